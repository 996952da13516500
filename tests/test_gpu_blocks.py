"""The Muon step on the blocks of stacked, fused and strided weights: bit for
bit muon_step on dense copies of the blocks (small blocks, whose chain runs in
one launch, against the oracle instead), and nothing outside them moves."""
import math

import pytest
import torch

import newton_schulz_matrix_b200 as nsm
import oracle
import parity_util
import synth

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def cut(t, block):
    """Dense copies of a tensor's blocks in the order of its status words."""
    r, c = block
    out = []
    for m in t.reshape(-1, *t.shape[-2:]):
        out += [m[i:i + r, j:j + c].clone() for i in range(0, m.shape[0], r) for j in range(0, m.shape[1], c)]
    return out


CASES = {
    # shape, block, view of the storage, W type, G type, hyper-parameters
    "heads": ((512, 384), (64, 384), None, "bf16", "bf16", {}),
    "head-columns": ((384, 512), (384, 64), None, "bf16", "bf16", {}),
    "fused-gate-up": ((3, 1024, 512), (512, 512), None, "bf16", "bf16", {}),
    "fused-tall": ((2, 600, 512), (600, 256), None, "bf16", "fp32", {}),
    "stack-of-stacks": ((2, 2, 256, 320), (256, 160), None, "fp16", "fp16", {"compute_dtype": "bf16"}),
    "strided-rows": ((2, 300, 520), (300, 260), "wide", "bf16", "bf16", {}),
    "unaligned": ((2, 514, 777), (257, 259), "odd", "bf16", "bf16", {}),
    "unaligned-fp32": ((300, 603), (300, 201), "odd", "fp32", "bf16", {"compute_dtype": "fp32"}),
    "fp32-tensor": ((2, 512, 640), (256, 320), "wide", "fp32", "fp32", {"compute_dtype": "fp32"}),
    "fp32-small": ((3, 64, 130), (32, 65), "odd", "fp32", "fp32", {"compute_dtype": "fp32"}),
    "gram": ((2, 512, 1536), (256, 768), "wide", "bf16", "bf16", {"mode": "gram_stabilized"}),
    "no-nesterov": ((320, 640), (320, 320), None, "fp32", "fp16", {"nesterov": False, "weight_decay": 0.0}),
    "rows-of-one": ((6, 48), (1, 48), None, "bf16", "bf16", {}),
    "column-of-one": ((40, 3), (40, 1), None, "bf16", "bf16", {}),
}


def make(shape, view, dtype, seed, std):
    """A tensor of `shape` inside a larger storage of sevens, and that storage."""
    pad = {None: 0, "wide": 24, "odd": 3}[view]
    store = torch.full(shape[:-2] + (shape[-2] + (2 if pad else 0), shape[-1] + pad), 7.0, dtype=dtype, device="cuda")
    first = 1 if view == "odd" else 0
    t = store[..., :shape[-2], first:first + shape[-1]]
    n = math.prod(shape)
    t.copy_(synth.gaussian(1, n, seed, "cuda", std=std).view(shape).to(dtype))
    return t, store


# 16-bit standard chains with n <= 128: one launch, another order of the sums
ONE_LAUNCH = ("heads", "head-columns", "rows-of-one", "column-of-one")


def check_weights(got, w, u, block, chain="fp16", coeffs=None, lr=0.02, wd=0.1):
    """W against the oracle: decay plus the step, whose O is within the 16-bit bar
    (2e-2, or 1.25 times what storing in the chain's type costs by itself), and
    half a step of W's type."""
    coeffs = coeffs or [oracle.QUINTIC] * 5
    x = u / (u.norm() + 1e-7)
    o = torch.from_numpy(oracle.ns_standard((x if block[0] <= block[1] else x.T).numpy(), coeffs))
    o = o if block[0] <= block[1] else o.T
    scale = lr * 0.2 * math.sqrt(max(block))
    ref = (1 - lr * wd) * w - scale * o
    tol = parity_util.tolerance(chain, parity_util.emulated_floor(u.numpy(), coeffs, "standard", chain=chain))
    err = float((got.double().cpu() - ref).norm())
    bound = tol * scale * float(o.norm()) + torch.finfo(got.dtype).eps / 2 * float(ref.norm()) + 1e-12
    assert err <= bound, (err, bound, tuple(block))


@pytest.mark.parametrize("name", sorted(CASES))
def test_blocks_step_as_dense_copies_do(name):
    shape, block, view, wdt, gdt, hp = CASES[name]
    (w, ws), (g, gs), (m, ms) = (make(shape, view, TYPES[wdt], 1, 0.05), make(shape, view, TYPES[gdt], 2, 1.0),
                                 make(shape, view, torch.float32, 3, 0.2))
    wd, gd, md = (cut(t, block) for t in (w, g, m))
    before = [t.clone() for t in (ws, gs, ms)]
    old = [[t.double().cpu() for t in ts] for ts in (wd, gd, md)]
    nsm.muon_step(wd, gd, md, **hp)
    status = torch.full((len(wd),), -1, dtype=torch.int32, device="cuda")
    nsm.muon_step_blocks([w], [g], [m], [block], status=status, **hp)
    assert status.tolist() == [0] * len(wd)
    for got, want in zip(cut(m, block), md):
        assert torch.equal(got, want)
    if name in ONE_LAUNCH:
        for got, w0, g0, m1 in zip(cut(w, block), old[0], old[1], md):
            check_weights(got, w0, 0.05 * g0 + 0.95 * m1.double().cpu(), block)
    else:
        for got, want in zip(cut(w, block), wd):
            assert torch.equal(got, want)
    # the storage around the blocks, and G, are as they were
    for t, view_, was in ((ws, w, before[0]), (ms, m, before[2])):
        view_.copy_(torch.zeros_like(view_))
        outside = t.clone()
        t.copy_(was)
        view_.copy_(torch.zeros_like(view_))
        assert torch.equal(outside, t)
    assert torch.equal(gs, before[1])


def test_parameters_of_several_kinds_in_one_call():
    """Heads, their transposes and whole matrices orient to common shapes and share batches; each gets its own result and status."""
    specs = [((4, 256, 640), (256, 320)), ((640, 512), (320, 256)), ((2, 320, 256), None), ((256, 320), None)]
    ws, gs, ms = [], [], []
    for i, (shape, _) in enumerate(specs):
        ws.append(make(shape, None, torch.bfloat16, 10 + i, 0.05)[0])
        gs.append(make(shape, None, torch.bfloat16, 20 + i, 1.0)[0])
        ms.append(make(shape, None, torch.float32, 30 + i, 0.2)[0])
    gs[1][400, 300] = float("nan")  # its block: rows 320.., columns 256..: the last of four
    blocks = [b for _, b in specs]
    dense = [[c for t, (s, b) in zip(ts, specs) for c in cut(t, b or s[-2:])] for ts in (ws, gs, ms)]
    want = torch.full((len(dense[0]),), -1, dtype=torch.int32, device="cuda")
    nsm.muon_step(*dense, status=want)
    status = torch.full_like(want, -1)
    nsm.muon_step_blocks(ws, gs, ms, blocks, status=status)
    assert torch.equal(status, want) and status.tolist() == [0] * 11 + [1] + [0] * 3
    got = [c for ts in (ws, ms) for t, (s, b) in zip(ts, specs) for c in cut(t, b or s[-2:])]
    for a, b in zip(got, dense[0] + dense[2]):
        assert torch.equal(a.view(torch.int16 if a.element_size() == 2 else torch.int32),
                           b.view(torch.int16 if b.element_size() == 2 else torch.int32))


def test_blocks_against_the_oracle():
    q5 = [oracle.QUINTIC] * 5
    w, g, m = (make((2, 256, 384), None, torch.float32, 40 + i, s)[0] for i, s in enumerate((0.05, 1.0, 0.2)))
    old = [t.double().cpu().numpy() for t in (w, g, m)]
    nsm.muon_step_blocks([w], [g], [m], [(128, 384)], compute_dtype="fp32")
    for e in range(2):
        for i in (0, 128):
            ref, mref, o = oracle.muon_step(*[t[e, i:i + 128] for t in old], lr=0.02, momentum=0.95, nesterov=True,
                                            weight_decay=0.1, scale_coef=0.2, eps=1e-7, coeffs=q5)
            step = torch.from_numpy(o).norm() * 0.02 * 0.2 * math.sqrt(384)
            # 1e-4 of the step (the fp32 bar) and half an fp32 step of the weights, three roundings
            assert (w[e, i:i + 128].double().cpu() - torch.from_numpy(ref)).norm() <= 1e-4 * step + 3 * 2.0 ** -24 * torch.from_numpy(ref).norm()
            assert (m[e, i:i + 128].double().cpu() - torch.from_numpy(mref)).norm() <= 3 * 2.0 ** -24 * torch.from_numpy(mref).norm()


def test_a_prepared_block_step_captures_and_uses_small_workspaces():
    shape, block = (4, 512, 512), (256, 512)
    w, g, m = (make(shape, None, dt, 50 + i, s)[0] for i, (dt, s) in enumerate(
        ((torch.bfloat16, 0.05), (torch.bfloat16, 1.0), (torch.float32, 0.2))))
    start = [w.clone(), m.clone()]
    nsm.muon_step_blocks([w], [g], [m], [block])
    nsm.muon_step_blocks([w], [g], [m], [block])
    want = [w.clone(), m.clone()]
    lo, hi = (f([w], [g], [m], [block]) for f in (nsm.muon_blocks_workspace_min, nsm.muon_blocks_workspace_size))
    assert lo < hi
    w.copy_(start[0]), m.copy_(start[1])
    step = nsm.MuonStep([w], [g], [m], blocks=[block], workspace_bytes=3 * lo)
    graph = step.capture()  # one eager step
    graph.replay()
    assert step.status.tolist() == [0] * 8
    for a, b in zip((w, m), want):
        assert torch.equal(a, b)
    w.copy_(start[0]), m.copy_(start[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(2):
        nsm.muon_step_blocks([w], [g], [m], [block], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip((w, m), want):
        assert torch.equal(a, b)


SMALL = [  # block, matrices, coefficients, chain, W type: one, two, four and eight CTAs a block, ragged slices
    ((128, 2048), 3, None, "fp16", "bf16"), ((2048, 128), 2, None, "fp16", "bf16"), ((64, 512), 2, None, "fp16", "fp32"),
    ((128, 513), 2, None, "fp16", "fp16"), ((100, 1100), 2, None, "fp16", "bf16"), ((17, 4096), 1, None, "fp16", "bf16"),
    ((3000, 33), 2, None, "fp16", "bf16"), ((128, 128), 5, None, "fp16", "bf16"), ((1, 640), 2, None, "fp16", "fp32"),
    ((5, 5), 3, None, "fp16", "bf16"), ((96, 1025), 2, None, "bf16", "bf16"), ((1537, 128), 1, None, "bf16", "fp32"),
    ((128, 700), 2, [oracle.CUBIC] * 7, "fp16", "bf16"), ((48, 2049), 1, [oracle.QUINTIC], "fp16", "fp32"),
    ((128, 1536), 2, [oracle.QUINTIC, oracle.CUBIC] * 3, "fp16", "bf16")]


@pytest.mark.parametrize("block,count,coeffs,chain,wdt", SMALL)
def test_small_blocks_in_one_launch(block, count, coeffs, chain, wdt):
    (w, _), (g, _), (m, _) = (make((count, *block), "odd" if block[1] % 2 else None, dt, 60 + i, s) for i, (dt, s) in enumerate(
        ((TYPES[wdt], 0.05), (torch.bfloat16, 1.0), (torch.float32, 0.2))))
    old = [t.double().cpu() for t in (w, g)]
    hp = {} if coeffs is None else {"coeffs": coeffs}
    nsm.muon_profile_begin()
    status = torch.full((count,), -1, dtype=torch.int32, device="cuda")
    nsm.muon_step_blocks([w], [g], [m], [None], status=status, compute_dtype=chain, **hp)
    assert "ns_block_kernel" in [r["kernel"] for r in nsm.muon_profile_end()]
    assert status.tolist() == [0] * count
    for e in range(count):
        check_weights(w[e], old[0][e], 0.05 * old[1][e] + 0.95 * m[e].double().cpu(), block, chain, coeffs)


def test_small_blocks_repeat_and_flag_what_is_not_finite():
    """Bit for bit the same twice and in a graph; a NaN or a zero gradient stays with its block."""
    shape, block = (512, 1024), (64, 1024)
    outs = []
    for mode in range(3):
        w, g, m = (make(shape, None, dt, 70 + i, s)[0] for i, (dt, s) in enumerate(
            ((torch.bfloat16, 0.05), (torch.bfloat16, 1.0), (torch.float32, 0.2))))
        g[70, 5] = float("nan")
        g[128:192], m[128:192] = 0, 0
        w0 = w.clone()
        step = nsm.MuonStep([w], [g], [m], blocks=[block])
        if mode == 2:
            graph = step.capture()
            w.copy_(w0), m.copy_(make(shape, None, torch.float32, 72, 0.2)[0])
            m[128:192] = 0
            graph.replay()
        else:
            step()
        assert step.status.tolist() == [0, 1, 0, 0, 0, 0, 0, 0]
        assert not w[64:128].isfinite().any() and w[128:].isfinite().all() and w[:64].isfinite().all()
        assert torch.equal(w[128:192], (0.998 * w0[128:192].float()).bfloat16())
        outs.append([t.view(torch.int16 if t.element_size() == 2 else torch.int32) for t in (w, m)])
    for o in outs[1:]:
        assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1])


def test_more_small_blocks_than_one_launch_takes():
    w, g, m = (make((600, 8, 256), None, dt, 80 + i, s)[0] for i, (dt, s) in enumerate(
        ((torch.bfloat16, 0.05), (torch.bfloat16, 1.0), (torch.float32, 0.2))))
    w2, m2 = w.clone(), m.clone()
    lo = nsm.muon_blocks_workspace_min([w], [g], [m], [None])
    nsm.muon_step_blocks([w], [g], [m], [None])
    nsm.muon_step_blocks([w2], [g], [m2], [None], workspace=torch.empty(20 * lo, dtype=torch.uint8, device="cuda"))
    assert torch.equal(w, w2) and torch.equal(m, m2)


@pytest.mark.parametrize("chain", ["fp16", "bf16"])
@pytest.mark.parametrize("block", [(64, 640), (640, 64), (33, 517), (517, 33), (128, 2049), (31, 95), (1, 1)])
def test_small_blocks_momentum_of_every_type_and_pitch(block, chain):
    """One launch reads G and M itself: G's types, pitches and alignments, both orientations and no Nesterov
    step give muon_step's momentum bit for bit and the oracle's weights; nothing else in the storages moves."""
    for i, (gdt, view, nesterov) in enumerate((("bf16", None, True), ("fp16", "wide", False), ("fp32", "odd", True),
                                               ("fp32", None, False), ("fp16", "odd", True))):
        shape = (2, block[0], 2 * block[1])
        (w, _), (g, _), (m, ms) = (make(shape, view, dt, 90 + 3 * i + k, s) for k, (dt, s) in enumerate(
            ((torch.float32, 0.05), (TYPES[gdt], 1.0), (torch.float32, 0.2))))
        wd, gd, md = (cut(t, block) for t in (w, g, m))
        old = [[t.double().cpu() for t in ts] for ts in (wd, gd)]
        hp = dict(nesterov=nesterov, compute_dtype=chain)
        nsm.muon_step(wd, gd, md, **hp)
        status = torch.full((4,), -1, dtype=torch.int32, device="cuda")
        nsm.muon_step_blocks([w], [g], [m], [block], status=status, **hp)
        assert status.tolist() == [0] * 4
        for got, want in zip(cut(m, block), md):
            assert torch.equal(got, want)
        for got, w0, g0, m1 in zip(cut(w, block), *old, md):
            m1 = m1.double().cpu()
            check_weights(got, w0, 0.05 * g0 + 0.95 * m1 if nesterov else m1, block, chain)
        m.fill_(7.0)
        assert bool((ms == 7).all())


def test_small_blocks_of_several_kinds_in_one_launch():
    """Blocks of one orientation share a launch, each with its own gradient type, pitch and orientation."""
    specs = [((2, 64, 320), "bf16", None), ((320, 64), "fp16", "wide"), ((64, 320), "fp32", "odd"), ((320, 64), "bf16", "odd")]
    ws, gs, ms = ([make(s, v, (torch.bfloat16, TYPES[d], torch.float32)[k], 120 + 3 * i + k, (0.05, 1.0, 0.2)[k])[0]
                   for i, (s, d, v) in enumerate(specs)] for k in range(3))
    one = [[t.clone() for t in ts] for ts in (ws, gs, ms)]
    nsm.muon_step_blocks(ws, gs, ms, [None] * 4)
    for i in range(4):
        nsm.muon_step_blocks([one[0][i]], [one[1][i]], [one[2][i]], [None])
        assert torch.equal(ws[i], one[0][i]) and torch.equal(ms[i], one[2][i])


@pytest.mark.parametrize("block,hp", [
    ((128, 4097), {}), ((64, 7168), {}), ((7168, 64), {}), ((128, 7168), {}), ((4100, 33), {"compute_dtype": "bf16"}),
    ((64, 384), {"coeffs": [oracle.CUBIC] * 65}), ((64, 384), {"mode": "gram"}), ((384, 64), {"mode": "gram_stabilized"}),
    ((128, 2048), {"mode": "gram_stabilized"}), ((33, 517), {"mode": "gram_stabilized", "restart_every": 1}),
    ((1, 48), {"mode": "gram"}), ((128, 7168), {"mode": "gram_stabilized"}),
    ((64, 384), {"mode": "gram", "gram_dtype": "bf16"}), ((100, 96), {"mode": "gram_stabilized", "compute_dtype": "fp32"})])
def test_small_blocks_that_one_launch_does_not_take(block, hp):
    """More than 4096 columns, more than 64 iterations, the Gram forms: muon_step's products, bit for bit."""
    odd = block[1] % 8 != 0
    (w, ws), (g, _), (m, ms) = (make((2, block[0], 2 * block[1]), "odd" if odd else None, dt, 150 + i, s) for i, (dt, s) in
                                enumerate(((torch.bfloat16, 0.05), (torch.bfloat16, 1.0), (torch.float32, 0.2))))
    wd, gd, md = (cut(t, block) for t in (w, g, m))
    nsm.muon_step(wd, gd, md, **hp)
    nsm.muon_profile_begin()
    status = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    nsm.muon_step_blocks([w], [g], [m], [block], status=status, **hp)
    assert "ns_block_kernel" not in [r["kernel"] for r in nsm.muon_profile_end()]
    assert status.tolist() == [0] * 4
    for got, want in zip(cut(w, block) + cut(m, block), wd + md):
        assert torch.equal(got, want)


def test_a_block_step_with_status_words_can_be_captured():
    """Kinds of blocks that take turns, so that the words come back in another order than the groups'."""
    shapes = [((4, 64, 96), (32, 96)), ((128, 80), (64, 40)), ((2, 64, 96), (32, 96)), ((64, 40), None), ((3, 64, 96), (32, 96))]
    (ws, gs, ms) = ([make(s, None, dt, 180 + 3 * i + k, std)[0] for i, (s, _) in enumerate(shapes)]
                    for k, (dt, std) in enumerate(((torch.bfloat16, 0.05), (torch.bfloat16, 1.0), (torch.float32, 0.2))))
    blocks = [b for _, b in shapes]
    gs[1][64:, 40:] = float("nan")  # the last of the second parameter's four blocks
    gs[4][1, :32, :32] = float("nan")  # the third of the last one's six
    want = [0] * 8 + [0, 0, 0, 1] + [0] * 4 + [0] + [0, 0, 1, 0, 0, 0]
    status = torch.full((len(want),), -1, dtype=torch.int32, device="cuda")
    assert nsm.muon_step_blocks(ws, gs, ms, blocks, status=status) is status
    assert status.tolist() == want
    shaped = torch.full((1, len(want)), -1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nsm.muon_step_blocks(ws, gs, ms, blocks, status=shaped)
    graph.replay()
    assert shaped[0].tolist()[8:12] == want[8:12] and shaped[0].tolist()[17:] == want[17:]


def test_a_workspace_of_another_type_counts_its_bytes():
    w, g, m = (make((2, 256, 320), None, dt, 200 + i, s)[0] for i, (dt, s) in enumerate(
        ((torch.bfloat16, 0.05), (torch.bfloat16, 1.0), (torch.float32, 0.2))))
    lo = nsm.muon_blocks_workspace_min([w], [g], [m], [None])
    step = nsm.MuonStep([w], [g], [m], blocks=[None], workspace=torch.empty(-(-lo // 4), dtype=torch.float32, device="cuda"))
    step()
    assert step.status.tolist() == [0, 0]


def test_one_launch_does_not_shrink_with_the_workspace():
    """The least workspace takes as many blocks a launch as the largest one, and writes nothing behind its end."""
    (w, _), (g, _), (m, _) = (make((600, 8, 256), None, dt, 210 + i, s) for i, (dt, s) in enumerate(
        ((torch.bfloat16, 0.05), (torch.bfloat16, 1.0), (torch.float32, 0.2))))
    w2, m2 = w.clone(), m.clone()
    lo = nsm.muon_blocks_workspace_min([w], [g], [m], [None])
    store = torch.full((lo + 4096,), 7, dtype=torch.uint8, device="cuda")
    launches = []
    for (a, b), ws in (((w, m), None), ((w2, m2), store[:lo])):
        nsm.muon_profile_begin()
        nsm.muon_step_blocks([a], [g], [b], [None], workspace=ws)
        launches.append({r["kernel"]: r["launches"] for r in nsm.muon_profile_end()}["ns_block_kernel"])
    assert launches == [2, 2]
    assert torch.equal(w, w2) and torch.equal(m, m2) and bool((store[lo:] == 7).all())


@pytest.mark.parametrize("block", [(192, 256), (256, 192), (200, 328), (300, 140), (257, 259), (516, 388)])
@pytest.mark.parametrize("gdt", ["bf16", "fp32"])
def test_alignment_does_not_show_in_the_bits(block, gdt):
    """A block is its dense copy bit for bit where the two are accessed differently: rows of whole 8s at odd
    pitches and addresses, other rows at pitches of whole 8s."""
    for i, (pad, first) in enumerate(((0, 0), (1, 1), (8, 0), (3, 2), (4, 4))):
        pitch = 2 * block[1] + pad
        for hp in ({}, {"compute_dtype": "fp32"}, {"compute_dtype": "bf16", "mode": "gram_stabilized"}, {"nesterov": False}):
            stores = [torch.full((2, block[0], -(-pitch // 8) * 8 + 8 if pad == 8 else pitch + first), 7.0, dtype=dt, device="cuda")
                      for dt in (torch.float32, TYPES[gdt], torch.float32)]
            w, g, m = (s[:, :, first:first + 2 * block[1]] for s in stores)
            for k, (t, std) in enumerate(((w, 0.05), (g, 1.0), (m, 0.2))):
                t.copy_(synth.gaussian(1, t.numel(), 230 + 3 * i + k, "cuda", std=std).view(t.shape))
            wd, gd, md = (cut(t, block) for t in (w, g, m))
            nsm.muon_step(wd, gd, md, **hp)
            nsm.muon_step_blocks([w], [g], [m], [block], **hp)
            for got, want in zip(cut(w, block) + cut(m, block), wd + md):
                assert torch.equal(got, want), (pad, first, hp)


@pytest.mark.parametrize("shape", [(384, 388), (100, 100), (516, 516), (300, 700), (256, 512), (257, 259)])
@pytest.mark.parametrize("hp", [{}, {"compute_dtype": "fp32"}, {"mode": "gram_stabilized"}], ids=["fp16", "fp32", "gram"])
def test_a_gradient_steps_alike_in_every_type_that_holds_it(shape, hp):
    """muon_step on the same values of G in bf16 and fp32, whose rows are aligned differently."""
    results = []
    for dt in (torch.bfloat16, torch.float32):
        w, m = (synth.gaussian(*shape, 250 + k, "cuda", std=std) for k, std in enumerate((0.05, 0.2)))
        g = synth.gaussian(*shape, 252, "cuda").bfloat16().to(dt)
        nsm.muon_step([w], [g], [m], **hp)
        results.append((w, m))
    for a, b in zip(*results):
        assert torch.equal(a, b)
