"""The expert-layer operators against plain 64-bit versions: routing (sort,
gather, combine and gradients), the experts' products and their gradients, and
a whole layer's training step into the Muon step."""
import os
import subprocess
import sys

import pytest
import torch

import newton_schulz_matrix_b200 as nsm
import oracle
from expert_util import U_NEAREST, U_TRUNCATED, close, f64, rows_ref, segments, sort_ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, HF, SF = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=SF):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def routing(seed, tokens, topk, experts, dropped=0.0, dtype=torch.int64):
    g = gen(seed)
    ids = torch.rand(tokens, experts, generator=g, device="cuda").topk(topk, dim=1).indices
    keep = torch.rand(tokens, topk, generator=g, device="cuda") >= dropped
    return torch.where(keep, ids, -1).to(dtype)


def pitched(t, pad):
    """The same matrix with `pad` elements between its rows, and that storage."""
    store = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    view = store[:, :t.shape[1]]
    view.copy_(t)
    return view


# ---------------------------------------------------------------- sort
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,topk,experts", [
    (1, 1, 1), (1, 8, 8), (3, 2, 1024), (32, 8, 216), (33, 3, 7), (1000, 8, 64), (1024, 8, 1023), (1025, 8, 64),
    (4097, 2, 1024), (20011, 3, 13), (70000, 8, 256)])
def test_sort_is_the_stable_order(tokens, topk, experts, dtype):
    ids = routing(1, tokens, min(topk, experts), experts, 0.1, dtype)
    got = nsm.muon_expert_sort(ids, experts)
    for g, r in zip(got, sort_ref(ids, experts)):
        assert g.dtype == torch.int32 and torch.equal(g.cpu(), r)


def test_sort_of_extreme_ids():
    """Ids outside the range (negative, beyond int32, the first one past the end) go to no expert; one expert may take all."""
    ids = torch.tensor([[0, 4], [5, -1], [2 ** 40, -2 ** 40], [2 ** 32, 2 ** 32 + 3], [4, 4]], device="cuda")
    for g, r in zip(nsm.muon_expert_sort(ids, 5), sort_ref(ids, 5)):
        assert torch.equal(g.cpu(), r)
    for tokens in (7, 30000):
        one = torch.full((tokens, 2), 3, device="cuda")
        none = torch.full((tokens, 2), -1, device="cuda", dtype=torch.int32)
        for ids in (one, none):
            for g, r in zip(nsm.muon_expert_sort(ids, 9), sort_ref(ids, 9)):
                assert torch.equal(g.cpu(), r)


def test_sort_of_no_token_and_of_pitched_ids():
    offsets, slot, source = nsm.muon_expert_sort(torch.empty(0, 4, dtype=torch.int64, device="cuda"), 6)
    assert offsets.tolist() == [0] * 7 and slot.shape == (0, 4) and source.numel() == 0
    wide = routing(2, 9000, 8, 32)
    for ids in (wide[:, 2:5], wide[::3, :4]):
        for g, r in zip(nsm.muon_expert_sort(ids, 32), sort_ref(ids, 32)):
            assert torch.equal(g.cpu(), r)


# ---------------------------------------------------------------- gather and combine
ROUTES = [  # tokens, topk, experts, cols, dropped, pad
    (1, 1, 1, 1, 0.0, 0), (1, 8, 16, 7168, 0.0, 0), (5, 3, 4, 17, 0.3, 0), (64, 8, 216, 2048, 0.0, 0),
    (257, 2, 8, 1001, 0.5, 0), (130, 6, 64, 96, 0.2, 8), (33, 11, 12, 130, 0.4, 2), (40, 4, 8, 264, 0.1, 3),
    (9, 2, 3, 8, 1.0, 0)]


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("tokens,topk,experts,cols,dropped,pad", ROUTES)
def test_gather_and_its_gradient(tokens, topk, experts, cols, dropped, pad, dtype):
    g = gen(3)
    offsets, slot, source = nsm.muon_expert_sort(routing(4, tokens, topk, experts, dropped), experts)
    x, dxs = pitched(randn(g, tokens, cols, dtype=dtype), pad), pitched(randn(g, tokens * topk, cols, dtype=dtype), pad)
    used = int(offsets[-1])
    dxs[used:] = float("nan")  # rows that no assignment names
    out = pitched(torch.full((tokens * topk, cols), 7.0, dtype=dtype, device="cuda"), pad)
    assert nsm.muon_expert_gather(x, slot, out=out) is out
    token = source[:used].long() // topk
    assert torch.equal(out[:used], x[token]) and bool((out[used:] == 7).all())
    dx = nsm.muon_expert_gather_backward(dxs, slot)
    rows, _ = rows_ref(torch.where(torch.arange(tokens * topk, device="cuda")[:, None] < used, dxs, 0), slot)
    close(dx, rows.sum(1), topk, rows.abs().sum(1), U_NEAREST)


@pytest.mark.parametrize("wdtype", [SF, BF])
@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("tokens,topk,experts,cols,dropped,pad", ROUTES)
def test_combine_and_its_gradients(tokens, topk, experts, cols, dropped, pad, dtype, wdtype):
    g = gen(5)
    offsets, slot, _ = nsm.muon_expert_sort(routing(6, tokens, topk, experts, dropped), experts)
    used = int(offsets[-1])
    ys, dy = pitched(randn(g, tokens * topk, cols, dtype=dtype), pad), pitched(randn(g, tokens, cols, dtype=dtype), pad)
    ys[used:] = float("inf")
    w = randn(g, tokens, topk, dtype=wdtype)
    w = torch.where(slot >= 0, w, float("nan"))  # the weight of a dropped assignment does not matter
    y = nsm.muon_expert_combine(ys, slot, w)
    rows, on = rows_ref(ys[:used], slot)
    w64 = torch.where(on, f64(w), 0.0)
    close(y, (w64[..., None] * rows).sum(1), topk, (w64[..., None] * rows).abs().sum(1), U_NEAREST)
    out = pitched(torch.full((tokens * topk, cols), 7.0, dtype=dtype, device="cuda"), pad)
    dys, dw = nsm.muon_expert_combine_backward(dy, ys, slot, w, out=out)
    assert dys is out and bool((dys[used:] == 7).all()) and dw.dtype == wdtype
    dy64 = f64(dy)[:, None, :]
    want = (w64[..., None] * dy64)
    picked, _ = rows_ref(dys, slot)
    close(dys[:used], want[on].new_zeros(used, cols).index_copy_(0, slot.cpu()[on].long(), want[on]), 1,
          want[on].new_zeros(used, cols).index_copy_(0, slot.cpu()[on].long(), want[on].abs()), U_NEAREST)
    close(dw, (rows * dy64).sum(2), cols, (rows * dy64).abs().sum(2), U_NEAREST)


def test_combine_without_weights_and_inf_in_a_taken_row():
    slot = torch.tensor([[0, -1], [1, 2]], dtype=torch.int32, device="cuda")
    ys = torch.tensor([[1.0, float("inf")], [2.0, 3.0], [4.0, float("nan")]], device="cuda")
    y = nsm.muon_expert_combine(ys, slot)
    assert y[0].tolist() == [1.0, float("inf")] and y[1, 0] == 6.0 and bool(y[1, 1].isnan())
    dys, dw = nsm.muon_expert_combine_backward(torch.ones(2, 2, device="cuda"), ys, slot)
    assert dw is None and dys.tolist() == [[1.0, 1.0]] * 3


def test_slots_outside_the_rows_are_skipped():
    """A slot beyond the sorted matrix (an output cut to a capacity) touches nothing."""
    g = gen(7)
    x = randn(g, 6, 40, dtype=BF)
    slot = torch.tensor([[0], [3], [4], [5], [2 ** 31 - 1], [-2 ** 31]], dtype=torch.int32, device="cuda")
    store = torch.full((6, 40), 7.0, dtype=BF, device="cuda")
    nsm.muon_expert_gather(x, slot, out=store[:4])
    assert torch.equal(store[0], x[0]) and torch.equal(store[3], x[1])
    assert bool((store[1:3] == 7).all()) and bool((store[4:] == 7).all())
    y = nsm.muon_expert_combine(store[:4], slot)
    assert torch.equal(y[:2], x[:2]) and not y[2:].any()
    dys, dw = nsm.muon_expert_combine_backward(x, store[:4], slot, torch.ones(6, 1, device="cuda"))
    assert dys.shape == (4, 40) and not dw[2:].any()


# ---------------------------------------------------------------- products
def offsets_of(counts, first=0):
    return torch.tensor([first] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


PRODUCTS = [  # counts, inner, outer
    ([1], 64, 64), ([0, 0, 3], 16, 8), ([5, 0, 17, 1], 72, 40), ([130, 64, 0, 255], 256, 264), ([256, 257, 511], 128, 512),
    ([33] * 20, 320, 136), ([700, 2, 0, 90], 1000, 520), ([15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65], 192, 256),
    ([1024], 512, 768)]


def product_case(seed, counts, inner, outer, dtype, tail=3, pad=0):
    g = gen(seed)
    rows = sum(counts) + tail
    xs, dys = pitched(randn(g, rows, inner, dtype=dtype), pad), pitched(randn(g, rows, outer, dtype=dtype), pad)
    # what lies behind the last expert's rows reaches no result
    xs[sum(counts):] = float("nan")
    dys[sum(counts):] = float("inf")
    return offsets_of(counts), xs, dys, randn(g, len(counts), outer, inner, dtype=dtype)


def check_products(offsets, xs, dys, w, u, dw_dtype=None):
    rows, inner, outer, dtype = xs.shape[0], xs.shape[1], dys.shape[1], xs.dtype
    y = torch.full((rows, outer), 7.0, dtype=dtype, device="cuda")
    dx = torch.full((rows, inner), 7.0, dtype=dtype, device="cuda")
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    nsm.muon_expert_product(xs, w, offsets, out=y, status=status)
    assert int(status) == 0
    nsm.muon_expert_input_grad(dys, w, offsets, out=dx, status=status)
    assert int(status) == 0
    dw = nsm.muon_expert_weight_grad(dys, xs, offsets, out_dtype=dw_dtype, status=status)
    assert int(status) == 0
    owned = torch.zeros(rows, dtype=torch.bool)
    for e, (lo, hi) in enumerate(segments(offsets, rows)):
        owned[lo:hi] = True
        x, d, m = f64(xs[lo:hi]), f64(dys[lo:hi]), f64(w[e])
        close(y[lo:hi], x @ m.T, inner, x.abs() @ m.abs().T, u, f"y of expert {e}")
        close(dx[lo:hi], d @ m, outer, d.abs() @ m.abs(), u, f"dx of expert {e}")
        close(dw[e], d.T @ x, hi - lo, d.abs().T @ x.abs(), u, f"dw of expert {e}")
    assert bool((y[~owned] == 7).all()) and bool((dx[~owned] == 7).all())


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("counts,inner,outer", PRODUCTS)
def test_products_and_gradients(counts, inner, outer, dtype):
    check_products(*product_case(11, counts, inner, outer, dtype), U_NEAREST if dtype == SF else U_TRUNCATED,
                   SF if counts[0] % 2 else None)


@pytest.mark.parametrize("dtype", [BF, SF])
@pytest.mark.parametrize("inner,outer,pad", [(33, 130, 0), (72, 41, 1), (64, 64, 3), (264, 1, 0), (1, 136, 8)])
def test_products_of_odd_widths_and_pitches(inner, outer, pad, dtype):
    check_products(*product_case(12, [7, 0, 66, 3], inner, outer, dtype, pad=pad),
                   U_NEAREST if dtype == SF else U_TRUNCATED)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("counts,inner,outer,pad", [([300, 0, 511, 37], 1021, 515, 0), ([700, 130], 770, 1023, 1),
                                                    ([90] * 12, 520, 1030, 4), ([40, 17, 2000], 336, 703, 0)])
def test_large_products_of_odd_widths(counts, inner, outer, pad, dtype):
    """Copied into aligned rows for the tensor cores; the results have rows of any alignment."""
    case = product_case(22, counts, inner, outer, dtype, pad=pad)
    nsm.muon_profile_begin()
    check_products(*case, U_TRUNCATED, SF if pad else None)
    prof = {r["kernel"]: r["launches"] for r in nsm.muon_profile_end()}
    assert prof == {"expert_product": 3}
    offsets, xs, dys, _ = case
    base = randn(gen(23), len(counts), outer, inner + 1)[:, :, 1:]
    out = base.clone()
    store = torch.full((len(counts), outer, inner + 3), 7.0, device="cuda")
    view = store[:, :, 1:inner + 1]
    view.copy_(base)
    nsm.muon_expert_weight_grad(dys, xs, offsets, out=view, accumulate=True)
    one = nsm.muon_expert_weight_grad(dys, xs, offsets, out_dtype=SF)
    for e, (lo, hi) in enumerate(segments(offsets, xs.shape[0])):
        d, x = f64(dys[lo:hi]), f64(xs[lo:hi])
        close(view[e], f64(out[e]) + d.T @ x, hi - lo + 1, f64(out[e]).abs() + d.abs().T @ x.abs(), U_TRUNCATED)
        close(one[e], d.T @ x, hi - lo, d.abs().T @ x.abs(), U_TRUNCATED)
    assert bool((store[:, :, 0] == 7).all()) and bool((store[:, :, inner + 1:] == 7).all())


@pytest.mark.parametrize("dtype", [BF, HF, SF])
def test_products_of_shared_weights(dtype):
    """One matrix for all experts (a stride of zero), small and large."""
    for counts, inner, outer in (([20, 0, 31], 64, 72), ([400, 0, 511], 768, 640)):
        offsets, xs, _, w = product_case(24, counts, inner, outer, dtype)
        shared = w[:1].expand(len(counts), outer, inner)
        y, ref = (nsm.muon_expert_product(xs, v, offsets) for v in (shared, shared.contiguous()))
        used = sum(counts)
        x, m = f64(xs[:used]), f64(w[0])
        close(y[:used], x @ m.T, inner, x.abs() @ m.abs().T, U_NEAREST if dtype == SF else U_TRUNCATED)
        close(ref[:used], x @ m.T, inner, x.abs() @ m.abs().T, U_NEAREST if dtype == SF else U_TRUNCATED)


@pytest.mark.parametrize("dtype", [BF, SF])
def test_products_of_strided_weights(dtype):
    """Weights that are part of a fused stack: every second half of the rows, a slice of the columns; dW written into one."""
    g = gen(13)
    counts = [40, 0, 300]
    offsets, xs, dys, _ = product_case(14, counts, 128, 96, dtype)
    fused = randn(g, 3, 2 * 96, 128 + 64, dtype=dtype)
    w = fused[:, 96:, 64:]
    check_products(offsets, xs, dys, w, U_NEAREST if dtype == SF else U_TRUNCATED)
    assert torch.equal(nsm.muon_expert_product(xs, w, offsets)[:340], nsm.muon_expert_product(xs, w.contiguous(), offsets)[:340])
    out = torch.full((3, 2 * 96, 128 + 64), 7.0, dtype=dtype, device="cuda")
    nsm.muon_expert_weight_grad(dys, xs, offsets, out=out[:, 96:, 64:])
    assert torch.equal(out[:, 96:, 64:], nsm.muon_expert_weight_grad(dys, xs, offsets))
    assert bool((out[:, :96] == 7).all()) and bool((out[:, :, :64] == 7).all())


@pytest.mark.parametrize("scale", [1, 9])
@pytest.mark.parametrize("dtype", [BF, HF, SF])
def test_nan_stays_with_its_expert(dtype, scale):
    """Inf and NaN in one expert's rows reach no other expert's results, whatever tile they share."""
    counts = [21 * scale, 9 * scale, 34 * scale, 100 * scale, 3 * scale]
    offsets, xs, dys, w = product_case(15, counts, 128, 64, dtype, tail=0)
    lo, hi = counts[0], counts[0] + counts[1]
    clean = [f(a, b, offsets) for f, a, b in ((nsm.muon_expert_product, xs, w), (nsm.muon_expert_input_grad, dys, w),
                                              (nsm.muon_expert_weight_grad, dys, xs))]
    xs[lo:hi], dys[lo:hi] = float("nan"), float("inf")
    dirty = [f(a, b, offsets) for f, a, b in ((nsm.muon_expert_product, xs, w), (nsm.muon_expert_input_grad, dys, w),
                                              (nsm.muon_expert_weight_grad, dys, xs))]
    rest = torch.cat([torch.arange(lo), torch.arange(hi, sum(counts))]).cuda()
    for a, b in zip(clean[:2], dirty[:2]):
        assert torch.equal(a[rest], b[rest])
    assert torch.equal(clean[2][[0, 2, 3, 4]], dirty[2][[0, 2, 3, 4]]) and not dirty[2][1].isfinite().any()


@pytest.mark.parametrize("dtype", [BF, SF])
@pytest.mark.parametrize("ends", [[5, 40, 40, 90], [-4, 20, 10, 2 ** 31 - 1], [50, 20, 60, 200], [0, 0, 0, 0], [100, 90, 80, 95]])
def test_offsets_are_clamped_to_the_rows(ends, dtype):
    """Offsets that start late, run backwards or past the end name the clamped rows and nothing else."""
    g = gen(16)
    xs, dys, w = randn(g, 80, 64, dtype=dtype), randn(g, 80, 72, dtype=dtype), randn(g, 3, 72, 64, dtype=dtype)
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    spans = segments(offsets, 80)
    y = torch.full((81, 72), 7.0, dtype=dtype, device="cuda")
    nsm.muon_expert_product(xs, w, offsets, out=y[:80])
    dw = nsm.muon_expert_weight_grad(dys, xs, offsets)
    u = U_NEAREST if dtype == SF else U_TRUNCATED
    owners = [[e for e, (lo, hi) in enumerate(spans) if lo <= p < hi] for p in range(81)]
    for p, own in enumerate(owners):
        if not own:
            assert bool((y[p] == 7).all())
        elif len(own) == 1:
            a, m = f64(xs[p]), f64(w[own[0]])
            close(y[p], m @ a, 64, m.abs() @ a.abs(), u)
    for e, (lo, hi) in enumerate(spans):
        d, x = f64(dys[lo:hi]), f64(xs[lo:hi])
        close(dw[e], d.T @ x, hi - lo, d.abs().T @ x.abs(), u)


@pytest.mark.parametrize("dtype", [BF, HF, SF])
def test_weight_gradients_accumulate(dtype):
    offsets, xs, dys, _ = product_case(17, [300, 0, 41], 136, 264, dtype)
    base = randn(gen(18), 3, 264, 136)
    out = base.clone()
    one = nsm.muon_expert_weight_grad(dys, xs, offsets, out_dtype=SF)
    assert nsm.muon_expert_weight_grad(dys, xs, offsets, out=out, accumulate=True) is out
    for e, (lo, hi) in enumerate(segments(offsets, xs.shape[0])):
        d, x = f64(dys[lo:hi]), f64(xs[lo:hi])
        u = U_NEAREST if dtype == SF else U_TRUNCATED
        close(out[e], f64(base[e]) + d.T @ x, hi - lo + 1, f64(base[e]).abs() + d.abs().T @ x.abs(), u)
    assert torch.equal(out[1], base[1]) and not one[1].any()


@pytest.mark.parametrize("rows,experts", [(1, 64), (8, 64), (200, 64), (3000, 300), (2000, 1024)])
def test_products_of_many_experts_with_few_rows(rows, experts):
    g = gen(19)
    to = torch.randint(0, experts, (rows,), generator=g, device="cuda").sort().values
    counts = torch.bincount(to, minlength=experts).tolist()
    check_products(*product_case(20, counts, 256, 128, BF, tail=0), U_TRUNCATED)


def test_products_repeat_bit_for_bit_and_on_another_stream():
    offsets, xs, dys, w = product_case(21, [70, 513, 1, 260], 512, 320, HF)
    used = int(offsets[-1])
    calls = [lambda **k: nsm.muon_expert_product(xs, w, offsets, **k)[:used],
             lambda **k: nsm.muon_expert_input_grad(dys, w, offsets, **k)[:used],
             lambda **k: nsm.muon_expert_weight_grad(dys, xs, offsets, out_dtype=SF, **k)]
    side = torch.cuda.Stream()
    for call in calls:
        first = call()
        assert torch.equal(first, call())
        side.wait_stream(torch.cuda.current_stream())
        other = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(first, other)


def test_products_of_no_row():
    offsets = torch.zeros(4, dtype=torch.int32, device="cuda")
    for dtype in (BF, SF):
        xs, dys, w = (torch.empty(s, dtype=dtype, device="cuda") for s in ((0, 64), (0, 72), (3, 72, 64)))
        assert nsm.muon_expert_product(xs, w, offsets).shape == (0, 72)
        assert nsm.muon_expert_input_grad(dys, w, offsets).shape == (0, 64)
        assert not nsm.muon_expert_weight_grad(dys, xs, offsets).any()
        out = torch.full((3, 72, 64), 7.0, device="cuda")
        assert bool((nsm.muon_expert_weight_grad(dys, xs, offsets, out=out, accumulate=True) == 7).all())
        y = nsm.muon_expert_combine(xs, torch.zeros(5, 2, dtype=torch.int32, device="cuda"))
        assert y.shape == (5, 64) and not y.any()


def test_rows_past_two_to_the_32_bytes_and_elements():
    """The last rows of a matrix of more than 2^32 elements, in every operator."""
    cols, rows = 4096, (1 << 20) + 4099
    big = torch.empty(rows, cols, dtype=BF, device="cuda")
    g = gen(41)
    counts = [70, 0, 131, 3]
    first = rows - sum(counts)
    offsets = offsets_of(counts, first)
    last = randn(g, sum(counts), cols, dtype=BF)
    big[first:] = last
    w = (randn(g, 4, 40, cols) / 64).to(BF)
    near = offsets_of(counts)
    y = nsm.muon_expert_product(big, w, offsets)
    assert torch.equal(y[first:], nsm.muon_expert_product(last, w, near))
    dys = torch.empty(rows, 40, dtype=BF, device="cuda")
    dys[first:] = randn(g, sum(counts), 40, dtype=BF)
    assert torch.equal(nsm.muon_expert_weight_grad(dys, big, offsets), nsm.muon_expert_weight_grad(dys[first:], last, near))
    slot = (first + torch.randperm(sum(counts), generator=g, device="cuda")).to(torch.int32).view(-1, 2)
    back = nsm.muon_expert_combine(big, slot)
    assert torch.equal(back, nsm.muon_expert_combine(last, slot - first))
    wts = torch.rand(*slot.shape, generator=g, device="cuda")
    ref_dys, ref_dw = nsm.muon_expert_combine_backward(back, last, slot - first, wts)
    got_dys, got_dw = nsm.muon_expert_combine_backward(back, big, slot, wts, out=big)
    assert torch.equal(got_dw, ref_dw) and torch.equal(got_dys[first:], ref_dys)
    nsm.muon_expert_gather(back, slot, out=big)
    assert torch.equal(big[slot.long()], back[:, None].expand(-1, 2, -1))
    wide = torch.empty(rows, cols, dtype=BF, device="cuda")
    nsm.muon_expert_input_grad(dys, w, offsets, out=wide)
    assert torch.equal(wide[first:], nsm.muon_expert_input_grad(dys[first:], w, near))


def test_the_first_calls_of_a_process_can_be_captured():
    """One-time set-up (shared-memory opt-ins, tensor maps) happens under a capture too."""
    code = """
import torch, sys
sys.path.insert(0, {root!r})
import newton_schulz_matrix_b200 as nsm
x, w = torch.randn(64, 64, device="cuda").bfloat16(), torch.randn(4, 64, 64, device="cuda").bfloat16()
ids, m = torch.randint(0, 4, (64, 2), device="cuda"), torch.zeros(4, 64, 64, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    offsets, slot, _ = nsm.muon_expert_sort(ids, 4)
    xs = nsm.muon_expert_gather(x, slot)
    h = nsm.muon_expert_product(xs, w, offsets)
    y = nsm.muon_expert_combine(h, slot)
    dw = nsm.muon_expert_weight_grad(h, xs, offsets)
    nsm.muon_step_blocks([w], [dw], [m], [(32, 64)])
w0 = w.clone()
g.replay()
torch.cuda.synchronize()
got = y.clone()
w.copy_(w0)
offsets, slot, _ = nsm.muon_expert_sort(ids, 4)
h = nsm.muon_expert_product(nsm.muon_expert_gather(x, slot), w, offsets)
assert torch.equal(got, nsm.muon_expert_combine(h, slot)) and got.any()
""".format(root=ROOT)
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300, cwd=ROOT)


# ---------------------------------------------------------------- together
def layer(x, ids, probs, w1, w2, blocks_dtype=BF):
    """Forward and backward of a two-product expert layer with relu-squared between, and all that it leaves."""
    experts = w1.shape[0]
    offsets, slot, _ = nsm.muon_expert_sort(ids, experts)
    xs = torch.zeros(ids.numel(), x.shape[1], dtype=x.dtype, device="cuda")
    nsm.muon_expert_gather(x, slot, out=xs)
    h = nsm.muon_expert_product(xs, w1, offsets, out=torch.zeros(ids.numel(), w1.shape[1], dtype=x.dtype, device="cuda"))
    a = torch.relu(h.float()).square().to(x.dtype)
    o = nsm.muon_expert_product(a, w2, offsets, out=torch.zeros(ids.numel(), w2.shape[1], dtype=x.dtype, device="cuda"))
    y = nsm.muon_expert_combine(o, slot, probs)

    def backward(dy):
        do, dprobs = nsm.muon_expert_combine_backward(dy, o, slot, probs, out=torch.zeros_like(o))
        dw2 = nsm.muon_expert_weight_grad(do, a, offsets)
        da = nsm.muon_expert_input_grad(do, w2, offsets, out=torch.zeros_like(a))
        dh = (da.float() * 2 * torch.relu(h.float())).to(x.dtype)
        dw1 = nsm.muon_expert_weight_grad(dh, xs, offsets)
        dxs = nsm.muon_expert_input_grad(dh, w1, offsets, out=torch.zeros_like(xs))
        return nsm.muon_expert_gather_backward(dxs, slot), dprobs, dw1, dw2, (dh, xs, offsets), (do, a, offsets)

    return y, backward


def layer_ref(x, ids, probs, w1, w2):
    """The same layer in 64 bits, one token and one assignment at a time."""
    y = []
    for t in range(x.shape[0]):
        row = torch.zeros(w2.shape[1], dtype=torch.float64)
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if 0 <= e < w1.shape[0]:
                row = row + probs[t, j] * (w2[e] @ torch.relu(w1[e] @ x[t]).square())
        y.append(row)
    return torch.stack(y)


@pytest.mark.parametrize("dtype", [SF, BF])
def test_a_layer_and_its_gradients(dtype):
    """Against the 64-bit layer, its autograd and its differences.  In fp32 the
    chain of four sums is within 1e-5 of the largest value (terms of at most
    136 products each, 136 * 2^-24 = 8e-6); in bf16 every stored matrix adds
    half a step of 2^-8 = 4e-3, eight stores on the longest path: 3.2e-2."""
    g = gen(30)
    tokens, topk, experts, width, hidden = 50, 3, 5, 64, 136
    ids = routing(31, tokens, topk, experts, 0.2)
    x, w1, w2 = (randn(g, tokens, width, dtype=dtype), (randn(g, experts, hidden, width) / 8).to(dtype),
                 (randn(g, experts, width, hidden) / 12).to(dtype))
    probs, dy = torch.rand(tokens, topk, generator=g, device="cuda"), randn(g, tokens, width, dtype=dtype)
    y, backward = layer(x, ids, probs, w1, w2)
    grads = backward(dy)[:4]
    leaves = [f64(t).requires_grad_() for t in (x, probs, w1, w2)]
    ref = layer_ref(leaves[0], ids.cpu(), *leaves[1:])
    want = torch.autograd.grad((ref * f64(dy)).sum(), leaves)
    tol = 1e-5 if dtype == SF else 3.2e-2
    for got, r in zip((y,) + grads, (ref.detach(),) + want):
        assert (f64(got) - r).norm() <= tol * r.norm(), float((f64(got) - r).norm() / r.norm())
    if dtype == SF:
        # the formula's gradient against central differences of the layer itself
        h = 2.0 ** -6
        for i, leaf in enumerate(leaves):
            step = torch.zeros_like(leaf)
            at = tuple(int(v) for v in torch.nonzero(want[i].abs() == want[i].abs().max())[0])
            step[at] = h
            up, down = ([(v + s * step).detach() if k == i else v.detach() for k, v in enumerate(leaves)] for s in (1, -1))
            slope = ((layer_ref(up[0], ids.cpu(), *up[1:]) - layer_ref(down[0], ids.cpu(), *down[1:])) * f64(dy)).sum() / (2 * h)
            # the layer is piecewise polynomial of degree 2 in each leaf: the central difference is exact off its kinks
            assert abs(float(grads[i].cpu()[at]) - float(slope)) <= 1e-2 * abs(float(slope))


def test_a_training_step_of_a_layer():
    """Route, multiply, differentiate and step: ExpertMuonStep in slices is the weight
    gradients followed by the block step, bit for bit, and the oracle's step on
    each expert's halves."""
    g = gen(32)
    tokens, topk, experts, width, hidden = 300, 2, 6, 128, 96
    ids = routing(33, tokens, topk, experts, 0.1)
    ids[ids == 4] = -1  # an expert without tokens: its momentum decays, its weights decay
    x = randn(g, tokens, width, dtype=BF)
    w1, w2 = (randn(g, experts, 2 * hidden, width) / 8).to(BF), (randn(g, experts, width, 2 * hidden) / 12).to(BF)
    moms = [randn(g, *w.shape) * 0.01 for w in (w1, w2)]
    moms[0][4], moms[1][4] = 0, 0
    probs = torch.rand(tokens, topk, generator=g, device="cuda")
    _, backward = layer(x, ids, probs, w1, w2)
    *_, dw1, dw2, f1, f2 = backward(randn(g, tokens, width, dtype=BF))
    blocks = [(hidden, width), None]
    pa, ma = [w1.clone(), w2.clone()], [m.clone() for m in moms]
    status = torch.full((3 * experts,), -1, dtype=torch.int32, device="cuda")
    nsm.muon_step_blocks(pa, [dw1, dw2], ma, blocks, status=status)
    assert status.tolist() == [0] * (3 * experts)
    for slice_bytes in (1, 2 * hidden * width * 2 * 4, 1 << 30):
        pb, mb = [w1.clone(), w2.clone()], [m.clone() for m in moms]
        step = nsm.ExpertMuonStep(pb, mb, blocks=blocks, slice_bytes=slice_bytes)
        step([f1, f2])
        assert step.status.tolist() == [0] * (3 * experts)
        for a, b in zip(pa + ma, pb + mb):
            assert torch.equal(a, b)
    q5 = [oracle.QUINTIC] * 5
    for w, dw, m, new, (r, c) in ((w1, dw1, moms[0], pa[0], blocks[0]), (w2, dw2, moms[1], pa[1], (width, 2 * hidden))):
        for e in range(experts):
            for i in range(0, w.shape[1], r):
                args = [f64(t[e, i:i + r]).numpy() for t in (w, dw, m)]
                ref, _, o = oracle.muon_step(*args, lr=0.02, momentum=0.95, nesterov=True, weight_decay=0.1,
                                             scale_coef=0.2, eps=1e-7, coeffs=q5)
                err = (f64(new[e, i:i + r]) - torch.from_numpy(ref)).norm()
                # 2e-2 of the step (the 16-bit chain's bar) and half a bf16 step of the weights
                step_norm = 0.02 * 0.2 * max(r, c) ** 0.5 * torch.from_numpy(o).norm()
                assert err <= 2e-2 * step_norm + 2.0 ** -8 * torch.from_numpy(ref).norm()


def test_expert_step_refuses_before_it_steps():
    g = gen(42)
    w, m = randn(g, 2, 64, 32, dtype=BF), torch.zeros(2, 64, 32, device="cuda")
    step = nsm.ExpertMuonStep([w, w.clone()], [m, m.clone()])
    good = (randn(g, 8, 64, dtype=BF), randn(g, 8, 32, dtype=BF), offsets_of([3, 5]))
    before = w.clone()
    for bad in ((good[0][:7], good[1], good[2]), (good[0].half(), good[1].half(), good[2]), (good[0], good[1], good[2].long()),
                (good[0], good[1], offsets_of([1, 2, 3])), (good[1], good[0], good[2]), (good[0].cpu(), good[1], good[2])):
        with pytest.raises(nsm.MuonError):
            step([good, bad])
    with pytest.raises(nsm.MuonError):
        step([good])
    assert torch.equal(w, before) and not m.any()
    step([good, good])
    assert not torch.equal(w, before)


def test_a_captured_layer_replays():
    """The whole run in one CUDA graph, replayed on other tokens and routes."""
    g = gen(34)
    tokens, topk, experts, width, hidden = 200, 2, 4, 64, 128
    x, ids = randn(g, tokens, width, dtype=BF), routing(35, tokens, topk, experts)
    probs, dy = torch.rand(tokens, topk, generator=g, device="cuda"), randn(g, tokens, width, dtype=BF)
    w1, w2 = (randn(g, experts, hidden, width) / 8).to(BF), (randn(g, experts, width, hidden) / 12).to(BF)
    moms = [torch.zeros(*w.shape, device="cuda") for w in (w1, w2)]
    step = nsm.ExpertMuonStep([w1, w2], moms, slice_bytes=hidden * width * 4)

    def run():
        y, backward = layer(x, ids, probs, w1, w2)
        out = backward(dy)
        step([out[4], out[5]])
        return (y,) + out[:4]

    start = [t.clone() for t in [w1, w2] + moms]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for seed in (36, 37):
        g = gen(seed)
        x.copy_(randn(g, tokens, width, dtype=BF))
        ids.copy_(routing(seed, tokens, topk, experts, 0.3))
        results = []
        for replay in (True, False):
            for t, s in zip([w1, w2] + moms, start):
                t.copy_(s)
            if replay:
                graph.replay()
                out = captured
            else:
                out = run()
            results.append([t.clone() for t in list(out) + [w1, w2] + moms])
        for a, b in zip(*results):
            assert torch.equal(a, b)


def test_expert_launches_are_profiled():
    offsets, xs, dys, w = product_case(38, [100, 28], 64, 64, BF)
    nsm.muon_profile_begin()
    offs, slot, _ = nsm.muon_expert_sort(routing(39, 64, 2, 4), 4)
    rows = nsm.muon_expert_gather(randn(gen(40), 64, 32, dtype=BF), slot)
    nsm.muon_expert_combine_backward(nsm.muon_expert_combine(rows, slot), rows, slot)
    nsm.muon_expert_product(xs, w, offsets)
    nsm.muon_expert_weight_grad(dys.float(), xs.float(), offsets)
    prof = {r["kernel"]: r for r in nsm.muon_profile_end()}
    for name in ("expert_sort", "expert_gather", "expert_combine", "expert_combine_backward"):
        assert prof[name]["launches"] == 1 and prof[name]["ms"] > 0, name
    assert sum(r["launches"] for name, r in prof.items() if name.startswith("expert_product")) == 2


# ---------------------------------------------------------------- forms of their own
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows", [4096, 4097, 16384, 16385])
def test_long_fp32_weight_gradients_keep_their_accuracy(rows, dtype):
    """fp32 dW of 16-bit operands at lengths around whole runs of 512 tokens.

    A run is 32 steps of 16 tokens, each of which truncates its sum: at most one
    step of 2^-23 relative to a partial sum that grows as sqrt(k), half of it on
    average, times the mean 0.72 of 1 / mantissa.  That is 0.36 * 2^-23 *
    sum sqrt(k / 32) = 9.4e-7 relative to the result, whatever the number of runs
    (they are added with round-to-nearest).  One sum over 4096 tokens would have
    256 steps and 7.3e-6, over 16384 2.9e-5: 1.5e-6 lies between."""
    counts = [rows, 513]
    offsets, xs, dys, _ = product_case(25, counts, 256, 264, dtype)
    dw = nsm.muon_expert_weight_grad(dys, xs, offsets, out_dtype=SF)
    for e, (lo, hi) in enumerate(segments(offsets, xs.shape[0])):
        ref = f64(dys[lo:hi]).T @ f64(xs[lo:hi])
        err = float((f64(dw[e]) - ref).norm() / ref.norm())
        assert err <= 1.5e-6, (e, err)
    out = torch.zeros_like(dw)
    nsm.muon_expert_weight_grad(dys, xs, offsets, out=out, accumulate=True)
    assert torch.equal(out, dw)


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("counts,inner,outer", [([40, 0, 300], 128, 96), ([3, 1, 0, 5], 64, 264)])
def test_products_of_permuted_stacks(counts, inner, outer, dtype):
    """Weights and dW whose experts alternate row by row: the expert stride is below the row pitch."""
    offsets, xs, dys, w = product_case(26, counts, inner, outer, dtype)
    permuted = w.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    assert permuted.stride(0) == inner < permuted.stride(1)
    check_products(offsets, xs, dys, permuted, U_NEAREST if dtype == SF else U_TRUNCATED)
    used = sum(counts)
    for call, rows in ((nsm.muon_expert_product, xs), (nsm.muon_expert_input_grad, dys)):
        assert torch.equal(call(rows, permuted, offsets)[:used], call(rows, w, offsets)[:used])
    for dw_dtype, accumulate in ((dtype, False), (SF, False), (SF, True)):
        store = torch.full((outer + 1, len(counts) + 1, inner), 7.0, dtype=dw_dtype, device="cuda")
        out = store[:outer, :len(counts)].permute(1, 0, 2)
        dense = torch.full((len(counts), outer, inner), 7.0, dtype=dw_dtype, device="cuda")
        nsm.muon_expert_weight_grad(dys, xs, offsets, out=out, accumulate=accumulate)
        nsm.muon_expert_weight_grad(dys, xs, offsets, out=dense, accumulate=accumulate)
        assert torch.equal(out, dense)
        assert bool((store[outer:] == 7).all()) and bool((store[:, len(counts):] == 7).all())


def test_expert_step_reports_its_weight_gradients():
    """Every slice has a word that its weight gradients write, eagerly and replayed; a set one flags the slice's blocks."""
    g = gen(43)
    w, m = randn(g, 3, 64, 32, dtype=BF), torch.zeros(3, 64, 32, device="cuda")
    step = nsm.ExpertMuonStep([w], [m], blocks=[(32, 32)], slice_bytes=1)
    factors = [(randn(g, 12, 64, dtype=BF), randn(g, 12, 32, dtype=BF), offsets_of([3, 5, 4]))]
    step(factors)
    assert len(step.words) == 3 and step.status.tolist() == [0] * 6
    step.words[1].fill_(2)
    assert step.status.tolist() == [0, 0, 2, 2, 0, 0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(factors)
    for run in (graph.replay, lambda: step(factors)):
        step.words[1].fill_(2)
        run()
        assert step.status.tolist() == [0] * 6


@pytest.mark.parametrize("dtype", [BF, HF, SF])
@pytest.mark.parametrize("counts,inner,outer", [([45, 44, 151, 66, 72, 0, 86], 7, 24), ([499], 325, 163), ([64, 33, 200], 171, 331),
                                                ([5, 6, 11, 0, 32], 15, 560), ([1, 40], 1, 3), ([300, 41], 518, 263)])
def test_results_of_ragged_rows_keep_what_lies_behind_them(counts, inner, outer, dtype):
    """Results whose rows start on 16 bytes and end inside 16: the columns behind them stay, and the operands'
    columns behind the rows (NaN) are not read."""
    def wide(*shape, fill=7.0, dt=dtype):
        store = torch.full((*shape[:-1], -(-shape[-1] // 8) * 8 + 8), fill, dtype=dt, device="cuda")
        return store[..., :shape[-1]], store[..., shape[-1]:]

    g = gen(44)
    rows, nan = sum(counts) + 2, float("nan")
    offsets = offsets_of(counts)
    (xs, _), (dys, _), (w, _) = (wide(*s, fill=nan) for s in ((rows, inner), (rows, outer), (len(counts), outer, inner)))
    for t in (xs, dys, w):
        t.copy_(randn(g, *t.shape, dtype=dtype))
    u = U_NEAREST if dtype == SF else U_TRUNCATED
    (y, behind_y), (dx, behind_dx) = wide(rows, outer), wide(rows, inner)
    nsm.muon_expert_product(xs, w, offsets, out=y)
    nsm.muon_expert_input_grad(dys, w, offsets, out=dx)
    results = []
    for dt, accumulate in ((dtype, False), (SF, False), (SF, True)):
        dw, behind = wide(len(counts), outer, inner, dt=dt)
        dw.zero_()
        nsm.muon_expert_weight_grad(dys, xs, offsets, out=dw, accumulate=accumulate)
        assert bool((behind == 7).all()), (dt, accumulate)
        results.append(dw)
    assert bool((behind_y == 7).all()) and bool((behind_dx == 7).all())
    assert bool((y[sum(counts):] == 7).all()) and bool((dx[sum(counts):] == 7).all())
    for e, (lo, hi) in enumerate(segments(offsets, rows)):
        x, d, m = f64(xs[lo:hi]), f64(dys[lo:hi]), f64(w[e])
        close(y[lo:hi], x @ m.T, inner, x.abs() @ m.abs().T, u)
        close(dx[lo:hi], d @ m, outer, d.abs() @ m.abs(), u)
        for dw in results:
            close(dw[e], d.T @ x, hi - lo, d.abs().T @ x.abs(), u)


def test_calls_at_once_from_several_threads():
    """Four threads, each on a stream of its own, run the operators and the block step at the same time, and get
    what one after the other gives."""
    import threading

    def work(seed, stream=None):
        g = gen(seed)
        counts = [300, 0, 41, 170]
        offsets, xs, dys, w = product_case(seed, counts, 256 + 8 * seed, 192, BF, tail=0)
        ids, m = routing(seed, 3000, 4, 64, 0.1), randn(g, 8, 64, 512) * 0.1
        p, gr = randn(g, 8, 64, 512, dtype=BF), randn(g, 8, 64, 512, dtype=BF)
        wm = torch.zeros(*w.shape, device="cuda")
        torch.cuda.current_stream().synchronize()
        out = []
        for _ in range(20):
            offs, slot, source = nsm.muon_expert_sort(ids, 64, stream=stream)
            y = nsm.muon_expert_product(xs, w, offsets, stream=stream)
            dw = nsm.muon_expert_weight_grad(dys, xs, offsets, out_dtype=SF, stream=stream)
            nsm.muon_step_blocks([p, w], [gr, dw], [m, wm], [(64, 256), None], stream=stream)
            out = [offs, slot, source, y, dw, p, m, w, wm]
        (stream or torch.cuda.current_stream()).synchronize()
        return out

    want = [work(60 + i) for i in range(4)]
    got, streams = [None] * 4, [torch.cuda.Stream() for _ in range(4)]

    def run(i):
        with torch.cuda.stream(streams[i]):
            got[i] = work(60 + i, streams[i])

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
