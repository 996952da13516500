"""Host-only checks of the expert-layer operators and the block step: argument
checks of the C ABI and of the binding, workspace sizes, without a GPU."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import newton_schulz_matrix_b200 as nsm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # a stand-in device pointer: nothing below launches


@pytest.fixture(scope="module")
def lib():
    from newton_schulz_matrix_b200 import build
    build.build()
    return nsm.load_library()


def test_sort_refusals(lib):
    size = lib.muon_expert_sort_workspace_size
    assert size(32, 8, 216) > 0 and size(0, 1, 1) > 0
    assert size(1 << 20, 8, 64) > 256  # several runs count apart
    for bad in ((-1, 8, 64), (32, 0, 64), (32, 8, 0), (32, 8, nsm.EXPERT_MAX + 1), (1 << 30, 8, 64), (1 << 27, 9, 64)):
        assert size(*bad) == 0
    ok = dict(ids=P, es=8, ld=8, tokens=1 << 17, topk=8, experts=64, offsets=P, slot=P, source=P, ws=P, bytes=0)
    # the workspace is too small: every other argument is right
    assert lib.muon_expert_sort(*ok.values(), None) == -3
    for change, rc in ((dict(es=2), -2), (dict(ids=None), -1), (dict(ids=P + 4), -1), (dict(ld=7), -1), (dict(topk=0), -1),
                       (dict(tokens=-1), -1), (dict(experts=0), -1), (dict(experts=2000), -1), (dict(offsets=None), -1),
                       (dict(offsets=P + 2), -1), (dict(slot=P + 1), -1), (dict(source=None), -1), (dict(ws=None), -1),
                       (dict(ws=P + 2), -1), (dict(tokens=1 << 29), -1)):
        assert lib.muon_expert_sort(*dict(ok, **change).values(), None) == rc, change


def test_route_refusals(lib):
    gather = dict(x=P, ld_x=64, slot=P, tokens=4, topk=2, cols=64, dtype=0, xs=P, ld_xs=64, rows=8)
    for change, rc in ((dict(ld_x=63), -1), (dict(x=None), -1), (dict(x=P + 1), -1), (dict(slot=None), -1),
                       (dict(slot=P + 2), -1), (dict(topk=0), -1), (dict(cols=0), -1), (dict(tokens=-1), -1),
                       (dict(dtype=3), -2), (dict(xs=P + 1), -1), (dict(ld_xs=10), -1), (dict(rows=-1), -1),
                       (dict(rows=(1 << 30) + 1), -1), (dict(cols=(1 << 30) + 1, ld_x=1 << 31, ld_xs=1 << 31), -1), (dict(dtype=2, x=P + 2), -1), (dict(tokens=1 << 30, topk=4), -1)):
        assert lib.muon_expert_gather(*dict(gather, **change).values(), None) == rc, change
    assert lib.muon_expert_gather(*dict(gather, tokens=0, slot=None, x=None).values(), None) == 0
    combine = dict(ys=P, ld_ys=64, rows=8, slot=P, w=P, wdt=2, tokens=4, topk=2, cols=64, dtype=0, y=P, ld_y=64)
    for change, rc in ((dict(ys=None), -1), (dict(ld_ys=1), -1), (dict(w=P + 2), -1), (dict(wdt=5), -2), (dict(y=None), -1),
                       (dict(ld_y=0), -1), (dict(dtype=-1), -2), (dict(slot=None), -1)):
        assert lib.muon_expert_combine(*dict(combine, **change).values(), None) == rc, change
    back = dict(dy=P, ld_dy=64, ys=P, ld_ys=64, rows=8, slot=P, w=P, wdt=2, tokens=4, topk=2, cols=64, dtype=0, dys=P,
                ld_dys=64, dw=P)
    for change, rc in ((dict(dy=None), -1), (dict(ld_dy=2), -1), (dict(ys=None), -1), (dict(dys=None), -1),
                       (dict(dw=P + 2), -1), (dict(w=None, wdt=9), -2), (dict(ld_dys=63), -1)):
        assert lib.muon_expert_combine_backward(*dict(back, **change).values(), None) == rc, change


def test_product_refusals(lib):
    fwd = dict(xs=P, ld_xs=64, w=P, ld_w=64, stride_w=64 * 32, offsets=P, experts=4, rows=10, inner=64, outer=32, dtype=0,
               y=P, ld_y=32, ws=None, ws_bytes=0, status=None)
    for change, rc in ((dict(xs=None), -1), (dict(ld_xs=63), -1), (dict(w=P + 1), -1), (dict(ld_w=1), -1),
                       (dict(stride_w=-1), -1), (dict(offsets=None), -1), (dict(offsets=P + 2), -1), (dict(experts=0), -1),
                       (dict(experts=1025), -1), (dict(rows=-1), -1), (dict(inner=0), -1), (dict(outer=0), -1),
                       (dict(dtype=4), -2), (dict(y=None), -1), (dict(ld_y=31), -1)):
        assert lib.muon_expert_product(*dict(fwd, **change).values(), None) == rc, change
    assert lib.muon_expert_product(*dict(fwd, rows=0, xs=None, y=None).values(), None) == 0
    dgrad = dict(fwd, xs=P, ld_xs=32, y=P, ld_y=64)
    for change, rc in ((dict(ld_xs=31), -1), (dict(ld_y=63), -1), (dict(dtype=9), -2), (dict(offsets=None), -1)):
        assert lib.muon_expert_input_grad(*dict(dgrad, **change).values(), None) == rc, change
    wgrad = dict(dys=P, ld_dys=32, xs=P, ld_xs=64, offsets=P, experts=4, rows=10, inner=64, outer=32, dtype=0, dw=P, ld_dw=64,
                 stride_dw=64 * 32, dw_dtype=0, accumulate=0, ws=None, ws_bytes=0, status=None)
    for change, rc in ((dict(dys=None), -1), (dict(xs=P + 1), -1), (dict(ld_dw=63), -1), (dict(dw=None), -1),
                       (dict(dw_dtype=1), -2), (dict(accumulate=1), -2), (dict(dtype=1), -2), (dict(stride_dw=0), -1),
                       (dict(stride_dw=-8), -1), (dict(dw_dtype=2, dw=P + 2), -1)):
        assert lib.muon_expert_weight_grad(*dict(wgrad, **change).values(), None) == rc, change


def test_workspaces_of_products(lib):
    """Only large 16-bit products with an operand that TMA cannot address take one: its rows, padded to 8 elements."""
    size = lib.muon_expert_workspace_size
    ok = dict(kind=0, a=P, ld_a=1024, b=P, ld_b=1024, stride_b=1024 * 512, experts=4, rows=2048, inner=1024, outer=512, dtype=0)
    assert size(*ok.values()) == 0
    rows, weights = 2048 * 1024 * 2, 4 * 512 * 1024 * 2
    for change, least in ((dict(a=P + 2), rows), (dict(ld_a=1025), rows), (dict(b=P + 8), weights), (dict(ld_b=1030), weights),
                          (dict(stride_b=1024 * 512 + 4), weights), (dict(stride_b=0), weights),
                          (dict(a=P + 2, ld_b=1028), rows + weights), (dict(kind=2, a=P + 2), 2048 * 512 * 2)):
        assert least <= size(*dict(ok, **change).values()) <= least + 1024, change
    odd = size(*dict(ok, inner=1021, ld_a=1021, ld_b=1021, stride_b=1021 * 512).values())
    assert rows + weights <= odd <= rows + weights + 1024  # 1021 columns in rows of 1024
    for change in (dict(a=P + 2, rows=4), dict(a=P + 2, dtype=2), dict(a=P + 2, kind=3), dict(a=P + 2, rows=-1),
                   dict(a=P + 2, experts=0), dict(a=P + 2, dtype=7), dict(a=P + 2, inner=0)):
        assert size(*dict(ok, **change).values()) == 0, change


def _block_group(ptr=P, rows=64, cols=128, count=2, down=1, across=1, wdt=0, gdt=0, ld=(256, 256, 256)):
    arrs = [(ctypes.c_void_p * count)(*[ptr + 2 * 128 * i for i in range(count)]) for _ in range(2)]
    arrs.append((ctypes.c_void_p * count)(*[P + 4 * 128 * i for i in range(count)]))
    return nsm._BlockGroup(rows, cols, count, down, across, wdt, gdt, *ld, *arrs), arrs


def test_block_step_refusals(lib):
    ns, _a = nsm._ns_params((nsm.QUINTIC,) * 5, "standard", 2, 1e-7, "fp16", "fp16")
    hp = nsm._hparams(0.02, 0.95, 0.1, 0.2, 1, ns)
    ws = ctypes.c_void_p(1 << 24)

    def call(group, n=1, ws=ws, size=1 << 30, hp=hp):
        return lib.muon_step_blocks((nsm._BlockGroup * 1)(group), n, ctypes.byref(hp), ws, size, None, None)

    good, keep = _block_group()
    size = lib.muon_blocks_workspace_size((nsm._BlockGroup * 1)(good), 1, ctypes.byref(hp))
    assert size == lib.muon_ns_workspace_size(2, 64, 128, ctypes.byref(ns))
    least = lib.muon_blocks_workspace_min((nsm._BlockGroup * 1)(good), 1, ctypes.byref(hp))
    assert least == lib.muon_ns_workspace_size(1, 64, 128, ctypes.byref(ns))
    tiled, keep1 = _block_group(down=3, across=2)
    assert lib.muon_blocks_workspace_size((nsm._BlockGroup * 1)(tiled), 1, ctypes.byref(hp)) == \
        lib.muon_ns_workspace_size(12, 64, 128, ctypes.byref(ns))
    assert call(good, n=0) == -1 and call(good, ws=None) == -1 and call(good, ws=ctypes.c_void_p((1 << 24) + 8)) == -1
    assert call(good, size=1024) == -3
    for kw, rc in ((dict(ptr=P + 1), -1), (dict(rows=0), -1), (dict(cols=-1), -1), (dict(wdt=3), -2), (dict(gdt=-1), -2),
                   (dict(ld=(127, 256, 256)), -1), (dict(down=0), -1), (dict(across=-1), -1), (dict(across=3), -1),
                   (dict(down=1 << 20), -1), (dict(down=1 << 16, across=1 << 16, cols=1, ld=(1 << 20,) * 3), -1), (dict(ld=(256, 0, 256)), -1), (dict(ld=(256, 256, 1 << 31)), -1)):
        bad, keep2 = _block_group(**kw)
        assert call(bad) == rc, kw
        assert lib.muon_blocks_workspace_size((nsm._BlockGroup * 1)(bad), 1, ctypes.byref(hp)) == 0
    # two-byte alignment is enough for 16-bit elements: refused for its size alone
    odd, keep3 = _block_group(ptr=P + 2)
    assert call(odd, size=1024) == -3
    nan = nsm._hparams(0.02, float("nan"), 0.1, 0.2, 1, ns)
    assert call(good, hp=nan) == -1


def test_the_binding_refuses_what_it_cannot_run():
    x, slot, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int64)
    w, offsets = torch.zeros(2, 3, 8), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: nsm.muon_expert_sort(ids, 4), lambda: nsm.muon_expert_gather(x, slot),
                 lambda: nsm.muon_expert_combine(x, slot), lambda: nsm.muon_expert_gather_backward(x, slot),
                 lambda: nsm.muon_expert_combine_backward(x, x, slot), lambda: nsm.muon_expert_product(x, w, offsets),
                 lambda: nsm.muon_expert_input_grad(x, w, offsets), lambda: nsm.muon_expert_weight_grad(x, x, offsets),
                 lambda: nsm.muon_step_blocks([x], [x], [x], [(2, 8)]), lambda: nsm.ExpertMuonStep([w], [w]),
                 lambda: nsm.ExpertMuonStep([], []), lambda: nsm.MuonStep([x], [x], [x], blocks=[(2, 8)])):
        with pytest.raises(nsm.MuonError):
            call()


class Fake:
    """A CUDA matrix for the binding's checks alone."""

    def __init__(self, shape, stride=None, dtype=torch.bfloat16, device="cuda:0"):
        self.shape = torch.Size(shape)
        self._stride = tuple(stride) if stride else tuple(torch.empty(shape, device="meta").stride())
        self.dtype, self.device, self.is_cuda = dtype, torch.device(device), True

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return P

    def is_contiguous(self):
        return self._stride == tuple(torch.empty(self.shape, device="meta").stride())


def test_shapes_types_and_devices_are_checked():
    bf, i32 = torch.bfloat16, torch.int32
    x, slot = Fake((4, 8)), Fake((4, 2), dtype=i32)
    w, offsets = Fake((2, 3, 8)), Fake((3,), dtype=i32)
    bad = [
        lambda: nsm.muon_expert_sort(Fake((4, 2), dtype=torch.int16), 4),
        lambda: nsm.muon_expert_sort(Fake((4,), dtype=i32), 4),
        lambda: nsm.muon_expert_sort(Fake((4, 2), dtype=i32), 0),
        lambda: nsm.muon_expert_sort(Fake((4, 2), dtype=i32), 1025),
        lambda: nsm.muon_expert_sort(Fake((4, 2), (1, 4), dtype=i32), 4),           # columns are not contiguous
        lambda: nsm.muon_expert_sort(Fake((4, 2), (0, 1), dtype=i32), 4),           # one row, broadcast
        lambda: nsm.muon_expert_gather(x, Fake((4, 2), dtype=torch.int64)),
        lambda: nsm.muon_expert_gather(x, Fake((5, 2), dtype=i32)),                 # another number of tokens
        lambda: nsm.muon_expert_gather(x, Fake((4, 2), dtype=i32, device="cuda:1")),
        lambda: nsm.muon_expert_gather(Fake((4, 8), dtype=torch.float64), slot),
        lambda: nsm.muon_expert_gather(Fake((4, 8), (1, 4)), slot),
        lambda: nsm.muon_expert_gather(Fake((4, 8), (0, 1)), slot),
        lambda: nsm.muon_expert_gather(x, slot, out=Fake((8, 9))),
        lambda: nsm.muon_expert_gather(x, slot, out=Fake((8, 8), dtype=torch.float16)),
        lambda: nsm.muon_expert_combine(x, slot, Fake((4, 3))),
        lambda: nsm.muon_expert_combine(x, slot, Fake((4, 2), (1, 4))),
        lambda: nsm.muon_expert_combine(x, slot, Fake((4, 2), device="cuda:1")),
        lambda: nsm.muon_expert_combine(x, slot, out=Fake((3, 8))),
        lambda: nsm.muon_expert_combine_backward(Fake((4, 9)), x, slot),
        lambda: nsm.muon_expert_combine_backward(Fake((4, 8), (0, 1)), x, slot),    # a broadcast gradient
        lambda: nsm.muon_expert_combine_backward(x, x, slot, out=Fake((5, 8))),
        lambda: nsm.muon_expert_product(x, Fake((2, 3, 9)), offsets),
        lambda: nsm.muon_expert_product(x, Fake((3, 3, 8)), offsets),
        lambda: nsm.muon_expert_product(x, Fake((2, 3, 8), dtype=torch.float16), offsets),
        lambda: nsm.muon_expert_product(x, w, Fake((3,), dtype=torch.int64)),
        lambda: nsm.muon_expert_product(x, w, Fake((1,), dtype=i32)),
        lambda: nsm.muon_expert_product(x, w, offsets, out=Fake((4, 4))),
        lambda: nsm.muon_expert_product(x, w, offsets, status=Fake((2,), dtype=i32)),
        lambda: nsm.muon_expert_input_grad(x, w, offsets),
        lambda: nsm.muon_expert_weight_grad(x, Fake((5, 8)), offsets),
        lambda: nsm.muon_expert_weight_grad(x, x, offsets, accumulate=True),
        lambda: nsm.muon_expert_weight_grad(x, x, offsets, out=Fake((2, 8, 9))),
        lambda: nsm.muon_expert_weight_grad(x, x, offsets, out=Fake((2, 8, 8)), out_dtype=torch.float32),
        lambda: nsm.muon_expert_weight_grad(x, x, offsets, out_dtype=torch.float64),
        lambda: nsm.muon_step_blocks([x], [x], [Fake((4, 8), dtype=torch.float32)], [(3, 8)]),
        lambda: nsm.muon_step_blocks([x], [x], [Fake((4, 8), dtype=torch.float32)], [(2, 8), None]),
        lambda: nsm.muon_step_blocks([x], [x], [x], [(2, 8)]),
        lambda: nsm.muon_step_blocks([x], [Fake((8, 4))], [Fake((4, 8), dtype=torch.float32)], [None]),
        lambda: nsm.muon_step_blocks([x], [Fake((4, 8), (0, 1))], [Fake((4, 8), dtype=torch.float32)], [None]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(nsm.MuonError):
            call()
            raise AssertionError(i)


def test_block_groups_name_every_block_once():
    """Pointers and status order of a strided stack, by hand."""
    w = Fake((2, 4, 6), (100, 10, 1))
    m = Fake((2, 4, 6), (24, 6, 1), dtype=torch.float32)
    groups, n, _keep, order = nsm._build_block_groups([w, w], [w, w], [m, m], [(2, 3), None])
    assert n == 2 and order == list(range(10))
    g = groups[0]
    assert (g.rows, g.cols, g.count, g.down, g.across, g.ld_w, g.ld_g, g.ld_m) == (2, 3, 2, 2, 2, 10, 10, 6)
    assert [g.W[i] - P for i in range(2)] == [0, 200] and [g.M[i] - P for i in range(2)] == [0, 96]
    g = groups[1]
    assert (g.rows, g.cols, g.count, g.down, g.across) == (4, 6, 2, 1, 1) and [g.W[i] - P for i in range(2)] == [0, 200]


def test_products_of_too_many_weight_rows(lib):
    """experts * outer is at most 2^34: above it tile counts would pass 32 bits."""
    outer = (1 << 25) + 1
    assert lib.muon_expert_product(P, 8, P, 8, 8 * outer, P, 512, 10, 8, outer, 0, P, outer, None, 0, None, None) == -1
    assert lib.muon_expert_input_grad(P, outer, P, 8, 8 * outer, P, 512, 10, 8, outer, 0, P, 8, None, 0, None, None) == -1
    assert lib.muon_expert_weight_grad(P, outer, P, 8, P, 512, 10, 8, outer, 0, P, 8, 8 * outer, 0, 0, None, 0, None, None) == -1


def test_a_timed_out_weight_gradient_flags_its_slice():
    """ExpertMuonStep.status: the word of a slice's weight gradients reaches every block of that slice, and no other."""
    class Step:
        def __init__(self, words):
            self.words = torch.tensor(words, dtype=torch.int32)

        def status_in_param_order(self):
            return self.words

    step = nsm.ExpertMuonStep.__new__(nsm.ExpertMuonStep)
    step.steps = [Step([0, 1, 0]), Step([0, 0]), Step([1])]
    step.words = torch.tensor([2, 0, 2], dtype=torch.int32).split(1)
    assert step.status.tolist() == [2, 3, 2, 0, 0, 3]


def test_blocks_that_share_memory_are_refused():
    """Two blocks of one launch must not update the same memory; gradients may be broadcast."""
    sf = torch.float32
    good, mom = Fake((2, 4, 6)), Fake((2, 4, 6), dtype=sf)
    for strides in ((0, 6, 1), (12, 6, 1), (23, 6, 1), (5, 10, 1), (6, 6, 1)):
        for call in (lambda t, m: nsm._build_block_groups([t], [good], [m], [(2, 3)]),
                     lambda t, m: nsm.ExpertMuonStep([t], [m], slice_bytes=1)):
            with pytest.raises(nsm.MuonError, match="overlaps"):
                call(Fake((2, 4, 6), strides), mom)
            with pytest.raises(nsm.MuonError, match="overlaps"):
                call(good, Fake((2, 4, 6), strides, dtype=sf))
        with pytest.raises(nsm.MuonError, match="overlaps"):
            nsm.muon_expert_weight_grad(Fake((5, 4)), Fake((5, 6)), Fake((3,), dtype=torch.int32), out=Fake((2, 4, 6), strides))
        assert nsm._build_block_groups([good], [Fake((2, 4, 6), (strides[0], 6, 1))], [mom], [None])[1] == 1
    # the experts of a permuted stack, the halves of fused columns, rows that interleave without meeting
    for strides in ((6, 12, 1), (6, 20, 1), (24, 6, 1), (9, 18, 1), (7, 15, 1)):
        assert nsm._build_block_groups([Fake((2, 4, 6), strides)], [good], [Fake((2, 4, 6), strides, dtype=sf)], [None])[1] == 1
    assert nsm._build_block_groups([Fake((3, 2, 2), (4, 6, 1))], [Fake((3, 2, 2))], [Fake((3, 2, 2), dtype=sf)], [None])[1] == 1


@pytest.mark.parametrize("shape", [(0, 4, 8), (2, 0, 8), (2, 4, 0)])
def test_empty_stacks_are_refused(shape):
    with pytest.raises(nsm.MuonError):
        nsm.ExpertMuonStep([Fake(shape)], [Fake(shape, dtype=torch.float32)])


def test_sizes_that_pass_32_bits_are_refused():
    """ctypes keeps the low 32 bits of an int argument: 2^32 + 4 tokens must not be sorted as 4."""
    i32, sf, big = torch.int32, torch.float32, 2 ** 32
    offsets, few, tall, wide = Fake((2,), dtype=i32), Fake((4, 8)), Fake((big + 4, 8)), Fake((1, big + 8))
    calls = [
        lambda: nsm.muon_expert_sort(Fake((big + 4, 1), dtype=i32), 8),
        lambda: nsm.muon_expert_sort(Fake((0, big + 1), dtype=i32), 8),
        lambda: nsm.muon_expert_sort(Fake((4, 2), dtype=i32), big + 8),
        lambda: nsm.muon_expert_gather(tall, Fake((big + 4, 1), dtype=i32)),
        lambda: nsm.muon_expert_gather(wide, Fake((1, 1), dtype=i32)),
        lambda: nsm.muon_expert_combine(few, Fake((big + 4, 1), dtype=i32)),
        lambda: nsm.muon_expert_combine(few, Fake((1 << 29, 4), dtype=i32)),
        lambda: nsm.muon_expert_combine(wide, Fake((1, 1), dtype=i32)),
        lambda: nsm.muon_expert_combine_backward(Fake((big + 4, 8)), few, Fake((big + 4, 1), dtype=i32)),
        lambda: nsm.muon_expert_product(few, Fake((1, big + 8, 8)), offsets),
        lambda: nsm.muon_expert_product(wide, Fake((1, 1, big + 8)), offsets),
        lambda: nsm.muon_expert_input_grad(wide, Fake((1, big + 8, 1)), offsets),
        lambda: nsm.muon_expert_weight_grad(few, Fake((4, big + 8)), offsets),
        lambda: nsm.muon_expert_weight_grad(few, few, Fake((big + 2,), dtype=i32)),
    ]
    for t, m in ((wide, Fake((1, big + 8), dtype=sf)), (Fake((big + 8, 1)), Fake((big + 8, 1), dtype=sf))):
        calls += [lambda t=t, m=m: nsm.muon_step_blocks([t], [t], [m], [None]),
                  lambda t=t, m=m: nsm.muon_blocks_workspace_size([t], [t], [m], [(1, 1)]),
                  lambda t=t, m=m: nsm.muon_step([t], [t], [m]),
                  lambda t=t: nsm.muon_ns_batched([t]), lambda t=t: nsm.muon_ns_batched_noalloc([t])]
    for i, call in enumerate(calls):
        try:
            call()
        except nsm.MuonError as e:
            assert "CUDA" not in str(e), (i, e)  # refused for its size, not by a launch
        else:
            raise AssertionError(i)


def test_status_and_workspace_are_checked_before_the_step():
    """A strided status would be refused by the copy behind the step, a strided workspace would be written in its gaps."""
    w, m, i32, u8 = Fake((2, 4, 8)), Fake((2, 4, 8), dtype=torch.float32), torch.int32, torch.uint8
    step = lambda **kw: nsm.muon_step_blocks([w], [w], [m], [None], **kw)
    ids = Fake((1 << 17, 8), dtype=i32)
    for call in (lambda: step(status=Fake((2,), (2,), dtype=i32)), lambda: step(workspace=Fake((1 << 24,), (2,), dtype=u8)),
                 lambda: step(workspace=Fake((1 << 24,), dtype=u8, device="cuda:1")),
                 lambda: nsm.muon_expert_sort(ids, 8, workspace=Fake((1 << 24,), (2,), dtype=u8)),
                 lambda: nsm.muon_expert_sort(ids, 8, workspace=Fake((1 << 24,), dtype=u8, device="cuda:1")),
                 lambda: nsm.MuonStep([w], [w], [m], blocks=[None], workspace=Fake((1 << 24,), (2,), dtype=u8)),
                 lambda: nsm.MuonStep([w], [w], [m], blocks=[None], workspace=Fake((1 << 24,), dtype=u8, device="cuda:1"))):
        with pytest.raises(nsm.MuonError, match="contiguous|is on"):
            call()


def test_no_exception_leaves_the_library(lib):
    """Host memory that runs out is an error code, not std::terminate (in a process of its own, with a bounded address space)."""
    code = """
import ctypes, resource, sys
sys.path.insert(0, {root!r})
import newton_schulz_matrix_b200 as nsm
lib = nsm.load_library()
ns, keep = nsm._ns_params((nsm.QUINTIC,) * 5, "standard", 2, 1e-7, "fp16", "fp16")
hp = nsm._hparams(0.02, 0.95, 0.1, 0.2, 1, ns)
n = 1 << 22
plain, blocks = (nsm._Group * n)(), (nsm._BlockGroup * n)()
one, ld = nsm._Group(8, 8, 0, 0, 0), nsm._BlockGroup(8, 8, 0, 1, 1, 0, 0, 8, 8, 8)
for array, item in ((plain, one), (blocks, ld)):
    raw = bytes(item)
    ctypes.memmove(array, raw * n, len(raw) * n)
    del raw
pages = int(open("/proc/self/statm").read().split()[0])
limit = pages * resource.getpagesize() + (64 << 20)
resource.setrlimit(resource.RLIMIT_AS, (limit, limit))
ws = ctypes.c_void_p(1 << 24)
for kind, array in (("muon", plain), ("muon_blocks", blocks)):
    assert getattr(lib, kind + "_workspace_size")(array, n, ctypes.byref(hp)) == 0, kind
    assert getattr(lib, kind + "_workspace_min")(array, n, ctypes.byref(hp)) == 0, kind
assert lib.muon_step(plain, n, ctypes.byref(hp), ws, 1 << 30, None, None) == -1
assert lib.muon_step_blocks(blocks, n, ctypes.byref(hp), ws, 1 << 30, None, None) == -1
""".format(root=ROOT)
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, (run.returncode, run.stderr[-500:])


def test_overlap_is_found_on_the_host_whatever_the_default_device():
    w, m = Fake((3, 2, 2), (4, 6, 1)), Fake((3, 2, 2), dtype=torch.float32)
    with torch.device("meta"):
        assert nsm._build_block_groups([w], [w], [m], [None])[1] == 1
        with pytest.raises(nsm.MuonError, match="overlaps"):
            nsm._build_block_groups([Fake((3, 2, 2), (4, 5, 1))], [w], [m], [None])
