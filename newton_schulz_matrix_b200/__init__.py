"""Python binding of libmuon (include/muon.h): the Muon optimizer step (on
whole matrices, or on the blocks of stacked and fused weights), batched
Newton-Schulz orthogonalisation, and the expert-layer operators whose weight
gradients the step takes, on NVIDIA B200.

This module only marshals arguments: it turns torch tensors into device
pointers, groups, hyper-parameter structs and the current CUDA stream, and calls
the C ABI through ctypes.  Every step of the computation runs in the library's
CUDA kernels.  There is no fallback: if ``libmuon.so`` is missing or no CUDA
device is present, the calls raise.

Build the library with ``python -m newton_schulz_matrix_b200.build``.
"""
from __future__ import annotations

import ctypes
import os
from typing import Sequence

import torch

__all__ = [
    "BF16", "FP16", "FP32", "STANDARD", "GRAM", "GRAM_STABILIZED", "QUINTIC", "CUBIC",
    "MuonError", "load_library", "library_path", "muon_step", "muon_ns_batched",
    "muon_workspace_size", "muon_workspace_min", "muon_ns_workspace_size", "muon_ns_flops",
    "muon_status_string", "muon_profile_begin", "muon_profile_end", "MuonStep", "StreamedMuonStep",
    "plan_slices", "muon_ns_batched_noalloc", "muon_step_blocks", "muon_blocks_workspace_size",
    "muon_blocks_workspace_min", "muon_expert_sort", "muon_expert_gather", "muon_expert_gather_backward",
    "muon_expert_combine", "muon_expert_combine_backward", "muon_expert_product", "muon_expert_input_grad",
    "muon_expert_weight_grad", "ExpertMuonStep", "EXPERT_MAX",
    "NOALLOC_SCRATCH_BYTES", "EXPORTED_SYMBOLS",
]

BF16, FP16, FP32 = 0, 1, 2
STANDARD, GRAM, GRAM_STABILIZED = 0, 1, 2
_MODE_NAMES = {"standard": STANDARD, "gram": GRAM, "gram_stabilized": GRAM_STABILIZED}
_DT_NAMES = {"bf16": BF16, "fp16": FP16, "fp32": FP32}
QUINTIC = (3.4445, -4.7750, 2.0315)
CUBIC = (1.5, -0.5, 0.0)
EXPORTED_SYMBOLS = (
    "muon_workspace_size", "muon_workspace_min", "muon_step", "muon_ns_workspace_size",
    "muon_ns_batched", "muon_ns_flops", "muon_status_string", "muon_profile_begin", "muon_profile_end",
    "muon_ns_batched_noalloc", "muon_blocks_workspace_size", "muon_blocks_workspace_min", "muon_step_blocks",
    "muon_expert_sort_workspace_size", "muon_expert_sort", "muon_expert_gather", "muon_expert_combine",
    "muon_expert_combine_backward", "muon_expert_product", "muon_expert_input_grad", "muon_expert_weight_grad",
    "muon_expert_workspace_size",
)
EXPERT_MAX = 1024
_EXPERT_MOST = 1 << 30  # rows, columns and tokens * topk of the expert operators
NOALLOC_SCRATCH_BYTES = 64 << 20

_HERE = os.path.dirname(os.path.abspath(__file__))
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_LIB = None


class MuonError(RuntimeError):
    pass


class _NSParams(ctypes.Structure):
    _fields_ = [("iters", ctypes.c_int), ("coeffs", ctypes.POINTER(ctypes.c_float)), ("mode", ctypes.c_int),
                ("restart_after", ctypes.c_int), ("eps", ctypes.c_float), ("compute_dtype", ctypes.c_int),
                ("gram_dtype", ctypes.c_int), ("restart_every", ctypes.c_int)]


class _Group(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("count", ctypes.c_int),
                ("w_dtype", ctypes.c_int), ("g_dtype", ctypes.c_int),
                ("W", ctypes.POINTER(ctypes.c_void_p)), ("G", ctypes.POINTER(ctypes.c_void_p)),
                ("M", ctypes.POINTER(ctypes.c_void_p))]


class _BlockGroup(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int), ("cols", ctypes.c_int), ("count", ctypes.c_int),
                ("down", ctypes.c_int), ("across", ctypes.c_int), ("w_dtype", ctypes.c_int), ("g_dtype", ctypes.c_int),
                ("ld_w", ctypes.c_longlong), ("ld_g", ctypes.c_longlong), ("ld_m", ctypes.c_longlong),
                ("W", ctypes.POINTER(ctypes.c_void_p)), ("G", ctypes.POINTER(ctypes.c_void_p)),
                ("M", ctypes.POINTER(ctypes.c_void_p))]


class _HParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("scale_coef", ctypes.c_float), ("nesterov", ctypes.c_int), ("ns", _NSParams)]


class _ProfEntry(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_char_p), ("launches", ctypes.c_int), ("ms", ctypes.c_double),
                ("flops", ctypes.c_double), ("exec_flops", ctypes.c_double), ("bytes", ctypes.c_double)]


def library_path() -> str:
    return os.environ.get("MUON_LIBRARY", os.path.join(_HERE, "libmuon.so"))


def load_library() -> ctypes.CDLL:
    """Load libmuon.so (raises if it has not been built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise MuonError(f"{path} is missing: build it with `python -m newton_schulz_matrix_b200.build`")
    lib = ctypes.CDLL(path)
    P = ctypes.c_void_p
    lib.muon_workspace_size.argtypes = [ctypes.POINTER(_Group), ctypes.c_int, ctypes.POINTER(_HParams)]
    lib.muon_workspace_size.restype = ctypes.c_size_t
    lib.muon_workspace_min.argtypes = [ctypes.POINTER(_Group), ctypes.c_int, ctypes.POINTER(_HParams)]
    lib.muon_workspace_min.restype = ctypes.c_size_t
    lib.muon_step.argtypes = [ctypes.POINTER(_Group), ctypes.c_int, ctypes.POINTER(_HParams), P, ctypes.c_size_t,
                              P, P]
    lib.muon_step.restype = ctypes.c_int
    lib.muon_ns_workspace_size.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(_NSParams)]
    lib.muon_ns_workspace_size.restype = ctypes.c_size_t
    lib.muon_ns_batched.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                    ctypes.c_int, ctypes.POINTER(_NSParams), P, ctypes.c_size_t, P, P]
    lib.muon_ns_batched.restype = ctypes.c_int
    lib.muon_ns_flops.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(_NSParams)]
    lib.muon_ns_flops.restype = ctypes.c_double
    lib.muon_ns_batched_noalloc.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_int,
                                            ctypes.c_int, ctypes.c_int, ctypes.POINTER(_NSParams), P, P]
    lib.muon_ns_batched_noalloc.restype = ctypes.c_int
    for name in ("muon_blocks_workspace_size", "muon_blocks_workspace_min"):
        getattr(lib, name).argtypes = [ctypes.POINTER(_BlockGroup), ctypes.c_int, ctypes.POINTER(_HParams)]
        getattr(lib, name).restype = ctypes.c_size_t
    lib.muon_step_blocks.argtypes = [ctypes.POINTER(_BlockGroup), ctypes.c_int, ctypes.POINTER(_HParams), P,
                                     ctypes.c_size_t, P, P]
    I, L = ctypes.c_int, ctypes.c_longlong
    lib.muon_expert_sort_workspace_size.argtypes = [I, I, I]
    lib.muon_expert_sort_workspace_size.restype = ctypes.c_size_t
    lib.muon_expert_sort.argtypes = [P, I, L, I, I, I, P, P, P, P, ctypes.c_size_t, P]
    lib.muon_expert_gather.argtypes = [P, L, P, I, I, I, I, P, L, L, P]
    lib.muon_expert_combine.argtypes = [P, L, L, P, P, I, I, I, I, I, P, L, P]
    lib.muon_expert_combine_backward.argtypes = [P, L, P, L, L, P, P, I, I, I, I, I, P, L, P, P]
    S = ctypes.c_size_t
    lib.muon_expert_workspace_size.argtypes = [I, P, L, P, L, L, I, L, I, I, I]
    lib.muon_expert_workspace_size.restype = S
    lib.muon_expert_product.argtypes = [P, L, P, L, L, P, I, L, I, I, I, P, L, P, S, P, P]
    lib.muon_expert_input_grad.argtypes = [P, L, P, L, L, P, I, L, I, I, I, P, L, P, S, P, P]
    lib.muon_expert_weight_grad.argtypes = [P, L, P, L, P, I, L, I, I, I, P, L, L, I, I, P, S, P, P]
    for name in ("muon_step_blocks", "muon_expert_sort", "muon_expert_gather", "muon_expert_combine",
                 "muon_expert_combine_backward", "muon_expert_product", "muon_expert_input_grad",
                 "muon_expert_weight_grad"):
        getattr(lib, name).restype = ctypes.c_int
    lib.muon_profile_begin.argtypes = []
    lib.muon_profile_begin.restype = ctypes.c_int
    lib.muon_profile_end.argtypes = [ctypes.POINTER(_ProfEntry), ctypes.c_int]
    lib.muon_profile_end.restype = ctypes.c_int
    lib.muon_status_string.argtypes = [ctypes.c_int]
    lib.muon_status_string.restype = ctypes.c_char_p
    _LIB = lib
    return lib


# ---------------------------------------------------------------------------
# argument marshalling
# ---------------------------------------------------------------------------
def _dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return BF16
    if t == torch.float16:
        return FP16
    if t == torch.float32:
        return FP32
    raise MuonError(f"unsupported dtype {t}")


def _code(v, names) -> int:
    return names[v] if isinstance(v, str) else int(v)


def _ns_params(coeffs, mode, restart_after, eps, compute_dtype, gram_dtype, restart_every=0):
    flat = [float(x) for abc in coeffs for x in abc]
    arr = (ctypes.c_float * len(flat))(*flat)
    p = _NSParams(len(flat) // 3, ctypes.cast(arr, ctypes.POINTER(ctypes.c_float)), _code(mode, _MODE_NAMES),
                  int(restart_after), float(eps), _code(compute_dtype, _DT_NAMES), _code(gram_dtype, _DT_NAMES),
                  int(restart_every))
    return p, arr


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _elsewhere(device: torch.device, stream, call, *args, **kw):
    """call(*args, **kw) with ``device`` current and, if a stream is given, that
    stream current too, so that what the call allocates belongs to it."""
    with torch.cuda.device(device):
        if stream is None:
            return call(*args, **kw)
        if not hasattr(stream, "cuda_stream"):
            handle = int(stream)
            stream = torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)
        if stream.device != device:
            raise MuonError(f"the stream is on {stream.device}, the tensors on {device}")
        with torch.cuda.stream(stream):
            return call(*args, **kw)


def _here(device: torch.device, stream) -> bool:
    """Whether a call on ``device`` can go out as things are: no stream asked for, the device current."""
    return stream is None and device.index == torch.cuda.current_device()


def _check_workspace(ws: torch.Tensor, device: torch.device):
    if ws.device != device:
        raise MuonError(f"the workspace is on {ws.device}, the tensors on {device}")
    if not ws.is_contiguous():
        raise MuonError("the workspace must be contiguous")


def _check_cuda(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise MuonError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise MuonError(f"{name} must be contiguous (row-major)")
    if t.dim() != 2:
        raise MuonError(f"{name} must be 2-D")


def _raise(rc: int, what: str):
    if rc != 0:
        raise MuonError(f"{what} failed: {rc} ({muon_status_string(rc)})")


def _sides(*sizes):
    """Refuses matrix sizes that the C structs' ints cannot hold (ctypes would keep their low 32 bits)."""
    if max(sizes) >= 1 << 31:
        raise MuonError(f"matrices have fewer than 2^31 rows and columns, not {max(sizes)}")


def _build_groups(params, grads, moms):
    """Group tensors by (shape, W dtype, G dtype) in first-appearance order."""
    keys = []
    index = {}
    for i, (w, g, m) in enumerate(zip(params, grads, moms)):
        _check_cuda(w, "param"); _check_cuda(g, "grad"); _check_cuda(m, "momentum")
        if w.shape != g.shape or w.shape != m.shape:
            raise MuonError("param, grad and momentum shapes differ")
        if m.dtype != torch.float32:
            raise MuonError("momentum buffers must be float32")
        _sides(*w.shape)
        k = (tuple(w.shape), _dtype_code(w.dtype), _dtype_code(g.dtype))
        if k not in index:
            index[k] = len(keys)
            keys.append((k, []))
        keys[index[k]][1].append(i)
    groups = (_Group * len(keys))()
    keep = []
    order = []
    for gi, ((shape, wdt, gdt), idx) in enumerate(keys):
        n = len(idx)
        W = (ctypes.c_void_p * n)(*[params[i].data_ptr() for i in idx])
        G = (ctypes.c_void_p * n)(*[grads[i].data_ptr() for i in idx])
        M = (ctypes.c_void_p * n)(*[moms[i].data_ptr() for i in idx])
        keep += [W, G, M]
        groups[gi] = _Group(shape[0], shape[1], n, wdt, gdt, W, G, M)
        order += idx
    return groups, len(keys), keep, order


def _matrices(t: torch.Tensor):
    """Addresses of the matrices of (..., R, C), in order."""
    at, es = [t.data_ptr()], t.element_size()
    for n, stride in zip(t.shape[:-2], t.stride()[:-2]):
        at = [p + o for p in at for o in range(0, n * stride * es, stride * es)] if stride else at * n
    return at


def _pitch(t: torch.Tensor, name: str) -> int:
    """The row pitch (in elements) of a matrix, or of the matrices of (..., R, C)."""
    *_, rows, cols = t.shape
    *_, ld, one = t.stride()
    if one != 1 and cols > 1:
        raise MuonError(f"{name} must have contiguous rows")
    if rows <= 1:
        return cols
    if ld < cols:
        raise MuonError(f"{name} has overlapping rows")
    return ld


def _apart(t: torch.Tensor, name: str):
    """Refuses a tensor to be written whose rows share memory: a leading stride of zero, windows that overlap."""
    cols, lead = t.shape[-1], sorted((s, n) for s, n in zip(t.stride()[:-1], t.shape[:-1]) if n > 1)
    span = cols  # elements from the first to the last of the dimensions so far
    for stride, n in lead:
        if stride < span:
            break
        span += (n - 1) * stride
    else:
        return
    starts = torch.zeros(1, dtype=torch.int64, device="cpu")  # strides that interleave: the rows themselves
    for stride, n in lead:
        starts = (starts[:, None] + stride * torch.arange(n, device="cpu")).view(-1)
    if bool((starts.sort().values.diff() < cols).any()):
        raise MuonError(f"{name} overlaps itself")


def _build_block_groups(params, grads, moms, blocks):
    """Block groups in first-appearance order, and the index of every grouped
    block in the order of the parameters' blocks (matrices, block rows, block
    columns)."""
    if len(blocks) != len(params):
        raise MuonError("blocks must have one entry per parameter")
    index, total = {}, 0
    for w, g, m, block in zip(params, grads, moms, blocks):
        for t, name in ((w, "param"), (g, "grad"), (m, "momentum")):
            if not t.is_cuda:
                raise MuonError(f"{name} must be a CUDA tensor")
            if t.device != params[0].device:
                raise MuonError(f"{name} is on {t.device}, not on {params[0].device}")
            if t.dim() < 2 or t.numel() == 0:
                raise MuonError(f"{name} must have at least two dimensions and no empty one")
        if w.shape != g.shape or w.shape != m.shape:
            raise MuonError("param, grad and momentum shapes differ")
        if m.dtype != torch.float32:
            raise MuonError("momentum buffers must be float32")
        _apart(w, "param")
        _apart(m, "momentum")
        rows, cols = w.shape[-2:]
        _sides(rows, cols)
        r, c = (rows, cols) if block is None else (int(block[0]), int(block[1]))
        if r < 1 or c < 1 or rows % r or cols % c:
            raise MuonError(f"blocks of {r} x {c} do not tile a {rows} x {cols} matrix")
        k = (r, c, rows // r, cols // c, _dtype_code(w.dtype), _dtype_code(g.dtype), _pitch(w, "param"),
             _pitch(g, "grad"), _pitch(m, "momentum"))
        entry = index.setdefault(k, ([], [], [], []))
        for t, out in zip((w, g, m), entry):
            out.extend(_matrices(t))
        n = w.numel() // (r * c)
        entry[3].extend(range(total, total + n))
        total += n
    groups = (_BlockGroup * len(index))()
    keep, order = [], []
    for gi, (k, (*ptrs, idx)) in enumerate(index.items()):
        arrays = [(ctypes.c_void_p * len(p))(*p) for p in ptrs]
        keep += arrays
        groups[gi] = _BlockGroup(k[0], k[1], len(ptrs[0]), *k[2:], *arrays)
        order += idx
    return groups, len(index), keep, order


def _hparams(lr, momentum, weight_decay, scale_coef, nesterov, ns):
    return _HParams(float(lr), float(momentum), float(weight_decay), float(scale_coef), int(bool(nesterov)), ns)


# ---------------------------------------------------------------------------
# public API (same names as the C ABI)
# ---------------------------------------------------------------------------
def muon_status_string(code: int) -> str:
    return load_library().muon_status_string(int(code)).decode()


def muon_ns_flops(rows: int, cols: int, coeffs=(QUINTIC,) * 5, mode="standard", restart_after=2,
                  restart_every=0) -> float:
    ns, _arr = _ns_params(coeffs, mode, restart_after, 1e-7, BF16, FP16, restart_every)
    return load_library().muon_ns_flops(rows, cols, ctypes.byref(ns))


def _step_args(params, grads, moms, lr, momentum, nesterov, weight_decay, scale_coef, eps, coeffs, mode,
               restart_after, compute_dtype, gram_dtype, restart_every=0, blocks=None):
    if not (len(params) == len(grads) == len(moms)) or len(params) == 0:
        raise MuonError("params, grads and moms must be non-empty lists of equal length")
    if blocks is None:
        groups, ng, keep, order = _build_groups(params, grads, moms)
    else:
        groups, ng, keep, order = _build_block_groups(params, grads, moms, blocks)
    ns, arr = _ns_params(coeffs, mode, restart_after, eps, compute_dtype, gram_dtype, restart_every)
    hp = _hparams(lr, momentum, weight_decay, scale_coef, nesterov, ns)
    return groups, ng, hp, (keep, arr), order


_STEP_DEFAULTS = dict(lr=0.02, momentum=0.95, nesterov=True, weight_decay=0.1, scale_coef=0.2, eps=1e-7,
                      coeffs=(QUINTIC,) * 5, mode="standard", restart_after=2, compute_dtype="fp16",
                      gram_dtype="fp16", restart_every=0)


def muon_workspace_size(params, grads, moms, **hp) -> int:
    a = dict(_STEP_DEFAULTS, **hp)
    groups, ng, h, _keep, _ = _step_args(params, grads, moms, **a)
    return int(load_library().muon_workspace_size(groups, ng, ctypes.byref(h)))


def muon_workspace_min(params, grads, moms, **hp) -> int:
    a = dict(_STEP_DEFAULTS, **hp)
    groups, ng, h, _keep, _ = _step_args(params, grads, moms, **a)
    return int(load_library().muon_workspace_min(groups, ng, ctypes.byref(h)))


def muon_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], moms: Sequence[torch.Tensor], *,
              workspace: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None,
              **hp) -> torch.Tensor | None:
    """One Muon step, in place on ``params`` and ``moms``.

    Keyword hyper-parameters (defaults: lr 0.02, momentum 0.95, nesterov True,
    weight_decay 0.1, scale_coef 0.2, eps 1e-7, five quintic iterations,
    mode "standard", restart_after 2, restart_every 0, compute_dtype "fp16",
    gram_dtype "fp16").
    ``compute_dtype`` is the storage type of the chain between the products
    (W and G keep their own types): "fp16" stores X0 = U / (||U|| + eps) and
    every product in binary16, "bf16" stores the raw U and the products in
    bfloat16 (8 x coarser), "fp32" runs 3xTF32 products.
    ``workspace`` is a CUDA uint8 tensor (allocated when None); ``status``, if
    given, is an int32 CUDA tensor with one word per parameter (in the order of
    ``params``) and receives the MUON_STATUS_* bits.
    """
    lib = load_library()
    a = dict(_STEP_DEFAULTS, **hp)
    groups, ng, h, keep, order = _step_args(params, grads, moms, **a)
    need = int(lib.muon_workspace_size(groups, ng, ctypes.byref(h)))
    if need == 0:
        raise MuonError("invalid arguments (workspace query returned 0)")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=params[0].device)
    st_grouped = None
    if status is not None:
        st_grouped = torch.empty(len(order), dtype=torch.int32, device=params[0].device)
    rc = lib.muon_step(groups, ng, ctypes.byref(h), ctypes.c_void_p(workspace.data_ptr()),
                       ctypes.c_size_t(workspace.numel() * workspace.element_size()),
                       ctypes.c_void_p(st_grouped.data_ptr() if st_grouped is not None else 0),
                       ctypes.c_void_p(_stream_handle(stream)))
    _raise(rc, "muon_step")
    if status is not None:
        status[torch.tensor(order, device=status.device)] = st_grouped
    return status


def muon_blocks_workspace_size(params, grads, moms, blocks, **hp) -> int:
    groups, ng, h, _keep, _ = _step_args(params, grads, moms, blocks=blocks, **dict(_STEP_DEFAULTS, **hp))
    return int(load_library().muon_blocks_workspace_size(groups, ng, ctypes.byref(h)))


def muon_blocks_workspace_min(params, grads, moms, blocks, **hp) -> int:
    groups, ng, h, _keep, _ = _step_args(params, grads, moms, blocks=blocks, **dict(_STEP_DEFAULTS, **hp))
    return int(load_library().muon_blocks_workspace_min(groups, ng, ctypes.byref(h)))


def muon_step_blocks(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], moms: Sequence[torch.Tensor],
                     blocks: Sequence, *, workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                     stream=None, **hp) -> torch.Tensor | None:
    """One Muon step on the blocks of stacked, fused or strided weights, in
    place on ``params`` and ``moms``.

    A parameter is (..., R, C) with contiguous rows and any other strides (an
    expert stack, a fused gate and up, a slice of either; a gradient's matrices
    may be the same memory, those of parameters and momentum buffers must not
    overlap, in one tensor or between them); its entry in ``blocks`` is the (rows, cols) of the blocks that tile each of its
    matrices, or None for whole matrices.  Every block is orthogonalised on its
    own, as muon_step does a matrix: (head_dim, hidden) splits a query
    projection into heads, (hidden, head_dim) an output projection.  ``status``
    has one word per block, in the order of the parameters, their matrices,
    block rows and block columns.  Hyper-parameters as for muon_step.
    """
    lib = load_library()
    groups, ng, h, _keep, order = _step_args(params, grads, moms, blocks=blocks, **dict(_STEP_DEFAULTS, **hp))
    need = int(lib.muon_blocks_workspace_size(groups, ng, ctypes.byref(h)))
    if need == 0:
        raise MuonError("invalid arguments (workspace query returned 0)")
    device = params[0].device
    if status is not None and (status.dtype != torch.int32 or status.numel() != len(order) or
                               status.device != device or not status.is_contiguous()):
        raise MuonError(f"status must be a contiguous int32 tensor of {len(order)} words on the parameters' device")
    if workspace is not None:
        _check_workspace(workspace, device)
    if not _here(device, stream):
        return _elsewhere(device, stream, muon_step_blocks, params, grads, moms, blocks, workspace=workspace,
                          status=status, **hp)
    ws = torch.empty(need, dtype=torch.uint8, device=device) if workspace is None else workspace
    grouped = None if status is None else torch.empty(len(order), dtype=torch.int32, device=device)
    _raise(lib.muon_step_blocks(groups, ng, ctypes.byref(h), ws.data_ptr(), ws.numel() * ws.element_size(),
                                None if grouped is None else grouped.data_ptr(), _raw_stream(device.index)),
           "muon_step_blocks")
    if status is not None:
        # words in a row at a time: an index tensor would have to come from the host, which a capture forbids
        flat, at = status.view(-1), [k for k, o in enumerate(order) if k == 0 or o != order[k - 1] + 1] + [len(order)]
        torch._foreach_copy_([flat[order[a]:order[a] + b - a] for a, b in zip(at, at[1:])],
                             [grouped[a:b] for a, b in zip(at, at[1:])])
    return status


def muon_ns_workspace_size(count: int, rows: int, cols: int, coeffs=(QUINTIC,) * 5, mode="standard",
                           restart_after=2, eps=1e-7, compute_dtype="fp16", gram_dtype="fp16",
                           restart_every=0) -> int:
    ns, _arr = _ns_params(coeffs, mode, restart_after, eps, compute_dtype, gram_dtype, restart_every)
    return int(load_library().muon_ns_workspace_size(count, rows, cols, ctypes.byref(ns)))


def muon_ns_batched(X: Sequence[torch.Tensor], *, coeffs=(QUINTIC,) * 5, mode="standard", restart_after=2,
                    eps=1e-7, compute_dtype=None, gram_dtype="fp16", workspace: torch.Tensor | None = None,
                    status: torch.Tensor | None = None, stream=None, restart_every=0) -> None:
    """Orthogonalise same-shape matrices in place (result has each input's shape).

    ``compute_dtype`` is the storage type of the chain: None picks "fp32" for
    fp32 inputs and "fp16" otherwise; "bf16" is also accepted.  fp32 chains run
    3xTF32 tensor-core products when the short side is at least 256, and a
    single fused launch per call for matrices small enough for one block's
    shared memory.  ``gram_dtype`` is the 16-bit type of the Gram chains.
    ``status``, if given, is an int32 CUDA tensor with one word per matrix.
    ``restart_every`` > 0 repeats the stabilised form's restart every that many
    iterations after ``restart_after``.
    """
    lib = load_library()
    if len(X) == 0:
        return
    for t in X:
        _check_cuda(t, "X")
        if t.shape != X[0].shape or t.dtype != X[0].dtype:
            raise MuonError("all matrices must share shape and dtype")
    rows, cols = X[0].shape
    _sides(rows, cols)
    dt = _dtype_code(X[0].dtype)
    if compute_dtype is None:
        compute_dtype = "fp32" if dt == FP32 else "fp16"
    ns, arr = _ns_params(coeffs, mode, restart_after, eps, compute_dtype, gram_dtype, restart_every)
    need = int(lib.muon_ns_workspace_size(len(X), rows, cols, ctypes.byref(ns)))
    if need == 0:
        raise MuonError("invalid arguments (workspace query returned 0)")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=X[0].device)
    ptrs = (ctypes.c_void_p * len(X))(*[t.data_ptr() for t in X])
    rc = lib.muon_ns_batched(ptrs, len(X), rows, cols, dt, ctypes.byref(ns), ctypes.c_void_p(workspace.data_ptr()),
                             ctypes.c_size_t(workspace.numel() * workspace.element_size()),
                             ctypes.c_void_p(status.data_ptr() if status is not None else 0),
                             ctypes.c_void_p(_stream_handle(stream)))
    _raise(rc, "muon_ns_batched")


def muon_profile_begin() -> None:
    """Start bracketing every library launch with CUDA events (tracing aid)."""
    _raise(load_library().muon_profile_begin(), "muon_profile_begin")


def muon_profile_end() -> list[dict]:
    """Stop profiling; per kernel kind: launches, device ms, algorithmic FLOPs,
    executed FLOPs (whole tensor-core tiles, triangles only for symmetric
    products, three MMAs per 3xTF32 product) and algorithmic bytes."""
    rows = (_ProfEntry * 32)()
    n = load_library().muon_profile_end(rows, 32)
    if n < 0:
        _raise(n, "muon_profile_end")
    return [dict(kernel=r.kernel.decode(), launches=r.launches, ms=r.ms, flops=r.flops, exec_flops=r.exec_flops,
                 bytes=r.bytes) for r in rows[:n]]


class MuonStep:
    """A prepared Muon step over a fixed set of tensors.

    Builds the C structs (groups, hyper-parameters) and the workspace once, so
    each call is a single C-ABI call with no per-step marshalling.  The tensors
    must stay alive and keep their storage for the object's lifetime.  With
    ``blocks`` it is muon_step_blocks: one status word per block.
    """

    def __init__(self, params, grads, moms, *, workspace_bytes: int | None = None,
                 workspace: torch.Tensor | None = None, blocks: Sequence | None = None, **hp):
        self._lib = load_library()
        a = dict(_STEP_DEFAULTS, **hp)
        self.hp = a
        self._groups, self._ng, self._h, self._keep, self.order = _step_args(params, grads, moms, blocks=blocks, **a)
        kind = "muon" if blocks is None else "muon_blocks"
        self._name = "muon_step" if blocks is None else "muon_step_blocks"
        self._step = getattr(self._lib, self._name)
        full = int(getattr(self._lib, kind + "_workspace_size")(self._groups, self._ng, ctypes.byref(self._h)))
        lo = int(getattr(self._lib, kind + "_workspace_min")(self._groups, self._ng, ctypes.byref(self._h)))
        if full == 0:
            raise MuonError("invalid arguments (workspace query returned 0)")
        self.workspace_needed = (lo, full)
        if workspace is not None:
            _check_workspace(workspace, params[0].device)
            if workspace.numel() * workspace.element_size() < lo:
                raise MuonError(f"workspace of {workspace.numel()} bytes is below the minimum {lo}")
            self.workspace = workspace
        else:
            size = full if workspace_bytes is None else max(lo, min(full, int(workspace_bytes)))
            self.workspace = torch.empty(size, dtype=torch.uint8, device=params[0].device)
        self.status = torch.zeros(len(self.order), dtype=torch.int32, device=params[0].device)
        self.count = len(self.order)

    def __call__(self, stream=None) -> None:
        if not _here(self.workspace.device, None):  # the tensors' device, not the current one
            return _elsewhere(self.workspace.device, stream, self)
        rc = self._step(self._groups, self._ng, ctypes.byref(self._h), ctypes.c_void_p(self.workspace.data_ptr()),
                        ctypes.c_size_t(self.workspace.nbytes), ctypes.c_void_p(self.status.data_ptr()),
                        ctypes.c_void_p(_stream_handle(stream)))
        _raise(rc, self._name)

    def capture(self, stream=None) -> "torch.cuda.CUDAGraph":
        """Record one step into a CUDA graph and return it; ``graph.replay()``
        then runs the whole launch chain with one launch call.  The step is run
        once eagerly first (one-time kernel set-up happens outside the capture),
        so each capture advances the optimizer state by one step.  Inputs are
        read from the same tensors at replay: update G in place between replays."""
        side = torch.cuda.Stream(device=self.workspace.device) if stream is None else stream
        side.wait_stream(torch.cuda.current_stream(self.workspace.device))
        with torch.cuda.stream(side):
            self(stream=side)
        torch.cuda.current_stream(self.workspace.device).wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            self(stream=side)
        return g

    def status_in_param_order(self) -> torch.Tensor:
        out = torch.empty_like(self.status)
        out[torch.tensor(self.order, device=out.device)] = self.status
        return out


def muon_ns_batched_noalloc(X: Sequence[torch.Tensor], *, coeffs=(QUINTIC,) * 5, mode="standard", restart_after=2,
                            eps=1e-7, compute_dtype=None, gram_dtype="fp16", status: torch.Tensor | None = None,
                            stream=None, restart_every=0) -> None:
    """muon_ns_batched with the library's fixed device scratch instead of a
    workspace: for callers that cannot allocate device memory at this point
    (their allocator owns the GPU, or allocation is forbidden after start-up).
    Matrices whose one-matrix workspace exceeds NOALLOC_SCRATCH_BYTES are
    rejected.  Calls share the scratch: do not let two of them overlap on the
    GPU.  The first call on a device must come before any stream capture."""
    lib = load_library()
    if len(X) == 0:
        return
    for t in X:
        _check_cuda(t, "X")
        if t.shape != X[0].shape or t.dtype != X[0].dtype:
            raise MuonError("all matrices must share shape and dtype")
    rows, cols = X[0].shape
    _sides(rows, cols)
    dt = _dtype_code(X[0].dtype)
    if compute_dtype is None:
        compute_dtype = "fp32" if dt == FP32 else "fp16"
    ns, arr = _ns_params(coeffs, mode, restart_after, eps, compute_dtype, gram_dtype, restart_every)
    ptrs = (ctypes.c_void_p * len(X))(*[t.data_ptr() for t in X])
    rc = lib.muon_ns_batched_noalloc(ptrs, len(X), rows, cols, dt, ctypes.byref(ns),
                                     ctypes.c_void_p(status.data_ptr() if status is not None else 0),
                                     ctypes.c_void_p(_stream_handle(stream)))
    _raise(rc, "muon_ns_batched_noalloc")


def plan_slices(shapes, nbytes, slice_bytes):
    """Slices of the streamed step: lists of tensor indices, at most
    ``slice_bytes`` each (a larger tensor gets a slice of its own), taken in
    order of decreasing short side (ties by index), so that the slices with
    the most orthogonalisation work per byte come first."""
    order = sorted(range(len(shapes)), key=lambda i: (-min(shapes[i][-2:]), i))
    slices, cur, acc = [], [], 0
    for i in order:
        if cur and acc + nbytes[i] > slice_bytes:
            slices.append(cur)
            cur, acc = [], 0
        cur.append(i)
        acc += nbytes[i]
    if cur:
        slices.append(cur)
    return slices


class StreamedMuonStep:
    """A Muon step fed from and returned to pinned host memory, with the PCIe
    copies overlapped with the orthogonalisation.

    The parameters are cut into slices (at most ``slice_bytes`` of gradients
    each), taken in order of decreasing short side: the orthogonalisation's
    work per byte grows with it, so the first slices give the next slices'
    copies the most compute to hide behind, and the last slices, whose
    copies cannot be hidden, are the cheapest.  Per slice, one stream copies the
    gradients host -> device, the compute stream runs the fused step on the
    slice, and a third stream copies the updated weights device -> host, so
    slice k's step runs while slice k+1's gradients arrive and slice k-1's
    weights leave.  Every slice shares one workspace (the steps are serialised
    on the compute stream).  Across calls, a slice's gradient buffer is not
    overwritten before the previous step has read it, nor its weights updated
    before the previous copy-out has read them.  The caller's current stream
    waits for the whole step at the end of each call.
    """

    def __init__(self, params, grads, moms, host_grads, host_params, *, slice_bytes: int = 512 << 20,
                 workspace_bytes: int | None = None, **hp):
        if not (len(params) == len(grads) == len(moms) == len(host_grads) == len(host_params)):
            raise MuonError("params, grads, moms and their host copies must have equal lengths")
        for h in list(host_grads) + list(host_params):
            if h.is_cuda or not h.is_pinned():
                raise MuonError("host buffers must be pinned CPU tensors")
        dev = params[0].device
        self.params, self.grads = list(params), list(grads)
        self.host_grads, self.host_params = list(host_grads), list(host_params)
        self.slices = plan_slices([tuple(g.shape) for g in self.grads],
                                  [g.numel() * g.element_size() for g in self.grads], slice_bytes)
        self.steps = [MuonStep([self.params[i] for i in idx], [self.grads[i] for i in idx],
                               [moms[i] for i in idx], workspace=None, workspace_bytes=1, **hp)
                      for idx in self.slices]
        need = max(st.workspace_needed[1] for st in self.steps)
        if workspace_bytes is not None:
            need = max(max(st.workspace_needed[0] for st in self.steps), min(need, int(workspace_bytes)))
        self.workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        for st in self.steps:
            st.workspace = self.workspace
        self.h2d = torch.cuda.Stream(device=dev)
        self.compute = torch.cuda.Stream(device=dev)
        self.d2h = torch.cuda.Stream(device=dev)
        n = len(self.slices)
        self._computed = [None] * n   # event: slice's step finished (its gradients are read)
        self._copied_out = [None] * n  # event: slice's weights are on the host

    def __call__(self) -> None:
        caller = torch.cuda.current_stream(self.workspace.device)
        for s in (self.h2d, self.compute, self.d2h):
            s.wait_stream(caller)
        done = []
        for k, idx in enumerate(self.slices):
            with torch.cuda.stream(self.h2d):
                if self._computed[k] is not None:
                    self.h2d.wait_event(self._computed[k])
                for i in idx:
                    self.grads[i].copy_(self.host_grads[i], non_blocking=True)
                arrived = torch.cuda.Event()
                arrived.record(self.h2d)
            self.compute.wait_event(arrived)
            if self._copied_out[k] is not None:
                self.compute.wait_event(self._copied_out[k])
            self.steps[k](stream=self.compute)
            ev = torch.cuda.Event()
            ev.record(self.compute)
            self._computed[k] = ev
            with torch.cuda.stream(self.d2h):
                self.d2h.wait_event(ev)
                for i in idx:
                    self.host_params[i].copy_(self.params[i], non_blocking=True)
                out = torch.cuda.Event()
                out.record(self.d2h)
            self._copied_out[k] = out
            done.append(out)
        for ev in done:
            caller.wait_event(ev)

    @property
    def status(self) -> torch.Tensor:
        return torch.cat([st.status_in_param_order() for st in self.steps])


# ---------------------------------------------------------------------------
# expert layers
# ---------------------------------------------------------------------------
_CODES = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}


def _matrix(t: torch.Tensor, name: str, device: torch.device, dtype: torch.dtype, rows: int, cols: int) -> int:
    """Checks a rows x cols matrix with contiguous rows; returns its row pitch."""
    if t.device != device or t.dtype != dtype or t.shape != (rows, cols):
        raise MuonError(f"{name} must be {dtype} ({rows}, {cols}) on {device}, not {t.dtype} {tuple(t.shape)} on {t.device}")
    return _pitch(t, name)


def _lead(t: torch.Tensor, name: str):
    """Checks a call's first matrix: (device, dtype, its code, rows, columns, row pitch)."""
    if not t.is_cuda or t.dim() != 2:
        raise MuonError(f"{name} must be a 2-D CUDA tensor")
    dtype, (rows, cols) = t.dtype, t.shape
    if dtype not in _CODES:
        raise MuonError(f"unsupported dtype {dtype}")
    if rows > _EXPERT_MOST or cols > _EXPERT_MOST:
        raise MuonError(f"{name} has more than 2^30 rows or columns: {rows} x {cols}")
    return t.device, dtype, _CODES[dtype], rows, cols, _pitch(t, name)


def _slot_arg(slot: torch.Tensor, device: torch.device):
    if slot.dtype != torch.int32 or slot.dim() != 2 or not slot.is_contiguous() or slot.device != device:
        raise MuonError(f"slot must be a contiguous 2-D int32 tensor on {device}")
    tokens, topk = slot.shape
    if topk < 1:
        raise MuonError("slot must have at least one column")
    if tokens * topk > _EXPERT_MOST:
        raise MuonError(f"slot has more than 2^30 entries: {tokens} x {topk}")
    return tokens, topk


def _weights_arg(weights: torch.Tensor, slot: torch.Tensor) -> int:
    if weights.device != slot.device or not weights.is_contiguous() or weights.shape != slot.shape:
        raise MuonError(f"weights must be contiguous {tuple(slot.shape)} on the slots' device")
    return _dtype_code(weights.dtype)


def muon_expert_sort(ids: torch.Tensor, experts: int, *, workspace: torch.Tensor | None = None, stream=None):
    """Sort the tokens' assignments by expert: (offsets, slot, source).

    ``ids`` is (tokens, topk) int32 or int64, as a router's topk gives it; an id
    outside [0, experts) goes to no expert (padding, or an expert on another
    GPU).  ``offsets`` (experts + 1): expert e owns the sorted rows
    [offsets[e], offsets[e + 1]).  ``slot`` (tokens, topk): the sorted row of an
    assignment, -1 where no expert takes it.  ``source`` (tokens * topk): the
    assignment (token * topk + j) of every sorted row, followed by those that
    no expert takes.  All int32, parts of one allocation; the sort is stable.
    """
    if not ids.is_cuda or ids.dim() != 2 or ids.dtype not in (torch.int32, torch.int64):
        raise MuonError("ids must be a 2-D int32 or int64 CUDA tensor")
    device = ids.device
    lib = load_library()
    tokens, topk = ids.shape
    need = 0
    if tokens * topk <= _EXPERT_MOST and topk <= _EXPERT_MOST and 0 < experts <= EXPERT_MAX:
        need = lib.muon_expert_sort_workspace_size(tokens, topk, experts)
    if need == 0:
        raise MuonError(f"cannot sort {tokens} x {topk} assignments to {experts} experts (workspace query returned 0)")
    ld, n, es = _pitch(ids, "ids"), tokens * topk, ids.element_size()
    if workspace is not None:
        _check_workspace(workspace, device)
    if not _here(device, stream):
        return _elsewhere(device, stream, muon_expert_sort, ids, experts, workspace=workspace)
    out = torch.empty(experts + 1 + 2 * n, dtype=torch.int32, device=device)
    offsets, slot, source = out.split_with_sizes((experts + 1, n, n))
    ws, ws_bytes = workspace, 0
    if ws is None and need > 256:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    if ws is not None:
        ws, ws_bytes = ws.data_ptr(), ws.numel() * ws.element_size()
    base = out.data_ptr()
    _raise(lib.muon_expert_sort(ids.data_ptr(), es, ld, tokens, topk, experts, base, base + 4 * (experts + 1),
                                base + 4 * (experts + 1 + n), ws, ws_bytes, _raw_stream(device.index)), "muon_expert_sort")
    return offsets, slot.view(tokens, topk), source


def muon_expert_gather(x: torch.Tensor, slot: torch.Tensor, *, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Lay the tokens' rows out by expert: out[slot[t, j]] = x[t].

    ``x`` is (tokens, cols), ``slot`` as from muon_expert_sort.  ``out`` (rows,
    cols) defaults to a new tensor of one row per assignment; rows that no slot
    names keep their contents, and slots outside it are skipped.
    """
    device, dtype, code, tokens, cols, ld = _lead(x, "x")
    topk = _slot_arg(slot, device)[1]
    if slot.shape[0] != tokens:
        raise MuonError(f"slot must have {tokens} rows, not {slot.shape[0]}")
    ld_out = cols if out is None else _matrix(out, "out", device, dtype, out.shape[0], cols)
    if not _here(device, stream):
        return _elsewhere(device, stream, muon_expert_gather, x, slot, out=out)
    if out is None:
        out = torch.empty(tokens * topk, cols, dtype=dtype, device=device)
    _raise(load_library().muon_expert_gather(x.data_ptr(), ld, slot.data_ptr(), tokens, topk, cols, code, out.data_ptr(),
                                             ld_out, out.shape[0], _raw_stream(device.index)), "muon_expert_gather")
    return out


def muon_expert_combine(ys: torch.Tensor, slot: torch.Tensor, weights: torch.Tensor | None = None, *,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Bring sorted rows back to their tokens: out[t] = sum_j weights[t, j] * ys[slot[t, j]].

    ``weights`` is (tokens, topk) of any supported type (None: ones).  An
    assignment that no expert takes adds nothing, whatever its weight.
    """
    device, dtype, code, rows, cols, ld = _lead(ys, "ys")
    tokens, topk = _slot_arg(slot, device)
    w, wdt = (None, 0) if weights is None else (weights.data_ptr(), _weights_arg(weights, slot))
    ld_out = cols if out is None else _matrix(out, "out", device, dtype, tokens, cols)
    if not _here(device, stream):
        return _elsewhere(device, stream, muon_expert_combine, ys, slot, weights, out=out)
    if out is None:
        out = torch.empty(tokens, cols, dtype=dtype, device=device)
    _raise(load_library().muon_expert_combine(ys.data_ptr(), ld, rows, slot.data_ptr(), w, wdt, tokens, topk, cols, code,
                                              out.data_ptr(), ld_out, _raw_stream(device.index)), "muon_expert_combine")
    return out


def muon_expert_gather_backward(dxs: torch.Tensor, slot: torch.Tensor, *, out: torch.Tensor | None = None,
                                stream=None) -> torch.Tensor:
    """The gradient of muon_expert_gather: out[t] = sum_j dxs[slot[t, j]]."""
    return muon_expert_combine(dxs, slot, None, out=out, stream=stream)


def muon_expert_combine_backward(dy: torch.Tensor, ys: torch.Tensor, slot: torch.Tensor,
                                 weights: torch.Tensor | None = None, *, out: torch.Tensor | None = None, stream=None):
    """The gradients of muon_expert_combine, (dys, dweights):
    dys[slot[t, j]] = weights[t, j] * dy[t] and dweights[t, j] = <dy[t], ys[slot[t, j]]>.

    ``out`` takes dys (a new tensor of ys's shape if None; rows that no slot
    names keep their contents).  dweights has the weights' type, zero where no
    expert takes the assignment; None if ``weights`` is None.
    """
    device, dtype, code, rows, cols, ld_ys = _lead(ys, "ys")
    tokens, topk = _slot_arg(slot, device)
    ld_dy = _matrix(dy, "dy", device, dtype, tokens, cols)
    w, wdt, dw, dwp = None, 0, None, None
    if weights is not None:
        w, wdt = weights.data_ptr(), _weights_arg(weights, slot)
    ld_out = cols if out is None else _matrix(out, "out", device, dtype, rows, cols)
    if not _here(device, stream):
        return _elsewhere(device, stream, muon_expert_combine_backward, dy, ys, slot, weights, out=out)
    if out is None:
        out = torch.empty(rows, cols, dtype=dtype, device=device)
    if weights is not None:
        dw = torch.empty_like(weights)
        dwp = dw.data_ptr()
    _raise(load_library().muon_expert_combine_backward(
        dy.data_ptr(), ld_dy, ys.data_ptr(), ld_ys, rows, slot.data_ptr(), w, wdt, tokens, topk, cols, code,
        out.data_ptr(), ld_out, dwp, _raw_stream(device.index)), "muon_expert_combine_backward")
    return out, dw


def _offsets_arg(offsets: torch.Tensor, device: torch.device) -> int:
    if offsets.device != device or offsets.dtype != torch.int32 or offsets.dim() != 1 or \
            not offsets.is_contiguous() or not 2 <= offsets.shape[0] <= EXPERT_MAX + 1:
        raise MuonError(f"offsets must be a contiguous int32 tensor of experts + 1 entries on the rows' device, for at "
                        f"most {EXPERT_MAX} experts")
    return offsets.shape[0] - 1


def _stack_arg(w: torch.Tensor, name: str, experts: int, device: torch.device, dtype: torch.dtype):
    """(outer, inner, row pitch, expert stride) of an (experts, outer, inner) stack."""
    if w.device != device or w.dtype != dtype or w.dim() != 3 or w.shape[0] != experts:
        raise MuonError(f"{name} must be {dtype} ({experts}, outer, inner) on {device}, not {w.dtype} {tuple(w.shape)} "
                        f"on {w.device}")
    _, outer, inner = w.shape
    if outer > _EXPERT_MOST or inner > _EXPERT_MOST:
        raise MuonError(f"{name} has more than 2^30 rows or columns an expert: {outer} x {inner}")
    return outer, inner, _pitch(w, name), w.stride(0) if experts > 1 else outer * inner


def _status_arg(status, device: torch.device):
    if status is None:
        return None
    if status.device != device or status.dtype != torch.int32 or status.numel() != 1:
        raise MuonError("status must be one int32 word on the rows' device")
    return status.data_ptr()


def _pack_space(kind: int, a, ld_a: int, b, ld_b: int, stride_b: int, experts: int, rows: int, inner: int, outer: int,
                code: int):
    """The workspace in which a product copies operands that TMA cannot address (None: it needs none)."""
    if code == FP32 or not ((a.data_ptr() | b.data_ptr()) | ((ld_a | ld_b | stride_b) << 1)) & 15 and (
            stride_b or kind == 2 or experts == 1):
        return None
    need = load_library().muon_expert_workspace_size(kind, a.data_ptr(), ld_a, b.data_ptr(), ld_b, stride_b, experts, rows,
                                                     inner, outer, code)
    return torch.empty(need, dtype=torch.uint8, device=a.device) if need else None


def muon_expert_product(xs: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *, out: torch.Tensor | None = None,
                        status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Every expert's rows times its weights: out[p] = w[e] @ xs[p] for the rows
    p of expert e, offsets[e] <= p < offsets[e + 1].

    ``xs`` is (rows, inner), ``w`` (experts, outer, inner) of the same type, both
    with contiguous rows and any other strides; ``offsets`` as from
    muon_expert_sort, read on the device.  Rows of ``out`` (rows, outer) that no
    expert owns keep their contents.  bf16 and fp16 run on the tensor cores
    (operands whose bases and strides are no multiples of 16 bytes after a copy
    into rows that are; small ones of that kind on the CUDA cores), fp32 on the
    CUDA cores.  ``status``: one int32 word, MUON_STATUS_TIMEOUT (2) where a
    device-side wait gave up and rows stayed unwritten; without it nothing
    reports that.
    """
    device, dtype, code, rows, width, ld = _lead(xs, "xs")
    experts = _offsets_arg(offsets, device)
    outer, inner, ld_w, stride_w = _stack_arg(w, "w", experts, device, dtype)
    if width != inner:
        raise MuonError(f"xs must have {inner} columns, not {width}")
    word = _status_arg(status, device)
    ld_out = outer if out is None else _matrix(out, "out", device, dtype, rows, outer)
    if not _here(device, stream):
        return _elsewhere(device, stream, muon_expert_product, xs, w, offsets, out=out, status=status)
    if out is None:
        out = torch.empty(rows, outer, dtype=dtype, device=device)
    ws = _pack_space(0, xs, ld, w, ld_w, stride_w, experts, rows, inner, outer, code)
    _raise(load_library().muon_expert_product(
        xs.data_ptr(), ld, w.data_ptr(), ld_w, stride_w, offsets.data_ptr(), experts, rows, inner, outer, code,
        out.data_ptr(), ld_out, None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), word, _raw_stream(device.index)), "muon_expert_product")
    return out


def muon_expert_input_grad(dys: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *,
                           out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                           stream=None) -> torch.Tensor:
    """The input gradient of muon_expert_product: out[p] = w[e]^T @ dys[p] for expert e's rows p."""
    device, dtype, code, rows, width, ld = _lead(dys, "dys")
    experts = _offsets_arg(offsets, device)
    outer, inner, ld_w, stride_w = _stack_arg(w, "w", experts, device, dtype)
    if width != outer:
        raise MuonError(f"dys must have {outer} columns, not {width}")
    word = _status_arg(status, device)
    ld_out = inner if out is None else _matrix(out, "out", device, dtype, rows, inner)
    if not _here(device, stream):
        return _elsewhere(device, stream, muon_expert_input_grad, dys, w, offsets, out=out, status=status)
    if out is None:
        out = torch.empty(rows, inner, dtype=dtype, device=device)
    ws = _pack_space(1, dys, ld, w, ld_w, stride_w, experts, rows, inner, outer, code)
    _raise(load_library().muon_expert_input_grad(
        dys.data_ptr(), ld, w.data_ptr(), ld_w, stride_w, offsets.data_ptr(), experts, rows, inner, outer, code,
        out.data_ptr(), ld_out, None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), word, _raw_stream(device.index)), "muon_expert_input_grad")
    return out


def muon_expert_weight_grad(dys: torch.Tensor, xs: torch.Tensor, offsets: torch.Tensor, *,
                            out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                            accumulate: bool = False, status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The weight gradients of muon_expert_product, (experts, outer, inner):
    dW[e] = sum of dys[p]^T xs[p] over expert e's rows, zero without rows.

    ``out_dtype`` (or ``out``'s type) is the operands' or float32; the stack's
    matrices are gradients as muon_step and muon_step_blocks take them.
    ``accumulate`` adds to a float32 ``out`` (gradient accumulation).
    """
    device, dtype, code, rows, outer, ld_dys = _lead(dys, "dys")
    if xs.dim() != 2 or xs.shape[1] > _EXPERT_MOST:
        raise MuonError(f"xs must be a matrix of at most 2^30 columns, not {tuple(xs.shape)}")
    inner = xs.shape[1]
    ld_xs = _matrix(xs, "xs", device, dtype, rows, inner)
    experts = _offsets_arg(offsets, device)
    word = _status_arg(status, device)
    if out is None:
        if accumulate:
            raise MuonError("accumulate needs out")
        out_dtype = out_dtype or dtype
        odt = _dtype_code(out_dtype)
        ld_out, stride_out = inner, outer * inner
    else:
        if out_dtype not in (None, out.dtype):
            raise MuonError(f"out is {out.dtype}, out_dtype {out_dtype}")
        odt = _dtype_code(out.dtype)
        if out.shape != (experts, outer, inner):
            raise MuonError(f"out must be {(experts, outer, inner)}, not {tuple(out.shape)}")
        _, _, ld_out, stride_out = _stack_arg(out, "out", experts, device, out.dtype)
        _apart(out, "out")
    if not _here(device, stream):
        return _elsewhere(device, stream, muon_expert_weight_grad, dys, xs, offsets, out=out, out_dtype=out_dtype,
                          accumulate=accumulate, status=status)
    if out is None:
        out = torch.empty(experts, outer, inner, dtype=out_dtype, device=device)
    ws = _pack_space(2, dys, ld_dys, xs, ld_xs, 0, experts, rows, inner, outer, code)
    _raise(load_library().muon_expert_weight_grad(
        dys.data_ptr(), ld_dys, xs.data_ptr(), ld_xs, offsets.data_ptr(), experts, rows, inner, outer, code,
        out.data_ptr(), ld_out, stride_out, odt, int(accumulate), None if ws is None else ws.data_ptr(),
        0 if ws is None else ws.numel(), word,
        _raw_stream(device.index)), "muon_expert_weight_grad")
    return out


class ExpertMuonStep:
    """A Muon step of expert stacks straight from the sorted tokens, without
    holding all of their gradients.

    ``params`` and ``moms`` are lists of (experts, outer, inner) stacks; a call
    takes, per stack, the (dys, xs, offsets) of its product's backward pass.  The
    experts are taken in slices whose gradients fit ``slice_bytes``: the slice's
    weight gradients go into one buffer that all slices share, and the block
    step on the slice consumes them, so a call needs that buffer and one
    workspace instead of a gradient per parameter.  The result is that of
    muon_expert_weight_grad followed by muon_step_blocks.  ``grad_dtype``: the
    buffer's type, the operands' (default: each stack's own) or float32.
    ``blocks`` as for muon_step_blocks, one entry per stack.  Calls share the
    buffer and the workspace and must not overlap on the GPU.

    A slice whose weight gradients hit a device-side timeout has stepped on an
    unfinished buffer: all of its blocks carry MUON_STATUS_TIMEOUT in ``status``,
    and their weights and momentum are to be restored from before the call.
    """

    def __init__(self, params, moms, *, blocks: Sequence | None = None, slice_bytes: int = 512 << 20,
                 grad_dtype: torch.dtype | None = None, **hp):
        if len(params) == 0 or len(params) != len(moms):
            raise MuonError("params and moms must be non-empty lists of equal length")
        blocks = [None] * len(params) if blocks is None else list(blocks)
        if len(blocks) != len(params):
            raise MuonError("blocks must have one entry per parameter")
        for w in params:
            if not w.is_cuda or w.dim() != 3 or w.device != params[0].device or w.numel() == 0:
                raise MuonError("params must be (experts, outer, inner) stacks on one device, none of them empty")
        for w, m in zip(params, moms):  # the slices are checked one by one below
            if w.shape != m.shape:
                raise MuonError("param and momentum shapes differ")
            _apart(w, "param")
            _apart(m, "momentum")
        self.device = params[0].device
        self.shapes = [tuple(w.shape) for w in params]
        dtypes = self.dtypes = [grad_dtype or w.dtype for w in params]
        self.slices = []  # (stack, first expert, last expert)
        most = 0
        for i, w in enumerate(params):
            one = w.shape[1] * w.shape[2] * dtypes[i].itemsize
            per = max(1, min(w.shape[0], slice_bytes // one))
            self.slices += [(i, e, min(e + per, w.shape[0])) for e in range(0, w.shape[0], per)]
            most = max(most, per * one)
        self._buffer = torch.empty(most, dtype=torch.uint8, device=self.device)
        self.grads, self.steps = [], []
        for i, e0, e1 in self.slices:
            shape = (e1 - e0,) + self.shapes[i][1:]
            n = shape[0] * shape[1] * shape[2] * dtypes[i].itemsize
            self.grads.append(self._buffer[:n].view(dtypes[i]).view(shape))
            self.steps.append(MuonStep([params[i][e0:e1]], [self.grads[-1]], [moms[i][e0:e1]], blocks=[blocks[i]],
                                       workspace_bytes=1, **hp))
        self.workspace = torch.empty(max(s.workspace_needed[1] for s in self.steps), dtype=torch.uint8,
                                     device=self.device)
        for step in self.steps:
            step.workspace = self.workspace
        # the status word of each slice's weight gradients
        self.words = torch.zeros(len(self.slices), dtype=torch.int32, device=self.device).split(1)

    def __call__(self, factors, stream=None) -> None:
        if len(factors) != len(self.shapes):
            raise MuonError("factors must have one (dys, xs, offsets) per stack")
        # everything is checked before the first slice steps
        for i, ((experts, outer, inner), (dys, xs, offsets)) in enumerate(zip(self.shapes, factors)):
            device, dtype, _, rows, cols, _ = _lead(dys, f"dys {i}")
            if device != self.device or cols != outer:
                raise MuonError(f"dys {i} must have {outer} columns on {self.device}")
            _matrix(xs, f"xs {i}", device, dtype, rows, inner)
            if _offsets_arg(offsets, device) != experts:
                raise MuonError(f"offsets {i} must have {experts + 1} entries")
            if self.dtypes[i] not in (dtype, torch.float32):
                raise MuonError(f"gradients {i} are held in {self.dtypes[i]}, dys is {dtype}")

        if not _here(self.device, stream):
            return _elsewhere(self.device, stream, self, factors)
        handle = _raw_stream(self.device.index)
        for (i, e0, e1), grad, word, step in zip(self.slices, self.grads, self.words, self.steps):
            dys, xs, offsets = factors[i]
            muon_expert_weight_grad(dys, xs, offsets[e0:e1 + 1], out=grad, status=word)
            step(stream=handle)

    @property
    def status(self) -> torch.Tensor:
        """The blocks' status words, each with its slice's weight gradients' word, in the order of the stacks,
        their experts and blocks."""
        return torch.cat([s.status_in_param_order() | word for s, word in zip(self.steps, self.words)])
