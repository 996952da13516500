"""Plain 64-bit versions of the expert-layer operators, and the error that a
right kernel may have against them.

A store to a type with unit eps is off by at most half a step, eps / 2 relative
to the value (and half the smallest subnormal below the normal range).  A sum
of n products in fp32 is off by at most n * u * sum |a_k b_k|, with u = 2^-24
where every addition rounds to nearest and u = 2^-23 where it may truncate (the
tensor cores).
"""
import torch

U_NEAREST, U_TRUNCATED = 2.0 ** -24, 2.0 ** -23
SUBNORMAL = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def f64(t):
    return t.detach().cpu().double()


def sort_ref(ids, experts):
    """(offsets, slot, source) by a plain loop."""
    flat = ids.cpu().reshape(-1).tolist()
    lists = [[] for _ in range(experts + 1)]
    for a, e in enumerate(flat):
        lists[e if 0 <= e < experts else experts].append(a)
    offsets, slot, source = [0], [-1] * len(flat), []
    for e in range(experts):
        for a in lists[e]:
            slot[a] = len(source)
            source.append(a)
        offsets.append(len(source))
    source += lists[experts]
    return (torch.tensor(offsets, dtype=torch.int32), torch.tensor(slot, dtype=torch.int32).view(ids.shape),
            torch.tensor(source, dtype=torch.int32))


def rows_ref(rows, slot):
    """(tokens, topk, cols) of the assignments' rows in 64 bits, zeros where there is none."""
    slot = slot.cpu().long()
    on = (slot >= 0) & (slot < rows.shape[0])
    picked = f64(rows)[slot.clamp(0, max(rows.shape[0] - 1, 0))] if rows.shape[0] else torch.zeros(
        *slot.shape, rows.shape[1], dtype=torch.float64)
    return torch.where(on[..., None], picked, 0.0), on


def segments(offsets, rows):
    ends = offsets.cpu().tolist()
    out = []
    for lo, hi in zip(ends[:-1], ends[1:]):
        lo = min(max(lo, 0), rows)
        out.append((lo, min(max(hi, lo), rows)))
    return out


def close(got, ref, terms, magnitude, u, what=""):
    """got within half a step of its type plus an fp32 sum's error of `terms` additions over `magnitude` = sum |a b|."""
    got, dt = f64(got), got.dtype
    bound = torch.finfo(dt).eps / 2 * (ref.abs() + terms * u * magnitude) + terms * u * magnitude + SUBNORMAL[dt]
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((got - ref).abs().max()), float(bound.max()),
                           torch.nonzero(bad)[:4].tolist())
