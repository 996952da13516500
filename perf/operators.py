"""Workloads of the expert-layer operators and of the Muon step on blocks.

Training an expert layer with Muon runs through these operators: the
assignments of tokens to experts are sorted (`sort`), the tokens' rows are laid
out by expert (`gather`), every expert multiplies its rows by its weights
(`product`, with both gradients), the results go back to their tokens with the
router's weights (`combine`, with both gradients), and the Muon step
orthogonalises the experts' stacked and fused weights block by block (`step`).

`own` False computes them with elementary torch operations in 32 bits, True
with this package's operators.
"""
import math

import torch

own = False

QUINTIC = (3.4445, -4.7750, 2.0315)
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MOST = 132_000 * 7168  # elements of the largest gathered matrix


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of a 32-sequence batch, routed to 8 of 216 experts: nothing but latency
        {"name": "sort decode", "op": "sort", "tokens": 32, "topk": 8, "experts": 216, "ids": "int64", "dropped": 0.0},
        # a training batch of 131072 tokens over 64 experts, a twentieth of them padding that goes to no expert
        {"name": "sort train", "op": "sort", "tokens": 131072, "topk": 8, "experts": 64, "ids": "int64", "dropped": 0.05},
        # a short ragged batch with an odd width: rows that start on no 16-byte boundary
        {"name": "gather odd", "op": "gather", "tokens": 777, "topk": 3, "experts": 13, "cols": 1001, "type": "fp32", "dropped": 0.2},
        # the Kimi-K2 width: 16384 tokens to 8 experts each, and the tokens' gradient back
        {"name": "gather K2", "op": "gather", "tokens": 16384, "topk": 8, "experts": 216, "cols": 7168, "type": "bf16", "dropped": 0.0},
        # a decoding batch's results back to their tokens, with the gradients (a short fine-tuning batch)
        {"name": "combine small", "op": "combine", "tokens": 64, "topk": 8, "experts": 216, "cols": 7168, "type": "fp16", "weights": "fp32", "dropped": 0.0},
        # the MoE set's width in training: 16384 tokens, 6 experts each, some padding
        {"name": "combine MoE", "op": "combine", "tokens": 16384, "topk": 6, "experts": 64, "cols": 2048, "type": "bf16", "weights": "fp32", "dropped": 0.05},
        # decoding: 192 rows over the MoE set's 64 experts (1408 x 2048); the weights' bytes count
        {"name": "product decode", "op": "product", "rows": 192, "experts": 64, "inner": 2048, "outer": 1408, "type": "bf16", "grads": False, "dw": "bf16", "tail": 0},
        # training the MoE set's up projections: forward and both gradients, unequal experts
        {"name": "product MoE", "op": "product", "rows": 49152, "experts": 64, "inner": 2048, "outer": 1408, "type": "bf16", "grads": True, "dw": "bf16", "tail": 1000},
        # eight of Kimi-K2's experts on one GPU, with gradients kept in fp32
        {"name": "product K2", "op": "product", "rows": 8192, "experts": 8, "inner": 7168, "outer": 2048, "type": "fp16", "grads": True, "dw": "fp32", "tail": 0},
        # small ragged experts in fp32, sizes that no vector width divides
        {"name": "product odd", "op": "product", "rows": 301, "experts": 7, "inner": 333, "outer": 130, "type": "fp32", "grads": True, "dw": "fp32", "tail": 5},
        # four 2048 x 2048 attention projections, each head (128 rows, or 128 columns of the output projection) on its own
        {"name": "step heads", "op": "step", "stack": 4, "rows": 2048, "cols": 2048, "block_rows": 128, "block_cols": 2048, "transposed": True, "weights": "bf16", "grads": "bf16"},
        # the MoE set's 64 experts with gate and up fused in one stacked 64 x 2816 x 2048 weight: 128 blocks
        {"name": "step experts", "op": "step", "stack": 64, "rows": 2816, "cols": 2048, "block_rows": 1408, "block_cols": 2048, "transposed": False, "weights": "bf16", "grads": "bf16"},
    ]


def _log(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def _width(rng, low, high):
    """A multiple of 8 mostly, any width else."""
    n = _log(rng, low, high)
    return n if rng.random() < 0.2 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(("sort", "gather", "combine", "product", "product", "step"))
    experts = _log(rng, 1, 256)
    topk = min(experts, rng.randint(1, 8))
    dropped = rng.choice((0.0, rng.uniform(0.0, 0.5)))
    if op == "sort":
        return {"op": op, "tokens": _log(rng, 1, 131072), "topk": topk, "experts": experts,
                "ids": rng.choice(("int32", "int64")), "dropped": dropped}
    if op in ("gather", "combine"):
        cols = _width(rng, 16, 7168)
        case = {"op": op, "tokens": min(_log(rng, 1, 16384), MOST // (2 * topk * cols)), "topk": topk, "experts": experts, "cols": cols,
                "type": rng.choice(("bf16", "fp16", "fp32")), "dropped": dropped}
        return dict(case, weights=rng.choice(("fp32", "bf16"))) if op == "combine" else case
    if op == "product":
        kind = rng.choice(("bf16", "fp16", "bf16", "fp16", "fp32"))
        high = 512 if kind == "fp32" else 2048
        return {"op": op, "rows": _log(rng, 8, 2048 if kind == "fp32" else 32768), "experts": _log(rng, 1, 32 if kind == "fp32" else 64),
                "inner": _width(rng, 32, high), "outer": _width(rng, 32, high), "type": kind,
                "grads": rng.random() < 0.7, "dw": rng.choice((kind, "fp32")), "tail": rng.choice((0, rng.randint(1, 100)))}
    block_rows, block_cols = _log(rng, 32, 1024), _log(rng, 32, 1024)
    return {"op": op, "stack": rng.randint(1, 8), "rows": block_rows * rng.randint(1, 3), "cols": block_cols * rng.randint(1, 3),
            "block_rows": block_rows, "block_cols": block_cols, "transposed": rng.random() < 0.5,
            "weights": rng.choice(("bf16", "bf16", "fp32")), "grads": rng.choice(("bf16", "fp32"))}


# ---------------------------------------------------------------- inputs
def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)


def _routing(g, tokens, topk, experts, dropped, dtype=torch.int64):
    """A router's choice of `topk` experts, popular and unpopular ones; -1 where padding goes to no expert."""
    logits = _randn(g, tokens, experts) + 0.5 * _randn(g, experts)
    ids = logits.topk(topk, dim=1).indices
    keep = torch.rand(tokens, 1, generator=g, device="cuda") >= dropped
    return torch.where(keep, ids, -1).to(dtype)


def _slots(ids, experts):
    key = torch.where((ids >= 0) & (ids < experts), ids, experts).reshape(-1).long()
    order = torch.argsort(key, stable=True)
    slot = torch.empty_like(order)
    slot[order] = torch.arange(order.numel(), device=order.device)
    return torch.where(key < experts, slot, -1).to(torch.int32).view(ids.shape)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, s = case, {"case": case}
    if c["op"] == "sort":
        s["ids"] = _routing(g, c["tokens"], c["topk"], c["experts"], c["dropped"], getattr(torch, c["ids"]))
    elif c["op"] in ("gather", "combine"):
        t, k, n, dt = c["tokens"], c["topk"], c["cols"], TYPES[c["type"]]
        s["slot"] = _slots(_routing(g, t, k, c["experts"], c["dropped"]), c["experts"])
        # one row more than the sorted rows: where the plain form sends what goes to no expert
        if c["op"] == "gather":
            s["x"] = _randn(g, t, n, dtype=dt)
            s["dxs"] = _randn(g, t * k, n, dtype=dt)
            s["xs"] = torch.zeros(t * k + 1, n, dtype=dt, device="cuda")
        else:
            s["ys"] = _randn(g, t * k, n, dtype=dt)
            s["dy"] = _randn(g, t, n, dtype=dt)
            s["weights"] = torch.softmax(_randn(g, t, k), dim=1).to(TYPES[c["weights"]])
            s["dys"] = torch.zeros(t * k + 1, n, dtype=dt, device="cuda")
    elif c["op"] == "product":
        e, r, i, o, dt = c["experts"], c["rows"], c["inner"], c["outer"], TYPES[c["type"]]
        share = torch.softmax(0.4 * _randn(g, e), dim=0)
        to = torch.multinomial(share, r, replacement=True, generator=g)
        counts = (to[:, None] == torch.arange(e, device="cuda")).sum(0) if e * r < 1 << 28 else torch.bincount(to, minlength=e)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["capacity"] = max(1, int(counts.max()))  # the plain form's rows of one expert
        s["xs"] = _randn(g, r + c["tail"], i, dtype=dt)
        s["w"] = _randn(g, e, o, i, dtype=dt, std=i ** -0.5)
        s["y"] = torch.zeros(r + c["tail"] + 1, o, dtype=dt, device="cuda")
        if c["grads"]:
            s["dys"] = _randn(g, r + c["tail"], o, dtype=dt)
            s["dxs"] = torch.zeros(r + c["tail"] + 1, i, dtype=dt, device="cuda")
    else:
        n, r, q = c["stack"], c["rows"], c["cols"]
        s["params"], s["grads"], s["moms"], s["blocks"] = [], [], [], []
        for part in range(2 if c["transposed"] and n > 1 else 1):
            # the last matrix of a transposed stack is split along its columns, as an output projection's heads are
            m = 1 if part else n - (1 if c["transposed"] and n > 1 else 0)
            shape = (m, q, r) if part else (m, r, q)
            block = (c["block_cols"], c["block_rows"]) if part else (c["block_rows"], c["block_cols"])
            s["params"].append(_randn(g, *shape, dtype=TYPES[c["weights"]], std=0.02))
            # a few strong directions and noise, as gradients of trained layers have
            low = _randn(g, m, shape[1], 64) @ _randn(g, m, 64, shape[2])
            s["grads"].append((low + 0.5 * _randn(g, *shape)).to(TYPES[c["grads"]]))
            s["moms"].append(_randn(g, *shape, std=0.1))
            s["blocks"].append(block)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    return {"sort": _sort, "gather": _gather, "combine": _combine, "product": _product, "step": _step}[state["case"]["op"]](state)


def _sort(s):
    ids, experts = s["ids"], s["case"]["experts"]
    if own:
        import newton_schulz_matrix_b200 as nsm
        return list(nsm.muon_expert_sort(ids, experts))
    key = torch.where((ids >= 0) & (ids < experts), ids, experts).reshape(-1)
    ordered, source = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ordered, torch.arange(experts + 1, device=ids.device, dtype=ids.dtype), out_int32=True)
    slot = torch.empty(key.numel(), dtype=torch.int32, device=ids.device)
    slot[source] = torch.arange(key.numel(), dtype=torch.int32, device=ids.device)
    slot = torch.where(key < experts, slot, -1).view(ids.shape)
    return [offsets, slot, source.to(torch.int32)]


def _rows_of(rows, slot):
    """The sorted rows of every token's assignments in 32 bits, zeros where it went to no expert."""
    picked = rows[slot.clamp(min=0).reshape(-1).long()].float().view(*slot.shape, -1)
    return torch.where((slot >= 0)[..., None], picked, 0.0)


def _to_rows(out, slot, rows):
    """out[slot] = rows; what has no slot goes to the row behind the last."""
    at = torch.where(slot >= 0, slot, out.shape[0] - 1).reshape(-1).long()
    out.index_copy_(0, at, rows.to(out.dtype))
    return out[:-1]


def _gather(s):
    x, slot, dxs = s["x"], s["slot"], s["dxs"]
    if own:
        import newton_schulz_matrix_b200 as nsm
        return [nsm.muon_expert_gather(x, slot, out=s["xs"][:-1]), nsm.muon_expert_gather_backward(dxs, slot)]
    xs = _to_rows(s["xs"], slot, x.repeat_interleave(slot.shape[1], dim=0))
    return [xs, _rows_of(dxs, slot).sum(1).to(x.dtype)]


def _combine(s):
    ys, dy, slot, weights = s["ys"], s["dy"], s["slot"], s["weights"]
    if own:
        import newton_schulz_matrix_b200 as nsm
        y = nsm.muon_expert_combine(ys, slot, weights)
        dys, dw = nsm.muon_expert_combine_backward(dy, ys, slot, weights, out=s["dys"][:-1])
        return [y, dys, dw]
    rows, w = _rows_of(ys, slot), weights.float()
    y = (rows * w[..., None]).sum(1).to(ys.dtype)
    dw = (rows * dy.float()[:, None, :]).sum(2).to(weights.dtype)
    dys = _to_rows(s["dys"], slot, (dy.float()[:, None, :] * w[..., None]).reshape(-1, dy.shape[1]))
    return [y, dys, dw]


def _product(s):
    c, xs, w, offsets = s["case"], s["xs"], s["w"], s["offsets"]
    if own:
        import newton_schulz_matrix_b200 as nsm
        out = [nsm.muon_expert_product(xs, w, offsets, out=s["y"][:-1])]
        if c["grads"]:
            out.append(nsm.muon_expert_input_grad(s["dys"], w, offsets, out=s["dxs"][:-1]))
            out.append(nsm.muon_expert_weight_grad(s["dys"], xs, offsets, out_dtype=TYPES[c["dw"]]))
        return out
    at = offsets[:-1, None] + torch.arange(s["capacity"], device=offsets.device, dtype=torch.int32)
    slot = torch.where(at < offsets[1:, None], at, -1)  # experts x capacity
    w32, x32 = w.float(), _rows_of(xs, slot)
    out = [_to_rows(s["y"], slot, (x32 @ w32.transpose(1, 2)).flatten(0, 1))]
    if c["grads"]:
        dy32 = _rows_of(s["dys"], slot)
        out.append(_to_rows(s["dxs"], slot, (dy32 @ w32).flatten(0, 1)))
        out.append((dy32.transpose(1, 2) @ x32).to(TYPES[c["dw"]]))
    return out


STEP = {"lr": 0.02, "momentum": 0.95, "weight_decay": 0.1, "scale_coef": 0.2}


def _blocks(t, block):
    """(..., R, C) as (blocks, rows, cols): a copy in the order of the tensor's matrices, block rows and block columns."""
    r, c = block
    t = t.reshape(-1, t.shape[-2] // r, r, t.shape[-1] // c, c)
    return t.transpose(2, 3).reshape(-1, r, c)


def _unblocks(b, shape, block):
    r, c = block
    return b.reshape(-1, shape[-2] // r, shape[-1] // c, r, c).transpose(2, 3).reshape(shape)


def _step(s):
    if own:
        import newton_schulz_matrix_b200 as nsm
        # fp32 weights ask for an fp32 iteration, 16-bit ones take the default (stored in fp16 between the products)
        compute = "fp32" if s["case"]["weights"] == "fp32" else "fp16"
        nsm.muon_step_blocks(s["params"], s["grads"], s["moms"], s["blocks"], compute_dtype=compute, **STEP)
        return [s["params"], s["moms"]]
    mu = STEP["momentum"]
    for w, grad, m, block in zip(s["params"], s["grads"], s["moms"], s["blocks"]):
        m.mul_(mu).add_(grad.float(), alpha=1 - mu)
        x = _blocks((1 - mu) * grad.float() + mu * m, block)
        tall = block[0] > block[1]
        x = x.transpose(1, 2) if tall else x
        x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + 1e-7)
        for _ in range(5):
            gram = x @ x.transpose(1, 2)
            x = QUINTIC[0] * x + (QUINTIC[1] * gram + QUINTIC[2] * (gram @ gram)) @ x
        x = _unblocks(x.transpose(1, 2) if tall else x, w.shape, block)
        scale = STEP["lr"] * STEP["scale_coef"] * math.sqrt(max(block))
        w.copy_((1 - STEP["lr"] * STEP["weight_decay"]) * w.float() - scale * x)
    return [s["params"], s["moms"]]


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "sort":
        n = c["tokens"] * c["topk"]
        return {"bytes": n * ((8 if c["ids"] == "int64" else 4) + 8) + 4 * (c["experts"] + 1), "flops": 0}
    if c["op"] in ("gather", "combine"):
        t, k, n, es = c["tokens"], c["topk"], c["cols"], 4 if c["type"] == "fp32" else 2
        rows = (1 - c["dropped"]) * t * k * n * es
        if c["op"] == "gather":  # x in and xs out; dxs in and dx out
            return {"bytes": 2 * (rows + t * n * es) + 8 * t * k, "flops": t * k * n}
        ws = 4 if c["weights"] == "fp32" else 2  # y: ys in, y out; gradients: ys and dy in, dys out
        return {"bytes": 3 * rows + 2 * t * n * es + t * k * (8 + 3 * ws), "flops": 5 * t * k * n}
    if c["op"] == "product":
        r, e, i, o, es = c["rows"], c["experts"], c["inner"], c["outer"], 4 if c["type"] == "fp32" else 2
        used = min(e, r)  # experts that can have rows
        b, f = (r * (i + o) + used * i * o) * es, 2 * r * i * o
        if c["grads"]:
            b += (r * (i + o) + used * i * o) * es + r * (i + o) * es + e * i * o * (4 if c["dw"] == "fp32" else 2)
            f *= 3
        return {"bytes": b, "flops": f}
    n, m = sorted((c["block_rows"], c["block_cols"]))
    elements = c["stack"] * c["rows"] * c["cols"]
    per = (4 if c["weights"] == "bf16" else 8) + (2 if c["grads"] == "bf16" else 4) + 8
    return {"bytes": elements * per, "flops": elements / (n * m) * 5 * (4 * m * n * n + 2 * n ** 3)}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "sort":
        return None
    if c["op"] in ("gather", "combine"):
        slot = s["slot"].cpu().reshape(-1).tolist()
        tokens, k = c["tokens"], c["topk"]
        token = torch.tensor([a // k for a, p in enumerate(slot) if p >= 0], device="cuda", dtype=torch.long)
        place = torch.tensor([a for a, p in enumerate(slot) if p >= 0], device="cuda", dtype=torch.long)
        row = torch.tensor([p for p in slot if p >= 0], device="cuda", dtype=torch.long)
        if c["op"] == "gather":
            xs = torch.zeros(tokens * k, c["cols"], dtype=torch.float64, device="cuda")
            xs[row] = s["x"].double()[token]
            dx = torch.zeros(tokens, c["cols"], dtype=torch.float64, device="cuda")
            return [xs, dx.index_add_(0, token, s["dxs"].double()[row])]
        w = s["weights"].double().reshape(-1)[place]
        rows, grads = s["ys"].double()[row], s["dy"].double()[token]
        y = torch.zeros(tokens, c["cols"], dtype=torch.float64, device="cuda").index_add_(0, token, w[:, None] * rows)
        dw = torch.zeros(tokens * k, dtype=torch.float64, device="cuda")
        dw[place] = torch.einsum("pc,pc->p", rows, grads)
        dys = torch.zeros(tokens * k, c["cols"], dtype=torch.float64, device="cuda")
        dys[row] = w[:, None] * grads
        return [y, dys, dw.view(tokens, k)]
    if c["op"] == "product":
        ends = s["offsets"].tolist()
        y = torch.zeros(s["xs"].shape[0], c["outer"], dtype=torch.float64, device="cuda")
        dx = torch.zeros(s["xs"].shape[0], c["inner"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(c["experts"], c["outer"], c["inner"], dtype=torch.float64, device="cuda")
        for e in range(c["experts"]):
            at = slice(ends[e], ends[e + 1])
            x, w = s["xs"][at].double(), s["w"][e].double()
            y[at] = x @ w.T
            if c["grads"]:
                dy = s["dys"][at].double()
                dx[at] = dy @ w
                dw[e] = dy.T @ x
        return [y, dx, dw] if c["grads"] else [y]
    params, moms = [], []
    for w, grad, m, (r, q) in zip(s["params"], s["grads"], s["moms"], s["blocks"]):
        w, grad, m = w.double(), grad.double(), m.double()
        m = 0.95 * m + 0.05 * grad
        u = 0.05 * grad + 0.95 * m
        w *= 1 - 0.02 * 0.1
        for matrix in range(w.shape[0]):
            for i in range(0, w.shape[1], r):
                for j in range(0, w.shape[2], q):
                    x = u[matrix, i:i + r, j:j + q]
                    x = x.T if r > q else x
                    x = x / (torch.linalg.norm(x) + 1e-7)
                    for _ in range(5):
                        gram = x @ x.T
                        x = QUINTIC[0] * x + QUINTIC[1] * gram @ x + QUINTIC[2] * gram @ (gram @ x)
                    w[matrix, i:i + r, j:j + q] -= 0.02 * 0.2 * math.sqrt(max(r, q)) * (x.T if r > q else x)
        params.append(w)
        moms.append(m)
    return [params, moms]
