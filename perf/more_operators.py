"""Timed cases of the experts' operators.

Operators:
  route   router logits to the chosen experts of every token and their weights
  plan    the chosen experts to rows sorted by expert: order (the choice that
          each row belongs to), place (its inverse), offsets (an expert's rows)
  up      rows of packed activations, gathered by the plan, through the gate
          and up matrices of their expert: h = silu(g) u as e4m3 codes with one
          scale per 128 features
  down    rows in the plan's order through the down matrix of their expert,
          then every token's weighted sum of its rows
  moe     from the activations and the chosen experts to the block's output:
          pack, plan, up, down, weighted sum and residual

Codes are e4m3 with one fp32 scale per row and 128 features of an activation
and per 128 x 128 block of a weight.

`own` selects between the plain torch form of an operator and the library's
kernels; the tool that times the file sets it.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
MOST_WEIGHTS = 64 * 3 * 1536 * 4096   # codes of the largest listed case
MOST_PRODUCTS = 4096 * 8 * 3 * 1536 * 4096


def listed():
    return [
        # one decoded token chooses its experts: latency only
        dict(name="route_token", op="route", T=1, E=64, k=8, dtype="bf16", score="softmax", bias=False, groups=1,
             top_groups=1, group_top=1, renormalise=True, scale=1.0, masked=False),
        # a prompt through a router balanced by a bias, choosing groups first
        dict(name="route_prompt", op="route", T=4096, E=256, k=8, dtype="f32", score="sigmoid", bias=True, groups=8,
             top_groups=4, group_top=2, renormalise=True, scale=2.5, masked=False),
        # an odd number of tokens and experts, some experts closed to some tokens, rows that have none left
        dict(name="route_masked", op="route", T=1003, E=60, k=4, dtype="f16", score="softmax", bias=False, groups=1,
             top_groups=1, group_top=1, renormalise=False, scale=1.0, masked=True),
        # a decode batch padded for a captured graph: a tenth of its tokens choose nothing
        dict(name="plan_batch", op="plan", T=64, E=128, k=8, padded=True),
        # the plan of a long prompt
        dict(name="plan_prompt", op="plan", T=8192, E=256, k=8, padded=False),
        # a decode batch: about two rows for each of the experts' matrices
        dict(name="up_batch", op="up", T=32, E=128, k=8, K=2048, I=768, bias=False, padded=False),
        # a prompt of odd length, widths that end inside a block, biases
        dict(name="up_odd", op="up", T=1531, E=24, k=4, K=1296, I=912, bias=True, padded=True),
        # the same batch through the down matrices
        dict(name="down_batch", op="down", T=32, E=128, k=8, K=768, N=2048, bias=False, padded=False, out="bf16"),
        # a prompt through the down matrices
        dict(name="down_prompt", op="down", T=4096, E=32, k=4, K=1024, N=2048, bias=False, padded=False, out="bf16"),
        # one decoded token through a whole expert block: its experts' weights are read once
        dict(name="moe_token", op="moe", T=1, E=64, k=8, K=4096, I=1536, dtype="bf16", bias=False, residual=True,
             padded=False),
        # a short prompt of odd sizes in binary16, some tokens padding
        dict(name="moe_short", op="moe", T=331, E=20, k=3, K=1280, I=656, dtype="f16", bias=True, residual=False,
             padded=True),
        # a prompt through a whole expert block
        dict(name="moe_prompt", op="moe", T=4096, E=64, k=8, K=4096, I=1536, dtype="bf16", bias=False, residual=True,
             padded=False),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "plan", "up", "down", "moe", "moe"])
    E = rng.choice([8, 16, 24, 60, 64, 96, 128, 160, 256])
    k = rng.randint(1, 8)
    T = _log_uniform(rng, 1, 8192)
    if op == "route":
        bias = rng.random() < 0.5
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2])
        top_groups = rng.randint(1, groups)
        return dict(op=op, T=min(T, 4096 * 256 // E), E=E, k=min(k, top_groups * (E // groups)),
                    dtype=rng.choice(["bf16", "f16", "f32", "f32"]), score=rng.choice(["softmax", "sigmoid"]),
                    bias=bias, groups=groups, top_groups=top_groups, group_top=rng.randint(1, 2),
                    renormalise=rng.random() < 0.6, scale=rng.choice([1.0, 1.0, 2.5]), masked=rng.random() < 0.4)
    padded = rng.random() < 0.4
    if op == "plan":
        return dict(op=op, T=T, E=E, k=k, padded=padded)
    K = max(16, _log_uniform(rng, 128, 4096) // 16 * 16)
    inner = max(16, _log_uniform(rng, 64, 2048) // 16 * 16)
    E = max(k, min(E, MOST_WEIGHTS // (3 * K * inner)))
    T = max(1, min(T, MOST_PRODUCTS // (3 * K * inner * k)))
    bias = rng.random() < 0.5
    if op == "up":
        return dict(op=op, T=T, E=E, k=k, K=K, I=inner, bias=bias, padded=padded)
    if op == "down":
        return dict(op=op, T=T, E=E, k=k, K=inner, N=K if rng.random() < 0.7 else K - rng.randint(1, 15), bias=bias,
                    padded=padded, out=rng.choice(["bf16", "f16", "f32"]))
    # the result of codes formed within the call hangs on which side of a
    # rounding border each code fell: 16-bit results alone
    return dict(op=op, T=T, E=E, k=k, K=K, I=inner, dtype=rng.choice(["bf16", "bf16", "f16"]), bias=bias,
                residual=rng.random() < 0.5, padded=padded)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _rand(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda")


def _activations(gen, M, K):
    """Unit normal values with a few outlier channels, as such activations have."""
    X = _randn(gen, M, K)
    X *= 1.0 + 29.0 * (_rand(gen, K) < 0.005)
    return X


def _codes(V, rows):
    """Codes and scales of V over blocks of `rows` x 128."""
    R, K = V.shape
    P = torch.zeros((R + rows - 1) // rows * rows, _blocks(K) * BLOCK, device=V.device)
    P[:R, :K] = V
    B = P.view(-1, rows, _blocks(K), BLOCK)
    amax = B.abs().amax(dim=(1, 3))
    s = amax / torch.full_like(amax, E4M3_MAX)
    q = torch.where(s[:, None, :, None] > 0, B / s[:, None, :, None], torch.zeros_like(B))
    q = q.clamp(-E4M3_MAX, E4M3_MAX).reshape(P.shape)[:R, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), s


def _matrices(gen, E, N, K, bias):
    """Codes [E,N,K], scales and biases of the experts' matrices."""
    q = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(E, _blocks(N), _blocks(K), device="cuda")
    for e in range(E):
        q[e], s[e] = _codes(K ** -0.5 * _randn(gen, N, K), BLOCK)
    return q, s, 0.1 * _randn(gen, E, N) if bias else None


def _choices(gen, T, E, k, padded):
    """Experts of every token, some of them more popular than others, and their weights."""
    logits = _randn(gen, T, E) + 0.5 * _randn(gen, E)
    w, e = torch.topk(torch.softmax(logits, dim=1), k, dim=1)
    w, e = w / w.sum(dim=1, keepdim=True), e.to(torch.int32)
    if padded:  # tokens that pad the batch choose nothing
        pad = _rand(gen, T) < 0.1
        e[pad] = -1
        w[pad] = 0.0
    return e.contiguous(), w.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s, op, T, E, k = dict(case), case["op"], case["T"], case["E"], case["k"]
    if op == "route":
        logits = 1.5 * _randn(gen, T, E) + 0.5 * _randn(gen, E)
        if case["masked"]:
            logits[_rand(gen, T, E) < 0.3] = -math.inf
            logits[_rand(gen, T) < 0.02] = -math.inf
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        s["bias_vector"] = 0.1 * _randn(gen, E) if case["bias"] else None
        s["experts"] = torch.empty(T, k, dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(T, k, device="cuda")
        return s
    s["experts"], s["weights"] = _choices(gen, T, E, k, case["padded"])
    if op in ("plan", "moe"):
        if op == "plan":
            s["order"] = torch.empty(T * k, dtype=torch.int32, device="cuda")
            s["place"] = torch.empty(T * k, dtype=torch.int32, device="cuda")
            s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
            return s
        s["X"] = _activations(gen, T, case["K"]).to(DTYPES[case["dtype"]])
        s["gate"] = _matrices(gen, E, case["I"], case["K"], case["bias"])
        s["up"] = _matrices(gen, E, case["I"], case["K"], case["bias"])
        s["down"] = _matrices(gen, E, case["K"], case["I"], case["bias"])
        s["R"] = _randn(gen, T, case["K"]).to(DTYPES[case["dtype"]]) if case["residual"] else None
        s["Y"] = torch.empty_like(s["X"])
        return s
    s["order"], s["place"], s["offsets"] = _plan(s["experts"], E)
    if op == "up":
        s["Qx"], s["sx"] = _codes(_activations(gen, T, case["K"]), 1)
        s["gate"] = _matrices(gen, E, case["I"], case["K"], case["bias"])
        s["up"] = _matrices(gen, E, case["I"], case["K"], case["bias"])
        # rows that the plan leaves free keep what the buffers hold
        s["Qh"] = torch.zeros(T * k, case["I"], dtype=torch.float8_e4m3fn, device="cuda")
        s["sh"] = torch.zeros(T * k, _blocks(case["I"]), device="cuda")
        return s
    s["Qh"], s["sh"] = _codes(_activations(gen, T * k, case["K"]), 1)
    s["down"] = _matrices(gen, E, case["N"], case["K"], case["bias"])
    s["rows"] = torch.zeros(T * k, case["N"], dtype=DTYPES[case["out"]], device="cuda")
    s["Y"] = torch.empty(T, case["N"], dtype=DTYPES[case["out"]], device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _widen(s, rows, cols, height):
    """Block scales as one factor per element."""
    return s.repeat_interleave(height, dim=0)[:rows].repeat_interleave(BLOCK, dim=1)[:, :cols]


def _decode(q, s, height):
    return q.float() * _widen(s, q.shape[0], q.shape[1], height)


def _plan(experts, E):
    """order, place and offsets of the choices; -1 is no choice."""
    e = experts.flatten().long()
    chosen = e >= 0
    counts = torch.zeros(E + 1, dtype=torch.int64, device=e.device)
    counts.scatter_add_(0, torch.where(chosen, e, E), torch.ones_like(e))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=e.device)
    offsets[1:] = torch.cumsum(counts[:E], 0)
    order = torch.sort(torch.where(chosen, e, E), stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(e.numel(), device=e.device)
    order = torch.where(torch.arange(e.numel(), device=e.device) < offsets[E], order, -1)
    return order.to(torch.int32), torch.where(chosen, place, -1).to(torch.int32), offsets.to(torch.int32)


def _route(s):
    # in 64 bits: which of two scores is larger hangs on their last digits
    l = s["logits"].double()
    closed = l == -math.inf
    if s["score"] == "softmax":
        m = l.max(dim=1, keepdim=True).values
        p = torch.where(closed, 0.0, torch.exp(l - m))
        total = p.sum(dim=1, keepdim=True)
        score = torch.where(total > 0, p / total, 0.0)
    else:
        score = torch.where(closed, 0.0, 1.0 / (1.0 + torch.exp(-l)))
    v = l if s["bias_vector"] is None else torch.where(closed, -math.inf, score + s["bias_vector"].double())
    if s["groups"] > 1:
        T, E = l.shape
        per = E // s["groups"]
        if s["group_top"] == 1:
            value = v.view(T, -1, per).max(dim=2).values
        else:
            w = score if s["bias_vector"] is None else v
            w = torch.where(closed, -math.inf, w).view(T, -1, per).sort(dim=2, descending=True).values
            value = w[:, :, 0] + torch.where(w[:, :, 1] > -math.inf, w[:, :, 1], 0.0)
        best = value.sort(dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        open_group = torch.zeros_like(value, dtype=torch.bool).scatter_(1, best, True)
        v = torch.where(open_group.repeat_interleave(per, dim=1), v, -math.inf)
    v, e = (t[:, :s["k"]] for t in v.sort(dim=1, descending=True, stable=True))
    w = score.gather(1, e)
    taken = v > -math.inf
    w = torch.where(taken, w, 0.0)
    if s["renormalise"]:
        total = w.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(taken, e, -1).to(torch.int32), (w * s["scale"]).float()


def _linear_rows(X, rows, offsets, q, s, bias, out):
    """out[i] = X[rows[i]] W_e^T + b_e for the rows i of every expert e."""
    for e in range(len(offsets) - 1):
        i, j = offsets[e], offsets[e + 1]
        if i < j:
            y = X[rows[i:j]] @ _decode(q[e], s[e], BLOCK).t()
            out[i:j] = y if bias is None else y + bias[e]
    return out


def _up(Qx, sx, order, offsets, k, gate, up):
    tokens = order.long() // k
    X, n, width = _decode(Qx, sx, 1), order.numel(), gate[0].shape[1]
    g = _linear_rows(X, tokens, offsets, *gate, torch.zeros(n, width, device=X.device))
    u = _linear_rows(X, tokens, offsets, *up, torch.zeros(n, width, device=X.device))
    return _codes(g / (1.0 + torch.exp(-g)) * u, 1)


def _combine(rows, place, weights):
    """Every token's weighted sum of its rows."""
    p = place.long().view(weights.shape)
    y = torch.zeros(weights.shape[0], rows.shape[1], device=rows.device)
    for j in range(weights.shape[1]):
        w = torch.where(p[:, j] >= 0, weights[:, j], 0.0)
        y += w[:, None] * rows[p[:, j].clamp_min(0)].float()
    return y


def _plain(s):
    if s["op"] == "route":
        return _route(s)
    if s["op"] == "plan":
        return _plan(s["experts"], s["E"])
    if s["op"] == "up":
        return _up(s["Qx"], s["sx"], s["order"], s["offsets"].tolist(), s["k"], s["gate"], s["up"])
    if s["op"] == "down":
        rows = torch.zeros(s["rows"].shape, device="cuda")
        rows = _linear_rows(_decode(s["Qh"], s["sh"], 1), torch.arange(rows.shape[0], device="cuda"),
                            s["offsets"].tolist(), *s["down"], rows).to(s["rows"].dtype)
        return rows, _combine(rows, s["place"], s["weights"]).to(rows.dtype)
    order, place, offsets = _plan(s["experts"], s["E"])
    offsets = offsets.tolist()
    Qx, sx = _codes(s["X"].float(), 1)
    Qh, sh = _up(Qx, sx, order, offsets, s["k"], s["gate"], s["up"])
    rows = _linear_rows(_decode(Qh, sh, 1), torch.arange(order.numel(), device="cuda"), offsets, *s["down"],
                        torch.zeros(order.numel(), s["K"], device="cuda"))
    y = _combine(rows, place, s["weights"])
    return (y if s["R"] is None else y + s["R"].float()).to(s["X"].dtype)


def run(state):
    s = state
    if not own:
        return _plain(s)
    from int8_hadamard_rotated_gb300 import ops
    if s["op"] == "route":
        kinds = {"softmax": ops.MOE_SOFTMAX, "sigmoid": ops.MOE_SIGMOID}
        return ops.moe_route(s["logits"], s["k"], score=kinds[s["score"]],
                             bias=s["bias_vector"], n_groups=s["groups"], top_groups=s["top_groups"],
                             group_top=s["group_top"], renormalise=s["renormalise"], scale=s["scale"],
                             experts=s["experts"], weights=s["weights"])
    if s["op"] == "plan":
        return ops.moe_plan(s["experts"], s["E"], order=s["order"], place=s["place"], offsets=s["offsets"])
    if s["op"] == "up":
        return ops.fp8_expert_swiglu(s["Qx"], s["sx"], s["order"], s["offsets"], s["k"], s["gate"], s["up"],
                                     Q_h=s["Qh"], s_h=s["sh"])
    if s["op"] == "down":
        rows = ops.fp8_expert_linear(s["Qh"], s["sh"], s["offsets"], s["down"], Y=s["rows"])
        return rows, ops.moe_combine(rows, s["place"], s["weights"], Y=s["Y"])
    return ops.fp8_moe(s["X"], s["experts"], s["weights"], s["gate"], s["up"], s["down"], residual=s["R"], Y=s["Y"])


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    T, E, k, op = case["T"], case["E"], case["k"], case["op"]
    n = T * k
    if op == "route":
        return {"bytes": T * E * SIZES[case["dtype"]] + 4 * E * case["bias"] + 8 * n, "flops": 8 * T * E}
    if op == "plan":
        return {"bytes": 12 * n + 4 * (E + 1), "flops": 4 * n}
    # the choices that are made, and the experts that tokens choosing evenly would reach
    n = n * 0.9 if case["padded"] else n
    reached = E * (1.0 - (1.0 - k / E) ** (n / k))
    K, wide = case["K"], case["N"] if op == "down" else case["I"]
    matrix = wide * K + 4 * _blocks(wide) * _blocks(K) + 4 * wide * case["bias"]
    if op == "up":
        return {"bytes": int(T * (K + 4 * _blocks(K)) + 2 * reached * matrix + n * (wide + 4 * _blocks(wide) + 4)),
                "flops": int(4 * n * K * wide)}
    if op == "down":
        b = SIZES[case["out"]]
        return {"bytes": int(n * (K + 4 * _blocks(K)) + reached * matrix + n * wide * b + T * wide * b + 8 * T * k),
                "flops": int(2 * n * K * wide + 2 * n * wide)}
    b = SIZES[case["dtype"]]
    return {"bytes": int(T * K * b * (2 + case["residual"]) + 3 * reached * matrix + 8 * T * k),
            "flops": int(6 * n * K * wide)}


def _rank_first(v, count):
    """Indices of the `count` largest of every row, the lowest first among equal ones."""
    out = []
    for row in v.split(max(1, (1 << 26) // v.shape[1] ** 2)):
        ahead = (row[:, None, :] > row[:, :, None]).sum(dim=2)
        same = (row[:, None, :] == row[:, :, None]).tril(-1).sum(dim=2)
        rank = ahead + same
        out.append(torch.zeros_like(rank).scatter_(1, rank, torch.arange(v.shape[1], device=v.device).expand_as(rank)))
    return torch.cat(out)[:, :count]


def _exact_route(s):
    l = s["logits"].double()
    open_ = torch.isfinite(l)
    score = torch.softmax(l, dim=1).nan_to_num(0.0) if s["score"] == "softmax" else torch.sigmoid(l)
    v = l
    if s["bias_vector"] is not None:
        v = (score + s["bias_vector"].double()).masked_fill(~open_, -math.inf)
    if s["groups"] > 1:
        T, per = l.shape[0], l.shape[1] // s["groups"]
        ranked = v if s["group_top"] == 1 or s["bias_vector"] is not None else score.masked_fill(~open_, -math.inf)
        ranked = ranked.view(T * s["groups"], per)
        top = ranked.gather(1, _rank_first(ranked, s["group_top"]))
        value = top[:, 0] if s["group_top"] == 1 else top[:, 0] + top[:, 1].masked_fill(top[:, 1] == -math.inf, 0.0)
        keep = _rank_first(value.view(T, -1), s["top_groups"])
        shut = torch.ones(T, s["groups"], dtype=torch.bool, device=l.device)
        shut[torch.arange(T, device=l.device)[:, None], keep] = False
        v = v.view(T, s["groups"], per).masked_fill(shut[:, :, None], -math.inf).view(T, -1)
    e = _rank_first(v, s["k"])
    none = v.gather(1, e) == -math.inf
    w = score.gather(1, e).masked_fill(none, 0.0)
    if s["renormalise"]:
        w = (w / w.sum(dim=1, keepdim=True)).nan_to_num(0.0)
    return e.masked_fill(none, -1), w * s["scale"]


def _exact_codes(X):
    """e4m3 values and fp32 scales of X (64 bits) per 128 features: of the fp32
    quotient, as the codes are defined, the nearest multiple, ties to even, of a
    step that is 2^-3 of the binade and at least 2^-9."""
    Q, scales = [], []
    for k in range(0, X.shape[1], BLOCK):
        x = X[:, k:k + BLOCK]
        s = (x.abs().max(dim=1).values / E4M3_MAX).float().double()
        z = (x / torch.where(s > 0, s, 1.0)[:, None]).float().double()
        step = torch.exp2(torch.floor(torch.log2(z.abs().clamp_min(2.0 ** -6))) - 3.0)
        Q.append(torch.clamp(torch.round(z / step) * step, -E4M3_MAX, E4M3_MAX))
        scales.append(s)
    return torch.cat(Q, 1), torch.stack(scales, 1)


def _exact_values(Q, s):
    return torch.cat([Q[:, BLOCK * j:BLOCK * (j + 1)].double() * s[:, j:j + 1].double() for j in range(s.shape[1])], 1)


def _exact_matrix(q, s):
    return torch.cat([_exact_values(q[BLOCK * i:BLOCK * (i + 1)], s[i:i + 1]) for i in range(s.shape[0])])


def _exact_linear(X, e, matrix):
    q, s, bias = matrix
    y = X @ _exact_matrix(q[e], s[e]).t()
    return y if bias is None else y + bias[e].double()


def _exact_by_expert(experts, E):
    """Every expert's choices (token times k plus slot), in order."""
    flat = experts.flatten()
    return [(flat == e).nonzero().flatten() for e in range(E)]


def _exact_h(X, c, e, s):
    x = X[torch.div(c, s["k"], rounding_mode="floor")]
    g, u = _exact_linear(x, e, s["gate"]), _exact_linear(x, e, s["up"])
    return _exact_codes(g * torch.sigmoid(g) * u)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    chosen = _exact_by_expert(s["experts"], case["E"])
    n = case["T"] * case["k"]
    if case["op"] == "plan":
        order = torch.cat(chosen)
        place = torch.full((n,), -1, dtype=torch.int64, device="cuda")
        place[order] = torch.arange(order.numel(), device="cuda")
        ends = torch.tensor([0] + [c.numel() for c in chosen], device="cuda").cumsum(0)
        free = torch.full((n - order.numel(),), -1, dtype=torch.int64, device="cuda")
        return torch.cat([order, free]), place, ends
    first = 0
    if case["op"] == "up":
        X = _exact_values(s["Qx"], s["sx"])
        Q = torch.zeros(n, case["I"], dtype=torch.float64, device="cuda")
        scales = torch.zeros(n, _blocks(case["I"]), dtype=torch.float64, device="cuda")
        for e, c in enumerate(chosen):
            if c.numel():
                Q[first:first + c.numel()], scales[first:first + c.numel()] = _exact_h(X, c, e, s)
            first += c.numel()
        return Q, scales
    weights = s["weights"].double().flatten()
    if case["op"] == "down":
        H = _exact_values(s["Qh"], s["sh"])
        rows = torch.zeros(n, case["N"], dtype=torch.float64, device="cuda")
        Y = torch.zeros(case["T"], case["N"], dtype=torch.float64, device="cuda")
        for e, c in enumerate(chosen):
            if c.numel():
                r = _exact_linear(H[first:first + c.numel()], e, s["down"])
                rows[first:first + c.numel()] = r
                Y.index_add_(0, torch.div(c, case["k"], rounding_mode="floor"), weights[c, None] * r)
            first += c.numel()
        return rows, Y
    X = _exact_values(*_exact_codes(s["X"].double()))
    Y = torch.zeros(case["T"], case["K"], dtype=torch.float64, device="cuda")
    for e, c in enumerate(chosen):
        if c.numel():
            r = _exact_linear(_exact_values(*_exact_h(X, c, e, s)), e, s["down"])
            Y.index_add_(0, torch.div(c, case["k"], rounding_mode="floor"), weights[c, None] * r)
    return Y if s["R"] is None else Y + s["R"].double()
