"""Timed cases of the block norms and the 8-bit floating-point linears.

Operators:
  norm    the norms around a transformer block, its gate and its residual in
          one pass: h' = a h + g * (b post(y)), u = modulate(pre(h')); u is
          stored as it is, or ("fp8") as e4m3 codes with one scale per 128
          features, which is what the linears read.
  pack    activations to e4m3 codes with one scale per row and 128 features.
  linear  Y = X W^T + bias with e4m3 weights, one scale per 128 x 128 block;
          X is packed within the call, or ("packed") comes as codes.

`own` selects between the plain torch form of an operator and the library's
kernels; the tool that times the file sets it.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # one decoded token through a sandwich of RMS norms: latency only
        dict(name="norm_token", op="norm", M=1, K=3072, dtype="bf16", post="rms", pre="rms", gate=False,
             modulate=False, samples=1, ragged=False, out="same"),
        # a diffusion transformer's block boundary: gated residual, LayerNorm
        # and modulation per sample, two samples of 2304 rows
        dict(name="norm_dit", op="norm", M=4608, K=3072, dtype="bf16", post="none", pre="layer", gate=True,
             modulate=True, samples=2, ragged=False, out="same"),
        # the same boundary feeding an 8-bit linear: codes instead of u, seven
        # packed samples of different lengths, RMS norms on both sides
        dict(name="norm_dit_fp8", op="norm", M=4608, K=3072, dtype="bf16", post="rms", pre="rms", gate=True,
             modulate=True, samples=7, ragged=True, out="fp8"),
        # an odd width and an odd row count in binary16
        dict(name="norm_odd", op="norm", M=1003, K=1283, dtype="f16", post="rms", pre="rms", gate=False,
             modulate=False, samples=1, ragged=False, out="same"),
        # the widest rows, an fp32 residual stream
        dict(name="norm_wide", op="norm", M=4608, K=12288, dtype="f32", post="rms", pre="rms", gate=True,
             modulate=False, samples=1, ragged=False, out="same"),
        # the packs of one token's and of a full batch's MLP activation
        dict(name="pack_token", op="pack", M=1, K=12288, dtype="bf16"),
        dict(name="pack_mlp", op="pack", M=4608, K=12288, dtype="bf16"),
        # one token through three projections that share its pack
        dict(name="linear_token", op="linear", M=1, K=3072, N=3072, count=3, dtype="bf16", out="bf16", packed=False,
             bias=True),
        # a decode batch through the MLP's down linear, codes from an earlier pack
        dict(name="linear_batch", op="linear", M=24, K=12288, N=3072, count=1, dtype="bf16", out="f32", packed=True,
             bias=True),
        # a short prompt through a U-Net-sized linear with an odd output width
        dict(name="linear_short", op="linear", M=331, K=1280, N=1283, count=1, dtype="f16", out="f16", packed=False,
             bias=False),
        # the diffusion transformer's projections, activations packed in the call
        dict(name="linear_dit", op="linear", M=4608, K=3072, N=3072, count=3, dtype="bf16", out="bf16", packed=False,
             bias=True),
        # the MLP's down linear: long sums, fp32 out
        dict(name="linear_down", op="linear", M=4608, K=12288, N=3072, count=1, dtype="bf16", out="f32", packed=True,
             bias=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "pack", "linear", "linear", "linear"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "norm":
        out = rng.choice(["same", "same", "fp8"])
        K = _log_uniform(rng, 64, 12288)
        K = max(16, K // 16 * 16) if out == "fp8" or rng.random() < 0.6 else K
        M = min(_log_uniform(rng, 1, 8192), 4608 * 12288 // K)
        samples = rng.randint(1, min(8, M))
        return dict(op=op, M=M, K=K, dtype=dtype, post=rng.choice(["none", "rms", "layer"]),
                    pre=rng.choice(["rms", "layer"]), gate=rng.random() < 0.6, modulate=rng.random() < 0.6,
                    samples=samples, ragged=rng.random() < 0.5, out=out)
    if op == "pack":
        K = max(16, _log_uniform(rng, 64, 12288) // 16 * 16)
        return dict(op=op, M=min(_log_uniform(rng, 1, 8192), 4608 * 12288 // K), K=K, dtype=dtype)
    K = max(16, _log_uniform(rng, 64, 12288) // 16 * 16)
    N = _log_uniform(rng, 64, 12288)
    N = max(8, N // 8 * 8) if rng.random() < 0.7 else N
    count = rng.randint(1, 3)
    M = min(_log_uniform(rng, 1, 8192), max(1, 4608 * 12288 * 3072 // (K * N * count)))
    packed = rng.random() < 0.5
    # an fp32 result of activations packed in the call hangs on which side of
    # a rounding border each code fell; it is drawn from given codes alone
    out = rng.choice(["bf16", "f16", "f32"]) if packed else rng.choice(["bf16", "f16"])
    return dict(op=op, M=M, K=K, N=N, count=count, dtype=dtype, out=out, packed=packed, bias=rng.random() < 0.5)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _activations(gen, M, K):
    """Unit normal values with a few outlier channels, as such activations have."""
    X = _randn(gen, M, K)
    X *= 1.0 + 29.0 * (torch.rand(K, generator=gen, device="cuda") < 0.005)
    return X


def _codes(V, rows):
    """Codes and scales of V over blocks of `rows` x 128."""
    R, K = V.shape
    P = torch.zeros(_blocks(K) * BLOCK, device=V.device).expand((R + rows - 1) // rows * rows, -1).clone()
    P[:R, :K] = V
    B = P.view(-1, rows, _blocks(K), BLOCK)
    amax = B.abs().amax(dim=(1, 3))
    s = amax / torch.full_like(amax, E4M3_MAX)
    q = torch.where(s[:, None, :, None] > 0, B / s[:, None, :, None], torch.zeros_like(B))
    q = q.clamp(-E4M3_MAX, E4M3_MAX).reshape(P.shape)[:R, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    M, K, dt = case["M"], case["K"], DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "norm":
        S = case["samples"]
        s["H"] = (2.0 * _activations(gen, M, K)).to(dt)
        s["Y"] = _activations(gen, M, K).to(dt)
        s["post_weight"] = 1.0 + 0.1 * _randn(gen, K) if case["post"] != "none" else None
        s["pre_weight"] = 1.0 + 0.1 * _randn(gen, K) if not case["modulate"] else None
        # gate, scale and shift are slices of one modulation row per sample
        mod = 0.3 * _randn(gen, S, 3 * K)
        s["gate_rows"] = mod[:, :K] if case["gate"] else None
        s["scale"] = mod[:, K:2 * K] if case["modulate"] else None
        s["shift"] = mod[:, 2 * K:] if case["modulate"] else None
        # rows of a sample are consecutive; ragged samples come with a row's sample
        cuts = torch.sort(torch.randperm(M, generator=gen, device="cuda")[:S - 1] if S > 1 else
                          torch.empty(0, dtype=torch.int64, device="cuda")).values
        rows = torch.arange(M, device="cuda")
        per = (M + S - 1) // S
        s["sample"] = (torch.bucketize(rows, cuts, right=True) if case["ragged"] else rows // per).to(torch.int32)
        s["rows_per_sample"] = 0 if case["ragged"] else per
        s["H_out"] = torch.empty_like(s["H"])
        if case["out"] == "fp8":
            s["Q"] = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
            s["s"] = torch.empty(M, _blocks(K), device="cuda")
        else:
            s["U"] = torch.empty_like(s["H"])
        return s
    X = _activations(gen, M, K)
    if case["op"] == "pack":
        s["X"] = X.to(dt)
        s["Q"] = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
        s["s"] = torch.empty(M, _blocks(K), device="cuda")
        return s
    if case["packed"]:
        s["Qx"], s["sx"] = _codes(X, 1)
    else:
        s["X"] = X.to(dt)
        s["workspace"] = torch.empty(M * K + 4 * M * _blocks(K) + 1024, dtype=torch.uint8, device="cuda")
    s["Qw"], s["sw"], s["b"], s["Ys"] = [], [], [], []
    for _ in range(case["count"]):
        q, w = _codes(0.02 * _randn(gen, case["N"], K), BLOCK)
        s["Qw"].append(q)
        s["sw"].append(w)
        s["b"].append(0.1 * _randn(gen, case["N"]) if case["bias"] else None)
        s["Ys"].append(torch.empty(M, case["N"], dtype=DTYPES[case["out"]], device="cuda"))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _norm(x, kind, weight):
    if kind == "layer":
        x = x - x.mean(dim=1, keepdim=True)
    if kind != "none":
        x = x / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS)
    return x if weight is None else x * weight


def _widen(s, rows, cols, height):
    """Block scales as one factor per element."""
    return s.repeat_interleave(height, dim=0)[:rows].repeat_interleave(BLOCK, dim=1)[:, :cols]


def _plain(s):
    if s["op"] == "norm":
        sample = s["sample"].long()
        v = _norm(s["Y"].float(), s["post"], s["post_weight"])
        if s["gate_rows"] is not None:
            v = v * s["gate_rows"][sample]
        h = s["H"].float() + v
        u = _norm(h, s["pre"], s["pre_weight"])
        if s["scale"] is not None:
            u = u + u * s["scale"][sample] + s["shift"][sample]
        if s["out"] == "fp8":
            return (h.to(s["H"].dtype), *_codes(u, 1))
        return h.to(s["H"].dtype), u.to(s["H"].dtype)
    if s["op"] == "pack":
        return _codes(s["X"].float(), 1)
    Qx, sx = (s["Qx"], s["sx"]) if s["packed"] else _codes(s["X"].float(), 1)
    X = Qx.float() * _widen(sx, s["M"], s["K"], 1)
    Ys = []
    for q, w, b in zip(s["Qw"], s["sw"], s["b"]):
        y = X @ (q.float() * _widen(w, s["N"], s["K"], BLOCK)).t()
        Ys.append((y if b is None else y + b).to(DTYPES[s["out"]]))
    return Ys


def run(state):
    s = state
    if not own:
        return _plain(s)
    from int8_hadamard_rotated_gb300 import ops
    if s["op"] == "norm":
        kind = {"none": ops.NORM_NONE, "rms": ops.NORM_RMS, "layer": ops.NORM_LAYER}
        args = dict(post_norm=kind[s["post"]], post_eps=EPS, post_weight=s["post_weight"], gate=s["gate_rows"],
                    pre_norm=kind[s["pre"]], pre_eps=EPS, pre_weight=s["pre_weight"], scale=s["scale"],
                    shift=s["shift"], row_sample=s["sample"] if s["ragged"] else None,
                    rows_per_sample=s["rows_per_sample"], H_out=s["H_out"])
        if s["out"] == "fp8":
            return ops.convrot_block_norm_fp8(s["H"], s["Y"], Q=s["Q"], s=s["s"], **args)
        return ops.convrot_block_norm(s["H"], s["Y"], U=s["U"], **args)
    if s["op"] == "pack":
        return ops.fp8_pack_activations(s["X"], Q_x=s["Q"], s_x=s["s"])
    if s["packed"]:
        return ops.fp8_linear_packed(s["Qx"], s["sx"], s["Qw"], s["sw"], s["b"], Ys=s["Ys"])
    return ops.fp8_linear(s["X"], s["Qw"], s["sw"], s["b"], Ys=s["Ys"], workspace=s["workspace"])


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    M, K = case["M"], case["K"]
    size = {"f32": 4, "f16": 2, "bf16": 2}
    b = size[case["dtype"]]
    if case["op"] == "norm":
        vectors = (case["gate"] + 2 * case["modulate"]) * case["samples"] + (case["post"] != "none") + \
            (not case["modulate"])
        out = M * K + 4 * M * _blocks(K) if case["out"] == "fp8" else M * K * b
        return {"bytes": 3 * M * K * b + out + 4 * K * vectors + 4 * M * case["ragged"], "flops": 16 * M * K}
    if case["op"] == "pack":
        return {"bytes": M * K * (b + 1) + 4 * M * _blocks(K), "flops": 3 * M * K}
    x = M * K + 4 * M * _blocks(K) if case["packed"] else M * K * b
    w = case["N"] * K + 4 * _blocks(case["N"]) * _blocks(K) + 4 * case["N"] * case["bias"]
    return {"bytes": x + case["count"] * (w + M * case["N"] * size[case["out"]]),
            "flops": 2 * M * K * case["N"] * case["count"]}


def _exact_norm(x, kind, weight):
    if kind == "rms":
        x = x * (x.square().mean(1, keepdim=True) + EPS).rsqrt()
    elif kind == "layer":
        x = (x - x.mean(1, keepdim=True)) * (x.var(1, correction=0, keepdim=True) + EPS).rsqrt()
    return x if weight is None else x * weight.double()


def _exact_codes(X):
    """e4m3 values and fp32 scales of X (64 bits) per 128 features: the nearest
    multiple, ties to even, of a step that is 2^-3 of the binade and at least 2^-9."""
    Q, scales = [], []
    for k in range(0, X.shape[1], BLOCK):
        x = X[:, k:k + BLOCK]
        s = (x.abs().max(dim=1).values / E4M3_MAX).float().double()
        z = x / torch.where(s > 0, s, 1.0)[:, None]
        step = torch.exp2(torch.floor(torch.log2(z.abs().clamp_min(2.0 ** -6))) - 3.0)
        Q.append(torch.clamp(torch.round(z / step) * step, -E4M3_MAX, E4M3_MAX))
        scales.append(s)
    return torch.cat(Q, 1), torch.stack(scales, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        pick = s["sample"].long()
        v = _exact_norm(s["Y"].double(), case["post"], s["post_weight"])
        if case["gate"]:
            v = v * s["gate_rows"].double()[pick]
        h = s["H"].double() + v
        u = _exact_norm(h, case["pre"], s["pre_weight"])
        if case["modulate"]:
            u = u * (1.0 + s["scale"].double()[pick]) + s["shift"].double()[pick]
        return (h, *_exact_codes(u)) if case["out"] == "fp8" else (h, u)
    if case["op"] == "pack":
        return _exact_codes(s["X"].double())
    Qx, sx = (s["Qx"].double(), s["sx"].double()) if case["packed"] else _exact_codes(s["X"].double())
    Ys = []
    for q, w, b in zip(s["Qw"], s["sw"], s["b"]):
        y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device="cuda")
        for i in range(0, case["N"], BLOCK):
            rows = q[i:i + BLOCK].double()
            for j in range(_blocks(case["K"])):
                k = slice(j * BLOCK, (j + 1) * BLOCK)
                y[:, i:i + BLOCK] += (sx[:, j:j + 1] * w[i // BLOCK, j].double()) * (Qx[:, k] @ rows[:, k].t())
        Ys.append(y if b is None else y + b.double())
    return Ys
