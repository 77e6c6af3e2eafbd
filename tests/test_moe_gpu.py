"""The experts' operators on the GPU against their 64-bit statements
(oracle/moe_oracle.py)."""
import numpy as np
import pytest
import torch

from gpu_common import host
from oracle import block_oracle as bo
from oracle import moe_oracle as mo

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U24 = 2.0 ** -24  # half a step of fp32
INF = float("inf")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def codes(t):
    return host(t.view(torch.uint8))


def dev_codes(Q):
    return torch.from_numpy(Q).cuda().view(torch.float8_e4m3fn)


def activations(seed, M, K, dtype="f32"):
    g = gen(seed)
    X = torch.randn(M, K, generator=g) * (1 + 29 * (torch.rand(K, generator=g) < 0.02))
    return X.to(DT[dtype])


def matrices(seed, E, N, K, bias):
    """The experts' matrices on the device, and as the statement has them."""
    r = np.random.default_rng(seed)
    W = r.normal(size=(E, N, K)).astype(np.float32) * np.float32(K ** -0.5)
    both = [bo.fp8_pack(w, 128) for w in W]
    q, s = np.stack([b[0] for b in both]), np.stack([b[1] for b in both])
    b = r.normal(size=(E, N)).astype(np.float32) * np.float32(0.1) if bias else None
    return (dev_codes(q), torch.from_numpy(s).cuda(), None if b is None else torch.from_numpy(b).cuda()), (q, s, b)


def choices(seed, T, E, k, dropped=0.0, only=None):
    """int32 [T,k] distinct experts per token (of `only`, where given), some -1."""
    r = np.random.default_rng(seed)
    pool = np.arange(E) if only is None else np.asarray(only)
    e = np.stack([r.permutation(pool)[:k] for _ in range(T)]).astype(np.int32)
    e[r.random((T, k)) < dropped] = -1
    w = r.random((T, k)).astype(np.float32)
    return e, w


def assert_within(y, ref, bound):
    """y off by half a step of its type and `bound`."""
    half = torch.finfo(y.dtype).eps / 2
    got = host(y.float()).astype(np.float64)
    bound = half * np.abs(ref) * (1 + half) + bound * (1 + half)
    if y.dtype == torch.float16:
        bound = bound + 2.0 ** -25  # half a subnormal step
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first {np.argwhere(bad)[0]}: {got[bad][0]} against {ref[bad][0]}"


# ---------------------------------------------------------------------------
# the router
# ---------------------------------------------------------------------------

def check_route(ops, logits, k, bias=None, **kw):
    score = {"softmax": ops.MOE_SOFTMAX, "sigmoid": ops.MOE_SIGMOID}
    e, w = ops.moe_route(logits, k, bias=None if bias is None else bias.cuda(),
                         **{n: score[v] if n == "score" else v for n, v in kw.items()})
    eo, wo = mo.route(host(logits.float()), k, bias=None if bias is None else bias.numpy(), **kw)
    np.testing.assert_array_equal(host(e), eo)
    # exp within 2 ulp, sums of up to 1024 scores (37 steps) and up to 32
    # weights, two divisions, the factor
    got = host(w)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(wo))
    np.testing.assert_allclose(got, wo, rtol=64 * U24, atol=1e-38)
    return host(e), got


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (7, 3), (60, 4), (64, 8), (65, 8), (160, 6), (256, 8), (511, 9), (1024, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_route(ops, E, k, score, dtype):
    for T in (1, 5, 130):
        L = (2 * torch.randn(T, E, generator=gen(E + T))).to(DT[dtype]).cuda()  # 16-bit logits are full of ties
        check_route(ops, L, k, score=score, renormalise=E % 2 == 0, scale=1.0 if E < 100 else 2.5)
        check_route(ops, L, k, bias=0.1 * torch.randn(E, generator=gen(E)), score=score)


@pytest.mark.parametrize("E,groups,top,k", [(8, 4, 2, 3), (64, 2, 1, 8), (160, 8, 3, 6), (256, 8, 4, 8), (96, 32, 7, 5),
                                            (1024, 16, 5, 8), (60, 5, 5, 4), (12, 12, 3, 3)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_route_groups(ops, E, groups, top, k, group_top):
    for score, biased, dtype in (("sigmoid", True, "f32"), ("softmax", False, "bf16"), ("softmax", True, "f16"),
                                 ("sigmoid", False, "f32")):
        L = (2 * torch.randn(77, E, generator=gen(E))).to(DT[dtype]).cuda()
        check_route(ops, L, k, bias=0.1 * torch.randn(E, generator=gen(1)) if biased else None, score=score,
                    n_groups=groups, top_groups=top, group_top=group_top)


def test_route_near_ties(ops):
    """Values that fp32 cannot tell apart: saturated sigmoids, scores that the
    bias makes nearly equal, scores that underflow."""
    E = 128
    L = torch.zeros(40, E)
    L[:20] = 18.0 + torch.rand(20, E, generator=gen(0))              # 1 - 1e-8: equal in fp32, not in 64 bits
    L[20:30] = -90.0 - 10 * torch.rand(10, E, generator=gen(1))      # exp(-l) overflows fp32
    L[30:] = 1e-4 * torch.randn(10, E, generator=gen(2))
    for score in ("sigmoid", "softmax"):
        for bias in (torch.zeros(E), -torch.sigmoid(L[35]), 1e-7 * torch.randn(E, generator=gen(3))):
            check_route(ops, L.cuda(), 8, bias=bias, score=score)
            check_route(ops, L.cuda(), 8, bias=bias, score=score, n_groups=8, top_groups=3)
        check_route(ops, L.cuda(), 8, score=score)
        check_route(ops, L.cuda(), 8, score=score, n_groups=4, top_groups=2, group_top=2)


@pytest.mark.parametrize("score,spread", [("sigmoid", 2.0 ** -22), ("softmax", 2.0 ** -16)])
@pytest.mark.parametrize("size", [4.0, 16.0, 60.0, 1000.0])
def test_route_groups_biases_of_opposite_sign(ops, size, score, spread):
    """Groups whose two largest values cancel: the sum is near 0, what their
    roundings may be off by is not. The groups' values lie about such a rounding
    apart."""
    E = 64
    bias = torch.full((E,), -4 * size)
    bias[0::8], bias[1::8] = size, -size
    L = size * spread * torch.randn(500, E, generator=gen(int(size)))
    for top, k in ((1, 2), (3, 6)):
        check_route(ops, L.cuda(), k, bias=bias, score=score, n_groups=8, top_groups=top, group_top=2)


def test_route_groups_whose_sum_overflows(ops):
    """Sums of two values past the fp32 range, next to one at its end."""
    bias = torch.zeros(40)
    for g, (a, b) in enumerate(((3.0e38, 3.0e38), (3.3e38, 3.2e38), (3.4e38, 2.0e31), (3.4e38, 1.0e31), (-3.0e38, -3.0e38))):
        bias[8 * g:8 * g + 8] = -3.2e38
        bias[8 * g + 3], bias[8 * g + 5] = b, a
    L = torch.randn(20, 40, generator=gen(12))
    for top in range(1, 6):
        check_route(ops, L.cuda(), 2 * top, bias=bias, score="sigmoid", n_groups=5, top_groups=top, group_top=2)


def test_route_closed_and_bad(ops):
    E = 24
    L = torch.randn(12, E, generator=gen(4))
    L[0] = -INF                     # nothing open
    L[1, 1:] = -INF                 # one
    L[2, 5:] = -INF                 # fewer than k
    L[3, 2] = float("nan")
    L[4, 3] = INF                   # softmax: no scores; sigmoid: 1
    L[5] = -3.0e38                  # finite, far from 0
    L[6, 0] = 3.0e38
    L[7, :12] = -INF                # whole groups
    L[8] = 0.0                      # all equal
    L[9, ::2] = -0.0
    L[9, 1::2] = 0.0
    bias = 0.2 * torch.randn(E, generator=gen(5))
    closing = bias.clone()
    closing[3] = -INF
    pushing = bias.clone()
    pushing[4] = INF
    for score in ("softmax", "sigmoid"):
        for b in (None, bias, closing, pushing):
            for groups in (dict(), dict(n_groups=4, top_groups=2, group_top=2), dict(n_groups=4, top_groups=2, group_top=1)):
                for r in (False, True):
                    e, w = check_route(ops, L.cuda(), 8, bias=b, score=score, renormalise=r, **groups)
        assert (e[0] == -1).all() and (w[0] == 0).all()
        assert np.isnan(w[3]).all() and (e[3] == np.arange(8)).all()
    nan = bias.clone()
    nan[7] = float("nan")
    e, w = check_route(ops, L.cuda(), 8, bias=nan)
    assert np.isnan(w).all()


def test_route_rows_apart(ops):
    base = torch.randn(33, 300, generator=gen(6)).cuda()
    for off, E in ((0, 64), (1, 65), (37, 256)):
        check_route(ops, base[:, off:off + E], 8)
    e, w = ops.moe_route(torch.empty(0, 16, device="cuda"), 4)
    assert e.shape == w.shape == (0, 4)


# ---------------------------------------------------------------------------
# the plan
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n,E", [(0, 5), (1, 1), (1, 1024), (31, 3), (32, 8), (33, 8), (1000, 60), (2049, 128),
                                 (4097, 256), (20000, 7), (65536, 256), (70001, 1024)])
def test_plan(ops, n, E):
    r = np.random.default_rng(n)
    e = r.integers(-1, E, size=n).astype(np.int32)
    if n > 100:
        e[10:90] = E - 1            # a run of one expert
        e[e == E // 2] = -1         # and an expert without rows
    order, place, offsets = (host(t) for t in ops.moe_plan(torch.from_numpy(e).cuda(), E))
    flat = np.where(e < 0, E, e)
    sort = np.argsort(flat, kind="stable").astype(np.int32)
    assert (offsets == np.searchsorted(flat[sort], np.arange(E + 1))).all()
    assert (order == np.where(np.arange(n) < offsets[E], sort, -1)).all()
    back = np.empty(n, np.int32)
    back[sort] = np.arange(n)
    assert (place == np.where(e < 0, -1, back)).all()
    if n <= 5000:
        for got, want in zip((order, place, offsets), mo.plan(e, E)):
            np.testing.assert_array_equal(got, want)
    assert ops.convrot_device_status() == ops.OK


@pytest.mark.parametrize("n,E", [(3000, 151), (3000, 152), (3000, 303), (3000, 304), (3000, 400), (5000, 607), (5000, 608),
                                 (9000, 1024), (12288, 64), (12288, 500), (12288, 1024), (12289, 64), (12289, 500),
                                 (12289, 1024), (300000, 130)])
def test_plan_at_its_borders(ops, n, E):
    """Where the experts per CTA change, and at the most choices of one launch."""
    r = np.random.default_rng(n + E)
    e = np.where(r.random(n) < 0.3, r.integers(0, 9, size=n), r.integers(-1, E, size=n)).astype(np.int32)
    e[e == E // 2] = -1
    order, place, offsets = (host(t) for t in ops.moe_plan(torch.from_numpy(e).cuda(), E))
    flat = np.where(e < 0, E, e)
    sort = np.argsort(flat, kind="stable").astype(np.int32)
    np.testing.assert_array_equal(offsets, np.searchsorted(flat[sort], np.arange(E + 1)))
    np.testing.assert_array_equal(order, np.where(np.arange(n) < offsets[E], sort, -1))
    back = np.empty(n, np.int32)
    back[sort] = np.arange(n)
    np.testing.assert_array_equal(place, np.where(e < 0, -1, back))
    assert ops.convrot_device_status() == ops.OK


def test_plan_out_of_range(ops):
    """Experts outside [-1, E) are dropped and reported."""
    for bad in (-2, 4, 2 ** 31 - 1, -2 ** 31):
        e = np.int32([0, 3, bad, 1, -1, 3])
        order, place, offsets = (host(t) for t in ops.moe_plan(torch.from_numpy(e).cuda(), 4))
        np.testing.assert_array_equal(order, [0, 3, 1, 5, -1, -1])
        np.testing.assert_array_equal(place, [0, 2, -1, 1, -1, 3])
        np.testing.assert_array_equal(offsets, [0, 1, 2, 2, 4])
        assert ops.convrot_device_status() == ops.ERR_ARG
        assert ops.convrot_device_status() == ops.OK


# ---------------------------------------------------------------------------
# the experts' linears
# ---------------------------------------------------------------------------

# (T, E, k, only): rows per expert from none to many, one expert that has all
SPREADS = [(1, 8, 1, None), (1, 8, 8, None), (3, 16, 2, None), (9, 4, 2, None), (40, 5, 3, None), (150, 6, 2, [1, 4]),
           (200, 3, 1, [1]), (700, 4, 2, None)]


def planned(seed, T, E, k, only, dropped):
    e, w = choices(seed, T, E, k, dropped, only)
    order, place, offsets = mo.plan(e, E)
    t = [torch.from_numpy(a).cuda() for a in (order, place, offsets)]
    return e, w, (order, place, offsets), t


@pytest.mark.parametrize("T,E,k,only", SPREADS)
@pytest.mark.parametrize("N,K", [(16, 16), (128, 128), (131, 656), (640, 1040)])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_expert_linear(ops, T, E, k, only, N, K, out):
    bias = N != 128
    _, _, (order, _, offsets), (d_order, _, d_offsets) = planned(T + N, T, E, k, only, 0.1 if T > 1 else 0.0)
    n, rows = T * k, int(offsets[E])
    dw, hw = matrices(N, E, N, K, bias)
    for gather in (False, True):
        Q, s = bo.fp8_pack(activations(T, T if gather else n, K).numpy())
        ref, mag = mo.expert_linear(Q, s, order[:rows] // k if gather else np.arange(rows), offsets, *hw)
        y = torch.full((n, N), 7.0, dtype=DT[out], device="cuda")
        ops.fp8_expert_linear(dev_codes(Q), torch.from_numpy(s).cuda(), d_offsets, dw,
                              order=d_order if gather else None, top_k=k, Y=y)
        assert_within(y[:rows], ref, mo.linear_error(mag, K))
        assert (host(y[rows:].float()) == 7.0).all()  # rows behind the last one stay as they were
    assert ops.convrot_device_status() == ops.OK


@pytest.mark.parametrize("T,E,k,only", SPREADS)
@pytest.mark.parametrize("I,K", [(16, 16), (128, 128), (144, 656), (656, 400)])
def test_expert_swiglu(ops, T, E, k, only, I, K):  # noqa: E741
    bias = I != 128
    _, _, (order, _, offsets), (d_order, _, d_offsets) = planned(T + I, T, E, k, only, 0.1 if T > 1 else 0.0)
    n, rows = T * k, int(offsets[E])
    dg, hg = matrices(I, E, I, K, bias)
    du, hu = matrices(I + 1, E, I, K, bias)
    for gather in (False, True):
        Q, s = bo.fp8_pack(activations(T, T if gather else n, K).numpy())
        src = order[:rows] // k if gather else np.arange(rows)
        g, ga = mo.expert_linear(Q, s, src, offsets, *hg)
        u, ua = mo.expert_linear(Q, s, src, offsets, *hu)
        h, dh = mo.swiglu(g, u, mo.linear_error(ga, K), mo.linear_error(ua, K))
        Qh = torch.full((n, I), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        sh = torch.full((n, bo.n_blocks(I)), 7.0, device="cuda")
        ops.fp8_expert_swiglu(dev_codes(Q), torch.from_numpy(s).cuda(), d_order if gather else None, d_offsets, k, dg,
                              du, Q_h=Qh, s_h=sh)
        got, sc = codes(Qh), host(sh)
        assert (got[rows:] == 0x55).all() and (sc[rows:] == 7.0).all()
        S = bo.widen(sc[:rows], rows, I)
        value = bo.e4m3_values()[got[:rows]] * S
        # the scale: the largest magnitude over 448; the codes: nearest
        for j in range(bo.n_blocks(I)):
            b = slice(128 * j, 128 * (j + 1))
            top, off = np.abs(h[:, b]).max(1), dh[:, b].max(1)
            assert (np.abs(sc[:rows, j] * 448.0 - top) <= off + top * 2 * U24).all()
        half = np.maximum(2.0 ** -4 * np.maximum(np.abs(value), np.abs(h)), 2.0 ** -10 * S)
        assert (np.abs(value - h) <= half * (1 + 1e-6) + dh + np.abs(h) * 4 * U24).all()
    assert ops.convrot_device_status() == ops.OK


@pytest.mark.parametrize("T,E,k,N,I,K", [(1, 1, 1, 1, 16, 48), (130, 1, 1, 1, 144, 272), (20, 1024, 4, 40, 32, 144),
                                          (2, 300, 8, 7, 48, 16), (6, 2, 1, 260, 144, 4240), (400, 2, 2, 33, 272, 4240)])
def test_expert_extremes(ops, T, E, k, N, I, K):  # noqa: E741
    """One expert and the most experts, one output feature, long K."""
    _, _, (order, _, offsets), (d_order, _, d_offsets) = planned(T, T, E, k, None, 0.0)
    dw, hw = matrices(1, E, N, K, True)
    dg, hg = matrices(2, E, I, K, True)
    du, hu = matrices(3, E, I, K, False)
    Q, s = bo.fp8_pack(activations(T, T, K).numpy())
    x, sx = dev_codes(Q), torch.from_numpy(s).cuda()
    src = order // k
    ref, mag = mo.expert_linear(Q, s, src, offsets, *hw)
    y = ops.fp8_expert_linear(x, sx, d_offsets, dw, order=d_order, top_k=k, out_dtype=torch.float32)
    assert_within(y, ref, mo.linear_error(mag, K))
    g, ga = mo.expert_linear(Q, s, src, offsets, *hg)
    u, ua = mo.expert_linear(Q, s, src, offsets, *hu)
    h, dh = mo.swiglu(g, u, mo.linear_error(ga, K), mo.linear_error(ua, K))
    Qh, sh = ops.fp8_expert_swiglu(x, sx, d_order, d_offsets, k, dg, du)
    S = bo.widen(host(sh), T * k, I)
    value = bo.e4m3_values()[codes(Qh)] * S
    half = np.maximum(2.0 ** -4 * np.maximum(np.abs(value), np.abs(h)), 2.0 ** -10 * S)
    assert (np.abs(value - h) <= half * (1 + 1e-6) + dh + np.abs(h) * 4 * U24).all()
    assert ops.convrot_device_status() == ops.OK


def test_expert_strides(ops):
    """Gate and up as halves of one array, experts apart; a Y with rows apart and at odd offsets."""
    E, I, K, T, k = 5, 144, 272, 70, 2  # noqa: E741
    _, _, (order, _, offsets), (d_order, _, d_offsets) = planned(3, T, E, k, None, 0.0)
    dg, _ = matrices(1, E, I, K, True)
    du, _ = matrices(2, E, I, K, True)
    q = torch.cat([dg[0].view(torch.uint8), du[0].view(torch.uint8)], 1).view(torch.float8_e4m3fn)
    s = torch.cat([dg[1], du[1]], 1)
    b = torch.cat([dg[2], du[2]], 1)
    nb = bo.n_blocks(I)
    Q, sx = ops.fp8_pack_activations(activations(4, T, K).cuda())
    want = ops.fp8_expert_swiglu(Q, sx, d_order, d_offsets, k, dg, du)
    got = ops.fp8_expert_swiglu(Q, sx, d_order, d_offsets, k, (q[:, :I], s[:, :nb], b[:, :I]),
                                (q[:, I:], s[:, nb:], b[:, I:]))
    assert (codes(got[0]) == codes(want[0])).all() and (host(got[1]) == host(want[1])).all()
    y = ops.fp8_expert_linear(Q, sx, d_offsets, dg, order=d_order, top_k=k)
    for off in (0, 1, 8):
        base = torch.zeros(T * k, I + 24, dtype=torch.bfloat16, device="cuda")
        ops.fp8_expert_linear(Q, sx, d_offsets, dg, order=d_order, top_k=k, Y=base[:, off:off + I])
        assert (host(base[:, off:off + I].float()) == host(y.float())).all()
        assert (host(base[:, :off].float()) == 0).all() and (host(base[:, off + I:].float()) == 0).all()


@pytest.mark.parametrize("rows", [[3] * 8, [130] * 8])
def test_swiglu_gates_far_below_zero(ops, rows):
    """Gates around where their sigmoid leaves the normal fp32 range (-87.3), next
    to up values that bring the products back: activations of zeros, so that g
    and u are the biases."""
    base = (-20.0, -60.0, -80.0, -87.0, -88.0, -90.0, -95.0, -101.0)
    E, K, I = len(base), 128, 144  # noqa: E741
    r = np.random.default_rng(1)
    g = (np.array(base)[:, None] - r.random((E, I))).astype(np.float32)
    u = (r.choice([-1.0, 1.0], (E, I)) * (1 + r.random((E, I))) * 1e30).astype(np.float32)
    q, s, _ = matrices(1, E, I, K, False)[0]
    n = sum(rows)
    x, sx = ops.fp8_pack_activations(torch.zeros(n, K, device="cuda"))
    offsets = torch.tensor([0] + rows).cumsum(0).to(torch.int32).cuda()
    Qh, sh = ops.fp8_expert_swiglu(x, sx, None, offsets, 1, (q, s, torch.from_numpy(g).cuda()),
                                   (q, s, torch.from_numpy(u).cuda()))
    S = bo.widen(host(sh), n, I)
    value = bo.e4m3_values()[codes(Qh)] * S
    which = np.repeat(np.arange(E), rows)
    zero = np.zeros((n, I))
    h, dh = mo.swiglu(g[which].astype(np.float64), u[which].astype(np.float64), zero, zero)
    # a sigmoid below 2^-126 is a multiple of 2^-149: half a step of its rounding, and of the exponential's
    dh = dh + np.abs(g[which].astype(np.float64) * u[which]) * 2.0 ** -149
    half = np.maximum(2.0 ** -4 * np.maximum(np.abs(value), np.abs(h)), 2.0 ** -10 * S)
    assert (np.abs(value - h) <= half * (1 + 1e-6) + dh + np.abs(h) * 4 * U24).all()


@pytest.mark.parametrize("E,rows", [(1, 5), (3, 4), (40, 3), (60, 20), (12, 40), (4, 100)])
@pytest.mark.parametrize("K", [512, 2048, 4096])
def test_results_whatever_the_scales_alignment(ops, E, rows, K):
    """The same values in scale arrays that start on 16 bytes, and on 4, with
    experts an odd distance apart: the same bits."""
    n, N = E * rows, 272
    r = np.random.default_rng(E)

    def codes_(*shape):
        return torch.from_numpy(r.integers(0, 0x70, shape).astype(np.uint8) | r.integers(0, 2, shape).astype(np.uint8) << 7)

    def scales(*shape):
        return torch.from_numpy((2.0 ** r.uniform(-6, 2, shape)).astype(np.float32)).cuda()

    def odd(t):  # the same, 4 bytes past a 16-byte boundary, the first axis apart by one more
        base = torch.zeros(1 + t.shape[0] * (t[0].numel() + 1), device="cuda")
        v = base[1:].view(t.shape[0], -1)[:, :-1].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 16 == 4
        return v

    x, q, q2 = (codes_(*d).cuda().view(torch.float8_e4m3fn) for d in ((n, K), (E, N, K), (E, N, K)))
    sx, s, s2 = scales(n, K // 128), scales(E, 3, K // 128), scales(E, 3, K // 128)
    offsets = (torch.arange(E + 1, dtype=torch.int32) * rows).cuda()
    base = torch.zeros(1 + sx.numel(), device="cuda")
    sx_odd = base[1:].view(sx.shape).copy_(sx)
    y = ops.fp8_expert_linear(x, sx, offsets, (q, s), out_dtype=torch.float32)
    h = ops.fp8_expert_swiglu(x, sx, None, offsets, 1, (q, s), (q2, s2))
    for args in ((sx_odd, s, s2), (sx, odd(s), odd(s2)), (sx_odd, odd(s), s2)):
        assert torch.equal(ops.fp8_expert_linear(x, args[0], offsets, (q, args[1]), out_dtype=torch.float32), y)
        z = ops.fp8_expert_swiglu(x, args[0], None, offsets, 1, (q, args[1]), (q2, args[2]))
        assert (codes(z[0]) == codes(h[0])).all() and torch.equal(z[1], h[1])


@pytest.mark.parametrize("E", [9, 20, 70, 300])
def test_many_rows_of_many_experts(ops, E):
    """The kernel for many rows per expert past its first eight and its first 32
    experts: uneven ones, whole eights without rows, several tiles of one."""
    r = np.random.default_rng(E)
    counts = r.integers(1, 180, size=E)
    counts[r.random(E) < 0.2] = 0
    counts[8:16] = 0
    counts[-3] = 700
    if E > 60:
        counts[24:48] = 0
        counts[64:66] = 256, 257
    short = 66 * E - counts.sum()  # over 64 rows on average
    if short > 0:
        counts[E - 2] += short
    e = r.permutation(np.repeat(np.arange(E), counts)).astype(np.int32)
    n, N, I, K = e.size, 40, 48, 144  # noqa: E741
    assert n // E > 64
    order = np.argsort(e, kind="stable").astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    d_order, d_offsets = torch.from_numpy(order).cuda(), torch.from_numpy(offsets).cuda()
    dw, hw = matrices(1, E, N, K, True)
    dg, hg = matrices(2, E, I, K, True)
    du, hu = matrices(3, E, I, K, False)
    Q, s = bo.fp8_pack(activations(E, n, K).numpy())
    x, sx = dev_codes(Q), torch.from_numpy(s).cuda()
    for src, d in ((order, d_order), (np.arange(n), None)):
        ref, mag = mo.expert_linear(Q, s, src, offsets, *hw)
        assert_within(ops.fp8_expert_linear(x, sx, d_offsets, dw, order=d), ref, mo.linear_error(mag, K))
        g, ga = mo.expert_linear(Q, s, src, offsets, *hg)
        u, ua = mo.expert_linear(Q, s, src, offsets, *hu)
        h, dh = mo.swiglu(g, u, mo.linear_error(ga, K), mo.linear_error(ua, K))
        Qh, sh = ops.fp8_expert_swiglu(x, sx, d, d_offsets, 1, dg, du)
        S = bo.widen(host(sh), n, I)
        value = bo.e4m3_values()[codes(Qh)] * S
        half = np.maximum(2.0 ** -4 * np.maximum(np.abs(value), np.abs(h)), 2.0 ** -10 * S)
        assert (np.abs(value - h) <= half * (1 + 1e-6) + dh + np.abs(h) * 4 * U24).all()
    assert ops.convrot_device_status() == ops.OK


def test_prepare_experts(ops):
    W = torch.randn(3, 130, 272, generator=gen(1)).cuda()
    Q, s = ops.fp8_prepare_experts(W)
    for e in range(3):
        q, t = ops.fp8_prepare_weight(W[e])
        assert (codes(Q[e]) == codes(q)).all() and (host(s[e]) == host(t)).all()


# ---------------------------------------------------------------------------
# the weighted sum, and all of it
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 8, 4096), (7, 3, 131), (33, 8, 640), (300, 32, 24)])
@pytest.mark.parametrize("rows,out", [("bf16", "bf16"), ("f32", "f16"), ("f16", "f32")])
def test_combine(ops, T, k, N, rows, out):
    r = np.random.default_rng(T + N)
    n = T * k
    R = torch.from_numpy(r.normal(size=(n, N)).astype(np.float32)).to(DT[rows]).cuda()
    place = r.permutation(n).astype(np.int32).reshape(T, k)
    place[r.random((T, k)) < 0.2] = -1
    w = r.normal(size=(T, k)).astype(np.float32)
    w[place < 0] = np.nan  # a choice without a row adds nothing, whatever its weight
    res = torch.from_numpy(r.normal(size=(T, N)).astype(np.float32)).to(DT[out]).cuda()
    for residual in (None, res):
        ref, mag = mo.combine(host(R.float()).astype(np.float64), place, w,
                              None if residual is None else host(res.float()))
        y = ops.moe_combine(R, torch.from_numpy(place).cuda(), torch.from_numpy(w).cuda(), residual=residual,
                            Y=torch.full((T, N), 9.0, dtype=DT[out], device="cuda"))
        assert_within(y, ref, (k + 1) * U24 * mag)
    z = res.clone()
    ops.moe_combine(R, torch.from_numpy(place).cuda(), torch.from_numpy(w).cuda(), residual=z, Y=z)
    assert (host(z.float()) == host(y.float())).all()


@pytest.mark.parametrize("T,E,k,only", SPREADS + [(2, 8, 4, None), (4, 8, 2, [2, 5]), (8, 16, 3, None), (9, 16, 3, None),
                                                  (64, 32, 4, None)])
@pytest.mark.parametrize("K,I,N,dtype,out", [(256, 128, 256, "bf16", "bf16"), (400, 144, 264, "f16", "f16"),
                                             (1040, 656, 133, "f32", "f32")])
def test_moe(ops, T, E, k, only, K, I, N, dtype, out):  # noqa: E741
    e, w = choices(T + K, T, E, k, 0.1 if T > 2 else 0.0, only)
    bias = K != 256
    dg, hg = matrices(1, E, I, K, bias)
    du, hu = matrices(2, E, I, K, bias)
    dd, hd = matrices(3, E, N, I, bias)
    X = activations(T, T, K, dtype)
    res = torch.randn(T, N, generator=gen(T)).to(DT[out]) if N != 264 else None
    ref, bound = mo.moe(X.float().numpy(), e, w, hg, hu, hd, None if res is None else res.float().numpy(),
                        rows_error=2.0 ** -11 if out == "bf16" else 0.0)  # rows in binary16 there
    y = ops.fp8_moe(X.cuda(), torch.from_numpy(e).cuda(), torch.from_numpy(w).cuda(), dg, du, dd,
                    residual=None if res is None else res.cuda(),
                    Y=torch.full((T, N), float("nan"), dtype=DT[out], device="cuda"))
    assert_within(y, ref, bound)
    assert ops.convrot_device_status() == ops.OK


@pytest.mark.parametrize("T,E,k,out,dtype", [(5, 200, 8, "bf16", "bf16"), (40, 200, 4, "f32", "f16"), (30, 303, 6, "bf16", "f32"),
                                             (30, 304, 6, "bf16", "bf16"), (60, 700, 8, "f16", "f16"), (25, 1024, 8, "f32", "f32"),
                                             (3300, 400, 4, "bf16", "bf16"), (3080, 300, 4, "f32", "f32")])
def test_moe_many_experts(ops, T, E, k, out, dtype):
    """The plans of more experts and choices inside fp8_moe."""
    K, I, N = 48, 32, 24  # noqa: E741
    e, w = choices(T, T, E, k, 0.1)
    dg, hg = matrices(1, E, I, K, True)
    du, hu = matrices(2, E, I, K, True)
    dd, hd = matrices(3, E, N, I, True)
    X = activations(T, T, K, dtype)
    ref, bound = mo.moe(X.float().numpy(), e, w, hg, hu, hd, rows_error=2.0 ** -11 if out == "bf16" else 0.0)
    y = ops.fp8_moe(X.cuda(), torch.from_numpy(e).cuda(), torch.from_numpy(w).cuda(), dg, du, dd, out_dtype=DT[out])
    assert_within(y, ref, bound)
    assert ops.convrot_device_status() == ops.OK


@pytest.mark.parametrize("k", [9, 12, 32])
@pytest.mark.parametrize("T", [3, 200])
def test_moe_many_choices_of_a_token(ops, T, k):
    """More rows than the weighted sum takes at once, with their powers of two."""
    E, K, I, N = 36, 144, 48, 264  # noqa: E741
    e, w = choices(T, T, E, k, 0.2)
    dg, hg = matrices(1, E, I, K, True)
    du, hu = matrices(2, E, I, K, True)
    dd, hd = matrices(3, E, N, I, True)
    X = activations(T, T, K, "bf16")
    ref, bound = mo.moe(X.float().numpy(), e, w, hg, hu, hd, rows_error=2.0 ** -11)
    y = ops.fp8_moe(X.cuda(), torch.from_numpy(e).cuda(), torch.from_numpy(w).cuda(), dg, du, dd)
    assert_within(y, ref, bound)


@pytest.mark.parametrize("T", [1, 40, 900])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_moe_strides(ops, T, dtype):
    """Rows of X, Y and the residual apart and at odd offsets, the residual in
    place: the results of dense arrays, and nothing written beside them."""
    E, k, K, I, N = 8, 2, 272, 144, 200  # noqa: E741
    X, e, w, gate, up, down = block(ops, T, E, k, K, I, N, T)
    X = X.to(DT[dtype])
    res = torch.randn(T, N, generator=gen(T)).to(DT[dtype]).cuda()
    want = ops.fp8_moe(X, e, w, gate, up, down, residual=res)
    plain = ops.fp8_moe(X, e, w, gate, up, down)
    for off in (1, 8):
        wide = torch.full((T, K + 25), 100.0, dtype=DT[dtype], device="cuda")
        wide[:, off:off + K] = X
        x = wide[:, off:off + K]
        y = torch.full((T, N + 19), 5.0, dtype=DT[dtype], device="cuda")
        y[:, off:off + N] = res
        z = y[:, off:off + N]
        assert torch.equal(ops.fp8_moe(x, e, w, gate, up, down), plain)
        assert torch.equal(ops.fp8_moe(x, e, w, gate, up, down, residual=z, Y=z), want)
        assert (y[:, :off] == 5).all() and (y[:, off + N:] == 5).all()
    z = res.clone()
    assert torch.equal(ops.fp8_moe(X, e, w, gate, up, down, residual=z, Y=z), want)


# ---------------------------------------------------------------------------
# the operators together
# ---------------------------------------------------------------------------

def block(ops, T, E, k, K, I, N, seed=0):  # noqa: E741
    """(X, experts, weights, gate, up, down) on the device, of random matrices packed there."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    mats = [(*ops.fp8_prepare_experts(r(E, n, m) * m ** -0.5), 0.1 * r(E, n)) for n, m in ((I, K), (I, K), (N, I))]
    e, w = ops.moe_route(r(T, E), k)
    return (r(T, K).to(torch.bfloat16), e, w, *mats)


@pytest.mark.parametrize("T,E,k", [(1, 16, 4), (5, 8, 2), (100, 16, 4), (300, 6, 2), (2000, 8, 4)])
def test_moe_is_its_parts(ops, T, E, k):
    """fp8_moe gives what the pack, the plan, the linears and the sum give one by one."""
    X, e, w, gate, up, down = block(ops, T, E, k, 400, 272, 384, T)
    e[T // 3] = -1
    res = torch.randn(T, 384, generator=gen(T)).cuda()
    got = ops.fp8_moe(X, e, w, gate, up, down, residual=res)
    assert got.dtype == torch.float32
    order, place, offsets = ops.moe_plan(e, E)
    h = ops.fp8_expert_swiglu(*ops.fp8_pack_activations(X), order, offsets, k, gate, up)
    rows = ops.fp8_expert_linear(*h, offsets, down, out_dtype=torch.float32)
    want = ops.moe_combine(rows, place, w, residual=res)
    assert torch.equal(got, want)
    assert ops.convrot_device_status() == ops.OK


def test_block_with_experts(ops):
    """A transformer block's MLP: norm, router, experts, residual; against 64 bits."""
    T, E, k, K, I = 90, 12, 3, 256, 144  # noqa: E741
    X, _, _, gate, up, down = block(ops, T, E, k, K, I, K, 7)
    router = torch.randn(E, K, generator=gen(8)).cuda() * K ** -0.5
    h, u = ops.convrot_block_norm(X, want_h=True)
    logits = u.float() @ router.t()
    e, w = ops.moe_route(logits, k, score=ops.MOE_SIGMOID, bias=0.05 * torch.randn(E, generator=gen(9)).cuda(), n_groups=4,
                         top_groups=2, scale=2.0)
    y = ops.fp8_moe(u, e, w, gate, up, down, residual=h)
    sets = [(codes(q), host(s), host(b)) for q, s, b in (gate, up, down)]
    ref, bound = mo.moe(host(u.float()), host(e), host(w), *sets, host(h.float()), rows_error=2.0 ** -11)
    assert_within(y, ref, bound)


def test_results_repeat(ops):
    """Bit for bit, also next to another call on another stream."""
    for T in (1, 40, 700):
        args = block(ops, T, 16, 4, 512, 256, 384, T)
        other = block(ops, 600, 16, 4, 512, 256, 384, T + 1)
        first = ops.fp8_moe(*args)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            z = ops.fp8_moe(*other, stream=side)
            assert torch.equal(ops.fp8_moe(*args), first)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(ops.fp8_moe(*other), z)
    assert ops.convrot_device_status() == ops.OK


@pytest.mark.parametrize("T", [1, 30, 500])
def test_captured_and_replayed(ops, T):
    """One graph of router, experts and sum, replayed on new inputs whose tokens
    choose other experts."""
    E, k, K, I, N = 8, 2, 256, 128, 200  # noqa: E741
    X, _, _, gate, up, down = block(ops, T, E, k, K, I, N)
    logits = torch.zeros(T, E, device="cuda")
    ws = torch.empty(ops.fp8_moe_workspace_size(T, K, I, N, k, E), dtype=torch.uint8, device="cuda")
    Y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")

    def run():
        e, w = ops.moe_route(logits, k)
        ops.fp8_moe(X, e, w, gate, up, down, Y=Y, workspace=ws)
        return e

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(4):
        g = torch.Generator(device="cuda").manual_seed(i)
        X.copy_(torch.randn(T, K, generator=g, device="cuda"))
        logits.copy_(torch.randn(T, E, generator=g, device="cuda") * 3)
        if i == 3:
            logits.fill_(-INF)  # no expert open: nothing is added
        Y.fill_(9.0)
        graph.replay()
        got = Y.clone()
        run()
        assert torch.equal(Y, got)
    assert (got == 0).all()


@pytest.mark.parametrize("counts", [[3, 5, 2], [40, 50, 30], [300, 20, 90]])
def test_non_finite_rows_stay_in_their_rows(ops, counts):
    """Infinities and NaN in some rows, next to others in the same tiles; rows
    behind the last one full of NaN codes."""
    E, K, I = len(counts), 272, 144  # noqa: E741
    n, total = sum(counts), sum(counts) + 37
    X = activations(3, total, K)
    clean = X.clone()
    bad = [0, counts[0], n - 1]
    X[0, 5], X[counts[0], 9], X[n - 1, 200] = INF, float("nan"), -INF
    X[n:] = float("nan")
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    gate, up = matrices(1, E, I, K, True)[0], matrices(2, E, I, K, True)[0]
    down = matrices(3, E, 200, I, True)[0]
    out = []
    for x in (X, clean):
        Qh = torch.zeros(total, I, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        h = ops.fp8_expert_swiglu(*ops.fp8_pack_activations(x.cuda()), None, offsets, 1, gate, up, Q_h=Qh,
                                  s_h=torch.zeros(total, 2, device="cuda"))
        y = ops.fp8_expert_linear(*h, offsets, down, Y=torch.zeros(total, 200, device="cuda"))
        out.append((codes(h[0]), host(h[1]), host(y)))
    good = [i for i in range(total) if i not in bad]
    for a, b in zip(*out):
        assert (a[good] == b[good]).all()
    assert not np.isfinite(out[0][2][bad]).any() and np.isfinite(out[0][2][good]).all()


def test_bf16_rows_keep_their_precision(ops):
    """fp8_moe's bf16 output, whose rows pass in binary16 with a power of two:
    large, small and zero rows, and outputs of an odd width."""
    T, E, k, K, I, N = 70, 4, 2, 128, 128, 133  # noqa: E741
    X, e, w, gate, up, down = block(ops, T, E, k, K, I, N, 5)
    for factor in (1.0, 1e30, 1e-30, 0.0):
        d = (down[0], down[1] * factor, down[2] * factor)
        want = ops.fp8_moe(X, e, w, gate, up, d, out_dtype=torch.float32)
        got = ops.fp8_moe(X, e, w, gate, up, d)
        order, place, offsets = ops.moe_plan(e, E)
        rows = ops.fp8_expert_linear(*ops.fp8_expert_swiglu(*ops.fp8_pack_activations(X), order, offsets, k, gate, up),
                                     offsets, d, out_dtype=torch.float32)
        mag = host(ops.moe_combine(rows.abs(), place, w)).astype(np.float64)
        # half a step of bf16, and half one of binary16 for every row
        bound = 2.0 ** -8 * np.abs(host(want)) + 2.0 ** -11 * mag * 1.01 + 8 * U24 * mag
        assert (np.abs(host(got.float()).astype(np.float64) - host(want)) <= bound).all(), factor


@pytest.mark.parametrize("T", [20, 700])
@pytest.mark.parametrize("size", [1.0, 1e30, 1e-30])
def test_bf16_rows_of_a_wide_range(ops, T, size):
    """Rows whose features differ by up to 2^60 within their block of 128: each is
    off by half a step of binary16, or by 2^-39 of the block's largest where that
    is more. Down matrices of zeros: the rows are the biases."""
    E, k, K, I, N = 6, 3, 128, 128, 272  # noqa: E741
    X, e, w, gate, up, down = block(ops, T, E, k, K, I, N, 5)
    r = np.random.default_rng(3)
    bias = (r.choice([-1.0, 1.0], (E, N)) * 2.0 ** r.uniform(-60, 0, (E, N)) * size).astype(np.float32)
    y = ops.fp8_moe(X, e, w, gate, up, (torch.zeros(E, N, I, device="cuda").to(torch.float8_e4m3fn),
                                        torch.ones(E, bo.n_blocks(N), 1, device="cuda"), torch.from_numpy(bias).cuda()))
    b = bias.astype(np.float64)
    top = bo.widen(np.stack([np.abs(b[:, j:j + 128]).max(1) for j in range(0, N, 128)], 1), E, N)
    off = np.maximum(2.0 ** -11 * np.abs(b), 2.0 ** -39 * top)
    rows = host(e).reshape(-1)  # a choice's row is its expert's
    place = np.arange(T * k, dtype=np.int32).reshape(T, k)
    ref, mag = mo.combine(b[rows], place, host(w))
    bound, _ = mo.combine(off[rows], place, host(w))
    # below 2^-126 bf16 values are multiples of 2^-126 2^-7: half a step is 2^-134,
    # where half a step relative to the value would be less
    assert_within(y, ref, bound + (k + 2) * U24 * mag + 2.0 ** -134)


def test_rows_past_31_bits(ops):
    """Sorted codes, outputs and rows of more than 2^31 bytes and elements."""
    T, k, E, K, N = 37500, 8, 4, 8192, 16
    n = T * k
    g = torch.Generator(device="cuda").manual_seed(1)
    e = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    X = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    Q, s = ops.fp8_pack_activations(X)
    W = (*ops.fp8_prepare_experts(torch.randn(E, N, K, generator=g, device="cuda")), None)
    order, place, offsets = ops.moe_plan(e, E)
    wide = torch.empty(n, 8192, dtype=torch.bfloat16, device="cuda")  # 2.5e9 elements
    y = ops.fp8_expert_linear(Q, s, offsets, W, order=order, top_k=k, Y=wide[:, 8176:])
    few = torch.arange(n - 40, n, device="cuda")
    t = order[few] // k
    x = ops.fp8_expert_linear(Q[t.long()].contiguous(), s[t.long()].contiguous(),
                              torch.tensor([0, 0, 0, 0, 40], dtype=torch.int32, device="cuda"), W)
    assert torch.allclose(y[few].float(), x.float(), rtol=2.0 ** -7, atol=1e-3 * float(x.float().abs().max()))
    w = torch.rand(T, k, generator=g, device="cuda")
    z = ops.moe_combine(wide[:, 8176:], place, w, out_dtype=torch.float32)
    last = place[-8:].long()
    want = (w[-1].double()[:, None] * wide[last][:, 8176:].double()).sum(0)
    assert torch.allclose(z[-1].double(), want, rtol=1e-5, atol=1e-5 * float(want.abs().max()))


def test_binding_refuses(ops):
    X, e, w, gate, up, down = block(ops, 6, 4, 2, 64, 32, 48)
    Q, s = ops.fp8_pack_activations(X)
    order, place, offsets = ops.moe_plan(e, 4)
    bad = [
        lambda: ops.moe_route(X[0], 2), lambda: ops.moe_route(X, 2, bias=torch.zeros(5, device="cuda")),
        lambda: ops.moe_route(X, 2, experts=torch.empty(6, 3, dtype=torch.int32, device="cuda")),
        lambda: ops.moe_plan(e.long(), 4), lambda: ops.moe_plan(e, 4, order=order[:-1]),
        lambda: ops.fp8_expert_linear(Q, s, offsets[:-1], gate), lambda: ops.fp8_expert_linear(Q, s[:, :0], offsets, gate),
        lambda: ops.fp8_expert_linear(Q, s, offsets, (gate[0].transpose(1, 2), gate[1])),
        lambda: ops.fp8_expert_linear(Q, s, offsets, (gate[0][0], gate[1])),
        lambda: ops.fp8_expert_swiglu(Q, s, order, offsets, 2, gate, down),
        lambda: ops.fp8_expert_swiglu(Q, s, order, offsets, 2, gate, tuple(x[:3] for x in up)),
        lambda: ops.moe_combine(X, place[:-1], w), lambda: ops.moe_combine(X, place, w, residual=X[:-1]),
        lambda: ops.fp8_moe(X, e, w[:, :1], gate, up, down), lambda: ops.fp8_moe(X, e, w, gate, up, gate),
        lambda: ops.fp8_moe(X, e, w, gate, up, down, residual=X),
        lambda: ops.fp8_prepare_experts(torch.zeros(4, 16, device="cuda"))]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, KeyError)):
            f()
            pytest.fail(f"call {i} was taken")
    for f in (lambda: ops.moe_route(X, 33), lambda: ops.moe_route(X, 2, n_groups=3),
              lambda: ops.fp8_moe(X, e, w, gate, up, down, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ops.ConvrotError):
            f()
    torch.cuda.synchronize()
