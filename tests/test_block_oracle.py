"""Facts that pin the 64-bit statements of the block norms and the 8-bit
floating-point linears, and the library's argument checks (no GPU)."""
import numpy as np
import pytest

from oracle import block_oracle as bo

A = [0x7f0000000000 + i * 0x10000000 for i in range(16)]  # fake, apart, 256-aligned addresses


@pytest.fixture(scope="session")
def L():
    from int8_hadamard_rotated_gb300 import build, ops
    build.build()
    return ops.lib()


def test_e4m3_values():
    v = bo.e4m3_values()
    assert v[0x7e] == 448.0 and np.isnan(v[0x7f]) and np.isnan(v[0xff])
    assert v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x39] == 1.125 and v[0xb8] == -1.0


def test_e4m3_encode_matches_torch_cast():
    import torch
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(0, s, 4000) for s in (1e-3, 1e-2, 1.0, 100.0)]).astype(np.float32)
    v = bo.e4m3_values()[:127]
    ties = ((v[1:] + v[:-1]) / 2).astype(np.float32)  # exact in fp32
    x = np.clip(np.concatenate([x, v.astype(np.float32), ties, -ties, np.nextafter(ties, 0, dtype=np.float32),
                                np.nextafter(ties, np.float32(1e9), dtype=np.float32), [0.0, -0.0]]), -448, 448)
    ref = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(bo.e4m3_encode(x.astype(np.float32)), ref)


def test_pack_facts():
    X = np.zeros((3, 272), np.float32)
    X[0, :128] = np.linspace(-5, 5, 128)
    X[1, 130] = 7.0
    X[2, 256:] = 1e-30
    Q, s = bo.fp8_pack(X)
    v = bo.e4m3_values()
    assert s.shape == (3, 3) and s[0, 1] == 0 and not Q[0, 128:].any()
    assert v[Q[1, 130]] == 448.0 and abs(float(s[1, 1]) * 448.0 - 7.0) < 1e-6
    d = v[Q] * bo.widen(s, 3, 272)
    assert np.all(np.abs(d - X) <= np.maximum(np.abs(X) * 2.0 ** -4, bo.widen(s, 3, 272) * 2.0 ** -10) * 1.00001)
    # one scale for all 128 rows of a weight's block
    Qw, sw = bo.fp8_pack(X, 128)
    assert sw.shape == (1, 3) and sw[0, 0] == s[0, 0] and v[Qw[1, 130]] == 448.0


def test_linear_facts():
    one = bo.e4m3_encode(np.ones((2, 200)))
    Y, mag = bo.fp8_linear(one, np.full((2, 2), 2.0), one, np.full((1, 2), 0.5), np.array([1.0, -1.0]))
    np.testing.assert_array_equal(Y, [[201, 199], [201, 199]])
    np.testing.assert_array_equal(mag, np.full((2, 2), 201.0))


def test_norm_facts():
    x = np.array([[1.0, -1.0, 1.0, -1.0]])
    assert np.allclose(bo.norm(x, bo.NORM_RMS, 3.0)[0], x / 2)          # 1 / sqrt(1 + 3)
    assert np.allclose(bo.norm(x + 5, bo.NORM_LAYER, 3.0)[0], x / 2)    # the mean is taken off
    h, u, _, _ = bo.block_norm(x, 2 * x, residual_scale=3.0, block_scale=0.5, gate=np.full((1, 4), 4.0),
                               pre=bo.NORM_NONE, scale=np.full((1, 4), 0.5), shift=np.full((1, 4), 10.0))
    assert np.allclose(h, 7 * x) and np.allclose(u, 10.5 * x + 10)


def test_pack_checks(L):
    from int8_hadamard_rotated_gb300 import ops
    f = L.fp8_pack_activations
    assert f(A[0], ops.BF16, 0, 256, 256, A[1], A[2], None) == ops.OK
    assert f(None, ops.BF16, 0, 256, 256, None, None, None) == ops.OK
    assert f(A[0], 3, 4, 256, 256, A[1], A[2], None) == ops.ERR_ARG
    assert f(None, ops.F32, 4, 256, 256, A[1], A[2], None) == ops.ERR_ARG
    assert f(A[0], ops.F32, 4, 256, 255, A[1], A[2], None) == ops.ERR_ARG          # rows overlap
    assert f(A[0], ops.F32, -1, 256, 256, A[1], A[2], None) == ops.ERR_ARG
    assert f(A[0], ops.F32, 4, 0, 256, A[1], A[2], None) == ops.ERR_ARG
    assert f(A[0], ops.F32, 4, 250, 256, A[1], A[2], None) == ops.ERR_ALIGN
    assert f(A[0], ops.F32, 4, 256, 256, A[1] + 8, A[2], None) == ops.ERR_ALIGN
    assert f(A[0] + 2, ops.F32, 4, 256, 256, A[1], A[2], None) == ops.ERR_ALIGN    # not on its elements
    assert f(A[0], ops.F32, 4, 256, 256, A[0] + 1024, A[2], None) == ops.ERR_ALIAS
    assert f(A[0], ops.F32, 4, 256, 256, A[1], A[1] + 16, None) == ops.ERR_ALIAS
    assert f(A[0], ops.F32, 1 << 31, 256, 256, A[1], A[2], None) == ops.ERR_UNSUPPORTED
    g = L.fp8_prepare_weight
    assert g(A[0], ops.F32, 0, 256, A[1], A[2], None) == ops.OK
    assert g(A[0], 9, 4, 256, A[1], A[2], None) == ops.ERR_ARG
    assert g(A[0], ops.F32, 4, 40, A[1], A[2], None) == ops.ERR_ALIGN
    assert g(A[0], ops.F32, 4, 256, A[0], A[2], None) == ops.ERR_ALIAS


def test_linear_checks(L):
    from int8_hadamard_rotated_gb300 import ops
    W = ops.convrot_fp8_weight
    f = L.fp8_linear_packed

    def call(ws, M=16, K=256, q=A[0], s=A[1], dt=ops.BF16, n=None):
        arr = (W * max(1, len(ws)))(*ws)
        return f(q, s, M, K, arr, len(ws) if n is None else n, dt, None)

    good = W(A[2], A[3], A[4], 64, A[5], 64)
    assert call([good], M=0) == ops.OK
    assert call([W(None, None, None, 0, None, 0)]) == ops.OK                       # nothing to compute
    assert call([good], n=0) == ops.ERR_ARG and call([good] * 9) == ops.ERR_ARG
    assert call([good], q=None) == ops.ERR_ARG and call([good], s=None) == ops.ERR_ARG
    assert call([good], dt=5) == ops.ERR_ARG and call([good], K=0) == ops.ERR_ARG
    assert call([W(A[2], None, None, 64, A[5], 64)]) == ops.ERR_ARG
    assert call([W(A[2], A[3], None, 64, A[5], 63)]) == ops.ERR_ARG
    assert call([W(A[2], A[3], None, -1, A[5], 64)]) == ops.ERR_ARG
    assert call([good], K=24) == ops.ERR_ALIGN and call([good], q=A[0] + 4) == ops.ERR_ALIGN
    assert call([W(A[2] + 8, A[3], None, 64, A[5], 64)]) == ops.ERR_ALIGN
    assert call([W(A[2], A[3], None, 64, A[5] + 1, 64)]) == ops.ERR_ALIGN
    assert call([W(A[2], A[3], None, 64, A[0] + 512, 64)]) == ops.ERR_ALIAS        # on the activations
    assert call([W(A[2], A[3], None, 64, A[2], 64)]) == ops.ERR_ALIAS              # on the weight
    assert call([good, W(A[6], A[7], None, 64, A[5], 64)]) == ops.ERR_ALIAS        # one output twice
    # column slices of one wide output are apart; one column more is not
    wide = [W(A[2], A[3], None, 64, A[5], 128), W(A[6], A[7], None, 64, A[5] + 128, 128)]
    assert call(wide) in (ops.ERR_DEVICE, ops.OK)
    wide[0].N = 65
    assert call(wide) == ops.ERR_ALIAS
    assert call([good], M=1 << 31) == ops.ERR_UNSUPPORTED


def test_linear_workspace_checks(L):
    from int8_hadamard_rotated_gb300 import ops
    W = ops.convrot_fp8_weight
    w = (W * 1)(W(A[2], A[3], None, 64, A[5], 64))
    need = L.fp8_linear_workspace_size(17, 272)
    assert need == (17 * 272 + 255) // 256 * 256 + (17 * 3 * 4 + 255) // 256 * 256
    assert L.fp8_linear_workspace_size(-1, 16) == 0 and L.fp8_linear_workspace_size(4, 0) == 0
    f = lambda ws, n, X=A[0], w=w: L.fp8_linear(X, ops.F32, 17, 272, 272, w, 1, ops.F32, ws, n, None)  # noqa: E731
    assert f(None, 0) == ops.ERR_WORKSPACE and f(A[6], need - 1) == ops.ERR_WORKSPACE
    assert f(A[6] + 8, need + 8) == ops.ERR_ALIGN
    assert f(A[0], need) == ops.ERR_ALIAS                                          # on X
    assert f(A[5], need) == ops.ERR_ALIAS                                          # on Y
    assert f(A[2], need) == ops.ERR_ALIAS                                          # on a weight
    assert f(A[6], need, w=(W * 1)(W(A[2], A[3], None, 64, A[0], 64))) == ops.ERR_ALIAS
    assert L.fp8_linear(None, ops.F32, 0, 272, 272, w, 1, ops.F32, None, 0, None) == ops.OK


def norm_args(**kw):
    from int8_hadamard_rotated_gb300 import ops
    a = ops.convrot_block_norm_args()
    base = dict(M=8, K=64, dtype=ops.F16, u_dtype=ops.F16, H=A[0], Y=A[1], ldh=64, ldy=64, residual_scale=1.0,
                block_scale=1.0, post_norm=1, pre_norm=2, post_eps=1e-6, pre_eps=1e-6, H_out=A[2], ldho=64, U=A[3],
                ldu=64)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(M=0, H=None, Y=None, H_out=None, U=None), "OK"),
    (dict(M=-1), "ERR_ARG"), (dict(K=0), "ERR_ARG"), (dict(dtype=4), "ERR_ARG"), (dict(u_dtype=4), "ERR_ARG"),
    (dict(post_norm=3), "ERR_ARG"), (dict(pre_norm=-1), "ERR_ARG"),
    (dict(pre_eps=-1.0), "ERR_ARG"), (dict(post_eps=float("nan")), "ERR_ARG"),
    (dict(residual_scale=float("inf")), "ERR_ARG"),
    (dict(H=None), "ERR_ARG"), (dict(H_out=None, U=None), "ERR_ARG"), (dict(Q=A[4]), "ERR_ARG"),
    (dict(U=None, Q=A[4]), "ERR_ARG"), (dict(ldh=63), "ERR_ARG"), (dict(ldy=1), "ERR_ARG"), (dict(ldu=0), "ERR_ARG"),
    (dict(gate=A[5]), "ERR_ARG"),                                    # no sample count
    (dict(gate=A[5], n_samples=1, Y=None), "ERR_ARG"),               # a gate of nothing
    (dict(gate=A[5], n_samples=2, ld_gate=63, rows_per_sample=4), "ERR_ARG"),
    (dict(gate=A[5], n_samples=2, ld_gate=64, rows_per_sample=3), "ERR_ARG"),   # 8 rows need 3 samples
    (dict(scale=A[5], n_samples=2, ld_mod=64, rows_per_sample=-1), "ERR_ARG"),
    (dict(H=A[0] + 1), "ERR_ALIGN"), (dict(pre_weight=A[5] + 2), "ERR_ALIGN"),
    (dict(U=None, Q=A[4] + 8, s=A[5]), "ERR_ALIGN"),
    (dict(U=None, Q=A[4], s=A[5], K=40), "ERR_ALIGN"),
    (dict(K=32769, ldh=32769, ldy=32769, ldho=32769, ldu=32769), "ERR_UNSUPPORTED"),
    (dict(H_out=A[0] + 16), "ERR_ALIAS"), (dict(H_out=A[0], ldho=65), "ERR_ALIAS"), (dict(H_out=A[1]), "ERR_ALIAS"),
    (dict(U=A[0]), "ERR_ALIAS"), (dict(U=A[2]), "ERR_ALIAS"),
    (dict(U=A[3], gate=A[3], n_samples=1), "ERR_ALIAS"),
    (dict(U=None, Q=A[4], s=A[4] + 64), "ERR_ALIAS"),
])
def test_norm_checks(L, change, status):
    import ctypes
    from int8_hadamard_rotated_gb300 import ops
    assert L.convrot_block_norm(ctypes.byref(norm_args(**change)), None) == getattr(ops, status)


def test_norm_accepts(L):
    """In place, column slices of one buffer, any alignment of the elements."""
    import ctypes
    from int8_hadamard_rotated_gb300 import ops
    assert L.convrot_block_norm(None, None) == ops.ERR_ARG
    for change in (dict(H_out=A[0]), dict(H_out=A[0] + 128, ldh=128, ldho=128), dict(U=A[3] + 2, ldu=67),
                   dict(U=None), dict(H_out=None, U=None, Q=A[4], s=A[5]), dict(Y=None, ldy=0)):
        assert L.convrot_block_norm(ctypes.byref(norm_args(**change)), None) in (ops.ERR_DEVICE, ops.OK)


def test_binding_refuses_host_tensors():
    import torch
    from int8_hadamard_rotated_gb300 import ops
    with pytest.raises(ValueError, match="CUDA"):
        ops.fp8_pack_activations(torch.zeros(4, 32))
    with pytest.raises(ValueError, match="CUDA"):
        ops.convrot_block_norm(torch.zeros(4, 32))


def test_row_limit(L):
    # rows are counted in 32 bits, with room for looking a tile past the last
    from int8_hadamard_rotated_gb300 import ops
    import ctypes
    W = ops.convrot_fp8_weight
    most, over = 0x7fff0000, 0x7fff0001
    for rows in (over, (1 << 31) - 1):
        assert L.fp8_pack_activations(A[0], ops.F32, rows, 16, 16, A[1], A[2], None) == ops.ERR_UNSUPPORTED
        assert L.fp8_prepare_weight(A[0], ops.F32, rows, 16, A[1], A[2], None) == ops.ERR_UNSUPPORTED
        assert L.fp8_linear_workspace_size(rows, 16) == 0
        w = (W * 1)(W(A[2], A[3], None, 64, A[5], 64))
        assert L.fp8_linear_packed(A[0], A[1], rows, 16, w, 1, ops.F32, None) == ops.ERR_UNSUPPORTED
        assert L.fp8_linear(A[0], ops.F32, rows, 16, 16, w, 1, ops.F32, A[6], 0, None) == ops.ERR_UNSUPPORTED
        w[0].N = w[0].ldy = rows
        assert L.fp8_linear_packed(A[0], A[1], 1, 16, w, 1, ops.F32, None) == ops.ERR_UNSUPPORTED
        assert L.convrot_block_norm(ctypes.byref(norm_args(M=rows, K=8)), None) == ops.ERR_UNSUPPORTED
    assert L.fp8_linear_workspace_size(most, 16) == most * 16 + most * 4


def test_norm_timeout_test_checks(L):
    import ctypes
    from int8_hadamard_rotated_gb300 import ops
    f = L.convrot_test_block_norm_timeout
    a = norm_args()
    assert f(None, 0, 1000, None) == ops.ERR_ARG
    assert f(ctypes.byref(a), 0, 0, None) == ops.ERR_ARG             # no limit
    assert f(ctypes.byref(a), 8, 1000, None) == ops.ERR_ARG          # no such row
    assert f(ctypes.byref(a), -1, 1000, None) == ops.ERR_ARG
    a.U = a.H
    assert f(ctypes.byref(a), 0, 1000, None) == ops.ERR_ALIAS


def test_linear_timeout_test_checks(L):
    from int8_hadamard_rotated_gb300 import ops
    W = ops.convrot_fp8_weight
    f = L.fp8_test_linear_timeout
    w = (W * 1)(W(A[2], A[3], A[4], 64, A[5], 64))
    assert f(A[0], A[1], 16, 256, w, 1, ops.BF16, 0, None) == ops.ERR_ARG          # no limit
    assert f(None, A[1], 16, 256, w, 1, ops.BF16, 1000, None) == ops.ERR_ARG
    assert f(A[0], A[1], 16, 24, w, 1, ops.BF16, 1000, None) == ops.ERR_ALIGN


def test_length_limit(L):
    """Places of K are counted in 32 bits, with steps of up to 8192 past the last."""
    from int8_hadamard_rotated_gb300 import ops
    W = ops.convrot_fp8_weight
    A = [0x7f0000000000 + i * 0x10000000000 for i in range(8)]  # apart by more than a row of 2^31 features
    most = 0x7fff0000
    w = (W * 1)(W(A[2], A[3], None, 1, A[5], 1))
    for K in (most + 16, (1 << 31) - 16):
        assert L.fp8_pack_activations(A[0], ops.F32, 1, K, K, A[1], A[4], None) == ops.ERR_UNSUPPORTED
        assert L.fp8_prepare_weight(A[0], ops.F32, 1, K, A[1], A[4], None) == ops.ERR_UNSUPPORTED
        assert L.fp8_linear_workspace_size(1, K) == 0
        assert L.fp8_linear_packed(A[0], A[1], 1, K, w, 1, ops.F32, None) == ops.ERR_UNSUPPORTED
        assert L.fp8_linear(A[0], ops.F32, 1, K, K, w, 1, ops.F32, A[6], 1 << 33, None) == ops.ERR_UNSUPPORTED
    assert L.fp8_linear_workspace_size(1, most) == most + (most // 128 * 4)


def fma32(a, b, c):
    """fp32 a b + c, rounded once: the product is exact in 64 bits, the sum is
    rounded to odd there, and then to fp32."""
    p, c = a.astype(np.float64) * b.astype(np.float64), c.astype(np.float64)
    s = p + c
    t = s - p
    err = (p - (s - t)) + (c - t)
    inexact_even = (err != 0) & (s.view(np.int64) & 1 == 0)
    toward = np.where((err > 0) == (s > 0), 1, -1)
    return (s.view(np.int64) + np.where(inexact_even, toward, 0)).view(np.float64).astype(np.float32)


def corrected_quotient(x, s):
    """The kernels' division: r = RN(1 / s), q0 = RN(x r), RN(q0 + RN(x - q0 s) r)."""
    r = np.float32(1) / s
    q0 = x * r
    return fma32(fma32(-q0, s, x), r, q0)


def test_fma32():
    from fractions import Fraction
    rng = np.random.default_rng(0)
    a, b = (rng.integers(1 << 23, 1 << 24, 300).astype(np.float32) for _ in range(2))
    c = (-(a * b)).astype(np.float32) * np.float32(1) + rng.integers(-4, 4, 300).astype(np.float32)
    for x, y, z, f in zip(a, b, c, fma32(a, b, c)):
        exact = Fraction(float(x)) * Fraction(float(y)) + Fraction(float(z))
        near = [f, np.nextafter(f, np.float32(np.inf)), np.nextafter(f, np.float32(-np.inf))]
        assert min(abs(Fraction(float(v)) - exact) for v in near) == abs(Fraction(float(f)) - exact)


def test_corrected_scale_is_the_ieee_quotient():
    """amax / 448 for every significand of amax."""
    for k in range(4):
        x = (np.arange(k << 21, (k + 1) << 21, dtype=np.int32) + np.float32(1).view(np.int32)).view(np.float32)
        s = np.full_like(x, 448)
        np.testing.assert_array_equal(corrected_quotient(x, s), x / s)


def test_corrected_quotients_at_rounding_borders():
    """x next to every rounding border of e4m3 times s: the last 2^14
    significands of s, where q0 is furthest from the quotient, and 2^14 others."""
    v = bo.e4m3_values()[:127]
    borders = np.unique(np.frexp((v[1:] + v[:-1]) / 2)[0] * 2)
    assert len(borders) == 16
    m = np.concatenate([np.arange((1 << 23) - (1 << 14), 1 << 23),
                        np.random.default_rng(0).integers(0, 1 << 23, 1 << 14)]).astype(np.int32)
    s = (m + np.float32(1).view(np.int32)).view(np.float32)
    furthest = 0.0
    for b in borders:
        x0 = (b * s.astype(np.float64)).astype(np.float32)
        for k in range(-5, 6):
            x = (x0.view(np.int32) + np.int32(k)).view(np.float32)
            q = x / s
            np.testing.assert_array_equal(corrected_quotient(x, s), q)
            off = np.abs((x * (np.float32(1) / s)).astype(np.float64) - x.astype(np.float64) / s) / np.spacing(q)
            furthest = max(furthest, float(off.max()))
    assert 1.0 < furthest < 1.5        # beyond what a proof by an exact remainder covers
