"""The 8-bit floating-point pack and linears on the GPU against their 64-bit
statements (oracle/block_oracle.py)."""
import numpy as np
import pytest
import torch

from gpu_common import host
from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U24 = 2.0 ** -24  # half a step of fp32


def codes(t):
    return host(t.view(torch.uint8))


def activations(seed, M, K, dtype="f32"):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(M, K, generator=g) * (1 + 29 * (torch.rand(K, generator=g) < 0.02))
    return X.to(DT[dtype]).cuda()


def packed(seed, R, K, rows=1):
    """Codes and scales on the device and on the host, packed by the statement."""
    X = np.random.default_rng(seed).normal(size=(R, K)).astype(np.float32)
    Q, s = bo.fp8_pack(X, rows)
    return torch.from_numpy(Q).cuda().view(torch.float8_e4m3fn), torch.from_numpy(s).cuda(), Q, s


def assert_linear(y, ref, mag, K):
    """Off by half a step of the output's type, and by the fp32 sums: at most
    one rounding per product and per block, one for each scale product and the
    bias, each of up to a whole step (the tensor cores may truncate)."""
    half = torch.finfo(y.dtype).eps / 2
    got = host(y.float()).astype(np.float64)
    bound = half * np.abs(ref) * (1 + half) + 2 * (128 + bo.n_blocks(K) + 4) * U24 * mag
    if y.dtype == torch.float16:
        bound = bound + 2.0 ** -25  # half a subnormal step
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} against {ref[bad][0]}"


@pytest.mark.parametrize("M,K,dtype", [(1, 16, "f32"), (1, 12288, "bf16"), (3, 144, "f16"), (37, 1040, "bf16"),
                                       (129, 3072, "f32"), (260, 1280, "f16"), (1000, 128, "bf16")])
def test_pack_is_the_definition(ops, M, K, dtype):
    X = activations(M + K, M, K, dtype)
    X[0, :16] = 0
    Q, s = ops.fp8_pack_activations(X)
    Qo, so = bo.fp8_pack(host(X.float()))
    np.testing.assert_array_equal(host(s), so)
    np.testing.assert_array_equal(codes(Q), Qo)


@pytest.mark.parametrize("N,K,dtype", [(1, 16, "f32"), (128, 128, "bf16"), (130, 272, "f16"), (1283, 1280, "f32")])
def test_weight_is_the_definition(ops, N, K, dtype):
    W = activations(N, N, K, dtype)
    Q, s = ops.fp8_prepare_weight(W)
    Qo, so = bo.fp8_pack(host(W.float()), 128)
    np.testing.assert_array_equal(host(s), so)
    np.testing.assert_array_equal(codes(Q), Qo)


def test_pack_rounding_borders(ops):
    """Quotients on and next to every rounding border, ties included: scale 1
    (a 448 in every block), a power of two and an inexact scale."""
    v = bo.e4m3_values()[:127].astype(np.float32)
    ties = (v[1:] + v[:-1]) / 2
    near = np.concatenate([ties, np.nextafter(ties, np.float32(0)), np.nextafter(ties, np.float32(500)), v, -ties,
                           np.float32([0.0, -0.0, 2.0 ** -10, 2.0 ** -11, 1e-30, 1e-42])])
    X = np.zeros((len(near) // 120 + 1) * 128, np.float32).reshape(-1, 128)
    X[:, 120] = 448
    X[:, :120].flat[:len(near)] = near
    for f in (1.0, 2.0 ** -30, 0.37, 3.3e4):
        Z = X * np.float32(f)
        Q, s = ops.fp8_pack_activations(torch.from_numpy(Z).cuda())
        Qo, so = bo.fp8_pack(Z)
        np.testing.assert_array_equal(host(s), so)
        np.testing.assert_array_equal(codes(Q), Qo)


def test_pack_extremes(ops):
    """Zero, subnormal, huge and non-finite blocks."""
    X = torch.zeros(8, 128)
    X[1] = torch.linspace(-1, 1, 128) * 1e-42        # the scale is subnormal or 0
    X[2, 5] = 2.0 ** -149
    X[3] = torch.linspace(-3.4e38, 3.4e38, 128)
    X[4] = torch.linspace(-1, 1, 128) * 1e-36        # 1 / scale would overflow
    X[5, 7] = float("inf")
    X[5, 8] = 1.0
    X[6, 9] = float("nan")
    X[7, 3] = -float("inf")
    X[7, 4] = float("nan")
    Q, s = (host(t) for t in (lambda r: (r[0].view(torch.uint8), r[1]))(ops.fp8_pack_activations(X.cuda())))
    Qo, so = bo.fp8_pack(X.numpy()[:5])
    np.testing.assert_array_equal(s[:5], so)
    np.testing.assert_array_equal(Q[:5], Qo)
    val = bo.e4m3_values()
    assert np.isinf(s[5, 0]) and np.isnan(s[6, 0]) and np.isnan(s[7, 0])
    with np.errstate(invalid="ignore"):
        assert np.isnan(val[Q[5:]] * s[5:]).all()    # nothing of such a block stays finite


def test_pack_strides_and_alignment(ops):
    """Column slices of a wider buffer, at offsets that are not 16-byte aligned."""
    base = activations(5, 40, 700, "bf16")
    for off, K in ((0, 256), (8, 256), (3, 272), (17, 16)):
        X = base[:, off:off + K]
        Q, s = ops.fp8_pack_activations(X)
        Qo, so = bo.fp8_pack(host(X.float().contiguous()))
        np.testing.assert_array_equal(host(s), so)
        np.testing.assert_array_equal(codes(Q), Qo)


# few rows (the weight rows on the tensor lanes), one tile of rows, several,
# pairs of CTAs; ragged rows, features and K on each
@pytest.mark.parametrize("M", [1, 16, 17, 33, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(16, 16), (128, 128), (130, 656), (640, 1280), (1283, 272)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_packed(ops, M, N, K, out):
    Qx, sx, qx, x = packed(M, M, K)
    Qw, sw, qw, w = packed(N + 1, N, K, 128)
    b = torch.randn(N, generator=torch.Generator().manual_seed(N)).cuda()
    for bias in (None, b):
        ref, mag = bo.fp8_linear(qx, x, qw, w, None if bias is None else host(bias))
        y = torch.full((M, N), float("nan"), dtype=DT[out], device="cuda")
        ops.fp8_linear_packed(Qx, sx, [Qw], [sw], [bias], Ys=[y])
        assert_linear(y, ref, mag, K)
    assert ops.convrot_device_status() == ops.OK


@pytest.mark.parametrize("M,N,K,out", [(2000, 3072, 1280, "bf16"), (2000, 3071, 528, "f16"), (1300, 9216, 256, "f32"),
                                       (9000, 512, 400, "f32"), (700, 5000, 3072, "f16")])
def test_linear_packed_many_tiles(ops, M, N, K, out):
    """Every tile of persistent launches: more tiles than CTAs."""
    Qx, sx, qx, x = packed(M, M, K)
    Qw, sw, qw, w = packed(N, N, K, 128)
    (y,) = ops.fp8_linear_packed(Qx, sx, [Qw], [sw], out_dtype=DT[out])
    assert_linear(y, *bo.fp8_linear(qx, x, qw, w), K)
    assert ops.convrot_device_status() == ops.OK


@pytest.mark.parametrize("M", [2, 100, 1500])
def test_linears_share_a_pack(ops, M):
    """Several linears of different widths (one empty) in one call, written
    into column slices of one output, whatever their alignment."""
    K, Ns = 784, [256, 0, 130, 1024, 16]
    X = activations(M, M, K, "bf16")
    qx, x = bo.fp8_pack(host(X.float()))
    ws = [packed(10 + j, n, K, 128) if n else (torch.empty(0, K, dtype=torch.float8_e4m3fn, device="cuda"),
                                               torch.empty(0, 7, device="cuda"), None, None) for j, n in enumerate(Ns)]
    for pad in (0, 3):
        wide = torch.full((M, sum(Ns) + pad), 7.0, dtype=torch.float16, device="cuda")
        Ys, at = [], pad
        for n in Ns:
            Ys.append(wide[:, at:at + n])
            at += n
        ops.fp8_linear(X, [w[0] for w in ws], [w[1] for w in ws], Ys=Ys)
        for y, w, n in zip(Ys, ws, Ns):
            if n:
                assert_linear(y, *bo.fp8_linear(qx, x, w[2], w[3]), K)
        assert (wide[:, :pad] == 7.0).all()
    assert ops.convrot_device_status() == ops.OK


@pytest.mark.parametrize("M", [3, 40, 300, 2500])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_outputs_inside_a_wider_array(ops, M, out):
    """Slices whose rows are 16-byte aligned (the bulk stores): what lies
    around them is left alone."""
    K, Ns = 400, [200, 1000]
    Qx, sx, qx, x = packed(M, M, K)
    ws = [packed(50 + n, n, K, 128) for n in Ns]
    wide = torch.full((M + 2, 1600), 5.0, dtype=DT[out], device="cuda")
    Ys = [wide[1:M + 1, 16:216], wide[1:M + 1, 232:1232]]
    ops.fp8_linear_packed(Qx, sx, [w[0] for w in ws], [w[1] for w in ws], Ys=Ys)
    for y, w in zip(Ys, ws):
        assert_linear(y, *bo.fp8_linear(qx, x, w[2], w[3]), K)
        y.fill_(5.0)
    assert (wide == 5.0).all()


def test_linear_is_repeatable_and_rows_are_independent(ops):
    """The same rows give the same bits, again and whatever rows follow within
    one kernel's range; every split of K adds in a fixed order."""
    Qx, sx, _, _ = packed(1, 64, 4096)
    Qw, sw, _, _ = packed(2, 384, 4096, 128)
    run = lambda m: ops.fp8_linear_packed(Qx[:m], sx[:m], [Qw], [sw], out_dtype=torch.float32)[0]  # noqa: E731
    a = run(64)
    for m in (64, 40):
        assert torch.equal(run(m), a[:m])


def test_linear_non_finite_rows(ops):
    """A NaN or infinity in one activation row reaches that row alone."""
    for M in (5, 200, 1200):
        X = activations(M, M, 512)
        X[1, 300] = float("nan")
        X[3, 5] = float("inf")
        Qw, sw, _, _ = packed(3, 2048, 512, 128)
        (y,) = ops.fp8_linear(X, [Qw], [sw])
        fine = torch.isfinite(y).all(1)
        assert not torch.isfinite(y[1]).any() and not torch.isfinite(y[3]).any()
        assert int(fine.sum()) == M - 2


def test_linear_empty(ops):
    Qw, sw, _, _ = packed(3, 64, 128, 128)
    (y,) = ops.fp8_linear(torch.empty(0, 128, device="cuda"), [Qw], [sw])
    assert y.shape == (0, 64)
    Q, s = ops.fp8_pack_activations(torch.empty(0, 128, device="cuda"))
    assert Q.shape == (0, 128) and s.shape == (0, 1)


def test_linear_on_another_stream_and_in_a_graph(ops):
    X = activations(9, 333, 768, "bf16")
    Qw, sw, _, _ = packed(4, 640, 768, 128)
    ref = ops.fp8_linear(X, [Qw], [sw])[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    (y,) = ops.fp8_linear(X, [Qw], [sw], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, ref)
    Y = torch.zeros_like(ref)
    ws = torch.empty(ops.fp8_linear_workspace_size(333, 768), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.fp8_linear(X, [Qw], [sw], Ys=[Y], workspace=ws)
    for k in range(2):
        X.copy_(activations(20 + k, 333, 768, "bf16"))
        graph.replay()
        assert torch.equal(Y, ops.fp8_linear(X, [Qw], [sw])[0])


def test_linear_offsets_past_32_bits(ops):
    """An output and an input buffer of more than 2^31 elements."""
    M, N, K = 70000, 32768, 16
    Qx, sx, qx, x = packed(6, M, K)
    Qw, sw, qw, w = packed(7, N, K, 128)
    (y,) = ops.fp8_linear_packed(Qx, sx, [Qw], [sw], out_dtype=torch.bfloat16)
    for r in (0, 65536, M - 3):
        assert_linear(y[r:r + 3], *bo.fp8_linear(qx[r:r + 3], x[r:r + 3], qw, w), K)
    del y
    wide = torch.empty(M, 32768, dtype=torch.bfloat16, device="cuda")
    X = wide[:, -256:]
    X.normal_()
    Q, s = ops.fp8_pack_activations(X)
    Qo, so = bo.fp8_pack(host(X[-5:].float()))
    np.testing.assert_array_equal(host(s[-5:]), so)
    np.testing.assert_array_equal(codes(Q[-5:]), Qo)


def test_linear_refusals(ops):
    X = activations(1, 8, 256)
    Qw, sw, _, _ = packed(3, 64, 256, 128)
    with pytest.raises(ops.ConvrotError) as e:
        ops.fp8_pack_activations(X[:, :40])
    assert e.value.status == ops.ERR_ALIGN
    for bad in (lambda: ops.fp8_linear(X.t(), [Qw], [sw]), lambda: ops.fp8_linear(X.double(), [Qw], [sw]),
                lambda: ops.fp8_linear(X, [Qw], [sw[:, :1]]), lambda: ops.fp8_linear(X, [Qw[:, :128]], [sw]),
                lambda: ops.fp8_linear(X, [], []), lambda: ops.fp8_linear(X, [Qw] * 9, [sw] * 9),
                lambda: ops.fp8_linear(X, [Qw], [sw], [sw[0]]), lambda: ops.fp8_linear(X, [Qw.cpu()], [sw]),
                lambda: ops.fp8_linear(X, [Qw], [sw], Ys=[torch.empty(8, 65, device="cuda")]),
                lambda: ops.fp8_linear(X[:1].expand(8, 256), [Qw], [sw]),
                lambda: ops.fp8_linear_packed(X, sw, [Qw], [sw])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ops.ConvrotError) as e:
        ops.fp8_linear(X, [Qw], [sw], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == ops.ERR_WORKSPACE


@pytest.mark.parametrize("M", [1, 2, 7, 15, 16])
@pytest.mark.parametrize("N,K", [(16, 16), (130, 656), (1283, 3072), (5000, 1040), (128, 12288)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f16")])
def test_few_rows_are_packed_alike(ops, M, N, K, dtype, out):
    """Up to 16 rows are packed inside the linear: the same result as of codes
    packed before, at any alignment of X."""
    Qw, sw, qw, w = packed(N + 1, N, K, 128)
    b = torch.randn(N, generator=torch.Generator().manual_seed(N)).cuda()
    wide = activations(M + N, M, K + 8, dtype)
    for off in (0, 3):
        X = wide[:, off:off + K]
        ref, mag = bo.fp8_linear(*bo.fp8_pack(host(X.float().contiguous())), qw, w, host(b))
        y = torch.full((M, N), float("nan"), dtype=DT[out], device="cuda")
        ops.fp8_linear(X, [Qw], [sw], [b], Ys=[y])
        assert_linear(y, ref, mag, K)
    assert ops.convrot_device_status() == ops.OK


def test_few_rows_non_finite(ops):
    X = activations(3, 9, 512)
    X[1, 300] = float("nan")
    X[3, 5] = float("inf")
    Qw, sw, _, _ = packed(3, 256, 512, 128)
    (y,) = ops.fp8_linear(X, [Qw], [sw])
    assert not torch.isfinite(y[[1, 3]]).any() and torch.isfinite(y[[0, 2, 4, 5, 6, 7, 8]]).all()


def test_few_rows_of_a_long_k(ops):
    """More blocks of K than the linear packs itself."""
    M, N, K = 3, 128, 24576
    X = activations(8, M, K)
    Qw, sw, qw, w = packed(9, N, K, 128)
    (y,) = ops.fp8_linear(X, [Qw], [sw])
    assert_linear(y, *bo.fp8_linear(*bo.fp8_pack(host(X)), qw, w), K)


# one kernel each: streamed weights (up to 8 rows), few rows, one wave of
# tiles, CTA pairs
@pytest.mark.parametrize("M,K", [(1, 3072), (3, 3072), (8, 3072), (1, 12288), (3, 12288), (8, 12288), (9, 12288),
                                 (300, 3072), (1500, 3072)])
def test_sums_are_fp32(ops, M, K):
    """The error of fp32 outputs against the 64-bit statement, root mean square
    over root mean square. Rounding the running sum to nearest after each of
    K / 128 <= 96 blocks gives sqrt(96) 2^-24 / sqrt 3 times the sum's own mean
    growth (0.71), 2.4e-7; eight steps of a block, each cut at 2^-23 of a block
    sum that is sqrt(128 / K) >= 0.1 of the result, give 3.4e-7 over 96 blocks;
    together 4.2e-7, doubled. Sums that keep 14 to 16 bits come to 1e-5 and
    more."""
    N = 2048
    Qx, sx, qx, x = packed(M, M, K)
    Qw, sw, qw, w = packed(N, N, K, 128)
    ref, _ = bo.fp8_linear(qx, x, qw, w)
    (y,) = ops.fp8_linear_packed(Qx, sx, [Qw], [sw], out_dtype=torch.float32)
    off = np.sqrt(np.mean((host(y).astype(np.float64) - ref) ** 2) / np.mean(ref ** 2))
    assert off <= 1e-6, off


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("N,K", [(16, 16), (130, 656), (1283, 3072), (5000, 1040), (128, 12288), (128, 12304)])
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f16", "bf16"), ("f32", "f16")])
def test_packing_in_the_call_equals_packing_before_it(ops, M, N, K, dtype, out):
    """Bit for bit: up to 4 rows of up to 12288 features are packed by the
    linear's own launch, more rows or features by a launch before it."""
    Qw, sw, qw, w = packed(N + 1, N, K, 128)
    b = torch.randn(N, generator=torch.Generator().manual_seed(N)).cuda()
    X = activations(M + N, M, K, dtype)
    (y,) = ops.fp8_linear(X, [Qw], [sw], [b], out_dtype=DT[out])
    Q, s = ops.fp8_pack_activations(X)
    (z,) = ops.fp8_linear_packed(Q, s, [Qw], [sw], [b], out_dtype=DT[out])
    assert torch.equal(y, z)
    assert_linear(y, *bo.fp8_linear(*bo.fp8_pack(host(X.float())), qw, w, host(b)), K)
    assert ops.convrot_device_status() == ops.OK


@pytest.mark.parametrize("M", [1, 8, 16, 200])
def test_nan_codes_of_finite_scales(ops, M):
    """A NaN code reaches the outputs that it enters, and no others."""
    Qx, sx, _, _ = packed(M, M, 256)
    Qw, sw, _, _ = packed(3, 64, 256, 128)
    Qw.view(torch.uint8)[7, 130] = 0x7f
    Qw.view(torch.uint8)[9, 3] = 0xff
    (y,) = ops.fp8_linear_packed(Qx, sx, [Qw], [sw], out_dtype=torch.float32)
    bad = torch.zeros(64, dtype=torch.bool, device="cuda")
    bad[[7, 9]] = True
    assert torch.isnan(y[:, bad]).all() and torch.isfinite(y[:, ~bad]).all()
