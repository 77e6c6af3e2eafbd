"""The block norms on the GPU against their 64-bit statement
(oracle/block_oracle.py)."""
import numpy as np
import pytest
import torch

from gpu_common import host
from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# Roundings of relative size 2^-24 on the way to a result: a row's sums add at
# most 32 elements per thread, 5 + 5 steps of lanes and warps and one division;
# the square root, the reciprocal, the affine forms and the final operations
# are ten more. Twice that, for the mean and for the deviation.
STEPS = 2 * (32 + 10 + 1 + 10) * 2.0 ** -24


def half(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return torch.finfo(t).tiny * torch.finfo(t).eps  # a subnormal step


def case(seed, M, K, dtype="bf16", gate=True, modulate=True, vectors=True, samples=3, ragged=True, y=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = dict(H=2 * r(M, K) * (1 + 29 * (torch.rand(K, generator=g) < 0.02)), Y=r(M, K) if y else None)
    t = {k: v if v is None else v.to(DT[dtype]).cuda() for k, v in t.items()}
    if vectors:
        for n in ("post_weight", "post_bias", "pre_weight", "pre_bias"):
            if y or n.startswith("pre"):
                t[n] = (0.2 * r(K) + ("weight" in n)).cuda()
    mod = 0.3 * r(samples, 3 * K).cuda()
    if gate and y:
        t["gate"] = mod[:, :K]
    if modulate:
        t["scale"], t["shift"] = mod[:, K:2 * K], mod[:, 2 * K:]
    per = -(-M // samples)
    if ragged:
        t["row_sample"] = torch.randint(0, samples, (M,), generator=g, dtype=torch.int32).cuda()
        sample = host(t["row_sample"])
    else:
        t["rows_per_sample"] = per
        sample = np.arange(M) // per
    return t, sample


def oracle(t, sample, post, pre, **kw):
    a = {k: host(v.float() if v.is_floating_point() else v) for k, v in t.items() if isinstance(v, torch.Tensor)}
    a.pop("row_sample", None)
    return bo.block_norm(a.pop("H"), a.pop("Y", None), post=post, pre=pre, sample=sample, **a, **kw)


def assert_near(got, ref, mag, what):
    x = host(got.float()).astype(np.float64)
    bound = half(got.dtype) * np.abs(ref) * 1.001 + STEPS * mag + tiny(got.dtype)
    bad = ~(np.abs(x - ref) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first {np.argwhere(bad)[0]}: {x[bad][0]} " \
                          f"against {ref[bad][0]}"


def assert_codes(Q, s, u, mag):
    """Codes and scales of an fp32 u that is itself off by up to STEPS * mag."""
    val, K = bo.e4m3_values(), u.shape[1]
    Q, s = host(Q.view(torch.uint8)), host(s).astype(np.float64)
    err = STEPS * mag
    for j in range(s.shape[1]):
        b = slice(j * 128, min(K, (j + 1) * 128))
        amax = np.abs(u[:, b]).max(1)
        assert np.all(np.abs(s[:, j] * 448 - amax) <= err[:, b].max(1) + amax * 2.0 ** -23 + 448 * 2.0 ** -149)
    w = bo.widen(s, *u.shape)
    d = np.abs(val[Q] * w - u)
    assert np.all(d <= np.maximum(np.abs(u) * 2.0 ** -4, w * 2.0 ** -10) * (1 + 2.0 ** -20) + 2 * err + w * 448 * 2.0 ** -23)


@pytest.mark.parametrize("M,K", [(1, 8), (5, 64), (37, 1280), (3, 3072), (310, 264), (2, 4104), (6, 8192),
                                 (9, 12288), (5, 16384),                                   # vector rows
                                 (4, 1), (7, 3), (65, 1283), (2, 12289), (1, 32768), (3, 20008)])  # any rows
@pytest.mark.parametrize("post,pre", [(1, 1), (0, 2), (2, 1), (2, 2), (0, 0)])
def test_norms(ops, M, K, post, pre):
    t, sample = case(M + K, M, K, ["bf16", "f16", "f32"][(M + K + post) % 3])
    h, u, hm, um = oracle(t, sample, post, pre)
    H, U = ops.convrot_block_norm(**t, post_norm=post, pre_norm=pre)
    assert_near(H, h, hm, "h")
    assert_near(U, u, um, "u")
    assert ops.convrot_device_status() == ops.OK


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("u_dtype", ["f32", "f16", "bf16"])
def test_types(ops, dtype, u_dtype):
    for K in (768, 771):
        t, sample = case(K, 70, K, dtype)
        h, u, hm, um = oracle(t, sample, 1, 2)
        H, U = ops.convrot_block_norm(**t, post_norm=1, pre_norm=2, u_dtype=DT[u_dtype])
        assert H.dtype == DT[dtype] and U.dtype == DT[u_dtype]
        assert_near(H, h, hm, "h")
        assert_near(U, u, um, "u")


@pytest.mark.parametrize("M,K,dtype", [(1, 16, "f32"), (37, 1280, "bf16"), (300, 3072, "bf16"), (5, 144, "f16"),
                                       (9, 12288, "f32"), (2, 32768, "f16"), (4, 16400, "bf16")])
@pytest.mark.parametrize("post,pre", [(1, 1), (0, 2), (0, 0)])
def test_codes(ops, M, K, dtype, post, pre):
    t, sample = case(M + K, M, K, dtype)
    h, u, hm, um = oracle(t, sample, post, pre)
    H, Q, s = ops.convrot_block_norm_fp8(**t, post_norm=post, pre_norm=pre)
    assert_near(H, h, hm, "h")
    assert_codes(Q, s, u, um)


def test_codes_are_the_packs(ops):
    """Without norms or vectors the codes are those of the residual sum itself."""
    for K, off in ((1280, 0), (1280, 1)):
        X = torch.randn(33, K + 8, generator=torch.Generator().manual_seed(K)).cuda()[:, off:off + K]
        _, Q, s = ops.convrot_block_norm_fp8(X, pre_norm=ops.NORM_NONE)
        Qp, sp = ops.fp8_pack_activations(X)
        assert torch.equal(s, sp) and torch.equal(Q.view(torch.uint8), Qp.view(torch.uint8))


@pytest.mark.parametrize("K", [640, 645])
@pytest.mark.parametrize("kw", [dict(gate=False), dict(modulate=False), dict(vectors=False), dict(y=False),
                                dict(samples=1, ragged=False), dict(samples=5, ragged=False),
                                dict(gate=False, modulate=False, vectors=False)])
def test_absent_parts(ops, K, kw):
    t, sample = case(K, 43, K, **kw)
    if "gate" not in t and "scale" not in t:
        t.pop("row_sample", None)
    scales = dict(residual_scale=0.75, block_scale=-1.5)
    h, u, hm, um = oracle({k: v for k, v in t.items() if k != "rows_per_sample"}, sample, 1, 1, **scales)
    H, U = ops.convrot_block_norm(**t, post_norm=1, pre_norm=1, **scales)
    assert_near(H, h, hm, "h")
    assert_near(U, u, um, "u")


def test_outputs_left_out_and_in_place(ops):
    for K in (512, 515):
        t, sample = case(3, 90, K)
        H, U = ops.convrot_block_norm(**t, post_norm=1, pre_norm=2)
        H1, none = ops.convrot_block_norm(**t, post_norm=1, pre_norm=2, want_u=False)
        none2, U1 = ops.convrot_block_norm(**t, post_norm=1, pre_norm=2, want_h=False)
        assert none is None and none2 is None and torch.equal(H, H1) and torch.equal(U, U1)
        h = t.pop("H").clone()
        H2, U2 = ops.convrot_block_norm(h, **t, post_norm=1, pre_norm=2, H_out=h)
        assert H2 is h and torch.equal(H, h) and torch.equal(U, U2)


def test_strides_and_alignment(ops):
    """Column slices of wider buffers: whole 16-byte pieces and not."""
    for off, K in ((0, 256), (8, 256), (1, 256), (5, 261)):
        g = torch.Generator().manual_seed(off)
        wide = torch.randn(50, 800, generator=g).to(torch.bfloat16).cuda()
        out = torch.full((50, 800), 3.0, dtype=torch.bfloat16, device="cuda")
        h, y, ho, u = wide[:, off:off + K], wide[:, 400 + off:400 + off + K], out[:, off:off + K], out[:, 400:400 + K]
        ref = bo.block_norm(host(h.float()), host(y.float()), post=1, pre=2)
        ops.convrot_block_norm(h, y, post_norm=1, pre_norm=2, H_out=ho, U=u)
        assert_near(ho, ref[0], ref[2], "h")
        assert_near(u, ref[1], ref[3], "u")
        assert (out[:, off + K:400] == 3.0).all() and (out[:, 400 + K:] == 3.0).all() and (out[:, :off] == 3.0).all()


def test_a_common_offset_does_not_cancel(ops):
    """LayerNorm of rows whose mean is 4096 times their deviation."""
    for K in (1024, 1027):
        x = torch.randn(16, K, generator=torch.Generator().manual_seed(1)).cuda() + 4096.0
        _, U = ops.convrot_block_norm(x, pre_norm=ops.NORM_LAYER)
        _, u, _, um = bo.block_norm(host(x), pre=2)
        assert_near(U, u, um, "u")
        assert float((U.var(1, correction=0) - 1).abs().max()) < 1e-3


def test_zero_constant_and_non_finite_rows(ops):
    for K in (384, 387):
        x = torch.randn(6, K, generator=torch.Generator().manual_seed(2)).cuda()
        x[0], x[1] = 0, 7.0
        x[2, 5], x[3, 9] = float("nan"), float("inf")
        for pre in (1, 2):
            _, U = ops.convrot_block_norm(x, pre_norm=pre)
            assert (U[0] == 0).all() and torch.isfinite(U[1]).all() and torch.isfinite(U[4:]).all()
            assert torch.isnan(U[2]).all() and torch.isnan(U[3, 9])
            if pre == 2:
                assert float(U[1].abs().max()) == 0.0


def test_sample_out_of_range_is_reported(ops):
    for K in (256, 259):
        t, sample = case(7, 12, K, samples=2)
        t["row_sample"][4], t["row_sample"][9] = 2, -1
        H, U = ops.convrot_block_norm(**t, post_norm=1, pre_norm=1)
        assert ops.convrot_device_status() == ops.ERR_ARG
        assert ops.convrot_device_status() == ops.OK
        assert torch.equal(H[4], t["H"][4])                       # gate 0
        fine = [r for r in range(12) if r not in (4, 9)]
        sample = host(t["row_sample"])[fine]
        sub = {k: v[fine] if k in ("H", "Y") else v for k, v in t.items()}
        h, u, hm, um = oracle(sub, sample, 1, 1)
        assert_near(H[fine], h, hm, "h")
        assert_near(U[fine], u, um, "u")


def test_samples_without_vectors_are_not_read(ops):
    """A row's sample means nothing without gate, scale or shift."""
    import ctypes
    for K in (256, 259):
        h = torch.randn(6, K, device="cuda")
        u = torch.empty_like(h)
        a = ops.convrot_block_norm_args()
        a.M, a.K, a.dtype, a.u_dtype, a.H, a.ldh, a.U, a.ldu = 6, K, ops.F32, ops.F32, h.data_ptr(), K, u.data_ptr(), K
        a.residual_scale, a.pre_norm, a.pre_eps = 1.0, ops.NORM_RMS, 1e-6
        sample = torch.full((6,), 77, dtype=torch.int32, device="cuda")
        a.row_sample = sample.data_ptr()
        assert ops.lib().convrot_block_norm(ctypes.byref(a), torch.cuda.current_stream().cuda_stream) == ops.OK
        assert ops.convrot_device_status() == ops.OK
        _, ref, _, mag = bo.block_norm(host(h))
        assert_near(u, ref, mag, "u")


def test_many_rows_repeat_bit_for_bit(ops):
    t, sample = case(8, 5000, 768)
    H, U = ops.convrot_block_norm(**t, post_norm=2, pre_norm=2)
    h, u, hm, um = oracle(t, sample, 2, 2)
    assert_near(H, h, hm, "h")
    assert_near(U, u, um, "u")
    for _ in range(2):
        H2, U2 = ops.convrot_block_norm(**t, post_norm=2, pre_norm=2)
        assert torch.equal(H, H2) and torch.equal(U, U2)


def test_offsets_past_32_bits(ops):
    """Rows of a buffer of more than 2^31 elements."""
    wide = torch.empty(70000, 32768, dtype=torch.bfloat16, device="cuda")
    for off in (32768 - 256, 32768 - 255):
        X = wide[:, off:]
        X.normal_()
        _, U = ops.convrot_block_norm(X, want_h=False)
        ref = bo.block_norm(host(X[-9:].float()))
        assert_near(U[-9:], ref[1], ref[3], "u")


def test_stream_graph_and_empty(ops):
    t, _ = case(9, 64, 512)
    ref = ops.convrot_block_norm(**t, post_norm=1, pre_norm=2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.convrot_block_norm(**t, post_norm=1, pre_norm=2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    out = [torch.zeros_like(v) for v in ref]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.convrot_block_norm(**t, post_norm=1, pre_norm=2, H_out=out[0], U=out[1])
    graph.replay()
    assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
    H, U = ops.convrot_block_norm(torch.empty(0, 64, device="cuda"))
    assert H.shape == U.shape == (0, 64)


def test_refusals(ops):
    x = torch.randn(8, 64, device="cuda")
    g = torch.randn(2, 64, device="cuda")
    for bad in (lambda: ops.convrot_block_norm(x.t()), lambda: ops.convrot_block_norm(x.double()),
                lambda: ops.convrot_block_norm(x, x.half()), lambda: ops.convrot_block_norm(x, x[:4]),
                lambda: ops.convrot_block_norm(x, pre_weight=g), lambda: ops.convrot_block_norm(x, pre_bias=g[0].half()),
                lambda: ops.convrot_block_norm(x, scale=g), lambda: ops.convrot_block_norm(x, U=torch.empty(8, 65, device="cuda")),
                lambda: ops.convrot_block_norm(x, scale=g, shift=g[:1], rows_per_sample=4),
                lambda: ops.convrot_block_norm(x, scale=g, row_sample=torch.zeros(8, device="cuda")),
                lambda: ops.convrot_block_norm(x, H_out=torch.empty(8, 64, device="cuda", dtype=torch.half)),
                lambda: ops.convrot_block_norm_fp8(x, Q=torch.empty(8, 64, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad, status in ((lambda: ops.convrot_block_norm(x, gate=g, rows_per_sample=4), ops.ERR_ARG),
                        (lambda: ops.convrot_block_norm(x, scale=g, rows_per_sample=3), ops.ERR_ARG),
                        (lambda: ops.convrot_block_norm(x, pre_norm=7), ops.ERR_ARG),
                        (lambda: ops.convrot_block_norm(x, pre_eps=-1.0), ops.ERR_ARG),
                        (lambda: ops.convrot_block_norm(x, H_out=x, U=x), ops.ERR_ALIAS),
                        (lambda: ops.convrot_block_norm_fp8(x[:, :40]), ops.ERR_ALIGN),
                        (lambda: ops.convrot_block_norm(torch.empty(2, 32769, device="cuda")), ops.ERR_UNSUPPORTED)):
        with pytest.raises(ops.ConvrotError) as e:
            bad()
        assert e.value.status == status


@pytest.mark.parametrize("M,K", [(11, 8200), (400, 9000), (7, 10240), (3, 9001)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vectors", [True, False])
def test_widths_between_8192_and_10240(ops, M, K, dtype, vectors):
    """Five units of eight features per lane, with and without vectors beside
    the staged rows, to u and to codes."""
    t, sample = case(M + K, M, K, dtype, vectors=vectors)
    h, u, hm, um = oracle(t, sample, 2, 1)
    H, U = ops.convrot_block_norm(**t, post_norm=2, pre_norm=1)
    assert_near(H, h, hm, "h")
    assert_near(U, u, um, "u")
    if K % 16 == 0:
        H, Q, s = ops.convrot_block_norm_fp8(**t, post_norm=2, pre_norm=1)
        assert_near(H, h, hm, "h")
        assert_codes(Q, s, u, um)
    assert ops.convrot_device_status() == ops.OK


@pytest.mark.parametrize("M", [1, 260])
def test_u_feeds_the_int8_linears(ops, M):
    """A bfloat16 residual stream in front of an INT8 linear: u leaves as
    binary16 or fp32, which the INT8 pack takes; the result is that of the same
    u held by the caller."""
    K, N, G = 1024, 256, 64
    t, sample = case(M, M, K, "bf16")
    W = torch.randn(N, K, generator=torch.Generator().manual_seed(5)).cuda()
    Q_w, s_w, Q16 = ops.convrot_prepare_weight(W, G)
    _, u, _, um = oracle(t, sample, 1, 2)
    for u_dtype in ("f16", "f32"):
        _, U = ops.convrot_block_norm(**t, post_norm=1, pre_norm=2, want_h=False, u_dtype=DT[u_dtype])
        assert_near(U, u, um, "u")
        (y,) = ops.convrot_linear(U, G, [Q16], [s_w], [None])
        # each operand is rounded to 8 bits: by up to 1 / 254 of its row's
        # largest rotated value, 1 / (254 sqrt 3) in the root mean square; that
        # largest of 1024 is within 6 times the row's root mean square
        ref = U.double() @ W.double().t()
        assert float((y.double() - ref).norm() / ref.norm()) < 2 * 6 / (254 * 3 ** 0.5)
    assert ops.convrot_device_status() == ops.OK


def test_gates_scales_and_shifts_of_no_sample(ops):
    """Refused for rows that need one, not taken for absent; and of no rows fine."""
    x, y = torch.randn(8, 64, device="cuda"), torch.randn(8, 64, device="cuda")
    none, two = torch.empty(0, 64, device="cuda"), torch.randn(2, 64, device="cuda")
    for bad in (lambda: ops.convrot_block_norm(x, y, gate=none), lambda: ops.convrot_block_norm(x, scale=none),
                lambda: ops.convrot_block_norm(x, shift=none), lambda: ops.convrot_block_norm_fp8(x, scale=none),
                lambda: ops.convrot_block_norm(x, y, gate=none, scale=two, rows_per_sample=4),
                lambda: ops.convrot_block_norm(x, scale=two, shift=none, rows_per_sample=4),
                lambda: ops.convrot_block_norm(x, scale=two[0]), lambda: ops.convrot_block_norm(x, scale=two[0, 0])):
        with pytest.raises(ValueError):
            bad()
    H, U = ops.convrot_block_norm(x[:0], y[:0], gate=none, scale=none, shift=none)
    assert H.shape == U.shape == (0, 64)
    assert ops.convrot_device_status() == ops.OK
