"""The block norms' failure path on the GPU, made to happen without faulting,
trapping or hanging anything: a test entry point leaves out the copies into
shared memory from one row on and shortens the limit of the waits, so that the
waits for those rows run out. Nothing is stored for them, the kernel records
CONVROT_ERR_TIMEOUT once and exits, and the next call is correct."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu

SENTINEL = 123.0


def arguments(ops, H, Y, H_out, U, vec, mod, codes):
    """LayerNorms on both sides with weights, a gate and modulation of two samples."""
    a = ops.convrot_block_norm_args()
    M, K = H.shape
    dtype = {torch.float32: ops.F32, torch.float16: ops.F16, torch.bfloat16: ops.BF16}[H.dtype]
    a.M, a.K, a.dtype, a.u_dtype, a.H, a.Y, a.ldh, a.ldy = M, K, dtype, dtype, H.data_ptr(), Y.data_ptr(), K, K
    a.residual_scale = a.block_scale = 1.0
    a.post_norm = a.pre_norm = ops.NORM_LAYER
    a.post_eps = a.pre_eps = 1e-6
    a.post_weight = a.pre_weight = vec.data_ptr()
    a.gate, a.scale, a.shift = (mod[:, i * K:].data_ptr() for i in range(3))
    a.ld_gate = a.ld_mod = 3 * K
    a.n_samples, a.rows_per_sample = 2, (M + 1) // 2
    a.H_out, a.ldho = H_out.data_ptr(), K
    if codes:
        a.Q, a.s = U[0].data_ptr(), U[1].data_ptr()
    else:
        a.U, a.ldu = U[0].data_ptr(), K
    return a


# one, two, four and eight warps to a row, and a row per block of 8 and of 16
# warps; a single row, few rows, and rings that are filled many times
@pytest.mark.parametrize("M,K,dtype", [(1, 64, "f32"), (5000, 256, "bf16"), (3000, 1280, "bf16"), (2000, 3072, "f16"),
                                       (40, 1024, "f32"), (600, 6144, "bf16"), (500, 12288, "f32"),
                                       (300, 16384, "bf16")])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_a_wait_that_runs_out_stores_nothing(ops, M, K, dtype, codes, where):
    g = torch.Generator().manual_seed(M)
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    H, Y = (torch.randn(M, K, generator=g).to(dt).cuda() for _ in range(2))
    vec, mod = (torch.randn(*s, generator=g).cuda() for s in ((K,), (2, 3 * K)))

    def outputs():
        o = [torch.full_like(H, SENTINEL)]
        return o + ([torch.full((M, K), 0x55, dtype=torch.uint8, device="cuda"),
                     torch.full((M, -(-K // 128)), SENTINEL, device="cuda")] if codes else
                    [torch.full_like(H, SENTINEL)])

    stream = torch.cuda.current_stream().cuda_stream
    ref, got = outputs(), outputs()
    untouched = [o.clone() for o in ref]
    a = arguments(ops, H, Y, ref[0], ref[1:], vec, mod, codes)
    assert ops.lib().convrot_block_norm(ctypes.byref(a), stream) == ops.OK
    assert ops.convrot_device_status() == ops.OK

    row = {"first": 0, "middle": M // 2, "last": M - 1}[where]
    a = arguments(ops, H, Y, got[0], got[1:], vec, mod, codes)
    assert ops.lib().convrot_test_block_norm_timeout(ctypes.byref(a), row, 200_000, stream) == ops.OK
    assert ops.convrot_device_status() == ops.ERR_TIMEOUT
    assert ops.convrot_device_status() == ops.OK          # reported once
    done = torch.stack([(x == r).all(1) for x, r in zip(got, ref)]).all(0)
    left = torch.stack([(x == u).all(1) for x, u in zip(got, untouched)]).all(0)
    assert (done | left).all() and not (done & left).any() and left[row:].all()
    # the rows before are complete, but for those that share a block's range
    per_block = M // torch.cuda.get_device_properties(0).multi_processor_count + 1
    assert int(done.sum()) >= row - per_block

    a = arguments(ops, H, Y, got[0], got[1:], vec, mod, codes)
    assert ops.lib().convrot_block_norm(ctypes.byref(a), stream) == ops.OK
    assert ops.convrot_device_status() == ops.OK
    for x, r in zip(got, ref):
        assert torch.equal(x, r)


def test_only_kernels_that_wait(ops):
    for K in (65, 16392):
        H = torch.zeros(4, K, device="cuda")
        out = torch.zeros(4, K, device="cuda")
        a = arguments(ops, H, H, out, [torch.zeros_like(out)], torch.ones(K, device="cuda"),
                      torch.zeros(2, 3 * K, device="cuda"), False)
        stream = torch.cuda.current_stream().cuda_stream
        assert ops.lib().convrot_test_block_norm_timeout(ctypes.byref(a), 0, 1000, stream) == ops.ERR_UNSUPPORTED
        torch.cuda.synchronize()
