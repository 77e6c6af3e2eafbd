"""The fp8 linears' failure path on the GPU, made to happen without faulting,
trapping or hanging anything: a test entry point leaves the last block of K of
the last tile out and shortens the limit of the waits, so that the waits for
that block run out. The kernel records CONVROT_ERR_TIMEOUT once and exits, the
other tiles are complete, that one is not written, and the next call is correct."""
import pytest
import torch

from test_fp8_linear_gpu import DT, packed

pytestmark = pytest.mark.gpu

# few rows (16, 32 and 64 columns of accumulators), one wave of tiles, CTA
# pairs: with the rows and features of a tile
SHAPES = [(9, [384], 1040, 16, 128), (24, [128, 200], 4096, 32, 128), (64, [1283], 272, 64, 128),
          (300, [640], 1280, 128, 128), (1000, [2304], 128, 128, 128), (3000, [2000, 1283], 528, 256, 256)]


def call(ops, Qx, sx, ws, Ys, wait_ns=None):
    arr = (ops.convrot_fp8_weight * len(ws))()
    for d, (q, s), y in zip(arr, ws, Ys):
        d.q, d.scale, d.bias, d.N, d.Y, d.ldy = q.data_ptr(), s.data_ptr(), None, q.shape[0], y.data_ptr(), y.shape[1]
    dt = {torch.float32: ops.F32, torch.float16: ops.F16, torch.bfloat16: ops.BF16}[Ys[0].dtype]
    M, K = Qx.shape
    stream = torch.cuda.current_stream().cuda_stream
    if wait_ns is None:
        return ops.lib().fp8_linear_packed(Qx.data_ptr(), sx.data_ptr(), M, K, arr, len(ws), dt, stream)
    return ops.lib().fp8_test_linear_timeout(Qx.data_ptr(), sx.data_ptr(), M, K, arr, len(ws), dt, wait_ns, stream)


def run_out(ops, M, Ns, K, out):
    """(outputs of a normal call, of one whose waits run out)"""
    Qx, sx, _, _ = packed(M, M, K)
    ws = [packed(n, n, K, 128)[:2] for n in Ns]
    ref, got = ([torch.full((M, n), 123.0, dtype=DT[out], device="cuda") for n in Ns] for _ in range(2))
    assert call(ops, Qx, sx, ws, ref) == ops.OK
    assert ops.convrot_device_status() == ops.OK
    assert call(ops, Qx, sx, ws, got, 1_000_000) == ops.OK
    assert ops.convrot_device_status() == ops.ERR_TIMEOUT
    assert ops.convrot_device_status() == ops.OK          # reported once
    again = [torch.full_like(y, 123.0) for y in ref]
    assert call(ops, Qx, sx, ws, again) == ops.OK
    assert ops.convrot_device_status() == ops.OK
    assert all(torch.equal(a, r) for a, r in zip(again, ref))
    return ref, got


@pytest.mark.parametrize("M,Ns,K,rows,cols", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_waits_that_run_out(ops, M, Ns, K, rows, cols, out):
    ref, got = run_out(ops, M, Ns, K, out)
    for y, r in zip(got[:-1], ref):
        assert torch.equal(y, r)
    m0, n0 = (M - 1) // rows * rows, (Ns[-1] - 1) // cols * cols      # the last tile
    assert torch.equal(got[-1][:m0], ref[-1][:m0]) and torch.equal(got[-1][:, :n0], ref[-1][:, :n0])


def test_streamed_weights_have_no_waits(ops):
    Qx, sx, _, _ = packed(8, 8, 256)
    y = torch.full((8, 64), 123.0, device="cuda")
    assert call(ops, Qx, sx, [packed(1, 64, 256, 128)[:2]], [y], 1000) == ops.ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert (y == 123.0).all()


@pytest.mark.parametrize("M,Ns,K,rows,cols", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_unfinished_sums_are_not_stored(ops, M, Ns, K, rows, cols, out):
    """Also where only one of the blocks of threads that share the tile's K
    waited in vain."""
    _, got = run_out(ops, M, Ns, K, out)
    m0, n0 = (M - 1) // rows * rows, (Ns[-1] - 1) // cols * cols
    assert (got[-1][m0:, n0:] == 123.0).all()


def test_one_status_call_clears_every_word(ops):
    """A linear's timeout and samples out of range of two types of block norm:
    the timeout is reported, and all are cleared."""
    Qx, sx, _, _ = packed(2, 16, 256)
    y = torch.empty(16, 128, device="cuda")
    for _ in range(2):
        for dtype in (torch.bfloat16, torch.float32):
            ops.convrot_block_norm(torch.ones(2, 64, dtype=dtype, device="cuda"), scale=torch.ones(2, 64, device="cuda"),
                                   row_sample=torch.tensor([0, 5], dtype=torch.int32, device="cuda"))
        assert call(ops, Qx, sx, [packed(1, 128, 256, 128)[:2]], [y], 100_000) == ops.OK
        assert ops.convrot_device_status() == ops.ERR_TIMEOUT
        assert ops.convrot_device_status() == ops.OK
