"""The expert linears' failure path on the GPU, made to happen without faulting,
trapping or hanging anything: a test entry point leaves the last block of K of
the last tile out and shortens the limit of the waits, so that the waits for
that block run out. The kernel records CONVROT_ERR_TIMEOUT once and exits, the
other tiles are complete, that one is not written, and the next call is correct."""
import pytest
import torch

from gpu_common import host
from test_moe_gpu import DT, bo, dev_codes, activations, matrices

pytestmark = pytest.mark.gpu

# rows of every expert, features, K, rows of a tile: few rows in tiles of 16 (K
# split over a cluster), 32 and 64 rows, many in tiles of 256
SHAPES = [([3, 0, 5], 200, 1040, 16), ([5] * 40, 640, 272, 16), ([20, 17, 30, 0, 25], 384, 528, 32),
          ([60, 10, 64, 70], 300, 400, 64), ([300, 0, 90, 400], 600, 1280, 256), ([700], 1100, 144, 256)]


def inputs(counts, K):
    n = sum(counts)
    Q, s = bo.fp8_pack(activations(n, n, K).numpy())
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    return dev_codes(Q), torch.from_numpy(s).cuda(), offsets


def last_tile(counts, tile):
    """First row of the last row tile, which belongs to the last expert that has rows."""
    n = sum(counts)
    last = [c for c in counts if c][-1]
    return n - last + (last - 1) // tile * tile


@pytest.mark.parametrize("counts,N,K,tile", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_linear_waits_that_run_out(ops, counts, N, K, tile, out):
    Q, s, offsets = inputs(counts, K)
    w, _ = matrices(N, len(counts), N, K, True)
    ref, got, again = (torch.full((sum(counts), N), 123.0, dtype=DT[out], device="cuda") for _ in range(3))
    ops.fp8_expert_linear(Q, s, offsets, w, Y=ref)
    assert ops.convrot_device_status() == ops.OK
    ops.fp8_test_expert_timeout(Q, s, offsets, w, 1_000_000, got)
    assert ops.convrot_device_status() == ops.ERR_TIMEOUT
    assert ops.convrot_device_status() == ops.OK          # reported once
    ops.fp8_expert_linear(Q, s, offsets, w, Y=again)
    assert ops.convrot_device_status() == ops.OK
    assert torch.equal(again, ref)
    m0, n0 = last_tile(counts, tile), (N - 1) // 256 * 256
    assert torch.equal(got[:m0], ref[:m0]) and torch.equal(got[:, :n0], ref[:, :n0])
    assert (got[m0:, n0:] == 123.0).all()


@pytest.mark.parametrize("counts,N,K,tile", [(c, N // 16 * 16, K, t) for c, N, K, t in SHAPES])
def test_swiglu_waits_that_run_out(ops, counts, N, K, tile):
    Q, s, offsets = inputs(counts, K)
    gate, _ = matrices(N, len(counts), N, K, True)
    up, _ = matrices(N + 1, len(counts), N, K, True)
    n = sum(counts)

    def empty():
        return (torch.full((n, N), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                torch.full((n, bo.n_blocks(N)), 7.0, device="cuda"))

    ref, got, again = empty(), empty(), empty()
    ops.fp8_expert_swiglu(Q, s, None, offsets, 1, gate, up, Q_h=ref[0], s_h=ref[1])
    ops.fp8_test_expert_timeout(Q, s, offsets, gate, 1_000_000, got[0], up=up, s_h=got[1])
    assert ops.convrot_device_status() == ops.ERR_TIMEOUT
    ops.fp8_expert_swiglu(Q, s, None, offsets, 1, gate, up, Q_h=again[0], s_h=again[1])
    assert ops.convrot_device_status() == ops.OK
    (rq, rs), (gq, gs), (aq, as_) = ((host(q.view(torch.uint8)), host(t)) for q, t in (ref, got, again))
    assert (aq == rq).all() and (as_ == rs).all()
    m0, n0 = last_tile(counts, tile), (N - 1) // 128 * 128
    assert (gq[:m0] == rq[:m0]).all() and (gq[:, :n0] == rq[:, :n0]).all()
    assert (gs[:m0] == rs[:m0]).all() and (gs[:, :n0 // 128] == rs[:, :n0 // 128]).all()
    assert (gq[m0:, n0:] == 0x55).all() and (gs[m0:, n0 // 128:] == 7.0).all()


def test_refusals(ops):
    Q, s, offsets = inputs([3, 2], 32)
    w, _ = matrices(1, 2, 16, 32, False)
    with pytest.raises(ops.ConvrotError):
        ops.fp8_test_expert_timeout(Q, s, offsets, w, 0, torch.empty(5, 16, device="cuda"))
    torch.cuda.synchronize()
