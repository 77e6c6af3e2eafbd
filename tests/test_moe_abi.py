"""The experts' entry points refuse bad calls before they touch a GPU (fake
device addresses: argument checks never dereference)."""
import ctypes

import pytest

BASE = 0x7f0000000000


def at(i):
    return BASE + i * 0x100000000


@pytest.fixture(scope="module")
def ops():
    from int8_hadamard_rotated_gb300 import build, ops as _ops
    build.build()
    _ops.lib()
    return _ops


def route_args(ops, **kw):
    a = ops.convrot_moe_route_args(T=5, n_experts=64, top_k=8, dtype=ops.F32, score=ops.MOE_SIGMOID, logits=at(0), ld=64,
                                   bias=at(1), n_groups=8, top_groups=4, group_top=2, renormalise=1, scale=1.0,
                                   experts=at(2), weights=at(3))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), "ARG"), (dict(n_experts=0), "ARG"), (dict(top_k=0), "ARG"), (dict(dtype=3), "ARG"),
    (dict(score=2), "ARG"), (dict(logits=None), "ARG"), (dict(experts=None), "ARG"), (dict(weights=None), "ARG"),
    (dict(ld=63), "ARG"), (dict(n_groups=0), "ARG"), (dict(n_groups=7), "ARG"), (dict(top_groups=0), "ARG"),
    (dict(top_groups=9), "ARG"), (dict(group_top=0), "ARG"), (dict(group_top=3), "ARG"), (dict(top_k=33), "ARG"),
    (dict(top_groups=1, top_k=9), "ARG"), (dict(scale=float("nan")), "ARG"), (dict(scale=float("inf")), "ARG"),
    (dict(n_experts=2048, ld=2048), "UNSUPPORTED"), (dict(top_groups=8, top_k=33), "UNSUPPORTED"),
    (dict(n_experts=128, ld=128, n_groups=64, top_groups=64), "UNSUPPORTED"), (dict(T=1 << 40), "UNSUPPORTED"),
    (dict(T=1 << 29), "UNSUPPORTED"), (dict(ld=1 << 41), "UNSUPPORTED"),
    (dict(logits=at(0) + 2), "ALIGN"), (dict(bias=at(1) + 1), "ALIGN"), (dict(experts=at(2) + 2), "ALIGN"),
    (dict(weights=at(3) + 3), "ALIGN"), (dict(experts=at(3)), "ALIAS"), (dict(weights=at(0) + 256), "ALIAS"),
    (dict(experts=at(1)), "ALIAS")])
def test_route_refusals(ops, kw, status):
    assert ops.lib().moe_route(ctypes.byref(route_args(ops, **kw)), None) == getattr(ops, "ERR_" + status)


def test_route_no_tokens(ops):
    assert ops.lib().moe_route(ctypes.byref(route_args(ops, T=0, logits=None, experts=None, weights=None)), None) == ops.OK
    assert ops.lib().moe_route(None, None) == ops.ERR_ARG


def test_plan_refusals(ops):
    f = ops.lib().moe_plan
    ok = [at(0), 100, 8, at(1), at(2), at(3), None, 0]

    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a, None)

    assert call(_1=-1) == ops.ERR_ARG and call(_2=0) == ops.ERR_ARG
    for i in (0, 3, 4, 5):
        assert call(**{f"_{i}": None}) == ops.ERR_ARG
        assert call(**{f"_{i}": at(i) + 2}) == ops.ERR_ALIGN
    assert call(_2=1025) == ops.ERR_UNSUPPORTED and call(_1=2 ** 31) == ops.ERR_UNSUPPORTED
    assert call(_3=at(0) + 396) == ops.ERR_ALIAS and call(_4=at(1)) == ops.ERR_ALIAS and call(_5=at(2) + 4) == ops.ERR_ALIAS
    # many choices need scratch, apart from the rest
    size = ops.moe_plan_workspace_size(100000, 8)
    assert ops.moe_plan_workspace_size(100, 8) == 0 < size
    assert ops.moe_plan_workspace_size(-1, 8) == ops.moe_plan_workspace_size(5, 0) == 0
    assert call(_1=100000) == ops.ERR_WORKSPACE
    assert call(_1=100000, _6=at(4), _7=size - 1) == ops.ERR_WORKSPACE
    assert call(_1=100000, _6=at(4) + 2, _7=size) == ops.ERR_ALIGN
    assert call(_1=100000, _6=at(2) + 4096, _7=size) == ops.ERR_ALIAS


def experts(ops, i, N=256, K=512, **kw):
    w = ops.convrot_experts(q=at(i), scale=at(i) + 0x40000000, bias=at(i) + 0x50000000, N=N, q_stride=N * K,
                            scale_stride=(N + 127) // 128 * ((K + 127) // 128), bias_stride=N)
    for k, v in kw.items():
        setattr(w, k, v)
    return w


def linear(ops, w=None, **kw):
    a = dict(Q=at(0), s=at(1), T=40, K=512, order=at(2), offsets=at(3), n=120, E=8, k=3, Y=at(4), ldy=256,
             dtype=ops.BF16, ws=None, size=0)
    a.update(kw)
    w = experts(ops, 8) if w is None else w
    return ops.lib().fp8_expert_linear(a["Q"], a["s"], a["T"], a["K"], a["order"], a["offsets"], a["n"], a["E"], a["k"],
                                       ctypes.byref(w), a["Y"], a["ldy"], a["dtype"], a["ws"], a["size"], None)


def test_linear_refusals(ops):
    for kw in (dict(T=-1), dict(n=-1), dict(K=0), dict(E=0), dict(k=0), dict(Q=None), dict(s=None), dict(offsets=None),
               dict(Y=None), dict(ldy=255), dict(dtype=7), dict(T=0), dict(order=None)):  # (40 rows cannot be 120)
        assert linear(ops, **kw) == ops.ERR_ARG, kw
    for kw in (dict(K=520), dict(Q=at(0) + 8), dict(s=at(1) + 2), dict(order=at(2) + 1), dict(offsets=at(3) + 2),
               dict(Y=at(4) + 1)):
        assert linear(ops, **kw) == ops.ERR_ALIGN, kw
    assert linear(ops, E=1025) == ops.ERR_UNSUPPORTED
    assert linear(ops, ldy=1 << 41) == ops.ERR_UNSUPPORTED
    for kw in (dict(Y=at(0) + 1024), dict(Y=at(1)), dict(Y=at(2) + 256), dict(Y=at(3)), dict(Y=at(8) + 4096),
               dict(Y=at(8) + 0x40000000), dict(Y=at(8) + 0x50000000)):
        assert linear(ops, **kw) == ops.ERR_ALIAS, kw
    for kw, status in ((dict(q=None), "ARG"), (dict(scale=None), "ARG"), (dict(N=-1), "ARG"), (dict(q_stride=256 * 512 - 16), "ARG"),
                       (dict(scale_stride=7), "ARG"), (dict(bias_stride=255), "ARG"), (dict(q=at(8) + 4), "ALIGN"),
                       (dict(q_stride=256 * 512 + 8), "ALIGN"), (dict(scale=at(8) + 0x40000002), "ALIGN"),
                       (dict(bias=at(8) + 0x50000001), "ALIGN"), (dict(q_stride=1 << 39), "UNSUPPORTED")):
        assert linear(ops, w=experts(ops, 8, **kw)) == getattr(ops, "ERR_" + status), kw
    assert linear(ops, n=0, Q=None, offsets=None, Y=None) == ops.OK
    assert linear(ops, w=experts(ops, 8, N=0), Y=None) == ops.OK


def test_linear_workspace(ops):
    """Many rows per expert, taken by an order, are sorted in scratch."""
    n, K, E = 3000, 512, 8
    size = ops.fp8_expert_workspace_size(n, K, E)
    assert size == n * K + (n * 4 * 4 + 255) // 256 * 256 and ops.fp8_expert_workspace_size(100, K, E) == 0
    assert ops.fp8_expert_workspace_size(n, 0, E) == ops.fp8_expert_workspace_size(n, K, 2000) == 0
    kw = dict(n=n, T=1000)
    assert linear(ops, **kw) == ops.ERR_WORKSPACE
    assert linear(ops, **kw, ws=at(5), size=size - 1) == ops.ERR_WORKSPACE
    assert linear(ops, **kw, ws=at(5) + 8, size=size) == ops.ERR_ALIGN
    for ws in (at(0) + 4096, at(1), at(2) + 256, at(4) + 512, at(8) + 512, at(8) + 0x50000000):
        assert linear(ops, **kw, ws=ws, size=size) == ops.ERR_ALIAS, hex(ws)


def test_swiglu_refusals(ops):
    def call(gate=None, up=None, **kw):
        a = dict(Q=at(0), s=at(1), T=40, K=512, order=at(2), offsets=at(3), n=120, E=8, k=3, Qh=at(4), sh=at(5), ws=None,
                 size=0)
        a.update(kw)
        g, u = gate or experts(ops, 8), up or experts(ops, 9)
        return ops.lib().fp8_expert_swiglu(a["Q"], a["s"], a["T"], a["K"], a["order"], a["offsets"], a["n"], a["E"],
                                           a["k"], ctypes.byref(g), ctypes.byref(u), a["Qh"], a["sh"], a["ws"],
                                           a["size"], None)

    assert call(Qh=None) == ops.ERR_ARG and call(sh=None) == ops.ERR_ARG
    assert call(up=experts(ops, 9, N=128)) == ops.ERR_ARG
    assert call(up=experts(ops, 9, q=None)) == ops.ERR_ARG
    assert call(gate=experts(ops, 8, N=250), up=experts(ops, 9, N=250)) == ops.ERR_ALIGN
    assert call(Qh=at(4) + 4) == ops.ERR_ALIGN and call(sh=at(5) + 2) == ops.ERR_ALIGN
    for kw in (dict(sh=at(4) + 256), dict(Qh=at(0)), dict(sh=at(3)), dict(Qh=at(9) + 512), dict(sh=at(8) + 0x40000000)):
        assert call(**kw) == ops.ERR_ALIAS, kw
    assert call(n=3000, T=1000) == ops.ERR_WORKSPACE
    assert call(n=0, T=0) == ops.OK


def test_more_choices_than_the_tokens_have(ops):
    """An order of more choices than T tokens make: a top_k left out or too
    small, which would read other tokens' rows."""
    assert linear(ops, k=1) == linear(ops, k=2) == ops.ERR_ARG
    assert linear(ops, n=121) == ops.ERR_ARG
    assert linear(ops, T=1 << 30, n=(1 << 30) + 1, k=1) == ops.ERR_ARG
    # as many choices as there are, fewer, and products past 31 bits, are taken (as far as the missing workspace)
    assert linear(ops, T=1000, n=3000) == linear(ops, T=1000, n=2900) == ops.ERR_WORKSPACE
    assert linear(ops, T=1000, n=3000, k=2 ** 31 - 1) == ops.ERR_WORKSPACE
    assert linear(ops, T=1 << 28, n=(1 << 28) + 1, k=1 << 30) == ops.ERR_ALIAS  # (Y reaches over the other arrays)
    # without an order top_k has no meaning
    assert linear(ops, T=3000, n=3000, order=None, k=1, Y=at(0)) == ops.ERR_ALIAS
    g, u = experts(ops, 8), experts(ops, 9)
    for k, status in ((1, ops.ERR_ARG), (2, ops.ERR_ARG), (3, ops.ERR_WORKSPACE)):
        assert ops.lib().fp8_expert_swiglu(at(0), at(1), 1000, 512, at(2), at(3), 3000, 8, k, ctypes.byref(g), ctypes.byref(u),
                                           at(4), at(5), None, 0, None) == status


def test_combine_refusals(ops):
    def call(**kw):
        a = dict(rows=at(0), rt=ops.BF16, ldr=256, n=120, place=at(1), w=at(2), T=40, k=3, N=256, res=at(3), ldres=256,
                 Y=at(4), ldy=256, yt=ops.F16)
        a.update(kw)
        return ops.lib().moe_combine(a["rows"], a["rt"], a["ldr"], a["n"], a["place"], a["w"], a["T"], a["k"], a["N"],
                                     a["res"], a["ldres"], a["Y"], a["ldy"], a["yt"], None)

    for kw in (dict(rows=None), dict(place=None), dict(w=None), dict(Y=None), dict(rt=5), dict(yt=-1), dict(ldr=255),
               dict(ldy=255), dict(ldres=255), dict(T=-1), dict(n=-1), dict(N=-1), dict(k=0)):
        assert call(**kw) == ops.ERR_ARG, kw
    assert call(k=33) == ops.ERR_UNSUPPORTED
    for kw in (dict(rows=at(0) + 1), dict(place=at(1) + 2), dict(w=at(2) + 1), dict(res=at(3) + 1), dict(Y=at(4) + 1)):
        assert call(**kw) == ops.ERR_ALIGN, kw
    for kw in (dict(Y=at(0) + 512), dict(Y=at(1)), dict(Y=at(2)), dict(Y=at(3) + 512), dict(Y=at(3), ldy=264)):
        assert call(**kw) == ops.ERR_ALIAS, kw
    assert call(T=0, Y=None) == ops.OK and call(N=0, Y=None, ldr=0, ldy=0, ldres=0) == ops.OK


def test_moe_refusals(ops):
    K, I, N, T, k, E = 512, 256, 384, 40, 3, 8  # noqa: E741
    size = ops.lib().fp8_moe_workspace_size(T, K, I, N, k, E, ops.BF16)
    assert size > 0
    for bad in ((-1, K, I, N, k, E, 2), (T, 0, I, N, k, E, 2), (T, K, 0, N, k, E, 2), (T, K, I, -1, k, E, 2),
                (T, K, I, N, 0, E, 2), (T, K, I, N, 33, E, 2), (T, K, I, N, k, 0, 2), (T, K, I, N, k, 1025, 2),
                (T, K, I, N, k, E, 3), (1 << 40, K, I, N, k, E, 2)):
        assert ops.lib().fp8_moe_workspace_size(*bad) == 0, bad

    def call(gate=None, up=None, down=None, ws=at(7), bytes_=size, **kw):
        g, u = gate or experts(ops, 8, I, K), up or experts(ops, 9, I, K)
        d = down or experts(ops, 10, N, I)
        ref = lambda w: ctypes.cast(ctypes.pointer(w), ctypes.c_void_p).value  # noqa: E731
        a = ops.convrot_moe_args(at(0), ops.BF16, T, K, K, at(1), at(2), k, E, ref(g), ref(u), ref(d), at(3), N, at(4), N,
                                 ops.BF16)
        for n, v in kw.items():
            setattr(a, n, v)
        return ops.lib().fp8_moe(ctypes.byref(a), ws, bytes_, None)

    for kw in (dict(T=-1), dict(K=0), dict(ldx=K - 1), dict(x_dtype=4), dict(y_dtype=4), dict(top_k=0), dict(n_experts=0),
               dict(X=None), dict(experts=None), dict(weights=None), dict(Y=None), dict(ldy=N - 1), dict(ld_res=N - 1),
               dict(gate=experts(ops, 8, I, K, q=None)), dict(up=experts(ops, 9, I - 16, K)),
               dict(down=experts(ops, 10, N, I, q_stride=N * I - 16))):
        assert call(**kw) == ops.ERR_ARG, kw
    for kw in (dict(top_k=33), dict(n_experts=1025), dict(ldx=1 << 41)):
        assert call(**kw) == ops.ERR_UNSUPPORTED, kw
    assert call(ws=None) == ops.ERR_WORKSPACE and call(bytes_=size - 1) == ops.ERR_WORKSPACE
    for kw in (dict(ws=at(7) + 8), dict(X=at(0) + 1), dict(experts=at(1) + 2), dict(Y=at(4) + 1), dict(residual=at(3) + 1),
               dict(weights=at(2) + 2), dict(gate=experts(ops, 8, I - 8, K), up=experts(ops, 9, I - 8, K))):
        assert call(**kw) == ops.ERR_ALIGN, kw
    for kw in (dict(Y=at(0)), dict(Y=at(1)), dict(Y=at(2)), dict(Y=at(3) + 2 * N), dict(Y=at(3), ldy=N + 8),
               dict(Y=at(7) + 256), dict(residual=at(7)), dict(X=at(7)), dict(ws=at(8)), dict(Y=at(10) + 1024)):
        assert call(**kw) == ops.ERR_ALIAS, kw
    assert call(T=0, X=None, Y=None) == ops.OK
    assert ops.lib().fp8_moe(None, None, 0, None) == ops.ERR_ARG


def test_binding_refusals(ops):
    """What the binding refuses by itself (CPU tensors never reach the library)."""
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        ops.moe_route(x, 2)
    with pytest.raises(ValueError):
        ops.moe_plan(torch.zeros(4, dtype=torch.int32), 3)
    with pytest.raises(ValueError):
        ops.fp8_prepare_experts(torch.zeros(2, 16, 16))
