"""Refusals of the routing-from-logits, gradient and adapter entry points:
host checks only, on fake addresses that are never dereferenced."""
import ctypes

import pytest

import top_routing_expert_gemm_b200 as moe
from top_routing_expert_gemm_b200 import build

INVALID, UNSUPPORTED, WORKSPACE, CUDA = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    build.build()
    return moe.lib()


def _p(addr=256):
    return ctypes.c_void_p(addr)


def _route(**kw):
    base = dict(T=64, n_experts=64, top_k=8, score=moe.MOE_SCORE_SIGMOID, n_groups=8, topk_groups=4, group_top=2)
    base.update(kw)
    return moe.make_route_config(**base)


def _topk(L, cfg, logits=256, bias=None, ids=256, w=256):
    return L.moe_route_topk(ctypes.byref(cfg) if cfg else None, _p(logits), _p(bias), _p(ids), _p(w), None)


def _back(L, cfg, logits=256, ids=256, g=256, counts=256, balance=0.0, z=0.0, grad=512):
    return L.moe_route_backward(ctypes.byref(cfg) if cfg else None, _p(logits), _p(ids), _p(g), _p(counts), balance,
                                z, _p(grad), None)


def test_route_config_struct_layout():
    assert ctypes.sizeof(moe.MoeRouteConfig) == 56
    assert moe.MoeRouteConfig.n_experts.offset == 16
    assert moe.MoeRouteConfig.weight_scale.offset == 48


@pytest.mark.parametrize("kw,want", [
    (dict(T=-1), INVALID), (dict(n_experts=0), INVALID), (dict(top_k=0), INVALID), (dict(n_groups=0), INVALID),
    (dict(n_groups=7), INVALID), (dict(topk_groups=0), INVALID), (dict(topk_groups=9), INVALID),
    (dict(top_k=9, topk_groups=1), INVALID), (dict(group_top=0), INVALID), (dict(group_top=3), INVALID),
    (dict(score=2), INVALID), (dict(renormalise=2), INVALID), (dict(logits_dtype=2), INVALID),
    (dict(logits_stride=63), INVALID), (dict(logits_stride=-64), INVALID),
    (dict(weight_scale=float("inf")), INVALID), (dict(weight_scale=float("nan")), INVALID),
    (dict(n_experts=1032, n_groups=8), UNSUPPORTED), (dict(top_k=17), UNSUPPORTED),
    (dict(n_experts=66, n_groups=33, topk_groups=33, top_k=1), UNSUPPORTED), (dict(T=1 << 28), UNSUPPORTED),
])
def test_route_config_refusals(L, kw, want):
    assert _topk(L, _route(**kw)) == want
    assert _back(L, _route(**kw)) == want


def test_route_argument_refusals(L):
    cfg = _route()
    assert _topk(L, None) == INVALID and _back(L, None) == INVALID
    for name in ("logits", "ids", "w"):
        assert _topk(L, cfg, **{name: None}) == INVALID
        assert _topk(L, cfg, **{name: 260}) == INVALID
    assert _topk(L, cfg, bias=8) == INVALID
    assert _topk(L, _route(T=0), logits=None, ids=None, w=None) == 0
    assert _back(L, cfg, logits=None) == INVALID and _back(L, cfg, grad=None) == INVALID
    assert _back(L, cfg, grad=256) == INVALID          # in place
    assert _back(L, cfg, ids=None) == INVALID          # grad_w without ids
    assert _back(L, cfg, balance=1.0, counts=None) == INVALID
    assert _back(L, cfg, balance=float("nan")) == INVALID and _back(L, cfg, z=float("inf")) == INVALID
    for name in ("logits", "ids", "g", "grad"):
        assert _back(L, cfg, **{name: 264}) == INVALID
    assert _back(L, _route(T=0), logits=None, grad=None) == 0


def _cfg(**kw):
    base = dict(T=64, d_model=256, n_experts=8, top_k=2, d_ff=512, dtype=moe.MOE_BF16, gating=1)
    base.update(kw)
    return moe.make_config(**base)


def test_combine_backward_refusals(L):
    def call(cfg, gy=256, yp=256, row=256, w=256, gp=256, gw=256):
        return L.moe_combine_backward(ctypes.byref(cfg) if cfg else None, _p(gy), _p(yp), _p(row), _p(w), _p(gp),
                                      _p(gw), None)
    assert call(None) == INVALID and call(_cfg(top_k=9)) == INVALID and call(_cfg(n_experts=2000)) == UNSUPPORTED
    assert call(_cfg(), gp=None, gw=None) == INVALID   # nothing asked for
    assert call(_cfg(), gy=None) == INVALID and call(_cfg(), row=None) == INVALID
    assert call(_cfg(), yp=None) == INVALID            # grad_w needs the rows
    assert call(_cfg(), w=None) == INVALID             # grad_y_perm needs the weights
    for name in ("gy", "yp", "row", "w", "gp", "gw"):
        assert call(_cfg(), **{name: 264}) == INVALID
    assert call(_cfg(T=0), gy=None, yp=None, row=None, w=None) == 0


def test_injected_launch_failure(L, monkeypatch):
    monkeypatch.setenv("MOE_FAULT", "launch")
    cfg = _cfg()
    assert _topk(L, _route()) == CUDA and _back(L, _route()) == CUDA
    assert L.moe_combine_backward(ctypes.byref(cfg), _p(), _p(), _p(), _p(), _p(), _p(), None) == CUDA
    assert _topk(L, _route(top_k=0)) == INVALID


# ------------------------------------------------------------------ adapters
def _plan(L, cfg, ad, offsets=256, perm=256, ta=256, plan=256, nb=1 << 40):
    return L.moe_adapter_plan(ctypes.byref(cfg), ctypes.byref(ad) if ad else None, _p(offsets), _p(perm), _p(ta),
                              _p(plan), nb, None)


def _apply(L, cfg, ad, which="down", plan=256, nb=1 << 40, x=256, a=256, b=256, scale=256, base=256, out=512):
    f = L.moe_adapter_gate_up if which == "gate_up" else L.moe_adapter_down
    return f(ctypes.byref(cfg), ctypes.byref(ad) if ad else None, _p(plan), nb, _p(x), _p(a), _p(b), _p(scale),
             _p(base), _p(out), None)


@pytest.mark.parametrize("kw,want", [
    (dict(n_adapters=0, rank=8), INVALID), (dict(n_adapters=-1, rank=8), INVALID), (dict(n_adapters=2, rank=0), INVALID),
    (dict(n_adapters=2, rank=12), INVALID), (dict(n_adapters=2, rank=8, shared=2), INVALID),
    (dict(n_adapters=2, rank=8, shared=1), INVALID),  # the layer has no shared expert
    (dict(n_adapters=2, rank=136), UNSUPPORTED), (dict(n_adapters=65537, rank=8), UNSUPPORTED),
])
def test_adapter_config_refusals(L, kw, want):
    ad = moe.make_adapter_config(**kw)
    assert moe.moe_adapter_plan_bytes(_cfg(), ad) == 0
    assert _plan(L, _cfg(), ad) == want and _apply(L, _cfg(), ad) == want and _apply(L, _cfg(), ad, "gate_up") == want


def test_adapter_argument_refusals(L):
    cfg, ad = _cfg(), moe.make_adapter_config(3, 16)
    need = moe.moe_adapter_plan_bytes(cfg, ad)
    assert need > 0 and need % 256 == 0
    assert _plan(L, cfg, None) == INVALID and _apply(L, cfg, None) == INVALID
    assert _plan(L, _cfg(top_k=9), ad) == INVALID
    many = _cfg(n_experts=1024)
    assert _plan(L, many, moe.make_adapter_config(8192, 8)) == UNSUPPORTED  # experts x adapters
    assert moe.moe_adapter_plan_bytes(many, moe.make_adapter_config(8191, 8)) > 0
    for name in ("offsets", "perm", "ta", "plan"):
        assert _plan(L, cfg, ad, **{name: None}) == INVALID
        assert _plan(L, cfg, ad, **{name: 264}) == INVALID
    assert _plan(L, cfg, ad, plan=16) == INVALID               # 256-byte alignment
    assert _plan(L, cfg, ad, nb=need - 1) == WORKSPACE and _apply(L, cfg, ad, nb=need - 1) == WORKSPACE
    sh = _cfg(n_shared=1, d_ff_shared=512)
    assert _plan(L, sh, moe.make_adapter_config(3, 16, 1)) == INVALID   # a shared expert has no dispatch
    for which in ("gate_up", "down"):
        for name in ("plan", "x", "a", "b", "scale", "base", "out"):
            assert _apply(L, cfg, ad, which, **{name: None}) == INVALID
            assert _apply(L, cfg, ad, which, **{name: 264}) == INVALID
        assert _apply(L, cfg, ad, which, x=512) == INVALID     # the result over the input
    assert _apply(L, cfg, ad, "gate_up", base=512) == INVALID  # SwiGLU halves the columns: not in place
    assert _apply(L, _cfg(T=0), ad, x=None, a=None, plan=None) == 0


def _forward(L, cfg, rc, ad, ws=256, nb=1 << 40, x=256, logits=256, wgu=256, wd=256, sgu=None, sd=None, y=256):
    return L.moe_forward_routed(ctypes.byref(cfg), ctypes.byref(rc), ctypes.byref(ad) if ad else None, _p(x),
                                _p(logits), None, _p(wgu), _p(wd), _p(sgu), _p(sd), _p(y), None, None, None, _p(ws),
                                nb, None)


def _layer_route(cfg, **kw):
    return moe.make_route_config(cfg.T, cfg.n_experts, cfg.top_k, moe.MOE_SCORE_SOFTMAX, **kw)


def test_forward_routed_refusals(L):
    cfg = _cfg()
    rc = _layer_route(cfg)
    need = moe.moe_forward_routed_workspace_bytes(cfg)
    assert need == moe.moe_workspace_bytes(cfg)
    assert _forward(L, cfg, rc, None, nb=need - 1) == WORKSPACE
    for bad in (dict(T=63), dict(n_experts=16), dict(top_k=3)):
        assert _forward(L, cfg, _layer_route(_cfg(**bad)), None) == INVALID
    for name in ("ws", "x", "logits", "wgu", "wd", "y"):
        assert _forward(L, cfg, rc, None, **{name: None}) == INVALID
        assert _forward(L, cfg, rc, None, **{name: 264}) == INVALID
    assert _forward(L, _cfg(n_shared=1, d_ff_shared=512), rc, None) == INVALID  # shared weights missing
    p = 256
    ad = moe.make_adapters(4, 16, p, p, p, p, p, p)
    more = moe.moe_forward_routed_workspace_bytes(cfg, ad)
    assert more > need + 128 * 2 * 512 * 2                     # the pre-activations
    assert _forward(L, cfg, rc, ad, nb=more - 1) == WORKSPACE
    assert moe.moe_forward_routed_workspace_bytes(cfg, moe.make_adapters(4, 16, p, p, a_down=p, b_down=p)) < more
    for bad in (moe.make_adapters(4, 16, None, p, p, p), moe.make_adapters(4, 16, p, None, p, p),
                moe.make_adapters(4, 16, p, p, p, None), moe.make_adapters(4, 16, p, p, b_down=p),
                moe.make_adapters(4, 12, p, p, p, p), moe.make_adapters(4, 16, p, p, 264, p),
                moe.make_adapters(4, 16, p, p, a_down_shared=p, b_down_shared=p)):
        assert moe.moe_forward_routed_workspace_bytes(cfg, bad) == 0
        assert _forward(L, cfg, rc, bad) == INVALID


def test_injected_launch_failure_of_the_adapter_calls(L, monkeypatch):
    monkeypatch.setenv("MOE_FAULT", "launch")
    cfg, ad = _cfg(), moe.make_adapter_config(3, 16)
    assert _plan(L, cfg, ad) == CUDA and _apply(L, cfg, ad) == CUDA and _apply(L, cfg, ad, "gate_up") == CUDA
    assert _forward(L, cfg, _layer_route(cfg), None) == CUDA
    assert _plan(L, cfg, ad, nb=16) == WORKSPACE


def test_adapter_struct_layouts():
    assert ctypes.sizeof(moe.MoeAdapterConfig) == 16
    assert ctypes.sizeof(moe.MoeAdapters) == 88 and moe.MoeAdapters.a_gate_up.offset == 24
    assert moe.moe_status_string(8) == "adapter id out of range"


def test_pair_limit_of_the_routed_experts_holds_beside_shared_adapters(L):
    """experts x adapters is limited for the routed experts' plan; the shared
    expert's plan has one pair per adapter."""
    cfg = _cfg(n_experts=1024, n_shared=1, d_ff_shared=512)
    rc = _layer_route(cfg)
    p, four = 256, dict(a_gate_up_shared=256, b_gate_up_shared=256, a_down_shared=256, b_down_shared=256)
    routed = (dict(a_gate_up=p, b_gate_up=p), dict(a_down=p, b_down=p),
              dict(a_gate_up=p, b_gate_up=p, a_down=p, b_down=p))
    for n in (8192, 40000, 65536):
        for part in routed:
            for ad in (moe.make_adapters(n, 16, p, p, **part), moe.make_adapters(n, 16, p, p, **part, **four)):
                assert moe.moe_forward_routed_workspace_bytes(cfg, ad) == 0
                assert _forward(L, cfg, rc, ad, sgu=p, sd=p) == UNSUPPORTED
        assert moe.moe_forward_routed_workspace_bytes(cfg, moe.make_adapters(n, 16, p, p, **four)) > 0
    for part in routed:
        assert moe.moe_forward_routed_workspace_bytes(cfg, moe.make_adapters(8191, 16, p, p, **part, **four)) > 0
