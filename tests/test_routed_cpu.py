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
