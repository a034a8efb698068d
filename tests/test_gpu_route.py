"""Routing from logits, its gradient and the combine's gradient on the GPU,
against the float64 oracle.

Tolerances.  One fp32 operation is off by u = 2^-24 of its result, expf by at
most 4 u.  A weight is a quotient of an exponential (its argument, a
difference of order 10, off by 10 u) and a sum of such (at most 37 additions):
below 2 (10 + 4 + 2) + 37 + 3 < 80 u.  Gradients multiply two or three such
factors and subtract sums of k or E of them: below 200 u of the largest term.
The last rounding is half a step: u in fp32, 2^-8 in bf16.
"""
import numpy as np
import pytest
import torch

import oracle
import top_routing_expert_gemm_b200 as moe

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {"f32": U, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
LOW = torch.finfo(torch.float32).min
SCORE = {"sigmoid": moe.MOE_SCORE_SIGMOID, "softmax": moe.MOE_SCORE_SOFTMAX}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _f64(t):
    return t.detach().cpu().double().numpy()


def _logits(T, E, dtype, seed, masks=0.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    wide = torch.full((T, E + pad), 99.0).to(DT[dtype])
    l = torch.randn(T, E, generator=g)
    if masks:
        off = torch.rand(T, E, generator=g) < masks
        kind = torch.randint(0, 3, (T, E), generator=g)
        l = l.to(DT[dtype])
        low = torch.finfo(DT[dtype]).min
        for i, v in enumerate((float("-inf"), float("nan"), low)):
            l[off & (kind == i)] = v
        if T > 2:
            l[T - 1] = low  # a padding row
            l[T // 2] = float("-inf")
    wide[:, :E] = l.to(DT[dtype])
    return wide.cuda()[:, :E]


def _cfg(l, k, score, G=1, Gk=1, gtop=1, renorm=1, scale=1.0):
    return moe.make_route_config(l.shape[0], l.shape[1], k, SCORE[score], G, Gk, gtop, renorm, scale,
                                 moe.MOE_BF16 if l.dtype == torch.bfloat16 else moe.MOE_F32, l.stride(0))


def _run(l, bias, cfg):
    ids = torch.full((cfg.T, cfg.top_k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((cfg.T, cfg.top_k), float("nan"), device="cuda")
    moe.moe_route_topk(cfg, l, bias, ids, w)
    torch.cuda.synchronize()
    return ids, w


def _check(l, bias, cfg, score, ids, w, dtype):
    want_ids, want_w, gap = oracle.route_logits(_f64(l), None if bias is None else _f64(bias), cfg.top_k, score,
                                                cfg.n_groups, cfg.topk_groups, cfg.group_top, bool(cfg.renormalise),
                                                float(cfg.weight_scale), dtype)
    # binary64 sums of two scores are off by a few 2^-53.  Of 512 choices within
    # 6e-8 (the closest case) the 8 first gaps are about 1.2e-10 each: one falls
    # below 1e-13 in 0.7% of the rows.
    sure = (gap > 1e-13) | (gap == 0.0)
    assert sure.mean() > 0.95
    got = ids.cpu().numpy()
    assert np.array_equal(got[sure], want_ids[sure])
    gw = _f64(w)
    assert np.all(np.abs(gw[sure] - want_w[sure]) <= 80 * U * want_w[sure] + 1e-37)
    return want_ids


SHAPES = [  # E, k, G, Gk, group_top
    (1, 1, 1, 1, 1), (5, 2, 1, 1, 1), (8, 2, 1, 1, 1), (60, 6, 1, 1, 1), (128, 4, 1, 1, 1), (256, 8, 8, 4, 2),
    (256, 8, 8, 4, 1), (160, 6, 8, 3, 2), (160, 6, 8, 3, 1), (64, 16, 32, 9, 2), (96, 5, 3, 2, 2), (256, 4, 2, 1, 2),
    (384, 8, 1, 1, 1), (1000, 13, 10, 3, 2), (1024, 16, 16, 4, 2), (32, 4, 32, 5, 2), (30, 3, 15, 4, 1),
]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,G,Gk,gtop", SHAPES)
@pytest.mark.parametrize("dtype,bias,masks,pad", [("f32", True, 0.0, 0), ("bf16", False, 0.3, 3),
                                                  ("f32", False, 0.1, 8), ("bf16", True, 0.7, 0)])
def test_route_matches_the_oracle(score, E, k, G, Gk, gtop, dtype, bias, masks, pad):
    l = _logits(53, E, dtype, E + k, masks, pad)
    b = (0.2 * torch.randn(E, generator=torch.Generator().manual_seed(1))).cuda() if bias else None
    renorm, scale = (1, 2.5) if (E + pad) % 2 else (int(score == "sigmoid"), 1.0)
    cfg = _cfg(l, k, score, G, Gk, gtop, renorm, scale)
    ids, w = _run(l, b, cfg)
    _check(l, b, cfg, score, ids, w, dtype)


@pytest.mark.parametrize("T", [1, 2, 3, 129, 20011])
def test_route_batch_sizes(T):
    """One row, odd batches, and more rows than the grid has warps."""
    l = _logits(T, 64, "f32", T)
    b = (0.1 * torch.randn(64, generator=torch.Generator().manual_seed(2))).cuda()
    cfg = _cfg(l, 6, "sigmoid", 8, 3, 2, 1, 2.5)
    ids, w = _run(l, b, cfg)
    rows = torch.arange(T)[:: max(1, T // 500)]
    sub = l[rows.cuda()]
    _check(sub, b, _cfg(sub, 6, "sigmoid", 8, 3, 2, 1, 2.5), "sigmoid", ids[rows.cuda()], w[rows.cuda()], "f32")
    again, w2 = _run(l, b, cfg)
    assert torch.equal(ids, again) and torch.equal(w, w2)


def _repeated(l, T=8219):
    """The rows of l over and over, in the same padded layout."""
    wide = torch.full((T, l.stride(0)), 99.0, device="cuda").to(l.dtype)
    wide[:, :l.shape[1]] = l.repeat(-(-T // l.shape[0]), 1)[:T]
    return wide[:, :l.shape[1]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,G,Gk,gtop", SHAPES + [(510, 7, 30, 4, 2), (512, 16, 1, 1, 1), (17, 3, 1, 1, 1)])
@pytest.mark.parametrize("dtype,bias,masks,pad", [("f32", True, 0.0, 0), ("bf16", False, 0.3, 3),
                                                  ("f32", False, 0.1, 8), ("bf16", True, 0.7, 0)])
def test_route_of_many_rows_matches_the_oracle(score, E, k, G, Gk, gtop, dtype, bias, masks, pad):
    """Batches large enough for four threads per row, on the rows of the test above."""
    few = _logits(53, E, dtype, E + k, masks, pad)
    l = _repeated(few)
    b = (0.2 * torch.randn(E, generator=torch.Generator().manual_seed(1))).cuda() if bias else None
    for renorm, scale in ((1, 2.5), (0, 1.0)):
        cfg = _cfg(l, k, score, G, Gk, gtop, renorm, scale)
        ids, w = _run(l, b, cfg)
        assert torch.equal(ids[53:106], ids[:53]) and torch.equal(ids[8162:8215], ids[:53])
        assert torch.equal(w[53:106], w[:53]) and torch.equal(w[8215], w[0])
        _check(few, b, _cfg(few, k, score, G, Gk, gtop, renorm, scale), score, ids[:53], w[:53], dtype)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E", [64, 512])
@pytest.mark.parametrize("G,Gk,gtop", [(1, 1, 1), (8, 3, 2), (8, 3, 1)])
def test_choices_closer_than_fp32_are_decided_as_the_logits_say(score, G, Gk, gtop, E):
    """A bias that cancels the scores to within half an fp32 step: every order
    hangs on bits that fp32 scores do not have."""
    T, k = 96, 8
    rng = np.random.default_rng(9)
    base = rng.standard_normal(E).astype(np.float32)
    l = np.repeat(base[None], T, 0)
    for _ in range(3):  # rows a few fp32 steps apart
        l = np.where(rng.random((T, E)) < 0.3, np.nextafter(l, np.float32(9)), l)
    s = oracle.route_scores(base.astype(np.float64), score)
    bias = torch.from_numpy((0.5 - s).astype(np.float32)).cuda()
    lt = torch.from_numpy(l).cuda()
    cfg = _cfg(lt, k, score, G, Gk, gtop)
    ids, w = _run(lt, bias, cfg)
    _check(lt, bias, cfg, score, ids, w, "f32")
    many = _repeated(lt)
    ids2, w2 = _run(many, bias, _cfg(many, k, score, G, Gk, gtop))
    _check(lt, bias, cfg, score, ids2[:T], w2[:T], "f32")
    assert torch.equal(ids2[-37:], ids2[8219 - 37 - T:8219 - T])


def test_ties_zero_bias_and_equal_rows_take_the_lowest_index():
    for E, G, Gk, gtop in ((40, 1, 1, 1), (64, 8, 2, 2), (30, 5, 2, 2)):
        l = torch.zeros(9, E, device="cuda")
        l[3:, 7] = 1.0
        for bias in (None, torch.zeros(E, device="cuda"), torch.full((E,), 0.25, device="cuda")):
            for score in ("sigmoid", "softmax"):
                cfg = _cfg(l, 3, score, G, Gk, gtop)
                ids, w = _run(l, bias, cfg)
                assert ids[:3].eq(torch.arange(3, device="cuda", dtype=torch.int32)).all()
                _check(l, bias, cfg, score, ids, w, "f32")
                many = _repeated(l)
                ids2, _ = _run(many, bias, _cfg(many, 3, score, G, Gk, gtop))
                assert torch.equal(ids2[9:18], ids) and torch.equal(ids2[8208:8217], ids)


def test_extreme_logits_and_biases():
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    l = torch.tensor([[inf, 1.0, -2.0, inf, 0.0], [-900.0, -901.0, -2000.0, low, nan], [1e30, -1e30, 3.0, 2.0, 1e30],
                      [-0.0, 0.0, -1e-40, 1e-40, -inf], [low, nan, -inf, low, nan], [88.0, 89.0, 300.0, -88.0, -300.0]],
                     device="cuda")
    for score in ("sigmoid", "softmax"):
        for renorm in (0, 1):
            cfg = _cfg(l, 3, score, renorm=renorm)
            ids, w = _run(l, None, cfg)
            # ranks by the logit: saturated scores do not tie
            assert ids.cpu().tolist() == [[0, 3, 1], [0, 1, 2], [0, 4, 2], [3, 0, 1], [-1] * 3, [2, 1, 0]]
            want_ids, want_w, _ = oracle.route_logits(_f64(l), None, 3, score, renormalise=bool(renorm))
            assert np.all(np.abs(_f64(w) - want_w) <= 80 * U * want_w + 1e-37)
            many = _repeated(l)
            ids2, w2 = _run(many, None, _cfg(many, 3, score, renorm=renorm))
            assert torch.equal(ids2[6:12], ids)
            assert np.all(np.abs(_f64(w2)[6:12] - want_w) <= 80 * U * want_w + 1e-37)
    b = torch.tensor([-inf, nan, inf, inf, -3.0], device="cuda")
    ids, w = _run(torch.zeros(2, 5, device="cuda"), b, _cfg(torch.zeros(2, 5, device="cuda"), 4, "softmax"))
    assert ids.cpu().tolist() == [[2, 3, 4, -1]] * 2
    assert torch.allclose(w, torch.tensor([[1 / 3, 1 / 3, 1 / 3, 0.0]], device="cuda").expand(2, 4))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("b,G,want", [
    # sums of a group's two best that pass fp32's range: 5e38 < 6e38 < inf
    ([2e38, 3e38, 3e38, 3e38, float("inf"), 0.0, 0.0, 0.0], 4, [4, 2, 3, 5]),
    ([2e38, 3e38, 0.0, 3e38, 3e38, 0.0, float("inf"), 0.0, 0.0], 3, [6, 3, 4, 5]),
    # an infinite bias beside excluded experts and equal choices: the fifth slot stays empty
    ([float("inf"), -float("inf"), float("inf"), 0.25, 0.25, float("nan"), -float("inf"), -float("inf")], 1,
     [0, 2, 3, 4, -1]),
])
def test_biases_past_the_range_of_fp32(score, b, G, want):
    bias = torch.tensor(b, device="cuda")
    for T in (1, 33, 8201):
        l = torch.zeros(T, len(b), device="cuda")
        ids, w = _run(l, bias, _cfg(l, len(want), score, G, min(G, 2), 2 if G > 1 else 1))
        assert torch.equal(ids.cpu(), torch.tensor(want, dtype=torch.int32).expand(T, -1))
        share = torch.tensor([1.0 if i >= 0 else 0.0 for i in want])
        assert torch.allclose(w.cpu(), (share / share.sum()).expand(T, -1))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("masked,b,G,want", [
    # sums of two of about -6.8e38 pass fp32's range, and still come before a group that is masked throughout
    ([0, 1], [0.0, 0.0, LOW, LOW, LOW, LOW, 0.5, 0.5], 4, [6, 7, 2, 3]),
    ([0, 1, 2], [0.0, 0.0, 0.0, LOW, LOW, LOW, 0.5, 0.5, 0.5], 3, [6, 7, 8, 3]),
    # and differ among themselves: -5e38 before -6e38, -4e38 before both
    ([], [-3e38, -3e38, -2e38, -3e38, -2e38, -2e38, -3e38, -3e38], 4, [2, 4, 5, 3]),
    ([], [-3e38, -3e38, -3e38, -2e38, -3e38, -3e38, -2e38, -2e38, -3e38], 3, [3, 6, 7, 4]),
])
def test_group_sums_below_the_range_of_fp32(score, masked, b, G, want):
    bias = torch.tensor(b, device="cuda")
    for T in (1, 33, 8201):
        l = torch.zeros(T, len(b), device="cuda")
        l[:, masked] = float("-inf")
        cfg = _cfg(l, len(want), score, G, 2, 2)
        ids, w = _run(l, bias, cfg)
        ref, _, _ = oracle.route_logits(_f64(l[:1]), _f64(bias), len(want), score, G, 2, 2)
        assert ref[0].tolist() == want
        assert torch.equal(ids.cpu(), torch.tensor(want, dtype=torch.int32).expand(T, -1))
        assert torch.allclose(w, torch.full_like(w, 0.25))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,k,G,Gk,gtop", [(64, 8, 8, 3, 2), (64, 6, 8, 2, 1), (30, 5, 5, 2, 2), (256, 12, 8, 4, 2),
                                           (40, 4, 1, 1, 1)])
@pytest.mark.parametrize("span", [24, 60, 120])
def test_saturated_scores_rank_by_their_logits(score, E, k, G, Gk, gtop, span):
    """Without a bias, or with zeros, scores that are equal in binary64 (sigmoids of
    logits above 37, differences of a denominator's last bit) still rank by the
    logits; whole numbers, so that logits tie too, and then the lower index wins.
    A group's sum of two is compared as a sum: equal ones keep the lower group; where
    its one best counts, that one's logit does, so the picks are those of a tenth
    of the logits, which does not saturate."""
    l = torch.randint(-span // 4, span + 1, (48, E), generator=torch.Generator().manual_seed(E + span)).float().cuda()
    l[5] = 50.0
    l[6, ::3] = float("-inf")
    want, want_w, _ = oracle.route_logits(_f64(l), None, k, score, G, Gk, gtop)
    if gtop == 1:
        want, _, _ = oracle.route_logits(0.1 * _f64(l), None, k, score, G, Gk, gtop)
        ls = np.vectorize(lambda v: -np.logaddexp(0.0, -v))(_f64(l)) if score == "sigmoid" else _f64(l)
        w = np.exp(np.take_along_axis(ls, want, 1) - np.take_along_axis(ls, want, 1).max(1, keepdims=True))
        want_w = w / w.sum(1, keepdims=True)
    many = _repeated(l)
    for bias in (None, torch.zeros(E, device="cuda")):
        ids, w = _run(l, bias, _cfg(l, k, score, G, Gk, gtop))
        assert np.array_equal(ids.cpu().numpy(), want)
        assert np.all(np.abs(_f64(w) - want_w) <= 80 * U * want_w + 1e-37)
        ids2, _ = _run(many, bias, _cfg(many, k, score, G, Gk, gtop))
        assert torch.equal(ids2[:48], ids) and torch.equal(ids2[48 * 170:48 * 171], ids)


def test_rows_past_32_bit_offsets():
    """Row strides that take the last rows past 2^32 bytes and 2^31 elements."""
    T, E, stride = 2100, 16, 1 << 20
    wide = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    l = torch.as_strided(wide, (T, E), (stride, 1))
    l.copy_(_logits(T, E, "bf16", 5))
    cfg = _cfg(l, 2, "softmax")
    assert (T - 1) * stride > 2 ** 31
    ids, w = _run(l, None, cfg)
    dense = l.contiguous()
    ids2, w2 = _run(dense, None, _cfg(dense, 2, "softmax"))
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    _check(dense[-64:], None, _cfg(dense[-64:], 2, "softmax"), "softmax", ids[-64:], w[-64:], "bf16")
    del wide, l
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ gradient
def _grad_check(l, ids, g, cfg, score, counts, balance, z, dtype, grad):
    want = oracle.route_backward(_f64(l), ids.cpu().numpy(), None if g is None else _f64(g), score,
                                 bool(cfg.renormalise), float(cfg.weight_scale),
                                 None if counts is None else counts.cpu().numpy(), balance, z, dtype)
    u = oracle.usable_logits(_f64(l), dtype)
    top = np.max(np.where(u > -np.inf, u, -1e30), axis=1)
    lse = np.where(top > -1e29, np.abs(top) + np.log(l.shape[1]), 0.0)
    mag = abs(cfg.weight_scale) * (np.max(np.abs(_f64(g)), axis=1) if g is not None else 0.0) \
        + abs(balance) * l.shape[1] / l.shape[0] + 2 * abs(z) / l.shape[0] * lse
    tol = HALF_STEP[dtype] * np.abs(want) + 200 * U * np.broadcast_to(mag, (l.shape[0],))[:, None] + 1e-40
    err = np.abs(_f64(grad) - want)
    assert np.all(err <= tol), float(np.max(err / tol))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("E,k,G,Gk,gtop", [s for s in SHAPES if s[0] in (1, 5, 60, 128, 256, 1000)])
@pytest.mark.parametrize("dtype,masks,pad,balance,z,weights", [
    ("f32", 0.0, 0, 0.0, 0.0, True), ("bf16", 0.3, 3, 0.01, 0.001, True), ("f32", 0.2, 4, 0.5, 0.0, True),
    ("bf16", 0.0, 8, 0.0, 0.25, True), ("f32", 0.5, 1, 0.5, 0.25, False)])
def test_route_backward_matches_the_oracle(score, renorm, E, k, G, Gk, gtop, dtype, masks, pad, balance, z, weights):
    l = _logits(41, E, dtype, E + 3 * k, masks, pad)
    cfg = _cfg(l, k, score, G, Gk, gtop, renorm, 2.5)
    ids, _ = _run(l, None, cfg)
    g = torch.randn(41, k, generator=torch.Generator().manual_seed(3)).cuda()
    if weights:
        g[ids < 0] = float("nan")  # an empty slot's gradient is never used
    counts = torch.bincount(ids[ids >= 0].long(), minlength=E).int()
    out = torch.full((41, E + pad), 77.0, dtype=l.dtype, device="cuda")
    grad = out[:, :E]
    moe.moe_route_backward(cfg, l, ids, g if weights else None, counts if balance else None, balance, z, grad)
    torch.cuda.synchronize()
    assert out[:, E:].eq(77.0).all()
    if weights:
        g = torch.nan_to_num(g)
    _grad_check(l, ids, g if weights else None, cfg, score, counts, balance, z, dtype, grad)


def test_route_backward_repeated_and_stray_ids():
    """Ids of the caller's own: a repeated id adds up, one outside [0, E) is an
    empty slot, one on a masked expert has no gradient."""
    l = torch.randn(6, 10, generator=torch.Generator().manual_seed(4))
    l[2, 5] = float("-inf")
    l = l.cuda()
    ids = torch.tensor([[1, 1, 3], [0, 9, 10], [5, 2, 1], [-1, -1, -1], [7, -3, 7], [2 ** 30, 4, 6]],
                       dtype=torch.int32, device="cuda")
    g = torch.randn(6, 3, generator=torch.Generator().manual_seed(5)).cuda()
    for score in ("sigmoid", "softmax"):
        for renorm in (0, 1):
            cfg = _cfg(l, 3, score, renorm=renorm)
            grad = torch.empty_like(l)
            moe.moe_route_backward(cfg, l, ids, g, None, 0.0, 0.0, grad)
            if renorm or score == "sigmoid":
                _grad_check(l, ids, g, cfg, score, None, 0.0, 0.0, "f32", grad)
            assert grad[3].eq(0).all() and grad[2, 5] == 0


def test_route_backward_counts_of_zero_and_empty_terms():
    l = torch.randn(4, 6, device="cuda")
    ids = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    grad = torch.full_like(l, 9.0)
    moe.moe_route_backward(_cfg(l, 2, "softmax"), l, ids, None, torch.zeros(6, dtype=torch.int32, device="cuda"), 1.0,
                           0.0, grad)
    assert grad.eq(0).all()
    grad.fill_(9.0)
    moe.moe_route_backward(_cfg(l, 2, "softmax"), l, None, None, None, 0.0, 0.0, grad)
    assert grad.eq(0).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("z", [0.0, 0.25])
def test_masked_experts_have_no_gradient_whatever_the_incoming_one_is(score, renorm, z):
    """An incoming gradient that is infinite or NaN stays in its row and out of the
    masked columns, and at a slot on a masked expert it is not used at all."""
    inf, nan = float("inf"), float("nan")
    l = torch.randn(6, 40, generator=torch.Generator().manual_seed(12)).cuda()
    l[:, 3], l[:, 20] = -inf, torch.finfo(torch.float32).min
    ids = torch.tensor([[0, 5, 39], [1, 2, 4], [3, 7, 8], [20, 3, 9], [6, 7, 8], [5, 6, 7]], dtype=torch.int32).cuda()
    g = torch.randn(6, 3, generator=torch.Generator().manual_seed(13)).cuda()
    g[1, 1], g[4, 0] = inf, nan                 # on picks that count
    g[2, 0], g[3, 0], g[3, 1] = nan, inf, nan   # on masked experts
    cfg = _cfg(l, 3, score, renorm=renorm)
    grad = torch.full_like(l, 77.0)
    moe.moe_route_backward(cfg, l, ids, g, None, 0.0, z, grad)
    torch.cuda.synchronize()
    assert grad[:, 3].eq(0).all() and grad[:, 20].eq(0).all()
    rows = [0, 2, 3, 5]
    _grad_check(l[rows], ids[rows], torch.nan_to_num(g[rows], posinf=0.0), _cfg(l[rows], 3, score, renorm=renorm), score,
                None, 0.0, z * 4 / 6, "f32", grad[rows])  # the penalty is a mean over 6 rows
    assert not grad[1].isfinite().all() and not grad[4].isfinite().all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("balance,z", [(0.0, 0.0), (0.5, 0.25)])
def test_gradients_of_repeated_and_stray_ids_match_the_oracle(score, renorm, balance, z):
    """Every slot of a repeated id counts with its own gradient, a stray id is an
    empty slot, a masked expert's slot adds nothing, with the penalties or without."""
    l = torch.randn(7, 10, generator=torch.Generator().manual_seed(4))
    l[2, 5] = float("-inf")
    l[6] = float("-inf")
    l = l.cuda()
    ids = torch.tensor([[1, 1, 3], [0, 9, 10], [5, 2, 1], [-1, -1, -1], [7, -3, 7], [2 ** 30, 4, 4], [3, 3, 8]],
                       dtype=torch.int32, device="cuda")
    g = torch.randn(7, 3, generator=torch.Generator().manual_seed(5)).cuda()
    counts = torch.arange(10, dtype=torch.int32, device="cuda")
    cfg = _cfg(l, 3, score, renorm=renorm, scale=2.5)
    grad = torch.full_like(l, 77.0)
    moe.moe_route_backward(cfg, l, ids, g, counts if balance else None, balance, z, grad)
    torch.cuda.synchronize()
    _grad_check(l, ids, g, cfg, score, counts, balance, z, "f32", grad)
    assert grad[6].eq(0).all() and grad[2, 5] == 0


def _far_logits(dtype):
    """Rows whose logits pass the end of fp32's exponential (88.72): every
    quarter from 80 to 110 of either sign beside ordinary logits, beside its half,
    and beside neighbours as far out."""
    v = torch.cat([torch.arange(320, 441) / 4, -torch.arange(320, 441) / 4])
    one = torch.ones_like(v)
    rows = torch.cat([torch.stack([v, 0.25 * one, -1.5 * one, v / 2], 1), torch.stack([-1.5 * one, v, one, 3 * one], 1),
                      torch.stack([v, v - 0.5, v - 1.0, v - 2.0], 1), torch.stack([v - 4.0, 0 * one, v, -v], 1)])
    return rows.to(DT[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_weights_of_logits_past_the_exponential_range(score, renorm, dtype):
    """All four experts are picked, so the order is the logits' own and every
    weight is checked.  Weights below 2^-126 may come out as 0 (the 1e-37)."""
    l = _far_logits(dtype)
    want_ids, want_w, _ = oracle.route_logits(_f64(l), None, 4, score, renormalise=bool(renorm), scale=2.5, dtype=dtype)
    for rows in (l, _repeated(l)):
        ids, w = _run(rows, None, _cfg(rows, 4, score, renorm=renorm, scale=2.5))
        n = l.shape[0]
        assert np.array_equal(ids[:n].cpu().numpy(), want_ids)
        assert np.all(np.abs(_f64(w)[:n] - want_w) <= 80 * U * want_w + 1e-37)
        if rows is not l:
            assert torch.equal(ids[n:2 * n], ids[:n]) and torch.equal(w[n:2 * n], w[:n])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("z", [0.0, 0.25])
def test_gradients_of_logits_past_the_exponential_range(score, renorm, dtype, z):
    l = _far_logits(dtype)
    T = l.shape[0]
    cfg = _cfg(l, 4, score, renorm=renorm, scale=2.5)
    ids, _ = _run(l, None, cfg)
    g = torch.randn(T, 4, generator=torch.Generator().manual_seed(6)).cuda()
    grad = torch.full_like(l, 77.0)
    moe.moe_route_backward(cfg, l, ids, g, None, 0.0, z, grad)
    torch.cuda.synchronize()
    _grad_check(l, ids, g, cfg, score, None, 0.0, z, dtype, grad)


# ------------------------------------------------------------------ combine
def _dispatch(T, E, k, seed, cap=None):
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    counts, offsets, perm, row_of = oracle.dispatch(ids, E, cap)
    return ids, counts, offsets, perm, torch.from_numpy(np.asarray(row_of).reshape(-1).astype(np.int32)).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,E,k,cap", [(1, 8, 4, 1, None), (37, 256, 8, 2, 5), (64, 520, 8, 3, None),
                                         (33, 1000, 16, 16, 20), (19, 4096, 8, 8, None), (300, 2880, 32, 4, 30)])
def test_combine_backward_matches_the_oracle(dtype, T, d, E, k, cap):
    _, _, _, _, row_of = _dispatch(T, E, k, T + d, cap)
    gen = torch.Generator().manual_seed(T)
    gy = torch.randn(T, d, generator=gen).to(DT[dtype]).cuda()
    yp = torch.randn(T * k, d, generator=gen).to(DT[dtype]).cuda()
    w = torch.rand(T, k, generator=gen).cuda()
    cfg = moe.make_config(T, d, E, k, 8, moe.MOE_BF16 if dtype == "bf16" else moe.MOE_F32, moe.MOE_SOFTMAX_TOPK)
    rows = torch.full((T * k, d), 5.5, dtype=DT[dtype], device="cuda")
    gw = torch.full((T, k), float("nan"), device="cuda")
    moe.moe_combine_backward(cfg, gy, yp, row_of, w, rows, gw)
    torch.cuda.synchronize()
    want_rows, want_w = oracle.combine_backward(_f64(gy), _f64(yp), row_of.cpu().numpy(), _f64(w), k)
    used = ~np.isnan(want_rows[:, 0])
    got = _f64(rows)
    assert np.all(got[~used] == 5.5)
    assert np.all(np.abs(got[used] - want_rows[used]) <= (HALF_STEP[dtype] + 2 * U) * np.abs(want_rows[used]) + 1e-40)
    absdot = np.array([[np.abs(_f64(gy[t])) @ np.abs(_f64(yp[max(0, int(row_of[t * k + s]))])) for s in range(k)]
                       for t in range(T)])
    assert np.all(np.abs(_f64(gw) - want_w) <= (d / 32 + 16) * U * absdot)
    # either output alone gives the same
    rows2, gw2 = torch.full_like(rows, 5.5), torch.empty_like(gw)
    moe.moe_combine_backward(cfg, gy, None, row_of, w, rows2, None)
    moe.moe_combine_backward(cfg, gy, yp, row_of, None, None, gw2)
    assert torch.equal(rows, rows2) and torch.equal(gw, gw2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,k", [(40003, 40, 2), (10007, 1032, 3)])
def test_combine_backward_of_more_tokens_than_blocks_and_in_place(dtype, T, d, k):
    """Blocks that take several tokens, against the formula in binary64 on the
    GPU; and the experts' rows replaced by their gradients."""
    _, _, _, _, row_of = _dispatch(T, 8, k, d, T * k // 9)
    gen = torch.Generator(device="cuda").manual_seed(T)
    gy = torch.randn(T, d, generator=gen, device="cuda").to(DT[dtype])
    yp = torch.randn(T * k, d, generator=gen, device="cuda").to(DT[dtype])
    w = torch.rand(T, k, generator=gen, device="cuda")
    cfg = moe.make_config(T, d, 8, k, 8, moe.MOE_BF16 if dtype == "bf16" else moe.MOE_F32, moe.MOE_SOFTMAX_TOPK)
    rows = torch.full((T * k, d), 5.5, dtype=DT[dtype], device="cuda")
    gw = torch.full((T, k), float("nan"), device="cuda")
    moe.moe_combine_backward(cfg, gy, yp, row_of, w, rows, gw)
    slot = torch.nonzero(row_of >= 0)[:, 0]
    row, g = row_of[slot].long(), gy[slot // k].double()
    want = g * w.reshape(-1)[slot, None].double()
    err = (rows[row].double() - want).abs()
    assert (err <= (HALF_STEP[dtype] + 2 * U) * want.abs() + 1e-40).all()
    free = torch.ones(T * k, dtype=torch.bool, device="cuda")
    free[row] = False
    assert free.any() and rows[free].eq(5.5).all()
    y = yp[row].double()
    want_w = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(want_w)
    want_w[slot], bound[slot] = (g * y).sum(1), (g * y).abs().sum(1)
    assert ((gw.reshape(-1).double() - want_w).abs() <= (d / 32 + 16) * U * bound).all()
    gw2 = torch.empty_like(gw)
    yp[free] = 5.5
    moe.moe_combine_backward(cfg, gy, yp, row_of, w, yp, gw2)
    assert torch.equal(yp, rows) and torch.equal(gw2, gw)


def test_combine_backward_refuses_the_incoming_gradient_as_its_output():
    """grad_y is read by tokens whose rows others write; y_perm's rows are each
    read and written by one token."""
    T, d = 37, 64
    row_of = torch.randperm(T, generator=torch.Generator().manual_seed(1)).int().cuda()
    gy, yp, w = torch.randn(T, d, device="cuda"), torch.randn(T, d, device="cuda"), torch.rand(T, 1, device="cuda")
    cfg = moe.make_config(T, d, 4, 1, 8, moe.MOE_F32, moe.MOE_SOFTMAX_TOPK)
    kept = gy.clone()
    with pytest.raises(moe.MoeError) as e:
        moe.moe_combine_backward(cfg, gy, yp, row_of, w, gy, torch.empty_like(w))
    assert e.value.status == 1
    torch.cuda.synchronize()
    assert torch.equal(gy, kept)


@pytest.mark.parametrize("score,renorm", [("sigmoid", 1), ("softmax", 0)])
@pytest.mark.parametrize("E,k,dtype", [(24, 3, "f32"), (300, 5, "bf16")])
def test_route_backward_of_more_rows_than_warps(score, renorm, E, k, dtype):
    """Warps that take several rows: the gradients of the rows alone (whose
    penalties are shares of a batch of their own)."""
    few = _logits(53, E, dtype, E, 0.2, 3)
    l = _repeated(few, 30011)
    g = torch.randn(53, k, generator=torch.Generator().manual_seed(8)).cuda()
    counts = torch.arange(1, E + 1, dtype=torch.int32, device="cuda")
    out = []
    for rows in (few, l):
        T = rows.shape[0]
        cfg = _cfg(rows, k, score, renorm=renorm, scale=1.5)
        ids, _ = _run(rows, None, cfg)
        grad = torch.full((T, E + 3), 77.0, dtype=rows.dtype, device="cuda")
        moe.moe_route_backward(cfg, rows, ids, g.repeat(-(-T // 53), 1)[:T].contiguous(), counts, 0.5 * T / 53,
                               0.25 * T / 53, grad[:, :E])
        assert grad[:, E:].eq(77.0).all()
        out.append(grad)
    # the coefficients, T / 53 times as large over T rows, are the same up to roundings of the division
    a, b = out[0].double(), out[1].double()[:53]
    mag = 1.5 * g.abs().max() + 0.5 * E / 53 + 0.5 / 53 * 10
    assert ((a - b).abs() <= 2 * HALF_STEP[dtype] * a.abs() + 8 * U * mag).all()
    for at in range(53, 30011 - 53, 53 * 47):
        assert torch.equal(out[1][at:at + 53], out[1][:53])


# ------------------------------------------------------------------ together
def test_router_gradient_through_the_layer():
    """route -> dispatch -> experts -> combine and back to the logits: the
    chained gradient equals the oracle's on the rows the GPU computed, and the
    layer's own outputs at logits +- h v differ as the oracle's do.

    L = <grad_y, y>.  y is a k-term fp32 sum per element and w is off by 80 u:
    a difference of two L is off by at most 2 * 90 u sum |grad_y||w y_perm|,
    divided by 2 h."""
    T, E, k, d, f = 48, 16, 4, 64, 96
    gen = torch.Generator().manual_seed(11)
    x = torch.randn(T, d, generator=gen).cuda()
    l = torch.randn(T, E, generator=gen).cuda()
    w_gu = (torch.randn(E, 2 * f, d, generator=gen) / d ** 0.5).cuda()
    w_d = (torch.randn(E, d, f, generator=gen) / f ** 0.5).cuda()
    gy = torch.randn(T, d, generator=gen).cuda()
    bias = (0.1 * torch.randn(E, generator=gen)).cuda()
    v = torch.randn(T, E, generator=gen).cuda()
    route = _cfg(l, k, "sigmoid", 4, 2, 2, 1, 2.0)
    cfg = moe.make_config(T, d, E, k, f, moe.MOE_F32, moe.MOE_SOFTMAX_TOPK)
    ws = torch.zeros(moe.moe_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    ids, w = _run(l, bias, route)
    counts = torch.empty(E, dtype=torch.int32, device="cuda")
    offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    perm = torch.empty(T * k, dtype=torch.int32, device="cuda")
    row_of = torch.empty(T * k, dtype=torch.int32, device="cuda")
    xp, yp = torch.empty(T * k, d, device="cuda"), torch.empty(T * k, d, device="cuda")
    y = torch.empty(T, d, device="cuda")
    moe.moe_permute(cfg, ids, x, counts, offsets, perm, row_of, xp, ws)
    moe.moe_grouped_ffn(cfg, xp, offsets, w_gu, w_d, yp, ws)
    gw, grad = torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda")
    moe.moe_combine_backward(cfg, gy, yp, row_of, w, None, gw)
    moe.moe_route_backward(route, l, ids, gw, counts, 0.01, 0.001, grad)
    assert moe.moe_device_status(ws) == 0
    _, want_gw = oracle.combine_backward(_f64(gy), _f64(yp), row_of.cpu().numpy(), _f64(w), k)
    want = oracle.route_backward(_f64(l), ids.cpu().numpy(), want_gw, "sigmoid", True, 2.0, counts.cpu().numpy(),
                                 0.01, 0.001)
    absw = np.array([[np.abs(_f64(gy[t])) @ np.abs(_f64(yp[int(row_of[t * k + s])])) for s in range(k)]
                     for t in range(T)])
    assert np.max(np.abs(_f64(grad) - want)) <= 200 * U * (2.0 * absw.max() + 1.0)

    h = 2.0 ** -7

    def layer(l2):  # same picks, weights of the shifted logits (k = E of the picked ones only)
        w2 = torch.empty_like(w)
        sub = torch.gather(l2, 1, ids.long()).contiguous()
        ids2 = torch.empty_like(ids)
        moe.moe_route_topk(_cfg(sub, k, "sigmoid", 1, 1, 1, 1, 2.0), sub, None, ids2, w2)
        back = torch.empty_like(w2).scatter_(1, ids2.long(), w2)
        moe.moe_combine(cfg, yp, row_of, back, None, y)
        return float((gy.double() * y.double()).sum())

    got = (layer(l + h * v) - layer(l - h * v)) / (2 * h)

    def obj(l2):
        return oracle.route_objective(l2, ids.cpu().numpy(), want_gw, "sigmoid", True, 2.0)
    lp, lm = _f64(l + h * v), _f64(l - h * v)
    want_diff = (obj(lp) - obj(lm)) / (2 * h)
    bound = 2 * 90 * U * float(np.sum(absw * _f64(w))) / (2 * h)
    assert abs(got - want_diff) <= bound
    # and that difference is the gradient's, up to h^2 times a third derivative of order 1 per logit
    flat = float(np.sum(oracle.route_backward(_f64(l), ids.cpu().numpy(), want_gw, "sigmoid", True, 2.0) * _f64(v)))
    assert abs(want_diff - flat) <= h * h * float(np.sum(absw[:, :, None] * np.abs(_f64(v))[:, None, :] ** 3))


def test_route_on_another_stream_and_in_a_graph():
    T, E, k = 77, 256, 8
    l = _logits(T, E, "f32", 1)
    b = (0.1 * torch.randn(E, generator=torch.Generator().manual_seed(2))).cuda()
    cfg = _cfg(l, k, "sigmoid", 8, 4, 2, 1, 2.5)
    want_ids, want_w = _run(l, b, cfg)
    g = torch.randn(T, k, device="cuda")
    want_grad = torch.empty_like(l)
    counts = torch.ones(E, dtype=torch.int32, device="cuda")
    moe.moe_route_backward(cfg, l, want_ids, g, counts, 0.01, 0.001, want_grad)
    ids, w, grad = torch.empty_like(want_ids), torch.empty_like(want_w), torch.empty_like(l)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    live = l.clone()
    with torch.cuda.graph(graph, stream=side):
        moe.moe_route_topk(cfg, live, b, ids, w)
        moe.moe_route_backward(cfg, live, ids, g, counts, 0.01, 0.001, grad)
    for shift in (0, 1):
        live.copy_(l.roll(shift, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, want_ids.roll(shift, 0)) and torch.equal(w, want_w.roll(shift, 0))
    live.copy_(l)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(grad, want_grad)


def test_route_refuses_host_tensors_and_keeps_outputs():
    l = torch.randn(4, 8)
    ids = torch.full((4, 2), -7, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    with pytest.raises(moe.MoeError) as e:
        moe.moe_route_topk(_cfg(l, 2, "softmax"), l, None, ids, w)
    assert e.value.status == 1
    torch.cuda.synchronize()
    assert ids.eq(-7).all()
