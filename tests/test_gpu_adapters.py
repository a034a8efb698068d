"""Low-rank adapters beside the expert projections, and the layer from router
logits with them, on the GPU against the float64 oracle.

Tolerances.  u = 2^-24.  U = A x sums K products in fp32: the tensor cores add
16 at a time and may drop bits below the last (4 u per step of the running
magnitude sum |a||x|), the warps and blocks add at most 40 partial sums more; in
fp32 layers a lane adds K / 32 terms.  U enters the second product as two bf16
values: 2^-17 of it is lost at most.  The second product adds r terms.  The sum
with the base is rounded (u), the activation costs under 20 u of its value, and
the result is rounded once: half a step, 2^-8 in bf16.
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


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _f64(t):
    return t.detach().cpu().double().numpy()


class Case:
    """Rows of a dispatched batch (or of a shared expert), adapters, weights."""

    def __init__(self, T, d, f, E, k, N, r, dtype, act="swiglu", shared=False, cap=None, pattern="random", seed=0):
        rng = np.random.default_rng(seed + T + d)
        gen = torch.Generator().manual_seed(seed + T * 7 + r)
        self.__dict__.update(T=T, d=d, f=f, E=E, k=k, N=N, r=r, dtype=dtype, act=act, shared=shared)
        self.cfg = moe.make_config(T, d, 1 if shared else E, 1 if shared else k, 8 if shared else f,
                                   moe.MOE_BF16 if dtype == "bf16" else moe.MOE_F32, moe.MOE_SOFTMAX_TOPK,
                                   n_shared=int(shared), d_ff_shared=f if shared else 0,
                                   expert_act=moe.MOE_ACT_SWIGLU if act == "swiglu" else moe.MOE_ACT_GELU)
        self.ad = moe.make_adapter_config(N, r, int(shared))
        if pattern == "random":
            ta = rng.integers(-1, N, T)
        elif pattern == "requests":  # runs of tokens
            ta = np.sort(rng.integers(-1, N, T))
        elif pattern == "none":
            ta = np.full(T, -1)
        elif pattern == "one":
            ta = np.full(T, N - 1)
        else:                        # bad ids and any negative value among good ones
            ta = rng.choice([-(2 ** 31), -1, 0, N - 1, N, 2 ** 31 - 1], T)
        self.ta = torch.from_numpy(ta.astype(np.int32)).cuda()
        self.offsets = self.perm = None
        self.rows = T if shared else T * k
        if shared:
            self.live, self.adapter, self.expert = T, ta, np.zeros(T, np.int64)
        else:
            ids = np.argsort(rng.random((T, E)) - (np.arange(E) == 1) * (T > 40), axis=1)[:, :k]  # expert 1 is hot
            counts, offsets, perm, _ = oracle.dispatch(ids, E, cap)
            self.live = int(offsets[-1])
            full = np.full(T * k, 2 ** 30, np.int32)  # behind the last row: never read
            full[:self.live] = np.asarray(perm).reshape(-1)[:self.live]
            self.offsets = torch.from_numpy(np.asarray(offsets).astype(np.int32)).cuda()
            self.perm = torch.from_numpy(full).cuda()
            self.adapter = ta[full[:self.live] // k]
            self.expert = np.repeat(np.arange(E), np.diff(offsets))
        self.gen = gen

    def tensors(self, which):
        K = self.d if which == "gate_up" else self.f
        n = self.d if which == "down" else (2 if self.act == "swiglu" else 1) * self.f
        E = 1 if self.shared else self.E

        def randn(*s, std=1.0):
            return (torch.randn(*s, generator=self.gen) * std).to(DT[self.dtype]).cuda()
        self.x, self.base = randn(self.rows, K), randn(self.rows, n)
        self.a = randn(self.N, E, self.r, K, std=K ** -0.5)
        self.b = randn(self.N, E, n, self.r, std=self.r ** -0.5)
        self.scale = torch.linspace(-2.0, 2.0, self.N + 1)[1:].cuda().contiguous()
        self.x[self.live:] = float("nan")
        self.base[self.live:] = float("nan")
        self.out = torch.full((self.rows, self.f if which == "gate_up" else self.d), 5.5, dtype=DT[self.dtype],
                              device="cuda")
        return self

    def plan(self, stream=None):
        p = torch.full((moe.moe_adapter_plan_bytes(self.cfg, self.ad),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN wherever nothing is written
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())  # the fill above
        moe.moe_adapter_plan(self.cfg, self.ad, self.offsets, self.perm, self.ta, p, stream=stream)
        return p

    def call(self, which, plan, out=None, base=None, stream=None):
        f = moe.moe_adapter_gate_up if which == "gate_up" else moe.moe_adapter_down
        f(self.cfg, self.ad, plan, self.x, self.a, self.b, self.scale, self.base if base is None else base,
          self.out if out is None else out, stream=stream)

    def check(self, which, out=None):
        out = _f64(self.out if out is None else out)
        n = self.live
        assert np.all(out[n:] == 5.5)
        x, base = _f64(self.x)[:n], _f64(self.base)[:n]
        a, b, s = _f64(self.a), _f64(self.b), _f64(self.scale)
        args = (self.adapter[:n], self.expert[:n])
        v = base + oracle.adapter_delta(x, *args, a, b, s)
        K = x.shape[1]
        steps = K / 16 + 40 if self.dtype == "bf16" else K / 32 + 60
        per = (4 if self.dtype == "bf16" else 1) * U
        mag = oracle.adapter_delta(np.abs(x), *args, np.abs(a), np.abs(b), np.abs(s))  # |s||B| |A||x|
        err = mag * (steps * per + self.r * per) + (2.0 ** -17) * self._abs_bu(x, a, b, s) + 2 * U * np.abs(v)
        if which == "down":
            want, tol = v, err + HALF_STEP[self.dtype] * np.abs(v)
        elif self.act == "swiglu":
            f = self.f
            want = oracle.silu(v[:, :f]) * v[:, f:]
            tol = 1.1 * (np.abs(v[:, f:]) + err[:, f:]) * err[:, :f] + np.abs(oracle.silu(v[:, :f])) * err[:, f:]
            tol = tol + (20 * U + HALF_STEP[self.dtype]) * np.abs(want)
        else:
            want = oracle.gelu(v)
            # 1 + erf cancels for negative v: its absolute error (8 u) is multiplied by v / 2
            tol = 1.13 * err + 8 * U * np.abs(v) + (20 * U + HALF_STEP[self.dtype]) * np.abs(want)
        bad = np.abs(out[:n] - want) - tol * (1 + 1e-6) - 1e-37
        assert np.all(bad <= 0), (float(bad.max()), float(np.max(np.abs(out[:n] - want) / tol)))

    def _abs_bu(self, x, a, b, s):
        if self.dtype == "f32":
            return 0.0
        out = np.zeros((x.shape[0], b.shape[2]))
        for i in range(x.shape[0]):
            n, e = int(self.adapter[i]), int(self.expert[i])
            if 0 <= n < self.N:
                out[i] = abs(s[n]) * (np.abs(b[n, e]) @ np.abs(a[n, e] @ x[i]))
        return out


CASES = [
    dict(T=1, d=64, f=64, E=4, k=2, N=3, r=8, dtype="bf16"),
    dict(T=1, d=4096, f=1024, E=8, k=2, N=16, r=16, dtype="bf16", pattern="one"),
    dict(T=5, d=8, f=8, E=3, k=2, N=2, r=8, dtype="bf16"),
    dict(T=37, d=200, f=264, E=8, k=2, N=5, r=24, dtype="bf16"),
    dict(T=64, d=1000, f=520, E=8, k=2, N=64, r=16, dtype="bf16"),
    dict(T=300, d=328, f=104, E=4, k=2, N=2, r=16, dtype="bf16", pattern="requests"),
    dict(T=300, d=328, f=104, E=4, k=2, N=2, r=32, dtype="bf16"),
    dict(T=257, d=136, f=72, E=2, k=2, N=3, r=64, dtype="bf16"),
    dict(T=200, d=72, f=136, E=2, k=1, N=2, r=8, dtype="bf16", act="gelu"),
    dict(T=130, d=264, f=600, E=4, k=3, N=7, r=128, dtype="bf16", act="gelu"),
    dict(T=90, d=72, f=88, E=4, k=2, N=2, r=48, dtype="bf16", cap=20),
    dict(T=513, d=64, f=80, E=1, k=1, N=6, r=16, dtype="bf16", shared=True),
    dict(T=33, d=2056, f=64, E=1, k=1, N=1, r=40, dtype="bf16", shared=True, act="gelu"),
    dict(T=70, d=96, f=64, E=4, k=2, N=3, r=16, dtype="bf16", pattern="none"),
    dict(T=70, d=96, f=64, E=4, k=2, N=3, r=16, dtype="bf16", pattern="stray"),
    dict(T=1, d=64, f=64, E=4, k=2, N=3, r=8, dtype="f32"),
    dict(T=37, d=200, f=264, E=8, k=2, N=5, r=24, dtype="f32"),
    dict(T=150, d=72, f=136, E=2, k=2, N=2, r=128, dtype="f32", act="gelu", cap=100),
    dict(T=260, d=520, f=40, E=1, k=1, N=4, r=16, dtype="f32", shared=True, pattern="requests"),
    dict(T=40, d=96, f=64, E=4, k=2, N=3, r=64, dtype="f32", pattern="stray"),
]


@pytest.mark.parametrize("which", ["gate_up", "down"])
@pytest.mark.parametrize("kw", CASES, ids=lambda kw: "-".join(str(v) for v in kw.values()))
def test_adapters_match_the_oracle(which, kw):
    c = Case(**kw).tensors(which)
    plan = c.plan()
    c.call(which, plan)
    st = moe.moe_device_status(plan)
    stray = bool(np.any(c.adapter[:c.live] >= c.N))
    assert st == (moe.MOE_ERR_BAD_ADAPTER_ID if stray else 0)
    c.check(which)
    # the plan serves again, and the same call gives the same bits
    out = torch.full_like(c.out, 5.5)
    c.call(which, plan, out)
    assert torch.equal(out, c.out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_down_in_place_equals_apart(dtype):
    c = Case(T=80, d=264, f=136, E=4, k=2, N=3, r=16, dtype=dtype, cap=30).tensors("down")
    plan = c.plan()
    c.call("down", plan)
    y = c.base.clone()
    y[c.live:] = 5.5
    c.call("down", plan, out=y, base=y)
    assert torch.equal(y, c.out)
    g = Case(T=80, d=264, f=136, E=4, k=2, N=3, r=16, dtype=dtype, act="gelu").tensors("gate_up")
    plan = g.plan()
    g.call("gate_up", plan)
    h = g.base.clone()
    g.call("gate_up", plan, out=h, base=h)
    assert torch.equal(h, g.out)


def test_row_results_do_not_depend_on_the_other_rows():
    """A request's rows come out bit for bit the same alone and in a batch of
    others whose tiles have the same size."""
    c = Case(T=40, d=256, f=128, E=4, k=2, N=6, r=16, dtype="bf16").tensors("gate_up")
    c.call("gate_up", c.plan())
    only = c.ta.clone()
    keep = int(c.adapter[0]) if c.adapter[0] >= 0 else 0
    only[c.ta != keep] = -1
    mine = torch.from_numpy(np.flatnonzero(c.adapter == keep)).cuda()
    first = c.out.clone()
    c.ta = only
    c.call("gate_up", c.plan())
    assert mine.numel() and torch.equal(c.out[mine], first[mine])


def test_adapters_on_a_side_stream_and_captured():
    c = Case(T=50, d=256, f=128, E=4, k=2, N=6, r=16, dtype="bf16").tensors("gate_up")
    c.call("gate_up", c.plan())
    want = c.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.full_like(want, 5.5)
    plan = c.plan(stream=side)
    side.wait_stream(torch.cuda.current_stream())
    c.call("gate_up", plan, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    out.fill_(5.5)
    live = c.ta.clone()
    with torch.cuda.graph(graph):
        moe.moe_adapter_plan(c.cfg, c.ad, c.offsets, c.perm, live, plan)
        c.call("gate_up", plan, out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    live.fill_(-1)
    graph.replay()
    torch.cuda.synchronize()
    f = c.f
    pre = _f64(c.base)
    h = oracle.silu(pre[:, :f]) * pre[:, f:]
    assert np.all(np.abs(_f64(out) - h) <= (2.0 ** -8 + 40 * U) * np.abs(h) + 1e-37)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("which", ["gate_up", "down"])
def test_what_no_row_uses_is_not_used(which, dtype):
    """NaN in the inputs of rows without an adapter and in the weights and scales
    of adapters that no token has."""
    c = Case(T=300, d=136, f=200, E=4, k=2, N=6, r=24, dtype=dtype).tensors(which)
    c.ta[c.ta == 2] = -1
    c.adapter = np.where(c.adapter == 2, -1, c.adapter)
    c.call(which, c.plan())
    want = c.out.clone()
    c.a[2], c.b[2], c.scale[2] = float("nan"), float("inf"), float("nan")
    c.x[:c.live][torch.from_numpy(c.adapter < 0).cuda()] = float("nan")
    c.out.fill_(5.5)
    c.call(which, c.plan())
    assert (c.adapter < 0).any() and torch.equal(c.out, want)
    assert c.out[:c.live].isfinite().all()


@pytest.mark.parametrize("T", [70, 700])
def test_plan_of_a_perm_that_ends_with_its_rows(T):
    """A capacity leaves fewer rows than slots; perm may hold just those."""
    c = Case(T=T, d=72, f=88, E=4, k=2, N=2, r=16, dtype="bf16", cap=T // 4).tensors("down")
    assert c.live < c.rows
    c.perm = c.perm[:c.live].clone()
    c.call("down", c.plan())
    c.check("down")


def test_captured_plan_of_several_chunks_replays_on_other_adapters():
    """A captured plan of more than one chunk clears its header and its chunks'
    states in every replay."""
    c = Case(T=900, d=136, f=200, E=4, k=2, N=6, r=16, dtype="bf16").tensors("down")
    want = []
    first, second = c.ta.clone(), c.ta.roll(17)
    for ta in (first, second):
        c.ta = ta
        c.out.fill_(5.5)
        c.call("down", c.plan())
        want.append(c.out.clone())
    live, plan = first.clone(), c.plan()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_adapter_plan(c.cfg, c.ad, c.offsets, c.perm, live, plan)
        c.call("down", plan)
    for i in (0, 1, 1, 0):
        live.copy_((first, second)[i])
        c.out.fill_(5.5)
        graph.replay()
        assert moe.moe_device_status(plan) == 0
        assert torch.equal(c.out, want[i])
    live.fill_(c.N)  # every id past the end: reported, and treated as none
    graph.replay()
    assert moe.moe_device_status(plan) == moe.MOE_ERR_BAD_ADAPTER_ID
    assert torch.equal(c.out[:c.live], c.base[:c.live])


@pytest.mark.parametrize("E,N,shared", [(1024, 8191, False), (1, 65536, True)])
def test_the_last_of_the_most_pairs(E, N, shared):
    """The largest numbers of experts and adapters: keys up to 2^31, weights past
    2^31 bytes apart.  Rows of the first and the last pair."""
    T, d, r = 300, 16, 8
    gen = torch.Generator(device="cuda").manual_seed(E)
    cfg = moe.make_config(T, d, E, 1, d, moe.MOE_BF16, moe.MOE_SOFTMAX_TOPK, n_shared=int(shared),
                          d_ff_shared=d if shared else 0)
    ad = moe.make_adapter_config(N, r, int(shared))
    plan = torch.empty(moe.moe_adapter_plan_bytes(cfg, ad), dtype=torch.uint8, device="cuda")
    offsets = perm = None
    expert = torch.zeros(T, dtype=torch.int64, device="cuda")
    if not shared:
        offsets = torch.full((E + 1,), 100, dtype=torch.int32, device="cuda")  # 100 rows of expert 0, 200 of the last
        offsets[0], offsets[E] = 0, T
        perm = torch.arange(T, dtype=torch.int32, device="cuda")
        expert[100:] = E - 1
    ta = torch.where(torch.arange(T, device="cuda") % 3 == 0, 0, N - 1).int()
    a = torch.zeros(N, E, r, d, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(N, E, d, r, dtype=torch.bfloat16, device="cuda")
    for n in (0, N - 1):
        for e in {0, E - 1}:
            a[n, e] = torch.randn(r, d, generator=gen, device="cuda")
            b[n, e] = torch.randn(d, r, generator=gen, device="cuda")
    scale = torch.ones(N, device="cuda")
    h, base = (torch.randn(T, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    y = torch.empty_like(base)
    moe.moe_adapter_plan(cfg, ad, offsets, perm, ta, plan)
    moe.moe_adapter_down(cfg, ad, plan, h, a, b, scale, base, y)
    assert moe.moe_device_status(plan) == 0
    A, B = a[ta.long(), expert].double(), b[ta.long(), expert].double()
    u, mag = torch.einsum("trd,td->tr", A, h.double()), torch.einsum("trd,td->tr", A.abs(), h.abs().double())
    want = base.double() + torch.einsum("tor,tr->to", B, u)
    tol = torch.einsum("tor,tr->to", B.abs(), mag) * (64 * U + 2.0 ** -17) + (2.0 ** -8 + 4 * U) * want.abs()
    assert ((y.double() - want).abs() <= tol).all()
    del a, b, A, B
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_calls_give_equal_results(dtype):
    """More chunks than one of rows, and tiles whose sums several blocks share."""
    c = Case(T=6000, d=64, f=2560, E=4, k=2, N=9, r=8, dtype=dtype).tensors("down")
    outs = []
    for _ in range(12):
        c.out.fill_(5.5)
        c.call("down", c.plan())
        outs.append(c.out.clone())
    assert all(torch.equal(o, outs[0]) for o in outs)
    c.check("down")


def test_calls_in_a_row_and_on_two_streams():
    """Plans, first and second projections one after the other with nothing
    between them, over two batches of different sizes, each on a stream of its
    own at the same time: as the same calls made alone."""
    cases = [Case(T=T, d=256, f=264, E=4, k=2, N=6, r=16, dtype="bf16", seed=T) for T in (40, 700)]
    streams = [torch.cuda.Stream() for _ in cases]
    alone, plans = [], []
    for c in cases:
        c.tensors("gate_up")
        c.down = Case.__new__(Case)
        c.down.__dict__.update(c.__dict__)
        c.down.tensors("down")
        plan = c.plan()
        c.call("gate_up", plan)
        c.down.call("down", plan)
        alone.append((c.out.clone(), c.down.out.clone()))
        plans.append(plan)
    none = [torch.full_like(c.ta, -1) for c in cases]
    got = []
    torch.cuda.synchronize()
    for i in range(20):
        for c, plan, s, other in zip(cases, plans, streams, none):
            with torch.cuda.stream(s):
                c.out.fill_(5.5)
                c.down.out.fill_(5.5)
                # a plan that the next one replaces at once, and a call on it
                moe.moe_adapter_plan(c.cfg, c.ad, c.offsets, c.perm, other, plan)
                c.call("gate_up", plan)
                moe.moe_adapter_plan(c.cfg, c.ad, c.offsets, c.perm, c.ta, plan)
                c.down.call("down", plan)
                c.call("gate_up", plan)
                got.append((c.out.clone(), c.down.out.clone()))
    torch.cuda.synchronize()
    for i, (h, y) in enumerate(got):
        assert torch.equal(h, alone[i % 2][0]) and torch.equal(y, alone[i % 2][1])


def test_shortest_wait_limit_is_right_or_reported_and_the_next_call_runs():
    """With a limit of 1 ns a wait of the expand that its first try does not end
    (a try may last until the data is there) expires: the call is right, or the
    plan's status word says that it is not; it ends either way, and the call
    after it (a new plan, the usual limit) is right."""
    c = Case(T=200, d=1024, f=2048, E=4, k=2, N=3, r=64, dtype="bf16").tensors("gate_up")
    usual = c.cfg.wait_limit_ns
    c.cfg.wait_limit_ns = 1
    plan = c.plan()
    c.call("gate_up", plan)
    st = moe.moe_device_status(plan)
    assert st in (0, moe.MOE_ERR_TIMEOUT)
    if st == 0:
        c.check("gate_up")
    c.cfg.wait_limit_ns = usual
    c.out.fill_(5.5)
    plan = c.plan()
    c.call("gate_up", plan)
    assert moe.moe_device_status(plan) == 0
    c.check("gate_up")


@pytest.mark.parametrize("which,r", [("gate_up", 8), ("gate_up", 128), ("down", 16), ("down", 64)])
def test_expand_waits_that_expire_end_the_call(which, r):
    """The plan is made with the usual limit, then the projection runs with 1 ns
    several times over: a warp of the expand whose lanes do not see a wait expire
    alike still leaves as one, so every call ends, right or with the status word
    set, and the next plan and call are right."""
    c = Case(T=1500, d=328, f=1032, E=4, k=2, N=3, r=r, dtype="bf16").tensors(which)
    usual = c.cfg.wait_limit_ns
    for _ in range(6):
        c.out.fill_(5.5)
        plan = c.plan()
        c.cfg.wait_limit_ns = 1
        c.call(which, plan)
        c.cfg.wait_limit_ns = usual
        st = moe.moe_device_status(plan)
        assert st in (0, moe.MOE_ERR_TIMEOUT)
        if st == 0:
            c.check(which)
    c.out.fill_(5.5)
    plan = c.plan()
    c.call(which, plan)
    assert moe.moe_device_status(plan) == 0
    c.check(which)


@pytest.mark.parametrize("dtype,T", [("bf16", 40), ("bf16", 700), ("f32", 40), ("f32", 700)])
@pytest.mark.parametrize("which", ["gate_up", "down"])
def test_a_plan_that_gave_up_is_not_used(which, dtype, T):
    """A chunk of the plan whose wait expired leaves its tiles unwritten and marks
    the plan in the word behind the tile count (byte 68); here a whole plan is
    marked by hand.  The projections then write nothing, and a new plan serves."""
    c = Case(T=T, d=264, f=136, E=4, k=2, N=3, r=16, dtype=dtype).tensors(which)
    plan = c.plan()
    head = plan[64:72].view(torch.int32)
    assert head[0] > 0 and head[1] == 0
    head[1] = 1
    c.call(which, plan)
    torch.cuda.synchronize()
    assert c.out.eq(5.5).all()
    moe.moe_adapter_plan(c.cfg, c.ad, c.offsets, c.perm, c.ta, plan)
    c.call(which, plan)
    assert moe.moe_device_status(plan) == 0
    c.check(which)


@pytest.mark.parametrize("kw", [
    dict(T=700, d=520, f=328, E=4, k=2, N=3, r=48, dtype="bf16", pattern="requests"),
    dict(T=900, d=1032, f=264, E=2, k=2, N=2, r=64, dtype="bf16", pattern="requests"),
    dict(T=1200, d=264, f=840, E=1, k=1, N=3, r=88, dtype="bf16", shared=True, pattern="requests"),
    dict(T=600, d=648, f=520, E=4, k=2, N=5, r=128, dtype="bf16", act="gelu"),
    dict(T=1100, d=136, f=200, E=2, k=1, N=2, r=128, dtype="f32", pattern="requests"),
], ids=lambda kw: "-".join(str(v) for v in kw.values()))
@pytest.mark.parametrize("which", ["gate_up", "down"])
def test_high_ranks_over_many_tiles(which, kw):
    """Ranks above 32 over batches of several chunks, with full tiles of long runs."""
    c = Case(**kw).tensors(which)
    plan = c.plan()
    c.call(which, plan)
    assert moe.moe_device_status(plan) == 0
    c.check(which)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_plan_waits_that_expire_leave_a_void_plan_or_a_right_one(dtype):
    """47 chunks with a limit of 1 ns: a plan whose chunks gave up says so and is
    not used, any other is right, and the next call (the usual limit) is right."""
    c = Case(T=6000, d=64, f=96, E=4, k=2, N=9, r=8, dtype=dtype).tensors("down")
    plan = c.plan()
    c.call("down", plan)
    want = c.out.clone()
    usual = c.cfg.wait_limit_ns
    for _ in range(40):
        c.out.fill_(5.5)
        c.cfg.wait_limit_ns = 1
        moe.moe_adapter_plan(c.cfg, c.ad, c.offsets, c.perm, c.ta, plan)
        c.cfg.wait_limit_ns = usual
        st = moe.moe_device_status(plan)
        assert st in (0, moe.MOE_ERR_TIMEOUT)
        assert (plan[64:72].view(torch.int32)[1] != 0) == (st != 0)
        c.call("down", plan)
        assert c.out.eq(5.5).all() if st else torch.equal(c.out, want)
    c.out.fill_(5.5)
    plan = c.plan()
    c.call("down", plan)
    assert moe.moe_device_status(plan) == 0
    c.check("down")


def test_plan_of_a_batch_with_long_runs_and_single_rows():
    """Chunks of the plan that end inside runs, tiles that end inside chunks: 700
    rows of one adapter, then every row another, then none."""
    c = Case(T=1100, d=64, f=64, E=1, k=1, N=300, r=8, dtype="bf16", shared=True)
    ta = np.concatenate([np.zeros(700), np.arange(300), np.full(100, -1)]).astype(np.int64)
    c.ta, c.adapter = torch.from_numpy(ta.astype(np.int32)).cuda(), ta
    c.tensors("down")
    plan = c.plan()
    c.call("down", plan)
    assert moe.moe_device_status(plan) == 0
    c.check("down")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("which,act", [("down", "swiglu"), ("gate_up", "swiglu"), ("gate_up", "gelu")])
def test_infinite_inputs_and_products_give_what_the_formula_gives(which, act, dtype):
    """Row by row: an infinite input, products of finite inputs that pass fp32's
    range, sums between bf16's largest value and fp32's, an infinite base, and a
    NaN input; the other rows are as without them."""
    c = Case(T=40, d=64, f=72, E=2, k=1, N=1, r=16, dtype=dtype, act=act, pattern="one").tensors(which)
    c.a.abs_()
    c.b.abs_().clamp_(min=0.01)
    c.a[..., :2] = 1.9921875
    c.x.abs_()
    c.scale.fill_(1.0)
    x, base = c.x, c.base
    clean = c.plan()
    c.call(which, clean)
    usual = c.out.clone()
    top = 3.3895313892515355e38
    x[3, 5] = float("inf")
    x[4, :2] = top                              # U = 1.35e39, infinite in fp32
    base[6] = float("inf")
    x[7, 1] = float("nan")
    x[8] = 0.0
    x[8, 0], x[8, 1] = 2.0 ** 127, 5e35         # U = 3.40e38: more than bf16's largest, less than fp32's
    c.call(which, clean)
    assert c.out[[3, 4, 6]].eq(float("inf")).all()
    assert c.out[7].isnan().all()
    rest = torch.tensor([i for i in range(40) if i not in (3, 4, 6, 7, 8)], device="cuda")
    assert torch.equal(c.out[rest], usual[rest])
    # the sum of row 8: small weights keep its result in range
    c.b.mul_(2.0 ** -100)
    c.call(which, clean)
    e = int(c.expert[8])
    delta = _f64(c.b[0, e]) @ (_f64(c.a[0, e]) @ _f64(x[8]))
    v = _f64(base[8]) + delta
    assert np.all(delta > 1e6) and np.abs(_f64(c.a[0, e]) @ _f64(x[8])).max() > top * (1 + 2.0 ** -9)
    f = c.f
    want = v if which == "down" else v[:f] * v[f:] if act == "swiglu" else v  # silu and gelu are the identity here
    # U: two products, one addition; as two bf16 values; r products; the rounding
    tol = 2 * (4 * U + 2.0 ** -17 + 16 * 4 * U + 20 * U) + HALF_STEP[dtype]
    assert np.all(np.abs(_f64(c.out[8]) - want) <= tol * np.abs(want))


# ------------------------------------------------------------------ the layer
def _layer(T, d, f, E, k, dtype, n_shared=0, act="swiglu", seed=0, e4m3=False, cap=0.0):
    gen = torch.Generator().manual_seed(seed)
    m = 2 if act == "swiglu" else 1

    def randn(*s, std=1.0):
        return (torch.randn(*s, generator=gen) * std).to(DT[dtype]).cuda()
    t = dict(x=randn(T, d), logits=torch.randn(T, E, generator=gen).cuda(),
             w_gu=randn(E, m * f, d, std=d ** -0.5), w_d=randn(E, d, f, std=f ** -0.5),
             s_gu=randn(1, m * f, d, std=d ** -0.5) if n_shared else None,
             s_d=randn(1, d, f, std=f ** -0.5) if n_shared else None)
    cfg = moe.make_config(T, d, E, k, f, moe.MOE_BF16 if dtype == "bf16" else moe.MOE_F32, moe.MOE_SOFTMAX_TOPK,
                          n_shared=n_shared, d_ff_shared=f if n_shared else 0, capacity_factor=cap,
                          expert_act=moe.MOE_ACT_SWIGLU if act == "swiglu" else moe.MOE_ACT_GELU,
                          weight_format=moe.MOE_W_E4M3 if e4m3 else moe.MOE_W_NATIVE)
    route = moe.make_route_config(T, E, k, moe.MOE_SCORE_SIGMOID, 2, 1 if k <= E // 2 else 2, 1, 1, 1.5)
    return cfg, route, t


def _blob(w):
    rows, cols = w.numel() // w.shape[-1], w.shape[-1]
    q = torch.empty(moe.moe_e4m3_weight_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    moe.moe_quantize_e4m3(w, rows, cols, q)
    return q


def _forward(cfg, route, t, ad=None, names=("w_gu", "w_d", "s_gu", "s_d")):
    y = torch.full((cfg.T, cfg.d_model), 5.5, dtype=t["x"].dtype, device="cuda")
    ids = torch.empty(cfg.T, cfg.top_k, dtype=torch.int32, device="cuda")
    w = torch.empty(cfg.T, cfg.top_k, device="cuda")
    counts = torch.empty(cfg.n_experts, dtype=torch.int32, device="cuda")
    ws = torch.full((max(256, moe.moe_forward_routed_workspace_bytes(cfg, ad)),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    moe.moe_forward_routed(cfg, route, ad, t["x"], t["logits"], None, *(t[n] for n in names), y, ids, w, counts, ws)
    return y, ids, w, counts, ws


@pytest.mark.parametrize("T,dtype,n_shared,cap", [(3, "bf16", 0, 0.0), (700, "bf16", 1, 0.0), (40, "f32", 1, 0.0),
                                                  (300, "bf16", 0, 0.5)])
def test_layer_without_adapters_is_the_chain_of_its_stages(T, dtype, n_shared, cap):
    cfg, route, t = _layer(T, 256, 192, 8, 2, dtype, n_shared, cap=cap)
    t["logits"][T // 2] = float("-inf")  # a padding token: only the shared expert sees it
    y, ids, w, counts, ws = _forward(cfg, route, t)
    assert moe.moe_device_status(ws) == 0  # empty slots are no error here
    assert ids[T // 2].eq(-1).all() and w[T // 2].eq(0).all()
    ws2 = torch.zeros(moe.moe_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
    moe.moe_route_topk(route, t["logits"], None, ids2, w2)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    c2, off = torch.empty_like(counts), torch.empty(9, dtype=torch.int32, device="cuda")
    perm = torch.empty(T * 2, dtype=torch.int32, device="cuda")
    row_of = torch.empty(T * 2, dtype=torch.int32, device="cuda")
    xp, yp = (torch.zeros(T * 2, 256, dtype=t["x"].dtype, device="cuda") for _ in range(2))
    moe.moe_permute(cfg, ids2, t["x"], c2, off, perm, row_of, xp, ws2)
    moe.moe_grouped_ffn(cfg, xp, off, t["w_gu"], t["w_d"], yp, ws2)
    ys = None
    if n_shared:
        one = moe.make_config(T, 256, 1, 1, 192, cfg.dtype, moe.MOE_SOFTMAX_TOPK)
        wso = torch.zeros(moe.moe_workspace_bytes(one), dtype=torch.uint8, device="cuda")
        ys = torch.empty(T, 256, dtype=t["x"].dtype, device="cuda")
        moe.moe_grouped_ffn(one, t["x"], torch.tensor([0, T], dtype=torch.int32, device="cuda"), t["s_gu"], t["s_d"],
                            ys, wso)
    want = torch.empty_like(y)
    moe.moe_combine(cfg, yp, row_of, w2, ys, want)
    torch.cuda.synchronize()
    assert torch.equal(counts, c2) and torch.equal(y, want)
    if not n_shared:
        assert y[T // 2].eq(0).all()


@pytest.mark.parametrize("T,E,k", [(2048, 256, 8), (1500, 60, 2), (400, 256, 4), (9000, 16, 2)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_layer_of_many_experts_with_empty_slots(T, E, k, e4m3):
    """Dispatches of several chunks (and of one, for the 400 tokens) with slots
    that no expert is left for: masked tokens, and tokens with fewer experts than
    slots.  Empty slots are no error, and the layer is what its stages make of the
    slots there are."""
    cfg, route, t = _layer(T, 128, 64, E, k, "bf16", e4m3=e4m3)
    g = torch.Generator().manual_seed(T)
    t["logits"][(torch.rand(T, generator=g) < 0.2).cuda()] = float("-inf")
    t["logits"][:, :E - 1] = t["logits"][:, :E - 1].masked_fill(
        (torch.rand(T, 1, generator=g) < 0.1).cuda(), torch.finfo(torch.float32).min)  # one expert left
    if e4m3:
        t["w_gu_q"], t["w_d_q"], t["s_gu_q"], t["s_d_q"] = _blob(t["w_gu"]), _blob(t["w_d"]), None, None
    names = ("w_gu_q", "w_d_q", "s_gu_q", "s_d_q") if e4m3 else ("w_gu", "w_d", "s_gu", "s_d")
    y, ids, w, counts, ws = _forward(cfg, route, t, None, names)
    assert moe.moe_device_status(ws) == 0
    empty = ids.eq(-1)
    assert empty.any() and (empty.sum(1) == k - 1).any() and w[empty].eq(0).all()
    used = ids[~empty].long()
    assert torch.equal(counts.long(), torch.bincount(used, minlength=E))
    # the stages, every empty slot sent to expert 0 with weight 0
    ids2 = torch.where(empty, torch.zeros_like(ids), ids)
    ws2 = torch.zeros(moe.moe_workspace_bytes(cfg), dtype=torch.uint8, device="cuda")
    c2, off = torch.empty_like(counts), torch.empty(E + 1, dtype=torch.int32, device="cuda")
    perm, row_of = (torch.empty(T * k, dtype=torch.int32, device="cuda") for _ in range(2))
    xp, yp = (torch.zeros(T * k, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_permute(cfg, ids2, t["x"], c2, off, perm, row_of, xp, ws2)
    moe.moe_grouped_ffn(cfg, xp, off, t[names[0]], t[names[1]], yp, ws2)
    want = torch.empty_like(y)
    moe.moe_combine(cfg, yp, row_of, w, None, want)
    assert moe.moe_device_status(ws2) == 0
    assert y[empty.all(1)].eq(0).all()
    # the same rows in other tiles: sums over k terms of products accumulated in another order, h and y_perm
    # rounded to bf16 (the layer's tolerance)
    assert float((y.float() - want.float()).abs().max()) <= 2e-2 * float(want.float().abs().max())


def _adapters(cfg, N, r, dtype, gen, shared, act="swiglu", std=0.5):
    m = 2 if act == "swiglu" else 1
    E, d, f = cfg.n_experts, cfg.d_model, cfg.d_ff

    def randn(*s, std=1.0):
        return (torch.randn(*s, generator=gen) * std).to(DT[dtype]).cuda()

    def four(E):
        return [randn(N, E, r, d, std=d ** -0.5), randn(N, E, m * f, r, std=std * r ** -0.5),
                randn(N, E, r, f, std=f ** -0.5), randn(N, E, d, r, std=std * r ** -0.5)]
    return four(E), four(1) if shared else [None] * 4


@pytest.mark.parametrize("T,dtype,n_shared,act,e4m3", [
    (1, "bf16", 1, "swiglu", False), (33, "bf16", 1, "swiglu", False), (700, "bf16", 1, "swiglu", False),
    (33, "bf16", 0, "gelu", False), (700, "bf16", 0, "gelu", False), (50, "f32", 1, "swiglu", False),
    (50, "f32", 0, "gelu", False), (33, "bf16", 1, "swiglu", True), (700, "bf16", 1, "swiglu", True)])
@pytest.mark.parametrize("parts", ["both", "gate_up", "down"])
def test_layer_with_adapters_matches_experts_with_merged_weights(T, dtype, n_shared, act, e4m3, parts):
    """Every token's experts with its adapter's product added to the weights, in
    float64.  Tolerances of the layer's other parity tests, relative to the
    largest output: 1e-4 in fp32, 2e-2 in bf16 (h, the pre-activations and the
    experts' outputs are rounded to bf16).  8-bit experts are compared with the
    8-bit scheme's values of the base weights and inputs, to 4e-2: the stored
    pre-activations move h by up to 2^-8, so about 2^-5 of its codes come out
    one step (2^-3.5 of the value) apart, 1.6% of an output's rms, whose
    largest of 1700 is 3.5 times that against a largest output of 3.5 rms."""
    E, k, d, f, N, r = 4, 2, 128, 96, 3, 16
    cfg, route, t = _layer(T, d, f, E, k, dtype, n_shared, act, seed=T, e4m3=e4m3)
    gen = torch.Generator().manual_seed(99)
    routed, shared = _adapters(cfg, N, r, dtype, gen, n_shared, act)
    if parts == "gate_up":
        routed[2:], shared[2:] = [None, None], [None, None]
    if parts == "down":
        routed[:2], shared[:2] = [None, None], [None, None]
    ta = ((torch.arange(T) + 1) % (N + 1) - 1).int().cuda()
    scale = torch.tensor([0.5, -1.0, 2.0], device="cuda")
    ad = moe.make_adapters(N, r, ta, scale, *routed, *shared)
    if e4m3:
        for n in ("w_gu", "w_d", "s_gu", "s_d"):
            t[n + "_q"] = _blob(t[n])
        y, ids, w, counts, ws = _forward(cfg, route, t, ad, ("w_gu_q", "w_d_q", "s_gu_q", "s_d_q"))
    else:
        y, ids, w, counts, ws = _forward(cfg, route, t, ad)
    assert moe.moe_device_status(ws) == 0
    x, sc, idn, wn = _f64(t["x"]), _f64(scale), ids.cpu().numpy(), _f64(w)

    def q(v):  # rows through the 8-bit codes
        if not e4m3:
            return v
        codes, s = oracle.quantize_rows_e4m3(v)
        return np.asarray(codes, np.float64) * np.asarray(s, np.float64).reshape(-1, 1)

    def expert(xt, gu, dn, n, e, four):
        gu, dn = q(_f64(gu)), q(_f64(dn))
        delta1 = delta2 = 0.0
        if n >= 0 and four[0] is not None:
            delta1 = sc[n] * _f64(four[1][n, e]) @ (_f64(four[0][n, e]) @ xt)
        v = gu @ q(xt[None])[0] + delta1
        h = oracle.silu(v[:f]) * v[f:] if act == "swiglu" else oracle.gelu(v)
        if n >= 0 and four[2] is not None:
            delta2 = sc[n] * _f64(four[3][n, e]) @ (_f64(four[2][n, e]) @ h)
        return dn @ (q(oracle.round_bf16(h)[None])[0] if e4m3 else h) + delta2

    tokens = sorted(set(range(min(T, 12))) | {T - 1, T // 2})
    want = np.zeros((len(tokens), d))
    for i, tok in enumerate(tokens):
        n = int(ta[tok])
        for s in range(k):
            e = int(idn[tok, s])
            want[i] += wn[tok, s] * expert(x[tok], t["w_gu"][e], t["w_d"][e], n, e, routed)
        if n_shared:
            want[i] += expert(x[tok], t["s_gu"][0], t["s_d"][0], n, 0, shared)
    got = _f64(y)[tokens]
    tol = 4e-2 if e4m3 else {"f32": 1e-4, "bf16": 2e-2}[dtype]
    assert np.max(np.abs(got - want)) <= tol * np.max(np.abs(want))


def test_layer_flags_bad_adapter_ids_and_replays():
    cfg, route, t = _layer(60, 128, 96, 4, 2, "bf16", 1)
    gen = torch.Generator().manual_seed(5)
    routed, shared = _adapters(cfg, 3, 16, "bf16", gen, True)
    ta = (torch.arange(60) % 3).int().cuda()
    scale = torch.ones(3, device="cuda")
    ad = moe.make_adapters(3, 16, ta, scale, *routed, *shared)
    y, ids, w, counts, ws = _forward(cfg, route, t, ad)
    assert moe.moe_device_status(ws) == 0
    y2 = torch.zeros_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_forward_routed(cfg, route, ad, t["x"], t["logits"], None, t["w_gu"], t["w_d"], t["s_gu"], t["s_d"],
                               y2, None, None, None, ws)
    graph.replay()
    assert moe.moe_device_status(ws) == 0 and torch.equal(y, y2)
    ta[7] = 3
    graph.replay()
    assert moe.moe_device_status(ws) == moe.MOE_ERR_BAD_ADAPTER_ID
    rest = torch.arange(60) != 7
    assert torch.equal(y[rest.cuda()], y2[rest.cuda()])
    ta[7] = -1
    graph.replay()
    assert moe.moe_device_status(ws) == 0


@pytest.mark.parametrize("T,dtype,cap,n_shared", [(300, "bf16", 0.75, 1), (700, "f32", 0.5, 1), (1100, "bf16", 1.0, 0)])
def test_layer_with_adapters_a_capacity_and_empty_slots(T, dtype, cap, n_shared):
    """Everything that leaves a slot out at once: masked tokens, tokens with one
    expert left, experts over their capacity, tokens without an adapter; the
    reference walks the slots in token order, in binary64.  Tolerances of the test
    above."""
    E, k, d, f, N, r = 4, 2, 128, 96, 3, 16
    cfg, route, t = _layer(T, d, f, E, k, dtype, n_shared, seed=T, cap=cap)
    gen = torch.Generator().manual_seed(T)
    t["logits"][:, 1] += 1.0  # a hot expert
    t["logits"][(torch.rand(T, generator=gen) < 0.1).cuda()] = float("-inf")
    t["logits"][:, 1:] = t["logits"][:, 1:].masked_fill((torch.rand(T, 1, generator=gen) < 0.1).cuda(), float("nan"))
    routed, shared = _adapters(cfg, N, r, dtype, gen, n_shared)
    ta = torch.randint(-1, N, (T,), generator=gen).int().cuda()
    scale = torch.tensor([0.5, -1.0, 2.0], device="cuda")
    y, ids, w, counts, ws = _forward(cfg, route, t, moe.make_adapters(N, r, ta, scale, *routed, *shared))
    assert moe.moe_device_status(ws) == 0
    C = moe.lib().moe_expert_capacity(cfg)
    x, sc, idn, wn, tan = _f64(t["x"]), _f64(scale), ids.cpu().numpy(), _f64(w), ta.cpu().numpy()

    def host(ts):
        return [None if v is None else _f64(v) for v in ts]
    r_w, s_w, (gu, dn, sgu, sdn) = host(routed), host(shared), host(t[n] for n in ("w_gu", "w_d", "s_gu", "s_d"))

    def expert(xt, gu, dn, n, e, four):
        v = gu @ xt
        if n >= 0:
            v = v + sc[n] * four[1][n, e] @ (four[0][n, e] @ xt)
        h = oracle.silu(v[:f]) * v[f:]
        o = dn @ h
        return o + sc[n] * four[3][n, e] @ (four[2][n, e] @ h) if n >= 0 else o

    want, seen, dropped = np.zeros((T, d)), np.zeros(E, np.int64), 0
    for tok in range(T):
        for s in range(k):
            e = int(idn[tok, s])
            if e < 0:
                continue
            seen[e] += 1
            if seen[e] > C:
                dropped += 1
                continue
            want[tok] += wn[tok, s] * expert(x[tok], gu[e], dn[e], tan[tok], e, r_w)
        if n_shared:
            want[tok] += expert(x[tok], sgu[0], sdn[0], tan[tok], 0, s_w)
    assert dropped > 0 and (idn < 0).any() and np.array_equal(counts.cpu().numpy(), seen)
    assert np.max(np.abs(_f64(y) - want)) <= {"f32": 1e-4, "bf16": 2e-2}[dtype] * np.max(np.abs(want))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T,d,f,E,k,act", [
    (2048, 2880, 2880, 16, 4, "swiglu"), (20, 4096, 3584, 8, 2, "swiglu"), (600, 1024, 1040, 4, 2, "gelu"),
    (1, 2048, 1408, 16, 4, "swiglu"), (3000, 512, 5776, 2, 1, "swiglu")])
def test_layer_of_real_widths_with_adapters_that_add_nothing(T, d, f, E, k, act, e4m3):
    """First products without their activation, at widths of many column tiles,
    under the batch and the decode GEMMs: with adapters of weight zero (B = 0) the
    layer is the one without adapters, but for the pre-activations' rounding to
    bf16 (and, with 8-bit experts, the codes of h that it moves).  Tolerances of
    the tests above; a misplaced column would be off by the outputs' own size."""
    N, r = 2, 16
    m = 2 if act == "swiglu" else 1
    gen = torch.Generator(device="cuda").manual_seed(T)

    def randn(*s, std=1.0):
        return torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=gen)
    t = dict(x=randn(T, d), logits=torch.randn(T, E, generator=gen, device="cuda"), w_gu=randn(E, m * f, d, std=d ** -0.5),
             w_d=randn(E, d, f, std=f ** -0.5), s_gu=None, s_d=None)
    cfg = moe.make_config(T, d, E, k, f, moe.MOE_BF16, moe.MOE_SOFTMAX_TOPK,
                          expert_act=moe.MOE_ACT_SWIGLU if act == "swiglu" else moe.MOE_ACT_GELU,
                          weight_format=moe.MOE_W_E4M3 if e4m3 else moe.MOE_W_NATIVE)
    route = moe.make_route_config(T, E, k, moe.MOE_SCORE_SOFTMAX)
    if e4m3:
        t["w_gu"], t["w_d"] = _blob(t["w_gu"]), _blob(t["w_d"])
    a1, b1 = randn(N, E, r, d), torch.zeros(N, E, m * f, r, dtype=torch.bfloat16, device="cuda")
    a2, b2 = randn(N, E, r, f), torch.zeros(N, E, d, r, dtype=torch.bfloat16, device="cuda")
    ta = (torch.arange(T, device="cuda") % 3 - 1).int()
    scale = torch.ones(N, device="cuda")
    want, ids, _, _, ws = _forward(cfg, route, t)
    assert moe.moe_device_status(ws) == 0
    for parts in ((a1, b1, a2, b2), (a1, b1, None, None), (None, None, a2, b2)):
        y, ids2, _, _, ws = _forward(cfg, route, t, moe.make_adapters(N, r, ta, scale, *parts))
        assert moe.moe_device_status(ws) == 0
        assert torch.equal(ids, ids2)
        if parts[0] is None:
            assert torch.equal(y, want)
        tol = 4e-2 if e4m3 else 2e-2
        assert float((y.float() - want.float()).abs().max()) <= tol * float(want.float().abs().max())
