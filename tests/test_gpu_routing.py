"""ep_route, ep_balance_loss and ep_route_backward against their 64-bit forms.

Tolerances count roundings of half a step, u = 2^-24 for fp32: an exponential
of x - m carries |x - m| u from its argument and 2u of its own, a log sigmoid
three times that; sums over up to 1024 experts pass through at most 22
additions (16 in a lane, 6 across lanes), and the balance sums through one per
token more; quotients and products add a handful.  DEPTH covers the constant
part, the spread of the logits enters per case.  bf16 gradients add half a
step, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import combine_ep_layout_09_amd as ep
import workloads
from tests import routing_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
DEPTH = 48


def spread(x):
    f = x[np.isfinite(x)].astype(np.float64)
    return min(float(f.max() - f.min()) + float(np.abs(f).max()), 128.0) if f.size else 0.0


def bound(x):
    return (3 * spread(x) + DEPTH) * U


class Case:
    def __init__(self, T, E, k, G=1, KG=1, score=0, norm=True, bf16=False, bias=False, pad=0.0,
                 B=1, scale=1.0, seed=0, gap=0, offset=0, logits=None):
        r = np.random.default_rng(seed + 1000 * T + E)
        self.rt = ep.Routing(T, E, k, G, KG, ("softmax", "sigmoid")[score], norm, B, scale)
        print(f"[gpu] {self.rt!r} bf16={bf16} bias={bias} pad={pad} gap={gap} offset={offset}",
              flush=True)
        x = torch.from_numpy((2.0 * r.standard_normal((T, E))).astype(np.float32)
                             if logits is None else logits.astype(np.float32))
        x = x.to(torch.bfloat16) if bf16 else x
        self.x = x.float().numpy()
        # rows `gap` elements further apart than E, the first `offset` elements in
        room = torch.full((offset + max(T, 1) * (E + gap),), float("nan"), dtype=x.dtype)
        view = room[offset:offset + T * (E + gap)].view(T, E + gap)[:, :E]
        view.copy_(x)
        self.room = room.to(DEV)
        self.logits = self.room[offset:offset + T * (E + gap)].view(T, E + gap)[:, :E]
        self.bias = (0.5 * r.standard_normal(E)).astype(np.float32) if bias else None
        self.valid = (r.random(T) >= pad).astype(np.uint8) if pad else None
        self.d_bias = None if self.bias is None else torch.from_numpy(self.bias).to(DEV)
        self.d_valid = None if self.valid is None else torch.from_numpy(self.valid).to(DEV)
        self.r, self.T, self.E, self.k, self.G, self.KG = r, T, E, k, G, KG
        self.score, self.norm, self.scale, self.B, self.bf16 = score, norm, scale, B, bf16

    def route(self):
        idx = torch.full((self.T, self.k), -7, dtype=torch.int32, device=DEV)
        w = torch.full((self.T, self.k), float("nan"), device=DEV)
        ep.ep_route(self.rt, self.logits, idx, w, expert_bias=self.d_bias, valid=self.d_valid)
        torch.cuda.synchronize()
        return idx, w

    def check_route(self, idx, w):
        want = ref.choose(self.x, self.k, self.G, self.KG, self.bias, self.valid)
        np.testing.assert_array_equal(idx.cpu().numpy(), want)
        ww = ref.weights(self.x, want, self.score, self.norm, self.scale, self.valid)
        got = w.cpu().numpy().astype(np.float64)
        assert (np.abs(got - ww) <= bound(self.x) * np.abs(ww) + 2.0 ** -126).all(), \
            np.abs(got - ww).max()
        return want

    def balance(self, idx, coef=0.25):
        B, E = self.B, self.E
        o = dict(counts=torch.full((B, E), -7, dtype=torch.int32, device=DEV),
                 mean_prob=torch.full((B, E), float("nan"), device=DEV),
                 num_valid=torch.full((B,), -7, dtype=torch.int32, device=DEV),
                 loss=torch.full((1,), float("nan"), device=DEV))
        n = ep.ep_balance_workspace_bytes(self.rt)
        space = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device=DEV)
        ep.ep_balance_loss(self.rt, self.logits, idx, coef, workspace=space[:n],
                           valid=self.d_valid, **o)
        torch.cuda.synchronize()
        assert (space[n:] == 0xFF).all()
        return o

    def check_balance(self, o, idx, coef=0.25):
        c, mean, n, loss = ref.balance(self.x, idx, self.score, coef, self.B, self.valid)
        np.testing.assert_array_equal(o["counts"].cpu().numpy(), c)
        np.testing.assert_array_equal(o["num_valid"].cpu().numpy(), n)
        tol = bound(self.x) + (self.T // self.B) * U
        got = o["mean_prob"].cpu().numpy()
        assert (np.abs(got - mean) <= tol * mean + 2.0 ** -126).all(), np.abs(got - mean).max()
        assert abs(float(o["loss"]) - loss) <= tol * abs(loss)
        return c, n

    def backward(self, idx, dw=None, coef=0.25, c=None, n=None, dloss=None):
        dx = torch.full((self.T, self.E), float("nan"), dtype=self.logits.dtype, device=DEV)
        to = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
        ep.ep_route_backward(self.rt, self.logits, idx, dx, d_weights=to(dw), coef=coef,
                             counts=to(c), num_valid=to(n),
                             d_loss=None if dloss is None else torch.tensor([dloss], device=DEV),
                             valid=self.d_valid)
        torch.cuda.synchronize()
        want, size = ref.gradient(self.x, idx.cpu().numpy(), self.score, self.norm, self.scale, dw,
                                  coef, c, n, dloss, self.valid)
        got = dx.float().cpu().numpy().astype(np.float64)
        half = 2.0 ** -8 if self.bf16 else U
        tol = (bound(self.x) + 8 * U) * size + half * np.abs(want) + 2.0 ** -126
        assert np.isfinite(got).all()
        assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / (size + 1e-30)).max()
        return dx

    def all(self):
        idx, w = self.route()
        want = self.check_route(idx, w)
        c, n = self.check_balance(self.balance(idx), want)
        dw = self.r.standard_normal((self.T, self.k)).astype(np.float32)
        self.backward(idx, dw=dw)
        self.backward(idx, c=c, n=n, dloss=1.5)
        self.backward(idx, dw=dw, c=c, n=n, dloss=-0.5)


CASES = [
    # T, E, k, G, KG: every lane mapping, powers of two and not
    dict(T=1, E=1, k=1), dict(T=1, E=256, k=8, G=8, KG=4), dict(T=3, E=5, k=5),
    dict(T=17, E=16, k=16), dict(T=33, E=17, k=3), dict(T=64, E=8, k=2), dict(T=65, E=60, k=6, G=6, KG=2),
    dict(T=50, E=64, k=6), dict(T=31, E=96, k=6, G=4, KG=3), dict(T=40, E=128, k=32),
    dict(T=200, E=200, k=9, G=8, KG=5), dict(T=129, E=256, k=32, G=64, KG=33),
    dict(T=20, E=257, k=4), dict(T=19, E=510, k=31, G=10, KG=1), dict(T=9, E=512, k=8, G=2, KG=1),
    dict(T=12, E=777, k=32, G=7, KG=3), dict(T=7, E=1024, k=32, G=64, KG=64),
]


@pytest.mark.parametrize("shape", CASES, ids=lambda s: "-".join(map(str, s.values())))
@pytest.mark.parametrize("score,norm,bf16", [(0, True, False), (0, False, True), (1, True, True),
                                             (1, False, False), (0, False, False)])
def test_shapes(shape, score, norm, bf16):
    Case(score=score, norm=norm, bf16=bf16, bias=score == 1, **shape).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("gap,offset", [(0, 1), (1, 0), (3, 5), (8, 8), (64, 0), (4, 4)])
def test_row_pitches_and_alignments(gap, offset, bf16):
    Case(37, 64, 6, bf16=bf16, gap=gap, offset=offset).all()
    Case(11, 256, 8, G=8, KG=4, bf16=bf16, gap=gap, offset=offset, score=1).all()
    Case(11, 300, 8, bf16=bf16, gap=gap, offset=offset, norm=False).all()


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("norm", [False, True])
def test_padding_sequences_and_scale(score, norm):
    Case(600, 64, 6, score=score, norm=norm, pad=0.4, B=6, scale=2.5).all()
    Case(96, 256, 8, G=8, KG=4, score=score, norm=norm, pad=0.3, B=96, bf16=True).all()
    Case(2048, 40, 4, score=score, norm=norm, pad=0.1, B=2).all()


def test_whole_sequences_without_valid_tokens():
    c = Case(64, 32, 4, B=4, pad=0.5)
    c.valid[:32] = 0
    c.d_valid = torch.from_numpy(c.valid).to(DEV)
    c.all()
    c.valid[:] = 0
    c.d_valid = torch.from_numpy(c.valid).to(DEV)
    c.all()


def _with_off(T, E, seed, values):
    r = np.random.default_rng(seed)
    x = (2 * r.standard_normal((T, E))).astype(np.float32)
    for i, v in enumerate(values):
        x[r.random((T, E)) < 0.15] = v
    x[0] = values[0]        # a row with nothing left
    if T > 2:
        x[1] = values[0]
        x[1, E // 2] = 0.5  # one expert left
        x[2, :E // 2] = values[-1]
    return x


@pytest.mark.parametrize("score,norm", [(0, True), (0, False), (1, True), (1, False)])
@pytest.mark.parametrize("E,G,KG", [(24, 1, 1), (24, 6, 2), (256, 8, 4), (700, 7, 3)])
def test_experts_switched_off(E, G, KG, score, norm):
    x = _with_off(30, E, 5, [-np.inf, np.nan, np.inf])
    Case(30, E, 8, G=G, KG=KG, score=score, norm=norm, logits=x, bias=True).all()
    Case(30, E, 8, G=G, KG=KG, score=score, norm=norm, logits=x, bf16=True, B=3).all()


@pytest.mark.parametrize("score,norm", [(0, True), (0, False), (1, True), (1, False)])
def test_lowest_values_and_wide_ranges(score, norm):
    low = float(np.finfo(np.float32).min)
    x = _with_off(20, 48, 6, [low, -200.0, -low])
    Case(20, 48, 6, score=score, norm=norm, logits=x).all()
    x = np.full((20, 48), low, np.float32)
    Case(20, 48, 6, score=score, norm=norm, logits=x).all()
    x = (-60 + 3 * np.random.default_rng(3).standard_normal((20, 48))).astype(np.float32)
    x[10:] += 100
    Case(20, 48, 6, G=4, KG=2, score=score, norm=norm, logits=x).all()


def test_a_bias_that_overflows_switches_an_expert_off():
    x = np.zeros((4, 16), np.float32)
    x[:, 3] = 3e38
    c = Case(4, 16, 16, logits=x)
    c.bias = np.linspace(0, 1, 16).astype(np.float32)
    c.bias[3] = 3e38
    c.bias[5] = np.nan
    c.d_bias = torch.from_numpy(c.bias).to(DEV)
    idx, w = c.route()
    c.check_route(idx, w)
    assert (idx[:, 14:] == -1).all()


@pytest.mark.parametrize("E,G,KG", [(16, 1, 1), (64, 8, 3), (256, 8, 4), (512, 1, 1)])
def test_ties_go_to_the_lowest_index(E, G, KG):
    r = np.random.default_rng(9)
    x = r.integers(-2, 3, (50, E)).astype(np.float32)
    x[x == 0] *= r.choice([-1.0, 1.0], (x == 0).sum())  # -0 and +0 are equal
    Case(50, E, 8, G=G, KG=KG, logits=x).all()
    Case(50, E, 8, G=G, KG=KG, logits=x, bf16=True, score=1).all()


@pytest.mark.parametrize("E,G,KG", [(8, 1, 1), (40, 5, 2), (100, 1, 1), (256, 2, 1), (256, 32, 9),
                                    (300, 3, 2), (512, 8, 4), (512, 16, 5), (512, 32, 32),
                                    (640, 2, 1), (1000, 1, 1), (1024, 4, 3), (1024, 16, 7),
                                    (1024, 32, 3)])
@pytest.mark.parametrize("bf16", [False, True])
def test_few_distinct_values(E, G, KG, bf16):
    """Lanes with several experts of one key, some of them past the k-th entry, groups
    of equal score, and rows with few experts or none left."""
    r = np.random.default_rng(E + G)
    for k in sorted({1, min(7, KG * (E // G)), min(32, KG * (E // G))}):
        x = r.integers(-2, 3, (60, E)).astype(np.float32)
        x[x == -2] = -np.inf
        x[:12] = np.where(r.random((12, E)) < 0.02, x[:12], np.nan)
        x[12:15] = 1.0
        x[15] = np.nan
        x[16:19] = np.where(r.random((3, E)) < 0.5, 0.0, -0.0)
        c = Case(60, E, k, G=G, KG=KG, score=1, bf16=bf16, pad=0.1, logits=x)
        c.check_route(*c.route())


def test_repeated_and_foreign_ids_in_the_gradient():
    c = Case(40, 64, 6)
    idx = c.r.integers(-2, 70, (40, 6)).astype(np.int32)
    idx[:, 3] = idx[:, 1]
    idx[:10] = 7
    d = torch.from_numpy(idx).to(DEV)
    cnt, n = c.check_balance(c.balance(d), idx)
    for norm in (True, False):
        for score in (0, 1):
            c2 = Case(40, 64, 6, score=score, norm=norm)
            dw = c2.r.standard_normal((40, 6)).astype(np.float32)
            c2.backward(d, dw=dw, c=cnt, n=n, dloss=0.7)
            a = c2.backward(d, dw=dw)
            b = c2.backward(d, dw=dw)
            assert torch.equal(a, b)


def test_nan_gradients_of_absent_entries_stay_out():
    c = Case(16, 32, 4)
    idx, _ = c.route()
    idx[:, 2] = -1
    dw = c.r.standard_normal((16, 4)).astype(np.float32)
    dw[:, 2] = np.nan
    dx = torch.empty((16, 32), device=DEV)
    ep.ep_route_backward(c.rt, c.logits, idx, dx, d_weights=torch.from_numpy(dw).to(DEV))
    dw[:, 2] = 0
    want, size = ref.gradient(c.x, idx.cpu().numpy(), 0, True, 1.0, dw)
    assert (np.abs(dx.cpu().numpy() - want) <= bound(c.x) * size + 1e-30).all()


def test_large_batches():
    Case(16384, 64, 6, bf16=True, B=4).all()
    Case(3001, 256, 8, G=8, KG=4, score=1, bias=True, pad=0.1).all()


def test_loss_joined_by_many_workgroups():
    """More partial sums than one workgroup adds.  One workspace serves problems of
    different sizes in turn, eager and replayed; equal calls give equal bits."""
    c = Case(5000, 256, 8, B=4, pad=0.1)
    small = Case(60, 16, 2, B=3)
    idx, w = c.route()
    want = c.balance(idx)
    c.check_balance(want, idx.cpu().numpy())
    idx_s, _ = small.route()
    want_s = small.balance(idx_s)
    n = ep.ep_balance_workspace_bytes(c.rt)
    space = torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV)
    got = {name: torch.empty_like(v) for name, v in want.items()}
    got_s = {name: torch.empty_like(v) for name, v in want_s.items()}

    def both():
        ep.ep_balance_loss(c.rt, c.logits, idx, 0.25, workspace=space, valid=c.d_valid, **got)
        ep.ep_balance_loss(small.rt, small.logits, idx_s, 0.25, workspace=space, **got_s)

    both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for rep in range(6):
        for t in (*got.values(), *got_s.values()):
            t.zero_()
        if rep % 2:
            both()
        else:
            g.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(got[name], want[name]), (rep, name)
            assert torch.equal(got_s[name], want_s[name]), (rep, name)


def test_no_tokens():
    c = Case(0, 64, 6, B=3)
    idx, w = c.route()
    o = c.balance(idx)
    assert (o["counts"] == 0).all() and (o["mean_prob"] == 0).all()
    assert (o["num_valid"] == 0).all() and float(o["loss"]) == 0.0
    ep.ep_route_backward(c.rt, c.logits, idx, torch.empty((0, 64), device=DEV),
                         d_weights=torch.empty((0, 6), device=DEV))
    torch.cuda.synchronize()


def test_rows_beyond_32_bit_offsets():
    """The last rows of a [40, 1024] view whose rows lie 2^26 + 8 elements
    apart: row 39 starts beyond 2^31 elements."""
    T, E, pitch = 40, 1024, (1 << 26) + 8
    x = (2 * np.random.default_rng(1).standard_normal((T, E))).astype(np.float32)
    room = torch.empty((T - 1) * pitch + E, dtype=torch.bfloat16, device=DEV)
    view = room.as_strided((T, E), (pitch, 1))
    view.copy_(torch.from_numpy(x))
    c = Case(T, E, 8, bf16=True, logits=x)
    c.logits = view
    c.all()


def test_choice_of_the_workloads_router():
    """The group-limited and plain choices of the synthetic workloads."""
    for E, k, G, KG in ((256, 8, 8, 4), (64, 6, 1, 1)):
        lg = np.random.default_rng(2).standard_normal((500, E)).astype(np.float32)
        want = (workloads.group_limited_topk(lg, k, G, KG) if G > 1
                else workloads._topk_desc(lg, k))
        c = Case(500, E, k, G=G, KG=KG, logits=lg)
        idx, _ = c.route()
        np.testing.assert_array_equal(idx.cpu().numpy(), want)


def test_gradient_against_differences():
    """Central differences of the 64-bit loss, step 2^-12: truncation is below
    step^2 / 6 times third derivatives (at most 6 of terms below 8 here)."""
    c = Case(6, 24, 4, score=1, norm=True, B=2)
    idx, _ = c.route()
    ih = idx.cpu().numpy()
    cnt, n = ref.counts(ih, 24, 2)
    dw = c.r.standard_normal((6, 4)).astype(np.float32)
    dx = c.backward(idx, dw=dw, c=cnt, n=n, dloss=1.0).cpu().numpy()

    def goal(x):
        return ((ref.weights(x, ih, 1, True) * dw).sum()
                + ref.balance(x, ih, 1, 0.25, 2)[3])

    h = 2.0 ** -12
    base = c.x.astype(np.float64)
    for t in range(6):
        for e in range(24):
            up, dn = base.copy(), base.copy()
            up[t, e] += h
            dn[t, e] -= h
            assert abs((goal(up) - goal(dn)) / (2 * h) - dx[t, e]) <= 8 * h * h + 1e-6


def test_graph_replays_and_two_streams():
    """One captured step, replayed between eager calls on another stream with
    its own buffers; every replay equals the eager result."""
    c = Case(700, 256, 8, G=8, KG=4, score=1, pad=0.1, B=7)
    e = Case(300, 64, 6, seed=4)
    want_e = e.route()
    T, E, k, B = 700, 256, 8, 7
    dw = torch.randn((T, k), device=DEV)
    dl = torch.ones(1, device=DEV)

    def buffers():
        return dict(idx=torch.empty((T, k), dtype=torch.int32, device=DEV),
                    w=torch.empty((T, k), device=DEV),
                    counts=torch.empty((B, E), dtype=torch.int32, device=DEV),
                    mean_prob=torch.empty((B, E), device=DEV),
                    num_valid=torch.empty(B, dtype=torch.int32, device=DEV),
                    loss=torch.empty(1, device=DEV), dx=torch.empty((T, E), device=DEV),
                    space=torch.empty(ep.ep_balance_workspace_bytes(c.rt), dtype=torch.uint8,
                                      device=DEV))

    def step(b):
        ep.ep_route(c.rt, c.logits, b["idx"], b["w"], valid=c.d_valid)
        ep.ep_balance_loss(c.rt, c.logits, b["idx"], 0.1, b["counts"], b["mean_prob"],
                           b["num_valid"], b["loss"], b["space"], valid=c.d_valid)
        ep.ep_route_backward(c.rt, c.logits, b["idx"], b["dx"], d_weights=dw, coef=0.1,
                             counts=b["counts"], num_valid=b["num_valid"], d_loss=dl,
                             valid=c.d_valid)

    eager, held = buffers(), buffers()
    step(eager)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(held)
    side = torch.cuda.Stream()
    for rep in range(4):
        for n, t in held.items():
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(side):
            idx2 = torch.empty((300, 6), dtype=torch.int32, device=DEV)
            w2 = torch.empty((300, 6), device=DEV)
            ep.ep_route(e.rt, e.logits, idx2, w2)
            step(eager)
        torch.cuda.synchronize()
        assert torch.equal(idx2, want_e[0]) and torch.equal(w2, want_e[1])
        for n in eager:
            if n != "space":
                assert torch.equal(eager[n], held[n]), (rep, n)


def test_prepared_calls():
    c = Case(100, 64, 6, B=2)
    idx, w = c.route()
    i2, w2 = torch.empty_like(idx), torch.empty_like(w)
    ep.prepare_route(c.rt, c.logits, i2, w2)()
    o = c.balance(idx)
    o2 = {n: torch.empty_like(t) for n, t in o.items()}
    space = torch.empty(ep.ep_balance_workspace_bytes(c.rt), dtype=torch.uint8, device=DEV)
    ep.prepare_balance_loss(c.rt, c.logits, idx, 0.25, workspace=space, **o2)()
    dw = torch.randn((100, 6), device=DEV)
    d1, d2 = torch.empty((100, 64), device=DEV), torch.empty((100, 64), device=DEV)
    ep.ep_route_backward(c.rt, c.logits, idx, d1, d_weights=dw)
    ep.prepare_route_backward(c.rt, c.logits, idx, d2, d_weights=dw)()
    torch.cuda.synchronize()
    assert torch.equal(idx, i2) and torch.equal(w, w2) and torch.equal(d1, d2)
    for n in o:
        assert torch.equal(o[n], o2[n])


def test_bool_padding_and_values_of_padded_rows():
    """Padding as torch.bool; what a padded row's logits hold does not matter."""
    c = Case(90, 128, 4, G=4, KG=2, score=1, pad=0.5, B=3)
    idx, w = c.route()
    o = c.balance(idx)
    dw = torch.randn((90, 4), device=DEV)

    def gradient(valid):
        dx = torch.empty((90, 128), device=DEV)
        ep.ep_route_backward(c.rt, c.logits, idx, dx, d_weights=dw, coef=0.1, counts=o["counts"],
                             num_valid=o["num_valid"], d_loss=torch.ones(1, device=DEV),
                             valid=valid)
        return dx

    d = gradient(c.d_valid)
    off = c.d_valid == 0
    c.logits[off] = float("nan")
    c.logits[off, ::3] = float("inf")
    c.d_valid = c.d_valid.bool()
    i2, w2 = c.route()
    o2 = c.balance(idx)
    assert torch.equal(idx, i2) and torch.equal(w, w2) and torch.equal(d, gradient(c.d_valid))
    assert all(torch.equal(o[n], o2[n]) for n in o)
    assert (d[off] == 0).all() and (idx[off] == -1).all() and (w[off] == 0).all()
