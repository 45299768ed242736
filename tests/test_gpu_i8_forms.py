"""ep_expert_i8 in each of its kernels' forms, the few-row kernel and row tiles of 64, 128 and
256 rows.  Which form a size takes is asserted by the launch rule's own arithmetic.

Without the activation outputs are compared bit for bit: the sum of the codes' products is
exact on both sides (in 64-bit floating point it stays below 2^53), then one rounding to
fp32, two fp32 products from the left and one rounding to bf16."""
import numpy as np
import pytest
import torch

import combine_ep_layout_09_amd as ep
import oracle

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SENTINEL = 0x5A5A


def cdiv(a, b):
    return -(-a // b)


def form(prob, mm):
    """Rows of a tile: 16 with the few-row kernel, 64, 128 or 256 with the many-row one."""
    entries, held = prob.num_tokens * prob.num_topk, prob.num_experts * prob.capacity
    filled = min(held, entries) if prob.capacity else entries
    experts = min(prob.num_experts, filled)
    n2 = mm.out_features * (1 + mm.activation)

    def tiles(mc):
        most = experts + filled // mc
        return min(prob.num_experts * cdiv(prob.capacity, mc), most) if prob.capacity else most

    def cost(mc, each):
        n = min(max(experts // 2 + filled // mc, experts), tiles(mc))
        return each * cdiv(n * cdiv(n2, 256), 256)

    if filled // experts <= 12 or tiles(16) * cdiv(n2, 64) <= 512:
        return 16
    costs = {64: cost(64, 10), 128: cost(128, 12), 256: cost(256, 16)}
    return min(costs, key=lambda mc: (costs[mc], mc))


def make_layout(idx, E, cap):
    r = oracle.layout(idx, E, cap)
    return r, ep.Layout(*(torch.from_numpy(np.ascontiguousarray(r[n], np.int32)).to(DEV)
                          for n in ("count", "offset", "slot_of", "src_of_slot", "status")))


def codes(shape, g):
    return torch.randint(-128, 128, shape, generator=g, device=DEV, dtype=torch.int8)


def exact_bits(q, row_scale, w, scale):
    """bf16 outputs of rows q [M, K] with weights w [N, K]."""
    s = q.double() @ w.double().t().contiguous()
    return (s.float() * row_scale[:, None] * scale[None]).bfloat16()


class One:
    """T rows of one expert."""

    def __init__(self, T, K, N, gated=0, want=None, seed=0, full=None):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed + K + N)
        self.T, self.K, self.N = T, K, N
        self.prob, self.mm = ep.Problem(T, 128, 1, 1), ep.ExpertI8(K, N, 1, gated)
        print(f"[gpu] {self.prob!r} {self.mm!r} tile {form(self.prob, self.mm)}", flush=True)
        assert want is None or form(self.prob, self.mm) == want
        n2 = N * (1 + gated)
        if full is None:
            self.q, self.w = codes((T, K), g), codes((1, n2, K), g)
        else:
            self.q = torch.full((T, K), full, dtype=torch.int8, device=DEV)
            self.w = torch.full((1, n2, K), -128, dtype=torch.int8, device=DEV)
        self.rs = 0.5 + torch.rand(T, generator=g, device=DEV)
        # values of a few units, a twentieth of the gates far below zero
        self.scale = (0.5 + torch.rand((1, n2), generator=g, device=DEV)) / (5920 * K ** 0.5)
        if gated:
            self.scale[0, :N:20] *= 60
        _, self.lay = make_layout(np.zeros((T, 1), np.int32), 1, 0)

    def run(self, rows=None):
        q, rs, lay, prob = self.q, self.rs, self.lay, self.prob
        if rows is not None:
            q, rs = q[rows].contiguous(), rs[rows].contiguous()
            prob = ep.Problem(len(rows), 128, 1, 1)
            _, lay = make_layout(np.zeros((len(rows), 1), np.int32), 1, 0)
        room = torch.full((len(q) * self.N + 64,), SENTINEL, dtype=torch.int16, device=DEV)
        out = room[:len(q) * self.N].view(torch.bfloat16).view(len(q), self.N)
        ep.ep_expert_i8(prob, self.mm, q, lay, self.w, self.scale, out, row_scales=rs)
        torch.cuda.synchronize()
        assert (room[len(q) * self.N:] == SENTINEL).all(), "written behind the last row"
        return out


FORMS = [(17, 16), (600, 64), (2000, 128), (6000, 256)]  # tokens and the form, at 4000 weight rows


@pytest.mark.parametrize("K", [784, 896])
@pytest.mark.parametrize("gated", [0, 1])
def test_a_row_has_the_same_bits_in_every_form(K, gated):
    """Beside other rows, in another place and by another kernel."""
    N = 2000 if gated else 4000
    whole = One(6000, K, N, gated, 256)
    outs = whole.run()
    everything = torch.arange(6000, device=DEV)
    for T, want in FORMS:
        prob = ep.Problem(T, 128, 1, 1)
        assert form(prob, whole.mm) == want
        assert torch.equal(whole.run(everything[:T]), outs[:T]), want
        turned = everything[-T:].flip(0)
        assert torch.equal(whole.run(turned), outs[turned]), want
    if not gated:
        assert torch.equal(outs, exact_bits(whole.q, whole.rs, whole.w[0], whole.scale[0]))


# stages of 128 channels: fewer than the ring holds, as many, one more, and a last one of 16
@pytest.mark.parametrize("K", [16, 112, 128, 144, 256, 272, 384, 400, 512, 528, 640, 2064, 7168])
@pytest.mark.parametrize("T,want", FORMS)
def test_sums_to_the_bit(T, want, K):
    T -= 3 * (T > 17)
    c = One(T, K, 3999, want=want)
    assert torch.equal(c.run(), exact_bits(c.q, c.rs, c.w[0], c.scale[0]))


# 65536 channels: the longest rows, and the largest sum, 2^30
LONGEST = [(20, 1300, 16), (600, 1300, 64), (3500, 1300, 128), (9000, 1300, 256)]


@pytest.mark.parametrize("T,N,want", LONGEST)
def test_longest_rows(T, N, want):
    c = One(T, 65536, N, want=want)
    assert torch.equal(c.run(), exact_bits(c.q, c.rs, c.w[0], c.scale[0]))


@pytest.mark.parametrize("full", [-128, 127])
@pytest.mark.parametrize("T,N,want", LONGEST)
def test_largest_sums_in_every_form(T, N, want, full):
    c = One(T, 65536, N, want=want, full=full)
    s = torch.full((T, N), float(full * -128 * 65536), device=DEV)
    assert torch.equal(c.run(), (s * c.rs[:, None] * c.scale).bfloat16())


class Routed:
    """bf16 or int8 rows of several experts, a workspace of its own."""

    def __init__(self, counts, cap, K, N, fmt, gated, want, seed=1):
        E = len(counts)
        idx = np.repeat(np.arange(E, dtype=np.int32), counts)[:, None]
        np.random.default_rng(seed).shuffle(idx)
        self.prob, self.mm = ep.Problem(len(idx), 128, 1, E, cap), ep.ExpertI8(K, N, fmt, gated)
        print(f"[gpu] {self.prob!r} {self.mm!r} tile {form(self.prob, self.mm)}", flush=True)
        assert form(self.prob, self.mm) == want
        self.ref, self.lay = make_layout(idx, E, cap)
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        R = ep.ep_num_recv_rows(self.prob)
        self.R, self.K, self.N, self.fmt, self.g = R, K, N, fmt, g
        self.w = codes((E, N * (1 + gated), K), g)
        self.scale = (0.5 + torch.rand(self.w.shape[:2], generator=g, device=DEV)) / (5920 * K ** 0.5)
        self.rows = torch.empty((R, K), dtype=torch.int8 if fmt else torch.bfloat16, device=DEV)
        self.rs = torch.empty(R, device=DEV) if fmt else None
        self.space = [torch.empty(max(16, ep.ep_expert_i8_workspace_bytes(self.prob, self.mm)),
                                  dtype=torch.uint8, device=DEV) for _ in range(2)]
        self.new_rows()

    def new_rows(self):
        if self.fmt:
            self.rows.copy_(codes(self.rows.shape, self.g))
            self.rs.copy_(0.5 + torch.rand(self.R, generator=self.g, device=DEV))
        else:
            self.rows.copy_(40 * torch.randn(self.rows.shape, generator=self.g, device=DEV))

    def call(self, out, which=0):
        ep.ep_expert_i8(self.prob, self.mm, self.rows, self.lay, self.w, self.scale, out,
                        row_scales=self.rs, workspace=self.space[which])

    def out(self):
        return torch.full((self.R, self.N), 5.0, dtype=torch.bfloat16, device=DEV)


@pytest.mark.parametrize("fmt", [0, 1])
def test_every_form_captured_and_replayed_at_once(fmt):
    """A graph of each form, replayed on streams of their own at the same time, beside eager
    calls with another workspace."""
    cases = [Routed([5, 0, 12, 9, 16, 1, 3, 7], 0, 512, 200, fmt, 1, 16),
             Routed([40, 70, 64, 0, 100, 33, 90, 61], 0, 384, 2050, fmt, 0, 64),
             Routed([100, 128, 130, 90, 70, 110, 60, 117], 320, 400, 4100, fmt, 1, 128),
             Routed([700, 900, 513, 1024, 650, 801, 0, 1000], 0, 272, 2049, fmt, 1, 256)]
    outs = [c.out() for c in cases]
    for c, o in zip(cases, outs):
        c.call(o)
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream() for _ in cases]
    for c, o in zip(cases, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.call(o)
    for turn in range(3):
        want = []
        for c in cases:
            c.new_rows()
            want.append(c.out())
            c.call(want[-1], 1)
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(5)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        again = [c.out() for c in cases]  # eager calls of the same form meanwhile
        for c, o in zip(cases, again):
            c.call(o, 1)
        torch.cuda.synchronize()
        for i, (o, a, w) in enumerate(zip(outs, again, want)):
            assert torch.equal(o, w) and torch.equal(a, w), (turn, i)
            filled = torch.from_numpy(cases[i].ref["src_of_slot"] >= 0).to(DEV)
            assert (o[~filled] == 5).all(), "rows that no entry fills were written"
            assert not (o[filled] == 5).all(1).any()


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("cap,want", [(9, 16), (48, 64), (120, 128), (1000, 256)])
def test_a_capacity_that_drops_rows_in_every_form(cap, want, fmt):
    """Counts above the capacity, by far for some experts, and below it."""
    counts = [cap * 3, cap + 1, cap, cap - 1, 1, 0, cap // 2, cap * 2] * 2
    c = Routed(counts, cap, 400, 4100 if want != 16 else 300, fmt, 0, want)
    out = c.out()
    c.call(out)
    torch.cuda.synchronize()
    for e, n in enumerate(counts):
        a, n = e * cap, min(n, cap)
        q, rs = (c.rows[a:a + n], c.rs[a:a + n]) if fmt else quant(c.rows[a:a + n])
        assert torch.equal(out[a:a + n], exact_bits(q, rs, c.w[e], c.scale[e])), e
        assert (out[a + n:a + cap] == 5).all()


def quant(x):
    """Codes and scales of bf16 rows: quotients in 64 bits, rounded to fp32 once, are
    those of an IEEE fp32 division (53 bits are more than twice 24 and two)."""
    if len(x) == 0:
        return x.to(torch.int8), x.new_empty(0, dtype=torch.float32)
    x = x.double()
    scale = (x.abs().amax(1) / 127).float()
    return (x / scale.double()[:, None]).float().round().to(torch.int8), scale
