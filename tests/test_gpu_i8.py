"""ep_dispatch_i8 to the bit, and ep_expert_i8 against the exact sums.

Tolerance of an output: the integer sum is exact; its conversion to fp32 and the two
factors round three times, then the result is rounded to bf16 (block_reference)."""
import numpy as np
import pytest
import torch

import combine_ep_layout_09_amd as ep
import oracle
from tests import block_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SENTINEL = 0x5A5A


def f64(t):
    return t.double().cpu().numpy()


def make_layout(idx, E, cap):
    r = oracle.layout(idx, E, cap)
    return r, ep.Layout(*(torch.from_numpy(np.ascontiguousarray(r[n], np.int32)).to(DEV)
                          for n in ("count", "offset", "slot_of", "src_of_slot", "status")))


def uniform(T, E, k, seed=0):
    r = np.random.default_rng(seed)
    return np.argsort(r.random((T, E)), 1)[:, :k].astype(np.int32)


# -------------------------------------------------------------------- dispatch

def rows_for_codes(T, H, seed):
    """bf16 rows with values next to the middles between codes, tiny and huge rows,
    zeros."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((T, H)) * np.exp2(r.integers(-6, 7, (T, 1)).astype(float))
    mid = (r.integers(-127, 127, (T, H)) + 0.5) / 127
    top = np.exp2(np.ceil(np.log2(np.abs(x).max(1, keepdims=True))))
    x = np.where(r.random((T, H)) < 0.4, mid * top, x)
    x[:, r.integers(0, H)] = top[:, 0]
    if T > 4:
        x[1] = 0
        x[2] *= 2.0 ** -126
        x[3] *= 2.0 ** 118
        x[4] = 2.0 ** -133 * r.integers(-3, 4, H)
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def check_dispatch(idx, E, cap, H, x=None):
    T, k = idx.shape
    prob = ep.Problem(T, H, k, E, cap)
    print(f"[gpu] dispatch_i8 {prob!r}", flush=True)
    r, lay = make_layout(idx, E, cap)
    R = ep.ep_num_recv_rows(prob)
    x = rows_for_codes(T, H, 7 * T + H) if x is None else x
    room = torch.full((R * H + 64,), 0x5A, dtype=torch.int8, device=DEV)
    scales = torch.full((R + 16,), 77.0, device=DEV)
    ep.ep_dispatch_i8(prob, x.to(DEV), lay, room[:R * H].view(R, H), scales[:R])
    torch.cuda.synchronize()
    q, s = ref.quant(x.float().numpy())
    want = np.full((R, H), 0x5A, np.int8)
    want_s = np.full(R, 77.0, np.float32)
    src = r["src_of_slot"]
    want[src >= 0], want_s[src >= 0] = q[src[src >= 0] // k], s[src[src >= 0] // k]
    got = room[:R * H].view(R, H).cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]
    assert np.array_equal(scales[:R].cpu().numpy(), want_s)
    assert (room[R * H:] == 0x5A).all() and (scales[R:] == 77.0).all()


@pytest.mark.parametrize("shape", [
    (1, 4, 2, 0, 8), (1, 256, 8, 0, 7168), (9, 8, 2, 0, 24), (64, 8, 2, 0, 256), (33, 16, 5, 4, 520),
    (128, 256, 8, 128, 1032), (20, 64, 7, 2, 512), (7, 3, 2, 0, 65536), (6, 8, 1, 0, 16392),
    (1500, 16, 4, 0, 1024), (1100, 16, 3, 150, 2056), (1030, 8, 2, 0, 4104), (1025, 4, 1, 0, 17000),
], ids=lambda s: "-".join(map(str, s)))
def test_dispatch(shape):
    T, E, k, cap, H = shape
    check_dispatch(uniform(T, E, k), E, cap, H)


def test_dispatch_of_unrouted_tokens():
    idx = uniform(60, 8, 3)
    idx[5] = -1
    idx[40:, 1] = 8
    check_dispatch(idx, 8, 0, 136)
    check_dispatch(np.full((6, 2), -1, np.int32), 4, 3, 64)


def test_every_quotient_of_a_scale():
    """All bf16 magnitudes up to the row's largest, for scales of every mantissa
    that bf16 rows can have, positive and negative."""
    H = 2 * 128 * 13
    rows = []
    for top in range(128):
        amax = (1 + top / 128) * 2.0 ** 3
        steps = np.exp2(np.arange(-9, 4)[:, None]) * (1 + np.arange(128) / 128)[None]
        v = steps.reshape(-1)
        v = np.where(v <= amax, v, amax)
        rows.append(np.concatenate([v, -v]))
    x = torch.from_numpy(np.array(rows, np.float32)).to(torch.bfloat16)
    assert x.shape == (128, H)
    check_dispatch(np.zeros((128, 1), np.int32), 1, 0, H, x)


# -------------------------------------------------------------------- products

class Case:
    def __init__(self, idx, E, cap, K, N, fmt, gated, seed=0, extreme=False):
        T, k = idx.shape
        r = np.random.default_rng(seed + K + 7 * N)
        self.E, self.cap, self.K, self.N, self.fmt, self.gated = E, cap, K, N, fmt, gated
        self.ref, self.lay = make_layout(idx, E, cap)
        self.prob = ep.Problem(T, 128, k, E, cap)
        self.mm = ep.ExpertI8(K, N, fmt, gated)
        R = self.R = ep.ep_num_recv_rows(self.prob)
        n2 = N * (2 if gated else 1)
        print(f"[gpu] {self.prob!r} {self.mm!r}", flush=True)
        used = self.ref["src_of_slot"] >= 0
        if extreme:
            self.w = np.full((E, n2, K), -128, np.int8)
            self.q = np.full((R, K), -128, np.int8)
        else:
            self.w = r.integers(-128, 128, (E, n2, K), dtype=np.int8)
            self.q = r.integers(-128, 128, (R, K), dtype=np.int8)
        # values of a few units at most, so that the gate's exponential is in range
        self.scale = ((0.5 + r.random((E, n2))) / (80 * 74 * np.sqrt(K))).astype(np.float32)
        self.rs = (0.5 + r.random(R)).astype(np.float32)
        if fmt == 0:
            x = torch.from_numpy(r.standard_normal((R, K)).astype(np.float32) * 40).to(torch.bfloat16)
            x[torch.from_numpy(~used)] = float("nan")
            self.q, self.rs = ref.quant(np.nan_to_num(x.float().numpy()))
            self.rows, self.row_scales = x.to(DEV), None
        else:
            self.rs[~used] = np.nan
            self.rows, self.row_scales = (torch.from_numpy(v).to(DEV) for v in (self.q, self.rs))
        # channels of experts that no entry names have NaN scales
        self.scale[self.ref["count"] == 0] = np.nan
        self.d_w, self.d_scale = torch.from_numpy(self.w).to(DEV), torch.from_numpy(self.scale).to(DEV)
        n = ep.ep_expert_i8_workspace_bytes(self.prob, self.mm)
        self.space = torch.full((n + 64,), 0xEE, dtype=torch.uint8, device=DEV)

    def call(self, out, stream=None):
        ep.ep_expert_i8(self.prob, self.mm, self.rows, self.lay, self.d_w, self.d_scale, out,
                        row_scales=self.row_scales, workspace=self.space[:-64], stream=stream)

    def run(self):
        room = torch.full((self.R * self.N + 64,), SENTINEL, dtype=torch.int16, device=DEV)
        out = room[:self.R * self.N].view(torch.bfloat16).view(self.R, self.N)
        self.call(out)
        torch.cuda.synchronize()
        assert (room[self.R * self.N:] == SENTINEL).all(), "written behind the last row"
        assert (self.space[-64:] == 0xEE).all(), "written behind the workspace"
        return out

    def check(self, out=None):
        out = self.run() if out is None else out
        bits, got = out.view(torch.int16).cpu().numpy(), f64(out)
        filled = np.zeros(self.R, bool)
        for e in range(self.E):
            a = e * self.cap if self.cap else int(self.ref["offset"][e])
            n = int(self.ref["count"][e])
            b = a + (min(n, self.cap) if self.cap else n)
            if a == b:
                continue
            filled[a:b] = True
            y, tol = ref.i8_products(self.q[a:b], self.rs[a:b], self.w[e], self.scale[e], self.gated)
            bad = ~(np.abs(got[a:b] - y) <= tol)
            assert not bad.any(), (e, np.argwhere(bad)[:5], np.abs(got[a:b] - y).max())
        assert (bits[~filled] == SENTINEL).all(), "rows that no entry fills were written"
        return out


SHAPES = [
    # T, E, k, cap, K, N
    (1, 8, 2, 0, 16, 1), (1, 256, 8, 0, 256, 40), (2, 4, 4, 0, 48, 33), (5, 3, 1, 0, 144, 64),
    (16, 8, 2, 0, 128, 65), (64, 8, 2, 0, 256, 100), (33, 5, 3, 0, 528, 31),
    (128, 16, 4, 40, 512, 96), (128, 16, 4, 3, 512, 48), (7, 1024, 4, 2, 64, 16),
    (130, 2, 2, 0, 640, 70), (100, 1, 1, 0, 384, 17), (300, 4, 2, 200, 1024, 128),
    (40, 8, 8, 40, 2064, 20), (3, 300, 3, 1, 256, 130), (700, 3, 2, 0, 208, 260),
    (1500, 4, 2, 0, 464, 300), (900, 2, 1, 500, 1040, 515),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fmt", [0, 1])
def test_shapes(shape, fmt, gated):
    T, E, k, cap, K, N = shape
    Case(uniform(T, E, k, seed=T + K), E, cap, K, N, fmt, gated).check()


@pytest.mark.parametrize("gated", [False, True])
def test_skewed_and_empty_experts(gated):
    """Every filling of a row tile: experts of 0, 1, 2, ... rows."""
    E = 40
    idx = np.concatenate([np.full(e, e, np.int32) for e in range(E)] +
                         [np.full(n, 3, np.int32) for n in (200,)])[:, None]
    np.random.default_rng(0).shuffle(idx)
    Case(idx, E, 0, 272, 130, 1, gated).check()
    Case(idx, E, 64, 272, 130, 0, gated).check()


def filled(counts):
    """One entry per token; experts with these numbers of rows, in any order."""
    idx = np.repeat(np.arange(len(counts), dtype=np.int32), counts)[:, None]
    np.random.default_rng(len(idx)).shuffle(idx)
    return idx


# rows of the experts: for row tiles of 256, of 128 and of 64 rows
MANY = {
    "256": [300, 1, 512, 0, 257, 700, 31, 240, 255, 129, 65, 900, 400, 128, 333, 177],
    "128": [80] * 30 + list(range(97, 129)) + [129, 256, 0, 1, 17, 63],
    "64": [20] * 40 + list(range(0, 66)) + [128, 129],
}


@pytest.mark.parametrize("K", [16, 80, 128, 272, 400, 512])
@pytest.mark.parametrize("N,gated", [(4100, False), (2049, True), (4097, False), (4352, False)])
@pytest.mark.parametrize("rows", MANY)
def test_many_rows(rows, N, gated, K):
    """Workgroups enough for each form of the many-row kernel: every filling of a row
    tile, channels that end inside a chunk, outputs that end inside a block, odd ones."""
    if rows != "256":
        N = N // 4 + N % 2
    counts = MANY[rows]
    c = Case(filled(counts), len(counts), 0, K, N, 1, gated)
    c.check()


def test_many_rows_in_the_fixed_capacity_layout():
    counts = MANY["256"]
    for cap in (300, 1000):
        Case(filled(counts), len(counts), cap, 208, 3600, 0, False).check()
    Case(filled(MANY["128"]), len(MANY["128"]), 120, 336, 1100, 0, True).check()


@pytest.mark.parametrize("T", [3, 400])
def test_largest_sums(T):
    """65536 products of -128 and -128: 2^30."""
    Case(np.zeros((T, 1), np.int32), 1, 0, 65536, 33, 1, False, extreme=True).check()


def test_ids_that_name_no_expert():
    idx = uniform(90, 8, 3)
    idx[::5] = -1
    idx[1::7, 2] = 1000
    for fmt in (0, 1):
        Case(idx, 8, 0, 160, 72, fmt, True).check()
        Case(idx, 8, 9, 160, 72, fmt, False).check()
    Case(np.full((5, 2), -1, np.int32), 4, 0, 64, 24, 0, False).check()


@pytest.mark.parametrize("fmt", [0, 1])
def test_no_tokens(fmt):
    prob, mm = ep.Problem(0, 128, 2, 4), ep.ExpertI8(64, 24, fmt)
    lay = ep.Layout(torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(5, dtype=torch.int32, device=DEV),
                    None, None, None)
    rows = torch.empty((0, 64), dtype=torch.int8 if fmt else torch.bfloat16, device=DEV)
    ep.ep_expert_i8(prob, mm, rows, lay, torch.zeros((4, 24, 64), dtype=torch.int8, device=DEV),
                    torch.zeros((4, 24), device=DEV), torch.empty((0, 24), dtype=torch.bfloat16, device=DEV),
                    row_scales=torch.empty(0, device=DEV),
                    workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()


def test_layout_of_another_problem_stays_inside():
    """Counts that add up to more rows than there are, and negative ones."""
    c = Case(uniform(60, 8, 2), 8, 0, 256, 64, 0, False)
    c.lay.count.fill_(1 << 30)
    c.lay.offset.fill_(1 << 30)
    c.rows.fill_(1.0)
    c.run()
    c.lay.count.fill_(-5)
    c.lay.offset.fill_(-5)
    assert (c.run().view(torch.int16) == SENTINEL).all()


@pytest.mark.parametrize("T", [20, 40])  # each kernel
def test_rows_and_weights_beyond_32_bit_offsets(T):
    """Weights of 4.5 GB and receive rows of 2.3 GB; the last expert's, at the end
    of both."""
    E, K, N, cap = 3, 65536, 23000, 12000
    idx = np.full((T, 1), 2, np.int32)
    idx[0] = 0
    r, lay = make_layout(idx, E, cap)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    w = torch.randint(-128, 128, (E, N, K), generator=g, device=DEV, dtype=torch.int8)
    q = torch.zeros((E * cap, K), dtype=torch.int8, device=DEV)
    at = torch.from_numpy(np.flatnonzero(r["src_of_slot"] >= 0)).to(DEV)
    q[at] = torch.randint(-128, 128, (T, K), generator=g, device=DEV, dtype=torch.int8)
    scale = torch.full((E, N), 2.0 ** -20, device=DEV)
    rs = torch.ones(E * cap, device=DEV)
    out = torch.zeros((E * cap, N), dtype=torch.bfloat16, device=DEV)
    prob = ep.Problem(T, 128, 1, E, cap)
    print("[gpu] products beyond 32-bit offsets", flush=True)
    ep.ep_expert_i8(prob, ep.ExpertI8(K, N, 1), q, lay, w, scale, out, row_scales=rs)
    torch.cuda.synchronize()
    for row in (0, int(at[-1])):
        e = row // cap
        for n in (0, 1, N // 2, N - 1):
            s = int((q[row].long() * w[e, n].long()).sum())
            want = s * 2.0 ** -20
            assert abs(float(out[row, n]) - want) <= (4 * ref.U + 2.0 ** -8) * abs(want)
    assert not out[1:cap].any()


def test_a_row_does_not_depend_on_the_others():
    """Few rows and many rows per expert, in any order: the sums are exact, so a
    row's bits are the same."""
    K, N = 784, 200
    r = np.random.default_rng(3)
    q = torch.from_numpy(r.integers(-128, 128, (600, K), dtype=np.int8)).to(DEV)
    w = torch.from_numpy(r.integers(-128, 128, (1, 2 * N, K), dtype=np.int8)).to(DEV)
    s = torch.full((1, 2 * N), 1e-4, device=DEV)
    rs = torch.from_numpy((r.random(600) + 0.1).astype(np.float32)).to(DEV)

    def products(rows):
        n = len(rows)
        _, lay = make_layout(np.zeros((n, 1), np.int32), 1, 0)
        out = torch.empty((n, N), dtype=torch.bfloat16, device=DEV)
        ep.ep_expert_i8(ep.Problem(n, 128, 1, 1), ep.ExpertI8(K, N, 1, 1), q[rows].contiguous(), lay, w, s,
                        out, row_scales=rs[rows].contiguous())
        return out

    everything = torch.arange(600, device=DEV)
    whole = products(everything)
    assert torch.equal(products(everything.flip(0)).flip(0), whole)
    for n in (1, 17, 100, 333):
        assert torch.equal(products(everything[:n]), whole[:n])


def test_replayed_graph_and_streams():
    a = Case(uniform(100, 16, 4), 16, 0, 512, 96, 0, True)
    b = Case(uniform(900, 4, 2), 4, 0, 384, 160, 0, False, seed=9)
    outs = [torch.zeros((c.R, c.N), dtype=torch.bfloat16, device=DEV) for c in (a, b)]
    for c, o in zip((a, b), outs):
        c.call(o)
    torch.cuda.synchronize()
    graphs = []
    for c, o in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(o)
        graphs.append(g)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for i in range(3):
        for c in (a, b):
            c.rows.copy_(torch.randn(c.R, c.K, device=DEV))
        want = []
        for c in (a, b):
            o = torch.zeros((c.R, c.N), dtype=torch.bfloat16, device=DEV)
            c.call(o)
            want.append(o)
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(5)
        torch.cuda.synchronize()
        for g, q in zip(graphs, (s, t)):
            with torch.cuda.stream(q):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), i


def test_layout_of_another_problem_dispatch():
    """Slots outside the receive rows are not followed."""
    T, H, k, E = 30, 128, 3, 8
    prob = ep.Problem(T, H, k, E)
    r, lay = make_layout(uniform(T, E, k), E, 0)
    lay.slot_of[::2] += T * k
    lay.slot_of[1::4] = -3
    x = torch.randn(T, H, device=DEV).bfloat16()
    q = torch.full((T * k, H), 0x5A, dtype=torch.int8, device=DEV)
    s = torch.full((T * k,), 77.0, device=DEV)
    ep.ep_dispatch_i8(prob, x, lay, q, s)
    torch.cuda.synchronize()
    want, scale = ref.quant(x.float().cpu().numpy())
    slot = lay.slot_of.cpu().numpy()
    there = np.zeros(T * k, bool)
    for t in range(T):
        for j in range(k):
            if 0 <= slot[t, j] < T * k:
                there[slot[t, j]] = True
                assert np.array_equal(q[slot[t, j]].cpu().numpy(), want[t])
                assert float(s[slot[t, j]]) == float(scale[t])
    assert (q.cpu().numpy()[~there] == 0x5A).all() and (s.cpu().numpy()[~there] == 77.0).all()


def test_binding_refuses():
    c = Case(uniform(6, 4, 2), 4, 0, 64, 24, 1, False)
    out = torch.empty((c.R, c.N), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(TypeError):
        ep.ep_expert_i8(c.prob, c.mm, c.rows.bfloat16(), c.lay, c.d_w, c.d_scale, out, row_scales=c.row_scales)
    with pytest.raises(TypeError):
        ep.ep_expert_i8(c.prob, c.mm, c.rows, c.lay, c.d_w.view(torch.uint8), c.d_scale, out, row_scales=c.row_scales)
    with pytest.raises((TypeError, ValueError)):
        ep.ep_expert_i8(c.prob, c.mm, c.rows, c.lay, c.d_w, c.d_scale, out)
    with pytest.raises(ValueError):
        ep.ep_expert_i8(c.prob, c.mm, c.rows, c.lay, c.d_w[:, :23].contiguous(), c.d_scale, out, row_scales=c.row_scales)
    with pytest.raises(ep.EpError):
        ep.ep_expert_i8(c.prob, ep.ExpertI8(64, 24, 0), torch.zeros((c.R, 64), dtype=torch.bfloat16, device=DEV),
                        c.lay, c.d_w, c.d_scale, out)
    x = torch.zeros((6, 64), dtype=torch.bfloat16, device=DEV)
    prob = ep.Problem(6, 64, 2, 4)
    q, s = torch.empty((12, 64), dtype=torch.int8, device=DEV), torch.empty(12, device=DEV)
    with pytest.raises(TypeError):
        ep.ep_dispatch_i8(prob, x.float(), c.lay, q, s)
    with pytest.raises(TypeError):
        ep.ep_dispatch_i8(prob, x, c.lay, q.view(torch.uint8), s)
    with pytest.raises(ValueError):
        ep.ep_dispatch_i8(prob, x, c.lay, q[:6], s)
