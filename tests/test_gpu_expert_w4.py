"""ep_expert_w4 against the 64-bit products.

Tolerance of an output: its products are exact; on the way into the fp32 sum a
product passes at most K / 4 + 8 additions (a quarter of the channels per wave,
three to join the waves), each rounding by 2^-24 of a partial sum that the
magnitudes of the products bound; row scales add one rounding per 128
channels, inside that count; the result is rounded to bf16 once, 2^-8.
"""
import numpy as np
import pytest
import torch

import combine_ep_layout_09_amd as ep
import oracle
import workloads
from tests import routing_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
SENTINEL = 0x5A5A  # a finite bf16 pattern that no test output produces by chance


def bf16_np(t):
    return t.float().cpu().numpy().astype(np.float64)


def make_layout(idx, E, cap):
    r = oracle.layout(idx, E, cap)
    lay = ep.Layout(*(torch.from_numpy(np.ascontiguousarray(r[n], np.int32)).to(DEV)
                      for n in ("count", "offset", "slot_of", "src_of_slot", "status")))
    return r, lay


def row_ranges(r, E, cap, R):
    for e in range(E):
        a = e * cap if cap else int(r["offset"][e])
        n = int(r["count"][e])
        yield e, a, a + (min(n, cap) if cap else n)


class Case:
    def __init__(self, idx, E, cap, K, N, fmt, gated, seed=0, scale_lo=118, scale_hi=124):
        T, k = idx.shape
        r = np.random.default_rng(seed + K + 7 * N)
        self.E, self.cap, self.K, self.N, self.fmt, self.gated = E, cap, K, N, fmt, gated
        self.ref, self.lay = make_layout(idx, E, cap)
        self.prob = ep.Problem(T, 128, k, E, cap, 0)
        self.mm = ep.ExpertW4(K, N, fmt, gated)
        R = self.R = ep.ep_num_recv_rows(self.prob)
        n2 = N * (2 if gated else 1)
        print(f"[gpu] {self.prob!r} {self.mm!r}", flush=True)
        self.codes = r.integers(0, 256, (E, n2, K // 2), dtype=np.uint8)
        self.scales = r.integers(scale_lo, scale_hi, (E, n2, K // 32), dtype=np.uint8)
        used = self.ref["src_of_slot"] >= 0
        if fmt:
            codes = r.integers(0, 256, (R, K), dtype=np.uint8)
            codes[(codes & 127) == 127] = 0x38
            codes[~used] = 0x7F  # NaN
            v = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
            if fmt == 1:
                s = (r.random((R, K // 128)) / 300).astype(np.float32)
                sv = s.astype(np.float64)
            else:
                s = r.integers(116, 121, (R, K // 128), dtype=np.uint8)
                sv = np.ldexp(1.0, s.astype(np.int32) - 127)
            s[~used] = 0xFF if fmt == 2 else np.nan
            self.x = v * np.repeat(sv, 128, 1)
            self.rows = torch.from_numpy(codes).to(DEV)
            self.row_scales = torch.from_numpy(s).to(DEV)
        else:
            x = torch.from_numpy(r.standard_normal((R, K)).astype(np.float32)).to(torch.bfloat16)
            x[torch.from_numpy(~used)] = float("nan")
            self.x = x.double().numpy()
            self.rows = x.to(DEV)
            self.row_scales = None
        # weights of experts that no entry names hold NaN scales
        self.scales[self.ref["count"] == 0] = 255
        self.d_codes = torch.from_numpy(self.codes).to(DEV)
        self.d_scales = torch.from_numpy(self.scales).to(DEV)

    def run(self):
        room = torch.full((self.R * self.N + 64,), SENTINEL, dtype=torch.int16, device=DEV)
        out = room[:self.R * self.N].view(torch.bfloat16).view(self.R, self.N)
        ep.ep_expert_w4(self.prob, self.mm, self.rows, self.lay, self.d_codes, self.d_scales, out,
                        row_scales=self.row_scales)
        torch.cuda.synchronize()
        assert (room[self.R * self.N:] == SENTINEL).all(), "written behind the last row"
        return out

    def check(self, out=None):
        out = self.run() if out is None else out
        bits = out.view(torch.int16).cpu().numpy()
        got = bf16_np(out)
        filled = np.zeros(self.R, bool)
        for e, a, b in row_ranges(self.ref, self.E, self.cap, self.R):
            if a == b:
                continue
            filled[a:b] = True
            y, mag = ref.products(self.x[a:b], self.codes[e], self.scales[e], self.gated)
            tol = (self.K / 4 + 8) * U * mag + 2.0 ** -8 * np.abs(y) + 2.0 ** -133
            bad = np.abs(got[a:b] - y) > tol
            assert not bad.any(), (e, np.argwhere(bad)[:5], np.abs(got[a:b] - y).max())
        assert (bits[~filled] == SENTINEL).all(), "rows that no entry fills were written"
        return out


def uniform(T, E, k, seed=0):
    r = np.random.default_rng(seed)
    return np.argsort(r.random((T, E)), 1)[:, :k].astype(np.int32)


SHAPES = [
    # T, E, k, cap, K, N
    (1, 8, 2, 0, 32, 1), (1, 256, 8, 0, 256, 40), (2, 4, 4, 0, 96, 33), (5, 3, 1, 0, 160, 64),
    (16, 8, 2, 0, 128, 65), (64, 8, 2, 0, 256, 100), (33, 5, 3, 0, 544, 31),
    (128, 16, 4, 40, 512, 96), (128, 16, 4, 3, 512, 48), (7, 1024, 4, 2, 64, 16),
    (130, 2, 2, 0, 640, 70), (100, 1, 1, 0, 384, 17), (300, 4, 2, 200, 1024, 128),
    (40, 8, 8, 40, 2080, 20), (3, 300, 3, 1, 256, 130),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_shapes(shape, fmt, gated):
    T, E, k, cap, K, N = shape
    if fmt:
        K = (K + 127) // 128 * 128
    Case(uniform(T, E, k), E, cap, K, N, fmt, gated).check()


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 129])
@pytest.mark.parametrize("fmt", [0, 1])
def test_rows_per_expert(m, fmt):
    """One expert with m rows between experts with one and none."""
    idx = np.concatenate([[0], np.full(m, 2), [4]]).astype(np.int32)[:, None]
    Case(idx, 6, 0, 256, 72, fmt, True).check()
    Case(idx, 6, 64, 256, 72, fmt, False).check()


SMALL = [0, 1, 9, 15, 16, 17, 24, 31, 32, 33, 20, 12]
LARGE = [0, 1, 33, 63, 64, 65, 100, 129, 48, 16, 5, 70]


@pytest.mark.parametrize("counts", [SMALL, LARGE], ids=["small", "large"])
@pytest.mark.parametrize("K,N,cap", [(32, 1, 0), (96, 33, 0), (256, 72, 64), (544, 130, 0),
                                     (1152, 260, 40), (4224, 33, 0), (4640, 5, 0), (8320, 3, 0)])
@pytest.mark.parametrize("fmt,gated", [(0, False), (0, True), (1, True), (2, False)])
def test_many_experts_with_many_rows(K, N, cap, counts, fmt, gated):
    """Row tiles of every filling, enough of them to occupy the card."""
    E = 228
    idx = np.repeat(np.arange(E), np.resize(counts, E)).astype(np.int32)[:, None]
    idx = np.random.default_rng(K).permutation(idx)
    Case(idx, E, cap, (K + 127) // 128 * 128 if fmt else K, N, fmt, gated).check()


def test_skewed_routing_and_foreign_ids():
    r = np.random.default_rng(3)
    idx = (r.zipf(1.3, (400, 6)) - 1).astype(np.int64)
    idx = np.where(idx < 16, idx, r.integers(-2, 20, idx.shape)).astype(np.int32)
    for cap in (0, 37):
        for gated in (False, True):
            Case(idx, 16, cap, 512, 80, 0, gated).check()


def test_no_rows():
    Case(np.zeros((0, 2), np.int32), 8, 0, 128, 32, 0, True).check()
    Case(np.full((9, 2), -1, np.int32), 8, 0, 128, 32, 0, True).check()
    Case(np.full((9, 2), 99, np.int32), 8, 4, 128, 32, 1, False).check()


def test_wide_input_and_repeat():
    c = Case(uniform(9, 4, 2), 4, 0, 7168, 96, 0, True)
    a = c.check().clone()
    assert torch.equal(a.view(torch.int16), c.run().view(torch.int16))
    Case(uniform(9, 4, 2), 4, 9, 65536, 16, 1, False).check()


def test_extreme_scales():
    """Scale bytes over the whole range, one per output: products from 2^-127
    up, infinities where they overflow, and NaN for byte 255."""
    K, N, E = 128, 256, 1
    c = Case(np.zeros((3, 1), np.int32), E, 0, K, N, 0, False)
    c.scales[:] = np.arange(256, dtype=np.uint8)[None, :, None]
    x = torch.zeros((3, K), dtype=torch.bfloat16)
    x[0, 5] = 1.0
    x[1, 70] = -2.0 ** -40
    x[2, 127] = 2.0 ** 40
    c.codes[:] = 0x25  # values 3 (even channels) and 1 (odd)
    c.rows, c.x = x.to(DEV), x.double().numpy()
    c.d_codes, c.d_scales = (torch.from_numpy(v).to(DEV) for v in (c.codes, c.scales))
    got = bf16_np(c.run())
    # a weight of 2^128 or more is infinite: 3 * 2^127, against 0 and not
    with np.errstate(invalid="ignore", over="ignore"):
        w = ref.decode_w4(c.codes[0], c.scales[0])
        w = np.where(np.abs(w) >= 2.0 ** 128, np.copysign(np.inf, w), w)
        want = (c.x[:, None] * w[None]).sum(2)
    assert np.isnan(want[:, 254:]).all() and np.isfinite(want[:, :254]).all()
    assert np.isnan(got[:, 254:]).all()
    got, want = got[:, :254], want[:, :254]
    over = np.abs(want) >= 2.0 ** 128
    assert np.isinf(got[over]).all() and (np.sign(got[over]) == np.sign(want[over])).all()
    normal = (np.abs(want) >= 2.0 ** -126) & ~over
    np.testing.assert_array_equal(got[normal], want[normal])
    assert (np.abs(got[np.abs(want) < 2.0 ** -126]) <= 2.0 ** -126).all()


def test_not_finite_rows_stay_in_their_outputs():
    c = Case(np.zeros((5, 1), np.int32), 2, 0, 256, 40, 0, True)
    clean = c.run().view(torch.int16).clone()
    c.rows[3, 17] = float("inf")
    c.rows[1, 200] = float("nan")
    got = c.run()
    keep = [0, 2, 4]
    assert torch.equal(got.view(torch.int16)[keep], clean[keep])
    assert not torch.isfinite(got[[1, 3]].float()).all()


def test_a_layout_of_another_problem_stays_inside():
    """Counts and offsets beyond the rows are cut to them."""
    c = Case(uniform(20, 4, 2), 4, 0, 128, 48, 0, False)
    c.lay.count += 1000
    c.lay.offset[2] = -5
    c.lay.offset[3] = 10 ** 9
    room = torch.full((c.R * c.N + 4096,), SENTINEL, dtype=torch.int16, device=DEV)
    out = room[:c.R * c.N].view(torch.bfloat16).view(c.R, c.N)
    ep.ep_expert_w4(c.prob, c.mm, c.rows, c.lay, c.d_codes, c.d_scales, out)
    torch.cuda.synchronize()
    assert (room[c.R * c.N:] == SENTINEL).all()


def test_weights_beyond_32_bit_offsets():
    """132 experts of 32 MiB of codes: the last experts' rows lie beyond
    2^32 bytes.  Only the last expert is named."""
    E, N, K = 132, 8192, 8192
    codes = torch.zeros((E, N, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.full((E, N, K // 32), 255, dtype=torch.uint8, device=DEV)
    r = np.random.default_rng(0)
    last = r.integers(0, 256, (N, K // 2), dtype=np.uint8)
    ls = r.integers(118, 124, (N, K // 32), dtype=np.uint8)
    codes[E - 1] = torch.from_numpy(last).to(DEV)
    scales[E - 1] = torch.from_numpy(ls).to(DEV)
    idx = np.full((2, 1), E - 1, np.int32)
    r0, lay = make_layout(idx, E, 0)
    x = torch.from_numpy(r.standard_normal((2, K)).astype(np.float32)).to(torch.bfloat16)
    out = torch.empty((2, N), dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_w4(ep.Problem(2, 128, 1, E), ep.ExpertW4(K, N), x.to(DEV), lay, codes, scales, out)
    torch.cuda.synchronize()
    y, mag = ref.products(x.double().numpy(), last, ls, False)
    assert (np.abs(bf16_np(out) - y) <= (K / 4 + 8) * U * mag + 2.0 ** -8 * np.abs(y)).all()


@pytest.mark.parametrize("cap,fp8", [(0, 0), (0, 2), (24, 1), (5, 1)])
def test_the_whole_layer(cap, fp8):
    """Gate logits to the layer's output through the public calls, as a
    program runs them: each stage is held to its own definition on what the
    stage before it left."""
    T, H, I, E, k = 48, 512, 160, 16, 4
    r = np.random.default_rng(8)
    dev = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    x = torch.from_numpy(r.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16)
    logits = dev((2 * r.standard_normal((T, E))).astype(np.float32))
    prob = ep.Problem(T, H, k, E, cap, fp8)
    rt = ep.Routing(T, E, k, 4, 2, "sigmoid")
    idx = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    lay, ws = ep.Layout.empty(prob, DEV), ep.alloc_workspace(prob, DEV)
    recv_x, recv_s = ep.alloc_recv(prob, DEV)
    recv_x.view(torch.uint8).fill_(0xFF)
    R = ep.ep_num_recv_rows(prob)
    c1, s1 = (r.integers(lo, hi, (E, 2 * I, n), dtype=np.uint8)
              for lo, hi, n in ((0, 256, H // 2), (118, 122, H // 32)))
    c2, s2 = (r.integers(lo, hi, (E, H, n), dtype=np.uint8)
              for lo, hi, n in ((0, 256, I // 2), (118, 122, I // 32)))
    h = torch.full((R, I), float("nan"), dtype=torch.bfloat16, device=DEV)
    eo = torch.full((R, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    dx, dc1, ds1, dc2, ds2 = x.to(DEV), dev(c1), dev(s1), dev(c2), dev(s2)
    up, down = ep.ExpertW4(H, I, fp8, 1), ep.ExpertW4(I, H)

    def layer():
        ep.ep_route(rt, logits, idx, w)
        ep.ep_layout_dispatch(prob, idx, lay, ws, dx, recv_x, recv_s)
        ep.ep_expert_w4(prob, up, recv_x, lay, dc1, ds1, h, row_scales=recv_s)
        ep.ep_expert_w4(prob, down, h, lay, dc2, ds2, eo)
        ep.ep_combine(prob, eo, lay, w, y)

    layer()
    torch.cuda.synchronize()
    ih = idx.cpu().numpy()
    np.testing.assert_array_equal(ih, ref.choose(logits.cpu().numpy(), k, 4, 2))
    lr = oracle.layout(ih, E, cap)
    np.testing.assert_array_equal(lay.count.cpu().numpy(), lr["count"])
    if fp8:
        v = recv_x.cpu().view(torch.float8_e4m3fn).double().numpy()
        s = recv_s.cpu().numpy()
        s = np.ldexp(1.0, s.astype(np.int32) - 127) if fp8 == 2 else s.astype(np.float64)
        xr = v * np.repeat(s, 128, 1)
    else:
        xr = bf16_np(recv_x)
    hv, ev, yv = bf16_np(h), bf16_np(eo), bf16_np(y)
    for e, a, b in row_ranges(lr, E, cap, R):
        for xin, got, cc, ss, gated, K in ((xr, hv, c1, s1, True, H), (hv, ev, c2, s2, False, I)):
            want, mag = ref.products(xin[a:b], cc[e], ss[e], gated)
            tol = (K / 4 + 8) * U * mag + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
            assert (np.abs(got[a:b] - want) <= tol).all()
    slot = lr["slot_of"].reshape(T, k)
    wv = w.cpu().numpy().astype(np.float64)
    want = sum(np.where(slot[:, j] >= 0, wv[:, j], 0)[:, None] * np.where(
        (slot[:, j] >= 0)[:, None], ev[np.maximum(slot[:, j], 0)], 0) for j in range(k))
    mag = sum(np.where(slot[:, j] >= 0, wv[:, j], 0)[:, None] * np.abs(np.where(
        (slot[:, j] >= 0)[:, None], ev[np.maximum(slot[:, j], 0)], 0)) for j in range(k))
    assert (np.abs(yv - want) <= 2.0 ** -8 * np.abs(want) + k * U * mag).all()

    # captured and replayed, with eager steps of another batch in between
    eager = y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    other = Case(uniform(64, 8, 2), 8, 0, 256, 100, 0, True)
    keep = other.run().view(torch.int16).clone()
    for rep in range(3):
        y.zero_()
        h.fill_(float("nan"))
        eo.fill_(float("nan"))
        g.replay()
        again = other.run()
        torch.cuda.synchronize()
        assert torch.equal(again.view(torch.int16), keep), rep
        assert torch.equal(y.view(torch.int16), eager.view(torch.int16)), rep


def test_two_streams_at_once():
    a = Case(uniform(64, 16, 4), 16, 0, 1024, 256, 0, True)
    b = Case(uniform(200, 8, 2), 8, 60, 512, 192, 1, False, seed=2)
    want = [c.run().view(torch.int16).clone() for c in (a, b)]
    outs = [torch.full((c.R, c.N), 0, dtype=torch.bfloat16, device=DEV) for c in (a, b)]
    for o in outs:
        o.view(torch.int16).fill_(SENTINEL)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        for c, o, st in zip((a, b), outs, s):
            ep.ep_expert_w4(c.prob, c.mm, c.rows, c.lay, c.d_codes, c.d_scales, o,
                            row_scales=c.row_scales, stream=st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o.view(torch.int16), w)


def test_prepared_call():
    c = Case(uniform(20, 8, 2), 8, 0, 256, 64, 2, True)
    want = c.run().view(torch.int16)
    out = torch.empty((c.R, c.N), dtype=torch.bfloat16, device=DEV)
    ep.prepare_expert_w4(c.prob, c.mm, c.rows, c.lay, c.d_codes, c.d_scales, out,
                         row_scales=c.row_scales)()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), want)


def test_the_decode_workloads_layout():
    """The decode batch: 128 tokens, 256 experts, k 8, capacity 128, FP8 rows."""
    wl = workloads.make(2, H=256)
    Case(wl.topk_idx, wl.E, wl.cap, 256, 48, 1, True).check()


@pytest.mark.parametrize("K,fmt", [(4640, 0), (8320, 0), (8704, 0), (8320, 1), (12288, 2)])
@pytest.mark.parametrize("T", [9, 60, 200])
def test_long_inputs(K, T, fmt):
    """Inputs whose scales take several turns through LDS, words and not, with
    few and many rows per expert."""
    Case(uniform(T, 2, 1), 2, 0, K, 68, fmt, True).check()
    Case(uniform(T, 2, 1), 2, 0, K, 131, fmt, False).check()


def test_one_expert_takes_everything():
    """All entries on one expert, every token on it twice: the other experts'
    weights are NaN and unread."""
    idx = np.full((150, 2), 5, np.int32)
    for fmt in (0, 1):
        Case(idx, 64, 0, 256, 100, fmt, True).check()
        Case(idx, 64, 17, 256, 100, fmt, False).check()
