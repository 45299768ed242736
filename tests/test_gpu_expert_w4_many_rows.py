"""ep_expert_w4 with many rows per expert: its many-row kernel at the widths that
models have.

Rows are small integers, scales powers of two near each other: every partial sum
is a whole number of units below 2^24, so that sums are exact in fp32 in any
order, and without the activation the outputs are the 64-bit products rounded
to bf16 once, bit for bit.  The activation adds, to exact gate and up values, an
exponential (2 units), a sum, a quotient and a product, and the rounding to bf16:
at most 6 * 2^-24 + 2^-8 of the result; below exp(-88) it is 0, which at these
magnitudes is under 1e-30.
"""
import numpy as np
import pytest
import torch

import combine_ep_layout_09_amd as ep
from tests import routing_reference as ref
from tests.test_gpu_expert_w4 import LARGE, SENTINEL, SMALL, make_layout, row_ranges, uniform

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E4M3_OF = np.array([0xC0, 0xB8, 0x00, 0x38, 0x40], np.uint8)  # -2 .. 2


def kernel_of(prob, mm):
    """The rows of a tile that launch_expert_w4's rule gives this problem: 64 or
    32 with the many-row kernel, 16 with the few-row one."""
    entries, held = prob.num_tokens * prob.num_topk, prob.num_experts * prob.capacity
    filled = min(held, entries) if prob.capacity else entries
    experts = min(prob.num_experts, filled)
    blocks = -(-mm.out_features * (1 + mm.activation) // 256)
    fp8 = mm.in_format != 0

    def many(rows, mc):
        return filled // experts > rows and (experts + filled // mc) * blocks > (200 if fp8 else 120)

    if not fp8 and many(40, 64):
        return 64
    return 32 if many(16 if fp8 else 8, 32) else 16


class Exact:
    def __init__(self, idx, E, cap, K, N, fmt, gated, seed=0):
        T, k = idx.shape
        r = np.random.default_rng(seed + K + 7 * N)
        self.E, self.cap, self.K, self.N, self.fmt, self.gated = E, cap, K, N, fmt, gated
        self.ref, self.lay = make_layout(idx, E, cap)
        self.prob, self.mm = ep.Problem(T, 128, k, E, cap, 0), ep.ExpertW4(K, N, fmt, gated)
        R = self.R = ep.ep_num_recv_rows(self.prob)
        print(f"[gpu] {self.prob!r} {self.mm!r} tile {kernel_of(self.prob, self.mm)}", flush=True)
        n2 = N * (2 if gated else 1)
        self.codes = r.integers(0, 256, (E, n2, K // 2), dtype=np.uint8)
        self.scales = r.integers(121, 124, (E, n2, K // 32), dtype=np.uint8)  # 2^-6 .. 2^-4
        self.scales[self.ref["count"] == 0] = 255  # not read
        used = self.ref["src_of_slot"] >= 0
        self.q = r.integers(0, 5, (R, K), dtype=np.uint8)
        self.row_scales = self.rs = None
        if fmt:
            rows = E4M3_OF[self.q]
            rows[~used] = 0x7F
            self.rows = torch.from_numpy(rows).to(DEV)
            b = r.integers(125, 128, (R, K // 128), dtype=np.uint8)  # 2^-2 .. 1
            self.rs = np.ldexp(1.0, b.astype(np.int32) - 127)
            b[~used] = 255
            s = b if fmt == 2 else np.where(used[:, None], self.rs, np.nan).astype(np.float32)
            self.row_scales = torch.from_numpy(s).to(DEV)
        else:
            self.rows = torch.from_numpy(self.q).to(DEV).to(torch.bfloat16) - 2
            self.rows[torch.from_numpy(~used).to(DEV)] = float("nan")
        self.d_codes = torch.from_numpy(self.codes).to(DEV)
        self.d_scales = torch.from_numpy(self.scales).to(DEV)

    def launch(self, out, stream=None):
        ep.ep_expert_w4(self.prob, self.mm, self.rows, self.lay, self.d_codes, self.d_scales, out,
                        row_scales=self.row_scales, stream=stream)

    def room(self):
        room = torch.full((self.R * self.N + 4096,), SENTINEL, dtype=torch.int16, device=DEV)
        return room, room[:self.R * self.N].view(torch.bfloat16).view(self.R, self.N)

    def run(self):
        room, out = self.room()
        self.launch(out)
        torch.cuda.synchronize()
        assert (room[self.R * self.N:] == SENTINEL).all(), "written behind the last row"
        return out

    def want(self, e, a, b, cols=slice(None)):
        """Exact gate (and up) values of rows a..b of expert e."""
        x = self.q[a:b].astype(np.float64) - 2
        if self.rs is not None:
            x *= np.repeat(self.rs[a:b], 128, 1)
        n = np.arange(self.N)[cols]
        n = np.concatenate([n, n + self.N]) if self.gated else n
        return x @ ref.decode_w4(self.codes[e][n], self.scales[e][n]).T

    def check(self, cols=slice(None)):
        out = self.run()
        filled = np.zeros(self.R, bool)
        got = out.float().cpu().numpy().astype(np.float64)
        for e, a, b in row_ranges(self.ref, self.E, self.cap, self.R):
            if a == b:
                continue
            filled[a:b] = True
            y, g = self.want(e, a, b, cols), got[a:b, cols]
            assert np.abs(y).max() < 2.0 ** (24 - 9)  # units of 2^-9: the sums are exact
            if self.gated:
                gate, up = np.split(y, 2, 1)
                with np.errstate(over="ignore"):
                    y = gate / (1.0 + np.exp(-gate)) * up
                bad = np.abs(g - y) > (6 * 2.0 ** -24 + 2.0 ** -8) * np.abs(y) + 1e-30
            else:
                bad = g != torch.from_numpy(y).to(torch.float32).to(torch.bfloat16).double().numpy()
            assert not bad.any(), (e, np.argwhere(bad)[:5])
        bits = out.view(torch.int16).cpu().numpy()
        assert (bits[~filled] == SENTINEL).all(), "rows that no entry fills were written"
        return out


def table(counts, E=228, seed=0):
    idx = np.repeat(np.arange(E), np.resize(counts, E)).astype(np.int32)[:, None]
    return np.random.default_rng(seed).permutation(idx)


# widths whose rows of scales are whole 16-byte pieces: one segment of 4096
# channels and less, exactly one, and parts and the whole of a second and third
@pytest.mark.parametrize("K,N", [(512, 260), (1536, 130), (4096, 33), (4608, 64), (7168, 40), (8704, 7)])
@pytest.mark.parametrize("counts,fmt,gated,cap,tile", [
    (SMALL, 0, True, 0, 32), (SMALL, 0, False, 24, 32), (LARGE, 0, True, 48, 64),
    (LARGE, 0, False, 0, 64), (SMALL, 2, False, 0, 32), (LARGE, 1, True, 48, 32),
    (LARGE, 2, True, 0, 32)])
def test_widths_of_models(K, N, counts, fmt, gated, cap, tile):
    c = Exact(table(counts), 228, cap, K, N, fmt, gated)
    assert kernel_of(c.prob, c.mm) == tile
    c.check()


# and some whose rows of scales are words, or no whole words
@pytest.mark.parametrize("K,fmt", [(640, 0), (4224, 1), (672, 0), (4192, 0)])
@pytest.mark.parametrize("counts", [SMALL, LARGE], ids=["small", "large"])
def test_other_widths(K, fmt, counts):
    c = Exact(table(counts), 228, 0, K, 70, fmt, True)
    assert kernel_of(c.prob, c.mm) > 16
    c.check()


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("gated", [False, True])
def test_rows_of_a_prompt(fmt, gated):
    """128 rows per expert in the mean, K 7168: 1024 tokens, 64 experts, k 8."""
    c = Exact(uniform(1024, 64, 8), 64, 0, 7168, 130, fmt, gated)
    assert kernel_of(c.prob, c.mm) == (32 if fmt else 64)
    c.check(slice(0, 130, 9))


def test_one_expert_takes_a_prompt():
    """4096 rows on one expert of many: its tiles are all there are."""
    for fmt in (0, 1):
        c = Exact(np.full((4096, 1), 5, np.int32), 64, 0, 512, 300, fmt, False)
        assert kernel_of(c.prob, c.mm) > 16
        c.check()


def many(fmt=0, counts=LARGE):
    c = Exact(table(counts), 228, 0, 1024, 72, fmt, True)
    assert kernel_of(c.prob, c.mm) == (64 if fmt == 0 and counts is LARGE else 32)
    return c


FORMS = pytest.mark.parametrize("fmt,counts", [(0, SMALL), (0, LARGE), (1, LARGE)])


@FORMS
def test_not_finite_rows_stay_in_their_outputs(fmt, counts):
    c = many(fmt, counts)
    clean = c.run().view(torch.int16).clone()
    bad = [3, 700, c.R - 1]
    if fmt:
        c.rows[bad, 17] = 0x7F
    else:
        c.rows[bad[:2], 17] = float("inf")
        c.rows[bad[2], 1000] = float("nan")
    got = c.run()
    keep = torch.ones(c.R, dtype=torch.bool, device=DEV)
    keep[bad] = False
    assert torch.equal(got.view(torch.int16)[keep], clean[keep])
    assert all(not torch.isfinite(got[b].float()).all() for b in bad)


@FORMS
def test_a_layout_of_another_problem_stays_inside(fmt, counts):
    """Counts beyond the rows are cut to them; run() looks behind the last row."""
    c = many(fmt, counts)
    c.lay.count[100:] += 1000
    c.lay.offset[50:] = 10 ** 9
    c.run()
    c.lay.count.fill_(2 ** 31 - 1)
    c.run()
    c.lay.count.fill_(-5)
    assert (c.run().view(torch.int16) == SENTINEL).all()


def test_repeats_streams_and_replays():
    """Equal bits on every call, on two streams at once, and from a graph that is
    replayed between eager calls."""
    cs = [many(0, LARGE), many(1, LARGE), many(0, SMALL)]
    want = [c.check().view(torch.int16).clone() for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [torch.zeros((c.R, c.N), dtype=torch.bfloat16, device=DEV) for c in cs]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, o, s in zip(cs, outs, streams):
            c.launch(o, stream=s)
    torch.cuda.synchronize()
    for o, w, c in zip(outs, want, cs):
        assert torch.equal(o.view(torch.int16), w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c, o in zip(cs, outs):
            c.launch(o)
    for rep in range(4):
        for o in outs:
            o.fill_(float("nan"))
        g.replay()
        again = cs[rep % 3].run()
        torch.cuda.synchronize()
        assert torch.equal(again.view(torch.int16), want[rep % 3])
        for o, w in zip(outs, want):
            assert torch.equal(o.view(torch.int16), w), rep


def test_weights_beyond_32_bit_offsets():
    """132 experts of 32 MiB of codes: the last one's rows lie beyond 2^32 bytes.
    It takes every entry; the others' scales are NaN."""
    E, N, K, T = 132, 8192, 8192, 132 * 9
    r = np.random.default_rng(0)
    last = r.integers(0, 256, (N, K // 2), dtype=np.uint8)
    ls = r.integers(121, 124, (N, K // 32), dtype=np.uint8)
    codes = torch.zeros((E, N, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.full((E, N, K // 32), 255, dtype=torch.uint8, device=DEV)
    codes[E - 1], scales[E - 1] = torch.from_numpy(last).to(DEV), torch.from_numpy(ls).to(DEV)
    _, lay = make_layout(np.full((T, 1), E - 1, np.int32), E, 0)
    q = r.integers(-2, 3, (T, K), dtype=np.int8)
    x = torch.from_numpy(q).to(DEV).to(torch.bfloat16)
    out = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    prob, mm = ep.Problem(T, 128, 1, E), ep.ExpertW4(K, N)
    assert kernel_of(prob, mm) == 32
    ep.ep_expert_w4(prob, mm, x, lay, codes, scales, out)
    torch.cuda.synchronize()
    cols = np.concatenate([np.arange(0, N, 173), [N - 1]])
    y = q.astype(np.float64) @ ref.decode_w4(last[cols], ls[cols]).T
    want = torch.from_numpy(y).to(torch.float32).to(torch.bfloat16)
    assert torch.equal(out[:, torch.from_numpy(cols).to(DEV)].cpu(), want)
