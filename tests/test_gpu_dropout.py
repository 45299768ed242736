"""ep_combine_dropout and ep_combine_backward against the 64-bit forms."""
import numpy as np
import pytest
import torch

import combine_ep_layout_09_amd as ep
import oracle
from tests import block_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SENTINEL = 0x5A5A  # a finite bf16 pattern that no test output produces by chance


def f64(t):
    return t.double().cpu().numpy()


def make_layout(idx, E, cap):
    r = oracle.layout(idx, E, cap)
    return r, ep.Layout(*(torch.from_numpy(np.ascontiguousarray(r[n], np.int32)).to(DEV)
                          for n in ("count", "offset", "slot_of", "src_of_slot", "status")))


def uniform(T, E, k, seed=0):
    r = np.random.default_rng(seed)
    return np.argsort(r.random((T, E)), 1)[:, :k].astype(np.int32)


class Case:
    def __init__(self, idx, E, cap, H, p, residual=True, seed=0):
        T, k = idx.shape
        r = np.random.default_rng(seed + 13 * T + H)
        self.T, self.k, self.E, self.cap, self.H, self.p = T, k, E, cap, H, p
        self.prob = ep.Problem(T, H, k, E, cap)
        print(f"[gpu] {self.prob!r} p {p} residual {residual}", flush=True)
        self.ref, self.lay = make_layout(idx, E, cap)
        self.slot = self.ref["slot_of"].reshape(T, k)
        R = self.R = ep.ep_num_recv_rows(self.prob)
        used = torch.from_numpy(self.ref["src_of_slot"] >= 0)
        eo = torch.from_numpy(r.standard_normal((R, H)).astype(np.float32)).to(torch.bfloat16)
        eo[~used] = float("nan")
        self.used, self.eo = used, eo.to(DEV)
        self.w = torch.from_numpy((r.random((T, k)) + 0.1).astype(np.float32)).to(DEV)
        self.rng = torch.from_numpy(r.integers(-2 ** 63, 2 ** 63, 2, dtype=np.int64)).to(DEV)
        self.dy = torch.from_numpy(r.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).to(DEV)
        self.res = None
        if residual:
            self.res = torch.from_numpy(r.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).to(DEV)

    def keep(self):
        seed, offset = (int(v) for v in self.rng.cpu())
        return ref.kept(self.T, self.H, self.p, seed, offset)

    def forward(self, rng="own", stream=None):
        room = torch.full((self.T * self.H + 64,), SENTINEL, dtype=torch.int16, device=DEV)
        y = room[:self.T * self.H].view(torch.bfloat16).view(self.T, self.H)
        ep.ep_combine_dropout(self.prob, self.eo, self.lay, self.w, self.p,
                              self.rng if rng == "own" else rng, y, residual=self.res, stream=stream)
        torch.cuda.synchronize()
        assert (room[self.T * self.H:] == SENTINEL).all(), "written behind the last row"
        return y

    def check_forward(self):
        got = f64(self.forward())
        want, bound = ref.combine(f64(self.eo), self.slot, f64(self.w), self.keep(), self.p,
                                  None if self.res is None else f64(self.res))
        off = np.abs(got - want)
        assert (off <= bound).all(), (np.argwhere(~(off <= bound))[:4], off.max())

    def backward(self, weights=True):
        room = torch.full((self.R * self.H + 64,), SENTINEL, dtype=torch.int16, device=DEV)
        deo = room[:self.R * self.H].view(torch.bfloat16).view(self.R, self.H)
        space = torch.full((self.T * self.k + 16,), 77.0, device=DEV)
        dw = space[:self.T * self.k].view(self.T, self.k)
        ep.ep_combine_backward(self.prob, self.dy, self.eo if weights else None, self.lay, self.w,
                               self.p, self.rng, deo, dw if weights else None)
        torch.cuda.synchronize()
        assert (room[self.R * self.H:] == SENTINEL).all() and (space[self.T * self.k:] == 77.0).all()
        return deo, dw

    def check_backward(self):
        deo, dw = self.backward()
        assert (deo.view(torch.int16).cpu()[~self.used] == SENTINEL).all(), "unused rows were written"
        rows, bounds, want, bound = ref.combine_grad(f64(self.dy), f64(self.eo), self.slot,
                                                     f64(self.w), self.keep(), self.p)
        off = np.abs(f64(dw) - want)
        assert (off <= bound).all(), (np.argwhere(~(off <= bound))[:4], off.max())
        got = f64(deo)
        for s, row in rows.items():
            off = np.abs(got[s] - row)
            assert (off <= bounds[s]).all(), (s, np.argwhere(~(off <= bounds[s]))[:4], off.max())
        return deo, dw


SHAPES = [
    # T, E, k, cap, H
    (1, 4, 1, 0, 8), (1, 256, 8, 0, 7168), (3, 8, 2, 0, 16), (5, 4, 3, 0, 1000), (64, 8, 2, 0, 256),
    (33, 16, 5, 4, 520), (40, 64, 7, 2, 512), (17, 8, 8, 0, 4096), (9, 32, 12, 0, 2056),
    (6, 64, 32, 3, 1288), (130, 5, 4, 0, 136), (2, 3, 2, 0, 65536), (7, 16, 6, 0, 16392),
    (300, 16, 6, 40, 3080),
]


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_shapes(shape, p):
    T, E, k, cap, H = shape
    c = Case(uniform(T, E, k, seed=T + k), E, cap, H, p, residual=T % 2 == 1)
    c.check_forward()
    c.check_backward()


def test_tokens_without_a_row():
    """Padding tokens and ids outside the experts: the skip connection alone, and
    gradients of nothing."""
    idx = uniform(50, 16, 4, seed=3)
    idx[7] = -1
    idx[20:24] = 99
    idx[30, 1:] = -1
    c = Case(idx, 16, 0, 264, 0.3)
    c.check_forward()
    _, dw = c.check_backward()
    y = c.forward()
    assert torch.equal(y[7], c.res[7]) and torch.equal(y[20:24], c.res[20:24])
    assert not dw[7].any() and not dw[30, 1:].any()
    c.res = None
    assert not c.forward()[7].any()


@pytest.mark.parametrize("H,k", [(16384, 3), (20480, 12), (33000, 4), (49160, 9)])
def test_rows_longer_than_a_workgroup_holds(H, k):
    c = Case(uniform(6, 32, k, seed=k), 32, 2, H, 0.1)
    c.check_forward()
    c.check_backward()


def test_an_expert_twice():
    """A token that names an expert twice has two rows there."""
    idx = uniform(60, 8, 4, seed=9)
    idx[:, 2] = idx[:, 0]
    idx[::3, 1] = idx[::3, 0]
    c = Case(idx, 8, 0, 520, 0.2)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("T", [40, 2100])
def test_without_dropout_it_is_the_combine(T):
    """p = 0 and no skip connection: the bits of ep_combine, in both launch forms."""
    c = Case(uniform(T, 32, 6), 32, 0, 7168, 0.0, residual=False)
    y = torch.empty_like(c.dy)
    ep.ep_combine(c.prob, c.eo, c.lay, c.w, y)
    assert torch.equal(c.forward(), y) and torch.equal(c.forward(rng=None), y)


@pytest.mark.parametrize("p", [2.0 ** -33, 0.1, 0.25, 0.999])
@pytest.mark.parametrize("T,H", [(3, 520), (2100, 7168)])
def test_mask_to_the_bit(T, H, p):
    """A sum of 1: what comes out is the factor or 0, by the generator's words.  The
    forward and the backward pass take the same mask, whatever form runs."""
    c = Case(uniform(T, 8, 1), 8, 0, H, p, residual=False)
    c.eo.fill_(1.0)
    c.w.fill_(1.0)
    c.dy.fill_(1.0)
    keep = torch.from_numpy(c.keep()).to(DEV)
    f = torch.tensor(1 / (1 - p), dtype=torch.float64).float().bfloat16().to(DEV)
    want = torch.where(keep, f, torch.zeros_like(f))
    assert torch.equal(c.forward(), want)
    deo, dw = c.backward()
    assert torch.equal(deo[c.lay.slot_of.view(-1).long()], want)
    n = keep.sum(1).double() / (1 - p)
    assert ((dw[:, 0].double() - n).abs() <= (ref.DOT_ADDS + 3) * ref.U * n).all()


def test_many_tokens():
    """Batches that take the forms for many tokens."""
    for T, H, k, cap in ((1500, 2048, 8, 0), (5000, 520, 3, 500)):
        c = Case(uniform(T, 16, k), 16, cap, H, 0.1)
        c.check_forward()
        c.check_backward()


def test_dropped_elements_do_not_pass_on_what_is_not_finite():
    c = Case(uniform(12, 8, 2), 8, 0, 512, 0.5)
    keep = torch.from_numpy(c.keep()).to(DEV)
    c.eo.fill_(float("inf"))
    y = c.forward()
    assert torch.equal(torch.where(keep, torch.zeros_like(y), y),
                       torch.where(keep, torch.zeros_like(c.res), c.res))
    assert torch.isinf(y[keep]).all()
    c.dy.fill_(float("nan"))
    deo, _ = c.backward(weights=False)
    rows = deo[c.lay.slot_of[:, 0].long()]
    assert not rows[~keep].any() and torch.isnan(rows[keep]).all()


@pytest.mark.parametrize("T,k,H", [(12, 2, 512), (30, 6, 4096), (9, 7, 16392), (2100, 8, 520)])
def test_gradients_do_not_take_what_is_not_finite_from_dropped_channels(T, k, H):
    """Infinities and NaN in the expert rows' and the gradient's dropped channels and
    an infinite weight: the output does not depend on any of them there."""
    c = Case(uniform(T, 8, k), 8, 0, H, 0.5)
    keep = torch.from_numpy(c.keep()).to(DEV)
    slot = c.lay.slot_of.long()
    clean, want = c.backward()
    for j in range(k):
        c.eo[slot[:, j]] = torch.where(keep, c.eo[slot[:, j]], float("inf") if j % 2 else float("nan"))
    c.dy = torch.where(keep, c.dy, float("-inf"))
    deo, dw = c.backward()
    assert torch.equal(dw, want) and torch.equal(deo, clean)
    c.w[:, 0] = float("inf")
    deo, dw = c.backward()
    assert torch.equal(dw, want)
    rows = deo[slot[:, 0]]
    assert not rows[~keep].any() and not torch.isfinite(rows[keep]).any()


def test_without_the_weights_gradient():
    c = Case(uniform(70, 16, 4), 16, 20, 1288, 0.2)
    deo, dw = c.backward()
    only, _ = c.backward(weights=False)
    assert torch.equal(deo.view(torch.int16), only.view(torch.int16))


def test_gradient_by_differences():
    """d_weights against differences of the forward call: the output is linear in a
    weight, so a difference is exact but for rounding to bf16."""
    c = Case(uniform(10, 8, 3), 8, 0, 1024, 0.25, residual=False)
    c.eo.copy_(torch.randint(-8, 9, c.eo.shape, device=DEV).float())
    c.dy.copy_(torch.randint(-8, 9, c.dy.shape, device=DEV).float())
    c.w.fill_(0.0)
    _, dw = c.backward()
    for j in range(3):
        c.w.fill_(0.0)
        c.w[:, j] = 3.0      # times 4 / 3 and a whole number of at most 8: whole, exact in bf16
        y = c.forward().double()
        want = (y * c.dy.double()).sum(1) / 3
        scale = (y * c.dy.double()).abs().sum(1) / 3
        assert ((dw[:, j].double() - want).abs() <= (ref.DOT_ADDS + 8) * ref.U * scale).all()


def test_other_offsets_and_seeds_give_other_masks():
    c = Case(uniform(16, 8, 1), 8, 0, 2048, 0.5, residual=False)
    base = c.rng.clone()
    seen = []
    for d in ((0, 0), (0, 1), (1, 0), (1 << 32, 0), (0, 1 << 32)):
        c.rng.copy_(base + torch.tensor(d, device=DEV))
        c.check_forward()
        seen.append(c.keep())
    for i in range(len(seen)):
        for j in range(i):
            assert 0.45 < (seen[i] == seen[j]).mean() < 0.55


def test_replayed_graph_takes_the_offset_of_the_moment():
    c = Case(uniform(200, 16, 4), 16, 0, 1032, 0.3)
    y, deo, dw = torch.empty_like(c.dy), torch.zeros_like(c.eo), torch.empty_like(c.w)

    def step():
        ep.ep_combine_dropout(c.prob, c.eo, c.lay, c.w, c.p, c.rng, y, residual=c.res)
        ep.ep_combine_backward(c.prob, c.dy, c.eo, c.lay, c.w, c.p, c.rng, deo, dw)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    last = None
    for i in range(4):
        c.rng[1] += 1
        step()
        torch.cuda.synchronize()
        want = [v.clone() for v in (y, deo, dw)]
        for v in (y, deo, dw):
            v.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((y, deo, dw), want):
            assert torch.equal(a, b), i
        assert last is None or not torch.equal(last, y)
        last = y.clone()


def test_two_streams():
    a = Case(uniform(100, 16, 4), 16, 0, 2048, 0.1)
    b = Case(uniform(2000, 8, 2), 8, 0, 1024, 0.4)
    want = [c.forward() for c in (a, b)] + [v for c in (a, b) for v in c.backward()]
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for i in range(3):
        y = [torch.empty_like(c.dy) for c in (a, b)]
        deo = [torch.full_like(c.eo, 0).view(torch.int16).fill_(SENTINEL).view(torch.bfloat16) for c in (a, b)]
        dw = [torch.empty_like(c.w) for c in (a, b)]
        torch.cuda.synchronize()
        for n, (c, q) in enumerate(((a, s), (b, t))):
            ep.ep_combine_dropout(c.prob, c.eo, c.lay, c.w, c.p, c.rng, y[n], residual=c.res, stream=q)
            ep.ep_combine_backward(c.prob, c.dy, c.eo, c.lay, c.w, c.p, c.rng, deo[n], dw[n], stream=q)
        torch.cuda.synchronize()
        for got, w in zip(y + [deo[0], dw[0], deo[1], dw[1]], want):
            assert torch.equal(got, w)


def test_layout_of_another_problem_stays_inside():
    """Slots outside the receive rows are not followed."""
    c = Case(uniform(40, 8, 3), 8, 0, 512, 0.2)
    c.lay.slot_of[::3] += c.R
    c.slot = np.where(f64(c.lay.slot_of) >= c.R, -1, f64(c.lay.slot_of)).astype(int)
    c.used = torch.zeros(c.R, dtype=torch.bool)
    c.used[torch.from_numpy(c.slot[c.slot >= 0])] = True
    c.check_forward()
    c.check_backward()


def test_binding_refuses():
    c = Case(uniform(4, 4, 2), 4, 0, 64, 0.1)
    y = torch.empty_like(c.dy)
    with pytest.raises(TypeError):
        ep.ep_combine_dropout(c.prob, c.eo.float(), c.lay, c.w, 0.1, c.rng, y)
    with pytest.raises(TypeError):
        ep.ep_combine_dropout(c.prob, c.eo, c.lay, c.w, 0.1, c.rng.int(), y)
    with pytest.raises(ValueError):
        ep.ep_combine_dropout(c.prob, c.eo, c.lay, c.w, 0.1, c.rng[:1], y)
    with pytest.raises(ValueError):
        ep.ep_combine_dropout(c.prob, c.eo, c.lay, c.w.t(), 0.1, c.rng, y)
    with pytest.raises(ep.EpError):
        ep.ep_combine_dropout(c.prob, c.eo, c.lay, c.w, 0.1, None, y)
    with pytest.raises(ep.EpError):
        ep.ep_combine_dropout(c.prob, c.eo, c.lay, c.w, 1.0, c.rng, y)
    with pytest.raises(ep.EpError):
        ep.ep_combine_dropout(c.prob, c.eo, c.lay, c.w, 0.1, c.rng, y, residual=y)
    with pytest.raises(ep.EpError):
        ep.ep_combine_backward(c.prob, c.dy, c.eo, c.lay, c.w, 0.1, c.rng, c.eo)
    with pytest.raises(ep.EpError):
        ep.ep_combine_backward(c.prob, c.dy, None, c.lay, c.w, 0.1, c.rng, torch.empty_like(c.eo),
                               torch.empty_like(c.w))
