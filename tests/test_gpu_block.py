"""The new calls together, as a program uses them: a training step through norm,
gate, dispatch, experts, combine with dropout and back, and a served layer in 8-bit
integers, eager and captured."""
import numpy as np
import pytest
import torch

import combine_ep_layout_09_amd as ep
from tests import block_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Step:
    """y = x + drop(sum_j w_j * scale_e(n_t)) with n = norm(x): every expert scales its
    rows by a vector of its own, so that the whole gradient can be followed."""

    def __init__(self, T=96, H=256, E=8, k=2, p=0.25):
        g = torch.Generator(device=DEV)
        g.manual_seed(11)
        self.T, self.H, self.E, self.k, self.p = T, H, E, k, p
        rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        self.x = rand(T, H).to(BF16)
        self.nw, self.nb = 1 + 0.2 * rand(H), 0.2 * rand(H)
        self.gate = rand(H, E) / np.sqrt(H)
        self.experts = (0.5 + torch.rand((E, H), generator=g, device=DEV)).to(BF16)
        self.dy = rand(T, H).to(BF16)
        self.rng = torch.tensor([1234567890123, 5], device=DEV)
        self.nm, self.prob = ep.Norm(T, H), ep.Problem(T, H, k, E)
        self.rt = ep.Routing(T, E, k)
        R = T * k
        empty = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
        self.n, self.mean, self.rstd = empty(T, H), empty(T, dtype=F32), empty(T, dtype=F32)
        self.logits, self.idx, self.w = empty(T, E, dtype=F32), empty(T, k, dtype=I32), empty(T, k, dtype=F32)
        self.lay, self.ws = ep.Layout.empty(self.prob, DEV), ep.alloc_workspace(self.prob, DEV)
        self.recv, self.eo, self.deo, self.drecv = (empty(R, H) for _ in range(4))
        self.y, self.dn, self.dx = (empty(T, H) for _ in range(3))
        self.dw, self.dlogits = empty(T, k, dtype=F32), empty(T, E, dtype=F32)
        self.dnw, self.dnb = empty(H, dtype=F32), empty(H, dtype=F32)
        self.space = empty(ep.ep_layer_norm_workspace_bytes(self.nm), dtype=torch.uint8)
        self.ones = torch.ones((T, k), device=DEV)

    def by_row(self):
        """Expert of each receive row."""
        at = torch.arange(self.T * self.k, dtype=I32, device=DEV)
        return torch.searchsorted(self.lay.offset[1:].contiguous(), at, right=True)

    def run(self):
        ep.ep_layer_norm(self.nm, self.x, self.nw, self.nb, self.n, mean=self.mean, rstd=self.rstd)
        torch.matmul(self.n.float(), self.gate, out=self.logits)
        ep.ep_route(self.rt, self.logits, self.idx, self.w)
        ep.ep_layout_dispatch(self.prob, self.idx, self.lay, self.ws, self.n, self.recv)
        scale = self.experts[self.by_row()]
        torch.mul(self.recv, scale, out=self.eo)
        ep.ep_combine_dropout(self.prob, self.eo, self.lay, self.w, self.p, self.rng, self.y,
                              residual=self.x)
        # and back
        ep.ep_combine_backward(self.prob, self.dy, self.eo, self.lay, self.w, self.p, self.rng,
                               self.deo, self.dw)
        torch.mul(self.deo, scale, out=self.drecv)
        ep.ep_combine(self.prob, self.drecv, self.lay, self.ones, self.dn)  # dispatch's gradient
        ep.ep_route_backward(self.rt, self.logits, self.idx, self.dlogits, d_weights=self.dw)
        self.dn.add_(self.dlogits @ self.gate.t().contiguous())
        ep.ep_layer_norm_backward(self.nm, self.x, self.dn, self.nw, self.mean, self.rstd, self.dx,
                                  d_weight=self.dnw, d_bias=self.dnb, workspace=self.space,
                                  d_skip=self.dy)

    def exact(self):
        """The same in 64 bits on the host, by automatic differentiation, for the experts
        that were chosen."""
        D = torch.float64
        x, nw, nb = (v.detach().cpu().to(D).requires_grad_() for v in (self.x, self.nw, self.nb))
        m = x.mean(1, keepdim=True)
        d = x - m
        n = d / torch.sqrt((d * d).mean(1, keepdim=True) + float(np.float32(1e-5))) * nw + nb
        logits = n @ self.gate.cpu().to(D)
        idx = self.idx.cpu().long()
        w = torch.softmax(logits.gather(1, idx), 1)
        s = sum(w[:, j:j + 1] * n * self.experts.cpu().to(D)[idx[:, j]] for j in range(self.k))
        keep = torch.from_numpy(ref.kept(self.T, self.H, self.p, *(int(v) for v in self.rng.cpu())))
        y = x + keep * s / (1 - self.p)
        grads = torch.autograd.grad((y * self.dy.cpu().to(D)).sum(), (x, nw, nb))
        return y.detach(), grads


def test_training_step():
    """Each intermediate tensor (the normalised rows, expert rows, their gradients)
    is rounded to bf16, 2^-9 of itself in the mean: a handful of such roundings on
    the way to every output."""
    s = Step()
    s.run()
    torch.cuda.synchronize()
    y, (dx, dnw, dnb) = s.exact()
    for name, got, want in (("y", s.y, y), ("dx", s.dx, dx), ("dw", s.dnw, dnw), ("db", s.dnb, dnb)):
        off = (got.cpu().double() - want).norm() / want.norm()
        assert off < 6 * 2.0 ** -8, (name, float(off))


def test_training_step_captured():
    """The whole step but the expert lookup of its layout replayed from a graph, with a new
    offset of the generator, beside an eager one."""
    s = Step()
    s.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    outs = ("y", "dx", "dnw", "dnb", "dw")
    for i in range(4):
        s.rng[1] += 7
        s.x.copy_(torch.randn(s.T, s.H, device=DEV))
        s.run()
        torch.cuda.synchronize()
        want = [getattr(s, n).clone() for n in outs]
        for n in outs:
            getattr(s, n).fill_(3)
        g.replay()
        torch.cuda.synchronize()
        for n, v in zip(outs, want):
            assert torch.equal(getattr(s, n), v), (i, n)


def served_layer(T, cap, captured):
    H, I, E, k = 512, 320, 16, 4
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    x, nw, nb = rand(T, H).to(BF16), 1 + 0.1 * rand(H), 0.1 * rand(H)
    gate = rand(H, E) / np.sqrt(H)
    codes = lambda *s: torch.randint(-127, 128, s, generator=g, device=DEV, dtype=torch.int8)  # noqa: E731
    up_w, down_w = codes(E, 2 * I, H), codes(E, H, I)
    up_s = (0.5 + torch.rand((E, 2 * I), generator=g, device=DEV)) / (73 * np.sqrt(H))
    down_s = (0.5 + torch.rand((E, H), generator=g, device=DEV)) / (73 * np.sqrt(I))
    nm, rt, prob = ep.Norm(T, H), ep.Routing(T, E, k), ep.Problem(T, H, k, E, cap)
    R = ep.ep_num_recv_rows(prob)
    n, y = torch.empty_like(x), torch.empty_like(x)
    logits, idx = torch.empty((T, E), device=DEV), torch.empty((T, k), dtype=I32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    lay, ws = ep.Layout.empty(prob, DEV), ep.alloc_workspace(prob, DEV)
    q, qs = torch.zeros((R, H), dtype=torch.int8, device=DEV), torch.zeros(R, device=DEV)
    h, out = torch.zeros((R, I), dtype=BF16, device=DEV), torch.zeros((R, H), dtype=BF16, device=DEV)
    up, down = ep.ExpertI8(H, I, in_format=1, activation=1), ep.ExpertI8(I, H, in_format=0)
    space = torch.empty(ep.ep_expert_i8_workspace_bytes(prob, down), dtype=torch.uint8, device=DEV)

    def run():
        ep.ep_layer_norm(nm, x, nw, nb, n)
        torch.matmul(n.float(), gate, out=logits)
        ep.ep_route(rt, logits, idx, w)
        ep.ep_layout(prob, idx, lay, ws)
        ep.ep_dispatch_i8(prob, n, lay, q, qs)
        ep.ep_expert_i8(prob, up, q, lay, up_w, up_s, h, row_scales=qs)
        ep.ep_expert_i8(prob, down, h, lay, down_w, down_s, out, workspace=space)
        ep.ep_combine_dropout(prob, out, lay, w, 0.0, None, y, residual=x)

    run()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for _ in range(3):
            eager = y.clone()
            y.fill_(0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, eager)
    # every stage from the tensors that the stage before left
    d = lambda t: t.double().cpu().numpy()  # noqa: E731
    slot = lay.slot_of.cpu().numpy()
    want, _ = ref.combine(d(out), slot, d(w), np.ones((T, H), bool), 0.0, d(x))
    assert np.abs(d(y) - want).max() <= 2.0 ** -7 * np.abs(want).max()
    qn, sn = ref.quant(d(n).astype(np.float32))
    for t in range(T):
        for j in range(k):
            r = slot[t, j]
            if r < 0:
                continue
            e = int(idx[t, j])
            assert np.array_equal(q[r].cpu().numpy(), qn[t]) and float(qs[r]) == float(sn[t])
            if t % 7 == 0:
                want, tol = ref.i8_products(qn[t:t + 1], sn[t:t + 1], up_w[e].cpu().numpy(),
                                            up_s[e].cpu().numpy(), True)
                assert (np.abs(d(h[r]) - want[0]) <= tol[0]).all()
                hq, hs = ref.quant(d(h[r:r + 1]).astype(np.float32))
                want, tol = ref.i8_products(hq, hs, down_w[e].cpu().numpy(), down_s[e].cpu().numpy(), False)
                assert (np.abs(d(out[r]) - want[0]) <= tol[0]).all()


@pytest.mark.parametrize("T,cap", [(1, 0), (40, 0), (40, 12), (300, 0)])
@pytest.mark.parametrize("captured", [False, True])
def test_served_layer(T, cap, captured):
    served_layer(T, cap, captured)


def test_no_tokens():
    """Batches without a token launch nothing."""
    prob = ep.Problem(0, 64, 2, 4)
    lay = ep.Layout(*(torch.zeros(n, dtype=I32, device=DEV) for n in (4, 5, 0, 0, 2)))
    x, w = torch.empty((0, 64), dtype=BF16, device=DEV), torch.empty((0, 2), device=DEV)
    rng = torch.zeros(2, dtype=torch.int64, device=DEV)
    ep.ep_combine_dropout(prob, x, lay, w, 0.5, rng, x.clone(), residual=x.clone())
    ep.ep_combine_backward(prob, x, x, lay, w, 0.5, rng, x.clone(), w.clone())
    ep.ep_dispatch_i8(prob, x, lay, torch.empty((0, 64), dtype=torch.int8, device=DEV),
                      torch.empty(0, device=DEV))
    torch.cuda.synchronize()


def test_prepared_calls():
    """The calls checked and marshalled once give what the plain ones give."""
    s = Step(T=50, H=264)
    s.run()
    torch.cuda.synchronize()
    want = {n: getattr(s, n).clone() for n in ("n", "mean", "rstd", "y", "deo", "dw", "dx", "dnw", "dnb")}
    q, qs = torch.zeros((100, 264), dtype=torch.int8, device=DEV), torch.zeros(100, device=DEV)
    mm = ep.ExpertI8(264 // 16 * 16, 40, 0)
    rows = torch.randn(100, mm.in_features, device=DEV).to(BF16)
    weights = torch.randint(-128, 128, (8, 40, mm.in_features), device=DEV, dtype=torch.int8)
    scales, out = torch.rand((8, 40), device=DEV), torch.zeros((100, 40), dtype=BF16, device=DEV)
    space = torch.empty(ep.ep_expert_i8_workspace_bytes(s.prob, mm), dtype=torch.uint8, device=DEV)
    ep.ep_dispatch_i8(s.prob, s.x, s.lay, q, qs)
    ep.ep_expert_i8(s.prob, mm, rows, s.lay, weights, scales, out, workspace=space)
    want.update(q=q.clone(), qs=qs.clone(), out=out.clone())
    calls = [
        ep.prepare_layer_norm(s.nm, s.x, s.nw, s.nb, s.n, mean=s.mean, rstd=s.rstd),
        ep.prepare_combine_dropout(s.prob, s.eo, s.lay, s.w, s.p, s.rng, s.y, residual=s.x),
        ep.prepare_combine_backward(s.prob, s.dy, s.eo, s.lay, s.w, s.p, s.rng, s.deo, s.dw),
        ep.prepare_layer_norm_backward(s.nm, s.x, s.dn, s.nw, s.mean, s.rstd, s.dx, d_weight=s.dnw,
                                       d_bias=s.dnb, workspace=s.space, d_skip=s.dy),
        ep.prepare_dispatch_i8(s.prob, s.x, s.lay, q, qs),
        ep.prepare_expert_i8(s.prob, mm, rows, s.lay, weights, scales, out, workspace=space),
    ]
    got = dict({n: getattr(s, n) for n in want if hasattr(s, n)}, q=q, qs=qs, out=out)
    for t in got.values():
        t.fill_(1)
    for call in calls:
        call()
    torch.cuda.synchronize()
    for n, t in want.items():
        assert torch.equal(got[n], t), n
