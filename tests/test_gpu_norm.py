"""ep_layer_norm and its backward pass against the 64-bit forms; the tolerances
count roundings (block_reference)."""
import numpy as np
import pytest
import torch

import combine_ep_layout_09_amd as ep
from tests import block_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SENTINEL = 0x5A


def f64(t):
    return t.double().cpu().numpy()


def pitched(a, dtype, pitch, first=0):
    """`a` as a [T, H] view of rows `pitch` elements apart, starting at element
    `first` of its memory; what lies between rows is NaN."""
    T, H = a.shape
    room = torch.full((first + max(T, 1) * pitch,), float("nan"), dtype=dtype, device=DEV)
    v = room[first:].view(-1, pitch)[:T, :H]
    v.copy_(torch.from_numpy(a))
    return v


def guarded(shape, dtype, first=0):
    """A tensor of sentinel bytes with more of them on both sides."""
    n = int(np.prod(shape))
    room = torch.empty(first + n + 64, dtype=dtype, device=DEV)
    room.view(torch.uint8).fill_(SENTINEL)
    return room, room[first:first + n].view(shape)


def untouched(room, first, n):
    b, size = room.view(torch.uint8), room.element_size()
    return bool((b[:first * size] == SENTINEL).all()) and bool((b[(first + n) * size:] == SENTINEL).all())


class Case:
    def __init__(self, T, H, xt, wt, seed=0, offset=0.0, pitch=None, first=0, eps=1e-5, params=True):
        r = np.random.default_rng(seed + 31 * T + H)
        print(f"[gpu] layer norm T {T} H {H} {xt} {wt} pitch {pitch} first {first}", flush=True)
        self.T, self.H, self.xt, self.wt, self.eps, self.first = T, H, xt, wt, eps, first
        self.nm = ep.Norm(T, H, eps)
        self.eps = float(np.float32(eps))
        pitch = pitch or H
        a = r.standard_normal((T, H)) * (0.2 + 3 * r.random(H)) + offset
        self.x = pitched(a, TYPES[xt], pitch, first)
        self.dy = pitched(r.standard_normal((T, H)), TYPES[xt], pitch + (pitch != H), first)
        self.w = self.b = None
        if params:
            self.w = pitched(1 + 0.5 * r.standard_normal((1, H)), TYPES[wt], H, first)[0]
            self.b = pitched(r.standard_normal((1, H)), TYPES[wt], H, first)[0]
        self.skip = pitched(r.standard_normal((T, H)), TYPES[xt], H, first)
        one, zero = np.ones(H), np.zeros(H)
        self.xn, self.dyn, self.skipn = f64(self.x), f64(self.dy), f64(self.skip)
        self.wn, self.bn = (f64(self.w), f64(self.b)) if params else (one, zero)

    def forward(self, stream=None):
        room, y = guarded((self.T, self.H), TYPES[self.xt], self.first)
        mean = torch.empty(self.T, device=DEV)
        rstd = torch.empty(self.T, device=DEV)
        ep.ep_layer_norm(self.nm, self.x, self.w, self.b, y, mean=mean, rstd=rstd, stream=stream)
        torch.cuda.synchronize()
        assert untouched(room, self.first, y.numel()), "written outside the rows"
        return y, mean, rstd

    def check_forward(self):
        got = self.forward()
        want = ref.norm(self.xn, self.wn, self.bn, self.eps)
        bounds = ref.norm_bounds(self.xn, self.wn, self.bn, self.eps, self.xt)
        for name, g, w, e in zip(("y", "mean", "rstd"), got, want, bounds):
            off = np.abs(f64(g) - w)
            assert (off <= e).all(), (name, np.argwhere(~(off <= e))[:4], off.max(), e.min())

    def backward(self, skip=True, params=True, stats=None):
        if stats is None:
            _, m, r = ref.norm(self.xn, self.wn, self.bn, self.eps)
            stats = [torch.from_numpy(v.astype(np.float32)).to(DEV) for v in (m, r)]
        self.stats = stats
        room, dx = guarded((self.T, self.H), TYPES[self.xt], self.first)
        rw, dw = guarded((self.H,), TYPES[self.wt], self.first)
        rb, db = guarded((self.H,), TYPES[self.wt], self.first)
        ws = torch.full((ep.ep_layer_norm_workspace_bytes(self.nm) + 64,), 0xFF, dtype=torch.uint8,
                        device=DEV)
        ep.ep_layer_norm_backward(self.nm, self.x, self.dy, self.w, *stats, dx,
                                  d_weight=dw if params else None, d_bias=db if params else None,
                                  workspace=ws[:-64] if params else None,
                                  d_skip=self.skip if skip else None)
        torch.cuda.synchronize()
        assert (ws[-64:] == 0xFF).all(), "written behind the workspace"
        for r, t in ((room, dx), (rw, dw), (rb, db)):
            assert untouched(r, self.first, t.numel()), "written outside an output"
        return dx, dw, db

    def check_backward(self, skip=True):
        got = self.backward(skip)
        m, r = (f64(v) for v in self.stats)
        args = (self.xn, self.dyn, self.wn, m, r, self.skipn if skip else None)
        want = ref.norm_grad(*args)
        bounds = ref.norm_grad_bounds(*args, self.xt, self.wt)
        for name, g, w, e in zip(("dx", "dw", "db"), got, want, bounds):
            off = np.abs(f64(g) - w)
            assert (off <= e).all(), (name, np.argwhere(~(off <= e))[:4], off.max(), e.min())


SIZES = [(1, 1), (3, 2), (1, 7168), (5, 8), (2, 9), (7, 64), (4, 511), (9, 512), (3, 513), (6, 1023),
         (130, 1409), (33, 2048), (17, 4096), (3, 4097), (5, 7168), (70, 100), (2, 8192), (2, 8200),
         (3, 12288), (2, 16384), (1, 20001), (2, 32776), (1, 65536), (2, 65535), (300, 40)]


@pytest.mark.parametrize("xt", ["bf16", "fp32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: f"{s[0]}x{s[1]}")
def test_sizes(size, xt):
    c = Case(*size, xt, "fp32" if size[0] % 2 else "bf16")
    c.check_forward()
    c.check_backward(skip=size[1] % 2 == 0)


@pytest.mark.parametrize("xt,wt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "bf16"),
                                   ("fp32", "fp32")])
@pytest.mark.parametrize("H,pitch,first", [(129, 131, 1), (512, 520, 0), (512, 515, 3), (1000, 1000, 1),
                                           (7, 9, 5)])
def test_types_pitches_and_alignments(xt, wt, H, pitch, first):
    c = Case(37, H, xt, wt, pitch=pitch, first=first)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("T,H", [(2000, 512), (1031, 7168), (4096, 136), (700, 2560), (5000, 33)])
def test_many_rows(T, H):
    c = Case(T, H, "bf16", "fp32")
    c.check_forward()
    c.check_backward()
    c = Case(T, min(H, 1000), "fp32", "fp32", pitch=1024)
    c.check_forward()
    c.check_backward(skip=False)


def test_without_parameters_and_optional_outputs():
    c = Case(19, 264, "bf16", "fp32", params=False)
    c.check_forward()
    c.check_backward()
    y, _, _ = c.forward()
    z = torch.empty_like(y)
    ep.ep_layer_norm(c.nm, c.x, None, None, z)
    dx, dw, db = c.backward()
    only, _, _ = c.backward(params=False)
    dw2 = torch.empty_like(dw)
    ws = torch.empty(ep.ep_layer_norm_workspace_bytes(c.nm), dtype=torch.uint8, device=DEV)
    dx2 = torch.empty_like(dx)
    ep.ep_layer_norm_backward(c.nm, c.x, c.dy, None, *c.stats, dx2, d_weight=dw2, workspace=ws,
                              d_skip=c.skip)
    torch.cuda.synchronize()
    assert torch.equal(y, z) and torch.equal(dx, only) and torch.equal(dx, dx2)
    assert torch.equal(dw, dw2)


@pytest.mark.parametrize("xt", ["bf16", "fp32"])
def test_far_from_zero_and_constant_rows(xt):
    """A mean far above the spread; rows of one value, whose variance is zero."""
    Case(11, 768, xt, "fp32", offset=200.0).check_forward()
    c = Case(5, 300, xt, "fp32")
    c.x[2] = 3.0
    c.xn = f64(c.x)
    y, mean, rstd = c.forward()
    assert float(mean[2]) == 3.0 and abs(float(rstd[2]) * np.sqrt(c.eps) - 1) < 1e-6
    off = np.abs(f64(y)[2] - c.bn)
    assert (off <= ref.half_step(xt) * np.abs(c.bn)).all()


def test_rows_that_are_not_finite_stay_by_themselves():
    c = Case(9, 520, "bf16", "fp32")
    y0, m0, r0 = c.forward()
    c.x[3, 7] = float("nan")
    c.x[5, 519] = float("inf")
    y, m, r = c.forward()
    fine = [0, 1, 2, 4, 6, 7, 8]
    assert torch.equal(y[fine], y0[fine]) and torch.equal(m[fine], m0[fine]) and torch.equal(r[fine], r0[fine])
    assert torch.isnan(y[3]).all() and torch.isnan(y[5]).all()


@pytest.mark.parametrize("T,H", [(1, 7168), (2, 7168), (4, 7168), (16, 1024)])
def test_few_rows_without_the_parameters_gradients(T, H):
    """The rows' gradient is the same with and without the sums over tokens."""
    print(f"[gpu] {T} x {H}", flush=True)
    r = np.random.default_rng(T)
    x, dy = (torch.from_numpy(r.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).to(DEV)
             for _ in range(2))
    w = torch.from_numpy(r.standard_normal(H).astype(np.float32)).to(DEV)
    nm = ep.Norm(T, H)
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    ep.ep_layer_norm(nm, x, w, None, y, mean, rstd)
    dx, only = torch.empty_like(x), torch.empty_like(x)
    space = torch.empty(ep.ep_layer_norm_workspace_bytes(nm), dtype=torch.uint8, device=DEV)
    ep.ep_layer_norm_backward(nm, x, dy, w, mean, rstd, dx, torch.empty_like(w),
                              torch.empty_like(w), space)
    ep.ep_layer_norm_backward(nm, x, dy, w, mean, rstd, only)
    assert torch.equal(dx, only)


def test_no_tokens():
    nm = ep.Norm(0, 48)
    x = torch.empty((0, 48), dtype=torch.bfloat16, device=DEV)
    f = torch.empty(0, device=DEV)
    w = torch.ones(48, device=DEV)
    ep.ep_layer_norm(nm, x, w, w.clone(), x.clone(), mean=f, rstd=f.clone())
    dw, db = torch.full((48,), 7.0, device=DEV), torch.full((48,), 7.0, device=DEV)
    ws = torch.empty(ep.ep_layer_norm_workspace_bytes(nm) + 256, dtype=torch.uint8, device=DEV)
    ep.ep_layer_norm_backward(nm, x, x.clone(), w, f, f.clone(), x.clone(), d_weight=dw, d_bias=db,
                              workspace=ws)
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()


def test_equal_calls_give_equal_bits_on_every_stream():
    c = Case(513, 1032, "bf16", "fp32")
    first = c.forward() + c.backward()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = c.forward() + c.backward(stats=c.stats)
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_replayed_graph():
    """Forward and backward captured, replayed on new rows beside eager calls."""
    c = Case(300, 1288, "bf16", "fp32")
    T, H = c.T, c.H
    y, mean, rstd = torch.empty_like(c.x), torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    dx, dw, db = torch.empty_like(c.x), torch.empty(H, device=DEV), torch.empty(H, device=DEV)
    ws = torch.empty(ep.ep_layer_norm_workspace_bytes(c.nm), dtype=torch.uint8, device=DEV)

    def step(ws):
        ep.ep_layer_norm(c.nm, c.x, c.w, c.b, y, mean=mean, rstd=rstd)
        ep.ep_layer_norm_backward(c.nm, c.x, c.dy, c.w, mean, rstd, dx, d_weight=dw, d_bias=db,
                                  workspace=ws, d_skip=c.skip)

    step(ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(ws)
    other = torch.empty_like(ws)
    for i in range(4):
        c.x.copy_(torch.randn(T, H, device=DEV))
        c.dy.copy_(torch.randn(T, H, device=DEV))
        step(other)
        torch.cuda.synchronize()
        want = [v.clone() for v in (y, mean, rstd, dx, dw, db)]
        for v in (y, mean, rstd, dx, dw, db):
            v.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((y, mean, rstd, dx, dw, db), want):
            assert torch.equal(a, b), i


def test_rows_beyond_32_bit_offsets():
    """Rows whose pitch takes the last one past 2^32 bytes and 2^31 elements."""
    T, H = 5, 520
    pitch = (1 << 29) + 8
    room = torch.empty(4 * pitch + H, dtype=torch.bfloat16, device=DEV)
    x = room.as_strided((T, H), (pitch, 1))
    x.copy_(torch.randn(T, H, device=DEV))
    w, b = torch.randn(H, device=DEV), torch.randn(H, device=DEV)
    dense = x.contiguous()
    nm = ep.Norm(T, H)
    outs = []
    for v in (x, dense):
        y, m, r = torch.empty_like(dense), torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        ep.ep_layer_norm(nm, v, w, b, y, mean=m, rstd=r)
        dx, dw, db = torch.empty_like(dense), torch.empty(H, device=DEV), torch.empty(H, device=DEV)
        ws = torch.empty(ep.ep_layer_norm_workspace_bytes(nm), dtype=torch.uint8, device=DEV)
        ep.ep_layer_norm_backward(nm, v, v, w, m, r, dx, d_weight=dw, d_bias=db, workspace=ws)
        outs.append((y, m, r, dx, dw, db))
    torch.cuda.synchronize()
    for a, c in zip(*outs):
        assert torch.equal(a, c)


def test_binding_refuses():
    T, H = 4, 64
    nm = ep.Norm(T, H)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    w, s = torch.ones(H, device=DEV), torch.ones(T, device=DEV)
    y = torch.empty_like(x)
    with pytest.raises(TypeError):
        ep.ep_layer_norm(nm, x.half(), w, w, y)
    with pytest.raises(TypeError):
        ep.ep_layer_norm(nm, x, w, w.bfloat16(), y)
    with pytest.raises(TypeError):
        ep.ep_layer_norm(nm, x, w, w, y.float())
    with pytest.raises(ValueError):
        ep.ep_layer_norm(nm, x[:, :32], w, w, y)
    with pytest.raises(ValueError):
        ep.ep_layer_norm(nm, torch.zeros((H, T), dtype=torch.bfloat16, device=DEV).t(), w, w, y)
    with pytest.raises(ValueError):
        ep.ep_layer_norm(nm, x[:1].expand(T, H), w, w, y)
    with pytest.raises(ep.EpError):
        ep.ep_layer_norm(nm, x, w, w, x)
    with pytest.raises(ep.EpError):
        ep.ep_layer_norm(nm, x, w, w, y, mean=s)
    with pytest.raises(ep.EpError):
        ep.ep_layer_norm_backward(nm, x, y, w, s, s, torch.empty_like(x), d_weight=torch.empty_like(w))
    with pytest.raises(TypeError):
        ep.ep_layer_norm_backward(nm, x, y.float(), w, s, s, torch.empty_like(x))
