"""Calls with more workgroups than one dimension of a grid holds (2^20), and rows too long for
a lane's two pieces where the products quantise them."""
import numpy as np
import pytest
import torch

import combine_ep_layout_09_amd as ep
from tests import block_reference as ref
from tests.test_gpu_i8_forms import codes, exact_bits, form, make_layout, quant

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def f64(t):
    return t.double().cpu().numpy()


def repeated(rows, T):
    return rows[torch.arange(T, device=DEV) % len(rows)]


def assert_repeats(t, few):
    """Every row equals the one `few` rows before."""
    for a in range(0, len(t) - few, 1 << 20):
        b = min(len(t) - few, a + (1 << 20))
        assert torch.equal(t[a:b], t[a + few:b + few]), a


@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
def test_layer_norm_of_more_rows_than_a_grid_dimension(xt):
    """Eight rows a workgroup: 2^23 rows and some, the last workgroup not full."""
    T, H, few = (1 << 23) + 11, 9, 997
    print(f"[gpu] norm T {T} H {H} {xt}", flush=True)
    r = np.random.default_rng(0)
    base = torch.from_numpy(r.standard_normal((few, H))).to(xt).to(DEV)
    w, b = (torch.from_numpy(r.standard_normal(H).astype(np.float32)).to(DEV) for _ in range(2))
    x = repeated(base, T)
    y = torch.full((T, H), 7.0, dtype=xt, device=DEV)
    mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    ep.ep_layer_norm(ep.Norm(T, H), x, w, b, y, mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    name = "bf16" if xt is torch.bfloat16 else "fp32"
    eps = float(np.float32(1e-5))
    want = ref.norm(f64(base), f64(w), f64(b), eps)
    for g, v, e in zip((y, mean, rstd), want, ref.norm_bounds(f64(base), f64(w), f64(b), eps, name)):
        assert (np.abs(f64(g[:few]) - v) <= e).all()
        assert_repeats(g, few)


def test_gradient_of_more_long_rows_than_a_grid_dimension():
    """A workgroup per row: 2^20 rows and some of 16392 channels, 34 GB; one set of rows is x
    and dy."""
    T, H, few = (1 << 20) + 5, 16392, 61
    print(f"[gpu] norm gradient T {T} H {H}", flush=True)
    r = np.random.default_rng(1)
    base = torch.from_numpy(r.standard_normal((few, H))).to(torch.bfloat16).to(DEV)
    w = torch.from_numpy(r.standard_normal(H).astype(np.float32)).to(DEV)
    x = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    for a in range(0, T, few * 4096):
        part = x[a:a + few * 4096]
        part.copy_(repeated(base, len(part)))
    _, m, s = ref.norm(f64(base), np.ones(H), np.zeros(H), 1e-5)
    m, s = (torch.from_numpy(v.astype(np.float32)).to(DEV) for v in (m, s))
    dx = torch.full((T, H), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_layer_norm_backward(ep.Norm(T, H), x, x, w, repeated(m, T), repeated(s, T), dx)
    torch.cuda.synchronize()
    args = (f64(base), f64(base), f64(w), f64(m), f64(s), None)
    want, _, _ = ref.norm_grad(*args)
    bound, _, _ = ref.norm_grad_bounds(*args, "bf16", "fp32")
    assert (np.abs(f64(dx[:few]) - want) <= bound).all()
    for a in range(0, T - few, 1 << 16):
        b = min(T - few, a + (1 << 16))
        assert torch.equal(dx[a:b], dx[a + few:b + few]), a


@pytest.mark.parametrize("T", [(1 << 20) + 77])
def test_products_of_more_bf16_rows_than_a_grid_dimension(T):
    """Rows quantised in the call, a workgroup for each of the first 2^20."""
    K, N, E = 32, 24, 3
    prob, mm = ep.Problem(T, 128, 1, E), ep.ExpertI8(K, N, 0)
    print(f"[gpu] {prob!r} {mm!r}", flush=True)
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    counts = [T // 2, 0, T - T // 2]
    i32 = dict(dtype=torch.int32, device=DEV)
    lay = ep.Layout(torch.tensor(counts, **i32), torch.tensor([0, T // 2, T // 2, T], **i32), None, None, None)
    x = (torch.randn((T, K), generator=g, device=DEV) * 40).bfloat16()
    w = codes((E, N, K), g)
    scale = torch.rand((E, N), generator=g, device=DEV) / 500
    space = torch.empty(ep.ep_expert_i8_workspace_bytes(prob, mm), dtype=torch.uint8, device=DEV)
    out = torch.full((T, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_i8(prob, mm, x, lay, w, scale, out, workspace=space)
    torch.cuda.synchronize()
    for e, (a, b) in enumerate(((0, T // 2), (0, 0), (T // 2, T))):
        if a < b:
            assert torch.equal(out[a:b], exact_bits(*quant(x[a:b]), w[e], scale[e])), e


def test_products_of_more_tiles_than_a_grid_dimension():
    """2^20 and more (row tile, output block) items: 1024 experts of 256 rows, 65536 gated
    outputs, 34 GB."""
    E, n, K, N = 1024, 256, 16, 65536
    T = E * n
    prob, mm = ep.Problem(T, 128, 1, E), ep.ExpertI8(K, N, 1, 1)
    print(f"[gpu] {prob!r} {mm!r}", flush=True)
    assert form(prob, mm) == 256 and (E + T // 256) * (2 * N // 256) >= 1 << 20
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    i32 = dict(dtype=torch.int32, device=DEV)
    lay = ep.Layout(torch.full((E,), n, **i32), torch.arange(E + 1, **i32) * n, None, None, None)
    q, w = codes((T, K), g), codes((E, 2 * N, K), g)
    rs = 0.5 + torch.rand(T, generator=g, device=DEV)
    scale = (0.5 + torch.rand((E, 2 * N), generator=g, device=DEV)) / 20000
    out = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_i8(prob, mm, q, lay, w, scale, out, row_scales=rs)
    torch.cuda.synchronize()
    for e in range(0, E, 16):
        assert torch.isfinite(out[e * n:(e + 16) * n]).all(), e
    # an expert by itself, whatever kernel takes it
    one, one_lay = ep.Problem(n, 128, 1, 1), make_layout(np.zeros((n, 1), np.int32), 1, 0)[1]
    for e in (0, 1, 127, 128, 511, 512, 770, 1022, 1023):
        want = torch.empty((n, N), dtype=torch.bfloat16, device=DEV)
        ep.ep_expert_i8(one, mm, q[e * n:(e + 1) * n].contiguous(), one_lay, w[e:e + 1].contiguous(),
                        scale[e:e + 1].contiguous(), want, row_scales=rs[e * n:(e + 1) * n].contiguous())
        assert torch.equal(out[e * n:(e + 1) * n], want), e


@pytest.mark.parametrize("cap", [0, 9])
@pytest.mark.parametrize("K", [16368, 16384, 16400, 32784, 65536])
def test_long_bf16_rows(K, cap):
    """Rows of one, two and up to eight pieces per lane, quantised in the call."""
    E, T, N = 3, 30, 40
    idx = np.random.default_rng(K).integers(0, E, (T, 1)).astype(np.int32)
    r, lay = make_layout(idx, E, cap)
    prob, mm = ep.Problem(T, 128, 1, E, cap), ep.ExpertI8(K, N, 0)
    print(f"[gpu] {prob!r} {mm!r}", flush=True)
    R = ep.ep_num_recv_rows(prob)
    g = torch.Generator(device=DEV)
    g.manual_seed(K)
    x = (torch.randn((R, K), generator=g, device=DEV) * 40).bfloat16()
    w = codes((E, N, K), g)
    scale = torch.rand((E, N), generator=g, device=DEV) / (500 * K ** 0.5)
    space = torch.empty(ep.ep_expert_i8_workspace_bytes(prob, mm), dtype=torch.uint8, device=DEV)
    out = torch.full((R, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_i8(prob, mm, x, lay, w, scale, out, workspace=space)
    torch.cuda.synchronize()
    for e in range(E):
        n = int(r["count"][e])
        a, n = (e * cap, min(n, cap)) if cap else (int(r["offset"][e]), n)
        assert torch.equal(out[a:a + n], exact_bits(*quant(x[a:a + n]), w[e], scale[e])), e
        if cap:
            assert (out[a + n:a + cap] == 7).all()
