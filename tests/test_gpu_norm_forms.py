"""Layer norm and its backward pass in every form of their kernels: two rows per load of
the weight at every number of pieces per lane, several turns of a workgroup, runs of several
rows.  Which form a size takes is asserted by the launch rule's own arithmetic.

The bounds are block_reference's.  Its sums over tokens count T / 256 + 64 additions.  The
longest way here is a part's rows, one after the other, then at most 16 groups or 4 waves
and 16 + 16 steps of the join: norm_grad_adds says how many, and that it is within them."""
import numpy as np
import pytest
import torch

import combine_ep_layout_09_amd as ep
from tests import block_reference as ref
from tests.test_gpu_norm import DEV, TYPES, Case, f64

pytestmark = pytest.mark.gpu


def cdiv(a, b):
    return -(-a // b)


def pieces_of(H, xt):
    return cdiv(H, 8 if xt == "bf16" else 4)


def norm_form(T, H, xt):
    """(lanes of a row, pieces of a lane, rows of a load of the weight) of the forward kernel."""
    pieces, L = pieces_of(H, xt), 64
    while L < 1024 and pieces > 8 * L:
        L *= 2
    while L < 1024 and L < pieces and T * (L // 64) < 2048:
        L *= 2
    return L, cdiv(pieces, L), 2 if T >= 4096 and pieces <= 8 * L else 1


def parts_of(T, H):
    return min(256, (1 << 21) // H, T)


def grad_form(T, H, xt):
    """(kernel, rows that a part's longest chain adds, parts): the kernel that reads rows once with V
    pieces per lane ("V1", "V2"), or the one for long rows ("long")."""
    pieces, most = pieces_of(H, xt), parts_of(T, H)
    if pieces <= 2048:
        V, B = (1, 2) if pieces <= 1024 else (2, 1)
        L = cdiv(cdiv(pieces, V), 64) * 64
        groups = 1024 // L
        turns = cdiv(T, groups * B)
        n = 1 if turns <= 2 else cdiv(turns, cdiv(turns, most))
        return f"V{V}", cdiv(turns, n) * B, n
    run = cdiv(T, most)
    return "long", cdiv(run, 4), cdiv(T, run)


def norm_grad_adds(T, H, xt):
    _, rows, parts = grad_form(T, H, xt)
    adds = rows + 16 + cdiv(parts, 16) + 16
    assert adds <= T / 256 + 64
    return adds


# Forward, two rows per load.  At 64 lanes a row every number of pieces, odd lengths among them;
# more lanes where a row has more than 512 pieces.
@pytest.mark.parametrize("xt", ["bf16", "fp32"])
@pytest.mark.parametrize("per", range(1, 9))
def test_two_rows_per_load(per, xt):
    T, P = 4097 + 2 * per, 8 if xt == "bf16" else 4
    H = 64 * P * per - (0 if per % 4 == 0 else 2 * per + 1)
    assert norm_form(T, H, xt) == (64, per, 2)
    Case(T, H, xt, "fp32" if per % 2 else "bf16").check_forward()


@pytest.mark.parametrize("T,H,xt,form", [
    (4097, 7168, "bf16", (128, 7, 2)), (4096, 4097, "bf16", (128, 5, 2)), (4100, 4096, "fp32", (128, 8, 2)),
    (4099, 2052, "fp32", (128, 5, 2)),
])
def test_two_rows_per_load_of_wide_rows(T, H, xt, form):
    assert norm_form(T, H, xt) == form
    Case(T, H, xt, "fp32").check_forward()


@pytest.mark.parametrize("T,H,xt,form", [
    (4097, 8200, "bf16", (256, 5, 2)), (4097, 16391, "bf16", (512, 5, 2)), (4097, 40001, "bf16", (1024, 5, 2)),
    (4097, 65536, "bf16", (1024, 8, 2)), (4097, 16385, "fp32", (1024, 5, 2)), (4097, 32768, "fp32", (1024, 8, 2)),
    (4097, 40000, "fp32", (1024, 10, 1)), (4097, 65535, "fp32", (1024, 16, 1)),
])
def test_many_rows_of_every_width(T, H, xt, form):
    """Rows from everywhere against the 64-bit form; the others by equality: a row is the
    same wherever it stands."""
    assert norm_form(T, H, xt) == form
    print(f"[gpu] layer norm T {T} H {H} {xt}", flush=True)
    few = 61
    r = np.random.default_rng(H)
    a = torch.from_numpy(r.standard_normal((few, H)) * (0.2 + 3 * r.random(H))).to(TYPES[xt]).to(DEV)
    x = a[torch.arange(T, device=DEV) % few].contiguous()
    w, b = (torch.from_numpy(v.astype(np.float32)).to(DEV)
            for v in (1 + 0.5 * r.standard_normal(H), r.standard_normal(H)))
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    ep.ep_layer_norm(ep.Norm(T, H), x, w, b, y, mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    eps = float(np.float32(1e-5))
    want = ref.norm(f64(a), f64(w), f64(b), eps)
    bounds = ref.norm_bounds(f64(a), f64(w), f64(b), eps, xt)
    for name, g, v, e in zip(("y", "mean", "rstd"), (y, mean, rstd), want, bounds):
        off = np.abs(f64(g[:few]) - v)
        assert (off <= e).all(), (name, np.argwhere(~(off <= e))[:4], off.max(), e.min())
        for t in range(few, T, few):
            part = g[t:t + few]
            assert torch.equal(part, g[:len(part)]), (name, t)


# Backward: sizes that give every workgroup several turns, the last ones fewer; one, two and
# more groups of lanes; runs of long rows, the last one shorter.
@pytest.mark.parametrize("T,H,xt,form", [
    (701, 12288, "bf16", ("V2", 5, 141)), (701, 16384, "bf16", ("V2", 6, 117)),
    (650, 8201, "bf16", ("V2", 3, 217)), (901, 16381, "bf16", ("V2", 8, 113)),
    (1000, 8192, "fp32", ("V2", 4, 250)), (777, 4097, "fp32", ("V2", 4, 195)),
    (1500, 8192, "bf16", ("V1", 6, 250)), (1601, 4095, "bf16", ("V1", 4, 201)),
    (1603, 2049, "bf16", ("V1", 4, 134)), (2049, 4096, "fp32", ("V1", 10, 205)),
])
def test_several_turns(T, H, xt, form):
    assert grad_form(T, H, xt) == form
    norm_grad_adds(T, H, xt)
    c = Case(T, H, xt, "fp32" if T % 2 else "bf16")
    c.check_backward(skip=H % 2 == 0)


@pytest.mark.parametrize("T,H,xt,form", [
    (301, 20001, "bf16", ("long", 1, 101)), (301, 32776, "bf16", ("long", 2, 61)),
    (301, 65536, "bf16", ("long", 3, 31)), (701, 12288, "fp32", ("long", 2, 141)),
    (301, 32777, "fp32", ("long", 2, 61)), (203, 65535, "fp32", ("long", 2, 29)),
])
def test_runs_of_several_long_rows(T, H, xt, form):
    assert grad_form(T, H, xt) == form
    norm_grad_adds(T, H, xt)
    c = Case(T, H, xt, "bf16" if T % 4 == 1 else "fp32")
    c.check_backward(skip=H % 2 == 1)


@pytest.mark.parametrize("T,H", [(701, 12288), (650, 8201), (301, 20001)])
def test_equal_bits_with_and_without_the_parameters(T, H):
    """The rows' gradient does not depend on what else is asked for, nor on the call."""
    c = Case(T, H, "bf16", "fp32")
    dx, dw, db = c.backward()
    again = c.backward(stats=c.stats)
    only, _, _ = c.backward(params=False, stats=c.stats)
    for a, b in zip((dx, dw, db), again):
        assert torch.equal(a, b)
    assert torch.equal(dx, only)
