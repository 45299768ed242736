"""ep_combine_dropout and ep_combine_backward in every form of their kernels: the persistent
one (exact and any k, one launch and several) with dropout and the skip connection, the
per-token one at every batch of entries, and the gradient's with one and two pieces per lane.
Which form a size takes is asserted by the launch rule's own arithmetic.  The bounds are
block_reference's; the 64-bit forms run on the GPU."""
import numpy as np
import pytest
import torch

import combine_ep_layout_09_amd as ep
from tests import block_reference as ref
from tests.test_gpu_dropout import Case, uniform

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def cdiv(a, b):
    return -(-a // b)


def launches(T, H, k):
    """Launches of the persistent form, 0 where the per-token form is taken."""
    waves = torch.cuda.get_device_properties(0).multi_processor_count * 16
    C = cdiv(H // 8, 64)
    n = cdiv(T * C, waves * 16)
    while cdiv(cdiv(T, n) * C, waves) > 16:
        n += 1
    return n if T * C >= waves and n <= 16 and T * C * k >= waves * 36 else 0


def grad_pieces(T, H, k):
    return 2 if H // 8 > 1024 or (T < 2048 and H // 8 > 128 and k >= 5) else 1


def check(c):
    """Forward and backward of a Case against the 64-bit forms."""
    keep = torch.from_numpy(c.keep()).to(DEV)
    slot = torch.from_numpy(c.slot.astype(np.int64)).to(DEV)
    f, U = 1 / (1 - c.p), ref.U
    w, dy = c.w.double(), c.dy.double()
    s, mag = torch.zeros_like(dy), torch.zeros_like(dy)
    g = torch.where(keep, dy * f, 0.0)
    y = c.forward()
    deo, dw = c.backward()
    assert (deo.view(torch.int16)[~c.used.to(DEV)] == 0x5A5A).all(), "unused rows were written"
    for j in range(c.k):
        there = slot[:, j] >= 0
        at = slot[:, j].clamp(min=0)
        eo = torch.where(there[:, None], c.eo[at].double(), 0.0)
        v = w[:, j:j + 1] * eo
        s += v
        mag += v.abs()
        want, size = (g * eo).sum(1), (g * eo).abs().sum(1)
        off = (dw[:, j].double() - want).abs()
        assert (off <= (ref.DOT_ADDS + 3) * U * size + 2.0 ** -140).all(), (j, off.max())
        d = (w[:, j:j + 1] * g)[there]
        off = (deo[at[there]].double() - d).abs()
        assert (off <= (4 * U + 2.0 ** -8) * d.abs() + 2.0 ** -133).all(), (j, off.max())
    want = torch.where(keep, s * f, 0.0)
    bound = torch.where(keep, (c.k + 3) * U * mag * f, 0.0)
    if c.res is not None:
        want = want + c.res.double()
    off = (y.double() - want).abs()
    bad = ~(off <= bound + (2 * U + 2.0 ** -8) * want.abs() + 2.0 ** -133)
    assert not bad.any(), (bad.nonzero()[:4], off.max())


PERSISTENT = [  # T, E, k, cap, H, launches
    (147501, 32, 1, 0, 72, 3), (25003, 16, 2, 0, 1032, 2), (3601, 64, 3, 0, 7168, 1), (4201, 16, 4, 1000, 4104, 1),
    (7501, 16, 5, 0, 2048, 1), (1801, 32, 6, 0, 7168, 1), (11003, 24, 7, 3000, 520, 1),
    (601, 16, 8, 0, 16392, 1), (66001, 64, 8, 0, 72, 2), (1401, 64, 8, 0, 7168, 1), (1201, 32, 9, 0, 7168, 1), (6201, 64, 12, 900, 520, 1),
    (1601, 64, 32, 0, 1288, 1),
]


@pytest.mark.parametrize("shape", PERSISTENT, ids=lambda s: "-".join(map(str, s)))
def test_persistent_form(shape):
    T, E, k, cap, H, n = shape
    assert launches(T, H, k) == n
    idx = uniform(T, E, k, seed=T)
    idx[5] = -1
    idx[T // 2:T // 2 + 40, 0] = E  # names no expert
    check(Case(idx, E, cap, H, 0.1 if k != 4 else 0.5, residual=k != 3))


@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 6, 7, 8, 11])
def test_per_token_form_with_two_pieces_per_lane(k):
    T, H = 701, 520
    assert launches(T, H, k) == 0
    check(Case(uniform(T, 16, k, seed=k), 16, 0, H, 0.2, residual=k % 2 == 0))


# the gradient: one piece per lane at every batch of entries and more entries than a batch, two
# pieces per lane likewise
@pytest.mark.parametrize("T,H,pieces", [(2049, 1032, 1), (150, 1024, 1), (150, 1288, 2), (150, 9000, 2)])
@pytest.mark.parametrize("k", [5, 6, 7, 8, 9, 17, 32])
def test_gradient_forms(T, H, pieces, k):
    assert grad_pieces(T, H, k) == pieces
    check(Case(uniform(T, 40, k, seed=k), 40, T * k // 40 if k % 2 else 0, H, 0.25))


@pytest.mark.parametrize("p", [0.1, 0.999])
def test_mask_of_the_persistent_form_to_the_bit(p):
    """A sum of 1: what comes out is the factor or 0, by the generator's words, in each of
    several launches."""
    T, H, k = 147501, 72, 1
    assert launches(T, H, k) == 3
    c = Case(uniform(T, 8, k), 8, 0, H, p, residual=False)
    c.eo.fill_(1.0)
    c.w.fill_(1.0)
    keep = torch.from_numpy(c.keep()).to(DEV)
    f = torch.tensor(1 / (1 - p), dtype=torch.float64).float().bfloat16().to(DEV)
    assert torch.equal(c.forward(), torch.where(keep, f, torch.zeros_like(f)))


def test_persistent_form_captured_with_another_offset():
    """Several launches in a graph, beside eager calls."""
    c = Case(uniform(66001, 64, 8), 64, 0, 72, 0.3)
    assert launches(c.T, c.H, c.k) == 2
    y = torch.empty_like(c.dy)

    def call(out):
        ep.ep_combine_dropout(c.prob, c.eo, c.lay, c.w, c.p, c.rng, out, residual=c.res)

    call(y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(y)
    last = None
    for i in range(3):
        c.rng[1] += 1
        want = torch.empty_like(y)
        call(want)
        y.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
        assert last is None or not torch.equal(last, want)
        last = want
