"""ep_balance_loss where a workgroup takes several passes over its tokens.

A mean probability passes, after its token's own roundings (test_gpu_routing's
bound), at most 32 fp32 additions in a lane, 6 across lanes and 16 over the
waves; the rest is fp64 and one rounding.  That count does not grow with the
number of tokens, and neither do the tolerances: LONG units of 2^-24.
"""
import numpy as np
import pytest
import torch

import combine_ep_layout_09_amd as ep
from tests import routing_reference as ref
from tests.test_gpu_routing import Case, U, bound

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
LONG = 32 + 6 + 16 + 2


def check(c, idx):
    """Against the reference; the loss adds its terms in fp64."""
    o = c.balance(idx)
    cnt, mean, n, loss = ref.balance(c.x, idx.cpu().numpy(), c.score, 0.25, c.B, c.valid)
    np.testing.assert_array_equal(o["counts"].cpu().numpy(), cnt)
    np.testing.assert_array_equal(o["num_valid"].cpu().numpy(), n)
    tol = bound(c.x) + LONG * U
    got = o["mean_prob"].cpu().numpy().astype(np.float64)
    assert (np.abs(got - mean) <= tol * mean + 2.0 ** -126).all(), np.abs(got - mean).max()
    assert abs(float(o["loss"]) - loss) <= tol * abs(loss)


def random_ids(c):
    return torch.from_numpy(c.r.integers(-1, c.E + 1, (c.T, c.k)).astype(np.int32)).to(DEV)


@pytest.mark.parametrize("T,E,B,pad", [
    (16385, 64, 1, 0.0),    # just above one pass: uneven runs, most of a last pass empty
    (16387, 200, 1, 0.2), (49155, 60, 3, 0.1), (50000, 64, 1, 0.3),
    (4097, 300, 1, 0.1), (9000, 300, 3, 0.0), (9001, 1024, 1, 0.2), (8196, 512, 2, 0.1)])
@pytest.mark.parametrize("score,bf16", [(0, True), (1, False)])
def test_several_passes(T, E, B, pad, score, bf16):
    c = Case(T, E, 3, score=score, bf16=bf16, B=B, pad=pad)
    check(c, random_ids(c))


def test_sequences_without_valid_tokens_in_several_passes():
    c = Case(60000, 32, 2, B=2, pad=0.5)
    c.valid[:30000] = 0
    c.valid[40000:45000] = 0
    c.d_valid = torch.from_numpy(c.valid).to(DEV)
    check(c, random_ids(c))


@pytest.mark.parametrize("B,T", [(512, 2048), (600, 3000), (2048, 2048)])
def test_many_short_sequences(B, T):
    """More outputs than one workgroup takes, one row of partial sums each."""
    c = Case(T, 64, 3, B=B, pad=0.2)
    check(c, random_ids(c))


@pytest.mark.parametrize("B,cycle", [(1, 1), (1, 7), (2, 1)])
def test_the_longest_batch(B, cycle):
    """2^25 tokens of `cycle` different rows: their mean probabilities are known
    in closed form."""
    T, E, k = 1 << 25, 17, 1
    rt = ep.Routing(T, E, k, num_seqs=B)
    print(f"[gpu] {rt!r} cycle={cycle}", flush=True)
    base = np.random.default_rng(cycle).standard_normal((cycle, E)).astype(np.float32)
    if cycle == 1:
        base[:] = 0.5
    rows = torch.from_numpy(base).to(torch.bfloat16)
    p = ref.probs(rows.float().numpy(), 0)
    logits = rows.to(DEV).repeat(-(-T // cycle), 1)[:T]
    idx = (torch.arange(T, device=DEV, dtype=torch.int32) % 5).view(T, 1)
    o = dict(counts=torch.empty((B, E), dtype=torch.int32, device=DEV),
             mean_prob=torch.empty((B, E), device=DEV),
             num_valid=torch.empty(B, dtype=torch.int32, device=DEV),
             loss=torch.empty(1, device=DEV))
    space = torch.empty(ep.ep_balance_workspace_bytes(rt), dtype=torch.uint8, device=DEV)
    ep.ep_balance_loss(rt, logits, idx, 1.0, workspace=space, **o)
    torch.cuda.synchronize()
    L = T // B
    tol = (bound(rows.float().numpy()) if cycle > 1 else 4 * U) + LONG * U
    total = 0.0
    for s in range(B):
        t0 = s * L
        of = lambda m, j: (t0 + L - j + m - 1) // m - (t0 - j + m - 1) // m  # noqa: E731
        cnt = np.array([of(5, e) if e < 5 else 0 for e in range(E)])
        mean = sum(of(cycle, j) * p[j] for j in range(cycle)) / L
        np.testing.assert_array_equal(o["counts"][s].cpu().numpy(), cnt)
        assert int(o["num_valid"][s]) == L
        got = o["mean_prob"][s].cpu().numpy().astype(np.float64)
        assert (np.abs(got - mean) <= tol * mean).all(), np.abs(got / mean - 1).max() / U
        total += float((cnt * mean).sum()) * E / (k * L)
    assert abs(float(o["loss"]) - total / B) <= tol * total / B
