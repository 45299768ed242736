"""The choice of experts by the scores of a sigmoid gate (choose_by_score).

The oracle's key is fp32(fp32(sigma(x)) + bias) with sigma in fp64, the choice
the plain one of those keys; weights and the calls after the choice are held to
the bounds of test_gpu_routing.  A key differs from the oracle's only where
sigma(x) lies within 2^-46 of a rounding border (about one value in 2^21), and
then by one unit, which changes a choice only if another key is that close.
"""
import ctypes

import numpy as np
import pytest
import torch

import combine_ep_layout_09_amd as ep
from tests import routing_reference as ref
from tests.test_gpu_routing import Case, _with_off, bound

DEV = "cuda:0"
F32 = np.float32


def sigma(x):
    """fp32 sigma(x), from fp64; NaN where x is not finite."""
    v = np.where(np.isfinite(x), x, 0.0).astype(np.float64)
    t = np.exp(-np.abs(v))
    return np.where(np.isfinite(x), np.where(v >= 0, 1.0, t) / (1.0 + t), np.nan).astype(F32)


def choose(x, k, G, KG, bias, valid):
    return ref.choose(sigma(x), k, G, KG, bias, valid)


class ByScore(Case):
    def __init__(self, *a, **kw):
        super().__init__(*a, score=1, **kw)
        self.rt.choose_by_score = 1
        print(f"[gpu] {self.rt!r}", flush=True)

    def check_route(self, idx, w):
        want = choose(self.x, self.k, self.G, self.KG, self.bias, self.valid)
        np.testing.assert_array_equal(idx.cpu().numpy(), want)
        ww = ref.weights(self.x, want, 1, self.norm, self.scale, self.valid)
        got = w.cpu().numpy().astype(np.float64)
        assert (np.abs(got - ww) <= bound(self.x) * np.abs(ww) + 2.0 ** -126).all()
        return want


@pytest.mark.gpu
@pytest.mark.parametrize("G,KG,bias", [(1, 1, True), (8, 4, True), (8, 4, False)])
def test_the_choice_of_a_sigmoid_gate(G, KG, bias):
    """A bias and group sums act on the scores: most tokens get other experts
    than by their logits."""
    c = ByScore(2048, 256, 8, G=G, KG=KG, bias=bias)
    want = c.check_route(*c.route())
    other = ref.choose(c.x, 8, G, KG, c.bias, None)
    differ = (np.sort(want, 1) != np.sort(other, 1)).any(1).mean()
    assert differ > (0.5 if bias else 0.05)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,G,KG", [
    (1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (3, 5, 5, 1, 1), (33, 17, 3, 1, 1), (65, 60, 6, 6, 2),
    (31, 96, 6, 4, 3), (40, 128, 32, 1, 1), (129, 256, 32, 64, 33), (19, 510, 31, 10, 1),
    (9, 512, 8, 2, 1), (12, 777, 32, 7, 3), (7, 1024, 32, 64, 64)])
@pytest.mark.parametrize("bf16", [False, True])
def test_shapes(T, E, k, G, KG, bf16):
    ByScore(T, E, k, G, KG, bf16=bf16, bias=True, norm=not bf16, scale=2.5).all()


@pytest.mark.gpu
def test_padding_sequences_and_pitches():
    ByScore(600, 64, 6, bias=True, pad=0.4, B=6).all()
    ByScore(96, 256, 8, G=8, KG=4, bias=True, pad=0.3, B=3, bf16=True, gap=3, offset=5).all()
    ByScore(37, 300, 8, bias=True, gap=64).all()


@pytest.mark.gpu
@pytest.mark.parametrize("E,G,KG", [(24, 1, 1), (24, 6, 2), (256, 8, 4), (700, 7, 3)])
def test_experts_switched_off(E, G, KG):
    """An infinite logit is off, though its sigmoid is finite."""
    x = _with_off(30, E, 5, [-np.inf, np.nan, np.inf])
    ByScore(30, E, 8, G=G, KG=KG, logits=x, bias=True).all()
    c = ByScore(30, E, 8, G=G, KG=KG, logits=x, bf16=True)
    c.bias = np.zeros(E, F32)
    c.bias[::5] = np.nan
    c.bias[1::5] = -np.inf
    c.d_bias = torch.from_numpy(c.bias).to(DEV)
    c.check_route(*c.route())


@pytest.mark.gpu
@pytest.mark.parametrize("G,KG", [(1, 1), (8, 3)])
def test_saturated_and_vanishing_scores(G, KG):
    """Scores that round to 1 or to 0 in fp32 tie and go to the lower index;
    between, every exponent of a score is reached."""
    r = np.random.default_rng(4)
    x = np.concatenate([r.uniform(10, 40, (40, 64)), r.uniform(-120, -80, (40, 64)),
                        r.uniform(-110, 30, (40, 64)), r.choice([-3e38, 3e38, -1e4, 89.0], (40, 64))])
    c = ByScore(160, 64, 8, G=G, KG=KG, logits=x)
    c.check_route(*c.route())
    c = ByScore(160, 64, 8, G=G, KG=KG, logits=x, bias=True)
    c.check_route(*c.route())


@pytest.mark.gpu
@pytest.mark.parametrize("E,G,KG", [(40, 5, 2), (256, 8, 4), (300, 3, 2), (1024, 16, 7)])
def test_few_distinct_values(E, G, KG):
    r = np.random.default_rng(E)
    x = r.integers(-2, 3, (60, E)).astype(F32)
    x[x == 0] *= r.choice([-1.0, 1.0], (x == 0).sum())
    c = ByScore(60, E, min(32, KG * (E // G)), G=G, KG=KG, logits=x, pad=0.1)
    c.check_route(*c.route())


@pytest.mark.gpu
def test_large_batch():
    ByScore(8192, 256, 8, G=8, KG=4, bias=True, pad=0.02, scale=2.5).all()


def test_refusals():
    lib, fake = ep.load_library(), 0x10000
    rt = ep.Routing(8, 64, 4, score="sigmoid", choose_by="scores")
    assert rt.choose_by_score == 1 and ep.Routing(8, 64, 4, score="sigmoid").choose_by_score == 0
    assert ep.ep_balance_workspace_bytes(rt) > 0
    with pytest.raises(ValueError, match="choose_by"):
        ep.Routing(8, 64, 4, choose_by="keys")

    def call():
        return lib.ep_route(ctypes.byref(rt), fake, 0, 64, None, None, fake, fake, None)

    rt.score = 0
    assert call() == ep.EP_ERR_UNSUPPORTED and ep.ep_balance_workspace_bytes(rt) == -1
    rt.score = 1
    for bad in (-1, 2):
        rt.choose_by_score = bad
        assert call() == ep.EP_ERR_ARG
