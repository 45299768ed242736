"""The plain forms that the GPU tests of layer norm, dropout and the 8-bit
products compare with, checked by themselves."""
import numpy as np
import pytest
import torch

from tests import block_reference as ref


# Known answers of Philox4x32-10 (its authors' published test vectors).
VECTORS = [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
]


@pytest.mark.parametrize("counter,key,words", VECTORS)
def test_generator(counter, key, words):
    got = ref.philox(np.array(counter, np.uint64), key)
    assert tuple(int(v) for v in got) == words


def test_mask_share():
    """The share of zeros lies within five deviations of p."""
    for p in (0.05, 0.5, 0.9):
        keep = ref.kept(512, 512, p, 1234567, 89)
        n = keep.size
        assert abs((~keep).sum() - p * n) < 5 * np.sqrt(n * p * (1 - p))
    assert ref.kept(7, 33, 0.0, 1, 2).all()


def test_norm_gradient_by_differences():
    """The gradient's formula against central differences of the forward one, in 64 bits."""
    r = np.random.default_rng(0)
    x, w, b, dy = (r.standard_normal(s) for s in ((3, 7), 7, 7, (3, 7)))
    _, m, rs = ref.norm(x, w, b, 1e-3)
    dx, dw, db = ref.norm_grad(x, dy, w, m, rs)
    h = 1e-5
    for arr, grad in ((x, dx), (w, dw), (b, db)):
        for i in np.ndindex(arr.shape):
            old = arr[i]
            arr[i] = old + h
            up = (ref.norm(x, w, b, 1e-3)[0] * dy).sum()
            arr[i] = old - h
            down = (ref.norm(x, w, b, 1e-3)[0] * dy).sum()
            arr[i] = old
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-7


def test_norm_against_torch():
    r = np.random.default_rng(1)
    x, w, b = r.standard_normal((5, 33)), r.standard_normal(33), r.standard_normal(33)
    y, _, _ = ref.norm(x, w, b, 1e-5)
    want = torch.nn.functional.layer_norm(*(torch.from_numpy(v) for v in (x,)), (33,),
                                          torch.from_numpy(w), torch.from_numpy(b), 1e-5)
    assert np.abs(y - want.numpy()).max() < 1e-12


def test_combine_gradient_by_differences():
    r = np.random.default_rng(2)
    T, k, H, p = 3, 2, 8, 0.3
    slot = np.array([[0, 4], [-1, 2], [5, 1]])
    eo, w, dy = r.standard_normal((6, H)), r.random((T, k)), r.standard_normal((T, H))
    keep = ref.kept(T, H, p, 5, 6)
    rows, _, dw, _ = ref.combine_grad(dy, eo, slot, w, keep, p)
    h = 1e-5

    def value():
        return (ref.combine(eo, slot, w, keep, p)[0] * dy).sum()

    for arr, grad in ((w, dw), (eo, np.stack([rows.get(s, np.zeros(H)) for s in range(6)]))):
        for i in np.ndindex(arr.shape):
            old = arr[i]
            arr[i] = old + h
            up = value()
            arr[i] = old - h
            down = value()
            arr[i] = old
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-7


def test_quant():
    x = np.array([[127, -127, 0.5, 1.5, 2.5, -0.5], [0] * 6, [1e-38, -3e-38, 2e-39, 0, 0, 0]])
    q, s = ref.quant(x)
    assert q[0].tolist() == [127, -127, 0, 2, 2, 0] and s[0] == 1
    assert not q[1].any() and s[1] == 0
    assert np.abs(q).max() <= 127
