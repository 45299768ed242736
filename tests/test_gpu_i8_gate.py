"""ep_expert_i8's gated activation over the whole range of a gate: from where silu
leaves fp32 (about -104) up to where it is the gate itself, in every kernel.

A row holds one code of 1 and zeros, so that gate and up are one weight times two
scales, exact but for the two products.  Tolerance of an output: block_reference's (the
exponential's argument, a few steps of exponential, sum, reciprocal and products, one
rounding to bf16), and half a step of fp32's subnormals, 2^-150, which silu itself may
be off by, times up.  bf16's own subnormals have steps of 2^-133."""
import numpy as np
import pytest
import torch

import combine_ep_layout_09_amd as ep
import oracle
from tests import block_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def contiguous_layout(T):
    """Every token's only entry goes to expert 0."""
    r = oracle.layout(np.zeros((T, 1), np.int32), 1, 0)
    return ep.Layout(*(torch.from_numpy(np.ascontiguousarray(r[n], np.int32)).to(DEV)
                       for n in ("count", "offset", "slot_of", "src_of_slot", "status")))


def steps(gates):
    """Scales and codes whose products are these gates to 2^-24."""
    code = np.where(np.abs(gates) < 1, 1, np.clip(np.rint(np.abs(gates)), 1, 127))
    return np.sign(gates) * code, np.where(gates == 0, 1.0, np.abs(gates) / code)


# T tokens of one expert: the few-row kernel, and row tiles of 64, 128 and 256 rows
@pytest.mark.parametrize("T,K", [(17, 64), (17, 128), (300, 64), (1000, 128), (2500, 64), (9000, 128)])
@pytest.mark.parametrize("up", [1.5, 2.0 ** 40, -2.0 ** 90])
def test_gates_of_every_size(T, K, up):
    gates = np.concatenate([
        np.linspace(-120, 60, 1801), np.linspace(-92, -85, 701), np.linspace(-46, -43, 301),
        -np.exp2(np.linspace(-100, 6, 300)), np.exp2(np.linspace(-100, 30, 300)), [0.0, -200.0, -1e30],
    ]).astype(np.float32).astype(np.float64)
    N = len(gates)
    code, size = steps(gates)
    r = np.random.default_rng(T + K)
    w = r.integers(-128, 128, (1, 2 * N, K), dtype=np.int8)
    at = 7  # the channel that the rows' only code stands in
    big = np.abs(gates) > 1e4
    code[big], size[big] = np.sign(gates[big]) * 100, np.abs(gates[big]) / 100
    w[0, :N, at], w[0, N:, at] = code.astype(np.int8), 1
    scale = np.concatenate([size, np.full(N, abs(up))])[None].astype(np.float32)
    if up < 0:
        w[0, N:, at] = -1
    q = np.zeros((T, K), np.int8)
    q[:, at] = 1
    rs = np.ones(T, np.float32)
    print(f"[gpu] gates T {T} K {K} N {N} up {up}", flush=True)
    out = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
    ep.ep_expert_i8(ep.Problem(T, 128, 1, 1), ep.ExpertI8(K, N, 1, 1), torch.from_numpy(q).to(DEV),
                    contiguous_layout(T), torch.from_numpy(w).to(DEV), torch.from_numpy(scale).to(DEV),
                    out, row_scales=torch.from_numpy(rs).to(DEV))
    torch.cuda.synchronize()
    assert torch.equal(out, out[:1].expand(T, N))
    got = out[0].double().cpu().numpy()
    with np.errstate(over="ignore"):
        want, tol = ref.i8_products(q[:1], rs[:1], w[0], scale[0], True)
    tol = tol[0] + 2.0 ** -150 * abs(up)
    off = np.abs(got - want[0])
    bad = ~(off <= tol)
    assert not bad.any(), [(gates[i], got[i], want[0, i]) for i in np.flatnonzero(bad)[:6]]
