"""The routing calls and ep_expert_w4 refuse tensors whose dimensions lie in
another order, whatever their number of elements (no GPU needed: every public
call here is refused before anything is enqueued)."""
import pytest
import torch

import combine_ep_layout_09_amd as ep

F32, I32, U8, BF16 = torch.float32, torch.int32, torch.uint8, torch.bfloat16
T, E, k, B, K, N = 12, 8, 4, 3, 64, 24


def test_split_and_merged_dimensions_are_accepted():
    for want, shapes in (((12, 4), [(12, 4), (48,), (3, 4, 4), (12, 2, 2), (1, 12, 4), (12, 4, 1)]),
                         ((8, 24, 32), [(8, 24, 32), (192, 32), (8, 768), (6144,), (2, 4, 24, 32)]),
                         ((12,), [(12,), (3, 4), (1, 12)]), ((1,), [(1,), (), (1, 1)]),
                         ((0, 4), [(0, 4), (0,), (2, 0, 4)])):
        for s in shapes:
            ep._arg(torch.zeros(s), "v", F32, want, -1)


@pytest.mark.parametrize("want,shape", [((12, 4), (4, 12)), ((12, 4), (6, 8)), ((12, 4), (16, 3)),
                                        ((8, 24, 32), (24, 8, 32)), ((8, 24, 32), (8, 32, 24)),
                                        ((8, 24, 32), (32, 192)), ((2, 12), (3, 8))])
def test_other_orders_are_refused(want, shape):
    with pytest.raises(ValueError, match="shape|elements"):
        ep._arg(torch.zeros(shape), "v", F32, want, -1)


@pytest.fixture
def on_host(monkeypatch):
    """Host tensors pass for those of one GPU in the checks."""
    monkeypatch.setattr(ep, "_device_of", lambda t, name: -1)


def swapped(t):
    return t.transpose(0, 1).contiguous()


@pytest.mark.parametrize("wrong", ["topk_idx", "topk_weights"])
def test_route(on_host, wrong):
    a = dict(logits=torch.zeros((T, E)), topk_idx=torch.zeros((T, k), dtype=I32),
             topk_weights=torch.zeros((T, k)))
    a[wrong] = swapped(a[wrong])
    with pytest.raises(ValueError, match=f"{wrong} has shape"):
        ep.ep_route(ep.Routing(T, E, k), **a)
    with pytest.raises(ValueError, match=f"{wrong} has shape"):
        ep.prepare_route(ep.Routing(T, E, k), **a)


@pytest.mark.parametrize("wrong", ["topk_idx", "counts", "mean_prob"])
def test_balance_loss(on_host, wrong):
    a = dict(logits=torch.zeros((T, E)), topk_idx=torch.zeros((T, k), dtype=I32),
             counts=torch.zeros((B, E), dtype=I32), mean_prob=torch.zeros((B, E)),
             num_valid=torch.zeros(B, dtype=I32), loss=torch.zeros(1),
             workspace=torch.zeros(1 << 20, dtype=U8))
    a[wrong] = swapped(a[wrong])
    with pytest.raises(ValueError, match=f"{wrong} has shape"):
        ep.ep_balance_loss(ep.Routing(T, E, k, num_seqs=B), coef=0.1, **a)


@pytest.mark.parametrize("wrong", ["topk_idx", "d_weights", "counts", "d_logits"])
def test_route_backward(on_host, wrong):
    a = dict(logits=torch.zeros((T, E)), topk_idx=torch.zeros((T, k), dtype=I32),
             d_logits=torch.zeros((T, E)), d_weights=torch.zeros((T, k)),
             counts=torch.zeros((B, E), dtype=I32), num_valid=torch.zeros(B, dtype=I32),
             d_loss=torch.zeros(1))
    a[wrong] = swapped(a[wrong])
    with pytest.raises(ValueError, match=f"{wrong} has shape"):
        ep.ep_route_backward(ep.Routing(T, E, k, num_seqs=B), coef=0.1, **a)


@pytest.mark.parametrize("wrong", ["rows", "codes", "scales", "out", "row_scales"])
def test_expert_w4(on_host, wrong):
    prob, R = ep.Problem(T, 128, k, E), T * k
    fmt = 1 if wrong == "row_scales" else 0
    Kf = 256 if fmt else K
    lay = ep.Layout(*(torch.zeros(n, dtype=I32) for n in (E, E + 1, R, R, 2)))
    a = dict(rows=torch.zeros((R, Kf), dtype=U8 if fmt else BF16),
             codes=torch.zeros((E, N, Kf // 2), dtype=U8),
             scales=torch.zeros((E, N, Kf // 32), dtype=U8), out=torch.zeros((R, N), dtype=BF16),
             row_scales=torch.zeros((R, Kf // 128)) if fmt else None)
    a[wrong] = swapped(a[wrong])
    with pytest.raises(ValueError, match=f"{wrong} has shape"):
        ep.ep_expert_w4(prob, ep.ExpertW4(Kf, N, fmt), layout=lay, **a)
