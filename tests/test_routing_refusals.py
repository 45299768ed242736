"""Host-side checks of the routing calls and of ep_expert_w4 (no GPU needed):
every call here fails its host checks, so nothing is enqueued."""
import ctypes

import pytest
import torch

import combine_ep_layout_09_amd as ep

FAKE = 0x10000  # never dereferenced
ARG, UNSUPPORTED, ALIGN = ep.EP_ERR_ARG, ep.EP_ERR_UNSUPPORTED, ep.EP_ERR_ALIGN
NAN, INF = float("nan"), float("inf")


def routing(**over):
    a = dict(num_tokens=8, num_experts=64, num_topk=4, num_groups=8, topk_groups=2, score=0,
             normalize=1, num_seqs=2, weight_scale=1.0)
    a.update(over)
    rt = ep.Routing(1, 1, 1)
    for n, v in a.items():
        setattr(rt, n, v)
    return rt


BAD = [
    (dict(num_tokens=-2), ARG), (dict(num_experts=0), ARG), (dict(num_topk=0), ARG),
    (dict(num_groups=0), ARG), (dict(topk_groups=0), ARG), (dict(num_seqs=0), ARG),
    (dict(score=2), ARG), (dict(score=-1), ARG), (dict(normalize=2), ARG), (dict(normalize=-1), ARG),
    (dict(weight_scale=NAN), ARG), (dict(weight_scale=INF), ARG),
    (dict(num_experts=1032), UNSUPPORTED), (dict(num_topk=33, topk_groups=8), UNSUPPORTED),
    (dict(num_experts=130, num_groups=65), UNSUPPORTED),
    (dict(num_tokens=1 << 21, num_seqs=1 << 21), UNSUPPORTED),
    (dict(num_experts=60), ARG), (dict(topk_groups=9), ARG), (dict(num_topk=17), ARG),
    (dict(num_seqs=3), ARG), (dict(num_tokens=1 << 30), UNSUPPORTED),
    (dict(num_tokens=(1 << 25) + 2), UNSUPPORTED),
]


@pytest.mark.parametrize("over,code", BAD, ids=str)
def test_bad_problems(over, code):
    lib, rt = ep.load_library(), routing(**over)
    R = ctypes.byref(rt)
    n = max(rt.num_experts, 1)
    assert lib.ep_route(R, FAKE, 0, n, None, None, FAKE, FAKE, None) == code
    assert lib.ep_balance_workspace_bytes(R) == -1
    assert lib.ep_balance_loss(R, FAKE, 0, n, FAKE, None, 0.1, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30,
                               None) == code
    assert lib.ep_route_backward(R, FAKE, 0, n, FAKE, FAKE, None, 0.1, FAKE, FAKE, FAKE, FAKE,
                                 None) == code


def test_null_problem():
    lib = ep.load_library()
    assert lib.ep_route(None, FAKE, 0, 64, None, None, FAKE, FAKE, None) == ARG
    assert lib.ep_balance_workspace_bytes(None) == -1
    assert lib.ep_expert_w4(None, None, FAKE, None, None, FAKE, FAKE, FAKE, None) == ARG


def test_route_arguments():
    lib, R = ep.load_library(), ctypes.byref(routing())
    f = lib.ep_route
    assert f(R, None, 0, 64, None, None, FAKE, FAKE, None) == ARG
    assert f(R, FAKE, 2, 64, None, None, FAKE, FAKE, None) == ARG
    assert f(R, FAKE, 0, 63, None, None, FAKE, FAKE, None) == ARG
    assert f(R, FAKE, 0, (1 << 31) + 1, None, None, FAKE, FAKE, None) == UNSUPPORTED
    assert f(R, FAKE, 0, 64, None, None, None, FAKE, None) == ARG
    assert f(R, FAKE, 0, 64, None, None, FAKE, None, None) == ARG
    assert f(R, FAKE + 2, 0, 64, None, None, FAKE, FAKE, None) == ALIGN
    assert f(R, FAKE + 1, 1, 64, None, None, FAKE, FAKE, None) == ALIGN
    assert f(R, FAKE, 0, 64, FAKE + 2, None, FAKE, FAKE, None) == ALIGN
    assert f(R, FAKE, 0, 64, None, None, FAKE + 1, FAKE, None) == ALIGN
    assert f(R, FAKE, 0, 64, None, None, FAKE, FAKE + 2, None) == ALIGN


def test_balance_arguments():
    lib, rt = ep.load_library(), routing()
    R, n = ctypes.byref(rt), ep.ep_balance_workspace_bytes(rt)
    assert n > 0 and n % 256 == 0

    def call(logits=FAKE, idx=FAKE, coef=0.1, c=FAKE, m=FAKE, v=FAKE, l=FAKE, ws=FAKE, size=n):
        return lib.ep_balance_loss(R, logits, 0, 64, idx, None, coef, c, m, v, l, ws, size, None)

    assert call(logits=None) == call(idx=None) == call(c=None) == call(m=None) == ARG
    assert call(v=None) == call(l=None) == call(ws=None) == call(size=n - 1) == ARG
    assert call(coef=NAN) == call(coef=INF) == ARG
    assert call(idx=FAKE + 2) == call(c=FAKE + 1) == call(m=FAKE + 2) == call(v=FAKE + 2) == ALIGN
    assert call(l=FAKE + 1) == call(ws=FAKE + 8) == ALIGN


def test_gradient_arguments():
    lib, R = ep.load_library(), ctypes.byref(routing())

    def call(logits=FAKE, idx=FAKE, dw=FAKE, coef=0.1, c=FAKE, n=FAKE, dl=FAKE, dx=FAKE, bf16=0):
        return lib.ep_route_backward(R, logits, bf16, 64, idx, dw, None, coef, c, n, dl, dx, None)

    assert call(logits=None) == call(dx=None) == call(dw=None, dl=None) == ARG
    assert call(idx=None) == call(c=None) == call(n=None) == call(coef=NAN) == ARG
    assert call(idx=FAKE + 1) == call(dw=FAKE + 2) == call(c=FAKE + 2) == call(n=FAKE + 2) == ALIGN
    assert call(dl=FAKE + 2) == call(dx=FAKE + 2) == call(dx=FAKE + 1, bf16=1) == ALIGN


def test_expert_arguments():
    lib, prob = ep.load_library(), ep.Problem(8, 128, 2, 16)

    def layout(**over):
        s = ep._LayoutPtrs()
        for f, _ in ep._LayoutPtrs._fields_:
            setattr(s, f, over.get(f, FAKE))
        return ctypes.byref(s)

    def call(mm=(256, 64, 0, 0), p=prob, rows=FAKE, rs=FAKE, lay=None, codes=FAKE, scales=FAKE,
             out=FAKE):
        m = ep.ExpertW4(*mm)
        return lib.ep_expert_w4(ctypes.byref(p), ctypes.byref(m), rows, rs, lay or layout(), codes,
                                scales, out, None)

    assert call(p=ep.Problem(8, 128, 2, 0)) == ARG
    assert call(p=ep.Problem(8, 128, 2, 2000)) == UNSUPPORTED
    assert call(mm=(0, 64, 0, 0)) == call(mm=(256, 0, 0, 0)) == ARG
    assert call(mm=(256, 64, 3, 0)) == call(mm=(256, 64, -1, 0)) == ARG
    assert call(mm=(256, 64, 0, 2)) == call(mm=(256, 64, 0, -1)) == ARG
    assert call(mm=(48, 64, 0, 0)) == call(mm=(96, 64, 1, 0)) == UNSUPPORTED
    assert call(mm=(65568, 64, 0, 0)) == call(mm=(256, 65537, 0, 0)) == UNSUPPORTED
    assert call(rows=None) == call(codes=None) == call(scales=None) == call(out=None) == ARG
    assert call(mm=(256, 64, 1, 0), rs=None) == ARG
    assert call(lay=layout(count=None)) == call(lay=layout(offset=None)) == ARG
    assert call(lay=layout(count=FAKE + 2)) == call(lay=layout(offset=FAKE + 1)) == ALIGN
    assert call(rows=FAKE + 8) == call(codes=FAKE + 4) == call(scales=FAKE + 1) == ALIGN
    assert call(out=FAKE + 2) == call(mm=(256, 64, 2, 0), rs=FAKE + 8) == ALIGN
    assert lib.ep_expert_w4(ctypes.byref(prob), None, FAKE, FAKE, layout(), FAKE, FAKE, FAKE,
                            None) == ARG


def test_python_binding_refuses():
    rt = ep.Routing(4, 8, 2)
    f32, i32 = torch.float32, torch.int32
    x, idx, w = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=i32), torch.zeros((4, 2))
    with pytest.raises(ValueError, match="GPU memory"):
        ep.ep_route(rt, x, idx, w)
    with pytest.raises(TypeError, match="torch.Tensor"):
        ep.ep_route(rt, None, idx, w)
    with pytest.raises(ValueError, match="GPU memory"):
        ep.ep_balance_loss(rt, x, idx, 0.1, idx, w, idx, w, w)
    with pytest.raises(ValueError, match="GPU memory"):
        ep.ep_route_backward(rt, x, idx, x, d_weights=w)
    with pytest.raises(ValueError, match="score"):
        ep.Routing(4, 8, 2, score="relu")
    prob, mm = ep.Problem(4, 128, 2, 8), ep.ExpertW4(32, 8)
    lay = ep.Layout(*(torch.zeros(n, dtype=i32) for n in (8, 9, 8, 8, 2)))
    with pytest.raises(ValueError, match="GPU memory"):
        ep.ep_expert_w4(prob, mm, torch.zeros((8, 32), dtype=torch.bfloat16), lay,
                        torch.zeros(8 * 8 * 16, dtype=torch.uint8),
                        torch.zeros(64, dtype=torch.uint8),
                        torch.zeros((8, 8), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="elements"):
        ep._arg(torch.zeros(3), "v", f32, 4, -1)
    with pytest.raises(TypeError, match="dtype"):
        ep._arg(torch.zeros(3), "v", i32, 3, -1)
    with pytest.raises(ValueError, match="contiguous"):
        ep._arg(torch.zeros((3, 4)).t(), "v", f32, 12, -1)
