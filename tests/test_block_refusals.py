"""Host-side checks of layer norm, of dropout in the combine and of the 8-bit
integer calls (no GPU needed): every call here fails its host checks, so nothing is
enqueued."""
import ctypes

import pytest
import torch

import combine_ep_layout_09_amd as ep

ARG, UNSUPPORTED, ALIGN = ep.EP_ERR_ARG, ep.EP_ERR_UNSUPPORTED, ep.EP_ERR_ALIGN
NAN, INF = float("nan"), float("inf")


def at(i):
    """Addresses that are never dereferenced, 2^40 bytes apart."""
    return (i + 1) << 40


def norm(T=8, H=64, eps=1e-5):
    return ep.Norm(T, H, eps)


def forward(nm, x=at(0), xb=1, xs=None, w=at(1), b=at(2), wb=1, y=at(3), m=at(4), r=at(5)):
    nm_p = None if nm is None else ctypes.byref(nm)
    xs = (nm.hidden if nm is not None else 64) if xs is None else xs
    return ep.load_library().ep_layer_norm(nm_p, x, xb, xs, w, b, wb, y, m, r, None)


def backward(nm, x=at(0), xb=1, xs=None, dy=at(1), gs=None, w=at(2), wb=1, m=at(3), r=at(4),
             skip=at(5), dx=at(6), dw=at(7), db=at(8), ws=at(9), size=1 << 30):
    nm_p = None if nm is None else ctypes.byref(nm)
    H = nm.hidden if nm is not None else 64
    return ep.load_library().ep_layer_norm_backward(
        nm_p, x, xb, H if xs is None else xs, dy, H if gs is None else gs, w, wb, m, r, skip, dx,
        dw, db, ws, size, None)


BAD_NORMS = [(norm(T=-1), ARG), (norm(H=0), ARG), (norm(eps=-1.0), ARG), (norm(eps=NAN), ARG),
             (norm(eps=INF), ARG), (norm(T=(1 << 25) + 1), UNSUPPORTED), (norm(H=65537), UNSUPPORTED)]


@pytest.mark.parametrize("nm,code", BAD_NORMS, ids=repr)
def test_bad_norms(nm, code):
    assert forward(nm, xs=1 << 20) == code
    assert backward(nm, xs=1 << 20, gs=1 << 20) == code
    assert ep.ep_layer_norm_workspace_bytes(nm) == -1


def test_layer_norm_arguments():
    nm = norm()
    assert forward(None) == ARG
    assert forward(nm, x=None) == ARG and forward(nm, y=None) == ARG
    assert forward(nm, xb=2) == ARG and forward(nm, wb=-1) == ARG
    assert forward(nm, xs=63) == ARG and forward(nm, xs=(1 << 31) + 1) == UNSUPPORTED
    assert forward(nm, m=None) == ARG and forward(nm, r=None) == ARG
    for over in (dict(x=at(0) + 1), dict(y=at(3) + 1), dict(w=at(1) + 1), dict(b=at(2) + 1),
                 dict(m=at(4) + 2), dict(r=at(5) + 2), dict(xb=0, x=at(0) + 2),
                 dict(xb=0, y=at(3) + 2), dict(wb=0, w=at(1) + 2), dict(wb=0, b=at(2) + 2)):
        assert forward(nm, **over) == ALIGN
    for over in (dict(y=at(0)), dict(y=at(0) + 8 * 64 * 2 - 2), dict(y=at(1)), dict(m=at(3) + 4),
                 dict(r=at(4)), dict(r=at(2)), dict(y=at(0) + 900, xs=1000)):
        assert forward(nm, **over) == ARG


def test_layer_norm_backward_arguments():
    nm = norm()
    need = ep.ep_layer_norm_workspace_bytes(nm)
    assert need > 0 and need % 256 == 0
    assert backward(None) == ARG
    for name in ("x", "dy", "m", "r", "dx"):
        assert backward(nm, **{name: None}) == ARG
    assert backward(nm, xb=2) == ARG and backward(nm, wb=2) == ARG
    assert backward(nm, xs=63) == ARG and backward(nm, gs=63) == ARG
    assert backward(nm, ws=None) == ARG and backward(nm, size=need - 1) == ARG
    assert backward(nm, ws=None, dw=None) == ARG
    for over in (dict(x=at(0) + 1), dict(dy=at(1) + 1), dict(w=at(2) + 1), dict(m=at(3) + 1),
                 dict(r=at(4) + 2), dict(skip=at(5) + 1), dict(dx=at(6) + 1), dict(dw=at(7) + 1),
                 dict(db=at(8) + 1), dict(ws=at(9) + 8), dict(xb=0, dx=at(6) + 2),
                 dict(xb=0, skip=at(5) + 2), dict(wb=0, dw=at(7) + 2)):
        assert backward(nm, **over) == ALIGN
    for over in (dict(dx=at(0)), dict(dx=at(1)), dict(dx=at(5)), dict(dw=at(8)), dict(dw=at(2)),
                 dict(ws=at(6)), dict(db=at(9) + 256)):
        assert backward(nm, **over) == ARG


def problem(T=8, H=64, k=2, E=4, cap=0):
    return ep.Problem(T, H, k, E, cap)


def layout(**over):
    a = dict(count=at(20), offset=at(21), slot_of=at(22), src_of_slot=at(23), status=at(24))
    a.update(over)
    return ep._LayoutPtrs(**a)


def combine(prob=None, eo=at(0), lay=None, w=at(1), res=at(2), p=0.1, rng=at(3), y=at(4)):
    prob, lay = prob or problem(), lay or layout()
    return ep.load_library().ep_combine_dropout(ctypes.byref(prob), eo, ctypes.byref(lay), w, res,
                                                p, rng, y, None)


def combine_grad(prob=None, dy=at(0), eo=at(1), lay=None, w=at(2), p=0.1, rng=at(3), deo=at(4),
                 dw=at(5)):
    prob, lay = prob or problem(), lay or layout()
    return ep.load_library().ep_combine_backward(ctypes.byref(prob), dy, eo, ctypes.byref(lay), w,
                                                 p, rng, deo, dw, None)


def dispatch(prob=None, x=at(0), lay=None, q=at(1), s=at(2)):
    prob, lay = prob or problem(), lay or layout()
    return ep.load_library().ep_dispatch_i8(ctypes.byref(prob), x, ctypes.byref(lay), q, s, None)


BAD_PROBLEMS = [(problem(T=-1), ARG), (problem(k=0), ARG), (problem(H=0), ARG),
                (problem(H=65), UNSUPPORTED), (problem(E=1025), UNSUPPORTED),
                (problem(k=33), UNSUPPORTED), (problem(T=(1 << 21) + 1), UNSUPPORTED),
                (problem(H=65544), UNSUPPORTED)]


@pytest.mark.parametrize("prob,code", BAD_PROBLEMS, ids=repr)
def test_bad_problems(prob, code):
    assert combine(prob) == code
    assert combine_grad(prob) == code
    assert dispatch(prob) == code


@pytest.mark.parametrize("p", [-0.1, 1.0, 1.5, NAN, INF])
def test_probability(p):
    assert combine(p=p) == ARG
    assert combine_grad(p=p) == ARG


def test_combine_dropout_arguments():
    for name in ("eo", "w", "y", "rng"):
        assert combine(**{name: None}) == ARG
    assert combine(lay=layout(slot_of=None)) == ARG
    for over in (dict(eo=at(0) + 8), dict(y=at(4) + 8), dict(res=at(2) + 8), dict(w=at(1) + 2),
                 dict(rng=at(3) + 4), dict(lay=layout(slot_of=at(22) + 2))):
        assert combine(**over) == ALIGN
    for over in (dict(y=at(0)), dict(y=at(2)), dict(y=at(1)), dict(y=at(0) + 16 * 64 * 2 - 16),
                 dict(y=at(22)), dict(y=at(3))):
        assert combine(**over) == ARG


def test_combine_backward_arguments():
    for name in ("dy", "w", "deo", "rng", "eo"):
        assert combine_grad(**{name: None}) == ARG
    for over in (dict(dy=at(0) + 8), dict(eo=at(1) + 8), dict(deo=at(4) + 8), dict(w=at(2) + 2),
                 dict(dw=at(5) + 2), dict(rng=at(3) + 4)):
        assert combine_grad(**over) == ALIGN
    for over in (dict(deo=at(0)), dict(deo=at(1)), dict(dw=at(2)), dict(dw=at(4) + 64)):
        assert combine_grad(**over) == ARG


def test_dispatch_i8_arguments():
    for name in ("x", "q", "s"):
        assert dispatch(**{name: None}) == ARG
    for over in (dict(x=at(0) + 8), dict(q=at(1) + 8), dict(s=at(2) + 2)):
        assert dispatch(**over) == ALIGN
    for over in (dict(q=at(0)), dict(s=at(0) + 64), dict(s=at(1) + 64)):
        assert dispatch(**over) == ARG


def expert(prob=None, mm=None, rows=at(0), rs=at(1), lay=None, w=at(2), s=at(3), out=at(4),
           ws=at(5), size=1 << 30):
    prob, lay, mm = prob or problem(), lay or layout(), mm or ep.ExpertI8(64, 48, 1)
    return ep.load_library().ep_expert_i8(ctypes.byref(prob), ctypes.byref(mm), rows, rs,
                                          ctypes.byref(lay), w, s, out, ws, size, None)


BAD_PRODUCTS = [((0, 8), ARG), ((16, 0), ARG), ((16, 8, 2), ARG), ((16, 8, -1), ARG),
                ((16, 8, 0, 2), ARG), ((24, 8), UNSUPPORTED), ((8, 8), UNSUPPORTED),
                ((65552, 8), UNSUPPORTED), ((16, 65537), UNSUPPORTED)]


@pytest.mark.parametrize("args,code", BAD_PRODUCTS)
def test_bad_products(args, code):
    mm = ep.ExpertI8(16, 8)
    for (name, _), v in zip(mm._fields_, args):
        setattr(mm, name, v)
    assert expert(mm=mm) == code
    assert ep.ep_expert_i8_workspace_bytes(problem(), mm) == -1


def test_expert_i8_arguments():
    lib = ep.load_library()
    assert lib.ep_expert_i8(None, None, at(0), at(1), None, at(2), at(3), at(4), None, 0, None) == ARG
    for name in ("rows", "rs", "w", "s", "out"):
        assert expert(**{name: None}) == ARG
    assert expert(lay=layout(count=None)) == ARG and expert(lay=layout(offset=None)) == ARG
    for over in (dict(rows=at(0) + 8), dict(w=at(2) + 8), dict(out=at(4) + 8), dict(s=at(3) + 2),
                 dict(rs=at(1) + 2), dict(lay=layout(count=at(20) + 2))):
        assert expert(**over) == ALIGN
    for over in (dict(out=at(0)), dict(out=at(1) - 64), dict(out=at(2)), dict(out=at(20))):
        assert expert(**over) == ARG
    bf16 = ep.ExpertI8(64, 48, 0)
    need = ep.ep_expert_i8_workspace_bytes(problem(), bf16)
    assert need >= 16 * 68 and need % 256 == 0
    assert ep.ep_expert_i8_workspace_bytes(problem(), ep.ExpertI8(64, 48, 1)) == 0
    assert expert(mm=bf16, ws=None) == ARG and expert(mm=bf16, size=need - 1) == ARG
    assert expert(mm=bf16, ws=at(5) + 8) == ALIGN
    assert expert(mm=bf16, ws=at(0)) == ARG and expert(mm=bf16, ws=at(4)) == ARG


def test_binding_refuses_host_tensors_and_wrong_types():
    T, H = 8, 64
    nm, prob = norm(), problem()
    x, w = torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(H, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x must be in GPU memory"):
        ep.ep_layer_norm(nm, x, w, w, x.clone())
    with pytest.raises(TypeError, match="x must be a torch.Tensor"):
        ep.ep_layer_norm(nm, None, w, w, x)
    with pytest.raises(ValueError, match="x must be in GPU memory"):
        ep.ep_layer_norm_backward(nm, x, x, w, w, w, x)
    lay = ep.Layout(*(torch.zeros(n, dtype=torch.int32) for n in (4, 5, 16, 16, 2)))
    with pytest.raises(ValueError, match="y must be in GPU memory"):
        ep.ep_combine_dropout(prob, x, lay, w, 0.1, None, x)
    with pytest.raises(ValueError, match="dy must be in GPU memory"):
        ep.ep_combine_backward(prob, x, x, lay, w, 0.1, None, x)
    with pytest.raises(ValueError, match="x must be in GPU memory"):
        ep.ep_dispatch_i8(prob, x, lay, x, w)
    with pytest.raises(ValueError, match="rows must be in GPU memory"):
        ep.ep_expert_i8(prob, ep.ExpertI8(64, 48), x, lay, x, w, x)
