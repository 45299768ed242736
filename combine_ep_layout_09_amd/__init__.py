"""MoE token dispatch / combine on one AMD MI355X: Python binding of libep.

The binding only marshals arguments: it checks dtypes, shapes and devices of
torch tensors, passes their device pointers and the current HIP stream to the
C ABI in include/ep.h, and turns a nonzero status into an exception.  Every
step of the computation runs in the HIP kernels of libep.so; there is no
Python or CPU fallback -- if libep.so cannot be loaded, calls raise.

Entry points (same names as the C ABI):
  ep_num_recv_rows(prob)                     -> R
  ep_layout_workspace_bytes(prob)            -> bytes
  ep_layout(prob, topk_idx, layout, workspace, stream=None)
  ep_dispatch(prob, x, layout, recv_x, recv_scales=None, stream=None)
  ep_layout_dispatch(prob, topk_idx, layout, workspace, x, recv_x, recv_scales=None,
                     stream=None)
  ep_layout_dispatch_noalloc(prob, topk_idx, layout, x, recv_x, recv_scales=None,
                             stream=None)   (workspace: the library's device array)
  ep_combine(prob, expert_out, layout, topk_weights, y, stream=None)
  ep_route(rt, logits, topk_idx, topk_weights, expert_bias=None, valid=None, stream=None)
  ep_balance_workspace_bytes(rt)             -> bytes
  ep_balance_loss(rt, logits, topk_idx, coef, counts, mean_prob, num_valid, loss,
                  workspace, valid=None, stream=None)
  ep_route_backward(rt, logits, topk_idx, d_logits, d_weights=None, coef=0.0,
                    counts=None, num_valid=None, d_loss=None, valid=None, stream=None)
  ep_expert_w4(prob, mm, rows, layout, codes, scales, out, row_scales=None, stream=None)
  ep_layer_norm(nm, x, weight, bias, y, mean=None, rstd=None, stream=None)
  ep_layer_norm_workspace_bytes(nm)          -> bytes
  ep_layer_norm_backward(nm, x, dy, weight, mean, rstd, dx, d_weight=None, d_bias=None,
                         workspace=None, d_skip=None, stream=None)
  ep_combine_dropout(prob, expert_out, layout, topk_weights, p, rng, y, residual=None,
                     stream=None)
  ep_combine_backward(prob, dy, expert_out, layout, topk_weights, p, rng, d_expert_out,
                      d_weights=None, stream=None)
  ep_dispatch_i8(prob, x, layout, recv_q, recv_scales, stream=None)
  ep_expert_i8_workspace_bytes(prob, mm)     -> bytes
  ep_expert_i8(prob, mm, rows, layout, weights, scales, out, row_scales=None,
               workspace=None, stream=None)
  ep_e4m3_encode(inp, out, stream=None)
  ep_strerror(code)

Helpers that allocate with torch (plumbing, outside the computation):
  Problem(...), Layout.empty(prob, device), alloc_workspace, alloc_recv,
  Routing(...), ExpertW4(...), Norm(...), ExpertI8(...).

The calls from ep_route on run on the GPU that holds their tensors,
by default on that GPU's current stream; tensors on several devices are
refused.

Prepared calls (prepare_layout / prepare_dispatch / prepare_combine / ...) check
and marshal the arguments once and return a callable that only issues the C
call, for loops that launch the same problem many times.
"""
import ctypes
import math
import os

__all__ = [
    "Problem", "Layout", "EpError", "ep_num_recv_rows", "ep_layout_workspace_bytes",
    "ep_layout", "ep_dispatch", "ep_combine", "ep_e4m3_encode", "ep_strerror",
    "alloc_workspace", "alloc_recv", "library_path", "load_library",
    "prepare_layout", "prepare_dispatch", "prepare_combine", "ep_layout_dispatch",
    "prepare_layout_dispatch", "ep_layout_dispatch_noalloc",
    "Routing", "ExpertW4", "ep_route", "ep_balance_workspace_bytes", "ep_balance_loss",
    "ep_route_backward", "ep_expert_w4", "prepare_route", "prepare_balance_loss",
    "prepare_route_backward", "prepare_expert_w4",
    "Norm", "ExpertI8", "ep_layer_norm", "ep_layer_norm_workspace_bytes",
    "ep_layer_norm_backward", "ep_combine_dropout", "ep_combine_backward", "ep_dispatch_i8",
    "ep_expert_i8_workspace_bytes", "ep_expert_i8", "prepare_layer_norm",
    "prepare_layer_norm_backward", "prepare_combine_dropout", "prepare_combine_backward",
    "prepare_dispatch_i8", "prepare_expert_i8",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libep.so")
_lib = None

EP_OK, EP_ERR_ARG, EP_ERR_UNSUPPORTED, EP_ERR_ALIGN, EP_ERR_HIP = 0, -1, -2, -3, -4


class EpError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed with status {code}: {ep_strerror(code)}")
        self.code = code


class Problem(ctypes.Structure):
    """ep_problem: T, H, k, E, capacity (0 = contiguous), use_fp8 (0 bf16,
    1 E4M3FN + fp32 scales, 2 E4M3FN + UE8M0 scale bytes)."""
    _fields_ = [("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("num_topk", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("use_fp8", ctypes.c_int32)]

    def __init__(self, num_tokens, hidden, num_topk, num_experts, capacity=0, use_fp8=0):
        super().__init__(num_tokens, hidden, num_topk, num_experts, capacity, int(use_fp8))

    def __repr__(self):
        return (f"Problem(T={self.num_tokens}, H={self.hidden}, k={self.num_topk}, "
                f"E={self.num_experts}, cap={self.capacity}, fp8={self.use_fp8})")


class Routing(ctypes.Structure):
    """ep_routing: T, E, k, groups and how many of them a token may use, the
    score ("softmax" / 0 or "sigmoid" / 1), whether a token's weights are
    normalised, sequences of the balance loss, factor of the weights, and
    whether the choice goes by "logits" / 0 or by "scores" / 1, as that of a
    model with a sigmoid gate does (sigmoid only)."""
    _fields_ = [("num_tokens", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("num_topk", ctypes.c_int32), ("num_groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("score", ctypes.c_int32),
                ("normalize", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("weight_scale", ctypes.c_float), ("choose_by_score", ctypes.c_int32)]

    _scores = {"softmax": 0, "sigmoid": 1, 0: 0, 1: 1}
    _choices = {"logits": 0, "scores": 1, 0: 0, 1: 1}

    def __init__(self, num_tokens, num_experts, num_topk, num_groups=1, topk_groups=1,
                 score="softmax", normalize=True, num_seqs=1, weight_scale=1.0,
                 choose_by="logits"):
        if score not in self._scores:
            raise ValueError(f"score is {score!r}, expected 'softmax' or 'sigmoid'")
        if choose_by not in self._choices:
            raise ValueError(f"choose_by is {choose_by!r}, expected 'logits' or 'scores'")
        ctypes.Structure.__init__(self, num_tokens, num_experts, num_topk, num_groups,
                                  topk_groups, self._scores[score], int(normalize), num_seqs,
                                  weight_scale, self._choices[choose_by])

    def __repr__(self):
        return (f"Routing(T={self.num_tokens}, E={self.num_experts}, k={self.num_topk}, "
                f"groups={self.topk_groups}/{self.num_groups}, "
                f"score={'sigmoid' if self.score else 'softmax'}, "
                f"choose_by={'scores' if self.choose_by_score else 'logits'}, "
                f"normalize={self.normalize}, "
                f"seqs={self.num_seqs}, scale={self.weight_scale})")


class ExpertW4(ctypes.Structure):
    """ep_expert_w4_t: K inputs, N outputs, format of the rows (0 bf16, 1 and 2
    E4M3FN as Problem.use_fp8) and activation (0 none, 1 silu(gate) * up)."""
    _fields_ = [("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32),
                ("in_format", ctypes.c_int32), ("activation", ctypes.c_int32)]

    def __init__(self, in_features, out_features, in_format=0, activation=0):
        super().__init__(in_features, out_features, int(in_format), int(activation))

    def __repr__(self):
        return (f"ExpertW4(K={self.in_features}, N={self.out_features}, "
                f"format={self.in_format}, activation={self.activation})")


class Norm(ctypes.Structure):
    """ep_norm: T rows of H channels and what is added to their variance."""
    _fields_ = [("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("eps", ctypes.c_float)]

    def __init__(self, num_tokens, hidden, eps=1e-5):
        super().__init__(num_tokens, hidden, eps)

    def __repr__(self):
        return f"Norm(T={self.num_tokens}, H={self.hidden}, eps={self.eps})"


class ExpertI8(ctypes.Structure):
    """ep_expert_i8_t: K inputs, N outputs, format of the rows (0 bf16, quantised
    by the call; 1 int8 with a scale per row) and activation (0 none,
    1 silu(gate) * up)."""
    _fields_ = [("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32),
                ("in_format", ctypes.c_int32), ("activation", ctypes.c_int32)]

    def __init__(self, in_features, out_features, in_format=0, activation=0):
        super().__init__(in_features, out_features, int(in_format), int(activation))

    def __repr__(self):
        return (f"ExpertI8(K={self.in_features}, N={self.out_features}, "
                f"format={self.in_format}, activation={self.activation})")


class _LayoutPtrs(ctypes.Structure):
    _fields_ = [("count", ctypes.c_void_p), ("offset", ctypes.c_void_p),
                ("slot_of", ctypes.c_void_p), ("src_of_slot", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


def library_path():
    return _LIB_PATH


def load_library():
    """Load libep.so, building it first only if no build exists."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        from . import build as _build
        _build.build()
    # torch ships its own HIP runtime under the same soname; loading it first
    # makes libep bind to that runtime, so torch's streams and memory are ours.
    _torch()
    lib = ctypes.CDLL(_LIB_PATH)
    P = ctypes.POINTER(Problem)
    L = ctypes.POINTER(_LayoutPtrs)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    lib.ep_num_recv_rows.restype = i64
    lib.ep_num_recv_rows.argtypes = [P]
    lib.ep_layout_workspace_bytes.restype = i64
    lib.ep_layout_workspace_bytes.argtypes = [P]
    lib.ep_layout.restype = ctypes.c_int
    lib.ep_layout.argtypes = [P, vp, L, vp, ctypes.c_size_t, vp]
    lib.ep_dispatch.restype = ctypes.c_int
    lib.ep_dispatch.argtypes = [P, vp, L, vp, vp, vp]
    lib.ep_layout_dispatch.restype = ctypes.c_int
    lib.ep_layout_dispatch.argtypes = [P, vp, L, vp, ctypes.c_size_t, vp, vp, vp, vp]
    lib.ep_layout_dispatch_noalloc.restype = ctypes.c_int
    lib.ep_layout_dispatch_noalloc.argtypes = [P, vp, L, vp, vp, vp, vp]
    lib.ep_combine.restype = ctypes.c_int
    lib.ep_combine.argtypes = [P, vp, L, vp, vp, vp]
    RT, i32, f32 = ctypes.POINTER(Routing), ctypes.c_int, ctypes.c_float
    lib.ep_route.restype = ctypes.c_int
    lib.ep_route.argtypes = [RT, vp, i32, i64, vp, vp, vp, vp, vp]
    lib.ep_balance_workspace_bytes.restype = i64
    lib.ep_balance_workspace_bytes.argtypes = [RT]
    lib.ep_balance_loss.restype = ctypes.c_int
    lib.ep_balance_loss.argtypes = [RT, vp, i32, i64, vp, vp, f32, vp, vp, vp, vp, vp,
                                    ctypes.c_size_t, vp]
    lib.ep_route_backward.restype = ctypes.c_int
    lib.ep_route_backward.argtypes = [RT, vp, i32, i64, vp, vp, vp, f32, vp, vp, vp, vp, vp]
    lib.ep_expert_w4.restype = ctypes.c_int
    lib.ep_expert_w4.argtypes = [P, ctypes.POINTER(ExpertW4), vp, vp, L, vp, vp, vp, vp]
    size, f64 = ctypes.c_size_t, ctypes.c_double
    NM, I8 = ctypes.POINTER(Norm), ctypes.POINTER(ExpertI8)
    lib.ep_layer_norm.restype = ctypes.c_int
    lib.ep_layer_norm.argtypes = [NM, vp, i32, i64, vp, vp, i32, vp, vp, vp, vp]
    lib.ep_layer_norm_workspace_bytes.restype = i64
    lib.ep_layer_norm_workspace_bytes.argtypes = [NM]
    lib.ep_layer_norm_backward.restype = ctypes.c_int
    lib.ep_layer_norm_backward.argtypes = [NM, vp, i32, i64, vp, i64, vp, i32, vp, vp, vp, vp,
                                           vp, vp, vp, size, vp]
    lib.ep_combine_dropout.restype = ctypes.c_int
    lib.ep_combine_dropout.argtypes = [P, vp, L, vp, vp, f64, vp, vp, vp]
    lib.ep_combine_backward.restype = ctypes.c_int
    lib.ep_combine_backward.argtypes = [P, vp, vp, L, vp, f64, vp, vp, vp, vp]
    lib.ep_dispatch_i8.restype = ctypes.c_int
    lib.ep_dispatch_i8.argtypes = [P, vp, L, vp, vp, vp]
    lib.ep_expert_i8_workspace_bytes.restype = i64
    lib.ep_expert_i8_workspace_bytes.argtypes = [P, I8]
    lib.ep_expert_i8.restype = ctypes.c_int
    lib.ep_expert_i8.argtypes = [P, I8, vp, vp, L, vp, vp, vp, vp, size, vp]
    lib.ep_e4m3_encode.restype = ctypes.c_int
    lib.ep_e4m3_encode.argtypes = [vp, vp, i64, vp]
    lib.ep_strerror.restype = ctypes.c_char_p
    lib.ep_strerror.argtypes = [ctypes.c_int]
    _lib = lib
    return lib


def ep_strerror(code):
    return load_library().ep_strerror(int(code)).decode()


def ep_num_recv_rows(prob):
    return int(load_library().ep_num_recv_rows(ctypes.byref(prob)))


def ep_layout_workspace_bytes(prob):
    return int(load_library().ep_layout_workspace_bytes(ctypes.byref(prob)))


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream_handle(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr(t, name, dtype=None, numel=None, allow_none=False):
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() and not t.is_cuda:
        raise ValueError(f"{name} must be in GPU memory")
    return t.data_ptr() if t.numel() else None


class Layout:
    """Device tensors written by ep_layout (int32): count [E], offset [E+1],
    slot_of [T, k], src_of_slot [R], status [2]."""

    def __init__(self, count, offset, slot_of, src_of_slot, status):
        self.count, self.offset, self.slot_of = count, offset, slot_of
        self.src_of_slot, self.status = src_of_slot, status

    @classmethod
    def empty(cls, prob, device="cuda"):
        torch = _torch()
        i32 = torch.int32
        R = ep_num_recv_rows(prob)
        if R < 0:
            raise ValueError(f"invalid problem {prob!r}")
        return cls(torch.empty(prob.num_experts, dtype=i32, device=device),
                   torch.empty(prob.num_experts + 1, dtype=i32, device=device),
                   torch.empty((prob.num_tokens, prob.num_topk), dtype=i32, device=device),
                   torch.empty(R, dtype=i32, device=device),
                   torch.empty(2, dtype=i32, device=device))

    def _struct(self, prob, check_all=True):
        T, k, E = prob.num_tokens, prob.num_topk, prob.num_experts
        torch = _torch()
        s = _LayoutPtrs()
        s.slot_of = _ptr(self.slot_of, "slot_of", torch.int32, T * k, allow_none=True)
        if check_all:
            s.count = _ptr(self.count, "count", torch.int32, E)
            s.offset = _ptr(self.offset, "offset", torch.int32, E + 1)
            s.src_of_slot = _ptr(self.src_of_slot, "src_of_slot", torch.int32,
                                 ep_num_recv_rows(prob), allow_none=True)
            s.status = _ptr(self.status, "status", torch.int32, 2)
        return s


def alloc_workspace(prob, device="cuda"):
    torch = _torch()
    n = ep_layout_workspace_bytes(prob)
    if n < 0:
        raise ValueError(f"invalid problem {prob!r}")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _scale_dtype(prob):
    """Block-scale element type: fp32 (use_fp8 = 1) or UE8M0 bytes (use_fp8 = 2)."""
    return _torch().uint8 if prob.use_fp8 == 2 else _torch().float32


def alloc_recv(prob, device="cuda"):
    """Receive buffers for dispatch: (recv_x, recv_scales or None)."""
    torch = _torch()
    R = ep_num_recv_rows(prob)
    if prob.use_fp8:
        return (torch.empty((R, prob.hidden), dtype=torch.uint8, device=device),
                torch.empty((R, prob.hidden // 128), dtype=_scale_dtype(prob), device=device))
    return torch.empty((R, prob.hidden), dtype=torch.bfloat16, device=device), None


def _check(fn, code):
    if code != EP_OK:
        raise EpError(fn, code)


def ep_layout(prob, topk_idx, layout, workspace, stream=None):
    torch = _torch()
    lib = load_library()
    idx = _ptr(topk_idx, "topk_idx", torch.int32, prob.num_tokens * prob.num_topk,
               allow_none=True)
    s = layout._struct(prob)
    ws = _ptr(workspace, "workspace", allow_none=True)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("ep_layout", lib.ep_layout(ctypes.byref(prob), idx, ctypes.byref(s), ws, nbytes,
                                      _stream_handle(stream)))


def ep_dispatch(prob, x, layout, recv_x, recv_scales=None, stream=None):
    torch = _torch()
    lib = load_library()
    T, H = prob.num_tokens, prob.hidden
    R = ep_num_recv_rows(prob)
    s = layout._struct(prob, check_all=False)
    xp = _ptr(x, "x", torch.bfloat16, T * H, allow_none=True)
    if prob.use_fp8:
        rp = _ptr(recv_x, "recv_x", (torch.uint8, torch.float8_e4m3fn), R * H, allow_none=True)
        sp = _ptr(recv_scales, "recv_scales", _scale_dtype(prob), R * (H // 128), allow_none=True)
    else:
        rp = _ptr(recv_x, "recv_x", torch.bfloat16, R * H, allow_none=True)
        sp = None
    _check("ep_dispatch", lib.ep_dispatch(ctypes.byref(prob), xp, ctypes.byref(s), rp, sp,
                                          _stream_handle(stream)))


def _layout_dispatch_args(prob, topk_idx, layout, workspace, x, recv_x, recv_scales):
    torch = _torch()
    T, H = prob.num_tokens, prob.hidden
    R = ep_num_recv_rows(prob)
    idx = _ptr(topk_idx, "topk_idx", torch.int32, T * prob.num_topk, allow_none=True)
    xp = _ptr(x, "x", torch.bfloat16, T * H, allow_none=True)
    s = layout._struct(prob)
    ws = _ptr(workspace, "workspace", allow_none=True)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if prob.use_fp8:
        rp = _ptr(recv_x, "recv_x", (torch.uint8, torch.float8_e4m3fn), R * H, allow_none=True)
        sp = _ptr(recv_scales, "recv_scales", _scale_dtype(prob), R * (H // 128), allow_none=True)
    else:
        rp = _ptr(recv_x, "recv_x", torch.bfloat16, R * H, allow_none=True)
        sp = None
    return s, (ctypes.byref(prob), idx, ctypes.byref(s), ws, nbytes, xp, rp, sp)


def ep_layout_dispatch(prob, topk_idx, layout, workspace, x, recv_x, recv_scales=None,
                       stream=None):
    lib = load_library()
    _s, args = _layout_dispatch_args(prob, topk_idx, layout, workspace, x, recv_x, recv_scales)
    _check("ep_layout_dispatch", lib.ep_layout_dispatch(*args, _stream_handle(stream)))


def ep_layout_dispatch_noalloc(prob, topk_idx, layout, x, recv_x, recv_scales=None,
                               stream=None):
    """ep_layout_dispatch with the library's own fixed device array as the
    workspace (nothing is allocated; calls that overlap on one GPU race)."""
    lib = load_library()
    _s, args = _layout_dispatch_args(prob, topk_idx, layout, None, x, recv_x, recv_scales)
    pr, idx, s, _ws, _nbytes, xp, rp, sp = args
    _check("ep_layout_dispatch_noalloc",
           lib.ep_layout_dispatch_noalloc(pr, idx, s, xp, rp, sp, _stream_handle(stream)))


def ep_combine(prob, expert_out, layout, topk_weights, y, stream=None):
    torch = _torch()
    lib = load_library()
    T, H, k = prob.num_tokens, prob.hidden, prob.num_topk
    R = ep_num_recv_rows(prob)
    s = layout._struct(prob, check_all=False)
    ep = _ptr(expert_out, "expert_out", torch.bfloat16, R * H, allow_none=True)
    wp = _ptr(topk_weights, "topk_weights", torch.float32, T * k, allow_none=True)
    yp = _ptr(y, "y", torch.bfloat16, T * H, allow_none=True)
    _check("ep_combine", lib.ep_combine(ctypes.byref(prob), ep, ctypes.byref(s), wp, yp,
                                        _stream_handle(stream)))


def ep_e4m3_encode(inp, out, stream=None):
    torch = _torch()
    lib = load_library()
    n = inp.numel()
    ip = _ptr(inp, "inp", torch.float32, allow_none=True)
    op = _ptr(out, "out", (torch.uint8, torch.float8_e4m3fn), n, allow_none=True)
    _check("ep_e4m3_encode", lib.ep_e4m3_encode(ip, op, n, _stream_handle(stream)))


class _Prepared:
    """A C-ABI call with its arguments checked and marshalled once.  Holds
    references to the tensors so their memory stays alive."""

    def __init__(self, name, fn, args, keep):
        self.name, self._fn, self._args, self._keep = name, fn, args, keep

    def __call__(self, stream=None):
        _check(self.name, self._fn(*self._args, _stream_handle(stream)))


def prepare_layout(prob, topk_idx, layout, workspace):
    torch = _torch()
    lib = load_library()
    idx = _ptr(topk_idx, "topk_idx", torch.int32, prob.num_tokens * prob.num_topk,
               allow_none=True)
    s = layout._struct(prob)
    nbytes = workspace.numel() * workspace.element_size()
    args = (ctypes.byref(prob), idx, ctypes.byref(s), _ptr(workspace, "workspace"), nbytes)
    return _Prepared("ep_layout", lib.ep_layout, args, (prob, s, topk_idx, layout, workspace))


def prepare_dispatch(prob, x, layout, recv_x, recv_scales=None):
    torch = _torch()
    lib = load_library()
    T, H = prob.num_tokens, prob.hidden
    R = ep_num_recv_rows(prob)
    xp = _ptr(x, "x", torch.bfloat16, T * H, allow_none=True)
    s = layout._struct(prob, check_all=False)
    if prob.use_fp8:
        rp = _ptr(recv_x, "recv_x", (torch.uint8, torch.float8_e4m3fn), R * H, allow_none=True)
        sp = _ptr(recv_scales, "recv_scales", _scale_dtype(prob), R * (H // 128), allow_none=True)
    else:
        rp = _ptr(recv_x, "recv_x", torch.bfloat16, R * H, allow_none=True)
        sp = None
    args = (ctypes.byref(prob), xp, ctypes.byref(s), rp, sp)
    return _Prepared("ep_dispatch", lib.ep_dispatch, args, (prob, s, x, layout, recv_x, recv_scales))


def prepare_combine(prob, expert_out, layout, topk_weights, y):
    torch = _torch()
    lib = load_library()
    T, H, k = prob.num_tokens, prob.hidden, prob.num_topk
    R = ep_num_recv_rows(prob)
    ep = _ptr(expert_out, "expert_out", torch.bfloat16, R * H, allow_none=True)
    wp = _ptr(topk_weights, "topk_weights", torch.float32, T * k, allow_none=True)
    yp = _ptr(y, "y", torch.bfloat16, T * H, allow_none=True)
    s = layout._struct(prob, check_all=False)
    args = (ctypes.byref(prob), ep, ctypes.byref(s), wp, yp)
    return _Prepared("ep_combine", lib.ep_combine, args,
                     (prob, s, expert_out, layout, topk_weights, y))


def prepare_layout_dispatch(prob, topk_idx, layout, workspace, x, recv_x, recv_scales=None):
    lib = load_library()
    s, args = _layout_dispatch_args(prob, topk_idx, layout, workspace, x, recv_x, recv_scales)
    return _Prepared("ep_layout_dispatch", lib.ep_layout_dispatch, args,
                     (prob, s, topk_idx, layout, workspace, x, recv_x, recv_scales))


# ------------------------------------------------- routing and expert products

def _device_of(t, name):
    """Index of the GPU that holds `t`."""
    try:
        dev = t.get_device()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if dev < 0:
        raise ValueError(f"{name} must be in GPU memory")
    return dev


def _runs(shape):
    """Sizes of the runs of memory that a contiguous tensor's dimensions mark."""
    n, out = 1, set()
    for d in reversed(shape):
        n *= d
        out.add(n)
    return out - {1}


def _arg(t, name, dtype, shape, dev, allow_none=False):
    """Pointer of a contiguous tensor on device `dev`, of `shape` (or of a number
    of elements, if that is an int).  Dimensions may be split or merged, as in
    [B, L, k] or [B * L * k] for [T, k]; other orders of them are refused."""
    if t is None and allow_none:
        return None
    try:  # what nearly every call passes, checked without naming what is wrong
        if (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                and t.get_device() == dev):
            return t.data_ptr()
    except AttributeError:
        pass
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    want = (shape,) if isinstance(shape, int) else shape
    if t.numel() != math.prod(want):
        raise ValueError(f"{name} has {t.numel()} elements, expected {math.prod(want)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.shape != want and t.numel():
        has, wants = _runs(t.shape), _runs(want)
        if not (has <= wants or wants <= has):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {want}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be in GPU memory, on cuda:{dev}")
    return t.data_ptr()


def _raw_stream(dev):
    """Handle of the current stream of device `dev`; the raw call costs 0.1 us,
    a torch.cuda.Stream object for it 1.1."""
    global _raw_stream
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        def raw(d):
            return torch.cuda.current_stream(d).cuda_stream
    _raw_stream = raw
    return raw(dev)


_gpus = None  # visible GPUs, once counted


def _issue(name, fn, args, dev, stream):
    """The C call on device `dev`, on its current stream by default."""
    global _gpus
    if _gpus is None:
        _gpus = _torch().cuda.device_count()
    if stream is None:
        handle = _raw_stream(dev)
    else:
        handle = stream if isinstance(stream, int) else stream.cuda_stream
    if _gpus == 1 or _torch().cuda.current_device() == dev:
        code = fn(*args, handle)
    else:
        with _torch().cuda.device(dev):
            code = fn(*args, handle)
    if code != EP_OK:
        raise EpError(name, code)


class _PreparedOn(_Prepared):
    """A prepared call that runs on the device of its tensors."""

    def __init__(self, name, fn, args, dev, keep):
        super().__init__(name, fn, args, keep)
        self._dev = dev

    def __call__(self, stream=None):
        _issue(self.name, self._fn, self._args, self._dev, stream)


def _logits_args(rt, logits):
    """Device, element type and row pitch of [T, E] logits, rows of any pitch."""
    torch = _torch()
    dev = _device_of(logits, "logits")
    if logits.dtype is torch.bfloat16:
        bf16 = 1
    elif logits.dtype is torch.float32:
        bf16 = 0
    else:
        raise TypeError(f"logits has dtype {logits.dtype}, expected float32 or bfloat16")
    T, E = rt.num_tokens, rt.num_experts
    if logits.shape != (T, E):
        raise ValueError(f"logits has shape {tuple(logits.shape)}, expected {(T, E)}")
    stride, inner = logits.stride()
    if inner != 1 and E > 1:
        raise ValueError("logits must be contiguous along the experts")
    if T <= 1:
        stride = E
    if stride < E:
        raise ValueError(f"logits rows overlap: row pitch {stride} below {E}")
    return dev, logits.data_ptr(), bf16, stride


def _valid_arg(rt, valid, dev):
    torch = _torch()
    u8 = torch.uint8
    dtype = u8 if getattr(valid, "dtype", None) is u8 else (u8, torch.bool)
    return _arg(valid, "valid", dtype, (rt.num_tokens,), dev)


def _route_args(rt, logits, topk_idx, topk_weights, expert_bias, valid):
    torch = _torch()
    dev, lp, bf16, stride = _logits_args(rt, logits)
    n = (rt.num_tokens, rt.num_topk)
    bp = vp = None
    if expert_bias is not None:
        bp = _arg(expert_bias, "expert_bias", torch.float32, (rt.num_experts,), dev)
    if valid is not None:
        vp = _valid_arg(rt, valid, dev)
    ip = _arg(topk_idx, "topk_idx", torch.int32, n, dev)
    wp = _arg(topk_weights, "topk_weights", torch.float32, n, dev)
    return dev, (ctypes.byref(rt), lp, bf16, stride, bp, vp, ip, wp)


def ep_route(rt, logits, topk_idx, topk_weights, expert_bias=None, valid=None, stream=None):
    lib = _lib or load_library()
    dev, args = _route_args(rt, logits, topk_idx, topk_weights, expert_bias, valid)
    _issue("ep_route", lib.ep_route, args, dev, stream)


def prepare_route(rt, logits, topk_idx, topk_weights, expert_bias=None, valid=None):
    lib = load_library()
    dev, args = _route_args(rt, logits, topk_idx, topk_weights, expert_bias, valid)
    return _PreparedOn("ep_route", lib.ep_route, args, dev,
                       (rt, logits, topk_idx, topk_weights, expert_bias, valid))


def ep_balance_workspace_bytes(rt):
    return int(load_library().ep_balance_workspace_bytes(ctypes.byref(rt)))


def _balance_args(rt, logits, topk_idx, coef, counts, mean_prob, num_valid, loss, workspace,
                  valid):
    torch = _torch()
    dev, lp, bf16, stride = _logits_args(rt, logits)
    T, E, B = rt.num_tokens, rt.num_experts, rt.num_seqs
    ip = _arg(topk_idx, "topk_idx", torch.int32, (T, rt.num_topk), dev)
    vp = None if valid is None else _valid_arg(rt, valid, dev)
    cp = _arg(counts, "counts", torch.int32, (B, E), dev)
    mp = _arg(mean_prob, "mean_prob", torch.float32, (B, E), dev)
    np_ = _arg(num_valid, "num_valid", torch.int32, (B,), dev)
    op = _arg(loss, "loss", torch.float32, (1,), dev)
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    wp = _arg(workspace, "workspace", workspace.dtype, workspace.shape, dev)
    nbytes = workspace.numel() * workspace.element_size()
    return dev, (ctypes.byref(rt), lp, bf16, stride, ip, vp, coef, cp, mp, np_, op, wp, nbytes)


def ep_balance_loss(rt, logits, topk_idx, coef, counts, mean_prob, num_valid, loss, workspace,
                    valid=None, stream=None):
    lib = _lib or load_library()
    dev, args = _balance_args(rt, logits, topk_idx, coef, counts, mean_prob, num_valid, loss,
                              workspace, valid)
    _issue("ep_balance_loss", lib.ep_balance_loss, args, dev, stream)


def prepare_balance_loss(rt, logits, topk_idx, coef, counts, mean_prob, num_valid, loss, workspace,
                         valid=None):
    lib = load_library()
    dev, args = _balance_args(rt, logits, topk_idx, coef, counts, mean_prob, num_valid, loss,
                              workspace, valid)
    return _PreparedOn("ep_balance_loss", lib.ep_balance_loss, args, dev,
                       (rt, logits, topk_idx, counts, mean_prob, num_valid, loss, workspace, valid))


def _route_backward_args(rt, logits, topk_idx, d_logits, d_weights, coef, counts, num_valid,
                         d_loss, valid):
    torch = _torch()
    dev, lp, bf16, stride = _logits_args(rt, logits)
    T, E, B = rt.num_tokens, rt.num_experts, rt.num_seqs
    n = (T, rt.num_topk)
    if d_weights is None and d_loss is None:
        raise ValueError("d_weights or d_loss is required")
    if d_weights is not None and topk_idx is None:
        raise ValueError("topk_idx is required with d_weights")
    if d_loss is not None and (counts is None or num_valid is None):
        raise ValueError("counts and num_valid are required with d_loss")
    ip = _arg(topk_idx, "topk_idx", torch.int32, n, dev, allow_none=True)
    gp = _arg(d_weights, "d_weights", torch.float32, n, dev, allow_none=True)
    vp = None if valid is None else _valid_arg(rt, valid, dev)
    cp = _arg(counts, "counts", torch.int32, (B, E), dev, allow_none=True)
    np_ = _arg(num_valid, "num_valid", torch.int32, (B,), dev, allow_none=True)
    sp = _arg(d_loss, "d_loss", torch.float32, (1,), dev, allow_none=True)
    dp = _arg(d_logits, "d_logits", logits.dtype, (T, E), dev)
    return dev, (ctypes.byref(rt), lp, bf16, stride, ip, gp, vp, coef, cp, np_, sp, dp)


def ep_route_backward(rt, logits, topk_idx, d_logits, d_weights=None, coef=0.0, counts=None,
                      num_valid=None, d_loss=None, valid=None, stream=None):
    lib = _lib or load_library()
    dev, args = _route_backward_args(rt, logits, topk_idx, d_logits, d_weights, coef, counts,
                                     num_valid, d_loss, valid)
    _issue("ep_route_backward", lib.ep_route_backward, args, dev, stream)


def prepare_route_backward(rt, logits, topk_idx, d_logits, d_weights=None, coef=0.0, counts=None,
                           num_valid=None, d_loss=None, valid=None):
    lib = load_library()
    dev, args = _route_backward_args(rt, logits, topk_idx, d_logits, d_weights, coef, counts,
                                     num_valid, d_loss, valid)
    return _PreparedOn("ep_route_backward", lib.ep_route_backward, args, dev,
                       (rt, logits, topk_idx, d_logits, d_weights, counts, num_valid, d_loss, valid))


def _expert_w4_args(prob, mm, rows, layout, codes, scales, out, row_scales):
    torch = _torch()
    dev = _device_of(rows, "rows")
    K, N, E, fmt = mm.in_features, mm.out_features, prob.num_experts, mm.in_format
    R = E * prob.capacity if prob.capacity else prob.num_tokens * prob.num_topk
    n2 = 2 * N if mm.activation == 1 else N
    u8 = torch.uint8
    s = _LayoutPtrs(_arg(layout.count, "count", torch.int32, (E,), dev),
                    _arg(layout.offset, "offset", torch.int32, (E + 1,), dev))
    if fmt == 0:
        rp = _arg(rows, "rows", torch.bfloat16, (R, K), dev)
        sp = None
    else:
        rp = _arg(rows, "rows", (u8, torch.float8_e4m3fn), (R, K), dev)
        sp = _arg(row_scales, "row_scales", u8 if fmt == 2 else torch.float32, (R, K // 128), dev)
    cp = _arg(codes, "codes", u8, (E, n2, K // 2), dev)
    wp = _arg(scales, "scales", u8, (E, n2, K // 32), dev)
    op = _arg(out, "out", torch.bfloat16, (R, N), dev)
    return dev, s, (ctypes.byref(prob), ctypes.byref(mm), rp, sp, ctypes.byref(s), cp, wp, op)


def ep_expert_w4(prob, mm, rows, layout, codes, scales, out, row_scales=None, stream=None):
    lib = _lib or load_library()
    dev, _s, args = _expert_w4_args(prob, mm, rows, layout, codes, scales, out, row_scales)
    _issue("ep_expert_w4", lib.ep_expert_w4, args, dev, stream)


def prepare_expert_w4(prob, mm, rows, layout, codes, scales, out, row_scales=None):
    lib = load_library()
    dev, s, args = _expert_w4_args(prob, mm, rows, layout, codes, scales, out, row_scales)
    return _PreparedOn("ep_expert_w4", lib.ep_expert_w4, args, dev,
                       (prob, mm, s, rows, layout, codes, scales, out, row_scales))


# ------------------------- layer norm, dropout in the combine, 8-bit integers

def _rows_arg(t, name, nm, dtype, dev):
    """Pointer and row pitch of a [T, H] tensor, rows of any pitch."""
    T, H = nm.num_tokens, nm.hidden
    try:  # what nearly every call passes
        if (t.dtype is dtype and t.shape == (T, H) and t.is_contiguous()
                and t.get_device() == dev):
            return t.data_ptr(), H
    except AttributeError:
        pass
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != (T, H):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(T, H)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be in GPU memory, on cuda:{dev}")
    stride, inner = t.stride()
    if inner != 1 and H > 1:
        raise ValueError(f"{name} must be contiguous along the channels")
    if T <= 1:
        stride = H
    if stride < H:
        raise ValueError(f"{name} rows overlap: row pitch {stride} below {H}")
    return t.data_ptr(), stride


def _is_bf16(t, name):
    """1 for a bf16 tensor, 0 for an fp32 one."""
    torch = _torch()
    dtype = getattr(t, "dtype", None)
    if dtype is torch.bfloat16:
        return 1
    if dtype is torch.float32:
        return 0
    raise TypeError(f"{name} has dtype {dtype}, expected float32 or bfloat16")


def _layer_norm_args(nm, x, weight, bias, y, mean, rstd):
    torch = _torch()
    dev = _device_of(x, "x")
    T, H = nm.num_tokens, nm.hidden
    x_bf16, w_bf16, wp, bp, mp, rp = _is_bf16(x, "x"), 0, None, None, None, None
    xp, stride = _rows_arg(x, "x", nm, x.dtype, dev)
    param = weight if weight is not None else bias
    if param is not None:
        w_bf16 = _is_bf16(param, "weight" if weight is not None else "bias")
        if weight is not None:
            wp = _arg(weight, "weight", param.dtype, (H,), dev)
        if bias is not None:
            bp = _arg(bias, "bias", param.dtype, (H,), dev)
    yp = _arg(y, "y", x.dtype, (T, H), dev)
    if mean is not None:
        mp = _arg(mean, "mean", torch.float32, (T,), dev)
    if rstd is not None:
        rp = _arg(rstd, "rstd", torch.float32, (T,), dev)
    return dev, (ctypes.byref(nm), xp, x_bf16, stride, wp, bp, w_bf16, yp, mp, rp)


def ep_layer_norm(nm, x, weight, bias, y, mean=None, rstd=None, stream=None):
    lib = _lib or load_library()
    dev, args = _layer_norm_args(nm, x, weight, bias, y, mean, rstd)
    _issue("ep_layer_norm", lib.ep_layer_norm, args, dev, stream)


def prepare_layer_norm(nm, x, weight, bias, y, mean=None, rstd=None):
    lib = load_library()
    dev, args = _layer_norm_args(nm, x, weight, bias, y, mean, rstd)
    return _PreparedOn("ep_layer_norm", lib.ep_layer_norm, args, dev,
                       (nm, x, weight, bias, y, mean, rstd))


def ep_layer_norm_workspace_bytes(nm):
    return int(load_library().ep_layer_norm_workspace_bytes(ctypes.byref(nm)))


def _workspace_arg(workspace, dev):
    """Pointer and bytes of a workspace that may be missing."""
    if workspace is None:
        return None, 0
    if not isinstance(workspace, _torch().Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    wp = _arg(workspace, "workspace", workspace.dtype, workspace.shape, dev)
    return wp, workspace.numel() * workspace.element_size()


def _layer_norm_backward_args(nm, x, dy, weight, mean, rstd, dx, d_weight, d_bias, workspace,
                              d_skip):
    torch = _torch()
    dev = _device_of(x, "x")
    T, H = nm.num_tokens, nm.hidden
    x_bf16, x_dtype, w_bf16, w_dtype = _is_bf16(x, "x"), x.dtype, 0, torch.float32
    for param, name in ((weight, "weight"), (d_weight, "d_weight"), (d_bias, "d_bias")):
        if param is not None:
            w_bf16, w_dtype = _is_bf16(param, name), param.dtype
            break
    xp, x_stride = _rows_arg(x, "x", nm, x_dtype, dev)
    gp, g_stride = _rows_arg(dy, "dy", nm, x_dtype, dev)
    wp = _arg(weight, "weight", w_dtype, (H,), dev, allow_none=True)
    mp = _arg(mean, "mean", torch.float32, (T,), dev)
    rp = _arg(rstd, "rstd", torch.float32, (T,), dev)
    sp = _arg(d_skip, "d_skip", x_dtype, (T, H), dev, allow_none=True)
    dp = _arg(dx, "dx", x_dtype, (T, H), dev)
    dwp = _arg(d_weight, "d_weight", w_dtype, (H,), dev, allow_none=True)
    dbp = _arg(d_bias, "d_bias", w_dtype, (H,), dev, allow_none=True)
    space, nbytes = _workspace_arg(workspace, dev)
    return dev, (ctypes.byref(nm), xp, x_bf16, x_stride, gp, g_stride, wp, w_bf16, mp, rp, sp, dp,
                 dwp, dbp, space, nbytes)


def ep_layer_norm_backward(nm, x, dy, weight, mean, rstd, dx, d_weight=None, d_bias=None,
                           workspace=None, d_skip=None, stream=None):
    lib = _lib or load_library()
    dev, args = _layer_norm_backward_args(nm, x, dy, weight, mean, rstd, dx, d_weight, d_bias,
                                          workspace, d_skip)
    _issue("ep_layer_norm_backward", lib.ep_layer_norm_backward, args, dev, stream)


def prepare_layer_norm_backward(nm, x, dy, weight, mean, rstd, dx, d_weight=None, d_bias=None,
                                workspace=None, d_skip=None):
    lib = load_library()
    dev, args = _layer_norm_backward_args(nm, x, dy, weight, mean, rstd, dx, d_weight, d_bias,
                                          workspace, d_skip)
    return _PreparedOn("ep_layer_norm_backward", lib.ep_layer_norm_backward, args, dev,
                       (nm, x, dy, weight, mean, rstd, dx, d_weight, d_bias, workspace, d_skip))


def _recv_rows(prob):
    return (prob.num_experts * prob.capacity if prob.capacity
            else prob.num_tokens * prob.num_topk)


def _slots(prob, layout, dev):
    s = _LayoutPtrs()
    s.slot_of = _arg(layout.slot_of, "slot_of", _torch().int32,
                     (prob.num_tokens, prob.num_topk), dev)
    return s


def _rng_arg(rng, dev):
    """{seed, offset} as two 64-bit words, int64 or uint64."""
    if rng is None:
        return None
    torch = _torch()
    i64 = torch.int64
    dtype = i64 if getattr(rng, "dtype", None) is i64 else (i64, torch.uint64)
    return _arg(rng, "rng", dtype, (2,), dev)


def _combine_dropout_args(prob, expert_out, layout, topk_weights, p, rng, y, residual):
    torch = _torch()
    dev = _device_of(y, "y")
    T, H, bf16 = prob.num_tokens, prob.hidden, torch.bfloat16
    s = _slots(prob, layout, dev)
    ep = _arg(expert_out, "expert_out", bf16, (_recv_rows(prob), H), dev)
    wp = _arg(topk_weights, "topk_weights", torch.float32, (T, prob.num_topk), dev)
    rp = _arg(residual, "residual", bf16, (T, H), dev, allow_none=True)
    gp = _rng_arg(rng, dev)
    yp = _arg(y, "y", bf16, (T, H), dev)
    return dev, s, (ctypes.byref(prob), ep, ctypes.byref(s), wp, rp, p, gp, yp)


def ep_combine_dropout(prob, expert_out, layout, topk_weights, p, rng, y, residual=None,
                       stream=None):
    lib = _lib or load_library()
    dev, _s, args = _combine_dropout_args(prob, expert_out, layout, topk_weights, p, rng, y,
                                          residual)
    _issue("ep_combine_dropout", lib.ep_combine_dropout, args, dev, stream)


def prepare_combine_dropout(prob, expert_out, layout, topk_weights, p, rng, y, residual=None):
    lib = load_library()
    dev, s, args = _combine_dropout_args(prob, expert_out, layout, topk_weights, p, rng, y,
                                         residual)
    return _PreparedOn("ep_combine_dropout", lib.ep_combine_dropout, args, dev,
                       (prob, s, expert_out, layout, topk_weights, rng, y, residual))


def _combine_backward_args(prob, dy, expert_out, layout, topk_weights, p, rng, d_expert_out,
                           d_weights):
    torch = _torch()
    dev = _device_of(dy, "dy")
    T, H, k, bf16 = prob.num_tokens, prob.hidden, prob.num_topk, torch.bfloat16
    R = _recv_rows(prob)
    s = _slots(prob, layout, dev)
    gp = _arg(dy, "dy", bf16, (T, H), dev)
    ep = _arg(expert_out, "expert_out", bf16, (R, H), dev, allow_none=True)
    wp = _arg(topk_weights, "topk_weights", torch.float32, (T, k), dev)
    rp = _rng_arg(rng, dev)
    dp = _arg(d_expert_out, "d_expert_out", bf16, (R, H), dev)
    dwp = _arg(d_weights, "d_weights", torch.float32, (T, k), dev, allow_none=True)
    return dev, s, (ctypes.byref(prob), gp, ep, ctypes.byref(s), wp, p, rp, dp, dwp)


def ep_combine_backward(prob, dy, expert_out, layout, topk_weights, p, rng, d_expert_out,
                        d_weights=None, stream=None):
    lib = _lib or load_library()
    dev, _s, args = _combine_backward_args(prob, dy, expert_out, layout, topk_weights, p, rng,
                                           d_expert_out, d_weights)
    _issue("ep_combine_backward", lib.ep_combine_backward, args, dev, stream)


def prepare_combine_backward(prob, dy, expert_out, layout, topk_weights, p, rng, d_expert_out,
                             d_weights=None):
    lib = load_library()
    dev, s, args = _combine_backward_args(prob, dy, expert_out, layout, topk_weights, p, rng,
                                          d_expert_out, d_weights)
    return _PreparedOn("ep_combine_backward", lib.ep_combine_backward, args, dev,
                       (prob, s, dy, expert_out, layout, topk_weights, rng, d_expert_out,
                        d_weights))


def _dispatch_i8_args(prob, x, layout, recv_q, recv_scales):
    torch = _torch()
    dev = _device_of(x, "x")
    T, H, R = prob.num_tokens, prob.hidden, _recv_rows(prob)
    s = _slots(prob, layout, dev)
    xp = _arg(x, "x", torch.bfloat16, (T, H), dev)
    qp = _arg(recv_q, "recv_q", torch.int8, (R, H), dev)
    sp = _arg(recv_scales, "recv_scales", torch.float32, (R,), dev)
    return dev, s, (ctypes.byref(prob), xp, ctypes.byref(s), qp, sp)


def ep_dispatch_i8(prob, x, layout, recv_q, recv_scales, stream=None):
    lib = _lib or load_library()
    dev, _s, args = _dispatch_i8_args(prob, x, layout, recv_q, recv_scales)
    _issue("ep_dispatch_i8", lib.ep_dispatch_i8, args, dev, stream)


def prepare_dispatch_i8(prob, x, layout, recv_q, recv_scales):
    lib = load_library()
    dev, s, args = _dispatch_i8_args(prob, x, layout, recv_q, recv_scales)
    return _PreparedOn("ep_dispatch_i8", lib.ep_dispatch_i8, args, dev,
                       (prob, s, x, layout, recv_q, recv_scales))


def ep_expert_i8_workspace_bytes(prob, mm):
    return int(load_library().ep_expert_i8_workspace_bytes(ctypes.byref(prob), ctypes.byref(mm)))


def _expert_i8_args(prob, mm, rows, layout, weights, scales, out, row_scales, workspace):
    torch = _torch()
    dev = _device_of(rows, "rows")
    K, N, E, R = mm.in_features, mm.out_features, prob.num_experts, _recv_rows(prob)
    n2 = 2 * N if mm.activation == 1 else N
    i8, f32, bf16 = torch.int8, torch.float32, torch.bfloat16
    s = _LayoutPtrs(_arg(layout.count, "count", torch.int32, (E,), dev),
                    _arg(layout.offset, "offset", torch.int32, (E + 1,), dev))
    sp = None
    if mm.in_format == 0:
        rp = _arg(rows, "rows", bf16, (R, K), dev)
    else:
        rp = _arg(rows, "rows", i8, (R, K), dev)
        sp = _arg(row_scales, "row_scales", f32, (R,), dev)
    wp = _arg(weights, "weights", i8, (E, n2, K), dev)
    cp = _arg(scales, "scales", f32, (E, n2), dev)
    op = _arg(out, "out", bf16, (R, N), dev)
    space, nbytes = _workspace_arg(workspace, dev) if mm.in_format == 0 else (None, 0)
    return dev, s, (ctypes.byref(prob), ctypes.byref(mm), rp, sp, ctypes.byref(s), wp, cp, op,
                    space, nbytes)


def ep_expert_i8(prob, mm, rows, layout, weights, scales, out, row_scales=None, workspace=None,
                 stream=None):
    lib = _lib or load_library()
    dev, _s, args = _expert_i8_args(prob, mm, rows, layout, weights, scales, out, row_scales,
                                    workspace)
    _issue("ep_expert_i8", lib.ep_expert_i8, args, dev, stream)


def prepare_expert_i8(prob, mm, rows, layout, weights, scales, out, row_scales=None,
                      workspace=None):
    lib = load_library()
    dev, s, args = _expert_i8_args(prob, mm, rows, layout, weights, scales, out, row_scales,
                                   workspace)
    return _PreparedOn("ep_expert_i8", lib.ep_expert_i8, args, dev,
                       (prob, mm, s, rows, layout, weights, scales, out, row_scales, workspace))
