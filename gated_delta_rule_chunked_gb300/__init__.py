"""GB300-native Kimi Delta Attention (KDA): chunked forward, backward and decode.

Python face of libkda.so (include/kda.h). Every step of the computation runs in
the library's CUDA kernels; this module only allocates outputs and workspaces
with PyTorch, passes raw device pointers and the current CUDA stream through
ctypes, and turns status codes into exceptions.

    o, hT, saved = kda_fwd(q, k, v, beta, g, cu_seqlens, h0, save=True)
    grads = kda_bwd(q, k, v, beta, g, dO, saved, cu_seqlens, h0, dhT)
    o = kda_step(q, k, v, beta, g, state, accept_len)     # state updated in place

and what stands around a recurrent layer: the selective scan behind its short convolution
(``ssm_fwd`` for prompts, ``ssm_step`` for decoding), the verification of drafted tokens
(``draft_verify``), and the norms, gate and residual sum around a block (``block_norm_fwd``,
``block_norm_bwd``). examples/draft_decode.py runs them together.

Shapes: q, k, v, g, dO [total, H, 128]; beta [total, H]; states [N, H, 128, 128]
(fp32, [key][value]); decode inputs carry an extra step axis: [N, L, H, ...].
"""
from __future__ import annotations

import ctypes as C
from typing import Optional

import torch

from . import _lib
from ._lib import KdaError

__all__ = ["kda_fwd", "kda_bwd", "kda_step", "fwd_args", "bwd_args", "KdaError", "library", "ssm_fwd", "ssm_step",
           "draft_verify", "block_norm_fwd", "block_norm_bwd"]


def library():
    """The loaded libkda.so handle (raises if it was not built)."""
    return _lib.load()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _io_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return _lib.KDA_BF16
    if t.dtype == torch.float32:
        return _lib.KDA_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _check_inputs(q, k, v, beta, g):
    for name, t in (("q", q), ("k", k), ("v", v), ("beta", beta), ("g", g)):
        if t is None and name == "v":
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if beta.dtype != torch.float32 or g.dtype != torch.float32:
        raise TypeError("beta and g must be float32")
    if k.dtype != q.dtype or (v is not None and v.dtype != q.dtype):
        raise TypeError("q, k and v must share one dtype")


def fwd_args(q, k, v, beta, g, cu_seqlens=None, h0=None, o=None, hT=None, saved=None,
             workspace=None, scale: float = 1.0, n_seqs: Optional[int] = None, dev_status=None,
             h0_identity: bool = False) -> _lib.FwdArgs:
    """Fill the C argument struct for kda_fwd from tensors (no allocation)."""
    a = _lib.FwdArgs()
    total, H, dk = q.shape
    a.n_seqs = (cu_seqlens.numel() - 1) if cu_seqlens is not None else (n_seqs or 1)
    a.total_tokens, a.heads, a.dk, a.dv, a.chunk = total, H, dk, (v.shape[2] if v is not None else dk), 64
    a.h0_identity = int(h0_identity)
    a.scale, a.io_dtype = scale, _io_dtype(q)
    a.cu_seqlens = _ptr(cu_seqlens)
    a.q, a.k, a.v, a.beta, a.g = _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g)
    a.h0, a.o, a.hT, a.saved = _ptr(h0), _ptr(o), _ptr(hT), _ptr(saved)
    a.workspace = _ptr(workspace)
    a.workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    a.dev_status = _ptr(dev_status)
    return a


def bwd_args(fa: _lib.FwdArgs, dO, dq, dk, dv, dbeta, dg, dh0=None, dhT=None, workspace=None) -> _lib.BwdArgs:
    b = _lib.BwdArgs()
    b.fwd = fa
    b.dO, b.dhT = _ptr(dO), _ptr(dhT)
    b.dq, b.dk, b.dv, b.dbeta, b.dg, b.dh0 = _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dbeta), _ptr(dg), _ptr(dh0)
    b.workspace = _ptr(workspace)
    b.workspace_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    return b


def _i32(cu_seqlens, device):
    if cu_seqlens is None:
        return None
    if cu_seqlens.device.type == "cpu":
        # through pinned memory, so the copy is enqueued on the current stream instead of
        # blocking the host until the stream reaches it
        return cu_seqlens.to(dtype=torch.int32).contiguous().pin_memory().to(device, non_blocking=True)
    return cu_seqlens.to(device=device, dtype=torch.int32).contiguous()


def kda_fwd(q, k, v, beta, g, cu_seqlens=None, h0=None, *, scale: float = 1.0, save: bool = False,
            final_state: bool = True, n_seqs: Optional[int] = None, dev_status=None):
    """Chunked KDA forward. Returns (o, hT or None, saved or None).

    ``saved`` (chunk-start states) is what kda_bwd needs; request it with save=True.
    Without cu_seqlens the tokens form ``n_seqs`` (default 1) equal sequences.
    ``dev_status`` (optional int32 device tensor, zeroed by the caller) receives
    KDA_ERR_TIMEOUT if a kernel gives up a bounded wait.
    """
    lib = library()
    _check_inputs(q, k, v, beta, g)
    dev = q.device
    cu = _i32(cu_seqlens, dev)
    N = (cu.numel() - 1) if cu is not None else (n_seqs or 1)
    H = q.shape[1]
    o = torch.empty_like(v)
    hT = torch.empty((N, H, 128, 128), dtype=torch.float32, device=dev) if final_state else None
    a = fwd_args(q, k, v, beta, g, cu, h0, o, hT, None, None, scale, n_seqs=N, dev_status=dev_status)
    saved = None
    if save:
        saved = torch.empty(lib.kda_saved_size(C.byref(a)), dtype=torch.uint8, device=dev)
        a.saved = saved.data_ptr()
    ws_bytes = lib.kda_fwd_workspace_size(C.byref(a))
    if ws_bytes == 0:
        _lib.check(lib.kda_fwd(C.byref(a), _stream(dev)))   # reports the argument error
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws_bytes
    _lib.check(lib.kda_fwd(C.byref(a), _stream(dev)))
    return o, hT, saved


def _fwd_states(q, k, v, beta, g, cu, h0, N, *, scale, h0_identity=False, out=None, ws=None):
    """One forward pass for its final states (and outputs into ``out`` when given). With
    ``ws`` (the workspace of an earlier pass on the same q, k, g, beta, cu) the chunk records
    are reused and only the scan runs; returns (hT, workspace)."""
    lib = library()
    dev = q.device
    hT = torch.empty((N, q.shape[1], 128, 128), dtype=torch.float32, device=dev)
    a = fwd_args(q, k, v, beta, g, cu, h0, out, hT, None, None, scale, n_seqs=N, h0_identity=h0_identity)
    ws_bytes = lib.kda_fwd_workspace_size(C.byref(a))
    if ws is None:
        ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    else:
        a.skip_prep = 1
    a.workspace, a.workspace_bytes = ws.data_ptr(), ws_bytes
    _lib.check(lib.kda_fwd(C.byref(a), _stream(dev)))
    return hT, ws


def kda_cp_combine(M, b, h0, n_segments: int):
    """States entering each segment: S_in[:, 0] = h0, S_in[:, k+1] = M[:, k] S_in[:, k] + b[:, k].

    M, b: [N, P, H, 128, 128] fp32 (maps and offsets of the segments); h0: [N, H, 128, 128]
    fp32 or None. Returns S_in [N, P, H, 128, 128].
    """
    lib = library()
    N, P, H = M.shape[:3]
    if P != n_segments or b.shape != M.shape or (h0 is not None and h0.shape != (N, H, 128, 128)):
        raise ValueError("M, b must be [N, P, H, 128, 128] and h0 [N, H, 128, 128]")
    s_in = torch.empty_like(M)
    a = _lib.CpArgs(N, P, H, 128, 128, M.data_ptr(), b.data_ptr(), _ptr(h0), s_in.data_ptr())
    _lib.check(lib.kda_cp_combine(C.byref(a), _stream(M.device)))
    return s_in


def kda_fwd_cp(q, k, v, beta, g, cu_seqlens=None, h0=None, *, n_segments: int, scale: float = 1.0,
               n_seqs: Optional[int] = None, dev_status=None):
    """Forward by context parallelism, emulated on one device (libkda's kda_fwd_cp): every
    sequence is cut into n_segments consecutive runs of whole chunks that are processed
    independently (as separate sequences), their affine maps combined, and the segments run
    again from the combined incoming states. Returns (o, hT) of the unsplit forward.
    """
    lib = library()
    _check_inputs(q, k, v, beta, g)
    dev = q.device
    cu = _i32(cu_seqlens, dev)
    N = (cu.numel() - 1) if cu is not None else (n_seqs or 1)
    H = q.shape[1]
    o = torch.empty_like(v)
    hT = torch.empty((N, H, 128, 128), dtype=torch.float32, device=dev)
    c = _lib.FwdCpArgs()
    c.fwd = fwd_args(q, k, v, beta, g, cu, None if h0 is None else h0.contiguous(), o, hT, None, None, scale,
                     n_seqs=N, dev_status=dev_status)
    c.n_segments = n_segments
    ws_bytes = lib.kda_fwd_cp_workspace_size(C.byref(c))
    if ws_bytes == 0:
        raise KdaError(_lib.KDA_ERR_INVALID_ARG, lib.kda_last_error().decode())
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    c.workspace, c.workspace_bytes = ws.data_ptr(), ws_bytes
    _lib.check(lib.kda_fwd_cp(C.byref(c), _stream(dev)))
    return o, hT


def _attnres_args(sources, w, eps, out=None, stats=None):
    S = len(sources)
    if not 1 <= S <= _lib.ATTNRES_MAX_SOURCES:
        raise ValueError("Attention Residuals takes 1..9 sources")
    T, d = sources[0].shape
    for x in sources:
        if x.shape != (T, d) or x.dtype != sources[0].dtype or not x.is_cuda or not x.is_contiguous():
            raise ValueError("sources must be contiguous CUDA tensors of one shape [T, d] and dtype")
    if w.dtype != torch.float32 or w.shape != (d,) or not w.is_contiguous():
        raise TypeError("w must be a contiguous float32 [d] tensor")
    a = _lib.AttnresFwdArgs()
    a.n_sources, a.tokens, a.dim, a.eps, a.io_dtype = S, T, d, eps, _io_dtype(sources[0])
    for i, x in enumerate(sources):
        a.src[i] = x.data_ptr()
    a.w, a.out = w.data_ptr(), _ptr(out)
    a.alpha, a.rstd, a.logit = (_ptr(t) for t in stats)
    return a


def attnres_fwd(sources, w, *, eps: float = 1e-6):
    """Attention Residuals forward: out = sum_i softmax_i(r_i (w . x_i)) x_i over the sources
    (r_i = 1 / RMS(x_i)). Returns (out [T, d], stats) with stats = (alpha, rstd, logit), each
    [T, S] fp32, which the backward takes."""
    lib = library()
    T, d = sources[0].shape
    dev = sources[0].device
    out = torch.empty_like(sources[0])
    stats = tuple(torch.empty((T, len(sources)), dtype=torch.float32, device=dev) for _ in range(3))
    a = _attnres_args(sources, w, eps, out, stats)
    _lib.check(lib.kda_attnres_fwd(C.byref(a), _stream(dev)))
    return out, stats


def attnres_bwd(sources, w, stats, d_out, *, eps: float = 1e-6):
    """Backward of attnres_fwd: returns (d_sources list, dw [d] fp32)."""
    lib = library()
    dev = sources[0].device
    if d_out.shape != sources[0].shape or d_out.dtype != sources[0].dtype or not d_out.is_contiguous():
        raise ValueError("d_out must match the sources")
    b = _lib.AttnresBwdArgs()
    b.fwd = _attnres_args(sources, w, eps, None, stats)
    d_src = [torch.empty_like(x) for x in sources]
    dw = torch.empty_like(w)
    b.d_out, b.dw = d_out.data_ptr(), dw.data_ptr()
    for i, x in enumerate(d_src):
        b.d_src[i] = x.data_ptr()
    ws_bytes = lib.kda_attnres_bwd_workspace_size(C.byref(b))
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=dev)
    b.workspace, b.workspace_bytes = ws.data_ptr(), ws_bytes
    _lib.check(lib.kda_attnres_bwd(C.byref(b), _stream(dev)))
    return d_src, dw


_ACT = {"none": _lib.KDA_ACT_NONE, "silu": _lib.KDA_ACT_SILU}


def _conv_args(x, weight, bias, cu, state_in, activation, n_seqs):
    if x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA tensor [T, C]")
    T, Cc = x.shape
    if weight.dtype != torch.float32 or weight.dim() != 2 or weight.shape[0] != Cc or not weight.is_contiguous():
        raise TypeError("weight must be a contiguous float32 [C, W] tensor")
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (Cc,)):
        raise TypeError("bias must be float32 [C]")
    W = weight.shape[1]
    if state_in is not None and (state_in.dtype != x.dtype or state_in.shape != (n_seqs, W - 1, Cc)
                                 or not state_in.is_contiguous()):
        raise ValueError("state_in must be a contiguous [N, W-1, C] tensor of x's dtype")
    a = _lib.ConvArgs()
    a.n_seqs, a.total_tokens, a.channels, a.width = n_seqs, T, Cc, W
    a.activation, a.io_dtype = _ACT[activation], _io_dtype(x)
    a.cu_seqlens, a.x, a.weight, a.bias, a.state_in = _ptr(cu), x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(state_in)
    return a


def conv_fwd(x, weight, bias=None, cu_seqlens=None, state_in=None, *, activation: str = "silu",
             n_seqs: Optional[int] = None):
    """Short causal depthwise convolution (width W = weight.shape[1]) with the convolution
    state of each sequence. Returns (y [T, C] in x's dtype, state_out [N, W-1, C])."""
    lib = library()
    cu = _i32(cu_seqlens, x.device)
    N = (cu.numel() - 1) if cu is not None else (n_seqs or 1)
    a = _conv_args(x, weight, bias, cu, state_in, activation, N)
    y = torch.empty_like(x)
    state_out = torch.empty((N, weight.shape[1] - 1, x.shape[1]), dtype=x.dtype, device=x.device)
    a.y, a.state_out = y.data_ptr(), _ptr(state_out) if state_out.numel() else None
    _lib.check(lib.kda_conv_fwd(C.byref(a), _stream(x.device)))
    return y, state_out


def conv_bwd(x, weight, bias, dy, cu_seqlens=None, state_in=None, d_state_out=None, *, activation: str = "silu",
             n_seqs: Optional[int] = None):
    """Backward of conv_fwd: returns a dict of fp32 gradients dx, dweight, dbias (None without a
    bias) and d_state_in."""
    lib = library()
    cu = _i32(cu_seqlens, x.device)
    N = (cu.numel() - 1) if cu is not None else (n_seqs or 1)
    if dy.shape != x.shape or dy.dtype != x.dtype or not dy.is_contiguous():
        raise ValueError("dy must match x")
    b = _lib.ConvBwdArgs()
    b.fwd = _conv_args(x, weight, bias, cu, state_in, activation, N)
    f32 = dict(dtype=torch.float32, device=x.device)
    W = weight.shape[1]
    dx, dweight = torch.empty(x.shape, **f32), torch.empty(weight.shape, **f32)
    dbias = torch.empty(x.shape[1], **f32) if bias is not None else None
    d_state_in = torch.empty((N, W - 1, x.shape[1]), **f32)
    if d_state_out is not None:
        d_state_out = d_state_out.to(torch.float32).contiguous()
    b.dy, b.d_state_out, b.dx, b.dweight = dy.data_ptr(), _ptr(d_state_out), dx.data_ptr(), dweight.data_ptr()
    b.dbias, b.d_state_in = _ptr(dbias), _ptr(d_state_in) if d_state_in.numel() else None
    ws_bytes = lib.kda_conv_bwd_workspace_size(C.byref(b))
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=x.device)
    b.workspace, b.workspace_bytes = ws.data_ptr(), ws_bytes
    _lib.check(lib.kda_conv_bwd(C.byref(b), _stream(x.device)))
    return {"dx": dx, "dweight": dweight, "dbias": dbias, "d_state_in": d_state_in}


def conv_step(x, weight, bias, state, accept_len=None, *, activation: str = "silu", state_indices=None,
              first_slot=None, out=None, dev_status=None):
    """Decode / verify L token slots per sequence through the short convolution: x [N, L, C];
    ``state`` [N, W-1, C] (or a pool [P, W-1, C] addressed by ``state_indices``) advanced in
    place through ``accept_len`` slots; slots before ``first_slot`` are padding. Returns y."""
    lib = library()
    if x.dim() != 3 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous CUDA tensor [N, L, C]")
    N, L, Cc = x.shape
    W = weight.shape[1]
    if state.dtype != x.dtype or state.shape[1:] != (W - 1, Cc) or not state.is_contiguous():
        raise ValueError("state must be a contiguous [P, W-1, C] tensor of x's dtype")
    i32 = lambda t: None if t is None else t.to(device=x.device, dtype=torch.int32).contiguous()
    acc, idx, first = i32(accept_len), i32(state_indices), i32(first_slot)
    if (idx is None and state.shape[0] != N) or (idx is not None and idx.numel() != N):
        raise ValueError("state has one slot per sequence unless state_indices [N] addresses a pool")
    y = torch.empty_like(x) if out is None else out
    a = _lib.ConvStepArgs()
    a.n_seqs, a.steps, a.channels, a.width = N, L, Cc, W
    a.activation, a.io_dtype = _ACT[activation], _io_dtype(x)
    a.x, a.weight, a.bias, a.state = x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(state) if state.numel() else None
    a.state_indices, a.n_slots, a.accept_len, a.first_slot = _ptr(idx), state.shape[0], _ptr(acc), _ptr(first)
    a.y, a.dev_status = y.data_ptr(), _ptr(dev_status)
    _lib.check(lib.kda_conv_step(C.byref(a), _stream(x.device)))
    return y


def kda_bwd(q, k, v, beta, g, dO, saved, cu_seqlens=None, h0=None, dhT=None, *, scale: float = 1.0,
            n_seqs: Optional[int] = None, initial_state_grad: bool = True, dev_status=None, out=None):
    """Backward of kda_fwd (``saved`` from kda_fwd(..., save=True) with the same inputs).

    Returns a dict of fp32 gradients: dq, dk, dv, dbeta, dg and dh0 (or None). ``out``, a dict
    with the same keys, supplies the gradient tensors to write (contiguous fp32 of the inputs'
    shapes; dh0 [N, H, 128, 128]) instead of fresh ones.
    """
    lib = library()
    _check_inputs(q, k, v, beta, g)
    dev = q.device
    cu = _i32(cu_seqlens, dev)
    N = (cu.numel() - 1) if cu is not None else (n_seqs or 1)
    H = q.shape[1]
    f32 = dict(dtype=torch.float32, device=dev)
    if out is not None:
        want = {"dq": q.shape, "dk": k.shape, "dv": v.shape, "dg": g.shape, "dbeta": beta.shape}
        for name, shape in want.items():
            t = out[name]
            if t.dtype != torch.float32 or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != dev:
                raise ValueError(f"out[{name!r}] must be a contiguous float32 tensor of shape {tuple(shape)} on {dev}")
        dq, dk, dv, dg, dbeta = (out[n] for n in ("dq", "dk", "dv", "dg", "dbeta"))
        dh0 = out.get("dh0") if initial_state_grad else None
        if dh0 is not None and (dh0.dtype != torch.float32 or tuple(dh0.shape) != (N, H, 128, 128)
                                or not dh0.is_contiguous()):
            raise ValueError("out['dh0'] must be a contiguous float32 [N, H, 128, 128] tensor")
    else:
        dq, dk, dv = torch.empty(q.shape, **f32), torch.empty(k.shape, **f32), torch.empty(v.shape, **f32)
        dg, dbeta = torch.empty(g.shape, **f32), torch.empty(beta.shape, **f32)
        dh0 = torch.empty((N, H, 128, 128), **f32) if initial_state_grad else None
    fa = fwd_args(q, k, v, beta, g, cu, h0, None, None, saved, None, scale, n_seqs=N, dev_status=dev_status)
    b = bwd_args(fa, dO, dq, dk, dv, dbeta, dg, dh0, dhT)
    ws_bytes = lib.kda_bwd_workspace_size(C.byref(b))
    if ws_bytes == 0:
        _lib.check(lib.kda_bwd(C.byref(b), _stream(dev)))
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    b.workspace, b.workspace_bytes = ws.data_ptr(), ws_bytes
    _lib.check(lib.kda_bwd(C.byref(b), _stream(dev)))
    return {"dq": dq, "dk": dk, "dv": dv, "dbeta": dbeta, "dg": dg, "dh0": dh0}


def step_args(q, k, v, beta, g, state, accept_len, o, scale: float = 1.0, state_indices=None,
              first_slot=None, dev_status=None) -> _lib.StepArgs:
    a = _lib.StepArgs()
    N, L, H, dk = q.shape
    a.n_seqs, a.steps, a.heads, a.dk, a.dv = N, L, H, dk, v.shape[3]
    a.scale, a.io_dtype = scale, _io_dtype(q)
    a.q, a.k, a.v, a.beta, a.g = _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g)
    a.state, a.accept_len, a.o = _ptr(state), _ptr(accept_len), _ptr(o)
    a.state_indices, a.first_slot, a.dev_status = _ptr(state_indices), _ptr(first_slot), _ptr(dev_status)
    a.n_slots = state.shape[0]
    return a


def kda_step(q, k, v, beta, g, state, accept_len=None, *, scale: float = 1.0, out=None, state_indices=None,
             first_slot=None, dev_status=None):
    """Decode / draft-verify L tokens per sequence; returns o [N, L, H, 128].

    ``state`` [N, H, 128, 128] fp32 (or a pool [P, H, 128, 128] addressed by
    ``state_indices`` [N]) is overwritten with the state after ``accept_len[i]`` token
    slots (left untouched where accept_len is 0; all L when None). Slots before
    ``first_slot[i]`` are padding: no state change, output not written. See
    include/kda.h for the verify-then-replay use of the two.
    """
    lib = library()
    _check_inputs(q, k, v, beta, g)
    if state.dtype != torch.float32 or not state.is_contiguous():
        raise TypeError("state must be a contiguous float32 tensor")
    i32 = lambda t: None if t is None else t.to(device=q.device, dtype=torch.int32).contiguous()
    acc, idx, first = i32(accept_len), i32(state_indices), i32(first_slot)
    N = q.shape[0]
    if (idx is None and state.shape[0] != N) or (idx is not None and idx.numel() != N):
        raise ValueError("state has one slot per sequence unless state_indices [N] addresses a pool")
    if first is not None and first.numel() != N:
        raise ValueError("first_slot must have one entry per sequence")
    o = torch.empty_like(v) if out is None else out
    a = step_args(q, k, v, beta, g, state, acc, o, scale, idx, first, dev_status)
    _lib.check(lib.kda_step(C.byref(a), _stream(q.device)))
    return o


# ---------------------------------------------------------------- around the recurrent core
# The current stream's handle without a Stream object around it, which would cost a small call several microseconds.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device) -> int:
    """The current stream of ``device``, which has to be the current device: the library launches there."""
    if device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {device}, the current device is cuda:{torch.cuda.current_device()}")
    return _raw_stream(device.index) if _raw_stream is not None else _stream(device)


def _need(t, name, dtype, shape, device):
    """Address of t, a contiguous tensor of this dtype and shape on CUDA device number ``device``, or an
    exception that names it."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)} on cuda:{device}")
    return t.data_ptr()


def _maybe(t, name, dtype, shape, device):
    return None if t is None else _need(t, name, dtype, shape, device)


def _ints(t, name, n, device):
    """Optional per-sequence int32 values on ``device`` (converted when they are not)."""
    if t is None:
        return None
    if t.numel() != n:
        raise ValueError(f"{name} must have one entry per sequence")
    if t.dtype is torch.int32 and t.get_device() == device.index and t.is_contiguous():
        return t
    return t.to(device=device, dtype=torch.int32).contiguous()


def _rows(t, name, T, heads, dim, like):
    """Row stride of a [T, heads, dim] view whose rows are dense."""
    if t.dtype != like.dtype:
        raise TypeError(f"{name} must share x's dtype")
    if t.shape != (T, heads, dim) or t.get_device() != like.get_device():
        raise ValueError(f"{name} must be [{T}, {heads}, {dim}] on {like.device}")
    row, head, channel = t.stride()
    if T == 0 or heads == 0:
        return heads * dim
    if channel != 1 or (heads > 1 and head != dim):
        raise ValueError(f"{name}'s rows must be dense (heads and channels side by side)")
    return row if T > 1 else heads * dim


def ssm_fwd(x, dt, a, b, c, cu_seqlens=None, h0=None, *, d_skip=None, dt_bias=None, dt_softplus: bool = True,
            final_state: bool = True, n_seqs: Optional[int] = None, dev_status=None):
    """Selective state space scan over packed prompts. Returns (y [T, H, P], hT or None).

    x [T, H, P] (P = 64 or 128), b and c [T, G, 128] in bfloat16 or float32 may be views into one
    row, such as conv_fwd's output split into [x | B | C]; dt [T, H], a [H], d_skip [H], dt_bias
    [H] are fp32, and the states h0, hT [N, H, 128, P] fp32 (row = state channel). Per token and
    head: h = softplus(dt + dt_bias), S = exp(h a) S + h B x^T, y = S^T C + d_skip x. For serving:
    there is no backward, and the results carry no gradient whatever the inputs require.
    """
    lib = library()
    if x.dim() != 3 or not x.is_cuda or b.dim() != 3:
        raise ValueError("x must be a CUDA tensor [T, H, P] and b [T, G, 128]")
    dev, di = x.device, x.get_device()
    (T, H, P), G = x.shape, b.shape[1]
    cu = cu_seqlens
    if cu is not None and (cu.dtype is not torch.int32 or cu.get_device() != di or not cu.is_contiguous()):
        cu = _i32(cu, dev)
    N = (cu.numel() - 1) if cu is not None else (n_seqs or 1)
    f32 = torch.float32
    D = b.shape[2]
    y = torch.empty((T, H, P), dtype=x.dtype, device=dev)
    hT = torch.empty((N, H, D, P), dtype=f32, device=dev) if final_state else None
    s = _lib.SsmArgs(
        N, T, H, G, P, D, _io_dtype(x), int(dt_softplus), _ptr(cu), x.data_ptr(), b.data_ptr(), c.data_ptr(),
        _rows(x, "x", T, H, P, x), _rows(b, "b", T, G, D, x), _rows(c, "c", T, G, D, x),
        _need(dt, "dt", f32, (T, H), di), _need(a, "a", f32, (H,), di), _maybe(dt_bias, "dt_bias", f32, (H,), di),
        _maybe(d_skip, "d_skip", f32, (H,), di), _maybe(h0, "h0", f32, (N, H, D, P), di), y.data_ptr(), _ptr(hT))
    s.dev_status = _ptr(dev_status)
    ws_bytes = lib.kda_ssm_fwd_workspace_size(C.byref(s))
    if ws_bytes:
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
        s.workspace, s.workspace_bytes = ws.data_ptr(), ws_bytes
    _lib.check(lib.kda_ssm_fwd(C.byref(s), _stream_of(dev)))
    return y, hT


def ssm_step(xbc, dt, a, conv_weight, conv_bias, conv_state, state, accept_len=None, *, groups: int = 1, d_skip=None,
             dt_bias=None, dt_softplus: bool = True, activation: str = "silu", state_indices=None, first_slot=None,
             out=None, dev_status=None):
    """Decode / verify L token slots per sequence through the short convolution and the
    selective scan; returns y [N, L, H, P].

    xbc [N, L, C] holds the raw rows [x | B | C], C = H P + 2 groups 128; ``conv_state``
    [N, W-1, C] (xbc's dtype) and ``state`` [N, H, 128, P] fp32, or pools addressed by
    ``state_indices`` [N], advance in place through ``accept_len`` slots; slots before
    ``first_slot`` are padding (their outputs are not written). conv_weight [C, W], conv_bias
    [C], dt [N, L, H], a, d_skip, dt_bias [H] are fp32.
    """
    lib = library()
    if xbc.dim() != 3 or not xbc.is_cuda or not xbc.is_contiguous() or state.dim() != 4 or conv_weight.dim() != 2:
        raise ValueError("xbc must be a contiguous CUDA tensor [N, L, C], state [slots, H, 128, P], conv_weight [C, W]")
    dev, di, f32 = xbc.device, xbc.get_device(), torch.float32
    N, L, Cc = xbc.shape
    slots, H, D, P = state.shape
    W = conv_weight.shape[1]
    if Cc != H * P + 2 * groups * D:
        raise ValueError(f"xbc has {Cc} channels, the heads and groups need {H * P + 2 * groups * D}")
    acc, idx = _ints(accept_len, "accept_len", N, dev), _ints(state_indices, "state_indices", N, dev)
    first = _ints(first_slot, "first_slot", N, dev)
    if idx is None and slots != N:
        raise ValueError("state has one slot per sequence unless state_indices [N] addresses a pool")
    y = torch.empty((N, L, H, P), dtype=xbc.dtype, device=dev) if out is None else out
    s = _lib.SsmStepArgs(
        N, L, H, groups, P, D, _io_dtype(xbc), int(dt_softplus), W, _ACT[activation], xbc.data_ptr(),
        _need(conv_weight, "conv_weight", f32, (Cc, W), di), _maybe(conv_bias, "conv_bias", f32, (Cc,), di),
        _need(conv_state, "conv_state", xbc.dtype, (slots, W - 1, Cc), di) if W > 1 else None,
        _need(dt, "dt", f32, (N, L, H), di), _need(a, "a", f32, (H,), di), _maybe(dt_bias, "dt_bias", f32, (H,), di),
        _maybe(d_skip, "d_skip", f32, (H,), di), _need(state, "state", f32, (slots, H, D, P), di), _ptr(idx), _ptr(acc),
        _ptr(first), slots, _need(y, "out", xbc.dtype, (N, L, H, P), di))
    s.dev_status = _ptr(dev_status)
    ws = torch.empty((N, L, Cc), dtype=f32, device=dev)   # the convolution's outputs: kda_ssm_step_workspace_size() bytes
    s.workspace, s.workspace_bytes = ws.data_ptr(), 4 * N * L * Cc
    _lib.check(lib.kda_ssm_step(C.byref(s), _stream_of(dev)))
    return y


def draft_verify(p, q, draft, u, noise, draft_len=None):
    """Speculative sampling from given random numbers: how many drafted tokens stand and which
    token follows. Returns int32 (accept_len [N], first_slot [N] = L - accept_len, tokens
    [N, L+1]: the accepted drafts, the next token, then -1).

    p [N, L+1, V] are the target's probabilities, q [N, L, V] the drafter's in the same dtype
    (bfloat16 or float32; None: the drafter is certain of its draft); draft [N, L] int32, u
    [N, L] fp32 uniforms in [0, 1), noise [N, V] fp32 Exp(1) variates, draft_len [N] optional
    lengths. Draft j stands while u q(x) < p(x); the next token wins the race r / noise over
    r = max(p - q, 0) after a rejection, r = p after the last draft (see include/kda.h).
    kda_step / conv_step / ssm_step then commit the accepted drafts either with ``accept_len``
    alone (slot j holds draft j) or with ``first_slot`` alone (the accepted drafts at the end of
    L slots, draft j in slot first_slot + j). Not with both: accept_len counts from slot 0, so
    only slots first_slot .. accept_len - 1 would be committed.
    """
    lib = library()
    if p.dim() != 3 or not p.is_cuda:
        raise ValueError("p must be a CUDA tensor [N, L+1, V]")
    dev, di, f32, i32 = p.device, p.get_device(), torch.float32, torch.int32
    N, L, V = p.shape[0], p.shape[1] - 1, p.shape[2]
    lens = _ints(draft_len, "draft_len", N, dev)
    accept, first = torch.empty(N, dtype=i32, device=dev), torch.empty(N, dtype=i32, device=dev)
    tokens = torch.empty((N, L + 1), dtype=i32, device=dev)
    s = _lib.DraftVerifyArgs(
        N, L, V, _io_dtype(p), _need(p, "p", p.dtype, (N, L + 1, V), di), _maybe(q, "q", p.dtype, (N, L, V), di),
        _need(draft, "draft", i32, (N, L), di), _ptr(lens), _need(u, "u", f32, (N, L), di),
        _need(noise, "noise", f32, (N, V), di), accept.data_ptr(), first.data_ptr(), tokens.data_ptr())
    _lib.check(lib.kda_draft_verify(C.byref(s), _stream_of(dev)))
    return accept, first, tokens


_GATE = {"sigmoid": _lib.KDA_GATE_SIGMOID, "silu": _lib.KDA_GATE_SILU}


def _block_norm_args(u, w_post, gate, gate_act, residual, scale, w_pre, eps):
    if u.dim() < 1 or not u.is_cuda or not u.is_contiguous():
        raise ValueError("u must be a contiguous CUDA tensor [..., d]")
    di, d, f32 = u.get_device(), u.shape[-1], torch.float32
    shape = u.shape
    n = _lib.BlockNormArgs(
        u.numel() // d if d else 0, d, eps, _io_dtype(u), _GATE[gate_act], u.data_ptr(),
        _maybe(gate, "gate", u.dtype, shape, di), _maybe(residual, "residual", u.dtype, shape, di),
        _maybe(w_post, "w_post", f32, (d,), di), _maybe(scale, "scale", f32, (d,), di),
        _maybe(w_pre, "w_pre", f32, (d,), di))
    return n


def block_norm_fwd(u, w_post, *, gate=None, gate_act: str = "silu", residual=None, scale=None, w_pre=None,
                   eps: float = 1e-6):
    """The norm after a block, its gate and residual scale, the residual sum and the norm before
    the next block, over rows u [..., d]:

        out = residual + scale * (w_post * rms_norm(u) * act(gate)),  normed = w_pre * rms_norm(out)

    w_post None leaves u as it is; gate, residual, scale and w_pre are optional. Returns (out,
    normed or None, stats); stats = (rstd_post, rstd_pre), fp32 [rows] or None, go to
    block_norm_bwd. With u the [T, H, d] output of the recurrent core this is its per-head
    output norm.
    """
    lib = library()
    n = _block_norm_args(u, w_post, gate, gate_act, residual, scale, w_pre, eps)
    out = torch.empty_like(u)
    normed = torch.empty_like(u) if w_pre is not None else None
    rstd = lambda on: torch.empty(n.rows, dtype=torch.float32, device=u.device) if on is not None else None
    stats = (rstd(w_post), rstd(w_pre))
    n.out, n.normed, n.rstd_post, n.rstd_pre = out.data_ptr(), _ptr(normed), _ptr(stats[0]), _ptr(stats[1])
    _lib.check(lib.kda_block_norm_fwd(C.byref(n), _stream_of(u.device)))
    return out, normed, stats


def block_norm_bwd(u, w_post, stats, d_out, d_normed=None, *, gate=None, gate_act: str = "silu", residual=None,
                   scale=None, w_pre=None, eps: float = 1e-6, dev_status=None):
    """Backward of block_norm_fwd (``stats`` from it, the same inputs). d_out and d_normed are the
    gradients of its two results, None for zero. Returns a dict: du, dgate, dresidual in u's
    dtype and dw_post, dscale, dw_pre fp32 [d], None where the input was absent."""
    lib = library()
    di, f32, shape = u.get_device(), torch.float32, u.shape
    n = _block_norm_args(u, w_post, gate, gate_act, residual, scale, w_pre, eps)
    rows, d = n.rows, n.dim
    if w_post is not None:
        n.rstd_post = _need(stats[0], "rstd_post", f32, (rows,), di)
    if w_pre is not None:
        n.rstd_pre = _need(stats[1], "rstd_pre", f32, (rows,), di)
    du = torch.empty_like(u)
    dgate, dresidual = (None if t is None else torch.empty_like(u) for t in (gate, residual))
    dw_post, dscale, dw_pre = (None if t is None else torch.empty_like(t) for t in (w_post, scale, w_pre))
    b = _lib.BlockNormBwdArgs(
        n, _maybe(d_out, "d_out", u.dtype, shape, di), _maybe(d_normed, "d_normed", u.dtype, shape, di), du.data_ptr(), _ptr(dgate),
        _ptr(dresidual), _ptr(dw_post), _ptr(dscale), _ptr(dw_pre))
    b.dev_status = _ptr(dev_status)
    ws_bytes = lib.kda_block_norm_bwd_workspace_size(C.byref(b))
    ws = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=u.device)
    b.workspace, b.workspace_bytes = ws.data_ptr(), ws_bytes
    _lib.check(lib.kda_block_norm_bwd(C.byref(b), _stream_of(u.device)))
    return {"du": du, "dgate": dgate, "dresidual": dresidual, "dw_post": dw_post, "dscale": dscale, "dw_pre": dw_pre}
