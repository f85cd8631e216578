"""torch-facing wrappers of the gated delta rule and of draft verification: shape checks,
output allocation, the inputs' device and its current stream.  Every step runs in the HIP
kernels of libkda.so; there is no CPU or PyTorch fallback."""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _lib
from .ops import _DT, _check_cu_host, _check_out, _ptr


def _tokens(name, t, heads, d, dtype, device):
    """q, k or v as rows of tokens: the heads of a token are dense, the tokens a fixed stride
    apart (a slice of a fused projection).  Returns the stride in elements."""
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    shape = t.shape
    if len(shape) < 3 or shape[-1] != d or shape[-2] != heads:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [..., {heads}, {d}]")
    if t.is_contiguous():
        return heads * d
    st = t.stride()
    if st[-1] != 1 or (heads > 1 and st[-2] != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous (strides {st})")
    if len(shape) == 4 and shape[0] > 1 and shape[1] > 1 and st[0] != shape[1] * st[1]:
        raise ValueError(f"{name}: tokens must be a fixed stride apart (strides {st})")
    if t.numel() == 0 or shape[:-2].numel() == 1:
        return heads * d  # no second token to stride to
    stride = st[0] if len(shape) == 4 and shape[1] == 1 else st[-3]
    if stride < heads * d:  # (0, an expanded tensor's, would mean dense)
        raise ValueError(f"{name}: tokens overlap (strides {st})")
    return stride


def _dense(name, t, shape, dtype, device):
    """A dense tensor of exactly this shape, dtype and device."""
    if t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _check_out(name, t, shape, dtype, device)


def _head_dims(q, v):
    if not q.is_cuda:
        raise ValueError("q must be a GPU tensor")
    if q.dtype not in _DT:
        raise ValueError(f"unsupported dtype {q.dtype}")
    qs, vs = q.shape, v.shape
    if len(qs) < 3 or len(vs) != len(qs):
        raise ValueError("q and v must be [..., heads, d] with the same number of dimensions")
    return qs[-2], vs[-2], qs[-1], vs[-1]


def _params(q, k, v, scale):
    hk, hv, dk, dv = _head_dims(q, v)
    lead = q.shape[:-2]
    if k.shape[:-2] != lead or v.shape[:-2] != lead:
        raise ValueError(f"q, k and v must lead with {tuple(lead)}: {tuple(k.shape)}, {tuple(v.shape)}")
    dt, dev = q.dtype, q.device
    return _lib.GdnParams(_DT[dt], hk, hv, dk, dv, scale, _tokens("q", q, hk, dk, dt, dev),
                          _tokens("k", k, hk, dk, dt, dev), _tokens("v", v, hv, dv, dt, dev))


class _on:
    """The call runs on the inputs' device and on that device's current stream."""

    __slots__ = ("device", "guard")

    def __init__(self, device):
        self.device, self.guard = device, None

    def __enter__(self):
        if self.device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(self.device)
            self.guard.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _lengths(q, cu_seqlens):
    """Host copy of the packed offsets, and the number of tokens."""
    if q.dim() == 4:
        if cu_seqlens is not None:
            raise ValueError("cu_seqlens is for packed [T_total, H, d] inputs")
        B, T = q.shape[:2]
        if B < 1:
            raise ValueError("the batch is empty")
        return [i * T for i in range(B + 1)], B * T
    if q.dim() != 3:
        raise ValueError("q must be [B, T, H, dk] or [T_total, H, dk]")
    if cu_seqlens is None:
        raise ValueError("packed [T_total, H, d] inputs need cu_seqlens")
    cu = cu_seqlens.tolist() if isinstance(cu_seqlens, torch.Tensor) else [int(x) for x in cu_seqlens]
    _check_cu_host(cu, q.shape[0])
    return cu, q.shape[0]


def gdn_chunk_prefill(q, k, v, log_alpha, beta, cu_seqlens: Optional[Sequence[int]] = None,
                      initial_state=None, output_final_state: bool = True, scale: float = 1.0,
                      out: Optional[torch.Tensor] = None,
                      final_state: Optional[torch.Tensor] = None):
    """The gated delta rule over whole sequences.

    Fixed length: q/k [B, T, HK, dk], v [B, T, HV, dv], log_alpha/beta fp32 [B, T, HV].
    Varlen: the same packed as [T_total, H, .] with cu_seqlens (N+1 entries; a device tensor
    is copied to the host, which waits for it).  HV is a multiple of HK: value head h reads
    key head h // (HV // HK).  q, k and v may be slices of one projection (tokens a fixed
    stride apart).  initial_state: fp32 [N, HV, dk, dv] or None; final_state may be the same
    tensor.  Returns (o, final_state or None); o has v's shape and dtype."""
    cu, T = _lengths(q, cu_seqlens)
    N, dev = len(cu) - 1, q.device
    p = _params(q, k, v, scale)
    hv, dk, dv = p.num_v_heads, p.dk, p.dv
    gshape = v.shape[:-1]
    _dense("log_alpha", log_alpha, gshape, torch.float32, dev)
    _dense("beta", beta, gshape, torch.float32, dev)
    if initial_state is not None:
        _dense("initial_state", initial_state, (N, hv, dk, dv), torch.float32, dev)
    if out is None:
        out = torch.empty_like(v, memory_format=torch.contiguous_format)
    else:
        _dense("out", out, v.shape, v.dtype, dev)
    if final_state is not None:
        _dense("final_state", final_state, (N, hv, dk, dv), torch.float32, dev)
    elif output_final_state:
        final_state = torch.empty((N, hv, dk, dv), dtype=torch.float32, device=dev)
    lib = _lib.load()
    with _on(dev) as stream:
        _lib.check(lib.kda_gdn_chunk_prefill(
            ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta),
            (ctypes.c_int32 * (N + 1))(*cu), N, _ptr(initial_state), _ptr(final_state), _ptr(out),
            stream))
    return out, final_state


def gdn_prefill_backward(q, k, v, log_alpha, beta, d_out,
                         cu_seqlens: Optional[Sequence[int]] = None, initial_state=None,
                         d_final_state=None, scale: float = 1.0,
                         workspace: Optional[torch.Tensor] = None):
    """Gradients of gdn_chunk_prefill.  Inputs as for gdn_chunk_prefill, d_out like o (dense),
    d_final_state fp32 [N, HV, dk, dv] or None.  Returns a dict with dq, dk, dv (dtypes and
    shapes of q, k, v), dlog_alpha and dbeta (fp32) and d_initial_state (fp32 [N, HV, dk, dv]).
    workspace: a uint8 tensor of at least kda_gdn_prefill_backward_workspace bytes, or None to
    allocate one."""
    cu, T = _lengths(q, cu_seqlens)
    N, dev = len(cu) - 1, q.device
    p = _params(q, k, v, scale)
    hv, dk, dv = p.num_v_heads, p.dk, p.dv
    gshape = v.shape[:-1]
    _dense("log_alpha", log_alpha, gshape, torch.float32, dev)
    _dense("beta", beta, gshape, torch.float32, dev)
    _dense("d_out", d_out, v.shape, v.dtype, dev)
    for name, t in (("initial_state", initial_state), ("d_final_state", d_final_state)):
        if t is not None:
            _dense(name, t, (N, hv, dk, dv), torch.float32, dev)
    new = lambda like, dtype: torch.empty(like.shape, dtype=dtype, device=dev)  # noqa: E731
    g = dict(dq=new(q, q.dtype), dk=new(k, k.dtype), dv=new(v, v.dtype), dlog_alpha=new(log_alpha, torch.float32),
             dbeta=new(beta, torch.float32),
             d_initial_state=torch.empty((N, hv, dk, dv), dtype=torch.float32, device=dev))
    lib, cu_h = _lib.load(), (ctypes.c_int32 * (N + 1))(*cu)
    with _on(dev) as stream:
        if workspace is None:
            need = lib.kda_gdn_prefill_backward_workspace(ctypes.byref(p), cu_h, N)
            if need < 0:
                raise _lib.KdaError(_lib.KDA_ERR_INVALID_ARGUMENT, lib.kda_last_error().decode())
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        else:
            _dense("workspace", workspace, (workspace.numel(),), torch.uint8, dev)
        _lib.check(lib.kda_gdn_prefill_backward(
            ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), cu_h, N,
            _ptr(initial_state), _ptr(d_out), _ptr(d_final_state), _ptr(g["dq"]), _ptr(g["dk"]),
            _ptr(g["dv"]), _ptr(g["dlog_alpha"]), _ptr(g["dbeta"]), _ptr(g["d_initial_state"]),
            _ptr(workspace), workspace.numel(), stream))
    return g


def gdn_recurrent(q, k, v, log_alpha, beta, state, steps: Optional[torch.Tensor] = None,
                  state_indices: Optional[torch.Tensor] = None, update_state: bool = True,
                  output: bool = True, scale: float = 1.0, out: Optional[torch.Tensor] = None):
    """The gated delta rule over 1..16 tokens of every sequence from its stored state, which is
    updated in place.

    q/k [N, K, HK, dk], v [N, K, HV, dv], log_alpha/beta fp32 [N, K, HV]; for one token the
    K axis may be left out.  state: fp32 [slots, HV, dk, dv]; sequence n's is
    state[state_indices[n]] (int32 GPU tensor) or state[n].  An index outside the slots marks a
    padded row (zero outputs, no state), and so does, where states are written, a slot that an
    earlier row names.  steps (int32 GPU tensor [N]): the state advances over the first steps[n]
    tokens only; update_state=False leaves it as it is (the outputs of drafts); output=False
    computes no outputs (the commit of their kept prefix).  Returns o shaped like v, or None."""
    hk, hv, dk, dv = _head_dims(q, v)
    if q.dim() == 3:
        N, K = q.shape[0], 1
    elif q.dim() == 4:
        N, K = q.shape[:2]
    else:
        raise ValueError("q must be [N, K, HK, dk] or [N, HK, dk]")
    dev = q.device
    p = _params(q, k, v, scale)
    gshape = v.shape[:-1]
    _dense("log_alpha", log_alpha, gshape, torch.float32, dev)
    _dense("beta", beta, gshape, torch.float32, dev)
    if state.dim() != 4:
        raise ValueError(f"state has shape {tuple(state.shape)}, expected [slots, {hv}, {dk}, {dv}]")
    slots = state.shape[0]
    _dense("state", state, (slots, hv, dk, dv), torch.float32, dev)
    for name, t in (("steps", steps), ("state_indices", state_indices)):
        if t is not None:
            _dense(name, t, (N,), torch.int32, dev)
    if not output:
        if out is not None:
            raise ValueError("out given but output=False")
    elif out is None:
        out = torch.empty_like(v, memory_format=torch.contiguous_format)
    else:
        _dense("out", out, v.shape, v.dtype, dev)
    if N == 0:
        return out
    lib = _lib.load()
    with _on(dev) as stream:
        _lib.check(lib.kda_gdn_recurrent(
            ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), N, K,
            _ptr(steps), _ptr(state_indices), slots, _ptr(state), int(update_state), _ptr(out),
            stream))
    return out


def spec_accept(target_probs, draft_probs, draft_tokens, uniforms,
                num_drafts: Optional[torch.Tensor] = None,
                accepted: Optional[torch.Tensor] = None, tokens: Optional[torch.Tensor] = None):
    """Verification of drafted tokens against the target's probabilities.

    target_probs [N, K+1, V], draft_probs [N, K, V] of the same dtype or None (certain drafts),
    draft_tokens int32 [N, K], uniforms fp32 [N, K+1] in [0, 1), num_drafts int32 [N] or None.
    Draft j is kept while uniforms[n, j] q_j(x_j) < p_j(x_j); uniforms[n, K] draws the next
    token.  Returns (accepted int32 [N], tokens int32 [N, K+1]: the kept drafts, the drawn
    token, then -1).  `accepted` is what spec_commit and gdn_recurrent(steps=) take."""
    if not target_probs.is_cuda:
        raise ValueError("target_probs must be a GPU tensor")
    if target_probs.dim() != 3 or target_probs.dtype not in _DT or target_probs.shape[1] < 1 or target_probs.shape[2] < 1:
        raise ValueError(f"target_probs must be bf16 or fp32 [N, K+1, V], got {tuple(target_probs.shape)} {target_probs.dtype}")
    N, K, V, dev = target_probs.shape[0], target_probs.shape[1] - 1, target_probs.shape[2], target_probs.device
    _dense("target_probs", target_probs, (N, K + 1, V), target_probs.dtype, dev)
    if draft_probs is not None:
        _dense("draft_probs", draft_probs, (N, K, V), target_probs.dtype, dev)
        if K == 0:
            draft_probs = None
    _dense("draft_tokens", draft_tokens, (N, K), torch.int32, dev)
    _dense("uniforms", uniforms, (N, K + 1), torch.float32, dev)
    if num_drafts is not None:
        _dense("num_drafts", num_drafts, (N,), torch.int32, dev)
    if accepted is None:
        accepted = torch.empty((N,), dtype=torch.int32, device=dev)
    else:
        _dense("accepted", accepted, (N,), torch.int32, dev)
    if tokens is None:
        tokens = torch.empty((N, K + 1), dtype=torch.int32, device=dev)
    else:
        _dense("tokens", tokens, (N, K + 1), torch.int32, dev)
    if N == 0:
        return accepted, tokens
    lib = _lib.load()
    with _on(dev) as stream:
        need = lib.kda_spec_accept_workspace(N, V)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        _lib.check(lib.kda_spec_accept(
            _DT[target_probs.dtype], N, K, V, _ptr(target_probs), _ptr(draft_probs),
            _ptr(draft_tokens), _ptr(uniforms), _ptr(num_drafts), _ptr(accepted),
            _ptr(tokens), _ptr(ws), ws.numel(), stream))
    return accepted, tokens
