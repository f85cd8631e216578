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
    dt, dev, qs, vs = q.dtype, q.device, q.shape, v.shape
    if k.shape != qs or vs[:-2] != qs[:-2]:
        raise ValueError(f"k must have q's shape {tuple(qs)} and v lead like it: {tuple(k.shape)}, {tuple(vs)}")
    for name, t in (("k", k), ("v", v)):
        if t.dtype != dt or t.device != dev:
            raise ValueError(f"{name} is {t.dtype} on {t.device}, q {dt} on {dev}")
    # (0: dense)
    return _lib.GdnParams(_DT[dt], hk, hv, dk, dv, scale,
                          0 if q.is_contiguous() else _tokens("q", q, hk, dk, dt, dev),
                          0 if k.is_contiguous() else _tokens("k", k, hk, dk, dt, dev),
                          0 if v.is_contiguous() else _tokens("v", v, hv, dv, dt, dev))


# The current stream's handle; the public way makes a Stream object for it (1.9 us against 0.1,
# of 12 that a small call takes).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(device, f, *args):
    """f(*args, stream) on the inputs' device and on that device's current stream."""
    index = device.index
    if index == torch.cuda.current_device():
        return _lib.check(f(*args, _raw_stream(index)))
    with torch.cuda.device(index):
        return _lib.check(f(*args, _raw_stream(index)))


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
        final_state = beta.new_empty((N, hv, dk, dv))
    _run(dev, _lib.load().kda_gdn_chunk_prefill, ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(),
         log_alpha.data_ptr(), beta.data_ptr(), (ctypes.c_int32 * (N + 1))(*cu), N, _ptr(initial_state),
         _ptr(final_state), out.data_ptr())
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
    g = dict(dq=q.new_empty(q.shape), dk=k.new_empty(k.shape), dv=v.new_empty(v.shape),
             dlog_alpha=beta.new_empty(gshape), dbeta=beta.new_empty(gshape),
             d_initial_state=beta.new_empty((N, hv, dk, dv)))
    lib, cu_h = _lib.load(), (ctypes.c_int32 * (N + 1))(*cu)
    if workspace is None:
        need = lib.kda_gdn_prefill_backward_workspace(ctypes.byref(p), cu_h, N)
        if need < 0:
            raise _lib.KdaError(_lib.KDA_ERR_INVALID_ARGUMENT, lib.kda_last_error().decode())
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    else:
        _dense("workspace", workspace, (workspace.numel(),), torch.uint8, dev)
    _run(dev, lib.kda_gdn_prefill_backward, ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(),
         log_alpha.data_ptr(), beta.data_ptr(), cu_h, N, _ptr(initial_state), d_out.data_ptr(),
         _ptr(d_final_state), g["dq"].data_ptr(), g["dk"].data_ptr(), g["dv"].data_ptr(), g["dlog_alpha"].data_ptr(),
         g["dbeta"].data_ptr(), g["d_initial_state"].data_ptr(), workspace.data_ptr(), workspace.numel())
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
    _run(dev, _lib.load().kda_gdn_recurrent, ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(),
         log_alpha.data_ptr(), beta.data_ptr(), N, K, _ptr(steps), _ptr(state_indices), slots, state.data_ptr(),
         int(update_state), _ptr(out))
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
        accepted = draft_tokens.new_empty((N,))
    else:
        _dense("accepted", accepted, (N,), torch.int32, dev)
    if tokens is None:
        tokens = draft_tokens.new_empty((N, K + 1))
    else:
        _dense("tokens", tokens, (N, K + 1), torch.int32, dev)
    if N == 0:
        return accepted, tokens
    lib = _lib.load()
    need = lib.kda_spec_accept_workspace(N, V)
    ws = uniforms.new_empty(need // 4)
    _run(dev, lib.kda_spec_accept, _DT[target_probs.dtype], N, K, V, target_probs.data_ptr(),
         _ptr(draft_probs), draft_tokens.data_ptr(), uniforms.data_ptr(), _ptr(num_drafts), accepted.data_ptr(),
         tokens.data_ptr(), ws.data_ptr(), need)
    return accepted, tokens
