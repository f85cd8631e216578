"""The gated delta rule and its reverse, and draft verification, in 64 bits on the CPU: plain
token loops written from the definitions, for tests.

    S <- e^{g_t} S;  u = beta_t (v_t - S^T k_t);  S <- S + k_t u^T;  o_t = scale S^T q_t
"""
from __future__ import annotations

import numpy as np
import torch


def f64(x):
    return None if x is None else x.detach().to("cpu", torch.float64)


def grouped(x, hv):
    """[T, HK, d] with each head repeated for the value heads that share it."""
    return x.repeat_interleave(hv // x.shape[1], dim=1)


def forward(q, k, v, la, be, cu, s0=None, scale=1.0, keep=False):
    """o [T, HV, dv], final states [N, HV, dk, dv] (and the state before each token)."""
    q, k, v, la, be, s0 = (f64(x) for x in (q, k, v, la, be, s0))
    T, hv, dv = v.shape
    dk, N = q.shape[2], len(cu) - 1
    q, k = grouped(q, hv) * scale, grouped(k, hv)
    o = torch.zeros(T, hv, dv, dtype=torch.float64)
    sf = torch.zeros(N, hv, dk, dv, dtype=torch.float64) if s0 is None else s0.clone()
    before = [None] * T
    for n in range(N):
        S = sf[n]
        for t in range(cu[n], cu[n + 1]):
            if keep:
                before[t] = S.clone()
            S = S * torch.exp(la[t])[:, None, None]
            u = be[t][:, None] * (v[t] - (k[t][:, None] @ S)[:, 0])
            S = S + k[t][:, :, None] * u[:, None]
            o[t] = (q[t][:, None] @ S)[:, 0]
        sf[n] = S
    return (o, sf, before) if keep else (o, sf)


def backward(q, k, v, la, be, cu, s0, do, dsf, scale=1.0):
    """Gradients of <o, do> + <S_final, dsf>: dq, dk, dv, dlog_alpha, dbeta, d_initial_state."""
    hk, hv = q.shape[1], v.shape[1]
    before = forward(q, k, v, la, be, cu, s0, scale, keep=True)[2]
    q, k, v, la, be, do, dsf = (f64(x) for x in (q, k, v, la, be, do, dsf))
    q, k = grouped(q, hv), grouped(k, hv)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dla, dbe = torch.zeros_like(la), torch.zeros_like(be)
    N = len(cu) - 1
    ds0 = torch.zeros(N, hv, q.shape[2], v.shape[2], dtype=torch.float64) if dsf is None else dsf.clone()
    col = lambda x: x[:, :, None]  # noqa: E731
    row = lambda x: x[:, None, :]  # noqa: E731
    for n in range(N):
        D = ds0[n]
        for t in reversed(range(cu[n], cu[n + 1])):
            a = torch.exp(la[t])[:, None, None]
            S = before[t] * a
            err = v[t] - (row(k[t]) @ S)[:, 0]
            b = be[t][:, None]
            new = S + col(k[t]) * row(b * err)
            dq[t] = scale * (new @ col(do[t]))[:, :, 0]
            D = D + scale * col(q[t]) * row(do[t])
            du = (row(k[t]) @ D)[:, 0]
            dk[t] = (D @ col(b * err))[:, :, 0] - (S @ col(b * du))[:, :, 0]
            dbe[t] = (du * err).sum(-1)
            dv[t] = b * du
            D = D - col(k[t]) * row(b * du)
            dla[t] = (D * S).sum((-1, -2))
            D = D * a
        ds0[n] = D
    shared = lambda x: x.reshape(x.shape[0], hk, hv // hk, -1).sum(2)  # noqa: E731
    return dict(dq=shared(dq), dk=shared(dk), dv=dv, dlog_alpha=dla, dbeta=dbe, d_initial_state=ds0)


def accept(p, q, x, u, counts=None):
    """accepted [N], tokens [N, K+1] by numpy in 64 bits, sequence by sequence."""
    p, u = f64(p).numpy(), f64(u).numpy()
    q = None if q is None else f64(q).numpy()
    x = x.cpu().numpy()
    N, K, V = p.shape[0], p.shape[1] - 1, p.shape[2]
    acc, tok = np.zeros(N, np.int32), np.full((N, K + 1), -1, np.int32)
    for n in range(N):
        m = K if counts is None else int(min(max(int(counts[n]), 0), K))
        a = 0
        while a < m:
            t = x[n, a]
            if not 0 <= t < V:
                break
            if not u[n, a] * (1.0 if q is None else q[n, a, t]) < p[n, a, t]:
                break
            a += 1
        with np.errstate(invalid="ignore"):
            base = np.where(p[n, a] > 0, p[n, a], 0.0)
            w = base
            if a < m:
                if q is None:
                    w = base.copy()
                    if 0 <= x[n, a] < V:
                        w[x[n, a]] = 0.0
                else:
                    d = p[n, a] - q[n, a]
                    w = np.where(d > 0, d, 0.0)
        if not w.sum() > 0:
            w = base
        acc[n], tok[n, :a] = a, x[n, :a]
        if w.sum() > 0:
            c = np.cumsum(w)
            at = np.nonzero((c > u[n, K] * c[-1]) & (w > 0))[0]
            tok[n, a] = at[0] if len(at) else np.nonzero(w > 0)[0][-1]
    return acc, tok


# -------------------------------------------------------------------------- inputs and bounds

def inputs(lens, hk, hv, dk, dv, dtype, seed, s0=True, device="cuda", decay=0.1, amp=1.0):
    """Packed seeded inputs: unit keys and queries, log-decays -decay softplus(N), write
    strengths sigmoid(N)."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    T, N = sum(lens), len(lens)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    cu = [sum(lens[:i]) for i in range(N + 1)]
    x = dict(q=unit(r(T, hk, dk)).to(dtype), k=unit(r(T, hk, dk)).to(dtype), v=(amp * r(T, hv, dv)).to(dtype),
             la=-decay * torch.nn.functional.softplus(r(T, hv)), be=torch.sigmoid(r(T, hv)),
             s0=0.3 * amp * r(N, hv, dk, dv) if s0 else None)
    return {n: None if t is None else t.to(device) for n, t in x.items()}, cu


def rel(got, ref):
    """2-norm of the difference over the reference's."""
    got, ref = f64(got), f64(ref)
    n = ref.norm().item()
    d = (got - ref).norm().item()
    return d / n if n else d


# fp32 results.  Products of the token loop are fp32 (2^-24 each) and sums over dk or 16 tokens
# at a time; those of the chunked form take their operands as pairs of 11-bit halves (2^-22
# each side).  A result is built from three such products in a row (S^T k, the chunk's solve,
# k u^T) whose sums of up to 128 terms of random sign grow the error of a term by at most
# sqrt(128) ~ 11 relative to the sum: 3 * 2 * 11 * 2^-22 = 1.6e-5.
TOL_F32 = 1.6e-5
# bf16 outputs: the stored rounding (at most 2^-8 of each value), and a readout whose three
# rounded operands (state, P, U) carry 11 bits: 3 * 2^-11.
TOL_BF16 = 2.0 ** -8 + 3 * 2.0 ** -11


def close(name, got, ref, dtype):
    assert torch.isfinite(got).all(), f"{name}: not finite"
    e = rel(got, ref)
    tol = TOL_BF16 if dtype == torch.bfloat16 else TOL_F32
    print(f"  {name}: {e:.2e} (tol {tol:.1e})", flush=True)
    assert e <= tol, f"{name}: {e:.3e} > {tol:.3e}"
