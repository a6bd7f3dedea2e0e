"""fp64 definitions of the operators of include/gdn_linattn.h (numpy, test infrastructure
only): linear attention with a decay for each head, token by token; the norm and rotation of
queries and keys; one step of beam search; the reordering of states."""
from __future__ import annotations

import numpy as np
import torch


def _np(t):
    return None if t is None else (t.detach().to("cpu", torch.float64).numpy() if isinstance(t, torch.Tensor)
                                   else np.asarray(t, np.float64))


def linear_attention(q, k, v, log_gate, h0=None, cu_seqlens=None, *, scale=1.0, snapshot_stride=0):
    """q, k (B,T,hk,dk), v (B,T,H,dv), log_gate (B,T,H) or (H,), h0 (N,H,dv,dk) or None.
    Returns (out (B,T,H,dv), final states, snapshots or None); rows outside every sequence are NaN."""
    q, k, v, g, h0 = (_np(x) for x in (q, k, v, log_gate, h0))
    B, T, H, dv = v.shape
    rep, dk = H // q.shape[2], q.shape[3]
    q, k = np.repeat(q, rep, axis=2) * scale, np.repeat(k, rep, axis=2)
    g = np.broadcast_to(g, (B, T, H))
    if cu_seqlens is None:
        spans = [(b * T, (b + 1) * T) for b in range(B)]
    else:
        cu = [int(c) for c in cu_seqlens]
        spans = list(zip(cu[:-1], cu[1:]))
    q, k, v, g = (x.reshape(B * T, *x.shape[2:]) for x in (q, k, v, g))
    out = np.full((B * T, H, dv), np.nan)
    fin = np.zeros((len(spans), H, dv, dk))
    snaps = np.zeros((len(spans), T // snapshot_stride, H, dv, dk)) if snapshot_stride else None
    for n, (a, b) in enumerate(spans):
        S = np.zeros((H, dv, dk)) if h0 is None else h0[n].copy()
        for t in range(a, b):
            S = np.exp(g[t])[:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
            out[t] = np.einsum("hij,hj->hi", S, q[t])
            if snapshot_stride and (t - a + 1) % snapshot_stride == 0:
                snaps[n, (t - a + 1) // snapshot_stride - 1] = S
        fin[n] = S
    return out.reshape(B, T, H, dv), fin, snaps


def norm_rope(x, positions, inv_freq, weight=None, *, eps=1e-6, weight_offset=0.0, interleaved=False):
    """x (B,T,heads,d), positions (B,T), inv_freq (rot/2,) or None."""
    x, w = _np(x), _np(weight)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * (weight_offset + w)
    if inv_freq is None or len(inv_freq) == 0:
        return y
    f = _np(inv_freq)
    angle = _np(positions)[:, :, None, None] * f
    c, s = np.cos(angle), np.sin(angle)
    half = len(f)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    z = y.copy()
    z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
    return z


def beam_select(logits, scores, K):
    """logits (B,W,V), scores (B,W) or None; returns (scores, parents, tokens), each (B,K)."""
    x = _np(logits)
    B, W, V = x.shape
    s = np.zeros((B, W)) if scores is None else _np(scores)
    out, par, tok = np.zeros((B, K)), np.zeros((B, K), np.int32), np.zeros((B, K), np.int32)
    for b in range(B):
        cand = []
        for w in range(W):
            row = x[b, w]
            with np.errstate(all="ignore"):
                m = row.max()
                lse = m + np.log(np.exp(row - m).sum())
            dead = not np.isfinite(s[b, w]) or not np.isfinite(lse)
            sc = np.full(V, -np.inf) if dead else (s[b, w] - lse) + row
            cand.append(sc)
        flat = np.concatenate(cand)
        order = np.lexsort((np.arange(W * V), -flat))[:K]
        out[b], par[b], tok[b] = flat[order], order // V, order % V
    return out, par, tok


def state_reorder(state, parent):
    """state (B*W, ...), parent (B,W) as numpy arrays; a parent outside 0 .. W-1 keeps its row."""
    B, W = parent.shape
    new = state.copy()
    for b in range(B):
        for w in range(W):
            p = int(parent[b, w])
            new[b * W + w] = state[b * W + (p if 0 <= p < W else w)]
    return new
