"""float64 oracle of the token operators: rotary positions, and linear
attention with a decay for each head.  Plain numpy, token by token, written
from the definitions."""

from __future__ import annotations

import math

import numpy as np


def _f64(x):
    if hasattr(x, "detach"):
        x = x.detach().double().cpu().numpy()
    return np.asarray(x, dtype=np.float64)


# ------------------------------------------------------------------ rotary


def rotary_frequencies(axis_pairs, base=10000.0, scaling="plain", factor=1.0, trained_length=4096.0,
                       beta_fast=32.0, beta_slow=1.0):
    """(radians per position of every pair, amplitude)."""
    out = []
    for P in axis_pairs:
        for i in range(P):
            w = base ** (-i / P)
            if scaling == "linear":
                w /= factor
            elif scaling == "ntk" and P > 1:
                w = (base * factor ** (P / (P - 1))) ** (-i / P)
            elif scaling == "yarn":
                def pair_of(turns):
                    # base^(-i / P) * trained_length = 2 pi turns
                    return P * math.log(trained_length / (2 * math.pi * turns)) / math.log(base)
                lo = max(math.floor(pair_of(beta_fast)), 0)
                hi = min(math.ceil(pair_of(beta_slow)), 2 * P - 1)
                stretched = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
                w = stretched * w / factor + (1 - stretched) * w
            out.append(w)
    return np.array(out), (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def grid_positions(grid, origin=(0, 0, 0)):
    """[axes, N] positions of a raster-ordered grid's tokens."""
    p = np.stack(np.unravel_index(np.arange(int(np.prod(grid))), tuple(grid)))
    return p + np.asarray(origin[: len(grid)])[:, None]


def rotate(x, positions, axis_pairs, freq, amplitude=1.0, layout="half", inverse=False):
    """x [B,H,N,d] turned (inverse: by the transpose).  positions [axes,N] or
    [B,axes,N]."""
    x = _f64(x)
    pos = _f64(positions)
    pos = np.broadcast_to(pos if pos.ndim == 3 else pos[None], (x.shape[0],) + pos.shape[-2:])
    y = x.copy()
    pairs = sum(axis_pairs)
    axis = np.repeat(np.arange(len(axis_pairs)), axis_pairs)
    for i in range(pairs):
        a, b = (i, i + pairs) if layout == "half" else (2 * i, 2 * i + 1)
        w = pos[:, axis[i]] * freq[i]                   # [B, N]
        c, s = amplitude * np.cos(w)[:, None], amplitude * np.sin(w)[:, None]
        if inverse:
            s = -s
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


# ------------------------------------------------------------------ decayed linear attention


def _decay(log_decay):
    return np.exp(_f64(log_decay))[None, :, None, None]


def _lens(lens, B, N):
    return np.full(B, N) if lens is None else np.clip(np.asarray(lens), 0, N)


def decay_forward(q, k, v, log_decay, lens=None, state=None, scale=None):
    """(out, state): S <- decay S + k_t v_t^T, out_t = scale q_t S."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, H, N, d = q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    n = _lens(lens, B, N)
    f = _decay(log_decay)
    S = np.zeros((B, H, d, d)) if state is None else _f64(state).copy()
    out = np.zeros_like(q)
    for t in range(N):
        on = np.nonzero(t < n)[0]
        if on.size == 0:
            break
        S[on] = f * S[on] + k[on, :, t, :, None] * v[on, :, t, None, :]
        out[on, :, t] = scale * np.einsum("bhk,bhkv->bhv", q[on, :, t], S[on])
    return out, S


def decay_backward(q, k, v, log_decay, dout, lens=None, state=None, dstate=None, scale=None):
    """(dq, dk, dv, gradient of the first state)."""
    q, k, v, dout = _f64(q), _f64(k), _f64(v), _f64(dout)
    B, H, N, d = q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    n = _lens(lens, B, N)
    f = _decay(log_decay)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(q), np.zeros_like(q)
    S = np.zeros((B, H, d, d)) if state is None else _f64(state).copy()
    for t in range(N):
        on = np.nonzero(t < n)[0]
        if on.size == 0:
            break
        S[on] = f * S[on] + k[on, :, t, :, None] * v[on, :, t, None, :]
        dq[on, :, t] = scale * np.einsum("bhkv,bhv->bhk", S[on], dout[on, :, t])
    # R: gradient of the state behind token t
    R = np.zeros((B, H, d, d)) if dstate is None else _f64(dstate).copy()
    for t in range(N - 1, -1, -1):
        on = np.nonzero(t < n)[0]
        if on.size == 0:
            continue
        R[on] += scale * q[on, :, t, :, None] * dout[on, :, t, None, :]
        dk[on, :, t] = np.einsum("bhkv,bhv->bhk", R[on], v[on, :, t])
        dv[on, :, t] = np.einsum("bhkv,bhk->bhv", R[on], k[on, :, t])
        R[on] *= f[0] if f.shape[0] == 1 else f[on]
    return dq, dk, dv, R
