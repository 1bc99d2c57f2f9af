"""The serving operators in plain 64-bit numpy, from their formulas in
include/ivit.h: linear layers with a low-rank adapter per request, the end of
a residual branch, differential attention.  ``>>`` on int64 is the floor
shift; every product and sum stays below 2^63.
"""
import numpy as np

from . import layernorm, shiftgelu


def _i64(a):
    return np.asarray(a, dtype=np.int64)


def _sat(v, bits=8):
    return np.clip(v, -(1 << (bits - 1)), (1 << (bits - 1)) - 1)


def _requant(acc, b, c, bits=8, rounding=0):
    v = acc * _i64(b)
    if rounding:
        v = v + np.where(_i64(c) > 0, np.int64(1) << np.maximum(_i64(c) - 1, 0), 0)
    return _sat(v >> _i64(c), bits)


def _matmul(a, b):
    """a b of int8-valued matrices: float64 holds every sum (below 2^53) exactly."""
    return (np.asarray(a, np.float64) @ np.asarray(b, np.float64)).astype(np.int64)


def linear_lora(X, W, bias, b, c, adapters, idx, rows, out_bits=8, skip=None, res=None, rounding=0, gelu=None):
    """Y [M x N] int8.  adapters (A [n,R,K], b_t, c_t [n,R], B [n,N,R]); gelu (I0, M, k_out, out) or None."""
    A, b_t, c_t, Bu = adapters
    acc = _matmul(X, W.T)
    if bias is not None:
        acc = acc + _i64(bias)
    for q, a in enumerate(idx):
        if 0 <= a < len(A):
            r = slice(q * rows, (q + 1) * rows)
            t = _requant(_matmul(X[r], A[a].T), b_t[a], c_t[a], 8, rounding)
            acc[r] += _matmul(t, Bu[a].T)
    o = _requant(acc, b, c, out_bits, rounding)
    if gelu is not None:
        return shiftgelu(o.astype(np.int8), *gelu)
    if skip is not None:
        o = _sat((res[0] * _i64(skip) + res[1] * o) >> res[2])
    return o.astype(np.int8)


def residual_norm(skip, branch, scale, b_skip, c, post=None, gate=None, gate_rows=1, pre=None):
    """(y, z); post and pre (gamma, beta, F, M_ln, out) or None."""
    n = layernorm(branch, *post) if post is not None else branch
    u = _i64(n)
    if gate is not None:
        u = u * _i64(gate)[np.arange(len(u)) // gate_rows]
    y = _sat((b_skip * _i64(skip) + _i64(scale) * u) >> c).astype(np.int8)
    return y, layernorm(y, *pre) if pre is not None else None


def _shift_exp(d, I0):
    neg = -(d + (d >> 1) - (d >> 4))
    q = neg // I0
    return (I0 - ((neg - q * I0 + 1) >> 1)) >> np.minimum(q, 62)


def diff_maps(L1, L2, I0, M, k_out, lam):
    """The two integer maps of logit rows L1, L2 [..., N]; the second weighted by lam / 2^M."""
    maps = []
    for L, num in ((L1, 1 << M), (L2, min(max(int(lam), 0), 1 << M))):
        e = _shift_exp(_i64(L) - _i64(L).max(-1, keepdims=True), I0)
        maps.append(((num // e.sum(-1, keepdims=True)) * e) >> (M - (k_out - 1)))
    return maps


def attention_diff(qkv, B, N, H, logit, k_s, I0, M, k_out, lam, out):
    """ctx [B*N x 128 H] int8."""
    D = 128 * H
    q, k, v = np.asarray(qkv).reshape(B, N, 3, H, 128).transpose(2, 0, 3, 1, 4)
    ctx = np.zeros((B, N, H, 128), np.int8)
    for i in range(B):
        for h in range(H):
            L = [_requant(_matmul(q[i, h, :, 64 * m:64 * m + 64], k[i, h, :, 64 * m:64 * m + 64].T), logit[0], logit[1],
                          k_s) for m in range(2)]
            p1, p2 = diff_maps(L[0], L[1], I0, M, k_out, lam[h])
            ctx[i, :, h] = _requant(_matmul(p1 - p2, v[i, h]), out[0], out[1])
    return ctx.reshape(B * N, D)
