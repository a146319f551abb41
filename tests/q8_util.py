"""Helpers of the 8-bit cache's tests: caches made on the host, the attention
over them in float64, and how far a kernel may be from it.

Tolerances, from the arithmetic (u32 = 2^-24; p_t the softmax weights, A the
output computed with |V|; L the largest sum of |q_c k_c| * |scale|):
 - a logit is off by at most (d + 4) u32 L, a weight relatively by twice that
   (numerator and denominator), a sum of n terms by (n + 16) u32 (the 16 covers
   the exponential's and the division's ulps):
       A (2 (d + 4) u32 L + (n + 16) u32);
 - the tensor-core paths round a query's small elements to 2^-10 units of which
   its largest has at least 224: a logit moves by 2^-10 / 224 max|q| sum|k_c|
   |scale|, a weight relatively by twice that (M its largest value):
       A 2 (2^-10 / 224) M;
   a weight to two e4m3 terms, at most 2^-9 of it, and the smallest weights to
   steps of 2^-13 where the largest p_t s_t (s_t the value row's scale) is at
   least 2^2: less than a step each, with a mean of 0 over the rows' dither, and
   together less than half a step each, 2^-16 of the largest, times codes up to
   448 (the shared prefix's fp16 weights stay within it):
       2^-9 A + n 2^-16 max_t(p_t s_t) 448;
 - bf16 outputs are rounded once: 2^-8 |o| (half a step), fp32: u32 |o|.
"""
import numpy as np
import torch

from grouped_query_attention_mqa_b200 import q8
from oracle import q8_oracle

U32 = 2.0 ** -24


def round_to(x, dtype):
    """float array -> (device tensor maker, float64 values) in the storage type."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32))
    t = t.to(torch.bfloat16) if dtype == "bf16" else t
    return t, t.double().numpy()


def rows(rng, shape, spread=1.0):
    """Normal rows whose magnitude varies from row to row (2^(spread * normal))."""
    return rng.standard_normal(shape) * np.exp2(spread * rng.standard_normal(shape[:-1] + (1,)))


def host_cache(rng, b, m_max, g, d_k, d_v=None, lens=None, spread=1.0):
    """(codes, exponents) pairs for K and V as uint8 arrays; with lens, rows at
    or past a sequence's length hold NaN codes and infinite scales."""
    out = []
    for d in (d_k, d_k if d_v is None else d_v):
        c, e = q8_oracle.quantise(rows(rng, (b, m_max, g, d), spread))
        e = np.ascontiguousarray(np.moveaxis(e, 2, 1))
        if lens is not None:
            for s, n in enumerate(lens):
                c[s, max(n, 0):] = 0x7F
                e[s, :, max(n, 0):] = 255
        out += [c, e]
    return out


def dev_cache(arrays):
    k, ke, v, ve = (torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in arrays)
    return q8.Cache(k.view(torch.float8_e4m3fn), ke, v.view(torch.float8_e4m3fn), ve)


def attention(q, parts, g, scale, dtype, two_terms):
    """(o, tolerance) [b, h, d_v] in float64.  ``parts``: per sequence, a list
    of (K, V, value row scales) with K [n, g, d_k], V [n, g, d_v], scales [n, g]
    whose rows together are the attended ones."""
    b, h, d_k = q.shape
    hq = h // g
    d_v = parts[0][0][1].shape[2]
    o, tol = np.zeros((b, h, d_v)), np.zeros((b, h, d_v))
    for s in range(b):
        K, V, S = (np.concatenate([p[i] for p in parts[s]]) for i in range(3))
        n = K.shape[0]
        if n == 0:
            continue
        for j in range(g):
            qs = q[s, j * hq:(j + 1) * hq]
            z = qs @ K[:, j].T * scale
            w = np.exp(z - z.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            ref, A = w @ V[:, j], w @ np.abs(V[:, j])
            L = (np.abs(qs) @ np.abs(K[:, j]).T).max() * abs(scale)
            t = A * (2 * (d_k + 4) * U32 * L + (n + 16) * U32)
            if two_terms:
                M = np.abs(qs).max(1, keepdims=True) * np.abs(K[:, j]).sum(1).max() * abs(scale)
                t = t + A * 2 * 2.0 ** -10 / 224 * M
                t = t + 2.0 ** -9 * A + n * 2.0 ** -16 * (w * S[:, j]).max(1, keepdims=True) * 448
            t = t + np.abs(ref) * (2.0 ** -8 if dtype == "bf16" else U32)
            o[s, j * hq:(j + 1) * hq], tol[s, j * hq:(j + 1) * hq] = ref, t
    return o, tol


def cache_parts(arrays, lens, window=0):
    """``attention``'s parts of a host cache: each sequence's attended rows."""
    k, ke, v, ve = arrays
    m_max = k.shape[1]
    out = []
    for s, n in enumerate(lens):
        n = min(max(int(n), 0), m_max)
        a = max(0, n - window) if window else 0
        K = q8_oracle.values(k[s:s + 1, a:n], ke[s:s + 1, :, a:n])[0]
        V = q8_oracle.values(v[s:s + 1, a:n], ve[s:s + 1, :, a:n])[0]
        out.append([(K, V, q8_oracle.scale_of(ve[s, :, a:n]).T)])
    return out


def assert_within(out, ref, tol, what=""):
    out = out.detach().double().cpu().numpy()
    assert out.shape == ref.shape
    assert np.isfinite(out).all(), f"{what}: non-finite output"
    over = np.abs(out - ref) - tol
    assert (over <= 0).all(), f"{what}: {over.max():.3e} past its tolerance (error {np.abs(out - ref).max():.3e})"
