"""The attention operators in float64 NumPy, from their definitions: packed
prompts, the weight each key received, the 4-bit cache, its decode step, and
eviction. Test infrastructure only; shares no code with the CUDA path.

"Escopo de Aplicação" (gist.science summary of "Reduced Matrix Multiplication:
Input-Adaptive Matrix-Product Reduction for LLM Inference") names the attention
sites; the cache format and the eviction rule are this library's own."""
from __future__ import annotations

import numpy as np

GROUP = 32


def visible(S_q: int, S_k: int, causal: bool) -> np.ndarray:
    """[S_q][S_k] bool: key k is seen by query q iff k <= q + S_k - S_q (causal)."""
    if not causal:
        return np.ones((S_q, S_k), dtype=bool)
    return np.arange(S_k)[None, :] <= np.arange(S_q)[:, None] + (S_k - S_q)


def attention(Q, K, V, scale: float, causal: bool):
    """One sequence, one head: (O, lse, P, S), rows that see no key 0 and -inf."""
    S = scale * (Q @ K.T)
    see = visible(Q.shape[0], K.shape[0], causal)
    X = np.where(see, S, -np.inf)
    m = np.max(X, axis=1, initial=-np.inf, keepdims=True)
    e = np.where(see, np.exp(X - np.where(np.isfinite(m), m, 0.0)), 0.0)
    total = e.sum(axis=1, keepdims=True)
    P = np.divide(e, total, out=np.zeros_like(e), where=total > 0)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(total))[:, 0]
    return P @ V, lse, P, S


def packed_attention(Q, K, V, cu_q, cu_k, scale: float, causal: bool):
    """Q [T_q][h_q][d], K, V [T_k][h_kv][d] -> (O, lse [h_q][T_q], w [h_kv][T_k],
    A, delta): A = sum_k P·|V| per output, and per row the largest visible
    scale·sum_c |q_c||k_c| (what a rounding bound of the scores scales with).
    Tokens of no sequence get NaN."""
    T_q, h_q, d = Q.shape
    T_k, h_kv, _ = K.shape
    O = np.full((T_q, h_q, d), np.nan)
    A = np.full((T_q, h_q, d), np.nan)
    lse = np.full((h_q, T_q), np.nan)
    mag = np.full((h_q, T_q), np.nan)
    w = np.full((h_kv, T_k), np.nan)
    for i in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[i], cu_q[i + 1], cu_k[i], cu_k[i + 1]
        w[:, k0:k1] = 0.0
        see = visible(q1 - q0, k1 - k0, causal)
        for h in range(h_q):
            g = h // (h_q // h_kv)
            o, l, P, _ = attention(Q[q0:q1, h], K[k0:k1, g], V[k0:k1, g], scale, causal)
            O[q0:q1, h], lse[h, q0:q1] = o, l
            A[q0:q1, h] = P @ np.abs(V[k0:k1, g])
            s_abs = scale * (np.abs(Q[q0:q1, h]) @ np.abs(K[k0:k1, g]).T)
            mag[h, q0:q1] = np.max(np.where(see, s_abs, 0.0), axis=1, initial=0.0)
            w[g, k0:k1] += P.sum(axis=0)
    return O, lse, w, A, mag


def to_bf16(x):
    """Nearest bfloat16 (ties to even) of float64 values in its normal range, as float64."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def quantise(x):
    """[..., d] -> (codes [..., d], step [..., d/32], minimum [..., d/32]); x holds
    values of f32 or bf16, and the step and the codes' quotients are formed in f32."""
    g = np.asarray(x, dtype=np.float32).reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    lo, hi = g.min(-1), g.max(-1)
    step = to_bf16((hi - lo) / np.float32(15)).astype(np.float32)
    mn = to_bf16(lo).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((g - mn[..., None]) / step[..., None])
    codes = np.where(step[..., None] > 0, np.clip(q, 0, 15), 0).astype(np.int64)
    return codes.reshape(x.shape), step.astype(np.float64), mn.astype(np.float64)


def dequantise(codes, step, mn):
    g = codes.reshape(*codes.shape[:-1], codes.shape[-1] // GROUP, GROUP).astype(np.float64)
    return (mn[..., None] + step[..., None] * g).reshape(codes.shape)


def pack_keys(codes):
    """Rows of key codes to bytes: 32-bit words [4][ng], word (j, g) nibble i = channel 32g + 8j + i."""
    d = codes.shape[-1]
    ng = d // GROUP
    out = np.zeros((*codes.shape[:-1], 4, ng), dtype="<u4")
    for j in range(4):
        for g in range(ng):
            for i in range(8):
                out[..., j, g] |= codes[..., 32 * g + 8 * j + i].astype(np.uint32) << np.uint32(4 * i)
    return np.ascontiguousarray(out).view(np.uint8).reshape(*codes.shape[:-1], d // 2)


def pack_values(codes):
    """Rows of value codes to bytes: 16-bit words [8][ng], word (r, g) nibble i = channel 32g + 8i + r."""
    d = codes.shape[-1]
    ng = d // GROUP
    out = np.zeros((*codes.shape[:-1], 8, ng), dtype="<u2")
    for r in range(8):
        for g in range(ng):
            for i in range(4):
                out[..., r, g] |= (codes[..., 32 * g + 8 * i + r] << (4 * i)).astype(np.uint16)
    return np.ascontiguousarray(out).view(np.uint8).reshape(*codes.shape[:-1], d // 2)


def kept_tokens(w, budget: int, sink: int, recent: int):
    """Indices (ascending) one (sequence, head) of len(w) tokens keeps."""
    n = len(w)
    if n <= budget:
        return np.arange(n)
    middle = np.arange(sink, n - recent)
    order = middle[np.argsort(-np.asarray(w, dtype=np.float64)[middle], kind="stable")]
    return np.sort(np.concatenate([np.arange(sink), order[:budget - sink - recent], np.arange(n - recent, n)]))
