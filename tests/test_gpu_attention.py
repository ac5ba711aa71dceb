"""Packed-prompt attention, key weights, the 4-bit cache with its decode step,
and eviction, against the definitions in float64 (oracle/attention_oracle.py).

Tolerances, from the arithmetic the header promises (u = 2^-24, h = 2^-8 the
half step of bf16):
  scores   products of bf16 are exact in f32; a sum of d of them along a tree
           of height at most d + 16, each addition off by at most 2u, is off by
           at most e = 2u·(d + 16)·scale·sum|q||k|; forming scale·s·log2(e) - m
           and the exponential adds at most 2^-20·(1 + |x|), |x| <= the same
           magnitude: E = e + 2^-20·(1 + 2·scale·sum|q||k|) absolute in the
           exponent, so a relative error of at most 1.1·E per probability
  lse      E + 2^-21·(1 + |lse|)
  O        probabilities rounded to bf16 before the product (h), scores (2.2·E
           for numerator and denominator), f32 sums (2^-18): all relative to
           A = sum P|V|; then the store: h·|O| for bf16
  weights  (1.1·E + |lse| error E) + f32 sums 2^-18, relative to the sum."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from input_adaptive_reduced_02_b200 import rmm
from oracle import attention_oracle as AO

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, H = 2.0 ** -24, 2.0 ** -8


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def score_error(mag, d):
    return 2 * U * (d + 16) * mag + 2.0 ** -20 * (1 + 2 * mag)


def cum(x):
    return [0] + list(np.cumsum(x))


def i32(x):
    return torch.tensor([int(v) for v in x], dtype=torch.int32, device=DEV)


def randn(*shape, seed=0, dtype=torch.bfloat16, mul=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * mul).to(dtype)


# q lengths, k lengths, h_q, h_kv, d, causal
PROMPTS = [
    ([1], [1], 1, 1, 8, True),
    ([5], [5], 2, 1, 16, True),
    ([130], [130], 4, 2, 64, True),
    ([257], [257], 8, 2, 128, True),
    ([64, 1, 0, 200, 3], [64, 1, 0, 200, 3], 6, 2, 80, True),      # an empty sequence in the middle
    ([1, 17, 129], [300, 17, 500], 8, 1, 128, True),               # earlier keys before the queries
    ([40, 9], [3, 0], 4, 4, 64, True),                             # rows that see no key, a sequence with none
    ([100, 33], [70, 260], 3, 3, 72, False),                       # no mask, odd sizes
    ([384], [384], 14, 2, 96, True),                               # 7 query heads to a key head
    ([150], [150], 24, 1, 64, True),                               # 24 query heads to one key head
    ([20], [700], 40, 8, 128, False),
    ([640, 513], [640, 1030], 2, 2, 128, True),
    ([33], [33], 128, 1, 32, True),                                # 128 query heads to one key head
]


def prompt_ids(c):
    return f"q{'-'.join(map(str, c[0]))}_k{'-'.join(map(str, c[1]))}_h{c[2]}-{c[3]}_d{c[4]}_{'c' if c[5] else 'f'}"


def make_prompt(case, seed, strided=False, tail=0):
    ql, kl, hq, hk, d, causal = case
    tq, tk = sum(ql) + tail, sum(kl) + tail
    if strided:  # one [tokens][heads] buffer of queries, keys and values, when the tokens agree; head-major otherwise
        Q = randn(hq, tq, d, seed=seed, mul=2.0).transpose(0, 1)
        KV = randn(tk, 2 * hk, d + 8, seed=seed + 1)
        K, V = KV[:, :hk, :d], KV[:, hk:, :d]
    else:
        Q, K, V = randn(tq, hq, d, seed=seed, mul=2.0), randn(tk, hk, d, seed=seed + 1), randn(tk, hk, d, seed=seed + 2)
    if tail:
        for t, n in ((Q, sum(ql)), (K, sum(kl)), (V, sum(kl))):
            t[n:] = float("nan")
    return Q, K, V, i32(cum(ql)), i32(cum(kl))


def check_prompt(case, Q, K, V, O, lse, scale):
    ql, kl, hq, hk, d, causal = case
    nq, nk = sum(ql), sum(kl)
    Or, lr, wr, A, mag = AO.packed_attention(f64(Q)[:nq], f64(K)[:nk], f64(V)[:nk], cum(ql), cum(kl), scale, causal)
    E = score_error(mag, d)
    got_l = f64(lse)[:, :nq]
    empty = np.isneginf(lr)
    assert np.array_equal(np.isneginf(got_l), empty)
    ok = ~empty
    assert np.all(np.abs(got_l[ok] - lr[ok]) <= (E + 2.0 ** -21 * (1 + np.abs(lr)))[ok])
    got = f64(O)[:nq]
    Et = E.T[:, :, None]
    tol = (H + 2.2 * Et + 2.0 ** -18) * A
    if O.dtype == torch.bfloat16:
        tol = tol + H * (np.abs(Or) + tol)
    bad = ~(np.abs(got - Or) <= tol + 1e-37)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, worst {np.nanmax(np.abs(got - Or) / (tol + 1e-37)):.2f}"
    return wr, E


@pytest.mark.parametrize("strided", [False, True], ids=["packed", "strided"])
@pytest.mark.parametrize("case", PROMPTS, ids=prompt_ids)
def test_prompt_and_key_weights(case, strided):
    ql, kl, hq, hk, d, causal = case
    scale = d ** -0.5
    Q, K, V, cq, ck = make_prompt(case, 11 + d + sum(ql), strided)
    st = rmm.status_word()
    for dt in (torch.bfloat16, torch.float32):
        O, lse = rmm.attn_prompt(Q, K, V, cq, ck, out_dtype=dt, causal=causal, status=st)
        wr, E = check_prompt(case, Q, K, V, O, lse, scale)
    w_in = torch.rand(hk, sum(kl), device=DEV)
    w = rmm.attn_key_weights(Q, K, lse, cq, ck, causal=causal, w_in=w_in, status=st)
    rmm.check(st)
    e = E.max(initial=0.0)
    ref = f64(w_in) + wr
    assert np.all(np.abs(f64(w) - ref) <= (2.1 * e + 2.0 ** -18) * ref + 1e-30)
    # in place, and from nothing
    w2 = rmm.attn_key_weights(Q, K, lse, cq, ck, causal=causal, w_in=w_in, out=w_in)
    assert torch.equal(w2, w) and w2 is w_in
    w0 = rmm.attn_key_weights(Q, K, lse, cq, ck, causal=causal)
    assert np.all(np.abs(f64(w0) - wr) <= (2.1 * e + 2.0 ** -18) * wr + 1e-30)


@pytest.mark.parametrize("case", [PROMPTS[3], PROMPTS[4], PROMPTS[5], PROMPTS[7]], ids=prompt_ids)
def test_memory_outside_the_sequences_is_neither_used_nor_written(case):
    ql, kl, hq, hk, d, causal = case
    tail = 37
    Q, K, V, cq, ck = make_prompt(case, 3, tail=tail)
    out = torch.full((sum(ql) + tail, hq, d + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((hq, sum(ql) + tail), 7.0, device=DEV)
    w = torch.full((hk, sum(kl) + tail), 7.0, device=DEV)
    st = rmm.status_word()
    rmm.attn_prompt(Q, K, V, cq, ck, causal=causal, out=out[:, :, :d], lse=lse, status=st)
    rmm.attn_key_weights(Q, K, lse, cq, ck, causal=causal, out=w, status=st)
    rmm.check(st)
    check_prompt(case, Q, K, V, out[:, :, :d], lse, d ** -0.5)
    assert (out[sum(ql):] == 7).all() and (out[:, :, d:] == 7).all() and (lse[:, sum(ql):] == 7).all()
    assert (w[:, sum(kl):] == 7).all() and torch.isfinite(w).all()


def test_prompt_without_boundaries_large_scores_and_scale():
    case = ([300], [300], 4, 2, 64, True)
    Q, K, V, cq, ck = make_prompt(case, 21)
    Q, K = Q * 30, K * 30  # scores of thousands: the softmax picks single keys
    a = rmm.attn_prompt(Q, K, V, scale=0.5)
    b = rmm.attn_prompt(Q, K, V, cq, ck, scale=0.5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_prompt(case, Q, K, V, *a, 0.5)


def test_nonfinite_queries_are_reported_and_stay_in_their_rows():
    case = ([200], [200], 2, 1, 128, True)
    Q, K, V, cq, ck = make_prompt(case, 5)
    O, lse = rmm.attn_prompt(Q, K, V, cq, ck)
    Q[100, 1, 3] = float("nan")
    st = rmm.status_word()
    O2, lse2 = rmm.attn_prompt(Q, K, V, cq, ck, status=st)
    keep = torch.ones(200, 2, dtype=torch.bool, device=DEV)
    keep[100, 1] = False
    assert torch.equal(O[keep], O2[keep]) and torch.isnan(O2[100, 1]).all()
    with pytest.raises(rmm.RMMError) as e:
        rmm.check(st)
    assert e.value.status == rmm.RMM_ERR_NONFINITE


def test_long_prompt_sampled_rows():
    """Rows of a long sequence against the definition (whole P would not fit a test)."""
    S, hq, hk, d = 5000, 8, 2, 128
    Q, K, V = randn(S, hq, d, seed=1, mul=2.0), randn(S, hk, d, seed=2), randn(S, hk, d, seed=3)
    O, lse = rmm.attn_prompt(Q, K, V, out_dtype=torch.bfloat16)
    w = rmm.attn_key_weights(Q, K, lse)
    assert abs(f64(w).sum() - S * hq) <= S * hq * 2.0 ** -12
    scale = d ** -0.5
    for h in (0, 5):
        rows = np.r_[0:3, 127:130, 255:258, 2500, 4095:4098, S - 2:S]
        q, k, v = f64(Q[:, h])[rows], f64(K[:, h // 4]), f64(V[:, h // 4])
        X = scale * q @ k.T
        X[np.arange(S)[None, :] > rows[:, None]] = -np.inf
        m = X.max(1, keepdims=True)
        P = np.exp(X - m)
        tot = P.sum(1, keepdims=True)
        P /= tot
        E = score_error((scale * np.abs(q) @ np.abs(k).T).max(1), d)[:, None]
        tol = (H + 2.2 * E + 2.0 ** -18) * (P @ np.abs(v))
        assert np.all(np.abs(f64(O[:, h])[rows] - P @ v) <= tol + H * (np.abs(P @ v) + tol))
        lr = (m + np.log(tot))[:, 0]
        assert np.all(np.abs(f64(lse[h])[rows] - lr) <= E[:, 0] + 2.0 ** -21 * (1 + np.abs(lr)))


# ---------------------------------------------------------------- the 4-bit cache
def stored(cache, b, h, n):
    """float64 values of the first n rows, decoded from the planes by the header's layout."""
    d, ng = cache.d, cache.d // 32
    kw = cache.kc[b, h, :n].cpu().numpy().view("<u4").reshape(n, 4, ng)
    vw = cache.vc[b, h, :n].cpu().numpy().view("<u2").reshape(n, 8, ng)
    kc, vc = np.zeros((n, d), np.int64), np.zeros((n, d), np.int64)
    for g in range(ng):
        for j in range(4):
            for i in range(8):
                kc[:, 32 * g + 8 * j + i] = (kw[:, j, g] >> np.uint32(4 * i)) & 15
        for r in range(8):
            for i in range(4):
                vc[:, 32 * g + 8 * i + r] = (vw[:, r, g].astype(np.int64) >> (4 * i)) & 15
    ks, vs = f64(cache.ks[b, h, :n]), f64(cache.vs[b, h, :n])
    return AO.dequantise(kc, ks[..., 0], ks[..., 1]), AO.dequantise(vc, vs[..., 0], vs[..., 1]), (kc, ks, vc, vs)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens,heads,d", [([1], 1, 32), ([3, 0, 70], 2, 64), ([40, 5], 3, 96), ([129], 2, 128)])
def test_store_matches_the_format(lens, heads, d, dtype):
    n, T, cap = len(lens), sum(lens), max(lens) + 9
    K, V = randn(T, heads, d, seed=d, dtype=dtype, mul=3.0), randn(T, heads, d + 3, seed=d + 1, dtype=dtype)[:, :, :d]
    K[0, 0, :32] = 2.5          # a constant group: step 0
    V[0, 0, 0] = 1000.0         # one far value
    start = [i % 4 for i in range(n)]
    cache = rmm.KV4Cache.empty(n, heads, cap, d)
    for t in (cache.kc, cache.vc):
        t.fill_(0xAB)
    cache.w.fill_(9.0)
    w_new = torch.rand(heads, T, device=DEV)
    st = rmm.status_word()
    rmm.kv4_store(cache, K, V, i32(start), i32(cum(lens)), w_new=w_new, status=st)
    rmm.check(st)
    cu = cum(lens)
    for b in range(n):
        for h in range(heads):
            s0, s1 = start[b], start[b] + lens[b]
            _, _, (kc, ks, vc, vs) = stored(cache, b, h, cap)
            for x, c, s in ((K, kc, ks), (V, vc, vs)):
                codes, step, mn = AO.quantise(x[cu[b]:cu[b + 1], h].float().cpu().numpy())
                assert np.array_equal(s[s0:s1, :, 0], step) and np.array_equal(s[s0:s1, :, 1], mn)
                assert np.array_equal(c[s0:s1], codes)
            # bytes as the layout says, and nothing else written
            assert np.array_equal(cache.kc[b, h, s0:s1].cpu().numpy(), AO.pack_keys(kc[s0:s1]))
            assert np.array_equal(cache.vc[b, h, s0:s1].cpu().numpy(), AO.pack_values(vc[s0:s1]))
            rest = torch.ones(cap, dtype=torch.bool, device=DEV)
            rest[s0:s1] = False
            assert (cache.kc[b, h][rest] == 0xAB).all() and (cache.vc[b, h][rest] == 0xAB).all()
            assert (cache.w[b, h][rest] == 9.0).all() and (cache.ks[b, h][rest] == 0).all()
            assert torch.equal(cache.w[b, h, s0:s1], w_new[h, cu[b]:cu[b + 1]])


def test_store_reports_slots_outside_the_cache_and_nonfinite_values():
    cache = rmm.KV4Cache.empty(2, 2, 8, 64)
    K, V = randn(2, 2, 64, seed=1), randn(2, 2, 64, seed=2)
    st = rmm.status_word()
    rmm.kv4_store(cache, K, V, i32([8, 3]), status=st)  # sequence 0 is full
    assert (cache.ks[0] == 0).all() and (cache.ks[1, :, 3] != 0).any()
    with pytest.raises(rmm.RMMError) as e:
        rmm.check(st)
    assert e.value.status == rmm.RMM_ERR_INVALID
    before = cache.ks.clone()
    rmm.kv4_store(cache, K, V, i32([-1, -5]), status=st)
    assert torch.equal(cache.ks, before)
    with pytest.raises(rmm.RMMError):
        rmm.check(st)
    K[1, 0, 5] = float("inf")
    rmm.kv4_store(cache, K, V, i32([0, 4]), status=st)
    with pytest.raises(rmm.RMMError) as e:
        rmm.check(st)
    assert e.value.status == rmm.RMM_ERR_NONFINITE


DECODES = [  # lens, cap, h_q, h_kv, d
    ([1], 1, 1, 1, 32),
    ([5, 0, 16], 17, 2, 1, 64),
    ([100], 128, 4, 4, 96),
    ([129, 128, 127], 130, 8, 2, 128),
    ([1000, 33], 1024, 14, 2, 128),
    ([700], 2000, 40, 8, 64),
    ([300, 1], 300, 24, 1, 128),   # 24 query heads to one key head
    ([64], 64, 33, 1, 96),         # 33 query heads to one key head
    ([4097, 2050], 5000, 16, 2, 128),
]


def filled_cache(lens, cap, hk, d, seed):
    n = len(lens)
    cache = rmm.KV4Cache.empty(n, hk, cap, d)
    T = sum(lens)
    K = randn(T, hk, d, seed=seed) + 2 * randn(1, hk, d, seed=seed + 1)
    V = randn(T, hk, d, seed=seed + 2)
    if T:
        rmm.kv4_store(cache, K, V, i32([0] * n), i32(cum(lens)))
    return cache


def check_decode(Q, cache, lens, O, lse, scale, w=None, w_in=None):
    n, hq, d = Q.shape
    gq = hq // cache.heads
    for b in range(n):
        for h in range(cache.heads):
            L = lens[b]
            k, v, (vc, vs) = (lambda a: (a[0], a[1], a[2][2:]))(stored(cache, b, h, L))
            vmag = AO.dequantise(vc, vs[..., 0], np.abs(vs[..., 1]))  # s·c + |m|
            q = f64(Q[b, h * gq:(h + 1) * gq])
            Or, lr, P, _ = AO.attention(q, k, v, scale, False)
            mag = np.max(scale * np.abs(q) @ (np.abs(k) + 0).T, axis=1, initial=0.0)
            kd = stored(cache, b, h, L)[2][:2]
            kmag = AO.dequantise(kd[0], kd[1][..., 0], np.abs(kd[1][..., 1]))
            mag = np.maximum(mag, np.max(scale * np.abs(q) @ kmag.T, axis=1, initial=0.0))
            E = score_error(mag, d)
            got, gl = f64(O[b, h * gq:(h + 1) * gq]), f64(lse[b, h * gq:(h + 1) * gq])
            if L == 0:
                assert (got == 0).all() and np.isneginf(gl).all()
                continue
            assert np.all(np.abs(gl - lr) <= E + 2.0 ** -21 * (1 + np.abs(lr)))
            # the probabilities times the steps, and the probabilities themselves, are rounded to bf16
            tol = (H + 2.2 * E[:, None] + 2.0 ** -18) * (P @ vmag)
            if O.dtype == torch.bfloat16:
                tol = tol + H * (np.abs(Or) + tol)
            err = np.abs(got - Or)
            assert np.all(err <= tol), f"worst {np.max(err / tol):.2f}"
            if w is not None:
                ref = P.sum(0) + (f64(w_in[b, h, :L]) if w_in is not None else 0.0)
                assert np.all(np.abs(f64(w[b, h, :L]) - ref) <= (2.1 * E.max() + 2.0 ** -18) * ref + 1e-30)


@pytest.mark.parametrize("case", DECODES, ids=lambda c: f"l{'-'.join(map(str, c[0]))}_h{c[2]}-{c[3]}_d{c[4]}")
def test_decode_on_the_4_bit_cache(case):
    lens, cap, hq, hk, d = case
    n = len(lens)
    cache = filled_cache(lens, cap, hk, d, seed=d + cap)
    for t in (cache.ks, cache.vs):  # slots past the lengths hold garbage
        for b in range(n):
            t[b, :, lens[b]:] = float("nan")
    Q = randn(hq, n, d, seed=9, mul=2.0).transpose(0, 1)
    L = i32(lens)
    O, lse, ws = rmm.kv4_attn(Q, cache, L, out_dtype=torch.bfloat16)
    rmm.check(ws)
    check_decode(Q, cache, lens, O, lse, d ** -0.5)
    cache.w.uniform_()
    w_in, w_out = cache.w.clone(), torch.full_like(cache.w, 5.0)
    O2, lse2, ws = rmm.kv4_attn(Q, cache, L, scale=0.3, w_in=w_in, w_out=w_out)
    rmm.check(ws)
    check_decode(Q, cache, lens, O2, lse2, 0.3, w_out, w_in)
    for b in range(n):
        assert (w_out[b, :, lens[b]:] == 5.0).all()
    O3, lse3, _ = rmm.kv4_attn(Q, cache, L, scale=0.3, w_in=cache.w, w_out=cache.w, workspace=ws)
    assert torch.equal(O3, O2) and torch.equal(lse3, lse2)
    for b in range(n):
        assert torch.equal(cache.w[b, :, :lens[b]], w_out[b, :, :lens[b]])
    O4, _, _ = rmm.kv4_attn(Q, cache, L, scale=0.3, w_out=w_out)
    assert torch.equal(O4, O2)
    check_decode(Q, cache, lens, O4, lse2, 0.3, w_out)


def test_decode_lengths_are_clamped_to_the_capacity():
    cache = filled_cache([64, 64], 64, 2, 64, seed=1)
    Q = randn(2, 4, 64, seed=2)
    a = rmm.kv4_attn(Q, cache, i32([64, 0]))
    b = rmm.kv4_attn(Q, cache, i32([1 << 30, -7]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------- eviction
EVICTS = [  # lens, cap, heads, budget, sink, recent
    ([10], 10, 1, 4, 1, 1),
    ([10, 3, 0, 8], 12, 2, 8, 2, 3),
    ([700, 1000, 64], 1000, 3, 64, 4, 16),
    ([5000], 5000, 2, 1000, 0, 0),
    ([513], 600, 2, 512, 0, 512),      # only the last ones
    ([513], 600, 1, 512, 512, 0),      # only the first ones
    ([2049, 2048], 4096, 2, 2047, 1, 1000),
    ([300], 400, 2, 1, 0, 0),
]


@pytest.mark.parametrize("in_place", [False, True], ids=["copy", "in_place"])
@pytest.mark.parametrize("case", EVICTS, ids=lambda c: f"l{'-'.join(map(str, c[0]))}_b{c[3]}_s{c[4]}_r{c[5]}")
def test_eviction(case, in_place):
    lens, cap, heads, budget, sink, recent = case
    n = len(lens)
    g = torch.Generator(device=DEV)
    g.manual_seed(cap)
    w = torch.rand(n, heads, cap, generator=g, device=DEV)
    w[:, 0] = (w[:, 0] * 4).floor()  # many ties
    w[:, :, ::7] = 0.0
    w[:, :, 3::11] = -0.0
    for b in range(n):
        w[b, :, lens[b]:] = float("nan")  # past the length: not looked at
    planes = [torch.randint(0, 255, (n, heads, cap, 64), dtype=torch.uint8, device=DEV, generator=g),
              torch.randn(n, heads, cap, 3, device=DEV, generator=g),            # 12-byte rows
              torch.randn(n, heads, cap, 128, device=DEV, generator=g).bfloat16(),
              torch.arange(cap, dtype=torch.int32, device=DEV).expand(n, heads, cap).contiguous(), w]
    orig = [p.clone() for p in planes]
    L = i32(lens)
    if in_place:
        L_out, idx, ws = rmm.cache_evict(w, L, planes, budget, sink, recent, lens_out=L)
        dst = planes
    else:
        dst = [torch.full((n, heads, budget + 3, *p.shape[3:]), 77, dtype=p.dtype, device=DEV) for p in planes]
        L_out, idx, ws = rmm.cache_evict(w, L, list(zip(planes, dst)), budget, sink, recent)
        for p, o in zip(planes, orig):
            assert torch.equal(p.view(torch.uint8), o.view(torch.uint8))
    rmm.check(ws)
    assert L_out.tolist() == [min(x, budget) for x in lens]
    for b in range(n):
        for h in range(heads):
            keep = AO.kept_tokens(f64(orig[4][b, h, :lens[b]]), budget, sink, recent)
            m = len(keep)
            assert idx[b, h, :m].tolist() == keep.tolist() and (idx[b, h, m:] == -1).all()
            at = torch.tensor(keep, dtype=torch.long, device=DEV)
            for p, o in zip(dst, orig):
                got, want = p[b, h, :m].contiguous(), o[b, h][at].contiguous()
                assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
                if not in_place:
                    assert (p[b, h, m:] == 77).all()


def test_eviction_reports_nan_weights():
    w = torch.rand(1, 1, 100, device=DEV)
    w[0, 0, 50] = float("nan")
    _, idx, ws = rmm.cache_evict(w, i32([100]), [], 40, 2, 2)
    with pytest.raises(rmm.RMMError) as e:
        rmm.check(ws)
    assert e.value.status == rmm.RMM_ERR_NONFINITE
    assert (idx.sort(-1).values == idx).all() and idx.unique().numel() == 40  # still a valid set of tokens


# ---------------------------------------------------------------- together
def serve(prompts, hq, hk, d, cap, budget, steps, rmm_calls=True):
    """A prompt pass, its keys into a 4-bit cache with their weights, then decode
    steps that evict whenever a cache is at its budget."""
    n = len(prompts)
    T = sum(prompts)
    Q, K, V = randn(T, hq, d, seed=1, mul=2.0), randn(T, hk, d, seed=2), randn(T, hk, d, seed=3)
    cu = i32(cum(prompts))
    O, lse = rmm.attn_prompt(Q, K, V, cu, cu)
    w = rmm.attn_key_weights(Q, K, lse, cu, cu)
    cache = rmm.KV4Cache.empty(n, hk, cap, d)
    rmm.kv4_store(cache, K, V, i32([0] * n), cu, w_new=w)
    lens = i32(prompts)
    out = []
    for s in range(steps):
        q, k, v = (randn(n, h, d, seed=100 + 3 * s + j, mul=m) for j, (h, m) in enumerate(((hq, 2.0), (hk, 1), (hk, 1))))
        rmm.kv4_store(cache, k, v, lens)
        lens = lens + 1
        o, l, ws = rmm.kv4_attn(q, cache, lens, w_in=cache.w, w_out=cache.w)
        rmm.check(ws)
        check_decode(q, cache, lens.tolist(), o, l, d ** -0.5)
        out.append(o)
        before = f64(cache.w)
        old = lens.tolist()
        _, idx, ws = rmm.cache_evict(cache.w, lens, cache.planes(), budget, sink=2, recent=8, lens_out=lens)
        rmm.check(ws)
        for b in range(n):
            for h in range(hk):
                keep = AO.kept_tokens(before[b, h, :old[b]], budget, 2, 8)
                assert idx[b, h, :len(keep)].tolist() == keep.tolist()
                assert np.array_equal(f64(cache.w)[b, h, :len(keep)], before[b, h][keep])
    return out, lens


def test_prompt_store_decode_and_evict_together():
    out, lens = serve([90, 200, 31], 8, 2, 64, cap=256, budget=64, steps=40)
    assert lens.tolist() == [64, 64, 64]
    again, _ = serve([90, 200, 31], 8, 2, 64, cap=256, budget=64, steps=40)
    assert all(torch.equal(a, b) for a, b in zip(out, again))  # the same bits every time


def test_captured_step_replays_and_two_streams_agree():
    """The decode step captured in a graph, replayed with other inputs; the calls
    on a side stream next to the same calls on another."""
    n, hq, hk, d, cap = 3, 8, 2, 128, 512
    lens = [500, 37, 255]
    cache = filled_cache(lens, cap, hk, d, seed=4)
    q, L = randn(n, hq, d, seed=1), i32(lens)
    k, v = randn(n, hk, d, seed=2), randn(n, hk, d, seed=3)
    w = torch.zeros(n, hk, cap, device=DEV)
    o, l, ws = rmm.kv4_attn(q, cache, L, w_out=w)
    pq = randn(300, hq, d, seed=8)
    pk = randn(300, hk, d, seed=9)
    po, pl = rmm.attn_prompt(pq, pk, pk)
    pw = rmm.attn_key_weights(pq, pk, pl)
    idx = torch.empty(n, hk, 64, dtype=torch.int32, device=DEV)
    lo = torch.empty_like(L)
    ews = rmm.cache_evict(w, L, [], 64, lens_out=lo, idx_out=idx)[2]
    want = [t.clone() for t in (po, pl, pw, idx, lo)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            rmm.kv4_store(cache, k, v, L - 1)
            rmm.kv4_attn(q, cache, L, out=o, lse=l, w_out=w, workspace=ws)
            rmm.attn_prompt(pq, pk, pk, out=po, lse=pl)
            rmm.attn_key_weights(pq, pk, pl, out=pw)
            rmm.cache_evict(w, L, [], 64, lens_out=lo, idx_out=idx, workspace=ews)
    torch.cuda.synchronize()
    for seed in (5, 6):
        q.copy_(randn(n, hq, d, seed=seed, mul=2.0))
        k.copy_(randn(n, hk, d, seed=seed + 10))
        for t in (po, pl, pw):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        check_decode(q, cache, lens, o, l, d ** -0.5, w)
        assert all(torch.equal(a, b) for a, b in zip((po, pl, pw), want[:3]))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    res = []
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            a = rmm.attn_prompt(pq, pk, pk)
            res.append((*a, rmm.attn_key_weights(pq, pk, a[1]), *rmm.kv4_attn(q, cache, L)[:2]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert torch.equal(res[0][0], want[0])


def test_empty_calls():
    z = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    O, lse = rmm.attn_prompt(z, z, z)
    assert O.shape == (0, 4, 64) and lse.shape == (4, 0)
    Q = randn(3, 4, 64)
    O, lse = rmm.attn_prompt(Q, z, z)  # no keys at all
    assert (O == 0).all() and torch.isneginf(lse).all()
    assert rmm.attn_key_weights(Q, z, lse).shape == (4, 0)
    w_in = torch.rand(4, 3, device=DEV)
    w = rmm.attn_key_weights(z, Q, torch.empty(4, 0, device=DEV), w_in=w_in)  # no queries
    assert torch.equal(w, w_in)
    cache = rmm.KV4Cache.empty(0, 2, 8, 64)
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    rmm.kv4_store(cache, z[:, :2], z[:, :2], e)
    _, _, ws = rmm.kv4_attn(z, cache, e)
    rmm.check(ws)
    _, _, ws = rmm.cache_evict(cache.w, e, cache.planes(), 4)
    rmm.check(ws)
