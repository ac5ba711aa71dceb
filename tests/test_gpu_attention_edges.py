"""The attention operators where their partitioning changes: many sequences,
more than one stretch per sequence, planes beyond 4 GB, capacities above what a
selection keeps in registers, values of extreme size. Tolerances as derived in
test_gpu_attention.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from input_adaptive_reduced_02_b200 import rmm
from oracle import attention_oracle as AO
from test_gpu_attention import (DEV, H, check_decode, check_prompt, cum, f64, filled_cache, i32, make_prompt, randn,
                                score_error)

pytestmark = pytest.mark.gpu


def test_prompt_of_many_sequences():
    rng = np.random.default_rng(1)
    ql = [int(x) for x in rng.integers(0, 40, 75)]  # three warps' worth of boundaries, some sequences empty
    kl = [q + int(x) for q, x in zip(ql, rng.integers(0, 90, 75))]
    case = (ql, kl, 6, 2, 64, True)
    Q, K, V, cq, ck = make_prompt(case, 2)
    O, lse = rmm.attn_prompt(Q, K, V, cq, ck)
    wr, E = check_prompt(case, Q, K, V, O, lse, 0.125)
    w = rmm.attn_key_weights(Q, K, lse, cq, ck)
    assert np.all(np.abs(f64(w) - wr) <= (2.1 * E.max() + 2.0 ** -18) * wr + 1e-30)


def test_head_major_output_and_boundaries_inside_the_tokens():
    """An output of [heads][tokens][d] memory, and a single sequence that is a part of the tokens."""
    case = ([200], [260], 4, 2, 96, True)
    Q, K, V, _, _ = make_prompt(case, 4)
    pad = lambda t, a, b: torch.cat((torch.full((a, *t.shape[1:]), float("nan"), dtype=t.dtype, device=DEV), t,  # noqa: E731
                                     torch.full((b, *t.shape[1:]), float("nan"), dtype=t.dtype, device=DEV)))
    Qp, Kp, Vp = pad(Q, 3, 9), pad(K, 5, 70), pad(V, 5, 70)
    out = torch.full((4, 212, 96), 7.0, device=DEV).transpose(0, 1)
    lse = torch.full((4, 212), 7.0, device=DEV)
    st = rmm.status_word()
    rmm.attn_prompt(Qp, Kp, Vp, i32([3, 203]), i32([5, 265]), out=out, lse=lse, status=st)
    w = torch.full((2, 335), 7.0, device=DEV)
    rmm.attn_key_weights(Qp, Kp, lse, i32([3, 203]), i32([5, 265]), out=w, status=st)
    rmm.check(st)
    wr, E = check_prompt(case, Q, K, V, out[3:203], lse[:, 3:203], 96 ** -0.5)
    assert (out[:3] == 7).all() and (out[203:] == 7).all() and (lse[:, :3] == 7).all() and (lse[:, 203:] == 7).all()
    assert (w[:, :5] == 7).all() and (w[:, 265:] == 7).all()
    assert np.all(np.abs(f64(w[:, 5:265]) - wr) <= (2.1 * E.max() + 2.0 ** -18) * wr + 1e-30)


def test_a_nan_query_reaches_only_the_weights_of_keys_it_sees():
    case = ([300], [300], 4, 1, 128, True)
    Q, K, V, cq, ck = make_prompt(case, 6)
    _, lse = rmm.attn_prompt(Q, K, V, cq, ck)
    w = rmm.attn_key_weights(Q, K, lse, cq, ck)
    Q[10, 2, 0] = float("nan")
    lse2 = lse.clone()
    lse2[2, 10] = float("nan")
    st = rmm.status_word()
    w2 = rmm.attn_key_weights(Q, K, lse2, cq, ck, status=st)
    assert torch.isnan(w2[:, :11]).all() and torch.equal(w2[:, 11:], w[:, 11:])
    with pytest.raises(rmm.RMMError) as e:
        rmm.check(st)
    assert e.value.status == rmm.RMM_ERR_NONFINITE


def test_key_weights_of_few_keys_and_many_queries():
    """Queries without causal order over one tile of keys: the clusters share them."""
    case = ([3000], [100], 4, 2, 64, False)
    Q, K, V, cq, ck = make_prompt(case, 8)
    _, lse = rmm.attn_prompt(Q, K, V, cq, ck, causal=False)
    w = rmm.attn_key_weights(Q, K, lse, cq, ck, causal=False)
    _, _, wr, _, mag = AO.packed_attention(f64(Q), f64(K), f64(V), [0, 3000], [0, 100], 0.125, False)
    E = score_error(mag, 64).max()
    assert np.all(np.abs(f64(w) - wr) <= (2.1 * E + 2.0 ** -18) * wr)
    assert torch.equal(w, rmm.attn_key_weights(Q, K, lse, cq, ck, causal=False))


@pytest.mark.parametrize("hq,hk,d", [(4, 1, 64), (3, 3, 32), (16, 2, 96), (20, 1, 128)])
def test_decode_of_many_sequences(hq, hk, d):
    """More sequences than threads of a block, empty ones among them; up to 4, 8 and 16 heads to a key head."""
    rng = np.random.default_rng(d)
    n, cap = 300, 70
    lens = [int(x) for x in rng.integers(0, cap + 1, n)]
    lens[0] = lens[-1] = lens[150] = 0
    cache = filled_cache(lens, cap, hk, d, seed=d)
    Q = randn(n, hq, d, seed=5, mul=2.0)
    w_out = torch.full((n, hk, cap), 3.0, device=DEV)
    O, lse, ws = rmm.kv4_attn(Q, cache, i32(lens), w_out=w_out)
    rmm.check(ws)
    pick = [0, 1, 2, 77, 149, 150, 151, 254, 255, 256, 257, 298, 299]
    sub = rmm.KV4Cache(*(t[pick].contiguous() for t in (cache.kc, cache.ks, cache.vc, cache.vs)))
    check_decode(Q[pick], sub, [lens[i] for i in pick], O[pick], lse[pick], d ** -0.5, w_out[pick])
    for b in range(n):
        assert (w_out[b, :, lens[b]:] == 3.0).all()
        if lens[b] == 0:
            assert (O[b] == 0).all() and torch.isneginf(lse[b]).all()
    total = torch.where(torch.arange(cap, device=DEV) < i32(lens)[:, None, None], w_out, 0.0).double().sum(-1)
    want = torch.tensor([float(hq // hk) if x else 0.0 for x in lens], dtype=torch.float64, device=DEV)[:, None]
    assert ((total - want).abs() <= want * 2.0 ** -12).all()


@pytest.mark.parametrize("mul", [1e-12, 1.0, 2.0 ** 40], ids=["tiny", "ones", "huge"])
def test_decode_of_values_of_any_size(mul):
    """Steps from 2^-40 to 2^40, queries and keys scaled against each other."""
    n, hq, hk, d, L = 2, 8, 2, 64, 100
    cache = rmm.KV4Cache.empty(n, hk, 128, d)
    K, V = randn(n * L, hk, d, seed=1).float() / mul, randn(n * L, hk, d, seed=2).float() * mul
    rmm.kv4_store(cache, K, V, i32([0, 0]), i32([0, L, 2 * L]))
    Q = (randn(n, hq, d, seed=3).float() * mul).bfloat16()
    Q[0, 0] = 0                      # a head of zeros: every token weighs the same
    Q[1, 1, 1:] = 0                  # one channel, next to nothing beside it
    Q[1, 1, 5] = mul * 2.0 ** -30
    O, lse, ws = rmm.kv4_attn(Q, cache, i32([L, L]))
    rmm.check(ws)
    check_decode(Q, cache, [L, L], O, lse, d ** -0.5)
    assert abs(lse[0, 0].item() - np.log(L)) < 1e-6


def test_decode_of_values_that_grow_along_the_sequence():
    """Steps from 2^-2 up to 2^28 and back, the probabilities of the small ones near 1 in some heads."""
    L, hq, hk, d = 400, 8, 2, 64
    cache = rmm.KV4Cache.empty(1, hk, L, d)
    t = torch.arange(L, device=DEV)
    grow = torch.exp2(torch.minimum(t, L - t).float() / 7).view(L, 1, 1)
    K, V = randn(L, hk, d, seed=1).float(), randn(L, hk, d, seed=2).float() * grow
    K[7] += 6.0  # a token of small values that takes most of the weight where the query is positive
    rmm.kv4_store(cache, K, V, i32([0]), i32([0, L]))
    Q = randn(1, hq, d, seed=3, mul=0.2)
    Q[0, ::2] = Q[0, ::2].abs()
    O, lse, ws = rmm.kv4_attn(Q, cache, i32([L]))
    rmm.check(ws)
    check_decode(Q, cache, [L], O, lse, d ** -0.5)


def test_decode_reports_nan_scales():
    cache = filled_cache([40, 40], 64, 1, 64, seed=1)
    cache.ks[1, 0, 17] = float("nan")
    O, lse, ws = rmm.kv4_attn(randn(2, 2, 64, seed=2), cache, i32([40, 40]))
    assert torch.isfinite(O[0]).all() and torch.isnan(lse[1]).all()
    with pytest.raises(rmm.RMMError) as e:
        rmm.check(ws)
    assert e.value.status == rmm.RMM_ERR_NONFINITE
    O, _, ws = rmm.kv4_attn(randn(2, 2, 64, seed=2), cache, i32([40, 17]), workspace=ws)  # not a cached token
    rmm.check(ws)
    assert torch.isfinite(O).all()


def test_planes_beyond_4_gib():
    """The last rows of a cache whose code planes are 4.3 GB each: zeros but for the last 40 tokens of one head."""
    hk, cap, d, n = 33, 1 << 21, 128, 40
    cache = rmm.KV4Cache.empty(1, hk, cap, d, weights=False)
    assert cache.kc.numel() > 1 << 32
    K, V = randn(n, hk, d, seed=1), randn(n, hk, d, seed=2)
    rmm.kv4_store(cache, K, V, i32([cap - n]), i32([0, n]))
    Q = randn(1, hk, d, seed=3, mul=2.0)
    O, lse, ws = rmm.kv4_attn(Q, cache, i32([cap]))
    rmm.check(ws)
    for h in (0, 16, 32):
        c, s, m = AO.quantise(K[:, h].float().cpu().numpy())
        k = AO.dequantise(c, s, m)
        c, s, m = AO.quantise(V[:, h].float().cpu().numpy())
        v, vmag = AO.dequantise(c, s, m), AO.dequantise(c, s, np.abs(m))
        q = f64(Q[0, h])
        x = d ** -0.5 * k @ q
        E = score_error(d ** -0.5 * (np.abs(k) @ np.abs(q)).max() * 3, d)  # |s·c| + |m| is at most 3 times a row here
        total = np.exp(x).sum() + (cap - n)
        p = np.exp(x) / total
        assert abs(lse[0, h].item() - np.log(total)) <= E + 2.0 ** -21 * 16
        assert np.all(np.abs(f64(O[0, h]) - p @ v) <= (H + 2.2 * E + 2.0 ** -18) * (p @ vmag))
    # the same rows through eviction: the last ones stay, the rest of the budget goes to the first zeros
    w = torch.zeros(1, hk, cap, device=DEV)
    dst = [torch.empty(1, hk, 64, *t.shape[3:], dtype=t.dtype, device=DEV) for t in (cache.kc, cache.ks)]
    L, idx, ws = rmm.cache_evict(w, i32([cap]), [(cache.kc, dst[0]), (cache.ks, dst[1])], 64, recent=n)
    rmm.check(ws)
    keep = torch.cat((torch.arange(24), torch.arange(cap - n, cap))).to(DEV)
    assert torch.equal(idx[0, 32].long(), keep)
    assert torch.equal(dst[0][0, 32], cache.kc[0, 32][keep]) and torch.equal(dst[1][0, 32], cache.ks[0, 32][keep])


@pytest.mark.parametrize("cap,n", [(2048, 2048), (2049, 2049), (8192, 8190), (8193, 8193), (40000, 39999)])
@pytest.mark.parametrize("kind", ["equal", "two_values", "spread", "negative", "subnormal"])
def test_eviction_at_every_selection_width(cap, n, kind):
    g = torch.Generator(device=DEV)
    g.manual_seed(cap)
    w = torch.rand(1, 2, cap, generator=g, device=DEV)
    w = {"equal": torch.full_like(w, 0.25), "two_values": (w > 0.7).float(), "spread": torch.exp(80 * w - 60),
         "negative": w - 0.5, "subnormal": w * 1e-40}[kind]
    budget, sink, recent = n // 3, 5, 100
    _, idx, ws = rmm.cache_evict(w, i32([n]), [], budget, sink, recent)
    rmm.check(ws)
    for h in range(2):
        assert idx[0, h].tolist() == AO.kept_tokens(f64(w[0, h, :n]), budget, sink, recent).tolist()


def test_eviction_in_place_of_wide_rows():
    """Rows in several column slices, several blocks of rows, beside a copied plane."""
    n, heads, cap, budget = 2, 2, 3000, 1700
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    w = torch.rand(n, heads, cap, generator=g, device=DEV)
    wide = torch.randn(n, heads, cap, 300, generator=g, device=DEV)       # 1200-byte rows
    odd = torch.randn(n, heads, cap, 7, generator=g, device=DEV)          # 28-byte rows
    copy = torch.randn(n, heads, cap, 48, generator=g, device=DEV).bfloat16()
    dst = torch.zeros(n, heads, cap, 48, device=DEV).bfloat16()
    old = [t.clone() for t in (w, wide, odd)]
    lens = i32([3000, 1699])
    out, idx, ws = rmm.cache_evict(w, lens, [wide, (copy, dst), odd, w], budget, 3, 50)
    rmm.check(ws)
    assert out.tolist() == [1700, 1699]
    for b in range(n):
        for h in range(heads):
            keep = AO.kept_tokens(f64(old[0][b, h, :lens[b].item()]), budget, 3, 50)
            at = torch.tensor(keep, dtype=torch.long, device=DEV)
            m = len(keep)
            for t, o in ((wide, old[1]), (odd, old[2]), (w, old[0]), (dst, copy)):
                assert torch.equal(t[b, h, :m], o[b, h][at])
            assert (dst[b, h, m:] == 0).all()


def test_store_rounds_as_the_definition_next_to_halves():
    """f32 values on and next to the borders between codes, groups far from zero, tiny and huge steps."""
    rng = np.random.default_rng(5)
    rows = []
    for scale, shift in ((1.0, 0.0), (15.0, -7.5), (1e-30, 0.0), (1e30, 0.0), (1.0, 4096.0), (3e-39, 0.0), (1e-3, -100.0)):
        x = np.concatenate(([0.0, 15.0], rng.integers(0, 15, 30) + 0.5 + rng.integers(-2, 3, 30) * 2.0 ** -19))
        rows.append(np.concatenate([x * scale + shift, rng.standard_normal(32) * scale + shift]))
    x = torch.tensor(np.array(rows), dtype=torch.float32, device=DEV)[:, None, :].contiguous()
    T = x.shape[0]
    cache = rmm.KV4Cache.empty(1, 1, T, 64)
    rmm.kv4_store(cache, x, x, i32([0]), i32([0, T]))
    codes, step, mn = AO.quantise(x[:, 0].cpu().numpy())
    normal = (step == 0) | (step >= 2.0 ** -126)  # bf16 subnormals: the oracle's rounding is for normal ones
    for plane, scales, pack in ((cache.kc, cache.ks, AO.pack_keys), (cache.vc, cache.vs, AO.pack_values)):
        assert np.array_equal(f64(scales)[0, 0, :, :, 0][normal], step[normal])
        ok = normal.all(1)
        assert np.array_equal(plane[0, 0].cpu().numpy()[ok], pack(codes)[ok])


def test_two_graphs_with_their_own_workspaces_interleave():
    n, hq, hk, d, cap = 2, 8, 2, 64, 256
    lens = [200, 131]
    cache = filled_cache(lens, cap, hk, d, seed=4)
    qs = [randn(n, hq, d, seed=s, mul=2.0) for s in (1, 2)]
    L = i32(lens)
    runs, want = [], []
    for q in qs:
        o, l, ws = rmm.kv4_attn(q, cache, L)
        want.append((o.clone(), l.clone()))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            rmm.kv4_attn(q, cache, L, out=o, lse=l, workspace=ws)
        runs.append((g, o, l, ws))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (g, *_r) in zip((s1, s2), runs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (g, o, l, ws), (wo, wl) in zip(runs, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)
        rmm.check(ws)
