"""The attention operators where a value, a size or a neighbour is unusual: rows
that a tile leaves idle, steps next to nothing, values of very different size in
one sequence, more (key, head) pairs than 31 bits hold, groups that overflow.
Tolerances as derived in test_gpu_attention.py unless a test derives its own."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from input_adaptive_reduced_02_b200 import rmm
from oracle import attention_oracle as AO
from test_gpu_attention import (DECODES, DEV, check_decode, check_prompt, cum, f64, filled_cache, i32, make_prompt, randn,
                                score_error, stored)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- idle rows of a prompt's tiles
def leave_in_shared_memory(value):
    """Every SM's last block of the prompt kernel leaves queries of this size in shared memory (128 live rows a tile)."""
    q = torch.full((2 * 148 * 64, 2, 128), value, dtype=torch.bfloat16, device=DEV)
    k = torch.ones(1, 1, 128, dtype=torch.bfloat16, device=DEV)
    rmm.attn_prompt(q, k, k, causal=False)


@pytest.mark.parametrize("hq,hk", [(3, 1), (14, 2), (24, 1)])
def test_prompt_bits_do_not_depend_on_what_ran_before(hq, hk):
    """Tiles with rows beyond the group's (128 is no multiple of 3, 7 or 24): queries of those rows are never loaded."""
    case = ([300], [900], hq, hk, 128, True)
    Q, K, V, cq, ck = make_prompt(case, 31)
    K[300:] *= 1.5  # the running maxima of the live rows grow by little from tile to tile
    want = None
    for left in (0.0, 40.0, -1.0, 3e4):
        leave_in_shared_memory(left)
        got = rmm.attn_prompt(Q, K, V, cq, ck)
        if want is None:
            want = got
            check_prompt(case, Q, K, V, *got, 128 ** -0.5)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), left


@pytest.mark.parametrize("hq,hk,d", [(3, 1, 64), (14, 2, 128), (8, 2, 128), (1, 1, 64)])
def test_a_sequence_has_the_same_bits_alone_and_packed(hq, hk, d):
    """The rows of a tile past the sequence's last query hold the next sequence's queries, here 60 times larger."""
    ql, kl = [50, 77], [1050, 600]
    Q, K, V, cq, ck = make_prompt((ql, kl, hq, hk, d, True), 32)
    K[350:1050] *= 1.5
    alone = rmm.attn_prompt(Q[:50].clone(), K[:1050].clone(), V[:1050].clone())
    Q[50:] *= 60
    O, lse = rmm.attn_prompt(Q, K, V, cq, ck)
    assert torch.equal(O[:50], alone[0]) and torch.equal(lse[:, :50], alone[1])
    Q[50:] = float("nan")  # unread by the first sequence in any form
    O, lse = rmm.attn_prompt(Q, K, V, cq, ck)
    assert torch.equal(O[:50], alone[0]) and torch.equal(lse[:, :50], alone[1])


# ---------------------------------------------------------------- steps of the decode's values
def growing_scores(n, L, hq, hk, d, log2_per_256):
    """Queries and keys whose scores grow along the sequence by so many powers of two per 256 tokens, a little uneven."""
    K, Q = randn(n * L, hk, d, seed=41, mul=0.05).float(), randn(n, hq, d, seed=42, mul=0.2).float()
    K[:, :, 0] = (torch.arange(L, device=DEV).float() * (log2_per_256 / 256)).repeat(n)[:, None]
    Q[:, :, 0] = d ** 0.5 * 0.6931471805599453
    return Q.bfloat16(), K


@pytest.mark.parametrize("hq,hk", [(32, 8), (8, 8), (64, 8), (96, 8)])
@pytest.mark.parametrize("size", [1e-35, 3e-37])
def test_decode_of_steps_next_to_nothing(size, hq, hk):
    """Steps of 2^-118 and 2^-123 beside a group of ordinary constants, more than one tile per warp, each raising the
    maximum by less than what is let through unscaled."""
    n, L, d = 16, 1024, 64
    Q, K = growing_scores(n, L, hq, hk, d, 6.0)
    V = randn(n * L, hk, d, seed=43).float() * size
    V[:, :, :32] = 3.0
    cache = rmm.KV4Cache.empty(n, hk, L, d)
    rmm.kv4_store(cache, K, V, i32([0] * n), i32(cum([L] * n)))
    assert 0 < cache.vs[..., 1, 0].float().max().item() < 2.0 ** -114
    w_out = torch.empty(n, hk, L, device=DEV)
    O, lse, ws = rmm.kv4_attn(Q, cache, i32([L] * n), w_out=w_out)
    rmm.check(ws)
    pick = [0, 7, 15]
    sub = rmm.KV4Cache(*(t[pick].contiguous() for t in (cache.kc, cache.ks, cache.vc, cache.vs)))
    check_decode(Q[pick], sub, [L] * 3, O[pick], lse[pick], d ** -0.5, w_out[pick])


def check_decode_f16(Q, cache, lens, O, lse, scale):
    """Outputs of dtype f32, by the header's arithmetic. p·step is rounded to f16: off by at most 2^-11 of itself, or,
    next to nothing, by half of the least f16 subnormal, 2^-25 under a power of two that keeps 4 times the head's
    largest p·step at 2^14 at least, so 2^-37 of that largest product; times codes up to 15. p·minimum and all
    sums stay in f32 (2^-18). Scores move numerator and denominator by 2.2·E."""
    n, hq, d = Q.shape
    gq = hq // cache.heads
    assert O.dtype == torch.float32
    for b in range(n):
        for h in range(cache.heads):
            k, v, (kc, ks, vc, vs) = stored(cache, b, h, lens[b])
            steps = AO.dequantise(vc, vs[..., 0], 0 * vs[..., 1])
            vmag = AO.dequantise(vc, vs[..., 0], np.abs(vs[..., 1]))
            kmag = np.maximum(np.abs(k), AO.dequantise(kc, ks[..., 0], np.abs(ks[..., 1])))
            q = f64(Q[b, h * gq:(h + 1) * gq])
            Or, lr, P, _ = AO.attention(q, k, v, scale, False)
            E = score_error(np.max(scale * np.abs(q) @ kmag.T, axis=1), d)
            largest = (P * vs[..., 0].max(1)).max(1)
            tol = 2.0 ** -11 * (P @ steps) + (2.2 * E[:, None] + 2.0 ** -18) * (P @ vmag)
            tol += (len(k) * 15 * 2.0 ** -37 * largest)[:, None]
            err = np.abs(f64(O[b, h * gq:(h + 1) * gq]) - Or)
            assert np.all(err <= tol), f"worst {np.max(err / tol):.2f}"
            gl = f64(lse[b, h * gq:(h + 1) * gq])
            assert np.all(np.abs(gl - lr) <= E + 2.0 ** -21 * (1 + np.abs(lr)))


@pytest.mark.parametrize("case", [c for c in DECODES if 0 not in c[0]],
                         ids=lambda c: f"l{'-'.join(map(str, c[0]))}_h{c[2]}-{c[3]}_d{c[4]}")
def test_decode_keeps_f16_of_the_probabilities_times_steps(case):
    lens, cap, hq, hk, d = case
    cache = filled_cache(lens, cap, hk, d, seed=7 * d + cap)
    Q = randn(len(lens), hq, d, seed=19, mul=2.0)
    O, lse, ws = rmm.kv4_attn(Q, cache, i32(lens))
    rmm.check(ws)
    check_decode_f16(Q, cache, lens, O, lse, d ** -0.5)


@pytest.mark.parametrize("at", [0, 5, 700], ids=lambda x: f"token{x}")
@pytest.mark.parametrize("ratio,below", [(24, 40), (31, 40), (60, 70), (100, 60)])
@pytest.mark.parametrize("hq,hk", [(8, 2), (16, 2), (24, 2)])
def test_decode_of_an_outlier_that_hardly_counts(hq, hk, ratio, below, at):
    """One token's values are 2^ratio times the others', its probability about 2^-below of theirs: where the others' p·step
    are the larger ones they keep their bits, and where its own is, it does."""
    L, d = 1000, 64
    K, V = randn(L, hk, d, seed=51, mul=0.05).float(), randn(L, hk, d, seed=52).float()
    Q = randn(1, hq, d, seed=53, mul=0.2).float()
    Q[:, :, 0] = d ** 0.5 * 0.6931471805599453
    K[:, :, 0] = 0.0
    K[at, :, 0] = -below
    V[at] *= 2.0 ** ratio
    Q = Q.bfloat16()
    cache = rmm.KV4Cache.empty(1, hk, L, d)
    rmm.kv4_store(cache, K, V, i32([0]), i32([0, L]))
    O, lse, ws = rmm.kv4_attn(Q, cache, i32([L]))
    rmm.check(ws)
    check_decode_f16(Q, cache, [L], O, lse, d ** -0.5)


# ---------------------------------------------------------------- long contexts
def test_key_weights_of_keys_2_to_31_pairs_before_the_queries():
    """Three new tokens of 128 query heads on one key head after 2^24 + 197 earlier ones: the first keys lie more than 2^31
    (query, head) pairs before the first query."""
    S_q, S_k, hq, d = 3, (1 << 24) + 200, 128, 8
    Q, K, V = randn(S_q, hq, d, seed=61), randn(S_k, 1, d, seed=62), randn(S_k, 1, d, seed=63)
    st = rmm.status_word()
    _, lse = rmm.attn_prompt(Q, K, V, status=st)
    w = rmm.attn_key_weights(Q, K, lse, status=st)
    rmm.check(st)
    scale = d ** -0.5
    q = Q.double().reshape(S_q * hq, d)
    for k0, k1 in ((0, 1000), (S_k // 2, S_k // 2 + 1000), (S_k - 1000, S_k)):
        x = scale * (q @ K[k0:k1, 0].double().T).reshape(S_q, hq, k1 - k0)
        seen = torch.arange(k0, k1, device=DEV) <= torch.arange(S_q, device=DEV)[:, None] + S_k - S_q
        ref = (torch.exp(x - lse.T.double()[:, :, None]) * seen[:, None]).sum((0, 1))
        E = score_error((scale * q.abs() @ K[k0:k1, 0].double().abs().T).max().item(), d)
        assert ((w[0, k0:k1] - ref).abs() <= (2.1 * E + 2.0 ** -18) * ref).all()
    # every row's probabilities add up to 1: a row's lse is off by E + 2^-21·(1 + |lse|) at most, |lse| < 32
    assert abs(w.double().sum().item() - S_q * hq) <= S_q * hq * 2.0 ** -14


# ---------------------------------------------------------------- store
@pytest.mark.parametrize("plane", [0, 1], ids=["keys", "values"])
@pytest.mark.parametrize("lo,hi,fits", [(-3e38, 3e38, False), (-2e38, 1e38, True), (-3.4e38, -3.39e38, False),
                                        (3.3895e38, 3.3895e38, True), (3.4e38, 3.4e38, False)])
def test_store_reports_steps_and_minima_that_overflow(lo, hi, fits, plane):
    """Finite values whose group's max - min overflows f32, or whose minimum overflows bf16 (largest 3.3895e38)."""
    kv = [randn(3, 2, 64, seed=s).float() for s in (71, 72)]
    kv[plane][1, 1, 32:] = torch.linspace(lo, hi, 32, dtype=torch.float64).float().to(DEV)
    kv[plane][1, 1, 32], kv[plane][1, 1, 63] = lo, hi
    assert torch.isfinite(kv[plane]).all()
    cache = rmm.KV4Cache.empty(1, 2, 3, 64)
    st = rmm.status_word()
    rmm.kv4_store(cache, *kv, i32([0]), i32([0, 3]), status=st)
    if fits:
        rmm.check(st)
        assert torch.isfinite(cache.ks).all() and torch.isfinite(cache.vs).all()
        return
    with pytest.raises(rmm.RMMError) as e:
        rmm.check(st)
    assert e.value.status == rmm.RMM_ERR_NONFINITE


# ---------------------------------------------------------------- refusals of the binding
def test_status_words_that_kernels_cannot_write_are_refused():
    q, k = randn(4, 2, 64), randn(4, 1, 64)
    lse = torch.zeros(2, 4, device=DEV)
    cache = rmm.KV4Cache.empty(1, 1, 8, 64)
    for bad in (rmm.status_word("cpu"), torch.zeros(1, dtype=torch.int64, device=DEV), torch.zeros(1, device=DEV)):
        for call in (lambda: rmm.attn_prompt(q, k, k, status=bad), lambda: rmm.attn_key_weights(q, k, lse, status=bad),
                     lambda: rmm.kv4_store(cache, k, k, i32([0]), i32([0, 4]), status=bad)):
            with pytest.raises(ValueError, match="status must be"):
                call()
    with pytest.raises(ValueError, match="workspace is on"):
        rmm.kv4_attn(q[:1], cache, i32([0]), workspace=rmm.Workspace(1 << 20, "cpu"))


def test_a_full_cache_reports_the_token_it_has_no_room_for():
    """Through the cache's own status word, without one from the caller."""
    cache = rmm.KV4Cache.empty(2, 1, 4, 64)
    lens, step = i32([3, 1]), randn(2, 1, 64)
    rmm.kv4_store(cache, step, step, lens)
    rmm.check(cache.status)
    rmm.kv4_store(cache, step, step, lens + 1)  # slot 4 of sequence 0
    assert (cache.ks[1, :, 2] != 0).any()
    with pytest.raises(rmm.RMMError) as e:
        rmm.check(cache.status)
    assert e.value.status == rmm.RMM_ERR_INVALID
    rmm.check(cache.status)  # reported once
    mine = rmm.status_word()
    rmm.kv4_store(cache, step, step, lens + 1, status=mine)
    rmm.check(cache.status)
    with pytest.raises(rmm.RMMError):
        rmm.check(mine)
    planes = (cache.kc, cache.ks, cache.vc, cache.vs, cache.w)
    assert rmm.KV4Cache(*planes).status is None and rmm.KV4Cache(*planes, status=mine).status is mine
    with pytest.raises(ValueError, match="status must be"):
        rmm.KV4Cache(*planes, status=rmm.status_word("cpu"))


def test_scales_and_flags_of_numpy_types():
    q, k = randn(4, 2, 64), randn(4, 1, 64)
    cache = rmm.KV4Cache.empty(4, 1, 8, 64)
    rmm.kv4_store(cache, k, k, i32([0] * 4))
    lse = rmm.attn_prompt(q, k, k, scale=0.25, causal=True)[1]
    for call in (lambda s, c: rmm.attn_prompt(q, k, k, scale=s, causal=c)[0],
                 lambda s, c: rmm.attn_key_weights(q, k, lse, scale=s, causal=c),
                 lambda s, c: rmm.kv4_attn(q, cache, i32([1] * 4), scale=s)[0]):
        assert torch.equal(call(np.float32(0.25), np.bool_(True)), call(0.25, True))


# ---------------------------------------------------------------- graphs
def test_the_reduced_products_in_a_captured_graph():
    """The fused calls of every route, captured once and replayed on other inputs."""
    A, B = randn(96, 512, seed=1), randn(512, 256, seed=2)
    x, n = randn(1, 512, seed=3), rmm.b_norms(B)
    L, V = randn(2, 64, 128, seed=4), randn(2, 128, 64, seed=5)

    def calls(outs, ws):
        c0, w0 = rmm.matmul_reduced(A, B, 0.5, out=outs[0], workspace=ws[0])
        c1, w1 = rmm.matmul_reduced_b_norms(x, B, n, 0.5, out=outs[1], workspace=ws[1])
        c2, _, w2 = rmm.pv_softmax_reduced(L, V, 0.5, out=outs[2], P=outs[3], workspace=ws[2])
        return [c0, c1, c2, _], [w0, w1, w2]

    outs, ws = calls([None] * 4, [None] * 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        calls(outs, ws)
    for seed in (11, 12):
        A.copy_(randn(96, 512, seed=seed))
        x.copy_(randn(1, 512, seed=seed + 20))
        L.copy_(randn(2, 64, 128, seed=seed + 40))
        g.replay()
        got = [t.clone() for t in outs]
        for w in ws:
            rmm.check(w)
        want, _ = calls([None] * 4, [None] * 3)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
