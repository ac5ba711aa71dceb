"""The attention operators where a value, a size or a neighbour is unusual: rows
that a tile leaves idle, steps next to nothing. Tolerances as derived in test_gpu_attention.py unless a
test derives its own."""
from __future__ import annotations

import pytest
import torch

from input_adaptive_reduced_02_b200 import rmm
from test_gpu_attention import DEV, check_decode, check_prompt, cum, i32, make_prompt, randn

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
