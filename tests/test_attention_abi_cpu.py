"""Host-side argument checks of the attention operators (no GPU): every refusal
comes back with its status and a message before any device work, and the
workspace helpers behave as documented."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from input_adaptive_reduced_02_b200 import rmm
from oracle import attention_oracle as AO

P = 1 << 20  # a pointer that is never followed: aligned to everything the checks ask for
BF16, F32 = rmm.RMM_BF16, rmm.RMM_F32
OK, INVALID, UNSUPPORTED = rmm.RMM_OK, rmm.RMM_ERR_INVALID, rmm.RMM_ERR_UNSUPPORTED
NAN = float("nan")


def call(name, base, changes):
    args = dict(base)
    assert set(changes) <= set(args), changes
    args.update(changes)
    status = getattr(rmm.lib(), name)(*args.values())
    return status, rmm.lib().rmm_last_error_string().decode()


PROMPT = dict(Q=P, q_ts=1024, q_hs=64, K=P, k_ts=256, k_hs=64, V=P, v_ts=256, v_hs=64, cu_q=P, cu_k=P, n_seq=2, T_q=10,
              T_k=12, h_q=16, h_kv=4, d=64, scale=0.125, causal=1, dtype=BF16, O=P, o_ts=1024, o_hs=64, out=BF16, lse=P,
              status=P, stream=None)


@pytest.mark.parametrize("changes,status,word", [
    (dict(Q=None), INVALID, "Q is NULL"), (dict(K=None), INVALID, "K is NULL"), (dict(V=None), INVALID, "V is NULL"),
    (dict(O=None), INVALID, "O is NULL"), (dict(Q=P + 8), INVALID, "aligned"), (dict(k_ts=260), INVALID, "multiples"),
    (dict(v_hs=68), INVALID, "multiples"), (dict(q_ts=32), INVALID, "too small"), (dict(k_hs=32), INVALID, "too small"),
    (dict(q_ts=-1024), INVALID, "too small"), (dict(o_ts=256, o_hs=64), INVALID, "overlap"),
    (dict(n_seq=-1), INVALID, "negative"), (dict(T_q=-1), INVALID, "negative"),
    (dict(n_seq=70000), UNSUPPORTED, "65535"), (dict(T_k=1 << 31), UNSUPPORTED, "tokens"),
    (dict(cu_q=None), INVALID, "single sequence"), (dict(cu_k=None), INVALID, "single sequence"),
    (dict(h_q=6), INVALID, "multiple of h_kv"), (dict(h_kv=0), INVALID, "multiple of h_kv"),
    (dict(h_q=516, q_ts=516 * 64, o_ts=516 * 64), UNSUPPORTED, "query heads"),
    (dict(d=0), INVALID, "d must"), (dict(d=60), UNSUPPORTED, "multiple of 8"), (dict(d=136), UNSUPPORTED, "at most 128"),
    (dict(scale=0.0), INVALID, "scale"), (dict(scale=-1.0), INVALID, "scale"), (dict(scale=NAN), INVALID, "scale"),
    (dict(scale=float("inf")), INVALID, "scale"), (dict(dtype=F32), UNSUPPORTED, "bf16"), (dict(dtype=7), INVALID, "dtype"),
    (dict(out=7), INVALID, "output dtype"),
])
def test_prompt_refusals(changes, status, word):
    got, text = call("rmm_attn_prompt", PROMPT, changes)
    assert got == status and word in text, (got, text)


def test_prompt_of_nothing_is_no_work():
    assert call("rmm_attn_prompt", PROMPT, dict(n_seq=0))[0] == OK
    assert call("rmm_attn_prompt", PROMPT, dict(T_q=0, Q=None, O=None))[0] == OK


WEIGHTS = dict(Q=P, q_ts=1024, q_hs=64, K=P, k_ts=256, k_hs=64, cu_q=P, cu_k=P, n_seq=2, T_q=10, T_k=12, h_q=16, h_kv=4,
               d=64, scale=0.125, causal=1, dtype=BF16, lse=P, w_in=None, w_out=P, status=None, stream=None)


@pytest.mark.parametrize("changes,status,word", [
    (dict(lse=None), INVALID, "lse"), (dict(w_out=None), INVALID, "w_out"), (dict(w_in=P + 64), INVALID, "overlap"),
    (dict(w_in=P - 64), INVALID, "overlap"), (dict(Q=P + 2), INVALID, "aligned"), (dict(dtype=F32), UNSUPPORTED, "bf16"),
    (dict(d=132), UNSUPPORTED, "multiple of 8"), (dict(scale=NAN), INVALID, "scale"),
])
def test_key_weight_refusals(changes, status, word):
    got, text = call("rmm_attn_key_weights", WEIGHTS, changes)
    assert got == status and word in text, (got, text)


STORE = dict(K=P, k_ts=256, k_hs=64, V=P, v_ts=256, v_hs=64, dtype=BF16, cu=P, start=P, n_seq=2, T=10, h_kv=4, d=64,
             cap=100, kc=P, ks=P, vc=P, vs=P, w_new=None, w=None, status=None, stream=None)


@pytest.mark.parametrize("changes,status,word", [
    (dict(K=None), INVALID, "NULL"), (dict(start=None), INVALID, "NULL"), (dict(kc=None), INVALID, "plane"),
    (dict(vs=None), INVALID, "plane"), (dict(ks=P + 4), INVALID, "aligned"), (dict(d=48), UNSUPPORTED, "32, 64, 96"),
    (dict(d=160), UNSUPPORTED, "32, 64, 96"), (dict(cap=0), INVALID, "cap"), (dict(cap=(1 << 21) + 1), UNSUPPORTED, "cap"),
    (dict(cu=None), INVALID, "one token per sequence"), (dict(w_new=P), INVALID, "w_new"),
    (dict(k_ts=63), INVALID, "too small"), (dict(n_seq=20000), UNSUPPORTED, "65535"), (dict(T=-1), INVALID, "negative"),
    (dict(h_kv=0), INVALID, "h_kv"), (dict(dtype=5), INVALID, "dtype"),
])
def test_store_refusals(changes, status, word):
    got, text = call("rmm_kv4_store", STORE, changes)
    assert got == status and word in text, (got, text)


DECODE = dict(Q=P, q_ss=1024, q_hs=64, kc=P, ks=P, vc=P, vs=P, lens=P, batch=2, h_q=16, h_kv=4, d=64, cap=100,
              scale=0.125, dtype=BF16, O=P, o_ss=1024, o_hs=64, out=F32, lse=None, w_in=None, w_out=None, ws=P,
              ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("changes,status,word", [
    (dict(Q=None), INVALID, "Q is NULL"), (dict(lens=None), INVALID, "lens"), (dict(vc=None), INVALID, "plane"),
    (dict(ws=None), INVALID, "workspace"), (dict(ws=P + 512), INVALID, "1 KiB"), (dict(ws_bytes=1024), INVALID, "too small"),
    (dict(w_in=P), INVALID, "w_in needs"), (dict(w_in=P + 4, w_out=P), INVALID, "overlap"),
    (dict(d=80), UNSUPPORTED, "32, 64, 96"), (dict(scale=0.0), INVALID, "scale"), (dict(dtype=F32), UNSUPPORTED, "bf16"),
    (dict(h_q=18), INVALID, "multiple of h_kv"), (dict(q_hs=60), INVALID, "too small"), (dict(out=9), INVALID, "dtype"),
    (dict(o_ss=64, o_hs=64), INVALID, "overlap"), (dict(batch=-1), INVALID, "negative"),
])
def test_decode_refusals(changes, status, word):
    got, text = call("rmm_kv4_attn", DECODE, changes)
    assert got == status and word in text, (got, text)


class Plane(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("row_bytes", ctypes.c_int64)]


EVICT = dict(w=P, lens=P, batch=2, heads=3, cap=100, budget=40, sink=4, recent=8, planes=None, n_planes=0, cap_out=40,
             lens_out=P, idx_out=None, ws=P, ws_bytes=1 << 30, stream=None)
FAR = P + (1 << 24)


@pytest.mark.parametrize("planes,changes,status,word", [
    ([], dict(w=None), INVALID, "NULL"), ([], dict(lens_out=None), INVALID, "NULL"), ([], dict(budget=0), INVALID, "budget"),
    ([], dict(budget=41), INVALID, "budget"), ([], dict(sink=33), INVALID, "exceed budget"),
    ([], dict(recent=-1), INVALID, "negative"), ([], dict(cap=(1 << 21) + 1), UNSUPPORTED, "cap"),
    ([], dict(heads=0), INVALID, "heads"), ([], dict(ws=None), INVALID, "workspace"),
    ([], dict(ws_bytes=1024), INVALID, "too small"), ([], dict(n_planes=1), INVALID, "planes"),
    ([(P, FAR, 16)] * 9, {}, UNSUPPORTED, "planes"), ([(P, FAR, 6)], {}, INVALID, "row_bytes"),
    ([(P, FAR, 8196)], {}, UNSUPPORTED, "row_bytes"), ([(P + 2, FAR, 16)], {}, INVALID, "4-byte"),
    ([(None, FAR, 16)], {}, INVALID, "NULL"), ([(P, P, 16)], {}, INVALID, "capacity"),
    ([(P, P + 1024, 16)], {}, INVALID, "overlap"), ([(P, FAR, 16), (P + (1 << 23), FAR + 64, 16)], {}, INVALID, "overlap"),
])
def test_eviction_refusals(planes, changes, status, word):
    arr = (Plane * max(1, len(planes)))(*[Plane(*p) for p in planes])
    base = dict(EVICT, planes=ctypes.cast(arr, ctypes.c_void_p) if planes else None, n_planes=len(planes))
    got, text = call("rmm_cache_evict", base, changes)
    assert got == status and word in text, (got, text)


def test_workspace_sizes():
    L = rmm.lib()
    assert rmm.kv4_attn_workspace_size(0, 8, 2, 64, 16) >= 1024  # the status word is there for an empty batch too
    for bad in ((-1, 8, 2, 64, 16), (1, 0, 2, 64, 16), (1, 8, 0, 64, 16), (1, 8, 2, 0, 16), (1, 8, 2, 64, 0)):
        assert L.rmm_kv4_attn_workspace_size(*bad, 0) == 0
    small, large = (rmm.kv4_attn_workspace_size(b, 32, 8, 128, 8192) for b in (1, 32))
    assert 0 < small < large
    # with weights: the scores of every query head and slot besides
    assert rmm.kv4_attn_workspace_size(3, 32, 8, 128, 1000, True) >= rmm.kv4_attn_workspace_size(3, 32, 8, 128, 1000) + \
        3 * 32 * 1000 * 4
    assert rmm.cache_evict_workspace_size(2, 3, 40) >= 1024 + 4 * 6 + 4 * 6 * 40
    assert L.rmm_cache_evict_workspace_size(1, 1, 0) == 0 and L.rmm_cache_evict_workspace_size(-1, 1, 1) == 0


def test_binding_refuses_what_it_can_see():
    """CPU tensors, wrong ranks and shapes: refused in Python, before the library is called."""
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        rmm.attn_prompt(q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        rmm.attn_key_weights(q, q, torch.zeros(2, 4))
    with pytest.raises(ValueError, match="CUDA"):
        rmm.KV4Cache(torch.zeros(1, 2, 8, 32, dtype=torch.uint8), q, q, q)
    with pytest.raises(ValueError, match="multiple of 32"):
        rmm.KV4Cache.empty(1, 1, 8, 48)
    with pytest.raises(ValueError, match="CUDA"):
        rmm.cache_evict(torch.zeros(1, 1, 8), torch.zeros(1, dtype=torch.int32), [], 4)


# ---------------------------------------------------------------- the oracle's own arithmetic
def test_oracle_layouts_round_trip_and_quantisation_bounds():
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 16, (5, 128))
    for pack, bits in ((AO.pack_keys, "<u4"), (AO.pack_values, "<u2")):
        b = pack(codes)
        assert b.shape == (5, 64)
        nibbles = np.stack([b & 15, b >> 4], -1).reshape(5, 128)
        assert np.array_equal(np.sort(nibbles, 1), np.sort(codes, 1))  # every code is there once
    x = rng.standard_normal((7, 96)).astype(np.float32) * 3
    c, s, m = AO.quantise(x)
    err = np.abs(AO.dequantise(c, s, m) - x)
    # half a step, plus what the rounded step and minimum (bf16, half a step of 2^-8 each) move the ends by
    bound = (0.5 * s + 15 * s * 2.0 ** -8 + np.abs(m) * 2.0 ** -8 + 1e-6)[..., None].repeat(32, -1).reshape(x.shape)
    assert np.all(err <= bound)
    flat = np.full((1, 32), 2.5, np.float32)
    c, s, m = AO.quantise(flat)
    assert (c == 0).all() and (s == 0).all() and (m == 2.5).all()


def test_oracle_attention_rows_without_keys_and_kept_tokens():
    q, k, v = np.ones((4, 8)), np.ones((2, 8)), np.arange(16.0).reshape(2, 8)
    o, lse, p, _ = AO.attention(q, k, v, 0.5, True)  # rows 0 and 1 see no key
    assert (o[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(p[2:].sum(1), 1)
    assert np.allclose(o[2], v[0]) and np.allclose(o[3], v.mean(0))
    assert AO.kept_tokens([5, 1, 3, 3, 2, 9], 4, 1, 1).tolist() == [0, 2, 3, 5]
    assert AO.kept_tokens([1, 2], 4, 1, 1).tolist() == [0, 1]
