"""Sizes of the attention operators at which a count would not fit its integer:
refused on the host, as are buffers of another device (no GPU)."""
from __future__ import annotations

import pytest
import torch

from input_adaptive_reduced_02_b200 import rmm
from test_attention_abi_cpu import DECODE, EVICT, PROMPT, STORE, UNSUPPORTED, WEIGHTS, call

WIDE = dict(d=8, q_ts=65535 * 8, q_hs=8, k_ts=65535 * 8, k_hs=8, h_q=65535, h_kv=65535, n_seq=65535)


@pytest.mark.parametrize("name,base,changes", [
    # blocks of every sequence and head: 2^32 - 131071, and just above 2^32, where the count would wrap round
    ("rmm_attn_prompt", PROMPT, dict(WIDE, v_ts=65535 * 8, v_hs=8, o_ts=65535 * 8, o_hs=8)),
    ("rmm_attn_prompt", PROMPT, dict(WIDE, v_ts=65535 * 8, v_hs=8, o_ts=65535 * 8, o_hs=8, T_q=1024)),
    ("rmm_attn_key_weights", WEIGHTS, WIDE), ("rmm_attn_key_weights", WEIGHTS, dict(WIDE, T_k=1024)),
    # products of two sizes that are 0 modulo 2^64
    ("rmm_kv4_store", STORE, dict(n_seq=1 << 32, h_kv=1 << 32)),
    ("rmm_kv4_attn", DECODE, dict(batch=1 << 62)),
    ("rmm_cache_evict", EVICT, dict(batch=1 << 32, heads=1 << 32)),
], ids=lambda x: x if isinstance(x, str) else "")
def test_counts_that_do_not_fit_are_refused(name, base, changes):
    got, text = call(name, base, changes)
    assert got == UNSUPPORTED, (got, text)


def test_workspace_sizes_of_refused_calls_are_zero():
    size = rmm.lib().rmm_kv4_attn_workspace_size
    assert size(65535, 8, 1, 64, 1 << 21, 1) > 0
    for bad in ((1 << 62, 8, 1, 64, 16), (1, 1 << 40, 1, 64, 16), (1, 8, 1 << 40, 64, 16), (1, 8, 1, 160, 16),
                (1, 8, 1, 64, (1 << 21) + 1)):
        assert size(*bad, 1) == 0
    size = rmm.lib().rmm_cache_evict_workspace_size
    assert size(65535, 8, 1 << 21) > 0
    for bad in ((1 << 32, 1 << 32, 16), (1, 1 << 62, 16), (1, 1, (1 << 21) + 1)):
        assert size(*bad) == 0


def test_status_words_and_workspaces_of_another_device_are_refused():
    """Their addresses would be written to by kernels of the call's device."""
    there, here = torch.device("cuda", 0), torch.device("cpu")
    assert rmm._status_ptr(None, there) is None
    word = rmm.status_word("cpu")
    assert rmm._status_ptr(word, here) == word.data_ptr()
    for bad, device in ((word, there), (torch.zeros(1, dtype=torch.int64), here), (torch.zeros(1), here),
                        (torch.zeros(0, dtype=torch.int32), here)):
        with pytest.raises(ValueError, match="status must be"):
            rmm._status_ptr(bad, device)
    ws = rmm.Workspace(64, "cpu")
    assert rmm._ensure_ws(ws, 64, here) is ws and rmm._ensure_ws(ws, 65, here) is not ws
    with pytest.raises(ValueError, match="workspace is on"):
        rmm._ensure_ws(ws, 64, there)


def test_host_tensors_never_reach_a_kernel():
    """The softmax calls' logits are not looked at before the stream is asked for: a tensor of no device has none."""
    L, V = torch.zeros(1, 8, 8), torch.zeros(1, 8, 16, dtype=torch.bfloat16)
    for call in (lambda: rmm.softmax_row_stats(L), lambda: rmm.softmax_score(L, torch.zeros(1, 8, 2)),
                 lambda: rmm.pv_softmax_reduced(L, V, 0.5)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
