"""The README's serving example runs as it stands and does what its calls do one by one."""
from __future__ import annotations

import os

import pytest
import torch

from input_adaptive_reduced_02_b200 import rmm
from test_gpu_attention import cum, i32, randn

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_serving_example():
    with open(README, encoding="utf-8") as f:
        code = f.read().split("## Serving", 1)[1].split("```python\n", 1)[1].split("```", 1)[0]
    lens, hq, heads, d, cap, budget, n = [300, 17, 263], 8, 2, 64, 320, 264, 12
    T, batch = sum(lens), len(lens)
    v = dict(Q=randn(T, hq, d, seed=1, mul=2.0), K=randn(T, heads, d, seed=2), V=randn(T, heads, d, seed=3),
             cu=i32(cum(lens)), start=i32([0] * batch), batch=batch, heads=heads, cap=cap, d=d, budget=budget,
             steps=[tuple(randn(batch, h, d, seed=10 * s + h) for h in (hq, heads, heads)) for s in range(n)])
    w = rmm.attn_key_weights(v["Q"], v["K"], rmm.attn_prompt(v["Q"], v["K"], v["V"], v["cu"], v["cu"])[1], v["cu"], v["cu"])
    cache = rmm.KV4Cache.empty(batch, heads, cap, d)
    rmm.kv4_store(cache, v["K"], v["V"], v["start"], v["cu"], w_new=w)
    L = i32(lens)
    for q, k, x in v["steps"]:
        rmm.kv4_store(cache, k, x, L)
        L = L + 1
        o = rmm.kv4_attn(q, cache, L, w_in=cache.w, w_out=cache.w)[0]
        rmm.cache_evict(cache.w, L, cache.planes(), budget, sink=4, recent=256, lens_out=L)
    exec(compile(code, README, "exec"), v)
    assert v["lens"].tolist() == [264, 29, 264] and torch.equal(v["lens"], L)
    assert torch.equal(v["o"], o) and torch.isfinite(o).all()
    assert all(torch.equal(a, b) for a, b in zip(v["cache"].planes(), cache.planes()))
