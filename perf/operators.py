"""Attention operators of the library as calls to be timed and compared: what a
serving program does with a prompt and then, token by token, with its cache.

  prompt   attention of packed prompts (causal or not, grouped heads) with the
           rows' log-sum-exp
  weights  the attention weight each key received, summed over the queries and
           over the query heads that share the key's head
  kv4      one decode step on a cache held in 4 bits: the step's new tokens are
           quantised into their slots, then one query token per sequence
           attends to its sequence's cached tokens (optionally adding its
           attention weights to the running sums)
  evict    a cache that has outgrown its budget keeps its first tokens, its
           last tokens and the ones of greatest accumulated weight

`own` chooses what `run` computes: the library's calls (True) or the same
operators written in elementary torch operations (False).
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
GROUP = 32  # channels that share one scale and one minimum in the 4-bit cache


# ---------------------------------------------------------------- cases
# heads: query heads, key/value heads and head dimension. "q" and "prefix" are
# per sequence: new tokens, and earlier tokens whose keys precede them.
_LISTED = [
    # a single short question: the call's latency is what the user waits for
    dict(name="prompt_short", op="prompt", q="203", prefix="0", h_q=32, h_kv=8, d=128, causal=True),
    # a batch of requests of very different lengths packed together
    dict(name="prompt_packed", op="prompt", q="1,17,300,1025,64,2048,777,3866", prefix="0,0,0,0,0,0,0,0", h_q=32,
         h_kv=8, d=128, causal=True),
    # the second chunk of a long document, one key head per query head, small heads
    dict(name="prompt_chunk", op="prompt", q="2048,1999", prefix="2048,4100", h_q=16, h_kv=16, d=64, causal=True),
    # a long document in one call
    dict(name="prompt_long", op="prompt", q="16384", prefix="0", h_q=32, h_kv=8, d=128, causal=True),
    # the weights of the packed batch, before its keys go into a bounded cache
    dict(name="weights_packed", op="weights", q="1,17,300,1025,64,2048,777,3866", prefix="0,0,0,0,0,0,0,0", h_q=32,
         h_kv=8, d=128, causal=True),
    # the weights of a long document
    dict(name="weights_long", op="weights", q="8192", prefix="0", h_q=32, h_kv=8, d=128, causal=True),
    # one conversation's next token: latency
    dict(name="kv4_single", op="kv4", lens="1000", new=1, cap=2048, h_q=32, h_kv=8, d=128, weights=False),
    # a decode batch of uneven lengths that keeps its keys' weights for eviction
    dict(name="kv4_batch", op="kv4", lens="ragged:32:8192:5", new=1, cap=8192, h_q=32, h_kv=8, d=128, weights=True),
    # few conversations over long contexts, eight query heads to a key head
    dict(name="kv4_long", op="kv4", lens="32768,32767,31001,29999,32768,20000,32100,32500", new=1, cap=32768, h_q=64,
         h_kv=8, d=128, weights=False),
    # a prompt's keys and values enter the cache, and the first token is decoded
    dict(name="kv4_fill", op="kv4", lens="4096,2500", new=0, cap=4500, h_q=16, h_kv=16, d=64, weights=True),
    # one conversation's bf16 cache goes over its budget by a block of tokens
    dict(name="evict_single", op="evict", lens="1088", cap=1280, budget=1024, sink=4, recent=256, h_kv=8, d=128,
         four_bit=False),
    # a batch's 4-bit caches are halved
    dict(name="evict_batch", op="evict", lens="ragged:32:8192:9", cap=8192, budget=4096, sink=4, recent=1024, h_kv=8,
         d=128, four_bit=True),
]


def listed():
    return [dict(c) for c in _LISTED]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_once(rng):
    op = rng.choice(["prompt", "prompt", "weights", "kv4", "kv4", "evict"])
    h_q, h_kv = rng.choice([(32, 8), (32, 8), (16, 16), (64, 8), (12, 4), (6, 1), (14, 2), (40, 8), (16, 1), (24, 1)])
    if op in ("prompt", "weights"):
        n = rng.choice([1, 1, 2, 3, 5, 8])
        q = [_log(rng, 1, 16384 if n == 1 else 4096) for _ in range(n)]
        pre = [rng.choice([0, 0, 0, _log(rng, 1, 4096)]) for _ in range(n)]
        return dict(op=op, q=",".join(map(str, q)), prefix=",".join(map(str, pre)), h_q=h_q, h_kv=h_kv,
                    d=rng.choice([128, 128, 64, 96, 80]), causal=rng.random() < 0.85)
    if op == "kv4":
        n = _log(rng, 1, 32)
        cap = _log(rng, 64, 32768)
        lens = [min(cap, _log(rng, 1, cap)) for _ in range(n)]
        return dict(op=op, lens=",".join(map(str, lens)), new=rng.choice([1, 1, 1, 0]), cap=cap, h_q=h_q, h_kv=h_kv,
                    d=rng.choice([128, 128, 64, 96]), weights=rng.random() < 0.5)
    n = _log(rng, 1, 32)
    cap = _log(rng, 64, 32768)
    lens = [min(cap, _log(rng, max(1, cap // 4), cap)) for _ in range(n)]
    budget = max(1, min(cap, _log(rng, max(1, cap // 8), cap)))
    sink = min(budget, rng.choice([0, 1, 4]))
    recent = rng.randint(0, budget - sink)
    return dict(op=op, lens=",".join(map(str, lens)), cap=cap, budget=budget, sink=sink, recent=recent, h_kv=h_kv,
                d=rng.choice([128, 128, 64, 96]), four_bit=rng.random() < 0.6)


def draw(rng):
    top = {}
    for c in _LISTED:
        w = work(c)
        t = top.setdefault(c["op"], [0.0, 0.0])
        t[0], t[1] = max(t[0], w["bytes"]), max(t[1], w["flops"])
    while True:
        c = _draw_once(rng)
        w = work(c)
        if w["bytes"] <= top[c["op"]][0] and w["flops"] <= top[c["op"]][1]:
            return c


def _ints(text):
    if text.startswith("ragged:"):  # "ragged:count:longest:step": uneven lengths from longest/8 up to longest
        _, n, top, step = text.split(":")
        n, top, step = int(n), int(top), int(step)
        return [top - (i * step * 7919) % (top - top // 8) for i in range(n)]
    return [int(x) for x in text.split(",")]


def _cum(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return out


def _pairs(q, pre, causal):
    """(query, key) pairs that see each other."""
    return sum(n * p + (n * (n + 1) // 2 if causal else n * n) for n, p in zip(q, pre))


def work(case):
    """Each input read once, each output written once; products of visible pairs only."""
    if case["op"] in ("prompt", "weights"):
        q, pre = _ints(case["q"]), _ints(case["prefix"])
        tq, tk = sum(q), sum(q) + sum(pre)
        pairs = _pairs(q, pre, case["causal"])
        d, hq, hk = case["d"], case["h_q"], case["h_kv"]
        if case["op"] == "prompt":
            return {"bytes": 2 * d * (hq * tq + 2 * hk * tk) + 2 * d * hq * tq + 4 * hq * tq,
                    "flops": 4 * d * hq * pairs}
        return {"bytes": 2 * d * (hq * tq + hk * tk) + 4 * hq * tq + 8 * hk * tk, "flops": 2 * d * hq * pairs}
    lens = _ints(case["lens"])
    d, hk = case["d"], case["h_kv"]
    row = d // 2 + 4 * (d // GROUP)  # one token of one head in one 4-bit plane pair (codes, scales)
    if case["op"] == "kv4":
        hq, n = case["h_q"], sum(lens)
        new = len(lens) if case["new"] else n
        old = n - new
        return {"bytes": 2 * row * hk * old + new * hk * 2 * (2 * d + row) + len(lens) * hq * d * 4 +
                (8 * hk * n if case["weights"] else 0),
                "flops": 4 * d * hq * n}
    keep = sum(min(x, case["budget"]) for x in lens)
    rows = 2 * (row if case["four_bit"] else 2 * d) + 4
    return {"bytes": hk * (4 * sum(lens) + 2 * rows * keep), "flops": hk * sum(lens)}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _qkv(g, tq, tk, hq, hk, d):
    """Queries, keys and values with what trained attention shows: a few key
    channels of each head far from zero, and heads of different sharpness."""
    bias = torch.zeros(hk, d, device=DEV)
    ch = torch.randint(0, d, (hk, 4), generator=g, device=DEV)
    bias.scatter_(1, ch, 3.0 * _randn(g, hk, 4))
    K = (_randn(g, tk, hk, d) + bias).to(torch.bfloat16)
    V = _randn(g, tk, hk, d).to(torch.bfloat16)
    sharp = 0.5 + 2.0 * torch.rand(hq, 1, generator=g, device=DEV)
    Q = (_randn(g, tq, hq, d) * sharp).to(torch.bfloat16)
    return Q, K, V


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    if case["op"] in ("prompt", "weights"):
        q, pre = _ints(case["q"]), _ints(case["prefix"])
        k = [a + b for a, b in zip(q, pre)]
        st["cu_q_host"], st["cu_k_host"] = _cum(q), _cum(k)
        st["cu_q"], st["cu_k"] = _i32(st["cu_q_host"]), _i32(st["cu_k_host"])
        st["Q"], st["K"], st["V"] = _qkv(g, sum(q), sum(k), case["h_q"], case["h_kv"], case["d"])
        st["scale"] = case["d"] ** -0.5
        if case["op"] == "weights":
            st["lse"] = _plain_lse(st)
            st["w_in"] = torch.rand(case["h_kv"], sum(k), generator=g, device=DEV)
        return st
    lens = _ints(case["lens"])
    n, cap, hk, d = len(lens), case["cap"], case["h_kv"], case["d"]
    st["lens_host"], st["lens"] = lens, _i32(lens)
    if case["op"] == "kv4":
        planes = {"kc": [], "ks": [], "vc": [], "vs": []}
        for _ in range(n):  # one sequence at a time: the unquantised cache of the batch is never held
            _, K, V = _qkv(g, 1, cap, 1, hk, d)
            for x, c, s, lay in ((K, "kc", "ks", _k_bytes), (V, "vc", "vs", _v_bytes)):
                codes, scales = _quantise(x.transpose(0, 1).float())
                planes[c].append(lay(codes))
                planes[s].append(scales)
        for name, rows in planes.items():
            st[name] = torch.stack(rows)
        st["w_in"] = torch.rand(n, hk, cap, generator=g, device=DEV) if case["weights"] else None
        st["w"] = torch.zeros(n, hk, cap, device=DEV) if case["weights"] else None
        new = [1] * n if case["new"] else lens
        st["Q"], st["K"], st["V"] = _qkv(g, n, sum(new), case["h_q"], hk, d)
        st["cu_host"] = _cum(new)
        st["cu"] = _i32(st["cu_host"])
        st["start_host"] = [a - b for a, b in zip(lens, new)]
        st["start"] = _i32(st["start_host"])
        st["scale"] = d ** -0.5
        return st
    # accumulated weights: a few keys hold most, many hold next to nothing, some exactly nothing
    w = torch.exp(2.5 * _randn(g, n, hk, cap) - 4.0)
    w *= (torch.rand(n, hk, cap, generator=g, device=DEV) > 0.02)
    st["w"] = w
    if case["four_bit"]:
        ng = d // GROUP
        src = [torch.randint(0, 256, (n, hk, cap, d // 2), generator=g, device=DEV, dtype=torch.uint8),
               _randn(g, n, hk, cap, ng, 2).to(torch.bfloat16),
               torch.randint(0, 256, (n, hk, cap, d // 2), generator=g, device=DEV, dtype=torch.uint8),
               _randn(g, n, hk, cap, ng, 2).to(torch.bfloat16)]
    else:
        src = [_randn(g, n, hk, cap, d).to(torch.bfloat16), _randn(g, n, hk, cap, d).to(torch.bfloat16)]
    st["src"] = src + [w]
    st["dst"] = [torch.zeros(n, hk, case["budget"], *x.shape[3:], dtype=x.dtype, device=DEV) for x in st["src"]]
    return st


# ---------------------------------------------------------------- the 4-bit format
# A row of d channels is cut into groups of 32. A group holds a bf16 minimum m,
# a bf16 step s = bf16((max - min) / 15) and a code c = clamp(round((x - m) / s),
# 0, 15) per channel (0 where s is 0); it stands for m + s·c.
def _quantise(x):
    xg = x.unflatten(-1, (-1, GROUP))
    lo = xg.amin(-1).to(torch.bfloat16)
    step = ((xg.amax(-1) - xg.amin(-1)) / 15.0).to(torch.bfloat16)
    lo32, step32 = lo.float().unsqueeze(-1), step.float().unsqueeze(-1)
    codes = torch.where(step32 > 0, torch.round((xg - lo32) / step32).clamp(0, 15), torch.zeros_like(xg))
    return codes.to(torch.uint8).flatten(-2), torch.stack((step, lo), -1)


def _value(codes, scales):
    s = scales.float()
    return (codes.unflatten(-1, (-1, GROUP)).float() * s[..., 0:1] + s[..., 1:2]).flatten(-2)


def _k_bytes(codes):
    """Keys: channel 32w + 8j + i is nibble i of 32-bit word w of the row's j-th quarter."""
    *lead, d = codes.shape
    x = codes.reshape(*lead, d // 32, 4, 4, 2).transpose(-4, -3)  # [j][w][i / 2][i % 2]
    return (x[..., 0] | (x[..., 1] << 4)).reshape(*lead, d // 2)


def _k_codes(b):
    *lead, n = b.shape
    x = torch.stack((b & 15, b >> 4), -1).reshape(*lead, 4, n // 16, 8)  # [j][w][i]
    return x.transpose(-3, -2).reshape(*lead, 2 * n)


def _v_bytes(codes):
    """Values: channel 32w + 8i + r is nibble i of 16-bit half-word w of the row's r-th eighth."""
    *lead, d = codes.shape
    x = codes.reshape(*lead, d // 32, 4, 8).movedim(-1, -3)  # [r][w][i]
    x = x.reshape(*lead, 8, d // 32, 2, 2)
    return (x[..., 0] | (x[..., 1] << 4)).reshape(*lead, d // 2)


def _v_codes(b):
    *lead, n = b.shape
    x = torch.stack((b & 15, b >> 4), -1).reshape(*lead, 8, n // 16, 4)  # [r][w][i]
    return x.movedim(-3, -1).reshape(*lead, 2 * n)


# ---------------------------------------------------------------- plain forms
def _chunks(nq, nk, hq):
    """Query rows at a time, so that the scores of all heads stay below 4 GB."""
    rows = max(1, min(nq, (1 << 30) // max(1, nk * hq)))
    return [(a, min(nq, a + rows)) for a in range(0, nq, rows)]


def _scores(st, i, a, b):
    """scale·q·k of rows a..b of sequence i over its keys, [h_kv][g·rows][keys], invisible keys -inf."""
    c = st["case"]
    q0, q1 = st["cu_q_host"][i], st["cu_q_host"][i + 1]
    k0, k1 = st["cu_k_host"][i], st["cu_k_host"][i + 1]
    g = c["h_q"] // c["h_kv"]
    q = st["Q"][q0 + a:q0 + b].float().reshape(b - a, c["h_kv"], g, c["d"]).permute(1, 2, 0, 3)
    k = st["K"][k0:k1].float().permute(1, 2, 0)
    s = torch.matmul(q.reshape(c["h_kv"], g * (b - a), c["d"]), k) * st["scale"]
    if c["causal"]:
        row = torch.arange(a, b, device=DEV) + (k1 - k0) - (q1 - q0)
        hidden = torch.arange(k1 - k0, device=DEV)[None, :] > row[:, None]
        s.view(c["h_kv"], g, b - a, k1 - k0).masked_fill_(hidden, float("-inf"))
    return s


def _sequences(st):
    for i in range(len(st["cu_q_host"]) - 1):
        nq = st["cu_q_host"][i + 1] - st["cu_q_host"][i]
        nk = st["cu_k_host"][i + 1] - st["cu_k_host"][i]
        for a, b in _chunks(nq, nk, st["case"]["h_q"]):
            yield i, a, b


def _plain_lse(st):
    c = st["case"]
    lse = torch.empty(c["h_q"], st["Q"].shape[0], device=DEV)
    for i, a, b in _sequences(st):
        s = _scores(st, i, a, b)
        m = s.amax(-1, keepdim=True)
        q0 = st["cu_q_host"][i]
        lse[:, q0 + a:q0 + b] = (m + torch.log(torch.exp(s - m).sum(-1, keepdim=True))).reshape(c["h_q"], b - a)
    return lse


def _plain_prompt(st):
    c = st["case"]
    g = c["h_q"] // c["h_kv"]
    O = torch.empty(st["Q"].shape, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(c["h_q"], st["Q"].shape[0], device=DEV)
    for i, a, b in _sequences(st):
        s = _scores(st, i, a, b)
        m = s.amax(-1, keepdim=True)
        p = s.sub_(m).exp_()
        total = p.sum(-1, keepdim=True)
        v = st["V"][st["cu_k_host"][i]:st["cu_k_host"][i + 1]].float().transpose(0, 1)
        o = torch.matmul(p, v) / total
        q0 = st["cu_q_host"][i]
        O[q0 + a:q0 + b] = o.reshape(c["h_kv"], g, b - a, c["d"]).permute(2, 0, 1, 3).reshape(b - a, c["h_q"], c["d"])
        lse[:, q0 + a:q0 + b] = (m + torch.log(total)).reshape(c["h_q"], b - a)
    return O, lse


def _plain_weights(st):
    c = st["case"]
    w = st["w_in"].clone()
    for i, a, b in _sequences(st):
        s = _scores(st, i, a, b)
        q0 = st["cu_q_host"][i]
        p = torch.exp(s - st["lse"][:, q0 + a:q0 + b].reshape(c["h_kv"], -1, 1))
        w[:, st["cu_k_host"][i]:st["cu_k_host"][i + 1]] += p.sum(1)
    return w


def _plain_kv4(st):
    c = st["case"]
    n, hk, d = len(st["lens_host"]), c["h_kv"], c["d"]
    g = c["h_q"] // hk
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), (st["cu"][1:] - st["cu"][:-1]).long(),
                                  output_size=st["K"].shape[0])
    slot = st["start"][seq] + torch.arange(st["K"].shape[0], device=DEV) - st["cu"][seq]
    for x, codes, scales, lay in ((st["K"], "kc", "ks", _k_bytes), (st["V"], "vc", "vs", _v_bytes)):
        q, s = _quantise(x.float())
        st[codes][seq, :, slot] = lay(q)
        st[scales][seq, :, slot] = s
    top = max(st["lens_host"])
    O = torch.empty(n, c["h_q"], d, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(n, c["h_q"], device=DEV)
    w = st["w"]
    step = max(1, (1 << 29) // (hk * top * d))  # sequences at a time: 2 GB of unpacked keys
    for b0 in range(0, n, step):
        b1 = min(n, b0 + step)
        k = _value(_k_codes(st["kc"][b0:b1, :, :top]), st["ks"][b0:b1, :, :top])
        q = st["Q"][b0:b1].float().reshape(b1 - b0, hk, g, d)
        s = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
        hidden = torch.arange(top, device=DEV)[None, :] >= st["lens"][b0:b1, None]
        s.masked_fill_(hidden[:, None, None, :], float("-inf"))
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        total = p.sum(-1, keepdim=True)
        p = p / total
        v = _value(_v_codes(st["vc"][b0:b1, :, :top]), st["vs"][b0:b1, :, :top])
        O[b0:b1] = torch.matmul(p, v).reshape(b1 - b0, c["h_q"], d)
        lse[b0:b1] = (m + torch.log(total)).reshape(b1 - b0, c["h_q"])
        if w is not None:
            w[b0:b1, :, :top] = torch.where(hidden[:, None, :], 0.0, st["w_in"][b0:b1, :, :top] + p.sum(2))
    return (O, lse) if w is None else (O, lse, w)


def _plain_evict(st):
    c = st["case"]
    n, hk, cap, budget = len(st["lens_host"]), c["h_kv"], c["cap"], c["budget"]
    t = torch.arange(cap, device=DEV)
    lens = st["lens"].long()[:, None, None]
    order = st["w"].clone()
    kept_always = (t < c["sink"]) | (t >= lens - c["recent"])
    order = torch.where(kept_always, torch.full_like(order, float("inf")), order)
    order = torch.where(t >= lens, torch.full_like(order, float("-inf")), order)
    rank = torch.sort(order, dim=-1, descending=True, stable=True).indices[..., :budget]
    m = torch.clamp(st["lens"].long(), max=budget)[:, None, None]
    slots = torch.arange(budget, device=DEV)
    rank = torch.where(slots < m, rank, cap)  # places past the kept ones sort last
    idx = torch.sort(rank, dim=-1).values
    live = idx < cap
    at = torch.where(live, idx, 0)
    out = []
    for src, dst in zip(st["src"], st["dst"]):
        rows = src.reshape(n, hk, cap, -1)
        got = torch.gather(rows, 2, at[..., None].expand(-1, -1, -1, rows.shape[-1]))
        dst.copy_(torch.where(live[..., None], got, torch.zeros_like(got)).reshape(dst.shape))
        out.append(dst)
    return [torch.where(live, idx, -1).int(), m.flatten().int(), *out]


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if not own:
        return {"prompt": _plain_prompt, "weights": _plain_weights, "kv4": _plain_kv4, "evict": _plain_evict}[c["op"]](
            state)
    from input_adaptive_reduced_02_b200 import rmm
    if c["op"] == "prompt":
        return rmm.attn_prompt(state["Q"], state["K"], state["V"], state["cu_q"], state["cu_k"], scale=state["scale"],
                               causal=c["causal"], out_dtype=torch.bfloat16)
    if c["op"] == "weights":
        return rmm.attn_key_weights(state["Q"], state["K"], state["lse"], state["cu_q"], state["cu_k"],
                                    scale=state["scale"], causal=c["causal"], w_in=state["w_in"])
    if c["op"] == "kv4":
        cache = rmm.KV4Cache(state["kc"], state["ks"], state["vc"], state["vs"])
        rmm.kv4_store(cache, state["K"], state["V"], state["start"], state["cu"])
        O, lse, state["ws"] = rmm.kv4_attn(state["Q"], cache, state["lens"], scale=state["scale"],
                                           out_dtype=torch.bfloat16,
                                           w_in=state["w_in"], w_out=state["w"], workspace=state.get("ws"))
        return (O, lse) if state["w"] is None else (O, lse, state["w"])
    lens, idx, state["ws"] = rmm.cache_evict(state["w"], state["lens"], list(zip(state["src"], state["dst"])),
                                             c["budget"], sink=c["sink"], recent=c["recent"],
                                             workspace=state.get("ws"))
    return [idx, lens, *state["dst"]]


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("prompt", "weights"):
        return _exact_prompt(st)
    if case["op"] == "kv4":
        return _exact_kv4(st)
    return None  # a selection and a copy: nothing is rounded


def _exact_prompt(st):
    c = st["case"]
    g = c["h_q"] // c["h_kv"]
    tq, tk = st["Q"].shape[0], st["K"].shape[0]
    Q, K, V = st["Q"].double(), st["K"].double(), st["V"].double()
    weights = c["op"] == "weights"
    O = None if weights else torch.zeros(tq, c["h_q"], c["d"], dtype=torch.float64, device=DEV)
    lse = torch.zeros(c["h_q"], tq, dtype=torch.float64, device=DEV)
    w = st["w_in"].double() if weights else None
    for i in range(len(st["cu_q_host"]) - 1):
        q0, q1 = st["cu_q_host"][i:i + 2]
        k0, k1 = st["cu_k_host"][i:i + 2]
        off = (k1 - k0) - (q1 - q0)
        for h in range(c["h_q"]):
            for a in range(q0, q1, 4096):
                b = min(q1, a + 4096)
                end = min(k1, k0 + (b - q0) + off) if c["causal"] else k1  # keys beyond are seen by no row here
                x = (Q[a:b, h] @ K[k0:end, h // g].T) * st["scale"]
                if c["causal"]:
                    last = torch.arange(a - q0, b - q0, device=DEV)[:, None] + off
                    x[torch.arange(end - k0, device=DEV)[None, :] > last] = -math.inf
                if weights:
                    w[h // g, k0:end] += torch.exp(x - st["lse"][h, a:b].double()[:, None]).sum(0)
                    continue
                lse[h, a:b] = torch.logsumexp(x, 1)
                O[a:b, h] = torch.exp(x - lse[h, a:b, None]) @ V[k0:end, h // g]
    return w if weights else (O, lse)


def _exact_kv4(st):
    c = st["case"]
    n, hk, d = len(st["lens_host"]), c["h_kv"], c["d"]
    g = c["h_q"] // hk
    O = torch.zeros(n, c["h_q"], d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(n, c["h_q"], dtype=torch.float64, device=DEV)
    w = None if st["w"] is None else torch.zeros(n, hk, c["cap"], dtype=torch.float64, device=DEV)
    ch = torch.arange(d, device=DEV)
    # where channel c's code lies: byte and shift
    k_byte = (ch % 32 // 8) * (d // 8) + 4 * (ch // 32) + ch % 8 // 2
    k_shift = 4 * (ch % 2)
    v_nib = ch % 32 // 8
    v_byte = (ch % 8) * (d // 16) + 2 * (ch // 32) + v_nib // 2
    v_shift = 4 * (v_nib % 2)

    def stored(codes, scales, byte, shift):
        q = (codes[..., byte] >> shift.to(torch.uint8)) & 15
        s = scales.double().repeat_interleave(GROUP, dim=-2)
        return q.double() * s[..., 0] + s[..., 1]

    def fresh(x):
        out = torch.empty(x.shape, dtype=torch.float64, device=DEV)
        for a in range(0, d, GROUP):
            y = x[..., a:a + GROUP].double()
            lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
            s = ((hi - lo) / 15).to(torch.bfloat16).double()
            q = torch.where(s > 0, torch.clamp(torch.round((y - lo) / s), 0, 15), 0.0)
            out[..., a:a + GROUP] = lo + s * q
        return out

    nk, nv = fresh(st["K"]), fresh(st["V"])
    for b in range(n):
        L, s0 = st["lens_host"][b], st["start_host"][b]
        t0, t1 = st["cu_host"][b:b + 2]
        for h in range(hk):
            k = torch.cat((stored(st["kc"][b, h, :s0], st["ks"][b, h, :s0], k_byte, k_shift), nk[t0:t1, h]))
            v = torch.cat((stored(st["vc"][b, h, :s0], st["vs"][b, h, :s0], v_byte, v_shift), nv[t0:t1, h]))
            x = st["Q"][b, h * g:(h + 1) * g].double() @ k.T * st["scale"]
            lse[b, h * g:(h + 1) * g] = torch.logsumexp(x, 1)
            p = torch.softmax(x, 1)
            O[b, h * g:(h + 1) * g] = p @ v
            if w is not None:
                w[b, h, :L] = st["w_in"][b, h, :L].double() + p.sum(0)
    return (O, lse) if w is None else (O, lse, w)
