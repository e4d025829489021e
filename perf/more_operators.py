"""The operators of the softmax-attention layers that stand between KDA layers, as cases that can be timed
and checked.

A hybrid stack keeps a few layers whose memory grows with the context. Their keys and values are held in 4
bits, in pages:

  norm_rope  RMSNorm of every query and key head and the position rotation, one pass   (kda_qk_norm_rope)
  append     new keys and values quantised as they are written into the cache, and what the cache then
             holds for them                                          (kda_kv4_append, kda_kv4_read)
  read       cached keys and values back as ordinary tensors                           (kda_kv4_read)
  attention  softmax attention of new queries over the cache                           (kda_kv4_attention)

``run`` computes them in plain torch operations, or through the library where ``own`` is true.

The cache is uint8 [pages, Hk, page_size / 16, 18 * D]. A block of 18 * D bytes holds 16 tokens of one
key/value head, and a group of 32 channels of a token shares one bf16 scale of five significant bits:

  keys    codes  [16 tokens][4 quarters j][D/32 groups g] words of 4 bytes: channels 32g + 8j + 0..7
          scales [16 tokens][D/32 groups]
  values  codes  [8 token pairs p][8 places][2 tokens of the pair][D/32 groups g] halves of 2 bytes; place
                 (r + 2p) mod 8 holds channels 32g + 8(r/2) + (r mod 2) + {0, 2, 4, 6}
          scales [8 token pairs][D/32 groups][2 tokens of the pair]

A word's lower half holds its even channels, the upper half its odd ones, and a half is its four 4-bit codes
(the first in the lowest bits) rotated left by three bits. Code c stands for (c - 8) * scale.
"""
import math

import torch

own = False

NORM_EPS = 1e-6
GROUP = 32              # channels that share a scale
SCALE_MIN = 2.0 ** -100
SCALE_MAX = 2.0 ** 123
ROPE_BASE = 500000.0

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a decode batch of 64 sequences with 96 query heads, far into long contexts
        {"name": "norm_rope_step_64", "op": "norm_rope", "T": 64, "Hq": 96, "Hk": 8, "D": 128, "R": 128,
         "dtype": "bf16", "interleaved": False, "far": 131072},
        # odd tokens, heads of 64 of which half the channels turn, neighbouring channels as pairs, fp32
        {"name": "norm_rope_ragged", "op": "norm_rope", "T": 1001, "Hq": 6, "Hk": 2, "D": 64, "R": 32,
         "dtype": "f32", "interleaved": True, "far": 1 << 20},
        # a large prefill batch
        {"name": "norm_rope_prefill", "op": "norm_rope", "T": 8192, "Hq": 64, "Hk": 8, "D": 128, "R": 128,
         "dtype": "bf16", "interleaved": False, "far": 8192},
        # one new token for each of 64 sequences
        {"name": "append_step_64", "op": "append", "B": 64, "new": 1, "L": 1024, "Hk": 8, "D": 128, "page": 64,
         "dtype": "bf16"},
        # five prompts of odd lengths joined to what is there, heads of 64, fp32, small pages
        {"name": "append_ragged", "op": "append", "B": 5, "new": 777, "L": 1500, "Hk": 3, "D": 64, "page": 16,
         "dtype": "f32"},
        # prompts of eight sequences, up to 4096 tokens each
        {"name": "append_prefill", "op": "append", "B": 8, "new": 4096, "L": 4096, "Hk": 8, "D": 128, "page": 64,
         "dtype": "bf16"},
        # a shared prefix handed to code that wants ordinary tensors: short, ragged, fp32
        {"name": "read_ragged", "op": "read", "B": 3, "L": 1201, "Hk": 3, "D": 64, "page": 32, "dtype": "f32"},
        # the same for eight long sequences
        {"name": "read_prefix", "op": "read", "B": 8, "L": 16384, "Hk": 8, "D": 128, "page": 64, "dtype": "bf16"},
        # one sequence decoding at 4K context: a call whose latency counts
        {"name": "attn_step_1", "op": "attention", "B": 1, "new": 1, "L": 4096, "Hq": 32, "Hk": 8, "D": 128,
         "page": 64, "dtype": "bf16", "causal": True, "window": 0},
        # the decode batch: 64 sequences of up to 8192 tokens, 96 query heads over 8 key/value heads
        {"name": "attn_step_64", "op": "attention", "B": 64, "new": 1, "L": 8192, "Hq": 96, "Hk": 8, "D": 128,
         "page": 64, "dtype": "bf16", "causal": True, "window": 0},
        # a few drafted tokens a sequence, odd lengths, a sliding window, three queries a head of 64, fp32
        {"name": "attn_ragged", "op": "attention", "B": 5, "new": 7, "L": 3001, "Hq": 9, "Hk": 3, "D": 64,
         "page": 16, "dtype": "f32", "causal": True, "window": 1000},
        # a 4096-token chunk of a prompt behind as many cached tokens
        {"name": "attn_prefill", "op": "attention", "B": 1, "new": 4096, "L": 8192, "Hq": 32, "Hk": 8, "D": 128,
         "page": 64, "dtype": "bf16", "causal": True, "window": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "read", "attention", "attention"])
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm_rope":
        hk = rng.randint(1, 8)
        hq = hk * rng.randint(1, 12)
        t = _log_int(rng, 1, min(8192, 8192 * 72 * 128 // ((hq + hk) * d * (2 if dtype == "f32" else 1))))
        return {"op": op, "T": t, "Hq": hq, "Hk": hk, "D": d, "R": rng.choice([d, d, d // 2]), "dtype": dtype,
                "interleaved": rng.random() < 0.3, "far": _log_int(rng, 8192, 1 << 20)}
    page = rng.choice([16, 32, 64, 128])
    hk = rng.randint(1, 8)
    if op == "append":
        b = _log_int(rng, 1, 64)
        new = 1 if rng.random() < 0.4 else _log_int(rng, 1, max(1, min(4096, 8 * 4096 // (b * (2 if dtype == "f32" else 1)))))
        return {"op": op, "B": b, "new": new, "L": new + _log_int(rng, 1, 1024), "Hk": hk, "D": d, "page": page,
                "dtype": dtype}
    if op == "read":
        b = _log_int(rng, 1, 64)
        return {"op": op, "B": b, "L": _log_int(rng, 64, min(16384, 8 * 8192 // b)), "Hk": hk, "D": d, "page": page,
                "dtype": dtype}
    hq = hk * rng.randint(1, 12)
    base = {"op": op, "Hk": hk, "Hq": hq, "D": d, "page": page, "dtype": dtype, "causal": rng.random() < 0.85,
            "window": rng.choice([0, 0, 0, _log_int(rng, 64, 2048)])}
    kind = rng.random()
    if kind < 0.5:  # decoding, sometimes with a few drafted tokens
        b = _log_int(rng, 1, 64)
        new = rng.choice([1, 1, 1, rng.randint(2, 8)])
        return {**base, "B": b, "new": new, "L": new + _log_int(rng, 64, min(32768, 64 * 6000 // b))}
    b = rng.randint(1, 4)  # prompts, in bf16 mostly
    if dtype == "f32":
        base["dtype"] = rng.choice(["f32", "bf16"])
    new = _log_int(rng, 16, (2048 if base["dtype"] == "bf16" else 512) // b)
    return {**base, "B": b, "new": new, "L": new + _log_int(rng, 1, 4096 // b)}


# ---------------------------------------------------------------- sizes of a case
def _lengths(case):
    """Tokens held for each sequence once the new ones are in: between half of L and L, the first with L."""
    length, new = case["L"], case.get("new", 1)
    return [max(min(length, new), length - (7919 * b) % (length // 2 + 1)) for b in range(case["B"])]


def _new(case):
    """New tokens of each sequence."""
    if case["op"] == "read":
        return _lengths(case)
    return [max(1, case["new"] - (case["new"] * 3 * b) // (4 * case["B"])) for b in range(case["B"])]


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    op, d, hk, dt = case["op"], case["D"], case["Hk"], _DTYPES[case["dtype"]]
    if op == "norm_rope":
        t, hq = case["T"], case["Hq"]
        # queries, keys and values of a token side by side, as their common projection leaves them
        x = (randn(t, (hq + 2 * hk) * d) * torch.exp(0.5 * randn(t, 1))).to(dt)
        q, k = x[:, :hq * d].unflatten(1, (hq, d)), x[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        freq = ROPE_BASE ** (-torch.arange(0, case["R"], 2, dtype=torch.float64, device=dev) / case["R"])
        return {"op": op, "q": q, "k": k, "q_weight": 0.5 + rand(d), "k_weight": 0.5 + rand(d), "freq": freq,
                "positions": torch.randint(0, case["far"], (t,), generator=gen, device=dev),
                "interleaved": case["interleaved"], "q_out": torch.empty((t, hq, d), dtype=dt, device=dev),
                "k_out": torch.empty((t, hk, d), dtype=dt, device=dev)}

    page, lens, new = case["page"], _lengths(case), _new(case)
    b, t = len(lens), sum(new)
    per_seq = (case["L"] + page - 1) // page
    used = [(n + page - 1) // page for n in lens]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=gen, device=dev).int()
    table = torch.zeros((b, per_seq), dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = order[at:at + n]
        at += n
    cache = torch.empty((pages, hk, page // 16, 18 * d), dtype=torch.uint8, device=dev)
    # keys and values of a model: channels of different size
    kc, vc = torch.exp(0.4 * randn(hk, 1, d)), torch.exp(0.3 * randn(hk, 1, d))
    step = max(1, (1 << 25) // (hk * page * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        cache[p:p + n] = _blocks(randn(n, hk, page, d) * kc, randn(n, hk, page, d) * vc)
    lens_t = torch.tensor(lens, dtype=torch.int64, device=dev)
    cu = torch.zeros(b + 1, dtype=torch.int64, device=dev)
    cu[1:] = torch.tensor(new, dtype=torch.int64, device=dev).cumsum(0)
    state = {"op": op, "cache": cache, "table": table, "lens": lens_t,
             "cu": None if t == b and op != "read" else cu, "longest": max(lens), "most": max(new)}
    if op == "append":
        state["k"] = (randn(t, hk, d) * kc.view(hk, d)).to(dt)
        state["v"] = (randn(t, hk, d) * vc.view(hk, d)).to(dt)
    if op != "attention":
        state["k_out"] = torch.empty((t, hk, d), dtype=dt, device=dev)
        state["v_out"] = torch.empty((t, hk, d), dtype=dt, device=dev)
        return state
    state["q"] = (1.5 * randn(t, case["Hq"], d)).to(dt)
    state["out"] = torch.empty_like(state["q"])
    state["lse"] = torch.empty((t, case["Hq"]), device=dev)
    state["causal"], state["window"] = case["causal"], case["window"]
    return state


# ---------------------------------------------------------------- the cache's format in plain operations
def _quantise(x):
    """x [..., D] -> codes int32 [..., D] and scales bf16 [..., D / 32]."""
    xg = x.double().unflatten(-1, (-1, GROUP))
    m = xg.abs().amax(-1)
    # a seventh of the largest magnitude, rounded up to five significant bits; in 64 bits, because values
    # next to a border between two scales or two codes are common
    last = (1 << 48) - 1
    s = (((m / 7.0).view(torch.int64) + last) & ~last).view(torch.float64).clamp(SCALE_MIN, SCALE_MAX)
    c = torch.round(xg / s[..., None]).clamp(-7, 7) + 8
    fine = torch.isfinite(m)
    c = torch.where(fine[..., None], c, 8.0)
    return c.to(torch.int32).flatten(-2), torch.where(fine, s, float("nan")).to(torch.bfloat16)


def _places(d, device):
    """Where a block of 9 * D 16-bit words holds a token's, [16, 9 * D / 16]: its D/4 halves of keys and D/4 of
    values (by group, word and half), its D/32 scales of keys and of values."""
    def ar(n):
        return torch.arange(n, device=device)

    g = d // GROUP
    t, grp, word, half = ar(16)[:, None, None, None], ar(g)[:, None, None], ar(4)[:, None], ar(2)
    keys = t * (d // 4) + word * (d // 16) + grp * 2 + half
    pair, r = t // 2, 2 * word + half
    values = 9 * d // 2 + pair * (d // 2) + ((r + 2 * pair) % 8) * (d // 16) + (t % 2) * g + grp
    t, grp = ar(16)[:, None], ar(g)
    key_scales = 4 * d + t * g + grp
    value_scales = 17 * d // 2 + (t // 2) * (2 * g) + 2 * grp + t % 2
    return torch.cat([keys.flatten(1), values.flatten(1), key_scales, value_scales], 1)


def _words(k, v):
    """Keys and values [..., D] -> a token's 16-bit words int16 [..., 9 * D / 16]."""
    parts, scales = [], []
    for x in (k, v):
        codes, s = _quantise(x)
        c = codes.unflatten(-1, (-1, 4, 4, 2))
        h = c[..., 0, :] | (c[..., 1, :] << 4) | (c[..., 2, :] << 8) | (c[..., 3, :] << 12)
        h = ((h << 3) | (h >> 13)) & 0xFFFF
        parts.append(((h ^ 0x8000) - 0x8000).to(torch.int16).flatten(-3))
        scales.append(s.view(torch.int16))
    return torch.cat(parts + scales, -1)


def _values(words, d):
    """The inverse: a token's words -> keys and values fp32 [..., D]."""
    g, out = d // GROUP, []
    *halves, ks, vs = words.split([d // 4, d // 4, g, g], -1)
    for h, s in zip(halves, (ks, vs)):
        h = h.to(torch.int32) & 0xFFFF
        h = ((h >> 3) | (h << 13)) & 0xFFFF
        c = torch.stack([(h >> (4 * i)) & 15 for i in range(4)], -1)             # [..., word and half, nibble]
        c = c.unflatten(-2, (-1, 2)).transpose(-1, -2).flatten(-3)
        out.append(((c - 8).float().unflatten(-1, (g, GROUP)) * s.contiguous().view(torch.bfloat16).float()[..., None])
                   .flatten(-2))
    return out


def _blocks(k, v):
    """Keys and values [..., page, D] -> cache blocks uint8 [..., page / 16, 18 * D]."""
    d = k.shape[-1]
    w = _words(k, v).unflatten(-2, (-1, 16)).flatten(-2)
    out = torch.empty_like(w)
    out[..., _places(d, w.device).flatten()] = w
    return out.view(torch.uint8)


def _token_slots(state, t):
    """Of each new token: its sequence, its number among the sequence's new tokens, its position."""
    dev, lens, cu = state["lens"].device, state["lens"], state["cu"]
    tok = torch.arange(t, device=dev)
    if cu is None:
        return tok, torch.zeros_like(tok), lens - 1
    seq = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    idx = tok - cu[seq]
    return seq, idx, lens[seq] - (cu[seq + 1] - cu[seq]) + idx


# ---------------------------------------------------------------- the operators
def run(state):
    op = state["op"]
    if own:
        from linear_attention_recurrence_02_gb300 import kda
        if op == "norm_rope":
            kda.kda_qk_norm_rope(state["q"], state["k"], state["q_out"], state["k_out"], state["positions"],
                                 state["freq"], q_weight=state["q_weight"], k_weight=state["k_weight"],
                                 eps=NORM_EPS, interleaved=state["interleaved"])
            return {"q": state["q_out"], "k": state["k_out"]}
        if op == "append":
            kda.kda_kv4_append(state["k"], state["v"], state["cache"], state["table"], state["lens"],
                               cu_seqlens=state["cu"])
            kda.kda_kv4_read(state["cache"], state["table"], state["lens"], state["k_out"], state["v_out"],
                             cu_seqlens=state["cu"])
            return {"k": state["k_out"], "v": state["v_out"], "cache": state["cache"]}
        if op == "read":
            kda.kda_kv4_read(state["cache"], state["table"], state["lens"], state["k_out"], state["v_out"],
                             cu_seqlens=state["cu"])
            return {"k": state["k_out"], "v": state["v_out"]}
        kda.kda_kv4_attention(state["q"], state["cache"], state["table"], state["lens"], state["out"],
                              cu_seqlens=state["cu"], causal=state["causal"], window=state["window"],
                              lse=state["lse"])
        return {"out": state["out"], "lse": state["lse"]}

    if op == "norm_rope":
        angle = state["positions"].double()[:, None] * state["freq"]
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        r = 2 * state["freq"].shape[0]

        def one(x, w):
            y = x.float()
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + NORM_EPS) * w
            turn, rest = y[..., :r], y[..., r:]
            if state["interleaved"]:
                a, b = turn[..., 0::2], turn[..., 1::2]
                turn = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
            else:
                a, b = turn[..., :r // 2], turn[..., r // 2:]
                turn = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
            return torch.cat([turn, rest], -1).to(x.dtype)

        return {"q": one(state["q"], state["q_weight"]), "k": one(state["k"], state["k_weight"])}

    cache, table, lens = state["cache"], state["table"], state["lens"]
    hk, page, d = cache.shape[1], cache.shape[2] * 16, cache.shape[3] // 18
    if op in ("append", "read"):
        t, dt = state["k_out"].shape[0], state["k_out"].dtype
        seq, _, pos = _token_slots(state, t)
        block = (table[seq, pos // page].long()[:, None] * hk + torch.arange(hk, device=pos.device)) * (page // 16)
        block = block + (pos % page // 16)[:, None]
        at = block[..., None] * (9 * d) + _places(d, pos.device)[pos % 16][:, None]          # [T, hk, 9 d / 16]
        held = cache.view(torch.int16).view(-1)
        if op == "append":
            held[at] = _words(state["k"], state["v"])
        k, v = _values(held[at], d)
        out = {"k": k.to(dt), "v": v.to(dt)}
        return {**out, "cache": cache} if op == "append" else out

    # attention: sequences padded to the longest, all heads of a key/value head as rows of one product
    q, b = state["q"], lens.shape[0]
    t, hq = q.shape[:2]
    most, longest = state["most"], state["longest"]
    seq, idx, pos = _token_slots(state, t)
    n = (longest + page - 1) // page
    words = cache.view(torch.int16)[table[:, :n].long()].transpose(1, 2).flatten(2, 3)       # [b, hk, blocks, 9 d]
    k, v = _values(words[..., _places(d, q.device)], d)                                      # [b, hk, blocks, 16, d]
    k, v = (x.flatten(2, 3)[:, :, :longest] for x in (k, v))
    live = torch.arange(longest, device=q.device) < lens[:, None]
    v = torch.where(live[:, None, :, None], v, 0.0)
    qp = torch.zeros((b, most, hq, d), device=q.device)
    qp[seq, idx] = q.float()
    posp = torch.full((b, most), -1, dtype=torch.int64, device=q.device)
    posp[seq, idx] = pos
    qp = qp.unflatten(2, (hk, hq // hk)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = torch.matmul(qp, k.transpose(-1, -2)) / math.sqrt(d)
    j = torch.arange(longest, device=q.device)
    see = live[:, None, :].expand(-1, most, -1)
    if state["causal"]:
        see = see & (j <= posp[..., None])
    if state["window"]:
        see = see & (j > posp[..., None] - state["window"])
    see = see.repeat_interleave(hq // hk, 1)[:, None]
    s = s.masked_fill_(~see, -math.inf)
    m = s.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(s.sub_(m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf)

    def rows(x):
        return x.unflatten(2, (most, hq // hk)).permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, idx]

    return {"out": rows(o).to(q.dtype), "lse": rows(lse)[..., 0]}


# ---------------------------------------------------------------- bytes and operations
def _seen(case):
    """Pairs of a new token and a cached one that it attends to, and cached tokens that are seen at all."""
    pairs = read = 0
    for n, new in zip(_lengths(case), _new(case)):
        lo = 0
        for pos in ((n - new, n - 1) if case["window"] == 0 else range(n - new, n)):
            hi = pos + 1 if case["causal"] else n
            first = max(0, pos - case["window"] + 1) if case["window"] else 0
            if case["window"]:
                pairs += hi - first
                lo = first if pos == n - new else lo
        if case["window"] == 0:
            pairs += new * n - (new * (new - 1) // 2 if case["causal"] else 0)
        read += n - lo
    return pairs, read


def work(case):
    size = {"bf16": 2, "f32": 4}[case["dtype"]]
    d, hk = case["D"], case["Hk"]
    if case["op"] == "norm_rope":
        e = case["T"] * (case["Hq"] + hk) * d
        return {"bytes": 2 * e * size + 8 * case["T"] + 8 * d + 4 * case["R"], "flops": 10 * e}
    held = 9 * d // 8  # bytes of a token's keys and values of one head in the cache
    if case["op"] in ("append", "read"):
        e = sum(_new(case)) * hk
        full = 2 * e * d * size
        return {"bytes": (2 if case["op"] == "append" else 1) * (full + e * held) + 12 * case["B"],
                "flops": 4 * e * d * (2 if case["op"] == "append" else 1)}
    pairs, read = _seen(case)
    t = sum(_new(case))
    return {"bytes": read * hk * held + 2 * t * case["Hq"] * d * size + 4 * t * case["Hq"],
            "flops": 4 * pairs * case["Hq"] * d}


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        turn = torch.exp(1j * (s["positions"].double()[:, None] * s["freq"]))[:, None]
        n = case["R"] // 2

        def one(x, w):
            y = x.double()
            y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["D"] + NORM_EPS) * w.double()
            if case["interleaved"]:
                z = torch.complex(y[..., 0:2 * n:2], y[..., 1:2 * n:2]) * turn
                y[..., 0:2 * n:2], y[..., 1:2 * n:2] = z.real, z.imag
            else:
                z = torch.complex(y[..., :n], y[..., n:2 * n]) * turn
                y[..., :n], y[..., n:2 * n] = z.real, z.imag
            return y

        return {"q": one(s["q"], s["q_weight"]), "k": one(s["k"], s["k_weight"])}

    def held(x):
        """The values that a cache holds for x [..., D]."""
        parts = []
        for c in range(0, case["D"], GROUP):
            y = x[..., c:c + GROUP].double()
            m = y.abs().max(-1, keepdim=True).values / 7.0
            e = torch.floor(torch.log2(m)) - 4
            sc = torch.clamp(torch.ceil(m / torch.exp2(e)) * torch.exp2(e), SCALE_MIN, SCALE_MAX)
            parts.append(torch.round(y / sc) * sc)
        return torch.cat(parts, -1)

    def token(b, lo, hi):
        """Keys and values of tokens lo..hi of sequence b, [hi - lo, Hk, D], straight from the cache's bits."""
        d, page = case["D"], case["page"]
        g = d // GROUP
        pos = torch.arange(lo, hi, device="cuda")
        blk = s["cache"][s["table"][b, pos // page].long(), :, (pos % page) // 16].to(torch.int32)  # [n, hk, 18d]
        tt = (pos % 16)[:, None]
        c = torch.arange(d, device="cuda")[None]
        grp, word, half, nib = c // 32, (c % 32) // 8, c % 2, (c % 8) // 2
        rr = 2 * word + half
        k_at = tt * (d // 2) + word * (d // 8) + grp * 4 + half * 2
        v_at = 9 * d + (tt // 2) * d + ((rr + 2 * (tt // 2)) % 8) * (d // 8) + (tt % 2) * (2 * g) + 2 * grp
        ks_at = 8 * d + tt * (2 * g) + 2 * grp
        vs_at = 17 * d + (tt // 2) * (4 * g) + grp * 4 + (tt % 2) * 2
        out = []
        for at, s_at in ((k_at, ks_at), (v_at, vs_at)):
            def u16(i):
                i = i[:, None, :].expand(-1, blk.shape[1], -1)
                return blk.gather(2, i) | (blk.gather(2, i + 1) << 8)
            bit = ((3 + 4 * nib) % 16)[:, None]
            w = u16(at)
            code = ((w | (w << 16)) >> bit) & 15
            e = u16(s_at)
            scale = (1 + (e & 127).double() / 128) * torch.exp2((e >> 7).double() - 127)
            out.append((code - 8).double() * scale)
        return out

    cu = [0]
    for n in _new(case):
        cu.append(cu[-1] + n)
    if case["op"] == "append":
        return {"k": held(s["k"]), "v": held(s["v"]), "cache": None}
    if case["op"] == "read":
        got = [token(b, n - m, n) for b, (n, m) in enumerate(zip(_lengths(case), _new(case)))]
        return {"k": torch.cat([x[0] for x in got]), "v": torch.cat([x[1] for x in got])}

    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    g = case["Hq"] // case["Hk"]
    for b, n in enumerate(_lengths(case)):
        k, v = token(b, 0, n)
        for h in range(case["Hk"]):
            for c in range(cu[b], cu[b + 1], 1024):
                e = min(c + 1024, cu[b + 1])
                pos = torch.arange(n - cu[b + 1] + c, n - cu[b + 1] + e, device="cuda")[:, None, None]
                z = s["q"][c:e, h * g:(h + 1) * g].double() @ k[:, h].t() / math.sqrt(case["D"])
                j = torch.arange(n, device="cuda")
                if case["causal"]:
                    z = torch.where(j <= pos, z, -math.inf)
                if case["window"]:
                    z = torch.where(j > pos - case["window"], z, -math.inf)
                lse[c:e, h * g:(h + 1) * g] = torch.logsumexp(z, -1)
                out[c:e, h * g:(h + 1) * g] = torch.softmax(z, -1) @ v[:, h]
    return {"out": out, "lse": lse}
