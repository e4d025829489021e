"""The 8-bit operators around a KDA layer, as cases that can be timed and checked.

Three operators carry a layer's activations in 8 bits (e4m3 with one fp32 scale for each token and
block of 128 channels) from the residual stream into the layer and out of it again:

  add_norm  h = x + residual; RMSNorm(h) * weight in 8 bits          (kda_add_rmsnorm_fp8)
  gated     RMSNorm(o) * weight * act(gate) in 8 bits                (kda_gated_rmsnorm_fp8)
  linear    the product of such activations with block-scaled 8-bit weights  (kda_fp8_linear)

``run`` computes them in plain torch operations, or through the library where ``own`` is true.
"""
import math

import torch

own = False

BLOCK = 128            # channels (and weight rows) that share a scale
E4M3_MAX = 448.0       # largest e4m3 value
AMAX_MIN = 2.0 ** -96  # a block's largest magnitude counts as at least this
NORM_EPS = 1e-6

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one sequence decoding, generic hidden size: a call whose latency is all that counts
        {"name": "add_norm_step_1", "op": "add_norm", "T": 1, "N": 4096, "dtype": "bf16", "res": "bf16"},
        # a decode batch of 64 whose residual stream is kept in fp32
        {"name": "add_norm_step_64", "op": "add_norm", "T": 64, "N": 8192, "dtype": "bf16", "res": "f32"},
        # an odd number of tokens, a last block of 16 channels, everything in fp32
        {"name": "add_norm_ragged", "op": "add_norm", "T": 1001, "N": 1040, "dtype": "f32", "res": "f32"},
        # a large prefill batch
        {"name": "add_norm_prefill", "op": "add_norm", "T": 8192, "N": 8192, "dtype": "bf16", "res": "bf16"},
        # the decode workload's output (64 sequences, 96 heads of 128)
        {"name": "gated_step_64", "op": "gated", "T": 64, "H": 96, "D": 128, "dtype": "bf16", "act": "sigmoid"},
        # heads of 64, of which the fifth leaves half a block, fp32, SiLU gate
        {"name": "gated_ragged", "op": "gated", "T": 333, "H": 5, "D": 64, "dtype": "f32", "act": "silu"},
        # the 4096-token prefill workload's output
        {"name": "gated_prefill", "op": "gated", "T": 4096, "H": 96, "D": 128, "dtype": "bf16", "act": "sigmoid"},
        # one token through the output-gate projection (96 heads of 128)
        {"name": "linear_step_1", "op": "linear", "M": 1, "K": 4096, "N": 12288, "out": "bf16"},
        # the decode batch through the q, k and v projections
        {"name": "linear_step_64", "op": "linear", "M": 64, "K": 4096, "N": 36864, "out": "bf16"},
        # odd tokens, a last K block of 16 channels, a last weight block of 104 rows, fp32 result
        {"name": "linear_ragged", "op": "linear", "M": 777, "K": 1040, "N": 1000, "out": "f32"},
        # a 4096-token prompt through the output projection
        {"name": "linear_out_prefill", "op": "linear", "M": 4096, "K": 12288, "N": 4096, "out": "bf16"},
        # a 4096-token prompt through the q, k and v projections
        {"name": "linear_qkv_prefill", "op": "linear", "M": 4096, "K": 4096, "N": 36864, "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["add_norm", "gated", "linear", "linear"])
    if op == "add_norm":
        n = 16 * _log_int(rng, 8, 512)
        t = _log_int(rng, 1, min(16384, 8192 * 8192 // n))
        return {"op": op, "T": t, "N": n, "dtype": rng.choice(["bf16", "f32"]),
                "res": rng.choice(["bf16", "f32", "none"])}
    if op == "gated":
        d, h = rng.choice([16, 32, 64, 128]), rng.randint(1, 96)
        t = _log_int(rng, 1, min(8192, 4096 * 96 * 128 // (h * d)))
        return {"op": op, "T": t, "H": h, "D": d, "dtype": rng.choice(["bf16", "f32"]),
                "act": rng.choice(["sigmoid", "silu"])}
    k, n = 16 * _log_int(rng, 8, 768), _log_int(rng, 16, 36864)
    if rng.random() < 0.7:
        n = max(8, n // 8 * 8)
    k = 16 * max(8, min(k // 16, 36864 * 4096 // n // 16))
    m = _log_int(rng, 1, 4096)
    return {"op": op, "M": m, "K": k, "N": n, "out": rng.choice(["bf16", "bf16", "f32"])}


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    f8 = torch.float8_e4m3fn
    op = case["op"]
    if op == "add_norm":
        t, n = case["T"], case["N"]
        dt = _DTYPES[case["dtype"]]
        res = _DTYPES.get(case["res"])
        # the residual stream of a deep model: channels of very different size, a few of them large
        channel = torch.exp(0.5 * randn(n)) * torch.where(rand(n) < 0.002, 50.0, 1.0)
        x = randn(t, n).to(dt)
        r = (2.0 * randn(t, n) * channel).to(res) if res is not None else None
        return {"op": op, "x": x, "residual": r, "weight": 0.5 + rand(n),
                "sum": torch.empty((t, n), dtype=res, device=dev) if res is not None else None,
                "y": torch.empty((t, n), dtype=f8, device=dev),
                "scales": torch.empty((_blocks(n), t), device=dev)}
    if op == "gated":
        t, h, d = case["T"], case["H"], case["D"]
        dt = _DTYPES[case["dtype"]]
        # rows (token, head) of different size, as attention outputs are
        o = (randn(t, h, d) * torch.exp(randn(t, h, 1))).to(dt)
        return {"op": op, "o": o, "gate": (2.0 * randn(t, h, d)).to(dt), "weight": 0.5 + rand(d),
                "act": case["act"], "y": torch.empty((t, h, d), dtype=f8, device=dev),
                "scales": torch.empty((_blocks(h * d), t), device=dev)}
    m, k, n = case["M"], case["K"], case["N"]
    # normal values that fill the e4m3 range as a block's quantisation leaves them: its largest at 448
    a = (randn(m, k) * 120.0).clamp_(-E4M3_MAX, E4M3_MAX).to(f8)
    w = (randn(n, k) * 110.0).clamp_(-E4M3_MAX, E4M3_MAX).to(f8)
    return {"op": op, "a": a, "w": w,
            "a_scales": torch.exp(0.5 * randn(_blocks(k), m)) / 120.0,
            "w_scales": torch.exp(0.3 * randn(_blocks(n), _blocks(k))) * (0.02 / 110.0),
            "y": torch.empty((m, n), dtype=_DTYPES[case["out"]], device=dev)}


def _quantise(y):
    """Values [T, n] in fp32 -> their e4m3 codes [T, n] and scales [blocks, T]."""
    t, n = y.shape
    nb = _blocks(n)
    yb = torch.nn.functional.pad(y, (0, nb * BLOCK - n)).reshape(t, nb, BLOCK)
    s = yb.abs().amax(-1).clamp_min(AMAX_MIN) / E4M3_MAX
    q = (yb / s[..., None]).reshape(t, nb * BLOCK)[:, :n]
    return q.to(torch.float8_e4m3fn), s.t().contiguous()


def run(state):
    op = state["op"]
    if own:
        from linear_attention_recurrence_02_gb300 import kda
        if op == "add_norm":
            kda.kda_add_rmsnorm_fp8(state["x"], state["weight"], state["y"], state["scales"],
                                    residual=state["residual"], sum_out=state["sum"], eps=NORM_EPS)
            return {"sum": state["sum"], "y": state["y"], "scales": state["scales"]}
        if op == "gated":
            kda.kda_gated_rmsnorm_fp8(state["o"], state["gate"], state["weight"], state["y"], state["scales"],
                                      act=state["act"], eps=NORM_EPS)
            return {"y": state["y"], "scales": state["scales"]}
        kda.kda_fp8_linear(state["a"], state["a_scales"], state["w"], state["w_scales"], state["y"])
        return {"y": state["y"]}

    if op == "add_norm":
        h = state["x"].float()
        r = state["residual"]
        if r is not None:
            h = h + r.float()
        y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + NORM_EPS) * state["weight"]
        q, s = _quantise(y)
        return {"sum": None if r is None else h.to(r.dtype), "y": q, "scales": s}
    if op == "gated":
        o, z = state["o"].float(), state["gate"].float()
        sig = 1.0 / (1.0 + torch.exp(-z))
        act = z * sig if state["act"] == "silu" else sig
        y = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + NORM_EPS) * state["weight"] * act
        t, h, d = y.shape
        q, s = _quantise(y.reshape(t, h * d))
        return {"y": q.reshape(t, h, d), "scales": s}
    a, w, y = state["a"], state["w"], state["y"]
    (m, k), n = a.shape, w.shape[0]
    af = a.float() * state["a_scales"].t().repeat_interleave(BLOCK, 1)[:, :k]
    wf = w.float() * state["w_scales"].repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return {"y": torch.matmul(af, wf.t()).to(y.dtype)}


def work(case):
    size = {"bf16": 2, "f32": 4, "none": 0}
    if case["op"] == "add_norm":
        e = case["T"] * case["N"]
        return {"bytes": e * (size[case["dtype"]] + 2 * size[case["res"]] + 1) + 4 * case["N"]
                + 4 * case["T"] * _blocks(case["N"]), "flops": 8 * e}
    if case["op"] == "gated":
        e = case["T"] * case["H"] * case["D"]
        return {"bytes": e * (2 * size[case["dtype"]] + 1) + 4 * case["D"]
                + 4 * case["T"] * _blocks(case["H"] * case["D"]), "flops": 12 * e}
    m, k, n = case["M"], case["K"], case["N"]
    return {"bytes": m * k + n * k + 4 * _blocks(k) * (m + _blocks(n)) + m * n * size[case["out"]],
            "flops": 2 * m * n * k}


def exact(case, seed):
    """The operators' definitions in 64 bits; 8-bit outputs as the values before their rounding to e4m3."""
    s = prepare(case, seed)

    def codes(y):
        t, n = y.shape
        out = torch.empty_like(y)
        scales = []
        for c in range(0, n, BLOCK):
            part = y[:, c:c + BLOCK]
            sc = torch.maximum(part.abs().max(dim=1).values,
                               torch.tensor(AMAX_MIN, dtype=torch.float64, device=y.device)) / E4M3_MAX
            out[:, c:c + BLOCK] = part / sc[:, None]
            scales.append(sc)
        return out, torch.stack(scales)

    def rms_rows(v):
        return v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + NORM_EPS)

    if case["op"] == "add_norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = h + s["residual"].double()
        y, sc = codes(rms_rows(h) * s["weight"].double())
        return {"sum": h if s["residual"] is not None else None, "y": y, "scales": sc}
    if case["op"] == "gated":
        g = s["gate"].double()
        act = torch.sigmoid(g)
        if case["act"] == "silu":
            act = act * g
        v = rms_rows(s["o"].double()) * s["weight"].double() * act
        y, sc = codes(v.reshape(case["T"], -1))
        return {"y": y.reshape(v.shape), "scales": sc}
    m, k, n = case["M"], case["K"], case["N"]
    acc = torch.zeros((m, n), dtype=torch.float64, device="cuda")
    rows = torch.arange(n, device="cuda") // BLOCK
    for b, c in enumerate(range(0, k, BLOCK)):
        part = s["a"][:, c:c + BLOCK].double() @ s["w"][:, c:c + BLOCK].double().t()
        acc += part * s["a_scales"][b].double()[:, None] * s["w_scales"][:, b].double()[rows][None, :]
    return {"y": acc}
