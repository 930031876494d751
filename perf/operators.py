"""Operators of a packed-document training step: what is measured, and their plain forms.

Three operators around the split backward of a stage:
  rotary      rotary positions on the query and key heads of a qkv tensor, forward and backward
  attention   softmax attention inside packed documents, with an optional prefix that every row of a
              document sees, a tanh cap on the scores and a bias that grows with the distance
  adamw       one AdamW step over the tensors of a layer, states in 32 or 8 bits, and the global
              gradient norm that clips it

`own` false: plain torch forms in float32 (float64 angles).  `own` true: the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

LOG2E = 1.0 / math.log(2.0)

# A layer of the 8B-shaped and the 70B-shaped stage, and the tiny transformer of the tests.
LAYERS = {
    "8b": dict(hidden=4096, ffn=14336, nh=32, nkv=8, hd=128),
    "70b": dict(hidden=8192, ffn=28672, nh=64, nkv=8, hd=128),
    "tiny": dict(hidden=256, ffn=512, nh=4, nkv=2, hd=64),
}


def _shape(name):
    s = LAYERS[name]
    return dict(nh=s["nh"], nkv=s["nkv"], hd=s["hd"])


def listed():
    r = dict(op="rotary", backward=False, offset=0, docs=0, layout=0)
    a = dict(op="attention", backward=False, docs=1, pad=0, prefix=0, cap=0.0, bias=False, layout=0)
    w = dict(op="adamw", tensors="layer", layout=0, master=True, grad16=False, stochastic=False)
    return [
        # one 128-token microbatch of the tests' small transformer: launch latency
        dict(r, name="rotary_tiny", tokens=128, **_shape("tiny"), rot=64, pairs="half", scaling="none"),
        # a layer of the 8B-shaped stage on packed documents, frequencies stretched for a longer context
        dict(r, name="rotary_8b", tokens=4096, **_shape("8b"), rot=128, pairs="half", scaling="banded", docs=9, layout=1),
        # the backward of a long sequence at far positions, half of each head rotated, 70B-shaped heads
        dict(r, name="rotary_far_70b_bwd", tokens=16384, **_shape("70b"), rot=64, pairs="interleaved", scaling="yarn",
             backward=True, offset=1000000),
        # a small ragged batch: five documents off every tile boundary and padding rows behind the last
        dict(a, name="attn_small", tokens=700, **_shape("tiny"), docs=5, pad=60, cap=30.0, layout=2),
        # a packed microbatch of the 8B-shaped layer, forward and backward
        dict(a, name="attn_docs_8b", tokens=4096, **_shape("8b"), docs=9, layout=1),
        dict(a, name="attn_docs_8b_bwd", tokens=4096, **_shape("8b"), docs=9, layout=1, backward=True),
        # the same layer with capped scores; prefix-visible prompts and a ragged end in the backward
        dict(a, name="attn_cap_8b", tokens=4096, **_shape("8b"), docs=2, cap=50.0, layout=3),
        dict(a, name="attn_cap_prefix_8b_bwd", tokens=4000, **_shape("8b"), docs=4, pad=37, prefix=300, cap=50.0, layout=4,
             backward=True),
        # one long document with a distance bias, heads of 64
        dict(a, name="attn_bias_long", tokens=16384, nh=16, nkv=4, hd=64, bias=True),
        # the optimizer of the tests' two-layer stage: 12 small tensors, clipped by their norm
        dict(w, name="adamw_tiny", model="tiny", n_layers=2, bits=32, clip=True),
        # one layer of the 8B-shaped stage: float32 states, clipped; then 8-bit states
        dict(w, name="adamw_8b", model="8b", n_layers=1, bits=32, clip=True),
        dict(w, name="adamw_8b_state8", model="8b", n_layers=1, bits=8, clip=False, stochastic=True),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of lo .. hi."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "attention", "attention", "adamw"])
    layout = rng.randrange(1, 1 << 20)
    heads = rng.choice([(4, 2, 64), (32, 8, 128), (64, 8, 128), (6, 3, 64), (2, 1, 128), (16, 4, 64), (5, 5, 128)])
    shape = dict(nh=heads[0], nkv=heads[1], hd=heads[2])
    if op == "rotary":
        return dict(op=op, tokens=_log(rng, 1, 16384), **shape, rot=rng.choice([16, 32, 48, 64, heads[2]]),
                    pairs=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "ntk", "yarn", "banded"]),
                    backward=rng.random() < 0.5, offset=rng.choice([0, 0, 4099, 1000003]), docs=rng.choice([0, 0, 3, 17]),
                    layout=layout)
    if op == "attention":
        tokens = _log(rng, 1, 3500 if heads[0] > 32 else 4096 if heads[0] > 16 else 8192)
        return dict(op=op, tokens=tokens, **shape, docs=min(tokens, rng.choice([1, 1, 2, 5, 12, 40])),
                    pad=rng.choice([0, 0, 1, 77]), prefix=rng.choice([0, 0, 1, 50, 400]),
                    cap=rng.choice([0.0, 0.0, 30.0, 50.0]), bias=rng.random() < 0.3, layout=layout,
                    backward=rng.random() < 0.6)
    bits = rng.choice([32, 8])
    return dict(op=op, tensors="ragged", model="", n_layers=_log(rng, 1, 14), layout=layout, bits=bits,
                total=_log(rng, 1000, 100000000), clip=bits == 32 and rng.random() < 0.5, master=rng.random() < 0.7,
                grad16=rng.random() < 0.3, stochastic=bits == 8 and rng.random() < 0.5)


# ---------------------------------------------------------------- the layout of a case (no tensors)


def _doc_bounds(case):
    """Row offsets of the documents: tokens - pad rows cut at seeded places; rows behind them are padding."""
    n = max(0, case["tokens"] - case.get("pad", 0))
    rng = random.Random(case["layout"])
    cuts = sorted(rng.randrange(n + 1) for _ in range(case["docs"] - 1)) if case["docs"] > 1 else []
    return [0] + cuts + [n]


def _prefixes(case):
    rng = random.Random(case["layout"] + 1)
    return [rng.randrange(case["prefix"] + 1) if case["prefix"] else 0 for _ in range(case["docs"])]


def _tensor_sizes(case):
    """(count, is a weight) of every tensor of the optimizer."""
    if case["tensors"] == "layer":
        s = LAYERS[case["model"]]
        h, f = s["hidden"], s["ffn"]
        one = [((s["nh"] + 2 * s["nkv"]) * s["hd"] * h, True), (h * h, True), (2 * f * h, True), (h * f, True),
               (h, False), (h, False)]
        return one * case["n_layers"]
    rng = random.Random(case["layout"])
    parts = [rng.random() ** 3 + 1e-3 for _ in range(case["n_layers"])]
    return [(max(1, int(case["total"] * p / sum(parts))), rng.random() < 0.8) for p in parts]


def _frequencies(case):
    """Angles per position (float64) of the pairs, and the factor on the rotated values."""
    rot, base, factor, context = case["rot"], 10000.0, 8.0, 8192.0
    i = np.arange(rot // 2, dtype=np.float64)
    kind, mag = case["scaling"], 1.0
    if kind == "ntk":
        base *= factor ** (rot / (rot - 2.0))
    freq = base ** (-2.0 * i / rot)
    if kind == "linear":
        freq = freq / factor
    elif kind == "yarn":
        at = lambda turns: rot * math.log(context / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))  # noqa: E731
        low, high = max(math.floor(at(32.0)), 0.0), min(math.ceil(at(1.0)), rot - 1.0)
        ramp = np.clip((i - low) / max(high - low, 1e-3), 0.0, 1.0)
        freq = freq / factor * ramp + freq * (1.0 - ramp)
        mag = 0.1 * math.log(factor) + 1.0
    elif kind == "banded":
        turns = context * freq / (2.0 * math.pi)
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
    return freq, mag


# ---------------------------------------------------------------- inputs

HYPER = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8)
DECAY, MAX_NORM, SEED = 0.1, 1.0, 20250
BLOCK = 256                                  # elements that share an 8-bit state's scale
M_TOP, V_TOP = 15.0 * 2 ** 14, 15.0 * 2 ** 30  # the largest 8-bit codes' values
TINY = float(np.finfo(np.float32).tiny)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    st = {"case": case}
    if case["op"] == "adamw":
        return _prepare_adamw(case, st, normal)
    t, nh, nkv, hd = case["tokens"], case["nh"], case["nkv"], case["hd"]
    w = (nh + 2 * nkv) * hd
    st["qkv"] = normal(t, w).to(torch.bfloat16)
    if case["op"] == "rotary":
        st["out"] = torch.empty(t, (nh + nkv) * hd, dtype=torch.bfloat16, device="cuda")
        pos = torch.arange(t, dtype=torch.int64)
        if case["docs"]:
            starts = torch.tensor(_doc_bounds(dict(case, pad=0)), dtype=torch.int64)
            pos = pos - starts[torch.searchsorted(starts, pos, right=True).clamp(max=case["docs"]) - 1]
        st["positions"] = (pos + case["offset"]).to(torch.int32).cuda()
        freq, st["magnitude"] = _frequencies(case)
        st["freq"] = torch.from_numpy(freq).cuda()
        # turns per position as 64-bit fixed-point fractions of a turn, as the library's table holds them
        turns = [int(f / (2.0 * math.pi) * 2.0 ** 64 + 0.5) & (2 ** 64 - 1) for f in freq.tolist()]
        st["turns"] = torch.from_numpy(np.array(turns, dtype=np.uint64).view(np.int64)).cuda()
        return st
    st["offsets"] = torch.tensor(_doc_bounds(case), dtype=torch.int32, device="cuda")
    st["prefix"] = torch.tensor(_prefixes(case), dtype=torch.int32, device="cuda") if case["prefix"] else None
    # slopes 2^-1 .. 2^-8 over the heads, as distance-biased models use
    st["slopes"] = torch.exp2(-8.0 * torch.arange(1, nh + 1, device="cuda") / nh) if case["bias"] else None
    if case["cap"]:  # scores large enough that the cap matters
        st["qkv"][:, : nh * hd] *= 8.0
    stride = max(128, (t + 127) // 128 * 128)
    st["a"] = torch.empty(t, nh * hd, dtype=torch.bfloat16, device="cuda")
    st["lse"] = torch.zeros(nh, stride, device="cuda")
    if case["backward"]:
        a, lse = _attention_forward(st)
        st["a"].copy_(a)
        st["lse"][:, :t] = lse
        st["da"] = normal(t, nh * hd).to(torch.bfloat16)
        st["dqkv"] = torch.empty_like(st["qkv"])
    return st


def _prepare_adamw(case, st, normal):
    """A training run some steps in: gradients of about 1e-3, moments that follow them."""
    st["step"] = 100
    st["tensors"] = []
    for n, weight in _tensor_sizes(case):
        t = {"grad": normal(n).mul_(1e-3), "param": normal(n).mul_(0.02 if weight else 0.1).add_(0.0 if weight else 1.0)}
        t["decay"] = DECAY if weight else 0.0
        if weight:
            p32 = t["param"]
            t["param"] = p32.to(torch.bfloat16)
            if case["master"]:
                t["master"] = p32
        if case["grad16"]:
            t["grad"] = t["grad"].to(torch.bfloat16)
        m, v = normal(n).mul_(3e-4), normal(n).mul_(1e-3).square_().add_(1e-9)
        if case["bits"] == 8:
            half = torch.tensor(0x8000, device="cuda")
            t["m"], t["m_scale"] = _pack(m, M_TOP, half, signed=True)
            t["v"], t["v_scale"] = _pack(v, V_TOP, half, signed=False)
        else:
            t["m"], t["v"] = m, v
        st["tensors"].append(t)
    st["grad_scale"] = torch.full((), 0.75, device="cuda")  # a loss scale's inverse, or a clip coefficient
    return st


# ---------------------------------------------------------------- plain forms


def _rotary(st):
    case, x = st["case"], st["qkv"]
    t, n, hd, r = case["tokens"], case["nh"] + case["nkv"], case["hd"], case["rot"]
    x = x[:, : n * hd].float().view(t, n, hd)
    angle = st["positions"].double()[:, None] * st["freq"][None, :]
    cos = (torch.cos(angle) * st["magnitude"]).float()[:, None, :]
    sin = (torch.sin(angle) * st["magnitude"]).float()[:, None, :]
    if case["backward"]:
        sin = -sin
    y = x.clone()
    if case["pairs"] == "half":
        a, b = x[..., : r // 2], x[..., r // 2 : r]
        y[..., : r // 2], y[..., r // 2 : r] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    return y.to(torch.bfloat16).view(t, n * hd)


def _scores(st):
    """(q, k, v, scores in float32, visible, what the cap's derivative is), heads as [kv head, group, rows, d]."""
    case = st["case"]
    t, nh, nkv, hd = case["tokens"], case["nh"], case["nkv"], case["hd"]
    x = st["qkv"].float()
    q = x[:, : nh * hd].view(t, nkv, nh // nkv, hd).permute(1, 2, 0, 3)
    k = x[:, nh * hd : (nh + nkv) * hd].view(t, nkv, 1, hd).permute(1, 2, 0, 3)
    v = x[:, (nh + nkv) * hd :].view(t, nkv, 1, hd).permute(1, 2, 0, 3)
    s = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(hd)
    slope = None
    if case["cap"]:
        s = torch.tanh(s / case["cap"])
        slope = 1.0 - s * s
        s = s * case["cap"]
    row = torch.arange(t, device="cuda", dtype=torch.int32)
    if case["bias"]:
        s = s - st["slopes"].view(nkv, nh // nkv, 1, 1) * (row[:, None] - row[None, :]).abs().float()
    doc = torch.searchsorted(st["offsets"], row, right=True) - 1
    inside = doc < case["docs"]
    doc = doc.clamp(max=case["docs"] - 1)
    at = row - st["offsets"][doc]
    seen = row[None, :] <= row[:, None]
    if st["prefix"] is not None:
        seen = seen | (at < st["prefix"][doc])[None, :]
    visible = seen & (doc[:, None] == doc[None, :]) & inside[:, None] & inside[None, :]
    return q, k, v, s, visible, slope


def _attention_forward(st):
    case = st["case"]
    t, nh, hd = case["tokens"], case["nh"], case["hd"]
    _, _, v, s, visible, _ = _scores(st)
    s = torch.where(visible, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    a = torch.matmul(p, v) / torch.where(total > 0.0, total, 1.0)
    lse = ((top + torch.log(total)) * LOG2E).view(nh, t)
    return a.permute(2, 0, 1, 3).reshape(t, nh * hd).to(torch.bfloat16), lse


def _attention_backward(st):
    case = st["case"]
    t, nh, nkv, hd = case["tokens"], case["nh"], case["nkv"], case["hd"]
    q, k, v, s, visible, slope = _scores(st)
    heads = lambda x: x.float().view(t, nkv, nh // nkv, hd).permute(1, 2, 0, 3)  # noqa: E731
    da, a = heads(st["da"]), heads(st["a"])
    lse = st["lse"][:, :t].view(nkv, nh // nkv, t, 1)
    p = torch.where(visible, torch.exp2(s * LOG2E - lse), 0.0)
    del s
    dv = torch.matmul(p.transpose(-1, -2), da).sum(1)
    ds = p * (torch.matmul(da, v.transpose(-1, -2)) - (da * a).sum(-1, keepdim=True))
    del p
    if slope is not None:
        ds = ds * slope
    ds = ds / math.sqrt(hd)
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(1)
    flat = lambda x: x.permute(1, 0, 2).reshape(t, nkv * hd)  # noqa: E731
    return torch.cat([dq.permute(2, 0, 1, 3).reshape(t, nh * hd), flat(dk), flat(dv)], 1).to(torch.bfloat16)


def _mix(x):
    """An xorshift-multiply mixing of 32-bit words (in int64)."""
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _noise(count, tensor, step):
    """The 32 random bits of every element of a tensor at a step."""
    key = _mix(torch.tensor((SEED ^ (step * 0x9E3779B1)) & 0xFFFFFFFF, device="cuda"))
    key = _mix((key + tensor * 0x85EBCA77) & 0xFFFFFFFF)
    return _mix(torch.arange(count, device="cuda") ^ key)


def _blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)


def _pack(x, top, noise16, signed):
    """8-bit codes of x, 256 elements to a scale: codes (8 + f) 2^(e - 1), the block's largest value at the top one."""
    blocks = _blocks(x)
    scale = (blocks.abs().amax(1) / top).clamp(min=TINY)
    z = (blocks.abs() * (1.0 / scale)[:, None]).clamp(max=top).view(-1)[: x.numel()]
    small = z < 8.0
    bits = torch.where(small, z + 8.0, z).view(torch.int32).to(torch.int64)
    code = ((bits + (noise16 << 4)) >> 20) - torch.where(small, 1040, 1032)
    if signed:
        code = code | torch.where(torch.signbit(x), 128, 0)
    else:  # what is not zero stays so: a second moment that vanished would blow the next update up
        code = torch.maximum(code, (z > 0.0).to(torch.int64))
    return code.to(torch.uint8), scale


def _unpack(code, scale, signed):
    c = code.to(torch.int32)
    mag = c & 127 if signed else c
    value = torch.where(mag < 8, mag.float(), ((mag + 1032) << 20).view(torch.float32))
    if signed:
        value = torch.where(c > 127, -value, value)
    return (_blocks(value) * scale[:, None]).view(-1)[: code.numel()]


def _adamw_one(case, st, t, index, scale):
    h, step = HYPER, st["step"]
    g = t["grad"].float()
    if scale is not None:
        g = g * scale
    small = case["bits"] == 8
    noise = _noise(g.numel(), index, step) if case["stochastic"] else None
    m = _unpack(t["m"], t["m_scale"], True) if small else t["m"]
    v = _unpack(t["v"], t["v_scale"], False) if small else t["v"]
    m = m * h["beta1"] + g * (1.0 - h["beta1"])
    v = v * h["beta2"] + (g * g) * (1.0 - h["beta2"])
    p = t["master"] if "master" in t else t["param"].float()
    denom = torch.sqrt(v) / math.sqrt(1.0 - h["beta2"] ** step) + h["eps"]
    p = p * (1.0 - h["lr"] * t["decay"]) - (h["lr"] / (1.0 - h["beta1"] ** step)) * (m / denom)
    if small:
        half = torch.tensor(0x8000, device="cuda")
        t["m"], t["m_scale"] = _pack(m, M_TOP, half if noise is None else noise & 0xFFFF, True)
        t["v"], t["v_scale"] = _pack(v, V_TOP, half if noise is None else noise >> 16, False)
        m, v = _unpack(t["m"], t["m_scale"], True), _unpack(t["v"], t["v_scale"], False)
    else:
        t["m"], t["v"] = m, v
    out = {"m": m, "v": v}
    if "master" in t:
        t["master"] = out["master"] = p
    elif noise is not None and t["param"].dtype == torch.bfloat16:  # no master copy: the parameter rounds by the noise too
        p = (((p.view(torch.int32).to(torch.int64) + (((noise * 0x9E3779B1) & 0xFFFFFFFF) >> 16)) >> 16) << 16).to(torch.int32).view(torch.float32)
    t["param"] = out["param"] = p.to(t["param"].dtype)
    return out


def _adamw(st):
    case = st["case"]
    scale, out = st["grad_scale"], {}
    if case["clip"]:
        norm = torch.sqrt(torch.stack([t["grad"].double().square().sum() for t in st["tensors"]]).sum())
        out["norm"] = norm.float()
        scale = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0).float()
    out["tensors"] = [_adamw_one(case, st, t, i, scale) for i, t in enumerate(st["tensors"])]
    st["step"] += 1
    return out


# ---------------------------------------------------------------- the library's calls


def _own_rotary(st):
    from backward_split_linear_gb300 import binding as zb

    case = st["case"]
    n, hd = case["nh"] + case["nkv"], case["hd"]
    call = zb.zb_op_rotary_backward if case["backward"] else zb.zb_op_rotary_forward
    call(st["qkv"], st["out"], st["positions"], st["turns"], st["magnitude"], case["tokens"], n, hd, case["rot"], case["pairs"],
         ld_x=(case["nh"] + 2 * case["nkv"]) * hd, ld_y=n * hd)
    return st["out"]


def _own_attention(st):
    from backward_split_linear_gb300 import binding as zb

    case = st["case"]
    t, heads = case["tokens"], (case["nh"], case["nkv"], case["hd"])
    if "plan" not in st:  # workspaces that the program keeps; their contents are written in every pass
        st["plan"] = torch.empty(zb.zb_op_attention_document_plan_bytes(t), dtype=torch.uint8, device="cuda")
        st["scratch"] = torch.empty(zb.zb_op_attention_document_scratch_bytes(t, case["nh"]), dtype=torch.uint8, device="cuda")
    plan = st["plan"]
    zb.zb_op_attention_document_plan(st["offsets"], st["prefix"], case["docs"], t, plan, plan.numel())
    if case["backward"]:
        zb.zb_op_attention_document_backward(st["qkv"], st["a"], st["da"], st["lse"], st["dqkv"], plan, st["slopes"],
                                             case["cap"], t, *heads, st["scratch"], st["scratch"].numel())
        return st["dqkv"]
    zb.zb_op_attention_document_forward(st["qkv"], st["a"], st["lse"], plan, st["slopes"], case["cap"], t, *heads)
    return st["a"], st["lse"][:, :t]


def _own_adamw(st):
    from backward_split_linear_gb300 import runtime

    case = st["case"]
    if "optimizer" not in st:  # the optimizer object of the program: it holds the tensors' table
        st["optimizer"] = runtime.AdamW([{k: v for k, v in t.items() if k != "decay"} | {"weight_decay": t["decay"]}
                                         for t in st["tensors"]], state_bits=case["bits"], stochastic=case["stochastic"],
                                        seed=SEED, step=st["step"] - 1, **HYPER)
    opt, out = st["optimizer"], {}
    if case["clip"]:
        out["norm"], scale = opt.grad_norm(MAX_NORM)
    else:
        scale = st["grad_scale"]
    opt.step(grad_scale=scale)
    states = opt.unpack_states() if case["bits"] == 8 else [(t["m"], t["v"]) for t in st["tensors"]]
    out["tensors"] = [{"m": m, "v": v} | {k: t[k] for k in ("master", "param") if k in t}
                      for t, (m, v) in zip(st["tensors"], states)]
    return out


def run(st):
    op = st["case"]["op"]
    if own:
        return {"rotary": _own_rotary, "attention": _own_attention, "adamw": _own_adamw}[op](st)
    if op == "rotary":
        return _rotary(st)
    if op == "attention":
        return _attention_backward(st) if st["case"]["backward"] else _attention_forward(st)
    return _adamw(st)


# ---------------------------------------------------------------- work and the definition in 64 bits


def _visible_pairs(case):
    pairs, off = 0, _doc_bounds(case)
    for d, pre in enumerate(_prefixes(case)):
        n = off[d + 1] - off[d]
        pre = min(pre, n)
        pairs += n * (n + 1) // 2 + pre * (pre - 1) // 2
    return pairs


def work(case):
    if case["op"] == "adamw":
        total = flops = 0.0
        for n, weight in _tensor_sizes(case):
            per = 2 if case["grad16"] else 4                           # the gradient
            per += 4 if not weight else (4 + 4 + 2 if case["master"] else 2 + 2)  # parameter read and written
            per += 4 if not weight else 0
            per += 16 if case["bits"] == 32 else 4 + 8 + 16 / BLOCK      # moments in and out (8 bits: values out too)
            total += per * n
            flops += 16.0 * n
        return {"bytes": total, "flops": flops}
    t, nh, nkv, hd = case["tokens"], case["nh"], case["nkv"], case["hd"]
    if case["op"] == "rotary":
        n = (nh + nkv) * hd
        return {"bytes": 4.0 * t * n + 4.0 * t, "flops": 3.0 * t * (nh + nkv) * case["rot"]}
    w = (nh + 2 * nkv) * hd
    pairs = max(1, _visible_pairs(case)) * nh
    if case["backward"]:
        return {"bytes": 2.0 * t * (2 * w + 2 * nh * hd) + 4.0 * t * nh, "flops": 10.0 * hd * pairs}
    return {"bytes": 2.0 * t * (w + nh * hd) + 4.0 * t * nh, "flops": 4.0 * hd * pairs}


def exact(case, seed):
    st = prepare(case, seed)
    return {"rotary": _exact_rotary, "attention": _exact_attention, "adamw": _exact_adamw}[case["op"]](case, st)


def _exact_rotary(case, st):
    """Pairs as complex numbers times magnitude * exp(+-i angle)."""
    t, n, hd, r = case["tokens"], case["nh"] + case["nkv"], case["hd"], case["rot"]
    y = st["qkv"][:, : n * hd].double().view(t, n, hd).clone()
    first = slice(0, r // 2) if case["pairs"] == "half" else slice(0, r, 2)
    second = slice(r // 2, r) if case["pairs"] == "half" else slice(1, r, 2)
    freq = torch.from_numpy(_frequencies(case)[0]).cuda()
    angle = torch.outer(st["positions"].double(), freq) * (-1.0 if case["backward"] else 1.0)
    turn = torch.polar(torch.full_like(angle, st["magnitude"]), angle)[:, None, :]
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y.view(t, n * hd)


def _exact_attention(case, st):
    """Document by document and head by head."""
    t, nh, nkv, hd = case["tokens"], case["nh"], case["nkv"], case["hd"]
    x = st["qkv"].double().view(t, nh + 2 * nkv, hd)
    off, pre = _doc_bounds(case), _prefixes(case)
    out = torch.zeros_like(x) if case["backward"] else torch.zeros(t, nh, hd, dtype=torch.float64, device="cuda")
    lse = torch.full((nh, t), -math.inf, dtype=torch.float64, device="cuda")
    for d in range(case["docs"]):
        rows = slice(off[d], off[d + 1])
        n = off[d + 1] - off[d]
        if n == 0:
            continue
        i = torch.arange(n, device="cuda")
        hidden = ~((i[None, :] <= i[:, None]) | (i < pre[d])[None, :])
        for h in range(nh):
            j = h // (nh // nkv)
            q, k, v = x[rows, h], x[rows, nh + j], x[rows, nh + nkv + j]
            s = q @ k.T / hd ** 0.5
            if case["cap"]:
                ratio = torch.tanh(s / case["cap"])
                s = ratio * case["cap"]
            if case["bias"]:
                s = s - st["slopes"][h].double() * (i[:, None] - i[None, :]).abs()
            s.masked_fill_(hidden, -math.inf)
            if not case["backward"]:
                lse[h, rows] = torch.logsumexp(s, 1) / math.log(2.0)
                out[rows, h] = torch.softmax(s, 1) @ v
                continue
            do, a = st["da"].double().view(t, nh, hd)[rows, h], st["a"].double().view(t, nh, hd)[rows, h]
            p = torch.exp(s - st["lse"][h, rows].double()[:, None] * math.log(2.0))
            out[rows, nh + nkv + j] += p.T @ do
            ds = p * (do @ v.T - (do * a).sum(1, keepdim=True))
            if case["cap"]:
                ds = ds * (1.0 - ratio ** 2)
            out[rows, h] = ds @ k / hd ** 0.5
            out[rows, nh + j] += ds.T @ q / hd ** 0.5
    if case["backward"]:
        return out.view(t, -1)
    return out.view(t, nh * hd), lse


def _exact_value(code, scale, signed):
    """The numbers that 8-bit codes stand for, by their table."""
    table = [float(c) if c < 8 else (8.0 + c % 8) * 2.0 ** (c // 8 - 1) for c in range(128 if signed else 256)]
    table = torch.tensor(table + [-x for x in table] if signed else table, dtype=torch.float64, device="cuda")
    return table[code.long()] * scale.double().repeat_interleave(BLOCK)[: code.numel()]


def _exact_adamw(case, st):
    h, step = HYPER, st["step"]
    scale, out = st["grad_scale"].double(), {}
    if case["clip"]:
        out["norm"] = math.sqrt(sum(float(torch.sum(t["grad"].double() ** 2)) for t in st["tensors"]))
        scale = min(1.0, MAX_NORM / (out["norm"] + 1e-6))
        out["norm"] = torch.tensor(out["norm"], dtype=torch.float64)
    out["tensors"] = []
    for t in st["tensors"]:
        g = t["grad"].double() * scale
        if case["bits"] == 8:
            m, v = _exact_value(t["m"], t["m_scale"], True), _exact_value(t["v"], t["v_scale"], False)
        else:
            m, v = t["m"].double(), t["v"].double()
        m = h["beta1"] * m + (1.0 - h["beta1"]) * g
        v = h["beta2"] * v + (1.0 - h["beta2"]) * g ** 2
        p = (t["master"] if "master" in t else t["param"]).double()
        p = p - h["lr"] * t["decay"] * p
        p = p - h["lr"] * (m / (1.0 - h["beta1"] ** step)) / ((v / (1.0 - h["beta2"] ** step)) ** 0.5 + h["eps"])
        kept = {"m": None, "v": None} if case["bits"] == 8 else {"m": m, "v": v}
        out["tensors"].append(kept | {k: p for k in ("master", "param") if k in t})
    return out
