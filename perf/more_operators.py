"""Operators of a feed-forward block with biases, norms on both sides and an 8-bit stash: what is measured, and their plain forms.

Three families around the split backward of a stage:
  linear      y = act(x w^T + bias) + residual with its checkpoints; the activation's backward and the bias gradient
              behind the dgrad of the linear that follows
  checkpoint  activations in 8 bits (32 columns of a row share a power of two), and the weight gradient from them
  norm        h = a x + b gate * PostNorm(y) and n = PreNorm(h) in one pass; its input and its weight gradients

`own` false: plain torch forms in float32.  `own` true: the library's calls.
"""
import math
import random

import torch

own = False

ACTIVATIONS = ["none", "relu", "gelu", "gelu_tanh", "silu", "relu2"]

# Hidden and feed-forward sizes of the 8B-shaped and the 70B-shaped stage, and of the tests' tiny transformer.
LAYERS = {"8b": (4096, 14336), "70b": (8192, 28672), "tiny": (256, 512)}


def listed():
    f = dict(op="linear", bias=True, residual=False, act="gelu", z="packed", packed=True)
    b = dict(op="linear_bwd", act="gelu", z="packed", bias=True)
    n = dict(gate="none", post="rms", pre="rms", a=1.0, b=1.0, beta=False)
    h, ffn = LAYERS["8b"]
    wide = LAYERS["70b"][0]
    small, small_ffn = LAYERS["tiny"]
    return [
        # one 128-token microbatch of the tests' small layer: launch latency
        dict(f, name="linear_tiny", tokens=128, inner=small, outer=small_ffn, act="silu", z="bf16", packed=False),
        # the up projection of an 8B-shaped block: pre-activation and output kept in 8 bits
        dict(f, name="linear_up_8b", tokens=4096, inner=h, outer=ffn),
        # its down projection with the residual, on a microbatch off every tile boundary
        dict(f, name="linear_down_ragged", tokens=1000, inner=ffn, outer=h, act="none", residual=True, z="none", packed=False),
        # B through the down projection and the activation, from the 8-bit pre-activation, with the up projection's bias gradient
        dict(b, name="linear_bwd_8b", tokens=4096, inner=ffn, outer=h),
        # the same on a small ragged batch with the pre-activation in bf16
        dict(b, name="linear_bwd_small", tokens=333, inner=small_ffn, outer=small, act="gelu_tanh", z="bf16"),
        # packing the normed activations of a 70B-shaped layer, and back
        dict(op="pack", name="pack_70b", tokens=4096, width=wide),
        # the up projection's weight gradient from its 8-bit input; and a small ragged one
        dict(op="weight", name="weight_8b", tokens=4096, inner=h, outer=ffn),
        dict(op="weight", name="weight_small", tokens=700, inner=small_ffn, outer=small),
        # between two blocks of the 8B-shaped layer: post norm, gate per channel, residual scale, next pre norm, 8-bit output
        dict(n, op="norm", name="norm_8b", tokens=4096, width=h, gate="channel", a=1.0, b=0.5, packed=True),
        # the small layer with layer norms and a gate per token
        dict(n, op="norm", name="norm_tiny_layer", tokens=128, width=small, gate="token", post="layer", pre="layer", beta=True,
             packed=False),
        # its input gradients for a 70B-shaped layer on a ragged batch
        dict(n, op="norm_bwd", name="norm_bwd_70b", tokens=3333, width=wide, gate="channel", a=0.7, b=0.5),
        # and the weight gradients of the 8B-shaped one
        dict(n, op="norm_weight", name="norm_weight_8b", tokens=4096, width=h, gate="channel", post="layer", pre="layer",
             beta=True, b=0.5),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of lo .. hi."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear_bwd", "pack", "weight", "norm", "norm_bwd", "norm_weight"])
    if op in ("linear", "linear_bwd", "weight"):
        most = 4096 * 4096 * 14336
        inner, outer = (64 * _log(rng, 1, 224) for _ in range(2))
        case = dict(op=op, tokens=_log(rng, 1, max(1, min(8192, most // (inner * outer)))), inner=inner, outer=outer)
        if op != "weight":
            case.update(act=rng.choice(ACTIVATIONS), bias=rng.random() < 0.7, z=rng.choice(["bf16", "packed"]))
        if op == "linear":
            case.update(residual=rng.random() < 0.5, packed=rng.random() < 0.5, z=rng.choice(["none", "bf16", "packed"]))
        return case
    width = 64 * _log(rng, 1, 256)
    case = dict(op=op, tokens=_log(rng, 1, max(1, min(16384, 4096 * 8192 // width))), width=width)
    if op != "pack":
        case.update(gate=rng.choice(["none", "channel", "token"]), post=rng.choice(["none", "rms", "layer"]),
                    pre=rng.choice(["none", "rms", "layer"]), a=rng.choice([1.0, 1.0, 0.7]), b=rng.choice([1.0, 0.5]),
                    beta=rng.random() < 0.5)
        if op == "norm":
            case.update(packed=case["pre"] != "none" and rng.random() < 0.5)
        if op == "norm_weight" and case["post"] == case["pre"] == "none":  # something has to be learned
            case.update(gate="channel")
    return case


# ---------------------------------------------------------------- inputs

EPS = 1e-5


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    bf16 = lambda x: x.to(torch.bfloat16)  # noqa: E731
    st, t = {"case": case}, case["tokens"]
    if case["op"] == "pack":
        # normed activations: a few channels far larger than the others, as trained models have them
        st["x"] = bf16(normal(t, case["width"]) * (1.0 + 20.0 * (normal(case["width"]) > 2.5)))
        return st
    if case["op"] in ("norm", "norm_bwd", "norm_weight"):
        return _prepare_norm(case, st, normal, bf16)
    k, n = case["inner"], case["outer"]
    if case["op"] == "linear":
        st["x"], st["w"] = bf16(normal(t, k)), bf16(normal(n, k) * k ** -0.5)
        st["bias"] = normal(n) * 0.1 if case["bias"] else None
        st["residual"] = bf16(normal(t, n)) if case["residual"] else None
        return st
    if case["op"] == "linear_bwd":
        # w of the linear behind the activation: [out, in] = [outer, inner]; z: what the activation read, [tokens, inner]
        st["dy"], st["w"], st["z"] = bf16(normal(t, n)), bf16(normal(n, k) * k ** -0.5), bf16(normal(t, k))
        if case["z"] == "packed":
            st["z_packed"] = _pack(st["z"])
        st["dbias"] = normal(k) if case["bias"] else None  # the sum over earlier microbatches
        return st
    st["dy"], st["dw"] = bf16(normal(t, n)), normal(n, k)
    st["x_packed"] = _pack(bf16(normal(t, k)))
    return st


def _prepare_norm(case, st, normal, bf16):
    t, w = case["tokens"], case["width"]
    # a residual stream larger than the branch, and a branch with a mean
    st["x"], st["y"] = bf16(3.0 * normal(t, w)), bf16(normal(t, w) + 0.3)
    for k in ("post", "pre"):
        st[k + "_gamma"] = 1.0 + 0.1 * normal(w) if case[k] != "none" else None
        st[k + "_beta"] = 0.1 * normal(w) if case[k] == "layer" and case["beta"] else None
    st["gate"] = {"none": None, "channel": 0.3 + 0.1 * normal(w), "token": bf16(torch.sigmoid(normal(t, w)))}[case["gate"]]
    if case["op"] == "norm":
        return st
    out = _norm(st)
    st["h"], st["stats"] = out["h"], out["stats"]
    st["dn"] = bf16(normal(t, w)) if case["pre"] != "none" else None
    if case["op"] == "norm_bwd":
        st["dres"] = bf16(normal(t, w))
        return st
    st["dh"] = bf16(normal(t, w))
    for k in ("post", "pre"):  # the sums over earlier microbatches
        for p in ("_gamma", "_beta"):
            st["d" + k + p] = normal(w) if st[k + p] is not None else None
    st["dgate"] = normal(w) if case["gate"] == "channel" else None
    return st


# ---------------------------------------------------------------- plain forms


def _act(z, kind):
    if kind == "relu":
        return torch.where(z > 0.0, z, 0.0)
    if kind == "relu2":
        return torch.where(z > 0.0, z * z, 0.0)
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _slope(z, kind):
    """The activation's derivative."""
    if kind == "relu":
        return (z > 0.0).float()
    if kind == "relu2":
        return torch.where(z > 0.0, 2.0 * z, 0.0)
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) / (2.0 * math.pi) ** 0.5
    if kind == "gelu_tanh":
        c = (2.0 / math.pi) ** 0.5
        th = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _pack(x):
    """8-bit codes of a bf16 matrix [rows, width] and one scale byte per 32 columns: a sign and a magnitude up to 127,
    in units of the power of two that takes the block's largest value to 127 at most."""
    blocks = x.float().view(x.shape[0], -1, 32)
    top = blocks.abs().amax(2)
    fine = torch.isfinite(blocks).all(2)
    # the exponent of the largest value, carried to the next one where its magnitude would round to 128
    scale = ((torch.where(fine, top, 1.0).view(torch.int32) + 0x10000) >> 23) - 6
    scale = scale.clamp(1, 248)
    unit = ((254 - scale) << 23).view(torch.float32)  # 2^(127 - scale)
    code = torch.round(blocks.abs() * unit[..., None]).clamp(max=127.0).to(torch.int32)
    code = code | torch.where(torch.signbit(blocks), 128, 0)
    code = torch.where(fine[..., None], code, 0)
    scale = torch.where(fine, scale, 255)
    return code.to(torch.uint8).view(x.shape), scale.to(torch.uint8)


def _unpack(codes, scales):
    c = codes.view(codes.shape[0], -1, 32).to(torch.int32)
    s = scales.to(torch.int32)
    unit = torch.where(s == 255, math.nan, (s << 23).view(torch.float32))
    value = (c & 127).float() * unit[..., None]
    return torch.where(c > 127, -value, value).view(codes.shape)


def _linear(st):
    case = st["case"]
    z = torch.matmul(st["x"].float(), st["w"].float().T)
    if st["bias"] is not None:
        z = z + st["bias"]
    y = _act(z, case["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    out = {"y": y.to(torch.bfloat16)}
    if case["z"] != "none":
        z = z.to(torch.bfloat16)
        out["z"] = z if case["z"] == "bf16" else _unpack(*_pack(z)).to(torch.bfloat16)
    if case["packed"]:
        out["y_packed"] = _unpack(*_pack(out["y"])).to(torch.bfloat16)
    return out


def _linear_bwd(st):
    case = st["case"]
    z = _unpack(*st["z_packed"]) if case["z"] == "packed" else st["z"].float()
    dz = torch.matmul(st["dy"].float(), st["w"].float()) * _slope(z, case["act"])
    out = {"dz": dz.to(torch.bfloat16)}
    if case["bias"]:
        st["dbias"] = out["dbias"] = st["dbias"] + dz.sum(0)
    return out


def _weight(st):
    st["dw"] = st["dw"] + torch.matmul(st["dy"].float().T, _unpack(*st["x_packed"]))
    return st["dw"]


def _moments(x, kind):
    """(mean, 1 / sqrt(variance + eps)) of rows; an RMS norm's mean is 0."""
    mean = x.mean(1) if kind == "layer" else torch.zeros(x.shape[0], device=x.device)
    d = x - mean[:, None]
    return mean, 1.0 / torch.sqrt((d * d).mean(1) + EPS)


def _normed(x, mean, rstd):
    return (x - mean[:, None]) * rstd[:, None]


def _affine(x, gamma, beta):
    return x * gamma if beta is None else x * gamma + beta


def _norm(st):
    case = st["case"]
    x, u = st["x"].float(), st["y"].float()
    none = torch.zeros(x.shape[0], device=x.device)
    stats = [none, none, none, none]
    if case["post"] != "none":
        stats[:2] = _moments(u, case["post"])
        u = _affine(_normed(u, *stats[:2]), st["post_gamma"], st["post_beta"])
    if st["gate"] is not None:
        u = u * st["gate"].float()
    out = {"h": (case["a"] * x + case["b"] * u).to(torch.bfloat16)}
    if case["pre"] != "none":
        h = out["h"].float()
        stats[2:] = _moments(h, case["pre"])
        out["n"] = _affine(_normed(h, *stats[2:]), st["pre_gamma"], st["pre_beta"]).to(torch.bfloat16)
        if case.get("packed"):
            out["n_packed"] = _unpack(*_pack(out["n"])).to(torch.bfloat16)
    out["stats"] = torch.stack(stats, 1)
    return out


def _norm_slope(d, xh, rstd, kind):
    """The input gradient of a norm: d is the gradient of its normed rows xh."""
    back = d - xh * (d * xh).mean(1, keepdim=True)
    if kind == "layer":
        back = back - d.mean(1, keepdim=True)
    return back * rstd[:, None]


def _norm_bwd(st):
    case, s = st["case"], st["stats"]
    dh = st["dres"].float()
    if case["pre"] != "none":
        hh = _normed(st["h"].float(), s[:, 2], s[:, 3])
        dh = dh + _norm_slope(st["dn"].float() * st["pre_gamma"], hh, s[:, 3], case["pre"])
    out = {"dh": dh.to(torch.bfloat16)}
    if case["a"] != 1.0:
        out["dx"] = (case["a"] * dh).to(torch.bfloat16)
    u = st["y"].float()
    if case["post"] != "none":
        yh = _normed(u, s[:, 0], s[:, 1])
        u = _affine(yh, st["post_gamma"], st["post_beta"])
    if case["gate"] == "token":
        out["dgate"] = (case["b"] * dh * u).to(torch.bfloat16)
    du = case["b"] * dh if st["gate"] is None else case["b"] * st["gate"].float() * dh
    if case["post"] != "none":
        du = _norm_slope(du * st["post_gamma"], yh, s[:, 1], case["post"])
    out["dy"] = du.to(torch.bfloat16)
    return out


NORM_GRADS = ("dpost_gamma", "dpost_beta", "dpre_gamma", "dpre_beta", "dgate")


def _norm_weight(st):
    case, s = st["case"], st["stats"]
    add = {}
    if case["pre"] != "none":
        dn = st["dn"].float()
        add["dpre_gamma"] = (dn * _normed(st["h"].float(), s[:, 2], s[:, 3])).sum(0)
        add["dpre_beta"] = dn.sum(0)
    u, du = st["y"].float(), case["b"] * st["dh"].float()
    if case["post"] != "none":
        yh = _normed(u, s[:, 0], s[:, 1])
        u = _affine(yh, st["post_gamma"], st["post_beta"])
        gated = du if st["gate"] is None else du * st["gate"].float()
        add["dpost_gamma"] = (gated * yh).sum(0)
        add["dpost_beta"] = gated.sum(0)
    if case["gate"] == "channel":
        add["dgate"] = (du * u).sum(0)
    for k in NORM_GRADS:
        if st[k] is not None:
            st[k] = st[k] + add[k]
    return {k: st[k] for k in NORM_GRADS if st[k] is not None}


# ---------------------------------------------------------------- the library's calls


def _empty(st, name, *shape, dtype=torch.bfloat16):
    """A buffer that the program keeps; its contents are written in every pass."""
    if name not in st:
        st[name] = torch.empty(*shape, dtype=dtype, device="cuda")
    return st[name]


def _packed(st, name, t, width):
    return (_empty(st, name + "_codes", t, width, dtype=torch.uint8),
            _empty(st, name + "_scales", t, width // 32, dtype=torch.uint8))


def _values(zb, st, name, packed):
    """What 8-bit codes stand for."""
    t, width = packed[0].shape
    out = _empty(st, name + "_values", t, width)
    zb.zb_op_checkpoint_unpack(packed, out, t, width)
    return out


def _own_linear(st):
    from backward_split_linear_gb300 import binding as zb

    case = st["case"]
    t, k, n = case["tokens"], case["inner"], case["outer"]
    out = {"y": _empty(st, "out", t, n)}
    z = _empty(st, "z_out", t, n) if case["z"] == "bf16" else None
    z8 = _packed(st, "z", t, n) if case["z"] == "packed" else None
    y8 = _packed(st, "y", t, n) if case["packed"] else None
    zb.zb_op_linear_activation_forward(st["x"], st["w"], st["bias"], st["residual"], out["y"], t, k, n, case["act"], z=z,
                                       z_packed=z8, y_packed=y8)
    if z is not None:
        out["z"] = z
    if z8 is not None:
        out["z"] = _values(zb, st, "z", z8)
    if y8 is not None:
        out["y_packed"] = _values(zb, st, "y", y8)
    return out


def _own_linear_bwd(st):
    from backward_split_linear_gb300 import binding as zb

    case = st["case"]
    t, k, n = case["tokens"], case["inner"], case["outer"]
    out = {"dz": _empty(st, "dz", t, k)}
    size = zb.zb_op_backward_input_activation_scratch_bytes(t, k)
    scratch = _empty(st, "scratch", max(16, size), dtype=torch.uint8)
    zb.zb_op_backward_input_activation(st["dy"], st["w"], None if case["z"] == "packed" else st["z"], out["dz"], t, k, n,
                                       case["act"], z_packed=st.get("z_packed"), dbias=st["dbias"], scratch=scratch)
    if case["bias"]:
        out["dbias"] = st["dbias"]
    return out


def _own_pack(st):
    from backward_split_linear_gb300 import binding as zb

    t, width = st["x"].shape
    packed = _packed(st, "x", t, width)
    zb.zb_op_checkpoint_pack(st["x"], packed, t, width)
    return _values(zb, st, "x", packed)


def _own_weight(st):
    from backward_split_linear_gb300 import binding as zb

    case = st["case"]
    t, k, n = case["tokens"], case["inner"], case["outer"]
    scratch = _empty(st, "scratch", zb.zb_op_backward_weight_checkpoint_scratch_bytes(t, k), dtype=torch.uint8)
    zb.zb_op_backward_weight_checkpoint(st["dy"], st["x_packed"], st["dw"], t, k, n, scratch)
    return st["dw"]


def _norm_op(zb, st):
    if "norm" not in st:  # the options that the program keeps beside its parameters
        case = st["case"]
        st["norm"] = zb.make_residual_norm(post=case["post"], pre=case["pre"], gate_kind=case["gate"], gate=st["gate"],
                                           post_gamma=st["post_gamma"], post_beta=st["post_beta"], pre_gamma=st["pre_gamma"],
                                           pre_beta=st["pre_beta"], residual_scale=case["a"], branch_scale=case["b"],
                                           post_eps=EPS, pre_eps=EPS)
    return st["norm"]


def _own_norm(st):
    from backward_split_linear_gb300 import binding as zb

    case = st["case"]
    t, w = case["tokens"], case["width"]
    out = {"h": _empty(st, "h", t, w), "stats": _empty(st, "stats", t, 4, dtype=torch.float32)}
    packed = None
    if case["pre"] != "none":
        out["n"] = _empty(st, "n", t, w)
        packed = _packed(st, "n", t, w) if case["packed"] else None
    zb.zb_op_residual_norm_forward(_norm_op(zb, st), st["x"], st["y"], out["h"], out.get("n"), out["stats"], t, w, n_packed=packed)
    if packed is not None:
        out["n_packed"] = _values(zb, st, "n", packed)
    return out


def _own_norm_bwd(st):
    from backward_split_linear_gb300 import binding as zb

    case = st["case"]
    t, w = case["tokens"], case["width"]
    out = {"dh": _empty(st, "dh", t, w), "dy": _empty(st, "dy", t, w)}
    if case["a"] != 1.0:
        out["dx"] = _empty(st, "dx", t, w)
    if case["gate"] == "token":
        out["dgate"] = _empty(st, "dgate", t, w)
    zb.zb_op_residual_norm_backward_input(_norm_op(zb, st), st["dn"], st["dres"], st["h"], st["y"], st["stats"], out["dh"],
                                          out["dy"], t, w, dx=out.get("dx"), dgate=out.get("dgate"))
    return out


def _own_norm_weight(st):
    from backward_split_linear_gb300 import binding as zb

    case = st["case"]
    t, w = case["tokens"], case["width"]
    scratch = _empty(st, "scratch", zb.zb_op_residual_norm_backward_weight_scratch_bytes(t, w), dtype=torch.uint8)
    zb.zb_op_residual_norm_backward_weight(_norm_op(zb, st), st["dn"], st["h"], st["dh"], st["y"], st["stats"], t, w, scratch,
                                           **{k: st[k] for k in NORM_GRADS})
    return {k: st[k] for k in NORM_GRADS if st[k] is not None}


def run(st):
    op = st["case"]["op"]
    if own:
        return {"linear": _own_linear, "linear_bwd": _own_linear_bwd, "pack": _own_pack, "weight": _own_weight,
                "norm": _own_norm, "norm_bwd": _own_norm_bwd, "norm_weight": _own_norm_weight}[op](st)
    if op == "pack":
        return _unpack(*_pack(st["x"])).to(torch.bfloat16)
    return {"linear": _linear, "linear_bwd": _linear_bwd, "weight": _weight, "norm": _norm, "norm_bwd": _norm_bwd,
            "norm_weight": _norm_weight}[op](st)


# ---------------------------------------------------------------- work and the definition in 64 bits

PACKED = 1.0 + 1.0 / 32.0  # bytes of an 8-bit value and its share of a scale


def work(case):
    t = case["tokens"]
    if case["op"] in ("linear", "linear_bwd", "weight"):
        k, n = case["inner"], case["outer"]
        flops = 2.0 * t * k * n
        if case["op"] == "weight":
            return {"bytes": 2.0 * t * n + PACKED * t * k + 8.0 * k * n, "flops": flops}
        if case["op"] == "linear":
            # 8-bit outputs are written as codes; the values that come back for them are not counted
            per = 2.0 + (2.0 if case["residual"] else 0.0) + (PACKED if case["packed"] else 0.0)
            per += {"none": 0.0, "bf16": 2.0, "packed": PACKED}[case["z"]]
            return {"bytes": 2.0 * t * k + 2.0 * k * n + 4.0 * n * case["bias"] + per * t * n, "flops": flops}
        per = 2.0 + (2.0 if case["z"] == "bf16" else PACKED)
        return {"bytes": 2.0 * t * n + 2.0 * k * n + per * t * k + 8.0 * k * case["bias"], "flops": flops}
    w = case["width"]
    if case["op"] == "pack":  # codes out, codes in, values out
        return {"bytes": (2.0 + 2.0 * PACKED + 2.0) * t * w, "flops": 4.0 * t * w}
    pre, token = case["pre"] != "none", case["gate"] == "token"
    if case["op"] == "norm":
        per = 6.0 + 2.0 * pre + (PACKED if case["packed"] else 0.0) + 2.0 * token
        return {"bytes": per * t * w + 16.0 * t, "flops": 16.0 * t * w}
    if case["op"] == "norm_bwd":
        per = 2.0 + 4.0 * pre + 4.0 + 2.0 * (case["post"] != "none" or token) + 4.0 * token + 2.0 * (case["a"] != 1.0)
        return {"bytes": per * t * w + 16.0 * t, "flops": 24.0 * t * w}
    branch = case["post"] != "none" or case["gate"] == "channel"
    per = 4.0 * pre + 4.0 * branch + 2.0 * (token and case["post"] != "none")
    return {"bytes": per * t * w + 16.0 * t, "flops": 8.0 * t * w}


def exact(case, seed):
    st = prepare(case, seed)
    return {"linear": _exact_linear, "linear_bwd": _exact_linear_bwd, "pack": lambda c, s: _exact_packed(s["x"].double()),
            "weight": _exact_weight, "norm": _exact_norm, "norm_bwd": _exact_norm_bwd,
            "norm_weight": _exact_norm_weight}[case["op"]](case, st)


def _exact_act(z, kind):
    if kind == "none":
        return z * 1.0
    if kind in ("relu", "relu2"):
        return torch.clamp(z, min=0.0) ** (1 if kind == "relu" else 2)
    if kind == "gelu":
        return z * torch.special.ndtr(z)
    return z * torch.sigmoid(z if kind == "silu" else 8.0 ** 0.5 * math.pi ** -0.5 * (z + 0.044715 * z ** 3))


def _rounded(x):
    return x.to(torch.bfloat16).double()


def _exact_packed(x):
    """The values that the 8-bit codes of bf16 numbers stand for: multiples of the smallest power of two (2^-126 at
    least) of which 127 reach the block's largest value, or that times 127.5 is above it."""
    b = x.view(x.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -126))) - 6.0)
    unit = torch.where(top >= 127.5 * unit, 2.0 * unit, unit).clamp(2.0 ** -126, 2.0 ** 121)
    return ((b / unit).round().clamp(-127.0, 127.0) * unit).view(x.shape)


def _exact_linear(case, st):
    z = st["x"].double() @ st["w"].double().T
    if st["bias"] is not None:
        z += st["bias"].double()
    y = _exact_act(z, case["act"])
    if st["residual"] is not None:
        y = y + st["residual"].double()
    out = {"y": y}
    if case["z"] != "none":
        out["z"] = z if case["z"] == "bf16" else _exact_packed(_rounded(z))
    if case["packed"]:
        out["y_packed"] = _exact_packed(_rounded(y))
    return out


def _exact_value(packed):
    """The numbers that 8-bit codes stand for, by their table."""
    codes, scales = packed
    table = torch.arange(128, dtype=torch.float64, device="cuda")
    table = torch.cat([table, -table])
    return table[codes.long()] * torch.exp2(scales.double() - 127.0).repeat_interleave(32, 1)


def _exact_linear_bwd(case, st):
    z = _exact_value(st["z_packed"]) if case["z"] == "packed" else st["z"].double()
    z.requires_grad_(True)
    (dz,) = torch.autograd.grad(_exact_act(z, case["act"]), z, st["dy"].double() @ st["w"].double())
    return {"dz": dz, "dbias": st["dbias"].double() + dz.sum(0)} if case["bias"] else {"dz": dz}


def _exact_weight(case, st):
    return torch.addmm(st["dw"].double(), st["dy"].double().T, _exact_value(st["x_packed"]))


def _exact_norm_of(x, kind, gamma, beta, stats=None):
    """A norm of rows and its moments."""
    if kind == "none":
        return x, [torch.zeros(x.shape[0], dtype=x.dtype, device="cuda")] * 2
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    rstd = ((x - mean).square().mean(1, keepdim=True) + EPS) ** -0.5
    y = (x - mean) * rstd * gamma
    return y if beta is None else y + beta, [mean[:, 0], rstd[:, 0]]


def _doubles(st):
    return {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in st.items()}


def _exact_norm(case, st):
    d = _doubles(st)
    u, s1 = _exact_norm_of(d["y"], case["post"], d["post_gamma"], d["post_beta"])
    h = case["a"] * d["x"] + case["b"] * (u if d["gate"] is None else u * d["gate"])
    out = {"h": h}
    n, s2 = _exact_norm_of(_rounded(h), case["pre"], d["pre_gamma"], d["pre_beta"])
    if case["pre"] != "none":
        out["n"] = n
        if case["packed"]:
            out["n_packed"] = _exact_packed(_rounded(n))
    out["stats"] = torch.stack(s1 + s2, 1)
    return out


def _exact_norm_bwd(case, st):
    """By differentiation in 64 bits."""
    d = _doubles(st)
    dh = d["dres"]
    if case["pre"] != "none":
        h = d["h"].requires_grad_(True)
        n, _ = _exact_norm_of(h, case["pre"], d["pre_gamma"], d["pre_beta"])
        dh = dh + torch.autograd.grad(n, h, d["dn"])[0]
    out = {"dh": dh}
    if case["a"] != 1.0:
        out["dx"] = case["a"] * dh
    y = d["y"].requires_grad_(True)
    u, _ = _exact_norm_of(y, case["post"], d["post_gamma"], d["post_beta"])
    gate = torch.ones_like(u) if d["gate"] is None else d["gate"].expand_as(u).clone()
    gate.requires_grad_(True)
    out["dy"], dgate = torch.autograd.grad(case["b"] * gate * u, [y, gate], dh)
    if case["gate"] == "token":
        out["dgate"] = dgate
    return out


def _exact_norm_weight(case, st):
    d = _doubles(st)
    known = [k for k in NORM_GRADS if st[k] is not None]
    for k in known:
        d[k[1:]] = d[k[1:]].requires_grad_(True)
    total = 0.0
    if case["pre"] != "none":
        total = (_exact_norm_of(d["h"], case["pre"], d["pre_gamma"], d["pre_beta"])[0] * d["dn"]).sum()
    u, _ = _exact_norm_of(d["y"], case["post"], d["post_gamma"], d["post_beta"])
    total = total + (case["b"] * (u if d["gate"] is None else u * d["gate"]) * d["dh"]).sum()
    return {k: d[k] + g for k, g in zip(known, torch.autograd.grad(total, [d[k[1:]] for k in known]))}
