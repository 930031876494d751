"""The feed-forward block's operators without a GPU: refusals, and the oracle's own identities."""
import ctypes

import numpy as np
import pytest

from backward_split_linear_gb300 import binding as zb
from oracle import block_ops as O
from parity import draw_bf16

FAKE = 1 << 20  # never dereferenced: the calls below fail their checks before any device call
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu", "relu2"]


def ckpt(codes=FAKE, scales=FAKE):
    return ctypes.byref(zb.zb_checkpoint(codes, scales))


# ---------------------------------------------------------------- refusals


def test_linear_refusals(zblib):
    def forward(**kw):
        a = {**dict(x=FAKE, w=FAKE, bias=FAKE, res=FAKE, y=2 * FAKE, z=None, z8=None, y8=None, t=8, k=64, n=64, act=2), **kw}
        return zblib.zb_op_linear_activation_forward(a["x"], a["w"], a["bias"], a["res"], a["y"], a["z"], a["z8"], a["y8"],
                                                     a["t"], a["k"], a["n"], a["act"], None)

    for kw in (dict(t=-1), dict(t=(1 << 24) + 1), dict(k=0), dict(k=96), dict(n=32), dict(n=-64), dict(n=(1 << 20) + 64)):
        assert forward(**kw) == -2, kw
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(x=FAKE + 2), dict(bias=FAKE + 4), dict(res=FAKE + 8), dict(act=-1),
               dict(act=6), dict(z=FAKE + 2), dict(z=FAKE, z8=ckpt()), dict(z8=ckpt(codes=None)), dict(y8=ckpt(scales=None)),
               dict(y8=ckpt(codes=FAKE + 4))):
        assert forward(**kw) == -1, kw

    def backward(**kw):
        a = {**dict(dy=FAKE, w=FAKE, z=FAKE, z8=None, dz=FAKE, db=None, t=8, k=64, n=64, act=2, s=FAKE, sb=1 << 20), **kw}
        return zblib.zb_op_backward_input_activation(a["dy"], a["w"], a["z"], a["z8"], a["dz"], a["db"], a["t"], a["k"], a["n"],
                                                     a["act"], a["s"], a["sb"], None)

    for kw in (dict(t=-1), dict(k=32), dict(n=100)):
        assert backward(**kw) == -2, kw
    for kw in (dict(dy=None), dict(w=FAKE + 2), dict(z=None), dict(z=FAKE, z8=ckpt()), dict(dz=None), dict(act=9),
               dict(z=None, z8=ckpt(scales=FAKE + 1)), dict(db=FAKE + 4)):
        assert backward(**kw) == -1, kw
    size = zb.zb_op_backward_input_activation_scratch_bytes(8, 64)
    assert size == 64 * 4
    for kw in (dict(s=None), dict(sb=size - 1), dict(s=FAKE + 4)):
        assert backward(db=FAKE, **kw) == -10, kw
    assert zb.zb_op_backward_input_activation_scratch_bytes(33, 128) == 2 * 128 * 4
    assert zb.zb_op_backward_input_activation_scratch_bytes(-1, 64) == 0


def test_activation_bias_and_checkpoint_refusals(zblib):
    act = zblib.zb_op_activation_backward
    assert act(FAKE, FAKE, None, FAKE, 8, 96, 2, None) == -2
    assert act(FAKE, None, None, FAKE, 8, 64, 2, None) == -1
    assert act(FAKE, FAKE, ckpt(), FAKE, 8, 64, 2, None) == -1
    assert act(None, FAKE, None, FAKE, 8, 64, 2, None) == -1
    bias = zblib.zb_op_backward_bias
    assert bias(FAKE, FAKE, 8, 65, FAKE, 1 << 20, None) == -2
    assert bias(FAKE, None, 8, 64, FAKE, 1 << 20, None) == -1
    assert bias(FAKE, FAKE, 8, 64, None, 1 << 20, None) == -10
    assert bias(FAKE, FAKE, 8, 64, FAKE, zb.zb_op_backward_bias_scratch_bytes(8, 64) - 1, None) == -10
    for call in (lambda x, c, t, w: zblib.zb_op_checkpoint_pack(x, c, t, w, None),
                 lambda x, c, t, w: zblib.zb_op_checkpoint_unpack(c, x, t, w, None)):
        assert call(FAKE, ckpt(), 8, 80) == -2
        assert call(FAKE, ckpt(), -8, 64) == -2
        assert call(FAKE, None, 8, 64) == -1
        assert call(None, ckpt(), 8, 64) == -1
        assert call(FAKE, ckpt(codes=FAKE + 8), 8, 64) == -1
        assert call(FAKE, ckpt(scales=None), 8, 64) == -1
    weight = zblib.zb_op_backward_weight_checkpoint
    need = zb.zb_op_backward_weight_checkpoint_scratch_bytes(8, 64)
    assert need >= 8 * 64 * 2
    assert weight(FAKE, ckpt(), FAKE, 8, 63, 64, FAKE, need, None) == -2
    assert weight(FAKE, None, FAKE, 8, 64, 64, FAKE, need, None) == -1
    assert weight(FAKE, ckpt(), None, 8, 64, 64, FAKE, need, None) == -1
    assert weight(FAKE, ckpt(), FAKE, 8, 64, 64, FAKE, need - 1, None) == -10
    assert weight(FAKE, ckpt(), FAKE, 8, 64, 64, None, need, None) == -10


def norm_op(**kw):
    a = dict(post="rms", pre="layer", gate_kind="channel", gate=FAKE, post_gamma=FAKE, pre_gamma=FAKE, pre_beta=FAKE)
    return zb.make_residual_norm(**{**a, **kw})


def test_residual_norm_refusals(zblib):
    def refused(code, fn, *args, **kw):
        with pytest.raises(zb.ZBError) as e:
            fn(*args, **kw)
        assert e.value.status == code, (args, kw)

    def forward(op=None, x=FAKE, y=FAKE, h=FAKE, n=FAKE, stats=FAKE, t=8, w=64, **kw):
        zb.zb_op_residual_norm_forward(op or norm_op(), x, y, h, n, stats, t, w, stream=0, **kw)

    for kw in (dict(t=-1), dict(w=96), dict(w=32768 + 64), dict(w=0)):
        refused(-2, forward, **kw)
    for kw in (dict(x=None), dict(y=FAKE + 2), dict(h=None), dict(n=None), dict(stats=None), dict(n=FAKE + 4),
               dict(n_packed=(FAKE, None)), dict(op=norm_op(pre="none", pre_gamma=None, pre_beta=None)),
               dict(op=norm_op(post_gamma=None)), dict(op=norm_op(post_beta=FAKE)), dict(op=norm_op(pre_eps=-1.0)),
               dict(op=norm_op(pre_eps=float("nan"))), dict(op=norm_op(gate=None)), dict(op=norm_op(gate_kind="none")),
               dict(op=norm_op(gate_kind="token", gate=None)), dict(op=norm_op(residual_scale=float("inf"))),
               dict(op=norm_op(branch_scale=float("nan"))), dict(op=norm_op(post="none"))):
        refused(-1, forward, **kw)
    bad = norm_op()
    bad.post_norm = 3
    refused(-1, forward, op=bad)

    def backward(op=None, dn=FAKE, dres=FAKE, h=FAKE, y=FAKE, stats=FAKE, dh=FAKE, dy=FAKE, t=8, w=64, **kw):
        zb.zb_op_residual_norm_backward_input(op or norm_op(), dn, dres, h, y, stats, dh, dy, t, w, stream=0, **kw)

    bare = dict(op=norm_op(pre="none", pre_gamma=None, pre_beta=None))
    for kw in (dict(dn=None), dict(h=None), dict(y=None), dict(dh=None), dict(dy=None), dict(stats=None), dict(dgate=FAKE),
               dict(dx=FAKE + 2), bare, dict(bare, dn=None, dres=None)):
        refused(-1, backward, **kw)
    refused(-2, backward, w=100)

    def weight(op=None, dn=FAKE, h=FAKE, dh=FAKE, y=FAKE, stats=FAKE, t=8, w=64, scratch=FAKE, scratch_bytes=1 << 20, **kw):
        zb.zb_op_residual_norm_backward_weight(op or norm_op(), dn, h, dh, y, stats, t, w, scratch, scratch_bytes, stream=0, **kw)

    for kw in (dict(dpost_beta=FAKE), dict(dpre_gamma=FAKE, dn=None), dict(dgate=FAKE, y=None), dict(dgate=FAKE + 4),
               dict(dgate=FAKE, op=norm_op(gate_kind="token")), dict(dpre_beta=FAKE, stats=None)):
        refused(-1, weight, **kw)
    need = zb.zb_op_residual_norm_backward_weight_scratch_bytes(8, 64)
    refused(-10, weight, dgate=FAKE, scratch_bytes=need - 1)
    refused(-10, weight, dgate=FAKE, scratch=None)
    assert zb.zb_op_residual_norm_backward_weight_scratch_bytes(8, 40000 // 64 * 64) == 0


def test_residual_norm_weight_takes_what_its_gradients_read(zblib):
    """A beta's gradient reads neither h nor y: the call gets past the checks of its arguments (and ends at the device's, or
    at the scratch)."""
    def status(**kw):
        a = {**dict(dn=FAKE, h=FAKE, dh=FAKE, y=FAKE), **{k: kw.pop(k) for k in ("dn", "h", "dh", "y") if k in kw}}
        with pytest.raises(zb.ZBError) as e:
            zb.zb_op_residual_norm_backward_weight(norm_op(post="layer", post_beta=FAKE), a["dn"], a["h"], a["dh"], a["y"], FAKE, 8, 64,
                                                   None, 0, stream=0, **kw)
        return e.value.status

    for kw in (dict(dpre_beta=FAKE, h=None, dh=None, y=None), dict(dpost_beta=FAKE, dn=None, h=None, y=None),
               dict(dgate=FAKE, dn=None, h=None), dict(dpre_gamma=FAKE, dh=None, y=None),
               dict(dpre_beta=FAKE, dpost_gamma=FAKE, h=None), dict(dpre_gamma=FAKE, dpost_beta=FAKE, y=None)):
        assert status(**kw) == -10, kw
    for kw in (dict(dpre_beta=FAKE, dn=None), dict(dpre_gamma=FAKE, h=None), dict(dpost_beta=FAKE, dh=None),
               dict(dpost_gamma=FAKE, y=None), dict(dgate=FAKE, y=None)):
        assert status(**kw) == -1, kw


def test_residual_norm_takes_every_finite_scale(zblib):
    largest = float(np.finfo(np.float32).max)
    for kw in (dict(residual_scale=largest), dict(branch_scale=-largest)):
        op = norm_op(**kw)  # W without a scratch: the options are checked ahead of it
        with pytest.raises(zb.ZBError) as e:
            zb.zb_op_residual_norm_backward_weight(op, FAKE, FAKE, FAKE, FAKE, FAKE, 8, 64, None, 0, dpre_gamma=FAKE, stream=0)
        assert e.value.status == -10, kw


# ---------------------------------------------------------------- the oracle


@pytest.mark.parametrize("kind", ACTS)
def test_slopes_are_the_differences_of_the_activations(kind):
    z = np.linspace(-7.0, 7.0, 113) + 0.0131  # off the corners
    d = 1e-5
    np.testing.assert_allclose(O.act_slope(z, kind), (O.act(z + d, kind) - O.act(z - d, kind)) / (2 * d), atol=1e-8)


def test_activations_in_closed_form():
    z = np.array([-3.0, 0.0, 3.0])
    for kind in ACTS[1:]:
        assert O.act(z, kind)[1] == 0.0
    for kind in ("gelu", "gelu_tanh", "silu"):  # act(z) - act(-z) = z
        np.testing.assert_allclose(O.act(z, kind) - O.act(-z, kind), z, atol=1e-15)
    assert O.act(z, "relu2")[2] == 9.0


def test_packed_values():
    _, x = draw_bf16(np.random.default_rng(0), (5, 128))
    x[0, :32] = 0.0
    x[1, 3] = np.inf
    x[2, 40:70] *= 2.0 ** 100
    x[3, :32] = 127.5                      # would round to 128 units: one scale up
    x[4, 0:32] = 127.5 * 2.0 ** 121        # the largest bf16 number
    x[4, 32:64] = 2.0 ** -133              # the smallest
    codes, scales = O.pack(x)
    v = O.unpack(codes, scales)
    unit = np.repeat(2.0 ** (scales.astype(np.float64) - 127.0), 32, axis=1)
    hole = np.repeat(scales == 255, 32, axis=1)
    assert hole[1, :32].all() and hole.sum() == 32 and np.isnan(v[hole]).all()
    assert np.all(np.abs(v - np.where(hole, 0.0, x))[~hole] <= 0.5 * unit[~hole])
    assert scales[0, 0] == 1 and scales[3, 0] == 128 and scales[4, 0] == 248 and scales[4, 1] == 1
    assert np.all((codes & 127)[4, :32] == 127)
    # the values are bf16 numbers: packing them again changes nothing
    again = O.unpack(*O.pack(np.where(hole, 0.0, v)))
    assert np.array_equal(again[~hole], v[~hole])


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post,pre", [("rms", "layer"), ("layer", "rms"), ("none", "layer"), ("rms", "none")])
def test_norm_gradients_are_differences(post, pre, gate):
    rng = np.random.default_rng(3)
    t, w = 3, 8
    draw = lambda *s: rng.standard_normal(s)  # noqa: E731
    par = dict(gate={"none": None, "channel": draw(w), "token": draw(t, w)}[gate])
    for k, kind in (("post", post), ("pre", pre)):
        par[k + "_gamma"] = None if kind == "none" else 1.0 + 0.3 * draw(w)
        par[k + "_beta"] = draw(w) if kind == "layer" else None
    x, y = draw(t, w), draw(t, w)
    cn, ch = draw(t, w), draw(t, w)  # the loss is <n, cn> + <h, ch>

    def loss(x=x, y=y, **kw):
        op = O.ResidualNorm(post, pre, a=0.7, b=0.4, **{**par, **kw})
        h = op.h(x, y)
        return np.sum(h * ch) + (np.sum(op.n(h) * cn) if pre != "none" else 0.0)

    op = O.ResidualNorm(post, pre, a=0.7, b=0.4, **par)
    got = op.backward(cn if pre != "none" else None, ch, op.h(x, y), y)
    named = {"dx": ("x", x), "dy": ("y", y)}
    named.update({"d" + k: (k, v) for k, v in par.items() if v is not None})
    for name, (arg, value) in named.items():
        g = got[name] if name != "dgate" or gate == "token" else got[name].sum(0)
        for _ in range(4):
            d = rng.standard_normal(value.shape)
            e = 1e-5
            diff = (loss(**{arg: value + e * d}) - loss(**{arg: value - e * d})) / (2 * e)
            np.testing.assert_allclose(np.sum(g * d), diff, rtol=1e-6, atol=1e-8, err_msg=name)
