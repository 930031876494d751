"""The training operators without a GPU: refusals, the frequency tables, and the oracle's own identities."""
import ctypes

import numpy as np
import pytest
import torch

from backward_split_linear_gb300 import binding as zb
from backward_split_linear_gb300.runtime import AdamW
from oracle import train_ops as O

FAKE = 1 << 20  # never dereferenced: the calls below fail their checks before any device call


def refused(name, fn, *args, **kw):
    with pytest.raises(zb.ZBError) as e:
        fn(*args, **kw)
    assert e.value.name == name


# ---------------------------------------------------------------- rotary


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
                                dict(scaling="yarn", factor=8.0, context=8192.0),
                                dict(scaling="banded", factor=8.0, context=8192.0, low=1.0, high=4.0)])
@pytest.mark.parametrize("rot,base", [(16, 10000.0), (64, 500000.0), (128, 10000.0), (1024, 10.0)])
def test_frequencies_equal_the_definitions(zblib, rot, base, kw):
    turns, g = zb.zb_rotary_frequencies(rot, base, **kw)
    f, g_ref = O.rotary_frequencies(rot, base, **kw)
    # a handful of float64 roundings (pow, the ramp) on either side, and half a unit of the 64-bit fraction
    np.testing.assert_allclose(np.array([t / 2.0 ** 64 for t in turns]), f / (2.0 * np.pi), rtol=64 * 2.0 ** -53,
                               atol=2.0 ** -65)
    assert abs(g - g_ref) <= 2.0 ** -24 * g_ref


def test_frequency_refusals(zblib):
    refused("ZB_ERR_SHAPE", zb.zb_rotary_frequencies, 24)
    refused("ZB_ERR_SHAPE", zb.zb_rotary_frequencies, 0)
    refused("ZB_ERR_SHAPE", zb.zb_rotary_frequencies, 1040)
    refused("ZB_ERR_ARG", zb.zb_rotary_frequencies, 64, 1.0)
    refused("ZB_ERR_ARG", zb.zb_rotary_frequencies, 64, float("nan"))
    refused("ZB_ERR_ARG", zb.zb_rotary_frequencies, 64, scaling="linear", factor=0.5)
    refused("ZB_ERR_ARG", zb.zb_rotary_frequencies, 64, scaling="yarn", factor=2.0)               # no context
    refused("ZB_ERR_ARG", zb.zb_rotary_frequencies, 64, scaling="banded", factor=2.0, context=8.0, low=4.0, high=4.0)
    bad = zb.zb_rotary_config(9, 64, 10000.0, 1.0, 0.0, 1.0, 4.0)
    out, mag = (ctypes.c_uint64 * 32)(), ctypes.c_float()
    assert zblib.zb_rotary_frequencies(ctypes.byref(bad), out, ctypes.byref(mag)) == -1


@pytest.mark.parametrize("op", ["zb_op_rotary_forward", "zb_op_rotary_backward"])
def test_rotary_refusals(zblib, op):
    ok = dict(x=FAKE, ld=128, y=2 * FAKE, ldy=128, pos=FAKE, turns=FAKE, mag=1.0, t=8, n=2, d=64, rot=64, pairs=0)

    def call(**kw):
        a = {**ok, **kw}
        return getattr(zblib, op)(a["x"], a["ld"], a["y"], a["ldy"], a["pos"], a["turns"], a["mag"], a["t"], a["n"], a["d"],
                                  a["rot"], a["pairs"], None)

    for kw in (dict(rot=8), dict(rot=24), dict(rot=80), dict(t=-1), dict(t=(1 << 24) + 1), dict(n=0), dict(d=60), dict(n=3, d=8),
               dict(ld=120), dict(ldy=132), dict(ld=64), dict(n=1 << 30), dict(n=1, d=2048, rot=2048, ld=2048, ldy=2048)):
        assert call(**kw) == -2, kw
    for kw in (dict(x=None), dict(y=None), dict(x=FAKE + 2), dict(pos=FAKE + 2), dict(turns=None), dict(pairs=2),
               dict(mag=float("nan")), dict(mag=float("inf")), dict(y=FAKE, ldy=192)):
        assert call(**kw) == -1, kw


def test_oracle_rotary_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((9, 2, 32))
    f, g = O.rotary_frequencies(16)
    for pairs in ("half", "interleaved"):
        y = O.rotary(x, np.arange(9) + 100, f, g, pairs)
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-12)
        np.testing.assert_allclose(O.rotary(y, np.arange(9) + 100, f, g, pairs, backward=True), x, atol=1e-12)
        # scores depend on the difference of positions alone
        z = O.rotary(x, np.arange(9) + 7, f, g, pairs)
        np.testing.assert_allclose(y[3, 0] @ y[8, 1], z[3, 0] @ z[8, 1], atol=1e-10)


# ---------------------------------------------------------------- AdamW


def tensors(n=300, bits=32, **kw):
    t = {"param": torch.zeros(n, dtype=torch.bfloat16), "grad": torch.zeros(n), "master": torch.zeros(n)}
    kind = torch.uint8 if bits == 8 else torch.float32
    t.update(m=torch.zeros(n, dtype=kind), v=torch.zeros(n, dtype=kind))
    if bits == 8:
        t.update(m_scale=torch.zeros((n + 255) // 256), v_scale=torch.zeros((n + 255) // 256))
    t.update(kw)
    return t


def test_adamw_table_refusals(zblib):
    zb.adamw_table([tensors(), tensors(bits=8)])
    for kw in (dict(grad=torch.zeros(299)), dict(param=torch.zeros(300, dtype=torch.float16)), dict(m=torch.zeros(10)),
               dict(master=torch.zeros(300, dtype=torch.bfloat16)), dict(grad=torch.zeros(600)[::2]), dict(v=None)):
        refused("ZB_ERR_ARG", zb.adamw_table, [tensors(**kw)])
    refused("ZB_ERR_ARG", zb.adamw_table, [tensors(bits=8, m_scale=torch.zeros(1))])
    refused("ZB_ERR_ARG", zb.adamw_table, [tensors(m=torch.zeros(300, device="meta"))])
    apart = torch.zeros((), device="meta")
    refused("ZB_ERR_ARG", AdamW, [tensors()], lr_device=apart)
    refused("ZB_ERR_ARG", AdamW([tensors()]).step, grad_scale=apart)


def test_adamw_refusals(zblib):
    def entry(**kw):
        a = dict(param=FAKE, master=FAKE, grad=FAKE, m=FAKE, v=FAKE, m_scale=FAKE, v_scale=FAKE, count=100, weight_decay=0.1,
                 param_dtype=0, grad_dtype=1, reserved=0)
        a.update(kw)
        return (zb.zb_adamw_tensor * 1)(zb.zb_adamw_tensor(*[a[k] for k, _ in zb.zb_adamw_tensor._fields_]))

    def step(table, cfg=None, step=1, n=1, **kw):
        cfg = cfg or zb.make_adamw_config(1e-3)
        zb.zb_op_adamw_step(table, n, cfg, step, stream=0, **kw)

    for kw in (dict(param=None), dict(grad=FAKE + 4), dict(m=None), dict(master=FAKE + 8), dict(param_dtype=2), dict(grad_dtype=5),
               dict(param_dtype=1), dict(weight_decay=float("nan"))):
        refused("ZB_ERR_ARG", step, entry(**kw))
    for kw in (dict(count=-1), dict(count=(1 << 40) + 1)):
        refused("ZB_ERR_SHAPE", step, entry(**kw))
    eight = zb.make_adamw_config(1e-3, state_bits=8)
    refused("ZB_ERR_ARG", step, entry(v_scale=None), eight)
    for kw in (dict(beta1=1.0), dict(beta2=-0.1), dict(eps=0.0), dict(lr=float("inf")), dict(state_bits=16)):
        refused("ZB_ERR_ARG", step, entry(), zb.make_adamw_config(**{"lr": 1e-3, **kw}))
    refused("ZB_ERR_ARG", step, entry(), step=0)
    refused("ZB_ERR_ARG", step, entry(), n=-1)
    refused("ZB_ERR_ARG", step, entry(), grad_scale=FAKE + 2)
    refused("ZB_ERR_ARG", step, entry(), step_device=FAKE + 4)
    nbytes = zb.zb_op_grad_norm_scratch_bytes(entry(), 1)
    assert nbytes >= 8 and zb.zb_op_grad_norm_scratch_bytes(entry(count=-1), 1) == 0
    refused("ZB_ERR_ARG", zb.zb_op_grad_norm, entry(), 1, 0.0, FAKE, FAKE, nbytes, stream=0)
    refused("ZB_ERR_ARG", zb.zb_op_grad_norm, entry(grad=None), 1, 1.0, FAKE, FAKE, nbytes, stream=0)
    refused("ZB_ERR_WORKSPACE", zb.zb_op_grad_norm, entry(), 1, 1.0, FAKE, FAKE, nbytes - 1, stream=0)
    refused("ZB_ERR_ARG", zb.zb_op_adamw_unpack, entry(m_scale=None), 1, [FAKE], [FAKE], stream=0)
    refused("ZB_ERR_ARG", zb.zb_op_adamw_unpack, entry(), 1, [None], [FAKE], stream=0)


@pytest.mark.parametrize("signed", [True, False])
def test_oracle_codes(signed):
    """Every code's value packs to itself, nearest rounding takes the nearer neighbour, and the noise decides the rest."""
    values = O.code_values(False)[: 128 if signed else 256]
    assert values[-1] == (O.M_TOP if signed else O.V_TOP) and np.all(np.diff(values) > 0)
    codes, scales = O.pack(values.astype(np.float32), signed, 0x8000)
    # the largest value's block scale is exactly 1
    assert np.array_equal(codes, np.arange(values.size)) and scales[0] == 1.0
    rng = np.random.default_rng(1)
    x = (np.exp(rng.uniform(-6, np.log(float(values[-1])), 255))).astype(np.float32)
    x = np.append(x, np.float32(values[-1]))
    got = O.unpack(*O.pack(x, signed, 0x8000), signed)
    near = values[np.abs(values[None, :] - x[:, None].astype(np.float64)).argmin(1)]
    if not signed:
        near = np.maximum(near, 1.0)
    assert np.array_equal(got, near.astype(np.float32))
    down, up = O.unpack(*O.pack(x, signed, 0), signed), O.unpack(*O.pack(x, signed, 0xFFFF), signed)
    assert np.all(down <= np.maximum(x, 0.0 if signed else 1.0)) and np.all(up >= x * (1 - 2.0 ** -16))


# ---------------------------------------------------------------- document attention


def test_document_refusals(zblib):
    nbytes = zb.zb_op_attention_document_plan_bytes(300)
    assert nbytes == 3 * (2 * 128 + 2) * 8 and zb.zb_op_attention_document_plan_bytes(0) == 0
    assert zb.zb_op_attention_document_plan_bytes(-1) == 0
    scratch = zb.zb_op_attention_document_scratch_bytes(300, 4)
    assert scratch >= 4 * 384 * 4 and zb.zb_op_attention_document_scratch_bytes(300, 0) == 0

    def plan(off=FAKE, pre=FAKE, n=2, t=300, p=FAKE, size=nbytes, pos=FAKE):
        zb.zb_op_attention_document_plan(off, pre, n, t, p, size, pos, stream=0)

    refused("ZB_ERR_SHAPE", plan, t=-1)
    refused("ZB_ERR_ARG", plan, n=0)
    refused("ZB_ERR_ARG", plan, n=(1 << 28) + 1)
    refused("ZB_ERR_ARG", plan, off=None)            # no offsets: one document
    refused("ZB_ERR_ARG", plan, off=FAKE + 2)
    refused("ZB_ERR_ARG", plan, pos=FAKE + 1)
    refused("ZB_ERR_WORKSPACE", plan, size=nbytes - 1)
    refused("ZB_ERR_WORKSPACE", plan, p=None)
    refused("ZB_ERR_WORKSPACE", plan, p=FAKE + 8)

    def fwd(qkv=FAKE, a=FAKE, lse=FAKE, p=FAKE, slopes=None, cap=0.0, t=300, nh=4, nkv=2, d=64):
        zb.zb_op_attention_document_forward(qkv, a, lse, p, slopes, cap, t, nh, nkv, d, stream=0)

    def bwd(qkv=FAKE, a=FAKE, da=FAKE, lse=FAKE, dqkv=FAKE, p=FAKE, slopes=None, cap=0.0, t=300, nh=4, nkv=2, d=64, s=FAKE,
            size=scratch):
        zb.zb_op_attention_document_backward(qkv, a, da, lse, dqkv, p, slopes, cap, t, nh, nkv, d, s, size, stream=0)

    for call in (fwd, bwd):
        for kw in (dict(d=96), dict(d=32), dict(nkv=3), dict(nkv=0), dict(t=-1), dict(t=(1 << 24) + 1),
                   dict(nh=(1 << 26) + 64, nkv=1)):
            refused("ZB_ERR_SHAPE", call, **kw)
        for kw in (dict(qkv=None), dict(a=FAKE + 2), dict(lse=None), dict(p=None), dict(p=FAKE + 8), dict(slopes=FAKE + 2),
                   dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(cap=1e-4), dict(cap=513.0), dict(cap=1e6)):
            refused("ZB_ERR_ARG", call, **kw)
    refused("ZB_ERR_ARG", bwd, da=None)
    refused("ZB_ERR_ARG", bwd, dqkv=FAKE + 4)
    refused("ZB_ERR_WORKSPACE", bwd, size=scratch - 1)
    refused("ZB_ERR_WORKSPACE", bwd, s=None)


@pytest.mark.parametrize("cap,slopes", [(0.0, None), (1.5, None), (0.0, [0.3, 0.02, 0.1, 0.0]), (2.0, [0.3, 0.02, 0.1, 0.0])])
def test_oracle_document_gradient_against_differences(cap, slopes):
    t, nh, nkv, d = 23, 4, 2, 8
    rng = np.random.default_rng(2)
    x, dy, u = (rng.standard_normal((t, w * d)) for w in (nh + 2 * nkv, nh, nh + 2 * nkv))
    see = O.document_visible(t, [1, 9, 9, 20], [3, 0, 20])
    f = lambda z: np.sum(O.document_attention(z, nh, nkv, d, see, cap, slopes)[0] * dy)  # noqa: E731
    h = 1e-5
    got = np.sum(O.document_attention_grad(dy, x, nh, nkv, d, see, cap, slopes) * u)
    # central differences: h^2 of truncation, 2^-53 / h of rounding, on sums of some hundreds of terms
    assert abs((f(x + h * u) - f(x - h * u)) / (2 * h) - got) < 1e-7 * max(1.0, abs(got))


def test_oracle_documents_are_independent_and_causal():
    from oracle import stage as S

    t, nh, nkv, d = 12, 2, 1, 8
    x = np.random.default_rng(3).standard_normal((t, 4 * d))
    see = O.document_visible(t, [0, 4, 8, 12])
    np.testing.assert_allclose(O.document_attention(x, nh, nkv, d, see)[0], S.attention_causal(x, nh, nkv, d, 4), atol=1e-12)
    dy = np.random.default_rng(4).standard_normal((t, 2 * d))
    np.testing.assert_allclose(O.document_attention_grad(dy, x, nh, nkv, d, see),
                               S.attention_causal_grad(dy, x, nh, nkv, d, 4), atol=1e-12)


# ---------------------------------------------------------------- stages of documents


def test_document_stage_refusals(zblib):
    tf = dict(kind="transformer", n_layers=2, hidden=256, ffn=512, n_heads=4, n_kv_heads=2, head_dim=64, max_tokens=256,
              max_inflight=2)
    standin = zb.zb_stage_workspace_bytes(zb.make_config(**tf))
    cfg = zb.make_config(**tf, attention="document")
    size = zb.zb_stage_workspace_bytes(cfg)
    assert size > standin
    assert zb.zb_stage_workspace_bytes(zb.make_config(**tf, attention="document", seq_len=128)) == 0
    assert zb.zb_stage_workspace_bytes(zb.make_config("mlp", 2, 256, 512, attention="document")) == 0
    names = ("w_qkv", "dw_qkv", "w_o", "dw_o", "w_gu", "dw_gu", "w_down", "dw_down", "gamma1", "dgamma1", "gamma2", "dgamma2")
    layers = [{k: FAKE for k in names}] * 2
    st = zb.zb_stage_create(cfg, layers, FAKE, size)
    try:
        opts = zb.zb_stage_set_attention
        opts(st)
        opts(st, 32, "interleaved", FAKE, 1.2, 30.0, FAKE)
        refused("ZB_ERR_SHAPE", opts, st, 24, "half", FAKE)
        refused("ZB_ERR_SHAPE", opts, st, 80, "half", FAKE)           # wider than a head
        refused("ZB_ERR_ARG", opts, st, 64, "half", None)
        refused("ZB_ERR_ARG", opts, st, 64, "half", FAKE, float("nan"))
        refused("ZB_ERR_ARG", opts, st, cap=-1.0)
        refused("ZB_ERR_ARG", opts, st, cap=600.0)
        refused("ZB_ERR_ARG", opts, st, slopes=FAKE + 2)
        fwd = zb.zb_stage_forward_documents
        refused("ZB_ERR_ARG", fwd, st, 0, FAKE, 10, FAKE, None, 0, FAKE, 0)
        refused("ZB_ERR_ARG", fwd, st, 0, FAKE, 10, None, None, 2, FAKE, 0)
        refused("ZB_ERR_ARG", fwd, st, 0, FAKE, 10, FAKE, None, (1 << 28) + 1, FAKE, 0)
        refused("ZB_ERR_ARG", fwd, st, 0, FAKE, 10, FAKE + 2, None, 2, FAKE, 0)
        refused("ZB_ERR_SHAPE", fwd, st, 0, FAKE, 257, FAKE, None, 2, FAKE, 0)
    finally:
        zb.zb_stage_destroy(st)
    causal = zb.make_config(**tf, attention="causal")
    st = zb.zb_stage_create(causal, layers, FAKE, zb.zb_stage_workspace_bytes(causal))
    try:
        zb.zb_stage_set_attention(st, 64, "half", FAKE)
        refused("ZB_ERR_ARG", zb.zb_stage_set_attention, st, cap=10.0)
        refused("ZB_ERR_ARG", zb.zb_stage_forward_documents, st, 0, FAKE, 10, FAKE, None, 2, FAKE, 0)
    finally:
        zb.zb_stage_destroy(st)
    st = zb.zb_stage_create(zb.make_config(**tf), layers, FAKE, standin)
    try:
        refused("ZB_ERR_ARG", zb.zb_stage_set_attention, st)
    finally:
        zb.zb_stage_destroy(st)


def test_oracle_document_stage_split_equals_differences():
    """The oracle's B of a layer with rotary positions and document attention against central differences of its F."""
    from oracle import stage as S

    rng = np.random.default_rng(9)
    T, H, F, nh, nkv, hd = 14, 32, 24, 4, 2, 8
    prm = {k: 0.3 * rng.standard_normal(s) for k, s in S.weight_shapes("transformer", H, F, nh, nkv, hd).items()}
    shp = dict(kind="transformer", hidden=H, ffn=F, n_heads=nh, n_kv_heads=nkv, head_dim=hd, eps=1e-5, attention="document",
               offsets=[1, 6, 12], prefix=[2, 0], cap=3.0, slopes=[0.1, 0.0, 0.2, 0.05],
               rotary=(np.array([1.0, 0.1]), 1.2, "interleaved"))
    x, dy, u = (rng.standard_normal((T, H)) for _ in range(3))
    _, saved = S.layer_forward(x, prm, shp)
    dx, _ = S.layer_backward_input(dy, prm, saved, shp)
    h = 1e-5
    f = lambda z: np.sum(S.layer_forward(z, prm, shp)[0] * dy)  # noqa: E731
    assert abs((f(x + h * u) - f(x - h * u)) / (2 * h) - np.sum(dx * u)) < 1e-6 * max(1.0, abs(np.sum(dx * u)))


def test_a_stage_keeps_the_tables_it_was_given(zblib):
    """The library and the kernels on a stream have their addresses: a second set_attention gives none of them back."""
    import gc
    import weakref

    from backward_split_linear_gb300 import synth
    from backward_split_linear_gb300.runtime import Stage

    inp = synth.stage_inputs("transformer", 1, 256, 512, 2, 1, 128, tokens=8, n_mb=1, seed=1)
    st = Stage.from_synth("transformer", 1, 256, 512, 2, 1, 128, 1e-5, 128, 1, inp["params"], device="cpu", attention="document")
    given, seen = [], []
    real = zb.zb_stage_set_attention

    def note(handle, rotary_dim, pairs, turns, magnitude, cap, slopes):
        given.append([None if t is None else weakref.ref(t) for t in (turns, slopes)])
        seen.append(turns.data_ptr() if turns is not None else 0)
        real(handle, rotary_dim, pairs, turns, magnitude, cap, slopes)

    zb.zb_stage_set_attention = note
    try:
        for base in (1e4, 5e5, 1e4):
            st.set_attention(rotary_dim=64, base=base, slopes=torch.ones(2))
        st.set_attention()
    finally:
        zb.zb_stage_set_attention = real
    gc.collect()
    assert all(ref is None or ref() is not None for pair in given for ref in pair)
    assert seen[0] == seen[2] != seen[1]  # the same frequencies again take no new table
    st.close()


def test_adamw_keeps_the_tensors_that_its_table_points_to(zblib):
    import gc
    import weakref

    t = tensors(bits=8)
    opt = AdamW([t], state_bits=8)
    refs = [weakref.ref(x) for x in t.values()]
    for name in list(t):
        t[name] = None  # a caller that swaps its gradients, or lets them go
    gc.collect()
    assert all(r() is not None for r in refs)
    assert opt.table[0].grad == opt.tensors[0]["grad"].data_ptr()


class Elsewhere:
    """A tensor of some device, as far as the checks look at one."""

    def __init__(self, like, device):
        self.like, self.device = like, torch.device(device)

    dtype = property(lambda self: self.like.dtype)

    def numel(self):
        return self.like.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE


def on(device, **kw):
    return {k: Elsewhere(t, device) for k, t in tensors(**kw).items()}


def test_adamw_takes_one_device(zblib, monkeypatch):
    """A launch reads every tensor from the current device: another index of the same type is another device."""
    zb.adamw_table([on("cuda:1"), on("cuda:1")])
    refused("ZB_ERR_ARG", zb.adamw_table, [on("cuda:0"), on("cuda:1")])
    refused("ZB_ERR_ARG", zb.adamw_table, [on("cuda:0"), tensors()])
    one, number = torch.zeros(()), torch.zeros((), dtype=torch.int64)
    for kw in (dict(lr_device=Elsewhere(one, "cuda:1")), dict(step_device=Elsewhere(number, "cuda:1")),
               dict(lr_device=Elsewhere(torch.zeros(0), "cuda:0")), dict(step_device=Elsewhere(number.new_zeros(2), "cuda:0")),
               dict(step_device=Elsewhere(one, "cuda:0"))):
        refused("ZB_ERR_ARG", AdamW, [on("cuda:0")], **kw)
    launched = []
    for name in ("zb_op_adamw_step", "zb_op_grad_norm", "zb_op_adamw_unpack"):
        monkeypatch.setattr(zb, name, lambda *a, **kw: launched.append(a))
    for bits in (32, 8):
        opt = AdamW([tensors(bits=bits)], state_bits=bits)  # the host's: no call may launch
        refused("ZB_ERR_ARG", opt.step)
        refused("ZB_ERR_ARG", opt.grad_norm)
        if bits == 8:
            refused("ZB_ERR_ARG", opt.unpack_states)
        opt.device, opt.index = torch.device("cuda:1"), 1  # as if all of it lay there
        monkeypatch.setattr(zb, "_current_device", lambda: 0)
        refused("ZB_ERR_ARG", opt.step)
        refused("ZB_ERR_ARG", opt.grad_norm)
        monkeypatch.setattr(zb, "_current_device", lambda: 1)
        for scale in (Elsewhere(one, "cuda:0"), Elsewhere(torch.zeros(0), "cuda:1"), Elsewhere(number, "cuda:1"), one):
            refused("ZB_ERR_ARG", opt.step, grad_scale=scale)
        assert not launched and opt.steps == 0
        opt.step(grad_scale=Elsewhere(one, "cuda:1"))
        opt.grad_norm()
        assert len(launched) == 2 and opt.steps == 1
        launched.clear()


@pytest.mark.parametrize("context", [1.0, 2.0, 4.0, 6.0, 6.5, 7.0, 50.0, 300.0, 8192.0, 1e7])
@pytest.mark.parametrize("rot,base", [(16, 10000.0), (128, 500000.0), (64, 3.0)])
def test_yarn_keeps_and_stretches_the_pairs_it_says(zblib, rot, base, context):
    """Pairs of fewer than `low` turns over the original context are stretched in full, pairs of more than `high` kept, the
    shortest contexts included.  In radians half a unit of the 64-bit fraction of a turn is 2 pi 2^-65."""
    near = dict(rtol=64 * 2.0 ** -53, atol=2.0 * np.pi * 2.0 ** -65)
    factor, low, high = 8.0, 1.0, 32.0
    turns, _ = zb.zb_rotary_frequencies(rot, base, "yarn", factor, context, low, high)
    got = np.array([t / 2.0 ** 64 for t in turns]) * 2.0 * np.pi
    f = base ** (-2.0 * np.arange(rot // 2) / rot)
    made = context * f / (2.0 * np.pi)
    for which, want in ((made < low * (1 - 1e-9), f / factor), (made > high * (1 + 1e-9), f)):
        np.testing.assert_allclose(got[which], want[which], **near)
    np.testing.assert_allclose(O.rotary_frequencies(rot, base, "yarn", factor, context, low, high)[0], got, **near)
