"""The feed-forward block's operators where their tests by size and kind do not come: gradients asked for alone, K split in a cluster."""
import pytest
import torch

from backward_split_linear_gb300 import binding as zb
from oracle import block_ops as O

pytestmark = pytest.mark.gpu


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def bytes_of(n):
    return torch.empty(max(16, n), dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- norms: one gradient, and only what it reads


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post", ["layer", "none"])
@pytest.mark.parametrize("t,w", [(37, 320), (300, 2112)])
def test_one_gradient_takes_only_what_it_reads(cuda_device, t, w, post, gate):
    normal = generator(t)
    bf16 = lambda *s: normal(*s).to(torch.bfloat16)  # noqa: E731
    par = dict(pre="layer", pre_gamma=normal(w), pre_beta=normal(w), gate_kind=gate, branch_scale=0.5)
    if post == "layer":
        par.update(post="layer", post_gamma=normal(w), post_beta=normal(w))
    if gate != "none":
        par.update(gate=normal(w) if gate == "channel" else bf16(t, w))
    op = zb.make_residual_norm(**par)
    x, y, dn, dh = (bf16(t, w) for _ in range(4))
    h, n, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(t, 4, device="cuda")
    zb.zb_op_residual_norm_forward(op, x, y, h, n, stats, t, w)
    scratch = bytes_of(zb.zb_op_residual_norm_backward_weight_scratch_bytes(t, w))
    reads = {"dpre_gamma": dict(dn=dn, h=h), "dpre_beta": dict(dn=dn)}
    if post == "layer":
        reads.update(dpost_gamma=dict(dh=dh, y=y), dpost_beta=dict(dh=dh))
    if gate == "channel":
        reads["dgate"] = dict(dh=dh, y=y)
    before = {k: normal(w) for k in reads}
    every = {k: v.clone() for k, v in before.items()}
    zb.zb_op_residual_norm_backward_weight(op, dn, h, dh, y, stats, t, w, scratch, **every)
    for k, given in reads.items():
        one = before[k].clone()
        a = {**dict(dn=None, h=None, dh=None, y=None), **given}
        zb.zb_op_residual_norm_backward_weight(op, a["dn"], a["h"], a["dh"], a["y"], stats, t, w, scratch, **{k: one})
        assert torch.equal(one, every[k]), k
    # a beta of one pair beside a gamma of the other
    pairs = [("dpre_beta", "dpost_gamma"), ("dpre_gamma", "dpost_beta")] if post == "layer" else []
    for names in pairs:
        some = {k: before[k].clone() for k in names}
        a = dict(dn=None, h=None, dh=None, y=None)
        for k in names:
            a.update(reads[k])
        zb.zb_op_residual_norm_backward_weight(op, a["dn"], a["h"], a["dh"], a["y"], stats, t, w, scratch, **some)
        for k in names:
            assert torch.equal(some[k], every[k]), k
    # the betas themselves, against float64
    for k, add in (("dpre_beta", dn.double()), ("dpost_beta", 0.5 * dh.double() * (par["gate"].double() if gate != "none" else 1.0))):
        if k in every:
            err = (every[k].double() - before[k].double() - add.sum(0)).abs()
            bar = (t + 4) * 2.0 ** -24 * add.abs().sum(0) + 2.0 ** -22 * (before[k].double().abs() + 1)
            assert bool((err <= bar).all()), k


# ---------------------------------------------------------------- K split among the CTA pairs of a cluster
#
# From K = 2048 on, where all units of 256 x 128 run at once: 25 units take two pairs each, 8 and 1 take four.

HALF = 2.0 ** -8
SPLIT = [(185, 2112, 3200), (300, 2304, 512), (33, 4160, 64)]


def placed(x, off):
    """x, or a copy of it that starts 16 bytes behind a 32-byte boundary."""
    if x is None or not off:
        return x
    if isinstance(x, tuple):
        return tuple(placed(v, off) for v in x)
    at = 16 // x.element_size()
    room = torch.zeros(x.numel() + at, dtype=x.dtype, device="cuda")
    room[at:].copy_(x.reshape(-1))
    assert room.data_ptr() % 32 == 0
    return room[at:].view(x.shape)


def codes_like(t, n, off=False):
    return placed((torch.zeros(t, n, dtype=torch.uint8, device="cuda"), torch.zeros(t, n // 32, dtype=torch.uint8, device="cuda")), off)


def slip(mass, k):
    """A sum of k terms of this mass, 1024 at most at a time on the tensor cores: 16 terms an addition that drops what falls below the
    last bit, some more inside, and float32 additions of the parts."""
    return ((min(k, 1024) / 16 + 4) * 2.0 ** -22 + (k / 128) * 2.0 ** -24) * mass


def within(got, ref, bar, what):
    err = (got.double() - ref).abs()
    assert bool((err <= bar).all()), f"{what}: {float((err / bar).max()):.3g} of the bar"


def on_gpu(f, x, kind):
    return torch.from_numpy(f(x.cpu().numpy(), kind)).cuda()


@pytest.mark.parametrize("off", [False, True])
@pytest.mark.parametrize("kind", ["none", "gelu", "relu2"])
@pytest.mark.parametrize("t,k,n", SPLIT)
def test_split_forward(cuda_device, t, k, n, kind, off):
    normal = generator(t + k)
    bf16 = lambda *s: normal(*s).to(torch.bfloat16)  # noqa: E731
    x, w, res, bias = bf16(t, k), (normal(n, k) * k ** -0.5).to(torch.bfloat16), bf16(t, n), normal(n)
    zz = x.double() @ w.double().t() + bias.double()
    s = slip(x.double().abs() @ w.double().abs().t() + bias.double().abs(), k)
    a = on_gpu(O.act, zz, kind)
    steep = 1.2 if kind != "relu2" else 2.0 * zz.abs() + s
    for r in (None, res):
        ref = a if r is None else a + r.double()
        bar = HALF * ref.abs() + 2.0 ** -12 * a.abs() + 2.0 ** -18 + steep * s + (0.0 if r is None else 2.0 ** -23 * r.double().abs())
        args = [placed(v, off) for v in (x, w, bias, r)]
        y, z, plain = (placed(torch.zeros_like(res), off) for _ in range(3))
        y8, z8 = codes_like(t, n, off), codes_like(t, n, off)
        zb.zb_op_linear_activation_forward(*args, y, t, k, n, kind, z=z, y_packed=y8)
        within(y, ref, bar, "y")
        within(z, zz, HALF * zz.abs() + s, "z")
        for packed, v in ((y8, y), (z8, z)):
            if packed is z8:
                again = torch.zeros_like(res)
                zb.zb_op_linear_activation_forward(*args, again, t, k, n, kind, z_packed=z8)
                assert torch.equal(again, y)
            c = codes_like(t, n)
            zb.zb_op_checkpoint_pack(v, c, t, n)
            assert torch.equal(c[0], packed[0]) and torch.equal(c[1], packed[1])
        # bf16 alone, and over the residual
        zb.zb_op_linear_activation_forward(*args, plain, t, k, n, kind)
        within(plain, ref, bar, "y alone")
        if r is not None:
            zb.zb_op_linear_activation_forward(*args, args[3], t, k, n, kind)
            assert torch.equal(args[3], plain)
    assert zb.zb_device_status() == (0, 0)


@pytest.mark.parametrize("off", [False, True])
@pytest.mark.parametrize("kind", ["none", "gelu", "relu2"])
@pytest.mark.parametrize("t,k,n", SPLIT)
def test_split_backward(cuda_device, t, k, n, kind, off):
    """dy [t, k], w [k, n], z [t, n]."""
    normal = generator(t + n)
    dy, w, z = normal(t, k).to(torch.bfloat16), (normal(k, n) * k ** -0.5).to(torch.bfloat16), (1.5 * normal(t, n)).to(torch.bfloat16)
    z8 = codes_like(t, n, off)
    zb.zb_op_checkpoint_pack(z, z8, t, n)
    values = torch.zeros_like(z)
    zb.zb_op_checkpoint_unpack(z8, values, t, n)
    ds = dy.double() @ w.double()
    s = slip(dy.double().abs() @ w.double().abs(), k)
    dy, w = placed(dy, off), placed(w, off)
    scratch = bytes_of(zb.zb_op_backward_input_activation_scratch_bytes(t, n))
    before = normal(n)
    for eight in (False, True):
        slope = on_gpu(O.act_slope, (values if eight else z).double(), kind)
        ref = ds * slope
        bar = (HALF + 2.0 ** -12) * ref.abs() + 2.0 ** -18 * ds.abs() + (slope.abs() + 0.1) * s
        zin, zin8 = (None, z8) if eight else (placed(z, off), None)
        dz, plain = (placed(torch.zeros_like(z), off) for _ in range(2))
        dbias = placed(before.clone(), off)
        zb.zb_op_backward_input_activation(dy, w, zin, dz, t, n, k, kind, z_packed=zin8, dbias=dbias, scratch=scratch)
        within(dz, ref, bar, "dz")
        each = 2.0 ** -18 * ds.abs() + (slope.abs() + 0.1) * s + t * 2.0 ** -24 * ref.abs()
        within(dbias, before.double() + ref.sum(0), each.sum(0) + 2.0 ** -22 * before.double().abs(), "dbias")
        zb.zb_op_backward_input_activation(dy, w, zin, plain, t, n, k, kind, z_packed=zin8)
        within(plain, ref, bar, "dz alone")
        if not eight:
            over = placed(z.clone(), off)
            zb.zb_op_backward_input_activation(dy, w, over, over, t, n, k, kind)
            assert torch.equal(over, plain)
    assert zb.zb_device_status() == (0, 0)


@pytest.mark.parametrize("off", [False, True])
@pytest.mark.parametrize("t,k,n", [(2111, 3200, 192), (2048, 128, 448)])
def test_split_weight(cuda_device, t, k, n, off):
    """dy [t, n], x [t, k], dw [n, k]: 25 units and 2."""
    normal = generator(t)
    dy, x = normal(t, n).to(torch.bfloat16), normal(t, k).to(torch.bfloat16)
    x8 = codes_like(t, k, off)
    zb.zb_op_checkpoint_pack(x, x8, t, k)
    zb.zb_op_checkpoint_unpack(x8, x, t, k)
    before = normal(n, k)
    scratch = bytes_of(zb.zb_op_backward_weight_checkpoint_scratch_bytes(t, k))
    dw = [placed(before.clone(), off) for _ in range(2)]
    for v in dw:
        zb.zb_op_backward_weight_checkpoint(placed(dy, off), x8, v, t, k, n, scratch)
    ref = before.double() + dy.double().t() @ x.double()
    s = slip(dy.double().abs().t() @ x.double().abs(), t)
    within(dw[0], ref, s + 2.0 ** -23 * (before.double().abs() + ref.abs()), "dw")
    assert torch.equal(*dw)
    assert zb.zb_device_status() == (0, 0)


# ---------------------------------------------------------------- B from the checkpoints that F wrote
#
# The largest second derivatives: gelu 2 phi(0) = 0.798, its tanh form 0.798 too (0.81 taken), silu 1/2, max(z, 0)^2 2.

CURVED = {"none": 0.0, "gelu": 0.81, "gelu_tanh": 0.81, "silu": 0.5, "relu2": 2.0}


def forward_and_slopes(kind, outlier):
    """F's bf16 z, y and 8-bit z of one layer, B through it from a z, dy w in float64 and its bound."""
    t, k, n = 200, 256, 640
    normal = generator(9)
    x, w = normal(t, k).to(torch.bfloat16), (normal(n, k) * k ** -0.5).to(torch.bfloat16)
    bias = 0.1 * normal(n)
    if outlier:
        w[5::32] *= 20.0
    y, z = (torch.empty(t, n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    z8 = codes_like(t, n)
    zb.zb_op_linear_activation_forward(x, w, bias, None, y, t, k, n, kind, z=z)
    zb.zb_op_checkpoint_pack(z, z8, t, n)
    dy, w2 = normal(t, k).to(torch.bfloat16), (normal(k, n) * k ** -0.5).to(torch.bfloat16)

    def back(z_given, packed):
        dz = torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
        zb.zb_op_backward_input_activation(dy, w2, z_given, dz, t, n, k, kind, z_packed=packed)
        return dz

    ds = dy.double() @ w2.double()
    return y, z, z8, back, ds, ds.abs() + slip(dy.double().abs() @ w2.double().abs(), k)


@pytest.mark.parametrize("outlier", [False, True])
@pytest.mark.parametrize("kind", sorted(CURVED))
def test_gradient_from_forwards_8_bits(cuda_device, kind, outlier):
    """Against the gradient from the bf16 z that F computed: the slope is off by its own slope times the code's error."""
    y, z, z8, back, _, most = forward_and_slopes(kind, outlier)
    values = torch.empty_like(z)
    zb.zb_op_checkpoint_unpack(z8, values, *z.shape)
    exact, got = back(z, None).double(), back(None, z8).double()
    # both are rounded to bf16, from float32 slopes and sums a little off
    fine = (HALF + 2.0 ** -12) * (exact.abs() + got.abs()) + 2.0 ** -17 * most
    within(got, exact, most * CURVED[kind] * (values.double() - z.double()).abs() + fine, kind)


@pytest.mark.parametrize("outlier", [False, True])
def test_relu_takes_its_output_for_z(cuda_device, outlier):
    """The bf16 y gives the gradient that the bf16 z gives, bit for bit.  8 bits lose it where a positive z reads as 0, and only
    there; the header says so."""
    y, z, z8, back, ds, _ = forward_and_slopes("relu", outlier)
    exact = back(z, None)
    assert torch.equal(back(y, None), exact)
    lost = (z > 0) & ((z8[0] & 127) == 0)
    assert int(lost.sum()) > 0
    got = back(None, z8)
    assert torch.equal(got[~lost], exact[~lost]) and not bool(got[lost].any())
    dy = ds.to(torch.bfloat16)  # the activation alone, likewise
    alone = [torch.empty_like(dy) for _ in range(2)]
    for v, zz in zip(alone, (z, y)):
        zb.zb_op_activation_backward(dy, zz, v, *z.shape, "relu")
    assert torch.equal(*alone)
