"""GPU parity of the feed-forward block's operators against the float64 oracle, element by element.

Bars.  A bf16 result is off by half a step, 2^-8 of its value (torch.finfo(bf16).eps / 2), plus the float32 arithmetic
before it.  A product of k terms on the tensor cores adds 16 of them at a time to a float32 sum and drops what falls
below its last bit: (k / 16 + 4) 2^-22 of the sum of the terms' magnitudes bounds that with room for the order inside an
instruction.  The activations and their slopes are taken to 2^-12 of the value plus 2^-18 (the fast exponential and
division have errors of a few 2^-23 times their argument, which stays below 100 where the result is not 0; the slopes
are sums of terms up to 1.2 that may cancel).  Float32 sums over t rows add t 2^-24 of the sum of magnitudes at most.
"""
import numpy as np
import pytest
import torch

from backward_split_linear_gb300 import binding as zb
from backward_split_linear_gb300.runtime import bf16_from_bits, f64_from_bf16
from oracle import block_ops as O
from parity import draw_bf16

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8
GUARD = 3  # rows behind the last, which every call leaves as they are
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu", "relu2"]


def out_rows(t, width, dtype=torch.bfloat16):
    """A buffer of t rows and some more, all of one recognisable value."""
    return torch.full((t + GUARD, width), 77, dtype=dtype, device="cuda")


def take(buf, t):
    assert torch.all(buf[t:] == 77), "rows behind the last were written"
    return f64_from_bf16(buf[:t]) if buf.dtype == torch.bfloat16 else buf[:t].cpu().numpy()


def packed_rows(t, width):
    return out_rows(t, width, torch.uint8), out_rows(t, width // 32, torch.uint8)


def take_packed(p, t):
    return take(p[0], t), take(p[1], t)


def f32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()


def draw_f32(rng, *shape):
    x = rng.standard_normal(shape, dtype=np.float32)
    return x.astype(np.float64), torch.from_numpy(x).cuda()


def scratch_of(n):
    return torch.full((max(16, n),), 255, dtype=torch.uint8, device="cuda")


def within(got, ref, bar, what=""):
    err = np.abs(np.asarray(got, dtype=np.float64) - ref)
    assert np.all(err <= bar), f"{what}: {np.max(err / np.maximum(bar, 1e-300)):.3g} of the bar"


def no_waits_ran_out():
    assert zb.zb_device_status() == (0, 0)


# ---------------------------------------------------------------- linear forward

SHAPES = [(1, 64, 64), (7, 128, 192), (128, 256, 512), (129, 64, 320), (255, 192, 64), (256, 256, 256), (300, 1024, 576),
          (513, 320, 1088)]


@pytest.mark.parametrize("t,k,n", SHAPES)
@pytest.mark.parametrize("kind", ACTS)
def test_forward(cuda_device, t, k, n, kind):
    rng = np.random.default_rng(t + n)
    xb, x = draw_bf16(rng, (t, k))
    wb, w = draw_bf16(rng, (n, k), std=1.5 / np.sqrt(k))
    rb, res = draw_bf16(rng, (t, n))
    bias, bias_dev = draw_f32(rng, n)
    xd, wd, rd = bf16_from_bits(xb), bf16_from_bits(wb), bf16_from_bits(rb)
    y, z = out_rows(t, n), out_rows(t, n)
    y8, z8 = packed_rows(t, n), packed_rows(t, n)
    zb.zb_op_linear_activation_forward(xd, wd, bias_dev, rd, y, t, k, n, kind, z=z, y_packed=y8)
    zz = x @ w.T + bias
    slip = (k / 16 + 4) * 2.0 ** -22 * (np.abs(x) @ np.abs(w).T + np.abs(bias))
    within(take(z, t), zz, HALF * np.abs(zz) + slip, "z")
    a = O.act(zz, kind)
    steep = 1.2 if kind != "relu2" else 2.0 * np.abs(zz) + slip
    bar = HALF * np.abs(a + res) + 2.0 ** -12 * np.abs(a) + 2.0 ** -18 + steep * slip + 2.0 ** -23 * np.abs(res)
    within(take(y, t), a + res, bar, "y")
    # the checkpoints are the packed forms of the stored tensors
    codes, scales = O.pack(take(y, t))
    assert np.array_equal(take_packed(y8, t)[0], codes) and np.array_equal(take_packed(y8, t)[1], scales)
    y2 = out_rows(t, n)
    zb.zb_op_linear_activation_forward(xd, wd, bias_dev, rd, y2, t, k, n, kind, z_packed=z8)
    assert torch.equal(y2, y)
    codes, scales = O.pack(take(z, t))
    assert np.array_equal(take_packed(z8, t)[0], codes) and np.array_equal(take_packed(z8, t)[1], scales)
    # nothing but y is asked for (its sums are then taken in another order), and y may be the residual
    y3 = out_rows(t, n)
    zb.zb_op_linear_activation_forward(xd, wd, bias_dev, rd, y3, t, k, n, kind)
    within(take(y3, t), a + res, bar, "y alone")
    zb.zb_op_linear_activation_forward(xd, wd, bias_dev, rd, rd, t, k, n, kind)
    assert torch.equal(rd, y3[:t])
    no_waits_ran_out()


def same_packed(p, x, t):
    """The 8-bit form that an epilogue wrote is the one that packing the bf16 tensor gives."""
    codes, scales = torch.empty_like(p[0][:t]), torch.empty_like(p[1][:t])
    zb.zb_op_checkpoint_pack(x, (codes, scales), t, x.shape[1])
    assert torch.equal(codes, p[0][:t]) and torch.equal(scales, p[1][:t])
    assert torch.all(p[0][t:] == 77) and torch.all(p[1][t:] == 77)


def product_slip(mass, k, most):
    """Bound of a product's error (the module's docstring) with sums of `most` terms at a time on the tensor cores."""
    return ((min(k, most) / 16 + 4) * 2.0 ** -22 + (k / 512) * 2.0 ** -24) * mass


# long inner sizes (sums in registers, the first ones longer; K split among CTA pairs), outputs of several waves of tiles whose
# last is cut in two or in four, and of one wave of tiles narrower than 256 columns
LONG = [(130, 4160, 320), (70, 1216, 192), (40, 2304, 64), (2600, 64, 2112), (2600, 128, 2048), (300, 64, 12672),
        (1000, 64, 4096), (1300, 64, 1984), (520, 128, 4160)]


@pytest.mark.parametrize("t,k,n", LONG)
def test_long_and_wide(cuda_device, t, k, n):
    rng = np.random.default_rng(k + n)
    xb, x = draw_bf16(rng, (t, k))
    wb, w = draw_bf16(rng, (n, k), std=1.0 / np.sqrt(k))
    bias, bias_dev = draw_f32(rng, n)
    xd, wd = bf16_from_bits(xb), bf16_from_bits(wb)
    y, z, y8, z8 = out_rows(t, n), out_rows(t, n), packed_rows(t, n), packed_rows(t, n)
    zb.zb_op_linear_activation_forward(xd, wd, bias_dev, None, y, t, k, n, "silu", z=z, y_packed=y8)
    zz = x @ w.T + bias
    mass = np.abs(x) @ np.abs(w).T + np.abs(bias)
    slip = product_slip(mass, k, 1024)
    within(take(z, t), zz, HALF * np.abs(zz) + slip, "z")
    a = O.act(zz, "silu")
    within(take(y, t), a, (HALF + 2.0 ** -12) * np.abs(a) + 2.0 ** -18 + 1.2 * slip, "y")
    y2 = out_rows(t, n)
    zb.zb_op_linear_activation_forward(xd, wd, bias_dev, None, y2, t, k, n, "silu", z_packed=z8)
    assert torch.equal(y2, y)
    same_packed(y8, y[:t], t)
    same_packed(z8, z[:t], t)
    plain = out_rows(t, n)
    zb.zb_op_linear_activation_forward(xd, wd, bias_dev, None, plain, t, k, n, "silu")
    within(take(plain, t), a, (HALF + 2.0 ** -12) * np.abs(a) + 2.0 ** -18 + 1.2 * product_slip(mass, k, k), "y alone")
    # B back through it: dy [t, k] of a linear [k, n] behind the activation
    db, dy = draw_bf16(rng, (t, k))
    w2 = bf16_from_bits(wb).t().contiguous()
    zq = O.unpack(take(z8[0], t), take(z8[1], t))
    ds, slope = dy @ w.T, O.act_slope(zq, "silu")
    mass = np.abs(dy) @ np.abs(w).T
    before, dbias = draw_f32(rng, n)
    scratch = scratch_of(zb.zb_op_backward_input_activation_scratch_bytes(t, n))
    for with_bias in (True, False):
        dz = out_rows(t, n)
        zb.zb_op_backward_input_activation(bf16_from_bits(db), w2, None, dz, t, n, k, "silu", z_packed=(z8[0], z8[1]),
                                           dbias=dbias if with_bias else None, scratch=scratch)
        slip = product_slip(mass, k, 1024 if with_bias else k)
        bar = (HALF + 2.0 ** -12) * np.abs(ds * slope) + 2.0 ** -18 * np.abs(ds) + (np.abs(slope) + 0.1) * slip
        within(take(dz, t), ds * slope, bar, "dz")
    each = 2.0 ** -18 * np.abs(ds) + (np.abs(slope) + 0.1) * product_slip(mass, k, 1024) + t * 2.0 ** -24 * np.abs(ds * slope)
    within(dbias.cpu().numpy(), before + (ds * slope).sum(0), each.sum(0) + 2.0 ** -22 * np.abs(before), "dbias")
    no_waits_ran_out()


@pytest.mark.parametrize("shift", [8, 24])
def test_tensors_at_16_byte_starts(cuda_device, shift):
    """Tensors that start 16 bytes off a 32-byte boundary give the same bits as aligned ones."""
    t, k, n = 70, 128, 192

    def off(x):
        """A copy of x that starts `shift` bf16 elements (codes: 16 bytes) into its storage."""
        at = shift if x.dtype == torch.bfloat16 else 16
        room = torch.zeros(x.numel() + at, dtype=x.dtype, device="cuda")
        room[at:].copy_(x.reshape(-1))
        return room[at:].view(x.shape)

    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, w, res, dy, w2 = draw(t, k), draw(n, k), draw(t, n), draw(t, k), draw(k, n)
    bias = torch.randn(n, generator=g, device="cuda")
    got = []
    for place in (lambda v: v, off):
        y, z = place(torch.zeros_like(res)), place(torch.zeros_like(res))
        y8 = tuple(place(torch.zeros(t, c, dtype=torch.uint8, device="cuda")) for c in (n, n // 32))
        z8 = tuple(place(torch.zeros(t, c, dtype=torch.uint8, device="cuda")) for c in (n, n // 32))
        zb.zb_op_linear_activation_forward(place(x), place(w), bias, place(res), y, t, k, n, "gelu", z=z, y_packed=y8)
        zb.zb_op_checkpoint_pack(z, z8, t, n)
        dz, dz8 = place(torch.zeros_like(res)), place(torch.zeros_like(res))
        zb.zb_op_backward_input_activation(place(dy), place(w2), z, dz, t, n, k, "gelu")
        zb.zb_op_backward_input_activation(place(dy), place(w2), None, dz8, t, n, k, "gelu", z_packed=z8)
        dw = torch.zeros(k, n, device="cuda")
        scratch = scratch_of(zb.zb_op_backward_weight_checkpoint_scratch_bytes(t, n))
        zb.zb_op_backward_weight_checkpoint(place(dy), y8, dw, t, n, k, scratch)
        got.append([y, z, *y8, *z8, dz, dz8, dw])
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_forward_without_options(cuda_device):
    t, k, n = 200, 128, 128
    rng = np.random.default_rng(0)
    xb, x = draw_bf16(rng, (t, k))
    wb, w = draw_bf16(rng, (n, k), std=0.1)
    y, plain = out_rows(t, n), torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
    zb.zb_op_linear_activation_forward(bf16_from_bits(xb), bf16_from_bits(wb), None, None, y, t, k, n)
    zb.zb_op_linear_forward(bf16_from_bits(xb), bf16_from_bits(wb), None, plain, t, k, n)
    assert torch.equal(y[:t], plain)
    take(y, t)


@pytest.mark.parametrize("kind", ACTS)
def test_values_out_of_range(cuda_device, kind):
    """Large and non-finite pre-activations: through a weight that copies x."""
    t, n = 4, 64
    x = torch.zeros(t, n, dtype=torch.bfloat16, device="cuda")
    probe = torch.tensor([float("nan"), float("inf"), 3e38, 1e19, 200.0, -200.0, -1e19, -3e38, 0.0], dtype=torch.bfloat16)
    for i in range(len(probe)):  # one row's inner product must not mix them: infinity times zero is NaN
        bias = torch.zeros(n, device="cuda")
        bias[5] = float(probe[i])
        y, z = out_rows(t, n), out_rows(t, n)
        y8 = packed_rows(t, n)
        eye = torch.eye(n, device="cuda").to(torch.bfloat16)
        zb.zb_op_linear_activation_forward(x, eye, bias, None, y, t, n, n, kind, z=z, y_packed=y8)
        got, v = float(take(y, t)[0, 5]), float(probe[i])
        if np.isnan(v):
            assert np.isnan(got)
            assert np.all(take_packed(y8, t)[1][:, 0] == 255) and np.all(take_packed(y8, t)[1][:, 1] != 255)
        elif np.isinf(v):
            assert got == v
        else:
            with np.errstate(over="ignore"):
                ref = float(torch.tensor(O.act(np.array([v]), kind)[0]).to(torch.bfloat16))
            assert got == ref or abs(got - ref) <= 2 * HALF * abs(ref) + 1e-30, (v, got, ref)
        assert np.all(take(y, t)[:, 6:] == 0.0)
        # and back: the slope of the stored z
        ones = torch.ones(t, n, dtype=torch.bfloat16, device="cuda")
        dz = out_rows(t, n)
        zb.zb_op_activation_backward(ones, z[:t], dz, t, n, kind)
        d = float(take(dz, t)[0, 5])
        if np.isnan(v):
            assert np.isnan(d) or kind == "none"
        elif np.isfinite(v) and abs(v) < 1e30:
            ref = O.act_slope(np.array([np.clip(v, -50, 50) if kind != "relu2" else v]), kind)[0]
            assert abs(d - ref) <= 2 * HALF * abs(ref) + 1e-9, (v, d, ref)


# ---------------------------------------------------------------- B


@pytest.mark.parametrize("t,n,k", SHAPES)
@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("eight", [False, True])
def test_backward_input(cuda_device, t, k, n, kind, eight):
    """dy [t, k], w [k, n], z [t, n]."""
    rng = np.random.default_rng(t + 2 * n)
    db, dy = draw_bf16(rng, (t, k))
    wb, w = draw_bf16(rng, (k, n), std=1.0 / np.sqrt(k))
    zbits, z = draw_bf16(rng, (t, n), std=1.5)
    zd = bf16_from_bits(zbits)
    z8 = None
    if eight:
        codes, scales = O.pack(z)
        z8 = (torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
        z = O.unpack(codes, scales)
    before, dbias = draw_f32(rng, n)
    dz = out_rows(t, n)
    scratch = scratch_of(zb.zb_op_backward_input_activation_scratch_bytes(t, n))
    args = (bf16_from_bits(db), bf16_from_bits(wb), None if eight else zd)
    zb.zb_op_backward_input_activation(*args, dz, t, n, k, kind, z_packed=z8, dbias=dbias, scratch=scratch)
    ds, slope = dy @ w, O.act_slope(z, kind)
    mass = np.abs(dy) @ np.abs(w)
    slip = (k / 16 + 4) * 2.0 ** -22 * mass
    bar = HALF * np.abs(ds * slope) + 2.0 ** -12 * np.abs(ds * slope) + 2.0 ** -18 * np.abs(ds) + (np.abs(slope) + 0.1) * slip
    within(take(dz, t), ds * slope, bar, "dz")
    # 512 terms at a time on the tensor cores (sums this short), k / 512 sums in registers
    slip = ((min(k, 512) / 16 + 4) * 2.0 ** -22 + (k / 512) * 2.0 ** -24) * mass
    each = 2.0 ** -18 * np.abs(ds) + (np.abs(slope) + 0.1) * slip + t * 2.0 ** -24 * np.abs(ds * slope)
    within(dbias.cpu().numpy(), before + (ds * slope).sum(0), each.sum(0) + 2.0 ** -22 * np.abs(before), "dbias")
    # without the bias gradient, and over z itself
    dz2 = zd.clone() if not eight else out_rows(t, n)
    zb.zb_op_backward_input_activation(args[0], args[1], None if eight else dz2, dz2, t, n, k, kind, z_packed=z8)
    within(f64_from_bf16(dz2[:t]), ds * slope, bar, "dz in place")
    # twice the same bits
    dz3, again = out_rows(t, n), f32(before)
    zb.zb_op_backward_input_activation(*args, dz3, t, n, k, kind, z_packed=z8, dbias=again, scratch=scratch)
    assert torch.equal(dz, dz3) and torch.equal(again, dbias)
    no_waits_ran_out()


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("kind", ACTS)
def test_activation_alone(cuda_device, kind, eight):
    t, n = 37, 192
    rng = np.random.default_rng(4)
    db, dy = draw_bf16(rng, (t, n))
    zbits, z = draw_bf16(rng, (t, n), std=2.0)
    zd, z8 = bf16_from_bits(zbits), None
    if eight:
        codes, scales = O.pack(z)
        z8, z = (torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()), O.unpack(codes, scales)
    dz, dyd = out_rows(t, n), bf16_from_bits(db)
    zb.zb_op_activation_backward(dyd, None if eight else zd, dz, t, n, kind, z_packed=z8)
    ref = dy * O.act_slope(z, kind)
    within(take(dz, t), ref, (HALF + 2.0 ** -12) * np.abs(ref) + 2.0 ** -18 * np.abs(dy), kind)
    zb.zb_op_activation_backward(dyd, None if eight else zd, dyd, t, n, kind, z_packed=z8)
    assert torch.equal(dyd, dz[:t])


@pytest.mark.parametrize("t,n", [(1, 64), (7, 192), (8, 256), (300, 320), (2049, 64), (1000, 2112)])
def test_bias_gradient(cuda_device, t, n):
    rng = np.random.default_rng(t)
    db, dy = draw_bf16(rng, (t, n))
    before, dbias = draw_f32(rng, n)
    scratch = scratch_of(zb.zb_op_backward_bias_scratch_bytes(t, n))
    zb.zb_op_backward_bias(bf16_from_bits(db), dbias, t, n, scratch)
    # each addend passes through at most t additions
    within(dbias.cpu().numpy(), before + dy.sum(0), t * 2.0 ** -24 * np.abs(dy).sum(0) + 2.0 ** -22 * (np.abs(before) + 1), "dbias")


# ---------------------------------------------------------------- 8-bit checkpoints


def odd_values(rng, t, width):
    """Ordinary blocks, and blocks at every border of the format."""
    bits, x = draw_bf16(rng, (t, width))
    bits = bits.copy()
    for r in range(t):
        kind = r % 8
        if kind == 1:
            bits[r, :32] = rng.integers(0, 1 << 16, 32)              # any bits, NaN and infinity among them
        elif kind == 2:
            bits[r, :] = rng.integers(0, 0x7f80, width)              # any finite positive
        elif kind == 3:
            bits[r, 32:64] = 0x7f7f                                  # the largest
        elif kind == 4:
            bits[r, :32] = rng.integers(0, 0x180, 32)                # subnormal and the smallest normal ones
        elif kind == 5:
            bits[r, :] = 0x8000                                      # minus zero
        elif kind == 6:
            bits[r, 7] = 0x42ff                                      # 127.5: carried to the next scale
    return bits


@pytest.mark.parametrize("t,width", [(1, 64), (24, 64), (33, 192), (130, 320), (9, 4160)])
def test_pack_and_unpack(cuda_device, t, width):
    rng = np.random.default_rng(width)
    bits = odd_values(rng, t, width)
    x = bf16_from_bits(bits)
    p = packed_rows(t, width)
    zb.zb_op_checkpoint_pack(x, p, t, width)
    codes, scales = O.pack(f64_from_bf16(x))
    assert np.array_equal(take(p[1], t), scales)
    assert np.array_equal(take(p[0], t), codes)
    back = out_rows(t, width)
    zb.zb_op_checkpoint_unpack(p, back, t, width)
    np.testing.assert_array_equal(take(back, t), O.unpack(codes, scales))


def test_unpack_any_bytes(cuda_device):
    t, width = 64, 256
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 256, (t, width)).astype(np.uint8)
    scales = rng.integers(0, 249, (t, width // 32)).astype(np.uint8)
    back = out_rows(t, width)
    zb.zb_op_checkpoint_unpack((torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()), back, t, width)
    np.testing.assert_array_equal(take(back, t), O.unpack(codes, scales))


@pytest.mark.parametrize("t,k,n", [(1, 64, 64), (63, 128, 64), (64, 64, 128), (65, 320, 192), (700, 512, 256), (513, 1088, 320),
                                   (1500, 256, 576), (4200, 64, 128), (64, 2624, 2688)])
def test_weight_from_8_bits(cuda_device, t, k, n):
    rng = np.random.default_rng(t + k)
    db, dy = draw_bf16(rng, (t, n))
    _, x = draw_bf16(rng, (t, k))
    codes, scales = O.pack(x)
    before, dw = draw_f32(rng, n, k)
    guard = torch.full((n + GUARD, k), 77.0, device="cuda")
    guard[:n] = dw
    p = (torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    scratch = scratch_of(zb.zb_op_backward_weight_checkpoint_scratch_bytes(t, k))
    zb.zb_op_backward_weight_checkpoint(bf16_from_bits(db), p, guard, t, k, n, scratch)
    v = O.unpack(codes, scales)
    slip = product_slip(np.abs(dy).T @ np.abs(v), t, 512)
    ref = before + dy.T @ v
    within(take(guard, n), ref, slip + 2.0 ** -23 * (np.abs(before) + np.abs(ref)), "dw")
    again = f32(before)
    zb.zb_op_backward_weight_checkpoint(bf16_from_bits(db), p, again, t, k, n, scratch)
    assert torch.equal(again, guard[:n])
    no_waits_ran_out()


# ---------------------------------------------------------------- norms around a block


def norm_case(rng, t, w, post, pre, gate, beta, a, b):
    par, dev = {}, {}
    for k, kind in (("post", post), ("pre", pre)):
        for name, scale, mid in (("_gamma", 0.1, 1.0), ("_beta", 0.1, 0.0)):
            if kind == "none" or (name == "_beta" and not (beta and kind == "layer")):
                par[k + name] = dev[k + name] = None
                continue
            v = (mid + scale * rng.standard_normal(w)).astype(np.float32)
            par[k + name], dev[k + name] = v.astype(np.float64), torch.from_numpy(v).cuda()
    par["gate"] = dev["gate"] = None
    if gate == "channel":
        par["gate"], dev["gate"] = draw_f32(rng, w)
    if gate == "token":
        bits, par["gate"] = draw_bf16(rng, (t, w))
        dev["gate"] = bf16_from_bits(bits)
    a, b = float(np.float32(a)), float(np.float32(b))
    eps = float(np.float32(1e-5))
    op = zb.make_residual_norm(post=post, pre=pre, gate_kind=gate, residual_scale=a, branch_scale=b, post_eps=eps, pre_eps=eps,
                               **dev)
    return op, O.ResidualNorm(post, pre, a=a, b=b, post_eps=eps, pre_eps=eps, **par)


NORMS = [("rms", "rms", "channel", False), ("layer", "layer", "token", True), ("none", "layer", "channel", False),
         ("rms", "none", "token", False), ("layer", "none", "none", True), ("none", "none", "channel", False),
         ("none", "rms", "none", False)]
SIZES = [(1, 64), (5, 192), (3, 256), (9, 320), (6, 576), (130, 1024), (7, 1088), (4, 2112), (5, 4096), (3, 4160), (2, 8256),
         (2, 16448), (1, 32768)]


def size_of(values, kind, gamma, beta):
    """Bound of a norm's terms: how large gamma (v - mean) rstd + beta gets before anything cancels."""
    if kind == "none":
        return np.abs(values)
    mean, rstd = O.norm_stats(values, kind, 1e-5)
    s = np.abs(gamma) * (np.abs(values) + np.abs(mean)[:, None]) * rstd[:, None]
    return s if beta is None else s + np.abs(beta)


@pytest.mark.parametrize("t,w", SIZES)
@pytest.mark.parametrize("post,pre,gate,beta", NORMS)
def test_residual_norm(cuda_device, t, w, post, pre, gate, beta):
    """F, B and W.  Sums over a row of w float32 terms go through 32 in a thread and a tree: 45 2^-24 of the sum of
    magnitudes, which 2^-18 of each term covers; statistics likewise."""
    rng = np.random.default_rng(t + w)
    a, b = (1.0, 0.5) if w % 128 else (0.7, 1.0)
    op, ref = norm_case(rng, t, w, post, pre, gate, beta, a, b)
    xb, x = draw_bf16(rng, (t, w), std=3.0)
    yb, y = draw_bf16(rng, (t, w))
    y = y + 2.0
    yb = y.astype(np.float32)
    yd = torch.from_numpy(yb).cuda().to(torch.bfloat16)
    y = f64_from_bf16(yd)
    xd = bf16_from_bits(xb)
    a, b = ref.a, ref.b
    h, n, stats = out_rows(t, w), out_rows(t, w) if pre != "none" else None, out_rows(t, 4, torch.float32)
    n8 = packed_rows(t, w) if pre != "none" else None
    zb.zb_op_residual_norm_forward(op, xd, yd, h, n, stats, t, w, n_packed=n8)
    fine = 2.0 ** -18
    gate_size = 1.0 if ref.gate is None else np.abs(ref.gate)
    usize = size_of(y, post, ref.post_gamma, ref.post_beta)
    want = ref.h(x, y)
    within(take(h, t), want, HALF * np.abs(want) + fine * (abs(a) * np.abs(x) + abs(b) * gate_size * usize), "h")
    hh = take(h, t)
    st = take(stats, t)
    for at, v, kind, eps in ((0, y, post, ref.post_eps), (2, hh, pre, ref.pre_eps)):
        mean, rstd = O.norm_stats(v, kind, eps)
        within(st[:, at], mean, fine * np.abs(v).mean(1), "mean")
        within(st[:, at + 1], rstd, fine * rstd, "rstd")
    if pre != "none":
        want = ref.n(hh)
        within(take(n, t), want, HALF * np.abs(want) + fine * size_of(hh, pre, ref.pre_gamma, ref.pre_beta), "n")
        codes, scales = O.pack(take(n, t))
        assert np.array_equal(take(n8[0], t), codes) and np.array_equal(take(n8[1], t), scales)
        only = packed_rows(t, w)
        zb.zb_op_residual_norm_forward(op, xd.clone(), yd, out_rows(t, w), None, out_rows(t, 4, torch.float32), t, w, n_packed=only)
        assert torch.equal(only[0], n8[0]) and torch.equal(only[1], n8[1])
    # in place over the residual stream
    over = xd.clone()
    zb.zb_op_residual_norm_forward(op, over, yd, over, n, stats, t, w)
    assert torch.equal(over, h[:t])

    # B
    rb, dres = draw_bf16(rng, (t, w))
    nb, dn = draw_bf16(rng, (t, w))
    dn = dn if pre != "none" else None
    dnd = bf16_from_bits(nb) if pre != "none" else None
    dresd = bf16_from_bits(rb)
    dh, dx, dy = (out_rows(t, w) for _ in range(3))
    dgate = out_rows(t, w) if gate == "token" else None
    zb.zb_op_residual_norm_backward_input(op, dnd, dresd, h[:t], yd, stats, dh, dy, t, w, dx=dx, dgate=dgate)
    got = ref.backward(dn, dres, hh, y)
    # what the terms of the two norms' backwards are made of, before they cancel
    def mass(d, v, kind, gamma):
        if kind == "none":
            return np.abs(d)
        mean, rstd = O.norm_stats(v, kind, 1e-5)
        hat = (np.abs(v) + np.abs(mean)[:, None]) * rstd[:, None]
        g = np.abs(d) * np.abs(gamma)
        return rstd[:, None] * (g + (hat + 1e-3) * (g * hat).mean(1, keepdims=True) + g.mean(1, keepdims=True))
    dsize = np.abs(dres) + (mass(dn, hh, pre, ref.pre_gamma) if pre != "none" else 0.0)
    within(take(dh, t), got["dh"], HALF * np.abs(got["dh"]) + fine * dsize, "dh")
    within(take(dx, t), got["dx"], HALF * np.abs(got["dx"]) + fine * abs(a) * dsize, "dx")
    if gate == "token":
        bar = HALF * np.abs(got["dgate"]) + 2 * fine * abs(b) * (dsize + np.abs(got["dh"])) * usize
        within(take(dgate, t), got["dgate"], bar, "dgate")
    bar = HALF * np.abs(got["dy"]) + 2 * fine * mass(abs(b) * gate_size * (dsize + np.abs(got["dh"])), y, post, ref.post_gamma)
    within(take(dy, t), got["dy"], bar, "dy")
    # dh over dres, no dx; and no gradient on the skip path
    over, dy2 = dresd.clone(), out_rows(t, w)
    zb.zb_op_residual_norm_backward_input(op, dnd, over, h[:t], yd, stats, over, dy2, t, w)
    assert torch.equal(over, dh[:t]) and torch.equal(dy2, dy)
    if pre != "none":
        alone, zero = out_rows(t, w), out_rows(t, w)
        zb.zb_op_residual_norm_backward_input(op, dnd, None, h[:t], yd, stats, alone, dy2, t, w)
        zb.zb_op_residual_norm_backward_input(op, dnd, torch.zeros_like(dresd), h[:t], yd, stats, zero, dy2, t, w)
        assert torch.equal(alone, zero)

    # W, from the stored dh
    dhh = take(dh, t)
    got = ref.backward(dn, dres, hh, y, dh=dhh)
    names = [k for k, v in (("dpost_gamma", ref.post_gamma), ("dpost_beta", ref.post_beta), ("dpre_gamma", ref.pre_gamma),
                            ("dpre_beta", ref.pre_beta)) if v is not None] + (["dgate"] if gate == "channel" else [])
    if not names:
        return
    grads, before = {}, {}
    for k in names:
        before[k], grads[k] = draw_f32(rng, w)
    scratch = scratch_of(zb.zb_op_residual_norm_backward_weight_scratch_bytes(t, w))
    zb.zb_op_residual_norm_backward_weight(op, dnd, h[:t], dh[:t], yd, stats, t, w, scratch, **grads)
    sums = {"dgate": np.abs(b * dhh) * usize, "dpre_beta": 0.0 if dn is None else np.abs(dn),
            "dpost_beta": np.abs(b * dhh) * gate_size}
    for k, v, kind, d in (("dpost_gamma", y, post, np.abs(b * dhh) * gate_size), ("dpre_gamma", hh, pre, dn)):
        if kind != "none":
            mean, rstd = O.norm_stats(v, kind, 1e-5)
            sums[k] = np.abs(d) * (np.abs(v) + np.abs(mean)[:, None]) * rstd[:, None]
    for k in names:
        want = (got[k].sum(0) if k == "dgate" else got[k])
        bar = (fine + t * 2.0 ** -24) * sums[k].sum(0) + 2.0 ** -22 * np.abs(before[k])
        within(grads[k].cpu().numpy(), before[k] + want, bar, k)
    # one gradient at a time: the same bits
    for k in names:
        one = f32(before[k])
        zb.zb_op_residual_norm_backward_weight(op, dnd, h[:t], dh[:t], yd, stats, t, w, scratch, **{k: one})
        assert torch.equal(one, grads[k]), k


@pytest.mark.parametrize("w", [64, 320, 4096, 4160, 11712])
def test_layer_norm_of_constant_rows(cuda_device, w):
    """A row of one value is its mean: the sum of w < 2^14 equal numbers of 8 bits is exact in float32, and so is its w-th part.
    The normed row is then 0, whatever the value: what is left is beta, rounded once, and gamma gets no gradient."""
    rng = np.random.default_rng(w)
    values = torch.tensor([1000.0, -0.37, 5e4, 0.0, 3e-5, -2.5], device="cuda").to(torch.bfloat16)
    t = values.numel()
    rows, zero = values[:, None].expand(t, w).contiguous(), torch.zeros(t, w, dtype=torch.bfloat16, device="cuda")
    gamma, beta = draw_f32(rng, w)[1], draw_f32(rng, w)[1]
    want = beta.to(torch.bfloat16).expand(t, w)
    op = zb.make_residual_norm(post="layer", post_gamma=gamma, post_beta=beta)
    h, stats, dy, dh = out_rows(t, w), out_rows(t, 4, torch.float32), out_rows(t, w), out_rows(t, w)
    zb.zb_op_residual_norm_forward(op, zero, rows, h, None, stats, t, w)
    assert torch.equal(h[:t], want) and torch.equal(stats[:t, 0], values.float())
    before = draw_f32(rng, w)[1]
    got, d = before.clone(), bf16_from_bits(draw_bf16(rng, (t, w))[0])
    scratch = scratch_of(zb.zb_op_residual_norm_backward_weight_scratch_bytes(t, w))
    zb.zb_op_residual_norm_backward_weight(op, None, None, d, rows, stats, t, w, scratch, dpost_gamma=got)
    assert torch.equal(got, before)
    op = zb.make_residual_norm(pre="layer", pre_gamma=gamma, pre_beta=beta)
    n = out_rows(t, w)
    zb.zb_op_residual_norm_forward(op, rows, zero, h, n, stats, t, w)
    assert torch.equal(h[:t], rows) and torch.equal(n[:t], want)
    got = before.clone()
    zb.zb_op_residual_norm_backward_weight(op, d, rows, None, None, stats, t, w, scratch, dpre_gamma=got)
    assert torch.equal(got, before)
    # dh over dn
    zb.zb_op_residual_norm_backward_input(op, d, zero, rows, None, stats, dh, dy, t, w)
    over = d.clone()
    zb.zb_op_residual_norm_backward_input(op, over, zero, rows, None, stats, over, dy, t, w)
    assert torch.equal(over, dh[:t])


def test_no_rows(cuda_device):
    op = zb.make_residual_norm(post="rms", post_gamma=torch.ones(64, device="cuda"))
    g = torch.ones(64, device="cuda")
    w = torch.zeros(64, 64, device="cuda").to(torch.bfloat16)
    nothing = (None, None)
    zb.zb_op_residual_norm_forward(op, None, None, None, None, None, 0, 64)
    zb.zb_op_residual_norm_backward_input(op, None, None, None, None, None, None, None, 0, 64)
    zb.zb_op_residual_norm_backward_weight(op, None, None, None, None, None, 0, 64, None, dpost_gamma=g)
    zb.zb_op_linear_activation_forward(None, w, None, None, None, 0, 64, 64, "gelu")
    zb.zb_op_backward_input_activation(None, w, None, None, 0, 64, 64, "gelu", dbias=g)
    zb.zb_op_activation_backward(None, None, None, 0, 64, "gelu")
    zb.zb_op_backward_bias(None, g, 0, 64, None)
    zb.zb_op_checkpoint_pack(None, nothing, 0, 64)
    zb.zb_op_checkpoint_unpack(nothing, None, 0, 64)
    zb.zb_op_backward_weight_checkpoint(None, nothing, torch.ones(64, 64, device="cuda"), 0, 64, 64, None)
    assert torch.all(g == 1.0)
    no_waits_ran_out()
