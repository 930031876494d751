"""GPU parity of the rotary positions against the float64 oracle.

Bar per element: the result's bf16 rounding, 2^-8 of its value (torch.finfo(bf16).eps / 2), plus the float32
arithmetic before it.  Cosine and sine carry at most 2^-22 (the angle's rounding to a float32 fraction of a turn, pi
2^-24, and two units of sincospi), products and the sum 2^-23 more: 2^-21 g (|a| + |b|) bounds it.
"""
import numpy as np
import pytest
import torch

from backward_split_linear_gb300 import binding as zb
from backward_split_linear_gb300.runtime import bf16_from_bits, f64_from_bf16
from oracle import train_ops as O
from parity import draw_bf16

pytestmark = pytest.mark.gpu


def turns_on_device(turns):
    return torch.from_numpy(np.array(turns, dtype=np.uint64).view(np.int64)).cuda()


def assert_rotated(got, ref, x, r, pairs, g):
    """The bar of the module's docstring; |a| + |b| of each element's pair."""
    size = np.abs(x[..., :r])
    if pairs == "half":
        s = size[..., : r // 2] + size[..., r // 2:]
        s = np.concatenate([s, s], axis=-1)
    else:
        s = np.repeat(size[..., 0::2] + size[..., 1::2], 2, axis=-1)
    bar = 2.0 ** -8 * np.abs(ref[..., :r]) + 2.0 ** -21 * g * s
    assert np.all(np.abs(got[..., :r] - ref[..., :r]) <= bar)
    assert np.array_equal(got[..., r:], x[..., r:])  # what does not turn passes unchanged


CASES = [  # tokens, heads, d, rotary, pairs, scaling
    (1, 3, 64, 64, "half", "none"), (1, 1, 64, 16, "interleaved", "none"), (7, 6, 64, 48, "half", "linear"),
    (129, 40, 128, 128, "half", "banded"), (130, 10, 128, 64, "interleaved", "yarn"), (513, 9, 64, 32, "interleaved", "ntk"),
    (33, 2, 160, 144, "half", "yarn"), (5, 4, 1024, 1024, "interleaved", "none"),
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("t,n,d,r,pairs,scaling", CASES)
def test_against_the_oracle(cuda_device, t, n, d, r, pairs, scaling, backward):
    rng = np.random.default_rng(t + d + r)
    bits, x = draw_bf16(rng, (t, n * d))
    high = 4.0 if scaling == "banded" else 32.0
    kw = dict(scaling=scaling, factor=1.0 if scaling == "none" else 8.0, context=8192.0)
    turns, g = zb.zb_rotary_frequencies(r, 10000.0, **kw)
    f, g_ref = O.rotary_frequencies(r, 10000.0, high=high, **kw)
    assert abs(g - g_ref) <= 2.0 ** -24 * g_ref
    positions = rng.integers(-(1 << 31), 1 << 31, t)
    positions[0] = 0
    y = torch.full((t, n * d), float("nan"), dtype=torch.bfloat16, device="cuda")
    op = zb.zb_op_rotary_backward if backward else zb.zb_op_rotary_forward
    op(bf16_from_bits(bits), y, torch.from_numpy(positions.astype(np.int32)).cuda(), turns_on_device(turns), g, t, n, d, r,
       pairs)
    # f is a float64, off by 2^-53 of itself, and the table by 2^-65 turns a position: at 2^31 positions 2^-22 radians
    xs = x.reshape(t, n, d)
    ref = O.rotary(xs, positions, f, g, pairs, backward)
    assert_rotated(f64_from_bf16(y).reshape(t, n, d), ref, xs, r, pairs, g)


def test_in_place_on_the_heads_of_qkv(cuda_device):
    """In place and out of place give the same bits; the value heads stay; positions default to the row number."""
    t, nh, nkv, d = 300, 6, 3, 64
    rng = np.random.default_rng(5)
    bits, x = draw_bf16(rng, (t, (nh + 2 * nkv) * d))
    turns, g = zb.zb_rotary_frequencies(d)
    dev = turns_on_device(turns)
    qkv = bf16_from_bits(bits)
    y = torch.zeros(t, (nh + nkv) * d + 64, dtype=torch.bfloat16, device="cuda")
    rows = torch.arange(t, dtype=torch.int32, device="cuda")
    w = (nh + 2 * nkv) * d
    zb.zb_op_rotary_forward(qkv, y, rows, dev, g, t, nh + nkv, d, d, ld_x=w, ld_y=y.shape[1])
    zb.zb_op_rotary_forward(qkv, qkv, None, dev, g, t, nh + nkv, d, d, ld_x=w, ld_y=w)
    assert torch.equal(qkv[:, : (nh + nkv) * d], y[:, : (nh + nkv) * d])
    assert torch.equal(qkv[:, (nh + nkv) * d:], bf16_from_bits(bits)[:, (nh + nkv) * d:])
    assert torch.all(y[:, (nh + nkv) * d:] == 0)
    # the backward is the inverse of the forward (g = 1): two roundings
    zb.zb_op_rotary_backward(qkv, qkv, None, dev, g, t, nh + nkv, d, d, ld_x=w, ld_y=w)
    back = f64_from_bf16(qkv)
    s = np.abs(x).reshape(t, -1, 2, d // 2)
    size = np.concatenate([s.sum(2)] * 2, axis=-1).reshape(t, w)
    assert np.all(np.abs(back - x) <= 2.0 ** -8 * np.abs(back) + 2.0 ** -8 * 2 * size)


def test_gradient_against_differences(cuda_device):
    """<R x, dy> = <x, R^T dy>: the backward is the forward's transpose, up to the bf16 roundings of both."""
    t, n, d, r = 64, 4, 64, 32
    rng = np.random.default_rng(8)
    xb, x = draw_bf16(rng, (t, n * d))
    db, dy = draw_bf16(rng, (t, n * d))
    turns, g = zb.zb_rotary_frequencies(r, scaling="yarn", factor=4.0, context=2048.0)
    dev = turns_on_device(turns)
    y, dx = (torch.empty(t, n * d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    zb.zb_op_rotary_forward(bf16_from_bits(xb), y, None, dev, g, t, n, d, r, "interleaved")
    zb.zb_op_rotary_backward(bf16_from_bits(db), dx, None, dev, g, t, n, d, r, "interleaved")
    y, dx = f64_from_bf16(y), f64_from_bf16(dx)
    bar = 2.0 ** -8 * (np.sum(np.abs(y * dy)) + np.sum(np.abs(x * dx)))
    assert abs(np.sum(y * dy) - np.sum(x * dx)) <= bar


def test_no_rows_and_another_stream(cuda_device):
    turns, g = zb.zb_rotary_frequencies(64)
    dev = turns_on_device(turns)
    zb.zb_op_rotary_forward(None, None, None, dev, g, 0, 4, 64, 64)
    x = torch.randn(50, 256, device="cuda").to(torch.bfloat16)
    y, z = torch.empty_like(x), torch.empty_like(x)
    zb.zb_op_rotary_forward(x, y, None, dev, g, 50, 4, 64, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    zb.zb_op_rotary_forward(x, z, None, dev, g, 50, 4, 64, 64, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, z)
