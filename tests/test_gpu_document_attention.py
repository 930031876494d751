"""GPU parity of the document attention (forward, backward, plan) against float64.

The plain form below is dense torch float64 on the GPU, from the definition; tests/test_train_ops_cpu.py ties the
numpy oracle to differences and this form to the oracle.  Bar per step: the one of the causal core (tests/parity.py),
relative Frobenius <= 5e-3 and max-abs <= 2e-2 max|ref|: the same roundings (P and dS to bf16, the results to bf16).
lse: float32 sums of products of at most 2^7 terms, each term's rounding 2^-24 of partial sums below 2^6 here, and
exponentials good to 2^-22: 2^-11 bounds it.
"""
import math

import numpy as np
import pytest
import torch

from backward_split_linear_gb300 import binding as zb
from backward_split_linear_gb300.runtime import bf16_from_bits
from oracle import train_ops as O
from parity import FRO_TOL, MAX_TOL, draw_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status_clean(cuda_device):
    zb.zb_device_status(reset=True)
    yield
    st, code = zb.zb_device_status()
    assert st == 0, f"device status word set: {code}"


def ints(values):
    return None if values is None else torch.tensor(values, dtype=torch.int32, device="cuda")


def make_plan(t, offsets, prefix=None, n_docs=None, positions=None):
    plan = torch.full((zb.zb_op_attention_document_plan_bytes(t),), 0xEE, dtype=torch.uint8, device="cuda")
    n = n_docs if n_docs is not None else (1 if offsets is None else len(offsets) - 1)
    zb.zb_op_attention_document_plan(ints(offsets), ints(prefix), n, t, plan, plan.numel(), positions)
    return plan


def forward(qkv, t, nh, nkv, d, plan, cap=0.0, slopes=None, stream=None, a=None):
    a = torch.full((t, nh * d), float("nan"), dtype=torch.bfloat16, device="cuda") if a is None else a
    lse = torch.full((nh, zb.zb_op_attention_stat_stride(t)), float("nan"), device="cuda")
    zb.zb_op_attention_document_forward(qkv, a, lse, plan, slopes, cap, t, nh, nkv, d, stream)
    return a, lse


def backward(qkv, a, da, lse, t, nh, nkv, d, plan, cap=0.0, slopes=None, stream=None):
    dqkv = torch.full((t, (nh + 2 * nkv) * d), float("nan"), dtype=torch.bfloat16, device="cuda")
    scratch = torch.full((zb.zb_op_attention_document_scratch_bytes(t, nh),), 0xEE, dtype=torch.uint8, device="cuda")
    zb.zb_op_attention_document_backward(qkv, a, da, lse, dqkv, plan, slopes, cap, t, nh, nkv, d, scratch, scratch.numel(),
                                         stream)
    return dqkv


def visible(t, offsets, prefix=None):
    i = torch.arange(t, device="cuda")
    off = torch.tensor(offsets, device="cuda")
    doc = torch.searchsorted(off, i, right=True) - 1
    live = (doc >= 0) & (doc < len(offsets) - 1)
    doc = doc.clamp(0, len(offsets) - 2)
    see = i[None, :] <= i[:, None]
    if prefix is not None:
        see = see | ((i - off[doc]) < torch.tensor(prefix, device="cuda")[doc])[None, :]
    return see & (doc[:, None] == doc[None, :]) & live[:, None] & live[None, :]


def reference(qkv, nh, nkv, d, see, cap=0.0, slopes=None, da=None):
    """(a, lse) and, with da, dqkv: float64, dense, hidden values replaced by zeros first."""
    t = qkv.shape[0]
    x = qkv.double().view(t, nh + 2 * nkv, d)
    q, k, v = x[:, :nh].transpose(0, 1), x[:, nh:nh + nkv].transpose(0, 1), x[:, nh + nkv:].transpose(0, 1)
    k, v = (y.repeat_interleave(nh // nkv, 0) for y in (k, v))
    s = q @ k.transpose(1, 2) / math.sqrt(d)
    deriv = 1.0
    if cap:
        r = torch.tanh(s / cap)
        s, deriv = cap * r, 1.0 - r * r
    if slopes is not None:
        i = torch.arange(t, device="cuda")
        s = s - slopes.double()[:, None, None] * (i[:, None] - i[None, :]).abs()
    s = s.masked_fill(~see, -math.inf)
    top = s.amax(2, keepdim=True).clamp(min=-1e300)
    p = torch.exp(s - top)
    total = p.sum(2, keepdim=True)
    lse = ((top + torch.log(total)) / math.log(2.0))[..., 0]
    p = p / total.clamp(min=1e-300)
    a = (p @ v).transpose(0, 1).reshape(t, nh * d)
    if da is None:
        return a, lse
    dy = da.double().view(t, nh, d).transpose(0, 1)
    dp = dy @ v.transpose(1, 2)
    ds = p * (dp - (p * dp).sum(2, keepdim=True)) * deriv / math.sqrt(d)
    fold = lambda y: y.view(nkv, nh // nkv, t, d).sum(1)  # noqa: E731
    out = torch.cat([ds @ k, fold(ds.transpose(1, 2) @ q), fold(p.transpose(1, 2) @ dy)], 0)
    return a, lse, out.transpose(0, 1).reshape(t, (nh + 2 * nkv) * d)


def cancelled(qkv, a, da, nh, d):
    """What is left of dq and dk where the formula gives zero (a row that sees one key: P = 1 and dP = D).  dP and D are
    float32 sums of the same d products in two orders: each is off by at most d 2^-24 of the sum of their sizes, and the
    difference meets a query or key, and the scale."""
    sums = (da.double() * a.double()).abs().view(da.shape[0], nh, d).sum(2).max()
    return float(2 * d * 2.0 ** -24 * sums * qkv.double().abs().max() / math.sqrt(d))


def assert_near(got, ref, what, floor=0.0):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    norm, top = float(ref.norm()), float(ref.abs().max()) if ref.numel() else 0.0
    d = got - ref
    if norm == 0.0:
        assert not d.numel() or float(d.abs().max()) <= floor, what
        return
    assert float(d.norm()) <= FRO_TOL * norm and float(d.abs().max()) <= MAX_TOL * top, \
        f"{what}: {float(d.norm()) / norm:.2e}, {float(d.abs().max()) / top:.2e}"


def assert_lse(lse, ref, t):
    got = lse[:, :t].double()
    assert torch.equal(torch.isneginf(got), torch.isneginf(ref))
    live = ~torch.isneginf(ref)
    if live.any():
        assert float((got - ref)[live].abs().max()) <= 2.0 ** -11


def draw(seed, t, nh, nkv, d, q_scale=1.0):
    rng = np.random.default_rng(seed)
    bits, _ = draw_bf16(rng, (t, (nh + 2 * nkv) * d))
    qkv = bf16_from_bits(bits)
    qkv[:, : nh * d] *= q_scale
    dbits, _ = draw_bf16(rng, (t, nh * d))
    return qkv, bf16_from_bits(dbits)


def slopes_of(nh):
    return torch.exp2(-6.0 * torch.arange(1, nh + 1, device="cuda") / nh)


def both_ways(seed, t, nh, nkv, d, offsets, prefix=None, cap=0.0, bias=False):
    """Forward and backward of one case against the plain form."""
    qkv, da = draw(seed, t, nh, nkv, d, 2.0 if cap else 1.0)
    slopes = slopes_of(nh) if bias else None
    plan = make_plan(t, offsets, prefix)
    a, lse = forward(qkv, t, nh, nkv, d, plan, cap, slopes)
    see = visible(t, [0, t] if offsets is None else offsets, prefix)
    ra, rl, rd = reference(qkv, nh, nkv, d, see, cap, slopes, da)
    assert_near(a, ra, "a")
    assert_lse(lse, rl, t)
    dqkv = backward(qkv, a, da, lse, t, nh, nkv, d, plan, cap, slopes)
    w, kw = nh * d, nkv * d
    floor = cancelled(qkv, a, da, nh, d)
    assert_near(dqkv[:, :w], rd[:, :w], "dq", floor)
    assert_near(dqkv[:, w:w + kw], rd[:, w:w + kw], "dk", floor)
    assert_near(dqkv[:, w + kw:], rd[:, w + kw:], "dv")
    dead = ~see.any(1)
    assert torch.all(a[dead] == 0) and torch.all(dqkv[dead] == 0)


LAYOUTS = [  # tokens, nh, nkv, d, offsets, prefix
    (1, 2, 1, 64, None, None),
    (1, 3, 3, 128, [0, 1], [1]),
    (3, 4, 2, 64, [0, 1, 2, 3], None),                              # documents of one token
    (127, 2, 2, 128, None, None),
    (128, 4, 1, 64, [0, 128], [128]),                               # everything sees everything
    (129, 4, 2, 128, [0, 0, 128, 128, 129], [3, 1, 0, 5]),          # empty documents, a prefix past the end
    (300, 6, 2, 64, [7, 100, 290], [20, 0]),                        # padding at both ends
    (513, 8, 2, 128, [0, 130, 131, 400, 513], None),
    (640, 5, 5, 64, [0, 640], [200]),
    (700, 16, 2, 128, [0, 64, 128, 192, 256, 500, 640], [1, 64, 63, 0, 150, 7]),
    (1100, 3, 1, 128, [0, 900, 1050], [-4, 33]),                    # a negative prefix, odd group
    (1500, 2, 1, 64, None, [700]),
]


@pytest.mark.parametrize("mode", ["plain", "cap", "bias", "cap+bias"])
@pytest.mark.parametrize("case", range(len(LAYOUTS)))
def test_forward_and_backward(case, mode):
    t, nh, nkv, d, offsets, prefix = LAYOUTS[case]
    both_ways(200 + case, t, nh, nkv, d, offsets, prefix, 3.0 if "cap" in mode else 0.0, "bias" in mode)


@pytest.mark.parametrize("mode", ["plain", "cap", "bias"])
def test_many_documents_of_every_length(mode):
    """Documents of 0 to 300 rows, so that every offset inside a tile starts one somewhere."""
    rng = np.random.default_rng(4)
    cuts = np.cumsum(np.concatenate([[5], rng.integers(0, 300, 24)])).tolist()
    both_ways(7, cuts[-1] + 61, 4, 2, 64, cuts, rng.integers(0, 40, 24).tolist(), 4.0 if mode == "cap" else 0.0, mode == "bias")


@pytest.mark.parametrize("mode", ["plain", "cap", "bias"])
@pytest.mark.parametrize("d", [64, 128])
def test_long_rows(mode, d):
    both_ways(9 + d, 4500, 2, 1, d, [0, 4400], [100], 6.0 if mode == "cap" else 0.0, mode == "bias")


def test_equals_the_causal_core_in_one_document():
    """The same formula as the causal core: both within one bar of float64, so within two of each other."""
    t, nh, nkv, d = 900, 4, 2, 128
    qkv, _ = draw(1, t, nh, nkv, d)
    a, lse = forward(qkv, t, nh, nkv, d, make_plan(t, None))
    b, lse_b = torch.empty_like(a), torch.zeros_like(lse)
    zb.zb_op_attention_causal_forward(qkv, b, lse_b, t, nh, nkv, d)
    assert float((a.double() - b.double()).norm()) <= 2 * FRO_TOL * float(b.double().norm())
    assert float((lse - lse_b)[:, :t].abs().max()) <= 2.0 ** -10


def test_large_scores_and_rising_maxima():
    """Scores in the hundreds that rise along the keys, for every other row: the running maximum moves all the way.  The
    softmax is nearly one-hot, so a alone is compared (dq and dk cancel)."""
    t, nh, nkv, d = 1024, 2, 1, 64
    rng = np.random.default_rng(2)
    sign = np.where(np.arange(t) % 2 == 0, 8.0, -8.0)
    q = sign[:, None] + 0.05 * rng.standard_normal((t, d))
    k = 5.0 * np.arange(t)[:, None] / t + 0.05 * rng.standard_normal((t, d))
    x = torch.from_numpy(np.concatenate([q, q, k, rng.standard_normal((t, d))], 1)).cuda().to(torch.bfloat16)
    offsets = [0, 300, 1024]
    for cap in (0.0, 400.0):
        a, _ = forward(x, t, nh, nkv, d, make_plan(t, offsets), cap)
        ra, _ = reference(x, nh, nkv, d, visible(t, offsets), cap)
        assert_near(a, ra, "a")


@pytest.mark.parametrize("cap,q_scale", [(1e-3, 2.0 ** -10), (1e-3, 1.0), (512.0, 32.0), (512.0, 256.0)])
@pytest.mark.parametrize("d", [64, 128])
def test_the_smallest_and_the_largest_cap(cap, q_scale, d):
    """Scores below the cap and far above it.  Scores around 512 leave a nearly one-hot softmax, whose dq and dk cancel:
    there a alone is compared."""
    t, nh, nkv, offsets = 600, 2, 1, [0, 350, 600]
    qkv, da = draw(31, t, nh, nkv, d, q_scale)
    see, plan = visible(t, offsets), make_plan(t, offsets)
    a, lse = forward(qkv, t, nh, nkv, d, plan, cap)
    ra, _, rd = reference(qkv, nh, nkv, d, see, cap, None, da)
    assert_near(a, ra, "a")
    if cap < 1.0:
        assert_near(backward(qkv, a, da, lse, t, nh, nkv, d, plan, cap), rd, "dqkv")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (5.0, False), (0.0, True)])
@pytest.mark.parametrize("d", [64, 128])
def test_values_that_are_not_finite_stay_where_they_are_seen(bad, cap, bias, d):
    """Padding rows and a whole document hold bad values, in the same tiles as clean rows; the clean documents' results
    are those of clean inputs.  A bad key and value at a document's end reach the rows from there on only."""
    t, nh, nkv = 420, 4, 2
    offsets, prefix = [10, 150, 200, 400], [5, 0, 9]
    qkv, da = draw(3, t, nh, nkv, d, 2.0 if cap else 1.0)
    slopes = slopes_of(nh) if bias else None
    see = visible(t, offsets, prefix)
    ra, rl, rd = reference(qkv, nh, nkv, d, see, cap, slopes, da)
    x, dy = qkv.clone(), da.clone()
    for rows in (slice(0, 10), slice(150, 200), slice(400, 420)):
        x[rows], dy[rows] = bad, bad
    plan = make_plan(t, offsets, prefix)
    a, lse = forward(x, t, nh, nkv, d, plan, cap, slopes)
    clean = torch.cat([torch.arange(10, 150), torch.arange(200, 400)]).cuda()
    assert_near(a[clean], ra[clean], "a")
    assert_lse(lse[:, clean], rl[:, clean], clean.numel())
    dqkv = backward(x, a, dy, lse, t, nh, nkv, d, plan, cap, slopes)
    assert_near(dqkv[clean], rd[clean], "dqkv")
    assert torch.all(a[:10] == 0) and torch.all(dqkv[400:] == 0)
    # the last key and value of the first document
    x = qkv.clone()
    x[149, nh * d:] = bad
    a, lse = forward(x, t, nh, nkv, d, plan, cap, slopes)
    keep = torch.cat([torch.arange(10, 149), torch.arange(150, 400)]).cuda()
    assert_near(a[keep], ra[keep], "a")
    assert not torch.isfinite(a[149].float()).any()
    # a bad gradient and query of one row: the keys it does not see, and every other row's dq, stay clean
    x, dy = qkv.clone(), da.clone()
    a, lse = forward(x, t, nh, nkv, d, plan, cap, slopes)
    dy[220] = bad
    dqkv = backward(x, a, dy, lse, t, nh, nkv, d, plan, cap, slopes)
    others = torch.tensor([i for i in range(t) if i != 220], device="cuda")
    assert_near(dqkv[others][:, : nh * d], rd[others][:, : nh * d], "dq")
    unseen = torch.cat([torch.arange(10, 200), torch.arange(221, 400)]).cuda()
    assert_near(dqkv[unseen][:, nh * d:], rd[unseen][:, nh * d:], "dk, dv")


@pytest.mark.parametrize("d", [64, 128])
def test_long_rows_with_values_that_are_not_finite(d):
    """One infinite value that every row sees sends every row to the pass over its own pairs: 12000 keys a row.  The
    other columns are those of clean inputs; batches of nothing but NaN give NaN, and end soon."""
    t, nh, nkv = 12000, 2, 1
    qkv, da = draw(21, t, nh, nkv, d)
    plan = make_plan(t, None)
    x = qkv.clone()
    x[0, (nh + nkv) * d] = float("inf")
    a, lse = forward(x, t, nh, nkv, d, plan)
    b, lse_b = forward(qkv, t, nh, nkv, d, plan)
    a3, b3 = a.view(t, nh, d), b.view(t, nh, d)
    assert torch.isposinf(a3[:, :, 0]).all()
    # both within one bar of the same numbers
    assert float((a3[:, :, 1:].double() - b3[:, :, 1:].double()).norm()) <= 2 * FRO_TOL * float(b3.double().norm())
    assert float((lse - lse_b)[:, :t].abs().max()) <= 2.0 ** -10
    dy = da.clone()
    dy[:, ::d] = 0.0  # the infinite column's gradient: 0 times infinity is NaN in D, so a and x lose it
    x[0, (nh + nkv) * d] = 0.0
    a3[:, :, 0] = 0.0
    da2 = dy.clone()
    da2[t - 1, 1] = float("inf")  # every key of the last row, and its dq
    dqkv = backward(x, a, da2, lse, t, nh, nkv, d, plan)
    want = backward(x, a, dy, lse, t, nh, nkv, d, plan)
    w = nh * d
    assert float((dqkv[:t - 1, :w].double() - want[:t - 1, :w].double()).norm()) <= 2 * FRO_TOL * float(want[:, :w].double().norm())
    assert not torch.isfinite(dqkv[t - 1, :d].float()).any() and torch.isfinite(dqkv[:, d:w].float()).all()
    dv, dv_want = dqkv[:, w + nkv * d:].double(), want[:, w + nkv * d:].double()
    assert torch.isposinf(dv[:, 1]).all()
    rest = [c for c in range(d) if c != 1]
    assert float((dv[:, rest] - dv_want[:, rest]).norm()) <= 2 * FRO_TOL * float(dv_want.norm())
    x.fill_(float("nan"))
    a, lse = forward(x, t, nh, nkv, d, plan)
    dqkv = backward(x, a, dy, lse, t, nh, nkv, d, plan)
    assert torch.isnan(a).all() and torch.isnan(lse[:, :t]).all() and torch.isnan(dqkv).all()


def test_plan_intervals_and_positions():
    t, offsets, prefix = 300, [7, 100, 100, 290], [20, 3, 0]
    pos = torch.full((t + 1,), -7, dtype=torch.int32, device="cuda")
    plan = make_plan(t, offsets, prefix, positions=pos)
    see = visible(t, offsets, prefix).cpu().numpy()
    nb = 3
    flat = plan.view(torch.int32).view(-1, 2).cpu().numpy()
    rows, cols = flat[: 128 * nb], flat[128 * nb: 256 * nb]
    for i in range(t):
        assert np.array_equal(np.nonzero(see[i])[0], np.arange(*rows[i]))
        assert np.array_equal(np.nonzero(see[:, i])[0], np.arange(*cols[i]))
    assert np.all(rows[t:] == 0) and np.all(cols[t:] == 0)
    starts = np.array([next((offsets[d] for d in range(3) if offsets[d] <= i < offsets[d + 1]), i) for i in range(t)])
    assert np.array_equal(pos.cpu().numpy()[:t], np.arange(t) - starts) and int(pos[t]) == -7
    for b, (first, end) in enumerate(flat[256 * nb: 256 * nb + nb]):
        assert np.array_equal(np.nonzero(see[128 * b: 128 * (b + 1)].any(0))[0][[0, -1]] // 128, [first, end - 1])


@pytest.mark.parametrize("offsets", [[50, 20, 400, -3, 90, 2000], [2 ** 31 - 1, 0, -2 ** 31, 5, 7, 9]])
def test_offsets_out_of_order_stay_inside(offsets):
    """Nonsense offsets give some mask, and neither faults nor hangs nor writes outside."""
    t, nh, nkv, d = 333, 2, 1, 64
    qkv, da = draw(5, t, nh, nkv, d)
    plan = make_plan(t, offsets, [2 ** 31 - 1, -5, 3, 2 ** 30, 1])
    flat = plan.view(torch.int32)
    assert int(flat.min()) >= 0 and int(flat.max()) <= t
    guard = torch.full((t + 40, nh * d), 3.0, dtype=torch.bfloat16, device="cuda")
    a, lse = forward(qkv, t, nh, nkv, d, plan, a=guard)
    backward(qkv, a, da, lse, t, nh, nkv, d, plan)
    assert torch.all(guard[t:] == 3.0)


def test_rows_behind_the_tokens_are_left_alone():
    t, nh, nkv, d = 200, 4, 2, 64
    qkv, da = draw(6, t + 56, nh, nkv, d)
    qkv[t:], da[t:] = float("nan"), float("nan")
    a = torch.full((t + 56, nh * d), 5.0, dtype=torch.bfloat16, device="cuda")
    dqkv = torch.full((t + 56, (nh + 2 * nkv) * d), 6.0, dtype=torch.bfloat16, device="cuda")
    plan = make_plan(t, [0, 70, 200])
    _, lse = forward(qkv, t, nh, nkv, d, plan, a=a)
    scratch = torch.empty(zb.zb_op_attention_document_scratch_bytes(t, nh), dtype=torch.uint8, device="cuda")
    zb.zb_op_attention_document_backward(qkv, a, da, lse, dqkv, plan, None, 0.0, t, nh, nkv, d, scratch, scratch.numel())
    assert torch.all(a[t:] == 5.0) and torch.all(dqkv[t:] == 6.0)
    ra, _, rd = reference(qkv[:t], nh, nkv, d, visible(t, [0, 70, 200]), da=da[:t])
    assert_near(a[:t], ra, "a")
    assert_near(dqkv[:t], rd, "dqkv")


def test_no_rows():
    zb.zb_op_attention_document_plan(None, None, 1, 0, None, 0)
    zb.zb_op_attention_document_forward(None, None, None, None, None, 0.0, 0, 4, 2, 64)
    zb.zb_op_attention_document_backward(None, None, None, None, None, None, None, 0.0, 0, 4, 2, 64, None, 0)


def test_the_same_bits_again_on_another_stream_and_in_graphs():
    """Two graphs on two streams at once, each with its own workspaces, give the eager call's bits."""
    t, nh, nkv, d = 1300, 8, 2, 128
    offsets, prefix = [0, 300, 310, 1200], [0, 4, 100]
    qkv, da = draw(8, t, nh, nkv, d)
    plan = make_plan(t, offsets, prefix)
    a, lse = forward(qkv, t, nh, nkv, d, plan, 20.0)
    dqkv = backward(qkv, a, da, lse, t, nh, nkv, d, plan, 20.0)
    off, pre = ints(offsets), ints(prefix)
    runs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        w = {"plan": torch.empty_like(plan), "a": torch.empty_like(a), "lse": torch.empty_like(lse),
             "dqkv": torch.empty_like(dqkv),
             "scratch": torch.empty(zb.zb_op_attention_document_scratch_bytes(t, nh), dtype=torch.uint8, device="cuda")}

        def calls(w=w, s=s):
            zb.zb_op_attention_document_plan(off, pre, 3, t, w["plan"], w["plan"].numel(), None, s)
            zb.zb_op_attention_document_forward(qkv, w["a"], w["lse"], w["plan"], None, 20.0, t, nh, nkv, d, s)
            zb.zb_op_attention_document_backward(qkv, w["a"], da, w["lse"], w["dqkv"], w["plan"], None, 20.0, t, nh, nkv, d,
                                                 w["scratch"], w["scratch"].numel(), s)

        s.wait_stream(torch.cuda.current_stream())
        calls()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            calls()
        runs.append((s, g, w))
    for _, _, w in runs:
        for x in (w["a"], w["dqkv"]):
            x.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, g, _ in runs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, _, w in runs:
        assert torch.equal(w["a"], a) and torch.equal(w["dqkv"], dqkv)
        assert torch.equal(w["lse"][:, :t], lse[:, :t])


def test_offsets_past_32_bits():
    """A qkv tensor of more than 2^31 elements: short documents at its start and end equal the same ones alone."""
    nh, nkv, d, n = 64, 8, 128, 120
    t = 212000
    assert t * (nh + 2 * nkv) * d > 2 ** 31
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    qkv = torch.randn(t, (nh + 2 * nkv) * d, generator=g, device="cuda", dtype=torch.bfloat16)
    da = torch.randn(t, nh * d, generator=g, device="cuda", dtype=torch.bfloat16)
    offsets = list(range(0, t - n, 90)) + [t - n, t]
    plan = make_plan(t, offsets)
    a, lse = forward(qkv, t, nh, nkv, d, plan)
    dqkv = backward(qkv, a, da, lse, t, nh, nkv, d, plan)
    for rows in (slice(0, 90), slice(t - n, t)):
        m = rows.stop - rows.start
        see = visible(m, [0, m])
        ra, _, rd = reference(qkv[rows], nh, nkv, d, see, da=da[rows])
        assert_near(a[rows], ra, "a")
        assert_near(dqkv[rows], rd, "dqkv")
    assert torch.isfinite(a.view(-1)[::1001].float()).all() and torch.isfinite(dqkv.view(-1)[::1001].float()).all()


def test_the_plain_form_equals_the_oracle():
    t, nh, nkv, d = 60, 4, 2, 64
    offsets, prefix = [3, 20, 20, 55], [4, 0, 50]
    qkv, da = draw(11, t, nh, nkv, d)
    slopes = slopes_of(nh)
    see = O.document_visible(t, offsets, prefix)
    assert np.array_equal(visible(t, offsets, prefix).cpu().numpy(), see)
    x, dy = qkv.double().cpu().numpy(), da.double().cpu().numpy()
    a, lse = O.document_attention(x, nh, nkv, d, see, 2.5, slopes.double().cpu().numpy())
    grad = O.document_attention_grad(dy, x, nh, nkv, d, see, 2.5, slopes.double().cpu().numpy())
    ra, rl, rd = (y.cpu().numpy() for y in reference(qkv, nh, nkv, d, visible(t, offsets, prefix), 2.5, slopes, da))
    np.testing.assert_allclose(ra, a, atol=1e-12)
    np.testing.assert_allclose(rd, grad, atol=1e-11)
    live = see.any(1)
    np.testing.assert_allclose(rl[:, live], lse[:, live], atol=1e-11)


@pytest.mark.parametrize("mode", ["plain", "cap", "bias"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_first", [1, 6])
@pytest.mark.parametrize("key", [float("inf"), 3e38])
def test_keys_of_no_weight_before_the_others(key, n_first, d, mode):
    """A document's first keys score -infinity (an infinite value, or a product past float32's range): they have no weight
    beside the finite scores behind them, whatever a document in the same tile holds.  Under a cap they score -cap."""
    t, nh, nkv, offsets, cap = 300, 4, 2, [0, 60, 290], 5.0 if mode == "cap" else 0.0
    qkv, da = draw(41, t, nh, nkv, d)
    x = qkv.view(t, nh + 2 * nkv, d)
    x[:, :nh, 3] = -(x[:, :nh, 3].abs() + 4.0)  # 4 times 3e38: past the range
    x[60:60 + n_first, nh:nh + nkv, 3] = key
    slopes = slopes_of(nh) if mode == "bias" else None
    see = O.document_visible(t, offsets)
    with np.errstate(invalid="ignore"):
        ra, rl = (torch.from_numpy(y).cuda() for y in O.document_attention(
            qkv.double().cpu().numpy(), nh, nkv, d, see, cap, None if slopes is None else slopes.double().cpu().numpy()))
    bad = qkv.clone()
    bad.view(t, nh + 2 * nkv, d)[20, nh + nkv:] = float("nan")  # the values of a key of the first document
    plan = make_plan(t, offsets)
    a, lse = forward(bad, t, nh, nkv, d, plan, cap, slopes)
    keep = torch.arange(60 if cap else 60 + n_first, 290, device="cuda")
    assert_near(a[keep], ra[keep], "a")
    assert_lse(lse[:, keep], rl[:, keep], keep.numel())
    if math.isinf(key) and not cap:
        assert torch.isnan(a[60:60 + n_first]).all()  # no key but those
    if math.isinf(key) or cap:
        return  # the formula's dq is 0 times infinity; the cap's slope at 3e38 is 0, as is its dk
    rd = reference(qkv, nh, nkv, d, visible(t, offsets), cap, slopes, da)[2]
    dqkv = backward(bad, a, da, lse, t, nh, nkv, d, plan, cap, slopes)
    assert_near(dqkv[keep], rd[keep], "dqkv")


@pytest.mark.parametrize("mode", ["plain", "bias", "cap"])
@pytest.mark.parametrize("nh,nkv,d", [(4, 2, 64), (4, 1, 128), (3, 3, 64), (3, 1, 128)])
def test_padding_gives_the_same_bits_whatever_it_holds(nh, nkv, d, mode):
    """Rows before the first and behind the last document, inside tiles that documents share and in tiles of their own."""
    t, offsets, prefix, cap = 900, [200, 330, 700], [20, 0], 5.0 if mode == "cap" else 0.0
    qkv, da = draw(51, t, nh, nkv, d)
    slopes = slopes_of(nh) if mode == "bias" else None
    plan = make_plan(t, offsets, prefix)
    pad = [slice(0, 200), slice(700, t)]
    kept = None
    # infinite scores, hidden as they are, would take a warp to the other form of the cap's tanh
    for value in (0.0, float("nan")) + (() if cap else (float("inf"), -float("inf"), 3e38)):
        x, dy = qkv.clone(), da.clone()
        for rows in pad:
            x[rows], dy[rows] = value, value
        a, lse = forward(x, t, nh, nkv, d, plan, cap, slopes)
        dqkv = backward(x, a, dy, lse, t, nh, nkv, d, plan, cap, slopes)
        assert torch.isneginf(lse[:, 700:t]).all() and all(not y[rows].any() for y in (a, dqkv) for rows in pad)
        if kept is None:
            kept = a, lse, dqkv
            ra, _, rd = reference(x, nh, nkv, d, visible(t, offsets, prefix), cap, slopes, dy)
            assert_near(a, ra, "a")
            assert_near(dqkv, rd, "dqkv")
        assert torch.equal(a, kept[0]) and torch.equal(dqkv, kept[2]) and torch.equal(lse[:, :t], kept[1][:, :t])
