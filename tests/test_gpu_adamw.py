"""GPU parity of the AdamW step, its 8-bit states and the gradient norm against the oracle.

Moments are compared bit for bit: their products and sums round separately, as numpy's float32 does.  Bar of a
float32 parameter: p (1 - lr wd) rounds twice and the final difference once, 3 x 2^-24 of |p|; the update carries
the moments' roundings, an approximate square root and division and the factors' own roundings, at most 16 units of
2^-24 of itself.  A bf16 parameter adds its rounding, 2^-8 of |p|.
"""
import numpy as np
import pytest
import torch

from backward_split_linear_gb300 import binding as zb
from backward_split_linear_gb300.runtime import AdamW, Stage, bf16_from_bits, f64_from_bf16
from backward_split_linear_gb300 import synth
from oracle import train_ops as O

pytestmark = pytest.mark.gpu

HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.95, eps=1e-8)


def draw(rng, n, bits, param="bf16", master=True, grad="f32", zero=False):
    """(device dict, float64 / integer host dict) of one tensor."""
    p = rng.standard_normal(n).astype(np.float32)
    g = (1e-3 * rng.standard_normal(n)).astype(np.float32)
    m = (1e-3 * rng.standard_normal(n)).astype(np.float32) * (0 if zero else 1)
    v = (1e-6 * rng.standard_normal(n) ** 2).astype(np.float32) * np.float32(0 if zero else 1)
    dev, host = {}, {}
    pt, gt = torch.from_numpy(p), torch.from_numpy(g)
    if grad == "bf16":
        gt = gt.to(torch.bfloat16)
    dev["grad"], host["grad"] = gt.cuda(), gt.float().numpy()
    if param == "bf16":
        dev["param"] = pt.to(torch.bfloat16).cuda()
        if master:
            dev["master"] = pt.clone().cuda()
        host["p"] = p if master else pt.to(torch.bfloat16).float().numpy()
    else:
        dev["param"], host["p"] = pt.clone().cuda(), p
    if bits == 8:
        for name, x, signed in (("m", m, True), ("v", v, False)):
            codes, scales = O.pack(x, signed, 0x8000)
            if zero:
                scales = np.zeros_like(scales)
            host[name] = O.unpack(codes, scales, signed)
            dev[name], dev[name + "_scale"] = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    else:
        host["m"], host["v"] = m, v
        dev["m"], dev["v"] = torch.from_numpy(m).cuda(), torch.from_numpy(v).cuda()
    return dev, host


def check(dev, host, step, decay, scale, bits, stochastic=False, seed=0, index=0):
    n = host["p"].size
    m, v = O.moments_f32(host["grad"], host["m"], host["v"], HYPER["beta1"], HYPER["beta2"], scale)
    g64 = host["grad"].astype(np.float64) * (1.0 if scale is None else float(np.float32(scale)))
    p, _, _ = O.adamw(host["p"].astype(np.float64), g64, host["m"].astype(np.float64), host["v"].astype(np.float64), step,
                      decay=decay, **HYPER)
    update = np.abs(p - host["p"] * (1.0 - HYPER["lr"] * decay))
    bar = 3 * 2.0 ** -24 * np.abs(host["p"]) + 16 * 2.0 ** -24 * update + 1e-37
    if "master" in dev:
        got = dev["master"].cpu().numpy()
        assert np.all(np.abs(got - p) <= bar)
        assert torch.equal(dev["param"], dev["master"].to(torch.bfloat16))
    elif dev["param"].dtype == torch.float32:
        assert np.all(np.abs(dev["param"].cpu().numpy() - p) <= bar)
    else:
        step_size = 2.0 ** -7 if stochastic else 2.0 ** -8  # to either neighbour, or to the nearest
        assert np.all(np.abs(f64_from_bf16(dev["param"]) - p) <= bar + step_size * np.abs(p) * (1 + 2.0 ** -8))
    if bits == 32:
        assert np.array_equal(dev["m"].cpu().numpy(), m) and np.array_equal(dev["v"].cpu().numpy(), v)
        return
    noise = O.noise32(seed, step, index, n) if stochastic else np.full(n, 0x80008000, dtype=np.uint64)
    for name, x, signed, bits16 in (("m", m, True, noise & np.uint64(0xFFFF)), ("v", v, False, noise >> np.uint64(16))):
        codes, scales = O.pack(x, signed, bits16)
        assert np.array_equal(dev[name + "_scale"].cpu().numpy(), scales)
        assert np.array_equal(dev[name].cpu().numpy(), codes)


SIZES = [1, 7, 8, 255, 256, 257, 2047, 2049, 70001]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,master,grad", [("bf16", True, "f32"), ("bf16", False, "bf16"), ("f32", False, "f32")])
def test_step_over_ragged_tensors(cuda_device, bits, param, master, grad):
    rng = np.random.default_rng(17)
    pairs = [draw(rng, n, bits, param, master, grad) for n in SIZES]
    opt = AdamW([d | {"weight_decay": 0.1 * (i % 2)} for i, (d, _) in enumerate(pairs)], state_bits=bits, step=6, **HYPER)
    opt.step()
    for i, (dev, host) in enumerate(pairs):
        check(dev, host, 7, 0.1 * (i % 2), None, bits)
    if bits == 8:
        for (m, v), (dev, _) in zip(opt.unpack_states(), pairs):
            for x, name, signed in ((m, "m", True), (v, "v", False)):
                want = O.unpack(dev[name].cpu().numpy(), dev[name + "_scale"].cpu().numpy(), signed)
                assert np.array_equal(x.cpu().numpy(), want)


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_scale_and_noise(cuda_device, bits):
    """New states are zero bytes; a device scale; stochastic rounding by the stated hash, tensor by tensor."""
    rng = np.random.default_rng(3)
    pairs = [draw(rng, n, bits, "bf16", i == 0, "f32", zero=True) for i, n in enumerate((3000, 5, 511))]
    opt = AdamW([d for d, _ in pairs], state_bits=bits, stochastic=True, seed=99, **HYPER)
    opt.step(grad_scale=torch.full((), 0.37, device="cuda"))
    for i, (dev, host) in enumerate(pairs):
        check(dev, host, 1, 0.0, 0.37, bits, stochastic=True, seed=99, index=i)


def test_more_tensors_than_one_launch_takes(cuda_device):
    rng = np.random.default_rng(4)
    pairs = [draw(rng, 1 + i % 5, 8) for i in range(150)]
    opt = AdamW([d for d, _ in pairs], state_bits=8, stochastic=True, seed=5, step=1, **HYPER)
    opt.step()
    for i, (dev, host) in enumerate(pairs):
        check(dev, host, 2, 0.0, None, 8, stochastic=True, seed=5, index=i)
    norm, _ = opt.grad_norm()
    want = np.sqrt(sum(np.sum(h["grad"].astype(np.float64) ** 2) for _, h in pairs))
    assert abs(float(norm) - want) <= 2.0 ** -22 * want


def test_empty_tensors_and_lists(cuda_device):
    rng = np.random.default_rng(6)
    pairs = [draw(rng, n, 32) for n in (0, 40, 0)]
    opt = AdamW([d for d, _ in pairs], **HYPER)
    opt.step()
    check(*pairs[1], 1, 0.0, None, 32)
    none = AdamW([])
    none.step()
    assert [float(x) for x in none.grad_norm()] == [0.0, 1.0]


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_without_a_finite_scale_writes_nothing(cuda_device, bits):
    rng = np.random.default_rng(7)
    dev, _ = draw(rng, 777, bits)
    before = {k: t.clone() for k, t in dev.items()}
    dev["grad"][5] = float("inf")
    opt = AdamW([dev], state_bits=bits, **HYPER)
    _, scale = opt.grad_norm(1.0)
    assert not np.isfinite(float(scale))
    opt.step(grad_scale=scale)
    for k, t in before.items():
        if k != "grad":
            assert torch.equal(dev[k], t), k


def test_extreme_moments_in_8_bits(cuda_device):
    """Blocks of zeros, of one tiny value and of values 10^30 apart keep their order, and no second moment vanishes."""
    n = 1024
    rng = np.random.default_rng(9)
    dev, host = draw(rng, n, 8, zero=True)
    g = np.zeros(n, dtype=np.float32)
    g[256] = 1e-30                                        # its square underflows: v = 0
    g[512:768] = np.float32(10.0) ** rng.uniform(-15, 15, 256)
    g[768:] = 1e-18 * rng.standard_normal(256)
    dev["grad"].copy_(torch.from_numpy(g))
    host["grad"] = g
    opt = AdamW([dev], state_bits=8, **HYPER)
    opt.step()
    check(dev, host, 1, 0.0, None, 8)
    v = O.moments_f32(g, host["m"], host["v"], HYPER["beta1"], HYPER["beta2"])[1]
    z = v * (1.0 / np.repeat(dev["v_scale"].cpu().numpy(), 256))
    assert np.all((dev["v"].cpu().numpy() > 0) == (z.astype(np.float32) > 0))
    assert torch.isfinite(dev["master"]).all()


@pytest.mark.parametrize("stochastic", [False, True])
def test_values_out_of_range_spare_their_block_in_8_bits(cuda_device, stochastic):
    """A gradient whose square overflows, an infinite and a NaN one: the moments of the elements beside them are the
    stated codes, and the next step's parameters are finite."""
    n, bad = 1024, {5: 2e19, 300: float("inf"), 301: -float("inf"), 700: float("nan")}
    dev, host = draw(np.random.default_rng(11), n, 8, master=False, param="f32")
    for i, g in bad.items():
        dev["grad"][i] = g
        host["grad"][i] = g
    opt = AdamW([dev], state_bits=8, step=3, stochastic=stochastic, seed=8, **HYPER)
    opt.step()
    m, v = O.moments_f32(host["grad"], host["m"], host["v"], HYPER["beta1"], HYPER["beta2"])
    noise = O.noise32(8, 4, 0, n) if stochastic else np.full(n, 0x80008000, dtype=np.uint64)
    for name, x, signed, bits16 in (("m", m, True, noise & np.uint64(0xFFFF)), ("v", v, False, noise >> np.uint64(16))):
        codes, scales = O.pack(x, signed, bits16)
        assert np.isfinite(scales).all() and np.array_equal(dev[name + "_scale"].cpu().numpy(), scales)
        ok = ~np.isnan(x)  # a NaN's sign is the hardware's
        assert np.array_equal(dev[name].cpu().numpy()[ok], codes[ok])
    dev["grad"].fill_(1e-3)
    opt.step()
    others = torch.tensor([i for i in range(n) if i not in bad], device="cuda")
    assert torch.isfinite(dev["param"][others]).all()


def test_stochastic_rounding_follows_a_slow_average(cuda_device):
    """v against a constant gradient: the nearest code cannot move by 5 % of a step, the stochastic one does.  Over 8192
    elements the mean's spread is 1/8 of a value / sqrt(8192), 0.14 %; four of those over 60 steps' geometric sum."""
    n = 8192
    ends = {}
    for stochastic in (False, True):
        rng = np.random.default_rng(10)
        dev, _ = draw(rng, n, 8, zero=True)
        dev["grad"].fill_(1e-3)
        opt = AdamW([dev], state_bits=8, stochastic=stochastic, seed=1, **HYPER)
        opt.step()
        dev["grad"].fill_(0.9e-3)
        dev["grad"][::256] = 1e-3   # holds each block's scale
        for _ in range(60):
            opt.step()
        _, v = opt.unpack_states()[0]
        ends[stochastic] = v.cpu().numpy().reshape(-1, 256)[:, 1:].mean()
    want = 1e-6 * 0.05 * 0.95 ** 60 + 0.81e-6 * (1 - 0.95 ** 60)
    assert abs(ends[True] - want) < 0.02 * want


def test_norm_range_and_repeatability(cuda_device):
    rng = np.random.default_rng(11)
    for size, g in ((3e25, "f32"), (1e-25, "f32"), (1.0, "bf16")):
        dev, host = draw(rng, 100003, 32, grad=g)
        x = host["grad"].astype(np.float64) * 1e3 * size
        dev["grad"] = (dev["grad"].double() * 1e3 * size).to(dev["grad"].dtype)
        x = dev["grad"].double().cpu().numpy()
        opt = AdamW([dev], **HYPER)
        norm, scale = (float(v) for v in opt.grad_norm(0.5 * size))
        want = np.sqrt(np.sum(x * x))
        assert abs(norm - want) <= 2.0 ** -20 * want
        assert abs(scale - min(1.0, 0.5 * size / (want + 1e-6))) <= 2.0 ** -20
        assert (norm, scale) == tuple(float(v) for v in opt.grad_norm(0.5 * size))


def test_captured_step_advances_on_the_device(cuda_device):
    """A graph of norm, step and the step number's increment, replayed, equals eager steps to the bias corrections'
    rounding (float32 powers on the device against float64 ones on the host)."""
    rng = np.random.default_rng(12)
    a, _ = draw(rng, 5000, 32)
    b = {k: t.clone() for k, t in a.items()}
    number = torch.ones((), dtype=torch.int64, device="cuda")
    lr = torch.full((), HYPER["lr"], device="cuda")
    graphed = AdamW([a], step_device=number, lr_device=lr, **HYPER)
    eager = AdamW([b], **HYPER)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        _, scale = graphed.grad_norm(0.01)
        graphed.step(grad_scale=scale)
        number.add_(1)
    for _ in range(5):
        graph.replay()
        eager.step(grad_scale=eager.grad_norm(0.01)[1])
    torch.cuda.synchronize()
    assert int(number) == 6
    assert torch.equal(a["m"], b["m"]) and torch.equal(a["v"], b["v"])
    # 1 - beta^t from expm1 of a float32 product: at most 4 units of 2^-24 of each factor, on updates below 1.1 lr each
    assert float((a["master"] - b["master"]).abs().max()) <= 5 * (3 * 2.0 ** -24 * 5.0 + 24 * 2.0 ** -24 * 4.0 * HYPER["lr"])


@pytest.mark.parametrize("bits", [32, 8])
def test_a_stage_takes_a_step(cuda_device, bits):
    """F, B, W, flush, clip and step through the stage's own objects; a step with W pending is refused."""
    inp = synth.stage_inputs("mlp", 2, 256, 512, tokens=96, n_mb=2, seed=3)
    st = Stage.from_synth("mlp", 2, 256, 512, max_tokens=96, max_inflight=2, params_bits=inp["params"])
    opt = AdamW.for_stage(st, lr=1e-2, weight_decay=0.1, state_bits=bits)
    masters = [{k: t["master"].cpu().numpy().copy() if "master" in t else t["param"].cpu().numpy().copy()
                for k, t in (("x", t),)}["x"] for t in opt.tensors]
    y, dx = (torch.empty(96, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i in range(2):
        st.forward(i, bf16_from_bits(inp["x"][i]), y)
        st.backward_input(i, bf16_from_bits(inp["dy"][i]), dx)
    with pytest.raises(zb.ZBError) as e:
        opt.step()
    assert e.value.name == "ZB_ERR_ORDER" and opt.steps == 0
    st.flush()
    norm, scale = opt.grad_norm(1.0)
    opt.step(grad_scale=scale)
    st.sync()
    total = np.sqrt(sum(float((t["grad"].double() ** 2).sum()) for t in opt.tensors))
    assert abs(float(norm) - total) <= 2.0 ** -20 * total
    for t, p0 in zip(opt.tensors, masters):
        g = t["grad"].double().cpu().numpy().reshape(-1) * float(scale)
        p0 = p0.reshape(-1).astype(np.float64)
        p, _, _ = O.adamw(p0, g, 0.0, 0.0, 1, 1e-2, 0.9, 0.95, 1e-8, t["weight_decay"])
        got = (t["master"] if "master" in t else t["param"]).double().cpu().numpy().reshape(-1)
        assert np.all(np.abs(got - p) <= 3 * 2.0 ** -24 * np.abs(p0) + 20 * 2.0 ** -24 * 1e-2)
        if "master" in t:
            assert torch.equal(t["param"].reshape(-1), t["master"].reshape(-1).to(torch.bfloat16))
    st.close()


def test_bf16_parameters_round_up_with_the_probability_of_their_remainder(cuda_device):
    """Bit for bit where the float32 result, known to its bar, does not lie at a carry: the bar is 2^-22 of the value
    beside a bf16 step of 2^-8, so fewer than one in 2^10 elements is undecided."""
    n = 70001
    dev, host = draw(np.random.default_rng(21), n, 32, master=False)
    opt = AdamW([dev | {"weight_decay": 0.1}], stochastic=True, seed=77, step=2, **HYPER)
    opt.step()
    f64 = {k: host[k].astype(np.float64) for k in ("p", "grad", "m", "v")}
    p, _, _ = O.adamw(f64["p"], f64["grad"], f64["m"], f64["v"], 3, decay=0.1, **HYPER)
    bar = 3 * 2.0 ** -24 * np.abs(f64["p"]) + 16 * 2.0 ** -24 * np.abs(p - f64["p"]) + 1e-37
    noise = ((O.noise32(77, 3, 0, n) * np.uint64(0x9E3779B1)) & np.uint64(0xFFFFFFFF)) >> np.uint64(16)
    low, high = ((np.maximum(np.abs(p) + s * bar, 0.0).astype(np.float32).view(np.uint32) + noise.astype(np.uint32)) >> 16
                 for s in (-1.0, 1.0))
    decided = (low == high) & (np.abs(p) > bar)
    assert decided.sum() > n - n // 1024
    got = dev["param"].view(torch.int16).cpu().numpy().view(np.uint16).astype(np.uint32)
    assert np.array_equal(got[decided] & 0x7FFF, low[decided])
    assert np.array_equal((got >> 15)[decided] == 1, (p < 0)[decided])


def test_a_parameter_below_half_a_step_moves_on_average(cuda_device):
    """Parameters of 1 with an update of 1e-3, against bf16 steps of 2^-8 below 1: rounded to the nearest none moves; with
    noise the mean does.  One element spreads by at most half a step, so 2^16 of them by 2^-17: six of those."""
    n = 1 << 16
    for stochastic in (False, True):
        dev, _ = draw(np.random.default_rng(22), n, 32, master=False, zero=True)
        dev["param"].fill_(1.0)
        dev["grad"].fill_(1.0)
        AdamW([dev], stochastic=stochastic, seed=3, **{**HYPER, "lr": 1e-3}).step()  # m / sqrt(v) is 1 in the first step
        mean = float(dev["param"].double().mean())
        assert mean == 1.0 if not stochastic else abs(mean - (1.0 - 1e-3)) < 6 * 2.0 ** -17


def test_the_nearest_code_stands_still(cuda_device):
    """The slow average of test_stochastic_rounding_follows_a_slow_average rounded to the nearest code, over the same
    steps: the codes are the oracle's, and their mean misses the average by more than the 2 % that the noise keeps to.
    (An element is pulled by 5 % of its distance from 0.81e-6 and moves a code by half of 1e-6 / 15 or more: at 13 / 15
    of its block's 0.956e-6, 7 % above the average, it stands.)"""
    n = 8192
    dev, host = draw(np.random.default_rng(10), n, 8, zero=True)
    opt = AdamW([dev], state_bits=8, **HYPER)
    m, v = host["m"], host["v"]
    for step in range(61):
        g = np.full(n, 0.9e-3 if step else 1e-3, dtype=np.float32)
        g[::256] = 1e-3
        dev["grad"].copy_(torch.from_numpy(g))
        opt.step()
        m, v = O.moments_f32(g, m, v, HYPER["beta1"], HYPER["beta2"])
        m, v = (O.unpack(*O.pack(x, signed, 0x8000), signed) for x, signed in ((m, True), (v, False)))
    got = opt.unpack_states()[0]
    assert np.array_equal(got[0].cpu().numpy(), m) and np.array_equal(got[1].cpu().numpy(), v)
    want = 1e-6 * 0.05 * 0.95 ** 60 + 0.81e-6 * (1 - 0.95 ** 60)
    assert abs(v.reshape(-1, 256)[:, 1:].mean() - want) > 0.02 * want
