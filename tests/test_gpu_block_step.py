"""A feed-forward block with biases, norms on both sides and an 8-bit stash, as a training step uses it: F, B and W of two
microbatches against float64 differentiation, from captured graphs, on other streams.

    h0 = x0 + b gate0 u0(y0)      n0 = PreNorm(h0)      (the block before)
    z1 = n0 W1^T + b1             y1 = act(z1)
    y2 = y1 W2^T + b2
    h1 = a h0 + b gate1 * PostNorm(y2),  n1 = PreNorm(h1)

Bar: relative Frobenius error.  A bf16 tensor costs 1.6e-3 (a uniform error of half a step at most), an 8-bit one 6.6e-3
(a third of a unit of a 92nd of a block's largest value, which lies 2.1 standard deviations out over 32 normal values).  A
gradient here has at most 8 bf16 tensors and 3 packed ones behind it, and they add in quadrature: sqrt(8 (1.6e-3)^2 + 3
(6.6e-3)^2) = 1.23e-2, times 1.5 for layers that amplify them (the norms' gammas and the slopes reach 1.2).
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from backward_split_linear_gb300 import binding as zb
from parity import errors

pytestmark = pytest.mark.gpu

H, F = 256, 576
BAR = 1.5 * float(np.sqrt(8 * 1.6e-3 ** 2 + 3 * 6.6e-3 ** 2))
EPS = 1e-5


def parameters(seed, act):
    g = torch.Generator()
    g.manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    bf = lambda x: x.to(torch.bfloat16)  # noqa: E731
    return dict(act=act, w1=bf(n(F, H) / H ** 0.5), b1=0.3 * n(F), w2=bf(n(H, F) / F ** 0.5), b2=0.3 * n(H), gate0=1.0 + 0.2 * n(H),
                gate1=0.5 + 0.2 * n(H), post=1.0 + 0.1 * n(H), pre0=1.0 + 0.1 * n(H), beta0=0.1 * n(H), pre1=1.0 + 0.1 * n(H))


def microbatch(seed, t):
    g = torch.Generator()
    g.manual_seed(seed)
    return {k: torch.randn(t, H, generator=g).to(torch.bfloat16) for k in ("x0", "y0", "dn1", "dres1")}


A1, B1 = 0.75, 0.5


class Block:
    """The calls of one block on the GPU; gradients accumulate over microbatches."""

    def __init__(self, par):
        self.act = par["act"]
        self.p = {k: v.cuda() for k, v in par.items() if k != "act"}
        p = self.p
        self.first = zb.make_residual_norm(pre="layer", gate_kind="channel", gate=p["gate0"], pre_gamma=p["pre0"],
                                           pre_beta=p["beta0"], pre_eps=EPS)
        self.second = zb.make_residual_norm(post="rms", pre="rms", gate_kind="channel", gate=p["gate1"], post_gamma=p["post"],
                                            pre_gamma=p["pre1"], residual_scale=A1, branch_scale=B1, post_eps=EPS, pre_eps=EPS)
        self.grads = {k: torch.zeros(v.shape, dtype=torch.float32, device="cuda") for k, v in p.items()}

    def buffers(self, t):
        bf = lambda w: torch.empty(t, w, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        pk = lambda w: (torch.empty(t, w, dtype=torch.uint8, device="cuda"),  # noqa: E731
                        torch.empty(t, w // 32, dtype=torch.uint8, device="cuda"))
        st = lambda: torch.empty(t, 4, device="cuda")  # noqa: E731
        sizes = [zb.zb_op_backward_input_activation_scratch_bytes(t, F), zb.zb_op_backward_bias_scratch_bytes(t, H),
                 zb.zb_op_backward_weight_checkpoint_scratch_bytes(t, F),
                 zb.zb_op_residual_norm_backward_weight_scratch_bytes(t, H)]
        return dict(t=t, h0=bf(H), n0=bf(H), n0_8=pk(H), s0=st(), y1=bf(F), z1_8=pk(F), y1_8=pk(F), y2=bf(H), h1=bf(H), n1=bf(H),
                    s1=st(), dh1=bf(H), dx=bf(H), dy2=bf(H), dz=bf(F), dn0=bf(H), dh0=bf(H), dy0=bf(H),
                    scratch=torch.empty(max(sizes), dtype=torch.uint8, device="cuda"))

    def step(self, m, b, stream=None):
        """F, B and W of one microbatch."""
        p, g, t, s = self.p, self.grads, b["t"], dict(stream=stream)
        zb.zb_op_residual_norm_forward(self.first, m["x0"], m["y0"], b["h0"], b["n0"], b["s0"], t, H, n_packed=b["n0_8"], **s)
        zb.zb_op_linear_activation_forward(b["n0"], p["w1"], p["b1"], None, b["y1"], t, H, F, self.act, z_packed=b["z1_8"],
                                           y_packed=b["y1_8"], **s)
        zb.zb_op_linear_activation_forward(b["y1"], p["w2"], p["b2"], None, b["y2"], t, F, H, **s)
        zb.zb_op_residual_norm_forward(self.second, b["h0"], b["y2"], b["h1"], b["n1"], b["s1"], t, H, **s)
        zb.zb_op_residual_norm_backward_input(self.second, m["dn1"], m["dres1"], b["h1"], b["y2"], b["s1"], b["dh1"], b["dy2"], t, H,
                                              dx=b["dx"], **s)
        zb.zb_op_backward_input_activation(b["dy2"], p["w2"], None, b["dz"], t, F, H, self.act, z_packed=b["z1_8"], dbias=g["b1"],
                                           scratch=b["scratch"], **s)
        zb.zb_op_backward_input(b["dz"], p["w1"], b["dn0"], t, H, F, **s)
        zb.zb_op_residual_norm_backward_input(self.first, b["dn0"], b["dx"], b["h0"], None, b["s0"], b["dh0"], b["dy0"], t, H, **s)
        zb.zb_op_backward_weight_checkpoint(b["dy2"], b["y1_8"], g["w2"], t, F, H, b["scratch"], **s)
        zb.zb_op_backward_bias(b["dy2"], g["b2"], t, H, b["scratch"], **s)
        zb.zb_op_backward_weight_checkpoint(b["dz"], b["n0_8"], g["w1"], t, H, F, b["scratch"], **s)
        zb.zb_op_residual_norm_backward_weight(self.second, m["dn1"], b["h1"], b["dh1"], b["y2"], b["s1"], t, H, b["scratch"],
                                               dpost_gamma=g["post"], dpre_gamma=g["pre1"], dgate=g["gate1"], **s)
        zb.zb_op_residual_norm_backward_weight(self.first, b["dn0"], b["h0"], b["dh0"], m["y0"], b["s0"], t, H, b["scratch"],
                                               dpre_gamma=g["pre0"], dpre_beta=g["beta0"], dgate=g["gate0"], **s)


def reference(par, mbs):
    """The block in float64, differentiated."""
    p = {k: v.double().requires_grad_(True) for k, v in par.items() if k != "act"}
    outs, total = [], 0.0

    def rms(x, gamma):
        return gamma * x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)

    acts = {"gelu": lambda z: z * torch.special.ndtr(z), "relu2": lambda z: torch.relu(z) ** 2, "silu": lambda z: z * torch.sigmoid(z)}
    for m in mbs:
        x0, y0 = (m[k].double().requires_grad_(True) for k in ("x0", "y0"))
        h0 = x0 + p["gate0"] * y0
        n0 = (h0 - h0.mean(1, keepdim=True)) / torch.sqrt(h0.var(1, unbiased=False, keepdim=True) + EPS) * p["pre0"] + p["beta0"]
        y2 = acts[par["act"]](n0 @ p["w1"].T + p["b1"]) @ p["w2"].T + p["b2"]
        h1 = A1 * h0 + B1 * p["gate1"] * rms(y2, p["post"])
        n1 = rms(h1, p["pre1"])
        total = total + (n1 * m["dn1"].double()).sum() + (h1 * m["dres1"].double()).sum()
        outs.append((x0, y0, h1, n1))
    total.backward()
    return {k: v.grad for k, v in p.items()}, outs


def cuda_batches(mbs):
    return [{k: v.cuda() for k, v in m.items()} for m in mbs]


@pytest.mark.parametrize("act", ["gelu", "relu2", "silu"])
def test_training_step_against_differentiation(cuda_device, act):
    par, mbs = parameters(1, act), [microbatch(2, 300), microbatch(3, 77)]
    block = Block(par)
    grads, outs = reference(par, mbs)
    for m, (x0, y0, h1, n1) in zip(cuda_batches(mbs), outs):
        b = block.buffers(m["x0"].shape[0])
        block.step(m, b)
        for name, got, ref in (("h1", b["h1"], h1), ("n1", b["n1"], n1), ("dx0", b["dh0"], x0.grad), ("dy0", b["dy0"], y0.grad)):
            fro, _ = errors(got.double().cpu().numpy(), ref.detach().numpy())
            assert fro <= BAR, (name, fro)
    for k, ref in grads.items():
        fro, _ = errors(block.grads[k].cpu().numpy(), ref.numpy())
        assert fro <= BAR, (k, fro)
    assert zb.zb_device_status() == (0, 0)


def eager(par, mbs, times=1):
    block = Block(par)
    bufs = [block.buffers(m["x0"].shape[0]) for m in mbs]
    for _ in range(times):
        for m, b in zip(mbs, bufs):
            block.step(m, b)
    torch.cuda.synchronize()
    return block, bufs


def assert_same(block, bufs, other, other_bufs):
    for k in block.grads:
        assert torch.equal(block.grads[k], other.grads[k]), k
    for b, o in zip(bufs, other_bufs):
        for k in b:
            if torch.is_tensor(b[k]) and k != "scratch":
                assert torch.equal(b[k], o[k]), k


def test_captured_and_replayed(cuda_device):
    """A step captured in a graph and replayed three times gives the bits of three eager ones, and replays take new inputs."""
    par, mbs = parameters(4, "gelu"), cuda_batches([microbatch(5, 200), microbatch(6, 333)])
    ref, ref_bufs = eager(par, mbs, times=3)
    block = Block(par)
    bufs = [block.buffers(m["x0"].shape[0]) for m in mbs]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for m, b in zip(mbs, bufs):
            block.step(m, b)
    for g in block.grads.values():
        assert torch.all(g == 0.0)  # captured, not run
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert_same(block, bufs, ref, ref_bufs)
    fresh = cuda_batches([microbatch(7, 200), microbatch(8, 333)])
    for m, f in zip(mbs, fresh):
        for k in m:
            m[k].copy_(f[k])
    for g in (*block.grads.values(), *ref.grads.values()):
        g.zero_()
    graph.replay()
    for m, b in zip(fresh, ref_bufs):
        ref.step(m, b)
    torch.cuda.synchronize()
    assert_same(block, bufs, ref, ref_bufs)


def test_two_streams_at_once(cuda_device):
    """Two blocks with buffers of their own, on two streams without an order between them, and on the default stream."""
    par, mbs = parameters(9, "silu"), cuda_batches([microbatch(10, 150)])
    ref, ref_bufs = eager(par, mbs, times=4)
    blocks = [Block(par) for _ in range(2)]
    bufs = [b.buffers(150) for b in blocks]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for block, b, s in zip(blocks, bufs, streams):
            block.step(mbs[0], b, stream=s)
    torch.cuda.synchronize()
    for block, b in zip(blocks, bufs):
        assert_same(block, [b], ref, ref_bufs)


def test_one_row_and_a_non_finite_one(cuda_device):
    """A microbatch of one token; a row that is not finite spoils no other row of the input gradients."""
    par = parameters(11, "gelu")
    mbs = cuda_batches([microbatch(12, 1), microbatch(13, 70)])
    ref, ref_bufs = eager(par, mbs)
    assert torch.all(torch.isfinite(ref_bufs[0]["dy0"]))
    bad = [mbs[0], {k: v.clone() for k, v in mbs[1].items()}]
    bad[1]["x0"][40, 3] = float("inf")
    block, bufs = eager(par, bad)
    rows = torch.arange(70, device="cuda") != 40
    for k in ("h0", "n0", "y1", "h1", "n1", "dh1", "dy2", "dz", "dn0", "dh0", "dy0"):
        assert torch.equal(bufs[1][k][rows], ref_bufs[1][k][rows]), k
    for k in ("n0", "y1", "n1", "dy0"):
        assert not torch.all(torch.isfinite(bufs[1][k][40])), k
    assert zb.zb_device_status() == (0, 0)


@pytest.mark.parametrize("t", [40, 1000])
def test_projection_into_document_attention(cuda_device, t):
    """The output projection's B, and the attention's backward right behind it on the stream: the attention's first kernel may
    start beside the projection's, and reads its result only once that has ended."""
    nh, nkv, d, out = 8, 4, 128, 1024
    g = torch.Generator()
    g.manual_seed(t)
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    qkv, w, dys = bf(t, (nh + 2 * nkv) * d), bf(out, nh * d), [bf(t, out) for _ in range(8)]
    new = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    plan = new(zb.zb_op_attention_document_plan_bytes(t), dtype=torch.uint8)
    offsets = torch.tensor([0, t // 3, t], dtype=torch.int32, device="cuda")
    zb.zb_op_attention_document_plan(offsets, None, 2, t, plan, plan.numel())
    a, lse = new(t, nh * d), new(nh, max(128, (t + 127) // 128 * 128), dtype=torch.float32)
    zb.zb_op_attention_document_forward(qkv, a, lse, plan, None, 0.0, t, nh, nkv, d)
    scratch = new(zb.zb_op_attention_document_scratch_bytes(t, nh), dtype=torch.uint8)

    def run(wait):
        da, outs = new(t, nh * d), []
        for dy in dys:
            dqkv = new(t, (nh + 2 * nkv) * d)
            outs.append(dqkv)
            zb.zb_op_backward_input_activation(dy, w, None, da, t, nh * d, out, "none")
            if wait:
                torch.cuda.synchronize()
            zb.zb_op_attention_document_backward(qkv, a, da, lse, dqkv, plan, None, 0.0, t, nh, nkv, d, scratch, scratch.numel())
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return outs

    for x, y in zip(run(True), run(False)):
        assert torch.equal(x, y)
    assert zb.zb_device_status() == (0, 0)


FIRST_CALL = """
import torch
import test_gpu_block_step as step
par, mbs = step.parameters(4, "gelu"), step.cuda_batches([step.microbatch(5, 200)])
block = step.Block(par)
bufs = [block.buffers(200)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
    block.step(mbs[0], bufs[0])
graph.replay()
torch.cuda.synchronize()
ref, ref_bufs = step.eager(par, mbs)
step.assert_same(block, bufs, ref, ref_bufs)
assert step.zb.zb_device_status() == (0, 0)
"""


def test_first_call_inside_a_capture(cuda_device):
    """A process whose first calls are captured: nothing is set up ahead of them that a capture would refuse."""
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]


def test_offsets_past_32_bits(cuda_device):
    """Tensors of 4.3e9 elements, all zeros but for the last row: it comes out as it does in a call of its own, and its
    products, the only ones that are not zero, are the weight gradients."""
    t, w = 2 ** 20 + 37, 4096
    g = torch.Generator()
    g.manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    zeros = lambda width, dtype=torch.bfloat16: torch.zeros(t, width, dtype=dtype, device="cuda")  # noqa: E731
    one = lambda width, dtype=torch.bfloat16: torch.zeros(1, width, dtype=dtype, device="cuda")  # noqa: E731
    row, small = n(1, w).to(torch.bfloat16), n(1, 64).to(torch.bfloat16)
    big, big_small = zeros(w), zeros(64)
    big[-1], big_small[-1] = row[0], small[0]

    # packing, F and B
    codes, scales = zeros(w, torch.uint8), zeros(w // 32, torch.uint8)
    c1, s1 = one(w, torch.uint8), one(w // 32, torch.uint8)
    zb.zb_op_checkpoint_pack(big, (codes, scales), t, w)
    zb.zb_op_checkpoint_pack(row, (c1, s1), 1, w)
    assert torch.equal(codes[-1:], c1) and torch.equal(scales[-1:], s1)
    weight, bias = (n(w, 64) / 8).to(torch.bfloat16), n(w)
    y, y1 = zeros(w), one(w)
    zb.zb_op_linear_activation_forward(big_small, weight, bias, None, y, t, 64, w, "gelu", z_packed=(codes, scales))
    zb.zb_op_linear_activation_forward(small, weight, bias, None, y1, 1, 64, w, "gelu", z_packed=(c1, s1))
    assert torch.equal(y[-1:], y1) and torch.equal(codes[-1:], c1) and torch.equal(scales[-1:], s1)
    back = (n(64, w) / 8).to(torch.bfloat16)
    db, db1 = (torch.zeros(w, device="cuda") for _ in range(2))
    scratch = torch.empty(zb.zb_op_backward_input_activation_scratch_bytes(t, w), dtype=torch.uint8, device="cuda")
    zb.zb_op_backward_input_activation(big_small, back, None, y, t, w, 64, "gelu", z_packed=(codes, scales), dbias=db, scratch=scratch)
    zb.zb_op_backward_input_activation(small, back, None, y1, 1, w, 64, "gelu", z_packed=(c1, s1), dbias=db1, scratch=scratch)
    assert torch.equal(y[-1:], y1) and torch.equal(db, db1) and torch.any(db != 0.0)
    assert torch.all(y[-2] == 0.0)

    # W from 8 bits
    zb.zb_op_checkpoint_pack(big, (codes, scales), t, w)
    scratch = torch.empty(zb.zb_op_backward_weight_checkpoint_scratch_bytes(t, w), dtype=torch.uint8, device="cuda")
    dw = torch.zeros(64, w, device="cuda")
    zb.zb_op_backward_weight_checkpoint(big_small, (codes, scales), dw, t, w, 64, scratch)
    zb.zb_op_checkpoint_unpack((codes, scales), y, t, w)
    assert torch.equal(dw, small[0].float()[:, None] * y[-1].float())
    del scratch, codes, scales

    # the norms
    gamma = 1.0 + 0.1 * n(w)
    op = zb.make_residual_norm(post="rms", pre="layer", post_gamma=gamma, pre_gamma=gamma)
    h, normed, st, h1, n1, st1 = zeros(w), zeros(w), zeros(4, torch.float32), one(w), one(w), one(4, torch.float32)
    zb.zb_op_residual_norm_forward(op, big, big, h, normed, st, t, w)
    zb.zb_op_residual_norm_forward(op, row, row, h1, n1, st1, 1, w)
    assert torch.equal(h[-1:], h1) and torch.equal(normed[-1:], n1) and torch.equal(st[-1:], st1)
    dh, dy, dh1, dy1 = zeros(w), y, one(w), one(w)
    zb.zb_op_residual_norm_backward_input(op, big, big, h, big, st, dh, dy, t, w)
    zb.zb_op_residual_norm_backward_input(op, row, row, h1, row, st1, dh1, dy1, 1, w)
    assert torch.equal(dh[-1:], dh1) and torch.equal(dy[-1:], dy1)
    scratch = torch.empty(zb.zb_op_residual_norm_backward_weight_scratch_bytes(t, w), dtype=torch.uint8, device="cuda")
    grads, grads1 = ([torch.zeros(w, device="cuda") for _ in range(2)] for _ in range(2))
    for a, (d, x, e, v, s, rows) in ((grads, (big, h, dh, big, st, t)), (grads1, (row, h1, dh1, row, st1, 1))):
        zb.zb_op_residual_norm_backward_weight(op, d, x, e, v, s, rows, w, scratch, dpost_gamma=a[0], dpre_gamma=a[1])
    for a, b in zip(grads, grads1):
        assert torch.equal(a, b) and torch.any(a != 0.0)
    assert zb.zb_device_status() == (0, 0)
