"""The feed-forward block's operators where their tests by size and kind do not come: gradients asked for alone."""
import pytest
import torch

from backward_split_linear_gb300 import binding as zb

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
