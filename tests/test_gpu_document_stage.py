"""A stage of packed documents as a training step uses it: rotary positions, document attention, F / B / W in a ZB-H1
order, flush, clip and AdamW, against the float64 oracle.

Bars: the causal stage's (tests/parity.py): eight roundings a layer, Frobenius <= 5e-3 sqrt(8 L), max <= 3e-2 max|ref|.
Rotary positions add one rounding of q and k forward and one of dq and dk backward, two of eight more: 5e-3 sqrt(10 L).
The cap's derivative is at most one and the distance bias has none, so neither widens them.
"""
import numpy as np
import pytest
import torch

from backward_split_linear_gb300 import binding as zb
from backward_split_linear_gb300 import synth
from backward_split_linear_gb300.runtime import AdamW, Stage, bf16_from_bits, f64_from_bf16
from oracle import stage as S
from oracle import train_ops as O
from parity import CAUSAL_MAX_TOL, FRO_TOL, assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _status_clean(cuda_device):
    zb.zb_device_status(reset=True)
    yield
    st, code = zb.zb_device_status()
    assert st == 0, f"device status word set: {code}"


def shape(L, H, F, nh, nkv, hd):
    return dict(kind="transformer", n_layers=L, hidden=H, ffn=F, n_heads=nh, n_kv_heads=nkv, head_dim=hd, eps=1e-5)


def close(got, ref, what, layers):
    assert_close(got, ref, what, FRO_TOL * float(np.sqrt(10 * layers)), CAUSAL_MAX_TOL)


def ints(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


CASES = [  # tokens of each microbatch, their documents and prefixes, heads, options
    # at least 256 tokens: D comes from the output projection's dgrad
    (2, 256, 512, 4, 2, 64, 300, [([0, 100, 290], [10, 0]), ([0, 300], None)],
     dict(rotary_dim=64, pairs="half", scaling="banded", factor=4.0, context=64.0, low=1.0, high=4.0, cap=20.0)),
    # fewer: D comes from the row kernel; part of each head turns; padding at both ends
    (1, 256, 512, 2, 1, 128, 131, [([3, 60, 60, 120], [5, 2, 70]), ([0, 131], [131]), ([0, 1, 2, 131], None)],
     dict(rotary_dim=32, pairs="interleaved", scaling="yarn", factor=4.0, context=64.0, slopes=True)),
    (2, 384, 512, 6, 2, 64, 256, [([0, 256], None)], dict()),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_training_step_against_the_oracle(case):
    L, H, F, nh, nkv, hd, T, batches, opts = CASES[case]
    m = len(batches)
    c = shape(L, H, F, nh, nkv, hd)
    inp = synth.stage_inputs("transformer", L, H, F, nh, nkv, hd, tokens=T, n_mb=m, seed=20 + case)
    st = Stage.from_synth("transformer", L, H, F, nh, nkv, hd, 1e-5, T, m, inp["params"], attention="document")
    opts = dict(opts)
    slopes = torch.exp2(-4.0 * torch.arange(1, nh + 1, device="cuda") / nh) if opts.pop("slopes", False) else None
    st.set_attention(slopes=slopes, **opts)
    rotary = None
    if opts.get("rotary_dim"):
        kw = {k: opts[k] for k in ("scaling", "factor", "context", "low", "high") if k in opts}
        rotary = O.rotary_frequencies(opts["rotary_dim"], 10000.0, **kw) + (opts["pairs"],)
    params = synth.params_f64(inp["params"])
    grads = S.zero_grads(params)
    y, dx = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    want, got = {}, {}
    for kind, mb in zb.zb_schedule("zbh1", 0, m, m):
        off, pre = batches[mb]
        shp = dict(c, attention="document", offsets=off, prefix=pre, cap=opts.get("cap", 0.0), rotary=rotary,
                   slopes=None if slopes is None else slopes.double().cpu().numpy())
        if kind == "F":
            if off == [0, T] and pre is None:
                st.forward(mb, bf16_from_bits(inp["x"][mb]), y)   # the call without documents
            else:
                st.forward(mb, bf16_from_bits(inp["x"][mb]), y, documents=ints(off), prefix=ints(pre))
            ref, saved = S.stage_forward(synth.bf16_to_f64(inp["x"][mb]), params, shp)
            close(f64_from_bf16(y), ref, f"y of {mb}", L)
            want[mb] = (saved, shp)
        elif kind == "B":
            st.backward_input(mb, bf16_from_bits(inp["dy"][mb]), dx)
            saved, shp = want[mb]
            ref, kept = S.stage_backward_input(synth.bf16_to_f64(inp["dy"][mb]), params, saved, shp)
            close(f64_from_bf16(dx), ref, f"dx of {mb}", L)
            got[mb] = kept
        elif mb % 2 == 0:  # the others wait for the flush
            st.backward_weight(mb)
    for mb in range(m):
        S.stage_backward_weight(grads, want[mb][0], got[mb], want[mb][1])
    st.flush()
    for li in range(L):
        for k, ref in grads[li].items():
            close(st.grads[li][k].cpu().numpy(), ref, f"d{k} of layer {li}", L)
    opt = AdamW.for_stage(st, lr=1e-3, state_bits=8 if case == 0 else 32)
    before = [t["param"].double().cpu().numpy().reshape(-1) for t in opt.tensors]
    norm, scale = opt.grad_norm(1.0)
    opt.step(grad_scale=scale)
    st.sync()
    total = np.sqrt(sum(float((g.double() ** 2).sum()) for layer in st.grads for g in layer.values()))
    assert abs(float(norm) - total) <= 2.0 ** -20 * total
    for t, p0 in zip(opt.tensors, before):
        g = t["grad"].double().cpu().numpy().reshape(-1) * float(scale)
        p, _, _ = O.adamw(p0, g, 0.0, 0.0, 1, 1e-3, 0.9, 0.95, 1e-8, t["weight_decay"])
        new = (t["master"] if "master" in t else t["param"]).double().cpu().numpy().reshape(-1)
        assert np.all(np.abs(new - p) <= 3 * 2.0 ** -24 * np.abs(p0) + 20 * 2.0 ** -24 * 1e-3)
    st.close()


def test_stash_feeds_the_oracle():
    """The attention core and its rotary positions apart from earlier roundings: a and dqkv from the stashed tensors."""
    L, H, F, nh, nkv, hd, T = 1, 512, 512, 4, 1, 128, 400
    off, pre = [0, 130, 390], [0, 40]
    inp = synth.stage_inputs("transformer", L, H, F, nh, nkv, hd, tokens=T, n_mb=1, seed=5)
    st = Stage.from_synth("transformer", L, H, F, nh, nkv, hd, 1e-5, T, 1, inp["params"], attention="document")
    st.set_attention(rotary_dim=128, cap=10.0)
    y, dx = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st.forward(0, bf16_from_bits(inp["x"][0]), y, documents=ints(off), prefix=ints(pre))
    st.sync()
    n1, qkv, a = (f64_from_bf16(st.stash(0, 0, k)) for k in ("n1", "qkv", "a"))
    prm = synth.params_f64(inp["params"])[0]
    shp = dict(shape(L, H, F, nh, nkv, hd), attention="document", offsets=off, prefix=pre, cap=10.0,
               rotary=O.rotary_frequencies(128) + ("half",))
    # qkv is rounded before and after the turn: two roundings of the projection's output
    assert_close(qkv, S._turned(n1 @ prm["w_qkv"].T, shp), "turned qkv")
    see = O.document_visible(T, off, pre)
    assert_close(a, O.document_attention(qkv, nh, nkv, hd, see, 10.0)[0], "a")
    assert np.all(a[390:] == 0.0)
    st.backward_input(0, bf16_from_bits(inp["dy"][0]), dx)
    st.sync()
    dh, dqkv = (f64_from_bf16(st.stash(0, 0, k)) for k in ("dh", "dqkv"))
    ref = S._turned(O.document_attention_grad(dh @ prm["w_o"], qkv, nh, nkv, hd, see, 10.0), shp, backward=True)
    assert_close(dqkv, ref, "dqkv")
    assert np.all(dqkv[390:] == 0.0)
    st.close()


def test_tensors_of_the_host_are_refused():
    inp = synth.stage_inputs("transformer", 1, 256, 512, 2, 1, 128, tokens=128, n_mb=1, seed=3)
    st = Stage.from_synth("transformer", 1, 256, 512, 2, 1, 128, 1e-5, 128, 1, inp["params"], attention="document")
    x, y = (torch.zeros(128, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    off = torch.tensor([0, 128], dtype=torch.int32)
    for call in (lambda: st.set_attention(slopes=torch.zeros(2)), lambda: st.set_attention(slopes=torch.zeros(1, device="cuda")),
                 lambda: st.forward(0, x, y, documents=off), lambda: st.forward(0, x, y, prefix=off[1:]),
                 lambda: st.forward(0, x, y, documents=off.cuda(), prefix=off.cuda())):
        with pytest.raises(zb.ZBError) as e:
            call()
        assert e.value.name == "ZB_ERR_ARG"
    st.forward(0, x, y, documents=off.cuda())  # and the stage still works
    st.close()


def test_rotary_in_a_causal_stage():
    L, H, F, nh, nkv, hd, T = 1, 256, 512, 4, 2, 64, 300
    inp = synth.stage_inputs("transformer", L, H, F, nh, nkv, hd, tokens=T, n_mb=1, seed=6)
    st = Stage.from_synth("transformer", L, H, F, nh, nkv, hd, 1e-5, T, 1, inp["params"], attention="causal", seq_len=128)
    st.set_attention(rotary_dim=64, pairs="interleaved")
    shp = dict(shape(L, H, F, nh, nkv, hd), attention="causal", seq_len=128, rotary=O.rotary_frequencies(64) + ("interleaved",))
    params = synth.params_f64(inp["params"])
    y, dx = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st.forward(0, bf16_from_bits(inp["x"][0]), y)
    ref, saved = S.stage_forward(synth.bf16_to_f64(inp["x"][0]), params, shp)
    close(f64_from_bf16(y), ref, "y", L)
    with pytest.raises(zb.ZBError) as e:
        st.set_attention()                      # a microbatch is in flight
    assert e.value.name == "ZB_ERR_ORDER"
    st.backward_input(0, bf16_from_bits(inp["dy"][0]), dx)
    ref, kept = S.stage_backward_input(synth.bf16_to_f64(inp["dy"][0]), params, saved, shp)
    close(f64_from_bf16(dx), ref, "dx", L)
    st.backward_weight(0)
    st.sync()
    grads = S.zero_grads(params)
    S.stage_backward_weight(grads, saved, kept, shp)
    close(st.grads[0]["w_qkv"].cpu().numpy(), grads[0]["w_qkv"], "dw_qkv", L)
    st.close()


def test_tracing_books_the_new_launches():
    L, H, F, nh, nkv, hd, T = 2, 256, 512, 4, 2, 64, 128
    inp = synth.stage_inputs("transformer", L, H, F, nh, nkv, hd, tokens=T, n_mb=1, seed=7)
    st = Stage.from_synth("transformer", L, H, F, nh, nkv, hd, 1e-5, T, 1, inp["params"], attention="document")
    st.set_attention(rotary_dim=64)
    y, dx = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    st.set_tracing(True)
    st.forward(0, bf16_from_bits(inp["x"][0]), y)
    st.backward_input(0, bf16_from_bits(inp["dy"][0]), dx)
    tr = st.read_tracing()
    assert tr["attn_forward"]["launches"] == L and tr["attn_backward"]["launches"] == 2 * L  # 128 tokens: the row kernel too
    # F rows: the plan, and per layer two norms, rotary and SwiGLU
    assert tr["row_forward"]["launches"] == 1 + 4 * L
    assert tr["row_backward_input"]["launches"] == 3 * L
    st.close()


def test_a_captured_stage_step_replays():
    """F, B and W of a documents' microbatch in a graph: replayed on new offsets in the same arrays, it gives the eager
    step's bits."""
    L, H, F, nh, nkv, hd, T = 1, 256, 512, 4, 2, 64, 300
    inp = synth.stage_inputs("transformer", L, H, F, nh, nkv, hd, tokens=T, n_mb=1, seed=8)
    runs = {}
    x, dy = bf16_from_bits(inp["x"][0]), bf16_from_bits(inp["dy"][0])
    for how in ("eager", "graph"):
        st = Stage.from_synth("transformer", L, H, F, nh, nkv, hd, 1e-5, T, 1, inp["params"], attention="document")
        st.set_attention(rotary_dim=64, cap=30.0)
        off = ints([0, 300, 300])
        y, dx = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))

        def step(stream=None):
            st.forward(0, x, y, stream, documents=off)
            st.backward_input(0, dy, dx, stream)
            st.backward_weight(0, stream)

        if how == "graph":
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            step(s)
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                step(s)
        off.copy_(ints([0, 77, 290]))
        st.zero_grads()
        g.replay() if how == "graph" else step()
        torch.cuda.synchronize()
        runs[how] = [y.clone(), dx.clone()] + [t.clone() for t in st.grads[0].values()]
        st.close()
    for a, b in zip(runs["eager"], runs["graph"]):
        assert torch.equal(a, b)


def test_new_attention_options_leave_the_old_tables_in_place():
    """A graph captured under one set of frequencies and slopes, and steps still queued on another stream, read their own
    after the stage has been given others and small tensors have been made."""
    L, H, F, nh, nkv, hd, T = 1, 256, 512, 4, 2, 64, 300
    inp = synth.stage_inputs("transformer", L, H, F, nh, nkv, hd, tokens=T, n_mb=1, seed=12)
    st = Stage.from_synth("transformer", L, H, F, nh, nkv, hd, 1e-5, T, 1, inp["params"], attention="document")
    x, dy = bf16_from_bits(inp["x"][0]), bf16_from_bits(inp["dy"][0])
    y, dx = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    off = ints([0, 77, 290])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        st.forward(0, x, y, s, documents=off)
        st.backward_input(0, dy, dx, s)
        st.backward_weight(0, s)

    def first():
        st.set_attention(rotary_dim=64, slopes=torch.exp2(-torch.arange(1.0, nh + 1, device="cuda")))
        s.wait_stream(torch.cuda.current_stream())

    def others():
        st.set_attention(rotary_dim=32, base=100.0, slopes=torch.full((nh,), 0.25, device="cuda"))
        return [torch.full((n,), 3, dtype=torch.int64, device="cuda") for n in [32, 16, 2] * 50]

    first()
    step()
    s.synchronize()
    want = y.clone(), dx.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    kept = others()
    y.zero_(), dx.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(dx, want[1])
    first()
    y.zero_(), dx.zero_()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        step()  # queued, not waited for
    kept += others()
    torch.cuda.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(dx, want[1])
    st.close()
