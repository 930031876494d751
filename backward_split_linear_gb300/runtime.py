"""Owning wrapper around a libzb stage: device weights, float32 accumulators, workspace.

Marshalling and ownership only; every step runs in libzb's kernels.
"""
from __future__ import annotations

import numpy as np
import torch

from . import binding as zb

# parameter name -> accumulator field of zb_layer_params
GRAD_FIELD = {"w_qkv": "dw_qkv", "w_o": "dw_o", "w_gu": "dw_gu", "w_down": "dw_down",
              "gamma1": "dgamma1", "gamma2": "dgamma2", "w": "dw"}


def bf16_from_bits(bits, device="cuda"):
    """uint16 bf16 bit patterns (numpy) -> torch.bfloat16 tensor on `device`."""
    t = torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16)
    return t.to(device)


def bits_from_bf16(t):
    """torch.bfloat16 tensor -> uint16 numpy bit patterns (host)."""
    return t.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def f64_from_bf16(t):
    return (bits_from_bf16(t).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


class Stage:
    """One pipeline stage on the current CUDA device."""

    def __init__(self, kind, n_layers, hidden, ffn, n_heads=0, n_kv_heads=0, head_dim=0, eps=1e-5,
                 max_tokens=128, max_inflight=1, params=None, device="cuda", attention="standin", seq_len=0):
        self.kind = kind
        self.hidden, self.ffn = hidden, ffn
        self.out_dim = ffn if kind == "linear" else hidden
        self.cfg = zb.make_config(kind, n_layers, hidden, ffn, n_heads, n_kv_heads, head_dim, eps,
                                  max_tokens, max_inflight, attention, seq_len)
        nbytes = zb.zb_stage_workspace_bytes(self.cfg)
        if nbytes == 0:
            raise zb.ZBError(-1, "zb_stage_workspace_bytes (invalid config)")
        self.workspace = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
        off = (-self.workspace.data_ptr()) % 256
        self.ws_ptr = self.workspace.data_ptr() + off
        self.ws_bytes = nbytes
        self.params = params  # list of dicts name -> device tensor
        self.grads = []
        layers = []
        for prm in params:
            d, g = {}, {}
            for name, t in prm.items():
                d[name] = t
                acc = torch.zeros(t.shape, dtype=torch.float32, device=device)
                g[name] = acc
                d[GRAD_FIELD[name]] = acc
            layers.append(d)
            self.grads.append(g)
        self.handle = zb.zb_stage_create(self.cfg, layers, self.ws_ptr, self.ws_bytes)
        # every table that the library was given (see set_attention), the frequencies' by their values
        self.turns, self.slopes = {}, []

    @staticmethod
    def from_synth(kind, n_layers, hidden, ffn, n_heads=0, n_kv_heads=0, head_dim=0, eps=1e-5,
                   max_tokens=128, max_inflight=1, params_bits=None, device="cuda", attention="standin", seq_len=0):
        params = []
        for layer in params_bits:
            params.append({k: (bf16_from_bits(v, device) if v.dtype == np.uint16
                               else torch.from_numpy(v).to(device)) for k, v in layer.items()})
        return Stage(kind, n_layers, hidden, ffn, n_heads, n_kv_heads, head_dim, eps, max_tokens,
                     max_inflight, params, device, attention, seq_len)

    def zero_grads(self):
        for g in self.grads:
            for t in g.values():
                t.zero_()

    def set_attention(self, rotary_dim=0, pairs="half", base=10000.0, scaling="none", factor=1.0, context=0.0, low=1.0,
                      high=None, cap=0.0, slopes=None):
        """Rotary positions, a tanh cap and distance slopes of the stage's softmax attention (see `zb_stage_set_attention`;
        the frequencies' arguments are those of `binding.zb_rotary_frequencies`).  `slopes`: float32 [n_heads].  The stage
        keeps the tables of earlier calls: a stream may still hold kernels that read them, and a captured graph always does."""
        turns, magnitude = None, 1.0
        if slopes is not None and (slopes.dtype != torch.float32 or not slopes.is_contiguous() or slopes.numel() != self.cfg.n_heads
                                   or slopes.device != self.workspace.device):
            raise zb.ZBError(-1, "Stage.set_attention (slopes are float32 [n_heads] on the stage's device)")
        if rotary_dim:
            values, magnitude = zb.zb_rotary_frequencies(rotary_dim, base, scaling, factor, context, low, high)
            turns = self.turns.get(tuple(values))
            if turns is None:
                turns = torch.from_numpy(np.array(values, dtype=np.uint64).view(np.int64)).to(self.workspace.device)
                self.turns[tuple(values)] = turns
        if slopes is not None and not any(slopes is t for t in self.slopes):
            self.slopes.append(slopes)
        zb.zb_stage_set_attention(self.handle, rotary_dim, pairs, turns, magnitude, cap, slopes)

    def forward(self, mb, x, y, stream=None, documents=None, prefix=None):
        """`documents`: int32 row offsets of packed documents (attention "document"), `prefix` their prefix lengths."""
        if documents is None and prefix is None:
            zb.zb_stage_forward(self.handle, mb, x, x.shape[0], y, stream)
            return
        for t, n in ((documents, None), (prefix, documents.numel() - 1 if documents is not None else 1)):
            if t is not None and (t.dtype != torch.int32 or not t.is_contiguous() or t.device != x.device
                                  or (n is not None and t.numel() != n)):
                raise zb.ZBError(-1, "Stage.forward (documents and prefix are contiguous int32 beside x)")
        zb.zb_stage_forward_documents(self.handle, mb, x, x.shape[0], documents, prefix,
                                      documents.numel() - 1 if documents is not None else 1, y, stream)

    def backward_input(self, mb, dy, dx, stream=None):
        zb.zb_backward_input(self.handle, mb, dy, dx, stream)

    def backward_weight(self, mb, stream=None):
        zb.zb_backward_weight(self.handle, mb, stream)

    def flush(self, stream=None):
        zb.zb_wgrad_flush(self.handle, stream)

    def sync(self, stream=None):
        zb.zb_stage_sync(self.handle, stream)

    def stats(self):
        return zb.zb_stage_stats(self.handle)

    def stash(self, mb, layer, name):
        """A view (no copy) of one stashed tensor of microbatch `mb`, layer `layer`, inside the
        workspace: bf16 [rows, cols] or float32 [rows, cols].  Valid until the microbatch's W."""
        ptr, rows, cols, eb = zb.zb_stage_stash_view(self.handle, mb, layer, name)
        off = ptr - self.workspace.data_ptr()
        nbytes = rows * cols * eb
        if off < 0 or off + nbytes > self.workspace.numel():
            raise zb.ZBError(-1, "zb_stage_stash_view (address outside the workspace)")
        raw = self.workspace[off:off + nbytes]
        return raw.view(torch.bfloat16 if eb == 2 else torch.float32).view(rows, cols)

    def set_tracing(self, enable):
        zb.zb_stage_set_tracing(self.handle, enable)

    def read_tracing(self, reset=True):
        return zb.zb_stage_read_tracing(self.handle, reset)

    def close(self):
        if self.handle:
            zb.zb_stage_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class AdamW:
    """AdamW over a list of tensors, or over a stage's parameters and accumulators (`for_stage`).

    Each entry of `tensors` is a dict with param, grad, m and v, and where they apply master, m_scale, v_scale and
    weight_decay (see `binding.adamw_table`).  The object keeps the tensors, the step number and the norm's scratch; it
    allocates nothing after it is made, so `grad_norm` and `step` can be captured into a graph (then with `step_device`,
    the device's step number, which the graph itself advances).
    """

    def __init__(self, tensors, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, state_bits=32, stochastic=False, seed=0, step=0,
                 step_device=None, lr_device=None):
        self.tensors = [dict(t) for t in tensors]  # the table has their addresses: not the caller's dicts, which may change
        self.table = zb.adamw_table(self.tensors)
        self.cfg = zb.make_adamw_config(lr, beta1, beta2, eps, state_bits, stochastic, seed)
        self.steps = step
        self.step_device, self.lr_device = step_device, lr_device
        want = torch.uint8 if state_bits == 8 else torch.float32
        if any(t["m"].dtype != want or t["v"].dtype != want for t in self.tensors):
            raise zb.ZBError(-1, f"AdamW (moments of {state_bits} bits are {want})")
        device = self.tensors[0]["param"].device if self.tensors else torch.device("cuda", zb._current_device())
        self.device = device
        self.index = device.index if device.type == "cuda" else None
        self._check_scalar("AdamW", "step_device", step_device, torch.int64)
        self._check_scalar("AdamW", "lr_device", lr_device, torch.float32)
        nbytes = zb.zb_op_grad_norm_scratch_bytes(self.table, len(self.tensors))
        self.scratch = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.norm = torch.zeros(4, dtype=torch.float32, device=device)  # norm, clip coefficient
        self.norm_views = (self.norm[0], self.norm[1])
        self.stage = None
        self._states = None

    @staticmethod
    def for_stage(stage, lr=1e-3, weight_decay=0.1, state_bits=32, master=True, **kw):
        """Over every parameter of a `Stage`, with fresh moments: weights decay, RMSNorm gammas do not.  `master`: float32
        copies of the bf16 weights."""
        tensors = []
        for prm, grads in zip(stage.params, stage.grads):
            for name, p in prm.items():
                n, dev = p.numel(), p.device
                t = {"param": p, "grad": grads[name], "weight_decay": weight_decay if p.dtype == torch.bfloat16 else 0.0}
                if master and p.dtype == torch.bfloat16:
                    t["master"] = p.float()
                for s in ("m", "v"):
                    t[s] = torch.zeros(n, dtype=torch.uint8 if state_bits == 8 else torch.float32, device=dev)
                    if state_bits == 8:
                        t[s + "_scale"] = torch.zeros((n + 255) // 256, dtype=torch.float32, device=dev)
                tensors.append(t)
        opt = AdamW(tensors, lr=lr, state_bits=state_bits, **kw)
        opt.stage = stage
        return opt

    def _check_scalar(self, call, name, t, dtype):
        if t is not None and (t.dtype != dtype or t.numel() != 1 or t.device != self.device):
            raise zb.ZBError(-1, f"{call} ({name} is one {dtype} on {self.device}, the tensors' device)")

    def _check_device(self, call):
        """The library launches on the current device, whose kernels must not read another one's memory or the host's."""
        if self.index is None or self.index != zb._current_device():
            raise zb.ZBError(-1, f"AdamW.{call} (the tensors lie on {self.device}, which is not the current device)")

    def grad_norm(self, max_norm=1.0, stream=None):
        """(norm, clip coefficient) of all the gradients: float32 scalars on the device, rewritten by the next call."""
        self._check_device("grad_norm")
        zb.zb_op_grad_norm(self.table, len(self.tensors), max_norm, self.norm, self.scratch, self.scratch.numel(), stream)
        return self.norm_views

    def step(self, grad_scale=None, stream=None):
        """One update (one that a scale which is not finite skips counts too).  A stage's weights must not change between F
        and W of a microbatch: its microbatches must all have run their W."""
        if self.stage is not None and self.stage.stats()[0] != 0:
            raise zb.ZBError(-3, "AdamW.step (microbatches of the stage still wait for their W)")
        if grad_scale is not self.norm_views[1]:
            self._check_scalar("AdamW.step", "grad_scale", grad_scale, torch.float32)
        self._check_device("step")
        zb.zb_op_adamw_step(self.table, len(self.tensors), self.cfg, self.steps + 1, grad_scale, self.lr_device,
                            self.step_device, stream)
        self.steps += 1

    def unpack_states(self, stream=None):
        """[(m, v)] as float32 values; 8-bit states are written into buffers that the next call rewrites."""
        if self.cfg.state_bits != 8:
            return [(t["m"], t["v"]) for t in self.tensors]
        self._check_device("unpack_states")
        if self._states is None:
            self._states = [tuple(torch.empty(t["m"].numel(), dtype=torch.float32, device=t["m"].device) for _ in range(2))
                            for t in self.tensors]
        zb.zb_op_adamw_unpack(self.table, len(self.tensors), [m for m, _ in self._states], [v for _, v in self._states],
                              stream)
        return self._states
