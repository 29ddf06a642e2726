"""MoELayer: the layer's weights, configuration and workspace in one object.

A convenience over the C ABI for callers that work in PyTorch: it allocates
the device workspace once (through torch), keeps the weights resident, and
calls ``moe_forward`` (inference), or ``moe_forward_train`` and
``moe_backward`` (training).  It adds no arithmetic of its own.
"""
from __future__ import annotations

import contextlib

import torch

from . import _binding as B


def _same(a, b) -> bool:
    """Both are tensors, and start at the same address."""
    return isinstance(a, torch.Tensor) and isinstance(b, torch.Tensor) and a.data_ptr() == b.data_ptr()


class MoELayer:
    """Token-choice top-k MoE layer (forward and backward)
    on one CUDA device.

    weights: w_router (D, E) fp32; w_gate, w_up (E, D, F); w_down (E, F, D) in
    the layer dtype (bf16 or fp32); optional router_bias (E) fp32.
    """

    def __init__(self, T: int, w_router, w_gate, w_up, w_down, K: int, capacity_factor=0.0,
                 router_bias=None, selection_bias=None, shared=None, experts=None, norm_weight=None,
                 norm_eps: float = 1e-6, **router_options):
        """router_options: score_func ("softmax" | "sigmoid"), renormalize,
        n_groups, topk_groups, route_scale (see moe_config in include/moe.h).
        selection_bias (E) fp32: DeepSeek-V3 bias, for selection only.
        shared: (w_gate_s (D, Fs), w_up_s (D, Fs), w_down_s (Fs, D)), a shared
        expert every token passes through.
        experts: None, or "mx8": inference reads the expert weights in 8 bits
        (moe_mx8_prepare_weight; quantize_experts() again after they change).
        norm_weight (D) fp32, norm_eps: the norm of forward_block and
        forward_block_train."""
        E, D, F = w_gate.shape
        dtype = "bf16" if w_gate.dtype == torch.bfloat16 else "f32"
        fs = 0 if shared is None else shared[0].shape[1]
        self.cfg = B.MoeConfig.make(T, D, F, E, K, dtype, capacity_factor, F_shared=fs,
                                    **router_options)
        self.shared = shared
        self.selection_bias = selection_bias
        st = B.check_config(self.cfg)
        if st != B.MOE_OK:
            raise B.MoEError(st, "MoELayer")
        self.device = w_gate.device
        self.w_router, self.w_gate, self.w_up, self.w_down = w_router, w_gate, w_up, w_down
        self.router_bias = router_bias
        nbytes = B.forward_workspace_size(self.cfg)
        self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
        self.torch_dtype = w_gate.dtype
        self.losses = torch.zeros(3, dtype=torch.float32, device=self.device)  # z, balance, entropy
        self.mean_prob = torch.zeros(E, dtype=torch.float32, device=self.device)
        self.counts = torch.zeros(E, dtype=torch.int32, device=self.device)
        # the router weight split once into the tensor-core router's bf16 terms
        # (moe_router_prepare); split again when w_router is replaced or changed
        # in place (tracked by the tensor's version counter)
        nb = B.router_terms_size(self.cfg)
        self.router_terms = torch.empty(nb, dtype=torch.uint8, device=self.device) if nb else None
        self._terms_of = None
        self.norm_weight, self.norm_eps = norm_weight, norm_eps
        if experts not in (None, "mx8"):
            raise ValueError('experts: None or "mx8"')
        self.mx8 = None
        if experts == "mx8":
            if shared is not None:
                raise ValueError("8-bit experts: a shared expert is not supported")
            nbytes = B.forward_mx8_workspace_size(self.cfg)
            if nbytes > self.workspace.numel():
                self.workspace = torch.zeros(nbytes, dtype=torch.uint8, device=self.device)
            self.quantize_experts()

    def quantize_experts(self, stream=None):
        """The expert weights into the 8-bit layout the layer's inference reads; call
        it again whenever the weights have changed."""
        if self.mx8 is None:
            out = []
            for w in (self.w_gate, self.w_up, self.w_down):
                E, k, n = w.shape
                out.append(torch.empty(E, n, k, dtype=torch.float8_e4m3fn, device=self.device))
                out.append(torch.empty(E, n, k // 32, dtype=torch.uint8, device=self.device))
            self.mx8 = tuple(out)
        for i, w in enumerate((self.w_gate, self.w_up, self.w_down)):
            B.moe_mx8_prepare_weight(w, self.mx8[2 * i], self.mx8[2 * i + 1], stream=stream)

    def _on_device(self):
        """The layer's device as the current one, for calls that go to the current
        device and its current stream."""
        if self.device.type != "cuda" or torch._C._cuda_getDevice() == self.device.index:
            return contextlib.nullcontext()
        return torch.cuda.device(self.device)

    def _terms(self, stream=None):
        if self.router_terms is None:
            return None
        key = (id(self.w_router), self.w_router.data_ptr(), self.w_router._version)
        if key != self._terms_of:
            B.moe_router_prepare(self.cfg, self.w_router, self.router_terms, stream=stream)
            self._terms_of = key
        return self.router_terms

    def forward(self, x, y=None, logit_noise=None, stats: bool = True, stream=None):
        """y = MoE(x) for x (T, D) on the device; returns y.  With stats the
        router's z-loss / balance loss / entropy, mean probabilities and counts are left in
        self.losses, self.mean_prob and self.counts."""
        if y is None:
            y = torch.empty_like(x)
        if self.mx8 is not None:
            return self._forward_mx8(x, y, logit_noise, stats, stream)
        B.moe_forward(self.cfg, x, self.w_router, self.w_gate, self.w_up, self.w_down, y,
                      self.workspace, w_router_terms=self._terms(stream),
                      router_bias=self.router_bias, logit_noise=logit_noise,
                      selection_bias=self.selection_bias, shared=self.shared,
                      losses=self.losses if stats else None,
                      mean_prob=self.mean_prob if stats else None,
                      counts=self.counts if stats else None, stream=stream)
        return y

    def _forward_mx8(self, x, y, logit_noise=None, stats=True, stream=None, xq=None, xs=None):
        with self._on_device():
            B.moe_forward_mx8(self.cfg, x, self.w_router, self.mx8, y, self.workspace, xq=xq, xs=xs,
                              w_router_terms=self._terms(stream), router_bias=self.router_bias,
                              logit_noise=logit_noise, selection_bias=self.selection_bias,
                              losses=self.losses if stats else None,
                              mean_prob=self.mean_prob if stats else None,
                              counts=self.counts if stats else None, stream=stream)
        return y

    def _check_rows(self, where, logit_noise=None, **rows):
        """The block's tensors are whole (T, D) batches of the layer's type on its device."""
        T, D, E = self.cfg.T, self.cfg.D, self.cfg.E
        specs = [(name, t, (self.torch_dtype,), T * D) for name, t in rows.items()]
        specs.append(("logit_noise", logit_noise, (torch.float32,), T * E))
        specs.append(("the layer's workspace", self.workspace, (torch.uint8,), self.workspace.numel()))
        B._check_tensors(where, specs)

    def _norm(self, where, x, residual, y, logit_noise, bits8=False, keep=False):
        """moe_rmsnorm into new buffers: (n, s, q, q_scales, rstd)."""
        if self.norm_weight is None:
            raise ValueError("the layer has no norm_weight")
        if residual is None and _same(x, y):
            raise ValueError(f"{where}: y must not be x, which is the sum the call returns")
        if self.mx8 is None:  # (moe_forward_mx8 checks its tensors itself)
            self._check_rows(where, logit_noise, x=x, residual=residual, y=y)
        n = torch.empty_like(x)
        s = torch.empty_like(x) if residual is not None else None
        q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device) if bits8 else None
        qs = torch.empty(x.shape[0], x.shape[1] // 32, dtype=torch.uint8, device=x.device) if bits8 else None
        rstd = torch.empty(x.shape[0], dtype=torch.float32, device=x.device) if keep else None
        B.moe_rmsnorm(x, self.norm_weight, n, residual=residual, s=s, rstd=rstd, q=q, q_scales=qs,
                      eps=self.norm_eps)
        return n, x if s is None else s, q, qs, rstd

    def forward_block(self, x, residual=None, y=None, logit_noise=None, stats: bool = True):
        """The pre-norm block: s = x + residual, y = MoE(norm(s)); returns (y, s),
        which the next block takes as its x and residual.  With 8-bit experts
        the norm writes the rows they read.  On the current stream."""
        n, s, q, qs, _ = self._norm("forward_block", x, residual, y, logit_noise, bits8=self.mx8 is not None)
        if y is None:
            y = torch.empty_like(x)
        if self.mx8 is not None:
            self._forward_mx8(n, y, logit_noise, stats, xq=q, xs=qs)
        else:
            with self._on_device():
                self.forward(n, y, logit_noise=logit_noise, stats=stats)
        return y, s

    def capture(self, x, y, logit_noise=None, stats: bool = True):
        """One forward over the buffers x -> y captured as a CUDA graph; returns
        the torch.cuda.CUDAGraph (graph.replay() runs the layer again on
        whatever x then holds).  The forward takes no host decision between
        its launches and never synchronises, so all of them form one graph;
        the first call runs outside the capture (one-time kernel attributes).
        Trace events must not be attached while capturing."""
        dev = self.device
        side = torch.cuda.Stream(dev)
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            self.forward(x, y, logit_noise=logit_noise, stats=stats)
        torch.cuda.current_stream(dev).wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.forward(x, y, logit_noise=logit_noise, stats=stats)
        return graph

    def forward_host(self, x_host, y_host, x_dev=None, y_dev=None, logit_noise=None,
                     stream=None):
        """End to end from host memory: copy x_host (pinned) in, run the layer,
        copy y out to y_host (pinned), all on one stream (asynchronous)."""
        s = stream or torch.cuda.current_stream(self.device)
        with torch.cuda.stream(s):
            if x_dev is None:
                x_dev = torch.empty(x_host.shape, dtype=x_host.dtype, device=self.device)
            if y_dev is None:
                y_dev = torch.empty_like(x_dev)
            x_dev.copy_(x_host, non_blocking=True)
            self.forward(x_dev, y_dev, logit_noise=logit_noise, stream=s)
            y_host.copy_(y_dev, non_blocking=True)
        return y_host

    def forward_host_stream(self, x_hosts, y_hosts, logit_noise=None, nbuf: int = 2,
                            events=None):
        """The layer over a sequence of host batches, end to end and pipelined.

        x_hosts / y_hosts: lists of pinned host tensors (T, D).  Three streams:
        the copy in of batch i+1 and the copy out of batch i-1 overlap the
        forward of batch i; device batches are double-buffered.  Returns the
        copy-out stream (synchronise on it, or on `events` when given: a pair of
        timing events recorded before the first copy in and after the last
        copy out)."""
        dev = self.device
        comp = torch.cuda.current_stream(dev)
        h2d = torch.cuda.Stream(dev)
        d2h = torch.cuda.Stream(dev)
        shape, dt = x_hosts[0].shape, x_hosts[0].dtype
        xd = [torch.empty(shape, dtype=dt, device=dev) for _ in range(nbuf)]
        yd = [torch.empty(shape, dtype=dt, device=dev) for _ in range(nbuf)]
        ev_in = [torch.cuda.Event() for _ in range(nbuf)]
        ev_done = [torch.cuda.Event() for _ in range(nbuf)]
        ev_out = [torch.cuda.Event() for _ in range(nbuf)]
        if events is not None:
            h2d.wait_stream(comp)
            events[0].record(h2d)
        for i, (xh, yh) in enumerate(zip(x_hosts, y_hosts)):
            b = i % nbuf
            with torch.cuda.stream(h2d):
                if i >= nbuf:
                    h2d.wait_event(ev_done[b])  # the forward of batch i-nbuf read xd[b]
                xd[b].copy_(xh, non_blocking=True)
                ev_in[b].record(h2d)
            comp.wait_event(ev_in[b])
            if i >= nbuf:
                comp.wait_event(ev_out[b])      # the copy out of batch i-nbuf read yd[b]
            self.forward(xd[b], yd[b], logit_noise=logit_noise, stream=comp)
            ev_done[b].record(comp)
            with torch.cuda.stream(d2h):
                d2h.wait_event(ev_done[b])
                yh.copy_(yd[b], non_blocking=True)
                ev_out[b].record(d2h)
        if events is not None:
            events[1].record(d2h)
        comp.wait_stream(d2h)
        return d2h

    # ----------------------------------------------------------- training
    def forward_train(self, x, y=None, logit_noise=None, stream=None):
        """forward() that keeps the activations moe_backward reads; the state
        buffer is allocated on first use."""
        if self.mx8 is not None:
            raise ValueError("8-bit experts are for inference: train a layer without them")
        if getattr(self, "state", None) is None:
            self.state = torch.zeros(B.train_state_size(self.cfg), dtype=torch.uint8,
                                     device=self.device)
        if y is None:
            y = torch.empty_like(x)
        B.moe_forward_train(self.cfg, x, self.w_router, self.w_gate, self.w_up, self.w_down, y,
                            self.state, router_bias=self.router_bias, logit_noise=logit_noise,
                            selection_bias=self.selection_bias, shared=self.shared,
                            losses=self.losses, mean_prob=self.mean_prob, counts=self.counts,
                            stream=stream)
        self._train_x = x
        self._block = None  # set again by forward_block_train
        return y

    def forward_block_train(self, x, residual=None, y=None, logit_noise=None):
        """forward_block() that keeps what backward_block() reads; returns (y, s)."""
        if self.mx8 is not None:
            raise ValueError("8-bit experts are for inference: train a layer without them")
        n, s, _, _, rstd = self._norm("forward_block_train", x, residual, y, logit_noise, keep=True)
        with self._on_device():
            y = self.forward_train(n, y, logit_noise=logit_noise)
        self._block = (s, rstd)
        return y, s

    def backward_block(self, dy, ds=None, c_balance: float = 0.0, c_z: float = 0.0, grads=None,
                       dlogits_add=None):
        """backward() of the last forward_block_train, through its norm: ds is the
        gradient that arrives at s (None: none), dx the gradient of x and of the
        residual alike, dgamma (D) fp32 the norm weight's."""
        if getattr(self, "_block", None) is None:
            raise RuntimeError("backward_block() needs a forward_block_train() first")
        s, rstd = self._block
        if grads is not None and _same(ds, grads["dx"]):
            raise ValueError("backward_block: ds must not be grads' dx, which is written before ds is read")
        self._check_rows("backward_block", dy=dy, ds=ds)
        with self._on_device():
            grads = self.backward(dy, c_balance, c_z, grads, dlogits_add=dlogits_add)
        if "dgamma" not in grads:
            grads["dgamma"] = torch.empty(s.shape[1], dtype=torch.float32, device=s.device)
        if getattr(self, "norm_workspace", None) is None:
            self.norm_workspace = torch.zeros(B.rmsnorm_backward_workspace_size(*s.shape), dtype=torch.uint8,
                                              device=s.device)
        B.moe_rmsnorm_backward(grads["dx"], s, self.norm_weight, rstd, grads["dx"], grads["dgamma"],
                               self.norm_workspace, ds=ds)
        return grads

    def balance_loss(self, seq_starts, token_mask=None, c_balance: float = 0.0, c_z: float = 0.0):
        """moe_balance_loss of the last forward_train's routing over the sequences
        seq_starts (S + 1) int32 and the tokens of token_mask: a dict of losses
        [z, balance], seq_loss (S), counts (S, E) and dlogits (T, E), the gradient
        of c_balance * balance + c_z * z that backward() adds as dlogits_add.  Malformed
        seq_starts show in the call's own workspace, also in the dict:
        moe_get_device_status(result["workspace"]).  On the current stream."""
        if getattr(self, "_train_x", None) is None:
            raise RuntimeError("balance_loss() needs a forward_train() first")
        if not isinstance(seq_starts, torch.Tensor) or seq_starts.numel() < 2:
            raise ValueError("balance_loss: seq_starts must be a tensor of S + 1 >= 2 borders")
        T, E, K, S = self.cfg.T, self.cfg.E, self.cfg.K, seq_starts.numel() - 1
        lo, io = B.train_state_router(self.cfg)
        logits = self.state[lo:lo + 4 * T * E].view(torch.float32)
        ids = self.state[io:io + 4 * T * K].view(torch.int32)
        f32 = dict(dtype=torch.float32, device=self.device)
        ws = torch.zeros(B.balance_workspace_size(self.cfg, S), dtype=torch.uint8, device=self.device)
        out = dict(losses=torch.empty(2, **f32), seq_loss=torch.empty(S, **f32), dlogits=torch.empty(T, E, **f32),
                   counts=torch.empty(S, E, dtype=torch.int32, device=self.device), workspace=ws)
        B.moe_balance_loss(self.cfg, logits, ids, seq_starts, out["counts"], out["losses"], out["seq_loss"], ws,
                           token_mask=token_mask, dlogits=out["dlogits"], c_balance=c_balance, c_z=c_z)
        return out

    def backward(self, dy, c_balance: float = 0.0, c_z: float = 0.0, grads=None, stream=None, dlogits_add=None):
        """Gradients of sum(dy * y) + c_balance * balance + c_z * z for the
        last forward_train; dlogits_add (T, E) fp32, a further gradient of the
        routing logits (balance_loss()'s), is added to theirs.  Returns a dict of dx (layer dtype) and fp32
        dw_router, db_router (when the layer has a router bias), dw_gate,
        dw_up, dw_down (and dshared); ``grads`` may pass that dict back to
        reuse its buffers."""
        x = getattr(self, "_train_x", None)
        if x is None:
            raise RuntimeError("backward() needs a forward_train() first")
        if getattr(self, "bwd_workspace", None) is None:
            self.bwd_workspace = torch.zeros(B.backward_workspace_size(self.cfg),
                                             dtype=torch.uint8, device=self.device)
        if grads is None:
            f32 = dict(dtype=torch.float32, device=self.device)
            grads = dict(dx=torch.empty_like(x),
                         dw_router=torch.empty(self.w_router.shape, **f32),
                         dw_gate=torch.empty(self.w_gate.shape, **f32),
                         dw_up=torch.empty(self.w_up.shape, **f32),
                         dw_down=torch.empty(self.w_down.shape, **f32))
            if self.router_bias is not None:
                grads["db_router"] = torch.empty(self.router_bias.shape, **f32)
            if self.shared is not None:
                grads["dshared"] = tuple(torch.empty(w.shape, **f32) for w in self.shared)
        B.moe_backward(self.cfg, x, self.w_router, self.w_gate, self.w_up, self.w_down, self.state,
                       dy, grads["dx"], grads["dw_router"], grads["dw_gate"], grads["dw_up"],
                       grads["dw_down"], self.bwd_workspace, c_balance=c_balance, c_z=c_z,
                       db_router=grads.get("db_router"), shared=self.shared,
                       dshared=grads.get("dshared"), stream=stream, dlogits_add=dlogits_add)
        return grads

    def update_selection_bias(self, gamma: float, stream=None):
        """One DeepSeek-V3 balancing step from the last forward's counts."""
        if self.selection_bias is None:
            raise ValueError("the layer has no selection bias")
        B.moe_update_selection_bias(self.cfg, self.counts, gamma, self.selection_bias, stream=stream)
