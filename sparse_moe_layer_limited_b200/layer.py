"""MoELayer: owns the device buffers of one layer shape and runs the forward
through the C-ABI calls (route -> dispatch -> experts -> combine -> bias update)
and, in BF16 mode, the layer backward."""
from __future__ import annotations

import torch

from . import _lib as L


class MoELayer:
    """DeepSeekMoE layer on one GPU.

    router_w [N, d] fp32, bias [N] fp32 (updated in place by forward), w13
    [N+1, 2f, d] packed (see moe_pack_w13), w2 [N+1, d, f]; for E4M3 the
    quantised weights and their 128x128-block scales.  All tensors must be on
    the same CUDA device.  Intermediate buffers are allocated once here.

    gather (BF16 only): GEMM1 reads each routed row straight from x through
    perm_tok (moe_expert_ffn_gathered) instead of a permuted copy; dispatch
    then writes no x_perm.

    fused_combine (BF16 only, not with gather): the combine runs inside
    GEMM2's epilogue (moe_expert_ffn_combine) instead of as its own kernel;
    the output is bit-identical.

    norm_w, norm_b [d] fp32 (norm_b optional): a layer norm in front of the
    layer (moe_layer_norm, norm_eps): routing and experts, the shared one
    included, read the normalised rows; backward then returns the gradient of
    the rows before the norm, and of its weight and bias."""

    def __init__(self, shape: L.MoEShape, router_w, bias, w13, w2, w13_scales=None,
                 w2_scales=None, gamma: float = 0.001, gather: bool = False,
                 fused_combine: bool = False, norm_w=None, norm_b=None, norm_eps: float = 1e-5):
        rc = L.check_shape(shape)
        if rc != L.OK:
            raise L.MoEError("moe_check_shape", rc)
        self.shape = s = shape
        self.router_w, self.bias, self.w13, self.w2 = router_w, bias, w13, w2
        self.w13_scales, self.w2_scales = w13_scales, w2_scales
        self.gamma = float(gamma)
        self.gather = bool(gather) and s.dtype == L.DTYPE_BF16
        self.fused_combine = (bool(fused_combine) and s.dtype == L.DTYPE_BF16
                              and not self.gather)
        dev = router_w.device
        i32 = dict(dtype=torch.int32, device=dev)
        xdt = L.x_torch_dtype(s)
        self.topk_idx = torch.empty(s.T, s.K, **i32)
        self.topk_gate = torch.empty(s.T, s.K, dtype=torch.float32, device=dev)
        self.counts = torch.empty(s.N, **i32)
        self.offsets = torch.empty(s.N + 1, **i32)
        self.perm_tok = torch.empty(s.T * s.K, **i32)
        self.slot = torch.empty(s.T, s.K, **i32)
        pdt = torch.float8_e4m3fn if s.dtype == L.DTYPE_E4M3 else xdt
        self.x_perm = (None if self.gather
                       else torch.empty(s.T * s.K, s.d, dtype=pdt, device=dev))
        self.x_perm_scales = (torch.empty(s.d // 128, (s.T * s.K + 3) // 4 * 4, dtype=torch.float32,
                                          device=dev)
                              if s.dtype == L.DTYPE_E4M3 else None)
        self.y_perm = torch.empty(s.T * s.K, s.d, dtype=xdt, device=dev)
        self.y_shared = torch.empty(s.T, s.d, dtype=xdt, device=dev)
        self.y = torch.empty(s.T, s.d, dtype=xdt, device=dev)
        self.ws = torch.zeros(L.workspace_size(s), dtype=torch.uint8, device=dev)
        if norm_w is None and norm_b is not None:
            raise ValueError("norm_b needs norm_w")
        self.norm_w, self.norm_b, self.norm_eps = norm_w, norm_b, float(norm_eps)
        if norm_w is not None:
            self.x_norm = torch.empty(s.T, s.d, dtype=xdt, device=dev)
            self.norm_mean = torch.empty(s.T, dtype=torch.float32, device=dev)
            self.norm_rstd = torch.empty(s.T, dtype=torch.float32, device=dev)

    def norm(self, x, stream=None):
        """The layer's rows after the norm in front of it (x itself without one)."""
        if self.norm_w is None:
            return x
        self._before_norm(x)
        L.moe_layer_norm(x, self.norm_w, self.norm_b, self.norm_eps, self.x_norm, self.norm_mean,
                         self.norm_rstd, stream)
        return self.x_norm

    def _before_norm(self, x):
        """Refuse the rows after the norm where those before it are read."""
        if self.norm_w is not None and x.data_ptr() == self.x_norm.data_ptr():
            raise ValueError("x: the rows before the norm in front of the layer are read here, "
                             "these are the ones that norm(x) returned")

    def _normed(self, x):
        """Refuse rows before the norm where those after it are read."""
        if self.norm_w is not None and x.data_ptr() != self.x_norm.data_ptr():
            raise ValueError("x: with a norm in front of the layer, the experts take the rows that "
                             "norm(x) returned")

    def route(self, x, stream=None):
        """Router on the rows before the norm (norm(x) runs here)."""
        s = self.shape
        x = self.norm(x, stream)
        L.moe_route(s, x, self.router_w, self.bias, self.topk_idx, self.topk_gate, self.counts,
                    self.ws, stream)

    def forward(self, x, update_bias: bool = True, stream=None):
        """y = shared(x) + sum_k gate_k expert_k(x); then (optionally) the bias
        update from this batch's counts.  Returns self.y (overwritten next call)."""
        s = self.shape
        x = self.norm(x, stream)
        L.moe_route(s, x, self.router_w, self.bias, self.topk_idx, self.topk_gate, self.counts,
                    self.ws, stream)
        L.moe_dispatch(s, x, self.topk_idx, self.counts, self.offsets, self.perm_tok, self.slot,
                       self.x_perm, self.x_perm_scales, self.ws, stream)
        self.experts_and_combine(x, stream)
        if update_bias:
            L.moe_bias_update(s, self.counts, self.bias, self.gamma, stream)
        return self.y

    def experts_and_combine(self, x, stream=None):
        """The expert GEMMs and the COMBINE step (one fused launch pair when
        fused_combine is set); writes self.y.  With a norm in front, x is what
        norm(x) returned; other rows are refused."""
        self._normed(x)
        s = self.shape
        if self.fused_combine:
            L.moe_expert_ffn_combine(s, self.x_perm, self.offsets, self.perm_tok, self.slot,
                                     self.topk_gate, x, self.w13, self.w2, self.y_perm,
                                     self.y_shared, self.y, self.ws, stream)
        else:
            self.experts(x, stream)
            L.moe_combine(s, self.y_perm, self.y_shared, self.slot, self.topk_gate, self.y,
                          stream)

    def experts(self, x, stream=None):
        """The expert GEMMs on the dispatched rows (gathered from x or read from x_perm); x as at
        experts_and_combine."""
        self._normed(x)
        s = self.shape
        if self.gather:
            L.moe_expert_ffn_gathered(s, x, self.perm_tok, self.offsets, self.w13, self.w2,
                                      self.y_perm, self.y_shared, self.ws, stream)
        else:
            L.moe_expert_ffn(s, self.x_perm, self.x_perm_scales, self.offsets, x, self.w13,
                             self.w2, self.w13_scales, self.w2_scales, self.y_perm,
                             self.y_shared, self.ws, stream)

    def backward(self, x, dy, w13t, w2t, weight_grads: bool = True, stream=None):
        """Gradients of the last forward (its routing held fixed) given
        dy = dL/dy [T, d], BF16 mode without gather, in the backward order
        COMBINE -> MLP_B -> MLP_W -> DISPATCH:
          moe_combine_backward -> moe_expert_ffn_backward_dx (-> _dw)
          -> moe_route_backward -> moe_dispatch_backward.
        w13t, w2t: the transposed weights (moe_transpose_weights).  Returns
        dict(dx [T, d] bf16, drouter [N, d] fp32, dgate [T, K] fp32, and with
        weight_grads dw13, dw2 laid out like w13, w2).  The bias gets no
        gradient (it only selects experts).  With a norm in front, x is the
        layer's input before it, dx is its gradient, and dnorm_w [d] and (with
        norm_b) dnorm_b [d] fp32 come as well."""
        s = self.shape
        if s.dtype != L.DTYPE_BF16 or self.gather:
            raise ValueError("the layer backward runs in BF16 mode on the x_perm path")
        self._before_norm(x)
        dev, xdt = x.device, L.x_torch_dtype(s)
        if getattr(self, "_bwd", None) is None:
            self._bwd = dict(
                ws=torch.zeros(L.backward_workspace_size(s), dtype=torch.uint8, device=dev),
                dy_perm=torch.empty(s.T * s.K, s.d, dtype=xdt, device=dev),
                dgate=torch.empty(s.T, s.K, dtype=torch.float32, device=dev),
                dx_perm=torch.empty(s.T * s.K, s.d, dtype=xdt, device=dev),
                dx_shared=torch.empty(s.T, s.d, dtype=xdt, device=dev),
                dlogit=torch.empty(s.T, s.K, dtype=torch.float32, device=dev),
                dx_route=torch.empty(s.T, s.d, dtype=torch.float32, device=dev))
        B = self._bwd
        x_in, x = x, (x if self.norm_w is None else self.x_norm)
        dx = torch.empty(s.T, s.d, dtype=xdt, device=dev)
        drouter = torch.empty(s.N, s.d, dtype=torch.float32, device=dev)
        L.moe_combine_backward(s, dy, self.y_perm, self.slot, self.topk_gate, B["dy_perm"],
                               B["dgate"], stream)
        L.moe_expert_ffn_backward_dx(s, self.x_perm, self.offsets, x, self.w13, w13t, w2t,
                                     B["dy_perm"], dy, B["dx_perm"], B["dx_shared"], B["ws"],
                                     stream)
        out = dict(dx=dx, drouter=drouter, dgate=B["dgate"])
        if weight_grads:
            out["dw13"] = torch.empty_like(self.w13)
            out["dw2"] = torch.empty_like(self.w2)
            L.moe_expert_ffn_backward_dw(s, self.x_perm, self.offsets, x, B["dy_perm"], dy,
                                         out["dw13"], out["dw2"], B["ws"], stream)
        L.moe_route_backward(s, x, self.router_w, self.topk_idx, B["dgate"], self.offsets,
                             self.perm_tok, self.slot, B["dlogit"], B["dx_route"], drouter,
                             stream)
        L.moe_dispatch_backward(s, B["dx_perm"], B["dx_shared"], self.slot, B["dx_route"], dx,
                                stream)
        if self.norm_w is not None:
            if "norm" not in B:
                B["norm"] = torch.empty(L.layer_norm_workspace_size(s.T, s.d), dtype=torch.uint8,
                                        device=dev)
            # dx has been rounded to the layer's type once, as it leaves a layer without a norm
            out["dx"] = torch.empty_like(dx)
            out["dnorm_w"] = torch.empty_like(self.norm_w)
            if self.norm_b is not None:
                out["dnorm_b"] = torch.empty_like(self.norm_b)
            L.moe_layer_norm_backward(dx, x_in, self.norm_w, self.norm_mean, self.norm_rstd,
                                      out["dx"], out["dnorm_w"], out.get("dnorm_b"), B["norm"],
                                      stream)
        return out

    def capture(self, x, update_bias: bool = True):
        """Record one forward (route, dispatch, experts, combine and, with
        update_bias, the bias update) on the buffer x into a CUDA graph, so
        that replay() reruns the whole step with one launch from the host.
        One eager forward runs first (it also moves the bias once) so that
        every launch-time set-up happens outside the capture.  The graph keeps
        x's address: copy each new batch into x before replay().  Returns the
        graph."""
        side = torch.cuda.Stream(x.device)
        side.wait_stream(torch.cuda.current_stream(x.device))
        with torch.cuda.stream(side):
            self.forward(x, update_bias)
        torch.cuda.current_stream(x.device).wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.forward(x, update_bias)
        self._graph = graph
        return graph

    def replay(self):
        """Rerun the captured step; returns self.y."""
        self._graph.replay()
        return self.y

    def backward_status(self, clear: bool = False) -> int:
        """Status word of the backward workspace (0 = no device-side problem)."""
        B = getattr(self, "_bwd", None)
        return 0 if B is None else L.moe_read_device_status(B["ws"], None, clear)

    def device_status(self, clear: bool = False) -> int:
        return L.moe_read_device_status(self.ws, None, clear)
