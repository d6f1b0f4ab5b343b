"""Whole layers - a KDA layer and a gated delta rule layer - on the library's kernels only.

Per token of each sequence (kimi_k3.c header comment, block "KDA per-head
recurrence"; struct Kda: W q, k, v, o, g, fa, fb, bp):

    q, k, v, g = W_q x, W_k x, W_v x, W_g x      one kda_linear over the stacked weights
    z, b       = W_fb (W_fa x), W_b x            kda_gate_proj
    o          = mixer(q, k, v, z, b, g)          kda_decode_token / kda_prefill (ShortConv4,
                                                  SiLU, L2, gates, delta rule, readout,
                                                  sigmoid(g) * RMSNorm_head)
    x'         = x + W_o o                        kda_linear with the residual

The residual add stands in for the model's residual stream (the pages' attention
residuals and the MoE/MLP blocks between KDA layers are other components). This module
only sequences library calls and owns their buffers; every product and every step of the
mixer runs in libkda's kernels.

The gated delta rule layer has the same frame around the recurrence with one decay per head:

    q, k, v, a, b = columns of W_in x              one product; its columns go on as they lie
    o             = kda_gdr_decode / kda_gdr_prefill
    x'            = x + W_o o

It is the recurrence between two products and no published model's layer: there is no short convolution, no
SiLU, no output norm and no gate around the recurrence. A model that has them applies them to the columns
and to o itself, between the library's calls.

The dense products of either layer run in BF16 (kda_linear) or, for weights given as
Fp8Weight, in FP8 (kda_quant_fp8 of the activations, kda_linear_fp8).
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import kda as K


@dataclass
class Fp8Weight:
    """A weight matrix [N, K] in E4M3 with one FP32 scale per 128 x 128 block."""
    q: torch.Tensor   # [N, K] float8_e4m3fn
    s: torch.Tensor   # [ceil(N / 128), ceil(K / 128)]

    @property
    def shape(self):
        return self.q.shape


def fp8_weight(w: torch.Tensor, stream=None) -> Fp8Weight:
    """w [N, K] (BF16 or FP32) quantised by kda_quant_fp8."""
    N, Kw = w.shape
    q = torch.empty(N, Kw, dtype=torch.float8_e4m3fn, device=w.device)
    s = torch.empty(-(-N // 128), -(-Kw // 128), dtype=torch.float32, device=w.device)
    K.kda_quant_fp8(w, q, s, block_rows=128, stream=stream)
    return Fp8Weight(q, s)


class Products:
    """The buffers of y = x W^T (+ r) for up to `rows` rows of x and the (N, K) of `shapes`."""

    def __init__(self, shapes, rows: int, device, fp8: bool):
        self.fp8 = fp8
        # the k split (and so the workspace) depends on the number of rows, up and down: the largest need of all of them
        query = K.kda_linear_fp8_workspace_bytes if fp8 else K.kda_linear_workspace_bytes
        ws = max(query(m, N, Kw) for N, Kw in shapes for m in range(1, rows + 1)) if rows else 256
        if fp8:
            Kmax = max(Kw for _, Kw in shapes)
            self.xq = torch.empty(rows * Kmax, dtype=torch.float8_e4m3fn, device=device)
            self.xs = torch.empty(rows * -(-Kmax // 128), dtype=torch.float32, device=device)
            self.ws = torch.zeros(ws, dtype=torch.uint8, device=device)  # the error word starts at 0
        else:
            self.ws = torch.empty(ws, dtype=torch.uint8, device=device)

    def __call__(self, x: torch.Tensor, w, y: torch.Tensor, r=None, ysplit: int = 0, stream=None) -> None:
        if isinstance(w, Fp8Weight) != self.fp8:
            raise TypeError("an FP8 runner takes Fp8Weight products, a BF16 runner BF16 tensors")
        if not self.fp8:
            K.kda_linear(x, w, y, self.ws, r=r, ysplit=ysplit, stream=stream)
            return
        n, Kx = x.shape
        xq, xs = self.xq[:n * Kx].view(n, Kx), self.xs[:n * -(-Kx // 128)].view(n, -(-Kx // 128))
        K.kda_quant_fp8(x, xq, xs, stream=stream)
        K.kda_linear_fp8(xq, xs, w.q, w.s, y, self.ws, r=r, ysplit=ysplit, stream=stream)


@dataclass
class KdaLayerWeights:
    """Device weights of one KDA layer (BF16 products, FP32 mixer parameters); w_qkvg and w_o may
    be Fp8Weight."""
    w_qkvg: torch.Tensor   # [4 H d, hidden]: rows of W_q, W_k, W_v, W_g in that order
    w_fa: torch.Tensor     # [d, hidden]
    w_fb: torch.Tensor     # [H d, d]
    w_b: torch.Tensor      # [H, hidden]
    w_o: torch.Tensor      # [hidden, H d]
    params: K.kda_layer_params  # conv_w, dt_bias, A_log, norm_w (FP32)


def random_layer_weights(H: int, d: int, hidden: int, gen: torch.Generator, device) -> KdaLayerWeights:
    """Synthetic weights: each projection ~ N(0, 1/fan_in) (so outputs come out ~ N(0, 1) for
    an input of unit variance), mixer parameters from the workload's distributions."""
    import math
    bf = torch.bfloat16
    D = H * d

    def mat(n, k):
        return (torch.randn(n, k, generator=gen, device=device) * k ** -0.5).to(bf).contiguous()

    conv_w = (torch.randn(3, D, 4, generator=gen, device=device) * 0.5).contiguous()
    dt_bias = torch.randn(D, generator=gen, device=device) * math.sqrt(0.5)
    A_log = torch.rand(H, generator=gen, device=device) * math.log(16.0)
    norm_w = 1.0 + torch.randn(d, generator=gen, device=device) * math.sqrt(0.1)
    return KdaLayerWeights(mat(4 * D, hidden), mat(d, hidden), mat(D, d), mat(H, hidden), mat(hidden, D),
                           K.kda_layer_params_from(conv_w, dt_bias, A_log, norm_w))


class KdaLayerRunner:
    """Buffers for running KDA layers on a batch of up to `rows` tokens at a time; fp8: with the
    stacked projection and W_o in FP8."""

    def __init__(self, cfg: K.kda_config_t, hidden: int, rows: int, device, fp8: bool = False):
        self.cfg = cfg
        self.hidden = hidden
        H, d = cfg.num_heads, cfg.head_dim
        D = H * d
        bf = torch.bfloat16
        self.rows = rows
        self.qkvg = torch.empty(4, rows, D, dtype=bf, device=device)
        self.z = torch.empty(rows, D, dtype=bf, device=device)
        self.b = torch.empty(rows, H, dtype=bf, device=device)
        self.o = torch.empty(rows, D, dtype=bf, device=device)
        self.products = Products([(4 * D, hidden), (hidden, D)], rows, device, fp8)
        self.ws_lin = self.products.ws
        self.ws_gp = torch.empty(K.kda_gate_proj_workspace_bytes(cfg, hidden, rows), dtype=torch.uint8, device=device)

    def _inputs(self, lw: KdaLayerWeights, x: torch.Tensor, stream):
        n = x.shape[0]
        D = self.o.shape[1]
        qkvg = self.qkvg.view(-1)[:4 * n * D].view(4, n, D)  # four contiguous [n, D] matrices
        self.products(x, lw.w_qkvg, qkvg, ysplit=self.o.shape[1], stream=stream)
        z, b = self.z[:n], self.b[:n]
        K.kda_gate_proj(self.cfg, x, lw.w_fa, lw.w_fb, lw.w_b, z, b, self.ws_gp, stream)
        return qkvg, z, b

    def decode(self, lw: KdaLayerWeights, st, slots: torch.Tensor, x: torch.Tensor, x_out: torch.Tensor,
               stream=None) -> None:
        """One decode token for each of the x.shape[0] rows (row r on slot slots[r]): x_out = x + W_o o."""
        n = x.shape[0]
        qkvg, z, b = self._inputs(lw, x, stream)
        o = self.o[:n]
        K.kda_decode_token(self.cfg, lw.params, st, slots, qkvg[0], qkvg[1], qkvg[2], z, b, qkvg[3], o, stream)
        self.products(o, lw.w_o, x_out, r=x, stream=stream)

    def prefill(self, lw: KdaLayerWeights, st, slots: torch.Tensor, cu_seqlens: torch.Tensor, cu_seqlens_host,
                x: torch.Tensor, x_out: torch.Tensor, stream=None) -> None:
        """Packed variable-length prefill of x.shape[0] tokens: x_out = x + W_o o."""
        n = x.shape[0]
        qkvg, z, b = self._inputs(lw, x, stream)
        o = self.o[:n]
        K.kda_prefill(self.cfg, lw.params, st, slots, cu_seqlens, cu_seqlens_host, qkvg[0], qkvg[1], qkvg[2], z, b,
                      qkvg[3], o, stream)
        self.products(o, lw.w_o, x_out, r=x, stream=stream)


@dataclass
class GdrLayerWeights:
    """Device weights of one gated delta rule layer; w_in and w_o BF16 or Fp8Weight."""
    w_in: torch.Tensor     # [gdr_width(cfg), hidden]: rows of W_q, W_k [Hk d], W_v [H d], W_a, W_b [H], then padding
    w_o: torch.Tensor      # [hidden, H d]
    params: K.kda_gdr_params  # A_log, dt_bias (FP32)


def gdr_width(cfg: K.kda_gdr_config_t) -> int:
    """Rows of w_in: q, k, v, a and b side by side, up to a multiple of 128 (what the BF16 product takes)."""
    n = (2 * cfg.num_qk_heads + cfg.num_heads) * cfg.head_dim + 2 * cfg.num_heads
    return -(-n // 128) * 128


def _capturing(stream) -> bool:
    """Whether the stream a call is given (a torch stream or its handle; None: the current one) is being captured."""
    if stream is None:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))):
        return torch.cuda.is_current_stream_capturing()


class GdrLayerRunner:
    """Buffers for running gated delta rule layers on a batch of up to `rows` tokens at a time, made on
    the current stream."""

    def __init__(self, cfg: K.kda_gdr_config_t, hidden: int, rows: int, device, fp8: bool = False):
        if cfg.io_dtype != K.KDA_BF16:
            raise ValueError("the layer's products are BF16")
        self.cfg, self.hidden, self.rows = cfg, hidden, rows
        D, W = cfg.num_heads * cfg.head_dim, gdr_width(cfg)
        self.proj = torch.empty(rows, W, dtype=torch.bfloat16, device=device)
        self.o = torch.empty(rows, D, dtype=torch.bfloat16, device=device)
        self.products = Products([(W, hidden), (hidden, D)], rows, device, fp8)
        self.ws = torch.empty(0, dtype=torch.uint8, device=device)
        self._captured = []  # workspaces that a captured prefill writes to

    def _inputs(self, lw: GdrLayerWeights, x: torch.Tensor, stream):
        n = x.shape[0]
        if n > self.rows:
            raise ValueError(f"{n} rows, the runner was made for {self.rows}")
        proj = self.proj[:n]
        self.products(x, lw.w_in, proj, stream=stream)
        H, Hk, d = self.cfg.num_heads, self.cfg.num_qk_heads, self.cfg.head_dim
        return (*torch.split(proj[:, :(2 * Hk + H) * d + 2 * H], [Hk * d, Hk * d, H * d, H, H], dim=1), self.o[:n])

    def decode(self, lw: GdrLayerWeights, S: torch.Tensor, src_slots: torch.Tensor, dst_slots: torch.Tensor, n: int,
               x: torch.Tensor, x_out: torch.Tensor, err=None, stream=None) -> None:
        """n tokens for each of src_slots.numel() sequences, rows r n + t of x: x_out = x + W_o o."""
        rows = self._inputs(lw, x, stream)
        K.kda_gdr_decode(self.cfg, lw.params, S, src_slots, dst_slots, n, *rows, err=err, stream=stream)
        self.products(rows[-1], lw.w_o, x_out, r=x, stream=stream)

    def prefill(self, lw: GdrLayerWeights, S: torch.Tensor, src_slots: torch.Tensor, dst_slots: torch.Tensor,
                cu_seqlens: torch.Tensor, cu_seqlens_host, x: torch.Tensor, x_out: torch.Tensor, err=None, stream=None) -> None:
        """Packed variable-length prefill of x.shape[0] tokens: x_out = x + W_o o. When a batch needs more
        chunks than any before, the workspace grows, which waits for the device; not while a graph is
        captured (run a prefill of that size first)."""
        need = K.kda_gdr_workspace_bytes(self.cfg, cu_seqlens_host)
        capturing = _capturing(stream)
        if self.ws.numel() < need:
            if capturing or torch.cuda.is_current_stream_capturing():  # neither capture would survive the waits below
                raise RuntimeError(f"the workspace must grow to {need} bytes: run a prefill of this size before one is captured")
            torch.cuda.synchronize(self.proj.device)  # calls on other streams may be using the old one
            self.ws = torch.empty(need, dtype=torch.uint8, device=self.proj.device)
            torch.cuda.synchronize(self.proj.device)  # and the new one's memory may have had another use
        if capturing and not any(w is self.ws for w in self._captured):
            self._captured.append(self.ws)  # a graph keeps writing to it
        rows = self._inputs(lw, x, stream)
        K.kda_gdr_prefill(self.cfg, lw.params, S, src_slots, dst_slots, cu_seqlens, cu_seqlens_host, *rows, self.ws,
                          err=err, stream=stream)
        self.products(rows[-1], lw.w_o, x_out, r=x, stream=stream)
