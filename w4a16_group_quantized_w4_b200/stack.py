"""A stack of mixture-of-experts layers held on one device.

The whole-model form of the hot path: every layer's gate/up and down weights arrive as bf16 (the
"unquantized" QAT export of "Repacked QAT Gemma 4 26B-A4B serves on one TPU v6e at 1.9x FP8
throughput", section "A repack, not a re-quantization"), are repacked on the device by
`w4_repack` into int4 codes and bf16 scales, and decode steps then run the four entry points layer
after layer ("The gap at 26B": 128 experts per layer, 8 active).  The pages give no blocks
between the MoE layers; a chained step feeds each layer the previous layer's output divided by
its root mean square (moe_rms_chain, no learned weight), with seeded router logits per layer.  A decode
step with attention (decode_step) puts an AttentionBlock in front of every expert layer, the usual
pre-norm residual block over a paged key/value cache.

Layouts (layer-major, so layer l's weights are contiguous slices):
  gate/up codes [L, E, 2I, H/8] int32, scales [L, E, 2I, H/32] bf16
  down    codes [L, E, H, I/8]  int32, scales [L, E, H, I/32]  bf16
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import api


@dataclass
class RepackReport:
    off_grid_gate_up: int
    off_grid_down: int
    group_m_gate_up: torch.Tensor     # uint8 [L*E*2I, H/32]
    group_m_down: torch.Tensor        # uint8 [L*E*H, I/32]


def _placed(x, stream):
    """Context in which calls without a stream run on `stream`, or on the current stream of x's device."""
    return torch.cuda.device(x.device) if stream is None else torch.cuda.stream(stream)


class AttentionBlock:
    """The attention half of a decoder layer on 4-bit weights, for one new token per sequence:

      h <- h + x;  n = norm(h) in 8-bit rows;  q, k, v = n Wqkv^T;  k, v into the cache;
      a = attention of q over the cache;  o = a Wo^T;  h <- h + o;  returns norm(h) for the expert layer.

    qkv_codes [(q_heads + 2 kv_heads) D, H/8] with scales [.., H/32], o_codes [H, q_heads D / 8] with
    scales [.., q_heads D / 32] (layout L1); norms: two bf16 [H] weights or None, with one eps.  Queries and
    keys are taken as the projection gives them; scale: what their products are multiplied by, 1 / sqrt(D) when
    None.  D, the cache's head_dim: one that attention takes (64, 128, 192 or 256)."""

    def __init__(self, qkv_codes, qkv_scales, o_codes, o_scales, cache: api.KVCache, q_heads: int,
                 norm_in=None, norm_out=None, softcap: float = 0.0, window: int = 0, scale: float | None = None,
                 eps: float = api.RMS_EPS):
        _, kv_heads, _, last = cache.k.shape
        self.dim = last * (8 if cache.kind == "int4" else 1)
        if self.dim not in (64, 128, 192, 256):
            raise ValueError(f"cache: attention takes a head_dim of 64, 128, 192 or 256, got {self.dim}")
        self.q_heads, self.kv_heads = q_heads, kv_heads
        if qkv_codes.shape[0] != (q_heads + 2 * kv_heads) * self.dim:
            raise ValueError("qkv_codes: rows must be (q_heads + 2 kv_heads) * head_dim")
        if o_codes.shape[1] * 8 != q_heads * self.dim:
            raise ValueError("o_codes: columns must be q_heads * head_dim / 8")
        self.qkv, self.o = (qkv_codes, qkv_scales), (o_codes, o_scales)
        self.cache, self.norm_in, self.norm_out = cache, norm_in, norm_out
        self.softcap, self.window, self.scale, self.eps = softcap, window, scale, eps

    def __call__(self, x, h, page_table, seq_lens, slots, stream=None, dev_status=None):
        """x bf16 [T, H] (the previous layer's output), h bf16 [T, H] the residual stream or None for
        the first layer; page_table, seq_lens as in kv_cache_attend (the new token counted), slots
        int64 [T] of the new rows -> (the expert layer's input, h).  dev_status: int32 [1] that the 8-bit linear, the
        write and the attention report to (a slot past the cache, a length or page out of range)."""
        with _placed(x, stream):
            T = x.shape[0]
            n, ns, h = api.w4_rms_add_q8(x, h, self.norm_in, eps=self.eps)
            rows = api.w4a8_linear(n, ns, *self.qkv, dev_status=dev_status).unflatten(1, (-1, self.dim))
            q, k, v = rows.split((self.q_heads, self.kv_heads, self.kv_heads), dim=1)
            self.cache.write(k, v, slots, dev_status=dev_status)
            a = self.cache.attend(q, page_table, seq_lens, scale=self.scale, softcap=self.softcap, window=self.window,
                                  dev_status=dev_status)
            o = api.w4a16_linear(a.view(T, -1), *self.o, ws=api.linear_scratch(T, *self.o[0].shape, x.device))
            return api.w4_rms_add(o, h, self.norm_out, eps=self.eps)


class MoEStack:
    """L layers of E experts (hidden H, expert intermediate I, top-k routing) on one device."""

    def __init__(self, L: int, E: int = 128, k: int = 8, H: int = 2816, I: int = 704, device="cuda"):
        self.L, self.E, self.k, self.H, self.I = L, E, k, H, I
        dev = torch.device(device)
        self.gu_codes = torch.empty((L, E, 2 * I, H // 8), dtype=torch.int32, device=dev)
        self.gu_scales = torch.empty((L, E, 2 * I, H // 32), dtype=torch.bfloat16, device=dev)
        self.dn_codes = torch.empty((L, E, H, I // 8), dtype=torch.int32, device=dev)
        self.dn_scales = torch.empty((L, E, H, I // 32), dtype=torch.bfloat16, device=dev)
        self._layers = {}

    # ------------------------------------------------------------------ repack
    def gate_up_rows(self) -> int:
        return self.L * self.E * 2 * self.I

    def down_rows(self) -> int:
        return self.L * self.E * self.H

    def repack(self, w_gate_up: torch.Tensor, w_down: torch.Tensor, stream=None) -> RepackReport:
        """w_gate_up bf16 [L*E*2I, H], w_down bf16 [L*E*H, I] (layer-major) -> this stack's codes
        and scales, through two w4_repack calls."""
        dev = self.gu_codes.device
        g_gu = torch.empty((self.gate_up_rows(), self.H // 32), dtype=torch.uint8, device=dev)
        g_dn = torch.empty((self.down_rows(), self.I // 32), dtype=torch.uint8, device=dev)
        off = torch.zeros(2, dtype=torch.int64, device=dev)
        api.w4_repack(w_gate_up, codes=self.gu_codes.view(-1, self.H // 8),
                      scales=self.gu_scales.view(-1, self.H // 32), group_m=g_gu,
                      off_grid_count=off[0:1], stream=stream)
        api.w4_repack(w_down, codes=self.dn_codes.view(-1, self.I // 8),
                      scales=self.dn_scales.view(-1, self.I // 32), group_m=g_dn,
                      off_grid_count=off[1:2], stream=stream)
        o = off.cpu()
        return RepackReport(int(o[0]), int(o[1]), g_gu, g_dn)

    # ------------------------------------------------------------------ decode
    def fusable(self, T: int) -> bool:
        """Whether T tokens fit the single-launch fused layer (moe_w4a16_layer)."""
        return api.moe_layer_fusable(T, self.E, self.k, self.H, self.I)

    def layer(self, l: int, T: int, fused: bool = False) -> api.MoELayer:
        """MoE layer l for T tokens (buffers allocated once per (l, T, fused)): the four-call
        path, or the single-launch fused layer when fused and T fits it."""
        fused = fused and self.fusable(T)
        key = (l, T, fused)
        if key not in self._layers:
            self._layers[key] = api.MoELayer(self.gu_codes[l], self.gu_scales[l], self.dn_codes[l],
                                             self.dn_scales[l], T, self.k, fused=fused)
        return self._layers[key]

    def step(self, xs, logits, stream=None, fused: bool = False):
        """One decode step through every layer with independent inputs: xs[l] bf16 [T, H],
        logits[l] f32 [T, E] -> the list of layer outputs y_l bf16 [T, H] (each layer's own
        buffer)."""
        T = xs[0].shape[0]
        return [self.layer(l, T, fused)(xs[l], logits[l], stream=stream) for l in range(self.L)]

    def chained_step(self, x0, logits, stream=None, fused: bool = False):
        """One decode step through the chained stack: layer 0 takes x0 bf16 [T, H]; layer l + 1
        takes moe_rms_chain(y_l).  Returns (the inputs x_l, the outputs y_l), device buffers
        owned by the stack (overwritten by the next chained step of the same T and path)."""
        T = x0.shape[0]
        key = ("chain", T, fused)
        if key not in self._layers:
            self._layers[key] = [torch.empty((T, self.H), dtype=torch.bfloat16, device=x0.device)
                                 for _ in range(self.L - 1)]
        xb = self._layers[key]
        xs, ys = [x0], []
        for l in range(self.L):
            y = self.layer(l, T, fused)(xs[l], logits[l], stream=stream)
            ys.append(y)
            if l + 1 < self.L:
                xs.append(api.moe_rms_chain(y, x_next=xb[l], stream=stream))
        return xs, ys

    def decode_step(self, x0, logits, blocks, page_table, seq_lens, slots, norm=None, stream=None,
                    fused: bool = False, dev_status=None, eps: float = api.RMS_EPS):
        """One decode step through attention and experts: layer l runs blocks[l] (AttentionBlock, each
        with its own cache; they share page_table, seq_lens and slots) and expert layer l on
        logits[l] f32 [T, E], around the residual stream that x0 bf16 [T, H] begins.  Returns
        (norm of the final residual stream with weight `norm` and eps, the stream), both bf16 [T, H].  Rows whose
        slot is negative and whose length is 0 are padding.  dev_status: int32 [1] that the blocks report to.  The expert layers share scratch and keep their
        buffers (allocated by the first step of a T and path: run one before capturing one): two steps must
        not overlap on the GPU, nor two captured ones be replayed at once."""
        if len(blocks) != self.L:
            raise ValueError(f"blocks: expected {self.L}, got {len(blocks)}")
        T = x0.shape[0]
        with _placed(x0, stream):
            y, h = x0, None
            for l, block in enumerate(blocks):
                x, h = block(y, h, page_table, seq_lens, slots, dev_status=dev_status)
                y = self.layer(l, T, fused)(x, logits[l])
            return api.w4_rms_add(y, h, norm, eps=eps)

    def expert_bytes(self) -> int:
        """Packed bytes of one expert (gate/up + down codes and scales)."""
        return (2 * self.I * self.H // 2 + 2 * self.I * self.H // 16 +
                self.H * self.I // 2 + self.H * self.I // 16)
