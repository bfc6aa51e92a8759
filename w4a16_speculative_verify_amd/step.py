"""One speculative-decoding verify step on the GPU (orchestration only).

The organisers' results page (section 3) describes the step: the target runs
one forward pass over the block of K+1 positions per sequence, its 8-bit
lm_head yields the greedy token of every row, and greedy acceptance keeps the
longest matching draft prefix plus the bonus token.  Here the target is a
chain of W4A16 linears (each reads the leading ``k_in`` columns of the
previous output; no activation function is modelled), with attention over a
paged cache between a layer's first two linears where a PagedMixer is given,
followed by the fused lm_head + argmax + verify launch.  Every launch goes to the
current stream through the C ABI; the object owns the activation buffers and
one workspace shared by the stream-ordered calls, so a step allocates
nothing and can be captured in a HIP graph.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (Chain, f16_gemm, f16_gemm_workspace_size, f16_lmhead_argmax_verify,
               gemm_workspace_size, lmhead_workspace_size, new_workspace, paged_attention,
               paged_attention_workspace_size, rope_inv_freq, rope_kv_append, w4a16_gemm,
               w8a16_lmhead_argmax_verify)


@dataclass
class DeviceLinear:
    qweight: torch.Tensor | None   # int32 [k/8, n]
    scales: torch.Tensor | None    # fp16 [k/g, n]
    qzeros: torch.Tensor | None    # int32 [k/g, n/8]
    k_in: int
    n_out: int
    alpha: float
    group_size: int = 128
    w16: torch.Tensor | None = None   # fp16 [n, k]: a half-precision linear instead


class PagedMixer:
    """Attention between the QKV and O linears of ``layers`` layers: rotary positions, the append
    of the block's keys and values to each layer's paged cache, and attention over it.

    All layers share the page table.  ``ctx_lens`` (int32 [batch], on the device) counts each
    sequence's tokens with the verify block's rows: set it, and ``block_table``, before a step;
    ``advance`` moves it on by what the step accepted, so that the next block overwrites the
    rejected drafts' places.  ``max_ctx`` is the most tokens a sequence will have.
    """

    def __init__(self, layers: int, batch: int, rows: int, hq: int, hkv: int, d: int, num_pages: int,
                 page_size: int, max_ctx: int, rope=None, interleaved: bool = False, device="cuda"):
        dev = torch.device(device)
        self.layers, self.batch, self.rows = layers, batch, rows
        self.hq, self.hkv, self.d, self.max_ctx, self.interleaved = hq, hkv, d, max_ctx, interleaved
        self.inv_freq, self.mscale = rope_inv_freq(d, device=dev) if rope is None else rope
        shape = (num_pages, hkv, page_size, d)
        self.k_cache = [torch.zeros(shape, dtype=torch.float16, device=dev) for _ in range(layers)]
        self.v_cache = [torch.zeros(shape, dtype=torch.float16, device=dev) for _ in range(layers)]
        self.block_table = torch.full((batch, -(-max_ctx // page_size)), -1, dtype=torch.int32,
                                      device=dev)
        self.ctx_lens = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.cu = torch.arange(0, (batch + 1) * rows, rows, dtype=torch.int32, device=dev)
        self.q = torch.empty((batch * rows, hq, d), dtype=torch.float16, device=dev)
        self.out = torch.empty((batch * rows, hq, d), dtype=torch.float16, device=dev)

    def workspace_size(self) -> int:
        return paged_attention_workspace_size(self.batch, self.rows, self.max_ctx, self.hq, self.hkv,
                                              self.d)

    def __call__(self, layer: int, qkv: torch.Tensor, workspace=None) -> torch.Tensor:
        """fp16 [batch * rows, hq * d] of layer ``layer`` from its QKV linear's output."""
        k, v = self.k_cache[layer], self.v_cache[layer]
        rope_kv_append(qkv, k, v, self.block_table, self.cu, self.ctx_lens, self.inv_freq, self.hq,
                       interleaved=self.interleaved, mscale=self.mscale, q_out=self.q)
        paged_attention(self.q, k, v, self.block_table, self.cu, self.ctx_lens, self.rows,
                        max_ctx=self.max_ctx, out=self.out, workspace=workspace)
        return self.out.view(self.batch * self.rows, self.hq * self.d)

    def advance(self, accepted_len: torch.Tensor):
        """The next block starts behind the accepted drafts and the target's own token."""
        self.ctx_lens.add_(accepted_len).add_(1)


class VerifyStep:
    def __init__(self, linears, lm_w, lm_s, m: int, batch: int, k_draft: int,
                 device="cuda", chain: bool | None = None, mixer: PagedMixer | None = None):
        if m != batch * (k_draft + 1):
            raise ValueError("rows must be batch * (k_draft + 1)")
        self.linears = list(linears)
        self.mixer = mixer
        if mixer is not None:
            if chain:
                raise ValueError("the one-launch chain has no attention between its linears")
            if mixer.batch != batch or mixer.rows != k_draft + 1:
                raise ValueError("the mixer's batch and rows must be the step's")
            self.per_layer = len(self.linears) // mixer.layers
            if self.per_layer < 2 or self.per_layer * mixer.layers != len(self.linears):
                raise ValueError("every layer needs the same linears, QKV and O first")
            for i in range(0, len(self.linears), self.per_layer):
                if self.linears[i].n_out < (mixer.hq + 2 * mixer.hkv) * mixer.d or \
                        self.linears[i + 1].k_in > mixer.hq * mixer.d:
                    raise ValueError(f"linears {i} and {i + 1} do not fit the mixer's heads")
        self.lm_w, self.lm_s = lm_w, lm_s
        self.m, self.batch, self.k = m, batch, k_draft
        dev = torch.device(device)
        # one output buffer per distinct (position-in-layer) width, reused across layers
        self.out = []
        cache = {}
        for i, lin in enumerate(self.linears):
            key = (i % 4, lin.n_out) if len(self.linears) % 4 == 0 else (i, lin.n_out)
            if key not in cache:
                cache[key] = torch.empty((m, lin.n_out), dtype=torch.float16, device=dev)
            self.out.append(cache[key])
        for i in range(1, len(self.out)):
            if self.out[i].data_ptr() == self.out[i - 1].data_ptr():
                raise ValueError("consecutive linears would share a buffer")
        need = max([f16_gemm_workspace_size(m, l.n_out, l.k_in) if l.w16 is not None
                    else gemm_workspace_size(m, l.n_out, l.k_in, l.group_size)
                    for l in self.linears] + [0])
        if lm_w is not None:
            need = max(need, lmhead_workspace_size(m, lm_w.shape[1], lm_w.shape[0]))
        if mixer is not None:
            need = max(need, mixer.workspace_size())
        self.workspace = new_workspace(need, dev)
        # one launch for the whole chain when the block fits the chain kernel
        self.chain = None
        if chain is None:
            chain = False
        if chain:
            self.chain = Chain([(l.qweight, l.scales, l.qzeros, l.alpha) for l in self.linears],
                               m, dev)
        self.target_ids = torch.empty(m, dtype=torch.int32, device=dev)
        self.max_logits = torch.empty(m, dtype=torch.float32, device=dev)
        self.accepted_len = torch.empty(batch, dtype=torch.int32, device=dev)
        self.out_tokens = torch.empty((batch, k_draft + 1), dtype=torch.int32, device=dev)

    def linears_only(self, x: torch.Tensor) -> torch.Tensor:
        """Run the chain of linears on x (fp16 [m, >= k_in of the first]), with the mixer behind each
        layer's first where there is one; returns the last output."""
        if self.chain is not None:
            return self.chain(x, out=self.out[-1])
        h = x
        for i, (lin, y) in enumerate(zip(self.linears, self.out)):
            if lin.w16 is not None:
                f16_gemm(h[:, :lin.k_in], lin.w16, alpha=lin.alpha, out=y, workspace=self.workspace)
            else:
                w4a16_gemm(h[:, :lin.k_in], lin.qweight, lin.scales, lin.qzeros, alpha=lin.alpha,
                           out=y, workspace=self.workspace, group_size=lin.group_size)
            h = y
            if self.mixer is not None and i % self.per_layer == 0:
                h = self.mixer(i // self.per_layer, y, self.workspace)
        return h

    def head(self, h: torch.Tensor, drafts: torch.Tensor, accepted_len=None, out_tokens=None):
        """Fused lm_head + argmax + greedy verify on the final hidden rows (an fp16 lm_head
        when no scales are given).  accepted_len / out_tokens: caller buffers for the
        verify's outputs (int32 [batch] / [batch, K+1]); the step's own by default."""
        acc = self.accepted_len if accepted_len is None else accepted_len
        out = self.out_tokens if out_tokens is None else out_tokens
        if self.lm_s is None:
            return f16_lmhead_argmax_verify(h, self.lm_w, drafts, target_ids=self.target_ids,
                                            max_logits=self.max_logits, accepted_len=acc,
                                            out_tokens=out, workspace=self.workspace)
        return w8a16_lmhead_argmax_verify(h, self.lm_w, self.lm_s, drafts,
                                          target_ids=self.target_ids, max_logits=self.max_logits,
                                          accepted_len=acc, out_tokens=out,
                                          workspace=self.workspace)

    def __call__(self, x: torch.Tensor, drafts: torch.Tensor, accepted_len=None, out_tokens=None):
        return self.head(self.linears_only(x), drafts, accepted_len, out_tokens)
