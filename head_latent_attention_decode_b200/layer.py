"""Device-memory plumbing around the C-ABI: upload a weight set, own the
repacked blob and a workspace, and call the entry points on torch tensors.

No arithmetic of the layer happens here; each method is one C-ABI call.
"""
from __future__ import annotations

import numpy as np
import torch

from . import (MLA_FP8_E4M3_ROW, MLA_ROW_LATENT_FIRST, make_config, mla_cache_block_bytes, mla_cache_read,
               mla_cache_write, mla_decode_attn, mla_decode_attn_prefix, mla_decode_qkv, mla_destroy,
               mla_init_weights, mla_latent_attn, mla_prefill, mla_prefix_workspace_bytes, mla_rope_cos_sin,
               mla_rope_cos_sin_inv_freq, mla_set_cache_dtype, mla_v4_qkv, mla_weights_bytes,
               mla_workspace_bytes, mla_workspace_init)

ACT_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def upload_weights(weights, device) -> dict:
    """workloads.Weights -> dict of device tensors in the C-ABI's storage dtypes."""
    s = weights.shape
    out = {}
    for name, arr in weights.dense.items():
        t = torch.from_numpy(np.ascontiguousarray(arr))
        out[name] = t.to(ACT_TORCH[s.weight_dtype]).to(device)
    for name, codes in weights.codes.items():
        out[name] = torch.from_numpy(np.ascontiguousarray(codes)).to(device)
        out[name + "_scale"] = torch.from_numpy(np.ascontiguousarray(weights.scales[name])).to(device)
    if weights.q_norm_w is not None:
        out["q_norm_w"] = torch.from_numpy(weights.q_norm_w).to(device)
    out["kv_norm_w"] = torch.from_numpy(weights.kv_norm_w).to(device)
    return out


class MlaLayer:
    """One layer's repacked weights (device) and C-ABI handle.

    The calls of a layer share one workspace, `ws`, made and enlarged as they need it. Calls on different
    streams are therefore put in order, each behind the calls before it. A captured graph keeps the workspace it
    was captured with; replays of graphs, and calls beside them, must not overlap on the GPU. `ws` holds the
    device flag of the calls made on it: a graph captured before any call has a workspace of its own."""

    def __init__(self, shape, weights, row_layout: int = MLA_ROW_LATENT_FIRST,
                 device: str = "cuda", softmax_scale: float = 0.0, attn_sink=None, cache_dtype: str | None = None):
        """cache_dtype: None for a cache in the activation dtype, "fp8" for the 8-bit cache."""
        if cache_dtype not in (None, "fp8"):
            raise ValueError(f"cache_dtype must be None or 'fp8', not {cache_dtype!r}")
        self.cache_dtype = cache_dtype
        self.shape = shape
        self.device = torch.device(device)
        self.act = ACT_TORCH[shape.act_dtype]
        self.row_layout = row_layout
        self.cfg = make_config(shape, row_layout, softmax_scale)
        nbytes = mla_weights_bytes(self.cfg)
        if nbytes == 0:
            raise ValueError(f"configuration not accepted by the library: {shape}")
        self.blob = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        src = upload_weights(weights, self.device) if not isinstance(weights, dict) else dict(weights)
        if attn_sink is not None:   # per-head sink logits, fp32 [n_heads]
            src["attn_sink"] = torch.as_tensor(attn_sink, dtype=torch.float32).to(self.device).contiguous()
        self.handle = mla_init_weights(self.cfg, src, self.blob)
        torch.cuda.current_stream(self.device).synchronize()
        del src
        if cache_dtype == "fp8":
            mla_set_cache_dtype(self.handle, MLA_FP8_E4M3_ROW)
        self.block_bytes = mla_cache_block_bytes(self.handle)
        self._cache_torch = torch.uint8 if cache_dtype == "fp8" else self.act
        self.ws = None
        self._graph_ws = []         # workspaces that captured graphs hold
        self._ws_for = (None, 0)    # the sizes that prefix_workspace was last asked for, and their bytes
        self._device_index = self.blob.get_device()
        self._ws_stream = self._ws_raw = None   # the stream of the last call, and its raw handle

    def close(self) -> None:
        """Release the library handle (the weight blob is torch memory)."""
        h = getattr(self, "handle", None)
        if h:
            mla_destroy(h)
            self.handle = None

    def __del__(self):
        # at interpreter shutdown the module's globals may already be gone
        if mla_destroy is not None:
            self.close()

    def _new_ws(self, need: int, head: int | None = None) -> torch.Tensor:
        ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        mla_workspace_init(ws[:head])
        return ws

    def _workspace(self, need: int) -> torch.Tensor:
        """A workspace of `need` bytes or more for a call on the current stream."""
        if torch._C._cuda_isCurrentStreamCapturing():
            # kept alive with the layer (a later call may need a larger one); one made here is the graph's own
            for ws in (self.ws, *self._graph_ws):
                if ws is not None and ws.numel() >= need:
                    break
            else:
                ws = self._new_ws(need, 256)   # at each replay: the device flag and the counters alone
            if all(w is not ws for w in self._graph_ws):
                self._graph_ws.append(ws)
            return ws
        if torch._C._cuda_getCurrentRawStream(self._device_index) != self._ws_raw:
            self._change_stream()
        if self.ws is None or self.ws.numel() < need:
            old, self.ws = self.ws, self._new_ws(need)
            if old is not None:
                self.ws[:4].copy_(old[:4])            # the device flag is sticky
                old.record_stream(self._ws_stream)    # the last calls on it may still run
        return self.ws

    def _change_stream(self):
        """The current stream waits for the calls made on the one before it."""
        stream, before = torch.cuda.current_stream(self.device), self._ws_stream
        if before is not None:
            with torch.cuda.stream(before):
                capturing = torch.cuda.is_current_stream_capturing()   # its earlier work was waited for then
            if not capturing:
                stream.wait_stream(before)
        self._ws_stream, self._ws_raw = stream, stream.cuda_stream

    def workspace(self, max_tokens: int, max_context_len: int = 1) -> torch.Tensor:
        return self._workspace(mla_workspace_bytes(self.handle, max(1, max_tokens), max(1, max_context_len)))

    def prefix_workspace(self, max_tokens: int, max_prefix_len: int, max_context_len: int) -> torch.Tensor:
        """A workspace for latent_attn and decode_attn_prefix (and every other call)."""
        sizes = (max_tokens, max_prefix_len, max_context_len)
        if sizes != self._ws_for[0]:
            need = mla_prefix_workspace_bytes(self.handle, max(1, max_tokens), max(0, max_prefix_len),
                                              max(1, max_context_len))
            if need == 0:
                raise ValueError("prefix_workspace: sizes not accepted by the library")
            self._ws_for = (sizes, need)
        return self._workspace(self._ws_for[1])

    def new_cache(self, n_blocks: int) -> torch.Tensor:
        """A zeroed paged cache: [n_blocks, 1, block_size, R], or [n_blocks, block bytes] uint8 if 8-bit."""
        if self.cache_dtype == "fp8":
            return torch.zeros((n_blocks, self.block_bytes), dtype=torch.uint8, device=self.device)
        return torch.zeros((n_blocks, 1, self.shape.block_size, self.shape.kv_row_dim), dtype=self.act,
                           device=self.device)

    def _check_cache(self, kv_cache):
        if kv_cache.dtype is not self._cache_torch or kv_cache.nbytes != kv_cache.shape[0] * self.block_bytes:
            raise ValueError(f"kv_cache does not hold blocks of this layer's cache ({self._cache_torch}, "
                             f"{self.block_bytes} bytes a block)")

    def _check_cache_bytes(self, kv_cache):
        """For the calls that took any tensor before: an 8-bit cache is checked, another only for its size."""
        if kv_cache is None:
            return
        if self.cache_dtype == "fp8":
            self._check_cache(kv_cache)
        elif kv_cache.nbytes < kv_cache.shape[0] * self.block_bytes:
            raise ValueError(f"kv_cache is smaller than its {kv_cache.shape[0]} blocks of {self.block_bytes} bytes")

    def _check_rows(self, rows):
        if rows.dtype != self.act or rows.dim() != 2 or rows.shape[1] != self.shape.kv_row_dim:
            raise ValueError(f"rows must be [n, {self.shape.kv_row_dim}] {self.act}")

    def cache_write(self, rows, kv_cache, slot_mapping):
        """rows [n, R] into the cache's flat rows slot_mapping (negative: skipped), quantised if it is 8-bit."""
        self._check_rows(rows)
        self._check_cache(kv_cache)
        ws = self._workspace(256) if self.ws is not None else self.workspace(1)   # the device flag alone
        mla_cache_write(self.handle, rows, kv_cache, slot_mapping, ws)
        return kv_cache

    def cache_read(self, kv_cache, slots, rows=None):
        """[n, R] in the activation dtype: the values of the cache's flat rows `slots`."""
        if rows is None:
            rows = torch.zeros((slots.numel(), self.shape.kv_row_dim), dtype=self.act, device=self.device)
        self._check_rows(rows)
        self._check_cache(kv_cache)
        ws = self._workspace(256) if self.ws is not None else self.workspace(1)   # the device flag alone
        mla_cache_read(self.handle, kv_cache, slots, rows, ws)
        return rows

    def _check_prefix(self, prefix_table, prefix_len):
        if prefix_len and (prefix_table is None or prefix_table.numel() * self.shape.block_size < prefix_len):
            raise ValueError("prefix_table does not cover prefix_len rows")

    def _check_query(self, q_abs, q_pe):
        s, a, p, act = self.shape, q_abs.shape, q_pe.shape, self.act
        n, heads = a[0], s.n_heads
        if a != (n, heads, s.kv_lora_rank) or p != (n, heads, s.qk_rope) or q_abs.dtype is not act or q_pe.dtype is not act:
            raise ValueError(f"q_abs must be [n, {s.n_heads}, {s.kv_lora_rank}] and q_pe [n, {s.n_heads}, {s.qk_rope}], {self.act}")

    def _check_out(self, n, out, head_out):
        s = self.shape
        if out.shape != (n, s.hidden) or out.dtype is not self.act:
            raise ValueError(f"out must be [{n}, {s.hidden}] {self.act}")
        if head_out is not None and (head_out.shape != (n, s.n_heads, s.v_dim) or head_out.dtype is not self.act):
            raise ValueError(f"head_out must be [{n}, {s.n_heads}, {s.v_dim}] {self.act}")

    def latent_attn(self, q_abs, q_pe, kv_cache, block_table, context_lens, max_context_len, prefix_table=None,
                    prefix_len: int = 0, o_lat=None, want_lse: bool = False):
        """(o_lat [n, H, r_kv], lse [n, H] fp32 or None) over the batch's shared prefix and each sequence's own rows."""
        self._check_query(q_abs, q_pe)
        self._check_cache(kv_cache)
        self._check_prefix(prefix_table, prefix_len)
        if o_lat is None:
            o_lat = torch.empty_like(q_abs)
        lse = torch.empty(q_abs.shape[:2], dtype=torch.float32, device=self.device) if want_lse else None
        ws = self.prefix_workspace(q_abs.shape[0], prefix_len, max_context_len)
        mla_latent_attn(self.handle, q_abs, q_pe, kv_cache, block_table, context_lens, max_context_len, o_lat, ws,
                        lse=lse, prefix_table=prefix_table, prefix_len=prefix_len)
        return o_lat, lse

    def decode_attn_prefix(self, q_abs, q_pe, kv_cache, prefix_table, prefix_len, block_table, context_lens,
                           max_context_len, out=None, head_out=None):
        """decode_attn over a prefix shared by the batch (its blocks in prefix_table) and each sequence's own rows."""
        self._check_query(q_abs, q_pe)
        self._check_cache(kv_cache)
        self._check_prefix(prefix_table, prefix_len)
        if out is None:
            out = torch.empty((q_abs.shape[0], self.shape.hidden), dtype=self.act, device=self.device)
        self._check_out(q_abs.shape[0], out, head_out)
        ws = self.prefix_workspace(q_abs.shape[0], prefix_len, max_context_len)
        mla_decode_attn_prefix(self.handle, q_abs, q_pe, kv_cache, prefix_table, prefix_len, block_table,
                               context_lens, max_context_len, out, ws, head_out=head_out)
        return out

    def rope(self, positions: torch.Tensor, inv_freq: torch.Tensor | None = None):
        """cos/sin [n, qk_rope/2] fp32 of the positions; inv_freq (device fp32
        [qk_rope/2], e.g. a YaRN table) replaces theta^(-2i/qk_rope)."""
        n = positions.numel()
        half = self.shape.qk_rope // 2
        cos = torch.empty((n, half), dtype=torch.float32, device=self.device)
        sin = torch.empty((n, half), dtype=torch.float32, device=self.device)
        if inv_freq is None:
            mla_rope_cos_sin(positions, self.shape.qk_rope, self.shape.rope_theta, cos, sin)
        else:
            mla_rope_cos_sin_inv_freq(positions, self.shape.qk_rope, inv_freq, cos, sin)
        return cos, sin

    def decode_qkv(self, hidden, cos, sin, kv_cache, slot_mapping, q_abs=None, q_pe=None, input_norm_w=None):
        s = self.shape
        n = hidden.shape[0]
        self._check_cache_bytes(kv_cache)
        if q_abs is None:
            q_abs = torch.empty((n, s.n_heads, s.kv_lora_rank), dtype=self.act, device=self.device)
        if q_pe is None:
            q_pe = torch.empty((n, s.n_heads, s.qk_rope), dtype=self.act, device=self.device)
        ws = self.workspace(n, 1)
        mla_decode_qkv(self.handle, hidden, cos, sin, kv_cache, slot_mapping, q_abs, q_pe, ws,
                       input_norm_w=input_norm_w)
        return q_abs, q_pe

    def decode_attn(self, q_abs, q_pe, kv_cache, block_table, context_lens, max_context_len,
                    out=None, head_out=None):
        s = self.shape
        n = q_abs.shape[0]
        self._check_cache_bytes(kv_cache)
        if out is None:
            out = torch.empty((n, s.hidden), dtype=self.act, device=self.device)
        ws = self.workspace(n, max_context_len)
        mla_decode_attn(self.handle, q_abs, q_pe, kv_cache, block_table, context_lens,
                        max_context_len, out, ws, head_out=head_out)
        return out

    def v4_qkv(self, hidden, cos, sin, kv_norm_w, q_out=None, kv_out=None):
        """DeepSeek-V4 QKV projection: (q [S, H, d_n + d_r], kv [S, r_kv + d_r])."""
        s = self.shape
        S = hidden.shape[0]
        if q_out is None:
            q_out = torch.empty((S, s.n_heads, s.qk_nope + s.qk_rope), dtype=self.act, device=self.device)
        if kv_out is None:
            kv_out = torch.empty((S, s.kv_lora_rank + s.qk_rope), dtype=self.act, device=self.device)
        ws = self.workspace(S, 1)
        mla_v4_qkv(self.handle, hidden, cos, sin, kv_norm_w, q_out, kv_out, ws)
        return q_out, kv_out

    def prefill(self, hidden, cos, sin, out=None, head_out=None, kv_cache=None, slot_mapping=None):
        s = self.shape
        S = hidden.shape[0]
        self._check_cache_bytes(kv_cache)
        if out is None:
            out = torch.empty((S, s.hidden), dtype=self.act, device=self.device)
        ws = self.workspace(S, 1)
        mla_prefill(self.handle, hidden, cos, sin, out, ws, head_out=head_out, kv_cache=kv_cache,
                    slot_mapping=slot_mapping)
        return out
