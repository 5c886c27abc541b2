"""Convenience layer over the C ABI: uploads weights with torch, owns a
library context and a set of canvas tensors, and reads results back.

No arithmetic of the method happens here; every step runs in the library's
kernels through the functions of this package.
"""
from __future__ import annotations

import contextlib
from dataclasses import dataclass
from typing import Dict, Optional

import numpy as np
import torch

from . import (DLM_BF16, DLM_F32, DLM_MASK, DLM_UNIFORM, dlm_canvas, dlm_canvas_init,
               dlm_canvas_stats, dlm_check, dlm_commit, dlm_create, dlm_debug_buffer,
               dlm_debug_logits, dlm_decode_block, dlm_decode_block_host, dlm_denoise_step, dlm_generate,
               dlm_destroy, dlm_kv_append, dlm_model_desc, dlm_paged_attention,
               dlm_paged_attention_workspace, dlm_paged_cache, dlm_paged_check,
               dlm_paged_kv_write, dlm_paged_resize, dlm_sampler_params, dlm_weights)

_NOTHING = contextlib.nullcontext()
_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
_NP_TYPESTR = {torch.float32: "<f4", torch.bfloat16: "<u2", torch.int32: "<i4",
               torch.uint8: "|u1"}


class _DevArray:
    """Zero-copy view of library-owned device memory for torch.as_tensor."""

    def __init__(self, ptr: int, shape, typestr: str):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr,
                                         "data": (int(ptr), False), "version": 2}


def host_to_device(a: np.ndarray, dtype: str, device) -> torch.Tensor:
    """numpy weights (bf16 bit patterns as uint16, or float32) -> device tensor."""
    if dtype == "bf16":
        t = torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    return t.to(device)


@dataclass
class Canvas:
    tokens: torch.Tensor
    committed: torch.Tensor
    step: torch.Tensor
    done: torch.Tensor
    eos_pos: torch.Tensor
    stats: torch.Tensor      # int32 [B][6]
    prev_cand: torch.Tensor  # int32 [B][C], adaptive stopping
    stable: torch.Tensor     # int32 [B], adaptive stopping

    @property
    def c(self) -> dlm_canvas:
        return dlm_canvas(self.tokens.data_ptr(), self.committed.data_ptr(),
                          self.step.data_ptr(), self.done.data_ptr(), self.eos_pos.data_ptr(),
                          self.prev_cand.data_ptr(), self.stable.data_ptr())

    def numpy(self) -> Dict[str, np.ndarray]:
        return {"tokens": self.tokens.cpu().numpy().astype(np.int64),
                "committed": self.committed.cpu().numpy().astype(bool),
                "step": self.step.cpu().numpy().astype(np.int64),
                "done": self.done.cpu().numpy().astype(bool),
                "eos_pos": self.eos_pos.cpu().numpy().astype(np.int64),
                "prev_cand": self.prev_cand.cpu().numpy().astype(np.int64),
                "stable": self.stable.cpu().numpy().astype(np.int64),
                "stats": self.stats.cpu().numpy()}

    def load(self, tokens, committed, step, done, eos_pos, prev_cand=None, stable=None) -> None:
        self.tokens.copy_(torch.as_tensor(np.asarray(tokens, dtype=np.int32)))
        self.committed.copy_(torch.as_tensor(np.asarray(committed, dtype=np.uint8)))
        self.step.copy_(torch.as_tensor(np.asarray(step, dtype=np.int32)))
        self.done.copy_(torch.as_tensor(np.asarray(done, dtype=np.uint8)))
        self.eos_pos.copy_(torch.as_tensor(np.asarray(eos_pos, dtype=np.int32)))
        if prev_cand is None:
            self.prev_cand.fill_(-1)
        else:
            self.prev_cand.copy_(torch.as_tensor(np.asarray(prev_cand, dtype=np.int32)))
        if stable is None:
            self.stable.zero_()
        else:
            self.stable.copy_(torch.as_tensor(np.asarray(stable, dtype=np.int32)))


def sampler_params(canvas: int, steps: int, threshold: float = 0.9, quota: int = 0,
                   corruption: str = "mask", entropy_bound: float = -1.0,
                   temperature: float = 0.0, t_max: float = 0.8, t_min: float = 0.4,
                   seed: int = 0, stability_steps: int = 1, stop_entropy: float = -1.0,
                   editing: int = 0, editing_threshold: float = 0.9) -> dlm_sampler_params:
    return dlm_sampler_params(canvas, steps, threshold, quota,
                              DLM_UNIFORM if corruption == "uniform" else DLM_MASK, editing,
                              entropy_bound, temperature, t_max, t_min, seed, stability_steps,
                              stop_entropy, editing_threshold)


class Session:
    """One library context for a model shape and its weights."""

    def __init__(self, shape, weights: Dict[str, np.ndarray], *, max_batch: int,
                 max_prefix: int, max_canvas: int, device="cuda:0", upload=None):
        self.shape = shape
        self.device = torch.device(device)
        self.dtype = _TORCH[shape.dtype]
        if upload is None:
            self.w = {k: host_to_device(v, shape.dtype, self.device) for k, v in weights.items()}
        else:
            self.w = upload
        desc = dlm_model_desc(shape.d_model, shape.n_heads, shape.n_kv_heads, shape.head_dim,
                              shape.vocab, DLM_BF16 if shape.dtype == "bf16" else DLM_F32,
                              float(shape.rope_theta), shape.mask_id, shape.eos_id,
                              max_batch, max_prefix, max_canvas,
                              2 if getattr(shape, "lm_nvfp4", False)
                              else (1 if getattr(shape, "lm_fp8", False) else 0))
        wts = dlm_weights(*(self.w[k].data_ptr() for k in
                            ("emb", "w_q", "w_k", "w_v", "w_o", "w_lm")))
        torch.cuda.synchronize(self.device)
        self.ctx = dlm_create(desc, wts)
        self.max_batch, self.max_prefix, self.max_canvas = max_batch, max_prefix, max_canvas

    def close(self) -> None:
        if getattr(self, "ctx", None):
            dlm_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- prefix -------------------------------------------------------------
    def kv_append_tokens(self, seq: int, tokens: np.ndarray, stream=None) -> None:
        t = torch.as_tensor(np.asarray(tokens, dtype=np.int32)).to(self.device)
        dlm_kv_append(self.ctx, seq, int(t.numel()), tokens=t, stream=stream)
        torch.cuda.synchronize(self.device)

    def kv_append_kv(self, seq: int, k: np.ndarray, v: np.ndarray, stream=None) -> None:
        """k, v: [Hkv][n][Dh] as bf16 bit patterns (uint16) or float32."""
        kt = host_to_device(k, self.shape.dtype, self.device)
        vt = host_to_device(v, self.shape.dtype, self.device)
        dlm_kv_append(self.ctx, seq, int(k.shape[1]), k=kt, v=vt, stream=stream)
        torch.cuda.synchronize(self.device)

    # -- canvas ---------------------------------------------------------------
    def new_canvas(self, batch: int, C: int) -> Canvas:
        dev = self.device
        return Canvas(torch.zeros((batch, C), dtype=torch.int32, device=dev),
                      torch.zeros((batch, C), dtype=torch.uint8, device=dev),
                      torch.zeros(batch, dtype=torch.int32, device=dev),
                      torch.zeros(batch, dtype=torch.uint8, device=dev),
                      torch.full((batch,), -1, dtype=torch.int32, device=dev),
                      torch.zeros((batch, 6), dtype=torch.int32, device=dev),
                      torch.full((batch, C), -1, dtype=torch.int32, device=dev),
                      torch.zeros(batch, dtype=torch.int32, device=dev))

    def init(self, cv: Canvas, p: dlm_sampler_params, stream=None) -> None:
        dlm_canvas_init(self.ctx, cv.c, cv.tokens.shape[0], p, stream=stream)

    def step(self, cv: Canvas, p: dlm_sampler_params, stream=None) -> None:
        dlm_denoise_step(self.ctx, cv.c, cv.tokens.shape[0], p, stats=cv.stats, stream=stream)

    def block(self, cv: Canvas, p: dlm_sampler_params, stream=None) -> None:
        dlm_decode_block(self.ctx, cv.c, cv.tokens.shape[0], p, stats=cv.stats, stream=stream)

    def commit(self, cv: Canvas, p: dlm_sampler_params, cand, conf, ent, stream=None) -> None:
        dlm_commit(self.ctx, cv.c, cv.tokens.shape[0], p, cand, conf, ent, stats=cv.stats,
                   stream=stream)

    def generate(self, cv: Canvas, p: dlm_sampler_params, n_blocks: int,
                 eos_early_stop: bool = True, stream=None) -> tuple:
        """(tokens [B][n_blocks*C] int32 on the device, blocks decoded)."""
        B, C = cv.tokens.shape
        out = torch.zeros((B, n_blocks * C), dtype=torch.int32, device=self.device)
        n = dlm_generate(self.ctx, cv.c, B, p, n_blocks, out, eos_early_stop=eos_early_stop,
                         stats=cv.stats, stream=stream)
        return out, n

    def check(self, stream=None) -> None:
        dlm_check(self.ctx, stream)

    # -- inspection ---------------------------------------------------------
    def buffer(self, which: int, shape, dtype: torch.dtype) -> torch.Tensor:
        ptr, nbytes = dlm_debug_buffer(self.ctx, which)
        n = int(np.prod(shape))
        assert n * torch.tensor([], dtype=dtype).element_size() <= nbytes
        t = torch.as_tensor(_DevArray(ptr, (n,), _NP_TYPESTR[dtype]), device=self.device)
        if dtype == torch.bfloat16:
            t = t.view(torch.bfloat16)
        return t.view(*shape)

    def logits(self, batch: int, C: int) -> torch.Tensor:
        out = torch.empty((batch * C, self.shape.vocab), dtype=torch.float32, device=self.device)
        dlm_debug_logits(self.ctx, batch, C, out)
        return out


class PagedCache:
    """A paged KV cache for a batch of sequences whose lengths differ: pages,
    block tables, free list and lengths as device tensors, and one step's calls
    in order -- resize(), write(), attend().  Nothing reads the lengths back, so
    a step can be captured into a CUDA graph (its tensors are then reused).

    Like a torch operation, every call runs on the cache's device, whichever is
    current, and on that device's current stream unless `stream` names another (a
    torch stream or a handle).  With a stream of its own a call does not wait for
    the current one, and the caller keeps its tensors until it is through; the
    tensor that attend() makes then belongs to that stream's pool."""

    def __init__(self, *, n_pages: int, page_size: int, n_heads: int, n_kv_heads: int,
                 head_dim: int, batch: int, max_len: int, max_new: int, dtype: str = "bf16",
                 device="cuda:0"):
        dev = torch.device(device)
        if dev.index is None:
            dev = torch.device(dev.type, torch.cuda.current_device())
        self.device = dev
        self.dtype = _TORCH[dtype]
        self.page_size, self.n_heads, self.batch, self.max_new = page_size, n_heads, batch, max_new
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        self.k = torch.empty(shape, dtype=self.dtype, device=dev)
        self.v = torch.empty(shape, dtype=self.dtype, device=dev)
        self.width = -(-max_len // page_size)
        self.table = torch.full((batch, self.width), -1, dtype=torch.int32, device=dev)
        self.free = torch.arange(n_pages, dtype=torch.int32, device=dev)
        self.n_free = torch.full((1,), n_pages, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.cu = torch.zeros(batch + 1, dtype=torch.int32, device=dev)
        self.slots = torch.full((max_new,), -1, dtype=torch.int64, device=dev)
        self.c = dlm_paged_cache(self.k.data_ptr(), self.v.data_ptr(), n_pages, page_size,
                                 n_kv_heads, head_dim, DLM_BF16 if dtype == "bf16" else DLM_F32)
        with torch.cuda.device(dev):
            self.work = torch.empty(dlm_paged_attention_workspace(self.c, n_heads),
                                    dtype=torch.uint8, device=dev)
            # the first call may come on any stream
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()

    def resize(self, new_lens: torch.Tensor, stream=None) -> None:
        """Lengths (int32 [batch], device) that the sequences are to have; a
        sequence that does not get its pages keeps its length (see .lens)."""
        if (new_lens.dtype != torch.int32 or new_lens.shape != (self.batch,) or
                not new_lens.is_contiguous()):
            raise ValueError("resize: new_lens is int32 [batch] without gaps")
        with self._on_device():
            dlm_paged_resize(self.lens, new_lens, self.lens, self.batch, self.table, self.width,
                             self.page_size, self.free, self.k.shape[0], self.n_free, self.n_free,
                             self.cu, self.slots, self.max_new, stream=self._stream(stream))

    def write(self, k: torch.Tensor, v: torch.Tensor, stream=None) -> None:
        """K and V of the last resize's new tokens, [<= max_new][n_kv_heads][head_dim]
        in sequence order (rows may be strided)."""
        if k.shape[0] != v.shape[0] or k.shape[0] > self.max_new:
            raise ValueError("write: k and v have one row per new token, at most max_new")
        heads = self.k.shape[1]
        ks, vs = self._stride(k, heads, "k"), self._stride(v, heads, "v")
        with self._on_device():
            dlm_paged_kv_write(self.c, k, v, self.slots, k.shape[0], k_stride=ks, v_stride=vs,
                               stream=self._stream(stream))

    def attend(self, q: torch.Tensor, mask_block: int, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Attention of the new tokens' queries [rows][n_heads][head_dim] over their
        sequences; mask_block 0 (every key), 1 (causal) or a block length, the same
        for the whole batch.  Rows of a sequence that the resize refused hold nothing
        of use, and rows behind the last sequence are not written."""
        qs = self._stride(q, self.n_heads, "q")
        if out is not None and out.shape != q.shape:
            raise ValueError("attend: out has q's shape")
        if lse is not None and (lse.dtype != torch.float32 or lse.shape != q.shape[:2] or
                                not lse.is_contiguous()):
            raise ValueError("attend: lse is float32 [rows][n_heads] without gaps")
        with self._on_device():
            s = self._stream(stream)
            if out is None and stream is None:
                out = torch.empty(q.shape, dtype=self.dtype, device=self.device)
            elif out is None:
                pool = s if isinstance(s, torch.cuda.Stream) else \
                    torch.cuda.ExternalStream(s.cuda_stream, device=self.device)
                with torch.cuda.stream(pool):
                    out = torch.empty(q.shape, dtype=self.dtype, device=self.device)
            dlm_paged_attention(self.c, q, out, self.cu, self.lens, self.table, self.width,
                                self.batch, q.shape[0], self.n_heads, mask_block, self.work, lse=lse,
                                q_stride=qs, o_stride=self._stride(out, self.n_heads, "out"), stream=s)
        return out

    def check(self, stream=None) -> None:
        """Wait for the stream; raises what the device recorded (dlm_paged_check)."""
        with self._on_device():
            dlm_paged_check(self._stream(stream))

    def _on_device(self):
        """The cache's device as the current one (a guard takes microseconds: only where needed)."""
        if torch.cuda.current_device() == self.device.index:
            return _NOTHING
        return torch.cuda.device(self.device)

    def _stream(self, stream):
        """The stream of a call: the one given, or the device's current one (its handle: a
        stream object of torch's takes microseconds to make)."""
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.device.index)
        if isinstance(stream, int):
            if stream in (0, 1):    # CUDA's names for the default stream
                return torch.cuda.default_stream(self.device)
            return torch.cuda.ExternalStream(stream, device=self.device)
        if getattr(stream, "device", self.device) != self.device:
            raise ValueError("PagedCache: a stream of another device")
        return stream

    def _stride(self, t: torch.Tensor, heads: int, what: str) -> int:
        """Elements between rows of [rows][heads][head_dim] (0: there is one at most)."""
        dim = self.k.shape[3]
        if (t.dtype != self.dtype or t.dim() != 3 or tuple(t.shape[1:]) != (heads, dim) or
                t.stride(2) != 1 or (heads > 1 and t.stride(1) != dim) or
                (t.shape[0] > 1 and t.stride(0) < heads * dim)):
            raise ValueError("%s: [rows][heads][head_dim] of the cache's type, heads without gaps "
                             "and rows that do not overlap" % what)
        return t.stride(0) if t.shape[0] > 1 else 0
