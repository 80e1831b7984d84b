"""The key/value cache in 4 bits: paged storage, append, read, attention and eviction.

Python face of the stagq_kv_* calls (include/stagq.h): argument checks and
marshalling only, everything runs in the native library.

    cache = KVCache(pages=512, kv_heads=8, head_dim=128)
    lengths += 1                                      # counts this step's token
    cache.append(k, v, table, lengths)                # k, v [B, 1, 8, 128]
    out = cache.attention(q, table, lengths, weights=w)
    kept, lengths = cache.evict(table, lengths, w, keep=4096, sinks=4, recent=256)
"""
from __future__ import annotations

import ctypes as C
import math
from typing import Optional, Tuple

from ._lib import KvAttn, KvCache, KvEvict, KvSeqs, KvTensor, check, lib


def _torch():
    import torch  # PyTorch only provides device memory and streams
    return torch


_DTYPES = None


def _dtypes():
    global _DTYPES
    if _DTYPES is None:
        torch = _torch()
        _DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
    return _DTYPES


class KVCache:
    """Keys and values of many sequences in 4 bits, in pages of page_tokens slots.

    A group of `group` channels of one token and kv head shares one pair
    (lo, s); a value is lo + s u, u in 0..15.  Sequences are given per call: an
    int32 page table [B, W] (any row stride) and int32 lengths [B], both on the
    cache's device.  lengths counts the tokens of the call.  A table entry
    outside [0, pages) stands for no page.

    page_tokens 32, 64, 128 or 256; head_dim 64, 96, 128 or 256; group 32, 64 or
    128 and a divisor of head_dim (64, or head_dim if smaller steps are needed: 32
    by default where 64 does not divide it).  buffer: a uint8 tensor to use (at
    least nbytes, 256-byte aligned); by default one is allocated, filled with 0.
    """

    def __init__(self, pages: int, kv_heads: int, head_dim: int, group: Optional[int] = None,
                 page_tokens: int = 64, device="cuda:0", buffer=None):
        torch = _torch()
        if group is None:
            group = 64 if head_dim % 64 == 0 else 32
        self._c = KvCache(int(pages), int(page_tokens), int(kv_heads), int(head_dim), int(group), 0, None, 0)
        n = int(lib().stagq_kv_bytes(C.byref(self._c)))
        if n == 0 and int(pages) != 0:
            check(-3, "stagq_kv_bytes")
        if buffer is None:
            buffer = torch.zeros(n, dtype=torch.uint8, device=device)
        if buffer.dtype != torch.uint8 or not buffer.is_contiguous() or buffer.numel() < n:
            raise ValueError(f"KVCache: buffer must be a contiguous uint8 tensor of at least {n} bytes")
        self.buffer = buffer
        self.device = buffer.device
        self.pages, self.page_tokens, self.kv_heads = int(pages), int(page_tokens), int(kv_heads)
        self.head_dim, self.group, self.nbytes = int(head_dim), int(group), n
        self._c.buf = buffer.data_ptr() or None
        self._c.bytes = buffer.numel()
        self._cp = C.addressof(self._c)

    # ------------------------------------------------------------ marshalling
    def _on(self, what, name, t, dtype, shape):
        """t is a tensor of this dtype and shape (None: any size) on the cache's device."""
        torch = _torch()
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: {name} must be a torch tensor")
        if t.dtype != dtype:
            raise ValueError(f"{what}: {name} must be {dtype}, not {t.dtype}")
        if t.device != self.device:
            raise ValueError(f"{what}: {name} is on {t.device}, the cache on {self.device}")
        if t.dim() != len(shape) or any(w is not None and w != s for w, s in zip(shape, t.shape)):
            want = ", ".join("*" if w is None else str(w) for w in shape)
            raise ValueError(f"{what}: {name} must have shape [{want}], not {list(t.shape)}")

    def _seqs(self, what, table, lengths) -> KvSeqs:
        torch = _torch()
        self._on(what, "table", table, torch.int32, (None, None))
        B, W = table.shape
        self._vector(what, "lengths", lengths, B)
        if W > 1 and table.stride(1) != 1:
            raise ValueError(f"{what}: the entries of a row of table must be adjacent")
        stride = table.stride(0) if B > 1 else W
        return KvSeqs(B, W, stride, table.data_ptr(), lengths.data_ptr())

    def _vector(self, what, name, t, n) -> None:
        self._on(what, name, t, _torch().int32, (n,))
        if n > 1 and t.stride(0) != 1:
            raise ValueError(f"{what}: {name} must be contiguous")

    def _rows(self, what, name, t, batch, heads, tokens=None, f32=True) -> KvTensor:
        torch = _torch()
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: {name} must be a torch tensor")
        code = _dtypes().get(t.dtype)
        if code is None or (code == 2 and not f32):
            raise ValueError(f"{what}: {name} must be float16, bfloat16{' or float32' if f32 else ''}, not {t.dtype}")
        self._on(what, name, t, t.dtype, (batch, tokens, heads, self.head_dim))
        if t.stride(3) != 1:
            raise ValueError(f"{what}: the channels of {name} must be adjacent")
        # strides of a size of one are never used; they may be anything
        sb, st, sh, _ = (0 if n == 1 else s for n, s in zip(t.shape, t.stride()))
        return KvTensor(t.data_ptr(), code, t.shape[1], t.shape[2], 0, sb, st, sh)

    def _columns(self, what, name, t, batch, need):
        self._on(what, name, t, _torch().float32, (batch, self.kv_heads, None))
        if t.shape[2] < need:
            raise ValueError(f"{what}: {name} has {t.shape[2]} slots per head, needs at least {need}")
        if t.shape[2] > 1 and t.stride(2) != 1:
            raise ValueError(f"{what}: the slots of {name} must be adjacent")

    def _reach(self, what, table, max_len) -> int:
        n = table.shape[1] * self.page_tokens
        if max_len is None:
            return n
        if max_len < 1:
            raise ValueError(f"{what}: max_len must be positive")
        return min(n, int(max_len))

    def _call(self, stream):
        """(stream, its pointer): the given stream or the device's current one."""
        torch = _torch()
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        elif stream.device != self.device:
            raise ValueError(f"stream is on {stream.device}, the cache on {self.device}")
        return stream, stream.cuda_stream

    class _Here:
        """The cache's device and the call's stream as current ones, for the call and what it allocates."""

        def __init__(self, stream):
            torch = _torch()
            self._ctx = None if (torch.cuda.current_device() == stream.device.index and
                                 torch.cuda.current_stream() == stream) else torch.cuda.stream(stream)

        def __enter__(self):
            if self._ctx is not None:
                self._ctx.__enter__()

        def __exit__(self, *a):
            if self._ctx is not None:
                self._ctx.__exit__(*a)

    # ------------------------------------------------------------- operators
    def append(self, k, v, table, lengths, new_lens=None, stream=None) -> None:
        """Quantise the rows of k and v [B, T, kv_heads, head_dim] (fp16, bf16 or
        fp32) into the cache: row i < n_b of sequence b becomes slot
        lengths[b] - n_b + i, with n_b = new_lens[b] or T.  Values are clamped to
        +-32768, NaN is held as 0.  The other slots keep what they hold."""
        B = table.shape[0] if hasattr(table, "shape") else 0
        seqs = self._seqs("append", table, lengths)
        kt = self._rows("append", "k", k, B, self.kv_heads)
        vt = self._rows("append", "v", v, B, self.kv_heads, k.shape[1])
        if k.dtype != v.dtype:
            raise ValueError(f"append: k is {k.dtype}, v {v.dtype}")
        if new_lens is not None:
            self._vector("append", "new_lens", new_lens, B)
        stream, ptr = self._call(stream)
        with self._Here(stream):
            check(lib().stagq_kv_append(self._cp, C.addressof(seqs), C.addressof(kt), C.addressof(vt),
                                        new_lens.data_ptr() if new_lens is not None else None, ptr),
                  "stagq_kv_append")

    def read(self, table, lengths, tokens: Optional[int] = None, start=None, dtype=None, k=None, v=None,
             stream=None) -> Tuple:
        """The values held, as (k, v) [B, tokens, kv_heads, head_dim]: row i is slot
        start[b] + i (start None: slot i; tokens None: the table's width).  Rows
        at or past lengths[b] are left as they are in a given k or v, and 0 in
        one allocated here (dtype: float32 unless given)."""
        torch = _torch()
        seqs = self._seqs("read", table, lengths)
        B = table.shape[0]
        if tokens is None:
            tokens = k.shape[1] if k is not None else table.shape[1] * self.page_tokens
        if start is not None:
            self._vector("read", "start", start, B)
        stream, ptr = self._call(stream)
        with self._Here(stream):
            shape = (B, int(tokens), self.kv_heads, self.head_dim)
            if dtype is None:
                dtype = k.dtype if k is not None else v.dtype if v is not None else torch.float32
            if k is None:
                k = torch.zeros(shape, dtype=dtype, device=self.device)
            if v is None:
                v = torch.zeros(shape, dtype=dtype, device=self.device)
            kt = self._rows("read", "k", k, B, self.kv_heads, int(tokens))
            vt = self._rows("read", "v", v, B, self.kv_heads, int(tokens))
            if k.dtype != v.dtype:
                raise ValueError(f"read: k is {k.dtype}, v {v.dtype}")
            check(lib().stagq_kv_read(self._cp, C.addressof(seqs),
                                      start.data_ptr() if start is not None else None, C.addressof(kt),
                                      C.addressof(vt), ptr), "stagq_kv_read")
        return k, v

    def attention(self, q, table, lengths, q_lens=None, scale: Optional[float] = None, causal: bool = True,
                  window: int = 0, max_len: Optional[int] = None, out=None, lse=None, weights=None, stream=None):
        """Attention of q [B, T, heads, head_dim] (fp16 or bf16; heads a multiple
        of kv_heads) over the cache; returns out, like q.

        Row i < q_lens[b] (None: T) stands at lengths[b] - q_lens[b] + i and sees
        the slots before lengths[b], up to its own where causal, and the last
        `window` of those where window > 0.  A row that sees nothing gives 0.
        Rows from q_lens[b] on are left as they are in a given out, and 0 in one
        allocated here.  scale: 1 / sqrt(head_dim) unless given.
          max_len  a bound of lengths known to the caller: sizes the launch (by
                   default the table's width); longer sequences are cut to it
          lse      fp32 [B, T, heads], contiguous: receives ln sum exp(scale q.k)
          weights  fp32 [B, kv_heads, >= max_len]: slot t gains the attention
                   weight it received, summed over rows and the kv head's heads
        """
        torch = _torch()
        seqs = self._seqs("attention", table, lengths)
        B = table.shape[0]
        if not isinstance(q, torch.Tensor):
            raise TypeError("attention: q must be a torch tensor")
        qt = self._rows("attention", "q", q, B, None, f32=False)
        heads = q.shape[2]
        if heads < 1 or heads % self.kv_heads:
            raise ValueError(f"attention: {heads} heads of q over {self.kv_heads} kv heads")
        if q_lens is not None:
            self._vector("attention", "q_lens", q_lens, B)
        reach = self._reach("attention", table, max_len)
        if lse is not None:
            self._on("attention", "lse", lse, torch.float32, (B, q.shape[1], heads))
            if not lse.is_contiguous():
                raise ValueError("attention: lse must be contiguous")
        if weights is not None:
            self._columns("attention", "weights", weights, B, reach)
        stream, ptr = self._call(stream)
        with self._Here(stream):
            if out is None:
                make = torch.empty if q_lens is None else torch.zeros
                out = make(q.shape, dtype=q.dtype, device=self.device)
            ot = self._rows("attention", "out", out, B, heads, q.shape[1], f32=False)
            if out.dtype != q.dtype:
                raise ValueError(f"attention: q is {q.dtype}, out {out.dtype}")
            a = KvAttn(qt, ot, q_lens.data_ptr() if q_lens is not None else None,
                       lse.data_ptr() if lse is not None else None,
                       weights.data_ptr() if weights is not None else None,
                       weights.stride(0) if weights is not None else 0,
                       weights.stride(1) if weights is not None else 0,
                       1.0 / math.sqrt(self.head_dim) if scale is None else float(scale),
                       1 if causal else 0, int(window), reach)
            need = int(lib().stagq_kv_attention_workspace(self._cp, C.addressof(seqs), C.addressof(a)))
            ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
            check(lib().stagq_kv_attention(self._cp, C.addressof(seqs), C.addressof(a),
                                           ws.data_ptr() if need else None, need, ptr), "stagq_kv_attention")
        return out

    def evict(self, table, lengths, weights, keep: int, sinks: int = 0, recent: int = 0,
              max_len: Optional[int] = None, out_table=None, weights_out=None, kept=None, out_lengths=None,
              stream=None) -> Tuple:
        """Keep the `keep` tokens of every sequence and kv head that accumulated
        the most attention weight; returns (kept, out_lengths).

        The first `sinks` and last `recent` tokens always stay (sinks + recent <=
        keep); ties go to the lowest slot; sequences of at most keep tokens stay
        whole.  The tokens that stay move together in their order, within their
        own pages, or to the pages of out_table [B, W'] (none of them among the
        pages read).  weights (fp32 [B, kv_heads, >= max_len]) moves along, in
        place or into weights_out, followed by 0.
          kept         int32 [B, kv_heads, keep]: the slots that stay, then -1
          out_lengths  int32 [B]: min(lengths, keep); may be lengths itself
        """
        torch = _torch()
        seqs = self._seqs("evict", table, lengths)
        B = table.shape[0]
        keep, sinks, recent = int(keep), int(sinks), int(recent)
        if keep < 1 or sinks < 0 or recent < 0 or sinks + recent > keep:
            raise ValueError(f"evict: sinks {sinks} and recent {recent} do not fit into keep {keep}")
        reach = self._reach("evict", table, max_len)
        self._columns("evict", "weights", weights, B, reach)
        if weights_out is None:
            weights_out = weights
        else:
            self._columns("evict", "weights_out", weights_out, B, reach)
        ow = os_ = 0
        if out_table is not None:
            self._on("evict", "out_table", out_table, torch.int32, (B, None))
            ow = out_table.shape[1]
            if ow > 1 and out_table.stride(1) != 1:
                raise ValueError("evict: the entries of a row of out_table must be adjacent")
            os_ = out_table.stride(0) if B > 1 else ow
            if ow * self.page_tokens < min(keep, reach):
                raise ValueError(f"evict: out_table holds {ow * self.page_tokens} tokens, needs {min(keep, reach)}")
        stream, ptr = self._call(stream)
        with self._Here(stream):
            if kept is None:
                kept = torch.empty((B, self.kv_heads, keep), dtype=torch.int32, device=self.device)
            else:
                self._on("evict", "kept", kept, torch.int32, (B, self.kv_heads, keep))
                if not kept.is_contiguous():
                    raise ValueError("evict: kept must be contiguous")
            if out_lengths is None:
                out_lengths = torch.empty(B, dtype=torch.int32, device=self.device)
            else:
                self._vector("evict", "out_lengths", out_lengths, B)
            e = KvEvict(weights.data_ptr(), weights_out.data_ptr(), weights.stride(0), weights.stride(1),
                        weights_out.stride(0), weights_out.stride(1), kept.data_ptr(), out_lengths.data_ptr(),
                        out_table.data_ptr() if out_table is not None else None, os_, ow, keep, sinks, recent,
                        reach, 0)
            need = int(lib().stagq_kv_evict_workspace(self._cp, C.addressof(seqs), C.addressof(e)))
            ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
            check(lib().stagq_kv_evict(self._cp, C.addressof(seqs), C.addressof(e),
                                       ws.data_ptr() if need else None, need, ptr), "stagq_kv_evict")
        return kept, out_lengths
