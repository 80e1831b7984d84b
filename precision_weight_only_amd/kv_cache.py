"""The key/value cache in 4 bits: paged storage, append, read, attention and eviction.

Python face of the stagq_kv_* calls (include/stagq.h): argument checks and
marshalling only, everything runs in the native library.

    cache = KVCache(pages=512, kv_heads=8, head_dim=128)
    lengths += 1                                      # counts this step's token
    cache.append(k, v, table, lengths)                # k, v [B, 1, 8, 128]
    out = cache.attention(q, table, lengths, weights=w)
    kept, lengths = cache.evict(table, lengths, w, keep=4096, sinks=4, recent=256)

A decode step makes two of these calls per layer, each a few microseconds on the
GPU, so the host's share counts: structs are packed as bytes (a third of the time
of ctypes structures), and every attribute of a tensor is looked at once.
"""
from __future__ import annotations

import math
from struct import Struct
from typing import Optional, Tuple

import torch

from ._lib import check, lib

# the current device and its current stream as a pointer, without building objects (about 2 us a call)
_device_index = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)

_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_I32, _F32 = torch.int32, torch.float32
# the structs of include/stagq.h, in their layout
_CACHE = Struct("iiiiiiQQ")        # stagq_kv_cache
_SEQS = Struct("iiqQQ")            # stagq_kv_seqs
_TENSOR = Struct("Qiiiiqqq")       # stagq_kv_tensor
_ATTN_REST = Struct("QQQqqfiiiii")  # stagq_kv_attn after its two tensors
_EVICT = Struct("QQqqqqQQQqiiiiii")  # stagq_kv_evict_args


class _On:
    """The device and stream of a call as current ones, for the call and what it allocates."""

    def __init__(self, device, stream):
        self._device = torch.cuda.device(device)
        self._stream = torch.cuda.stream(stream) if stream is not None else None

    def __enter__(self):
        self._device.__enter__()
        if self._stream is not None:
            self._stream.__enter__()

    def __exit__(self, *a):
        if self._stream is not None:
            self._stream.__exit__(*a)
        self._device.__exit__(*a)


def _fail(what, name, t, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: {name} must be a torch tensor")
    if t.dtype != dtype:
        raise ValueError(f"{what}: {name} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{what}: {name} is on {t.device}, the cache on {device}")
    want = ", ".join("*" if w is None else str(w) for w in shape)
    raise ValueError(f"{what}: {name} must have shape [{want}], the last size contiguous, not {list(t.shape)} with "
                     f"strides {t.stride()}")


class KVCache:
    """Keys and values of many sequences in 4 bits, in pages of page_tokens slots.

    A group of `group` channels of one token and kv head shares one pair
    (lo, s); a value is lo + s u, u in 0..15.  Sequences are given per call: an
    int32 page table [B, W] (any row stride) and int32 lengths [B], both on the
    cache's device.  lengths counts the tokens of the call.  A table entry
    outside [0, pages) stands for no page.

    page_tokens 32, 64, 128 or 256; head_dim 64, 96, 128 or 256; group 32, 64 or
    128 and a divisor of head_dim (by default 64, or 32 where 64 is none).
    buffer: a uint8 tensor to use (at least nbytes, 256-byte aligned); by default
    one is allocated, filled with 0.

    The calls answer with values only: none of them records a gradient.  Tensors
    that a call writes must not overlap themselves (an expanded one does).

    Every call runs on the given stream, or the device's current one, and
    returns without waiting for it.  Workspaces come from torch's allocator on
    that stream, one per call, so calls on several streams and captured ones do
    not share any.
    """

    def __init__(self, pages: int, kv_heads: int, head_dim: int, group: Optional[int] = None,
                 page_tokens: int = 64, device="cuda:0", buffer=None):
        if group is None:
            group = 64 if head_dim % 64 == 0 else 32
        shape = (int(pages), int(page_tokens), int(kv_heads), int(head_dim), int(group), 0)
        n = int(lib().stagq_kv_bytes(_CACHE.pack(*shape, 0, 0)))
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
        self._c = _CACHE.pack(*shape, buffer.data_ptr(), buffer.numel())
        self._scale = 1.0 / math.sqrt(self.head_dim)
        self._lib = lib()
        self._needs = {}   # workspace bytes of attention by everything they depend on

    # ------------------------------------------------------------ marshalling
    def _seqs(self, what, table, lengths):
        """(batch, table width, packed struct)."""
        dev = self.device
        if not isinstance(table, torch.Tensor) or table.dtype != _I32 or table.device != dev or table.dim() != 2:
            _fail(what, "table", table, _I32, (None, None), dev)
        (B, W), (row, one) = table.shape, table.stride()
        if one != 1 and W > 1:
            _fail(what, "table", table, _I32, (None, None), dev)
        return B, W, _SEQS.pack(B, W, row if B > 1 else W, table.data_ptr(), self._vector(what, "lengths", lengths, B))

    def _vector(self, what, name, t, n) -> int:
        if t is None:
            if name == "lengths":
                raise TypeError(f"{what}: lengths must be a torch tensor")
            return 0
        if (not isinstance(t, torch.Tensor) or t.dtype != _I32 or t.device != self.device or t.shape != (n,)
                or not t.is_contiguous()):
            _fail(what, name, t, _I32, (n,), self.device)
        return t.data_ptr()

    def _rows(self, what, name, t, batch, tokens, heads, f32=True):
        """(tokens, heads, packed struct) of a [batch, tokens, heads, head_dim] tensor (None: any)."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: {name} must be a torch tensor")
        code = _DTYPES.get(t.dtype, 3)
        if code > (2 if f32 else 1):
            raise ValueError(f"{what}: {name} must be float16, bfloat16{' or float32' if f32 else ''}, not {t.dtype}")
        if t.dim() != 4 or t.device != self.device:
            _fail(what, name, t, t.dtype, (batch, tokens, heads, self.head_dim), self.device)
        (b, n, h, d), (sb, st, sh, sd) = t.shape, t.stride()
        if (b != batch or d != self.head_dim or sd != 1 or (tokens is not None and n != tokens)
                or (heads is not None and h != heads)):
            _fail(what, name, t, t.dtype, (batch, tokens, heads, self.head_dim), self.device)
        # the stride of a size of one is never used and may be anything
        return n, h, _TENSOR.pack(t.data_ptr(), code, n, h, 0, sb if b > 1 else 0, st if n > 1 else 0, sh if h > 1 else 0)

    def _columns(self, what, name, t, batch, need):
        """(address, stride of a sequence, of a head) of fp32 [batch, kv_heads, >= need]."""
        if (not isinstance(t, torch.Tensor) or t.dtype != _F32 or t.device != self.device or t.dim() != 3
                or t.shape[0] != batch or t.shape[1] != self.kv_heads):
            _fail(what, name, t, _F32, (batch, self.kv_heads, None), self.device)
        sb, sh, one = t.stride()
        if t.shape[2] < need:
            raise ValueError(f"{what}: {name} has {t.shape[2]} slots per head, needs at least {need}")
        if one != 1 and t.shape[2] > 1:
            _fail(what, name, t, _F32, (batch, self.kv_heads, None), self.device)
        return t.data_ptr(), sb, sh

    def _reach(self, what, width, max_len) -> int:
        n = width * self.page_tokens
        if max_len is None:
            return n
        if max_len < 1:
            raise ValueError(f"{what}: max_len must be positive")
        return min(n, int(max_len))

    def _run(self, stream, call):
        """call(stream pointer) with the cache's device, and the given stream, current."""
        index = self.device.index
        if stream is None:
            if _device_index() == index:
                return call(_raw_stream(index))
            with _On(self.device, None):
                return call(_raw_stream(index))
        if stream.device != self.device:
            raise ValueError(f"stream is on {stream.device}, the cache on {self.device}")
        with _On(self.device, stream):
            return call(stream.cuda_stream)

    # ------------------------------------------------------------- operators
    def append(self, k, v, table, lengths, new_lens=None, stream=None) -> None:
        """Quantise the rows of k and v [B, T, kv_heads, head_dim] (fp16, bf16 or
        fp32) into the cache: row i < n_b of sequence b becomes slot
        lengths[b] - n_b + i, with n_b = new_lens[b] or T.  Values are clamped to
        +-32768, NaN is held as 0.  The other slots keep what they hold."""
        B, _, seqs = self._seqs("append", table, lengths)
        n, _, kt = self._rows("append", "k", k, B, None, self.kv_heads)
        _, _, vt = self._rows("append", "v", v, B, n, self.kv_heads)
        if k.dtype != v.dtype:
            raise ValueError(f"append: k is {k.dtype}, v {v.dtype}")
        new = self._vector("append", "new_lens", new_lens, B)
        self._run(stream, lambda st: check(self._lib.stagq_kv_append(self._c, seqs, kt, vt, new, st), "stagq_kv_append"))

    def read(self, table, lengths, tokens: Optional[int] = None, start=None, dtype=None, k=None, v=None,
             stream=None) -> Tuple:
        """The values held, as (k, v) [B, tokens, kv_heads, head_dim]: row i is slot
        start[b] + i (start None: slot i; tokens None: the table's width).  Rows
        whose slot is not in 0 .. lengths[b] - 1 are left as they are in a given k
        and v, and 0 in ones allocated here (dtype: float32 unless given)."""
        B, W, seqs = self._seqs("read", table, lengths)
        at = self._vector("read", "start", start, B)
        if (k is None) != (v is None):
            raise ValueError("read: give k and v, or neither")
        if tokens is None:
            tokens = W * self.page_tokens if k is None else k.shape[1]

        def call(st):
            nonlocal k, v
            fresh = k is None
            if fresh:
                kind = dtype or _F32
                if kind not in _DTYPES:
                    raise ValueError(f"read: dtype must be float16, bfloat16 or float32, not {kind}")
                h, d = self.kv_heads, self.head_dim
                both = torch.empty((2, B, tokens, h, d), dtype=kind, device=self.device)
                k, v = both.unbind(0)
                rest = (_DTYPES[kind], tokens, h, 0, tokens * h * d, h * d, d)
                kt, vt = _TENSOR.pack(k.data_ptr(), *rest), _TENSOR.pack(v.data_ptr(), *rest)
            else:
                _, _, kt = self._rows("read", "k", k, B, tokens, self.kv_heads)
                _, _, vt = self._rows("read", "v", v, B, tokens, self.kv_heads)
                if k.dtype != v.dtype:
                    raise ValueError(f"read: k is {k.dtype}, v {v.dtype}")
            check(self._lib.stagq_kv_read(self._c, seqs, at, kt, vt, 1 if fresh else 0, st), "stagq_kv_read")
            return k, v

        return self._run(stream, call)

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
        B, W, seqs = self._seqs("attention", table, lengths)
        n, heads, qt = self._rows("attention", "q", q, B, None, None, False)
        if heads < 1 or heads % self.kv_heads:
            raise ValueError(f"attention: {heads} heads of q over {self.kv_heads} kv heads")
        ql = self._vector("attention", "q_lens", q_lens, B)
        reach = self._reach("attention", W, max_len)
        window = int(window)
        if not 0 <= window < 2 ** 31:
            raise ValueError(f"attention: window must be 0 (none) or a number of slots below 2^31, not {window}")
        ls = 0
        if lse is not None:
            if (not isinstance(lse, torch.Tensor) or lse.dtype != _F32 or lse.device != self.device
                    or lse.shape != (B, n, heads) or not lse.is_contiguous()):
                _fail("attention", "lse", lse, _F32, (B, n, heads), self.device)
            ls = lse.data_ptr()
        w, wb, wh = (0, 0, 0) if weights is None else self._columns("attention", "weights", weights, B, reach)

        def call(st):
            nonlocal out
            fresh = out is None
            if fresh:
                out = torch.empty(q.shape, dtype=q.dtype, device=self.device)
                d = self.head_dim
                ot = _TENSOR.pack(out.data_ptr(), _DTYPES[q.dtype], n, heads, 0, n * heads * d, heads * d, d)
            else:
                _, _, ot = self._rows("attention", "out", out, B, n, heads, False)
                if out.dtype != q.dtype:
                    raise ValueError(f"attention: q is {q.dtype}, out {out.dtype}")
            a = qt + ot + _ATTN_REST.pack(ql, ls, w, wb, wh, self._scale if scale is None else scale,
                                          1 if causal else 0, window, reach, 1 if fresh and ql else 0, 0)
            key = (B, n, heads, window, reach, ls != 0, w != 0)
            need = self._needs.get(key)
            first = need is None
            if first:
                need = self._lib.stagq_kv_attention_workspace(self._c, seqs, a)
            ws = torch.empty(need, dtype=torch.uint8, device=self.device).data_ptr() if need else 0
            status = self._lib.stagq_kv_attention(self._c, seqs, a, ws, need, st)
            if status:
                check(status, "stagq_kv_attention")
            if first and len(self._needs) < 4096:   # not that of a refused call, which is 0
                self._needs[key] = need
            return out

        return self._run(stream, call)

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
        B, W, seqs = self._seqs("evict", table, lengths)
        keep, sinks, recent = int(keep), int(sinks), int(recent)
        if keep < 1 or sinks < 0 or recent < 0 or sinks + recent > keep:
            raise ValueError(f"evict: sinks {sinks} and recent {recent} do not fit into keep {keep}")
        reach = self._reach("evict", W, max_len)
        w, wb, wh = self._columns("evict", "weights", weights, B, reach)
        o, ob, oh = (w, wb, wh) if weights_out is None else self._columns("evict", "weights_out", weights_out, B, reach)
        ot = ow = os_ = 0
        if out_table is not None:
            if (not isinstance(out_table, torch.Tensor) or out_table.dtype != _I32 or out_table.device != self.device
                    or out_table.dim() != 2 or out_table.shape[0] != B
                    or (out_table.shape[1] > 1 and out_table.stride(1) != 1)):
                _fail("evict", "out_table", out_table, _I32, (B, None), self.device)
            ow = out_table.shape[1]
            os_ = out_table.stride(0) if B > 1 else ow
            ot = out_table.data_ptr()
            if ow * self.page_tokens < min(keep, reach):
                raise ValueError(f"evict: out_table holds {ow * self.page_tokens} tokens, needs {min(keep, reach)}")

        def call(st):
            nonlocal kept, out_lengths
            if kept is None:
                kept = torch.empty((B, self.kv_heads, keep), dtype=_I32, device=self.device)
            elif (not isinstance(kept, torch.Tensor) or kept.dtype != _I32 or kept.device != self.device
                    or kept.shape != (B, self.kv_heads, keep) or not kept.is_contiguous()):
                _fail("evict", "kept", kept, _I32, (B, self.kv_heads, keep), self.device)
            if out_lengths is None:
                out_lengths = torch.empty(B, dtype=_I32, device=self.device)
            e = _EVICT.pack(w, o, wb, wh, ob, oh, kept.data_ptr(), self._vector("evict", "out_lengths", out_lengths, B),
                            ot, os_, ow, keep, sinks, recent, reach, 0)
            need = self._lib.stagq_kv_evict_workspace(self._c, seqs, e)
            ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
            check(self._lib.stagq_kv_evict(self._c, seqs, e, ws.data_ptr() if need else 0, need, st), "stagq_kv_evict")
            return kept, out_lengths

        return self._run(stream, call)
