"""The key/value cache on the CPU: its layout, its oracle, and every refusal of
the library and the binding (nothing is launched)."""
import ctypes as C
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

import precision_weight_only_amd as pwo
from oracle import kv_oracle

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

EINVAL, ESHAPE, EALIGN, ESIZE = -1, -3, -5, -8


class KvCache(C.Structure):
    _fields_ = [
        ("pages", C.c_int32), ("page_tokens", C.c_int32), ("kv_heads", C.c_int32), ("head_dim", C.c_int32),
        ("group", C.c_int32), ("spare", C.c_int32), ("buf", C.c_void_p), ("bytes", C.c_uint64),
    ]


class KvSeqs(C.Structure):
    _fields_ = [
        ("batch", C.c_int32), ("table_width", C.c_int32), ("table_stride", C.c_int64), ("table", C.c_void_p),
        ("lengths", C.c_void_p),
    ]


class KvTensor(C.Structure):
    _fields_ = [
        ("data", C.c_void_p), ("dtype", C.c_int32), ("tokens", C.c_int32), ("heads", C.c_int32),
        ("spare", C.c_int32), ("stride_seq", C.c_int64), ("stride_token", C.c_int64), ("stride_head", C.c_int64),
    ]


class KvAttn(C.Structure):
    _fields_ = [
        ("q", KvTensor), ("out", KvTensor), ("q_lens", C.c_void_p), ("lse", C.c_void_p), ("weights", C.c_void_p),
        ("weights_stride_seq", C.c_int64), ("weights_stride_head", C.c_int64), ("scale", C.c_float),
        ("causal", C.c_int32), ("window", C.c_int32), ("max_len", C.c_int32), ("zero_rest", C.c_int32),
        ("spare", C.c_int32),
    ]


class KvEvict(C.Structure):
    _fields_ = [
        ("weights", C.c_void_p), ("weights_out", C.c_void_p), ("weights_stride_seq", C.c_int64),
        ("weights_stride_head", C.c_int64), ("out_stride_seq", C.c_int64), ("out_stride_head", C.c_int64),
        ("kept", C.c_void_p), ("out_lengths", C.c_void_p), ("out_table", C.c_void_p),
        ("out_table_stride", C.c_int64), ("out_table_width", C.c_int32), ("keep", C.c_int32), ("sinks", C.c_int32),
        ("recent", C.c_int32), ("max_len", C.c_int32), ("spare", C.c_int32),
    ]


def test_packed_structs_have_the_layout_of_the_header():
    from precision_weight_only_amd import kv_cache as m
    assert m._CACHE.size == C.sizeof(KvCache) and m._SEQS.size == C.sizeof(KvSeqs)
    assert m._TENSOR.size == C.sizeof(KvTensor) and m._EVICT.size == C.sizeof(KvEvict)
    assert 2 * m._TENSOR.size + m._ATTN_REST.size == C.sizeof(KvAttn)
    c = KvCache.from_buffer_copy(m._CACHE.pack(1, 2, 3, 4, 5, 0, 6, 7))
    assert (c.pages, c.page_tokens, c.kv_heads, c.head_dim, c.group, c.buf, c.bytes) == (1, 2, 3, 4, 5, 6, 7)
    t = m._TENSOR.pack(1, 2, 3, 4, 0, 5, 6, 7)
    a = KvAttn.from_buffer_copy(t + t + m._ATTN_REST.pack(1, 2, 3, 4, 5, 0.5, 6, 7, 8, 9, 0))
    assert (a.out.data, a.out.stride_head, a.q_lens, a.lse, a.weights) == (1, 7, 1, 2, 3)
    assert (a.weights_stride_head, a.scale, a.causal, a.window, a.max_len, a.zero_rest) == (5, 0.5, 6, 7, 8, 9)
    e = KvEvict.from_buffer_copy(m._EVICT.pack(*range(1, 17)))
    assert [getattr(e, f) for f, _ in KvEvict._fields_] == list(range(1, 17))


def test_layout_uses_every_byte_once(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    exe = str(tmp_path / "kv_layout")
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", os.path.join(ROOT, "precision_weight_only_amd", "csrc"),
                    os.path.join(ROOT, "tests", "native", "kv_layout.cpp"), "-o", exe], check=True, timeout=120)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "layout ok" in r.stdout, r.stdout


# ------------------------------------------------------------------ oracle --
def test_oracle_codes_are_the_nearest_with_ties_upward():
    # lo = -1, s = fp16(2 / 15): values on both sides of a border and on it
    s = float(np.float16(np.float32(2.0) / np.float32(15.0)))
    x = np.zeros(32)
    x[0], x[1] = -1.0, 1.0
    x[2] = -1.0 + 2.5 * s
    x[3] = np.nextafter(x[2], -2.0)
    u, lo, st = kv_oracle.quantise(x, 32)
    assert lo[0] == -1.0 and st[0] == s and u[2] == 3 and u[3] == 2 and u[0] == 0 and u[1] == 15
    v = kv_oracle.values(u, lo, st)
    assert np.abs(v - x).max() <= 0.5 * s + 15 * s * 2.0 ** -11   # half a step, and s itself half an ulp off


def test_oracle_constant_group_clamp_and_nan():
    u, lo, s = kv_oracle.quantise(np.full(64, 3.25), 32)
    assert (u == 0).all() and (lo == 3.25).all() and (s == 0).all()
    x = np.zeros(32)
    x[:3] = np.inf, -np.inf, np.nan
    v = kv_oracle.values(*kv_oracle.quantise(x, 32))
    assert np.isfinite(v).all() and v[1] == -32768.0 and abs(v[0] - 32768.0) <= 32.0
    assert abs(v[2]) <= 0.5 * 4368.0 + 1


def test_oracle_attention_by_hand():
    # two tokens, D = 32 with k = e_0 * (0, 1): softmax of (0, z)
    k, v = np.zeros((2, 32)), np.zeros((2, 32))
    k[1, 0], v[1] = 15.0, 30.0
    kq, vq = kv_oracle.quantise(k, 32), kv_oracle.quantise(v, 32)
    q = np.zeros((1, 1, 32))
    q[0, 0, 0] = math.log(3.0) / 15.0
    r = kv_oracle.attention(q, kq, vq, 1.0)
    assert np.allclose(r["out"], 22.5) and np.allclose(r["weights"], [0.25, 0.75]) and np.allclose(r["lse"], math.log(4))
    r = kv_oracle.attention(q, kq, vq, 1.0, absent=(0, 1))
    assert (r["out"] == 0).all() and (r["lse"] == -np.inf).all() and (r["weights"] == 0).all()
    r = kv_oracle.attention(np.repeat(q, 3, 0), kq, vq, 1.0)   # more rows than tokens: the first sees nothing
    assert (r["out"][0] == 0).all() and r["lse"][0, 0] == -np.inf and np.allclose(r["lse"][1, 0], 0.0)


def test_oracle_evict_ties_and_ends():
    w = np.array([0, 5, 1, 1, 1, 0, 0, 2, 0, 0], float)
    assert kv_oracle.evict(w, 6, 1, 2).tolist() == [0, 1, 2, 7, 8, 9]
    assert kv_oracle.evict(w, 5, 2, 3).tolist() == [0, 1, 7, 8, 9]
    assert kv_oracle.evict(w, 10, 0, 0).tolist() == list(range(10))
    assert kv_oracle.evict(np.array([0.0, np.nan, 3.0]), 1, 0, 0).tolist() == [1]


# ---------------------------------------------------------- library refusals --
def _cache(**kw):
    f = dict(pages=8, page_tokens=64, kv_heads=2, head_dim=128, group=64, spare=0, buf=4096, bytes=1 << 40)
    f.update(kw)
    return KvCache(**f)


def _seqs(**kw):
    f = dict(batch=3, table_width=4, table_stride=4, table=4096, lengths=4096)
    f.update(kw)
    return KvSeqs(**f)


def _tensor(**kw):
    f = dict(data=4096, dtype=0, tokens=2, heads=2, spare=0, stride_seq=512, stride_token=256, stride_head=128)
    f.update(kw)
    return KvTensor(**f)


def _attn(q=None, out=None, **kw):
    q = q or _tensor(heads=4, stride_token=512, stride_seq=1024)
    if out is None:
        out = type(q).from_buffer_copy(q)
        out.data = 8192
    f = dict(q=q, out=out, q_lens=None, lse=None, weights=None, weights_stride_seq=0, weights_stride_head=0,
             scale=0.1, causal=1, window=0, max_len=0, zero_rest=0, spare=0)
    f.update(kw)
    return KvAttn(**f)


def _evict(**kw):
    f = dict(weights=4096, weights_out=4096, weights_stride_seq=512, weights_stride_head=256, out_stride_seq=512,
             out_stride_head=256, kept=4096, out_lengths=4096, out_table=8192, out_table_stride=4, out_table_width=4,
             keep=10, sinks=2, recent=3, max_len=0, spare=0)
    f.update(kw)
    return KvEvict(**f)


A = C.addressof


def _rows_calls(c, s, k, v, counts=None):
    lib = pwo.lib()
    return {lib.stagq_kv_append(A(c), A(s), A(k), A(v), counts, None),
            lib.stagq_kv_read(A(c), A(s), counts, A(k), A(v), 0, None)}


BAD_CACHES = [(dict(page_tokens=48), ESHAPE), (dict(kv_heads=0), ESHAPE), (dict(kv_heads=1025), ESHAPE),
              (dict(head_dim=80), ESHAPE), (dict(group=48), ESHAPE), (dict(head_dim=96, group=64), ESHAPE),
              (dict(pages=-1), ESHAPE), (dict(buf=None), EINVAL), (dict(buf=4096 + 16), EALIGN), (dict(bytes=1000), ESIZE)]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_refused_caches(bad, status):
    lib = pwo.lib()
    c, s, t = _cache(**bad), _seqs(), _tensor()
    assert _rows_calls(c, s, t, t) == {status}
    assert lib.stagq_kv_attention(A(c), A(s), A(_attn()), None, 0, None) == status
    assert lib.stagq_kv_evict(A(c), A(s), A(_evict()), None, 0, None) == status


@pytest.mark.parametrize("bad,status", [
    (dict(batch=-1), EINVAL), (dict(table_width=-1), EINVAL), (dict(table=None), EINVAL), (dict(lengths=None), EINVAL),
    (dict(table=4098), EALIGN), (dict(lengths=4097), EALIGN), (dict(table_stride=3), EINVAL),
    (dict(batch=(1 << 20) + 1), ESHAPE)])
def test_refused_sequences(bad, status):
    lib = pwo.lib()
    c, s, t = _cache(), _seqs(**bad), _tensor()
    assert _rows_calls(c, s, t, t) == {status}
    assert lib.stagq_kv_attention(A(c), A(s), A(_attn()), None, 0, None) == status
    assert lib.stagq_kv_evict(A(c), A(s), A(_evict()), None, 0, None) == status


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=3), EINVAL), (dict(data=None), EINVAL), (dict(data=4104), EALIGN), (dict(heads=3), ESHAPE),
    (dict(tokens=-1), ESHAPE), (dict(stride_seq=-8), EINVAL), (dict(stride_token=252), EALIGN),
    (dict(stride_head=4), EALIGN)])
def test_refused_tensors(bad, status):
    lib = pwo.lib()
    c, s = _cache(), _seqs()
    assert _rows_calls(c, s, _tensor(**bad), _tensor()) == {status}
    assert _rows_calls(c, s, _tensor(), _tensor(**bad)) == {status}
    f = dict(heads=4, stride_token=512, stride_seq=1024)
    f.update(bad)
    assert lib.stagq_kv_attention(A(c), A(s), A(_attn(q=_tensor(**f))), None, 0, None) == status


def test_refused_pairs_of_tensors():
    c, s = _cache(), _seqs()
    assert _rows_calls(c, s, _tensor(), _tensor(dtype=1)) == {EINVAL}
    assert _rows_calls(c, s, _tensor(), _tensor(tokens=3)) == {EINVAL}
    assert _rows_calls(c, s, _tensor(), _tensor(), counts=4098) == {EALIGN}
    # sizes past one launch
    big = _tensor(tokens=(1 << 31) - 64)
    assert _rows_calls(c, s, big, big) == {ESHAPE}


@pytest.mark.parametrize("bad,status", [
    (dict(window=-1), EINVAL), (dict(window=4, causal=0), EINVAL), (dict(max_len=-1), EINVAL),
    (dict(scale=math.inf), EINVAL), (dict(scale=-1e31), EINVAL), (dict(scale=math.nan), EINVAL), (dict(lse=4098), EALIGN), (dict(q_lens=4097), EALIGN),
    (dict(weights=4098), EALIGN), (dict(weights=4096, weights_stride_seq=-1), EINVAL),
    (dict(out=_tensor(heads=4, dtype=1)), EINVAL), (dict(out=_tensor(heads=4, tokens=5)), EINVAL),
    (dict(q=_tensor(heads=5)), ESHAPE), (dict(out=_tensor(heads=4, stride_token=512, stride_seq=1024)), EINVAL), (dict(q=_tensor(heads=4, dtype=2)), EINVAL)])
def test_refused_attention(bad, status):
    a = _attn(**bad)
    assert pwo.lib().stagq_kv_attention(A(_cache()), A(_seqs()), A(a), None, 0, None) == status
    assert pwo.lib().stagq_kv_attention_workspace(A(_cache()), A(_seqs()), A(a)) == 0


def test_attention_workspace_is_checked():
    lib = pwo.lib()
    c, s, a = _cache(pages=100000), _seqs(table_width=4000, table_stride=4000), _attn()
    need = lib.stagq_kv_attention_workspace(A(c), A(s), A(a))
    assert need > 0 and need % 256 == 0
    assert lib.stagq_kv_attention(A(c), A(s), A(a), None, need, None) == EINVAL
    assert lib.stagq_kv_attention(A(c), A(s), A(a), 4096 + 64, need, None) == EALIGN
    assert lib.stagq_kv_attention(A(c), A(s), A(a), 4096, need - 1, None) == ESIZE


@pytest.mark.parametrize("bad,status", [
    (dict(keep=0), EINVAL), (dict(sinks=-1), EINVAL), (dict(recent=-1), EINVAL), (dict(sinks=6, recent=5), EINVAL),
    (dict(max_len=-2), EINVAL), (dict(weights=None), EINVAL), (dict(weights_out=None), EINVAL), (dict(kept=None), EINVAL),
    (dict(out_lengths=None), EINVAL), (dict(kept=4097), EALIGN), (dict(weights=4098), EALIGN),
    (dict(out_stride_head=-1), EINVAL), (dict(out_stride_head=128), EINVAL), (dict(out_table_stride=3), EINVAL), (dict(keep=200, out_table_width=3), ESIZE),
    (dict(out_table=4096), EINVAL)])
def test_refused_eviction(bad, status):
    e = _evict(**bad)
    assert pwo.lib().stagq_kv_evict(A(_cache()), A(_seqs()), A(e), None, 0, None) == status


def test_eviction_in_place_needs_its_workspace():
    lib = pwo.lib()
    c, s, e = _cache(), _seqs(), _evict(out_table=None)
    need = lib.stagq_kv_evict_workspace(A(c), A(s), A(e))
    assert need == 3 * 2 * 1 * (32 * 128 + 256 * 2)
    assert lib.stagq_kv_evict(A(c), A(s), A(e), None, need, None) == EINVAL
    assert lib.stagq_kv_evict(A(c), A(s), A(e), 4096 + 8, need, None) == EALIGN
    assert lib.stagq_kv_evict(A(c), A(s), A(e), 4096, need - 1, None) == ESIZE
    assert lib.stagq_kv_evict_workspace(A(c), A(s), A(_evict())) == 0
    # many slots are selected from in parts, with a workspace of their own
    wide = _seqs(table_width=1000, table_stride=1000)
    e = _evict(weights_stride_seq=1 << 17, weights_stride_head=1 << 16, out_stride_seq=1 << 17, out_stride_head=1 << 16)
    assert lib.stagq_kv_evict_workspace(A(c), A(wide), A(e)) > 0
    assert lib.stagq_kv_evict(A(c), A(wide), A(e), None, 1 << 30, None) == EINVAL


@pytest.mark.parametrize("bad", [dict(stride_seq=0), dict(stride_token=0), dict(stride_head=0), dict(stride_head=120),
                                 dict(stride_token=128), dict(stride_seq=256), dict(stride_seq=1 << 62)])
def test_what_is_written_may_not_overlap_itself(bad):
    lib = pwo.lib()
    c, s = _cache(), _seqs(batch=3)
    f = dict(heads=4, stride_token=512, stride_seq=1024)
    f.update(bad)
    assert lib.stagq_kv_attention(A(c), A(s), A(_attn(out=_tensor(data=8192, **f))), None, 0, None) == EINVAL
    t, far = _tensor(**bad), _tensor(data=1 << 30)
    assert lib.stagq_kv_read(A(c), A(s), None, A(t), A(far), 0, None) == EINVAL
    assert lib.stagq_kv_read(A(c), A(s), None, A(far), A(t), 0, None) == EINVAL
    assert lib.stagq_kv_read(A(c), A(s), None, A(far), A(far), 0, None) == EINVAL


@pytest.mark.parametrize("seq,head", [(0, 256), (512, 0), (512, 255), (511, 256), (256, 256)])
def test_weights_written_may_not_overlap(seq, head):
    lib = pwo.lib()
    c, s = _cache(), _seqs(batch=3)   # 2 heads of up to 256 slots
    assert lib.stagq_kv_attention(A(c), A(s), A(_attn(weights=1 << 20, weights_stride_seq=seq, weights_stride_head=head)),
                                  None, 0, None) == EINVAL
    e = _evict(weights_out=1 << 20, out_stride_seq=seq, out_stride_head=head)
    assert lib.stagq_kv_evict(A(c), A(s), A(e), None, 0, None) == EINVAL


def test_null_structs_and_empty_calls():
    lib = pwo.lib()
    c, s, t = _cache(), _seqs(), _tensor()
    assert lib.stagq_kv_bytes(None) == 0
    for args in ((None, A(s), A(t), A(t)), (A(c), None, A(t), A(t)), (A(c), A(s), None, A(t)), (A(c), A(s), A(t), None)):
        assert lib.stagq_kv_append(*args, None, None) == EINVAL
    assert lib.stagq_kv_attention(A(c), A(s), None, None, 0, None) == EINVAL
    assert lib.stagq_kv_evict(A(c), A(s), None, None, 0, None) == EINVAL
    none = _seqs(batch=0, table=None, lengths=None)
    assert _rows_calls(c, none, _tensor(data=None), _tensor(data=None)) == {0}
    assert _rows_calls(c, s, _tensor(tokens=0, data=None), _tensor(tokens=0, data=None)) == {0}
    assert lib.stagq_kv_attention(A(c), A(none), A(_attn()), None, 0, None) == 0
    assert lib.stagq_kv_evict(A(c), A(none), A(_evict()), None, 0, None) == 0


def test_cache_bytes():
    # 32 tokens x (128 / 2 x 2 bytes of codes + 2 groups x 2 x 4 bytes of pairs) per head
    assert pwo.lib().stagq_kv_bytes(A(_cache(pages=3))) == 3 * 2 * 64 * (128 + 16)
    assert pwo.KVCache(5, 3, 96, page_tokens=32, device="cpu").nbytes == 5 * 3 * 32 * (96 + 24)


# ---------------------------------------------------------- binding refusals --
def _i32(*a):
    return torch.tensor(a, dtype=torch.int32)


def test_binding_refuses_before_any_call():
    c = pwo.KVCache(8, 2, 128, device="cpu")
    assert c.group == 64 and pwo.KVCache(1, 1, 96, device="cpu").group == 32
    with pytest.raises(pwo.StagQError):
        pwo.KVCache(8, 2, 80, device="cpu")
    with pytest.raises(ValueError):
        pwo.KVCache(8, 2, 128, buffer=torch.zeros(16, dtype=torch.uint8))
    table, lengths = torch.zeros(3, 4, dtype=torch.int32), _i32(1, 2, 3)
    k = torch.zeros(3, 1, 2, 128, dtype=torch.float16)
    q = torch.zeros(3, 1, 4, 128, dtype=torch.float16)
    for bad in (dict(table=table.long()), dict(table=table[:2]), dict(table=table.t()), dict(lengths=lengths.long()),
                dict(lengths=lengths[:2]), dict(lengths=_i32(1, 0, 2, 0, 3, 0)[::2]), dict(k=k.double()), dict(k=k[:, :, :1]),
                dict(k=k.transpose(2, 3)), dict(v=k.float()), dict(v=k[:2]), dict(new_lens=lengths.float())):
        a = dict(k=k, v=k, table=table, lengths=lengths)
        a.update(bad)
        with pytest.raises(ValueError):
            c.append(**a)
    with pytest.raises(TypeError):
        c.append(k.numpy(), k, table, lengths)
    w = torch.zeros(3, 2, 256)
    for bad in (dict(q=q.float()), dict(q=q[:, :, :3]), dict(q=q[..., :64]), dict(q_lens=lengths.long()),
                dict(max_len=0), dict(lse=torch.zeros(3, 4)), dict(lse=torch.zeros(3, 1, 8)[..., ::2]),
                dict(weights=w[..., :255]), dict(weights=w.half()), dict(weights=w.transpose(1, 2))):
        a = dict(q=q, table=table, lengths=lengths)
        a.update(bad)
        with pytest.raises(ValueError):
            c.attention(**a)
    for bad in (dict(keep=0), dict(sinks=-1), dict(sinks=8, recent=3), dict(weights=w[..., :100]), dict(weights=w[:2]),
                dict(weights_out=w[..., :100]), dict(out_table=table.long()), dict(out_table=table[:, :0])):
        a = dict(table=table, lengths=lengths, weights=w, keep=10)
        a.update(bad)
        with pytest.raises(ValueError):
            c.evict(**a)
    with pytest.raises(ValueError):
        c.read(table, lengths, start=lengths.long())
