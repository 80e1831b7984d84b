"""The key/value cache in 4 bits on the GPU against its float64 oracle.

Reads are exact: lo + s u rounded once.  Attention is held to a bound per
element, counted from the roundings on its way (h = eps / 2 of the output type,
u16 = 2^-11 the fp16 rounding):
  z     every product goes through the matrix instruction, whose alignment may
        drop 2^-19 of the largest product, and a few binary32 sums: dz <= 2^-17
        Z, Z = scale sum |q| (|lo| + s u) (reach_z).  Where many rows run together
        the keys are first rounded to fp16: dz grows by u16 scale sum |q| |k|
        (keys_z).  A probability is then off by a factor e^(2 dz).
  P V   the products p s are rounded to fp16 (u16 of sum P s u, `code`), or,
        where many rows run together, p and v each (2 u16 of sum P |v|, `size`).
  out   h |out|, and half of the smallest fp16 number.
Every case prints its name before it touches the GPU.
"""
import math

import numpy as np
import pytest

from oracle import kv_oracle

pytestmark = pytest.mark.gpu
U16 = 2.0 ** -11


def _say(*a):
    print("[gpu]", *a, flush=True)


@pytest.fixture(scope="module")
def pwo():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import precision_weight_only_amd as m   # raises if libstagq.so is missing
    return m


def _torch():
    import torch
    return torch


class Case:
    """Sequences in a cache whose unused slots hold arbitrary bits."""

    def __init__(self, pwo, lens, Hkv=2, D=128, g=64, P=64, seed=0, dtype="float16", extra_width=0, scale_v=1.0):
        torch = _torch()
        self.dt = getattr(torch, dtype)
        self.lens, self.Hkv, self.D, self.g, self.P = list(lens), Hkv, D, g, P
        rng = np.random.default_rng([seed, D, g])
        B, L = len(lens), max(max(lens), 1)
        k = rng.standard_normal((B, L, Hkv, D)) * (0.5 + np.abs(rng.standard_normal((Hkv, D)))) + rng.standard_normal((Hkv, D))
        v = rng.standard_normal((B, L, Hkv, D)) * scale_v
        self.k = torch.from_numpy(k).to(self.dt).cuda()
        self.v = torch.from_numpy(v).to(self.dt).cuda()
        need = [-(-n // P) for n in lens]
        width = max(max(need), 1) + extra_width
        perm = rng.permutation(sum(need) + 2)
        table = np.full((B, width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at: at + n]
            at += n
        self.table = torch.from_numpy(table).cuda()
        self.pages = sum(need) + 2
        self.lengths = torch.tensor(list(lens), dtype=torch.int32).cuda()
        nbytes = pwo.KVCache(self.pages, Hkv, D, group=g, page_tokens=P, device="cpu").nbytes
        junk = torch.from_numpy(rng.integers(0, 256, nbytes, dtype=np.uint8))
        junk[::2] = 0xff   # among it NaN and infinities as pairs
        self.cache = pwo.KVCache(self.pages, Hkv, D, group=g, page_tokens=P, buffer=junk.cuda())
        self.rng = rng

    def fill(self):
        self.cache.append(self.k, self.v, self.table, self.lengths, new_lens=self.lengths)
        return self

    def quant(self, b, h):
        f = lambda x: kv_oracle.quantise(x[b, : self.lens[b], h].double().cpu().numpy(), self.g)
        return f(self.k), f(self.v)

    def queries(self, T, Hq, spread=0.6):
        torch = _torch()
        q = self.rng.standard_normal((len(self.lens), T, Hq, self.D)) * spread
        return torch.from_numpy(q).to(self.dt if self.dt != torch.float32 else torch.float16).cuda()


def _np(t):
    return t.double().cpu().numpy()


def check_attention(case, q, out, q_lens=None, scale=None, causal=True, window=0, lse=None, weights=None, before=None,
                    absent=lambda b: ()):
    torch = _torch()
    B, T, Hq, D = q.shape
    gq = Hq // case.Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    h_out = torch.finfo(q.dtype).eps / 2
    out, qn = _np(out), _np(q)
    worst = 0.0
    for b, n in enumerate(case.lens):
        t = T if q_lens is None else q_lens[b]
        for h in range(case.Hkv):
            kq, vq = case.quant(b, h)
            if n == 0:
                assert (out[b, :t, h * gq:(h + 1) * gq] == 0).all()
                if lse is not None:
                    assert (_np(lse)[b, :t, h * gq:(h + 1) * gq] == -np.inf).all()
                continue
            r = kv_oracle.attention(qn[b, :t, h * gq:(h + 1) * gq], kq, vq, scale, causal, window, absent(b))
            dz = 2.0 ** -17 * r["reach_z"] + U16 * r["keys_z"]
            assert (dz < 0.3).all()
            err = np.abs(out[b, :t, h * gq:(h + 1) * gq] - r["out"])
            tol = (h_out * np.abs(r["out"]) + 2.0 ** -25 + U16 * np.maximum(r["code"], 2 * r["size"]) * 1.01
                   + np.expm1(2 * dz)[..., None] * r["size"])
            worst = max(worst, float((err / tol).max()))
            assert (err <= tol).all(), f"seq {b} head {h}: {float((err / tol).max())} of the bound"
            if lse is not None:
                got, want = _np(lse)[b, :t, h * gq:(h + 1) * gq], r["lse"]
                none = want == -np.inf
                assert (got[none] == -np.inf).all()
                assert (np.abs(got[~none] - want[~none]) <= (dz + 2.0 ** -21 * (1 + np.abs(want)))[~none]).all()
            if weights is not None:
                got = _np(weights)[b, h, :n] - 0.0
                base = before[b, h, :n]
                # A weight is exp(z - lse): what lse may be off by in 32 bits, the bound
                # of it above, is an error of the exponent next to z's.  (Where z is
                # exactly 0, scale 0, dz is 0 and this is all that is left: 150 slots,
                # lse 5.01, one step of which is 4.8e-7 of the weight; log2, its
                # product with ln 2 and back are three roundings of that size.)
                seen = np.abs(r["lse"][np.isfinite(r["lse"])])
                off = 2 * (dz.max() if dz.size else 0.0) + 2.0 ** -21 * (1 + (seen.max() if seen.size else 0.0))
                tol_w = np.expm1(off) * r["weights"] + 2.0 ** -20 * (base + r["weights"]) + 1e-30
                assert (np.abs(got - base - r["weights"]) <= tol_w).all()
    _say(f"worst {worst:.3f} of the bound")


# ------------------------------------------------------------ append, read ----
SHAPES = [(64, 64, 32), (64, 32, 64), (96, 32, 64), (128, 128, 256), (128, 64, 64), (128, 32, 128), (256, 128, 64),
          (256, 64, 32), (256, 32, 64)]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("D,g,P", SHAPES)
def test_append_and_read_are_exact(pwo, D, g, P, dtype):
    _say("append", D, g, P, dtype)
    torch = _torch()
    c = Case(pwo, [1, 0, 33, 130, 64], D=D, g=g, P=P, dtype=dtype, Hkv=3).fill()
    k, v = c.cache.read(c.table, c.lengths, tokens=140)
    for b, n in enumerate(c.lens):
        assert (k[b, n:] == 0).all() and (v[b, n:] == 0).all()
        for h in range(3 if n else 0):
            for got, f in zip((k, v), c.quant(b, h)):
                assert np.array_equal(got[b, :n, h].cpu().numpy(), kv_oracle.values(*f).astype(np.float32))
    # the other types, a start, rows left alone
    start = torch.tensor([0, 0, 5, 100, -3], dtype=torch.int32).cuda()
    for dt in (torch.float16, torch.bfloat16):
        a = torch.full((5, 40, 3, D), 7.0, dtype=dt, device="cuda")
        b2 = a.clone()
        c.cache.read(c.table, c.lengths, start=start, k=a, v=b2)
        for b, n in enumerate(c.lens):
            s = int(start[b])
            for i in range(40):
                want = k[b, s + i].to(dt) if 0 <= s + i < n else torch.full_like(a[b, i], 7.0)
                assert torch.equal(a[b, i], want)
                want = v[b, s + i].to(dt) if 0 <= s + i < n else torch.full_like(a[b, i], 7.0)
                assert torch.equal(b2[b, i], want)


def test_append_borders_and_wide_values(pwo):
    """Values on, just below and just above every border, huge and tiny steps, NaN, infinities."""
    _say("append borders")
    torch = _torch()
    rng = np.random.default_rng(5)
    n, D, g = 96, 64, 32
    x = rng.standard_normal((n, 2, g)).astype(np.float16).astype(np.float64)
    x *= (2.0 ** rng.integers(-12, 12, (n, 2)))[..., None]
    x = x.astype(np.float16).astype(np.float32)
    for t in range(n):
        for h in range(2):
            _, lo, s = kv_oracle.quantise(x[t, h], g)
            inner = [i for i in range(g) if x[t, h, i] not in (x[t, h].min(), x[t, h].max())][:12]
            for m, i in enumerate(inner):
                border = np.float32(lo[0] + (m + 0.5) * s[0])   # exact in binary32 where it matters
                x[t, h, i] = [border, np.nextafter(border, np.float32(-1e9)), np.nextafter(border, np.float32(1e9))][(t + m) % 3]
    x[0, 0, 3], x[1, 0, 4], x[2, 0, 5], x[3, 1, 6], x[4, 1, 7] = np.nan, np.inf, -np.inf, 1e30, -1e30
    x[5], x[6, 0], x[7] = 0.0, -3.5, 1e-30
    xs = torch.from_numpy(x.reshape(1, n, 1, D)).cuda()
    cache = pwo.KVCache(4, 1, D, group=g, page_tokens=32)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32).cuda()
    lengths = torch.tensor([n], dtype=torch.int32).cuda()
    cache.append(xs, -xs, table, lengths)
    k, v = cache.read(table, lengths, tokens=n)
    for got, y in ((k, x), (v, -x)):
        want = kv_oracle.values(*kv_oracle.quantise(y.reshape(n, D), g)).astype(np.float32)
        assert np.array_equal(got[0, :, 0].cpu().numpy(), want)
        assert np.isfinite(want).all()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_append_token_by_token_equals_all_at_once(pwo, dtype):
    """Steps of 1, 3, 31, 32 and 33 tokens give the same bytes as one call; strided rows, slots before and
    after the step keep what they hold, also where a step starts before slot 0 or has no page."""
    _say("append steps", dtype)
    torch = _torch()
    c = Case(pwo, [100, 70], D=128, g=64, P=32, dtype=dtype, Hkv=2)
    one = c.cache.buffer.clone()
    c.fill()
    other = pwo.KVCache(c.pages, 2, 128, group=64, page_tokens=32, buffer=one)
    fused = torch.stack([c.k, c.v], 2)   # rows of k and v side by side
    done = [0, 0]
    for step in (1, 3, 31, 32, 33, 1):
        now = [min(d + step, n) for d, n in zip(done, c.lens)]
        new = [a - d for a, d in zip(now, done)]
        rows = torch.full((2, step + 2, 2, 2, 128), float("nan"), dtype=c.dt, device="cuda")
        for b in range(2):
            rows[b, : new[b]] = fused[b, done[b]: now[b]]
        i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
        other.append(rows[:, :, 0], rows[:, :, 1], c.table, i32(now), new_lens=i32(new))
        done = now
    assert done == c.lens
    ka, va = c.cache.read(c.table, c.lengths)
    kb, vb = other.read(c.table, c.lengths)
    assert torch.equal(ka, kb) and torch.equal(va, vb)
    keep = other.buffer.clone()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32).cuda()
    other.append(c.k, c.v, c.table, i32([0, -5]), new_lens=i32([40, 40]))       # before slot 0
    other.append(c.k, c.v, c.table, c.lengths, new_lens=i32([0, -3]))           # nothing
    bad = c.table.clone()
    bad[0], bad[1] = -1, 1 << 30
    other.append(c.k, c.v, bad, c.lengths, new_lens=c.lengths)                  # no pages
    other.append(c.k, c.v, c.table, i32([2000000000, 2000000000]))              # past the table
    assert torch.equal(other.buffer, keep)
    k, v = other.read(bad, c.lengths, tokens=100)
    assert (k == 0).all() and (v == 0).all()


# -------------------------------------------------------------- attention ----
DECODE = [
    # D, g, P, Hkv, gq, lens, dtype, window
    (64, 64, 32, 2, 1, [1, 5, 64, 131], "float16", 0),
    (64, 32, 64, 1, 7, [0, 31, 32, 33], "bfloat16", 0),
    (96, 32, 128, 3, 4, [200, 1, 77], "float16", 50),
    (128, 64, 64, 2, 4, [1000, 3, 0, 517], "float16", 0),
    (128, 128, 256, 2, 8, [300, 700], "bfloat16", 0),
    (128, 32, 32, 1, 16, [650], "float16", 64),
    (128, 64, 64, 1, 24, [333, 40], "float16", 0),
    (128, 64, 64, 1, 48, [90, 257], "bfloat16", 33),
    (256, 128, 64, 2, 2, [129, 600], "float16", 0),
    (256, 64, 32, 1, 20, [65], "bfloat16", 0),
    (256, 32, 64, 1, 3, [400, 2], "float16", 1),
]


@pytest.mark.parametrize("D,g,P,Hkv,gq,lens,dtype,window", DECODE)
def test_one_token(pwo, D, g, P, Hkv, gq, lens, dtype, window):
    _say("one token", D, g, P, Hkv, gq, lens, dtype, window)
    torch = _torch()
    c = Case(pwo, lens, Hkv, D, g, P, dtype=dtype, extra_width=3).fill()
    q = c.queries(1, Hkv * gq)
    lse = torch.full(q.shape[:3], 5.0, device="cuda")
    w = torch.rand(len(lens), Hkv, c.table.shape[1] * P, device="cuda")
    before = _np(w)
    out = c.cache.attention(q, c.table, c.lengths, window=window, lse=lse, weights=w)
    check_attention(c, q, out, window=window, lse=lse, weights=w, before=before)
    for b, n in enumerate(lens):
        assert np.array_equal(_np(w)[b, :, n:], before[b, :, n:])
    again = c.cache.attention(q, c.table, c.lengths, window=window, max_len=max(lens))
    check_attention(c, q, again, window=window)


LONG = [
    # rows of few heads, sequences long enough for the grid to share their steps
    # D, g, P, Hkv, gq, T, lens, dtype, window
    (128, 64, 64, 2, 4, 1, [2100, 0, 1, 1500], "float16", 0),
    (128, 128, 32, 1, 2, 2, [3000, 40], "bfloat16", 0),
    (64, 64, 256, 3, 1, 4, [1100, 1030, 64], "float16", 0),
    (256, 128, 64, 1, 3, 1, [1500, 2], "float16", 0),
    (256, 64, 32, 2, 1, 3, [1200], "bfloat16", 1100),
    (128, 64, 64, 1, 4, 1, [5000, 300], "float16", 2000),
    (64, 64, 32, 1, 1, 1, [70 * i % 1300 for i in range(70)], "float16", 0),          # more sequences than lanes
    (128, 64, 64, 8, 1, 1, [1100] + [1] * 130, "bfloat16", 0),                         # most at their first token
    (64, 64, 64, 8, 2, 2, [1300, 0] + [3] * 20, "float16", 0),                         # items enough for one workgroup each
    (256, 128, 64, 8, 4, 1, [1300, 0, 1290] + [2] * 20, "bfloat16", 0),
    (128, 64, 32, 4, 1, 1, [9000] + [40 * i for i in range(3)], "float16", 0),
]


@pytest.mark.parametrize("D,g,P,Hkv,gq,T,lens,dtype,window", LONG)
def test_few_rows_of_long_sequences(pwo, D, g, P, Hkv, gq, T, lens, dtype, window):
    _say("few rows, long", D, g, P, Hkv, gq, T, lens[:4], dtype, window)
    torch = _torch()
    c = Case(pwo, lens, Hkv, D, g, P, dtype=dtype, seed=14, extra_width=1).fill()
    q = c.queries(T, Hkv * gq)
    ql = [min(T, n) for n in lens]
    lse = torch.full(q.shape[:3], 5.0, device="cuda")
    w = torch.rand(len(lens), Hkv, c.table.shape[1] * P, device="cuda")
    before = _np(w)
    out = c.cache.attention(q, c.table, c.lengths, q_lens=torch.tensor(ql, dtype=torch.int32).cuda(), window=window, lse=lse,
                            weights=w)
    check_attention(c, q, out, q_lens=ql, window=window, lse=lse, weights=w, before=before)
    for b, n in enumerate(lens):
        assert (out[b, ql[b]:] == 0).all() and (lse[b, ql[b]:] == 5.0).all()
        assert np.array_equal(_np(w)[b, :, n:], before[b, :, n:])


def test_a_refused_call_leaves_nothing_behind(pwo):
    """The same call with an argument put right works (its workspace is not that of the refused one)."""
    _say("refused, then right")
    torch = _torch()
    c = Case(pwo, [1500, 1300], 2, 128, 64, 64, seed=17).fill()
    q = c.queries(1, 4)
    for bad in (dict(scale=math.inf), dict(out=q), dict(window=5, causal=False)):
        with pytest.raises(pwo.StagQError):
            c.cache.attention(q, c.table, c.lengths, **bad)
    with pytest.raises(ValueError):
        c.cache.attention(q, c.table, c.lengths, window=-1)
    with pytest.raises(pwo.StagQError):
        c.cache.attention(q, c.table, c.lengths, out=torch.zeros_like(q[:1]).expand(2, -1, -1, -1))
    check_attention(c, q, c.cache.attention(q, c.table, c.lengths))
    check_attention(c, q, c.cache.attention(q, c.table, c.lengths, window=5), window=5)


def test_no_pages(pwo):
    """A table of width 0, and a cache of no pages."""
    _say("no pages")
    torch = _torch()
    c = Case(pwo, [5, 0], 2, 64, 64, 32, seed=18)
    kv = torch.zeros(2, 1, 2, 64, dtype=c.dt, device="cuda")
    for cache, table in ((c.cache, c.table[:, :0]), (pwo.KVCache(0, 2, 64, page_tokens=32), c.table)):
        for T in (1, 5, 40):
            q = c.queries(T, 4)
            lse = torch.zeros(q.shape[:3], device="cuda")
            w = torch.ones(2, 2, table.shape[1] * 32, device="cuda")
            cache.append(kv, kv, table, c.lengths)
            out = cache.attention(q, table, c.lengths, lse=lse, weights=w)
            assert (out == 0).all() and (lse == -math.inf).all() and (w == 1).all()
        k, v = cache.read(table, c.lengths, tokens=3)
        assert (k == 0).all() and (v == 0).all()
    kept, n = c.cache.evict(c.table[:, :0], c.lengths, torch.ones(2, 2, 0, device="cuda"), keep=3)
    assert (kept == -1).all() and (n == 0).all()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("D,g,T,gq", [(64, 64, 40, 2), (96, 32, 9, 2), (128, 128, 29, 4), (128, 64, 1, 3), (256, 32, 20, 4)])
@pytest.mark.parametrize("window", [1, 2])
def test_lse_of_rows_that_see_one_or_two_slots(pwo, D, g, T, gq, window, dtype):
    """lse holds 32 bits also where nothing averages out: z is off by 2^-22 of its terms (products of 22-bit parts, sums
    in binary32), and e^z sums in binary32 (2^-22 with the logarithm and its scales)."""
    _say("lse", D, g, T, gq, window, dtype)
    torch = _torch()
    c = Case(pwo, [200], 1, D, g, 64, dtype=dtype, seed=24).fill()
    q = c.queries(T, gq)
    lse = torch.zeros(q.shape[:3], device="cuda")
    c.cache.attention(q, c.table, c.lengths, window=window, lse=lse)
    r = kv_oracle.attention(_np(q)[0], *c.quant(0, 0), 1 / math.sqrt(D), True, window)
    assert (np.abs(_np(lse)[0] - r["lse"]) <= 2.0 ** -22 * (2 + np.abs(r["lse"]) + r["reach_z"])).all()


@pytest.mark.parametrize("lens", [[9000, 300, 8500], [17000, 300, 16500]])
def test_eviction_of_many_slots_into_its_own_lengths(pwo, lens):
    """out_lengths may be lengths itself, also where the selection takes several launches."""
    _say("own lengths")
    torch = _torch()
    c = Case(pwo, lens, 1, 64, 64, 128, seed=19).fill()
    w = torch.rand(3, 1, c.table.shape[1] * 128, device="cuda")
    cache2 = pwo.KVCache(c.pages, 1, 64, page_tokens=128, buffer=c.cache.buffer.clone())
    w2, l2 = w.clone(), c.lengths.clone()
    kept, n = c.cache.evict(c.table, c.lengths, w, keep=400, sinks=4, recent=100)
    kept2, n2 = cache2.evict(c.table, l2, w2, keep=400, sinks=4, recent=100, out_lengths=l2)
    assert n2 is l2 and n.tolist() == [400, 300, 400] and torch.equal(n, l2)
    assert torch.equal(kept, kept2) and torch.equal(w, w2)
    assert all(torch.equal(a, b) for a, b in zip(c.cache.read(c.table, n), cache2.read(c.table, n)))


@pytest.mark.parametrize("T", [1, 3, 40])
@pytest.mark.parametrize("scale", [-0.09, 0.0])
def test_other_scales(pwo, T, scale):
    """A negative scale turns the order of the scores; 0 gives the mean of what is seen."""
    _say("scale", T, scale)
    torch = _torch()
    c = Case(pwo, [150, 20], 1, 128, 64, 64, seed=15).fill()
    q = c.queries(T, 4)
    lse = torch.zeros(q.shape[:3], device="cuda")
    w = torch.zeros(2, 1, c.table.shape[1] * 64, device="cuda")
    out = c.cache.attention(q, c.table, c.lengths, scale=scale, lse=lse, weights=w)
    check_attention(c, q, out, scale=scale, lse=lse, weights=w, before=np.zeros(w.shape))


def test_split_chunk_of_a_long_sequence(pwo):
    """Rows enough for the tiles, slots enough for their splits to be joined."""
    _say("split chunk")
    torch = _torch()
    c = Case(pwo, [3000], 1, 128, 64, 64, seed=16).fill()
    q = c.queries(12, 4)
    lse = torch.zeros(q.shape[:3], device="cuda")
    w = torch.zeros(1, 1, c.table.shape[1] * 64, device="cuda")
    out = c.cache.attention(q, c.table, c.lengths, lse=lse, weights=w)
    check_attention(c, q, out, lse=lse, weights=w, before=np.zeros(w.shape))


MANY = [
    (64, 32, 32, 2, 2, [70, 9], 6, None, "float16", True, 0),
    (64, 64, 64, 1, 1, [300], 300, None, "bfloat16", True, 0),
    (96, 32, 64, 1, 3, [150, 20], 40, [40, 11], "float16", True, 0),
    (128, 64, 64, 2, 4, [200, 90, 0], 70, [70, 33, 0], "float16", True, 0),
    (128, 64, 32, 1, 4, [260], 131, None, "bfloat16", True, 40),
    (128, 128, 128, 2, 1, [129, 64], 64, None, "float16", False, 0),
    (128, 32, 64, 1, 5, [100], 100, None, "float16", True, 1),
    (128, 64, 64, 1, 4, [20, 50], 60, None, "float16", True, 0),     # more rows than tokens: empty rows
    (128, 64, 64, 1, 2, [700], 17, None, "float16", True, 0),
    (256, 64, 32, 1, 2, [140], 70, None, "bfloat16", True, 0),
    (256, 32, 64, 1, 1, [200], 33, None, "float16", False, 0),
    (256, 128, 64, 1, 3, [95], 95, [80], "float16", True, 30),
]


@pytest.mark.parametrize("D,g,P,Hkv,gq,lens,T,q_lens,dtype,causal,window", MANY)
def test_many_rows(pwo, D, g, P, Hkv, gq, lens, T, q_lens, dtype, causal, window):
    _say("many rows", D, g, P, Hkv, gq, lens, T, q_lens, dtype, causal, window)
    torch = _torch()
    c = Case(pwo, lens, Hkv, D, g, P, dtype=dtype, seed=3).fill()
    # q a slice of a wider row, with rows past q_lens that must not be read
    wide = torch.full((len(lens), T, Hkv * gq + 2 * Hkv, D), float("nan"), dtype=c.dt, device="cuda")
    wide[:, :, : Hkv * gq] = c.queries(T, Hkv * gq)
    q = wide[:, :, : Hkv * gq]
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32).cuda()
    lse = torch.full(q.shape[:3], 5.0, device="cuda")
    w = torch.zeros(len(lens), Hkv, c.table.shape[1] * P, device="cuda")
    before = _np(w)
    out = torch.full_like(wide, 9.0)[:, :, : Hkv * gq]
    got = c.cache.attention(q, c.table, c.lengths, q_lens=ql, causal=causal, window=window, out=out, lse=lse, weights=w)
    assert got is out
    check_attention(c, q, out, q_lens=q_lens, causal=causal, window=window, lse=lse, weights=w, before=before)
    for b in range(len(lens)):
        t = T if q_lens is None else q_lens[b]
        assert (out[b, t:] == 9.0).all() and (lse[b, t:] == 5.0).all()
        assert (_np(w)[b, :, lens[b]:] == 0).all()
    if ql is not None:
        mine = c.cache.attention(q, c.table, c.lengths, q_lens=ql, causal=causal, window=window)
        for b in range(len(lens)):
            assert torch.equal(mine[b, : q_lens[b]], out[b, : q_lens[b]]) and (mine[b, q_lens[b]:] == 0).all()


@pytest.mark.parametrize("T", [1, 5, 80])
def test_missing_pages_are_masked(pwo, T):
    _say("missing pages", T)
    torch = _torch()
    c = Case(pwo, [300, 90], 2, 128, 64, 32, seed=8).fill()
    c.table[0, 2] = -1
    c.table[0, 5] = c.pages
    c.table[1, :] = -(1 << 31)
    gone = [[s for s in range(300) if s // 32 in (2, 5)], list(range(90))]
    q = c.queries(T, 8)
    lse = torch.zeros(q.shape[:3], device="cuda")
    w = torch.zeros(2, 2, c.table.shape[1] * 32, device="cuda")
    out = c.cache.attention(q, c.table, c.lengths, lse=lse, weights=w)
    check_attention(c, q, out, lse=lse, weights=w, before=np.zeros(w.shape), absent=lambda b: gone[b])


@pytest.mark.parametrize("scale_v", [2.0 ** -9, 300.0])
@pytest.mark.parametrize("T", [1, 90])
def test_value_scales_and_a_dominant_token(pwo, T, scale_v):
    """Small and large V, and one token that outweighs the others by far: the bound is relative to what counts."""
    _say("value scales", T, scale_v)
    torch = _torch()
    c = Case(pwo, [900], 1, 128, 64, 64, seed=4, scale_v=scale_v)
    q = c.queries(T, 4)
    c.k[0, 0, 0] = (q[0, 0, 0].float() * 2.5).to(c.dt)
    c.fill()
    out = c.cache.attention(q, c.table, c.lengths)
    check_attention(c, q, out)


def test_query_extremes(pwo):
    """Rows of zeros, tiny and large magnitudes: every row is scaled by itself; an infinity stays in its row."""
    _say("query extremes")
    torch = _torch()
    for dtype in ("float16", "bfloat16"):
        c = Case(pwo, [100], 1, 128, 64, 64, seed=6, dtype=dtype).fill()
        q = c.queries(1, 8)
        q[0, 0, 0] = 0
        q[0, 0, 1] *= 2.0 ** -12
        q[0, 0, 2] = 0
        q[0, 0, 2, 5] = 30.0
        out = c.cache.attention(q, c.table, c.lengths)
        check_attention(c, q, out)
        bad = q.clone()
        bad[0, 0, 3, 7] = float("inf")
        got = c.cache.attention(bad, c.table, c.lengths)
        rest = [0, 1, 2, 4, 5, 6, 7]
        assert torch.equal(got[0, 0, rest], out[0, 0, rest])


def test_max_len_cuts_and_lengths_are_clamped(pwo):
    _say("max_len")
    torch = _torch()
    c = Case(pwo, [200], 1, 64, 32, 32, seed=9).fill()
    q = c.queries(1, 2)
    cut = Case(pwo, [200], 1, 64, 32, 32, seed=9).fill()
    cut.lens = [96]
    out = c.cache.attention(q, c.table, c.lengths, max_len=96)
    check_attention(cut, q, out)
    out = c.cache.attention(q, c.table, torch.tensor([-7], dtype=torch.int32).cuda())
    assert (out == 0).all()
    out = c.cache.attention(q, c.table, torch.tensor([2000000000], dtype=torch.int32).cuda(), max_len=200)
    check_attention(c, q, out)


# ---------------------------------------------------------------- eviction ----
def check_evict(c, w, keep, sinks, recent, kept, lengths, wout, read):
    for b, n in enumerate(c.lens):
        assert int(lengths[b]) == min(n, keep)
        for h in range(c.Hkv):
            want = kv_oracle.evict(w[b, h, :n], keep, sinks, recent)
            m = len(want)
            got = kept[b, h].cpu().numpy()
            assert np.array_equal(got[:m], want) and (got[m:] == -1).all()
            assert np.array_equal(wout[b, h, :m].cpu().numpy(), w[b, h, want])
            assert (wout[b, h, m:] == 0).all()
            if m == 0:
                continue
            for x, f in zip(read, c.quant(b, h)):
                assert np.array_equal(x[b, :m, h].cpu().numpy(), kv_oracle.values(*f).astype(np.float32)[want])


EVICT = [
    (64, 32, 32, [100, 33, 0, 5], 33, 4, 10), (128, 64, 64, [1500, 700], 400, 0, 0), (128, 64, 64, [2500], 1, 0, 0),
    (128, 128, 64, [200, 90], 64, 4, 60), (96, 32, 128, [300], 299, 0, 299), (256, 64, 32, [130, 131], 65, 65, 0),
    (256, 32, 256, [600], 128, 1, 3), (64, 64, 64, [5000], 1100, 3, 200),
    # more slots than one workgroup selects from
    (64, 64, 64, [8500, 0, 30, 12289], 5000, 4, 300), (64, 64, 256, [20000, 9000], 9500, 0, 0), (64, 64, 64, [9000], 40, 30, 10),
    (64, 64, 64, [8300], 10000, 1, 1),
    (64, 64, 64, [16500, 0, 30, 24577], 5000, 4, 300), (64, 64, 64, [17000], 40, 30, 10), (64, 64, 64, [16400], 18000, 1, 1),
    (64, 64, 64, [16384, 4096, 4097], 700, 3, 5),
]


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("D,g,P,lens,keep,sinks,recent", EVICT)
def test_evict(pwo, D, g, P, lens, keep, sinks, recent, inplace):
    _say("evict", D, g, P, lens, keep, sinks, recent, inplace)
    torch = _torch()
    c = Case(pwo, lens, 2, D, g, P, seed=7).fill()
    B, W = c.table.shape
    w = c.rng.choice([0.0, -0.0, 0.5, 0.5, 1.5, 2.0 ** -140, 7.0, -2.0], (B, 2, W * P))
    w[:, :, ::3] = c.rng.standard_normal(w[:, :, ::3].shape) ** 2
    w = w.astype(np.float32)
    wt = torch.from_numpy(w).cuda()
    if inplace:
        kept, lengths = c.cache.evict(c.table, c.lengths, wt, keep, sinks=sinks, recent=recent, out_lengths=c.lengths)
        assert lengths is c.lengths
        wout, table, cache = wt, c.table, c.cache
    else:
        per = -(-keep // P)
        big = pwo.KVCache(c.pages + B * per, 2, D, group=g, page_tokens=P)
        big.buffer[: c.cache.nbytes] = c.cache.buffer
        table = (torch.arange(B * per, dtype=torch.int32, device="cuda").flip(0).view(B, per) + c.pages).contiguous()
        wout = torch.full_like(wt, 3.0)
        kept, lengths = big.evict(c.table, c.lengths, wt, keep, sinks=sinks, recent=recent, out_table=table, weights_out=wout)
        cache = big
        assert torch.equal(big.buffer[: c.cache.nbytes], c.cache.buffer) and np.array_equal(wt.cpu().numpy(), w)
    read = cache.read(table, lengths, tokens=keep)
    check_evict(c, w, keep, sinks, recent, kept, lengths, wout, read)


@pytest.mark.parametrize("n", [400, 9000, 17000])
def test_evict_nan_infinity_and_all_equal(pwo, n):
    _say("evict extremes", n)
    torch = _torch()
    c = Case(pwo, [n], 1, 64, 64, 32, seed=2).fill()
    i = np.arange(c.table.shape[1] * 32)
    for w in (0.0 * i, np.full(i.shape, np.inf), np.where(i % 7 == 0, np.nan, 1.0), np.where(i % 5 == 0, -np.inf, 0.0)):
        w = w.astype(np.float32)[None, None]
        wt = torch.from_numpy(w.copy()).cuda()
        kept, _ = c.cache.evict(c.table, c.lengths, wt, 100, sinks=2, recent=9, weights_out=torch.empty_like(wt),
                                out_table=torch.full((1, 4), -1, dtype=torch.int32, device="cuda"))   # no page: nothing moves
        assert np.array_equal(kept[0, 0].cpu().numpy(), kv_oracle.evict(w[0, 0, :n], 100, 2, 9))


# ------------------------------------------------------- together, captured ----
def test_a_run_together(pwo):
    """A prompt, decode steps that accumulate weights, an eviction, more steps: every output against the oracle run
    on the values as they were fed in."""
    _say("run together")
    torch = _torch()
    c = Case(pwo, [90, 57], 2, 128, 64, 32, seed=11, extra_width=2).fill()
    q0 = c.queries(90, 8)
    ql = c.lengths.clone()
    w = torch.zeros(2, 2, c.table.shape[1] * 32, device="cuda")
    out = c.cache.attention(q0, c.table, c.lengths, q_lens=ql, weights=w)
    check_attention(c, q0, out, q_lens=c.lens, weights=w, before=np.zeros(w.shape))
    keep = 40
    before = w.cpu().numpy()
    kept, lengths = c.cache.evict(c.table, c.lengths, w, keep, sinks=2, recent=8, out_lengths=c.lengths)
    read = c.cache.read(c.table, lengths, tokens=keep)
    check_evict(c, before, keep, 2, 8, kept, lengths, w, read)
    # from here on every kv head has its own past
    past = [[[x[b, kept[b, h].long(), h] for x in (c.k, c.v)] for h in range(2)] for b in range(2)]
    for step in range(3):
        rows = [torch.from_numpy(c.rng.standard_normal((2, 1, 2, 128))).to(c.dt).cuda() for _ in range(2)]
        lengths += 1
        c.cache.append(rows[0], rows[1], c.table, lengths)
        q = c.queries(1, 8)
        got = c.cache.attention(q, c.table, lengths, weights=w)
        for b in range(2):
            for h in range(2):
                past[b][h] = [torch.cat([p, r[b, :, h]]) for p, r in zip(past[b][h], rows)]
                one = Case.__new__(Case)
                one.lens, one.Hkv, one.D, one.g, one.dt = [keep + step + 1], 1, 128, 64, c.dt
                one.k, one.v = (x[None, :, None] for x in past[b][h])
                check_attention(one, q[b:b + 1, :, h * 4:h * 4 + 4], got[b:b + 1, :, h * 4:h * 4 + 4])


def test_captured_steps_replay(pwo):
    """Append and attention (long enough for a join, with weights) captured in one graph and replayed, with eager work
    between the replays: equal to the eager loop, bit for bit."""
    _say("captured")
    torch = _torch()
    lens = [2000, 37]
    runs = []
    for captured in (False, True):
        c = Case(pwo, [n + 8 for n in lens], 2, 128, 64, 64, seed=13)
        c.cache.buffer.zero_()
        lengths = torch.tensor(lens, dtype=torch.int32).cuda()
        c.cache.append(c.k[:, :2000], c.v[:, :2000], c.table, lengths, new_lens=lengths)
        w = torch.zeros(2, 2, c.table.shape[1] * 64, device="cuda")
        k, v = c.k[:, :1].clone(), c.v[:, :1].clone()
        q = c.queries(1, 8)
        out = torch.empty_like(q)

        def step():
            lengths.add_(1)
            c.cache.append(k, v, c.table, lengths)
            c.cache.attention(q, c.table, lengths, out=out, weights=w)

        graph = None
        if captured:
            keep = (lengths.clone(), w.clone(), c.cache.buffer.clone())
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            lengths.copy_(keep[0]); w.copy_(keep[1]); c.cache.buffer.copy_(keep[2])
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        outs = []
        for i in range(5):
            k.copy_(c.k[:, i:i + 1] * 0.5)
            v.copy_(c.v[:, i:i + 1] * 0.5)
            q.mul_(1.01)
            graph.replay() if captured else step()
            torch.cuda.synchronize()
            _ = c.cache.attention(q, c.table, lengths)   # eager work between the replays
            outs.append(out.clone())
        runs.append((outs, w.clone(), lengths.clone(), c.cache.buffer.clone()))
    a, b = runs
    assert all(torch.equal(x, y) for x, y in zip(a[0], b[0]))
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])


@pytest.mark.parametrize("lens,keep", [([300, 41], 90), ([9000, 100], 500), ([17000, 100], 500)])
def test_captured_chunk_and_eviction_replay(pwo, lens, keep):
    """A chunk appended, attended to with weights and evicted in place, with the lengths updated in place, captured in
    one graph: every replay equals the eager calls, bit for bit."""
    _say("captured chunk", lens)
    torch = _torch()
    c = Case(pwo, lens, 2, 64, 64, 64, seed=21, extra_width=1)
    c.cache.buffer.zero_()
    k, v, q, start = c.k[:, :40].clone(), c.v[:, :40].clone(), c.queries(40, 4), c.lengths.clone()
    new = torch.tensor([40, 9], dtype=torch.int32).cuda()
    w = torch.rand(2, 2, c.table.shape[1] * 64, device="cuda")
    out, lse = torch.empty_like(q), torch.zeros(q.shape[:3], device="cuda")
    kept = torch.empty(2, 2, keep, dtype=torch.int32, device="cuda")
    c.fill()
    state = [t.clone() for t in (c.cache.buffer, c.lengths, w)]

    def step():
        c.cache.append(k, v, c.table, c.lengths, new_lens=new)
        c.cache.attention(q, c.table, c.lengths, q_lens=new, out=out, lse=lse, weights=w)
        c.cache.evict(c.table, c.lengths, w, keep=keep, sinks=4, recent=16, kept=kept, out_lengths=c.lengths)

    def reset(i):
        for t, s in zip((c.cache.buffer, c.lengths, w), state):
            t.copy_(s)
        k.copy_(c.k[:, :40] * (0.5 + i))
        q.mul_(1.01)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for t in (c.cache.buffer, c.lengths, w, out, lse, kept)]

    q0, runs, graph = q.clone(), [], None
    for captured in (False, True):
        q.copy_(q0), out.zero_(), lse.zero_(), reset(0)
        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            q.copy_(q0), out.zero_(), lse.zero_(), reset(0)
        for i in range(4):
            reset(i)
            graph.replay() if captured else step()
            runs.append(results())
            _ = c.cache.attention(q, c.table, c.lengths)
    for a, b in zip(runs[:4], runs[4:]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T", [1, 6, 40])
def test_a_row_that_is_not_finite_stays_alone(pwo, T):
    """NaN or an infinity in a row of q: that row is NaN, the others are what they are without it."""
    _say("NaN row", T)
    torch = _torch()
    c = Case(pwo, [200, 1200], 1, 128, 64, 64, seed=22).fill()
    q = c.queries(T, 3)
    clean = c.cache.attention(q, c.table, c.lengths)
    bad = q.clone()
    bad[0, 0, 1, 5] = math.nan
    bad[1, T - 1, 2, 7] = math.inf
    out = c.cache.attention(bad, c.table, c.lengths)
    hit = torch.zeros(q.shape[:3], dtype=torch.bool, device="cuda")
    hit[0, 0, 1] = hit[1, T - 1, 2] = True
    assert out[hit].isnan().all()
    # the reference that exponents are taken from may move at another slot: one more rounding of each p, and of out
    assert (out[~hit].double() - clean[~hit].double()).abs().max() <= 2.0 ** -9 * float(clean.abs().max())


def test_every_call_on_a_given_stream(pwo):
    _say("given stream")
    torch = _torch()
    side = torch.cuda.Stream()
    res = []
    for stream in (None, side):
        c = Case(pwo, [150, 70], 2, 64, 64, 32, seed=23)
        c.cache.buffer.zero_()
        w = torch.zeros(2, 2, c.table.shape[1] * 32, device="cuda")
        q = c.queries(2, 4)
        torch.cuda.synchronize()
        c.cache.append(c.k, c.v, c.table, c.lengths, new_lens=c.lengths, stream=stream)
        out = c.cache.attention(q, c.table, c.lengths, weights=w, stream=stream)
        kept, n = c.cache.evict(c.table, c.lengths, w, keep=50, stream=stream)
        k, v = c.cache.read(c.table, n, tokens=50, stream=stream)
        side.synchronize()
        torch.cuda.synchronize()
        res.append((out, kept, n, k, v, w))
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_two_streams_at_once(pwo):
    """Calls on two streams (each with its own workspace) give what they give alone."""
    _say("two streams")
    torch = _torch()
    cs = [Case(pwo, [3001], 2, 128, 64, 64, seed=20 + i).fill() for i in range(2)]
    qs = [c.queries(1, 8) for c in cs]
    alone = [c.cache.attention(q, c.table, c.lengths) for c, q in zip(cs, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[], []]
    for _ in range(4):
        for i in (0, 1):
            got[i].append(cs[i].cache.attention(qs[i], cs[i].table, cs[i].lengths, stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(g, alone[i]) for g in got[i])


def test_offsets_past_32_bits(pwo):
    """Pages that begin past 4 GiB of the buffer."""
    _say("far pages")
    torch = _torch()
    page = 8 * 64 * (128 + 16)
    pages = (1 << 32) // page + 40
    cache = pwo.KVCache(pages, 8, 128, buffer=torch.empty(pages * page, dtype=torch.uint8, device="cuda"))
    c = Case(pwo, [150], 8, 128, 64, 64, seed=1)
    c.table = torch.tensor([[pages - 1, 3, pages - 20]], dtype=torch.int32).cuda()
    c.cache = cache
    c.fill()
    q = c.queries(1, 32)
    check_attention(c, q, cache.attention(q, c.table, c.lengths))
    k, v = cache.read(c.table, c.lengths, tokens=150)
    for h in (0, 7):
        for got, f in zip((k, v), c.quant(0, h)):
            assert np.array_equal(got[0, :, h].cpu().numpy(), kv_oracle.values(*f).astype(np.float32))
