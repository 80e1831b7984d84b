// The key/value cache in 4 bits: quantising new tokens into the pages, and
// reading the values back.
//
// One workgroup takes one block (32 tokens) of one kv head (a single token: one
// wave).  The kernels move each value once; V, whose codes lie eight tokens to
// a dword, is turned in LDS.
#include "stagq_kv_host.h"

namespace stagq {
namespace kv {

constexpr int kRowThreads = 256;

// x >= lo + b, exactly: t + err is x - lo without rounding, and since t is
// x - lo rounded to nearest and b (a multiple of s / 2 with 5 + 11 bits) is a
// binary32 number, only t == b needs the remainder.
__device__ __forceinline__ bool reaches(float t, float err, float b) { return t > b || (t == b && err >= 0.0f); }

// Code of one value: the nearest by a division, then its two borders exactly.
__device__ __forceinline__ uint32_t code_of(float x, float lo, float s, float r) {
  const float t = x - lo, bb = t - x;
  const float err = (x - (t - bb)) + (-lo - bb);
  float u = floorf(fminf(fmaxf(fmaf(t, r, 0.5f), 0.0f), 15.0f));
  if (u < 15.0f && reaches(t, err, (u + 0.5f) * s)) u += 1.0f;
  else if (u > 0.0f && !reaches(t, err, (u - 0.5f) * s)) u -= 1.0f;
  return uint32_t(u);
}

// Eight neighbouring channels of one token: codes (one per element of u) and
// the group's pair lo | s << 16.  LANES = group / 8 neighbouring lanes hold a
// group.  The quotient is off by less than 2^-18 (t and 1 / s each to 2^-23, at
// most 15.5 of it, and the sum's rounding), so only values within 2^-17 of a
// border need the exact comparison; a wave takes it if any of its lanes does
// (under 1 % of the time; it costs as much as all the rest).
template <int LANES>
__device__ __forceinline__ uint32_t quantise8(float* f, uint32_t* u) {
  float mn = kClamp, mx = -kClamp;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    f[i] = f[i] != f[i] ? 0.0f : fminf(fmaxf(f[i], -kClamp), kClamp);
    mn = fminf(mn, f[i]);
    mx = fmaxf(mx, f[i]);
  }
#pragma unroll
  for (int d = 1; d < LANES; d *= 2) {
    mn = fminf(mn, __shfl_xor(mn, d));
    mx = fmaxf(mx, __shfl_xor(mx, d));
  }
  const _Float16 lo16 = (_Float16)mn;
  const float step = (mx - mn) / 15.0f;
  const _Float16 s16 = (_Float16)step;
  const float lo = (float)lo16, s = (float)s16;
  const float r = s > 0.0f ? __builtin_amdgcn_rcpf(s) : 0.0f;   // s = 0: code 0
  bool near = false;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float q = fmaf(f[i] - lo, r, 0.5f);
    near |= fabsf(q - rintf(q)) < 7.62939453125e-6f;
    u[i] = uint32_t(fminf(fmaxf(q, 0.0f), 15.0f));
  }
  if (__any(near)) {
#pragma unroll
    for (int i = 0; i < 8; i++) u[i] = s > 0.0f ? code_of(f[i], lo, s, r) : 0u;
  }
  return bits_half(lo16) | (bits_half(s16) << 16);
}

__device__ __forceinline__ uint32_t pack_codes(const uint32_t* u) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; e++) w |= u[e] << (4 * nibble(e));
  return w;
}

struct RowsParams {
  Cache c;
  Tensor k, v;
  const int* counts;  // append: new_lens; read: start
  int blocks;         // blocks per sequence in the grid
  int zero_rest;      // read: rows without a slot are set to 0
};

// Workgroup -> (block of the sequence's range, head, sequence).
__device__ __forceinline__ void place(const RowsParams& p, int& blk, int& head, int& b) {
  const unsigned i = blockIdx.x, hb = i / unsigned(p.blocks);
  blk = int(i - hb * unsigned(p.blocks));
  b = int(hb / unsigned(p.c.heads));
  head = int(hb - unsigned(b) * unsigned(p.c.heads));
}

template <int D, int G>
__global__ void __launch_bounds__(kRowThreads) append_kernel(const RowsParams p) {
  constexpr int CH = D / 8, LANES = D / G / 8;
  __shared__ __attribute__((aligned(16))) uint8_t vc[kBlock][D];
  int i, head, b;
  place(p, i, head, b);
  const int T = p.k.tokens;
  const int n = p.counts ? min(max(p.counts[b], 0), T) : T;
  const int64_t len = p.c.lengths[b], start = len - n;
  const int64_t blk = (start > 0 ? start : 0) / kBlock + i;
  const int64_t at = blk * kBlock;
  const int lo = int(max(max(start, int64_t(0)), at) - at), hi = int(max(min(len - at, int64_t(kBlock)), int64_t(0)));
  if (lo >= hi) return;
  uint8_t* base = block_at<D, G>(p.c, b, head, at);
  if (!base) return;
  const int esz = p.k.dtype == STAGQ_F32 ? 4 : 2;
  const int items = (hi - lo) * CH;
  for (int it = threadIdx.x; it < items; it += kRowThreads) {
    const int tok = lo + it / CH, ch = it % CH;
    const int64_t row = at + tok - start;
    float f[8], g[8];
    unpack8(p.k.data + (b * p.k.sb + row * p.k.st + head * p.k.sh + ch * 8) * esz, p.k.dtype, f);
    unpack8(p.v.data + (b * p.v.sb + row * p.v.st + head * p.v.sh + ch * 8) * esz, p.v.dtype, g);
    uint32_t u[8];
    uint32_t pair = quantise8<LANES>(f, u);
    *reinterpret_cast<uint32_t*>(base + kcode_at(D, G, tok >> 4, (ch & 3) * 16 + (tok & 15), ch >> 2)) = pack_codes(u);
    if (ch % LANES == 0) *reinterpret_cast<uint32_t*>(base + kpair_at(G, tok, ch / LANES)) = pair;
    pair = quantise8<LANES>(g, u);
    u2_t w = {u[0] | u[1] << 8 | u[2] << 16 | u[3] << 24, u[4] | u[5] << 8 | u[6] << 16 | u[7] << 24};
    *reinterpret_cast<u2_t*>(&vc[tok][ch * 8]) = w;
    if (ch % LANES == 0) {
      uint8_t* m = base + vstep_at(G, vset(tok), velem(tok), ch / LANES);
      *reinterpret_cast<uint16_t*>(m) = uint16_t(pair >> 16);
      *reinterpret_cast<uint16_t*>(m + 16) = uint16_t(pair);
    }
  }
  __syncthreads();
  // V: a dword holds eight tokens of one channel; those outside the range keep
  // their nibbles.  A thread turns four channels of a set of tokens.
  for (int it = threadIdx.x; it < D; it += kRowThreads) {
    const int set = it / (D / 4), c4 = (it % (D / 4)) * 4;
    uint32_t w[4] = {0, 0, 0, 0}, mask = 0;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const int tok = vtoken(set, e);
      if (tok >= lo && tok < hi) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(&vc[tok][c4]);
        mask |= 15u << (4 * nibble(e));
#pragma unroll
        for (int k = 0; k < 4; k++) w[k] |= ((x >> (8 * k)) & 15u) << (4 * nibble(e));
      }
    }
    if (!mask) continue;
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const int c = c4 + k;
      uint32_t* dst = reinterpret_cast<uint32_t*>(base + vcode_at(D, G, set * 16 + (c & 15), c >> 4));
      *dst = mask == 0xffffffffu ? w[k] : (w[k] | (*dst & ~mask));
    }
  }
}

// One new token per sequence, the decode step: a wave per sequence and kv head,
// its first D / 8 lanes for K and the next for V (at 256 channels all), each
// with eight channels.  Nothing but a chain of loads bounds it (length, page,
// the eight dwords of V that keep their other nibbles), so there is no LDS and
// no barrier, and the rows are requested first.
template <int D, int G>
__global__ void __launch_bounds__(256) append_one_kernel(const RowsParams p) {
  constexpr int CH = D / 8, LANES = D / G / 8;
  const int lane = threadIdx.x & 63;
  const unsigned hb = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (hb >= unsigned(p.c.batch) * unsigned(p.c.heads)) return;
  const int b = int(hb / unsigned(p.c.heads)), head = int(hb - unsigned(b) * unsigned(p.c.heads));
  const bool is_v = lane >= CH, mine = lane < 2 * CH;
  const int ch = mine ? lane - (is_v ? CH : 0) : 0;
  const int esz = p.k.dtype == STAGQ_F32 ? 4 : 2;
  float f[8];
  const Tensor& t = p.k;
  const int64_t at_k = b * p.k.sb + head * p.k.sh + ch * 8, at_v = b * p.v.sb + head * p.v.sh + ch * 8;
  unpack8(is_v ? p.v.data + at_v * esz : p.k.data + at_k * esz, t.dtype, f);
  const int n = p.counts ? p.counts[b] : 1;
  const int64_t slot = int64_t(p.c.lengths[b]) - 1;
  if (n <= 0 || slot < 0) return;
  uint8_t* base = block_at<D, G>(p.c, b, head, slot);
  if (!base) return;
  const int tok = int(slot) & (kBlock - 1);
  uint32_t* dst[8];
  uint32_t old[8];
#pragma unroll
  for (int e = 0; e < 8; e++) {
    const int c = ch * 8 + e;
    dst[e] = reinterpret_cast<uint32_t*>(base + vcode_at(D, G, vset(tok) * 16 + (c & 15), c >> 4));
    old[e] = mine && is_v ? *dst[e] : 0u;
  }
  uint32_t u[8];
  const uint32_t pair = quantise8<LANES>(f, u);
  if (!mine) return;
  if (!is_v) {
    *reinterpret_cast<uint32_t*>(base + kcode_at(D, G, tok >> 4, (ch & 3) * 16 + (tok & 15), ch >> 2)) = pack_codes(u);
    if (ch % LANES == 0) *reinterpret_cast<uint32_t*>(base + kpair_at(G, tok, ch / LANES)) = pair;
    return;
  }
  const int shift = 4 * nibble(velem(tok));
#pragma unroll
  for (int e = 0; e < 8; e++) *dst[e] = (old[e] & ~(15u << shift)) | u[e] << shift;
  if (ch % LANES == 0) {
    uint8_t* m = base + vstep_at(G, vset(tok), velem(tok), ch / LANES);
    *reinterpret_cast<uint16_t*>(m) = uint16_t(pair >> 16);
    *reinterpret_cast<uint16_t*>(m + 16) = uint16_t(pair);
  }
}

__device__ __forceinline__ void store8(uint8_t* dst, int dtype, const float* f) {
  if (dtype == STAGQ_F32) {
    f4_t a = {f[0], f[1], f[2], f[3]}, b = {f[4], f[5], f[6], f[7]};
    *reinterpret_cast<f4_t*>(dst) = a;
    *reinterpret_cast<f4_t*>(dst + 16) = b;
  } else {
    u4_t v;
    for (int i = 0; i < 4; i++) v[i] = uint32_t(to_16(f[2 * i], dtype)) | uint32_t(to_16(f[2 * i + 1], dtype)) << 16;
    *reinterpret_cast<u4_t*>(dst) = v;
  }
}

template <int D, int G>
__global__ void __launch_bounds__(kRowThreads) read_kernel(const RowsParams p) {
  constexpr int CH = D / 8, LANES = D / G / 8, NV = D / 16;
  __shared__ uint8_t vc[kBlock][D];
  int i, head, b;
  place(p, i, head, b);
  const int64_t start = p.counts ? p.counts[b] : 0, end = start + p.k.tokens;
  const int64_t at = ((start >> 5) + i) * kBlock;   // block of slots; those below 0 hold nothing
  const int64_t held = p.c.lengths[b];
  // rows [lo, hi) of the block are in the tensors, [lo, has) of them in the cache
  const int lo = int(max(start, at) - at), hi = int(max(min(end - at, int64_t(kBlock)), int64_t(0)));
  const int has = at < 0 ? 0 : int(max(min(held - at, int64_t(hi)), int64_t(0)));
  const int last = p.zero_rest ? hi : has;
  if (lo >= last) return;
  const uint8_t* base = has > lo ? block_at<D, G>(p.c, b, head, at) : nullptr;   // null: the rows are 0
  if (base) {
    for (int it = threadIdx.x; it < 64 * NV; it += kRowThreads) {
      const int lane = it & 63, ct = it >> 6, set = lane >> 4, c = ct * 16 + (lane & 15);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(base + vcode_at(D, G, lane, ct));
#pragma unroll
      for (int e = 0; e < 8; e++) vc[vtoken(set, e)][c] = (w >> (4 * nibble(e))) & 15u;
    }
  }
  __syncthreads();
  const int esz = p.k.dtype == STAGQ_F32 ? 4 : 2;
  const int items = (last - lo) * CH;
  for (int it = threadIdx.x; it < items; it += kRowThreads) {
    const int tok = lo + it / CH, ch = it % CH;
    const int64_t row = at + tok - start;
    float f[8] = {0, 0, 0, 0, 0, 0, 0, 0}, g[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (base && tok < has) {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(
          base + kcode_at(D, G, tok >> 4, (ch & 3) * 16 + (tok & 15), ch >> 2));
      const uint32_t pair = *reinterpret_cast<const uint32_t*>(base + kpair_at(G, tok, ch / LANES));
      const float klo = half_bits(pair & 0xffffu), ks = half_bits(pair >> 16);
      const uint8_t* m = base + vstep_at(G, vset(tok), velem(tok), ch / LANES);
      const float vs = half_bits(*reinterpret_cast<const uint16_t*>(m));
      const float vlo = half_bits(*reinterpret_cast<const uint16_t*>(m + 16));
#pragma unroll
      for (int e = 0; e < 8; e++) {
        f[e] = fmaf(ks, float((w >> (4 * nibble(e))) & 15u), klo);
        g[e] = fmaf(vs, float(vc[tok][ch * 8 + e]), vlo);
      }
    }
    store8(p.k.data + (b * p.k.sb + row * p.k.st + head * p.k.sh + ch * 8) * esz, p.k.dtype, f);
    store8(p.v.data + (b * p.v.sb + row * p.v.st + head * p.v.sh + ch * 8) * esz, p.v.dtype, g);
  }
}

struct LaunchAppend {
  RowsParams p;
  hipStream_t st;
  template <int D, int G>
  int go() {
    const int64_t heads = int64_t(p.c.batch) * p.c.heads;
    if (p.k.tokens == 1)
      hipLaunchKernelGGL((append_one_kernel<D, G>), dim3(unsigned((heads + 3) / 4)), dim3(256), 0, st, p);
    else
      hipLaunchKernelGGL((append_kernel<D, G>), dim3(unsigned(heads * p.blocks)), dim3(kRowThreads), 0, st, p);
    return launched();
  }
};
struct LaunchRead {
  RowsParams p;
  hipStream_t st;
  template <int D, int G>
  int go() {
    const unsigned n = unsigned(int64_t(p.c.batch) * p.c.heads * p.blocks);
    hipLaunchKernelGGL((read_kernel<D, G>), dim3(n), dim3(kRowThreads), 0, st, p);
    return launched();
  }
};

static int check_rows(const stagq_kv_cache* c, const stagq_kv_seqs* q, const stagq_kv_tensor* k,
                      const stagq_kv_tensor* v, const int32_t* counts, RowsParams* p) {
  int st = check_cache(c);
  if (st == STAGQ_OK) st = check_seqs(c, q);
  if (st != STAGQ_OK) return st;
  if (!k || !v) return STAGQ_EINVAL;
  st = check_tensor(*k, c->kv_heads, true, q->batch);
  if (st == STAGQ_OK) st = check_tensor(*v, c->kv_heads, true, q->batch);
  if (st != STAGQ_OK) return st;
  if (k->dtype != v->dtype || k->tokens != v->tokens) return STAGQ_EINVAL;
  if (misaligned(counts, 4)) return STAGQ_EALIGN;
  p->c = make_cache(c, q);
  p->k = make_tensor(*k);
  p->v = make_tensor(*v);
  p->counts = counts;
  // T rows from any slot on touch at most (T + 30) / 32 + 1 blocks
  p->blocks = k->tokens == 0 ? 0 : (k->tokens + kBlock - 2) / kBlock + 1;
  if (!launchable(int64_t(q->batch) * c->kv_heads * p->blocks, kRowThreads)) return STAGQ_ESHAPE;
  return STAGQ_OK;
}

}  // namespace kv
}  // namespace stagq

using namespace stagq::kv;

extern "C" {

size_t stagq_kv_bytes(const stagq_kv_cache* c) {
  if (!c || !supported(c->pages, c->page_tokens, c->kv_heads, c->head_dim, c->group)) return 0;
  return size_t(uint64_t(c->pages) * page_bytes(c->page_tokens, c->kv_heads, c->head_dim, c->group));
}

int stagq_kv_append(const stagq_kv_cache* c, const stagq_kv_seqs* q, const stagq_kv_tensor* k,
                    const stagq_kv_tensor* v, const int32_t* new_lens, void* hip_stream) {
  RowsParams p;
  const int st = check_rows(c, q, k, v, new_lens, &p);
  if (st != STAGQ_OK) return st;
  if (q->batch == 0 || p.blocks == 0 || c->pages == 0) return STAGQ_OK;
  return by_shape(c, LaunchAppend{p, static_cast<hipStream_t>(hip_stream)});
}

int stagq_kv_read(const stagq_kv_cache* c, const stagq_kv_seqs* q, const int32_t* start, const stagq_kv_tensor* k,
                  const stagq_kv_tensor* v, int zero_rest, void* hip_stream) {
  RowsParams p;
  const int st = check_rows(c, q, k, v, start, &p);
  if (st != STAGQ_OK) return st;
  if (q->batch == 0 || p.blocks == 0) return STAGQ_OK;
  if (k->data == v->data || !disjoint(*k, q->batch, c->head_dim) || !disjoint(*v, q->batch, c->head_dim)) return STAGQ_EINVAL;
  p.zero_rest = zero_rest;
  return by_shape(c, LaunchRead{p, static_cast<hipStream_t>(hip_stream)});
}

}  // extern "C"
