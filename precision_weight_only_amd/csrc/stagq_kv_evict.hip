// Eviction from the key/value cache in 4 bits by accumulated attention weight.
//
// select: one workgroup per sequence and kv head finds the weight of the
// lightest token that stays (a radix select over the order-preserving bits, 8
// at a time), then writes the slots that stay in order and gathers their
// weights.  gather: one workgroup per block of 32 tokens that stay and kv head
// moves their codes and pairs.  All counts are integers, so no result depends
// on the order of the atomics.
#include "stagq_kv_host.h"

namespace stagq {
namespace kv {

constexpr int kSelectThreads = 1024;

struct EvictParams {
  Cache c;
  const float* w;
  float* wout;
  int64_t wsb, wsh, osb, osh;
  int* kept;
  int* out_lengths;
  const int* out_table;   // null: the tokens go to `stage` first
  int64_t out_stride;
  int out_width;
  uint8_t* stage;         // [batch][kv head][block][block bytes]
  int keep, sinks, recent;
  int64_t max_len;
  int blocks;             // of 32 tokens that stay, per sequence
};

__device__ __forceinline__ int seq_len(const EvictParams& p, int b) {
  const int64_t len = p.c.lengths[b];
  return int(len < 0 ? 0 : len > p.max_len ? p.max_len : len);
}

// Weights in order as unsigned numbers: NaN highest, -0 = +0.
__device__ __forceinline__ uint32_t order_of(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const EvictParams p) {
  constexpr int NW = kSelectThreads / 64;
  __shared__ int hist[256];
  __shared__ int found_bin, found_rest;
  __shared__ int n_above[NW], n_equal[NW];
  const int hk = int(blockIdx.x % unsigned(p.c.heads)), b = int(blockIdx.x / unsigned(p.c.heads));
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = seq_len(p, b), m = min(n, p.keep);
  const float* w = p.w + b * p.wsb + hk * p.wsh;
  int* kept = p.kept + (int64_t(b) * p.c.heads + hk) * p.keep;
  if (n <= p.keep) {
    for (int i = tid; i < p.keep; i += kSelectThreads) kept[i] = i < n ? i : -1;
  } else {
    // the middle [sinks, end) gives `want` tokens
    const int end = n - p.recent, want = p.keep - p.sinks - p.recent;
    uint32_t prefix = 0, mask = 0;
    int rest = want;
    if (want > 0) {
      for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int i = p.sinks + tid; i < end; i += kSelectThreads) {
          const uint32_t k = order_of(w[i]);
          if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
        }
        __syncthreads();
        if (wave == 0) {   // bins from the highest: 4 per lane, lane 0 the top ones
          int c[4], total = 0;
          for (int i = 0; i < 4; i++) { c[i] = hist[255 - (lane * 4 + i)]; total += c[i]; }
          int before = total;
          for (int d = 1; d < 64; d *= 2) { const int o = __shfl_up(before, d); if (lane >= d) before += o; }
          before -= total;
          for (int i = 0; i < 4; i++) {
            if (before < rest && before + c[i] >= rest) { found_bin = 255 - (lane * 4 + i); found_rest = rest - before; }
            before += c[i];
          }
        }
        __syncthreads();
        prefix |= uint32_t(found_bin) << shift;
        mask |= 255u << shift;
        rest = found_rest;
        __syncthreads();
      }
    }
    // stays: the ends, those above prefix, and the first `rest` equal to it
    const int per = (n + NW * 64 - 1) / (NW * 64) * 64;
    const int from = min(wave * per, n), to = min(from + per, n);
    auto look = [&](int i, bool& above, bool& equal) {
      above = equal = false;
      if (i >= to) return;
      if (i < p.sinks || i >= end) { above = true; return; }
      if (want == 0) return;
      const uint32_t k = order_of(w[i]);
      above = k > prefix;
      equal = k == prefix;
    };
    int na = 0, ne = 0;
    for (int i = from; i < to; i += 64) {
      bool a, e;
      look(i + lane, a, e);
      na += __popcll(__ballot(a));
      ne += __popcll(__ballot(e));
    }
    if (lane == 0) { n_above[wave] = na; n_equal[wave] = ne; }
    __syncthreads();
    int above = 0, equal = 0;   // before this wave's part
    for (int i = 0; i < wave; i++) { above += n_above[i]; equal += n_equal[i]; }
    const uint64_t below = (uint64_t(1) << lane) - 1;
    for (int i = from; i < to; i += 64) {
      bool a, e;
      look(i + lane, a, e);
      const uint64_t ma = __ballot(a), me = __ballot(e);
      const int eq_rank = equal + __popcll(me & below);
      const int at = above + __popcll(ma & below) + min(eq_rank, rest);
      if ((a || (e && eq_rank < rest)) && at < p.keep) kept[at] = i + lane;
      above += __popcll(ma);
      equal += __popcll(me);
    }
  }
  __threadfence_block();
  __syncthreads();
  // Weights move to lower or equal places, in tiles: a tile is read before it
  // is written, and later tiles read past it.
  float* wo = p.wout + b * p.osb + hk * p.osh;
  for (int i0 = 0; i0 < m; i0 += kSelectThreads) {
    const int i = i0 + tid;
    const float v = i < m ? w[kept[i]] : 0.0f;
    __syncthreads();
    if (i < m) wo[i] = v;
  }
  __syncthreads();
  for (int64_t i = m + tid; i < p.max_len; i += kSelectThreads) wo[i] = 0.0f;
}

template <int D, int G>
__device__ __forceinline__ uint8_t* out_block(const EvictParams& p, int b, int hk, int blk) {
  const int64_t slot = int64_t(blk) * kBlock, e = slot >> p.c.shift;
  const int* table = p.out_table ? p.out_table : p.c.table;
  const int64_t stride = p.out_table ? p.out_stride : p.c.table_stride;
  if (e >= (p.out_table ? p.out_width : p.c.width)) return nullptr;
  const int page = table[int64_t(b) * stride + e];
  if (page < 0 || page >= p.c.pages) return nullptr;
  return p.c.buf + uint64_t(page) * p.c.page_bytes + uint64_t(hk) * p.c.head_bytes +
         uint32_t((slot & ((int64_t(1) << p.c.shift) - 1)) / kBlock) * block_bytes(D, G);
}

template <int D, int G>
__global__ void __launch_bounds__(256) gather_kernel(const EvictParams p) {
  constexpr int NK = D / 32, NV = D / 16;
  __shared__ const uint8_t* src[kBlock];
  __shared__ int tok[kBlock];
  unsigned id = blockIdx.x;
  const int blk = int(id % unsigned(p.blocks)); id /= unsigned(p.blocks);
  const int hk = int(id % unsigned(p.c.heads)), b = int(id / unsigned(p.c.heads));
  const int m = min(seq_len(p, b), p.keep);
  if (blk == 0 && hk == 0 && threadIdx.x == 0) p.out_lengths[b] = m;
  if (blk * kBlock >= m) return;
  uint8_t* dst = p.stage ? p.stage + ((int64_t(b) * p.c.heads + hk) * p.blocks + blk) * int64_t(block_bytes(D, G))
                         : out_block<D, G>(p, b, hk, blk);
  if (!dst) return;
  if (threadIdx.x < kBlock) {
    const int i = blk * kBlock + threadIdx.x;
    const uint8_t* s = nullptr;
    int t = 0;
    if (i < m) {
      const int slot = p.kept[(int64_t(b) * p.c.heads + hk) * p.keep + i];
      s = block_at<D, G>(p.c, b, hk, slot);
      t = slot % kBlock;
    }
    src[threadIdx.x] = s;
    tok[threadIdx.x] = t;
  }
  __syncthreads();
  // K: every dword belongs to one token.
  for (int it = threadIdx.x; it < 2 * 64 * NK; it += 256) {
    const int ks = it % NK, lane = (it / NK) & 63, u = it / (64 * NK), t = u * 16 + (lane & 15);
    const uint8_t* s = src[t];
    uint32_t w = 0;
    if (s) w = *reinterpret_cast<const uint32_t*>(s + kcode_at(D, G, tok[t] >> 4, (lane & 48) | (tok[t] & 15), ks));
    *reinterpret_cast<uint32_t*>(dst + kcode_at(D, G, u, lane, ks)) = w;
  }
  for (int it = threadIdx.x; it < kBlock * G; it += 256) {
    const int t = it % kBlock, g = it / kBlock;
    const uint8_t* s = src[t];
    uint32_t w = 0;
    uint16_t vs = 0, vl = 0;
    if (s) {
      w = *reinterpret_cast<const uint32_t*>(s + kpair_at(G, tok[t], g));
      const uint8_t* v = s + vstep_at(G, vset(tok[t]), velem(tok[t]), g);
      vs = *reinterpret_cast<const uint16_t*>(v);
      vl = *reinterpret_cast<const uint16_t*>(v + 16);
    }
    *reinterpret_cast<uint32_t*>(dst + kpair_at(G, t, g)) = w;
    uint8_t* v = dst + vstep_at(G, vset(t), velem(t), g);
    *reinterpret_cast<uint16_t*>(v) = vs;
    *reinterpret_cast<uint16_t*>(v + 16) = vl;
  }
  // V: a dword takes one nibble from each of its eight tokens.
  for (int it = threadIdx.x; it < 64 * NV; it += 256) {
    const int lane = it & 63, ct = it >> 6, set = lane >> 4;
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const int t = vtoken(set, e);
      const uint8_t* s = src[t];
      if (!s) continue;
      const uint32_t x = *reinterpret_cast<const uint32_t*>(s + vcode_at(D, G, vset(tok[t]) * 16 + (lane & 15), ct));
      w |= ((x >> (4 * nibble(velem(tok[t])))) & 15u) << (4 * nibble(e));
    }
    *reinterpret_cast<uint32_t*>(dst + vcode_at(D, G, lane, ct)) = w;
  }
}

// The staged blocks to their pages.
template <int D, int G>
__global__ void __launch_bounds__(256) place_kernel(const EvictParams p) {
  unsigned id = blockIdx.x;
  const int blk = int(id % unsigned(p.blocks)); id /= unsigned(p.blocks);
  const int hk = int(id % unsigned(p.c.heads)), b = int(id / unsigned(p.c.heads));
  if (blk * kBlock >= min(seq_len(p, b), p.keep)) return;
  uint8_t* dst = out_block<D, G>(p, b, hk, blk);
  if (!dst) return;
  const uint8_t* s = p.stage + ((int64_t(b) * p.c.heads + hk) * p.blocks + blk) * int64_t(block_bytes(D, G));
  for (uint32_t i = threadIdx.x * 16; i < block_bytes(D, G); i += 256 * 16)
    *reinterpret_cast<u4_t*>(dst + i) = *reinterpret_cast<const u4_t*>(s + i);
}

struct LaunchEvict {
  EvictParams p;
  hipStream_t st;
  template <int D, int G>
  int go() {
    const unsigned heads = unsigned(p.c.batch) * unsigned(p.c.heads);
    hipLaunchKernelGGL(select_kernel, dim3(heads), dim3(kSelectThreads), 0, st, p);
    int s = launched();
    if (s != STAGQ_OK) return s;
    hipLaunchKernelGGL((gather_kernel<D, G>), dim3(heads * unsigned(p.blocks)), dim3(256), 0, st, p);
    s = launched();
    if (s != STAGQ_OK || !p.stage) return s;
    hipLaunchKernelGGL((place_kernel<D, G>), dim3(heads * unsigned(p.blocks)), dim3(256), 0, st, p);
    return launched();
  }
};

static int check_evict(const stagq_kv_cache* c, const stagq_kv_seqs* q, const stagq_kv_evict_args* e) {
  int st = check_cache(c);
  if (st == STAGQ_OK) st = check_seqs(c, q);
  if (st != STAGQ_OK) return st;
  if (!e || e->keep < 1 || e->sinks < 0 || e->recent < 0 || e->max_len < 0) return STAGQ_EINVAL;
  if (int64_t(e->sinks) + e->recent > e->keep) return STAGQ_EINVAL;
  if (q->batch == 0) return STAGQ_OK;
  if (!e->kept || !e->out_lengths) return STAGQ_EINVAL;
  if (reach(c, q, e->max_len) > 0 && (!e->weights || !e->weights_out)) return STAGQ_EINVAL;
  if (e->weights_stride_seq < 0 || e->weights_stride_head < 0 || e->out_stride_seq < 0 || e->out_stride_head < 0)
    return STAGQ_EINVAL;
  if (misaligned(e->weights, 4) || misaligned(e->weights_out, 4) || misaligned(e->kept, 4) ||
      misaligned(e->out_lengths, 4) || misaligned(e->out_table, 4))
    return STAGQ_EALIGN;
  if (e->out_table) {
    if (e->out_table_width < 0 || (q->batch > 1 && e->out_table_stride < e->out_table_width)) return STAGQ_EINVAL;
    if (int64_t(e->out_table_width) * c->page_tokens < (e->keep < reach(c, q, e->max_len) ? e->keep : reach(c, q, e->max_len)))
      return STAGQ_ESIZE;
  }
  const int64_t blocks = (int64_t(e->keep) + kBlock - 1) / kBlock;
  const int64_t heads = int64_t(q->batch) * c->kv_heads;
  if (!launchable(heads * blocks, 256) || !launchable(heads, kSelectThreads)) return STAGQ_ESHAPE;
  return STAGQ_OK;
}

// Tokens that can stay: keep, or all slots within reach.
static int evict_blocks(const stagq_kv_cache* c, const stagq_kv_seqs* q, const stagq_kv_evict_args* e) {
  const int64_t r = reach(c, q, e->max_len), m = e->keep < r ? e->keep : r;
  return int(m > 0 ? (m + kBlock - 1) / kBlock : 1);
}

}  // namespace kv
}  // namespace stagq

using namespace stagq::kv;

extern "C" {

size_t stagq_kv_evict_workspace(const stagq_kv_cache* c, const stagq_kv_seqs* q, const stagq_kv_evict_args* e) {
  if (check_evict(c, q, e) != STAGQ_OK || e->out_table) return 0;
  return size_t(q->batch) * c->kv_heads * size_t(evict_blocks(c, q, e)) * block_bytes(c->head_dim, c->head_dim / c->group);
}

int stagq_kv_evict(const stagq_kv_cache* c, const stagq_kv_seqs* q, const stagq_kv_evict_args* e, void* workspace,
                   size_t workspace_bytes, void* hip_stream) {
  const int st = check_evict(c, q, e);
  if (st != STAGQ_OK) return st;
  if (q->batch == 0) return STAGQ_OK;
  const size_t need = stagq_kv_evict_workspace(c, q, e);
  if (need > 0 && !workspace) return STAGQ_EINVAL;
  if (misaligned(workspace, 256)) return STAGQ_EALIGN;
  if (workspace_bytes < need) return STAGQ_ESIZE;
  EvictParams p;
  p.c = make_cache(c, q);
  p.w = e->weights;
  p.wout = e->weights_out;
  p.wsb = e->weights_stride_seq;
  p.wsh = e->weights_stride_head;
  p.osb = e->out_stride_seq;
  p.osh = e->out_stride_head;
  p.kept = e->kept;
  p.out_lengths = e->out_lengths;
  p.out_table = e->out_table;
  p.out_stride = e->out_table_stride;
  p.out_width = e->out_table_width;
  p.stage = e->out_table ? nullptr : static_cast<uint8_t*>(workspace);
  p.keep = e->keep;
  p.sinks = e->sinks;
  p.recent = e->recent;
  p.max_len = reach(c, q, e->max_len);
  p.blocks = evict_blocks(c, q, e);
  return by_shape(c, LaunchEvict{p, static_cast<hipStream_t>(hip_stream)});
}

}  // extern "C"
