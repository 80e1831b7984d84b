// Eviction from the key/value cache in 4 bits by accumulated attention weight.
//
// The slots that stay: a radix select over the order-preserving bits of the
// weights (11, 11 and 10 of them) finds the lightest that stays, and a count of
// heavier and equal ones gives every slot its place.  Up to kSmall slots one
// workgroup per sequence and kv head does it all (select_kernel).  Beyond, one
// workgroup would take 72 to 111 us at 65536 slots (its compute unit reads the
// weights five times and counts in one LDS), so the slots are cut into parts of
// 4096: count_kernel counts the first digit per part, sort_kernel adds the counts
// up, counts the heavier slots and sets aside those with the deciding digit,
// settle_kernel (one workgroup again, over those few) finds the weight itself and
// where every part's slots go, write_kernel writes them.  Many weights are
// exactly 0 and would meet in one counter: they are counted by ballot.
// gather: one workgroup per block of 32 tokens that stay and kv head moves their
// codes, pairs and weights.  All counts are integers, so no result depends on
// the order of the atomics.
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
  int parts;              // of 4096 slots; 0: one workgroup per sequence and head selects
  uint8_t* parts_ws;
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

constexpr int kWaves = kSelectThreads / 64, kBins = 2048;
constexpr int kPart = 4 * kSelectThreads;   // slots of a part, four per thread
// Up to here select_kernel, of at most 16 keys a thread.  8 kv heads, keep 1024,
// with the gather: at 16384 slots 25 us against 31 us in parts, at 12000 22
// against 30 us (32 sequences 71 against 96 us); with 32 keys a thread 32768
// slots take 43 us against 33 us in parts (8 sequences 65 against 58 us).
constexpr int kSmall = 4 * kPart;
constexpr uint32_t kZeroKey = 0x80000000u;
// Keys below that of -inf: slots that stay anyway, and slots past the end.
constexpr uint32_t kEnd = 1u, kPast = 0u;

// One sequence and kv head.
struct Item {
  int n, m, end, want;   // tokens; that stay; the middle [sinks, end) gives `want`
  const float* w;
  int* kept;
};
__device__ __forceinline__ Item item_of(const EvictParams& p, int b, int hk) {
  Item t;
  t.n = seq_len(p, b);
  t.m = min(t.n, p.keep);
  t.end = t.n - p.recent;
  t.want = p.keep - p.sinks - p.recent;
  t.w = p.w + b * p.wsb + hk * p.wsh;
  t.kept = p.kept + (int64_t(b) * p.c.heads + hk) * p.keep;
  return t;
}
__device__ __forceinline__ uint32_t key_at(const EvictParams& p, const Item& t, int i) {
  return i >= t.n ? kPast : i < p.sinks || i >= t.end ? kEnd : order_of(t.w[i]);
}
__device__ __forceinline__ int shift_of(int pass) { return pass == 0 ? 21 : pass == 1 ? 10 : 0; }
__device__ __forceinline__ uint32_t digit_mask(int pass) { return pass == 2 ? 1023u : 2047u; }

struct SelectLds {
  int hist[kBins];
  int wave_sum[kWaves];
  int bin, rest;
  int above[kWaves], equal[kWaves];
};
__device__ __forceinline__ void clear_hist(SelectLds& s) {
  for (int i = threadIdx.x; i < kBins; i += kSelectThreads) s.hist[i] = 0;
  __syncthreads();
}
// Counts 64 keys; returns those that are 0, for the caller to add in one go.
__device__ __forceinline__ int count_key(SelectLds& s, uint32_t k, uint32_t prefix, uint32_t mask, int pass) {
  const bool in = k > kEnd && (k & mask) == prefix, zero = in && k == kZeroKey;
  if (in && !zero) atomicAdd(&s.hist[(k >> shift_of(pass)) & digit_mask(pass)], 1);
  return __popcll(__ballot(zero));
}
__device__ __forceinline__ void count_zeros(SelectLds& s, int zeros, int pass) {
  if ((threadIdx.x & 63) == 0 && zeros) atomicAdd(&s.hist[(kZeroKey >> shift_of(pass)) & digit_mask(pass)], zeros);
}
// c0 and c1: counts of the bins 2047 - 2 tid and the one below.  Finds the bin
// in which the count from the highest reaches `rest`: s.bin, and in s.rest how
// many of it stay.
__device__ __forceinline__ void find_bin(SelectLds& s, int c0, int c1, int rest) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b0 = kBins - 1 - 2 * tid;
  int upto = c0 + c1;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) { const int o = __shfl_up(upto, d); if (lane >= d) upto += o; }
  if (lane == 63) s.wave_sum[wave] = upto;
  __syncthreads();
  for (int i = 0; i < wave; i++) upto += s.wave_sum[i];
  const int before = upto - c0 - c1;
  if (before < rest && before + c0 >= rest) { s.bin = b0; s.rest = rest - before; }
  else if (before + c0 < rest && upto >= rest) { s.bin = b0 - 1; s.rest = rest - before - c0; }
  __syncthreads();
}

// Places of 64 slots' keys: `above` and `equal` stay so far, of those equal to
// prefix the first `rest`.
__device__ __forceinline__ void place_key(const EvictParams& p, const Item& t, int slot, uint32_t k, uint32_t prefix, int rest,
                                          int& above, int& equal) {
  const uint64_t below = (uint64_t(1) << (threadIdx.x & 63)) - 1;
  const bool a = k == kEnd || k > prefix, e = k == prefix;
  const uint64_t ma = __ballot(a), me = __ballot(e);
  const int eq_rank = equal + __popcll(me & below);
  const int at = above + __popcll(ma & below) + min(eq_rank, rest);
  if ((a || (e && eq_rank < rest)) && at < p.keep) t.kept[at] = slot;
  above += __popcll(ma);
  equal += __popcll(me);
}
// Per wave: how many of its keys are above prefix (or stay anyway), and equal.
__device__ __forceinline__ void tally_key(uint32_t k, uint32_t prefix, int& above, int& equal) {
  above += __popcll(__ballot(k == kEnd || k > prefix));
  equal += __popcll(__ballot(k == prefix));
}

// In place: weights move to lower or equal places, in tiles: a tile is read
// before it is written, and later tiles read past it.
__device__ __forceinline__ void weights_in_place(const EvictParams& p, const Item& t, float* wo) {
  for (int i0 = 0; i0 < t.m; i0 += kSelectThreads) {
    const int i = i0 + threadIdx.x;
    const float v = i < t.m ? t.w[t.kept[i]] : 0.0f;
    __syncthreads();
    if (i < t.m) wo[i] = v;
  }
  __syncthreads();
  for (int64_t i = t.m + threadIdx.x; i < p.max_len; i += kSelectThreads) wo[i] = 0.0f;
}

// PER: keys of a thread.
template <int PER>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const EvictParams p) {
  __shared__ SelectLds s;
  const int hk = int(blockIdx.x % unsigned(p.c.heads)), b = int(blockIdx.x / unsigned(p.c.heads));
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Item t = item_of(p, b, hk);
  if (t.n <= p.keep) {
    for (int i = tid; i < p.keep; i += kSelectThreads) t.kept[i] = i < t.n ? i : -1;
  } else {
    const int each = (t.n + kWaves * 64 - 1) / (kWaves * 64), from = wave * each * 64 + lane;   // each <= PER
    uint32_t key[PER];
#pragma unroll
    for (int e = 0; e < PER; e++) key[e] = e < each ? key_at(p, t, from + e * 64) : kPast;
    // (with nothing wanted of the middle: prefix above all keys but NaN, of which 0 stay)
    uint32_t prefix = t.want > 0 ? 0u : 0xffffffffu, mask = 0;
    int rest = t.want;
    for (int pass = 0; pass < 3 && t.want > 0; pass++) {
      clear_hist(s);
      int zeros = 0;
#pragma unroll
      for (int e = 0; e < PER; e++)
        if (e < each) zeros += count_key(s, key[e], prefix, mask, pass);
      count_zeros(s, zeros, pass);
      __syncthreads();
      find_bin(s, s.hist[kBins - 1 - 2 * tid], s.hist[kBins - 2 - 2 * tid], rest);
      prefix |= uint32_t(s.bin) << shift_of(pass);
      mask |= digit_mask(pass) << shift_of(pass);
      rest = s.rest;
    }
    int above = 0, equal = 0;
#pragma unroll
    for (int e = 0; e < PER; e++) tally_key(key[e], prefix, above, equal);
    if (lane == 0) { s.above[wave] = above; s.equal[wave] = equal; }
    __syncthreads();
    above = equal = 0;
    for (int i = 0; i < wave; i++) { above += s.above[i]; equal += s.equal[i]; }
#pragma unroll
    for (int e = 0; e < PER; e++)
      if (e < each) place_key(p, t, from + e * 64, key[e], prefix, rest, above, equal);
  }
  if (p.wout != p.w) return;   // else the gather kernel moves the weights
  __threadfence_block();
  __syncthreads();
  weights_in_place(p, t, p.wout + b * p.osb + hk * p.osh);
}

// ------------------------------------------------------- many slots: parts ----
// Workspace of one item: [parts][2048] counts of the first digit, [parts][4096]
// keys with the deciding one, [parts] PartInfo, and the Verdict.
struct PartInfo {
  int aside, above, equal, spare;   // keys set aside; then (settle) where the part's slots begin
};
struct Verdict {
  uint32_t prefix;
  int rest;
};
struct PartsWs {
  int* hist;
  uint32_t* keys;
  PartInfo* info;
  Verdict* verdict;
};
__host__ __device__ inline size_t parts_bytes(int parts) {   // of one item
  return size_t(parts) * (kBins * 4 + kPart * 4 + sizeof(PartInfo)) + 256;
}
__device__ __forceinline__ PartsWs parts_ws(const EvictParams& p, int item) {
  uint8_t* at = p.parts_ws + size_t(item) * parts_bytes(p.parts);
  PartsWs r;
  r.hist = reinterpret_cast<int*>(at);
  r.keys = reinterpret_cast<uint32_t*>(r.hist + size_t(p.parts) * kBins);
  r.info = reinterpret_cast<PartInfo*>(r.keys + size_t(p.parts) * kPart);
  r.verdict = reinterpret_cast<Verdict*>(r.info + p.parts);
  return r;
}
struct PartOf {
  Item t;
  PartsWs ws;
  int part, parts, from;   // of the item's parts; first slot of the thread (then 64 further, four times)
};
__device__ __forceinline__ PartOf part_of(const EvictParams& p) {
  const int item = blockIdx.y, b = item / p.c.heads;
  PartOf r;
  r.t = item_of(p, b, item - b * p.c.heads);
  r.ws = parts_ws(p, item);
  r.part = blockIdx.x;
  r.parts = (r.t.n + kPart - 1) / kPart;
  r.from = r.part * kPart + int(threadIdx.x >> 6) * 256 + int(threadIdx.x & 63);
  return r;
}

__global__ void __launch_bounds__(kSelectThreads) count_kernel(const EvictParams p) {
  __shared__ SelectLds s;
  const PartOf o = part_of(p);
  if (o.t.n <= p.keep || o.part >= o.parts || o.t.want == 0) return;
  uint32_t k[4];
#pragma unroll
  for (int e = 0; e < 4; e++) k[e] = key_at(p, o.t, o.from + e * 64);
  clear_hist(s);
  int zeros = 0;
#pragma unroll
  for (int e = 0; e < 4; e++) zeros += count_key(s, k[e], 0u, 0u, 0);
  count_zeros(s, zeros, 0);
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kSelectThreads) o.ws.hist[size_t(o.part) * kBins + i] = s.hist[i];
}

__global__ void __launch_bounds__(kSelectThreads) sort_kernel(const EvictParams p) {
  __shared__ SelectLds s;
  const PartOf o = part_of(p);
  if (o.t.n <= p.keep || o.part >= o.parts || o.t.want == 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t k[4];
#pragma unroll
  for (int e = 0; e < 4; e++) k[e] = key_at(p, o.t, o.from + e * 64);
  int c0 = 0, c1 = 0;
#pragma unroll 8
  for (int i = 0; i < o.parts; i++) {
    const int2 c = *reinterpret_cast<const int2*>(o.ws.hist + size_t(i) * kBins + kBins - 2 - 2 * tid);
    c0 += c.y;
    c1 += c.x;
  }
  find_bin(s, c0, c1, o.t.want);
  const uint32_t bin = uint32_t(s.bin);
  int above = 0, aside = 0;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    above += __popcll(__ballot(k[e] == kEnd || (k[e] > kEnd && (k[e] >> 21) > bin)));
    aside += __popcll(__ballot(k[e] > kEnd && (k[e] >> 21) == bin));
  }
  if (lane == 0) { s.above[wave] = above; s.equal[wave] = aside; }
  __syncthreads();
  int at = 0, all = 0, sum = 0;
  for (int i = 0; i < kWaves; i++) {
    if (i < wave) at += s.equal[i];
    all += s.equal[i];
    sum += s.above[i];
  }
  uint32_t* keys = o.ws.keys + size_t(o.part) * kPart;
  const uint64_t below = (uint64_t(1) << lane) - 1;
#pragma unroll
  for (int e = 0; e < 4; e++) {
    const bool in = k[e] > kEnd && (k[e] >> 21) == bin;
    const uint64_t m = __ballot(in);
    if (in) keys[at + __popcll(m & below)] = k[e];
    at += __popcll(m);
  }
  if (tid == 0) {
    o.ws.info[o.part] = PartInfo{all, sum, 0, 0};
    if (o.part == 0) *o.ws.verdict = Verdict{bin << 21, s.rest};
  }
}

__global__ void __launch_bounds__(kSelectThreads) settle_kernel(const EvictParams p) {
  __shared__ SelectLds s;
  const int item = blockIdx.x, b = item / p.c.heads;
  const Item t = item_of(p, b, item - b * p.c.heads);
  if (t.n <= p.keep || t.want == 0) return;
  const PartsWs ws = parts_ws(p, item);
  const int parts = (t.n + kPart - 1) / kPart;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint32_t prefix = ws.verdict->prefix, mask = 2047u << 21;
  int rest = ws.verdict->rest;
  for (int pass = 1; pass < 3; pass++) {
    clear_hist(s);
    int zeros = 0;
    for (int i = wave; i < parts; i += kWaves) {   // a wave per part
      const int n = ws.info[i].aside;
      const uint32_t* keys = ws.keys + size_t(i) * kPart;
#pragma unroll 4
      for (int e = 0; e < n; e += 64) zeros += count_key(s, e + lane < n ? keys[e + lane] : kPast, prefix, mask, pass);
    }
    count_zeros(s, zeros, pass);
    __syncthreads();
    find_bin(s, s.hist[kBins - 1 - 2 * tid], s.hist[kBins - 2 - 2 * tid], rest);
    prefix |= uint32_t(s.bin) << shift_of(pass);
    mask |= digit_mask(pass) << shift_of(pass);
    rest = s.rest;
  }
  for (int i = wave; i < parts; i += kWaves) {
    const PartInfo in = ws.info[i];
    const uint32_t* keys = ws.keys + size_t(i) * kPart;
    int above = in.above, equal = 0;
#pragma unroll 4
    for (int e = 0; e < in.aside; e += 64) tally_key(e + lane < in.aside ? keys[e + lane] : kPast, prefix, above, equal);
    if (lane == 0) ws.info[i] = PartInfo{in.aside, above, equal, 0};
  }
  __threadfence_block();
  __syncthreads();
  if (wave == 0) {   // where the parts begin
    int above = 0, equal = 0;
    for (int i0 = 0; i0 < parts; i0 += 64) {
      PartInfo in = {0, 0, 0, 0};
      if (i0 + lane < parts) in = ws.info[i0 + lane];
      int a = in.above, e = in.equal;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int x = __shfl_up(a, d), y = __shfl_up(e, d);
        if (lane >= d) { a += x; e += y; }
      }
      if (i0 + lane < parts) ws.info[i0 + lane] = PartInfo{in.aside, above + a - in.above, equal + e - in.equal, 0};
      above += __shfl(a, 63);
      equal += __shfl(e, 63);
    }
    if (lane == 0) *ws.verdict = Verdict{prefix, rest};
  }
}

__global__ void __launch_bounds__(kSelectThreads) write_kernel(const EvictParams p) {
  __shared__ SelectLds s;
  const PartOf o = part_of(p);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (o.t.n <= p.keep) {   // all stay; the last part also writes what is past the slots
    const int to = o.part == p.parts - 1 ? p.keep : min((o.part + 1) * kPart, p.keep);
    for (int i = o.part * kPart + tid; i < to; i += kSelectThreads) o.t.kept[i] = i < o.t.n ? i : -1;
    return;
  }
  if (o.part >= o.parts) return;
  uint32_t k[4];
#pragma unroll
  for (int e = 0; e < 4; e++) k[e] = key_at(p, o.t, o.from + e * 64);
  uint32_t prefix = 0xffffffffu;   // only the ends stay
  int rest = 0, above = 0, equal = 0;
  if (o.t.want > 0) {
    const PartInfo in = o.ws.info[o.part];
    prefix = o.ws.verdict->prefix;
    rest = o.ws.verdict->rest;
    above = in.above;
    equal = in.equal;
  } else {   // the ends before this part
    const int at = o.part * kPart;
    above = min(at, p.sinks) + max(at - o.t.end, 0);
  }
  int na = 0, ne = 0;
#pragma unroll
  for (int e = 0; e < 4; e++) tally_key(k[e], prefix, na, ne);
  if (lane == 0) { s.above[wave] = na; s.equal[wave] = ne; }
  __syncthreads();
  for (int i = 0; i < wave; i++) { above += s.above[i]; equal += s.equal[i]; }
#pragma unroll
  for (int e = 0; e < 4; e++) place_key(p, o.t, o.from + e * 64, k[e], prefix, rest, above, equal);
}

__global__ void __launch_bounds__(kSelectThreads) weights_kernel(const EvictParams p) {
  const int item = blockIdx.x, b = item / p.c.heads, hk = item - b * p.c.heads;
  weights_in_place(p, item_of(p, b, hk), p.wout + b * p.osb + hk * p.osh);
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

__device__ __forceinline__ void or_word(Chunk<3>::type& w, int k, uint32_t v) { w.v[k] |= v; }
__device__ __forceinline__ void or_word(u4_t& w, int k, uint32_t v) { w[k] |= v; }

template <int D, int G>
__global__ void __launch_bounds__(256) gather_kernel(const EvictParams p) {
  constexpr int NK = D / 32, NV = D / 16, CK = kchunk(D), CV = vchunk(D);
  __shared__ const uint8_t* src[kBlock];
  __shared__ int tok[kBlock];
  unsigned id = blockIdx.x;
  const int blk = int(id % unsigned(p.blocks)); id /= unsigned(p.blocks);
  const int hk = int(id % unsigned(p.c.heads)), b = int(id / unsigned(p.c.heads));
  const int m = min(seq_len(p, b), p.keep);
  if (blk == 0 && hk == 0 && threadIdx.x == 0) p.out_lengths[b] = m;
  if (p.wout != p.w) {   // an equal part of the weights, each once
    const int64_t part = (p.max_len + p.blocks - 1) / p.blocks, to = min((blk + 1) * part, p.max_len);
    const float* w = p.w + b * p.wsb + hk * p.wsh;
    const int* kept = p.kept + (int64_t(b) * p.c.heads + hk) * p.keep;
    float* wo = p.wout + b * p.osb + hk * p.osh;
    for (int64_t i = blk * part + threadIdx.x; i < to; i += 256) wo[i] = i < m ? w[kept[i]] : 0.0f;
  }
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
  // Codes, a lane's chunk of up to 16 bytes at a time.  K: a chunk belongs to one
  // token.  V: every dword takes one nibble from each of its eight tokens.  A
  // token without a page is read from the block's first (and gives 0), so that
  // all loads are under way together.
  constexpr int KI = 2 * 64 * (NK / CK), VI = 64 * (NV / CV);
  typedef typename Chunk<CK>::type KW;
  typedef typename Chunk<CV>::type VW;
  const uint8_t* any = nullptr;
  for (int t = 0; t < kBlock && !any; t++) any = src[t];
  if (any) {
    for (int it = threadIdx.x; it < KI; it += 256) {
      const int lane = it & 63, c = (it >> 6) % (NK / CK), u = (it >> 6) / (NK / CK), t = u * 16 + (lane & 15);
      const uint8_t* s = src[t];
      KW w = *reinterpret_cast<const KW*>((s ? s : any) + kcode_at(D, G, tok[t] >> 4, (lane & 48) | (tok[t] & 15), c * CK));
      if (!s) w = KW{};
      *reinterpret_cast<KW*>(dst + kcode_at(D, G, u, lane, c * CK)) = w;
    }
    for (int it = threadIdx.x; it < VI; it += 256) {
      const int lane = it & 63, c = it >> 6, set = lane >> 4;
      VW w = {};
      VW x[8];
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const int t = vtoken(set, e);
        const uint8_t* s = src[t];
        x[e] = *reinterpret_cast<const VW*>((s ? s : any) + vcode_at(D, G, vset(tok[t]) * 16 + (lane & 15), c * CV));
      }
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const int t = vtoken(set, e), from = 4 * nibble(velem(tok[t]));
        const uint32_t keep = src[t] ? 15u : 0u;
#pragma unroll
        for (int k = 0; k < CV; k++) or_word(w, k, ((x[e][k] >> from) & keep) << (4 * nibble(e)));
      }
      *reinterpret_cast<VW*>(dst + vcode_at(D, G, lane, c * CV)) = w;
    }
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
    if (p.parts == 0) {
      const dim3 grid(heads), threads(kSelectThreads);
      if (p.max_len <= 4 * kSelectThreads) hipLaunchKernelGGL(select_kernel<4>, grid, threads, 0, st, p);
      else if (p.max_len <= 8 * kSelectThreads) hipLaunchKernelGGL(select_kernel<8>, grid, threads, 0, st, p);
      else hipLaunchKernelGGL(select_kernel<16>, grid, threads, 0, st, p);
    } else {
      const dim3 grid(unsigned(p.parts), heads), threads(kSelectThreads);
      hipLaunchKernelGGL(count_kernel, grid, threads, 0, st, p);
      hipLaunchKernelGGL(sort_kernel, grid, threads, 0, st, p);
      hipLaunchKernelGGL(settle_kernel, dim3(heads), threads, 0, st, p);
      hipLaunchKernelGGL(write_kernel, grid, threads, 0, st, p);
      if (p.wout == p.w) hipLaunchKernelGGL(weights_kernel, dim3(heads), threads, 0, st, p);
    }
    int s = launched();
    if (s != STAGQ_OK) return s;
    hipLaunchKernelGGL((gather_kernel<D, G>), dim3(heads * unsigned(p.blocks)), dim3(256), 0, st, p);
    s = launched();
    if (s != STAGQ_OK || !p.stage) return s;
    hipLaunchKernelGGL((place_kernel<D, G>), dim3(heads * unsigned(p.blocks)), dim3(256), 0, st, p);
    return launched();
  }
};

static int64_t parts_of(int64_t slots) { return slots <= kSmall ? 1 : (slots + kPart - 1) / kPart; }

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
  if (!disjoint(reach(c, q, e->max_len), q->batch, e->out_stride_seq, c->kv_heads, e->out_stride_head)) return STAGQ_EINVAL;
  if (e->weights == e->weights_out &&
      (e->weights_stride_seq != e->out_stride_seq || e->weights_stride_head != e->out_stride_head))
    return STAGQ_EINVAL;
  if (misaligned(e->weights, 4) || misaligned(e->weights_out, 4) || misaligned(e->kept, 4) ||
      misaligned(e->out_lengths, 4) || misaligned(e->out_table, 4))
    return STAGQ_EALIGN;
  if (e->out_table) {
    if (e->out_table == q->table) return STAGQ_EINVAL;   // the same pages: NULL is the call for that
    if (e->out_table_width < 0 || (q->batch > 1 && e->out_table_stride < e->out_table_width)) return STAGQ_EINVAL;
    if (int64_t(e->out_table_width) * c->page_tokens < (e->keep < reach(c, q, e->max_len) ? e->keep : reach(c, q, e->max_len)))
      return STAGQ_ESIZE;
  }
  const int64_t blocks = (int64_t(e->keep) + kBlock - 1) / kBlock;
  const int64_t heads = int64_t(q->batch) * c->kv_heads;
  const int64_t parts = parts_of(reach(c, q, e->max_len));
  if (!launchable(heads * blocks, 256) || !launchable(heads * parts, kSelectThreads)) return STAGQ_ESHAPE;
  if (parts > 1 && heads > 65535) return STAGQ_ESHAPE;   // y of the grid
  return STAGQ_OK;
}

// Tokens that can stay: keep, or all slots within reach.
static int evict_blocks(const stagq_kv_cache* c, const stagq_kv_seqs* q, const stagq_kv_evict_args* e) {
  const int64_t r = reach(c, q, e->max_len), m = e->keep < r ? e->keep : r;
  return int(m > 0 ? (m + kBlock - 1) / kBlock : 1);
}

// Workspace: the staged blocks of an eviction in place, then that of the parts.
static size_t stage_bytes(const stagq_kv_cache* c, const stagq_kv_seqs* q, const stagq_kv_evict_args* e) {
  if (e->out_table) return 0;
  const size_t n = size_t(q->batch) * c->kv_heads * size_t(evict_blocks(c, q, e)) * block_bytes(c->head_dim, c->head_dim / c->group);
  return (n + 255) / 256 * 256;
}
static size_t select_bytes(const stagq_kv_cache* c, const stagq_kv_seqs* q, const stagq_kv_evict_args* e) {
  const int64_t r = reach(c, q, e->max_len);
  return r <= kSmall ? 0 : size_t(q->batch) * c->kv_heads * parts_bytes(int(parts_of(r)));
}

}  // namespace kv
}  // namespace stagq

using namespace stagq::kv;

extern "C" {

size_t stagq_kv_evict_workspace(const stagq_kv_cache* c, const stagq_kv_seqs* q, const stagq_kv_evict_args* e) {
  if (check_evict(c, q, e) != STAGQ_OK) return 0;
  return stage_bytes(c, q, e) + select_bytes(c, q, e);
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
  p.parts = p.max_len <= kSmall ? 0 : int(parts_of(p.max_len));
  p.parts_ws = static_cast<uint8_t*>(workspace) + stage_bytes(c, q, e);
  return by_shape(c, LaunchEvict{p, static_cast<hipStream_t>(hip_stream)});
}

}  // extern "C"
