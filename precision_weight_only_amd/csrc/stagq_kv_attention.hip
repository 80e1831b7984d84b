// Attention over the key/value cache in 4 bits.
//
// Query rows of a sequence that share a kv head (tokens x q heads of the kv
// head, row = token * heads + head) run together.  For a row q and slot t with
// pairs (lo, s) and codes u per group g of channels,
//   q . k_t = sum_g  s_{t,g} (q . u_t)_g + lo_{t,g} (sum of q over g),
// so the codes go into the matrix instruction as they are (see codes8) and the
// pairs meet the 32-bit sums; likewise with probabilities p_t
//   out_c = sum_t (p_t s_{t,g(c)}) u_{t,c} + sum_t p_t lo_{t,g(c)}.
// One pass over the slots with a running reference r per row, p_t = 2^(z_t - r)
// (z in binary orders: scale log2 e folded in), and the sums of p, p lo and
// p s u in binary32; they are multiplied by 2^(old r - new r) when r moves.
#include "stagq_kv_host.h"

namespace stagq {
namespace kv {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNone = -1e30f;  // reference of a row that has seen nothing
constexpr int kRowTile = 16;
constexpr int kWantedGroups = 512;  // two workgroups per CU
// Blocks of a split of attend_rows where the grid is filled twice, and workgroups
// up to which they may be fewer (a block per wave): 16 rows of 2000 slots take 10
// against 11 us, 32 rows of 4 x 1000 16 against 19 us; but fewer everywhere,
// 32 rows of 4 x 2000 28 against 20 us and 16 rows of 8000 14 against 12 us.
constexpr int kMinBlocks = 8, kSingleGroups = 256;
// Rules of plan(), measured with 8 kv heads of 128 channels unless said otherwise.
// Blocks of a split of attend_tiles: 8 against 16 took 49 against 54 us with 256
// rows of 12001 slots and 22 against 31 us with 128 rows of 2000, but 55 against
// 50 us with 1024 rows of 2000; 32 took 60, 49 and 65 us.
constexpr int kMinTileBlocks = 8;
// Rows beyond which attend_tiles takes over from attend_rows, without and with
// weights (whose second pass after attend_rows, weigh_kernel, is the slower one
// there): 20 rows of 8192 slots take 16 us in attend_rows and 29 us in
// attend_tiles; 64 rows 22 and 24 us, of 16 sequences of 2000 slots 52 and 55 us;
// 128 rows of those 58 and 71 us, but of 8192 slots and with 256 channels
// attend_tiles is as fast or faster.  With weights 32 rows take 24 and 38 us of
// 8192 slots, 63 and 58 us of 16 x 2000, and 64 rows 33 and 35, 97 and 80 us.
constexpr int kManyRows = 64, kManyRowsWeighed = 32;
// Up to this many rows z is kept for the weights: of 2, 4 and 8 rows of 32 x 2000
// slots 29, 31 and 35 us, 69, 69 and 72 us if it is computed again.
constexpr int kStashRows = 8;
// attend_few, steps of 64 slots: an item has a workgroup of its own up to
// kOwnSteps steps (a sequence of 12 steps 10.8 us, one of 16 13.1 us and shared
// 11.4 us, one of 24 shared 11.5 us), and up to one step per kItemsPerStep items
// (128 sequences of 2000 slots, 32 steps: 63 against 67 us, ragged 43 against 51;
// 32 sequences: 23 against 27 and 22 against 24 us; but 4 sequences 21 against
// 18 us).
constexpr int kOwnSteps = 12, kItemsPerStep = 8;

struct AttnParams {
  Cache c;
  Tensor q, out;
  const int* q_lens;
  float* lse;
  float* weights;
  int64_t wsb, wsh;
  float* part;      // sums of the parts of rows, [part row][D]
  float* part_rl;   // and their references and sums of p, [part row][2]
  float scale2;     // scale * log2 e
  unsigned gq, gq_inv;  // q heads per kv head, and floor(2^32 / gq), at most 2^32 - 1
  int causal, window, zero_rest;
  float* stash;     // or z (binary orders) of [batch][kv head][row][stash_len]
  int64_t stash_len;
  uint8_t* q_frags; // or the query operands of attend_tiles, [batch][kv head][16 rows][D / 32 + 1] KB
  float* q_units;   // and what their products are multiplied by, per row
  int64_t q_tiles;  // 16-row tiles per sequence and head
  int64_t max_len;
  int chunk;        // slots of a split
  int nsplit, tiles, tile_rows;
  int rows;         // tokens * gq
  int shared;       // attend_few: workgroups that share all steps evenly; 0: one per sequence and head
  int2* where;      // then, by sequence and head: its first part and their number
};

// The token of a row: row / gq, from the reciprocal, which is at most one short.
__device__ __forceinline__ int token_of(const AttnParams& p, int row) {
  const unsigned q = __umulhi(unsigned(row), p.gq_inv);
  return int(unsigned(row) - q * p.gq >= p.gq ? q + 1 : q);
}

// What a sequence and a tile of rows see: slots [lo, hi), lo down to two blocks.
struct Span {
  int64_t len;
  int ql, rows;     // query tokens and rows of the sequence
  int64_t lo, hi;
};
__device__ __forceinline__ void seq_span(const AttnParams& p, int length, int q_len, Span& s) {
  const int64_t len = length;
  s.len = len < 0 ? 0 : len > p.max_len ? p.max_len : len;
  s.ql = min(max(q_len, 0), p.q.tokens);
  s.rows = s.ql * int(p.gq);
}
__device__ __forceinline__ int q_len_of(const AttnParams& p, int b) { return p.q_lens ? p.q_lens[b] : p.q.tokens; }
__device__ __forceinline__ void seq_span(const AttnParams& p, int b, Span& s) {
  seq_span(p, p.c.lengths[b], q_len_of(p, b), s);
}
__device__ __forceinline__ void tile_span(const AttnParams& p, int row0, Span& s) {
  const int last = min(row0 + p.tile_rows, s.rows) - 1;
  const int64_t first_pos = s.len - s.ql + token_of(p, row0), last_pos = s.len - s.ql + token_of(p, last);
  s.hi = p.causal ? max(min(last_pos + 1, s.len), int64_t(0)) : s.len;
  s.lo = p.window > 0 ? max(first_pos - p.window + 1, int64_t(0)) & ~int64_t(2 * kBlock - 1) : 0;
}
__device__ __forceinline__ int used_splits(const AttnParams& p, const Span& s) {
  return s.hi <= s.lo ? 0 : int((s.hi - s.lo + p.chunk - 1) / p.chunk);
}
// Slots [from, to) that a row sees.
__device__ __forceinline__ void row_span(const AttnParams& p, const Span& s, int row, int64_t& from, int64_t& to) {
  const int64_t pos = s.len - s.ql + token_of(p, row);
  to = p.causal ? min(pos + 1, s.len) : s.len;
  from = p.window > 0 ? max(pos - p.window + 1, int64_t(0)) : 0;
}

__device__ __forceinline__ const uint8_t* q_row(const AttnParams& p, int b, int hk, int row) {
  const int t = token_of(p, row), h = (hk - t) * int(p.gq) + row;
  return p.q.data + (b * p.q.sb + t * p.q.st + h * p.q.sh) * 2;
}
__device__ __forceinline__ uint16_t* out_row(const AttnParams& p, int b, int hk, int row) {
  const int t = token_of(p, row), h = (hk - t) * int(p.gq) + row;
  return reinterpret_cast<uint16_t*>(p.out.data) + (b * p.out.sb + t * p.out.st + h * p.out.sh);
}
__device__ __forceinline__ void put_lse(const AttnParams& p, int b, int hk, int row, float ref, float sum) {
  const int t = token_of(p, row), h = (hk - t) * int(p.gq) + row;
  const float v = sum == 0.0f ? -__builtin_inff() : (ref + __log2f(sum)) * kLn2;
  p.lse[(int64_t(b) * p.q.tokens + t) * p.q.heads + h] = v;
}
__device__ __forceinline__ int64_t part_row(const AttnParams& p, int b, int hk, int split, int row) {
  return ((int64_t(b) * p.c.heads + hk) * p.nsplit + split) * p.rows + row;
}

// Four channels of a row's result from its sums.
__device__ __forceinline__ void put_out(const AttnParams& p, int b, int hk, int row, int c, f4_t o, float sum) {
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  u2_t w;
  w[0] = uint32_t(to_16(o[0] * inv, p.q.dtype)) | uint32_t(to_16(o[1] * inv, p.q.dtype)) << 16;
  w[1] = uint32_t(to_16(o[2] * inv, p.q.dtype)) | uint32_t(to_16(o[3] * inv, p.q.dtype)) << 16;
  *reinterpret_cast<u2_t*>(out_row(p, b, hk, row) + c) = w;
}
template <int D>
__device__ __forceinline__ void zero_rows(const AttnParams& p, int b, int hk, int row, int end) {
  for (int it = threadIdx.x; it < (end - row) * (D / 4); it += blockDim.x)
    *reinterpret_cast<u2_t*>(out_row(p, b, hk, row + it / (D / 4)) + (it % (D / 4)) * 4) = u2_t{0u, 0u};
}

// Query rows as operands.  fp16 rows go in as they are.  bf16 rows are scaled by
// a power of two per row (see row_scale) and rounded to fp16; the result undoes
// the scale.  All loads are issued before the first is used.
template <int N>
__device__ __forceinline__ float amax_bf16(const u4_t* raw) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i++)
#pragma unroll
    for (int e = 0; e < 8; e++) amax = fmaxf(amax, fabsf(bf16_of(raw[i], e)));
  return amax;
}
template <int N>
__device__ __forceinline__ void bf16_to_half(const u4_t* raw, float m, h8_t* out) {
#pragma unroll
  for (int i = 0; i < N; i++)
#pragma unroll
    for (int e = 0; e < 8; e++) out[i][e] = (_Float16)(bf16_of(raw[i], e) * m);
}
// Sum of N times eight values as rounded, exact products into binary32.
template <int N>
__device__ __forceinline__ float sum8(const h8_t* q) {
  const h2_t one = {(_Float16)1.0f, (_Float16)1.0f};
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i++) {
    a = __builtin_amdgcn_fdot2(__builtin_shufflevector(q[i], q[i], 0, 1), one, a, false);
    a = __builtin_amdgcn_fdot2(__builtin_shufflevector(q[i], q[i], 2, 3), one, a, false);
    a = __builtin_amdgcn_fdot2(__builtin_shufflevector(q[i], q[i], 4, 5), one, a, false);
    a = __builtin_amdgcn_fdot2(__builtin_shufflevector(q[i], q[i], 6, 7), one, a, false);
  }
  return a;
}
// A lane's share of a 16-row tile: row n = lane & 15, channels 32 ks + 8 (lane >> 4) + e.
template <int D>
__device__ __forceinline__ void load_q(const AttnParams& p, int b, int hk, int row, bool there, h8_t* qf, float* unit) {
  constexpr int NK = D / 32;
  const int set = (threadIdx.x & 63) >> 4;
  u4_t raw[NK];
  const uint8_t* src = q_row(p, b, hk, there ? row : 0);
#pragma unroll
  for (int ks = 0; ks < NK; ks++) {
    raw[ks] = u4_t{0u, 0u, 0u, 0u};
    if (there) raw[ks] = *reinterpret_cast<const u4_t*>(src + (32 * ks + 8 * set) * 2);
  }
  *unit = 1.0f;
  if (p.q.dtype == STAGQ_F16) {
#pragma unroll
    for (int ks = 0; ks < NK; ks++) qf[ks] = __builtin_bit_cast(h8_t, raw[ks]);
  } else {
    const float m = row_scale(max_sets(amax_bf16<NK>(raw)));
    bf16_to_half<NK>(raw, m, qf);
    *unit = 1.0f / m;
  }
}

// The waves' sums of a tile of ROWS rows meet in LDS: [wave][row][D + 4] floats,
// then the references and sums of p, [wave][row] each.
constexpr uint32_t join_bytes(int waves, int rows, int D) { return uint32_t(waves * rows * (D + 4 + 2) * 4); }
__device__ __forceinline__ void join_refs(float* sums, int waves, int rows, int D, int wave, int row, float ref, float l) {
  float* refs = sums + waves * rows * (D + 4);
  refs[wave * rows + row] = ref;
  refs[(waves + wave) * rows + row] = l;
}
// Add them up in a fixed order and write the rows from row0 on: the result where
// `all` slots of the rows are in, else the part that starts at part row `at`.
template <int D, int NW, int ROWS>
__device__ __forceinline__ void join_waves(const AttnParams& p, const Span& s, const float* sums, int b, int hk, int row0,
                                           bool all, int64_t at) {
  constexpr int LD = D + 4;
  const float* refs = sums + NW * ROWS * LD;
  const float* ls = refs + NW * ROWS;
  for (int it = threadIdx.x; it < ROWS * (D / 4); it += NW * 64) {
    const int r = it / (D / 4), c = (it % (D / 4)) * 4, row = row0 + r;
    if (row >= s.rows) {
      if (p.zero_rest && all && row < p.rows)
        *reinterpret_cast<u2_t*>(out_row(p, b, hk, row) + c) = u2_t{0u, 0u};
      continue;
    }
    float m = refs[r], l = 0.0f;
#pragma unroll
    for (int w = 1; w < NW; w++) m = fmaxf(m, refs[w * ROWS + r]);
    f4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < NW; w++) {
      const float f = exp2_fast(refs[w * ROWS + r] - m);
      l = fmaf(ls[w * ROWS + r], f, l);
      o += *reinterpret_cast<const f4_t*>(sums + (w * ROWS + r) * LD + c) * f;
    }
    if (all) {
      put_out(p, b, hk, row, c, o, l);
      if (p.lse && c == 0) put_lse(p, b, hk, row, m, l);
    } else {
      *reinterpret_cast<f4_t*>(p.part + (at + r) * D + c) = o;
    }
    if (p.part_rl && c == 0) { p.part_rl[(at + r) * 2] = m; p.part_rl[(at + r) * 2 + 1] = l; }
  }
}

// p s goes into fp16: the reference lies `lift` below the row's largest z, so
// that the largest step seen times 2^lift is near 2^8 (limit 2^15).  Then a
// product is lost only 2^-33 below the largest, whatever the scale of V.  smax:
// largest step of what comes next, the same in all lanes.
__device__ __forceinline__ void lift_of(float smax, float& lift, float& s_limit) {
  if (smax > s_limit) {
    const int e = (__builtin_bit_cast(int, fmaxf(smax, 5.9604645e-8f)) >> 23) - 127;   // 2^e <= smax
    lift = float(8 - e);
    s_limit = exp2_fast(float(e + 7));
  }
}

// ------------------------------------------------- few rows per kv head ----
// A tile is NQ x 16 rows; a workgroup takes one split of the slots, its waves
// every NW-th block of 32.  A wave keeps its rows' q and sums in registers and
// moves blocks through a ring of its own in LDS: the block is one contiguous
// piece in operand order, so it is copied there by direct loads that hold no
// registers while they are under way, DEPTH - 1 blocks ahead.  No barrier in
// the loop: a wave waits for its own loads only.
constexpr int ring_waves(int D) { return D == 256 ? 2 : 4; }
template <int D, int G>
struct Ring {
  static constexpr int NW = ring_waves(D);
  static constexpr uint32_t BB = block_bytes(D, G);
  static constexpr int DEPTH = D == 64 ? 4 : 3;              // a workgroup's rings fit in 64 KB, two of them in a CU
  static constexpr int LOADS = int((BB + 1023) / 1024);      // of a wave per block
  static constexpr uint32_t BYTES = NW * DEPTH * BB;
};

// Copy a block to LDS (byte offset `to`, the same in all lanes): every load
// instruction moves 1 KB, lane l's 16 bytes to `to` + 16 l.
// STREAM: read once, the non-temporal policy.
template <uint32_t BB, bool STREAM = true>
__device__ __forceinline__ void copy_block(const uint8_t* from, uint32_t to, int lane) {
  const uint8_t* mine = from + lane * 16;
#pragma unroll
  for (uint32_t i = 0; i < BB; i += 1024) {
    if (BB - i >= 1024 || uint32_t(lane) * 16 < BB - i) {
      if (STREAM)
        asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off nt"
                     : : "v"(mine + i), "s"(to + i) : "memory", "m0");
      else
        asm volatile("s_mov_b32 m0, %1\n\tglobal_load_lds_dwordx4 %0, off"
                     : : "v"(mine + i), "s"(to + i) : "memory", "m0");
    }
  }
}
template <int N>
__device__ __forceinline__ void wait_loads() {   // until at most N loads of the wave are under way
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

template <int D, int G, int NQ>
__global__ void __launch_bounds__(ring_waves(D) * 64, D == 256 || (G == 4 && NQ == 2) ? 1 : 2) attend_rows(const AttnParams p) {
  typedef Ring<D, G> R;
  constexpr int NK = D / 32, NV = D / 16, KG = NK / G, VG = NV / G, NW = R::NW, DEPTH = R::DEPTH;
  constexpr int CK = kchunk(D), CV = vchunk(D);
  constexpr int LD = D + 4;
  constexpr uint32_t JOIN = join_bytes(NW, kRowTile, D);
  __shared__ __attribute__((aligned(16))) uint8_t lds[R::BYTES > JOIN ? R::BYTES : JOIN];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, set = lane >> 4;
  const int split = blockIdx.x, b = blockIdx.z;
  const int tile = p.tiles == 1 ? 0 : blockIdx.y / unsigned(p.c.heads), hk = blockIdx.y - tile * p.c.heads;
  Span s;
  seq_span(p, b, s);
  const int row0 = tile * NQ * kRowTile;
  if (row0 >= s.rows) {
    if (p.zero_rest && p.nsplit == 1) zero_rows<D>(p, b, hk, row0, min(row0 + NQ * kRowTile, p.rows));
    return;
  }
  tile_span(p, row0, s);
  const int used = used_splits(p, s);
  if (split >= used && p.nsplit > 1) return;   // an only split writes the zeros of a tile that sees nothing
  const int64_t begin = s.lo + int64_t(split) * p.chunk, end = min(begin + p.chunk, s.hi);
  const int nblk = end > begin ? int((end - begin + kBlock - 1) / kBlock) : 0;
  const int mine = nblk > wave ? (nblk - wave + NW - 1) / NW : 0;

  // lane i holds the page of the wave's block i; -1: none
  int page = -1;
  {
    const int64_t slot = begin + int64_t(wave + lane * NW) * kBlock;
    const int64_t e = slot >> p.c.shift;
    if (lane < mine && e < p.c.width) page = p.c.table[int64_t(b) * p.c.table_stride + e];
    if (page >= p.c.pages) page = -1;
  }
  const int64_t in_page = (int64_t(1) << p.c.shift) - 1;
  const uint32_t ring = uint32_t(uintptr_t((__attribute__((address_space(3))) void*)lds)) + uint32_t(wave) * DEPTH * R::BB;
  // A block without a page is copied from page 0 all the same (the count of
  // loads under way stays known) and then left out.
  auto fetch = [&](int i) {
    const int pg = max(__builtin_amdgcn_readlane(page, i), 0);
    const int64_t slot = begin + int64_t(wave + i * NW) * kBlock;
    copy_block<R::BB>(p.c.buf + uint64_t(pg) * p.c.page_bytes + uint64_t(hk) * p.c.head_bytes +
                          uint32_t((slot & in_page) / kBlock) * R::BB,
                      ring + uint32_t(i % DEPTH) * R::BB, lane);
  };
#pragma unroll
  for (int i = 0; i < DEPTH - 1; i++)
    if (i < mine) fetch(i);

  h8_t qf[NQ][NK];
  float qsum[NQ][G], z_unit[NQ], ref[NQ], top[NQ], psum[NQ], plo[NQ][G];
  int64_t from[NQ], to[NQ];
  f4_t acc[NQ][NV];
#pragma unroll
  for (int t = 0; t < NQ; t++) {
    const int row = row0 + t * kRowTile + n;
    const bool there = row < s.rows;
    float unit;
    load_q<D>(p, b, hk, row, there, qf[t], &unit);
    z_unit[t] = p.scale2 * kCodeUnit * unit;
#pragma unroll
    for (int g = 0; g < G; g++) {
      qsum[t][g] = sum_sets(sum8<KG>(qf[t] + g * KG)) * (1.0f / kCodeUnit);
      plo[t][g] = 0.0f;
    }
    from[t] = to[t] = 0;
    if (there) row_span(p, s, row, from[t], to[t]);
    ref[t] = top[t] = kNone;
    psum[t] = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; c++) acc[t][c] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // slots that every row of the tile sees: [all_from, all_to)
  int64_t all_from = 0, all_to = s.len;
  {
    int64_t f, t;
    row_span(p, s, row0, f, t);
    all_to = t;
    row_span(p, s, min(row0 + NQ * kRowTile, s.rows) - 1, f, t);
    all_from = f;
  }
  float lift = 0.0f, s_limit = -1.0f;
  float* stash = nullptr;   // z of row n, if it is kept for the weights
  if (NQ == 1 && p.stash && row0 + n < s.rows)
    stash = p.stash + ((int64_t(b) * p.c.heads + hk) * p.rows + row0 + n) * p.stash_len;

#pragma unroll 1
  for (int i = 0; i < mine; i++) {
    if (i + DEPTH - 1 < mine) {
      fetch(i + DEPTH - 1);
      wait_loads<R::LOADS * (DEPTH - 1)>();
    } else {
      wait_loads<0>();
    }
    const int64_t slot0 = begin + int64_t(wave + i * NW) * kBlock;
    if (__builtin_amdgcn_readlane(page, i) < 0) {
      if (stash) {
        const f4_t none = {-__builtin_inff(), -__builtin_inff(), -__builtin_inff(), -__builtin_inff()};
        *reinterpret_cast<f4_t*>(stash + slot0 + 4 * set) = none;
        *reinterpret_cast<f4_t*>(stash + slot0 + 16 + 4 * set) = none;
      }
      continue;
    }
    const uint8_t* blk = lds + (wave * DEPTH + i % DEPTH) * R::BB;
    const bool whole = slot0 >= all_from && slot0 + kBlock <= all_to;
    u4_t vs[G], vl[G];
#pragma unroll
    for (int g = 0; g < G; g++) {
      vs[g] = *reinterpret_cast<const u4_t*>(blk + vstep_at(G, set, 0, g));
      vl[g] = *reinterpret_cast<const u4_t*>(blk + vstep_at(G, set, 0, g) + 16);
    }
    if (!whole) {   // pairs of slots that hold nothing yet may be anything
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (slot0 + vtoken(set, e) >= s.len)
#pragma unroll
          for (int g = 0; g < G; g++) {
            const uint32_t keep = (e & 1) ? 0x0000ffffu : 0xffff0000u;
            vs[g][e / 2] &= keep;
            vl[g][e / 2] &= keep;
          }
    }
    float smax;
    {
      h2_t m = {(_Float16)0.0f, (_Float16)0.0f};
#pragma unroll
      for (int g = 0; g < G; g++)
#pragma unroll
        for (int e = 0; e < 4; e++) m = __builtin_elementwise_max(m, __builtin_bit_cast(h2_t, (uint32_t)vs[g][e]));
      smax = fmaxf((float)m[0], (float)m[1]);
    }
    float z[NQ][8];
#pragma unroll
    for (int u = 0; u < 2; u++) {
      h8_t kf[NK];
#pragma unroll
      for (int k = 0; k < NK / CK; k++) {
        const auto w = *reinterpret_cast<const typename Chunk<CK>::type*>(blk + kcode_at(D, G, u, lane, k * CK));
#pragma unroll
        for (int x = 0; x < CK; x++) kf[k * CK + x] = codes8(w[x]);
      }
      u4_t kp[G];
#pragma unroll
      for (int g = 0; g < G; g++) kp[g] = *reinterpret_cast<const u4_t*>(blk + kpair_at(G, 16 * u + 4 * set, g));
#pragma unroll
      for (int t = 0; t < NQ; t++) {
        float zz[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int g = 0; g < G; g++) {
          f4_t a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int ks = g * KG; ks < (g + 1) * KG; ks++)
            a = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[ks], qf[t][ks], a, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; r++) {
            const h2_t pair = __builtin_bit_cast(h2_t, (uint32_t)kp[g][r]);
            zz[r] = fmaf((float)pair[1], a[r], zz[r]);
            zz[r] = fmaf((float)pair[0], qsum[t][g], zz[r]);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; r++) z[t][u * 4 + r] = zz[r] * z_unit[t];
      }
    }
    if (!whole) {
#pragma unroll
      for (int t = 0; t < NQ; t++)
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const int64_t slot = slot0 + vtoken(set, e);
          z[t][e] = slot >= from[t] && slot < to[t] ? z[t][e] : -__builtin_inff();
        }
    }
    if (NQ == 1 && stash) {
      const f4_t a = {z[0][0], z[0][1], z[0][2], z[0][3]}, c = {z[0][4], z[0][5], z[0][6], z[0][7]};
      *reinterpret_cast<f4_t*>(stash + slot0 + 4 * set) = a;
      *reinterpret_cast<f4_t*>(stash + slot0 + 16 + 4 * set) = c;
    }
    bool moves = smax > s_limit;
    float mx[NQ];
#pragma unroll
    for (int t = 0; t < NQ; t++) {
      mx[t] = fmaxf(fmaxf(fmaxf(z[t][0], z[t][1]), fmaxf(z[t][2], z[t][3])),
                    fmaxf(fmaxf(z[t][4], z[t][5]), fmaxf(z[t][6], z[t][7])));
      moves |= mx[t] > top[t];
    }
    if (__any(moves)) {   // rare: the reference of some row moves
      float sm = max_sets(smax);
#pragma unroll
      for (int d = 1; d < 16; d *= 2) sm = fmaxf(sm, __shfl_xor(sm, d));
      lift_of(sm, lift, s_limit);
#pragma unroll
      for (int t = 0; t < NQ; t++) {
        top[t] = fmaxf(top[t], max_sets(mx[t]));
        const float r = top[t] - lift, f = exp2_fast(ref[t] - r);
        ref[t] = r;
        psum[t] *= f;
#pragma unroll
        for (int g = 0; g < G; g++) plo[t][g] *= f;
#pragma unroll
        for (int c = 0; c < NV; c++) acc[t][c] *= f;
      }
    }
#pragma unroll
    for (int t = 0; t < NQ; t++)
#pragma unroll
      for (int e = 0; e < 8; e++) {
        z[t][e] = exp2_fast(z[t][e] - ref[t]);   // p from here on
        psum[t] += z[t][e];
      }
    typename Chunk<CV>::type w[NV / CV];
#pragma unroll
    for (int k = 0; k < NV / CV; k++)
      w[k] = *reinterpret_cast<const typename Chunk<CV>::type*>(blk + vcode_at(D, G, lane, k * CV));
    // p s as the sum of two fp16 (22 bits): one alone costs more than the
    // rounding of an fp16 result, since the code part is cancelled by p lo.
#pragma unroll
    for (int g = 0; g < G; g++) {
      const h8_t sv = __builtin_bit_cast(h8_t, vs[g]), lv = __builtin_bit_cast(h8_t, vl[g]);
      h8_t hi[NQ], rest[NQ];
#pragma unroll
      for (int t = 0; t < NQ; t++)
#pragma unroll
        for (int e = 0; e < 8; e++) {
          plo[t][g] = fmaf(z[t][e], (float)lv[e], plo[t][g]);
          const float ps = z[t][e] * (float)sv[e];
          hi[t][e] = (_Float16)ps;
          rest[t][e] = (_Float16)(ps - (float)hi[t][e]);
        }
#pragma unroll
      for (int c = g * VG; c < (g + 1) * VG; c++) {
        const h8_t vf = codes8(w[c / CV][c % CV]);
#pragma unroll
        for (int t = 0; t < NQ; t++) {
          acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, hi[t], acc[t][c], 0, 0, 0);
          acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, rest[t], acc[t][c], 0, 0, 0);
        }
      }
    }
  }

  float* sums = reinterpret_cast<float*>(lds);
  for (int t = 0; t < NQ; t++) {
    __syncthreads();
    const float l = sum_sets(psum[t]);
    float lo[G];
#pragma unroll
    for (int g = 0; g < G; g++) lo[g] = sum_sets(plo[t][g]);
#pragma unroll
    for (int c = 0; c < NV; c++) {
      f4_t o;
#pragma unroll
      for (int r = 0; r < 4; r++) o[r] = fmaf(acc[t][c][r], kCodeUnit, lo[c / VG]);
      *reinterpret_cast<f4_t*>(sums + (wave * kRowTile + n) * LD + 16 * c + 4 * set) = o;
    }
    if (set == 0) join_refs(sums, NW, kRowTile, D, wave, n, ref[t], l);
    __syncthreads();
    join_waves<D, NW, kRowTile>(p, s, sums, b, hk, row0 + t * kRowTile, p.nsplit == 1,
                                part_row(p, b, hk, split, row0 + t * kRowTile));
  }
}

// ------------------------------------------ up to four rows per kv head ----
// The decode step of most models: one token, at most four q heads per kv head.
// In attend_rows twelve of the sixteen columns would idle and its vector work
// (58 % of the cycles at 131001 slots; matrix 12 %) would bound it.  Here the
// matrix instruction is the one of sixteen 4 x 4 x 4 products: four rows against
// 64 slots (lane = slot for K, then four slots of row lane & 3 per lane), and
// for V the product of one set of four slots, its probabilities broadcast from
// the four lanes that hold them, with 64 channels (lane = channel).  Per 64
// slots that is a quarter of the vector work outside the unpacking of codes,
// at the same matrix cycles.
// Waves, rings and the running reference as in attend_rows; a step is two
// blocks, and the next step's are under way.
constexpr int few_waves(int D) { return D == 256 ? 2 : 4; }
constexpr int kFewRows = 4;
constexpr int kFewDepth = 4;   // blocks of a ring

// Steps of a sequence, the same for all its kv heads.
__device__ __forceinline__ int few_steps(const AttnParams& p, Span& s) {
  if (s.rows == 0) { s.lo = s.hi = 0; return 0; }
  tile_span(p, 0, s);
  return s.hi <= s.lo ? 0 : int((s.hi - s.lo + 2 * kBlock - 1) / (2 * kBlock));
}
__device__ __forceinline__ int few_steps(const AttnParams& p, int b) {
  Span s;
  seq_span(p, b, s);
  return few_steps(p, s);
}
__device__ __forceinline__ int prefix64(int v) {   // inclusive, over the wave
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    if (int(threadIdx.x & 63) >= d) v += o;
  }
  return v;
}
// Where lengths differ, the host (which does not know them) cannot cut the work
// evenly: all steps of all sequences and heads are numbered, and workgroup w
// takes the `quota` from w quota on, across heads and sequences.  Beginning an
// item (sequence, head) takes as long as some steps: it is charged kItemCost
// numbers after its last step (without them a workgroup that met ten heads of a
// one-token sequence took 59 us where the others took 15).  An item that starts
// at number `first` and has n > 0 steps is in the workgroups first / quota ..
// (first + n - 1) / quota, and its part in workgroup w is part w + item, which
// no two parts share.
// At least a step per wave: one sequence of 2000 slots takes 11.5 us, with 8 13.7
// and with 16 17.4 us (of 8000 13.6, 14.7 and 19 us, of 32000 all 19 us).
constexpr int kMinQuota = 4;
constexpr int kItemCost = 8;
__device__ __forceinline__ int few_cost(const AttnParams& p, int b) {
  const int n = few_steps(p, b);
  return n > 0 ? n + kItemCost : 0;
}
// Numbers of all sequences.
__device__ __forceinline__ int few_total(const AttnParams& p) {
  int sum = 0;
  for (int b0 = 0; b0 < p.c.batch; b0 += 64) {
    const int b = b0 + (threadIdx.x & 63);
    int v = b < p.c.batch ? few_cost(p, b) * p.c.heads : 0;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    sum += __builtin_amdgcn_readfirstlane(v);
  }
  return sum;
}

// LDS of attend_few: the waves' rings (later their sums), then a copy of the
// query rows per wave.
template <int D, int G>
struct FewLds {
  static constexpr uint32_t RING = few_waves(D) * kFewDepth * block_bytes(D, G);
  static constexpr uint32_t JOIN = join_bytes(few_waves(D), kFewRows, D);
  static constexpr uint32_t Q = RING > JOIN ? RING : JOIN;
  static constexpr uint32_t BYTES = Q + few_waves(D) * kFewRows * D * 2;
};

// `steps` steps from step `first` of one sequence and kv head.
template <int D, int G>
__device__ __forceinline__ void few_segment(const AttnParams& p, const Span& s, int b, int hk, int first, int steps, bool all,
                                            int64_t at_part, uint8_t* lds) {
  constexpr int NW = few_waves(D), NK = D / 32, NH = D / 64, KG = NK / G, CK = kchunk(D), LD = D + 4;
  constexpr uint32_t BB = block_bytes(D, G);
  constexpr int LOADS = 2 * int((BB + 1023) / 1024);   // of a wave per step
  // (opaque, so that what hangs on it is not kept in registers across segments)
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int j = lane & 3, quad = lane >> 2;   // row, and set of four slots of the step
  const int64_t begin = s.lo + int64_t(first) * 2 * kBlock, end = min(begin + int64_t(steps) * 2 * kBlock, s.hi);
  const int mine = steps > wave ? (steps - wave + NW - 1) / NW : 0;

  // lane i holds the page of the wave's block i (two per step); -1: none
  int page = -1;
  {
    const int64_t slot = begin + int64_t((wave + (lane >> 1) * NW) * 2 + (lane & 1)) * kBlock;
    const int64_t e = slot >> p.c.shift;
    if ((lane >> 1) < mine && slot < end && e < p.c.width) page = p.c.table[int64_t(b) * p.c.table_stride + e];
    if (page >= p.c.pages) page = -1;
  }
  const int64_t in_page = (int64_t(1) << p.c.shift) - 1;
  const uint32_t ring = uint32_t(uintptr_t((__attribute__((address_space(3))) void*)lds)) + uint32_t(wave) * kFewDepth * BB;
  auto fetch = [&](int i) {   // a block without a page is copied from page 0 and left out
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int pg = max(__builtin_amdgcn_readlane(page, 2 * i + h), 0);
      const int64_t slot = begin + int64_t((wave + i * NW) * 2 + h) * kBlock;
      copy_block<BB>(p.c.buf + uint64_t(pg) * p.c.page_bytes + uint64_t(hk) * p.c.head_bytes +
                         uint32_t((slot & in_page) / kBlock) * BB,
                     ring + uint32_t((2 * i + h) % kFewDepth) * BB, lane);
    }
  };
  if (mine > 0) fetch(0);

  // The rows come in once per wave, CH lanes a row, are scaled (bf16) and turned
  // through LDS: lane j + 4 n then holds row j.
  constexpr int CH = D / 8, LOADQ = kFewRows * CH > 64 ? kFewRows * CH / 64 : 1;
  h8_t qf[CH];
  float qsum[G], z_unit = p.scale2 * kCodeUnit;
  const bool there = j < s.rows;
  {
    h8_t* stage = reinterpret_cast<h8_t*>(lds + FewLds<D, G>::Q) + wave * kFewRows * CH;
    u4_t raw[LOADQ];
#pragma unroll
    for (int i = 0; i < LOADQ; i++) {
      const int row = (i * 64 + lane) / CH, ch = lane % CH;
      raw[i] = u4_t{0u, 0u, 0u, 0u};
      if (row < min(s.rows, kFewRows)) raw[i] = *reinterpret_cast<const u4_t*>(q_row(p, b, hk, row) + ch * 16);
    }
    float unit[kFewRows];
#pragma unroll
    for (int i = 0; i < LOADQ; i++) {
      const int row = (i * 64 + lane) / CH, ch = lane % CH;
      h8_t h = __builtin_bit_cast(h8_t, raw[i]);
      float m = 1.0f;
      if (p.q.dtype != STAGQ_F16) {
        float amax = amax_bf16<1>(&raw[i]);
#pragma unroll
        for (int d = 1; d < CH; d *= 2) amax = fmaxf(amax, __shfl_xor(amax, d));
        m = row_scale(amax);
        bf16_to_half<1>(&raw[i], m, &h);
      }
#pragma unroll
      for (int r = i * 64 / CH; r < (i + 1) * 64 / CH && r < kFewRows; r++)
        unit[r] = 1.0f / __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, m), r * CH - i * 64));
      if (row < kFewRows) stage[row * CH + ch] = h;
    }
    z_unit *= j == 0 ? unit[0] : j == 1 ? unit[1] : j == 2 ? unit[2] : unit[3];
#pragma unroll
    for (int c = 0; c < CH; c++) qf[c] = stage[j * CH + c];
  }
#pragma unroll
  for (int g = 0; g < G; g++) qsum[g] = sum8<CH / G>(qf + g * (CH / G)) * (1.0f / kCodeUnit);
  int64_t from = 0, to = 0;
  if (there) row_span(p, s, j, from, to);
  int64_t all_from, all_to;   // slots that every row sees
  {
    int64_t f, t;
    row_span(p, s, 0, f, all_to);
    row_span(p, s, s.rows - 1, all_from, t);
  }
  float* stash = nullptr;
  if (p.stash && there) stash = p.stash + ((int64_t(b) * p.c.heads + hk) * p.rows + j) * p.stash_len;

  float ref = kNone, top = kNone, psum = 0.0f, plo[G], lift = 0.0f, s_limit = -1.0f;
  f4_t acc[NH], more[NH];   // of the two parts of p s
#pragma unroll
  for (int g = 0; g < G; g++) plo[g] = 0.0f;
#pragma unroll
  for (int h = 0; h < NH; h++) acc[h] = more[h] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll 1
  for (int i = 0; i < mine; i++) {
    if (i + 1 < mine) {
      fetch(i + 1);
      wait_loads<LOADS>();
    } else {
      wait_loads<0>();
    }
    const int64_t slot0 = begin + int64_t(wave + i * NW) * 2 * kBlock;
    const uint8_t* step = lds + (wave * kFewDepth + (2 * i) % kFewDepth) * BB;   // its two blocks are neighbours
    const bool gone0 = __builtin_amdgcn_readlane(page, 2 * i) < 0, gone1 = __builtin_amdgcn_readlane(page, 2 * i + 1) < 0;
    const bool whole = slot0 >= all_from && slot0 + 2 * kBlock <= all_to && !gone0 && !gone1;
    // scores: lane = slot for the codes, then slots 4 quad .. 4 quad + 3 of row j
    f4_t a[G][2];
#pragma unroll
    for (int g = 0; g < G; g++) a[g][0] = a[g][1] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
    {
      const uint8_t* kb = step + (lane >> 5) * BB;
      const int u = (lane >> 4) & 1, t = lane & 15;
#pragma unroll
      for (int c = 0; c < 4; c++)
#pragma unroll
        for (int k = 0; k < NK / CK; k++) {
          const auto w = *reinterpret_cast<const typename Chunk<CK>::type*>(kb + kcode_at(D, G, u, c * 16 + t, k * CK));
#pragma unroll
          for (int x = 0; x < CK; x++) {
            const int ks = k * CK + x;
            const h8_t f = codes8(w[x]);
            const h8_t q = qf[ks * 4 + c];
            a[ks / KG][0] = __builtin_amdgcn_mfma_f32_4x4x4f16(low4(f), low4(q), a[ks / KG][0], 0, 0, 0);
            a[ks / KG][1] = __builtin_amdgcn_mfma_f32_4x4x4f16(high4(f), high4(q), a[ks / KG][1], 0, 0, 0);
          }
        }
    }
    const uint8_t* mb = step + (quad >> 3) * BB;   // the block of the lane's four slots
    const int q8 = quad & 7;
    float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    h4_t vs[G], vl[G];
#pragma unroll
    for (int g = 0; g < G; g++) {
      const u4_t kp = *reinterpret_cast<const u4_t*>(mb + kpair_at(G, 4 * q8, g));
      vs[g] = *reinterpret_cast<const h4_t*>(mb + vstep_at(G, q8 & 3, 4 * (q8 >> 2), g));
      vl[g] = *reinterpret_cast<const h4_t*>(mb + vstep_at(G, q8 & 3, 4 * (q8 >> 2), g) + 16);
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const h2_t pair = __builtin_bit_cast(h2_t, (uint32_t)kp[r]);
        z[r] = fmaf((float)pair[1], a[g][0][r] + a[g][1][r], z[r]);
        z[r] = fmaf((float)pair[0], qsum[g], z[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; r++) z[r] *= z_unit;
    if (!whole) {
      const bool gone = quad < 8 ? gone0 : gone1;
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const int64_t slot = slot0 + 4 * quad + r;
        z[r] = slot >= from && slot < to && !gone ? z[r] : -__builtin_inff();
        if (slot >= s.len || gone)   // pairs of slots that hold nothing may be anything
#pragma unroll
          for (int g = 0; g < G; g++) vs[g][r] = vl[g][r] = (_Float16)0.0f;
      }
    }
    if (stash && slot0 + 4 * quad < p.stash_len) *reinterpret_cast<f4_t*>(stash + slot0 + 4 * quad) = f4_t{z[0], z[1], z[2], z[3]};
    h2_t sm2 = {(_Float16)0.0f, (_Float16)0.0f};
#pragma unroll
    for (int g = 0; g < G; g++) {
      sm2 = __builtin_elementwise_max(sm2, __builtin_shufflevector(vs[g], vs[g], 0, 1));
      sm2 = __builtin_elementwise_max(sm2, __builtin_shufflevector(vs[g], vs[g], 2, 3));
    }
    const float smax = fmaxf((float)sm2[0], (float)sm2[1]);
    const float mx = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
    if (__any(smax > s_limit || mx > top)) {   // rare: the reference of some row moves
      float sm = max_quads(smax);
      sm = fmaxf(sm, __shfl_xor(sm, 1));
      sm = fmaxf(sm, __shfl_xor(sm, 2));
      lift_of(sm, lift, s_limit);
      top = fmaxf(top, max_quads(mx));
      const float r = top - lift, f = exp2_fast(ref - r);
      ref = r;
      psum *= f;
#pragma unroll
      for (int g = 0; g < G; g++) plo[g] *= f;
#pragma unroll
      for (int q = 0; q < 4; q++) {
        const float fq = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), q));
#pragma unroll
        for (int h = 0; h < NH; h++) {
          acc[h][q] *= fq;
          more[h][q] *= fq;
        }
      }
    }
    h4_t hi[G], rest[G];   // p s as the sum of two fp16, see attend_rows
#pragma unroll
    for (int r = 0; r < 4; r++) {
      const float pe = exp2_fast(z[r] - ref);
      psum += pe;
#pragma unroll
      for (int g = 0; g < G; g++) {
        plo[g] = fmaf(pe, (float)vl[g][r], plo[g]);
        const float ps = pe * (float)vs[g][r];
        hi[g][r] = (_Float16)ps;
        rest[g][r] = (_Float16)(ps - (float)hi[g][r]);
      }
    }
    // V: lane = channel 64 h + lane; a dword holds two sets of four slots
#define STAGQ_KV_PV(HB, C)                                                                                        \
  {                                                                                                               \
    _Pragma("unroll") for (int h = 0; h < NH; h++) {                                                              \
      const uint32_t w = *reinterpret_cast<const uint32_t*>(step + HB * BB +                                      \
                                                            vcode_at(D, G, C * 16 + (lane & 15), 4 * h + (lane >> 4))); \
      const h8_t f = codes8(w);                                                                                   \
      const int g = h * G / NH;                                                                                   \
      acc[h] = __builtin_amdgcn_mfma_f32_4x4x4f16(hi[g], low4(f), acc[h], 4, 8 * HB + C, 0);                           \
      more[h] = __builtin_amdgcn_mfma_f32_4x4x4f16(rest[g], low4(f), more[h], 4, 8 * HB + C, 0);                       \
      acc[h] = __builtin_amdgcn_mfma_f32_4x4x4f16(hi[g], high4(f), acc[h], 4, 8 * HB + 4 + C, 0);                       \
      more[h] = __builtin_amdgcn_mfma_f32_4x4x4f16(rest[g], high4(f), more[h], 4, 8 * HB + 4 + C, 0);                   \
    }                                                                                                             \
  }
    STAGQ_KV_PV(0, 0) STAGQ_KV_PV(0, 1) STAGQ_KV_PV(0, 2) STAGQ_KV_PV(0, 3)
    STAGQ_KV_PV(1, 0) STAGQ_KV_PV(1, 1) STAGQ_KV_PV(1, 2) STAGQ_KV_PV(1, 3)
#undef STAGQ_KV_PV
  }

  float* sums = reinterpret_cast<float*>(lds);
  __syncthreads();
  const float l = sum_quads(psum);
#pragma unroll
  for (int g = 0; g < G; g++) plo[g] = sum_quads(plo[g]);
#pragma unroll
  for (int h = 0; h < NH; h++)
#pragma unroll
    for (int q = 0; q < 4; q++) {
      const float lo = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, plo[h * G / NH]), q));
      sums[(wave * kFewRows + q) * LD + 64 * h + lane] = fmaf(acc[h][q] + more[h][q], kCodeUnit, lo);
    }
  if (quad == 0) join_refs(sums, NW, kFewRows, D, wave, j, ref, l);
  __syncthreads();
  join_waves<D, NW, kFewRows>(p, s, sums, b, hk, 0, all, at_part);
}

template <int D, int G>
__global__ void __launch_bounds__(few_waves(D) * 64, D == 256 ? 1 : 2) attend_few(const AttnParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[FewLds<D, G>::BYTES];
  const int lane = threadIdx.x & 63, w = blockIdx.x;
  const bool own = p.shared == 0;
  int pos = 0, end = 1, quota = 1;
  // sequences in sets of 64: `seen` numbers before the set; lane i's sequence has
  // this length, this many rows, and ends at number seen + upto
  int set = 0, seen = 0, length = 0, q_len = 0, cost = 0, upto = 0;
  auto look = [&](int from) {
    length = q_len = 0;
    if (from + lane < p.c.batch) {
      length = p.c.lengths[from + lane];
      q_len = q_len_of(p, from + lane);
    }
    Span s;
    seq_span(p, length, q_len, s);
    const int n = few_steps(p, s);
    cost = n > 0 ? n + kItemCost : 0;
    upto = prefix64(cost * p.c.heads);
  };
  if (!own) {
    look(0);
    int total = __builtin_amdgcn_readlane(upto, 63);
    if (p.c.batch > 64) total = few_total(p);
    quota = max(int((unsigned(total) + unsigned(p.shared) - 1) / unsigned(p.shared)), kMinQuota);
    pos = w * quota;   // below 2^31, see plan
    end = min(total - pos, quota) + pos;
  }
  bool more = false;
#pragma unroll 1
  while (pos < end) {
    int b = blockIdx.z, hk = blockIdx.y, first = 0, take, n;
    int64_t part = (int64_t(b) * p.c.heads + hk) * kFewRows;
    Span s;
    if (own) {
      seq_span(p, b, s);
      take = n = few_steps(p, s);
      pos = end;
    } else {
      int in_set = __builtin_amdgcn_readlane(upto, 63);
      while (pos - seen >= in_set) {
        seen += in_set;
        set += 64;
        look(set);
        in_set = __builtin_amdgcn_readlane(upto, 63);
      }
      const int i = __builtin_amdgcn_readfirstlane(__ffsll(__ballot(upto > pos - seen)) - 1);
      const int c = __builtin_amdgcn_readlane(cost, i);
      const int into = pos - seen - (__builtin_amdgcn_readlane(upto, i) - c * p.c.heads);   // of the sequence's numbers
      seq_span(p, __builtin_amdgcn_readlane(length, i), __builtin_amdgcn_readlane(q_len, i), s);
      n = few_steps(p, s);
      b = set + i;
      hk = into / c;
      first = into - hk * c;
      take = min(c - first, end - pos);
      const int64_t item = int64_t(b) * p.c.heads + hk;
      part = (w + item) * kFewRows;
      if (first == 0 && threadIdx.x == 0) p.where[item] = int2{int(w + item), (pos + n - 1) / quota - w + 1};
      pos += take;
      take = min(take, n - first);
      if (take <= 0) continue;   // what was left of the item is its charge
    }
    if (more) __syncthreads();   // the last segment's sums have been read
    few_segment<D, G>(p, s, b, hk, first, take, take == n, part, lds);
    more = true;
  }
}

// The parts that make up the rows of a sequence and kv head: `count` of them,
// part k's row r at first + k stride + r.  done: the rows are written already.
struct Parts {
  int64_t first, stride;
  int count;
  bool done;
};
__device__ __forceinline__ Parts parts_of(const AttnParams& p, const Span& s, int b, int hk) {
  if (p.tile_rows != kFewRows) return Parts{part_row(p, b, hk, 0, 0), p.rows, used_splits(p, s), p.nsplit == 1};
  const int64_t item = int64_t(b) * p.c.heads + hk;
  const int n = few_steps(p, b);
  if (p.shared == 0) return Parts{item * kFewRows, kFewRows, n > 0 ? 1 : 0, true};
  if (n == 0) return Parts{0, 0, 0, false};
  const int2 at = p.where[item];
  return Parts{int64_t(at.x) * kFewRows, kFewRows, at.y, at.y == 1};
}

// Join the splits of a row, in a fixed order: D / 4 lanes hold the row, and the
// workgroup's groups of lanes take every NG-th split.
template <int D>
__device__ __forceinline__ void join_row(const AttnParams& p, unsigned id, float* lds) {
  constexpr int LV = D / 4, NG = 256 / LV;
  const int row = int(id % unsigned(p.rows)); id /= unsigned(p.rows);
  const int hk = int(id % unsigned(p.c.heads)), b = int(id / unsigned(p.c.heads));
  Span s;
  seq_span(p, b, s);
  if (row >= s.rows) {
    if (p.zero_rest) zero_rows<D>(p, b, hk, row, row + 1);
    return;
  }
  tile_span(p, row / p.tile_rows * p.tile_rows, s);
  const Parts parts = parts_of(p, s, b, hk);
  if (parts.done) return;
  const int used = parts.count;
  const int64_t first = parts.first + row;
  const int lane = threadIdx.x & 63, group = threadIdx.x / LV, c = (threadIdx.x % LV) * 4;
  float m = kNone;
  for (int i = lane; i < used; i += 64) m = fmaxf(m, p.part_rl[(first + i * parts.stride) * 2]);
#pragma unroll
  for (int d = 1; d < 64; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
  float l = 0.0f;
  f4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
  if (group < NG)
#pragma unroll 4
    for (int i = group; i < used; i += NG) {
      const int64_t at = first + i * parts.stride;
      const float f = exp2_fast(p.part_rl[at * 2] - m);
      l = fmaf(p.part_rl[at * 2 + 1], f, l);
      o += *reinterpret_cast<const f4_t*>(p.part + at * D + c) * f;
    }
  if (group < NG) {
    *reinterpret_cast<f4_t*>(lds + group * (D + 4) + c) = o;
    if (c == 0) lds[group * (D + 4) + D] = l;
  }
  __syncthreads();
  if (group == 0) {
    for (int i = 1; i < NG; i++) {
      o += *reinterpret_cast<const f4_t*>(lds + i * (D + 4) + c);
      l += lds[i * (D + 4) + D];
    }
    put_out(p, b, hk, row, c, o, l);
    if (p.lse && c == 0) put_lse(p, b, hk, row, m, l);
  }
}

// Weights of 1024 slots from the z that attend_rows kept.
__device__ __forceinline__ void weigh_stash(const AttnParams& p, unsigned id, float* lds) {
  const unsigned per = unsigned((p.max_len + 1023) / 1024);
  const int64_t slot = int64_t(id % per) * 1024 + threadIdx.x * 4; id /= per;
  const int hk = int(id % unsigned(p.c.heads)), b = int(id / unsigned(p.c.heads));
  Span s;
  seq_span(p, b, s);
  if (s.rows == 0) return;
  tile_span(p, 0, s);
  const Parts parts = parts_of(p, s, b, hk);
  const int used = parts.count;
  if (slot - threadIdx.x * 4 >= s.hi || used == 0) return;
  // the rows' log-sum-exp: 32 lanes per row (at most 8 rows)
  const int r = threadIdx.x >> 5, l32 = threadIdx.x & 31;
  float m = kNone, l = 0.0f;
  if (r < s.rows) {
    const int64_t first = parts.first + r;
    for (int i = l32; i < used; i += 32) m = fmaxf(m, p.part_rl[(first + i * parts.stride) * 2]);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) m = fmaxf(m, __shfl_xor(m, d));
    for (int i = l32; i < used; i += 32) {
      const int64_t at = (first + i * parts.stride) * 2;
      l = fmaf(p.part_rl[at + 1], exp2_fast(p.part_rl[at] - m), l);
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2) l += __shfl_xor(l, d);
    if (l32 == 0) lds[r] = l == 0.0f ? __builtin_inff() : m + __log2f(l);
  }
  __syncthreads();
  if (slot >= s.hi || slot + 4 <= s.lo) return;
  const float* z = p.stash + (int64_t(b) * p.c.heads + hk) * p.rows * p.stash_len + slot;
  f4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = 0; i < s.rows; i++) {
    const f4_t x = *reinterpret_cast<const f4_t*>(z + i * p.stash_len);
#pragma unroll
    for (int k = 0; k < 4; k++) sum[k] += exp2_fast(x[k] - lds[i]);
  }
  float* w = p.weights + b * p.wsb + hk * p.wsh + slot;
#pragma unroll
  for (int k = 0; k < 4; k++)
    if (slot + k < s.hi) w[k] += sum[k];
}

// What follows attend_rows in one launch: rows to join, then slots to weigh.
template <int D>
__global__ void __launch_bounds__(256) finish_kernel(const AttnParams p, unsigned joins) {
  __shared__ float lds[(256 / (D / 4)) * (D + 4)];
  if (blockIdx.x < joins) join_row<D>(p, blockIdx.x, lds);
  else weigh_stash(p, blockIdx.x - joins, lds);
}

// ------------------------------------------------ many rows per kv head ----
// Prompts and chunks of them.  A workgroup holds 128 rows (64 at 256 channels),
// 32 per wave, and walks over 64 slots at a time: the four waves unpack a quarter each of the
// tile into LDS, in operand order, so that a fragment is 1 KB read and written
// in lane order without conflicts; every fragment serves 32 rows of each wave.
//   K  goes in as its codes (u / 256, exact), and s meets the 32-bit sums of its
//      group; sum lo (sum of q) is a product of its own, of the lo of all groups
//      with the sums of q, split in two fp16.  (With lo + s u rounded to fp16 in
//      one fragment the scores lose more than an fp16 result shows: relative
//      error 4.4e-4 instead of 2.9e-4 at 12001 slots, where its own rounding
//      makes 2.1e-4.)
//   V  goes in as lo + s u, rounded to fp16 once; so do the probabilities.
// The codes of the next tile are loaded while this one is computed, and unpacked
// into the other buffer after it: one barrier per tile.  The row sums are
// of the probabilities before their rounding, in binary32 (a matrix product of
// the rounded ones with 1 is 1.7 % faster, but leaves lse off by up to 1.5e-4 in
// rows that see two slots).
constexpr int kTileSlots = 64;
// 16-row tiles of a wave (two hold too many registers at 256 channels), rows of a workgroup
constexpr int big_tiles(int D) { return D == 256 ? 1 : 2; }
constexpr int big_rows(int D) { return 64 * big_tiles(D); }
constexpr float kTileLift = 14.0f;   // p <= 2^14 in fp16; lost only below 2^-38 of the largest

template <int D, int G>
struct TileRegs {
  static constexpr int NK = D / 32, NV = D / 16, CK = kchunk(D), VH = NV / 2, VG = NV / G, GH = (VH + VG - 1) / VG;
  static constexpr int CV = VH < vchunk(D) ? VH : vchunk(D);
  typename Chunk<CK>::type k[NK / CK];   // unit `wave` of the tile
  uint32_t kp[G];
  typename Chunk<CV>::type v[VH / CV];   // half `wave & 1` of the channels of block `wave >> 1`
  u4_t vs[GH], vl[GH];

  __device__ __forceinline__ void load(const uint8_t* base, int lane, int wave) {
    const int u = wave & 1, half = wave & 1, g0 = half * VH / VG;
#pragma unroll
    for (int g = 0; g < G; g++) kp[g] = *reinterpret_cast<const uint32_t*>(base + kpair_at(G, 16 * u + (lane & 15), g));
#pragma unroll
    for (int i = 0; i < NK / CK; i++)
      k[i] = *reinterpret_cast<const typename Chunk<CK>::type*>(base + kcode_at(D, G, u, lane, i * CK));
#pragma unroll
    for (int g = 0; g < GH; g++) {
      const uint8_t* at = base + vstep_at(G, lane >> 4, 0, g0 + g);
      vs[g] = *reinterpret_cast<const u4_t*>(at);
      vl[g] = *reinterpret_cast<const u4_t*>(at + 16);
    }
#pragma unroll
    for (int i = 0; i < VH / CV; i++)
      v[i] = *reinterpret_cast<const typename Chunk<CV>::type*>(base + vcode_at(D, G, lane, half * VH + i * CV));
  }
  // Pairs of slots from `left` on (of the block) become 0, and with them the values.
  __device__ __forceinline__ void cut(int left, int lane, int wave) {
    if (16 * (wave & 1) + (lane & 15) >= left)
#pragma unroll
      for (int g = 0; g < G; g++) kp[g] = 0u;
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (vtoken(lane >> 4, e) >= left)
#pragma unroll
        for (int g = 0; g < GH; g++) {
          const uint32_t keep = (e & 1) ? 0x0000ffffu : 0xffff0000u;
          vs[g][e / 2] &= keep;
          vl[g][e / 2] &= keep;
        }
  }
  // kb, vb, lb: fragments; sb: s [unit][group][16 slots].
  __device__ __forceinline__ void store(h8_t* kb, h8_t* vb, h8_t* lb, _Float16* sb, int lane, int wave) const {
    const int blk = wave >> 1, half = wave & 1;
#pragma unroll
    for (int ks = 0; ks < NK; ks++) {
      const uint32_t w = k[ks / CK][ks % CK];
      h8_t f;
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const h2_t x = code_pair_256th(w, i);
        f[2 * i] = x[0];
        f[2 * i + 1] = x[1];
      }
      kb[(wave * NK + ks) * 64 + lane] = f;
    }
    h8_t f;   // sets 0 and 1: lo of group e against the two parts of the sums of q
#pragma unroll
    for (int e = 0; e < 8; e++) f[e] = e < G && lane < 32 ? __builtin_bit_cast(h2_t, kp[e < G ? e : 0])[0] : (_Float16)0.0f;
    lb[wave * 64 + lane] = f;
    if (lane < 16)
#pragma unroll
      for (int g = 0; g < G; g++) sb[(wave * G + g) * 16 + lane] = __builtin_bit_cast(h2_t, kp[g])[1];
#pragma unroll
    for (int i = 0; i < VH; i++) {
      const int c = half * VH + i;
      u4_t vsg, vlg;
      if constexpr (VH % VG == 0 || VG % VH == 0) {
        vsg = vs[VH % VG == 0 ? i / VG : 0];
        vlg = vl[VH % VG == 0 ? i / VG : 0];
      } else {   // a group lies across the halves
        const int g = c / VG - half * VH / VG;
        vsg = vs[0];
        vlg = vl[0];
#pragma unroll
        for (int x = 1; x < GH; x++)
          if (g == x) { vsg = vs[x]; vlg = vl[x]; }
      }
      const uint32_t w = v[i / CV][i % CV];
      h8_t f;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const h2_t x = __builtin_elementwise_fma(code_pair(w, e), __builtin_bit_cast(h2_t, (uint32_t)vsg[e]),
                                                 __builtin_bit_cast(h2_t, (uint32_t)vlg[e]));
        f[2 * e] = x[0];
        f[2 * e + 1] = x[1];
      }
      vb[(blk * NV + c) * 64 + lane] = f;
    }
  }
};

// The sums of q over its groups as an operand, divided by 256 and split in two
// fp16: set 0 the rounded ones, set 1 what is left (e = group).
template <int NK, int G>
__device__ __forceinline__ h8_t sums_operand(const h8_t* qf, int set) {
  constexpr int KG = NK / G;
  h8_t r;
#pragma unroll
  for (int e = 0; e < 8; e++) {
    r[e] = (_Float16)0.0f;
    if (e < G) {
      const float q = sum_sets(sum8<KG>(qf + (e < G ? e : 0) * KG)) * (1.0f / 256.0f);
      const _Float16 hi = (_Float16)q;
      r[e] = set == 0 ? hi : set == 1 ? (_Float16)(q - (float)hi) : (_Float16)0.0f;
    }
  }
  return r;
}
// q . k / 256 of NT 16-row tiles and the tile's four units of 16 slots.
template <int NT, int NK, int G>
__device__ __forceinline__ void scores(const h8_t* kb, const h8_t* lb, const _Float16* sb, const h8_t (*qf)[NK],
                                       const h8_t* qs, int lane, f4_t (*z)[4]) {
  constexpr int KG = NK / G;
  const f4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int u = 0; u < 4; u++) {
    if (NK == 8) __builtin_amdgcn_sched_barrier(0);   // or the loads of all units are hoisted, and spilled
    const h8_t lf = lb[u * 64 + lane];
#pragma unroll
    for (int t = 0; t < NT; t++) z[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(lf, qs[t], zero, 0, 0, 0);
#pragma unroll
    for (int g = 0; g < G; g++) {
      f4_t a[NT];
#pragma unroll
      for (int t = 0; t < NT; t++) a[t] = zero;
#pragma unroll
      for (int ks = g * KG; ks < (g + 1) * KG; ks++) {
        const h8_t kf = kb[(u * NK + ks) * 64 + lane];
#pragma unroll
        for (int t = 0; t < NT; t++) a[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[t][ks], a[t], 0, 0, 0);
      }
      const h4_t s = *reinterpret_cast<const h4_t*>(sb + (u * G + g) * 16 + 4 * (lane >> 4));
#pragma unroll
      for (int r = 0; r < 4; r++)
#pragma unroll
        for (int t = 0; t < NT; t++) z[t][u][r] = fmaf((float)s[r], a[t][r], z[t][u][r]);
    }
  }
}

// p from z, its sums, and p V.  EXACT: p as the sum of two fp16, for fp16
// results: with V rounded as well, one alone makes their error 1.6 times that of
// their own rounding (two: 1.4); bf16 results are eight times as coarse.
template <bool EXACT, int NT, int NV>
__device__ __forceinline__ void weigh_values(const f4_t (*z)[4], const float* z_unit, const float* ref, const h8_t* vb,
                                             int lane, float* sum, f4_t (*acc)[NV]) {
#pragma unroll
  for (int h = 0; h < 2; h++) {
    h8_t pf[NT], rest[NT];
#pragma unroll
    for (int t = 0; t < NT; t++) {
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const float x = exp2_fast(fmaf(z[t][2 * h + (e >> 2)][e & 3], z_unit[t], -ref[t]));
        pf[t][e] = (_Float16)x;
        if (EXACT) rest[t][e] = (_Float16)(x - (float)pf[t][e]);
        sum[t] += x;
      }
    }
#pragma unroll
    for (int c = 0; c < NV; c++) {
      const h8_t vf = vb[(h * NV + c) * 64 + lane];
#pragma unroll
      for (int t = 0; t < NT; t++) {
        acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[t], acc[t][c], 0, 0, 0);
        if (EXACT) acc[t][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, rest[t], acc[t][c], 0, 0, 0);
      }
    }
  }
}

// fp16 rows of q scaled as bf16 ones are (exact): the second part of the sums
// over 256 would be subnormal, and lse off by 1e-6 of its size instead of 3e-7.
template <int NK>
__device__ __forceinline__ float scale_half(h8_t* qf) {
  float amax = 0.0f;
#pragma unroll
  for (int ks = 0; ks < NK; ks++)
#pragma unroll
    for (int e = 0; e < 8; e++) amax = fmaxf(amax, fabsf((float)qf[ks][e]));
  const float m = row_scale(max_sets(amax));
#pragma unroll
  for (int ks = 0; ks < NK; ks++)
#pragma unroll
    for (int e = 0; e < 8; e++) qf[ks][e] = (_Float16)((float)qf[ks][e] * m);
  return 1.0f / m;
}

template <int D, int G, bool EXACT>
__global__ void __launch_bounds__(256, D == 256 ? 1 : 2) attend_tiles(const AttnParams p) {
  constexpr int NK = D / 32, NV = D / 16, NT = big_tiles(D);
  __shared__ h8_t kbuf[2][4 * NK * 64], vbuf[2][2 * NV * 64], lbuf[2][4 * 64];
  __shared__ __attribute__((aligned(16))) _Float16 sbuf[2][4 * G * 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, set = lane >> 4;
  // heads change fastest, so that an XCD's L2 keeps to few of them; the tiles
  // that see most come first
  const int hk = blockIdx.x, b = blockIdx.z;
  const int tile = p.tiles - 1 - int(blockIdx.y / unsigned(p.nsplit)), split = int(blockIdx.y % unsigned(p.nsplit));
  Span s;
  seq_span(p, b, s);
  const int row0 = tile * big_rows(D);
  if (row0 >= s.rows) {
    if (p.zero_rest && p.nsplit == 1) zero_rows<D>(p, b, hk, row0, min(row0 + big_rows(D), p.rows));
    return;
  }
  tile_span(p, row0, s);
  if (split >= used_splits(p, s) && split > 0) return;   // split 0 leaves its operands, and zeros if it is the only one
  const int begin = int(s.lo) + split * p.chunk, end = int(min(int64_t(begin) + p.chunk, s.hi));
  const int ntile = end > begin ? (end - begin + kTileSlots - 1) / kTileSlots : 0;

  const int wrow = row0 + wave * 16 * NT;
  h8_t qf[NT][NK], qs[NT];
  float z_unit[NT], ref[NT], top[NT];
  int from[NT], to[NT];
  f4_t acc[NT][NV];
  float sum[NT];   // of the lane's slots
#pragma unroll
  for (int t = 0; t < NT; t++) {
    const int row = wrow + t * 16 + n;
    const bool there = row < s.rows;
    float unit;
    load_q<D>(p, b, hk, row, there, qf[t], &unit);
    if (EXACT) unit = scale_half<NK>(qf[t]);   // fp16
    z_unit[t] = fabsf(p.scale2) * 256.0f * unit;
    if (p.scale2 < 0.0f)   // the sign goes to q, so that the largest product is the largest z
#pragma unroll
      for (int ks = 0; ks < NK; ks++) qf[t][ks] = -qf[t][ks];
    if (z_unit[t] < 0x1p-126f) {   // a scale of 0: z is 0 by q, as -inf, what is not seen, may not meet a factor of 0
      z_unit[t] = 1.0f;
#pragma unroll
      for (int ks = 0; ks < NK; ks++) qf[t][ks] = h8_t{};
    }
    qs[t] = sums_operand<NK, G>(qf[t], set);
    if (p.q_frags && split == 0) {   // for the weights
      const int64_t rt = (int64_t(b) * p.c.heads + hk) * p.q_tiles + (wrow + t * 16) / 16;
      h8_t* to = reinterpret_cast<h8_t*>(p.q_frags) + rt * (NK + 1) * 64 + lane;
#pragma unroll
      for (int ks = 0; ks < NK; ks++) to[ks * 64] = qf[t][ks];
      to[NK * 64] = qs[t];
      if (set == 0) p.q_units[rt * 16 + n] = z_unit[t];
    }
    int64_t f = 0, e = 0;
    if (there) row_span(p, s, row, f, e);
    from[t] = int(f);
    to[t] = int(e);
    ref[t] = top[t] = kNone;
    sum[t] = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; c++) acc[t][c] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  // what some row of the wave sees, and what all of them see
  int any_from = 0, any_to = 0, all_from = 0, all_to = 0;
  if (wrow < s.rows) {
    int64_t f0, t0, f1, t1;
    row_span(p, s, wrow, f0, t0);
    row_span(p, s, min(wrow + 16 * NT, s.rows) - 1, f1, t1);
    any_from = int(f0); any_to = int(t1); all_from = int(f1); all_to = int(t0);
  }

  int page[2];   // of the two blocks of tile (64 k + lane)
  const int mask = (1 << p.c.shift) - 1;
  auto pages = [&](int i0) {
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int slot = begin + (i0 + lane) * kTileSlots + h * kBlock;
      page[h] = -1;
      if (i0 + lane < ntile && (slot >> p.c.shift) < p.c.width)
        page[h] = p.c.table[int64_t(b) * p.c.table_stride + (slot >> p.c.shift)];
      if (page[h] >= p.c.pages) page[h] = -1;
    }
  };
  TileRegs<D, G> regs;
  bool gone[2][2];   // by buffer and block
  auto load = [&](int i) {
    if ((i & 63) == 0) pages(i);
    const int pg0 = __builtin_amdgcn_readlane(page[0], i & 63), pg1 = __builtin_amdgcn_readlane(page[1], i & 63);
    gone[1][0] = pg0 < 0;
    gone[1][1] = pg1 < 0;
    const int pg = wave < 2 ? pg0 : pg1, slot = begin + i * kTileSlots + (wave >> 1) * kBlock;
    // a block without a page is read from page 0 and cut away
    regs.load(p.c.buf + uint64_t(max(pg, 0)) * p.c.page_bytes + uint64_t(hk) * p.c.head_bytes +
                  uint32_t((slot & mask) / kBlock) * block_bytes(D, G), lane, wave);
    const int left = pg < 0 ? 0 : int(s.len) - slot;
    if (left < kBlock) regs.cut(left, lane, wave);
  };
  if (ntile > 0) {
    load(0);
    regs.store(kbuf[0], vbuf[0], lbuf[0], sbuf[0], lane, wave);
  }

#pragma unroll 1
  for (int i = 0; i < ntile; i++) {
    gone[0][0] = gone[1][0];
    gone[0][1] = gone[1][1];
    __syncthreads();
    if (i + 1 < ntile) load(i + 1);
    const int slot0 = begin + i * kTileSlots;
    if (slot0 < any_to && slot0 + kTileSlots > any_from) {
      const h8_t* kb = kbuf[i & 1];
      const h8_t* vb = vbuf[i & 1];
      f4_t z[NT][4];
      scores<NT, NK, G>(kb, lbuf[i & 1], sbuf[i & 1], qf, qs, lane, z);
      if (slot0 < all_from || slot0 + kTileSlots > all_to || gone[0][0] || gone[0][1]) {
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
          for (int u = 0; u < 4; u++)
#pragma unroll
            for (int r = 0; r < 4; r++) {
              const int slot = slot0 + 16 * u + 4 * set + r;
              z[t][u][r] = slot >= from[t] && slot < to[t] && !gone[0][u >> 1] ? z[t][u][r] : -__builtin_inff();
            }
      }
      float mx[NT];
      bool moves = false;
#pragma unroll
      for (int t = 0; t < NT; t++) {
        float m = z[t][0][0];
#pragma unroll
        for (int u = 0; u < 4; u++)
#pragma unroll
          for (int r = 0; r < 4; r++) m = fmaxf(m, z[t][u][r]);
        mx[t] = m * z_unit[t];
        moves |= mx[t] > top[t];
      }
      if (__any(moves)) {
#pragma unroll
        for (int t = 0; t < NT; t++) {
          top[t] = fmaxf(top[t], max_sets(mx[t]));
          const float r = top[t] - kTileLift, f = exp2_fast(ref[t] - r);
          ref[t] = r;
          sum[t] *= f;
#pragma unroll
          for (int c = 0; c < NV; c++) acc[t][c] *= f;
        }
      }
      weigh_values<EXACT, NT, NV>(z, z_unit, ref, vb, lane, sum, acc);
    }
    if (i + 1 < ntile) {
      const int o = (i + 1) & 1;
      regs.store(kbuf[o], vbuf[o], lbuf[o], sbuf[o], lane, wave);
    }
  }

#pragma unroll
  for (int t = 0; t < NT; t++) {
    const int row = wrow + t * 16 + n;
    const float l = sum_sets(sum[t]);
    if (row >= s.rows) {
      if (p.zero_rest && p.nsplit == 1 && row < p.rows)
#pragma unroll
        for (int c = 0; c < NV; c++)
          *reinterpret_cast<u2_t*>(out_row(p, b, hk, row) + 16 * c + 4 * set) = u2_t{0u, 0u};
      continue;
    }
    if (p.nsplit == 1) {
#pragma unroll
      for (int c = 0; c < NV; c++) put_out(p, b, hk, row, 16 * c + 4 * set, acc[t][c], l);
      if (p.lse && set == 0) put_lse(p, b, hk, row, ref[t], l);
    } else if (ntile > 0) {
      const int64_t at = part_row(p, b, hk, split, row);
#pragma unroll
      for (int c = 0; c < NV; c++) *reinterpret_cast<f4_t*>(p.part + at * D + 16 * c + 4 * set) = acc[t][c];
      if (set == 0) { p.part_rl[at * 2] = ref[t]; p.part_rl[at * 2 + 1] = l; }
    }
  }
}

// Weight of every cached slot: the sum of P over the sequence's rows, from the
// rows' log-sum-exp.  A wave owns one block of 32 slots, so no two waves add to
// one slot and the order of the sums is fixed.
template <int D, int G>
__global__ void __launch_bounds__(256) weigh_kernel(const AttnParams p) {
  constexpr int NK = D / 32, KG = NK / G, CK = kchunk(D);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, set = lane >> 4;
  unsigned id = blockIdx.x;
  const unsigned per = unsigned((p.max_len + 4 * kBlock - 1) / (4 * kBlock));
  const int64_t slot0 = (int64_t(id % per) * 4 + wave) * kBlock; id /= per;
  const int hk = int(id % unsigned(p.c.heads)), b = int(id / unsigned(p.c.heads));
  Span s;
  seq_span(p, b, s);
  if (slot0 >= s.len || s.rows == 0) return;
  const uint8_t* base = block_at<D, G>(p.c, b, hk, slot0);
  if (!base) return;
  h8_t kf[2][NK];
  u4_t kp[2][G];
#pragma unroll
  for (int u = 0; u < 2; u++) {
#pragma unroll
    for (int g = 0; g < G; g++) kp[u][g] = *reinterpret_cast<const u4_t*>(base + kpair_at(G, 16 * u + 4 * set, g));
#pragma unroll
    for (int i = 0; i < NK / CK; i++) {
      const auto w = *reinterpret_cast<const typename Chunk<CK>::type*>(base + kcode_at(D, G, u, lane, i * CK));
#pragma unroll
      for (int x = 0; x < CK; x++) {
        kf[u][i * CK + x] = codes8(w[x]);
      }
    }
  }
  float sum[8] = {};
  const float* lse = p.lse + int64_t(b) * p.q.tokens * p.q.heads;
  for (int row0 = 0; row0 < s.rows; row0 += kRowTile) {
    const int row = row0 + n;
    const bool there = row < s.rows;
    int64_t from = 0, to = 0;
    if (there) row_span(p, s, row, from, to);
    if (!__any(from < slot0 + kBlock && to > slot0)) continue;
    h8_t qf[NK];
    float unit;
    load_q<D>(p, b, hk, row, there, qf, &unit);
    const float z_unit = p.scale2 * kCodeUnit * unit;
    const int t = token_of(p, row);
    const float l = there ? lse[int64_t(t) * p.q.heads + (hk - t) * int(p.gq) + row] : 0.0f;
    const float l2 = l * kLog2e;
    float z[8] = {};
#pragma unroll
    for (int g = 0; g < G; g++) {
      const float qs = sum_sets(sum8<KG>(qf + g * KG)) * (1.0f / kCodeUnit);
#pragma unroll
      for (int u = 0; u < 2; u++) {
        f4_t a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ks = g * KG; ks < (g + 1) * KG; ks++)
          a = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[u][ks], qf[ks], a, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const h2_t pair = __builtin_bit_cast(h2_t, (uint32_t)kp[u][g][r]);
          z[u * 4 + r] = fmaf((float)pair[1], a[r], z[u * 4 + r]);
          z[u * 4 + r] = fmaf((float)pair[0], qs, z[u * 4 + r]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const int64_t slot = slot0 + vtoken(set, e);
      sum[e] += slot >= from && slot < to ? exp2_fast(z[e] * z_unit - l2) : 0.0f;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; e++)
#pragma unroll
    for (int d = 1; d < 16; d *= 2) sum[e] += __shfl_xor(sum[e], d);
  if (n == 0) {
    float* w = p.weights + b * p.wsb + hk * p.wsh;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      const int64_t slot = slot0 + vtoken(set, e);
      if (slot < s.len) w[slot] += sum[e];
    }
  }
}

// Weights after attend_tiles, which leaves its query operands behind.  A wave
// holds 64 slots of K in registers and goes through the rows that may see them,
// 16 at a time; the operands come through LDS, 32 rows ahead by direct loads
// shared by the four waves.  Per 16 rows and 64 slots: 20 matrix instructions
// and about 130 others (16 of them exponentials), so vector work bounds it, at
// about half of what attend_tiles takes for the same scores.
template <int D, int G>
__global__ void __launch_bounds__(256, D == 256 ? 1 : 2) weigh_tiles(const AttnParams p) {
  constexpr int NK = D / 32, KG = NK / G, CK = kchunk(D), FR = NK + 1;   // 1 KB fragments of 16 rows
  constexpr int kStage = 2;                                              // row tiles per stage
  __shared__ h8_t qbuf[2][kStage * FR * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, set = lane >> 4;
  const int hk = blockIdx.x, b = blockIdx.z;
  Span s;
  seq_span(p, b, s);
  const int group0 = int(blockIdx.y) * 4 * kTileSlots, slot0 = group0 + wave * kTileSlots;
  if (group0 >= s.len || s.rows == 0) return;
  // tokens [t0, t1) of the queries see some slot of the workgroup
  const int behind = int(s.len) - s.ql;
  const int t0 = p.causal ? max(group0 - behind, 0) : 0;
  const int t1 = p.window > 0 ? int(min(int64_t(group0) + 4 * kTileSlots - 1 + p.window - behind, int64_t(s.ql))) : s.ql;
  if (t0 >= t1) return;
  const int rt0 = t0 * int(p.gq) / 16, rt1 = (t1 * int(p.gq) + 15) / 16;

  const int64_t item = int64_t(b) * p.c.heads + hk;
  const h8_t* frags = reinterpret_cast<const h8_t*>(p.q_frags) + item * p.q_tiles * FR * 64;
  const uint32_t to = uint32_t(uintptr_t((__attribute__((address_space(3))) void*)&qbuf[0][0]));
  auto fetch = [&](int i) {   // stage i: every wave copies every fourth KB
#pragma unroll
    for (int k = 0; k < (kStage * FR + 3) / 4; k++) {
      const int f = wave + k * 4;
      if (f < kStage * FR && rt0 + i * kStage + f / FR < p.q_tiles)
        copy_block<1024, false>(reinterpret_cast<const uint8_t*>(frags + (int64_t(rt0 + i * kStage) * FR + f) * 64),
                         to + uint32_t(i & 1) * uint32_t(sizeof(qbuf[0])) + uint32_t(f) * 1024u, lane);
    }
  };
  const int stages = (rt1 - rt0 + kStage - 1) / kStage;
  fetch(0);

  h8_t kf[4][NK], lf[4];
  h4_t ks4[4][G];
  bool gone[2];
#pragma unroll
  for (int h = 0; h < 2; h++) {
    const int first = slot0 + h * kBlock;
    const uint8_t* base = first < s.len ? block_at<D, G>(p.c, b, hk, first) : nullptr;
    gone[h] = base == nullptr;
#pragma unroll
    for (int v = 0; v < 2; v++) {
      const int u = 2 * h + v;
      uint32_t lo[G];
#pragma unroll
      for (int g = 0; g < G; g++) {
        u4_t kp = {0u, 0u, 0u, 0u};
        lo[g] = 0u;
        if (base) {
          kp = *reinterpret_cast<const u4_t*>(base + kpair_at(G, 16 * v + 4 * set, g));
          lo[g] = *reinterpret_cast<const uint32_t*>(base + kpair_at(G, 16 * v + n, g));
        }
#pragma unroll
        for (int r = 0; r < 4; r++) ks4[u][g][r] = __builtin_bit_cast(h2_t, (uint32_t)kp[r])[1];
      }
#pragma unroll
      for (int e = 0; e < 8; e++)
        lf[u][e] = e < G && lane < 32 ? __builtin_bit_cast(h2_t, lo[e < G ? e : 0])[0] : (_Float16)0.0f;
#pragma unroll
      for (int i = 0; i < NK / CK; i++) {
        typename Chunk<CK>::type w = {};
        if (base) w = *reinterpret_cast<const typename Chunk<CK>::type*>(base + kcode_at(D, G, v, lane, i * CK));
#pragma unroll
        for (int x = 0; x < CK; x++)
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const h2_t c = code_pair_256th(w[x], e);
            kf[u][i * CK + x][2 * e] = c[0];
            kf[u][i * CK + x][2 * e + 1] = c[1];
          }
      }
    }
  }
  f4_t sum[4];
#pragma unroll
  for (int u = 0; u < 4; u++) sum[u] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const f4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const float* lse = p.lse + int64_t(b) * p.q.tokens * p.q.heads;
  const bool holes = gone[0] || gone[1] || slot0 + kTileSlots > s.len;

#pragma unroll 1
  for (int i = 0; i < stages; i++) {
    wait_loads<0>();
    __syncthreads();   // the stage is there, and the other buffer has been read
    if (i + 1 < stages) fetch(i + 1);
#pragma unroll
    for (int k = 0; k < kStage; k++) {
      const int rt = rt0 + i * kStage + k, row = rt * 16 + n;
      if (rt >= rt1) continue;
      int from = 0, to_ = 0;
      float l2 = 0.0f, unit = 0.0f;
      if (row < s.rows) {
        int64_t f, t;
        row_span(p, s, row, f, t);
        from = int(f);
        to_ = int(t);
        const int tok = token_of(p, row);
        l2 = lse[int64_t(tok) * p.q.heads + (hk - tok) * int(p.gq) + row] * kLog2e;
        unit = p.q_units[item * p.q_tiles * 16 + row];
      }
      // rows of the tile: first .. last; what all of them see
      int64_t f0, e0, f1, e1;
      row_span(p, s, rt * 16, f0, e0);
      row_span(p, s, min(rt * 16 + 16, s.rows) - 1, f1, e1);
      if (e1 <= slot0 || f0 >= slot0 + kTileSlots) continue;
      const bool whole = !holes && f1 <= slot0 && e0 >= slot0 + kTileSlots && rt * 16 + 16 <= s.rows;
      const h8_t* qb = &qbuf[i & 1][k * FR * 64];
      h8_t qf[NK];
#pragma unroll
      for (int ks = 0; ks < NK; ks++) qf[ks] = qb[ks * 64 + lane];
      const h8_t qs = qb[NK * 64 + lane];
#pragma unroll
      for (int u = 0; u < 4; u++) {
        f4_t z = __builtin_amdgcn_mfma_f32_16x16x32_f16(lf[u], qs, zero, 0, 0, 0);
#pragma unroll
        for (int g = 0; g < G; g++) {
          f4_t a = zero;
#pragma unroll
          for (int ks = g * KG; ks < (g + 1) * KG; ks++)
            a = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[u][ks], qf[ks], a, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < 4; r++) z[r] = fmaf((float)ks4[u][g][r], a[r], z[r]);
        }
        if (whole) {
#pragma unroll
          for (int r = 0; r < 4; r++) sum[u][r] += exp2_fast(fmaf(z[r], unit, -l2));
        } else {
#pragma unroll
          for (int r = 0; r < 4; r++) {
            const int slot = slot0 + 16 * u + 4 * set + r;
            const float w = exp2_fast(fmaf(z[r], unit, -l2));
            sum[u][r] += slot >= from && slot < to_ && !gone[u >> 1] ? w : 0.0f;
          }
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < 4; u++)
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
      for (int d = 1; d < 16; d *= 2) sum[u][r] += __shfl_xor(sum[u][r], d);
  if (n == 0) {
    float* w = p.weights + b * p.wsb + hk * p.wsh;
#pragma unroll
    for (int u = 0; u < 4; u++)
#pragma unroll
      for (int r = 0; r < 4; r++) {
        const int slot = slot0 + 16 * u + 4 * set + r;
        if (slot < s.len) w[slot] += sum[u][r];
      }
  }
}

// ------------------------------------------------------------- dispatch ----
struct Plan {
  enum { FEW, ROWS, TILES } kind;
  int nq, tile_rows, tiles, chunk, nsplit, shared;
  bool stash;
  int64_t stash_len, groups, joins, weighs;
  int64_t q_tiles;
  size_t part, rl, lse, z, where, frags, units, total;   // offsets in the workspace, its size
};

// Variants and splits by shape alone.
static bool plan(const stagq_kv_cache* c, const stagq_kv_seqs* q, const stagq_kv_attn* a, Plan* pl) {
  const int gq = a->q.heads / c->kv_heads;
  const int64_t rows = int64_t(a->q.tokens) * gq;
  if (rows > (int64_t(1) << 30)) return false;
  const int waves = ring_waves(c->head_dim);
  const int64_t all = c->pages > 0 ? reach(c, q, a->max_len) : 0;   // without pages there is nothing to see
  const int64_t heads = int64_t(q->batch) * c->kv_heads;
  auto spanned = [&](int tile_rows) {   // slots a tile's rows see at most, from the start of two blocks
    const int64_t most = int64_t(a->window) + (tile_rows + gq - 1) / gq + 1 + 2 * kBlock;
    return a->window > 0 && most < all ? most : all;
  };
  // attend_few: a set of 64 channels has to share its pair; step numbers are below 2^30
  const int64_t steps = (spanned(kFewRows) + 2 * kBlock - 1) / (2 * kBlock), cost = steps + kItemCost;
  const bool few = rows <= kFewRows && c->group >= 64 && heads * cost < (int64_t(1) << 30);
  pl->kind = few ? Plan::FEW : rows > (a->weights ? kManyRowsWeighed : kManyRows) ? Plan::TILES : Plan::ROWS;
  pl->nq = rows > kRowTile && c->head_dim < 256 ? 2 : 1;   // attend_rows
  pl->tile_rows = few ? kFewRows : pl->kind == Plan::TILES ? big_rows(c->head_dim) : pl->nq * kRowTile;
  pl->tiles = int((rows + pl->tile_rows - 1) / pl->tile_rows);
  const int64_t base = heads * pl->tiles;
  pl->shared = 0;
  pl->nsplit = pl->chunk = 1;
  size_t part_rows;
  if (few) {
    // An item (sequence and head) has a workgroup of its own where it is short, or
    // where there are items enough to even the grid out by themselves; else the
    // grid shares all steps.  most: steps of a workgroup, 32 per wave (a
    // page-table entry per lane and block).
    const int64_t most = few_waves(c->head_dim) * 32;
    if (steps > kOwnSteps && (steps > most || steps * kItemsPerStep > heads)) {
      const int64_t need = (heads * cost + most - 1) / most;
      pl->shared = int((need + kWantedGroups - 1) / kWantedGroups * kWantedGroups);
    }
    part_rows = size_t(pl->shared + heads) * kFewRows;
    pl->groups = pl->shared ? pl->shared : heads;
  } else {
    const int64_t blocks = (spanned(pl->tile_rows) + kBlock - 1) / kBlock;
    const int64_t wanted = base > 0 ? (kWantedGroups + base - 1) / base : 1;
    const bool big = pl->kind == Plan::TILES;
    const int64_t least = big ? kMinTileBlocks : kMinBlocks, unit = big ? 2 : waves;
    int64_t per = (blocks + wanted - 1) / wanted;
    per = per < least ? least : per;
    if (!big) {   // few blocks: one workgroup per CU rather than longer splits
      const int64_t single = base > 0 ? (kSingleGroups + base - 1) / base : 1;
      int64_t one = (blocks + single - 1) / single;
      one = one < waves ? waves : one;
      per = one < per ? one : per;
    }
    if (!big && per > 64 * waves) per = 64 * waves;   // 64 blocks per wave at most
    per = (per + unit - 1) / unit * unit;
    pl->chunk = int(per) * kBlock;
    pl->nsplit = int(blocks ? (blocks + per - 1) / per : 1);
    part_rows = size_t(heads) * pl->nsplit * size_t(rows);
    pl->groups = base * pl->nsplit;
  }
  const bool split = pl->nsplit > 1 || pl->shared > 0;
  pl->stash = a->weights && rows <= kStashRows;
  pl->stash_len = (all + kBlock - 1) / kBlock * kBlock;
  pl->joins = split ? heads * rows : 0;
  pl->q_tiles = int64_t(pl->tiles) * pl->tile_rows / 16;
  const int64_t slots = pl->stash ? 1024 : pl->kind == Plan::TILES ? 4 * kTileSlots : 4 * kBlock;   // of a workgroup
  pl->weighs = !a->weights ? 0 : heads * ((all + slots - 1) / slots);
  if (pl->weighs > 0 && pl->kind == Plan::TILES && (all + slots - 1) / slots > 65535) return false;
  // y and z of the grid
  if (q->batch > 65535 || int64_t(pl->tiles) * (pl->kind == Plan::TILES ? pl->nsplit : c->kv_heads) > 65535) return false;
  if (!launchable(pl->groups, 256) || !launchable(pl->joins + pl->weighs, 256)) return false;
  size_t o = 0;
  auto take = [&](bool used, size_t bytes) {
    const size_t at = o;
    if (used) o += (bytes + 255) / 256 * 256;
    return at;
  };
  pl->part = take(split, part_rows * c->head_dim * 4);
  pl->rl = take(split || pl->stash, part_rows * 8);
  pl->lse = take(a->weights && !pl->stash && !a->lse, size_t(q->batch) * a->q.tokens * a->q.heads * 4);
  pl->z = take(pl->stash, size_t(heads) * rows * pl->stash_len * 4);
  pl->where = take(pl->shared > 0, size_t(heads) * sizeof(int2));
  const bool frags = a->weights && pl->kind == Plan::TILES;
  pl->frags = take(frags, size_t(heads) * pl->q_tiles * (c->head_dim / 32 + 1) * 1024);
  pl->units = take(frags, size_t(heads) * pl->q_tiles * 16 * 4);
  pl->total = o;
  return true;
}

struct LaunchAttention {
  AttnParams p;
  Plan pl;
  hipStream_t st;
  template <int D, int G>
  int go() {
    const dim3 grid(unsigned(pl.nsplit), unsigned(pl.tiles * p.c.heads), unsigned(p.c.batch)), threads(Ring<D, G>::NW * 64);
    if (pl.kind == Plan::TILES) {
      const dim3 tiles(unsigned(p.c.heads), unsigned(pl.tiles * pl.nsplit), unsigned(p.c.batch));
      if (p.q.dtype == STAGQ_F16) hipLaunchKernelGGL((attend_tiles<D, G, true>), tiles, dim3(256), 0, st, p);
      else hipLaunchKernelGGL((attend_tiles<D, G, false>), tiles, dim3(256), 0, st, p);
    } else if (pl.kind == Plan::FEW) {
      const dim3 shares = p.shared ? dim3(unsigned(p.shared)) : grid;
      if constexpr (D / G >= 64) hipLaunchKernelGGL((attend_few<D, G>), shares, dim3(few_waves(D) * 64), 0, st, p);
    } else if (pl.nq == 1) {
      hipLaunchKernelGGL((attend_rows<D, G, 1>), grid, threads, 0, st, p);
    } else {
      if constexpr (D < 256) hipLaunchKernelGGL((attend_rows<D, G, 2>), grid, threads, 0, st, p);
    }
    int s = launched();
    if (s != STAGQ_OK) return s;
    const int64_t more = pl.joins + (pl.stash ? pl.weighs : 0);
    if (more > 0) {
      hipLaunchKernelGGL((finish_kernel<D>), dim3((unsigned)more), dim3(256), 0, st, p, unsigned(pl.joins));
      s = launched();
      if (s != STAGQ_OK) return s;
    }
    if (pl.weighs > 0 && pl.kind == Plan::TILES) {
      const dim3 groups(unsigned(p.c.heads), unsigned((p.max_len + 4 * kTileSlots - 1) / (4 * kTileSlots)), unsigned(p.c.batch));
      hipLaunchKernelGGL((weigh_tiles<D, G>), groups, dim3(256), 0, st, p);
      s = launched();
    } else if (pl.weighs > 0 && !pl.stash) {
      hipLaunchKernelGGL((weigh_kernel<D, G>), dim3((unsigned)pl.weighs), dim3(256), 0, st, p);
      s = launched();
    }
    return s;
  }
};

static int check_attention(const stagq_kv_cache* c, const stagq_kv_seqs* q, const stagq_kv_attn* a) {
  int st = check_cache(c);
  if (st == STAGQ_OK) st = check_seqs(c, q);
  if (st != STAGQ_OK) return st;
  if (!a) return STAGQ_EINVAL;
  if (a->q.heads < 1 || a->q.heads % c->kv_heads) return STAGQ_ESHAPE;
  st = check_tensor(a->q, a->q.heads, false, q->batch);
  if (st == STAGQ_OK) st = check_tensor(a->out, a->q.heads, false, q->batch);
  if (st != STAGQ_OK) return st;
  if (a->q.dtype != a->out.dtype || a->q.tokens != a->out.tokens) return STAGQ_EINVAL;
  if (a->out.data && a->out.data == a->q.data) return STAGQ_EINVAL;   // q is read until the end
  if (a->window < 0 || (a->window > 0 && !a->causal) || a->max_len < 0) return STAGQ_EINVAL;
  if (!(fabsf(a->scale) <= 0x1p100f)) return STAGQ_EINVAL;   // NaN, infinite or so large that its products are
  if (misaligned(a->q_lens, 4) || misaligned(a->lse, 4) || misaligned(a->weights, 4)) return STAGQ_EALIGN;
  if (a->weights && (a->weights_stride_seq < 0 || a->weights_stride_head < 0)) return STAGQ_EINVAL;
  if (!disjoint(a->out, q->batch, c->head_dim)) return STAGQ_EINVAL;
  if (a->weights && !disjoint(reach(c, q, a->max_len), q->batch, a->weights_stride_seq, c->kv_heads, a->weights_stride_head))
    return STAGQ_EINVAL;
  return STAGQ_OK;
}

}  // namespace kv
}  // namespace stagq

using namespace stagq::kv;

extern "C" {

size_t stagq_kv_attention_workspace(const stagq_kv_cache* c, const stagq_kv_seqs* q, const stagq_kv_attn* a) {
  Plan pl;
  if (check_attention(c, q, a) != STAGQ_OK || !plan(c, q, a, &pl)) return 0;
  return pl.total;
}

int stagq_kv_attention(const stagq_kv_cache* c, const stagq_kv_seqs* q, const stagq_kv_attn* a, void* workspace,
                       size_t workspace_bytes, void* hip_stream) {
  const int st = check_attention(c, q, a);
  if (st != STAGQ_OK) return st;
  if (q->batch == 0 || a->q.tokens == 0) return STAGQ_OK;
  Plan pl;
  if (!plan(c, q, a, &pl)) return STAGQ_ESHAPE;
  if (pl.total > 0 && !workspace) return STAGQ_EINVAL;
  if (misaligned(workspace, 256)) return STAGQ_EALIGN;
  if (workspace_bytes < pl.total) return STAGQ_ESIZE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  AttnParams p;
  p.c = make_cache(c, q);
  p.q = make_tensor(a->q);
  p.out = make_tensor(a->out);
  p.q_lens = a->q_lens;
  p.lse = a->lse ? a->lse : a->weights && !pl.stash ? reinterpret_cast<float*>(ws + pl.lse) : nullptr;
  p.weights = a->weights;
  p.wsb = a->weights_stride_seq;
  p.wsh = a->weights_stride_head;
  p.part = reinterpret_cast<float*>(ws + pl.part);
  p.part_rl = pl.nsplit > 1 || pl.shared > 0 || pl.stash ? reinterpret_cast<float*>(ws + pl.rl) : nullptr;
  p.stash = pl.stash ? reinterpret_cast<float*>(ws + pl.z) : nullptr;
  p.stash_len = pl.stash_len;
  p.q_frags = a->weights && pl.kind == Plan::TILES ? ws + pl.frags : nullptr;
  p.q_units = reinterpret_cast<float*>(ws + pl.units);
  p.q_tiles = pl.q_tiles;
  p.zero_rest = a->zero_rest != 0;
  p.scale2 = a->scale * kLog2e;
  p.gq = unsigned(a->q.heads / c->kv_heads);
  p.gq_inv = p.gq == 1 ? 0xffffffffu : unsigned((uint64_t(1) << 32) / p.gq);
  p.causal = a->causal != 0;
  p.window = a->window;
  p.max_len = c->pages > 0 ? reach(c, q, a->max_len) : 0;
  p.chunk = pl.chunk;
  p.nsplit = pl.nsplit;
  p.shared = pl.shared;
  p.where = reinterpret_cast<int2*>(ws + pl.where);
  p.tiles = pl.tiles;
  p.tile_rows = pl.tile_rows;
  p.rows = a->q.tokens * int(p.gq);
  return by_shape(c, LaunchAttention{p, pl, static_cast<hipStream_t>(hip_stream)});
}

}  // extern "C"
