// Host checks shared by the entry points of the key/value cache.
#pragma once
#include <stdint.h>

#include "stagq_kv_device.h"

namespace stagq {
namespace kv {

inline bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

inline int check_cache(const stagq_kv_cache* c) {
  if (!c) return STAGQ_EINVAL;
  if (!supported(c->pages, c->page_tokens, c->kv_heads, c->head_dim, c->group)) return STAGQ_ESHAPE;
  if (c->pages > 0 && !c->buf) return STAGQ_EINVAL;
  if (misaligned(c->buf, 256)) return STAGQ_EALIGN;
  if (c->bytes < stagq_kv_bytes(c)) return STAGQ_ESIZE;
  return STAGQ_OK;
}

inline int check_seqs(const stagq_kv_cache* c, const stagq_kv_seqs* q) {
  if (!q || q->batch < 0 || q->table_width < 0) return STAGQ_EINVAL;
  if (q->batch == 0) return STAGQ_OK;
  if (!q->lengths || (q->table_width > 0 && !q->table)) return STAGQ_EINVAL;
  if (misaligned(q->table, 4) || misaligned(q->lengths, 4)) return STAGQ_EALIGN;
  if (q->batch > 1 && q->table_stride < q->table_width) return STAGQ_EINVAL;
  if (q->batch > (1 << 20) || int64_t(q->table_width) * c->page_tokens > (int64_t(1) << 30)) return STAGQ_ESHAPE;   // slots are 31-bit numbers
  return STAGQ_OK;
}

// heads: as many as the tensor must have; f32: whether fp32 is taken.
inline int check_tensor(const stagq_kv_tensor& t, int heads, bool f32, int batch) {
  if (t.dtype != STAGQ_F16 && t.dtype != STAGQ_BF16 && !(f32 && t.dtype == STAGQ_F32)) return STAGQ_EINVAL;
  if (t.tokens < 0 || t.heads != heads) return STAGQ_ESHAPE;
  if (batch == 0 || t.tokens == 0) return STAGQ_OK;
  if (!t.data) return STAGQ_EINVAL;
  if (t.stride_seq < 0 || t.stride_token < 0 || t.stride_head < 0) return STAGQ_EINVAL;
  if (misaligned(t.data, 16) || t.stride_seq % 8 || t.stride_token % 8 || t.stride_head % 8) return STAGQ_EALIGN;
  return STAGQ_OK;
}

// Whether an array that a call writes is free of overlaps with itself: rows of
// `inner` adjacent elements, and the strides nested (each one covers what the
// smaller ones span).
inline bool disjoint(int64_t inner, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2 = 1, int64_t s2 = 0) {
  int64_t n[3] = {n0, n1, n2}, s[3] = {s0, s1, s2}, extent = inner;
  for (int done = 0; done < 3; done++) {
    int at = -1;
    for (int i = 0; i < 3; i++)
      if (n[i] > 1 && (at < 0 || s[i] < s[at])) at = i;
    if (at < 0) return true;
    if (s[at] < extent) return false;
    if (s[at] > INT64_MAX / 4 / n[at]) return false;
    extent += s[at] * (n[at] - 1);
    n[at] = 1;
  }
  return true;
}
inline bool disjoint(const stagq_kv_tensor& t, int batch, int head_dim) {
  return disjoint(head_dim, batch, t.stride_seq, t.tokens, t.stride_token, t.heads, t.stride_head);
}

inline Cache make_cache(const stagq_kv_cache* c, const stagq_kv_seqs* q) {
  Cache r;
  r.buf = static_cast<uint8_t*>(c->buf);
  r.table = q->table;
  r.lengths = q->lengths;
  r.table_stride = q->table_stride;
  r.page_bytes = page_bytes(c->page_tokens, c->kv_heads, c->head_dim, c->group);
  r.head_bytes = uint32_t(head_bytes(c->page_tokens, c->head_dim, c->group));
  r.pages = c->pages;
  r.width = q->table_width;
  r.shift = __builtin_ctz(unsigned(c->page_tokens));
  r.heads = c->kv_heads;
  r.batch = q->batch;
  return r;
}

inline Tensor make_tensor(const stagq_kv_tensor& t) {
  return Tensor{static_cast<uint8_t*>(t.data), t.dtype, t.tokens, t.heads, t.stride_seq, t.stride_token, t.stride_head};
}

// Slots a call may reach: max_len (0: all) within the table.
inline int64_t reach(const stagq_kv_cache* c, const stagq_kv_seqs* q, int32_t max_len) {
  const int64_t all = int64_t(q->table_width) * c->page_tokens;
  return max_len > 0 && max_len < all ? max_len : all;
}

// A launch holds fewer than 2^31 workgroups and 2^32 threads.
inline bool launchable(int64_t groups, int threads) { return groups * threads < (int64_t(1) << 32); }

// Calls f.template operator()<D, G>() for the cache's head size and groups.
template <class F>
inline int by_shape(const stagq_kv_cache* c, F f) {
  const int G = c->head_dim / c->group;
  switch (c->head_dim) {
    case 64: return G == 1 ? f.template go<64, 1>() : f.template go<64, 2>();
    case 96: return f.template go<96, 3>();
    case 128:
      return G == 1 ? f.template go<128, 1>() : G == 2 ? f.template go<128, 2>() : f.template go<128, 4>();
    default:
      return G == 2 ? f.template go<256, 2>() : G == 4 ? f.template go<256, 4>() : f.template go<256, 8>();
  }
}

inline int launched() { return hipGetLastError() == hipSuccess ? STAGQ_OK : STAGQ_EHIP; }

}  // namespace kv
}  // namespace stagq
