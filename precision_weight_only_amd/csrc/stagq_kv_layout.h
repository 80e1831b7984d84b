// Layout of the paged key/value cache in 4 bits, shared by its host checks and
// the gfx950 kernels.
//
// A page holds page_tokens (P = 32, 64, 128 or 256) consecutive tokens of one
// sequence for every kv head; head by head, each head's P / 32 "blocks" of 32
// tokens in order.  A block is what one wave reads per step, and its codes lie
// in the order in which the lanes of a 16 x 16 x 32 matrix instruction take
// their operands, so a lane loads its own dwords and only masks them:
//
//   K pairs   2 units x G groups x 16 tokens x 4 B   (fp16 lo | fp16 s << 16)
//   V pairs   G groups x 4 token sets x (8 fp16 s, 8 fp16 lo)
//   K codes   2 units x 64 lanes x D/32 dwords
//   V codes   64 lanes x D/16 dwords
//
// with D = head_dim, G = D / group, j = lane / 16 throughout:
//
//   K: unit u holds tokens 16u .. 16u + 15 of the block.  Lane j * 16 + t of
//      unit u, dword ks: channels 32 ks + 8 j + e, e = 0..7, of token 16 u + t.
//   V: token set j holds the tokens 4j + e (e = 0..3) and 16 + 4j + (e - 4)
//      (e = 4..7): the tokens whose scores a lane of set j holds after the
//      product with K, so the probabilities feed the second product from the
//      registers they were computed in.  Lane j * 16 + c, dword ct: channel
//      16 ct + c of the tokens e = 0..7 of set j.
//   Element e of a dword sits in nibble e / 2 + 4 (e mod 2): nibbles i and
//      i + 4 lie at the same place of the dword's two 16-bit halves and hold
//      the neighbours (2i, 2i + 1).
//
// A lane's dwords lie together in chunks of up to 16 bytes (kchunk, vchunk
// dwords), and the 64 lanes' chunks one after another, so every load of a wave
// is one contiguous piece.
#pragma once
#include <stddef.h>
#include <stdint.h>

#ifdef __HIPCC__
#define STAGQ_KV_HD __host__ __device__ constexpr
#else
#define STAGQ_KV_HD constexpr
#endif

namespace stagq {
namespace kv {

constexpr int kBlock = 32;          // tokens of a block
constexpr int kMaxHeads = 1024;     // kv heads of a cache, at most
constexpr float kClamp = 32768.0f;  // largest magnitude held (lo + 15 s stays finite in fp16)

STAGQ_KV_HD int kchunk(int D) { return D / 32 < 4 ? D / 32 : 4; }
STAGQ_KV_HD int vchunk(int D) { return (D / 16) % 4 == 0 ? 4 : 3; }

STAGQ_KV_HD uint32_t pair_bytes(int G) { return 128u * G; }  // of K or of V, per block
STAGQ_KV_HD uint32_t off_vpair(int G) { return 128u * G; }
STAGQ_KV_HD uint32_t off_kcode(int G) { return 256u * G; }
STAGQ_KV_HD uint32_t off_vcode(int D, int G) { return 256u * G + 16u * D; }
STAGQ_KV_HD uint32_t block_bytes(int D, int G) { return 256u * G + 32u * D; }

// Byte offsets inside a block.
STAGQ_KV_HD uint32_t kpair_at(int G, int token, int g) {
  return uint32_t(((token >> 4) * G + g) * 16 + (token & 15)) * 4u;
}
STAGQ_KV_HD int vset(int token) { return (token & 15) >> 2; }
STAGQ_KV_HD int velem(int token) { return (token & 3) + 4 * (token >> 4); }
STAGQ_KV_HD int vtoken(int set, int e) { return 4 * set + (e & 3) + 16 * (e >> 2); }
STAGQ_KV_HD uint32_t vstep_at(int G, int set, int e, int g) {  // s; lo 16 bytes further
  return off_vpair(G) + uint32_t((g * 4 + set) * 16 + e) * 2u;
}
STAGQ_KV_HD uint32_t kcode_at(int D, int G, int unit, int lane, int ks) {
  const int c = kchunk(D);
  return off_kcode(G) + uint32_t(((unit * (D / 32 / c) + ks / c) * 64 + lane) * c + ks % c) * 4u;
}
STAGQ_KV_HD uint32_t vcode_at(int D, int G, int lane, int ct) {
  const int c = vchunk(D);
  return off_vcode(D, G) + uint32_t(((ct / c) * 64 + lane) * c + ct % c) * 4u;
}
STAGQ_KV_HD int nibble(int e) { return (e >> 1) + 4 * (e & 1); }

inline bool supported(int pages, int P, int heads, int D, int g) {
  if (pages < 0 || heads < 1 || heads > kMaxHeads) return false;
  if (P != 32 && P != 64 && P != 128 && P != 256) return false;
  if (D != 64 && D != 96 && D != 128 && D != 256) return false;
  return (g == 32 || g == 64 || g == 128) && D % g == 0;
}
inline uint64_t head_bytes(int P, int D, int g) { return uint64_t(P / kBlock) * block_bytes(D, D / g); }
inline uint64_t page_bytes(int P, int heads, int D, int g) { return head_bytes(P, D, g) * uint64_t(heads); }

}  // namespace kv
}  // namespace stagq
