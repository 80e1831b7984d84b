// Every byte of a block of the key/value cache belongs to exactly one pair
// half or code dword, in every shape.
#include <cstdio>
#include <vector>

#include "stagq_kv_layout.h"

using namespace stagq::kv;

static int fail(const char* what, int D, int G) {
  std::printf("%s D=%d G=%d\n", what, D, G);
  return 1;
}

int main() {
  const int shapes[][2] = {{64, 1}, {64, 2}, {96, 3}, {128, 1}, {128, 2}, {128, 4}, {256, 2}, {256, 4}, {256, 8}};
  for (auto& sh : shapes) {
    const int D = sh[0], G = sh[1];
    std::vector<int> used(block_bytes(D, G), 0);
    auto take = [&](uint32_t at, int n) {
      for (int i = 0; i < n; i++) {
        if (at + i >= used.size()) return false;
        used[at + i]++;
      }
      return true;
    };
    for (int t = 0; t < kBlock; t++)
      for (int g = 0; g < G; g++) {
        if (!take(kpair_at(G, t, g), 4)) return fail("K pair past the block", D, G);
        if (!take(vstep_at(G, vset(t), velem(t), g), 2) || !take(vstep_at(G, vset(t), velem(t), g) + 16, 2))
          return fail("V pair past the block", D, G);
        if (vtoken(vset(t), velem(t)) != t) return fail("token sets", D, G);
      }
    for (int lane = 0; lane < 64; lane++) {
      for (int u = 0; u < 2; u++)
        for (int ks = 0; ks < D / 32; ks++)
          if (!take(kcode_at(D, G, u, lane, ks), 4)) return fail("K codes past the block", D, G);
      for (int ct = 0; ct < D / 16; ct++)
        if (!take(vcode_at(D, G, lane, ct), 4)) return fail("V codes past the block", D, G);
    }
    for (int u : used)
      if (u != 1) return fail("a byte is not used once", D, G);
    if (block_bytes(D, G) % 16) return fail("block size", D, G);
    int seen = 0;
    for (int e = 0; e < 8; e++) seen |= 1 << nibble(e);
    if (seen != 255) return fail("nibbles", D, G);
    if (!supported(1, 32, 1, D, D / G)) return fail("supported", D, G);
  }
  if (supported(1, 48, 1, 128, 64) || supported(1, 64, 0, 128, 64) || supported(1, 64, 1, 80, 16) ||
      supported(-1, 64, 1, 128, 64) || supported(1, 64, 1, 96, 64) || supported(1, 64, 1, 64, 128))
    return fail("unsupported shapes taken", 0, 0);
  std::printf("layout ok\n");
  return 0;
}
