// Which kernel of the 8-bit product runs, and how it is cut: host code alone,
// a function of the sizes and the output's type.
#pragma once
#include <stddef.h>

#include <algorithm>

namespace moe {

// How the tile kernels cut a product, and what it then takes, in us: 8 for the
// ends of a kernel; of a turn (256 tiles, one a CU) 1.75 a block for tiles of
// 256 x 256, 1.15 for 256 rows x 128 tokens, 1.45 for 128 x 256 with fp32 sums.
// The first kind reads least per product, the second fills turns better:
// 4096 tokens and 6144 rows of 7168 are 384 of the first (half of the second
// turn empty, 207 us), 768 of the second (three turns, 199), or 256 of the first
// and then 256 of the second (186, all on one card).  Where the tiles are fewer than the CUs, K is
// split into about one work-group a CU, of four blocks at least, and the parts'
// sums are written and read at 3 TB/s.
struct TilePlan {
  int rows;  // bf16 out: rows in tiles of the first kind
  int splits;
  double us;
};
inline TilePlan tile_plan(int T, int N, int K, bool out_bf16) {
  const long long kb = (K + 127) / 128, CUS = 256;
  auto up = [](long long a, long long b) { return (a + b - 1) / b; };
  const long long small = out_bf16 ? up(N, 256) * up(T, 128) : up(N, 128) * up(T, 256);
  const double step = out_bf16 ? 1.15 : 1.45;
  const long long s = std::max(1LL, std::min(std::min(CUS / small, kb / 4), 16LL));
  TilePlan best{0, (int)s, 8 + step * (double)(up(kb, s) * up(small * s, CUS)) + (s > 1 ? 2.6e-6 * s * T * N : 0.0)};
  if (!out_bf16 || s > 1) return best;
  // whole turns of the first kind, or all of it
  const long long tn = up(N, 256), tt = up(T, 256);
  for (long long turns = 1; turns <= up(tn * tt, CUS); ++turns) {
    const long long n = std::min(tn, turns * CUS / tt);
    if (n == 0) continue;
    const double us = 8 + (double)kb * (1.75 * (double)up(n * tt, CUS) + step * (double)up((tn - n) * up(T, 128), CUS));
    if (us < best.us) best = {(int)(256 * n), 1, us};
  }
  return best;
}
// Whether the stream kernel is taken above 64 tokens: its work-groups of 32 rows
// and 64 tokens take 0.38 us a block, one a CU at a time.  Measured at K = 7168,
// stream against tiles in us, (tokens, rows), bf16 out then fp32 out:
// (128, 6144) 48 / 27, 48 / 34; (512, 6144) 137 / 43, 136 / 66; (1024, 895)
// 46 / 25, 46 / 30; (301, 895) 23.8 / 21.7, 23.9 / 25.1; (512, 895) 24.5 / 23,
// 25 / 27; at K = 512 (300, 3584) 11 / 11, 11 / 14.  Where they are within some
// 5 % of each other the rule may take the slower: it does at (301, 895) to fp32
// and at (512, 895) to bf16.
inline bool stream_fits(const TilePlan &tile, int T, int N, int K) {
  const long long groups = (long long)((N + 31) / 32) * ((T + 63) / 64);
  return 2.5 + 0.38 * ((K + 127) / 128) * (double)((groups + 255) / 256) <= tile.us;
}

struct Fp8Plan {
  bool stream;
  TilePlan tile;  // unless stream
};
inline Fp8Plan fp8_plan(int T, int N, int K, bool out_bf16) {
  // Up to 64 tokens the stream kernel, whose sums are fp32 in both outputs, so
  // that decode batches of any size round alike.  To fp32 the tiles are no
  // faster where there are rows ((64, 6144) 28 / 30 us, (33, 3584) 16.4 / 20.7);
  // to bf16 they are from about 64 tokens on ((64, 6144) 28 / 21, (64, 895)
  // 20 / 15, (33, 3584) 16.5 / 15.5).
  if (T <= 64) return {true, {}};
  const TilePlan tile = tile_plan(T, N, K, out_bf16);
  return {stream_fits(tile, T, N, K), tile};
}

// bytes of the parts' sums, for either output
inline size_t fp8_partial_bytes(int T, int N, int K) {
  size_t need = 0;
  for (const bool out_bf16 : {false, true}) {
    const Fp8Plan p = fp8_plan(T, N, K, out_bf16);
    if (!p.stream && p.tile.splits > 1) need = std::max(need, (size_t)p.tile.splits * T * ((N + 3) / 4) * 16);
  }
  return need;
}

}  // namespace moe
