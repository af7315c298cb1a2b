// Which kernels of the MXFP4 products run, and how they are cut: host code alone, a
// function of the sizes.
#pragma once
#include <stddef.h>

#include <algorithm>

namespace moe {

// How a product of T rows and N columns over K is cut, and what it then takes, in us.
//
// Stream: work-groups of 32 columns and up to 64 rows, whose eight waves take the
// stages of 256 inputs in turn; one on a CU at a time.
// Tiles: work-groups of 256 columns and `rows` rows (64 to 256).  With more of them
// than CUs (256) the first `cut` column tiles may have 256 rows, which read least for
// a product, and the others fewer, which fill the last round better.  Where tiles are
// fewer than the CUs K may be split, and the parts' sums are joined.
//
// Measured, bf16 out, K = 7168 unless said, us: stream / tiles of 64 rows / of 128 /
// of 256 (K split so that all CUs have a part), and what this rule takes:
// (tokens, columns) (32, 3584) 8.9 / 14.9 / - / -, stream; (64, 3584) 13.4 / 17.4,
// stream; (64, 7168, K 33792) 61 / 38, tiles; (128, 3584) 14.6 / 17.8 / 21.5, stream;
// (301, 895) 14.1 / 16.9 / 19.7 / 22.2, stream; (512, 3584) 51 / 21.9 / 24.1 / 34,
// tiles of 64; (1024, 3584) 87 / 25.2 / 31.1 / 38.7; (2048, 3584) 166 / 51 / 38.7 /
// 52.7, tiles of 128; (4096, 4096) - / 108 / 80 / 68, tiles of 256; (4096, 6144)
// - / 151 / 114 / 110, one round of 256 rows and one of 128: 105.
struct Mx4Plan {
  bool stream;
  int rows, cut, splits;
  double us;
};

constexpr long long MX4_CUS = 256;
inline long long mx4_up(long long a, long long b) { return (a + b - 1) / b; }

inline double mx4_stream_us(int T, int N, int K) {
  const long long stages = mx4_up(K, 256), groups = mx4_up(N, 32) * mx4_up(T, 64);
  const double stage = T <= 16 ? 1.7 : T <= 32 ? 2.4 : 3.3;  // of eight waves
  return 1.0 + stage * (double)(mx4_up(groups, MX4_CUS) * mx4_up(stages, 8));
}
// the ends of a kernel of such tiles, and a stage of them on every CU
inline double mx4_ends_us(int rows) { return rows <= 64 ? 4.5 : rows <= 128 ? 5.0 : rows <= 192 ? 6.0 : 7.5; }
inline double mx4_stage_us(int rows) { return rows <= 64 ? 0.75 : rows <= 128 ? 1.1 : rows <= 192 ? 1.45 : 1.85; }

inline Mx4Plan mx4_plan(int T, int N, int K) {
  const long long stages = mx4_up(K, 256), pairs = mx4_up(K, 512), nb = mx4_up(N, 256);
  Mx4Plan best{true, 0, 0, 1, mx4_stream_us(T, N, K)};
  if (T <= 16) return best;  // a tile would be three quarters empty
  const double out = 0.4e-6 * T * N;                               // rows written
  const double in = ((double)N + T) * K * (17.0 / 32.0) / 5.3e6;  // operands read once
  for (int rows = 64; rows <= 256; rows += 64) {
    const long long tiles = mx4_up(T, rows) * nb;
    for (long long s = 1; s <= std::min(pairs, 16LL) && (s == 1 || tiles * s <= MX4_CUS); ++s) {
      const long long per = s > 1 ? 2 * mx4_up(pairs, s) : stages;
      const double join = s > 1 ? 6.0 + 0.3 * (double)s + 0.5e-6 * (double)s * T * N : 0.0;
      const double run = mx4_stage_us(rows) * (double)(mx4_up(tiles * s, MX4_CUS) * per);
      const double us = mx4_ends_us(rows) + out + join + std::max(run, in);
      if (us < best.us) best = {false, rows, 0, (int)s, us};
    }
    // whole rounds of the largest tiles first
    const long long tt = mx4_up(T, 256);
    for (long long rounds = 1; rows < 256 && rounds <= 64; ++rounds) {
      const long long cut = rounds * MX4_CUS / tt;
      if (cut >= nb) break;
      if (cut == 0) continue;
      const double run = (double)stages * (mx4_stage_us(256) * (double)mx4_up(cut * tt, MX4_CUS) +
                                           mx4_stage_us(rows) * (double)mx4_up((nb - cut) * mx4_up(T, rows), MX4_CUS));
      const double us = mx4_ends_us(256) + out + std::max(run, in);
      if (us < best.us) best = {false, rows, (int)cut, 1, us};
    }
  }
  return best;
}

// bytes of the parts' sums
inline size_t mx4_partial_bytes(int T, int N, int K) {
  const Mx4Plan p = mx4_plan(T, N, K);
  return !p.stream && p.splits > 1 ? (size_t)p.splits * T * ((N + 3) / 4) * 16 : 0;
}

// ---- expert products
constexpr int MX4_TILE_ROWS = 256;  // rows of a tile, at most

// An expert's rows up to which its weights are streamed by waves of their own.  The down product of 256
// tokens over 64 experts, four each, uneven: 61 us at 16, 61 at 8, 68 at 24, 69 at 32; gate and up of 64
// tokens 94, 91, 101, 105; of 1024 tokens, two each, 168, 169, 188, 184.
// With 32 rows an expert on average and more, tiles take them all, as the few that the others would have are
// not worth a launch behind them: of 4096 tokens, two of 112 experts each, gate and up 339 with both, 330 with
// tiles alone, down 191 and 184; of 1024 tokens, two of 64 each, down 116 and 100 (with experts' weights e^1.5
// apart, the rows with a few of them, 67 and 71).
inline int mx4_few_rows(int E, int P) { return P >= 32LL * E ? 0 : 16; }
inline int mx4_few_chunks(int E, int P) { return mx4_few_rows(E, P) > 0 ? std::min(E, P) : 0; }
inline int mx4_many_chunks(int E, int P) { return P / MX4_TILE_ROWS + std::min(E, P / (mx4_few_rows(E, P) + 1)); }
// work-groups of the stream kernel for a chunk
inline int mx4_stream_groups(int N, bool pair) { return (N + (pair ? 63 : 127)) / (pair ? 64 : 128); }
// chunks of up to 64 rows, at most, of work-groups that look for them themselves
inline int mx4_found_chunks(int E, int P) { return P / 64 + std::min(E, P); }
// Few work-groups do so, in place of a launch before, and stream whatever rows an expert has.  That saves the list
// and, at decode, an empty launch, and loses where experts have many rows, as their weights are read once for every
// 64.  Both sides at the layer's sizes (gate and up / down), experts x rows each, us, found / listed: 1 x 1 10 / 13,
// 8 / 11; 16 x 1 42 / 40, 21 / 24; 8 x 16 26 / 31, 14 / 18; 16 x 16 44 / 47, 25 / 29; 4 x 32 19 / 23, 14 / 17; 1 x 256
// 25 / 37, 20 / 28.  Lost: 4 x 64 29 / 24, 21 / 17; 4 x 128 45 / 29, 22 / 21; 8 x 64 50 / 29, 25 / 23; 4 x 256 62 / 42,
// 36 / 31.  Past 1024 work-groups: 16 x 32 54 / 52, 30 / 29; 16 x 64 77 / 54, 42 / 31; 4 x 512 113 / 45, 65 / 36.  Small
// layers: 32 x 32 of 128 x 128 6.9 / 10.1, 5.7 / 9.3, of 768 x 512 11.5 / 12.8, 8.0 / 10.9; 8 x 256 of 768 x 512
// 16 / 22, 11 / 16; past 1024, 32 x 128 of 768 x 512 25 / 17, 15 / 15.  A rule on rows an expert would take lists from
// some 64 of them in four experts and more where the weights are large.
inline bool mx4_finds_chunks(int E, int P, int groups) { return (long long)mx4_found_chunks(E, P) * groups <= 1024; }

}  // namespace moe
