// Dense product of e4m3 operands with a scale per block of 128:
//   out[t, n] (+)= sum_b sx[t, b] sw[n / 128, b] sum_{k in block b} x[t, k] w[n, k]
//
// Weight rows are the matrix instruction's M side, tokens its N side; a lane
// holds 32 bytes of its row per block, and which 32 does not matter as long as
// both operands agree, because the whole block has one scale.
//
// The 8-bit matrix instructions of gfx950 align a group's products to the
// largest and drop what lies some 14 bits below: on normally distributed
// operands a sum is off by 1.5e-5 of its root mean square, on uniformly random
// codes by 5e-5 (measured; products that fit the window are exact).  fp32
// outputs therefore take the codes as bf16 (exact) through the bf16
// instruction, whose sums are fp32 (1e-8 and 8e-8 on the same operands).
#include <algorithm>

#include "fp8_plan.h"
#include "kernels.h"
#include "quant8.h"

namespace moe {
namespace {

// eight codes as bf16, exact
MOE_DEV bf16x8_t codes_to_bf16(uint32_t a, uint32_t b) {
  const bf16x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
  const bf16x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
  const bf16x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
  const bf16x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
  bf16x8_t r;
  r[0] = p0[0]; r[1] = p0[1]; r[2] = p1[0]; r[3] = p1[1];
  r[4] = p2[0]; r[5] = p2[1]; r[6] = p3[0]; r[7] = p3[1];
  return r;
}

typedef int i32x8_t __attribute__((ext_vector_type(8)));
// c + 16 rows times 16 columns over a block's 128 codes, times 2^(a - 127) of
// the row and 2^(b - 127) of the column: bytes 1 and 0 of `scales`
MOE_DEV f32x4_t mfma_f8(const u32x4_t (&w)[2], const u32x4_t (&x)[2], f32x4_t c, uint32_t scales) {
  i32x8_t a, b;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = (int)w[i >> 2][i & 3];
    b[i] = (int)x[i >> 2][i & 3];
  }
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 1, (int)scales, 0, (int)scales);
}

// value(s) of an output row, four consecutive columns from n on
template <typename O>
MOE_DEV void store_cols(O *row, int n, int N, bool vec, int accumulate, f32x4_t v) {
  if constexpr (sizeof(O) == 4) {
    if (vec && n + 3 < N) {
      f32x4_t *p = reinterpret_cast<f32x4_t *>(row + n);
      *p = accumulate ? *p + v : v;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < N) row[n + r] = accumulate ? row[n + r] + v[r] : v[r];
    }
  } else {
    bf16x4_t b;
#pragma unroll
    for (int r = 0; r < 4; ++r) b[r] = to_bf16(v[r]);
    if (vec && n + 3 < N) {
      *reinterpret_cast<bf16x4_t *>(row + n) = b;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < N) reinterpret_cast<__bf16 *>(row)[n + r] = b[r];
    }
  }
}

// Few tokens: the weights are the whole cost.  A work-group owns 16 MT weight
// rows and 16 NT tokens; its NW waves take the K blocks in turn, so that at any
// time they read a contiguous NW * 128 bytes of each row, and keep U blocks in
// flight each.  Both operands come straight from memory (the tokens' rows stay
// in the L2).  The waves' sums meet in LDS and are added in wave order.
template <int NT, int MT, int NW, int U, bool E8, typename O>
__global__ __launch_bounds__(64 * NW) void fp8_stream_kernel(Fp8Args g) {
  __shared__ f32x4_t part[NW][MT][NT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kg = lane >> 4;
  const int n0 = 16 * MT * blockIdx.x, t0 = 16 * NT * blockIdx.y;
  const int K = g.K, kb = (K + 127) / 128;
  const int nrows = min(16 * MT, g.N - n0), ntok = min(16 * NT, g.T - t0);
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(g.w + (long long)n0 * K, (uint32_t)nrows * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.x + t0 * g.ldx, (uint32_t)((ntok - 1) * g.ldx + K));
  const __amdgpu_buffer_rsrc_t xsr = make_rsrc(g.sx + t0 * g.ldsx, (uint32_t)((ntok - 1) * g.ldsx + kb));
  uint32_t wo[MT], xo[NT], xso[NT];
#pragma unroll
  for (int m = 0; m < MT; ++m) wo[m] = (uint32_t)min(16 * m + r16, nrows - 1) * (uint32_t)K + 16 * kg;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int t = min(16 * i + r16, ntok - 1);
    xo[i] = (uint32_t)(t * g.ldx) + 16 * kg;
    xso[i] = (uint32_t)(t * g.ldsx);
  }
  const long long srow = (long long)(n0 / 128) * kb;  // 16 MT divides 128

  f32x4_t acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[m][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int b0 = wave; b0 < kb; b0 += NW * U) {
    u32x4_t w[U][MT][2], x[U][NT][2];
    uint32_t xs[U][NT];
    float ws[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // blocks past the end re-read the last one, with a scale of zero
      const int b = min(b0 + NW * u, kb - 1);
      const uint32_t k0 = 128u * b;
      // a block that ends inside: its lanes past K read out of range, zeros
      const uint32_t d[2] = {k0 + 16 * kg < (uint32_t)K ? 0u : 0x70000000u,
                             k0 + 16 * kg + 64 < (uint32_t)K ? 64u : 0x70000000u};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int m = 0; m < MT; ++m) w[u][m][h] = buf_load16(wr, wo[m] + d[h], k0);
#pragma unroll
        for (int i = 0; i < NT; ++i) x[u][i][h] = buf_load16(xr, xo[i] + d[h], k0);
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) xs[u][i] = __builtin_amdgcn_raw_buffer_load_b8(xsr, xso[i], b, 0);
      if constexpr (E8) {
        const uint32_t e = static_cast<const uint8_t *>(g.sw)[srow + b];
        // 2^(e - 127); byte 0 is the subnormal 2^-127, 255 is NaN
        ws[u] = __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7FC00000u : e << 23);
      } else {
        ws[u] = static_cast<const float *>(g.sw)[srow + b];
      }
      if (b0 + NW * u >= kb) ws[u] = 0.f;
    }
    __builtin_amdgcn_sched_barrier(0);  // every load of the round is on its way before the first product
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f32x4_t p[MT][NT];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        bf16x8_t xb[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) xb[i] = codes_to_bf16(x[u][i][q >> 1][2 * (q & 1)], x[u][i][q >> 1][2 * (q & 1) + 1]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const bf16x8_t wb = codes_to_bf16(w[u][m][q >> 1][2 * (q & 1)], w[u][m][q >> 1][2 * (q & 1) + 1]);
#pragma unroll
          for (int i = 0; i < NT; ++i)
            p[m][i] = mfma_16x16x32(wb, xb[i], q == 0 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : p[m][i]);
        }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float sc = e8m0_to_float(xs[u][i]) * ws[u];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[m][i][r] = fmaf(p[m][i][r], sc, acc[m][i][r]);
      }
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) part[wave][m][i][lane] = acc[m][i];
  __syncthreads();
  for (int e = threadIdx.x; e < MT * NT * 64; e += 64 * NW) {
    const int m = e / (64 * NT), i = (e >> 6) % NT, l = e & 63;
    f32x4_t v = part[0][m][i][l];
#pragma unroll
    for (int q = 1; q < NW; ++q) v += part[q][m][i][l];
    const int t = 16 * i + (l & 15);
    if (t < ntok)
      store_cols<O>(static_cast<O *>(g.out) + (t0 + t) * g.ldo, n0 + 16 * m + 4 * (l >> 4), g.N, g.vec_out,
                    g.accumulate, v);
  }
}

// ---- many tokens
// A work-group of eight waves owns 64 MT weight rows and 32 NT tokens, a wave of
// it 16 MT rows and 16 NT tokens; K may be split over work-groups, whose sums
// fp8_join_kernel adds.  Both operands pass through ST LDS stages of one block
// of 128, filled by direct loads of rows' whole 128 bytes between the products.
//
// A row's 128 bytes are eight pieces of 16; piece p of row r lies at position
// p ^ (r / 2 % 8), so the 16 rows that a quarter wave reads at once, two to a
// 256-byte line of LDS, fall on different banks.
//
// F8 takes the 8-bit instruction.  With e8m0 weight scales both scales go
// through it, onto the sum (which keeps fp32's precision there: what the
// instruction drops is measured against the products, not the sum: measured
// within 2 units in the sum's last place); fp32 scales multiply a block's sum
// onto the fp32 sum, between the next tokens' products.  Without F8 the codes go
// through the bf16 instruction.
//
// 4096 x 6144 x 7168, the kernel alone, call after call, by card: 173 to 187 us
// to bf16 with fp32 scales (1.9 to 2.1 PFLOP/s), 162 to 174 with e8m0 scales
// (2.1 to 2.2), 327 to 343 to fp32 (1.05 to 1.1; the library's bf16 product of
// 8192^3 runs at 1.25, its 8-bit one without block scales takes 154 us here).
// What bounds the first is the issue of products and multiply-adds: without the
// latter (e8m0 scales) it is 11 us shorter, a third of the waves' cycles wait
// for an issue slot, and the 8-bit instructions are busy for 48 % of them; alone,
// fed from LDS one read each, these reach 3.0 PFLOP/s, 120 us.  Tried and slower,
// at a time when the kernel took 193 to 199: weights straight to the registers of
// the one wave that needs them (291: such a load touches 16 rows for 64 bytes
// each), 192 rows a tile (205), all of a block's loads at its start (+9).
constexpr int SCB = 8;   // blocks whose scales are in LDS at a time

// 16 bytes of LDS at a + O, issued without waiting
template <int O>
MOE_DEV void tread(uint32_t a, u32x4_t &v) {
  static_assert(O >= 0 && O < 65536, "offset field");
  asm volatile("ds_read_b128 %0, %1 offset:%2" : "=&v"(v) : "v"(a), "n"(O) : "memory");
}
template <int N>
MOE_DEV void twait() {
  asm volatile("s_waitcnt lgkmcnt(%0)" ::"n"(N) : "memory");
}
// ties a register to the wait before: its users stay behind it
MOE_DEV void ttie(u32x4_t &v) { asm volatile("" : "+v"(v)); }

template <int MT, int NT, int ST>
struct TileLds {
  uint8_t w[ST][64 * MT * 128], x[ST][32 * NT * 128];  // codes by stage
  // products of the scales, or both bytes, by block, the tile's block of rows,
  // half of the tokens, token % 16 and the wave's tile of tokens
  float s[SCB][MT > 2 ? 2 : 1][2][16][NT];
};

// tile `work` of tiles_n x tiles_t x splits, of rows from row0 on
template <int MT, int NT, int ST, bool F8, bool E8, typename O>
MOE_DEV void fp8_tile(const Fp8Args &g, int work, int row0, int tiles_n, int tiles_t, int splits, float *partial,
                      TileLds<MT, NT, ST> &l) {
  constexpr int TN = 64 * MT, TT = 32 * NT;
  // scales that are all powers of two go through the instruction, onto the sum
  constexpr bool ACC = F8 && E8;
  constexpr int WL = TN / 64, XL = TT / 64;  // direct loads of a wave per block, 8 rows each
  const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, kg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wn = wave & 3, wt = wave >> 2;
  // a few row tiles next to each other, then the next tokens: what an XCD works
  // on at a time is near square
  const int split = work / (tiles_n * tiles_t), id = work - split * tiles_n * tiles_t;
  const int per = 4 * tiles_t, grp = id / per, in = id - grp * per, gn = min(4, tiles_n - 4 * grp);
  const int n0 = row0 + (4 * grp + in % gn) * TN, t0 = in / gn * TT;
  const int K = g.K, kb = (K + 127) / 128;
  const int first = (int)((long long)split * kb / splits), nblk = (int)((long long)(split + 1) * kb / splits) - first;
  const int nrows = min(TN, g.N - n0), ntok = min(TT, g.T - t0);
  // rows and tokens past the end are out of range: zeros
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(g.w + (long long)n0 * K, (uint32_t)nrows * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.x + t0 * g.ldx, (uint32_t)((ntok - 1) * g.ldx + K));
  // direct load u of this wave fills rows 8 (8 u + wave) ..: lane i's 16 bytes
  // land at position i % 8 of row i / 8; the swizzle repeats every 16 rows, so
  // the piece is the same for every u
  const int r0 = 8 * wave + (lane >> 3), piece = (lane & 7) ^ (r0 >> 1 & 7);
  const uint32_t wo = (uint32_t)r0 * (uint32_t)K + 16 * piece, xo = (uint32_t)(r0 * g.ldx) + 16 * piece;
  const uint32_t wstep = 64u * (uint32_t)K, xstep = (uint32_t)(64 * g.ldx);
  // load u of block b of this split: the weights' first, then the tokens'
  auto request = [&](int stage, int b, auto uc) {
    constexpr int u = decltype(uc)::value;
    const uint32_t k0 = 128u * min(first + b, kb - 1);  // past the last block that one again, unused
    // of a block that ends inside, pieces past K read out of range
    const uint32_t out = k0 + 16 * piece < (uint32_t)K ? 0u : 0x70000000u;
    if constexpr (u < WL)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, (lds_void *)(l.w[stage] + (8 * u + wave) * 1024), 16,
                                               wo + u * wstep + out, k0, 0, 0);
    else if constexpr (u < WL + XL)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (lds_void *)(l.x[stage] + (8 * (u - WL) + wave) * 1024), 16,
                                               xo + (u - WL) * xstep + out, k0, 0, 0);
  };
  // the scales of blocks b0 .. b0 + SCB / 2 - 1, a token and half of the blocks
  // a thread: requested by one step, put into their half of the buffer by the next
  constexpr int SB = 512 / TT, SU = SCB / 2 / SB, SH = TN > 128 ? 2 : 1;
  const int st = tid & (TT - 1), su = wave / (TT / 64);
  uint32_t sx[SU], sw[SU][SH];
  auto request_scales = [&](int b0) {
#pragma unroll
    for (int u = 0; u < SU; ++u) {
      const int at = min(first + b0 + su + SB * u, kb - 1);
      sx[u] = g.sx[(t0 + min(st, ntok - 1)) * g.ldsx + at];
#pragma unroll
      for (int h = 0; h < SH; ++h) {
        const long long wi = (long long)(min(n0 + 128 * h, g.N - 1) / 128) * kb + at;
        if constexpr (E8) sw[u][h] = static_cast<const uint8_t *>(g.sw)[wi];
        else sw[u][h] = static_cast<const uint32_t *>(g.sw)[wi];
      }
    }
  };
  auto put_scales = [&](int b0) {
#pragma unroll
    for (int u = 0; u < SU; ++u)
#pragma unroll
      for (int h = 0; h < SH; ++h) {
        float *const to = &l.s[(b0 + su + SB * u) % SCB][h][st / (TT / 2)][st & 15][(st >> 4) % NT];
        if constexpr (ACC) {
          *reinterpret_cast<uint32_t *>(to) = sx[u] | sw[u][h] << 8;
          continue;
        }
        // a byte is 2^(e - 127); 0 is the subnormal 2^-127, 255 is NaN
        const uint32_t e = sw[u][h], f = !E8 ? e : e == 0 ? 0x00400000u : e == 255 ? 0x7FC00000u : e << 23;
        *to = e8m0_to_float(sx[u]) * __uint_as_float(f);
      }
  };

  f32x4_t acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[m][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const uint32_t sz = r16 >> 1;
  uint32_t wa[2], xa[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t at = 128 * r16 + 16 * ((kg + 4 * q) ^ sz);
    wa[q] = lds_addr(l.w[0]) + 2048 * MT * wn + at;
    xa[q] = lds_addr(l.x[0]) + 2048 * NT * wt + at;
  }
  const uint32_t sa = lds_addr(reinterpret_cast<const uint8_t *>(l.s[0][16 * MT * wn >= 128][wt][r16]));
  constexpr int SBYTES = sizeof(l.s[0]);

  static_for<ST - 1>([&](auto sc) {
    constexpr int s = decltype(sc)::value;
    static_for<WL + XL>([&](auto uc) { request(s, s, uc); });
  });
  request_scales(0);
  put_scales(0);
  twait<0>();  // in LDS before the first barrier (later ones are, by the reads' own waits behind them)
  auto step = [&](auto hc, int b) {
    constexpr int h = decltype(hc)::value;
    // this block has landed (of three stages: what was requested since is the
    // next), and every wave is done with the one before, whose stage is filled below
    __builtin_amdgcn_s_waitcnt(vmcnt_imm((WL + XL) * (ST - 2)));
    __builtin_amdgcn_s_barrier();
    if (b % (SCB / 2) == 0) request_scales(b + SCB / 2);
    else if (b % (SCB / 2) == 1) put_scales(b - 1 + SCB / 2);  // whose half nobody reads any more
    u32x4_t sc[NT / 4], w[MT][2], x[2][2];
    const uint32_t wh[2] = {wa[0] + h * TN * 128, wa[1] + h * TN * 128}, xh[2] = {xa[0] + h * TT * 128, xa[1] + h * TT * 128};
    auto read_x = [&](auto ic) {
      constexpr int i = decltype(ic)::value;
      tread<2048 * i>(xh[0], x[i & 1][0]);
      tread<2048 * i>(xh[1], x[i & 1][1]);
    };
    static_for<NT / 4>([&](auto qc) { tread<16 * decltype(qc)::value>(sa + b % SCB * SBYTES, sc[decltype(qc)::value]); });
    read_x(std::integral_constant<int, 0>{});
    static_for<MT>([&](auto mc) {
      constexpr int m = decltype(mc)::value;
      tread<2048 * m>(wh[0], w[m][0]);
      tread<2048 * m>(wh[1], w[m][1]);
    });
    read_x(std::integral_constant<int, 1>{});
    f32x4_t p[2][MT];
    bf16x8_t wb[F8 ? 1 : MT][4];
    auto add = [&](int i, int m) {
      const float f = __uint_as_float(sc[i >> 2][i & 3]);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[m][i][r] = fmaf(p[i & 1][m][r], f, acc[m][i][r]);
    };
    static_for<NT>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      if constexpr (i > 0) {
        if constexpr (i + 1 < NT) {
          read_x(std::integral_constant<int, i + 1>{});
          twait<2>();
        } else {
          twait<0>();
        }
        ttie(x[i & 1][0]);
        ttie(x[i & 1][1]);
      }
      // the loads into the free stage, spread over the products (of two stages:
      // the first half, the rest is their time to land)
      constexpr int over = ST == 2 ? NT / 2 : NT, per = (WL + XL + over - 1) / over;
      if constexpr (i < over)
        static_for<per>([&](auto uc) {
          request((h + ST - 1) % ST, b + ST - 1, std::integral_constant<int, per * i + decltype(uc)::value>{});
        });
      if constexpr (F8) {
        static_for<MT>([&](auto mc) {
          constexpr int m = decltype(mc)::value;
          if constexpr (i == 0) {  // the weights as they come
            twait<2 * (MT - 1 - m) + 2>();
            if constexpr (m == 0) {
#pragma unroll
              for (int q = 0; q < NT / 4; ++q) ttie(sc[q]);
              ttie(x[0][0]);
              ttie(x[0][1]);
            }
            ttie(w[m][0]);
            ttie(w[m][1]);
          }
          if constexpr (ACC) {
            acc[m][i] = mfma_f8(w[m], x[i & 1], acc[m][i], sc[i >> 2][i & 3]);
          } else {
            p[i & 1][m] = mfma_f8(w[m], x[i & 1], f32x4_t{0.f, 0.f, 0.f, 0.f}, 0x7F7Fu);
            if constexpr (i > 0) add(i - 1, m);
          }
        });
      } else {
        if constexpr (i == 0) {
          twait<2>();
#pragma unroll
          for (int q = 0; q < NT / 4; ++q) ttie(sc[q]);
          ttie(x[0][0]);
          ttie(x[0][1]);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            ttie(w[m][0]);
            ttie(w[m][1]);
#pragma unroll
            for (int c = 0; c < 4; ++c) wb[m][c] = codes_to_bf16(w[m][c >> 1][2 * (c & 1)], w[m][c >> 1][2 * (c & 1) + 1]);
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bf16x8_t xb = codes_to_bf16(x[i & 1][c >> 1][2 * (c & 1)], x[i & 1][c >> 1][2 * (c & 1) + 1]);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            p[i & 1][m] = mfma_16x16x32(wb[m][c], xb, c == 0 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : p[i & 1][m]);
        }
        if constexpr (i > 0) {
#pragma unroll
          for (int m = 0; m < MT; ++m) add(i - 1, m);
        }
      }
    });
    if constexpr (!ACC) {
#pragma unroll
      for (int m = 0; m < MT; ++m) add(NT - 1, m);
    }
  };
  for (int b = 0; b < nblk; b += ST)
    static_for<ST>([&](auto hc) {
      if (b + decltype(hc)::value < nblk) step(hc, b + decltype(hc)::value);
    });
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  const int nw = n0 + 16 * MT * wn, ldp = (g.N + 3) & ~3;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int t = TT / 2 * wt + 16 * i + r16;
    if (t < ntok)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int n = nw + 16 * m + 4 * kg;
        if (splits > 1) store_cols<float>(partial + ((long long)split * g.T + t0 + t) * ldp, n, ldp, true, 0, acc[m][i]);
        else store_cols<O>(static_cast<O *>(g.out) + (t0 + t) * g.ldo, n, g.N, g.vec_out, g.accumulate, acc[m][i]);
      }
  }
}

// block -> tile of `total`, as xcd_logical
MOE_DEV int tile_of(int block, int total) {
  const int t8 = (total + 7) & ~7, id = (block & 7) * (t8 >> 3) + (block >> 3);
  return block < t8 && id < total ? id : -1;
}

// fp32 out: tiles of 128 rows and 256 tokens
template <bool E8>
__global__ __launch_bounds__(512, 2) void fp8_tile_f32_kernel(Fp8Args g, int splits, float *partial) {
  __shared__ __attribute__((aligned(1024))) TileLds<2, 8, 2> l;
  const int tn = (g.N + 127) / 128, tt = (g.T + 255) / 256, work = tile_of(blockIdx.x, tn * tt * splits);
  if (work >= 0) fp8_tile<2, 8, 2, false, E8, float>(g, work, 0, tn, tt, splits, partial, l);
}

// bf16 out: tiles of 256 rows and 256 tokens for the first rows, of 256 rows and
// 128 tokens for the others; K is split where there are none of the first kind
template <bool E8>
__global__ __launch_bounds__(512, 2) void fp8_tile_bf16_kernel(Fp8Args g, int rows, int splits, float *partial) {
  __shared__ __attribute__((aligned(1024))) union L {
    TileLds<4, 8, 2> big;
    TileLds<4, 4, 3> small;
    __device__ L() {}
  } l;
  const int tn = rows / 256, tt = (g.T + 255) / 256, big = (tn * tt + 7) & ~7;
  if ((int)blockIdx.x < big) {
    const int work = tile_of(blockIdx.x, tn * tt);
    if (work >= 0) fp8_tile<4, 8, 2, true, E8, uint16_t>(g, work, 0, tn, tt, 1, partial, l.big);
    return;
  }
  const int sn = max(g.N - rows + 255, 0) / 256, st = (g.T + 127) / 128, work = tile_of(blockIdx.x - big, sn * st * splits);
  if (work >= 0) fp8_tile<4, 4, 3, true, E8, uint16_t>(g, work, rows, sn, st, splits, partial, l.small);
}

// the splits' sums in order, four columns a thread
template <typename O>
__global__ __launch_bounds__(256) void fp8_join_kernel(Fp8Args g, int splits, const float *partial) {
  const int per = (g.N + 3) / 4;  // rows of partial are whole groups of four
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, stride = (long long)g.T * per;
  if (i >= stride) return;
  const int t = (int)(i / per), n = 4 * (int)(i - (long long)t * per);
  const f32x4_t *p = reinterpret_cast<const f32x4_t *>(partial) + i;
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int s = 0; s < splits; ++s) v += p[s * stride];
  store_cols<O>(static_cast<O *>(g.out) + t * g.ldo, n, g.N, g.vec_out, g.accumulate, v);
}

template <int NT, int MT, int NW, int U>
void stream_by_type(const Fp8Args &g, bool e8, bool out_bf16, hipStream_t st) {
  const dim3 gr((unsigned)((g.N + 16 * MT - 1) / (16 * MT)), (unsigned)((g.T + 16 * NT - 1) / (16 * NT))), blk(64 * NW);
  if (e8) {
    if (out_bf16) hipLaunchKernelGGL((fp8_stream_kernel<NT, MT, NW, U, true, uint16_t>), gr, blk, 0, st, g);
    else hipLaunchKernelGGL((fp8_stream_kernel<NT, MT, NW, U, true, float>), gr, blk, 0, st, g);
  } else {
    if (out_bf16) hipLaunchKernelGGL((fp8_stream_kernel<NT, MT, NW, U, false, uint16_t>), gr, blk, 0, st, g);
    else hipLaunchKernelGGL((fp8_stream_kernel<NT, MT, NW, U, false, float>), gr, blk, 0, st, g);
  }
}

}  // namespace

size_t fp8_workspace_bytes(int T, int N, int K) { return fp8_partial_bytes(T, N, K); }

hipError_t launch_fp8_gemm(const Fp8Args &g, bool e8, bool out_bf16, void *ws, hipStream_t st) {
  const Fp8Plan plan = fp8_plan(g.T, g.N, g.K, out_bf16);
  const TilePlan &p = plan.tile;
  if (!plan.stream) {
    float *partial = static_cast<float *>(ws);
    auto up8 = [](int v) { return (unsigned)((v + 7) & ~7); };
    const dim3 blk(512);
    if (out_bf16) {
      const int rest = std::max(g.N - p.rows, 0);
      const dim3 gr(up8(p.rows / 256 * ((g.T + 255) / 256)) + up8((rest + 255) / 256 * ((g.T + 127) / 128) * p.splits));
      if (e8) hipLaunchKernelGGL(fp8_tile_bf16_kernel<true>, gr, blk, 0, st, g, p.rows, p.splits, partial);
      else hipLaunchKernelGGL(fp8_tile_bf16_kernel<false>, gr, blk, 0, st, g, p.rows, p.splits, partial);
    } else {
      const dim3 gr(up8((g.N + 127) / 128 * ((g.T + 255) / 256) * p.splits));
      if (e8) hipLaunchKernelGGL(fp8_tile_f32_kernel<true>, gr, blk, 0, st, g, p.splits, partial);
      else hipLaunchKernelGGL(fp8_tile_f32_kernel<false>, gr, blk, 0, st, g, p.splits, partial);
    }
    if (p.splits > 1) {
      const dim3 jr((unsigned)(((long long)g.T * ((g.N + 3) / 4) + 255) / 256));
      if (out_bf16) hipLaunchKernelGGL(fp8_join_kernel<uint16_t>, jr, dim3(256), 0, st, g, p.splits, partial);
      else hipLaunchKernelGGL(fp8_join_kernel<float>, jr, dim3(256), 0, st, g, p.splits, partial);
    }
  } else if (g.T <= 16) {
    // Two row tiles a work-group halve the tokens' loads, which are as many as the
    // weights', where rows are many: 6144 (192 work-groups) is the fewest at which
    // that was measured faster, 3584 the most at which it was slower.  Long rows
    // keep 16 waves busy.  Measured at (tokens, N, K), the three below
    // in order: (16, 7168, 33792) 61 / 72 / 74 us, (4, 7168, 33792) 53 / 56 / 59,
    // (16, 6144, 7168) 16.3 / 18.2 / 19.3, (16, 3584, 7168) 14.2 / 10.4 / 11.4,
    // (1, 7168, 33792) 48.2 / 46.1 / 49.7, (4, 6144, 1024) - / 10.9 / 9.0.
    if (g.T > 1 && g.N >= 6144) stream_by_type<1, 2, 8, 2>(g, e8, out_bf16, st);
    else if (g.K >= 4096) stream_by_type<1, 1, 16, 1>(g, e8, out_bf16, st);
    else stream_by_type<1, 1, 8, 4>(g, e8, out_bf16, st);
  } else if (g.T <= 32) {
    stream_by_type<2, 1, 8, 2>(g, e8, out_bf16, st);
  } else if (g.K >= 4096 && (g.N + 15LL) / 16 * ((g.T + 63) / 64) <= 256) {
    // one row tile a work-group while that is one work-group a CU at most: 33
    // tokens, 3584 x 7168 16.4 us (with two 19.6), 64 and 895 x 7168 20.2 (23.5);
    // with 384 work-groups 42 (28.2 at 64 tokens, 6144 x 7168), and short rows
    // gain nothing (40 tokens, 2048 x 2048 10.6 against 10.0)
    stream_by_type<4, 1, 8, 1>(g, e8, out_bf16, st);
  } else {
    stream_by_type<4, 2, 8, 1>(g, e8, out_bf16, st);
  }
  return hipGetLastError();
}

}  // namespace moe
