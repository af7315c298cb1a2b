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
// 16 rows times 16 columns over a block's 128 codes, scales of one
MOE_DEV f32x4_t mfma_f8(const u32x4_t (&w)[2], const u32x4_t (&x)[2]) {
  i32x8_t a, b;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a[i] = (int)w[i >> 2][i & 3];
    b[i] = (int)x[i >> 2][i & 3];
  }
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 127, 0, 127);
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
// A work-group of four waves owns 64 MT weight rows and 16 NT tokens; a wave has
// 16 MT rows and all the tokens.  So no two waves need the same weights: those
// go from memory straight to registers, one block of 128 ahead, and only the
// tokens' codes pass through LDS (two buffers, one barrier a block), which
// halves the reads that bound a tile with both operands in LDS.  Two work-groups
// a CU cover each other's waits.
//
// A row's 128 bytes of a block are eight pieces of 16; piece p of row t lies at
// position p ^ (t / 2 % 8), so the 16 rows that a quarter wave reads at once,
// two to a 256-byte line of LDS, fall on different banks.
//
// F8: a block's sum by the 8-bit instruction, from zero, then times both scales
// onto the fp32 sum.  Otherwise the codes go through the bf16 instruction.
template <int MT, int NT, bool F8, bool E8, typename O>
__global__ __launch_bounds__(256, 2) void fp8_tile_kernel(Fp8Args g, int tiles_n, int tiles_t) {
  constexpr int TN = 64 * MT, TT = 16 * NT;  // tile
  constexpr int PIECES = TT * 8 / 256;       // 16-byte pieces of the tokens' codes a thread moves
  __shared__ u32x4_t lx[2][TT * 8];
  __shared__ float ls[2][TT];
  const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, kg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int id = xcd_logical(tiles_n * tiles_t);
  if (id < 0) return;
  // eight row tiles next to each other, then the next tokens: what an XCD works
  // on at a time is near square
  const int per = 8 * tiles_t, grp = id / per, in = id - grp * per, gn = min(8, tiles_n - 8 * grp);
  const int n0 = (8 * grp + in % gn) * TN, t0 = in / gn * TT;
  const int K = g.K, kb = (K + 127) / 128;
  const int nw = n0 + 16 * MT * wave;  // the wave's rows
  const int nrows = min(max(g.N - nw, 0), 16 * MT), ntok = min(TT, g.T - t0);
  // rows and tokens past the end are out of range: zeros
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(g.w + (long long)min(nw, g.N - 1) * K, (uint32_t)nrows * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.x + t0 * g.ldx, (uint32_t)((ntok - 1) * g.ldx + K));
  const __amdgpu_buffer_rsrc_t sr = make_rsrc(g.sx + t0 * g.ldsx, (uint32_t)((ntok - 1) * g.ldsx + kb));
  const uint32_t wo = (uint32_t)r16 * (uint32_t)K + 16 * kg;
  const int xrow = tid >> 3, xp = tid & 7;
  const uint32_t xo = (uint32_t)(xrow * g.ldx) + 16 * xp, xstep = (uint32_t)(32 * g.ldx);
  const uint32_t so = (uint32_t)((tid & (TT - 1)) * g.ldsx);
  const long long srow = (long long)(min(nw, g.N - 1) / 128) * kb;  // 16 MT divides 128

  struct Block {
    u32x4_t w[MT][2], x[PIECES];
    uint32_t s;
  };
  auto request = [&](Block &q, int b) {
    b = min(b, kb - 1);  // past the last block that one again, unused
    const uint32_t k0 = 128u * b, none = 0x70000000u;
    // a block that ends inside: pieces past K read out of range
    const uint32_t d[2] = {k0 + 16 * kg < (uint32_t)K ? 0u : none, k0 + 16 * kg + 64 < (uint32_t)K ? 64u : none};
    const uint32_t dx = k0 + 16 * xp < (uint32_t)K ? 0u : none;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) q.w[m][h] = buf_load16(wr, wo + 16u * m * (uint32_t)K + d[h], k0);
#pragma unroll
    for (int u = 0; u < PIECES; ++u) q.x[u] = buf_load16(xr, xo + u * xstep + dx, k0);
    q.s = __builtin_amdgcn_raw_buffer_load_b8(sr, so, b, 0);
  };
  auto put = [&](const Block &q, int buf) {
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
      const int t = xrow + 32 * u;
      lx[buf][8 * t + (xp ^ (t >> 1 & 7))] = q.x[u];
    }
    if (tid < TT) ls[buf][tid] = e8m0_to_float(q.s);
  };
  auto weight_scale = [&](int b) {
    if constexpr (E8) {
      const uint32_t e = static_cast<const uint8_t *>(g.sw)[srow + b];
      // 2^(e - 127); byte 0 is the subnormal 2^-127, 255 is NaN
      return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7FC00000u : e << 23);
    } else {
      return static_cast<const float *>(g.sw)[srow + b];
    }
  };

  f32x4_t acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[m][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const Block &q, int buf, float sw) {
    bf16x8_t wb[F8 ? 1 : MT][4];
    if constexpr (!F8) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) wb[m][c] = codes_to_bf16(q.w[m][c >> 1][2 * (c & 1)], q.w[m][c >> 1][2 * (c & 1) + 1]);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int t = 16 * i + r16, sz = t >> 1 & 7;
      u32x4_t x[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) x[h] = lx[buf][8 * t + ((kg + 4 * h) ^ sz)];
      const float sc = ls[buf][t] * sw;
      f32x4_t p[MT];
      if constexpr (F8) {
#pragma unroll
        for (int m = 0; m < MT; ++m) p[m] = mfma_f8(q.w[m], x);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bf16x8_t xb = codes_to_bf16(x[c >> 1][2 * (c & 1)], x[c >> 1][2 * (c & 1) + 1]);
#pragma unroll
          for (int m = 0; m < MT; ++m) p[m] = mfma_16x16x32(wb[m][c], xb, c == 0 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : p[m]);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[m][i][r] = fmaf(p[m][r], sc, acc[m][i][r]);
    }
  };

  Block q[2];
  request(q[0], 0);
  put(q[0], 0);
  __syncthreads();
  for (int b = 0; b < kb; b += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float sw = b + h < kb ? weight_scale(b + h) : 0.f;
      request(q[h ^ 1], b + h + 1);
      __builtin_amdgcn_sched_barrier(0);  // on its way before the products
      if (b + h < kb) multiply(q[h], h, sw);
      put(q[h ^ 1], h ^ 1);
      __syncthreads();
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int t = 16 * i + r16;
    if (t < ntok)
#pragma unroll
      for (int m = 0; m < MT; ++m)
        store_cols<O>(static_cast<O *>(g.out) + (t0 + t) * g.ldo, nw + 16 * m + 4 * kg, g.N, g.vec_out, g.accumulate,
                      acc[m][i]);
  }
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

template <int MT, int NT, bool F8, typename O>
void tile_by_type(const Fp8Args &g, bool e8, hipStream_t st) {
  const int tn = (g.N + 64 * MT - 1) / (64 * MT), tt = (g.T + 16 * NT - 1) / (16 * NT);
  const dim3 gr((unsigned)((tn * tt + 7) / 8 * 8)), blk(256);
  if (e8) hipLaunchKernelGGL((fp8_tile_kernel<MT, NT, F8, true, O>), gr, blk, 0, st, g, tn, tt);
  else hipLaunchKernelGGL((fp8_tile_kernel<MT, NT, F8, false, O>), gr, blk, 0, st, g, tn, tt);
}

}  // namespace

size_t fp8_workspace_bytes(int T, int N, int K) { return 0; }

hipError_t launch_fp8_gemm(const Fp8Args &g, bool e8, bool out_bf16, void *ws, hipStream_t st) {
  if (g.T > 64) {
    if (out_bf16) tile_by_type<4, 8, true, uint16_t>(g, e8, st);
    else tile_by_type<2, 8, false, float>(g, e8, st);
  } else if (g.T <= 16) stream_by_type<1, 1, 8, 4>(g, e8, out_bf16, st);
  else if (g.T <= 32) stream_by_type<2, 1, 8, 2>(g, e8, out_bf16, st);
  else stream_by_type<4, 2, 8, 1>(g, e8, out_bf16, st);
  return hipGetLastError();
}

}  // namespace moe
