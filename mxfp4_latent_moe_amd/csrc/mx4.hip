// MXFP4 on both sides: rows of values to and from the format, and products
//   out[p, n] (+)= sum_b 2^(sx[p, b] - 127) 2^(sw[n, b] - 127) sum_{k in b} x[p, k] w[n, k]
// over blocks b of 32, dense or with the rows sorted by expert and each expert's
// own w; for a pair of matrices SiTU-GLU of the two products, which can be
// written in MXFP4 again.
//
// The 4-bit matrix instructions take both operands' codes and scale bytes as
// they are.  Their sums are fp32's: over chains of 7168 products with scales
// spread over 2^40 they are off by 1 to 2e-7 of the result's rms, where adding
// in order in fp32 is by 3 to 6e-7 (measured), so every output type uses them.
#include <algorithm>

#include "kernels.h"
#include "mx4_plan.h"
#include "quant4.h"

namespace moe {
namespace {

typedef float f32x8_t __attribute__((ext_vector_type(8)));

MOE_DEV float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
MOE_DEV float widen(float v) { return v; }

// the maximum over the four neighbouring lanes of a block
MOE_DEV uint32_t max4(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));  // lanes 1 0 3 2
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));  // 2 3 0 1
}

// Rows of fp32 or bf16 values in MXFP4: a block is four lanes of 8 values, read in
// 16-byte loads, one pass.  vec: rows' chunks of 8 are whole and aligned.  Memory is
// the bound: 16384 x 3584 fp32 50 us, 5.3 TB/s read and written; a row of 7168 2.4 us.
template <typename X>
__global__ __launch_bounds__(256) void quantize4_kernel(const X *__restrict__ x, long long ldx, long long T, int K,
                                                        int vec, int ocp, uint8_t *__restrict__ q, long long ldq,
                                                        uint8_t *__restrict__ qs, long long ldqs) {
  const int kb = (K + MX4_BLOCK - 1) / MX4_BLOCK;
  const long long first = 64LL * blockIdx.x, t0 = first / kb;  // of the work-group
  const int b0 = (int)(first - t0 * kb) + (threadIdx.x >> 2), r = b0 / kb, b = b0 - r * kb;
  const long long t = t0 + r;
  const int c = b * MX4_BLOCK + 8 * (threadIdx.x & 3);
  f32x8_t v{};
  if (t < T) {
    const X *row = x + t * ldx + c;
    if (vec) {
      if (c < K) {
        const u32x4_t *p = reinterpret_cast<const u32x4_t *>(row);
        const u32x4_t a = p[0];
        if constexpr (sizeof(X) == 4) {
          const u32x4_t e = p[1];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i < 4 ? a[i & 3] : e[i & 3]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __uint_as_float((i & 1) ? (a[i >> 1] & 0xFFFF0000u) : (a[i >> 1] << 16));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c + i < K ? widen(row[i]) : 0.f;
    }
  }
  // magnitudes compare as their bit patterns, infinities and NaN above all
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  const uint32_t sb = mx4_scale_byte(max4(m), ocp);
  const float inv = mx4_inverse(sb);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= inv;
  const uint32_t codes = sb == 255u ? 0u : mx4_codes(v);
  if (t >= T) return;
  uint8_t *to = q + t * ldq + c / 2;
  if (vec) {
    if (c < K) *reinterpret_cast<uint32_t *>(to) = codes;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + 2 * i < K) to[i] = (uint8_t)(codes >> (8 * i));
  }
  if ((threadIdx.x & 3) == 0) qs[t * ldqs + b] = (uint8_t)sb;
}

// and back, eight values a thread: 16384 x 3584 to bf16 24 us, 6.2 TB/s
template <typename O>
__global__ __launch_bounds__(256) void dequantize4_kernel(const uint8_t *__restrict__ q, long long ldq,
                                                          const uint8_t *__restrict__ qs, long long ldqs, long long T,
                                                          int K, int vec, O *__restrict__ out, long long ldo) {
  const int per = (K + 7) / 8;
  const long long first = 256LL * blockIdx.x, t0 = first / per;
  const int i0 = (int)(first - t0 * per) + threadIdx.x, r = i0 / per, c = 8 * (i0 - r * per);
  const long long t = t0 + r;
  if (t >= T) return;
  const uint8_t *from = q + t * ldq + c / 2;
  uint32_t codes = 0;
  if (vec) {
    codes = *reinterpret_cast<const uint32_t *>(from);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + 2 * i < K) codes |= (uint32_t)from[i] << (8 * i);
  }
  const float s = mx4_scale(qs[t * ldqs + c / MX4_BLOCK]);
  f32x8_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto p = i == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0)
                   : i == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1)
                   : i == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2)
                            : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
    v[2 * i] = p[0] * s;
    v[2 * i + 1] = p[1] * s;
  }
  O *to = out + t * ldo + c;
  if constexpr (sizeof(O) == 2) {
    bf16x8_t b;
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = to_bf16(v[i]);
    if (vec) {
      *reinterpret_cast<bf16x8_t *>(to) = b;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < K) reinterpret_cast<__bf16 *>(to)[i] = b[i];
    }
  } else {
    if (vec) {
      reinterpret_cast<f32x4_t *>(to)[0] = f32x4_t{v[0], v[1], v[2], v[3]};
      reinterpret_cast<f32x4_t *>(to)[1] = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < K) to[i] = v[i];
    }
  }
}

// ---- products

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// c + 16 rows times 16 columns over 128 codes, scaled by byte J of each operand's
// scales: a lane holds one of four blocks of row (column) lane % 16
template <int J>
MOE_DEV f32x4_t mfma_4_16(u32x4_t w, u32x4_t x, f32x4_t c, uint32_t sw, uint32_t sx) {
  const i32x4_t w4 = __builtin_bit_cast(i32x4_t, w), x4 = __builtin_bit_cast(i32x4_t, x);
  const i32x8_t a = __builtin_shufflevector(w4, w4, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8_t b = __builtin_shufflevector(x4, x4, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, J, (int)sw, J, (int)sx);
}

// tanh x as a fraction: x P(x^2) over Q(x^2), both of degree 4 with positive
// coefficients, fitted for the least relative error over |x| <= 9 (4.4e-8; in fp32
// 3.1e-7), past which tanh is within 3.1e-8 of its limit.  NaN stays NaN.
MOE_DEV void tanh_ratio(float x, float &num, float &den) {
  const float c = __builtin_elementwise_minimum(__builtin_elementwise_maximum(x, -9.0f), 9.0f), t = c * c;
  float p = 2.6083236265e-11f, q = 1.5188552638e-9f;
  p = fmaf(p, t, 4.0252043476e-8f);
  q = fmaf(q, t, 6.4172485281e-7f);
  p = fmaf(p, t, 6.8273161560e-6f);
  q = fmaf(q, t, 5.0540962548e-5f);
  p = fmaf(p, t, 2.6134811924e-4f);
  q = fmaf(q, t, 9.1238942696e-4f);
  num = c * fmaf(p, t, 0.001953125f);
  den = fmaf(q, t, 0.001953125f);
}

// SiTU-GLU of a tile's sums: 32 instructions a value where situ_glu has 43.  Denominators lie
// between 2^-9 and 1, so that their product overflows where 1 + exp(-g) does (there the result is 0).
// Each beta goes to its own fraction, as the product of the two may leave fp32's range, and the
// reciprocal to the first, which it can only take to 0 and never from infinity to NaN.
MOE_DEV float situ4(float g, float u, float beta, float beta_lin) {
  float ng, dg, nu, du;
  tanh_ratio(g * __builtin_amdgcn_rcpf(beta), ng, dg);
  tanh_ratio(u * __builtin_amdgcn_rcpf(beta_lin), nu, du);
  const float ds = 1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f);
  return (beta * ng * __builtin_amdgcn_rcpf(dg * du * ds)) * (beta_lin * nu);
}

// an expert's rows [row, row + n) of a grouped product, or rows of the dense one
struct Chunk {
  int expert, row, n;
};

// The experts' sorted rows as chunks, an expert's one after the other: experts of
// up to `few` rows on the list few_list, one chunk each, the others on many_list in
// chunks of at most `most` rows, blocks of 64 shared evenly, with a chunk's number
// within its expert << 16 | how many those are.  Bad offsets give wrong
// chunks but none outside the P rows and the lists' sizes.
__global__ __launch_bounds__(1024) void mx4_plan_kernel(const int32_t *offsets, int E, int P, int few, int most,
                                                        int few_cap, int4 *few_list, int32_t *few_count, int many_cap,
                                                        int4 *many_list, int32_t *many_count) {
  __shared__ int tot[2][16];
  const int e = threadIdx.x, lane = e & 63, wave = e >> 6;
  int lo = 0, ne = 0;
  if (e < E) {
    lo = min(max(offsets[e], 0), P);
    ne = min(max(offsets[e + 1], lo), P) - lo;
  }
  int n[2] = {ne > 0 && ne <= few ? 1 : 0, ne > few ? (ne + most - 1) / most : 0}, at[2], sum[2] = {0, 0};
#pragma unroll
  for (int l = 0; l < 2; ++l) {
    int x = n[l];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(x, d, 64);
      if (lane >= d) x += y;
    }
    if (lane == 63) tot[l][wave] = x;
    at[l] = x - n[l];
  }
  __syncthreads();
  for (int w = 0; w < 16; ++w)
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      if (w < wave) at[l] += tot[l][w];
      sum[l] += tot[l][w];
    }
  if (n[0] && at[0] < few_cap) few_list[at[0]] = int4{e, lo, ne, 0};
  const int listed = min(n[1], many_cap - at[1]);
  const long long blocks = (ne + 63) / 64;  // of 64 rows
  for (int i = 0; i < listed; ++i) {
    const int from = 64 * (int)(blocks * i / n[1]), to = min(64 * (int)(blocks * (i + 1) / n[1]), ne);
    many_list[at[1] + i] = int4{e, lo + from, to - from, i << 16 | listed};
  }
  if (e == 0) {
    *few_count = min(sum[0], few_cap);
    *many_count = min(sum[1], many_cap);
  }
}

// four columns n .. of row p in the output's type
template <int OUT>
MOE_DEV void store4(const Mx4Args &g, long long p, int n, f32x4_t v) {
  if constexpr (OUT == MX4_OUT_F32) {
    float *to = static_cast<float *>(g.out) + p * g.ldo + n;
    if (g.vec_out && n + 3 < g.N) {
      f32x4_t *q = reinterpret_cast<f32x4_t *>(to);
      *q = g.accumulate ? *q + v : v;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < g.N) to[r] = g.accumulate ? to[r] + v[r] : v[r];
    }
  } else {
    __bf16 *to = static_cast<__bf16 *>(g.out) + p * g.ldo + n;
    bf16x4_t b;
#pragma unroll
    for (int r = 0; r < 4; ++r) b[r] = to_bf16(v[r]);
    if (g.vec_out && n + 3 < g.N) {
      *reinterpret_cast<bf16x4_t *>(to) = b;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < g.N) to[r] = b[r];
    }
  }
}

// the row of x that sorted row p of the product reads
MOE_DEV int x_row(const Mx4Args &g, int p) { return g.map == nullptr ? p : g.map[p] / g.div; }

// 16 bytes of LDS at a + O, issued without waiting
template <int O>
MOE_DEV void tread(uint32_t a, u32x4_t &v) {
  static_assert(O >= 0 && O < 65536, "offset field");
  asm volatile("ds_read_b128 %0, %1 offset:%2" : "=&v"(v) : "v"(a), "n"(O) : "memory");
}
template <int O>
MOE_DEV void tread2(uint32_t a, uint32_t &v) {
  static_assert(O >= 0 && O < 65536, "offset field");
  asm volatile("ds_read_u16 %0, %1 offset:%2" : "=&v"(v) : "v"(a), "n"(O) : "memory");
}
template <int O>
MOE_DEV void tread4(uint32_t a, uint32_t &v) {
  static_assert(O >= 0 && O < 65536, "offset field");
  asm volatile("ds_read_b32 %0, %1 offset:%2" : "=&v"(v) : "v"(a), "n"(O) : "memory");
}
template <int N>
MOE_DEV void twait() {
  asm volatile("s_waitcnt lgkmcnt(%0)" ::"n"(N < 15 ? N : 15) : "memory");
}
// ties a register to the wait before: its users stay behind it
template <typename V>
MOE_DEV void ttie(V &v) {
  asm volatile("" : "+v"(v));
}

// The chunk of number `want` where no list of them was made: every work-group
// counts the experts' chunks itself.  NW waves; false: there are fewer.
template <int NW>
MOE_DEV bool find_chunk(const Mx4Args &g, int rows, int want, Chunk &c, int *lds) {
  constexpr int PER = MX4_MAX_E / (64 * NW);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int lo[PER], ne[PER], n = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = PER * tid + i;
    lo[i] = ne[i] = 0;
    if (e < g.n_experts) {
      lo[i] = min(max(g.offsets[e], 0), g.P);
      ne[i] = min(max(g.offsets[e + 1], lo[i]), g.P) - lo[i];
      n += (ne[i] + rows - 1) / rows;
    }
  }
  int x = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  if (lane == 63) lds[wave] = x;
  if (tid == 0) lds[NW + 2] = 0;
  __syncthreads();
  int at = x - n;
#pragma unroll
  for (int w = 0; w < NW; ++w)
    if (w < wave) at += lds[w];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int k = want - at, nch = (ne[i] + rows - 1) / rows;
    if (k >= 0 && k < nch) {
      lds[NW] = PER * tid + i;
      lds[NW + 1] = lo[i] + k * rows;
      lds[NW + 2] = min(rows, ne[i] - k * rows);
    }
    at += nch;
  }
  __syncthreads();
  c = Chunk{lds[NW], lds[NW + 1], lds[NW + 2]};
  return c.n > 0;
}

// ---- few rows: the weights are the whole cost
//
// A wave owns 32 weight rows (32 columns of the result, of a pair 16 of each
// matrix) and 16 NT rows of x, and has a ring of its own in LDS, ST stages of 256
// inputs, that direct loads of rows' whole 128 bytes fill: no wave waits for
// another while it streams, and the waves of a CU keep some 100 KB on their way.
// x comes straight to registers, a stage ahead (the rows stay in the L2).  KS waves
// of a work-group share their columns and take the stages of K in turn (at any time
// they read a contiguous KS * 128 bytes of a row); their sums meet in LDS and are
// added in order.
//
// In LDS piece p (16 bytes, a block) of row r lies at position p ^ (r / 2 % 8), as
// the 16 rows that a quarter wave reads at once, two to a 256-byte line, then fall
// on different banks.  Product j of a stage takes piece 2 kg + j from the lanes of
// group kg (the groups' K need not be neighbours in memory), so that a lane's two
// scale bytes of a stage are neighbours, of which the instruction selects one.
//
// Loads of two bytes a lane cost as much as those of sixteen.  With SG (scale rows
// are whole dwords apart and aligned) the scales of two stages come into LDS by one
// direct load for 32 rows, 16 bytes a row; without it byte by byte to registers
// (16 tokens, 7168 x 33792: 39 us in place of 31 with x's scale rows strided; K of
// 33824, whose scale rows are no whole dwords, 47).
//
// Bound by the weights.  One token: 3584 x 7168 5.9 us, 7168 x 33792 25 us, 5.1 TB/s;
// 16 tokens 31 us, 4.2 TB/s, where half as many bytes of x as of weights come to a
// CU.  Gate and up of one token's 16 experts 41 us, 4.5 TB/s; of 16 tokens through 896
// experts (some 230 of them in use) 425 to 440 us, 6.1 TB/s, down 211 to 218 (505 and
// 248 in a process that had allocated and freed other large weights before).
constexpr int STREAM_STAGE = 32 * 128;
constexpr int stream_st(int nt) { return nt == 1 ? 4 : 3; }
constexpr int stream_group(int nt) { return 1024 + 512 * nt; }  // the weights' scales, then x's
constexpr int STREAM_WAVE = 19 * 1024;  // LDS of a wave: the ring and two groups of scales
constexpr bool stream_fits(int nt) { return stream_st(nt) * STREAM_STAGE + 2 * stream_group(nt) <= STREAM_WAVE; }
static_assert(stream_fits(1) && stream_fits(2) && stream_fits(4), "LDS of a wave");

// 16 bytes a lane straight into LDS (the host's pass over this code knows of 4 only)
MOE_DEV void lds_load(__amdgpu_buffer_rsrc_t r, uint8_t *to, uint32_t voff, uint32_t soff) {
#ifdef __HIP_DEVICE_COMPILE__
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)to, 16, voff, soff, 0, 0);
#endif
}

// two neighbouring scale bytes
MOE_DEV uint32_t load_scales(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t at) {
  const uint32_t lo = __builtin_amdgcn_raw_buffer_load_b8(r, off, at, 0);
  return lo | (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(r, off + 1, at, 0) << 8;
}

// what a stage takes from registers: pieces of x, and without SG the scales
template <int NT>
struct StreamRegs {
  u32x4_t x[NT][2];
  uint32_t sx[NT], sw[2];
};

template <int NT, bool PAIR, bool SG, int KS>
MOE_DEV void mx4_stream(const Mx4Args &g, const Chunk &c, int block, uint8_t *lds) {
  constexpr int ST = stream_st(NT), SB = STREAM_STAGE, GB = stream_group(NT), DL = 4;
  constexpr int RL = SG ? 2 * NT : 4 * NT + 4;  // register loads of a stage
  constexpr int GL = !SG ? 0 : (PAIR ? 2 : 1) + (NT == 4 ? 2 : 1);  // of a group of scales
  constexpr int CW = PAIR ? 16 : 32;
  const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, kg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kbytes = g.K / 2, kb = g.K / 32, stages = (g.K + 255) / 256;
  const int n0 = CW * block, part = KS == 1 ? 0 : wave % KS;
  // a wave whose columns are past the last one only keeps the barriers whole
  const int nrows = __builtin_amdgcn_readfirstlane(max(min(CW, g.N - n0), 0));
  // stage s of this wave is stage part + KS s of K
  const int count = nrows > 0 ? (stages - part + KS - 1) / KS : 0;
  uint8_t *const ring = lds + wave * STREAM_WAVE, *const groups = ring + ST * SB;
  constexpr uint32_t OUT = 0x80000000u;  // past the end of every buffer

  __amdgpu_buffer_rsrc_t wr[PAIR ? 2 : 1], sr[PAIR ? 2 : 1];
#pragma unroll
  for (int m = 0; m < (PAIR ? 2 : 1); ++m) {
    const long long row = (long long)c.expert * g.N + n0;
    wr[m] = make_rsrc(g.w[m] + row * kbytes, (uint32_t)nrows * (uint32_t)kbytes);
    sr[m] = make_rsrc(g.sw[m] + row * kb, (uint32_t)nrows * (uint32_t)kb);
  }
  // gathered rows are found from the first row of x, others from the chunk's own
  const long long base = g.map != nullptr ? 0 : c.row;
  const int xrows = g.map != nullptr ? g.x_rows : c.n;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.x + base * g.ldx, (uint32_t)((xrows - 1) * g.ldx + kbytes));
  const __amdgpu_buffer_rsrc_t xsr = make_rsrc(g.sx + base * g.ldsx, (uint32_t)((xrows - 1) * g.ldsx + kb));
  const int l8 = lane >> 3;
  uint32_t piece[2], vw[DL];
#pragma unroll
  for (int q = 0; q < 2; ++q) piece[q] = 16 * ((lane & 7) ^ (4 * q + (lane >> 4)));
#pragma unroll
  for (int u = 0; u < DL; ++u)  // 8 rows a load; the second matrix's are loads 2 and 3
    vw[u] = (uint32_t)(8 * (PAIR ? u & 1 : u) + l8) * (uint32_t)kbytes + piece[u & 1];
  auto request = [&](int s) {  // stage s of this wave's part
    uint8_t *const at = ring + (s % ST) * SB;
    const uint32_t k0 = 128u * (part + KS * s);
    // of a stage that ends inside, pieces past K read out of range: zeros
    const uint32_t past[2] = {k0 + piece[0] < (uint32_t)kbytes ? 0u : OUT, k0 + piece[1] < (uint32_t)kbytes ? 0u : OUT};
#pragma unroll
    for (int u = 0; u < DL; ++u)
      lds_load(wr[PAIR ? u >> 1 : 0], at + 1024 * u, vw[u] | past[u & 1], k0);
  };
  // the weights go out before anything about x's rows is known
  for (int s = 0; s < min(ST - 1, count); ++s) request(s);

  uint32_t so[2], xo[NT], xso[NT];
#pragma unroll
  for (int m = 0; m < 2; ++m) so[m] = (uint32_t)min((PAIR ? 0 : 16 * m) + r16, nrows - 1) * (uint32_t)kb + 2 * kg;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    // rows past the chunk read out of range
    const bool in = 16 * i + r16 < c.n;
    const uint32_t r = in ? (uint32_t)(x_row(g, c.row + 16 * i + r16) - (int)base) : 0u;
    xo[i] = in ? r * (uint32_t)g.ldx + 32 * kg : OUT;
    xso[i] = in ? r * (uint32_t)g.ldsx + 2 * kg : OUT;
  }
  using Regs = StreamRegs<NT>;
  auto load = [&](Regs &v, int s) {
    const uint32_t k0 = 128u * (part + KS * s), b0 = 8u * (part + KS * s);
    const uint32_t past = b0 + 2 * kg < (uint32_t)kb ? 0u : OUT, past2 = b0 + 2 * kg + 1 < (uint32_t)kb ? 0u : OUT;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      v.x[i][0] = buf_load16(xr, xo[i] | past, k0);
      v.x[i][1] = buf_load16(xr, (xo[i] + 16) | past2, k0);
      if constexpr (!SG) v.sx[i] = load_scales(xsr, xso[i] | past, b0);
    }
    if constexpr (!SG) {
#pragma unroll
      for (int m = 0; m < 2; ++m) v.sw[m] = load_scales(sr[PAIR ? m : 0], so[m] | past, b0);
    }
  };
  // scales of stages 2 q and 2 q + 1, [stage][row][16], of a pair the one matrix's and
  // then the other's; a row's bytes past its end are others'
  uint32_t vg = 0, vgx[2] = {0, 0};
  if constexpr (SG) {
    vg = (uint32_t)min(PAIR ? r16 : lane & 31, max(nrows - 1, 0)) * (uint32_t)kb + 8 * KS * (PAIR ? lane >> 4 : lane >> 5);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int r = NT == 4 ? lane : lane % (16 * NT), later = NT == 4 ? q : lane / (16 * NT);
      vgx[q] = r < c.n && later < 2 ? (uint32_t)(x_row(g, c.row + r) - (int)base) * (uint32_t)g.ldsx + 8 * KS * later : OUT;
    }
  }
  auto request_scales = [&](int q) {
    if constexpr (SG) {
      uint8_t *const at = groups + (q & 1) * GB;
      const uint32_t b0 = 8u * (part + KS * 2 * q);
      if constexpr (PAIR) {  // half a wave's lanes for each matrix
        if (lane < 32) lds_load(sr[0], at, vg, b0);
        if (lane < 32) lds_load(sr[PAIR ? 1 : 0], at + 512, vg, b0);
      } else {
        lds_load(sr[0], at, vg, b0);
      }
      if (NT > 1 || lane < 32) lds_load(xsr, at + 1024, vgx[0], b0);
      if constexpr (NT == 4) lds_load(xsr, at + 2048, vgx[1], b0);
    }
  };

  f32x4_t acc[2][NT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[m][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  uint32_t frag[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) frag[j] = lds_addr(ring) + 128 * r16 + 16 * ((2 * kg + j) ^ (r16 >> 1));
  const uint32_t sfrag = lds_addr(groups) + 16 * r16 + 2 * kg;
  // In the order of their requests: registers of stage s, at even s the scales of
  // s + 2 and s + 3, stage s + ST - 1.  MORE: such a stage is left; else `more` says so.
  auto step = [&](auto oddc, auto morec, bool more, int s, Regs &now, Regs &next) {
    constexpr bool odd = decltype(oddc)::value, MORE = decltype(morec)::value;
    load(next, min(s + 1, count - 1));
    __builtin_amdgcn_sched_barrier(0);  // the waits count loads in this order
    if (!odd && (MORE || s + 2 < count)) request_scales(s / 2 + 1);
    // this stage, its registers and scales have landed; requested since are later ones'
    if (MORE || more) {
      request(s + ST - 1);
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(DL * (ST - 2) + RL + (odd ? 0 : GL)));
    } else {
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(RL));  // near the end fewer are on their way
    }
    __builtin_amdgcn_sched_barrier(0);
    const uint32_t at = (s % ST) * SB;
    u32x4_t w[2][2];
    uint32_t sw[2], sx[NT];
    if constexpr (SG) {
      const uint32_t sa = sfrag + (s / 2 & 1) * GB, swa = sa + (odd ? PAIR ? 256 : 512 : 0), sxa = sa + 1024 + (odd ? 256 * NT : 0);
      tread2<0>(swa, sw[0]);
      tread2<PAIR ? 512 : 256>(swa, sw[1]);
      static_for<NT>([&](auto ic) { tread2<256 * decltype(ic)::value>(sxa, sx[decltype(ic)::value]); });
    } else {
#pragma unroll
      for (int m = 0; m < 2; ++m) sw[m] = now.sw[m];
#pragma unroll
      for (int i = 0; i < NT; ++i) sx[i] = now.sx[i];
    }
    tread<0>(frag[0] + at, w[0][0]);
    tread<2048>(frag[0] + at, w[1][0]);
    tread<0>(frag[1] + at, w[0][1]);
    tread<2048>(frag[1] + at, w[1][1]);
    // scale bytes past K are of other rows: one in their place
    const int in = kb - 8 * (part + KS * s) - 2 * kg;
    const uint32_t mask = in >= 2 ? 0xFFFFu : in <= 0 ? 0u : 0xFFu;
    twait<2>();
    ttie(w[0][0]);
    ttie(w[1][0]);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if constexpr (SG) ttie(sw[m]);
      sw[m] = (sw[m] & mask) | (0x7F7Fu & ~mask);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if constexpr (SG) ttie(sx[i]);
      sx[i] = (sx[i] & mask) | (0x7F7Fu & ~mask);
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[m][i] = mfma_4_16<0>(w[m][0], now.x[i][0], acc[m][i], sw[m], sx[i]);
    twait<0>();
    ttie(w[0][1]);
    ttie(w[1][1]);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[m][i] = mfma_4_16<1>(w[m][1], now.x[i][1], acc[m][i], sw[m], sx[i]);
  };
  if (count > 0) {
    const std::false_type even;
    const std::true_type odd;
    Regs a, b;
    request_scales(0);
    load(a, 0);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // the first stages went out in another order than the rest
    __builtin_amdgcn_sched_barrier(0);
    const int most = count - (ST - 1);  // steps that request a stage
    int s = 0;
    for (; s + 1 < most; s += 2) {
      step(even, std::true_type{}, true, s, a, b);
      step(odd, std::true_type{}, true, s + 1, b, a);
    }
    for (;;) {  // s is even
      step(even, std::false_type{}, s < most, s, a, b);
      if (++s >= count) break;
      step(odd, std::false_type{}, s < most, s, b, a);
      if (++s >= count) break;
    }
  }

  if constexpr (KS > 1) {
    f32x4_t *const mine = reinterpret_cast<f32x4_t *>(ring);  // its own loads have landed
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) mine[64 * (NT * m + i) + lane] = acc[m][i];
    __syncthreads();
    // tile by tile in turn over the waves that share them
    const int w0 = wave - part;
    for (int t = part; t < 2 * NT; t += KS) {
      f32x4_t v = {0.f, 0.f, 0.f, 0.f};
      for (int q = 0; q < KS; ++q)
        v += reinterpret_cast<const f32x4_t *>(lds + (w0 + q) * STREAM_WAVE)[64 * t + lane];
      const int m = t / NT, r = 16 * (t % NT) + r16, n = n0 + 16 * m + 4 * kg;
      if (r < c.n) {
        if (g.out_kind == MX4_OUT_BF16) store4<MX4_OUT_BF16>(g, c.row + r, n, v);
        else store4<MX4_OUT_F32>(g, c.row + r, n, v);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int r = 16 * i + r16;
    const long long p = c.row + r;
    if constexpr (PAIR) {
      f32x4_t v;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = situ4(acc[0][i][k], acc[1][i][k], g.beta, g.beta_lin);
      const int n = n0 + 4 * kg;
      if (g.out_kind == MX4_OUT_MX4) {
        // a block of the result is this wave's columns and its neighbour's
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max(top, __float_as_uint(v[k]) & 0x7FFFFFFFu);
        top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
        uint32_t *const tops = reinterpret_cast<uint32_t *>(lds);
        __syncthreads();  // rings (and the tops of the tile before) are done with
        if (kg == 0) tops[16 * wave + r16] = top;
        __syncthreads();
        top = max(top, tops[16 * (wave ^ 1) + r16]);
        const uint32_t sb = mx4_scale_byte(top, false);
        v *= mx4_inverse(sb);
        uint32_t q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], 1.0f, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], 1.0f, 1);
        if (r < c.n && n < g.N) {
          *reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(g.out) + p * g.ldo + n / 2) =
              sb == 255u ? (uint16_t)0 : (uint16_t)q;
          if (lane < 16 && n0 % 32 == 0) g.os[p * g.ldos + n0 / 32] = (uint8_t)sb;
        }
      } else if (r < c.n) {
        if (g.out_kind == MX4_OUT_BF16) store4<MX4_OUT_BF16>(g, p, n, v);
        else store4<MX4_OUT_F32>(g, p, n, v);
      }
    } else if (r < c.n) {
      const float pw = g.pair_weight != nullptr ? g.pair_weight[g.pair[p]] : 1.f;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const f32x4_t v = acc[m][i] * pw;
        if (g.out_kind == MX4_OUT_BF16) store4<MX4_OUT_BF16>(g, p, n0 + 16 * m + 4 * kg, v);
        else store4<MX4_OUT_F32>(g, p, n0 + 16 * m + 4 * kg, v);
      }
    }
  }
}

template <int MAXT, bool PAIR, bool SG, int KS>
MOE_DEV void mx4_stream_rows(const Mx4Args &g, const Chunk &c, int block, uint8_t *lds) {
  if (MAXT == 1 || c.n <= 16) mx4_stream<1, PAIR, SG, KS>(g, c, block, lds);
  else if (MAXT == 2 || c.n <= 32) mx4_stream<(MAXT < 2 ? MAXT : 2), PAIR, SG, KS>(g, c, block, lds);
  else mx4_stream<MAXT, PAIR, SG, KS>(g, c, block, lds);
}

// work-groups of 4 waves with a block of columns each, two on a CU (grouped), or of
// 8 that share one (dense); chunks of at most 16 MAXT rows
template <int MAXT, bool PAIR, bool SG, int KS>
__global__ __launch_bounds__(KS == 1 ? 256 : 512, 2) void mx4_stream_kernel(Mx4Args g) {
  constexpr int NW = KS == 1 ? 4 : 8, BLOCKS = NW / KS;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NW * STREAM_WAVE];
  const int nb = ((g.N + (PAIR ? 15 : 31)) / (PAIR ? 16 : 32) + BLOCKS - 1) / BLOCKS;  // work-groups a chunk
  Chunk c;
  int nblk;
  if (KS > 1) {  // dense
    const int logical = xcd_logical((g.P + 16 * MAXT - 1) / (16 * MAXT) * nb);
    if (logical < 0) return;
    const int ci = logical / nb;
    nblk = logical - ci * nb;
    c = Chunk{0, 16 * MAXT * ci, min(16 * MAXT, g.P - 16 * MAXT * ci)};
  } else if (g.chunks != nullptr) {
    const int logical = xcd_logical(*g.chunk_count * nb);
    if (logical < 0) return;
    const int ci = logical / nb;
    nblk = logical - ci * nb;
    const int4 v = g.chunks[ci];
    c = Chunk{v.x, v.y, v.z};
  } else {
    const int ci = blockIdx.x / nb;
    nblk = blockIdx.x - ci * nb;
    if (!find_chunk<NW>(g, 16 * MAXT, ci, c, reinterpret_cast<int *>(lds))) return;
    __syncthreads();  // lds is the rings' from here on
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int block = nblk * BLOCKS + wave / KS;
  // the same in every lane, which buffer descriptors need
  c = Chunk{__builtin_amdgcn_readfirstlane(c.expert), __builtin_amdgcn_readfirstlane(c.row),
            __builtin_amdgcn_readfirstlane(c.n)};
  mx4_stream_rows<MAXT, PAIR, SG, KS>(g, c, block, lds);
}

// ---- many rows
// A work-group of eight waves owns 256 weight rows (of a pair, 128 of each matrix)
// and 64 NT rows of x; a wave of it 64 weight rows and half of the rows, 2 x NT
// tiles of 32 x 32.  Both operands pass through ST LDS stages of
// 256 inputs, filled by direct loads of rows' whole 128 bytes between the products.
//
// A row's 128 bytes are eight pieces of 16, a block of 32 codes each; piece p of
// row r lies at position p ^ (r / 2 % 8), so the 16 rows that a quarter wave reads
// at once, two to a 256-byte line of LDS, fall on different banks.  Product j of a
// stage takes piece 4 h + j from the lanes of half h: the two halves of the
// instruction's K need not be neighbours in memory, and the four scale bytes that
// a lane needs in a stage are then one dword, from which the instruction selects
// byte j.  Scales come into LDS 16 bytes a row, two stages at a time.
//
// SG: scale rows are whole dwords apart and aligned, so that those 16 bytes can be
// loaded directly; else they come byte by byte through registers: 16 loads of a byte a
// lane for two stages, and one register spilled for a pair, two without.  So K whose
// blocks are no multiple of four is slow: 4096 x 6144 x 7200 180 us where 7168 takes
// 109, K = 2880 70 where 2816 takes 49, gate and up of 16384 tokens, two of 112 experts
// each, 934 at K = 3616 for 614 at 3584.
//
// A stage of 256 rows takes 1.86 us on all CUs: its loads alone 1.65 (1.33 with more
// room to wait for them), its products 1.33, its LDS reads 0.70, reads and products
// 1.57.  4096 x 6144 x 7168 101 to 116 us with the card's clock, 3.1 to 3.6 PFLOP/s.  Slower: waves of 64 x 256 (119 for
// 110), stages of 128 inputs four deep (2.09 for 1.86).  Of a pair, the 64 values a
// lane of SiTU-GLU come on top, 9 of an item's 45 us at K = 3584: gate and up of 4096
// tokens, four of 16 experts each, 291 us, without it 234; work-groups that stay and
// request their next item before they write one need some 70 registers more than
// there are (16384 tokens, two of 112 experts each: 815 us for 669).  With some 70 rows
// an expert the weights are the bound, 3.9 TB/s with two stages of them on their way
// (4096 tokens, two of 112 experts each: 337 us); tiles of half the size two on a CU
// took 348, a dword of each row of the stage after asked for into the L2 358.
typedef float f32x16_t __attribute__((ext_vector_type(16)));

// c + 32 rows times 32 columns over 64 codes, scaled by byte J of each operand's scales
template <int J>
MOE_DEV f32x16_t mfma_4_32(u32x4_t w, u32x4_t x, f32x16_t c, uint32_t sw, uint32_t sx) {
  const i32x4_t w4 = __builtin_bit_cast(i32x4_t, w), x4 = __builtin_bit_cast(i32x4_t, x);
  const i32x8_t a = __builtin_shufflevector(w4, w4, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8_t b = __builtin_shufflevector(x4, x4, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 4, 4, J, (int)sw, J, (int)sx);
}

constexpr int TILE_ROWS = MX4_TILE_ROWS;  // rows of x
constexpr int TILE_COLS = 256;    // weight rows
constexpr int GROUP_BYTES = (TILE_COLS + TILE_ROWS) * 16;  // scales of two stages
constexpr int stages_of(int nt) { return nt <= 2 ? 3 : 2; }
constexpr int stage_bytes(int nt) { return (TILE_COLS + 64 * nt) * 128; }
constexpr int tile_lds(int nt) { return stages_of(nt) * stage_bytes(nt) + 2 * GROUP_BYTES; }
constexpr int max_lds(int nt) { return nt == 0 ? 0 : tile_lds(nt) > max_lds(nt - 1) ? tile_lds(nt) : max_lds(nt - 1); }
constexpr int TILE_LDS = max_lds(4);
static_assert(TILE_LDS <= 160 * 1024, "LDS of a CU");

// rows c of x times weight rows of columns n0 .., stages first .. first + count - 1 of K (first even)
template <int NT, bool PAIR, bool SG>
MOE_DEV void mx4_tile(const Mx4Args &g, const Chunk &c, int n0, int first, int count, float *partial, uint8_t *lds) {
  constexpr int ST = stages_of(NT), SB = stage_bytes(NT), GB = GROUP_BYTES;
  constexpr int WL = 4, XL = NT;  // direct loads of a wave per stage, 8 rows each
  const int tid = threadIdx.x, lane = tid & 63, r32 = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wn = wave & 3, wt = wave >> 2;
  const int kbytes = g.K / 2, kb = g.K / 32;
  const int ncols = min(PAIR ? TILE_COLS / 2 : TILE_COLS, g.N - n0);
  uint8_t *const groups = lds + ST * SB;

  // columns and rows past the end are out of range: zeros
  __amdgpu_buffer_rsrc_t wr[PAIR ? 2 : 1], sr[PAIR ? 2 : 1];
#pragma unroll
  for (int m = 0; m < (PAIR ? 2 : 1); ++m) {
    const long long row = (long long)c.expert * g.N + n0;
    wr[m] = make_rsrc(g.w[m] + row * kbytes, (uint32_t)ncols * (uint32_t)kbytes);
    sr[m] = make_rsrc(g.sw[m] + row * kb, (uint32_t)ncols * (uint32_t)kb);
  }
  const long long base = g.map != nullptr ? 0 : c.row;
  const int xrows = g.map != nullptr ? g.x_rows : c.n;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.x + base * g.ldx, (uint32_t)((xrows - 1) * g.ldx + kbytes));
  const __amdgpu_buffer_rsrc_t xsr = make_rsrc(g.sx + base * g.ldsx, (uint32_t)((xrows - 1) * g.ldsx + kb));
  constexpr uint32_t OUT = 0x80000000u;  // past the end of every buffer
  auto row_of = [&](int r) { return (uint32_t)(x_row(g, c.row + r) - (int)base); };

  // direct load u of this wave fills 8 rows of a stage: lane i's 16 bytes land at
  // position i % 8 of row i / 8
  const int l8 = lane >> 3;
  uint32_t piece[2], vw[WL], vx[XL];
#pragma unroll
  for (int q = 0; q < 2; ++q) piece[q] = 16 * ((lane & 7) ^ (4 * q + (lane >> 4)));
#pragma unroll
  for (int u = 0; u < WL; ++u) {
    const int n = 32 * (PAIR ? wave >> 1 : wave) + 8 * u + l8;  // of a pair, even waves the first matrix's rows
    vw[u] = (uint32_t)n * (uint32_t)kbytes + piece[u & 1];
  }
  // what to add where stage b ends inside; stages after the last are read as the last, unused
  auto past = [&](int b, uint32_t p) { return 128u * (first + min(b, count - 1)) + p < (uint32_t)kbytes ? 0u : OUT; };
  // load u of stage b, to the place at `place` of the ring
  auto request = [&](uint32_t place, int b, const uint32_t (&out)[2], auto uc) {
    constexpr int u = decltype(uc)::value;
    uint8_t *const at = lds + place;
    const uint32_t k0 = 128u * (first + min(b, count - 1));
    if constexpr (u < WL)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wr[PAIR ? wave & 1 : 0], (lds_void *)(at + (32 * wave + 8 * u) * 128), 16,
                                               vw[u] | out[u & 1], k0, 0, 0);
    else if constexpr (u < WL + XL)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          xr, (lds_void *)(at + (TILE_COLS + 8 * (8 * (u - WL) + wave)) * 128), 16, vx[u - WL] | out[wave & 1], k0, 0, 0);
  };
  // the first stages' weights go out before anything about x's rows is known
  static_for<ST - 1>([&](auto sc) {
    constexpr int s = decltype(sc)::value;
    const uint32_t out[2] = {past(s, piece[0]), past(s, piece[1])};
    static_for<WL>([&](auto uc) { request(s * SB, s, out, uc); });
  });
#pragma unroll
  for (int u = 0; u < XL; ++u) {
    const int r = 8 * (8 * u + wave) + l8;
    vx[u] = r < c.n ? row_of(r) * (uint32_t)g.ldx + piece[wave & 1] : OUT;
  }
  // scales of stages 2 q and 2 q + 1: [row][16], a row a lane; waves 0 to 3 the
  // weights' (of a pair first one matrix's 128 rows, then the other's), the others x's
  const int sr_row = 64 * (PAIR && wt == 0 ? wn & 1 : wn) + lane;
  const uint32_t vs = wt == 0 ? (uint32_t)sr_row * (uint32_t)kb : sr_row < c.n ? row_of(sr_row) * (uint32_t)g.ldsx : OUT;
  const __amdgpu_buffer_rsrc_t srsrc = wt != 0 ? xsr : PAIR && wn >= 2 ? sr[PAIR ? 1 : 0] : sr[0];
  u32x4_t held;  // without SG: on their way through registers
  auto request_scales = [&](int q) {
    const uint32_t at = 16u * (first / 2 + min(q, (count - 1) / 2));
    if constexpr (SG) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(srsrc, (lds_void *)(groups + (q & 1) * GB + 1024 * wave), 16,
                                               vs, at, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t a = __builtin_amdgcn_raw_buffer_load_b8(srsrc, vs | (at + i < (uint32_t)kb ? 0u : OUT), at + i, 0);
        held[i >> 2] = i & 3 ? held[i >> 2] | a << (8 * (i & 3)) : a;
      }
    }
  };
  auto put_scales = [&](int q) {
    if constexpr (!SG) reinterpret_cast<u32x4_t *>(groups + (q & 1) * GB)[tid] = held;
  };

  request_scales(0);
  static_for<ST - 1>([&](auto sc) {
    constexpr int s = decltype(sc)::value;
    const uint32_t out[2] = {past(s, piece[0]), past(s, piece[1])};
    static_for<XL>([&](auto uc) { request(s * SB, s, out, std::integral_constant<int, WL + decltype(uc)::value>{}); });
  });
  put_scales(0);
  // they went out in another order than the rest (of two stages, the first step waits for all)
  if constexpr (ST > 2) __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));

  f32x16_t acc[2][NT];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[m][i][r] = 0.f;
  // Sums stay in accumulation registers: left to itself, the compiler moves some of
  // them to others and back within the loop.
  auto hold = [&] {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) asm volatile("" : "+a"(acc[m][i]));
  };
  uint32_t frag[4];  // this lane's piece of row r32 for product j
#pragma unroll
  for (int j = 0; j < 4; ++j) frag[j] = lds_addr(lds) + 128 * r32 + 16 * ((4 * h + j) ^ (r32 >> 1 & 7));
  const uint32_t sfrag = lds_addr(groups) + 16 * r32 + 4 * h;

  // the order of a stage's LDS reads: the scales, the first product's weights and D
  // rows' pieces; then with each tile the rows' piece D tiles on, and with a
  // product's first tile the next product's weights
  constexpr int F = 4 * NT, D = NT == 1 ? 2 : 3;
  uint32_t place = 0;  // of this stage in the ring
  auto step = [&](auto oddc, int b) {
    constexpr bool odd = decltype(oddc)::value;
    hold();
    // this stage has landed (what was requested since is the next ones), and every
    // wave is done with the one before, whose place is filled below
    if constexpr (!SG) twait<0>();
    __builtin_amdgcn_s_waitcnt(vmcnt_imm((WL + XL) * (ST - 2)));
    __builtin_amdgcn_s_barrier();
    if constexpr (odd) put_scales(b / 2 + 1);
    else request_scales(b / 2 + 1);
    u32x4_t w[2][2], x[D + 1];
    uint32_t sw[2], sx[NT];
    const uint32_t sa = sfrag + (b / 2 & 1) * GB + (odd ? 8 : 0);
    const uint32_t swa = sa + (PAIR ? 512 : 1024) * wn, sxa = sa + 512 * NT * wt;
    uint32_t fx[4], fw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      fw[j] = frag[j] + place + 8192 * wn;
      fx[j] = frag[j] + place + 4096 * NT * wt;
    }
    auto read_w = [&](auto jc) {
      constexpr int j = decltype(jc)::value;
      tread<0>(fw[j], w[j & 1][0]);
      tread<4096>(fw[j], w[j & 1][1]);
    };
    auto read_x = [&](auto fc) {
      constexpr int f = decltype(fc)::value;
      tread<TILE_COLS * 128 + 4096 * (f % NT)>(fx[f / NT], x[f % (D + 1)]);
    };
    tread4<0>(swa, sw[0]);
    tread4<PAIR ? 2048 : 512>(swa, sw[1]);
    static_for<NT>([&](auto ic) { tread4<TILE_COLS * 16 + 512 * decltype(ic)::value>(sxa, sx[decltype(ic)::value]); });
    read_w(std::integral_constant<int, 0>{});
    static_for<D>([&](auto fc) { read_x(fc); });
    const uint32_t out[2] = {past(b + ST - 1, piece[0]), past(b + ST - 1, piece[1])};
    const uint32_t next = place == 0 ? (ST - 1) * SB : place - SB;  // the place that stage b - 1 had
    // scale bytes past K are of other rows: one in their place
    const int in = kb - 8 * (first + b) - 4 * h;
    const uint32_t mask = in >= 4 ? 0xFFFFFFFFu : in <= 0 ? 0u : (1u << (8 * in)) - 1u;
    static_for<F>([&](auto fc) {
      constexpr int f = decltype(fc)::value, j = f / NT, i = f % NT;
      if constexpr (f + D < F) read_x(std::integral_constant<int, f + D>{});
      if constexpr (i == 0 && j < 3) read_w(std::integral_constant<int, j + 1>{});
      // reads behind the last one that this tile needs: rows' piece f (issued with
      // tile f - D), and at a product's first tile the weights issued with the last
      // product's first; weights are two reads
      constexpr int from = f < D ? 0 : f - D + 1;          // tiles since piece f went out, this one among them
      constexpr int xs_behind = (f + D < F ? f + D : F - 1) - f;
      constexpr int ws_behind = [] {
        int n = 0;
        for (int q = from; q <= f; ++q)
          if (q % NT == 0 && q / NT < 3) n += 2;
        return n;
      }();
      // the weights of product j went out with tile (j - 1) NT, behind that tile's piece
      constexpr int w_at = (j - 1) * NT;
      constexpr int w_behind = j == 0 ? D : [] {
        int n = 0;
        for (int q = w_at + 1; q <= f; ++q) {
          if (q + D < F) ++n;
          if (q % NT == 0 && q / NT < 3) n += 2;
        }
        return n;
      }();
      constexpr int behind = xs_behind + ws_behind;
      twait<(i == 0 && w_behind < behind) ? w_behind : behind>();
      ttie(x[f % (D + 1)]);
      if constexpr (i == 0) {
        ttie(w[j & 1][0]);
        ttie(w[j & 1][1]);
      }
      if constexpr (f == 0) {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          ttie(sw[m]);
          sw[m] = (sw[m] & mask) | (0x7F7F7F7Fu & ~mask);
        }
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          ttie(sx[q]);
          sx[q] = (sx[q] & mask) | (0x7F7F7F7Fu & ~mask);
        }
      }
      // the loads into the free stage, spread over the products (of two stages:
      // the first half, the rest is their time to land)
      constexpr int over = ST == 2 ? F / 2 : F, per = (WL + XL + over - 1) / over;
      if constexpr (f < over)
        static_for<per>([&](auto uc) {
          request(next, b + ST - 1, out, std::integral_constant<int, per * f + decltype(uc)::value>{});
        });
#pragma unroll
      for (int m = 0; m < 2; ++m) acc[m][i] = mfma_4_32<j>(w[j & 1][m], x[f % (D + 1)], acc[m][i], sw[m], sx[i]);
    });
  };
  for (int b = 0;;) {
    step(std::false_type{}, b);
    place = place == (ST - 1) * SB ? 0 : place + SB;
    if (++b >= count) break;
    step(std::true_type{}, b);
    place = place == (ST - 1) * SB ? 0 : place + SB;
    if (++b >= count) break;
  }
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  __syncthreads();  // LDS is free
  hold();

  // A wave's 32 rows of a tile and their columns go through its part of LDS, so
  // that neighbouring lanes write neighbouring columns.
  constexpr int CW = PAIR ? 32 : 64, LD = CW + 4;
  float *const turn = reinterpret_cast<float *>(lds) + wave * 32 * 68;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
#pragma unroll
    for (int m = 0; m < (PAIR ? 1 : 2); ++m) {
      f32x4_t v[4];  // columns 8 q + 4 h ..
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (PAIR) v[q][k] = situ4(acc[0][i][4 * q + k], acc[1][i][4 * q + k], g.beta, g.beta_lin);
          else v[q][k] = acc[m][i][4 * q + k];
        }
      if (PAIR && g.out_kind == MX4_OUT_MX4) {
        const int nb = n0 + 32 * wn;  // a block of the result
        uint32_t top = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int k = 0; k < 4; ++k) top = max(top, __float_as_uint(v[q][k]) & 0x7FFFFFFFu);
        top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
        const uint32_t sb = mx4_scale_byte(top, false);
        const float inv = mx4_inverse(sb);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] *= inv;
        // this half's codes, 16 bits of each 8 columns
        uint32_t q01 = mx4_codes(__builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
        uint32_t q23 = mx4_codes(__builtin_shufflevector(v[2], v[3], 0, 1, 2, 3, 4, 5, 6, 7));
        if (sb == 255u) q01 = q23 = 0;
        // the lower half writes columns 0..15 of the block, the upper one 16..31
        const uint32_t mine = h ? q23 : q01, other = (uint32_t)__shfl_xor((int)(h ? q01 : q23), 32, 64);
        const uint32_t lo = h ? other : mine, hi = h ? mine : other;  // columns 8 q + 0..3 and 8 q + 4..7
        const u32x2_t o = {(lo & 0xFFFFu) | hi << 16, lo >> 16 | (hi & 0xFFFF0000u)};
        const int r = 32 * (NT * wt + i) + r32;
        if (r < c.n && nb < g.N) {
          const long long p = c.row + r;
          *reinterpret_cast<u32x2_t *>(static_cast<uint8_t *>(g.out) + p * g.ldo + nb / 2 + 8 * h) = o;
          if (h == 0) g.os[p * g.ldos + nb / 32] = (uint8_t)sb;
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) *reinterpret_cast<f32x4_t *>(turn + r32 * LD + 32 * m + 8 * q + 4 * h) = v[q];
      }
    }
    if (PAIR && g.out_kind == MX4_OUT_MX4) continue;
    const int r0 = 32 * (NT * wt + i);
    // W columns a lane and a row of the tile every CW / W lanes
    auto rows = [&](auto wc, auto &&put) {
      constexpr int W = decltype(wc)::value, RS = 64 * W / CW;
      const int rl = lane / (CW / W), nl = W * (lane % (CW / W));
      f32x4_t v[32 / RS][W / 4];
#pragma unroll
      for (int q = 0; q < 32 / RS; ++q)
#pragma unroll
        for (int k = 0; k < W / 4; ++k) v[q][k] = *reinterpret_cast<const f32x4_t *>(turn + (rl + RS * q) * LD + nl + 4 * k);
#pragma unroll
      for (int q = 0; q < 32 / RS; ++q)
        if (r0 + rl + RS * q < c.n) put(c.row + r0 + rl + RS * q, n0 + CW * wn + nl, v[q]);
    };
    if (partial != nullptr) {
      const int ldp = (g.N + 3) & ~3;
      rows(std::integral_constant<int, 4>{}, [&](long long p, int n, f32x4_t(&v)[1]) {
        if (n < g.N) *reinterpret_cast<f32x4_t *>(partial + p * ldp + n) = v[0];
      });
    } else if (g.out_kind == MX4_OUT_BF16) {
      rows(std::integral_constant<int, 8>{}, [&](long long p, int n, f32x4_t(&v)[2]) {
        if (!PAIR && g.pair_weight != nullptr) {
          const float pw = g.pair_weight[g.pair[p]];
          v[0] *= pw;
          v[1] *= pw;
        }
        if (g.vec_out == 2 && n + 7 < g.N) {
          bf16x8_t b;
#pragma unroll
          for (int k = 0; k < 8; ++k) b[k] = to_bf16(v[k >> 2][k & 3]);
          *reinterpret_cast<bf16x8_t *>(static_cast<__bf16 *>(g.out) + p * g.ldo + n) = b;
        } else {
          store4<MX4_OUT_BF16>(g, p, n, v[0]);
          store4<MX4_OUT_BF16>(g, p, n + 4, v[1]);
        }
      });
    } else {
      rows(std::integral_constant<int, 4>{}, [&](long long p, int n, f32x4_t(&v)[1]) {
        if (!PAIR && g.pair_weight != nullptr) v[0] *= g.pair_weight[g.pair[p]];
        store4<MX4_OUT_F32>(g, p, n, v[0]);
      });
    }
  }
}

// block -> item of `total`, as xcd_logical
MOE_DEV int tile_of(int block, int total) {
  const int t8 = (total + 7) & ~7, id = (block & 7) * (t8 >> 3) + (block >> 3);
  return block < t8 && id < total ? id : -1;
}

// chunk and column tile of item i of chunks * cols: four column tiles next to each
// other, then the next chunk, so that what an XCD works on at a time is near square
MOE_DEV void tile_at(int i, int chunks, int cols, int &chunk, int &col) {
  const int per = 4 * chunks, grp = i / per, in = i - grp * per, gn = min(4, cols - 4 * grp);
  chunk = in / gn;
  col = 4 * grp + in - chunk * gn;
}

// grouped: an item is a chunk and a tile of columns.  Dense: tiles of 256 rows for
// the first `cut` column tiles, of `rows` for the others, whose K may be split
template <bool PAIR, bool SG>
__global__ __launch_bounds__(512, 2) void mx4_tile_kernel(Mx4Args g, int rows, int cut, int splits, float *partial) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[TILE_LDS];
  constexpr int COLS = PAIR ? TILE_COLS / 2 : TILE_COLS;
  const int nb = (g.N + COLS - 1) / COLS, pairs = (g.K + 511) / 512, stages = (g.K + 255) / 256;
  int nblk, cj, first = 0, count = stages;
  Chunk c;
  float *part = nullptr;
  if (g.chunks != nullptr) {
    const int logical = xcd_logical(*g.chunk_count * nb);
    if (logical < 0) return;
    const int ci = logical / nb, info = g.chunks[ci].w, c0 = ci - (info >> 16);  // the expert's first
    tile_at(logical - c0 * nb, info & 0xFFFF, nb, cj, nblk);
    const int4 v = g.chunks[c0 + cj];
    c = Chunk{v.x, v.y, v.z};
  } else {
    const int big = cut * ((g.P + TILE_ROWS - 1) / TILE_ROWS), big8 = (big + 7) & ~7;
    const bool is_big = (int)blockIdx.x < big8;
    const int each = is_big ? TILE_ROWS : rows, cols = is_big ? cut : nb - cut, chunks = (g.P + each - 1) / each;
    const int parts = is_big ? 1 : splits;
    const int logical = tile_of(is_big ? blockIdx.x : blockIdx.x - big8, chunks * cols * parts);
    if (logical < 0) return;
    const int split = logical / (chunks * cols), item = logical - split * chunks * cols;
    tile_at(item, chunks, cols, cj, nblk);
    if (!is_big) nblk += cut;
    c = Chunk{0, each * cj, min(each, g.P - each * cj)};
    if (parts > 1) {
      first = 2 * (int)((long long)split * pairs / parts);
      count = min(stages, 2 * (int)((long long)(split + 1) * pairs / parts)) - first;
      part = partial + (long long)split * g.P * ((g.N + 3) & ~3);
    }
  }
  const int n0 = nblk * COLS;
  switch ((c.n + 63) / 64) {
    case 1: mx4_tile<1, PAIR, SG>(g, c, n0, first, count, part, lds); break;
    case 2: mx4_tile<2, PAIR, SG>(g, c, n0, first, count, part, lds); break;
    case 3: mx4_tile<3, PAIR, SG>(g, c, n0, first, count, part, lds); break;
    default: mx4_tile<4, PAIR, SG>(g, c, n0, first, count, part, lds); break;
  }
}

// the splits' sums in order, four columns a thread
template <int OUT>
__global__ __launch_bounds__(256) void mx4_join_kernel(Mx4Args g, int splits, const float *partial) {
  const int per = (g.N + 3) / 4;  // rows of partial are whole groups of four
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, stride = (long long)g.P * per;
  if (i >= stride) return;
  const int t = (int)(i / per), n = 4 * (int)(i - (long long)t * per);
  const f32x4_t *p = reinterpret_cast<const f32x4_t *>(partial) + i;
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int s = 0; s < splits; ++s) v += p[s * stride];
  store4<OUT>(g, t, n, v);
}

// scale rows that can be loaded 16 bytes at a time
bool scales_in_groups(const Mx4Args &g) {
  auto ok = [](const uint8_t *p, long long ld) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0 && ld % 4 == 0; };
  return ok(g.sx, g.ldsx) && ok(g.sw[0], g.K / 32) && (g.w[1] == nullptr || ok(g.sw[1], g.K / 32));
}
template <int MAXT, bool PAIR, int KS>
void launch_stream(const Mx4Args &g, long long groups, hipStream_t st) {
  const dim3 gr((unsigned)((groups + 7) / 8 * 8)), blk(KS == 1 ? 256 : 512);
  if (scales_in_groups(g)) hipLaunchKernelGGL((mx4_stream_kernel<MAXT, PAIR, true, KS>), gr, blk, 0, st, g);
  else hipLaunchKernelGGL((mx4_stream_kernel<MAXT, PAIR, false, KS>), gr, blk, 0, st, g);
}

constexpr long long PART_THREADS = 1LL << 31;  // a grid holds fewer than 2^32 threads

}  // namespace

hipError_t launch_quantize4(const void *x, bool x_bf16, long long ldx, int T, int K, bool vec, bool ocp, uint8_t *q,
                            long long ldq, uint8_t *qs, long long ldqs, hipStream_t st) {
  const int kb = (K + MX4_BLOCK - 1) / MX4_BLOCK;
  const long long part = std::max(1LL, PART_THREADS / 4 / kb);  // rows; 4 threads a block
  const dim3 blk(256);
  for (long long t = 0; t < T; t += part) {
    const long long n = std::min(T - t, part);
    const dim3 gr((unsigned)((n * kb + 63) / 64));
    if (x_bf16)
      hipLaunchKernelGGL((quantize4_kernel<uint16_t>), gr, blk, 0, st, static_cast<const uint16_t *>(x) + t * ldx, ldx,
                         n, K, (int)vec, (int)ocp, q + t * ldq, ldq, qs + t * ldqs, ldqs);
    else
      hipLaunchKernelGGL((quantize4_kernel<float>), gr, blk, 0, st, static_cast<const float *>(x) + t * ldx, ldx, n, K,
                         (int)vec, (int)ocp, q + t * ldq, ldq, qs + t * ldqs, ldqs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_dequantize4(const uint8_t *q, long long ldq, const uint8_t *qs, long long ldqs, int T, int K, bool vec,
                              void *out, bool out_bf16, long long ldo, hipStream_t st) {
  const int per = (K + 7) / 8;
  const long long part = std::max(1LL, PART_THREADS / per);
  const dim3 blk(256);
  for (long long t = 0; t < T; t += part) {
    const long long n = std::min(T - t, part);
    const dim3 gr((unsigned)((n * per + 255) / 256));
    if (out_bf16)
      hipLaunchKernelGGL((dequantize4_kernel<uint16_t>), gr, blk, 0, st, q + t * ldq, ldq, qs + t * ldqs, ldqs, n, K,
                         (int)vec, static_cast<uint16_t *>(out) + t * ldo, ldo);
    else
      hipLaunchKernelGGL((dequantize4_kernel<float>), gr, blk, 0, st, q + t * ldq, ldq, qs + t * ldqs, ldqs, n, K,
                         (int)vec, static_cast<float *>(out) + t * ldo, ldo);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

namespace {
void launch_tiles(const Mx4Args &g, long long groups, int rows, int cut, int splits, float *partial, hipStream_t st) {
  const dim3 gr((unsigned)groups), blk(512);
  if (scales_in_groups(g)) {
    if (g.w[1] != nullptr) hipLaunchKernelGGL((mx4_tile_kernel<true, true>), gr, blk, 0, st, g, rows, cut, splits, partial);
    else hipLaunchKernelGGL((mx4_tile_kernel<false, true>), gr, blk, 0, st, g, rows, cut, splits, partial);
  } else {
    if (g.w[1] != nullptr) hipLaunchKernelGGL((mx4_tile_kernel<true, false>), gr, blk, 0, st, g, rows, cut, splits, partial);
    else hipLaunchKernelGGL((mx4_tile_kernel<false, false>), gr, blk, 0, st, g, rows, cut, splits, partial);
  }
}
long long up8(long long v) { return (v + 7) / 8 * 8; }

}  // namespace

size_t mx4_workspace_bytes(int T, int N, int K) { return mx4_partial_bytes(T, N, K); }

hipError_t launch_mx4_gemm(const Mx4Args &g, void *ws, hipStream_t st) {
  const Mx4Plan p = mx4_plan(g.P, g.N, g.K);
  if (p.stream) {
    const int nb = (g.N + 31) / 32;
    if (g.P <= 16) launch_stream<1, false, 8>(g, nb, st);
    else if (g.P <= 32) launch_stream<2, false, 8>(g, nb, st);
    else launch_stream<4, false, 8>(g, (long long)nb * ((g.P + 63) / 64), st);
    return hipGetLastError();
  }
  const int nb = (g.N + TILE_COLS - 1) / TILE_COLS;
  const long long big = (long long)p.cut * ((g.P + TILE_ROWS - 1) / TILE_ROWS);
  const long long rest = (long long)(nb - p.cut) * ((g.P + p.rows - 1) / p.rows) * p.splits;
  launch_tiles(g, up8(big) + up8(rest), p.rows, p.cut, p.splits, static_cast<float *>(ws), st);
  if (p.splits > 1) {
    const dim3 jr((unsigned)(((long long)g.P * ((g.N + 3) / 4) + 255) / 256));
    if (g.out_kind == MX4_OUT_BF16)
      hipLaunchKernelGGL(mx4_join_kernel<MX4_OUT_BF16>, jr, dim3(256), 0, st, g, p.splits, static_cast<const float *>(ws));
    else
      hipLaunchKernelGGL(mx4_join_kernel<MX4_OUT_F32>, jr, dim3(256), 0, st, g, p.splits, static_cast<const float *>(ws));
  }
  return hipGetLastError();
}

size_t mx4_expert_workspace_bytes(int E, int P, int, int) {
  return 256 + (size_t)(mx4_few_chunks(E, P) + mx4_many_chunks(E, P)) * sizeof(int4);
}

hipError_t launch_mx4_expert(const Mx4Args &a, void *ws, hipStream_t st) {
  Mx4Args g = a;
  const int E = g.n_experts, groups = mx4_stream_groups(g.N, g.w[1] != nullptr);
  const bool pair = g.w[1] != nullptr;
  if (mx4_finds_chunks(E, g.P, groups)) {
    const int chunks = mx4_found_chunks(E, g.P);
    if (pair) launch_stream<4, true, 1>(g, (long long)chunks * groups, st);
    else launch_stream<4, false, 1>(g, (long long)chunks * groups, st);
    return hipGetLastError();
  }
  int32_t *count = static_cast<int32_t *>(ws);
  int4 *few = reinterpret_cast<int4 *>(static_cast<char *>(ws) + 256), *many = few + mx4_few_chunks(E, g.P);
  hipLaunchKernelGGL(mx4_plan_kernel, dim3(1), dim3(1024), 0, st, g.offsets, E, g.P, mx4_few_rows(E, g.P), TILE_ROWS,
                     mx4_few_chunks(E, g.P), few, count, mx4_many_chunks(E, g.P), many, count + 1);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (mx4_many_chunks(E, g.P) > 0) {
    g.chunks = many;
    g.chunk_count = count + 1;
    launch_tiles(g, up8((long long)mx4_many_chunks(E, g.P) * ((g.N + (pair ? 127 : 255)) / (pair ? 128 : 256))), 0, 0, 1, nullptr, st);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (mx4_few_chunks(E, g.P) == 0) return hipSuccess;
  g.chunks = few;
  g.chunk_count = count;
  if (pair) launch_stream<1, true, 1>(g, (long long)mx4_few_chunks(E, g.P) * groups, st);
  else launch_stream<1, false, 1>(g, (long long)mx4_few_chunks(E, g.P) * groups, st);
  return hipGetLastError();
}

}  // namespace moe
