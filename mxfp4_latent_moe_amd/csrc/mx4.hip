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

// Rows of fp32 or bf16 values in MXFP4: a block is four lanes of 8 values.
// vec: rows' chunks of 8 are whole and aligned.
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

// and back, eight values a thread
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

// c + 16 rows times 16 columns over 128 codes: a lane holds block lane / 16 of
// row (column) lane % 16, and that block's scale byte
MOE_DEV f32x4_t mfma_4_16(u32x4_t w, u32x4_t x, f32x4_t c, uint32_t sw, uint32_t sx) {
  const i32x4_t w4 = __builtin_bit_cast(i32x4_t, w), x4 = __builtin_bit_cast(i32x4_t, x);
  const i32x8_t a = __builtin_shufflevector(w4, w4, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8_t b = __builtin_shufflevector(x4, x4, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, 0, (int)sw, 0, (int)sx);
}

// an expert's rows [row, row + n) of a grouped product, or rows of the dense one
struct Chunk {
  int expert, row, n;
};

// Chunks of at most `rows` sorted rows, an expert's one after the other.  Bad
// offsets give wrong chunks but none outside the P rows and the list's `cap`.
__global__ __launch_bounds__(1024) void mx4_plan_kernel(const int32_t *offsets, int E, int P, int rows, int cap,
                                                        int4 *chunks, int32_t *count) {
  __shared__ int tot[16];
  const int e = threadIdx.x, lane = e & 63, wave = e >> 6;
  int lo = 0, ne = 0;
  if (e < E) {
    lo = min(max(offsets[e], 0), P);
    ne = min(max(offsets[e + 1], lo), P) - lo;
  }
  const int nch = (ne + rows - 1) / rows;
  int x = nch;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  if (lane == 63) tot[wave] = x;
  __syncthreads();
  int at = x - nch, sum = 0;
  for (int w = 0; w < 16; ++w) {
    if (w < wave) at += tot[w];
    sum += tot[w];
  }
  for (int i = 0; i < nch && at + i < cap; ++i)
    chunks[at + i] = int4{e, lo + i * rows, min(rows, ne - i * rows), 0};
  if (e == 0) *count = min(sum, cap);
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

// Few rows: the weights are the whole cost.  A work-group owns 32 columns of the
// result (of a pair, 32 weight rows of each matrix) and 16 NT rows; its NW waves
// take steps of 128 inputs in turn, so that at any time they read a contiguous
// NW * 64 bytes of each weight row, U steps in flight each.  Both operands come
// straight from memory, the rows from the L2.  The waves' sums meet in LDS and
// are added in wave order.
template <int NT, int NW, int U, bool PAIR, int OUT>
__global__ __launch_bounds__(64 * NW) void mx4_stream_kernel(Mx4Args g) {
  constexpr int NM = PAIR ? 2 : 1;
  __shared__ f32x4_t part[NW][NM][2][NT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kg = lane >> 4;
  const int K = g.K, kbytes = K / 2, kb = K / 32, steps = (K + 127) / 128;
  const int nb = (g.N + 31) / 32;
  const int total = (g.chunks != nullptr ? *g.chunk_count : (g.P + 16 * NT - 1) / (16 * NT)) * nb;
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    const int ci = item / nb, n0 = 32 * (item - ci * nb);
    Chunk c{0, 16 * NT * ci, min(16 * NT, g.P - 16 * NT * ci)};
    if (g.chunks != nullptr) {
      const int4 v = g.chunks[ci];
      c = Chunk{v.x, v.y, v.z};
    }
    const int nrows = min(32, g.N - n0);
    __amdgpu_buffer_rsrc_t wr[NM], sr[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      const long long row = (long long)c.expert * g.N + n0;
      wr[m] = make_rsrc(g.w[m] + row * kbytes, (uint32_t)nrows * (uint32_t)kbytes);
      sr[m] = make_rsrc(g.sw[m] + row * kb, (uint32_t)nrows * (uint32_t)kb);
    }
    // gathered rows are found from the first row of x, others from the chunk's own
    const long long base = g.map != nullptr ? 0 : c.row;
    const int xrows = g.map != nullptr ? g.x_rows : c.n;
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.x + base * g.ldx, (uint32_t)((xrows - 1) * g.ldx + kbytes));
    const __amdgpu_buffer_rsrc_t xsr = make_rsrc(g.sx + base * g.ldsx, (uint32_t)((xrows - 1) * g.ldsx + kb));
    uint32_t wo[2], so[2], xo[NT], xso[NT];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int r = min(16 * m + r16, nrows - 1);
      wo[m] = (uint32_t)r * (uint32_t)kbytes + 16 * kg;
      so[m] = (uint32_t)r * (uint32_t)kb + kg;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int r = x_row(g, c.row + min(16 * i + r16, c.n - 1)) - (int)base;
      xo[i] = (uint32_t)r * (uint32_t)g.ldx + 16 * kg;
      xso[i] = (uint32_t)r * (uint32_t)g.ldsx + kg;
    }
    f32x4_t acc[NM][2][NT];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[m][j][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int b0 = wave; b0 < steps; b0 += NW * U) {
      u32x4_t w[U][NM][2], x[U][NT];
      uint32_t sw[U][NM][2], sx[U][NT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // steps past the end, and lanes whose block is past it, read out of range: codes of zero
        const int b = b0 + NW * u;
        const bool in = 4 * b + kg < kb;
        const uint32_t past = in ? 0u : 0x80000000u;
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            w[u][m][j] = buf_load16(wr[m], wo[j] + past, 64u * b);
            sw[u][m][j] = __builtin_amdgcn_raw_buffer_load_b8(sr[m], so[j] + past, 4u * b, 0);
          }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          x[u][i] = buf_load16(xr, xo[i] + past, 64u * b);
          sx[u][i] = __builtin_amdgcn_raw_buffer_load_b8(xsr, xso[i] + past, 4u * b, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // every load of the round is on its way before the first product
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < NT; ++i)
              acc[m][j][i] = mfma_4_16(w[u][m][j], x[u][i], acc[m][j][i], sw[u][m][j], sx[u][i]);
    }
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i) part[wave][m][j][i][lane] = acc[m][j][i];
    __syncthreads();
    // eight neighbouring threads a row, four columns each
    for (int e = threadIdx.x; e < 128 * NT; e += 64 * NW) {
      const int t = e >> 3, j = e >> 2 & 1, h = e & 3, l = 16 * h + (t & 15), i = t >> 4;
      f32x4_t v[NM];
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        v[m] = part[0][m][j][i][l];
#pragma unroll
        for (int q = 1; q < NW; ++q) v[m] += part[q][m][j][i][l];
      }
      if constexpr (PAIR) {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[0][r] = situ_glu(v[0][r], v[1][r], g.beta, g.beta_lin);
      }
      const int n = n0 + 16 * j + 4 * h;
      const long long p = c.row + t;
      if (!PAIR && g.pair_weight != nullptr && t < c.n) v[0] *= g.pair_weight[g.pair[p]];
      if constexpr (OUT == MX4_OUT_MX4) {
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < 4; ++r) m = max(m, __float_as_uint(v[0][r]) & 0x7FFFFFFFu);
        m = max4(m);
        m = max(m, (uint32_t)__shfl_xor((int)m, 4, 64));
        const uint32_t sb = mx4_scale_byte(m, false);
        v[0] *= mx4_inverse(sb);
        uint32_t q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0][0], v[0][1], 1.0f, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0][2], v[0][3], 1.0f, 1);
        if (t < c.n) {
          *reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(g.out) + p * g.ldo + n / 2) =
              sb == 255u ? (uint16_t)0 : (uint16_t)q;
          if ((e & 7) == 0) g.os[p * g.ldos + n / 32] = (uint8_t)sb;
        }
      } else {
        if (t < c.n) store4<OUT>(g, p, n, v[0]);
      }
    }
    __syncthreads();  // part is free again
  }
}

template <int NT, int NW, int U>
void stream_by_type(const Mx4Args &g, int max_items, hipStream_t st) {
  const dim3 gr((unsigned)std::min(max_items, 1 << 20)), blk(64 * NW);
  if (g.w[1] != nullptr) {
    if (g.out_kind == MX4_OUT_F32) hipLaunchKernelGGL((mx4_stream_kernel<NT, NW, U, true, MX4_OUT_F32>), gr, blk, 0, st, g);
    else if (g.out_kind == MX4_OUT_BF16) hipLaunchKernelGGL((mx4_stream_kernel<NT, NW, U, true, MX4_OUT_BF16>), gr, blk, 0, st, g);
    else hipLaunchKernelGGL((mx4_stream_kernel<NT, NW, U, true, MX4_OUT_MX4>), gr, blk, 0, st, g);
  } else {
    if (g.out_kind == MX4_OUT_F32) hipLaunchKernelGGL((mx4_stream_kernel<NT, NW, U, false, MX4_OUT_F32>), gr, blk, 0, st, g);
    else hipLaunchKernelGGL((mx4_stream_kernel<NT, NW, U, false, MX4_OUT_BF16>), gr, blk, 0, st, g);
  }
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
constexpr int CHUNK_ROWS = 64;
int max_chunks(int E, int P) { return P / CHUNK_ROWS + std::min(E, P); }
}  // namespace

size_t mx4_workspace_bytes(int, int, int) { return 0; }

hipError_t launch_mx4_gemm(const Mx4Args &g, void *, hipStream_t st) {
  const int nb = (g.N + 31) / 32;
  if (g.P <= 16) stream_by_type<1, 8, 4>(g, nb, st);
  else stream_by_type<4, 4, 2>(g, (g.P + 63) / 64 * nb, st);
  return hipGetLastError();
}

size_t mx4_expert_workspace_bytes(int E, int P, int, int) { return 256 + (size_t)max_chunks(E, P) * sizeof(int4); }

hipError_t launch_mx4_expert(const Mx4Args &a, const int32_t *offsets, int E, void *ws, hipStream_t st) {
  Mx4Args g = a;
  int32_t *count = static_cast<int32_t *>(ws);
  int4 *chunks = reinterpret_cast<int4 *>(static_cast<char *>(ws) + 256);
  const int cap = max_chunks(E, g.P);
  hipLaunchKernelGGL(mx4_plan_kernel, dim3(1), dim3(1024), 0, st, offsets, E, g.P, CHUNK_ROWS, cap, chunks, count);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  g.chunks = chunks;
  g.chunk_count = count;
  stream_by_type<4, 4, 2>(g, cap * ((g.N + 31) / 32), st);
  return hipGetLastError();
}

}  // namespace moe
