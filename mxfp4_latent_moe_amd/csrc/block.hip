// The norms around the block.
//
//   pre:   n = x / sqrt(mean(x^2) + eps) * gamma, as bf16 and / or as e4m3
//          codes with a power-of-two scale per 128 channels (quant8.h)
//   post:  out = r + s g (y / sqrt(mean(y^2) + eps) * gamma), with the gate g
//          absent, one per token, one per channel or one per value, as given
//          or through a sigmoid; then, if asked, the next block's pre-norm of
//          the row of out as it is stored
//
// Both are bound by memory: a row is read once, stays in registers through its
// reductions and is written once.  One work-group per row: NT threads of 8
// consecutive channels each, NC rounds of them, so a thread's loads are 16 or
// 32 bytes wide and all in flight before the first sum.  Sums of squares are
// held in fp32: 8 NC values in a thread, then a butterfly over the wave and a
// fixed-order sum over the waves, so a row's result does not depend on the
// other rows or the launch.
//
// Measured, 4096 rows of 7168: pre from fp32 to bf16 33 us (176 MB, 5.3 TB/s; a
// copy of 1 GiB runs at 5.07), 4001 rows post with a gate per channel in fp32
// 66 us (344 MB, 5.2 TB/s).  One row takes 2.4 to 4.5 us.
#include <algorithm>

#include "kernels.h"
#include "quant8.h"

namespace moe {
namespace {

typedef float f32x8_t __attribute__((ext_vector_type(8)));

template <typename T>
MOE_DEV f32x8_t widen8(const u32x4_t &a, const u32x4_t &b) {
  f32x8_t v;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 2) {
      v[i] = __uint_as_float((i & 1) ? (a[i >> 1] & 0xFFFF0000u) : (a[i >> 1] << 16));
    } else {
      v[i] = __uint_as_float(i < 4 ? a[i & 3] : b[i & 3]);
    }
  }
  return v;
}
MOE_DEV float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
MOE_DEV float widen(float v) { return v; }

// eight channels from c on; past the row's end zeros.  vec: the row's chunks
// are whole and 16-byte aligned.
template <typename T>
MOE_DEV f32x8_t load8(const T *row, int c, int H, bool vec) {
  if (vec) {
    u32x4_t a{0, 0, 0, 0}, b{0, 0, 0, 0};
    if (c < H) {
      const u32x4_t *p = reinterpret_cast<const u32x4_t *>(row + c);
      a = p[0];
      if constexpr (sizeof(T) == 4) b = p[1];
    }
    return widen8<T>(a, b);
  }
  f32x8_t v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = c + i < H ? widen(row[c + i]) : 0.f;
  return v;
}

// the value as it is stored, back in fp32
template <typename T>
MOE_DEV f32x8_t store8(T *row, int c, int H, bool vec, f32x8_t v) {
  if constexpr (sizeof(T) == 2) {
    bf16x8_t b;
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = to_bf16(v[i]);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = from_bf16(b[i]);
    if (vec) {
      if (c < H) *reinterpret_cast<bf16x8_t *>(row + c) = b;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < H) reinterpret_cast<__bf16 *>(row)[c + i] = b[i];
    }
  } else {
    if (vec) {
      if (c < H) {
        reinterpret_cast<f32x4_t *>(row + c)[0] = f32x4_t{v[0], v[1], v[2], v[3]};
        reinterpret_cast<f32x4_t *>(row + c)[1] = f32x4_t{v[4], v[5], v[6], v[7]};
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < H) row[c + i] = v[i];
    }
  }
  return v;
}

template <int NT>
MOE_DEV float block_sum(float s, float *red) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) t += red[i];
  return t;
}

template <int NC>
MOE_DEV float square_sum(const f32x8_t (&v)[NC]) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    f32x8_t q = v[j] * v[j];
    s += ((q[0] + q[1]) + (q[2] + q[3])) + ((q[4] + q[5]) + (q[6] + q[7]));
  }
  return s;
}

MOE_DEV float rms_factor(float ss, int H, float eps) { return 1.0f / sqrtf(ss / (float)H + eps); }

// the normed row in the forms asked for
template <int NT, int NC>
MOE_DEV void write_normed(const NormOut &o, long long t, int H, bool vec, const f32x8_t (&v)[NC], float f) {
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = 8 * (threadIdx.x + NT * j);
    f32x8_t n = v[j] * f * load8<uint16_t>(o.gamma, c, H, vec);
    if (o.n != nullptr) store8<uint16_t>(o.n + t * o.ldn, c, H, vec, n);
    if (o.q != nullptr) {
      // a block of 128 channels is 16 neighbouring lanes; lanes past the row hold zeros
      uint32_t lo, hi;
      const uint32_t sb = q8_block(n, lo, hi);
      uint8_t *q = o.q + t * o.ldq;
      if (vec) {
        if (c < H) *reinterpret_cast<u32x2_t *>(q + c) = u32x2_t{lo, hi};
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c + i < H) q[c + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
      }
      if ((threadIdx.x & 15) == 0 && c < H) o.qs[t * o.ldqs + c / Q8_BLOCK] = (uint8_t)sb;
    }
  }
}

template <typename X, int NT, int NC>
__global__ __launch_bounds__(NT) void pre_norm_kernel(const X *__restrict__ x, long long ldx, int H, float eps,
                                                      int vec, NormOut o) {
  __shared__ float red[NT / 64];
  const long long t = blockIdx.x;
  f32x8_t v[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) v[j] = load8<X>(x + t * ldx, 8 * (threadIdx.x + NT * j), H, vec);
  const float f = rms_factor(block_sum<NT>(square_sum<NC>(v), red), H, eps);
  write_normed<NT, NC>(o, t, H, vec, v, f);
}

template <typename Y, typename R, int NT, int NC>
__global__ __launch_bounds__(NT) void post_norm_kernel(PostNormArgs a) {
  __shared__ float red[2][NT / 64];
  const long long t = blockIdx.x;
  const int H = a.H;
  const bool vec = a.vec;
  f32x8_t y[NC], r[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j)
    y[j] = load8<Y>(static_cast<const Y *>(a.y) + t * a.ldy, 8 * (threadIdx.x + NT * j), H, vec);
#pragma unroll
  for (int j = 0; j < NC; ++j)
    r[j] = load8<R>(static_cast<const R *>(a.resid) + t * a.ldr, 8 * (threadIdx.x + NT * j), H, vec);
  float f = 1.f;
  if (a.gamma != nullptr) f = rms_factor(block_sum<NT>(square_sum<NC>(y), red[0]), H, a.eps);
  auto squash = [&](float g) { return a.gate_sigmoid ? 1.0f / (1.0f + expf(-g)) : g; };
  float gt = 1.f;  // one gate for the row
  if (a.gate != nullptr && !a.gate_channels)
    gt = squash(a.gate_bf16 ? widen(static_cast<const uint16_t *>(a.gate)[t * a.ldg])
                            : static_cast<const float *>(a.gate)[t * a.ldg]);
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = 8 * (threadIdx.x + NT * j);
    f32x8_t b = y[j];
    if (a.gamma != nullptr) b = b * f * load8<uint16_t>(a.gamma, c, H, vec);
    b = b * a.scale;
    if (a.gate_channels) {
      f32x8_t g = a.gate_bf16 ? load8<uint16_t>(static_cast<const uint16_t *>(a.gate) + t * a.ldg, c, H, vec)
                              : load8<float>(static_cast<const float *>(a.gate) + t * a.ldg, c, H, vec);
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] *= squash(g[i]);
    } else if (a.gate != nullptr) {
      b = b * gt;
    }
    r[j] = store8<R>(static_cast<R *>(a.out) + t * a.ldo, c, H, vec, r[j] + b);
    if (c >= H) r[j] = f32x8_t{};
    else if (!vec) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i >= H) r[j][i] = 0.f;
    }
  }
  if (a.next.gamma == nullptr) return;
  const float fn = rms_factor(block_sum<NT>(square_sum<NC>(r), red[1]), H, a.eps);
  write_normed<NT, NC>(a.next, t, H, vec, r, fn);
}

// e4m3 codes and scales of rows of fp32 or bf16 values: a block of 128 is 16
// lanes of 8 values, one pass, bound by memory: 4096 rows of 7168 bf16 20.8 us
// (88 MB, 4.2 TB/s).  Two and four blocks a thread took 2% and 16% longer.
template <typename X>
__global__ __launch_bounds__(256) void quantize8_kernel(const X *__restrict__ x, long long ldx, long long T, int K,
                                                        int vec, uint8_t *__restrict__ q, long long ldq,
                                                        uint8_t *__restrict__ qs, long long ldqs) {
  const int kb = (K + Q8_BLOCK - 1) / Q8_BLOCK;
  const long long first = 16LL * blockIdx.x, t0 = first / kb;  // of the work-group
  const int b0 = (int)(first - t0 * kb) + (threadIdx.x >> 4), r = b0 / kb, b = b0 - r * kb;
  const long long t = t0 + r;
  const int c = b * Q8_BLOCK + 8 * (threadIdx.x & 15);
  f32x8_t v{};
  if (t < T) v = load8<X>(x + t * ldx, c, K, vec);
  uint32_t lo, hi;
  const uint32_t sb = q8_block(v, lo, hi);
  if (t >= T) return;
  uint8_t *row = q + t * ldq;
  if (vec) {
    if (c < K) *reinterpret_cast<u32x2_t *>(row + c) = u32x2_t{lo, hi};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < K) row[c + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
  }
  if ((threadIdx.x & 15) == 0) qs[t * ldqs + b] = (uint8_t)sb;
}

constexpr int NORM_NT = 512;
// Rows up to 1024 wide have fewer threads: 4096 rows of 256, pre with codes 5.2
// us (with 512 threads 12.7), post with the next pre-norm 6.4 (17.0).
constexpr int NORM_NARROW = 128;

template <typename X>
void pre_by_width(const X *x, long long ldx, int T, int H, float eps, bool vec, const NormOut &o, hipStream_t st) {
  const dim3 gr((unsigned)T), blk(NORM_NT);
  if (H <= 8 * NORM_NARROW)
    hipLaunchKernelGGL((pre_norm_kernel<X, NORM_NARROW, 1>), gr, dim3(NORM_NARROW), 0, st, x, ldx, H, eps, (int)vec, o);
  else if (H <= 8 * NORM_NT)
    hipLaunchKernelGGL((pre_norm_kernel<X, NORM_NT, 1>), gr, blk, 0, st, x, ldx, H, eps, (int)vec, o);
  else if (H <= 16 * NORM_NT)
    hipLaunchKernelGGL((pre_norm_kernel<X, NORM_NT, 2>), gr, blk, 0, st, x, ldx, H, eps, (int)vec, o);
  else
    hipLaunchKernelGGL((pre_norm_kernel<X, NORM_NT, 4>), gr, blk, 0, st, x, ldx, H, eps, (int)vec, o);
}

template <typename Y, typename R>
void post_by_width(const PostNormArgs &a, hipStream_t st) {
  const dim3 gr((unsigned)a.T), blk(NORM_NT);
  if (a.H <= 8 * NORM_NARROW)
    hipLaunchKernelGGL((post_norm_kernel<Y, R, NORM_NARROW, 1>), gr, dim3(NORM_NARROW), 0, st, a);
  else if (a.H <= 8 * NORM_NT)
    hipLaunchKernelGGL((post_norm_kernel<Y, R, NORM_NT, 1>), gr, blk, 0, st, a);
  else if (a.H <= 16 * NORM_NT)
    hipLaunchKernelGGL((post_norm_kernel<Y, R, NORM_NT, 2>), gr, blk, 0, st, a);
  else
    hipLaunchKernelGGL((post_norm_kernel<Y, R, NORM_NT, 4>), gr, blk, 0, st, a);
}

}  // namespace

static_assert(NORM_MAX_H == 32 * NORM_NT, "the widest row the norm kernels hold");

// A grid holds fewer than 2^32 threads: one that passes that comes out shorter,
// without an error.  Longer calls go out in parts.
constexpr long long PART_THREADS = 1LL << 31;
constexpr int PART_ROWS = (int)(PART_THREADS / NORM_NT);

// the rows from t on
static NormOut rows_from(NormOut o, long long t) {
  if (o.n != nullptr) o.n += t * o.ldn;
  if (o.q != nullptr) {
    o.q += t * o.ldq;
    o.qs += t * o.ldqs;
  }
  return o;
}

hipError_t launch_pre_norm(const void *x, bool x_bf16, long long ldx, int T, int H, float eps, bool vec,
                           const NormOut &o, hipStream_t st) {
  for (long long t = 0; t < T; t += PART_ROWS) {
    const int n = (int)std::min<long long>(T - t, PART_ROWS);
    if (x_bf16) pre_by_width(static_cast<const uint16_t *>(x) + t * ldx, ldx, n, H, eps, vec, rows_from(o, t), st);
    else pre_by_width(static_cast<const float *>(x) + t * ldx, ldx, n, H, eps, vec, rows_from(o, t), st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_post_norm(const PostNormArgs &a, bool y_bf16, bool r_bf16, hipStream_t st) {
  const int yb = y_bf16 ? 2 : 4, rb = r_bf16 ? 2 : 4, gb = a.gate_bf16 ? 2 : 4;
  for (long long t = 0; t < a.T; t += PART_ROWS) {
    PostNormArgs p = a;
    p.T = (int)std::min<long long>(a.T - t, PART_ROWS);
    p.y = static_cast<const char *>(a.y) + t * a.ldy * yb;
    p.resid = static_cast<const char *>(a.resid) + t * a.ldr * rb;
    p.out = static_cast<char *>(a.out) + t * a.ldo * rb;
    if (a.gate != nullptr) p.gate = static_cast<const char *>(a.gate) + t * a.ldg * gb;
    p.next = rows_from(a.next, t);
    if (y_bf16) {
      if (r_bf16) post_by_width<uint16_t, uint16_t>(p, st);
      else post_by_width<uint16_t, float>(p, st);
    } else {
      if (r_bf16) post_by_width<float, uint16_t>(p, st);
      else post_by_width<float, float>(p, st);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_quantize8(const void *x, bool x_bf16, long long ldx, int T, int K, bool vec, uint8_t *q,
                            long long ldq, uint8_t *qs, long long ldqs, hipStream_t st) {
  const int kb = (K + Q8_BLOCK - 1) / Q8_BLOCK;
  const long long part = std::max(1LL, PART_THREADS / 16 / kb);  // rows; 16 threads a block
  const dim3 blk(256);
  for (long long t = 0; t < T; t += part) {
    const long long n = std::min(T - t, part);
    const dim3 gr((unsigned)((n * kb + 15) / 16));
    if (x_bf16)
      hipLaunchKernelGGL((quantize8_kernel<uint16_t>), gr, blk, 0, st, static_cast<const uint16_t *>(x) + t * ldx, ldx,
                         n, K, (int)vec, q + t * ldq, ldq, qs + t * ldqs, ldqs);
    else
      hipLaunchKernelGGL((quantize8_kernel<float>), gr, blk, 0, st, static_cast<const float *>(x) + t * ldx, ldx, n, K,
                         (int)vec, q + t * ldq, ldq, qs + t * ldqs, ldqs);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
