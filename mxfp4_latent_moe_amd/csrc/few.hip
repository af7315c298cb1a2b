// The whole layer for a few tokens (T <= 4) in two kernels.
//
// At these sizes every weight of the layer that the tokens touch is read once
// and used for at most four columns, so the layer is one weight stream of the
// router, the latent projections, the shared experts and the chosen experts,
// and what costs time beside it are the places where the stream stops: kernel
// boundaries, and steps that wait for a step before them.
//
//   few_front_kernel  logits = x W_r^T and z = x W_d^T (both need x alone)
//   few_layer_kernel  everything else, as work items in one list:
//       top-k (a token) | shared gate/up (16 rows) | expert gate/up (32 rows) |
//       shared down (16 rows) | expert down (64 rows) | combine (256 columns) |
//       up_proj (16 rows)
//     A work-group takes items from the list in order, by a ticket counter.
//     An item that needs another step's results waits for that step's counter;
//     the steps are ordered so that the results are usually there: the shared
//     experts' items, which need only x, fill the time of the top-k and of the
//     last expert gate/up items.
//
// Every wait ends, whatever part of the grid is resident: an item waits only
// for items with smaller tickets, tickets are handed out in order to
// work-groups that are running, and a work-group works its tickets off in
// order (it holds at most the one it works on and the next).  So the smallest
// unfinished ticket is always at work and waits for nothing unfinished.
//
// Arithmetic: weight rows on the MFMA's M side, on its N side up to 15 columns.
// x is exact in bf16.  z, the hidden activations and the normed latent are kept
// as three bf16 planes (a = a1 + a2 + a3, exact for normal fp32), three columns
// per token, so every product is that of the fp32 value with the exact weight;
// sums are fp32.  The columns cost nothing: the kernel waits for weights.  The
// eight waves of a work-group take the K steps in turn; their sums are added
// in wave order, so results do not depend on the schedule.  RMSNorm's factor is
// one number per token and is applied to up_proj's sums.
#include <atomic>

#include "kernels.h"
#include "topk.h"

namespace moe {
namespace {

constexpr int FW = 8;             // waves per work-group
constexpr int FTHR = 64 * FW;
constexpr int MT_GU = 2;          // 16-row tiles per matrix of an expert gate/up item
constexpr int MT_DN = 4;          // of an expert down item
constexpr int CMB = 256;          // columns of a combine item

// counters, one per 128-byte line
enum { C_TICKET = 0, C_TOPK = 32, C_READY = 64, C_SGU = 96, C_EGU = 128, C_SDN = 160, C_EDN = 192, C_CMB = 224 };

MOE_DEV int32_t load_count(const int32_t *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
MOE_DEV int32_t add_count(int32_t *p) { return __hip_atomic_fetch_add(p, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
// this wave's stores are visible on the device before its next atomic
MOE_DEV void release() { __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent"); }
MOE_DEV void acquire() { __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent"); }
// counts one finished wave of an item
MOE_DEV void done(int32_t *p) {
  release();
  if (lane_id() == 0) add_count(p);
}

MOE_DEV void split3(float a, __bf16 &h, __bf16 &m, __bf16 &l) {
  h = to_bf16(a);
  const float r = a - from_bf16(h);
  m = to_bf16(r);
  l = to_bf16(r - from_bf16(m));
}
// Four consecutive values k0 .. k0 + 3 (k0 a multiple of 4) of a row kept in
// planes: octet o of the row holds its three planes' eight values one after
// the other, 48 bytes.
MOE_DEV void store_planes(uint16_t *row, int k0, f32x4_t v) {
  bf16x4_t h, m, l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __bf16 a, b, c;
    split3(v[i], a, b, c);
    h[i] = a;
    m[i] = b;
    l[i] = c;
  }
  uint16_t *p = row + (k0 >> 3) * 24 + (k0 & 4);
  *reinterpret_cast<bf16x4_t *>(p) = h;
  *reinterpret_cast<bf16x4_t *>(p + 8) = m;
  *reinterpret_cast<bf16x4_t *>(p + 16) = l;
}

// the N-side operand of a product: lane column c's row, by octets
struct Cols {
  __amdgpu_buffer_rsrc_t r;
  uint32_t off;      // byte offset of the lane's column
  uint32_t ostride;  // bytes between octets
};

// acc[t] += tile t (16 rows x K) * columns, over the K steps of this wave.
// W[t]: first byte of the tile, nrows its rows (bf16 [16][K] or packed
// [16][K/2] with scales S[t] [16][K/32]).
template <int WF, int NT, int U>
MOE_DEV void product(f32x4_t (&acc)[NT], const uint8_t *const (&W)[NT], const uint8_t *const (&S)[NT], int nrows,
                     int K, const Cols &b, int wave) {
  constexpr int WR = WF == W_MXFP4 ? 1 : 4;
  constexpr uint32_t STEP = WF == W_MXFP4 ? 64 : 256;
  const int lane = lane_id(), r16 = lane & 15, kg = lane >> 4;
  const uint32_t row_bytes = WF == W_MXFP4 ? K / 2 : 2 * K;
  const int nks = K / 128;
  const int row = min(r16, nrows - 1);
  const uint32_t wo = row * row_bytes + 16 * kg, so = row * (K / 32);
  __amdgpu_buffer_rsrc_t wr[NT], sr[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    wr[t] = make_rsrc(W[t], nrows * row_bytes);
    if constexpr (WF == W_MXFP4) sr[t] = make_rsrc(S[t], nrows * (K / 32));
  }
  for (int s0 = wave; s0 < nks; s0 += FW * U) {
    u32x4_t w[U][NT][WR], x[U][4];
    uint32_t sc[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t s = min(s0 + FW * u, nks - 1);  // past the end: the last step again, not used
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < WR; ++j) w[u][t][j] = buf_load16(wr[t], wo + 64 * j, s * STEP);
        if constexpr (WF == W_MXFP4) sc[u][t] = buf_load4(sr[t], so, 4 * s);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t s = min(s0 + FW * u, nks - 1);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[u][j] = buf_load16(b.r, b.off + (WF == W_MXFP4 ? 4 * kg + j : 4 * j + kg) * b.ostride, 16 * s * b.ostride);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + FW * u >= nks) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8_t xb = __builtin_bit_cast(bf16x8_t, x[u][j]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          bf16x8_t a;
          if constexpr (WF == W_MXFP4) a = fp4x8_to_bf16(w[u][t][0][j], e8m0_to_float((sc[u][t] >> (8 * kg)) & 0xFFu));
          else a = __builtin_bit_cast(bf16x8_t, w[u][t][j]);
          acc[t] = mfma_16x16x32(a, xb, acc[t]);
        }
      }
    }
  }
}

// columns that are rows of x: column c is token c
MOE_DEV Cols cols_x(const uint16_t *x, int T, int H) {
  return Cols{make_rsrc(x, (uint32_t)T * H * 2), (uint32_t)min(lane_id() & 15, T - 1) * H * 2, 16u};
}
// columns that are planes: column 3 j + p is plane p of row[j]; past 3 n the first column
MOE_DEV Cols cols_planes(const uint16_t *planes, uint32_t bytes, int K, int n, const int32_t (&row)[FEW_MAX_T]) {
  const int c = lane_id() & 15, j = c / 3;
  int q = row[0];
#pragma unroll
  for (int i = 1; i < FEW_MAX_T; ++i) q = j == i && i < n ? row[i] : q;
  return Cols{make_rsrc(planes, bytes), (uint32_t)q * (uint32_t)K * 6u + (j < n ? 16u * (c - 3 * j) : 0u), 48u};
}

// the waves' sums of tile t, in wave order
MOE_DEV f32x4_t wave_sum(const f32x4_t (*part)[MT_DN][64], int t) {
  f32x4_t v = part[0][t][lane_id()];
#pragma unroll
  for (int q = 1; q < FW; ++q) v += part[q][t][lane_id()];
  return v;
}
// the three planes' columns of a token together, in its first column
MOE_DEV f32x4_t plane_sum(f32x4_t v) {
  f32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = v[i] + (__shfl_down(v[i], 1, 64) + __shfl_down(v[i], 2, 64));
  return r;
}

// ---- x W_r^T and x W_d^T, 16 rows a work-group
__global__ __launch_bounds__(FTHR, 4) void few_front_kernel(FewArgs a) {
  __shared__ f32x4_t part[FW][MT_DN][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < FEW_COUNTERS; i += FTHR) a.counters[i] = 0;
  const int nb_r = (a.E + 15) / 16;
  const bool router = (int)blockIdx.x < nb_r;
  const int n0 = 16 * (router ? blockIdx.x : blockIdx.x - nb_r);
  const int N = router ? a.E : a.L;
  f32x4_t acc[1] = {f32x4_t{0.f, 0.f, 0.f, 0.f}};
  const uint8_t *W[1] = {reinterpret_cast<const uint8_t *>((router ? a.w_router : a.w_down) + (long long)n0 * a.H)};
  const uint8_t *S[1] = {nullptr};
  product<W_BF16, 1, 2>(acc, W, S, min(16, N - n0), a.H, cols_x(a.x, a.T, a.H), wave);
  part[wave][0][lane] = acc[0];
  __syncthreads();
  if (wave != 0) return;
  const f32x4_t v = wave_sum(part, 0);
  const int t = lane & 15, n = n0 + 4 * (lane >> 4);
  if (t >= a.T) return;
  if (router) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < N) a.logits[(long long)t * N + n + r] = v[r];
  } else {
    store_planes(a.z + (long long)t * a.L * 3, n, v);
  }
}

struct TopkLds {
  uint32_t key[64 * SLOTS];
  float sg[64 * SLOTS];
  int sel[32];
  float s[32];
  uint32_t kl[32];
};

// one token's selection, by the whole work-group
MOE_DEV void topk_item(const FewArgs &a, int t, TopkLds &l) {
  for (int e = threadIdx.x; e < 64 * SLOTS; e += FTHR) {
    uint32_t key = 0u;  // slots past E: below every real expert
    float sg = 0.f;
    if (e < a.E) {
      sg = sigmoid(a.logits[(long long)t * a.E + e]);
      float b = sg + a.bias[e];
      if (b != b) b = -INFINITY;
      key = order_key(b);
    }
    l.key[e] = key;
    l.sg[e] = sg;
  }
  __syncthreads();
  const int lane = lane_id();
  if (threadIdx.x < 64) {
    uint32_t key[SLOTS];
    float sg[SLOTS];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      key[i] = l.key[lane + 64 * i];
      sg[i] = l.sg[lane + 64 * i];
    }
    uint32_t th, kp1;
    select_topk(key, sg, a.k, lane, l.sel, l.s, l.kl, th, kp1);
  }
  __syncthreads();
  if (threadIdx.x >= 64) return;
  write_topk(t, a.k, lane, l.sel, l.s, l.kl, nullptr, 0, a.ids, a.wts);
  if (a.topk_ids != nullptr) write_topk(t, a.k, lane, l.sel, l.s, l.kl, nullptr, 0, a.topk_ids, a.topk_w);
  release();
  int last = 0;
  if (lane == 0) last = add_count(a.counters + C_TOPK) == a.T - 1;
  if (!__builtin_amdgcn_readfirstlane(last)) return;
  // the last token's wave makes the list of experts, each at its first pair
  acquire();
  const int P = a.T * a.k;
  int base = 0;
  for (int p0 = 0; p0 < P; p0 += 64) {
    const int p = p0 + lane;
    int e = -1;
    bool first = p < P;
    if (first) {
      e = a.ids[p];
      for (int q = 0; q < p / a.k * a.k; ++q) first &= a.ids[q] != e;
    }
    const uint64_t m = __ballot(first);
    if (first) {
      const int slot = base + lanes_below(m);
      a.list->expert[slot] = e;
      int n = 0;
      for (int q = p; q < P; ++q)
        if (a.ids[q] == e) a.list->pair[slot][n++] = q;
      a.list->npair[slot] = n;
    }
    base += __popcll(m);
  }
  if (lane == 0) a.list->n = base;
  release();
  if (lane == 0) add_count(a.counters + C_READY);
}

// until *p reaches n; the whole work-group, whose waves then see what was counted
MOE_DEV void wait_for(const int32_t *p, int n) {
  if (threadIdx.x == 0)
    while (load_count(p) < n) __builtin_amdgcn_s_sleep(1);
  __syncthreads();
  acquire();
}

__global__ __launch_bounds__(FTHR, 4) void few_layer_kernel(FewArgs a) {
  __shared__ union {
    f32x4_t part[2][FW][MT_DN][64];
    TopkLds topk;
  } lds;
  __shared__ int next_ticket[2];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id();
  const int col = lane & 15, rg = lane >> 4;
  const int T = a.T, H = a.H, L = a.L, I = a.I, S = a.S;
  const int P = T * a.k;
  int32_t *cnt = a.counters;
  const int n_sgu = S / 16, n_sdn = S > 0 ? H / 16 : 0;
  const int nb_gu = I / (16 * MT_GU), nb_dn = L / (16 * MT_DN), nb_cmb = (L + CMB - 1) / CMB;
  const int end_topk = T, end_sgu = end_topk + n_sgu;
  int end_egu = 0x7FFFFFFF, end_sdn = 0, end_edn = 0, end_cmb = 0, end = 0x7FFFFFFF;
  int n_active = 0;
  int seen = 0;  // steps whose results this work-group has waited for

  if (threadIdx.x == 0) next_ticket[0] = add_count(cnt + C_TICKET);
  __syncthreads();
  int par = 0;
  for (;;) {
    const int item = __builtin_amdgcn_readfirstlane(next_ticket[par]);
    // the next ticket, ready after this item's barrier
    if (threadIdx.x == 0) next_ticket[par ^ 1] = add_count(cnt + C_TICKET);
    if (item >= end_sgu && !(seen & 1)) {
      wait_for(cnt + C_READY, 1);
      seen |= 1;
      n_active = __builtin_amdgcn_readfirstlane(a.list->n);
      end_egu = end_sgu + n_active * nb_gu;
      end_sdn = end_egu + n_sdn;
      end_edn = end_sdn + n_active * nb_dn;
      end_cmb = end_edn + T * nb_cmb;
      end = end_cmb + H / 16;
    }
    if (item >= end) break;
    auto &part = lds.part[par];
    par ^= 1;

    if (item < end_topk) {
      topk_item(a, item, lds.topk);
      __syncthreads();  // the selection's LDS is the sums' too
      continue;
    }
    if (item < end_sgu) {
      const long long r0 = 16LL * (item - end_topk);
      const uint8_t *W[2] = {reinterpret_cast<const uint8_t *>(a.sh_gate + r0 * H),
                             reinterpret_cast<const uint8_t *>(a.sh_up + r0 * H)};
      const uint8_t *Sc[2] = {nullptr, nullptr};
      f32x4_t acc[2] = {};
      product<W_BF16, 2, 1>(acc, W, Sc, 16, H, cols_x(a.x, T, H), wave);
      part[wave][0][lane] = acc[0];
      part[wave][1][lane] = acc[1];
      __syncthreads();
      if (wave == 0) {
        const f32x4_t g = wave_sum(part, 0), u = wave_sum(part, 1);
        f32x4_t h;
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = situ_glu(g[r], u[r], a.beta, a.beta_lin);
        if (col < T) store_planes(a.hs + (long long)col * S * 3, (int)r0 + 4 * rg, h);
        done(cnt + C_SGU);
      }
      continue;
    }
    if (item < end_egu) {
      const int i = item - end_sgu, slot = i / nb_gu, r0 = (i - slot * nb_gu) * 16 * MT_GU;
      const long long e = a.list->expert[slot];
      const int np = a.list->npair[slot];
      int32_t tok[FEW_MAX_T];
#pragma unroll
      for (int j = 0; j < FEW_MAX_T; ++j) tok[j] = j < np ? a.list->pair[slot][j] / a.k : 0;
      const uint8_t *W[2 * MT_GU], *Sc[2 * MT_GU];
#pragma unroll
      for (int t = 0; t < 2 * MT_GU; ++t) {
        const long long row = e * I + r0 + 16 * (t % MT_GU);
        W[t] = (t < MT_GU ? a.w1 : a.w3) + row * (L / 2);
        Sc[t] = (t < MT_GU ? a.s1 : a.s3) + row * (L / 32);
      }
      f32x4_t acc[2 * MT_GU] = {};
      product<W_MXFP4, 2 * MT_GU, 2>(acc, W, Sc, 16, L, cols_planes(a.z, (uint32_t)T * L * 6u, L, np, tok), wave);
#pragma unroll
      for (int t = 0; t < 2 * MT_GU; ++t) part[wave][t][lane] = acc[t];
      __syncthreads();
      if (wave < MT_GU) {
        const f32x4_t g = plane_sum(wave_sum(part, wave)), u = plane_sum(wave_sum(part, wave + MT_GU));
        f32x4_t h;
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = situ_glu(g[r], u[r], a.beta, a.beta_lin);
        const int j = col / 3;
        if (col == 3 * j && j < np)
          store_planes(a.h + (long long)a.list->pair[slot][j] * I * 3, r0 + 16 * wave + 4 * rg, h);
        done(cnt + C_EGU);
      }
      continue;
    }
    if (item < end_sdn) {
      if (!(seen & 2)) wait_for(cnt + C_SGU, n_sgu);
      seen |= 2;
      const long long r0 = 16LL * (item - end_egu);
      const uint8_t *W[1] = {reinterpret_cast<const uint8_t *>(a.sh_down + r0 * S)};
      const uint8_t *Sc[1] = {nullptr};
      const int32_t tok[FEW_MAX_T] = {0, 1, 2, 3};
      f32x4_t acc[1] = {};
      product<W_BF16, 1, 2>(acc, W, Sc, 16, S, cols_planes(a.hs, (uint32_t)T * S * 6u, S, T, tok), wave);
      part[wave][0][lane] = acc[0];
      __syncthreads();
      if (wave == 0) {
        const f32x4_t v = plane_sum(wave_sum(part, 0));
        const int j = col / 3;
        if (col == 3 * j && j < T) *reinterpret_cast<f32x4_t *>(a.sd + (long long)j * H + r0 + 4 * rg) = v;
        done(cnt + C_SDN);
      }
      continue;
    }
    if (item < end_edn) {
      if (!(seen & 4)) wait_for(cnt + C_EGU, n_active * nb_gu * MT_GU);
      seen |= 4;
      const int i = item - end_sdn, slot = i / nb_dn, r0 = (i - slot * nb_dn) * 16 * MT_DN;
      const long long e = a.list->expert[slot];
      const int np = a.list->npair[slot];
      int32_t pair[FEW_MAX_T];
#pragma unroll
      for (int j = 0; j < FEW_MAX_T; ++j) pair[j] = j < np ? a.list->pair[slot][j] : 0;
      const uint8_t *W[MT_DN], *Sc[MT_DN];
#pragma unroll
      for (int t = 0; t < MT_DN; ++t) {
        const long long row = e * L + r0 + 16 * t;
        W[t] = a.w2 + row * (I / 2);
        Sc[t] = a.s2 + row * (I / 32);
      }
      f32x4_t acc[MT_DN] = {};
      product<W_MXFP4, MT_DN, 2>(acc, W, Sc, 16, I, cols_planes(a.h, (uint32_t)P * I * 6u, I, np, pair), wave);
#pragma unroll
      for (int t = 0; t < MT_DN; ++t) part[wave][t][lane] = acc[t];
      __syncthreads();
      if (wave < MT_DN) {
        const f32x4_t v = plane_sum(wave_sum(part, wave));
        const int j = col / 3;
        if (col == 3 * j && j < np)
          *reinterpret_cast<f32x4_t *>(a.y + (long long)a.list->pair[slot][j] * L + r0 + 16 * wave + 4 * rg) = v;
        done(cnt + C_EDN);
      }
      continue;
    }
    if (item < end_cmb) {
      if (!(seen & 8)) wait_for(cnt + C_EDN, n_active * nb_dn * MT_DN);
      seen |= 8;
      const int i = item - end_edn, t = i / nb_cmb, blk = i - t * nb_cmb;
      const int c = blk * CMB + 4 * lane;
      f32x4_t v = {0.f, 0.f, 0.f, 0.f};
      if (c < L)
        for (int j = wave; j < a.k; j += FW) {
          const int p = t * a.k + j;
          v += a.wts[p] * *reinterpret_cast<const f32x4_t *>(a.y + (long long)p * L + c);
        }
      part[wave][0][lane] = v;
      __syncthreads();
      if (wave == 0) {
        v = wave_sum(part, 0);
        float ss = v[0] * v[0] + v[1] * v[1] + v[2] * v[2] + v[3] * v[3];
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) ss += __shfl_xor(ss, d, 64);
        if (c < L) {
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] *= __uint_as_float((uint32_t)a.gamma[c + r] << 16);
          store_planes(a.yn + (long long)t * L * 3, c, v);
        }
        if (lane == 0) a.ss[t * nb_cmb + blk] = ss;
        done(cnt + C_CMB);
      }
      continue;
    }
    if (!(seen & 16)) {
      wait_for(cnt + C_CMB, T * nb_cmb);
      if (S > 0) wait_for(cnt + C_SDN, n_sdn);
    }
    seen |= 16;
    const long long r0 = 16LL * (item - end_cmb);
    const uint8_t *W[1] = {reinterpret_cast<const uint8_t *>(a.w_up + r0 * L)};
    const uint8_t *Sc[1] = {nullptr};
    const int32_t tok[FEW_MAX_T] = {0, 1, 2, 3};
    f32x4_t acc[1] = {};
    product<W_BF16, 1, 2>(acc, W, Sc, 16, L, cols_planes(a.yn, (uint32_t)T * L * 6u, L, T, tok), wave);
    part[wave][0][lane] = acc[0];
    __syncthreads();
    if (wave == 0) {
      f32x4_t v = plane_sum(wave_sum(part, 0));
      const int j = col / 3;
      if (col == 3 * j && j < T) {
        float ss = 0.f;
        for (int q = 0; q < nb_cmb; ++q) ss += a.ss[j * nb_cmb + q];
        v = v * (1.0f / sqrtf(ss / (float)L + a.eps));
        const long long o = (long long)j * H + r0 + 4 * rg;
        if (S > 0) v += *reinterpret_cast<const f32x4_t *>(a.sd + o);
        *reinterpret_cast<f32x4_t *>(a.out + o) = v;
      }
    }
  }
}

}  // namespace

static_assert(FEW_COUNTERS > C_CMB, "every counter is cleared");

hipError_t launch_few(const FewArgs &a, hipStream_t st) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= 64) return hipErrorInvalidDevice;
  static std::atomic<int> cus[64];
  int ncu = cus[dev].load();
  if (ncu == 0) {
    e = hipDeviceGetAttribute(&ncu, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    cus[dev].store(ncu);
  }
  hipLaunchKernelGGL(few_front_kernel, dim3((unsigned)((a.E + 15) / 16 + a.L / 16)), dim3(FTHR), 0, st, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(few_layer_kernel, dim3((unsigned)(2 * ncu)), dim3(FTHR), 0, st, a);
  return hipGetLastError();
}

}  // namespace moe
