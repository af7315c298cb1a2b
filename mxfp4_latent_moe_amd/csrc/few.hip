// The whole layer for a few tokens (T <= 4) in six kernels on one stream.
//
// At these sizes every weight of the layer that the tokens touch is read once
// and used for at most four tokens, so the layer is one weight stream of the
// router, the latent projections, the shared experts and the chosen experts,
// and what costs time beside it are the places where the stream stops.  Steps
// that need nothing from each other share a launch:
//
//   few_front_kernel   logits = x W_r^T | z = x W_d^T
//   few_shared_kernel  top-k and the list of chosen experts (one work-group) |
//                      shared gate/up, which hides it
//   few_expert<gate/up>
//   few_expert<down>   expert down | shared down, which fills its last wave
//   few_combine_kernel sum over a token's experts, times gamma; squares' sums
//   few_up_kernel      up_proj, times RMSNorm's factor, plus the shared experts
//
// Arithmetic: weight rows on the MFMA's M side, on its N side up to 12 columns.
// x is exact in bf16.  z, the hidden activations and the normed latent are kept
// as three bf16 planes (a = a1 + a2 + a3, exact for normal fp32), three columns
// per token, so every product is that of the fp32 value with the exact weight;
// sums are fp32.  The columns cost nothing: the kernel waits for weights.
// RMSNorm's factor is one number per token and is applied to up_proj's sums.
// Every sum has one order, so results do not depend on the schedule.
//
// Measured (hidden 7168, latent 3584, 16 of 896 experts of 3072, 6144 shared):
// 157 us for one token, 224 for two, 303 to 315 for four, 4.2 to 4.8 TB/s of the
// bytes the layer cannot do without; the layer's calls one by one take 181, 230
// and 318.  Of the 157 us about 4 a kernel are the launch and its cold code, and
// some more go to work-groups that do not divide over the CUs: of gate/up's 384
// half of the CUs have two and the others one (48 us, 3.9 TB/s; at four tokens,
// with some 61 distinct experts, 5.2).  One resident kernel that hands work items
// from step to step by counters in place of launches took 177, 247 and 350 us:
// its waves could not keep the weights flowing through the steps' ends.
// Requests further ahead are no faster: two groups of K steps ahead in the
// expert products 50 against 46 us at one token (one work-group a CU fits), and
// in the bf16 products four steps a round 58 against 38.
#include <algorithm>
#include <atomic>

#include "kernels.h"
#include "topk.h"

namespace moe {
namespace {

constexpr int FNW = 8;           // waves of a work-group
constexpr int FTHR = 64 * FNW;
constexpr int SU = 3;            // K steps a round of the shared gate/up
constexpr int CMB = 256;         // columns of a combine work-group
constexpr int AHEAD = 1;         // groups of K steps requested ahead, of
constexpr int D = 4;             // K steps (128 values) each
constexpr int ROWS = 16 * FNW;   // weight rows of an expert item whose waves split the rows

MOE_DEV int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

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

// the N-side operand of a dense product: its rows, and the lane's column
struct Cols {
  const void *base;
  uint32_t bytes;
  uint32_t off;      // of the lane's column
  uint32_t ostride;  // bytes between octets
};
// columns that are rows of x: column c is token c
MOE_DEV Cols cols_x(const uint16_t *x, int T, int H) {
  return Cols{x, (uint32_t)T * H * 2, (uint32_t)min(lane_id() & 15, T - 1) * H * 2, 16};
}
// columns of rows kept in planes: column 3 t + p is plane p of row t
MOE_DEV Cols cols_planes(const uint16_t *x, int T, int K) {
  const int c = min(lane_id() & 15, 3 * T - 1), t = c / 3;
  return Cols{x, (uint32_t)T * K * 6, (uint32_t)t * K * 6 + 16 * (c - 3 * t), 48};
}

// 16 rows of bf16 weights (the last of nrows again past them) times the
// columns: this wave's share of the K steps, every FNW-th, one requested ahead.
// Steps past the end are out of the buffers' range: zeros.
MOE_DEV f32x4_t dense_part(const uint16_t *W, int nrows, int K, const Cols &b, int wave) {
  const int lane = lane_id(), kg = lane >> 4;
  const int nks = K / 128;
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(W, nrows * 2u * K), br = make_rsrc(b.base, b.bytes);
  const uint32_t wo = min(lane & 15, nrows - 1) * 2u * K + 16 * kg, bo = b.off + kg * b.ostride;
  u32x4_t q[2][4], x[2][4];
  auto request = [&](int slot, int s) {
    const uint32_t ws = s < nks ? s * 256 : 0x70000000u, xs = s < nks ? s * 16 * b.ostride : 0x70000000u;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[slot][j] = buf_load16(wr, wo + 64 * j, ws);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[slot][j] = buf_load16(br, bo + 4 * j * b.ostride, xs);
  };
  request(0, wave);
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = wave; s < nks; s += 2 * FNW) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      request(i ^ 1, s + FNW * (i + 1));
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc = mfma_16x16x32(__builtin_bit_cast(bf16x8_t, q[i][j]), __builtin_bit_cast(bf16x8_t, x[i][j]), acc);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  return acc;
}
// the waves' sums, in wave order
MOE_DEV f32x4_t wave_sum(const f32x4_t (*part)[64]) {
  f32x4_t v = part[0][lane_id()];
#pragma unroll
  for (int i = 1; i < FNW; ++i) v += part[i][lane_id()];
  return v;
}
// the whole work-group's product; true in the wave that has it
MOE_DEV bool dense_tile(f32x4_t &v, const uint16_t *W, int nrows, int K, const Cols &b, f32x4_t (*part)[64]) {
  const int wave = uni(threadIdx.x >> 6);
  part[wave][lane_id()] = dense_part(W, nrows, K, b, wave);
  __syncthreads();
  if (wave != 0) return false;
  v = wave_sum(part);
  return true;
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
  __shared__ f32x4_t part[FNW][64];
  const int lane = lane_id();
  const int nb_r = (a.E + 15) / 16;
  const bool router = (int)blockIdx.x < nb_r;
  const int n0 = 16 * (router ? blockIdx.x : blockIdx.x - nb_r);
  const int N = router ? a.E : a.L;
  f32x4_t v;
  if (!dense_tile(v, (router ? a.w_router : a.w_down) + (long long)n0 * a.H, min(16, N - n0), a.H,
                     cols_x(a.x, a.T, a.H), part))
    return;
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
  int sel[FEW_MAX_T][32];
  float s[FEW_MAX_T][32];
  uint32_t kl[FEW_MAX_T][32];
};

// The selection, a wave per token, and the list of chosen experts: each with
// the pairs that use it, FEW_ROWS pairs an entry.  An expert's entries follow
// one another.
MOE_DEV void topk_group(const FewArgs &a, TopkLds &l) {
  const int t = uni(threadIdx.x >> 6), lane = lane_id();
  if (t < a.T) {
    uint32_t key[SLOTS];  // 0 for slots past E: below every real expert
    float sg[SLOTS], lg[SLOTS], bi[SLOTS];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      const int e = min(lane + 64 * i, a.E - 1);
      lg[i] = a.logits[(long long)t * a.E + e];
      bi[i] = a.bias[e];
    }
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      sg[i] = sigmoid(lg[i]);
      float b = sg[i] + bi[i];
      if (b != b) b = -INFINITY;
      key[i] = lane + 64 * i < a.E ? order_key(b) : 0u;
    }
    uint32_t th, kp1;
    select_topk<false>(key, sg, a.k, lane, l.sel[t], l.s[t], l.kl[t], th, kp1);
  }
  __syncthreads();
  if (t < a.T && lane < a.k) {
    float sum = 0.f;
    for (int q = 0; q < a.k; ++q) sum += l.s[t][q];
    const int p = t * a.k + lane;
    const float w = l.s[t][lane] / sum;
    a.wts[p] = w;
    if (a.topk_ids != nullptr) {
      a.topk_ids[p] = l.sel[t][lane];
      a.topk_w[p] = w;
    }
  }
  if (t != 0) return;
  const int P = a.T * a.k;
  int base = 0;
  for (int p0 = 0; p0 < P; p0 += 64) {
    const int p = p0 + lane, t0 = min(p, P - 1) / a.k;
    const int e = l.sel[t0][min(p, P - 1) - t0 * a.k];
    bool first = p < P;
    int n = 0, pair[FEW_MAX_T];
    // a token's ids differ, so each other token holds e once at most
    for (int t1 = 0; t1 < a.T; ++t1)
      for (int q = 0; q < a.k; ++q)
        if (l.sel[t1][q] == e) {
          if (t1 < t0) first = false;
#pragma unroll
          for (int i = 0; i < FEW_MAX_T; ++i)
            if (i == n) pair[i] = t1 * a.k + q;
          ++n;
        }
    // one entry or two
    const uint64_t m1 = __ballot(first), m2 = __ballot(first && n > FEW_ROWS);
    if (first) {
      const int slot = base + lanes_below(m1) + lanes_below(m2);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int left = n - FEW_ROWS * h;
        if (left <= 0) continue;
        FewEntry &en = a.list->entry[slot + h];
        en.expert = e;
        en.npair = min(left, FEW_ROWS);
#pragma unroll
        for (int i = 0; i < FEW_ROWS; ++i)
          if (i < left) en.pair[i] = pair[FEW_ROWS * h + i];
      }
    }
    base += __popcll(m1) + __popcll(m2);
  }
  if (lane == 0) a.list->n = base;
}

// ---- top-k; shared gate/up, eight rows of both matrices a work-group
__global__ __launch_bounds__(FTHR, 4) void few_shared_kernel(FewArgs a) {
  __shared__ union {
    f32x4_t part[FNW][64];
    TopkLds topk;
  } l;
  if (blockIdx.x == 0) {
    topk_group(a, l.topk);
    return;
  }
  const int wave = uni(threadIdx.x >> 6), lane = lane_id(), kg = lane >> 4, r16 = lane & 15;
  const int r0 = 8 * (blockIdx.x - 1), nks = a.H / 128;
  const char *const w = reinterpret_cast<const char *>((r16 < 8 ? a.sh_gate : a.sh_up) + (long long)(r0 + (r16 & 7)) * a.H);
  const char *const x = reinterpret_cast<const char *>(a.x + (long long)min(r16, a.T - 1) * a.H);
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int s0 = wave; s0 < nks; s0 += FNW * SU) {
    u32x4_t q[SU][4], c[SU][4];
#pragma unroll
    for (int u = 0; u < SU; ++u) {
#pragma unroll
      for (int j = 0; j < 4; ++j) q[u][j] = c[u][j] = u32x4_t{0u, 0u, 0u, 0u};
      const int s = s0 + FNW * u;
      if (s < nks) {
        const uint32_t o = s * 256 + 16 * kg;
#pragma unroll
        for (int j = 0; j < 4; ++j) q[u][j] = *reinterpret_cast<const u32x4_t *>(w + o + 64 * j);
#pragma unroll
        for (int j = 0; j < 4; ++j) c[u][j] = *reinterpret_cast<const u32x4_t *>(x + o + 64 * j);
      }
    }
    __builtin_amdgcn_sched_barrier(0);  // every load of the round is on its way before the first product
#pragma unroll
    for (int u = 0; u < SU; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc = mfma_16x16x32(__builtin_bit_cast(bf16x8_t, q[u][j]), __builtin_bit_cast(bf16x8_t, c[u][j]), acc);
  }
  l.part[wave][lane] = acc;
  __syncthreads();
  if (wave != 0) return;
  const f32x4_t v = wave_sum(l.part);
  f32x4_t h;  // rows 4 kg ..: the first half of the wave has gate's sums, the second up's
#pragma unroll
  for (int r = 0; r < 4; ++r) h[r] = situ_glu(v[r], __shfl_down(v[r], 32, 64), a.beta, a.beta_lin);
  if (lane < 32 && r16 < a.T) store_planes(a.hs + (long long)r16 * a.S * 3, r0 + 4 * kg, h);
}

// ---- expert products
// An item is 128 weight rows (of both matrices for gate/up), 16 a wave, of a
// list entry; a work-group has a contiguous range of the items.  Each wave
// streams its rows over the whole of K, four K steps (256 contiguous bytes a
// row) a group, one group ahead, across items; the entry's columns sit in LDS
// and are staged when the entry changes.  KSPLIT: an item is 16 rows, the waves
// take the groups of K by turns and their sums are added in wave order: where
// there are few items, a wave's groups one after the other are what takes time
// (two experts of 256 x 3328: gate/up 8.8 us, 20.2 without).
template <bool PAIR, bool KSPLIT>
MOE_DEV void expert_items(const FewArgs &a, u32x4_t *lds, f32x4_t (*part)[2][64], int group, int groups) {
  constexpr int IROWS = KSPLIT ? 16 : ROWS, KS = KSPLIT ? FNW : 1;
  constexpr int NM = PAIR ? 2 : 1;
  const int wave = uni(threadIdx.x >> 6), lane = lane_id(), kg = lane >> 4, r16 = lane & 15;
  const int N = PAIR ? a.I : a.L, K = PAIR ? a.L : a.I;
  const int nks = K / 128, ng = (nks + D - 1) / D, nb = N / IROWS;
  const int wrow = KSPLIT ? 0 : 16 * wave, ks = KSPLIT ? wave : 0;  // the wave's rows of an item, its first group
  const int ngw = (ng + KS - 1) / KS;
  const int nc = 3 * min(a.T, FEW_ROWS);
  const uint32_t row_bytes = K / 2, srow_bytes = K / 32;
  // read through the constant address space: the scalar unit's reads stay off
  // the counter that paces the weight ring
  typedef __attribute__((address_space(4))) const int32_t const_i32;
  const_i32 *list = (const_i32 *)a.list;
  constexpr int ENTRY = sizeof(FewEntry) / 4;
  const int n_items = list[0] * nb;
  const int i_begin = (int)((long long)group * n_items / groups);
  const int i_end = (int)((long long)(group + 1) * n_items / groups);
  if (i_begin >= i_end) return;

  int l_item = i_begin, l_g = 0;
  __amdgpu_buffer_rsrc_t wr[NM], sr[NM];
  uint32_t wo = 0, so = 0;
  auto set_load_item = [&](int it) {
    const int c = uni(it / nb);
    const long long e = list[1 + ENTRY * c];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      wr[m] = make_rsrc((PAIR ? (m ? a.w3 : a.w1) : a.w2) + e * N * row_bytes, (uint32_t)N * row_bytes);
      sr[m] = make_rsrc((PAIR ? (m ? a.s3 : a.s1) : a.s2) + e * N * srow_bytes, (uint32_t)N * srow_bytes);
    }
    const uint32_t n = (it - c * nb) * IROWS + wrow + r16;
    wo = n * row_bytes + kg * 16;
    so = n * srow_bytes;
  };
  set_load_item(i_begin);
  u32x4_t wq[AHEAD + 1][D][NM], sq[AHEAD + 1][NM];
  // Past the last item the requests go on, all to one line, so that the count
  // of loads in flight stays the same.  A last group that is not whole reads
  // on into the next row (codes are finite; their columns are zeros).
  auto load_group = [&](int bi) {
    const bool live = l_item < i_end;
    const uint32_t w0 = live ? wo : 0u, s0 = live ? so : 0u, q0 = live ? min(ks + KS * l_g, ng - 1) * D : 0u;
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int m = 0; m < NM; ++m) wq[bi][d][m] = buf_load16(wr[m], w0, (q0 + d) * 64u);
#pragma unroll
    for (int m = 0; m < NM; ++m) sq[bi][m] = buf_load16(sr[m], s0, q0 * 4u);
    if (++l_g == ngw) {
      l_g = 0;
      if (++l_item < i_end) set_load_item(l_item);
    }
  };
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) load_group(i);

  // columns of K steps past the end are zeros
  for (int i = 16 * nks * nc + threadIdx.x; i < 16 * D * ng * nc; i += FTHR) lds[i] = u32x4_t{0u, 0u, 0u, 0u};
  int staged = -1, npair = 0, pair0 = 0, pair1 = 0;
  const u32x4_t *const src = reinterpret_cast<const u32x4_t *>(PAIR ? a.z : a.h);
  auto stage = [&](int c) {
    if (c == staged) return;
    npair = uni(list[1 + ENTRY * c + 1]);
    pair0 = uni(list[1 + ENTRY * c + 2]);
    pair1 = npair > 1 ? uni(list[1 + ENTRY * c + 3]) : pair0;
    __syncthreads();  // every wave is done with the previous entry's columns
    const int pieces = K / 8 * 3;
    const u32x4_t *const row0 = src + (long long)(PAIR ? pair0 / a.k : pair0) * pieces;
    const u32x4_t *const row1 = src + (long long)(PAIR ? pair1 / a.k : pair1) * pieces;
    constexpr int B = 3;  // pieces of a row that a thread requests at once
    for (int i0 = threadIdx.x; i0 < pieces; i0 += B * FTHR) {
      u32x4_t v[2][B];
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const int i = min(i0 + FTHR * u, pieces - 1);
        v[0][u] = row0[i];
        v[1][u] = row1[i];
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const int i = min(i0 + FTHR * u, pieces - 1);
        u32x4_t *const to = lds + i / 3 * nc + i % 3;
        to[0] = v[0][u];
        if (npair > 1) to[3] = v[1][u];
      }
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // nothing of this is counted against the ring
    __syncthreads();
    staged = c;
  };
  const u32x4_t *const col = lds + kg * 4 * nc + min(r16, nc - 1);

  int item = i_begin, c = uni(item / nb), g = 0;
  stage(c);
  f32x4_t acc[NM];
#pragma unroll
  for (int m = 0; m < NM; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto finish = [&]() {
    if constexpr (KSPLIT) {
      __syncthreads();  // the sums of the item before have been read
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        part[wave][m][lane] = acc[m];
        acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      }
      __syncthreads();
      if (wave != 0) return;
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        acc[m] = part[0][m][lane];
#pragma unroll
        for (int q = 1; q < FNW; ++q) acc[m] += part[q][m][lane];
      }
    }
    const int n0 = (item - c * nb) * IROWS + wrow + 4 * kg, j = r16 / 3;
    f32x4_t v = plane_sum(acc[0]);
    if constexpr (PAIR) {
      const f32x4_t u = plane_sum(acc[NM - 1]);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = situ_glu(v[r], u[r], a.beta, a.beta_lin);
    }
    if (r16 == 3 * j && j < npair) {
      const int p = j == 0 ? pair0 : pair1;
      if constexpr (PAIR) store_planes(a.h + (long long)p * N * 3, n0, v);
      else *reinterpret_cast<f32x4_t *>(a.y + (long long)p * N + n0) = v;
    }
#pragma unroll
    for (int m = 0; m < NM; ++m) acc[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  };
  // the groups of the work-group's items, a ring's turn an iteration; groups
  // past the last one are multiplied and dropped
  for (int left = (i_end - i_begin) * ngw; left > 0; left -= AHEAD + 1) {
#pragma unroll
    for (int b = 0; b <= AHEAD; ++b) {
      load_group((b + AHEAD) % (AHEAD + 1));
      __builtin_amdgcn_sched_barrier(0);
      const int gg = ks + KS * g;
      if (!KSPLIT || gg < ng) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
          float sc[NM];
#pragma unroll
          for (int m = 0; m < NM; ++m)
            sc[m] = gg * D + d < nks ? e8m0_to_float((sq[b][m][d] >> (8 * kg)) & 0xFFu) : 1.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bf16x8_t x = __builtin_bit_cast(bf16x8_t, col[(16 * (gg * D + d) + j) * nc]);
#pragma unroll
            for (int m = 0; m < NM; ++m) acc[m] = mfma_16x16x32(fp4x8_to_bf16(wq[b][d][m][j], sc[m]), x, acc[m]);
          }
        }
      }
      if (++g == ngw) {
        g = 0;
        if (item < i_end) {
          finish();
          if (++item < i_end) {
            c = uni(item / nb);
            stage(c);
          }
        }
      }
    }
  }
}

// gate/up; down with the shared experts' down products behind it
template <bool PAIR, bool KSPLIT>
__global__ __launch_bounds__(FTHR, 2) void few_expert_kernel(FewArgs a, int groups) {
  extern __shared__ u32x4_t lds[];
  __shared__ f32x4_t part[KSPLIT ? FNW : 1][2][64];
  if ((int)blockIdx.x < groups) {
    expert_items<PAIR, KSPLIT>(a, lds, part, blockIdx.x, groups);
    return;
  }
  if constexpr (!PAIR) {
    const int lane = lane_id(), n0 = 16 * (blockIdx.x - groups);
    f32x4_t v;
    if (!dense_tile(v, a.sh_down + (long long)n0 * a.S, 16, a.S, cols_planes(a.hs, a.T, a.S),
                       reinterpret_cast<f32x4_t(*)[64]>(lds)))
      return;
    v = plane_sum(v);
    const int col = lane & 15, t = col / 3;
    if (col == 3 * t && t < a.T)
      *reinterpret_cast<f32x4_t *>(a.sd + (long long)t * a.H + n0 + 4 * (lane >> 4)) = v;
  }
}

// ---- 256 columns of a token's combined latent, times gamma, and their squares' sum
__global__ __launch_bounds__(64) void few_combine_kernel(FewArgs a) {
  const int lane = lane_id(), L = a.L;
  const int t = blockIdx.y, c = blockIdx.x * CMB + 4 * lane;
  const float wt = lane < a.k ? a.wts[t * a.k + lane] : 0.f;
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  for (int q0 = 0; q0 < a.k; q0 += 16) {
    f32x4_t y[16];  // all requested at once; past the last slot that one again, unused
#pragma unroll
    for (int q = 0; q < 16; ++q)
      y[q] = *reinterpret_cast<const f32x4_t *>(a.y + (long long)(t * a.k + min(q0 + q, a.k - 1)) * L + min(c, L - 4));
#pragma unroll
    for (int q = 0; q < 16; ++q)
      if (q0 + q < a.k) v += __shfl(wt, q0 + q, 64) * y[q];
  }
  if (c >= L) v = f32x4_t{0.f, 0.f, 0.f, 0.f};
  float ss = v[0] * v[0] + v[1] * v[1] + v[2] * v[2] + v[3] * v[3];
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) ss += __shfl_xor(ss, d, 64);
  if (c < L) {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] *= __uint_as_float((uint32_t)a.gamma[c + r] << 16);
    store_planes(a.yn + (long long)t * L * 3, c, v);
  }
  if (lane == 0) a.ss[t * gridDim.x + blockIdx.x] = ss;
}

// ---- up_proj, 16 rows a work-group
__global__ __launch_bounds__(FTHR, 4) void few_up_kernel(FewArgs a, int nb_cmb) {
  __shared__ f32x4_t part[FNW][64];
  const int lane = lane_id(), n0 = 16 * blockIdx.x;
  f32x4_t v;
  if (!dense_tile(v, a.w_up + (long long)n0 * a.L, 16, a.L, cols_planes(a.yn, a.T, a.L), part)) return;
  v = plane_sum(v);
  const int col = lane & 15, t = col / 3;
  if (col != 3 * t || t >= a.T) return;
  float ss = 0.f;
  for (int q = 0; q < nb_cmb; ++q) ss += a.ss[t * nb_cmb + q];
  v = v * (1.0f / sqrtf(ss / (float)a.L + a.eps));
  const long long o = (long long)t * a.H + n0 + 4 * (lane >> 4);
  if (a.S > 0) v += *reinterpret_cast<const f32x4_t *>(a.sd + o);
  *reinterpret_cast<f32x4_t *>(a.out + o) = v;
}

}  // namespace

// LDS of an expert kernel's columns, and of the shared experts' sums beside it
static size_t columns_bytes(int T, int K) {
  const int ng = (K / 128 + D - 1) / D;
  const size_t b = (size_t)3 * (T < FEW_ROWS ? T : FEW_ROWS) * ng * D * 256;
  return b > FNW * 64 * 16 ? b : FNW * 64 * 16;
}

// An expert kernel: K split over the waves where the items of 128 rows are fewer
// than half of the CUs, by a rule without T, so that a token's result does not
// depend on its company; K is long; and there is room for the sums.  Measured
// with / without: gate/up of K = 3328 8.8 / 20.2 us, 2944 12.8 / 20.4, 2048 8.5 /
// 15.5; down (one matrix a wave) of 1792 8.9 / 8.2, of 256 6.1 / 5.4.  Two
// work-groups a CU where their columns fit, and no more than there can be items;
// `more` follow.
template <bool PAIR>
static hipError_t launch_expert(const FewArgs &a, int ncu, int N, int K, int more, hipStream_t st) {
  const size_t lds = columns_bytes(a.T, K);
  const int items = a.k * (N / ROWS);  // of a token
  const bool split = FEW_MAX_T * items < ncu / 2 && K >= (PAIR ? 2048 : 2560) && columns_bytes(FEW_MAX_T, K) <= 128 * 1024;
  const int groups = std::min(ncu * (lds <= 60 * 1024 ? 2 : 1), a.T * items * (split ? FNW : 1));
  auto *fn = split ? &few_expert_kernel<PAIR, true> : &few_expert_kernel<PAIR, false>;
  if (lds > 60 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(fn), hipFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(fn, dim3((unsigned)(groups + more)), dim3(FTHR), lds, st, a, groups);
  return hipGetLastError();
}

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
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(few_shared_kernel, dim3((unsigned)(1 + a.S / 8)), dim3(FTHR), 0, st, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if ((e = launch_expert<true>(a, ncu, a.I, a.L, 0, st)) != hipSuccess) return e;
  if ((e = launch_expert<false>(a, ncu, a.L, a.I, a.S > 0 ? a.H / 16 : 0, st)) != hipSuccess) return e;
  const int nb = (a.L + CMB - 1) / CMB;
  hipLaunchKernelGGL(few_combine_kernel, dim3((unsigned)nb, (unsigned)a.T), dim3(64), 0, st, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(few_up_kernel, dim3((unsigned)(a.H / 16)), dim3(FTHR), 0, st, a, nb);
  return hipGetLastError();
}

}  // namespace moe
