// Selection of the k largest biased scores of a token, shared by the routing
// kernels and the few-token layer.  Order: larger biased score first, then the
// lower expert index; NaN ranks last.
#pragma once
#include <math.h>

#include "common.h"

namespace moe {

constexpr int SLOTS = 16;  // experts per lane: E <= 64 * SLOTS = 1024

// Order-preserving map of a biased score onto uint32 (larger score, larger
// key); -0 is folded onto +0 so the two compare equal, as floats do.
MOE_DEV uint32_t order_key(float b) {
  uint32_t u = __float_as_uint(b);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
MOE_DEV float key_value(uint32_t key) { return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key); }

MOE_DEV float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// lanes below this one with their bit set in m
MOE_DEV int lanes_below(uint64_t m) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}

// The k-th largest key of a wavefront's SLOTS x 64 keys and the selection
// (see above): the selected ids, scores and keys go to sel / s / kl in
// ascending id order; th is the k-th largest key, kp1 the (k+1)-th.
// GAP false: the search ends as soon as a candidate has exactly k keys at or
// above it; th is then that candidate and kp1 the largest key below it.
template <bool GAP = true>
MOE_DEV void select_topk(const uint32_t (&key)[SLOTS], const float (&sg)[SLOTS], int k, int lane, int *sel,
                         float *s, uint32_t *kl, uint32_t &th_out, uint32_t &kp1_out) {
  auto count_ge = [&](uint32_t c) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) n += __popcll(__ballot(key[i] >= c));
    return n;
  };
  uint32_t th = 0u;  // the largest c with at least k keys >= c: the k-th largest key
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t c = th | (1u << bit);
    const int n = count_ge(c);
    if (n >= k) th = c;
    if constexpr (!GAP)
      if (n == k) break;
  }
  int above = 0, at_or_above = 0;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    above += __popcll(__ballot(key[i] > th));
    at_or_above += __popcll(__ballot(key[i] >= th));
  }
  // (k+1)-th largest: th again if more keys equal it, else the largest key below it
  uint32_t below = 0u;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) below = max(below, key[i] < th ? key[i] : 0u);
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) below = max(below, (uint32_t)__shfl_xor((int)below, d, 64));
  kp1_out = at_or_above > k ? th : below;
  th_out = th;

  int need = k - above;  // keys equal to th that are selected, lowest indices first
  int pos = 0;
#pragma unroll
  for (int i = 0; i < SLOTS; ++i) {
    const uint64_t eq = __ballot(key[i] == th);
    const bool pick = key[i] > th || (key[i] == th && lanes_below(eq) < need);
    need -= min(__popcll(eq), max(need, 0));
    const uint64_t m = __ballot(pick);
    if (pick) {
      const int q = pos + lanes_below(m);
      sel[q] = lane + 64 * i;
      s[q] = sg[i];
      kl[q] = key[i];
    }
    pos += __popcll(m);
  }
}

// Weights of token t from its selection (after a barrier that makes the
// selection visible): the selected sigmoid scores over their sum, with the
// capped-promotion rule when a promoted mask is given.
MOE_DEV void write_topk(int t, int k, int lane, const int *sel, const float *s, const uint32_t *kl,
                        const uint8_t *promoted, int k_hi, int32_t *ids, float *w) {
  float sum = 0.f;
  for (int q = 0; q < k; ++q) sum += s[q];
  if (lane < k) {
    const int id = sel[lane];
    float wt = s[lane] / sum;
    if (promoted != nullptr && promoted[id]) {
      // capped promotion: a promoted expert with k_hi selected promoted experts
      // ahead of it in routing order (larger key, or equal key and lower id)
      // has its contribution dropped; the other weights stay as they are
      const uint32_t my = kl[lane];
      int ahead = 0;
      for (int q = 0; q < k; ++q) {
        const int o = sel[q];
        const uint32_t ok = kl[q];
        ahead += (promoted[o] && (ok > my || (ok == my && o < id))) ? 1 : 0;
      }
      if (ahead >= k_hi) wt = 0.f;
    }
    ids[(long long)t * k + lane] = id;
    w[(long long)t * k + lane] = wt;
  }
}

}  // namespace moe
