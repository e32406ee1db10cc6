// route_decide.cuh -- one token's routing decision by one warp: scoring, group-limited top-k with
// certification, the full ranking, and the gates (definitions in router.cu). Lane l holds the
// logits of experts l, l + 32, ... (EPL = E / 32 per lane, rounded up).
#pragma once

#include <float.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

struct VE {
  double v;
  int e;
};

// Order-preserving key of a double: a larger value has a larger key. -0 is taken as +0 first, so
// that the two have one key as they compare equal.
__device__ __forceinline__ unsigned long long order_key(double v) {
  const unsigned long long b = (unsigned long long)__double_as_longlong(v + 0.0);
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// The value of an order key (-0 comes back as +0).
__device__ __forceinline__ double key_value(unsigned long long key) {
  return __longlong_as_double((long long)((key >> 63) ? (key & 0x7FFFFFFFFFFFFFFFull) : ~key));
}

// Largest value of the warp (two warp reductions over its order key, then the value itself).
__device__ __forceinline__ double warp_max(double v) {
  const unsigned long long key = order_key(v);
  const unsigned hi = (unsigned)(key >> 32), lo = (unsigned)key;
  const unsigned best_hi = __reduce_max_sync(kFull, hi);
  const unsigned best_lo = __reduce_max_sync(kFull, hi == best_hi ? lo : 0u);
  const int src = __ffs(__ballot_sync(kFull, hi == best_hi && lo == best_lo)) - 1;
  return __shfl_sync(kFull, v, src);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}

__device__ __forceinline__ double sigmoid_d(double z) { return 1.0 / (1.0 + exp(-z)); }

// sqrt(softplus(z)) ("sqrtsoftplus", page "15. DeepSeek: MLA, MoE and MTP", section V4).
__device__ __forceinline__ double sqrtsoftplus_d(double z) { return sqrt(fmax(z, 0.0) + log1p(exp(-fabs(z)))); }

// Raw score of the routers that add a selection bias.
__device__ __forceinline__ double raw_score(int score_fn, double z) {
  return score_fn == MOE_SCORE_SQRTSOFTPLUS ? sqrtsoftplus_d(z) : sigmoid_d(z);
}

template <int EPL>
__device__ __forceinline__ double pick(const double (&r)[EPL], int j) {
  double out = 0.0;
#pragma unroll
  for (int i = 0; i < EPL; ++i)
    if (i == j) out = r[i];
  return out;
}

// Selection values: softmax ranks the logits; sigmoid ranks s + bias.
template <int EPL>
__device__ __forceinline__ void selection_values(const RouteArgs& a, const double (&l)[EPL], double (&v)[EPL],
                                                 bool (&valid)[EPL]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 32 * j;
    valid[j] = e < a.E;
    if (valid[j])
      v[j] = a.score_fn != MOE_SCORE_SOFTMAX ? raw_score(a.score_fn, l[j]) + (a.bias ? (double)a.bias[e] : 0.0) : l[j];
    else
      v[j] = -INFINITY;
  }
}

// Group limit with per-expert uncertainty (bit j of `exact`: value is binary64;
// otherwise it may be off by delta_v). Sets *elig (bits over j) to the experts
// of the kept groups. Returns false when the group cut is not certain, with the
// inexact experts that could decide it in *mark. An expert can be in its group's
// true top two only if v >= (second largest v) - 2 delta_v; once all of those
// are exact the group score is exact.
template <int EPL>
__device__ bool decide_groups_32(const RouteArgs& a, const double (&v)[EPL], const bool (&valid)[EPL], uint32_t exact,
                                 double delta_v, uint32_t* elig, uint32_t* mark, unsigned long long* keys);

template <int EPL>
__device__ bool decide_groups(const RouteArgs& a, const double (&v)[EPL], const bool (&valid)[EPL], uint32_t exact,
                              double delta_v, uint32_t* elig, uint32_t* mark, unsigned long long* keys) {
  const int lane = threadIdx.x & 31;
  const int per = a.E / a.G;
  // groups of 32 experts, one per lane slot: every group's reduction at once (below)
  if (per == 32 && a.G == EPL) return decide_groups_32<EPL>(a, v, valid, exact, delta_v, elig, mark, keys);
  double gs[kMaxGroups], gu[kMaxGroups], t2s[kMaxGroups];
  for (int g = 0; g < a.G; ++g) {
    double t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = lane + 32 * j;
      if (valid[j] && e / per == g) {
        if (v[j] > t1) {
          t2 = t1;
          t1 = v[j];
        } else if (v[j] > t2) {
          t2 = v[j];
        }
      }
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      const double o1 = __shfl_xor_sync(kFull, t1, off);
      const double o2 = __shfl_xor_sync(kFull, t2, off);
      const double hi = fmax(t1, o1);
      const double lo = fmax(fmin(t1, o1), fmax(t2, o2));
      t1 = hi;
      t2 = lo;
    }
    bool inexact_cand = false;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = lane + 32 * j;
      if (valid[j] && e / per == g && !((exact >> j) & 1u) && v[j] >= t2 - 2.0 * delta_v) inexact_cand = true;
    }
    gs[g] = t1 + t2;
    gu[g] = __any_sync(kFull, inexact_cand) ? 2.0 * delta_v : 0.0;
    t2s[g] = t2;
  }
  uint32_t keep = 0;
  double min_kept = INFINITY, max_drop = -INFINITY;
  for (int g = 0; g < a.G; ++g) {
    int better = 0;
    for (int h = 0; h < a.G; ++h) better += (gs[h] > gs[g]) || (gs[h] == gs[g] && h < g);
    if (better < a.topk_group) {
      keep |= 1u << g;
      min_kept = fmin(min_kept, gs[g] - gu[g]);
    } else {
      max_drop = fmax(max_drop, gs[g] + gu[g]);
    }
  }
  bool ok = true;
  uint32_t m = 0;
  if (a.topk_group < a.G && !(min_kept > max_drop)) {
    uint32_t involved = 0;
    for (int g = 0; g < a.G; ++g) {
      const bool kept = (keep >> g) & 1u;
      if (gu[g] > 0.0 && (kept ? gs[g] - gu[g] <= max_drop : gs[g] + gu[g] >= min_kept)) involved |= 1u << g;
    }
    if (involved) {
      ok = false;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int e = lane + 32 * j;
        if (valid[j] && ((involved >> (e / per)) & 1u) && !((exact >> j) & 1u) && v[j] >= t2s[e / per] - 2.0 * delta_v)
          m |= 1u << j;
      }
    }
  }
  uint32_t el = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 32 * j;
    if (valid[j] && ((keep >> (e / per)) & 1u)) el |= 1u << j;
  }
  *elig = el;
  *mark = m;
  return ok;
}

// decide_groups for groups of exactly 32 experts with G = EPL: lane slot j of every lane holds
// expert lane + 32 j, which is in group j, so the two best values of all groups are reduced across
// the warp together (independent shuffle chains), with no per-expert group arithmetic.
template <int EPL>
__device__ bool decide_groups_32(const RouteArgs& a, const double (&v)[EPL], const bool (&valid)[EPL], uint32_t exact,
                                 double delta_v, uint32_t* elig, uint32_t* mark, unsigned long long* keys) {
  // The two best values of every group (the largest and the largest of the rest, equal to the
  // first on a tie) on integer order keys, which order like the values (binary64 comparisons and
  // min/max are slow next to integer ones when many warps decide at once). Group g is slot g of
  // every lane; through the warp's shared scratch each group goes to 32 / EPL lanes of EPL keys
  // each, which take their two best and merge them by shuffles, instead of one chain of warp
  // reductions per group and rank.
  const int lane = threadIdx.x & 31;
  constexpr int LPG = 32 / EPL;  // lanes per group
  __syncwarp();  // the scratch's previous readers are done
#pragma unroll
  for (int g = 0; g < EPL; ++g) keys[g * 32 + lane] = order_key(valid[g] ? v[g] : -INFINITY);
  __syncwarp();
  unsigned long long k1 = 0ull, k2 = 0ull;  // 0 is below the key of every value, -inf included
  const unsigned long long* mine = keys + (lane / LPG) * 32 + (lane % LPG) * EPL;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const unsigned long long kk = mine[(i + lane) % EPL];
    if (kk > k1) {
      k2 = k1;
      k1 = kk;
    } else if (kk > k2) {
      k2 = kk;
    }
  }
#pragma unroll
  for (int off = 1; off < LPG; off <<= 1) {
    const unsigned long long o1 = __shfl_xor_sync(kFull, k1, off);
    const unsigned long long o2 = __shfl_xor_sync(kFull, k2, off);
    const unsigned long long lo1 = k1 < o1 ? k1 : o1, hi2 = k2 > o2 ? k2 : o2;
    k1 = k1 > o1 ? k1 : o1;
    k2 = lo1 > hi2 ? lo1 : hi2;
  }
  double t1[EPL], t2[EPL];
#pragma unroll
  for (int g = 0; g < EPL; ++g) {
    t1[g] = key_value(__shfl_sync(kFull, k1, g * LPG));
    t2[g] = key_value(__shfl_sync(kFull, k2, g * LPG));
  }
  double gs[EPL], gu[EPL];
#pragma unroll
  for (int g = 0; g < EPL; ++g) {
    // an inexact expert could be among the group's true top two if v >= second best - 2 delta_v
    const bool cand = valid[g] && !((exact >> g) & 1u) && v[g] >= t2[g] - 2.0 * delta_v;
    gs[g] = t1[g] + t2[g];
    gu[g] = __any_sync(kFull, cand) ? 2.0 * delta_v : 0.0;
  }
  uint32_t keep = 0;
  double min_kept = INFINITY, max_drop = -INFINITY;
  unsigned long long gk[EPL];  // group scores as order keys: larger score, larger key
#pragma unroll
  for (int g = 0; g < EPL; ++g) gk[g] = order_key(gs[g]);
#pragma unroll
  for (int g = 0; g < EPL; ++g) {
    int better = 0;
#pragma unroll
    for (int h = 0; h < EPL; ++h) better += (gk[h] > gk[g]) || (gk[h] == gk[g] && h < g);
    if (better < a.topk_group) {
      keep |= 1u << g;
      min_kept = fmin(min_kept, gs[g] - gu[g]);
    } else {
      max_drop = fmax(max_drop, gs[g] + gu[g]);
    }
  }
  bool ok = true;
  uint32_t m = 0;
  if (a.topk_group < a.G && !(min_kept > max_drop)) {
    uint32_t involved = 0;
#pragma unroll
    for (int g = 0; g < EPL; ++g) {
      const bool kept = (keep >> g) & 1u;
      if (gu[g] > 0.0 && (kept ? gs[g] - gu[g] <= max_drop : gs[g] + gu[g] >= min_kept)) involved |= 1u << g;
    }
    if (involved) {
      ok = false;
#pragma unroll
      for (int g = 0; g < EPL; ++g)
        if (valid[g] && ((involved >> g) & 1u) && !((exact >> g) & 1u) && v[g] >= t2[g] - 2.0 * delta_v) m |= 1u << g;
    }
  }
  *elig = 0;
#pragma unroll
  for (int g = 0; g < EPL; ++g)
    if (valid[g] && ((keep >> g) & 1u)) *elig |= 1u << g;
  *mark = m;
  return ok;
}

// Top-k selection of one token with per-expert uncertainty. l[j] is the logit
// of expert lane + 32j; bit j of `exact` says it is the binary64 value,
// otherwise it is the binary32 GEMM result whose selection value may be off by
// up to delta_v. Writes the k kept experts to rank[0..k). Returns true when
// every comparison the decision depends on is certain: strictly separated
// intervals, or both sides exact (exact ties then follow the index rule).
// Otherwise sets, in *refine, the inexact experts an uncertain comparison involves.
template <int EPL>
__device__ bool decide(const RouteArgs& a, const double (&l)[EPL], uint32_t exact, double delta_v, int16_t* rank,
                       int* n_ranked, uint32_t* refine, unsigned long long* keys) {
  const int lane = threadIdx.x & 31;
  double v[EPL];
  bool valid[EPL];
  selection_values<EPL>(a, l, v, valid);
  auto unc = [&](int j) { return ((exact >> j) & 1u) ? 0.0 : delta_v; };
  bool ok = true;
  uint32_t mark = 0;
  uint32_t elig_mask = 0;
  if (a.G > 1) {
    if (!decide_groups<EPL>(a, v, valid, exact, delta_v, &elig_mask, &mark, keys)) ok = false;
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (valid[j]) elig_mask |= 1u << j;
  }
  int n_elig = __popc(elig_mask);
#pragma unroll
  for (int off = 16; off; off >>= 1) n_elig += __shfl_xor_sync(kFull, n_elig, off);
  const int want = min(n_elig, a.k);
  uint32_t taken = 0;
  double prev_lo = 0.0;
  int prev_e = -1;
  bool prev_exact = true;
  double top_lo = INFINITY;  // min over the kept experts of v - u
  unsigned long long vk[EPL];  // selection values as order keys
#pragma unroll
  for (int j = 0; j < EPL; ++j) vk[j] = order_key(v[j]);
  for (int r = 0; r < want; ++r) {
    // this lane's best untaken eligible expert (lower j first on equal keys), then the warp's
    unsigned long long bk = 0ull;
    int bj = -1;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (((elig_mask & ~taken) >> j) & 1u && (bj < 0 || vk[j] > bk)) {
        bk = vk[j];
        bj = j;
      }
    // the lowest expert index among the lanes holding the best key: lane + 32 j, so the lowest j,
    // then the lowest lane
    const unsigned bhi = __reduce_max_sync(kFull, bj >= 0 ? (unsigned)(bk >> 32) : 0u);
    const unsigned blo = __reduce_max_sync(kFull, bj >= 0 && (unsigned)(bk >> 32) == bhi ? (unsigned)bk : 0u);
    const bool top = bj >= 0 && (unsigned)(bk >> 32) == bhi && (unsigned)bk == blo;
    const unsigned be = __reduce_min_sync(kFull, top ? (unsigned)(lane + 32 * bj) : 0xFFFFFFFFu);
    VE best;
    best.e = (int)be;
    best.v = __shfl_sync(kFull, pick(v, bj < 0 ? 0 : bj), (int)(be & 31));
    const int owner = best.e & 31, jb = best.e >> 5;
    const bool b_exact = __shfl_sync(kFull, (int)((exact >> jb) & 1u), owner) != 0;
    const double bu = b_exact ? 0.0 : delta_v;
    if (lane == owner) taken |= 1u << jb;
    if (r > 0 && !(prev_exact && b_exact) && !(prev_lo > best.v + bu)) {
      // adjacent order not certain: refine whichever of the two is inexact
      ok = false;
      if (!prev_exact && (prev_e & 31) == lane) mark |= 1u << (prev_e >> 5);
      if (!b_exact && lane == owner) mark |= 1u << jb;
    }
    prev_lo = best.v - bu;
    prev_e = best.e;
    prev_exact = b_exact;
    top_lo = fmin(top_lo, best.v - bu);
    if (lane == 0) rank[r] = (int16_t)best.e;
  }
  if (want < n_elig) {
    // The cut between the k kept experts and every eligible expert below them.
    double below_hi = -INFINITY;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (((elig_mask & ~taken) >> j) & 1u) below_hi = fmax(below_hi, v[j] + unc(j));
    below_hi = warp_max(below_hi);
    if (!(top_lo > below_hi)) {
      bool any = false;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        if (!((elig_mask >> j) & 1u) || ((exact >> j) & 1u)) continue;
        const bool mine = (taken >> j) & 1u;
        if (mine ? v[j] - delta_v <= below_hi : v[j] + delta_v >= top_lo) {
          mark |= 1u << j;
          any = true;
        }
      }
      if (__any_sync(kFull, any)) ok = false;
    }
  }
  *n_ranked = want;
  *refine = mark;
  __syncwarp();
  return ok;
}

// Full ranking of one token's eligible experts (the capacity rule needs it),
// by a bitonic sort across the warp: position p = lane * EPL + j. Each element
// carries its expert index and exactness. After the sort, adjacent pairs are
// certified like the top-k pairs; uncertain inexact experts are flagged in
// `flags` (per-warp shared, one byte per expert) and returned in *refine.
template <int EPL>
__device__ bool decide_full(const RouteArgs& a, const double (&l)[EPL], uint32_t exact, double delta_v,
                            int16_t* rank, uint8_t* flags, int* n_ranked, uint32_t* refine,
                            unsigned long long* keys) {
  const int lane = threadIdx.x & 31;
  const int E = a.E;
  double v0[EPL];
  bool valid[EPL];
  selection_values<EPL>(a, l, v0, valid);
  uint32_t elig_mask = 0;
  bool ok = true;
  uint32_t mark = 0;
  if (a.G > 1) {
    if (!decide_groups<EPL>(a, v0, valid, exact, delta_v, &elig_mask, &mark, keys)) ok = false;
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (valid[j]) elig_mask |= 1u << j;
  }
  // keys in sort layout: lane holds positions lane*EPL .. lane*EPL+EPL-1. The sort compares the
  // values' integer order keys (binary64 comparisons are slow next to integer ones when many
  // warps sort at once); the values come back from the keys afterwards.
  unsigned long long kk[EPL];
  int ke[EPL];  // expert | exact << 16, or -1 for empty
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 32 * j;
    const bool el = (elig_mask >> j) & 1u;
    kk[j] = order_key(el ? v0[j] : -INFINITY);
    ke[j] = el ? (e | (int)(((exact >> j) & 1u) << 16)) : (0x7FFF | (1 << 16));
  }
  auto key_better = [](unsigned long long ka, int ea, unsigned long long kb, int eb) {
    return ka > kb || (ka == kb && ea < eb);
  };
  constexpr int S = 32 * EPL;
#pragma unroll
  for (int k = 2; k <= S; k <<= 1) {
#pragma unroll
    for (int d = k >> 1; d > 0; d >>= 1) {
      if (d < EPL) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const int jp = j ^ d;
          if (jp > j) {
            const int p = lane * EPL + j;
            const bool up = (p & k) == 0;  // block sorted best-first
            const bool swap = up ? key_better(kk[jp], ke[jp] & 0xFFFF, kk[j], ke[j] & 0xFFFF)
                                 : key_better(kk[j], ke[j] & 0xFFFF, kk[jp], ke[jp] & 0xFFFF);
            if (swap) {
              const unsigned long long tk = kk[j];
              kk[j] = kk[jp];
              kk[jp] = tk;
              const int te = ke[j];
              ke[j] = ke[jp];
              ke[jp] = te;
            }
          }
        }
      } else {
        const int ld = d / EPL;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          const unsigned long long ok_ = __shfl_xor_sync(kFull, kk[j], ld);
          const int oe = __shfl_xor_sync(kFull, ke[j], ld);
          const int p = lane * EPL + j;
          const bool up = (p & k) == 0;
          const bool lower = (lane & ld) == 0;  // this element sits at the smaller position
          const bool other_better = key_better(ok_, oe & 0xFFFF, kk[j], ke[j] & 0xFFFF);
          // the smaller position keeps the better key in an ascending block
          const bool take = (lower == up) ? other_better : !other_better;
          if (take) {
            kk[j] = ok_;
            ke[j] = oe;
          }
        }
      }
    }
  }
  double kv[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) kv[j] = key_value(kk[j]);
  int n_elig = __popc(elig_mask);
#pragma unroll
  for (int off = 16; off; off >>= 1) n_elig += __shfl_xor_sync(kFull, n_elig, off);
  // certify adjacent pairs (p, p+1) inside the eligible prefix
  const double nxt_v = __shfl_down_sync(kFull, kv[0], 1);
  const int nxt_e = __shfl_down_sync(kFull, ke[0], 1);
  bool any_flag = false;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int p = lane * EPL + j;
    if (p + 1 >= n_elig) continue;
    const double vb = (j + 1 < EPL) ? kv[(j + 1) % EPL] : nxt_v;
    const int eb = (j + 1 < EPL) ? ke[(j + 1) % EPL] : nxt_e;
    const bool ea_exact = (ke[j] >> 16) & 1, eb_exact = (eb >> 16) & 1;
    const double ua = ea_exact ? 0.0 : delta_v, ub = eb_exact ? 0.0 : delta_v;
    if (!(ea_exact && eb_exact) && !(kv[j] - ua > vb + ub)) {
      if (!ea_exact) flags[ke[j] & 0xFFFF] = 1;
      if (!eb_exact) flags[eb & 0xFFFF] = 1;
      any_flag = true;
    }
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int p = lane * EPL + j;
    if (p < n_elig) rank[p] = (int16_t)(ke[j] & 0xFFFF);
  }
  if (__any_sync(kFull, any_flag)) {
    ok = false;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = lane + 32 * j;
      if (e < E && flags[e]) {
        mark |= 1u << j;
        flags[e] = 0;
      }
    }
  }
  __syncwarp();
  *n_ranked = n_elig;
  *refine = mark;
  return ok;
}

// Gate weights of the slots in idx[0..k) (entries < 0 are dropped slots).
// Lane j < k returns the weight of slot j.
// s_val: this warp's kMaxTopK doubles of shared memory.
template <int EPL>
__device__ float gates(const RouteArgs& a, const double (&l)[EPL], const int* idx_of_slot, double* s_val) {
  const int lane = threadIdx.x & 31;
  double m = -INFINITY;
  if (a.score_fn == MOE_SCORE_SOFTMAX) {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (lane + 32 * j < a.E) m = fmax(m, l[j]);
    m = warp_max(m);
  }
  double z = 0.0;
  if (a.score_fn == MOE_SCORE_SOFTMAX) {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (lane + 32 * j < a.E) z += exp(l[j] - m);
    z = warp_sum(z);
  }
  // the logit of each kept expert to its slot's lane (the lane owning the expert writes it), then
  // every slot's score at once
  for (int r = 0; r < a.k; ++r) {
    const int e = idx_of_slot[r];
    if (e >= 0 && (e & 31) == lane) s_val[r] = pick(l, e >> 5);
  }
  __syncwarp();
  double mine = 0.0;
  const int e_mine = lane < a.k ? idx_of_slot[lane] : -1;
  if (e_mine >= 0) {
    const double le = s_val[lane];
    mine = a.score_fn == MOE_SCORE_SOFTMAX ? exp(le - m) / z : raw_score(a.score_fn, le);
  }
  __syncwarp();  // s_val is the next token's
  double denom = 1.0;
  if (a.renorm) denom = warp_sum(lane < a.k ? mine : 0.0);
  // a dropped slot weighs 0, also when every slot of the token was dropped
  const bool kept = lane < a.k && idx_of_slot[lane] >= 0;
  return kept ? (float)(mine / denom * (double)a.rsf) : 0.0f;
}

}  // namespace
}  // namespace moe
