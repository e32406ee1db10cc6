// decode.cuh -- what the one-kernel layers for few tokens share (decode_simt.cu, decode_tc.cu):
// arguments, the counters that order the work inside the launch, the router in binary64, the plan
// of active experts and the combine.
//
// The layer of n <= 64 tokens is one launch. Its work is cut into units that thread blocks claim
// from counters in the workspace, in this order: E4M3 rows of x (FP8), router logits, routing
// decisions, gate/up tiles (shared experts first), down tiles. A unit waits only for units that
// were claimed before it, so some block is running each of them and every wait ends, whatever
// share of the grid is resident: no cooperative launch, and calls on several streams may overlap
// on the GPU. Waits are bounded all the same (kDecodeTimeoutNs).
//
// Sums are deterministic: no floating-point atomics; the block that finishes the last down tile of
// a column range adds that range's expert rows in slot order.
#pragma once

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "route_decide.cuh"

namespace moe {
namespace {

constexpr uint64_t kDecodeTimeoutNs = 2000000000ull;  // 2 s for any single wait

// Counter words (zeroed before the launch).
enum {
  kCtrAbort = 0,
  kCtrQuant,       // E4M3 rows handed out / finished
  kCtrQuantDone,
  kCtrLogit,       // router units
  kCtrLogitDone,
  kCtrToken,       // routing decisions
  kCtrTokenDone,
  kCtrTile,        // gate/up and down tiles
  kCtrExpert = 16  // [E + 1] finished gate/up tiles per expert (E: shared), then [column ranges] finished down tiles
};

__device__ __forceinline__ int ld_acquire(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ int add_release(int32_t* p, int v) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// One thread waits until *p >= target. False once the call is abandoned.
__device__ __noinline__ inline bool wait_counter(const int32_t* p, int target, int32_t* ctr, moe_diag* status) {
  if (ld_acquire(p) >= target) return true;
  const uint64_t t0 = ptx::globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (ld_acquire(p) >= target) return true;
    if ((it & 63u) == 0) {
      if (ld_acquire(ctr + kCtrAbort)) return false;
      if (ptx::globaltimer() - t0 > kDecodeTimeoutNs) {
        atomicExch(ctr + kCtrAbort, 1);
        set_status(status, MOE_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

// ---- E4M3 activations --------------------------------------------------------------

// The codes of a 1 x 128 tile, four values per lane of the warp, and its scale byte.
__device__ __forceinline__ uint32_t quantize_tile(const float (&v)[4], uint32_t* byte) {
  float m = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
  for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
  const int e = ue8m0_exponent(m);
  *byte = (uint32_t)(e + 127);
  return e4m3x4(v[0], v[1], v[2], v[3], pow2_neg(e));
}

// Tile i of x's n * d / 128 (row by row), by one warp.
__device__ __forceinline__ void quantize_x_tile(const DecodeArgs& a, int64_t i) {
  const int lane = threadIdx.x & 31;
  const uint2 raw = __ldg(reinterpret_cast<const uint2*>(a.x) + i * 32 + lane);
  const float v[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u), __uint_as_float(raw.y << 16),
                      __uint_as_float(raw.y & 0xFFFF0000u)};
  uint32_t byte;
  const uint32_t q = quantize_tile(v, &byte);
  reinterpret_cast<uint32_t*>(a.xq)[i * 32 + lane] = q;
  if (lane == 0) a.xs[i] = (uint8_t)byte;
}

// ---- router ------------------------------------------------------------------------

// 16 bytes of activations or router weights as binary32 (8 bf16 or 4 binary32 values).
template <typename T>
struct Chunk {
  static constexpr int N = 16 / sizeof(T);
};
__device__ __forceinline__ void unpack(const uint4& raw, float (&v)[8]) {
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(u[j] << 16);
    v[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(const uint4& raw, float (&v)[4]) {
  v[0] = __uint_as_float(raw.x), v[1] = __uint_as_float(raw.y), v[2] = __uint_as_float(raw.z), v[3] = __uint_as_float(raw.w);
}

// Experts per router unit: the units spread over the grid.
__host__ __device__ inline int router_unit(int E, int grid) { return (E + grid - 1) / grid; }

constexpr int kRouterTokens = 4;  // tokens of one dot-product item: each weight is converted once for them

// Binary64 logits of experts [e0, e1) for every token, by the NW warps of a block (warp `w`; `part`:
// NW * 2 * kRouterTokens doubles). Exact products, binary64 sums. Items are (expert, four tokens),
// cut along d when there are fewer of them than warps; a cut item's parts are added in order.
// `sync` is a barrier of these warps.
template <typename T, int NW, typename Sync>
__device__ void router_logits_unit(const DecodeArgs& a, int e0, int e1, int w, double* part, Sync sync) {
  constexpr int C = Chunk<T>::N;
  const int lane = threadIdx.x & 31;
  const int groups = (a.n + kRouterTokens - 1) / kRouterTokens;
  const int items = (e1 - e0) * groups;
  const int cuts = items >= NW ? 1 : NW / items;
  const int chunks = a.d / C;  // d % 8 == 0
  const int per = (chunks + cuts - 1) / cuts;
  for (int it = w; it < items * cuts; it += NW) {
    const int item = it / cuts, cut = it % cuts;
    const int e = e0 + item / groups, t0 = (item % groups) * kRouterTokens;
    const uint4* wr = reinterpret_cast<const uint4*>(static_cast<const T*>(a.w_router) + (int64_t)e * a.d);
    const uint4* xr = reinterpret_cast<const uint4*>(static_cast<const T*>(a.x));
    double acc[kRouterTokens] = {};
    const int c1 = min(chunks, (cut + 1) * per);
#pragma unroll 2
    for (int c = cut * per + lane; c < c1; c += 32) {
      float wv[C];
      unpack(__ldg(wr + c), wv);
      double wd[C];
#pragma unroll
      for (int j = 0; j < C; ++j) wd[j] = (double)wv[j];
#pragma unroll
      for (int q = 0; q < kRouterTokens; ++q) {
        if (t0 + q >= a.n) break;
        float xv[C];
        unpack(__ldg(xr + (int64_t)(t0 + q) * chunks + c), xv);
#pragma unroll
        for (int j = 0; j < C; ++j) acc[q] = fma((double)xv[j], wd[j], acc[q]);
      }
    }
#pragma unroll
    for (int q = 0; q < kRouterTokens; ++q) {
      if (t0 + q >= a.n) break;
      const double s = warp_sum(acc[q]);
      if (lane == 0) {
        if (cuts == 1)
          a.logits[(int64_t)(t0 + q) * a.E + e] = s;
        else
          part[it * kRouterTokens + q] = s;  // it < items * cuts <= NW
      }
    }
  }
  if (cuts == 1) return;
  sync();
  if (w == 0)
    for (int i = lane; i < items * kRouterTokens; i += 32) {
      const int item = i / kRouterTokens, q = i % kRouterTokens;
      const int t = (item % groups) * kRouterTokens + q;
      if (t >= a.n) continue;
      double s = 0.0;
      for (int cut = 0; cut < cuts; ++cut) s += part[(item * cuts + cut) * kRouterTokens + q];
      a.logits[(int64_t)t * a.E + e0 + item / groups] = s;
    }
  sync();  // `part` is the next unit's
}

// Scratch of one deciding warp.
struct DecideScratch {
  int16_t rank[kMaxExperts];
  int idx[kMaxTopK];
  double val[kMaxTopK];
  unsigned long long keys[kMaxExperts];
};

// Token t's experts and gates from its binary64 logits, by one warp.
template <int EPL>
__device__ void decide_token(const DecodeArgs& a, int t, DecideScratch* sc) {
  const int lane = threadIdx.x & 31;
  RouteArgs r{};
  r.bias = a.bias;
  r.E = a.E;
  r.k = a.k;
  r.G = a.G;
  r.topk_group = a.topk_group;
  r.score_fn = a.score_fn;
  r.renorm = a.renorm;
  r.rsf = a.rsf;
  double l[EPL];
  uint32_t exact = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 32 * j;
    l[j] = e < a.E ? __ldcg(a.logits + (int64_t)t * a.E + e) : 0.0;
    exact |= 1u << j;
  }
  int nr = 0;
  uint32_t refine = 0;
  decide<EPL>(r, l, exact, 0.0, sc->rank, &nr, &refine, sc->keys);  // exact logits: every comparison is certain
  if (lane < a.k) sc->idx[lane] = lane < nr ? (int)sc->rank[lane] : -1;
  __syncwarp();
  const float g = gates<EPL>(r, l, sc->idx, sc->val);
  if (lane < a.k) {
    a.topk_idx[t * a.k + lane] = sc->idx[lane];
    a.topk_w[t * a.k + lane] = g;
  }
  __syncwarp();
}

__device__ inline void decide_token_any(const DecodeArgs& a, int t, DecideScratch* sc) {
  if (a.E <= 32)
    decide_token<1>(a, t, sc);
  else if (a.E <= 64)
    decide_token<2>(a, t, sc);
  else if (a.E <= 128)
    decide_token<4>(a, t, sc);
  else
    decide_token<8>(a, t, sc);
}

// ---- plan --------------------------------------------------------------------------

// The batch's routing in shared memory: which tokens each expert holds (n <= 64 bits), the first
// row of each expert when the slots are ordered by expert and token, and the active experts.
struct DecodePlan {
  unsigned long long mask[kMaxExperts];
  int32_t off[kMaxExperts + 1];
  int16_t act[kMaxExperts];
  int32_t n_act;
};

__device__ __forceinline__ unsigned long long token_mask(int n) { return n >= 64 ? ~0ull : (1ull << n) - 1ull; }

// Row of token t among the slots of expert e.
__device__ __forceinline__ int slot_row(const DecodePlan& p, int e, int t) {
  return p.off[e] + __popcll(p.mask[e] & ((1ull << t) - 1ull));
}

// Built by NT threads (tid 0 .. NT-1, warp 0 among them) from the finished decisions.
template <int NT, typename Sync>
__device__ void build_plan(const DecodeArgs& a, DecodePlan* p, int tid, Sync sync) {
  for (int e = tid; e < kMaxExperts; e += NT) p->mask[e] = 0ull;
  sync();
  for (int s = tid; s < a.n * a.k; s += NT) {
    const int e = __ldcg(a.topk_idx + s);
    if (e >= 0) atomicOr(&p->mask[e], 1ull << (s / a.k));
  }
  sync();
  if (tid < 32) {
    constexpr int PER = kMaxExperts / 32;
    int c[PER], rows = 0, live = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      c[j] = __popcll(p->mask[tid * PER + j]);
      rows += c[j];
      live += c[j] > 0;
    }
    int r = rows, v = live;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int ro = __shfl_up_sync(kFull, r, off), vo = __shfl_up_sync(kFull, v, off);
      if (tid >= off) r += ro, v += vo;
    }
    if (tid == 31) {
      p->off[kMaxExperts] = r;
      p->n_act = v;
    }
    r -= rows;
    v -= live;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      p->off[tid * PER + j] = r;
      if (c[j]) p->act[v++] = (int16_t)(tid * PER + j);
      r += c[j];
    }
  }
  sync();
}

// counts and diag of the call, by one block.
template <int NT>
__device__ void write_counts(const DecodeArgs& a, const DecodePlan& p, int tid) {
  if (a.counts)
    for (int e = tid; e < a.E; e += NT) a.counts[e] = __popcll(p.mask[e]);
  if (a.diag && tid < 32) {
    int most = 0;
    for (int e = tid; e < a.E; e += 32) most = max(most, __popcll(p.mask[e]));
    most = __reduce_max_sync(kFull, most);
    if (tid == 0) {
      a.diag->overflowed = 0;
      a.diag->dropped = a.n * a.k - p.off[kMaxExperts];
      a.diag->refined_tokens = 0;
      a.diag->max_load = most;
      a.diag->refined_logits = 0;
    }
  }
}

}  // namespace
}  // namespace moe
