// decode.cuh -- what the layers for few tokens share (decode_router.cu, decode_simt.cu,
// decode_tc.cu): the counters that order the work inside a launch, the routing decision, the plan of
// active experts.
//
// The layer of n <= 64 tokens is two launches. The first (decode_router.cu) computes the router
// logits, quantises x where the experts want E4M3, and clears the counters; the second is set up
// meanwhile (programmatic dependent launch) and does the rest. Its work is cut into units that
// thread blocks claim from counters in the workspace, in this order: routing decisions, gate/up
// tiles (shared experts first), down tiles. A unit waits only for units that were claimed before
// it, so some block is running each of them and every wait ends, whatever share of the grid is
// resident: no cooperative launch, and calls on several streams may overlap on the GPU. Waits are
// bounded all the same (kDecodeWaitCycles).
//
// Sums are deterministic: no floating-point atomics; whichever block adds the expert rows of a
// column range takes them in slot order.
#pragma once

#include "common.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
// Counter words (zeroed before the launch).
enum {
  kCtrAbort = 0,
  kCtrToken,       // routing decisions handed out / finished
  kCtrTokenDone,
  kCtrTile,        // gate/up and down tiles handed out
  kCtrExpert = 16  // [E + 1] finished gate/up tiles per expert (E: shared), then [column ranges] finished down
                   // tiles, then (gate/up tiles cut along k) [E * tiles + shared tiles] finished parts
};
constexpr int kMinColumns = 32;  // output columns of a down tile, at least
// Up to here every block decides the tokens itself: a decision takes 1.5 us, handing it on through
// global memory as long again.
constexpr int kSelfTokens = 2;

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

// One thread waits until *p >= target. False once the call is abandoned. (The limit is read off the SM's clock, which
// takes a few cycles; %globaltimer takes long enough to delay a wait that ends meanwhile.)
__device__ __noinline__ inline bool wait_counter(const int32_t* p, int target, int32_t* ctr, moe_diag* status, int64_t limit) {
  if (ld_acquire(p) >= target) return true;
  const long long t0 = clock64();
  for (uint32_t it = 1;; ++it) {
    if (ld_acquire(p) >= target) return true;
    if ((it & 63u) == 0) {
      if (ld_acquire(ctr + kCtrAbort)) return false;
      if (clock64() - t0 > limit) {
        atomicExch(ctr + kCtrAbort, 1);
        set_status(status, MOE_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

// ---- routing decision --------------------------------------------------------------

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}

// Order-preserving key of a double: a larger value has a larger key; never 0. -0 is taken as +0
// first, so that the two have one key as they compare equal.
__device__ __forceinline__ unsigned long long order_key(double v) {
  const unsigned long long b = (unsigned long long)__double_as_longlong(v + 0.0);
  const unsigned long long key = (b >> 63) ? ~b : (b | 0x8000000000000000ull);
  return key ? key : 1ull;
}

struct __align__(16) DecideScratch {
  uint32_t hi[kMaxExperts];             // upper halves of the selection keys; 0: not eligible
  unsigned long long top[kMaxExperts];  // each warp's k best keys, best first (0: none)
  int16_t top_e[kMaxExperts];           // and their experts
  uint8_t place[kMaxExperts];           // an expert's slot
  unsigned long long key[kMaxExperts];
  unsigned long long group[kMaxGroups];
  double best[2][kMaxGroups];
  double part[8];
  double val[kMaxTopK];
  int idx[kMaxTopK];
};

// The block's largest value (SUM: sum) of v over the first `warps` warps, in a fixed order.
template <bool SUM, typename Sync>
__device__ __noinline__ double block_reduce(double v, double* part, int tid, int warps, Sync sync) {
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    const double o = __shfl_xor_sync(kFull, v, off);
    v = SUM ? v + o : fmax(v, o);
  }
  if ((tid & 31) == 0) part[tid >> 5] = v;
  sync();
  v = part[0];
  for (int i = 1; i < warps; ++i) v = SUM ? v + part[i] : fmax(v, part[i]);
  sync();
  return v;
}

// Token t's experts and gates from its binary64 logits (definitions in router.cu) to out_idx and
// out_w, by 256 threads, an expert each; `bias` is the thread's expert's.
// An expert's place is the number of better ones: first in its warp, by the upper halves of the keys
// (a warp with two equal halves counts the whole keys), then each warp's k best among those of all.
// Counting costs 1.5 us at E = 256, top-8 of 4 of 8 groups. One warp walking top-k rounds with eight
// experts a lane took 49 us (its code, run once, comes from memory), counting whole keys 3.6 us.
template <typename Sync>
__device__ void decide_token(const DecodeArgs& a, int t, float bias, DecideScratch* sc, int tid, Sync sync, int* out_idx,
                             float* out_w) {
  const int e = tid, lane = tid & 31, w0 = tid & ~31;
  const bool live = e < a.E;
  const double l = live ? __ldcg(a.logits + (int64_t)t * a.E + e) : 0.0;
  double score = l;  // what the gate is made of
  if (a.score_fn == MOE_SCORE_SIGMOID)
    score = 1.0 / (1.0 + exp(-l));
  else if (a.score_fn == MOE_SCORE_SQRTSOFTPLUS)
    score = sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
  const double sel = score + (double)bias;
  unsigned long long key = live ? order_key(sel) : 0ull;
  sc->key[e] = key;
  sc->place[e] = 0xFF;
  if (a.G > 1) {
    // the two best of each group, then the groups by their sum (ties: the lower group)
    const int per = a.E / a.G, g = e / per;
    if (per == 32) {  // a group is a warp
      if (live) {
        const unsigned hi = (unsigned)(key >> 32), lo = (unsigned)key;
        const unsigned h1 = __reduce_max_sync(kFull, hi), l1 = __reduce_max_sync(kFull, hi == h1 ? lo : 0u);
        const int first = __ffs(__ballot_sync(kFull, hi == h1 && lo == l1)) - 1;
        const unsigned hr = lane == first ? 0u : hi;
        const unsigned h2 = __reduce_max_sync(kFull, hr), l2 = __reduce_max_sync(kFull, hr == h2 ? lo : 0u);
        const int second = __ffs(__ballot_sync(kFull, hr == h2 && lo == l2)) - 1;
        const double b = __shfl_sync(kFull, sel, first) + __shfl_sync(kFull, sel, second);
        if (lane == 0) sc->group[g] = order_key(b);
      }
    } else {
      sync();
      if (live) {
        int better = 0;
#pragma unroll 4
        for (int f = g * per; f < (g + 1) * per; ++f) {
          const unsigned long long o = sc->key[f];
          better += (o > key) | ((o == key) & (f < e));
        }
        if (better < 2) sc->best[better][g] = sel;
        if (per == 1) sc->best[1][g] = -INFINITY;
      }
      sync();
      if (tid < a.G) sc->group[tid] = order_key(sc->best[0][tid] + sc->best[1][tid]);
    }
    sync();
    if (live) {
      const unsigned long long mine = sc->group[g];
      int better = 0;
#pragma unroll 8
      for (int h = 0; h < a.G; ++h) better += (sc->group[h] > mine) | ((sc->group[h] == mine) & (h < g));
      if (better >= a.topk_group) sc->key[e] = key = 0ull;
    }
  }
  sc->hi[e] = (uint32_t)(key >> 32);
  if (a.score_fn == MOE_SCORE_SOFTMAX) {
    const int warps = (a.E + 31) / 32;
    const double m = block_reduce<false>(live ? l : -INFINITY, sc->part, tid, warps, sync);
    score = live ? exp(l - m) : 0.0;
    // (over the kept slots the sum of all experts cancels)
    if (!a.renorm) score /= block_reduce<true>(score, sc->part, tid, warps, sync);
  }
  const int per_warp = min(a.k, 32);
  if (w0 < a.E) {
    unsigned long long* top = sc->top + (w0 >> 5) * per_warp;
    if (lane < per_warp) top[lane] = 0ull;
    __syncwarp();  // the warp's keys and empty list
    const uint32_t mine = (uint32_t)(key >> 32);
    int better = 0, same = 0;
#pragma unroll
    for (int f = 0; f < 32; f += 4) {
      const uint4 o = *reinterpret_cast<const uint4*>(sc->hi + w0 + f);
      better += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
      same += (o.x == mine) + (o.y == mine) + (o.z == mine) + (o.w == mine);
    }
    if (__any_sync(kFull, key && same > 1)) {
      better = 0;
      for (int f = 0; f < 32; ++f) {
        const unsigned long long o = sc->key[w0 + f];
        better += (o > key) | ((o == key) & (f < lane));
      }
    }
    if (key && better < per_warp) {
      top[better] = key;
      sc->top_e[(w0 >> 5) * per_warp + better] = (int16_t)e;
    }
  }
  sync();
  // every candidate against the others, four lanes a candidate
  const int count = (a.E + 31) / 32 * per_warp;
  for (int c0 = 0; c0 < count; c0 += 64) {
    const int c = c0 + (tid >> 2);
    const unsigned long long mine = c < count ? sc->top[c] : 0ull;
    const int ce = mine ? sc->top_e[c] : 0;
    int better = 0;
    if (mine) {
#pragma unroll 4
      for (int f = tid & 3; f < count; f += 4) {
        const unsigned long long o = sc->top[f];
        better += (o > mine) | ((o == mine) & (sc->top_e[f] < ce));
      }
    }
    better += __shfl_xor_sync(kFull, better, 1);
    better += __shfl_xor_sync(kFull, better, 2);
    if (mine && (tid & 3) == 0 && better < a.k) sc->place[ce] = (uint8_t)better;
  }
  sync();
  const int slot = sc->place[e];
  if (slot < a.k) {
    sc->idx[slot] = e;
    sc->val[slot] = score;
  }
  sync();
  if (tid < 32) {
    const double v = tid < a.k ? sc->val[tid] : 0.0;
    const double denom = a.renorm ? warp_sum(v) : 1.0;
    if (tid < a.k) {
      out_idx[tid] = sc->idx[tid];
      out_w[tid] = (float)(v / denom * (double)a.rsf);
    }
  }
  sync();
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

// Built by NT threads (tid 0 .. NT-1, warp 0 among them) from the finished decisions at idx and w;
// slot_w and slot_r (given: [n * k]) receive each slot's gate and its row. The masks are zero.
template <int NT, typename Sync>
__device__ void build_plan(const DecodeArgs& a, const int* idx, const float* w, DecodePlan* p, float* slot_w,
                           uint16_t* slot_r, int tid, Sync sync) {
  const int slots = a.n * a.k;
  // idx and w: global memory written in this launch (never through L1), or shared memory
  const volatile int* vi = idx;
  const volatile float* vw = w;
  // the first NT slots stay in registers: most batches have no more
  const int e0 = tid < slots ? vi[tid] : 0;
  const float g0 = tid < slots ? vw[tid] : 0.0f;
  for (int s = tid; s < slots; s += NT) atomicOr(&p->mask[s == tid ? e0 : vi[s]], 1ull << (s / a.k));
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
    int both = rows << 16 | live;  // at most 2048 rows, 256 experts
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(kFull, both, off);
      if (tid >= off) both += o;
    }
    if (tid == 31) {
      p->off[kMaxExperts] = both >> 16;
      p->n_act = both & 0xFFFF;
    }
    int r = (both >> 16) - rows, v = (both & 0xFFFF) - live;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      p->off[tid * PER + j] = r;
      if (c[j]) p->act[v++] = (int16_t)(tid * PER + j);
      r += c[j];
    }
  }
  sync();
  if (slot_w)
    for (int s = tid; s < slots; s += NT) {
      slot_w[s] = s == tid ? g0 : vw[s];
      slot_r[s] = (uint16_t)slot_row(*p, s == tid ? e0 : vi[s], s / a.k);
    }
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
      a.diag->dropped = 0;
      a.diag->refined_tokens = 0;
      a.diag->max_load = most;
      a.diag->refined_logits = 0;
    }
  }
}

// Launch that may begin before the kernel in front of it has ended; every kernel launched so waits
// for that end (griddepcontrol.wait) before it touches global memory.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), int grid, int block, size_t smem, cudaStream_t s, const Args&... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void wait_for_earlier_kernels() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace
}  // namespace moe
