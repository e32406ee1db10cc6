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

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr uint64_t kDecodeTimeoutNs = 2000000000ull;  // 2 s for any single wait

// Counter words (zeroed before the launch).
enum {
  kCtrAbort = 0,
  kCtrQuant,       // E4M3 rows handed out / finished
  kCtrQuantDone,
  kCtrLogit,       // router units
  kCtrLogitDone,
  kCtrToken,       // routing decisions, a block each
  kCtrTokenDone,
  kCtrTile,        // gate/up and down tiles
  kCtrExpert = 16  // [E + 1] finished gate/up tiles per expert (E: shared), then [column ranges] finished down
                   // tiles, then (gate/up tiles cut along k) [E * tiles + shared tiles] finished parts
};
constexpr int kMinColumns = 32;  // output columns of a down tile, at least

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

// A binary32 value times 2^-896 as a binary64, exact for every finite value (subnormals and zeros
// included: the fields only move): three integer operations, where the conversion instruction runs
// at 4 lanes a clock and SM and made the logits of 64 tokens take 150 us.
__device__ __forceinline__ double widened(float v) {
  const int u = __float_as_int(v);
  return __hiloint2double((u >> 3) & (int)0x8FFFFFFF, u << 29);
}
// A router weight gets 2^512 (two steps: 2^(896 + 512) is past the range), so that its products with
// widened activations are 2^-384 of the true ones, far from both ends of the range.
__device__ __forceinline__ double widened_weight(float v) { return widened(v) * 0x1p1000 * 0x1p408; }
constexpr double kWidenLogit = 0x1p384;

constexpr int kRouterTokens = 4;  // tokens of one dot-product item: each weight is widened once for them

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}

// Binary64 logits of experts e0 and (pair) e0 + 1 for every token, by the NW warps of a block (warp
// `w`; `part`: NW * 2 * kRouterTokens doubles). Products of bf16 values are exact, sums are binary64.
// Items are groups of TOK tokens, cut along d when there are fewer of them than warps; a cut item's
// parts are added in order. The loads of BATCH steps are issued before their products: a step whose
// loads wait on branches took a memory latency per token. A row with a NaN or an infinity gets NaN
// logits (the widening alone would take them for finite values). `sync` is a barrier of these warps.
template <typename T, int NW, int TOK, int BATCH, typename Sync>
__device__ void router_logits_pair(const DecodeArgs& a, int e0, bool pair, int w, double* part, Sync sync) {
  constexpr int C = Chunk<T>::N;
  const int lane = threadIdx.x & 31;
  const int items = (a.n + TOK - 1) / TOK;
  const int cuts = items >= NW ? 1 : NW / items;
  const int chunks = a.d / C;  // d % 8 == 0
  const int per = (chunks + cuts - 1) / cuts;
  const uint4* w0 = reinterpret_cast<const uint4*>(static_cast<const T*>(a.w_router) + (int64_t)e0 * a.d);
  const uint4* w1 = pair ? w0 + chunks : w0;
  for (int it = w; it < items * cuts; it += NW) {
    const int item = it / cuts, cut = it % cuts, t0 = item * TOK;
    const int last = min(TOK, a.n - t0) - 1;
    const uint4* xr = reinterpret_cast<const uint4*>(a.x) + (int64_t)t0 * chunks;
    double acc[2][TOK] = {};
    float odd[2] = {}, odd_x[TOK] = {};  // NaN once a value is not finite
    const int c1 = min(chunks, (cut + 1) * per);
    for (int c0 = cut * per; c0 < c1; c0 += 32 * BATCH) {
      uint4 r0[BATCH], r1[BATCH], rx[BATCH][TOK];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int c = c0 + 32 * b + lane;
        const bool in = c < c1;
        r0[b] = in ? __ldg(w0 + c) : make_uint4(0, 0, 0, 0);
        r1[b] = in ? __ldg(w1 + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < TOK; ++q)  // past the last token: its row again, not stored
          rx[b][q] = in ? __ldg(xr + (int64_t)min(q, last) * chunks + c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        float v0[C], v1[C];
        unpack(r0[b], v0);
        unpack(r1[b], v1);
        double d0[C], d1[C];
#pragma unroll
        for (int j = 0; j < C; ++j) {
          d0[j] = widened_weight(v0[j]);
          d1[j] = widened_weight(v1[j]);
          odd[0] = fmaf(v0[j], 0.0f, odd[0]);
          odd[1] = fmaf(v1[j], 0.0f, odd[1]);
        }
#pragma unroll
        for (int q = 0; q < TOK; ++q) {
          float xv[C];
          unpack(rx[b][q], xv);
#pragma unroll
          for (int j = 0; j < C; ++j) {
            const double xd = widened(xv[j]);
            acc[0][q] = fma(xd, d0[j], acc[0][q]);
            acc[1][q] = fma(xd, d1[j], acc[1][q]);
            odd_x[q] = fmaf(xv[j], 0.0f, odd_x[q]);
          }
        }
      }
    }
#pragma unroll
    for (int q = 0; q < TOK; ++q)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const double s = warp_sum(acc[p][q] * kWidenLogit + (double)(odd[p] + odd_x[q]));
        if (lane != 0 || (p && !pair) || q > last) continue;
        if (cuts == 1)
          a.logits[(int64_t)(t0 + q) * a.E + e0 + p] = s;
        else
          part[(it * 2 + p) * TOK + q] = s;  // it < items * cuts <= NW
      }
  }
  if (cuts == 1) return;
  sync();
  if (w == 0)
    for (int i = lane; i < items * 2 * TOK; i += 32) {
      const int item = i / (2 * TOK), p = i / TOK % 2, q = i % TOK;
      const int t = item * TOK + q;
      if (t >= a.n || (p && !pair)) continue;
      double s = 0.0;
      for (int cut = 0; cut < cuts; ++cut) s += part[((item * cuts + cut) * 2 + p) * TOK + q];
      a.logits[(int64_t)t * a.E + e0 + p] = s;
    }
  sync();  // `part` is the next pair's
}

template <typename T, int NW, typename Sync>
__device__ void router_logits_unit(const DecodeArgs& a, int e0, int e1, int w, double* part, Sync sync) {
  for (int e = e0; e < e1; e += 2) {
    if (a.n == 1)
      router_logits_pair<T, NW, 1, 4>(a, e, e + 1 < e1, w, part, sync);
    else
      router_logits_pair<T, NW, kRouterTokens, 2>(a, e, e + 1 < e1, w, part, sync);
  }
}

// Order-preserving key of a double: a larger value has a larger key; never 0. -0 is taken as +0
// first, so that the two have one key as they compare equal.
__device__ __forceinline__ unsigned long long order_key(double v) {
  const unsigned long long b = (unsigned long long)__double_as_longlong(v + 0.0);
  const unsigned long long key = (b >> 63) ? ~b : (b | 0x8000000000000000ull);
  return key ? key : 1ull;
}

struct __align__(16) DecideScratch {
  unsigned long long key[kMaxExperts];  // selection values; 0: not eligible
  unsigned long long top[kMaxExperts];  // each warp's k best keys and experts, best first
  int16_t top_e[kMaxExperts];
  unsigned long long group[kMaxGroups];
  double best[2][kMaxGroups];
  double part[8];
  double val[kMaxTopK];
  int idx[kMaxTopK];
};

// The block's largest value (SUM: sum) of v over 256 threads, in a fixed order.
template <bool SUM, typename Sync>
__device__ __noinline__ double block_reduce(double v, double* part, int tid, Sync sync) {
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    const double o = __shfl_xor_sync(kFull, v, off);
    v = SUM ? v + o : fmax(v, o);
  }
  if ((tid & 31) == 0) part[tid >> 5] = v;
  sync();
  v = part[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) v = SUM ? v + part[i] : fmax(v, part[i]);
  sync();
  return v;
}

// Token t's experts and gates from its binary64 logits (definitions in router.cu), by 256 threads,
// an expert each: an expert's place is the number of better keys, counted over shared memory, first
// in its warp, then for each warp's k best among those of all. `bias` is the thread's expert's. One
// warp walking top-k rounds with eight experts a lane took 49 us at E = 256: its code does not fit
// the instruction cache, and a block runs it once. The counts are free of branches: with a short-
// circuit the lanes of a tie test ran one by one.
template <typename Sync>
__device__ void decide_token(const DecodeArgs& a, int t, float bias, DecideScratch* sc, int tid, Sync sync) {
  const int e = tid;
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
  sync();
  if (a.G > 1) {
    // the two best of each group, then the groups by their sum (ties: the lower group)
    const int per = a.E / a.G, g = e / per;
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
    sync();
    if (live) {
      const unsigned long long mine = sc->group[g];
      int better = 0;
      for (int h = 0; h < a.G; ++h) better += (sc->group[h] > mine) | ((sc->group[h] == mine) & (h < g));
      if (better >= a.topk_group) sc->key[e] = key = 0ull;
    }
    sync();
  }
  if (a.score_fn == MOE_SCORE_SOFTMAX) {
    const double m = block_reduce<false>(live ? l : -INFINITY, sc->part, tid, sync);
    score = live ? exp(l - m) : 0.0;
    const double z = block_reduce<true>(score, sc->part, tid, sync);
    if (live) score /= z;  // (a quotient of 0 takes the division's slow path, ten times as long)
  }
  {
    const int w0 = tid & ~31, per_warp = min(a.k, 32);
    int better = 0;
    if (w0 < a.E) {
#pragma unroll 8
      for (int f = 0; f < 32; ++f) {
        const unsigned long long o = sc->key[w0 + f];
        better += (o > key) | ((o == key) & (w0 + f < e));
      }
    } else {
      better = tid & 31;
    }
    if (better < per_warp) {  // experts past E and groups left out come last, with key 0
      sc->top[(w0 >> 5) * per_warp + better] = key;
      sc->top_e[(w0 >> 5) * per_warp + better] = (int16_t)e;
    }
    sync();
    if (key && better < per_warp) {
      const int count = (a.E + 31) / 32 * per_warp;
      better = 0;
#pragma unroll 8
      for (int f = 0; f < count; ++f) {
        const unsigned long long o = sc->top[f];
        better += (o > key) | ((o == key) & (sc->top_e[f] < e));
      }
      if (better < a.k) {
        sc->idx[better] = e;
        sc->val[better] = score;
      }
    }
  }
  sync();
  if (tid < 32) {
    const double v = tid < a.k ? sc->val[tid] : 0.0;
    const double denom = a.renorm ? warp_sum(v) : 1.0;
    if (tid < a.k) {
      a.topk_idx[t * a.k + tid] = sc->idx[tid];
      a.topk_w[t * a.k + tid] = (float)(v / denom * (double)a.rsf);  // lanes with a slot only, as above
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

// Built by NT threads (tid 0 .. NT-1, warp 0 among them) from the finished decisions; slot_w and
// slot_r (given: [n * k]) receive each slot's gate and its row. The masks are zero.
template <int NT, typename Sync>
__device__ void build_plan(const DecodeArgs& a, DecodePlan* p, float* slot_w, uint16_t* slot_r, int tid, Sync sync) {
  const int slots = a.n * a.k;
  // the first NT slots stay in registers: most batches have no more
  const int e0 = tid < slots ? __ldcg(a.topk_idx + tid) : -1;
  const float g0 = tid < slots ? __ldcg(a.topk_w + tid) : 0.0f;
  for (int s = tid; s < slots; s += NT) {
    const int e = s == tid ? e0 : __ldcg(a.topk_idx + s);
    atomicOr(&p->mask[e], 1ull << (s / a.k));
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
      const int e = s == tid ? e0 : __ldcg(a.topk_idx + s);
      slot_w[s] = s == tid ? g0 : __ldcg(a.topk_w + s);
      slot_r[s] = (uint16_t)slot_row(*p, e, s / a.k);
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

}  // namespace
}  // namespace moe
