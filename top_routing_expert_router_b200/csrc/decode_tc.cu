// decode_tc.cu -- the layer for few tokens on the tcgen05 tensor cores: bf16 and FP8 experts
// (decode.cuh has the scheme).
//
// The weights are the M side: a tile is two blocks of 128 weight rows (gate and up rows of the same
// 128 hidden columns; 256 output columns of a down matrix) times N token columns, N = the tokens
// rounded up to 16. D0 and D1, 128 x N binary32 each in TMEM, hold a token per column, so a gate/up
// tile multiplies every token of the batch and stores the columns of the expert's tokens: no row is
// gathered and no operand is padded to 128 rows. bf16 experts keep h as the sum of two bf16 rows (16 bits:
// y then carries one rounding, where one bf16 row made its error 1.4 times as large); the two are columns
// side by side of a down tile's MMA, added in the epilogue, and the weights are read once. (silu's __expf is within
// 2^-19 of itself for |g| < 20, below h's 16 bits.) At N <= 64 the MMAs take under a tenth of the time the weights
// take to arrive. Layers of large matrices are bound by HBM (DeepSeek-V3 and Mixtral shapes: 0.97 to 1.02 of the copy
// rate from four tokens on, 0.77 to 0.89 at one). Small and medium ones are not: a tile then costs its hand-overs and
// an epilogue that grows with the tokens and not with the bytes (38 tokens, four FP8 experts of 1408 x 3584: 73 us for
// 9 us of bytes; 64 tokens, 64 bf16 experts of 1408 x 2048: 216 for 174).
//
// One CTA per SM, 384 threads, warp-specialised:
//   warp 0      claims tiles and copies their weights (TMA, 128-byte swizzle) into a ring of 32 KB
//               stages, running ahead of everything else: at the turn from gate/up to down tiles the
//               ring already holds down weights while other CTAs finish h.
//   warp 2      copies the token operand of each stage (x, or h once its expert's gate/up tiles are
//               finished) and, for FP8, writes the stage's scale words.
//   warp 1      owns TMEM and issues the MMAs; tcgen05.commit frees stages.
//   warps 4-7   routing decisions and the plan, then the epilogue: SwiGLU and h (FP8: its E4M3 tile, whose 128 columns are
//               the tile's 128 lanes) or the down tile's rows, and at last the combine.
//   warps 8-11  routing decisions and the plan.
// The shared experts' tiles need no routing and come first, so the weights stream while tokens are
// decided. FP8 scales ride in the MMA (kind::mxf8f6f4.block_scale): one scale word holds four 128-wide
// k blocks, so every fourth stage carries scale words, copied into TMEM by tcgen05.cp.
#include <cuda.h>
#include <limits.h>

#include "decode.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kThreads = 384;
constexpr int kRouterWarps = 8, kRouterThreads = 32 * kRouterWarps;  // warps 4..11
static_assert(kRouterThreads == kMaxExperts, "a router thread per expert");
constexpr int kRows = 128;                  // weight rows of an MMA
constexpr int kKB = 128;                    // bytes of k per stage and row
constexpr int kABytes = kRows * kKB;        // one weight block
constexpr int kSfBytes = 512;
constexpr int kColumns = 2 * kRows;         // output columns of a down tile
constexpr int kCombineTokens = 8;           // tokens of a combine unit
constexpr int kMaxStages = 8;
constexpr int kQueue = 4;                   // tiles published ahead of the slowest reader
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfCol0 = 256;           // FP8: after two pairs of accumulators of at most 64 columns (bf16: of 128)
constexpr uint32_t kSfCols = 12;            // per slot: D0's rows, D1's rows, the tokens
constexpr size_t kSmemLimit = 232448;
// Few experts leave few tiles for the SMs, and one SM draws at most about 65 GB/s, so tiles are cut along
// k. A part of a gate/up tile costs a round trip through L2; down tiles join their parts in the combine.
// Gate/up: at most as many parts as keep them within one turn of the SMs, each of at least what the ring
// holds, kMinPart k blocks; from three quarters of a turn to eight turns, halves (past one turn only of tiles
// of twice kLongPart k blocks or more: 264 tiles of 32 blocks take 85 us whole, 88 halved). Fewer for many
// tokens, whose parts one block joins (gate_parts): 55 tokens and 2 shared tiles of 110 blocks 145 us in 16
// parts, 87 in four; 59 tokens and 18 shared tiles of 17 blocks 89 us in two, 72 whole.
// Down: parts within two turns, of at least kMinPart blocks, or three turns in at most kWideParts parts of
// twice kMinPart (64 tiles of 44 blocks: 65 us in four parts, 68 in six); halves from one to two turns.
// Measured, one token unless said: 16 gate/up tiles 81 us whole, 40.5 in nine parts; 96 tiles 66.8 us
// whole, 76.4 halved; 128 tiles and 252 down tiles (DeepSeek-V3 shapes, FP8) 79 us with both halved, 83 with
// either whole; 224 gate/up tiles (Mixtral shapes) 132 us whole, 121 halved, 131 in three; its 32 down
// tiles of 7.3 MB 200 us whole, 121 in nine parts; 160 and 80 tiles (d = 4096, five experts of 4096) 111 us
// whole and in three, 94 halved and in five; 896 and 128 tiles (Mixtral, 4 tokens) 337 us whole and
// halved, 321 halved and in three.
constexpr int kSms = 148, kMinPart = 6, kMaxParts = 16, kLongPart = 20, kWideParts = 9;

struct __align__(16) Ctl {
  uint64_t full[kMaxStages];   // weights' and tokens' arrivals
  uint64_t empty[kMaxStages];
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];
  uint64_t tile_full[kQueue];
  uint64_t tile_empty[kQueue];  // read by the MMA, the token producer and four epilogue warps
  uint64_t plan_ready;
  uint64_t drain;
  int32_t tile[kQueue];
  uint32_t tmem_base;
  int32_t abort;
  uint32_t armed[2];           // stages that the weight and the token warp have armed, written as they leave
  int32_t ticket;
  int32_t routed;              // every token's decision was seen
  int32_t last;
  float4 amax[4];              // FP8: a token's largest |h| per epilogue warp, four tokens at a time
  int32_t sel_e[kSelfTokens * kMaxTopK];  // the block's own decisions
  float sel_w[kSelfTokens * kMaxTopK];
  DecideScratch decide;
  DecodePlan plan;
};

struct DecodeMaps {
  CUtensorMap gate, up, down, sgate, sup, sdown, x, h, hs;
};

struct TcShape {
  int32_t n_cols;       // token columns: n rounded up to 16
  int32_t stages;
  int32_t stage_bytes;
  int32_t sf_off;       // bytes from the ring to the stages' scale words (FP8)
  int32_t slot_off;     // to the combine's slots
  int32_t ctl_off;
};

__device__ __noinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, Ctl* ctl, int32_t* ctr, moe_diag* st, int64_t limit) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try(b, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try(b, parity)) return true;
    if ((it & 255u) == 0) {
      if (*reinterpret_cast<volatile int32_t*>(&ctl->abort)) return false;
      if (clock64() - t0 > limit) {
        atomicExch(&ctl->abort, 1);
        atomicExch(ctr + kCtrAbort, 1);
        set_status(st, MOE_ERR_TIMEOUT);
        return false;
      }
    }
  }
}

__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// kind::f16 (bf16 A and B) and kind::mxf8f6f4 (E4M3, UE8M0 scales; scale byte `id` of the words)
// instruction descriptors: binary32 D, K-major operands, M = 128, N = n.
__device__ __forceinline__ uint32_t idesc_bf16(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}
__device__ __forceinline__ uint32_t idesc_fp8(int n, int id) {
  return ((uint32_t)id << 4) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(kRows >> 4) << 24) |
         ((uint32_t)id << 29);
}
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)
      : "memory");
}
__device__ __forceinline__ void sf_copy(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// A weight tile's copy: each weight is read once a call, so its lines leave L2 first and the rest
// (instructions, x, h, router weights) stays.
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_2d_hint(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t c0, int32_t c1,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4}], "
      "[%2], %5;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}

// Orders generic writes before, and async-proxy (TMA) reads after, across the release/acquire pair between them.
__device__ __forceinline__ void fence_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// Barrier of COUNT threads. bar.sync wants whole warps: lanes that left a loop apart meet first.
template <int ID, int COUNT>
__device__ __forceinline__ void named_sync() {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "n"(COUNT) : "memory");
}

// Four columns of each of two accumulators (32 lanes).
__device__ __forceinline__ void tmem_ld4x2(uint32_t a0, uint32_t a1, float (&v0)[4], float (&v1)[4]) {
  uint32_t x[4], y[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
               : "r"(a0));
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
               : "r"(a1));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v0[i] = __uint_as_float(x[i]);
    v1[i] = __uint_as_float(y[i]);
  }
}

// Barrier of COUNT threads that tells each whether all of them came with `v`.
template <int ID, int COUNT>
__device__ __forceinline__ bool named_and(bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(ID), "n"(COUNT)
      : "memory");
  return r != 0;
}

// A tile's place in the layer.
struct Tile {
  int e;        // expert, or E for the shared ones
  int r0;       // first weight row (down: output column) of the tile
  int down;
  int Ie;       // hidden width of the expert
  int part, parts;  // which part of the k axis, of how many
  int kb0, kb1; // its k blocks
  int row0, m;  // the expert's token rows: slots row0 .. row0 + m (shared: every token)
  unsigned long long mask;
};

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 1) decode_tc_kernel(const __grid_constant__ DecodeMaps maps,
                                                               const __grid_constant__ DecodeArgs a,
                                                               const __grid_constant__ TcShape sh) {
  constexpr int KE = FP8 ? 128 : 64;  // elements of k per stage
  constexpr int HR = FP8 ? 1 : 2;     // rows of h for a token's slot
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + sh.ctl_off);
  float* slot_w = reinterpret_cast<float*>(smem + sh.slot_off);           // [n * k] gates
  uint16_t* slot_r = reinterpret_cast<uint16_t*>(slot_w + a.n * a.k);     // [n * k] expert output rows
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int N = sh.n_cols, stages = sh.stages;
  const uint32_t dcols = (uint32_t)(N * HR);  // columns of an accumulator
  const int shared = a.Is > 0;
  const int tiles1 = (a.I + kRows - 1) / kRows, tiles1s = (a.Is + kRows - 1) / kRows;
  const int tiles2 = (a.d + kColumns - 1) / kColumns;

  if (threadIdx.x == 0) {
    ctl->abort = 0;
    for (int s = 0; s < stages; ++s) {
      mbar_init(&ctl->full[s], 2);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&ctl->tmem_full[b], 1);
      mbar_init(&ctl->tmem_empty[b], 4);
    }
    for (int q = 0; q < kQueue; ++q) {
      mbar_init(&ctl->tile_full[q], 1);
      mbar_init(&ctl->tile_empty[q], 6);
    }
    mbar_init(&ctl->plan_ready, kRouterWarps);
    mbar_init(&ctl->drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 3 && lane < 9)  // the first copies do not wait for their descriptors
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.gate + lane)) : "memory");
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl->tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem_base = ctl->tmem_base;
  wait_for_earlier_kernels();

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return mbar_try(smem_u32(bar), parity) || mbar_wait(bar, parity, ctl, a.ctr, a.status, a.wait_cycles);
  };
  const int count1 = tiles1 * a.cut.s1, count1s = tiles1s * a.cut.s1s;  // an expert's gate/up tiles, parts counted
  const int count2 = tiles2 * a.cut.s2, count2s = shared * tiles2 * a.cut.s2s;
  auto tile_of = [&](int t) {
    Tile tl;
    const int first2 = t < count1s ? INT_MAX : count1s + ctl->plan.n_act * count1;  // the plan is ready past the first tiles
    tl.down = t >= first2;
    int u, local, parts, per;
    if (tl.down) {
      local = t - first2;
      u = local < count2s ? -1 : (local - count2s) / count2;
      local = u < 0 ? local : (local - count2s) % count2;
      parts = u < 0 ? a.cut.s2s : a.cut.s2;
      per = u < 0 ? a.cut.per2s : a.cut.per2;
      tl.r0 = local / parts * kColumns;
    } else {
      u = t < count1s ? -1 : (t - count1s) / count1;
      local = u < 0 ? t : (t - count1s) % count1;
      parts = u < 0 ? a.cut.s1s : a.cut.s1;
      per = u < 0 ? a.cut.per1s : a.cut.per1;
      tl.r0 = local / parts * kRows;
    }
    tl.part = local % parts;
    tl.parts = parts;
    tl.e = u < 0 ? a.E : ctl->plan.act[u];
    tl.Ie = u < 0 ? a.Is : a.I;
    tl.kb0 = tl.part * per;
    tl.kb1 = min(tl.kb0 + per, ((tl.down ? tl.Ie : a.d) + KE - 1) / KE);
    tl.mask = u < 0 ? token_mask(a.n) : ctl->plan.mask[tl.e];
    tl.row0 = u < 0 ? 0 : ctl->plan.off[tl.e];
    tl.m = __popcll(tl.mask);
    return tl;
  };
  // Whether a tile's second weight block has any row.
  auto two_blocks = [&](const Tile& tl) { return !tl.down || tl.r0 + kRows < a.d; };
  // Token columns of a tile: all of them, or a routed down tile's own rows.
  auto columns = [&](const Tile& tl) { return tl.down && tl.e < a.E ? (tl.m + 15) & ~15 : N; };

  if (warp == 0) {
    // ================= weights =================
    if (lane == 0) {
      int stage = 0, q = 0;
      uint32_t phase = 0, qphase = 0, armed = 0;
      bool ok = true;
      const uint64_t policy = evict_first_policy();
      int total = INT_MAX, next = atomicAdd(a.ctr + kCtrTile, 1);
      while (ok) {
        const int t = next;
        if (t >= count1s && total == INT_MAX) {
          if (!(ok = wait(&ctl->plan_ready, 0))) break;
          total = count1s + count2s + ctl->plan.n_act * (count1 + count2);
        }
        if (!(ok = wait(&ctl->tile_empty[q], qphase ^ 1u))) break;
        ctl->tile[q] = t < total ? t : -1;
        mbar_arrive(&ctl->tile_full[q]);
        if (++q == kQueue) q = 0, qphase ^= 1u;
        if (t >= total) break;
        next = atomicAdd(a.ctr + kCtrTile, 1);
        const Tile tl = tile_of(t);
        const bool s = tl.e == a.E, two = two_blocks(tl);
        const CUtensorMap* m0 = tl.down ? (s ? &maps.sdown : &maps.down) : (s ? &maps.sgate : &maps.gate);
        const CUtensorMap* m1 = tl.down ? m0 : (s ? &maps.sup : &maps.up);
        const int y0 = (s ? 0 : tl.e * (tl.down ? a.d : a.I)) + tl.r0, y1 = tl.down ? y0 + kRows : y0;
        for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
          if (!(ok = wait(&ctl->empty[stage], phase ^ 1u))) break;
          uint8_t* sa = smem + stage * sh.stage_bytes;
          mbar_expect_tx(&ctl->full[stage], two ? 2 * kABytes : kABytes);
          tma_load_2d_hint(sa, m0, &ctl->full[stage], kb * KE, y0, policy);
          if (two) tma_load_2d_hint(sa + kABytes, m1, &ctl->full[stage], kb * KE, y1, policy);
          ++armed;
          if (++stage == stages) stage = 0, phase ^= 1u;
        }
      }
      ctl->armed[0] = armed;
    }
  } else if (warp == 1) {
    // ================= MMA =================
    if (lane == 0) {
      int stage = 0, q = 0, i = 0;
      uint32_t phase = 0, qphase = 0;
      [[maybe_unused]] uint32_t sf_slot = 0;  // FP8: scale words of four k blocks, two slots in turn
      bool ok = true;
      for (;; ++i) {
        if (!(ok = wait(&ctl->tile_full[q], qphase))) break;
        const int t = ctl->tile[q];
        if (t < 0) break;
        const Tile tl = tile_of(t);
        mbar_arrive(&ctl->tile_empty[q]);
        if (++q == kQueue) q = 0, qphase ^= 1u;
        const int buf = i & 1;
        if (!(ok = wait(&ctl->tmem_empty[buf], ((uint32_t)(i >> 1) & 1u) ^ 1u))) break;
        fence_after();
        const uint32_t d0 = tmem_base + buf * 2 * dcols, d1 = d0 + dcols;
        const bool two = two_blocks(tl);
        const int cols = columns(tl) * (tl.down ? HR : 1);
        for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
          if (!(ok = wait(&ctl->full[stage], phase))) break;
          fence_after();
          const uint32_t sa = smem_u32(smem + stage * sh.stage_bytes);
          const uint64_t a0 = sw128_desc(sa), a1 = sw128_desc(sa + kABytes), b = sw128_desc(sa + 2 * kABytes);
          if constexpr (FP8) {
            if ((kb & 3) == 0) sf_slot ^= 1u;
            const uint32_t sf = tmem_base + kSfCol0 + kSfCols * sf_slot;
            if ((kb & 3) == 0) {
              const uint32_t ss = smem_u32(smem + sh.sf_off + stage * 3 * kSfBytes);
              sf_copy(sf, sf_desc(ss));
              sf_copy(sf + 4, sf_desc(ss + kSfBytes));
              sf_copy(sf + 8, sf_desc(ss + 2 * kSfBytes));
            }
            const uint32_t id = idesc_fp8(cols, kb & 3);
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // 32 codes = 32 bytes
              mma_fp8(d0, a0 + (uint64_t)(2 * k), b + (uint64_t)(2 * k), id, sf, sf + 8, ((kb - tl.kb0) | k) != 0);
              if (two) mma_fp8(d1, a1 + (uint64_t)(2 * k), b + (uint64_t)(2 * k), id, sf + 4, sf + 8, ((kb - tl.kb0) | k) != 0);
            }
          } else {
            const uint32_t id = idesc_bf16(cols);
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // 16 bf16 = 32 bytes
              mma_bf16(d0, a0 + (uint64_t)(2 * k), b + (uint64_t)(2 * k), id, ((kb - tl.kb0) | k) != 0);
              if (two) mma_bf16(d1, a1 + (uint64_t)(2 * k), b + (uint64_t)(2 * k), id, ((kb - tl.kb0) | k) != 0);
            }
          }
          mma_commit(&ctl->empty[stage]);
          if (++stage == stages) stage = 0, phase ^= 1u;
        }
        if (!ok) break;
        mma_commit(&ctl->tmem_full[buf]);
      }
    }
  } else if (warp == 2) {
    // ================= tokens (and FP8 scale words) =================
    int stage = 0, q = 0;
    uint32_t phase = 0, qphase = 0, armed = 0;
    auto all = [&](bool v) { return __shfl_sync(kFull, (int)v, 0) != 0; };
    for (;;) {
      if (!all(lane != 0 || wait(&ctl->tile_full[q], qphase))) break;
      __syncwarp();
      const int t = *reinterpret_cast<volatile int32_t*>(&ctl->tile[q]);
      if (t < 0) break;
      const Tile tl = tile_of(t);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->tile_empty[q]);
      if (++q == kQueue) q = 0, qphase ^= 1u;
      bool ok = true;
      if (lane == 0) {
        if (tl.down) ok = wait_counter(a.ctr + kCtrExpert + tl.e, tl.e == a.E ? tiles1s : tiles1, a.ctr, a.status, a.wait_cycles);  // its h
        fence_async_global();
        if (!ok) atomicExch(&ctl->abort, 1);
      }
      if (!all(ok)) break;
      __syncwarp();  // lane 0's acquire comes before every lane's reads of h's scale bytes: a shuffle orders no memory
      const bool s = tl.e == a.E;
      const CUtensorMap* m = !tl.down ? &maps.x : (s ? &maps.hs : &maps.h);
      const int cols = columns(tl), nkb = (tl.down ? tl.Ie : a.d) / KE;  // FP8: scale bytes per row
      // scale bytes: rows of the token operand, and the two weight blocks
      const uint8_t *tok = nullptr, *w0 = nullptr, *w1 = nullptr;
      if constexpr (FP8) {
        if (tl.down) {
          tok = s ? a.hs_scale : a.h_scale + (int64_t)tl.row0 * nkb;
          w0 = (s ? a.ss_down : a.s_down + (int64_t)tl.e * (a.d / 128) * nkb) + (int64_t)(tl.r0 / 128) * nkb;
          w1 = two_blocks(tl) ? w0 + nkb : w0;
        } else {
          tok = a.xs;
          const int64_t at = (s ? 0 : (int64_t)tl.e * (a.I / 128) * nkb) + (int64_t)(tl.r0 / 128) * nkb;
          w0 = (s ? a.ss_gate : a.s_gate) + at;
          w1 = (s ? a.ss_up : a.s_up) + at;
        }
      }
      const int rows = tl.down && !s ? tl.m : a.n;
      auto word = [&](const uint8_t* p, int kb, bool own) {  // scale bytes of k blocks kb .. kb + 3
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (kb + j < nkb) w |= (uint32_t)(own ? __ldcg(p + kb + j) : __ldg(p + kb + j)) << (8 * j);
        return w;
      };
      uint32_t wt0 = 0, wt1 = 0, ww0 = 0, ww1 = 0;
      auto fetch = [&](int kb) {  // lane l holds token rows l and l + 32
        if (kb >= tl.kb1) return;
        wt0 = lane < rows ? word(tok + (int64_t)lane * nkb, kb, true) : 0u;
        wt1 = lane + 32 < rows ? word(tok + (int64_t)(lane + 32) * nkb, kb, true) : 0u;
        ww0 = word(w0, kb, false);
        ww1 = word(w1, kb, false);
      };
      if constexpr (FP8) fetch(tl.kb0);
      for (int kb = tl.kb0; kb < tl.kb1; ++kb) {
        if (!all(lane != 0 || wait(&ctl->empty[stage], phase ^ 1u))) {
          ok = false;
          break;
        }
        uint8_t* sb = smem + stage * sh.stage_bytes + 2 * kABytes;
        if (FP8 && (kb & 3) == 0) {
          uint4* sf = reinterpret_cast<uint4*>(smem + sh.sf_off + stage * 3 * kSfBytes);
          sf[lane] = make_uint4(ww0, ww0, ww0, ww0);
          sf[32 + lane] = make_uint4(ww1, ww1, ww1, ww1);
          sf[64 + lane] = make_uint4(wt0, wt1, 0u, 0u);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          fetch(kb + 4);
        }
        __syncwarp();
        if (lane == 0) {
          const int parts = tl.down ? HR : 1, apart = s ? a.n : a.n * a.k;  // rows of h between a slot's two
          mbar_expect_tx(&ctl->full[stage], (uint32_t)(parts * cols) * kKB);
          ++armed;
          for (int p = 0; p < parts; ++p) {
            if (tl.down && !s)
              for (int c = 0; c < cols; c += 16)
                tma_load_2d(sb + (p * cols + c) * kKB, m, &ctl->full[stage], kb * KE, p * apart + tl.row0 + c);
            else
              tma_load_2d(sb + p * cols * kKB, m, &ctl->full[stage], kb * KE, p * apart);
          }
        }
        if (++stage == stages) stage = 0, phase ^= 1u;
      }
      if (!ok) break;
    }
    if (lane == 0) ctl->armed[1] = armed;
  } else if (warp >= 4) {
    // ================= router =================
    const int tid = threadIdx.x - 128, rw = warp - 4;
    auto sync = [] { named_sync<1, kRouterThreads>(); };
    ctl->plan.mask[tid] = 0ull;
    const float bias = a.bias && tid < a.E ? __ldg(a.bias + tid) : 0.0f;
    const bool self = a.n <= kSelfTokens;
    bool ok = true;
    if (self) {
      for (int t = 0; t < a.n; ++t)
        decide_token(a, t, bias, &ctl->decide, tid, sync, ctl->sel_e + t * a.k, ctl->sel_w + t * a.k);
      if (blockIdx.x == 0 && tid < a.n * a.k) a.topk_idx[tid] = ctl->sel_e[tid], a.topk_w[tid] = ctl->sel_w[tid];
    } else {
      for (;;) {
        if (tid == 0) ctl->ticket = atomicAdd(a.ctr + kCtrToken, 1);
        sync();
        const int t = ctl->ticket;
        if (t >= a.n) break;
        decide_token(a, t, bias, &ctl->decide, tid, sync, a.topk_idx + t * a.k, a.topk_w + t * a.k);
        if (tid == 0) add_release(a.ctr + kCtrTokenDone, 1);  // decide_token ends with a barrier
      }
      if (tid == 0) {
        ctl->routed = wait_counter(a.ctr + kCtrTokenDone, a.n, a.ctr, a.status, a.wait_cycles);
        if (!ctl->routed) atomicExch(&ctl->abort, 1);
      }
      sync();
      ok = ctl->routed != 0;  // one answer for all: the barriers below count every router warp
    }
    if (ok) {
      build_plan<kRouterThreads>(a, self ? ctl->sel_e : a.topk_idx, self ? ctl->sel_w : a.topk_w, &ctl->plan, slot_w, slot_r, tid,
                                 sync);
      sync();
      if (lane == 0) mbar_arrive(&ctl->plan_ready);
      if (blockIdx.x == 0 && rw >= 4) write_counts<kRouterThreads - 128>(a, ctl->plan, tid - 128);
    }
    if (ok && rw < 4) {
      // ================= epilogue (warps 4..7) =================
      const int r = rw * 32 + lane;  // weight row of the tile: TMEM lane (quarter rw = warp % 4)
      int q = 0, i = 0;
      uint32_t qphase = 0;
      // Combine: y of 256 columns and eight tokens a unit: each slot's parts in order, the slots in order,
      // the shared experts last. Four columns a thread, two tokens at once. For a few tokens the block
      // that finishes a column range adds it at once (Mixtral shapes n=1: 132 us a call, 133.4 otherwise); for
      // more, the units are spread over the blocks after their tiles (nobody waits for a unit, so each
      // block has its own): with one block adding all tokens of a range, 64 tokens took 28 SMs about 30 us
      // after the last weight had arrived.
      const bool few = a.n <= 4;
      const int chunks = (a.n + kCombineTokens - 1) / kCombineTokens;
      const int parts = ctl->plan.n_act * a.cut.s2 + shared * a.cut.s2s;  // down tiles of a column range
      bool tiles_left = true;
      int unit = few ? INT_MAX : (int)blockIdx.x;
      for (;;) {
        int u;
        if (tiles_left) {
          const int buf = i & 1;
          bool go = wait(&ctl->tile_full[q], qphase);
          const int t = go ? *reinterpret_cast<volatile int32_t*>(&ctl->tile[q]) : 0;
          if (go && t >= 0) go = wait(&ctl->tmem_full[buf], (uint32_t)(i >> 1) & 1u);
          // one answer for the four warps: the barriers below count all of them
          if (!named_and<2, 128>(go)) break;
          if (t < 0) {
            tiles_left = false;
            continue;
          }
          ++i;
          const Tile tl = tile_of(t);
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->tile_empty[q]);
          if (++q == kQueue) q = 0, qphase ^= 1u;
          fence_after();
          const uint32_t d0 = tmem_base + ((uint32_t)(rw * 32) << 16) + buf * 2 * dcols, d1 = d0 + dcols;
          const bool s = tl.e == a.E;
          auto release = [&] {  // the accumulators are read
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->tmem_empty[buf]);
          };
          // what the four warps wrote is visible to whoever sees the count (the barrier puts it before
          // thread 0's release, which is cumulative; a fence in every thread cost 2 us a call); true for
          // the count's last
          auto count = [&](int32_t* p, int target) {
            fence_async_global();  // h is read by TMA
            named_sync<2, 128>();
            if (r == 0) ctl->last = add_release(p, 1) + 1 == target;
            named_sync<2, 128>();
            return ctl->last != 0;
          };
          if (!tl.down) {
            const int c = tl.r0 + r;  // hidden column
            float* part = a.gu + (s ? (int64_t)a.n * a.k * a.cut.s1 * 2 * a.I : 0);  // [rows, parts, 2, Ie]
            if (tl.parts > 1) {
              int row = tl.row0;
              for (int t0 = 0; t0 < N; t0 += 4) {
                const uint32_t mine = (uint32_t)(tl.mask >> t0) & 15u;
                if (!mine) continue;
                float g[4], u[4];
                tmem_ld4x2(d0 + (uint32_t)t0, d1 + (uint32_t)t0, g, u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  if (!((mine >> j) & 1u)) continue;
                  float* o = part + ((int64_t)row++ * tl.parts + tl.part) * 2 * tl.Ie + c;
                  if (c < tl.Ie) o[0] = g[j], o[tl.Ie] = u[j];
                }
              }
              release();
              // the block that brings a tile's last part adds the parts, in order, and goes on with the sums
              if (!count(a.ctr + kCtrExpert + a.E + 1 + (a.d + kMinColumns - 1) / kMinColumns + tl.e * tiles1 + tl.r0 / kRows,
                         tl.parts))
                continue;
            }
            int row = tl.row0;
            for (int t0 = 0; t0 < N; t0 += 4) {  // four at a time: more, unrolled, missed the instruction cache
              const uint32_t mine = (uint32_t)(tl.mask >> t0) & 15u;
              if (!mine) continue;
              float g[4], u[4];
              if (tl.parts > 1) {
                // the four tokens' parts, four at a time: 32 loads in flight (a token after the other took about
                // a microsecond each: 29 tokens, five experts and a shared one in four parts 70 us, 54 so)
                const float* o[4];
                bool on[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  g[j] = u[j] = 0.0f;
                  on[j] = ((mine >> j) & 1u) && c < tl.Ie;
                  o[j] = part + (int64_t)(row + __popc(mine & ((1u << j) - 1u))) * tl.parts * 2 * tl.Ie + c;
                }
                for (int p0 = 0; p0 < tl.parts; p0 += 4) {
                  float vg[4][4], vu[4][4];
#pragma unroll
                  for (int p = 0; p < 4; ++p)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                      const bool in = on[j] && p0 + p < tl.parts;
                      vg[p][j] = in ? __ldcg(o[j] + (int64_t)(p0 + p) * 2 * tl.Ie) : 0.0f;
                      vu[p][j] = in ? __ldcg(o[j] + (int64_t)(p0 + p) * 2 * tl.Ie + tl.Ie) : 0.0f;
                    }
#pragma unroll
                  for (int p = 0; p < 4; ++p)
#pragma unroll
                    for (int j = 0; j < 4; ++j) g[j] += vg[p][j], u[j] += vu[p][j];
                }
              } else {
                tmem_ld4x2(d0 + (uint32_t)t0, d1 + (uint32_t)t0, g, u);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) g[j] = silu(g[j]) * u[j];
              if constexpr (FP8) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  if (!((mine >> j) & 1u)) continue;
                  g[j] = to_f32(from_f32<bf16>(g[j]));
                  const float v = fabsf(g[j]);  // a NaN is left out of the maximum
                  const unsigned top = __reduce_max_sync(kFull, v >= 0.0f ? __float_as_uint(v) : 0u);
                  if (lane == 0) reinterpret_cast<float*>(&ctl->amax[j])[rw] = __uint_as_float(top);
                }
                named_sync<2, 128>();
                uint8_t* hq = static_cast<uint8_t*>(s ? a.hs : a.h);
                uint8_t* hb = s ? a.hs_scale : a.h_scale;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  if (!((mine >> j) & 1u)) continue;
                  const float4 m4 = ctl->amax[j];
                  const int e = ue8m0_exponent(fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w)));
                  hq[(int64_t)row * tl.Ie + c] = (uint8_t)__nv_cvt_float_to_fp8(g[j] * pow2_neg(e), __NV_SATFINITE, __NV_E4M3);
                  if (r == 0) hb[(int64_t)row * (tl.Ie / 128) + tl.r0 / 128] = (uint8_t)(e + 127);
                  ++row;
                }
                named_sync<2, 128>();  // amax is the next columns'
              } else {
                bf16* h = static_cast<bf16*>(s ? a.hs : a.h);
                bf16* h2 = h + (int64_t)(s ? a.n : a.n * a.k) * tl.Ie;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  if (!((mine >> j) & 1u)) continue;
                  const bf16 top = from_f32<bf16>(g[j]);
                  const float rest = fabsf(to_f32(top)) < INFINITY ? g[j] - to_f32(top) : 0.0f;
                  if (c < tl.Ie) {
                    h[(int64_t)row * tl.Ie + c] = top;
                    h2[(int64_t)row * tl.Ie + c] = from_f32<bf16>(rest);
                  }
                  ++row;
                }
              }
            }
            if (tl.parts == 1) release();
            count(a.ctr + kCtrExpert + tl.e, INT_MAX);
            continue;
          }
          {
            const int64_t rows = s ? a.n : (int64_t)a.n * a.k;
            float* out = (s ? a.es : a.eo) + (tl.part * rows + tl.row0) * a.d;
            const bool two = two_blocks(tl);
            for (int t0 = 0; t0 < tl.m; t0 += 4) {
              float v0[4], v1[4];
              tmem_ld4x2(d0 + (uint32_t)t0, (two ? d1 : d0) + (uint32_t)t0, v0, v1);
              if constexpr (HR == 2) {
                float u0[4], u1[4];
                const uint32_t at = (uint32_t)(columns(tl) + t0);
                tmem_ld4x2(d0 + at, (two ? d1 : d0) + at, u0, u1);
#pragma unroll
                for (int j = 0; j < 4; ++j) v0[j] += u0[j], v1[j] += u1[j];
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if (t0 + j >= tl.m) break;
                float* o = out + (int64_t)(t0 + j) * a.d + tl.r0 + r;
                if (tl.r0 + r < a.d) o[0] = v0[j];
                if (tl.r0 + kRows + r < a.d) o[kRows] = v1[j];
              }
            }
          }
          release();
          if (!count(a.ctr + kCtrExpert + a.E + 1 + tl.r0 / kColumns, parts) || !few) continue;
          u = tl.r0 / kColumns;
        } else {
          if (unit >= tiles2 * chunks) break;
          u = unit;
          unit += gridDim.x;
          bool done = true;
          if (r == 0) done = wait_counter(a.ctr + kCtrExpert + a.E + 1 + u % tiles2, parts, a.ctr, a.status, a.wait_cycles);
          if (!named_and<2, 128>(done)) break;
        }
        const int c = u % tiles2 * kColumns + 4 * (r & 63);
        if (c >= a.d) continue;
        const int64_t nk = (int64_t)a.n * a.k;
        const int first = u / tiles2 * kCombineTokens, end = min(a.n, first + kCombineTokens);
        for (int ta = first + (r >> 6); ta < end; ta += 4) {
          const int tb = ta + 2;
          const bool two = tb < end;
          float4 ya = make_float4(0.0f, 0.0f, 0.0f, 0.0f), yb = ya;
          auto add = [&](float4& y, const float* p, float w) {
            const float4 o = __ldcg(reinterpret_cast<const float4*>(p));
            y.x = fmaf(w, o.x, y.x);
            y.y = fmaf(w, o.y, y.y);
            y.z = fmaf(w, o.z, y.z);
            y.w = fmaf(w, o.w, y.w);
          };
          int j = 0, p = 0;
#pragma unroll 8
          for (int i2 = 0; i2 < a.k * a.cut.s2; ++i2) {
            add(ya, a.eo + (p * nk + slot_r[ta * a.k + j]) * a.d + c, slot_w[ta * a.k + j]);
            if (two) add(yb, a.eo + (p * nk + slot_r[tb * a.k + j]) * a.d + c, slot_w[tb * a.k + j]);
            if (++p == a.cut.s2) p = 0, ++j;
          }
          if (shared) {
#pragma unroll 4
            for (p = 0; p < a.cut.s2s; ++p) {
              add(ya, a.es + ((int64_t)p * a.n + ta) * a.d + c, 1.0f);
              if (two) add(yb, a.es + ((int64_t)p * a.n + tb) * a.d + c, 1.0f);
            }
          }
          auto store = [&](int t, const float4& y) {
            __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(static_cast<bf16*>(a.y) + (int64_t)t * a.d + c);
            o[0] = __floats2bfloat162_rn(y.x, y.y);
            o[1] = __floats2bfloat162_rn(y.z, y.w);
          };
          store(ta, ya);
          if (two) store(tb, yb);
        }
      }
    }
  }

  __syncwarp();  // lanes that had no part in their warp's work
  fence_before();
  __syncthreads();
  fence_after();
  if (ctl->abort) {
    // An abandoned call: wherever each warp stopped, nothing that writes this block's shared or tensor memory outlives
    // it. Of a stage's two arrivals (weights, tokens) one may be missing: the other's copies land in a phase that its
    // substitute completes. (A stage is armed again only after both came, so the two counts differ by one at most.)
    if (threadIdx.x == 0)
      for (int s = 0; s < stages; ++s) {
        auto fills = [&](uint32_t armed) { return armed > (uint32_t)s ? (armed - 1 - s) / stages + 1 : 0u; };
        const uint32_t w = fills(ctl->armed[0]), t = fills(ctl->armed[1]), most = w > t ? w : t;
        if (w != t) mbar_arrive(&ctl->full[s]);
        if (most) mbar_drain(&ctl->full[s], (most - 1) & 1u);
      }
    if (threadIdx.x == 32) {  // the thread that issued the MMAs
      mma_commit(&ctl->drain);
      mbar_drain(&ctl->drain, 0);
    }
  }
  if (warp == 1) {
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
  }
}

// ---- host side ---------------------------------------------------------------------
// 2-D tensor [rows, cols] (cols contiguous), box [box_rows, 128 bytes], 128-byte swizzle.
bool make_map(CUtensorMap* m, bool fp8, const void* base, int64_t rows, int64_t cols, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const int64_t b = fp8 ? 1 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(cols * b)};
  const cuuint32_t box[2] = {(cuuint32_t)(kKB / b), (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
            strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool FP8>
cudaError_t launch_t(const DecodeArgs& a, const DecodeMaps& maps, const TcShape& sh, int grid, size_t smem, cudaStream_t s) {
  static std::atomic<uint64_t> attr;
  const cudaError_t e = set_smem_limit(attr, (const void*)decode_tc_kernel<FP8>, kSmemLimit);
  if (e != cudaSuccess) return e;
  return launch_early(decode_tc_kernel<FP8>, grid, kThreads, smem, s, maps, a, sh);
}

// A k axis of nkb blocks in about `p` parts, each of at least kMinPart blocks (FP8: of whole scale
// words, four blocks).
void split_k(int64_t p, int64_t nkb, bool fp8, int32_t* parts, int32_t* per) {
  if (p > nkb / kMinPart) p = nkb / kMinPart;
  if (p > kMaxParts) p = kMaxParts;
  if (p < 1) p = 1;
  *per = (int32_t)align_up(nkb > 0 ? ceil_div(nkb, p) : 1, fp8 ? 4 : 1);
  *parts = nkb > 0 ? (int32_t)ceil_div(nkb, *per) : 1;
}

}  // namespace

// Most parts of a gate/up tile when there are `tiles` of nkb blocks.
static int64_t gate_parts_limit(int64_t tiles, int64_t nkb) {
  if (tiles <= 0) return 1;
  const bool halved = tiles >= kSms * 3 / 4 && (tiles < kSms || (tiles < 8 * kSms && nkb >= 2 * kLongPart));
  int64_t p = halved ? 2 : kSms / tiles;
  if (p > nkb / kMinPart) p = nkb / kMinPart;
  if (p > kMaxParts) p = kMaxParts;
  return p > 1 ? p : 1;
}

// Of up to `limit` parts the number that is done first, for a tile of `tokens` rows: in quarters of a
// microsecond, a block of k takes 2, a join 6 and, by fours of tokens and of parts, 4.
static int64_t gate_parts(int64_t limit, int64_t nkb, int64_t tokens) {
  const int64_t fours = ceil_div(tokens, 4);
  int64_t best = 1, least = 2 * nkb;
  for (int64_t p = 2; p <= limit; ++p) {
    const int64_t cost = 2 * nkb / p + 6 + fours * (p > 4 ? p : 4);
    if (cost <= least) best = p, least = cost;
  }
  return best;
}

DecodeSplits decode_splits(int64_t n, int32_t d, int32_t E, int32_t k, int32_t I, int32_t Is, int32_t dtype) {
  DecodeSplits c{1, 0, 1, 0, 1, 0, 1, 0};
  if (dtype == MOE_F32) return c;
  const int64_t ke = dtype == MOE_FP8 ? 128 : 64;
  const int64_t active = n * k < E ? n * k : E;  // experts at most
  const int64_t tiles1 = active * ceil_div(I, kRows), tiles1s = ceil_div(Is, kRows);
  const int64_t tiles2 = (active + (Is > 0)) * ceil_div(d, kColumns);
  const bool fp8 = dtype == MOE_FP8;
  const int64_t kb1 = ceil_div(d, ke);
  split_k(gate_parts(gate_parts_limit(tiles1, kb1), kb1, ceil_div(n * k, active)), kb1, fp8, &c.s1, &c.per1);
  split_k(gate_parts(gate_parts_limit(tiles1s, kb1), kb1, n), kb1, fp8, &c.s1s, &c.per1s);
  auto parts2 = [&](int64_t nkb) {
    const int64_t two = tiles2 >= kSms && tiles2 < 2 * kSms ? 2 : 2 * kSms / tiles2;
    int64_t three = 3 * kSms / tiles2;
    if (three > nkb / (2 * kMinPart)) three = nkb / (2 * kMinPart);
    if (three > kWideParts) three = kWideParts;
    return two > three ? two : three;
  };
  split_k(parts2(ceil_div(I, ke)), ceil_div(I, ke), fp8, &c.s2, &c.per2);
  split_k(parts2(ceil_div(Is, ke)), ceil_div(Is, ke), fp8, &c.s2s, &c.per2s);
  return c;
}

// Fewer tokens may be cut into more parts, so each count is the most that any call of up to n tokens
// has. While the tokens' slots name an expert each (mk <= E), s1 * mk <= max(mk, 16 * kSms / gate/up tiles
// of an expert) and s2 * mk, s2s * m <= max(mk, 4 * kSms / down tiles); past that the limits no longer change.
DecodeRows decode_rows(int64_t n, int32_t d, int32_t E, int32_t k, int32_t I, int32_t Is, int32_t dtype) {
  const int64_t nk = n * k, kb1 = ceil_div(d, dtype == MOE_FP8 ? 128 : 64);
  if (dtype == MOE_F32) return DecodeRows{0, 0, nk, Is > 0 ? n : 0};
  const DecodeSplits c = decode_splits(n, d, E, k, I, Is, dtype);
  auto most = [](int64_t rows, int64_t parts, int64_t bound) {
    const int64_t small = rows * kMaxParts < bound ? rows * kMaxParts : bound;
    return rows * parts > small ? rows * parts : small;
  };
  const int64_t tiles1 = ceil_div(I, kRows), tiles1s = ceil_div(Is, kRows), tiles2 = ceil_div(d, kColumns);
  return DecodeRows{most(nk, gate_parts_limit((nk < E ? nk : E) * tiles1, kb1), 16 * kSms / tiles1),
                    Is > 0 ? n * gate_parts_limit(tiles1s, kb1) : 0, most(nk, c.s2, 4 * kSms / tiles2),
                    Is > 0 ? most(n, c.s2s, 4 * kSms / tiles2) : 0};
}

int64_t decode_counters(int32_t d, int32_t E, int32_t I, int32_t Is) {
  return kCtrExpert + E + 1 + ceil_div(d, kMinColumns) + E * ceil_div(I, kRows) + ceil_div(Is, kRows);
}

bool decode_tc_supported() { return encode_fn() != nullptr; }

cudaError_t launch_decode_tc(const DecodeArgs& a, cudaStream_t s) {
  const bool fp8 = a.dtype == MOE_FP8;
  TcShape sh{};
  sh.n_cols = (int32_t)align_up(a.n, 16);
  const int halves = fp8 ? 1 : 2;  // rows of h for a token's slot
  sh.stage_bytes = 2 * kABytes + halves * sh.n_cols * kKB;
  const int64_t slots = align_up((int64_t)a.n * a.k * 6, 16);
  const int64_t sf = fp8 ? 3 * kSfBytes : 0;  // scale words, outside the stages to keep those on 1024 bytes
  const int64_t fit = ((int64_t)kSmemLimit - 1024 - slots - (int64_t)sizeof(Ctl)) / (sh.stage_bytes + sf);
  sh.stages = (int32_t)(fit < kMaxStages ? fit : kMaxStages);
  sh.sf_off = sh.stages * sh.stage_bytes;
  sh.slot_off = sh.sf_off + sh.stages * (int32_t)sf;
  sh.ctl_off = sh.slot_off + (int32_t)slots;
  const size_t smem = 1024 + (size_t)sh.ctl_off + sizeof(Ctl);
  if (sh.stages < 2) return cudaErrorInvalidValue;
  DecodeMaps m;
  const int64_t E = a.E, nk = (int64_t)a.n * a.k;
  bool ok = make_map(&m.gate, fp8, a.w_gate, E * a.I, a.d, kRows) && make_map(&m.up, fp8, a.w_up, E * a.I, a.d, kRows) &&
            make_map(&m.down, fp8, a.w_down, E * a.d, a.I, kRows) &&
            make_map(&m.x, fp8, fp8 ? a.xq : a.x, a.n, a.d, sh.n_cols) && make_map(&m.h, fp8, a.h, halves * nk, a.I, 16);
  m.sgate = m.sup = m.gate;
  m.sdown = m.down;
  m.hs = m.h;
  if (a.Is > 0)
    ok = ok && make_map(&m.sgate, fp8, a.ws_gate, a.Is, a.d, kRows) && make_map(&m.sup, fp8, a.ws_up, a.Is, a.d, kRows) &&
         make_map(&m.sdown, fp8, a.ws_down, a.d, a.Is, kRows) && make_map(&m.hs, fp8, a.hs, halves * a.n, a.Is, sh.n_cols);
  if (!ok) return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (sms <= 0) sms = 148;
  return fp8 ? launch_t<true>(a, m, sh, sms, smem, s) : launch_t<false>(a, m, sh, sms, smem, s);
}

}  // namespace moe
