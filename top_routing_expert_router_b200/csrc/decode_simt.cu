// decode_simt.cu -- the layer for few tokens on the CUDA cores: binary32 (decode.cuh has the scheme).
//
//   h[r, i]  = silu(x_t . gate_e[i]) * (x_t . up_e[i])   for slot row r of token t, expert e
//   o[r, c]  = h[r] . down_e[c],   y[t] = sum_j w_tj o[row(t, j)] + shared(x_t)
// A tile is 64 weight rows (32 gate and the same 32 up rows, or 64 output columns of a down matrix),
// a warp has eight of them and multiplies them with up to eight token rows at once: lane l holds k
// elements 4 l .. 4 l + 3 of each 128-wide chunk, and the 8 x tokens sums meet at the end of the rows
// by halving exchanges. Weights come through a ring of cp.async copies, each slot written and read by
// one thread, so no barrier guards them; a tile's first chunks are on their way before the tile in
// front of it is summed up. Token rows come through L1. With many tiles and up to eight tokens an expert
// this is bound by HBM (80 experts of 1536 x 5120, 24 tokens: 1134 us for 1021); more tokens are taken in
// passes over the tile (from L2) and bound by the FMA rate: 64 tokens need 64 FMAs for each four bytes,
// 2.9 times as long as the bytes take. Tiles are not cut along k, so a few of them leave most of the GPU
// waiting (58 tokens, six experts of 3040 x 216, 24 down tiles for 296 blocks: 174 us for 7; four tokens, 44
// experts of 96 x 2800: 46 for 7).
#include "decode.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRows = 8;                     // weight rows of a warp
constexpr int kColumns = kWarps * kRows;     // output columns of a down tile
constexpr int kHidden = kColumns / 2;        // hidden columns of a gate/up tile
constexpr int kChunk = 128;                  // k elements of a ring slot
constexpr int kDepth = 3;                    // slots: 96 KB of weights in flight, two blocks an SM
constexpr int kMaxTokens = 8;                // token rows of a pass
static_assert(kColumns >= kMinColumns, "counters of the down tiles");

struct Shared {
  DecodePlan plan;
  float slot_w[MOE_DECODE_MAX_TOKENS * kMaxTopK];
  uint16_t slot_r[MOE_DECODE_MAX_TOKENS * kMaxTopK];
  int32_t sel_e[kSelfTokens * kMaxTopK];
  float sel_w[kSelfTokens * kMaxTopK];
  union {
    DecideScratch decide;
    float4 ring[kDepth][kRows][kThreads];
  };
  uint8_t tok[2][MOE_DECODE_MAX_TOKENS];
  int32_t ticket;
  int32_t ok;
};

// 16 bytes, or zeros where !on.
__device__ __forceinline__ void copy16(void* smem, const void* global, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(global),
               "r"(on ? 16 : 0)
               : "memory");
}

struct Tile {
  int e;        // expert, or E for the shared ones
  int r0;       // first hidden column, or output column
  int down;
  int K;        // length of the weight rows
  int rows;     // hidden or output columns there are
  int row0, m;  // the expert's slots: rows row0 .. row0 + m (shared: every token)
  unsigned long long mask;
  const float *w0, *w1;  // gate and up, or down twice
};

template <int T>
struct Sums {
  float v[kRows / 2 * T * 2];  // [pair of weight rows][token][which of the pair]
};

// One pass over a tile's rows: sums with T token rows at base + row[t] * K.
template <int T, typename Fetch>
__device__ __forceinline__ void pass_sums(Shared& sm, const Tile& tl, const float* base, const int (&row)[kMaxTokens],
                                          Fetch fetch, Sums<T>& s) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < kRows * T; ++i) s.v[i] = 0.0f;
  const int chunks = (tl.K + kChunk - 1) / kChunk;
  const float* p[T];
#pragma unroll
  for (int t = 0; t < T; ++t) p[t] = base + (int64_t)row[t] * tl.K + 4 * lane;
  int slot = 0;
  for (int c = 0; c < chunks; ++c) {
    const bool in = c * kChunk + 4 * lane < tl.K;
    float4 x[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
      x[t] = in ? *reinterpret_cast<const float4*>(p[t] + c * kChunk) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float4 w = sm.ring[slot][r][threadIdx.x];
#pragma unroll
      for (int t = 0; t < T; ++t) {
        float& a = s.v[((r >> 1) * T + t) * 2 + (r & 1)];
        a = fmaf(w.x, x[t].x, a);
        a = fmaf(w.y, x[t].y, a);
        a = fmaf(w.z, x[t].z, a);
        a = fmaf(w.w, x[t].w, a);
      }
    }
    fetch(c + kDepth, slot);
    if (++slot == kDepth) slot = 0;
  }
  // after the last chunk: kDepth empty groups are pending, and the slots are free
  constexpr int V = kRows * T;
  int left = V;
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    if (left > 2) {  // exchange halves: each lane keeps the half of its bit
      left >>= 1;
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        if (i >= left) break;
        const float send = lane & off ? s.v[i] : s.v[i + left], keep = lane & off ? s.v[i + left] : s.v[i];
        s.v[i] = keep + __shfl_xor_sync(kFull, send, off);
      }
    } else {
      s.v[0] += __shfl_xor_sync(kFull, s.v[0], off);
      s.v[1] += __shfl_xor_sync(kFull, s.v[1], off);
    }
  }
}

// Stores a pass's sums: lane l ends up with pair q = l >> (5 - steps) of the halving.
template <int T>
__device__ __forceinline__ void store_sums(const Tile& tl, const Sums<T>& s, float* out, int m0, int m, int ld) {
  constexpr int kPairs = kRows / 2 * T;
  constexpr int kShift = T == 8 ? 0 : T == 4 ? 1 : T == 2 ? 2 : 3;
  static_assert(kPairs << kShift == 32, "lanes of a pair");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane >> kShift, i = q / T, t = q % T;
  if ((lane & ((1 << kShift) - 1)) != 0 || m0 + t >= m) return;
  if (!tl.down) {
    const int c = tl.r0 + warp * (kRows / 2) + i;
    const float g = s.v[0];
    if (c < tl.rows) out[(int64_t)(m0 + t) * ld + c] = g / (1.0f + expf(-g)) * s.v[1];
  } else {
    const int c = tl.r0 + warp * kRows + 2 * i;  // even, and so are the columns
    if (c < tl.rows) *reinterpret_cast<float2*>(out + (int64_t)(m0 + t) * ld + c) = make_float2(s.v[0], s.v[1]);
  }
}

__global__ void __launch_bounds__(kThreads, 2) decode_simt_kernel(const __grid_constant__ DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& sm = *reinterpret_cast<Shared*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto sync = [] { __syncthreads(); };
  auto claim = [&](int which) {
    __syncthreads();
    if (tid == 0) sm.ticket = atomicAdd(a.ctr + which, 1);
    __syncthreads();
    return sm.ticket;
  };
  auto finish = [&](int32_t* p) {  // what the block wrote is visible to whoever sees the count
    __syncthreads();
    if (tid == 0) sm.ticket = add_release(p, 1);
    __syncthreads();
    return sm.ticket;
  };
  auto wait = [&](const int32_t* p, int target) {
    __syncthreads();
    if (tid == 0) sm.ok = wait_counter(p, target, a.ctr, a.status, a.wait_cycles);
    __syncthreads();
    return sm.ok != 0;
  };
  wait_for_earlier_kernels();
  sm.plan.mask[tid] = 0ull;
  const float bias = a.bias && tid < a.E ? __ldg(a.bias + tid) : 0.0f;
  const bool self = a.n <= kSelfTokens;
  if (self) {
    for (int t = 0; t < a.n; ++t)
      decide_token(a, t, bias, &sm.decide, tid, sync, sm.sel_e + t * a.k, sm.sel_w + t * a.k);
    if (blockIdx.x == 0 && tid < a.n * a.k) a.topk_idx[tid] = sm.sel_e[tid], a.topk_w[tid] = sm.sel_w[tid];
  } else {
    for (int t; (t = claim(kCtrToken)) < a.n;) {
      decide_token(a, t, bias, &sm.decide, tid, sync, a.topk_idx + t * a.k, a.topk_w + t * a.k);
      finish(a.ctr + kCtrTokenDone);
    }
    if (!wait(a.ctr + kCtrTokenDone, a.n)) return;
  }
  build_plan<kThreads>(a, self ? sm.sel_e : a.topk_idx, self ? sm.sel_w : a.topk_w, &sm.plan, sm.slot_w, sm.slot_r, tid, sync);
  if (blockIdx.x == 0) write_counts<kThreads>(a, sm.plan, tid);

  const int shared = a.Is > 0;
  const int tiles1 = (a.I + kHidden - 1) / kHidden, tiles1s = (a.Is + kHidden - 1) / kHidden;
  const int tiles2 = (a.d + kColumns - 1) / kColumns;
  const int first2 = tiles1s + sm.plan.n_act * tiles1;
  const int total = first2 + (sm.plan.n_act + shared) * tiles2;
  auto tile_of = [&](int t) {
    Tile tl;
    tl.down = t >= first2;
    int u;
    if (tl.down) {
      u = (t - first2) / tiles2 - shared;
      tl.r0 = (t - first2) % tiles2 * kColumns;
    } else {
      u = t < tiles1s ? -1 : (t - tiles1s) / tiles1;
      tl.r0 = (u < 0 ? t : (t - tiles1s) % tiles1) * kHidden;
    }
    const bool s = u < 0;
    tl.e = s ? a.E : sm.plan.act[u];
    const int Ie = s ? a.Is : a.I;
    tl.K = tl.down ? Ie : a.d;
    tl.rows = tl.down ? a.d : Ie;
    tl.mask = s ? token_mask(a.n) : sm.plan.mask[tl.e];
    tl.row0 = s ? 0 : sm.plan.off[tl.e];
    tl.m = __popcll(tl.mask);
    const int64_t at = s ? 0 : (int64_t)tl.e * a.I * a.d;
    tl.w0 = static_cast<const float*>(tl.down ? (s ? a.ws_down : a.w_down) : (s ? a.ws_gate : a.w_gate)) + at;
    tl.w1 = tl.down ? tl.w0 : static_cast<const float*>(s ? a.ws_up : a.w_up) + at;
    return tl;
  };
  // Chunk c of the warp's eight rows into a slot (zeros past the row; rows past the last are its again).
  auto copy_chunk = [&](const Tile& tl, int c, int slot) {
    const int k = c * kChunk + 4 * lane;
    if (c * kChunk < tl.K) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int row = tl.down ? tl.r0 + warp * kRows + r : tl.r0 + warp * (kRows / 2) + (r >> 1);
        const float* w = (r & 1 ? tl.w1 : tl.w0) + (int64_t)min(row, tl.rows - 1) * tl.K;
        copy16(&sm.ring[slot][r][tid], w + (k < tl.K ? k : 0), k < tl.K);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto start = [&](const Tile& tl) {
    for (int c = 0; c < kDepth; ++c) copy_chunk(tl, c, c);
  };
  __syncthreads();  // the decisions' scratch is the ring's
  int t = claim(kCtrTile), which = 0;
  Tile tl;
  if (t < total) {
    tl = tile_of(t);
    start(tl);
  }
  float* h = static_cast<float*>(a.h);
  float* hs = static_cast<float*>(a.hs);
  while (t < total) {
    const bool s = tl.e == a.E;
    if (tl.down && !wait(a.ctr + kCtrExpert + tl.e, s ? tiles1s : tiles1)) break;
    uint8_t* tok = sm.tok[which];
    which ^= 1;
    if (tid < a.n && (tl.mask >> tid & 1ull)) tok[__popcll(tl.mask & ((1ull << tid) - 1ull))] = (uint8_t)tid;
    const int next = claim(kCtrTile);  // (a barrier: tok is written)
    Tile ahead = tl;
    if (next < total) ahead = tile_of(next);
    const float* base = tl.down ? (s ? hs : h) + (int64_t)tl.row0 * tl.K : static_cast<const float*>(a.x);
    float* out = tl.down ? (s ? a.es : a.eo + (int64_t)tl.row0 * a.d) : (s ? hs : h) + (int64_t)tl.row0 * tl.rows;
    for (int m0 = 0; m0 < tl.m; m0 += kMaxTokens) {
      const int mm = min(kMaxTokens, tl.m - m0);
      int row[kMaxTokens];
#pragma unroll
      for (int q = 0; q < kMaxTokens; ++q) {
        const int r = m0 + min(q, mm - 1);
        row[q] = tl.down ? r : tok[r];
      }
      const bool last = m0 + kMaxTokens >= tl.m;
      auto fetch = [&](int c, int slot) { copy_chunk(tl, c, slot); };
      auto run = [&](auto sums) {
        pass_sums(sm, tl, base, row, fetch, sums);
        // the next pass's, or the next tile's, first chunks set out
        if (!last)
          start(tl);
        else if (next < total)
          start(ahead);
        store_sums(tl, sums, out, m0, tl.m, tl.rows);
      };
      if (mm == 1)
        run(Sums<1>{});
      else if (mm == 2)
        run(Sums<2>{});
      else if (mm <= 4)
        run(Sums<4>{});
      else
        run(Sums<8>{});
    }
    int32_t* done = a.ctr + kCtrExpert + (tl.down ? a.E + 1 + tl.r0 / kColumns : tl.e);
    // the last expert's tile of these columns adds them up, the slots in order, the shared experts last
    if (finish(done) + 1 == sm.plan.n_act + shared && tl.down) {
      for (int i = tid; i < a.n * kColumns; i += kThreads) {
        const int t2 = i / kColumns, c = tl.r0 + i % kColumns;
        if (c >= a.d) continue;
        float y = 0.0f;
#pragma unroll 4
        for (int j = 0; j < a.k; ++j)
          y = fmaf(sm.slot_w[t2 * a.k + j], __ldcg(a.eo + (int64_t)sm.slot_r[t2 * a.k + j] * a.d + c), y);
        if (shared) y += __ldcg(a.es + (int64_t)t2 * a.d + c);
        static_cast<float*>(a.y)[(int64_t)t2 * a.d + c] = y;
      }
    }
    t = next;
    tl = ahead;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace

cudaError_t launch_decode_simt(const DecodeArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> attr;
  const cudaError_t e = set_smem_limit(attr, (const void*)decode_simt_kernel, sizeof(Shared));
  if (e != cudaSuccess) return e;
  return launch_early(decode_simt_kernel, 148 * 2, kThreads, sizeof(Shared), s, a);
}

}  // namespace moe
