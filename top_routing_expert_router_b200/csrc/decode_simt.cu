// decode_simt.cu -- the layer for few tokens on the CUDA cores: binary32 (decode.cuh has the scheme).
//
//   h[r, i]  = silu(x_t . gate_e[i]) * (x_t . up_e[i])   for slot row r of token t, expert e
//   o[r, c]  = h[r] . down_e[c],   y[t] = sum_j w_tj o[row(t, j)] + shared(x_t)
// A warp takes one weight row (gate and up rows together) and multiplies it with up to
// kTokens token rows held against it, so each weight is loaded once per kTokens tokens.
// Sums are binary32.
#include <type_traits>

#include "decode.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kTokens = 8;     // token rows a weight row is multiplied with in one pass
constexpr int kColumns = kMinColumns;  // output columns of a down tile

template <int DT>
struct Types;
template <>
struct Types<MOE_F32> {
  using Act = float;
  static constexpr int N = 4;      // weights of one 16-byte load
  static constexpr int ROWS = 32;  // weight rows of a gate/up tile
};
template <>
struct Types<MOE_BF16> {
  using Act = bf16;
  static constexpr int N = 8;
  static constexpr int ROWS = 32;
};
template <>
struct Types<MOE_FP8> {
  using Act = uint8_t;  // x and h enter as E4M3 codes
  static constexpr int N = 16;
  static constexpr int ROWS = 128;  // one scale tile of h
};

struct Shared {
  DecodePlan plan;
  float slot_w[MOE_DECODE_MAX_TOKENS * kMaxTopK];
  uint16_t slot_r[MOE_DECODE_MAX_TOKENS * kMaxTopK];
  int32_t sel_e[kSelfTokens * kMaxTopK];
  float sel_w[kSelfTokens * kMaxTopK];
  union {
    DecideScratch decide;
    float h[MOE_DECODE_MAX_TOKENS][128];
  };
  uint8_t tok[MOE_DECODE_MAX_TOKENS];
  int32_t ticket;
  int32_t ok;
};

__device__ __forceinline__ void unpack(const uint4& raw, float (&v)[16]) {
  const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[j / 2] >> (16 * (j & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}

__device__ __forceinline__ float scale_of(uint8_t byte) { return exp2f((float)((int)byte - 127)); }

// acc[q] = (row w of W) . (token row q) for up to kTokens rows, by one warp. FP8: `scale` and
// `act_scale` ([rows, K / 128]) are the UE8M0 bytes.
template <int DT, typename Act>
__device__ __forceinline__ void dots(const Act* w, const uint8_t* scale, const Act* base, const uint8_t* act_scale, int K,
                                     const int (&row)[kTokens], int m, float (&acc)[kTokens]) {
  constexpr int N = Types<DT>::N;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int q = 0; q < kTokens; ++q) acc[q] = 0.0f;
#pragma unroll 2
  for (int c = lane * N; c < K; c += 32 * N) {
    float wv[N];
    unpack(__ldg(reinterpret_cast<const uint4*>(w + c)), wv);
    float s = 1.0f;
    if constexpr (DT == MOE_FP8) s = scale_of(__ldg(scale + c / 128));
#pragma unroll
    for (int q = 0; q < kTokens; ++q) {
      if (q >= m) break;
      float av[N];
      unpack(__ldcg(reinterpret_cast<const uint4*>(base + (int64_t)row[q] * K + c)), av);  // may be this launch's own
      float t = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) t = fmaf(wv[j], av[j], t);
      if constexpr (DT == MOE_FP8)
        acc[q] = fmaf(s * scale_of(__ldcg(act_scale + (int64_t)row[q] * (K / 128) + c / 128)), t, acc[q]);
      else
        acc[q] += t;
    }
  }
#pragma unroll
  for (int q = 0; q < kTokens; ++q)
#pragma unroll
    for (int off = 16; off; off >>= 1) acc[q] += __shfl_xor_sync(kFull, acc[q], off);
}

template <int DT>
__global__ void __launch_bounds__(kThreads) decode_simt_kernel(DecodeArgs a) {
  using T = Types<DT>;
  using Act = typename T::Act;                                            // x, h and the weights as multiplied
  using Out = typename std::conditional<DT == MOE_FP8, bf16, Act>::type;  // the router's x and y
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
    if (tid == 0) sm.ok = wait_counter(p, target, a.ctr, a.status);
    __syncthreads();
    return sm.ok != 0;
  };
  wait_for_earlier_kernels();
  const Act* x = DT == MOE_FP8 ? reinterpret_cast<const Act*>(a.xq) : static_cast<const Act*>(a.x);
  sm.plan.mask[tid] = 0ull;
  const float bias = a.bias && tid < a.E ? __ldg(a.bias + tid) : 0.0f;
  const bool self = a.n <= kSelfTokens;
  if (self) {
    for (int t = 0; t < a.n; ++t)
      decide_token(a, t, bias, &sm.decide, tid, sync, sm.sel_e + t * a.k, sm.sel_w + t * a.k);
    if (blockIdx.x == 0)
      for (int s = tid; s < a.n * a.k; s += kThreads) a.topk_idx[s] = sm.sel_e[s], a.topk_w[s] = sm.sel_w[s];
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
  const int tiles1 = (a.I + T::ROWS - 1) / T::ROWS, tiles1s = (a.Is + T::ROWS - 1) / T::ROWS;
  const int tiles2 = (a.d + kColumns - 1) / kColumns;
  const int first2 = tiles1s + sm.plan.n_act * tiles1;
  const int total = first2 + (sm.plan.n_act + shared) * tiles2;
  Act* h = static_cast<Act*>(a.h);
  Act* hs = static_cast<Act*>(a.hs);
  for (int t; (t = claim(kCtrTile)) < total;) {
    // expert e (a.E: the shared ones), weight rows [i0, i1) of its matrices
    const bool down = t >= first2;
    int e, i0, i1;
    if (down) {
      const int u = (t - first2) / tiles2 - shared;
      e = u < 0 ? a.E : sm.plan.act[u];
      i0 = (t - first2) % tiles2 * kColumns;
      i1 = min(a.d, i0 + kColumns);
    } else {
      const bool s = t < tiles1s;
      e = s ? a.E : sm.plan.act[(t - tiles1s) / tiles1];
      i0 = (s ? t : (t - tiles1s) % tiles1) * T::ROWS;
      i1 = min(s ? a.Is : a.I, i0 + T::ROWS);
    }
    const bool sh = e == a.E;
    const unsigned long long mask = sh ? token_mask(a.n) : sm.plan.mask[e];
    const int m = __popcll(mask), row0 = sh ? 0 : sm.plan.off[e];
    if (tid < a.n && (mask >> tid & 1ull)) sm.tok[__popcll(mask & ((1ull << tid) - 1ull))] = (uint8_t)tid;
    const int Ie = sh ? a.Is : a.I;
    if (!down) {
      __syncthreads();
      const int64_t at = sh ? 0 : (int64_t)e * a.I * a.d;
      const Act* wg = static_cast<const Act*>(sh ? a.ws_gate : a.w_gate) + at;
      const Act* wu = static_cast<const Act*>(sh ? a.ws_up : a.w_up) + at;
      const int64_t sat = sh ? 0 : (int64_t)e * ((a.I + 127) / 128) * (a.d / 128);
      const uint8_t* sg = DT == MOE_FP8 ? (sh ? a.ss_gate : a.s_gate) + sat : nullptr;
      const uint8_t* su = DT == MOE_FP8 ? (sh ? a.ss_up : a.s_up) + sat : nullptr;
      Act* out = sh ? hs : h;
      for (int i = i0 + warp; i < i1; i += kWarps) {
        for (int m0 = 0; m0 < m; m0 += kTokens) {
          const int mm = min(kTokens, m - m0);
          int row[kTokens];
#pragma unroll
          for (int q = 0; q < kTokens; ++q) row[q] = sm.tok[q < mm ? m0 + q : 0];
          float g[kTokens], u[kTokens];
          dots<DT>(wg + (int64_t)i * a.d, DT == MOE_FP8 ? sg + (i / 128) * (a.d / 128) : nullptr, x, a.xs, a.d, row, mm, g);
          dots<DT>(wu + (int64_t)i * a.d, DT == MOE_FP8 ? su + (i / 128) * (a.d / 128) : nullptr, x, a.xs, a.d, row, mm, u);
#pragma unroll
          for (int q = 0; q < kTokens; ++q)
            if (q < mm && lane == q) {
              const float v = g[q] / (1.0f + expf(-g[q])) * u[q];
              if constexpr (DT == MOE_FP8)
                sm.h[m0 + q][i - i0] = to_f32(from_f32<bf16>(v));
              else
                out[(int64_t)(row0 + m0 + q) * Ie + i] = from_f32<Act>(v);
            }
        }
      }
      if constexpr (DT == MOE_FP8) {
        __syncthreads();
        for (int r = warp; r < m; r += kWarps) {
          const float v[4] = {sm.h[r][4 * lane], sm.h[r][4 * lane + 1], sm.h[r][4 * lane + 2], sm.h[r][4 * lane + 3]};
          uint32_t byte;
          const uint32_t q = quantize_tile(v, &byte);
          reinterpret_cast<uint32_t*>(out + (int64_t)(row0 + r) * Ie + i0)[lane] = q;
          if (lane == 0) (sh ? a.hs_scale : a.h_scale)[(int64_t)(row0 + r) * (Ie / 128) + i0 / 128] = (uint8_t)byte;
        }
      }
      finish(a.ctr + kCtrExpert + e);
      continue;
    }
    if (!wait(a.ctr + kCtrExpert + e, sh ? tiles1s : tiles1)) return;
    const Act* wd = static_cast<const Act*>(sh ? a.ws_down : a.w_down) + (sh ? 0 : (int64_t)e * a.d * a.I);
    const uint8_t* sd = DT == MOE_FP8 ? (sh ? a.ss_down : a.s_down + (int64_t)e * (a.d / 128) * (a.I / 128)) : nullptr;
    const Act* in = (sh ? hs : h) + (int64_t)row0 * Ie;
    const uint8_t* in_scale = DT == MOE_FP8 ? (sh ? a.hs_scale : a.h_scale + (int64_t)row0 * (a.I / 128)) : nullptr;
    float* out = sh ? a.es : a.eo + (int64_t)row0 * a.d;
    for (int i = i0 + warp; i < i1; i += kWarps)
      for (int m0 = 0; m0 < m; m0 += kTokens) {
        const int mm = min(kTokens, m - m0);
        int row[kTokens];
#pragma unroll
        for (int q = 0; q < kTokens; ++q) row[q] = m0 + (q < mm ? q : 0);
        float o[kTokens];
        dots<DT>(wd + (int64_t)i * Ie, DT == MOE_FP8 ? sd + (i / 128) * (Ie / 128) : nullptr, in, in_scale, Ie, row, mm, o);
#pragma unroll
        for (int q = 0; q < kTokens; ++q)
          if (q < mm && lane == q) out[(int64_t)(m0 + q) * a.d + i] = o[q];
      }
    // the last expert's tile of these columns adds them up
    if (finish(a.ctr + kCtrExpert + a.E + 1 + i0 / kColumns) + 1 < sm.plan.n_act + shared) continue;
    for (int i = tid; i < a.n * kColumns; i += kThreads) {
      const int t2 = i / kColumns, c = i0 + i % kColumns;
      if (c >= i1) continue;
      float s = 0.0f;
      for (int j = 0; j < a.k; ++j) {
        s = fmaf(sm.slot_w[t2 * a.k + j], __ldcg(a.eo + (int64_t)sm.slot_r[t2 * a.k + j] * a.d + c), s);
      }
      if (shared) s += __ldcg(a.es + (int64_t)t2 * a.d + c);
      static_cast<Out*>(a.y)[(int64_t)t2 * a.d + c] = from_f32<Out>(s);
    }
  }
}

template <int DT>
cudaError_t launch_t(const DecodeArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> attr;
  const cudaError_t e = set_smem_limit(attr, (const void*)decode_simt_kernel<DT>, sizeof(Shared));
  if (e != cudaSuccess) return e;
  return launch_early(decode_simt_kernel<DT>, 148 * 2, kThreads, sizeof(Shared), s, a);
}

}  // namespace

cudaError_t launch_decode_simt(const DecodeArgs& a, cudaStream_t s) {
  if (a.dtype == MOE_F32) return launch_t<MOE_F32>(a, s);
  if (a.dtype == MOE_BF16) return launch_t<MOE_BF16>(a, s);
  return launch_t<MOE_FP8>(a, s);
}

}  // namespace moe
