// The router of the MoE layer: top-k of the (biased) expert logits with
// softmax weights, and its gradient.  It produces the routing ids and fp32
// weights that the permutation and the combine consume ("miniTE報告、NVFP4強化
// 学習の安定性を検証", fourth paragraph: device-side metadata; the pages do
// not describe the router itself).
//
// Mathematics, per token with logits l_e (fp32), optional selection bias b_e
// and key_e = l_e + b_e:
//   ids = the k largest keys, largest first, ties to the lower expert; keys
//         that are -inf or NaN are never chosen (id -1, weight 0);
//   TOPK_SOFTMAX: w_j = scale * exp(l_j - m) / sum over the chosen;
//   SOFTMAX:      w_j = scale * exp(l_j - lse), lse = log sum_e exp(l_e);
//   prob_sum_e = sum over tokens of p_e = exp(l_e - lse).
// Backward (u_j = scale * dw_j):
//   TOPK_SOFTMAX: dl[id_j] += q_j (u_j - sum_i q_i u_i), q = softmax of the chosen;
//   SOFTMAX:      dl[id_j] += p_j u_j, and dl_e -= p_e sum_j p_j u_j;
//   dl_e += p_e (dlse + dS_e - sum_e' p_e' dS_e'), terms with p = 0 left out:
//           the lse of a row without experts is -inf, and so is the gradient of
//           its square.
// All arithmetic is fp32.
//
// Layout.  A group of L lanes serves one token, each lane holding V logits in
// registers: L = 16 (four tokens per wave; every reduction stays inside a DPP
// row) up to 256 experts and k <= 16, else a whole wave.  Vectors of W
// consecutive logits per lane (16 bytes of fp32) when E and the pointers
// allow it.  Lane i holds experts e(v) = (v / W) * W * L + i * W + v % W, so a
// lower v is a lower expert and ties resolve in order.
//
// Exponentials and logarithms are the hardware's (__expf, __logf): their errors
// are those of fp32 roundings (weights are off by 6e-8 relative, as with exact
// functions), and gates are not worth more instructions.
//
// Bounds, measured (E = 128, k = 8, fp32): the rounds.  One is some 46
// instructions for the four tokens of a wave: 3 maxima over 8 registers (three
// at a time), 4 across the lanes, 16 to find the winner's expert, 4 across, 16
// to take it out.  With lse and sums the vector ALU issues 59% of the time and
// waves wait 57% of theirs: the reductions of a round depend on one another.  16 tokens 3.9 us (a launch and one trip to memory); 16384
// tokens with lse and sums 10 to 11 us (0.9 TB/s), the last sum 2 to 4 us,
// where 512 smaller workgroups and floating-point keys took 11.6 and 10.6.  The
// gradient of 8192 tokens 6.0 us (1.5 TB/s; 5.6 without the test for
// probabilities of 0).
#include <type_traits>

#include "common.hpp"

namespace nvfp4moe {
namespace {

constexpr int kRouterThreads = 256;
constexpr int kProbSumBlocks = 256;  // workgroups that leave partial sums of the probabilities

constexpr float kNegInf = -__builtin_inff();

// Reductions over a token's L lanes; every lane receives the result.  (With a
// zero for lanes that have no source, which do not occur, the compiler folds
// the rotation into the operation.)
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kRor = 0x120;  // row_ror:n is 0x120 + n (rows of 16 lanes)

template <int L>
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, dpp_f<kRor + 8>(v));
  v = fmaxf(v, dpp_f<kRor + 4>(v));
  v = fmaxf(v, dpp_f<kRor + 2>(v));
  v = fmaxf(v, dpp_f<kRor + 1>(v));
  if constexpr (L == 64) {
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    v = fmaxf(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }
template <int L>
__device__ __forceinline__ uint32_t group_umax(uint32_t v) {
  v = umax(v, dpp_u<kRor + 8>(v));
  v = umax(v, dpp_u<kRor + 4>(v));
  v = umax(v, dpp_u<kRor + 2>(v));
  v = umax(v, dpp_u<kRor + 1>(v));
  if constexpr (L == 64) {
    v = umax(v, __shfl_xor(v, 16, 64));
    v = umax(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t group_umin(uint32_t v) {
  v = umin(v, dpp_u<kRor + 8>(v));
  v = umin(v, dpp_u<kRor + 4>(v));
  v = umin(v, dpp_u<kRor + 2>(v));
  v = umin(v, dpp_u<kRor + 1>(v));
  if constexpr (L == 64) {
    v = umin(v, __shfl_xor(v, 16, 64));
    v = umin(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  v += dpp_f<kRor + 8>(v);
  v += dpp_f<kRor + 4>(v);
  v += dpp_f<kRor + 2>(v);
  v += dpp_f<kRor + 1>(v);
  if constexpr (L == 64) {
    v += __shfl_xor(v, 16, 64);
    v += __shfl_xor(v, 32, 64);
  }
  return v;
}

// Keys as unsigned integers of the same order; 0 is "never chosen" (-inf, NaN
// and what has been taken).
__device__ __forceinline__ uint32_t sortable(float s) {
  const int b = __float_as_int(s);
  return s > kNegInf ? (uint32_t)(b ^ ((b >> 31) | (int)0x80000000)) : 0u;
}
__device__ __forceinline__ float unsortable(uint32_t u) {
  const int b = (int)u;
  return __int_as_float(b ^ (~(b >> 31) | (int)0x80000000));
}

// Expert of register v of group lane i.
template <int L, int W>
__device__ __forceinline__ int expert_of(int v, int i) {
  return (v / W) * W * L + i * W + v % W;
}

// The lane's V logits of one row (`fill` past E).
template <int L, int V, int W, bool BF16>
__device__ __forceinline__ void load_row(const void* __restrict__ base, int64_t row, int E, int i, float fill,
                                         float (&out)[V]) {
#pragma unroll
  for (int b = 0; b < V / W; ++b) {
    const int e = b * W * L + i * W;
    if constexpr (W == 4) {
      if (e < E) {  // E % 4 == 0: the vector is whole
        if constexpr (BF16) {
          const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(base) + row * E + e);
          out[4 * b] = bf16_lo(w.x);
          out[4 * b + 1] = bf16_hi(w.x);
          out[4 * b + 2] = bf16_lo(w.y);
          out[4 * b + 3] = bf16_hi(w.y);
        } else {
          const float4 w = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + row * E + e);
          out[4 * b] = w.x;
          out[4 * b + 1] = w.y;
          out[4 * b + 2] = w.z;
          out[4 * b + 3] = w.w;
        }
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) out[4 * b + u] = fill;
      }
    } else {
      if (e < E) {
        if constexpr (BF16)
          out[b] = bf16_lo(reinterpret_cast<const uint16_t*>(base)[row * E + e]);
        else
          out[b] = reinterpret_cast<const float*>(base)[row * E + e];
      } else {
        out[b] = fill;
      }
    }
  }
}
template <int L, int V, int W, bool BF16>
__device__ __forceinline__ void store_row(void* __restrict__ base, int64_t row, int E, int i, const float (&v)[V]) {
#pragma unroll
  for (int b = 0; b < V / W; ++b) {
    const int e = b * W * L + i * W;
    if (e >= E) continue;
    if constexpr (W == 4) {
      if constexpr (BF16)
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(base) + row * E + e) =
            make_uint2(pack_bf16x2(v[4 * b], v[4 * b + 1]), pack_bf16x2(v[4 * b + 2], v[4 * b + 3]));
      else
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + row * E + e) =
            make_float4(v[4 * b], v[4 * b + 1], v[4 * b + 2], v[4 * b + 3]);
    } else {
      if constexpr (BF16)
        reinterpret_cast<uint16_t*>(base)[row * E + e] = (uint16_t)f32_to_bf16_rne(v[b]);
      else
        reinterpret_cast<float*>(base)[row * E + e] = v[b];
    }
  }
}
template <bool BF16>
__device__ __forceinline__ float load_logit(const void* __restrict__ base, int64_t at) {
  if constexpr (BF16) return bf16_lo(reinterpret_cast<const uint16_t*>(base)[at]);
  else return reinterpret_cast<const float*>(base)[at];
}

// max and sum of exp(l - max) over a token's logits, which become exp(l -
// max).  All -inf: zeros.
template <int L, int V>
__device__ __forceinline__ void row_softmax(float (&l)[V], float& m, float& sum) {
  m = l[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
  m = group_max<L>(m);
  sum = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    l[v] = m > kNegInf || l[v] != l[v] ? __expf(l[v] - m) : 0.0f;
    sum += l[v];
  }
  sum = group_sum<L>(sum);
}

// SUM: the per-expert sums of probabilities are wanted.  Without them one
// token per group; with them large workgroups walk the tokens, so that few
// partial rows are left to add up.
template <int L, int V, int W, bool BF16, bool SUM, int THREADS>
__global__ __launch_bounds__(THREADS) void router_kernel(const void* __restrict__ logits, int64_t T, int E, int k,
                                                         const float* __restrict__ bias, int score, float scale,
                                                         int32_t* __restrict__ ids, float* __restrict__ w,
                                                         float* __restrict__ lse, float* __restrict__ partial) {
  constexpr int G = THREADS / L;  // tokens in flight per workgroup
  const int i = threadIdx.x % L, g = threadIdx.x / L;
  float acc[SUM ? V : 1];
#pragma unroll
  for (int v = 0; v < (SUM ? V : 1); ++v) acc[v] = 0.0f;

  for (int64_t t = (int64_t)blockIdx.x * G + g; t < T; t += (int64_t)gridDim.x * G) {
    float l[V];
    load_row<L, V, W, BF16>(logits, t, E, i, kNegInf, l);
    // Selection: k rounds of "largest key, lowest expert", each taking the
    // winner out.
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_of<L, W>(v, i);
      key[v] = sortable(l[v] + (bias && e < E ? bias[e] : 0.0f));  // (+0 also turns -0 into +0)
    }
    int mine = -1;  // lane j keeps the j-th choice and its logit
    float c = kNegInf;
    for (int j = 0; j < k; ++j) {
      uint32_t best = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) best = umax(best, key[v]);
      best = group_umax<L>(best);
      if (best == 0) break;  // uniform in the group: nothing is left
      uint32_t at = 0xFFFFFFFFu;
#pragma unroll
      for (int v = V - 1; v >= 0; --v)
        if (key[v] == best) at = (uint32_t)expert_of<L, W>(v, i);
      at = group_umin<L>(at);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if ((uint32_t)expert_of<L, W>(v, i) == at) key[v] = 0u;
      if (i == j) {
        mine = (int)at;
        c = unsortable(best);
      }
    }
    if (bias && mine >= 0) c = load_logit<BF16>(logits, t * E + mine);
    float m = 0.0f, sum = 1.0f;
    if (SUM || lse || score == NVFP4MOE_ROUTER_SOFTMAX) row_softmax<L, V>(l, m, sum);
    float wt;
    if (score == NVFP4MOE_ROUTER_TOPK_SOFTMAX) {
      const float mc = group_max<L>(c);
      const float ex = mine >= 0 ? __expf(c - mc) : 0.0f;
      const float den = group_sum<L>(ex);  // every lane takes part, chosen or not
      wt = mine >= 0 ? scale * (ex / den) : 0.0f;
    } else {
      wt = mine >= 0 ? scale * (__expf(c - m) / sum) : 0.0f;
    }
    if (i < k) {
      ids[t * k + i] = mine;
      w[t * k + i] = wt;
    }
    if (lse && i == 0) lse[t] = sum == 0.0f ? kNegInf : m + __logf(sum);
    if constexpr (SUM) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += l[v] * inv;
    }
  }

  if constexpr (SUM) {
    // A wave's groups meet in its lanes, the waves in LDS, always in the same
    // order.
    constexpr int NW = THREADS / 64;
    __shared__ float red[NW * L * V];
    const int lane = threadIdx.x & 63, wid = threadIdx.x / 64;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if constexpr (L == 16) {
        acc[v] += __shfl_xor(acc[v], 16, 64);
        acc[v] += __shfl_xor(acc[v], 32, 64);
      }
      if (lane < L) red[(wid * V + v) * L + i] = acc[v];
    }
    __syncthreads();
    for (int x = threadIdx.x; x < L * V; x += THREADS) {
      const int e = expert_of<L, W>(x / L, x % L);
      float s = red[x];
#pragma unroll
      for (int q = 1; q < NW; ++q) s += red[q * L * V + x];
      if (e < E) partial[(int64_t)blockIdx.x * E + e] = s;
    }
  }
}

// prob_sum[e] = sum of the workgroups' partial rows, in a fixed order: 16
// experts per workgroup, 64 rows at a time.
__global__ __launch_bounds__(1024) void prob_sum_kernel(const float* __restrict__ partial, int rows, int E,
                                                        float* __restrict__ out) {
  __shared__ float red[16 * 16];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4, e = blockIdx.x * 16 + c;
  float s = 0.0f;
  if (e < E)
#pragma unroll 4
    for (int q = r; q < rows; q += 64) s += partial[(int64_t)q * E + e];
  s += __shfl_xor(s, 16, 64);
  s += __shfl_xor(s, 32, 64);
  if ((threadIdx.x & 63) < 16) red[(threadIdx.x >> 6) * 16 + c] = s;
  __syncthreads();
  if (threadIdx.x < 16 && e < E) {
    s = red[c];
#pragma unroll
    for (int q = 1; q < 16; ++q) s += red[q * 16 + c];
    out[e] = s;
  }
}

template <int L, int V, int W, bool BF16, bool OUT_BF16>
__global__ __launch_bounds__(kRouterThreads) void router_bwd_kernel(
    const void* __restrict__ logits, int64_t T, int E, int k, const int32_t* __restrict__ ids, int score, float scale,
    const float* __restrict__ dw, const float* __restrict__ lse, const float* __restrict__ dlse,
    const float* __restrict__ dsum, void* __restrict__ dl) {
  constexpr int G = kRouterThreads / L;
  const int i = threadIdx.x % L, g = threadIdx.x / L;
  const int64_t t = (int64_t)blockIdx.x * G + g;
  if (t >= T) return;
  const bool all = score == NVFP4MOE_ROUTER_SOFTMAX;
  const bool full = all || dlse || dsum;  // the probabilities of every expert take part

  // This lane's choice (lane j: the j-th).
  int id = -1;
  float u = 0.0f;
  if (i < k) {
    id = ids[t * k + i];
    if (id >= E) id = -1;
    if (id >= 0 && dw) u = scale * dw[t * k + i];
  }
  const float c = id >= 0 ? load_logit<BF16>(logits, t * E + id) : kNegInf;

  float p[V], L_t = 0.0f;
  bool empty = false;
  if (full) {
    load_row<L, V, W, BF16>(logits, t, E, i, kNegInf, p);
    if (lse) {
      L_t = lse[t];
    } else {
      float m, sum, ex[V];
#pragma unroll
      for (int v = 0; v < V; ++v) ex[v] = p[v];
      row_softmax<L, V>(ex, m, sum);
      L_t = sum == 0.0f ? kNegInf : m + __logf(sum);
    }
    empty = L_t == kNegInf;
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = empty ? 0.0f : __expf(p[v] - L_t);
  }

  // Gradient of the chosen entries.
  float gj, dot;
  if (all) {
    gj = id >= 0 && !empty ? __expf(c - L_t) * u : 0.0f;
    dot = group_sum<L>(gj);
  } else {
    const float mc = group_max<L>(c);
    const float ex = id >= 0 ? __expf(c - mc) : 0.0f;
    const float den = group_sum<L>(ex);
    const float q = id >= 0 ? ex / den : 0.0f;
    const float qu = group_sum<L>(q * u);
    gj = id >= 0 ? q * (u - qu) : 0.0f;
    dot = 0.0f;
  }

  float d[V];
#pragma unroll
  for (int v = 0; v < V; ++v) d[v] = 0.0f;
  if (full) {
    float base = dlse ? dlse[t] - dot : -dot, s[V];
    if (dsum) {
      float mean = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = expert_of<L, W>(v, i);
        s[v] = e < E ? dsum[e] : 0.0f;
        mean += p[v] == 0.0f ? 0.0f : p[v] * s[v];
      }
      base -= group_sum<L>(mean);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = p[v] == 0.0f ? 0.0f : p[v] * (dsum ? base + s[v] : base);
  }
  for (int j = 0; j < k; ++j) {
    const int src = (threadIdx.x & 63) / L * L + j;  // lane j of this token's group
    const int at = __shfl(id, src, 64);
    const float add = __shfl(gj, src, 64);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (expert_of<L, W>(v, i) == at) d[v] += add;
  }
  store_row<L, V, W, OUT_BF16>(dl, t, E, i, d);
}

// Calls f(lanes, values per lane, vector width) for the smallest layout that
// holds E experts and k choices.
template <class F>
void with_layout(int E, int k, bool vec, F f) {
#define NVR(L, V)                                                                       \
  do {                                                                                  \
    if (vec) f(std::integral_constant<int, L>(), std::integral_constant<int, V>(), std::integral_constant<int, 4>()); \
    else f(std::integral_constant<int, L>(), std::integral_constant<int, V>(), std::integral_constant<int, 1>());     \
  } while (0)
  if (k <= 16 && E <= 64) NVR(16, 4);
  else if (k <= 16 && E <= 128) NVR(16, 8);
  else if (k <= 16 && E <= 256) NVR(16, 16);
  else if (E <= 512) NVR(64, 8);
  else if (E <= 1024) NVR(64, 16);
  else NVR(64, 64);
#undef NVR
}

constexpr int kRouterMaxExperts = 4096;

// Workgroup sizes with probability sums: as large as the registers allow.
constexpr int sum_threads(int V) { return V <= 16 ? 1024 : 256; }

int64_t prob_sum_rows(int64_t T, int E, int k) {
  const int64_t per = k <= 16 && E <= 256 ? 1024 / 16 : E <= 1024 ? 1024 / 64 : 256 / 64;
  const int64_t n = cdiv(T, per);
  return n < kProbSumBlocks ? n : kProbSumBlocks;
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" size_t moe_router_workspace_size(int64_t T, int E, int k) {
  if (T < 0 || E < 1 || k < 1) return 0;
  return (size_t)(prob_sum_rows(T, E, k) * E * 4);
}

extern "C" int moe_router(const void* logits, int logits_dtype, int64_t T, int E, int k, const float* bias, int score,
                          float scale, int32_t* topk_ids, float* topk_w, float* lse, float* prob_sum, void* workspace,
                          size_t ws_bytes, nvfp4moe_stream_t stream) {
  if (T < 0 || E < 1 || k < 1) return NVFP4MOE_EINVAL;
  if (logits_dtype != NVFP4MOE_F32 && logits_dtype != NVFP4MOE_BF16) return NVFP4MOE_EINVAL;
  if (score != NVFP4MOE_ROUTER_TOPK_SOFTMAX && score != NVFP4MOE_ROUTER_SOFTMAX) return NVFP4MOE_EINVAL;
  if (T > 0 && (!logits || !topk_ids || !topk_w)) return NVFP4MOE_EINVAL;
  if (E > kRouterMaxExperts || k > 64 || k > E) return NVFP4MOE_ESHAPE;
  if (T * k > 0x7FFFFFFFLL) return NVFP4MOE_ESHAPE;
  const int lb = dtype_bytes(logits_dtype);
  if (!aligned(logits, lb) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(lse, 4) ||
      !aligned(prob_sum, 4) || !aligned(workspace, 4))
    return NVFP4MOE_ESHAPE;
  if (prob_sum && T > 0 && (!workspace || ws_bytes < moe_router_workspace_size(T, E, k))) return NVFP4MOE_EWORKSPACE;
  const int arch = check_arch();
  if (arch != NVFP4MOE_OK) return arch;
  hipStream_t st = as_stream(stream);
  if (T == 0) {
    if (prob_sum) fill_u32_kernel<<<1, 256, 0, st>>>(reinterpret_cast<uint32_t*>(prob_sum), 0u, E);
    return launch_status();
  }
  const bool bf = logits_dtype == NVFP4MOE_BF16;
  float* partial = prob_sum ? reinterpret_cast<float*>(workspace) : nullptr;
  with_layout(E, k, E % 4 == 0 && aligned(logits, 4 * lb), [&](auto Lc, auto Vc, auto Wc) {
    constexpr int L = decltype(Lc)::value, V = decltype(Vc)::value, W = decltype(Wc)::value;
    int64_t grid = cdiv(T, kRouterThreads / L);
    if (grid > kMaxStreamGrid) grid = kMaxStreamGrid;
    if (prob_sum) grid = prob_sum_rows(T, E, k);
#define NVR_GO(B, S, N)                                                                                             \
  router_kernel<L, V, W, B, S, N><<<(unsigned)grid, N, 0, st>>>(logits, T, E, k, bias, score, scale, topk_ids, topk_w, \
                                                                lse, partial)
    constexpr int N = sum_threads(V);
    if (bf) {
      if (prob_sum) NVR_GO(true, true, N);
      else NVR_GO(true, false, kRouterThreads);
    } else {
      if (prob_sum) NVR_GO(false, true, N);
      else NVR_GO(false, false, kRouterThreads);
    }
#undef NVR_GO
  });
  if (prob_sum)
    prob_sum_kernel<<<(unsigned)cdiv(E, 16), 1024, 0, st>>>(partial, (int)prob_sum_rows(T, E, k), E, prob_sum);
  return launch_status();
}

extern "C" int moe_router_bwd(const void* logits, int logits_dtype, int64_t T, int E, int k, const int32_t* topk_ids,
                              int score, float scale, const float* d_topk_w, const float* lse, const float* d_lse,
                              const float* d_prob_sum, void* d_logits, int d_dtype, nvfp4moe_stream_t stream) {
  if (T < 0 || E < 1 || k < 1) return NVFP4MOE_EINVAL;
  if (logits_dtype != NVFP4MOE_F32 && logits_dtype != NVFP4MOE_BF16) return NVFP4MOE_EINVAL;
  if (d_dtype != NVFP4MOE_F32 && d_dtype != NVFP4MOE_BF16) return NVFP4MOE_EINVAL;
  if (score != NVFP4MOE_ROUTER_TOPK_SOFTMAX && score != NVFP4MOE_ROUTER_SOFTMAX) return NVFP4MOE_EINVAL;
  if (T > 0 && (!logits || !topk_ids || !d_logits)) return NVFP4MOE_EINVAL;
  if (E > kRouterMaxExperts || k > 64 || k > E) return NVFP4MOE_ESHAPE;
  if (T * k > 0x7FFFFFFFLL) return NVFP4MOE_ESHAPE;
  const int lb = dtype_bytes(logits_dtype), db = dtype_bytes(d_dtype);
  if (!aligned(logits, lb) || !aligned(d_logits, db) || !aligned(topk_ids, 4) || !aligned(d_topk_w, 4) ||
      !aligned(lse, 4) || !aligned(d_lse, 4) || !aligned(d_prob_sum, 4))
    return NVFP4MOE_ESHAPE;
  const int arch = check_arch();
  if (arch != NVFP4MOE_OK) return arch;
  if (T == 0) return NVFP4MOE_OK;
  hipStream_t st = as_stream(stream);
  const bool bf = logits_dtype == NVFP4MOE_BF16, obf = d_dtype == NVFP4MOE_BF16;
  with_layout(E, k, E % 4 == 0 && aligned(logits, 4 * lb) && aligned(d_logits, 4 * db), [&](auto Lc, auto Vc, auto Wc) {
    constexpr int L = decltype(Lc)::value, V = decltype(Vc)::value, W = decltype(Wc)::value;
    // A dispatch has fewer than 2^32 work-items: tokens beyond that go in
    // launches of their own.
    constexpr int64_t kSlice = kMaxStreamGrid * (kRouterThreads / L);
    for (int64_t t0 = 0; t0 < T; t0 += kSlice) {
      const int64_t n = T - t0 < kSlice ? T - t0 : kSlice, grid = cdiv(n, kRouterThreads / L);
      const void* x = reinterpret_cast<const uint8_t*>(logits) + t0 * E * lb;
      void* d = reinterpret_cast<uint8_t*>(d_logits) + t0 * E * db;
      const float *dw = d_topk_w ? d_topk_w + t0 * k : nullptr, *ls = lse ? lse + t0 : nullptr,
                  *dl = d_lse ? d_lse + t0 : nullptr;
#define NVR_GO(B, O)                                                                                            \
  router_bwd_kernel<L, V, W, B, O><<<(unsigned)grid, kRouterThreads, 0, st>>>(x, n, E, k, topk_ids + t0 * k, score, \
                                                                              scale, dw, ls, dl, d_prob_sum, d)
      if (bf) {
        if (obf) NVR_GO(true, true);
        else NVR_GO(true, false);
      } else {
        if (obf) NVR_GO(false, true);
        else NVR_GO(false, false);
      }
    }
#undef NVR_GO
  });
  return launch_status();
}
