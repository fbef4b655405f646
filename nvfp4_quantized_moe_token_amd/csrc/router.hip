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
//   dl_e += p_e (dlse + dS_e - sum_e' p_e' dS_e').
// All arithmetic is fp32.
//
// Layout.  A group of L lanes serves one token, each lane holding V logits in
// registers: L = 16 (four tokens per wave; every reduction stays inside a DPP
// row) up to 256 experts and k <= 16, else a whole wave.  Vectors of W
// consecutive logits per lane (16 bytes of fp32) when E and the pointers
// allow it.  Lane i holds experts e(v) = (v / W) * W * L + i * W + v % W, so a
// lower v is a lower expert and ties resolve in order.
#include <type_traits>

#include "common.hpp"

namespace nvfp4moe {
namespace {

constexpr int kRouterThreads = 256;
constexpr int kProbSumBlocks = 512;  // workgroups that leave partial sums of the probabilities

constexpr float kNegInf = -__builtin_inff();

// Reductions over a token's L lanes; every lane receives the result.
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  const int i = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(i, i, CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ int dpp_i(int v) {
  return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
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
template <int L>
__device__ __forceinline__ int group_min(int v) {
  int o;
  o = dpp_i<kRor + 8>(v); v = o < v ? o : v;
  o = dpp_i<kRor + 4>(v); v = o < v ? o : v;
  o = dpp_i<kRor + 2>(v); v = o < v ? o : v;
  o = dpp_i<kRor + 1>(v); v = o < v ? o : v;
  if constexpr (L == 64) {
    o = __shfl_xor(v, 16, 64); v = o < v ? o : v;
    o = __shfl_xor(v, 32, 64); v = o < v ? o : v;
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

// max and sum of exp(l - max) over a token's logits.  All -inf: sum 0.
template <int L, int V>
__device__ __forceinline__ void row_softmax(const float (&l)[V], float& m, float& sum) {
  m = l[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
  m = group_max<L>(m);
  sum = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) sum += m > kNegInf || l[v] != l[v] ? __expf(l[v] - m) : 0.0f;
  sum = group_sum<L>(sum);
}

// AUX: the lse and/or the per-expert sums of probabilities are wanted.
// Without them one token per group; with the sums the groups walk the tokens
// so that every workgroup leaves one partial row.
template <int L, int V, int W, bool BF16, bool AUX>
__global__ __launch_bounds__(kRouterThreads) void router_kernel(const void* __restrict__ logits, int64_t T, int E,
                                                                int k, const float* __restrict__ bias, int score,
                                                                float scale, int32_t* __restrict__ ids,
                                                                float* __restrict__ w, float* __restrict__ lse,
                                                                float* __restrict__ partial) {
  constexpr int G = kRouterThreads / L;  // tokens in flight per workgroup
  const int i = threadIdx.x % L, g = threadIdx.x / L;
  float acc[AUX ? V : 1];
#pragma unroll
  for (int v = 0; v < (AUX ? V : 1); ++v) acc[v] = 0.0f;

  for (int64_t t = (int64_t)blockIdx.x * G + g; t < T; t += (int64_t)gridDim.x * G) {
    float l[V];
    load_row<L, V, W, BF16>(logits, t, E, i, kNegInf, l);
    // Selection: k rounds of "largest key, lowest expert", each taking the
    // winner out.
    float key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_of<L, W>(v, i);
      const float s = l[v] + (bias && e < E ? bias[e] : 0.0f);  // (+0 also turns -0 into +0)
      key[v] = s == s ? s : kNegInf;
    }
    int mine = -1;  // lane j keeps the j-th choice
    for (int j = 0; j < k; ++j) {
      float best = key[0];
#pragma unroll
      for (int v = 1; v < V; ++v) best = fmaxf(best, key[v]);
      best = group_max<L>(best);
      if (!(best > kNegInf)) break;  // uniform in the group: nothing is left
      int at = 0x7FFFFFFF;
#pragma unroll
      for (int v = V - 1; v >= 0; --v)
        if (key[v] == best) at = expert_of<L, W>(v, i);
      at = group_min<L>(at);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (expert_of<L, W>(v, i) == at) key[v] = kNegInf;
      if (i == j) mine = at;
    }
    float m = 0.0f, sum = 1.0f;
    if (AUX || score == NVFP4MOE_ROUTER_SOFTMAX) row_softmax<L, V>(l, m, sum);
    const float c = mine >= 0 ? load_logit<BF16>(logits, t * E + mine) : kNegInf;
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
    if constexpr (AUX) {
      if (lse && i == 0) lse[t] = sum == 0.0f ? kNegInf : m + __logf(sum);
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += m > kNegInf || l[v] != l[v] ? __expf(l[v] - m) * inv : 0.0f;
    }
  }

  if constexpr (AUX) {
    if (partial) {
      // The groups' sums meet in LDS, in the order of the groups.
      __shared__ float red[kRouterThreads * V];
#pragma unroll
      for (int v = 0; v < V; ++v) red[v * kRouterThreads + threadIdx.x] = acc[v];
      __syncthreads();
      for (int x = threadIdx.x; x < L * V; x += kRouterThreads) {
        const int v = x / L, ii = x % L, e = expert_of<L, W>(v, ii);
        float s = 0.0f;
        for (int q = 0; q < G; ++q) s += red[v * kRouterThreads + q * L + ii];
        if (e < E) partial[(int64_t)blockIdx.x * E + e] = s;
      }
    }
  }
}

// prob_sum[e] = sum of the workgroups' partial rows, in a fixed order.
__global__ __launch_bounds__(256) void prob_sum_kernel(const float* __restrict__ partial, int rows, int E,
                                                       float* __restrict__ out) {
  __shared__ float red[256];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4, e = blockIdx.x * 16 + c;
  float s = 0.0f;
  if (e < E)
    for (int q = r; q < rows; q += 16) s += partial[(int64_t)q * E + e];
  red[threadIdx.x] = s;
  __syncthreads();
  if (r == 0 && e < E) {
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
      float m, sum;
      row_softmax<L, V>(p, m, sum);
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
        mean += p[v] * s[v];
      }
      base -= group_sum<L>(mean);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = p[v] * (dsum ? base + s[v] : base);
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

int64_t prob_sum_rows(int64_t T, int E, int k) {
  const int64_t per = k <= 16 && E <= 256 ? kRouterThreads / 16 : kRouterThreads / 64;
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
  const bool bf = logits_dtype == NVFP4MOE_BF16, aux = lse || prob_sum;
  float* partial = prob_sum ? reinterpret_cast<float*>(workspace) : nullptr;
  with_layout(E, k, E % 4 == 0 && aligned(logits, 4 * lb), [&](auto Lc, auto Vc, auto Wc) {
    constexpr int L = decltype(Lc)::value, V = decltype(Vc)::value, W = decltype(Wc)::value;
    int64_t grid = cdiv(T, kRouterThreads / L);
    if (grid > kMaxStreamGrid) grid = kMaxStreamGrid;
    if (prob_sum) grid = prob_sum_rows(T, E, k);
#define NVR_GO(B, A)                                                                                          \
  router_kernel<L, V, W, B, A><<<(unsigned)grid, kRouterThreads, 0, st>>>(logits, T, E, k, bias, score, scale, \
                                                                          topk_ids, topk_w, lse, partial)
    if (bf) {
      if (aux) NVR_GO(true, true);
      else NVR_GO(true, false);
    } else {
      if (aux) NVR_GO(false, true);
      else NVR_GO(false, false);
    }
#undef NVR_GO
  });
  if (prob_sum)
    prob_sum_kernel<<<(unsigned)cdiv(E, 16), 256, 0, st>>>(partial, (int)prob_sum_rows(T, E, k), E, prob_sum);
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
    const int64_t grid = cdiv(T, kRouterThreads / L);
#define NVR_GO(B, O)                                                                                       \
  router_bwd_kernel<L, V, W, B, O><<<(unsigned)grid, kRouterThreads, 0, st>>>(logits, T, E, k, topk_ids, score, scale, \
                                                                              d_topk_w, lse, d_lse, d_prob_sum, d_logits)
    if (bf) {
      if (obf) NVR_GO(true, true);
      else NVR_GO(true, false);
    } else {
      if (obf) NVR_GO(false, true);
      else NVR_GO(false, false);
    }
#undef NVR_GO
  });
  return launch_status();
}
