// Quantization to 8-bit integers with one fp32 scale per row: a token's for
// activations, an output channel's for weights (the operands of
// grouped_gemm_int8; "miniTE報告、NVFP4強化学習の安定性を検証", fourth paragraph:
// token-wise quantization, contiguous layout, op fusion).
//
// Mathematics, per row with amax a, in IEEE fp32:
//   s = a / 127,  q = rne(x / s) clamped to [-127, 127]; all zeros when s is 0.
// (x / s passes 127 only where s is subnormal.)  A row that holds an infinity
// or a NaN gets that infinity or a NaN as its scale and zeros as codes: its
// products are NaN.
//
// Layout.  Sixteen lanes per row up to 768 elements, a wave up to 4096, 16
// consecutive elements a lane and step, kept in registers between the maximum and the encoding; a workgroup
// per row beyond, which reads the row a second time (from the cache).  The
// permutation's form encodes a token once and writes its k rows.
//
// Measured (us): H of 65536 x 768 bf16 25 to 29 (151 MB, 5.2 to 6 TB/s; 45 with a
// wave per row and divisions: the vector ALU then took longer than the memory);
// the gate+up weights of 128 experts, 196608 x 2048, 210 (5.8 TB/s); 8192 tokens
// of 2048 to 65536 permuted rows 30 (5.5 TB/s).
#include "common.hpp"

namespace nvfp4moe {
namespace {

struct Int8Params {
  const uint4* x;
  int64_t rows;  // of x
  int64_t K;
  int8_t* q;
  float* scales;
  const int32_t* dest;  // scatter: rows of x go to dest[row * k + j]
  const int32_t* offsets;
  int64_t R;
  int k, E;
};

template <bool BF16>
__device__ __forceinline__ void load16(const uint4* x, int64_t at, float (&v)[16]) {  // at: in 16 elements
  if (BF16) {
    const uint4 w0 = x[2 * at], w1 = x[2 * at + 1];
    const uint32_t ws[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[2 * i] = bf16_lo(ws[i]);
      v[2 * i + 1] = bf16_hi(ws[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 w = x[4 * at + i];
      v[4 * i] = __uint_as_float(w.x);
      v[4 * i + 1] = __uint_as_float(w.y);
      v[4 * i + 2] = __uint_as_float(w.z);
      v[4 * i + 3] = __uint_as_float(w.w);
    }
  }
}

// Greatest |v| by its bits: infinities above every number, NaNs above those.
__device__ __forceinline__ uint32_t amax_bits16(uint32_t m, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t m) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
  return m;
}

// What a row's elements are divided by.  x / s correctly rounded is one product
// and two fused multiply-adds with the rounded reciprocal y of s (Markstein:
// q = x y, r = x - q s exactly, q + r y rounds as x / s does), where neither y nor
// r leaves the normal range or the code is 0 anyway; `direct` scales, below
// 2^-90, take the division itself.
struct Divisor {
  float s, y;
  bool live, direct;
};
__device__ __forceinline__ Divisor divisor(uint32_t amax_bits) {
  Divisor d;
  d.s = __uint_as_float(amax_bits) / 127.0f;
  d.y = 1.0f / d.s;
  d.live = amax_bits < 0x7F800000u && d.s > 0.0f;  // positive and finite
  d.direct = d.s < 0x1p-90f;
  return d;
}

// Codes of 16 elements (element i in byte i).  The clamp comes before the
// rounding, which is to whole numbers either way; adding 1.5 * 2^23 rounds to
// nearest even and leaves the whole number's low byte in the sum's.
template <bool DIRECT>
__device__ __forceinline__ uint4 encode16_by(const float (&v)[16], const Divisor& d) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = v[4 * i + j], q = x * d.y;
      const float t = DIRECT ? x / d.s : __builtin_fmaf(__builtin_fmaf(-q, d.s, x), d.y, q);
      b[j] = __float_as_uint(__builtin_amdgcn_fmed3f(t, -127.0f, 127.0f) + 12582912.0f);
    }
    w[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0C0C0400u),
                                 __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), 0x05040100u);
    w[i] = d.live ? w[i] : 0u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 encode16(const float (&v)[16], const Divisor& d) {
  return d.direct ? encode16_by<true>(v, d) : encode16_by<false>(v, d);
}

// LANES lanes per row of at most NC * LANES * 16 elements; NC == 0: a workgroup.
template <bool BF16, int LANES, int NC, bool SCATTER>
__global__ __launch_bounds__(256) void int8_quantize_kernel(Int8Params p) {
  constexpr int NT = LANES, GROUPS = 256 / NT;
  static_assert(NC ? LANES == 16 || LANES == 64 : LANES == 256, "lanes of a row");
  const int t = threadIdx.x % NT;
  const int64_t n16 = p.K / 16, first = (int64_t)blockIdx.x * GROUPS + threadIdx.x / NT,
                step = (int64_t)gridDim.x * GROUPS;
  uint4* q = reinterpret_cast<uint4*>(p.q);
  const auto put = [&](int64_t row, int64_t u, uint4 codes) {
    if constexpr (SCATTER) {
      for (int j = 0; j < p.k; ++j) {
        const int32_t r = p.dest[row * p.k + j];
        if (r >= 0) q[(int64_t)r * n16 + u] = codes;
      }
    } else {
      q[row * n16 + u] = codes;
    }
  };
  for (int64_t row = first; row < p.rows; row += step) {
    float v[NC ? NC : 1][16];
    uint32_t m = 0;
    if constexpr (NC > 0) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (c * NT + t < n16) load16<BF16>(p.x, row * n16 + c * NT + t, v[c]);
        else
#pragma unroll
          for (int i = 0; i < 16; ++i) v[c][i] = 0.0f;
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) m = amax_bits16(m, v[c]);
      m = lanes_max<NT>(m);
    } else {
      __shared__ uint32_t red[4];
      for (int64_t u = t; u < n16; u += NT) {
        load16<BF16>(p.x, row * n16 + u, v[0]);
        m = amax_bits16(m, v[0]);
      }
      m = lanes_max<64>(m);
      __syncthreads();  // the row before has been read
      if ((t & 63) == 0) red[t >> 6] = m;
      __syncthreads();
      m = max(max(red[0], red[1]), max(red[2], red[3]));
    }
    const Divisor d = divisor(m);
    if constexpr (NC > 0) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (c * NT + t < n16) put(row, c * NT + t, encode16(v[c], d));
    } else {
      for (int64_t u = t; u < n16; u += NT) {
        load16<BF16>(p.x, row * n16 + u, v[0]);
        put(row, u, encode16(v[0], d));
      }
    }
    if (t == 0) {
      if constexpr (SCATTER) {
        for (int j = 0; j < p.k; ++j) {
          const int32_t r = p.dest[row * p.k + j];
          if (r >= 0) p.scales[r] = d.s;
        }
      } else {
        p.scales[row] = d.s;
      }
    }
  }
  if constexpr (SCATTER) {  // rows of skipped assignments: zeros
    int64_t valid = p.offsets[p.E];
    valid = valid < 0 ? 0 : valid > p.R ? p.R : valid;
    for (int64_t row = valid + first; row < p.R; row += step) {
      for (int64_t u = t; u < n16; u += NT) q[row * n16 + u] = make_uint4(0, 0, 0, 0);
      if (t == 0) p.scales[row] = 0.0f;
    }
  }
}

template <bool SCATTER>
int launch(const Int8Params& p, bool bf16, hipStream_t st) {
  const bool bf = bf16;
#define NVQ(B, L, NC)                                                                                         \
  do {                                                                                                        \
    const int64_t n = cdiv(p.rows > 0 ? p.rows : 1, 256 / (L));                                               \
    int8_quantize_kernel<B, L, NC, SCATTER><<<(unsigned)(n < kMaxStreamGrid ? n : kMaxStreamGrid), 256, 0, st>>>(p); \
  } while (0)
#define NVQ2(L, NC)           \
  do {                        \
    if (bf) NVQ(true, L, NC); \
    else NVQ(false, L, NC);   \
  } while (0)
  if (p.K <= 256) NVQ2(16, 1);
  else if (p.K <= 512) NVQ2(16, 2);
  else if (p.K <= 768) NVQ2(16, 3);
  else if (p.K <= 1024) NVQ2(64, 1);
  else if (p.K <= 2048) NVQ2(64, 2);
  else if (p.K <= 4096) NVQ2(64, 4);
  else NVQ2(256, 0);
#undef NVQ2
#undef NVQ
  return launch_status();
}

}  // namespace

// Enqueue the quantize-scatter of T token rows of D elements into the permuted
// rows given by dest (metadata already enqueued; T > 0, D % 16 == 0; rows of no
// elements get scales of 0).
int int8_quantize_scatter_launch(const void* x, int x_dtype, int64_t T, int k, int64_t D, const int32_t* dest,
                                 const int32_t* offsets, int E, int8_t* q, float* scales, hipStream_t st) {
  Int8Params p{};
  p.x = reinterpret_cast<const uint4*>(x);
  p.rows = T;
  p.K = D;
  p.q = q;
  p.scales = scales;
  p.dest = dest;
  p.offsets = offsets;
  p.R = T * k;
  p.k = k;
  p.E = E;
  return launch<true>(p, x_dtype == NVFP4MOE_BF16, st);
}

}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" int int8_quantize(const void* x, int x_dtype, int64_t rows, int64_t K, int8_t* q, float* scales,
                             nvfp4moe_stream_t stream) {
  if (rows < 0 || K < 0) return NVFP4MOE_EINVAL;
  if (x_dtype != NVFP4MOE_F32 && x_dtype != NVFP4MOE_BF16) return NVFP4MOE_EINVAL;
  if (rows > 0 && (!scales || (K > 0 && (!x || !q)))) return NVFP4MOE_EINVAL;
  if (K % 16 != 0 || !aligned(x, 16) || !aligned(q, 16) || !aligned(scales, 4)) return NVFP4MOE_ESHAPE;
  const int arch = check_arch();
  if (arch != NVFP4MOE_OK) return arch;
  if (rows == 0) return NVFP4MOE_OK;
  Int8Params p{};
  p.x = reinterpret_cast<const uint4*>(x);
  p.rows = rows;
  p.K = K;
  p.q = q;
  p.scales = scales;
  return launch<false>(p, x_dtype == NVFP4MOE_BF16, as_stream(stream));
}
