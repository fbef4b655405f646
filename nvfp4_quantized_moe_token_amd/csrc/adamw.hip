// AdamW over many tensors in one launch, with moments in fp32 or in 8 bits.
//
// The learner's update after the backward pass; the pages name the learner
// but no optimizer ("miniTE ускоряет RL в NVFP4 на B300", intro), so this is
// the published rule with decoupled weight decay:
//   g = grad * grad_scale
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g g
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// in fp32, one rounding per operation (contraction is off), so that the
// moments are the same bits on every launch shape.
//
// 8-bit moments: blocks of 256 consecutive elements share one fp32 scale.
//   m: E4M3 of m / s_m, s_m = max |m| * fl(1 / 448).
//   v: an unsigned format with 3 mantissa bits and 2^-32 of range below the
//      block's max s_v: code c > 0 stands for the float with bits
//      (c + 762) << 20 (254 is 1.0, 255 NaN), code 0 for zero.  v is kept as
//      itself, not as its root, so that rounding is unbiased in v.
// Both are rounded stochastically: with b2 = 0.999 a step moves v by less
// than half a code, and round-to-nearest would freeze it.  The random bits
// are a hash of (seed, step, tensor, element), so a step is reproducible.  A
// positive v never becomes 0 (an update divides by its root).  The update
// itself uses the unrounded moments.
// bf16 parameters (no fp32 master) are rounded stochastically too, for the
// same reason.
//
// Layout.  One wave takes one 256-element block: 4 consecutive elements per
// lane (16-byte loads of fp32), so the scale of a block is one wave
// reduction and nothing is shared between waves.  A workgroup takes kChunk
// consecutive elements of one tensor; the tensors' pointers and first
// workgroups travel in the kernel arguments, 72 tensors per launch (56
// with 8-bit moments).
// The bound is HBM: 30 bytes per element with fp32 moments, a bf16 copy and
// fp32 gradients, 18 with 8-bit moments.  604 M elements: 3.41 ms (5.3 TB/s)
// and 2.16 ms (5.1 TB/s; 2.37 when every wave raised the betas to the step
// itself), reading 8-bit moments back 1.13 ms (5.3 TB/s).  A copy of 4 GiB
// reaches 4.6 TB/s, a fill 6.8.
#include <math.h>

#include "nvfp4_codec.hpp"

namespace nvfp4moe {
namespace {

constexpr int kStateBlock = NVFP4MOE_ADAMW_BLOCK;  // elements per 8-bit scale: one wave, 4 per lane
constexpr int kWaveBlocks = 4;                     // blocks per wave
constexpr int kChunk = 4 * kWaveBlocks * kStateBlock;  // elements per workgroup (4 waves)
static_assert(kStateBlock == 256, "one wave holds a block");

struct Tensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  uint16_t* copy;
  int64_t n;
};
struct Scales {
  float* m;
  float* v;
};
template <bool STATE8>
struct Args {
  static constexpr bool kState8 = STATE8;
  static constexpr int kMaxTensors = STATE8 ? 56 : 72;  // per launch: their records fit 4 KiB of arguments
  Tensor t[kMaxTensors];
  Scales s[STATE8 ? kMaxTensors : 1];
  int32_t first[kMaxTensors + 1];  // first workgroup of each tensor
  int32_t n_tensors;
  int32_t base;                    // ordinal of t[0] in the caller's list
  uint32_t seed;
  float lr, wd, b1, c1, b2, c2, eps;
  float rate, inv_root;            // of `step` and `lr`, when neither comes from the device
  double beta1, beta2;
  int64_t step;
  const int64_t* step_dev;
  const float* lr_dev;
  const float* grad_scale;
  const int32_t* skip;
};
static_assert(sizeof(Args<false>) <= 4096 && sizeof(Args<true>) <= 4096, "kernel arguments");

// The tensor of this workgroup.
template <bool STATE8>
__device__ __forceinline__ int tensor_of_group(const Args<STATE8>& a) {
  int ti = 0;
#pragma unroll
  for (int step = 64; step > 0; step >>= 1)
    if (ti + step < a.n_tensors && a.first[ti + step] <= (int)blockIdx.x) ti += step;
  return ti;
}

// The bias corrections of step t: lr / (1 - b1^t) and 1 / sqrt(1 - b2^t), the
// powers by repeated squaring in fp64.  The same operations on the host and on
// the device, so a captured step gives the same bits.
__host__ __device__ inline double power(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1, b *= b)
    if (t & 1) r *= b;
  return r;
}
__host__ __device__ inline float corrected_rate(float lr, double beta1, int64_t t) {
  return (float)((double)lr / (1.0 - power(beta1, t)));
}
__host__ __device__ inline float corrected_root(double beta2, int64_t t) {
  return (float)(1.0 / sqrt(1.0 - power(beta2, t)));
}

// 32-bit mixer: multiply and xor-shift, constants from the fractional digits
// of the golden ratio and the square root of 3.
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B9u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ (x >> 16);
}
__device__ __forceinline__ uint32_t random_bits(uint32_t key, int64_t i) {
  return mix(((uint32_t)i * 0x9E3779B1u) ^ key ^ ((uint32_t)((uint64_t)i >> 32) * 0x6A09E667u));
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __builtin_inff(); }

// First moment x with block scale s > 0 (r: 16 random bits).  Not finite: NaN.
__device__ __forceinline__ uint32_t encode_m(float x, float s, uint32_t r) {
  const uint32_t sign = (__float_as_uint(x) >> 24) & 0x80u;
  if (!finite(x)) return sign | 0x7Fu;
  if (!(s > 0.0f)) return sign;
  const float y = fminf(fabsf(x) / s, 448.0f);
  // below the normal range the codes are steps of 2^-9
  if (y < 0.015625f) return sign | (uint32_t)(int)__builtin_floorf(y * 512.0f + (float)r * 0x1p-16f);
  return sign | (((__float_as_uint(y) + (r << 4)) >> 20) - (120u << 3));
}
__device__ __forceinline__ uint32_t encode_v(float x, float s, uint32_t r) {
  if (!finite(x)) return 255u;
  if (!(x > 0.0f)) return 0u;  // (then s, the block's maximum, is positive too)
  const float y = x / s;       // 0 when x is below 2^-149 of s: the lowest code all the same
  const int c = (int)((__float_as_uint(y) + (r << 4)) >> 20) - 762;
  return (uint32_t)(c < 1 ? 1 : c > 254 ? 254 : c);
}
__device__ __forceinline__ float decode_v(uint32_t c, float s) {
  if (c == 0) return 0.0f;
  if (c == 255) return __builtin_nanf("");
  return __uint_as_float((c + 762u) << 20) * s;
}

// 4 consecutive values at element i of a tensor; `whole` (wave-uniform): the
// block lies inside the tensor and its vectors are aligned.
template <bool BF16>
__device__ __forceinline__ void load4(const void* base, int64_t i, int64_t n, bool whole, float (&v)[4]) {
  if (whole) {
    if constexpr (BF16) {
      const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(base) + i);
      v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    } else {
      const float4 w = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + i);
      v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (i + q >= n) v[q] = 0.0f;
      else if constexpr (BF16) v[q] = bf16_lo(reinterpret_cast<const uint16_t*>(base)[i + q]);
      else v[q] = reinterpret_cast<const float*>(base)[i + q];
    }
  }
}
__device__ __forceinline__ void store4_f32(void* base, int64_t i, int64_t n, bool whole, const float (&v)[4]) {
  float* f = reinterpret_cast<float*>(base);
  if (whole) {
    *reinterpret_cast<float4*>(f + i) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < n) f[i + q] = v[q];
  }
}
__device__ __forceinline__ void store4_u16(uint16_t* base, int64_t i, int64_t n, bool whole, uint32_t lo, uint32_t hi) {
  if (whole) {
    *reinterpret_cast<uint2*>(base + i) = make_uint2(lo, hi);
  } else {
    const uint32_t w[2] = {lo, hi};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < n) base[i + q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
  }
}
__device__ __forceinline__ uint32_t load4_u8(const void* base, int64_t i, int64_t n, bool whole) {
  const uint8_t* b = reinterpret_cast<const uint8_t*>(base);
  if (whole) return *reinterpret_cast<const uint32_t*>(b + i);
  uint32_t w = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (i + q < n) w |= (uint32_t)b[i + q] << (8 * q);
  return w;
}
__device__ __forceinline__ void store4_u8(void* base, int64_t i, int64_t n, bool whole, uint32_t w) {
  uint8_t* b = reinterpret_cast<uint8_t*>(base);
  if (whole) {
    *reinterpret_cast<uint32_t*>(b + i) = w;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (i + q < n) b[i + q] = (uint8_t)(w >> (8 * q));
  }
}

template <bool P_BF16, bool G_BF16, bool STATE8>
__global__ __launch_bounds__(256) void adamw_kernel(const Args<STATE8> a) {
  if (a.skip && *a.skip != 0) return;
  const int ti = tensor_of_group(a);
  const Tensor& t = a.t[ti];
  const Scales& sc = a.s[STATE8 ? ti : 0];
  const int64_t n = t.n;
  const int64_t chunk = (int64_t)((int)blockIdx.x - a.first[ti]) * kChunk;
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;

  const int64_t step = a.step_dev ? *a.step_dev : a.step;
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
  float rate = a.rate, inv_root = a.inv_root;
  if (a.step_dev || a.lr_dev) {
    rate = corrected_rate(lr, a.beta1, step);
    inv_root = corrected_root(a.beta2, step);
  }
  const float keep = 1.0f - lr * a.wd;
  uint32_t key = 0;
  if (STATE8 || P_BF16) key = mix(mix(mix(a.seed) + (uint32_t)step) + (uint32_t)(a.base + ti));
  const uintptr_t addr = (uintptr_t)t.p | (uintptr_t)t.g | (uintptr_t)t.copy;
  const bool vec = (addr & 15) == 0 && (STATE8 ? (((uintptr_t)t.m | (uintptr_t)t.v) & 3) == 0
                                               : (((uintptr_t)t.m | (uintptr_t)t.v) & 15) == 0);

#pragma unroll 2
  for (int b = 0; b < kWaveBlocks; ++b) {
    const int64_t i0 = chunk + (int64_t)(b * 4 + wid) * kStateBlock;
    if (i0 >= n) break;
    const bool whole = vec && i0 + kStateBlock <= n;
    const int64_t i = i0 + lane * 4;
    float p[4], g[4], m[4], v[4];
    load4<P_BF16>(t.p, i, n, whole, p);
    load4<G_BF16>(t.g, i, n, whole, g);
    if constexpr (STATE8) {
      const uint32_t mc = load4_u8(t.m, i, n, whole), vc = load4_u8(t.v, i, n, whole);
      const float sm = sc.m[i0 / kStateBlock], sv = sc.v[i0 / kStateBlock];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        m[q] = e4m3_decode((mc >> (8 * q)) & 0xFF) * sm;
        v[q] = decode_v((vc >> (8 * q)) & 0xFF, sv);
      }
    } else {
      load4<false>(t.m, i, n, whole, m);
      load4<false>(t.v, i, n, whole, v);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float gq = g[q] * gs;
      m[q] = a.b1 * m[q] + a.c1 * gq;
      v[q] = a.b2 * v[q] + a.c2 * (gq * gq);
      p[q] = p[q] * keep - rate * (m[q] / (sqrtf(v[q]) * inv_root + a.eps));
    }
    uint32_t r[4];
    if (STATE8 || P_BF16) {
#pragma unroll
      for (int q = 0; q < 4; ++q) r[q] = random_bits(key, i + q);
    }
    if constexpr (P_BF16) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t bits = __float_as_uint(p[q]);
        w[q] = finite(p[q]) ? (bits + (mix(r[q] + 0x6A09E667u) >> 16)) >> 16 : f32_to_bf16_rne(p[q]);
      }
      store4_u16(reinterpret_cast<uint16_t*>(t.p), i, n, whole, w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    } else {
      store4_f32(t.p, i, n, whole, p);
      if (t.copy) store4_u16(t.copy, i, n, whole, pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]));
    }
    if constexpr (STATE8) {
      float am = 0.0f, av = 0.0f;  // over the finite values (elements past n are zeros)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        am = fmaxf(am, finite(m[q]) ? fabsf(m[q]) : 0.0f);
        av = fmaxf(av, finite(v[q]) ? v[q] : 0.0f);
      }
      am = wave_max(am);
      av = wave_max(av);
      const float sm = am * (1.0f / 448.0f);
      uint32_t mc = 0, vc = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        mc |= encode_m(m[q], sm, r[q] >> 16) << (8 * q);
        vc |= encode_v(v[q], av, r[q] & 0xFFFFu) << (8 * q);
      }
      store4_u8(t.m, i, n, whole, mc);
      store4_u8(t.v, i, n, whole, vc);
      if (lane == 0) {
        sc.m[i0 / kStateBlock] = sm;
        sc.v[i0 / kStateBlock] = av;
      }
    } else {
      store4_f32(t.m, i, n, whole, m);
      store4_f32(t.v, i, n, whole, v);
    }
  }
}

// fp32 values of 8-bit moments.
__global__ __launch_bounds__(256) void adamw_read_kernel(const Args<true> a) {
  const int ti = tensor_of_group(a);
  const Tensor& t = a.t[ti];
  const Scales& sc = a.s[ti];
  float* om = reinterpret_cast<float*>(t.p);
  float* ov = reinterpret_cast<float*>(t.copy);
  const int64_t n = t.n, chunk = (int64_t)((int)blockIdx.x - a.first[ti]) * kChunk;
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const bool vec = (((uintptr_t)om | (uintptr_t)ov) & 15) == 0 && (((uintptr_t)t.m | (uintptr_t)t.v) & 3) == 0;
#pragma unroll
  for (int b = 0; b < kWaveBlocks; ++b) {
    const int64_t i0 = chunk + (int64_t)(b * 4 + wid) * kStateBlock;
    if (i0 >= n) break;
    const bool whole = vec && i0 + kStateBlock <= n;
    const int64_t i = i0 + lane * 4;
    const uint32_t mc = load4_u8(t.m, i, n, whole), vc = load4_u8(t.v, i, n, whole);
    const float sm = sc.m[i0 / kStateBlock], sv = sc.v[i0 / kStateBlock];
    float m[4], v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      m[q] = e4m3_decode((mc >> (8 * q)) & 0xFF) * sm;
      v[q] = decode_v((vc >> (8 * q)) & 0xFF, sv);
    }
    store4_f32(om, i, n, whole, m);
    store4_f32(ov, i, n, whole, v);
  }
}

// Fills launches of up to kMaxTensors tensors and calls go(args, workgroups)
// for each; tensors without elements are left out.
template <bool STATE8, class F>
int for_launches(const nvfp4moe_adamw_tensor* list, int count, Args<STATE8>& a, F go) {
  a.n_tensors = 0;
  int64_t groups = 0;
  for (int i = 0; i <= count; ++i) {
    const int64_t n = i < count ? list[i].n : 0, need = cdiv(n, kChunk);
    // the ordinals of a launch's tensors are consecutive: an empty tensor keeps its place
    if (i == count || a.n_tensors == a.kMaxTensors || groups + need > 0x7FFFFFFFLL) {
      if (groups > 0) {
        a.first[a.n_tensors] = (int32_t)groups;
        const int rc = go(a, (unsigned)groups);
        if (rc != NVFP4MOE_OK) return rc;
      }
      a.n_tensors = 0;
      groups = 0;
      if (i == count) break;
    }
    if (a.n_tensors == 0) a.base = i;
    const nvfp4moe_adamw_tensor& s = list[i];
    a.t[a.n_tensors] = Tensor{s.param, s.grad, s.exp_avg, s.exp_avg_sq, reinterpret_cast<uint16_t*>(s.param_bf16), n};
    if (STATE8) a.s[a.n_tensors] = Scales{s.avg_scale, s.avg_sq_scale};
    a.first[a.n_tensors++] = (int32_t)groups;
    groups += need;
  }
  return NVFP4MOE_OK;
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" int adamw_step(const nvfp4moe_adamw_tensor* tensors, int count, int param_dtype, int grad_dtype,
                          int state_bits, double lr, double beta1, double beta2, double eps, double weight_decay,
                          int64_t step, const int64_t* step_dev, const float* lr_dev, const float* grad_scale,
                          const int32_t* skip, uint32_t seed, nvfp4moe_stream_t stream) {
  if (count < 0 || (count > 0 && !tensors)) return NVFP4MOE_EINVAL;
  if (param_dtype != NVFP4MOE_F32 && param_dtype != NVFP4MOE_BF16) return NVFP4MOE_EINVAL;
  if (grad_dtype != NVFP4MOE_F32 && grad_dtype != NVFP4MOE_BF16) return NVFP4MOE_EINVAL;
  if (state_bits != 8 && state_bits != 32) return NVFP4MOE_EINVAL;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0)) return NVFP4MOE_EINVAL;
  if (!step_dev && step < 1) return NVFP4MOE_EINVAL;
  const int pb = dtype_bytes(param_dtype), gb = dtype_bytes(grad_dtype), sb = state_bits / 8;
  for (int i = 0; i < count; ++i) {
    const nvfp4moe_adamw_tensor& t = tensors[i];
    if (t.n < 0) return NVFP4MOE_EINVAL;
    if (t.param_bf16 && param_dtype != NVFP4MOE_F32) return NVFP4MOE_EINVAL;
    if (t.n == 0) continue;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return NVFP4MOE_EINVAL;
    if (state_bits == 8 && (!t.avg_scale || !t.avg_sq_scale)) return NVFP4MOE_EINVAL;
    if (t.n > (int64_t)kChunk * 0x7FFFFFFFLL) return NVFP4MOE_ESHAPE;
    if (!aligned(t.param, pb) || !aligned(t.grad, gb) || !aligned(t.exp_avg, sb) || !aligned(t.exp_avg_sq, sb) ||
        !aligned(t.avg_scale, 4) || !aligned(t.avg_sq_scale, 4) || !aligned(t.param_bf16, 2))
      return NVFP4MOE_ESHAPE;
  }
  if (!aligned(step_dev, 8) || !aligned(lr_dev, 4) || !aligned(grad_scale, 4) || !aligned(skip, 4))
    return NVFP4MOE_ESHAPE;
  const int arch = check_arch();
  if (arch != NVFP4MOE_OK) return arch;
  hipStream_t st = as_stream(stream);
  const bool p16 = param_dtype == NVFP4MOE_BF16, g16 = grad_dtype == NVFP4MOE_BF16;
  auto run = [&](auto a) {
    constexpr bool S = decltype(a)::kState8;
    a.seed = seed;
    a.lr = (float)lr;
    a.wd = (float)weight_decay;
    a.b1 = (float)beta1;
    a.c1 = (float)(1.0 - beta1);
    a.b2 = (float)beta2;
    a.c2 = (float)(1.0 - beta2);
    a.eps = (float)eps;
    a.beta1 = beta1;
    a.beta2 = beta2;
    a.step = step;
    a.rate = step > 0 ? corrected_rate(a.lr, beta1, step) : 0.0f;
    a.inv_root = step > 0 ? corrected_root(beta2, step) : 0.0f;
    a.step_dev = step_dev;
    a.lr_dev = lr_dev;
    a.grad_scale = grad_scale;
    a.skip = skip;
    return for_launches(tensors, count, a, [&](const Args<S>& args, unsigned grid) {
      if (p16 && g16) adamw_kernel<true, true, S><<<grid, 256, 0, st>>>(args);
      else if (p16) adamw_kernel<true, false, S><<<grid, 256, 0, st>>>(args);
      else if (g16) adamw_kernel<false, true, S><<<grid, 256, 0, st>>>(args);
      else adamw_kernel<false, false, S><<<grid, 256, 0, st>>>(args);
      return launch_status();
    });
  };
  return state_bits == 8 ? run(Args<true>{}) : run(Args<false>{});
}

extern "C" int adamw_read_state(const nvfp4moe_adamw_tensor* tensors, int count, float* const* avg_out,
                                float* const* avg_sq_out, nvfp4moe_stream_t stream) {
  if (count < 0 || (count > 0 && (!tensors || !avg_out || !avg_sq_out))) return NVFP4MOE_EINVAL;
  for (int i = 0; i < count; ++i) {
    const nvfp4moe_adamw_tensor& t = tensors[i];
    if (t.n < 0) return NVFP4MOE_EINVAL;
    if (t.n == 0) continue;
    if (!t.exp_avg || !t.exp_avg_sq || !t.avg_scale || !t.avg_sq_scale || !avg_out[i] || !avg_sq_out[i])
      return NVFP4MOE_EINVAL;
    if (t.n > (int64_t)kChunk * 0x7FFFFFFFLL) return NVFP4MOE_ESHAPE;
    if (!aligned(t.avg_scale, 4) || !aligned(t.avg_sq_scale, 4) || !aligned(avg_out[i], 4) ||
        !aligned(avg_sq_out[i], 4))
      return NVFP4MOE_ESHAPE;
  }
  const int arch = check_arch();
  if (arch != NVFP4MOE_OK) return arch;
  hipStream_t st = as_stream(stream);
  Args<true> a = {};
  return for_launches(tensors, count, a, [&](Args<true>& args, unsigned grid) {
    for (int i = 0; i < args.n_tensors; ++i) {
      args.t[i].p = avg_out[args.base + i];
      args.t[i].copy = reinterpret_cast<uint16_t*>(avg_sq_out[args.base + i]);
    }
    adamw_read_kernel<<<grid, 256, 0, st>>>(args);
    return launch_status();
  });
}
