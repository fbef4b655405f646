// SiLU-gated expert activation between the two grouped GEMMs, with the amax
// of its output folded in so the requantization reuses it ("miniTE報告、
// NVFP4強化学習の安定性を検証", fourth paragraph: op fusion, amax reuse).
// H = silu(G) * U with Y1 = [G | U] per row; fp32 math, bf16 storage.
#include "mx_codec.hpp"

namespace nvfp4moe {
namespace {

__global__ __launch_bounds__(256) void silu_fwd_kernel(const uint16_t* __restrict__ y1, int64_t R, int64_t F,
                                                       uint16_t* __restrict__ h, float* __restrict__ amax_out) {
  const int64_t n8 = F / 8;
  const int64_t total = R * n8;
  float m = 0.0f;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / n8, c = (i - r * n8) * 8;
    const uint4 gw = *reinterpret_cast<const uint4*>(y1 + r * 2 * F + c);
    const uint4 uw = *reinterpret_cast<const uint4*>(y1 + r * 2 * F + F + c);
    const uint32_t g[4] = {gw.x, gw.y, gw.z, gw.w}, u[4] = {uw.x, uw.y, uw.z, uw.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float g0 = bf16_lo(g[j]), g1 = bf16_hi(g[j]);
      const float h0 = silu_gate(g0, bf16_lo(u[j]));
      const float h1 = silu_gate(g1, bf16_hi(u[j]));
      o[j] = pack_bf16x2(h0, h1);
      m = fmaxf(m, fmaxf(fabsf(bf16_lo(o[j])), fabsf(bf16_hi(o[j]))));
    }
    *reinterpret_cast<uint4*>(h + r * F + c) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  if (amax_out) block_atomic_max<256>(amax_out, m);
}

// dY1 = [dG | dU] from dH and Y1; with amax_out, max |dY1| (the max of the
// fp32 results rounded once to bf16, equal to the max of the stored values)
// with one atomic per workgroup.
template <int P>
__global__ __launch_bounds__(256) void silu_bwd_kernel(const uint16_t* __restrict__ y1, const uint16_t* __restrict__ dh,
                                                       int64_t R, int64_t F, uint16_t* __restrict__ dy1,
                                                       float* __restrict__ amax_out) {
  const int64_t n8 = F / 8;
  const int64_t total = R * n8;
  float m = 0.0f;
  // P pieces of 8 per thread and step, 256 apart: every load of the step is
  // issued before its first store.  A wave's memory counter retires in
  // order, so a load issued after a store also waits for that store; with
  // the capped grid of the amax variant a thread takes many pieces, and a
  // load-store-load loop would wait on every store.  Pieces past the end
  // load the last piece again (valid memory, an element of the tensor, so
  // the max is unchanged) and store nothing.
  for (int64_t base = blockIdx.x * (256ll * P) + threadIdx.x; base < total;
       base += (int64_t)gridDim.x * 256 * P) {
    uint4 gw[P], uw[P], dw[P];
    int64_t at[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t i0 = base + 256 * p, i = i0 < total ? i0 : total - 1;
      const int64_t r = i / n8, c = (i - r * n8) * 8;
      at[p] = r * 2 * F + c;
      gw[p] = *reinterpret_cast<const uint4*>(y1 + r * 2 * F + c);
      uw[p] = *reinterpret_cast<const uint4*>(y1 + r * 2 * F + F + c);
      dw[p] = *reinterpret_cast<const uint4*>(dh + r * F + c);
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const uint32_t g[4] = {gw[p].x, gw[p].y, gw[p].z, gw[p].w}, u[4] = {uw[p].x, uw[p].y, uw[p].z, uw[p].w};
      const uint32_t d[4] = {dw[p].x, dw[p].y, dw[p].z, dw[p].w};
      uint32_t og[4], ou[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float gg[2] = {bf16_lo(g[j]), bf16_hi(g[j])}, uu[2] = {bf16_lo(u[j]), bf16_hi(u[j])};
        float dd[2] = {bf16_lo(d[j]), bf16_hi(d[j])};
        float rg[2], ru[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float sg = sigmoid_f32(gg[q]);
          const float dsilu = sg * (1.0f + gg[q] * (1.0f - sg));
          rg[q] = dd[q] * uu[q] * dsilu;
          ru[q] = dd[q] * gg[q] * sg;
          m = fmaxf(m, fmaxf(fabsf(rg[q]), fabsf(ru[q])));
        }
        og[j] = pack_bf16x2(rg[0], rg[1]);
        ou[j] = pack_bf16x2(ru[0], ru[1]);
      }
      if (base + 256 * p < total) {
        *reinterpret_cast<uint4*>(dy1 + at[p]) = make_uint4(og[0], og[1], og[2], og[3]);
        *reinterpret_cast<uint4*>(dy1 + at[p] + F) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
      }
    }
  }
  if (amax_out) block_atomic_max<256>(amax_out, bf16_lo(pack_bf16x2(m, m)));
}

// dY1 and H from Y1 kept as MXINT8 (codes [R][2F], scales [R][2F / 32]): the
// gate's backward of a forward pass that stored neither Y1 nor H in bf16.  H is
// taken from the same values, for the weight gradient of the product it went
// into.  HBM bound: 2 F (33/32) + 2 F bytes a row in, 4 F + 2 F out.  A thread
// takes 16 features: whole 16-byte accesses of every tensor.  65536 rows of 768
// features, 506 MB: 85 to 94 us (5.4 to 5.9 TB/s).
__global__ __launch_bounds__(256) void silu_bwd_mx_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                          const uint4* __restrict__ dh, int64_t R, int64_t F,
                                                          uint4* __restrict__ dy1, uint4* __restrict__ h) {
  const int64_t n16 = F / 16, total = R * n16;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / n16, c = i - r * n16;  // row, 16-feature piece
    const int64_t at = r * 2 * n16 + c;
    const uint4 gq = reinterpret_cast<const uint4*>(q)[at], uq = reinterpret_cast<const uint4*>(q)[at + n16];
    const uint4 d0 = dh[2 * i], d1 = dh[2 * i + 1];
    const float gs = int8_step(s[at >> 1]), us = int8_step(s[(at + n16) >> 1]);  // (n16 is even)
    const uint32_t g[4] = {gq.x, gq.y, gq.z, gq.w}, u[4] = {uq.x, uq.y, uq.z, uq.w};
    const uint32_t d[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
    uint32_t og[8], ou[8], oh[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float rg[2], ru[2], rh[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int e = 2 * j + k;
        const float gv = decode_int8((int8_t)(g[e / 4] >> (8 * (e % 4))), gs);
        const float uv = decode_int8((int8_t)(u[e / 4] >> (8 * (e % 4))), us);
        const float dv = k ? bf16_hi(d[j]) : bf16_lo(d[j]);
        const float sg = sigmoid_f32(gv);
        rg[k] = dv * uv * (sg * (1.0f + gv * (1.0f - sg)));
        ru[k] = dv * gv * sg;
        rh[k] = gv * sg * uv;
      }
      og[j] = pack_bf16x2(rg[0], rg[1]);
      ou[j] = pack_bf16x2(ru[0], ru[1]);
      oh[j] = pack_bf16x2(rh[0], rh[1]);
    }
    dy1[2 * at] = make_uint4(og[0], og[1], og[2], og[3]);
    dy1[2 * at + 1] = make_uint4(og[4], og[5], og[6], og[7]);
    dy1[2 * (at + n16)] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
    dy1[2 * (at + n16) + 1] = make_uint4(ou[4], ou[5], ou[6], ou[7]);
    if (h) {
      h[2 * i] = make_uint4(oh[0], oh[1], oh[2], oh[3]);
      h[2 * i + 1] = make_uint4(oh[4], oh[5], oh[6], oh[7]);
    }
  }
}

// With an amax the grid is capped (one same-address atomic per workgroup).
inline unsigned grid_for(int64_t work) {
  const int64_t g = cdiv(work, 256);
  return (unsigned)(g < 1 ? 1 : g > kAmaxGrid ? kAmaxGrid : g);
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" int silu_gate_fwd(const void* y1, int64_t R, int64_t F, void* h, float* amax_out,
                             nvfp4moe_stream_t stream) {
  if (R < 0 || F < 0) return NVFP4MOE_EINVAL;
  if (R * F > 0 && (!y1 || !h)) return NVFP4MOE_EINVAL;
  if (F % 8 != 0 || !aligned(y1, 16) || !aligned(h, 16)) return NVFP4MOE_ESHAPE;
  const int arch = check_arch();
  if (arch != NVFP4MOE_OK) return arch;
  hipStream_t st = as_stream(stream);
  if (amax_out) fill_u32_kernel<<<1, 64, 0, st>>>(reinterpret_cast<uint32_t*>(amax_out), 0u, 1);
  if (R * F > 0)
    silu_fwd_kernel<<<grid_for(R * F / 8), 256, 0, st>>>(reinterpret_cast<const uint16_t*>(y1), R, F,
                                                          reinterpret_cast<uint16_t*>(h), amax_out);
  return launch_status();
}

extern "C" int silu_gate_bwd(const void* y1, const void* dh, int64_t R, int64_t F, void* dy1, float* amax_out,
                             nvfp4moe_stream_t stream) {
  if (R < 0 || F < 0) return NVFP4MOE_EINVAL;
  if (R * F > 0 && (!y1 || !dh || !dy1)) return NVFP4MOE_EINVAL;
  if (F % 8 != 0 || !aligned(y1, 16) || !aligned(dh, 16) || !aligned(dy1, 16)) return NVFP4MOE_ESHAPE;
  if (amax_out && !aligned(amax_out, 4)) return NVFP4MOE_ESHAPE;
  const int arch = check_arch();
  if (arch != NVFP4MOE_OK) return arch;
  hipStream_t st = as_stream(stream);
  if (amax_out) fill_u32_kernel<<<1, 64, 0, st>>>(reinterpret_cast<uint32_t*>(amax_out), 0u, 1);
  if (R * F == 0) return launch_status();
  // The amax variant's capped grid gives each thread several pieces, four
  // per step (measured on the 8k-token dY1: 0.099 -> 0.095 ms); without the
  // amax one piece per thread is faster (0.088 against 0.090 ms).
  const uint16_t* y1b = reinterpret_cast<const uint16_t*>(y1);
  const uint16_t* dhb = reinterpret_cast<const uint16_t*>(dh);
  uint16_t* dy1b = reinterpret_cast<uint16_t*>(dy1);
  if (amax_out) {
    silu_bwd_kernel<4><<<grid_for(cdiv(R * F / 8, 4)), 256, 0, st>>>(y1b, dhb, R, F, dy1b, amax_out);
  } else {
    int64_t grid = cdiv(R * F / 8, 256);
    if (grid > kMaxStreamGrid) grid = kMaxStreamGrid;
    silu_bwd_kernel<1><<<(unsigned)grid, 256, 0, st>>>(y1b, dhb, R, F, dy1b, nullptr);
  }
  return launch_status();
}

extern "C" int silu_gate_bwd_mx(const uint8_t* q_y1, const uint8_t* s_y1, const void* dh, int64_t R, int64_t F,
                                void* dy1, void* h, nvfp4moe_stream_t stream) {
  if (R < 0 || F < 0) return NVFP4MOE_EINVAL;
  if (R > 0 && F > 0 && (!q_y1 || !s_y1 || !dh || !dy1)) return NVFP4MOE_EINVAL;
  if (F % 32 != 0 || !aligned(q_y1, 16) || !aligned(dh, 16) || !aligned(dy1, 16) || !aligned(h, 16))
    return NVFP4MOE_ESHAPE;
  const int arch = check_arch();
  if (arch != NVFP4MOE_OK) return arch;
  if (R == 0 || F == 0) return NVFP4MOE_OK;
  int64_t grid = cdiv(R * (F / 16), 256);
  if (grid > kMaxStreamGrid) grid = kMaxStreamGrid;
  silu_bwd_mx_kernel<<<(unsigned)grid, 256, 0, as_stream(stream)>>>(q_y1, s_y1, reinterpret_cast<const uint4*>(dh), R, F,
                                                                    reinterpret_cast<uint4*>(dy1),
                                                                    reinterpret_cast<uint4*>(h));
  return launch_status();
}
