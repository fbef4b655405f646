// Grouped MXFP4 x MXFP4 GEMM over the contiguous per-expert layout: both
// operands E2M1 with one E8M0 scale per 32 elements along K,
//   C[r][n] = sum over blocks b of 2^(sa + sb - 254) * sum_i a_i b_i,
// accumulated in fp32 by gfx950's scaled MFMA (v_mfma_scale_f32_32x32x64_f8f6f4
// with both operands 4-bit), which takes codes and scales as they are stored.
// The 4-bit experts' products are the ones the report's ablation ends at
// ("miniTE報告、NVFP4強化学習の安定性を検証", third paragraph: W4A4; fourth:
// grouped GEMM, op fusion); this is the format that this GPU multiplies
// natively.
//
// The kernel and its epilogues are in gemm_codes.hpp.
//
// Bounds and measurements (us of the kernel, several sets of inputs in turn; 128
// experts, top-8).  A 256x256 tile of 8 waves, 64x128 each, reads 0.75 KiB of LDS
// per MFMA.  64x64 waves (128x256 and 256x128 tiles, or two workgroups per CU)
// read a third more and lose more than finer tiles save: gate+up of 8192 tokens
// 209 (198 by now) against 216 to 244.  Stages of 128 elements and a ring of four
// are no faster either (155 against 138 for a dense 4096 x 8192 x 8192 product,
// 4.0 PFLOP/s): lines are then read in halves.
//   gate+up, 8192 tokens (65536 rows, 768 features, K = 2048)      198
//   down, 16384 tokens, skewed routing (N = 2048, K = 768)         199
//   gate+up, 8192 tokens, H quantized and nothing else stored      174
//   the same with Y1 and H stored too                              221
//   the same with Y1 in 8 bits instead (the learner's checkpoint)  207
//   the skewed product with fp32 output (266 of bytes)             269
//   N = 1536, K = 2048, 16 tokens, which reach 84 of the experts (140 MB)
//                                                     26 to 28 (5.0 to 5.4 TB/s)
// Without any epilogue the first two take 129 and 117, where the MFMAs alone need
// 52 and 47: a workgroup's stores and SiLU are not hidden behind its products,
// since its accumulators fill the registers and its stages the LDS; the loop
// itself is held up by its operands' way to LDS and by row padding (a fifth of
// gate+up's MFMAs).
#include "gemm_codes.hpp"

namespace nvfp4moe {
namespace {

// Tiles by the mean rows per expert (the host does not know more): with few rows
// the work is reading the weights, so the row block is small and the ring three
// stages deep; with many it is the MFMAs, the LDS reads that feed them and the
// stores.  The row block is one that most experts' rows fit in, up to 256, where
// blocks of 192 need two.  Measured kernel times in us (before any non-temporal
// access), 128 experts, random routing, gate+up with Y1 and H stored (768
// features, K = 2048) and down (N = 2048, K = 768):
//   rows      gate+up, blocks of           down, blocks of
//             32     64    192    256      32     64    192    256
//    16     37.6   40.7   50.6   61.2    22.9   25.0   31.6   34.8
//    32     44.0   42.5   51.7   60.6    25.4   25.9   31.6   35.3
//    64     59.7   56.1   56.9   65.9    35.4   32.3   36.1   39.0
//    80     71.0   63.7   59.9   68.0    40.6   38.2   36.6   39.7
//    96     89.6   68.0   64.9   71.3    43.0   37.6   38.0   41.5
//   128    112.5   88.1   75.5   79.2    52.8   44.1   40.6   44.8
//   160    130.1   97.8   94.0   85.0    63.0   52.2   46.8   46.2
//   208    162.1  123.9  116.9   92.3    80.3   62.4   64.1   48.8
//   512    354.1  268.9  210.0  210.1   220.4  176.0  126.2  125.3
// Near the end of the blocks of 192 (other inputs each time; 192, 256):
//   144                   78.8   81.7                   45.1   47.6
//   152                   81.0   83.4                   45.4   48.4
//   160                   91.8   85.2                   49.1   49.2
template <int EPI, bool OUT32>
int launch_epi(const Params& p, hipStream_t st) {
  if (p.M <= 24 * (int64_t)p.E) return launch_tiles<MXFP4, 32, 256, 1, 4, 3, true, EPI, OUT32>(p, st);
  if (p.M <= 72 * (int64_t)p.E) return launch_tiles<MXFP4, 64, 256, 1, 4, 3, true, EPI, OUT32>(p, st);
  if (p.M <= 152 * (int64_t)p.E) return launch_tiles<MXFP4, 192, 256, 2, 4, 2, true, EPI, OUT32>(p, st);
  if (p.M <= kOnceRows * p.E) return launch_tiles<MXFP4, 256, 256, 4, 2, 2, true, EPI, OUT32>(p, st);
  return launch_tiles<MXFP4, 256, 256, 4, 2, 2, false, EPI, OUT32>(p, st);
}

// Argument checks shared by both entry points, then the launch parameters.
int check_operands(const uint8_t* a_q, const uint8_t* a_s, const uint8_t* b_q, const uint8_t* b_s,
                   const int32_t* expert_offsets, int E, int64_t M_total, int64_t N, int64_t K, Params& p) {
  if (E < 1 || M_total < 0 || N < 0 || K < 0) return NVFP4MOE_EINVAL;
  if (!expert_offsets) return NVFP4MOE_EINVAL;
  if (M_total > 0 && N > 0 && K > 0 && (!a_q || !a_s || !b_q || !b_s)) return NVFP4MOE_EINVAL;
  if (K % 128 != 0 || N % 32 != 0) return NVFP4MOE_ESHAPE;
  // a tile's operand region is read through 32-bit offsets
  if (M_total >= 0x7FFFFF00LL || N > (1 << 20) || K > (1 << 22)) return NVFP4MOE_ESHAPE;
  if (!aligned(a_q, 16) || !aligned(b_q, 16) || !aligned(a_s, 4) || !aligned(b_s, 4) || !aligned(expert_offsets, 4))
    return NVFP4MOE_ESHAPE;
  p = Params{};
  p.a = a_q;
  p.b = b_q;
  p.as = a_s;
  p.bs = b_s;
  p.offsets = expert_offsets;
  p.M = M_total;
  p.N = N;
  p.K = K;
  p.E = E;
  return NVFP4MOE_OK;
}

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" int grouped_gemm_mxfp4(const uint8_t* a_q, const uint8_t* a_s, const uint8_t* b_q, const uint8_t* b_s,
                                  const int32_t* expert_offsets, int E, int64_t M_total, int64_t N, int64_t K, void* c,
                                  int c_dtype, nvfp4moe_stream_t stream) {
  Params p;
  if (c_dtype != NVFP4MOE_F32 && c_dtype != NVFP4MOE_BF16) return NVFP4MOE_EINVAL;
  if (M_total > 0 && N > 0 && !c) return NVFP4MOE_EINVAL;
  const int rc = check_operands(a_q, a_s, b_q, b_s, expert_offsets, E, M_total, N, K, p);
  if (rc != NVFP4MOE_OK) return rc;
  if (!aligned(c, 16)) return NVFP4MOE_ESHAPE;
  const int arch = check_arch();
  if (arch != NVFP4MOE_OK) return arch;
  if (M_total == 0 || N == 0) return NVFP4MOE_OK;
  p.c = c;
  hipStream_t st = as_stream(stream);
  return c_dtype == NVFP4MOE_F32 ? launch_epi<EPI_PLAIN, true>(p, st) : launch_epi<EPI_PLAIN, false>(p, st);
}

namespace {
int silu_gate_impl(const uint8_t* a_q, const uint8_t* a_s, const uint8_t* b_q, const uint8_t* b_s,
                   const int32_t* expert_offsets, int E, int64_t M_total, int64_t F, int64_t K, void* y1, void* h,
                   float* amax_out, uint8_t* q_h, uint8_t* s_h, uint8_t* q_y1, uint8_t* s_y1, nvfp4moe_stream_t stream) {
  Params p;
  if (F < 0 || F > 0x3FFFFFFFLL) return F < 0 ? NVFP4MOE_EINVAL : NVFP4MOE_ESHAPE;
  if ((q_h != nullptr) != (s_h != nullptr)) return NVFP4MOE_EINVAL;
  if (M_total > 0 && F > 0 && !h && !q_h) return NVFP4MOE_EINVAL;
  const int rc = check_operands(a_q, a_s, b_q, b_s, expert_offsets, E, M_total, 2 * F, K, p);
  if (rc != NVFP4MOE_OK) return rc;
  if (F % 128 != 0 || 2 * F * (K / 2) >= (1LL << 31)) return NVFP4MOE_ESHAPE;  // gate and up rows: one region
  if (!aligned(y1, 16) || !aligned(h, 16) || !aligned(q_h, 4) || !aligned(q_y1, 16) || !aligned(s_y1, 2) || !aligned(amax_out, 4))
    return NVFP4MOE_ESHAPE;
  const int arch = check_arch();
  if (arch != NVFP4MOE_OK) return arch;
  hipStream_t st = as_stream(stream);
  if (amax_out) fill_u32_kernel<<<1, 64, 0, st>>>(reinterpret_cast<uint32_t*>(amax_out), 0u, 1);
  if (M_total == 0 || F == 0) return launch_status();
  p.c = y1;
  p.h = h;
  p.amax = amax_out;
  p.hq = q_h;
  p.hs = s_h;
  p.yq = q_y1;
  p.ys = s_y1;
  if (q_y1) return launch_epi<EPI_SILU_C, false>(p, st);
  return q_h ? launch_epi<EPI_SILU_Q, false>(p, st) : launch_epi<EPI_SILU, false>(p, st);
}
}  // namespace

extern "C" int grouped_gemm_mxfp4_silu_gate(const uint8_t* a_q, const uint8_t* a_s, const uint8_t* b_q,
                                            const uint8_t* b_s, const int32_t* expert_offsets, int E, int64_t M_total,
                                            int64_t F, int64_t K, void* y1, void* h, float* amax_out, uint8_t* q_h,
                                            uint8_t* s_h, nvfp4moe_stream_t stream) {
  return silu_gate_impl(a_q, a_s, b_q, b_s, expert_offsets, E, M_total, F, K, y1, h, amax_out, q_h, s_h, nullptr, nullptr,
                        stream);
}

extern "C" int grouped_gemm_mxfp4_silu_gate_ckpt(const uint8_t* a_q, const uint8_t* a_s, const uint8_t* b_q,
                                                 const uint8_t* b_s, const int32_t* expert_offsets, int E,
                                                 int64_t M_total, int64_t F, int64_t K, void* y1, void* h,
                                                 float* amax_out, uint8_t* q_h, uint8_t* s_h, uint8_t* q_y1,
                                                 uint8_t* s_y1, nvfp4moe_stream_t stream) {
  if (M_total > 0 && F > 0 && (!q_y1 || !s_y1)) return NVFP4MOE_EINVAL;
  return silu_gate_impl(a_q, a_s, b_q, b_s, expert_offsets, E, M_total, F, K, y1, h, amax_out, q_h, s_h, q_y1, s_y1,
                        stream);
}
