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
// blocks of 192 need two.  Measured kernel times in us (weights non-temporal up to
// 240 rows), 128 experts, random routing, three sets of inputs in turn, gate+up with
// Y1 and H stored (768 features, K = 2048) and down (N = 2048, K = 768):
//   rows     gate+up, blocks of            down, blocks of
//              32     64    192    256       32     64    192    256
//    16     44.2   46.2                   25.1   26.5
//    20     45.5   46.2                   26.3   26.9
//    24     50.2   47.0                   28.2   27.1
//    32     54.7   48.1                   29.9   27.7
//    48     62.9   57.4                   35.5   32.4
//    64     74.1   62.2   62.9   65.9     40.9   35.0   36.6   39.3
//    72     81.3   69.4   63.3   66.6     46.1   40.3   37.6   40.3
//    80     85.4   69.7   63.8   67.8     47.8   40.1   37.7   40.6
//    96     96.4   69.8   67.0   70.3     52.4   40.6   39.1   42.2
//   112    102.6   78.8   66.8   70.1     59.4   45.7   40.7   43.9
//   128    117.6   88.2   69.7   73.1     65.2   49.1   41.4   45.5
//   144    127.0   98.0   71.6   75.0     72.8   57.3   42.2   46.5
//   152    135.5   98.3   73.3   76.2     75.5   57.6   42.9   46.5
//   160    141.6  100.7   78.0   76.9     79.7   59.3   44.6   46.6
//   200           121.7  104.8   81.7            72.4   61.5   54.7
//   256           144.8  122.0  119.3            86.2   70.0   66.3
//   272           151.3  125.9  130.7            89.1   71.7   76.4
//   288           155.6  128.9  131.7            92.3   73.7   80.2
//   320           170.9  134.0  137.6           101.9   78.1   80.1
//   352           183.9  150.5  144.5           112.6   87.5   85.9
//   384           200.8  164.3  149.9           124.3   95.2   91.9
//   512           266.0  199.1  192.8           171.7  121.2  117.0
//  1024           477.8  372.9  333.3           290.1  224.5  205.9
// The borders are those of an earlier table, without non-temporal accesses.  By this
// one they cost at most 5% but at 21 to 24 rows (blocks of 64: up to 6% less), 65 to 72
// (192: 9%) and 257 to 320 (192: up to 8%).
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
