// Grouped W8A8 GEMM over the contiguous per-expert layout: 8-bit integers with
// one fp32 scale per row (token) of A and per row (output channel) of B_e,
//   C[r][n] = (float)(sum_k a[r][k] b[n][k]) * as[r] * bs[e][n],
// the sum exact in int32 (v_mfma_i32_32x32x32_i8; K <= 131072 keeps it below
// 2^31, but for one sum that is told apart), then three fp32 roundings: of the
// sum and of the two products.
// The 8-bit integer form of the experts' products stands beside the report's
// W4A8 and W4A4 ("miniTE報告、NVFP4強化学習の安定性を検証", third paragraph: the
// precisions compared; fourth: grouped GEMM, op fusion).
//
// The kernel and its epilogues are in gemm_codes.hpp.
//
// Bounds and measurements (us of the kernel, several sets of inputs in turn; 128
// experts, top-8).
//   gate+up, 8192 tokens (65536 rows, 768 features, K = 2048)      288 to 295 (1.4 PFLOP/s)
//   the same, H stored alone                                       263 to 272
//   the same, H and Y1 in 8 bits                                   297
//   down, 8192 tokens (N = 2048, K = 768)                          175
//   down, 16384 tokens, skewed routing                             293 to 298 (1.4 PFLOP/s)
//   the same, fp32 output                                          372 to 377
//   dense, 4096 x 8192 x 8192                                      228 (2.4 PFLOP/s)
//   N = 1536, K = 2048, 16 tokens, which reach 84 of the experts
//                                  (264 MB of weights)             40 to 41 (6.4 to 6.6 TB/s)
// The dense product is held by power: the clock falls to 1.7 GHz, where the MFMAs
// alone take 154 us, and LDS reads and loads add to the energy and so to the time
// (35 and 28 us when taken away singly); torch's integer product of 8192 x 8192 x
// 8192 reaches 2.5 PFLOP/s.  Gate+up: 224 without an epilogue, 185 without MFMAs
// (the operands' way from HBM: 128-byte pieces of 2 KiB rows, 614 MB at 3.3 TB/s
// by the L2's misses), 178 without loads, 150 with MFMAs and barriers alone (119
// of MFMAs, a quarter of them row padding: while they run, the fragments read and
// the stages written take all of the LDS's 128 bytes a cycle, 96 and 32); the
// epilogue's arithmetic (scales, SiLU, rounding: 20 each for SiLU and for the
// 8-bit codes) and stores come on top, as a workgroup fills a CU's registers and
// LDS.  Measured instead and not kept: four waves of 128x128 (dense 236, skewed
// 386); two workgroups per CU of 128x128 (309, 367) or of 128x256 with 64-byte
// stages (281, 369); rings of three and four 64-byte stages (no change); loads
// that bring lines of later stages to the L2 (20 more); leaving out waves without
// rows (no change); accumulators in vector registers (no change, 16 tokens 3 us
// slower); half of a tile's stores held in registers until the next tile's first
// stages (no change); staggered starts (no change).
#include "gemm_codes.hpp"

namespace nvfp4moe {
namespace {

// Tiles by the mean rows per expert (the host does not know more).  Up to 112 rows
// the work is reading the weights: small row blocks and a ring three stages deep.
// Then it is the MFMAs, the operands' way to LDS and the stores; blocks of 192
// where most experts' rows fit in one, or in two of them where they take two of
// 256 as well.  Measured kernel times in us (weights non-temporal up to 240 rows),
// 128 experts, random routing, three sets of inputs in turn, gate+up with H stored
// (768 features, K = 2048) and down (N = 2048, K = 768):
//   rows     gate+up, blocks of                   down, blocks of
//              32     64    128    192    256       32     64    128    192    256
//    16     65.7   67.9   70.9                   39.0   39.5   42.6
//    20     68.9   68.2   71.6                   41.0   40.4   43.4
//    24     75.1   69.1   72.2                   43.9   41.2   44.1
//    32     79.0   70.3   73.3                   46.1   41.8   44.5
//    40     88.6   71.5   75.8                   53.5   43.5   46.0
//    48     94.7   84.0   76.4                   55.2   49.3   46.7
//    64    122.5   93.5   78.8   90.8   99.8     64.5   55.6   48.4   57.5   62.3
//    96    155.0  105.4   85.3   96.1  104.9     80.5   62.1   52.0   60.4   65.3
//   112    151.3  115.7   98.0   96.2  104.5     87.9   69.2   60.5   61.6   68.0
//   128    173.1  134.0  115.7   98.1  105.5     98.2   75.0   66.9   63.2   68.1
//   144    182.6  150.2  131.3   99.4  109.4    108.8   86.4   82.6   63.6   69.8
//   152    190.5  155.1  132.5  101.3  108.8    114.2   86.6   84.1   65.4   70.5
//   160    200.1  153.5  129.4  107.6  107.3    118.6   89.6   83.1   68.0   70.4
//   200           171.6  127.6  149.5  115.3           106.9   82.5   93.0   75.7
//   256           196.2  163.0  169.2  166.9           127.2  100.9  110.3  106.6
//   272           202.6  179.3  170.8  188.1           131.5  107.8  110.3  121.6
//   288           208.4  183.7  172.5  190.9           135.7  114.3  110.9  125.4
//   320           229.2  189.5  177.2  195.3           149.0  117.0  115.1  126.8
//   352           245.2  197.3  197.4  200.6           163.2  127.8  130.2  129.0
//   384           262.2  219.1  221.6  201.8           178.7  139.8  141.5  134.3
//   512           343.9  277.6  256.5  261.9           244.7  180.2  172.6  175.7
//  1024           625.7  503.5  474.8  454.1           408.2  330.0  312.6  300.2
// The borders are those of an earlier table, without non-temporal accesses.  By this
// one they cost at most 5% but from 145 to 159 rows (blocks of 192: up to 9% less)
// and from 257 to 272 (blocks of 128 or 192: up to 12% less).
template <int EPI, bool OUT32>
int launch_epi(const Params& p, hipStream_t st) {
  const int64_t E = p.E, M = p.M;
  if (M <= 20 * E) return launch_tiles<INT8, 32, 256, 1, 4, 3, true, EPI, OUT32>(p, st);
  if (M <= 40 * E) return launch_tiles<INT8, 64, 256, 1, 4, 3, true, EPI, OUT32>(p, st);
  if (M <= 112 * E) return launch_tiles<INT8, 128, 256, 2, 4, 3, true, EPI, OUT32>(p, st);
  if (M <= 144 * E) return launch_tiles<INT8, 192, 256, 2, 4, 2, true, EPI, OUT32>(p, st);
  if (M <= kOnceRows * E) return launch_tiles<INT8, 256, 256, 4, 2, 2, true, EPI, OUT32>(p, st);
  if (M > 272 * E && M <= 352 * E) return launch_tiles<INT8, 192, 256, 2, 4, 2, false, EPI, OUT32>(p, st);
  return launch_tiles<INT8, 256, 256, 4, 2, 2, false, EPI, OUT32>(p, st);
}

// Argument checks shared by both entry points, then the launch parameters.
int check_operands(const int8_t* a_q, const float* a_s, const int8_t* b_q, const float* b_s,
                   const int32_t* expert_offsets, int E, int64_t M_total, int64_t N, int64_t K, Params& p) {
  if (E < 1 || M_total < 0 || N < 0 || K < 0) return NVFP4MOE_EINVAL;
  if (!expert_offsets) return NVFP4MOE_EINVAL;
  if (M_total > 0 && N > 0 && (!a_s || !b_s || (K > 0 && (!a_q || !b_q)))) return NVFP4MOE_EINVAL;
  if (K % 16 != 0 || N % 32 != 0) return NVFP4MOE_ESHAPE;
  // a tile's operand region is read through 32-bit offsets; the sums stay exact
  if (M_total >= 0x7FFFFF00LL || N > (1 << 20) || K > kLongestInt8) return NVFP4MOE_ESHAPE;
  if (!aligned(a_q, 16) || !aligned(b_q, 16) || !aligned(a_s, 4) || !aligned(b_s, 4) || !aligned(expert_offsets, 4))
    return NVFP4MOE_ESHAPE;
  p = Params{};
  p.a = reinterpret_cast<const uint8_t*>(a_q);
  p.b = reinterpret_cast<const uint8_t*>(b_q);
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

extern "C" int grouped_gemm_int8(const int8_t* a_q, const float* a_s, const int8_t* b_q, const float* b_s,
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

extern "C" int grouped_gemm_int8_silu_gate(const int8_t* a_q, const float* a_s, const int8_t* b_q, const float* b_s,
                                           const int32_t* expert_offsets, int E, int64_t M_total, int64_t F, int64_t K,
                                           void* y1, void* h, float* amax_out, uint8_t* q_y1, uint8_t* s_y1,
                                           nvfp4moe_stream_t stream) {
  Params p;
  if (F < 0 || F > 0x3FFFFFFFLL) return F < 0 ? NVFP4MOE_EINVAL : NVFP4MOE_ESHAPE;
  if ((q_y1 != nullptr) != (s_y1 != nullptr)) return NVFP4MOE_EINVAL;
  if (M_total > 0 && F > 0 && !h) return NVFP4MOE_EINVAL;
  const int rc = check_operands(a_q, a_s, b_q, b_s, expert_offsets, E, M_total, 2 * F, K, p);
  if (rc != NVFP4MOE_OK) return rc;
  if (F % 128 != 0 || 2 * F * K >= (1LL << 31)) return NVFP4MOE_ESHAPE;  // gate and up rows: one region
  if (!aligned(y1, 16) || !aligned(h, 16) || !aligned(q_y1, 16) || !aligned(s_y1, 2) || !aligned(amax_out, 4)) return NVFP4MOE_ESHAPE;
  const int arch = check_arch();
  if (arch != NVFP4MOE_OK) return arch;
  hipStream_t st = as_stream(stream);
  if (amax_out) fill_u32_kernel<<<1, 64, 0, st>>>(reinterpret_cast<uint32_t*>(amax_out), 0u, 1);
  if (M_total == 0 || F == 0) return launch_status();
  p.c = y1;
  p.h = h;
  p.amax = amax_out;
  p.yq = q_y1;
  p.ys = s_y1;
  return q_y1 ? launch_epi<EPI_SILU_C, false>(p, st) : launch_epi<EPI_SILU, false>(p, st);
}
