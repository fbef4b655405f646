// The grouped GEMM kernel of the operands that are kept as codes and go to the
// matrix instructions as they are stored: MXFP4 x MXFP4 (fp32 accumulation in
// the scaled MFMA, E8M0 scales per 32 along K) and 8-bit integers (exact int32
// accumulation, one fp32 scale per row of A and of B applied in the epilogue).
// gemm_mxfp4.hip and gemm_int8.hip instantiate it and hold their measurements.
//
// Data movement.  Codes and scales go HBM -> LDS by buffer loads that write
// LDS directly; rows past an expert's end or past N read as zeros.  A stage
// holds 128 bytes of codes per row (one cache line: 256 4-bit or 128 8-bit
// reduction elements), 16-byte units XOR-swizzled by row; a fragment of either
// format is one unit per lane.  MX scales travel 16 bytes a row, for two stages
// at once; the integers' scales once per tile, with its first stage.  A ring of
// S stages runs S - 1 ahead of the computation, across the ends of tiles; one
// wait and one workgroup barrier per stage.
//
// Scheduling is that of the other grouped GEMMs: a persistent grid, each
// workgroup finds its tiles from the device offsets (up to 64 of them at a
// time), tiles in contiguous ranges per XCD with the row blocks of an expert
// next to each other.
//
// Epilogues.  The tile leaves in pieces of 64 or 128 bytes per row, put together
// by exchanges between the lanes of a wave (through LDS the int8 gate+up with Y1
// in 8 bits took 14 us more).  SiLU gate: tiles hold matching gate and up columns;
// Y1 is rounded to bf16 and H = silu(G) * U is taken from the rounded values, as
// the standalone kernel does; optionally H is quantized to MXFP4 on the way out,
// or the rounded Y1 to MXINT8, the form in which the backward pass takes it back.
#pragma once

#include "gemm_tiles.hpp"
#include "mx_codec.hpp"

namespace nvfp4moe {
namespace {

enum Fmt { MXFP4, INT8 };
// SiLU gate: H (and Y1 if asked for); _Q: H in MXFP4 too; _C: Y1 in MXINT8 too,
// and H in MXFP4 if asked for (MXFP4 products).
enum Epi { EPI_PLAIN = 0, EPI_SILU = 1, EPI_SILU_Q = 2, EPI_SILU_C = 3 };

struct Params {
  const uint8_t* a;
  const uint8_t* b;
  const void* as;  // MXFP4: E8M0 bytes [rows][K / 32]; INT8: fp32 [rows]
  const void* bs;
  const int32_t* offsets;
  void* c;      // plain: C; SiLU: Y1 or NULL
  void* h;      // SiLU: H or NULL
  float* amax;  // SiLU: max |H| (cleared before the launch) or NULL
  uint8_t* hq;  // SiLU_Q, SiLU_C: codes and scales of H (SiLU_C: or NULL)
  uint8_t* hs;
  uint8_t* yq;  // SiLU_C: codes and scales of Y1
  uint8_t* ys;
  int64_t M, N, K;
  int E, n_tiles;
  bool stream;  // C or Y1 is stored past the caches
};

constexpr int kRowB = 128;          // code bytes per row and stage: one cache line
constexpr int kOffsetsInLds = 512;  // experts whose offsets are kept in LDS
constexpr int kTiles = 64;          // tiles looked up at a time
// C, or Y1, of so many bytes (352 MB) is stored non-temporally: the 256 MB cache
// behind the L2s would not hold it for whoever reads it next, and the operands stay
// there instead.  Measured (us, down of 16384 skewed tokens, 537 MB, other inputs each
// time): MXFP4 210 -> 199, fp32 output 289 -> 269, int8 306 -> 295 (of the same
// inputs, which the cache then holds, 207 -> 161 and 303 -> 266).  Layer forward, whose combine reads C
// next, MXFP4 and int8, cached and non-temporal: 8192 tokens (268 MB) 367, 370 and
// 553, 555; 10240 (336 MB) 434, 436 and 653, 649; 12288 (403 MB) 522, 513 and 778,
// 766; 16384 679, 658 and 1012, 993, with Y1 (403 MB) kept too 798, 768 and 1071,
// 1051.
constexpr int64_t kStreamBytes = 336LL << 20;
// Up to so many rows per expert in the mean most experts have one row block, so
// each of B's lines is read once: its loads are non-temporal and leave the caches
// to what is read again.  Measured (us, cached and non-temporal, gate+up with H
// alone (MXFP4: quantized) | down; several inputs in turn), rows per expert:
//             int8                        MXFP4
//      1   51.3  45.9 | 28.8  25.7     30.2  27.4 | 17.0  17.4
//     32   77.2  70.3 | 44.0  41.3     46.5  42.3 | 28.2  27.4
//    128  110.5 101.5 | 65.6  65.1     65.9  64.2 | 43.6  42.5
//    200  127.9 118.2 | 81.0  76.4     76.7  73.2 | 54.2  50.0
//    240  151.8 144.5 | 96.0  89.9     92.8  89.4 | 62.6  60.2
//    288  175.6 184.8 | 114  114      124.9 124.0 | 83.7  82.7
//    384  209   238   | 137  147      129.5 125.4 | 94.2  93.1
// (16384 skewed tokens, 1024 rows, the same inputs: 270, 314 | MXFP4 169, 220.)  Skewed
// routing of up to 256 rows in the mean: -6 to +2%.
// The rule does not ask for the weights' bytes: a model of several layers finds them
// in HBM whatever their size.  Products of 16, 64, 200 rows per expert (us, cached and
// non-temporal), several sets of weights in turn | the same ones again and again, which
// a cache may then hold (what a single small layer gives up):
//   int8   32 x 1536 x 2048, 101 MB  22.3 20.4  27.3 25.1  40.5 38.9 | 18.8 18.9  22.2 24.0  33.5 37.9
//          64 x 1536 x 2048, 201 MB  41.0 36.8  49.7 48.1  79.1 72.2 | 32.8 35.1  40.8 45.0  66.3 72.0
//          4 x 8192 x 8192, 268 MB   65.0 60.6  73.3 68.5 112.0 102  | 47.6 59.0  57.2 67.0  94.8 101
//   MXFP4  32 x 1536 x 2048, 50 MB   15.7 14.7  23.9 23.0  27.7 26.7 | 12.8 12.5  20.0 21.4  22.7 25.0
//          128 x 2048 x 768, 101 MB  26.0 24.3  35.5 34.5  56.2 53.8 | 22.5 22.6  32.0 37.1  44.4 53.1
//          4 x 8192 x 8192, 134 MB   43.1 40.0  45.2 43.4  69.7 65.7 | 26.8 38.3  31.2 41.5  51.0 64.7
// Layer forward of 512 tokens, MXFP4, 32 experts, top-4: 59.0 58.7 | 52.5 57.7; 128 experts, top-8
// (302 MB): 99.0 91.7 | 97.4 91.6.
constexpr int64_t kOnceRows = 240;

typedef __attribute__((address_space(3))) const i32x4_t lds_i32x4_t;
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) const u32x2_t lds_u32x2_t;

typedef int32_t i32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) const float lds_f32_t;
typedef __attribute__((address_space(3))) const f32x4_t lds_f32x4_t;

// A fragment: 16 bytes of codes (the scaled instruction's operand has room for
// 32), and an accumulator.
template <int FMT>
struct Operands {
  typedef i32x8_t Frag;
  typedef f32x16_t Acc;
};
template <>
struct Operands<INT8> {
  typedef i32x4_t Frag;
  typedef i32x16_t Acc;
};
template <int FMT>
__device__ __forceinline__ typename Operands<FMT>::Frag frag(uint32_t at) {
  const i32x4_t v = *(lds_i32x4_t*)(uintptr_t)at;
  if constexpr (FMT == MXFP4) return (i32x8_t){v[0], v[1], v[2], v[3], 0, 0, 0, 0};
  else return v;
}

// 16-byte unit u of code row r lies at unit u ^ swz(r).  The swizzle repeats
// every 32 rows, so a wave's fragments differ by constant offsets, and unit
// 2c + h of chunk c is one XOR away from unit h.
__device__ __forceinline__ int swz(int r) { return kswz(r & 31); }

// Accumulators stay in the accumulation registers until an element is used:
// left to itself the compiler moves whole blocks to vector registers at the
// end of the k-loop and spills.  settle() waits out the MFMA -> read latency,
// which the compiler does not see here; element() then reads one.
__device__ __forceinline__ void settle() { asm volatile("s_nop 15\n\ts_nop 15"); }
__device__ __forceinline__ float element(float a) {
  float v;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(a));
  return v;
}
// dma16 of lines that no other workgroup reads soon (non-temporal).
__device__ __forceinline__ void dma16_once(__amdgpu_buffer_rsrc_t r, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds" ::"s"(
                   __builtin_amdgcn_readfirstlane(lds)),
               "v"(voff), "s"(r)
               : "memory", "m0");
}
// A buffer region of less than 2^31 bytes: reads past it are zeros, writes are
// dropped.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t region(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, kRawBufferWord3);
}
// Four consecutive elements: the accumulator's, or for the integers the sums
// (each rounded to 24 bits) times the row's scale, then the columns'.
template <int FMT>
__device__ __forceinline__ f32x4_t elements(const typename Operands<FMT>::Acc& a, int g, float rs, f32x4_t cs) {
  f32x4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (FMT == MXFP4) {
      v[i] = element(a[4 * g + i]);
    } else {
      int32_t n;
      asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(n) : "a"(a[4 * g + i]));
      v[i] = (float)n * rs * cs[i];
    }
  }
  return v;
}
// The integers' sums reach from -127 * 128 K to 128 * 128 K: with the longest K a
// row and a column of -128 throughout give 2^31, one more than int32 holds, which
// arrives as the lowest number (no other sum is as low).  The number below it,
// 2^31 - 1, is 2^31 in fp32.
constexpr int64_t kLongestInt8 = 1 << 17;
__device__ __forceinline__ int32_t unwrapped(int32_t a) {
  int32_t v;
  asm volatile("v_accvgpr_read_b32 %1, %0\n\t"
               "v_cmp_eq_u32 vcc, %2, %1\n\t"
               "v_subbrev_co_u32 %1, vcc, 0, %1, vcc\n\t"
               "v_accvgpr_write_b32 %0, %1"
               : "+a"(a), "=&v"(v)
               : "s"(0x80000000u)
               : "vcc");
  return a;
}
__device__ __forceinline__ void bf16x4(f32x4_t v, uint32_t* w) {
  w[0] = pack_bf16x2(v[0], v[1]);
  w[1] = pack_bf16x2(v[2], v[3]);
}

// Exchanges between lanes.  swap_halves: a's upper half of the wave against b's
// lower one; swap_quarters: the same in each half, with quarters.
__device__ __forceinline__ void swap_halves(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap_quarters(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ uint32_t max_of_halves(uint32_t v) {
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(r[0], r[1]);
}
// Row of an operand block of 32 that its LDS row m holds (B's): the rows go in
// such an order that a lane's elements of a block's tile, MFMA columns 8 g +
// 4 (l / 32) + 0..3 for g = 0..3, are the columns 16 (l / 32) + 0..15.
__device__ __forceinline__ int column(int m) { return (m & ~31) | (m & 3) | ((m & 24) >> 1) | ((m & 4) << 2); }
// Exchange between neighbouring lanes (rows l and l ^ 1): afterwards a holds the
// even lane's row and b the odd one's, in each an even lane what was in its a, an
// odd lane what was in b.
// (Written out because the compiler keeps each move apart from its selection, twice
// the instructions.  The waits are those between a register's write and its read by
// another lane, before and behind.)
__device__ __forceinline__ void turn(uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {  // (a, b) and (c, d)
  uint32_t t, u;
  asm("s_mov_b32 vcc_lo, 0xAAAAAAAA\n\t"
      "s_mov_b32 vcc_hi, 0xAAAAAAAA\n\t"
      "v_cndmask_b32_dpp %0, %2, %4, vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %1, %3, %5, vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "s_not_b64 vcc, vcc\n\t"
      "v_cndmask_b32_dpp %2, %4, %2, vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "v_cndmask_b32_dpp %3, %5, %3, vcc quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf\n\t"
      "s_nop 1"
      : "=&v"(t), "=&v"(u), "+v"(a), "+v"(c)
      : "v"(b), "v"(d)
      : "vcc", "scc");
  b = t;
  d = u;
}
// A block's words, 32 bytes of a row per lane: afterwards words 0..3 are 16
// bytes of row l % 32 without its bit 0, unit 2 (l / 32) + l % 2 of 64 bytes, and
// words 4..7 those of the next row.
__device__ __forceinline__ void turn8(uint32_t (&w)[8]) {
#pragma unroll
  for (int k = 0; k < 4; k += 2) turn(w[k], w[k + 4], w[k + 1], w[k + 5]);
}
// A 16-byte store at one register offset.  With part of the offset in a scalar
// register the compiler takes the data registers as free at once and may write
// them in the next instruction; the store was then seen to take the new value of
// its third register (32 x 32 blocks of codes, in some lanes).
template <int HINT = 0>
__device__ __forceinline__ void store16(i32x4_t v, __amdgpu_buffer_rsrc_t r, uint32_t at) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, at, 0, HINT);
}
// Of two such quadruples side by side, a of 64 bytes of rows and b of the next 64:
// afterwards a holds row l % 16 without bit 0, unit 4 ((l / 16) % 2) + 2 (l / 32) +
// l % 2 of 128 bytes, and b the same of the row 16 further.
__device__ __forceinline__ void line(uint32_t* a, uint32_t* b) {
#pragma unroll
  for (int k = 0; k < 4; ++k) swap_quarters(a[k], b[k]);
}
__device__ __forceinline__ i32x4_t four(const uint32_t* w) { return (i32x4_t){(int)w[0], (int)w[1], (int)w[2], (int)w[3]}; }
// The quadruples of a and b to their places; as a stream (non-temporal) or not.
__device__ __forceinline__ void store_four(bool stream, __amdgpu_buffer_rsrc_t r, const uint32_t (&a)[8],
                                           const uint32_t (&b)[8], uint32_t a0, uint32_t b0, uint32_t a1, uint32_t b1) {
  if (stream) {
    store16<2>(four(a), r, a0);
    store16<2>(four(b), r, b0);
    store16<2>(four(a + 4), r, a1);
    store16<2>(four(b + 4), r, b1);
  } else {
    store16(four(a), r, a0);
    store16(four(b), r, b0);
    store16(four(a + 4), r, a1);
    store16(four(b + 4), r, b1);
  }
}

template <int FMT, int BM, int BN, int WM, int WN, int S, bool ONCE, int EPI, bool OUT32>
__global__ __launch_bounds__(WM* WN * 64, WM* WN / 4) void codes_kernel(Params p) {
  constexpr int NW = WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 32, FN = WTN / 32;
  static_assert(FM >= 1 && FN >= 2 && WTM % 32 == 0 && WTN % 64 == 0, "wave tiling");
  constexpr bool SILU = EPI != EPI_PLAIN;
  constexpr uint32_t GROUP = 8;
  // Scale rows of A (whole loads), and the scales' ring: of two stages' scales,
  // or of tiles'.  The loads run up to S tiles ahead of an epilogue.
  constexpr int SA = FMT == INT8 ? 256 : BM < 64 ? 64 : BM, SROW = FMT == INT8 ? 4 : 16;
  constexpr int AT_B = BM * kRowB, STAGE = AT_B + BN * kRowB;  // codes of A, then B
  constexpr int SBUF = (SA + BN) * SROW, SRING = (FMT == INT8 ? S + 1 : S) * SBUF;
  // 1 KiB loads of 8 code rows, and of 64 (MX) or 256 rows of scales, dealt to the waves in
  // turn; every wave issues NDMA per stage, whatever is left over landing in a
  // pad, so that its waits are constants.
  constexpr int A_LOADS = BM / 8, B_LOADS = BN / 8, SC_LOADS = (SA + BN) * SROW / 1024;
  constexpr int A_INSTR = A_LOADS / NW, B_INSTR = B_LOADS / NW, SC_INSTR = (SC_LOADS + NW - 1) / NW;
  constexpr int NDMA = A_INSTR + B_INSTR + SC_INSTR, HALF = (NDMA + 1) / 2;
  static_assert(A_LOADS % NW == 0 && B_LOADS % NW == 0 && NW % 4 == 0, "the rows of a wave's loads agree modulo 32");
  constexpr int AHEAD = (S - 2) * NDMA;  // loads of this wave that are younger than the stage waited for
  static_assert(S >= 2 && AHEAD + 32 <= 63, "pipeline depth");

  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * STAGE + SRING + 1024];
  __shared__ __attribute__((aligned(16))) int4 s_tile[2 * kTiles];  // this workgroup's tiles: expert, n-tile, first and end row
  __shared__ int32_t s_off[kOffsetsInLds + 1];                      // row offsets
  __shared__ int32_t s_blk[kOffsetsInLds + 1];                      // row blocks before each expert
  __shared__ int s_blocks;
  static_assert(sizeof(smem) + sizeof(s_tile) + sizeof(s_off) + sizeof(s_blk) + 64 <= 160 * 1024, "LDS");
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wid / WN, wn = wid % WN;
  const uint32_t smem_lds = (uint32_t)(uintptr_t)(const lds_void_t*)smem, scales = smem_lds + S * STAGE,
                 pad = scales + SRING;
  const bool off_in_lds = p.E <= kOffsetsInLds;
  lds_i32_t* off_lds = (lds_i32_t*)s_off;
  if (off_in_lds)
    for (int i = threadIdx.x; i <= p.E; i += NW * 64) s_off[i] = p.offsets[i];
  __syncthreads();
  if (wid == 0) {
    if (off_in_lds) {
      int base = 0;
      for (int e0 = 0; e0 < p.E; e0 += 64) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < p.E) expert_range(off_lds, e, p.M, lo, hi);
        int incl = (hi - lo + BM - 1) / BM;
        const int cnt = incl;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const int v = __shfl_up(incl, o, 64);
          if (lane >= o) incl += v;
        }
        if (e < p.E) s_blk[e] = base + incl - cnt;
        base += __shfl(incl, 63, 64);
      }
      if (lane == 0) {
        s_blk[p.E] = base;
        s_blocks = base;
      }
    } else {
      const int blocks = count_row_blocks<BM>(p.offsets, p.E, p.M);
      if (lane == 0) s_blocks = blocks;
    }
  }
  __syncthreads();
  const int64_t total = (int64_t)__builtin_amdgcn_readfirstlane(s_blocks) * p.n_tiles;
  const int xcd = blockIdx.x & 7;
  const int64_t t_step = gridDim.x >> 3, t_first = total * xcd / 8 + (blockIdx.x >> 3), t_end = total * (xcd + 1) / 8;
  const int my_tiles = t_first < t_end ? (int)((t_end - t_first + t_step - 1) / t_step) : 0;

  // Looks up this workgroup's tiles i0 .. i0 + 63, one per lane, into half
  // (i0 / 64) % 2 of s_tile.  Every wave does so for itself and writes the same
  // values.  The tiles of an expert go by groups of GROUP row blocks, n-tile-major
  // within a group: the 32 tiles that an XCD has in work at once are then at most
  // 8 by 4, 12 panels of operands in its L2 where whole columns of row blocks
  // would be 33.
  auto look_up = [&](int i0) {
    int4 t = make_int4(-1, 0, 0, 0);
    if (off_in_lds) {
      if (i0 + lane < my_tiles) {
        const uint32_t nt = (uint32_t)p.n_tiles, L = (uint32_t)(t_first + (i0 + lane) * t_step), slot = L / nt;
        int e = 0, hi_e = p.E;  // the last expert with no more than `slot` blocks before it
        while (hi_e - e > 1) {
          const int mid = (e + hi_e) >> 1;
          if ((uint32_t)s_blk[mid] <= slot) e = mid;
          else hi_e = mid;
        }
        int lo, hi;
        expert_range(off_lds, e, p.M, lo, hi);
        const uint32_t in = L - (uint32_t)s_blk[e] * nt, cnt = (uint32_t)(s_blk[e + 1] - s_blk[e]);
        if (in < cnt * nt) {  // (always, with ascending offsets)
          const uint32_t b0 = in / (GROUP * nt) * GROUP, r = in - b0 * nt, size = cnt - b0 < GROUP ? cnt - b0 : GROUP;
          t.x = e;
          t.y = (int)(r / size);
          t.z = lo + (int)(b0 + r % size) * BM;
          t.w = hi - t.z < BM ? hi : t.z + BM;
        }
      }
    } else {
      for (int i = 0; i < kTiles && i0 + i < my_tiles; ++i) {
        int e = -1, n = 0;
        int64_t r0 = 0, r1 = 0;
        const bool ok = find_tile<BM, true>(p.offsets, p.E, p.M, t_first + (i0 + i) * t_step, p.n_tiles, e, r0, r1, n);
        if (lane == i && ok) t = make_int4(e, n, (int)r0, (int)r1);
      }
    }
    s_tile[(i0 & kTiles) + lane] = t;
  };
  // Tile i of this workgroup, in scalar registers (expert -1: none).
  auto tile = [&](int i) {
    int4 t = make_int4(-1, 0, 0, 0);
    if (i < my_tiles) {
      t = s_tile[i & (2 * kTiles - 1)];
      t.x = __builtin_amdgcn_readfirstlane(t.x);
      t.y = __builtin_amdgcn_readfirstlane(t.y);
      t.z = __builtin_amdgcn_readfirstlane(t.z);
      t.w = __builtin_amdgcn_readfirstlane(t.w);
    }
    return t;
  };

  // Loads.  A lane's byte offsets of its first loads of a tile; load i adds
  // 8 NW i rows (gate and up granules of 32 rows alternate, and 8 NW is a
  // multiple of 32).  Scales are read 16 bytes a row, for two stages at once:
  // every row is a cache line of its own, and a load of 64 lines takes the
  // address unit 64 to 110 cycles however short they are (measured; a 1 KiB
  // load of whole lines takes 16).
  const int64_t F = p.N / 2;
  const uint32_t rowb = (uint32_t)(FMT == INT8 ? p.K : p.K / 2), srow = FMT == INT8 ? 4u : (uint32_t)(p.K / 32);
  const int lrow = wid * 8 + lane / 8, lunit = (lane & 7) ^ swz(lrow);
  const uint32_t la0 = (uint32_t)lrow * rowb + lunit * 16;
  const uint32_t lb0 = (uint32_t)(SILU ? gate_up_row(column(lrow), F, 0) : column(lrow)) * rowb + lunit * 16;
  uint32_t ls0[SC_INSTR];
#pragma unroll
  for (int x = 0; x < SC_INSTR; ++x) {
    const int idx = wid + NW * x;
    constexpr int ROWS = 1024 / SROW;  // rows a load; 16 bytes a lane
    const bool is_a = idx * ROWS < SA;
    const int row = (is_a ? idx * ROWS : idx * ROWS - SA) + lane * (16 / SROW);
    const bool real = idx < SC_LOADS && (!is_a || row < BM);
    ls0[x] = real ? (uint32_t)(is_a ? row : SILU ? gate_up_row(column(row), F, 0) : column(row)) * srow : kOOB;
  }
  constexpr int KS = FMT == INT8 ? kRowB : 2 * kRowB;       // reduction elements per stage
  const int nk = p.K > 0 ? (int)((p.K + KS - 1) / KS) : 1;  // (K == 0: one stage of zeros)
  // The last stage may be short (MXFP4: by half): units past the row are not
  // read (zeros), and the MX scales of its upper chunks, which would be the
  // next row's, are taken as 0.
  const uint32_t beyond = p.K % KS != 0 && (FMT == INT8 ? lunit * 16 >= p.K % KS : lunit >= 4) ? kOOB : 0u;
  // The load cursor: stage ld_kt of tile ld_i, always S - 1 stages ahead of the
  // computation.  Behind the last tile its regions are empty and its loads go
  // to the pad.
  int ld_i = 0, ld_kt = 0;
  uint32_t ld_slot = 0, ld_sbuf = 0, la = 0, lb = 0;
  bool ld_on = true;
  __amdgpu_buffer_rsrc_t ra, rb, rsc[SC_INSTR];
  auto regions = [&]() {
    const int4 t = tile(ld_i);
    ld_on = t.x >= 0;
    const int64_t n0 = (int64_t)t.y * BN, brow = ld_on ? (int64_t)t.x * p.N + (SILU ? n0 / 2 : n0) : 0;
    const uint32_t left = (uint32_t)p.N - (uint32_t)n0 / (SILU ? 2 : 1);
    const uint32_t nv = !ld_on ? 0u : SILU || left < BN ? left : BN, mv = (uint32_t)(t.w - t.z);
    ra = region(p.a + t.z * (int64_t)rowb, mv * rowb);
    rb = region(p.b + brow * (int64_t)rowb, nv * rowb);
#pragma unroll
    for (int x = 0; x < SC_INSTR; ++x) {
      const bool is_a = (wid + NW * x) * (1024 / SROW) < SA;
      const uint8_t *as = reinterpret_cast<const uint8_t*>(p.as), *bs = reinterpret_cast<const uint8_t*>(p.bs);
      rsc[x] = is_a ? region(as + t.z * (int64_t)srow, mv * srow) : region(bs + brow * (int64_t)srow, nv * srow);
    }
  };
  auto offsets = [&]() {
    const bool last = ld_kt + 1 == nk;
    la = (la0 + (uint32_t)ld_kt * kRowB) | (last ? beyond : 0u);
    lb = (lb0 + (uint32_t)ld_kt * kRowB) | (last ? beyond : 0u);
  };
  auto dma = [&](int x) __attribute__((always_inline)) {  // load x of NDMA of the cursor's stage
    if (x < A_INSTR) {
      dma16(ra, ld_on ? smem_lds + ld_slot + (wid + NW * x) * 1024 : pad, la + (uint32_t)(8 * NW * x) * rowb);
    } else if (x < A_INSTR + B_INSTR) {
      const int i = x - A_INSTR;
      const uint32_t row = (uint32_t)(SILU ? gate_up_row(8 * NW * i, F, 0) : 8 * NW * i);
      const uint32_t to = ld_on ? smem_lds + ld_slot + AT_B + (wid + NW * i) * 1024 : pad;
      if constexpr (ONCE) dma16_once(rb, to, lb + row * rowb);
      else dma16(rb, to, lb + row * rowb);
    } else {
      const int i = x - A_INSTR - B_INSTR;
      const bool real = (SC_LOADS % NW == 0 || wid + NW * i < SC_LOADS) && ld_on && (FMT == INT8 ? ld_kt == 0 : (ld_kt & 1) == 0);
      const uint32_t at = ls0[i] + (FMT == INT8 ? 0u : (uint32_t)ld_kt * 8);
      if (S == 2) {  // (no wait counts loads)
        if (real) dma16(rsc[i], scales + ld_sbuf + (wid + NW * i) * 1024, at);
      } else {
        dma16(rsc[i], real ? scales + ld_sbuf + (wid + NW * i) * 1024 : pad, real ? at : kOOB);
      }
    }
  };
  auto advance = [&]() {
    ld_slot = ld_slot + STAGE == S * STAGE ? 0 : ld_slot + STAGE;
    if ((FMT == MXFP4 && (ld_kt & 1)) || ld_kt + 1 == nk) ld_sbuf = ld_sbuf + SBUF == SRING ? 0 : ld_sbuf + SBUF;
    if (++ld_kt == nk) {
      ld_kt = 0;
      ++ld_i;
      if ((ld_i & (kTiles - 1)) == 0) look_up(ld_i);
      regions();
    }
    offsets();
  };

  // This lane's fragment addresses in slot 0: row lane % 32 of the wave's
  // first row block, unit lane / 32; and its first scale words.
  const uint32_t unit0 = (lane & 31) * kRowB + (((lane >> 5) ^ swz(lane & 31)) << 4);
  const uint32_t fa0 = smem_lds + wm * WTM * kRowB + unit0, fb0 = smem_lds + AT_B + wn * WTN * kRowB + unit0;
  const uint32_t sa0 = scales + (wm * WTM + (lane & 31)) * 16, sb0 = scales + (SA + wn * WTN + (lane & 31)) * 16;
  const int sh = 8 * (lane >> 5);

  typename Operands<FMT>::Frag fa[2][FM], fb[2][FN];
  u32x2_t wa[FM], wb[FN];  // scale words of the next stage as read
  int sa[FM], sb[FN];      // of the chunks in work
  auto read = [&](uint32_t slot, int c) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[c & 1][j] = frag<FMT>(((fb0 + slot) ^ (32 * c)) + j * 32 * kRowB);
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[c & 1][i] = frag<FMT>(((fa0 + slot) ^ (32 * c)) + i * 32 * kRowB);
  };
  auto read_scales = [&](uint32_t at) __attribute__((always_inline)) {
    if constexpr (FMT == INT8) return;
#pragma unroll
    for (int j = 0; j < FN; ++j) wb[j] = *(lds_u32x2_t*)(uintptr_t)(sb0 + at + j * 512);
#pragma unroll
    for (int i = 0; i < FM; ++i) wa[i] = *(lds_u32x2_t*)(uintptr_t)(sa0 + at + i * 512);
  };
  // Bytes h and h + 2 of word w of a stage's two (h = lane / 32) to bytes 0 and
  // 2; none of them when bits is 0.
  auto take_scales = [&](int w, uint32_t bits) __attribute__((always_inline)) {
    if constexpr (FMT == INT8) return;
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = (int)__builtin_amdgcn_ubfe(wa[i][w], sh, bits);
#pragma unroll
    for (int j = 0; j < FN; ++j) sb[j] = (int)__builtin_amdgcn_ubfe(wb[j][w], sh, bits);
  };
  typename Operands<FMT>::Acc acc[FM][FN];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  };
  // MFMA x of FM * FN of chunk c: byte 0 or 2 of the scale words.  B first:
  // the result is the transposed tile.
  auto mfma = [&](int c, int x) __attribute__((always_inline)) {
    const int i = x / FN, j = x % FN;
    if constexpr (FMT == INT8)
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[c & 1][j], fa[c & 1][i], acc[i][j], 0, 0, 0);
    else if (c & 1)
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[1][j], fa[1][i], acc[i][j], 4, 4, 2, sb[j], 2, sa[i]);
    else
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[0][j], fa[0][i], acc[i][j], 4, 4, 0, sb[j], 0, sa[i]);
  };
  // Keeps MFMAs x and x + 1 where they are written (they would be sunk behind
  // the branches that follow).
  auto pin = [&](int x) __attribute__((always_inline)) {
    asm volatile("" : "+a"(acc[x / FN][x % FN]), "+a"(acc[(x + 1) / FN][(x + 1) % FN]));
  };
  // Chunk c's MFMAs with loads x0 .. x1 - 1 spread among them (all waves'
  // loads at once would keep the address unit busy longer than the chunk).
  auto chunk = [&](int c, int x0, int x1, bool issue) __attribute__((always_inline)) {
    constexpr int G = FM * FN / 2;  // pairs of MFMAs
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      mfma(c, 2 * g);
      mfma(c, 2 * g + 1);
      pin(2 * g);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int x = x0; x < x1; ++x)
        if ((x - x0) * G / (x1 - x0) == g && issue) dma(x);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  float tile_amax = 0.0f;
  if (my_tiles > 0) {
    look_up(0);
    regions();
    offsets();
#pragma unroll 1
    for (int s = 0; s < S - 1; ++s) {
#pragma unroll
      for (int x = 0; x < NDMA; ++x) dma(x);
      advance();
    }
#pragma unroll
    for (int x = 0; x < HALF; ++x) dma(x);
    wait_vmcnt<AHEAD + HALF>();
    lds_barrier();
    read(0, 0);
    read_scales(0);
  }
  // Ring slot and scale buffer (MX: plus 8 for the second of two stages; the
  // integers': of the tile) of the stage in work.
  uint32_t slot = 0, so = 0;
  int fresh = 0, nst = 0;     // stages whose wait must allow for the last epilogue's nst stores
  bool rest = true;           // the cursor's stage has loads left to issue
#pragma unroll 1
  for (int it = 0; it < my_tiles; ++it) {
    const int4 cur = tile(it);
    const int64_t m0 = cur.z, m_end = cur.w, n0 = (int64_t)cur.y * BN;
    clear();
#pragma unroll 1
    for (int kt = 0; kt < nk; ++kt) {
      const bool last = kt + 1 == nk;
      // Each chunk's fragments are read under the MFMAs of the one before.
      take_scales(0, 24);
      read(slot, 1);
      chunk(0, HALF, NDMA, rest);
      if (rest) advance();
      rest = true;
      read(slot, 2);
      chunk(1, 0, 0, false);
      take_scales(1, last && p.K % KS != 0 ? 0 : 24);
      read(slot, 3);
      chunk(2, 0, 0, false);
      // The last chunk's fragments are in registers, so the slot is free once
      // every wave is here; the next stage has landed.  Stores of an epilogue
      // are younger than the loads of the S stages after it and need not have
      // finished.
      if (fresh == 0) {
        wait_vmcnt<AHEAD>();
      } else {
        --fresh;
        if (nst >= 32) wait_vmcnt<AHEAD + 32>();
        else if (nst >= 16) wait_vmcnt<AHEAD + 16>();
        else wait_vmcnt<AHEAD>();
      }
      lds_barrier();
      slot = slot + STAGE == S * STAGE ? 0 : slot + STAGE;
      if constexpr (FMT == MXFP4) {
        if ((kt & 1) || last) {
          so = (so & ~15u) + SBUF;
          if (so == SRING) so = 0;
        } else {
          so += 8;
        }
      }
      read(slot, 0);
      read_scales(so);
      chunk(3, 0, HALF, true);
    }
    // The rest of the cursor's stage goes before the epilogue's stores.
#pragma unroll
    for (int x = HALF; x < NDMA; ++x) dma(x);
    advance();
    rest = false;
    fresh = S - 1;
    nst = 0;

    // Epilogue.  The B fragment is the MFMA's first operand, so lane l holds
    // output row l % 32 and, by the order of B's rows in LDS, 16 consecutive
    // columns of each block.  Neighbouring lanes exchange registers until a store
    // writes 64 bytes of 16 rows, pairs of units in pairs of lanes: with units in
    // higher lane bits alone a quad of lanes touches four rows, and a CU's stores
    // to the L2 take half as long again (31 against 20 us for eight 128 KiB tiles on
    // every CU; to HBM 38.5 against 37).  Where nothing but C leaves, quarters of
    // the wave exchange too and a store writes whole lines (skewed product 212
    // against 224 us).  Rows past the expert's end are past the store's region.
    settle();
    if constexpr (FMT == INT8) {
      if (p.K == kLongestInt8) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = unwrapped(acc[i][j][r]);
      }
    }
    int ln = lane;
    asm volatile("" : "+v"(ln));  // (what follows from it is not kept from tile to tile: registers)
    const int hh = ln >> 5;
    const int r2 = ln & 30, u4 = 2 * hh + (ln & 1);         // row and 16-byte unit after turn8()
    const int r4 = ln & 14, u8 = ((ln >> 4) & 1) * 4 + u4;  // and after line()
    const uint32_t tile_rows = (uint32_t)(cur.w - cur.z);
    // The integers' scales of this lane's row of row block i, and of its columns
    // 16 hh + 4 g + 0..3 of column block j (rows 8 g + 4 hh + 0..3 of B in LDS).
    auto row_scale = [&](int i) __attribute__((always_inline)) {
      if constexpr (FMT == INT8) return *(lds_f32_t*)(uintptr_t)(scales + so + (wm * WTM + i * 32 + (ln & 31)) * 4);
      else return 0.0f;
    };
    auto col_scales = [&](int j, int g) __attribute__((always_inline)) {
      if constexpr (FMT == INT8)
        return *(lds_f32x4_t*)(uintptr_t)(scales + so + (SA + wn * WTN + j * 32 + 8 * g + 4 * hh) * 4);
      else return (f32x4_t){0, 0, 0, 0};
    };
    if constexpr (SILU) {
      const uint32_t yb = (uint32_t)p.N * 2, hb = (uint32_t)F * 2, qb = (uint32_t)F / 2, eb = (uint32_t)F / 32;
      uint16_t *Yp = reinterpret_cast<uint16_t*>(p.c), *Hp = reinterpret_cast<uint16_t*>(p.h);
      const __amdgpu_buffer_rsrc_t ry = region(Yp + m0 * p.N, tile_rows * yb), rh = region(Hp + m0 * F, tile_rows * hb);
      const __amdgpu_buffer_rsrc_t rq = region(p.hq + m0 * qb, tile_rows * qb), re = region(p.hs + m0 * eb, tile_rows * eb);
      const uint32_t kqb = (uint32_t)p.N, keb = (uint32_t)p.N / 32;  // row bytes of Y1's codes and scales
      const __amdgpu_buffer_rsrc_t rkq = region(p.yq + m0 * kqb, tile_rows * kqb), rke = region(p.ys + m0 * keb, tile_rows * keb);
      constexpr int P = FN >= 4 ? 2 : 1;  // pairs of a gate and an up block that leave together
      const uint32_t lr = ln & 31;      // codes and scales of one pair leave with a row per two lanes
      const uint32_t vq = lr * qb + hh * (P == 2 ? 16 : 8), ve = P == 2 ? lr * eb + hh : hh == 0 ? lr * eb : kOOB;
      const uint32_t vkq = P == 2 ? r2 * kqb + ((ln & 1) * 2 + hh) * 16 : lr * kqb + hh * 16, vke = lr * keb + hh * ((uint32_t)F / 32);
      const bool want_q = EPI == EPI_SILU_Q || (EPI == EPI_SILU_C && FMT == MXFP4 && p.hq);
      // Stores P blocks of 32 columns (paired up) at `at` of the region's rows.
      auto leave = [&](bool stream, uint32_t (&w)[P][8], __amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t rb) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < P; ++q) turn8(w[q]);
        at += r2 * rb + u4 * 16;
        if constexpr (P == 2) {
          store_four(stream, r, w[0], w[1], at, at + 64, at + rb, at + rb + 64);
        } else {
          store16(four(w[0]), r, at);
          store16(four(w[0] + 4), r, at + rb);
        }
      };
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const float rs = row_scale(i);
#pragma unroll
        for (int j = 0; j < FN; j += 2 * P) {
          // Y1 is rounded to bf16 first: H is the gate of the stored values.
          uint32_t gv[P][8], uv[P][8], hv[P][8];  // columns 16 hh + 4 g + 0..3 in words 2 g and 2 g + 1
#pragma unroll
          for (int q = 0; q < P; ++q) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              bf16x4(elements<FMT>(acc[i][j + 2 * q], g, rs, col_scales(j + 2 * q, g)), gv[q] + 2 * g);
              bf16x4(elements<FMT>(acc[i][j + 2 * q + 1], g, rs, col_scales(j + 2 * q + 1, g)), uv[q] + 2 * g);
            }
          }
          const uint32_t row = wm * WTM + i * 32, f = (uint32_t)n0 / 2 + wn * (WTN / 2) + j * 16;
          // The words are unpacked anew by each step that reads them (their halves
          // kept as floats from one to the next would spill).
          auto anew = [&](uint32_t (&y)[P][8]) __attribute__((always_inline)) {
#pragma unroll
            for (int q = 0; q < P; ++q)
#pragma unroll
              for (int w = 0; w < 8; ++w) asm volatile("" : "+v"(y[q][w]));
          };
          if constexpr (EPI == EPI_SILU_C) {
            uint32_t sc[2] = {0, 0};  // scale bytes of the P blocks, gate and up
#pragma unroll
            for (int t = 0; t < 2; ++t) {  // gate, up
              uint32_t d[P][4];
#pragma unroll
              for (int q = 0; q < P; ++q) {
                const uint32_t(&y)[8] = t ? uv[q] : gv[q];
                uint32_t am = 0;
#pragma unroll
                for (int w = 0; w < 8; ++w) am = max_abs_bf16x2(am, y[w]);
                am = max_of_halves(max_of_pair(am));
                const Int8Encoder e = int8_encoder(am);
                sc[t] |= (uint32_t)int8_scale(am) << (8 * q);
                anew(t ? uv : gv);
                // (the way that takes every block: a second one for tiny blocks
                // would spill)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                  const float v[4] = {bf16_lo(y[2 * g]), bf16_hi(y[2 * g]), bf16_lo(y[2 * g + 1]), bf16_hi(y[2 * g + 1])};
                  d[q][g] = encode4_int8<true>(v, e);
                }
              }
              if constexpr (P == 2) {  // 64 columns of every other row
#pragma unroll
                for (int k = 0; k < 4; k += 2) turn(d[0][k], d[1][k], d[0][k + 1], d[1][k + 1]);
              }
#pragma unroll
              for (int q = 0; q < P; ++q) store16(four(d[q]), rkq, vkq + (row + q) * kqb + t * (uint32_t)F + f);
              anew(t ? uv : gv);
              __builtin_amdgcn_sched_barrier(0);  // registers
            }
            const uint32_t s = hh ? sc[1] : sc[0];
            if constexpr (P == 2) __builtin_amdgcn_raw_buffer_store_b16((uint16_t)s, rke, vke, row * keb + f / 32, 0);
            else __builtin_amdgcn_raw_buffer_store_b8((uint8_t)s, rke, vke, row * keb + f / 32, 0);
          }
#pragma unroll
          for (int q = 0; q < P; ++q)
#pragma unroll
            for (int w = 0; w < 8; ++w)
              hv[q][w] = pack_bf16x2(silu_gate(bf16_lo(gv[q][w]), bf16_lo(uv[q][w])), silu_gate(bf16_hi(gv[q][w]), bf16_hi(uv[q][w])));
          if (Yp) {
#pragma unroll
            for (int t = 0; t < 2; ++t) leave(p.stream, t ? uv : gv, ry, row * yb + (t * (uint32_t)F + f) * 2, yb);
          }
          if (p.amax || want_q) {
            uint32_t d[P][2];
            int se[P];
#pragma unroll
            for (int q = 0; q < P; ++q) {
              // (rows past the end hold 0 or NaN, which the maximum passes over)
              float am = 0.0f;
#pragma unroll
              for (int w = 0; w < 8; ++w) am = fmaxf(am, fmaxf(fabsf(bf16_lo(hv[q][w])), fabsf(bf16_hi(hv[q][w]))));
              tile_amax = fmaxf(tile_amax, am);
              if (want_q) {
                // the two halves hold the 32 features of one block of one row
                se[q] = shared_exp<2>(__uint_as_float(max_of_halves(__float_as_uint(am))));
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                  float v[8];
#pragma unroll
                  for (int w = 0; w < 4; ++w) {
                    v[2 * w] = bf16_lo(hv[q][4 * t + w]);
                    v[2 * w + 1] = bf16_hi(hv[q][4 * t + w]);
                  }
                  d[q][t] = encode8_e2m1(v, se[q]);
                }
              }
            }
            if (want_q) {
              const uint32_t at = row * qb + f / 2, es = row * eb + f / 32;
              if constexpr (P == 2) {  // a block per half of the wave
                swap_halves(d[0][0], d[1][0]);
                swap_halves(d[0][1], d[1][1]);
                store16((i32x4_t){(int)d[0][0], (int)d[0][1], (int)d[1][0], (int)d[1][1]}, rq, vq + at);
                __builtin_amdgcn_raw_buffer_store_b8((uint8_t)((hh ? se[1] : se[0]) + 127), re, ve + es, 0, 0);
              } else {
                __builtin_amdgcn_raw_buffer_store_b64((u32x2_t){d[0][0], d[0][1]}, rq, vq, at, 0);
                __builtin_amdgcn_raw_buffer_store_b8((uint8_t)(se[0] + 127), re, ve, es, 0);
              }
            }
          }
          if (Hp) leave(false, hv, rh, row * hb + f * 2, hb);
          nst += P * ((Yp ? 4 : 0) + (Hp ? 2 : 0)) + (want_q ? 2 : 0) + (EPI == EPI_SILU_C ? 2 * P + 1 : 0);
          __builtin_amdgcn_sched_barrier(0);  // P pairs at a time: registers
        }
      }
    } else {
      constexpr uint32_t EB = OUT32 ? 4 : 2;  // bytes per element
      const uint32_t cb = (uint32_t)p.N * EB;
      const __amdgpu_buffer_rsrc_t rc = region(reinterpret_cast<uint8_t*>(p.c) + m0 * cb, tile_rows * cb);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const float rs = row_scale(i);
        const uint32_t row = wm * WTM + i * 32;
        if constexpr (OUT32) {
          // after line() lane bit 4 is unit bit 1 and lane / 32 unit bit 2
          const uint32_t vo = r4 * cb + (4 * hh + 2 * ((ln >> 4) & 1) + (ln & 1)) * 16;
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            const uint32_t col = (uint32_t)n0 + wn * WTN + j * 32;
            if (col >= (uint32_t)p.N) continue;  // (N % 32 == 0)
            uint32_t w[2][8];  // units 0 and 2, 1 and 3 of this lane's 64 bytes
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const f32x4_t e = elements<FMT>(acc[i][j], g, rs, col_scales(j, g));
#pragma unroll
              for (int k = 0; k < 4; ++k) w[g >> 1][(g & 1) * 4 + k] = __float_as_uint(e[k]);
            }
            // unit 4 h + g of 128 bytes: bit 0 to lane bit 0, bit 1 to lane bit 4
#pragma unroll
            for (int q = 0; q < 2; ++q) turn8(w[q]);
#pragma unroll
            for (int part = 0; part < 2; ++part) line(w[0] + 4 * part, w[1] + 4 * part);
            const uint32_t at = vo + row * cb + col * EB;
            store_four(p.stream, rc, w[0], w[1], at, at + 16 * cb, at + cb, at + 17 * cb);
            nst += 4;
            __builtin_amdgcn_sched_barrier(0);  // one block at a time: registers
          }
        } else {
          const uint32_t vc = r4 * cb + u8 * 16;
#pragma unroll
          for (int j = 0; j < FN; j += 2) {
            const uint32_t col = (uint32_t)n0 + wn * WTN + j * 32;
            if (col >= (uint32_t)p.N) continue;  // (N % 32 == 0)
            uint32_t w[2][8];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
              for (int g = 0; g < 4; ++g) bf16x4(elements<FMT>(acc[i][j + t], g, rs, col_scales(j + t, g)), w[t] + 2 * g);
              turn8(w[t]);
            }
            // (N may end between the two blocks: units 4..7 are then dropped)
            const uint32_t at = (u8 < 4 || col + 32 < (uint32_t)p.N ? vc : kOOB) + row * cb + col * EB;
#pragma unroll
            for (int part = 0; part < 2; ++part) line(w[0] + 4 * part, w[1] + 4 * part);
            store_four(p.stream, rc, w[0], w[1], at, at + 16 * cb, at + cb, at + 17 * cb);
            nst += 4;
            __builtin_amdgcn_sched_barrier(0);  // two blocks at a time: registers
          }
        }
      }
    }
    if constexpr (FMT == INT8) so = so + SBUF == SRING ? 0 : so + SBUF;
  }

  wait_vmcnt<0>();  // no load may land after the workgroup's LDS is given away
  if constexpr (SILU) {
    if (p.amax) {
      __shared__ float red[NW];
      const float m = wave_max(tile_amax);
      if (lane == 0) red[wid] = m;
      __syncthreads();
      if (threadIdx.x == 0) {
        float v = red[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) v = fmaxf(v, red[i]);
        atomicMax(reinterpret_cast<unsigned int*>(p.amax), __float_as_uint(v));
      }
    }
  }
}

// Resident workgroups per CU (the same on every gfx950 device).
template <int FMT, int BM, int BN, int WM, int WN, int S, bool ONCE, int EPI, bool OUT32>
int resident_per_cu() {
  static int cached = 0;
  if (cached > 0) return cached;
  int occ = 0;
  if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&occ, codes_kernel<FMT, BM, BN, WM, WN, S, ONCE, EPI, OUT32>, WM * WN * 64,
                                                   0) != hipSuccess ||
      occ < 1)
    occ = 1;
  cached = occ;
  return occ;
}

template <int FMT, int BM, int BN, int WM, int WN, int S, bool ONCE, int EPI, bool OUT32>
int launch_tiles(const Params& p0, hipStream_t st) {
  Params p = p0;
  p.n_tiles = (int)cdiv(p.N, BN);
  p.stream = p.M * p.N * (OUT32 ? 4 : 2) >= kStreamBytes;  // (SiLU: Y1)
  const int64_t upper = (cdiv(p.M, BM) + p.E) * p.n_tiles;  // tiles at most
  if (upper > 0x7FFFFFFFLL) return NVFP4MOE_ESHAPE;
  int64_t grid = (int64_t)device_cu_count() * resident_per_cu<FMT, BM, BN, WM, WN, S, ONCE, EPI, OUT32>();
  if (grid > upper) grid = upper;
  grid = cdiv(grid, 8) * 8;  // whole XCD rounds
  codes_kernel<FMT, BM, BN, WM, WN, S, ONCE, EPI, OUT32><<<(unsigned)grid, WM * WN * 64, 0, st>>>(p);
  return launch_status();
}

}  // namespace
}  // namespace nvfp4moe
