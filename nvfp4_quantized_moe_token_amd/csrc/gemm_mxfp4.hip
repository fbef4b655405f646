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
// Data movement.  Codes and scales go HBM -> LDS by buffer loads that write
// LDS directly; rows past an expert's end or past N read as zeros.  A stage
// holds 256 reduction elements: 128 bytes of codes per row (one cache line),
// 16-byte units XOR-swizzled by row.  Scales travel 16 bytes a row, for two
// stages at once.  A ring of S stages runs S - 1 ahead of the computation,
// across the ends of tiles; one wait and one workgroup barrier per stage.
//
// Scheduling is that of the other grouped GEMMs: a persistent grid, each
// workgroup finds its tiles from the device offsets (up to 64 of them at a
// time), tiles in contiguous ranges per XCD with the row blocks of an expert
// next to each other.
//
// Epilogues.  The tile leaves through LDS in pieces of 64 bytes per row.  SiLU
// gate: tiles hold matching gate and up columns; Y1 is rounded to bf16 and
// H = silu(G) * U is taken from the rounded values, as the standalone kernel
// does; optionally H is quantized to MXFP4 on the way out.
//
// Bounds and measurements (us of the kernel; 128 experts, top-8).  A 256x256
// tile of 8 waves, 64x128 each, reads 0.75 KiB of LDS per MFMA; by the counters
// the LDS is then busy 81% as long as the MFMAs (gate+up of 8192 tokens; 107% in
// the skewed product, its epilogue included), writes of the loads not counted.
// 64x64 waves (128x256 and 256x128 tiles, or two workgroups per CU) read a third
// more and lose more than finer tiles save: gate+up of 8192 tokens 209 against
// 216 to 244.  Stages of 128 elements and a
// ring of four are no faster either (155 against 138 for a dense 4096 x 8192 x
// 8192 product, 4.0 PFLOP/s): lines are then read in halves.
//   gate+up, 8192 tokens (65536 rows, 768 features, K = 2048)      210
//   down, 16384 tokens, skewed routing (N = 2048, K = 768)         243
//   gate+up, 8192 tokens, H quantized and nothing else stored      181
//   the same with Y1 and H stored too (the learner's form)         235
//   the skewed product with fp32 output (266 of bytes)             328
//   gate+up, 512 tokens    51 (4.2 TB/s)     down, 512 tokens       30
//   N = 1536, K = 2048, 16 tokens, which reach 84 of the experts (140 MB)
//                                                     28 to 33 (4.3 to 4.9 TB/s)
// In copies without their stores the first two take 170 and 161, without any
// epilogue 129 and 117, where the MFMAs alone need 52 and 47: a workgroup's
// stores and SiLU are not hidden behind its products, since its accumulators
// fill the registers and its stages the LDS; the loop itself is held up by its
// LDS reads and by row padding (a fifth of gate+up's MFMAs).
#include "gemm_tiles.hpp"
#include "mx_codec.hpp"

namespace nvfp4moe {
namespace {

enum Epi { EPI_PLAIN = 0, EPI_SILU = 1, EPI_SILU_Q = 2 };

struct Params {
  const uint8_t* a;
  const uint8_t* b;
  const uint8_t* as;
  const uint8_t* bs;
  const int32_t* offsets;
  void* c;      // plain: C; SiLU: Y1 or NULL
  void* h;      // SiLU: H or NULL
  float* amax;  // SiLU: max |H| (cleared before the launch) or NULL
  uint8_t* hq;  // SiLU_Q: codes and scales of H
  uint8_t* hs;
  int64_t M, N, K;
  int E, n_tiles;
};

constexpr int kKS = 256;            // reduction elements per stage: 128 bytes of codes per row, one cache line
constexpr int kRowB = kKS / 2;      // code bytes per row
constexpr int kOffsetsInLds = 512;  // experts whose offsets are kept in LDS
constexpr int kTiles = 64;          // tiles looked up at a time
constexpr int kWaveOut = 1024;      // bytes of a wave's epilogue staging: 16 rows of 64 bytes

typedef __attribute__((address_space(3))) const i32x4_t lds_i32x4_t;
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) const u32x2_t lds_u32x2_t;

// A fragment: 16 bytes of codes (the instruction's operand has room for 32).
__device__ __forceinline__ i32x8_t frag(uint32_t at) {
  const i32x4_t v = *(lds_i32x4_t*)(uintptr_t)at;
  return (i32x8_t){v[0], v[1], v[2], v[3], 0, 0, 0, 0};
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
// A buffer region of less than 2^31 bytes: reads past it are zeros, writes are
// dropped.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t region(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, kRawBufferWord3);
}
// Four consecutive elements as bf16.
__device__ __forceinline__ uint2 bf16x4(const f32x16_t& a, int g) {
  const float x = element(a[4 * g]), y = element(a[4 * g + 1]), z = element(a[4 * g + 2]), w = element(a[4 * g + 3]);
  return make_uint2(pack_bf16x2(x, y), pack_bf16x2(z, w));
}

template <int BM, int BN, int WM, int WN, int S, int EPI, bool OUT32>
__global__ __launch_bounds__(WM* WN * 64, WM* WN / 4) void mxfp4_kernel(Params p) {
  constexpr int NW = WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 32, FN = WTN / 32;
  static_assert(FM >= 1 && FN >= 2 && WTM % 32 == 0 && WTN % 64 == 0, "wave tiling");
  constexpr bool SILU = EPI != EPI_PLAIN;
  constexpr int SA = BM < 64 ? 64 : BM;                    // scale rows of A (whole loads)
  constexpr int AT_B = BM * kRowB, STAGE = AT_B + BN * kRowB;  // codes of A, then B
  constexpr int SBUF = (SA + BN) * 16;                     // scales of two stages
  // 1 KiB loads of 8 code rows, and of 64 rows of scales, dealt to the waves in
  // turn; every wave issues NDMA per stage, whatever is left over landing in a
  // pad, so that its waits are constants.
  constexpr int A_LOADS = BM / 8, B_LOADS = BN / 8, SC_LOADS = (SA + BN) / 64;
  constexpr int A_INSTR = A_LOADS / NW, B_INSTR = B_LOADS / NW, SC_INSTR = (SC_LOADS + NW - 1) / NW;
  constexpr int NDMA = A_INSTR + B_INSTR + SC_INSTR, HALF = (NDMA + 1) / 2;
  static_assert(A_LOADS % NW == 0 && B_LOADS % NW == 0 && NW % 4 == 0, "the rows of a wave's loads agree modulo 32");
  constexpr int AHEAD = (S - 2) * NDMA;  // loads of this wave that are younger than the stage waited for
  static_assert(S >= 2 && AHEAD + 32 <= 63, "pipeline depth");

  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * (STAGE + SBUF) + NW * kWaveOut + 1024];
  __shared__ __attribute__((aligned(16))) int4 s_tile[2 * kTiles];  // this workgroup's tiles: expert, n-tile, first and end row
  __shared__ int32_t s_off[kOffsetsInLds + 1];                      // row offsets
  __shared__ int32_t s_blk[kOffsetsInLds + 1];                      // row blocks before each expert
  __shared__ int s_blocks;
  static_assert(sizeof(smem) + sizeof(s_tile) + sizeof(s_off) + sizeof(s_blk) + 64 <= 160 * 1024, "LDS");
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wid / WN, wn = wid % WN;
  const uint32_t smem_lds = (uint32_t)(uintptr_t)(const lds_void_t*)smem, scales = smem_lds + S * STAGE,
                 out = S * (STAGE + SBUF) + wid * kWaveOut, pad = smem_lds + S * (STAGE + SBUF) + NW * kWaveOut;
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
  // values.  The tiles of an expert are numbered n-tile-major (its row blocks
  // that share a weight panel are neighbours and run side by side on one XCD).
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
          t.x = e;
          t.y = (int)(in / cnt);
          t.z = lo + (int)(in % cnt) * BM;
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
  const uint32_t rowb = (uint32_t)(p.K / 2), srow = (uint32_t)(p.K / 32);
  const int lrow = wid * 8 + lane / 8, lunit = (lane & 7) ^ swz(lrow);
  const uint32_t la0 = (uint32_t)lrow * rowb + lunit * 16;
  const uint32_t lb0 = (uint32_t)(SILU ? gate_up_row(lrow, F, 0) : lrow) * rowb + lunit * 16;
  uint32_t ls0[SC_INSTR];
#pragma unroll
  for (int x = 0; x < SC_INSTR; ++x) {
    const int idx = wid + NW * x;
    const bool is_a = idx * 64 < SA;
    const int row = (is_a ? idx * 64 : idx * 64 - SA) + lane;
    const bool real = idx < SC_LOADS && (!is_a || row < BM);
    ls0[x] = real ? (uint32_t)(SILU && !is_a ? gate_up_row(row, F, 0) : row) * srow : kOOB;
  }
  const int nk = p.K > 0 ? (int)((p.K + kKS - 1) / kKS) : 1;  // (K == 0: one stage of zeros)
  // The last stage may hold 128 elements only: its upper units are not read
  // (zeros), and the scales of its upper chunks, which would be the next
  // row's, are taken as 0.
  const uint32_t beyond = p.K % kKS != 0 && lunit >= 4 ? kOOB : 0u;
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
      const bool is_a = (wid + NW * x) * 64 < SA;
      rsc[x] = is_a ? region(p.as + t.z * (int64_t)srow, mv * srow) : region(p.bs + brow * (int64_t)srow, nv * srow);
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
      dma16(rb, ld_on ? smem_lds + ld_slot + AT_B + (wid + NW * i) * 1024 : pad, lb + row * rowb);
    } else {
      const int i = x - A_INSTR - B_INSTR;
      const bool real = (SC_LOADS % NW == 0 || wid + NW * i < SC_LOADS) && ld_on && (ld_kt & 1) == 0;
      if (S == 2) {  // (no wait counts loads)
        if (real) dma16(rsc[i], scales + ld_sbuf + (wid + NW * i) * 1024, ls0[i] + (uint32_t)ld_kt * 8);
      } else {
        dma16(rsc[i], real ? scales + ld_sbuf + (wid + NW * i) * 1024 : pad, real ? ls0[i] + (uint32_t)ld_kt * 8 : kOOB);
      }
    }
  };
  auto advance = [&]() {
    ld_slot = ld_slot + STAGE == S * STAGE ? 0 : ld_slot + STAGE;
    if ((ld_kt & 1) || ld_kt + 1 == nk) ld_sbuf = ld_sbuf + SBUF == S * SBUF ? 0 : ld_sbuf + SBUF;
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

  i32x8_t fa[2][FM], fb[2][FN];
  u32x2_t wa[FM], wb[FN];  // scale words of the next stage as read
  int sa[FM], sb[FN];      // of the chunks in work
  auto read = [&](uint32_t slot, int c) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[c & 1][j] = frag(((fb0 + slot) ^ (32 * c)) + j * 32 * kRowB);
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[c & 1][i] = frag(((fa0 + slot) ^ (32 * c)) + i * 32 * kRowB);
  };
  auto read_scales = [&](uint32_t at) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < FN; ++j) wb[j] = *(lds_u32x2_t*)(uintptr_t)(sb0 + at + j * 512);
#pragma unroll
    for (int i = 0; i < FM; ++i) wa[i] = *(lds_u32x2_t*)(uintptr_t)(sa0 + at + i * 512);
  };
  // Bytes h and h + 2 of word w of a stage's two (h = lane / 32) to bytes 0 and
  // 2; none of them when bits is 0.
  auto take_scales = [&](int w, uint32_t bits) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = (int)__builtin_amdgcn_ubfe(wa[i][w], sh, bits);
#pragma unroll
    for (int j = 0; j < FN; ++j) sb[j] = (int)__builtin_amdgcn_ubfe(wb[j][w], sh, bits);
  };
  f32x16_t acc[FM][FN];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  };
  // MFMA x of FM * FN of chunk c: byte 0 or 2 of the scale words.  B first:
  // the result is the transposed tile.
  auto mfma = [&](int c, int x) __attribute__((always_inline)) {
    const int i = x / FN, j = x % FN;
    if (c & 1)
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
  uint32_t slot = 0, so = 0;  // ring slot and scale buffer (plus 8 for the second of two stages) of the stage in work
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
      take_scales(1, last && p.K % kKS != 0 ? 0 : 24);
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
      if ((kt & 1) || last) {
        so = (so & ~15u) + SBUF;
        if (so == S * SBUF) so = 0;
      } else {
        so += 8;
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
    // output row l % 32 and, for g = 0..3, the four consecutive columns
    // 8 g + 4 (l / 32) + 0..3 in registers 4g..4g+3.  Pieces of 16 rows and 64
    // bytes pass through a staging area of the wave's own, so that a store
    // writes 64 consecutive bytes of each row (which cost a CU what whole lines
    // do, 20 cycles a KiB; 32-byte pieces cost 32); the next tile's stages land
    // meanwhile.  LDS serves a wave in order: nothing is waited for between a
    // piece's writes and reads but the data, and a block is stored while the
    // next one passes.  Rows past the expert's end are past the store's region.
    settle();
    const int rq = lane & 15, hh = lane >> 5, half = (lane >> 4) & 1;  // this lane's row in its half
    uint8_t* reg = smem + out;
    const int pr = lane >> 2, pu = lane & 3;  // row and 16-byte unit of a piece on its way out
    uint8_t* put_at = reg + rq * 64 + 8 * hh;
    const uint8_t* get_at = reg + pr * 64 + ((pu ^ (pr >> 2)) << 4);
    auto put = [&](const uint2 (&w)[4], int part) __attribute__((always_inline)) {
      if (half == part) {
#pragma unroll
        for (int g = 0; g < 4; ++g) *reinterpret_cast<uint2*>(put_at + ((g ^ (rq >> 2)) << 4)) = w[g];
      }
    };
    auto get = [&]() __attribute__((always_inline)) {
      asm volatile("" ::: "memory");  // other lanes' writes
      const i32x4_t v = *reinterpret_cast<const i32x4_t*>(get_at);
      asm volatile("" ::: "memory");
      return v;
    };
    const uint32_t tile_rows = (uint32_t)(cur.w - cur.z);
    if constexpr (SILU) {
      const uint32_t yb = (uint32_t)p.N * 2, hb = (uint32_t)F * 2, qb = (uint32_t)F / 2, eb = (uint32_t)F / 32;
      uint16_t *Yp = reinterpret_cast<uint16_t*>(p.c), *Hp = reinterpret_cast<uint16_t*>(p.h);
      const __amdgpu_buffer_rsrc_t ry = region(Yp + m0 * p.N, tile_rows * yb), rh = region(Hp + m0 * F, tile_rows * hb);
      const __amdgpu_buffer_rsrc_t rq_ = region(p.hq + m0 * qb, tile_rows * qb), re = region(p.hs + m0 * eb, tile_rows * eb);
      const uint32_t vy = pr * yb + pu * 16, vh = pr * hb + pu * 16, vq = pr * qb + pu * 4, ve = pu == 0 ? pr * eb : kOOB;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int j = 0; j < FN; j += 2) {
          // Y1 is rounded to bf16 first: H is the gate of the stored values.
          uint2 gv[4], uv[4];
          i32x4_t o[2][3];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            gv[g] = bf16x4(acc[i][j], g);
            uv[g] = bf16x4(acc[i][j + 1], g);
          }
          if (Yp) {
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              put(gv, part);
              o[part][0] = get();
              put(uv, part);
              o[part][1] = get();
            }
          }
#pragma unroll
          for (int g = 0; g < 4; ++g)
            gv[g] = make_uint2(pack_bf16x2(silu_gate(bf16_lo(gv[g].x), bf16_lo(uv[g].x)),
                                           silu_gate(bf16_hi(gv[g].x), bf16_hi(uv[g].x))),
                               pack_bf16x2(silu_gate(bf16_lo(gv[g].y), bf16_lo(uv[g].y)),
                                           silu_gate(bf16_hi(gv[g].y), bf16_hi(uv[g].y))));
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            put(gv, part);
            o[part][2] = get();
          }
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const uint32_t row = wm * WTM + i * 32 + part * 16, f = (uint32_t)n0 / 2 + wn * (WTN / 2) + j * 16;
            if (Yp) {
              __builtin_amdgcn_raw_buffer_store_b128(o[part][0], ry, vy, row * yb + f * 2, 0);
              __builtin_amdgcn_raw_buffer_store_b128(o[part][1], ry, vy, row * yb + hb + f * 2, 0);
            }
            const i32x4_t h = o[part][2];
            if (Hp) __builtin_amdgcn_raw_buffer_store_b128(h, rh, vh, row * hb + f * 2, 0);
            if (EPI == EPI_SILU_Q || p.amax) {
              // (rows past the end hold 0 or NaN, which the maximum passes over)
              float hf[8], am = 0.0f;
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                hf[2 * w] = bf16_lo((uint32_t)h[w]);
                hf[2 * w + 1] = bf16_hi((uint32_t)h[w]);
                am = fmaxf(am, fmaxf(fabsf(hf[2 * w]), fabsf(hf[2 * w + 1])));
              }
              tile_amax = fmaxf(tile_amax, am);
              if constexpr (EPI == EPI_SILU_Q) {
                // four lanes hold the 32 features of one block of one row
                am = fmaxf(am, __shfl_xor(am, 1, 64));
                am = fmaxf(am, __shfl_xor(am, 2, 64));
                const int se = shared_exp<2>(am);
                __builtin_amdgcn_raw_buffer_store_b32(encode8_e2m1(hf, se), rq_, vq, row * qb + f / 2, 0);
                __builtin_amdgcn_raw_buffer_store_b8((uint8_t)(se + 127), re, ve, row * eb + f / 32, 0);
              }
            }
          }
          nst += 2 * ((Yp ? 2 : 0) + (Hp ? 1 : 0) + (EPI == EPI_SILU_Q ? 2 : 0));
          __builtin_amdgcn_sched_barrier(0);  // one block at a time: registers
        }
      }
    } else {
      constexpr uint32_t EB = OUT32 ? 4 : 2;  // bytes per element
      const uint32_t cb = (uint32_t)p.N * EB;
      const __amdgpu_buffer_rsrc_t rc = region(reinterpret_cast<uint8_t*>(p.c) + m0 * cb, tile_rows * cb);
      const uint32_t vc = pr * cb + pu * 16;
      i32x4_t v[2][OUT32 ? 2 : 1], before[2][OUT32 ? 2 : 1];
      auto store = [&](int x, const i32x4_t (&w)[2][OUT32 ? 2 : 1]) __attribute__((always_inline)) {  // block x
        const uint32_t row = wm * WTM + (x / FN) * 32, col = (uint32_t)n0 + wn * WTN + (x % FN) * 32;
        if (col < (uint32_t)p.N) {  // (N % 32 == 0)
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (uint32_t q = 0; q < EB / 2; ++q)
              __builtin_amdgcn_raw_buffer_store_b128(w[part][q], rc, vc, (row + part * 16) * cb + col * EB + q * 64, 0);
          nst += EB;
        }
      };
#pragma unroll
      for (int x = 0; x < FM * FN; ++x) {
        const f32x16_t& a = acc[x / FN][x % FN];
        if constexpr (OUT32) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {  // 16 columns at a time
            float4 w[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const int b = 8 * q + 4 * g;
              w[g] = make_float4(element(a[b]), element(a[b + 1]), element(a[b + 2]), element(a[b + 3]));
            }
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              if (half == part) {
#pragma unroll
                for (int g = 0; g < 2; ++g)
                  *reinterpret_cast<float4*>(reg + rq * 64 + (((2 * g + hh) ^ (rq >> 2)) << 4)) = w[g];
              }
              v[part][q] = get();
            }
          }
        } else {
          uint2 w[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) w[g] = bf16x4(a, g);
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            put(w, part);
            v[part][0] = get();
          }
        }
        if (x > 0) store(x - 1, before);
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (uint32_t q = 0; q < EB / 2; ++q) before[part][q] = v[part][q];
        __builtin_amdgcn_sched_barrier(0);  // one block at a time: registers
      }
      store(FM * FN - 1, before);
    }
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
template <int BM, int BN, int WM, int WN, int S, int EPI, bool OUT32>
int resident_per_cu() {
  static int cached = 0;
  if (cached > 0) return cached;
  int occ = 0;
  if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&occ, mxfp4_kernel<BM, BN, WM, WN, S, EPI, OUT32>, WM * WN * 64,
                                                   0) != hipSuccess ||
      occ < 1)
    occ = 1;
  cached = occ;
  return occ;
}

template <int BM, int BN, int WM, int WN, int S, int EPI, bool OUT32>
int launch_tiles(const Params& p0, hipStream_t st) {
  Params p = p0;
  p.n_tiles = (int)cdiv(p.N, BN);
  const int64_t upper = (cdiv(p.M, BM) + p.E) * p.n_tiles;  // tiles at most
  if (upper > 0x7FFFFFFFLL) return NVFP4MOE_ESHAPE;
  int64_t grid = (int64_t)device_cu_count() * resident_per_cu<BM, BN, WM, WN, S, EPI, OUT32>();
  if (grid > upper) grid = upper;
  grid = cdiv(grid, 8) * 8;  // whole XCD rounds
  mxfp4_kernel<BM, BN, WM, WN, S, EPI, OUT32><<<(unsigned)grid, WM * WN * 64, 0, st>>>(p);
  return launch_status();
}

// Tiles by the mean rows per expert (the host does not know more): with few
// rows the work is reading the weights, so the row block is small and the ring
// three stages deep; with many it is the MFMAs, the LDS reads that feed them
// and the stores.  The row block is one that most experts' rows fit in, up to
// 256, where blocks of 192 need two.  Measured kernel times in us, 128 experts,
// gate+up (768 features, K = 2048) and down (N = 2048, K = 768):
//   rows      gate+up, blocks of           down, blocks of
//             32     64    192    256      32     64    192    256
//    16     45.4   48.8          67.5
//    32     56.1   51.0          68.8    30.3   30.2          41.0
//    64     74.6   64.9   67.2   71.9    41.5   35.6   38.4   42.0
//    80            72.5   69.2   73.9           43.3   39.9   43.4
//    96     96.9   75.2   72.1   76.6    54.2   44.1   40.6   44.5
//   128    119.7   91.6   75.8   79.5    67.8   53.2   43.2   46.3
//   160                   79.9   85.5                  47.3   49.3
//   208                  118.7   96.1                  67.9   55.6
template <int EPI, bool OUT32>
int launch_epi(const Params& p, hipStream_t st) {
  if (p.M <= 24 * (int64_t)p.E) return launch_tiles<32, 256, 1, 4, 3, EPI, OUT32>(p, st);
  if (p.M <= 72 * (int64_t)p.E) return launch_tiles<64, 256, 1, 4, 3, EPI, OUT32>(p, st);
  if (p.M <= 176 * (int64_t)p.E) return launch_tiles<192, 256, 2, 4, 2, EPI, OUT32>(p, st);
  return launch_tiles<256, 256, 4, 2, 2, EPI, OUT32>(p, st);
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

extern "C" int grouped_gemm_mxfp4_silu_gate(const uint8_t* a_q, const uint8_t* a_s, const uint8_t* b_q,
                                            const uint8_t* b_s, const int32_t* expert_offsets, int E, int64_t M_total,
                                            int64_t F, int64_t K, void* y1, void* h, float* amax_out, uint8_t* q_h,
                                            uint8_t* s_h, nvfp4moe_stream_t stream) {
  Params p;
  if (F < 0 || F > 0x3FFFFFFFLL) return F < 0 ? NVFP4MOE_EINVAL : NVFP4MOE_ESHAPE;
  if ((q_h != nullptr) != (s_h != nullptr)) return NVFP4MOE_EINVAL;
  if (M_total > 0 && F > 0 && !h && !q_h) return NVFP4MOE_EINVAL;
  const int rc = check_operands(a_q, a_s, b_q, b_s, expert_offsets, E, M_total, 2 * F, K, p);
  if (rc != NVFP4MOE_OK) return rc;
  if (F % 128 != 0 || 2 * F * (K / 2) >= (1LL << 31)) return NVFP4MOE_ESHAPE;  // gate and up rows: one region
  if (!aligned(y1, 16) || !aligned(h, 16) || !aligned(q_h, 4) || !aligned(amax_out, 4)) return NVFP4MOE_ESHAPE;
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
  return q_h ? launch_epi<EPI_SILU_Q, false>(p, st) : launch_epi<EPI_SILU, false>(p, st);
}
