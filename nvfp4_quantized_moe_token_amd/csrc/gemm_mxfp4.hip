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
// 16-byte units XOR-swizzled by row, and the row's 8 scale bytes as two words
// in two planes (elements 0..127 and 128..255), so that a lane's word serves
// two MFMAs (the instruction selects the byte).  A ring of S stages keeps
// S - 1 in flight; one wait and one workgroup barrier per stage.
//
// Scheduling is that of the other grouped GEMMs: a persistent grid, each
// workgroup finds its tiles from the device offsets, tiles in contiguous
// ranges per XCD with the row blocks of an expert next to each other.
//
// Epilogues.  Plain: the tile leaves through LDS, so that every store writes
// whole lines.  SiLU gate: tiles hold matching gate and up columns; Y1 is
// rounded to bf16 and H = silu(G) * U is taken from the rounded values, as the
// standalone kernel does; optionally H is quantized to MXFP4 on the way out.
#include "gemm_tiles.hpp"
#include "mx_codec.hpp"

namespace nvfp4moe {
namespace {

constexpr int kKS = 256;  // reduction elements per stage

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

// Code rows are 128 bytes; 16-byte unit u of row r lies at unit u ^ swz(r).  The
// swizzle repeats every 32 rows, so a wave's fragments differ by constant
// offsets, and unit 2c + h of chunk c is one XOR away from unit h.
__device__ __forceinline__ int swz(int r) { return kswz(r & 31); }

typedef __attribute__((address_space(3))) const i32x4_t lds_i32x4_t;
typedef __attribute__((address_space(3))) const uint32_t lds_u32_t;
// 32 codes at an LDS byte address; the operand's upper four registers are not
// read for a 4-bit format.
__device__ __forceinline__ i32x8_t frag(uint32_t at) {
  const i32x4_t v = *(lds_i32x4_t*)(uintptr_t)at;
  return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}

template <int BM, int BN, int WM, int WN, int S, int EPI, bool OUT32>
__global__ __launch_bounds__(WM* WN * 64, WM* WN / 4) void mxfp4_kernel(Params p) {
  constexpr int NW = WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 32, FN = WTN / 32;
  static_assert(FM >= 1 && FN >= 1 && WTM % 32 == 0 && WTN % 32 == 0, "wave tiling");
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && BN % 64 == 0, "whole loads per wave");
  constexpr bool SILU = EPI != EPI_PLAIN;
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  constexpr int SA = BM < 64 ? 64 : BM;          // scale rows of A (whole 64-lane loads)
  constexpr int PLANE = (SA + BN) * 4;           // one scale word per row
  constexpr int AT_A = 2 * PLANE, AT_B = AT_A + A_BYTES, STAGE = AT_B + B_BYTES;  // scales, A, B
  static_assert(STAGE % 128 == 0 && AT_A % 128 == 0, "the chunk XOR stays inside a row");
  constexpr int A_INSTR = BM / (8 * NW), B_INSTR = BN / (8 * NW);
  constexpr int SC_BLK = (SA + BN) / 64, SC_LOADS = 2 * SC_BLK;  // loads of 64 words per stage
  constexpr int SC_INSTR = (SC_LOADS + NW - 1) / NW;             // per wave; the excess lands in a pad
  constexpr int NDMA = A_INSTR + B_INSTR + SC_INSTR;
  static_assert(S >= 2 && NDMA * (S - 2) <= 63, "pipeline depth");

  __shared__ __attribute__((aligned(1024))) uint8_t smem[S * STAGE + 256];
  __shared__ int64_t s_tile[5];  // expert, first row, end row, row-block count, n-tile
  constexpr int kOffLds = 1025;
  __shared__ int32_t s_off[kOffLds];
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wid / WN, wn = wid % WN;
  const uint32_t smem_lds = (uint32_t)(uintptr_t)(const lds_void_t*)smem;
  const bool off_in_lds = p.E < kOffLds;
  lds_i32_t* off_lds = (lds_i32_t*)s_off;
  if (off_in_lds)
    for (int i = threadIdx.x; i <= p.E; i += NW * 64) s_off[i] = p.offsets[i];
  if (wid == 0) {
    const int blocks = count_row_blocks<BM>(p.offsets, p.E, p.M);
    if (lane == 0) s_tile[3] = blocks;
  }
  __syncthreads();
  const int64_t total = s_tile[3] * p.n_tiles;
  const int xcd = blockIdx.x & 7;
  const int64_t t_end = total * (xcd + 1) / 8, t_step = gridDim.x >> 3;

  // A lane's byte offsets in the regions of a tile: the same for every tile;
  // a stage adds a fixed number of bytes per row.
  const int64_t rowb = p.K / 2, srow = p.K / 32, gate_f = SILU ? p.N / 2 : 0;
  uint32_t oa[A_INSTR], ob[B_INSTR], os[SC_INSTR];
  // every load of a wave has the same rows modulo 32, so its lane takes the
  // same 16-byte unit of each row
  static_assert((8 * NW) % 32 == 0, "rows of a wave's loads, modulo 32");
  const uint32_t unit16 = ((lane & 7) ^ swz(wid * 8 + lane / 8)) << 4;
#pragma unroll
  for (int i = 0; i < A_INSTR; ++i) {
    const int row = (wid + NW * i) * 8 + lane / 8;
    oa[i] = (uint32_t)(row * rowb) + unit16;
  }
#pragma unroll
  for (int i = 0; i < B_INSTR; ++i) {
    const int row = (wid + NW * i) * 8 + lane / 8;
    const int64_t grow = SILU ? gate_up_row(row, gate_f, 0) : row;
    ob[i] = (uint32_t)(grow * rowb) + unit16;
  }
#pragma unroll
  for (int i = 0; i < SC_INSTR; ++i) {
    const int idx = wid + NW * i, blk = idx % SC_BLK, plane = idx / SC_BLK;
    const bool is_a = blk * 64 < SA;
    const int row = (is_a ? blk * 64 : blk * 64 - SA) + lane;
    const bool real = idx < SC_LOADS && (!is_a || row < BM);
    const int64_t grow = SILU && !is_a ? gate_up_row(row, gate_f, 0) : row;
    os[i] = real ? (uint32_t)(grow * srow + plane * 4) : kOOB;
  }

  // This lane's fragment addresses in slot 0: row lane % 32 of the wave's
  // first row block, unit lane / 32; and its scale words in plane 0.
  const uint32_t unit0 = (lane & 31) * 128 + (((lane >> 5) ^ swz(lane)) << 4);
  const uint32_t fa0 = smem_lds + AT_A + wm * WTM * 128 + unit0, fb0 = smem_lds + AT_B + wn * WTN * 128 + unit0;
  const uint32_t sa0 = smem_lds + (wm * WTM + (lane & 31)) * 4, sb0 = smem_lds + (SA + wn * WTN + (lane & 31)) * 4;

  float tile_amax = 0.0f;
  for (int64_t L = total * xcd / 8 + (blockIdx.x >> 3); L < t_end; L += t_step) {
    lds_barrier();  // every wave is done with the previous tile's LDS and s_tile
    if (wid == 0) {
      int e = -1, nt = 0;
      int64_t r0 = 0, r1 = 0;
      const bool ok = off_in_lds ? find_tile<BM, true>(off_lds, p.E, p.M, L, p.n_tiles, e, r0, r1, nt)
                                 : find_tile<BM, true>(p.offsets, p.E, p.M, L, p.n_tiles, e, r0, r1, nt);
      if (lane == 0) {
        s_tile[0] = ok ? e : -1;
        s_tile[1] = r0;
        s_tile[2] = r1;
        s_tile[4] = nt;
      }
    }
    lds_barrier();
    const int expert = __builtin_amdgcn_readfirstlane((int)s_tile[0]);
    if (expert < 0) break;  // uniform: only when offsets changed under the kernel
    const int64_t m0 = uniform64(s_tile[1]), m_end = uniform64(s_tile[2]), n0 = uniform64(s_tile[4]) * BN;

    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.a + m0 * rowb, (m_end - m0) * rowb);
    const __amdgpu_buffer_rsrc_t rsa = make_rsrc(p.as + m0 * srow, (m_end - m0) * srow);
    const int64_t brow = (int64_t)expert * p.N + (SILU ? n0 / 2 : n0);
    const int64_t nv = SILU ? p.N - n0 / 2 : p.N - n0 < BN ? p.N - n0 : BN;
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.b + brow * rowb, nv * rowb);
    const __amdgpu_buffer_rsrc_t rsb = make_rsrc(p.bs + brow * srow, nv * srow);

    auto load_stage = [&](int64_t kt, int slot) {
      const uint32_t st = smem_lds + slot * STAGE;
      const uint32_t k0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)(kt * kKS));
      // K % 256 == 128: the second half of the last stage reads as zeros
      const uint32_t left = (uint32_t)p.K - k0;
      const bool in_k = unit16 * 2 < left;
#pragma unroll
      for (int i = 0; i < A_INSTR; ++i) dma16(ra, st + AT_A + (wid + NW * i) * 1024, in_k ? oa[i] + k0 / 2 : kOOB);
#pragma unroll
      for (int i = 0; i < B_INSTR; ++i) dma16(rb, st + AT_B + (wid + NW * i) * 1024, in_k ? ob[i] + k0 / 2 : kOOB);
#pragma unroll
      for (int i = 0; i < SC_INSTR; ++i) {
        const int idx = wid + NW * i, blk = idx % SC_BLK, plane = idx / SC_BLK;
        const uint32_t at = idx < SC_LOADS ? st + plane * PLANE + blk * 256
                                           : smem_lds + S * STAGE;
        dma4(blk * 64 < SA ? rsa : rsb, at, (uint32_t)plane * 128 < left ? os[i] + k0 / 32 : kOOB);
      }
    };

    f32x16_t acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

    const int64_t nk = (p.K + kKS - 1) / kKS;
    // A wave whose rows all lie past the expert's end skips its MFMAs (it
    // still loads and takes part in the barriers).
    const bool active = m_end - m0 > wm * WTM;
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
      if (s < nk) load_stage(s, s);

    for (int64_t kt = 0; kt < nk; ++kt) {
      const int64_t ahead = nk - 1 - kt < S - 2 ? nk - 1 - kt : S - 2;
      wait_steps_ahead<S - 2, NDMA>((int)ahead);
      lds_barrier();
      if (kt + S - 1 < nk) load_stage(kt + S - 1, (int)((kt + S - 1) % S));
      const uint32_t slot = (uint32_t)__builtin_amdgcn_readfirstlane((int)(kt % S)) * STAGE;

      if (active) {
        i32x8_t fa[2][FM], fb[2][FN];
        int sa[2][FM], sb[2][FN];  // by half of the stage
        auto read = [&](int c) {
#pragma unroll
          for (int i = 0; i < FM; ++i) fa[c & 1][i] = frag(((fa0 + slot) ^ (32 * c)) + i * 4096);
#pragma unroll
          for (int j = 0; j < FN; ++j) fb[c & 1][j] = frag(((fb0 + slot) ^ (32 * c)) + j * 4096);
          if ((c & 1) == 0) {
            // this half's scale words: byte 2 (c % 2) + h belongs to chunk c
            const int sh = 8 * (lane >> 5);
#pragma unroll
            for (int i = 0; i < FM; ++i)
              sa[c >> 1][i] = (int)(*(lds_u32_t*)(uintptr_t)(sa0 + slot + (c >> 1) * PLANE + i * 128) >> sh);
#pragma unroll
            for (int j = 0; j < FN; ++j)
              sb[c >> 1][j] = (int)(*(lds_u32_t*)(uintptr_t)(sb0 + slot + (c >> 1) * PLANE + j * 128) >> sh);
          }
        };
        read(0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2 * (FM + FN), 0);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          // of the waves sharing a SIMD the one behind in the stage issues first
          if (c == 0) __builtin_amdgcn_s_setprio(1);
          else if (c == 2) __builtin_amdgcn_s_setprio(0);
          if (c + 1 < 4) read(c + 1);
#pragma unroll
          for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) {
              // B first: the result is the transposed tile (see the epilogue)
              if (c & 1)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[1][j], fa[1][i], acc[i][j], 4, 4, 2,
                                                                            sb[c >> 1][j], 2, sa[c >> 1][i]);
              else
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[0][j], fa[0][i], acc[i][j], 4, 4, 0,
                                                                            sb[c >> 1][j], 0, sa[c >> 1][i]);
            }
          if (c + 1 < 4)
            interleave_mfma_ds<FM * FN, (FM + FN) * 2>();
          else
            interleave_mfma_ds<FM * FN, 0>();
        }
      }
    }

    // Epilogue.  The B fragment is the MFMA's first operand, so lane l holds
    // output row l % 32 and, for g = 0..3, the four consecutive columns
    // 8 g + 4 (l / 32) + 0..3 in registers 4g..4g+3.  Each wave passes its
    // 32-row blocks through a private LDS region (the ring is free).
    lds_barrier();
    const int q = lane & 31, hh = lane >> 5;
    if constexpr (SILU) {
      constexpr int FW = WTN / 2;      // features per wave
      constexpr int CH = FW / 8;       // 16-byte chunks per row and part
      constexpr int PART = 32 * FW * 2;
      static_assert(WTN % 64 == 0 && (CH & (CH - 1)) == 0 && NW * 2 * PART <= S * STAGE, "SiLU staging");
      uint16_t* Yp = reinterpret_cast<uint16_t*>(p.c);
      uint16_t* Hp = reinterpret_cast<uint16_t*>(p.h);
      const int64_t F = p.N / 2, f0 = n0 / 2 + wn * FW;
      uint8_t* reg = smem + wid * 2 * PART;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int64_t row0 = m0 + wm * WTM + i * 32;
        if (row0 >= m_end) break;
#pragma unroll
        for (int jj = 0; jj < FN / 2; ++jj)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x16_t& ga = acc[i][2 * jj];
            const f32x16_t& ua = acc[i][2 * jj + 1];
            const int off = q * (FW * 2) + (((jj * 4 + g) ^ (q & (CH - 1))) << 4) + 8 * hh;
            *reinterpret_cast<uint2*>(reg + off) =
                make_uint2(pack_bf16x2(ga[4 * g], ga[4 * g + 1]), pack_bf16x2(ga[4 * g + 2], ga[4 * g + 3]));
            *reinterpret_cast<uint2*>(reg + PART + off) =
                make_uint2(pack_bf16x2(ua[4 * g], ua[4 * g + 1]), pack_bf16x2(ua[4 * g + 2], ua[4 * g + 3]));
          }
#pragma unroll
        for (int t = 0; t < 32 * CH / 64; ++t) {
          const int r = t * (64 / CH) + lane / CH, ch = lane % CH;
          const int off = r * (FW * 2) + ((ch ^ (r & (CH - 1))) << 4);
          const int64_t row = row0 + r, f = f0 + ch * 8;
          const uint4 vg = *reinterpret_cast<const uint4*>(reg + off);
          const uint4 vu = *reinterpret_cast<const uint4*>(reg + PART + off);
          const uint32_t gw[4] = {vg.x, vg.y, vg.z, vg.w}, uw[4] = {vu.x, vu.y, vu.z, vu.w};
          float hv[8];
          uint32_t hw[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            hw[w] = pack_bf16x2(silu_gate(bf16_lo(gw[w]), bf16_lo(uw[w])), silu_gate(bf16_hi(gw[w]), bf16_hi(uw[w])));
            hv[2 * w] = bf16_lo(hw[w]);
            hv[2 * w + 1] = bf16_hi(hw[w]);
          }
          const bool valid = row < m_end;
          float am = 0.0f;
#pragma unroll
          for (int w = 0; w < 8; ++w) am = fmaxf(am, fabsf(hv[w]));
          if (valid) {
            tile_amax = fmaxf(tile_amax, am);
            if (Yp) {
              *reinterpret_cast<uint4*>(Yp + row * p.N + f) = vg;
              *reinterpret_cast<uint4*>(Yp + row * p.N + F + f) = vu;
            }
            if (Hp) *reinterpret_cast<uint4*>(Hp + row * F + f) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
          }
          if constexpr (EPI == EPI_SILU_Q) {
            // lanes ch .. ch ^ 3 hold the 32 features of one block of one row
            am = fmaxf(am, __shfl_xor(am, 1, 64));
            am = fmaxf(am, __shfl_xor(am, 2, 64));
            const int se = shared_exp<2>(am);
            const uint32_t codes = encode8_e2m1(hv, se);
            if (valid) {
              *reinterpret_cast<uint32_t*>(p.hq + row * (F / 2) + f / 2) = codes;
              if ((ch & 3) == 0) p.hs[row * (F / 32) + f / 32] = (uint8_t)(se + 127);
            }
          }
        }
      }
    } else {
      constexpr int EB = OUT32 ? 4 : 2;        // bytes per element
      constexpr int CH = WTN * EB / 16;        // 16-byte chunks per row
      constexpr int REGION = 32 * WTN * EB;
      static_assert(NW * REGION <= S * STAGE && (CH & (CH - 1)) == 0, "epilogue staging");
      uint8_t* reg = smem + wid * REGION;
      const int64_t col0 = n0 + wn * WTN;
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int64_t row0 = m0 + wm * WTM + i * 32;
        if (row0 >= m_end) break;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const f32x16_t& a = acc[i][j];
            if constexpr (OUT32) {
              const int ch = j * 8 + 2 * g + hh;
              *reinterpret_cast<float4*>(reg + q * (WTN * 4) + ((ch ^ (q & (CH - 1))) << 4)) =
                  make_float4(a[4 * g], a[4 * g + 1], a[4 * g + 2], a[4 * g + 3]);
            } else {
              const int ch = j * 4 + g;
              *reinterpret_cast<uint2*>(reg + q * (WTN * 2) + ((ch ^ (q & (CH - 1))) << 4) + 8 * hh) =
                  make_uint2(pack_bf16x2(a[4 * g], a[4 * g + 1]), pack_bf16x2(a[4 * g + 2], a[4 * g + 3]));
            }
          }
#pragma unroll 4
        for (int t = 0; t < 32 * CH / 64; ++t) {
          const int r = t * (64 / CH) + lane / CH, ch = lane % CH;
          const uint4 v = *reinterpret_cast<const uint4*>(reg + r * (WTN * EB) + ((ch ^ (r & (CH - 1))) << 4));
          const int64_t row = row0 + r, col = col0 + ch * (16 / EB);
          if (row < m_end && col < p.N)
            *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(p.c) + (row * p.N + col) * EB) = v;
        }
      }
    }
  }

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
// rows the work is reading the weights, so the row block is small and the
// ring deep; with many it is the MFMAs and the LDS reads that feed them.
template <int EPI, bool OUT32>
int launch_epi(const Params& p, hipStream_t st) {
  if (p.M <= 32 * (int64_t)p.E) return launch_tiles<32, 256, 1, 4, 4, EPI, OUT32>(p, st);
  if (p.M <= 96 * (int64_t)p.E) return launch_tiles<64, 256, 1, 4, 3, EPI, OUT32>(p, st);
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
  if (M_total > 0x7FFFFFFFLL || N > 0x7FFFFFFFLL || K > (1 << 22)) return NVFP4MOE_ESHAPE;
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
