// Device helpers shared by the grouped GEMM kernels: waits and barriers, the
// LDS-direct loads and the swizzles of their tiles, and the lookup of a tile
// among the experts' row blocks.
#pragma once

#include "common.hpp"

namespace nvfp4moe {
namespace {

typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(8))) int i32x8_t;
typedef __attribute__((ext_vector_type(4))) int i32x4_t;
typedef __attribute__((address_space(3))) void lds_void_t;

__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A wave-uniform 64-bit value moved to scalar registers.
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Wait until at most min(n, MAX) vector memory operations are outstanding
// (n wave-uniform).
template <int MAX>
__device__ __forceinline__ void wait_vmcnt_upto(int n) {
  if constexpr (MAX <= 0) {
    wait_vmcnt<0>();
  } else {
    if (n >= MAX)
      wait_vmcnt<MAX>();
    else
      wait_vmcnt_upto<MAX - 1>(n);
  }
}
constexpr int kMaxEpilogueStores = 32;

// Wait until at most `ahead` steps of NDMA loads each are outstanding
// (ahead in [0, MAX], wave-uniform).
template <int MAX, int NDMA>
__device__ __forceinline__ void wait_steps_ahead(int ahead) {
  if constexpr (MAX <= 0) {
    wait_vmcnt<0>();
  } else {
    if (ahead >= MAX)
      wait_vmcnt<MAX * NDMA>();
    else
      wait_steps_ahead<MAX - 1, NDMA>(ahead);
  }
}

// One wave-wide LDS-direct load: lane l's `size` bytes land at LDS byte
// address lds + size*l (lds wave-uniform).  Issued as inline assembly so the
// compiler does not make every later LDS read wait for it: the kernel keeps
// the count of its own loads (s_waitcnt vmcnt) and orders LDS with barriers.
// `lds` goes through readfirstlane: under register pressure the compiler may
// hold a uniform value in a vector register, which the scalar operand cannot
// take (a no-op when it is already scalar).
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t r, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(
                   __builtin_amdgcn_readfirstlane(lds)),
               "v"(voff), "s"(r)
               : "memory", "m0");
}
// The same with 4 bytes per lane: lane l's word lands at lds + 4*l (probed).
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(__builtin_amdgcn_readfirstlane(lds)),
               "v"(voff), "s"(r)
               : "memory", "m0");
}
// K-major bf16 tile: chunk c (8 elements) of row r at byte r*128 + 16*(c ^ kswz(r)).
__device__ __forceinline__ int kswz(int r) { return (r ^ (r >> 3)) & 7; }
// Swizzle of a K-major tile with ROWB-byte rows (128: kswz; 64: (r / 2) % 4),
// conflict-free for 16-byte reads of the same chunk in 8 consecutive rows.
template <int ROWB>
__device__ __forceinline__ int rswz(int r) {
  if constexpr (ROWB == 128) return kswz(r);
  else return (r >> 1) & 3;
}
// MN-major bf16 tile: chunk c of reduction row k at byte k*rowbytes + 16*(c ^ mswz(k)).
// Any 4 consecutive rows k = 4i..4i+3 then put a transposed read's 32- and
// 64-byte row segments on disjoint banks.
__device__ __forceinline__ int mswz(int k) { return (0xCA60 >> ((k & 3) * 4)) & 15; }  // {0, 6, 10, 12}
// Clamped [lo, hi) row range of expert e.  `off` is the global offsets array
// or its copy in LDS.
typedef __attribute__((address_space(3))) const int32_t lds_i32_t;
template <class OffPtr>
__device__ __forceinline__ void expert_range(OffPtr off, int e, int64_t M, int& lo, int& hi) {
  lo = off[e];
  hi = off[e + 1];
  lo = lo < 0 ? 0 : lo > M ? (int)M : lo;
  hi = hi < lo ? lo : hi > M ? (int)M : hi;
}

// Number of BM-row blocks over all experts.  Runs on one whole wave.
template <int BM>
__device__ int count_row_blocks(const int32_t* __restrict__ off, int E, int64_t M) {
  const int lane = threadIdx.x & 63;
  int total = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    int cnt = 0;
    if (e < E) {
      int lo, hi;
      expert_range(off, e, M, lo, hi);
      cnt = (hi - lo + BM - 1) / BM;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) cnt += __shfl_xor(cnt, o, 64);
    total += cnt;
  }
  return total;
}

// Map row block `slot` to (expert, first row, end row) by a prefix sum of
// per-expert block counts.  Runs on one whole wave; false past the last block.
// Tile L of the row-grouped layouts: its expert, row range and n-tile.  The
// tiles of one expert are numbered n-tile-major when NMAJOR (the expert's
// row blocks that share a weight panel are neighbours, so they run side by
// side on one XCD), row-block-major otherwise.  Tile numbers stay below 2^31
// (checked at launch), so the divisions are 32-bit ones.
template <int BM, bool NMAJOR, class OffPtr>
__device__ bool find_tile(OffPtr off, int E, int64_t M, int64_t L64, int n_tiles, int& e_out,
                          int64_t& r0, int64_t& r1, int& n_out) {
  const int lane = threadIdx.x & 63;
  const uint32_t L = (uint32_t)L64, nt = (uint32_t)n_tiles;
  const uint32_t slot = L / nt;  // the expert's tiles span its row blocks x n_tiles
  uint32_t running = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, hi = 0, cnt = 0;
    if (e < E) {
      expert_range(off, e, M, lo, hi);
      cnt = (hi - lo + BM - 1) / BM;
    }
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o, 64);
      if (lane >= o) incl += v;
    }
    const uint32_t total = (uint32_t)__shfl(incl, 63, 64);
    if (slot < running + total) {
      const bool mine = slot >= running + incl - cnt && slot < running + incl;
      const uint64_t mask = __ballot(mine);
      const int srcl = __ffsll((unsigned long long)mask) - 1;
      e_out = __shfl(e, srcl, 64);
      const int lo_s = __shfl(lo, srcl, 64), hi_s = __shfl(hi, srcl, 64), ex = __shfl(incl - cnt, srcl, 64);
      const uint32_t cnt_s = (uint32_t)__shfl(cnt, srcl, 64);
      const uint32_t rb0 = running + (uint32_t)ex;  // the expert's first row block
      uint32_t rb;
      if (NMAJOR) {
        const uint32_t t = L - rb0 * nt;
        n_out = (int)(t / cnt_s);
        rb = t % cnt_s;
      } else {
        n_out = (int)(L % nt);
        rb = slot - rb0;
      }
      r0 = lo_s + (int64_t)rb * BM;
      r1 = r0 + BM < hi_s ? r0 + BM : hi_s;
      return true;
    }
    running += total;
  }
  return false;
}

// Gate+up tiles of the SiLU-gate epilogue: tile row r (of 256) is expert row
// gate_f * ((r / 32) % 2) + j0 + 32 * (r / 64) + r % 32, so 32-row granules
// alternate gate and up rows of the same 32 features; each wave's pair of
// adjacent 32-column MFMA blocks then holds matching gate and up columns.
__device__ __forceinline__ int64_t gate_up_row(int r, int64_t gate_f, int64_t j0) {
  return ((r >> 5) & 1) * gate_f + j0 + ((r >> 6) << 5) + (r & 31);
}

// Scheduling hint: N_MFMA MFMAs with N_DS LDS reads interleaved one after
// each MFMA (the reads feed the next sub-step), then any reads left over.
template <int N_MFMA, int N_DS>
__device__ __forceinline__ void interleave_mfma_ds() {
  if constexpr (N_MFMA > 0) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // one MFMA
    if constexpr (N_DS > 0) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // one DS read
    interleave_mfma_ds<N_MFMA - 1, (N_DS > 0 ? N_DS - 1 : 0)>();
  } else if constexpr (N_DS > 0) {
    __builtin_amdgcn_sched_group_barrier(0x100, N_DS, 0);
  }
}

}  // namespace
}  // namespace nvfp4moe
