// Layer norm in front of the layer, and its RMS form (the norm of the Qwen3
// layers whose shapes the library's workloads take), forward and backward with
// the reduction of the weight's and bias's gradients ("miniTE報告、NVFP4強化学習
// の安定性を検証", first paragraph: the learner's update in BF16; the pages name
// no norm).
//
// Mathematics, per row x of D elements, m its mean (RMS: 0):
//   r = 1 / sqrt(mean((x - m)^2) + eps),  h = (x - m) r,  y = h w + b
//   g = dy w,  dx = r (g - mean(g) - h mean(g h))     (RMS: without mean(g))
//   dw = sum over rows of dy h,  db = sum over rows of dy
// All sums are fp32; the variance is the mean square of the differences, taken
// from registers after the mean.  A mean far from 0 is off by the rounding of its
// sum; rows whose mean is more than 16 deviations take the differences' own mean
// out too (without it the variance was off by up to percents at 2^20 deviations;
// always taking it out costs 16384 x 2048 bf16 33.5 us for 28.6).
//
// Layout.  A row belongs to one wave up to 2048 elements (512 if they are read
// singly), to a workgroup beyond; its elements stay in registers from the load
// to the store, so every tensor is read once and written once.  Lanes take 8
// consecutive elements where the row length and the pointers allow 16-byte
// accesses, single ones otherwise.  Groups go round over the rows and keep the
// weights, and in the backward pass the columns' sums, in registers.  The
// sums of a workgroup go to the workspace as one row, and a second launch adds
// those rows in order: no atomics, the same bits every time.  Few rows take one
// launch, some workgroups of which sum columns while the others write dx.
//
// Bounds and measurements (us).  HBM: 16384 x 2048 bf16 forward 27 to 28 (134 MB at
// 4.8 TB/s, other inputs each time; 20 of the same), gradient of 8192 x 2048 (bf16
// rows, fp32 dy) 28 and 4 for the sums of 256 workgroups (10 when each thread of
// 256 added 32 of them one after another); of the same inputs together 27, 31 when
// the next row's loads branch on its type (each branch then waits for the other's),
// 29 with two rows in flight; a wave for rows of 2048 with twice the columns a lane
// 49.  16 rows of 2048: 3.5.  Odd lengths, by single elements: 16384 x 2047 bf16
// forward 85 to 90, 4096 x 6001 fp32 59 to 66.
#include <type_traits>

#include "common.hpp"

namespace nvfp4moe {
namespace {

constexpr int kNormMaxD = 16384;
constexpr int kNormBwdBlocks = 256;  // rows of partial sums at most
// The mean's square over the variance from which the mean is corrected.  Its error
// is at most 86 roundings (a thread's 64 elements, then the lanes and waves), 2^-17
// of it: below this ratio that adds no more than 2^-26 to the variance.
constexpr float kNormFar = 256.0f;
// Up to so many rows the gradient takes one launch, whatever their length and type:
// a compromise, since the two are level near 330 rows at 512 columns, 400 at 2048,
// and past 1024 at an odd length.  Measured (us through the C entry point, both
// gradients; one launch and two):
//   rows   512 columns   2048         2557 fp32    8192
//     16   3.7   6.9     3.5   8.0    4.8   9.1    3.6   7.5
//    256   5.9   7.2     5.8   8.7    5.2  11.1   10.7  17.0
//    512   9.5   7.2     9.5   9.4    7.4  13.4   22.3  17.8
//   1024  17.2   7.6    21.2  10.9   14.5  15.8   43.3  22.3
constexpr int kNormFewRows = 384;

struct NormParams {
  const void* x;
  const void* dy;
  const void* w;
  const void* b;
  const float* mean_in;
  const float* rstd_in;
  void* out;  // y or dx
  float* mean;
  float* rstd;
  float* part;  // backward: [2][gridDim.x][D] partial sums of dw, db
  float* dw;    // the same at once (few rows)
  float* db;
  int64_t T;
  int D;
  float eps;
  bool x_bf16, dy_bf16, w_bf16, out_bf16, rms, want_dw, want_db;
};

// Elements (c * NT + t) * W + 0..W-1, c < NC, of a row, zeros past its end.
template <int NT, int NC, int W>
__device__ __forceinline__ void load_row(const void* base, bool bf16, int64_t at, int D, int t, float (&v)[NC * W]) {
  if (bf16) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + at;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * NT + t) * W;
      if constexpr (W == 8) {
        uint4 q = make_uint4(0, 0, 0, 0);
        if (col < D) q = *reinterpret_cast<const uint4*>(p + col);
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[c * W + 2 * i] = bf16_lo(u[i]);
          v[c * W + 2 * i + 1] = bf16_hi(u[i]);
        }
      } else {
        v[c] = col < D ? bf16_lo(p[col]) : 0.0f;
      }
    }
  } else {
    const float* p = reinterpret_cast<const float*>(base) + at;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * NT + t) * W;
      if constexpr (W == 8) {
        float4 a = make_float4(0, 0, 0, 0), b = a;
        if (col < D) {
          a = *reinterpret_cast<const float4*>(p + col);
          b = *reinterpret_cast<const float4*>(p + col + 4);
        }
        const float u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c * W + i] = u[i];
      } else {
        v[c] = col < D ? p[col] : 0.0f;
      }
    }
  }
}

// The same as they are stored, by buffer loads of `row`, a region of D elements
// or of none: no branch, so that nothing waits for them before values().
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_region(const void* base, bool bf16, int64_t at, int n, bool live) {
  const int size = bf16 ? 2 : 4;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(reinterpret_cast<const uint8_t*>(base)) + at * size, (short)0,
                                           live ? n * size : 0, kRawBufferWord3);
}
template <int NT, int NC, int W>
__device__ __forceinline__ void load_raw(__amdgpu_buffer_rsrc_t row, bool bf16, int t, uint32_t (&v)[NC * W]) {
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const uint32_t col = (c * NT + t) * W;
    if constexpr (W == 8) {
      const uint32_t off = col * (bf16 ? 2 : 4);
      const u32x4_t a = __builtin_amdgcn_raw_buffer_load_b128(row, off, 0, 0);
      const u32x4_t b = __builtin_amdgcn_raw_buffer_load_b128(row, bf16 ? kOOB : off + 16, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[c * 8 + i] = a[i];
        v[c * 8 + 4 + i] = b[i];
      }
    } else {
      if (bf16) v[c] = __builtin_amdgcn_raw_buffer_load_b16(row, col * 2, 0, 0);
      else v[c] = __builtin_amdgcn_raw_buffer_load_b32(row, col * 4, 0, 0);
    }
  }
}
template <int NC, int W>
__device__ __forceinline__ void values(const uint32_t (&raw)[NC * W], bool bf16, float (&v)[NC * W]) {
  if (bf16) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if constexpr (W == 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[c * W + 2 * i] = bf16_lo(raw[c * W + i]);
          v[c * W + 2 * i + 1] = bf16_hi(raw[c * W + i]);
        }
      } else {
        v[c] = bf16_lo(raw[c]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NC * W; ++i) v[i] = __uint_as_float(raw[i]);
  }
}

template <int NT, int NC, int W>
__device__ __forceinline__ void store_row(void* base, bool bf16, int64_t at, int D, int t, const float (&v)[NC * W]) {
  if (bf16) {
    uint16_t* p = reinterpret_cast<uint16_t*>(base) + at;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * NT + t) * W;
      if (col >= D) continue;
      if constexpr (W == 8) {
        const float* a = v + c * W;
        *reinterpret_cast<uint4*>(p + col) = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                                        pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
      } else {
        p[col] = (uint16_t)f32_to_bf16_rne(v[c]);
      }
    }
  } else {
    float* p = reinterpret_cast<float*>(base) + at;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int col = (c * NT + t) * W;
      if (col >= D) continue;
      if constexpr (W == 8) {
        const float* a = v + c * W;
        *reinterpret_cast<float4*>(p + col) = make_float4(a[0], a[1], a[2], a[3]);
        *reinterpret_cast<float4*>(p + col + 4) = make_float4(a[4], a[5], a[6], a[7]);
      } else {
        p[col] = v[c];
      }
    }
  }
}

// Sums over the NT threads of a row (a wave, or several: the GROUPS rows of the
// workgroup then call this together); every thread of a row receives the same
// bits.  `turn` alternates between two buffers, so one barrier a call is enough.
template <int NT, int N, int GROUPS>
__device__ __forceinline__ void row_sums(float (&s)[N], int& turn) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor(s[i], o, 64);
  if constexpr (NT > 64) {
    __shared__ float red[2][2][GROUPS * NT / 64];
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((threadIdx.x & 63) == 0) red[turn][i][threadIdx.x >> 6] = s[i];
    __syncthreads();
    const int first = threadIdx.x / NT * (NT / 64);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float a = red[turn][i][first];
#pragma unroll
      for (int w = 1; w < NT / 64; ++w) a += red[turn][i][first + w];
      s[i] = a;
    }
    turn ^= 1;
  }
}

template <int NT>
constexpr int threads() {
  return NT < 256 ? 256 : NT;
}

template <int NT, int NC, int W>
__global__ __launch_bounds__(threads<NT>()) void norm_fwd_kernel(NormParams p) {
  constexpr int N = NC * W, GROUPS = threads<NT>() / NT;
  const int t = threadIdx.x % NT, D = p.D;
  const float inv_d = 1.0f / (float)D;
  float w[N], b[N];
  if (p.w) load_row<NT, NC, W>(p.w, p.w_bf16, 0, D, t, w);
  if (p.b) load_row<NT, NC, W>(p.b, p.w_bf16, 0, D, t, b);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!p.w) w[i] = 1.0f;
    if (!p.b) b[i] = 0.0f;
  }
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * GROUPS + threadIdx.x / NT; row < p.T; row += (int64_t)gridDim.x * GROUPS) {
    float v[N];
    load_row<NT, NC, W>(p.x, p.x_bf16, row * D, D, t, v);
    float m = 0.0f;
    if (!p.rms) {
      float s[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < N; ++i) s[0] += v[i];
      row_sums<NT, 1, GROUPS>(s, turn);
      m = s[0] * inv_d;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < W; ++i) v[c * W + i] = (c * NT + t) * W < D ? v[c * W + i] - m : 0.0f;
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < N; ++i) s[0] += v[i] * v[i];
    row_sums<NT, 1, GROUPS>(s, turn);
    float ms = s[0] * inv_d;
    if (m * m > kNormFar * ms) {  // (the same in all threads of the row; RMS: m is 0)
      s[0] = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) s[0] += v[i];
      row_sums<NT, 1, GROUPS>(s, turn);
      const float off = s[0] * inv_d;  // what the rounding of the first sum left in the differences
      ms = fmaxf(ms - off * off, 0.0f);
      m += off;
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] -= off;
    }
    const float r = 1.0f / sqrtf(ms + p.eps);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] * r * w[i] + b[i];
    store_row<NT, NC, W>(p.out, p.out_bf16, row * D, D, t, v);
    if (t == 0) {
      if (p.mean) p.mean[row] = m;
      if (p.rstd) p.rstd[row] = r;
    }
  }
}

// Threads of a backward workgroup: eight waves of a row each, so that few
// workgroups, whose sums the second launch adds, keep two waves per SIMD.
template <int NT>
constexpr int bwd_threads() {
  return NT < 512 ? 512 : NT;
}

template <int NT, int NC, int W>
__global__ __launch_bounds__(bwd_threads<NT>()) void norm_bwd_kernel(NormParams p) {
  constexpr int N = NC * W, GROUPS = bwd_threads<NT>() / NT;
  // The next row is on its way while one is in work, where the registers allow.
  constexpr bool AHEAD = 7 * N + 24 <= (bwd_threads<NT>() > 512 ? 128 : 256);
  const int t = threadIdx.x % NT, D = p.D;
  const float inv_d = 1.0f / (float)D;
  float w[N], dw[N], db[N];
  if (p.w) load_row<NT, NC, W>(p.w, p.w_bf16, 0, D, t, w);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!p.w) w[i] = 1.0f;
    dw[i] = db[i] = 0.0f;
  }
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
  int64_t row = (int64_t)blockIdx.x * GROUPS + group;
  uint32_t nx[AHEAD ? N : 1], ndy[AHEAD ? N : 1];  // the next row as stored
  float nr = 0.0f, nm = 0.0f;
  const auto next = [&](int64_t at) __attribute__((always_inline)) {
    const bool live = at < p.T;
    if constexpr (AHEAD) {
      load_raw<NT, NC, W>(row_region(p.x, p.x_bf16, at * D, D, live), p.x_bf16, t, nx);
      load_raw<NT, NC, W>(row_region(p.dy, p.dy_bf16, at * D, D, live), p.dy_bf16, t, ndy);
      nr = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(row_region(p.rstd_in, false, at, 1, live), 0, 0, 0));
      nm = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(row_region(p.mean_in, false, at, 1, live && !p.rms), 0, 0, 0));
    }
  };
  // (The groups of a workgroup that share a barrier per row go round together,
  // the last ones perhaps without a row.)
  const bool together = NT > 64;
  next(row);
  for (; together ? row - group < p.T : row < p.T; row += step) {
    const bool live = row < p.T;
    float h[N], dy[N], r = 0.0f, m = 0.0f;
    if constexpr (AHEAD) {
      values<NC, W>(nx, p.x_bf16, h);
      values<NC, W>(ndy, p.dy_bf16, dy);
      r = nr;
      m = nm;
    } else if (live) {
      load_row<NT, NC, W>(p.x, p.x_bf16, row * D, D, t, h);
      load_row<NT, NC, W>(p.dy, p.dy_bf16, row * D, D, t, dy);
      r = p.rstd_in[row];
      m = p.rms ? 0.0f : p.mean_in[row];
    }
    float s[2] = {0.0f, 0.0f};
    if (live) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = c * W; i < c * W + W; ++i) {
          h[i] = (c * NT + t) * W < D ? (h[i] - m) * r : 0.0f;
          dw[i] += dy[i] * h[i];
          db[i] += dy[i];
          dy[i] *= w[i];
          s[0] += dy[i] * h[i];
          s[1] += dy[i];
        }
    }
    next(row + step);
    if (p.out) {
      row_sums<NT, 2, GROUPS>(s, turn);
      const float gh = s[0] * inv_d, g = p.rms ? 0.0f : s[1] * inv_d;
      if (live) {
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = r * (dy[i] - g - h[i] * gh);
        store_row<NT, NC, W>(p.out, p.out_bf16, row * D, D, t, h);
      }
    }
  }
  // This workgroup's sums.
  float* to = p.part + (int64_t)blockIdx.x * D;
  const int64_t db_at = (int64_t)gridDim.x * D;
  if constexpr (GROUPS == 1) {
    if (p.want_dw) store_row<NT, NC, W>(to, false, 0, D, t, dw);
    if (p.want_db) store_row<NT, NC, W>(to + db_at, false, 0, D, t, db);
  } else {
    __shared__ __attribute__((aligned(16))) float sum[NT * N];
    for (int which = 0; which < 2; ++which) {
      if (!(which ? p.want_db : p.want_dw)) continue;
      for (int g = 0; g < GROUPS; ++g) {  // the groups add their sums in turn
        if ((int)threadIdx.x / NT == g) {
          float a[N];
          if (g > 0) load_row<NT, NC, W>(sum, false, 0, D, t, a);
#pragma unroll
          for (int i = 0; i < N; ++i) a[i] = (g > 0 ? a[i] : 0.0f) + (which ? db[i] : dw[i]);
          if (g + 1 < GROUPS) store_row<NT, NC, W>(sum, false, 0, D, t, a);
          else store_row<NT, NC, W>(to + which * db_at, false, 0, D, t, a);
        }
        __syncthreads();
      }
    }
  }
}

// Few rows: one launch.  The first workgroups take 32 columns each and sum them
// over all rows, which the cache then holds for the others, each of which takes
// rows and writes dx.
template <int NT, int NC, int W>
__global__ __launch_bounds__(bwd_threads<NT>()) void norm_bwd_few_kernel(NormParams p, int strips) {
  constexpr int N = NC * W, BT = bwd_threads<NT>(), GROUPS = BT / NT;
  const int D = p.D;
  if ((int)blockIdx.x < strips) {
    constexpr int G = BT / 32;  // threads of a column
    __shared__ float red[2][32][G + 1];
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
    float dw = 0.0f, db = 0.0f;
    if (col < D) {
#pragma unroll 4
      for (int64_t t = g; t < p.T; t += G) {
        const int64_t at = t * D + col;
        const float x = p.x_bf16 ? bf16_lo(reinterpret_cast<const uint16_t*>(p.x)[at]) : reinterpret_cast<const float*>(p.x)[at];
        const float dy = p.dy_bf16 ? bf16_lo(reinterpret_cast<const uint16_t*>(p.dy)[at]) : reinterpret_cast<const float*>(p.dy)[at];
        dw += dy * ((x - (p.rms ? 0.0f : p.mean_in[t])) * p.rstd_in[t]);
        db += dy;
      }
    }
    red[0][c][g] = dw;
    red[1][c][g] = db;
    __syncthreads();
    const int oc = threadIdx.x / G, og = threadIdx.x % G, out = blockIdx.x * 32 + oc;
    dw = red[0][oc][og];
    db = red[1][oc][og];
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) {
      dw += __shfl_xor(dw, o, 64);
      db += __shfl_xor(db, o, 64);
    }
    if (og == 0 && out < D) {
      if (p.dw) p.dw[out] = dw;
      if (p.db) p.db[out] = db;
    }
    return;
  }
  const int t = threadIdx.x % NT;
  const int64_t row = ((int64_t)blockIdx.x - strips) * GROUPS + threadIdx.x / NT;
  const bool live = row < p.T;
  const float inv_d = 1.0f / (float)D;
  float h[N], g[N], w[N], s[2] = {0.0f, 0.0f}, r = 0.0f;
  if (live) {
    load_row<NT, NC, W>(p.x, p.x_bf16, row * D, D, t, h);
    load_row<NT, NC, W>(p.dy, p.dy_bf16, row * D, D, t, g);
    if (p.w) load_row<NT, NC, W>(p.w, p.w_bf16, 0, D, t, w);
    r = p.rstd_in[row];
    const float m = p.rms ? 0.0f : p.mean_in[row];
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = c * W; i < c * W + W; ++i) {
        h[i] = (c * NT + t) * W < D ? (h[i] - m) * r : 0.0f;
        if (p.w) g[i] *= w[i];
        s[0] += g[i] * h[i];
        s[1] += g[i];
      }
  }
  int turn = 0;
  row_sums<NT, 2, GROUPS>(s, turn);
  if (live) {
    const float gh = s[0] * inv_d, gm = p.rms ? 0.0f : s[1] * inv_d;
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = r * (g[i] - gm - h[i] * gh);
    store_row<NT, NC, W>(p.out, p.out_bf16, row * D, D, t, h);
  }
}

// Column sums of rows partial sums (at most kNormBwdBlocks): 32 columns a
// workgroup, 32 groups of 8 rows, whose loads are all in flight at once.
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float* part, int rows, int D, float* dw, float* db) {
  __shared__ float red[32][33];
  const float* from = part + (int64_t)blockIdx.y * rows * D;
  float* to = blockIdx.y ? db : dw;
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  constexpr int PER = kNormBwdBlocks / 32;
  float v[PER], s = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) v[i] = to && col < D && g + 32 * i < rows ? from[(int64_t)(g + 32 * i) * D + col] : 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) s += v[i];
  red[c][g] = s;
  __syncthreads();
  // the columns' sums: 32 lanes each
  s = red[threadIdx.x >> 5][threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  const int out = blockIdx.x * 32 + (threadIdx.x >> 5);
  if ((threadIdx.x & 31) == 0 && to && out < D) to[out] = s;
}

// Kernels by the row's length: a wave a row, then several.
template <int NT_, int NC_, int W_>
struct Shape {
  static constexpr int NT = NT_, NC = NC_, W = W_;
};
template <class F>
void by_length(int D, bool vec, F&& f) {
  if (vec) {
    if (D <= 512) return f(Shape<64, 1, 8>{});
    if (D <= 1024) return f(Shape<64, 2, 8>{});
    if (D <= 2048) return f(Shape<64, 4, 8>{});
    if (D <= 4096) return f(Shape<256, 2, 8>{});
    if (D <= 8192) return f(Shape<256, 4, 8>{});
    return f(Shape<256, 8, 8>{});
  }
  if (D <= 128) return f(Shape<64, 2, 1>{});
  if (D <= 512) return f(Shape<64, 8, 1>{});
  if (D <= 2048) return f(Shape<256, 8, 1>{});
  if (D <= 4096) return f(Shape<256, 16, 1>{});
  return f(Shape<1024, 16, 1>{});
}
// The backward pass keeps three times as much per column in registers.
template <class F>
void bwd_by_length(int D, bool vec, F&& f) {
  if (vec) {
    if (D <= 512) return f(Shape<64, 1, 8>{});
    if (D <= 1024) return f(Shape<64, 2, 8>{});
    if (D <= 2048) return f(Shape<128, 2, 8>{});
    if (D <= 4096) return f(Shape<256, 2, 8>{});
    if (D <= 8192) return f(Shape<512, 2, 8>{});
    return f(Shape<1024, 2, 8>{});
  }
  if (D <= 128) return f(Shape<64, 2, 1>{});
  if (D <= 512) return f(Shape<64, 8, 1>{});
  if (D <= 2048) return f(Shape<256, 8, 1>{});
  if (D <= 4096) return f(Shape<256, 16, 1>{});
  return f(Shape<1024, 16, 1>{});
}

bool is_float(int dt) { return dt == NVFP4MOE_F32 || dt == NVFP4MOE_BF16; }

}  // namespace
}  // namespace nvfp4moe

using namespace nvfp4moe;

extern "C" int layer_norm(const void* x, int x_dtype, int64_t T, int64_t D, const void* w, const void* b, int w_dtype,
                          float eps, int kind, void* y, int y_dtype, float* mean, float* rstd,
                          nvfp4moe_stream_t stream) {
  if (T < 0 || D < 0 || !is_float(x_dtype) || !is_float(y_dtype) || ((w || b) && !is_float(w_dtype)))
    return NVFP4MOE_EINVAL;
  if (kind != NVFP4MOE_NORM_LAYER && kind != NVFP4MOE_NORM_RMS) return NVFP4MOE_EINVAL;
  if (!(eps >= 0.0f) || (kind == NVFP4MOE_NORM_RMS && mean)) return NVFP4MOE_EINVAL;
  if (T > 0 && (!x || !y)) return NVFP4MOE_EINVAL;
  if (D < 1 || D > kNormMaxD) return NVFP4MOE_ESHAPE;
  const int xb = dtype_bytes(x_dtype), yb = dtype_bytes(y_dtype), wb = w || b ? dtype_bytes(w_dtype) : 1;
  if (!aligned(x, xb) || !aligned(y, yb) || !aligned(w, wb) || !aligned(b, wb) || !aligned(mean, 4) || !aligned(rstd, 4))
    return NVFP4MOE_ESHAPE;
  const int arch = check_arch();
  if (arch != NVFP4MOE_OK) return arch;
  if (T == 0) return NVFP4MOE_OK;
  NormParams p{};
  p.x = x;
  p.w = w;
  p.b = b;
  p.out = y;
  p.mean = mean;
  p.rstd = rstd;
  p.T = T;
  p.D = (int)D;
  p.eps = eps;
  p.x_bf16 = x_dtype == NVFP4MOE_BF16;
  p.w_bf16 = w_dtype == NVFP4MOE_BF16;
  p.out_bf16 = y_dtype == NVFP4MOE_BF16;
  p.rms = kind == NVFP4MOE_NORM_RMS;
  hipStream_t st = as_stream(stream);
  const bool vec = D % 8 == 0 && aligned(x, 16) && aligned(y, 16) && aligned(w, 16) && aligned(b, 16);
  by_length(p.D, vec, [&](auto shape) {
    constexpr int NT = decltype(shape)::NT, NC = decltype(shape)::NC, W = decltype(shape)::W;
    const int64_t n = cdiv(T, threads<NT>() / NT);
    norm_fwd_kernel<NT, NC, W><<<(unsigned)(n < kStreamBlocks ? n : kStreamBlocks), threads<NT>(), 0, st>>>(p);
  });
  return launch_status();
}

extern "C" size_t layer_norm_bwd_workspace_size(int64_t T, int64_t D) {
  if (T <= kNormFewRows || D < 1 || D > kNormMaxD) return 0;
  return (size_t)(2 * kNormBwdBlocks * D * 4);
}

extern "C" int layer_norm_bwd(const void* dy, int dy_dtype, const void* x, int x_dtype, int64_t T, int64_t D,
                              const void* w, int w_dtype, const float* mean, const float* rstd, int kind, void* dx,
                              int dx_dtype, float* dw, float* db, void* workspace, size_t ws_bytes,
                              nvfp4moe_stream_t stream) {
  if (T < 0 || D < 0 || !is_float(dy_dtype) || !is_float(x_dtype) || (w && !is_float(w_dtype)) ||
      (dx && !is_float(dx_dtype)))
    return NVFP4MOE_EINVAL;
  if (kind != NVFP4MOE_NORM_LAYER && kind != NVFP4MOE_NORM_RMS) return NVFP4MOE_EINVAL;
  if (T > 0 && (!dy || !x || !rstd || (kind == NVFP4MOE_NORM_LAYER && !mean) || (!dx && !dw && !db)))
    return NVFP4MOE_EINVAL;
  if (D < 1 || D > kNormMaxD) return NVFP4MOE_ESHAPE;
  const int xb = dtype_bytes(x_dtype), yb = dtype_bytes(dy_dtype), wb = w ? dtype_bytes(w_dtype) : 1,
            ob = dx ? dtype_bytes(dx_dtype) : 1;
  if (!aligned(x, xb) || !aligned(dy, yb) || !aligned(w, wb) || !aligned(dx, ob) || !aligned(mean, 4) ||
      !aligned(rstd, 4) || !aligned(dw, 4) || !aligned(db, 4))
    return NVFP4MOE_ESHAPE;
  if (T > kNormFewRows && (dw || db)) {
    if (!workspace || ws_bytes < layer_norm_bwd_workspace_size(T, D)) return NVFP4MOE_EWORKSPACE;
    if (!aligned(workspace, 16)) return NVFP4MOE_ESHAPE;
  }
  const int arch = check_arch();
  if (arch != NVFP4MOE_OK) return arch;
  hipStream_t st = as_stream(stream);
  if (T == 0) {
    const unsigned blocks = (unsigned)cdiv(D, 256);
    if (dw) fill_u32_kernel<<<blocks, 256, 0, st>>>(reinterpret_cast<uint32_t*>(dw), 0u, D);
    if (db) fill_u32_kernel<<<blocks, 256, 0, st>>>(reinterpret_cast<uint32_t*>(db), 0u, D);
    return launch_status();
  }
  NormParams p{};
  p.x = x;
  p.dy = dy;
  p.w = w;
  p.mean_in = mean;
  p.rstd_in = rstd;
  p.out = dx;
  p.part = reinterpret_cast<float*>(workspace);
  p.T = T;
  p.D = (int)D;
  p.x_bf16 = x_dtype == NVFP4MOE_BF16;
  p.dy_bf16 = dy_dtype == NVFP4MOE_BF16;
  p.w_bf16 = w_dtype == NVFP4MOE_BF16;
  p.out_bf16 = dx_dtype == NVFP4MOE_BF16;
  p.rms = kind == NVFP4MOE_NORM_RMS;
  p.want_dw = dw != nullptr;
  p.want_db = db != nullptr;
  p.dw = dw;
  p.db = db;
  const bool vec = D % 8 == 0 && aligned(x, 16) && aligned(dy, 16) && aligned(w, 16) && aligned(dx, 16);
  if (T <= kNormFewRows) {
    const int strips = dw || db ? (int)cdiv(D, 32) : 0;
    bwd_by_length(p.D, vec, [&](auto shape) {
      constexpr int NT = decltype(shape)::NT, NC = decltype(shape)::NC, W = decltype(shape)::W;
      const int64_t rows = dx ? cdiv(T, bwd_threads<NT>() / NT) : 0;
      norm_bwd_few_kernel<NT, NC, W><<<(unsigned)(strips + rows), bwd_threads<NT>(), 0, st>>>(p, strips);
    });
    return launch_status();
  }
  int64_t blocks = kNormBwdBlocks;
  bwd_by_length(p.D, vec, [&](auto shape) {
    constexpr int NT = decltype(shape)::NT, NC = decltype(shape)::NC, W = decltype(shape)::W;
    const int64_t n = cdiv(T, bwd_threads<NT>() / NT);
    if (n < blocks) blocks = n;
    norm_bwd_kernel<NT, NC, W><<<(unsigned)blocks, bwd_threads<NT>(), 0, st>>>(p);
  });
  const int rc = launch_status();
  if (rc != NVFP4MOE_OK || (!dw && !db)) return rc;
  norm_sum_kernel<<<dim3((unsigned)cdiv(D, 32), db ? 2 : 1), 1024, 0, st>>>(p.part, (int)blocks, p.D, dw, db);
  return launch_status();
}
