// Root-mean-square norm with the residual's addition, forward and backward.
//
//   forward : h = x + res            H = bf16(h)
//             Y = bf16(h rstd w),    rstd = 1 / sqrt(mean(h^2) + eps)
//             codes, scales: the MXFP8 form of Y (optional)
//   backward: t = dY w, n = h rstd
//             dX = bf16(rstd (t - n mean(t n)) + dH)
//             dW = bf16(sum over rows of dY n)
//
// About ten operations per element against 2 bytes read or written for each
// tensor: HBM-bound, so every tensor is touched once. A row stays in the
// registers of its threads (a wave, or a whole block; VPT vectors of 8
// elements each) between the sums and the outputs. The sums of the forward run
// over the unrounded fp32 h = x + res; Y is rounded once. The MXFP8 codes are
// those of the rounded Y, as quant_pack_mxfp8 gives them, so that both outputs
// stand for one value (the MX-native forward does not read them: it takes bf16
// and quantizes it into an order of its own).
//
// Measured (MI355X): forward 4096 x 4096 with H 22 us (6.0 TB/s), 8192 x 8192
// with H, Y and MXFP8 108 us (5.6 TB/s), one row of 4096 2.8 us; backward with
// dH 4096 x 4096 23 us, with dW too 28 us and 4 for the sum of its partials
// (4.2 TB/s), 8192 x 8192 106 and 5 (4.8 TB/s), 4097 x 5003 50 to 54 us.
//
// Rows of any length: a row of D % 8 != 0 elements starts at an address that
// is a multiple of 2 only. The forward issues its 16-byte accesses there all
// the same (global memory takes them at any alignment on amdhsa; 4097 rows of
// 5003: 5.1 TB/s), the row's last D % 8 elements one by one. The backward, with
// three tensors to read for one to write, loses half its rate that way: there
// a thread's vectors are the memory's aligned ones, which lie 0 to 7 elements
// before the row's (the same shift for all the tensors of a row), and the
// elements of the neighbouring rows are masked out.
#pragma once

#include "common.hpp"
#include "mx.hpp"

namespace lora4 {
namespace norm {

// 1024 threads x 2 vectors of 8; one vector less for rows that start unaligned
constexpr int MAX_D = 16384, MAX_D_UNALIGNED = 16376;

struct FwdParams {
  const uint16_t *X;
  const uint16_t *R;      // residual, or nullptr
  const uint16_t *w;
  int64_t M;
  int D;
  float eps;
  uint16_t *H;            // x + res, or nullptr
  uint16_t *Y;            // or nullptr
  uint8_t *codes;         // MXFP8 of Y, or nullptr
  uint8_t *scales;
};

struct BwdParams {
  const uint16_t *dY;
  const uint16_t *H;
  const uint16_t *w;
  const uint16_t *dH;     // gradient that reaches h past the norm, or nullptr
  int64_t M;
  int D;
  float eps;
  uint16_t *dX;
  float *dw_part;         // [gridDim.x][D] partial sums of dW, or nullptr
};

// Elements 8 v .. 8 v + 7 of a row (zero past D).
__device__ __forceinline__ u32x4_t load_vec(const uint16_t *row, int v, int D) {
  if (8 * v + 8 <= D) return *reinterpret_cast<const u32x4_a2_t *>(row + 8 * v);
  u32x4_t r = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (8 * v + e < D) r[e >> 1] |= (uint32_t)row[8 * v + e] << (16 * (e & 1));
  return r;
}

__device__ __forceinline__ void store_vec(uint16_t *row, int v, int D, u32x4_t x) {
  if (8 * v + 8 <= D) {
    *reinterpret_cast<u32x4_a2_t *>(row + 8 * v) = x;
    return;
  }
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (8 * v + e < D) row[8 * v + e] = (uint16_t)(x[e >> 1] >> (16 * (e & 1)));
}

__device__ __forceinline__ float lo_f32(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f32(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Sums of a and b over a row's threads: a wave (WAVE), or the block, through
// `red`, one of two LDS buffers used in turn, so that one barrier is enough.
template <bool WAVE>
__device__ __forceinline__ void row_sum2(float &a, float &b, float (*red)[2]) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (!WAVE) {
    if ((threadIdx.x & 63) == 0) {
      red[threadIdx.x >> 6][0] = a;
      red[threadIdx.x >> 6][1] = b;
    }
    __syncthreads();
    a = 0.0f;
    b = 0.0f;
    const int waves = blockDim.x >> 6;
    for (int i = 0; i < waves; ++i) {
      a += red[i][0];
      b += red[i][1];
    }
  }
}

constexpr int WAVE_ROWS = 4;   // rows per block of 256 threads (WAVE)
constexpr int MAX_WAVES = 16;

// Rows blockIdx.x * RPB + .., in steps of gridDim.x * RPB (as the backward).
template <bool WAVE, int VPT, bool MX>
__global__ __launch_bounds__(WAVE ? 64 * WAVE_ROWS : 64 * MAX_WAVES) void k_rmsnorm_fwd(FwdParams p) {
  __shared__ float red[2][MAX_WAVES][2];
  constexpr int RPB = WAVE ? WAVE_ROWS : 1;
  const int tid = WAVE ? threadIdx.x & 63 : threadIdx.x, sub = WAVE ? threadIdx.x >> 6 : 0;
  const int TPR = WAVE ? 64 : blockDim.x;
  const int D = p.D;
  u32x4_t wv[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = tid + j * TPR;
    wv[j] = u32x4_t{0u, 0u, 0u, 0u};
    if (8 * v < D) wv[j] = load_vec(p.w, v, D);
  }
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPB + sub; row < p.M; row += (int64_t)gridDim.x * RPB) {
    const uint16_t *x = p.X + row * D;
    u32x4_t xv[VPT], rv[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = tid + j * TPR;
      xv[j] = u32x4_t{0u, 0u, 0u, 0u};
      if (8 * v < D) xv[j] = load_vec(x, v, D);
    }
    if (p.R) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = tid + j * TPR;
        rv[j] = u32x4_t{0u, 0u, 0u, 0u};
        if (8 * v < D) rv[j] = load_vec(p.R + row * D, v, D);
      }
    }
    float h[VPT][8];
    float ss = 0.0f, none = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[j][2 * e] = lo_f32(xv[j][e]);
        h[j][2 * e + 1] = hi_f32(xv[j][e]);
        if (p.R) {
          h[j][2 * e] += lo_f32(rv[j][e]);
          h[j][2 * e + 1] += hi_f32(rv[j][e]);
        }
        ss += h[j][2 * e] * h[j][2 * e] + h[j][2 * e + 1] * h[j][2 * e + 1];
      }
    // (H may be X or R itself: this thread has read all it writes)
    if (p.H) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = tid + j * TPR;
        if (8 * v < D)
          store_vec(p.H + row * D, v, D,
                    u32x4_t{pack_bf16x2(h[j][0], h[j][1]), pack_bf16x2(h[j][2], h[j][3]),
                            pack_bf16x2(h[j][4], h[j][5]), pack_bf16x2(h[j][6], h[j][7])});
      }
    }
    row_sum2<WAVE>(ss, none, red[turn]);
    turn ^= 1;
    const float rstd = 1.0f / sqrtf(ss / (float)D + p.eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = tid + j * TPR;
      u32x4_t y;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        y[e] = pack_bf16x2(h[j][2 * e] * rstd * lo_f32(wv[j][e]), h[j][2 * e + 1] * rstd * hi_f32(wv[j][e]));
      if (p.Y && 8 * v < D) store_vec(p.Y + row * D, v, D, y);
      if constexpr (MX) {
        // D % 32 == 0: the four lanes of a quad hold one 32-element block, or
        // none of them does
        uint32_t a = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) a = max(a, max(y[e] & 0x7FFFu, (y[e] >> 16) & 0x7FFFu));
        a = max(a, (uint32_t)__shfl_xor((int)a, 1));
        a = max(a, (uint32_t)__shfl_xor((int)a, 2));
        const int Xe = mx::mx8_exponent(a);
        const float scale = __uint_as_float((uint32_t)(127 - Xe) << 23);   // 2^-Xe
        if (8 * v < D) {
          *reinterpret_cast<u32x2_t *>(p.codes + row * D + 8 * v) =
              u32x2_t{mx::mx8_code2(y[0], scale) | (mx::mx8_code2(y[1], scale) << 16),
                      mx::mx8_code2(y[2], scale) | (mx::mx8_code2(y[3], scale) << 16)};
          if ((v & 3) == 0) p.scales[row * (D >> 5) + (v >> 2)] = (uint8_t)(Xe + 127);
        }
      }
    }
  }
}

// Rows blockIdx.x * RPB + .., in steps of gridDim.x * RPB. With DW each thread
// keeps the sums of its columns over the block's rows in registers and writes
// them out once (dw_part, RPB rows of partials per block), summed in a fixed
// order by k_col_sum; there are few blocks then (their partials cost traffic),
// and in blocks of up to four waves the next row's loads are issued before a
// row is worked on (two register sets in turn), so that a block keeps memory
// busy over its reductions; wider blocks rather share a CU. MAXW: waves of the
// largest block this instantiation runs with.
//
// Loads and whole-vector stores go through a buffer descriptor of the row, so
// that lanes past its end need no branch (one after a load makes it wait).
// EDGE (D % 8 != 0): rows of one block are a multiple of 8 apart (or there is
// one), so that the shift of their aligned vectors, and with it a thread's
// columns, are the same for all; the neighbouring rows' elements in the first
// and the last vector are masked out and not written. (The widest of these with
// dW, blocks of 16 waves, spills 37 registers: 128 are all that 16 waves leave.)
template <bool WAVE, int VPT, bool DW, int MAXW, bool EDGE>
__global__ __launch_bounds__(WAVE ? 64 * WAVE_ROWS : 64 * MAXW) void k_rmsnorm_bwd(BwdParams p) {
  __shared__ float red[2][MAX_WAVES][2];
  constexpr int RPB = WAVE ? WAVE_ROWS : 1;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tid = WAVE ? threadIdx.x & 63 : threadIdx.x, sub = WAVE ? wave : 0;
  const int TPR = WAVE ? 64 : blockDim.x;
  const int D = p.D;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + sub;
  // elements from the aligned vector's start to the row's: this thread's vector
  // j holds columns c0[j] .. + 7, at byte 16 (tid + j TPR) of the row's vectors
  const int shift = EDGE ? (int)((row * D) & 7) : 0;
  const uint32_t bytes = (uint32_t)((shift + D) * 2 + 3) & ~3u;
  int c0[VPT];
  u32x4_t wv[VPT], mask[EDGE ? VPT : 1];
  float dw[DW ? VPT : 1][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    c0[j] = 8 * (tid + j * TPR) - shift;
    wv[j] = u32x4_t{0u, 0u, 0u, 0u};
    if (c0[j] >= 0 && c0[j] + 8 <= D) wv[j] = *reinterpret_cast<const u32x4_a2_t *>(p.w + c0[j]);
    if constexpr (EDGE) {
      mask[j] = u32x4_t{~0u, ~0u, ~0u, ~0u};
      if (c0[j] < 0 || c0[j] + 8 > D) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (c0[j] + e >= 0 && c0[j] + e < D) wv[j][e >> 1] |= (uint32_t)p.w[c0[j] + e] << (16 * (e & 1));
          else mask[j][e >> 1] &= 0xFFFF0000u >> (16 * (e & 1));
        }
      }
    }
    if constexpr (DW)
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
  }
  struct Row {
    u32x4_t h[VPT], y[VPT], g[VPT];
  };
  auto load = [&](Row &r, int64_t row) {
    const int64_t at = row * D - shift;
    const big::rsrc_t hs = big::make_rsrc(p.H + at, bytes), ys = big::make_rsrc(p.dY + at, bytes);
    const big::rsrc_t gs = big::make_rsrc(p.dH ? p.dH + at : p.H, p.dH ? bytes : 0u);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const uint32_t off = 16u * (tid + j * TPR);
      r.h[j] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(hs, off, 0, 0));
      r.y[j] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(ys, off, 0, 0));
      r.g[j] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(gs, off, 0, 0));
    }
  };
  int turn = 0;
  auto work = [&](Row &r, int64_t row) {
    float ss = 0.0f, st = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (EDGE) {
          r.h[j][e] &= mask[j][e];
          r.y[j][e] &= mask[j][e];
        }
        const float h0 = lo_f32(r.h[j][e]), h1 = hi_f32(r.h[j][e]);
        ss += h0 * h0 + h1 * h1;
        st += lo_f32(r.y[j][e]) * lo_f32(wv[j][e]) * h0 + hi_f32(r.y[j][e]) * hi_f32(wv[j][e]) * h1;
      }
    row_sum2<WAVE>(ss, st, red[turn]);
    turn ^= 1;
    const float rstd = 1.0f / sqrtf(ss / (float)D + p.eps);
    const float c = st / (float)D * rstd * rstd;   // mean(t n) rstd
    const big::rsrc_t os = big::make_rsrc(p.dX + (row * D - shift), bytes);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      u32x4_t o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float h0 = lo_f32(r.h[j][e]), h1 = hi_f32(r.h[j][e]);
        const float y0 = lo_f32(r.y[j][e]), y1 = hi_f32(r.y[j][e]);
        const float d0 = rstd * (y0 * lo_f32(wv[j][e]) - h0 * c) + lo_f32(r.g[j][e]);
        const float d1 = rstd * (y1 * hi_f32(wv[j][e]) - h1 * c) + hi_f32(r.g[j][e]);
        o[e] = pack_bf16x2(d0, d1);
        if constexpr (DW) {
          dw[j][2 * e] += y0 * (h0 * rstd);
          dw[j][2 * e + 1] += y1 * (h1 * rstd);
        }
      }
      const bool whole = !EDGE || (c0[j] >= 0 && c0[j] + 8 <= D);
      __builtin_amdgcn_raw_buffer_store_b128(o, os, whole ? 16u * (tid + j * TPR) : big::OOB, 0, 0);
      if constexpr (EDGE) {
        if (!whole) {
          uint16_t *dst = p.dX + row * D + c0[j];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c0[j] + e >= 0 && c0[j] + e < D) dst[e] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
  };
  if constexpr (DW && (WAVE || MAXW <= 4)) {
    Row a, b;
    if (row < p.M) load(a, row);
    while (row < p.M) {
      const int64_t next = row + step;
      if (next < p.M) load(b, next);
      work(a, row);
      if (next >= p.M) break;
      row = next + step;
      if (row < p.M) load(a, row);
      work(b, next);
    }
  } else {
    for (; row < p.M; row += step) {
      Row a;
      load(a, row);
      work(a, row);
    }
  }
  if constexpr (DW) {
    float *dst = p.dw_part + ((int64_t)blockIdx.x * RPB + sub) * D;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c0[j] + e >= 0 && c0[j] + e < D) dst[c0[j] + e] = dw[j][e];
  }
}

// out[c] = bf16(sum over i < n of part[i][c]), c < D: 32 columns per block,
// 32 threads to a column (thread q of them sums rows q, q + 32, ..), joined in
// LDS in a fixed order. One block per 32 columns and z (z: independent sums,
// part + z * n * D, out + z * D).
static __global__ __launch_bounds__(1024) void k_col_sum(const float *part, int n, int D, uint16_t *out) {
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  part += (int64_t)blockIdx.y * n * D;
  float a = 0.0f;
  if (col < D) {
    int i = q;
    for (; i + 7 * 32 < n; i += 8 * 32) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = part[(int64_t)(i + 32 * u) * D + col];
#pragma unroll
      for (int u = 0; u < 8; ++u) a += v[u];
    }
    for (; i < n; i += 32) a += part[(int64_t)i * D + col];
  }
  s[q][c] = a;
  __syncthreads();
  if (q == 0 && col < D) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][c];
    out[(int64_t)blockIdx.y * D + col] = to_bf16(t);
  }
}

}  // namespace norm
}  // namespace lora4
