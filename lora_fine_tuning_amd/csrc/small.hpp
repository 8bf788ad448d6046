// The base product for few tokens (single-token decoding, small serving
// batches, experts with a handful of rows each):
//
//   P = X deq(W)^T + (s Z) B^T for up to 16 MT tokens of a group,
//   with the gated or the fused epilogue (fwd::Epi).
//
// Bound: reading the packed base once (about half a byte per element; at one
// token 2 flops per element). A workgroup owns 16 columns (gated: the same 16
// of gate and up) and all its NW waves split the reduction among them, so that
// the base's bytes are spread over thousands of waves, each with several
// 16-byte loads per lane in flight, and no partial sums leave the workgroup
// (the waves' sums are joined in LDS). A wave takes chunks of 128 elements
// (two 64 x 64 tiles of the storage) in turn with the others:
//
//  * lane l holds row l % 16 of the block and, with q = l / 16, elements
//    64 (q % 2) + 32 (q / 2) .. +31 of the chunk: 16 bytes of codes under one
//    NF4 scale (one MXFP4 scale, two NVFP4 scales), so a load instruction
//    reads two whole 512-byte pieces of the storage, and lanes l and l + 32
//    share a run, hence half an NF4 table each (big::make_table_pair);
//  * the codes decode straight into MFMA operands: the 32 elements are four
//    operands of v_mfma_f32_16x16x32_bf16 in the reduction order 8 kk + ..
//    of every lane, and the tokens' X (second operand) is read in that order.
//
// PF register sets of a chunk's codes, scales and X are in flight. Token rows
// past the group's last repeat its last row (their results are not stored).
#pragma once

#include "gemm_fwd.hpp"

namespace lora4 {
namespace small {

using big::OOB;
using big::rsrc_t;

struct Params {
  PackedW W;              // groups: P per row group (P = 2: gate, up)
  const uint16_t *X;      // [M, K]
  int64_t M, K, N;
  const int64_t *offsets;
  int groups;             // row groups
  int r;
  const uint16_t *sZ;     // [M, P r] bf16, s Z
  const uint16_t *B;      // [groups P][N, r]
  int act;
  uint16_t *out;          // [M, N]
  uint16_t *pre;          // gated: [M, 2 N]; fused: [M, N]; or nullptr
  const uint16_t *bias;   // fused: [groups][N] or nullptr
  const uint16_t *residual;   // fused: [M, N] or nullptr
  int nblocks;            // blocks of 16 columns; block b: slot b / nblocks
  Nf4Table tab;
};

// As map_row_tile, with the 64 lanes of a wave looking through 64 groups at a
// time (a grid of few-token slots runs over every expert).
__device__ __forceinline__ RowTile map_row_tile_wave(int slot, int BM, const int64_t *offsets, int groups,
                                                     int64_t M) {
  if (offsets == nullptr) return map_row_tile(slot, BM, nullptr, 1, M);
  RowTile t{-1, 0, 0};
  const int lane = threadIdx.x & 63;
  int64_t base = 0;   // slots of the groups before e0
  for (int e0 = 0; e0 < groups; e0 += 64) {
    const int e = e0 + lane;
    int64_t a = 0, b = 0;
    if (e < groups) {
      a = offsets[e];
      b = offsets[e + 1];
    }
    const int nt = (int)((b - a + BM - 1) / BM);
    int incl = nt;   // inclusive prefix sum over the lanes
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o);
      if (lane >= o) incl += v;
    }
    const int64_t first = base + incl - nt;
    const unsigned long long hit = __ballot(slot >= first && slot < first + nt);
    if (hit) {
      const int src = __ffsll(hit) - 1;
      t.group = e0 + src;
      const int s = __shfl((int)(slot - first), src);
      t.row0 = __shfl((long long)a, src) + (int64_t)s * BM;
      t.row_end = __shfl((long long)b, src);
      return t;
    }
    base += __shfl(incl, 63);
  }
  return t;
}

// ---------------------------------------------------------------------------
// Z = X A^T for few tokens: one workgroup per 16 tokens x 16 rank columns, its
// 16 waves taking 32-wide chunks of the reduction in turn, joined in LDS.
// ---------------------------------------------------------------------------

struct ZParams {
  const uint16_t *X;      // [M, K]
  const uint16_t *A;      // [groups][R, K]
  int64_t M, K;
  int R;                  // rank columns (P r)
  float s;
  const int64_t *offsets;
  int groups;
  uint16_t *sZ;           // [M, R] bf16(s Z)
  uint16_t *Z;            // [M, R] bf16(Z) or nullptr
  int jblocks;            // blocks of 16 rank columns; block b: slot b / jblocks
};

constexpr int Z_WAVES = 16;

static __global__ __launch_bounds__(64 * Z_WAVES) void k_small_z(ZParams p) {
  __shared__ f32x4_t red[Z_WAVES][64];
  const RowTile rt = map_row_tile_wave(blockIdx.x / p.jblocks, 16, p.offsets, p.groups, p.M);
  if (rt.group < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 15, q = lane >> 4;
  const int j0 = (blockIdx.x % p.jblocks) * 16;
  const int64_t last = min(rt.row0 + 16, rt.row_end) - 1;
  const int64_t tok = min(rt.row0 + lr, last);
  const uint16_t *x = p.X + tok * p.K + 8 * q;
  const uint16_t *a = p.A + ((int64_t)rt.group * p.R + min(j0 + lr, p.R - 1)) * p.K + 8 * q;
  const int64_t chunks = p.K >> 5;   // (K % 32 == 0)
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  constexpr int U = 8;
  int64_t c = wave;
  for (; c + (U - 1) * Z_WAVES < chunks; c += U * Z_WAVES) {
    u32x4_t av[U], xv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      av[u] = *reinterpret_cast<const u32x4_t *>(a + (c + u * Z_WAVES) * 32);
      xv[u] = *reinterpret_cast<const u32x4_t *>(x + (c + u * Z_WAVES) * 32);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) acc = mfma_16x16x32(av[u], xv[u], acc);
  }
  {
    u32x4_t av[U], xv[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c + u * Z_WAVES < chunks) {
        av[u] = *reinterpret_cast<const u32x4_t *>(a + (c + u * Z_WAVES) * 32);
        xv[u] = *reinterpret_cast<const u32x4_t *>(x + (c + u * Z_WAVES) * 32);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c + u * Z_WAVES < chunks) acc = mfma_16x16x32(av[u], xv[u], acc);
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (threadIdx.x < 64) {
    f32x4_t z = red[0][lane];
#pragma unroll
    for (int w = 1; w < Z_WAVES; ++w) z += red[w][lane];
    // lane: rank columns j0 + 4 q + e of token lr
    if (rt.row0 + lr <= last) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = j0 + 4 * q + e;
        if (j < p.R) {
          p.sZ[(rt.row0 + lr) * p.R + j] = to_bf16(z[e] * p.s);
          if (p.Z) p.Z[(rt.row0 + lr) * p.R + j] = to_bf16(z[e]);
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The base product
// ---------------------------------------------------------------------------

__host__ __device__ constexpr int lds_bytes(int P, int MT, int NW) { return NW * P * MT * 64 * 16; }

template <int FMT, int EPI, int MT, int NW>
__global__ __launch_bounds__(64 * NW) void k_small(Params p) {
  constexpr int P = EPI == fwd::EPI_GATED ? 2 : 1;
  constexpr int PF = MT == 1 ? 4 : MT == 2 ? 3 : 2;   // chunks in flight
  extern __shared__ __attribute__((aligned(16))) f32x4_t red[];   // [NW][P][MT][64]
  const RowTile rt = map_row_tile_wave(blockIdx.x / p.nblocks, 16 * MT, p.offsets, p.groups, p.M);
  if (rt.group < 0) return;
  const int g = rt.group;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int lr = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)(blockIdx.x % p.nblocks) * 16;
  const int rows = (int)min(rt.row_end - rt.row0, (int64_t)16 * MT);
  const int64_t KB = p.W.KB;
  const int K = (int)p.K;

  // ---- the base: row n0 + lr (a padding row past N reads zeros) --------------
  constexpr int sc_bytes = FMT == FMT_NF4 ? 4 : 1;
  constexpr int sc_tile = FMT == FMT_MXFP4 ? 128 : FMT == FMT_NVFP4 ? 256 : 64 * sc_bytes;
  const int64_t rb = n0 >> 6;
  const int i0 = (int)(n0 & 63) + lr;
  rsrc_t w_rs[P], s_rs[P], s2_rs[P];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int64_t gw = (int64_t)g * P + j;
    w_rs[j] = big::make_rsrc(p.W.codes + gw * p.W.g_codes + rb * KB * 2048, big::clamp_bytes(KB * 2048));
    s_rs[j] = big::make_rsrc(reinterpret_cast<const uint8_t *>(p.W.scales) + gw * p.W.g_scales * sc_bytes +
                                 rb * KB * sc_tile,
                             big::clamp_bytes(KB * sc_tile));
    s2_rs[j] = FMT == FMT_NF4_DQ ? big::make_rsrc(p.W.scales2 + gw * p.W.g_scales2,
                                                  big::clamp_bytes(p.W.g_scales2 * 4))
                                 : w_rs[j];
  }
  const uint32_t c_off = (uint32_t)((q & 1) * 2048 + i0 * 32 + (q >> 1) * 16);
  const uint32_t s_off =
      (uint32_t)((q & 1) * sc_tile + (FMT == FMT_MXFP4   ? i0 * 2 + (q >> 1)
                                      : FMT == FMT_NVFP4 ? i0 * 4 + (q >> 1) * 2
                                                         : i0 * sc_bytes));
  const int64_t s2_row = (n0 + lr) * (p.K >> 6) + (q & 1);
  const int k_lane = 64 * (q & 1) + 32 * (q >> 1);   // first element within a chunk

  // ---- tokens -----------------------------------------------------------------
  const rsrc_t x_rs = big::make_rsrc(p.X + rt.row0 * p.K, big::clamp_bytes((int64_t)rows * p.K * 2));
  uint32_t x_off[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) x_off[m] = (uint32_t)((min(16 * m + lr, rows - 1) * p.K + k_lane) * 2);

  struct Set {
    u32x4_t c[P];
    uint32_t sc[P], c2[P];
    u32x4_t x[MT][4];
  };
  // (a lane whose 32 elements lie past K loads zeros, base and tokens)
  auto load = [&](Set &s, int chunk) {
    const bool in = chunk * 128 + k_lane < K;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      s.c[j] = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(w_rs[j], in ? c_off : OOB, chunk * 4096, 0));
      const int so = chunk * 2 * sc_tile;
      if constexpr (FMT == FMT_NF4) {
        s.sc[j] = __builtin_amdgcn_raw_buffer_load_b32(s_rs[j], in ? s_off : OOB, so, 0);
      } else if constexpr (FMT == FMT_NVFP4) {
        s.sc[j] = __builtin_amdgcn_raw_buffer_load_b16(s_rs[j], in ? s_off : OOB, so, 0);
      } else {
        s.sc[j] = __builtin_amdgcn_raw_buffer_load_b8(s_rs[j], in ? s_off : OOB, so, 0);
      }
      if constexpr (FMT == FMT_NF4_DQ)
        s.c2[j] = __builtin_amdgcn_raw_buffer_load_b32(
            s2_rs[j], in ? (uint32_t)(((s2_row + 2 * chunk) >> 8) * 4) : OOB, 0, 0);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        s.x[m][kk] = __builtin_bit_cast(
            u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(x_rs, in ? x_off[m] + 16 * kk : OOB, chunk * 256, 0));
  };

  const uint32_t sel = big::sel_base();
  float qh[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) qh[i] = (lane >> 5) ? p.tab.q[8 + i] : p.tab.q[i];
  f32x4_t acc[P][MT];
#pragma unroll
  for (int j = 0; j < P; ++j)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[j][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](const Set &s) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      u32x4_t w[4];
      if constexpr (FMT == FMT_MXFP4) {
        const float sc = e8m0_to_f32(s.sc[j] & 0xFFu);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) w[kk] = big::decode8_mxfp4(s.c[j][kk], sc);
      } else if constexpr (FMT == FMT_NVFP4) {
        const float s0 = e4m3_to_f32(s.sc[j] & 0xFFu), s1 = e4m3_to_f32((s.sc[j] >> 8) & 0xFFu);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) w[kk] = decode8_nvfp4(s.c[j][kk], kk < 2 ? s0 : s1);
      } else {
        float c;
        if constexpr (FMT == FMT_NF4) c = __builtin_bit_cast(float, s.sc[j]);
        else c = e4m3_to_f32(s.sc[j] & 0xFFu) * __builtin_bit_cast(float, s.c2[j]);
        const big::RunTable T = big::make_table_pair(c, qh, sel);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) w[kk] = big::decode8_nf4(T, s.c[j][kk]);
      }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[j][m] = mfma_16x16x32(w[kk], s.x[m][kk], acc[j][m]);
    }
  };

  const int chunks = (K + 127) >> 7;
  const int n_own = chunks > wave ? (chunks - wave + NW - 1) / NW : 0;   // chunks wave, wave + NW, ..
  Set set[PF];
#pragma unroll
  for (int u = 0; u < PF; ++u) load(set[u], wave + u * NW);
  for (int i = 0; i < n_own; i += PF) {
#pragma unroll
    for (int u = 0; u < PF; ++u) {
      if (i + u < n_own) {
        compute(set[u]);
        load(set[u], wave + (i + u + PF) * NW);
      }
    }
  }

  // ---- rank-r product, 32 rank columns per step, the steps dealt to the waves
  for (int j0 = 32 * wave; j0 < p.r; j0 += 32 * NW) {
    const int jr = j0 + 8 * q;
    const bool vec = (p.r & 7) == 0;
    auto rank8 = [&](const uint16_t *src, bool ok) -> u32x4_t {   // src[0 .. 7], zero past r
      uint32_t w4[4] = {0u, 0u, 0u, 0u};
      if (ok && jr < p.r) {
        if (vec) return *reinterpret_cast<const u32x4_t *>(src);
        for (int e = 0; e < 8; ++e)
          if (jr + e < p.r) w4[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
      }
      return u32x4_t{w4[0], w4[1], w4[2], w4[3]};
    };
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int64_t n = n0 + lr;
      const u32x4_t b = rank8(p.B + (((int64_t)g * P + j) * p.N + n) * p.r + jr, n < p.N);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int64_t row = rt.row0 + min(16 * m + lr, rows - 1);
        acc[j][m] = mfma_16x16x32(b, rank8(p.sZ + row * (P * p.r) + j * p.r + jr, true), acc[j][m]);
      }
    }
  }

  // ---- join the waves; each item is 4 consecutive columns of one token --------
#pragma unroll
  for (int j = 0; j < P; ++j)
#pragma unroll
    for (int m = 0; m < MT; ++m) red[((wave * P + j) * MT + m) * 64 + lane] = acc[j][m];
  __syncthreads();
  for (int it = threadIdx.x; it < MT * 64; it += 64 * NW) {
    f32x4_t v[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      v[j] = red[j * MT * 64 + it];
#pragma unroll
      for (int w = 1; w < NW; ++w) v[j] += red[(w * P + j) * MT * 64 + it];
    }
    const int tok = 16 * (it >> 6) + (it & 15);
    const int64_t n = n0 + 4 * ((it >> 4) & 3);
    if (tok >= rows || n >= p.N) continue;
    const int64_t row = rt.row0 + tok;
    const bool vec = (p.N & 3) == 0;   // then the four columns are whole and 8-byte aligned
    auto put = [&](uint16_t *dst, const float (&o)[4]) {
      if (vec) {
        *reinterpret_cast<u32x2_t *>(dst) = u32x2_t{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < p.N) dst[e] = to_bf16(o[e]);
      }
    };
    float o[4];
    if constexpr (EPI == fwd::EPI_GATED) {
      if (p.pre) {
        const float gv[4] = {v[0][0], v[0][1], v[0][2], v[0][3]}, uv[4] = {v[1][0], v[1][1], v[1][2], v[1][3]};
        put(p.pre + row * 2 * p.N + n, gv);
        put(p.pre + row * 2 * p.N + p.N + n, uv);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = act_value(v[0][e], p.act) * v[1][e];
    } else {
      if (p.bias) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < p.N) v[0][e] += bf16_bits_to_f32(p.bias[g * p.N + n + e]);
      }
      if (p.pre) {
        const float pv[4] = {v[0][0], v[0][1], v[0][2], v[0][3]};
        put(p.pre + row * p.N + n, pv);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = act_value(v[0][e], p.act);
      if (p.residual) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < p.N) o[e] += bf16_bits_to_f32(p.residual[row * p.N + n + e]);
      }
    }
    put(p.out + row * p.N + n, o);
  }
}

}  // namespace small
}  // namespace lora4
