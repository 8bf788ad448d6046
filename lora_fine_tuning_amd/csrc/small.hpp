// The base product for few tokens (single-token decoding, small serving
// batches, experts with a few rows each):
//
//   P = X deq(W)^T + (s Z) B^T for up to XT (4 or 8) tokens of a group,
//   with the gated or the fused epilogue (fwd::Epi).
//
// Bound: reading the packed base once (about half a byte per element; at one
// token 2 flops per element), and for NF4 the decode (3.5 VALU instructions
// per element and lane). A workgroup owns 16 columns (gated: the same 16 of
// gate and up) and all its NW waves split the reduction among them, so that
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
//    of every lane;
//  * the chunk of X, XT rows of 256 bytes, takes XT / 4 load instructions of
//    one 16-byte piece per lane, and goes through the wave's own LDS into the
//    operand layout. (Loading each lane's operand straight from memory takes
//    four instructions of duplicates and 16 registers per chunk in flight;
//    with these 4 to 8, a wave needs at most 128 registers and four of them
//    share a SIMD.)
//
// PF register sets of a chunk's codes, scales and X are in flight. Token rows
// past the group's last repeat its last row (their results are not stored).
//
// Measured (MI355X), one token: gated 4096 -> 2 x 14336 NF4 22 us (3.0 TB/s;
// the VALU is busy 13 us of it, and of the 896 workgroups some CUs have 4 and
// others 3), MXFP4 14 us (4.5 TB/s), 8192 -> 2 x 28672 48 us (5.2 TB/s); one
// projection, 14336 -> 4096 NVFP4, 4 tokens, 13 us (2.5 TB/s: as many bytes of X
// as of codes). k_small_z in front of each takes 4 us.
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
  const float *zpart;     // [zsplits][M, P r] partial sums of Z
  int zsplits;
  float s;
  uint16_t *Z;            // [M, P r] bf16 output (of the blocks of columns 0 ..), or nullptr
  const uint16_t *B;      // [groups P][N, r]
  int act;
  uint16_t *out;          // [M, N]
  uint16_t *pre;          // gated: [M, 2 N]; fused: [M, N]; or nullptr
  const uint16_t *bias;   // fused: [groups][N] or nullptr
  const uint16_t *residual;   // fused: [M, N] or nullptr
  int nblocks;            // blocks of 16 columns; block b: slot b / nblocks
  Nf4Table tab;
};

// ---------------------------------------------------------------------------
// Z = X A^T for few tokens: one workgroup per 16 tokens x 16 rank columns x
// one of `splits` ranges of the reduction, its four waves taking 32-wide chunks
// in turn, joined in LDS. The consumer adds the ranges' fp32 sums up, so a long
// reduction costs one pass of loads instead of many in a row: 3 to 4 us, which
// is a launch and two memory latencies (24 tokens, 8192 -> 128 columns: 6 us).
// ---------------------------------------------------------------------------

struct ZParams {
  const uint16_t *X;      // [M, K]
  const uint16_t *A;      // [groups][R, K]
  int64_t M, K;
  int R;                  // rank columns (P r)
  const int64_t *offsets;
  int groups;
  float *part;            // [splits][M, R]
  int jblocks, splits;    // block b: range b % splits, rank block b / splits % jblocks, then the slot
  int64_t per;            // chunks per range
};

constexpr int Z_WAVES = 4;
constexpr int Z_CHUNKS = 8;   // chunks a wave has in flight

static __global__ __launch_bounds__(64 * Z_WAVES) void k_small_z(ZParams p) {
  __shared__ f32x4_t red[Z_WAVES][64];
  const int split = blockIdx.x % p.splits, rest = blockIdx.x / p.splits;
  const RowTile rt = map_row_tile_wave(rest / p.jblocks, 16, p.offsets, p.groups, p.M);
  if (rt.group < 0) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 15, q = lane >> 4;
  const int j0 = (rest % p.jblocks) * 16;
  const int64_t last = min(rt.row0 + 16, rt.row_end) - 1;
  const int64_t tok = min(rt.row0 + lr, last);
  const uint16_t *x = p.X + tok * p.K + 8 * q;
  const uint16_t *a = p.A + ((int64_t)rt.group * p.R + min(j0 + lr, p.R - 1)) * p.K + 8 * q;
  const int64_t all = p.K >> 5;   // (K % 32 == 0)
  const int64_t end = min((split + 1) * p.per, all);
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int64_t c = split * p.per + wave; c < end; c += Z_CHUNKS * Z_WAVES) {
    u32x4_t av[Z_CHUNKS], xv[Z_CHUNKS];
#pragma unroll
    for (int u = 0; u < Z_CHUNKS; ++u)
      if (c + u * Z_WAVES < end) {
        av[u] = *reinterpret_cast<const u32x4_t *>(a + (c + u * Z_WAVES) * 32);
        xv[u] = *reinterpret_cast<const u32x4_t *>(x + (c + u * Z_WAVES) * 32);
      }
#pragma unroll
    for (int u = 0; u < Z_CHUNKS; ++u)
      if (c + u * Z_WAVES < end) acc = mfma_16x16x32(av[u], xv[u], acc);
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (threadIdx.x < 64) {
    f32x4_t z = red[0][lane];
#pragma unroll
    for (int w = 1; w < Z_WAVES; ++w) z += red[w][lane];
    // lane: rank columns j0 + 4 q + e of token lr
    if (rt.row0 + lr <= last) {
      float *dst = p.part + ((int64_t)split * p.M + rt.row0 + lr) * p.R;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j0 + 4 * q + e < p.R) dst[j0 + 4 * q + e] = z[e];
    }
  }
}

// ---------------------------------------------------------------------------
// The base product
// ---------------------------------------------------------------------------

__host__ __device__ constexpr int lds_bytes(int P, int XT, int NW) { return NW * (P * 64 * 16 + XT * 256); }

template <int FMT, int EPI, int XT, int NW>
__global__ __launch_bounds__(64 * NW, 4) void k_small(Params p) {
  constexpr int P = EPI == fwd::EPI_GATED ? 2 : 1;
  constexpr int PF = P == 2 ? 3 : 4;   // chunks in flight (one more or fewer: within 3%)
  constexpr int XL = XT / 4;   // X loads per chunk
  extern __shared__ __attribute__((aligned(16))) f32x4_t lds[];   // [NW][P][64] sums, then [NW][XT][16] X pieces
  // Blocks go to the XCDs in turn: the four column blocks of one 64-row block
  // of the storage are taken by blocks of one XCD, so that the lines of scales
  // they share (and the codes' memory pages) are fetched by one L2.
  int b = blockIdx.x;
  const int whole = (int)(gridDim.x & ~31u);
  if (b < whole) b = (b & ~31) + ((b & 7) << 2) + ((b >> 3) & 3);
  const RowTile rt = map_row_tile_wave(b / p.nblocks, XT, p.offsets, p.groups, p.M);
  if (rt.group < 0) return;
  const int g = rt.group;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int lr = lane & 15, q = lane >> 4;
  const int64_t n0 = (int64_t)(b % p.nblocks) * 16;
  const int rows = (int)min(rt.row_end - rt.row0, (int64_t)XT);
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
  // piece (kk, token, q) of the chunk is the 16 bytes at element 64 (q % 2) +
  // 32 (q / 2) + 8 kk of the token: load u of lane l takes piece number
  // 64 u + l = (kk XT + token) 4 + q, and so it lies in LDS
  uint32_t x_off[XL];
  int x_k[XL];
#pragma unroll
  for (int u = 0; u < XL; ++u) {
    const int id = 64 * u + lane, pq = id & 3, tok = (id >> 2) % XT, kk = id / (4 * XT);
    x_k[u] = 64 * (pq & 1) + 32 * (pq >> 1) + 8 * kk;
    x_off[u] = (uint32_t)((min(tok, rows - 1) * p.K + x_k[u]) * 2);
  }
  f32x4_t *red = lds;
  u32x4_t *xs = reinterpret_cast<u32x4_t *>(lds + NW * P * 64) + wave * (XT * 16);
  const u32x4_t *x_rd = xs + (lr < XT ? lr : XT - 1) * 4 + q;   // operand kk at x_rd[kk * 4 XT]

  struct Set {
    u32x4_t c[P];
    uint32_t sc[P], c2[P];
    u32x4_t x[XL];
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
    for (int u = 0; u < XL; ++u)
      s.x[u] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                               x_rs, chunk * 128 + x_k[u] < K ? x_off[u] : OOB, chunk * 256, 0));
  };

  const uint32_t sel = big::sel_base();
  float qh[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) qh[i] = (lane >> 5) ? p.tab.q[8 + i] : p.tab.q[i];
  f32x4_t acc[P];
#pragma unroll
  for (int j = 0; j < P; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto compute = [&](const Set &s) {
    // (a wave's LDS accesses run in order: the last chunk's reads are done)
#pragma unroll
    for (int u = 0; u < XL; ++u) xs[64 * u + lane] = s.x[u];
    u32x4_t x[4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) x[kk] = x_rd[kk * 4 * XT];
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
      for (int kk = 0; kk < 4; ++kk) acc[j] = mfma_16x16x32(w[kk], x[kk], acc[j]);
    }
  };

  // ---- rank-r product: 32 rank columns per step, the steps dealt to the waves.
  // (Before the base's loads are issued: among them it costs 30 registers
  // more than there are, and its own latency is hidden by the other waves.)
  for (int j0 = 32 * wave; j0 < p.r; j0 += 32 * NW) {
    const int jr = j0 + 8 * q;
    const bool vec = (p.r & 7) == 0;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int64_t n = n0 + lr;
      u32x4_t b = {0u, 0u, 0u, 0u};
      if (n < p.N && jr < p.r) {
        const uint16_t *src = p.B + (((int64_t)g * P + j) * p.N + n) * p.r + jr;
        if (vec) {
          b = *reinterpret_cast<const u32x4_t *>(src);
        } else {
          for (int e = 0; e < 8; ++e)
            if (jr + e < p.r) b[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
        }
      }
      // eight columns of this lane's token: the ranges added up in order
      const int64_t row = rt.row0 + min(lr, rows - 1);
      float z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = 0.0f;
      if (jr < p.r) {
        const float *src = p.zpart + row * (P * p.r) + j * p.r + jr;
        const int64_t stride = p.M * (P * p.r);
        if (vec) {
#pragma unroll 4
          for (int k = 0; k < p.zsplits; ++k) {
            const f32x4_t lo = *reinterpret_cast<const f32x4_t *>(src + k * stride);
            const f32x4_t hi = *reinterpret_cast<const f32x4_t *>(src + k * stride + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              z[e] += lo[e];
              z[4 + e] += hi[e];
            }
          }
        } else {
          for (int k = 0; k < p.zsplits; ++k)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (jr + e < p.r) z[e] += src[k * stride + e];
        }
        if (p.Z && n0 == 0 && lr < rows) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (jr + e < p.r) p.Z[row * (P * p.r) + j * p.r + jr + e] = to_bf16(z[e]);
        }
      }
      acc[j] = mfma_16x16x32(b, big::pack_scaled8(z, p.s), acc[j]);
    }
  }
  asm volatile("" ::: "memory");

  const int chunks = (K + 127) >> 7;
  const int n_own = chunks > wave ? (chunks - wave + NW - 1) / NW : 0;   // chunks wave, wave + NW, ..
  Set set[PF];
#pragma unroll
  for (int u = 0; u < PF; ++u) {
    load(set[u], wave + u * NW);
    __builtin_amdgcn_sched_barrier(0);   // (the waits count loads in this order)
  }
  // (the groups of PF chunks run without conditions, so that every wait in
  // them counts exactly the loads behind it; loads past the last chunk are out
  // of range and return zeros)
  int i = 0;
  for (; i + PF <= n_own; i += PF) {
#pragma unroll
    for (int u = 0; u < PF; ++u) {
      compute(set[u]);
      load(set[u], wave + (i + u + PF) * NW);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int u = 0; u < PF; ++u)
    if (i + u < n_own) compute(set[u]);

  // ---- join the waves; a thread has 4 consecutive columns of one token ---------
#pragma unroll
  for (int j = 0; j < P; ++j) red[(wave * P + j) * 64 + lane] = acc[j];
  __syncthreads();
  if (threadIdx.x < 64) {
    f32x4_t v[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      v[j] = red[j * 64 + lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) v[j] += red[(w * P + j) * 64 + lane];
    }
    const int tok = lr;
    const int64_t n = n0 + 4 * q;
    if (tok >= rows || n >= p.N) return;
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
