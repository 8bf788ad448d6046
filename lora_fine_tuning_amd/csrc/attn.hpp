// Causal attention over packed sequences with grouped heads: forward (whole
// prompts, chunks and single tokens over a cache) and backward.
//
// Per sequence with Lq queries and Lk keys, query i sees the keys
// j <= i + Lk - Lq:
//
//   S = scale Q K^T,  P = softmax of a row's visible S,  O = P V,
//   lse = log(sum exp S)
//   backward: delta = sum_d dO O,  P = exp(S - lse),  dP = dO V^T,
//   dS = P (dP - delta),  dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO
//
// Packed rows: the G = Hq / Hkv query heads of a key head are rows of one
// matrix, row i G + g for query i and head g of the group. A tile of rows
// reads its keys and values once for all heads of the group, single tokens
// over a cache fill their tiles G times better, and dK, dV are sums over rows
// that need no second pass over the heads.
//
// Products run on v_mfma_f32_32x32x16_bf16 in the transposed form: a wave
// computes S^T = K Q^T, so that a lane's 16 results of a 32 x 32 block belong
// to one row (its column lane % 32), and the softmax is lane-local but for one
// exchange between the two lane halves. Result register r of half h holds
// key 8 (r / 4) + 4 h + r % 4. As second operand of the next product
// (O^T = V^T P^T) a lane half supplies 8 keys per 16-deep step; the reduction's
// order is free, so the 16 keys of a step are taken in the order in which the
// registers hold them, and V is fetched to match: two transposing reads of
// rows 16 b + 4 h .. +3 and 16 b + 8 + 4 h .. +3. P never passes through LDS.
//
// LDS tiles of [rows][D] bf16 (rows of 128 or 256 bytes) are filled by direct
// loads, 16 bytes a lane; a row's 16-byte chunks are stored at
// chunk ^ row_swz(row), which keeps both kinds of read off each other's banks.
// Rows past a sequence's end and columns past D are out of the descriptor's
// range and read as zeros, so that nothing of another sequence (or of a cache's
// unfilled part) enters a product, NaN included.
#pragma once

#include <type_traits>

#include "common.hpp"
#include "gemm_big.hpp"

namespace lora4 {
namespace attn {

using big::rsrc_t;

constexpr int THREADS = 256;
constexpr int ROWS = 128;     // packed query rows of a forward or dQ tile (32 a wave)
constexpr int KEYS = 64;      // keys of a step of these
constexpr int BKEYS = 128;    // keys of a dK, dV tile (32 a wave)
constexpr int BROWS = 64;     // packed query rows of a step of it
constexpr uint32_t OOB = big::OOB;
constexpr float SLACK = 8.0f; // binary orders a weight may exceed 1 by (see k_attn_fwd)
constexpr float LOG2E = 1.44269504088896340736f;

struct Params {
  const uint16_t *Q, *K, *V;
  int64_t ldq, ldk, ldv;      // elements between tokens
  int64_t Tq, Tk;
  int seqs;
  int Hq, Hkv, G, D;
  uint32_t gmagic, gone;      // ceil(2^32 / G) and 0; for G == 1 0 and all ones
  float scale;
  const int64_t *qo, *ko, *kl;
  int slots;                  // row tiles (forward, dQ) or key tiles (dK, dV) of the grid
  int splits;                 // key ranges (forward) or row ranges (dK, dV) per tile
  uint16_t *O;                // [Tq][Hq][D]
  float *lse;                 // [Tq][Hq] or null
  float *part;                // splits > 1: fp32 partials
  float *part_ml;             // forward: [splits][Tq Hq][2] running maximum and sum
  // backward
  const uint16_t *dO;
  const uint16_t *Oin;        // the forward's O
  float *stat;                // [2][Tq][Hq]: lse log2 e and delta, made by k_attn_dq
  uint16_t *dQ, *dK, *dV;
  int64_t lddq, lddk, lddv;
};

// Query of packed row r, exact for r < 2^32 / G (which the host checks).
__device__ __forceinline__ uint32_t row_query(const Params &p, uint32_t r) {
  return __umulhi(r, p.gmagic) + (r & p.gone);
}

// One tile of the grid.
struct Tile {
  int64_t q0, k0;   // the sequence's first query and key
  int Lq, Lk;
  int tile;         // tile of the sequence, -1: none
};

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : x > hi ? hi : x; }

// Sequence s, its ranges held inside the tensors whatever the offsets say.
__device__ __forceinline__ void seq_range(const Params &p, int s, int64_t &q0, int64_t &Lq, int64_t &k0, int64_t &Lk) {
  if (p.qo) {
    q0 = clamp64(p.qo[s], 0, p.Tq);
    Lq = clamp64(p.qo[s + 1], q0, p.Tq) - q0;
  } else {
    q0 = 0;
    Lq = p.Tq;
  }
  if (p.ko) {
    k0 = clamp64(p.ko[s], 0, p.Tk);
    Lk = clamp64(p.ko[s + 1], k0, p.Tk) - k0;
  } else {
    k0 = 0;
    Lk = p.Tk;
  }
  if (p.kl) Lk = clamp64(p.kl[s], 0, Lk);
}

// The slot-th tile of the batch: sequences in order, each cut into tiles of
// `per` packed rows (BY_KEYS: keys). The lanes of a wave look through 64
// sequences at a time.
template <bool BY_KEYS>
__device__ __forceinline__ Tile map_tile(const Params &p, int slot, int per) {
  Tile t{0, 0, 0, 0, -1};
  const int lane = threadIdx.x & 63;
  int64_t base = 0;
  for (int s0 = 0; s0 < p.seqs; s0 += 64) {
    int64_t q0 = 0, Lq = 0, k0 = 0, Lk = 0;
    if (s0 + lane < p.seqs) seq_range(p, s0 + lane, q0, Lq, k0, Lk);
    const int nt = (int)(((BY_KEYS ? Lk : Lq * p.G) + per - 1) / per);
    int incl = nt;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(incl, o);
      if (lane >= o) incl += v;
    }
    const int64_t first = base + incl - nt;
    const unsigned long long hit = __ballot(slot >= first && slot < first + nt);
    if (hit) {
      const int src = __builtin_amdgcn_readfirstlane(__ffsll(hit) - 1);
      t.tile = __builtin_amdgcn_readfirstlane(__shfl((int)(slot - first), src));
      t.q0 = uniform64(__shfl((long long)q0, src));
      t.k0 = uniform64(__shfl((long long)k0, src));
      t.Lq = __builtin_amdgcn_readfirstlane(__shfl((int)Lq, src));
      t.Lk = __builtin_amdgcn_readfirstlane(__shfl((int)Lk, src));
      return t;
    }
    base += __shfl(incl, 63);
  }
  return t;
}

// Block -> (slot, key head, split). Consecutive blocks go to consecutive XCDs:
// with eight key heads (or a group of eight of more) a head's blocks share one
// XCD's L2, whatever their slots.
struct Job {
  int slot, head, split;
};
__device__ __forceinline__ Job map_job(const Params &p) {
  int id = blockIdx.x;
  const int hw = p.Hkv % 8 == 0 ? 8 : p.Hkv;   // heads side by side
  const int per = p.slots * p.splits * hw;
  const int g = id / per;
  id -= g * per;
  Job j;
  j.head = g * hw + id % hw;
  id /= hw;
  j.split = id % p.splits;
  j.slot = id / p.splits;
  return j;
}

// ---------------------------------------------------------------------------
// LDS tiles
// ---------------------------------------------------------------------------

// Bytes of a tile row for DC 32-element column blocks, and the swizzle. A
// 16-byte-per-lane read takes 16 lanes at a time (256 bytes, 64 banks): 16
// consecutive rows at one chunk, which land in 16 different places. A
// transposing read takes 32 lanes at a time: four consecutive rows (from a
// multiple of four) of 64 bytes, which land in the four quarters.
template <int DC>
struct Lds {
  static constexpr int CH = DC <= 2 ? 8 : 16;     // 16-byte chunks of a row
  static constexpr int RW = CH * 8;               // elements of a row
  static __device__ __forceinline__ int swz(int row) {
    return CH == 16 ? ((row & 3) << 2) | ((row >> 2) & 3) : (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
  }
  static __device__ __forceinline__ int at(int row, int chunk) { return row * RW + ((chunk ^ swz(row)) << 3); }
};

__device__ __forceinline__ void load_lds16(const rsrc_t &r, uint16_t *dst, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 16, voff, 0, 0, 0);
}

// Key or value tile: NR rows from key k of the descriptor (whose range ends with
// the sequence) into LDS. Lane l of a wave writes the l-th 16 bytes of 1 KB.
template <int DC, int NR>
__device__ __forceinline__ void load_kv(const rsrc_t &r, uint16_t *lds, int64_t ld, int D, int wave, int lane) {
  using T = Lds<DC>;
  constexpr int RPI = 64 / T::CH;          // rows of one load instruction
  constexpr int NI = NR / RPI / 4;         // instructions per wave
  const int rl = lane / T::CH, cp = lane % T::CH;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int row = (i * 4 + wave) * RPI + rl;
    const int c = cp ^ T::swz(row);
    load_lds16(r, lds + (i * 4 + wave) * 512, c * 8 < D ? (uint32_t)(row * (int)ld * 2 + c * 16) : OOB);
  }
}

// A operand of 16 reduction columns from kk * 16 of the 32 rows from row0 (the rows
// are the product's rows).
template <int DC>
__device__ __forceinline__ u32x4_t frag_rows(const uint16_t *lds, int row0, int kk, int lane) {
  return lds_read_b128(lds + Lds<DC>::at(row0 + (lane & 31), 2 * kk + (lane >> 5)));
}

// A operand of a product that reduces over the tile's rows: columns 32 db ..
// +31 as its rows, the 16 rows from row0 in the order of the result registers.
template <int DC>
__device__ __forceinline__ u32x4_t frag_cols(const uint16_t *lds, int row0, int db, int lane) {
  const int h = lane >> 5, i = lane & 15;
  const int col = db * 32 + ((lane >> 4) & 1) * 16 + (i & 3) * 4;
  const int r = row0 + 4 * h + (i >> 2);
  const u32x2_t lo = lds_read_tr16(lds + Lds<DC>::at(r, col >> 3) + (col & 7));
  const u32x2_t hi = lds_read_tr16(lds + Lds<DC>::at(r + 8, col >> 3) + (col & 7));
  return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
}

// 8 result registers (one 16-row step) as bf16 operand.
__device__ __forceinline__ u32x4_t pack8(const f32x16_t &v, int r0) {
  return u32x4_t{pack_bf16x2(v[r0], v[r0 + 1]), pack_bf16x2(v[r0 + 2], v[r0 + 3]), pack_bf16x2(v[r0 + 4], v[r0 + 5]),
                 pack_bf16x2(v[r0 + 6], v[r0 + 7])};
}

// Scheduling hints: the next `n` MFMAs, LDS reads, of the block go here. The
// compiler by itself reads each operand just before its product and waits.
template <int N>
__device__ __forceinline__ void sched_mfma() {
  __builtin_amdgcn_sched_group_barrier(0x008, N, 0);
}
template <int N>
__device__ __forceinline__ void sched_read() {
  __builtin_amdgcn_sched_group_barrier(0x100, N, 0);
}

// The values of both lane halves, lower first.
struct Halves {
  float lo, hi;
};
__device__ __forceinline__ Halves both_halves(float x) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return {__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])};
}
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// B operand straight from memory: this lane's row, 8 columns from 16 kk + 8 h.
// Columns past D take the row's first ones: the other operand is zero there. (All
// loads without a condition: a branch to each cost more than the loads.)
template <int DC>
__device__ __forceinline__ void load_row_frags(u32x4_t (&f)[2 * DC], const uint16_t *row, int D, int h) {
#pragma unroll
  for (int kk = 0; kk < 2 * DC; ++kk) {
    const int c = 16 * kk + 8 * h;
    f[kk] = ldg_b128_cached(row + (c < D ? c : 0));
  }
}

// This lane's row of a transposed result [32 DC columns][rows] times a, as bf16.
template <int DC>
__device__ __forceinline__ void store_row(uint16_t *dst, const f32x16_t (&acc)[DC], float a, int D, int h) {
#pragma unroll
  for (int db = 0; db < DC; ++db)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = db * 32 + 8 * i + 4 * h;
      if (c < D)
        *reinterpret_cast<u32x2_t *>(dst + c) =
            u32x2_t{pack_bf16x2(acc[db][4 * i] * a, acc[db][4 * i + 1] * a),
                    pack_bf16x2(acc[db][4 * i + 2] * a, acc[db][4 * i + 3] * a)};
    }
}

template <int DC>
__device__ __forceinline__ void store_row_f32(float *dst, const f32x16_t (&acc)[DC], int D, int h) {
#pragma unroll
  for (int db = 0; db < DC; ++db)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = db * 32 + 8 * i + 4 * h;
      if (c < D)
        *reinterpret_cast<f32x4_t *>(dst + c) =
            f32x4_t{acc[db][4 * i], acc[db][4 * i + 1], acc[db][4 * i + 2], acc[db][4 * i + 3]};
    }
}

// Keys or values of one head, a tile of KEYS after another, to the sequence's end
// (64-bit addresses: a cache may be longer than a descriptor's range).
struct KvStream {
  const uint16_t *at;   // first row of the next tile
  int64_t bytes;        // from there to the end
  int64_t step;         // elements per tile
  __device__ __forceinline__ KvStream(const uint16_t *X, int64_t ld, const Params &p, const Tile &t, int head, int k)
      : at(X + (t.k0 + k) * ld + head * p.D), bytes((((int64_t)t.Lk - k - 1) * ld + p.D) * 2), step(KEYS * ld) {}
  __device__ __forceinline__ rsrc_t next() {
    const rsrc_t r = big::make_rsrc(at, (uint32_t)(bytes >> 31) ? 0x7FFFFFFFu : (uint32_t)bytes);
    at += step;
    bytes -= step * 2;
    return r;
  }
};

// Runs body(step, stage) for the steps from s0, the stage (0, 1, 0, ..) a
// constant: LDS addresses of both stages are immediate offsets.
template <typename F>
__device__ __forceinline__ void two_stages(int s0, int s1, F &&body) {
  for (int s = s0; s < s1; ++s) {
    body(s, std::integral_constant<int, 0>{});
    if (++s >= s1) break;
    body(s, std::integral_constant<int, 1>{});
  }
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------

// O of a tile of 128 packed rows, 32 to a wave, over its keys, 64 to a step. Per
// row a running reference m and sum l: weights are 2^(c S - m), and m moves (O and
// l rescaled) only when a score passes it by more than SLACK binary orders.
// P is rounded to bf16 for its product with V (a weight's error of 2^-8 of itself
// is that of the values it multiplies); l is the sum of the unrounded weights. Keys
// behind a row's last are left out by a branch that only edge steps take.
//
// Bound: one token's rows, by the caches' bytes (24 tokens over 5 to 32 thousand
// keys, 64 heads: 363-373 us for 1.91 GB, 5.2 TB/s) or, over one short cache, by the
// latency of 4 steps (7 us). Long prompts, by the matrix cores at the clock the card
// holds under them: 32768 tokens, 40 heads 9.5-9.9 ms, 1110-1150 TFLOP/s, products
// in flight 59-63 % of the cycles at 1.62-1.65 GHz, no LDS bank conflicts; the rest of
// the issue is exp2, the row maxima and the packing of P. Two blocks a CU (256
// registers a wave) let one's softmax run under the other's products. LDS reads
// ahead of their products, stage offsets as constants and the lazy reference took
// this prompt from 11.2 to 9.7 ms. Packed 4096 tokens, 32 heads: 48 us for 27.4
// GFLOP, prologues and tiles of few keys.
template <int DC>
__global__ __launch_bounds__(THREADS, 2) void k_attn_fwd(Params p) {
  using T = Lds<DC>;
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];
  constexpr int TE = KEYS * T::RW;   // elements of one tile
  // K and V of two steps: K0 V0 K1 V1

  Job j = map_job(p);
  const Tile t = map_tile<false>(p, p.slots - 1 - j.slot, ROWS);   // long rows of keys first
  if (t.tile < 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int h = lane >> 5;
  const int R = t.Lq * p.G;
  const int off = t.Lk - t.Lq;

  // this lane's row
  const int r = t.tile * ROWS + wave * 32 + (lane & 31);
  const bool row_ok = r < R;
  const int qi = (int)row_query(p, (uint32_t)(row_ok ? r : R - 1));
  const int64_t oi = (t.q0 + qi) * p.Hq + j.head * p.G + ((row_ok ? r : R - 1) - qi * p.G);   // (token, head)
  u32x4_t qf[2 * DC];
  load_row_frags<DC>(qf, p.Q + (t.q0 + qi) * p.ldq + (oi - (t.q0 + qi) * p.Hq) * p.D, p.D, h);

  // keys that the block's last row sees, and that all of the wave's rows see
  const int q_hi = (int)row_query(p, (uint32_t)min(R - 1, t.tile * ROWS + ROWS - 1));
  const int q_lo = (int)row_query(p, (uint32_t)min(R - 1, t.tile * ROWS + wave * 32));
  const int kend = min(t.Lk, q_hi + off + 1);
  int nt = kend > 0 ? (kend + KEYS - 1) / KEYS : 0;
  int t0 = 0;
  if (p.splits > 1) {
    const int per = (nt + p.splits - 1) / p.splits;
    t0 = min(nt, j.split * per);
    nt = min(nt, t0 + per);
  }
  const int full = min(t.Lk, q_lo + off + 1);   // keys seen by every row of the wave

  f32x16_t acc[DC];
#pragma unroll
  for (int i = 0; i < DC; ++i) acc[i] = f32x16_t{};
  float m = -INFINITY, l[2] = {0.0f, 0.0f};
  const float c = p.scale * LOG2E;
  const int lim = qi + off;   // last key this lane's row sees

  // keys that any row of the wave sees (none where it has no rows)
  const int wr0 = t.tile * ROWS + wave * 32;
  const int wend = wr0 < R ? min(kend, (int)row_query(p, (uint32_t)min(R - 1, wr0 + 31)) + off + 1) : 0;
  KvStream ks(p.K, p.ldk, p, t, j.head, t0 * KEYS), vs(p.V, p.ldv, p, t, j.head, t0 * KEYS);
  auto issue = [&](int stage) {
    uint16_t *dst = smem + stage * 2 * TE;
    load_kv<DC, KEYS>(ks.next(), dst, p.ldk, p.D, wave, lane);
    load_kv<DC, KEYS>(vs.next(), dst + TE, p.ldv, p.D, wave, lane);
  };

  if (t0 < nt) issue(0);
  two_stages(t0, nt, [&](int s, auto stage) __attribute__((always_inline)) {
    constexpr int ST = decltype(stage)::value;
    __builtin_amdgcn_s_waitcnt(0x0F70);   // this wave's loads of step s have landed
    __syncthreads();                      // everyone's have, and step s - 1 is done with
    if (s + 1 < nt) issue(ST ^ 1);
    const uint16_t *Ks = smem + ST * 2 * TE, *Vs = Ks + TE;
    const int k0 = s * KEYS;
    if (k0 >= wend) return;   // (no row of the wave sees these keys)

    __builtin_amdgcn_s_setprio(1);   // products before the other wave's softmax (1 % of a long prompt)
    f32x16_t sc[2];
    u32x4_t vf[DC];
#pragma unroll
    for (int kk = 0; kk < 2 * DC; ++kk)
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
        sc[kb] = mfma_32x32x16(frag_rows<DC>(Ks, kb * 32, kk, lane), qf[kk], kk == 0 ? f32x16_t{} : sc[kb]);
#pragma unroll
    for (int db = 0; db < DC; ++db) vf[db] = frag_cols<DC>(Vs, 0, db, lane);
    // four reads ahead of the products, V's first operands behind the last ones
    sched_read<4>();
#pragma unroll
    for (int i = 0; i < 4 * DC - 4; ++i) {
      sched_mfma<1>();
      sched_read<1>();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sched_mfma<1>();
      sched_read<(2 * DC + 3) / 4>();
    }
    __builtin_amdgcn_s_setprio(0);
    if (k0 + KEYS > full) {
      asm volatile("");   // a branch, not 32 selects in every step
      const int lk = lim - k0 - 4 * h;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (kb * 32 + 8 * (i >> 2) + (i & 3) > lk) sc[kb][i] = -INFINITY;
    }
    float mt = sc[0][0];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) mt = fmaxf(mt, sc[kb][i]);
    const Halves mh = both_halves(mt);
    mt = fmaxf(mh.lo, mh.hi);
    // The reference m follows the running maximum only where a row's has grown by
    // more than SLACK binary orders (always in the first step): weights up to
    // 2^SLACK lose nothing in bf16 and fp32, and the rescaling is rare.
    if (__ballot((mt - m) * c > SLACK)) {
      const float mn = fmaxf(m, mt);
      const float a = mn == m ? 1.0f : exp2_hw((m - mn) * c);
#pragma unroll
      for (int i = 0; i < DC; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][e] *= a;
      l[0] *= a;
      l[1] *= a;
      m = mn;
    }
    const float mc = m == -INFINITY ? 0.0f : m * c;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float e = exp2_hw(__builtin_fmaf(sc[kb][i], c, -mc));
        sc[kb][i] = e;
        l[i & 1] += e;
      }
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const u32x4_t pf = pack8(sc[b >> 1], (b & 1) * 8);
#pragma unroll
      for (int db = 0; db < DC; ++db) {
        acc[db] = mfma_32x32x16(vf[db], pf, acc[db]);
        if (b < 3) vf[db] = frag_cols<DC>(Vs, (b + 1) * 16, db, lane);
      }
    }
#pragma unroll
    for (int i = 0; i < 3 * DC; ++i) {
      sched_mfma<1>();
      sched_read<2>();
    }
    sched_mfma<DC>();
    __builtin_amdgcn_s_setprio(0);
  });

  const Halves lh = both_halves(l[0] + l[1]);
  const float ls = lh.lo + lh.hi;
  if (!row_ok) return;
  if (p.splits > 1) {
    const int64_t pi = (int64_t)j.split * p.Tq * p.Hq + oi;
    store_row_f32<DC>(p.part + pi * p.D, acc, p.D, h);
    if (h == 0) {
      p.part_ml[2 * pi] = m * c;
      p.part_ml[2 * pi + 1] = ls;
    }
    return;
  }
  store_row<DC>(p.O + oi * p.D, acc, ls > 0.0f ? 1.0f / ls : (ls == 0.0f ? 0.0f : ls), p.D, h);
  if (p.lse && h == 0) p.lse[oi] = ls == 0.0f ? -INFINITY : m * p.scale + __logf(ls);
}

// Joins the key ranges of a row: a wave to a row; a lane to a range for its
// maximum and sum, then to two columns. Bound by latency: 24 tokens, 64 heads over 20
// ranges 5.5-6.0 us, 3 chunks of 333 tokens, 14 heads over 4 ranges 7.1-7.3.
constexpr int MAX_SPLITS = 64;
static __global__ __launch_bounds__(THREADS) void k_attn_join(Params p) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t rows = p.Tq * p.Hq;
  if (row >= rows) return;
  const int64_t q = row / p.Hq;
  if (p.qo && (q < p.qo[0] || q >= p.qo[p.seqs])) return;   // rows of no sequence
  float ms = -INFINITY, ls = 0.0f;
  if (lane < p.splits) {
    const float *ml = p.part_ml + 2 * (lane * rows + row);
    ms = ml[0];
    ls = ml[1];
  }
  float mx = ls != 0.0f ? ms : -INFINITY;   // (a NaN is not 0)
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
  const float as = ls != 0.0f ? exp2_hw(ms - mx) : 0.0f;
  float l = as * ls;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) l += __shfl_xor(l, o);
  float o0 = 0.0f, o1 = 0.0f;
  const int d = lane * 2;
  // The ranges that count (one without keys has a sum of 0), asked for by all lanes:
  // a lane whose columns are past D still holds a range's sum.
  const unsigned long long counts = __ballot(ls != 0.0f);
  for (int s0 = 0; s0 < p.splits; s0 += 8) {
    f32x2_t v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      v[u] = f32x2_t{0.0f, 0.0f};
      if ((counts >> (s0 + u) & 1) && d < p.D)   // (s0 + u < 64, and no bits from p.splits on)
        v[u] = *reinterpret_cast<const f32x2_t *>(p.part + ((s0 + u) * rows + row) * p.D + d);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float a = __shfl(as, s0 + u);
      o0 = __builtin_fmaf(a, v[u][0], o0);
      o1 = __builtin_fmaf(a, v[u][1], o1);
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (d < p.D) *reinterpret_cast<uint32_t *>(p.O + row * p.D + d) = pack_bf16x2(o0 * inv, o1 * inv);
  if (p.lse && lane == 0) p.lse[row] = l == 0.0f ? -INFINITY : mx * (1.0f / LOG2E) + __logf(l);
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

// dQ: a tile of rows over its keys, as the forward. It also makes the rows' delta
// for k_attn_dkv, which runs after it: delta from the bf16 O is off by O's
// rounding, which shows as rows of dS that do not sum to zero; their fp32 sum is
// added to it, so that dK is free of that error. dQ keeps it (it would take the
// product P K as well) but in the rows that see at most 32 keys: their delta is the
// sum of P dP, which took dQ's error over 16 tokens of peaked scores from 0.0046 to
// 0.0024 of its norm and over 64 from 0.0035 to 0.0028, for 1.5 % of the time. O's
// rounding weighs most where few keys carry a row's weight, whether or not it sees
// more: 500 to 700 tokens with scores of deviation 0.25, 2.25, 9 and 36 have dQ off by
// 0.0024, 0.0028, 0.0053 and 0.0066 of its norm.
//
// S and dP are made here and in k_attn_dkv: seven products instead of five, but no
// sums of dQ over key tiles in memory, whose order would change the results. dS is
// rounded to bf16 for dS K (an error of 2^-8 of each term; a second product of what
// that drops cost 15 to 25 % of the time). Bound by the matrix cores: 8192 tokens,
// 64 heads 1.40-1.52 ms, 1.08-1.18 PFLOP/s of its three products, in flight 64 % of
// the cycles at 1.65 GHz; packed 4096 tokens, 32 heads 69-80 us.
template <int DC>
__global__ __launch_bounds__(THREADS, 2) void k_attn_dq(Params p) {
  using T = Lds<DC>;
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];
  constexpr int TE = KEYS * T::RW;

  Job j = map_job(p);
  const Tile t = map_tile<false>(p, p.slots - 1 - j.slot, ROWS);
  if (t.tile < 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int h = lane >> 5;
  const int R = t.Lq * p.G;
  const int off = t.Lk - t.Lq;

  const int r = t.tile * ROWS + wave * 32 + (lane & 31);
  const bool row_ok = r < R;
  const int qi = (int)row_query(p, (uint32_t)(row_ok ? r : R - 1));
  const int64_t oi = (t.q0 + qi) * p.Hq + j.head * p.G + ((row_ok ? r : R - 1) - qi * p.G);
  const int64_t hd = (oi - (t.q0 + qi) * p.Hq) * p.D;   // the head's first column
  u32x4_t qf[2 * DC], of[2 * DC];
  load_row_frags<DC>(qf, p.Q + (t.q0 + qi) * p.ldq + hd, p.D, h);
  load_row_frags<DC>(of, p.dO + oi * p.D, p.D, h);
  const float ls = p.lse[oi];
  // a row that saw no key has no gradient: P = exp2(-inf) = 0
  const float lse2 = ls == -INFINITY ? INFINITY : ls * LOG2E;
  float dl = 0.0f;
#pragma unroll
  for (int kk = 0; kk < 2 * DC; ++kk) {
    const int col = 16 * kk + 8 * h;
    u32x4_t o = ldg_b128_cached(p.Oin + oi * p.D + (col < p.D ? col : 0));
    if (col >= p.D) o = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      dl = __builtin_fmaf(bf16_bits_to_f32(o[e] & 0xFFFFu), bf16_bits_to_f32(of[kk][e] & 0xFFFFu), dl);
      dl = __builtin_fmaf(bf16_bits_to_f32(o[e] >> 16), bf16_bits_to_f32(of[kk][e] >> 16), dl);
    }
  }
  const Halves dh = both_halves(dl);
  dl = dh.lo + dh.hi;
  float rest = 0.0f;   // sum of the row's dS

  const int q_hi = (int)row_query(p, (uint32_t)min(R - 1, t.tile * ROWS + ROWS - 1));
  const int q_lo = (int)row_query(p, (uint32_t)min(R - 1, t.tile * ROWS + wave * 32));
  const int kend = min(t.Lk, q_hi + off + 1);
  const int nt = kend > 0 ? (kend + KEYS - 1) / KEYS : 0;
  const int full = min(t.Lk, q_lo + off + 1);

  f32x16_t acc[DC];
#pragma unroll
  for (int i = 0; i < DC; ++i) acc[i] = f32x16_t{};
  const float c = p.scale * LOG2E;
  const int lim = qi + off;

  // keys that any row of the wave sees (none where it has no rows)
  const int wr0 = t.tile * ROWS + wave * 32;
  const int wend = wr0 < R ? min(kend, (int)row_query(p, (uint32_t)min(R - 1, wr0 + 31)) + off + 1) : 0;
  KvStream ks(p.K, p.ldk, p, t, j.head, 0), vs(p.V, p.ldv, p, t, j.head, 0);
  auto issue = [&](int stage) {
    uint16_t *dst = smem + stage * 2 * TE;
    load_kv<DC, KEYS>(ks.next(), dst, p.ldk, p.D, wave, lane);
    load_kv<DC, KEYS>(vs.next(), dst + TE, p.ldv, p.D, wave, lane);
  };

  if (nt > 0) issue(0);
  two_stages(0, nt, [&](int s, auto stage) __attribute__((always_inline)) {
    constexpr int ST = decltype(stage)::value;
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
    if (s + 1 < nt) issue(ST ^ 1);
    const uint16_t *Ks = smem + ST * 2 * TE, *Vs = Ks + TE;
    const int k0 = s * KEYS;
    if (k0 >= wend) return;
    const bool edge = k0 + KEYS > full;
    const int lk = lim - k0 - 4 * h;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      f32x16_t sc = f32x16_t{}, dp = f32x16_t{};
      u32x4_t cf[DC];
#pragma unroll
      for (int kk = 0; kk < 2 * DC; ++kk) {
        sc = mfma_32x32x16(frag_rows<DC>(Ks, kb * 32, kk, lane), qf[kk], sc);
        dp = mfma_32x32x16(frag_rows<DC>(Vs, kb * 32, kk, lane), of[kk], dp);
      }
#pragma unroll
      for (int db = 0; db < DC; ++db) cf[db] = frag_cols<DC>(Ks, kb * 32, db, lane);
      sched_read<4>();
#pragma unroll
      for (int i = 0; i < 4 * DC - 4; ++i) {
        sched_mfma<1>();
        sched_read<1>();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sched_mfma<1>();
        sched_read<(2 * DC + 3) / 4>();
      }
      if (kb == 0 && s == 0 && full <= 32) {
        // rows that see no key past these 32: delta from P and dP themselves
        float d = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (8 * (i >> 2) + (i & 3) <= lk) d = __builtin_fmaf(exp2_hw(__builtin_fmaf(sc[i], c, -lse2)), dp[i], d);
          asm volatile("" : "+v"(d));   // (one at a time: registers)
        }
        const Halves both = both_halves(d);
        if (lim < 32) dl = both.lo + both.hi;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[i] = exp2_hw(__builtin_fmaf(sc[i], c, -lse2)) * (dp[i] - dl);
      if (edge) {
        asm volatile("");   // a branch, not selects in every step
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (kb * 32 + 8 * (i >> 2) + (i & 3) > lk) sc[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) rest += sc[i];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const u32x4_t df = pack8(sc, b * 8);
#pragma unroll
        for (int db = 0; db < DC; ++db) {
          acc[db] = mfma_32x32x16(cf[db], df, acc[db]);
          if (b == 0) cf[db] = frag_cols<DC>(Ks, kb * 32 + 16, db, lane);
        }
      }
#pragma unroll
      for (int i = 0; i < DC; ++i) {
        sched_mfma<1>();
        sched_read<2>();
      }
      sched_mfma<DC>();
    }
  });
  const Halves rh = both_halves(rest);
  if (!row_ok) return;
  if (h == 0) {
    p.stat[oi] = lse2;
    p.stat[p.Tq * p.Hq + oi] = dl + (rh.lo + rh.hi);
  }
  store_row<DC>(p.dQ + (t.q0 + qi) * p.lddq + hd, acc, p.scale, p.D, h);
}

// dK, dV: a tile of keys (32 a wave, K and V in registers) over the packed rows
// that see them, 64 to a step. P and dS are rounded to bf16 for P^T dO and dS^T Q
// (2^-8 of each term); both sums stay in registers over all rows.
//
// Bound by registers: K, V, dK and dV of a wave take 192 of 256, so the reads of Q
// and dO run only 3 products ahead. 8192 tokens, 64 heads over 8 key heads 2.18-2.33
// ms, 0.94-1.0 PFLOP/s of its four products, in flight 49 % of the cycles at 1.6-1.8
// GHz; packed 4096 tokens, 32 heads over 8 101-119 us. First form 6.7 ms (63 registers
// spilled); without spills 3.1, statistics of the rows by direct loads 2.5, ranges and
// reads without branches 2.3. One wave a SIMD with 512 registers took 5.7 ms (moves
// between the two register files), V in LDS with 32-row steps 2.6-2.7, row ranges of
// equal work 2.8-3.7 (they end in tiles of many sizes).
template <int DC>
__global__ __launch_bounds__(THREADS, 2) void k_attn_dkv(Params p) {
  using T = Lds<DC>;
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];
  constexpr int TE = BROWS * T::RW;
  constexpr int RPI = 64 / T::CH, NI = BROWS / RPI / 4;
  // Q and dO of two steps, then lse (times log2 e) and delta of their rows
  float *stat = reinterpret_cast<float *>(smem + 4 * TE);   // [2][2][BROWS]

  Job j = map_job(p);
  const Tile t = map_tile<true>(p, j.slot, BKEYS);
  if (t.tile < 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, lane0 = lane;
  const int h = lane >> 5;
  const int R = t.Lq * p.G;
  const int off = t.Lk - t.Lq;

  const int kt = t.tile * BKEYS;                   // the tile's first key
  const int key = kt + wave * 32 + (lane & 31);    // this lane's
  const bool key_ok = key < t.Lk;
  const int64_t kr = t.k0 + (key_ok ? key : t.Lk - 1);
  u32x4_t kf[2 * DC], vf[2 * DC];
  load_row_frags<DC>(kf, p.K + kr * p.ldk + j.head * p.D, p.D, h);
  load_row_frags<DC>(vf, p.V + kr * p.ldv + j.head * p.D, p.D, h);

  // rows from the first query that sees the tile's first key
  const int64_t r_lo = (int64_t)max(0, kt - off) * p.G;
  const int s_lo = (int)(r_lo / BROWS), s_hi = (R + BROWS - 1) / BROWS;
  int s0 = min(s_lo, s_hi), s1 = s_hi;
  if (p.splits > 1) {
    const int per = (s1 - s0 + p.splits - 1) / p.splits;
    s0 = min(s1, s0 + j.split * per);
    s1 = min(s1, s0 + per);
  }
  constexpr int AHEAD = 3;   // reads ahead of their products
  // from this row on every row sees every key of the wave
  const int64_t full = (int64_t)max(0, kt + wave * 32 + 31 - off) * p.G;

  f32x16_t dk[DC], dv[DC];
#pragma unroll
  for (int i = 0; i < DC; ++i) dk[i] = dv[i] = f32x16_t{};
  const float c = p.scale * LOG2E;

  // The wave's first row with a key to see of its own.
  const int64_t mine = (int64_t)max(0, kt + wave * 32 - off) * p.G;
  auto issue = [&](int s, int stage) {
    const int r0 = s * BROWS;
    const int q0 = (int)row_query(p, (uint32_t)r0);
    uint16_t *dst = smem + stage * 2 * TE;
    uint32_t ln = (uint32_t)lane0;
    pin(ln);   // (see below)
    const int lane = (int)ln;
    const int64_t left = (int64_t)t.Lq - q0;
    const int64_t ldo = (int64_t)p.Hq * p.D;
    const rsrc_t rq = big::make_rsrc(p.Q + (t.q0 + q0) * p.ldq, big::clamp_bytes(((left - 1) * p.ldq + ldo) * 2));
    const rsrc_t ro = big::make_rsrc(p.dO + (t.q0 + q0) * ldo, big::clamp_bytes(left * ldo * 2));
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int row = (i * 4 + wave) * RPI + lane / T::CH;
      const int ch = (lane % T::CH) ^ T::swz(row);
      const uint32_t q = row_query(p, (uint32_t)(r0 + row));
      const uint32_t hd = (uint32_t)(j.head * p.G + (r0 + row) - (int)q * p.G) * (uint32_t)p.D + (uint32_t)ch * 8;
      const bool ok = ch * 8 < p.D && r0 + row < R;
      load_lds16(rq, dst + (i * 4 + wave) * 512, ok ? ((q - q0) * (uint32_t)p.ldq + hd) * 2 : OOB);
      load_lds16(ro, dst + TE + (i * 4 + wave) * 512, ok ? ((q - q0) * (uint32_t)ldo + hd) * 2 : OOB);
    }
    // a row to a lane: the first wave loads lse, the second delta (rows that are
    // not there: zeros, as Q and dO, which make zeros of their products)
    if (wave < 2) {
      const uint32_t q = row_query(p, (uint32_t)(r0 + lane));
      const uint32_t at = (q - q0) * (uint32_t)p.Hq + (uint32_t)(j.head * p.G + (r0 + lane) - (int)q * p.G);
      const rsrc_t rs = big::make_rsrc(p.stat + (wave * p.Tq + t.q0 + q0) * p.Hq, big::clamp_bytes(left * p.Hq * 4));
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rs, (__attribute__((address_space(3))) void *)(stat + (stage * 2 + wave) * BROWS), 4,
          r0 + lane < R ? at * 4 : OOB, 0, 0, 0);
    }
  };

  if (s0 < s1) issue(s0, 0);
  two_stages(s0, s1, [&](int s, auto stage) __attribute__((always_inline)) {
    constexpr int ST = decltype(stage)::value;
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
    if (s + 1 < s1) issue(s + 1, ST ^ 1);
    if ((int64_t)(s + 1) * BROWS <= mine) return;   // (no row sees the wave's keys)
    const uint16_t *Qs = smem + ST * 2 * TE, *Os = Qs + TE;
    const float *sl = stat + ST * 2 * BROWS;
    const bool edge = (int64_t)s * BROWS < full;
#pragma unroll 1
    for (int rb = 0; rb < 2; ++rb) {
      // (opaque: the operand addresses are made where they are used, not kept over
      // the loop, which has no registers to spare)
      uint32_t ln = (uint32_t)lane0;
      pin(ln);
      const int lane = (int)ln, h = lane >> 5;
      f32x16_t sc = f32x16_t{}, dp = f32x16_t{};
#pragma unroll
      for (int kk = 0; kk < 2 * DC; ++kk) {
        sc = mfma_32x32x16(frag_rows<DC>(Qs, rb * 32, kk, lane), kf[kk], sc);
        dp = mfma_32x32x16(frag_rows<DC>(Os, rb * 32, kk, lane), vf[kk], dp);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i > 0) __builtin_amdgcn_sched_barrier(0);
        const int row = rb * 32 + 8 * i + 4 * h;
        const f32x4_t l4 = *reinterpret_cast<const f32x4_t *>(sl + row);
        const f32x4_t d4 = *reinterpret_cast<const f32x4_t *>(sl + BROWS + row);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float pe = exp2_hw(__builtin_fmaf(sc[4 * i + e], c, -l4[e]));
          dp[4 * i + e] = pe * (dp[4 * i + e] - d4[e]);
          sc[4 * i + e] = pe;
        }
      }
      if (edge) {
        asm volatile("");   // a branch, not selects in every step
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t r = (uint32_t)(s * BROWS + rb * 32 + 8 * (i >> 2) + 4 * h + (i & 3));
          if (key > (int)row_query(p, r) + off) sc[i] = dp[i] = 0.0f;
        }
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        __builtin_amdgcn_sched_barrier(0);
        const u32x4_t pf = pack8(sc, b * 8), df = pack8(dp, b * 8);
#pragma unroll
        for (int db = 0; db < DC; ++db) {
          dv[db] = mfma_32x32x16(frag_cols<DC>(Os, rb * 32 + b * 16, db, lane), pf, dv[db]);
          dk[db] = mfma_32x32x16(frag_cols<DC>(Qs, rb * 32 + b * 16, db, lane), df, dk[db]);
        }
      }
    }
  });
  if (!key_ok) return;
  if (p.splits > 1) {
    const int64_t n = p.Tk * p.Hkv * p.D;
    float *dst = p.part + 2 * j.split * n + (kr * p.Hkv + j.head) * p.D;
    store_row_f32<DC>(dst, dk, p.D, h);
    store_row_f32<DC>(dst + n, dv, p.D, h);
    return;
  }
  store_row<DC>(p.dK + kr * p.lddk + j.head * p.D, dk, p.scale, p.D, h);
  store_row<DC>(p.dV + kr * p.lddv + j.head * p.D, dv, 1.0f, p.D, h);
}

// Sums the row ranges' dK (times scale) and dV in order: 4 columns a thread. The
// grid runs over the key slots, so that keys of no sequence are left alone. Bound by
// the partials' bytes: 8192 keys, 8 heads, 3 ranges 41-42 us (235 MB, 5.6 TB/s), 4096
// keys, 4 ranges 24.
static __global__ __launch_bounds__(THREADS) void k_attn_dkv_sum(Params p) {
  const Tile t = map_tile<true>(p, blockIdx.x, 16);
  if (t.tile < 0) return;
  const int64_t n = p.Tk * p.Hkv * p.D;
  const int w = p.Hkv * p.D;
  const int keys = min(16, t.Lk - t.tile * 16);
  for (int i = (blockIdx.y * THREADS + threadIdx.x) * 4; i < keys * w; i += gridDim.y * THREADS * 4) {
    const int64_t kr = t.k0 + t.tile * 16 + i / w;
    const int col = i % w;
    const float *src = p.part + kr * w + col;
    f32x4_t a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll 4
    for (int s = 0; s < p.splits; ++s) {
      a += *reinterpret_cast<const f32x4_t *>(src + 2 * s * n);
      b += *reinterpret_cast<const f32x4_t *>(src + (2 * s + 1) * n);
    }
    *reinterpret_cast<u32x2_t *>(p.dK + kr * p.lddk + col) =
        u32x2_t{pack_bf16x2(a[0] * p.scale, a[1] * p.scale), pack_bf16x2(a[2] * p.scale, a[3] * p.scale)};
    *reinterpret_cast<u32x2_t *>(p.dV + kr * p.lddv + col) =
        u32x2_t{pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
  }
}

// The kernels as the host code launches them: by address, so that they compile
// as a unit of their own (attn.hip). dc: 32-element column blocks of a head.
int col_blocks(int D);
const void *fwd_kernel(int dc);
const void *join_kernel();
const void *dq_kernel(int dc);
const void *dkv_kernel(int dc);
const void *dkv_sum_kernel();

}  // namespace attn
}  // namespace lora4
