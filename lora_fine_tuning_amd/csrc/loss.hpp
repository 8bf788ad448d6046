// Softmax cross entropy over a large vocabulary behind a frozen head, with the
// gradient of its input, in pieces of the vocabulary:
//
//   l = X W^T,  loss_i = log(sum_v exp l_iv) - l_it,
//   dX_i = w_i (softmax(l_i) - onehot(t_i)) W
//
// The logits are never kept. With the gradient wanted, one pass makes both:
// for each piece of the vocabulary
//
//   E = exp(l - ref) of the piece's logits, target column left out   (bf16)
//   S += the row sums of E (unrounded),  acc += E W_piece            (fp32)
//
// and at the end dX = w (acc / (S + s_t) - S / (S + s_t) W_t), s_t = exp(l_t -
// ref): two products of the size of the logits where a second pass for them
// would take three. The row's reference is the logit of its own target, which
// is a term of the sum, so that no term that counts can underflow; loss =
// log1p(S) keeps its digits where the target is nearly certain, and p_t - 1 =
// -S / (S + s_t) does not cancel. A strip of logits more than REF_SLACK binary
// orders above the reference is stored against its own maximum instead, and
// k_loss_join brings the row onto the new reference.
//
// Rows without a target (prompts, padding) are left out before the products:
// the rows that count are copied together once (k_loss_rows).
//
// Both products run on v_mfma_f32_32x32x16_bf16, operands by direct loads into LDS
// stages of 64-deep slabs: tiles of 256 x 256 by eight waves with two stages, or,
// for few tokens or few words, 64 tokens x 128 by four waves with three stages,
// two blocks to a CU. The vocabulary
// (the hidden columns) is the first operand, so that a lane's results belong to
// one token: its row's maximum and sum are lane-local but for one exchange, and
// its stores are contiguous.
#pragma once

#include "common.hpp"
#include "gemm_big.hpp"

namespace lora4 {
namespace loss {

using big::OOB;
using big::rsrc_t;

constexpr int BKS = 64;              // reduction step

// A tile: WV x WT waves, each of AV x 2 blocks of 32 x 32; the first operand is the
// words (hidden columns), the second the tokens.
template <int WV_, int WT_, int AV_, int STAGES_>
struct Shape {
  static constexpr int WV = WV_, WT = WT_, AV = AV_, STAGES = STAGES_;
  static constexpr int NW = WV * WT, THREADS = 64 * NW;
  static constexpr int VT = 32 * AV * WV, TT = 64 * WT;   // words, tokens
  static constexpr int STRIP = 32 * AV;                   // words of a wave: one maximum and sum per row
  static constexpr int SLAB_V = VT * BKS, SLAB_T = TT * BKS, STAGE = SLAB_V + SLAB_T;   // elements
  static constexpr size_t LDS_BYTES = (size_t)STAGES * STAGE * 2;
  static constexpr int PER_CU = NW == 8 ? 1 : 2;
};
using Big = Shape<2, 4, 4, 2>;
using Small = Shape<4, 1, 1, 3>;
constexpr int TILE = 256;            // pieces of the vocabulary are multiples of it

constexpr float LOG2E = 1.44269504088896340736f;
constexpr float REF_SLACK = 64.0f;   // binary orders a logit may lie above its row's reference

struct Params {
  const uint16_t *X;        // bf16 [M][K]
  const uint16_t *W;        // bf16 [V][K]
  const int64_t *target;    // [M]
  const float *weight;      // [M] or null: 1 / rows that count
  int64_t M, K, V;
  int64_t ignore;
  // the rows that count, together
  int *count;               // [0] rows
  int *row;                 // [M] their rows
  int *tgt;                 // [M] their targets (-1: out of range)
  uint16_t *Xc;             // [M][K]
  float *lt;                // [M] target's logit
  float *ref;               // [M] reference
  float *S;                 // [M] sum over the other words
  // a chunk of them and a piece of the vocabulary
  int64_t row0;             // first (of the rows that count)
  int rows;                 // rows of the chunk (a multiple of the tiles')
  int64_t v0;               // first word
  int64_t cols, piece;      // words, and those of all pieces but the last
  uint16_t *E;              // [rows][lde]
  int64_t lde;              // a multiple of TILE
  int strip, strips;        // words of a strip, strips of the piece's tiles
  float *strip_ref, *strip_sum;   // [strips][live rows]
  float *acc;               // [splits][live rows, whole tiles][K]
  int dt, dv;               // tokens and hidden columns of acc's tiles
  int side;                 // blocks of acc's product that run side by side
  int total_block;          // k_loss_finish makes total
  int first;                // first piece: acc is written, not added to
  int tiles_m, tiles_n;
  // outputs
  float *loss, *lse, *total;
  uint16_t *dX;
};

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ void load_lds16(const rsrc_t &r, uint16_t *dst, uint32_t voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 16, voff, soff, 0, 0);
}

// Item of the grid: consecutive blocks go to consecutive XCDs, each of which takes
// a contiguous range of the n items, so that its blocks share operands in its L2.
__device__ __forceinline__ int xcd_item(int id, int n) {
  const int per = (n + 7) / 8;
  const int t = (id & 7) * per + (id >> 3);
  return (id >> 3) < per && t < n ? t : -1;
}

// Tile t in grouped order: runs of RUN row tiles walked column by column.
constexpr int RUN = 8;
__device__ __forceinline__ void grouped(int t, int tiles_m, int tiles_n, int &tm, int &tn) {
  const int g = t / (RUN * tiles_n), r = t - g * RUN * tiles_n;
  const int rows = min(RUN, tiles_m - g * RUN);
  tn = r / rows;
  tm = g * RUN + (r - tn * rows);
}

// A ROWS x 64 slab (rows of ld elements, the reduction contiguous) into the
// tile64 layout. The 1-KB blocks (8 rows) go to the NW waves in turn.
template <int ROWS, int NW>
struct SlabLoad {
  static constexpr int N = ROWS / 8 / NW;   // loads of a wave
  uint32_t voff[N];
  int chunk;        // logical 16-byte chunk this lane fetches (the same in all blocks: NW is even)
  __device__ __forceinline__ SlabLoad(int64_t ld, int wave, int lane) {
    const int rl = lane >> 3;
    // block b = NW i + wave: rows 8 b .. 8 b + 7
    chunk = (lane & 7) ^ ((((wave & 1) << 2) | (rl >> 1)) & 7);
#pragma unroll
    for (int i = 0; i < N; ++i) voff[i] = (uint32_t)((((NW * i + wave) * 8 + rl) * ld + chunk * 8) * 2);
  }
  __device__ __forceinline__ void issue(const rsrc_t &r, uint16_t *lds, int k0, int R, int wave) const {
    const bool edge = k0 + chunk * 8 >= R;
#pragma unroll
    for (int i = 0; i < N; ++i) load_lds16(r, lds + (NW * i + wave) * 512, edge ? OOB : voff[i], k0 * 2);
  }
};

// Operand of 16 reduction columns of the 32 rows from row0.
__device__ __forceinline__ u32x4_t frag(const uint16_t *lds, int row0, int kk, int lane) {
  return lds_read_b128(lds + tile64_swz(row0 + (lane & 31), 2 * kk + (lane >> 5)));
}

// The main loop of both products. Operands of one 16-deep piece are read from LDS
// while the products of the piece before run, and the step's one barrier stands
// between its third and its last piece: there the next step's slabs have landed,
// and everyone has read the last piece of this step's, so that the loads after
// next go into its stage. No product waits at the barrier.
//   issue(step, stage): the step's loads, LOADS instructions of every wave (also
//     past the last step, where nothing is in range, so that the loads in flight
//     at each wait are a constant); read(stage, kk, frags): the operands of piece
//     kk; mma(frags).
constexpr int wait_imm(int vm, int lgkm) { return (vm & 15) | (7 << 4) | (lgkm << 8) | ((vm >> 4) << 14); }

template <int STAGES, int LOADS, int MFMAS, int READS, typename Frags, typename Issue, typename Read, typename Mma>
__device__ __forceinline__ void pipeline(int s0, int s1, Issue &&issue, Read &&read, Mma &&mma) {
  if (s0 >= s1) return;
  Frags f0, f1;
#pragma unroll
  for (int i = 0; i < STAGES; ++i) issue(s0 + i, i);
  __builtin_amdgcn_s_waitcnt(wait_imm((STAGES - 1) * LOADS, 15));
  __syncthreads();
  read(0, 0, f0);
  // MFMAs with the next piece's reads spread over them
  auto hints = [&]() __attribute__((always_inline)) {
    constexpr int GROUPS = MFMAS > 2 ? MFMAS - 2 : 1;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                         // MFMA
      __builtin_amdgcn_sched_group_barrier(0x100, (READS + GROUPS - 1) / GROUPS, 0);   // LDS reads
    }
    __builtin_amdgcn_sched_group_barrier(0x008, MFMAS - GROUPS, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  int stage = 0;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    const int next = stage + 1 == STAGES ? 0 : stage + 1;
    read(stage, 1, f1);
    mma(f0);
    hints();
    read(stage, 2, f0);
    mma(f1);
    hints();
    read(stage, 3, f1);
    mma(f0);
    hints();
    __builtin_amdgcn_s_waitcnt(wait_imm((STAGES - 2) * LOADS, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    issue(s + STAGES, stage);
    read(next, 0, f0);   // (past the last step: not used)
    mma(f1);
    hints();
    stage = next;
  }
  __builtin_amdgcn_s_waitcnt(wait_imm(0, 15));   // (no load into LDS outlives the block)
}

template <int AV>
struct Frags {
  u32x4_t a[AV], b[2];
};

// ---------------------------------------------------------------------------
// The rows that count
// ---------------------------------------------------------------------------

// Rows of a batch whose blocks find the rows that count each for themselves, four
// rows to a thread (a launch less, 3-5 us; the targets are read from the L2).
constexpr int SHORT = 1024;

// The rows whose target is not `ignore`, in order: one block of NT threads looks at
// [0, M) and calls put(index among them, row, target) for each; returns their
// number. Every thread of the block takes part.
template <int NT, typename Put>
__device__ __forceinline__ int find_rows(const Params &p, int *wsum, Put &&put) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int base = 0;
  for (int64_t i0 = 0; i0 < p.M; i0 += NT) {
    const int64_t i = i0 + threadIdx.x;
    const int64_t t = i < p.M ? p.target[i] : p.ignore;
    const bool in = t != p.ignore;
    const unsigned long long b = __ballot(in);
    __syncthreads();   // (the round before is done with wsum)
    if (lane == 0) wsum[wave] = __popcll(b);
    __syncthreads();
    int before = base;
    for (int w = 0; w < NT / 64; ++w) {
      if (w < wave) before += wsum[w];
      base += wsum[w];
    }
    if (in) put(before + __popcll(b & ((1ull << lane) - 1)), (int)i, t >= 0 && t < p.V ? (int)t : -1);
  }
  return base;
}

// One block.
static __global__ __launch_bounds__(1024) void k_loss_rows(Params p) {
  __shared__ int wsum[16];
  const int n = find_rows<1024>(p, wsum, [&](int at, int row, int tgt) {
    p.row[at] = row;
    p.tgt[at] = tgt;
  });
  if (threadIdx.x == 0) *p.count = n;
}

// A wave to a row that counts: its X beside the others', and the logit of its
// target (NaN for a target that is no word or whose logit is +infinity: the row's
// outputs become NaN). And a wave to a row that does not: loss, lse and dX of row i
// are zero. FIND: without k_loss_rows before it (M <= SHORT). Bound by latency and
// X's bytes, which are written once more: 4096 rows of 4096 20 us, 2048 of 5120 14, 8
// rows 7.
template <bool FIND>
__global__ __launch_bounds__(256) void k_loss_target(Params p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int at = blockIdx.x * 4 + wave;
  int count, row = 0, t = 0;
  if constexpr (FIND) {
    __shared__ int wsum[4], mine[4][2];
    count = find_rows<256>(p, wsum, [&](int i, int r, int g) {
      if (blockIdx.x == 0) {
        p.row[i] = r;
        p.tgt[i] = g;
      }
      if (i / 4 == (int)blockIdx.x) {
        mine[i & 3][0] = r;
        mine[i & 3][1] = g;
      }
    });
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.count = count;
    __syncthreads();
    row = mine[wave][0];
    t = mine[wave][1];
  } else {
    count = *p.count;
    if (at < count) {
      row = p.row[at];
      t = p.tgt[at];
    }
  }
  if (at < p.M && p.target[at] == p.ignore) {
    if (lane == 0) {
      p.loss[at] = 0.0f;
      if (p.lse) p.lse[at] = 0.0f;
    }
    if (p.dX)
      for (int64_t k = lane * 8; k < p.K; k += 512)
        *reinterpret_cast<u32x4_t *>(p.dX + (int64_t)at * p.K + k) = u32x4_t{0u, 0u, 0u, 0u};
  }
  if (at >= count) return;
  const uint16_t *x = p.X + (int64_t)row * p.K;
  const uint16_t *w = p.W + (int64_t)max(t, 0) * p.K;
  uint16_t *xc = p.Xc + (int64_t)at * p.K;
  float s = 0.0f;
  for (int64_t k = lane * 8; k < p.K; k += 512) {
    const u32x4_t a = ldg_b128_cached(x + k), b = ldg_b128_cached(w + k);
    *reinterpret_cast<u32x4_t *>(xc + k) = a;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s = __builtin_fmaf(bf16_bits_to_f32(a[i] & 0xFFFFu), bf16_bits_to_f32(b[i] & 0xFFFFu), s);
      s = __builtin_fmaf(bf16_bits_to_f32(a[i] >> 16), bf16_bits_to_f32(b[i] >> 16), s);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if (lane == 0) {
    if (t < 0 || s == INFINITY) s = __builtin_nanf("");
    p.lt[at] = s;
    p.ref[at] = s;
    p.S[at] = 0.0f;
  }
}

// ---------------------------------------------------------------------------
// Logits of a piece: strip maxima and sums, and E
// ---------------------------------------------------------------------------

// Rows between strips: those that count (lines of few rows hold many strips).
__device__ __forceinline__ int strip_ld(int live) { return (live + 7) & ~7; }

// The tile's results: wave (wv, wt) holds the words of a strip, AV blocks, of
// tokens 64 wt .. + 63 (2 blocks). The epilogue takes the strip's maximum and the sum
// of exp(l - reference) of every row in registers, in fp32, and with GRAD stores E, which
// is rounded to bf16 for its product with W (2^-8 of each term, as the operand that a
// softmax rounded to bf16 would be).
//
// Bound by the matrix cores at the clock the card holds under them (products in flight
// 61 % of the cycles at 1.9 GHz): 3686 rows, 4096 -> 32768 with E 831-868 us, 1.14-1.19
// PFLOP/s (a library product of the same operands, whose logits are then in memory,
// 1.39); 2048 rows, 5120 -> 32003 without 522-553, 1.21-1.29 PFLOP/s. Few rows, by the
// head's bytes: 8 rows, 4096 -> 128256 170-195 us, 5.4-6.2 TB/s. 32-deep stages, five of
// them, took 865 us where two of 64 took 840.
template <bool GRAD, typename T>
__global__ __launch_bounds__(T::THREADS, 2) void k_loss_logits(Params p) {
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];
  const int item = xcd_item(blockIdx.x, p.tiles_m * p.tiles_n);
  if (item < 0) return;
  int tm, tn;
  grouped(item, p.tiles_m, p.tiles_n, tm, tn);
  const int live = min(*p.count - (int)p.row0, p.rows);   // rows of this chunk that count
  if (tm * T::TT >= live) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wv = wave % T::WV, wt = wave / T::WV, h = lane >> 5;
  const int64_t v0 = p.v0 + (int64_t)tn * T::VT;   // first word of the tile
  const int64_t t0 = p.row0 + (int64_t)tm * T::TT;
  const int K = (int)p.K;
  const rsrc_t wr = big::make_rsrc(p.W + v0 * p.K, big::clamp_bytes(min((int64_t)T::VT, p.V - v0) * p.K * 2));
  const rsrc_t xr = big::make_rsrc(p.Xc + t0 * p.K, big::clamp_bytes((int64_t)min(T::TT, live - tm * T::TT) * p.K * 2));
  const SlabLoad<T::VT, T::NW> lw(p.K, wave, lane);
  const SlabLoad<T::TT, T::NW> lx(p.K, wave, lane);

  f32x16_t acc[T::AV][2];
#pragma unroll
  for (int i = 0; i < T::AV; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x16_t{};

  using F = Frags<T::AV>;
  pipeline<T::STAGES, lw.N + lx.N, 2 * T::AV, T::AV + 2, F>(
      0, (K + BKS - 1) / BKS,
      [&](int s, int stage) __attribute__((always_inline)) {
        uint16_t *dst = smem + stage * T::STAGE;
        lw.issue(wr, dst, s * BKS, K, wave);
        lx.issue(xr, dst + T::SLAB_V, s * BKS, K, wave);
      },
      [&](int stage, int kk, F &f) __attribute__((always_inline)) {
        const uint16_t *Ws = smem + stage * T::STAGE, *Xs = Ws + T::SLAB_V;
#pragma unroll
        for (int i = 0; i < T::AV; ++i) f.a[i] = frag(Ws, wv * T::STRIP + i * 32, kk, lane);
#pragma unroll
        for (int j = 0; j < 2; ++j) f.b[j] = frag(Xs, wt * 64 + j * 32, kk, lane);
      },
      [&](const F &f) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < T::AV; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = mfma_32x32x16(f.a[i], f.b[j], acc[i][j]);
      });

  // word of register r of block i: vw + 32 i + 8 (r / 4) + r % 4
  const int vw = wv * T::STRIP + 4 * h;
  const int strip = tn * T::WV + wv;
  const int vend = (int)min((int64_t)T::VT, p.V - v0);   // words of the tile that exist
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int tl = tm * T::TT + wt * 64 + j * 32 + (lane & 31);   // row of the chunk
    const bool ok = tl < live;
    const int64_t at = p.row0 + tl;
    const float ref = ok ? p.ref[at] : INFINITY;
    // the target as a word of this lane's (its register), where it is one
    const int64_t rel = ok ? (int64_t)p.tgt[at] - v0 - vw : -1;
    const int own = rel >= 0 && rel < T::STRIP ? (int)rel : -1;
    if (__ballot(own >= 0) || vend < T::VT) {   // (few strips hold a target or the vocabulary's end)
      asm volatile("");   // a branch, not selects in every tile
#pragma unroll
      for (int i = 0; i < T::AV; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int at_r = 32 * i + 8 * (r >> 2) + (r & 3);
          if (at_r == own || vw + at_r >= vend) acc[i][j][r] = -INFINITY;
        }
    }
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < T::AV; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) mx = fmaxf(mx, acc[i][j][r]);
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float rs = (mx - ref) * LOG2E > REF_SLACK ? mx : ref;
    float sum = 0.0f;
    const float rl = rs == -INFINITY ? 0.0f : rs * LOG2E;   // (a strip of -infinity alone: zeros)
#pragma unroll
    for (int i = 0; i < T::AV; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float e = exp2_hw(__builtin_fmaf(acc[i][j][r], LOG2E, -rl));
        acc[i][j][r] = e;
        sum += e;
      }
    sum += __shfl_xor(sum, 32);
    if (ok) {
      if (h == 0) p.strip_ref[(int64_t)strip * strip_ld(live) + tl] = rs;
      else p.strip_sum[(int64_t)strip * strip_ld(live) + tl] = sum;
    }
    if constexpr (GRAD) {
      if (!ok) continue;   // (both halves of a row)
      uint16_t *dst = p.E + (int64_t)tl * p.lde + tn * T::VT + wv * T::STRIP;
#pragma unroll
      for (int i = 0; i < T::AV; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          // the lane halves trade, so that each holds 8 words in a row
          const f32x16_t &c = acc[i][j];
          const auto w0 = __builtin_amdgcn_permlane32_swap(pack_bf16x2(c[8 * q], c[8 * q + 1]),
                                                           pack_bf16x2(c[8 * q + 4], c[8 * q + 5]), false, false);
          const auto w1 = __builtin_amdgcn_permlane32_swap(pack_bf16x2(c[8 * q + 2], c[8 * q + 3]),
                                                           pack_bf16x2(c[8 * q + 6], c[8 * q + 7]), false, false);
          *reinterpret_cast<u32x4_t *>(dst + i * 32 + q * 16 + h * 8) = u32x4_t{w0[0], w1[0], w0[1], w1[1]};
        }
    }
  }
}

// Word ranges of the product acc += E W, from the rows that count (which the device alone
// knows): as many as the chip takes in one round, of at least 8 steps each.
struct Split {
  int n, steps;      // ranges, 64-word steps of a range
  int64_t stride;    // elements of acc between ranges
};
__device__ __forceinline__ Split split_of(const Params &p, int live, int64_t cols) {
  const int tiles_m = (min(live, p.rows) + p.dt - 1) / p.dt;
  const int tiles = max(1, tiles_m * (int)((p.K + p.dv - 1) / p.dv));
  const int steps = (int)((cols + BKS - 1) / BKS);
  Split s;
  s.n = max(1, min(p.side / tiles, steps / 8));
  s.steps = (steps + s.n - 1) / s.n;
  s.stride = (int64_t)tiles_m * p.dt * p.K;
  return s;
}

// The strips of a piece into the rows' sums. NR rows to a block, 1024 / NR threads
// to a row (32 rows read whole lines; few rows have more threads each: 8 rows of
// 1002 strips 10 us with 256 threads a row, 31 with 32). Where a strip had to take a
// reference of its own, the row gets the largest, and its E and acc are brought onto
// it (E is rounded a second time). Bound by latency: 3686 rows of 256 strips 11 us.
template <bool GRAD, int NR>
__global__ __launch_bounds__(1024) void k_loss_join(Params p) {
  constexpr int NT = 1024 / NR;
  __shared__ float red[NT][NR + 1], sums[NT][NR + 1];
  __shared__ float nref[NR], fac[NR];
  __shared__ int moved[NR];
  const int tx = threadIdx.x % NR, ty = threadIdx.x / NR;   // row, strip group
  const int live = min(*p.count - (int)p.row0, p.rows), ld = strip_ld(live);
  const int tl = blockIdx.x * NR + tx;
  if ((int)blockIdx.x * NR >= live) return;
  const int strips = p.strips;
  const bool ok = tl < live;
  const int64_t at = p.row0 + tl;
  const float ref = ok ? p.ref[at] : 0.0f;
  float mx = ref;
  bool nan = ref != ref, other = false;
  if (ok)
    for (int s0 = ty; s0 < strips; s0 += 4 * NT) {
      float r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        r[u] = s0 + u * NT < strips ? p.strip_ref[(int64_t)(s0 + u * NT) * ld + tl] : ref;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        nan |= r[u] != r[u];
        other |= r[u] != ref;
        mx = fmaxf(mx, r[u]);
      }
    }
  red[ty][tx] = nan ? __builtin_nanf("") : mx;
  if (ty == 0) moved[tx] = 0;
  __syncthreads();
  if (other) moved[tx] = 1;   // (every writer writes 1)
  for (int n = NT / 2; n > 0; n /= 2) {
    if (ty < n) {
      const float a = red[ty][tx], b = red[ty + n][tx];
      red[ty][tx] = (a != a || b != b) ? __builtin_nanf("") : fmaxf(a, b);
    }
    __syncthreads();
  }
  const float m = red[0][tx];
  if (ty == 0) nref[tx] = m;
  float sum = 0.0f;
  if (ok)
    for (int s0 = ty; s0 < strips; s0 += 4 * NT) {
      float r[4], v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = (int64_t)(s0 + u * NT) * ld + tl;
        r[u] = s0 + u * NT < strips ? p.strip_ref[i] : m;
        v[u] = s0 + u * NT < strips ? p.strip_sum[i] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) sum += r[u] == m ? v[u] : v[u] * exp2_hw((r[u] - m) * LOG2E);
    }
  sums[ty][tx] = sum;
  __syncthreads();
  for (int n = NT / 2; n > 0; n /= 2) {
    if (ty < n) sums[ty][tx] += sums[ty + n][tx];
    __syncthreads();
  }
  if (ty == 0 && ok) {
    const float f = ref == m ? 1.0f : exp2_hw((ref - m) * LOG2E);
    p.S[at] = p.S[at] * f + sums[0][tx];
    p.ref[at] = m;
    fac[tx] = f;
  }
  if constexpr (GRAD) {
    __syncthreads();
    for (int r = 0; r < NR; ++r) {
      const int row = blockIdx.x * NR + r;
      if (row >= live || !moved[r]) continue;   // uniform
      for (int64_t c = threadIdx.x; c < (int64_t)strips * p.strip; c += 1024) {
        const float sr = p.strip_ref[(c / p.strip) * ld + row];
        if (sr == nref[r]) continue;
        uint16_t *e = p.E + (int64_t)row * p.lde + c;
        *e = to_bf16(bf16_bits_to_f32(*e) * exp2_hw((sr - nref[r]) * LOG2E));
      }
      if (!p.first && fac[r] != 1.0f) {
        const Split sp = split_of(p, live, p.piece);
        for (int s = 0; s < sp.n; ++s)
          for (int64_t k = threadIdx.x; k < p.K; k += 1024) p.acc[s * sp.stride + (int64_t)row * p.K + k] *= fac[r];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// acc += E W_piece
// ---------------------------------------------------------------------------

// W slab: 64 words x VT hidden columns (rows of 512 or 256 bytes, 16-byte chunk c
// of row v at c ^ ((v & 3) << 2): the transposing read takes four rows of 64 bytes
// at a time, which land in the four quarters of the banks).
template <int VT>
__device__ __forceinline__ int wat(int v, int c) {
  return v * VT + ((c ^ ((v & 3) << 2)) << 3);
}

template <int VT>
__device__ __forceinline__ u32x4_t frag_w(const uint16_t *lds, int v0, int col0, int lane) {
  const int h = lane >> 5, i = lane & 15;
  const int col = col0 + ((lane >> 4) & 1) * 16 + (i & 3) * 4;
  const int v = v0 + 8 * h + (i >> 2);
  const u32x2_t lo = lds_read_tr16(lds + wat<VT>(v, col >> 3) + (col & 7));
  const u32x2_t hi = lds_read_tr16(lds + wat<VT>(v + 4, col >> 3) + (col & 7));
  return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
}

// acc of a tile of tokens and hidden columns over a range of the piece's words, fp32,
// added to the pieces' before it. The head is read as it lies, the reduction over its
// rows, by transposing LDS reads. Bound by the matrix cores (61 % of the cycles at 1.9
// GHz): 3686 rows, 32768 words, 4096 columns 764-837 us, 1.18-1.30 PFLOP/s (a library
// product 1.23); 933 rows, 50021 words, 2080 columns in 7 ranges on their XCDs 199 us,
// with ranges on any XCD 352. Two stages of 64; five of 32 took 808 us beside 777.
template <typename T>
__global__ __launch_bounds__(T::THREADS, 2) void k_loss_dx(Params p) {
  extern __shared__ __attribute__((aligned(16))) uint16_t smem[];
  const int live = min(*p.count - (int)p.row0, p.rows);
  if (live <= 0) return;
  // the piece's ranges, in the first piece's number (the last one may be shorter)
  const Split sp = split_of(p, live, p.piece);
  const int tiles_m = (live + T::TT - 1) / T::TT, tiles = tiles_m * p.tiles_n;
  // (range by range: an XCD's blocks are tiles of one or two ranges, which share
  // their words' W and E; the tiles of each range over all XCDs took 1.5 times as
  // long, 933 rows of 2080 over 50021 words)
  const int item = xcd_item(blockIdx.x, tiles * sp.n);
  if (item < 0) return;
  const int split = item / tiles;
  int tm, tn;
  grouped(item - split * tiles, tiles_m, p.tiles_n, tm, tn);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int wk = wave % T::WV, wt = wave / T::WV, h = lane >> 5;
  const int c0 = tn * T::VT;                // first hidden column
  const int K = (int)p.K;
  const int R = (int)p.cols;
  const int s0 = split * sp.steps, s1 = min((R + BKS - 1) / BKS, s0 + sp.steps);

  // E: the tile's rows that count (lde covers whole tiles, zero past the last word)
  const rsrc_t er = big::make_rsrc(p.E + (int64_t)tm * T::TT * p.lde,
                                   big::clamp_bytes((int64_t)min(T::TT, live - tm * T::TT) * p.lde * 2));
  const SlabLoad<T::TT, T::NW> le(p.lde, wave, lane);
  // W: a 1-KB block is WR words; lane's word lane / CPR of it, chunk lane % CPR
  constexpr int CPR = T::VT / 8, WR = 64 / CPR, WN = BKS / WR / T::NW;
  const int wrow = lane / CPR, wpos = lane % CPR;

  f32x16_t acc[T::AV][2];
#pragma unroll
  for (int i = 0; i < T::AV; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x16_t{};
  using F = Frags<T::AV>;
  pipeline<T::STAGES, WN + le.N, 2 * T::AV, 2 * T::AV + 2, F>(
      s0, s1,
      [&](int s, int stage) __attribute__((always_inline)) {
        uint16_t *dst = smem + stage * T::STAGE;
        const int64_t v = p.v0 + (int64_t)s * BKS, left = p.v0 + p.cols - v;
        const rsrc_t wr = big::make_rsrc(p.W + (left > 0 ? v : 0) * p.K,
                                         big::clamp_bytes(min((int64_t)BKS, left) * p.K * 2));
#pragma unroll
        for (int i = 0; i < WN; ++i) {
          const int w = WR * (T::NW * i + wave) + wrow;
          const int c = c0 + (wpos ^ ((w & 3) << 2)) * 8;
          load_lds16(wr, dst + (T::NW * i + wave) * 512, c < K ? (uint32_t)((w * K + c) * 2) : OOB, 0);
        }
        le.issue(er, dst + T::SLAB_V, s * BKS, (int)p.lde, wave);
      },
      [&](int stage, int kk, F &f) __attribute__((always_inline)) {
        const uint16_t *Ws = smem + stage * T::STAGE, *Es = Ws + T::SLAB_V;
#pragma unroll
        for (int i = 0; i < T::AV; ++i) f.a[i] = frag_w<T::VT>(Ws, kk * 16, wk * T::STRIP + i * 32, lane);
#pragma unroll
        for (int j = 0; j < 2; ++j) f.b[j] = frag(Es, wt * 64 + j * 32, kk, lane);
      },
      [&](const F &f) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < T::AV; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) acc[i][j] = mfma_32x32x16(f.a[i], f.b[j], acc[i][j]);
      });
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int tl = tm * T::TT + wt * 64 + j * 32 + (lane & 31);
    if (tl >= live) continue;
    const int col = c0 + wk * T::STRIP + 4 * h;
    float *dst = p.acc + split * sp.stride + (int64_t)tl * p.K + col;
#pragma unroll
    for (int i = 0; i < T::AV; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (col + i * 32 + q * 8 >= K) continue;
        f32x4_t v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        f32x4_t *d = reinterpret_cast<f32x4_t *>(dst + i * 32 + q * 8);
        if (!p.first) v += *d;
        *d = v;
      }
  }
}

// ---------------------------------------------------------------------------
// Outputs
// ---------------------------------------------------------------------------

__device__ __forceinline__ float row_weight(const Params &p, int row, int count) {
  return p.weight ? p.weight[row] : 1.0f / (float)count;
}

// Loss and lse - ref of a row. The target's own term is 1 where the reference is
// its logit, as it mostly is.
struct RowLoss {
  float loss, up, sum;
};
__device__ __forceinline__ RowLoss row_loss(const Params &p, int64_t at) {
  const float S = p.S[at], lt = p.lt[at], ref = p.ref[at];
  RowLoss r;
  r.sum = S + (ref == lt ? 1.0f : exp2_hw((lt - ref) * LOG2E));
  r.up = ref == lt ? log1pf(S) : logf(r.sum);
  r.loss = ref == lt ? r.up : r.up + (ref - lt);
  if (ref == -INFINITY) r.loss = r.sum = __builtin_nanf("");   // no logit above -infinity
  return r;
}

// total = sum of weight times loss over the rows that count: one block of NT
// threads, in a fixed order.
template <int NT>
__device__ __forceinline__ void sum_total(const Params &p, int count) {
  __shared__ float red[NT / 64];
  float s = 0.0f;
  for (int i = threadIdx.x; i < count; i += NT) s += row_weight(p, p.row[i], count) * row_loss(p, i).loss;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.0f;
    for (int w = 0; w < NT / 64; ++w) t += red[w];
    *p.total = t;
  }
}

// A wave to 512 columns of a row of the chunk (column block blockIdx.y): dX = w
// (acc - S W_t) / (S + s_t), and by the first the row's loss. Bound by acc's bytes
// (3686 rows of 4096 23 us). The last block in x,
// where there is one more than the rows need, makes total.
static __global__ __launch_bounds__(256) void k_loss_finish(Params p) {
  const int lane = threadIdx.x & 63;
  const int tl = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int count = *p.count;
  if (p.total_block && blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0) sum_total<256>(p, count);
    return;
  }
  const int64_t at = p.row0 + tl;
  if (at >= count || tl >= p.rows) return;
  const int row = p.row[at];
  const float S = p.S[at];
  const RowLoss r = row_loss(p, at);
  const float sum = r.sum;
  if (blockIdx.y == 0 && lane == 0) {
    p.loss[row] = r.loss;
    if (p.lse) p.lse[row] = r.up + p.ref[at];
  }
  const int64_t k = blockIdx.y * 512 + lane * 8;
  if (!p.dX || k >= p.K) return;
  const float w = row_weight(p, row, count);
  const float a = w / sum, b = a * S;
  const u32x4_t wv = ldg_b128_cached(p.W + (int64_t)max(p.tgt[at], 0) * p.K + k);
  const Split sp = split_of(p, (int)min((int64_t)p.rows, count - p.row0), p.piece);
  const float *src = p.acc + (int64_t)tl * p.K + k;
  f32x4_t lo = {0.0f, 0.0f, 0.0f, 0.0f}, hi = lo;
  for (int s0 = 0; s0 < sp.n; s0 += 4) {
    f32x4_t q[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float *at_u = src + (int64_t)min(s0 + u, sp.n - 1) * sp.stride;
      q[u][0] = *reinterpret_cast<const f32x4_t *>(at_u);
      q[u][1] = *reinterpret_cast<const f32x4_t *>(at_u + 4);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (s0 + u < sp.n) {
        lo += q[u][0];
        hi += q[u][1];
      }
  }
  float o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float we = bf16_bits_to_f32((wv[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
    o[e] = __builtin_fmaf(a, e < 4 ? lo[e & 3] : hi[e & 3], -(b * we));
  }
  *reinterpret_cast<u32x4_t *>(p.dX + (int64_t)row * p.K + k) =
      u32x4_t{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])};
}

// total by itself, of several chunks.
static __global__ __launch_bounds__(1024) void k_loss_total(Params p) { sum_total<1024>(p, *p.count); }

// The kernels as the host code launches them: by address, so that they compile
// as a unit of their own (loss.hip).
const void *rows_kernel();
const void *target_kernel(bool find);
const void *logits_kernel(bool grad, bool small);
const void *join_kernel(bool grad, int rows);
const void *dx_kernel(bool small);
const void *finish_kernel();
const void *total_kernel();

}  // namespace loss
}  // namespace lora4
