// Host side of the feed-forward operators (included by lora4.hip behind its
// planning and dispatch helpers): validation, workspace layout and launch
// order of the RMS norm, the gated projections and the linear with an epilogue.
//
//   gated forward   : Z = X A^T, both projections' A as one operand of 2 r rows
//                     (k_small_z, or the rank-r row pass for many rows), then
//                     k_small, or the gated tiles, whole or split and summed
//   gated backward  : [Z pass] -> k_act_dz (dG, dU, partial dZ) -> dX over
//                     both projections as one reduction -> dA, dB
//   fused forward   : as the gated, with one projection
//   fused backward  : with an activation as the gated, with one projection and
//                     dbias; else dbias and the plain layer's backward
#pragma once

namespace {

// ---------------------------------------------------------------------------
// Launch by kernel address (ffn.hpp)
// ---------------------------------------------------------------------------

template <typename... Args>
lora4_status launch_grid(const char *name, const void *fn, dim3 grid, int threads, size_t lds, hipStream_t st,
                         Args... args) {
  if (lds > 64 * 1024) TRY(set_lds_limit(fn, lds));
  void *argv[] = {(void *)&args...};
  return launch_timed(name, st, [&] {
    (void)hipLaunchKernel(fn, grid, dim3((unsigned)threads), argv, lds, st);
  });
}

template <typename... Args>
lora4_status launch_fn(const char *name, const void *fn, int64_t blocks, int threads, size_t lds, hipStream_t st,
                       Args... args) {
  if (blocks <= 0) return LORA4_OK;
  if (blocks > INT32_MAX) return LORA4_ERR_SHAPE;
  return launch_grid(name, fn, dim3((unsigned)blocks), threads, lds, st, args...);
}

bool all_aligned16(std::initializer_list<const void *> ps) {
  for (const void *p : ps)
    if (p && !aligned16(p)) return false;
  return true;
}

// ---------------------------------------------------------------------------
// RMS norm
// ---------------------------------------------------------------------------

// Blocks of the norm's grids: enough for the chip to be full several times
// over (rows beyond them are walked in steps of the grid).
constexpr int64_t NORM_MAX_BLOCKS = 1 << 16;
// Blocks with dW: each keeps a row of fp32 sums to be added up afterwards, so
// as many as are on the chip at a time, by their registers (blocks of up to four
// waves, which hold two rows: 8 waves per CU; wider ones 16, with masks 12). A
// multiple of 8 (see k_rmsnorm_bwd), unless every row has a block.
int norm_rows_per_block(ffn::NormShape s) { return s.threads == 64 ? norm::WAVE_ROWS : 1; }

int64_t norm_dw_blocks(int64_t M, int64_t D) {
  const ffn::NormShape s = ffn::norm_shape((int)D);
  const int64_t waves = s.threads == 64 ? norm::WAVE_ROWS : s.threads / 64;
  const int64_t per_cu = std::max<int64_t>(1, (waves <= 4 ? 8 : D % 8 == 0 ? 16 : 12) / waves);
  const int64_t need = ceil_div(M, norm_rows_per_block(s));
  return std::min(std::max<int64_t>(8, per_cu * cu_count() / 8 * 8), need);
}

size_t norm_ws_bytes(int64_t M, int64_t D) {
  const ffn::NormShape s = ffn::norm_shape((int)D);
  return align256((size_t)std::max<int64_t>(1, norm_dw_blocks(M, D)) * norm_rows_per_block(s) * D * 4);
}

lora4_status check_norm(int64_t M, int64_t D, float eps) {
  if (M < 0 || M > (int64_t(1) << 31) || D < 1 ||
      D > (D % 8 == 0 ? norm::MAX_D : norm::MAX_D_UNALIGNED))
    return LORA4_ERR_SHAPE;
  if (!std::isfinite(eps) || eps < 0.0f) return LORA4_ERR_SHAPE;
  return LORA4_OK;
}

// dW of zero rows
lora4_status fill_zero(uint16_t *p, int64_t n, hipStream_t st) {
  return launch_args("fill_zero", k_fill_u16, dim3((unsigned)ceil_div(n, 256)), dim3(256), st, p, n, (uint16_t)0);
}

lora4_status norm_forward(const uint16_t *X, const uint16_t *R, const uint16_t *w, int64_t M, int64_t D, float eps,
                          uint16_t *H, uint16_t *Y, uint8_t *codes, uint8_t *scales, hipStream_t st) {
  TRY(check_norm(M, D, eps));
  if (codes && D % 32 != 0) return LORA4_ERR_SHAPE;
  if (!w || (M > 0 && !X) || (!codes) != (!scales) || (M > 0 && !Y && !codes) || (H && !R && M > 0))
    return LORA4_ERR_NULL;
  if (!all_aligned16({X, R, w, H, Y, codes, scales})) return LORA4_ERR_ALIGN;
  if (M == 0) return LORA4_OK;
  const norm::FwdParams p{X, R, w, M, (int)D, eps, H, Y, codes, scales};
  const ffn::NormShape s = ffn::norm_shape((int)D);
  const int64_t blocks = std::min(NORM_MAX_BLOCKS, ceil_div(M, norm_rows_per_block(s)));
  return launch_fn("rmsnorm_fwd", ffn::norm_fwd_kernel(s, codes != nullptr), blocks,
                   s.threads == 64 ? 64 * norm::WAVE_ROWS : s.threads, 0, st, p);
}

lora4_status norm_backward(const uint16_t *dY, const uint16_t *H, const uint16_t *w, const uint16_t *dH, int64_t M,
                           int64_t D, float eps, uint16_t *dX, uint16_t *dW, void *ws, size_t ws_bytes,
                           hipStream_t st) {
  TRY(check_norm(M, D, eps));
  if (!w || (M > 0 && (!dY || !H || !dX))) return LORA4_ERR_NULL;
  if (!all_aligned16({dY, H, w, dH, dX, dW, ws})) return LORA4_ERR_ALIGN;
  if (dW && M > 0 && (!ws || ws_bytes < norm_ws_bytes(M, D))) return LORA4_ERR_WORKSPACE;
  if (M == 0) return dW ? fill_zero(dW, D, st) : LORA4_OK;
  const ffn::NormShape s = ffn::norm_shape((int)D);
  const int64_t per = norm_rows_per_block(s);
  const int64_t blocks = dW ? norm_dw_blocks(M, D) : std::min(NORM_MAX_BLOCKS, ceil_div(M, per));
  const norm::BwdParams p{dY, H, w, dH, M, (int)D, eps, dX, dW ? reinterpret_cast<float *>(ws) : nullptr};
  TRY(launch_fn("rmsnorm_bwd", ffn::norm_bwd_kernel(s, dW != nullptr, D % 8 != 0), blocks,
                s.threads == 64 ? 64 * norm::WAVE_ROWS : s.threads, 0, st, p));
  if (!dW) return LORA4_OK;
  return launch_fn("rmsnorm_dw", ffn::col_sum_kernel(), ceil_div(D, 32), 1024, 0, st, (const float *)ws,
                   (int)(blocks * per), (int)D, dW);
}

// ---------------------------------------------------------------------------
// Gated and fused forward
// ---------------------------------------------------------------------------

// An operator's base: E row groups with P projections each (gated: 2, W's
// groups 2 e and 2 e + 1).
struct Ffn {
  const lora4_W *W;
  int epi;       // fwd::EPI_GATED or fwd::EPI_FUSED
  int P;
  int64_t E;
  int64_t M;
  int r;
};

// Tokens per group up to which the few-token kernel runs: one slot of it, and
// two for one projection without groups (14336 -> 4096, NF4, 16 tokens: 25 us
// against 39 with the split tiles; gated, 4096 -> 14336: 38 against 39,
// 8192 -> 28672 MXFP4: 99 against 73; 16 experts of 2048 x 7168: 77 against 45).
constexpr int64_t SMALL_ROWS = 8;

// Forced schedule for tests and measurements (LORA4_FFN_ROWS): 4 or 8 the
// few-token kernel with that many tokens per slot; 1064, 1128 or 1256 the
// tiles of 64, 128 or 256 rows; 2032, 2064 or 2128 the tiles of that many rows
// with their reduction split; anything else or unset: automatic.
int ffn_policy() {
  const char *e = std::getenv("LORA4_FFN_ROWS");
  if (!e) return 0;
  const int v = std::atoi(e);
  for (int ok : {4, 8, 1064, 1128, 1256, 2032, 2064, 2128})
    if (v == ok) return v;
  return 0;
}

struct FfnPlan {
  bool small;
  int xt, nw;           // small: tokens per slot, waves
  int rows;             // tiles: rows per tile
  bool split;           // tiles: their reduction in ksplit ranges of split_steps 64-deep steps
  int ksplit, split_steps;
  int64_t slots, cblocks;
  bool z_small;         // Z by k_small_z (z_splits ranges of z_per chunks), else by the rank-r row pass
  int z_splits;
  int64_t z_per;
  SkSched zs;           // the rank-r row pass's schedule
  bool z_tail;          // the tiles' tail adds up Z's range partials
  size_t off_sz, off_zpart, off_part, bytes;
};

// The tiles and split of the reduction with the least estimated time. Measured
// (gated, NF4 and MXFP4 bases of 4096 x 14336 and 8192 x 28672, 16 experts of
// 7168 x 2048, fused 14336 -> 4096): a 64-deep step of a tile takes about
// `alone` us on a CU of its own, and `shared` us of the CU where several share
// one (`occ` at a time); starting a tile and writing it out about 4 us; a split
// reduction another launch of about 6 us and its partial sums' way through
// memory. Shapes a few percent apart in this estimate are as close in time.
struct TileShape {
  int rows, cols;      // per tile (gated: columns of each projection)
  bool split;
  int occ;
  double alone, shared;   // 0: DEEP_STEP
};
// The deep tiles (fwd::deep_tile) of 256 columns are bound by their decode,
// on a CU of their own or not: NF4's by table lookups, the others' by conversions.
constexpr double DEEP_STEP_NF4 = 0.75, DEEP_STEP = 0.52;
constexpr TileShape GATED_TILES[] = {
    {64, 128, false, 2, 0, 0}, {128, 128, false, 1, 0.95, 0.95}, {256, 128, false, 1, 1.7, 1.7},
    {32, 128, true, 3, 0, 0},  {64, 128, true, 2, 0, 0},         {128, 128, true, 1, 0.95, 0.95},
};
constexpr TileShape FUSED_TILES[] = {
    {64, 128, false, 2, 0.55, 0.5}, {128, 128, false, 2, 0.62, 0.6}, {256, 256, false, 1, 1.7, 1.7},
    {32, 256, true, 3, 0, 0},        {64, 256, true, 2, 0, 0},        {128, 256, true, 1, 0.95, 0.95},
};

void choose_tiles(const Ffn &f, int64_t M, int pol, int64_t cus, FfnPlan &p) {
  const int64_t N = f.W->N, steps = ceil_div(f.W->K, fwd::BKS), extra = f.E > 1 ? std::min(f.E, M) : 0;
  double best = 0;
  for (const TileShape &s : f.epi == fwd::EPI_GATED ? GATED_TILES : FUSED_TILES) {
    if (pol && pol != (s.split ? 2000 : 1000) + s.rows) continue;
    const int64_t slots = ceil_div(M, s.rows) + extra, cb = ceil_div(N, s.cols);
    // tiles with rows: one for each group, and a group's last one is half full on average
    const double tiles = (double)cb * (f.E > 1 ? std::max((double)extra, (double)M / s.rows + 0.5 * (double)extra)
                                               : (double)ceil_div(M, s.rows));
    const double deep = f.W->format == LORA4_NF4 || f.W->format == LORA4_NF4_DQ ? DEEP_STEP_NF4 : DEEP_STEP;
    double alone = s.alone > 0 ? s.alone : deep, shared = s.shared > 0 ? s.shared : deep;
    // groups of few rows run the 256-row tiles' shorter code; the largest of
    // uneven groups sets the pace, with about twice the mean (16 experts of
    // 7168 x 2048, 16 rows each: 65 us; 64-row split tiles 77)
    if (f.E > 1 && s.rows == 256 && 2 * M <= 128 * f.E) alone = shared = 2 * M <= 64 * f.E ? deep : 0.95;
    // a split: as many ranges (of at least four steps) as keep the chip full once
    int64_t per = steps, ks = 1;
    if (s.split) {
      const int64_t want = std::min<int64_t>((int64_t)((double)(s.occ * cus) / tiles), steps / 4);
      if (want < 2 && !pol) continue;
      per = ceil_div(steps, std::max<int64_t>(1, want));
      ks = ceil_div(steps, per);
    }
    const double blocks = tiles * (double)ks;
    const double rounds = std::ceil(blocks / (double)(s.occ * cus));
    const double each = std::max(1.0, blocks / (rounds * (double)cus));   // blocks on a CU at a time
    const double step = s.occ == 1 ? alone : std::max(alone, each * shared);
    double t = rounds * (step * (double)per + 4.0);
    if (s.split) t += 6.0 + blocks * s.rows * (4 * 64 * 4) * 2 / 4.0e6;
    if (p.rows == 0 || t < best) {
      best = t;
      p.rows = s.rows;
      p.slots = slots;
      p.cblocks = cb;
      p.split = s.split;
      p.ksplit = (int)ks;
      p.split_steps = s.split ? (int)per : 1 << 30;
    }
  }
}

// Rows up to which k_small_z makes the Z of the tiles.
constexpr int64_t Z_SMALL_ROWS = 1024;

FfnPlan ffn_plan(const Ffn &f) {
  FfnPlan p{};
  const int64_t M = std::max<int64_t>(f.M, 1), N = f.W->N, K = f.W->K;
  const int64_t extra = f.E > 1 ? std::min(f.E, M) : 0;   // slots cut short at the ends of groups with rows
  const int64_t cus = cu_count();
  const int pol = ffn_policy();
  const int R = f.P * f.r;
  const int64_t mean = ceil_div(M, f.E);
  p.ksplit = 1;
  p.split_steps = 1 << 30;
  p.small = pol ? pol < 1000 : mean <= (f.P == 1 && f.E == 1 ? 2 : 1) * SMALL_ROWS;
  int64_t max_zsplits = big::A2_MAX_PARTS;
  if (p.small) {
    p.xt = pol ? pol : mean <= 4 ? 4 : 8;
    p.slots = ceil_div(M, p.xt) + extra;
    p.cblocks = ceil_div(N, 16);
    // about 14 waves per CU
    const int64_t groups = p.slots * p.cblocks;
    p.nw = groups >= 3 * cus ? 4 : groups >= 3 * cus / 2 ? 8 : 16;
    // (every workgroup of the base product reads the ranges' partials of its
    // tokens: at most 16 KB)
    max_zsplits = std::max<int64_t>(1, std::min<int64_t>(16, 4096 / (std::min<int64_t>(M, p.xt) * R)));
  } else {
    choose_tiles(f, M, pol, cus, p);
  }
  p.z_small = p.small || f.M <= Z_SMALL_ROWS;
  size_t off = 0;
  auto take = [&](size_t b) {
    const size_t o = off;
    off += align256(b);
    return o;
  };
  if (p.z_small) {
    // ranges of one pass of loads each, while they do not fill the chip anyway
    const int64_t chunks = K / 32, blocks = (ceil_div(M, 16) + extra) * ceil_div(R, 16);
    p.z_splits = (int)std::max<int64_t>(
        1, std::min({ceil_div(chunks, small::Z_WAVES * small::Z_CHUNKS), max_zsplits, 8 * cus / blocks}));
    p.z_per = ceil_div(chunks, p.z_splits);
    p.z_splits = (int)ceil_div(chunks, p.z_per);
    p.off_zpart = take((size_t)p.z_splits * M * R * 4);
  } else {
    p.zs = sk_sched(f.M, K, R, f.E, 0);
    p.z_tail = p.zs.ranges > 1 && p.zs.ranges <= big::A2_MAX_PARTS;
    p.off_sz = take((size_t)M * R * 2);
    p.off_zpart = take(sk_part_bytes_for(f.M, K, R, f.E, 0));
  }
  if (p.split)
    p.off_part = take((size_t)p.slots * p.cblocks * p.ksplit * 4 * p.rows * 64 * 4);
  p.bytes = std::max<size_t>(off, 256);
  return p;
}

lora4_status check_ffn(const Ffn &f, int act, float s, const int64_t *offs) {
  TRY(check_W(f.W));
  if (f.P == 2 && f.W->groups % 2 != 0) return LORA4_ERR_SHAPE;
  if (act < LORA4_ACT_NONE || act > LORA4_ACT_GELU_TANH) return LORA4_ERR_FORMAT;
  if (f.M < 0 || f.M > (int64_t(1) << 31)) return LORA4_ERR_SHAPE;
  if (f.r < 1 || f.r > 256 / f.P) return LORA4_ERR_SHAPE;
  if (!std::isfinite(s)) return LORA4_ERR_SHAPE;
  if (f.E > 1 && !offs) return LORA4_ERR_NULL;
  if (f.E == 1 && offs) return LORA4_ERR_SHAPE;
  // 32-bit buffer offsets within a group's base and a row tile
  Base b{f.W, f.W->groups, false};
  if (!big_fits(f.W->K, f.M, packed_of(b))) return LORA4_ERR_SHAPE;
  return LORA4_OK;
}

struct FfnOut {
  uint16_t *out, *pre, *Z;
  const uint16_t *bias, *residual;
};

lora4_status ffn_forward(const Ffn &f, int act, const uint16_t *X, const uint16_t *A, const uint16_t *B, float s,
                         const int64_t *offs, const FfnOut &o, void *ws, size_t ws_bytes, hipStream_t st) {
  TRY(check_ffn(f, act, s, offs));
  if (!A || !B || (f.M > 0 && (!X || !o.out))) return LORA4_ERR_NULL;
  if (!all_aligned16({X, A, B, offs, o.out, o.pre, o.Z, o.bias, o.residual, ws})) return LORA4_ERR_ALIGN;
  const FfnPlan pl = ffn_plan(f);
  if (!ws || ws_bytes < pl.bytes) return LORA4_ERR_WORKSPACE;
  if (f.M == 0) return LORA4_OK;
  const lora4_W *W = f.W;
  const PackedW pw = packed_of(Base{W, W->groups, false});
  const int R = f.P * f.r;   // rank columns of a row group
  float *zpart = ws_at<float>(ws, pl.off_zpart);
  if (pl.z_small) {
    small::ZParams z{};
    z.X = X;
    z.A = A;
    z.M = f.M;
    z.K = W->K;
    z.R = R;
    z.offsets = offs;
    z.groups = (int)f.E;
    z.part = zpart;
    z.jblocks = (int)ceil_div(R, 16);
    z.splits = pl.z_splits;
    z.per = pl.z_per;
    const int64_t zslots = ceil_div(f.M, 16) + (f.E > 1 ? std::min(f.E, f.M) : 0);
    TRY(launch_fn("small_z", ffn::small_z_kernel(), zslots * z.jblocks * z.splits, 64 * small::Z_WAVES, 0, st, z));
  }
  if (pl.small) {
    small::Params p{};
    p.W = pw;
    p.X = X;
    p.M = f.M;
    p.K = W->K;
    p.N = W->N;
    p.offsets = offs;
    p.groups = (int)f.E;
    p.r = f.r;
    p.zpart = zpart;
    p.zsplits = pl.z_splits;
    p.s = s;
    p.Z = o.Z;
    p.B = B;
    p.act = act;
    p.out = o.out;
    p.pre = o.pre;
    p.bias = o.bias;
    p.residual = o.residual;
    p.nblocks = (int)pl.cblocks;
    p.tab = nf4_table();
    return launch_fn(f.P == 2 ? "small_gated" : "small_fused", ffn::small_kernel(W->format, f.epi, pl.xt, pl.nw),
                     pl.slots * pl.cblocks, 64 * pl.nw, small::lds_bytes(f.P, pl.xt, pl.nw), st, p);
  }
  uint16_t *sZ = ws_at<uint16_t>(ws, pl.off_sz);
  big::Params q = big_params(mat(X, W->K), pw, W->K, mat(sZ, R), mat(B, f.r, W->N * f.r), R, f.M, W->N, offs, f.E,
                             o.out, W->N);
  if (pl.z_small) {
    const TailParts tp{zpart, pl.z_splits, s, o.Z, 1.0f, nullptr, 0.0f};
    apply_tail_parts(q, &tp);
  } else {
    uint16_t *z1 = o.Z ? o.Z : sZ, *z2 = o.Z ? sZ : nullptr;
    TRY(rows_skinny(0, X, W->K, A, W->K, (int64_t)R * W->K, W->K, f.M, R, offs, f.E, z1, o.Z ? 1.0f : s, z2, s, zpart,
                    pl.z_tail, st));
    if (pl.z_tail) {
      const TailParts tp{zpart, pl.zs.ranges, s, o.Z, 1.0f, nullptr, 0.0f};
      apply_tail_parts(q, &tp);
    }
  }
  q.act = act;
  q.pre = o.pre;
  q.bias = o.bias;
  q.residual = o.residual;
  q.tiles_n = (int)pl.cblocks;
  q.nslots = (int)pl.slots;
  const int64_t blocks = pl.slots * pl.cblocks * pl.ksplit;
  if (blocks > INT32_MAX) return LORA4_ERR_SHAPE;
  q.nblocks = (int)blocks;
  const char *name = f.P == 2 ? "gemm_gated" : "gemm_fused";
  if (pl.split) {
    q.ksplit = pl.ksplit;
    q.split_steps = pl.split_steps;
    q.Cpart = ws_at<float>(ws, pl.off_part);
    TRY(launch_fn(name, ffn::split_kernel(W->format, f.epi, pl.rows), blocks, fwd::THREADS,
                  (size_t)fwd::epi_lds_bytes(pl.rows, 2, true), st, q));
    const int64_t pieces = pl.slots * pl.cblocks * 4 * pl.rows * (f.P == 2 ? 4 : 8);
    return launch_fn("epilogue", ffn::epi_reduce_kernel(f.epi), ceil_div(pieces, 256), 256, 0, st, q, pl.rows);
  }
  const int nj = f.P == 2 || pl.rows == 256 ? 2 : 1;
  return launch_fn(name, ffn::tile_kernel(W->format, f.epi, pl.rows, pl.rows == 256 && f.E > 1), blocks, fwd::THREADS,
                   (size_t)fwd::epi_lds_bytes(pl.rows, nj, false), st, q);
}

// ---------------------------------------------------------------------------
// Backward of the gated projections, and of one projection with an activation
// ---------------------------------------------------------------------------

// The bases of a group's projections as one base of P Np rows (Np: N rounded
// up to whole row blocks; the padding rows dequantize to zero): the reduction
// of dX runs over the gradients of both.
PackedW joint_base(const lora4_W *W, int P, int64_t Np) {
  PackedW p = packed_of(Base{W, W->groups, false});
  p.N = P * Np;
  if (P == 2) {
    p.half = Np;
    p.half_s2 = p.g_scales2;
    p.g_codes *= 2;
    p.g_scales *= 2;
    p.g_scales2 *= 2;
  }
  return p;
}

constexpr int64_t ACT_DZ_BLOCKS = 1024;   // blocks wanted of k_act_dz
constexpr int ACT_DZ_RANGES = 32;

// How dX is made: the library's own choice for the plain layer (the 256 x 256
// dgrad where its tiles fill the chip, else the 128 x 128 kernel), or the
// 256 x 256 dgrad with the reduction split over blocks.
// LORA4_FFN_DGRAD forces it for tests and measurements: "split" or "own".
int dgrad_policy() {
  const char *e = std::getenv("LORA4_FFN_DGRAD");
  if (!e) return 0;
  const std::string v(e);
  return v == "split" ? 1 : v == "own" ? 2 : 0;
}

struct FfnBwdPlan {
  int64_t Np;
  PackedW pw;
  lora4_W Wv;        // the joint base as make_plan sees it
  Plan pl;           // its dgrad plan
  bool dx_split;     // dX by the split dgrad, in dx_ranges ranges of dx_steps steps
  int dx_ranges, dx_steps;
  int64_t dx_slots;
  int64_t slots;     // row slots of k_act_dz
  int ranges, steps;
  int rt, msplit_a, msplit_b;
  int64_t tq_a, tq_b, ncnt;
  size_t off_z, off_skpart, off_dz, off_grad, off_dzpart, off_col, off_pa, off_pb, off_cnt, off_partx, bytes;
};

FfnBwdPlan ffn_bwd_plan(const Ffn &f, bool dbias) {
  FfnBwdPlan p{};
  const lora4_W *W = f.W;
  const int64_t M = std::max<int64_t>(f.M, 1), K = W->K, N = W->N, G = f.P * f.E;
  const int64_t extra = f.E > 1 ? std::min(f.E, M) : 0;
  const int R = f.P * f.r;
  p.Np = w_blocks(N) * 64;
  p.pw = joint_base(W, f.P, p.Np);
  p.Wv = *W;
  p.Wv.N = f.P * p.Np;
  p.Wv.groups = f.E;
  p.pl = make_plan(1, Base{&p.Wv, f.E, false}, f.M, R);
  {
    const int64_t ld = f.P * p.Np, steps = ceil_div(ld, dgrad::BKS), cus = cu_count();
    p.dx_slots = ceil_div(M, dgrad::BM) + extra;
    const int64_t tiles = p.dx_slots * ceil_div(K, dgrad::BN);
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>({cus / std::max<int64_t>(tiles, 1), steps / 4, 32}));
    p.dx_steps = (int)ceil_div(steps, want);
    p.dx_ranges = (int)ceil_div(steps, p.dx_steps);
    // Estimated times, us: 1.9 a step, the partial sums' way through memory, and
    // an extra launch; against the 128 x 128 kernel's rate, on few blocks and on
    // many. Measured
    // (NF4, 4096 x 4096): 512 rows 52 against 73 us, 2048 rows 92 against 137;
    // gated 4096 x 14336, 1024 rows: 224 against 767; 1024 x 2048 (MXFP4), 256
    // rows: 33 against 25.
    const double t_split = 1.9 * p.dx_steps + 16.0 + 2.0 * p.dx_ranges * (double)M * (double)K * 4 / 4.0e6;
    const int64_t own_slots = ceil_div(M, BM_MAIN) + extra;
    const double t_own = 20.0 + 2.0 * (double)own_slots * BM_MAIN * (double)K * (double)ld /
                                    (own_slots * ceil_div(K, BN_MAIN) < cus ? 3.6e8 : 5.2e8);
    const int pol = dgrad_policy();
    const bool fits = big_fits(ld, M, p.pw) && big_policy() < 0;
    p.dx_split = fits && pol != 2 && !dgrad_taken(ld, ld, f.M, p.pw, K, f.E) && (pol == 1 || t_split < t_own);
  }
  p.slots = ceil_div(M, 64) + extra;
  const int64_t all = p.Np / 64;
  const int64_t want = std::min<int64_t>({ceil_div(ACT_DZ_BLOCKS, p.slots), ACT_DZ_RANGES, all});
  p.steps = (int)ceil_div(all, std::max<int64_t>(1, want));
  p.ranges = (int)ceil_div(all, p.steps);
  p.rt = skinny_tile(f.r);
  p.tq_a = ceil_div(K, TN_BQ);
  p.tq_b = ceil_div(N, TN_BQ);
  const int64_t rtiles = ceil_div(f.r, p.rt), mavg = std::max<int64_t>(1, M / f.E);
  auto msplit = [&](int64_t qtiles) {
    const int64_t tiles = rtiles * qtiles * G;
    const int64_t w = ceil_div(TARGET_WG * 16 / p.rt, std::max<int64_t>(tiles, 1));
    return (int)std::max<int64_t>(1, std::min<int64_t>({w, std::max<int64_t>(1, mavg / 256), 65535 / G}));
  };
  p.msplit_a = msplit(p.tq_a);
  p.msplit_b = msplit(p.tq_b);
  p.ncnt = rtiles * (p.tq_a + p.tq_b) * G;
  size_t off = 0;
  auto take = [&](size_t b) {
    const size_t o = off;
    off += align256(b);
    return o;
  };
  const size_t mr = (size_t)M * R;
  p.off_z = take(mr * 2);
  p.off_skpart = take(sk_part_bytes_for(f.M, K, R, f.E, 0));
  p.off_dz = take(mr * 2);
  p.off_grad = take((size_t)M * f.P * p.Np * 2);
  p.off_dzpart = take((size_t)p.ranges * mr * 4);
  p.off_col = take(dbias ? (size_t)p.slots * N * 4 : 0);
  p.off_pa = take((size_t)p.msplit_a * G * f.r * K * 4);
  p.off_pb = take((size_t)p.msplit_b * G * f.r * N * 4);
  p.off_cnt = take((size_t)p.ncnt * 4);
  const int64_t parts = p.dx_split ? p.dx_ranges : p.pl.lds_splits > 1 ? p.pl.lds_splits : 0;
  p.off_partx = take((size_t)parts * M * K * 4);
  p.bytes = off;
  return p;
}

lora4_status ffn_backward(const Ffn &f, int act, const uint16_t *X, const uint16_t *dY, const uint16_t *pre,
                          const uint16_t *A, const uint16_t *B, float s, const int64_t *offs, const uint16_t *Z,
                          uint16_t *dX, uint16_t *dA, uint16_t *dB, uint16_t *dbias, void *ws, size_t ws_bytes,
                          hipStream_t st) {
  const FfnBwdPlan p = ffn_bwd_plan(f, dbias != nullptr);
  if (!ws || ws_bytes < p.bytes) return LORA4_ERR_WORKSPACE;
  const lora4_W *W = f.W;
  const int64_t K = W->K, N = W->N, G = f.P * f.E, ld = f.P * p.Np;
  const int r = f.r, R = f.P * r;
  if (f.M == 0) {
    TRY(fill_zero(dA, G * r * K, st));
    if (dbias) TRY(fill_zero(dbias, f.E * N, st));
    return fill_zero(dB, G * N * r, st);
  }
  const uint16_t *Zu = Z;
  if (!Zu) {
    uint16_t *Zw = ws_at<uint16_t>(ws, p.off_z);
    TRY(rows_skinny(0, X, K, A, K, (int64_t)R * K, K, f.M, R, offs, f.E, Zw, 1.0f, nullptr, 0.0f,
                    ws_at<float>(ws, p.off_skpart), false, st));
    Zu = Zw;
  }
  // the gradients before the activation and the partial sums of dZ; the first
  // block clears the arrival counters of the dA / dB tiles
  uint16_t *grad = ws_at<uint16_t>(ws, p.off_grad), *dZ = ws_at<uint16_t>(ws, p.off_dz);
  float *zpart = ws_at<float>(ws, p.off_dzpart), *col = dbias ? ws_at<float>(ws, p.off_col) : nullptr;
  unsigned *cnt = ws_at<unsigned>(ws, p.off_cnt);
  {
    actbwd::DzParams q{dY,   pre,     B,     f.M, N,   p.Np,   r,     act, offs, (int)f.E,
                       grad, p.steps, zpart, col, cnt, p.ncnt};
    const void *fn = ffn::act_dz_kernel(f.P, r <= 16 ? 1 : r <= 32 ? 2 : r <= 64 ? 4 : r <= 128 ? 8 : 16);
    void *argv[] = {&q};
    TRY(launch_timed("act_dz", st, [&] {
      (void)hipLaunchKernel(fn, dim3((unsigned)p.slots, (unsigned)p.ranges), dim3(actbwd::THREADS), argv, 0, st);
    }));
  }
  if (dbias) {
    const int E = (int)f.E;
    int64_t M = f.M, n = N;
    void *argv[] = {&col, (void *)&offs, (void *)&E, &M, &n, &dbias};
    const void *sum = ffn::col_sum_slots_kernel();
    TRY(launch_timed("dbias_sum", st, [&] {
      (void)hipLaunchKernel(sum, dim3((unsigned)ceil_div(N, 32), (unsigned)f.E), dim3(1024), argv, 0, st);
    }));
  }
  // dZ = s (..): by the dgrad's tail where it takes partial sums, else here
  const bool big = p.dx_split || dgrad_taken(ld, ld, f.M, p.pw, K, f.E);
  const bool tail = p.ranges <= big::A2_MAX_PARTS && big;
  const TailParts tp{zpart, p.ranges, s, dZ, s, nullptr, 0.0f};
  if (!tail)
    TRY(reduce_bf16("reduce_dz", zpart, p.ranges, f.M * R, f.M * R, dZ, s, nullptr, 0.0f, st));
  // dX = [dG dU] [deq(Wg); deq(Wu)] + dZ [Ag; Au]
  float *partx = ws_at<float>(ws, p.off_partx);
  if (p.dx_split) {
    big::Params q = big_params(mat(grad, ld), p.pw, ld, mat(dZ, R), mat(A, K, (int64_t)R * K), R, f.M, K, offs, f.E,
                               dX, K);
    if (tail) apply_tail_parts(q, &tp);
    q.nslots = (int)p.dx_slots;
    q.ksplit = p.dx_ranges;
    q.split_steps = p.dx_steps;
    q.Cpart = partx;
    TRY(launch_fn("gemm_nn_dgrad", ffn::dgrad_split_kernel(W->format), p.dx_slots * q.tiles_n * p.dx_ranges,
                  dgrad::THREADS, (size_t)dgrad::lds_bytes(), st, q));
    TRY(reduce_bf16("reduce_dx", partx, p.dx_ranges, f.M * K, f.M * K, dX, 1.0f, nullptr, 0.0f, st));
  } else {
    NnParams q{};
    q.A = mat(grad, ld);
    q.W = p.pw;
    q.R = ld;
    q.A2 = mat(dZ, R);
    q.B2 = mat(A, K, (int64_t)R * K);
    q.r2 = R;
    q.M = f.M;
    q.Nc = K;
    q.offsets = offs;
    q.groups = (int)f.E;
    q.Rsplit = ld;
    q.out = GemmOut{dX, K, nullptr, 0, 1.0f};
    q.tab = nf4_table();
    dim3 grid((unsigned)ceil_div(K, BN_MAIN), (unsigned)p.pl.row_slots, 1);
    TRY(run_nn_main_fmt(W->format, q, grid, p.pl, partx, tail ? &tp : nullptr, st));
  }
  // dA = dZ^T X and dB = s [dG dU]^T Z, per projection
  TnParams pa{};
  pa.U = mat(dZ, R);
  pa.V = mat(X, K);
  pa.P = r;
  pa.Q = K;
  pa.M = f.M;
  pa.offsets = offs;
  pa.groups = (int)G;
  pa.splits = p.msplit_a;
  pa.part = ws_at<float>(ws, p.off_pa);
  pa.cnt = cnt;
  pa.out = dA;
  pa.alpha = 1.0f;
  pa.transpose_out = 0;
  pa.half_shift = f.P - 1;
  pa.u_half = f.P == 2 ? r : 0;
  pa.v_half = 0;
  TnParams pb = pa;
  pb.U = mat(Zu, R);
  pb.V = mat(grad, ld);
  pb.Q = N;
  pb.splits = p.msplit_b;
  pb.part = ws_at<float>(ws, p.off_pb);
  pb.cnt = cnt + ceil_div(r, p.rt) * p.tq_a * G;
  pb.out = dB;
  pb.alpha = s;
  pb.transpose_out = 1;
  pb.v_half = f.P == 2 ? p.Np : 0;
  return run_tn2("gemm_tn_dA_dB", p.rt, pa, pb, (int)p.tq_a, (int)(p.msplit_a * G), (int)p.tq_b,
                 (int)(p.msplit_b * G), st);
}

// Backward of one projection without an activation: the plain layer's, and the
// column sums of dY.
struct ColPlan {
  int64_t xblocks;
  int splits;          // row ranges of k_col_part per group
  size_t bytes;
};

ColPlan col_plan(const Ffn &f) {
  ColPlan p{};
  const int64_t M = std::max<int64_t>(f.M, 1), N = f.W->N;
  p.xblocks = ceil_div(N, actbwd::COL_BLOCK);
  // about 1024 blocks, of at least 16 rows each
  p.splits = (int)std::max<int64_t>(1, std::min<int64_t>(ceil_div(1024, p.xblocks * f.E), ceil_div(M, 16 * f.E)));
  p.bytes = align256((size_t)f.E * p.splits * 4 * N * 4);
  return p;
}

lora4_status col_sums(const Ffn &f, const uint16_t *dY, const int64_t *offs, uint16_t *dbias, void *ws,
                      hipStream_t st) {
  if (f.M == 0) return fill_zero(dbias, f.E * f.W->N, st);
  const ColPlan p = col_plan(f);
  float *part = reinterpret_cast<float *>(ws);
  actbwd::ColParams q{dY, f.M, (int)f.W->N, offs, (int)f.E, part};
  const void *fn = ffn::col_part_kernel();
  void *argv[] = {&q};
  TRY(launch_timed("dbias_part", st, [&] {
    (void)hipLaunchKernel(fn, dim3((unsigned)p.xblocks, (unsigned)p.splits, (unsigned)f.E), dim3(actbwd::THREADS),
                          argv, 0, st);
  }));
  const int n = p.splits * 4, D = (int)f.W->N;
  void *sargv[] = {&part, (void *)&n, (void *)&D, &dbias};
  const void *sum = ffn::col_sum_kernel();
  return launch_timed("dbias_sum", st, [&] {
    (void)hipLaunchKernel(sum, dim3((unsigned)ceil_div(D, 32), (unsigned)f.E), dim3(1024), sargv, 0, st);
  });
}

size_t fused_bwd_bytes(const Ffn &f, bool act, bool dbias) {
  if (act) return ffn_bwd_plan(f, dbias).bytes;
  return (dbias ? col_plan(f).bytes : 0) + make_plan(1, Base{f.W, f.E, false}, f.M, f.r).bytes;
}

}  // namespace
