// Host side of the vocabulary loss (included by lora4.hip behind its dispatch
// helpers): validation, workspace layout and launch order.
//
//   [k_loss_rows ->] k_loss_target -> per chunk of rows:
//       per piece of the vocabulary: k_loss_logits -> k_loss_join [-> k_loss_dx]
//       k_loss_finish
//   [-> k_loss_total]
//
// How many rows count is known on the device alone: the grids cover all M, and
// blocks past the last row that counts end at once.
#pragma once

namespace {

// Rows of a chunk at most, and bytes of E (a chunk's rows by a piece's words): a
// piece is wide enough that adding its part to acc in memory is small beside its
// product, and narrow enough that E stays far below the logits' size.
constexpr int64_t LOSS_CHUNK = 4096;
constexpr int64_t LOSS_E_BYTES = int64_t(256) << 20;

// The tiles of a launch.
struct LossTiles {
  bool small;
  int tt, vt, wv, strip, side, threads;   // (side: blocks that run side by side)
  size_t lds;
};
template <typename T>
LossTiles loss_tiles_of(bool small, int cus) {
  return {small, T::TT, T::VT, T::WV, T::STRIP, T::PER_CU * cus, T::THREADS, T::LDS_BYTES};
}

// Forced tiles for tests and measurements (LORA4_LOSS_TILES): small or big.
int loss_tiles_policy() {
  const char *e = std::getenv("LORA4_LOSS_TILES");
  return !e ? 0 : std::strcmp(e, "small") == 0 ? 1 : std::strcmp(e, "big") == 0 ? 2 : 0;
}

// Microseconds of a 64-deep step and of a tile's start and end, by tile: big tiles
// do eight times the work of small ones in 2.4 times the time, one to a CU instead
// of two, and want many steps and tiles enough for every CU. Measured beside the
// estimate (small / big, us): logits of 512 tokens, 4096 -> 32000 212 / 118, of 256
// 111 / 109, of 1000, 4600 -> 2070 61 / 107, of 2753, 792 -> 5813 59 / 36; gradients
// of the same 193 / 126, 104 / 80, 43 / 34, 63 / 43, of 300 tokens, 24639 -> 1024
// 27 / 35.
double loss_round_us(bool small, double steps) {
  return small ? 0.8 * steps + 4.0 : 1.75 * steps + 9.0;
}

// Estimated time of the logits, `rows` tokens by V words over K, with tiles t.
double loss_logits_us(const LossTiles &t, int64_t rows, int64_t K, int64_t V) {
  const int64_t tiles = ceil_div(rows, t.tt) * ceil_div(V, t.vt);
  return (double)ceil_div(tiles, t.side) * loss_round_us(t.small, (double)ceil_div(K, loss::BKS));
}

// That of acc: `rows` tokens by K columns over `words`, in the ranges of split_of;
// the ranges are read again when they are summed.
double loss_acc_us(const LossTiles &t, int64_t rows, int64_t K, int64_t words) {
  const int64_t tiles = std::max<int64_t>(1, ceil_div(rows, t.tt) * ceil_div(K, t.vt));
  const int64_t steps = ceil_div(words, loss::BKS);
  const int64_t n = std::max<int64_t>(1, std::min(t.side / tiles, steps / 8));
  return (double)ceil_div(tiles * n, t.side) * loss_round_us(t.small, (double)ceil_div(steps, n)) +
         1e-6 * (double)n * (double)rows * (double)K;
}

// The two kinds of tiles: [0] big, [1] small.
struct LossKinds {
  const int cus = cu_count();
  LossTiles t[2] = {loss_tiles_of<loss::Big>(false, cus), loss_tiles_of<loss::Small>(true, cus)};
  int forced = loss_tiles_policy();
  int logits(int64_t rows, int64_t K, int64_t V) const {
    if (forced) return forced == 1;
    return loss_logits_us(t[1], rows, K, V) < loss_logits_us(t[0], rows, K, V);
  }
  // how much longer acc takes on big tiles (0: those, where they take as long)
  double acc_gap(int64_t rows, int64_t K, int64_t V) const {
    if (forced) return forced == 1 ? 1.0 : -1.0;
    return loss_acc_us(t[0], rows, K, V) - loss_acc_us(t[1], rows, K, V);
  }
};

struct LossPlan {
  LossTiles lt, dt;    // tiles of the logits and of acc
  int64_t chunk;       // rows of a chunk, a multiple of the tiles'
  int64_t piece;       // words of a piece, a multiple of TILE
  size_t off_row, off_tgt, off_xc, off_lt, off_ref, off_s, off_sref, off_ssum, off_e, off_acc, bytes;
};

// Words of a piece at most (the strips' maxima and sums, and 32-bit offsets in E).
constexpr int64_t LOSS_PIECE = int64_t(1) << 19;

// Forced width of a piece for tests (LORA4_LOSS_PIECE, in words).
int64_t loss_piece_policy() {
  const char *e = std::getenv("LORA4_LOSS_PIECE");
  return e ? std::max<int64_t>(1, ceil_div(std::atoi(e), loss::TILE)) : LOSS_PIECE / loss::TILE;
}

lora4_status check_loss_sizes(int64_t M, int64_t K, int64_t V) {
  if (M < 0 || M > (int64_t(1) << 30) || V < 1 || V > (int64_t(1) << 30) || K < 8 || K % 8 != 0 || K > (1 << 20))
    return LORA4_ERR_SHAPE;
  return LORA4_OK;
}

// A plan of M tokens with tiles lt and dt in chunks of `rows` (at most LOSS_CHUNK,
// rounded up to the tiles), pieces of at most `widest` tiles of words.
LossPlan loss_layout(bool grad, int64_t M, int64_t rows, int64_t K, int64_t V, const LossTiles &lt,
                     const LossTiles &dt, int64_t widest) {
  constexpr int64_t T = loss::TILE;
  LossPlan pl{};
  pl.lt = lt;
  pl.dt = dt;
  const int64_t unit = std::max(pl.lt.tt, pl.dt.tt);
  pl.chunk = std::max<int64_t>(unit, ceil_div(rows, unit) * unit);
  const int64_t tiles_v = ceil_div(V, T);
  int64_t piece = std::min(tiles_v, widest);
  if (grad) {
    piece = std::max<int64_t>(1, std::min(piece, LOSS_E_BYTES / (pl.chunk * 2 * T)));
  }
  pl.piece = piece * T;
  size_t off = 256;   // the count
  auto take = [&](size_t n) {
    const size_t at = off;
    off += align256(std::max<size_t>(n, 1));
    return at;
  };
  pl.off_row = take((size_t)M * 4);
  pl.off_tgt = take((size_t)M * 4);
  pl.off_xc = take((size_t)M * K * 2);
  pl.off_lt = take((size_t)M * 4);
  pl.off_ref = take((size_t)M * 4);
  pl.off_s = take((size_t)M * 4);
  const size_t strips = (size_t)(pl.piece / pl.lt.strip) * pl.chunk * 4;
  pl.off_sref = take(strips);
  pl.off_ssum = take(strips);
  if (grad) {
    pl.off_e = take((size_t)pl.chunk * pl.piece * 2);
    // the chunk's rows once, or as many ranges of fewer as fill the chip (split_of)
    pl.off_acc = take((size_t)std::max(pl.chunk, pl.dt.side / ceil_div(K, pl.dt.vt) * pl.dt.tt) * K * 4);
  }
  pl.bytes = off;
  return pl;
}

LossPlan loss_plan(bool grad, int64_t M, int64_t K, int64_t V) {
  const LossKinds k;
  const int64_t rows = std::min(M, LOSS_CHUNK);
  return loss_layout(grad, M, rows, K, V, k.t[k.logits(rows, K, V)], k.t[k.acc_gap(rows, K, V) > 0.0],
                     loss_piece_policy());
}

// Bytes that the plan of any batch of up to M tokens fits in: a shorter one may take
// small tiles, whose strips are four times as many, or wider pieces. The logits' tiles
// and the chunk are the same for all rows of a block of 64, and acc's gap is linear in
// them (where it is close to 0 at an end, both kinds count), so that the ends of each
// block say it all. On the host 0.1 us a block, 7 us for a whole chunk.
size_t loss_workspace(bool grad, int64_t M, int64_t K, int64_t V) {
  const LossKinds k;
  const int64_t top = std::min(M, LOSS_CHUNK), widest = loss_piece_policy();
  size_t most = 256;   // (of no tokens: the count)
  for (int64_t lo = 1; lo <= top; lo += 64) {
    const int64_t hi = std::min(top, lo + 63);
    const LossTiles &lt = k.t[k.logits(hi, K, V)];
    const double a = k.acc_gap(lo, K, V), b = k.acc_gap(hi, K, V);
    if (std::min(a, b) < 1e-6) most = std::max(most, loss_layout(grad, M, hi, K, V, lt, k.t[0], widest).bytes);
    if (std::max(a, b) > -1e-6) most = std::max(most, loss_layout(grad, M, hi, K, V, lt, k.t[1], widest).bytes);
  }
  return most;
}

lora4_status head_loss(const uint16_t *X, const uint16_t *W, const int64_t *targets, const float *weights, int64_t M,
                       int64_t K, int64_t V, int64_t ignore, float *out_loss, float *lse, float *total, uint16_t *dX,
                       void *ws, size_t ws_bytes, hipStream_t st) {
  TRY(check_loss_sizes(M, K, V));
  if (!W || (M > 0 && (!X || !targets || !out_loss))) return LORA4_ERR_NULL;
  if (!all_aligned16({X, W, targets, weights, out_loss, lse, total, dX, ws})) return LORA4_ERR_ALIGN;
  const bool grad = dX != nullptr;
  if (!ws || ws_bytes < loss_workspace(grad, M, K, V)) return LORA4_ERR_WORKSPACE;
  const LossPlan pl = loss_plan(grad, M, K, V);
  loss::Params p{};
  p.X = X;
  p.W = W;
  p.target = targets;
  p.weight = weights;
  p.M = M;
  p.K = K;
  p.V = V;
  p.ignore = ignore;
  p.count = ws_at<int>(ws, 0);
  p.row = ws_at<int>(ws, pl.off_row);
  p.tgt = ws_at<int>(ws, pl.off_tgt);
  p.Xc = ws_at<uint16_t>(ws, pl.off_xc);
  p.lt = ws_at<float>(ws, pl.off_lt);
  p.ref = ws_at<float>(ws, pl.off_ref);
  p.S = ws_at<float>(ws, pl.off_s);
  p.rows = (int)pl.chunk;
  p.E = ws_at<uint16_t>(ws, pl.off_e);
  p.lde = pl.piece;
  p.strip_ref = ws_at<float>(ws, pl.off_sref);
  p.strip_sum = ws_at<float>(ws, pl.off_ssum);
  p.acc = ws_at<float>(ws, pl.off_acc);
  p.piece = pl.piece;
  p.strip = pl.lt.strip;
  p.dt = pl.dt.tt;
  p.dv = pl.dt.vt;
  p.side = pl.dt.side;
  p.loss = out_loss;
  p.lse = lse;
  p.total = total;
  p.dX = dX;
  const bool find = M > 0 && M <= loss::SHORT;
  if (!find) TRY(launch_fn("loss_rows", loss::rows_kernel(), 1, 1024, 0, st, p));
  if (M > 0) TRY(launch_fn("loss_target", loss::target_kernel(find), ceil_div(M, 4), 256, 0, st, p));
  p.total_block = total && M > 0 && M <= pl.chunk;   // (every row's sum is there by then)
  for (int64_t row0 = 0; row0 < M; row0 += pl.chunk) {
    p.row0 = row0;
    const int64_t rows = std::min(pl.chunk, M - row0);
    for (int64_t v0 = 0; v0 < V; v0 += pl.piece) {
      p.v0 = v0;
      p.cols = std::min(pl.piece, V - v0);
      p.first = v0 == 0;
      p.tiles_m = (int)ceil_div(rows, pl.lt.tt);
      p.tiles_n = (int)ceil_div(p.cols, pl.lt.vt);
      p.strips = p.tiles_n * pl.lt.wv;
      TRY(launch_fn("loss_logits", loss::logits_kernel(grad, pl.lt.small),
                    ceil_div((int64_t)p.tiles_m * p.tiles_n, 8) * 8, pl.lt.threads, pl.lt.lds, st, p));
      const int nr = rows <= 256 ? 4 : 32;
      TRY(launch_fn("loss_join", loss::join_kernel(grad, nr), ceil_div(rows, nr), 1024, 0, st, p));
      if (!grad) continue;
      p.tiles_m = (int)ceil_div(rows, pl.dt.tt);
      p.tiles_n = (int)ceil_div(K, pl.dt.vt);
      // all tiles once, or ranges of fewer up to what runs side by side (split_of)
      const int64_t items = std::max<int64_t>((int64_t)p.tiles_m * p.tiles_n, p.side);
      TRY(launch_fn("loss_dx", loss::dx_kernel(pl.dt.small), ceil_div(items, 8) * 8, pl.dt.threads, pl.dt.lds, st, p));
    }
    const dim3 grid((unsigned)(ceil_div(rows, 4) + p.total_block), grad ? (unsigned)ceil_div(K, 512) : 1u);
    TRY(launch_grid("loss_finish", loss::finish_kernel(), grid, 256, 0, st, p));
  }
  return total && !p.total_block ? launch_fn("loss_total", loss::total_kernel(), 1, 1024, 0, st, p) : LORA4_OK;
}

}  // namespace
