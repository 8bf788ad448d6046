// The kernels of the feed-forward operators (norm.hpp, small.hpp, act_bwd.hpp
// and the tiles of gemm_fwd.hpp with an epilogue) as the host code launches
// them: by address, so that their instantiations compile as a unit of their
// own (ffn.hip), beside lora4.hip.
#pragma once

#include "act_bwd.hpp"
#include "gemm_dgrad.hpp"
#include "gemm_fwd.hpp"
#include "norm.hpp"
#include "small.hpp"

namespace lora4 {
namespace ffn {

// Row norms: a wave to a row (threads 64, 4 rows to a block of 256) or a block
// of `threads` to a row, vpt vectors of 8 to a thread.
struct NormShape {
  int threads, vpt;
};
NormShape norm_shape(int D);
const void *norm_fwd_kernel(NormShape s, bool mx);
const void *norm_bwd_kernel(NormShape s, bool dw, bool edge);   // edge: D % 8 != 0
const void *col_sum_kernel();

// Forward tiles with an epilogue (epi: fwd::EPI_GATED, fwd::EPI_FUSED).
// Gated tiles are 128 columns of both projections; fused tiles 256 columns
// (rows 256) or 128. short_rows: with the shorter code for the last row tiles
// of a group (rows 256 only).
const void *tile_kernel(int fmt, int epi, int rows, bool short_rows);

// The same with the reduction split over blocks (rows 32, 64 or 128; 128
// columns of both projections or 256), and the sum of their partials.
const void *split_kernel(int fmt, int epi, int rows);
const void *epi_reduce_kernel(int epi);

// Few tokens: up to xt (4, 8) tokens of a group, nw (4, 8, 16) waves.
const void *small_kernel(int fmt, int epi, int xt, int nw);
const void *small_z_kernel();

// Gradient of the activation and dZ: projections 1 or 2; tj: 16-column blocks of
// the rank, 1, 2, 4, 8 or 16 (16 with one projection only).
const void *act_dz_kernel(int projections, int tj);
const void *col_part_kernel();
const void *col_sum_slots_kernel();

// The 256 x 256 dgrad with its reduction split over blocks.
const void *dgrad_split_kernel(int fmt);

}  // namespace ffn
}  // namespace lora4
