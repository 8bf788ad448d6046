// Instantiations of the feed-forward operators' kernels (ffn.hpp).
#include "ffn.hpp"

namespace lora4 {
namespace ffn {

namespace {

template <typename K>
const void *addr(K *k) {
  return reinterpret_cast<const void *>(k);
}

template <bool WAVE, int VPT>
const void *norm_fwd(bool mx) {
  return mx ? addr(norm::k_rmsnorm_fwd<WAVE, VPT, true>) : addr(norm::k_rmsnorm_fwd<WAVE, VPT, false>);
}

template <bool WAVE, int VPT, int MAXW>
const void *norm_bwd(bool dw, bool edge) {
  if (edge)
    return dw ? addr(norm::k_rmsnorm_bwd<WAVE, VPT, true, MAXW, true>)
              : addr(norm::k_rmsnorm_bwd<WAVE, VPT, false, MAXW, true>);
  return dw ? addr(norm::k_rmsnorm_bwd<WAVE, VPT, true, MAXW, false>)
            : addr(norm::k_rmsnorm_bwd<WAVE, VPT, false, MAXW, false>);
}

template <int FMT, int EPI>
const void *tile(int rows, bool short_rows) {
  constexpr int NJ_SMALL = EPI == fwd::EPI_GATED ? 2 : 1;
  if (rows == 64) return addr(fwd::k_gemm_fwd_epi<FMT, EPI, 64, NJ_SMALL, false>);
  if (rows == 128) return addr(fwd::k_gemm_fwd_epi<FMT, EPI, 128, NJ_SMALL, false>);
  return short_rows ? addr(fwd::k_gemm_fwd_epi<FMT, EPI, 256, 2, true>)
                    : addr(fwd::k_gemm_fwd_epi<FMT, EPI, 256, 2, false>);
}

template <int FMT, int EPI>
const void *split(int rows) {
  return rows == 32   ? addr(fwd::k_gemm_fwd_split<FMT, EPI, 32>)
         : rows == 64 ? addr(fwd::k_gemm_fwd_split<FMT, EPI, 64>)
                      : addr(fwd::k_gemm_fwd_split<FMT, EPI, 128>);
}

template <int FMT>
const void *split_of(int epi, int rows) {
  return epi == fwd::EPI_GATED ? split<FMT, fwd::EPI_GATED>(rows) : split<FMT, fwd::EPI_FUSED>(rows);
}

template <int FMT, int EPI, int XT>
const void *small_xt(int nw) {
  return nw == 4   ? addr(small::k_small<FMT, EPI, XT, 4>)
         : nw == 8 ? addr(small::k_small<FMT, EPI, XT, 8>)
                   : addr(small::k_small<FMT, EPI, XT, 16>);
}

template <int FMT>
const void *tile_of(int epi, int rows, bool short_rows) {
  return epi == fwd::EPI_GATED ? tile<FMT, fwd::EPI_GATED>(rows, short_rows)
                               : tile<FMT, fwd::EPI_FUSED>(rows, short_rows);
}

template <int FMT>
const void *small_of(int epi, int xt, int nw) {
  if (epi == fwd::EPI_GATED)
    return xt == 4 ? small_xt<FMT, fwd::EPI_GATED, 4>(nw) : small_xt<FMT, fwd::EPI_GATED, 8>(nw);
  return xt == 4 ? small_xt<FMT, fwd::EPI_FUSED, 4>(nw) : small_xt<FMT, fwd::EPI_FUSED, 8>(nw);
}

}  // namespace

// One wave per row up to 1024 elements; above, a block of as many waves as
// hold the row at two vectors per thread.
NormShape norm_shape(int D) {
  // (the backward's aligned vectors of a row: one more where rows are unaligned)
  const int nv = D % 8 == 0 ? D / 8 : (D + 14) / 8;
  if (nv <= 128) return {64, nv <= 64 ? 1 : 2};
  return {64 * ((nv + 127) / 128), 2};
}

const void *norm_fwd_kernel(NormShape s, bool mx) {
  if (s.threads == 64) return s.vpt == 1 ? norm_fwd<true, 1>(mx) : norm_fwd<true, 2>(mx);
  return norm_fwd<false, 2>(mx);
}

const void *norm_bwd_kernel(NormShape s, bool dw, bool edge) {
  if (s.threads == 64) return s.vpt == 1 ? norm_bwd<true, 1, 4>(dw, edge) : norm_bwd<true, 2, 4>(dw, edge);
  return s.threads <= 256   ? norm_bwd<false, 2, 4>(dw, edge)
         : s.threads <= 512 ? norm_bwd<false, 2, 8>(dw, edge)
                            : norm_bwd<false, 2, 16>(dw, edge);
}

const void *col_sum_kernel() { return addr(norm::k_col_sum); }

const void *tile_kernel(int fmt, int epi, int rows, bool short_rows) {
  switch (fmt) {
    case FMT_NF4: return tile_of<FMT_NF4>(epi, rows, short_rows);
    case FMT_NF4_DQ: return tile_of<FMT_NF4_DQ>(epi, rows, short_rows);
    case FMT_MXFP4: return tile_of<FMT_MXFP4>(epi, rows, short_rows);
    default: return tile_of<FMT_NVFP4>(epi, rows, short_rows);
  }
}

const void *split_kernel(int fmt, int epi, int rows) {
  switch (fmt) {
    case FMT_NF4: return split_of<FMT_NF4>(epi, rows);
    case FMT_NF4_DQ: return split_of<FMT_NF4_DQ>(epi, rows);
    case FMT_MXFP4: return split_of<FMT_MXFP4>(epi, rows);
    default: return split_of<FMT_NVFP4>(epi, rows);
  }
}

const void *epi_reduce_kernel(int epi) {
  return epi == fwd::EPI_GATED ? addr(fwd::k_epi_reduce<fwd::EPI_GATED>) : addr(fwd::k_epi_reduce<fwd::EPI_FUSED>);
}

const void *small_kernel(int fmt, int epi, int xt, int nw) {
  switch (fmt) {
    case FMT_NF4: return small_of<FMT_NF4>(epi, xt, nw);
    case FMT_NF4_DQ: return small_of<FMT_NF4_DQ>(epi, xt, nw);
    case FMT_MXFP4: return small_of<FMT_MXFP4>(epi, xt, nw);
    default: return small_of<FMT_NVFP4>(epi, xt, nw);
  }
}

const void *small_z_kernel() { return addr(small::k_small_z); }

const void *act_dz_kernel(int projections, int tj) {
  if (projections == 2) {
    switch (tj) {
      case 1: return addr(actbwd::k_act_dz<2, 1>);
      case 2: return addr(actbwd::k_act_dz<2, 2>);
      case 4: return addr(actbwd::k_act_dz<2, 4>);
      default: return addr(actbwd::k_act_dz<2, 8>);
    }
  }
  switch (tj) {
    case 1: return addr(actbwd::k_act_dz<1, 1>);
    case 2: return addr(actbwd::k_act_dz<1, 2>);
    case 4: return addr(actbwd::k_act_dz<1, 4>);
    case 8: return addr(actbwd::k_act_dz<1, 8>);
    default: return addr(actbwd::k_act_dz<1, 16>);
  }
}

const void *col_part_kernel() { return addr(actbwd::k_col_part); }
const void *col_sum_slots_kernel() { return addr(actbwd::k_col_sum_slots); }

const void *dgrad_split_kernel(int fmt) {
  switch (fmt) {
    case FMT_NF4: return addr(dgrad::k_gemm_dgrad<FMT_NF4, false, false, true>);
    case FMT_NF4_DQ: return addr(dgrad::k_gemm_dgrad<FMT_NF4_DQ, false, true, true>);
    case FMT_MXFP4: return addr(dgrad::k_gemm_dgrad<FMT_MXFP4, false, false, true>);
    default: return addr(dgrad::k_gemm_dgrad<FMT_NVFP4, false, false, true>);
  }
}

}  // namespace ffn
}  // namespace lora4
