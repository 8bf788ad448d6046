// Host side of attention (included by lora4.hip behind its dispatch helpers):
// validation, workspace layout and launch order.
//
//   forward  : k_attn_fwd, over ranges of the keys where the row tiles alone do
//              not fill the chip, then k_attn_join
//   backward : k_attn_dq (and delta) -> k_attn_dkv (over ranges of the rows
//              where the key tiles do not fill the chip, then k_attn_dkv_sum)
#pragma once

namespace {

struct AttnPlan {
  int dc;
  int64_t slots, kslots;   // tiles of packed rows, and of keys
  int splits, ksplits;     // forward's key ranges, dK and dV's row ranges
  size_t off_part, bytes;
};

lora4_status check_attn_sizes(int64_t Tq, int64_t Tk, int64_t seqs, int32_t Hq, int32_t Hkv, int32_t D) {
  if (Tq < 0 || Tk < 0 || seqs < 1 || seqs > (1 << 20) || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > 64 ||
      D < 8 || D % 8 != 0)
    return LORA4_ERR_SHAPE;
  if (D > 128) return LORA4_ERR_UNIMPLEMENTED;
  const int64_t G = Hq / Hkv;
  // 32-bit packed rows (also exactly divided by G with one multiplication) and keys
  if (Hq > 65535 || Tq > (int64_t(1) << 30) || Tk > (int64_t(1) << 30) || Tq * Hq >= (int64_t(1) << 31) ||
      (Tq * G + attn::ROWS) * G >= (int64_t(1) << 32))
    return LORA4_ERR_SHAPE;
  return LORA4_OK;
}

// Blocks that keep the chip busy: two a CU.
int64_t attn_full_grid() { return 2 * (int64_t)cu_count(); }

AttnPlan attn_plan(int which, int64_t Tq, int64_t Tk, int64_t seqs, int Hq, int Hkv, int D) {
  AttnPlan pl{};
  const int64_t G = Hq / Hkv;
  pl.dc = attn::col_blocks(D);
  // every sequence may end with a tile that is not full
  pl.slots = std::min(Tq * G / attn::ROWS + seqs, Tq * G);
  pl.kslots = std::min(Tk / attn::BKEYS + seqs, Tk);
  pl.splits = pl.ksplits = 1;
  const int64_t keys = Tk / seqs, rows = Tq * G / seqs;   // the lengths are on the device: means
  if (which == 0) {
    const int64_t blocks = std::max<int64_t>(1, std::max(Tq * G / attn::ROWS, std::min(seqs, Tq)) * Hkv);
    const int64_t most = std::max<int64_t>(1, keys / (4 * attn::KEYS));
    // Single tokens (rows of one wave) over caches of different fill: eight blocks a
    // CU, so that a long cache does not end last (24 tokens over 5 to 32 thousand keys,
    // 64 heads: 367 us, with two a CU 429). Else two, more only add to the join
    // (3 chunks of 333 tokens, 14 heads: 36 us, with four a CU 40, with one 43).
    const int64_t full = (rows <= 32 ? 4 : 1) * attn_full_grid();
    pl.splits = (int)std::min<int64_t>(std::min<int64_t>(attn::MAX_SPLITS, most), std::max<int64_t>(1, full / blocks));
    pl.bytes = 256;
    if (pl.splits > 1) {
      pl.off_part = align256((size_t)pl.splits * Tq * Hq * 8);
      pl.bytes = std::max(pl.bytes, pl.off_part + align256((size_t)pl.splits * Tq * Hq * D * 4));
    }
  } else {
    const int64_t blocks = std::max<int64_t>(1, std::max(Tk / attn::BKEYS, std::min(seqs, Tk)) * Hkv);
    // Ranges of at least eight steps, as each costs its partials; where the blocks are
    // fewer than the CUs, of at least two (a sequence of 531 tokens, 32 over 8 heads: 4
    // ranges 65 us, 8 56; three of together 531: 1 range 56, 2 46, 5 42).
    const int64_t steps = rows / attn::BROWS;
    const int64_t most = std::max<int64_t>({1, steps / 8, std::min(steps / 2, cu_count() / blocks)});
    // Four blocks a CU where the key tiles give fewer: the first keys of a sequence
    // are seen by all of its rows, the last by few, and the long blocks start first
    // (packed 4096 tokens, 8 key heads: 1, 2, 4, 8 ranges 195, 141, 119, 141 us, their
    // sums 0, 14, 24, 56). One more where it leaves each 256 steps, whose partials
    // are little beside them (8192 tokens, 64 heads: 2 ranges 2481 + 29, 3 2327 + 42).
    pl.ksplits = (int)std::min<int64_t>(std::min<int64_t>(16, most),
                                        std::max<int64_t>(1, ceil_div(2 * attn_full_grid(), blocks)));
    if (steps / (pl.ksplits + 1) >= 256) ++pl.ksplits;
    pl.off_part = align256((size_t)std::max<int64_t>(1, Tq * Hq) * 8);
    pl.bytes = pl.off_part + (pl.ksplits > 1 ? align256((size_t)pl.ksplits * 2 * Tk * Hkv * D * 4) : 0);
  }
  return pl;
}

size_t attn_workspace(int which, int64_t Tq, int64_t Tk, int64_t seqs, int32_t Hq, int32_t Hkv, int32_t D) {
  if (check_attn_sizes(Tq, Tk, seqs, Hq, Hkv, D) != LORA4_OK) return 0;
  return attn_plan(which, Tq, Tk, seqs, Hq, Hkv, D).bytes;
}

bool bad_stride(int64_t ld, int64_t width) { return ld < width || ld % 8 != 0 || ld > (1 << 22); }

lora4_status check_attn(const lora4_attn *a) {
  if (!a) return LORA4_ERR_NULL;
  TRY(check_attn_sizes(a->Tq, a->Tk, a->seqs, a->Hq, a->Hkv, a->D));
  // (the kernels take scale log2 e)
  if (!(a->scale > 0.0f) || !std::isfinite(a->scale * attn::LOG2E)) return LORA4_ERR_SHAPE;
  const int64_t wq = (int64_t)a->Hq * a->D, wk = (int64_t)a->Hkv * a->D;
  if (bad_stride(a->ldq, wq) || bad_stride(a->ldk, wk) || bad_stride(a->ldv, wk)) return LORA4_ERR_SHAPE;
  if (!a->q_offsets && a->seqs != 1) return LORA4_ERR_NULL;
  if (a->q_offsets && !a->k_offsets && a->Tk != a->Tq) return LORA4_ERR_SHAPE;
  if (!a->q_offsets && a->k_offsets) return LORA4_ERR_SHAPE;   // both or the queries' alone
  return LORA4_OK;
}

attn::Params attn_params(const lora4_attn *a, const uint16_t *Q, const uint16_t *K, const uint16_t *V) {
  attn::Params p{};
  p.Q = Q;
  p.K = K;
  p.V = V;
  p.ldq = a->ldq;
  p.ldk = a->ldk;
  p.ldv = a->ldv;
  p.Tq = a->Tq;
  p.Tk = a->Tk;
  p.seqs = (int)a->seqs;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.G = a->Hq / a->Hkv;
  p.D = a->D;
  p.gmagic = p.G == 1 ? 0u : (uint32_t)(((uint64_t(1) << 32) + p.G - 1) / p.G);
  p.gone = p.G == 1 ? ~0u : 0u;
  p.scale = a->scale;
  p.qo = a->q_offsets;
  p.ko = a->k_offsets ? a->k_offsets : a->q_offsets;
  p.kl = a->k_lengths;
  p.splits = 1;
  return p;
}

// LDS of a step's two tiles, twice, and (dK, dV) the rows' statistics.
size_t attn_lds(int dc, bool stats) {
  return (size_t)4 * 64 * (dc <= 2 ? 128 : 256) + (stats ? 2 * 2 * attn::BROWS * 4 : 0);
}

lora4_status attn_forward(const lora4_attn *a, const uint16_t *Q, const uint16_t *K, const uint16_t *V, uint16_t *O,
                          float *lse, void *ws, size_t ws_bytes, hipStream_t st) {
  TRY(check_attn(a));
  if (a->Tq == 0) return LORA4_OK;
  if (!Q || !O || (a->Tk > 0 && (!K || !V))) return LORA4_ERR_NULL;
  if (!all_aligned16({Q, K, V, O, lse, a->q_offsets, a->k_offsets, a->k_lengths, ws})) return LORA4_ERR_ALIGN;
  const AttnPlan pl = attn_plan(0, a->Tq, a->Tk, a->seqs, a->Hq, a->Hkv, a->D);
  if (!ws || ws_bytes < pl.bytes) return LORA4_ERR_WORKSPACE;
  attn::Params p = attn_params(a, Q, K, V);
  p.O = O;
  p.lse = lse;
  p.slots = (int)pl.slots;
  p.splits = pl.splits;
  p.part_ml = ws_at<float>(ws, 0);
  p.part = ws_at<float>(ws, pl.off_part);
  TRY(launch_fn("attn_fwd", attn::fwd_kernel(pl.dc), pl.slots * a->Hkv * pl.splits, attn::THREADS,
                attn_lds(pl.dc, false), st, p));
  if (pl.splits == 1) return LORA4_OK;
  return launch_fn("attn_join", attn::join_kernel(), ceil_div(a->Tq * a->Hq, 4), attn::THREADS, 0, st, p);
}

lora4_status attn_backward(const lora4_attn *a, const uint16_t *Q, const uint16_t *K, const uint16_t *V,
                           const uint16_t *O, const float *lse, const uint16_t *dO, uint16_t *dQ, uint16_t *dK,
                           uint16_t *dV, int64_t lddq, int64_t lddk, int64_t lddv, void *ws, size_t ws_bytes,
                           hipStream_t st) {
  TRY(check_attn(a));
  const int64_t wq = (int64_t)a->Hq * a->D, wk = (int64_t)a->Hkv * a->D;
  if (bad_stride(lddq, wq) || bad_stride(lddk, wk) || bad_stride(lddv, wk)) return LORA4_ERR_SHAPE;
  if ((a->Tq > 0 && (!Q || !O || !lse || !dO || !dQ)) || (a->Tk > 0 && (!K || !V || !dK || !dV))) return LORA4_ERR_NULL;
  if (!all_aligned16({Q, K, V, O, lse, dO, dQ, dK, dV, a->q_offsets, a->k_offsets, a->k_lengths, ws}))
    return LORA4_ERR_ALIGN;
  const AttnPlan pl = attn_plan(1, a->Tq, a->Tk, a->seqs, a->Hq, a->Hkv, a->D);
  // (no grid is refused after another was launched)
  if (pl.slots * a->Hkv > INT32_MAX || pl.kslots * a->Hkv * pl.ksplits > INT32_MAX) return LORA4_ERR_SHAPE;
  if (!ws || ws_bytes < pl.bytes) return LORA4_ERR_WORKSPACE;
  attn::Params p = attn_params(a, Q, K, V);
  p.lse = const_cast<float *>(lse);
  p.dO = dO;
  p.Oin = O;
  p.stat = ws_at<float>(ws, 0);
  p.dQ = dQ;
  p.dK = dK;
  p.dV = dV;
  p.lddq = lddq;
  p.lddk = lddk;
  p.lddv = lddv;
  p.part = ws_at<float>(ws, pl.off_part);
  if (a->Tq > 0) {
    p.slots = (int)pl.slots;
    TRY(launch_fn("attn_dq", attn::dq_kernel(pl.dc), pl.slots * a->Hkv, attn::THREADS, attn_lds(pl.dc, false), st, p));
  }
  if (a->Tk == 0) return LORA4_OK;
  p.slots = (int)pl.kslots;
  p.splits = pl.ksplits;
  TRY(launch_fn("attn_dkv", attn::dkv_kernel(pl.dc), pl.kslots * a->Hkv * pl.ksplits, attn::THREADS,
                attn_lds(pl.dc, true), st, p));
  if (pl.ksplits == 1) return LORA4_OK;
  // blocks of 16 keys, or of parts of their columns where those are few (1024 tokens,
  // 32 over 8 heads, 8 ranges: the backward 112 us without parts, 84 with)
  const int64_t blocks = a->Tk / 16 + a->seqs;
  const int64_t parts = std::min(ceil_div(16 * wk, 4 * attn::THREADS), ceil_div(8 * cu_count(), blocks));
  return launch_grid("attn_dkv_sum", attn::dkv_sum_kernel(), dim3((unsigned)blocks, (unsigned)parts), attn::THREADS, 0,
                     st, p);
}

}  // namespace
