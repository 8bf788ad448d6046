// Instantiations of the attention kernels (attn.hpp).
#include "attn.hpp"

namespace lora4 {
namespace attn {

namespace {
template <typename K>
const void *addr(K *k) {
  return reinterpret_cast<const void *>(k);
}
}  // namespace

int col_blocks(int D) { return D <= 64 ? 2 : D <= 96 ? 3 : 4; }

const void *fwd_kernel(int dc) {
  return dc == 2 ? addr(k_attn_fwd<2>) : dc == 3 ? addr(k_attn_fwd<3>) : addr(k_attn_fwd<4>);
}
const void *join_kernel() { return addr(k_attn_join); }
const void *dq_kernel(int dc) {
  return dc == 2 ? addr(k_attn_dq<2>) : dc == 3 ? addr(k_attn_dq<3>) : addr(k_attn_dq<4>);
}
const void *dkv_kernel(int dc) {
  return dc == 2 ? addr(k_attn_dkv<2>) : dc == 3 ? addr(k_attn_dkv<3>) : addr(k_attn_dkv<4>);
}
const void *dkv_sum_kernel() { return addr(k_attn_dkv_sum); }

}  // namespace attn
}  // namespace lora4
