// Instantiations of the vocabulary loss's kernels (loss.hpp).
#include "loss.hpp"

namespace lora4 {
namespace loss {

namespace {
template <typename K>
const void *addr(K *k) {
  return reinterpret_cast<const void *>(k);
}
}  // namespace

const void *rows_kernel() { return addr(k_loss_rows); }
const void *target_kernel(bool find) { return find ? addr(k_loss_target<true>) : addr(k_loss_target<false>); }
const void *logits_kernel(bool grad, bool small) {
  if (small) return grad ? addr(k_loss_logits<true, Small>) : addr(k_loss_logits<false, Small>);
  return grad ? addr(k_loss_logits<true, Big>) : addr(k_loss_logits<false, Big>);
}
const void *join_kernel(bool grad, int rows) {
  if (rows == 4) return grad ? addr(k_loss_join<true, 4>) : addr(k_loss_join<false, 4>);
  return grad ? addr(k_loss_join<true, 32>) : addr(k_loss_join<false, 32>);
}
const void *dx_kernel(bool small) { return small ? addr(k_loss_dx<Small>) : addr(k_loss_dx<Big>); }
const void *finish_kernel() { return addr(k_loss_finish); }
const void *total_kernel() { return addr(k_loss_total); }

}  // namespace loss
}  // namespace lora4
