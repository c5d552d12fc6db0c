// The gated delta rule with one decay per head: the gradients, fp32 I/O.
#include "kda_gd_grad.hpp"

namespace kda {
namespace gd {
hipError_t grad_pass_fp32(const GradArgs &a, int K, int V, hipStream_t st) { return grad_by_k<false, true, 2>(a, K, V, st); }
}  // namespace gd
}  // namespace kda
