// The gated delta rule with one decay per head: the gradients, bf16 I/O beside fp32 gates.
#include "kda_gd_grad.hpp"

namespace kda {
namespace gd {
hipError_t grad_pass_bf16_gates_fp32(const GradArgs &a, int K, int V, bool y_fp32, hipStream_t st) {
    return y_fp32 ? grad_by_k<true, true, 3>(a, K, V, st) : grad_by_k<true, false, 3>(a, K, V, st);
}
}  // namespace gd
}  // namespace kda
