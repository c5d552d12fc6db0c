// Linear attention with one decay per head: the gradients, bf16 I/O.
#include "kda_hd_core.hpp"

namespace kda {
namespace hd {
namespace {
template <int K, int V, int VT, bool DG, bool YF>
hipError_t launch(const GradArgs &g, hipStream_t st) {
    const dim3 grid = grid_of(g.dv, g.dv.tiles + 2 * g.dk.tiles);
    hipLaunchKernelGGL((kda_hd_grad_kernel<true, K, V, VT, DG, YF>), grid, dim3(VT * 4), 0, st, g);
    return hipGetLastError();
}
template <int K, int V>
hipError_t by_kind(const GradArgs &g, bool dg, bool y_fp32, hipStream_t st) {
    constexpr int VT = grad_tile(K, V, true);
    if (y_fp32) return dg ? launch<K, V, VT, true, true>(g, st) : launch<K, V, VT, false, true>(g, st);
    return dg ? launch<K, V, VT, true, false>(g, st) : launch<K, V, VT, false, false>(g, st);
}
template <int K>
hipError_t by_v(const GradArgs &g, int V, bool dg, bool y_fp32, hipStream_t st) {
    return V == 32 ? by_kind<K, 32>(g, dg, y_fp32, st) : V == 64 ? by_kind<K, 64>(g, dg, y_fp32, st) : by_kind<K, 128>(g, dg, y_fp32, st);
}
}  // namespace
hipError_t grad_pass_bf16(const GradArgs &g, int K, int V, bool dg, bool y_fp32, hipStream_t st) {
    return K == 32 ? by_v<32>(g, V, dg, y_fp32, st) : K == 64 ? by_v<64>(g, V, dg, y_fp32, st) : by_v<128>(g, V, dg, y_fp32, st);
}
}  // namespace hd
}  // namespace kda
