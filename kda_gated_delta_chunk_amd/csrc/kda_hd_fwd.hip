// Linear attention with one decay per head: the forward pass and the increments of the segments' states.
#include "kda_hd_core.hpp"

namespace kda {
namespace hd {
namespace {
template <bool BF, int KD, int VT>
hipError_t fwd_kv(const CoreArgs &a, hipStream_t st) {
    const dim3 grid = grid_of(a, a.tiles);
    hipLaunchKernelGGL((kda_hd_fwd_kernel<BF, KD, VT>), grid, dim3(VT * 4), 0, st, a);
    return hipGetLastError();
}
template <bool BF, int KD>
hipError_t fwd_k(const CoreArgs &a, int vt, hipStream_t st) {
    if (vt == 32) return fwd_kv<BF, KD, 32>(a, st);
    if (vt == 64) return fwd_kv<BF, KD, 64>(a, st);
    if constexpr (BF) return fwd_kv<BF, KD, 128>(a, st);
    return hipErrorInvalidValue;
}
template <bool BF>
hipError_t fwd_b(const CoreArgs &a, int K, int vt, hipStream_t st) {
    return K == 32 ? fwd_k<BF, 32>(a, vt, st) : K == 64 ? fwd_k<BF, 64>(a, vt, st) : fwd_k<BF, 128>(a, vt, st);
}
template <bool BF, int KD, int VT>
hipError_t inc_kv(const CoreArgs &f, const CoreArgs *r, hipStream_t st) {
    const dim3 grid = grid_of(f, r ? 2 * f.tiles : f.tiles);
    hipLaunchKernelGGL((kda_hd_inc_kernel<BF, KD, VT>), grid, dim3(VT * 4), 0, st, f, r ? *r : f, (int)(r != nullptr));
    return hipGetLastError();
}
template <bool BF>
hipError_t inc_b(const CoreArgs &f, const CoreArgs *r, int K, int vt, hipStream_t st) {
    if (vt == 32)
        return K == 32 ? inc_kv<BF, 32, 32>(f, r, st) : K == 64 ? inc_kv<BF, 64, 32>(f, r, st) : inc_kv<BF, 128, 32>(f, r, st);
    return K == 32 ? inc_kv<BF, 32, 64>(f, r, st) : K == 64 ? inc_kv<BF, 64, 64>(f, r, st) : inc_kv<BF, 128, 64>(f, r, st);
}
}  // namespace
hipError_t fwd_pass(bool bf16, const CoreArgs &a, int K, int vt, hipStream_t st) {
    return bf16 ? fwd_b<true>(a, K, vt, st) : fwd_b<false>(a, K, vt, st);
}
hipError_t inc_pass(bool bf16, const CoreArgs &f, const CoreArgs *r, int K, int vt, hipStream_t st) {
    return bf16 ? inc_b<true>(f, r, K, vt, st) : inc_b<false>(f, r, K, vt, st);
}
}  // namespace hd
}  // namespace kda
