// Driver of the gated delta rule's, the rotary axes' and the checkpoints' host code under AddressSanitizer: entry points
// with rejected arguments, the workspace queries over many sizes, and, on a host without a GPU, valid arguments up to the
// device check.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>

#include "../../include/kda.h"

static int checks = 0;
#define CHECK(x)                                              \
    do {                                                      \
        ++checks;                                             \
        if (!(x)) {                                           \
            printf("failed: %s (line %d)\n", #x, __LINE__);   \
            exit(1);                                          \
        }                                                     \
    } while (0)

int main(int argc, char **) {  // an argument: there is a GPU, no valid calls on these addresses
    const bool run_valid = argc == 1;
    char *p = (char *)(1 << 20);
    const size_t M = 1 << 24;
    auto at = [&](int i) { return (void *)(p + i * M); };
    auto f = [&](int i) { return (float *)at(i); };
    auto ok = [&](kda_status_t s) { return s == KDA_ERROR_NO_DEVICE; };
    for (int io = -1; io <= 2; ++io)
        for (int64_t T : {(int64_t)-1, (int64_t)0, (int64_t)1, (int64_t)4097, (int64_t)1 << 20, (int64_t)1 << 31})
            for (int H : {0, 1, 6, 96, 1 << 16})
                for (int Hk : {0, 1, 3, 4})
                    for (int K : {0, 32, 96, 128})
                        for (int N : {0, 1, 7})
                            for (int packed : {0, 1}) {
                                const size_t a = kda_gd_chunk_fwd_workspace_bytes(1, T, H, Hk, K, 64, N, packed,
                                                                                  (kda_dtype_t)io);
                                const size_t b = kda_gd_chunk_bwd_workspace_bytes(1, T, H, Hk, K, 64, N, packed,
                                                                                  (kda_dtype_t)io);
                                CHECK((a == 0) == (b == 0) && a <= b);
                            }
    CHECK(kda_gd_chunk_fwd(nullptr, at(1), at(2), at(3), at(4), nullptr, nullptr, 1, 64, 4, 2, 32, 64, 1, KDA_DTYPE_BF16,
                           KDA_DTYPE_BF16, 1.f, at(5), f(6), at(7), M, nullptr) == KDA_ERROR_INVALID_VALUE);
    CHECK(kda_gd_chunk_bwd(at(0), at(1), at(2), at(3), at(4), nullptr, nullptr, at(5), nullptr, 1, 64, 4, 2, 32, 96, 1,
                           KDA_DTYPE_BF16, KDA_DTYPE_FP32, 1.f, at(6), at(7), at(8), at(9), at(10), f(11), at(12), M,
                           nullptr) == KDA_ERROR_NOT_SUPPORTED);
    CHECK(kda_gd_decode_step(at(0), at(1), at(2), at(3), at(4), f(5), at(5), 2, 4, 2, 32, 64, KDA_DTYPE_BF16,
                             KDA_DTYPE_BF16, 1.f, nullptr) == KDA_ERROR_INVALID_VALUE);
    CHECK(kda_rotary_axes(at(0), nullptr, (double *)at(2), (int32_t *)at(3), (int32_t *)at(4), at(5), nullptr, 8, 17, 4, 0,
                          64, 64, KDA_DTYPE_BF16, KDA_ROTARY_HALF, 0, 1.f, nullptr) == KDA_ERROR_NOT_SUPPORTED);
    CHECK(kda_checkpoint8_save(at(0), (int8_t *)at(0), f(2), 4, 33, KDA_DTYPE_BF16, nullptr) == KDA_ERROR_INVALID_VALUE);
    CHECK(kda_checkpoint8_restore((int8_t *)at(0), f(1), at(2), 4, 0, KDA_DTYPE_BF16, nullptr) == KDA_ERROR_INVALID_VALUE);
    CHECK(kda_layer_norm_bwd_checkpoint8(at(0), (int8_t *)at(1), f(2), f(3), f(4), at(5), at(6), f(7), f(8), nullptr, 6, 3,
                                         33, 1e-5f, 1, KDA_DTYPE_BF16, at(9), M, nullptr) == KDA_ERROR_INVALID_VALUE);
    if (run_valid) {
        CHECK(ok(kda_gd_chunk_fwd(at(0), at(1), at(2), at(3), at(4), nullptr, nullptr, 1, 64, 4, 2, 32, 64, 1,
                                  KDA_DTYPE_BF16, KDA_DTYPE_FP32, 1.f, at(5), f(6), at(7), M, nullptr)));
        CHECK(ok(kda_gd_chunk_bwd(at(0), at(1), at(2), at(3), at(4), nullptr, nullptr, at(5), nullptr, 1, 64, 4, 2, 32, 64,
                                  1, KDA_DTYPE_BF16, KDA_DTYPE_BF16, 1.f, at(6), at(7), at(8), at(9), at(10), f(11),
                                  at(12), M, nullptr)));
        CHECK(ok(kda_gd_decode_step(at(0), at(1), at(2), at(3), at(4), f(5), at(6), 2, 4, 2, 32, 64, KDA_DTYPE_FP32,
                                    KDA_DTYPE_FP32, 1.f, nullptr)));
        CHECK(ok(kda_rotary_axes(at(0), at(1), (double *)at(2), (int32_t *)at(3), (int32_t *)at(4), at(0), at(1), 8, 3, 4,
                                 2, 64, 64, KDA_DTYPE_BF16, KDA_ROTARY_INTERLEAVED, 1, 1.f, nullptr)));
        CHECK(ok(kda_checkpoint8_save(at(0), (int8_t *)at(1), f(2), 4, 33, KDA_DTYPE_BF16, nullptr)));
        CHECK(ok(kda_checkpoint8_restore((int8_t *)at(0), f(1), at(2), 4, 33, KDA_DTYPE_FP32, nullptr)));
        CHECK(ok(kda_layer_norm_bwd_checkpoint8(at(0), (int8_t *)at(1), f(2), f(3), f(4), at(5), at(6), f(7), f(8), at(9),
                                                6, 3, 33, 1e-5f, 1, KDA_DTYPE_BF16, at(10), M, nullptr)));
    }
    printf("all checks passed (%d)\n", checks);
    return 0;
}
