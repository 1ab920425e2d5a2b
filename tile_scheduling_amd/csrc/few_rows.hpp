// The product with a fused epilogue for few rows of A (one token, a small decoding batch):
// bound by reading B once.  Declarations; kernels in few_rows.hip.
#pragma once

#include "epilogue.hpp"

namespace ts {

constexpr int kFewRows = 32;   // largest M of these kernels, but for int8 operands
// Largest M with int8 operands as well: with more rows, as far as the rows of A, which every workgroup reads, cost less than
// tiles that leave most CUs idle (figures at many_kernel, few_rows.hip).
inline int few_rows_most(bool int8, long long N, long long K) {
    return int8 && N <= 8192 ? (K <= 2048 ? 128 : K <= 4096 ? 64 : kFewRows) : kFewRows;
}

struct FewArgs {
    const void *A, *B;
    void* C;
    int M, N, K;
    long long lda, ldb, ldc;   // elements; A [M][K]; B [N][K] or [K][N]
    const void *bias, *aux_in;
    void* aux_out;
    long long ld_in, ld_out;
    const float *scale_a, *scale_b;
    int bias_type, act, grad;
    int tiles, xcds;           // workgroups; XCDs they are dealt over
    uint8_t* kept;             // preact in 8 bits, as in EpiArgs (16-bit operands)
    long long ld_kept;
};

// Enqueues the kernel for operands of type ab (ELT_*) and C of type c; b_kmaj: B stored [N][K].  False
// if that failed.
bool launch_few_rows(FewArgs& g, int ab, int c, bool b_kmaj, hipStream_t stream);

}  // namespace ts
