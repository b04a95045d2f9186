// The orthogonalised update's products, between its two files.
#pragma once
#include <cuda_fp16.h>

#include "linear_internal.h"

namespace mhc {

constexpr float kNsScale = 4096.f;                  // what every matrix is held times
constexpr float kNsMostUnit = 16.f;                 // what a is below: P has it on its diagonal, and fp16 holds kNsScale times that
constexpr int kNsMostCtas = 152;                    // that share a product, at most an item each, or a pair of them
// Scratch of the products: parts of split sums ([CTAs][tile columns, 256 at most][128]), and counters.
constexpr size_t kNsPartsBytes = static_cast<size_t>(kNsMostCtas) * 256 * 128 * 4;
constexpr size_t kNsCounters = 32 + 10 * kNsMostCtas;

// a I + b A + c A A = c (A + h I)^2 + (a - c h^2) I with h = b / 2c: A is kept with h on its diagonal, and is not
// read again. Where c h^2 is far above the coefficients that would cancel, and b A is added instead.
struct NsPolynomial {
    float of_square, of_a, shift, of_unit;          // of A A, of A; what A has on its diagonal, and the result
};
inline NsPolynomial ns_polynomial(float a, float b, float c, bool may_complete) {
    const double h = c != 0.f ? b / (2. * c) : 0., square = c * h * h;
    const double size = (a < 0.f ? -a : a) + (b < 0.f ? -b : b) + (c < 0.f ? -c : c);
    if (may_complete && c != 0.f && (square < 0. ? -square : square) <= 4. * size && (h < 0. ? -h : h) <= 8.)
        return {c, 0.f, static_cast<float>(h), static_cast<float>(a - square)};
    return {c, b, 0.f, a};
}

struct NsCall {
    int batch, m, n, steps;
    float a, b, c;
    __half *x[2][2], *mat[4][2];                    // X in turn, matrices [p][p]; hi and lo
    long long x_pitch, x_size, p_pitch, p_size;
    void *out;
    int out_dtype;
    float *parts;
    unsigned int *counters;                         // zero
};
// A side of at most 128 and the other of at most 2048 (64: 4096, 32: 8192) by a cluster of at most `ctas` CTAs, 16 of them where the
// device holds such a cluster.
bool ns_small_fits_in(int m, int n, int ctas);
bool ns_small_fits(int m, int n);
int launch_ns_small(const OrthogonalArgs &a, const NsPolynomial &f, unsigned int *status, bool pdl, cudaStream_t s);
int launch_ns(const NsCall &c, unsigned int *status, cudaStream_t s);

}  // namespace mhc
