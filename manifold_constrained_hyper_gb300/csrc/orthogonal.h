// The orthogonalised update's products, between its two files.
#pragma once
#include <cuda_fp16.h>

#include "linear_internal.h"

namespace mhc {

constexpr float kNsScale = 4096.f;                  // what every matrix is held times
constexpr int kNsMostPairs = 76;                    // pairs of CTAs that share a product
// Scratch of the products: parts of split sums ([items][2][tile columns][128], at most an item a pair and
// 256 columns), and counters.
constexpr size_t kNsPartsBytes = static_cast<size_t>(kNsMostPairs) * 2 * 256 * 128 * 4;
constexpr size_t kNsCounters = 32 + 13 * 2 * kNsMostPairs;

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
int launch_ns(const NsCall &c, unsigned int *status, cudaStream_t s);

}  // namespace mhc
