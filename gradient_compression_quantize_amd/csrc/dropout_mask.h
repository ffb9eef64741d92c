// dropout_mask.h -- the dropout mask as a function of (seed, worker, index):
// shared by the dropout kernels and the norm/residual kernels.
//
// Value i takes word i mod 4 of Philox4x32-10(key = seed, counter =
// (i/4 low, i/4 high, worker, 2)); u_i = (r >> 8) * 2^-24, the uniform of the
// stochastic rounding, and the value is kept where u_i >= p. As integers:
// r >= ceil(p * 2^24) * 2^8. The mask is drawn again wherever it is needed,
// so it costs no memory; it does not depend on the values or their type.
#pragma once

#include <cmath>

#include "philox.h"
#include "values.h"

namespace gcq {
namespace {

constexpr uint32_t kPurposeDropout = 2;

// What a launch needs to know of a mask. `step`, if not NULL, is a device
// counter added to the seed, so that a captured launch draws a new mask at
// every replay.
struct DropoutArgs {
    uint32_t cut;  // kept where r >= cut
    bool some;     // whether anything can be dropped (cut > 0)
    bool all;      // p = 1: everything is, whatever the draw
    float scale;   // 1 / (1 - p) rounded once
    uint32_t worker;
    uint64_t seed;
    const uint64_t* step;
};

inline bool dropout_p_ok(double p) { return p >= 0.0 && p <= 1.0; }

inline DropoutArgs dropout_args(double p, uint64_t seed, uint32_t worker, const uint64_t* step)
{
    DropoutArgs a;
    a.all = std::ceil(p * 16777216.0) >= 16777216.0;
    a.cut = a.all ? 0xFFFFFFFFu : uint32_t(std::ceil(p * 16777216.0)) << 8;
    a.some = a.cut > 0;
    a.scale = a.all ? 0.0f : float(1.0 / (1.0 - p));
    a.worker = worker;
    a.seed = seed;
    a.step = step;
    return a;
}

__device__ __forceinline__ uint64_t dropout_key(const DropoutArgs& a)
{
    return a.step ? a.seed + *a.step : a.seed;
}

// The words of a slot; of p = 1, words that drop everything.
__device__ __forceinline__ U4 dropout_words(const DropoutArgs& a, uint64_t key, uint64_t slot)
{
    if (a.all)
        return U4{0, 0, 0, 0};
    return philox4x32_10(U4{uint32_t(slot), uint32_t(slot >> 32), a.worker, kPurposeDropout},
                         uint32_t(key), uint32_t(key >> 32));
}

// x * scale where kept, else 0 (whatever x holds).
__device__ __forceinline__ float dropout_apply(const DropoutArgs& a, uint32_t r, float x)
{
    return r >= a.cut ? x * a.scale : 0.0f;
}

// The word of value i alone.
__device__ __forceinline__ uint32_t dropout_word(const DropoutArgs& a, uint64_t key, uint64_t i)
{
    const U4 r = dropout_words(a, key, i >> 2);
    const uint32_t lo = (i & 1) ? r.y : r.x, hi = (i & 1) ? r.w : r.z;
    return (i & 2) ? hi : lo;
}

}  // namespace
}  // namespace gcq
