// linear_xent.hip -- softmax cross entropy of a linear layer over a large
// vocabulary, and its gradient; the logits are never kept.
//
//   l_nv = <hidden_n, weight_v>,  lse_n = log sum_v exp(l_nv),
//   loss_n = lse_n - l_n,target(n)
//   G_nv = dloss_n (exp(l_nv - lse_n) - [v = target(n)])
//   dhidden = G weight,  dweight = G^T hidden
//
// Loss: one product whose tiles end in the running maximum and sum of their
// part of the vocabulary; a wave for each token joins the parts.
// Gradient: piece by piece of the vocabulary, the logits are computed again
// and turned into G in the tile's registers; G of one piece is the only
// matrix of tokens x vocabulary that is ever in memory, and the two products
// of the gradient read it back.
//
// Bound by the matrix cores and, for narrow models, by what G costs: 8192 x
// 30522 x 768 bf16 takes 361 to 395 us for the loss (0.97 to 1.06 PFLOP/s: six
// turns of k a tile, then its epilogue) and 1.81 to 1.87 ms for a gradient with
// fp32 dweight (a third of it in tiles of G, whose 1 GB of stores no other
// tile's products run under); 8192 x 64000 x 4096 takes 10.7 to 10.9 ms for the
// gradient (1.2 PFLOP/s). A few tokens are bound by bytes: bf16 ones read the
// matrix once (14.5 us for one token of 30522 x 768, floor 9.1), but fp32
// weights, and 16-bit ones with D off a multiple of 128, are copied first.
#include <algorithm>
#include <limits>
#include <string>
#include <type_traits>

#include "mfma_product.h"

namespace gcq {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;       // log2(e) rounded
constexpr float kLog2eRest = 1.92596299112661746887e-8f; // what that rounding left
constexpr float kLn2 = 0.69314718055994530942f;

// exp(x) for x <= 0 (and a little above): 2^(x log2 e) by v_exp_f32, the
// rounding of the product put back as a factor.
__device__ __forceinline__ float exp_neg(float x)
{
    const float hi = x * kLog2e;
    const float lo = __builtin_fmaf(x, kLog2e, -hi) + x * kLog2eRest;
    const float r = __builtin_amdgcn_exp2f(hi);
    return r == 0.0f ? 0.0f : __builtin_fmaf(r, lo * kLn2, r);
}

// Whether row n has a target among the rows of the vocabulary.
__device__ __forceinline__ bool has_target(const int64_t* target, size_t n, int64_t ignore, size_t V)
{
    const int64_t t = target[n];
    return t != ignore && t >= 0 && size_t(t) < V;
}

// ---- operands as planes --------------------------------------------------------

constexpr int kRowThreads = 256, kRowWaves = kRowThreads / kWave;

// A row's values c .. c + 7 (zeros behind d), whatever the alignment.
template <typename T>
__device__ __forceinline__ void load8(const T* row, size_t c, size_t d, float (&v)[8])
{
    typedef T Vec __attribute__((ext_vector_type(8)));
    typedef Vec VecAny __attribute__((aligned(sizeof(T))));
    if (c + 8 <= d) {
        const auto x = __builtin_convertvector(*reinterpret_cast<const VecAny*>(row + c), vec_of<float, 8>);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = x[k];
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        v[k] = c + k < d ? float(row[c + k]) : 0.0f;
}

// max(m, |x|) over the finite ones of eight values
__device__ __forceinline__ float largest_finite(float m, const float (&v)[8])
{
#pragma unroll
    for (int k = 0; k < 8; ++k)
        m = fabsf(v[k]) <= std::numeric_limits<float>::max() ? fmaxf(m, fabsf(v[k])) : m;
    return m;
}

// What the scale of a matrix goes by: the largest finite |x| of its rows (of
// those with a target, if `target` is not NULL), a maximum for each workgroup.
constexpr unsigned kMaxParts = 1024;

struct MaxOf {
    const void* src;
    bool f32;  // else of the inputs' type
    size_t rows, d;
    const int64_t* target;
    float* parts;
    unsigned nparts;
};

// A launch takes the maxima of up to three matrices, and lays out up to two
// and sets an exponent: blockIdx.y says which.
struct MaxOfAll {
    MaxOf of[3];
};

__device__ __forceinline__ float workgroup_max(float m)
{
    __shared__ float lds[kRowWaves];
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1)
        m = fmaxf(m, __shfl_xor(m, off));
    if ((threadIdx.x & (kWave - 1)) == 0)
        lds[threadIdx.x / kWave] = m;
    __syncthreads();
    m = lds[0];
    for (int w = 1; w < kRowWaves; ++w)
        m = fmaxf(m, lds[w]);
    return m;
}

template <typename T>
__device__ __forceinline__ void largest(const MaxOf& a, int64_t ignore, size_t V)
{
    const T* src = static_cast<const T*>(a.src);
    const int lane = threadIdx.x & (kWave - 1);
    float m = 0.0f;
    for (size_t r = size_t(blockIdx.x) * kRowWaves + threadIdx.x / kWave; r < a.rows; r += size_t(a.nparts) * kRowWaves) {
        if (a.target && !has_target(a.target, r, ignore, V))
            continue;
        const T* row = src + r * a.d;
#pragma unroll 2
        for (size_t c = lane * 8; c < a.d; c += kWave * 8) {
            float v[8];
            load8(row, c, a.d, v);
            m = largest_finite(m, v);
        }
    }
    m = workgroup_max(m);
    if (threadIdx.x == 0)
        a.parts[blockIdx.x] = m;
}

template <typename T>
__global__ __launch_bounds__(kRowThreads) void largest_kernel(MaxOfAll all, int64_t ignore, size_t V)
{
    const MaxOf a = blockIdx.y == 0 ? all.of[0] : blockIdx.y == 1 ? all.of[1] : all.of[2];
    if (blockIdx.x >= a.nparts)
        return;
    if (a.f32)
        largest<float>(a, ignore, V);
    else
        largest<T>(a, ignore, V);
}

// src [rows][d] -> planes [rows_out][d_out] (d_out a multiple of 8), one
// behind the other, of bf16 as it is or of fp16, scaled so that the largest
// finite value comes to [2^14, 2^15): that of the matrix where `parts` is not
// NULL, that of each row, with an exponent of its own, where by_row is set.
// Zeros behind the last column and row, and in the rows that have no target if
// `target` is not NULL: what such rows hold, NaN included, reaches nothing. One
// wave a row. Without an `out` only the exponent is set.
struct PlanesOf {
    const void* src;
    size_t rows, d;
    uint16_t* out;
    size_t rows_out, d_out;
    const int64_t* target;
    const float* parts;
    unsigned nparts;
    int* exponent;  // one, or one a row
    bool by_row;
};

// The power of two that brings m, the largest value, to [2^14, 2^15).
__device__ __forceinline__ int exponent_for(float m) { return m > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(m) : 0; }

struct PlanesOfAll {
    PlanesOf of[3];
};

template <typename T, bool kF16, int kPlanes>
__global__ __launch_bounds__(kRowThreads) void planes_kernel(PlanesOfAll all, int64_t ignore, size_t V)
{
    const PlanesOf a = blockIdx.y == 0 ? all.of[0] : blockIdx.y == 1 ? all.of[1] : all.of[2];
    if (size_t(blockIdx.x) * kRowWaves >= std::max<size_t>(a.out ? a.rows_out : 0, 1))
        return;
    int scale = 0;
    if (kF16 && a.parts) {
        float m = 0.0f;
        for (unsigned k = threadIdx.x; k < a.nparts; k += kRowThreads)
            m = fmaxf(m, a.parts[k]);
        m = workgroup_max(m);
        scale = exponent_for(m);
        if (blockIdx.x == 0 && threadIdx.x == 0)
            *a.exponent = scale;
    }
    if (!a.out)
        return;
    const T* src = static_cast<const T*>(a.src);
    const int lane = threadIdx.x & (kWave - 1);
    for (size_t r = size_t(blockIdx.x) * kRowWaves + threadIdx.x / kWave; r < a.rows_out;
         r += size_t(gridDim.x) * kRowWaves) {
        const bool live = r < a.rows && (!a.target || has_target(a.target, r, ignore, V));
        if (kF16 && a.by_row) {
            float m = 0.0f;
            for (size_t c = lane * 8; live && c < a.d; c += kWave * 8) {
                float v[8];
                load8(src + r * a.d, c, a.d, v);
                m = largest_finite(m, v);
            }
#pragma unroll
            for (int off = kWave / 2; off > 0; off >>= 1)
                m = fmaxf(m, __shfl_xor(m, off));
            scale = exponent_for(m);
            if (lane == 0)
                a.exponent[r] = scale;
        }
#pragma unroll 2
        for (size_t c = lane * 8; c < a.d_out; c += kWave * 8) {
            float v[8] = {};
            if (live)
                load8(src + r * a.d, c, a.d, v);
#pragma unroll
            for (int plane = 0; plane < kPlanes; ++plane) {
                s16x8 w;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (!kF16) {
                        w[k] = __builtin_bit_cast(short, bf16_t(v[k]));
                        continue;
                    }
                    if (plane == 0)
                        v[k] = __builtin_amdgcn_ldexpf(v[k], scale);
                    const f16_t h = f16_t(v[k]);
                    w[k] = __builtin_bit_cast(short, h);
                    // an infinity or NaN stays in the first plane alone
                    v[k] = fabsf(float(h)) <= 65504.0f ? (v[k] - float(h)) * 0x1p11f : 0.0f;
                }
                *reinterpret_cast<s16x8*>(a.out + plane * (a.rows_out * a.d_out) + r * a.d_out + c) = w;
            }
        }
    }
}

// What sums of products of scaled operands are multiplied by, as an exponent:
// of row n of b, if its rows have exponents of their own.
__device__ __forceinline__ int unscale(const MatOperand& a, const MatOperand& b, uint32_t n = 0)
{
    return -((a.exponent ? *a.exponent : 0) + (b.exponent ? b.exponent[b.by_row ? n : 0] : 0));
}

// ---- tiles of the logits -------------------------------------------------------

template <bool kF16, int TA, int TB, int WA, int WB>
struct LogitTile {
    using Product = TileProduct<kF16, false, false, TA, TB, WA, WB>;
    static constexpr int kRowsA = TA / WA, kRowsB = TB / WB;  // of one wave
};

struct LossPart {
    float top, sum;  // the maximum, and the sum of exp(l - top)
};

// Vocabulary tile x token tile, of the rows v0 .. v0 + v - 1 of the
// vocabulary, which `weight` begins with; their parts are part0 and on. A
// wave's part of a token's row is kRowsA logits, half of them in each half of
// the wave.
template <bool kF16, int TA, int TB, int WA, int WB>
__global__ __launch_bounds__(WA* WB* kWave, 2) void loss_tiles_kernel(
    MatOperand weight, MatOperand hidden, ProductShape sh, uint32_t N, uint32_t v0, uint32_t v, uint32_t V,
    const int64_t* __restrict__ target, LossPart* __restrict__ parts, uint32_t nparts, uint32_t part0,
    float* __restrict__ target_logit)
{
    using L = LogitTile<kF16, TA, TB, WA, WB>;
    using P = typename L::Product;
    GCQ_TILE_BUFFERS(lds, TA, TB);
    uint32_t ta, tb;
    tile_of(xcd_contiguous(blockIdx.x, gridDim.x), sh.tiles_a, sh.tiles_b, ta, tb);
    typename P::Acc acc;
    P::run(weight, hidden, sh, ta * TA, tb * TB, 0, sh.turns * sh.segments, lds, acc);

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wa = wave % WA, wb = wave / WA;
    const uint32_t a_wave = ta * TA + wa * L::kRowsA;
#pragma unroll
    for (int j = 0; j < P::RB; ++j) {
        const uint32_t n = tb * TB + wb * L::kRowsB + j * 32 + acc_col(lane);
        const int64_t t = n < N ? target[n] : -1;
        if (kF16) {
            const int back = unscale(weight, hidden, min(n, N - 1));
#pragma unroll
            for (int i = 0; i < P::RA; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    acc.v[i][j][e] = __builtin_amdgcn_ldexpf(acc.v[i][j][e], back);
        }
        // the target's place in this wave's part, if it is there: it hardly
        // ever is, and only the last tile reaches past the vocabulary
        const uint32_t at = t >= 0 && t < int64_t(V) ? uint32_t(t) - (v0 + a_wave) : 0xFFFFFFFFu;
        if (__any(at < uint32_t(L::kRowsA))) {
            float mine = 0.0f;
            bool found = false;
#pragma unroll
            for (int i = 0; i < P::RA; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (i * 32 + acc_row(e, lane) == at) {
                        mine = acc.v[i][j][e];
                        found = true;
                    }
            if (found)
                target_logit[n] = mine;
        }
        if (a_wave + L::kRowsA > v) {
            const uint32_t left = v > a_wave ? v - a_wave : 0;
#pragma unroll
            for (int i = 0; i < P::RA; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (i * 32 + acc_row(e, lane) >= left)
                        acc.v[i][j][e] = -INFINITY;
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < P::RA; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                top = fmaxf(top, acc.v[i][j][e]);
        top = fmaxf(top, __shfl_xor(top, 32));
        // exp(l - top) = 2^((l - top) log2 e). The difference comes first: l log2
        // e - top log2 e in one fma is off by the rounding of the second, 2^-24
        // |top| of the sum, and by everything past |top| = 1e9. A part that
        // holds no logit above -inf adds nothing.
        const float ref = top == -INFINITY ? 0.0f : top;
        float sums[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < P::RA; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                sums[e & 3] += __builtin_amdgcn_exp2f((acc.v[i][j][e] - ref) * kLog2e);
        float sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
        sum += __shfl_xor(sum, 32);
        if (lane < 32 && n < N)
            parts[size_t(n) * nparts + part0 + ta * WA + wa] = LossPart{top, sum};
    }
}

// One wave for each token joins the parts of its row. The loss of a token whose
// target leads is log(sum) with a sum near 1, far below lse: the target's logit
// is taken from the maximum, before the logarithm's bits are lost in lse.
constexpr int kJoinThreads = 256;

__global__ __launch_bounds__(kJoinThreads) void loss_join_kernel(
    const LossPart* __restrict__ parts, uint32_t nparts, const float* __restrict__ target_logit,
    const int64_t* __restrict__ target, int64_t ignore, uint32_t N, uint32_t V,
    float* __restrict__ loss, float* __restrict__ lse)
{
    const int lane = threadIdx.x & (kWave - 1);
    for (uint32_t n = blockIdx.x * (kJoinThreads / kWave) + threadIdx.x / kWave; n < N;
         n += gridDim.x * (kJoinThreads / kWave)) {
        float top = -INFINITY, sum = 0.0f;
        for (uint32_t k = lane; k < nparts; k += kWave) {
            const LossPart p = parts[size_t(n) * nparts + k];
            const float both = fmaxf(top, p.top), ref = both == -INFINITY ? 0.0f : both;
            sum = sum * exp_neg(top - ref) + p.sum * exp_neg(p.top - ref);
            top = both;
        }
#pragma unroll
        for (int off = kWave / 2; off > 0; off >>= 1) {
            const float t2 = __shfl_xor(top, off), s2 = __shfl_xor(sum, off);
            const float both = fmaxf(top, t2), ref = both == -INFINITY ? 0.0f : both;
            sum = sum * exp_neg(top - ref) + s2 * exp_neg(t2 - ref);
            top = both;
        }
        if (lane == 0) {
            // (the sum holds exp(0), whatever its rounding left of it)
            const float rest = logf(sum < 1.0f ? 1.0f : sum);
            lse[n] = top + rest;
            const int64_t t = target[n];
            float x = 0.0f;
            if (t != ignore)
                x = t >= 0 && t < int64_t(V) ? (top - target_logit[n]) + rest
                                             : std::numeric_limits<float>::quiet_NaN();
            loss[n] = x;
        }
    }
}

// G of one piece: columns v0 .. of the vocabulary, for rows 0 .. rows_out - 1
// (zeros from N on, and behind the vocabulary). Each wave turns its part of
// the tile into rows of G through LDS, so that the stores are whole rows.
struct GradOut {
    uint16_t* plane0;  // [rows_out][ld]
    size_t plane_stride;
    uint32_t ld, rows_out;
    const int* exponent;  // fp16 planes hold G times 2^exponent
};

// One plane of bf16, or kPlanes of fp16.
template <bool kF16, int TA, int TB, int WA, int WB, int kPlanes>
__global__ __launch_bounds__(WA* WB* kWave, 2) void logit_grad_kernel(
    MatOperand weight, MatOperand hidden, ProductShape sh, uint32_t N, uint32_t v0, uint32_t V,
    const int64_t* __restrict__ target, int64_t ignore, const float* __restrict__ lse,
    const float* __restrict__ dloss, GradOut out)
{
    using L = LogitTile<kF16, TA, TB, WA, WB>;
    using P = typename L::Product;
    GCQ_TILE_BUFFERS(lds, TA, TB);
    uint32_t ta, tb;
    tile_of(xcd_contiguous(blockIdx.x, gridDim.x), sh.tiles_a, sh.tiles_b, ta, tb);
    typename P::Acc acc;
    P::run(weight, hidden, sh, ta * TA, tb * TB, 0, sh.turns * sh.segments, lds, acc);

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wa = wave % WA, wb = wave / WA;
    const uint32_t a_wave = ta * TA + wa * L::kRowsA, b_wave = tb * TB + wb * L::kRowsB;

    const int back = kF16 ? unscale(weight, hidden) : 0, up = kF16 ? *out.exponent : 0;

    // this wave's buffer, for its turn of values into rows
    static_assert(P::kWaves <= kBuffers || (P::kWaves <= 2 * kBuffers && TA == TB), "a buffer for each wave");
    uint16_t* part = lds.a[0];
#pragma unroll
    for (int k = 1; k < P::kWaves; ++k)
        part = wave == k ? (k < kBuffers ? lds.a[k] : lds.b[k - kBuffers]) : part;

#pragma unroll
    for (int j = 0; j < P::RB; ++j) {
        const uint32_t n = b_wave + j * 32 + acc_col(lane);
        bool live = n < N;
        uint32_t at = 0xFFFFFFFFu;  // the target's place in this wave's part
        float z = 0.0f, d = 0.0f;
        if (live) {
            const int64_t tn = target[n];
            live = tn != ignore && tn >= 0 && tn < int64_t(V);
            at = live ? uint32_t(tn) - (v0 + a_wave) : at;
            z = live ? lse[n] : 0.0f;
            d = live ? dloss[n] : 0.0f;
        }
        // p, from the difference l - lse: its error goes by that, and not by the
        // size of lse. In one plane in the end, p takes two roundings of (l -
        // lse) log2 e, 2^-24 of it each, some 1e-6 of p
#pragma unroll
        for (int i = 0; i < P::RA; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float l = kF16 ? __builtin_amdgcn_ldexpf(acc.v[i][j][e], back) : acc.v[i][j][e];
                acc.v[i][j][e] = kPlanes == 1 ? __builtin_amdgcn_exp2f((l - z) * kLog2e) : exp_neg(l - z);
            }
        if (__any(at < uint32_t(L::kRowsA))) {
#pragma unroll
            for (int i = 0; i < P::RA; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    acc.v[i][j][e] -= i * 32 + acc_row(e, lane) == at ? 1.0f : 0.0f;
        }
        // a row without a target holds zeros, whatever its logits were
        if (__any(!live)) {
#pragma unroll
            for (int i = 0; i < P::RA; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    acc.v[i][j][e] = live ? acc.v[i][j][e] : 0.0f;
        }
        if (v0 + a_wave + L::kRowsA > V) {
            const uint32_t left = V > v0 + a_wave ? V - (v0 + a_wave) : 0;
#pragma unroll
            for (int i = 0; i < P::RA; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    acc.v[i][j][e] = i * 32 + acc_row(e, lane) >= left ? 0.0f : acc.v[i][j][e];
        }
#pragma unroll
        for (int i = 0; i < P::RA; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc.v[i][j][e] = kF16 ? __builtin_amdgcn_ldexpf(acc.v[i][j][e] * d, up) : acc.v[i][j][e] * d;
    }
    // this wave's part of 32 tokens at a time, all planes of them
    constexpr int kCols = L::kRowsA, kChunks = kCols / 8;
    constexpr int kPlanePart = 32 * kCols;
    static_assert(kPlanes * kPlanePart <= TA * kStageK, "the planes fit a buffer");
#pragma unroll
    for (int j = 0; j < P::RB; ++j) {
        const int row = int(acc_col(lane));
#pragma unroll
        for (int i = 0; i < P::RA; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = acc.v[i][j][q * 4 + e];
                const int col = i * 32 + 8 * q + 4 * (lane >> 5);
                uint16_t* to = part + row * kCols + ((col >> 3) ^ (row & (kChunks - 1))) * 8 + (col & 4);
#pragma unroll
                for (int plane = 0; plane < kPlanes; ++plane) {
                    s16x4 w;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (!kF16) {
                            w[e] = __builtin_bit_cast(short, bf16_t(x[e]));
                            continue;
                        }
                        const f16_t h = f16_t(x[e]);
                        w[e] = __builtin_bit_cast(short, h);
                        x[e] = (x[e] - float(h)) * 0x1p11f;
                    }
                    *reinterpret_cast<s16x4*>(to + plane * kPlanePart) = w;
                }
            }
        wave_lds_sync();
        constexpr int kRows = kWave / kChunks;
#pragma unroll
        for (int plane = 0; plane < kPlanes; ++plane)
#pragma unroll
            for (int r = 0; r < 32; r += kRows) {
                const int from = r + lane / kChunks, chunk = lane % kChunks;
                const uint32_t n = b_wave + j * 32 + from;
                const s16x8 w = *reinterpret_cast<const s16x8*>(
                    part + plane * kPlanePart + from * kCols + ((chunk ^ (from & (kChunks - 1))) << 3));
                if (n < out.rows_out)
                    *reinterpret_cast<s16x8*>(out.plane0 + plane * out.plane_stride + size_t(n) * out.ld +
                                               a_wave + chunk * 8) = w;
            }
        wave_lds_sync();
    }
}

// ---- the two products of the gradient ----------------------------------------

// Where a product's tiles go: out[b][a], rows of ld values.
template <typename T>
struct ProductOut {
    T* p;
    size_t ld, split_stride;  // split s writes at p + s * split_stride
    uint32_t na, nb;          // valid columns and rows
    bool vec;                 // four values from a multiple of 4 on are aligned to their size
    bool add;                 // onto what is there
};

template <bool kF16, bool kBK, int TA, int TB, int WA, int WB, typename T>
__global__ __launch_bounds__(WA* WB* kWave, 2) void product_kernel(MatOperand A, MatOperand B,
                                                                  ProductShape sh, ProductOut<T> out)
{
    using P = TileProduct<kF16, true, kBK, TA, TB, WA, WB>;
    GCQ_TILE_BUFFERS(lds, TA, TB);
    const uint32_t id = xcd_contiguous(blockIdx.x, gridDim.x);
    const uint32_t tiles = sh.tiles_a * sh.tiles_b, split = id / tiles;
    uint32_t ta, tb;
    tile_of(id - split * tiles, sh.tiles_a, sh.tiles_b, ta, tb);
    const uint64_t all = uint64_t(sh.turns) * sh.segments;
    typename P::Acc acc;
    P::run(A, B, sh, ta * TA, tb * TB, uint32_t(all * split / sh.splits),
           uint32_t(all * (split + 1) / sh.splits), lds, acc);

    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wa = wave % WA, wb = wave / WA;
    const int back = kF16 ? unscale(A, B) : 0;
    T* p = out.p + split * out.split_stride;
#pragma unroll
    for (int j = 0; j < P::RB; ++j) {
        const uint32_t b = tb * TB + wb * (TB / WB) + j * 32 + acc_col(lane);
        if (b >= out.nb)
            continue;
#pragma unroll
        for (int i = 0; i < P::RA; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t a = ta * TA + wa * (TA / WA) + i * 32 + acc_row(4 * q, lane);
                T* o = p + size_t(b) * out.ld + a;
                vec_of<float, 4> w;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = kF16 ? __builtin_amdgcn_ldexpf(acc.v[i][j][q * 4 + e], back) : acc.v[i][j][q * 4 + e];
                if (out.vec && a + 4 <= out.na) {
                    auto* o4 = reinterpret_cast<vec_of<T, 4>*>(o);
                    if (out.add)
                        w += __builtin_convertvector(*o4, vec_of<float, 4>);
                    *o4 = __builtin_convertvector(w, vec_of<T, 4>);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (a + e < out.na)
                            o[e] = T(out.add ? float(o[e]) + w[e] : w[e]);
                }
            }
    }
}

// out[r][c] = sum over splits, in their order, of slab[s][r][c].
constexpr int kSumThreads = 256;

template <typename T>
__global__ __launch_bounds__(kSumThreads) void sum_splits_kernel(const float* __restrict__ slab,
                                                                 size_t ld, size_t split_stride,
                                                                 uint32_t splits, size_t rows, size_t d,
                                                                 T* __restrict__ out)
{
    // four columns a lane: slabs are padded to a multiple of 4
    const size_t quads = ld / 4, total = rows * quads;
    const bool vec = (d & 3) == 0 && (reinterpret_cast<uintptr_t>(out) & (4 * sizeof(T) - 1)) == 0;
    for (size_t q = size_t(blockIdx.x) * kSumThreads + threadIdx.x; q < total;
         q += size_t(gridDim.x) * kSumThreads) {
        const size_t r = q / quads, c = (q - r * quads) * 4;
        vec_of<float, 4> v = *reinterpret_cast<const vec_of<float, 4>*>(slab + r * ld + c);
        for (uint32_t s = 1; s < splits; ++s)
            v += *reinterpret_cast<const vec_of<float, 4>*>(slab + s * split_stride + r * ld + c);
        T* o = out + r * d + c;
        if (vec) {
            *reinterpret_cast<vec_of<T, 4>*>(o) = __builtin_convertvector(v, vec_of<T, 4>);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + e < d)
                    o[e] = T(v[e]);
        }
    }
}

// ---- host side -----------------------------------------------------------------

size_t align256(size_t b) { return (b + 255) & ~size_t(255); }
size_t round_up(size_t a, size_t b) { return ceil_div(a, b) * b; }

// Room for consecutive buffers in a workspace.
struct Carver {
    size_t used = 0;
    size_t take(size_t bytes)
    {
        const size_t at = used;
        used += align256(bytes);
        return at;
    }
};

// Sizes the index arithmetic of the kernels holds: 32-bit tokens, vocabulary
// and channels, 32-bit byte offsets within a tile of 256 rows.
constexpr size_t kMaxTokens = size_t(1) << 28, kMaxVocab = size_t(1) << 28, kMaxChannels = size_t(1) << 20;
constexpr size_t kMaxTiles = size_t(1) << 22, kMaxPiece = size_t(1) << 21;

int check_sizes(const char* what, size_t N, size_t V, size_t D, int dtype)
{
    if (!dtype_bytes(dtype))
        return fail(GC_EINVAL, std::string(what) + ": unknown dtype");
    if (V == 0 || D == 0)
        return fail(GC_EINVAL, std::string(what) + ": the vocabulary and the hidden size must be at least 1");
    if (N > kMaxTokens || V > kMaxVocab || D > kMaxChannels)
        return fail(GC_EUNSUPPORTED, std::string(what) + ": sizes beyond 2^28 tokens, 2^28 rows of the "
                                                         "vocabulary or 2^20 channels");
    // a launch has fewer than 2^32 threads: 2^22 tiles of 256 x 256
    if (ceil_div(N, 256) * ceil_div(V, 256) > kMaxTiles || ceil_div(N, 256) * ceil_div(D, 256) > kMaxTiles ||
        ceil_div(std::min(V, kMaxPiece), 256) * ceil_div(D, 256) > kMaxTiles)
        return fail(GC_EUNSUPPORTED, std::string(what) + ": a product of more than 2^22 tiles of 256 x 256");
    return GC_OK;
}

// How a call computes. bf16 operands are multiplied as they are where no more
// is asked than 16 bits of a gradient; everything else in fp16: fp16 inputs as
// they are, others scaled by a power of two, fp32 ones in two planes. (fp16
// holds a bf16 value exactly down to 2^-31 of the largest one of the matrix,
// and to 2^-39 of that one below.)
struct Mode {
    bool f16;       // matrix products in fp16
    bool scaled;    // inputs scaled, from copies
    int planes;     // of the inputs
};

Mode mode_of(int dtype, bool wide)
{
    if (dtype == GC_BF16 && !wide)
        return Mode{false, false, 1};
    return Mode{true, dtype != GC_F16, dtype == GC_F32 ? 2 : 1};
}

// Whether the product can read the matrix where it is: rows aligned for
// 16-byte loads, whole turns.
bool direct_ok(const void* p, size_t D, const Mode& m) { return !m.scaled && D % kTurnK == 0 && aligned16(p); }

// An operand's planes: the matrix itself, or copies in the workspace, which
// has room for them whatever the address.
struct PlaneRoom {
    size_t rows, d, off, parts, exponent;
    int planes;
    bool by_row;  // each row has a scale of its own
};

PlaneRoom plane_room(Carver& c, size_t rows, size_t D, const Mode& m, bool by_row = false)
{
    PlaneRoom r{};
    r.rows = rows;
    r.d = round_up(D, kTurnK);
    r.planes = m.planes;
    r.off = c.take(r.planes * rows * r.d * 2);
    r.by_row = by_row;
    r.parts = c.take(by_row ? 0 : kMaxParts * sizeof(float));
    r.exponent = c.take((by_row ? rows : 1) * sizeof(int));
    return r;
}

unsigned stride_grid(size_t items, size_t per)
{
    return unsigned(std::max<size_t>(1, std::min(ceil_div(items, per), max_grid_blocks())));
}

// What has to be done before the products, in at most two launches.
struct Preparation {
    MaxOfAll max{};
    PlanesOfAll planes{};
    int nmax = 0, nplanes = 0;

    void scale_by(const void* src, bool f32, size_t rows, size_t d, const int64_t* target, float* parts)
    {
        max.of[nmax++] = MaxOf{src, f32, rows, d, target, parts,
                               unsigned(std::min<size_t>(ceil_div(rows, kRowWaves), kMaxParts))};
    }

    // The exponent of the matrix that scale_by was called for last.
    void lay_out(PlanesOf p, bool scaled)
    {
        if (scaled) {
            p.parts = max.of[nmax - 1].parts;
            p.nparts = max.of[nmax - 1].nparts;
        }
        planes.of[nplanes++] = p;
    }

    void launch(int dtype, const Mode& mode, int64_t ignore, size_t V, hipStream_t stream) const
    {
        unsigned parts = 0;
        for (int k = 0; k < nmax; ++k)
            parts = std::max(parts, max.of[k].nparts);
        size_t rows = 1;
        for (int k = 0; k < nplanes; ++k)
            rows = std::max(rows, planes.of[k].out ? planes.of[k].rows_out : 0);
        const dim3 grid(unsigned(std::min<size_t>(ceil_div(rows, kRowWaves), 256 * 8)), unsigned(nplanes));
        with_dtype(dtype, [&](auto t) {
            using T = decltype(t);
            if (nmax)
                hipLaunchKernelGGL(largest_kernel<T>, dim3(parts, unsigned(nmax)), dim3(kRowThreads), 0, stream, max,
                                   ignore, V);
            if (!nplanes)
                return 0;
            const auto launch = [&](auto kernel) {
                hipLaunchKernelGGL(kernel, grid, dim3(kRowThreads), 0, stream, planes, ignore, V);
            };
            if constexpr (std::is_same_v<T, float>)
                launch(planes_kernel<T, true, 2>);
            else if constexpr (std::is_same_v<T, f16_t>)
                launch(planes_kernel<T, true, 1>);
            else
                launch(mode.f16 ? planes_kernel<T, true, 1> : planes_kernel<T, false, 1>);
            return 0;
        });
    }
};

// Describes src as an operand by rows: as it is, or as planes in the workspace
// that `prep` is to lay out. With a `target`, rows that have none become zeros
// and the scale takes no notice of them.
MatOperand make_operand(Preparation& prep, const void* src, size_t rows, size_t D, const Mode& mode, int dtype,
                        const PlaneRoom& room, char* ws, const int64_t* target)
{
    MatOperand m{};
    if (!target && direct_ok(src, D, mode)) {
        m.plane0 = static_cast<const uint16_t*>(src);
        m.ld = uint32_t(D);
        m.extent = uint32_t(rows);
        return m;
    }
    uint16_t* out = reinterpret_cast<uint16_t*>(ws + room.off);
    int* exponent = mode.scaled ? reinterpret_cast<int*>(ws + room.exponent) : nullptr;
    const bool by_row = mode.scaled && room.by_row, whole = mode.scaled && !by_row;
    if (whole)
        prep.scale_by(src, dtype == GC_F32, rows, D, target, reinterpret_cast<float*>(ws + room.parts));
    prep.lay_out(PlanesOf{src, rows, D, out, room.rows, room.d, target, nullptr, 0, exponent, by_row}, whole);
    m.plane0 = out;
    m.plane_stride = room.rows * room.d;
    m.ld = uint32_t(room.d);
    m.extent = uint32_t(room.rows);
    m.exponent = exponent;
    m.by_row = by_row;
    return m;
}

// ---- loss

// Tiles of 256 x 256 read the least and need some rounds of 256 of them; what
// has fewer than half a round takes smaller ones, two of which share a compute
// unit. V = 30522, D = 768, us:
//   tokens        1     32     64    128    256    512
//   128 x 64   14.5   16.5   16.2
//   128 x 128                19.4   19.1   25.6   39.8
//   256 x 256  24.7   25.1   21.6   21.0   27.2   31.1
constexpr int kTile = 256, kSmallTile = 128, kLogitWavesA = 2;
constexpr size_t kCus = 256;

// A range of the vocabulary and the tiles that it takes.
struct LogitRange {
    size_t v0, v;
    int ta, tb;
    size_t tiles_a() const { return ceil_div(v, ta); }
};

struct LogitPlan {
    LogitRange range[2];
    int count;
};

// The logits of N rows. A last round of 256 x 256 tiles that would leave more
// than half of the chip empty goes as tiles of 128 x 128 instead: 1001 x 33333
// x 1001 fp32, 524 tiles, took 333 us in three rounds, 308 in two and the rest.
LogitPlan logit_plan(size_t N, size_t V, bool few_rows)
{
    LogitPlan p{};
    p.count = 1;
    if (few_rows && N <= 64) {
        p.range[0] = LogitRange{0, V, kSmallTile, 64};
        return p;
    }
    const size_t tb = ceil_div(N, kTile), tiles = tb * ceil_div(V, kTile);
    if (tiles <= kCus / 2) {
        p.range[0] = LogitRange{0, V, kSmallTile, kSmallTile};
        return p;
    }
    p.range[0] = LogitRange{0, V, kTile, kTile};
    const size_t whole = tiles / kCus * kCus / tb;  // tiles of the vocabulary in whole rounds
    if (whole > 0 && whole * kTile < V) {
        const LogitRange rest{whole * kTile, V - whole * kTile, kSmallTile, kSmallTile};
        if (rest.tiles_a() * ceil_div(N, kSmallTile) <= 2 * kCus) {
            p.range[0].v = whole * kTile;
            p.range[1] = rest;
            p.count = 2;
        }
    }
    return p;
}

struct LossLayout {
    Mode mode;
    LogitPlan plan;
    PlaneRoom weight, hidden;
    size_t parts, target_logit, nparts, total;
};

LossLayout loss_layout(size_t N, size_t V, size_t D, int dtype)
{
    LossLayout L{};
    Carver c;
    L.mode = mode_of(dtype, dtype != GC_BF16);
    L.plan = logit_plan(N, V, true);
    L.weight = plane_room(c, V, D, L.mode);
    // a scale for each token, so that none costs another one bits
    L.hidden = plane_room(c, N, D, L.mode, true);
    for (int k = 0; k < L.plan.count; ++k)
        L.nparts += L.plan.range[k].tiles_a() * kLogitWavesA;
    L.parts = c.take(N * L.nparts * sizeof(LossPart));
    L.target_logit = c.take(N * 4);
    L.total = c.used;
    return L;
}

// ---- gradient

// G of one piece is kept to about this many bytes. A larger piece means fewer
// partial results and better filled rounds of tiles, a smaller one less memory
// (and G in the 256 MB of the last-level cache): 8192 x 30522 x 768 with an
// fp32 gradient took 2858, 2352, 2200, 2317 and 2221 us with 128, 256, 512,
// 1024 and 2048 MB; 8192 x 64000 x 4096 in bf16 10.96, 10.83, 10.83, 10.73 and
// 10.75 ms.
constexpr size_t kPieceBytes = size_t(512) << 20;

// Tile and splits of k of one of the gradient's products.
struct ProductPlan {
    int tile;
    uint32_t splits;
};

struct GradLayout {
    Mode mode;
    PlaneRoom weight, hidden;
    size_t n_pad, piece, pieces;  // rows of G, vocabulary of one piece
    int g_planes, h_planes, w_planes;  // of G: in memory, in each product
    size_t g, g_parts, g_exponent, h_slab, w_slab, total;
    size_t d4;  // row length of the slabs
    ProductPlan h, w;
};

// Splits of a product of `tiles` tiles over `turns` turns: as many as find a
// compute unit each, at least 4 turns long. Filling several rounds of 256
// tiles with more of them cost more in partial results than it gave: 8192 x
// 30522 x 768 with an fp32 gradient (192 tiles of 128 turns into 16384 x 768)
// took 1974 us with 4 splits, 1884 with 1.
//
// Few tiles are smaller ones: of 128 x 128, two share a compute unit. The
// fp32 gradient of 100 x 3001 x 256 took 63 us with tiles of 256 alone, 46
// with these; that of 600 x 5000 x 500, whose dweight is 40 tiles of 256, 100
// and 90; that of 4000 x 9000 x 1024, whose dhidden is 64, 770 and 812.
constexpr size_t kFewTiles = 48;

ProductPlan product_plan(size_t rows, size_t D, size_t turns)
{
    ProductPlan p{};
    p.tile = ceil_div(rows, kTile) * ceil_div(D, kTile) <= kFewTiles ? kSmallTile : kTile;
    const size_t tiles = ceil_div(rows, p.tile) * ceil_div(D, p.tile), room = p.tile == kTile ? kCus : 2 * kCus;
    p.splits = uint32_t(std::max<size_t>(1, std::min(room / tiles, turns / 4)));
    return p;
}

// Planes of G for a gradient of the type: one, rounded to the 16 bits that the
// gradient is rounded to as well, or two. A 16-bit gradient thus carries two
// roundings to its type where one cannot be avoided: it is some 1.4 times as
// far from 64 bits (1.75 at most in 60 sizes). A second plane would undo that
// and take 2.20 ms for 8192 x 30522 x 768, where one takes 1.25; who needs it
// asks for fp32.
int g_planes(int dtype) { return dtype == GC_F32 ? 2 : 1; }

// Planes for dweight. One plane of fp16 ends at 2^-39 of the largest |dloss|,
// far above what a bf16 dweight holds of the rows of rare tokens: next to an
// fp32 dhidden, for which both planes are there, it takes both.
int w_planes(const Mode& m, int dtype, int dw_dtype) { return dtype == GC_BF16 && m.f16 ? 2 : g_planes(dw_dtype); }

ProductShape grad_shape(int planes_a, int planes_g)
{
    ProductShape sh{};
    set_pairs(sh, planes_a, planes_g);
    return sh;
}

// Tiles of the vocabulary of one piece: all of them if that is at most `most`
// (two pieces of 4000 x 9000 x 1024 took 500 us, one 400), else at least half
// of `most`. The pieces' products for dweight run in rounds of 256 tiles, which some
// sizes fill better than others; splits and pieces cost their partial results
// (about 4 TB/s, in turns of 3.4 us). 8192 x 30522 x 768 with an fp32
// gradient: 1955 us in pieces of 64 tiles (192 of dweight), 1890 in pieces of
// 42 (126, in two splits).
size_t piece_tiles(size_t most, size_t N, size_t V, size_t D, size_t h_turns_a_tile, size_t w_turns)
{
    const size_t all = ceil_div(V, kTile), from = std::max<size_t>(most / 2, 1);
    if (all <= most)
        return all;
    constexpr double kTurnBytes = 4e12 * 3.4e-6;
    size_t best = most;
    double least = 0.0;
    for (size_t p = best; p >= from; p -= std::max<size_t>(p / 64, 1)) {
        const auto turns = [&](size_t tiles) {
            const ProductPlan w = product_plan(tiles * kTile, D, w_turns), h = product_plan(N, D, tiles * h_turns_a_tile);
            const size_t room = w.tile == kTile ? kCus : 2 * kCus;
            const double a_turn = w.tile == kTile ? 1.0 : 0.5;
            return double(ceil_div(ceil_div(tiles * kTile, w.tile) * ceil_div(D, w.tile) * w.splits, room)) *
                       double(ceil_div(w_turns, w.splits)) * a_turn +
                   (w.splits > 1 ? double(w.splits * tiles * kTile * D) * 8.0 / kTurnBytes : 0.0) +
                   double(h.splits * N * D) * 8.0 / kTurnBytes;
        };
        const double t = double(all / p) * turns(p) + (all % p ? turns(all % p) : 0.0);
        if (p == best || t < least) {
            best = p;
            least = t;
        }
        if (p == 1)
            break;
    }
    return best;
}

GradLayout grad_layout(size_t N, size_t V, size_t D, int dtype, int dh_dtype, int dw_dtype)
{
    GradLayout L{};
    Carver c;
    L.mode = mode_of(dtype, dh_dtype == GC_F32 || dw_dtype == GC_F32);
    L.weight = plane_room(c, V, D, L.mode);
    L.n_pad = round_up(N, kTurnK);
    L.hidden = plane_room(c, L.n_pad, D, L.mode);
    L.d4 = round_up(D, 4);
    L.h_planes = g_planes(dh_dtype);
    L.w_planes = w_planes(L.mode, dtype, dw_dtype);
    L.g_planes = std::max(L.h_planes, L.w_planes);
    const size_t h_turns = kTile / kTurnK * grad_shape(L.weight.planes, L.h_planes).segments;  // of a tile of the vocabulary
    const size_t w_turns = L.n_pad / kTurnK * grad_shape(L.hidden.planes, L.w_planes).segments;
    const size_t most = std::min(std::max<size_t>(kPieceBytes / (L.n_pad * 2 * L.g_planes * kTile), 1), kMaxPiece / kTile);
    L.piece = piece_tiles(most, N, V, D, h_turns, w_turns) * kTile;
    L.pieces = ceil_div(V, L.piece);
    L.g = c.take(L.g_planes * L.n_pad * L.piece * 2);
    L.g_parts = c.take(kMaxParts * sizeof(float));
    L.g_exponent = c.take(sizeof(int));
    L.h = product_plan(N, D, L.piece / kTile * h_turns);
    L.w = product_plan(L.piece, D, w_turns);
    L.h_slab = c.take(L.h.splits > 1 || L.pieces > 1 ? L.h.splits * N * L.d4 * 4 : 0);
    L.w_slab = c.take(L.w.splits > 1 ? L.w.splits * L.piece * L.d4 * 4 : 0);
    L.total = c.used;
    return L;
}

// A product into `out` of type T.
template <bool kBK, typename T>
void launch_product(const MatOperand& A, const MatOperand& B, ProductShape sh, int tile, const ProductOut<T>& out,
                    bool f16, hipStream_t stream)
{
    sh.tiles_a = uint32_t(ceil_div(out.na, tile));
    sh.tiles_b = uint32_t(ceil_div(out.nb, tile));
    const dim3 grid(sh.tiles_a * sh.tiles_b * sh.splits);
    const auto either = [&](auto f) {
        constexpr bool kF16 = decltype(f)::value;
        if (tile == kTile)
            hipLaunchKernelGGL((product_kernel<kF16, kBK, kTile, kTile, 2, 4, T>), grid, dim3(8 * kWave), 0, stream, A,
                               B, sh, out);
        else
            hipLaunchKernelGGL((product_kernel<kF16, kBK, kSmallTile, kSmallTile, 2, 2, T>), grid, dim3(4 * kWave), 0,
                               stream, A, B, sh, out);
    };
    if (f16)
        either(std::true_type());
    else if constexpr (!std::is_same_v<T, f16_t>)
        either(std::false_type());
}

template <bool kBK>
void launch_product_any(const MatOperand& A, const MatOperand& B, const ProductShape& sh, int tile, void* out,
                        int dtype, size_t nb, size_t D, bool f16, hipStream_t stream)
{
    with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        ProductOut<T> o{};
        o.p = static_cast<T*>(out);
        o.ld = D;
        o.na = uint32_t(D);
        o.nb = uint32_t(nb);
        o.vec = D % 4 == 0 && aligned_to(out, 4 * sizeof(T));
        launch_product<kBK, T>(A, B, sh, tile, o, f16, stream);
        return 0;
    });
}

void launch_sum(const float* slab, size_t d4, size_t split_stride, uint32_t splits, size_t rows, size_t D,
                void* out, int dtype, hipStream_t stream)
{
    with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        hipLaunchKernelGGL(sum_splits_kernel<T>, dim3(stride_grid(rows * (d4 / 4), kSumThreads)),
                           dim3(kSumThreads), 0, stream, slab, d4, split_stride, splits, rows, D,
                           static_cast<T*>(out));
        return 0;
    });
}

__global__ __launch_bounds__(kSumThreads) void zero_kernel(uint16_t* out, size_t n)
{
    for (size_t i = size_t(blockIdx.x) * kSumThreads + threadIdx.x; i < n; i += size_t(gridDim.x) * kSumThreads)
        out[i] = 0;
}

// bytes: even, as every type's size is.
void launch_zero(void* out, size_t bytes, hipStream_t stream)
{
    hipLaunchKernelGGL(zero_kernel, dim3(stride_grid(bytes / 2, kSumThreads)), dim3(kSumThreads), 0, stream,
                       static_cast<uint16_t*>(out), bytes / 2);
}

}  // namespace
}  // namespace gcq

using namespace gcq;

GCQ_API int linear_xent_loss(const void* hidden, const void* weight, int dtype, size_t N, size_t V,
                             size_t D, const int64_t* target, int64_t ignore_index, float* loss,
                             float* lse, void* ws, size_t* ws_bytes, hipStream_t stream)
{
    clear_error();
    if (int rc = check_sizes("linear_xent_loss", N, V, D, dtype))
        return rc;
    if (!ws_bytes)
        return fail(GC_EINVAL, "linear_xent_loss: ws_bytes is NULL");
    const LossLayout L = loss_layout(N, V, D, dtype);
    if (!ws) {
        *ws_bytes = L.total;
        return GC_OK;
    }
    if (N == 0)
        return GC_OK;
    const size_t b = dtype_bytes(dtype);
    if (!hidden || !weight || !target || !loss || !lse || !aligned_to(hidden, b) || !aligned_to(weight, b) ||
        !aligned_to(target, 8) || !aligned4(loss) || !aligned4(lse))
        return fail(GC_EINVAL, "linear_xent_loss: a buffer is NULL or misaligned");
    if (!aligned16(ws) || *ws_bytes < L.total)
        return fail(GC_EINVAL, "linear_xent_loss: workspace too small or not 16-byte aligned");
    char* w = static_cast<char*>(ws);
    Preparation prep;
    const MatOperand wo = make_operand(prep, weight, V, D, L.mode, dtype, L.weight, w, nullptr);
    const MatOperand ho = make_operand(prep, hidden, N, D, L.mode, dtype, L.hidden, w, nullptr);
    prep.launch(dtype, L.mode, ignore_index, V, stream);
    ProductShape sh{};
    sh.turns = uint32_t(round_up(D, kTurnK) / kTurnK);
    set_pairs(sh, L.weight.planes, L.hidden.planes);
    sh.splits = 1;
    LossPart* parts = reinterpret_cast<LossPart*>(w + L.parts);
    float* tl = reinterpret_cast<float*>(w + L.target_logit);
    size_t part0 = 0;
    for (int k = 0; k < L.plan.count; ++k) {
        const LogitRange& r = L.plan.range[k];
        MatOperand wr = wo;
        wr.plane0 += r.v0 * wo.ld;
        wr.extent = uint32_t(r.v);
        sh.tiles_a = uint32_t(r.tiles_a());
        sh.tiles_b = uint32_t(ceil_div(N, r.tb));
        const dim3 grid(sh.tiles_a * sh.tiles_b);
        const auto tiles = [&](auto kernel, int waves) {
            hipLaunchKernelGGL(kernel, grid, dim3(waves * kWave), 0, stream, wr, ho, sh, uint32_t(N), uint32_t(r.v0),
                               uint32_t(r.v), uint32_t(V), target, parts, uint32_t(L.nparts), uint32_t(part0), tl);
        };
        const auto either = [&](auto f16) {
            constexpr bool kF16 = decltype(f16)::value;
            if (r.tb == 64)
                tiles(loss_tiles_kernel<kF16, kSmallTile, 64, kLogitWavesA, 2>, 4);
            else if (r.tb == kSmallTile)
                tiles(loss_tiles_kernel<kF16, kSmallTile, kSmallTile, kLogitWavesA, 2>, 4);
            else
                tiles(loss_tiles_kernel<kF16, kTile, kTile, kLogitWavesA, 4>, 8);
        };
        if (L.mode.f16)
            either(std::true_type());
        else
            either(std::false_type());
        part0 += r.tiles_a() * kLogitWavesA;
    }
    hipLaunchKernelGGL(loss_join_kernel, dim3(stride_grid(N, kJoinThreads / kWave)), dim3(kJoinThreads), 0,
                       stream, parts, uint32_t(L.nparts), tl, target, ignore_index, uint32_t(N), uint32_t(V),
                       loss, lse);
    return check_launch("linear_xent_loss");
}

GCQ_API int linear_xent_grad(const void* hidden, const void* weight, int dtype, size_t N, size_t V,
                             size_t D, const int64_t* target, int64_t ignore_index, const float* lse,
                             const float* dloss, void* dhidden, int dhidden_dtype, void* dweight,
                             int dweight_dtype, void* ws, size_t* ws_bytes, hipStream_t stream)
{
    clear_error();
    if (int rc = check_sizes("linear_xent_grad", N, V, D, dtype))
        return rc;
    if ((dhidden_dtype != dtype && dhidden_dtype != GC_F32) || (dweight_dtype != dtype && dweight_dtype != GC_F32))
        return fail(GC_EINVAL, "linear_xent_grad: a gradient has the inputs' type or fp32");
    if (!ws_bytes)
        return fail(GC_EINVAL, "linear_xent_grad: ws_bytes is NULL");
    if (!ws) {
        // (of no tokens too: a workspace of no bytes would ask again)
        *ws_bytes = grad_layout(std::max<size_t>(N, 1), V, D, dtype, dhidden_dtype, dweight_dtype).total;
        return GC_OK;
    }
    const size_t b = dtype_bytes(dtype);
    if (!aligned_to(dhidden, dtype_bytes(dhidden_dtype)) || !aligned_to(dweight, dtype_bytes(dweight_dtype)))
        return fail(GC_EINVAL, "linear_xent_grad: a gradient is misaligned");
    if (N == 0) {
        if (dweight)
            launch_zero(dweight, V * D * dtype_bytes(dweight_dtype), stream);
        return check_launch("linear_xent_grad");
    }
    if (!hidden || !weight || !target || !lse || !dloss || !aligned_to(hidden, b) || !aligned_to(weight, b) ||
        !aligned_to(target, 8) || !aligned4(lse) || !aligned4(dloss))
        return fail(GC_EINVAL, "linear_xent_grad: a buffer is NULL or misaligned");
    const GradLayout L = grad_layout(N, V, D, dtype, dhidden_dtype, dweight_dtype);
    if (!aligned16(ws) || *ws_bytes < L.total)
        return fail(GC_EINVAL, "linear_xent_grad: workspace too small or not 16-byte aligned");
    if (!dhidden && !dweight)
        return GC_OK;

    char* w = static_cast<char*>(ws);
    Preparation prep;
    const MatOperand wo = make_operand(prep, weight, V, D, L.mode, dtype, L.weight, w, nullptr);
    // always a copy: rows without a target become zeros
    const MatOperand ho = make_operand(prep, hidden, N, D, L.mode, dtype, L.hidden, w, target);
    GradOut g{};
    MatOperand go{};
    if (L.mode.f16) {
        int* exponent = reinterpret_cast<int*>(w + L.g_exponent);
        prep.scale_by(dloss, true, N, 1, target, reinterpret_cast<float*>(w + L.g_parts));
        prep.lay_out(PlanesOf{nullptr, 0, 0, nullptr, 0, 0, nullptr, nullptr, 0, exponent, false}, true);
        go.exponent = g.exponent = exponent;
    }
    prep.launch(dtype, L.mode, ignore_index, V, stream);
    go.plane0 = g.plane0 = reinterpret_cast<uint16_t*>(w + L.g);
    go.plane_stride = g.plane_stride = L.n_pad * L.piece;
    go.ld = g.ld = uint32_t(L.piece);
    g.rows_out = uint32_t(L.n_pad);
    float* h_slab = reinterpret_cast<float*>(w + L.h_slab);
    float* w_slab = reinterpret_cast<float*>(w + L.w_slab);
    const bool h_direct = L.h.splits == 1 && L.pieces == 1;

    for (size_t v0 = 0; v0 < V; v0 += L.piece) {
        const size_t vp = std::min(L.piece, V - v0);
        MatOperand wp = wo;
        wp.plane0 += v0 * wo.ld;
        wp.extent = uint32_t(vp);
        ProductShape sh{};
        sh.turns = uint32_t(round_up(D, kTurnK) / kTurnK);
        set_pairs(sh, L.weight.planes, L.hidden.planes);
        const LogitPlan plan = logit_plan(L.n_pad, vp, false);
        sh.splits = 1;
        for (int k = 0; k < plan.count; ++k) {
            const LogitRange& r = plan.range[k];
            MatOperand wr = wp;
            wr.plane0 += r.v0 * wo.ld;
            wr.extent = uint32_t(r.v);
            GradOut gr = g;
            gr.plane0 += r.v0;
            sh.tiles_a = uint32_t(r.tiles_a());
            sh.tiles_b = uint32_t(ceil_div(L.n_pad, r.tb));
            const dim3 grid(sh.tiles_a * sh.tiles_b);
            const auto logits = [&](auto whole, auto small) {
                const auto launch = [&](auto kernel, int waves) {
                    hipLaunchKernelGGL(kernel, grid, dim3(waves * kWave), 0, stream, wr, ho, sh, uint32_t(N),
                                       uint32_t(v0 + r.v0), uint32_t(V), target, ignore_index, lse, dloss, gr);
                };
                if (r.tb == kTile)
                    launch(whole, 8);
                else
                    launch(small, 4);
            };
            if (!L.mode.f16)
                logits(logit_grad_kernel<false, kTile, kTile, 2, 4, 1>,
                       logit_grad_kernel<false, kSmallTile, kSmallTile, 2, 2, 1>);
            else if (L.g_planes == 1)
                logits(logit_grad_kernel<true, kTile, kTile, 2, 4, 1>,
                       logit_grad_kernel<true, kSmallTile, kSmallTile, 2, 2, 1>);
            else
                logits(logit_grad_kernel<true, kTile, kTile, 2, 4, 2>,
                       logit_grad_kernel<true, kSmallTile, kSmallTile, 2, 2, 2>);
        }
        if (dhidden) {
            MatOperand A = wp, B = go;
            A.extent = uint32_t(wo.ld);
            A.krows = uint32_t(vp);
            B.extent = uint32_t(N);
            ProductShape ps = grad_shape(L.weight.planes, L.h_planes);
            ps.turns = uint32_t(ceil_div(vp, kTurnK));
            ps.splits = L.h.splits;
            if (h_direct) {
                launch_product_any<false>(A, B, ps, L.h.tile, dhidden, dhidden_dtype, N, D, L.mode.f16, stream);
            } else {
                ProductOut<float> o{h_slab, L.d4, N * L.d4, uint32_t(L.d4), uint32_t(N), true, v0 > 0};
                launch_product<false, float>(A, B, ps, L.h.tile, o, L.mode.f16, stream);
            }
        }
        if (dweight) {
            MatOperand A = ho, B = go;
            A.extent = uint32_t(ho.ld);
            A.krows = B.krows = uint32_t(L.n_pad);
            B.extent = uint32_t(L.piece);
            ProductShape ps = grad_shape(L.hidden.planes, L.w_planes);
            ps.turns = uint32_t(L.n_pad / kTurnK);
            ps.splits = L.w.splits;
            char* out = static_cast<char*>(dweight) + v0 * D * dtype_bytes(dweight_dtype);
            if (L.w.splits == 1) {
                launch_product_any<true>(A, B, ps, L.w.tile, out, dweight_dtype, vp, D, L.mode.f16, stream);
            } else {
                ProductOut<float> o{w_slab, L.d4, L.piece * L.d4, uint32_t(L.d4), uint32_t(vp), true, false};
                launch_product<true, float>(A, B, ps, L.w.tile, o, L.mode.f16, stream);
                launch_sum(w_slab, L.d4, L.piece * L.d4, L.w.splits, vp, D, out, dweight_dtype, stream);
            }
        }
    }
    if (dhidden && !h_direct)
        launch_sum(h_slab, L.d4, N * L.d4, L.h.splits, N, D, dhidden, dhidden_dtype, stream);
    return check_launch("linear_xent_grad");
}
