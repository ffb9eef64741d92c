// row_team.h -- a row of values in the registers of a team of threads: shared by
// the norms (norm_residual.hip, layer_norm.hip).
//
// A team is a wave for rows of up to four 16-byte vectors a lane, then 4 to 16
// waves. Sums over columns are exchanged within the team; sums over rows leave
// one partial row a workgroup, which a second launch adds in their order.
#pragma once

#include "dropout_mask.h"

namespace gcq {
namespace {

constexpr size_t kMaxNormD = 16384;

template <int N>
struct Int {
    static constexpr int value = N;
};

// ---- a row in the registers of a team -----------------------------------------

// Vector v of team lane t is v * kTeam + t; kAligned: every row starts on 16
// bytes and holds whole vectors (otherwise the loads and stores are aligned
// to the element alone, and a row's last values go one at a time).
template <typename T, int kTeam, int kVecs, bool kAligned>
struct Row {
    static constexpr int V = kVec<T>;
    static constexpr int kWg = kTeam < 256 ? 256 : kTeam;
    static constexpr int kTeams = kWg / kTeam;  // of a workgroup
    using F = vec_f32<T>;
    typedef T Raw __attribute__((ext_vector_type(kVec<T>)));
    typedef Raw RawAny __attribute__((aligned(sizeof(T))));

    static __device__ __forceinline__ uint32_t col(int v, int t) { return (v * kTeam + t) * V; }

    static __device__ __forceinline__ Raw load_raw(const T* row, uint32_t c, uint32_t d)
    {
        if (kAligned)
            return c < d ? *reinterpret_cast<const Raw*>(row + c) : Raw{};
        if (c + V <= d)
            return *reinterpret_cast<const RawAny*>(row + c);
        Raw r = {};
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (c + e < d)
                r[e] = row[c + e];
        return r;
    }

    static __device__ __forceinline__ void load(Raw (&r)[kVecs], const T* p, size_t row, uint32_t d, int t)
    {
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
            r[v] = load_raw(p + row * d, col(v, t), d);
    }

    static __device__ __forceinline__ F wide(Raw r) { return __builtin_convertvector(r, F); }

    static __device__ __forceinline__ void store(T* row, uint32_t c, uint32_t d, F x)
    {
        const Raw r = __builtin_convertvector(x, Raw);
        if (kAligned) {
            if (c < d)
                *reinterpret_cast<Raw*>(row + c) = r;
            return;
        }
        if (c + V <= d) {
            *reinterpret_cast<RawAny*>(row + c) = r;
            return;
        }
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (c + e < d)
                row[c + e] = r[e];
    }

    // x where bit e of `bits` is set, else 0 (whatever x holds).
    static __device__ __forceinline__ float keep(uint32_t bits, int e, float x)
    {
        return u2f(f2u(x) & uint32_t(int32_t(bits << (31 - e)) >> 31));
    }

    // Which team of the workgroup this is, for every lane of a wave the same.
    static __device__ __forceinline__ int team()
    {
        return kTeams == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / kTeam);
    }

    // fp32 values of columns, which are aligned to 4 bytes: 1 where there is no
    // array.
    typedef float Cols __attribute__((ext_vector_type(kVec<T>)));
    typedef Cols ColsAny __attribute__((aligned(4)));

    static __device__ __forceinline__ F columns(const float* p, uint32_t c, uint32_t d)
    {
        if (!p)
            return F{} + 1.0f;
        if (c + V <= d)
            return *reinterpret_cast<const ColsAny*>(p + c);
        F f = {};
        if (!kAligned) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (c + e < d)
                    f[e] = p[c + e];
        }
        return f;
    }

    static __device__ __forceinline__ void store_columns(float* p, uint32_t c, uint32_t d, F x)
    {
        if (c + V <= d) {
            *reinterpret_cast<ColsAny*>(p + c) = x;
        } else if (!kAligned) {
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (c + e < d)
                    p[c + e] = x[e];
        }
    }

    // Whether the values i .. i + V - 1 of the mask are kept, a bit each; i mod
    // 4 is the same for a whole row.
    static __device__ __forceinline__ uint32_t mask(const DropoutArgs& a, uint64_t key, uint64_t i)
    {
        const uint32_t phase = kAligned ? 0 : __builtin_amdgcn_readfirstlane(uint32_t(i) & 3);
        uint32_t w[V + 4];
#pragma unroll
        for (int s = 0; s < V / 4; ++s) {
            const U4 r = dropout_words(a, key, (i >> 2) + s);
            w[4 * s] = r.x;
            w[4 * s + 1] = r.y;
            w[4 * s + 2] = r.z;
            w[4 * s + 3] = r.w;
        }
        if (phase) {
            const U4 r = dropout_words(a, key, (i >> 2) + V / 4);
            w[V] = r.x;
            w[V + 1] = r.y;
            w[V + 2] = r.z;
#pragma unroll
            for (int e = 0; e < V; ++e)
                w[e] = phase == 1 ? w[e + 1] : phase == 2 ? w[e + 2] : w[e + 3];
        }
        uint32_t bits = 0;
#pragma unroll
        for (int e = 0; e < V; ++e)
            bits |= w[e] >= a.cut ? 1u << e : 0u;
        return bits;
    }
};

// Sum over a wave, in every lane: four DPP steps within each row of 16 lanes
// (quad_perm xor 1 and xor 2, row_half_mirror, row_mirror), then the rows.
__device__ __forceinline__ float wave_sum(float x)
{
    const auto step = [](float v, auto ctrl) {
        return v + u2f(uint32_t(__builtin_amdgcn_update_dpp(0, int(f2u(v)), decltype(ctrl)::value, 0xF, 0xF, true)));
    };
    x = step(x, Int<0xB1>());
    x = step(x, Int<0x4E>());
    x = step(x, Int<0x141>());
    x = step(x, Int<0x140>());
    const auto row = [x](int lane) { return u2f(uint32_t(__builtin_amdgcn_readlane(int(f2u(x)), lane))); };
    return (row(0) + row(16)) + (row(32) + row(48));
}

// Sums over a team; every lane gets them. Teams of several waves are whole
// workgroups and exchange through LDS, alternating between two halves so that
// one barrier an exchange suffices.
template <int kTeam, int kCount>
struct TeamSum {
    static constexpr int kWaves = kTeam / kWave;

    static __device__ __forceinline__ void run(float (&x)[kCount], float* lds, int& half)
    {
#pragma unroll
        for (int k = 0; k < kCount; ++k)
            x[k] = wave_sum(x[k]);
        if (kWaves == 1)
            return;
        float* at = lds + half * (kWaves * kCount);
        half ^= 1;
        const int wave = threadIdx.x / kWave;
        if ((threadIdx.x & (kWave - 1)) == 0) {
#pragma unroll
            for (int k = 0; k < kCount; ++k)
                at[k * kWaves + wave] = x[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kCount; ++k) {
            x[k] = at[k * kWaves];
            for (int w = 1; w < kWaves; ++w)
                x[k] += at[k * kWaves + w];
        }
    }
};

// ---- sums over rows -------------------------------------------------------------

// out[k][c] = sum over the `count` partial rows of k, in a fixed order: 16
// threads a column take every 16th row, and their sums are added in order.
constexpr int kSumCols = 64, kSumRows = 16;

struct PartSum {
    const float* part;
    float* out;
    uint32_t count;  // partial rows of one output row
    uint32_t rows;   // output rows
};

__global__ __launch_bounds__(kSumCols* kSumRows) void sum_parts_kernel(PartSum a, PartSum b, PartSum c, uint32_t d)
{
    __shared__ float lds[kSumRows][kSumCols];
    const uint32_t col = blockIdx.x * kSumCols + threadIdx.x % kSumCols, r = threadIdx.x / kSumCols;
    for (uint32_t row = blockIdx.y; row < a.rows + b.rows + c.rows; row += gridDim.y) {
        uint32_t k = row;
        PartSum p = a;
        if (k >= a.rows) {
            k -= a.rows;
            p = b;
            if (k >= b.rows) {
                k -= b.rows;
                p = c;
            }
        }
        float s = 0.0f;
        if (col < d)
#pragma unroll 8
            for (uint32_t i = r; i < p.count; i += kSumRows)
                s += p.part[(size_t(k) * p.count + i) * d + col];
        lds[r][threadIdx.x % kSumCols] = s;
        __syncthreads();
        if (r == 0 && col < d) {
            for (int i = 1; i < kSumRows; ++i)
                s += lds[i][threadIdx.x];
            p.out[size_t(k) * d + col] = s;
        }
        __syncthreads();
    }
}

// Calls f(team, vecs), as integral constants, with the smallest team that
// holds a row of d values.
template <typename T, typename F>
void with_team(size_t d, F f)
{
    // at most 16 values a lane
    constexpr int M = 16 / kVec<T>;
    const size_t vecs = ceil_div(d, kVec<T>);
    if (vecs <= 64)
        f(Int<64>(), Int<1>());
    else if (vecs <= 128)
        f(Int<64>(), Int<2>());
    else if (vecs <= 64 * M)
        f(Int<64>(), Int<M>());
    else if (vecs <= 128 * M)
        f(Int<256>(), Int<M / 2>());
    else if (vecs <= 256 * M)
        f(Int<256>(), Int<M>());
    else if (vecs <= 512 * M)
        f(Int<512>(), Int<M>());
    else
        f(Int<1024>(), Int<M>());
}

}  // namespace
}  // namespace gcq
