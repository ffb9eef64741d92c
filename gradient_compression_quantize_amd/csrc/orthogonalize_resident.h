// orthogonalize_resident.h -- the whole iteration of a small matrix in one
// workgroup and one launch (orthogonalize.hip says what is computed).
//
// Small means that X fits a compute unit: its 32 x 32 blocks stay in the registers
// of 8 waves from the norm to the result, fp32, in the layout of the matrix cores,
// and its first plane (or both) in LDS, where A, P and the waves' products read
// it. The tiled products need some 17 launches of 4 us and more for the same: 64 x
// 576 takes 80 us with them and 34 here, 128 x 256 77 and 37, 32 x 1024 of both
// planes 102 and 37; 48 of 64 x 576, a compute unit each, 102 and 37. A step takes
// some 4.4 us, four barriers and what LDS and the matrix cores answer in between.
//
// The smaller side r is padded to RP = 32, 64 or 128, the other one, c, to blocks
// of 32, and each wave owns every eighth 32 of c. Of a block, a lane holds 4
// values of a row side by side (16 bytes of the matrix at a time), and LDS the
// matrix as it lies: where a product needs it the other way, it reads it through
// the transposing load (a tall one in A = X' X, a wide one in P X). The blocks of
// A are split over the waves, over c too where there are fewer of them than
// waves.
#pragma once

#include "mfma_product.h"

namespace gcq {
namespace {

constexpr int kResidentWaves = 8;

// Coefficients of up to 64 steps.
constexpr int kMaxSteps = 64;
struct Coefficients {
    float v[kMaxSteps][3];
};

// A matrix of fp16 in LDS, rows of kLength values, in 16-byte chunks that an XOR
// of the row spreads over the 64 banks: the same chunk of 16 rows, which by_rows
// reads in one clock, and 64 bytes of four rows, which by_k does: 256 x 128 takes
// 41 us, 46 with the row itself (spread for by_k too, rows of 64 are slower: 576 x
// 64 41 us instead of 38).
template <int kLength>
struct LdsMatrix {
    static constexpr int kChunks = kLength / 8, kSpread = kChunks < 16 ? kChunks : 16, kRowsOfBanks = 16 / kSpread;
    typedef __attribute__((address_space(3))) uint16_t lds_u16;
    lds_u16* p;

    __device__ __forceinline__ lds_u16* at(int row, int col) const
    {
        const int r = (row / kRowsOfBanks) & (kSpread - 1);
        const int chunk = (col >> 3) ^ (kSpread == 16 ? 4 * (r & 3) + (r >> 2) : r);
        return p + row * kLength + chunk * 8 + (col & 7);
    }

    // Fragment of 32 rows x 16 k, the k of a row side by side.
    __device__ __forceinline__ s16x8 by_rows(int row0, int k0, int lane) const
    {
        typedef __attribute__((address_space(3))) const s16x8 lds_s16x8;
        return *(lds_s16x8*)at(row0 + (lane & 31), k0 + 8 * (lane >> 5));
    }

    // Fragment of 32 columns x 16 k, the k of a column below one another.
    __device__ __forceinline__ s16x8 by_k(int col0, int k0, int lane) const
    {
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const int g = lane >> 4, j = lane & 15;
        const int row = k0 + 8 * (g >> 1) + (j >> 2), col = col0 + 16 * (g & 1) + 4 * (j & 3);
        union {
            s16x4 h[2];
            s16x8 v;
        } u;
        u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at(row, col));
        u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at(row + 4, col));
        return u.v;
    }

    // The four values of a row from a column (a multiple of 4) on.
    __device__ __forceinline__ f16x4 quad(int row, int col) const
    {
        typedef __attribute__((address_space(3))) const f16x4 lds_f16x4;
        return *(lds_f16x4*)at(row, col);
    }
    __device__ __forceinline__ void set_quad(int row, int col, f16x4 v) const
    {
        typedef __attribute__((address_space(3))) f16x4 lds_f16x4;
        *(lds_f16x4*)at(row, col) = v;
    }
};

// One plane of a matrix or two that add up to it.
template <int kLength, int kPlanes>
struct LdsPlanes {
    LdsMatrix<kLength> plane[kPlanes];

    __device__ __forceinline__ void set(int row, int col, f32x4 v) const
    {
        const f16x4 p0 = __builtin_convertvector(v, f16x4);
        plane[0].set_quad(row, col, p0);
        if (kPlanes == 2)
            plane[kPlanes - 1].set_quad(row, col, __builtin_convertvector(v - __builtin_convertvector(p0, f32x4), f16x4));
    }

    __device__ __forceinline__ f32x4 get(int row, int col) const
    {
        f32x4 v = __builtin_convertvector(plane[0].quad(row, col), f32x4);
        if (kPlanes == 2)
            v += __builtin_convertvector(plane[kPlanes - 1].quad(row, col), f32x4);
        return v;
    }
};

// acc += a b of all pairs of planes but that of two second ones.
template <int kPlanes>
__device__ __forceinline__ f32x16 multiply_planes(const s16x8 (&a)[kPlanes], const s16x8 (&b)[kPlanes], f32x16 acc)
{
    const auto one = [](s16x8 x, s16x8 y, f32x16 z) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), z, 0, 0, 0);
    };
    if (kPlanes == 2) {
        acc = one(a[0], b[kPlanes - 1], acc);
        acc = one(a[kPlanes - 1], b[0], acc);
    }
    return one(a[0], b[0], acc);
}

// What a matrix is read from: values of `dtype`, or gradients (fp32) that move
// the momenta.
struct ResidentIn {
    PtrTable<void> x;
    PtrTable<float> momenta, new_momenta;
    Momentum mo;
    int dtype;
    bool momentum;
    uint32_t m, n;
    float eps;
};

// A value of 16 bits: bf16 or fp16.
__device__ __forceinline__ float from16(uint16_t bits, bool bf16)
{
    return bf16 ? u2f(uint32_t(bits) << 16) : float(__builtin_bit_cast(f16_t, bits));
}

__device__ __forceinline__ uint16_t to16(float v, bool bf16)
{
    return bf16 ? __builtin_bit_cast(uint16_t, bf16_t(v)) : __builtin_bit_cast(uint16_t, f16_t(v));
}

// RB: RP / 32; NB: 32s of c a wave owns; kTall: c is the number of rows.
template <int RB, int NB, int kPlanes, bool kTall>
__global__ __launch_bounds__(kResidentWaves* kWave, 2) void resident_kernel(ResidentIn in, Coefficients coef, int steps,
                                                                            LastOut last)
{
    constexpr int RP = 32 * RB, CP = kResidentWaves * NB * 32;
    // of A: a wave's blocks, and how many waves share one
    constexpr int kBlocks = RB * RB, kSplit = kBlocks < kResidentWaves ? kResidentWaves / kBlocks : 1;
    constexpr int kOwn = kBlocks > kResidentWaves ? kBlocks / kResidentWaves : 1;
    constexpr int kSums = (kSplit - 1) * kBlocks * 1024 * 4, kAP = 2 * kPlanes * RP * RP * 2;
    __shared__ uint16_t lds_x[kPlanes * CP * RP];
    // A and P, and before them the sums of the waves that share a block
    __shared__ uint16_t lds_ap[(kSums > kAP ? kSums : kAP) / 2];
    __shared__ __attribute__((aligned(16))) float diagonal_a[RP], diagonal_p[RP];
    __shared__ double norm_parts[kResidentWaves];
    typedef __attribute__((address_space(3))) uint16_t lds_u16;
    LdsPlanes<kTall ? RP : CP, kPlanes> X;
    LdsPlanes<RP, kPlanes> A, P;
#pragma unroll
    for (int k = 0; k < kPlanes; ++k) {
        X.plane[k].p = (lds_u16*)lds_x + k * CP * RP;
        A.plane[k].p = (lds_u16*)lds_ap + k * RP * RP;
        P.plane[k].p = (lds_u16*)lds_ap + (kPlanes + k) * RP * RP;
    }
    float* const sums = reinterpret_cast<float*>(lds_ap);

    // (locals, so that the arguments' tables are read where they lie)
    const uint32_t matrix = blockIdx.x;
    const void* const from = in.x.p[matrix];
    const float* const m0 = in.momenta.p[matrix];
    float* const m1 = const_cast<float*>(in.new_momenta.p[matrix]);
    const void* const weights = last.weights.p[matrix];
    void* const out = const_cast<void*>(last.out.p[matrix]);
    const Momentum mo = in.mo;
    const bool momentum = in.momentum, moves = last.update;
    const int in_dtype = in.dtype, out_dtype = last.dtype;
    const uint32_t m = in.m, n = in.n;
    const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int blocks = int(((kTall ? m : n) + 31) / 32);
    const auto owns = [&](int nb) { return nb * kResidentWaves + wave < blocks; };
    // Row of this lane's values in block (nb, i), and column of its quad q.
    const auto row_of = [&](int nb, int i, int l) {
        return (kTall ? nb * kResidentWaves + wave : i) * 32 + int(acc_col(l));
    };
    const auto col_of = [&](int nb, int i, int q, int l) {
        return (kTall ? i : nb * kResidentWaves + wave) * 32 + int(acc_row(4 * q, l));
    };

    // The values of block (nb, i) from or to a matrix in memory, by buffer
    // instructions: one that does not exist lies behind the last, where loads
    // give 0 and stores do nothing, so that there are no branches and all loads
    // are on their way together. Four at a time where each row holds whole
    // quads. Places are found anew each time: kept, they would take as many
    // registers as the values.
    const auto each_quad = [&](int nb, int i, auto f) {
        int l = lane;
        asm volatile("" : "+v"(l));
        const uint32_t row = row_of(nb, i, l);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t col = col_of(nb, i, q, l);
            f(q, row < m && col < n ? row * n + col : 1u << 28, n - col);
        }
    };
    const auto get = [&](const void* p, int dtype, int nb, int i, f32x16& v) {
        const bool wide = dtype == GC_F32, bf16 = dtype == GC_BF16;
        const auto at = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, m * n * (wide ? 4 : 2), 0x00020000);
        const bool whole = n % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 3) == 0;
        if (wide && whole)
            each_quad(nb, i, [&](int q, uint32_t first, uint32_t) {
                const u32x4 w = __builtin_amdgcn_raw_buffer_load_b128(at, first * 4, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[4 * q + e] = u2f(w[e]);
            });
        else if (whole)
            each_quad(nb, i, [&](int q, uint32_t first, uint32_t) {
                const auto w = __builtin_amdgcn_raw_buffer_load_b64(at, first * 2, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[4 * q + e] = from16(uint16_t(w[e / 2] >> 16 * (e % 2)), bf16);
            });
        else
            each_quad(nb, i, [&](int q, uint32_t first, uint32_t left) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t one = uint32_t(e) < left ? first + e : 1u << 28;
                    v[4 * q + e] = wide ? u2f(__builtin_amdgcn_raw_buffer_load_b32(at, one * 4, 0, 0))
                                        : from16(__builtin_amdgcn_raw_buffer_load_b16(at, one * 2, 0, 0), bf16);
                }
            });
    };
    const auto put = [&](void* p, int dtype, int nb, int i, const f32x16& v) {
        const bool wide = dtype == GC_F32, bf16 = dtype == GC_BF16;
        const auto at = __builtin_amdgcn_make_buffer_rsrc(p, 0, m * n * (wide ? 4 : 2), 0x00020000);
        const bool whole = n % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 3) == 0;
        if (wide && whole)
            each_quad(nb, i, [&](int q, uint32_t first, uint32_t) {
                u32x4 w;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = f2u(v[4 * q + e]);
                __builtin_amdgcn_raw_buffer_store_b128(w, at, first * 4, 0, 0);
            });
        else if (whole)
            each_quad(nb, i, [&](int q, uint32_t first, uint32_t) {
                vec_of<uint32_t, 2> w;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    w[e] = to16(v[4 * q + 2 * e], bf16) | uint32_t(to16(v[4 * q + 2 * e + 1], bf16)) << 16;
                __builtin_amdgcn_raw_buffer_store_b64(w, at, first * 2, 0, 0);
            });
        else
            each_quad(nb, i, [&](int q, uint32_t first, uint32_t left) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t one = uint32_t(e) < left ? first + e : 1u << 28;
                    if (wide)
                        __builtin_amdgcn_raw_buffer_store_b32(f2u(v[4 * q + e]), at, one * 4, 0, 0);
                    else
                        __builtin_amdgcn_raw_buffer_store_b16(to16(v[4 * q + e], bf16), at, one * 2, 0, 0);
                }
            });
    };

    // One or two 32s of c at a time, the others moving up: their loads are on
    // their way together, and the code of all NB, which the first waves to come
    // by have to fetch, is that of these.
    constexpr int kAtOnce = NB > 1 ? 2 : 1;
    f32x16 x[NB][RB];
    const auto columns = [&](auto f) {
#pragma unroll 1
        for (int nb = 0; nb < NB; nb += kAtOnce) {
            f32x16 v[kAtOnce][RB];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
                for (int i = 0; i < RB; ++i)
                    v[k][i] = x[k][i];
            if (owns(nb))
                f(nb, v);
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
                for (int i = 0; i < RB; ++i)
                    x[k][i] = k + kAtOnce < NB ? x[(k + kAtOnce) % NB][i] : v[(k + kAtOnce) % NB % kAtOnce][i];
        }
    };
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < RB; ++i)
            x[nb][i] = f32x16{};
    double sum = 0.0;
    columns([&](int nb, f32x16 (&v)[kAtOnce][RB]) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
            for (int i = 0; i < RB; ++i)
                get(from, in_dtype, nb + k, i, v[k][i]);
        if (momentum) {
            f32x16 old[kAtOnce][RB];  // (new momenta may be the old ones: all are read first)
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
                for (int i = 0; i < RB; ++i)
                    get(m0, GC_F32, nb + k, i, old[k][i]);
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
                for (int i = 0; i < RB; ++i) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float g = v[k][i][e] * mo.grad_scale, now = mix(g, old[k][i][e], mo);
                        old[k][i][e] = now;
                        v[k][i][e] = mo.nesterov ? mix(g, now, mo) : now;
                    }
                    put(m1, GC_F32, nb + k, i, old[k][i]);
                }
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    sum = __builtin_fma(double(v[k][i][e]), double(v[k][i][e]), sum);
    });
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1)
        sum += __shfl_xor(sum, off);
    if (lane == 0)
        norm_parts[wave] = sum;
    __syncthreads();
    sum = norm_parts[0];
    for (int w = 1; w < kResidentWaves; ++w)
        sum += norm_parts[w];
    // times 2^14 / (norm + eps): its power of two by itself, as the quotient may
    // be past fp32 where the values are not
    int power;
    const float factor = float(frexp(1.0 / (sqrt(sum) + double(in.eps)), &power));
    power += kXExp;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                x[nb][i][e] = __builtin_amdgcn_ldexpf(x[nb][i][e], power) * factor;

    const auto quad_of = [](const f32x16& v, int q) {
        f32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = v[4 * q + e];
        return w;
    };
    for (int s = 0; s < steps; ++s) {
        const float ca = coef.v[s][0], cb = coef.v[s][1], cc = coef.v[s][2];
        int lane = threadIdx.x & (kWave - 1);
        asm volatile("" : "+v"(lane));  // places in LDS are found anew in each step, too
        // X into LDS
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            if (owns(nb)) {
#pragma unroll
                for (int i = 0; i < RB; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        X.set(row_of(nb, i, lane), col_of(nb, i, q, lane), quad_of(x[nb][i], q));
            }
        __syncthreads();

        // A = X X'
        f32x16 acc[kOwn];
        const int part = kSplit > 1 ? wave / kBlocks : 0;
        const auto block = [&](int o) { return kSplit > 1 ? wave % kBlocks : wave * kOwn + o; };
#pragma unroll
        for (int o = 0; o < kOwn; ++o)
            acc[o] = f32x16{};
        for (int k = part; k < 2 * blocks; k += kSplit) {
#pragma unroll
            for (int o = 0; o < kOwn; ++o) {
                s16x8 fa[kPlanes], fb[kPlanes];
#pragma unroll
                for (int p = 0; p < kPlanes; ++p) {
                    const auto of = [&](int first) {
                        return kTall ? X.plane[p].by_k(first, 16 * k, lane) : X.plane[p].by_rows(first, 16 * k, lane);
                    };
                    fa[p] = of(block(o) / RB * 32);
                    fb[p] = of(block(o) % RB * 32);
                }
                acc[o] = multiply_planes<kPlanes>(fa, fb, acc[o]);
            }
        }
        // (row and column of a quad of a block: the product is symmetric, so
        // that four values below one another are four side by side)
        const auto quad_place = [&](int o, int q, int& row, int& col) {
            col = block(o) / RB * 32 + int(acc_row(4 * q, lane));
            row = block(o) % RB * 32 + int(acc_col(lane));
        };
        // On the diagonal of a block of the diagonal lies at most one of a lane's
        // values, the one of this index (else 16): it leaves for `to` and becomes 0.
        const int n = lane & 31, own = (n >> 2 & 1) == lane >> 5 ? (n >> 3) * 4 + (n & 3) : 16;
        const auto take_diagonal = [&](f32x16& v, int o, float* to, float times, float more) {
            if (block(o) / RB != block(o) % RB)
                return;
            float d = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                d = e == own ? v[e] : d;
                v[e] = e == own ? 0.0f : v[e];
            }
            if (own < 16)
                to[block(o) / RB * 32 + n] = __builtin_fmaf(d, times, more);
        };
        if (kSplit > 1) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (part > 0)
                    sums[(((part - 1) * kBlocks + block(0)) * 16 + e) * kWave + lane] = acc[0][e];
            __syncthreads();
            if (part == 0) {
#pragma unroll
                for (int k = 0; k < kSplit - 1; ++k)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        acc[0][e] += sums[((k * kBlocks + block(0)) * 16 + e) * kWave + lane];
            }
            __syncthreads();
        }
        if (part == 0) {
#pragma unroll
            for (int o = 0; o < kOwn; ++o) {
                acc[o] *= pow2<kAExp - 2 * kXExp>;
                take_diagonal(acc[o], o, diagonal_a, pow2<-kAExp>, 0.0f);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    int row, col;
                    quad_place(o, q, row, col);
                    A.set(row, col, quad_of(acc[o], q));
                }
            }
        }
        __syncthreads();

        // P = b A + c A^2
        if (part == 0) {
#pragma unroll
            for (int o = 0; o < kOwn; ++o)
                acc[o] = f32x16{};
            for (int k = 0; k < RP; k += 16) {
#pragma unroll
                for (int o = 0; o < kOwn; ++o) {
                    s16x8 fa[kPlanes], fb[kPlanes];
#pragma unroll
                    for (int p = 0; p < kPlanes; ++p) {
                        fa[p] = A.plane[p].by_rows(block(o) / RB * 32, k, lane);
                        fb[p] = A.plane[p].by_rows(block(o) % RB * 32, k, lane);
                    }
                    acc[o] = multiply_planes<kPlanes>(fa, fb, acc[o]);
                }
            }
#pragma unroll
            for (int o = 0; o < kOwn; ++o) {
                const float d = diagonal_a[block(o) % RB * 32 + int(acc_col(lane))];
                const float of_row = (cb + cc * d) * pow2<kPExp - kAExp>, of_col = cc * pow2<kPExp - kAExp>;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    int row, col;
                    quad_place(o, q, row, col);
                    const f32x4 a = A.get(row, col), da = *reinterpret_cast<const f32x4*>(diagonal_a + col);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[o][4 * q + e] = __builtin_fmaf(a[e], __builtin_fmaf(of_col, da[e], of_row),
                                                           acc[o][4 * q + e] * (cc * pow2<kPExp - 2 * kAExp>));
                }
                take_diagonal(acc[o], o, diagonal_p, pow2<-kPExp>, (cb + cc * d) * d);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    int row, col;
                    quad_place(o, q, row, col);
                    P.set(row, col, quad_of(acc[o], q));
                }
            }
        }
        __syncthreads();

        // X = a X + P X (X P of a tall one)
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f32x4 d;
                if (kTall)
                    d = *reinterpret_cast<const f32x4*>(diagonal_p + i * 32 + acc_row(4 * q, lane));
                else
                    d = f32x4{} + diagonal_p[i * 32 + acc_col(lane)];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float self = (ca + d[e]) * pow2<kPExp>;
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
                        x[nb][i][4 * q + e] *= self;
                }
            }
#pragma unroll 1  // (or what all its turns read is held at once)
        for (int k = 0; k < RP; k += 16) {
            s16x8 fp[RB][kPlanes];
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int p = 0; p < kPlanes; ++p)
                    fp[i][p] = P.plane[p].by_rows(i * 32, k, lane);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                if (!owns(nb))
                    break;
                const int first = (nb * kResidentWaves + wave) * 32;
                s16x8 fx[kPlanes];
#pragma unroll
                for (int p = 0; p < kPlanes; ++p)
                    fx[p] = kTall ? X.plane[p].by_rows(first, k, lane) : X.plane[p].by_k(first, k, lane);
#pragma unroll
                for (int i = 0; i < RB; ++i)
                    x[nb][i] = kTall ? multiply_planes<kPlanes>(fp[i], fx, x[nb][i])
                                     : multiply_planes<kPlanes>(fx, fp[i], x[nb][i]);
            }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < RB; ++i)
                x[nb][i] *= pow2<-kPExp>;
        // (each wave writes again only the part of X that it alone has read in
        // the update; the others are done with it since the barrier behind A)
    }

    float keep = 0.0f, times = last.scale * pow2<-kXExp>;
    if (moves) {
        const float lr = last.lr_scale ? last.lr * *last.lr_scale : last.lr;
        keep = __builtin_fmaf(-lr, last.decay, 1.0f);
        times = -lr * last.scale * pow2<-kXExp>;
    }
    columns([&](int nb, f32x16 (&v)[kAtOnce][RB]) {
        f32x16 w[kAtOnce][RB] = {};
        if (moves) {
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
                for (int i = 0; i < RB; ++i)
                    get(weights, out_dtype, nb + k, i, w[k][i]);
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
#pragma unroll
            for (int i = 0; i < RB; ++i) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    v[k][i][e] = moves ? __builtin_fmaf(w[k][i][e], keep, v[k][i][e] * times) : v[k][i][e] * times;
                put(out, out_dtype, nb + k, i, v[k][i]);
            }
    });
}

// Calls f(RB, NB, planes), as integral constants, for the resident kernel of a
// matrix of r x c, if there is one: X has to fit 128 registers a lane and, next
// to A and P, 160 KB of LDS.
template <typename F>
bool with_resident(size_t r, size_t c, bool both, F f)
{
    const size_t rb = r <= 32 ? 1 : r <= 64 ? 2 : 4, nb = ceil_div(ceil_div(c, 32), kResidentWaves);
    const auto call = [&](auto RB, auto NB, auto planes) {
        f(RB, NB, planes);
        return true;
    };
    using std::integral_constant;
    const integral_constant<int, 1> one;
    const integral_constant<int, 2> two;
    const integral_constant<int, 4> four;
    if (r > 128 || nb > 4)
        return false;
    if (rb == 1)
        return both ? (nb == 1 ? call(one, one, two) : call(one, four, two))
                    : (nb == 1 ? call(one, one, one) : call(one, four, one));
    if (nb == 1 && !(rb == 4 && both))
        return rb == 4 ? call(four, one, one) : both ? call(two, one, two) : call(two, one, one);
    return rb == 2 && !both ? call(two, four, one) : false;
}

}  // namespace
}  // namespace gcq
