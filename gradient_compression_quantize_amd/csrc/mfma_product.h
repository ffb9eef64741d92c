// mfma_product.h -- the tiled bf16 matrix product under linear_xent.hip.
//
// out[b][a] = sum over segments, sum over k of A(a, k) * B(b, k), fp32 sums in
// the matrix cores. An operand is a matrix of bf16 in one of two layouts:
//   by rows (kKRows = false): row a holds its k values contiguously;
//   by k    (kKRows = true):  row k holds the values of all a contiguously.
// The second is read out of LDS with the transposing load (ds_read_b64_tr_b16:
// in each 16 lanes, lane j brings the 4 values of row j/4 at columns 4 (j % 4)
// and lane i receives column i of the 4 rows), so that no operand is ever
// transposed in memory.
//
// Precision: an operand of more than 8 significant bits is held as up to three
// planes of bf16, x = p0 + p1 + p2, each the rounding of what the ones before
// left (at most 2^-8 of it, so 2^-8, 2^-16 and 2^-24 of x after one, two and
// three). A product then runs over segments, one for each pair (i, j) of
// planes with i + j up to a limit: what a limit of 2 drops is 2^-24 of a term,
// what a limit of 1 drops 2^-16.
//
// A workgroup of kWavesA x kWavesB waves owns a tile of kTA x kTB outputs. A
// stage is 64 values of k of both operands, moved straight into LDS
// (buffer_load ... lds, 16 bytes a lane) while the stage before it is
// multiplied. LDS holds 16-byte chunks permuted by an XOR of the row, which
// the loads apply to their global addresses (LDS-direct loads write lane after
// lane) and the fragment reads to their LDS addresses.
#pragma once

#include "values.h"

namespace gcq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kStageK = 64;

struct MatOperand {
    const bf16_t* plane0;
    size_t plane_stride;  // values from plane to plane
    uint32_t ld;          // values from row to row: a multiple of 8
    uint32_t extent;  // by rows: rows that may be read; by k: columns that may be read (a multiple of 8)
    uint32_t krows;   // by k: rows that may be read (a last stage past them reads the last one again,
                      // against zeros of the other operand)
};

struct ProductShape {
    uint32_t stages;    // of one segment: ceil(k / 64)
    uint32_t segments;  // pairs of planes: 1 .. 6
    uint32_t pair_a, pair_b;  // the planes of segment s: two bits each, at bit 2 s
    uint32_t tiles_a, tiles_b, splits;
};

// The pairs (i, j) of planes with i + j <= limit.
inline void set_pairs(ProductShape& sh, int planes_a, int planes_b, int limit)
{
    sh.segments = sh.pair_a = sh.pair_b = 0;
    for (int i = 0; i < planes_a; ++i)
        for (int j = 0; j < planes_b && i + j <= limit; ++j) {
            sh.pair_a |= uint32_t(i) << (2 * sh.segments);
            sh.pair_b |= uint32_t(j) << (2 * sh.segments);
            ++sh.segments;
        }
}

// What one lane and wave move of an operand's stage, T rows (or columns) wide.
template <bool kKRows, int T, int kWaves>
struct StageLoader {
    static constexpr int kLoads = T / 8 / kWaves;  // 1 KB wave loads
    static_assert(kLoads >= 1, "every wave moves at least one load");
    static constexpr int kChunks = T / 8;                 // by k: 16-byte chunks of a row
    static constexpr int kRowsPerLoad = 1024 / (2 * T);   // by k
    uint32_t off[kLoads];  // by rows: byte offset of each load; by k: of its columns alone
    uint32_t row;          // by k: the first load's row
    int wave;

    // XOR on the chunk index of LDS row `row` (see the file comment).
    static __device__ __forceinline__ uint32_t swizzle(uint32_t row)
    {
        return kKRows ? 2 * (row & 3) : row & 7;
    }

    __device__ __forceinline__ void init(const MatOperand& m, uint32_t first, int wave_, int lane)
    {
        wave = wave_;
        row = wave * kLoads * kRowsPerLoad + lane / kChunks;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            if (kKRows) {
                const uint32_t chunk = (lane % kChunks) ^ swizzle(row + j * kRowsPerLoad);
                off[j] = min(first + chunk * 8, m.extent - 8) * 2;
            } else {
                const uint32_t r = (wave * kLoads + j) * 8 + lane / 8;
                const uint32_t chunk = (lane & 7) ^ swizzle(r);
                off[j] = min(first + r, m.extent - 1) * m.ld * 2 + chunk * 16;
            }
        }
    }

    // Enqueues the stage from k0 on of plane p into lds.
    __device__ __forceinline__ void load(const MatOperand& m, const bf16_t* p, uint32_t k0, bf16_t* lds) const
    {
        const bf16_t* base = p + (kKRows ? size_t(k0) * m.ld : size_t(k0));
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<bf16_t*>(base), 0, 0xFFFFFFFFu,
                                                            0x00020000);
        const uint32_t last = m.krows - 1 - k0;  // by k: the last row of the stage that may be read
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            // rows of a stage and the bytes of a row fit 24 bits
            const uint32_t o =
                kKRows ? __umul24(min(row + j * kRowsPerLoad, last), m.ld * 2) + off[j] : off[j];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (__attribute__((address_space(3))) void*)(lds + (wave * kLoads + j) * 512), 16, o, 0, 0, 0);
        }
    }
};

// Fragments of 32 rows (or columns) x 16 k: lane l holds row l % 32, k values
// 8 (l / 32) .. + 7.
template <bool kKRows, int T>
struct FragmentReader {
    uint32_t base;  // byte offset of this lane at fragment 0, k 0

    __device__ __forceinline__ void init(uint32_t first, int lane)
    {
        if (kKRows) {
            const uint32_t g = lane >> 4, j = lane & 15;
            const uint32_t row = 8 * (g >> 1) + (j >> 2);
            const uint32_t col = first + 16 * (g & 1) + 4 * (j & 3);
            base = row * (2 * T) + (((col >> 3) ^ (2 * (row & 3))) << 4) + ((col & 4) << 1);
        } else {
            const uint32_t row = first + (lane & 31);
            base = row * 128 + (((lane >> 5) ^ (row & 7)) << 4);
        }
    }

    // Fragment f (32 f rows on), k values 16 kk on.
    __device__ __forceinline__ bf16x8 read(const bf16_t* lds, int f, int kk) const
    {
        if (kKRows) {
            typedef __attribute__((address_space(3))) s16x4* lds_ptr;
            // chunk + 4 f under the XOR of bits 1 and 2: bit 2 of 4 f meets it, the rest adds
            const char* p = reinterpret_cast<const char*>(lds) + (base ^ (uint32_t(f) << 6)) + kk * 16 * (2 * T);
            union {
                s16x4 h[2];
                bf16x8 v;
            } u;
            u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p));
            u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * (2 * T)));
            return u.v;
        }
        const char* p = reinterpret_cast<const char*>(lds) + (base ^ (uint32_t(kk) << 5)) + f * (32 * 128);
        return *reinterpret_cast<const bf16x8*>(p);
    }
};

template <bool kAK, bool kBK, int TA, int TB, int WA, int WB>
struct TileProduct {
    static constexpr int kWaves = WA * WB;
    static constexpr int kThreads = kWaves * kWave;
    static constexpr int RA = TA / WA / 32, RB = TB / WB / 32;  // 32 x 32 products of a wave
    using LoadA = StageLoader<kAK, TA, kWaves>;
    using LoadB = StageLoader<kBK, TB, kWaves>;

    struct Acc {
        f32x16 v[RA][RB];
    };

    // Multiplies stages [s0, s1) of the tile at (a0, b0). The four buffers
    // are LDS variables of their own, so that the compiler knows which loads
    // a fragment read has to wait for.
    static __device__ __forceinline__ void run(const MatOperand& A, const MatOperand& B,
                                               const ProductShape& sh, uint32_t a0, uint32_t b0,
                                               uint32_t s0, uint32_t s1, bf16_t* la0, bf16_t* la1,
                                               bf16_t* lb0, bf16_t* lb1, Acc& acc)
    {
        const int lane = threadIdx.x & (kWave - 1);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        const int wa = wave % WA, wb = wave / WA;
        LoadA ga;
        LoadB gb;
        ga.init(A, a0, wave, lane);
        gb.init(B, b0, wave, lane);
        FragmentReader<kAK, TA> fa;
        FragmentReader<kBK, TB> fb;
        fa.init(wa * (TA / WA), lane);
        fb.init(wb * (TB / WB), lane);
#pragma unroll
        for (int i = 0; i < RA; ++i)
#pragma unroll
            for (int j = 0; j < RB; ++j)
                acc.v[i][j] = f32x16{};

        // the stage that is fetched next
        uint32_t seg = s0 / sh.stages, k0 = (s0 - seg * sh.stages) * kStageK;
        const auto fetch = [&](bf16_t* la, bf16_t* lb) {
            const uint32_t pa = (sh.pair_a >> (2 * seg)) & 3, pb = (sh.pair_b >> (2 * seg)) & 3;
            ga.load(A, A.plane0 + pa * A.plane_stride, k0, la);
            gb.load(B, B.plane0 + pb * B.plane_stride, k0, lb);
            k0 += kStageK;
            if (k0 == sh.stages * kStageK) {
                k0 = 0;
                ++seg;
            }
        };
        // the fragments of the next 16 values of k are read while these are
        // multiplied
        const auto multiply = [&](const bf16_t* la, const bf16_t* lb) {
            bf16x8 a[2][RA], b[2][RB];
            const auto read = [&](int kk) {
#pragma unroll
                for (int j = 0; j < RB; ++j)
                    b[kk & 1][j] = fb.read(lb, j, kk);
#pragma unroll
                for (int i = 0; i < RA; ++i)
                    a[kk & 1][i] = fa.read(la, i, kk);
            };
            read(0);
#pragma unroll
            for (int kk = 0; kk < kStageK / 16; ++kk) {
                if (kk + 1 < kStageK / 16)
                    read(kk + 1);
#pragma unroll
                for (int i = 0; i < RA; ++i)
#pragma unroll
                    for (int j = 0; j < RB; ++j)
                        acc.v[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[kk & 1][i], b[kk & 1][j],
                                                                              acc.v[i][j], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (s0 >= s1)
            return;
        // One barrier a stage: behind it every wave's loads of the stage are in
        // LDS and every wave is done with the buffers that the next stage's
        // loads then overwrite.
        fetch(la0, lb0);
        uint32_t s = s0;
        for (; s + 2 <= s1; s += 2) {
            stage_ready();
            fetch(la1, lb1);
            multiply(la0, lb0);
            stage_ready();
            if (s + 2 < s1)
                fetch(la0, lb0);
            multiply(la1, lb1);
        }
        stage_ready();
        if (s < s1) {
            multiply(la0, lb0);
            workgroup_sync();
        }
    }

    static __device__ __forceinline__ void stage_ready()
    {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        workgroup_sync();
    }

    static __device__ __forceinline__ void workgroup_sync()
    {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }
};

// Row (of A) and column (of B) of value i of a lane's 32 x 32 product.
__device__ __forceinline__ uint32_t acc_row(int i, int lane) { return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3); }
__device__ __forceinline__ uint32_t acc_col(int lane) { return lane & 31; }

// Tile of workgroup id: each XCD takes a contiguous range of ids, and ids run
// through patches of 8 tiles of B, so that the workgroups that share an L2 at
// one time share operands too.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t tiles_a, uint32_t tiles_b, uint32_t& ta,
                                        uint32_t& tb)
{
    constexpr uint32_t kPatch = 8;
    const uint32_t per = kPatch * tiles_a, patch = id / per, in = id - patch * per;
    const uint32_t height = min(kPatch, tiles_b - patch * kPatch);
    ta = in / height;
    tb = patch * kPatch + in % height;
}

}  // namespace
}  // namespace gcq
