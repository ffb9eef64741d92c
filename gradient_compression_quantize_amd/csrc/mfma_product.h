// mfma_product.h -- the tiled matrix product under linear_xent.hip.
//
// out[b][a] = sum over segments, sum over k of A(a, k) * B(b, k), 16-bit
// factors, fp32 sums in the matrix cores. An operand is a matrix of bf16 or
// fp16 in one of two layouts:
//   by rows (kKRows = false): row a holds its k values contiguously;
//   by k    (kKRows = true):  row k holds the values of all a contiguously.
// The second is read out of LDS with the transposing load (ds_read_b64_tr_b16:
// in each 16 lanes, lane j brings the 4 values of row j/4 at columns 4 (j % 4)
// and lane i receives column i of the 4 rows), so that no operand is ever
// transposed in memory.
//
// Precision: an operand of more than 11 significant bits is held as two planes
// of fp16, x = p0 + 2^-11 p1, p0 the rounding of x (off by at most 2^-11 of it)
// and p1 that of the rest times 2^11: together they are within 2^-22 of x, as
// long as x is within 2^-28 of the largest value (which the caller scales to
// [2^14, 2^15)), and below that within 2^-50 of the largest value (half of
// 2^-24, the smallest fp16, times 2^-11). A product then runs over segments,
// one for each pair of planes: first those of one p1, whose sum is then
// multiplied by 2^-11, then p0 p0. The pair of two p1, at most 2^-22 of a term,
// is left out.
//
// A workgroup of WA x WB waves owns a tile of TA x TB outputs. k advances in
// stages of 32 values of both operands, moved straight into LDS
// (buffer_load ... lds, 16 bytes a lane) by way of four buffers: while stage s
// is multiplied, s + 1 is there (its first fragments are read under the last
// products of s), s + 2 is on its way and s + 3 is asked for. LDS holds 16-byte
// chunks permuted by an XOR of the row, which the loads apply to their global
// addresses (LDS-direct loads write lane after lane) and the fragment reads to
// their LDS addresses.
//
// Measured on 8192 x 64000 x 4096 bf16: 1.13 to 1.27 PFLOP/s (torch's library
// product of that shape: 1.50). The matrix cores are busy 62 to 70% of the
// cycles, and power holds the clock near 1.7 GHz: the first form, two stages of
// 64 k with the reads of one stage behind its barrier, kept them busy 46% at
// 2.16 GHz and was a tenth slower. Tiles of 128 x 128, two to a compute unit,
// were a fifth slower; four waves of 128 x 128 outputs each half as fast;
// s_setprio around the products made no difference.
#pragma once

#include "values.h"

namespace gcq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kStageK = 32;
constexpr int kBuffers = 4;

// k is padded to whole turns of the four buffers.
constexpr int kTurnK = kBuffers * kStageK;

struct MatOperand {
    const uint16_t* plane0;
    size_t plane_stride;  // values from plane to plane
    uint32_t ld;          // values from row to row: a multiple of 8
    uint32_t extent;  // by rows: rows that may be read; by k: columns that may be read (a multiple of 8)
    uint32_t krows;   // by k: rows that may be read (what lies past them reads the last one again, against
                      // zeros of the other operand)
    const int* exponent;  // values are held times 2^exponent; NULL: 0
    bool by_row;          // row r times 2^exponent[r]
};

struct ProductShape {
    uint32_t turns;     // of one segment: ceil(k / 128)
    uint32_t segments;  // pairs of planes: 1 .. 3
    uint32_t pair_a, pair_b;  // the planes of segment s: two bits each, at bit 2 s
    uint32_t fold;      // segments whose sum is multiplied by 2^-11: the first so many
    uint32_t tiles_a, tiles_b, splits;
};

// The pairs (0, 1), (1, 0), (0, 0) of planes, as far as they exist.
inline void set_pairs(ProductShape& sh, int planes_a, int planes_b)
{
    sh.segments = sh.pair_a = sh.pair_b = 0;
    const auto add = [&](uint32_t i, uint32_t j) {
        sh.pair_a |= i << (2 * sh.segments);
        sh.pair_b |= j << (2 * sh.segments);
        ++sh.segments;
    };
    if (planes_b == 2)
        add(0, 1);
    if (planes_a == 2)
        add(1, 0);
    sh.fold = sh.segments;
    add(0, 0);
}

// What one lane and wave move of an operand's stage, T rows (or columns) wide.
template <bool kKRows, int T, int kWaves>
struct StageLoader {
    static constexpr int kLoads = T / 16 / kWaves;  // 1 KB wave loads
    static_assert(kLoads >= 1, "every wave moves at least one load");
    static constexpr int kChunks = T / 8;                // by k: 16-byte chunks of a row
    static constexpr int kRowsPerLoad = 1024 / (2 * T);  // by k
    uint32_t off[kLoads];  // by rows: byte offset of each load from the tile's first row; by k: of its columns alone
    uint32_t row;          // by k: the first load's row
    size_t origin;         // by rows: values before the tile's first row
    int wave;

    // XOR on the chunk index of LDS row `row`, so that what is read in one
    // clock covers the 64 banks (256 bytes): by rows (64 bytes each) the same
    // chunk of 16 rows, by k 64 bytes of 4 rows. SQ_LDS_BANK_CONFLICT is zero;
    // covering 32 banks alone left it at half of SQ_LDS_IDX_ACTIVE.
    static __device__ __forceinline__ uint32_t swizzle(uint32_t row)
    {
        return kKRows ? 4 * (row & 3) : (row >> 2) & 3;
    }

    __device__ __forceinline__ void init(const MatOperand& m, uint32_t first, int wave_, int lane)
    {
        wave = wave_;
        origin = kKRows ? 0 : size_t(first) * m.ld;
        row = wave * kLoads * kRowsPerLoad + lane / kChunks;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            if (kKRows) {
                const uint32_t chunk = (lane % kChunks) ^ swizzle(row + j * kRowsPerLoad);
                off[j] = min(first + chunk * 8, m.extent - 8) * 2;
            } else {
                const uint32_t r = (wave * kLoads + j) * 16 + lane / 4;
                const uint32_t chunk = (lane & 3) ^ swizzle(r);
                // 255 rows of up to 2^22 bytes
                off[j] = min(r, m.extent - 1 - first) * m.ld * 2 + chunk * 16;
            }
        }
    }

    // Where the stage from k0 on of plane p starts, as a descriptor of `bytes`
    // bytes: of none, its loads fetch nothing.
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t stage(const MatOperand& m, const uint16_t* p, uint32_t k0,
                                                            uint32_t bytes) const
    {
        // (by k: not past the last row)
        const uint16_t* base = p + (kKRows ? size_t(min(k0, m.krows - 1)) * m.ld : origin + k0);
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), 0, bytes, 0x00020000);
    }

    // Enqueues load j of the stage into lds.
    __device__ __forceinline__ void load(const MatOperand& m, __amdgpu_buffer_rsrc_t at, uint32_t k0, int j,
                                         uint16_t* lds) const
    {
        // by k: the last row of the stage that may be read; rows of a stage
        // and the bytes of a row fit 24 bits
        const uint32_t last = m.krows - 1 - min(k0, m.krows - 1);
        const uint32_t o = kKRows ? __umul24(min(row + j * kRowsPerLoad, last), m.ld * 2) + off[j] : off[j];
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            at, (__attribute__((address_space(3))) void*)(lds + (wave * kLoads + j) * 512), 16, o, 0, 0, 0);
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
            base = row * (2 * T) + (((col >> 3) ^ StageLoader<true, T, 1>::swizzle(row)) << 4) + ((col & 4) << 1);
        } else {
            const uint32_t row = first + (lane & 31);
            base = row * (2 * kStageK) + (((lane >> 5) ^ StageLoader<false, T, 1>::swizzle(row)) << 4);
        }
    }

    // Fragment f (32 f rows on), k values 16 kk on.
    __device__ __forceinline__ s16x8 read(const uint16_t* lds, int f, int kk) const
    {
        if (kKRows) {
            typedef __attribute__((address_space(3))) s16x4* lds_ptr;
            // 4 f chunks on: the XOR reaches bits 2 and 3 of the chunk, which 4 f meets too
            const char* p = reinterpret_cast<const char*>(lds) + (base ^ (uint32_t(f) << 6)) + kk * 16 * (2 * T);
            union {
                s16x4 h[2];
                s16x8 v;
            } u;
            u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p));
            u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * (2 * T)));
            return u.v;
        }
        const char* p = reinterpret_cast<const char*>(lds) + (base ^ (uint32_t(kk) << 5)) + f * (32 * 2 * kStageK);
        return *reinterpret_cast<const s16x8*>(p);
    }
};

// The LDS of a tile, as variables of their own, so that the compiler knows
// which loads a fragment read has to wait for.
struct TileBuffers {
    uint16_t *a[kBuffers], *b[kBuffers];
};

#define GCQ_TILE_BUFFERS(name, TA, TB)                                                                       \
    __shared__ uint16_t name##_a0[(TA) * kStageK], name##_a1[(TA) * kStageK], name##_a2[(TA) * kStageK],       \
        name##_a3[(TA) * kStageK], name##_b0[(TB) * kStageK], name##_b1[(TB) * kStageK],                     \
        name##_b2[(TB) * kStageK], name##_b3[(TB) * kStageK];                                                \
    const TileBuffers name = {{name##_a0, name##_a1, name##_a2, name##_a3},                                  \
                              {name##_b0, name##_b1, name##_b2, name##_b3}}

// kF16: fp16 operands, else bf16.
template <bool kF16, bool kAK, bool kBK, int TA, int TB, int WA, int WB>
struct TileProduct {
    static constexpr int kWaves = WA * WB;
    static constexpr int RA = TA / WA / 32, RB = TB / WB / 32;  // 32 x 32 products of a wave
    using LoadA = StageLoader<kAK, TA, kWaves>;
    using LoadB = StageLoader<kBK, TB, kWaves>;

    struct Acc {
        f32x16 v[RA][RB];
    };

    // Multiplies turns [t0, t1) of the tile at (a0, b0). LDS is free for
    // other use when it returns.
    static __device__ __forceinline__ void run(const MatOperand& A, const MatOperand& B, const ProductShape& sh,
                                               uint32_t a0, uint32_t b0, uint32_t t0, uint32_t t1,
                                               const TileBuffers& lds, Acc& acc)
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
        if (t0 >= t1)
            return;

        // the stage that is fetched next: its place in the planes, and how
        // many are left
        const uint32_t k_end = sh.turns * kTurnK;
        uint32_t seg = t0 / sh.turns, k0 = (t0 - seg * sh.turns) * kTurnK, left = (t1 - t0) * kBuffers;
        struct Fetch {
            __amdgpu_buffer_rsrc_t a, b;
            uint32_t k0;
        };
        const auto next_stage = [&]() {
            const uint32_t pa = (sh.pair_a >> (2 * seg)) & 3, pb = (sh.pair_b >> (2 * seg)) & 3;
            // (readfirstlane keeps what the compiler would select in vector
            // registers in scalar ones)
            const uint32_t bytes = __builtin_amdgcn_readfirstlane(left ? 0xFFFFFFFFu : 0u);
            const Fetch f = {ga.stage(A, A.plane0 + pa * A.plane_stride, k0, bytes),
                             gb.stage(B, B.plane0 + pb * B.plane_stride, k0, bytes), k0};
            left -= bytes & 1;
            k0 += kStageK;
            const uint32_t over = __builtin_amdgcn_readfirstlane(k0 == k_end ? 1u : 0u);
            seg += over;
            k0 -= over * k_end;
            return f;
        };
        constexpr int kLoads = LoadA::kLoads + LoadB::kLoads;
        const auto load = [&](const Fetch& f, int j, int buffer) {
            if (j < LoadA::kLoads)
                ga.load(A, f.a, f.k0, j, lds.a[buffer]);
            else if (j < kLoads)
                gb.load(B, f.b, f.k0, j - LoadA::kLoads, lds.b[buffer]);
        };

#pragma unroll
        for (int s = 0; s < kBuffers - 1; ++s) {
            const Fetch f = next_stage();
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                load(f, j, s);
        }
        wait_loads<2 * kLoads>();
        s16x8 a[2][RA], b[2][RB];
#pragma unroll
        for (int j = 0; j < RB; ++j)
            b[0][j] = fb.read(lds.b[0], j, 0);
#pragma unroll
        for (int i = 0; i < RA; ++i)
            a[0][i] = fa.read(lds.a[0], i, 0);

        const uint32_t fold = sh.fold * sh.turns;
        for (uint32_t t = t0; t < t1; ++t) {
            if (t == fold && t > t0)
                scale(acc);
#pragma unroll
            for (int s = 0; s < kBuffers; ++s) {
                // behind the barrier stage s + 1 is in LDS for everybody, and
                // nobody reads the buffer of s - 1 any more, which s + 3 takes
                wait_loads<kLoads>();
                const Fetch f = next_stage();
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const int from = kk == 0 ? s : (s + 1) % kBuffers;
                    // each row of products runs over the reads of a fragment
                    // of the next 16 k and one load
#pragma unroll
                    for (int i = 0; i < (RA > RB ? RA : RB); ++i) {
                        if (i < RB)
                            b[kk ^ 1][i] = fb.read(lds.b[from], i, kk ^ 1);
                        if (i < RA)
                            a[kk ^ 1][i] = fa.read(lds.a[from], i, kk ^ 1);
                        constexpr int kSteps = 2 * (RA > RB ? RA : RB), kEach = (kLoads + kSteps - 1) / kSteps;
#pragma unroll
                        for (int e = 0; e < kEach; ++e)
                            load(f, (kk * (RA > RB ? RA : RB) + i) * kEach + e, (s + kBuffers - 1) % kBuffers);
                        if (i < RA) {
#pragma unroll
                            for (int j = 0; j < RB; ++j)
                                acc.v[i][j] = multiply(a[kk][i], b[kk][j], acc.v[i][j]);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
        }
        if (t1 <= fold)
            scale(acc);
        wait_loads<0>();
    }

    static __device__ __forceinline__ f32x16 multiply(s16x8 a, s16x8 b, f32x16 c)
    {
        if constexpr (kF16)
            return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b),
                                                          c, 0, 0, 0);
        else
            return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                           __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }

    // The sum of the segments of a second plane, in the first one's units.
    static __device__ __forceinline__ void scale(Acc& acc)
    {
#pragma unroll
        for (int i = 0; i < RA; ++i)
#pragma unroll
            for (int j = 0; j < RB; ++j)
                acc.v[i][j] *= 0x1p-11f;
    }

    // Waits until all but the last N loads of this wave are in LDS, then for
    // every wave of the workgroup to get there.
    template <int N>
    static __device__ __forceinline__ void wait_loads()
    {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
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
