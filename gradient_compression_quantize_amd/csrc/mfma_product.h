// mfma_product.h -- the tiled matrix product under linear_xent.hip and
// orthogonalize.hip.
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
// is left out. (orthogonalize.hip holds p1 as it is, in a range of its own: kPlain.)
//
// A workgroup of WA x WB waves owns a tile of TA x TB outputs. k advances in
// stages of 32 values of both operands, moved straight into LDS
// (buffer_load ... lds, 16 bytes a lane) by way of four buffers (eight of small
// tiles: kRing): while stage s is multiplied, s + 1 is there (its first fragments
// are read under the last products of s), s + 2 is on its way and s + 3 is asked
// for. LDS holds 16-byte chunks permuted by an XOR of the row, which the loads
// apply to their global addresses (LDS-direct loads write lane after lane) and
// the fragment reads to their LDS addresses.
//
// Measured on 8192 x 64000 x 4096 bf16: 1.13 to 1.27 PFLOP/s (torch's library
// product of that shape: 1.50). The matrix cores are busy 62 to 70% of the
// cycles, and power holds the clock near 1.7 GHz (4096 x 4096 x 4096 fp16: 1.0 to
// 1.1 PFLOP/s of random values, 1.7 of zeros): the first form, two stages of
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
// kPlain: every row of every stage of an operand by k may be read (else the last
// one that may be stands for those behind it). kPaired (of kPlain): rows hold 16
// values of the first plane, then those of the second, and so on, and a stage is 16
// values of k of both.
template <bool kKRows, int T, int kWaves, bool kPlain = false, bool kPaired = false>
struct StageLoader {
    static_assert(kPlain || !kPaired, "paired planes are plain");
    static constexpr int kLoads = T / 16 / kWaves;  // 1 KB wave loads
    static_assert(kLoads >= 1, "every wave moves at least one load");
    static constexpr int kWidth = kPaired ? 2 * T : T;        // by k: values of a row
    static constexpr int kChunks = kWidth / 8;                // its 16-byte chunks
    static constexpr int kRowsPerLoad = 1024 / (2 * kWidth);
    static constexpr bool kClamped = kKRows && !kPlain;
    // byte offset of each load: by rows from the tile's first row, by k from
    // the stage's first row (clamped: of its columns alone)
    uint32_t off[kLoads];
    uint32_t row;   // by k: the first load's row
    uint32_t step;  // bytes from stage to stage
    size_t origin;  // by rows: values before the tile's first row
    int wave;

    // XOR on the chunk index of LDS row `row`, so that what is read in one
    // clock covers the 64 banks (256 bytes): by rows (64 bytes each) the same
    // chunk of 16 rows, by k 64 bytes of 4 rows, in halves that lie 64 bytes apart
    // where planes are paired; rows of 128 bytes are two to the 256.
    // SQ_LDS_BANK_CONFLICT is zero; covering 32 banks alone left it at half of
    // SQ_LDS_IDX_ACTIVE.
    static __device__ __forceinline__ uint32_t swizzle(uint32_t row)
    {
        if (!kKRows)
            return (row >> 2) & 3;
        return kPaired ? 2 * (row & 1) + 4 * (row & 2) : kWidth >= 128 ? 4 * (row & 3) : 2 * (row & 2);
    }

    __device__ __forceinline__ void init(const MatOperand& m, uint32_t first, int wave_, int lane)
    {
        wave = wave_;
        origin = kKRows ? 0 : size_t(first) * m.ld;
        step = 2 * kStageK * (kKRows ? m.ld / (kPaired ? 2 : 1) : 1);
        row = wave * kLoads * kRowsPerLoad + lane / kChunks;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            if (kKRows) {
                const uint32_t r = row + j * kRowsPerLoad, chunk = (lane % kChunks) ^ swizzle(r);
                constexpr uint32_t kOf = kPaired ? 2 : 1;
                off[j] = min(kOf * first + chunk * 8, kOf * m.extent - 8) * 2 + (kClamped ? 0 : __umul24(r, m.ld * 2));
            } else {
                const uint32_t r = (wave * kLoads + j) * 16 + lane / 4;
                const uint32_t chunk = (lane & 3) ^ swizzle(r);
                // 255 rows of up to 2^22 bytes
                off[j] = min(r, m.extent - 1 - first) * m.ld * 2 + chunk * 16;
            }
        }
    }

    // The turn from k0 on of plane p.
    __device__ __forceinline__ const uint16_t* turn(const MatOperand& m, const uint16_t* p, uint32_t k0) const
    {
        return p + (kKRows ? size_t(k0) * m.ld : origin + (kPaired ? 2 * k0 : k0));
    }

    // A descriptor of `bytes` bytes from p on: of none, its loads fetch nothing.
    static __device__ __forceinline__ __amdgpu_buffer_rsrc_t view(const uint16_t* p, uint32_t bytes)
    {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(p), 0, bytes, 0x00020000);
    }

    // Enqueues load j of stage s of the turn from k0 on, which starts at p (and
    // in `at`), into lds.
    __device__ __forceinline__ void load(const MatOperand& m, const uint16_t* p, uint32_t bytes,
                                         __amdgpu_buffer_rsrc_t at, uint32_t k0, int s, int j, uint16_t* lds) const
    {
        const auto to = (__attribute__((address_space(3))) void*)(lds + (wave * kLoads + j) * 512);
        if (kClamped) {
            // not past the last row that may be read (a turn starts in front of
            // it); rows of a stage and the bytes of a row fit 24 bits
            const uint32_t k = k0 + s * kStageK, first = min(k, m.krows - 1), last = m.krows - 1 - first;
            const uint32_t o = __umul24(min(row + j * kRowsPerLoad, last), m.ld * 2) + off[j];
            __builtin_amdgcn_raw_ptr_buffer_load_lds(view(p + size_t(first - k0) * m.ld, bytes), to, 16, o, 0, 0, 0);
        } else {
            // (an offset in the instruction itself would move the place in LDS too)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(at, to, 16, off[j], s * step, 0, 0);
        }
    }
};

// Fragments of 32 rows (or columns) x 16 k: lane l holds row l % 32, k values
// 8 (l / 32) .. + 7.
template <bool kKRows, int T, bool kPaired = false>
struct FragmentReader {
    using Stage = StageLoader<kKRows, T, 1, kPaired, kPaired>;
    static constexpr int kRow = 2 * Stage::kWidth;  // by k: bytes of a row

    uint32_t base;  // byte offset of this lane at fragment 0, k 0

    __device__ __forceinline__ void init(uint32_t first, int lane)
    {
        if (kKRows) {
            const uint32_t g = lane >> 4, j = lane & 15;
            const uint32_t row = 8 * (g >> 1) + (j >> 2);
            const uint32_t col = (first + 16 * (g & 1)) * (kPaired ? 2 : 1) + 4 * (j & 3);
            base = row * kRow + (((col >> 3) ^ Stage::swizzle(row)) << 4) + ((col & 4) << 1);
        } else {
            const uint32_t row = first + (lane & 31);
            base = row * (2 * kStageK) + (((lane >> 5) ^ Stage::swizzle(row)) << 4);
        }
    }

    // Fragment f (32 f rows on), k values 16 kk on (kPaired: plane kk).
    __device__ __forceinline__ s16x8 read(const uint16_t* lds, int f, int kk) const
    {
        if (kKRows) {
            typedef __attribute__((address_space(3))) s16x4* lds_ptr;
            // 4 f chunks on (8 f, and 2 for the second plane): the XOR of the row
            // reaches bits of the chunk that these meet too
            const uint32_t at = kPaired ? base ^ (uint32_t(f) << 7 | uint32_t(kk) << 5) : base ^ (uint32_t(f) << 6);
            const char* p = reinterpret_cast<const char*>(lds) + at + (kPaired ? 0 : kk * 16 * kRow);
            union {
                s16x4 h[2];
                s16x8 v;
            } u;
            u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p));
            u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * kRow));
            return u.v;
        }
        const char* p = reinterpret_cast<const char*>(lds) + (base ^ (uint32_t(kk) << 5)) + f * (32 * 2 * kStageK);
        return *reinterpret_cast<const s16x8*>(p);
    }
};

// The LDS of a tile, as variables of their own, so that the compiler knows
// which loads a fragment read has to wait for: a ring of four, or of eight.
struct TileBuffers {
    uint16_t *a[2 * kBuffers], *b[2 * kBuffers];
};

#define GCQ_FOUR_BUFFERS(name, values) \
    __shared__ uint16_t name##0[values], name##1[values], name##2[values], name##3[values]

#define GCQ_TILE_BUFFERS(name, TA, TB)                                             \
    GCQ_FOUR_BUFFERS(name##_a, (TA) * kStageK);                                     \
    GCQ_FOUR_BUFFERS(name##_b, (TB) * kStageK);                                     \
    const TileBuffers name = {{name##_a0, name##_a1, name##_a2, name##_a3}, \
                              {name##_b0, name##_b1, name##_b2, name##_b3}}

// (of a ring of four the others are not there: nothing reads them)
#define GCQ_TILE_RING(name, T, ring)                                                                       \
    GCQ_FOUR_BUFFERS(name##_a, (T) * kStageK);                                                              \
    GCQ_FOUR_BUFFERS(name##_b, (T) * kStageK);                                                              \
    GCQ_FOUR_BUFFERS(name##_c, (ring) == 8 ? (T) * kStageK : 1);                                            \
    GCQ_FOUR_BUFFERS(name##_d, (ring) == 8 ? (T) * kStageK : 1);                                            \
    const TileBuffers name = {                                                                             \
        {name##_a0, name##_a1, name##_a2, name##_a3, name##_c0, name##_c1, name##_c2, name##_c3}, \
        {name##_b0, name##_b1, name##_b2, name##_b3, name##_d0, name##_d1, name##_d2, name##_d3}}

// kF16: fp16 operands, else bf16. kPlain: as of StageLoader, and planes that add
// up as they are: no sum of segments is scaled. kPaired: of two such planes in both
// operands all pairs but that of two second ones, as one segment: its turns are
// of kTurnK / 2 values of k, whose planes are fetched and read out of LDS once for
// all three products: 512 tiles of 128 x 128 over 2048 k in 116 us, 145 as three
// segments; 256 of 256 x 256 in 181 and 191. kRing: buffers of a tile; 8 keep seven
// stages on their way, for small tiles, whose stages are over before what was asked
// for three of them ago has come: 256 tiles of 64 x 64 over 8192 k in 34 us instead
// of 48, over 768 in 7.6 instead of 8.0 (512, two to a compute unit: 72 and 64).
template <bool kF16, bool kAK, bool kBK, int TA, int TB, int WA, int WB, bool kPlain = false, bool kPaired = false,
          int kRing = kBuffers>
struct TileProduct {
    static constexpr int kWaves = WA * WB;
    static constexpr int RA = TA / WA / 32, RB = TB / WB / 32;  // 32 x 32 products of a wave
    using LoadA = StageLoader<kAK, TA, kWaves, kPlain, kPaired>;
    using LoadB = StageLoader<kBK, TB, kWaves, kPlain, kPaired>;
    static constexpr int kOfTurn = kPaired ? kTurnK / 2 : kTurnK;
    static_assert(kRing == kBuffers || (kRing == 2 * kBuffers && kPlain), "a ring of one turn or two");

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
        FragmentReader<kAK, TA, kPaired> fa;
        FragmentReader<kBK, TB, kPaired> fb;
        fa.init(wa * (TA / WA), lane);
        fb.init(wb * (TB / WB), lane);
#pragma unroll
        for (int i = 0; i < RA; ++i)
#pragma unroll
            for (int j = 0; j < RB; ++j)
                acc.v[i][j] = f32x16{};
        if (t0 >= t1)
            return;

        // the turn that is fetched next: its place in the planes, and how many
        // are left. Set once a turn: scalar instructions of every stage are
        // what all waves go through behind its barrier before their first
        // product.
        const uint32_t k_end = sh.turns * kOfTurn;
        uint32_t seg = t0 / sh.turns, k0 = (t0 - seg * sh.turns) * kOfTurn, left = t1 - t0;
        struct Fetch {
            __amdgpu_buffer_rsrc_t a, b;
            const uint16_t *pa, *pb;
            uint32_t k0, bytes;
        };
        const auto next_turn = [&]() {
            const uint32_t i = (sh.pair_a >> (2 * seg)) & 3, j = (sh.pair_b >> (2 * seg)) & 3;
            Fetch f;
            f.pa = ga.turn(A, A.plane0 + i * A.plane_stride, k0);
            f.pb = gb.turn(B, B.plane0 + j * B.plane_stride, k0);
            // (readfirstlane keeps what the compiler would select in vector
            // registers in scalar ones)
            f.bytes = __builtin_amdgcn_readfirstlane(left ? 0xFFFFFFFFu : 0u);
            f.k0 = k0;
            f.a = LoadA::view(f.pa, f.bytes);
            f.b = LoadB::view(f.pb, f.bytes);
            left -= f.bytes & 1;
            k0 += kOfTurn;
            const uint32_t over = __builtin_amdgcn_readfirstlane(k0 == k_end ? 1u : 0u);
            seg += over;
            k0 -= over * k_end;
            return f;
        };
        constexpr int kLoads = LoadA::kLoads + LoadB::kLoads;
        const auto load = [&](const Fetch& f, int s, int j) {
            if (j < LoadA::kLoads)
                ga.load(A, f.pa, f.bytes, f.a, f.k0, s % kBuffers, j, lds.a[s]);
            else if (j < kLoads)
                gb.load(B, f.pb, f.bytes, f.b, f.k0, s % kBuffers, j - LoadA::kLoads, lds.b[s]);
        };

        Fetch f = next_turn();
#pragma unroll
        for (int s = 0; s < kRing - 1; ++s) {
            if (s > 0 && s % kBuffers == 0)
                f = next_turn();
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                load(f, s, j);
        }
        wait_loads<(kRing - 2) * kLoads>();
        if constexpr (kPaired) {
            // Fragments of a second plane come in under the products of the two
            // first ones, those of the next stage's first planes under the third
            // products (b's beside those in use).
            s16x8 a[2][RA], b[3][RB];
#pragma unroll
            for (int j = 0; j < RB; ++j)
                b[0][j] = fb.read(lds.b[0], j, 0);
#pragma unroll
            for (int i = 0; i < RA; ++i)
                a[0][i] = fa.read(lds.a[0], i, 0);
            for (uint32_t t = t0; t < t1; t += kRing / kBuffers) {
#pragma unroll
                for (int s = 0; s < kRing; ++s) {
                    if (s > 0 && s % kBuffers == 0 && t + s / kBuffers == t1)
                        break;
                    wait_loads<(kRing - 3) * kLoads>();
                    constexpr int kSteps = 3 * (RA > RB ? RA : RB), kEach = (kLoads + kSteps - 1) / kSteps;
                    const int now = s & 1, next = now ^ 1, to = (s + 1) % kRing;
#pragma unroll
                    for (int phase = 0; phase < 3; ++phase)
#pragma unroll
                        for (int i = 0; i < (RA > RB ? RA : RB); ++i) {
                            if (phase == 0 && i < RB)
                                b[2][i] = fb.read(lds.b[s], i, 1);
                            if (phase == 0 && i < RA)
                                a[1][i] = fa.read(lds.a[s], i, 1);
                            if (phase == 2 && i < RB)
                                b[next][i] = fb.read(lds.b[to], i, 0);
                            if (phase == 2 && i < RA)
                                a[0][i] = fa.read(lds.a[to], i, 0);
#pragma unroll
                            for (int e = 0; e < kEach; ++e)
                                load(f, (s + kRing - 1) % kRing, (phase * (RA > RB ? RA : RB) + i) * kEach + e);
                            if (i < RA) {
#pragma unroll
                                for (int j = 0; j < RB; ++j)
                                    acc.v[i][j] = multiply(a[phase == 2 ? 1 : 0][i], b[phase == 1 ? 2 : now][j], acc.v[i][j]);
                            }
                            __builtin_amdgcn_sched_barrier(0);
                        }
                    if (s % kBuffers == 0)
                        f = next_turn();
                }
            }
            wait_loads<0>();
            return;
        }
        s16x8 a[2][RA], b[2][RB];
#pragma unroll
        for (int j = 0; j < RB; ++j)
            b[0][j] = fb.read(lds.b[0], j, 0);
#pragma unroll
        for (int i = 0; i < RA; ++i)
            a[0][i] = fa.read(lds.a[0], i, 0);

        const uint32_t fold = sh.fold * sh.turns;
        for (uint32_t t = t0; t < t1; t += kRing / kBuffers) {
            if (!kPlain && t == fold && t > t0)
                scale(acc);
#pragma unroll
            for (int s = 0; s < kRing; ++s) {
                if (s > 0 && s % kBuffers == 0 && t + s / kBuffers == t1)
                    break;
                // behind the barrier stage s + 1 is in LDS for everybody, and
                // nobody reads the buffer of s - 1 any more, which s + 3 (of a
                // ring of four) takes
                wait_loads<(kRing - 3) * kLoads>();
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const int from = kk == 0 ? s : (s + 1) % kRing;
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
                            load(f, (s + kRing - 1) % kRing, (kk * (RA > RB ? RA : RB) + i) * kEach + e);
                        if (i < RA) {
#pragma unroll
                            for (int j = 0; j < RB; ++j)
                                acc.v[i][j] = multiply(a[kk][i], b[kk][j], acc.v[i][j]);
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
                // the stages behind the last one of this turn are the next one's
                if (s % kBuffers == 0)
                    f = next_turn();
            }
        }
        if (!kPlain && t1 <= fold)
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
