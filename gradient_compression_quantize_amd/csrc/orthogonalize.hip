// orthogonalize.hip -- the nearest thing to an orthogonal matrix that a few
// products reach (Newton-Schulz), and the optimiser step around it.
//
//   X_0 = u / (|u|_F + eps),  X <- a X + P X,  P = b A + c A^2,  A = X X^T
// with A of the smaller side (of a tall matrix A = X^T X and X <- a X + X P).
// Every singular value s of X becomes a s + b s^3 + c s^5, the singular vectors
// stay.
//
// A step of the iteration is three products: A and A^2 are symmetric, so that
// only the tiles on and below the diagonal are computed and written twice; the
// third ends in the sum with a X, in the last step in the output itself (the
// scaled update, or the new weights). A tall matrix is never transposed: its
// products read it by k (mfma_product.h).
//
// Precision. X is carried to 22 bits, as two planes of fp16 that add up to it; A
// and P are held in one plane or two. The operands of the products are the first planes alone
// (off by at most 2^-11 of a value) where the result is kept in bf16, else both
// (three products each). a X never loses what the operands round away: its
// roundings would grow with the small singular values, 3.4 times a step, up to
// 500 times, while those of P X shrink with s^2. The diagonals of A and P, near 1
// and -3 where other entries are far below, are held apart in fp32 and enter by
// themselves,
//   (A^2)_ij = (O^2)_ij + (A_ii + A_jj) A_ij,  (A^2)_ii = (O^2)_ii + A_ii^2
//   (a X + P X)_i = (a + P_ii) X_i + (what is off the diagonal of P) X
// with O = A off its diagonal: rounded to 11 bits, they would scale whole rows. Of
// 64 x 576 the result of one plane is then 5e-4 off 64 bits instead of 2e-3.
// X is held times 2^14, A times 2^12, P times 2^10: entries are at most a singular
// value (s, s^2, ..) in size, and the first ones of X, of 4096 x 4096, near 2^-12.
// Second planes end at 2^-39 in X, at 2^-37 in A and 2^-35 in P, where they only
// are factors of something below 1 next to a X.
//
// Five steps of one plane take 1.46 to 1.62 ms for 4096 x 4096 (1.37 TFLOP, halves
// of symmetric products left out: 0.85 to 0.94 PFLOP/s) and 7.2 to 7.6 ms for 25088 x
// 4096 (0.88 to 0.93 PFLOP/s); of both 1.78 to 1.93 ms for the step of 48 x 768 x 768
// (three products: 0.68 to 0.73 PFLOP/s). Large symmetric products are 136 or 144
// tiles on 256 compute units (25088 x 4096: 470 to 485 us, 0.87 to 0.90 PFLOP/s), the
// updates next to them (1.0 PFLOP/s at 4096) bound by the power that holds the clock
// (mfma_product.h); one of 768 x 768, 123 us, by its 17 launches of 5 to 8 us; up to
// some 128 x 256 orthogonalize_resident.h goes without them. Both sides are held
// padded to 128: 48 of 16 x 16384, 50 MB of values, take 1.19 ms and 815 MB of
// workspace.
#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "mfma_product.h"

namespace gcq {
namespace {

constexpr int kXExp = 14, kAExp = 12, kPExp = 10;

constexpr float power_of_two(int e)
{
    return e == 0 ? 1.0f : e > 0 ? 2.0f * power_of_two(e - 1) : 0.5f * power_of_two(e + 1);
}

// 2^kExp: as a constant (a call with constant arguments stays a call).
template <int kExp>
constexpr float pow2 = power_of_two(kExp);

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// ---- the norm, and the first X -------------------------------------------------

constexpr int kThreads = 256;

// Up to this many partial sums of squares a matrix.
constexpr uint32_t kMaxParts = 1024;

// Eight values of a row of n, from column c on (zeros behind the last),
// whatever the alignment.
template <typename T>
__device__ __forceinline__ vec_of<float, 8> load8(const T* row, size_t c, size_t n)
{
    typedef T Vec __attribute__((ext_vector_type(8)));
    typedef Vec VecAny __attribute__((aligned(sizeof(T))));
    if (c + 8 <= n)
        return __builtin_convertvector(*reinterpret_cast<const VecAny*>(row + c), vec_of<float, 8>);
    vec_of<float, 8> v = {};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (c + k < n)
            v[k] = float(row[c + k]);
    return v;
}

__device__ __forceinline__ double workgroup_sum(double x)
{
    __shared__ double lds[kThreads / kWave];
#pragma unroll
    for (int off = kWave / 2; off > 0; off >>= 1)
        x += __shfl_xor(x, off);
    if ((threadIdx.x & (kWave - 1)) == 0)
        lds[threadIdx.x / kWave] = x;
    __syncthreads();
    x = lds[0];
    for (int w = 1; w < kThreads / kWave; ++w)
        x += lds[w];
    return x;
}

// The two passes below move memory only: the step of 4 x 2048 x 8192 takes 141 us for
// gradients and momenta to norms and new momenta, 150 us from both to X (5.7 and 5.4
// TB/s).

// What the update is made of: a matrix as it is, or the gradient and the
// momentum, which the first pass over them moves on.
struct Momentum {
    float grad_scale;
    float weight;   // the smaller one of beta and 1 - beta
    bool far;       // it is the gradient's
    bool nesterov;
};

// (1 - beta) g + beta m of g scaled, and of the momentum, old or new. It starts at
// the end with the larger weight, whose value enters unrounded: from the other one,
// m would be rounded at the size of m - g, which is that of g where gradients are
// noise (6 times the momenta at beta 0.95: 1.7e-7 off 64 bits instead of 2.7e-8).
__device__ __forceinline__ float mix(float g, float m, const Momentum& mo)
{
    const float from = mo.far ? m : g, to = mo.far ? g : m;
    return __builtin_fmaf(mo.weight, to - from, from);
}

// parts[matrix][workgroup] = sum of squares of its share of u, in 64 bits: no
// size of its values overflows or vanishes. Workgroups of one matrix take its
// values in turn, matrices are contiguous. Also zeros `zero`, what the products
// read of the workspace and do not write.
template <typename T, bool kMomentum>
__global__ __launch_bounds__(kThreads) void norm_kernel(PtrTable<T> x, PtrTable<float> momenta,
                                                        PtrTable<float> new_momenta, Momentum mo, size_t values,
                                                        double* __restrict__ parts, u32x4* __restrict__ zero,
                                                        size_t zeros)
{
    const size_t k = blockIdx.y;
    const T* src = x.p[k];
    double sum = 0.0;
    const size_t stride = size_t(gridDim.x) * kThreads * 8;
    for (size_t i = (size_t(blockIdx.x) * kThreads + threadIdx.x) * 8; i < values; i += stride) {
        vec_of<float, 8> v = load8(src, i, values);
        if (kMomentum) {
            const vec_of<float, 8> old = load8(momenta.p[k], i, values);
            vec_of<float, 8> now;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float g = v[e] * mo.grad_scale;
                now[e] = mix(g, old[e], mo);
                v[e] = mo.nesterov ? mix(g, now[e], mo) : now[e];
            }
            float* to = const_cast<float*>(new_momenta.p[k]) + i;
            typedef vec_of<float, 8> VecAny __attribute__((aligned(4)));
            if (i + 8 <= values) {
                *reinterpret_cast<VecAny*>(to) = now;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (i + e < values)
                        to[e] = now[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sum = __builtin_fma(double(v[e]), double(v[e]), sum);
    }
    sum = workgroup_sum(sum);
    if (threadIdx.x == 0)
        parts[k * gridDim.x + blockIdx.x] = sum;
    const size_t all = size_t(gridDim.x) * gridDim.y * kThreads;
    for (size_t i = (k * gridDim.x + blockIdx.x) * kThreads + threadIdx.x; i < zeros; i += all)
        zero[i] = u32x4{0, 0, 0, 0};
}

// Eight values as two planes: x = p0 + p1 to 2^-22 of it.
typedef vec_of<float, 8> f32x8;
typedef vec_of<f16_t, 4> f16x4;

struct Planes8 {
    f16x8 p0, p1;
};

__device__ __forceinline__ Planes8 split8(f32x8 v)
{
    Planes8 s;
    s.p0 = __builtin_convertvector(v, f16x8);
    s.p1 = __builtin_convertvector(v - __builtin_convertvector(s.p0, f32x8), f16x8);
    return s;
}

__device__ __forceinline__ f32x8 join8(Planes8 s)
{
    return __builtin_convertvector(s.p0, f32x8) + __builtin_convertvector(s.p1, f32x8);
}

__device__ __forceinline__ f16x8 load_plane(const uint16_t* p) { return *reinterpret_cast<const f16x8*>(p); }
__device__ __forceinline__ void store_plane(uint16_t* p, f16x8 v) { *reinterpret_cast<f16x8*>(p) = v; }

// A matrix of the workspace, of each of `count`: `rows` rows of ld values, which
// hold `cols` values of the first plane, then those of the second if there is one
// - or, where products read both, 16 of one and 16 of the other in turn.
struct Held {
    uint16_t* p;
    size_t matrix_stride;
    uint32_t ld, rows, cols;
};

__device__ __forceinline__ uint16_t* held_at(const Held& h, size_t matrix) { return h.p + matrix * h.matrix_stride; }

// Where the value of a plane in column c is in its row (those up to the next
// multiple of 16 follow it).
__device__ __forceinline__ size_t held_in_row(const Held& h, bool both, uint32_t c, int plane)
{
    return both ? size_t(c & ~15u) * 2 + plane * 16 + (c & 15) : size_t(plane) * h.cols + c;
}

// X_0 of each matrix, zeros behind its last row and column.
template <typename T, bool kMomentum>
__global__ __launch_bounds__(kThreads) void first_kernel(PtrTable<T> x, PtrTable<float> new_momenta, Momentum mo,
                                                         size_t m, size_t n, float eps,
                                                         const double* __restrict__ parts, uint32_t nparts, Held to,
                                                         bool both)
{
    const size_t k = blockIdx.y;
    double sum = 0.0;
    for (uint32_t i = threadIdx.x; i < nparts; i += kThreads)
        sum += parts[k * nparts + i];
    sum = workgroup_sum(sum);
    const double factor = double(pow2<kXExp>) / (sqrt(sum) + double(eps));
    const uint32_t chunks = to.cols / 8;
    const size_t total = size_t(to.rows) * chunks;
    for (size_t i = size_t(blockIdx.x) * kThreads + threadIdx.x; i < total; i += size_t(gridDim.x) * kThreads) {
        const size_t r = i / chunks, c = (i - r * chunks) * 8;
        vec_of<float, 8> v = {};
        if (r < m && c < n) {
            v = load8(x.p[k] + r * n, c, n);
            if (kMomentum) {
                const vec_of<float, 8> mom = load8(new_momenta.p[k] + r * n, c, n);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = mo.nesterov ? mix(v[e] * mo.grad_scale, mom[e], mo) : mom[e];
            }
            // (a factor that overflows fp32 belongs to values that do not)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e] = float(double(v[e]) * factor);
        }
        const Planes8 s = split8(v);
        uint16_t* o = held_at(to, k) + r * to.ld;
        store_plane(o + held_in_row(to, both, uint32_t(c), 0), s.p0);
        store_plane(o + held_in_row(to, both, uint32_t(c), 1), s.p1);
    }
}

// ---- products --------------------------------------------------------------------

// Tile `id` on or below the diagonal: ta <= tb.
__device__ __forceinline__ void triangle_of(uint32_t id, uint32_t& ta, uint32_t& tb)
{
    tb = uint32_t((sqrtf(8.0f * float(id) + 1.0f) - 1.0f) * 0.5f);
    // (the root may be off by one step)
    while (tb * (tb + 1) / 2 > id)
        --tb;
    while ((tb + 1) * (tb + 2) / 2 <= id)
        ++tb;
    ta = id - tb * (tb + 1) / 2;
}

struct Tiles {
    uint32_t per_matrix;
    uint32_t a, b;  // of a product that is not symmetric
    float* slab;    // of one over several ranges of k: what each leaves
};

template <int T>
struct Waves {
    static constexpr int a = 2, b = T == 256 ? 4 : 2, threads = a * b * kWave;
    // buffers of a tile: 1024 x 1024 takes 136 us, 161 with four
    static constexpr int ring = T == 64 ? 8 : 4;
};

// What a wave's products leave through: its part of the tile, 32 rows of b at a
// time, turned in the LDS that the product has left, so that a lane loads and
// stores 16 bytes of a row and a wave whole rows of its part. As the matrix cores
// leave them, 4 values of 32 rows each, the update of 4096 x 4096 took 221 us
// instead of 141.
template <int T>
struct Part {
    using W = Waves<T>;
    static constexpr int kCols = T / W::a, kRowsB = T / W::b;  // of a wave
    // (addresses of LDS throughout: as a generic one the choice of the buffer
    // would become a table, and LDS has no addresses to put there)
    typedef __attribute__((address_space(3))) uint16_t lds_u16;
    lds_u16* buffer;
    uint32_t a, b;  // where the wave's part starts
    int lane;

    __device__ __forceinline__ Part(const TileBuffers& lds, uint32_t a_first, uint32_t b_first)
    {
        static_assert(W::a * W::b <= 2 * kBuffers, "a buffer for each wave");
        static_assert(32 * kCols * 4 <= T * kStageK * 2, "32 rows of 4 bytes a value fit a buffer");
        lane = threadIdx.x & (kWave - 1);
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
        buffer = (lds_u16*)lds.a[0];
#pragma unroll
        for (int k = 1; k < W::a * W::b; ++k) {
            lds_u16* const p = (lds_u16*)(k < kBuffers ? lds.a[k % kBuffers] : lds.b[k % kBuffers]);
            buffer = wave == k ? p : buffer;
        }
        a = a_first + wave % W::a * kCols;
        b = b_first + wave / W::a * kRowsB;
    }
};

// The part as fp32, to be combined with what a lane loads beside it: 16-byte
// chunks that an XOR of the row spreads over the banks.
template <int T>
struct PartRows : Part<T> {
    using Part<T>::kCols, Part<T>::buffer, Part<T>::lane;
    static constexpr int kChunks = kCols / 4;
    static constexpr int kLanes = kCols / 8, kStep = kWave / kLanes, kPasses = 32 / kStep;
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
    using Part<T>::Part;

    __device__ __forceinline__ lds_f32x4* chunk(int row, int c) const
    {
        return (lds_f32x4*)(buffer + 2 * row * kCols + ((c ^ (row & (kChunks - 1))) << 3));
    }

    // Products [i][j] of all i into the image.
    template <typename Acc>
    __device__ __forceinline__ void fill(const Acc& acc, int j) const
    {
        const int row = int(acc_col(lane));
#pragma unroll
        for (int i = 0; i < kCols / 32; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = acc.v[i][j][4 * q + e];
                *chunk(row, i * 8 + 2 * q + (lane >> 5)) = v;
            }
        wave_lds_sync();
    }

    // Row and column (from the part's) of this lane's values in a pass.
    __device__ __forceinline__ int row(int pass) const { return pass * kStep + lane / kLanes; }
    __device__ __forceinline__ int col() const { return lane % kLanes * 8; }

    __device__ __forceinline__ f32x8 get(int pass) const
    {
        f32x8 v;
        v.lo = *chunk(row(pass), col() / 4);
        v.hi = *chunk(row(pass), col() / 4 + 1);
        return v;
    }
};

// The part as fp16, one plane or two one behind the other, made in the layout of
// the matrix cores: rows of it are then only copied, and those of its transpose
// come out of the transposing load (mfma_product.h).
template <int T>
struct PartPlanes : Part<T> {
    using Part<T>::kCols, Part<T>::buffer, Part<T>::lane;
    static constexpr int kChunks = kCols / 8, kPlane = 32 * kCols;  // chunks of 16 bytes a row
    static constexpr int kStep = kWave / kChunks, kPasses = 32 / kStep;
    typedef __attribute__((address_space(3))) f16x8 lds_f16x8;
    typedef __attribute__((address_space(3))) f16x4 lds_f16x4;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    using Part<T>::Part;

    __device__ __forceinline__ typename Part<T>::lds_u16* at(int plane, int row, int col) const
    {
        return buffer + plane * kPlane + row * kCols + (((col >> 3) ^ (row & (kChunks - 1))) << 3) + (col & 7);
    }

    // The 32 rows of a matrix from row b0 on into the image, as far as they exist.
    __device__ __forceinline__ void bring(const uint16_t* matrix, const Held& h, bool both, int planes, uint32_t b0) const
    {
        const uint32_t a = this->a + col();
        for (int plane = 0; plane < planes; ++plane) {
            const uint16_t* from = matrix + held_in_row(h, both, a, plane);
            f16x8 v[kPasses];
#pragma unroll
            for (int p = 0; p < kPasses; ++p) {
                v[p] = f16x8{};
                if (a < h.cols && b0 + row(p) < h.rows)
                    v[p] = load_plane(from + size_t(b0 + row(p)) * h.ld);
            }
#pragma unroll
            for (int p = 0; p < kPasses; ++p)
                *eight(plane, p) = v[p];
        }
        wave_lds_sync();
    }

    // The image into those rows.
    __device__ __forceinline__ void leave(uint16_t* matrix, const Held& h, bool both, int planes, uint32_t b0) const
    {
        const uint32_t a = this->a + col();
        for (int plane = 0; plane < planes; ++plane) {
            uint16_t* to = matrix + held_in_row(h, both, a, plane);
#pragma unroll
            for (int p = 0; p < kPasses; ++p) {
                const f16x8 v = *eight(plane, p);
                if (a < h.cols && b0 + row(p) < h.rows)
                    store_plane(to + size_t(b0 + row(p)) * h.ld, v);
            }
        }
    }

    // The four values that the matrix cores leave this lane in [i][.], q.
    __device__ __forceinline__ lds_f16x4* quad(int plane, int i, int q) const
    {
        return (lds_f16x4*)at(plane, int(acc_col(lane)), i * 32 + 8 * q + 4 * (lane >> 5));
    }

    // Those of all q: out of the image, and into it.
    __device__ __forceinline__ void read(f32x4 (&v)[4], int i, bool both) const
    {
        f16x4 p0[4], p1[4] = {};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            p0[q] = *quad(0, i, q);
            if (both)
                p1[q] = *quad(1, i, q);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            v[q] = __builtin_convertvector(p0[q], f32x4) + __builtin_convertvector(p1[q], f32x4);
    }

    __device__ __forceinline__ void write(const f32x4 (&v)[4], int i, bool both) const
    {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const f16x4 p0 = __builtin_convertvector(v[q], f16x4);
            *quad(0, i, q) = p0;
            if (both)
                *quad(1, i, q) = __builtin_convertvector(v[q] - __builtin_convertvector(p0, f32x4), f16x4);
        }
    }

    // Row and column of this lane's eight values in a pass over the rows.
    __device__ __forceinline__ int row(int pass) const { return pass * kStep + lane / kChunks; }
    __device__ __forceinline__ int col() const { return lane % kChunks * 8; }
    __device__ __forceinline__ lds_f16x8* eight(int plane, int pass) const
    {
        return (lds_f16x8*)at(plane, row(pass), col());
    }

    // Of the transpose: column turned_col(), rows turned_row() .. + 7.
    static constexpr int kTurnedPasses = kCols / 16;
    __device__ __forceinline__ int turned_col(int pass) const { return pass * 16 + (lane & 15); }
    __device__ __forceinline__ int turned_row() const { return lane / 16 * 8; }
    __device__ __forceinline__ f16x8 turned(int plane, int pass) const
    {
        const int r = turned_row() + (lane >> 2 & 3), c = pass * 16 + 4 * (lane & 3);
        union {
            s16x4 h[2];
            f16x8 v;
        } u;
        u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at(plane, r, c));
        u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at(plane, r + 4, c));
        return u.v;
    }
};

// A value for each column of a wave's part (0 behind the last), in LDS.
template <int T>
struct Columns {
    static constexpr int kCols = T / Waves<T>::a, kAll = Waves<T>::a * Waves<T>::b * kCols;
    typedef __attribute__((address_space(3))) float lds_f32;
    typedef __attribute__((address_space(3))) const f32x4 lds_f32x4;
    lds_f32* own;
    int lane;

    __device__ __forceinline__ Columns(float (&lds)[kAll], const float* p, uint32_t a, uint32_t cols)
    {
        lane = threadIdx.x & (kWave - 1);
        own = (lds_f32*)lds + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * kCols;
        for (int c = lane; c < kCols; c += kWave)
            own[c] = a + c < cols ? p[a + c] : 0.0f;
        wave_lds_sync();
    }

    // At the columns of the products that the matrix cores leave this lane.
    __device__ __forceinline__ f32x4 quad(int i, int q) const
    {
        return *(lds_f32x4*)(own + i * 32 + 8 * q + 4 * (lane >> 5));
    }
};

// A symmetric product S = V V^T of the rows (by k: columns) of V, and what is
// made of it: A = S (kSquare = false), or P = b A + c A^2 of V, A off its
// diagonal. Diagonals go to (and come from) arrays of their own, [matrix][side].
struct SymmetricOut {
    Held to;
    bool both;  // planes
    float b, c;
    const float* from_diagonal;  // of A, if kSquare
    float* diagonal;
};

template <bool kKRows, bool kSquare, int T, bool kBoth>
__global__ __launch_bounds__(Waves<T>::threads, 2) void symmetric_kernel(MatOperand V, size_t matrix_stride,
                                                                         ProductShape sh, Tiles tiles, SymmetricOut out)
{
    constexpr int WA = Waves<T>::a, WB = Waves<T>::b;
    using P = TileProduct<true, kKRows, kKRows, T, T, WA, WB, true, kBoth, Waves<T>::ring>;
    GCQ_TILE_RING(lds, T, Waves<T>::ring);
    const uint32_t id = xcd_contiguous(blockIdx.x, gridDim.x), range = id / tiles.per_matrix;
    const uint32_t matrix = range / sh.splits, split = range - matrix * sh.splits;
    uint32_t ta, tb;
    triangle_of(id - range * tiles.per_matrix, ta, tb);
    V.plane0 += matrix * matrix_stride;
    const uint32_t turns = sh.turns * sh.segments;
    typename P::Acc acc;
    P::run(V, V, sh, ta * T, tb * T, uint32_t(uint64_t(turns) * split / sh.splits),
           uint32_t(uint64_t(turns) * (split + 1) / sh.splits), lds, acc);

    if (!kSquare && sh.splits > 1) {  // the sums as the lanes hold them, for join_kernel
        const int lane = threadIdx.x & (kWave - 1);
        f32x4* to = reinterpret_cast<f32x4*>(tiles.slab) + (size_t(id) * (WA * WB) + threadIdx.x / kWave) * (P::RA * P::RB * 256);
#pragma unroll
        for (int i = 0; i < P::RA; ++i)
#pragma unroll
            for (int j = 0; j < P::RB; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    f32x4 v;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = acc.v[i][j][4 * q + e];
                    to[((i * P::RB + j) * 4 + q) * kWave + lane] = v;
                }
        return;
    }
    using Rows = PartPlanes<T>;
    const Rows part(lds, ta * T, tb * T);
    uint16_t* to = held_at(out.to, matrix);
    const uint32_t side = out.to.rows;
    float* diagonal = out.diagonal + size_t(matrix) * side;
    const float* old = kSquare ? out.from_diagonal + size_t(matrix) * side : nullptr;
    constexpr int planes = kBoth ? 2 : 1;
    __shared__ float of_columns[Columns<T>::kAll];
    const Columns<T> of_col(of_columns, old, part.a, kSquare ? side : 0);  // A's diagonal
#pragma unroll
    for (int j = 0; j < P::RB; ++j) {
        const uint32_t b0 = part.b + j * 32, b = b0 + acc_col(part.lane);
        if (kSquare)  // A's part of V, which lies as P does
            part.bring(V.plane0, out.to, kBoth, planes, b0);
        const float db = kSquare && b < side ? old[b] : 0.0f;
#pragma unroll
        for (int i = 0; i < P::RA; ++i) {
            f32x4 v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[q][e] = acc.v[i][j][4 * q + e] * (kSquare ? out.c * pow2<kPExp - 2 * kAExp> : pow2<kAExp - 2 * kXExp>);
            if (kSquare) {
                const float own = (out.b + out.c * db) * pow2<kPExp - kAExp>, each = out.c * pow2<kPExp - kAExp>;
                f32x4 A[4];
                part.read(A, i, kBoth);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x4 da = of_col.quad(i, q);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[q][e] = __builtin_fmaf(A[q][e], __builtin_fmaf(each, da[e], own), v[q][e]);
                }
            }
            if (ta == tb) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (part.a + i * 32 + acc_row(4 * q + e, part.lane) == b && b < side) {
                            // (A is 0 there in the planes)
                            const float more = kSquare ? (out.b + out.c * db) * db : 0.0f;
                            diagonal[b] = __builtin_fmaf(v[q][e], pow2<kSquare ? -kPExp : -kAExp>, more);
                            v[q][e] = 0.0f;
                        }
            }
            part.write(v, i, kBoth);
        }
        wave_lds_sync();
        part.leave(to, out.to, kBoth, planes, b0);
        if (ta != tb) {
            for (int plane = 0; plane < planes; ++plane) {
                uint16_t* p = to + held_in_row(out.to, kBoth, b0 + part.turned_row(), plane);
#pragma unroll
                for (int k = 0; k < Rows::kTurnedPasses; ++k) {
                    const uint32_t row = part.a + part.turned_col(k);
                    const f16x8 v = part.turned(plane, k);
                    if (row < side && b0 + part.turned_row() < side)
                        store_plane(p + size_t(row) * out.to.ld, v);
                }
            }
        }
        wave_lds_sync();
    }
}

// A of what the ranges of k have left: one workgroup for each 32 x 32 block of each
// tile adds its 4 KB of every range, in their order.
template <int T>
__global__ __launch_bounds__(kThreads) void join_kernel(const f32x4* __restrict__ slab, uint32_t splits, Tiles tiles,
                                                        SymmetricOut out)
{
    constexpr int WA = Waves<T>::a, WB = Waves<T>::b, RA = T / WA / 32, RB = T / WB / 32, kBlocks = WA * WB * RA * RB;
    __shared__ float turned[32][33];
    const uint32_t tile_id = blockIdx.x / kBlocks, block = blockIdx.x - tile_id * kBlocks;
    const uint32_t matrix = tile_id / tiles.per_matrix, tile = tile_id - matrix * tiles.per_matrix;
    uint32_t ta, tb;
    triangle_of(tile, ta, tb);
    const f32x4* from = slab + (size_t(matrix) * splits * tiles.per_matrix + tile) * (kBlocks * 256) + block * 256 + threadIdx.x;
    const size_t stride = size_t(tiles.per_matrix) * (kBlocks * 256);
    f32x4 v = {};
#pragma unroll 8
    for (uint32_t s = 0; s < splits; ++s)
        v += from[s * stride];
    v *= pow2<kAExp - 2 * kXExp>;

    const uint32_t wave = block / (RA * RB), in = block % (RA * RB), lane = threadIdx.x & (kWave - 1);
    const uint32_t a0 = ta * T + wave % WA * (T / WA) + in / RB * 32, b0 = tb * T + wave / WA * (T / WB) + in % RB * 32;
    const uint32_t side = out.to.rows;
    if (a0 >= side || b0 >= side)
        return;
    const uint32_t a = acc_row(threadIdx.x / kWave * 4, lane), b = acc_col(lane);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (a0 + a + e == b0 + b) {
            out.diagonal[size_t(matrix) * side + b0 + b] = v[e] * pow2<-kAExp>;
            v[e] = 0.0f;
        }
    const auto store = [&](uint32_t row, uint32_t col, f32x4 x) {
        uint16_t* p = held_at(out.to, matrix) + size_t(row) * out.to.ld;
        const f16x4 p0 = __builtin_convertvector(x, f16x4);
        *reinterpret_cast<f16x4*>(p + held_in_row(out.to, out.both, col, 0)) = p0;
        if (out.both)
            *reinterpret_cast<f16x4*>(p + held_in_row(out.to, true, col, 1)) =
                __builtin_convertvector(x - __builtin_convertvector(p0, f32x4), f16x4);
    };
    store(b0 + b, a0 + a, v);
    if (ta == tb)
        return;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        turned[a + e][b] = v[e];
    __syncthreads();
    const uint32_t row = threadIdx.x / 8, col = threadIdx.x % 8 * 4;
    store(a0 + row, b0 + col, f32x4{turned[row][col], turned[row][col + 1], turned[row][col + 2], turned[row][col + 3]});
}

// P = b A of a step without a second power; `rows` of all matrices.
__global__ __launch_bounds__(kThreads) void scale_kernel(Held A, Held P, bool both, float b, size_t rows,
                                                         const float* __restrict__ from_diagonal,
                                                         float* __restrict__ diagonal)
{
    const float f = b * pow2<kPExp - kAExp>;
    const size_t chunks = A.cols / 8, all = rows * chunks;
    for (size_t i = size_t(blockIdx.x) * kThreads + threadIdx.x; i < all; i += size_t(gridDim.x) * kThreads) {
        const size_t row = i / chunks, c = i - row * chunks;
        if (c == 0)
            diagonal[row] = b * from_diagonal[row];
        const size_t at0 = row * A.ld + held_in_row(A, both, uint32_t(c) * 8, 0);
        const size_t at1 = row * A.ld + held_in_row(A, both, uint32_t(c) * 8, 1);
        Planes8 s = {};
        s.p0 = load_plane(A.p + at0);
        if (both)
            s.p1 = load_plane(A.p + at1);
        s = split8(join8(s) * f);
        store_plane(P.p + at0, s.p0);
        if (both)
            store_plane(P.p + at1, s.p1);
    }
}

// What the last step writes: out = scale X, or new weights = (1 - lr decay)
// weights - lr scale X.
struct LastOut {
    PtrTable<void> weights, out;
    int dtype;
    bool update;
    uint32_t m, n;
    float scale, lr, decay;
    const float* lr_scale;
};

template <typename T>
__device__ __forceinline__ void write_last(const LastOut& o, uint32_t matrix, size_t r, uint32_t c, f32x8 x,
                                           float keep, float factor)
{
    const size_t at = r * o.n + c;
    T* to = static_cast<T*>(const_cast<void*>(o.out.p[matrix])) + at;
    const T* w = o.update ? static_cast<const T*>(o.weights.p[matrix]) + at : nullptr;
    typedef T Vec __attribute__((ext_vector_type(8)));
    typedef Vec VecAny __attribute__((aligned(sizeof(T))));
    x *= factor;
    if (c + 8 <= o.n) {
        if (w) {
            const f32x8 old = __builtin_convertvector(*reinterpret_cast<const VecAny*>(w), f32x8);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = __builtin_fmaf(old[e], keep, -x[e]);
        }
        *reinterpret_cast<VecAny*>(to) = __builtin_convertvector(x, Vec);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (c + e < o.n)
            to[e] = T(w ? __builtin_fmaf(float(w[e]), keep, -x[e]) : x[e]);
}

}  // namespace
}  // namespace gcq

#include "orthogonalize_resident.h"

namespace gcq {
namespace {

// out[b][a] = X[b][a] * a_coef + sum over k of A(a, k) B(b, k): of a wide X, A
// is X by k and B is P; of a tall one, A is P and B is X. kLast: the last step.
struct UpdateOut {
    Held from, to;
    float a;
    const float* diagonal;  // of P, [matrix][side]
    uint32_t side;
};

template <bool kTall, bool kLast, int T, bool kBoth>
__global__ __launch_bounds__(Waves<T>::threads, 2) void update_kernel(MatOperand A, size_t a_stride, MatOperand B,
                                                                      size_t b_stride, ProductShape sh, Tiles tiles,
                                                                      UpdateOut out, LastOut last)
{
    constexpr int WA = Waves<T>::a, WB = Waves<T>::b;
    using P = TileProduct<true, !kTall, false, T, T, WA, WB, true, kBoth, Waves<T>::ring>;
    GCQ_TILE_RING(lds, T, Waves<T>::ring);
    const uint32_t id = xcd_contiguous(blockIdx.x, gridDim.x), matrix = id / tiles.per_matrix;
    uint32_t ta, tb;
    tile_of(id - matrix * tiles.per_matrix, tiles.a, tiles.b, ta, tb);
    A.plane0 += matrix * a_stride;
    B.plane0 += matrix * b_stride;
    typename P::Acc acc;
    P::run(A, B, sh, ta * T, tb * T, 0, sh.turns * sh.segments, lds, acc);

    const PartPlanes<T> part(lds, ta * T, tb * T);
    const uint16_t* from = held_at(out.from, matrix);
    const float* diagonal = out.diagonal + size_t(matrix) * out.side;
    const uint32_t rows = out.from.rows, cols = out.from.cols;
    __shared__ float of_columns[Columns<T>::kAll];
    const Columns<T> of_col(of_columns, diagonal, part.a, kTall ? cols : 0);
    const PartRows<T> whole(lds, ta * T, tb * T);
    float keep = 1.0f, factor = last.scale * pow2<-kXExp>;
    if (kLast && last.update) {
        const float lr = last.lr_scale ? last.lr * *last.lr_scale : last.lr;
        keep = __builtin_fmaf(-lr, last.decay, 1.0f);
        factor = lr * last.scale * pow2<-kXExp>;
    }
#pragma unroll
    for (int j = 0; j < P::RB; ++j) {
        const uint32_t b0 = part.b + j * 32, b = b0 + acc_col(part.lane);
        part.bring(from, out.from, kBoth, 2, b0);
        const float of_row = out.a + (!kTall && b < rows ? diagonal[b] : 0.0f);
#pragma unroll
        for (int i = 0; i < P::RA; ++i) {
            f32x4 v[4];
            part.read(v, i, true);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const f32x4 of_cols = kTall ? of_col.quad(i, q) : f32x4{};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float self = kTall ? of_cols[e] + out.a : of_row;
                    v[q][e] = __builtin_fmaf(v[q][e], self, acc.v[i][j][4 * q + e] * pow2<-kPExp>);
                    if (kLast)
                        acc.v[i][j][4 * q + e] = v[q][e];
                }
            }
            if (!kLast)
                part.write(v, i, true);
        }
        wave_lds_sync();
        if (!kLast) {
            part.leave(held_at(out.to, matrix), out.to, kBoth, 2, b0);
            wave_lds_sync();
            continue;
        }
        whole.fill(acc, j);
        const uint32_t a = whole.a + whole.col();
#pragma unroll
        for (int p = 0; p < PartRows<T>::kPasses; ++p) {
            const uint32_t row = b0 + whole.row(p);
            const f32x8 v = whole.get(p);
            if (a >= last.n || row >= last.m)
                continue;
            if (last.dtype == GC_F32)
                write_last<float>(last, matrix, row, a, v, keep, factor);
            else if (last.dtype == GC_BF16)
                write_last<bf16_t>(last, matrix, row, a, v, keep, factor);
            else
                write_last<f16_t>(last, matrix, row, a, v, keep, factor);
        }
        wave_lds_sync();
    }
}

// ---- host side -----------------------------------------------------------------

size_t round_up(size_t a, size_t b) { return ceil_div(a, b) * b; }

constexpr size_t kMaxSide = size_t(1) << 20, kMaxSmallSide = size_t(1) << 15, kMaxTiles = size_t(1) << 22;
void place(Held& h, char* ws) { h.p = reinterpret_cast<uint16_t*>(ws + reinterpret_cast<size_t>(h.p)); }

MatOperand operand(const Held& h)
{
    MatOperand o{};
    o.plane0 = h.p;
    o.ld = h.ld;
    return o;
}

size_t triangle_tiles(size_t side, size_t t) { return ceil_div(side, t) * (ceil_div(side, t) + 1) / 2; }
size_t all_tiles(size_t a, size_t b, size_t t) { return ceil_div(a, t) * ceil_div(b, t); }

// How a product goes: its tiles, and over how many ranges of k.
struct Plan {
    int tile;
    uint32_t splits;
};

// Microseconds of `tiles` tiles of T over `turns` turns of 128 k, from what a turn
// was measured to take (random values, 4096 and 16384 k): alone on a compute unit
// with half of the chip's at work 2.8 (T = 256), 1.05 (128), 0.52 (64), with all of
// them 3.9, 1.3 and 0.55; two to a compute unit 2.8 (128) and 1.15 (64). Tiles of
// 256 then come in rounds, the others fill in as places become free.
double tiles_cost(int T, double tiles, double turns)
{
    const double cus = 256.0, places = T == 256 ? cus : 2.0 * cus;
    const double few = T == 256 ? 2.8 : T == 128 ? 1.05 : 0.52, one = T == 256 ? 3.9 : T == 128 ? 1.3 : 0.55;
    const double full = T == 256 ? 3.9 : T == 128 ? 2.8 : 1.15, end = T == 256 ? 8.0 : T == 128 ? 4.0 : 3.0;
    double turn, rounds = 1.0;
    if (tiles <= cus / 2)
        turn = few;
    else if (tiles <= cus)
        turn = few + (one - few) * (tiles / (cus / 2) - 1.0);
    else if (tiles <= places)
        turn = one + (full - one) * (tiles - cus) / (places - cus);
    else {
        turn = full;
        rounds = T == 256 ? std::ceil(tiles / places) : tiles / places + 0.25;
    }
    return rounds * (turns * turn + end);
}

// Of the tiles of 256, 128 and 64, and of 1, 2, 4 .. ranges of at least four turns
// each, what costs least. A turn of both planes is as long as 2.6 of one with
// tiles of 256, 2.3 with smaller ones. Several ranges leave their sums in memory
// (written and read at some 4 TB/s) for another launch (5 us): all five steps of 64
// x 16384 take 99 us with 32 ranges, 327 with one, of 256 x 2304 106 and 127. With
// tiles of one size alone: 4096 x 4096 1.59 ms with 256, 1.94 with 128, 2.82 with
// 64; 768 x 768 369, 191 and 121 us; 48 of them 1054, 975 and 1287.
template <typename Tiles>
Plan plan_of(size_t count, size_t k, bool both, bool may_split, Tiles tiles)
{
    Plan best{};
    double least = 0.0;
    const size_t turns = k / kTurnK * (both ? 2 : 1);
    for (int T = 256; T >= 64; T /= 2) {
        const double n = double(count * tiles(T)), turn = both ? (T == 256 ? 1.3 : 1.15) : 1.0;
        for (uint32_t s = 1; s == 1 || (may_split && s * 4 <= turns && n * s <= 1024.0); s *= 2) {
            const double t = tiles_cost(T, n * s, double(ceil_div(turns, s)) * turn) +
                             (s > 1 ? 5.0 + n * s * T * T * 8.0 / 4e6 : 0.0);
            if (best.tile == 0 || t < least) {
                best = Plan{T, s};
                least = t;
            }
        }
    }
    return best;
}

// Calls f with the tile, and whether products are of both planes, as integral
// constants.
template <typename F>
void with_tile(int tile, bool both, F f)
{
    const auto with = [&](auto t) {
        if (both)
            f(t, std::true_type());
        else
            f(t, std::false_type());
    };
    if (tile == 256)
        with(std::integral_constant<int, 256>());
    else if (tile == 128)
        with(std::integral_constant<int, 128>());
    else
        with(std::integral_constant<int, 64>());
}

ProductShape shape_of(size_t k, bool both)
{
    ProductShape sh{};
    sh.turns = uint32_t(k / (both ? kTurnK / 2 : kTurnK));
    sh.segments = 1;
    sh.splits = 1;
    return sh;
}

struct Layout {
    size_t m, n, small;     // small: the side of A
    bool tall, both;        // both: products of both planes
    bool resident;          // one workgroup a matrix, without a workspace
    Plan gram, square, update;
    size_t slab;            // of gram's ranges
    Held x[2], A, P;        // their p: an offset into the workspace
    size_t parts, diagonals[2], zero, zeros, total;  // bytes; diagonals of A and P
    uint32_t nparts;
};

Layout layout_of(size_t count, size_t m, size_t n, bool both)
{
    Layout L{};
    L.m = m;
    L.n = n;
    L.tall = m > n;
    L.both = both;
    L.small = std::min(m, n);
    L.resident = with_resident(L.small, std::max(m, n), both, [](auto, auto, auto) {});
    if (L.resident)
        return L;
    const size_t rows = round_up(m, kTurnK), cols = round_up(n, kTurnK), side = round_up(L.small, kTurnK);
    size_t used = 0;
    const auto take = [&](size_t bytes) {
        const size_t at = used;
        used += (bytes + 255) & ~size_t(255);
        return at;
    };
    const auto hold = [&](size_t r, size_t cols, int planes) {
        Held h{};
        h.matrix_stride = r * cols * planes;
        h.ld = uint32_t(cols * planes);
        h.cols = uint32_t(cols);
        h.rows = uint32_t(r);
        h.p = reinterpret_cast<uint16_t*>(take(count * h.matrix_stride * 2));
        return h;
    };
    L.nparts = uint32_t(std::min<size_t>(kMaxParts, ceil_div(m * n, kThreads * 8 * 4)));
    L.parts = take(count * L.nparts * sizeof(double));
    L.x[0] = hold(rows, cols, 2);
    L.zero = used;
    L.x[1] = hold(rows, cols, 2);
    L.A = hold(side, side, both ? 2 : 1);
    L.P = hold(side, side, both ? 2 : 1);
    L.diagonals[0] = take(count * side * sizeof(float));
    L.diagonals[1] = take(count * side * sizeof(float));
    L.zeros = used - L.zero;
    L.gram = plan_of(count, L.tall ? rows : cols, both, true, [&](int T) { return triangle_tiles(L.small, T); });
    L.square = plan_of(count, side, both, false, [&](int T) { return triangle_tiles(L.small, T); });
    L.update = plan_of(count, side, both, false, [&](int T) { return all_tiles(m, n, T); });
    const size_t T = L.gram.tile;
    L.slab = take(L.gram.splits > 1 ? count * L.gram.splits * triangle_tiles(L.small, T) * T * T * 4 : 0);
    // Tiles of 64 leave padding unwritten (128 is what it goes by), which then
    // has to be zero from the start.
    const auto half = [](size_t v) { return round_up(v, 64) % kTurnK != 0; };
    const bool leaves = ((L.gram.tile == 64 || L.square.tile == 64) && half(L.small)) ||
                        (L.update.tile == 64 && (half(m) || half(n)));
    L.zeros = leaves ? L.zeros : 0;
    L.total = used;
    return L;
}


template <bool kKRows, bool kSquare>
void launch_symmetric(const Held& v, const Plan& plan, size_t side, size_t k, size_t count, const SymmetricOut& out,
                      float* slab, hipStream_t stream)
{
    MatOperand o = operand(v);
    o.extent = kKRows ? v.cols : v.rows;
    o.krows = v.rows;
    ProductShape sh = shape_of(k, out.both);
    sh.splits = plan.splits;
    with_tile(plan.tile, out.both, [&](auto t, auto both) {
        constexpr int T = decltype(t)::value;
        Tiles tiles{};
        tiles.per_matrix = uint32_t(triangle_tiles(side, T));
        tiles.slab = slab;
        const size_t all = tiles.per_matrix * count;
        hipLaunchKernelGGL((symmetric_kernel<kKRows, kSquare, T, decltype(both)::value>), dim3(unsigned(all * plan.splits)),
                           dim3(Waves<T>::threads), 0, stream, o, v.matrix_stride, sh, tiles, out);
        if (plan.splits > 1)
            hipLaunchKernelGGL(join_kernel<T>, dim3(unsigned(all * (T / 32) * (T / 32))), dim3(kThreads), 0, stream,
                               reinterpret_cast<const f32x4*>(slab), plan.splits, tiles, out);
    });
}

template <bool kTall, bool kLast>
void launch_update(const Layout& L, size_t count, const UpdateOut& out, const LastOut& last, hipStream_t stream)
{
    MatOperand X = operand(out.from), P = operand(L.P);
    X.extent = kTall ? out.from.rows : out.from.cols;
    X.krows = out.from.rows;
    P.extent = L.P.rows;
    const ProductShape sh = shape_of(L.P.cols, L.both);
    with_tile(L.update.tile, L.both, [&](auto t, auto both) {
        constexpr int T = decltype(t)::value;
        constexpr bool kBoth = decltype(both)::value;
        Tiles tiles{};
        tiles.a = uint32_t(ceil_div(L.n, T));
        tiles.b = uint32_t(ceil_div(L.m, T));
        tiles.per_matrix = tiles.a * tiles.b;
        const dim3 grid(unsigned(tiles.per_matrix * count));
        if (kTall)
            hipLaunchKernelGGL((update_kernel<kTall, kLast, T, kBoth>), grid, dim3(Waves<T>::threads), 0, stream, P,
                               L.P.matrix_stride, X, out.from.matrix_stride, sh, tiles, out, last);
        else
            hipLaunchKernelGGL((update_kernel<kTall, kLast, T, kBoth>), grid, dim3(Waves<T>::threads), 0, stream, X,
                               out.from.matrix_stride, P, L.P.matrix_stride, sh, tiles, out, last);
    });
}

// The iteration, from X_0 in L.x[0] on.
template <bool kTall>
void iterate(const Layout& L, size_t count, const float* coefficients, int steps, const LastOut& last, char* ws,
             hipStream_t stream)
{
    float* of_a = reinterpret_cast<float*>(ws + L.diagonals[0]);
    float* of_p = reinterpret_cast<float*>(ws + L.diagonals[1]);
    for (int s = 0; s < steps; ++s) {
        const float a = coefficients[3 * s], b = coefficients[3 * s + 1], c = coefficients[3 * s + 2];
        const Held &from = L.x[s & 1], &to = L.x[(s + 1) & 1];
        launch_symmetric<kTall, false>(from, L.gram, L.small, kTall ? from.rows : from.cols, count,
                                       SymmetricOut{L.A, L.both, 0.0f, 0.0f, nullptr, of_a},
                                       reinterpret_cast<float*>(ws + L.slab), stream);
        if (c != 0.0f) {
            launch_symmetric<false, true>(L.A, L.square, L.small, L.A.cols, count,
                                          SymmetricOut{L.P, L.both, b, c, of_a, of_p}, nullptr, stream);
        } else {
            const size_t rows = count * L.A.rows;
            hipLaunchKernelGGL(scale_kernel, dim3(unsigned(std::min<size_t>(ceil_div(rows * L.A.cols / 8, kThreads), 2048))),
                               dim3(kThreads), 0, stream, L.A, L.P, L.both, b, rows, of_a, of_p);
        }
        if (s + 1 < steps)
            launch_update<kTall, false>(L, count, UpdateOut{from, to, a, of_p, L.P.rows}, last, stream);
        else
            launch_update<kTall, true>(L, count, UpdateOut{from, to, a, of_p, L.P.rows}, last, stream);
    }
}

struct Call {
    const char* what;
    size_t count, m, n;
    int out_dtype;      // of the accuracy asked for
    const float* coefficients;
    int steps;
    float eps;
    void* ws;
    size_t* ws_bytes;
};

int refuse(const Call& c, const char* why, gc_status code = GC_EINVAL) { return fail(code, std::string(c.what) + ": " + why); }

// What both entry points check; 1: a query of the workspace, answered.
int check_call(const Call& c, Layout& L)
{
    if (!dtype_bytes(c.out_dtype))
        return refuse(c, "unknown dtype");
    if (c.count < 1 || c.count > GC_MAX_WORKERS)
        return refuse(c, "the number of matrices must lie in 1 .. 64");
    if (c.m > kMaxSide || c.n > kMaxSide || std::min(c.m, c.n) > kMaxSmallSide ||
        c.count * all_tiles(c.m, c.n, 256) > kMaxTiles)
        return refuse(c, "sides beyond 2^20 (the smaller one 2^15), or more than 2^22 tiles of 256 x 256",
                      GC_EUNSUPPORTED);
    if (!c.ws_bytes)
        return refuse(c, "ws_bytes is NULL");
    L = layout_of(c.count, c.m, c.n, c.out_dtype != GC_BF16);
    if (!c.ws) {
        *c.ws_bytes = std::max<size_t>(L.total, 256);
        return 1;
    }
    if (c.steps < 1 || c.steps > kMaxSteps || !c.coefficients)
        return refuse(c, "1 to 64 steps of three coefficients each");
    for (int k = 0; k < 3 * c.steps; ++k)
        if (!std::isfinite(c.coefficients[k]))
            return refuse(c, "a coefficient is not finite");
    if (!(c.eps >= 0.0f) || !std::isfinite(c.eps))
        return refuse(c, "eps must not be negative");
    if (!aligned16(c.ws) || *c.ws_bytes < L.total)
        return refuse(c, "workspace too small or not 16-byte aligned");
    if (L.resident)
        return GC_OK;
    place(L.x[0], static_cast<char*>(c.ws));
    place(L.x[1], static_cast<char*>(c.ws));
    place(L.A, static_cast<char*>(c.ws));
    place(L.P, static_cast<char*>(c.ws));
    return GC_OK;
}

// Copies `count` pointers, each to values of `bytes` bytes.
template <typename T>
bool take_pointers(PtrTable<T>& t, const void* const* p, size_t count, size_t bytes)
{
    for (size_t k = 0; k < count; ++k) {
        if (!p || !p[k] || !aligned_to(p[k], bytes))
            return false;
        t.p[k] = static_cast<const T*>(p[k]);
    }
    return true;
}

// The buffers of a call in memory, to find outputs that lie in others: whether
// those are read first goes by the size of the matrices.
class Buffers {
public:
    void reads(const void* p, size_t bytes) { add(p, bytes, false); }
    // An output; `own`: the input that may be in its place.
    void writes(const void* p, size_t bytes, const void* own, size_t own_bytes)
    {
        const bool in_place = p == own;
        add(p, in_place ? std::max(bytes, own_bytes) : bytes, true);
        if (own && !in_place)
            add(own, own_bytes, false);
    }

    bool overlap()
    {
        std::sort(all_, all_ + count_, [](const One& a, const One& b) { return a.first < b.first; });
        uintptr_t end = 0, end_of_outputs = 0;
        for (size_t k = 0; k < count_; ++k) {
            const One& o = all_[k];
            if (o.first < (o.output ? end : end_of_outputs))
                return true;
            end = std::max(end, o.last);
            end_of_outputs = o.output ? std::max(end_of_outputs, o.last) : end_of_outputs;
        }
        return false;
    }

private:
    struct One {
        uintptr_t first, last;
        bool output;
    };
    void add(const void* p, size_t bytes, bool output)
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        all_[count_++] = One{at, at + bytes, output};
    }
    One all_[5 * GC_MAX_WORKERS];
    size_t count_ = 0;
};

// What a call reads: matrices of `dtype`, or gradients and momenta.
struct In {
    PtrTable<void> x;
    int dtype;
    bool momentum;
    PtrTable<float> momenta, new_momenta;
    Momentum mo;
};

int run_resident(const Call& c, const Layout& L, const In& in, const LastOut& last, hipStream_t stream)
{
    ResidentIn r{};
    r.x = in.x;
    r.momenta = in.momenta;
    r.new_momenta = in.new_momenta;
    r.mo = in.mo;
    r.dtype = in.dtype;
    r.momentum = in.momentum;
    r.m = uint32_t(L.m);
    r.n = uint32_t(L.n);
    r.eps = c.eps;
    Coefficients coef{};
    for (int k = 0; k < 3 * c.steps; ++k)
        coef.v[k / 3][k % 3] = c.coefficients[k];
    with_resident(L.small, std::max(L.m, L.n), L.both, [&](auto RB, auto NB, auto planes) {
        const auto launch = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3(unsigned(c.count)), dim3(kResidentWaves * kWave), 0, stream, r, coef,
                               c.steps, last);
        };
        constexpr int kRB = decltype(RB)::value, kNB = decltype(NB)::value, kPlanes = decltype(planes)::value;
        if (L.tall)
            launch(resident_kernel<kRB, kNB, kPlanes, true>);
        else
            launch(resident_kernel<kRB, kNB, kPlanes, false>);
    });
    return check_launch(c.what);
}

template <typename T, bool kMomentum>
void launch_first(const Call& c, const Layout& L, const In& in, hipStream_t stream)
{
    char* ws = static_cast<char*>(c.ws);
    double* parts = reinterpret_cast<double*>(ws + L.parts);
    PtrTable<T> x{};
    for (size_t k = 0; k < c.count; ++k)
        x.p[k] = static_cast<const T*>(in.x.p[k]);
    hipLaunchKernelGGL((norm_kernel<T, kMomentum>), dim3(L.nparts, unsigned(c.count)), dim3(kThreads), 0, stream, x,
                       in.momenta, in.new_momenta, in.mo, c.m * c.n, parts, reinterpret_cast<u32x4*>(ws + L.zero),
                       L.zeros / 16);
    const size_t chunks = L.x[0].matrix_stride / 8;
    hipLaunchKernelGGL((first_kernel<T, kMomentum>),
                       dim3(unsigned(std::min<size_t>(ceil_div(chunks, kThreads * 4), kMaxParts)), unsigned(c.count)),
                       dim3(kThreads), 0, stream, x, in.new_momenta, in.mo, c.m, c.n, c.eps, parts, L.nparts, L.x[0], L.both);
}

int run_call(const Call& c, const Layout& L, const In& in, const LastOut& last, hipStream_t stream)
{
    if (L.resident)
        return run_resident(c, L, in, last, stream);
    if (in.momentum)
        launch_first<float, true>(c, L, in, stream);
    else
        with_dtype(in.dtype, [&](auto e) {
            launch_first<decltype(e), false>(c, L, in, stream);
            return 0;
        });
    char* ws = static_cast<char*>(c.ws);
    if (L.tall)
        iterate<true>(L, c.count, c.coefficients, c.steps, last, ws, stream);
    else
        iterate<false>(L, c.count, c.coefficients, c.steps, last, ws, stream);
    return check_launch(c.what);
}

}  // namespace
}  // namespace gcq

using namespace gcq;

GCQ_API int orthogonalize(const void* const* x, int count, size_t m, size_t n, int dtype, const float* coefficients,
                          int steps, float eps, float scale, void* const* out, int out_dtype, void* ws,
                          size_t* ws_bytes, hipStream_t stream)
{
    clear_error();
    const Call c{"orthogonalize", size_t(std::max(count, 0)), m, n, out_dtype, coefficients, steps, eps, ws, ws_bytes};
    Layout L;
    if (int rc = check_call(c, L))
        return rc > 0 ? GC_OK : rc;
    if (!dtype_bytes(dtype))
        return refuse(c, "unknown dtype");
    if (m == 0 || n == 0)
        return GC_OK;
    In in{};
    LastOut last{};
    if (!take_pointers(in.x, x, c.count, dtype_bytes(dtype)) ||
        !take_pointers(last.out, out, c.count, dtype_bytes(out_dtype)))
        return refuse(c, "a matrix is NULL or misaligned");
    Buffers at;
    for (size_t k = 0; k < c.count; ++k)
        at.writes(out[k], m * n * dtype_bytes(out_dtype), x[k], m * n * dtype_bytes(dtype));
    if (at.overlap())
        return refuse(c, "an out overlaps another matrix (out[k] may be x[k] itself)");
    last.dtype = out_dtype;
    last.m = uint32_t(m);
    last.n = uint32_t(n);
    last.scale = scale;
    in.dtype = dtype;
    return run_call(c, L, in, last, stream);
}

GCQ_API int muon_step(const float* const* grads, int count, size_t m, size_t n, const float* const* momenta,
                      const void* const* weights, int dtype, int update_dtype, const float* coefficients, int steps,
                      float eps, float grad_scale, double momentum, int nesterov, float lr, const float* lr_scale,
                      float weight_decay, float update_scale, float* const* new_momenta, void* const* new_weights,
                      void* ws, size_t* ws_bytes, hipStream_t stream)
{
    clear_error();
    const Call c{"muon_step", size_t(std::max(count, 0)), m, n, update_dtype, coefficients, steps, eps, ws, ws_bytes};
    Layout L;
    if (int rc = check_call(c, L))
        return rc > 0 ? GC_OK : rc;
    const size_t b = dtype_bytes(dtype);
    if (!b)
        return refuse(c, "unknown dtype");
    if (!(momentum >= 0.0 && momentum < 1.0))
        return refuse(c, "momentum must lie in [0, 1)");
    if (!std::isfinite(grad_scale) || !std::isfinite(lr) || !std::isfinite(weight_decay) ||
        !std::isfinite(update_scale))
        return refuse(c, "a scale, rate or decay is not finite");
    if (!aligned4(lr_scale))
        return refuse(c, "lr_scale is misaligned");
    if (m == 0 || n == 0)
        return GC_OK;
    In in{};
    LastOut last{};
    if (!take_pointers(in.x, reinterpret_cast<const void* const*>(grads), c.count, 4) ||
        !take_pointers(in.momenta, reinterpret_cast<const void* const*>(momenta), c.count, 4) ||
        !take_pointers(in.new_momenta, reinterpret_cast<const void* const*>(new_momenta), c.count, 4) ||
        !take_pointers(last.weights, weights, c.count, b) || !take_pointers(last.out, new_weights, c.count, b))
        return refuse(c, "a matrix is NULL or misaligned");
    Buffers at;
    for (size_t k = 0; k < c.count; ++k) {
        at.reads(grads[k], m * n * 4);
        at.writes(new_momenta[k], m * n * 4, momenta[k], m * n * 4);
        at.writes(new_weights[k], m * n * b, weights[k], m * n * b);
    }
    if (at.overlap())
        return refuse(c, "new momenta or weights overlap another matrix (they may be the old ones themselves)");
    last.dtype = dtype;
    last.update = true;
    last.m = uint32_t(m);
    last.n = uint32_t(n);
    last.scale = update_scale;
    last.lr = lr;
    last.decay = weight_decay;
    last.lr_scale = lr_scale;
    in.dtype = GC_F32;
    in.momentum = true;
    in.mo = Momentum{grad_scale, float(std::min(momentum, 1.0 - momentum)), momentum >= 0.5, nesterov != 0};
    return run_call(c, L, in, last, stream);
}
