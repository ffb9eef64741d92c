// norm_residual.hip -- the path between two blocks of a transformer, and its
// gradient: the norm behind a block, its dropout, its gate, the scaled
// residual sum, and the norm in front of the next block.
//
//   u = y rstd(y) post,   z = s x + gate drop(u),   h = z rstd(z) pre
//   rstd(v) = (mean v^2 + eps)^-1/2
//
// A row is held in the registers of its team of threads (a wave up to four
// 16-byte vectors a lane, then 4 to 16 waves), so that each activation is
// read once and written once. A team takes a contiguous range of rows and
// keeps what its columns need of the gains and the gate in registers.
//
// Gradient, with t the whole gradient of z, q = gate mask post yhat:
//   t = dz + rstd_z (dh pre - zhat c1),  c1 = mean(dh pre zhat)
//   dx = s t,   dy = rstd_y (t gate mask post - yhat c2)
//   c2 = mean(t q) = mean(q (dz + rstd_z dh pre)) - rstd_z c1 mean(q zhat)
// so one exchange of three sums serves both means. The gradients of the gains
// and the gate are sums over rows: a workgroup adds its rows in registers,
// writes one partial row, and a second launch adds the partial rows in their
// order.
//
// Bound by HBM: 16384 x 4096 bf16 with dropout takes 112 us forward (537 MB,
// 4.8 TB/s) and 166 us backward (805 MB, 4.8 TB/s), a plain copy moving 5.2.
// The backward pass has some 60 vector instructions a value, about 105 us of
// them: they have to run under the loads, which the row fetched ahead does.
//
// Past 4096 values a row the backward kernels spill registers (teams of 8
// waves 72 bytes of scratch a lane in 16-bit types and 264 in fp32, of 16 waves
// 224 to 256; off 16 bytes up to 860), and so does the forward one in fp32 past
// 8192: 4096 x 8192 bf16 takes 100 us backward (floor 78), 4096 x 12288 301
// (117). Gates of a few rows each start with nothing fetched ahead and exchange
// their sums: 16383 x 1024 bf16 with 5461 gates takes 78 us backward (floor 48).
#include "dropout_mask.h"

#include <algorithm>
#include <string>

namespace gcq {
namespace {

constexpr size_t kMaxNormD = 16384;

template <int N>
struct Int {
    static constexpr int value = N;
};

struct NormArgs {
    const float *post, *gate, *pre;  // NULL: 1 and no norm, 1, no h
    size_t rows, rows_per_gate;
    uint32_t d;
    float scale, eps, inv_d;
    DropoutArgs drop;
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

// ---- forward --------------------------------------------------------------------
//
// Outputs may be the inputs' own buffers: a thread writes only the values that
// it alone has read before. kAll: every optional argument is there.

template <typename T, int kTeam, int kVecs, bool kAligned, bool kAll>
__global__ __launch_bounds__(kTeam < 256 ? 256 : kTeam) void norm_residual_kernel(
    const T* x, const T* y, NormArgs a, T* z, T* h, float* rstd_post, float* rstd_pre, size_t teams)
{
    using R = Row<T, kTeam, kVecs, kAligned>;
    using F = typename R::F;
    __shared__ float lds[2 * (kTeam / kWave)];
    int half = 0;
    const bool has_post = kAll || a.post, has_pre = kAll || a.pre;
    const int t = threadIdx.x % kTeam;
    const size_t team = size_t(blockIdx.x) * R::kTeams + R::team();
    if (team >= teams)
        return;  // only teams of one wave share a workgroup
    const size_t lo = a.rows * team / teams, hi = a.rows * (team + 1) / teams;
    if (lo >= hi)
        return;
    const uint64_t key = dropout_key(a.drop);
    F w[kVecs], pre[kVecs];  // gate * post of the current group, and pre
    size_t group_end = 0;  // the first row of the next group
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
        pre[v] = R::columns(a.pre, R::col(v, t), a.d);
    typename R::Raw rx[kVecs], ry[kVecs];
    R::load(rx, x, lo, a.d, t);
    R::load(ry, y, lo, a.d, t);
    for (size_t row = lo; row < hi; ++row) {
        if (row >= group_end) {
            const size_t group = row / a.rows_per_gate;
            group_end = (group + 1) * a.rows_per_gate;
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const uint32_t c = R::col(v, t);
                w[v] = R::columns(a.post, c, a.d) * R::columns(a.gate ? a.gate + group * a.d : nullptr, c, a.d);
            }
        }
        F fx[kVecs], fy[kVecs];
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            fx[v] = R::wide(rx[v]);
            fy[v] = R::wide(ry[v]);
        }
        if (row + 1 < hi) {  // under this row's arithmetic
            R::load(rx, x, row + 1, a.d, t);
            R::load(ry, y, row + 1, a.d, t);
        }
        float rp = 1.0f;
        if (has_post) {
            float s[1] = {0.0f};
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
#pragma unroll
                for (int e = 0; e < R::V; ++e)
                    s[0] = __builtin_fmaf(fy[v][e], fy[v][e], s[0]);
            TeamSum<kTeam, 1>::run(s, lds, half);
            rp = 1.0f / sqrtf(s[0] * a.inv_d + a.eps);
            if (t == 0)
                rstd_post[row] = rp;
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const uint32_t c = R::col(v, t);
            F b = fy[v] * rp * w[v];
            if (a.drop.some) {
                const uint32_t kept = R::mask(a.drop, key, uint64_t(row) * a.d + c);
#pragma unroll
                for (int e = 0; e < R::V; ++e)  // 0 where dropped, whatever y holds
                    b[e] = R::keep(kept, e, b[e] * a.drop.scale);
            }
#pragma unroll
            for (int e = 0; e < R::V; ++e) {
                fx[v][e] = __builtin_fmaf(fx[v][e], a.scale, b[e]);
                s[0] = __builtin_fmaf(fx[v][e], fx[v][e], s[0]);
            }
            R::store(z + row * a.d, c, a.d, fx[v]);
        }
        if (has_pre) {
            TeamSum<kTeam, 1>::run(s, lds, half);
            const float rz = 1.0f / sqrtf(s[0] * a.inv_d + a.eps);
            if (t == 0)
                rstd_pre[row] = rz;
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
                R::store(h + row * a.d, R::col(v, t), a.d, fx[v] * rz * pre[v]);
        }
    }
}

// ---- backward -------------------------------------------------------------------

struct NormGradArgs {
    const float *rstd_post, *rstd_pre;
    float *part_post, *part_pre;  // [workgroups][d]
    float* gate_out;              // [gate strips][d]: partial rows, or dgate itself
    size_t strips_per_gate;       // > 1: a gate's rows are split over so many strips
    size_t gates_per_strip;       // > 1: a strip has so many gates (then strips_per_gate is 1)
};

// One workgroup for each strip of rows; its teams take the rows in turn. The
// rows of a strip share a gate, or the strip holds whole gates.
template <typename T, int kTeam, int kVecs, bool kAligned, bool kAll>
__global__ __launch_bounds__(kTeam < 256 ? 256 : kTeam) void norm_residual_grad_kernel(
    const T* z, const T* y, const T* dz, const T* dh, NormArgs a, NormGradArgs g, T* dx, T* dy)
{
    using R = Row<T, kTeam, kVecs, kAligned>;
    using F = typename R::F;
    // exchanges of a team of several waves, or the sum over teams of one wave
    constexpr int kLds = R::kTeams > 1 ? (R::kTeams - 1) * kTeam * kVecs * R::V : 2 * 3 * (kTeam / kWave);
    __shared__ float lds[kLds];
    int half = 0;
    const bool has_post = kAll || a.post, has_pre = kAll || a.pre, has_dz = kAll || dz;
    const int t = threadIdx.x % kTeam, team = R::team();
    const uint64_t key = dropout_key(a.drop);
    const float factor = a.drop.some ? a.drop.scale : 1.0f;
    const size_t strip = blockIdx.x;
    const size_t gates = a.rows / a.rows_per_gate;
    // gates [g_lo, g_hi) of this strip, and its rows of the first one
    const size_t g_lo = g.strips_per_gate > 1 ? strip / g.strips_per_gate : strip * g.gates_per_strip;
    const size_t g_hi = g.strips_per_gate > 1 ? g_lo + 1 : std::min(g_lo + g.gates_per_strip, gates);

    F pre[kVecs], sum_pre[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        pre[v] = R::columns(a.pre, R::col(v, t), a.d);
        sum_pre[v] = F{};
    }
    // teams of one wave: sums over the workgroup's teams end in team 0
    const auto over_teams = [&](F (&s)[kVecs]) {
        if (R::kTeams == 1)
            return;
        __syncthreads();
        if (team > 0) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
#pragma unroll
                for (int e = 0; e < R::V; ++e)
                    lds[(((team - 1) * kVecs + v) * R::V + e) * kTeam + t] = s[v][e];
        }
        __syncthreads();
        if (team == 0) {
            for (int o = 0; o < R::kTeams - 1; ++o)
#pragma unroll
                for (int v = 0; v < kVecs; ++v)
#pragma unroll
                    for (int e = 0; e < R::V; ++e)
                        s[v][e] += lds[((o * kVecs + v) * R::V + e) * kTeam + t];
        }
    };
    // s times r and the columns of f (1 for NULL), onto what this thread wrote there
    // before if `more`
    const auto write = [&](float* p, const F (&s)[kVecs], float r, const float* f, bool more) {
        if (R::kTeams > 1 && team > 0)
            return;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const uint32_t c = R::col(v, t);
            F x = s[v] * r * R::columns(f, c, a.d);
            if (more)
                x += R::columns(p, c, a.d);
            R::store_columns(p, c, a.d, x);
        }
    };

    for (size_t gate = g_lo; gate < g_hi; ++gate) {
        size_t lo = gate * a.rows_per_gate, hi = lo + a.rows_per_gate;
        if (g.strips_per_gate > 1) {
            const size_t s = strip - gate * g.strips_per_gate, n = a.rows_per_gate;
            hi = lo + n * (s + 1) / g.strips_per_gate;
            lo = lo + n * s / g.strips_per_gate;
        }
        // the gate, the post gain and 1 / (1 - p) enter as one factor w; with
        // A = sum of t kept yhat over the rows of a gate, dgate = A post / (1 -
        // p), and dpost is the sum of A gate / (1 - p) over the gates
        F w[kVecs], sum[kVecs];
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const uint32_t c = R::col(v, t);
            w[v] = R::columns(a.gate ? a.gate + gate * a.d : nullptr, c, a.d) * R::columns(a.post, c, a.d) * factor;
            sum[v] = F{};
        }
        typename R::Raw next_y[kVecs], next_dz[kVecs], next_z[kVecs], next_dh[kVecs];
        float next_rz = 0.0f, next_ry = 1.0f;
        const auto fetch = [&](size_t row) {
            R::load(next_y, y, row, a.d, t);
            if (has_dz)
                R::load(next_dz, dz, row, a.d, t);
            if (has_pre) {
                R::load(next_z, z, row, a.d, t);
                R::load(next_dh, dh, row, a.d, t);
                next_rz = g.rstd_pre[row];
            }
            if (has_post)
                next_ry = g.rstd_post[row];
        };
        // the next row's loads run under this row's arithmetic; a workgroup of
        // 1024 threads, which has 128 registers a lane, takes them row by row
        constexpr bool kAhead = kTeam < 1024;
        if (kAhead && lo + team < hi)
            fetch(lo + team);
        for (size_t row = lo + team; row < hi; row += R::kTeams) {
            if (!kAhead)
                fetch(row);
            const float rz = next_rz, ry = next_ry;
            F zn[kVecs], yn[kVecs], e[kVecs], p[kVecs];
            uint32_t kept[kVecs];
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                yn[v] = R::wide(next_y[v]);
                e[v] = has_dz ? R::wide(next_dz[v]) : F{};
                zn[v] = has_pre ? R::wide(next_z[v]) : F{};
                p[v] = has_pre ? R::wide(next_dh[v]) : F{};
            }
            if (kAhead && row + R::kTeams < hi)
                fetch(row + R::kTeams);
            float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const uint32_t c = R::col(v, t);
                yn[v] *= ry;
                kept[v] = ~0u;
                if (a.drop.some) {
                    kept[v] = R::mask(a.drop, key, uint64_t(row) * a.d + c);
                    if (!has_post) {  // a dropped y takes no part, whatever it holds
#pragma unroll
                        for (int k = 0; k < R::V; ++k)
                            yn[v][k] = R::keep(kept[v], k, yn[v][k]);
                    }
                }
                zn[v] *= rz;
#pragma unroll
                for (int k = 0; k < R::V; ++k) {
                    sum_pre[v][k] = __builtin_fmaf(p[v][k], zn[v][k], sum_pre[v][k]);
                    const float gp = p[v][k] * pre[v][k];
                    const float q = w[v][k] * R::keep(kept[v], k, yn[v][k]);
                    e[v][k] = __builtin_fmaf(gp, rz, e[v][k]);
                    s[0] = __builtin_fmaf(gp, zn[v][k], s[0]);
                    s[1] = __builtin_fmaf(q, e[v][k], s[1]);
                    s[2] = __builtin_fmaf(q, zn[v][k], s[2]);
                }
            }
            TeamSum<kTeam, 3>::run(s, lds, half);
            const float c1 = rz * (s[0] * a.inv_d);
            const float c2 = has_post ? ry * ((s[1] - c1 * s[2]) * a.inv_d) : 0.0f;
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const uint32_t c = R::col(v, t);
                F out;
#pragma unroll
                for (int k = 0; k < R::V; ++k) {
                    e[v][k] = __builtin_fmaf(-c1, zn[v][k], e[v][k]);
                    const float wm = R::keep(kept[v], k, e[v][k]);
                    sum[v][k] = __builtin_fmaf(wm, yn[v][k], sum[v][k]);
                    const float direct = wm * w[v][k] * ry;
                    // (without a norm y is in no mean, whatever it holds)
                    out[k] = has_post ? __builtin_fmaf(-c2, yn[v][k], direct) : direct;
                }
                R::store(dx + row * a.d, c, a.d, e[v] * a.scale);
                R::store(dy + row * a.d, c, a.d, out);
            }
        }
        over_teams(sum);
        if (g.part_post)
            write(g.part_post + strip * a.d, sum, factor, a.gate ? a.gate + gate * a.d : nullptr, gate > g_lo);
        if (g.gate_out)
            write(g.gate_out + (g.strips_per_gate > 1 ? strip : gate) * a.d, sum, factor, a.post, false);
    }
    if (g.part_pre) {
        over_teams(sum_pre);
        write(g.part_pre + strip * a.d, sum_pre, 1.0f, nullptr, false);
    }
}

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

// ---- host side --------------------------------------------------------------------

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

// Waves of one launch: 8 a compute unit, each with a contiguous range of
// rows. 16384 x 4096 bf16: 117 us, against 169, 138, 134 and 136 with 4, 6, 10
// and 16; rows dealt out in turn instead took 205. Teams of 16 waves (more than
// 8192 values a row) come to one workgroup for every other compute unit, which
// leaves half of them idle: 4096 x 12288 bf16 takes 168 us, floor 78.
constexpr size_t kForwardWaves = 256 * 8;

// Strips of the backward launch, each of which leaves a partial row: one
// workgroup a compute unit, two where a row is one wave's. 16384 x 4096 bf16
// (teams of four waves): 170 us with 256, 177 with 512; 4095 x 1001 fp32 (of
// one wave): 36 us with 256, 32 with 512.
constexpr size_t kGradStrips = 256, kMaxGradStrips = 512;

struct GradStrips {
    size_t strips, per_gate, gates_per;
};

GradStrips grad_strips(size_t rows, size_t gates, size_t most)
{
    GradStrips s{};
    const size_t rows_per_gate = rows / gates;
    if (gates >= most / 2) {
        s.per_gate = 1;
        s.gates_per = ceil_div(gates, most);
        s.strips = ceil_div(gates, s.gates_per);
    } else {
        // at least four rows a strip
        s.per_gate = std::max<size_t>(1, std::min(most / gates, rows_per_gate / 4));
        s.gates_per = 1;
        s.strips = gates * s.per_gate;
    }
    return s;
}

struct GradRoom {
    size_t post, pre, gate, total;
};

// Room for the most strips, whatever the type.
GradRoom grad_room(size_t rows, size_t d, size_t gates)
{
    const GradStrips s = rows ? grad_strips(rows, gates, kMaxGradStrips) : GradStrips{};
    GradRoom r{};
    const size_t part = (s.strips * d * 4 + 255) & ~size_t(255);
    r.post = 0;
    r.pre = part;
    r.gate = 2 * part;
    r.total = 3 * part;
    return r;
}

int check_shape(const char* what, size_t rows, size_t d, size_t gates, int dtype, double p, const uint64_t* step)
{
    if (!dtype_bytes(dtype))
        return fail(GC_EINVAL, std::string(what) + ": unknown dtype");
    if (d == 0)
        return fail(GC_EINVAL, std::string(what) + ": a row must hold at least one value");
    if (d > kMaxNormD || rows > (size_t(1) << 40))
        return fail(GC_EUNSUPPORTED, std::string(what) + ": rows of more than 16384 values, or over 2^40 rows");
    if (gates == 0 || gates > (size_t(1) << 31) || (rows && rows % gates))
        return fail(GC_EINVAL, std::string(what) + ": the gate's rows must divide the rows");
    if (!dropout_p_ok(p))
        return fail(GC_EINVAL, std::string(what) + ": p must lie in [0, 1]");
    if (!aligned_to(step, 8))
        return fail(GC_EINVAL, std::string(what) + ": step must be 8-byte aligned");
    return GC_OK;
}

NormArgs norm_args(size_t rows, size_t d, const float* post, const float* gate, size_t gates, const float* pre,
                   float scale, float eps, double p, uint64_t seed, uint32_t worker, const uint64_t* step)
{
    NormArgs a{};
    a.post = post;
    a.gate = gate;
    a.pre = pre;
    a.rows = rows;
    a.rows_per_gate = rows / gates;
    a.d = uint32_t(d);
    a.scale = scale;
    a.eps = eps;
    a.inv_d = float(1.0 / double(d));
    a.drop = dropout_args(p, seed, worker, step);
    return a;
}

}  // namespace
}  // namespace gcq

using namespace gcq;

GCQ_API int norm_residual(const void* x, const void* y, int dtype, size_t rows, size_t d, const float* post_gain,
                          const float* gate, size_t gates, const float* pre_gain, float residual_scale, float eps,
                          double p, uint64_t seed, uint32_t worker, const uint64_t* step, void* z, void* h,
                          float* rstd_post, float* rstd_pre, hipStream_t stream)
{
    clear_error();
    if (int rc = check_shape("norm_residual", rows, d, gates, dtype, p, step))
        return rc;
    if (!(eps >= 0.0f))
        return fail(GC_EINVAL, "norm_residual: eps must not be negative");
    if (rows == 0)
        return GC_OK;
    const size_t b = dtype_bytes(dtype);
    if (!x || !y || !z || (pre_gain && (!h || !rstd_pre)) || (post_gain && !rstd_post))
        return fail(GC_EINVAL, "norm_residual: a buffer is NULL");
    if (!pre_gain && h)
        return fail(GC_EINVAL, "norm_residual: h without pre_gain");
    if (!aligned_to(x, b) || !aligned_to(y, b) || !aligned_to(z, b) || !aligned_to(h, b) || !aligned4(post_gain) ||
        !aligned4(gate) || !aligned4(pre_gain) || !aligned4(rstd_post) || !aligned4(rstd_pre))
        return fail(GC_EINVAL, "norm_residual: a buffer is misaligned");
    const NormArgs a = norm_args(rows, d, post_gain, gate, gates, pre_gain, residual_scale, eps, p, seed, worker, step);
    with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const bool aligned = d * b % 16 == 0 && aligned16(x) && aligned16(y) && aligned16(z) && aligned16(h);
        with_team<T>(d, [&](auto team, auto vecs) {
            constexpr int kTeam = decltype(team)::value, kVecs = decltype(vecs)::value;
            constexpr int kWg = kTeam < 256 ? 256 : kTeam;
            const size_t teams = std::min(rows, kForwardWaves / (kTeam / kWave));
            const dim3 grid(unsigned(ceil_div(teams, kWg / kTeam)));
            const auto launch = [&](auto kernel) {
                hipLaunchKernelGGL(kernel, grid, dim3(kWg), 0, stream, static_cast<const T*>(x),
                                   static_cast<const T*>(y), a, static_cast<T*>(z), static_cast<T*>(h), rstd_post,
                                   rstd_pre, teams);
            };
            if (aligned && post_gain && pre_gain)
                launch(norm_residual_kernel<T, kTeam, kVecs, true, true>);
            else if (aligned)
                launch(norm_residual_kernel<T, kTeam, kVecs, true, false>);
            else
                launch(norm_residual_kernel<T, kTeam, kVecs, false, false>);
        });
        return 0;
    });
    return check_launch("norm_residual");
}

GCQ_API int norm_residual_grad(const void* z, const void* y, int dtype, size_t rows, size_t d,
                               const float* post_gain, const float* gate, size_t gates, const float* pre_gain,
                               float residual_scale, double p, uint64_t seed, uint32_t worker, const uint64_t* step,
                               const float* rstd_post, const float* rstd_pre, const void* dz, const void* dh, void* dx,
                               void* dy, float* dpost_gain, float* dgate, float* dpre_gain, void* ws, size_t* ws_bytes,
                               hipStream_t stream)
{
    clear_error();
    if (int rc = check_shape("norm_residual_grad", rows, d, gates, dtype, p, step))
        return rc;
    if (!ws_bytes)
        return fail(GC_EINVAL, "norm_residual_grad: ws_bytes is NULL");
    const GradRoom room = grad_room(rows, d, gates);
    if (!ws) {
        *ws_bytes = std::max<size_t>(room.total, 256);
        return GC_OK;
    }
    const size_t b = dtype_bytes(dtype);
    if ((dpost_gain && !post_gain) || (dgate && !gate) || (dpre_gain && !pre_gain))
        return fail(GC_EINVAL, "norm_residual_grad: a gradient of a gain or gate that is NULL");
    if (rows && (!z || !y || !dx || !dy || (!dz && !dh) || (pre_gain ? !dh || !rstd_pre : dh != nullptr) ||
                 (post_gain && !rstd_post)))
        return fail(GC_EINVAL, "norm_residual_grad: a buffer is NULL (or dh is given without pre_gain)");
    if (!aligned_to(z, b) || !aligned_to(y, b) || !aligned_to(dz, b) || !aligned_to(dh, b) || !aligned_to(dx, b) ||
        !aligned_to(dy, b) || !aligned4(post_gain) || !aligned4(gate) || !aligned4(pre_gain) ||
        !aligned4(rstd_post) || !aligned4(rstd_pre) || !aligned4(dpost_gain) || !aligned4(dgate) ||
        !aligned4(dpre_gain))
        return fail(GC_EINVAL, "norm_residual_grad: a buffer is misaligned");
    if (!aligned16(ws) || *ws_bytes < room.total)
        return fail(GC_EINVAL, "norm_residual_grad: workspace too small or not 16-byte aligned");
    GradStrips s{};
    if (rows)
        with_dtype(dtype, [&](auto t) {
            with_team<decltype(t)>(d, [&](auto team, auto) {
                s = grad_strips(rows, gates, decltype(team)::value == kWave ? kMaxGradStrips : kGradStrips);
            });
            return 0;
        });
    char* w = static_cast<char*>(ws);
    PartSum sums[3] = {};
    int n = 0;
    const auto add = [&](float* out, size_t off, size_t count, size_t out_rows) {
        sums[n++] = PartSum{reinterpret_cast<const float*>(w + off), out, uint32_t(count), uint32_t(out_rows)};
    };
    if (dpost_gain)
        add(dpost_gain, room.post, s.strips, 1);
    if (dpre_gain)
        add(dpre_gain, room.pre, s.strips, 1);
    if (dgate && (rows == 0 || s.per_gate > 1))
        add(dgate, room.gate, rows ? s.per_gate : 0, gates);
    if (rows) {
        const NormArgs a = norm_args(rows, d, post_gain, gate, gates, pre_gain, residual_scale, 0.0f, p, seed, worker,
                                     step);
        NormGradArgs g{};
        g.rstd_post = rstd_post;
        g.rstd_pre = rstd_pre;
        g.part_post = dpost_gain ? reinterpret_cast<float*>(w + room.post) : nullptr;
        g.part_pre = dpre_gain ? reinterpret_cast<float*>(w + room.pre) : nullptr;
        g.gate_out = !dgate ? nullptr : s.per_gate > 1 ? reinterpret_cast<float*>(w + room.gate) : dgate;
        g.strips_per_gate = s.per_gate;
        g.gates_per_strip = s.gates_per;
        with_dtype(dtype, [&](auto t) {
            using T = decltype(t);
            const bool aligned = d * b % 16 == 0 && aligned16(z) && aligned16(y) && aligned16(dz) && aligned16(dh) &&
                                 aligned16(dx) && aligned16(dy);
            with_team<T>(d, [&](auto team, auto vecs) {
                constexpr int kTeam = decltype(team)::value, kVecs = decltype(vecs)::value;
                const auto launch = [&](auto kernel) {
                    hipLaunchKernelGGL(kernel, dim3(unsigned(s.strips)), dim3(kTeam < 256 ? 256 : kTeam), 0, stream,
                                       static_cast<const T*>(z), static_cast<const T*>(y), static_cast<const T*>(dz),
                                       static_cast<const T*>(dh), a, g, static_cast<T*>(dx), static_cast<T*>(dy));
                };
                if (aligned && post_gain && pre_gain && dz)
                    launch(norm_residual_grad_kernel<T, kTeam, kVecs, true, true>);
                else if (aligned)
                    launch(norm_residual_grad_kernel<T, kTeam, kVecs, true, false>);
                else
                    launch(norm_residual_grad_kernel<T, kTeam, kVecs, false, false>);
            });
            return 0;
        });
        if (int rc = check_launch("norm_residual_grad"))
            return rc;
    }
    uint32_t out_rows = 0;
    for (const PartSum& p : sums)
        out_rows += p.rows;
    if (out_rows)
        hipLaunchKernelGGL(sum_parts_kernel, dim3(unsigned(ceil_div(d, kSumCols)), std::min(out_rows, 65535u)),
                           dim3(kSumCols * kSumRows), 0, stream, sums[0], sums[1], sums[2], uint32_t(d));
    return check_launch("norm_residual_grad (sums)");
}
