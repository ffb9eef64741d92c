// layer_norm.hip -- layer norm behind a block's dropout and residual sum, and
// its gradient.
//
//   z = x + drop(y),   h = (z - mean) rstd gain + bias
//   mean = mean(z),  rstd = (mean (z - mean)^2 + eps)^-1/2
//
// A row is held in the registers of its team (row_team.h), so that each
// activation is read once and written once and the deviations are taken from
// the mean itself. A wave finds the mean and the squares around it of its own
// part of the row; a team of several waves joins them in one exchange,
//   sum (z - mean)^2 = sum over waves of (squares + count (mean_w - mean)^2),
// which loses nothing where the mean is far larger than the deviations, or where
// there are none.
//
// Gradient, with zhat = (z - mean) rstd and g = dh gain:
//   dx = dz + rstd (g - mean(g) - zhat mean(g zhat)),  dy = dx mask / (1 - p)
//   dgain = sum over rows of dh zhat,  dbias = sum over rows of dh
// Both means go through one exchange. The sums over rows stay in registers,
// leave one partial row a workgroup, and a second launch adds those in order.
//
// HBM bounds it: 16384 x 4096 bf16 takes 52 us forward (two activations, 5.2 TB/s,
// what a large copy reaches) and 83 us backward (three, 4.8 TB/s, 5 us of it the
// second launch); 8192 x 768 bf16 with dropout and sum 12.9 us (four, 3.9 TB/s) and
// backward 19 us (five, 3.3 TB/s: two short launches); 4095 x 1001 fp32 backward with
// dropout 24 us (five, 3.4 TB/s: rows off 16 bytes draw two masks for four values).
// 16-bit rows past 8192 values, whose teams are alone on a compute unit, are
// farthest from it: 4096 x 12288 57 us forward (3.5 TB/s) and 82 backward (3.7). Of 16
// x 768 the kernel takes 3 us, the call 7.5.
#include "row_team.h"

#include <algorithm>
#include <string>

namespace gcq {
namespace {

struct LayerNormArgs {
    const float *gain, *bias;  // NULL: 1 and 0
    size_t rows;
    uint32_t d;
    float eps, inv_d;
    DropoutArgs drop;
};

// Columns of an optional array that is 0 where it is missing.
template <typename R>
__device__ __forceinline__ typename R::F columns_or_zero(const float* p, uint32_t c, uint32_t d)
{
    return p ? R::columns(p, c, d) : typename R::F{};
}

// Values of a row that wave w of a team holds.
template <typename R, int kTeam, int kVecs>
__device__ __forceinline__ float wave_count(int w, uint32_t d)
{
    uint32_t n = 0;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const uint32_t first = R::col(v, w * kWave);
        n += d > first ? min(d - first, uint32_t(kWave * R::V)) : 0;
    }
    return float(n);
}

// A sum and its quotient round by some 2^-24 of the mean each, which is all that a
// row of one value has for deviations: eps = 1e-12 would make them the size of the
// gain. The deviations u from the mean, exact there, say how far it is off: sum u / n.
// Not where they are above a 16th of the mean, as their sum then rounds by more than
// the row's, nor of NaN or infinities: most rows are only asked.
// q: sum u^2, inv: 1 / n.
__device__ __forceinline__ bool mean_is_coarse(float mean, float q, float inv)
{
    return q * inv * 256.0f < mean * mean && q < __builtin_inff();
}

// r: sum u.
__device__ __forceinline__ void correct_mean(float& mean, float& q, float r, float inv)
{
    const float more = r * inv;
    mean += more;
    q = fmaxf(__builtin_fmaf(-r, more, q), 0.0f);
}

// Mean of the row x (zeros behind column d), and sum of squares around it.
template <typename R, int kTeam, int kVecs, bool kAligned>
__device__ __forceinline__ void mean_and_squares(const typename R::F (&x)[kVecs], uint32_t d, float inv_d, int t,
                                                 float* lds, int& half, float& mean, float& squares)
{
    constexpr int kWaves = kTeam / kWave;
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int e = 0; e < R::V; ++e)
            s += x[v][e];
    s = wave_sum(s);
    const int wave = kWaves == 1 ? 0 : __builtin_amdgcn_readfirstlane(t / kWave);
    const float count = wave_count<R, kTeam, kVecs>(wave, d);
    const float inv = kWaves == 1 ? inv_d : count > 0.0f ? 1.0f / count : 0.0f;
    float own = s * inv;
    const auto deviation = [&](int v, int e, float from) {
        return R::col(v, t) + (kAligned ? 0 : e) < d ? x[v][e] - from : 0.0f;
    };
    float q = 0.0f, r = 0.0f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int e = 0; e < R::V; ++e) {
            const float u = deviation(v, e, own);
            q = __builtin_fmaf(u, u, q);
        }
    q = wave_sum(q);
    if (mean_is_coarse(own, q, inv)) {  // (the same in every lane)
        float from = own;
        asm volatile("" : "+v"(from));  // (or the deviations are held until here, 4 to 9 registers)
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int e = 0; e < R::V; ++e)
                r += deviation(v, e, from);
        correct_mean(own, q, wave_sum(r), inv);
    }
    if (kWaves == 1) {
        mean = own;
        squares = q;
        return;
    }
    float* at = lds + half * (3 * kWaves);
    half ^= 1;
    if ((t & (kWave - 1)) == 0) {
        at[wave] = s;
        at[kWaves + wave] = q;
        at[2 * kWaves + wave] = own;
    }
    __syncthreads();
    s = 0.0f;
    for (int w = 0; w < kWaves; ++w)
        s += at[w];
    mean = s * inv_d;
    // the same once more, of the waves' means
    q = r = squares = 0.0f;
    for (int w = 0; w < kWaves; ++w) {
        const float n = wave_count<R, kTeam, kVecs>(w, d);
        const float u = n > 0.0f ? at[2 * kWaves + w] - mean : 0.0f;
        q = __builtin_fmaf(n * u, u, q);
        r = __builtin_fmaf(n, u, r);
        squares += at[kWaves + w];
    }
    if (mean_is_coarse(mean, q, inv_d))
        correct_mean(mean, q, r, inv_d);
    squares += q;
}

// ---- forward --------------------------------------------------------------------
//
// Outputs may be the inputs' own buffers: a thread writes only the values that
// it alone has read before. kSub: there is a y.

template <typename T, int kTeam, int kVecs, bool kAligned, bool kSub>
__global__ __launch_bounds__(kTeam < 256 ? 256 : kTeam) void layer_norm_kernel(
    const T* x, const T* y, LayerNormArgs a, T* z, T* h, float* mean_out, float* rstd_out, size_t teams)
{
    using R = Row<T, kTeam, kVecs, kAligned>;
    using F = typename R::F;
    __shared__ float lds[6 * (kTeam / kWave)];
    int half = 0;
    const int t = threadIdx.x % kTeam;
    const size_t team = size_t(blockIdx.x) * R::kTeams + R::team();
    if (team >= teams)
        return;  // only teams of one wave share a workgroup
    const size_t lo = a.rows * team / teams, hi = a.rows * (team + 1) / teams;
    if (lo >= hi)
        return;
    const uint64_t key = kSub ? dropout_key(a.drop) : 0;
    F gain[kVecs], bias[kVecs];
    typename R::Raw rx[kVecs], ry[kVecs];
    R::load(rx, x, lo, a.d, t);
    if (kSub)
        R::load(ry, y, lo, a.d, t);
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        gain[v] = R::columns(a.gain, R::col(v, t), a.d);
        bias[v] = columns_or_zero<R>(a.bias, R::col(v, t), a.d);
    }
    for (size_t row = lo; row < hi; ++row) {
        F f[kVecs], fy[kVecs];
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            f[v] = R::wide(rx[v]);
            if (kSub)
                fy[v] = R::wide(ry[v]);
        }
        if (row + 1 < hi) {  // under this row's arithmetic
            R::load(rx, x, row + 1, a.d, t);
            if (kSub)
                R::load(ry, y, row + 1, a.d, t);
        }
        if (kSub) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const uint32_t c = R::col(v, t);
                if (a.drop.some) {
                    const uint32_t kept = R::mask(a.drop, key, uint64_t(row) * a.d + c);
#pragma unroll
                    for (int e = 0; e < R::V; ++e)  // 0 where dropped, whatever y holds
                        fy[v][e] = R::keep(kept, e, fy[v][e] * a.drop.scale);
                }
                f[v] += fy[v];
                if (z)
                    R::store(z + row * a.d, c, a.d, f[v]);
            }
        }
        float mean, squares;
        mean_and_squares<R, kTeam, kVecs, kAligned>(f, a.d, a.inv_d, t, lds, half, mean, squares);
        const float rstd = 1.0f / sqrtf(squares * a.inv_d + a.eps);
        if (t == 0) {
            if (mean_out)
                mean_out[row] = mean;
            if (rstd_out)
                rstd_out[row] = rstd;
        }
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            F out;
#pragma unroll
            for (int e = 0; e < R::V; ++e)
                out[e] = __builtin_fmaf((f[v][e] - mean) * rstd, gain[v][e], bias[v][e]);
            R::store(h + row * a.d, R::col(v, t), a.d, out);
        }
    }
}

// ---- backward -------------------------------------------------------------------

// One workgroup for each strip of rows; its teams take the rows in turn. kSub:
// there is a dz or a dy.
template <typename T, int kTeam, int kVecs, bool kAligned, bool kSub>
__global__ __launch_bounds__(kTeam < 256 ? 256 : kTeam) void layer_norm_grad_kernel(
    const T* z, const T* dh, const T* dz, LayerNormArgs a, const float* mean, const float* rstd, T* dx, T* dy,
    float* part_gain, float* part_bias)
{
    using R = Row<T, kTeam, kVecs, kAligned>;
    using F = typename R::F;
    // exchanges of a team of several waves, or the sum over teams of one wave
    constexpr int kLds = R::kTeams > 1 ? (R::kTeams - 1) * kTeam * kVecs * R::V : 2 * 2 * (kTeam / kWave);
    __shared__ float lds[kLds];
    int half = 0;
    const int t = threadIdx.x % kTeam, team = R::team();
    const uint64_t key = kSub ? dropout_key(a.drop) : 0;
    const bool has_dz = kSub && dz, has_dy = kSub && dy;
    const size_t strip = blockIdx.x, strips = gridDim.x;
    const size_t lo = a.rows * strip / strips, hi = a.rows * (strip + 1) / strips;

    F gain[kVecs], sum_gain[kVecs], sum_bias[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        gain[v] = R::columns(a.gain, R::col(v, t), a.d);
        sum_gain[v] = F{};
        sum_bias[v] = F{};
    }
    typename R::Raw next_z[kVecs], next_dh[kVecs], next_dz[kVecs];
    float next_mean = 0.0f, next_rstd = 0.0f;
    const auto fetch = [&](size_t row) {
        R::load(next_z, z, row, a.d, t);
        R::load(next_dh, dh, row, a.d, t);
        if (has_dz)
            R::load(next_dz, dz, row, a.d, t);
        next_mean = mean[row];
        next_rstd = rstd[row];
    };
    // the next row's loads run under this row's arithmetic; a workgroup of
    // 1024 threads, which has 128 registers a lane, takes them row by row
    constexpr bool kAhead = kTeam < 1024;
    if (kAhead && lo + team < hi)
        fetch(lo + team);
    for (size_t row = lo + team; row < hi; row += R::kTeams) {
        if (!kAhead)
            fetch(row);
        const float mu = next_mean, r = next_rstd;
        F zn[kVecs], g[kVecs], more[kVecs];
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            zn[v] = R::wide(next_z[v]);
            g[v] = R::wide(next_dh[v]);
            more[v] = has_dz ? R::wide(next_dz[v]) : F{};
        }
        if (kAhead && row + R::kTeams < hi)
            fetch(row + R::kTeams);
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int e = 0; e < R::V; ++e) {
                zn[v][e] = (zn[v][e] - mu) * r;
                sum_gain[v][e] = __builtin_fmaf(g[v][e], zn[v][e], sum_gain[v][e]);
                sum_bias[v][e] += g[v][e];
                g[v][e] *= gain[v][e];  // (0 behind the last column)
                s[0] += g[v][e];
                s[1] = __builtin_fmaf(g[v][e], zn[v][e], s[1]);
            }
        TeamSum<kTeam, 2>::run(s, lds, half);
        const float c0 = s[0] * a.inv_d, c1 = s[1] * a.inv_d;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const uint32_t c = R::col(v, t);
            F out;
#pragma unroll
            for (int e = 0; e < R::V; ++e)
                out[e] = __builtin_fmaf(r, __builtin_fmaf(-c1, zn[v][e], g[v][e] - c0), more[v][e]);
            R::store(dx + row * a.d, c, a.d, out);
            if (!has_dy)
                continue;
            if (a.drop.some) {
                const uint32_t kept = R::mask(a.drop, key, uint64_t(row) * a.d + c);
#pragma unroll
                for (int e = 0; e < R::V; ++e)
                    out[e] = R::keep(kept, e, out[e] * a.drop.scale);
            }
            R::store(dy + row * a.d, c, a.d, out);
        }
    }
    const auto leave = [&](float* p, F (&s)[kVecs]) {
        if (R::kTeams > 1) {  // of teams of one wave, team 0 adds the others' sums
            __syncthreads();
            if (team > 0) {
#pragma unroll
                for (int v = 0; v < kVecs; ++v)
#pragma unroll
                    for (int e = 0; e < R::V; ++e)
                        lds[(((team - 1) * kVecs + v) * R::V + e) * kTeam + t] = s[v][e];
            }
            __syncthreads();
            if (team > 0)
                return;
            for (int o = 0; o < R::kTeams - 1; ++o)
#pragma unroll
                for (int v = 0; v < kVecs; ++v)
#pragma unroll
                    for (int e = 0; e < R::V; ++e)
                        s[v][e] += lds[((o * kVecs + v) * R::V + e) * kTeam + t];
        }
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
            R::store_columns(p + strip * a.d, R::col(v, t), a.d, s[v]);
    };
    if (part_gain)
        leave(part_gain, sum_gain);
    if (part_bias)
        leave(part_bias, sum_bias);
}

// ---- host side --------------------------------------------------------------------

// Teams of one forward launch, each with a contiguous range of rows: 64 waves a
// compute unit in all, twice what it holds, so that some start while others end.
// 16384 x 4096 bf16: 52.0 us, against 58.4, 60.3 and 56.2 with 8, 16 and 32 and 54.5
// with 128; 4096 x 8192 with dropout 57.6 (65.7, 58.5, 59.1, 61.4). Teams of 16 waves
// do with 32: 4096 x 12288 68.9 (118 with 8, 67.1 with 16, 76.2 with 64). (All with
// the waves' means found once more from their sums, by a division each; the last is
// 57.3 now.)
constexpr size_t forward_teams(int team)
{
    return 256 * (team == 1024 ? 32 : 64) / (team / kWave);
}

// Strips of the backward launch, each of which leaves a partial row. With 1024 (512
// for teams of several waves) 16384 x 4096 bf16 takes 88.9 us instead of 83.2 and
// 4095 x 1001 fp32 34.4 instead of 24.6; with 256, the latter 26.6.
constexpr size_t kWaveStrips = 512, kTeamStrips = 256;

// At least four rows a strip.
size_t grad_strips(size_t rows, bool one_wave)
{
    return std::max<size_t>(1, std::min(one_wave ? kWaveStrips : kTeamStrips, rows / 4));
}

struct GradRoom {
    size_t gain, bias, total;
};

// Room for the most strips, whatever the type.
GradRoom grad_room(size_t rows, size_t d)
{
    const size_t part = (grad_strips(rows, true) * d * 4 + 255) & ~size_t(255);
    return GradRoom{0, part, 2 * part};
}

int check_shape(const char* what, size_t rows, size_t d, int dtype, double p, const uint64_t* step)
{
    if (!dtype_bytes(dtype))
        return fail(GC_EINVAL, std::string(what) + ": unknown dtype");
    if (d == 0)
        return fail(GC_EINVAL, std::string(what) + ": a row must hold at least one value");
    if (d > kMaxNormD || rows > (size_t(1) << 40))
        return fail(GC_EUNSUPPORTED, std::string(what) + ": rows of more than 16384 values, or over 2^40 rows");
    if (!dropout_p_ok(p))
        return fail(GC_EINVAL, std::string(what) + ": p must lie in [0, 1]");
    if (!aligned_to(step, 8))
        return fail(GC_EINVAL, std::string(what) + ": step must be 8-byte aligned");
    return GC_OK;
}

LayerNormArgs layer_norm_args(size_t rows, size_t d, const float* gain, const float* bias, float eps, double p,
                              uint64_t seed, uint32_t worker, const uint64_t* step)
{
    LayerNormArgs a{};
    a.gain = gain;
    a.bias = bias;
    a.rows = rows;
    a.d = uint32_t(d);
    a.eps = eps;
    a.inv_d = float(1.0 / double(d));
    a.drop = dropout_args(p, seed, worker, step);
    return a;
}

}  // namespace
}  // namespace gcq

using namespace gcq;

GCQ_API int layer_norm(const void* x, const void* y, int dtype, size_t rows, size_t d, const float* gain,
                       const float* bias, float eps, double p, uint64_t seed, uint32_t worker, const uint64_t* step,
                       void* z, void* h, float* mean, float* rstd, hipStream_t stream)
{
    clear_error();
    if (int rc = check_shape("layer_norm", rows, d, dtype, p, step))
        return rc;
    if (!(eps >= 0.0f))
        return fail(GC_EINVAL, "layer_norm: eps must not be negative");
    if (z && !y)
        return fail(GC_EINVAL, "layer_norm: z without y (it is x)");
    if (rows == 0)
        return GC_OK;
    const size_t b = dtype_bytes(dtype);
    if (!x || !h)
        return fail(GC_EINVAL, "layer_norm: a buffer is NULL");
    if (!aligned_to(x, b) || !aligned_to(y, b) || !aligned_to(z, b) || !aligned_to(h, b) || !aligned4(gain) ||
        !aligned4(bias) || !aligned4(mean) || !aligned4(rstd))
        return fail(GC_EINVAL, "layer_norm: a buffer is misaligned");
    const LayerNormArgs a = layer_norm_args(rows, d, gain, bias, eps, p, seed, worker, step);
    with_dtype(dtype, [&](auto e) {
        using T = decltype(e);
        const bool aligned = d * b % 16 == 0 && aligned16(x) && aligned16(y) && aligned16(z) && aligned16(h);
        with_team<T>(d, [&](auto team, auto vecs) {
            constexpr int kTeam = decltype(team)::value, kVecs = decltype(vecs)::value;
            constexpr int kWg = kTeam < 256 ? 256 : kTeam;
            const size_t teams = std::min(rows, forward_teams(kTeam));
            const dim3 grid(unsigned(ceil_div(teams, kWg / kTeam)));
            const auto launch = [&](auto kernel) {
                hipLaunchKernelGGL(kernel, grid, dim3(kWg), 0, stream, static_cast<const T*>(x),
                                   static_cast<const T*>(y), a, static_cast<T*>(z), static_cast<T*>(h), mean, rstd,
                                   teams);
            };
            if (aligned && y)
                launch(layer_norm_kernel<T, kTeam, kVecs, true, true>);
            else if (aligned)
                launch(layer_norm_kernel<T, kTeam, kVecs, true, false>);
            else if (y)
                launch(layer_norm_kernel<T, kTeam, kVecs, false, true>);
            else
                launch(layer_norm_kernel<T, kTeam, kVecs, false, false>);
        });
        return 0;
    });
    return check_launch("layer_norm");
}

GCQ_API int layer_norm_grad(const void* z, const void* dh, const void* dz, int dtype, size_t rows, size_t d,
                            const float* gain, double p, uint64_t seed, uint32_t worker, const uint64_t* step,
                            const float* mean, const float* rstd, void* dx, void* dy, float* dgain, float* dbias,
                            void* ws, size_t* ws_bytes, hipStream_t stream)
{
    clear_error();
    if (int rc = check_shape("layer_norm_grad", rows, d, dtype, p, step))
        return rc;
    if (!ws_bytes)
        return fail(GC_EINVAL, "layer_norm_grad: ws_bytes is NULL");
    const GradRoom room = grad_room(rows, d);
    if (!ws) {
        *ws_bytes = room.total;
        return GC_OK;
    }
    const size_t b = dtype_bytes(dtype);
    if (rows && (!z || !dh || !dx || !mean || !rstd))
        return fail(GC_EINVAL, "layer_norm_grad: a buffer is NULL");
    if (!aligned_to(z, b) || !aligned_to(dh, b) || !aligned_to(dz, b) || !aligned_to(dx, b) || !aligned_to(dy, b) ||
        !aligned4(gain) || !aligned4(mean) || !aligned4(rstd) || !aligned4(dgain) || !aligned4(dbias))
        return fail(GC_EINVAL, "layer_norm_grad: a buffer is misaligned");
    if (!aligned16(ws) || *ws_bytes < room.total)
        return fail(GC_EINVAL, "layer_norm_grad: workspace too small or not 16-byte aligned");
    char* w = static_cast<char*>(ws);
    float* part_gain = dgain ? reinterpret_cast<float*>(w + room.gain) : nullptr;
    float* part_bias = dbias ? reinterpret_cast<float*>(w + room.bias) : nullptr;
    size_t strips = 0;
    if (rows) {
        const LayerNormArgs a = layer_norm_args(rows, d, gain, nullptr, 0.0f, p, seed, worker, step);
        with_dtype(dtype, [&](auto e) {
            using T = decltype(e);
            const bool aligned = d * b % 16 == 0 && aligned16(z) && aligned16(dh) && aligned16(dz) && aligned16(dx) &&
                                 aligned16(dy);
            with_team<T>(d, [&](auto team, auto vecs) {
                constexpr int kTeam = decltype(team)::value, kVecs = decltype(vecs)::value;
                strips = grad_strips(rows, kTeam == kWave);
                const auto launch = [&](auto kernel) {
                    hipLaunchKernelGGL(kernel, dim3(unsigned(strips)), dim3(kTeam < 256 ? 256 : kTeam), 0, stream,
                                       static_cast<const T*>(z), static_cast<const T*>(dh),
                                       static_cast<const T*>(dz), a, mean, rstd, static_cast<T*>(dx),
                                       static_cast<T*>(dy), part_gain, part_bias);
                };
                if (!aligned)
                    launch(layer_norm_grad_kernel<T, kTeam, kVecs, false, true>);
                else if (dz || dy)
                    launch(layer_norm_grad_kernel<T, kTeam, kVecs, true, true>);
                else
                    launch(layer_norm_grad_kernel<T, kTeam, kVecs, true, false>);
            });
            return 0;
        });
        if (int rc = check_launch("layer_norm_grad"))
            return rc;
    }
    PartSum sums[3] = {};
    int n = 0;
    if (dgain)
        sums[n++] = PartSum{part_gain, dgain, uint32_t(strips), 1};
    if (dbias)
        sums[n++] = PartSum{part_bias, dbias, uint32_t(strips), 1};
    if (n)
        hipLaunchKernelGGL(sum_parts_kernel, dim3(unsigned(ceil_div(d, kSumCols)), unsigned(n)),
                           dim3(kSumCols * kSumRows), 0, stream, sums[0], sums[1], sums[2], uint32_t(d));
    return check_launch("layer_norm_grad (sums)");
}
