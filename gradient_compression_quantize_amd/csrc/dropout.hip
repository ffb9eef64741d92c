// dropout.hip -- dropout whose mask is never stored, and its gradient.
//
// out_i = (keep_i ? x_i / (1 - p) : 0) + residual_i with the mask of
// dropout_mask.h, computed in fp32 and rounded once to the values' type. The
// gradient is the same map with the same mask, without a residual.
//
// Bound by HBM, with the Philox rounds (20 products of 32 x 32 bits for four
// values) close behind for 16-bit types: 67,108,864 bf16 values in 48 us, 5.6
// TB/s of reads and writes, where a plain copy of 1 GB moves 5.2.
#include "dropout_mask.h"

#include <algorithm>

namespace gcq {
namespace {

constexpr int kThreads = 256;

// 16-byte vectors a lane has in flight.
constexpr int kUnroll = 2;

// One workgroup tile is kThreads * kUnroll vectors, lane-contiguous.
// offset4: the Philox slot of value 0 (the mask's offset is a multiple of 4
// here, so that every vector starts on a slot). A lane loads before it
// draws, so the Philox rounds run under the loads. kLoop = false: one tile
// per workgroup.
template <typename T, bool kResidual, bool kLoop>
__global__ __launch_bounds__(kThreads) void dropout_vec_kernel(const T* x, const T* residual,
                                                               T* out, size_t n, uint64_t offset4,
                                                               DropoutArgs a, size_t ntiles)
{
    constexpr int V = kVec<T>;
    const uint64_t key = dropout_key(a);
    for (size_t tile = blockIdx.x; tile < ntiles; tile += gridDim.x) {
        const size_t c0 = tile * (kThreads * kUnroll) + threadIdx.x;
        if ((tile + 1) * (kThreads * kUnroll * V) <= n) {
            vec_f32<T> v[kUnroll], r[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                v[u] = load_vec(x + (c0 + u * kThreads) * V);
                if (kResidual)
                    r[u] = load_vec(residual + (c0 + u * kThreads) * V);
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const size_t c = c0 + u * kThreads;
                if (a.some) {
#pragma unroll
                    for (int s = 0; s < V / 4; ++s) {
                        const U4 w = dropout_words(a, key, offset4 + c * (V / 4) + s);
                        v[u][4 * s] = dropout_apply(a, w.x, v[u][4 * s]);
                        v[u][4 * s + 1] = dropout_apply(a, w.y, v[u][4 * s + 1]);
                        v[u][4 * s + 2] = dropout_apply(a, w.z, v[u][4 * s + 2]);
                        v[u][4 * s + 3] = dropout_apply(a, w.w, v[u][4 * s + 3]);
                    }
                }
                if (kResidual)
                    v[u] += r[u];
                store_vec(out + c * V, v[u]);
            }
        } else {
            // the last tile, a value at a time
            for (size_t i = tile * (kThreads * kUnroll * V) + threadIdx.x; i < n; i += kThreads) {
                float v = float(x[i]);
                if (a.some)
                    v = dropout_apply(a, dropout_word(a, key, offset4 * 4 + i), v);
                if (kResidual)
                    v += float(residual[i]);
                out[i] = T(v);
            }
        }
        if (!kLoop)
            break;
    }
}

// Buffers off 16-byte alignment, or an offset off a multiple of 4: a lane
// takes the (up to four) values of one Philox slot, a value at a time.
template <typename T, bool kResidual>
__global__ __launch_bounds__(kThreads) void dropout_slot_kernel(const T* x, const T* residual,
                                                                T* out, size_t n, uint64_t offset,
                                                                DropoutArgs a)
{
    const uint64_t key = dropout_key(a);
    const unsigned head = unsigned(offset & 3);  // values of slot 0 before value 0
    const size_t nslots = (n + head + 3) >> 2;
    for (size_t q = size_t(blockIdx.x) * kThreads + threadIdx.x; q < nslots;
         q += size_t(gridDim.x) * kThreads) {
        const U4 w = a.some ? dropout_words(a, key, (offset >> 2) + q) : U4{0, 0, 0, 0};
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const size_t j = q * 4 + k;  // index + head
            if (j >= head && j - head < n) {
                const size_t i = j - head;
                float v = float(x[i]);
                if (a.some)
                    v = dropout_apply(a, words[k], v);
                if (kResidual)
                    v += float(residual[i]);
                out[i] = T(v);
            }
        }
    }
}

template <typename T, bool kResidual>
void launch_dropout(const T* x, const T* residual, T* out, size_t n, uint64_t offset,
                    const DropoutArgs& a, hipStream_t stream)
{
    if (aligned16(x) && aligned16(out) && aligned16(residual) && (offset & 3) == 0) {
        const size_t ntiles = ceil_div(n, size_t(kThreads) * kUnroll * kVec<T>);
        const dim3 grid(unsigned(std::min(ntiles, max_grid_blocks())));
        if (ntiles > grid.x)
            hipLaunchKernelGGL((dropout_vec_kernel<T, kResidual, true>), grid, dim3(kThreads), 0,
                               stream, x, residual, out, n, offset >> 2, a, ntiles);
        else
            hipLaunchKernelGGL((dropout_vec_kernel<T, kResidual, false>), grid, dim3(kThreads), 0,
                               stream, x, residual, out, n, offset >> 2, a, ntiles);
        return;
    }
    const size_t nslots = ceil_div(n + (offset & 3), 4);
    const dim3 grid(unsigned(std::min(ceil_div(nslots, kThreads), max_grid_blocks())));
    hipLaunchKernelGGL((dropout_slot_kernel<T, kResidual>), grid, dim3(kThreads), 0, stream, x,
                       residual, out, n, offset, a);
}

int dropout_impl(const char* what, const void* x, const void* residual, size_t n, int dtype,
                 double p, uint64_t seed, uint32_t worker, uint64_t offset, const uint64_t* step,
                 void* out, hipStream_t stream)
{
    clear_error();
    const size_t b = dtype_bytes(dtype);
    if (!b)
        return fail(GC_EINVAL, std::string(what) + ": unknown dtype");
    if (!dropout_p_ok(p))
        return fail(GC_EINVAL, std::string(what) + ": p must lie in [0, 1]");
    if (n > SIZE_MAX / 8 || (n && offset > UINT64_MAX - (n - 1)))
        return fail(GC_EINVAL, std::string(what) + ": offset + n exceeds 2^64");
    if (!aligned_to(step, 8))
        return fail(GC_EINVAL, std::string(what) + ": step must be 8-byte aligned");
    if (n == 0)
        return GC_OK;
    if (!x || !out || !aligned_to(x, b) || !aligned_to(out, b) || !aligned_to(residual, b))
        return fail(GC_EINVAL, std::string(what) + ": a buffer is NULL or misaligned");
    const DropoutArgs a = dropout_args(p, seed, worker, step);
    with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const T* xt = static_cast<const T*>(x);
        if (residual)
            launch_dropout<T, true>(xt, static_cast<const T*>(residual), static_cast<T*>(out), n,
                                    offset, a, stream);
        else
            launch_dropout<T, false>(xt, nullptr, static_cast<T*>(out), n, offset, a, stream);
        return 0;
    });
    return check_launch(what);
}

}  // namespace
}  // namespace gcq

using namespace gcq;

GCQ_API int dropout(const void* x, const void* residual, size_t n, int dtype, double p,
                    uint64_t seed, uint32_t worker, uint64_t offset, const uint64_t* step,
                    void* out, hipStream_t stream)
{
    return dropout_impl("dropout", x, residual, n, dtype, p, seed, worker, offset, step, out,
                        stream);
}

GCQ_API int dropout_backward(const void* grad_out, size_t n, int dtype, double p, uint64_t seed,
                             uint32_t worker, uint64_t offset, const uint64_t* step, void* grad_in,
                             hipStream_t stream)
{
    return dropout_impl("dropout_backward", grad_out, nullptr, n, dtype, p, seed, worker, offset,
                        step, grad_in, stream);
}
