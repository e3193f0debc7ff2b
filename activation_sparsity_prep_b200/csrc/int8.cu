// int8.cu -- linear in 8-bit integers with a scale for each token and
// channel (sm_100a):
//   Y[i, j] = x_scale[i] * w_scale[j] * sum_k x[i, k] w[j, k] [+ bias[j]].
// The sum is exact in int32 (K <= 65536, so |sum| <= 2^30); it is rounded
// once to fp32, scaled, biased, and rounded to the output's type.
#include "common.cuh"
#include "ops_common.cuh"
#include "ops_internal.h"

namespace sharq {
namespace {

__device__ __forceinline__ void store_out(const Int8Launch& a, int64_t i, int j, int sum) {
    float y = (float)sum * a.x_scale[i] * a.w_scale[j];
    if (a.bias)
        y += a.bias_fp32 ? static_cast<const float*>(a.bias)[j]
                         : __bfloat162float(static_cast<const __nv_bfloat16*>(a.bias)[j]);
    if (a.y_fp32) static_cast<float*>(a.Y)[i * a.N + j] = y;
    else          static_cast<__nv_bfloat16*>(a.Y)[i * a.N + j] = __float2bfloat16_rn(y);
}

// A warp computes R channels for MT tokens on the dot-product units, its
// lanes striding K in 16-byte pieces.
template <int MT, int R>
__global__ void __launch_bounds__(256)
dot_kernel(const Int8Launch a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int j0 = (blockIdx.x * 8 + warp) * R;
    const int64_t i0 = (int64_t)blockIdx.y * MT;
    if (j0 >= a.N) return;
    const int4* w[R];
    const int4* x[MT];
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = reinterpret_cast<const int4*>(a.w + (int64_t)min(j0 + r, a.N - 1) * a.K);
#pragma unroll
    for (int m = 0; m < MT; ++m) x[m] = reinterpret_cast<const int4*>(a.x + min(i0 + m, a.M - 1) * a.K);
    int acc[MT][R] = {};
    for (int c = lane; c < a.K / 16; c += 32) {
        int4 wv[R];
#pragma unroll
        for (int r = 0; r < R; ++r) wv[r] = w[r][c];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int4 xv = x[m][c];
#pragma unroll
            for (int r = 0; r < R; ++r)
                acc[m][r] = __dp4a(wv[r].x, xv.x, __dp4a(wv[r].y, xv.y, __dp4a(wv[r].z, xv.z, __dp4a(wv[r].w, xv.w, acc[m][r]))));
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int sum = __reduce_add_sync(kFull, acc[m][r]);
            if (lane == 0 && i0 + m < a.M && j0 + r < a.N) store_out(a, i0 + m, j0 + r, sum);
        }
}

template <int MT>
cudaError_t launch_dot(const Int8Launch& p, cudaStream_t s) {
    constexpr int R = 4;
    dim3 grid((unsigned)((p.N + 8 * R - 1) / (8 * R)), 1);
    // grid.y holds at most 65535 token tiles: longer batches go in parts
    Int8Launch q = p;
    for (int64_t i = 0; i < p.M; i += (int64_t)MT * 65535) {
        q.M = p.M - i < (int64_t)MT * 65535 ? p.M - i : (int64_t)MT * 65535;
        q.x = p.x + i * p.K;
        q.x_scale = p.x_scale + i;
        q.Y = static_cast<char*>(p.Y) + i * p.N * (p.y_fp32 ? 4 : 2);
        grid.y = (unsigned)((q.M + MT - 1) / MT);
        dot_kernel<MT, R><<<grid, 256, 0, s>>>(q);
        if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_linear_int8(const Int8Launch& p, cudaStream_t s, int) {
    if (p.M == 0) return cudaSuccess;
    return p.M == 1 ? launch_dot<1>(p, s) : p.M <= 4 ? launch_dot<4>(p, s) : launch_dot<8>(p, s);
}

}  // namespace sharq
