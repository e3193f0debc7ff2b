// norm.cu -- the residual addition of a block with the norms, gate and
// modulation around it, and the 8-bit quantiser of a row (sm_100a).
//
//   u  = h, or RMSNorm(h) * post_gamma          (the norm after the block)
//   x' = x + alpha * gate * u                   (residual stream)
//   y  = norm(x') [* gamma + beta] [* (1 + scale) + shift]
//                                               (the norm before the next block)
// y leaves as bf16, or as 8-bit codes with one scale a row:
//   a = max |y|, row_scale = a / 127, code = rne(y * (127 / a)).
//
// One block owns a row and holds it in registers from the load to the
// stores, so every input is read once and every output written once; the
// kernel is bound by memory.  All statistics are fp32 over the unrounded x',
// reduced in an order that depends on K alone: a row's result does not
// depend on the rows around it.
#include "common.cuh"
#include "ops_common.cuh"
#include "ops_internal.h"

namespace sharq {
namespace {

__device__ __forceinline__ uint32_t quantize4(const float* v, float inv) {
    int q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(q[i]) : "f"(v[i] * inv));
    return (q[0] & 0xff) | (q[1] & 0xff) << 8 | (q[2] & 0xff) << 16 | (uint32_t)q[3] << 24;
}

// V chunks of 8 elements a thread: chunk i of a thread is i * blockDim + tid.
template <int V, bool XF32, int THREADS>
__global__ void __launch_bounds__(THREADS)
residual_norm_kernel(const NormLaunch a) {
    __shared__ float red[2][32];
    int turn = 0;
    const int64_t row = blockIdx.x;
    const int chunks = a.K >> 3;
    const float inv_k = 1.0f / (float)a.K;
    float t[V][8];

#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        if (c < chunks) load8<XF32>(a.x, row * a.ldx + c * 8, t[i]);
        else
#pragma unroll
            for (int j = 0; j < 8; ++j) t[i][j] = 0.0f;
    }
    const int64_t group = a.gate || a.scale || a.shift ? row / a.group_rows : 0;
    if (a.h) {
        float u[V][8];
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            if (c < chunks) load8(a.h, a.h_fp32, row * a.ldh + c * 8, u[i]);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) u[i][j] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(u[i][j], u[i][j], ss);
        }
        float r = 1.0f;
        if (a.post_gamma) r = 1.0f / sqrtf(block_reduce<false>(ss, red, turn) * inv_k + a.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            if (c >= chunks) continue;
            float g[8];
            if (a.post_gamma) {
                load8(a.post_gamma, a.norm_fp32, c * 8, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[i][j] *= r * g[j];
            }
            if (a.gate) {
                load8(a.gate, a.mod_fp32, group * a.ld_gate + c * 8, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[i][j] *= g[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) t[i][j] = fmaf(a.alpha, u[i][j], t[i][j]);
        }
    }
    if (a.out_x) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            if (c < chunks) store8<XF32>(a.out_x, row * a.ldo + c * 8, t[i]);
        }
    }
    if (!a.y && !a.codes) return;

    if (a.norm) {
        float mean = 0.0f;
        if (a.norm == 2) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) s += t[i][j];
            mean = block_reduce<false>(s, red, turn) * inv_k;
        }
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool in = i * blockDim.x + threadIdx.x < chunks;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                t[i][j] = in ? t[i][j] - mean : 0.0f;
                ss = fmaf(t[i][j], t[i][j], ss);
            }
        }
        const float r = 1.0f / sqrtf(block_reduce<false>(ss, red, turn) * inv_k + a.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            if (c >= chunks) continue;
            float g[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) t[i][j] *= r;
            if (a.gamma) {
                load8(a.gamma, a.norm_fp32, c * 8, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) t[i][j] *= g[j];
            }
            if (a.beta) {
                load8(a.beta, a.norm_fp32, c * 8, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) t[i][j] += g[j];
            }
            if (a.scale) {
                load8(a.scale, a.mod_fp32, group * a.ld_scale + c * 8, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) t[i][j] = fmaf(t[i][j], g[j], t[i][j]);
            }
            if (a.shift) {
                load8(a.shift, a.mod_fp32, group * a.ld_shift + c * 8, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) t[i][j] += g[j];
            }
        }
    }
    if (a.y) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            if (c < chunks) store8<false>(a.y, row * a.K + c * 8, t[i]);
        }
    }
    if (a.codes) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(t[i][j]));
        m = block_reduce<true>(m, red, turn);
        // below 2^-100 the reciprocal could overflow: such a row is zero
        const bool live = m >= 7.8886091e-31f;
        const float inv = live ? __fdiv_rn(127.0f, m) : 0.0f;
        if (threadIdx.x == 0) a.row_scale[row] = live ? __fdiv_rn(m, 127.0f) : 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            if (c < chunks)
                *reinterpret_cast<uint2*>(a.codes + row * a.K + c * 8) =
                    make_uint2(quantize4(t[i], inv), quantize4(t[i] + 4, inv));
        }
    }
}

template <int V, int THREADS>
cudaError_t launch_v(const NormLaunch& p, cudaStream_t s) {
    const int threads = ((p.K / 8 + V - 1) / V + 31) / 32 * 32;
    if (p.x_fp32) residual_norm_kernel<V, true, THREADS><<<(unsigned)p.M, threads, 0, s>>>(p);
    else          residual_norm_kernel<V, false, THREADS><<<(unsigned)p.M, threads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_residual_norm(const NormLaunch& p, cudaStream_t s) {
    if (p.M == 0) return cudaSuccess;
    // as few chunks a thread as keep the block at 512 threads: the row's
    // loads are then all in flight at once
    if (p.K <= 4096) return launch_v<1, 512>(p, s);
    if (p.K <= 8192) return launch_v<2, 512>(p, s);
    if (p.K <= 16384) return launch_v<4, 512>(p, s);
    return launch_v<8, 512>(p, s);
}

}  // namespace sharq
