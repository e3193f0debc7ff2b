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
// One block works on a row at a time and holds it in registers from the load
// to the stores, so every input is read once and every output written once;
// the kernel is bound by memory.  All statistics are fp32 over the unrounded x',
// reduced in an order that depends on K alone: a row's result does not
// depend on the rows around it.
#include <algorithm>
#include <atomic>

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

// Bytes of one row of x, and of x and h, in a stage of the ring.
__host__ __device__ inline uint32_t x_bytes(const NormLaunch& a) { return (uint32_t)a.K * (a.x_fp32 ? 4 : 2); }
__host__ __device__ inline uint32_t row_bytes(const NormLaunch& a) {
    return x_bytes(a) + (a.h ? (uint32_t)a.K * (a.h_fp32 ? 4 : 2) : 0);
}

constexpr int kMaxRing = 8;

// Starts the copies of a row's x and h into a stage.
__device__ __forceinline__ void fetch(const NormLaunch& a, int64_t row, uint8_t* stage, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, row_bytes(a));
    bulk_load(stage, static_cast<const uint8_t*>(a.x) + row * a.ldx * (a.x_fp32 ? 4 : 2), x_bytes(a), bar);
    if (a.h)
        bulk_load(stage + x_bytes(a), static_cast<const uint8_t*>(a.h) + row * a.ldh * (a.h_fp32 ? 4 : 2),
                  row_bytes(a) - x_bytes(a), bar);
}

// V chunks of 8 elements a thread: chunk i of a thread is i * blockDim + tid.
// RING: a block walks rows blockIdx, blockIdx + gridDim, ... and keeps the
// next `stages` of them coming into shared memory by bulk copies, so that
// reads are in flight while it waits in its reductions; without it a block
// has one row, loaded straight into registers (few rows: no start-up).  Both
// do the same arithmetic.
template <int V, bool XF32, bool RING>
__global__ void __launch_bounds__(512, RING && V <= 2 ? 2 : 1)
residual_norm_kernel(const __grid_constant__ NormLaunch a, int stages) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][32];
    __shared__ uint64_t full[kMaxRing];
    int turn = 0;
    const int chunks = a.K >> 3;
    const float inv_k = 1.0f / (float)a.K;
    const int64_t step = gridDim.x;
    if (RING) {
        if (threadIdx.x == 0) {
            for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
            fence_barrier_init();
            for (int s = 0; s < stages; ++s)
                if (blockIdx.x + s * step < a.M) fetch(a, blockIdx.x + s * step, ring + s * row_bytes(a), &full[s]);
        }
        __syncthreads();
    }
    int s = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += step) {
        float t[V][8];
        const uint8_t* stage = ring + s * row_bytes(a);
        if (RING) wait_bar(&full[s], phase);              // a wait that gives up is recorded; the row is then wrong
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            if (c < chunks) load8<XF32>(RING ? stage : a.x, (RING ? 0 : row * a.ldx) + c * 8, t[i]);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) t[i][j] = 0.0f;
        }
        const int64_t group = a.group_rows < a.M ? (int64_t)((uint32_t)row / (uint32_t)a.group_rows) : 0;
        if (a.h) {
            float u[V][8];
            float ss = 0.0f;
            const void* h = RING ? static_cast<const void*>(stage + x_bytes(a)) : a.h;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * blockDim.x + threadIdx.x;
                if (c < chunks) load8(h, a.h_fp32, (RING ? 0 : row * a.ldh) + c * 8, u[i]);
                else
#pragma unroll
                    for (int j = 0; j < 8; ++j) u[i][j] = 0.0f;
            }
            if (RING) {
                __syncthreads();                          // the stage is read: its next row may come
                if (threadIdx.x == 0 && row + stages * step < a.M)
                    fetch(a, row + stages * step, ring + s * row_bytes(a), &full[s]);
            }
            float r = 1.0f;
            if (a.post_gamma) {
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss = fmaf(u[i][j], u[i][j], ss);
                r = 1.0f / sqrtf(block_reduce<false>(ss, red, turn) * inv_k + a.eps);
            }
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
        } else if (RING) {
            __syncthreads();
            if (threadIdx.x == 0 && row + stages * step < a.M)
                fetch(a, row + stages * step, ring + s * row_bytes(a), &full[s]);
        }
        if (a.out_x) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int c = i * blockDim.x + threadIdx.x;
                if (c < chunks) store8<XF32>(a.out_x, row * a.ldo + c * 8, t[i]);
            }
        }
        if (a.norm) {
            float mean = 0.0f;
            if (a.norm == 2) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum += t[i][j];
                mean = block_reduce<false>(sum, red, turn) * inv_k;
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
        if (!RING) return;
        if (++s == stages) { s = 0; phase ^= 1; }
    }
}

template <int V, bool XF32>
cudaError_t launch_v(const NormLaunch& p, cudaStream_t s, int sms) {
    const int threads = ((p.K / 8 + V - 1) / V + 31) / 32 * 32;
    // blocks an SM, and the rows each keeps coming
    const uint32_t bytes = row_bytes(p);
    const int resident = std::max(1, std::min({1024 / threads, 16, (int)(200 * 1024 / bytes)}));
    const int stages = std::max(1, std::min(kMaxRing, (int)(200 * 1024 / (resident * bytes))));
    if (p.M <= (int64_t)resident * sms) {
        residual_norm_kernel<V, XF32, false><<<(unsigned)p.M, threads, 0, s>>>(p, 0);
        return cudaGetLastError();
    }
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !done[dev].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(residual_norm_kernel<V, XF32, true>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
        if (e != cudaSuccess) return e;
        if (dev < 64) done[dev].store(true, std::memory_order_release);
    }
    residual_norm_kernel<V, XF32, true><<<(unsigned)(resident * sms), threads, stages * bytes, s>>>(p, stages);
    return cudaGetLastError();
}

template <int V>
cudaError_t launch_x(const NormLaunch& p, cudaStream_t s, int sms) {
    return p.x_fp32 ? launch_v<V, true>(p, s, sms) : launch_v<V, false>(p, s, sms);
}

}  // namespace

unsigned take_status_norm() { return take_tu_status(); }

cudaError_t launch_residual_norm(const NormLaunch& p, cudaStream_t s, int sms) {
    if (p.M == 0) return cudaSuccess;
    // at most 512 threads; the split of a row depends on K alone
    if (p.K <= 2048) return launch_x<1>(p, s, sms);
    if (p.K <= 8192) return launch_x<2>(p, s, sms);
    if (p.K <= 16384) return launch_x<4>(p, s, sms);
    return launch_x<8>(p, s, sms);
}

}  // namespace sharq
