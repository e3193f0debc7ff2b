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
// reduced in an order that depends on K and on the parts of the call: a row's
// result does not depend on the rows around it.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "ops_common.cuh"
#include "ops_internal.h"

namespace sharq {
namespace {

// Codes of four elements: the product is rounded to fp32, then to the nearest
// integer (even on ties) by adding 1.5 * 2^23, whose low byte is the code.  A
// conversion instruction would run at an eighth of the rate.
__device__ __forceinline__ uint32_t quantize4(f2 a, f2 b, float inv) {
    float v[4];
    split_f2(a, v[0], v[1]);
    split_f2(b, v[2], v[3]);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __float_as_uint(__fadd_rn(__fmul_rn(v[i], inv), 12582912.0f));
    return __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
}

// Bytes of one row of x, and of x and h, in a stage of the ring.
__host__ __device__ inline uint32_t x_bytes(const NormLaunch& a) { return (uint32_t)a.K * (a.x_fp32 ? 4 : 2); }
__host__ __device__ inline uint32_t row_bytes(const NormLaunch& a) {
    return x_bytes(a) + (a.h ? (uint32_t)a.K * (a.h_fp32 ? 4 : 2) : 0);
}

constexpr int kMaxRing = 8;
constexpr int kRingBytes = 216 * 1024;    // shared memory that an SM's blocks share

// The vectors of a row come down to three: x' = x + r u P and y = r (x' - mean)
// A + B with P = post_gamma gate alpha, A = gamma (1 + scale) and
// B = beta (1 + scale) + shift.
__device__ __forceinline__ void vector_p(const NormLaunch& a, int64_t group, int k, f2 (&p)[4]) {
    const f2 alpha = make_f2(a.alpha, a.alpha);
    f2 g[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = alpha;
    if (a.post_gamma) {
        load8(a.post_gamma, a.norm_fp32, k, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = mul2(p[j], g[j]);
    }
    if (a.gate) {
        load8(a.gate, a.mod_fp32, group * a.ld_gate + k, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) p[j] = mul2(p[j], g[j]);
    }
}
__device__ __forceinline__ void vectors_ab(const NormLaunch& a, int64_t group, int k, f2 (&m)[4], f2 (&c)[4]) {
    const f2 one = make_f2(1.0f, 1.0f);
    f2 scale[4], g[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) { scale[j] = one; m[j] = one; c[j] = 0; }
    if (a.scale) {
        load8(a.scale, a.mod_fp32, group * a.ld_scale + k, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = scale[j] = add2(one, g[j]);
    }
    if (a.shift) load8(a.shift, a.mod_fp32, group * a.ld_shift + k, c);
    if (a.beta) {
        load8(a.beta, a.norm_fp32, k, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = fma2(g[j], scale[j], c[j]);
    }
    if (a.gamma) {
        load8(a.gamma, a.norm_fp32, k, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = mul2(g[j], scale[j]);
    }
}

// Starts the copies of a row's x and, at h_at, h into a stage.
__device__ __forceinline__ void fetch(const NormLaunch& a, int64_t row, uint8_t* stage, uint32_t h_at, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, row_bytes(a));
    bulk_load(stage, static_cast<const uint8_t*>(a.x) + row * a.ldx * (a.x_fp32 ? 4 : 2), x_bytes(a), bar);
    if (a.h)
        bulk_load(stage + h_at, static_cast<const uint8_t*>(a.h) + row * a.ldh * (a.h_fp32 ? 4 : 2),
                  row_bytes(a) - x_bytes(a), bar);
}

// The row's 8-bit codes and scale.  NaN and infinities reach the scale, so that
// a product with the row is not finite either.
template <int V>
__device__ __forceinline__ void write_codes(const NormLaunch& a, int64_t row, const f2 (&t)[V][4], float (&red)[2][32],
                                            int& turn) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo, hi;
            split_f2(t[i][j], lo, hi);
            m = max_nan(m, max_nan(fabsf(lo), fabsf(hi)));
        }
    m = block_reduce<true>(m, red, turn);
    // below 2^-100 the reciprocal could overflow: such a row is zero
    const bool live = !(m < 7.8886091e-31f);
    const float inv = live ? __fdiv_rn(127.0f, m) : 0.0f;
    if (threadIdx.x == 0) a.row_scale[row] = live ? __fdiv_rn(m, 127.0f) : 0.0f;
    int8_t* out = a.codes + row * a.K;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        if (c < a.K >> 3)
            *reinterpret_cast<uint2*>(out + c * 8) =
                make_uint2(quantize4(t[i][0], t[i][1], inv), quantize4(t[i][2], t[i][3], inv));
    }
}

// V chunks of 8 elements a thread: chunk i of a thread is i * blockDim + tid.
// RING: a block walks rows blockIdx, blockIdx + gridDim, ...; the next
// `stages` of them come into shared memory by bulk copies, so that reads are
// in flight while it waits in its reductions, and P, A and B are made once
// (again where a row's modulation group differs from the last one's).
// Without it a block has one row, loaded straight into registers (few rows:
// no start-up).  Both do the same arithmetic.
template <int V, bool XF32, bool RING>
__global__ void __launch_bounds__(512, RING && V <= 2 ? 2 : 1)
residual_norm_kernel(const __grid_constant__ NormLaunch a, int stages) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][32];
    __shared__ uint64_t full[kMaxRing];
    int turn = 0;
    const int tid = threadIdx.x, width = blockDim.x;
    const int chunks = a.K >> 3;
    const float inv_k = 1.0f / (float)a.K;
    const bool affine = a.gamma || a.scale, shifted = a.beta || a.shift;
    const bool scaled = a.post_gamma || a.gate || a.alpha != 1.0f;
    const uint32_t row_size = RING ? row_bytes(a) : 0;
    chain_begin();
    if (RING) {
        if (tid == 0) {
            for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
            fence_barrier_init();
            for (int s = 0; s < stages; ++s)
                if (blockIdx.x + s * (int64_t)gridDim.x < a.M)
                    fetch(a, blockIdx.x + s * (int64_t)gridDim.x, ring + s * row_size, x_bytes(a), &full[s]);
        }
        __syncthreads();
    }
    f2* const vec_p = reinterpret_cast<f2*>(ring + stages * row_size);       // [K / 2] each, where present
    f2* const vec_a = vec_p + (scaled ? a.K >> 1 : 0);
    f2* const vec_b = vec_a + (affine ? a.K >> 1 : 0);
    int64_t made = -1;
    int s = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const int64_t group = a.group_rows < a.M ? (int64_t)((uint32_t)row / (uint32_t)a.group_rows) : 0;
        if (RING && group != made) {
            // a thread reads only what it writes here: no barrier
            made = group;
            for (int c = tid; c < chunks; c += width) {
                f2 p[4], m[4];
                if (scaled) {
                    vector_p(a, group, c * 8, p);
                    store8<true>(vec_p, c * 8, p);
                }
                vectors_ab(a, group, c * 8, m, p);
                if (affine) store8<true>(vec_a, c * 8, m);
                if (shifted) store8<true>(vec_b, c * 8, p);
            }
        }
        f2 t[V][4];
        const uint8_t* stage = ring + s * row_size;
        if (RING) wait_bar(&full[s], phase);              // a wait that gives up is recorded; the row is then wrong
        const void* x = RING ? static_cast<const void*>(stage) : static_cast<const uint8_t*>(a.x) + row * a.ldx * (XF32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * width + tid;
            if (c < chunks) load8<XF32>(x, c * 8, t[i]);
            else
#pragma unroll
                for (int j = 0; j < 4; ++j) t[i][j] = 0;
        }
        if (a.h) {
            f2 u[V][4];
            const void* h = RING ? static_cast<const void*>(stage + x_bytes(a))
                                 : static_cast<const uint8_t*>(a.h) + row * a.ldh * (a.h_fp32 ? 4 : 2);
            if (a.h_fp32) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int c = i * width + tid;
                    if (c < chunks) load8<true>(h, c * 8, u[i]);
                    else
#pragma unroll
                        for (int j = 0; j < 4; ++j) u[i][j] = 0;
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int c = i * width + tid;
                    if (c < chunks) load8<false>(h, c * 8, u[i]);
                    else
#pragma unroll
                        for (int j = 0; j < 4; ++j) u[i][j] = 0;
                }
            }
            if (a.post_gamma) {
                f2 ss = 0;
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) ss = fma2(u[i][j], u[i][j], ss);
                float lo, hi;
                split_f2(ss, lo, hi);
                const float r = rsqrtf(block_reduce<false>(lo + hi, red, turn) * inv_k + a.eps);
                const f2 rr = make_f2(r, r);
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) u[i][j] = mul2(u[i][j], rr);
            }
            if (scaled) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int c = i * width + tid;
                    if (c < chunks) {
                        f2 p[4];
                        if (RING) load8<true>(vec_p, c * 8, p);
                        else      vector_p(a, group, c * 8, p);
#pragma unroll
                        for (int j = 0; j < 4; ++j) t[i][j] = fma2(u[i][j], p[j], t[i][j]);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) t[i][j] = add2(u[i][j], t[i][j]);
            }
        }
        if (RING) {
            __syncthreads();                              // the stage is read: its next row may come
            const int64_t next = row + stages * (int64_t)gridDim.x;
            if (tid == 0 && next < a.M) fetch(a, next, ring + s * row_size, x_bytes(a), &full[s]);
        }
        if (a.out_x) {
            uint8_t* out = static_cast<uint8_t*>(a.out_x) + row * a.ldo * (XF32 ? 4 : 2);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i * width + tid < chunks) store8<XF32>(out, (i * width + tid) * 8, t[i]);
        }
        if (a.norm) {
            float lo, hi;
            if (a.norm == 2) {
                f2 sum = 0;
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum = add2(sum, t[i][j]);
                split_f2(sum, lo, hi);
                const float mean = block_reduce<false>(lo + hi, red, turn) * inv_k;
                const f2 minus = make_f2(-mean, -mean);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i * width + tid < chunks)
#pragma unroll
                        for (int j = 0; j < 4; ++j) t[i][j] = add2(t[i][j], minus);
            }
            f2 ss = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) ss = fma2(t[i][j], t[i][j], ss);
            split_f2(ss, lo, hi);
            const float r = rsqrtf(block_reduce<false>(lo + hi, red, turn) * inv_k + a.eps);
            const f2 rr = make_f2(r, r);
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) t[i][j] = mul2(t[i][j], rr);
            if (RING) {
                if (affine)
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (i * width + tid < chunks) {
                            f2 m[4];
                            load8<true>(vec_a, (i * width + tid) * 8, m);
#pragma unroll
                            for (int j = 0; j < 4; ++j) t[i][j] = mul2(t[i][j], m[j]);
                        }
                if (shifted)
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (i * width + tid < chunks) {
                            f2 c[4];
                            load8<true>(vec_b, (i * width + tid) * 8, c);
#pragma unroll
                            for (int j = 0; j < 4; ++j) t[i][j] = add2(t[i][j], c[j]);
                        }
            } else if (affine || shifted) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i * width + tid < chunks) {
                        f2 m[4], c[4];
                        vectors_ab(a, group, (i * width + tid) * 8, m, c);
                        if (affine)
#pragma unroll
                            for (int j = 0; j < 4; ++j) t[i][j] = mul2(t[i][j], m[j]);
                        if (shifted)
#pragma unroll
                            for (int j = 0; j < 4; ++j) t[i][j] = add2(t[i][j], c[j]);
                    }
            }
        }
        if (a.y) {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.y) + row * a.K;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i * width + tid < chunks) store8<false>(out, (i * width + tid) * 8, t[i]);
        }
        if (a.codes) write_codes<V>(a, row, t, red, turn);
        if (!RING) return;
        if (++s == stages) { s = 0; phase ^= 1; }
    }
}

// The usual row: every vector has one bf16 source (P = post_gamma or gate,
// A = gamma or 1 + scale, B = beta or shift), alpha is 1 and h is bf16.  The
// ring form with the vectors held raw in registers and the norms fixed at
// compile time: the general form issues 480 instructions a warp and row at
// V = 2, most of them on flags and addresses, and leaves room for fewer
// blocks.  A stage is padded with zeros to whole chunks of the block, so that
// only stores look at the row's end.  The arithmetic is the general form's.
template <int V, bool XF32, int NORM, int H>      // H: 0 no h, 1 added, 2 normed and added
__global__ void __launch_bounds__(512, V <= 2 ? 2 : 1)
residual_norm_fast_kernel(const __grid_constant__ NormLaunch a, int stages) {
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float red[2][32];
    __shared__ uint64_t full[kMaxRing];
    int turn = 0;
    const int tid = threadIdx.x, width = blockDim.x;
    const float inv_k = 1.0f / (float)a.K;
    const int chunks = a.K >> 3;
    const bool last = (V - 1) * width + tid < chunks;     // of a thread's chunks only the last can lie past the row
    const uint32_t pitch_x = V * width * 8 * (XF32 ? 4 : 2), pitch = pitch_x + (H ? V * width * 16 : 0);
    chain_begin();
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
        fence_barrier_init();
        for (int s = 0; s < stages; ++s)
            if (blockIdx.x + s * (int64_t)gridDim.x < a.M)
                fetch(a, blockIdx.x + s * (int64_t)gridDim.x, ring + s * pitch, pitch_x, &full[s]);
    }
    if (!last)
        for (int s = 0; s < stages; ++s) {
            const f2 zero[4] = {0, 0, 0, 0};
            store8<XF32>(ring + s * pitch, ((V - 1) * width + tid) * 8, zero);
            if (H) store8<false>(ring + s * pitch + pitch_x, ((V - 1) * width + tid) * 8, zero);
        }
    __syncthreads();
    const bool has_p = H && (a.post_gamma || a.gate), has_a = NORM && (a.gamma || a.scale);
    const bool has_b = NORM && (a.beta || a.shift), plus_one = a.scale != nullptr;
    const f2 one = make_f2(1.0f, 1.0f);
    uint4 vp[V], va[V], vb[V];
    int64_t made = -1;
    int s = 0;
    uint32_t phase = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const int64_t group = a.group_rows < a.M ? (int64_t)((uint32_t)row / (uint32_t)a.group_rows) : 0;
        if (group != made) {
            made = group;
            const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.gate ? a.gate : a.post_gamma) + (a.gate ? group * a.ld_gate : 0);
            const __nv_bfloat16* m = static_cast<const __nv_bfloat16*>(a.scale ? a.scale : a.gamma) + (a.scale ? group * a.ld_scale : 0);
            const __nv_bfloat16* c = static_cast<const __nv_bfloat16*>(a.shift ? a.shift : a.beta) + (a.shift ? group * a.ld_shift : 0);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int at = i * width + tid;
                vp[i] = va[i] = vb[i] = make_uint4(0, 0, 0, 0);
                if (i == V - 1 && !last) continue;
                if (has_p) vp[i] = reinterpret_cast<const uint4*>(p)[at];
                if (has_a) va[i] = reinterpret_cast<const uint4*>(m)[at];
                if (has_b) vb[i] = reinterpret_cast<const uint4*>(c)[at];
            }
        }
        wait_bar(&full[s], phase);                        // a wait that gives up is recorded; the row is then wrong
        f2 t[V][4], u[V][4];
        const uint8_t* stage = ring + s * pitch;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            load8<XF32>(stage, (i * width + tid) * 8, t[i]);
            if (H) load8<false>(stage + pitch_x, (i * width + tid) * 8, u[i]);
        }
        __syncthreads();                                  // the stage is read: its next row may come
        const int64_t next = row + stages * (int64_t)gridDim.x;
        if (tid == 0 && next < a.M) fetch(a, next, ring + s * pitch, pitch_x, &full[s]);
        float lo, hi;
        if (H == 2) {
            f2 ss = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) ss = fma2(u[i][j], u[i][j], ss);
            split_f2(ss, lo, hi);
            const float r = rsqrtf(block_reduce<false>(lo + hi, red, turn) * inv_k + a.eps);
            const f2 rr = make_f2(r, r);
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) u[i][j] = mul2(u[i][j], rr);
        }
        if (H) {
            if (has_p) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint32_t w[4] = {vp[i].x, vp[i].y, vp[i].z, vp[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) t[i][j] = fma2(u[i][j], bf16x2_f2(w[j]), t[i][j]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) t[i][j] = add2(u[i][j], t[i][j]);
            }
        }
        if (a.out_x) {
            uint8_t* out = static_cast<uint8_t*>(a.out_x) + row * a.ldo * (XF32 ? 4 : 2);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < V - 1 || last) store8<XF32>(out, (i * width + tid) * 8, t[i]);
        }
        if (NORM) {
            if (NORM == 2) {
                f2 sum = 0;
#pragma unroll
                for (int i = 0; i < V; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum = add2(sum, t[i][j]);
                split_f2(sum, lo, hi);
                const float mean = block_reduce<false>(lo + hi, red, turn) * inv_k;
                const f2 minus = make_f2(-mean, -mean);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i < V - 1 || last)
#pragma unroll
                        for (int j = 0; j < 4; ++j) t[i][j] = add2(t[i][j], minus);
            }
            f2 ss = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) ss = fma2(t[i][j], t[i][j], ss);
            split_f2(ss, lo, hi);
            const float r = rsqrtf(block_reduce<false>(lo + hi, red, turn) * inv_k + a.eps);
            const f2 rr = make_f2(r, r);
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) t[i][j] = mul2(t[i][j], rr);
            if (has_a) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint32_t w[4] = {va[i].x, va[i].y, va[i].z, va[i].w};
                    if (plus_one) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) t[i][j] = mul2(t[i][j], add2(one, bf16x2_f2(w[j])));
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) t[i][j] = mul2(t[i][j], bf16x2_f2(w[j]));
                    }
                }
            }
            if (has_b) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint32_t w[4] = {vb[i].x, vb[i].y, vb[i].z, vb[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) t[i][j] = add2(t[i][j], bf16x2_f2(w[j]));
                }
            }
        }
        if (a.y) {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.y) + row * a.K;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < V - 1 || last) store8<false>(out, (i * width + tid) * 8, t[i]);
        }
        if (a.codes) write_codes<V>(a, row, t, red, turn);
        if (++s == stages) { s = 0; phase ^= 1; }
    }
}

template <class Fn>
cudaError_t ring_limit_once(std::atomic<bool> (&done)[64], Fn kernel) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
    return e;
}

// Blocks of `threads` threads that an SM's registers hold.
template <class Fn>
int by_registers(std::atomic<int>& regs, Fn kernel, int threads) {
    int r = regs.load(std::memory_order_relaxed);
    if (!r) {
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, kernel) != cudaSuccess) return 1;
        regs.store(r = (at.numRegs + 7) / 8 * 8, std::memory_order_relaxed);
    }
    return std::max(1, 65536 / (r * threads));
}

// Returns cudaErrorNotSupported where a row does not fit the ring twice or the
// modulation changes before a block has used it a few times.
template <int V, bool XF32, int NORM, int H>
cudaError_t launch_fast(const NormLaunch& p, int threads, cudaStream_t s, int sms) {
    const auto kernel = residual_norm_fast_kernel<V, XF32, NORM, H>;
    static std::atomic<int> regs;
    // as many blocks an SM as its registers hold and as leave each two rows
    const int pitch = V * threads * 8 * ((XF32 ? 4 : 2) + (H ? 2 : 0));
    int resident = std::min({32, 2048 / threads, by_registers(regs, kernel, threads)});
    while (resident > 1 && kRingBytes / resident - 1024 < 2 * pitch) --resident;
    const int stages = std::min(kMaxRing, (kRingBytes / resident - 1024) / pitch);
    if (stages < 2 || ((p.gate || p.scale || p.shift) && p.group_rows < (int64_t)2 * resident * sms))
        return cudaErrorNotSupported;
    static std::atomic<bool> done[64];
    if (cudaError_t e = ring_limit_once(done, kernel); e != cudaSuccess) return e;
    const unsigned grid = (unsigned)std::min<int64_t>(p.M, (int64_t)resident * sms);
    return launch_chained(kernel, dim3(grid), threads, stages * pitch, s, 1, p, stages);
}

template <int V, bool XF32>
cudaError_t launch_fast_any(const NormLaunch& p, int threads, cudaStream_t s, int sms) {
    const int h = !p.h ? 0 : p.post_gamma ? 2 : 1;
    if constexpr (V > 4) {
        // longer rows: registers for the plain quantiser only
        return p.norm || h ? cudaErrorNotSupported : launch_fast<V, XF32, 0, 0>(p, threads, s, sms);
    } else {
        switch (p.norm * 3 + h) {
            case 0: return launch_fast<V, XF32, 0, 0>(p, threads, s, sms);
            case 1: return launch_fast<V, XF32, 0, 1>(p, threads, s, sms);
            case 2: return launch_fast<V, XF32, 0, 2>(p, threads, s, sms);
            case 3: return launch_fast<V, XF32, 1, 0>(p, threads, s, sms);
            case 4: return launch_fast<V, XF32, 1, 1>(p, threads, s, sms);
            case 5: return launch_fast<V, XF32, 1, 2>(p, threads, s, sms);
            case 6: return launch_fast<V, XF32, 2, 0>(p, threads, s, sms);
            case 7: return launch_fast<V, XF32, 2, 1>(p, threads, s, sms);
            default: return launch_fast<V, XF32, 2, 2>(p, threads, s, sms);
        }
    }
}

template <int V, bool XF32>
cudaError_t launch_v(const NormLaunch& p, cudaStream_t s, int sms) {
    const int threads = ((p.K / 8 + V - 1) / V + 31) / 32 * 32;
    const int most = std::max(1, std::min(16, 1024 / threads));
    const int row = (int)row_bytes(p);
    const bool mod = p.gate || p.scale || p.shift;
    const bool few = p.M <= (int64_t)most * sms;          // a block a row: no ring
    const bool plain = p.alpha == 1.0f && !p.h_fp32 && !p.norm_fp32 && !p.mod_fp32 && !(p.post_gamma && p.gate) &&
                       !(p.gamma && p.scale) && !(p.beta && (p.shift || p.scale));
    if (!few && plain) {
        const cudaError_t e = launch_fast_any<V, XF32>(p, threads, s, sms);
        if (e != cudaErrorNotSupported) return e;
    }
    // the general ring: its vectors lie behind the rows.  Not for few rows,
    // rows too long for it, or modulation that changes before a block has
    // used it a few times
    const int vecs = ((p.post_gamma || p.gate || p.alpha != 1.0f ? 1 : 0) + (p.gamma || p.scale ? 1 : 0) +
                      (p.beta || p.shift ? 1 : 0)) * p.K * 4;
    int resident = most;
    while (resident > 1 && kRingBytes / resident - 1024 < vecs + 2 * row) --resident;
    if (few || kRingBytes - 1024 < vecs + 2 * row || (mod && p.group_rows < (int64_t)2 * resident * sms)) {
        return launch_chained(residual_norm_kernel<V, XF32, false>, dim3((unsigned)p.M), threads, 0, s, 1, p, 0);
    }
    const int stages = std::min(kMaxRing, (kRingBytes / resident - 1024 - vecs) / row);
    static std::atomic<bool> done[64];
    if (cudaError_t e = ring_limit_once(done, residual_norm_kernel<V, XF32, true>); e != cudaSuccess) return e;
    return launch_chained(residual_norm_kernel<V, XF32, true>, dim3((unsigned)(resident * sms)), threads,
                          stages * row + vecs, s, 1, p, stages);
}

template <int V>
cudaError_t launch_x(const NormLaunch& p, cudaStream_t s, int sms) {
    return p.x_fp32 ? launch_v<V, true>(p, s, sms) : launch_v<V, false>(p, s, sms);
}

}  // namespace

unsigned take_status_norm() { return take_tu_status(); }

cudaError_t launch_residual_norm(const NormLaunch& p, cudaStream_t s, int sms) {
    if (p.M == 0) return cudaSuccess;
    // At most 512 threads; the split of a row depends on K and on the parts of
    // the call, not on M.  Four chunks a thread halve what a row's reductions
    // and flags cost a warp, and pay where that counts: the bf16 quantiser and
    // two norms (4096 x 3584: 12.2 -> 9.9 us, 22.6 -> 21.4 us); with one
    // reduction and more bytes two chunks keep more warps resident (8190 x
    // 5120 fp32: 84 against 94 us).  The bound is where a norm into 8 bits
    // crosses (4096 rows, two chunks against four: K = 2816 14.4 and 17.9 us,
    // 3200 16.1 and 16.0, 4096 19.0 and 17.3); the quantiser alone and two norms
    // gain from 1024 on, by a tenth (2560: 8.9 and 8.6, 18.2 and 17.2).
    const bool long_work = p.K > 3200 && !p.x_fp32 && (!p.h || p.post_gamma);
    if (p.K <= 256) return launch_x<1>(p, s, sms);
    if (p.K <= 8192 && !long_work) return launch_x<2>(p, s, sms);
    if (p.K <= 16384) return launch_x<4>(p, s, sms);
    return launch_x<8>(p, s, sms);
}

}  // namespace sharq
