// ops_common.cuh -- device helpers of the operators around the linears
// (norm.cu, route.cu, int8.cu): vector loads and stores of bf16 / fp32
// rows, warp and block reductions in a fixed order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace sharq {

constexpr unsigned kFull = 0xffffffffu;

// Chained launches (launch_chained in ops_internal.h): a kernel may be placed
// on the SMs while the one before it on its stream still runs.  chain_begin()
// comes before a kernel's first access to memory that others write: it waits
// until that kernel has ended and its writes are visible, and lets the next
// one be placed.  What is set up before it (barriers, tensor memory, the
// weight on its way into L2) costs no time after it.
__device__ __forceinline__ void chain_begin() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// Two fp32 values in one register pair: sm_100 adds, multiplies and fuses both
// in one instruction.
using f2 = unsigned long long;

__device__ __forceinline__ f2 make_f2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split_f2(f2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 bf16x2_f2(uint32_t w) { return make_f2(bf16_lo(w), bf16_hi(w)); }

// Eight consecutive elements as four pairs, and back.
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t at, f2 (&v)[4]) {
    if constexpr (F32) {
        const ulonglong2* q = reinterpret_cast<const ulonglong2*>(static_cast<const float*>(p) + at);
        const ulonglong2 a = q[0], b = q[1];
        v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
        v[0] = bf16x2_f2(w.x); v[1] = bf16x2_f2(w.y); v[2] = bf16x2_f2(w.z); v[3] = bf16x2_f2(w.w);
    }
}
__device__ __forceinline__ void load8(const void* p, int f32, int64_t at, f2 (&v)[4]) {
    if (f32) load8<true>(p, at, v);
    else     load8<false>(p, at, v);
}
__device__ __forceinline__ uint32_t pack_f2(f2 v) {
    float lo, hi;
    split_f2(v, lo, hi);
    return pack_bf16(lo, hi);
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t at, const f2 (&v)[4]) {
    if constexpr (F32) {
        ulonglong2* q = reinterpret_cast<ulonglong2*>(static_cast<float*>(p) + at);
        q[0] = make_ulonglong2(v[0], v[1]);
        q[1] = make_ulonglong2(v[2], v[3]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + at) =
            make_uint4(pack_f2(v[0]), pack_f2(v[1]), pack_f2(v[2]), pack_f2(v[3]));
    }
}

// Eight consecutive elements at element offset `at` (16-byte aligned).
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
    if constexpr (F32) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        const float4 a = q[0], b = q[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
        v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
        v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
    }
}

// One rounding (nearest even) per element where the destination is bf16.
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&v)[8]) {
    if constexpr (F32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + at) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

// The larger value, NaN where one of them is (fmaxf would take the other).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = max_nan(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

// Bounded wait: a few hundred tries, each of which suspends the thread by
// itself, then mbar_wait(), which times them by the global timer.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait(bar, parity);
}

// Sum (or maximum, NaN if any is) over the block, returned to every thread.  `red` holds
// two sets of 32 words; successive calls alternate between them, so one
// block barrier a call is enough.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float (&red)[2][32], int& turn) {
    v = MAX ? warp_max_nan(v) : warp_sum(v);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return v;
    float* r = red[turn & 1];
    ++turn;
    if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    v = lane < nw ? r[lane] : 0.0f;      // zero is the identity of both (maxima are of magnitudes)
    return MAX ? warp_max_nan(v) : warp_sum(v);
}

}  // namespace sharq
