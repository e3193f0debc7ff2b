// route.cu -- routing to experts: the choice of each token's experts, the
// dispatch order that the grouped linear reads, and the weighted sum of the
// expert outputs back to the tokens (sm_100a).  The formulas are in
// include/sharq.h.
#include "common.cuh"
#include "ops_common.cuh"
#include "ops_internal.h"

namespace sharq {
namespace {

constexpr int kRouteWarps = 8;
constexpr int kMaxRouteExperts = 512;
constexpr float kNegInf = -__builtin_inff();

// Order-preserving integer of a float (no NaN; both zeros alike).
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}

// Largest value over the warp and the lowest index that has it.
__device__ __forceinline__ void warp_argmax(float& v, int& e) {
    const uint32_t u = ordered(v);
    const uint32_t m = __reduce_max_sync(kFull, u);
    e = (int)__reduce_min_sync(kFull, u == m ? (uint32_t)e : 0x7fffffffu);
    v = from_ordered(m);
}
__device__ __forceinline__ void warp_argmax(double& v, int& e) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const double w = __shfl_xor_sync(kFull, v, o);
        const int f = __shfl_xor_sync(kFull, e, o);
        if (w > v || (w == v && f < e)) { v = w; e = f; }
    }
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// The choice for one token by one warp; lane l holds experts l, 32 + l, ...
// (l[j] = -inf where masked).  F = float returns false when two scores that
// the choice compares lie within the error of their fp32 evaluation; the
// caller then repeats it in double, so that the experts are those of the
// formula and not of its rounding.  Without a bias the scores' order is that
// of the logits, which needs no evaluation.
template <int NPL, typename F>
__device__ bool choose(const float (&l)[NPL], const float (&b)[NPL], const RouteLaunch& a, int lane,
                       F* scratch, int& id_out, float& w_out) {
    constexpr bool kFp32 = sizeof(F) == 4;
    F s[NPL], key[NPL];
    // |error| of an fp32 score: a relative part from exp, sum and quotient,
    // an absolute one from rounding score + bias
    const float rel = a.sigmoid ? 4.8e-7f : 1.9e-6f;      // 2^-21, 2^-19
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < NPL; ++j) s[j] = l[j] > kNegInf ? F(1) / (F(1) + exp_of(-F(l[j]))) : F(0);
    } else {
        float m = l[0];
#pragma unroll
        for (int j = 1; j < NPL; ++j) m = fmaxf(m, l[j]);
        m = warp_max(m);
        F sum = 0;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            s[j] = l[j] > kNegInf ? exp_of(F(l[j]) - F(m)) : F(0);
            sum += s[j];
        }
        sum = warp_sum(sum);
        const F r = sum > F(0) ? F(1) / sum : F(0);
#pragma unroll
        for (int j = 0; j < NPL; ++j) s[j] *= r;
    }
    const bool scored = a.bias != nullptr;
#pragma unroll
    for (int j = 0; j < NPL; ++j)
        key[j] = !(l[j] > kNegInf) ? F(kNegInf) : scored ? s[j] + F(b[j]) : F(l[j]);

    if (a.groups > 1) {
        const int gs = a.E / a.groups;
        const bool by_score = scored || a.group_top2;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            const int e = j * 32 + lane;
            if (e < a.E)
                scratch[e] = a.group_top2 && !scored ? (l[j] > kNegInf ? s[j] : F(kNegInf)) : key[j];
        }
        __syncwarp();
        F top = F(kNegInf), second = F(kNegInf);
        if (lane < a.groups) {
            // rotated start: the lanes' group strides would share a bank
            int at = lane % gs;
            for (int i = 0; i < gs; ++i) {
                const F v = scratch[lane * gs + at];
                at = at + 1 == gs ? 0 : at + 1;
                if (v > top) { second = top; top = v; }
                else if (v > second) second = v;
            }
            if (a.group_top2 && second > F(kNegInf)) top += second;
        }
        uint32_t chosen = 0;
        F last = 0;
        for (int r = 0; r <= a.topk_groups && r < a.groups; ++r) {
            F v = top;
            int g = lane;
            warp_argmax(v, g);
            if (!(v > F(kNegInf))) break;
            if (r == a.topk_groups) {
                if (kFp32 && by_score && last - v <= F(4.0f * (2.0f * rel + 2.4e-7f * (1.0f + fabsf((float)last)))))
                    return false;
                break;
            }
            chosen |= 1u << g;
            last = v;
            if (lane == g) top = F(kNegInf);
        }
        const uint32_t recip = ((1u << 20) + gs - 1) / gs;      // e * recip >> 20 == e / gs below 512
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            const uint32_t g = (uint32_t)(j * 32 + lane) * recip >> 20;
            if (!(chosen >> (g & 31) & 1u)) key[j] = F(kNegInf);
        }
    }

    int id = -1;
    F w = 0, prev = 0, prev_s = 0;
    const int rounds = kFp32 && scored ? a.k + 1 : a.k;         // one more to see the gap behind the last
    for (int r = 0; r < rounds; ++r) {
        F v = key[0];
        int e = lane;
#pragma unroll
        for (int j = 1; j < NPL; ++j)
            if (key[j] > v) { v = key[j]; e = j * 32 + lane; }
        warp_argmax(v, e);
        if (!(v > F(kNegInf))) break;
        F sv = 0;
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if (j * 32 + lane == e) { sv = s[j]; key[j] = F(kNegInf); }
        sv = __shfl_sync(kFull, sv, e & 31);
        if (kFp32 && scored && r > 0 &&
            prev - v <= F(2.0f * rel * fmaxf((float)prev_s, (float)sv) + 2.4e-7f * (1.0f + fmaxf(fabsf((float)prev), fabsf((float)v)))))
            return false;
        prev = v;
        prev_s = sv;
        if (r < a.k && lane == r) { id = e; w = sv; }
    }
    if (a.renormalize) {
        const F sum = warp_sum(w);
        w = sum > F(0) ? w / sum : F(0);
    }
    id_out = id;
    w_out = (float)(w * F(a.scale));
    return true;
}

// One warp a token.
template <int NPL, bool F32>
__global__ void __launch_bounds__(kRouteWarps * 32)
route_kernel(const RouteLaunch a) {
    extern __shared__ double route_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
    if (t >= a.T) return;
    double* scratch = route_smem + warp * a.E;
    float l[NPL], b[NPL];
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        const int e = j * 32 + lane;
        float v = kNegInf, w = 0.0f;
        if (e < a.E) {
            if (F32) v = static_cast<const float*>(a.logits)[t * a.ld + e];
            else     v = __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[t * a.ld + e]);
            if (a.bias) w = a.bias[e];
        }
        const bool live = v > kNegInf && w > kNegInf;           // false for NaN too
        l[j] = live ? v : kNegInf;
        b[j] = live ? w : 0.0f;
    }
    int id;
    float w;
    if (!choose<NPL, float>(l, b, a, lane, reinterpret_cast<float*>(scratch), id, w))
        choose<NPL, double>(l, b, a, lane, scratch, id, w);
    if (lane < a.k) {
        a.ids[t * a.k + lane] = id;
        a.weights[t * a.k + lane] = w;
    }
}

template <int NPL>
cudaError_t launch_route_n(const RouteLaunch& p, cudaStream_t s) {
    const unsigned grid = (unsigned)((p.T + kRouteWarps - 1) / kRouteWarps);
    const size_t smem = p.groups > 1 ? (size_t)kRouteWarps * p.E * sizeof(double) : 0;
    if (p.fp32) route_kernel<NPL, true><<<grid, kRouteWarps * 32, smem, s>>>(p);
    else        route_kernel<NPL, false><<<grid, kRouteWarps * 32, smem, s>>>(p);
    return cudaGetLastError();
}

// ---------------------------------------------------------- dispatch ------
// Stable counting sort of the n = T * k choices by expert, in one cluster:
// every warp owns a run of consecutive choices and a histogram row in shared
// memory; the rows are scanned over the block's warps, the block totals over
// the cluster (distributed shared memory) and the experts, and a second walk
// over the same run places each choice.  Equal ids inside a group of 32 are
// ranked by a warp match.  No workspace, no atomics: the order is fixed.
constexpr int kDispWarps = 32;

template <int C>
__global__ void __launch_bounds__(kDispWarps * 32)
dispatch_kernel(const DispatchLaunch a) {
    extern __shared__ int disp_smem[];
    int* hist = disp_smem;                        // [kDispWarps][E]
    int* total = hist + kDispWarps * a.E;         // [E] this block's counts
    int* start = total + a.E;                     // [E] first slot of this block's rows
    __shared__ int wsum[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = C > 1 ? (int)cluster_ctarank() : 0;
    const int64_t per = (a.n + (int64_t)C * kDispWarps * 32 - 1) / ((int64_t)C * kDispWarps * 32) * 32;
    const int64_t first = ((int64_t)rank * kDispWarps + warp) * per;
    const int64_t end = first + per < a.n ? first + per : a.n;
    int* mine = hist + warp * a.E;

    for (int i = threadIdx.x; i < kDispWarps * a.E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    for (int64_t i = first + lane; i - lane < end; i += 32) {
        const int e = i < end ? a.ids[i] : -1;
        const bool ok = e >= 0 && e < a.E;
        const unsigned peers = __match_any_sync(kFull, ok ? e : -1);
        if (ok && lane == __ffs(peers) - 1) mine[e] += __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    // exclusive scan of each expert's counts over the block's warps
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int sum = 0;
        for (int w = 0; w < kDispWarps; ++w) {
            const int v = hist[w * a.E + e];
            hist[w * a.E + e] = sum;
            sum += v;
        }
        total[e] = sum;
    }
    if (C > 1) cluster_sync_all();
    else       __syncthreads();
    // experts' first slots: exclusive scan over the experts (E <= blockDim)
    int all = 0, before = 0;
    const int e = threadIdx.x;
    if (e < a.E) {
        for (int r = 0; r < C; ++r) {
            const int v = C > 1 ? __float_as_int(ld_shared_cluster_f32(&total[e], r)) : total[e];
            if (r < rank) before += v;
            all += v;
        }
    }
    int inc = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += wsum[w];
    int live = 0;
    for (int w = 0; w < kDispWarps; ++w) live += wsum[w];
    if (e < a.E) {
        start[e] = base + inc - all + before;
        if (rank == 0) a.offsets[e] = base + inc - all;
    }
    if (rank == 0 && threadIdx.x == 0) a.offsets[a.E] = live;
    __syncthreads();
    for (int64_t i = first + lane; i - lane < end; i += 32) {
        const int e2 = i < end ? a.ids[i] : -1;
        const bool ok = e2 >= 0 && e2 < a.E;
        const unsigned peers = __match_any_sync(kFull, ok ? e2 : -1);
        int at = 0;
        if (ok) at = start[e2] + mine[e2] + __popc(peers & ((1u << lane) - 1u));
        __syncwarp();
        if (ok && lane == __ffs(peers) - 1) mine[e2] += __popc(peers);
        __syncwarp();
        if (i < end) {
            a.position[i] = ok ? at : -1;
            if (ok) a.row_index[at] = (int)(i / a.k);
        }
    }
    // slots behind the last live one name row 0: valid rows of no expert
    for (int64_t i = live + (int64_t)rank * blockDim.x + threadIdx.x; i < a.n; i += (int64_t)C * blockDim.x)
        a.row_index[i] = 0;
    if (C > 1) cluster_sync_all();                // no block leaves while its totals are read
}

template <int C>
cudaError_t launch_dispatch_c(const DispatchLaunch& p, cudaStream_t s) {
    const size_t smem = (size_t)(kDispWarps + 2) * p.E * sizeof(int);
    if (cudaError_t e = cudaFuncSetAttribute(dispatch_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)((kDispWarps + 2) * kMaxRouteExperts * sizeof(int)));
        e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(kDispWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, dispatch_kernel<C>, p);
}

// ----------------------------------------------------------- combine ------
// out[t] = residual[t] + sum_j weights[t, j] * Y[position[t, j]], fp32, j
// ascending, the residual last, one rounding.  One block a token and 2048
// columns; a thread owns 8 columns and issues the loads of up to 8 experts'
// rows together: bound by memory.
template <bool YF32, bool OF32>
__global__ void __launch_bounds__(256)
combine_kernel(const CombineLaunch a) {
    const int64_t t = blockIdx.x;
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * 8;
    if (c >= a.N) return;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int j0 = 0; j0 < a.k; j0 += 8) {
        float v[8][8], w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] = 0.0f;
            int64_t at = -1;
            if (j0 + j < a.k) {
                at = a.position[t * a.k + j0 + j];
                w[j] = a.weights[t * a.k + j0 + j];
            }
            const bool ok = at >= 0 && at < a.rows;
            if (ok) load8<YF32>(a.Y, at * a.N + c, v[j]);
            else {
                w[j] = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = fmaf(w[j], v[j][i], sum[i]);
    }
    if (a.residual) {
        float r[8];
        load8<OF32>(a.residual, t * a.N + c, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += r[i];
    }
    store8<OF32>(a.out, t * a.N + c, sum);
}

}  // namespace

cudaError_t launch_route(const RouteLaunch& p, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    if (p.E <= 32) return launch_route_n<1>(p, s);
    if (p.E <= 64) return launch_route_n<2>(p, s);
    if (p.E <= 128) return launch_route_n<4>(p, s);
    if (p.E <= 256) return launch_route_n<8>(p, s);
    return launch_route_n<16>(p, s);
}

cudaError_t launch_dispatch(const DispatchLaunch& p, cudaStream_t s) {
    // one block covers 4 choices a thread; beyond that a cluster of 8
    return p.n <= 4096 ? launch_dispatch_c<1>(p, s) : launch_dispatch_c<8>(p, s);
}

cudaError_t launch_combine(const CombineLaunch& p, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    const int chunks = p.N / 8;
    const int threads = chunks < 256 ? (chunks + 31) / 32 * 32 : 256;
    const dim3 grid((unsigned)p.T, (unsigned)((chunks + threads - 1) / threads));
    if (p.y_fp32) {
        if (p.out_fp32) combine_kernel<true, true><<<grid, threads, 0, s>>>(p);
        else            combine_kernel<true, false><<<grid, threads, 0, s>>>(p);
    } else {
        if (p.out_fp32) combine_kernel<false, true><<<grid, threads, 0, s>>>(p);
        else            combine_kernel<false, false><<<grid, threads, 0, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace sharq
