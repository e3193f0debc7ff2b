// ops_internal.h -- host-side launch interfaces between the C ABI layer and
// the operators around the linears.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace sharq {

// Launches a kernel so that it may be placed on the SMs before the previous
// kernel of its stream has ended; every kernel launched so begins with
// chain_begin() (ops_common.cuh).  cluster: blocks of a cluster.
template <class... P, class... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster,
                           const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Rows of the residual stream: x' = x + alpha * gate * post(h), y = norm(x')
// (see sharq_residual_norm in include/sharq.h).
struct NormLaunch {
    const void* x;
    const void* h;              // null: x' = x
    const void* post_gamma;     // null: no norm of h
    const void* gate;           // null: 1
    const void* gamma;
    const void* beta;
    const void* scale;
    const void* shift;
    void* out_x;                // null: x' is not stored
    void* y;                    // bf16, or null
    int8_t* codes;              // 8-bit y with one scale a row, or null
    float* row_scale;
    int64_t ldx, ldh, ld_gate, ld_scale, ld_shift, ldo;
    int64_t M;
    int64_t group_rows;         // rows that share one row of gate, scale and shift
    int K;
    int norm;                   // 0 none, 1 RMS, 2 layer
    int x_fp32, h_fp32, norm_fp32, mod_fp32;
    float alpha, eps;
};
cudaError_t launch_residual_norm(const NormLaunch& p, cudaStream_t s, int sms);

struct RouteLaunch {
    const void* logits;
    const float* bias;          // null: none
    int32_t* ids;
    float* weights;
    int64_t ld, T;
    int E, k;
    int fp32, sigmoid, groups, topk_groups, group_top2, renormalize;
    float scale;
    // set by launch_route for its kernels
    int group_size;
    int group_whole;            // a group is a power-of-two number of whole lanes
    int group_shift;            // log2 of the lanes that share a group
    int vectors;                // rows can be loaded in vectors
    int bias_vectors;           // the biases can be loaded in vectors
};

struct DispatchLaunch {
    const int32_t* ids;
    int32_t* row_index;
    int32_t* offsets;
    int32_t* position;
    int64_t n;                  // T * k
    int E, k;
};
cudaError_t launch_dispatch(const DispatchLaunch& p, cudaStream_t s);
// order: also build the dispatch order of the ids written, or null.
cudaError_t launch_route(const RouteLaunch& p, const DispatchLaunch* order, cudaStream_t s, int sms);

struct CombineLaunch {
    const void* Y;
    const int32_t* position;
    const float* weights;
    const void* residual;       // null: none
    void* out;
    int64_t T, rows;
    int k, N, y_fp32, out_fp32; // the residual has the output's type
};
cudaError_t launch_combine(const CombineLaunch& p, cudaStream_t s);

struct Int8Launch {
    const int8_t* x;
    const float* x_scale;
    const int8_t* w;
    const float* w_scale;
    const void* bias;           // null: none
    void* Y;
    int64_t M;
    int N, K, bias_fp32, y_fp32;
};
cudaError_t launch_linear_int8(const Int8Launch& p, cudaStream_t s, int sms);

// Read and clear the device status words of these files.
unsigned take_status_norm();
unsigned take_status_int8();

}  // namespace sharq
