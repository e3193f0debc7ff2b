// int8.cu -- linear in 8-bit integers with a scale for each token and
// channel (sm_100a):
//   Y[i, j] = (x_scale[i] * sum_k x[i, k] w[j, k]) * w_scale[j] [+ bias[j]].
// The sum is exact in int32 (K <= 65536, so |sum| <= 2^30), whatever the
// order; it is rounded once to fp32, scaled, scaled and biased in one fused
// step, and rounded to the output's type.  Every form below ends in the same
// finish(), so a row's result does not depend on the batch around it.
//
// Three forms:
//   dot     one or two tokens: a warp for two or four channels on the
//           dot-product units, bound by streaming the weight;
//   swapped up to 64 tokens (128 in narrow, long layers): 128 channels x all
//           tokens on the tensor cores (the weight is the M-side operand), K
//           split over a cluster so that narrow layers use every SM; bound by
//           the weight;
//   tiled   128 or 256 tokens x up to 256 channels a tile, persistent, bound
//           by the tensor cores.
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "ops_common.cuh"
#include "ops_internal.h"

namespace sharq {
namespace {

__device__ __forceinline__ float finish(int sum, float xs, float ws, float bias) {
    return __fmaf_rn(__fmul_rn(__int2float_rn(sum), xs), ws, bias);
}

__device__ __forceinline__ float bias_at(const Int8Launch& a, int64_t j) {
    if (!a.bias) return 0.0f;
    return a.bias_fp32 ? static_cast<const float*>(a.bias)[j]
                       : __bfloat162float(static_cast<const __nv_bfloat16*>(a.bias)[j]);
}

__device__ __forceinline__ void store_one(const Int8Launch& a, int64_t i, int64_t j, float y) {
    if (a.y_fp32) static_cast<float*>(a.Y)[i * a.N + j] = y;
    else          static_cast<__nv_bfloat16*>(a.Y)[i * a.N + j] = __float2bfloat16_rn(y);
}

// ---------------------------------------------------------------- dot -----
// A warp computes R channels for MT tokens, its lanes striding K in 16-byte
// pieces.
constexpr int kDotWarps = 4;

template <int MT, int R>
__global__ void __launch_bounds__(kDotWarps * 32)
dot_kernel(const Int8Launch a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int j0 = (blockIdx.x * kDotWarps + warp) * R;
    chain_begin();
    if (j0 >= a.N) return;
    const int4* w[R];
    const int4* x[MT];
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = reinterpret_cast<const int4*>(a.w + (int64_t)min(j0 + r, a.N - 1) * a.K);
#pragma unroll
    for (int m = 0; m < MT; ++m) x[m] = reinterpret_cast<const int4*>(a.x + min((int64_t)m, a.M - 1) * a.K);
    int acc[MT][R] = {};
#pragma unroll (8 / R)
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
            if (lane == 0 && m < a.M && j0 + r < a.N)
                store_one(a, m, j0 + r, finish(sum, a.x_scale[m], a.w_scale[j0 + r], bias_at(a, j0 + r)));
        }
}

template <int MT>
cudaError_t launch_dot(const Int8Launch& p, cudaStream_t s) {
    // two channels a warp where there are few, for more warps; four where there
    // are many, for fewer loads of the tokens (1 x 14336 x 4096: 11.7 against
    // 13.6 us; 1 x 4096 x 4096: 3.7 against 3.5 us)
    const int channels = kDotWarps * (p.N > 8192 ? 4 : 2);
    const dim3 grid((unsigned)((p.N + channels - 1) / channels));
    return p.N > 8192 ? launch_chained(dot_kernel<MT, 4>, grid, kDotWarps * 32, 0, s, 1, p)
                      : launch_chained(dot_kernel<MT, 2>, grid, kDotWarps * 32, 0, s, 1, p);
}

// ------------------------------------------------------- tensor cores -----
constexpr int kRows = 128;                    // rows of the M-side operand of a tile
constexpr int kStep = 128;                    // K a pipeline stage: one 128-byte swizzled row
constexpr uint32_t kABytes = kRows * kStep;
constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 8;                  // blocks of a cluster that share a tile's K
constexpr int kSwappedTokens = 128;           // most tokens of the swapped form
constexpr int kI8Threads = 192;               // TMA warp, MMA warp, four epilogue warps

struct alignas(8) I8Barriers {
    uint64_t full[kMaxStages];
    uint64_t empty[kMaxStages];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint32_t tmem_base;
};

// D (s32, tensor memory) (+)= A (s8, shared) x B (s8, shared)^T, 32 of K.
__device__ __forceinline__ void tc_mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

// The same over a pair of blocks: each holds 128 rows of A and D and half of
// B's rows at the same shared-memory offsets; the even block issues.
__device__ __forceinline__ void tc_mma_i8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

// Arrives on the barrier at this offset in both blocks of the pair once all
// prior tcgen05 operations of this thread finish.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}

// Cluster address of `p` in the even block of the pair.
__device__ __forceinline__ uint32_t even_addr(const void* p) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}

// TMA load into this block's shared memory that completes on the even block's
// barrier.  One block reads each tile: no multicast.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const void* tmap, uint64_t* bar, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%3, %4}], [%2];"
                 :: "r"(smem_u32(dst)), "l"(tmap), "r"(even_addr(bar)), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ void mbar_arrive_even(uint64_t* bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(even_addr(bar)) : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(dst_smem)), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(taddr), "r"(ncols) : "memory");
}

// Instruction descriptor: s32 accumulator (2 at bit 4), signed 8-bit A and B
// (1 at bits 7 and 10), N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t i8_idesc(int n, int m = kRows) {
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

struct Geometry {
    int bn;                  // rows of the N-side operand of a tile
    int stages;
    int sub;                 // k-steps a stage
    int mt, nt;              // tiles along the M-side and the N-side operand
    int bn2, nt2;            // tiled form: narrower tiles behind the nt of width bn, or none
    int n_fast;              // tile walk: N-side fastest
    int split;               // swapped form: blocks of a cluster that share a tile's K
    uint32_t tmem_cols;
};

__device__ __forceinline__ void epilogue_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// One lane of a converged warp.  The TMA and MMA warps run their loops with
// all lanes and elect one around the instructions: loop state and descriptors
// then stay in uniform registers, and an issued MMA costs a few cycles
// instead of the 66 of a loop that only lane 0 runs.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// TMA prefetch of a box into L2.
__device__ __forceinline__ void tma_prefetch_2d(const void* tmap, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" :: "l"(tmap), "r"(x), "r"(y) : "memory");
}

// Place in the ring of stages: the stage's index and the parity of its phase.
struct Ring {
    uint32_t s, phase;
    __device__ __forceinline__ void next(int stages) {
        if (++s == (uint32_t)stages) { s = 0; phase ^= 1; }
    }
};

// Issues the TMA loads of k-steps [k0, k1) of one tile, `sub` a stage, each
// k-step `bytes` into its `block` of the stage.  PAIR: both blocks' loads
// complete on the even block's barrier, which expects the bytes of both.
template <bool PAIR>
__device__ __forceinline__ bool produce(const CUtensorMap* ta, const CUtensorMap* tb, I8Barriers* bars, uint8_t* smem,
                                        uint32_t block, uint32_t bytes, const Geometry& g, Ring& at, int k0, int k1,
                                        int arow, int brow, bool lead = true) {
    for (int k = k0; k < k1; k += g.sub, at.next(g.stages)) {
        if (!__all_sync(kFull, wait_bar(&bars->empty[at.s], at.phase ^ 1))) return false;
        uint8_t* st = smem + at.s * g.sub * block;
        const int n = min(g.sub, k1 - k);
        if (elect_one()) {
            if (!PAIR || lead) mbar_arrive_expect_tx(&bars->full[at.s], (PAIR ? 2 : 1) * n * bytes);
            for (int i = 0; i < n; ++i, st += block) {
                if constexpr (PAIR) {
                    tma_load_2d_pair(st, ta, &bars->full[at.s], (k + i) * kStep, arow);
                    tma_load_2d_pair(st + kABytes, tb, &bars->full[at.s], (k + i) * kStep, brow);
                } else {
                    tma_load_2d(st, ta, &bars->full[at.s], (k + i) * kStep, arow);
                    tma_load_2d(st + kABytes, tb, &bars->full[at.s], (k + i) * kStep, brow);
                }
            }
        }
        __syncwarp();
    }
    return true;
}

// Waits (bounded) for the loads still in flight after an early end: each stage's
// last issued phase.
__device__ __forceinline__ void drain(I8Barriers* bars, int stages, Ring at, bool wrapped) {
    for (int i = 0; i < stages; ++i) {
        const uint32_t parity = i < (int)at.s ? at.phase : at.phase ^ 1;
        if (i < (int)at.s || wrapped) wait_bar(&bars->full[i], parity);
    }
}

// Multiplies nk staged k-steps into the accumulator at tensor-memory address d.
template <bool PAIR>
__device__ __forceinline__ bool multiply(I8Barriers* bars, uint64_t desc0, uint32_t block, const Geometry& g, Ring& at,
                                         int nk, uint32_t d, uint32_t idesc) {
    for (int k = 0; k < nk; k += g.sub, at.next(g.stages)) {
        if (!__all_sync(kFull, wait_bar(&bars->full[at.s], at.phase))) return false;
        tc_fence_after();
        const uint64_t stage = desc0 + at.s * (g.sub * block >> 4);
        const int n = min(g.sub, nk - k);
        if (elect_one()) {
            for (int i = 0; i < n; ++i) {
                const uint64_t da = stage + i * (block >> 4), db = da + (kABytes >> 4);
#pragma unroll
                for (int j = 0; j < kStep / 32; ++j) {
                    if constexpr (PAIR) tc_mma_i8_pair(d, da + 2 * j, db + 2 * j, idesc, (k | i | j) ? 1u : 0u);
                    else                tc_mma_i8(d, da + 2 * j, db + 2 * j, idesc, (k | i | j) ? 1u : 0u);
                }
            }
            if constexpr (PAIR) tc_commit_pair(&bars->empty[at.s]);
            else                tc_commit(&bars->empty[at.s]);
        }
        __syncwarp();
    }
    return true;
}

template <bool PAIR>
__device__ __forceinline__ uint8_t* setup(uint8_t* raw, const Geometry& g, uint32_t block, I8Barriers*& bars,
                                          uint8_t*& tail) {
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    tail = smem + g.stages * g.sub * block;
    bars = reinterpret_cast<I8Barriers*>(tail);
    tail += (sizeof(I8Barriers) + 127) / 128 * 128;
    if (threadIdx.x == 0) {
        for (int s = 0; s < g.stages; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bars->acc_full[b], 1);
            mbar_init(&bars->acc_empty[b], PAIR ? 8 : 4);
        }
        fence_barrier_init();
    }
    if (threadIdx.x >> 5 == 1) {
        if constexpr (PAIR) tmem_alloc_pair(&bars->tmem_base, g.tmem_cols);
        else { tmem_alloc(&bars->tmem_base, g.tmem_cols); tmem_relinquish(); }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync_all();                         // the other block's barriers are ready too
    tc_fence_after();
    return smem;
}

// Tile t of the tiled form: its row tile, first column and width.
struct Tile { int m, col, width; };
__device__ __forceinline__ Tile tile_at(const Geometry& g, int t) {
    const int full = g.mt * g.nt;
    const bool wide = t < full;
    const int nt = wide ? g.nt : g.nt2, bn = wide ? g.bn : g.bn2;
    if (!wide) t -= full;
    int m, n;
    if (g.n_fast) { m = t / nt; n = t - m * nt; }
    else          { n = t / g.mt; m = t - n * g.mt; }
    return {m, (wide ? 0 : g.nt * g.bn) + n * bn, bn};
}

// Tiled form.  A = tokens, B = channels; two accumulators of bn columns, so
// the next tile's MMAs run while the epilogue drains the previous one.  PAIR:
// a tile is 256 tokens over two blocks of a cluster, each loading its 128
// tokens and half of the channels: a third less traffic from L2 for a tile as
// wide (single blocks of 256 columns ask for 19 TB/s and wait for it).  A
// thread drains one token's columns, 128 bytes of output at a time, through
// a staging buffer that turns them into whole 128-byte row segments.
template <bool YF32, bool PAIR>
__global__ void __launch_bounds__(kI8Threads, 1)
tiled_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
             const __grid_constant__ CUtensorMap tb2, const Int8Launch a, const Geometry g) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    constexpr int kShare = PAIR ? 2 : 1;                  // blocks that share a tile's channels
    const uint32_t block = kABytes + g.bn / kShare * kStep;
    I8Barriers* bars;
    uint8_t* tail;
    uint8_t* smem = setup<PAIR>(smem_raw, g, block, bars, tail);
    const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t tmem = __shfl_sync(kFull, bars->tmem_base, 0);
    const int nk = (a.K + kStep - 1) / kStep;
    const int tiles = g.mt * (g.nt + g.nt2);
    const int rank = PAIR ? (int)(blockIdx.x & 1) : 0;     // place in the pair
    const int first = PAIR ? blockIdx.x >> 1 : blockIdx.x, step = PAIR ? gridDim.x >> 1 : gridDim.x;
    constexpr int kTileRows = kShare * kRows;
    chain_begin();

    if (warp == 0) {
        if (elect_one()) { prefetch_tmap(&ta); prefetch_tmap(&tb); }
        __syncwarp();
        Ring at{0, 0};
        int done = 0;
        for (int t = first; t < tiles; t += step, done = 1) {
            const Tile w = tile_at(g, t);
            const int brows = w.width / kShare;           // channels that this block loads
            if (!produce<PAIR>(&ta, w.width == g.bn ? &tb : &tb2, bars, smem, block, kABytes + brows * kStep, g, at, 0, nk,
                               w.m * kTileRows + rank * kRows, w.col + rank * brows, rank == 0)) {
                if (rank == 0) drain(bars, g.stages, at, done || at.phase);
                break;
            }
        }
    } else if (warp == 1 && rank == 0) {
        Ring at{0, 0};
        const uint64_t desc0 = sdesc_sw128(smem_u32(smem));
        uint32_t tc = 0;
        for (int t = first; t < tiles; t += step, ++tc) {
            const uint32_t buf = tc & 1, use = tc >> 1;
            if (use > 0 && !__all_sync(kFull, wait_bar(&bars->acc_empty[buf], (use - 1) & 1))) break;
            tc_fence_after();
            if (!multiply<PAIR>(bars, desc0, block, g, at, nk, tmem + buf * g.bn, i8_idesc(tile_at(g, t).width, kTileRows)))
                break;
            if (elect_one()) {
                if constexpr (PAIR) tc_commit_pair(&bars->acc_full[buf]);
                else                tc_commit(&bars->acc_full[buf]);
            }
            __syncwarp();
        }
    } else if (warp >= 2) {
        constexpr int kCols = YF32 ? 32 : 64;             // columns of one staged 128-byte row segment
        const int q = warp & 3;
        const uint32_t lane_off = (uint32_t)(q * 32) << 16;
        uint8_t* stage = tail + q * 4096;                 // [32 rows][128 bytes], 16-byte units swizzled by row
        float* col_scale = reinterpret_cast<float*>(tail + 4 * 4096);
        float* col_bias = col_scale + 256;
        const int et = threadIdx.x - 64;
        const bool vec = (int64_t)a.N % (YF32 ? 4 : 8) == 0;
        uint32_t tc = 0;
        bool ok = true;                                   // after a wait that gave up: keep step, store nothing
        for (int t = first; t < tiles; t += step, ++tc) {
            const Tile w = tile_at(g, t);
            const int64_t row0 = (int64_t)w.m * kTileRows + rank * kRows + q * 32, col0 = w.col;
            epilogue_bar();                               // the previous tile's columns are no longer read
            for (int c = et; c < w.width; c += 128) {
                const bool in = col0 + c < a.N;
                col_scale[c] = in ? a.w_scale[col0 + c] : 0.0f;
                col_bias[c] = in ? bias_at(a, col0 + c) : 0.0f;
            }
            epilogue_bar();
            const float xs = row0 + lane < a.M ? a.x_scale[row0 + lane] : 0.0f;
            const uint32_t buf = tc & 1, use = tc >> 1;
            ok = __all_sync(kFull, ok && wait_bar(&bars->acc_full[buf], use & 1));
            tc_fence_after();
            if (!ok) continue;
            for (int c0 = 0; c0 < w.width; c0 += kCols) {
                uint32_t v[kCols];
#pragma unroll
                for (int h = 0; h < kCols; h += 32)
                    tmem_ld_32x32b_x32(tmem + buf * g.bn + lane_off + c0 + h, *reinterpret_cast<uint32_t(*)[32]>(v + h));
                tmem_ld_wait();
                if (c0 + kCols >= w.width) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (PAIR) mbar_arrive_even(&bars->acc_empty[buf]);
                        else                mbar_arrive(&bars->acc_empty[buf]);
                    }
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {             // 16-byte units of the row segment
                    uint4 o;
                    uint32_t* word = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (YF32) {
                            const int c = u * 4 + i;
                            word[i] = __float_as_uint(finish((int)v[c], xs, col_scale[c0 + c], col_bias[c0 + c]));
                        } else {
                            const int c = u * 8 + i * 2;
                            word[i] = pack_bf16(finish((int)v[c], xs, col_scale[c0 + c], col_bias[c0 + c]),
                                             finish((int)v[c + 1], xs, col_scale[c0 + c + 1], col_bias[c0 + c + 1]));
                        }
                    }
                    *reinterpret_cast<uint4*>(stage + lane * 128 + ((u ^ (lane & 7)) << 4)) = o;
                }
                __syncwarp();
                if (vec) {
                    constexpr int kPer = YF32 ? 4 : 8;    // elements of a unit
                    const int u = lane & 7;
                    const int64_t col = col0 + c0 + u * kPer;
#pragma unroll
                    for (int r8 = 0; r8 < 8; ++r8) {
                        const int r = r8 * 4 + (lane >> 3);
                        const uint4 o = *reinterpret_cast<const uint4*>(stage + r * 128 + ((u ^ (r & 7)) << 4));
                        if (row0 + r < a.M && col < a.N)
                            *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.Y) +
                                                      ((row0 + r) * a.N + col) * (YF32 ? 4 : 2)) = o;
                    }
                } else {
                    for (int r = 0; r < 32 && row0 + r < a.M; ++r)
                        for (int c = lane; c < kCols; c += 32) {
                            if (col0 + c0 + c >= a.N) continue;
                            const int byte = c * (YF32 ? 4 : 2);
                            const uint8_t* from = stage + r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15);
                            if constexpr (YF32)
                                static_cast<float*>(a.Y)[(row0 + r) * a.N + col0 + c0 + c] = *reinterpret_cast<const float*>(from);
                            else
                                static_cast<uint16_t*>(a.Y)[(row0 + r) * a.N + col0 + c0 + c] = *reinterpret_cast<const uint16_t*>(from);
                        }
                }
                __syncwarp();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync_all();                         // neither block leaves while the other may signal it
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem, g.tmem_cols);
        else                tmem_dealloc(tmem, g.tmem_cols);
    }
}

// Swapped form.  A = 128 channels, B = all M <= bn tokens; the `split` blocks
// of a cluster take a run of k-steps each, leave their int32 partial tiles in
// shared memory, and every block then adds up and finishes its share of the
// tokens over distributed shared memory (integer sums: exact in any order),
// a warp a token, four channels a lane, the ranks' loads in flight together.
__device__ __forceinline__ int4 ld_shared_cluster_v4(const int* p, uint32_t rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    int4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

__global__ void __launch_bounds__(kI8Threads)
swapped_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx, const Int8Launch a,
               const Geometry g) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t block = kABytes + g.bn * kStep;
    I8Barriers* bars;
    uint8_t* tail;
    uint8_t* smem = setup<false>(smem_raw, g, block, bars, tail);
    const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t tmem = __shfl_sync(kFull, bars->tmem_base, 0);
    const int nk = (a.K + kStep - 1) / kStep;
    const int tile = blockIdx.x / g.split, rank = blockIdx.x - tile * g.split;
    const int k0 = (int)((int64_t)nk * rank / g.split), k1 = (int)((int64_t)nk * (rank + 1) / g.split);
    int* partial = reinterpret_cast<int*>(smem);          // [tokens][128], over the stages once they are consumed
    float* xs = reinterpret_cast<float*>(tail);           // [kSwappedTokens] token scales
    const int M = (int)a.M;
    if (warp == 0) {
        // the weight's first stages into L2 before the wait
        if (elect_one()) {
            prefetch_tmap(&tw); prefetch_tmap(&tx);
            for (int k = k0; k < min(k1, k0 + g.stages); ++k) tma_prefetch_2d(&tw, k * kStep, tile * kRows);
        }
        __syncwarp();
    }
    chain_begin();

    if (warp == 0) {
        Ring at{0, 0};
        if (!produce<false>(&tw, &tx, bars, smem, block, block, g, at, k0, k1, tile * kRows, 0))
            drain(bars, g.stages, at, at.phase);
    } else if (warp == 1) {
        Ring at{0, 0};
        if (multiply<false>(bars, sdesc_sw128(smem_u32(smem)), block, g, at, k1 - k0, tmem, i8_idesc(g.bn)) && elect_one())
            tc_commit(&bars->acc_full[0]);
    }
    __syncwarp();
    if (warp >= 2) {
        const int q = warp & 3;
        const int jl = q * 32 + lane;
        const int64_t j = (int64_t)tile * kRows + jl;
        for (int i = threadIdx.x - 64; i < M; i += 128) xs[i] = a.x_scale[i];
        const float ws = j < a.N ? a.w_scale[j] : 0.0f, bias = j < a.N ? bias_at(a, j) : 0.0f;
        epilogue_bar();
        const bool ok = __all_sync(kFull, wait_bar(&bars->acc_full[0], 0));
        tc_fence_after();
        if (ok) {
            for (int c0 = 0; c0 < M; c0 += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(tmem + ((uint32_t)(q * 32) << 16) + c0, v);
                tmem_ld_wait();
                if (g.split > 1) {
                    // bn tokens of room: those past M are written and not read
#pragma unroll
                    for (int i = 0; i < 16; ++i) partial[(c0 + i) * kRows + jl] = (int)v[i];
                } else if (j < a.N) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c0 + i < M) store_one(a, c0 + i, j, finish((int)v[i], xs[c0 + i], ws, bias));
                }
            }
        }
        __syncwarp();
    }
    if (g.split > 1) {
        cluster_sync_all();
        const int t0 = M * rank / g.split, t1 = M * (rank + 1) / g.split;
        const int64_t j = (int64_t)tile * kRows + lane * 4;
        if (t0 + warp < t1 && j < a.N) {
            float ws[4], bias[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                ws[c] = j + c < a.N ? a.w_scale[j + c] : 0.0f;
                bias[c] = j + c < a.N ? bias_at(a, j + c) : 0.0f;
            }
            for (int i = t0 + warp; i < t1; i += kI8Threads / 32) {
                int4 v[kMaxSplit];
#pragma unroll
                for (int r = 0; r < kMaxSplit; ++r)
                    if (r < g.split) v[r] = ld_shared_cluster_v4(&partial[i * kRows + lane * 4], r);
                int4 sum = v[0];
#pragma unroll
                for (int r = 1; r < kMaxSplit; ++r)
                    if (r < g.split) { sum.x += v[r].x; sum.y += v[r].y; sum.z += v[r].z; sum.w += v[r].w; }
                const float y[4] = {finish(sum.x, xs[i], ws[0], bias[0]), finish(sum.y, xs[i], ws[1], bias[1]),
                                    finish(sum.z, xs[i], ws[2], bias[2]), finish(sum.w, xs[i], ws[3], bias[3])};
                const int64_t to = (int64_t)i * a.N + j;
                if (a.N % 4 == 0) {
                    if (a.y_fp32) *reinterpret_cast<float4*>(static_cast<float*>(a.Y) + to) = make_float4(y[0], y[1], y[2], y[3]);
                    else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.Y) + to) =
                             make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (j + c < a.N) store_one(a, i, j + c, y[c]);
                }
            }
        }
        __syncwarp();
        cluster_sync_all();                               // no block leaves while its partial tile is read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) { tc_fence_after(); tmem_dealloc(tmem, g.tmem_cols); }
}

// ------------------------------------------------------------------ host --

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_tiled() {
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeFn>(p);
        return static_cast<EncodeFn>(nullptr);
    }();
    return fn;
}

// [rows, K] bytes in boxes of box_rows x 128, 128-byte swizzle; what lies
// past the rows or past K reads as zero.
bool make_map(CUtensorMap* m, const void* base, int64_t rows, int K, int box_rows) {
    EncodeFn fn = encode_tiled();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)K};
    cuuint32_t box[2] = {(cuuint32_t)kStep, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class Fn>
cudaError_t smem_limit_once(std::atomic<bool> (&done)[64], Fn kernel) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
    return e;
}

constexpr uint32_t kBarBytes = (sizeof(I8Barriers) + 127) / 128 * 128;
constexpr uint32_t kEpilogueBytes = 4 * 4096 + 2 * 256 * 4;

uint32_t tmem_cols(int n) {
    uint32_t c = 32;
    while (c < (uint32_t)n) c *= 2;
    return c;
}

template <bool YF32, bool PAIR>
cudaError_t launch_tiled_t(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tb2, const Int8Launch& p,
                           const Geometry& g, size_t smem, int grid, cudaStream_t s) {
    static std::atomic<bool> done[64];
    if (cudaError_t e = smem_limit_once(done, tiled_kernel<YF32, PAIR>); e != cudaSuccess) return e;
    return launch_chained(tiled_kernel<YF32, PAIR>, dim3((unsigned)grid), kI8Threads, smem, s, PAIR ? 2 : 1, ta, tb, tb2, p, g);
}

// Time of a tile of this width a k-step, in units of 1.3 ns, measured over 128
// k-steps: pairs of blocks 113, 176, 237, 313 ns for 64 to 256 channels,
// single blocks (half as many rows) 120, 220, 297, 396 ns.
int64_t tile_cost(bool pair, int bn) {
    if (bn == 64) return pair ? 88 : 92;
    return pair ? 30 + bn * 83 / 100 : bn + 47;
}

// Shape and order of the tiles.  All of one width, or 256 wide for as many
// whole waves as there are and narrower behind, so that a last wave of a few
// tiles does not take a whole tile's time (4096 x 3584: 224 pair tiles are
// 3.03 waves).
bool plan_tiles(const Int8Launch& p, int sms, Geometry& g) {
    int64_t best = 0;
    bool pair = false;
    for (int two = 1; two >= 0; --two) {
        const int rows = two ? 2 * kRows : kRows, units = two ? sms / 2 : sms;
        const int64_t mt = (p.M + rows - 1) / rows;
        auto take = [&](int bn, int64_t nt, int bn2, int64_t nt2) {
            // the unit with most work is the first, or the first without one more wide tile
            const int64_t wide = mt * nt, all = wide + mt * nt2;
            int64_t cost = 0;
            for (const int64_t c : {(int64_t)0, wide % units}) {
                const int64_t n1 = (wide - c + units - 1) / units, n = (all - c + units - 1) / units;
                cost = std::max(cost, n1 * tile_cost(two, bn) + (n - n1) * tile_cost(two, bn2));
            }
            if (best && cost >= best) return;
            best = cost;
            pair = two;
            g.bn = bn; g.nt = (int)nt; g.bn2 = bn2; g.nt2 = (int)nt2; g.mt = (int)mt;
        };
        for (int bn = 256; bn >= 64; bn -= 64) take(bn, (p.N + bn - 1) / bn, 64, 0);
        const int64_t waves = mt * ((p.N + 255) / 256) / units;
        for (int64_t w = std::max<int64_t>(1, waves - 1); w <= waves; ++w) {
            const int64_t nt = std::min<int64_t>(w * units / mt, p.N / 256);
            const int64_t rest = p.N - nt * 256;
            if (nt > 0 && rest > 0)
                for (int bn = 192; bn >= 64; bn -= 64) take(256, nt, bn, (rest + bn - 1) / bn);
        }
    }
    return pair;
}

cudaError_t launch_tiled(const Int8Launch& p, cudaStream_t s, int sms) {
    Geometry g{};
    sms = std::max(2, sms);
    const bool pair = plan_tiles(p, sms, g);
    g.n_fast = p.M > p.N;                                 // the smaller operand stays in L2
    g.split = 1;
    g.tmem_cols = tmem_cols(2 * g.bn);
    const int share = pair ? 2 : 1;
    // the narrowest tiles: two k-steps a stage, half the barrier steps for their
    // MMAs (128 k-steps of 64 channels: 30.6 -> 25.0 us, pairs 35.2 -> 25.8; no
    // gain from 128 channels on, where fewer stages cost more)
    g.sub = g.bn <= 64 ? 2 : 1;
    const uint32_t stride = g.sub * (kABytes + g.bn / share * kStep);
    g.stages = std::min<int>(kMaxStages, (int)((227 * 1024 - 1024 - kBarBytes - kEpilogueBytes) / stride));
    const size_t smem = 1024 + g.stages * stride + kBarBytes + kEpilogueBytes;
    CUtensorMap ta, tb, tb2;
    if (!make_map(&ta, p.x, p.M, p.K, kRows) || !make_map(&tb, p.w, p.N, p.K, g.bn / share)) return cudaErrorInvalidValue;
    if (g.nt2) {
        if (!make_map(&tb2, p.w, p.N, p.K, g.bn2 / share)) return cudaErrorInvalidValue;
    } else {
        tb2 = tb;
    }
    const int64_t tiles = (int64_t)g.mt * (g.nt + g.nt2);
    if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
    const int grid = share * (int)std::min<int64_t>(tiles, sms / share);
    if (pair)
        return p.y_fp32 ? launch_tiled_t<true, true>(ta, tb, tb2, p, g, smem, grid, s)
                        : launch_tiled_t<false, true>(ta, tb, tb2, p, g, smem, grid, s);
    return p.y_fp32 ? launch_tiled_t<true, false>(ta, tb, tb2, p, g, smem, grid, s)
                    : launch_tiled_t<false, false>(ta, tb, tb2, p, g, smem, grid, s);
}

cudaError_t launch_swapped(const Int8Launch& p, cudaStream_t s, int sms) {
    Geometry g{};
    g.bn = (int)((p.M + 15) / 16 * 16);
    g.mt = (p.N + kRows - 1) / kRows;
    g.nt = 1;
    g.sub = 1;
    g.tmem_cols = tmem_cols(g.bn);
    const int nk = (p.K + kStep - 1) / kStep;
    // Fewer tiles than SMs: split K over a cluster, each block keeping at least
    // 4 k-steps: the split that leaves an SM the fewest k-steps, one block or two
    // to the SM, where clusters fill about seven eighths of the places and their
    // sum costs a few k-steps (6144 x 4096: 144 blocks in clusters of three take
    // 7.5 us, 96 in pairs 6.2; 10240 x 8192: 80 blocks 19.3 us, 240 in clusters
    // of three 15.8; 12288 x 4096: 96 blocks 12.1 us, 768 in eights 14.4).
    g.split = 1;
    const int places = sms * 7 / 8;
    int least = 2 * nk;
    for (int split = 2; split <= std::min(kMaxSplit, nk / 4) && g.mt * split <= 2 * places; ++split) {
        const int held = g.mt * split <= places ? 1 : 2;
        const int cost = 2 * held * ((nk + split - 1) / split) + 6 + split;
        if (cost < least) { least = cost; g.split = split; }
    }
    const uint32_t stride = kABytes + g.bn * kStep;
    // two blocks an SM: one loads while the other finishes
    constexpr uint32_t kExtra = kBarBytes + kSwappedTokens * 4;
    const uint32_t room = 112 * 1024 - 1024 - kExtra;
    g.stages = std::min<int>({kMaxStages, (int)(room / stride), std::max(2, (nk + g.split - 1) / g.split)});
    // the partial tiles, bn x 512 bytes, lie over the stages: two stages of 16 KB
    // and bn x 128 bytes hold them up to bn = 128
    const size_t smem = 1024 + g.stages * stride + kExtra;
    CUtensorMap tw, tx;
    if (!make_map(&tw, p.w, p.N, p.K, kRows) || !make_map(&tx, p.x, p.M, p.K, g.bn)) return cudaErrorInvalidValue;
    static std::atomic<bool> done[64];
    if (cudaError_t e = smem_limit_once(done, swapped_kernel); e != cudaSuccess) return e;
    return launch_chained(swapped_kernel, dim3((unsigned)(g.mt * g.split)), kI8Threads, smem, s, g.split, tw, tx, p, g);
}

}  // namespace

unsigned take_status_int8() { return take_tu_status(); }

cudaError_t launch_linear_int8(const Int8Launch& p, cudaStream_t s, int sms) {
    if (p.M == 0) return cudaSuccess;
    // One or two tokens: the dot form starts sooner (4096 x 4096: 3.1 and 3.4
    // us against 4.7), but its warps walk long rows alone (4096 x 14336: 15
    // against 13 us), and over a large weight it streams slower (28672 x 4096:
    // 21.9 and 24.6 against 20.4 us; two tokens, 5120 x 5120: 6.0 against 5.2).
    const int64_t bytes = (int64_t)p.N * p.K;
    if (p.K <= 8192 && p.M <= 2 && bytes <= (p.M == 1 ? 64 << 20 : 24 << 20))
        return p.M == 1 ? launch_dot<1>(p, s) : launch_dot<2>(p, s);
    // Up to 64 tokens, unless K is short: nothing to split, and the tiled form
    // has less to set up (48 x 1024 x 1024: 4.5 against 5.9 us).  Up to 128 where
    // K is long and there are too few channels for tiles on every SM (N x K, tiled
    // against swapped, us; 72 tokens: 4096 x 14336 19.4 and 15.8, 4736 x 14336 20.5
    // and 18.8, 8192 x 14336 26.3 and 30.2, 4096 x 4096 8.9 and 8.2; 128 tokens:
    // 19.5 and 18.4, 20.4 and 22.2, 26.8 and 35.0, 8.9 and 9.9; 4096 x 8192: 13.1 and
    // 11.4 for 72, 13.1 and 13.2 for 128).
    if (p.K > 1024 && p.M <= (p.K >= 8192 && p.N <= 64 * sms / 2 ? kSwappedTokens : 64)) return launch_swapped(p, s, sms);
    return launch_tiled(p, s, sms);
}

}  // namespace sharq
