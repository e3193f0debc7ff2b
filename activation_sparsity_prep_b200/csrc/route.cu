// route.cu -- routing to experts: the choice of each token's experts, the
// dispatch order that the grouped linear reads, and the weighted sum of the
// expert outputs back to the tokens (sm_100a).  The formulas are in
// include/sharq.h.
#include <algorithm>
#include <atomic>

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
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return a > b ? a : b; }
__device__ __forceinline__ float smaller(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return a < b ? a : b; }

// Lane i of the warp that routes a token holds experts NPL i .. NPL i + NPL-1:
// a row is loaded in vectors, and a gather in lane order is in expert order.
// -inf where masked: beyond E, a logit or a bias of -inf or NaN.
template <int NPL, bool F32>
__device__ __forceinline__ void load_vectors(const RouteLaunch& a, int64_t t, int e0, float (&l)[NPL]) {
    constexpr int kBytes = NPL * (F32 ? 4 : 2);
    uint32_t w[(kBytes + 3) / 4];
    const char* p = static_cast<const char*>(a.logits) + (t * a.ld + e0) * (F32 ? 4 : 2);
    if constexpr (kBytes >= 16)
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
            *reinterpret_cast<uint4*>(w + 4 * i) = *reinterpret_cast<const uint4*>(p + 16 * i);
    else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
    else if constexpr (kBytes == 4) w[0] = *reinterpret_cast<const uint32_t*>(p);
    else w[0] = *reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        const float v = F32 ? __uint_as_float(w[j]) : j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
        l[j] = fmaxf(v, kNegInf);                         // -inf for NaN
    }
}

__device__ __forceinline__ float logit_at(const RouteLaunch& a, int64_t at) {
    return a.fp32 ? static_cast<const float*>(a.logits)[at]
                  : __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[at]);
}

template <int NPL>
__device__ __forceinline__ void load_logits(const RouteLaunch& a, int64_t t, int lane, float (&l)[NPL]) {
    const int e0 = lane * NPL;
#pragma unroll
    for (int j = 0; j < NPL; ++j) l[j] = kNegInf;
    if (a.vectors) {                                      // whole lanes, aligned
        if (e0 < a.E) {
            if (a.fp32) load_vectors<NPL, true>(a, t, e0, l);
            else        load_vectors<NPL, false>(a, t, e0, l);
        }
    } else {
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if (e0 + j < a.E) l[j] = fmaxf(logit_at(a, t * a.ld + e0 + j), kNegInf);
    }
}

// The biases of a lane's experts, -inf where they mask; whether any does.  In
// vectors: single loads with the lanes' stride cost a warp of few tokens a fifth
// of its time (16383 x 256, sigmoid with bias: 16.3 against 13.3 us).
template <int NPL>
__device__ __forceinline__ bool load_bias(const RouteLaunch& a, int lane, float (&b)[NPL]) {
    bool masks = false;
#pragma unroll
    for (int j = 0; j < NPL; ++j) b[j] = 0.0f;
    if (a.bias && NPL % 4 == 0 && a.bias_vectors) {
        if (lane * NPL < a.E)
#pragma unroll
            for (int j = 0; j + 3 < NPL; j += 4) {
                const float4 v = *reinterpret_cast<const float4*>(a.bias + lane * NPL + j);
                b[j] = v.x; b[j + 1] = v.y; b[j + 2] = v.z; b[j + 3] = v.w;
            }
    } else if (a.bias) {
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if (lane * NPL + j < a.E) b[j] = a.bias[lane * NPL + j];
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        b[j] = fmaxf(b[j], kNegInf);
        masks |= !(b[j] > kNegInf);
    }
    return __any_sync(kFull, masks);
}

// Largest value over the warp.
__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Makes `top` the group's score, the sum of its two largest where top2 is set,
// and returns the larger magnitude of its terms.
template <typename F>
__device__ __forceinline__ float group_sum(int top2, F& top, F second) {
    float size = fabsf((float)top);
    if (top2 && second > F(kNegInf)) {
        size = fmaxf(size, fabsf((float)second));
        top += second;
    }
    return size;
}

// Whether fp32 cannot tell the kept groups from those left behind: some lane's
// kept group comes within the errors of another's that is not.  A group's score
// is off by up to rel for each of its two scores of at most 1 and by 2^-24 of the
// terms for each of their roundings and of the sum's, so the error follows the
// terms, which can be far larger than a sum that cancels; twice that is allowed.
// A sum past the range of fp32 is no score (-inf would drop the group).
__device__ __forceinline__ bool groups_close(float score, float size, bool kept, float rel) {
    const float err = 2.0f * (2.0f * rel + 2.4e-7f * (1.0f + size));
    const float low = -redux_max(kept ? err - score : kNegInf);
    const float high = redux_max(!kept && score > kNegInf ? score + err : kNegInf);
    return low <= high || __any_sync(kFull, size < -kNegInf && !(fabsf(score) < -kNegInf));
}

// The choice for one token by one warp, a search round for each expert.
// F = float returns false when two scores that the choice compares lie within
// the error of their fp32 evaluation, or a chosen score is about to underflow;
// the caller then repeats it in double, so that the experts are those of the
// formula and not of its rounding.  Without a bias the scores' order is that
// of the logits, which needs no evaluation.
template <int NPL, typename F>
__device__ bool choose(const RouteLaunch& a, int64_t t, int lane, F* scratch) {
    constexpr bool kFp32 = sizeof(F) == 4;
    float l[NPL], b[NPL];
    load_logits(a, t, lane, l);
    load_bias(a, lane, b);
    F s[NPL], key[NPL];
#pragma unroll
    for (int j = 0; j < NPL; ++j)
        if (!(b[j] > kNegInf)) l[j] = kNegInf;
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
            const int e = lane * NPL + j;
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
        }
        const float size = group_sum(a.group_top2, top, second);
        const F own = top;
        uint32_t chosen = 0;
        for (int r = 0; r < a.topk_groups && r < a.groups; ++r) {
            F v = top;
            int g = lane;
            warp_argmax(v, g);
            if (!(v > F(kNegInf))) break;
            chosen |= 1u << g;
            if (lane == g) top = F(kNegInf);
        }
        if constexpr (kFp32) {
            if (by_score && groups_close(own, size, chosen >> lane & 1u, rel)) return false;
        }
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if (!(chosen >> ((lane * NPL + j) / gs & 31) & 1u)) key[j] = F(kNegInf);
    }

    int id = -1;
    F w = 0, prev = 0, prev_s = 0;
    const int rounds = kFp32 && scored ? a.k + 1 : a.k;         // one more to see the gap behind the last
    for (int r = 0; r < rounds; ++r) {
        F v = key[0];
        int e = lane * NPL;
#pragma unroll
        for (int j = 1; j < NPL; ++j)
            if (key[j] > v) { v = key[j]; e = lane * NPL + j; }
        warp_argmax(v, e);
        if (!(v > F(kNegInf))) break;
        F sv = 0;
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if (lane * NPL + j == e) { sv = s[j]; key[j] = F(kNegInf); }
        sv = __shfl_sync(kFull, sv, e / NPL);
        if (kFp32 && scored && r > 0 &&
            prev - v <= F(2.0f * rel * fmaxf((float)prev_s, (float)sv) + 2.4e-7f * (1.0f + fmaxf(fabsf((float)prev), fabsf((float)v)))))
            return false;
        prev = v;
        prev_s = sv;
        if (r < a.k && lane == r) { id = e; w = sv; }
    }
    if (a.renormalize) {
        const F sum = warp_sum(w);
        if (kFp32 && __any_sync(kFull, id >= 0 && w < F(1e-30f))) return false;
        w = sum > F(0) ? w / sum : F(0);
    }
    if (lane < a.k) {
        a.ids[t * a.k + lane] = id;
        a.weights[t * a.k + lane] = (float)(w * F(a.scale));
    }
    return true;
}

// Per-warp shared memory of the fast choice.
struct RouteScratch {
    double key[36];                      // floats in the fp32 form; padded to a multiple of four
    int expert[32];
};

__device__ __forceinline__ float fast_exp(float v) {           // ex2.approx: 2^-22 + |v| 2^-23 relative
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 1.4426950408889634f));
    return r;
}
__device__ __forceinline__ double fast_exp(double v) { return exp(v); }
__device__ __forceinline__ float quotient(float a, float b) { return __fdividef(a, b); }
__device__ __forceinline__ float reciprocal(float a) {        // rcp.approx: one ulp
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}
__device__ __forceinline__ double reciprocal(double a) { return 1.0 / a; }
__device__ __forceinline__ double quotient(double a, double b) { return a / b; }

// How many groups are better than this lane's group g with score `top`: larger,
// or as large with a lower index.
template <typename F>
__device__ __forceinline__ int group_rank(F top, int g, const RouteLaunch& a) {
    int rank = 0;
    for (int h = 0; h < a.groups; ++h) {
        const F v = __shfl_sync(kFull, top, h << a.group_shift);
        rank += v > top || (v == top && h < g);
    }
    return rank;
}

// Masks the keys outside the groups that a token may use; `of` holds what a
// group's score is made of.  Returns false when the last kept and the first
// dropped group are too close for fp32 (checked where scores are inexact).
// 1 << group_shift lanes share a group: where a group is a power-of-two
// number of whole lanes from their registers, else through shared memory,
// each lane reading every p-th of the group's experts.
template <int NPL, typename F>
__device__ __forceinline__ bool keep_groups(const F (&of)[NPL], F (&key)[NPL], const RouteLaunch& a, int lane,
                                            bool inexact, float rel, F* scratch) {
    F top = F(kNegInf), second = F(kNegInf);
    const int p = 1 << a.group_shift, g = lane >> a.group_shift;
    if (a.group_whole) {
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            second = larger(second, smaller(top, of[j]));
            top = larger(top, of[j]);
        }
    } else {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if (lane * NPL + j < a.E) scratch[lane * NPL + j] = of[j];
        __syncwarp();
        const int gs = a.group_size, sub = lane & (p - 1);
        if (g < a.groups) {
            const int n = (gs + p - 1) >> a.group_shift;
            int it = g % n;                               // rotated start: groups would share a bank
            for (int i = 0; i < n; ++i) {
                const int at = (it << a.group_shift) + sub;
                const F v = at < gs ? scratch[g * gs + at] : F(kNegInf);
                it = it + 1 == n ? 0 : it + 1;
                second = larger(second, smaller(top, v));
                top = larger(top, v);
            }
        }
    }
    for (int o = 1; o < p; o <<= 1) {
        const F t = __shfl_xor_sync(kFull, top, o), u = __shfl_xor_sync(kFull, second, o);
        second = larger(smaller(top, t), larger(second, u));
        top = larger(top, t);
    }
    const float size = group_sum(a.group_top2, top, second);
    if (g >= a.groups) top = F(kNegInf);
    // the groups not under the topk_groups-th largest score; where equal scores
    // make them too many, by rank with the lower index first
    const bool live = top > F(kNegInf);
    bool kept;
    if constexpr (sizeof(F) == 4) {
        float left = top, bound = kNegInf;
        for (int r = 0; r < a.topk_groups; ++r) {
            bound = redux_max(left);
            if (left == bound) left = kNegInf;
        }
        kept = live && top >= bound;
        if (inexact && groups_close(top, size, kept, rel)) return false;
        if (__popc(__ballot_sync(kFull, kept)) > a.topk_groups << a.group_shift) {
            if (inexact) return false;
            const int rank = group_rank(top, g, a);       // a warp step: outside any lane's condition
            kept = live && rank < a.topk_groups;
        }
    } else {
        const int rank = group_rank(top, g, a);
        kept = live && rank < a.topk_groups;
    }
    if (a.group_whole) {
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if (!kept) key[j] = F(kNegInf);
    } else {
        const uint32_t lanes = __ballot_sync(kFull, kept);
        const uint32_t recip = ((1u << 20) + a.group_size - 1) / a.group_size;      // e * recip >> 20 == e / size below 512
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            const uint32_t h = (uint32_t)(lane * NPL + j) * recip >> 20;
            if (!(lanes >> ((h << a.group_shift) & 31) & 1u)) key[j] = F(kNegInf);
        }
    }
    return true;
}

enum Choice { kChosen, kTooClose, kTooMany };

// Ranks of the gathered experts by score + bias in double: lane i < count has
// expert e.  Not inlined: few tokens need it, and its registers would cost the
// others theirs.
template <int NPL>
__device__ __noinline__ int exact_rank(const RouteLaunch* a, int64_t t, int lane, int count, int e, RouteScratch* sh) {
    double score = 0.0, m = 0.0, sum = 1.0;
    if (!a->sigmoid) {
        float l[NPL], b[NPL];
        load_logits(*a, t, lane, l);
        load_bias(*a, lane, b);
        float top = kNegInf;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            if (!(b[j] > kNegInf)) l[j] = kNegInf;
            top = fmaxf(top, l[j]);
        }
        m = redux_max(top);
        sum = 0.0;
        for (int j = 0; j < NPL; ++j) sum += exp((double)l[j] - m);
        sum = warp_sum(sum);
    }
    if (lane < count) {
        const double x = logit_at(*a, t * a->ld + e);
        score = (a->sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - m) / sum) + (double)a->bias[e];
    }
    __syncwarp();
    if (lane < count) sh->key[lane] = score;
    __syncwarp();
    int rank = 0;
    for (int i = 0; i < count; ++i) rank += sh->key[i] > score || (sh->key[i] == score && i < lane);
    __syncwarp();
    return rank;
}

// The choice without a search round for each expert.  The k-th largest of the
// 32 lane maxima bounds the k-th largest key from below, so the few keys not
// under it are gathered, in expert order, and ranked against one another.
// What a token costs is instructions, not memory (issue slots 71 % busy, DRAM 9 %):
// 16383 tokens of 256 experts, sigmoid with bias, took 13.8 M warp instructions
// and 30 us with search rounds, and take 12.6 us so.  F = float ranks close
// candidates in double, and leaves close groups and scores about to underflow to
// F = double (kTooClose), which gathers on its keys rounded to fp32, an
// order-preserving step, and ranks the keys themselves.  Nothing is written
// unless kChosen is returned.
template <int NPL, bool SCORED, bool GROUPS, typename F>
__device__ __forceinline__ Choice choose_fast(const RouteLaunch& a, int64_t t, int lane, const float (&b)[NPL],
                                              bool bias_masks, F* scratch, RouteScratch& sh) {
    constexpr bool kFp32 = sizeof(F) == 4;
    constexpr bool scored = SCORED;                                      // a bias: keys are not the logits
    const bool need_all = SCORED || (GROUPS && a.group_top2);            // every score, not just the chosen ones'
    const float rel = a.sigmoid ? 4.8e-7f : 1.9e-6f;                     // see choose(); the fast exponential is within both
    F key[NPL];
    F m = 0, r = 1;
    {
        float l[NPL];
        load_logits(a, t, lane, l);
        if (SCORED && bias_masks)
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (!(b[j] > kNegInf)) l[j] = kNegInf;
        if (!a.sigmoid && (need_all || !a.renormalize)) {
            float top = l[0];
#pragma unroll
            for (int j = 1; j < NPL; ++j) top = fmaxf(top, l[j]);
            top = redux_max(top);
            m = top > kNegInf ? top : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < NPL; ++j) key[j] = l[j];
    }
    if (need_all) {
        F s[NPL];
        if (a.sigmoid) {
#pragma unroll
            for (int j = 0; j < NPL; ++j) s[j] = reciprocal(F(1) + fast_exp(-key[j]));
        } else {
            F sum = 0;
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                s[j] = fast_exp(key[j] - m);
                sum += s[j];
            }
            sum = warp_sum(sum);
            r = sum > F(0) ? quotient(F(1), sum) : F(0);
#pragma unroll
            for (int j = 0; j < NPL; ++j) s[j] *= r;
        }
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            s[j] = key[j] > F(kNegInf) ? (SCORED ? s[j] + F(b[j]) : s[j]) : F(kNegInf);
            if (scored) key[j] = s[j];
        }
        if (GROUPS && !keep_groups(s, key, a, lane, true, rel, scratch)) return kTooClose;
    } else {
        if (!a.sigmoid && !a.renormalize) {
            F sum = 0;
#pragma unroll
            for (int j = 0; j < NPL; ++j) sum += exp_of(key[j] - m);     // 0 where masked
            sum = warp_sum(sum);
            r = sum > F(0) ? quotient(F(1), sum) : F(0);
        }
        if (GROUPS) keep_groups(key, key, a, lane, false, rel, scratch);
    }

    // the bound: one more than k where the gap behind the last choice counts
    float top = (float)key[0];
#pragma unroll
    for (int j = 1; j < NPL; ++j) top = fmaxf(top, (float)key[j]);
    float bound = kNegInf;
    const int rounds = scored ? a.k + 1 : a.k;
#pragma unroll 2
    for (int i = 0; i < rounds; ++i) {
        bound = redux_max(top);
        if (top == bound) top = kNegInf;                  // lanes with equal maxima go together: a lower bound still
    }
    // keys that fp32 may have put on the wrong side of the bound are gathered too
    const float slack = kFp32 && scored ? 2.0f * rel + 2.4e-7f * (1.0f + fabsf(bound)) : 0.0f;
    bound = fmaxf(bound - slack, -3.4028235e38f);         // masked keys stay out
    int n = 0;
#pragma unroll
    for (int j = 0; j < NPL; ++j) n += (float)key[j] >= bound;
    // the lanes' counts summed a binary digit at a time: ballots, no chain of
    // shuffles
    int at = 0, count = 0;
#pragma unroll
    for (int o = 0; 1 << o <= NPL; ++o) {
        const uint32_t has = __ballot_sync(kFull, n >> o & 1);
        at += __popc(has & ((1u << lane) - 1u)) << o;
        count += __popc(has) << o;
    }
    if (count > 32) return kTooMany;
    F* gathered = reinterpret_cast<F*>(sh.key);
    __syncwarp();                                         // the previous token's reads are done
    if (n) {
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if ((float)key[j] >= bound) {
                gathered[at] = key[j];
                sh.expert[at] = lane * NPL + j;
                ++at;
            }
    }
    if (lane < 4) gathered[count + lane] = F(kNegInf);
    __syncwarp();
    const bool mine = lane < count;
    const F v = mine ? gathered[lane] : F(kNegInf);
    const int e = mine ? sh.expert[lane] : 0;
    int rank = 0;
    if constexpr (kFp32) {
        for (int i = 0; i < count; i += 4) {
            const float4 w = *reinterpret_cast<const float4*>(gathered + i);
            rank += (w.x > v) + (w.y > v) + (w.z > v) + (w.w > v);
        }
        // equal keys (both zeros alike): the lower index first
        rank += __popc(__match_any_sync(kFull, __float_as_uint(v + 0.0f)) & ((1u << lane) - 1u));
        if (scored) {
            // neighbours in rank order; a score is at most 1
            __syncwarp();
            if (mine) gathered[rank] = v;
            __syncwarp();
            bool close = false;
            if (lane < a.k && lane + 1 < count) {
                const float p = (float)gathered[lane], q = (float)gathered[lane + 1];
                close = p - q <= 2.0f * rel + 2.4e-7f * (1.0f + fmaxf(fabsf(p), fabsf(q)));
            }
            if (__any_sync(kFull, close)) rank = exact_rank<NPL>(&a, t, lane, count, e, &sh);
        }
    } else {
        for (int i = 0; i < count; ++i) rank += gathered[i] > v || (gathered[i] == v && i < lane);
    }
    const bool chosen = mine && rank < a.k;
    F x = v;
    if (scored && mine) x = logit_at(a, t * a.ld + e);
    F score;
    if (a.sigmoid) {
        score = quotient(F(1), F(1) + exp_of(-x));
    } else {
        // the sum over all experts cancels where weights are renormalised
        F c = m;
        if (a.renormalize) {
            c = F(redux_max(chosen ? (float)x : kNegInf));
            if (kFp32 && need_all && c - m < F(-80)) return kTooClose;
            if (!kFp32 && need_all && exp_of(c - m) == F(0)) r = 0;      // every chosen score is 0
        }
        score = exp_of(x - c) * (!a.renormalize || r == F(0) ? r : F(1));
    }
    F w = chosen ? score : F(0);
    if (a.renormalize) {
        const F sum = warp_sum(w);
        if (kFp32 && a.sigmoid && __any_sync(kFull, chosen && w < F(1e-30f))) return kTooClose;
        w = sum > F(0) ? quotient(w, sum) : F(0);
    }
    const int64_t to = t * a.k;
    if (chosen) {
        a.ids[to + rank] = e;
        a.weights[to + rank] = (float)(w * F(a.scale));
    }
    if (lane >= count && lane < a.k) {
        a.ids[to + lane] = -1;
        a.weights[to + lane] = 0.0f;
    }
    return kChosen;
}

// What the fp32 form leaves undecided.  Not inlined: its registers (the scores
// in double) would halve the resident warps of the fp32 form.
template <int NPL, bool SCORED, bool GROUPS>
__device__ __noinline__ void choose_slow(const RouteLaunch* a, int64_t t, int lane, Choice why, double* scratch,
                                         RouteScratch* sh) {
    if (why == kTooClose) {
        float b[NPL];
        const bool masks = load_bias(*a, lane, b);
        why = choose_fast<NPL, SCORED, GROUPS>(*a, t, lane, b, masks, scratch, *sh);
    }
    if (why == kTooMany && !choose<NPL>(*a, t, lane, reinterpret_cast<float*>(scratch))) choose<NPL>(*a, t, lane, scratch);
}

// One warp routes token t.  scratch: E doubles of this warp.
template <int NPL, bool SCORED, bool GROUPS>
__device__ __forceinline__ void route_token(const RouteLaunch& a, int64_t t, int lane, const float (&b)[NPL],
                                            bool bias_masks, double* scratch, RouteScratch& sh) {
    const Choice c = choose_fast<NPL, SCORED, GROUPS>(a, t, lane, b, bias_masks, reinterpret_cast<float*>(scratch), sh);
    if (c != kChosen) choose_slow<NPL, SCORED, GROUPS>(&a, t, lane, c, scratch, &sh);
}

// One warp a token, a warp walking several.
template <int NPL, bool SCORED, bool GROUPS>
__global__ void __launch_bounds__(kRouteWarps * 32, NPL <= 8 ? 4 : 2)
route_kernel(const __grid_constant__ RouteLaunch a) {
    extern __shared__ double route_smem[];
    __shared__ alignas(16) RouteScratch sh[kRouteWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float b[NPL];
    chain_begin();
    const bool masks = load_bias(a, lane, b);
    for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < a.T; t += (int64_t)gridDim.x * kRouteWarps)
        route_token<NPL, SCORED, GROUPS>(a, t, lane, b, masks, route_smem + warp * a.E, sh[warp]);
}

// ---------------------------------------------------------- dispatch ------
// Stable counting sort of the n = T * k choices by expert, in one cluster:
// every warp owns a run of consecutive choices and a histogram row in shared
// memory; the rows are scanned over the block's warps, the block totals over
// the cluster (distributed shared memory) and the experts, and a second walk
// over the same run places each choice.  Equal ids inside a group of 32 are
// ranked by ballots, so the order is fixed; no workspace.
constexpr int kDispWarps = 32;
constexpr int kBatch = 8;            // groups of 32 choices whose loads are in flight together
constexpr int kHeld = 2;             // groups of a run short enough to stay in registers

// ids[first + 32 b + lane], -1 where there is none or no such expert
template <int B>
__device__ __forceinline__ void load_batch(const DispatchLaunch& a, int64_t at, int64_t end, int lane, int (&e)[B]) {
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const int64_t i = at + b * 32 + lane;
        e[b] = i < end ? a.ids[i] : -1;
    }
#pragma unroll
    for (int b = 0; b < B; ++b)
        if ((unsigned)e[b] >= (unsigned)a.E) e[b] = -1;
}

// Lanes that hold the same expert (any set for e < 0).  One ballot a bit of
// the expert: the warp match instruction takes a step for each distinct value,
// and here nearly all are.
__device__ __forceinline__ unsigned same_expert(int e, int bits) {
    unsigned peers = kFull;
    for (int b = 0; b < bits; ++b) {
        const bool set = e >> b & 1;
        const unsigned with = __ballot_sync(kFull, set);
        peers &= set ? with : ~with;
    }
    return peers & __ballot_sync(kFull, e >= 0);
}

// Exclusive scan of v over the block's 1024 threads; sum: the total.
__device__ __forceinline__ int block_scan(int v, int* wsum, int& sum) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += u;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int w = wsum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, w, o);
        if (lane >= o) w += u;
    }
    sum = __shfl_sync(kFull, w, 31);
    const int before = warp ? __shfl_sync(kFull, w, warp - 1) : 0;
    return before + inc - v;
}

template <int C>
__device__ __forceinline__ void dispatch_body(const DispatchLaunch& a, int* smem, int* wsum) {
    int* hist = smem;                             // [kDispWarps][E]
    int* total = hist + kDispWarps * a.E;         // [E] this block's counts
    int* start = total + a.E;                     // [E] first slot of this block's rows
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = C > 1 ? (int)cluster_ctarank() : 0;
    const int64_t per = (a.n + (int64_t)C * kDispWarps * 32 - 1) / ((int64_t)C * kDispWarps * 32) * 32;
    const int64_t first = ((int64_t)rank * kDispWarps + warp) * per;
    const int64_t end = first + per < a.n ? first + per : a.n;
    int* mine = hist + warp * a.E;
    const int bits = 32 - __clz(a.E - 1);          // 0 for one expert

    for (int i = threadIdx.x; i < kDispWarps * a.E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    // a short run is ranked as it is counted and stays in registers; a longer
    // one is counted now and walked again, its ranks under its stores (131064
    // choices: 11.6 against 14.9 us held, 2048: 3.2 against 3.0)
    const bool once = per <= kHeld * 32;
    int held[kHeld], local[kHeld];
    if (once) {
        load_batch(a, first, end, lane, held);
#pragma unroll
        for (int b = 0; b < kHeld; ++b) {
            if (first + b * 32 >= end) break;
            const unsigned peers = same_expert(held[b], bits);
            if (held[b] >= 0) local[b] = mine[held[b]] + __popc(peers & ((1u << lane) - 1u));
            __syncwarp();
            if (held[b] >= 0 && lane == __ffs(peers) - 1) mine[held[b]] += __popc(peers);
            __syncwarp();
        }
    } else {
        for (int64_t at = first; at < end; at += kBatch * 32) {
            int e[kBatch];
            load_batch(a, at, end, lane, e);
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
                if (e[b] >= 0) atomicAdd(&mine[e[b]], 1);     // counts only: their order does not matter
        }
    }
    __syncthreads();
    // exclusive scan of each expert's counts over the block's warps
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int sum = 0;
#pragma unroll 8
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
    const int x = threadIdx.x;
    if (x < a.E) {
#pragma unroll
        for (int r = 0; r < C; ++r) {
            const int v = C > 1 ? __float_as_int(ld_shared_cluster_f32(&total[x], r)) : total[x];
            if (r < rank) before += v;
            all += v;
        }
    }
    int live;
    const int base = block_scan(all, wsum, live);
    if (x < a.E) {
        start[x] = base + before;
        if (rank == 0) a.offsets[x] = base;
    }
    if (rank == 0 && threadIdx.x == 0) a.offsets[a.E] = live;
    __syncthreads();
    auto place = [&](int64_t i, int slot) {
        if (i < end) {
            a.position[i] = slot;
            if (slot >= 0) a.row_index[slot] = (int)((uint32_t)i / (uint32_t)a.k);
        }
    };
    if (once) {
#pragma unroll
        for (int b = 0; b < kHeld; ++b) {
            if (first + b * 32 >= end) break;
            place(first + b * 32 + lane, held[b] >= 0 ? start[held[b]] + mine[held[b]] + local[b] : -1);
        }
    } else {
        for (int64_t at = first; at < end; at += kBatch * 32) {
            int e[kBatch];
            load_batch(a, at, end, lane, e);
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (at + b * 32 >= end) break;
                const unsigned peers = same_expert(e[b], bits);
                int slot = -1;
                if (e[b] >= 0) slot = start[e[b]] + mine[e[b]] + __popc(peers & ((1u << lane) - 1u));
                __syncwarp();
                if (e[b] >= 0 && lane == __ffs(peers) - 1) mine[e[b]] += __popc(peers);
                __syncwarp();
                place(at + b * 32 + lane, slot);
            }
        }
    }
    // slots behind the last live one name row 0: valid rows of no expert
    for (int64_t i = live + rank * blockDim.x + threadIdx.x; i < a.n; i += C * blockDim.x) a.row_index[i] = 0;
    if (C > 1) cluster_sync_all();                // no block leaves while its totals are read
}

template <int C>
__global__ void __launch_bounds__(kDispWarps * 32)
dispatch_kernel(const DispatchLaunch a) {
    extern __shared__ int disp_smem[];
    __shared__ int wsum[32];
    chain_begin();
    dispatch_body<C>(a, disp_smem, wsum);
}

// Few tokens: the choice and the dispatch order by one block, in one launch
// (against two: 16 x 128, top 8: 4.0 against 4.2 us, 32 tokens 4.7 against 4.3;
// 256 experts with bias and groups, 8 tokens 5.7 against 5.6, 32 7.4 against 5.8;
// outside a captured graph the second launch also costs the host its time).
constexpr int kFusedTokens = 16;

template <int NPL, bool SCORED, bool GROUPS>
__global__ void __launch_bounds__(kDispWarps * 32)
route_dispatch_kernel(const __grid_constant__ RouteLaunch r, const DispatchLaunch d) {
    extern __shared__ double route_smem[];
    __shared__ alignas(16) RouteScratch sh[kDispWarps];
    __shared__ int wsum[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float b[NPL];
    chain_begin();
    const bool masks = load_bias(r, lane, b);
    for (int64_t t = warp; t < r.T; t += kDispWarps)
        route_token<NPL, SCORED, GROUPS>(r, t, lane, b, masks, route_smem + warp * r.E, sh[warp]);
    __syncthreads();                              // the block's own ids, written to global memory, are read back
    dispatch_body<1>(d, reinterpret_cast<int*>(route_smem), wsum);
}

template <class Fn>
cudaError_t allow_smem(std::atomic<bool> (&done)[64], Fn kernel, size_t bytes, bool wide_cluster = false) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && wide_cluster)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && dev < 64) done[dev].store(true, std::memory_order_release);
    return e;
}

constexpr size_t dispatch_smem(int E) { return (size_t)(kDispWarps + 2) * E * sizeof(int); }

template <int C>
cudaError_t launch_dispatch_c(const DispatchLaunch& p, cudaStream_t s) {
    static std::atomic<bool> done[64];
    if (cudaError_t e = allow_smem(done, dispatch_kernel<C>, dispatch_smem(kMaxRouteExperts), C > 8); e != cudaSuccess)
        return e;
    return launch_chained(dispatch_kernel<C>, dim3(C), kDispWarps * 32, dispatch_smem(p.E), s, C, p);
}

template <int NPL, bool SCORED, bool GROUPS>
cudaError_t launch_route_v(const RouteLaunch& p, const DispatchLaunch* order, cudaStream_t s, int sms) {
    if (order && p.T <= kFusedTokens) {
        // scratch of 32 warps and, later, the histograms
        const size_t smem = std::max((size_t)kDispWarps * p.E * sizeof(double), dispatch_smem(p.E));
        static std::atomic<bool> done[64];
        if (cudaError_t e = allow_smem(done, route_dispatch_kernel<NPL, SCORED, GROUPS>,
                                       (size_t)kDispWarps * kMaxRouteExperts * sizeof(double));
            e != cudaSuccess)
            return e;
        return launch_chained(route_dispatch_kernel<NPL, SCORED, GROUPS>, dim3(1), kDispWarps * 32, smem, s, 1, p, *order);
    }
    const int64_t blocks = std::min<int64_t>((p.T + kRouteWarps - 1) / kRouteWarps, (int64_t)sms * 8);
    const size_t smem = p.groups > 1 ? (size_t)kRouteWarps * p.E * sizeof(double) : 0;
    if (cudaError_t e = launch_chained(route_kernel<NPL, SCORED, GROUPS>, dim3((unsigned)blocks), kRouteWarps * 32, smem, s, 1, p);
        e != cudaSuccess)
        return e;
    return order ? launch_dispatch(*order, s) : cudaSuccess;
}

template <int NPL>
cudaError_t launch_route_n(const RouteLaunch& given, const DispatchLaunch* order, cudaStream_t s, int sms) {
    RouteLaunch p = given;
    p.group_size = p.E / p.groups;
    const int lanes = p.group_size / NPL;
    p.group_whole = p.group_size % NPL == 0 && (lanes & (lanes - 1)) == 0;
    const int most = p.group_whole ? lanes : 32 / p.groups;
    while ((2 << p.group_shift) <= most) ++p.group_shift;
    // whole lanes of experts, every lane's first on a boundary of its vector
    const int size = p.fp32 ? 4 : 2, align = std::min(16, NPL * size);
    p.vectors = p.E % NPL == 0 && p.ld * size % align == 0 && reinterpret_cast<uintptr_t>(p.logits) % align == 0;
    p.bias_vectors = p.E % NPL == 0 && reinterpret_cast<uintptr_t>(p.bias) % 16 == 0;
    if (p.bias) return p.groups > 1 ? launch_route_v<NPL, true, true>(p, order, s, sms) : launch_route_v<NPL, true, false>(p, order, s, sms);
    return p.groups > 1 ? launch_route_v<NPL, false, true>(p, order, s, sms) : launch_route_v<NPL, false, false>(p, order, s, sms);
}

// ----------------------------------------------------------- combine ------
// out[t] = residual[t] + sum_j weights[t, j] * Y[position[t, j]], fp32, j
// ascending, the residual last, one rounding.  A thread owns 8 columns of one
// token and issues the loads of J experts' rows before it uses the first:
// bound by memory.
__device__ __forceinline__ void widen(const uint4& w, float (&v)[8]) {
    v[0] = bf16_lo(w.x); v[1] = bf16_hi(w.x); v[2] = bf16_lo(w.y); v[3] = bf16_hi(w.y);
    v[4] = bf16_lo(w.z); v[5] = bf16_hi(w.z); v[6] = bf16_lo(w.w); v[7] = bf16_hi(w.w);
}
__device__ __forceinline__ void widen(const float4 (&w)[2], float (&v)[8]) {
    v[0] = w[0].x; v[1] = w[0].y; v[2] = w[0].z; v[3] = w[0].w;
    v[4] = w[1].x; v[5] = w[1].y; v[6] = w[1].z; v[7] = w[1].w;
}

template <bool F32> struct Raw8 { uint4 w; };
template <> struct Raw8<true> { float4 w[2]; };

// CONST: through the read-only path (memory that the kernel does not write).
template <bool F32, bool CONST = true>
__device__ __forceinline__ Raw8<F32> load_raw(const void* p, int64_t at) {
    Raw8<F32> r;
    if constexpr (F32) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        r.w[0] = CONST ? __ldg(q) : q[0];
        r.w[1] = CONST ? __ldg(q + 1) : q[1];
    } else {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
        r.w = CONST ? __ldg(q) : *q;
    }
    return r;
}

template <bool YF32, bool OF32, int J>
__global__ void __launch_bounds__(256, J < 8 ? 0 : YF32 ? 2 : 4)
combine_kernel(const CombineLaunch a) {
    const int64_t t = blockIdx.x;
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * 8;
    chain_begin();
    if (c >= a.N) return;
    float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const int32_t* position = a.position + t * a.k;
    const float* weights = a.weights + t * a.k;
    // the residual loads under the experts' rows
    Raw8<OF32> res;
    if (a.residual) res = load_raw<OF32, false>(a.residual, t * a.N + c);
    for (int j0 = 0; j0 < a.k; j0 += J) {
        Raw8<YF32> v[J];
        bool in[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t at = j0 + j < a.k ? position[j0 + j] : -1;
            in[j] = at >= 0 && at < a.rows;
            if (in[j]) v[j] = load_raw<YF32>(a.Y, at * a.N + c);
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (!in[j]) continue;                        // uniform over the block
            const float w = weights[j0 + j];
            float x[8];
            widen(v[j].w, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = fmaf(w, x[i], sum[i]);
        }
    }
    if (a.residual) {
        float r[8];
        widen(res.w, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += r[i];
    }
    store8<OF32>(a.out, t * a.N + c, sum);
}

template <bool YF32, bool OF32>
cudaError_t launch_combine_t(const CombineLaunch& p, cudaStream_t s) {
    const int chunks = p.N / 8;
    // small blocks: a token's last loads hold back few others (4096 x 8 x 2048:
    // 31.4 us with 64 threads, 31.9 with 128; 8192 x 2 x 5120: 54.8 against
    // 58.2 with 256)
    const int threads = std::min(64, (chunks + 31) / 32 * 32);
    const dim3 grid((unsigned)p.T, (unsigned)((chunks + threads - 1) / threads));
    if (p.k <= 2) return launch_chained(combine_kernel<YF32, OF32, 2>, grid, threads, 0, s, 1, p);
    if (p.k <= 4) return launch_chained(combine_kernel<YF32, OF32, 4>, grid, threads, 0, s, 1, p);
    return launch_chained(combine_kernel<YF32, OF32, 8>, grid, threads, 0, s, 1, p);
}

}  // namespace

cudaError_t launch_route(const RouteLaunch& p, const DispatchLaunch* order, cudaStream_t s, int sms) {
    if (p.T == 0) return order ? launch_dispatch(*order, s) : cudaSuccess;
    if (p.E <= 32) return launch_route_n<1>(p, order, s, sms);
    if (p.E <= 64) return launch_route_n<2>(p, order, s, sms);
    if (p.E <= 128) return launch_route_n<4>(p, order, s, sms);
    if (p.E <= 256) return launch_route_n<8>(p, order, s, sms);
    return launch_route_n<16>(p, order, s, sms);
}

namespace {
// Whether the device places a cluster of 16 blocks of the dispatch kernel at
// its largest (16 is beyond the portable size).
bool wide_cluster_fits() {
    static std::atomic<int> known[64];                    // 0 not asked, 1 no, 2 yes
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64)
        if (const int k = known[dev].load(std::memory_order_relaxed)) return k == 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(kDispWarps * 32);
    cfg.dynamicSmemBytes = dispatch_smem(kMaxRouteExperts);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    const bool fits = cudaFuncSetAttribute(dispatch_kernel<16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)cfg.dynamicSmemBytes) == cudaSuccess &&
                      cudaFuncSetAttribute(dispatch_kernel<16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                      cudaOccupancyMaxActiveClusters(&n, dispatch_kernel<16>, &cfg) == cudaSuccess && n > 0;
    if (!fits) cudaGetLastError();
    if (dev < 64) known[dev].store(fits ? 2 : 1, std::memory_order_relaxed);
    return fits;
}
}  // namespace

cudaError_t launch_dispatch(const DispatchLaunch& p, cudaStream_t s) {
    // one block covers up to 2 choices a thread; beyond that a cluster does, of
    // 16 blocks where the device places one (32768 choices: 6.5 us against 7.8
    // with 8, 4800: 5.5 against 5.2; 4096 with one block 6.4)
    if (p.n <= 2048) return launch_dispatch_c<1>(p, s);
    return p.n > 8192 && wide_cluster_fits() ? launch_dispatch_c<16>(p, s) : launch_dispatch_c<8>(p, s);
}

cudaError_t launch_combine(const CombineLaunch& p, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    if (p.y_fp32) return p.out_fp32 ? launch_combine_t<true, true>(p, s) : launch_combine_t<true, false>(p, s);
    return p.out_fp32 ? launch_combine_t<false, true>(p, s) : launch_combine_t<false, false>(p, s);
}

}  // namespace sharq
