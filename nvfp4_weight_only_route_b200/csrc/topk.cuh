// topk.cuh -- top-k experts and softmax weights of one token's router logits, by one warp.
#pragma once

#include "common.cuh"

namespace tfmoe {

// One warp per token: k rounds of a warp arg-max over (logit desc, index asc),
// then softmax over the selected logits (max-subtracted, fp32).
constexpr int kMaxEPerLane = 8;   // E <= 256

// Order-preserving key of a finite fp32 logit: a larger logit has a larger key, and -0
// counts as +0 (equal logits tie). No finite logit maps to key 0.
__device__ __forceinline__ uint32_t logit_key(float v) {
    uint32_t b = __float_as_uint(v);
    if ((b << 1) == 0u) b = 0u;
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// One warp selects a token's top k experts: k rounds, each a lane-local best (largest key,
// lowest expert on ties) followed by a warp-wide max of the keys and a min of the expert ids
// that hold it (two redux.sync), so ties go to the lower expert index. With m shared slots the
// row continues with slots k..k+m-1 = experts E..E+m-1 at weight 1 (the shared expert).
__device__ __forceinline__ void topk_warp(const float *row, int E, int k, int32_t *ids_row, float *w_row,
                                          int32_t *ids_copy = nullptr, int m = 0)
{
    const int lane = threadIdx.x & 31;
    float v[kMaxEPerLane];
    uint32_t key[kMaxEPerLane];
    uint32_t taken = 0;                       // bit i: candidate lane + 32 i used or absent
#pragma unroll
    for (int i = 0; i < kMaxEPerLane; ++i) {
        const int e = lane + 32 * i;
        v[i] = (e < E) ? __ldcg(row + e) : 0.f;
        key[i] = logit_key(v[i]);
        if (e >= E) taken |= 1u << i;
    }
    float sel_first = 0.f, my_sel = 0.f;
    int my_id = -1;
    for (int s = 0; s < k; ++s) {
        uint32_t bk = 0u;
        float bv = 0.f;
#pragma unroll
        for (int i = 0; i < kMaxEPerLane; ++i) {
            if (!(taken & (1u << i)) && key[i] > bk) {   // strict: the lower i (lower expert) keeps ties
                bk = key[i];
                bv = v[i];
            }
        }
        const uint32_t mk = __reduce_max_sync(0xffffffffu, bk);
        uint32_t mine = 0xffffffffu;
#pragma unroll
        for (int i = kMaxEPerLane - 1; i >= 0; --i)
            if (!(taken & (1u << i)) && key[i] == mk) mine = (uint32_t)(lane + 32 * i);
        const uint32_t win = __reduce_min_sync(0xffffffffu, mine);
        const float wv = __shfl_sync(0xffffffffu, bv, (int)(win & 31u));
        if ((int)(win & 31u) == lane) taken |= 1u << (win >> 5);
        if (s == 0) sel_first = wv;
        if (lane == s) { my_sel = wv; my_id = (int)win; }
    }
    const float ex = (lane < k) ? expf(my_sel - sel_first) : 0.f;
    float den = ex;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (lane < k) {
        ids_row[lane] = my_id;
        w_row[lane] = ex / den;
        if (ids_copy) ids_copy[lane] = my_id;
    } else if (lane < k + m) {
        ids_row[lane] = E + lane - k;
        w_row[lane] = 1.f;
        if (ids_copy) ids_copy[lane] = E + lane - k;
    }
}

}  // namespace tfmoe
