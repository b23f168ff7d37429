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

// The logit of a key (+0 for a zero of either sign).
__device__ __forceinline__ float logit_of_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// The top k experts of one token by one warp: lane s < k ends with the s-th expert's id and its softmax
// weight over the k selected logits. Each lane keeps its best remaining expert (largest key, lower
// expert on ties); a round takes the warp's largest key and the lowest expert that holds it (two
// redux.sync), so ties go to the lower expert index, and only the winner's lane searches its next best.
template <int kPerLane>
__device__ __forceinline__ void topk_lanes(const float *row, int E, int k, int &my_id, float &my_w)
{
    const int lane = threadIdx.x & 31;
    uint32_t key[kPerLane];
    uint32_t left = 0;                        // bit i: candidate lane + 32 i remains
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const int e = lane + 32 * i;
        const bool in = e < E;
        key[i] = in ? logit_key(__ldcg(row + e)) : 0u;
        left |= in ? 1u << i : 0u;
    }
    uint32_t best_key = 0u, best_id = 0xffffffffu;
    auto search = [&]() {
        best_key = 0u;
        best_id = 0xffffffffu;
#pragma unroll
        for (int i = kPerLane - 1; i >= 0; --i)           // downwards: the lower expert keeps ties
            if ((left & (1u << i)) && key[i] >= best_key) {
                best_key = key[i];
                best_id = (uint32_t)(lane + 32 * i);
            }
    };
    search();
    uint32_t first = 0u, mine = 0u;
    my_id = -1;
    for (int s = 0; s < k; ++s) {
        const uint32_t mk = __reduce_max_sync(0xffffffffu, best_key);
        const uint32_t win = __reduce_min_sync(0xffffffffu, best_key == mk ? best_id : 0xffffffffu);
        if (s == 0) first = mk;
        if (lane == s) { mine = mk; my_id = (int)win; }
        if (best_id == win) {
            left &= ~(1u << (win >> 5));
            search();
        }
    }
    const float ex = (lane < k) ? expf(logit_of_key(mine) - logit_of_key(first)) : 0.f;
    float den = ex;
    for (int o = k <= 8 ? 4 : 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);   // lanes from k on hold 0
    my_w = ex / den;
}
__device__ __forceinline__ void topk_select(const float *row, int E, int k, int &my_id, float &my_w) {
    if (E <= 128) topk_lanes<4>(row, E, k, my_id, my_w);
    else topk_lanes<kMaxEPerLane>(row, E, k, my_id, my_w);
}

// As topk_select, into the token's rows of ids and weights. With m shared slots the rows continue with
// slots k..k+m-1 = experts E..E+m-1 at weight 1 (the shared expert).
__device__ __forceinline__ void topk_warp(const float *row, int E, int k, int32_t *ids_row, float *w_row,
                                          int32_t *ids_copy = nullptr, int m = 0)
{
    const int lane = threadIdx.x & 31;
    int id;
    float w;
    topk_select(row, E, k, id, w);
    if (lane >= k) { id = E + lane - k; w = 1.f; }
    if (lane < k + m) {
        ids_row[lane] = id;
        w_row[lane] = w;
        if (ids_copy) ids_copy[lane] = id;
    }
}

}  // namespace tfmoe
