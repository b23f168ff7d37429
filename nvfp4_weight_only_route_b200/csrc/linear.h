// linear.h -- the handle and the launchers of the NVFP4 matrix product (tfmoe_linear_*).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace tfmoe {

// What the epilogue of one output needs. Weight rows are those of the tiled matrix: with a
// gated activation row 2j is gate row j and row 2j+1 up row j, so N outputs have 2N rows.
struct LinearEpilogue {
    const float *global0, *global1;   // [1] per-tensor multipliers (gate, up when gated)
    const float *bias;                // [N], gated [2N]; NULL = none
    const uint16_t *residual;         // bf16 or NULL
    int64_t ldr;
    void *out;
    int64_t ldo;
    int N;
    int act;                          // tfmoe_activation
    int out_fp32;
};

struct Linear {
    tfmoe_linear_desc desc{};
    int device = 0;
    int num_sms = 0;
    bool loaded = false;
    int rows = 0;                     // weight rows: N, or 2N when gated
    int RT = 0, KT = 0;               // row tiles of 128, column tiles of 64 (zero filled)
    void *w_block = nullptr;
    void *ws_block = nullptr;
    uint8_t *codes = nullptr;         // [RT][KT] tiles of kTileCodeBytes, words in the order 0 2 4 6 1 3 5 7
    uint8_t *scales = nullptr;        // [RT][KT] slabs of kTileScaleBytes
    float *global = nullptr;          // [2]
    float *bias = nullptr;            // [rows]
    int32_t *err_word = nullptr;
    int32_t *tickets = nullptr;       // arrivals per row tile (streaming) or split tile, 0 between calls
    size_t zero_bytes = 0;            // err_word and tickets, at the start of the workspace
    float *partial = nullptr;         // sums of cut row tiles
    int32_t last_launches = 0;
    bool test_timeout = false;        // the next forward takes the timeout path (a test aid)
};

constexpr uint32_t kLinearTestWaitNs = 1000000;

inline bool linear_gated(const Linear &L) { return L.desc.activation == TFMOE_ACT_SWIGLU; }

cudaError_t launch_linear_repack(const Linear &L, const tfmoe_linear_weights &w, cudaStream_t s);
bool linear_stream_fits(const Linear &L, int T);
// Estimated times in clocks, for the choice between the two where both can.
double linear_stream_clocks(const Linear &L, int T), linear_tc_clocks(const Linear &L, int T);
cudaError_t linear_stream_setup(const Linear &L);
size_t linear_stream_partial_floats(const Linear &L);
cudaError_t launch_linear_stream(Linear &L, const uint16_t *x, int64_t ldx, int T, const LinearEpilogue &ep,
                                 cudaStream_t s, int *launches);
cudaError_t linear_tc_setup(const Linear &L);
size_t linear_tc_partial_floats(const Linear &L);
cudaError_t launch_linear_tc(Linear &L, const uint16_t *x, int64_t ldx, int T, const LinearEpilogue &ep,
                             cudaStream_t s, int *launches);

// GELU: y Phi(y). 1 + erf cancels for negative y (4 % off at y = -5, zero from -5.6 on), so the tail is computed
// by itself: for v = |y|, Phi(-v) = e^{-v^2/2} t q(1 - t) with t = 1 / (1 + c v), where t q is half the scaled
// complementary error function, smooth in t. q is a polynomial fitted by reweighted least squares over v <= 14.6
// (below -14.5 the tail is under the smallest fp32): of degree 9 and c = 25/64 to 2^-26.9; with Fast, for outputs
// that are rounded to bf16, of degree 5 and c = 29/64 to 2^-16.9, and with the one-instruction exponential of a
// rounded v^2. (4096 x 2048 x 8192 with bf16 out: Fast 132 us, without it 137, CUDA's erfcf 154, the cancelling form 130.)
template <bool Fast>
__device__ __forceinline__ float gelu(float y) {
    constexpr float kFine[] = {0.5f, -0.521293163f, 0.0958522633f, 0.119704634f, 0.00993833877f, -0.0561364889f,
                               0.0359269567f, -0.0946980417f, 0.096099481f, -0.029562287f};
    constexpr float kCoarse[] = {0.499998093f, -0.380580723f, -0.0397436433f, 0.0596017055f, 0.11025656f, -0.0689856187f};
    constexpr int kDegree = Fast ? 5 : 9;
    const float v = fminf(fabsf(y), 15.0f), t = rcp_approx(fmaf(v, Fast ? 0.453125f : 0.390625f, 1.0f)), s = 1.0f - t;
    float q = Fast ? kCoarse[kDegree] : kFine[kDegree];
#pragma unroll
    for (int i = kDegree - 1; i >= 0; --i) q = fmaf(q, s, Fast ? kCoarse[i] : kFine[i]);
    const float v2 = v * v;
    float e = Fast ? __expf(-0.5f * v2) : expf(-0.5f * v2);
    if (!Fast) e = fmaf(e, -0.5f * fmaf(v, v, -v2), e);       // what the rounding of v^2 lost
    const float tail = q * t * e;
    return y * (y < 0.f ? tail : 1.0f - tail);                // a NaN stays a NaN
}

// Activations in fp32. expf and the division are CUDA's own fp32 functions (a few units in the last place).
__device__ __forceinline__ float activate(float y, int act) {
    switch (act) {
    case TFMOE_ACT_RELU: return y < 0.f ? 0.f : y;            // a NaN stays a NaN
    case TFMOE_ACT_SILU: return y / (1.0f + expf(-y));
    case TFMOE_ACT_GELU: return gelu<false>(y);
    case TFMOE_ACT_GELU_TANH:
        // (1 + tanh(z)) / 2 = 1 / (1 + e^-2z), z = sqrt(2/pi) (y + 0.044715 y^3)
        return y / (1.0f + expf(-1.5957691216057308f * (y + 0.044715f * y * y * y)));
    default: return y;
    }
}

// The finished value of output n of token t from its accumulated sum(s) without multiplier.
__device__ __forceinline__ float finish_output(const LinearEpilogue &ep, int t, int n, float s0, float s1, float g0,
                                               float g1) {
    float y = s0 * g0;
    if (ep.bias) y += __ldg(ep.bias + n);
    if (ep.act == TFMOE_ACT_SWIGLU) {
        float u = s1 * g1;
        if (ep.bias) u += __ldg(ep.bias + ep.N + n);
        y = activate(y, TFMOE_ACT_SILU) * u;
    } else {
        y = activate(y, ep.act);
    }
    if (ep.residual) y += bf16_bits_to_float(ep.residual[(int64_t)t * ep.ldr + n]);
    return y;
}

__device__ __forceinline__ void store_output(const LinearEpilogue &ep, int t, int n, float v) {
    if (ep.out_fp32) static_cast<float *>(ep.out)[(int64_t)t * ep.ldo + n] = v;
    else static_cast<uint16_t *>(ep.out)[(int64_t)t * ep.ldo + n] = float_to_bf16_bits_rn(v);
}

}  // namespace tfmoe
