// decode.cu -- the whole MoE layer for a few tokens in one kernel (tfmoe_forward_decode).
//
// A decode step reads its active experts' 4-bit weights once (DGX Spark GB10 bandwidth-budget
// page, section "Mechanism: decode is bandwidth-bound, prefill is compute-bound"); what the chain
// of launches adds to that is a ramp up and down of the stream per projection and one CTA's tail per
// step. Here one CTA per SM stays for the whole layer, and the weight stream (stream.cuh) runs
// through it without a break:
//
//   router     CTA c takes the experts c, c + G, ...: fp64 logits, exact as in the other paths
//   barrier 0  (x becomes the operand rows meanwhile)
//   plan       every CTA takes the top k of all tokens and lists the active experts; the producer
//              warp now knows every byte this CTA will read: its run of the active experts' gate/up
//              tiles, then its run of their down tiles, and does not stop until it has read both
//   gate/up    sums of the run's pieces -> global
//   barrier 1  (the ring fills with down tiles meanwhile)
//   down       per expert of the run: a = silu(G) U from the pieces, as operand rows; sums -> global
//   barrier 2
//   combine    out = bf16(sum_s g_s y_s + residual), slots in order, the tiles of 128 outputs spread over
//              the SMs; with norm weights one CTA per token, which then has the row for its RMS norm
//
// The down run's first tiles are on chip before barrier 1 opens: a ring's worth of bytes (10 slots, 184 KB per SM,
// with one token; 8, 147 KB, with 8 tokens of H 2048; 4, 74 KB, with 14 of H 4096). All sums across CTAs are added
// in a fixed order: equal calls give equal bits.
//
// Measured, calls in a row on rotating weights: H 2048, I 768, E 128, top 8 with one token 22.6 us, with 8 tokens 47
// (137 MB: 2.9 TB/s over all), with shared expert, residual and norm 53; H 4096, I 1536, 14 tokens
// 189 (810 MB: 4.3 TB/s); H 4096, I 2688, E 256, one token 48 (151 MB: 3.2 TB/s). By device timestamps (weights out of
// L2, the slowest CTA) the gate/up stream of 8 tokens runs at 4.2 TB/s, that of the 14 at 5.5, of the large layer's one at
// 4.3; outside the two streams are 7 us before them, 4 to 5 of barrier 1 and a rows and 4 of barrier 2 and combine with 8 tokens.
//
// a is rounded to f16 times a power of two per token and expert: 11 significant bits, exact
// range within 2^-39 of the row's largest (8 times finer than bf16, at no cost: f16 is what the
// product runs on).
//
// The grid barriers need every CTA resident: a cooperative launch. Each wait is bounded; after a
// timeout a CTA goes through the barriers without waiting, and CTA 0 may then set a counter back before the last
// CTA has arrived at it. What is left in the counters is wrong until the host's tfmoe_sync_status
// clears them with the error word (which ends the waits of the calls before that).
#include <algorithm>

#include "internal.h"
#include "stream.cuh"
#include "topk.cuh"

namespace tfmoe {
namespace {

using namespace stream;

constexpr int kArrivalStride = 32;                       // one 128-byte line per counter
constexpr int kMaxSlotsPerToken = 32;
constexpr int kMaxPairs = kMaxTokens * kMaxSlotsPerToken;
static_assert(kMaxPairs <= kConsumerThreads, "one thread per pair");
constexpr uint32_t kTestWaitNs = 1000000;

struct DecodeArgs {
    const uint16_t *x;
    int T, H, I, E, k, m;                                // m: slots of the shared expert
    const uint16_t *router_w;
    const float *bias;
    const uint8_t *gu_codes, *gu_scales, *d_codes, *d_scales;
    const float *gate_global, *up_global, *down_global;
    float *logits;
    int32_t *ids;
    float *topk_w;
    float *gu_part, *d_part;                             // sums of the pieces, see piece_at
    uint32_t *arrivals;                                  // [3] lines, 0 between calls (or left for the next call to clear)
    const uint16_t *residual, *norm_w;
    uint16_t *out, *out_norm;
    double eps;
    int slots, debug;
    uint32_t row_area;
    uint32_t test_wait_ns;
    int32_t *err_word;
};

// The routing of the call, in shared memory. A pair is (token, slot), t * (k + m) + s; rows are pairs
// ordered by (expert, token).
struct Plan {
    int32_t ids[kMaxPairs];
    float w[kMaxPairs];
    uint32_t sel[kMaxTokens][8];                         // experts of a token, one bit each
    uint8_t slot[kMaxTokens][256];                       // a token's slot for each of its experts
    int16_t list[256], poff[256], eidx[256];             // active experts; their first row; place in the list
    uint8_t cnt[256];                                    // their tokens
    uint8_t tok[kMaxPairs];                              // token of a row
    uint8_t ei[kMaxPairs];                               // place in the list of a row's expert
    int16_t row[kMaxPairs];                              // row of a pair
    int n_act;
};

// Where the sums [column][128 rows] of CTA c's piece of row tile rt of an expert with m tokens and
// first row `poff` lie, in floats. Going to the next tile moves by m columns or more and to the next CTA
// by T >= m, so the pieces, at most RT * pairs + G * T columns in all, do not overlap.
__device__ __forceinline__ size_t piece_at(int poff, int RT, int rt, int m, uint32_t c, int T) {
    return (size_t)(uint32_t)(poff * RT + rt * m + (int)c * T) * 128u;
}

// The runs of a phase: no more of them than windows, so that a small layer is not cut into pieces whose
// joining costs more than their reading.
__device__ __forceinline__ Runs runs_of(int units, uint32_t G) {
    return Runs((uint32_t)units, min(G, (uint32_t)(units + kWindow - 1) / kWindow));
}

__device__ __forceinline__ void grid_arrive(uint32_t *counter) {
    consumer_sync();
    if (threadIdx.x == 0) {
        __threadfence();                                 // the CTA's writes, ordered by the barrier above
        atomicAdd(counter, 1u);
    }
}
__device__ __forceinline__ void grid_wait(const Ring &r, uint32_t *counter, uint32_t target) {
    if (threadIdx.x == 0) {
        const uint64_t t0 = global_timer_ns();
        for (int n = 1;; ++n) {
            uint32_t v;
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
            if (v >= target || *r.abort_flag) break;
            if (n % 64) continue;
            if (*reinterpret_cast<volatile int32_t *>(r.err_word) & DEV_ERR_WAIT_TIMEOUT) { *r.abort_flag = 1; break; }
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                atomicOr(r.err_word, DEV_ERR_WAIT_TIMEOUT);
                *r.abort_flag = 1;
                break;
            }
        }
    }
    consumer_sync();
}

// A finite bf16 value as a double times 2^-896: its bits moved to the double's exponent and fraction. bf16
// subnormals become the right double subnormals. (Infinities and NaN would become 2^-768 times 1 to 2, a
// finite number: router_logits looks for them.)
__device__ __forceinline__ double shifted_double_lo(uint32_t u) {
    return __hiloint2double((int)(((uint32_t)((int)(u << 16) >> 3)) & 0x8FFFE000u), 0);
}
__device__ __forceinline__ double shifted_double_hi(uint32_t u) {
    return __hiloint2double((int)(((uint32_t)((int)u >> 3)) & 0x8FFFE000u), 0);
}

// Logits of the CTA's experts for every token: the columns of each (expert, token) are split over `wpt` warps.
__device__ void router_logits(const DecodeArgs &a, double *part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chunks = a.H / 8, G = (int)gridDim.x;
    const int pairs = (a.E - (int)blockIdx.x + G - 1) / G * a.T;     // none for a CTA past the experts
    int wpt = kConsumers;
    while (wpt > 1 && wpt * pairs > kConsumers) wpt >>= 1;
    const int p = warp % wpt;
    for (int first = 0; first < pairs; first += kConsumers / wpt) {
        const int pair = first + warp / wpt, t = pair % a.T, e = (int)blockIdx.x + pair / a.T * G;
        const uint4 *xrow = reinterpret_cast<const uint4 *>(a.x + (size_t)t * a.H);
        const uint4 *wrow = reinterpret_cast<const uint4 *>(a.router_w + (size_t)e * a.H);
        double acc = 0.0;
        uint32_t top = 0;                                // largest magnitude bits of x, in both halves
        if (pair < pairs) {
            for (int i0 = p * 32 + lane; i0 < chunks; i0 += 4 * 32 * wpt) {
                uint4 wv[4], xv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = i0 + j * 32 * wpt;
                    wv[j] = i < chunks ? __ldg(wrow + i) : make_uint4(0, 0, 0, 0);
                    xv[j] = i < chunks ? xrow[i] : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    top = max_bits(xv[j], top);
                    const uint32_t wu[4] = {wv[j].x, wv[j].y, wv[j].z, wv[j].w}, xu[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        acc = fma(shifted_double_lo(xu[q]), (double)bf16_bits_to_float(wu[q] & 0xFFFFu), acc);
                        acc = fma(shifted_double_hi(xu[q]), (double)bf16_bits_to_float(wu[q] >> 16), acc);
                    }
                }
            }
            if (__any_sync(0xffffffffu, max(top >> 16, top & 0xFFFFu) >= 0x7F80u)) {
                // x holds an infinity or a NaN here: the slice once more with converted values, so that the logit is
                // the infinity or NaN that the sum of products is (the scaling back leaves those as they are)
                acc = 0.0;
#pragma unroll 1
                for (int i = p * 32 + lane; i < chunks; i += 32 * wpt) {
                    const uint4 w4 = __ldg(wrow + i), x4 = xrow[i];
                    const uint32_t wu[4] = {w4.x, w4.y, w4.z, w4.w}, xu[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        acc = fma((double)bf16_bits_to_float(xu[q] & 0xFFFFu), (double)bf16_bits_to_float(wu[q] & 0xFFFFu), acc);
                        acc = fma((double)bf16_bits_to_float(xu[q] >> 16), (double)bf16_bits_to_float(wu[q] >> 16), acc);
                    }
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
            if (lane == 0) part[warp] = acc;
        }
        consumer_sync();
        const int mine = first + (int)threadIdx.x;
        if ((int)threadIdx.x < kConsumers / wpt && mine < pairs) {
            const int te = mine % a.T, ee = (int)blockIdx.x + mine / a.T * G;
            double v = 0.0;
            for (int i = 0; i < wpt; ++i) v += part[threadIdx.x * wpt + i];
            float l = (float)(v * 0x1p896);
            if (a.bias) l = l + __ldg(a.bias + ee);
            if (a.debug && !isfinite(l)) atomicOr(a.err_word, DEV_ERR_NONFINITE);
            a.logits[(size_t)te * a.E + ee] = l;
        }
        consumer_sync();
    }
}

// Top k of every token (a warp each) and the plan of the call (a thread per expert).
__device__ void make_plan(const DecodeArgs &a, Plan &pl) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x, kx = a.k + a.m;
    if (warp < a.T) {
        int id;
        float w;
        topk_select(a.logits + (size_t)warp * a.E, a.E, a.k, id, w);
        if (lane >= a.k) { id = a.E + lane - a.k; w = 1.f; }
        if (lane < kx) {
            const int p = warp * kx + lane;
            pl.ids[p] = id;
            pl.w[p] = w;
            pl.slot[warp][id] = (uint8_t)lane;
            atomicOr(&pl.sel[warp][id >> 5], 1u << (id & 31));
            if (blockIdx.x == 0) {
                a.ids[p] = id;
                a.topk_w[p] = w;
            }
        }
    }
    consumer_sync();
    if (tid < 256) {                                     // expert tid: its place, first row and tokens
        const int word = tid >> 5;
        const uint32_t below = (1u << lane) - 1u;
        // lane l < 8: the active experts of word l and their rows; a scan gives those before each word
        uint32_t any = 0, mine = 0, n = 0;
        int rows = 0;
        if (lane < 8)
#pragma unroll 4
            for (int i = 0; i < a.T; ++i) {
                const uint32_t s = pl.sel[i][lane];
                any |= s;
                n += (uint32_t)__popc(s) << 16;
            }
        n += __popc(any);
        uint32_t incl = n;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const uint32_t before = __shfl_sync(0xffffffffu, incl - n, word), own = __shfl_sync(0xffffffffu, any, word);
        if (tid == 7) pl.n_act = (int)(incl & 0xffffu);
        rows = (int)(before >> 16);
        const int idx = (int)(before & 0xffffu) + __popc(own & below);
#pragma unroll 4
        for (int i = 0; i < a.T; ++i) {
            const uint32_t s = pl.sel[i][word];
            rows += __popc(s & below);
            mine |= ((s >> lane) & 1u) << i;
        }
        if (mine) {
            pl.list[idx] = (int16_t)tid;
            pl.cnt[idx] = (uint8_t)__popc(mine);
            pl.poff[idx] = (int16_t)rows;
            pl.eidx[tid] = (int16_t)idx;
            for (int r = rows; mine; mine &= mine - 1, ++r) {
                const int t = __ffs(mine) - 1;
                pl.tok[r] = (uint8_t)t;
                pl.ei[r] = (uint8_t)idx;
                pl.row[t * kx + pl.slot[t][tid]] = (int16_t)r;
            }
        }
    }
    consumer_sync();
}

// a = silu(G) U of the plan's rows [ra, rb) as operand rows 0, 1, ..., from the gate/up pieces. A thread holds
// the values of its first kHold items between finding the row's largest and writing; the rest is computed again.
// Two items' loads are in flight at a time: with one, 8 rows of 768 took 7 us of latency, with four, the code
// of one token's few items cost it 1 us.
template <int kHold>
__device__ void prepare_a(const DecodeArgs &a, const Plan &pl, int ra, int rb, const Runs &r1, uint8_t *rows, uint32_t *emax) {
    const int RT = a.I / 64, KT = a.H / kTileK, KT2 = a.I / kTileK, half = a.I / 2;
    const size_t stride = (size_t)a.T * 32;              // from a tile's piece to its next, in float4
    // an item is two neighbouring outputs of one row; a warp's 32 items share the row and the row tile
    struct Place { const float4 *p; uint32_t n; float g0, g1; };
    auto place = [&](int item) {
        const int r = item / half, jp = item - r * half, rt = jp >> 5, ei = pl.ei[ra + r], e = pl.list[ei];
        const uint32_t q = (uint32_t)(ei * RT + rt) * (uint32_t)KT, ca = r1.owner(q);
        return Place{reinterpret_cast<const float4 *>(a.gu_part + piece_at(pl.poff[ei], RT, rt, pl.cnt[ei], ca, a.T) +
                                                      (ra + r - pl.poff[ei]) * 128) + (jp & 31),
                     r1.owner(q + KT - 1) - ca + 1, __ldg(a.gate_global + e), __ldg(a.up_global + e)};
    };
    // The values of kBatch items, their loads in flight together; an item past the last is the last once more.
    constexpr int kBatch = 2;
    const int items = (rb - ra) * half;
    auto values = [&](int item, float2 *out) {
        Place w[kBatch];
        float4 v[kBatch], u[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            w[j] = place(min(item + j * kConsumerThreads, items - 1));
            v[j] = __ldcg(w[j].p);
            u[j] = __ldcg(w[j].n > 1 ? w[j].p + stride : w[j].p);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            float4 s = v[j];
            auto add = [&](const float4 &o) { s.x += o.x; s.y += o.y; s.z += o.z; s.w += o.w; };
            if (w[j].n > 1) add(u[j]);
            for (uint32_t i = 2; i < w[j].n; ++i) add(__ldcg(w[j].p + i * stride));
            out[j] = make_float2(silu_f32(s.x * w[j].g0) * (s.y * w[j].g1), silu_f32(s.z * w[j].g0) * (s.w * w[j].g1));
        }
    };
    float2 hold[kHold];
    auto note = [&](int item, float2 v) {
        const uint32_t bits = max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu);
        const uint32_t b = __reduce_max_sync(0xffffffffu, bits >> 23);
        if ((threadIdx.x & 31) == 0) atomicMax(&emax[item / half], b);
    };
    for (int i = threadIdx.x; i < rb - ra; i += kConsumerThreads) emax[i] = 0;
    consumer_sync();
    // a warp's lanes have items of one row, all of them or none (half is a multiple of 32)
    for (int j0 = 0, item = threadIdx.x; item < items; j0 += kBatch, item += kBatch * kConsumerThreads) {
        float2 v[kBatch];
        values(item, v);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (item + j * kConsumerThreads < items) note(item + j * kConsumerThreads, v[j]);
#pragma unroll
            for (int h = 0; h < kHold; h += kBatch)
                if (j0 == h) hold[h + j] = v[j];
        }
    }
    consumer_sync();
    auto put = [&](int item, float2 v) {
        const int r = item / half, j = 2 * (item - r * half);
        const float up = up_of(emax[r]);
        *reinterpret_cast<__half2 *>(rows + r * row_bytes(KT2) + chunk_offset(j & ~7) + (j & 7) * 2) =
            __floats2half2_rn(v.x * up, v.y * up);
    };
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
        const int item = threadIdx.x + j * kConsumerThreads;
        if (item < items) put(item, hold[j]);
    }
    for (int item = threadIdx.x + kHold * kConsumerThreads; item < items; item += kBatch * kConsumerThreads) {
        float2 v[kBatch];
        values(item, v);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (item + j * kConsumerThreads < items) put(item + j * kConsumerThreads, v[j]);
    }
    consumer_sync();
}

// The weighted sum of token t's slots (plus the residual) at h = 128 rt + 4 lane and the three after it, by one
// warp, rounded to bf16: two words.
__device__ __forceinline__ uint2 combine128(const DecodeArgs &a, const Plan &pl, int t, int rt, const Runs &r2) {
    const int lane = threadIdx.x & 31, kx = a.k + a.m, RT = a.H / kTileRows, KT = a.I / kTileK;
    // lane s finds the pieces of slot s
    uint32_t base = 0, n = 0;
    float w = 0.f;
    if (lane < kx) {
        const int p = t * kx + lane, ei = pl.eidx[pl.ids[p]], poff = pl.poff[ei], m = pl.cnt[ei];
        const uint32_t q = (uint32_t)(ei * RT + rt) * (uint32_t)KT, ca = r2.owner(q);
        base = (uint32_t)(piece_at(poff, RT, rt, m, ca, a.T) + (pl.row[p] - poff) * 128);
        n = r2.owner(q + KT - 1) - ca + 1;
        w = pl.w[p];
    }
    const size_t at = (size_t)t * a.H + rt * 128 + 4 * lane;
    const uint2 res = a.residual ? *reinterpret_cast<const uint2 *>(a.residual + at) : make_uint2(0u, 0u);
    const uint32_t most = __reduce_max_sync(0xffffffffu, n);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [](float4 &s, const float4 &o) { s.x += o.x; s.y += o.y; s.z += o.z; s.w += o.w; };
    constexpr int kS = 8;                                // slots in flight, two pieces of each
    for (int s0 = 0; s0 < kx; s0 += kS) {
        float4 v[kS], u[kS];
        auto load = [&](float4 (&o)[kS], uint32_t i) {
#pragma unroll
            for (int j = 0; j < kS; ++j) {
                const uint32_t b = __shfl_sync(0xffffffffu, base, (s0 + j) & 31), c = __shfl_sync(0xffffffffu, n, (s0 + j) & 31);
                o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (s0 + j < kx && i < c) o[j] = __ldcg(reinterpret_cast<const float4 *>(a.d_part + b + i * a.T * 128u) + lane);
            }
        };
        load(v, 0);
        for (uint32_t i = 1; i < most; ++i) {
            load(u, i);
#pragma unroll
            for (int j = 0; j < kS; ++j) add(v[j], u[j]);
        }
#pragma unroll
        for (int j = 0; j < kS; ++j) {
            const float g = __shfl_sync(0xffffffffu, w, (s0 + j) & 31);
            if (s0 + j < kx) {
                acc.x = fmaf(g, v[j].x, acc.x);
                acc.y = fmaf(g, v[j].y, acc.y);
                acc.z = fmaf(g, v[j].z, acc.z);
                acc.w = fmaf(g, v[j].w, acc.w);
            }
        }
    }
    if (a.residual) add(acc, make_float4(bf16_bits_to_float(res.x & 0xFFFFu), bf16_bits_to_float(res.x >> 16),
                                         bf16_bits_to_float(res.y & 0xFFFFu), bf16_bits_to_float(res.y >> 16)));
    const uint2 o = make_uint2((uint32_t)float_to_bf16_bits_rn(acc.x) | ((uint32_t)float_to_bf16_bits_rn(acc.y) << 16),
                               (uint32_t)float_to_bf16_bits_rn(acc.z) | ((uint32_t)float_to_bf16_bits_rn(acc.w) << 16));
    *reinterpret_cast<uint2 *>(a.out + at) = o;
    return o;
}

struct Layout {
    uint32_t rows, sums, zeros, emax, bars, total;
    // row_area: for the T rows of x and, later, the a rows of as many experts as fit
    __host__ __device__ Layout(int T, uint32_t row_area, int slots) {
        rows = (uint32_t)slots * kSlotBytes;
        sums = rows + row_area;
        zeros = sums + 2u * T * kSumStride * 4;
        emax = zeros + 256;                              // of the x rows and the a rows
        bars = emax + (kMaxTokens + kMaxPairs) * 4;
        total = bars + (2 * kMaxSlots + 3) * 8;          // full, empty, planned, never, abort flag
    }
};

// The gate/up pieces of the units [u, end) once more, from global memory without rounding x.
__device__ __forceinline__ void exact_gate_up(const DecodeArgs &a, const Plan &pl, uint32_t u, uint32_t end) {
    consumer_sync();                                     // the pieces' first sums are written
    for (Pieces p(u, end, a.I / 64, a.H / kTileK); p.valid(); p.next()) {
        const int m = pl.cnt[p.ei], poff = pl.poff[p.ei];
        const size_t tile = ((size_t)pl.list[p.ei] * p.RT + p.rt) * p.KT;
        float *dst = a.gu_part + piece_at(poff, p.RT, p.rt, m, blockIdx.x, a.T);
        for (int i = threadIdx.x; i < m * 128; i += kConsumerThreads)
            dst[i] = exact_dot<false>(a.gu_codes + tile * kTileCodeBytes, a.gu_scales + tile * kTileScaleBytes, p.ka, p.kb, i & 127,
                                      a.x + (size_t)pl.tok[poff + (i >> 7)] * a.H, a.H);
    }
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const DecodeArgs a)
{
    using In = std::conditional_t<NT == 1, WindowConsumer<NT>, PairConsumer<NT>>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Plan pl;
    __shared__ double part[kConsumers];
    const int KT1 = a.H / kTileK, RT1 = a.I / 64, KT2 = a.I / kTileK, RT2 = a.H / kTileRows;
    const Layout lay(a.T, a.row_area, a.slots);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + lay.bars);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t G = gridDim.x, c = blockIdx.x;
    Ring ring;
    ring.slots = smem_u32(smem);
    ring.full = smem_u32(bars);
    ring.empty = ring.full + 8u * kMaxSlots;
    ring.zeros = smem_u32(smem + lay.zeros);
    ring.n = a.slots;
    ring.early = false;
    ring.abort_flag = reinterpret_cast<volatile int32_t *>(bars + 2 * kMaxSlots + 2);
    ring.err_word = a.err_word;
    const uint32_t planned = ring.full + 8u * (2 * kMaxSlots);
    if (warp == kConsumers) {
        if (lane < a.slots) {
            mbar_init(bars + lane, 1);
            mbar_init(bars + kMaxSlots + lane, In::kArrivals);
        }
        if (lane == 0) {
            mbar_init(bars + 2 * kMaxSlots, 1);
            mbar_init(bars + 2 * kMaxSlots + 1, 1);      // no thread ever arrives on this one
            *ring.abort_flag = 0;
        }
        fence_mbar_init();
    }
    if (threadIdx.x < kMaxTokens * 8) reinterpret_cast<uint32_t *>(pl.sel)[threadIdx.x] = 0;
    if (threadIdx.x < kMaxTokens) {
        reinterpret_cast<uint32_t *>(smem + lay.emax)[threadIdx.x] = 0;
        reinterpret_cast<uint32_t *>(smem + lay.sums)[threadIdx.x] = 0xFFFFFFFFu;   // the rows' smallest, before there are sums
    }
    if (threadIdx.x < 64) reinterpret_cast<uint32_t *>(smem + lay.zeros)[threadIdx.x] = 0;
    __syncthreads();

    if (warp >= kConsumers) {
        give_registers();
        if (warp == kConsumers && lane == 0 && wait(ring, planned, 0)) {
            Cursor cur;
            uint32_t issued = 0;
            bool ok = true;
            auto nothing = [](uint32_t) {};
            auto run = [&](const uint8_t *codes, const uint8_t *scales, int RT, int KT) {
                const Runs r = runs_of(pl.n_act * RT * KT, G);
                for (Pieces p(r.first(c), r.end(c), RT, KT); p.valid() && ok; p.next()) {
                    const size_t tile = ((size_t)pl.list[p.ei] * RT + p.rt) * KT;
                    ok = produce_piece(ring, cur, issued, codes + tile * kTileCodeBytes, scales + tile * kTileScaleBytes, p.ka,
                                       p.kb, nothing);
                }
            };
            run(a.gu_codes, a.gu_scales, RT1, KT1);
            run(a.d_codes, a.d_scales, RT2, KT2);
            if (*ring.abort_flag) drain(ring, cur, issued);
        }
        return;
    }

    take_registers();
    uint32_t *emax = reinterpret_cast<uint32_t *>(smem + lay.emax);
    uint8_t *rows = smem + lay.rows;
    uint32_t *arrive0 = a.arrivals, *arrive1 = a.arrivals + kArrivalStride, *arrive2 = a.arrivals + 2 * kArrivalStride;

    router_logits(a, part);
    grid_arrive(arrive0);
    const bool wide = convert_rows<8 * NT, false>(a.x, a.H, rows, a.T, a.H, KT1, emax, reinterpret_cast<uint32_t *>(smem + lay.sums),
                                                  [](int) { return true; });
    grid_wait(ring, arrive0, G);
    // counter 2 still holds the last call's arrivals; everyone's next use of it is behind barrier 1
    if (c == 0 && threadIdx.x == 0) *arrive2 = 0;
    if (a.test_wait_ns && c == 0 && threadIdx.x == 0) {
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait_sleep_at(planned + 8u, 0))
            if (global_timer_ns() - t0 > a.test_wait_ns) {
                atomicOr(a.err_word, DEV_ERR_WAIT_TIMEOUT);
                *ring.abort_flag = 1;
                break;
            }
    }
    make_plan(a, pl);
    if (threadIdx.x == 0) mbar_arrive_at(planned);

    // gate/up, then down: one loop, so that both run the same code
    In in(ring);
    float *buf = reinterpret_cast<float *>(smem + lay.sums), *other = buf + a.T * kSumStride;   // of sums, in turn
    const int n_act = uniform(pl.n_act);
    const Runs r1 = runs_of(n_act * RT1 * KT1, G), r2 = runs_of(n_act * RT2 * KT2, G);
    const uint32_t rows_at = ring.slots + lay.rows;
    const int g = lane >> 2, t = lane & 3;
    // the a rows of as many of the down run's experts as fit are prepared together: rows [r0, r_end)
    const int fit = (int)(a.row_area / row_bytes(KT2));
    int r0 = 0, r_end = 0;
#pragma unroll 1
    for (int down = 0; down < 2; ++down) {
        if (down) {
            if (wide) exact_gate_up(a, pl, r1.first(c), r1.end(c));   // x rows that f16 cannot hold
            grid_arrive(arrive1);
        }
        const int RT = down ? RT2 : RT1, KT = down ? KT2 : KT1;
        const uint32_t rb = row_bytes(KT);
        const uint32_t *em = down ? emax + kMaxTokens : emax;
        Pieces p(down ? r2.first(c) : r1.first(c), down ? r2.end(c) : r1.end(c), RT, KT);
        // the a rows of expert ei of the run and of those after it that fit: [r0, r_end)
        auto next_rows = [&](int ei) {
            const int last = (int)((p.end - 1) / ((uint32_t)RT2 * KT2));
            r0 = uniform(pl.poff[ei]);
            int el = ei;
            while (el < last && pl.poff[el + 1] + pl.cnt[el + 1] - r0 <= fit) ++el;
            r_end = uniform(pl.poff[el] + pl.cnt[el]);
        };
        if (p.valid()) {
            in.fetch(p.windows() + p.rest());
            if (down) next_rows(p.ei);
        }
        bool prepared = false;
        if (down) {
            grid_wait(ring, arrive1, G);
            if (c == 0 && threadIdx.x == 0) *arrive0 = 0;
        }
        while (p.valid()) {
            const int ei = p.ei, m = uniform(pl.cnt[ei]), poff = uniform(pl.poff[ei]);
            float scale = 1.f;
            if (down) {
                if (!prepared || poff >= r_end) {
                    if (prepared) {
                        next_rows(ei);
                        consumer_sync();                 // the rows in use are free
                    }
                    prepare_a<NT == 1 ? 8 : 4>(a, pl, r0, r_end, r1, rows, emax + kMaxTokens);
                    prepared = true;
                }
                scale = __ldg(a.down_global + pl.list[ei]);
            }
            // the lane's operand rows and the factors of its sums: columns are the expert's tokens
            uint32_t xa[NT];
            float f[NT][2];
            auto row = [&](int col) { return (uint32_t)(down ? poff - r0 + col : pl.tok[poff + col]); };
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                xa[n] = rows_at + row(8 * n + g < m ? 8 * n + g : 0) * rb;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int col = 8 * n + 2 * t + j;
                    f[n][j] = col < m ? inverse_up(em[row(col)]) * scale : 0.f;
                }
            }
            float *dst = (down ? a.d_part : a.gu_part) + piece_at(poff, RT, p.rt, m, c, a.T) + (2 * t) * 128 + (warp & 7) * 16 + g;
            const bool two = m > 8;
            do {
                Acc<NT> acc;
                acc.clear();
                in.piece(p.ka, p.kb, p.rest(), xa, two, acc);
                join_pairs<NT>(acc, buf, m, [&](int n, int j, float v) {
                    if (8 * n + 2 * t + (j & 1) < m) dst[(8 * n + (j & 1)) * 128 + 8 * (j >> 1)] = v * f[n][j & 1];
                });
                float *const swap = buf;
                buf = other;
                other = swap;
                dst += m * 128;                          // the next tile's columns follow this one's
                p.next();
            } while (p.valid() && p.ei == ei);
        }
    }
    grid_arrive(arrive2);
    if ((int)c >= (a.norm_w ? a.T : a.T * RT2)) return;
    grid_wait(ring, arrive2, G);
    if (c == 0 && threadIdx.x == 0) *arrive1 = 0;
    if (!a.norm_w) {
        // a few tiles for every SM rather than all of them for a few
        for (int i = (int)c + warp * (int)G; i < a.T * RT2; i += (int)G * kConsumers) combine128(a, pl, i / RT2, i % RT2, r2);
        return;
    }
    // one CTA per token: the row in shared memory, its fp64 sum of squares, the norm (as combine.cu)
    for (int t = (int)c; t < a.T; t += (int)G) {
        uint2 *keep = reinterpret_cast<uint2 *>(rows);
        double ss = 0.0;
        for (int rt = warp; rt < RT2; rt += kConsumers) {
            const uint2 o = combine128(a, pl, t, rt, r2);
            keep[rt * 32 + lane] = o;
            const float x[4] = {bf16_bits_to_float(o.x & 0xFFFFu), bf16_bits_to_float(o.x >> 16),
                                bf16_bits_to_float(o.y & 0xFFFFu), bf16_bits_to_float(o.y >> 16)};
#pragma unroll
            for (int j = 0; j < 4; ++j) ss = fma((double)x[j], (double)x[j], ss);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane == 0) part[warp] = ss;
        consumer_sync();
        double tot = 0.0;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) tot += part[w];
        const double r = 1.0 / sqrt(tot / (double)a.H + a.eps);
        for (int rt = warp; rt < RT2; rt += kConsumers) {
            const uint2 o = keep[rt * 32 + lane];
            const uint2 gm = *reinterpret_cast<const uint2 *>(a.norm_w + rt * 128 + 4 * lane);
            const uint32_t ow[2] = {o.x, o.y}, gw[2] = {gm.x, gm.y};
            uint32_t nw[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const double lo = (double)bf16_bits_to_float(ow[j] & 0xFFFFu) * r * (double)bf16_bits_to_float(gw[j] & 0xFFFFu);
                const double hi = (double)bf16_bits_to_float(ow[j] >> 16) * r * (double)bf16_bits_to_float(gw[j] >> 16);
                nw[j] = (uint32_t)double_to_bf16_bits_rn(lo) | ((uint32_t)double_to_bf16_bits_rn(hi) << 16);
            }
            *reinterpret_cast<uint2 *>(a.out_norm + (size_t)t * a.H + rt * 128 + 4 * lane) = make_uint2(nw[0], nw[1]);
        }
        consumer_sync();
    }
}

// Dynamic shared memory: 227 KB less the static part and the 1 KB the runtime keeps per CTA.
constexpr int kSmemLimit = 227 * 1024 - 1024 - (int)sizeof(Plan) - (int)sizeof(double) * kConsumers - 256;
constexpr int kMinSlots = 3;     // 55 KB in flight per SM still cover the latency of HBM

// Whether a call runs the kernel for one tile of 8 tokens. Its groups take alternate windows, which wants a
// ring of at least 4 slots; where the rows leave fewer, the kernel for two tiles runs.
bool one_tile(int T, int slots) { return T <= 8 && slots >= 4; }

uint32_t least_rows(const Layer &L, int T) { return (uint32_t)T * row_bytes(std::max(L.desc.hidden, L.desc.intermediate) / kTileK); }
int decode_slots(const Layer &L, int T) {
    const int left = kSmemLimit - (int)Layout(T, least_rows(L, T), 0).total;
    const int n = left < 0 ? 0 : std::min(kMaxSlots, left / kSlotBytes);
    return one_tile(T, n) ? n & ~1 : n;                  // an even number: WindowConsumer
}
// What the slots leave goes to the rows: a run that crosses into another expert then prepares both at once
// (one token, 4096 x 2688: 3 us of the CTAs that do).
uint32_t decode_row_area(const Layer &L, int T) {
    const uint32_t least = least_rows(L, T);
    return least + (((uint32_t)kSmemLimit - Layout(T, least, decode_slots(L, T)).total) & ~255u);
}

int decode_workspace_tokens(const Layer &L) { return std::min(L.desc.max_tokens, kMaxTokens); }

}  // namespace

int decode_max_tokens(const Layer &L) {
    int T = decode_workspace_tokens(L);
    while (T > 0 && decode_slots(L, T) < kMinSlots) --T;
    return T;
}

size_t decode_gu_floats(const Layer &L) {
    const size_t T = decode_workspace_tokens(L);
    return (T * token_slots(L) * (L.desc.intermediate / 64) + (size_t)L.num_sms * T) * 128;
}
size_t decode_d_floats(const Layer &L) {
    const size_t T = decode_workspace_tokens(L);
    return (T * token_slots(L) * (L.desc.hidden / kTileRows) + (size_t)L.num_sms * T) * 128;
}
size_t decode_arrival_words() { return 3 * kArrivalStride; }

cudaError_t decode_setup(const Layer &)
{
    cudaError_t e = cudaFuncSetAttribute(decode_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(decode_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    return e;
}

cudaError_t launch_decode(Layer &L, const uint16_t *x, int T, const uint16_t *residual, const uint16_t *norm_w,
                          uint16_t *out, uint16_t *out_norm, cudaStream_t s, int *launches)
{
    DecodeArgs a{};
    a.x = x;
    a.T = T; a.H = L.desc.hidden; a.I = L.desc.intermediate; a.E = L.desc.num_experts; a.k = L.desc.top_k;
    a.m = shared_slots(L);
    a.router_w = L.w.router_w;
    a.bias = L.desc.has_router_bias ? L.w.router_bias : nullptr;
    a.gu_codes = L.w.gu_codes; a.gu_scales = L.w.gu_scales;
    a.d_codes = L.w.d_codes; a.d_scales = L.w.d_scales;
    a.gate_global = L.w.gate_global; a.up_global = L.w.up_global; a.down_global = L.w.down_global;
    a.logits = L.ws.logits; a.ids = L.ws.ids; a.topk_w = L.ws.topk_w;
    a.gu_part = L.ws.dec_gu; a.d_part = L.ws.dec_d;
    a.arrivals = L.ws.dec_arrivals;
    a.residual = residual; a.norm_w = norm_w; a.out = out; a.out_norm = out_norm;
    a.eps = (double)L.desc.norm_eps;
    a.slots = decode_slots(L, T);
    a.row_area = decode_row_area(L, T);
    a.debug = (L.desc.flags & TFMOE_FLAG_DEBUG_CHECKS) ? 1 : 0;
    a.test_wait_ns = (L.desc.flags & TFMOE_FLAG_TEST_TIMEOUT) && !L.decode_timed_out ? kTestWaitNs : 0;
    L.decode_timed_out = true;
    a.err_word = L.ws.err_word;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(L.num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout(T, a.row_area, a.slots).total;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, one_tile(T, a.slots) ? decode_kernel<1> : decode_kernel<2>, a);
    *launches += 1;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tfmoe
