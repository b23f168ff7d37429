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
//   combine    out = bf16(sum_s g_s y_s + residual), slots in order; with norm weights one CTA per
//              token, which then has the row for its RMS norm
//
// The down run's first tiles are on chip before barrier 1 opens, so HBM idles only where a ring's
// worth of bytes (about 180 KB per SM, 4 us) does not cover a barrier. All sums across CTAs are added
// in a fixed order: equal calls give equal bits.
//
// a is rounded to f16 times a power of two per token and expert: 11 significant bits, exact
// range within 2^-39 of the row's largest (8 times finer than bf16, at no cost: f16 is what the
// product runs on).
//
// The grid barriers need every CTA resident: a cooperative launch. Each wait is bounded; after a
// timeout every CTA still arrives at every barrier, so that the arrival counters end where they
// should, and the host's tfmoe_sync_status clears them.
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
    uint32_t test_wait_ns;
    int32_t *err_word;
};

// The routing of the call, in shared memory. A pair is (token, slot), t * (k + m) + s; rows are pairs
// ordered by (expert, token).
struct Plan {
    int32_t ids[kMaxPairs];
    float w[kMaxPairs];
    uint32_t sel[kMaxTokens][8];                         // experts of a token, one bit each
    int16_t list[256], poff[256], eidx[256];             // active experts; their first row; place in the list
    uint8_t cnt[256];                                    // their tokens
    uint8_t tok[kMaxPairs];                              // token of a row
    int16_t row[kMaxPairs];                              // row of a pair
    int n_act;
};

// Where the sums [column][128 rows] of CTA c's piece of row tile rt of an expert with m tokens and
// first row `poff` lie, in floats. Going to the next tile moves by m columns or more and to the next CTA
// by T >= m, so the pieces, at most RT * pairs + G * T columns in all, do not overlap.
__device__ __forceinline__ size_t piece_at(int poff, int RT, int rt, int m, uint32_t c, int T) {
    return (size_t)(uint32_t)(poff * RT + rt * m + (int)c * T) * 128u;
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

// A bf16 value as a double times 2^-896: its bits moved to the double's exponent and fraction. bf16
// subnormals become the right double subnormals; infinities and NaN become 2^-768 times 1 to 2, which
// the scaling back turns into an infinite logit.
__device__ __forceinline__ double shifted_double_lo(uint32_t u) {
    return __hiloint2double((int)(((uint32_t)((int)(u << 16) >> 3)) & 0x8FFFE000u), 0);
}
__device__ __forceinline__ double shifted_double_hi(uint32_t u) {
    return __hiloint2double((int)(((uint32_t)((int)u >> 3)) & 0x8FFFE000u), 0);
}

// Logits of the CTA's experts for every token: each token's columns are split over `wpt` warps.
__device__ void router_logits(const DecodeArgs &a, double *part) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int wpt = kConsumers;
    while (wpt * a.T > kConsumers) wpt >>= 1;
    const int t = warp / wpt, p = warp % wpt, chunks = a.H / 8;
    const uint4 *xrow = reinterpret_cast<const uint4 *>(a.x + (size_t)t * a.H);
    for (int e = blockIdx.x; e < a.E; e += gridDim.x) {
        const uint4 *wrow = reinterpret_cast<const uint4 *>(a.router_w + (size_t)e * a.H);
        double acc = 0.0;
        if (t < a.T) {
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
                    const uint32_t wu[4] = {wv[j].x, wv[j].y, wv[j].z, wv[j].w}, xu[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        acc = fma(shifted_double_lo(xu[q]), (double)bf16_bits_to_float(wu[q] & 0xFFFFu), acc);
                        acc = fma(shifted_double_hi(xu[q]), (double)bf16_bits_to_float(wu[q] >> 16), acc);
                    }
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
            if (lane == 0) part[warp] = acc;
        }
        consumer_sync();
        if (threadIdx.x < a.T) {
            double v = 0.0;
            for (int i = 0; i < wpt; ++i) v += part[threadIdx.x * wpt + i];
            float l = (float)(v * 0x1p896);
            if (a.bias) l = l + __ldg(a.bias + e);
            if (a.debug && !isfinite(l)) atomicOr(a.err_word, DEV_ERR_NONFINITE);
            a.logits[(size_t)threadIdx.x * a.E + e] = l;
        }
        consumer_sync();
    }
}

// Top k of every token and the plan of the call.
__device__ void make_plan(const DecodeArgs &a, Plan &pl) {
    const int warp = threadIdx.x >> 5, tid = threadIdx.x, kx = a.k + a.m;
    if (warp < a.T) topk_warp(a.logits + (size_t)warp * a.E, a.E, a.k, pl.ids + warp * kx, pl.w + warp * kx, nullptr, a.m);
    consumer_sync();
    const bool pair = tid < a.T * kx;
    const int t = tid / kx, e = pair ? pl.ids[tid] : 0;
    if (pair) {
        atomicOr(&pl.sel[t][e >> 5], 1u << (e & 31));
        if (blockIdx.x == 0) {
            a.ids[tid] = e;
            a.topk_w[tid] = pl.w[tid];
        }
    }
    consumer_sync();
    if (tid < 256) {                                     // expert tid: its place, first row and tokens
        const int word = tid >> 5;
        const uint32_t below = (1u << (tid & 31)) - 1u;
        int idx = 0, rows = 0, n = 0;
        for (int w = 0; w <= word; ++w) {
            uint32_t any = 0;
            for (int i = 0; i < a.T; ++i) {
                const uint32_t s = pl.sel[i][w];
                any |= s;
                rows += __popc(w < word ? s : s & below);
                if (w == word) n += (s >> (tid & 31)) & 1u;
            }
            idx += __popc(w < word ? any : any & below);
        }
        if (n) {
            pl.list[idx] = (int16_t)tid;
            pl.cnt[idx] = (uint8_t)n;
            pl.poff[idx] = (int16_t)rows;
            pl.eidx[tid] = (int16_t)idx;
        }
        if (tid == 255) pl.n_act = idx + (n ? 1 : 0);
    }
    consumer_sync();
    if (pair) {
        int col = 0;
        for (int i = 0; i < t; ++i) col += (pl.sel[i][e >> 5] >> (e & 31)) & 1u;
        const int r = pl.poff[pl.eidx[e]] + col;
        pl.tok[r] = (uint8_t)t;
        pl.row[tid] = (int16_t)r;
    }
    consumer_sync();
}

// One piece through the consumers: the sums of m columns, times factor(column), to dst [m][128].
template <int NT, class RowOf, class Factor>
__device__ __forceinline__ void run_piece(const Ring &r, Cursor &c, const Lane &ln, int ka, int kb, int m, RowOf row_of,
                                          Factor factor, float *buf, float *dst) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint32_t xa[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) xa[n] = row_of(8 * n + g < m ? 8 * n + g : 0);
    Acc<NT> acc;
    acc.clear();
    consume_piece<NT>(r, c, ln, ka, kb, xa, acc);
    // the second half's sums go through shared memory (two buffers in turn, so one barrier per piece)
    const int row = (warp & 7) * 16 + g;
    if (warp >= 8) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = 8 * n + 2 * t + (j & 1);
                if (col < m) buf[col * kSumStride + row + 8 * (j >> 1)] = acc.sum(n, j);
            }
    }
    consumer_sync();
    if (warp < 8) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = 8 * n + 2 * t + (j & 1), rr = row + 8 * (j >> 1);
                if (col < m) dst[col * 128 + rr] = (acc.sum(n, j) + buf[col * kSumStride + rr]) * factor(col);
            }
    }
}

// a = silu(G) U of the m tokens of list entry ei as operand rows, from the gate/up pieces.
__device__ void prepare_a(const DecodeArgs &a, const Plan &pl, int ei, uint32_t U1, uint32_t G, uint8_t *rows,
                          uint32_t *emax, uint32_t *emax_next) {
    const int RT = a.I / 64, KT = a.H / kTileK, KT2 = a.I / kTileK, half = a.I / 2;
    const int m = pl.cnt[ei], poff = pl.poff[ei], e = pl.list[ei];
    const float g0 = __ldg(a.gate_global + e), g1 = __ldg(a.up_global + e);
    // item: two neighbouring outputs of one column; a warp's 32 items share the column and the row tile
    auto value = [&](int item) {
        const int col = item / half, jp = item - col * half, rt = jp >> 5;
        const uint32_t q = (uint32_t)(ei * RT + rt) * (uint32_t)KT;
        const uint32_t ca = owner(q, U1, G), cb = owner(q + KT - 1, U1, G);
        const float4 *src = reinterpret_cast<const float4 *>(a.gu_part + piece_at(poff, RT, rt, m, ca, a.T) + col * 128) + (jp & 31);
        float4 s = __ldcg(src);
#pragma unroll 4
        for (uint32_t c = ca + 1; c <= cb; ++c) {
            const float4 v = __ldcg(src + (size_t)(c - ca) * a.T * 32);
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        return make_float2(silu_f32(s.x * g0) * (s.y * g1), silu_f32(s.z * g0) * (s.w * g1));
    };
    constexpr int kHold = 4;
    float2 hold[kHold];
    const int items = m * half;
    auto note = [&](int item, float2 v) {
        const uint32_t bits = max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu);
        const uint32_t b = __reduce_max_sync(0xffffffffu, bits >> 23);
        if ((threadIdx.x & 31) == 0) atomicMax(&emax[item / half], b);
    };
    consumer_sync();                                     // the rows and the other exponents are free
    if (threadIdx.x < kMaxTokens) emax_next[threadIdx.x] = 0;
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
        const int item = threadIdx.x + j * kConsumerThreads;
        if (item < items) hold[j] = value(item);
    }
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
        const int item = threadIdx.x + j * kConsumerThreads;
        if (item < items) note(item, hold[j]);
    }
    for (int item = threadIdx.x + kHold * kConsumerThreads; item < items; item += kConsumerThreads) note(item, value(item));
    consumer_sync();
    auto put = [&](int item, float2 v) {
        const int col = item / half, j = 2 * (item - col * half);
        const float up = up_of(emax[col]);
        *reinterpret_cast<__half2 *>(rows + col * row_bytes(KT2) + chunk_offset(j & ~7) + (j & 7) * 2) =
            __floats2half2_rn(v.x * up, v.y * up);
    };
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
        const int item = threadIdx.x + j * kConsumerThreads;
        if (item < items) put(item, hold[j]);
    }
    for (int item = threadIdx.x + kHold * kConsumerThreads; item < items; item += kConsumerThreads) put(item, value(item));
    consumer_sync();
}

// The weighted sum of token t's slots (plus the residual) at h = 64 hb + 2 lane and h + 1, by one warp.
__device__ __forceinline__ float2 combine64(const DecodeArgs &a, const Plan &pl, int t, int hb, uint32_t U2, uint32_t G) {
    const int lane = threadIdx.x & 31, kx = a.k + a.m, RT = a.H / kTileRows, KT = a.I / kTileK, rt = hb >> 1;
    // lane s finds the pieces of slot s
    uint32_t base = 0, n = 0;
    float w = 0.f;
    if (lane < kx) {
        const int p = t * kx + lane, ei = pl.eidx[pl.ids[p]], poff = pl.poff[ei], m = pl.cnt[ei];
        const uint32_t q = (uint32_t)(ei * RT + rt) * (uint32_t)KT;
        const uint32_t ca = owner(q, U2, G), cb = owner(q + KT - 1, U2, G);
        base = (uint32_t)(piece_at(poff, RT, rt, m, ca, a.T) + (pl.row[p] - poff) * 128);
        n = cb - ca + 1;
        w = pl.w[p];
    }
    const uint32_t col = (uint32_t)(hb & 1) * 64u + 2u * lane;
    float2 acc = make_float2(0.f, 0.f);
    for (int s0 = 0; s0 < kx; s0 += 8) {
        float2 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = __shfl_sync(0xffffffffu, base, (s0 + j) & 31);
            if (s0 + j < kx) v[j] = __ldcg(reinterpret_cast<const float2 *>(a.d_part + b + col));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = __shfl_sync(0xffffffffu, base, (s0 + j) & 31), c = __shfl_sync(0xffffffffu, n, (s0 + j) & 31);
            const float g = __shfl_sync(0xffffffffu, w, (s0 + j) & 31);
            if (s0 + j >= kx) continue;
#pragma unroll 2
            for (uint32_t i = 1; i < c; ++i) {
                const float2 u = __ldcg(reinterpret_cast<const float2 *>(a.d_part + b + i * a.T * 128u + col));
                v[j].x += u.x;
                v[j].y += u.y;
            }
            acc.x = fmaf(g, v[j].x, acc.x);
            acc.y = fmaf(g, v[j].y, acc.y);
        }
    }
    if (a.residual) {
        const uint32_t r = *reinterpret_cast<const uint32_t *>(a.residual + (size_t)t * a.H + hb * 64 + 2 * lane);
        acc.x += bf16_bits_to_float(r & 0xFFFFu);
        acc.y += bf16_bits_to_float(r >> 16);
    }
    return acc;
}

struct Layout {
    uint32_t rows, sums, zeros, emax, bars, total;
    __host__ __device__ Layout(int T, int KT1, int KT2, int slots) {
        rows = (uint32_t)slots * kSlotBytes;
        sums = rows + (uint32_t)T * row_bytes(KT1 > KT2 ? KT1 : KT2);
        zeros = sums + 2u * T * kSumStride * 4;
        emax = zeros + 256;                              // x rows, a rows of the experts in turn
        bars = emax + 3 * kMaxTokens * 4;
        total = bars + (2 * kMaxSlots + 3) * 8;          // full, empty, planned, never, abort flag
    }
};

__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const DecodeArgs a)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Plan pl;
    __shared__ double part[kConsumers];
    const int KT1 = a.H / kTileK, RT1 = a.I / 64, KT2 = a.I / kTileK, RT2 = a.H / kTileRows;
    const Layout lay(a.T, KT1, KT2, a.slots);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + lay.bars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t G = gridDim.x, c = blockIdx.x;
    Ring ring;
    ring.slots = smem_u32(smem);
    ring.full = smem_u32(bars);
    ring.empty = ring.full + 8u * kMaxSlots;
    ring.zeros = smem_u32(smem + lay.zeros);
    ring.n = a.slots;
    ring.abort_flag = reinterpret_cast<volatile int32_t *>(bars + 2 * kMaxSlots + 2);
    ring.err_word = a.err_word;
    const uint32_t planned = ring.full + 8u * (2 * kMaxSlots);
    if (warp == kConsumers) {
        if (lane < a.slots) {
            mbar_init(bars + lane, 1);
            mbar_init(bars + kMaxSlots + lane, kConsumers);
        }
        if (lane == 0) {
            mbar_init(bars + 2 * kMaxSlots, 1);
            mbar_init(bars + 2 * kMaxSlots + 1, 1);      // no thread ever arrives on this one
            *ring.abort_flag = 0;
        }
        fence_mbar_init();
    }
    if (threadIdx.x < kMaxTokens * 8) reinterpret_cast<uint32_t *>(pl.sel)[threadIdx.x] = 0;
    if (threadIdx.x < 3 * kMaxTokens) reinterpret_cast<uint32_t *>(smem + lay.emax)[threadIdx.x] = 0;
    if (threadIdx.x < 64) reinterpret_cast<uint32_t *>(smem + lay.zeros)[threadIdx.x] = 0;
    __syncthreads();

    if (warp == kConsumers) {
        if (lane == 0 && wait(ring, planned, 0)) {
            Cursor cur;
            uint32_t issued = 0;
            bool ok = true;
            auto nothing = [](uint32_t) {};
            auto run = [&](const uint8_t *codes, const uint8_t *scales, int RT, int KT) {
                const uint32_t U = (uint32_t)pl.n_act * RT * KT, Gs = min(G, U);
                const uint32_t u1 = c < Gs ? first_unit(c + 1, U, Gs) : 0u;
                for (uint32_t u = first_unit(c, U, Gs); u < u1 && ok;) {
                    const uint32_t q = u / KT, ei = q / RT;
                    const int ka = (int)(u - q * KT), kb = (int)min((uint32_t)KT, ka + (u1 - u));
                    const size_t tile = ((size_t)pl.list[ei] * RT + (q - ei * RT)) * KT;
                    ok = produce_piece(ring, cur, issued, codes + tile * kTileCodeBytes, scales + tile * kTileScaleBytes, ka,
                                       kb, nothing);
                    u += kb - ka;
                }
            };
            run(a.gu_codes, a.gu_scales, RT1, KT1);
            run(a.d_codes, a.d_scales, RT2, KT2);
            if (*ring.abort_flag) drain(ring, cur, issued);
        }
        return;
    }

    uint32_t *emax = reinterpret_cast<uint32_t *>(smem + lay.emax);
    uint8_t *rows = smem + lay.rows;
    float *sums = reinterpret_cast<float *>(smem + lay.sums);
    uint32_t *arrive0 = a.arrivals, *arrive1 = a.arrivals + kArrivalStride, *arrive2 = a.arrivals + 2 * kArrivalStride;

    router_logits(a, part);
    grid_arrive(arrive0);
    convert_rows<8>(a.x, a.H, rows, a.T, a.H, KT1, emax, [](int) { return true; });
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

    const Lane ln;
    Cursor cur;
    int buf = 0;
    const uint32_t U1 = (uint32_t)pl.n_act * RT1 * KT1, U2 = (uint32_t)pl.n_act * RT2 * KT2;
    // the CTAs that stream: no more than there are units, so that each has some
    const uint32_t G1 = min(G, U1), G2 = min(G, U2);
    const uint32_t rows_at = ring.slots + lay.rows;
    {
        const uint32_t u1 = c < G1 ? first_unit(c + 1, U1, G1) : 0u, rb = row_bytes(KT1);
        for (uint32_t u = first_unit(c, U1, G1); u < u1;) {
            const uint32_t q = u / KT1, ei = q / RT1;
            const int rt = (int)(q - ei * RT1), ka = (int)(u - q * KT1), kb = (int)min((uint32_t)KT1, ka + (u1 - u));
            const int m = pl.cnt[ei], poff = pl.poff[ei];
            auto row_of = [&](int col) { return rows_at + pl.tok[poff + col] * rb; };
            auto factor = [&](int col) { return inverse_up(emax[pl.tok[poff + col]]); };
            float *dst = a.gu_part + piece_at(poff, RT1, rt, m, c, a.T), *sb = sums + buf * a.T * kSumStride;
            if (m <= 8) run_piece<1>(ring, cur, ln, ka, kb, m, row_of, factor, sb, dst);
            else run_piece<2>(ring, cur, ln, ka, kb, m, row_of, factor, sb, dst);
            buf ^= 1;
            u += kb - ka;
        }
    }
    grid_arrive(arrive1);
    grid_wait(ring, arrive1, G);
    if (c == 0 && threadIdx.x == 0) *arrive0 = 0;
    {
        const uint32_t u1 = c < G2 ? first_unit(c + 1, U2, G2) : 0u, rb = row_bytes(KT2);
        int have = -1, set = 0;
        float dg = 0.f;
        for (uint32_t u = first_unit(c, U2, G2); u < u1;) {
            const uint32_t q = u / KT2;
            const int ei = (int)(q / RT2);
            const int rt = (int)(q - (uint32_t)ei * RT2), ka = (int)(u - q * KT2), kb = (int)min((uint32_t)KT2, ka + (u1 - u));
            const int m = pl.cnt[ei], poff = pl.poff[ei];
            if (ei != have) {
                have = ei;
                set ^= 1;
                dg = __ldg(a.down_global + pl.list[ei]);
                prepare_a(a, pl, ei, U1, G1, rows, emax + (1 + set) * kMaxTokens, emax + (2 - set) * kMaxTokens);
            }
            const uint32_t *ea = emax + (1 + set) * kMaxTokens;
            auto row_of = [&](int col) { return rows_at + (uint32_t)col * rb; };
            auto factor = [&](int col) { return inverse_up(ea[col]) * dg; };
            float *dst = a.d_part + piece_at(poff, RT2, rt, m, c, a.T), *sb = sums + buf * a.T * kSumStride;
            if (m <= 8) run_piece<1>(ring, cur, ln, ka, kb, m, row_of, factor, sb, dst);
            else run_piece<2>(ring, cur, ln, ka, kb, m, row_of, factor, sb, dst);
            buf ^= 1;
            u += kb - ka;
        }
    }
    grid_arrive(arrive2);
    const int blocks = a.H / 64;
    if (a.norm_w ? (int)c >= a.T : (int)c * kConsumers >= a.T * blocks) return;
    grid_wait(ring, arrive2, G);
    if (c == 0 && threadIdx.x == 0) *arrive1 = 0;
    if (!a.norm_w) {
        for (int i = (int)c * kConsumers + warp; i < a.T * blocks; i += (int)G * kConsumers) {
            const int t = i / blocks, hb = i - t * blocks;
            const float2 v = combine64(a, pl, t, hb, U2, G2);
            *reinterpret_cast<uint32_t *>(a.out + (size_t)t * a.H + hb * 64 + 2 * lane) =
                (uint32_t)float_to_bf16_bits_rn(v.x) | ((uint32_t)float_to_bf16_bits_rn(v.y) << 16);
        }
        return;
    }
    // one CTA per token: the row in shared memory, its fp64 sum of squares, the norm (as combine.cu)
    for (int t = (int)c; t < a.T; t += (int)G) {
        uint32_t *keep = reinterpret_cast<uint32_t *>(rows);
        double ss = 0.0;
        for (int hb = warp; hb < blocks; hb += kConsumers) {
            const float2 v = combine64(a, pl, t, hb, U2, G2);
            const uint32_t lo = float_to_bf16_bits_rn(v.x), hi = float_to_bf16_bits_rn(v.y);
            *reinterpret_cast<uint32_t *>(a.out + (size_t)t * a.H + hb * 64 + 2 * lane) = lo | (hi << 16);
            keep[hb * 32 + lane] = lo | (hi << 16);
            const double x0 = bf16_bits_to_float(lo), x1 = bf16_bits_to_float(hi);
            ss = fma(x0, x0, ss);
            ss = fma(x1, x1, ss);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane == 0) part[warp] = ss;
        consumer_sync();
        double tot = 0.0;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) tot += part[w];
        const double r = 1.0 / sqrt(tot / (double)a.H + a.eps);
        for (int hb = warp; hb < blocks; hb += kConsumers) {
            const uint32_t o = keep[hb * 32 + lane];
            const uint32_t gm = *reinterpret_cast<const uint32_t *>(a.norm_w + hb * 64 + 2 * lane);
            const double lo = (double)bf16_bits_to_float(o & 0xFFFFu) * r * (double)bf16_bits_to_float(gm & 0xFFFFu);
            const double hi = (double)bf16_bits_to_float(o >> 16) * r * (double)bf16_bits_to_float(gm >> 16);
            *reinterpret_cast<uint32_t *>(a.out_norm + (size_t)t * a.H + hb * 64 + 2 * lane) =
                (uint32_t)double_to_bf16_bits_rn(lo) | ((uint32_t)double_to_bf16_bits_rn(hi) << 16);
        }
        consumer_sync();
    }
}

// Dynamic shared memory: 227 KB less the static part and the 1 KB the runtime keeps per CTA.
constexpr int kSmemLimit = 227 * 1024 - 1024 - (int)sizeof(Plan) - (int)sizeof(double) * kConsumers - 256;
constexpr int kMinSlots = 3;     // 55 KB in flight per SM still cover the latency of HBM

int decode_slots(const Layer &L, int T) {
    const int left = kSmemLimit - (int)Layout(T, L.desc.hidden / kTileK, L.desc.intermediate / kTileK, 0).total;
    return left < 0 ? 0 : std::min(kMaxSlots, left / kSlotBytes);
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
    return cudaFuncSetAttribute(decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
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
    a.debug = (L.desc.flags & TFMOE_FLAG_DEBUG_CHECKS) ? 1 : 0;
    a.test_wait_ns = (L.desc.flags & TFMOE_FLAG_TEST_TIMEOUT) ? kTestWaitNs : 0;
    a.err_word = L.ws.err_word;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(L.num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout(T, a.H / kTileK, a.I / kTileK, a.slots).total;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_kernel, a);
    *launches += 1;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tfmoe
