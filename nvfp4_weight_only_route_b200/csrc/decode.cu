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

// a = silu(G) U of the plan's rows [ra, rb) as operand rows 0, 1, ..., from the gate/up pieces.
__device__ void prepare_a(const DecodeArgs &a, const Plan &pl, int ra, int rb, const Runs &r1, uint8_t *rows, uint32_t *emax) {
    const int RT = a.I / 64, KT = a.H / kTileK, KT2 = a.I / kTileK, half = a.I / 2;
    const size_t stride = (size_t)a.T * 32;              // from a tile's piece to its next, in float4
    // an item is two neighbouring outputs of one row; a warp's 32 items share the row and the row tile
    auto value = [&](int item) {
        const int r = item / half, jp = item - r * half, rt = jp >> 5, ei = pl.ei[ra + r], e = pl.list[ei];
        const float g0 = __ldg(a.gate_global + e), g1 = __ldg(a.up_global + e);
        const uint32_t q = (uint32_t)(ei * RT + rt) * (uint32_t)KT, ca = r1.owner(q), n = r1.owner(q + KT - 1) - ca + 1;
        const float4 *p = reinterpret_cast<const float4 *>(a.gu_part + piece_at(pl.poff[ei], RT, rt, pl.cnt[ei], ca, a.T) +
                                                           (ra + r - pl.poff[ei]) * 128) + (jp & 31);
        float4 v[4], s = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](const float4 &u) { s.x += u.x; s.y += u.y; s.z += u.z; s.w += u.w; };
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i == 0 || i < (int)n) v[i] = __ldcg(p + i * stride);
        s = v[0];
#pragma unroll
        for (int i = 1; i < 4; ++i)
            if (i < (int)n) add(v[i]);
        for (uint32_t i = 4; i < n; ++i) add(__ldcg(p + i * stride));
        return make_float2(silu_f32(s.x * g0) * (s.y * g1), silu_f32(s.z * g0) * (s.w * g1));
    };
    constexpr int kHold = 3;
    float2 hold[kHold];
    const int items = (rb - ra) * half;
    auto note = [&](int item, float2 v) {
        const uint32_t bits = max(__float_as_uint(v.x) & 0x7FFFFFFFu, __float_as_uint(v.y) & 0x7FFFFFFFu);
        const uint32_t b = __reduce_max_sync(0xffffffffu, bits >> 23);
        if ((threadIdx.x & 31) == 0) atomicMax(&emax[item / half], b);
    };
    for (int i = threadIdx.x; i < rb - ra; i += kConsumerThreads) emax[i] = 0;
    consumer_sync();
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
    for (int item = threadIdx.x + kHold * kConsumerThreads; item < items; item += kConsumerThreads) put(item, value(item));
    consumer_sync();
}

// The weighted sum of token t's slots (plus the residual) at h = 64 hb + 2 lane and h + 1, by one warp.
__device__ __forceinline__ float2 combine64(const DecodeArgs &a, const Plan &pl, int t, int hb, const Runs &r2) {
    const int lane = threadIdx.x & 31, kx = a.k + a.m, RT = a.H / kTileRows, KT = a.I / kTileK, rt = hb >> 1;
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
    const uint32_t col = (uint32_t)(hb & 1) * 64u + 2u * lane, most = __reduce_max_sync(0xffffffffu, n);
    float2 acc = make_float2(0.f, 0.f);
    for (int s0 = 0; s0 < kx; s0 += 8) {
        float2 v[8], u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = __shfl_sync(0xffffffffu, base, (s0 + j) & 31), c = __shfl_sync(0xffffffffu, n, (s0 + j) & 31);
            v[j] = u[j] = make_float2(0.f, 0.f);
            const float2 *src = reinterpret_cast<const float2 *>(a.d_part + b + col);
            if (s0 + j < kx && c > 0) v[j] = __ldcg(src);
            if (s0 + j < kx && c > 1) u[j] = __ldcg(src + a.T * 64);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) { v[j].x += u[j].x; v[j].y += u[j].y; }
        for (uint32_t i = 2; i < most; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = __shfl_sync(0xffffffffu, base, (s0 + j) & 31), c = __shfl_sync(0xffffffffu, n, (s0 + j) & 31);
                u[j] = make_float2(0.f, 0.f);
                if (s0 + j < kx && i < c) u[j] = __ldcg(reinterpret_cast<const float2 *>(a.d_part + b + i * a.T * 128u + col));
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) { v[j].x += u[j].x; v[j].y += u[j].y; }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float g = __shfl_sync(0xffffffffu, w, (s0 + j) & 31);
            if (s0 + j < kx) {
                acc.x = fmaf(g, v[j].x, acc.x);
                acc.y = fmaf(g, v[j].y, acc.y);
            }
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
        emax = zeros + 256;                              // of the x rows and the a rows
        bars = emax + (kMaxTokens + kMaxPairs) * 4;
        total = bars + (2 * kMaxSlots + 3) * 8;          // full, empty, planned, never, abort flag
    }
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const DecodeArgs a)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Plan pl;
    __shared__ double part[kConsumers];
    const int KT1 = a.H / kTileK, RT1 = a.I / 64, KT2 = a.I / kTileK, RT2 = a.H / kTileRows;
    const Layout lay(a.T, KT1, KT2, a.slots);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + lay.bars);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
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
    if (threadIdx.x < kMaxTokens) reinterpret_cast<uint32_t *>(smem + lay.emax)[threadIdx.x] = 0;
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
    convert_rows<8, false>(a.x, a.H, rows, a.T, a.H, KT1, emax, [](int) { return true; });
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
    Consumer<NT> in(ring);
    float *buf = reinterpret_cast<float *>(smem + lay.sums), *other = buf + a.T * kSumStride;   // of sums, in turn
    const int n_act = uniform(pl.n_act);
    const Runs r1 = runs_of(n_act * RT1 * KT1, G), r2 = runs_of(n_act * RT2 * KT2, G);
    const uint32_t rows_at = ring.slots + lay.rows;
    const int g = lane >> 2, t = lane & 3;
    // the a rows of as many of the down run's experts as fit are prepared together: rows [r0, r_end)
    const int fit = (int)((uint32_t)a.T * row_bytes(KT1 > KT2 ? KT1 : KT2) / row_bytes(KT2));
    int r0 = 0, r_end = 0;
#pragma unroll 1
    for (int down = 0; down < 2; ++down) {
        if (down) {
            grid_arrive(arrive1);
            grid_wait(ring, arrive1, G);
            if (c == 0 && threadIdx.x == 0) *arrive0 = 0;
        }
        const int RT = down ? RT2 : RT1, KT = down ? KT2 : KT1;
        const uint32_t rb = row_bytes(KT);
        const uint32_t *em = down ? emax + kMaxTokens : emax;
        Pieces p(down ? r2.first(c) : r1.first(c), down ? r2.end(c) : r1.end(c), RT, KT);
        if (p.valid()) in.fetch();
        while (p.valid()) {
            const int ei = p.ei, m = uniform(pl.cnt[ei]), poff = uniform(pl.poff[ei]);
            float scale = 1.f;
            if (down) {
                if (poff >= r_end) {
                    const int last = (int)((p.end - 1) / ((uint32_t)RT2 * KT2));
                    int el = ei;
                    while (el < last && pl.poff[el + 1] + pl.cnt[el + 1] - poff <= fit) ++el;
                    r0 = poff;
                    r_end = uniform(pl.poff[el] + pl.cnt[el]);
                    consumer_sync();                     // the rows in use are free
                    prepare_a(a, pl, r0, r_end, r1, rows, emax + kMaxTokens);
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
                in.piece(p.ka, p.kb, p.more(), xa, two, acc);
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
    const int blocks = a.H / 64;
    if (a.norm_w ? (int)c >= a.T : (int)c * kConsumers >= a.T * blocks) return;
    grid_wait(ring, arrive2, G);
    if (c == 0 && threadIdx.x == 0) *arrive1 = 0;
    if (!a.norm_w) {
        for (int i = (int)c * kConsumers + warp; i < a.T * blocks; i += (int)G * kConsumers) {
            const int t = i / blocks, hb = i - t * blocks;
            const float2 v = combine64(a, pl, t, hb, r2);
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
            const float2 v = combine64(a, pl, t, hb, r2);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, T <= 8 ? decode_kernel<1> : decode_kernel<2>, a);
    *launches += 1;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tfmoe
