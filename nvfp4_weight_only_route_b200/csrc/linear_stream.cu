// linear_stream.cu -- the streaming regime of the NVFP4 matrix product: up to 16 tokens, bound by
// the weight bytes over HBM bandwidth (stream.cuh has the stream and the arithmetic).
//
// The x rows become f16 times a power of two per row and CTA (exact for every element within
// 2^28 of the largest one the CTA uses; smaller ones are rounded to 2^-39 of the largest) and stay
// in shared memory. A row tile that one CTA owns is finished there. One that is cut by CTA borders
// leaves its pieces' sums in global memory (at most two pieces per CTA: its first and its last), and
// the CTA that arrives last at the tile's counter adds them in CTA order and finishes it: no
// CTA waits for another, so the launch needs no co-residency, and equal calls give equal bits.
// The launch is a programmatic dependent of the one before it: the weights, which no kernel
// writes, start to stream before that kernel has ended.
#include <algorithm>

#include "linear.h"
#include "stream.cuh"

namespace tfmoe {
namespace {

using namespace stream;

struct StreamArgs {
    const uint8_t *codes, *scales;
    const uint16_t *x;
    int64_t ldx;
    int T, K, RT, KT, slots;
    float *partial;          // [2 G][T][128]: the first and the last piece of every CTA
    int32_t *tickets;        // [RT] arrivals per row tile, left at 0
    int32_t *err_word;
    LinearEpilogue ep;
};

// Shared memory after the slots: token rows, sums, zeros, per-row exponents, barriers.
struct Layout {
    uint32_t x, sums, zeros, emax, bars, total;
    __host__ __device__ Layout(int T, int KT, int slots) {
        x = (uint32_t)slots * kSlotBytes;
        sums = x + (uint32_t)T * row_bytes(KT);
        zeros = sums + kMaxTokens * kSumStride * 4;
        emax = zeros + 256;
        bars = emax + kMaxTokens * 4;
        total = bars + (2 * kMaxSlots + 2) * 8;          // full, empty, token rows landed, abort flag
    }
};

// Outputs of row tile rt from sums[token][row] (per-token factor 2^-sh in inv).
__device__ __forceinline__ void finish_tile(const StreamArgs &a, int rt, const float *sums, const uint32_t *emax,
                                            float g0, float g1) {
    const bool gated = a.ep.act == TFMOE_ACT_SWIGLU;
    const int per = gated ? 64 : 128;
    for (int i = threadIdx.x; i < a.T * per; i += kConsumerThreads) {
        const int t = i / per, j = i % per, n = rt * per + j;
        if (n >= a.ep.N) continue;
        const float inv = emax ? inverse_up(emax[t]) : 1.f;
        const float *s = sums + t * kSumStride + (gated ? 2 * j : j);
        store_output(a.ep, t, n, finish_output(a.ep, t, n, s[0] * inv, gated ? s[1] * inv : 0.f, g0, g1));
    }
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) linear_stream_kernel(const StreamArgs a)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int last[2];
    const Layout lay(a.T, a.KT, a.slots);
    float *sums = reinterpret_cast<float *>(smem + lay.sums);
    uint32_t *emax = reinterpret_cast<uint32_t *>(smem + lay.emax);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + lay.bars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Ring ring;
    ring.slots = smem_u32(smem);
    ring.full = smem_u32(bars);
    ring.empty = ring.full + 8u * kMaxSlots;
    ring.zeros = smem_u32(smem + lay.zeros);
    ring.n = a.slots;
    ring.abort_flag = reinterpret_cast<volatile int32_t *>(bars + 2 * kMaxSlots + 1);
    ring.err_word = a.err_word;
    const uint32_t xfull = ring.full + 8u * (2 * kMaxSlots);
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.slots; ++i) {
            mbar_init(bars + i, 1);
            mbar_init(bars + kMaxSlots + i, kConsumers);
        }
        mbar_init(bars + 2 * kMaxSlots, 1);
        *ring.abort_flag = 0;
        fence_mbar_init();
    }
    if (threadIdx.x < kMaxTokens) emax[threadIdx.x] = 0;
    if (threadIdx.x < 64) reinterpret_cast<uint32_t *>(smem + lay.zeros)[threadIdx.x] = 0;
    __syncthreads();
    grid_dep_launch_dependents();

    const uint32_t G = gridDim.x, c = blockIdx.x, U = (uint32_t)a.RT * a.KT;
    const uint32_t u0 = first_unit(c, U, G), u1 = first_unit(c + 1, U, G);
    const int q0 = (int)(u0 / a.KT), k0 = (int)(u0 % a.KT);           // u0 < u1: G <= U
    const int q1 = (int)((u1 - 1) / a.KT), k1 = (int)((u1 - 1) % a.KT) + 1;
    // the columns this CTA uses: [xa0, xb0) and, when its run wraps into the next row tile, [0, xb1)
    const bool all = q1 > q0 + 1 || (q1 == q0 + 1 && k1 >= (k0 & ~1));
    const int xa0 = all ? 0 : (k0 & ~1) * kTileK, xb0 = min(a.K, (q1 > q0 ? a.KT : (k1 + 1) & ~1) * kTileK);
    const int xb1 = all || q1 == q0 ? 0 : min(xa0, ((k1 + 1) & ~1) * kTileK);
    if (warp == kConsumers) {
        if (lane == 0) {
            Cursor cur;
            uint32_t issued = 0;
            // One slot of weights, which no kernel writes, then the rows, then the rest: rows behind a
            // full ring would wait for 150 KB of weights.
            bool ok = true, rows = false;
            for (int q = q0; q <= q1 && ok; ++q) {
                const int ka = q == q0 ? k0 : 0, kb = q == q1 ? k1 : a.KT;
                const uint8_t *codes = a.codes + (size_t)q * a.KT * kTileCodeBytes;
                const uint8_t *scales = a.scales + (size_t)q * a.KT * kTileScaleBytes;
                int k = ka;
                if (!rows) {
                    k = min(kb, (ka & ~(kWindow - 1)) + kWindow);
                    ok = produce_piece(ring, cur, issued, codes, scales, ka, k);
                    rows = true;
                    grid_dep_wait();
                    const uint32_t bytes = (uint32_t)(xb0 - xa0 + xb1) * 2u;
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                                 ::"r"(xfull), "r"(bytes * a.T) : "memory");
                    for (int t = 0; t < a.T; ++t) {
                        const uint32_t dst = ring.slots + lay.x + t * row_bytes(a.KT);
                        const uint16_t *src = a.x + (int64_t)t * a.ldx;
                        bulk_at(dst + xa0 * 2, src + xa0, (uint32_t)(xb0 - xa0) * 2u, xfull);
                        if (xb1) bulk_at(dst, src, (uint32_t)xb1 * 2u, xfull);
                    }
                }
                if (ok) ok = produce_piece(ring, cur, issued, codes, scales, k, kb);
            }
            if (*ring.abort_flag) {
                drain(ring, cur, issued);
                const uint64_t t0 = global_timer_ns();
                while (!mbar_try_wait_sleep_at(xfull, 0) && global_timer_ns() - t0 < kWaitLimitNs / 4) {
                }
            }
        }
        return;
    }

    const bool gated = a.ep.act == TFMOE_ACT_SWIGLU;
    const float g0 = __ldg(a.ep.global0), g1 = gated ? __ldg(a.ep.global1) : 0.f;
    grid_dep_wait();                                        // before anything another kernel may write
    wait(ring, xfull, 0);
    convert_rows(smem + lay.x, a.T, a.K, a.KT, emax,
                 [&](int kg) { return (kg * 128 >= xa0 && kg * 128 < xb0) || kg * 128 < xb1; });

    const Lane ln;
    uint32_t xa[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = 8 * n + (lane >> 2);
        xa[n] = ring.slots + lay.x + (uint32_t)(t < a.T ? t : 0) * row_bytes(a.KT);
    }
    Cursor cur;
    Acc<NT> acc;
    bool cut[2] = {false, false};
    for (int q = q0; q <= q1; ++q) {
        const int ka = q == q0 ? k0 : 0, kb = q == q1 ? k1 : a.KT;
        acc.clear();
        consume_piece<NT>(ring, cur, ln, ka, kb, xa, acc);
        join_parities<NT>(acc, sums, a.T);
        if (kb - ka == a.KT) {
            finish_tile(a, q, sums, emax, g0, g1);
        } else {
            cut[q != q0] = true;
            float *mine = a.partial + (size_t)(2 * c + (q != q0)) * a.T * 128;
            for (int i = threadIdx.x; i < a.T * 128; i += kConsumerThreads)
                mine[i] = sums[(i >> 7) * kSumStride + (i & 127)] * inverse_up(emax[i >> 7]);
        }
        if (q < q1) consumer_sync();                        // sums are free again
    }
    if (!cut[0] && !cut[1]) return;
    consumer_sync();
    if (threadIdx.x < 2) {
        int is_last = 0;
        __threadfence();                                    // the whole CTA's pieces, ordered by the barrier
        if (cut[threadIdx.x]) {
            const uint32_t q = threadIdx.x ? q1 : q0;
            const uint32_t ca = owner(q * a.KT, U, G), cb = owner((q + 1) * a.KT - 1, U, G);
            is_last = atomicAdd(a.tickets + q, 1) == (int)(cb - ca);
            if (is_last) a.tickets[q] = 0;                  // for the next call
            __threadfence();
        }
        last[threadIdx.x] = is_last;
    }
    consumer_sync();
    for (int p = 0; p < 2; ++p) {
        if (!last[p]) continue;
        const uint32_t q = p ? q1 : q0;
        const uint32_t ca = owner(q * a.KT, U, G), cb = owner((q + 1) * a.KT - 1, U, G);
        const size_t stride = (size_t)2 * a.T * 32;         // in float4
        for (int i = threadIdx.x; i < a.T * 32; i += kConsumerThreads) {
            // only the first of the tile's CTAs can have started before the tile
            const float4 *src = reinterpret_cast<const float4 *>(a.partial) + ca * stride + i;
            float4 v = __ldcg(src + (first_unit(ca, U, G) / a.KT != q) * (stride / 2));
            for (uint32_t cc = ca + 1; cc <= cb; cc += 4) {
                float4 p4[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (cc + j <= cb) p4[j] = __ldcg(src + (cc + j - ca) * stride);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (cc + j <= cb) { v.x += p4[j].x; v.y += p4[j].y; v.z += p4[j].z; v.w += p4[j].w; }
            }
            *reinterpret_cast<float4 *>(sums + (i >> 5) * kSumStride + (i & 31) * 4) = v;
        }
        consumer_sync();
        finish_tile(a, q, sums, nullptr, g0, g1);
        consumer_sync();
    }
}

constexpr int kSmemLimit = 227 * 1024 - 1024;   // the static part and the runtime's own 1 KB stay outside

int slots_for(int T, int KT) {
    const int left = kSmemLimit - (int)Layout(T, KT, 0).total;
    return std::min(kMaxSlots, left / kSlotBytes);
}

}  // namespace

// The streaming regime needs the token rows and a ring of at least 4 slots (74 KB: enough bytes in
// flight for HBM) in shared memory.
bool linear_stream_fits(const Linear &L, int T) { return T <= kMaxTokens && slots_for(T, L.KT) >= 4; }

cudaError_t linear_stream_setup(const Linear &)
{
    cudaError_t e = cudaFuncSetAttribute(linear_stream_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(linear_stream_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    return e;
}

size_t linear_stream_partial_floats(const Linear &L) {
    return (size_t)2 * L.num_sms * std::min<int>(L.desc.max_tokens, kMaxTokens) * 128;
}

cudaError_t launch_linear_stream(Linear &L, const uint16_t *x, int64_t ldx, int T, const LinearEpilogue &ep,
                                 cudaStream_t s, int *launches)
{
    StreamArgs a{};
    a.codes = L.codes; a.scales = L.scales;
    a.x = x; a.ldx = ldx;
    a.T = T; a.K = L.desc.in_features; a.RT = L.RT; a.KT = L.KT;
    a.slots = slots_for(T, L.KT);
    a.partial = L.partial; a.tickets = L.tickets; a.err_word = L.err_word;
    a.ep = ep;
    const int grid = (int)std::min<int64_t>(L.num_sms, (int64_t)L.RT * L.KT);
    const size_t smem = Layout(T, L.KT, a.slots).total;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, T <= 8 ? linear_stream_kernel<1> : linear_stream_kernel<2>, a);
    *launches += 1;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tfmoe
