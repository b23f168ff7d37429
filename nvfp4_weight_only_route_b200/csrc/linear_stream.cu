// linear_stream.cu -- the streaming regime of the NVFP4 matrix product: up to 16 tokens, bound by
// the weight bytes over HBM bandwidth (stream.cuh has the stream and the arithmetic).
//
// The x rows become f16 times a power of two per row and CTA and stay in shared memory: exact as long as the
// elements that the CTA uses of a row lie within 2^31 of one another. A CTA that finds others takes its pieces'
// sums from exact_dot instead. A row tile that one CTA owns is finished there. One that is cut by CTA borders
// leaves its pieces' sums in global memory (at most two pieces per CTA: its first and its last), and
// the CTA that arrives last at the tile's counter adds them in CTA order and finishes it: no
// CTA waits for another, so the launch needs no co-residency, and equal calls give equal bits.
// Measured, calls in a row on rotating weights: 1 x 2048 x 4096 8.3 us, 8 x 4096 x 32001 with fp32 out 22.7 (75 MB: 3.3 TB/s
// over all). Fitted to calls on one matrix, which L2 may hold: a start of 7 us (one row) to 12 (16 rows), and 0.42 to
// 0.65 us per window of 18.4 KB and SM (HBM's pace is 0.42).
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
    uint32_t test_wait_ns;   // > 0: CTA 0's producer waits that long for nothing and times out
    LinearEpilogue ep;
};

// Shared memory after the slots: token rows, two buffers of sums (the first also a joined tile's), zeros, per-row exponents, barriers.
struct Layout {
    uint32_t x, sums, zeros, emax, bars, total;
    __host__ __device__ Layout(int T, int KT, int slots) {
        x = (uint32_t)slots * kSlotBytes;
        sums = x + (uint32_t)T * row_bytes(KT);
        zeros = sums + 2u * T * kSumStride * 4;
        emax = zeros + 256;
        bars = emax + kMaxTokens * 4;
        total = bars + (2 * kMaxSlots + 2) * 8;          // full, empty, rows requested, abort flag
    }
};

// Outputs of row tile rt from its joined sums[token][row].
__device__ __forceinline__ void finish_tile(const StreamArgs &a, int rt, const float *sums, float g0, float g1) {
    const bool gated = a.ep.act == TFMOE_ACT_SWIGLU;
    const int per = gated ? 64 : 128;
    for (int i = threadIdx.x; i < a.T * per; i += kConsumerThreads) {
        const int t = i / per, j = i % per, n = rt * per + j;
        if (n >= a.ep.N) continue;
        const float *s = sums + t * kSumStride + (gated ? 2 * j : j);
        store_output(a.ep, t, n, finish_output(a.ep, t, n, s[0], gated ? s[1] : 0.f, g0, g1));
    }
}

// The CTA's pieces once more, from global memory without rounding x; the products above stored nothing.
__device__ __forceinline__ void exact_pieces(const StreamArgs &a, int q0, int k0, int q1, int k1, float *sums, float g0, float g1) {
    for (int q = q0; q <= q1; ++q) {
        const int ka = q == q0 ? k0 : 0, kb = q == q1 ? k1 : a.KT;
        const bool cut = kb - ka < a.KT;
        float *mine = a.partial + (size_t)(2 * blockIdx.x + (q != q0)) * a.T * 128;
        consumer_sync();                                    // the sums are free
        for (int i = threadIdx.x; i < a.T * 128; i += kConsumerThreads) {
            const int t = i >> 7, row = i & 127;
            const float v = exact_dot<true>(a.codes + (size_t)q * a.KT * kTileCodeBytes, a.scales + (size_t)q * a.KT * kTileScaleBytes,
                                            ka, kb, row, a.x + (int64_t)t * a.ldx, a.K);
            if (cut) mine[i] = v;
            else sums[t * kSumStride + row] = v;
        }
        if (cut) continue;
        consumer_sync();
        finish_tile(a, q, sums, g0, g1);
    }
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) linear_stream_kernel(const StreamArgs a)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int join[2][3];                              // per cut piece: last to arrive, first and last CTA of the tile
    const Layout lay(a.T, a.KT, a.slots);
    float *sums = reinterpret_cast<float *>(smem + lay.sums);
    uint32_t *emax = reinterpret_cast<uint32_t *>(smem + lay.emax);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + lay.bars);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    Ring ring;
    ring.slots = smem_u32(smem);
    ring.full = smem_u32(bars);
    ring.empty = ring.full + 8u * kMaxSlots;
    ring.zeros = smem_u32(smem + lay.zeros);
    ring.n = a.slots;
    ring.early = true;
    ring.abort_flag = reinterpret_cast<volatile int32_t *>(bars + 2 * kMaxSlots + 1);
    const uint32_t requested = ring.full + 8u * (2 * kMaxSlots);
    ring.err_word = a.err_word;
    const uint32_t c = blockIdx.x;
    const Runs runs((uint32_t)a.RT * a.KT, gridDim.x);
    const uint32_t u0 = runs.first(c), u1 = runs.first(c + 1);
    const int q0 = (int)(u0 / a.KT), k0 = (int)(u0 - (uint32_t)q0 * a.KT);                   // u0 < u1: G <= U
    const int q1 = (int)((u1 - 1) / a.KT), k1 = (int)(u1 - 1 - (uint32_t)q1 * a.KT) + 1;
    grid_dep_launch_dependents();
    if (warp >= kConsumers) {
        give_registers();
        if (warp > kConsumers) return;
        if (lane < a.slots) {
            mbar_init(bars + lane, 1);
            mbar_init(bars + kMaxSlots + lane, WindowConsumer<NT>::kArrivals);
        }
        if (lane == 0) {
            mbar_init(bars + 2 * kMaxSlots, kConsumers);
            *ring.abort_flag = 0;
        }
        fence_mbar_init();
        __syncwarp();
        asm volatile("bar.arrive 10, %0;" ::"n"(kConsumerThreads + 32) : "memory");   // the consumers wait there
        if (lane == 0) {
            Cursor cur;
            uint32_t issued = 0;
            bool ok = true;
            if (a.test_wait_ns && c == 0) {                 // nobody else fills the first slot
                const uint64_t t0 = global_timer_ns();
                while (ok && !mbar_try_wait_sleep_at(ring.full, 0)) ok = global_timer_ns() - t0 <= a.test_wait_ns;
                atomicOr(a.err_word, DEV_ERR_WAIT_TIMEOUT);
                *ring.abort_flag = 1;
            }
            // Two slots at once, the rest behind the requests for the token rows: rows queued behind
            // a whole ring of weights arrive 3 us later.
            auto rows_first = [&](uint32_t n) { if (n == 2) wait(ring, requested, 0); };
            for (int q = q0; q <= q1 && ok; ++q)
                ok = produce_piece(ring, cur, issued, a.codes + (size_t)q * a.KT * kTileCodeBytes,
                                   a.scales + (size_t)q * a.KT * kTileScaleBytes, q == q0 ? k0 : 0, q == q1 ? k1 : a.KT, rows_first);
            if (*ring.abort_flag) drain(ring, cur, issued);
        }
        return;
    }

    take_registers();
    uint32_t *low = reinterpret_cast<uint32_t *>(sums);      // before there are sums
    if (threadIdx.x < kMaxTokens) {
        emax[threadIdx.x] = 0;
        low[threadIdx.x] = 0xFFFFFFFFu;
    }
    if (threadIdx.x < 64) reinterpret_cast<uint32_t *>(smem + lay.zeros)[threadIdx.x] = 0;
    const bool gated = a.ep.act == TFMOE_ACT_SWIGLU;
    const float g0 = __ldg(a.ep.global0), g1 = gated ? __ldg(a.ep.global1) : 0.f;
    asm volatile("bar.sync 10, %0;" ::"n"(kConsumerThreads + 32) : "memory");
    grid_dep_wait();                                        // before anything another kernel may write
    const bool all = q1 > q0 + 1;
    const bool wide = convert_rows<8 * NT, true>(a.x, a.ldx, smem + lay.x, a.T, a.K, a.KT, emax, low, [&](int kg) {
        const bool from = kg >= k0 / 2, to = kg <= (k1 - 1) / 2;
        return all || (q1 == q0 ? from && to : from || to);
    }, requested);
    const int joined = wide ? 0 : a.T;                      // columns of sums to finish

    uint32_t xa[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = 8 * n + (lane >> 2);
        xa[n] = ring.slots + lay.x + (uint32_t)(t < a.T ? t : 0) * row_bytes(a.KT);
    }
    WindowConsumer<NT> in(ring);
    Acc<NT> acc;
    // windows of the piece of row tile q
    auto windows = [&](int q) {
        const int ka = q == q0 ? k0 & ~(kWindow - 1) : 0, kb = q == q1 ? k1 : a.KT;
        return (kb - ka + kWindow - 1) / kWindow;
    };
    auto rest = [&](int q) { return q == q1 ? 0 : min(2, windows(q + 1) + (q + 1 < q1 ? 1 : 0)); };
    in.fetch(windows(q0) + rest(q0));
    const bool cut[2] = {k0 > 0 || (q0 == q1 && k1 < a.KT), q1 > q0 && k1 < a.KT};   // the first and the last piece
    for (int q = q0; q <= q1; ++q) {
        const int ka = q == q0 ? k0 : 0, kb = q == q1 ? k1 : a.KT;
        acc.clear();
        in.piece(ka, kb, rest(q), xa, true, acc);
        float *buf = sums + ((q - q0) & 1) * a.T * kSumStride;
        const int row0 = (warp & 7) * 16 + (lane >> 2), col0 = 2 * (lane & 3);
        if (kb - ka < a.KT) {
            float *mine = a.partial + (size_t)(2 * c + (q != q0)) * a.T * 128;
            join_pairs<NT>(acc, buf, joined, [&](int i, int j, float v) {
                const int col = 8 * i + col0 + (j & 1), row = row0 + 8 * (j >> 1);
                if (col < a.T) mine[col * 128 + row] = v * inverse_up(emax[col]);
            });
        } else if (gated) {
            join_pairs<NT>(acc, buf, joined, [&](int i, int j, float v) {
                const int col = 8 * i + col0 + (j & 1), row = row0 + 8 * (j >> 1);
                const float other = __shfl_xor_sync(0xffffffffu, v, 4);          // the neighbouring row
                const int n = (q * 128 + row) >> 1;
                if ((row & 1) || col >= a.T || n >= a.ep.N) return;
                const float inv = inverse_up(emax[col]);
                store_output(a.ep, col, n, finish_output(a.ep, col, n, v * inv, other * inv, g0, g1));
            });
        } else {
            join_pairs<NT>(acc, buf, joined, [&](int i, int j, float v) {
                const int col = 8 * i + col0 + (j & 1), row = row0 + 8 * (j >> 1);
                const int n = q * 128 + row;
                if (col < a.T && n < a.ep.N)
                    store_output(a.ep, col, n, finish_output(a.ep, col, n, v * inverse_up(emax[col]), 0.f, g0, g1));
            });
        }
    }
    if (wide) exact_pieces(a, q0, k0, q1, k1, sums, g0, g1);
    if (!cut[0] && !cut[1]) return;
    consumer_sync();
    if (threadIdx.x < 2) {
        int is_last = 0;
        __threadfence();                                    // the whole CTA's pieces, ordered by the barrier
        if (cut[threadIdx.x]) {
            const uint32_t q = threadIdx.x ? q1 : q0;
            const uint32_t ca = runs.owner(q * a.KT), cb = runs.owner((q + 1) * a.KT - 1);
            is_last = atomicAdd(a.tickets + q, 1) == (int)(cb - ca);
            if (is_last) a.tickets[q] = 0;                  // for the next call
            __threadfence();
            join[threadIdx.x][1] = (int)(2 * ca + (runs.first(ca) / a.KT != q));
            join[threadIdx.x][2] = (int)(2 * cb);
        }
        join[threadIdx.x][0] = is_last;
    }
    consumer_sync();
    for (int p = 0; p < 2; ++p) {
        if (!join[p][0]) continue;
        // the pieces of the tile: only its first CTA can have started before it, so the others' are their first
        const int pa = join[p][1], pb = join[p][2], stride = a.T * 32;   // in float4
        for (int i = threadIdx.x; i < a.T * 32; i += kConsumerThreads) {
            const float4 *src = reinterpret_cast<const float4 *>(a.partial) + i;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            int s0 = pa;
            do {
                float4 p4[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int s1 = j == 0 ? s0 : (s0 & ~1) + 2 * j;
                    if (s1 <= pb) p4[j] = __ldcg(src + (size_t)s1 * stride);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if ((j == 0 ? s0 : (s0 & ~1) + 2 * j) > pb) continue;
                    v.x += p4[j].x; v.y += p4[j].y; v.z += p4[j].z; v.w += p4[j].w;
                }
                s0 = (s0 & ~1) + 16;
            } while (s0 <= pb);
            *reinterpret_cast<float4 *>(sums + (i >> 5) * kSumStride + (i & 31) * 4) = v;
        }
        consumer_sync();
        finish_tile(a, p ? q1 : q0, sums, g0, g1);
        consumer_sync();
    }
}

constexpr int kSmemLimit = 227 * 1024 - 1024;   // the static part and the runtime's own 1 KB stay outside

int slots_for(int T, int KT) {
    const int left = kSmemLimit - (int)Layout(T, KT, 0).total;
    return std::min(kMaxSlots, left / kSlotBytes) & ~1;     // an even number: WindowConsumer
}

}  // namespace

// The streaming regime needs the token rows and a ring of at least 4 slots (74 KB: enough bytes in
// flight for HBM) in shared memory.
bool linear_stream_fits(const Linear &L, int T) { return T <= kMaxTokens && slots_for(T, L.KT) >= 4; }

// The estimated time of a call in clocks of an SM, to set beside the tcgen05 regime's: a start (token rows,
// first weights, joined tiles) that grows with the rows, and the SM's windows of the weight stream. Fitted to
// launches of 1 to 16 tokens over 12 matrices. With few windows and many rows tcgen05 wins (16 x 4096 x 2 x 2688:
// 10.9 us against 15.6), with many windows this regime (8 x 4096 x 32001: 22.7 us against 33.3).
double linear_stream_clocks(const Linear &L, int T) {
    const double windows = (double)L.RT * L.KT / L.num_sms / kWindow;
    return T <= 8 ? 13000.0 + 520.0 * (T - 1) + 830.0 * windows : 21500.0 + 190.0 * (T - 9) + 1250.0 * windows;
}

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
    a.test_wait_ns = L.test_timeout ? kLinearTestWaitNs : 0;
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
