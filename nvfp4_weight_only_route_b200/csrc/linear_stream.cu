// linear_stream.cu -- the streaming regime of the NVFP4 matrix product: up to 16 tokens, bound by
// the weight bytes over HBM bandwidth (stream.cuh has the stream and the arithmetic).
//
// The x rows become f16 times a power of two per row and CTA (exact for every element within
// 2^28 of the largest one the CTA uses; smaller ones are rounded to 2^-39 of the largest) and stay
// in shared memory. A row tile that one CTA owns is finished there. One that is cut by CTA borders
// leaves its pieces' sums in global memory, and the CTA that arrives last at the tile's counter
// adds them in CTA order and finishes it: no CTA waits for another, so the launch needs no
// co-residency, and equal calls give equal bits.
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
        total = bars + 2 * kMaxSlots * 8 + 16;
    }
};

// Outputs of row tile rt from sums[token][row] (per-token factor 2^-sh in inv).
__device__ __forceinline__ void finish_tile(const StreamArgs &a, int rt, const float *sums, const uint32_t *emax) {
    const bool gated = a.ep.act == TFMOE_ACT_SWIGLU;
    const float g0 = __ldg(a.ep.global0), g1 = gated ? __ldg(a.ep.global1) : 0.f;
    const int per = gated ? 64 : 128;
    for (int i = threadIdx.x; i < a.T * per; i += kConsumerThreads) {
        const int t = i / per, j = i % per, n = rt * per + j;
        if (n >= a.ep.N) continue;
        const float inv = emax ? __uint_as_float((uint32_t)(254 - up_field(emax[t])) << 23) : 1.f;
        const float *s = sums + t * kSumStride + (gated ? 2 * j : j);
        store_output(a.ep, t, n, finish_output(a.ep, t, n, s[0] * inv, gated ? s[1] * inv : 0.f, g0, g1));
    }
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1) linear_stream_kernel(const StreamArgs a)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int is_last;
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
    ring.abort_flag = reinterpret_cast<volatile int32_t *>(bars + 2 * kMaxSlots);
    ring.err_word = a.err_word;
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.slots; ++i) {
            mbar_init(bars + i, 1);
            mbar_init(bars + kMaxSlots + i, kConsumers / 2);
        }
        *ring.abort_flag = 0;
        fence_mbar_init();
    }
    if (threadIdx.x < kMaxTokens) emax[threadIdx.x] = 0;
    if (threadIdx.x < 64) reinterpret_cast<uint32_t *>(smem + lay.zeros)[threadIdx.x] = 0;
    __syncthreads();

    const uint32_t G = gridDim.x, c = blockIdx.x, U = (uint32_t)a.RT * a.KT;
    const uint32_t u0 = first_unit(c, U, G), u1 = first_unit(c + 1, U, G);
    const int q0 = (int)(u0 / a.KT), k0 = (int)(u0 % a.KT);           // u0 < u1: G <= U
    const int q1 = (int)((u1 - 1) / a.KT), k1 = (int)((u1 - 1) % a.KT) + 1;
    if (warp == kConsumers) {
        if (lane == 0) {
            Cursor cur;
            uint32_t issued = 0;
            bool ok = true;
            for (int q = q0; q <= q1 && ok; ++q) {
                const int ka = q == q0 ? k0 : 0, kb = q == q1 ? k1 : a.KT;
                const size_t tile = (size_t)q * a.KT + ka;
                ok = produce_piece(ring, cur, issued, a.codes + tile * kTileCodeBytes, a.scales + tile * kTileScaleBytes,
                                   kb - ka);
            }
            if (*ring.abort_flag) drain(ring, cur, issued);
        }
        return;
    }

    // x -> f16 rows in shared memory, for the column groups (128 columns) this CTA uses
    {
        const int KG = (a.KT + 1) / 2, chunks = KG * 16;
        const bool all = q1 > q0 + 1;
        auto used = [&](int kg) {
            if (all) return true;
            if (q1 == q0) return kg >= k0 / 2 && kg <= (k1 - 1) / 2;
            return kg >= k0 / 2 || kg <= (k1 - 1) / 2;
        };
        int tpr = kConsumerThreads;                         // threads per row
        while (tpr * a.T > kConsumerThreads) tpr >>= 1;
        const int t = threadIdx.x / tpr, i0 = threadIdx.x % tpr;
        const uint16_t *row = a.x + (int64_t)t * a.ldx;
        uint32_t e = 0;
        if (t < a.T)
            for (int i = i0; i < chunks; i += tpr)
                if (i * 8 < a.K && used(i >> 4)) e = max(e, max_exponent(__ldg(reinterpret_cast<const uint4 *>(row + i * 8))));
        e = __reduce_max_sync(0xffffffffu, e);              // tpr is at least 32: a warp serves one row
        if (lane == 0 && t < a.T) atomicMax(&emax[t], e);
        consumer_sync();
        if (t < a.T) {
            const float up = __uint_as_float((uint32_t)up_field(emax[t]) << 23);
            uint8_t *dst = smem + lay.x + t * row_bytes(a.KT);
            for (int i = i0; i < chunks; i += tpr)
                if (used(i >> 4))
                    *reinterpret_cast<uint4 *>(dst + chunk_offset(i * 8)) =
                        i * 8 < a.K ? bf16x8_to_f16(__ldg(reinterpret_cast<const uint4 *>(row + i * 8)), up)
                                    : make_uint4(0, 0, 0, 0);
        }
        consumer_sync();
    }

    uint32_t xa[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int t = 8 * n + (lane >> 2);
        xa[n] = smem_u32(smem + lay.x) + (uint32_t)(t < a.T ? t : 0) * row_bytes(a.KT);
    }
    Cursor cur;
    uint32_t par = 0;
    Acc<NT> acc;
    for (int q = q0; q <= q1; ++q) {
        const int ka = q == q0 ? k0 : 0, kb = q == q1 ? k1 : a.KT;
        acc.clear();
        consume_piece<NT>(ring, cur, par, ka, kb - ka, xa, acc);
        join_parities<NT>(acc, sums, a.T);
        if (kb - ka == a.KT) {
            finish_tile(a, q, sums, emax);
            consumer_sync();                                // sums are free again
            continue;
        }
        // a cut row tile: leave the piece, and add the pieces if this CTA is the tile's last
        float *mine = a.partial + (size_t)(2 * c + (q != q0)) * a.T * 128;
        for (int i = threadIdx.x; i < a.T * 128; i += kConsumerThreads) {
            const int t = i >> 7;
            mine[i] = sums[t * kSumStride + (i & 127)] * __uint_as_float((uint32_t)(254 - up_field(emax[t])) << 23);
        }
        __threadfence();
        consumer_sync();
        const uint32_t ca = owner((uint32_t)q * a.KT, U, G), cb = owner((uint32_t)(q + 1) * a.KT - 1, U, G);
        if (threadIdx.x == 0) {
            is_last = atomicAdd(a.tickets + q, 1) == (int)(cb - ca);
            if (is_last) a.tickets[q] = 0;                  // for the next call
            __threadfence();
        }
        consumer_sync();
        if (is_last) {
            for (int i = threadIdx.x; i < a.T * 128; i += kConsumerThreads) {
                float v = 0.f;
                for (uint32_t cc = ca; cc <= cb; ++cc) {
                    const uint32_t s = 2 * cc + (first_unit(cc, U, G) / a.KT != (uint32_t)q);
                    v += __ldcg(a.partial + (size_t)s * a.T * 128 + i);
                }
                sums[(i >> 7) * kSumStride + (i & 127)] = v;
            }
            consumer_sync();
            finish_tile(a, q, sums, nullptr);
        }
        consumer_sync();
    }
}

constexpr int kSmemLimit = 227 * 1024 - 1024;   // the static part and the runtime's own 1 KB stay outside

int slots_for(int T, int KT) {
    const int left = kSmemLimit - (int)Layout(T, KT, 0).total;
    return std::min(kMaxSlots, left / kSlotBytes);
}

}  // namespace

// The streaming regime needs the token rows and a ring of at least 8 slots (75 KB: enough bytes in
// flight for HBM) in shared memory.
bool linear_stream_fits(const Linear &L, int T) { return T <= kMaxTokens && slots_for(T, L.KT) >= 8; }

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
    if (T <= 8) linear_stream_kernel<1><<<grid, kThreads, smem, s>>>(a);
    else linear_stream_kernel<2><<<grid, kThreads, smem, s>>>(a);
    *launches += 1;
    return cudaGetLastError();
}

}  // namespace tfmoe
