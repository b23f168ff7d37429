// stream.cuh -- the weight stream of the few-token kernels (the NVFP4 matrix product's streaming
// regime, linear_stream.cu, and the one-kernel MoE layer, decode.cu).
//
// A few tokens times an NVFP4 matrix take the weight bytes over HBM bandwidth, so the work is
// cut by bytes: the matrix is a line of units of 128 rows x 64 columns (4608 bytes, contiguous in
// the tiled layout), and CTA c of G takes the units [c U / G, (c + 1) U / G). Every SM streams the
// same number of bytes, in a few long runs, whatever the matrix's shape. A run of units
// inside one row tile is a piece; a row tile cut by a CTA border has its pieces' sums added
// afterwards in CTA order, so equal calls give equal bits.
//
// One producer lane fills a ring of slots with bulk copies; a slot holds a group of one or two
// consecutive units of a piece. 16 consumer warps: warp w takes 16 rows (w mod 8) of the groups
// whose running number has the parity w / 8. The product runs on mma.sync m16n8k16 (f16 in, fp32
// sums), rows of weights against up to 8 tokens per instruction: the tensor core is idle most of
// the time either way, and this form needs no tensor memory round trip for a few tokens. What has
// to keep up with HBM (23 bytes = 41 weights per clock and SM) is the decode, one conversion
// and one scale multiplication per two weights; on CUDA cores the products would add an FMA per
// weight and token.
//
// The order of the reduction is free, so the lanes read what they can use: lane (g, t) = (l / 4,
// l % 4) owns rows g and g + 8 and the t-th 32-column half of the group: one 16-byte load per row,
// and chunk i (8 columns) of every lane's half forms the k indices of two instructions. The
// halves are copied 32 bytes apart from a multiple of 128 (and the second unit's scales
// likewise), which spreads the four lanes of a row over the banks. Token operands are stored
// in that order too: [128 columns][chunk 0..3][half 0..3][8 values].
#pragma once

#include "common.cuh"
#include "internal.h"

namespace tfmoe {
namespace stream {

constexpr int kConsumers = 16;                           // warps
constexpr int kConsumerThreads = 32 * kConsumers;
constexpr int kThreads = kConsumerThreads + 32;          // + the producer warp
constexpr int kHalfStride = kTileCodeBytes / 2 + 32;     // 2080
constexpr int kScaleAt = 4 * kHalfStride;                // 8320
constexpr int kScaleStride = kTileScaleBytes + 32;       // 544
constexpr int kSlotBytes = kScaleAt + kScaleStride + kTileScaleBytes;   // 9376
static_assert(kSlotBytes % 16 == 0, "bulk copies need 16-byte aligned slots");
constexpr int kMaxSlots = 24;
constexpr int kMaxTokens = 16;                           // two n = 8 tiles

// Shared-memory bytes of one token's operand row for K = 64 KT columns. The 64 bytes at the
// end put consecutive rows on the other half of the banks.
__host__ __device__ constexpr uint32_t row_bytes(int KT) { return (uint32_t)((KT + 1) / 2) * 256u + 64u; }
// Byte offset of the 8-value chunk holding column k (a multiple of 8) inside its row.
__host__ __device__ constexpr uint32_t chunk_offset(int k) {
    return (uint32_t)(k >> 7) * 256u + (uint32_t)((k >> 3) & 3) * 64u + (uint32_t)((k >> 5) & 3) * 16u;
}

// First unit of CTA c, and the CTA that owns unit u, when U units are cut into G runs.
__host__ __device__ __forceinline__ uint32_t first_unit(uint32_t c, uint32_t U, uint32_t G) {
    return (uint32_t)((uint64_t)c * U / G);
}
__host__ __device__ __forceinline__ uint32_t owner(uint32_t u, uint32_t U, uint32_t G) {
    return (uint32_t)((((uint64_t)u + 1) * G - 1) / U);
}

struct Ring {
    uint32_t slots, full, empty;          // shared addresses
    uint32_t zeros;                       // shared address of 256 zero bytes
    int n;                                // slots in use
    volatile int32_t *abort_flag;         // shared
    int32_t *err_word;                    // global
};

// Bounded wait: false once another thread has given up or after kWaitLimitNs (recorded).
__device__ __forceinline__ bool wait(const Ring &r, uint32_t bar, uint32_t parity) {
    if (mbar_try_wait_at(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        for (int i = 0; i < 4; ++i)
            if (mbar_try_wait_sleep_at(bar, parity)) return true;
        if (*r.abort_flag) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            atomicOr(r.err_word, DEV_ERR_WAIT_TIMEOUT);
            *r.abort_flag = 1;
            return false;
        }
    }
}

// Slot and phase of a running group number, advanced without dividing.
struct Cursor {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void advance(int by, int n) {
        slot += by;
        while (slot >= n) { slot -= n; phase ^= 1u; }
    }
};

__device__ __forceinline__ void bulk_at(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// The producer's side: put one piece (units consecutive units from `codes` / `scales`) into the
// ring. `issued` counts the groups. Returns false after an abort.
__device__ __forceinline__ bool produce_piece(const Ring &r, Cursor &c, uint32_t &issued, const uint8_t *codes,
                                              const uint8_t *scales, int units) {
    for (int u = 0; u < units; u += 2) {
        const int n = min(2, units - u);
        const uint32_t full = r.full + 8u * c.slot, slot = r.slots + (uint32_t)c.slot * kSlotBytes;
        if (issued >= (uint32_t)r.n && !wait(r, r.empty + 8u * c.slot, c.phase ^ 1u)) return false;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                     ::"r"(full), "r"((uint32_t)n * (kTileCodeBytes + kTileScaleBytes)) : "memory");
        for (int i = 0; i < n; ++i) {
            const uint8_t *cp = codes + (size_t)(u + i) * kTileCodeBytes;
            bulk_at(slot + (2 * i) * kHalfStride, cp, kTileCodeBytes / 2, full);
            bulk_at(slot + (2 * i + 1) * kHalfStride, cp + kTileCodeBytes / 2, kTileCodeBytes / 2, full);
            bulk_at(slot + kScaleAt + i * kScaleStride, scales + (size_t)(u + i) * kTileScaleBytes, kTileScaleBytes,
                    full);
        }
        c.advance(1, r.n);
        ++issued;
    }
    return true;
}

// After an abort: let the copies still in flight land (bounded) before the CTA exits.
__device__ __forceinline__ void drain(const Ring &r, const Cursor &end, uint32_t issued) {
    const int k = (int)min(issued, (uint32_t)r.n);
    Cursor c = end;
    for (int i = 0; i < k; ++i) {
        if (c.slot == 0) { c.slot = r.n; c.phase ^= 1u; }
        --c.slot;
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait_sleep_at(r.full + 8u * c.slot, c.phase) && global_timer_ns() - t0 < kWaitLimitNs / 4) {
        }
    }
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, __half2 b) {
    const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&a), b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Sums of one warp: 16 rows x 8 NT tokens, two sets that alternate so that consecutive
// instructions do not wait for one another. Lane (g, t): rows g (c[0..1]) and g + 8 (c[2..3]),
// tokens 2t and 2t + 1 of the tile.
template <int NT>
struct Acc {
    float c[2][NT][4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) c[i][n][j] = 0.f;
    }
    __device__ __forceinline__ float sum(int n, int j) const { return c[0][n][j] + c[1][n][j]; }
};

// One group: `units` (1 or 2) units whose first column tile is kt. xa: the lane's token row per
// n-tile (token 8 n + g; any valid row where there is no such token). Products E2M1 * E4M3 are
// exact in f16 (at most 6 significant bits, 2^-10 to 2688).
template <int NT>
__device__ __forceinline__ void consume_group(uint32_t slot, int units, int kt, int rows16, const uint32_t (&xa)[NT],
                                              uint32_t zeros, Acc<NT> &acc) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const bool live = (t >> 1) < units;
    const uint32_t code = slot + (uint32_t)t * kHalfStride + (uint32_t)(rows16 + g) * 16u;
    const uint32_t scale = slot + kScaleAt + (uint32_t)(t >> 1) * kScaleStride + (uint32_t)(rows16 + g) * 4u + (t & 1) * 2u;
    const int kl = kt + (t >> 1);
    const uint32_t xo = (uint32_t)(kl >> 1) * 256u + (uint32_t)((kl & 1) * 2 + (t & 1)) * 16u;
    const uint4 c0 = lds128(code), c1 = lds128(code + 128);
    // a lane without a unit multiplies zeros by zero scales (zero times what an earlier group or an
    // infinite activation left there could be a NaN)
    const uint32_t s0 = live ? lds16(scale) : 0u, s1 = live ? lds16(scale + 32) : 0u;
    const uint32_t h0 = e4m3x2_to_f16x2(s0), h1 = e4m3x2_to_f16x2(s1);
    const __half2 v0 = *reinterpret_cast<const __half2 *>(&h0), v1 = *reinterpret_cast<const __half2 *>(&h1);
    const __half2 sc0[2] = {__low2half2(v0), __high2half2(v0)}, sc1[2] = {__low2half2(v1), __high2half2(v1)};
    const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a[4], b[4];
        e2m1x8_to_f16x2x4(w0[i], a);
        e2m1x8_to_f16x2x4(w1[i], b);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = mul_f16x2(a[j], sc0[i >> 1]);
            b[j] = mul_f16x2(b[j], sc1[i >> 1]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 x = lds128((live ? xa[n] + xo : zeros) + 64u * i);
            mma_f16(acc.c[0][n], a[0], b[0], a[1], b[1], x.x, x.y);
            mma_f16(acc.c[1][n], a[2], b[2], a[3], b[3], x.z, x.w);
        }
    }
}

// One piece: this warp's share of its groups. `c` is at the piece's first group, whose running
// number has parity `par0`.
template <int NT>
__device__ __forceinline__ void consume_piece(const Ring &r, Cursor &c, uint32_t &par0, int kt, int units,
                                              const uint32_t (&xa)[NT], Acc<NT> &acc) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rows16 = (warp & 7) * 16;
    const int groups = (units + 1) / 2;
    int first = (int)((uint32_t)(warp >> 3) ^ par0);       // 0 or 1: the warp's first group
    Cursor my = c;
    if (first) my.advance(1, r.n);
    for (int gi = first; gi < groups; gi += 2) {
        wait(r, r.full + 8u * my.slot, my.phase);
        __syncwarp();
        consume_group<NT>(r.slots + (uint32_t)my.slot * kSlotBytes, min(2, units - 2 * gi), kt + 2 * gi, rows16, xa,
                          r.zeros, acc);
        __syncwarp();
        if (lane == 0) mbar_arrive_at(r.empty + 8u * my.slot);
        my.advance(2, r.n);
    }
    c.advance(groups, r.n);
    par0 ^= (uint32_t)groups & 1u;
}

// Barrier among the consumer warps.
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumerThreads) : "memory"); }

// Add the two parities' sums of a piece: sums[token][row] (stride kSumStride floats) for `m`
// tokens. Ends with a consumer barrier, after which every consumer may read it; the next call
// must come after another barrier.
constexpr int kSumStride = 132;
template <int NT>
__device__ __forceinline__ void join_parities(const Acc<NT> &acc, float *sums, int m) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int row = (warp & 7) * 16 + g;
    for (int par = 1; par >= 0; --par) {
        if ((warp >> 3) == par) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int col = 8 * n + 2 * t + (j & 1);
                    if (col >= m) continue;
                    float *p = sums + col * kSumStride + row + 8 * (j >> 1);
                    *p = par ? acc.sum(n, j) : *p + acc.sum(n, j);
                }
        }
        consumer_sync();
    }
}

// Eight bf16 values (as loaded) times `up`, rounded to f16.
__device__ __forceinline__ uint4 bf16x8_to_f16(const uint4 &v, float up) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 h = __floats2half2_rn(bf16_bits_to_float(u[j] & 0xFFFFu) * up, bf16_bits_to_float(u[j] >> 16) * up);
        o[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ uint32_t max_exponent(const uint4 &v) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    uint32_t e = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) e = max(e, max((u[j] >> 7) & 0xFFu, (u[j] >> 23) & 0xFFu));
    return e;
}
// The power of two that brings a row whose largest exponent field is emax just below 2^15, as the
// exponent field of its float; the inverse's field is 254 minus it.
__device__ __forceinline__ int up_field(uint32_t emax) {
    return 127 + max(-120, min(120, 14 - ((int)emax - 127)));
}

}  // namespace stream
}  // namespace tfmoe
