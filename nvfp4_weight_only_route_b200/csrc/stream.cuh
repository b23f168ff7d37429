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
// One producer lane fills a ring of slots with bulk copies; a slot holds the units of a piece whose
// column tiles lie in one aligned window of four (two copies: a bulk copy costs the issuing
// lane about 100 clocks, so small ones would set the pace). 16 consumer warps: warp w takes 16 rows
// (w mod 8) of pair w / 8 of every window. The product runs on mma.sync m16n8k16 (f16 in, fp32
// sums), rows of weights against up to 8 tokens per instruction: the tensor core is idle most of
// the time either way, and this form needs no tensor memory round trip for a few tokens. What has
// to keep up with HBM (23 bytes = 41 weights per clock and SM) is the decode, one conversion
// and one scale multiplication per two weights: measured alone, two units take 272 clocks of an SM
// (8 tokens) or 405 (16 tokens) against 400 at HBM speed. On CUDA cores the products would add an
// FMA per weight and token.
//
// The order of the reduction is free, so the lanes read what they can use: lane (g, t) = (l / 4,
// l % 4) owns rows g and g + 8 and the t-th 32-column half of the pair, four chunks of 8 columns (one
// word of codes each) in the order t, t + 1, t + 2, t + 3 (mod 4), which puts the 32 lanes on
// different banks. Chunk i of every lane forms the k indices of two instructions. Token operands
// are stored in that order too: [128 columns][step 0..3][half 0..3][8 values].
#pragma once

#include "common.cuh"
#include "internal.h"

namespace tfmoe {
namespace stream {

constexpr int kConsumers = 16;                           // warps
constexpr int kConsumerThreads = 32 * kConsumers;
constexpr int kThreads = kConsumerThreads + 32;          // + the producer warp
constexpr int kWindow = 4;                               // column tiles per slot
constexpr int kScaleAt = kWindow * kTileCodeBytes;       // 16384
constexpr int kSlotBytes = kScaleAt + kWindow * kTileScaleBytes;   // 18432
static_assert(kSlotBytes % 128 == 0, "bulk copies need 16-byte aligned slots");
constexpr int kMaxSlots = 12;
constexpr int kMaxTokens = 16;                           // two n = 8 tiles

// Shared-memory bytes of one token's operand row for K = 64 KT columns. The 64 bytes at the
// end put consecutive rows on the other half of the banks.
__host__ __device__ constexpr uint32_t row_bytes(int KT) { return (uint32_t)((KT + 1) / 2) * 256u + 64u; }
// Byte offset of the 8-value chunk holding column k (a multiple of 8) inside its row.
__host__ __device__ constexpr uint32_t chunk_offset(int k) {
    return (uint32_t)(k >> 7) * 256u + (uint32_t)(((k >> 3) - (k >> 5)) & 3) * 64u + (uint32_t)((k >> 5) & 3) * 16u;
}

// First unit of CTA c, and the CTA that owns unit u, when U units are cut into G runs. The
// handles keep U below 2^24 and G is the SM count, so the products fit 32 bits.
__host__ __device__ __forceinline__ uint32_t first_unit(uint32_t c, uint32_t U, uint32_t G) { return c * U / G; }
__host__ __device__ __forceinline__ uint32_t owner(uint32_t u, uint32_t U, uint32_t G) { return ((u + 1) * G - 1) / U; }

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
        if (slot >= n) { slot -= n; phase ^= 1u; }
    }
};

__device__ __forceinline__ void bulk_at(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// The producer's side: put the column tiles [ka, kb) of one row tile into the ring, whose codes
// and scales start at `codes` and `scales` (those of column tile 0); before(n) runs ahead of the n-th
// slot. Returns false after an abort.
template <class Before>
__device__ __forceinline__ bool produce_piece(const Ring &r, Cursor &c, uint32_t &issued, const uint8_t *codes,
                                              const uint8_t *scales, int ka, int kb, Before before) {
    for (int k = ka; k < kb;) {
        before(issued);
        const int at = k % kWindow, n = min(kWindow - at, kb - k);
        const uint32_t full = r.full + 8u * c.slot, slot = r.slots + (uint32_t)c.slot * kSlotBytes;
        if (issued >= (uint32_t)r.n && !wait(r, r.empty + 8u * c.slot, c.phase ^ 1u)) return false;
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                     ::"r"(full), "r"((uint32_t)n * (kTileCodeBytes + kTileScaleBytes)) : "memory");
        bulk_at(slot + at * kTileCodeBytes, codes + (size_t)k * kTileCodeBytes, n * kTileCodeBytes, full);
        bulk_at(slot + kScaleAt + at * kTileScaleBytes, scales + (size_t)k * kTileScaleBytes, n * kTileScaleBytes, full);
        c.advance(1, r.n);
        ++issued;
        k += n;
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
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
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

// What a consumer lane needs of its place, computed once.
struct Lane {
    uint32_t code[4];      // offsets of the lane's four words of row g inside a window's pair, step by step
    uint32_t scale;        // offset of row g's two scale bytes
    uint32_t sel[2];       // prmt selectors: (scale of step 0, of step 2), (of step 1, of step 3)
    uint32_t x;            // offset inside 128 columns of a token row
    int unit;              // the lane's unit of a window
    __device__ __forceinline__ Lane() {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int row = (warp & 7) * 16 + g;
        unit = 2 * (warp >> 3) + (t >> 1);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            code[i] = (uint32_t)(unit * kTileCodeBytes + (t & 1) * (kTileCodeBytes / 2) + row * 16 + ((i + t) & 3) * 4);
        scale = (uint32_t)(kScaleAt + unit * kTileScaleBytes + row * 4 + (t & 1) * 2);
        sel[0] = (t >> 1) ? 0x1032u : 0x3210u;               // steps 0 and 2 are in different 16-column blocks,
        sel[1] = (((1 + t) & 3) >> 1) ? 0x1032u : 0x3210u;   // and so are steps 1 and 3
        x = (uint32_t)(warp >> 3) * 256u + (uint32_t)t * 16u;
    }
};

// The codes and scales of the lane's rows of one pair, in registers.
struct Pair {
    uint32_t w0[4], w1[4], s0, s1;
    __device__ __forceinline__ void load(uint32_t slot, const Lane &ln) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w0[i] = lds32(slot + ln.code[i]);
            w1[i] = lds32(slot + ln.code[i] + 128u);
        }
        s0 = lds16(slot + ln.scale);
        s1 = lds16(slot + ln.scale + 32u);
    }
};

// One pair of a window. x: the lane's operands (token 8 n + g; any valid row where there is no such
// token) at the pair's columns. Products E2M1 * E4M3 are exact in f16 (at most 6 significant
// bits, 2^-10 to 2688).
template <int NT>
__device__ __forceinline__ void consume_pair(const Pair &p, const Lane &ln, const uint32_t (&x)[NT], Acc<NT> &acc) {
    const uint32_t h0 = e4m3x2_to_f16x2(p.s0), h1 = e4m3x2_to_f16x2(p.s1);
    __half2 v0[2], v1[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t a = __byte_perm(h0, 0, ln.sel[j]), b = __byte_perm(h1, 0, ln.sel[j]);
        v0[j] = *reinterpret_cast<const __half2 *>(&a);
        v1[j] = *reinterpret_cast<const __half2 *>(&b);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a[4], b[4];
        e2m1x8_to_f16x2x4(p.w0[i], a);
        e2m1x8_to_f16x2x4(p.w1[i], b);
        const __half2 sa = i < 2 ? __low2half2(v0[i & 1]) : __high2half2(v0[i & 1]);
        const __half2 sb = i < 2 ? __low2half2(v1[i & 1]) : __high2half2(v1[i & 1]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = mul_f16x2(a[j], sa);
            b[j] = mul_f16x2(b[j], sb);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint4 xv = lds128(x[n] + 64u * i);
            mma_f16(acc.c[0][n], a[0], b[0], a[1], b[1], xv.x, xv.y);
            mma_f16(acc.c[1][n], a[2], b[2], a[3], b[3], xv.z, xv.w);
        }
    }
}

// One piece, the column tiles [ka, kb) of a row tile: this warp's share of its windows. xa: the
// lane's token rows. Whole windows run two at a time: the next one's codes are read (and its slot
// handed back) before the current one is multiplied.
template <int NT>
__device__ __forceinline__ void consume_piece(const Ring &r, Cursor &c, const Lane &ln, int ka, int kb,
                                              const uint32_t (&xa)[NT], Acc<NT> &acc) {
    const int lane = threadIdx.x & 31;
    int w = ka & ~(kWindow - 1);
    uint32_t x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) x[n] = xa[n] + ln.x + (uint32_t)w * 128u;
    auto step = [&]() {
        w += kWindow;
#pragma unroll
        for (int n = 0; n < NT; ++n) x[n] += kWindow * 128u;
    };
    auto fetch = [&](Pair &p) {
        wait(r, r.full + 8u * c.slot, c.phase);
        p.load(r.slots + (uint32_t)c.slot * kSlotBytes, ln);
        __syncwarp();
        if (lane == 0) mbar_arrive_at(r.empty + 8u * c.slot);
        c.advance(1, r.n);
    };
    // a window of which the piece has only some units: a lane without a unit multiplies zeros by zero
    // scales (zero times what an earlier window or an infinite activation left there could be a NaN)
    auto part = [&]() {
        Pair p;
        fetch(p);
        const bool live = w + ln.unit >= ka && w + ln.unit < kb;
        if (!live) p.s0 = p.s1 = 0u;
        uint32_t xl[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) xl[n] = live ? x[n] : r.zeros;
        if (__any_sync(0xffffffffu, live)) consume_pair<NT>(p, ln, xl, acc);
        step();
    };
    if (w < ka || w + kWindow > kb) part();
    int whole = (kb - w) / kWindow;
    if (whole > 0) {
        Pair p0, p1;
        fetch(p0);
        for (; whole >= 2; whole -= 2) {
            fetch(p1);
            consume_pair<NT>(p0, ln, x, acc);
            step();
            if (whole > 2) fetch(p0);
            consume_pair<NT>(p1, ln, x, acc);
            step();
        }
        if (whole) {
            consume_pair<NT>(p0, ln, x, acc);
            step();
        }
    }
    if (w < kb) part();
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
// Largest magnitude bits of eight bf16 values, in both halves of a word (not yet joined).
__device__ __forceinline__ uint32_t max_bits(const uint4 &v, uint32_t m) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(u[j] & 0x7FFF7FFFu));
    return m;
}
// The power of two that brings a row whose largest exponent field is emax just below 2^15, as the
// exponent field of its float; the inverse's field is 254 minus it.
__device__ __forceinline__ int up_field(uint32_t emax) {
    return 127 + max(-120, min(120, 14 - ((int)emax - 127)));
}
__device__ __forceinline__ float up_of(uint32_t emax) { return __uint_as_float((uint32_t)up_field(emax) << 23); }
__device__ __forceinline__ float inverse_up(uint32_t emax) {
    return __uint_as_float((uint32_t)(254 - up_field(emax)) << 23);
}

// T bf16 rows of K values in global memory (ld apart, 16-byte aligned) become operand rows in shared
// memory (row_bytes(KT) apart), by all consumers: f16 times a power of two per row (exact for every
// element within 2^28 of the row's largest; smaller ones are rounded to 2^-39 of it), columns from K
// on zero. Only the 128-column groups for which used(group) holds are read and written. emax[t] (zero
// before) receives the rows' largest exponent fields. Ends with a consumer barrier. A thread
// keeps up to kHeld chunks in registers between finding the maximum and converting; what lies beyond
// is read again. requested: an
// mbarrier that every consumer warp arrives at once its first loads are on the way.
template <int kHeld, class Used>
__device__ __forceinline__ void convert_rows(const uint16_t *x, int64_t ld, uint8_t *rows, int T, int K, int KT,
                                             uint32_t *emax, Used used, uint32_t requested = 0) {
    const int chunks = ((KT + 1) / 2) * 16;
    int tpr = kConsumerThreads;                              // threads per row, at least a warp
    while (tpr * T > kConsumerThreads) tpr >>= 1;
    const int t = threadIdx.x / tpr, i0 = threadIdx.x % tpr;
    const uint4 *row = reinterpret_cast<const uint4 *>(x + (int64_t)t * ld);
    uint4 v[kHeld];
    if (t < T) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            const int i = i0 + j * tpr;
            v[j] = i * 8 < K && used(i >> 4) ? row[i] : make_uint4(0, 0, 0, 0);
        }
    }
    if (requested && (threadIdx.x & 31) == 0) mbar_arrive_at(requested);
    if (t < T) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < kHeld; ++j) m = max_bits(v[j], m);
#pragma unroll 4
        for (int i = i0 + kHeld * tpr; i * 8 < K; i += tpr)
            if (used(i >> 4)) m = max_bits(row[i], m);
        const uint32_t e = __reduce_max_sync(0xffffffffu, max(m >> 23, (m >> 7) & 0xFFu));
        if ((threadIdx.x & 31) == 0) atomicMax(&emax[t], e);
    }
    consumer_sync();
    if (t < T) {
        const float up = up_of(emax[t]);
        uint8_t *dst = rows + t * row_bytes(KT);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            const int i = i0 + j * tpr;
            if (i < chunks && used(i >> 4)) *reinterpret_cast<uint4 *>(dst + chunk_offset(i * 8)) = bf16x8_to_f16(v[j], up);
        }
#pragma unroll 4
        for (int i = i0 + kHeld * tpr; i < chunks; i += tpr)
            if (used(i >> 4))
                *reinterpret_cast<uint4 *>(dst + chunk_offset(i * 8)) =
                    i * 8 < K ? bf16x8_to_f16(row[i], up) : make_uint4(0, 0, 0, 0);
    }
    consumer_sync();
}

}  // namespace stream
}  // namespace tfmoe
