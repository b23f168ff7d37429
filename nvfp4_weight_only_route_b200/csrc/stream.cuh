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
// (w mod 8), and the two groups of 8 share the windows (the consumers' classes below); the two warps of a row group add
// their sums at the end of a piece. (Two groups that take whole pieces in turn need no joining, but leave 8
// warps to keep up with HBM: the 14-token wide layer took 216 us instead of 188.)
// The product runs on mma.sync m16n8k16 (f16 in, fp32 sums), rows of weights against up to 8 tokens
// per instruction: the tensor core is idle most of the time either way, and this form needs no
// tensor memory round trip for a few tokens. What has to keep up with HBM (23 bytes = 41 weights
// per clock and SM) is the decode, one conversion (measured: 36 lanes per clock and SM) and one
// scale multiplication per two weights: a window needs about 570 clocks of an SM's conversions against
// 800 at HBM speed. On CUDA cores the products would add an FMA per weight and token.
//
// The order of the reduction is free, so the lanes read what they can use: lane (g, t) = (l / 4,
// l % 4) owns rows g and g + 8 and the t-th 32-column half of a pair of units, four chunks of 8 columns
// (one word of codes each); step i takes chunk i xor t, which puts the 32 lanes on different banks.
// The chunks of a step form the k indices of two instructions. Token operands are stored in that
// order too: [128 columns][step 0..3][half 0..3][8 values].
#pragma once

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace tfmoe {
namespace stream {

constexpr int kConsumers = 16;                           // warps
constexpr int kConsumerThreads = 32 * kConsumers;
constexpr int kThreads = kConsumerThreads + 128;         // + the producer's warpgroup, of which one lane works
// A scheduler's four consumer warps and its share of the producer's group: 640 threads start with 96
// registers each (61440 in all); the consumers take 112, the producer's warps keep 24 (60416).
constexpr int kConsumerRegs = 112, kProducerRegs = 24;
static_assert(kConsumerThreads * kConsumerRegs + 128 * kProducerRegs <= kThreads * 96, "register split");
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs)); }
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs)); }
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
    return (uint32_t)(k >> 7) * 256u + (uint32_t)(((k >> 3) ^ (k >> 5)) & 3) * 64u + (uint32_t)((k >> 5) & 3) * 16u;
}

// U units cut into G runs: the first unit of run c, and the run that holds unit u. The handles keep
// U at 2^24 or less (256 experts of 16384 x 16384) and G is at most the SM count, so the products fit 32 bits. A quotient below G is
// found by one multiplication with the reciprocal (relative error below 2^-22) and a correction.
struct Runs {
    uint32_t U, G;
    float rcp;
    __device__ __forceinline__ Runs(uint32_t units, uint32_t most) : U(units), G(min(units, most)), rcp(1.0f / (float)units) {}
    __device__ __forceinline__ uint32_t first(uint32_t c) const { return c * U / G; }
    __device__ __forceinline__ uint32_t end(uint32_t c) const { return c < G ? first(c + 1) : 0u; }
    __device__ __forceinline__ uint32_t owner(uint32_t u) const {
        const uint32_t n = (u + 1) * G - 1;
        uint32_t q = (uint32_t)((float)n * rcp);
        const int r = (int)(n - q * U);                    // within +-U: fits
        if (r < 0) --q;
        else if ((uint32_t)r >= U) ++q;
        return q;
    }
};

struct Ring {
    uint32_t slots, full, empty;          // shared addresses
    uint32_t zeros;                       // shared address of 256 zero bytes
    int n;                                // slots in use
    bool early;                           // the kernel may have started before the one ahead of it has ended
    volatile int32_t *abort_flag;         // shared
    int32_t *err_word;                    // global
};

// Bounded wait: false once another thread has given up or after kWaitLimitNs (recorded). In a kernel that started
// early the time of the kernel ahead does not count: when the limit passes, that one is waited for and the
// clock set back, once.
__device__ __forceinline__ bool wait(const Ring &r, uint32_t bar, uint32_t parity) {
    if (mbar_try_wait_at(bar, parity)) return true;
    uint64_t t0 = global_timer_ns();
    bool again = r.early;
    while (true) {
        for (int i = 0; i < 4; ++i)
            if (mbar_try_wait_sleep_at(bar, parity)) return true;
        if (*r.abort_flag) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            if (again) {
                again = false;
                grid_dep_wait();
                t0 = global_timer_ns();
                continue;
            }
            atomicOr(r.err_word, DEV_ERR_WAIT_TIMEOUT);
            *r.abort_flag = 1;
            return false;
        }
    }
}

// The same by a whole warp, which goes on together.
__device__ __forceinline__ void wait_warp(const Ring &r, uint32_t bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait_at(bar, parity))) return;
    wait(r, bar, parity);
    __syncwarp();
}

// A value that is the same in every lane, in a form the compiler takes as such: loops and branches on
// values from shared memory are otherwise compiled for lanes that may part, which slowed the
// product's loop by half.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Slot and phase of a running group number, advanced without dividing.
struct Cursor {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step(int n) {
        if (++slot == n) { slot = 0; phase ^= 1u; }
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
        c.step(r.n);
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
    uint32_t code[4];      // offsets of the lane's four words of row g inside a window's pair `pair`, step by step
    uint32_t scale;        // offset of row g's two scale bytes
    uint32_t sel;          // prmt selector: (scale of steps 0 and 1, of steps 2 and 3)
    uint32_t x;            // offset inside a window's columns of a token row
    int unit;              // the lane's unit of a window
    bool first;            // lane 0
    __device__ __forceinline__ explicit Lane(int pair) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int row = (warp & 7) * 16 + g;
        unit = 2 * pair + (t >> 1);
        first = lane == 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            code[i] = (uint32_t)(unit * kTileCodeBytes + (t & 1) * (kTileCodeBytes / 2) + row * 16 + (i ^ t) * 4);
        scale = (uint32_t)(kScaleAt + unit * kTileScaleBytes + row * 4 + (t & 1) * 2);
        sel = (t >> 1) ? 0x1032u : 0x3210u;                  // steps 0 and 1 are in 16-column block t / 2
        x = (uint32_t)pair * 256u + (uint32_t)t * 16u;
        // kept in registers, not worked out anew in every window
        asm volatile("" : "+r"(code[0]), "+r"(code[1]), "+r"(code[2]), "+r"(code[3]), "+r"(scale), "+r"(sel), "+r"(x));
    }
};

// The consumers' two groups of 8 warps share the windows in one of two ways, which the two classes below are. A
// warp always holds the codes of its next pair of units: each word is replaced by the next pair's as soon as it
// is converted, across windows and pieces, and a slot is handed back when the last of it is read.
//
// WindowConsumer: a group takes both pairs of every second window: one wait, one hand-back and one set of
// counters for two pairs (0.42 us per window and SM against 0.48 with one token row, on weights that L2 holds; HBM's
// pace is 0.42). The ring has an
// even number of slots, so that a group's windows are all the phases of every second slot, in order: a
// group that saw only some phases of a slot could take an older phase's parity for the one it waits for.
template <int NT>
struct WindowConsumer {
    static constexpr int kArrivals = kConsumers / 2;     // that free a slot
    const Ring &r;
    Lane ln;
    uint32_t slot, bar, phase;         // the slot to read next, its full barrier, its phase
    uint32_t slot0, end;               // the group's first slot, one past the last full barrier
    uint32_t w0[4], w1[4], s0, s1;     // codes of rows g and g + 8, their scales
    bool mine;                         // the next window to come is this group's
    __device__ __forceinline__ explicit WindowConsumer(const Ring &ring)
        : r(ring), ln(0), phase(0), end(ring.full + 8u * ring.n) {
        const uint32_t group = (uint32_t)uniform((int)(threadIdx.x >> 8));
        slot = slot0 = ring.slots + group * kSlotBytes;
        bar = ring.full + 8u * group;
        mine = group == 0;
    }
    template <int P>
    __device__ __forceinline__ void load(int i) {
        constexpr uint32_t at = (uint32_t)P * 2u * kTileCodeBytes;
        w0[i] = lds32(slot + ln.code[i] + at);
        w1[i] = lds32(slot + ln.code[i] + (at + 128u));
    }
    template <int P>
    __device__ __forceinline__ void load_scales() {
        constexpr uint32_t at = (uint32_t)P * 2u * kTileScaleBytes;
        s0 = lds16(slot + ln.scale + at);
        s1 = lds16(slot + ln.scale + (at + 32u));
    }
    __device__ __forceinline__ void release() {
        __syncwarp();
        if (ln.first) mbar_arrive_at(bar + 8u * kMaxSlots);
        slot += 2u * kSlotBytes;
        bar += 16u;
        if (bar >= end) {
            slot = slot0;
            bar -= 8u * r.n;
            phase ^= 1u;
        }
    }
    // A run of `windows` windows begins: the group's first pair of it.
    __device__ __forceinline__ void fetch(int windows) {
        if (windows <= (mine ? 0 : 1)) return;
        wait_warp(r, bar, phase);
#pragma unroll
        for (int i = 0; i < 4; ++i) load<0>(i);
        load_scales<0>();
    }
    // Pair P of the group's units of the window in hand, with scales sa and sb, against the first N of NT tiles
    // of tokens; x + at: the lane's operands (token 8 n + g; any valid row where there is no such token) at the
    // pair's columns. Fetches the next pair: the window's second, or with `next` the first one of
    // the group's next window. Products E2M1 * E4M3 are exact in f16 (at most 6 significant bits, 2^-10 to 2688).
    template <int N, int P>
    __device__ __forceinline__ void multiply(const uint32_t (&x)[NT], uint32_t at, uint32_t sa, uint32_t sb, bool next, Acc<NT> &acc) {
        const uint32_t h0 = __byte_perm(e4m3x2_to_f16x2(sa), 0, ln.sel), h1 = __byte_perm(e4m3x2_to_f16x2(sb), 0, ln.sel);
        const __half2 v0 = *reinterpret_cast<const __half2 *>(&h0), v1 = *reinterpret_cast<const __half2 *>(&h1);
        // (without a next window the loads read the slot all the same, and nobody uses them)
        if (P == 1 && next) wait_warp(r, bar, phase);
        load_scales<1 - P>();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t a[4], b[4];
            e2m1x8_to_f16x2x4(w0[i], a);
            e2m1x8_to_f16x2x4(w1[i], b);
            load<1 - P>(i);
            const __half2 ma = i < 2 ? __low2half2(v0) : __high2half2(v0), mb = i < 2 ? __low2half2(v1) : __high2half2(v1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[j] = mul_f16x2(a[j], ma);
                b[j] = mul_f16x2(b[j], mb);
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint4 xv = lds128(x[n] + at + 64u * i);
                mma_f16(acc.c[0][n], a[0], b[0], a[1], b[1], xv.x, xv.y);
                mma_f16(acc.c[1][n], a[2], b[2], a[3], b[3], xv.z, xv.w);
            }
        }
        if (P == 0) release();
    }
    // One piece, the column tiles [ka, kb) of a row tile; the first pair of the group's next window is held
    // where it has one. rest: windows of the run behind the piece, as far as 2. xa: the lane's token rows; `two`:
    // the second tile of tokens has some.
    __device__ __forceinline__ void piece(int ka, int kb, int rest, const uint32_t (&xa)[NT], bool two, Acc<NT> &acc) {
        const int w0th = ka & ~(kWindow - 1), all = (kb - w0th + kWindow - 1) / kWindow;
        int i = mine ? 0 : 1;
        mine = mine != ((all & 1) != 0);
        uint32_t x[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) x[n] = xa[n] + ln.x + (uint32_t)(w0th + i * kWindow) * 128u;
#pragma unroll 1
        for (; i < all; i += 2) {
            const int w = w0th + i * kWindow;
            const bool next = i + 2 < all + rest;
            if (w >= ka && w + kWindow <= kb) {
                if (NT == 1 || two) {
                    multiply<NT, 0>(x, 0u, s0, s1, next, acc);
                    multiply<NT, 1>(x, 256u, s0, s1, next, acc);
                } else {
                    multiply<1, 0>(x, 0u, s0, s1, next, acc);
                    multiply<1, 1>(x, 256u, s0, s1, next, acc);
                }
            } else {
                // a window of which the piece has only some units: a lane without a unit multiplies zeros by zero scales
                // (zero times what an earlier window or an infinite activation left there could be a NaN)
                auto part = [&](auto pair) {
                    constexpr int P = decltype(pair)::value;
                    const int u = w + 2 * P + ln.unit;
                    const bool live = u >= ka && u < kb;
                    uint32_t xl[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) xl[n] = live ? x[n] + 256u * P : r.zeros;
                    multiply<NT, P>(xl, 0u, live ? s0 : 0u, live ? s1 : 0u, next, acc);
                };
                part(std::integral_constant<int, 0>());
                part(std::integral_constant<int, 1>());
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) x[n] += 2 * kWindow * 128u;
        }
    }
};

// PairConsumer: a group takes one pair of every window, and a slot is free as soon as both groups hold its codes.
// For rings of few slots and experts of few tokens: the wide layer at 14 tokens (4 slots) takes 176 us with it and
// 187 with the other, the matrix product 16 x 4096 x 32001 (4 slots, every column used) 30.8 and 29.4.
template <int NT>
struct PairConsumer {
    static constexpr int kArrivals = kConsumers;
    const Ring &r;
    Lane ln;
    uint32_t slot, bar, phase;         // the slot to read next, its full barrier, its phase
    uint32_t end;                      // one past the last full barrier
    uint32_t w0[4], w1[4], s0, s1;     // codes of rows g and g + 8, their scales
    __device__ __forceinline__ explicit PairConsumer(const Ring &ring)
        : r(ring), ln((int)(threadIdx.x >> 8)), slot(ring.slots), bar(ring.full), phase(0), end(ring.full + 8u * ring.n) {}

    __device__ __forceinline__ void release() {
        __syncwarp();
        if (ln.first) mbar_arrive_at(bar + 8u * kMaxSlots);
        slot += kSlotBytes;
        bar += 8u;
        if (bar == end) {
            slot = r.slots;
            bar = r.full;
            phase ^= 1u;
        }
    }
    // A run of `windows` windows begins, at least one.
    __device__ __forceinline__ void fetch(int) {
        wait_warp(r, bar, phase);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w0[i] = lds32(slot + ln.code[i]);
            w1[i] = lds32(slot + ln.code[i] + 128u);
        }
        s0 = lds16(slot + ln.scale);
        s1 = lds16(slot + ln.scale + 32u);
        release();
    }
    // One pair of units, with scales sa and sb, against the first N of NT tiles of tokens; x: the lane's
    // operands (token 8 n + g; any valid row where there is no such token) at the pair's columns. `next`:
    // fetch the next window's. Products E2M1 * E4M3 are exact in f16 (at most 6 significant bits,
    // 2^-10 to 2688).
    template <int N>
    __device__ __forceinline__ void multiply(const uint32_t (&x)[NT], uint32_t sa, uint32_t sb, bool next, Acc<NT> &acc) {
        const uint32_t h0 = __byte_perm(e4m3x2_to_f16x2(sa), 0, ln.sel), h1 = __byte_perm(e4m3x2_to_f16x2(sb), 0, ln.sel);
        const __half2 v0 = *reinterpret_cast<const __half2 *>(&h0), v1 = *reinterpret_cast<const __half2 *>(&h1);
        if (next) wait_warp(r, bar, phase);
        // (without a next window the loads read the slot all the same, and nobody uses them)
        s0 = lds16(slot + ln.scale);
        s1 = lds16(slot + ln.scale + 32u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t a[4], b[4];
            e2m1x8_to_f16x2x4(w0[i], a);
            e2m1x8_to_f16x2x4(w1[i], b);
            w0[i] = lds32(slot + ln.code[i]);
            w1[i] = lds32(slot + ln.code[i] + 128u);
            const __half2 ma = i < 2 ? __low2half2(v0) : __high2half2(v0), mb = i < 2 ? __low2half2(v1) : __high2half2(v1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[j] = mul_f16x2(a[j], ma);
                b[j] = mul_f16x2(b[j], mb);
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const uint4 xv = lds128(x[n] + 64u * i);
                mma_f16(acc.c[0][n], a[0], b[0], a[1], b[1], xv.x, xv.y);
                mma_f16(acc.c[1][n], a[2], b[2], a[3], b[3], xv.z, xv.w);
            }
        }
        if (next) release();
    }
    // One piece, the column tiles [ka, kb) of a row tile, whose first window is held; with `rest` > 0 another
    // piece follows, whose first window is held afterwards. xa: the lane's token rows; `two`: the
    // second tile of tokens has some.
    __device__ __forceinline__ void piece(int ka, int kb, int rest, const uint32_t (&xa)[NT], bool two, Acc<NT> &acc) {
        const bool more = rest > 0;
        uint32_t x[NT];
        int w = ka & ~(kWindow - 1);
#pragma unroll
        for (int n = 0; n < NT; ++n) x[n] = xa[n] + ln.x + (uint32_t)w * 128u;
        auto step = [&]() {
            w += kWindow;
#pragma unroll
            for (int n = 0; n < NT; ++n) x[n] += kWindow * 128u;
        };
        // a window of which the piece has only some units: a lane without a unit multiplies zeros by zero scales
        // (zero times what an earlier window or an infinite activation left there could be a NaN)
        auto part = [&]() {
            const bool live = w + ln.unit >= ka && w + ln.unit < kb;
            uint32_t xl[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) xl[n] = live ? x[n] : r.zeros;
            multiply<NT>(xl, live ? s0 : 0u, live ? s1 : 0u, more || w + kWindow < kb, acc);
            step();
        };
        if (w < ka) part();
        const int whole = (kb - w) / kWindow;
        const bool after = more || w + whole * kWindow < kb;
#pragma unroll 1
        for (int i = whole; i > 0; --i) {
            if (NT == 1 || two) multiply<NT>(x, s0, s1, i > 1 || after, acc);
            else multiply<1>(x, s0, s1, i > 1 || after, acc);
#pragma unroll
            for (int n = 0; n < NT; ++n) x[n] += kWindow * 128u;
        }
        w += whole * kWindow;
        if (w < kb) part();
    }
};

// The pieces of a run [u, end) of units, row tile after row tile: ka..kb of row tile rt (of RT) of expert
// ei. Stepping takes no division.
struct Pieces {
    uint32_t u, end;
    int RT, KT, ei, rt, ka, kb;
    __device__ __forceinline__ Pieces(uint32_t first, uint32_t last, int row_tiles, int col_tiles)
        : u(first), end(last), RT(row_tiles), KT(col_tiles) {
        const uint32_t q = u / (uint32_t)KT;
        ei = (int)(q / (uint32_t)RT);
        rt = (int)(q - (uint32_t)ei * RT);
        ka = (int)(u - q * KT);
        kb = (int)min((uint32_t)KT, ka + (end - u));
    }
    __device__ __forceinline__ bool valid() const { return u < end; }
    // Windows of the piece; windows of the run behind it, as far as 2.
    __device__ __forceinline__ int windows() const { return (kb - (ka & ~(kWindow - 1)) + kWindow - 1) / kWindow; }
    __device__ __forceinline__ int rest() const {
        const int left = (int)(end - u) - (kb - ka);
        return left == 0 ? 0 : left > min(KT, kWindow) ? 2 : 1;
    }
    __device__ __forceinline__ void next() {
        u += kb - ka;
        if (++rt == RT) { rt = 0; ++ei; }
        ka = 0;
        kb = (int)min((uint32_t)KT, end - u);
    }
};

// Barrier among the consumer warps.
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumerThreads) : "memory"); }

// The sums of a finished piece: warps 8 to 15 hand theirs to warps 0 to 7 through `buf` ([column][128
// rows], kSumStride floats a column), and those call f(n, j, sum) for their values, every lane of a warp
// in each call: column 8 n + 2 t + (j & 1) of m (beyond m where only other lanes have one), row
// 16 warp + g + 8 (j >> 1). The two warps of a row group meet at a barrier of
// their own; two buffers in turn make it one meeting per piece.
constexpr int kSumStride = 132;
template <int NT, class F>
__device__ __forceinline__ void join_pairs(const Acc<NT> &acc, float *buf, int m, F f) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float *mine = buf + 2 * t * kSumStride + (warp & 7) * 16 + g;
    if (warp >= 8) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (8 * n + 2 * t + (j & 1) < m) mine[(8 * n + (j & 1)) * kSumStride + 8 * (j >> 1)] = acc.sum(n, j);
    }
    asm volatile("bar.sync %0, 64;" ::"r"(2 + (warp & 7)) : "memory");
    if (warp < 8) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (8 * n + (j & 1) >= m) continue;          // no lane has a column below m
                const int col = 8 * n + 2 * t + (j & 1);
                const float other = col < m ? mine[(8 * n + (j & 1)) * kSumStride + 8 * (j >> 1)] : 0.f;
                f(n, j, acc.sum(n, j) + other);
            }
    }
}

// Eight bf16 values (as loaded) times `up`, rounded to f16; in the order 0 2 4 6 1 3 5 7 when the weights'
// words are kept so (the matrix product's).
template <bool EvenFirst>
__device__ __forceinline__ uint4 bf16x8_to_f16(const uint4 &v, float up) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    float lo[4], hi[4];
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        lo[j] = bf16_bits_to_float(u[j] & 0xFFFFu) * up;
        hi[j] = bf16_bits_to_float(u[j] >> 16) * up;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 h = !EvenFirst ? __floats2half2_rn(lo[j], hi[j])
                          : j < 2    ? __floats2half2_rn(lo[2 * j], lo[2 * j + 1])
                                     : __floats2half2_rn(hi[2 * j - 4], hi[2 * j - 3]);
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
// Smallest magnitude bits less one of eight bf16 values, zeros left out (they become 0xFFFF), in both halves of a word.
__device__ __forceinline__ uint32_t min_bits(const uint4 &v, uint32_t m) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t less;
        asm("add.u16x2 %0, %1, %2;" : "=r"(less) : "r"(u[j] & 0x7FFF7FFFu), "r"(0xFFFFFFFFu));
        asm("min.u16x2 %0, %0, %1;" : "+r"(m) : "r"(less));
    }
    return m;
}
// Whether a row has elements that its f16 operand cannot hold: the last bit of an element, 2^(field - 134), has to be
// at least f16's last one, 2^-24, times the row's power of two, so the fields may be 31 apart. low: min_bits of the row. A row with
// an infinity or a NaN is not one of these: its outputs are infinite or NaN whatever its other elements are.
__device__ __forceinline__ bool wide_row(uint32_t emax, uint32_t low) {
    return emax < 255u && (int)emax - max((int)((low + 1) >> 7), 1) > 31;
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
// memory (row_bytes(KT) apart), by all consumers: f16 times a power of two per row, columns from K
// on zero. Only the 128-column groups for which used(group) holds are read and written. emax[t] and low[t] (0
// and ~0 before) receive the rows' largest exponent fields and smallest magnitudes (low is free afterwards).
// Returns whether a row's elements lie too far apart for that (wide_row; an element then loses bits, and is 0 more
// than 2^39 below the largest); what needs those rows takes exact_dot instead. Ends with a consumer barrier. A thread
// keeps up to kHeld chunks in registers between finding the maximum and converting; what lies beyond
// is read again. requested: an
// mbarrier that every consumer warp arrives at once its first loads are on the way.
template <int kHeld, bool EvenFirst, class Used>
__device__ __forceinline__ bool convert_rows(const uint16_t *x, int64_t ld, uint8_t *rows, int T, int K, int KT,
                                             uint32_t *emax, uint32_t *low, Used used, uint32_t requested = 0) {
    const int chunks = ((KT + 1) / 2) * 16;
    int tpr = kConsumerThreads;                              // threads per row, at least a warp
    while (tpr * T > kConsumerThreads) tpr >>= 1;
    const int t = threadIdx.x / tpr, i0 = threadIdx.x % tpr;
    const uint4 *row = reinterpret_cast<const uint4 *>(x + (int64_t)t * ld);
    const int rounds = (chunks + tpr - 1) / tpr;
    uint4 v[kHeld];
    if (t < T) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            const int i = i0 + j * tpr;
            v[j] = make_uint4(0, 0, 0, 0);
            if (j < rounds && i * 8 < K && used(i >> 4)) v[j] = row[i];
        }
    }
    if (requested && (threadIdx.x & 31) == 0) mbar_arrive_at(requested);
    if (t < T) {
        uint32_t m = 0, n = 0xFFFFFFFFu;
#pragma unroll
        for (int j = 0; j < kHeld; ++j)
            if (j < rounds) {
                m = max_bits(v[j], m);
                n = min_bits(v[j], n);
            }
#pragma unroll 4
        for (int i = i0 + kHeld * tpr; i * 8 < K; i += tpr)
            if (used(i >> 4)) {
                const uint4 r = row[i];
                m = max_bits(r, m);
                n = min_bits(r, n);
            }
        const uint32_t e = __reduce_max_sync(0xffffffffu, max(m >> 23, (m >> 7) & 0xFFu));
        const uint32_t l = __reduce_min_sync(0xffffffffu, min(n >> 16, n & 0xFFFFu));
        if ((threadIdx.x & 31) == 0) {
            atomicMax(&emax[t], e);
            atomicMin(&low[t], l);
        }
    }
    consumer_sync();
    const int lane = threadIdx.x & 31;
    const bool wide = __any_sync(0xffffffffu, lane < T && wide_row(emax[lane < T ? lane : 0], low[lane < T ? lane : 0]));
    if (t < T) {
        const float up = up_of(emax[t]);
        uint8_t *dst = rows + t * row_bytes(KT);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            const int i = i0 + j * tpr;
            if (j >= rounds) break;
            if (i < chunks && used(i >> 4)) *reinterpret_cast<uint4 *>(dst + chunk_offset(i * 8)) = bf16x8_to_f16<EvenFirst>(v[j], up);
        }
#pragma unroll 4
        for (int i = i0 + kHeld * tpr; i < chunks; i += tpr)
            if (used(i >> 4))
                *reinterpret_cast<uint4 *>(dst + chunk_offset(i * 8)) =
                    i * 8 < K ? bf16x8_to_f16<EvenFirst>(row[i], up) : make_uint4(0, 0, 0, 0);
    }
    consumer_sync();
    return wide;
}

// The sum of x w over the column tiles [ka, kb) of one row (of 128) of a row tile, from global memory in fp32 FMAs
// (the products are exact): what takes the place of a piece's product where convert_rows finds rows too wide for f16.
// Rarely needed (activations 2^31 and more apart in one row) and slow: 8 x 4096 x 32001 takes 304 us with it and 22
// without, the decode layer of 8 tokens 282 and 44, the product of one token 1 x 2048 x 4096 16 and 8.
template <bool EvenFirst>
__device__ __forceinline__ float exact_dot(const uint8_t *codes, const uint8_t *scales, int ka, int kb, int row, const uint16_t *x, int K) {
    float s = 0.f;
#pragma unroll 1
    for (int k = ka; k < kb; ++k) {
        const uint8_t *ct = codes + (size_t)k * kTileCodeBytes + row * 16;
        const uint32_t sc = *reinterpret_cast<const uint32_t *>(scales + (size_t)k * kTileScaleBytes + row * 4);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            const uint4 c4 = *reinterpret_cast<const uint4 *>(ct + h * (kTileCodeBytes / 2));
            const uint32_t words[4] = {c4.x, c4.y, c4.z, c4.w}, two = e4m3x2_to_f16x2(sc >> (16 * h) & 0xFFFFu);
            const __half2 m = *reinterpret_cast<const __half2 *>(&two);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int col = k * kTileK + h * 32 + w * 8;
                if (col >= K) break;                     // K is a multiple of 16: a chunk is inside or not
                const uint4 xv = *reinterpret_cast<const uint4 *>(x + col);
                const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
                uint32_t f[4];
                e2m1x8_to_f16x2x4(words[w], f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 wv = f16x2_to_float2(mul_f16x2(f[j], w < 2 ? __low2half2(m) : __high2half2(m)));
                    // the pair's columns: 2j and 2j + 1, or with the even columns first 0 2, 4 6, 1 3, 5 7
                    const uint32_t lo = EvenFirst ? xw[2 * (j & 1)] : xw[j], hi = EvenFirst ? xw[2 * (j & 1) + 1] : xw[j];
                    const bool odd = EvenFirst && j >= 2;
                    s = fmaf(bf16_bits_to_float(odd ? lo >> 16 : lo & 0xFFFFu), wv.x, s);
                    s = fmaf(bf16_bits_to_float(odd || !EvenFirst ? hi >> 16 : hi & 0xFFFFu), wv.y, s);
                }
            }
        }
    }
    return s;
}

}  // namespace stream
}  // namespace tfmoe
