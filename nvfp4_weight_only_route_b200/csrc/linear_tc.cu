// linear_tc.cu -- the tensor-core regime of the NVFP4 matrix product: more tokens than the streaming
// regime takes, bound by the bf16 tensor pipe (large T) or by latency (short prompts).
//
// A tile is 128 weight rows (MMA M) x N <= 192 tokens (MMA N), the reduction in stages of 64. The weights are
// decoded to bf16 in registers and stored into tensor memory as the A operand; the bf16 token rows
// come by TMA (128-byte swizzle) into shared memory as the B operand: no rounding of either. Per CTA
// (one per SM, 24 warps):
//   warp 0       token tiles (TMA) into a ring that the MMA commits free
//   warp 2       codes and scales of four stages at a time (two bulk copies) into a ring that the decoders free
//   warp 1       owns tensor memory, issues four MMAs of K = 16 per stage
//   warps 4-15   three decode warpgroups taking every third stage, a thread per weight row
//   warps 16-23  epilogue, two warpgroups taking alternate 16-token steps of the accumulator
// Tensor memory: two accumulators of 192 columns, so that a tile's epilogue runs under the next tile's
// products, and four decoded stages of 32 columns: all 512.
//
// What bounds the main loop is the issue: four MMAs, a commit and a barrier wait keep the issuing warp
// about 380 clocks, as long as a stage's MMAs take at N = 192 (two waits and two commits: 680). So a
// stage's decoders wait for its token tile too, one barrier tells the issuer of both operands, one commit
// frees both (the A slot of stage g, a quarter of a shorter ring, was stage g - 4's), and the next
// stage's barrier is asked while the current MMAs are issued. (One accumulator of 224 columns that the
// epilogue takes into 112 registers a thread at once was as fast at 7234 tokens, but its 50 KB of
// straight-line code came from memory in every launch: 28 us against 16 at 601 tokens.)
//
// Measured: 7234 x 4096 x 2 x 2688 with SwiGLU 221 us from rest (1.44 PFLOP/s, 0.87 of the measured bf16 burst),
// 229 to 235 us in a row, where the power limit holds the clock (1.37, 0.98 of the measured sustained rate).
// 601 x 2688 x 1001 13.4 us, 100 x 1536 x 4096 9.7, 16 x 4096 x 2 x 2688 10.9. Copying codes and scales stage by
// stage kept the copying thread busier than the MMAs (250 us). Two CTAs per tile (cta_group::2, half the token
// bytes for each) gave 213 us from rest and 221 in a row and nothing at fewer tokens: not worth a second set
// of kernels.
//
// The decode: a stage must be decoded in the time of its MMAs (2 N clocks, 384 at N = 192). A conversion
// to f16 and on to bf16 would take about 410 clocks per stage of an SM's conversion rate (36 lanes per clock
// for E2M1, 63 for f16 -> f32). So the code's bits are placed instead: sign at bit 15 and the three
// magnitude bits at 8..6 of a bf16 are that E2M1 value times 2^-126, its subnormal included; one
// bf16x2 multiplication by the block scale times 2^112 gives value * scale * 2^-14 exactly (at most 6
// significant bits, 2^-24 to 0.17), and 2^14 joins the multiplier in the epilogue. The tiled layout
// keeps the eight codes of a word in the order 0 2 4 6 1 3 5 7, so that a shift brings the codes of
// columns 2j and 2j + 1 to the same place of both halves; a product by 2^6 + 2^12 puts magnitude and sign
// where they belong in one instruction, which the integer multiplier does beside the logic unit.
//
// Few tiles leave SMs idle, so their reductions are split: CTA (tile, split) leaves its sums in global memory,
// and the CTA that arrives last at the tile's counter adds them in split order and finishes the tile, with
// the decode warps' help (601 tokens: 16.3 us by the epilogue warps alone).
// No CTA waits for another; equal calls give equal bits.
#include <cuda.h>

#include <algorithm>

#include "linear.h"

namespace tfmoe {
namespace {

constexpr int kM = 128;
constexpr int kMaxN = 192;
constexpr int kStages = 6, kAStages = 4, kDBufs = 2;
constexpr int kWindow = 4, kWindows = 4;     // stages per window of codes and scales, windows in the ring
constexpr int kDqGroups = 3, kEpiGroups = 2;
constexpr int kDqWarp0 = 4, kEpiWarp0 = kDqWarp0 + 4 * kDqGroups;
constexpr int kThreads = 32 * (kEpiWarp0 + 4 * kEpiGroups);
constexpr int kJoinGroups = kDqGroups + kEpiGroups, kJoinThreads = 128 * kJoinGroups;
constexpr uint32_t kACol = kDBufs * kMaxN, kTmemCols = 512;
static_assert(kACol + kAStages * 32 <= kTmemCols, "tensor memory");
static_assert(kAStages < kStages, "an A slot's last use is told by the barrier of its stage");
constexpr int kBBytes = kMaxN * 128;
constexpr int kMaxSplits = 8;

struct TcSmem {
    uint8_t b[kStages][kBBytes];             // 1024-byte aligned
    uint8_t codes[kWindows][kWindow * kTileCodeBytes];
    uint8_t scales[kWindows][kWindow * kTileScaleBytes];
    uint64_t bfull[kStages], ready[kStages], done[kStages];   // token tile landed; both operands there; MMAs complete
    uint64_t cfull[kWindows], cempty[kWindows];
    uint64_t dfull[kDBufs], dempty[kDBufs];
    uint64_t mma_done;
    uint32_t tmem_base;
    int32_t abort_flag;
    int32_t is_last;
};

struct TcArgs {
    const uint8_t *codes, *scales;
    int T, RT, KT, N, splits, items;         // items: tiles * splits
    float *partial;                          // [items][N][128]
    int32_t *tickets;                        // [tiles], left at 0
    int32_t *err_word;
    uint32_t test_wait_ns;                   // > 0: CTA 0's token copies wait that long for nothing and time out
    LinearEpilogue ep;
};

// Bounded wait. The kernel may have started before the one ahead of it has ended, whose time does not count: when the
// limit passes, that one is waited for and the clock set back, once. (A function of its own: inlined in the
// dozen places that wait, its code costs the product of 100 tokens 0.2 us.)
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int32_t *abort_flag, int32_t *err) {
    for (int again = 1;; --again) {
        const uint64_t t0 = global_timer_ns();
        do {
            for (int i = 0; i < 4; ++i)
                if (mbar_try_wait_sleep_at(bar, parity)) return true;
            if (*abort_flag) return false;
        } while (global_timer_ns() - t0 <= kWaitLimitNs);
        if (!again) break;
        grid_dep_wait();
    }
    atomicOr(err, DEV_ERR_WAIT_TIMEOUT);
    *abort_flag = 1;
    return false;
}
__device__ __forceinline__ bool wait_or_abort(TcSmem &sm, uint64_t *bar, uint32_t parity, int32_t *err) {
    return mbar_try_wait(bar, parity) || wait_long(smem_u32(bar), parity, &sm.abort_flag, err);
}
__device__ __forceinline__ bool wait_warp(TcSmem &sm, uint64_t *bar, uint32_t parity, int32_t *err) {
    return __all_sync(0xffffffffu, wait_or_abort(sm, bar, parity, err));
}

// Whether a phase is complete, without waiting.
__device__ __forceinline__ bool test_now(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr) {
    // K-major, 128-byte swizzle, 1024 bytes between groups of 8 rows
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1u << 16) | ((uint64_t)(1024u >> 4) << 32) |
           ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}
// kind::f16, A and B bf16 K-major, D fp32, M = 128.
__device__ __forceinline__ uint32_t instr_desc(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kM >> 4) << 24);
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %5, %5, %5}, p;\n\t}"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(0u));
}
__device__ __forceinline__ bool elect_one() {
    uint32_t pred = 0;
    asm volatile("{\n\t.reg .b32 rx;\n\t.reg .pred px;\n\telect.sync rx|px, %1;\n\t@px mov.s32 %0, 1;\n\t}"
                 : "+r"(pred) : "r"(0xffffffffu));
    return pred != 0;
}
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void join_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kJoinThreads) : "memory"); }

// The block scales of two E4M3 bytes times 2^112, each in both halves of a bf16x2.
__device__ __forceinline__ void scale_pairs(uint32_t two, uint32_t &lo, uint32_t &hi) {
    const float2 f = f16x2_to_float2(e4m3x2_to_f16x2(two));
    const uint32_t a = __float_as_uint(f.x * 0x1p112f), b = __float_as_uint(f.y * 0x1p112f);
    lo = __byte_perm(a, 0, 0x3232);              // an E4M3 value fills 4 significant bits: its fp32 is a bf16
    hi = __byte_perm(b, 0, 0x3232);
}
// Eight codes (order 0 2 4 6 1 3 5 7) times the scale pair -> four bf16x2, columns in order.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t scale, uint32_t *o) {
    constexpr uint32_t kKeep = 0x81C081C0u;
    const uint32_t w8 = w >> 8;
    // a code times 2^6 + 2^12: its magnitude at bits 8..6, its sign at bit 15, and copies that the mask drops
    const uint32_t v[4] = {(w & 0x000F000Fu) * 4160u & kKeep, (w & 0x00F000F0u) * 260u & kKeep,
                           (w8 & 0x000F000Fu) * 4160u & kKeep, (w8 & 0x00F000F0u) * 260u & kKeep};
#pragma unroll
    for (int j = 0; j < 4; ++j) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o[j]) : "r"(v[j]), "r"(scale));
}

struct Item {
    int tile, split, rt, t0, k0, k1;
    __device__ __forceinline__ Item(const TcArgs &a, int i) {
        tile = i / a.splits;
        split = i - tile * a.splits;
        const int tt = tile / a.RT;              // row tiles first: concurrent tiles share token rows
        rt = tile - tt * a.RT;
        t0 = tt * a.N;
        k0 = split * a.KT / a.splits;
        k1 = (split + 1) * a.KT / a.splits;
    }
};

// The activation for outputs that are rounded to bf16: exponential and reciprocal one instruction each
// (relative errors of a few units of fp32). fp32 outputs take CUDA's own functions (linear.h).
__device__ __forceinline__ float activate_fast(float y, int act) {
    switch (act) {
    case TFMOE_ACT_SILU: return silu_f32(y);
    case TFMOE_ACT_GELU: return gelu<true>(y);
    case TFMOE_ACT_GELU_TANH: {
        const float z = 1.5957691216057308f * (y + 0.044715f * y * y * y);
        return y * rcp_approx(1.0f + __expf(-z));
    }
    default: return activate(y, act);
    }
}

// One epilogue thread's place: its output column and where its next step's tokens lie.
template <int Act, bool Fast, int Groups>
struct Finisher {
    static constexpr bool kGated = Act == TFMOE_ACT_SWIGLU;
    static constexpr int kTok = kGated ? 8 : 16;   // tokens of a step that this lane finishes
    const LinearEpilogue &ep;
    int T, t;                                      // the call's tokens; the step's first one of this lane
    bool odd, in;
    float g0, g1, b0, b1;
    const uint16_t *res;
    char *out;

    // gated: an even lane has gate row j of a step's 16 tokens, the odd lane after it up row j; the even lane
    // finishes tokens 0..7, the odd one 8..15
    __device__ __forceinline__ Finisher(const LinearEpilogue &e, int tokens, int rt, int q, int first, float m0, float m1)
        : ep(e), T(tokens), odd(kGated && (q & 1)), g0(m0), g1(m1) {
        const int n = kGated ? (rt * kM + q) >> 1 : rt * kM + q;
        in = n < ep.N;
        b0 = ep.bias && in ? __ldg(ep.bias + n) : 0.f;
        b1 = kGated && ep.bias && in ? __ldg(ep.bias + ep.N + n) : 0.f;
        t = first + (odd ? 8 : 0);
        res = ep.residual ? ep.residual + (int64_t)t * ep.ldr + n : nullptr;
        out = static_cast<char *>(ep.out) + ((int64_t)t * ep.ldo + n) * (Fast ? 2 : 4);
    }
    // A step's 16 sums of this lane's weight row; the next step is 16 Groups tokens on. The residual is
    // loaded for eight tokens before any of them is stored: out may be the residual, so the compiler moves no
    // load ahead of a store, and one load at a time would cost its latency per token.
    __device__ __forceinline__ void step(const uint32_t (&s)[16]) {
        const int64_t ob = ep.ldo * (Fast ? 2 : 4);
#pragma unroll
        for (int h = 0; h < kTok; h += 8) {
            uint32_t rv[8];
            if (res) {
                const uint16_t *p = res;
#pragma unroll
                for (int i = 0; i < 8; ++i, p += ep.ldr) rv[i] = in && t + i < T ? *p : 0u;
            }
            char *p = out;
#pragma unroll
            for (int i = 0; i < 8; ++i, p += ob) {
                float v;
                if (kGated) {
                    const float lo = __uint_as_float(s[i]), hi = __uint_as_float(s[i + 8]);
                    const float keep = odd ? hi : lo, got = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
                    const float gate = fmaf(odd ? got : keep, g0, b0), up = fmaf(odd ? keep : got, g1, b1);
                    v = (Fast ? silu_f32(gate) : activate(gate, TFMOE_ACT_SILU)) * up;
                } else {
                    const float y = fmaf(__uint_as_float(s[h + i]), g0, b0);
                    v = Fast ? activate_fast(y, Act) : activate(y, Act);
                }
                if (res) v += bf16_bits_to_float(rv[i]);
                if (in && t + i < T) {
                    if (Fast) *reinterpret_cast<uint16_t *>(p) = float_to_bf16_bits_rn(v);
                    else *reinterpret_cast<float *>(p) = v;
                }
            }
            const int ahead = h + 8 < kTok ? 8 : 16 * Groups + 8 - kTok;
            if (res) res += ahead * ep.ldr;
            out += ahead * ob;
            t += ahead;
        }
    }
};

template <int Act, bool Fast>
__global__ void __launch_bounds__(kThreads, 1) linear_tc_kernel(const __grid_constant__ CUtensorMap xmap, const TcArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    TcSmem &sm = *reinterpret_cast<TcSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) { mbar_init(&sm.bfull[s], 1); mbar_init(&sm.ready[s], 4); mbar_init(&sm.done[s], 1); }
        for (int s = 0; s < kWindows; ++s) { mbar_init(&sm.cfull[s], 1); mbar_init(&sm.cempty[s], 4 * kDqGroups); }
        for (int s = 0; s < kDBufs; ++s) { mbar_init(&sm.dfull[s], 1); mbar_init(&sm.dempty[s], 4 * kEpiGroups); }
        mbar_init(&sm.mma_done, 1);
        sm.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&sm.tmem_base)), "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_before();
    __syncthreads();
    tc_after();
    grid_dep_launch_dependents();
    const uint32_t tmem = sm.tmem_base;
    int32_t *err = a.err_word;

    if (warp == 0 || warp == 2) {
        if (lane == 0) {
            const bool tokens = warp == 0;
            const int nst = tokens ? kStages : kWindows, step = tokens ? 1 : kWindow;
            uint64_t *full = tokens ? sm.bfull : sm.cfull, *empty = tokens ? sm.done : sm.cempty;
            if (tokens) grid_dep_wait();         // the weights are nobody's output; the tokens may be
            uint32_t issued = 0, ph = 0;
            int s = 0;
            bool ok = true;
            if (a.test_wait_ns && tokens && blockIdx.x == 0) {       // nobody else fills the first stage
                const uint64_t t0 = global_timer_ns();
                while (ok && !mbar_try_wait_sleep(&full[0], 0)) ok = global_timer_ns() - t0 <= a.test_wait_ns;
                atomicOr(err, DEV_ERR_WAIT_TIMEOUT);
                *reinterpret_cast<volatile int32_t *>(&sm.abort_flag) = 1;
            }
            for (int i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
                const Item it(a, i);
                for (int kt = it.k0; kt < it.k1; kt += step) {
                    ok = wait_or_abort(sm, &empty[s], ph ^ 1u, err);
                    if (!ok) break;
                    if (tokens) {
                        mbar_arrive_expect_tx(&full[s], (uint32_t)a.N * 128u);
                        tma_load_2d(sm.b[s], &xmap, kt * kTileK, it.t0, &full[s]);
                    } else {
                        // a row tile's stages follow one another in both arrays
                        const size_t tile = (size_t)it.rt * a.KT + kt;
                        const uint32_t n = (uint32_t)min(kWindow, it.k1 - kt);
                        mbar_arrive_expect_tx(&full[s], n * (kTileCodeBytes + kTileScaleBytes));
                        bulk_g2s(sm.codes[s], a.codes + tile * kTileCodeBytes, n * kTileCodeBytes, &full[s]);
                        bulk_g2s(sm.scales[s], a.scales + tile * kTileScaleBytes, n * kTileScaleBytes, &full[s]);
                    }
                    ++issued;
                    if (++s == nst) { s = 0; ph ^= 1u; }
                }
            }
            if (*reinterpret_cast<volatile int32_t *>(&sm.abort_flag)) {
                // aborted: let the copies already issued land before the CTA exits (bounded)
                for (uint32_t j = issued > (uint32_t)nst ? issued - nst : 0; j < issued; ++j) {
                    const uint64_t t0 = global_timer_ns();
                    while (!mbar_try_wait_sleep(&full[j % nst], (j / nst) & 1u) && global_timer_ns() - t0 < kWaitLimitNs / 4) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        const uint64_t bdesc0 = smem_desc(smem_u32(sm.b[0]));
        int s = 0;
        uint32_t ph = 0, n_item = 0, g = 0;
        bool ok = true;
        for (int i = blockIdx.x; i < a.items && ok; i += gridDim.x, ++n_item) {
            const Item it(a, i);
            const uint32_t idesc = instr_desc(min(a.N, (a.T - it.t0 + 15) & ~15));
            const int buf = (int)(n_item % kDBufs);
            ok = wait_warp(sm, &sm.dempty[buf], ((n_item / kDBufs) & 1u) ^ 1u, err);
            if (!ok) break;
            const uint32_t d = tmem + (uint32_t)buf * kMaxN;
            bool here = test_now(&sm.ready[s], ph);
            for (int kt = it.k0; kt < it.k1; ++kt, ++g) {
                if (!__all_sync(0xffffffffu, here)) {
                    ok = wait_warp(sm, &sm.ready[s], ph, err);
                    if (!ok) break;
                }
                tc_after();
                // the next stage's barrier is asked while this one's MMAs are issued
                const int sn = s + 1 == kStages ? 0 : s + 1;
                const uint32_t pn = ph ^ (sn == 0 ? 1u : 0u);
                here = test_now(&sm.ready[sn], pn);
                if (elect_one()) {
                    const uint64_t bd = bdesc0 + (uint64_t)(s * (kBBytes >> 4));
                    const uint32_t ad = tmem + kACol + (g % kAStages) * 32u;
                    mma_ts(d, ad, bd, idesc, kt != it.k0);
                    mma_ts(d, ad + 8u, bd + 2u, idesc, 1u);
                    mma_ts(d, ad + 16u, bd + 4u, idesc, 1u);
                    mma_ts(d, ad + 24u, bd + 6u, idesc, 1u);
                    commit(&sm.done[s]);
                }
                __syncwarp();
                s = sn;
                ph = pn;
            }
            if (!ok) break;
            if (elect_one()) commit(&sm.dfull[buf]);
            __syncwarp();
        }
        // on every path: tensor memory and the stages stay in use until the MMAs issued are complete
        if (elect_one()) commit(&sm.mma_done);
        __syncwarp();
    } else if (warp >= kDqWarp0 && warp < kEpiWarp0) {
        const int gq = (warp - kDqWarp0) >> 2, q = (warp & 3) * 32 + lane;
        const uint32_t acol = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kACol;
        // this group's stages are the running numbers gq, gq + 3, ...; ring places are kept, not divided for
        // Every warp passes every window, those without a stage of its own too: a barrier's phase is then
        // never two ahead of a warp that waits for it.
        int s = gq, sa = gq, skip = gq;
        uint32_t ps = 0, seen = 0, base = 0;     // windows passed, windows before this item
        bool ok = true;
        for (int i = blockIdx.x; i < a.items && ok; i += gridDim.x) {
            const Item it(a, i);
            int kt = it.k0 + skip;
            for (; kt < it.k1; kt += kDqGroups) {
                const uint32_t j = (uint32_t)(kt - it.k0), win = base + j / kWindow, at = j % kWindow, w4 = win % kWindows;
                while (seen <= win) {
                    ok = wait_warp(sm, &sm.cfull[seen % kWindows], seen / kWindows & 1u, err);
                    if (!ok) break;
                    if (seen++ < win && lane == 0) mbar_arrive(&sm.cempty[(seen - 1) % kWindows]);
                }
                if (!ok) break;
                const uint8_t *codes = sm.codes[w4] + at * kTileCodeBytes + q * 16;
                const uint4 c0 = *reinterpret_cast<const uint4 *>(codes), c1 = *reinterpret_cast<const uint4 *>(codes + 2048);
                const uint32_t sc4 = *reinterpret_cast<const uint32_t *>(sm.scales[w4] + at * kTileScaleBytes + q * 4);
                __syncwarp();
                // the window's last stage of this group
                if (lane == 0 && (at + kDqGroups >= kWindow || kt + kDqGroups >= it.k1)) mbar_arrive(&sm.cempty[w4]);
                uint32_t sp[4], r[32];
                scale_pairs(sc4 & 0xFFFFu, sp[0], sp[1]);
                scale_pairs(sc4 >> 16, sp[2], sp[3]);
                const uint32_t words[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
                for (int w = 0; w < 8; ++w) decode8(words[w], sp[w >> 1], r + 4 * w);
                // the A slot was stage g - 4's, kStages - 4 places on in the ring: its MMAs are complete (the
                // barrier's next phase, stage g + 2's, cannot end before this stage is decoded; stages 0..3 find the
                // phase before the first complete)
                const int sd = s + kStages - kAStages < kStages ? s + kStages - kAStages : s - kAStages;
                ok = wait_warp(sm, &sm.done[sd], sd > s ? ps ^ 1u : ps, err);
                if (!ok) break;
                tc_after();
                const uint32_t col = acol + (uint32_t)sa * 32u;
                tmem_st16(col, r);
                tmem_st16(col + 16u, r + 16);
                ok = wait_warp(sm, &sm.bfull[s], ps, err);
                tc_wait_st();                    // after an abort too: tensor memory is freed at the end
                if (!ok) break;
                tc_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.ready[s]);
                if ((s += kDqGroups) >= kStages) { s -= kStages; ps ^= 1u; }
                if ((sa += kDqGroups) >= kAStages) sa -= kAStages;
            }
            skip = kt - it.k1;                   // of the next item's first stages
            base += (uint32_t)(it.k1 - it.k0 + kWindow - 1) / kWindow;
        }
    } else if (warp >= kEpiWarp0) {
        const int eg = (warp - kEpiWarp0) >> 2, q = (warp & 3) * 32 + lane;
        const uint32_t d = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float g0 = __ldg(a.ep.global0) * 0x1p14f, g1 = Act == TFMOE_ACT_SWIGLU ? __ldg(a.ep.global1) * 0x1p14f : 0.f;
        grid_dep_wait();
        uint32_t n_item = 0;
        for (int i = blockIdx.x; i < a.items; i += gridDim.x, ++n_item) {
            const Item it(a, i);
            const int steps = (min(a.N, a.T - it.t0) + 15) >> 4;
            const int buf = (int)(n_item % kDBufs);
            const bool ok = wait_warp(sm, &sm.dfull[buf], (n_item / kDBufs) & 1u, err);
            if (!ok) break;
            tc_after();
            const uint32_t dcol = d + (uint32_t)buf * kMaxN;
            auto load = [&](int st, uint32_t (&r)[16]) {
                tmem_ld16(dcol + (uint32_t)(16 * st), r);
                tc_wait_ld();
                if (st + kEpiGroups >= steps) {  // the warp's last read of the accumulator
                    tc_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.dempty[buf]);
                }
            };
            if (eg >= steps && lane == 0) mbar_arrive(&sm.dempty[buf]);
            if (a.splits > 1) {
                float *mine = a.partial + ((size_t)i * a.N + 16 * eg) * kM + q;
#pragma unroll 1
                for (int st = eg; st < steps; st += kEpiGroups) {
                    uint32_t r[16];
                    load(st, r);
#pragma unroll
                    for (int c = 0; c < 16; ++c) mine[c * kM] = __uint_as_float(r[c]);
                    mine += 16 * kEpiGroups * kM;
                }
                continue;
            }
            Finisher<Act, Fast, kEpiGroups> fin(a.ep, a.T, it.rt, q, it.t0 + 16 * eg, g0, g1);
#pragma unroll 1
            for (int st = eg; st < steps; st += kEpiGroups) {
                uint32_t r[16];
                load(st, r);
                fin.step(r);
            }
        }
    }
    // A split item is its CTA's only one (the grid is one wave): the decode and epilogue warps, all free by
    // now, join the tile in the CTA that arrives last. (After an abort they still meet here.)
    if (a.splits > 1 && warp >= kDqWarp0) {
        const Item it(a, (int)blockIdx.x);
        join_sync();
        if (threadIdx.x == kDqWarp0 * 32) {
            __threadfence();                     // the CTA's sums, ordered by the barrier
            const int last = atomicAdd(a.tickets + it.tile, 1) == a.splits - 1;
            if (last) a.tickets[it.tile] = 0;
            __threadfence();
            sm.is_last = last;
        }
        join_sync();
        if (sm.is_last) {
            grid_dep_wait();                     // the residual may be the kernel before's
            const int jg = (warp - kDqWarp0) >> 2, q = (warp & 3) * 32 + lane, steps = (min(a.N, a.T - it.t0) + 15) >> 4;
            const float g0 = __ldg(a.ep.global0) * 0x1p14f, g1 = Act == TFMOE_ACT_SWIGLU ? __ldg(a.ep.global1) * 0x1p14f : 0.f;
            Finisher<Act, Fast, kJoinGroups> fin(a.ep, a.T, it.rt, q, it.t0 + 16 * jg, g0, g1);
            const float *src = a.partial + ((size_t)it.tile * a.splits * a.N + 16 * jg) * kM + q;
            const size_t next = (size_t)a.N * kM;    // from a split's sums to the next's
#pragma unroll 1
            for (int st = jg; st < steps; st += kJoinGroups, src += 16 * kJoinGroups * kM) {
                // two splits' sums in flight at a time; added in split order
                uint32_t r[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) r[c] = 0u;
#pragma unroll 1
                for (int sp = 0; sp < a.splits; sp += 2) {
                    const float *p = src + sp * next, *p1 = sp + 1 < a.splits ? p + next : p;
                    float u[2][16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) { u[0][c] = __ldcg(p + c * kM); u[1][c] = __ldcg(p1 + c * kM); }
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float v = __uint_as_float(r[c]) + u[0][c];
                        r[c] = __float_as_uint(sp + 1 < a.splits ? v + u[1][c] : v);
                    }
                }
                fin.step(r);
            }
        }
    }
    __syncthreads();
    if (warp == 1) {
        if (lane == 0) mbar_wait_bounded(&sm.mma_done, 0, err);
        __syncwarp();
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
}

using TcKernel = void (*)(const CUtensorMap, const TcArgs);
template <bool Fast>
TcKernel tc_kernel(int act) {
    switch (act) {
    case TFMOE_ACT_RELU: return linear_tc_kernel<TFMOE_ACT_RELU, Fast>;
    case TFMOE_ACT_SILU: return linear_tc_kernel<TFMOE_ACT_SILU, Fast>;
    case TFMOE_ACT_GELU: return linear_tc_kernel<TFMOE_ACT_GELU, Fast>;
    case TFMOE_ACT_GELU_TANH: return linear_tc_kernel<TFMOE_ACT_GELU_TANH, Fast>;
    case TFMOE_ACT_SWIGLU: return linear_tc_kernel<TFMOE_ACT_SWIGLU, Fast>;
    default: return linear_tc_kernel<TFMOE_ACT_NONE, Fast>;
    }
}
TcKernel tc_kernel(const Linear &L) {
    return L.desc.flags & TFMOE_FLAG_OUT_FP32 ? tc_kernel<false>(L.desc.activation) : tc_kernel<true>(L.desc.activation);
}

constexpr size_t kSmemBytes = sizeof(TcSmem) + 1024;

struct TcPlan {
    int N, splits;
    double clocks;
};

// The tile width and the number of splits with the least estimated time, in clocks of an SM, fitted to
// launches of 1 to 7234 tokens over 40 weight matrices. A stage of 64 columns takes the round of its barriers and
// its MMAs; a launch ends with its last epilogue (about 30 clocks a token); splits add the sums' way to
// global memory and back.
TcPlan make_tc_plan(const Linear &L, int T) {
    TcPlan best{16, 1, 1e30};
    for (int N = 16; N <= kMaxN; N += 16) {
        const int64_t tiles = (int64_t)L.RT * ((T + N - 1) / N);
        for (int S = 1; S <= kMaxSplits && S <= L.KT; ++S) {
            if (S > 1 && tiles * S > L.num_sms) break;         // the workspace holds one wave of sums
            const int64_t waves = (tiles * S + L.num_sms - 1) / L.num_sms;
            const double stage = 420.0 + 1.1 * N, stages = (double)((L.KT + S - 1) / S);
            double t = (double)waves * (stages * stage + 600.0) + 30.0 * N + 5200.0;
            if (S > 1) t += 3500.0 + 10.0 * N + (300.0 + 9.0 * N) * S;
            if (t < best.clocks) best = {N, S, t};
        }
        if (N >= T) break;
    }
    return best;
}

}  // namespace

cudaError_t linear_tc_setup(const Linear &L)
{
    return cudaFuncSetAttribute(tc_kernel(L), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
}

double linear_tc_clocks(const Linear &L, int T) { return make_tc_plan(L, T).clocks; }

size_t linear_tc_partial_floats(const Linear &L) {
    return (size_t)L.num_sms * std::min(kMaxN, (L.desc.max_tokens + 15) & ~15) * kM;
}

cudaError_t launch_linear_tc(Linear &L, const uint16_t *x, int64_t ldx, int T, const LinearEpilogue &ep, cudaStream_t s,
                             int *launches)
{
    const TcPlan plan = make_tc_plan(L, T);
    TcArgs a{};
    a.codes = L.codes; a.scales = L.scales;
    a.T = T; a.RT = L.RT; a.KT = L.KT;
    a.N = plan.N; a.splits = plan.splits;
    a.items = L.RT * ((T + plan.N - 1) / plan.N) * plan.splits;
    a.partial = L.partial; a.tickets = L.tickets; a.err_word = L.err_word;
    a.test_wait_ns = L.test_timeout ? kLinearTestWaitNs : 0;
    a.ep = ep;
    CUtensorMap map;
    if (encode_tensor_map_2d(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, const_cast<uint16_t *>(x), (uint64_t)L.desc.in_features,
                             (uint64_t)T, (uint64_t)ldx * 2, (uint32_t)kTileK, (uint32_t)plan.N,
                             CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(std::min(L.num_sms, a.items));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, tc_kernel(L), map, a);
    *launches += 1;
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tfmoe
