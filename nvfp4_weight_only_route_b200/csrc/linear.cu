// linear.cu -- the C ABI of the NVFP4 matrix product (tfmoe_linear_* in tfmoe.h): argument
// checks, weight storage and repacking, and the choice of the regime.
#include <algorithm>
#include <cstdlib>
#include <new>

#include "linear.h"

using namespace tfmoe;

struct tfmoe_linear {
    Linear impl;
};

namespace tfmoe {
namespace {

// One thread per (tiled row, column tile) copies 32 code bytes and 4 scale bytes into the
// 128 x 64 tile layout of repack.cu, except that the eight codes of a word are kept in the order
// 0 2 4 6 1 3 5 7 (linear_tc.cu says why); rows and columns past the matrix are zero. The source
// may start anywhere and its rows are K/2 and K/16 bytes long, so it is read byte by byte.
__global__ void __launch_bounds__(256) linear_repack_kernel(
    const uint8_t *__restrict__ codes0, const uint8_t *__restrict__ scales0, const uint8_t *__restrict__ codes1,
    const uint8_t *__restrict__ scales1, int rows, int K, int RT, int KT, uint8_t *__restrict__ out_codes,
    uint8_t *__restrict__ out_scales)
{
    const size_t n = (size_t)RT * kTileRows * KT;
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x) {
        const int kt = (int)(i % KT), r = (int)(i / KT);
        const bool up = codes1 && (r & 1);
        const int src = codes1 ? r >> 1 : r;
        const uint8_t *c = (up ? codes1 : codes0) + (size_t)src * (K / 2) + (size_t)kt * 32;
        const uint8_t *sc = (up ? scales1 : scales0) + (size_t)src * (K / 16) + (size_t)kt * 4;
        const int nc = r < rows ? min(32, K / 2 - kt * 32) : 0, ns = r < rows ? min(4, K / 16 - kt * 4) : 0;
        const size_t tile = (size_t)(r / kTileRows) * KT + kt;
        uint8_t *ct = out_codes + tile * kTileCodeBytes + (r % kTileRows) * 16;
        uint8_t *st = out_scales + tile * kTileScaleBytes + (r % kTileRows) * 4;
        for (int w = 0; w < 8; ++w) {
            uint32_t lo = 0, hi = 0;                     // codes 0 2 4 6 and 1 3 5 7
            for (int b = 0; b < 4; ++b) {
                const uint32_t v = 4 * w + b < nc ? c[4 * w + b] : 0u;
                lo |= (v & 15u) << (4 * b);
                hi |= (v >> 4) << (4 * b);
            }
            *reinterpret_cast<uint32_t *>(ct + (w >> 2) * 2048 + (w & 3) * 4) = lo | hi << 16;
        }
        for (int b = 0; b < 4; ++b) st[b] = b < ns ? sc[b] : 0;
    }
}

}  // namespace

cudaError_t launch_linear_repack(const Linear &L, const tfmoe_linear_weights &w, cudaStream_t s)
{
    const bool gated = linear_gated(L);
    linear_repack_kernel<<<4 * L.num_sms, 256, 0, s>>>(w.codes, w.scales, gated ? w.up_codes : nullptr,
                                                       gated ? w.up_scales : nullptr, L.rows, L.desc.in_features,
                                                       L.RT, L.KT, L.codes, L.scales);
    return cudaGetLastError();
}

}  // namespace tfmoe

namespace {

struct DeviceGuard {
    int prev = -1;
    bool changed = false;
    explicit DeviceGuard(int dev) {
        if (cudaGetDevice(&prev) == cudaSuccess && prev != dev) changed = (cudaSetDevice(dev) == cudaSuccess);
    }
    ~DeviceGuard() { if (changed) cudaSetDevice(prev); }
};

tfmoe_status cuda_fail(cudaError_t e, const char *where) {
    return record_error(e == cudaErrorMemoryAllocation ? TFMOE_ERR_OOM : TFMOE_ERR_CUDA, "%s: %s (%s)", where,
                        cudaGetErrorName(e), cudaGetErrorString(e));
}

// T rows of `width` bytes, `stride` bytes apart.
struct Rows {
    uintptr_t at;
    uint64_t width, stride;
    int T;
    uint64_t span() const { return (uint64_t)(T - 1) * stride + width; }
};

// Whether two row sets share a byte. Rows of one stride that do not wrap share bytes only where
// their column ranges do (two slices of one wider buffer); for other strides touching spans
// count as overlapping.
bool overlap(const Rows &a, const Rows &b) {
    if (!a.at || !b.at) return false;
    if (a.at >= b.at + b.span() || b.at >= a.at + a.span()) return false;
    if (a.stride != b.stride || a.T == 1) return true;
    const uint64_t d = a.at <= b.at ? (b.at - a.at) % a.stride : (a.stride - (a.at - b.at) % a.stride) % a.stride;
    return !(d >= a.width && d + b.width <= a.stride);
}

}  // namespace

extern "C" {

tfmoe_status tfmoe_linear_create(const tfmoe_linear_desc *desc, tfmoe_linear **out)
{
    if (!out) return record_error(TFMOE_ERR_INVALID_ARG, "tfmoe_linear_create: out is NULL");
    *out = nullptr;
    if (!desc) return record_error(TFMOE_ERR_INVALID_ARG, "tfmoe_linear_create: desc is NULL");
    const tfmoe_linear_desc d = *desc;
    if (d.in_features <= 0 || d.in_features % 16)
        return record_error(TFMOE_ERR_INVALID_ARG, "in_features (%d) must be a positive multiple of 16", d.in_features);
    if (d.out_features <= 0) return record_error(TFMOE_ERR_INVALID_ARG, "out_features (%d) must be >= 1", d.out_features);
    if (d.max_tokens <= 0) return record_error(TFMOE_ERR_INVALID_ARG, "max_tokens (%d) must be >= 1", d.max_tokens);
    if (d.activation < TFMOE_ACT_NONE || d.activation > TFMOE_ACT_SWIGLU)
        return record_error(TFMOE_ERR_INVALID_ARG, "unknown activation %d", d.activation);
    if ((d.flags & TFMOE_FLAG_FORCE_GEMV) && (d.flags & TFMOE_FLAG_FORCE_MMA))
        return record_error(TFMOE_ERR_INVALID_ARG, "FORCE_GEMV and FORCE_MMA are exclusive");
    if (d.flags & ~(TFMOE_FLAG_FORCE_GEMV | TFMOE_FLAG_FORCE_MMA | TFMOE_FLAG_OUT_FP32 | TFMOE_FLAG_TEST_TIMEOUT))
        return record_error(TFMOE_ERR_INVALID_ARG, "unknown flag bits 0x%x", d.flags);
    if (d.in_features > (1 << 16) || d.out_features > (1 << 20) || d.max_tokens > (1 << 20))
        return record_error(TFMOE_ERR_UNSUPPORTED, "tfmoe_linear supports in_features <= 65536, out_features <= 2^20 and "
                            "max_tokens <= 2^20 (got %d, %d, %d)", d.in_features, d.out_features, d.max_tokens);
    const char *fail_env = getenv("TFMOE_FAIL_ALLOC");
    if (fail_env && atoi(fail_env) != 0)
        return record_error(TFMOE_ERR_OOM, "tfmoe_linear_create: allocation failure injected by TFMOE_FAIL_ALLOC");

    tfmoe_linear *h = new (std::nothrow) tfmoe_linear();
    if (!h) return record_error(TFMOE_ERR_OOM, "tfmoe_linear_create: host allocation failed");
    Linear &L = h->impl;
    L.desc = d;
    L.test_timeout = (d.flags & TFMOE_FLAG_TEST_TIMEOUT) != 0;
    L.rows = linear_gated(L) ? 2 * d.out_features : d.out_features;
    L.RT = (L.rows + kTileRows - 1) / kTileRows;
    L.KT = (d.in_features + kTileK - 1) / kTileK;
    cudaError_t e = cudaGetDevice(&L.device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&L.num_sms, cudaDevAttrMultiProcessorCount, L.device);
    if (e != cudaSuccess) { delete h; return cuda_fail(e, "tfmoe_linear_create: device query"); }
    const size_t tiles = (size_t)L.RT * L.KT;
    const size_t small = 256 + (((size_t)L.rows * 4 + 255) & ~(size_t)255);      // global, bias
    e = cudaMalloc(&L.w_block, tiles * (kTileCodeBytes + kTileScaleBytes) + small);
    L.zero_bytes = (256 + (size_t)std::max(L.RT, L.num_sms) * 4 + 255) & ~(size_t)255;
    const size_t sums = std::max(linear_stream_partial_floats(L), linear_tc_partial_floats(L));
    if (e == cudaSuccess) e = cudaMalloc(&L.ws_block, L.zero_bytes + sums * 4);
    if (e == cudaSuccess) e = cudaMemset(L.ws_block, 0, L.zero_bytes);
    if (e == cudaSuccess) e = linear_stream_setup(L);
    if (e == cudaSuccess) e = linear_tc_setup(L);
    if (e != cudaSuccess) {
        cudaGetLastError();
        if (L.w_block) cudaFree(L.w_block);
        if (L.ws_block) cudaFree(L.ws_block);
        delete h;
        return cuda_fail(e, "tfmoe_linear_create");
    }
    L.codes = static_cast<uint8_t *>(L.w_block);
    L.scales = L.codes + tiles * kTileCodeBytes;
    L.global = reinterpret_cast<float *>(L.scales + tiles * kTileScaleBytes);
    L.bias = L.global + 64;
    L.err_word = static_cast<int32_t *>(L.ws_block);
    L.tickets = L.err_word + 64;
    L.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(L.ws_block) + L.zero_bytes);
    *out = h;
    return record_ok();
}

tfmoe_status tfmoe_linear_load_weights(tfmoe_linear *lin, const tfmoe_linear_weights *w)
{
    if (!lin || !w) return record_error(TFMOE_ERR_INVALID_ARG, "tfmoe_linear_load_weights: NULL argument");
    Linear &L = lin->impl;
    const bool gated = linear_gated(L);
    if (!w->codes || !w->scales || !w->global || (gated && (!w->up_codes || !w->up_scales || !w->up_global)))
        return record_error(TFMOE_ERR_INVALID_ARG, "tfmoe_linear_load_weights: a required weight pointer is NULL");
    if (L.desc.has_bias && !w->bias)
        return record_error(TFMOE_ERR_INVALID_ARG, "tfmoe_linear_load_weights: has_bias but bias is NULL");
    const void *f32[] = {w->global, gated ? w->up_global : nullptr, L.desc.has_bias ? w->bias : nullptr};
    for (const void *p : f32)
        if (reinterpret_cast<uintptr_t>(p) & 3u)
            return record_error(TFMOE_ERR_INVALID_ARG, "tfmoe_linear_load_weights: fp32 arrays must be 4-byte aligned");
    DeviceGuard dg(L.device);
    cudaStream_t s;
    // the caller's tensors may still be being written, and forwards may still read the old weights
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaStreamCreateWithFlags(&s, cudaStreamNonBlocking);
    if (e != cudaSuccess) return cuda_fail(e, "tfmoe_linear_load_weights: stream");
    e = cudaMemcpyAsync(L.global, w->global, 4, cudaMemcpyDeviceToDevice, s);
    if (e == cudaSuccess && gated) e = cudaMemcpyAsync(L.global + 1, w->up_global, 4, cudaMemcpyDeviceToDevice, s);
    if (e == cudaSuccess && L.desc.has_bias)
        e = cudaMemcpyAsync(L.bias, w->bias, (size_t)L.rows * 4, cudaMemcpyDeviceToDevice, s);
    if (e == cudaSuccess) e = launch_linear_repack(L, *w, s);
    const cudaError_t e2 = cudaStreamSynchronize(s);
    cudaStreamDestroy(s);
    if (e == cudaSuccess) e = e2;
    if (e != cudaSuccess) { L.loaded = false; return cuda_fail(e, "tfmoe_linear_load_weights"); }
    L.loaded = true;
    return record_ok();
}

tfmoe_status tfmoe_linear_forward(tfmoe_linear *lin, const uint16_t *x, int64_t ldx, int32_t T,
                                  const uint16_t *residual, int64_t ldr, void *out, int64_t ldo, void *cuda_stream)
{
    const char *who = "tfmoe_linear_forward";
    if (!lin) return record_error(TFMOE_ERR_INVALID_ARG, "%s: lin is NULL", who);
    Linear &L = lin->impl;
    L.last_launches = 0;
    if (!L.loaded) return record_error(TFMOE_ERR_NOT_LOADED, "%s: weights not loaded", who);
    if (T < 0 || T > L.desc.max_tokens)
        return record_error(TFMOE_ERR_INVALID_ARG, "%s: T=%d outside [0, max_tokens=%d]", who, T, L.desc.max_tokens);
    if (T == 0) return record_ok();
    if (!x || !out) return record_error(TFMOE_ERR_INVALID_ARG, "%s: x or out is NULL", who);
    const int K = L.desc.in_features, N = L.desc.out_features;
    const bool f32 = (L.desc.flags & TFMOE_FLAG_OUT_FP32) != 0;
    const int64_t lim = 1LL << 40;
    if (ldx < K || ldo < N || (residual && ldr < N) || ldx > lim || ldo > lim || (residual && ldr > lim))
        return record_error(TFMOE_ERR_INVALID_ARG, "%s: row strides ldx=%lld, ldr=%lld, ldo=%lld must hold a row "
                            "(K=%d, N=%d)", who, (long long)ldx, (long long)ldr, (long long)ldo, K, N);
    if ((reinterpret_cast<uintptr_t>(x) & 15u) || ldx % 8)
        return record_error(TFMOE_ERR_INVALID_ARG, "%s: x must be 16-byte aligned and ldx (%lld) a multiple of 8", who,
                            (long long)ldx);
    if ((reinterpret_cast<uintptr_t>(residual) & 1u) || (reinterpret_cast<uintptr_t>(out) & (f32 ? 3u : 1u)))
        return record_error(TFMOE_ERR_INVALID_ARG, "%s: residual and out must be aligned to their element", who);
    if ((L.desc.flags & TFMOE_FLAG_FORCE_GEMV) && !linear_stream_fits(L, T))
        return record_error(TFMOE_ERR_UNSUPPORTED, "%s: the streaming regime takes at most 16 tokens whose rows fit in "
                            "shared memory (T=%d, K=%d)", who, T, K);
    const uint64_t es = f32 ? 4 : 2;
    const Rows rx{reinterpret_cast<uintptr_t>(x), (uint64_t)K * 2, (uint64_t)ldx * 2, T};
    const Rows ro{reinterpret_cast<uintptr_t>(out), (uint64_t)N * es, (uint64_t)ldo * es, T};
    const Rows rr{reinterpret_cast<uintptr_t>(residual), (uint64_t)N * 2, (uint64_t)ldr * 2, T};
    const bool in_place = !f32 && residual == out && (ldr == ldo || T == 1);
    if (overlap(rx, ro) || (residual && !in_place && overlap(rr, ro)))
        return record_error(TFMOE_ERR_INVALID_ARG, "%s: out overlaps x or residual (only residual == out, bf16, with the "
                            "same ld is allowed)", who);

    DeviceGuard dg(L.device);
    LinearEpilogue ep{};
    ep.global0 = L.global;
    ep.global1 = L.global + 1;
    ep.bias = L.desc.has_bias ? L.bias : nullptr;
    ep.residual = residual;
    ep.ldr = ldr;
    ep.out = out;
    ep.ldo = ldo;
    ep.N = N;
    ep.act = L.desc.activation;
    ep.out_fp32 = f32;
    int n = 0;
    const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    bool stream = linear_stream_fits(L, T) && !(L.desc.flags & TFMOE_FLAG_FORCE_MMA);
    if (stream && !(L.desc.flags & TFMOE_FLAG_FORCE_GEMV)) stream = linear_stream_clocks(L, T) <= linear_tc_clocks(L, T);
    const cudaError_t e = stream ? launch_linear_stream(L, x, ldx, T, ep, s, &n) : launch_linear_tc(L, x, ldx, T, ep, s, &n);
    L.last_launches = n;
    L.test_timeout = false;
    if (e != cudaSuccess) return cuda_fail(e, who);
    return record_ok();
}

tfmoe_status tfmoe_linear_sync_status(tfmoe_linear *lin, void *cuda_stream)
{
    if (!lin) return record_error(TFMOE_ERR_INVALID_ARG, "tfmoe_linear_sync_status: lin is NULL");
    Linear &L = lin->impl;
    DeviceGuard dg(L.device);
    const cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    cudaError_t e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "tfmoe_linear_sync_status");
    int32_t word = 0;
    e = cudaMemcpy(&word, L.err_word, sizeof word, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && word != 0) {
        // done before this returns: the next forward may run on any stream
        e = cudaMemsetAsync(L.ws_block, 0, L.zero_bytes, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    if (e != cudaSuccess) return cuda_fail(e, "tfmoe_linear_sync_status: error word");
    if (word) return record_error(TFMOE_ERR_TIMEOUT, "a device-side wait timed out (word 0x%x)", word);
    return record_ok();
}

int32_t tfmoe_linear_last_launch_count(tfmoe_linear *lin) { return lin ? lin->impl.last_launches : 0; }

void tfmoe_linear_destroy(tfmoe_linear *lin)
{
    if (!lin) return;
    {
        DeviceGuard dg(lin->impl.device);
        if (lin->impl.w_block) cudaFree(lin->impl.w_block);
        if (lin->impl.ws_block) cudaFree(lin->impl.ws_block);
    }
    delete lin;
}

}  // extern "C"
