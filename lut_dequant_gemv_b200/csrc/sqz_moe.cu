// sqz_moe.cu -- host side of the mixture-of-experts layer declared in
// include/sqz.h.  Every argument is checked on the host before any CUDA call.
#include <new>

#include "fp8_host.cuh"
#include "kernels_moe.cuh"

struct sqz_moe {
    sqz_moe_desc d;
    int device = 0, sms = 0, smem = 0;
    int tiles_i = 0, tiles_h = 0;
    CUtensorMap map_w13, map_w2;
};

namespace {

using namespace sqz::f8;
namespace M = sqz::moe;

constexpr int kSharedSlack = 1024;  // alignment of the ring

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// The workspace's parts for a call of `tokens`; the counters come first, at
// places that do not depend on the tokens.
struct Layout {
    size_t cnt1, cnt2, logits, xq, sx, hq, sh, part1, part2, total;
    Layout(const sqz_moe& m, int tokens) {
        const size_t pairs = (size_t)tokens * m.d.top_k;
        size_t at = up256(sizeof(M::Header));
        const auto take = [&](size_t bytes) {
            const size_t here = at;
            at += up256(bytes);
            return here;
        };
        cnt1 = take((size_t)m.d.experts * m.tiles_i * 4);
        cnt2 = take((size_t)m.tiles_h * 4);
        logits = take((size_t)tokens * m.d.experts * 8);
        xq = take((size_t)tokens * M::kDigits * m.tiles_h * 128);
        sx = take((size_t)tokens * m.tiles_h * 4);
        hq = take(pairs * M::kDigits * m.tiles_i * 128);
        sh = take(pairs * m.tiles_i * 4);
        part1 = take((size_t)m.sms * 2 * tokens * 256 * 4);
        part2 = take((size_t)m.sms * 2 * tokens * 128 * 4);
        total = at;
    }
};

sqz_status check_handle(const sqz_moe* m) {
    if (!m) return host_fail(SQZ_ERR_INVALID_ARG, "moe is NULL");
    return SQZ_OK;
}

}  // namespace

extern "C" SQZ_API sqz_status sqz_create_moe(const sqz_moe_desc* desc, sqz_moe_t* out) {
    if (!out) return host_fail(SQZ_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (!desc) return host_fail(SQZ_ERR_INVALID_ARG, "desc is NULL");
    const sqz_moe_desc& d = *desc;
    if (d.experts < 1 || d.experts > SQZ_MOE_MAX_EXPERTS)
        return host_fail(SQZ_ERR_INVALID_ARG, "experts=%d outside [1, %d]", d.experts, SQZ_MOE_MAX_EXPERTS);
    if (d.top_k < 1 || d.top_k > SQZ_MOE_MAX_TOP_K || d.top_k > d.experts)
        return host_fail(SQZ_ERR_INVALID_ARG, "top_k=%d outside [1, min(%d, experts=%d)]", d.top_k, SQZ_MOE_MAX_TOP_K,
                         d.experts);
    if (d.hidden < 16 || d.inter < 16 || d.hidden % 16 || d.inter % 16)
        return host_fail(SQZ_ERR_INVALID_ARG, "hidden=%d and inter=%d must be positive multiples of 16", d.hidden,
                         d.inter);
    // (the kernel's column indexes are 32 bits and run past the end by up to a step of the CTA)
    if (d.hidden > 1 << 30 || d.inter > 1 << 30)
        return host_fail(SQZ_ERR_UNSUPPORTED, "hidden=%d or inter=%d too large (at most 2^30)", d.hidden, d.inter);
    if (d.x_type != SQZ_TYPE_F16 && d.x_type != SQZ_TYPE_BF16)
        return host_fail(SQZ_ERR_INVALID_ARG, "x_type=%d: fp16 or bf16 expected", d.x_type);
    if (d.renormalize != 0 && d.renormalize != 1)
        return host_fail(SQZ_ERR_INVALID_ARG, "renormalize=%d: 0 or 1 expected", d.renormalize);
    if (!d.router || !d.w13 || !d.w13_scale || !d.w2 || !d.w2_scale)
        return host_fail(SQZ_ERR_INVALID_ARG, "router, w13, w2 or their scales are NULL");
    if (d.ld_router < d.hidden)
        return host_fail(SQZ_ERR_INVALID_ARG, "ld_router=%lld < hidden=%d", (long long)d.ld_router, d.hidden);
    if (reinterpret_cast<uintptr_t>(d.w13) % 16 || reinterpret_cast<uintptr_t>(d.w2) % 16)
        return host_fail(SQZ_ERR_INVALID_ARG, "w13 and w2 must start on a 16-byte boundary");
    if (reinterpret_cast<uintptr_t>(d.router) % 2 || reinterpret_cast<uintptr_t>(d.w13_scale) % 4 ||
        reinterpret_cast<uintptr_t>(d.w2_scale) % 4)
        return host_fail(SQZ_ERR_INVALID_ARG, "router must be 2-byte and the scales 4-byte aligned");
    const int64_t tiles_i = (d.inter + 127) / 128, tiles_h = (d.hidden + 127) / 128;
    if (tiles_i * tiles_h * (int64_t)(d.experts < M::kMaxPairs ? d.experts : M::kMaxPairs) > INT32_MAX)
        return host_fail(SQZ_ERR_UNSUPPORTED, "experts x hidden x inter too large (2^31 blocks of 128 x 128)");
    DeviceSizes dev;
    sqz_status st = device_sizes(&dev);
    if (st != SQZ_OK) return st;
    sqz_moe* m = new (std::nothrow) sqz_moe;
    if (!m) return host_fail(SQZ_ERR_OOM, "no host memory for the handle");
    m->d = d;
    m->device = dev.device;
    m->sms = dev.sms < M::kMaxGrid ? dev.sms : M::kMaxGrid;
    m->smem = dev.smem;
    m->tiles_i = (int)tiles_i;
    m->tiles_h = (int)tiles_h;
    st = tile_map(&m->map_w13, d.w13, d.hidden, d.inter, d.hidden, 128, (int64_t)d.experts * 2,
                  (int64_t)d.inter * d.hidden);
    if (st == SQZ_OK)
        st = tile_map(&m->map_w2, d.w2, d.inter, d.hidden, d.inter, 128, d.experts, (int64_t)d.inter * d.hidden);
    if (st != SQZ_OK) {
        delete m;
        return st;
    }
    *out = m;
    return SQZ_OK;
}

extern "C" SQZ_API sqz_status sqz_destroy_moe(sqz_moe_t moe) {
    delete moe;
    return SQZ_OK;
}

extern "C" SQZ_API sqz_status sqz_moe_workspace_bytes(sqz_moe_t moe, int32_t tokens, int64_t* bytes) {
    if (!bytes) return host_fail(SQZ_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    const sqz_status st = check_handle(moe);
    if (st != SQZ_OK) return st;
    if (tokens < 1 || tokens > SQZ_MOE_MAX_TOKENS)
        return host_fail(SQZ_ERR_INVALID_ARG, "tokens=%d outside [1, %d]", tokens, SQZ_MOE_MAX_TOKENS);
    *bytes = (int64_t)Layout(*moe, tokens).total;
    return SQZ_OK;
}

extern "C" SQZ_API sqz_status sqz_moe_forward(sqz_moe_t moe, const void* x, int32_t tokens, int64_t ldx, void* y,
                                              int64_t ldy, int32_t* ids, float* weights, void* workspace,
                                              int64_t workspace_bytes, void* stream) {
    sqz_status st = check_handle(moe);
    if (st != SQZ_OK) return st;
    if (tokens < 0 || tokens > SQZ_MOE_MAX_TOKENS)
        return host_fail(SQZ_ERR_INVALID_ARG, "tokens=%d outside [0, %d]", tokens, SQZ_MOE_MAX_TOKENS);
    if (tokens == 0) return SQZ_OK;
    if (!x || !y || !workspace) return host_fail(SQZ_ERR_INVALID_ARG, "x, y or workspace is NULL");
    const sqz_moe_desc& d = moe->d;
    if (ldx < d.hidden || ldy < d.hidden)
        return host_fail(SQZ_ERR_INVALID_ARG, "ldx=%lld or ldy=%lld < hidden=%d", (long long)ldx, (long long)ldy,
                         d.hidden);
    if (reinterpret_cast<uintptr_t>(x) % 2 || reinterpret_cast<uintptr_t>(y) % 2 ||
        reinterpret_cast<uintptr_t>(ids) % 4 || reinterpret_cast<uintptr_t>(weights) % 4)
        return host_fail(SQZ_ERR_INVALID_ARG, "x, y, ids or weights are not aligned to their types");
    if (reinterpret_cast<uintptr_t>(workspace) % 256)
        return host_fail(SQZ_ERR_INVALID_ARG, "workspace must start on a 256-byte boundary");
    const Layout L(*moe, tokens);
    if (workspace_bytes < (int64_t)L.total)
        return host_fail(SQZ_ERR_INVALID_ARG, "workspace_bytes=%lld, %lld needed for %d tokens",
                         (long long)workspace_bytes, (long long)L.total, tokens);
    DeviceSizes dev;
    if ((st = device_sizes(&dev)) != SQZ_OK) return st;
    if (dev.device != moe->device)
        return host_fail(SQZ_ERR_INVALID_ARG, "the handle was made on device %d, the current device is %d", moe->device,
                         dev.device);
    uint8_t* w = static_cast<uint8_t*>(workspace);
    M::Params p{};
    p.x = static_cast<const uint16_t*>(x);
    p.ldx = ldx;
    p.router = static_cast<const uint16_t*>(d.router);
    p.ld_router = d.ld_router;
    p.s13 = d.w13_scale;
    p.s2 = d.w2_scale;
    p.y = y;
    p.ldy = ldy;
    p.ids = ids;
    p.weights = weights;
    p.head = reinterpret_cast<M::Header*>(w);
    p.cnt1 = reinterpret_cast<int*>(w + L.cnt1);
    p.cnt2 = reinterpret_cast<int*>(w + L.cnt2);
    p.logits = reinterpret_cast<float*>(w + L.logits);
    p.logits_lo = p.logits + (size_t)tokens * d.experts;
    p.xq = w + L.xq;
    p.sx = reinterpret_cast<float*>(w + L.sx);
    p.hq = w + L.hq;
    p.sh = reinterpret_cast<float*>(w + L.sh);
    p.part1 = reinterpret_cast<float*>(w + L.part1);
    p.part2 = reinterpret_cast<float*>(w + L.part2);
    p.tokens = tokens;
    p.experts = d.experts;
    p.top_k = d.top_k;
    p.hidden = d.hidden;
    p.inter = d.inter;
    p.tiles_i = moe->tiles_i;
    p.tiles_h = moe->tiles_h;
    p.hpad = moe->tiles_h * 128;
    p.ipad = moe->tiles_i * 128;
    p.renormalize = d.renormalize;
    p.vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ldx % 8 == 0 && reinterpret_cast<uintptr_t>(d.router) % 16 == 0 &&
            d.ld_router % 8 == 0;
    p.stage_bytes = 16384 + M::b_rows(tokens) * 128;
    const int fixed = kSharedSlack + 2 * tokens * 128 * 4 + M::scratch_bytes(tokens, d.experts) + (int)sizeof(M::Shared);
    p.stages = (moe->smem - fixed) / p.stage_bytes;
    if (p.stages > M::kMaxRing) p.stages = M::kMaxRing;
    CUtensorMap mx, mh;
    if ((st = tile_map(&mx, p.xq, p.hpad, (int64_t)tokens * M::kDigits, p.hpad, M::kDigits)) != SQZ_OK) return st;
    if ((st = tile_map(&mh, p.hq, p.ipad, (int64_t)tokens * d.top_k * M::kDigits, p.ipad, M::kDigits)) != SQZ_OK)
        return st;
    const bool bf16 = d.x_type == SQZ_TYPE_BF16;
    const auto kernel = bf16 ? M::moe_kernel<true> : M::moe_kernel<false>;
    static std::atomic<uint64_t> ready[2];
    if ((st = allow_smem(kernel, dev, &ready[bf16])) != SQZ_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)moe->sms);
    cfg.blockDim = dim3(M::kThreads);
    cfg.dynamicSmemBytes = (size_t)(fixed + p.stages * p.stage_bytes);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    SQZ_F8_TRY(cudaLaunchKernelEx(&cfg, kernel, moe->map_w13, moe->map_w2, mx, mh, p), "moe launch");
    return SQZ_OK;
}

extern "C" SQZ_API sqz_status sqz_moe_status(void* workspace, void* stream, int32_t* status) {
    if (!status || !workspace) return host_fail(SQZ_ERR_INVALID_ARG, "workspace or status is NULL");
    *status = 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    SQZ_F8_TRY(cudaStreamIsCapturing(s, &cap), "cudaStreamIsCapturing");
    if (cap != cudaStreamCaptureStatusNone)
        return host_fail(SQZ_ERR_UNSUPPORTED, "the stream is being captured into a CUDA graph; reading the status "
                                              "synchronises, which a capture cannot contain");
    M::Header h{};
    SQZ_F8_TRY(cudaMemcpyAsync(&h, workspace, sizeof h, cudaMemcpyDeviceToHost, s), "reading the status");
    SQZ_F8_TRY(cudaStreamSynchronize(s), "reading the status");
    *status = h.status;
    if (h.status & 1)
        return host_fail(SQZ_ERR_TIMEOUT, "a bounded device wait gave up (status 0x%x): y of the affected call is "
                                          "undefined; zero the workspace before its next use", h.status);
    return SQZ_OK;
}
