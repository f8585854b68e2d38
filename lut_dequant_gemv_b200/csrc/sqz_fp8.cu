// sqz_fp8.cu -- host side of the block-scaled 8-bit quantizer and matrix
// product declared in include/sqz.h.  Every argument is checked on the host
// before any CUDA call.
#include <algorithm>

#include "fp8_host.cuh"
#include "kernels_fp8.cuh"
#include "timeouts.cuh"

namespace {

using namespace sqz::f8;

// Counts, on every GPU, the CTAs of products whose bounded wait gave up; read by
// sqz_fp8_status, which reports each once.
__device__ uint32_t g_fp8_timeouts;
constexpr int kMaxDevices = 256;
sqz::ReportedTimeouts g_reported[kMaxDevices];

sqz_status timeout_count(uint32_t** out) {
    void* p = nullptr;
    SQZ_F8_TRY(cudaGetSymbolAddress(&p, g_fp8_timeouts), "cudaGetSymbolAddress(fp8 timeouts)");
    *out = static_cast<uint32_t*>(p);
    return SQZ_OK;
}

bool aligned16(const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 16 == 0; }

template <class Params>
cudaError_t launch(void (*kernel)(const Params), dim3 grid, int threads, const Params& prm, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, prm);
}

template <bool BF16, bool E5M2, int ALIGN>
cudaError_t launch_quantize(const QuantParams& p, int block_rows, int sms, cudaStream_t s) {
    if (block_rows == 1) {
        const int64_t blocks = p.batch * p.rows * p.nblocks;
        if (blocks <= (int64_t)sms * 32 * 4)
            return launch(fp8_quantize_rows_kernel<BF16, E5M2, ALIGN, 1>, dim3((unsigned)((blocks + 31) / 32)), 256, p, s);
        const int64_t ctas = (blocks + 63) / 64, most = (int64_t)sms * 8 * 4;  // then each strides
        return launch(fp8_quantize_rows_kernel<BF16, E5M2, ALIGN, 2>, dim3((unsigned)(ctas < most ? ctas : most)), 256,
                      p, s);
    }
    return launch(fp8_quantize_tiles_kernel<BF16, E5M2, ALIGN>,
                  dim3((unsigned)p.nblocks, (unsigned)(p.batch * ((p.rows + 127) / 128))), 256, p, s);
}

template <bool BF16, bool E5M2>
cudaError_t launch_quantize(const QuantParams& p, int block_rows, int align, int sms, cudaStream_t s) {
    switch (align) {
        case kWhole: return launch_quantize<BF16, E5M2, kWhole>(p, block_rows, sms, s);
        case 16: return launch_quantize<BF16, E5M2, 16>(p, block_rows, sms, s);
        case 8: return launch_quantize<BF16, E5M2, 8>(p, block_rows, sms, s);
        case 4: return launch_quantize<BF16, E5M2, 4>(p, block_rows, sms, s);
        default: return launch_quantize<BF16, E5M2, 2>(p, block_rows, sms, s);
    }
}

// ------------------------------------------------------------ the product
int round_pow2(int v) {
    int p = 16;
    while (p < v) p *= 2;
    return p;
}

template <int TB>
sqz_status launch_few(const CUtensorMap& mw, const CUtensorMap& ma, GemmParams p, int splits, int stages,
                      const DeviceSizes& d, cudaStream_t s) {
    static std::atomic<uint64_t> ready;
    const sqz_status st = allow_smem(fp8_gemm_few_kernel<TB>, d, &ready);
    if (st != SQZ_OK) return st;
    p.stages = stages;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)splits, (unsigned)((p.n + 127) / 128), (unsigned)((p.m + TB - 1) / TB));
    cfg.blockDim = dim3(FewShape<TB>::kThreads);
    cfg.dynamicSmemBytes = (size_t)FewShape<TB>::smem_bytes(stages);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    SQZ_F8_TRY(cudaLaunchKernelEx(&cfg, fp8_gemm_few_kernel<TB>, mw, ma, p), "fp8 product launch");
    return SQZ_OK;
}

template <int BN, int V>
sqz_status launch_many(const CUtensorMap& mw, const CUtensorMap& ma, GemmParams p, const DeviceSizes& d,
                       cudaStream_t s) {
    static std::atomic<uint64_t> ready;
    const sqz_status st = allow_smem(fp8_gemm_many_kernel<BN, V>, d, &ready);
    if (st != SQZ_OK) return st;
    p.tiles_m = (p.m + 255) / 256;
    p.tiles_n = (p.n + BN - 1) / BN;
    const int stages = (d.smem - 512 - ManyShape<BN>::smem_bytes(0)) / ManyShape<BN>::kStageBytes;  // 512: static
    p.stages = stages > 8 ? 8 : stages;
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, pairs = d.sms / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    cfg.blockDim = dim3(ManyShape<BN>::kThreads);
    cfg.dynamicSmemBytes = (size_t)ManyShape<BN>::smem_bytes(p.stages);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    SQZ_F8_TRY(cudaLaunchKernelEx(&cfg, fp8_gemm_many_kernel<BN, V>, mw, ma, p), "fp8 product launch");
    return SQZ_OK;
}

// By the alignment of y's rows: 16 bytes, or 4, 2 or 1 values (of up to 8 bytes) at once.
template <int BN>
sqz_status launch_many(const CUtensorMap& mw, const CUtensorMap& ma, const GemmParams& p, const DeviceSizes& d,
                       cudaStream_t s) {
    if (p.out_align >= 16) return launch_many<BN, 0>(mw, ma, p, d, s);
    switch (p.out_align / (p.out_type == SQZ_TYPE_F32 ? 4 : 2)) {
        case 4: return launch_many<BN, 4>(mw, ma, p, d, s);
        case 2: return launch_many<BN, 2>(mw, ma, p, d, s);
        default: return launch_many<BN, 1>(mw, ma, p, d, s);
    }
}

// Rows of a few-row kernel's token tile; up to here it takes the call whatever W
// is (4096 x 4096: 64 rows 10 us, by the many-row kernel 13).
constexpr int kFewRows = 64;

// Which kernel takes a product, and how it cuts it.
struct Plan {
    bool many;       // many rows of A
    int tile_w;      // many: columns of y a tile (rows of W); few: 128
    int tile_a;      // many: 256; few: rows of A a tile, 16, 32 or 64
    int splits;      // few: CTAs of a cluster that share K
};

Plan plan_product(int32_t m, int32_t n, int32_t k, int sms) {
    const int nkb = (k + 127) / 128;
    const int64_t row_blocks = ((int64_t)n + 127) / 128;
    // Many rows: the width of the tiles with the least rounds of the pairs of SMs
    // times a tile's time for a block of K, which measured 0.29, 0.35 and 0.56 us
    // for 64, 128 and 256 columns: about 180 + 1.5 width ns.
    const int64_t tm = ((int64_t)m + 255) / 256, pairs = std::max(1, sms / 2);
    int bn = 256;
    int64_t many = INT64_MAX;
    for (int width : {256, 192, 160, 128, 64}) {
        const int64_t tiles = tm * (((int64_t)n + width - 1) / width);
        const int64_t ns = 5000 + (tiles + pairs - 1) / pairs * nkb * (180 + width * 3 / 2);
        if (ns < many) many = ns, bn = width;
    }
    // Few rows: K split over up to 8 CTAs of a cluster, while the grid stays
    // within 7/8 of the two CTAs an SM has room for: clusters do not fill the
    // rest, and those left over run alone (16 x 5120 x 13824: 4, 6 and 7 CTAs
    // 16.4, 16.6 and 24.5 us; 1 x 5120 x 5120: 8.1, 7.5 and 11.6 us).
    const int tb = m < kFewRows ? round_pow2(m) : kFewRows;
    const int64_t blocks = row_blocks * (((int64_t)m + tb - 1) / tb);
    int splits = (int)std::min<int64_t>(std::min(8, nkb), (int64_t)sms * 7 / 4 / blocks);
    if (splits < 1) splits = 1;
    // Beyond 64 rows the few-row kernel serves products with so little W that the
    // many-row kernel's pairs would stand idle (it does not split K): a CTA's block
    // of K takes about 400 ns (100 x 300 x 13824: 39 us, 12 this way; 128 x 4096 x
    // 4096: 13.1 and 11.9).
    const int64_t few = 5000 + (blocks * splits + sms - 1) / sms * ((nkb + splits - 1) / splits) * 400;
    if ((m <= kFewRows || few < many) && row_blocks <= 65535) return {false, 128, tb, splits};
    return {true, bn, 256, 1};
}

sqz_status check_matrix(const sqz_fp8_matrix* x, const char* name, int64_t rows, int32_t k) {
    if (!x) return host_fail(SQZ_ERR_INVALID_ARG, "%s is NULL", name);
    if (x->format != SQZ_FP8_E4M3 && x->format != SQZ_FP8_E5M2)
        return host_fail(SQZ_ERR_INVALID_ARG, "%s: unknown 8-bit format %d", name, x->format);
    if (rows == 0 || k == 0) return SQZ_OK;
    if (!x->q || !x->scale) return host_fail(SQZ_ERR_INVALID_ARG, "%s: codes or scales are NULL", name);
    if (x->ld < k) return host_fail(SQZ_ERR_INVALID_ARG, "%s: ld=%lld < k=%d", name, (long long)x->ld, k);
    if (x->ld_scale < (k + 127) / 128)
        return host_fail(SQZ_ERR_INVALID_ARG, "%s: ld_scale=%lld < %d blocks", name, (long long)x->ld_scale,
                         (k + 127) / 128);
    if (!aligned16(x->q, x->ld))
        return host_fail(SQZ_ERR_INVALID_ARG, "%s: codes must start on a 16-byte boundary with a pitch (ld) that is a "
                                              "multiple of 16", name);
    if (x->ld >= (int64_t)1 << 40) return host_fail(SQZ_ERR_INVALID_ARG, "%s: ld too large", name);
    if (reinterpret_cast<uintptr_t>(x->scale) % 4)
        return host_fail(SQZ_ERR_INVALID_ARG, "%s: scales must be 4-byte aligned", name);
    return SQZ_OK;
}

}  // namespace

extern "C" SQZ_API sqz_status sqz_fp8_quantize(const void* x, int32_t x_type, int64_t batch, int32_t rows,
                                               int32_t cols, int64_t ldx, int32_t block_rows, int32_t format,
                                               uint8_t* q, int64_t ldq, float* scale, int64_t ld_scale, void* stream) {
    if (x_type != SQZ_TYPE_F16 && x_type != SQZ_TYPE_BF16)
        return host_fail(SQZ_ERR_INVALID_ARG, "x_type=%d: fp16 or bf16 expected", x_type);
    if (format != SQZ_FP8_E4M3 && format != SQZ_FP8_E5M2)
        return host_fail(SQZ_ERR_INVALID_ARG, "unknown 8-bit format %d", format);
    if (block_rows != 1 && block_rows != 128)
        return host_fail(SQZ_ERR_INVALID_ARG, "block_rows=%d: 1 or 128 expected", block_rows);
    if (batch < 0 || rows < 0 || cols < 0)
        return host_fail(SQZ_ERR_INVALID_ARG, "negative size (batch=%lld, rows=%d, cols=%d)", (long long)batch, rows,
                         cols);
    if (rows > INT32_MAX - 127 || cols > INT32_MAX - 127) return host_fail(SQZ_ERR_INVALID_ARG, "rows or cols too large");
    if (batch == 0 || rows == 0 || cols == 0) return SQZ_OK;
    if (!x || !q || !scale) return host_fail(SQZ_ERR_INVALID_ARG, "x, q or scale is NULL");
    const int nblocks = (cols + 127) / 128;
    if (ldx < cols || ldq < cols || ld_scale < nblocks)
        return host_fail(SQZ_ERR_INVALID_ARG, "ldx=%lld, ldq=%lld or ld_scale=%lld too small for %d columns",
                         (long long)ldx, (long long)ldq, (long long)ld_scale, cols);
    if (!aligned16(q, ldq))
        return host_fail(SQZ_ERR_INVALID_ARG, "q must start on a 16-byte boundary with a pitch (ldq) that is a multiple "
                                              "of 16");
    if (reinterpret_cast<uintptr_t>(x) % 2 || reinterpret_cast<uintptr_t>(scale) % 4)
        return host_fail(SQZ_ERR_INVALID_ARG, "x must be 2-byte and scale 4-byte aligned");
    if (batch > (int64_t)1 << 31 || (block_rows == 128 && batch * ((rows + 127) / 128) > 65535) ||
        batch * rows > ((int64_t)1 << 62) / nblocks)
        return host_fail(SQZ_ERR_UNSUPPORTED, "too many row blocks (at most 65535 of 128 rows in one call)");
    DeviceSizes d;
    const sqz_status st = device_sizes(&d);
    if (st != SQZ_OK) return st;
    QuantParams p{};
    p.x = static_cast<const uint16_t*>(x);
    p.ldx = ldx;
    p.q = q;
    p.ldq = ldq;
    p.scale = scale;
    p.lds = ld_scale;
    p.batch = batch;
    p.rows = rows;
    p.cols = cols;
    p.nblocks = nblocks;
    int align = 16;  // of every row
    while (align > 2 && (reinterpret_cast<uintptr_t>(x) % align || ldx * 2 % align)) align /= 2;
    if (align == 16 && cols % 128 == 0) align = kWhole;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool bf16 = x_type == SQZ_TYPE_BF16, e5m2 = format == SQZ_FP8_E5M2;
    const cudaError_t e = bf16 ? e5m2 ? launch_quantize<true, true>(p, block_rows, align, d.sms, s)
                                      : launch_quantize<true, false>(p, block_rows, align, d.sms, s)
                          : e5m2 ? launch_quantize<false, true>(p, block_rows, align, d.sms, s)
                                 : launch_quantize<false, false>(p, block_rows, align, d.sms, s);
    SQZ_F8_TRY(e, "fp8 quantize launch");
    return SQZ_OK;
}

extern "C" SQZ_API sqz_status sqz_fp8_gemm(const sqz_fp8_matrix* a, const sqz_fp8_matrix* w, int32_t m, int32_t n,
                                           int32_t k, void* y, int64_t ldy, int32_t y_type, void* stream) {
    if (m < 0 || n < 0 || k < 0) return host_fail(SQZ_ERR_INVALID_ARG, "negative size (m=%d, n=%d, k=%d)", m, n, k);
    if (m > INT32_MAX - 256 || n > INT32_MAX - 256 || k > INT32_MAX - 256)
        return host_fail(SQZ_ERR_INVALID_ARG, "size too large (m=%d, n=%d, k=%d)", m, n, k);
    if (y_type != SQZ_TYPE_F16 && y_type != SQZ_TYPE_BF16 && y_type != SQZ_TYPE_F32)
        return host_fail(SQZ_ERR_INVALID_ARG, "unknown y_type %d", y_type);
    sqz_status st = check_matrix(a, "a", m, k);
    if (st != SQZ_OK) return st;
    if ((st = check_matrix(w, "w", n, k)) != SQZ_OK) return st;
    if (m == 0 || n == 0) return SQZ_OK;
    if (!y) return host_fail(SQZ_ERR_INVALID_ARG, "y is NULL");
    if (ldy < n) return host_fail(SQZ_ERR_INVALID_ARG, "ldy=%lld < n=%d", (long long)ldy, n);
    const int out_bytes = y_type == SQZ_TYPE_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(y) % out_bytes) return host_fail(SQZ_ERR_INVALID_ARG, "y is not aligned to its type");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (k == 0) {  // an empty sum (+0 is all-zero bits in every output type)
        SQZ_F8_TRY(cudaMemset2DAsync(y, (size_t)ldy * out_bytes, 0, (size_t)n * out_bytes, (size_t)m, s), "clearing y");
        return SQZ_OK;
    }
    DeviceSizes d;
    if ((st = device_sizes(&d)) != SQZ_OK) return st;
    GemmParams p{};
    p.sa = a->scale;
    p.ld_sa = a->ld_scale;
    p.sw = w->scale;
    p.ld_sw = w->ld_scale;
    p.y = y;
    p.ldy = ldy;
    p.m = m;
    p.n = n;
    p.nkb = (k + 127) / 128;
    p.out_type = y_type;
    p.out_align = 32;
    while (p.out_align > 2 && (reinterpret_cast<uintptr_t>(y) % p.out_align || ldy * out_bytes % p.out_align))
        p.out_align /= 2;
    if ((st = timeout_count(&p.status)) != SQZ_OK) return st;
    CUtensorMap mw, ma;
    const Plan plan = plan_product(m, n, k, d.sms);
    if (!plan.many) {
        const int tb = plan.tile_a, splits = plan.splits;
        if ((st = tile_map(&mw, w->q, k, n, w->ld, 128)) != SQZ_OK) return st;
        if ((st = tile_map(&ma, a->q, k, m, a->ld, tb)) != SQZ_OK) return st;
        p.idesc = instr_desc(w->format, a->format, 128, tb);
        const int per_cta = (p.nkb + splits - 1) / splits;
        const int stage = tb * 128 + 16384 + (tb + 4) * 4;
        int stages = (d.smem / 2 - 4096) / stage;  // two CTAs share an SM
        if (stages > kMaxStages) stages = kMaxStages;
        if (stages > per_cta) stages = per_cta;
        if (stages < 1 || (int64_t)stages * (16384 + tb * 128) < (int64_t)tb * 512) stages = (tb * 512) / (16384 + tb * 128) + 1;
        switch (tb) {
            case 16: return launch_few<16>(mw, ma, p, splits, stages, d, s);
            case 32: return launch_few<32>(mw, ma, p, splits, stages, d, s);
            default: return launch_few<64>(mw, ma, p, splits, stages, d, s);
        }
    }
    const int bn = plan.tile_w;
    if ((st = tile_map(&mw, w->q, k, n, w->ld, bn / 2)) != SQZ_OK) return st;
    if ((st = tile_map(&ma, a->q, k, m, a->ld, 128)) != SQZ_OK) return st;
    p.idesc = instr_desc(a->format, w->format, 256, bn);
    switch (bn) {
        case 256: return launch_many<256>(mw, ma, p, d, s);
        case 192: return launch_many<192>(mw, ma, p, d, s);
        case 160: return launch_many<160>(mw, ma, p, d, s);
        case 128: return launch_many<128>(mw, ma, p, d, s);
        default: return launch_many<64>(mw, ma, p, d, s);
    }
}

extern "C" SQZ_API sqz_status sqz_fp8_status(void* stream, int32_t* status) {
    if (!status) return host_fail(SQZ_ERR_INVALID_ARG, "status is NULL");
    *status = 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    SQZ_F8_TRY(cudaStreamIsCapturing(s, &cap), "cudaStreamIsCapturing");
    if (cap != cudaStreamCaptureStatusNone)
        return host_fail(SQZ_ERR_UNSUPPORTED, "the stream is being captured into a CUDA graph; reading the status "
                                              "synchronises, which a capture cannot contain");
    int device = 0;
    SQZ_F8_TRY(cudaGetDevice(&device), "cudaGetDevice");
    if (device >= kMaxDevices)
        return host_fail(SQZ_ERR_UNSUPPORTED, "device %d: at most %d are told apart", device, kMaxDevices);
    uint32_t* count = nullptr;
    const sqz_status st = timeout_count(&count);
    if (st != SQZ_OK) return st;
    uint32_t h = 0;
    SQZ_F8_TRY(cudaMemcpyAsync(&h, count, sizeof h, cudaMemcpyDeviceToHost, s), "reading the status");
    SQZ_F8_TRY(cudaStreamSynchronize(s), "reading the status");
    if (g_reported[device].take(h)) {
        *status = 1;
        return host_fail(SQZ_ERR_TIMEOUT, "a bounded device wait gave up (status 0x1): y of the affected call is "
                                          "undefined");
    }
    return SQZ_OK;
}

extern "C" SQZ_API sqz_status sqz_fp8_plan_query(int32_t m, int32_t n, int32_t k, int32_t sm_count,
                                                 sqz_fp8_plan_info* out) {
    if (!out) return host_fail(SQZ_ERR_INVALID_ARG, "out is NULL");
    *out = sqz_fp8_plan_info{};
    if (m < 1 || n < 1 || k < 1 || m > INT32_MAX - 256 || n > INT32_MAX - 256 || k > INT32_MAX - 256)
        return host_fail(SQZ_ERR_INVALID_ARG, "m=%d, n=%d or k=%d outside [1, 2^31 - 257]", m, n, k);
    if (sm_count < 2) return host_fail(SQZ_ERR_INVALID_ARG, "sm_count=%d: at least 2 expected", sm_count);
    const Plan p = plan_product(m, n, k, sm_count);
    out->many_rows = p.many;
    out->tile_rows = p.tile_a;
    out->tile_cols = p.tile_w;
    out->splits = p.splits;
    return SQZ_OK;
}
