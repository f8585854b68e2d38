// kernels_moe.cuh -- a whole mixture-of-experts layer for a few tokens in one
// cooperative kernel.
//
//   l = x R^T, p = softmax(l), the top_k experts of each token by l (ties: the
//   lowest index), h_e = silu(W1_e x) * (W3_e x), y = sum_e g_e W2_e h_e
//
// with W1, W3, W2 in 8 bits and one fp32 scale per 128 x 128 block.
//
// What bounds it: a few tokens read every weight of the experts they reach
// once, so the floor is those bytes at HBM speed; everything else is kept out
// of the stream's way.
//
// Activations at full precision on 8-bit tensor cores.  Weights go to the
// tensor cores as they are stored (no decoding in the SMs), so the
// activations have to be 8-bit too -- but not rounded to it: a value is the
// sum of four e4m3 digits, v = s (d0 + d1/16 + d2/256 + d3/4096), s the power
// of two that puts the largest value of a block of 128 in [128, 256).  Each
// digit is the rounded remainder of the ones before it, 16 times larger, so
// four digits carry 19 bits of a block's large values (fp16 has 11, bf16 8:
// both exact) and an absolute error of 2^-29 of the block's largest for small
// ones.  (Blocks whose largest is below 2^-110 are scaled as if it were that.)  A
// token is then four columns of the product, weights take the 128
// lanes (the MMA's M), and the digits' columns are joined in fp32 when the
// block's sum is scaled.
//
// Work.  A persistent CTA per SM; three phases with two grid-wide barriers:
//   0  router logits (in fp64: they are compared) and the digits of x, spread over
//      all warps of the grid;
//   1  every CTA routes for itself (the logits are a few KB), then gate and
//      up products: units (expert, 128 columns of the inner size, block of K)
//      in one sequence cut evenly over the CTAs, so that no SM is left with a
//      whole tile more than another.  Pieces of a tile meet in the workspace;
//      the CTA that brings the last one adds them in CTA order (bitwise
//      reproducible whoever is last), applies silu(gate) * up and writes the
//      digits of h;
//   2  down products: units (128 rows of y, expert, block of the inner size),
//      cut the same way; a token's experts are added in registers and shared
//      memory before anything leaves the SM, and the last piece of a row tile
//      writes y.
// The weights' ring runs through phases 1 and 2 without a stop: the first
// tiles of phase 2 are on their way while the CTA waits for the last h.
//
// Measured: 8 tokens, 128 experts, top 8, 4096/1408: 153 to 172 us for the 48 to
// 56 experts that random tokens reach (5.6 TB/s; 6.3 in phase 1); one token, 8
// experts, top 2, 4096/11008: 66 us (4.1 TB/s); 32 tokens, 32 experts, top 4,
// 2560/1008: 77 us; one token, 64 experts, top 6, 2048/1408: 34 us, of which the
// weights' time is 8.  The rest is latency, and most of that is instructions not
// in the cache the one time they run: routing 3.5 us after the first barrier, a
// tile's end 5 us (the counter's round trip 1.5, the join 1.5 to 3, h and its
// digits 0.5 to 3).  Code on those paths is kept short: unrolling the digits'
// loop and the join made 32 tokens 8 % slower.
//
// Warps: 0 weights (TMA), 1 TMEM and matrix instructions, 2 digits of x or h
// (TMA, four rows a token) and scales, 3 idle after phase 1's routing,
// 4-11 promotion (phase 1: 4-7 gate rows, 8-11 up rows; phase 2: both halves
// hold the rows, alternate groups of four tokens).
#pragma once

#include "fp8_common.cuh"

namespace sqz {
namespace moe {

using namespace f8;

constexpr int kMaxTokens = 32;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 16;
constexpr int kMaxPairs = kMaxTokens * kMaxTopK;
constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRing = 12;
constexpr int kScaleSlots = 8;
constexpr int kMaxBufs = 8;  // accumulators in tensor memory (a power of two; see kernels_fp8.cuh)
constexpr int kDigits = 4;
constexpr int kMaxGrid = 256;  // CTAs (one per SM)

// Start of the caller's workspace.  Zero before the first call; every call
// leaves the tile counters zero and the barrier counter a multiple of the
// grid.
struct Header {
    unsigned long long arrived;  // grid-wide barrier arrivals, ever
    int status;
    int pad;
};

struct Params {
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* router;
    int64_t ld_router;
    const float* s13;  // [experts][2][tiles_i][nkb_h]
    const float* s2;   // [experts][tiles_h][nkb_i]
    void* y;
    int64_t ldy;
    int32_t* ids;    // [tokens][top_k] or nullptr
    float* weights;  // [tokens][top_k] or nullptr
    // workspace
    Header* head;
    int* cnt1;       // [experts * tiles_i]
    int* cnt2;       // [tiles_h]
    float* logits;     // [tokens][experts]
    float* logits_lo;  // what rounding the logits to fp32 left out, the same way
    uint8_t* xq;     // [tokens][4][hpad]
    float* sx;       // [tokens][nkb_h]
    uint8_t* hq;     // [pairs][4][ipad]
    float* sh;       // [pairs][nkb_i]
    float* part1;    // [grid][2][tokens][256]
    float* part2;    // [grid][2][tokens][128]
    int tokens, experts, top_k, hidden, inter;
    int tiles_i, tiles_h;  // also the blocks of K of the down and the gate/up products
    int hpad, ipad;
    int renormalize, vec;
    int stages, stage_bytes;
};

__host__ __device__ inline int b_rows(int tokens) { return (kDigits * tokens + 15) / 16 * 16; }

// Shared memory of the logits' shares and, later, of the warps' logit keys.
__host__ __device__ inline int scratch_bytes(int tokens, int experts) {
    const int keys = (tokens < kWarps ? tokens : kWarps) * experts * 4, share = kWarps * 32 * 8;
    return ((keys > share ? keys : share) + 127) / 128 * 128;
}

template <bool BF16>
__device__ __forceinline__ float to_float(uint16_t h) {
    return BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}

// ---------------------------------------------------------- grid barrier
__device__ __forceinline__ unsigned long long ld_acquire(const unsigned long long* p) {
    unsigned long long v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
// Release and acquire at GPU scope (__threadfence is sequentially consistent,
// which nothing here needs, and slower).
__device__ __forceinline__ void fence_gpu() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// One thread of a CTA arrives, and later waits for the round its arrival
// belongs to.  The grid is launched cooperatively (every CTA is resident), and
// the wait is bounded all the same (about four seconds).
__device__ __forceinline__ unsigned long long grid_arrive(Header* h) {
    fence_gpu();
    const unsigned long long old = atomicAdd(&h->arrived, 1ull);
    return (old / gridDim.x + 1) * gridDim.x;
}
__device__ __forceinline__ bool grid_wait(const Header* h, unsigned long long target, volatile int* dead) {
    const long long t0 = clock64();
    while (ld_acquire(&h->arrived) < target) {
        if (*dead || clock64() - t0 > 8000000000ll) {
            *dead = 1;
            return false;
        }
    }
    fence_gpu();
    return true;
}

// ------------------------------------------------------------ digits of v
// Power of two that brings values up to `max_bits` (fp32 bits) into [128,
// 256): the factor, and its inverse, which scales the sums back.  Exponents
// below 2^-110 are treated as 2^-110 (both stay normal numbers).
__device__ __forceinline__ float digit_scale(uint32_t max_bits, float* factor) {
    int e = (int)(max_bits >> 23) - 127;
    if (max_bits == 0 || max_bits >= 0x7F800000u) e = 7;  // zeros, or the digits are NaN
    if (e < -110) e = -110;
    *factor = __uint_as_float((uint32_t)(7 - e + 127) << 23);
    return __uint_as_float((uint32_t)(e - 7 + 127) << 23);
}
// The four digits of v (already scaled), lowest byte first; NaN for a value
// that is not finite.
__device__ __forceinline__ uint32_t digits_of(float v) {
    uint32_t out = 0;
    if (!(fabsf(v) < __int_as_float(0x7F800000))) return 0x7F7F7F7Fu;
#pragma unroll
    for (int p = 0; p < kDigits; ++p) {
        uint16_t code;
        uint32_t back;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(code) : "f"(0.f), "f"(v));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(code));
        out |= (uint32_t)(code & 0xFF) << (8 * p);
        v = (v - __half2float(__ushort_as_half((uint16_t)(back & 0xFFFF)))) * 16.f;
    }
    return out;
}

// ------------------------------------------------------------ phase 0
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = BF16 ? __uint_as_float(w[j] << 16) : h2f((uint16_t)w[j]);
        v[2 * j + 1] = BF16 ? __uint_as_float(w[j] & 0xFFFF0000u) : h2f((uint16_t)(w[j] >> 16));
    }
}
// Eight values from column c of a row of the router (zeros past `hidden`; a vector
// load when rows are 16-byte aligned), or of x: plain loads, since y, which this
// kernel writes later, may be x.
template <bool BF16, bool X>
__device__ __forceinline__ void load8(const uint16_t* row, int c, const Params& p, float (&v)[8]) {
    if (p.vec) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (c < p.hidden) u = X ? ld_u128(row + c) : ldg_u128(row + c);
        unpack8<BF16>(u, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = c + j < p.hidden ? to_float<BF16>(X ? ld_u16(row + c + j) : __ldg(row + c + j)) : 0.f;
    }
}

// The logits of expert e for tokens [t_begin, t_end): the warp's share of the
// columns (runs of 256, 8 a lane), then the lanes' sums; lane t returns token
// t's.
// Products and sums are in fp64: the choice of experts is a comparison, and in
// fp32 two logits closer than their sums' error would change places.
// The expert's row is held in registers (two runs at a time), so a token costs
// its own loads only; four tokens' sums cross the lanes together.
template <bool BF16>
__device__ __forceinline__ double logits_share(const Params& p, int e, int t_begin, int t_end, int warp,
                                               int lane) {
    const uint16_t* r = p.router + (int64_t)e * p.ld_router;
    double mine = 0.;
    for (int c0 = warp * 256; c0 < p.hidden; c0 += 2 * kWarps * 256) {
        const int c[2] = {c0 + lane * 8, c0 + kWarps * 256 + lane * 8};
        const int runs = c0 + kWarps * 256 < p.hidden ? 2 : 1;
        double rd[2][8];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float rf[8];
            load8<BF16, false>(r, c[k], p, rf);
#pragma unroll
            for (int j = 0; j < 8; ++j) rd[k][j] = rf[j];
        }
#pragma unroll 1
        for (int t0 = t_begin; t0 < t_end; t0 += 4) {
            double s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[i] = 0.;
                if (t0 + i >= t_end) continue;
                const uint16_t* x = p.x + (int64_t)(t0 + i) * p.ldx;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (k >= runs) break;
                    float xf[8];
                    load8<BF16, true>(x, c[k], p, xf);
#pragma unroll
                    for (int j = 0; j < 8; ++j) s[i] = fma(rd[k][j], (double)xf[j], s[i]);
                }
            }
            // lanes 8 i .. 8 i + 7 end with token t0 + i
            const bool up2 = lane & 16, up1 = lane & 8;
            double k0 = up2 ? s[2] : s[0], k1 = up2 ? s[3] : s[1];
            k0 += __shfl_xor_sync(0xffffffffu, up2 ? s[0] : s[2], 16);
            k1 += __shfl_xor_sync(0xffffffffu, up2 ? s[1] : s[3], 16);
            double v = up1 ? k1 : k0;
            v += __shfl_xor_sync(0xffffffffu, up1 ? k0 : k1, 8);
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            v = __shfl_sync(0xffffffffu, v, (lane - t0) * 8 & 31);
            if (lane >= t0 && lane < t0 + 4) mine += v;
        }
    }
    return mine;
}

// Digits of block kb of token t: lane holds four consecutive values.
template <bool BF16>
__device__ __forceinline__ void x_digits_unit(const Params& p, int t, int kb, int lane) {
    float v[4];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int c = kb * kBlockK + lane * 4 + j;
        v[j] = c < p.hidden ? to_float<BF16>(ld_u16(p.x + (int64_t)t * p.ldx + c)) : 0.f;
        m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    float f;
    const float s = digit_scale(m, &f);
    uint32_t d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = digits_of(v[j] * f);
#pragma unroll
    for (int q = 0; q < kDigits; ++q) {
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) w |= ((d[j] >> (8 * q)) & 0xFF) << (8 * j);
        *reinterpret_cast<uint32_t*>(p.xq + ((int64_t)t * kDigits + q) * p.hpad + kb * kBlockK + lane * 4) = w;
    }
    if (lane == 0) p.sx[t * p.tiles_h + kb] = s;
}

// ------------------------------------------------------------ routing
struct Routing {
    uint32_t mask[kMaxExperts];     // tokens of each expert, one bit each
    uint16_t base[kMaxExperts];     // first row of the expert's tokens
    uint16_t active[kMaxPairs];     // experts with tokens, ascending
    uint16_t id[kMaxPairs];         // [token][slot]
    float weight[kMaxPairs];        // [token][slot]
    uint8_t row_token[kMaxPairs];   // [row]: rows sorted by expert, then token
    float row_weight[kMaxPairs];
    int n_active, n_most;  // experts with tokens; the most tokens one has
};

// Logits as unsigned integers of the same order, +0 and -0 alike, NaN (1)
// below every number; 0 is left for what is taken.
__device__ __forceinline__ uint32_t logit_key(float l) {
    const uint32_t u = __float_as_uint(l + 0.f);
    return l != l ? 1u : (u & 0x80000000u ? ~u : u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return k == 1u ? __int_as_float(0x7FFFFFFF) : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Of the experts whose fp32 logits are the same, `key`: the one that has most
// beyond it, the lowest index where that is equal too (the whole warp).
__device__ __noinline__ uint32_t best_of_equals(const float* lo, const uint32_t* keys, uint32_t key, int experts,
                                                int lane) {
    uint32_t k = 0, at = 0xffffffffu;
#pragma unroll 4
    for (int e = lane; e < experts; e += 32) {
        const uint32_t v = keys[e] == key ? logit_key(__ldcg(lo + e)) : 0;
        if (v > k) k = v, at = e;
    }
    return __reduce_min_sync(0xffffffffu, k == __reduce_max_sync(0xffffffffu, k) ? at : 0xffffffffu);
}

// The choice of one token by one warp: top_k rounds of the warp's best
// (highest logit, lowest index).  `keys`: the warp's copy, [experts].
__device__ __forceinline__ void route_token(const Params& p, Routing* R, uint32_t* keys, int t, int lane) {
    const float* l = p.logits + t * p.experts;
    uint32_t best = 0;
#pragma unroll 4
    for (int e = lane; e < p.experts; e += 32) {
        const uint32_t k = logit_key(__ldcg(l + e));
        keys[e] = k;
        best = max(best, k);
    }
    const float top = key_logit(__reduce_max_sync(0xffffffffu, best));
    float sum = 0.f;  // NaN if any logit is (key_logit)
#pragma unroll 2
    for (int e = lane; e < p.experts; e += 32) sum += expf(key_logit(keys[e]) - top);
    sum = warp_sum(sum);
    uint32_t mine = 0;  // lane j: the j-th choice's key
    int mine_id = 0;
#pragma unroll 1
    for (int j = 0; j < p.top_k; ++j) {
        uint32_t k = 0, at = 0xffffffffu;
        bool again = false;  // the lane has its best key more than once
#pragma unroll 4
        for (int e = lane; e < p.experts; e += 32) {
            const uint32_t v = keys[e];
            again = v == k || (again && v < k);
            if (v > k) k = v, at = e;
        }
        const uint32_t high = __reduce_max_sync(0xffffffffu, k);
        uint32_t e = __reduce_min_sync(0xffffffffu, k == high ? at : 0xffffffffu);
        if (__any_sync(0xffffffffu, k == high && (again || at != e)) && high > 1u)
            e = best_of_equals(p.logits_lo + t * p.experts, keys, high, p.experts, lane);
        if ((int)(e & 31) == lane) keys[e] = 0;  // (the lane that reads it)
        if (lane == j) mine = high, mine_id = (int)e;
    }
    float w = lane < p.top_k ? expf(key_logit(mine) - top) / sum : 0.f;
    if (p.renormalize) w = w / warp_sum(w);
    if (lane < p.top_k) {
        R->id[t * p.top_k + lane] = (uint16_t)mine_id;
        R->weight[t * p.top_k + lane] = w;
        atomicOr(&R->mask[mine_id], 1u << t);
        if (blockIdx.x == 0) {
            if (p.ids) p.ids[t * p.top_k + lane] = mine_id;
            if (p.weights) p.weights[t * p.top_k + lane] = w;
        }
    }
}

// Active experts in ascending order, the first row of each (one
// warp).
__device__ __forceinline__ void list_experts(const Params& p, Routing* R, int lane) {
    int n = 0, rows = 0, most = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 32) {
        const int e = e0 + lane;
        const int c = e < p.experts ? __popc(R->mask[e]) : 0;
        const uint32_t on = __ballot_sync(0xffffffffu, c > 0);
        if (on == 0) continue;
        most = max(most, c);
        int pre = c;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, pre, off);
            if (lane >= off) pre += o;
        }
        if (c > 0) {
            R->active[n + __popc(on & ((1u << lane) - 1))] = (uint16_t)e;
            R->base[e] = (uint16_t)(rows + pre - c);
        }
        n += __popc(on);
        rows += __shfl_sync(0xffffffffu, pre, 31);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) R->n_active = n, R->n_most = most;
}

// -------------------------------------------------------- unit sequences
// `total` units cut evenly: CTA c has [cuts[c], cuts[c + 1]), cuts[c] =
// floor(total c / grid) (in 32 bits: the remainder times c stays below grid^2).
__device__ __forceinline__ void make_cuts(int* cuts, int total) {
    const int g = gridDim.x, q = total / g, r = total - q * g;
    for (int c = threadIdx.x; c <= g; c += kThreads) cuts[c] = q * c + r * c / g;
}
// The last CTA that starts at or before unit u: the one that has it.
__device__ __forceinline__ int owner(const int* cuts, int u) {
    int lo = 0, hi = gridDim.x;  // cuts[lo] <= u < cuts[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cuts[mid] <= u) lo = mid; else hi = mid;
    }
    return lo;
}

// Sums of a tile's pieces in CTA order: four consecutive floats at `at` and
// four more 1024 floats further on (256 threads cover a run of 1024).  Pieces
// lie [CTA][at the tile's start: 1, later: 0][size floats], `size` of them in
// use; this CTA's own is passed in.  The loads of up to eight pieces are in
// flight together.
struct Joined {
    float4 v[2];
};
__device__ __forceinline__ Joined join4(const Joined& own, const float* pieces, int64_t size, int at, const int* cuts,
                                        int c0, int c1, int first, int used) {
    Joined s;
    s.v[0] = s.v[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool two = at + 1024 < used;
    for (int cb = c0; cb <= c1; cb += 8) {
        float4 w[2][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = min(cb + j, c1), from = cuts[c];
            const bool on = cb + j <= c1 && from < cuts[c + 1];
            const float4* src =
                reinterpret_cast<const float4*>(pieces + (c * 2 + (from > first ? 0 : 1)) * size + at);
            w[0][j] = w[1][j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (on && c == blockIdx.x) {
                w[0][j] = own.v[0], w[1][j] = own.v[1];
            } else if (on) {
                w[0][j] = __ldcg(src);
                if (two) w[1][j] = __ldcg(src + 256);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s.v[k].x += w[k][j].x, s.v[k].y += w[k][j].y, s.v[k].z += w[k][j].z, s.v[k].w += w[k][j].w;
    }
    return s;
}

// Four consecutive columns of y (hidden is a multiple of 16: all or none).
template <bool BF16>
__device__ __forceinline__ void store_y(const Params& p, int token, int col, const float4& v) {
    if (col >= p.hidden) return;
    const int64_t at = token * p.ldy + col;
    const int type = BF16 ? kBF16 : kF16;
    store_out(p.y, at, type, v.x);
    store_out(p.y, at + 1, type, v.y);
    store_out(p.y, at + 2, type, v.z);
    store_out(p.y, at + 3, type, v.w);
}

struct Shared {
    Routing route;
    uint64_t full[kMaxRing], empty[kMaxRing], sfull[kScaleSlots], sempty[kScaleSlots], tfull[kMaxBufs], tempty[kMaxBufs];
    float scale[kScaleSlots][kMaxTokens + 2];  // token (or row) scales, the two weight scales
    uint32_t taddr;
    uint64_t h_arrived;              // the CTA's last h is written and its arrival posted
    unsigned long long h_target;     // the barrier round of that arrival
    int dead, last, owners[2];
    int cuts[2][kMaxGrid + 1];       // units of the two products by CTA
    __align__(16) uint32_t max_bits[kMaxTokens][4];
};

__device__ __forceinline__ void bar_promotion() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// The four digits' columns of four tokens joined (16 columns of tensor memory).
__device__ __forceinline__ float joined(const uint32_t (&d)[16], int i) {
    float v = __uint_as_float(d[4 * i + 3]);
    v = fmaf(v, 0.0625f, __uint_as_float(d[4 * i + 2]));
    v = fmaf(v, 0.0625f, __uint_as_float(d[4 * i + 1]));
    return fmaf(v, 0.0625f, __uint_as_float(d[4 * i]));
}
// acc[j][i] += scale * sw * sum for n tokens, groups of four from `first` on,
// `step` apart: group first + step j in acc[j].  Whether the scales' products
// (lane: token) stay in range is asked while tensor memory answers; if one does
// not, lane t splits those of token t.
template <int GROUPS>
__device__ __forceinline__ void promote(float (&acc)[GROUPS][4], uint32_t taddr, const float* sc, float sw, int n,
                                        int first, int step, int lane) {
    if (4 * first >= n) return;
    uint32_t d[16];
    tmem_ld16(taddr + first * 16, d);
    const bool plain = __all_sync(0xffffffffu, lane >= n || in_range(sc[lane] * sw));
    tmem_wait_ld(d);
    if (plain) {
#pragma unroll
        for (int j = 0; j < GROUPS; ++j) {
            const int b = first + j * step;
            if (4 * b >= n) break;
            if (j > 0) {
                tmem_ld16(taddr + b * 16, d);
                tmem_wait_ld(d);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(joined(d, i), sc[4 * b + i] * sw, acc[j][i]);
        }
    } else {
        const ScalePair own = split_scales(sc[lane], sw);
#pragma unroll
        for (int j = 0; j < GROUPS; ++j) {
            const int b = first + j * step;
            if (4 * b < n) {
                tmem_ld16(taddr + b * 16, d);
                tmem_wait_ld(d);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[j][i] = fmaf(joined(d, i) * __shfl_sync(0xffffffffu, own.first, 4 * b + i),
                                     __shfl_sync(0xffffffffu, own.s, 4 * b + i), acc[j][i]);
            }
        }
    }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1) moe_kernel(const __grid_constant__ CUtensorMap map_w13,
                                                          const __grid_constant__ CUtensorMap map_w2,
                                                          const __grid_constant__ CUtensorMap map_x,
                                                          const __grid_constant__ CUtensorMap map_h, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    float* sums = reinterpret_cast<float*>(ring + p.stages * p.stage_bytes);  // [2][tokens][128]
    uint8_t* scratch = reinterpret_cast<uint8_t*>(sums + 2 * p.tokens * 128);  // phase 0 and routing
    Shared* S = reinterpret_cast<Shared*>(scratch + scratch_bytes(p.tokens, p.experts));
    Routing* R = &S->route;
    volatile int* dead = &S->dead;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int nkb1 = p.tiles_h, nkb2 = p.tiles_i;  // blocks of K of the two products

    // an expert's tokens in as many groups (of whole fours) as there are CTAs for
    int groups = max(1, min((p.tokens + 3) / 4, (int)gridDim.x / p.experts));
    const int per_group = ((p.tokens + 3) / 4 + groups - 1) / groups * 4;
    groups = (p.tokens + per_group - 1) / per_group;
    if (blockIdx.x < p.experts * groups)  // the router's row on its way while x is split
        for (int c = threadIdx.x * 64; c < p.hidden; c += kThreads * 64)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.router + blockIdx.x / groups * p.ld_router + c));
    if (warp == 1) tmem_alloc(&S->taddr, 512);
    if (warp == 2 && lane == 0) {
        tma_prefetch_map(&map_w13);
        tma_prefetch_map(&map_x);
        tma_prefetch_map(&map_w2);
        tma_prefetch_map(&map_h);
    }
    if (threadIdx.x == 0) {
        S->dead = 0;
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&S->full[i], 1 + 1);
            mbar_init(&S->empty[i], 1);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&S->sfull[i], 32);
            mbar_init(&S->sempty[i], 8);
        }
        for (int i = 0; i < kMaxBufs; ++i) {
            mbar_init(&S->tfull[i], 1);
            mbar_init(&S->tempty[i], 8);
        }
        mbar_init(&S->h_arrived, 1);
        fence_mbar_init();
    }
    for (int e = threadIdx.x; e < p.experts; e += kThreads) R->mask[e] = 0;
    // ---- phase 0: logits and the digits of x
    double* share = reinterpret_cast<double*>(scratch);  // [kWarps][32]
    for (int u = gridDim.x - 1 - blockIdx.x + gridDim.x * warp; u < p.tokens * nkb1; u += gridDim.x * kWarps)
        x_digits_unit<BF16>(p, u / nkb1, u % nkb1, lane);
    for (int u = blockIdx.x; u < p.experts * groups; u += gridDim.x) {
        const int e = u / groups, t0 = (u - e * groups) * per_group, t1 = min(t0 + per_group, p.tokens);
        share[warp * 32 + lane] = logits_share<BF16>(p, e, t0, t1, warp, lane);
        __syncthreads();
        const int t = t0 + threadIdx.x;
        if (t < t1) {
            double v = 0.;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += share[w * 32 + t];
            const float l = (float)v;
            p.logits[t * p.experts + e] = l;
            p.logits_lo[t * p.experts + e] = fabsf(l) < __int_as_float(0x7F800000) ? (float)(v - l) : 0.f;
        }
        __syncthreads();
    }
    fence_proxy_all();  // the digits are read by TMA
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t taddr = S->taddr;
    if (threadIdx.x == 0) grid_wait(p.head, grid_arrive(p.head), dead);
    __syncthreads();

    // ---- routing, by every CTA for itself
    if (!*dead) {
        uint32_t* keys = reinterpret_cast<uint32_t*>(scratch) + warp * p.experts;
        for (int t = warp; t < p.tokens; t += kWarps) {
            route_token(p, R, keys, t, lane);
            __syncwarp();
        }
    }
    __syncthreads();
    if (warp == 0) list_experts(p, R, lane);
    __syncthreads();

    const int n_act = *dead ? 0 : R->n_active;
    // columns of an accumulator: what the expert with the most tokens needs
    const uint32_t cols = b_rows(*dead ? 1 : R->n_most);
    uint32_t bufs = kMaxBufs, bufs_log = 3;
    while (bufs * 2 * cols > 512) bufs /= 2, --bufs_log;
    const int total1 = n_act * p.tiles_i * nkb1, total2 = p.tiles_h * n_act * nkb2;
    for (int i = threadIdx.x; i < (*dead ? 0 : p.tokens * p.top_k); i += kThreads) {
        const int t = i / p.top_k, e = R->id[i];
        const int row = R->base[e] + __popc(R->mask[e] & ((1u << t) - 1));
        R->row_token[row] = (uint8_t)t;
        R->row_weight[row] = R->weight[i];
    }
    make_cuts(S->cuts[0], total1);
    make_cuts(S->cuts[1], total2);
    __syncthreads();
    const int u1a = S->cuts[0][blockIdx.x], u1b = S->cuts[0][blockIdx.x + 1];
    const int u2a = S->cuts[1][blockIdx.x], u2b = S->cuts[1][blockIdx.x + 1];

    if (warp == 0) {  // ---------------------------------------------- weights
        int st = 0, ph = 0;
        bool alive = true;
        if (u1a < u1b) {
            int kb = u1a % nkb1, ti = u1a / nkb1 % p.tiles_i, a = u1a / nkb1 / p.tiles_i, e = R->active[a];
            for (int u = u1a; u < u1b && alive; ++u) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!(alive = wait_warp(&S->empty[st], ph ^ 1, dead))) break;
                    if (elect_one()) {
                        mbar_expect_tx(&S->full[st], kTileBytes);
                        tma_load_3d(ring + st * p.stage_bytes, &map_w13, &S->full[st], kb * kBlockK, ti * 128, 2 * e + half);
                    }
                    __syncwarp();
                    if (++st == p.stages) st = 0, ph ^= 1;
                }
                if (++kb == nkb1) {
                    kb = 0;
                    if (++ti == p.tiles_i && ++a < n_act) e = R->active[a];
                    if (ti == p.tiles_i) ti = 0;
                }
            }
        }
        if (u2a < u2b) {
            int kb = u2a % nkb2, a = u2a / nkb2 % n_act, rt = u2a / nkb2 / n_act, e = R->active[a];
            for (int u = u2a; u < u2b && alive; ++u) {
                if (!(alive = wait_warp(&S->empty[st], ph ^ 1, dead))) break;
                if (elect_one()) {
                    mbar_expect_tx(&S->full[st], kTileBytes);
                    tma_load_3d(ring + st * p.stage_bytes, &map_w2, &S->full[st], kb * kBlockK, rt * 128, e);
                }
                __syncwarp();
                if (++st == p.stages) st = 0, ph ^= 1;
                if (++kb == nkb2) {
                    kb = 0;
                    if (++a == n_act) a = 0, ++rt;
                    e = R->active[a];
                }
            }
        }
        if (!alive) let_copies_land();
    } else if (warp == 1) {  // ---------------------------- matrix instructions
        const uint32_t idesc = instr_desc(0, 0, 128, cols);
        int st = 0, ph = 0;
        uint32_t it = 0;
        bool alive = true;
        Ahead next;
        next.ask(&S->full[0], 0, &S->tempty[0], 1);
        for (int u = u1a; u < u1b; ++u) {
            const int buf = it & (bufs - 1), gate = st;
            alive = next.wait(&S->full[st], ph, &S->tempty[buf], ((it >> bufs_log) & 1) ^ 1, dead);
            if (!alive) break;
            if (++st == p.stages) st = 0, ph ^= 1;
            const int up = st;
            const bool up_there = mbar_test(&S->full[st], ph);
            tc_fence_after();
            const uint32_t at = smem_u32(ring + gate * p.stage_bytes), digits = at + kTileBytes;
            if (elect_one()) mma_block(taddr + buf * 2 * cols, at, digits, idesc);
            __syncwarp();
            if (!__all_sync(0xffffffffu, up_there)) alive = wait_warp(&S->full[st], ph, dead);
            if (!alive) break;
            tc_fence_after();
            if (++st == p.stages) st = 0, ph ^= 1;
            ++it;
            next.ask(&S->full[st], ph, &S->tempty[it & (bufs - 1)], ((it >> bufs_log) & 1) ^ 1);
            if (elect_one()) {  // the up tile shares the gate tile's digits
                mma_block(taddr + (buf * 2 + 1) * cols, smem_u32(ring + up * p.stage_bytes), digits, idesc);
                mma_commit(&S->tfull[buf]);
                mma_commit(&S->empty[gate]);
                mma_commit(&S->empty[up]);
            }
            __syncwarp();
        }
        for (int u = u2a; u < u2b && alive; ++u) {
            const int buf = it & (bufs - 1), used = st;
            alive = next.wait(&S->full[st], ph, &S->tempty[buf], ((it >> bufs_log) & 1) ^ 1, dead);
            if (!alive) break;
            tc_fence_after();
            if (++st == p.stages) st = 0, ph ^= 1;
            ++it;
            next.ask(&S->full[st], ph, &S->tempty[it & (bufs - 1)], ((it >> bufs_log) & 1) ^ 1);
            const uint32_t at = smem_u32(ring + used * p.stage_bytes);
            if (elect_one()) {
                mma_block(taddr + buf * 2 * cols, at, at + kTileBytes, idesc);
                mma_commit(&S->tfull[buf]);
                mma_commit(&S->empty[used]);
            }
            __syncwarp();
        }
        if (!alive) let_copies_land();
    } else if (warp == 2) {  // ------------------------ digits and their scales
        int st = 0, ph = 0;
        uint32_t it = 0;
        bool alive = true;
        fence_proxy_all();  // the digits of x were written by threads before the grid's barrier
        for (int u = u1a; u < u1b && alive;) {
            const int tile = u / nkb1, k0 = u - tile * nkb1, k1 = min(nkb1, k0 + u1b - u);
            const int a = tile / p.tiles_i, ti = tile - a * p.tiles_i, e = R->active[a], n = __popc(R->mask[e]);
            const int t = lane < n ? R->row_token[R->base[e] + lane] : 0;
            const float* sx = p.sx + t * nkb1;
            const float* sw = p.s13 + (((int64_t)e * 2 + (lane & 1)) * p.tiles_i + ti) * nkb1;
            for (int kb = k0; kb < k1; ++kb, ++it) {
                const int slot = it % kScaleSlots;
                alive = __all_sync(0xffffffffu, wait_alive(&S->sempty[slot], ((it / kScaleSlots) & 1) ^ 1, dead) &&
                                                    wait_alive(&S->empty[st], ph ^ 1, dead));
                if (!alive) break;
                if (lane == 0) mbar_expect_tx(&S->full[st], (uint32_t)n * kDigits * kBlockK);
                __syncwarp();
                if (lane < n)
                    tma_load_2d(ring + st * p.stage_bytes + kTileBytes + lane * kDigits * kBlockK, &map_x, &S->full[st],
                                kb * kBlockK, t * kDigits);
                if (lane < n) cp_async4(&S->scale[slot][lane], sx + kb);
                if (lane < 2) cp_async4(&S->scale[slot][kMaxTokens + lane], sw + kb);
                cp_async_arrive(&S->sfull[slot]);
                if (++st == p.stages) st = 0, ph ^= 1;
                // the up tile's stage brings no digits of its own
                alive = __all_sync(0xffffffffu, wait_alive(&S->empty[st], ph ^ 1, dead));
                if (!alive) break;
                if (lane == 0) mbar_arrive(&S->full[st]);
                if (++st == p.stages) st = 0, ph ^= 1;
            }
            u += k1 - k0;
        }
        // every h of the grid has to be there
        if (u2a < u2b && alive) {
            bool ok = true;
            if (lane == 0) ok = wait_alive(&S->h_arrived, 0, dead) && grid_wait(p.head, S->h_target, dead);
            __syncwarp();  // what lane 0 has acquired, for the lanes that read it (a vote orders no memory)
            alive = __all_sync(0xffffffffu, ok);
            fence_proxy_all();
        }
        for (int u = u2a; u < u2b && alive;) {
            const int run = u / nkb2, k0 = u - run * nkb2, k1 = min(nkb2, k0 + u2b - u), rt = run / n_act;
            const int e = R->active[run - rt * n_act], n = __popc(R->mask[e]), row = R->base[e] + (lane < n ? lane : 0);
            const float* sh = p.sh + (int64_t)row * nkb2;
            const float* sw = p.s2 + ((int64_t)e * p.tiles_h + rt) * nkb2;
            for (int kb = k0; kb < k1; ++kb, ++it) {
                const int slot = it % kScaleSlots;
                alive = __all_sync(0xffffffffu, wait_alive(&S->sempty[slot], ((it / kScaleSlots) & 1) ^ 1, dead) &&
                                                    wait_alive(&S->empty[st], ph ^ 1, dead));
                if (!alive) break;
                if (lane == 0) mbar_expect_tx(&S->full[st], (uint32_t)n * kDigits * kBlockK);
                __syncwarp();
                if (lane < n)
                    tma_load_2d(ring + st * p.stage_bytes + kTileBytes + lane * kDigits * kBlockK, &map_h, &S->full[st],
                                kb * kBlockK, row * kDigits);
                if (lane < n) cp_async4(&S->scale[slot][lane], sh + kb);
                if (lane == 0) cp_async4(&S->scale[slot][kMaxTokens], sw + kb);
                cp_async_arrive(&S->sfull[slot]);
                if (++st == p.stages) st = 0, ph ^= 1;
            }
            u += k1 - k0;
        }
    } else if (warp >= 4) {  // ------------------------------------- promotion
        const int group = (warp - 4) / 4, r = (warp & 3) * 32 + lane;
        const int pt = threadIdx.x - 128;  // 0 .. 255
        const bool first_thread = pt == 0;
        const uint32_t lanes = taddr + ((uint32_t)(warp & 3) << 21);
        uint32_t it = 0;
        // Once a wait has given up, the warps stop waiting but keep step (they
        // meet at barriers); the results are then undefined.
        bool alive = true;
        // Waits for unit `it`: its scales and its sums.  Returns the scales.
        const auto unit_ready = [&]() -> const float* {
            const int slot = it % kScaleSlots;
            if (alive)
                alive = __all_sync(0xffffffffu, wait_alive(&S->sfull[slot], (it / kScaleSlots) & 1, dead) &&
                                                    wait_alive(&S->tfull[it & (bufs - 1)], (it >> bufs_log) & 1, dead));
            tc_fence_after();
            return S->scale[slot];
        };
        const auto unit_done = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&S->tempty[it & (bufs - 1)]);
                mbar_arrive(&S->sempty[it % kScaleSlots]);
            }
            ++it;
        };
        // The CTAs that have the units [first, first + whole), for the join: looked
        // up while the counter's answer is on its way.
        const auto find_owners = [&](const int* cuts, int first, int whole) {
            S->owners[0] = owner(cuts, first);
            S->owners[1] = owner(cuts, first + whole - 1);
        };
        // Whether the other CTAs' pieces of a tile are all there: then this CTA
        // completes it, and its own piece need not leave the SM.  (Asked for the
        // tile a CTA ends inside of, when it had others before: the next CTAs start
        // with that tile's rest.)
        const auto others_done = [&](int* counter, int len, const int* cuts, int first, int whole) {
            bar_promotion();
            if (first_thread) {
                int done;
                asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(done) : "l"(counter) : "memory");
                find_owners(cuts, first, whole);
                S->last = done + len == whole;
                if (S->last) *counter = 0;  // for the next call
            }
            bar_promotion();
            return S->last != 0;
        };
        // Adds `len` of a tile's `whole` units to its counter once the pieces
        // of all 256 threads are written; true for the CTA that completes it.
        const auto is_last = [&](int* counter, int len, const int* cuts, int first, int whole) {
            bar_promotion();
            if (first_thread) {  // its release covers what the barrier has ordered before it
                int old;
                asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;"
                             : "=r"(old)
                             : "l"(counter), "r"(len)
                             : "memory");
                find_owners(cuts, first, whole);
                S->last = old + len == whole;
                if (S->last) *counter = 0;  // for the next call
            }
            bar_promotion();
            return S->last != 0;
        };

        for (int u = u1a; u < u1b;) {
            const int tile = u / nkb1, k0 = u - tile * nkb1, len = min(nkb1 - k0, u1b - u);
            const int a = tile / p.tiles_i, ti = tile - a * p.tiles_i, e = R->active[a];
            const int n = __popc(R->mask[e]), row0 = R->base[e];
            float acc[8][4];
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i / 4][i % 4] = 0.f;
            for (int i = 0; i < len; ++i) {
                const float* sc = unit_ready();
                promote(acc, lanes + ((it & (bufs - 1)) * 2 + group) * cols, sc, sc[kMaxTokens + group], n, 0, 1, lane);
                unit_done();
            }
            // From here on in shared memory, token by token: [token][gate, up rows]
            float* own = sums + group * 128 + r;
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                if (4 * b >= n) break;  // (few tokens fetch few instructions)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (4 * b + i < n) own[(4 * b + i) * 256] = acc[b][i];
            }
            bool mine = len == nkb1;
            if (!mine) {  // a piece: at the tile's start (then the CTA's last tile) or not (then its first)
                const int slot = k0 > 0 ? 0 : 1;
                const int first = tile * nkb1;
                mine = slot == 1 && u1b - u1a > len && others_done(p.cnt1 + tile, len, S->cuts[0], first, nkb1);
                if (!mine) {
                    float* dst = p.part1 + (int64_t)(blockIdx.x * 2 + slot) * p.tokens * 256 + group * 128 + r;
#pragma unroll 2
                    for (int i = 0; i < n; ++i) __stcg(dst + i * 256, own[i * 256]);
                    mine = is_last(p.cnt1 + tile, len, S->cuts[0], first, nkb1);
                }
                if (mine) {
                    const int used = n * 256, c0 = S->owners[0], c1 = S->owners[1];
                    for (int i = pt * 4; i < used; i += 2048) {
                        Joined s;
                        s.v[0] = *reinterpret_cast<const float4*>(sums + i);
                        if (i + 1024 < used) s.v[1] = *reinterpret_cast<const float4*>(sums + i + 1024);
                        s = join4(s, p.part1, (int64_t)p.tokens * 256, i, S->cuts[0], c0, c1, first, used);
                        *reinterpret_cast<float4*>(sums + i) = s.v[0];
                        if (i + 1024 < used) *reinterpret_cast<float4*>(sums + i + 1024) = s.v[1];
                    }
                }
            }
            if (mine) {  // h = silu(gate) * up, and its digits; group g takes the tokens of its parity
                bar_promotion();
#pragma unroll 1
                for (int i = group; i < n; i += 2) {
                    const float g = sums[i * 256 + r], h = g / (1.f + expf(-g)) * sums[i * 256 + 128 + r];
                    sums[i * 256 + r] = h;
                    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(h) & 0x7FFFFFFFu);
                    if (lane == 0) S->max_bits[i][warp & 3] = m;
                }
                bar_promotion();
#pragma unroll 1
                for (int i = group; i < n; i += 2) {
                    const uint4 m = *reinterpret_cast<const uint4*>(S->max_bits[i]);
                    float f;
                    const float s = digit_scale(max(max(m.x, m.y), max(m.z, m.w)), &f);
                    const uint32_t d = digits_of(sums[i * 256 + r] * f);
                    uint8_t* dst = p.hq + (int64_t)(row0 + i) * kDigits * p.ipad + ti * 128 + r;
#pragma unroll
                    for (int q = 0; q < kDigits; ++q) dst[(int64_t)q * p.ipad] = (uint8_t)(d >> (8 * q));
                    if (r == 0) p.sh[(int64_t)(row0 + i) * nkb2 + ti] = s;
                }
            }
            bar_promotion();  // `sums` is read
            u += len;
        }
        fence_proxy_all();  // the digits are read by TMA
        bar_promotion();
        if (first_thread) {
            S->h_target = grid_arrive(p.head);
            mbar_arrive(&S->h_arrived);
        }

        for (int u = u2a; u < u2b;) {
            const int per = n_act * nkb2, rt = u / per, k0 = u - rt * per, len = min(per - k0, u2b - u);
            float* own = sums + group * p.tokens * 128 + r;  // [token][128], this thread's row
            for (int t = 0; t < p.tokens; ++t) own[t * 128] = 0.f;
            for (int v = k0; v < k0 + len;) {
                const int a = v / nkb2, kb = v - a * nkb2, run = min(nkb2 - kb, k0 + len - v);
                const int e = R->active[a], n = __popc(R->mask[e]), row0 = R->base[e];
                float acc[4][4];
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i / 4][i % 4] = 0.f;
                for (int i = 0; i < run; ++i) {
                    const float* sc = unit_ready();
                    promote(acc, lanes + (it & (bufs - 1)) * 2 * cols, sc, sc[kMaxTokens], n, group, 2, lane);
                    unit_done();
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int row = (2 * (i / 4) + group) * 4 + i % 4;
                    if (row < n)
                        own[R->row_token[row0 + row] * 128] =
                            fmaf(R->row_weight[row0 + row], acc[i / 4][i % 4], own[R->row_token[row0 + row] * 128]);
                }
                v += run;
            }
            bar_promotion();
            // the two groups' sums meet; a thread takes four rows of a token
            const int used = p.tokens * 128, slot = k0 > 0 ? 0 : 1;
            const auto met = [&](int i) {
                float4 v = *reinterpret_cast<const float4*>(sums + i);
                const float4 w = *reinterpret_cast<const float4*>(sums + used + i);
                v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
                return v;
            };
            if (len == per) {
                for (int i = pt * 4; i < used; i += 1024) store_y<BF16>(p, i / 128, rt * 128 + i % 128, met(i));
            } else {
                const int first = rt * per;
                bool mine = slot == 1 && u2b - u2a > len && others_done(p.cnt2 + rt, len, S->cuts[1], first, per);
                if (!mine) {
                    float* dst = p.part2 + (int64_t)(blockIdx.x * 2 + slot) * used;
                    for (int i = pt * 4; i < used; i += 1024) __stcg(reinterpret_cast<float4*>(dst + i), met(i));
                    mine = is_last(p.cnt2 + rt, len, S->cuts[1], first, per);
                }
                if (mine) {
                    const int c0 = S->owners[0], c1 = S->owners[1];
                    for (int i = pt * 4; i < used; i += 2048) {
                        Joined s;
                        s.v[0] = met(i);
                        if (i + 1024 < used) s.v[1] = met(i + 1024);
                        s = join4(s, p.part2, used, i, S->cuts[1], c0, c1, first, used);
                        store_y<BF16>(p, i / 128, rt * 128 + i % 128, s.v[0]);
                        if (i + 1024 < used) store_y<BF16>(p, i / 128 + 8, rt * 128 + i % 128, s.v[1]);
                    }
                }
            }
            bar_promotion();  // `sums` is read
            u += len;
        }
    }
    __syncwarp();  // a warp whose lanes parted in its role meets again: the barrier counts whole warps
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(taddr, 512);
    if (threadIdx.x == 0 && *dead) atomicOr(&p.head->status, 1);
}

}  // namespace moe
}  // namespace sqz
