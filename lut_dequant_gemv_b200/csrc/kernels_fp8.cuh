// kernels_fp8.cuh -- 8-bit floating point with one fp32 scale per block of
// 128 columns: the quantizer and the matrix product.
#pragma once

#include <type_traits>

#include "fp8_common.cuh"

namespace sqz {
namespace f8 {

// ------------------------------------------------------------- quantizer
// scale = max|x| / F over a block (F the largest finite code; 1 for a block
// of zeros), code = x / scale rounded to nearest even.
//
// The maximum is taken over the values' bit patterns without the sign: the
// order of non-negative floats is that of their bits, and NaN, above
// infinity, wins, so a block that holds one gets a NaN scale.
//
// The quotient: with y = 1 / scale correctly rounded and q0 = x y,
// q0 - (q0 scale - x) y is x / scale correctly rounded (Markstein 1990) as
// long as no step under- or overflows: three operations where a division
// takes over ten (the kernel would be bound by them, not by its 3 bytes per
// element).  The remainder q0 scale - x has bits down to 2^-47 of x, and a
// quotient that does not round to code 0 is at least 2^-18, so scales from 2^-80
// on keep it exact; blocks whose scale is outside [2^-80, 2^120] (or NaN, or
// infinite) divide.
//
// Measured: 4096 x 13824 bf16 in 1 x 128 blocks 32.4 us, 5.3 TB/s (0.81 of the
// copy rate), bound by instructions (75 % of the issue slots, 15 an element,
// half of them the quotients' and the maxima's); 11000 x 4100 fp16 in 128 x 128
// blocks 30 us, 4.5 TB/s, with 62 % of the issue slots: a CTA's loads, barrier and
// stores follow one another, and the other three of its SM fill the gaps only in
// part; a row of 4096 1.6 us.
struct Quotient {
    float scale, inv;
    __device__ __forceinline__ explicit Quotient(float s) : scale(s), inv(1.f / s) {}
    __device__ __forceinline__ bool divides() const { return !(scale >= 0x1p-80f && scale <= 0x1p120f); }
    // (The remainder's sign is such that -0 / scale stays -0.)
    __device__ __forceinline__ float operator()(float x) const {
        const float q = x * inv;
        return fmaf(-fmaf(q, scale, -x), inv, q);
    }
};

template <bool E5M2>
__device__ __forceinline__ uint32_t code2(float lo, float hi) {
    uint16_t r;
    if (E5M2)
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool BF16>
__device__ __forceinline__ float x_to_float(uint32_t h) {
    if (BF16) return __uint_as_float(h << 16);
    return __half2float(__ushort_as_half((uint16_t)h));
}

// Eight consecutive elements of a row from column c, as they are stored
// (zeros past the edge).  ALIGN: the alignment in bytes that x and its pitch
// have, so the width of the loads; kWhole: 16, and no row ends inside a block
// (the edge's tests were a tenth of the instructions).
constexpr int kWhole = 32;
struct Raw8 {
    uint32_t w[4];
};
template <int ALIGN>
__device__ __forceinline__ Raw8 load8(const uint16_t* row, int c, int cols) {
    Raw8 v;
    if (ALIGN == kWhole || (ALIGN > 2 && c + 8 <= cols)) {
        const char* p = reinterpret_cast<const char*>(row + c);
        if (ALIGN >= 16) {
            const uint4 u = ld_once_u128(p);
            v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
        } else if (ALIGN == 8) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint2 u = ld_u64(p + 8 * i);
                v.w[2 * i] = u.x, v.w[2 * i + 1] = u.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v.w[i] = ld_u32(p + 4 * i);
        }
    } else {
        uint16_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = c + i < cols ? ld_u16(row + c + i) : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) v.w[i] = h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
    }
    return v;
}
// The largest magnitude's bits of eight elements, two at a time (16-bit bit
// patterns order as their values do).
__device__ __forceinline__ uint32_t max_bits8(const Raw8& v, uint32_t m) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, v.w[i] & 0x7FFF7FFFu);
    return m;
}
template <bool BF16>
__device__ __forceinline__ uint32_t fp32_bits(uint32_t m) {
    return __float_as_uint(x_to_float<BF16>(max(m & 0xFFFFu, m >> 16)));
}

// The codes of eight elements; `divides`: by.divides() (rare: a loop).
template <bool BF16, bool E5M2>
__device__ __forceinline__ uint2 codes8(const Raw8& raw, const Quotient& by, bool divides) {
    uint32_t w[4];
    if (divides) {
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            const uint32_t h = i == 0 ? raw.w[0] : i == 1 ? raw.w[1] : i == 2 ? raw.w[2] : raw.w[3];
            const uint32_t c2 = code2<E5M2>(x_to_float<BF16>(h & 0xFFFF) / by.scale, x_to_float<BF16>(h >> 16) / by.scale);
            if (i == 0) w[0] = c2;
            if (i == 1) w[1] = c2;
            if (i == 2) w[2] = c2;
            if (i == 3) w[3] = c2;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = code2<E5M2>(by(x_to_float<BF16>(raw.w[i] & 0xFFFF)), by(x_to_float<BF16>(raw.w[i] >> 16)));
        }
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}
// Eight codes to columns c .. of a row (rows are 16-byte aligned).
template <int ALIGN>
__device__ __forceinline__ void store_codes(uint8_t* __restrict__ row, int c, int cols, const uint2& q) {
    if (ALIGN == kWhole || c + 8 <= cols) {
        *reinterpret_cast<uint2*>(row + c) = q;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < cols) row[c + i] = (uint8_t)((i < 4 ? q.x >> (8 * i) : q.y >> (8 * (i - 4))) & 0xFF);
    }
}

template <bool E5M2>
__device__ __forceinline__ float scale_of(uint32_t max_bits) {
    if (max_bits == 0) return 1.f;
    const float m = __uint_as_float(max_bits), f = E5M2 ? 57344.f : 448.f, inv = 1.f / f;  // (a constant)
    if (!(m >= 0x1p-90f && m <= 0x1p126f)) return m / f;
    const float q = m * inv;
    return fmaf(fmaf(-q, f, m), inv, q);  // correctly rounded, as above
}

struct QuantParams {
    const uint16_t* x;
    int64_t ldx;
    uint8_t* q;
    int64_t ldq;
    float* scale;
    int64_t lds;
    int64_t batch;
    int rows, cols, nblocks;  // nblocks = scale blocks of a row
};

// Blocks of 1 x 128: 8 lanes hold a block, 16 elements each (two loads), so
// that the block's own work (two divisions, the maximum's shuffles, addresses)
// is spread over more elements -- the kernel is bound by its instructions --
// and have kAhead blocks in flight: one where the blocks do not fill the SMs (a
// token), else two.  A warp takes 4 kAhead consecutive blocks a step and strides
// over all rows x blocks.
template <bool BF16, bool E5M2, int ALIGN, int kAhead>
__global__ void __launch_bounds__(256) fp8_quantize_rows_kernel(const QuantParams p) {
    pdl_launch_dependents();
    pdl_wait_previous();
    const int part = (threadIdx.x & 7) * 16;  // of the block
    const int64_t total = p.batch * p.rows * p.nblocks;
    const bool narrow = total <= 0x7fffffff;  // 32-bit division (the 64-bit one costs as much as a block)
    const int64_t step = (int64_t)gridDim.x * (blockDim.x / 8) * kAhead;
    // the loop's bound is the same for the whole warp: its shuffles need every lane
    for (int64_t first = ((int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32) * 4 * kAhead; first < total;
         first += step) {
        Raw8 v[kAhead][2];
        int64_t row[kAhead];
        int b[kAhead];
        const int64_t at = first + ((threadIdx.x >> 3) & 3);
        row[0] = narrow ? (int64_t)((uint32_t)at / (uint32_t)p.nblocks) : at / p.nblocks;
        b[0] = (int)(at - row[0] * p.nblocks);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (i > 0) {
                row[i] = row[i - 1], b[i] = b[i - 1] + 4;
                while (b[i] >= p.nblocks) b[i] -= p.nblocks, ++row[i];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (at + 4 * i < total)
                    v[i][k] = load8<ALIGN>(p.x + row[i] * p.ldx, b[i] * kBlockK + part + 8 * k, p.cols);
                else
                    v[i][k].w[0] = v[i][k].w[1] = v[i][k].w[2] = v[i][k].w[3] = 0;
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            uint32_t m = max_bits8(v[i][1], max_bits8(v[i][0], 0));
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
            const float s = scale_of<E5M2>(fp32_bits<BF16>(m));
            if (at + 4 * i >= total) continue;
            const int c = b[i] * kBlockK + part;
            const Quotient by(s);
            uint8_t* q = p.q + row[i] * p.ldq;
            const bool divides = by.divides();
            const uint2 lo = codes8<BF16, E5M2>(v[i][0], by, divides), hi = codes8<BF16, E5M2>(v[i][1], by, divides);
            if (ALIGN == kWhole || c + 16 <= p.cols) {
                *reinterpret_cast<uint4*>(q + c) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            } else {
                store_codes<ALIGN>(q, c, p.cols, lo);
                store_codes<ALIGN>(q, c + 8, p.cols, hi);
            }
            if (part == 0) p.scale[row[i] * p.lds + b[i]] = s;
        }
    }
}

// Blocks of 128 x 128: one CTA per block, the block in registers (64 elements
// a thread, all its loads in flight) between the maximum and the division, so
// x is read once.
template <bool BF16, bool E5M2, int ALIGN>
__global__ void __launch_bounds__(256, 4) fp8_quantize_tiles_kernel(const QuantParams p) {
    pdl_launch_dependents();
    pdl_wait_previous();
    __shared__ uint32_t part[8];
    const int row_blocks = (p.rows + 127) / 128;
    const int64_t z = blockIdx.y / row_blocks;
    const int rb = (int)(blockIdx.y - z * row_blocks), b = blockIdx.x;
    const int r0 = rb * 128 + (threadIdx.x >> 4), c = b * kBlockK + (threadIdx.x & 15) * 8;
    const uint16_t* x = p.x + z * p.rows * p.ldx;
    uint8_t* q = p.q + z * p.rows * p.ldq;
    Raw8 v[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        if (r < p.rows)
            v[i] = load8<ALIGN>(x + (int64_t)r * p.ldx, c, p.cols);
        else
            v[i].w[0] = v[i].w[1] = v[i].w[2] = v[i].w[3] = 0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max_bits8(v[i], m);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, part[i]);
    const float s = scale_of<E5M2>(fp32_bits<BF16>(m));
    const Quotient by(s);
    const auto write = [&](bool divides) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = r0 + 16 * i;
            if (r < p.rows && (ALIGN == kWhole || c < p.cols))
                store_codes<ALIGN>(q + (int64_t)r * p.ldq, c, p.cols, codes8<BF16, E5M2>(v[i], by, divides));
        }
    };
    if (by.divides())
        write(true);
    else
        write(false);
    if (threadIdx.x == 0) p.scale[(z * row_blocks + rb) * p.lds + b] = s;
}

// -------------------------------------------------------- matrix product
// y[m][n] = sum_b sa[m][b] sw[n / 128][b] * (sum over the 128 k of block b of
// a[m][k] w[n][k]).  The inner sum is four tcgen05 matrix instructions into
// tensor memory; the outer one is carried in fp32 registers, one fused
// multiply-add per output and block ("promotion").  Blocks with a product of
// scales outside fp32's normal numbers take two factors (split_scales); the
// few-row kernel's promotion asks while tensor memory answers, the many-row
// kernel's leaves it to the warp that copies the scales.

struct GemmParams {
    const float* sa;
    int64_t ld_sa;
    const float* sw;
    int64_t ld_sw;
    void* y;
    int64_t ldy;
    uint32_t* status;
    int m, n, nkb;  // nkb = blocks of K
    int out_type;
    uint32_t idesc;
    int stages;
    int tiles_m, tiles_n;  // many-row kernel
    int out_align;         // alignment of y's rows in bytes: 32, 16 or less
};

constexpr int kMaxStages = 12;

// Few rows of A (up to 64): bound by reading W.  The weights take the 128
// lanes (MMA "A", 128 rows of W) and the TB tokens the columns, so a tile
// costs the tensor cores little however few tokens there are, and the K axis
// is split over the CTAs of a cluster, whose partial sums meet in distributed
// shared memory in rank order: no workspace, no atomics, the same bits every
// run.
//
// Measured: 16 x 5120 x 13824 16.0 us, 4.4 TB/s with about 4 us of launch,
// first copies and the sums' meeting (16 x 18944 x 32768: 6.1 TB/s); 1 x 4096 x
// 4096 6.1 us; 32 x 5120 x 5120 9.4; 64 x 5120 x 13824 19.9.
//
//   warp 0: TMA loads of W and A tiles into a ring of stages
//   warp 1: TMEM allocation, matrix instructions into a ring of accumulators
//   warp 2: the block's scales into the stage (4-byte asynchronous copies)
//   warps 3-6: promotion; thread = a row of W
template <int TB>
struct FewShape {
    static constexpr int kStageBytes = kTileBytes + TB * kBlockK;
    static constexpr int kScaleFloats = TB + 4;  // TB token scales, the weights' scale
    // A block's way from the matrix instruction through the promotion and back
    // to a free accumulator takes over a thousand cycles (barriers, mostly): two
    // accumulators let a CTA do a block every 820, eight one every 550 (half the
    // tensor memory, so that two CTAs share an SM).
    static constexpr int kBufs = 256 / TB < 8 ? 256 / TB : 8;
    static constexpr int kTmemCols = kBufs * TB;
    static constexpr int kThreads = 224;
    static int smem_bytes(int stages) { return 1024 + stages * (kStageBytes + kScaleFloats * 4); }
};

template <int TB>
__global__ void __launch_bounds__(224) fp8_gemm_few_kernel(const __grid_constant__ CUtensorMap map_w,
                                                            const __grid_constant__ CUtensorMap map_a,
                                                            const GemmParams p) {
    using S = FewShape<TB>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tfull[S::kBufs], tempty[S::kBufs];
    __shared__ uint32_t taddr_s;
    __shared__ int dead_s;
    uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    float* scales = reinterpret_cast<float*>(ring + p.stages * S::kStageBytes);
    volatile int* dead = &dead_s;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int splits = gridDim.x, rank = blockIdx.x;
    const int row0 = blockIdx.y * 128, tok0 = blockIdx.z * TB;
    const int kb0 = (int)((int64_t)p.nkb * rank / splits), kb1 = (int)((int64_t)p.nkb * (rank + 1) / splits);
    const int nk = kb1 - kb0;

    if (warp == 1) tmem_alloc(&taddr_s, S::kTmemCols);
    if (threadIdx.x == 0) {
        dead_s = 0;
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&full[i], 1 + 32);
            mbar_init(&empty[i], 1 + 4);
        }
        for (int i = 0; i < S::kBufs; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 4);
        }
        fence_mbar_init();
        tma_prefetch_map(&map_w);
        tma_prefetch_map(&map_a);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t taddr = taddr_s;
    pdl_launch_dependents();
    pdl_wait_previous();

    float acc[TB];
    if (warp == 0) {
        int st = 0, ph = 0, it = 0;
        for (; it < nk; ++it) {
            if (!wait_warp(&empty[st], ph ^ 1, dead)) break;
            uint8_t* at = ring + st * S::kStageBytes;
            if (elect_one()) {
                mbar_expect_tx(&full[st], S::kStageBytes);
                tma_load_2d(at, &map_w, &full[st], (kb0 + it) * kBlockK, row0);
                tma_load_2d(at + kTileBytes, &map_a, &full[st], (kb0 + it) * kBlockK, tok0);
            }
            __syncwarp();
            if (++st == p.stages) st = 0, ph ^= 1;
        }
        if (it < nk) let_copies_land();
    } else if (warp == 1) {
        int st = 0, ph = 0, it = 0;
        Ahead next;
        next.ask(&full[0], 0, &tempty[0], 1);
        for (; it < nk; ++it) {
            const int buf = it % S::kBufs, used = st;
            if (!next.wait(&full[st], ph, &tempty[buf], ((it / S::kBufs) & 1) ^ 1, dead)) break;
            tc_fence_after();
            if (++st == p.stages) st = 0, ph ^= 1;
            next.ask(&full[st], ph, &tempty[(it + 1) % S::kBufs], (((it + 1) / S::kBufs) & 1) ^ 1);
            const uint32_t at = smem_u32(ring + used * S::kStageBytes);
            if (elect_one()) {
                mma_block(taddr + buf * TB, at, at + kTileBytes, p.idesc);
                mma_commit(&tfull[buf]);
                mma_commit(&empty[used]);
            }
            __syncwarp();
        }
        if (it < nk) let_copies_land();
    } else if (warp == 2) {
        int st = 0, ph = 0;
        const float* sw = p.sw + (int64_t)blockIdx.y * p.ld_sw;
        for (int it = 0; it < nk; ++it) {
            if (!__all_sync(0xffffffffu, wait_alive(&empty[st], ph ^ 1, dead))) break;
            float* dst = scales + st * S::kScaleFloats;
            const int kb = kb0 + it;
#pragma unroll
            for (int t = lane; t < TB; t += 32)  // (a column of no token is never stored: any scale does)
                if (tok0 + t < p.m) cp_async4(dst + t, p.sa + (int64_t)(tok0 + t) * p.ld_sa + kb);
            if (lane == 0) cp_async4(dst + TB, sw + kb);
            cp_async_arrive(&full[st]);
            if (++st == p.stages) st = 0, ph ^= 1;
        }
    } else {
#pragma unroll
        for (int t = 0; t < TB; ++t) acc[t] = 0.f;
        const uint32_t lanes = taddr + ((uint32_t)(warp & 3) << 21);
        const bool no_token = tok0 + lane % TB >= p.m, no_later = TB > 32 ? tok0 + lane + TB - 32 >= p.m : no_token;
        int st = 0, ph = 0;
        for (int it = 0; it < nk; ++it) {
            const int buf = it % S::kBufs;
            bool ok = wait_alive(&full[st], ph, dead);  // the scales of the stage
            ok = ok && wait_alive(&tfull[buf], (it / S::kBufs) & 1, dead);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const float* sc = scales + st * S::kScaleFloats;
            const float sw = sc[TB];
            uint32_t d[16];
            tmem_ld16(lanes + buf * TB, d);
            // The first columns' scales, and whether all products of scales are normal
            // numbers, while tensor memory answers.
            constexpr int kHead = TB < 32 ? TB : 32;
            float s[kHead];
#pragma unroll
            for (int j = 0; j < kHead; ++j) {
                s[j] = sc[j] * sw;
                asm volatile("" : "+f"(s[j]));  // (here, not behind the branch)
            }
            const float mine = sc[lane % TB] * sw, later = TB > 32 ? sc[lane + TB - 32] * sw : mine;
            const bool plain = __all_sync(0xffffffffu, (in_range(mine) | no_token) & (in_range(later) | no_later));
            tmem_wait_ld(d);
            if (plain) {
#pragma unroll
                for (int c = 0; c < TB; c += 16) {
                    if (c > 0) {
                        tmem_ld16(lanes + buf * TB + c, d);
                        tmem_wait_ld(d);
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        acc[c + j] = fmaf(__uint_as_float(d[j]), c < kHead ? s[c % kHead + j] : sc[c + j] * sw, acc[c + j]);
                }
            } else {  // lane t splits the scales of tokens t and t + 32
                const ScalePair own = split_scales(sc[lane % TB], sw), own32 = split_scales(sc[(lane + 32) % TB], sw);
#pragma unroll
                for (int c = 0; c < TB; c += 16) {
                    tmem_ld16(lanes + buf * TB + c, d);
                    tmem_wait_ld(d);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const ScalePair& from = c + j < 32 ? own : own32;
                        const float f = __shfl_sync(0xffffffffu, from.first, (c + j) & 31);
                        acc[c + j] =
                            fmaf(__uint_as_float(d[j]) * f, __shfl_sync(0xffffffffu, from.s, (c + j) & 31), acc[c + j]);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&tempty[buf]);
                mbar_arrive(&empty[st]);
            }
            if (++st == p.stages) st = 0, ph ^= 1;
        }
    }
    __syncwarp();  // a warp whose lanes parted in its role meets again: the barrier counts whole warps
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(taddr, S::kTmemCols);
    if (threadIdx.x == 0 && *dead) atomicAdd(p.status, 1u);

    const int tokens = min(TB, p.m - tok0);
    const int r = (warp & 3) * 32 + lane;  // row of W in the tile (promotion warps)
    if (splits == 1) {
        if (warp >= 3 && row0 + r < p.n) {
#pragma unroll
            for (int t = 0; t < TB; ++t)
                if (t < tokens) store_out(p.y, (int64_t)(tok0 + t) * p.ldy + row0 + r, p.out_type, acc[t]);
        }
        return;
    }
    float* red = reinterpret_cast<float*>(ring);  // every copy into the ring has been read
    if (warp >= 3) {
#pragma unroll
        for (int t = 0; t < TB; ++t)
            if (t < tokens) red[t * 128 + r] = acc[t];
    }
    cluster_sync();
    // Rows that this CTA finishes (fours, so that a load is 16 bytes); the loads
    // from all CTAs are in flight together.
    const int rows = (128 + 4 * splits - 1) / (4 * splits) * 4, first = rank * rows;
    for (int i = threadIdx.x; i < rows / 4 * tokens; i += S::kThreads) {
        const int t = i / (rows / 4), rr = first + i % (rows / 4) * 4;
        if (rr >= 128 || row0 + rr >= p.n) continue;
        float4 part[8];
#pragma unroll
        for (int c = 0; c < 8; ++c)
            part[c] = c < splits ? ld_cluster4(red + t * 128 + rr, c) : make_float4(0.f, 0.f, 0.f, 0.f);
        float4 v = part[0];
#pragma unroll
        for (int c = 1; c < 8; ++c) v.x += part[c].x, v.y += part[c].y, v.z += part[c].z, v.w += part[c].w;
        const int64_t at = (int64_t)(tok0 + t) * p.ldy + row0 + rr;
        store_out(p.y, at, p.out_type, v.x);
        if (row0 + rr + 1 < p.n) store_out(p.y, at + 1, p.out_type, v.y);
        if (row0 + rr + 2 < p.n) store_out(p.y, at + 2, p.out_type, v.z);
        if (row0 + rr + 3 < p.n) store_out(p.y, at + 3, p.out_type, v.w);
    }
    cluster_sync();  // the other CTAs have read this one's sums
}

// Many rows of A: tiles of 256 rows of A x BN rows of W, by pairs of CTAs (one
// CTA an SM, persistent): each CTA loads its own 128 rows of A and half of W's
// rows, and the matrix instructions (cta_group::2) read W's halves from both.
// Alone, a CTA with a 128 x 256 tile would have 48 KB a block of K written to
// its shared memory and 48 KB read from it for 512 cycles of matrix
// instructions, more than the 128 bytes a cycle it has.
//
// A thread of the promotion holds one row of A and BN / 2 columns: the block's
// scale is then one or two numbers per thread (the row's scale times those of
// the 128-row blocks of W that its columns lie in).  Packed fp32 multiply-adds
// measured slower here than plain ones.
//
// What bounds it, by the clocks of a CTA's roles (cycles a block of K):
//   64 columns, eight accumulators: 495, of which the issuing warp spends 340 on
//   the instructions of the block (four products, two commits, the next polls) and
//   155 waiting.  The matrix instructions themselves take 128: the issue is what
//   every width pays, and most of the 180 ns that a block costs at any width.
//   256 columns, two accumulators: 935, of which the issue takes 335, a wait for
//   an accumulator 485 and one for a stage 110.  The promotion has 935 as well:
//   487 of reads, 248 of the last multiply-adds and its loop, 198 of waiting: an
//   accumulator's way through it is what the issue waits for.
// 8192 x 11008 x 4096 in 356 to 363 us (2.05 PFLOP/s, tensor pipe 47 %; 422 us
// under the power cap, 1.75).
//
//   warp 0: TMA ring (the full barriers live in the even CTA, the empty ones
//   in both), warp 1: TMEM and, in the even CTA, matrix instructions, warp 2:
//   scales, sixteen blocks of K ahead (a wait for each block's would cost the
//   promotion 200 cycles; loads into its registers stall its reads of tensor
//   memory), and whether their products stay in range, warps 3-10: promotion
//   (warp % 4 = the 32 lanes it may read; first or second half of the columns)
template <int BN>
struct ManyShape {
    static constexpr int kRowsW = BN / 2;  // of W, in each CTA
    static constexpr int kStageBytes = kTileBytes + kRowsW * kBlockK;
    static constexpr int kBufs = 512 / BN;  // accumulators that take turns
    static constexpr int kTmemCols = kBufs * BN > 256 ? 512 : 256;  // (allocated in powers of two)
    static constexpr int kPromotionWarps = 8;
    static constexpr int kThreads = 96 + kPromotionWarps * 32;
    static constexpr int kCols = BN / 2;   // columns of a thread
    static constexpr bool kOneBlock = 256 % BN == 0;  // ... lie in one block of 128 rows of W (else in two)
    static constexpr int kChunk = 16;      // columns of a load from tensor memory
    // scales of kScaleRun blocks of K at a time, [four blocks][128 rows of A, 2 for W][4]
    static constexpr int kScaleRun = 16;
    static constexpr int kScaleRows = 128 + 2;
    // a promotion warp's 32 rows x 16 columns on their way to unaligned rows of y
    static constexpr int kTurnPitch = 17;
    static constexpr int kTurnFloats = 32 * kTurnPitch;
    static int smem_bytes(int stages) {
        return 1024 + stages * kStageBytes + 2 * kScaleRun * kScaleRows * 4 + kPromotionWarps * kTurnFloats * 4;
    }
};

// V consecutive values (2 to 8 bytes, aligned to their size) to y.
template <int V>
__device__ __forceinline__ void store_few(const GemmParams& p, int64_t at, const float (&v)[V]) {
    if (V == 1 || (V == 4 && p.out_type == kF32)) {  // (four fp32 would be 16 bytes: never asked for)
        store_out(p.y, at, p.out_type, v[0]);
    } else if (p.out_type == kF32) {
        *reinterpret_cast<float2*>(static_cast<float*>(p.y) + at) = make_float2(v[0], v[V > 1 ? 1 : 0]);
    } else {
        uint32_t w[V / 2 + 1];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if (p.out_type == kF16) {
                const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        uint16_t* y = static_cast<uint16_t*>(p.y) + at;
        if (V == 4)
            *reinterpret_cast<uint2*>(y) = make_uint2(w[0], w[V / 4]);
        else
            *reinterpret_cast<uint32_t*>(y) = w[0];
    }
}

// Rows of y that are not 16-byte aligned: 16 columns of the warp's 32 rows at a
// time are turned through shared memory, so that neighbouring lanes write
// neighbouring values, V each (a lane writing its own row 2 to 8 bytes at a time
// costs a line of L1 per lane and store: 398 x 4799 x 7308 51 us, turned 33).
// `turn`: the warp's buffer; lane = row row0 + lane of y, v its values from
// column col0 on.
template <int V, int N, int PITCH>
__device__ __forceinline__ void store_turned(const GemmParams& p, int64_t row0, int col0, int lane, float* turn,
                                             const float (&v)[N]) {
    constexpr int kLanes = 16 / V, kRows = 32 / kLanes;  // lanes of a row, rows of a store
    const int lc = lane % kLanes * V, lr = lane / kLanes;
#pragma unroll
    for (int c = 0; c < N; c += 16) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) turn[lane * PITCH + j] = v[c + j];
        __syncwarp();
        const int col = col0 + c + lc;
        int64_t at = (row0 + lr) * p.ldy + col;
#pragma unroll 4
        for (int r = lr; r < 32; r += kRows, at += kRows * p.ldy) {
            float a[V];
#pragma unroll
            for (int j = 0; j < V; ++j) a[j] = turn[r * PITCH + lc + j];
            if (row0 + r >= p.m) continue;
            if (col + V <= p.n) {
                store_few<V>(p, at, a);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (col + j < p.n) store_out(p.y, at + j, p.out_type, a[j]);
            }
        }
    }
    __syncwarp();
}

// The first `left` of N consecutive values to a row of y that is 16-byte
// aligned (p.out_align), 32 bytes at a time up to its end.
template <int N>
__device__ __forceinline__ void store_row(const GemmParams& p, int64_t at, int left, const float (&v)[N]) {
    if (p.out_type == kF32) {
#pragma unroll
        for (int j = 0; j < N; j += 8) {
            if (j + 8 <= left) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[j + i]);
                st_global_32b(static_cast<float*>(p.y) + at + j, w, p.out_align);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (j + i < left) static_cast<float*>(p.y)[at + j + i] = v[j + i];
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 16) {
            if (j + 16 <= left) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (p.out_type == kF16) {
                        const __half2 h = __floats2half2_rn(v[j + 2 * i], v[j + 2 * i + 1]);
                        w[i] = *reinterpret_cast<const uint32_t*>(&h);
                    } else {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(v[j + 2 * i], v[j + 2 * i + 1]);
                        w[i] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                }
                st_global_32b(static_cast<uint16_t*>(p.y) + at + j, w, p.out_align);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (j + i < left) store_out(p.y, at + j + i, p.out_type, v[j + i]);
            }
        }
    }
}

// The warp's lanes' sums in tensor memory times a factor: `first` before column
// `split` (a multiple of 16), `later` from there on.  The rare path of odd scales:
// in tensor memory and in a loop, so that it takes nothing from the registers
// and the unrolled reads of the others (a branch among those costs them a third).
__device__ __forceinline__ void scale_sums(uint32_t taddr, int cols, int split, float first, float later) {
#pragma unroll 1
    for (int c = 0; c < cols; c += 16) {
        const float f = c < split ? first : later;
        uint32_t d[16];
        tmem_ld16(taddr + c, d);
        tmem_wait_ld(d);
#pragma unroll
        for (int j = 0; j < 16; ++j) d[j] = __float_as_uint(__uint_as_float(d[j]) * f);
        tmem_st16(taddr + c, d);
    }
    tmem_wait_st();
}

// V: 0 for 16-byte aligned rows of y, else the values of a store (see above).
template <int BN, int V>
__global__ void __launch_bounds__(ManyShape<BN>::kThreads, 1) fp8_gemm_many_kernel(
    const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a, const GemmParams p) {
    using S = ManyShape<BN>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tfull[S::kBufs], tempty[S::kBufs];
    __shared__ uint64_t sfull[2], sempty[2];
    __shared__ uint32_t taddr_s;
    __shared__ int dead_s, odd_s[2];  // odd_s: whether a run's scales take two factors
    uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    float* scales = reinterpret_cast<float*>(ring + p.stages * S::kStageBytes);
    volatile int* dead = &dead_s;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = (int)cluster_rank(), pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;

    if (warp == 1) tmem_alloc_pair(&taddr_s, S::kTmemCols);
    if (threadIdx.x == 0) {
        dead_s = 0;
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < S::kBufs; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * S::kPromotionWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&sempty[i], S::kPromotionWarps);
        }
        fence_mbar_init();
        tma_prefetch_map(&map_w);
        tma_prefetch_map(&map_a);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // the other CTA's barriers are ready
    tc_fence_after();
    const uint32_t taddr = taddr_s;
    pdl_launch_dependents();
    pdl_wait_previous();

    if (warp == 0) {
        int st = 0, ph = 0;
        bool alive = true;
        const uint32_t leader_full = cluster_addr(full, 0);
        for (int64_t tile = pair; tile < tiles && alive; tile += pairs) {
            const int tn = (int)(tile / p.tiles_m), tm = (int)(tile - (int64_t)tn * p.tiles_m);
            // a CTA whose rows all lie past the last one multiplies the first ones
            const int row0 = tm * 256 + rank * 128 < p.m ? tm * 256 + rank * 128 : 0;
            for (int kb = 0; kb < p.nkb; ++kb) {
                if (!(alive = wait_warp(&empty[st], ph ^ 1, dead))) break;
                const uint32_t bar = leader_full + st * 8;
                uint8_t* at = ring + st * S::kStageBytes;
                if (elect_one()) {
                    if (rank == 0) mbar_expect_tx(&full[st], 2 * S::kStageBytes);
                    tma_load_2d_pair(at, &map_a, bar, kb * kBlockK, row0);
                    tma_load_2d_pair(at + kTileBytes, &map_w, bar, kb * kBlockK, tn * BN + rank * S::kRowsW);
                }
                __syncwarp();
                if (++st == p.stages) st = 0, ph ^= 1;
            }
        }
        // The last arrivals on this CTA's empty barriers come from the even CTA:
        // they are here before this one leaves.
        for (int i = 0; i < p.stages && alive; ++i) {
            alive = wait_warp(&empty[st], ph ^ 1, dead);
            if (++st == p.stages) st = 0, ph ^= 1;
        }
        if (!alive) let_copies_land();
    } else if (warp == 1) {
        if (rank == 0) {
            int st = 0, ph = 0;
            uint32_t it = 0;
            bool alive = true;
            Ahead next;
            next.ask(&full[0], 0, &tempty[0], 1);
            for (int64_t tile = pair; tile < tiles && alive; tile += pairs) {
                for (int kb = 0; kb < p.nkb; ++kb) {
                    const int buf = it % S::kBufs, used = st;
                    alive = next.wait(&full[st], ph, &tempty[buf], ((it / S::kBufs) & 1) ^ 1, dead);
                    if (!alive) break;
                    tc_fence_after();
                    if (++st == p.stages) st = 0, ph ^= 1;
                    ++it;
                    next.ask(&full[st], ph, &tempty[it % S::kBufs], ((it / S::kBufs) & 1) ^ 1);
                    const uint32_t at = smem_u32(ring + used * S::kStageBytes);
                    if (elect_one()) {
                        mma_block_pair(taddr + buf * BN, at, at + kTileBytes, p.idesc);
                        mma_commit_pair(&tfull[buf]);
                        mma_commit_pair(&empty[used]);
                    }
                    __syncwarp();
                }
            }
            if (!alive) let_copies_land();
        }
    } else if (warp == 2) {
        uint32_t runs = 0;
        bool alive = true;
        const int w_blocks = (p.n + 127) / 128;
        for (int64_t tile = pair; tile < tiles && alive; tile += pairs) {
            const int tn = (int)(tile / p.tiles_m), tm = (int)(tile - (int64_t)tn * p.tiles_m);
            for (int k0 = 0; k0 < p.nkb; k0 += S::kScaleRun, ++runs) {
                if (!(alive = wait_warp(&sempty[runs & 1], ((runs >> 1) & 1) ^ 1, dead))) break;
                float* dst = scales + (runs & 1) * S::kScaleRun * S::kScaleRows;
                // A half-warp copies a row's run of consecutive scales: few lines of
                // L1 a copy, whatever the pitch.  (What belongs to no row is never
                // stored: any scale does.)
                const int k = k0 + (lane & 15), at = (lane & 15) / 4 * 4 * S::kScaleRows + (lane & 3);
                const int rows = min(128, p.m - (tm * 256 + rank * 128)), wb = tn * BN / 128 + lane / 16;
                if (k < p.nkb) {
                    const float* sa = p.sa + (int64_t)(tm * 256 + rank * 128) * p.ld_sa + k;
                    for (int i = lane / 16; i < rows; i += 2) cp_async4(dst + at + 4 * i, sa + (int64_t)i * p.ld_sa);
                    if (wb < w_blocks) cp_async4(dst + at + 4 * (128 + lane / 16), p.sw + wb * p.ld_sw + k);
                }
                cp_async_commit();
                cp_async_wait<0>();
                __syncwarp();
                // The least and the largest of each side's magnitudes (bits order as
                // values): products that they keep in range need no second factor.
                uint32_t least = __float_as_uint(1.f), most = least, least_w = least, most_w = least;
                for (int i = lane; i < rows; i += 32) {
#pragma unroll
                    for (int q = 0; q < S::kScaleRun / 4; ++q) {
                        const uint4 a = *reinterpret_cast<const uint4*>(dst + 4 * (q * S::kScaleRows + i));
                        const uint32_t v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (k0 + 4 * q + j < p.nkb)
                                least = min(least, v[j] & 0x7FFFFFFFu), most = max(most, v[j] & 0x7FFFFFFFu);
                    }
                }
                if (k < p.nkb && wb < w_blocks) {
                    const uint32_t v = __float_as_uint(dst[at + 4 * (128 + lane / 16)]) & 0x7FFFFFFFu;
                    least_w = min(least_w, v), most_w = max(most_w, v);
                }
                least = __reduce_min_sync(0xffffffffu, least), least_w = __reduce_min_sync(0xffffffffu, least_w);
                most = __reduce_max_sync(0xffffffffu, most), most_w = __reduce_max_sync(0xffffffffu, most_w);
                if (lane == 0) {
                    odd_s[runs & 1] = !in_range(__uint_as_float(least) * __uint_as_float(least_w)) ||
                                      !in_range(__uint_as_float(most) * __uint_as_float(most_w));
                    mbar_arrive(&sfull[runs & 1]);
                }
                __syncwarp();
            }
        }
    } else {
        const int group = (warp - 3) / 4;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes = taddr + ((uint32_t)(warp & 3) << 21) + group * S::kCols;
        const uint32_t leader_tempty = cluster_addr(tempty, 0);
        float* turn = scales + 2 * S::kScaleRun * S::kScaleRows + (warp - 3) * S::kTurnFloats;
        uint32_t it = 0, runs = 0;
        bool alive = true;
        for (int64_t tile = pair; tile < tiles && alive; tile += pairs) {
            const int tn = (int)(tile / p.tiles_m), tm = (int)(tile - (int64_t)tn * p.tiles_m);
            const int64_t row = (int64_t)tm * 256 + rank * 128 + r;
            const int col0 = tn * BN + group * S::kCols;
            // the block of W that the thread's first column lies in (of the
            // tile's), and its first column of the next one
            const int block = col0 / 128 - tn * BN / 128, split = (col0 / 128 + 1) * 128 - col0;
            float acc[S::kCols];
#pragma unroll
            for (int j = 0; j < S::kCols; ++j) acc[j] = 0.f;
            // Block kb of the run whose scales are at sc; `odd`: with two factors.
            const auto promote = [&](const float* sc, int kb, auto odd) {
                const int buf = it % S::kBufs;
                const float* quad = sc + kb / 4 * 4 * S::kScaleRows + kb % 4;
                float s0 = quad[4 * r] * quad[4 * (128 + block)];
                float s1 = S::kOneBlock ? s0 : quad[4 * r] * quad[4 * (128 + 1)];
                if (!(alive = wait_warp(&tfull[buf], (it / S::kBufs) & 1, dead))) return;
                tc_fence_after();
                if (odd) {
                    const ScalePair f0 = split_scales(quad[4 * r], quad[4 * (128 + block)]);
                    const ScalePair f1 = S::kOneBlock ? f0 : split_scales(quad[4 * r], quad[4 * (128 + 1)]);
                    s0 = f0.s, s1 = f1.s;
                    scale_sums(lanes + buf * BN, S::kCols, S::kOneBlock ? S::kCols : split, f0.first, f1.first);
                }
#pragma unroll
                for (int c = 0; c < S::kCols; c += S::kChunk) {
                    uint32_t d[S::kChunk];
                    tmem_ld16(lanes + buf * BN + c, d);
                    tmem_wait_ld(d);
                    if (c + S::kChunk == S::kCols) {  // the accumulator is read
                        tc_fence_before();
                        __syncwarp();
                        if (elect_one()) mbar_arrive_cluster(leader_tempty + buf * 8);
                    }
#pragma unroll
                    for (int j = 0; j < S::kChunk; ++j)
                        acc[c + j] = fmaf(__uint_as_float(d[j]), S::kOneBlock || c < split ? s0 : s1, acc[c + j]);
                }
                ++it;
            };
            for (int k0 = 0; k0 < p.nkb && alive; k0 += S::kScaleRun, ++runs) {
                if (!(alive = wait_warp(&sfull[runs & 1], (runs >> 1) & 1, dead))) break;
                const float* sc = scales + (runs & 1) * S::kScaleRun * S::kScaleRows;
                const int len = min(S::kScaleRun, p.nkb - k0);
                if (!odd_s[runs & 1]) {
#pragma unroll 1
                    for (int kb = 0; kb < len && alive; ++kb) promote(sc, kb, std::false_type());
                } else {  // (a loop of its own: a test of each block in the other one costs it 3 to 30 %)
#pragma unroll 1
                    for (int kb = 0; kb < len && alive; ++kb) promote(sc, kb, std::true_type());
                }
                __syncwarp();
                if (elect_one()) mbar_arrive(&sempty[runs & 1]);
            }
            if (!alive) continue;
            if (V == 0) {
                if (row < p.m) store_row<S::kCols>(p, row * p.ldy + col0, p.n - col0, acc);
            } else {
                store_turned<V == 0 ? 1 : V, S::kCols, S::kTurnPitch>(p, row - lane, col0, lane, turn, acc);
            }
        }
    }
    __syncwarp();  // a warp whose lanes parted in its role meets again: the barrier counts whole warps
    __syncthreads();
    cluster_sync();  // nothing of the other CTA is on its way here any more
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(taddr, S::kTmemCols);
    if (threadIdx.x == 0 && *dead) atomicAdd(p.status, 1u);
}

}  // namespace f8
}  // namespace sqz
