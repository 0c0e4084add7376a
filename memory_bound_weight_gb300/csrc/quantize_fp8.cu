// quantize_fp8.cu -- 8-bit floating point with a scale for each block of 128:
// activations by row and 128 columns (optionally of the RMS-normed row), weights
// by 128 x 128, and both back.
//
//   s = max|x| / 448,  code = e4m3(x / s),  value = s * code
//
// Both divisions are IEEE fp32, the code is rounded to nearest even, a block of
// zeros has s = 0 and codes 0. A block that holds a NaN or an infinity reads as
// NaN: its scale is one, or is infinite, which makes the quotients zero and NaN.
//
// The quotients are Markstein's (IBM J. Res. Dev. 1990), q = x r, q + (x - q s) r
// with the correctly rounded reciprocal r, one for a block: correctly rounded where
// the remainder x - q s is, which holds for s in [2^-60, 2^60] and every x whose
// quotient is 2^-10 or more; a smaller one is code 0 whatever its last bit. Other
// scales take the division itself.
//
// What bounds it: memory, for large ones (rows of 4096 x 18944: 39.8 us, 5.85 TB/s;
// weights 18944 x 3584: 35 us, 5.8 TB/s; values back 56 us, 6.0 TB/s), and launch and a
// chain of dependent steps for small ones (one row: 1.7 us, normed 2.6). Normed rows:
// instructions and latency (4000 x 3584: 16.4 us, 2.6 TB/s; 20000 x 3328: 62 us). What
// it cost on the way there: the roots of those 4000 rows in 64 bits by every thread 70 us;
// 8 columns a lane in place of 16 (rows 19 us in place of 10.6); a branch per quotient for
// scales out of range, and 64-bit divisions of indexes, a third more.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device.cuh"
#include "internal.h"

namespace mbw {

namespace {

struct Divide {
    float s, r;
    bool plain;
    __device__ __forceinline__ explicit Divide(float scale) : s(scale) {
        plain = s >= 0x1p-60f && s <= 0x1p60f;
        r = plain ? __frcp_rn(s) : 0.f;
    }
    template <bool PLAIN>
    __device__ __forceinline__ float of(float x) const {
        if (PLAIN) {
            const float q = x * r;
            return fmaf(fmaf(-q, s, x), r, q);
        }
        return s == 0.f ? 0.f : __fdiv_rn(x, s);
    }
};

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// 8 bf16 values as codes.
template <bool PLAIN>
__device__ __forceinline__ uint2 codes8(const uint4& v, const Divide& d) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = to_e4m3x2(d.of<PLAIN>(bf16lo_to_f32(w[i])), d.of<PLAIN>(bf16hi_to_f32(w[i])));
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
// The largest magnitude of 8 bf16 values, as bits in both halves; those of a NaN are the largest.
__device__ __forceinline__ uint32_t largest8(uint32_t m, const uint4& v) {
    return __vmaxu2(__vmaxu2(__vmaxu2(m, v.x & 0x7FFF7FFFu), __vmaxu2(v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu)), v.w & 0x7FFF7FFFu);
}
__device__ __forceinline__ float scale_of(uint32_t most) {
    const float m = __uint_as_float(max(most >> 16, most & 0xFFFFu) << 16);
    if (m >= 0x1p-90f && m <= 0x1p120f) {  // the quotient as above, of the correctly rounded 1/448
        const float r = 0x1.24924ap-9f, q = m * r;
        return fmaf(fmaf(-q, 448.0f, m), r, q);
    }
    return __fdiv_rn(m, 448.0f);
}
// 16 columns a lane, 8 lanes a block: the reciprocal and the block's maximum are a third of the instructions with 8 columns.
struct Words {
    uint4 a, b;
};
__device__ __forceinline__ Words load16(const uint16_t* p, bool wide) {  // wide: p lies on 32 bytes
    Words v;
    if (wide)
        asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v.a.x), "=r"(v.a.y), "=r"(v.a.z), "=r"(v.a.w), "=r"(v.b.x), "=r"(v.b.y), "=r"(v.b.z), "=r"(v.b.w) : "l"(p));
    else
        v.a = ld_ro16(p), v.b = ld_ro16(p + 8);
    return v;
}
__device__ __forceinline__ uint32_t largest_of_block(const Words& v) {
    uint32_t m = largest8(largest8(0, v.a), v.b);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return m;
}
__device__ __forceinline__ void put16(uint8_t* q, const Words& v, const Divide& d) {
    uint2 a, b;
    if (d.plain)
        a = codes8<true>(v.a, d), b = codes8<true>(v.b, d);
    else
        a = codes8<false>(v.a, d), b = codes8<false>(v.b, d);
    *reinterpret_cast<uint4*>(q) = make_uint4(a.x, a.y, b.x, b.y);
}

constexpr int kThreads = 256;

// Rows as they are: eight lanes take a block of 128 columns, two blocks at a time, whose loads go together.
constexpr int kBatch = 4;
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const uint16_t* __restrict__ X, int64_t stride, uint8_t* __restrict__ Q,
                                                                 float* __restrict__ S, int64_t M, int KB) {
    constexpr int BATCH = 2;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t blocks = M * KB, step = (int64_t)gridDim.x * (kThreads / 8);
    const int lane = threadIdx.x & 7, part = (threadIdx.x >> 3) & 3;
    const bool dense = stride == (int64_t)KB * 128, wide = ((uintptr_t)X & 31) == 0 && stride % 16 == 0;
    // a warp's four parts go round equally often
    for (int64_t b0 = (int64_t)blockIdx.x * (kThreads / 8) + (threadIdx.x / 32) * 4; b0 < blocks; b0 += BATCH * step) {
        Words v[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int64_t b = b0 + i * step + part;
            v[i].a = v[i].b = make_uint4(0, 0, 0, 0);
            if (b < blocks) {
                int64_t at = b * 128;
                if (!dense) {
                    const int64_t row = blocks < (1ll << 31) ? (int64_t)((uint32_t)b / (uint32_t)KB) : b / KB;
                    at = row * stride + (b - row * KB) * 128;
                }
                v[i] = load16(X + at + lane * 16, wide);
            }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int64_t b = b0 + i * step + part;
            const float s = scale_of(largest_of_block(v[i]));
            if (b < blocks) {
                put16(Q + b * 128 + lane * 16, v[i], Divide(s));
                if (lane == 0) S[b] = s;
            }
        }
    }
}

// The sum of a and b without loss, in two floats (Knuth's two-sum).
__device__ __forceinline__ void add2(float& hi, float& lo, float x) {
    const float s = hi + x, t = s - hi;
    lo += (hi - (s - t)) + (x - t);
    hi = s;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{.reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z;}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
// 8 bf16 values times r and their weights, rounded to bf16, as norm_word.
__device__ __forceinline__ uint4 normed(const uint4& v, float r, const uint4& g) {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w}, w[4] = {g.x, g.y, g.z, g.w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(bf16lo_to_f32(x[j]) * r * bf16lo_to_f32(w[j]), bf16hi_to_f32(x[j]) * r * bf16hi_to_f32(w[j]));
        o[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}
// 1 / sqrt(sum / k + eps) rounded to fp32, the sum and eps in two floats each: the approximation r0 and the step of Newton's
// method from its error 1 - v r0^2, in which the products' remainders (by fma) are kept; off by 2^-44 before its rounding.
// (In 64 bits by every thread, the roots of 4000 rows took 70 us.)
__device__ __forceinline__ float inverse_root(float hi, float lo, float k, float eps_hi, float eps_lo) {
    float v = __fdiv_rn(hi, k), low = __fdiv_rn(fmaf(-v, k, hi) + lo, k) + eps_lo;
    add2(v, low, eps_hi);
    const float vh = v + low, vl = low - (vh - v);
    const float r = rsqrtf(vh), p = r * r, pl = fmaf(r, r, -p), t = vh * p, tl = fmaf(vh, p, -t);
    const float e = ((1.f - t) - tl) - fmaf(vh, pl, vl * p);
    return fmaf(0.5f * e, r, r);
}

// The mean of squares, then the codes of bf16(x * r * w), r = 1 / sqrt(mean + eps) rounded to fp32, from the row held in
// registers as far as they go. The sum is kept in two floats (squares of bf16 are exact), so that r is that of the exact
// mean but for 2^-40, and the codes do not hang on the order of the sum. Where the squares pass fp32 or would vanish in it
// the sum is taken again in 64 bits.
// ALONE: a CTA has a row; else each warp has one, which waits for no other and holds it up to 3584 columns: of many short
// rows. Alone and by warps, us: 800 rows of 2048 6.2, 5.7, of 3584 6.7, 7.5; 1200 rows of 2048 7.8, 6.0, of 3584 8.6, 8.2, of
// 4096 (whose end a warp reads twice) 8.9, 9.3, of 5120 10.8, 12.3; 4000 rows of 1024 18.5, 8.7, of 3584 22.9, 16.5, of 4096
// 23.4, 19.4, of 5120 29.0, 24.7, of 8192 33.7, 43.3. The bounds are those of 3584 and 4096 columns: narrower rows would go by
// warps from 500 to 800 rows on, and wider ones of up to 5120 from some 2000 on.
constexpr int kManyRows = 1200, kShortRow = 4096;
template <bool ALONE>
__global__ void __launch_bounds__(kThreads) quantize_norm_kernel(const uint16_t* __restrict__ X, int64_t stride, uint8_t* __restrict__ Q,
                                                                 float* __restrict__ S, int64_t M, int KB, const uint16_t* __restrict__ W,
                                                                 double eps) {
    constexpr int LANES = ALONE ? kThreads : 32, HELD = ALONE ? 2 : 7;  // threads of a row, and of its words what each holds
    __shared__ float sh_hi[kThreads / 32], sh_lo[kThreads / 32];
    __shared__ double sh_d[kThreads / 32];
    const float eps_hi = (float)eps, eps_lo = (float)(eps - (double)eps_hi);
    pdl_launch_dependents();
    pdl_wait();
    const bool wide = ((uintptr_t)X & 31) == 0 && stride % 16 == 0;
    const int words = KB * 8, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, me = ALONE ? threadIdx.x : lane;  // words of 16 columns
    const int turns = (words + LANES - 1) / LANES;
    for (int64_t row = ALONE ? blockIdx.x : (int64_t)blockIdx.x * (kThreads / 32) + warp; row < M; row += ALONE ? gridDim.x : (int64_t)gridDim.x * (kThreads / 32)) {
        const uint16_t* x = X + row * stride;
        Words held[HELD];
        auto load = [&](int i) {
            Words v;
            v.a = v.b = make_uint4(0, 0, 0, 0);
            if (me + i * LANES < words) v = load16(x + (me + i * LANES) * 16, wide);
            return v;
        };
#pragma unroll
        for (int i = 0; i < HELD; ++i) held[i] = load(i);
        float hi4[4] = {0.f, 0.f, 0.f, 0.f}, lo4[4] = {0.f, 0.f, 0.f, 0.f};  // four sums, which do not wait for each other
        auto add = [&](const Words& v) {
            const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float a = bf16lo_to_f32(w[j]), b = bf16hi_to_f32(w[j]);
                add2(hi4[2 * j & 3], lo4[2 * j & 3], a * a);
                add2(hi4[2 * j + 1 & 3], lo4[2 * j + 1 & 3], b * b);
            }
        };
        if (ALONE) {
#pragma unroll
            for (int i = 0; i < HELD; ++i)
                if (i < turns) add(held[i]);
        } else {
            // Two sums of pairs, begun with a power of two of at least the largest square of what is held, so that a sum is never
            // less than what is added, and what it loses is x^2 - (s' - s), exactly: four instructions for two squares in
            // place of 16 (4000 x 3584: 17.8 -> 16.5 us; alone, with 48 registers, 300 rows took 5.4 us in place of 4.4).
            uint32_t largest = 0;
#pragma unroll
            for (int i = 0; i < HELD; ++i) largest = largest8(largest8(largest, held[i].a), held[i].b);
            const float above = 2.f * __uint_as_float(max(largest & 0x7F80u, largest >> 16 & 0x7F80u) << 16), start = above * above;
            float2 sums[2] = {make_float2(start, start), make_float2(start, start)}, lost[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 minus = make_float2(-1.f, -1.f), one = make_float2(1.f, 1.f);
#pragma unroll
            for (int i = 0; i < HELD; ++i)
                if (i < turns) {
                    const uint32_t w[8] = {held[i].a.x, held[i].a.y, held[i].a.z, held[i].a.w, held[i].b.x, held[i].b.y, held[i].b.z, held[i].b.w};
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 v = make_float2(bf16lo_to_f32(w[j]), bf16hi_to_f32(w[j])), before = sums[j & 1];
                        sums[j & 1] = fma2(v, v, before);
                        lost[j & 1] = fma2(fma2(v, v, fma2(sums[j & 1], minus, before)), one, lost[j & 1]);
                    }
                }
            // exact: the sums and their beginning are multiples of the sums' last places
            hi4[0] = sums[0].x - start, hi4[1] = sums[0].y - start, hi4[2] = sums[1].x - start, hi4[3] = sums[1].y - start;
            lo4[0] = lost[0].x, lo4[1] = lost[0].y, lo4[2] = lost[1].x, lo4[3] = lost[1].y;
        }
        for (int i = HELD; i < turns; ++i) add(load(i));
        float hi = hi4[0], lo = (lo4[0] + lo4[1]) + (lo4[2] + lo4[3]);
        add2(hi, lo, hi4[1]), add2(hi, lo, hi4[2]), add2(hi, lo, hi4[3]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float h = __shfl_xor_sync(0xFFFFFFFFu, hi, o), l = __shfl_xor_sync(0xFFFFFFFFu, lo, o);
            add2(hi, lo, h);
            lo += l;
        }
        if (ALONE) {
            if (lane == 0) sh_hi[warp] = hi, sh_lo[warp] = lo;
            __syncthreads();
            hi = lo = 0.f;
#pragma unroll
            for (int i = 0; i < kThreads / 32; ++i) add2(hi, lo, sh_hi[i]), lo += sh_lo[i];
        }
        float r;
        if (hi >= 0x1p-80f && hi <= 0x1p100f) {  // the same for all of the row's threads
            r = inverse_root(hi, lo, (float)(KB * 128.0), eps_hi, eps_lo);
        } else {
            double sum = 0.0;
            for (int i = 0; i < turns; ++i) {
                const Words v = load(i);
                const uint32_t w[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
                for (int j = 0; j < 8; ++j) {
                    const double a = (double)bf16lo_to_f32(w[j]), b = (double)bf16hi_to_f32(w[j]);
                    sum += a * a + b * b;
                }
            }
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            if (ALONE) {
                if (lane == 0) sh_d[warp] = sum;
                __syncthreads();
                sum = 0.0;
                for (int i = 0; i < kThreads / 32; ++i) sum += sh_d[i];
            }
            r = (float)(1.0 / sqrt(sum / (KB * 128.0) + eps));
        }
        // The words' steps side by side, so that their loads, shuffles and quotients wait together. A block's lanes go together.
        auto norm = [&](int i, Words& v) {
            const int at = me + i * LANES;
            if (at >= words) return;
            const uint4 *w = reinterpret_cast<const uint4*>(W + at * 16), wa = __ldg(w), wb = __ldg(w + 1);
            v.a = normed(v.a, r, wa), v.b = normed(v.b, r, wb);
        };
        auto put = [&](int i, const Words& v, uint32_t most) {
            const int at = me + i * LANES;
            if (at >= words) return;
            const float s = scale_of(most);
            put16(Q + (row * words + at) * 16, v, Divide(s));
            if ((lane & 7) == 0) S[row * KB + at / 8] = s;
        };
#pragma unroll
        for (int i = 0; i < HELD; ++i) norm(i, held[i]);
        uint32_t most[HELD];
#pragma unroll
        for (int i = 0; i < HELD; ++i) most[i] = largest_of_block(held[i]);
#pragma unroll
        for (int i = 0; i < HELD; ++i) put(i, held[i], most[i]);
        for (int i = HELD; i < turns; ++i) {
            Words v = load(i);
            norm(i, v);
            const uint32_t m = largest_of_block(v);
            put(i, v, m);
        }
        if (ALONE) __syncthreads();  // the sums are rewritten for the next row
    }
}

// Weights: a CTA takes a block of 128 x 128, held in its registers.
__global__ void __launch_bounds__(kThreads, 4) quantize_blocks_kernel(const uint16_t* __restrict__ W, uint8_t* __restrict__ Q, float* __restrict__ S,
                                                                      int64_t N, int KB, int64_t blocks) {
    __shared__ uint32_t sh_most[kThreads / 32];
    const int lane = threadIdx.x & 7, r0 = threadIdx.x >> 3;
    const int64_t K = (int64_t)KB * 128;
    const bool wide = ((uintptr_t)W & 31) == 0;
    for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
        const int64_t n0 = blk / KB * 128;
        const int64_t at = (int64_t)(blk % KB) * 128 + lane * 16;
        Words v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t n = n0 + r0 + 32 * i;
            v[i].a = v[i].b = make_uint4(0, 0, 0, 0);
            if (n < N) v[i] = load16(W + n * K + at, wide);
        }
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = largest8(largest8(m, v[i].a), v[i].b);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if ((threadIdx.x & 31) == 0) sh_most[threadIdx.x >> 5] = m;
        __syncthreads();
        m = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) m = __vmaxu2(m, sh_most[i]);
        const float s = scale_of(m);
        const Divide d(s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t n = n0 + r0 + 32 * i;
            if (n < N) put16(Q + n * K + at, v[i], d);
        }
        if (threadIdx.x == 0) S[blk] = s;
        __syncthreads();  // sh_most is rewritten for the next block
    }
}

__device__ __forceinline__ float4 values4(uint32_t q, float s) {
    uint32_t a, b;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)q));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(q >> 16)));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a)), y = __half22float2(*reinterpret_cast<const __half2*>(&b));
    return make_float4(x.x * s, x.y * s, y.x * s, y.y * s);
}

// Values of activations' codes, four a thread and turn: a warp's 32 are a block's.
__global__ void __launch_bounds__(kThreads) dequant_rows_kernel(const uint32_t* __restrict__ Q, const float* __restrict__ S, float4* __restrict__ out, int64_t words) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; i0 < words; i0 += kBatch * step) {
        uint32_t q[kBatch];
        float s[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int64_t i = i0 + j * step;
            q[j] = i < words ? Q[i] : 0, s[j] = i < words ? S[i / 32] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (i0 + j * step < words) out[i0 + j * step] = values4(q[j], s[j]);
    }
}

// Values of weights' codes: a CTA takes a block of 128 x 128, a warp a row of it at a time.
__global__ void __launch_bounds__(kThreads) dequant_blocks_kernel(const uint8_t* __restrict__ Q, const float* __restrict__ S, float* __restrict__ out,
                                                                  int64_t N, int KB, int64_t blocks) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t K = (int64_t)KB * 128;
    for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
        const int64_t n0 = blk / KB * 128, at = (blk % KB) * 128 + (threadIdx.x & 31) * 4;
        const float s = S[blk];
        for (int r = threadIdx.x >> 5; r < 128; r += kBatch * (kThreads / 32)) {
            uint32_t q[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int64_t n = n0 + r + j * (kThreads / 32);
                q[j] = n < N ? *reinterpret_cast<const uint32_t*>(Q + n * K + at) : 0;
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int64_t n = n0 + r + j * (kThreads / 32);
                if (n < N) *reinterpret_cast<float4*>(out + n * K + at) = values4(q[j], s);
            }
        }
    }
}

// As quantize.cu's: behind it a product on the same stream reads finished weights, which it does before its wait.
__global__ void fp8_weights_written_kernel() {}

template <typename... P, typename... A>
cudaError_t launch_pdl(void (*fn)(P...), int64_t grid, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attrs[1];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

int64_t waves(int64_t ctas, int per_sm) {
    const int64_t cap = (int64_t)device_sm_count() * per_sm;
    return ctas < cap ? ctas : cap;
}

}  // namespace

cudaError_t launch_quantize_fp8_rows(const uint16_t* X, int64_t stride, uint8_t* Q, float* S, int64_t M, int64_t K, const uint16_t* norm_w,
                                     double eps, cudaStream_t s) {
    const int KB = (int)(K / 128);
    if (norm_w && (M < kManyRows || K > kShortRow)) return launch_pdl(quantize_norm_kernel<true>, waves(M, 8), s, X, stride, Q, S, M, KB, norm_w, eps);
    if (norm_w) return launch_pdl(quantize_norm_kernel<false>, waves((M + kThreads / 32 - 1) / (kThreads / 32), 16), s, X, stride, Q, S, M, KB, norm_w, eps);
    return launch_pdl(quantize_rows_kernel, waves((M * KB + kThreads / 8 - 1) / (kThreads / 8), 16), s, X, stride, Q, S, M, KB);
}

cudaError_t launch_quantize_fp8_blocks(const uint16_t* W, uint8_t* Q, float* S, int64_t N, int64_t K, cudaStream_t s) {
    const int KB = (int)(K / 128);
    const int64_t blocks = (N + 127) / 128 * KB;
    count_launch();
    quantize_blocks_kernel<<<(unsigned)waves(blocks, 64), kThreads, 0, s>>>(W, Q, S, N, KB, blocks);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launch();
    fp8_weights_written_kernel<<<1, 32, 0, s>>>();
    return cudaGetLastError();
}

cudaError_t launch_dequant_fp8(const uint8_t* Q, const float* S, float* out, int64_t M, int64_t K, int rows_per_scale, cudaStream_t s) {
    const int KB = (int)(K / 128);
    if (rows_per_scale == 1) {
        const int64_t words = M * K / 4;
        return launch_pdl(dequant_rows_kernel, waves((words + kThreads - 1) / kThreads, 8), s, reinterpret_cast<const uint32_t*>(Q), S,
                          reinterpret_cast<float4*>(out), words);
    }
    const int64_t blocks = (M + 127) / 128 * KB;
    return launch_pdl(dequant_blocks_kernel, waves(blocks, 8), s, Q, S, out, M, KB, blocks);
}

}  // namespace mbw
