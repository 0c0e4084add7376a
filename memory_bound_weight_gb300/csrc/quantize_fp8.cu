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
    __device__ __forceinline__ float operator()(float x) const {
        if (plain) {
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
__device__ __forceinline__ uint2 codes8(const uint4& v, const Divide& d) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = to_e4m3x2(d(bf16lo_to_f32(w[i])), d(bf16hi_to_f32(w[i])));
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
// The largest magnitude of 8 bf16 values, as bits in both halves; those of a NaN are the largest.
__device__ __forceinline__ uint32_t largest8(uint32_t m, const uint4& v) {
    return __vmaxu2(__vmaxu2(__vmaxu2(m, v.x & 0x7FFF7FFFu), __vmaxu2(v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu)), v.w & 0x7FFF7FFFu);
}
__device__ __forceinline__ float scale_of(uint32_t most) {
    return __fdiv_rn(__uint_as_float(max(most >> 16, most & 0xFFFFu) << 16), 448.0f);
}
// A block's 16 lanes of 8 columns each.
__device__ __forceinline__ uint32_t largest_of_block(uint32_t m) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return m;
}

constexpr int kThreads = 256;

// Rows as they are: a half-warp takes a block of 128 columns. Nothing of it is used twice, so that many small CTAs keep
// enough loads under way.
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const uint16_t* __restrict__ X, int64_t stride, uint8_t* __restrict__ Q,
                                                                 float* __restrict__ S, int64_t M, int KB) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t blocks = M * KB, step = (int64_t)gridDim.x * (kThreads / 16);
    const int lane = threadIdx.x & 15;
    // every lane of a warp goes round as often as the other block's
    for (int64_t b0 = (int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x / 32) * 2; b0 < blocks; b0 += step) {
        const int64_t b = b0 + ((threadIdx.x >> 4) & 1);
        const bool there = b < blocks;
        const int64_t row = there ? b / KB : 0;
        const int kb = there ? (int)(b - row * KB) : 0;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (there) v = *reinterpret_cast<const uint4*>(X + row * stride + kb * 128 + lane * 8);
        const float s = scale_of(largest_of_block(largest8(0, v)));
        if (there) {
            *reinterpret_cast<uint2*>(Q + b * 128 + lane * 8) = codes8(v, Divide(s));
            if (lane == 0) S[b] = s;
        }
    }
}

// The sum of a and b without loss, in two floats (Knuth's two-sum).
__device__ __forceinline__ void add2(float& hi, float& lo, float x) {
    const float s = hi + x, t = s - hi;
    lo += (hi - (s - t)) + (x - t);
    hi = s;
}

// A row's CTA: the mean of squares, then the codes of bf16(x * r * w), r = 1 / sqrt(mean + eps) rounded to fp32, from the
// row held in registers as far as they go. The sum is kept in two floats (squares of bf16 are exact), so that r is that of
// the exact mean but for 2^-40, and the codes do not hang on the order of the sum. Where the squares pass fp32 or would
// vanish in it the sum is taken again in 64 bits.
constexpr int kHeld = 4;  // words of 8 columns a thread
__global__ void __launch_bounds__(kThreads) quantize_norm_kernel(const uint16_t* __restrict__ X, int64_t stride, uint8_t* __restrict__ Q,
                                                                 float* __restrict__ S, int64_t M, int KB, const uint16_t* __restrict__ W,
                                                                 double eps) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ float sh_hi[kThreads / 32], sh_lo[kThreads / 32];
    __shared__ double sh_d[kThreads / 32];
    const int words = KB * 16, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int turns = (words + kThreads - 1) / kThreads;
    for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
        const uint4* x = reinterpret_cast<const uint4*>(X + row * stride);
        uint4 held[kHeld];
        float hi = 0.f, lo = 0.f;
        auto add = [&](const uint4& v) {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = bf16lo_to_f32(w[j]), b = bf16hi_to_f32(w[j]);
                add2(hi, lo, a * a);
                add2(hi, lo, b * b);
            }
        };
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int at = threadIdx.x + i * kThreads;
            held[i] = at < words ? x[at] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (i < turns) add(held[i]);
        for (int i = kHeld; i < turns; ++i) {
            const int at = threadIdx.x + i * kThreads;
            if (at < words) add(x[at]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float h = __shfl_xor_sync(0xFFFFFFFFu, hi, o), l = __shfl_xor_sync(0xFFFFFFFFu, lo, o);
            add2(hi, lo, h);
            lo += l;
        }
        if (lane == 0) sh_hi[warp] = hi, sh_lo[warp] = lo;
        __syncthreads();
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) sum += (double)sh_hi[i] + (double)sh_lo[i];
        if (!(sum >= 0x1p-80 && sum <= 0x1p125)) {  // the same for the whole CTA
            double d = 0.0;
            for (int at = threadIdx.x; at < words; at += kThreads) {
                const uint4 v = x[at];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                for (int j = 0; j < 4; ++j) {
                    const double a = (double)bf16lo_to_f32(w[j]), b = (double)bf16hi_to_f32(w[j]);
                    d += a * a + b * b;
                }
            }
            for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
            if (lane == 0) sh_d[warp] = d;
            __syncthreads();
            sum = 0.0;
            for (int i = 0; i < kThreads / 32; ++i) sum += sh_d[i];
        }
        const float r = (float)(1.0 / sqrt(sum / (double)(KB * 128) + eps));
        auto put = [&](int at, const uint4& raw) {  // a warp's lanes go together: words is a multiple of 16
            const bool there = at < words;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (there) v = norm_word(raw, r, W + at * 8);
            const float s = scale_of(largest_of_block(largest8(0, v)));
            if (there) {
                *reinterpret_cast<uint2*>(Q + row * words * 8 + at * 8) = codes8(v, Divide(s));
                if ((lane & 15) == 0) S[row * KB + at / 16] = s;
            }
        };
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (i < turns) put(threadIdx.x + i * kThreads, held[i]);
        for (int i = kHeld; i < turns; ++i) {
            const int at = threadIdx.x + i * kThreads;
            put(at, at < words ? x[at] : make_uint4(0, 0, 0, 0));
        }
        __syncthreads();  // the sums are rewritten for the next row
    }
}

// Weights: a CTA takes a block of 128 x 128, held in its registers.
__global__ void __launch_bounds__(kThreads) quantize_blocks_kernel(const uint16_t* __restrict__ W, uint8_t* __restrict__ Q, float* __restrict__ S,
                                                                   int64_t N, int KB, int64_t blocks) {
    __shared__ uint32_t sh_most[kThreads / 32];
    const int lane = threadIdx.x & 15, r0 = threadIdx.x >> 4;
    const int64_t K = (int64_t)KB * 128;
    for (int64_t blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
        const int64_t n0 = blk / KB * 128;
        const int64_t at = (int64_t)(blk % KB) * 128 + lane * 8;
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t n = n0 + r0 + 16 * i;
            v[i] = n < N ? *reinterpret_cast<const uint4*>(W + n * K + at) : make_uint4(0, 0, 0, 0);
        }
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = largest8(m, v[i]);
        m = largest_of_block(m);
        m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
        if ((threadIdx.x & 31) == 0) sh_most[threadIdx.x >> 5] = m;
        __syncthreads();
        m = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) m = __vmaxu2(m, sh_most[i]);
        const float s = scale_of(m);
        const Divide d(s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t n = n0 + r0 + 16 * i;
            if (n < N) *reinterpret_cast<uint2*>(Q + n * K + at) = codes8(v[i], d);
        }
        if (threadIdx.x == 0) S[blk] = s;
        __syncthreads();  // sh_most is rewritten for the next block
    }
}

// Values of codes, 8 a thread; rows_per_scale is 1 (activations) or 128 (weights).
__global__ void __launch_bounds__(kThreads) dequant_fp8_kernel(const uint8_t* __restrict__ Q, const float* __restrict__ S, float* __restrict__ out,
                                                               int64_t words, int KB, int rows_per_scale) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < words; i += step) {
        const int64_t row = i / (KB * 16);
        const int kb = (int)(i - row * (KB * 16)) / 16;
        const uint2 q = reinterpret_cast<const uint2*>(Q)[i];
        const float s = S[row / rows_per_scale * KB + kb];
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)((j < 2 ? q.x : q.y) >> (j & 1) * 16)));
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
            f[2 * j] = v.x * s, f[2 * j + 1] = v.y * s;
        }
        float4* to = reinterpret_cast<float4*>(out) + 2 * i;
        to[0] = make_float4(f[0], f[1], f[2], f[3]);
        to[1] = make_float4(f[4], f[5], f[6], f[7]);
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
    if (norm_w) return launch_pdl(quantize_norm_kernel, waves(M, 8), s, X, stride, Q, S, M, KB, norm_w, eps);
    return launch_pdl(quantize_rows_kernel, waves((M * KB + kThreads / 16 - 1) / (kThreads / 16), 32), s, X, stride, Q, S, M, KB);
}

cudaError_t launch_quantize_fp8_blocks(const uint16_t* W, uint8_t* Q, float* S, int64_t N, int64_t K, cudaStream_t s) {
    const int KB = (int)(K / 128);
    const int64_t blocks = (N + 127) / 128 * KB;
    count_launch();
    quantize_blocks_kernel<<<(unsigned)waves(blocks, 16), kThreads, 0, s>>>(W, Q, S, N, KB, blocks);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launch();
    fp8_weights_written_kernel<<<1, 32, 0, s>>>();
    return cudaGetLastError();
}

cudaError_t launch_dequant_fp8(const uint8_t* Q, const float* S, float* out, int64_t M, int64_t K, int rows_per_scale, cudaStream_t s) {
    const int64_t words = M * K / 8;
    return launch_pdl(dequant_fp8_kernel, waves((words + kThreads - 1) / kThreads, 32), s, Q, S, out, words, (int)(K / 128), rows_per_scale);
}

}  // namespace mbw
