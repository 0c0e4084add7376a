// logprobs.cu -- log probabilities of given tokens, the distribution's entropy
// and its most likely tokens, from the logits of the LM head product.
//
// With y = scale * x over the V logits of a row, M = max y at its lowest index
// i*, S' = sum over i != i* of e^(y_i - M), T = sum e^(y_i - M) (M - y_i):
//   log p_t = (y_t - M) - log1p(S'),   H = log1p(S') + T / (1 + S')
// Keeping the largest term out of the sum leaves log1p exact where one token
// has nearly all the probability, and both terms of H are positive: nothing
// cancels. Tokens are ordered by logit, then by the lower index; the rank is
// the target's place in that order, from 1. Logits of minus infinity have
// probability 0; a row of them alone has log probabilities of minus infinity
// and entropy 0. A NaN or plus infinity makes the row's numbers NaN.
//
// One CTA per row; one pass for the maximum, one for the sums and the rank,
// one per top token.
#include <cuda_runtime.h>

#include <math_constants.h>

#include "device.cuh"
#include "internal.h"

namespace mbw {

namespace {

__device__ int g_logprobs_range;  // a target was not below V

constexpr int kThreads = 256;

struct Cand {  // a logit and its index; better: larger, then the lower index
    float x;
    int i;
};
__device__ __forceinline__ bool better(float x, int i, float y, int j) { return x > y || (x == y && i < j); }

__device__ Cand block_best(Cand c, Cand* sm) {
    for (int o = 16; o > 0; o >>= 1) {
        const float x = __shfl_xor_sync(0xFFFFFFFFu, c.x, o);
        const int i = __shfl_xor_sync(0xFFFFFFFFu, c.i, o);
        if (better(x, i, c.x, c.i)) c.x = x, c.i = i;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = c;
    __syncthreads();
    c = sm[0];
    for (int w = 1; w < kThreads / 32; ++w)
        if (better(sm[w].x, sm[w].i, c.x, c.i)) c = sm[w];
    return c;
}

template <typename T>
__device__ T block_sum(T v, T* sm) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < kThreads / 32; ++w) v += sm[w];
    return v;
}

__device__ __forceinline__ float logit(const uint16_t* p, int64_t i) { return bf16lo_to_f32(p[i]); }
__device__ __forceinline__ float logit(const float* p, int64_t i) { return p[i]; }

template <typename T>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(LogprobArgs a) {
    __shared__ Cand sc[kThreads / 32];
    __shared__ float sf[kThreads / 32];
    __shared__ int si[kThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t r = blockIdx.x;
    const T* x = static_cast<const T*>(a.logits) + r * a.row_stride;
    const int V = (int)a.V;
    int t = a.targets ? a.targets[r] : -1;
    if (t >= V) {
        if (threadIdx.x == 0) atomicExch(&g_logprobs_range, 1);
        t = -1;
    }
    Cand best = {-CUDART_INF_F, 0x7FFFFFFF};
    float nan = 0.f;
    for (int i = threadIdx.x; i < V; i += kThreads) {
        const float v = logit(x, i);
        if (v != v) nan = v;
        if (better(v, i, best.x, best.i)) best = {v, i};
    }
    best = block_best(best, sc);
    nan = block_sum(nan, sf);
    const bool none = best.x == -CUDART_INF_F;
    const float top = best.x, xt = t >= 0 ? logit(x, t) : 0.f;
    float s = 0.f, e = 0.f;
    int before = 0;
    for (int i = threadIdx.x; i < V; i += kThreads) {
        const float v = logit(x, i);
        if (better(v, i, xt, t)) ++before;
        if (i == best.i || v == -CUDART_INF_F) continue;
        const float y = (v - top) * a.scale, p = expf(y);
        if (p > 0.f) s += p, e -= p * y;
    }
    s = block_sum(s, sf) + nan + (none ? 0.f : top - top);
    e = block_sum(e, sf);
    before = block_sum(before, si);
    const float lse = log1pf(s);
    if (threadIdx.x == 0) {
        if (a.logprob) a.logprob[r] = t < 0 ? 0.f : none ? -CUDART_INF_F + nan : (xt - top) * a.scale - lse;
        if (a.rank) a.rank[r] = t < 0 ? 0 : 1 + before;
        if (a.entropy) a.entropy[r] = none ? nan : lse + e / (1.f + s);
    }
    for (int k = 0; k < a.top_k; ++k) {
        if (k > 0) {  // the best one behind the last
            const Cand last = best;
            best = {-CUDART_INF_F, 0x7FFFFFFF};
            for (int i = threadIdx.x; i < V; i += kThreads) {
                const float v = logit(x, i);
                if (better(last.x, last.i, v, i) && better(v, i, best.x, best.i)) best = {v, i};
            }
            best = block_best(best, sc);
        }
        if (threadIdx.x == 0) {
            const bool no = best.x == -CUDART_INF_F;
            if (a.top_ids) a.top_ids[r * a.top_k + k] = no ? -1 : best.i;
            if (a.top_logprobs)
                a.top_logprobs[r * a.top_k + k] = no ? -CUDART_INF_F + nan : (best.x - top) * a.scale - lse;
        }
    }
}

}  // namespace

size_t token_logprobs_workspace() { return 0; }

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.M, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attrs[1];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, a.fp32 ? token_logprobs_kernel<float> : token_logprobs_kernel<uint16_t>, a);
}

int logprobs_take_range() {
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_logprobs_range, sizeof(int)) != cudaSuccess) return -1;
    if (v) cudaMemcpyToSymbol(g_logprobs_range, &z, sizeof(int));
    return v;
}

}  // namespace mbw
