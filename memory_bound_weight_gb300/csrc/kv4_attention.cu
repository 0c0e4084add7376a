// kv4_attention.cu -- attention of one or several query tokens per request
// over the 4-bit paged cache (layout in kv4.cuh).
//
//   o_h = sum_t p_t v_t,  p = softmax over the keys t a query sees of
//   scale * q_h . k_t,  k_t = s n + m from codes n, likewise v_t
//
// Query i of a request with n queries and ctx cached tokens (its own among
// them) sits at position ctx - n + i and sees the keys t <= position, and with
// a window w those with t > position - w. A query that sees no key gets zeros
// and a log-sum-exp of minus infinity.
//
// One warp per (query, head): lanes share the dimensions, one pass over the
// keys with the running maximum and sum of the softmax.
#include <cuda_runtime.h>

#include <math_constants.h>

#include "internal.h"
#include "kv4.cuh"

namespace mbw {

namespace {

__device__ int g_kv4_attn_range;  // a page id, length or query offset was out of range

template <int D, int G>
__global__ void __launch_bounds__(128) kv4_attention_kernel(Kv4AttnArgs a) {
    constexpr int E = D / 32;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= (int64_t)a.T * a.q_heads) return;
    const int t = (int)(row / a.q_heads), h = (int)(row % a.q_heads), kvh = h / (a.q_heads / a.kv_heads);
    // the request that token t belongs to: the last one whose queries start at or before it
    int b = 0, first = 0, next = a.T;
    if (a.q_starts) {
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            (a.q_starts[mid] <= t ? lo : hi) = mid;
        }
        b = lo, first = a.q_starts[b], next = a.q_starts[b + 1];
    } else {
        const int n = a.T / a.B;
        b = t / n, first = b * n, next = first + n;
    }
    int ctx = a.ctx_lens[b];
    const int64_t cap = (int64_t)a.table_width * a.page_size;
    bool bad = ctx > cap;
    if (bad) ctx = (int)cap;
    const int pos = ctx - (next - t);
    const int begin = a.window ? max(0, pos - a.window + 1) : 0;
    float q[E], o[E], m = -CUDART_INF_F, l = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        q[i] = bf16lo_to_f32(a.q[t * a.q_stride + (int64_t)h * D + lane + 32 * i]) * a.scale;
        o[i] = 0.f;
    }
    if (t >= first && t < next)
        for (int key = begin; key <= pos; ++key) {
            int page = a.table[b * a.table_stride + key / a.page_size];
            if (page < 0 || page >= a.num_pages) bad = true, page = 0;
            const int in_page = key % a.page_size, tok = in_page & 15;
            const uint8_t* blk = a.pages + (((int64_t)page * a.kv_heads + kvh) * (a.page_size / 16) + in_page / 16) *
                                               (int64_t)kv4_block_bytes(D, G);
            float x = 0.f, v[E];
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const int d = lane + 32 * i;
                const uint32_t kw = *reinterpret_cast<const uint32_t*>(blk + kv4_k_word(D, tok, d / 8));
                const uint32_t vw = *reinterpret_cast<const uint32_t*>(blk + kv4_v_word(D, tok, d % 8, d / 64));
                const float2 mk = kv4_pair(*reinterpret_cast<const uint32_t*>(blk + kv4_meta(D, G, tok, d / G, 0)));
                const float2 mv = kv4_pair(*reinterpret_cast<const uint32_t*>(blk + kv4_meta(D, G, tok, d / G, 1)));
                x = fmaf(q[i], fmaf(mk.x, (float)((kw >> (4 * (d % 8))) & 15u), mk.y), x);
                v[i] = fmaf(mv.x, (float)((vw >> (4 * (d % 64 / 8))) & 15u), mv.y);
            }
            x = warp_sum(x);
            const float n = fmaxf(m, x), f = m == -CUDART_INF_F ? 0.f : expf(m - n), p = x == -CUDART_INF_F ? 0.f : expf(x - n);
            l = l * f + p;
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = o[i] * f + p * v[i];
            m = n;
        }
    const float r = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < E; ++i) store_out(a.out, t * a.out_stride + (int64_t)h * D + lane + 32 * i, o[i] * r, a.out_f32);
    if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -CUDART_INF_F : m + logf(l);
    if (bad && lane == 0) atomicExch(&g_kv4_attn_range, 1);
}

}  // namespace

size_t kv4_attention_workspace(int head_dim) {
    (void)head_dim;
    return 0;
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, cudaStream_t s) {
    const int64_t rows = (int64_t)a.T * a.q_heads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + 3) / 4), 1, 1);
    cfg.blockDim = dim3(128, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attrs[1];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    count_launch();
    if (a.group == 32)
        return cudaLaunchKernelEx(&cfg, a.head_dim == 64 ? kv4_attention_kernel<64, 32> : a.head_dim == 128
                                      ? kv4_attention_kernel<128, 32> : kv4_attention_kernel<256, 32>, a);
    return cudaLaunchKernelEx(&cfg, a.head_dim == 64 ? kv4_attention_kernel<64, 64> : a.head_dim == 128
                                  ? kv4_attention_kernel<128, 64> : kv4_attention_kernel<256, 64>, a);
}

int kv4_attn_take_range() {
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv4_attn_range, sizeof(int)) != cudaSuccess) return -1;
    if (v) cudaMemcpyToSymbol(g_kv4_attn_range, &z, sizeof(int));
    return v;
}

}  // namespace mbw
