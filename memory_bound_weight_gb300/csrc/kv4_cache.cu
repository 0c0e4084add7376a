// kv4_cache.cu -- writing the 4-bit paged key/value cache: kv4_append rotates
// queries and keys by their position, quantizes keys and values and stores
// them in their pages; kv4_gather reads values back.
//
// Rotation: of the first R dimensions of a head, (a, b) -> (a cos - b sin,
// b cos + a sin) for the pairs (i, i + R/2), or (2i, 2i + 1) interleaved, with
// cos and sin of the token's position from a table in fp32.
//
// Quantization, per token, head and group of G dimensions, of the bf16 values x
// (keys: the rotated ones, rounded to fp32 and then to bf16, as a bf16 cache
// would hold them): m = fp16(min x), s = fp16((max x - m) / 15),
// code = clamp(rint((x - m) / s), 0, 15), 0 where s = 0; each step one IEEE
// fp32 operation. With the rotation summed to about twice fp32's precision
// below, a code is a function of the inputs alone, not of the order of
// operations. A NaN or a value beyond fp16 (one that would round to its infinity)
// makes its whole group NaN when it is read, so it is not lost: a minimum beyond it
// by itself, a maximum through a scale that is none. Finite scales are then at most
// 8704, (65280 + 65280) / 15 with the largest bf16 values within fp16, which the
// attention kernels' operands rely on.
//
// What bounds it: for one token or some dozens the launch and its three dependent
// loads (2.4 and 1.8 us of append and gather, in a graph); for many, instructions at
// an occupancy that does not hide all of their latency: some 2400 for a token of 28 +
// 8 rows, issue slots 61% busy by 38% of the warps. 8192 tokens, 147 MB, take 32 us,
// 4.6 TB/s, and 8 us to read back.
#include <cuda_runtime.h>

#include <math_constants.h>

#include "internal.h"
#include "kv4.cuh"

namespace mbw {

namespace {

__device__ int g_kv4_cache_range;  // a slot or position was out of range

constexpr int kAppendThreads = 128;

// p1 - p2 of the exact products a * c and b * s (b * c and -a * s for the other
// component): both products split into their fp32 value and remainder, the
// values added with the remainder of that addition. About 2^-45 off before the
// final rounding, so it is the correctly rounded fp32 result but for inputs
// that a 64-bit sum cannot tell apart either.
__device__ __forceinline__ float rot_exact(float a, float c, float b, float s) {
    const float p = __fmul_rn(a, c), pe = __fmaf_rn(a, c, -p);
    const float r = __fmul_rn(b, s), re = __fmaf_rn(b, s, -r);
    const float h = __fadd_rn(p, r);
    const float z = __fsub_rn(h, p);
    const float e = __fadd_rn(__fsub_rn(p, __fsub_rn(h, z)), __fsub_rn(r, z));
    const float x = __fadd_rn(h, __fadd_rn(e, __fadd_rn(pe, re)));
    return x == x ? x : h;  // an infinity stays one: the remainders of infinite products are NaN
}

// The same for two values of a query, which are only rounded: a c + b s with the second product's remainder taken
// along (Kahan's form; Jeannerod, Louvet and Muller 2013: at most 1.5 ulp off), in pairs of fp32: five instructions
// for two values, where rot_exact takes twenty-six. NaN for an infinity, as its scores would be.
__device__ __forceinline__ void rot_near2(const float* a, const float* c, const float* b, const float* s, float* z) {
    asm("{.reg .b64 a, c, b, s, n, w, m, e;\n"
        " mov.b64 a, {%2, %3};\n mov.b64 c, {%4, %5};\n mov.b64 b, {%6, %7};\n mov.b64 s, {%8, %9};\n mov.b64 n, {%10, %11};\n"
        " mul.rn.f32x2 w, b, s;\n mul.rn.f32x2 m, b, n;\n"   // the product and its negative
        " fma.rn.f32x2 e, b, s, m;\n fma.rn.f32x2 w, a, c, w;\n add.rn.f32x2 w, w, e;\n mov.b64 {%0, %1}, w;}"
        : "=f"(z[0]), "=f"(z[1])
        : "f"(a[0]), "f"(a[1]), "f"(c[0]), "f"(c[1]), "f"(b[0]), "f"(b[1]), "f"(s[0]), "f"(s[1]), "f"(-s[0]), "f"(-s[1]));
}

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Page and place of a slot; 32-bit division where it does.
__device__ __forceinline__ int64_t page_of(int64_t slot, int page_size, int& place) {
    const int64_t page = slot >> 32 ? slot / page_size : (int64_t)((uint32_t)slot / (uint32_t)page_size);
    place = (int)(slot - page * page_size);
    return page;
}

__device__ __forceinline__ void unpack8(uint4 v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16lo_to_f32(w[i]);
        x[2 * i + 1] = bf16hi_to_f32(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes of the lane's 8 values (nibble i: value i) and its group's (scale,
// minimum); a group is G / 8 neighbouring lanes.
template <int G>
__device__ __forceinline__ uint32_t quantize8(const float* x, uint32_t& meta) {
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = min_nan(lo, x[i]);
        hi = max_nan(hi, x[i]);
    }
#pragma unroll
    for (int o = 1; o < G / 8; o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
        hi = max_nan(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
    }
    const __half mh = __float2half_rn(lo);
    const float m = __half2float(mh);
    const __half sh = __float2half_rn(hi < 65520.f ? __fdiv_rn(__fsub_rn(hi, m), 15.0f) : CUDART_NAN_F);
    const float s = __half2float(sh);
    meta = (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(mh) << 16);
    // (x - m) / s, correctly rounded, as Markstein (IBM J. Res. Dev. 1990) gets it from the correctly rounded
    // reciprocal: q = d r, q + (d - q s) r. One reciprocal for eight quotients. (Where s is infinite or no number, so
    // is the group's value, whatever its codes.)
    const float r = s != 0.f ? __frcp_rn(s) : 0.f;
    // Clamped before it is rounded, which gives the same; 1.5 2^23 more puts the rounded value into the low bits.
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float d = __fsub_rn(x[i], m), q = __fmul_rn(d, r);
        const float n = fminf(fmaxf(__fmaf_rn(__fmaf_rn(-q, s, d), r, q), 0.f), 15.f);
        codes |= (__float_as_uint(__fadd_rn(n, 12582912.f)) & 15u) << (4 * i);
    }
    return codes;
}

// Transpose of 8 x 8 nibbles over 8 neighbouring lanes: lane s gives nibbles
// g = 0 .. 7, lane g gets nibbles s = 0 .. 7. Three exchanges of halves.
__device__ __forceinline__ uint32_t transpose_nibbles(uint32_t v, int lane) {
    uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, v, 4);
    v = (lane & 4) ? ((v & 0xFFFF0000u) | (o >> 16)) : ((v & 0x0000FFFFu) | (o << 16));
    o = __shfl_xor_sync(0xFFFFFFFFu, v, 2);
    v = (lane & 2) ? ((v & 0xFF00FF00u) | ((o >> 8) & 0x00FF00FFu)) : ((v & 0x00FF00FFu) | ((o << 8) & 0xFF00FF00u));
    o = __shfl_xor_sync(0xFFFFFFFFu, v, 1);
    v = (lane & 1) ? ((v & 0xF0F0F0F0u) | ((o >> 4) & 0x0F0F0F0Fu)) : ((v & 0x0F0F0F0Fu) | ((o << 4) & 0xF0F0F0F0u));
    return v;
}

// One thread holds 8 dimensions of a head row, D / 8 neighbouring lanes a row;
// a CTA, or each of its warps, takes one token and `rows` of its Hq + 2 Hkv
// rows from row0 on.
template <int D, int G>
__global__ void __launch_bounds__(kAppendThreads) kv4_append_kernel(Kv4AppendArgs a, int rows, int tokens) {
    constexpr int LPR = D / 8;
    const int SLOTS = kAppendThreads / LPR / tokens;  // rows at a time
    pdl_launch_dependents();
    pdl_wait();
    const int tid = tokens > 1 ? threadIdx.x & 31 : threadIdx.x;  // among the token's threads
    const int64_t t = (int64_t)blockIdx.x * tokens + (tokens > 1 ? threadIdx.x >> 5 : 0);
    if (t >= a.T) return;  // a whole warp
    const int lane = threadIdx.x & 31, l = threadIdx.x % LPR, sub = tid / LPR;
    const int total = a.q_heads + 2 * a.kv_heads;
    const int row0 = blockIdx.y * rows, row1 = min(row0 + rows, total);

    // One row of each slot at a time, the next one's load under way: queries, then keys and values.
    const int q1 = min(row1, a.q_heads), kv0 = max(row0, a.q_heads) - a.q_heads, kv1 = row1 - a.q_heads;
    const uint16_t* q_at = a.q + t * a.q_stride + 8 * l;
    uint16_t* q_to = a.q_out + t * a.q_out_stride + 8 * l;
    const uint16_t* k_at = a.k + t * a.k_stride + 8 * l;  // row r < kv_heads, then the values' rows
    const uint16_t* v_at = a.v + t * a.v_stride - (int64_t)a.kv_heads * D + 8 * l;
    auto load_q = [&](int r) { return r < q1 ? *reinterpret_cast<const uint4*>(q_at + r * D) : make_uint4(0, 0, 0, 0); };
    auto load_kv = [&](int r) {
        return r < kv1 ? *reinterpret_cast<const uint4*>((r < a.kv_heads ? k_at : v_at) + r * D) : make_uint4(0, 0, 0, 0);
    };
    uint4 q_next = load_q(row0 + sub), kv_next = load_kv(kv0 + sub);

    int64_t slot = a.slots[t];
    if (slot >= a.num_slots) {
        if (tid == 0) atomicExch(&g_kv4_cache_range, 1);
        slot = -1;
    }
    // cos and sin of the lane's 8 dimensions; sin carries the sign of its term
    float c[8], s[8];
    int partner = l;  // lane of the row that holds the other component (half layout)
    bool rotated = false;
    if (a.cos_sin) {
        int64_t pos = a.positions[t];
        if (pos < 0 || pos >= a.max_pos) {
            if (tid == 0) atomicExch(&g_kv4_cache_range, 1);
            pos = 0;
        }
        const float* cs = a.cos_sin + pos * a.rotary;
        const int half = a.rotary / 2;
        rotated = 8 * l < a.rotary;
        if (rotated) {
            if (a.interleaved) {
                const float4 vc = *reinterpret_cast<const float4*>(cs + 4 * l);
                const float4 vs = *reinterpret_cast<const float4*>(cs + half + 4 * l);
                c[0] = c[1] = vc.x, c[2] = c[3] = vc.y, c[4] = c[5] = vc.z, c[6] = c[7] = vc.w;
                s[1] = vs.x, s[3] = vs.y, s[5] = vs.z, s[7] = vs.w;
                s[0] = -vs.x, s[2] = -vs.y, s[4] = -vs.z, s[6] = -vs.w;
            } else {
                const bool second = 8 * l >= half;
                const int i0 = second ? 8 * l - half : 8 * l;
                partner = second ? l - half / 8 : l + half / 8;
                const float sign = second ? 1.f : -1.f;
                const float4* vc = reinterpret_cast<const float4*>(cs + i0);
                const float4* vs = reinterpret_cast<const float4*>(cs + half + i0);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 x = vc[i], y = vs[i];
                    c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
                    s[4 * i] = sign * y.x, s[4 * i + 1] = sign * y.y;
                    s[4 * i + 2] = sign * y.z, s[4 * i + 3] = sign * y.w;
                }
            }
        }
    }
    int in_page;
    const int64_t page = page_of(slot < 0 ? 0 : slot, a.page_size, in_page);
    const int tok = in_page & 15, nblk = a.page_size / 16;

    const int from = lane - l % 32 + partner;  // LPR <= 32 and rows start at multiples of LPR
    // The row's other components of the lane's pairs; every lane of the warp takes part.
    auto partners = [&](uint4 raw, const float* x, float* y) {
        if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[i ^ 1];
        } else {
            raw.x = __shfl_sync(0xFFFFFFFFu, raw.x, from);
            raw.y = __shfl_sync(0xFFFFFFFFu, raw.y, from);
            raw.z = __shfl_sync(0xFFFFFFFFu, raw.z, from);
            raw.w = __shfl_sync(0xFFFFFFFFu, raw.w, from);
            unpack8(raw, y);
        }
    };
    for (int r0 = row0; r0 < q1; r0 += SLOTS) {  // the same for a token's threads: the shuffles need every lane
        const int r = r0 + sub;
        uint4 raw = q_next;
        q_next = load_q(r + SLOTS);
        if (a.cos_sin) {
            float x[8], y[8], z[8];
            unpack8(raw, x);
            partners(raw, x, y);
#pragma unroll
            for (int i = 0; i < 8; i += 2) rot_near2(x + i, c + i, y + i, s + i, z + i);
            if (rotated) raw = pack8(z);
        }
        if (r < q1) *reinterpret_cast<uint4*>(q_to + r * D) = raw;
    }
    for (int r0 = kv0; r0 < kv1; r0 += SLOTS) {
        const int r = r0 + sub;
        uint4 raw = kv_next;
        kv_next = load_kv(r + SLOTS);
        const bool key = r < a.kv_heads;
        float x[8];
        unpack8(raw, x);
        if (a.cos_sin && r0 < a.kv_heads) {
            float y[8], z[8];
            partners(raw, x, y);
            if (key && rotated) {
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] = rot_exact(x[i], c[i], y[i], s[i]);
                unpack8(pack8(z), x);
            }
        }
        uint32_t meta;
        const uint32_t codes = quantize8<G>(x, meta);
        const uint32_t turned = transpose_nibbles(codes, lane);
        if (r < kv1 && slot >= 0) {
            uint8_t* blk = a.pages + ((page * a.kv_heads + (key ? r : r - a.kv_heads)) * nblk + in_page / 16) *
                                         (int64_t)kv4_block_bytes(D, G);
            *reinterpret_cast<uint32_t*>(blk + (key ? kv4_k_word(D, tok, l) : kv4_v_word(D, tok, l % 8, l / 8))) = key ? codes : turned;
            if (l % (G / 8) == 0) *reinterpret_cast<uint32_t*>(blk + kv4_meta(D, G, tok, l / (G / 8), !key)) = meta;
        }
    }
}

// One thread per 8 dimensions of one (token, head): K from its word; V's words are read one a lane and transposed
// over 8 lanes, as they were written.
template <int D, int G>
__global__ void __launch_bounds__(256) kv4_gather_kernel(Kv4GatherArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int LPR = D / 8;
    const int64_t n = a.T * a.kv_heads * LPR;
    const int lane = threadIdx.x & 31;
    for (int64_t i0 = blockIdx.x * (int64_t)blockDim.x; i0 < n; i0 += (int64_t)gridDim.x * blockDim.x) {
        const int64_t i = i0 + threadIdx.x;
        const bool on = i < n;  // whole rows of lanes: n is a multiple of LPR
        const int l = threadIdx.x % LPR;
        const int64_t row = on ? i / LPR : 0;  // token * kv_heads + head
        const int64_t t = row >> 32 ? row / a.kv_heads : (int64_t)((uint32_t)row / (uint32_t)a.kv_heads);
        const int h = (int)(row - t * a.kv_heads);
        int64_t slot = a.slots[t];
        if (slot >= a.num_slots) {
            atomicExch(&g_kv4_cache_range, 1);
            slot = -1;
        }
        int in_page;
        const int64_t page = page_of(slot < 0 ? 0 : slot, a.page_size, in_page);  // a padding token reads slot 0 and drops it
        const int tok = in_page & 15;
        const uint8_t* blk = a.pages + ((page * a.kv_heads + h) * (a.page_size / 16) + in_page / 16) *
                                           (int64_t)kv4_block_bytes(D, G);
        const float2 mk = kv4_pair(*reinterpret_cast<const uint32_t*>(blk + kv4_meta(D, G, tok, 8 * l / G, 0)));
        const float2 mv = kv4_pair(*reinterpret_cast<const uint32_t*>(blk + kv4_meta(D, G, tok, 8 * l / G, 1)));
        const uint32_t kw = *reinterpret_cast<const uint32_t*>(blk + kv4_k_word(D, tok, l));
        const uint32_t vw = transpose_nibbles(*reinterpret_cast<const uint32_t*>(blk + kv4_v_word(D, tok, l % 8, l / 8)), lane);
        float k[8], v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            k[j] = slot < 0 ? 0.f : fmaf(mk.x, (float)((kw >> (4 * j)) & 15u), mk.y);
            v[j] = slot < 0 ? 0.f : fmaf(mv.x, (float)((vw >> (4 * j)) & 15u), mv.y);
        }
        if (on) {
            *reinterpret_cast<uint4*>(a.k + row * D + 8 * l) = pack8(k);
            *reinterpret_cast<uint4*>(a.v + row * D + 8 * l) = pack8(v);
        }
    }
}

template <typename F, typename A, typename... R>
cudaError_t launch_pdl(F* fn, dim3 grid, int threads, cudaStream_t s, const A& a, R... rest) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attrs[1];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, fn, a, rest...);
}

#define KV4_FOR(D, G, fn)                                      \
    ((G) == 32 ? ((D) == 64 ? fn<64, 32> : (D) == 128 ? fn<128, 32> : fn<256, 32>) \
               : ((D) == 64 ? fn<64, 64> : (D) == 128 ? fn<128, 64> : fn<256, 64>))

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t s) {
    // Few tokens: a CTA of 4 warps takes the rows it holds at a time, so that a token is done soonest. Many: one warp
    // takes a whole token, and what is done once per token and thread is done for all its rows (8192 tokens of 28 + 8
    // rows: 1030 instructions a warp and 4 warps a token become some 2400).
    const int total = a.q_heads + 2 * a.kv_heads;
    const int tokens = a.T >= (int64_t)device_sm_count() * 16 ? kAppendThreads / 32 : 1;
    const int slots = kAppendThreads / (a.head_dim / 8);
    int rows = slots;
    if (tokens > 1)
        rows = total;
    else
        while (rows < total && a.T * ((total + rows - 1) / rows) > (int64_t)device_sm_count() * 16) rows += slots;
    const int groups = (total + rows - 1) / rows;
    auto fn = KV4_FOR(a.head_dim, a.group, kv4_append_kernel);
    return launch_pdl(fn, dim3((unsigned)((a.T + tokens - 1) / tokens), (unsigned)groups), kAppendThreads, s, a, rows, tokens);
}

cudaError_t launch_kv4_gather(const Kv4GatherArgs& a, cudaStream_t s) {
    const int64_t n = a.T * a.kv_heads * (a.head_dim / 8);
    const int64_t blocks = (n + 255) / 256, cap = (int64_t)device_sm_count() * 16;
    auto fn = KV4_FOR(a.head_dim, a.group, kv4_gather_kernel);
    return launch_pdl(fn, dim3((unsigned)(blocks < cap ? blocks : cap)), 256, s, a);
}

int kv4_cache_take_range() {
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv4_cache_range, sizeof(int)) != cudaSuccess) return -1;
    if (v) cudaMemcpyToSymbol(g_kv4_cache_range, &z, sizeof(int));
    return v;
}

}  // namespace mbw
