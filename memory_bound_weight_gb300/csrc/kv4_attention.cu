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
// Mathematics. No value is dequantized. The codes enter m16n8k16 exactly, as
// fp16 subnormals: the bits 0 .. 3 of a halfword are the number n 2^-24, the
// bits 4 .. 7 alone n 2^-20, and the matrix unit multiplies subnormals exactly.
// Keys are the rows (a lane's A operand comes straight from the cache's bytes),
// the query rows that share the KV head (heads of the group x query tokens, 8
// per n-tile) the columns:
//   q . k = sum over groups of  s * sum q n  +  m * sum q
// q is scaled by a power of two per row so that its largest entry lies in
// [2^14, 2^15), and by another 2^-4 at the places of the 2^-20 codes: fp16 then
// holds bf16 entries exactly down to 2^-24 of the largest, smaller ones to
// within 2^-35 of it. The softmax weight p enters as w = fp16(4 p s), one per
// group:
//   sum p (s n + m) = [sum w n - 8 sum w] / 4 + sum p (m + 8 s)
// with the same rounded w in both sums, so that its rounding (2^-11) acts on
// the centred code n - 8 only; 8 sum w comes from a constant tile. p <= 1
// against the running maximum and s <= 8737 in fp16, so w cannot overflow; the
// factor 4 moves w's subnormal range to p s < 1.5e-5. Scores, maxima, sums and
// outputs are fp32.
//
// Unpacking is thus one AND per pair and a shift for every other pair. It runs
// on the ALU pipe at half rate, which bounded the forms before: with a shift
// per pair and an OR into 16 + n, and with HADD2 to n - 8.
//
// Work. A block of 16 tokens of one KV head is 2304 bytes in one piece (D =
// 128, G = 64), read once; each warp streams blocks of its own through a ring
// of shared memory (cp.async) with its own softmax state. The grid is one wave;
// the blocks of all (request, KV head, query tile) items are one line, cut
// into equal shares (each CTA derives the same cut from the lengths on the
// device), so ragged batches and single long contexts load every SM alike. An
// item cut between CTAs leaves its parts in the workspace, and the CTA that
// arrives last joins them in their order, so the result does not depend on who
// that is.
#include <cuda_runtime.h>

#include <math_constants.h>

#include <type_traits>

#include "internal.h"
#include "kv4.cuh"

namespace mbw {

namespace {

__device__ int g_kv4_attn_range;  // a page id, length or query offset was out of range

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8x8 transpose of 16-bit values over the warp: lane 4 i + j holds row i, columns 2j and 2j + 1.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Nibbles 0 and 4, 1 and 5, 2 and 6, 3 and 7 of a word as fp16 pairs: n 2^-24, n 2^-20, n 2^-24, n 2^-20.
__device__ __forceinline__ void unpack(uint32_t w, uint32_t* p) {
    const uint32_t v = w >> 8;
    p[0] = w & 0x000F000Fu;
    p[1] = w & 0x00F000F0u;
    p[2] = v & 0x000F000Fu;
    p[3] = v & 0x00F000F0u;
}

// The same less 8, n - 8 each: 1024 + n and 64 + n (an OR into the bits) less 1032 and 72.
__device__ __forceinline__ void unpack_centred(uint32_t w, uint32_t* p) {
    uint32_t x[4];
    unpack(w, x);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(x[i] | (i & 1 ? 0x54005400u : 0x64006400u)), "r"(i & 1 ? 0x54805480u : 0x64086408u));
}

// The NG (scale, minimum) pairs of a token.
template <int NG>
__device__ __forceinline__ void load_meta(const uint8_t* p, uint32_t* m) {
    if (NG == 1) m[0] = *reinterpret_cast<const uint32_t*>(p);
    if (NG == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        m[0] = v.x, m[1] = v.y;
    }
    if (NG >= 4)
#pragma unroll
        for (int i = 0; i < NG / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[i];
            m[4 * i] = v.x, m[4 * i + 1] = v.y, m[4 * i + 2] = v.z, m[4 * i + 3] = v.w;
        }
}

struct Request {
    int q0, nq, ctx, fb, units, qt;
    long long cost;  // units of all its items
};

template <int D, int G, int NT, int NW, int NB, int DEPTH>
struct Shape {
    static constexpr int NG = D / G, J = D / 32, BB = kv4_block_bytes(D, G), ROWS = 8 * NT;
    static constexpr int U = NW * NB;  // blocks of a unit: one step of every warp
    static constexpr int STAGE = NB * BB, RING = NW * DEPTH * STAGE;
    static constexpr int PAD = 68;  // floats of a merge row: 64 dimensions, 4 to spread the banks
    static constexpr int MERGE = NW * 8 * PAD * 4;
    static constexpr int QS = NT > 1 ? J * NT * 512 : 0;
    static constexpr int QSUM = NT > 1 ? (NG + 1) * ROWS * 4 : 0;
    static constexpr int SMEM = RING + MERGE + QS + QSUM + 2 * NW * ROWS * 4;
    static constexpr int MOST = RING / (4 * ROWS) - 2;  // most parts whose factors the drained ring holds
    static constexpr int PART = ROWS * (D + 2);  // floats of a part: rows of D, then M and L of each
};

template <int D, int G, int NT, int NW, int NB, int DEPTH, int OCC>
__global__ void __launch_bounds__(NW * 32, OCC) kv4_attention_kernel(Kv4AttnArgs a, int split) {
    using S = Shape<D, G, NT, NW, NB, DEPTH>;
    constexpr int NG = S::NG, J = S::J, BB = S::BB, ROWS = S::ROWS, THREADS = NW * 32, NV = D / 64;
    // V's codes as they are and 8 sum w from a constant tile; or, where several n-tiles share their unpacking, n - 8
    constexpr bool RAW = NT == 1;
    extern __shared__ __align__(16) uint8_t smem[];
    float* buf = reinterpret_cast<float*>(smem + S::RING);  // [NW][8][PAD]
    uint4* qs = reinterpret_cast<uint4*>(smem + S::RING + S::MERGE);
    float* qsums = reinterpret_cast<float*>(smem + S::RING + S::MERGE + S::QS);
    float* sm_m = reinterpret_cast<float*>(smem + S::RING + S::MERGE + S::QS + S::QSUM);
    float* sm_l = sm_m + NW * ROWS;
    __shared__ long long sh_scan[NW + 1];
    __shared__ long long sh_found[2];
    __shared__ int sh_last[2];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int gq = a.q_heads / a.kv_heads, bpp = a.page_size / 16;
    const float sl2 = fabsf(a.scale) * 1.44269504088896340736f;
    bool bad = false;

    pdl_launch_dependents();
    pdl_wait();

    auto request = [&](int b) {
        Request r;
        int q0, q1;
        if (a.q_starts) {
            const int s0 = a.q_starts[b], s1 = a.q_starts[b + 1];
            q0 = min(max(s0, 0), a.T);
            q1 = min(max(s1, q0), a.T);
            if (q0 != s0 || q1 != s1) bad = true;
        } else {
            const int n = a.T / a.B;
            q0 = b * n, q1 = q0 + n;
        }
        const long long cap = (long long)a.table_width * a.page_size;
        int ctx = max(a.ctx_lens[b], 0);
        if (ctx > cap) bad = true, ctx = (int)cap;
        r.q0 = q0, r.nq = q1 - q0, r.ctx = ctx;
        r.fb = a.window ? max(0, ctx - r.nq - a.window + 1) / 16 : 0;
        const int nblk = (ctx + 15) / 16 - r.fb;
        r.units = max(1, (nblk + S::U - 1) / S::U);
        r.qt = (int)(((long long)r.nq * gq + ROWS - 1) / ROWS);
        r.cost = (long long)r.units * r.qt * a.kv_heads;
        return r;
    };
    // exclusive prefix of v over the CTA's threads, and the total
    auto scan = [&](long long v, long long& total) {
        long long x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) sh_scan[warp] = x;
        __syncthreads();
        long long before = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < warp) before += sh_scan[w];
            total += sh_scan[w];
        }
        return before + x - v;
    };

    // ---- this CTA's share [u0, u1) of the units of all items ----
    long long W = 0, mine = 0, excl = 0;
    for (int base = 0; base < a.B; base += THREADS) {
        mine = base + tid < a.B ? request(base + tid).cost : 0;
        long long total;
        excl = scan(mine, total);
        W += total;
    }
    const long long C = W < gridDim.x ? W : gridDim.x;
    if ((long long)blockIdx.x >= C) {
        if (bad) atomicExch(&g_kv4_attn_range, 1);
        return;
    }
    const long long u0 = (long long)blockIdx.x * W / C, u1 = ((long long)blockIdx.x + 1) * W / C;
    {
        long long run = 0;
        for (int base = 0; base < a.B; base += THREADS) {
            long long total = W;
            if (a.B > THREADS) {
                mine = base + tid < a.B ? request(base + tid).cost : 0;
                excl = scan(mine, total);
            }
            if (u0 >= run + excl && u0 < run + excl + mine) sh_found[0] = base + tid, sh_found[1] = run + excl;
            run += total;
            if (run > u0) break;  // the same for every thread
        }
        __syncthreads();
    }
    int b = (int)sh_found[0];
    long long start = sh_found[1];  // units before request b
    Request rq = request(b);

    // ---- segments: what this CTA takes of one item ----
    struct Segment {
        int q0, nq, ctx, h, f0;   // the request's queries and length, KV head, first query row of the tile
        int bs, be, nsteps;       // blocks, and this warp's steps over them
        int pos_lo, pos_hi;       // positions of the tile's first and last query
        bool whole;               // the item is this CTA's alone
        long long iu0;            // the item's first unit
        int units;
        const int32_t* table;
    };
    long long u = u0;
    auto next_segment = [&](Segment& sg) {
        while (u < u1) {
            while (u >= start + rq.cost) {
                start += rq.cost;
                rq = request(++b);
            }
            const long long item = (u - start) / rq.units, iu0 = start + item * rq.units;
            const int s0 = (int)(u - iu0);
            int s1 = rq.units;
            if (split) {
                if (u1 - iu0 < s1) s1 = (int)(u1 - iu0);
            } else if (s0 != 0) {  // its first unit is another CTA's, and so is the item
                u = iu0 + rq.units;
                continue;
            }
            u = iu0 + s1;
            sg.q0 = rq.q0, sg.nq = rq.nq, sg.ctx = rq.ctx, sg.iu0 = iu0, sg.units = rq.units;
            sg.h = (int)(item / rq.qt), sg.f0 = (int)(item % rq.qt) * ROWS;
            sg.whole = s0 == 0 && s1 == rq.units;
            const int i_last = min(rq.nq - 1, (sg.f0 + ROWS - 1) / gq);
            sg.pos_lo = rq.ctx - rq.nq + sg.f0 / gq, sg.pos_hi = rq.ctx - rq.nq + i_last;
            const int k_lo = a.window ? max(0, sg.pos_lo - a.window + 1) : 0;
            sg.bs = max(rq.fb + s0 * S::U, k_lo / 16);
            sg.be = max(sg.bs, min(rq.fb + s1 * S::U, (sg.pos_hi + 16) / 16));
            sg.nsteps = sg.be > sg.bs + warp * NB ? (sg.be - sg.bs - warp * NB + S::U - 1) / S::U : 0;
            sg.table = a.table + (long long)b * a.table_stride;
            return true;
        }
        return false;
    };

    // ---- copies: the lane's block offset among the 32 of the steps win * 32 / NB ..., -1 past the end ----
    constexpr int SPW = 32 / NB;
    auto offsets = [&](const Segment& sg, int win) -> long long {
        const int k = win * SPW + lane / NB;
        const int blk = sg.bs + (k * NW + warp) * NB + lane % NB;
        if (k >= sg.nsteps || blk >= sg.be) return -1;
        const int p = blk / bpp;
        int page = sg.table[p];
        if (page < 0 || page >= a.num_pages) bad = true, page = 0;
        return (((long long)page * a.kv_heads + sg.h) * bpp + (blk - p * bpp)) * BB;
    };
    const uint8_t* my_ring = smem + warp * DEPTH * S::STAGE;
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(my_ring) + lane * 16;
    const uint8_t* pages = a.pages + lane * 16;
    long long off = -1, off_next = -1;
    auto issue = [&](const Segment& sg, int k) {
        if (k < sg.nsteps) {
            if (k % SPW == 0) {
                off = k == 0 ? offsets(sg, 0) : off_next;
                if (k + SPW < sg.nsteps) off_next = offsets(sg, k / SPW + 1);
            }
#pragma unroll
            for (int sub = 0; sub < NB; ++sub) {
                const long long o = __shfl_sync(0xFFFFFFFFu, off, (k % SPW) * NB + sub);
                if (o >= 0) {
                    const uint32_t dst = ring_at + (uint32_t)((k % DEPTH) * S::STAGE + sub * BB);
                    const uint8_t* src = pages + o;
#pragma unroll
                    for (int i = 0; i < (BB + 511) / 512; ++i)
                        if (i < BB / 512 || lane < BB % 512 / 16)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + i * 512), "l"(src + i * 512) : "memory");
                }
            }
        }
        cp_async_commit();
    };

    struct Pending {  // an item of which this CTA wrote a part
        int q0, nq, h, f0, parts0, parts;
    };
    __shared__ Pending pend[2];  // the one that begins before this CTA's share, the one that begins within
    if (tid < 2) pend[tid].parts = 0;

    // dimensions d .. d + 3 of query row f: the sum of the weighted values, the maximum and the sum of the weights
    auto store = [&](int q0, int h, int f, int d, float4 s, float m, float l) {
        const int qi = f / gq;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const long long row = q0 + qi;
        const int head = h * gq + f - qi * gq;
        const long long at = row * a.out_stride + (long long)head * D + d;
        if (a.out_f32) {
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
        } else {
            const __nv_bfloat162 p = __floats2bfloat162_rn(s.x * inv, s.y * inv);
            const __nv_bfloat162 q = __floats2bfloat162_rn(s.z * inv, s.w * inv);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
        }
        if (a.lse && d == 0)
            a.lse[row * a.q_heads + head] = l == 0.f ? -CUDART_INF_F : (m + log2f(l) - 2.f) * 0.69314718055994530942f;
    };

    Segment sg;
    bool more = next_segment(sg);
    if (more)
        for (int k = 0; k < DEPTH - 1; ++k) issue(sg, k);

    while (more) {
        const int f0 = sg.f0, nsteps = sg.nsteps, bs = sg.bs, be = sg.be, h = sg.h;
        // ---- the queries as B operands, and their sums over each group ----
        // word pairs of dimensions 32 j + 8 c + (0, 4), (1, 5), (2, 6), (3, 7) of row 8 nt + g
        uint32_t qf[NT == 1 ? J : 1][4];
        float qsum[NT == 1 ? NG : 1][2], qscale[2];
        int posc[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) posc[nt][e] = sg.ctx - sg.nq + min(sg.nq - 1, (f0 + 8 * nt + 2 * c + e) / gq);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (NT > 1 && warp != nt % NW) continue;
            const int f = f0 + 8 * nt + g, i = f / gq;
            const uint16_t* src = a.q + (long long)(sg.q0 + i) * a.q_stride + (long long)(h * gq + f - i * gq) * D + 8 * c;
            float sum[NG];
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) sum[gr] = 0.f;
            uint4 v[J];
            uint32_t big = 0;  // the largest |q| of the row, as bf16 bits
#pragma unroll
            for (int j = 0; j < J; ++j) {
                v[j] = make_uint4(0, 0, 0, 0);
                if (i < sg.nq) v[j] = *reinterpret_cast<const uint4*>(src + 32 * j);
                big = __vmaxu2(__vmaxu2(big, v[j].x & 0x7FFF7FFFu), __vmaxu2(v[j].y & 0x7FFF7FFFu,
                               __vmaxu2(v[j].z & 0x7FFF7FFFu, v[j].w & 0x7FFF7FFFu)));
            }
            big = __vmaxu2(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
            big = __vmaxu2(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
            const uint32_t ex = max(max(big >> 16, big & 0xFFFFu) >> 7, 20u);  // its biased exponent
            // to 2^14, and back with the codes' 2^24 (in two factors: either is a normal number)
            const float up = copysignf(__uint_as_float((268u - ex) << 23), a.scale), down = __uint_as_float((ex - 14u) << 23) * (sl2 * 16777216.f);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const uint32_t x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
                uint32_t hw[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const float q0 = bf16lo_to_f32(x[d]) * up, q1 = bf16hi_to_f32(x[d]) * up;
                    sum[j * 32 / G] += q0 + q1;
                    const __half2 hh = __floats2half2_rn(q0, q1 * 0.0625f);  // odd places hold n 2^-20
                    hw[d] = *reinterpret_cast<const uint32_t*>(&hh);
                }
                const uint4 w = make_uint4(__byte_perm(hw[0], hw[2], 0x5410), __byte_perm(hw[0], hw[2], 0x7632),
                                           __byte_perm(hw[1], hw[3], 0x5410), __byte_perm(hw[1], hw[3], 0x7632));
                if (NT == 1)
                    qf[j][0] = w.x, qf[j][1] = w.y, qf[j][2] = w.z, qf[j][3] = w.w;
                else
                    qs[(j * NT + nt) * 32 + lane] = w;
            }
            if (NT == 1) {
                qscale[0] = __shfl_sync(0xFFFFFFFFu, down, 8 * c);
                qscale[1] = __shfl_sync(0xFFFFFFFFu, down, 8 * c + 4);
            } else if (c == 0) {
                qsums[NG * ROWS + 8 * nt + g] = down;
            }
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                sum[gr] += __shfl_xor_sync(0xFFFFFFFFu, sum[gr], 1);
                sum[gr] = (sum[gr] + __shfl_xor_sync(0xFFFFFFFFu, sum[gr], 2)) * 0x1p-24f;
                if (NT == 1) {
                    qsum[gr][0] = __shfl_sync(0xFFFFFFFFu, sum[gr], 8 * c);
                    qsum[gr][1] = __shfl_sync(0xFFFFFFFFu, sum[gr], 8 * c + 4);
                } else if (c == 0) {
                    qsums[gr * ROWS + 8 * nt + g] = sum[gr];
                }
            }
        }
        if (NT > 1) __syncthreads();

        float o[NT][D / 16][4], z[RAW ? NG : 1][4], r[NT][NG][2], M[NT][2], L[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                r[nt][gr][0] = r[nt][gr][1] = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) z[RAW ? gr : 0][e] = 0.f;
            }
            M[nt][0] = M[nt][1] = -CUDART_INF_F;
            L[nt][0] = L[nt][1] = 0.f;
        }

        // scores are kept as s and m give them; col_scale (>= 0) takes those of a column to powers of two
        auto col_scale = [&](int nt, int e) { return NT == 1 ? qscale[e] : qsums[NG * ROWS + 8 * nt + 2 * c + e]; };

        for (int k = 0; k < nsteps; ++k) {
            cp_async_wait<DEPTH - 2>();
            __syncwarp();  // the step's copies of every lane are there, and step k - 1 is read
            issue(sg, k + DEPTH - 1);
            const uint8_t* stage = my_ring + (k % DEPTH) * NB * BB;
            const int blk0 = bs + (k * NW + warp) * NB;

            // scores y of NB blocks: rows g and g + 8 (tokens), columns 2c and 2c + 1 of each n-tile
            float y[NB][NT][4];
#pragma unroll
            for (int sub = 0; sub < NB; ++sub) {
                const uint8_t* blk = stage + sub * BB;
                uint32_t km[2][NG];
                load_meta<NG>(blk + kv4_meta(D, G, g, 0, 0), km[0]);
                load_meta<NG>(blk + kv4_meta(D, G, g + 8, 0, 0), km[1]);
                uint32_t kw[2][J];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (D == 64) {
                        const uint2 v = *reinterpret_cast<const uint2*>(blk + (g + 8 * t) * 32 + c * 8);
                        kw[t][0] = v.x, kw[t][1] = v.y;
                    } else {
#pragma unroll
                        for (int p = 0; p < D / 128; ++p) {
                            const uint4 v = *reinterpret_cast<const uint4*>(blk + p * 1024 + (g + 8 * t) * 64 + c * 16);
                            kw[t][4 * p] = v.x, kw[t][4 * p + 1] = v.y, kw[t][4 * p + 2] = v.z, kw[t][4 * p + 3] = v.w;
                        }
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) y[sub][nt][0] = y[sub][nt][1] = y[sub][nt][2] = y[sub][nt][3] = 0.f;
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                    float acc[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
                    for (int j = gr * G / 32; j < (gr + 1) * G / 32; ++j) {
                        uint32_t n0[4], n1[4];
                        unpack(kw[0][j], n0);
                        unpack(kw[1][j], n1);
                        const uint32_t a0[4] = {n0[0], n1[0], n0[1], n1[1]}, a1[4] = {n0[2], n1[2], n0[3], n1[3]};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            uint4 q;
                            if (NT == 1)
                                q = make_uint4(qf[j][0], qf[j][1], qf[j][2], qf[j][3]);
                            else
                                q = qs[(j * NT + nt) * 32 + lane];
                            mma_f16(acc[nt], a0, q.x, q.y);
                            mma_f16(acc[nt], a1, q.z, q.w);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const float2 sm = kv4_pair(km[t][gr]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float2 qq;
                            if (NT == 1)
                                qq = make_float2(qsum[gr][0], qsum[gr][1]);
                            else
                                qq = *reinterpret_cast<const float2*>(qsums + gr * ROWS + 8 * nt + 2 * c);
                            y[sub][nt][2 * t] = fmaf(sm.y, qq.x, fmaf(sm.x, acc[nt][2 * t], y[sub][nt][2 * t]));
                            y[sub][nt][2 * t + 1] = fmaf(sm.y, qq.y, fmaf(sm.x, acc[nt][2 * t + 1], y[sub][nt][2 * t + 1]));
                        }
                    }
                }
            }
            // Some key of this step may be unseen by some row, or lie past the segment.
            const bool edge = blk0 + NB > be || (blk0 + NB) * 16 - 1 > sg.pos_lo ||
                              (a.window && blk0 * 16 <= sg.pos_hi - a.window);
            uint32_t seen = 0xFFFFFFFFu;
            static_assert(NB * NT * 4 <= 32, "one bit per score");
            if (edge) {
#pragma unroll
                for (int sub = 0; sub < NB; ++sub)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int t = (blk0 + sub) * 16 + g + 8 * (e >> 1), p = posc[nt][e & 1];
                            if (blk0 + sub >= be || t > p || (a.window && t <= p - a.window)) {
                                y[sub][nt][e] = -CUDART_INF_F;
                                seen &= ~(1u << ((sub * NT + nt) * 4 + e));
                            }
                        }
            }
            bool raise = false;
#pragma unroll
            for (int sub = 0; sub < NB; ++sub)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) raise |= y[sub][nt][e] > M[nt][e & 1];
            if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = M[nt][e];
#pragma unroll
                        for (int sub = 0; sub < NB; ++sub) m = fmaxf(m, fmaxf(y[sub][nt][e], y[sub][nt][2 + e]));
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, w));
                        const float f = M[nt][e] == -CUDART_INF_F ? 0.f : exp2_fast((M[nt][e] - m) * col_scale(nt, e));
                        M[nt][e] = m;
                        L[nt][e] *= f;
#pragma unroll
                        for (int gr = 0; gr < NG; ++gr) {
                            r[nt][gr][e] *= f;
                            if (RAW) z[gr][e] *= f, z[gr][2 + e] *= f;
                        }
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) o[nt][i][e] *= f, o[nt][i][2 + e] *= f;
                    }
            }
            // weights 4 p
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f = col_scale(nt, e), m = M[nt][e] == -CUDART_INF_F ? 0.f : fmaf(-M[nt][e], f, 2.f);
#pragma unroll
                    for (int sub = 0; sub < NB; ++sub) {
                        y[sub][nt][e] = exp2_fast(fmaf(y[sub][nt][e], f, m));
                        y[sub][nt][2 + e] = exp2_fast(fmaf(y[sub][nt][2 + e], f, m));
                        L[nt][e] += y[sub][nt][e] + y[sub][nt][2 + e];
                    }
                }
            auto values = [&](auto edge_step) {
                constexpr bool EDGE = decltype(edge_step)::value;
#pragma unroll
                for (int sub = 0; sub < NB; ++sub) {
                    const uint8_t* blk = stage + sub * BB;
                    uint32_t vm[2][NG];
                    load_meta<NG>(blk + kv4_meta(D, G, g, 0, 1), vm[0]);
                    load_meta<NG>(blk + kv4_meta(D, G, g + 8, 0, 1), vm[1]);
                    uint32_t vw[4 * NV];  // word (h, b, w)
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const uint4 v = *reinterpret_cast<const uint4*>(blk + 8 * D + i * 512 + lane * 16);
                        vw[4 * i] = v.x, vw[4 * i + 1] = v.y, vw[4 * i + 2] = v.z, vw[4 * i + 3] = v.w;
                    }
                    uint32_t pb[NT][NG][2];  // w of tokens (2c, 2c + 1) and (2c + 8, 2c + 9), row g: B operands
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const float2 sm = kv4_pair(vm[t][gr]);
                            const float mid = fmaf(8.f, sm.x, sm.y);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float w0 = y[sub][nt][2 * t] * sm.x, w1 = y[sub][nt][2 * t + 1] * sm.x;
                                if (EDGE) {  // what is unseen may be no number
                                    const uint32_t on = seen >> ((sub * NT + nt) * 4 + 2 * t);
                                    if (on & 1) r[nt][gr][0] = fmaf(y[sub][nt][2 * t], mid, r[nt][gr][0]); else w0 = 0.f;
                                    if (on & 2) r[nt][gr][1] = fmaf(y[sub][nt][2 * t + 1], mid, r[nt][gr][1]); else w1 = 0.f;
                                } else {
                                    r[nt][gr][0] = fmaf(y[sub][nt][2 * t], mid, r[nt][gr][0]);
                                    r[nt][gr][1] = fmaf(y[sub][nt][2 * t + 1], mid, r[nt][gr][1]);
                                }
                                const __half2 hw = __floats2half2_rn(w0, w1);
                                pb[nt][gr][t] = transpose8x8(*reinterpret_cast<const uint32_t*>(&hw));
                            }
                        }
                    if (RAW) {
                        const uint32_t k8[4] = {0x00080008u, 0x00800080u, 0x00080008u, 0x00800080u};  // 8 as the codes' rows hold it
#pragma unroll
                        for (int gr = 0; gr < NG; ++gr) mma_f16(z[gr], k8, pb[0][gr][0], pb[0][gr][1]);
                    }
#pragma unroll
                    for (int w = 0; w < NV; ++w) {
                        // halfword pairs of tokens (2c, 2c + 1), lower and upper slots, for h = 0 and 1
                        uint32_t lo[2], hi[2];
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            lo[t] = __byte_perm(vw[2 * t * NV + w], vw[(2 * t + 1) * NV + w], 0x5410);
                            hi[t] = __byte_perm(vw[2 * t * NV + w], vw[(2 * t + 1) * NV + w], 0x7632);
                        }
                        uint32_t l0[4], l1[4], h0[4], h1[4];
                        if (RAW) {
                            unpack(lo[0], l0), unpack(lo[1], l1), unpack(hi[0], h0), unpack(hi[1], h1);
                        } else {
                            unpack_centred(lo[0], l0), unpack_centred(lo[1], l1);
                            unpack_centred(hi[0], h0), unpack_centred(hi[1], h1);
                        }
                        const uint32_t f[4][4] = {{l0[0], l0[1], l1[0], l1[1]}, {l0[2], l0[3], l1[2], l1[3]},
                                                  {h0[0], h0[1], h1[0], h1[1]}, {h0[2], h0[3], h1[2], h1[3]}};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                constexpr int T0 = 4;
                                const int gr = (T0 * w + i) * 16 / G;
                                mma_f16(o[nt][T0 * w + i], f[i], pb[nt][gr][0], pb[nt][gr][1]);
                            }
                    }
                }
            };
            if (edge)
                values(std::true_type());
            else
                values(std::false_type());
        }
        cp_async_wait<0>();

        // the next segment's first copies run while this one's warps are joined
        const Segment done = sg;
        more = next_segment(sg);
        if (more)
            for (int k = 0; k < DEPTH - 1; ++k) issue(sg, k);

        // ---- join the warps, then write the item or this CTA's part of it ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) {
                    L[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, L[nt][e], w);
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) r[nt][gr][e] += __shfl_xor_sync(0xFFFFFFFFu, r[nt][gr][e], w);
                }
                if (g == 0) {
                    sm_m[warp * ROWS + 8 * nt + 2 * c + e] = M[nt][e] * col_scale(nt, e);
                    sm_l[warp * ROWS + 8 * nt + 2 * c + e] = L[nt][e];
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const int gr = i * 16 / G;
                    if (RAW) {
                        o[nt][i][e] = fmaf(o[nt][i][e] - z[gr][e], 0x1p24f, r[nt][gr][e]);
                        o[nt][i][2 + e] = fmaf(o[nt][i][2 + e] - z[gr][2 + e], 0x1p20f, r[nt][gr][e]);
                    } else {
                        o[nt][i][e] += r[nt][gr][e];
                        o[nt][i][2 + e] += r[nt][gr][e];
                    }
                }
            }
        float* part = nullptr;
        if (!done.whole) {
            const bool begins = done.iu0 >= u0;  // the item's other parts are later CTAs'
            part = static_cast<float*>(a.workspace) + 1024 + (2 * (long long)blockIdx.x + begins) * S::PART;
            if (tid == 0) {
                Pending& p = pend[begins];
                p.q0 = done.q0, p.nq = done.nq, p.h = h, p.f0 = f0;
                p.parts0 = (int)(((done.iu0 + 1) * C - 1) / W);
                p.parts = (int)(((done.iu0 + done.units) * C - 1) / W) - p.parts0 + 1;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int hd = 0; hd < D / 64; ++hd) {
                if (nt + hd > 0) __syncthreads();  // the buffer is read
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        buf[(warp * 8 + 2 * c + (e & 1)) * S::PAD + 16 * i + g + 8 * (e >> 1)] = o[nt][4 * hd + i][e];
                __syncthreads();
                for (int i = tid; i < 128; i += THREADS) {
                    const int row = i / 16, d = i % 16 * 4, f = f0 + 8 * nt + row;
                    if (f >= done.nq * gq) continue;
                    float m = -CUDART_INF_F, l = 0.f;
#pragma unroll
                    for (int w = 0; w < NW; ++w) m = fmaxf(m, sm_m[w * ROWS + 8 * nt + row]);
                    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        const float mw = sm_m[w * ROWS + 8 * nt + row], x = mw == -CUDART_INF_F ? 0.f : exp2_fast(mw - m);
                        const float4 v = *reinterpret_cast<const float4*>(buf + (w * 8 + row) * S::PAD + d);
                        l = fmaf(x, sm_l[w * ROWS + 8 * nt + row], l);
                        s.x = fmaf(x, v.x, s.x), s.y = fmaf(x, v.y, s.y), s.z = fmaf(x, v.z, s.z), s.w = fmaf(x, v.w, s.w);
                    }
                    if (done.whole) {
                        store(done.q0, h, f, 64 * hd + d, s, m, l);
                    } else {
                        *reinterpret_cast<float4*>(part + (8 * nt + row) * D + 64 * hd + d) = s;
                        if (hd == 0 && d == 0) {
                            part[ROWS * D + 8 * nt + row] = m;
                            part[ROWS * D + ROWS + 8 * nt + row] = l;
                        }
                    }
                }
            }
        __syncthreads();  // the buffers are free for the next segment
    }
    if (bad) atomicExch(&g_kv4_attn_range, 1);

    // ---- parts: the CTA that arrives last at an item joins them ----
    if (pend[0].parts + pend[1].parts == 0) return;
    __threadfence();
    __syncthreads();
    if (tid < 2) {
        sh_last[tid] = 0;
        const int n = tid ? pend[1].parts : pend[0].parts, at = tid ? pend[1].parts0 : pend[0].parts0;
        if (n) sh_last[tid] = atomicInc(static_cast<unsigned*>(a.workspace) + at, (unsigned)n - 1) == (unsigned)n - 1;  // wraps to 0 behind the last
        __threadfence();
    }
    __syncthreads();
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (!sh_last[which]) continue;
        const Pending p = pend[which];
        const int n = p.parts;
        // CTA j's part: slot 2j, or 2j + 1 where the item begins within it, that is at parts0
        const float* base = static_cast<const float*>(a.workspace) + 1024;
        auto at = [&](int j) { return base + (2 * (long long)(p.parts0 + j) + (j == 0)) * S::PART; };
        // factors 2^(m_j - m) and the joined m and l of each row, one warp a row
        float* fac = reinterpret_cast<float*>(smem);
        float* joined = fac + ROWS * n;
        for (int row = warp; row < ROWS; row += NW) {
            float m = -CUDART_INF_F, l = 0.f;
            for (int j = lane; j < n; j += 32) {
                const float mj = __ldcg(at(j) + ROWS * D + row);
                fac[row * n + j] = mj;
                m = fmaxf(m, mj);
            }
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, w));
            for (int j = lane; j < n; j += 32) {
                const float mj = fac[row * n + j], x = mj == -CUDART_INF_F ? 0.f : exp2_fast(mj - m);
                fac[row * n + j] = x;
                l = fmaf(x, __ldcg(at(j) + ROWS * D + ROWS + row), l);
            }
            l = warp_sum(l);
            if (lane == 0) joined[2 * row] = m, joined[2 * row + 1] = l;
        }
        __syncthreads();
        for (int i = tid; i < ROWS * D / 4; i += THREADS) {
            const int row = i / (D / 4), d = i % (D / 4) * 4, f = p.f0 + row;
            if (f >= p.nq * gq) continue;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int j = 0; j < n; ++j) {
                const float x = fac[row * n + j];
                const float4 v = __ldcg(reinterpret_cast<const float4*>(at(j) + row * D + d));
                s.x = fmaf(x, v.x, s.x), s.y = fmaf(x, v.y, s.y), s.z = fmaf(x, v.z, s.z), s.w = fmaf(x, v.w, s.w);
            }
            store(p.q0, p.h, f, d, s, joined[2 * row], joined[2 * row + 1]);
        }
        __syncthreads();
    }
}

constexpr int kMaxCtas = 1024;  // counters in the workspace's first 4 KB

struct Entry {
    const void* fn;
    int threads, smem, occ, rows, part, most;
};

template <int D, int G, int NT, int NW, int NB, int DEPTH, int OCC>
Entry entry() {
    using S = Shape<D, G, NT, NW, NB, DEPTH>;
    static_assert(S::SMEM * OCC <= 225 * 1024, "shared memory of the CTAs of an SM");
    return {(const void*)kv4_attention_kernel<D, G, NT, NW, NB, DEPTH, OCC>, NW * 32, S::SMEM, OCC, S::ROWS, S::PART, S::MOST};
}

// rows: query rows per KV head of an average request; few: fewer items than SMs, so each is cut over several.
template <int D, int G>
Entry pick(int rows, bool few) {
    // columns: as few n-tiles as hold the rows of an average request, at most what the registers hold
    if constexpr (D == 256) {
        return rows <= 8 || G == 32 ? entry<D, G, 1, 4, 1, 4, 2>() : entry<D, G, G == 32 ? 1 : 2, 4, 1, 4, 2>();
    } else {
        if (rows <= 8) return few ? entry<D, G, 1, 16, 2, D == 64 ? 4 : 2, 1>() : entry<D, G, 1, 4, 2, D == 64 ? 4 : 3, D == 64 ? 4 : 3>();
        if (rows <= 16 || (D == 128 && G == 32)) return entry<D, G, 2, 4, 1, 4, D == 64 ? 3 : 2>();
        return entry<D, G, D == 128 && G == 32 ? 2 : 4, 4, 1, 4, 2>();
    }
}

Entry pick_for(int head_dim, int group, int rows, bool few) {
    if (group == 32)
        return head_dim == 64 ? pick<64, 32>(rows, few) : head_dim == 128 ? pick<128, 32>(rows, few) : pick<256, 32>(rows, few);
    return head_dim == 64 ? pick<64, 64>(rows, few) : head_dim == 128 ? pick<128, 64>(rows, few) : pick<256, 64>(rows, few);
}

// One wave, at most as many CTAs as counters and as the buffer of a joining CTA holds factors for.
int grid_of(const Entry& e, int sms) {
    int n = sms * e.occ;
    if (n > kMaxCtas) n = kMaxCtas;
    return n < e.most ? n : e.most;
}
size_t workspace_of(const Entry& e, int grid) { return 4096 + (size_t)grid * 2 * e.part * sizeof(float); }

}  // namespace

size_t kv4_attention_workspace(int head_dim) {
    size_t most = 0;
    for (int group : {32, 64})
        for (int rows : {8, 16, 32})
            for (bool few : {false, true}) {
                const Entry e = pick_for(head_dim, group, rows, few);
                const size_t n = workspace_of(e, grid_of(e, device_sm_count()));
                most = n > most ? n : most;
            }
    return most;
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, cudaStream_t s) {
    const int sms = device_sm_count();
    const int64_t rows = ((int64_t)a.T * (a.q_heads / a.kv_heads) + a.B - 1) / a.B;
    const Entry e = pick_for(a.head_dim, a.group, (int)(rows < 64 ? rows : 64), (int64_t)a.B * a.kv_heads <= sms);
    cudaError_t err = cudaFuncSetAttribute(e.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, e.smem);
    if (err != cudaSuccess) return err;
    const int grid = grid_of(e, sms);
    int split = a.ws_bytes >= workspace_of(e, grid) ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)e.threads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)e.smem;
    cfg.stream = s;
    cudaLaunchAttribute attrs[1];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    count_launch();
    Kv4AttnArgs args = a;
    void* params[2] = {&args, &split};
    return cudaLaunchKernelExC(&cfg, e.fn, params);
}

int kv4_attn_take_range() {
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv4_attn_range, sizeof(int)) != cudaSuccess) return -1;
    if (v) cudaMemcpyToSymbol(g_kv4_attn_range, &z, sizeof(int));
    return v;
}

}  // namespace mbw
