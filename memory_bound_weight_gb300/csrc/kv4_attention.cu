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
// Mathematics. No value is dequantized. The codes enter m16n8k16 exactly, with
// the keys as rows (a lane's A operand comes straight from the cache's bytes)
// and the query rows that share the KV head (heads of the group x query
// tokens, 8 per n-tile) as columns:
//   q . k = sum over groups of  s * sum q (16 + n)  +  (m - 16 s) * sum q
// 16 + n is 0x4180 | n << 3 in bf16: one shift and one LOP3 per pair. The
// softmax weight p enters as w = fp16(4 p s), one per group, and
//   sum p (s n + m) = [sum w (16 + n) - 24 sum w] / 4 + sum p (m + 8 s)
// with the same rounded w in both sums, so that its rounding (2^-11) only acts
// on the centred code n - 8, not on the offset. p <= 1 against the running
// maximum, s <= 8737 in fp16, so w cannot overflow; the factor 4 moves w's
// subnormal range to p s < 1.5e-5. Scores, maxima, sums and outputs are fp32.
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

__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(bits));
    return r;
}

// Nibbles S and S + 4 of a word as the bf16 pair (16 + n, 16 + n').
template <int S>
__device__ __forceinline__ uint32_t k_pair(uint32_t w) {
    return and_or(S == 0 ? w << 3 : w >> (S == 0 ? 0 : 4 * S - 3), 0x00780078u, 0x41804180u);
}
// Nibble S of both halfwords as the fp16 pair (16 + n, 16 + n').
template <int S>
__device__ __forceinline__ uint32_t v_pair(uint32_t w) {
    return and_or(S == 0 ? w << 6 : S == 1 ? w << 2 : S == 2 ? w >> 2 : w >> 6, 0x03C003C0u, 0x4C004C00u);
}

struct Request {
    int q0, nq, ctx, fb, units, qt;
    long long cost;  // units of all its items
};

template <int D, int G, int NT, int NW, int NB, int DEPTH>
struct Shape {
    static constexpr int NG = D / G, J = D / 32, BB = kv4_block_bytes(D, G), ROWS = 8 * NT;
    static constexpr int U = NW * NB;  // blocks of a unit: one step of every warp
    static constexpr int RING = NW * DEPTH * NB * BB;
    static constexpr int MERGE = NW * 8 * (D + 4) * 4;
    static constexpr int BUF = RING > MERGE ? RING : MERGE;
    static constexpr int QS = NT > 1 ? J * NT * 512 : 0;
    static constexpr int QSUM = NT > 1 ? NG * ROWS * 4 : 0;
    static constexpr int SMEM = BUF + QS + QSUM + 2 * NW * ROWS * 4;
    static constexpr int PART = ROWS * (D + 2);  // floats of a part: rows of D, then M and L of each
};

template <int D, int G, int NT, int NW, int NB, int DEPTH, int OCC>
__global__ void __launch_bounds__(NW * 32, OCC) kv4_attention_kernel(Kv4AttnArgs a, int split) {
    using S = Shape<D, G, NT, NW, NB, DEPTH>;
    constexpr int NG = S::NG, J = S::J, BB = S::BB, ROWS = S::ROWS, THREADS = NW * 32, NV = D / 64;
    constexpr bool ZMMA = NT * NG <= 4;  // 24 sum w by the matrix unit (a constant tile), or in the weights' layout
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* ring = smem;
    uint4* qs = reinterpret_cast<uint4*>(smem + S::BUF);
    float* qsums = reinterpret_cast<float*>(smem + S::BUF + S::QS);
    float* sm_m = reinterpret_cast<float*>(smem + S::BUF + S::QS + S::QSUM);
    float* sm_l = sm_m + NW * ROWS;
    __shared__ long long sh_scan[NW + 1];
    __shared__ long long sh_found[2];
    __shared__ int sh_last;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int gq = a.q_heads / a.kv_heads, bpp = a.page_size / 16;
    const float sl2 = a.scale * 1.44269504088896340736f;
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

    for (long long u = u0; u < u1;) {
        while (u >= start + rq.cost) {
            start += rq.cost;
            rq = request(++b);
        }
        const long long item = (u - start) / rq.units, iu0 = start + item * rq.units;
        const int s0 = (int)(u - iu0);
        const int h = (int)(item / rq.qt), f0 = (int)(item % rq.qt) * ROWS;
        int s1 = rq.units;
        if (split) {
            if (u1 - iu0 < s1) s1 = (int)(u1 - iu0);
        } else if (s0 != 0) {  // its first unit is another CTA's, and so is the item
            u = iu0 + rq.units;
            continue;
        }
        u = iu0 + s1;

        // ---- the blocks [bs, be) of this segment ----
        const int i_last = min(rq.nq - 1, (f0 + ROWS - 1) / gq);
        const int pos_lo = rq.ctx - rq.nq + f0 / gq, pos_hi = rq.ctx - rq.nq + i_last;
        const int k_lo = a.window ? max(0, pos_lo - a.window + 1) : 0;
        const int bs = max(rq.fb + s0 * S::U, k_lo / 16);
        const int be = max(bs, min(rq.fb + s1 * S::U, (pos_hi + 16) / 16));
        const int32_t* table = a.table + (long long)b * a.table_stride;
        const int nsteps = be > bs + warp * NB ? (be - bs - warp * NB + S::U - 1) / S::U : 0;

        // byte offset of the lane's block among the 32 of steps win * 32 / NB ...; -1 past the end
        auto offsets = [&](int win) -> long long {
            const int k = win * (32 / NB) + lane / NB;
            const int blk = bs + (k * NW + warp) * NB + lane % NB;
            if (k >= nsteps || blk >= be) return -1;
            const int p = blk / bpp;
            int page = table[p];
            if (page < 0 || page >= a.num_pages) bad = true, page = 0;
            return (((long long)page * a.kv_heads + h) * bpp + (blk - p * bpp)) * BB;
        };
        long long off = offsets(0), off_next = nsteps > 32 / NB ? offsets(1) : -1;
        uint8_t* my_ring = ring + warp * DEPTH * NB * BB;
        auto issue = [&](int k) {
            if (k < nsteps) {
                constexpr int SPW = 32 / NB;
                if (k % SPW == 0 && k > 0) {
                    off = off_next;
                    if (k + SPW < nsteps) off_next = offsets(k / SPW + 1);
                }
#pragma unroll
                for (int sub = 0; sub < NB; ++sub) {
                    const long long o = __shfl_sync(0xFFFFFFFFu, off, (k % SPW) * NB + sub);
                    if (o >= 0) {
                        uint8_t* dst = my_ring + ((k % DEPTH) * NB + sub) * BB;
                        for (int i = lane; i < BB / 16; i += 32) cp_async16(dst + i * 16, a.pages + o + i * 16);
                    }
                }
            }
            cp_async_commit();
        };
        for (int k = 0; k < DEPTH - 1; ++k) issue(k);

        // ---- the queries as B operands, and their sums over each group ----
        // word pairs of dimensions 32 j + 8 c + (0, 4), (1, 5), (2, 6), (3, 7) of row 8 nt + g
        uint32_t qf[NT == 1 ? J : 1][4];
        float qsum[NT == 1 ? NG : 1][2];
        int posc[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) posc[nt][e] = rq.ctx - rq.nq + min(rq.nq - 1, (f0 + 8 * nt + 2 * c + e) / gq);
        if (NT > 1) __syncthreads();  // the last segment's readers
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (NT > 1 && warp != nt % NW) continue;
            const int f = f0 + 8 * nt + g, i = f / gq;
            const uint16_t* src = a.q + (long long)(rq.q0 + i) * a.q_stride + (long long)(h * gq + f - i * gq) * D + 8 * c;
            float sum[NG];
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) sum[gr] = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (i < rq.nq) v = *reinterpret_cast<const uint4*>(src + 32 * j);
                sum[j * 32 / G] += ((bf16lo_to_f32(v.x) + bf16hi_to_f32(v.x)) + (bf16lo_to_f32(v.y) + bf16hi_to_f32(v.y))) +
                                   ((bf16lo_to_f32(v.z) + bf16hi_to_f32(v.z)) + (bf16lo_to_f32(v.w) + bf16hi_to_f32(v.w)));
                const uint4 w = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                           __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
                if (NT == 1)
                    qf[j][0] = w.x, qf[j][1] = w.y, qf[j][2] = w.z, qf[j][3] = w.w;
                else
                    qs[(j * NT + nt) * 32 + lane] = w;
            }
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                sum[gr] += __shfl_xor_sync(0xFFFFFFFFu, sum[gr], 1);
                sum[gr] += __shfl_xor_sync(0xFFFFFFFFu, sum[gr], 2);
                if (NT == 1) {
                    qsum[gr][0] = __shfl_sync(0xFFFFFFFFu, sum[gr], 8 * c);
                    qsum[gr][1] = __shfl_sync(0xFFFFFFFFu, sum[gr], 8 * c + 4);
                } else if (c == 0) {
                    qsums[gr * ROWS + 8 * nt + g] = sum[gr];
                }
            }
        }
        if (NT > 1) __syncthreads();

        float o[NT][D / 16][4], z[ZMMA ? NT : 1][ZMMA ? NG : 1][4], r[NT][NG][2], M[NT][2], L[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                r[nt][gr][0] = r[nt][gr][1] = 0.f;
                if (ZMMA) z[nt][gr][0] = z[nt][gr][1] = z[nt][gr][2] = z[nt][gr][3] = 0.f;
            }
            M[nt][0] = M[nt][1] = -CUDART_INF_F;
            L[nt][0] = L[nt][1] = 0.f;
        }

        for (int k = 0; k < nsteps; ++k) {
            cp_async_wait<DEPTH - 2>();
            __syncwarp();  // the step's copies of every lane are there, and step k - 1 is read
            issue(k + DEPTH - 1);
            const uint8_t* stage = my_ring + (k % DEPTH) * NB * BB;
            const int blk0 = bs + (k * NW + warp) * NB;

            // scores y of NB blocks: rows g and g + 8 (tokens), columns 2c and 2c + 1 of each n-tile
            float y[NB][NT][4];
#pragma unroll
            for (int sub = 0; sub < NB; ++sub) {
                const uint8_t* blk = stage + sub * BB;
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
                        const uint32_t a0[4] = {k_pair<0>(kw[0][j]), k_pair<0>(kw[1][j]), k_pair<1>(kw[0][j]), k_pair<1>(kw[1][j])};
                        const uint32_t a1[4] = {k_pair<2>(kw[0][j]), k_pair<2>(kw[1][j]), k_pair<3>(kw[0][j]), k_pair<3>(kw[1][j])};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            uint4 q;
                            if (NT == 1)
                                q = make_uint4(qf[j][0], qf[j][1], qf[j][2], qf[j][3]);
                            else
                                q = qs[(j * NT + nt) * 32 + lane];
                            mma_bf16(acc[nt], a0, q.x, q.y);
                            mma_bf16(acc[nt], a1, q.z, q.w);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const float2 sm = kv4_pair(*reinterpret_cast<const uint32_t*>(blk + kv4_meta(D, G, g + 8 * t, gr, 0)));
                        const float low = fmaf(-16.f, sm.x, sm.y);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float2 qq;
                            if (NT == 1)
                                qq = make_float2(qsum[gr][0], qsum[gr][1]);
                            else
                                qq = *reinterpret_cast<const float2*>(qsums + gr * ROWS + 8 * nt + 2 * c);
                            y[sub][nt][2 * t] = fmaf(low, qq.x, fmaf(sm.x, acc[nt][2 * t], y[sub][nt][2 * t]));
                            y[sub][nt][2 * t + 1] = fmaf(low, qq.y, fmaf(sm.x, acc[nt][2 * t + 1], y[sub][nt][2 * t + 1]));
                        }
                    }
                }
            }
            // Some key of this step may be unseen by some row, or lie past the segment.
            const bool edge = blk0 + NB > be || (blk0 + NB) * 16 - 1 > pos_lo ||
                              (a.window && blk0 * 16 <= pos_hi - a.window);
            uint32_t seen = 0xFFFFFFFFu;
            static_assert(NB * NT * 4 <= 32, "one bit per score");
            bool raise = false;
#pragma unroll
            for (int sub = 0; sub < NB; ++sub)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float v = y[sub][nt][e] * sl2;
                        if (edge) {
                            const int t = (blk0 + sub) * 16 + g + 8 * (e >> 1), p = posc[nt][e & 1];
                            if (blk0 + sub >= be || t > p || (a.window && t <= p - a.window)) {
                                v = -CUDART_INF_F;
                                seen &= ~(1u << ((sub * NT + nt) * 4 + e));
                            }
                        }
                        y[sub][nt][e] = v;
                        raise |= v > M[nt][e & 1];
                    }
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
                        const float f = M[nt][e] == -CUDART_INF_F ? 0.f : exp2_fast(M[nt][e] - m);
                        M[nt][e] = m;
                        L[nt][e] *= f;
#pragma unroll
                        for (int gr = 0; gr < NG; ++gr) {
                            r[nt][gr][e] *= f;
                            if (ZMMA) z[nt][gr][e] *= f, z[nt][gr][2 + e] *= f;
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
                    const float m = 2.f - (M[nt][e] == -CUDART_INF_F ? 0.f : M[nt][e]);
#pragma unroll
                    for (int sub = 0; sub < NB; ++sub) {
                        y[sub][nt][e] = exp2_fast(y[sub][nt][e] + m);
                        y[sub][nt][2 + e] = exp2_fast(y[sub][nt][2 + e] + m);
                        L[nt][e] += y[sub][nt][e] + y[sub][nt][2 + e];
                    }
                }
#pragma unroll
            for (int sub = 0; sub < NB; ++sub) {
                const uint8_t* blk = stage + sub * BB;
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
                        const float2 sm = kv4_pair(*reinterpret_cast<const uint32_t*>(blk + kv4_meta(D, G, g + 8 * t, gr, 1)));
                        const float mid = fmaf(8.f, sm.x, sm.y);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float w[2], x[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                w[e] = y[sub][nt][2 * t + e] * sm.x;
                                x[e] = y[sub][nt][2 * t + e] * mid;
                            }
                            if (edge) {  // what is unseen may be no number
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (!(seen >> ((sub * NT + nt) * 4 + 2 * t + e) & 1)) w[e] = x[e] = 0.f;
                            }
                            const __half2 hw = __floats2half2_rn(w[0], w[1]);
                            if (!ZMMA) {
                                const float2 back = __half22float2(hw);
                                x[0] = fmaf(-24.f, back.x, x[0]);
                                x[1] = fmaf(-24.f, back.y, x[1]);
                            }
                            r[nt][gr][0] += x[0];
                            r[nt][gr][1] += x[1];
                            pb[nt][gr][t] = transpose8x8(*reinterpret_cast<const uint32_t*>(&hw));
                        }
                    }
                if (ZMMA) {
                    const uint32_t k24[4] = {0x4E004E00u, 0x4E004E00u, 0x4E004E00u, 0x4E004E00u};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int gr = 0; gr < NG; ++gr) mma_f16(z[nt][gr], k24, pb[nt][gr][0], pb[nt][gr][1]);
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
                    const uint32_t f[4][4] = {{v_pair<0>(lo[0]), v_pair<1>(lo[0]), v_pair<0>(lo[1]), v_pair<1>(lo[1])},
                                              {v_pair<2>(lo[0]), v_pair<3>(lo[0]), v_pair<2>(lo[1]), v_pair<3>(lo[1])},
                                              {v_pair<0>(hi[0]), v_pair<1>(hi[0]), v_pair<0>(hi[1]), v_pair<1>(hi[1])},
                                              {v_pair<2>(hi[0]), v_pair<3>(hi[0]), v_pair<2>(hi[1]), v_pair<3>(hi[1])}};
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
        }
        cp_async_wait<0>();

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
                    sm_m[warp * ROWS + 8 * nt + 2 * c + e] = M[nt][e];
                    sm_l[warp * ROWS + 8 * nt + 2 * c + e] = L[nt][e];
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const int gr = i * 16 / G;
                    const float add = ZMMA ? r[nt][gr][e] - z[nt][gr][e] : r[nt][gr][e];
                    o[nt][i][e] += add;
                    o[nt][i][2 + e] += add;
                }
            }
        const bool whole = s0 == 0 && s1 == rq.units;
        long long parts0 = 0, parts1 = 0;  // first and last CTA of the item
        float* part = nullptr;
        if (!whole) {
            parts0 = ((iu0 + 1) * C - 1) / W;
            parts1 = ((iu0 + rq.units) * C - 1) / W;
            part = static_cast<float*>(a.workspace) + 1024 + (2 * (long long)blockIdx.x + (iu0 >= u0)) * S::PART;
        }
        float* buf = reinterpret_cast<float*>(smem);  // [NW][8][D + 4], over the drained ring
        for (int nt = 0; nt < NT; ++nt) {
            __syncthreads();
#pragma unroll
            for (int n = 0; n < NT; ++n)
                if (n == nt) {
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            buf[(warp * 8 + 2 * c + (e & 1)) * (D + 4) + 16 * i + g + 8 * (e >> 1)] = o[n][i][e];
                }
            __syncthreads();
            for (int i = tid; i < 8 * D / 4; i += THREADS) {
                const int row = i / (D / 4), d = i % (D / 4) * 4, f = f0 + 8 * nt + row;
                if (f >= rq.nq * gq) continue;
                float m = -CUDART_INF_F, l = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) m = fmaxf(m, sm_m[w * ROWS + 8 * nt + row]);
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < NW; ++w) {
                    const float mw = sm_m[w * ROWS + 8 * nt + row], x = mw == -CUDART_INF_F ? 0.f : exp2_fast(mw - m);
                    const float4 v = *reinterpret_cast<const float4*>(buf + (w * 8 + row) * (D + 4) + d);
                    l = fmaf(x, sm_l[w * ROWS + 8 * nt + row], l);
                    s.x = fmaf(x, v.x, s.x), s.y = fmaf(x, v.y, s.y), s.z = fmaf(x, v.z, s.z), s.w = fmaf(x, v.w, s.w);
                }
                if (whole) {
                    const int qi = f / gq;
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    const long long row_at = rq.q0 + qi;
                    const int head = h * gq + f - qi * gq;
                    const long long at = row_at * a.out_stride + (long long)head * D + d;
                    if (a.out_f32) {
                        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) =
                            make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
                    } else {
                        const __nv_bfloat162 p = __floats2bfloat162_rn(s.x * inv, s.y * inv), q = __floats2bfloat162_rn(s.z * inv, s.w * inv);
                        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
                            make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
                    }
                    if (a.lse && d == 0)
                        a.lse[row_at * a.q_heads + head] = l == 0.f ? -CUDART_INF_F : (m + log2f(l) - 2.f) * 0.69314718055994530942f;
                } else {
                    *reinterpret_cast<float4*>(part + (8 * nt + row) * D + d) = s;
                    if (d == 0) {
                        part[ROWS * D + 8 * nt + row] = m;
                        part[ROWS * D + ROWS + 8 * nt + row] = l;
                    }
                }
            }
        }
        if (!whole) {
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const unsigned n = (unsigned)(parts1 - parts0);
                sh_last = atomicInc(static_cast<unsigned*>(a.workspace) + parts0, n) == n;  // wraps to 0 behind the last
                __threadfence();
            }
            __syncthreads();
            if (sh_last) {
                const long long n = parts1 - parts0 + 1;
                // CTA j's part: slot 2j, or 2j + 1 where the item begins within (only at j = parts0)
                const bool in0 = iu0 >= parts0 * W / C;
                const float* base = static_cast<const float*>(a.workspace) + 1024;
                for (int i = tid; i < ROWS * D / 4; i += THREADS) {
                    const int row = i / (D / 4), d = i % (D / 4) * 4, f = f0 + row;
                    if (f >= rq.nq * gq) continue;
                    auto at = [&](long long j) { return base + (2 * (parts0 + j) + (j == 0 && in0)) * S::PART; };
                    float m = -CUDART_INF_F, l = 0.f;
                    for (long long j = 0; j < n; ++j) m = fmaxf(m, __ldcg(at(j) + ROWS * D + row));
                    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                    for (long long j = 0; j < n; ++j) {
                        const float* p = at(j);
                        const float mj = __ldcg(p + ROWS * D + row), x = mj == -CUDART_INF_F ? 0.f : exp2_fast(mj - m);
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(p + row * D + d));
                        l = fmaf(x, __ldcg(p + ROWS * D + ROWS + row), l);
                        s.x = fmaf(x, v.x, s.x), s.y = fmaf(x, v.y, s.y), s.z = fmaf(x, v.z, s.z), s.w = fmaf(x, v.w, s.w);
                    }
                    const int qi = f / gq;
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    const long long row_at = rq.q0 + qi;
                    const int head = h * gq + f - qi * gq;
                    const long long o_at = row_at * a.out_stride + (long long)head * D + d;
                    if (a.out_f32) {
                        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + o_at) =
                            make_float4(s.x * inv, s.y * inv, s.z * inv, s.w * inv);
                    } else {
                        const __nv_bfloat162 p = __floats2bfloat162_rn(s.x * inv, s.y * inv), q = __floats2bfloat162_rn(s.z * inv, s.w * inv);
                        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o_at) =
                            make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
                    }
                    if (a.lse && d == 0)
                        a.lse[row_at * a.q_heads + head] = l == 0.f ? -CUDART_INF_F : (m + log2f(l) - 2.f) * 0.69314718055994530942f;
                }
            }
        }
        __syncthreads();  // the buffers are free for the next segment
    }
    if (bad) atomicExch(&g_kv4_attn_range, 1);
}

constexpr int kMaxCtas = 1024;  // counters in the workspace's first 4 KB

struct Entry {
    const void* fn;
    int threads, smem, occ, rows, part;
};

template <int D, int G, int NT, int NW, int NB, int DEPTH, int OCC>
Entry entry() {
    using S = Shape<D, G, NT, NW, NB, DEPTH>;
    static_assert(S::SMEM * OCC <= 225 * 1024, "shared memory of the CTAs of an SM");
    return {(const void*)kv4_attention_kernel<D, G, NT, NW, NB, DEPTH, OCC>, NW * 32, S::SMEM, OCC, S::ROWS, S::PART};
}

template <int D, int G>
Entry pick(int rows) {
    // columns: as few n-tiles as hold the rows of an average request, at most what the registers hold
    if constexpr (D == 256) {
        return rows <= 8 ? entry<D, G, 1, 4, 1, 4, 2>() : entry<D, G, 2, 4, 1, 4, 2>();
    } else {
        if (rows <= 8) return entry<D, G, 1, 4, 2, 3, D == 64 ? 4 : 3>();
        if (rows <= 16 || (D == 128 && G == 32)) return entry<D, G, 2, 4, 1, 4, D == 64 ? 3 : 2>();
        return entry<D, G, D == 128 && G == 32 ? 2 : 4, 4, 1, 4, 2>();
    }
}

Entry pick_for(int head_dim, int group, int rows) {
    if (group == 32) return head_dim == 64 ? pick<64, 32>(rows) : head_dim == 128 ? pick<128, 32>(rows) : pick<256, 32>(rows);
    return head_dim == 64 ? pick<64, 64>(rows) : head_dim == 128 ? pick<128, 64>(rows) : pick<256, 64>(rows);
}

}  // namespace

size_t kv4_attention_workspace(int head_dim) {
    size_t most = 0;
    for (int group : {32, 64})
        for (int rows : {8, 16, 32}) {
            const Entry e = pick_for(head_dim, group, rows);
            const size_t n = 4096 + (size_t)device_sm_count() * e.occ * 2 * e.part * sizeof(float);
            most = n > most ? n : most;
        }
    return most;
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, cudaStream_t s) {
    const int64_t avg = ((int64_t)a.T * (a.q_heads / a.kv_heads) + a.B - 1) / a.B;
    const Entry e = pick_for(a.head_dim, a.group, (int)(avg < 64 ? avg : 64));
    cudaError_t err = cudaFuncSetAttribute(e.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, e.smem);
    if (err != cudaSuccess) return err;
    int grid = device_sm_count() * e.occ;
    if (grid > kMaxCtas) grid = kMaxCtas;
    int split = a.ws_bytes >= 4096 + (size_t)grid * 2 * e.part * sizeof(float) ? 1 : 0;
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
