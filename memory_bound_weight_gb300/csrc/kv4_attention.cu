// kv4_attention.cu -- attention of one or several query tokens per request
// over the 4-bit paged cache (layout in kv4.cuh). Chunks of a prompt, many query
// rows per KV head, are kv4_attention_tc.cu's; the choice is at the launch below.
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
// within 2^-35 of it. The softmax weight p enters as w = fp16(2^u p s), one per
// group:
//   sum p (s n + m) = [sum w n - 8 sum w] / 2^u + sum p (m + 8 s)
// with the same rounded w in both sums, so that its rounding (2^-11) acts on
// the centred code n - 8 only; 8 sum w comes from a constant tile. p refers to a
// maximum that follows the true one only when it has grown by 2^3, so that what was
// summed seldom has to be taken to another, and u follows the largest scale so far:
// 2^u s is below 2^12, and was between 2^10 and 2^11 when that scale came. So w < 2^15,
// and a weight keeps its 11 bits down to p = 2^-24 and is lost only below 2^-35,
// whatever the size of the values. (With 4 p s the many small weights beside a large
// one were lost where values are small: at 1e-4 the sum of 2000 of them, half the
// result.) Each lane looks at the scales of its share of a step's tokens. Scores,
// maxima, sums and outputs are fp32.
//
// Unpacking is thus one AND per pair and a shift for every other pair. It runs
// on the ALU pipe at half rate, which bounded the forms before: with a shift
// per pair and an OR into 16 + n, and with HADD2 to n - 8.
//
// Work. A block of 16 tokens of one KV head is 2304 bytes in one piece (D =
// 128, G = 64), read once; each warp streams blocks through a ring of shared
// memory of its own (cp.async) with its own softmax state. The blocks of all
// (request, KV head, query tile) items are one line, cut into equal shares for
// the workers of a one-wave grid, each item lengthened by what an item costs
// besides its blocks. The cut is made on the device from the lengths, so a
// captured call follows them. An item cut between workers leaves its parts in
// the workspace, and the worker that arrives last joins them in their order, so
// that the result does not depend on who that is.
//   Many items: each warp is a worker, and no warp waits for another. (With the
// four warps of a CTA as one worker, joining them at every item, 64 requests of
// 300 to 16000 tokens took 82 us, and with blocks handed out by a counter 95 to 103.)
//   Few items, each cut many times: a CTA of 16 warps is one, and its warps are
// joined in shared memory, so that fewer parts go through the workspace (1 request
// of 65536 tokens: 21 us, of 4 heads and a part per SM; 145 with warps as workers).
//
// What bounds it: 64 requests of 300 to 16000 tokens, 308 MB, take 66 us, 4.6 TB/s;
// the time of a further token is that of 6.0 TB/s, 88% of what a copy reaches, and 13
// us are the start (lengths, block table and first block one behind the other), ends
// that are not even, and the join of parts. One request of 1024 tokens takes 11.0 us,
// all of it such latencies.
#include <cuda_runtime.h>

#include <math_constants.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "kv4.cuh"

namespace mbw {

namespace {

__device__ int g_kv4_attn_range;  // a page id, length or query offset was out of range

// A weight's exponent is formed in one operation, the score times its factor less the maximum's, which is rounded; from
// maxima of this size on (in powers of two) that rounding, 2^-10 of a power here and as many as a float holds further out,
// would show, and the difference of the scores is taken first.
constexpr float kFar = 16384.f;
// Growth of a maximum, in powers of two, that is let pass before what was summed is taken to it.
constexpr int kSlack = 3;

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
    int q0, nq, ctx;  // its queries and its length
    int fb;           // first block that a query sees
    uint32_t units;   // of the line
    uint32_t tiles;   // items: KV heads x query tiles
    int qt;           // query tiles
};

// COOP: the NW warps of a CTA are one worker; else each warp is.
template <int D, int G, int NT, int NW, int NB, int DEPTH, bool COOP>
struct Shape {
    static constexpr int NG = D / G, J = D / 32, BB = kv4_block_bytes(D, G), ROWS = 8 * NT;
    static constexpr int WORKERS = COOP ? 1 : NW;       // of a CTA
    static constexpr int STEP = (COOP ? NW : 1) * NB;   // blocks that a worker takes at a time
    static constexpr int STAGE = NB * BB, RING = NW * DEPTH * STAGE;
    static constexpr int PAD = D + 4;  // floats of a row that warps are joined in: 4 to spread the banks
    static constexpr int QS = NT > 1 ? WORKERS * J * NT * 512 : 0;
    static constexpr int QSUM = NT > 1 ? WORKERS * (NG + 1) * ROWS * 4 : 0;
    static constexpr int JOIN = COOP ? NW * 8 * PAD * 4 : 0;  // over the ring, which is drained then
    static constexpr int BUF = RING > JOIN ? RING : JOIN;
    static constexpr int SMEM = BUF + QS + QSUM + (COOP ? 2 * (NW + 1) * ROWS * 4 : 0) + (NW * 32 + 1) * 16;
    static constexpr int PART = ROWS * (D + 2);  // floats of a part: its sums, then m and l of each row
};

// The workspace begins with a counter of finished parts per worker; an item cut between workers has that of its first.
constexpr int kCounters = 4096;

// SHARED: the first shared_len tokens' part is there already (kv4_attention_tc.cu); the items are those of the others, and what
// they give is joined to it as it is stored.
template <int D, int G, int NT, int NW, int NB, int DEPTH, int OCC, bool COOP, bool SHARED>
__global__ void __launch_bounds__(NW * 32, OCC) kv4_attention_kernel(Kv4AttnArgs a, int split, int shift) {
    using S = Shape<D, G, NT, NW, NB, DEPTH, COOP>;
    constexpr int NG = S::NG, J = S::J, BB = S::BB, ROWS = S::ROWS, THREADS = NW * 32, NV = D / 64;
    // V's codes as they are and 8 sum w from a constant tile; or, where several n-tiles share their unpacking, n - 8
    constexpr bool RAW = NT == 1;
    // Units that an item costs besides its own (a warp's line), and the units from which on it is worth their parts' way
    // through the workspace to share them: of a worker at least, of an item that CTAs cut.
    constexpr uint32_t EXTRA = 4, LEAST = 4;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int own = COOP ? 0 : warp;  // the worker in the CTA
    uint4* qs = reinterpret_cast<uint4*>(smem + S::BUF) + own * J * NT * 32;
    float* qsums = reinterpret_cast<float*>(smem + S::BUF + S::QS) + own * (NG + 1) * ROWS;
    float* sm_m = reinterpret_cast<float*>(smem + S::BUF + S::QS + S::QSUM);  // [NW + 1][ROWS], the last joined
    float* sm_l = sm_m + (NW + 1) * ROWS;
    // the line before each thread's requests, and q0, nq and ctx of the one where a thread has no more
    uint4* prefix = reinterpret_cast<uint4*>(smem + S::SMEM) - (THREADS + 1);
    struct Pending {  // an item of which the worker wrote a part
        int q0, nq, h, f0;
        uint32_t first, n;
    };
    __shared__ Pending sh_pend[S::WORKERS][2];  // one that begins before the worker's share, one that begins within
    __shared__ uint32_t sh_scan[NW], sh_items[NW];
    __shared__ uint32_t sh_last[S::WORKERS][2];
    auto sync = [&]() {  // the worker's threads
        if (COOP)
            __syncthreads();
        else
            __syncwarp();
    };

    const int gq = a.q_heads / a.kv_heads, bpp = a.page_size / 16;
    const float sl2 = fabsf(a.scale) * 1.44269504088896340736f;
    uint32_t* counters = static_cast<uint32_t*>(a.workspace);
    float* parts = reinterpret_cast<float*>(counters + kCounters);
    bool bad = false, falls = false;
    if ((COOP ? tid : lane) < 2) sh_pend[own][COOP ? tid : lane].n = 0;

    pdl_launch_dependents();
    // SHARED: what this kernel reads is there, since the shared part's kernel starts it behind its own wait; only that kernel's
    // results are waited for, where they are joined. But that wait was another grid's: the fence sees to it that nothing
    // is read here from a first-level cache that is older (0.2 us of 39: 64 requests behind 8192 tokens).
    if (SHARED)
        __threadfence();
    else
        pdl_wait();

    // ---- the line: per item, EXTRA and its units of STEP << shift blocks ----
    const int unit = S::STEP << shift;
    const int cap = a.table_width * a.page_size;  // at most MBW_MAX_DIM
    auto sized = [&](int q0, int nq, int ctx) {
        Request r;
        r.q0 = q0, r.nq = nq, r.ctx = ctx;
        r.fb = kv4_first_seen(ctx - nq, a.window) / 16;
        if (SHARED) r.fb = max(r.fb, a.shared_len / 16);
        r.units = max(1u, ((uint32_t)(SHARED ? max((ctx + 15) / 16 - r.fb, 0) : (ctx + 15) / 16 - r.fb) + unit - 1) / unit);
        r.qt = ((uint32_t)nq * gq + ROWS - 1) / ROWS;  // at most MBW_MAX_DIM query rows
        r.tiles = (uint32_t)r.qt * a.kv_heads;
        return r;
    };
    auto request = [&](int b) {
        int q0, q1;
        if (a.q_starts) {
            const int s0 = a.q_starts[b], s1 = a.q_starts[b + 1];
            q0 = min(max(s0, 0), a.T);
            q1 = min(max(s1, q0), a.T);
            if (q0 != s0 || q1 != s1) bad = true;
            if (s1 < s0) falls = true;
        } else {
            const int n = a.T / a.B;
            q0 = b * n, q1 = q0 + n;
        }
        int ctx = max(a.ctx_lens[b], 0);
        if (ctx > cap) bad = true, ctx = cap;
        return sized(q0, q1 - q0, ctx);
    };
    const int stride = (a.B + THREADS - 1) / THREADS;  // requests per thread
    // COOP: places are pieces of one item each, as many as the item's units are of all among the CTAs, so that no CTA
    // has to end one item and begin another (a CTA whose share spanned two took 8 us longer).
    float per_unit = 0.f;  // pieces
    if (COOP) {
        float n = 0.f;  // the same in every CTA
        for (int i = 0; i < stride; ++i) {
            const int b = tid * stride + i;
            if (b < a.B) {
                const Request r = request(b);
                n += (float)r.tiles * (float)r.units;
            }
        }
        n = warp_sum(n);
        if (lane == 0) sh_scan[warp] = __float_as_uint(n);
        __syncthreads();
        n = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) n += __uint_as_float(sh_scan[w]);
        per_unit = split ? fminf((float)gridDim.x / n, 1.f) : 0.f;
        __syncthreads();
    }
    auto pieces_of = [&](const Request& r) { return r.units < LEAST ? 1u : max(1u, (uint32_t)((float)r.units * per_unit)); };
    auto places_of = [&](const Request& r) { return COOP ? pieces_of(r) : r.units + EXTRA; };  // of an item
    uint32_t W, items = 0;
    {
        uint32_t x = 0, n = 0;
        uint4 mine = make_uint4(0, 0, 0, 0);
        for (int i = 0; i < stride; ++i) {
            const int b = tid * stride + i;
            if (b < a.B) {
                const Request r = request(b);
                x += r.tiles * places_of(r), n += r.tiles;
                mine.y = r.q0, mine.z = r.nq, mine.w = r.ctx;
            }
        }
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        uint32_t sum = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) sh_scan[warp] = sum, sh_items[warp] = n;
        __syncthreads();
        uint32_t before = 0;
        W = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const uint32_t y = sh_scan[w];
            if (w < warp) before += y;
            W += y, items += sh_items[w];
        }
        mine.x = before + sum - x;
        prefix[tid] = mine;
        if (tid == 0) prefix[THREADS].x = W;
        // Offsets that fall make ranges that overlap, and more items than the launch left room for: then there is no work.
        if (__syncthreads_or(falls)) W = 0;
    }
    // Warps: as many as items at least; worker i of C has the places [i each + min(i, rest), ...). CTAs: one place, and
    // where there are more pieces than CTAs the others behind it.
    const uint32_t all = gridDim.x * S::WORKERS, C = COOP ? all : max(1u, min(all, max(items, W / LEAST)));
    const uint32_t each = W / C, rest = W - each * C;
    const uint32_t me = COOP ? blockIdx.x : warp * gridDim.x + blockIdx.x;  // neighbours on different SMs
    auto start_of = [&](uint32_t i) { return i * each + min(i, rest); };
    auto owner_of = [&](uint32_t p) {
        const uint32_t big = rest * (each + 1);
        return p < big ? p / (each + 1) : rest + (p - big) / each;
    };
    uint32_t pos = COOP ? me : me < C ? start_of(me) : W;
    const uint32_t end = COOP ? W : me < C ? start_of(me + 1) : W;

    // ---- copies: the lane's block offset among the 32 of the steps win * 32 / NB ..., -1 past the end ----
    constexpr int SPW = 32 / NB, STRIDE = COOP ? NW : 1;
    const int at = COOP ? warp : 0;  // the warp's place in a step
    int bs = 0, be = 0, nsteps = 0, h = 0;
    const int32_t* table = a.table;
    auto offsets = [&](int win) -> long long {
        const int k = win * SPW + lane / NB;
        const int blk = bs + (k * STRIDE + at) * NB + lane % NB;
        if (k >= nsteps || blk >= be) return -1;
        const int p = blk / bpp;
        int page = table[p];
        if (page < 0 || page >= a.num_pages) bad = true, page = 0;
        return (((long long)page * a.kv_heads + h) * bpp + (blk - p * bpp)) * BB;
    };
    const uint8_t* my_ring = smem + warp * DEPTH * S::STAGE;
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(my_ring) + lane * 16;
    const uint8_t* pages = a.pages + lane * 16;
    long long off = -1, off_next = -1;
    auto issue = [&](int k) {
        if (k < nsteps) {
            if (k % SPW == 0) {
                off = k == 0 ? offsets(0) : off_next;
                if (k + SPW < nsteps) off_next = offsets(k / SPW + 1);
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

    float o[NT][D / 16][4], z[RAW ? NG : 1][4], r[NT][NG][2], M[NT][2], L[NT][2];

    // SHARED: of a row's maximum and sum here (of 4 p) and its shared part, the factors of their outputs, and their sum's log2.
    struct Joint {
        float own, shared[kKv4SharedParts], lse;
    };
    const long long all_rows = (long long)a.T * a.q_heads;  // of a part
    auto joint = [&](long long at, float m, float l) {
        const float x = l == 0.f ? -CUDART_INF_F : m + log2f(l) - 2.f;
        float y[kKv4SharedParts], top = x;
#pragma unroll
        for (int p = 0; p < kKv4SharedParts; ++p) y[p] = p < a.shared_parts ? __ldcg(a.shared_lse + p * all_rows + at) : -CUDART_INF_F;
#pragma unroll
        for (int p = 0; p < kKv4SharedParts; ++p) top = fmaxf(top, y[p]);
        const float ex = x == -CUDART_INF_F ? 0.f : exp2_fast(x - top);
        float sum = ex;
        Joint j;
#pragma unroll
        for (int p = 0; p < kKv4SharedParts; ++p) {
            j.shared[p] = y[p] == -CUDART_INF_F ? 0.f : exp2_fast(y[p] - top);
            sum += j.shared[p];
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        j.own = l == 0.f ? 0.f : ex * inv / l;
#pragma unroll
        for (int p = 0; p < kKv4SharedParts; ++p) j.shared[p] *= inv;
        j.lse = sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * 0.69314718055994530942f;
        return j;
    };
    // Outputs of rows f0 .. f0 + ROWS - 1 from the sums in o, by one warp.
    auto store = [&](int q0, int nq, int hh, int f0) {
        if (SHARED) pdl_wait();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float inv[2];
            if constexpr (SHARED) {
                // Both columns' loads go together, two parts at a time, the first beside the log sums: a join is a few loads
                // behind one another, not a few a column and part.
                constexpr int PARTS = 2;
                long long at[2];
                bool in[2];
                float v[PARTS][2][D / 8];
                auto fetch = [&](int p) {
#pragma unroll
                    for (int t = 0; t < PARTS; ++t)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int i = 0; i < D / 8; ++i)
                                v[t][e][i] = in[e] && p + t < a.shared_parts ? __ldcg(a.shared_out + ((p + t) * all_rows + at[e]) * D + g + 8 * i) : 0.f;
                };
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int f = f0 + 8 * nt + 2 * c + e, qi = f / gq;
                    in[e] = f < nq * gq;
                    at[e] = in[e] ? (long long)(q0 + qi) * a.q_heads + hh * gq + f - qi * gq : 0;
                }
                fetch(0);
                const Joint j[2] = {joint(at[0], M[nt][0], L[nt][0]), joint(at[1], M[nt][1], L[nt][1])};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (a.lse && g == 0 && in[e]) a.lse[at[e]] = j[e].lse;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) o[nt][i][e] *= j[e].own, o[nt][i][2 + e] *= j[e].own;
                }
#pragma unroll
                for (int p = 0; p < kKv4SharedParts; p += PARTS) {
                    if (p >= a.shared_parts) break;
                    if (p) fetch(p);
#pragma unroll
                    for (int t = 0; t < PARTS; ++t)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                o[nt][i][e] = fmaf(v[t][e][2 * i], j[e].shared[p + t], o[nt][i][e]);
                                o[nt][i][2 + e] = fmaf(v[t][e][2 * i + 1], j[e].shared[p + t], o[nt][i][2 + e]);
                            }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                inv[e] = SHARED ? 1.f : L[nt][e] == 0.f ? 0.f : 1.f / L[nt][e];
                const int f = f0 + 8 * nt + 2 * c + e, qi = f / gq;
                if (f >= nq * gq) continue;
                const long long row = q0 + qi;
                const int head = hh * gq + f - qi * gq;
                if (!SHARED && a.lse && g == 0)
                    a.lse[row * a.q_heads + head] =
                        L[nt][e] == 0.f ? -CUDART_INF_F : (M[nt][e] + log2f(L[nt][e]) - 2.f) * 0.69314718055994530942f;
                if (a.out_f32) {
                    float* to = static_cast<float*>(a.out) + row * a.out_stride + (long long)head * D + g;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) to[16 * i] = o[nt][i][e] * inv[e], to[16 * i + 8] = o[nt][i][2 + e] * inv[e];
                }
            }
            if (a.out_f32) continue;
            // pairs of columns of a dimension become pairs of dimensions of column g
            const int f = f0 + 8 * nt + g, qi = f / gq;
            uint16_t* to = static_cast<uint16_t*>(a.out) + (long long)(q0 + qi) * a.out_stride + (long long)(hh * gq + f - qi * gq) * D + 2 * c;
            const bool there = f < nq * gq;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(o[nt][i][2 * t] * inv[0], o[nt][i][2 * t + 1] * inv[1]);
                    const uint32_t w = transpose8x8(*reinterpret_cast<const uint32_t*>(&v));
                    if (there) *reinterpret_cast<uint32_t*>(to + 16 * i + 8 * t) = w;
                }
        }
    };
    // A part is the o of a warp as it lies in its lanes, then M and L of each row.
    auto put_part = [&](uint32_t slot) {
        float* part = parts + (long long)slot * S::PART;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                reinterpret_cast<float4*>(part)[(nt * (D / 16) + i) * 32 + lane] = make_float4(o[nt][i][0], o[nt][i][1], o[nt][i][2], o[nt][i][3]);
            if (g == 0) {
                *reinterpret_cast<float2*>(part + ROWS * D + 8 * nt + 2 * c) = make_float2(M[nt][0], M[nt][1]);
                *reinterpret_cast<float2*>(part + ROWS * D + ROWS + 8 * nt + 2 * c) = make_float2(L[nt][0], L[nt][1]);
            }
        }
    };
    // Adds the parts of an item to o, M and L, in their order; some at a time are on their way.
    // Piece j's part lies in its slot 0, or 1 where the item begins with it.
    auto add_parts = [&](uint32_t first, uint32_t n) {
        constexpr int BATCH = NT * D <= 64 ? 4 : NT * D <= 128 ? 2 : 1;
        for (uint32_t j = 0; j < n; j += BATCH) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float2 m[BATCH], l[BATCH];
                float4 v[BATCH][D / 16];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const uint32_t q = j + k;
                    m[k] = make_float2(-CUDART_INF_F, -CUDART_INF_F), l[k] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) v[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (q < n) {
                        const float* part = parts + (long long)(2 * (first + q) + (q == 0)) * S::PART;
                        m[k] = __ldcg(reinterpret_cast<const float2*>(part + ROWS * D + 8 * nt + 2 * c));
                        l[k] = __ldcg(reinterpret_cast<const float2*>(part + ROWS * D + ROWS + 8 * nt + 2 * c));
#pragma unroll
                        for (int i = 0; i < D / 16; ++i) v[k][i] = __ldcg(reinterpret_cast<const float4*>(part) + (nt * (D / 16) + i) * 32 + lane);
                    }
                }
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const float m0 = fmaxf(M[nt][0], m[k].x), m1 = fmaxf(M[nt][1], m[k].y);
                    const float f0 = M[nt][0] == -CUDART_INF_F ? 0.f : exp2_fast(M[nt][0] - m0);
                    const float f1 = M[nt][1] == -CUDART_INF_F ? 0.f : exp2_fast(M[nt][1] - m1);
                    const float x0 = m[k].x == -CUDART_INF_F ? 0.f : exp2_fast(m[k].x - m0);
                    const float x1 = m[k].y == -CUDART_INF_F ? 0.f : exp2_fast(m[k].y - m1);
                    M[nt][0] = m0, M[nt][1] = m1;
                    L[nt][0] = fmaf(L[nt][0], f0, l[k].x * x0), L[nt][1] = fmaf(L[nt][1], f1, l[k].y * x1);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        o[nt][i][0] = fmaf(o[nt][i][0], f0, v[k][i].x * x0), o[nt][i][1] = fmaf(o[nt][i][1], f1, v[k][i].y * x1);
                        o[nt][i][2] = fmaf(o[nt][i][2], f0, v[k][i].z * x0), o[nt][i][3] = fmaf(o[nt][i][3], f1, v[k][i].w * x1);
                    }
                }
            }
        }
    };
    auto clear = [&]() {
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
    };
    // COOP: the parts of an item joined by all the CTA's threads, each four values of a lane's o, in groups of threads
    // that take every GROUPS-th part; the groups meet in shared memory.
    auto join_parts = [&](const Pending& p) {
        constexpr int VALUES = NT * (D / 16) * 32, GROUPS = THREADS / VALUES > 1 ? THREADS / VALUES : 1, BATCH = 4;
        struct Sum {
            float4 s;
            float2 m, l;
        };
        Sum* meet = reinterpret_cast<Sum*>(smem);
        if (SHARED) pdl_wait();
        auto join = [&](Sum& x, float4 v, float2 m, float2 l) {
            const float m0 = fmaxf(x.m.x, m.x), m1 = fmaxf(x.m.y, m.y);
            const float f0 = x.m.x == -CUDART_INF_F ? 0.f : exp2_fast(x.m.x - m0), f1 = x.m.y == -CUDART_INF_F ? 0.f : exp2_fast(x.m.y - m1);
            const float g0 = m.x == -CUDART_INF_F ? 0.f : exp2_fast(m.x - m0), g1 = m.y == -CUDART_INF_F ? 0.f : exp2_fast(m.y - m1);
            x.m = make_float2(m0, m1);
            x.l = make_float2(fmaf(x.l.x, f0, l.x * g0), fmaf(x.l.y, f1, l.y * g1));
            x.s = make_float4(fmaf(x.s.x, f0, v.x * g0), fmaf(x.s.y, f1, v.y * g1), fmaf(x.s.z, f0, v.z * g0), fmaf(x.s.w, f1, v.w * g1));
        };
        for (int i0 = 0; i0 < VALUES; i0 += THREADS / GROUPS) {
            const int i = i0 + tid % (THREADS / GROUPS), group = tid / (THREADS / GROUPS), ln = i & 31, tile = i / 32;
            const int col = 8 * (tile / (D / 16)) + 2 * (ln & 3);
            Sum x = {make_float4(0.f, 0.f, 0.f, 0.f), make_float2(-CUDART_INF_F, -CUDART_INF_F), make_float2(0.f, 0.f)};
            for (uint32_t j = group; j < p.n; j += GROUPS * BATCH) {
                float4 v[BATCH];
                float2 m[BATCH], l[BATCH];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const uint32_t q = j + k * GROUPS;
                    v[k] = make_float4(0.f, 0.f, 0.f, 0.f), m[k] = make_float2(-CUDART_INF_F, -CUDART_INF_F), l[k] = make_float2(0.f, 0.f);
                    if (q < p.n) {
                        const float* part = parts + (long long)(p.first + q) * S::PART;
                        v[k] = __ldcg(reinterpret_cast<const float4*>(part) + i);
                        m[k] = __ldcg(reinterpret_cast<const float2*>(part + ROWS * D + col));
                        l[k] = __ldcg(reinterpret_cast<const float2*>(part + ROWS * D + ROWS + col));
                    }
                }
#pragma unroll
                for (int k = 0; k < BATCH; ++k) join(x, v[k], m[k], l[k]);
            }
            if (GROUPS > 1) {
                if (group > 0) meet[tid] = x;
                __syncthreads();
                if (group == 0)
                    for (int w = 1; w < GROUPS; ++w) {
                        const Sum y = meet[tid + w * (THREADS / GROUPS)];
                        join(x, y.s, y.m, y.l);
                    }
                __syncthreads();
            }
            if (group > 0) continue;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int f = p.f0 + col + e, qi = f / gq;
                if (f >= p.nq * gq) continue;
                const float m = e ? x.m.y : x.m.x, l = e ? x.l.y : x.l.x, inv = l == 0.f ? 0.f : 1.f / l;
                const long long row = p.q0 + qi;
                const int head = p.h * gq + f - qi * gq, d = 16 * (tile % (D / 16)) + (ln >> 2);
                const long long to = row * a.out_stride + (long long)head * D + d;
                if constexpr (SHARED) {
                    const long long at = row * a.q_heads + head;
                    const Joint j = joint(at, m, l);
                    float v0 = (e ? x.s.y : x.s.x) * j.own, v1 = (e ? x.s.w : x.s.z) * j.own;
#pragma unroll
                    for (int p = 0; p < kKv4SharedParts; ++p)
                        if (p < a.shared_parts) {
                            const float* from = a.shared_out + (p * all_rows + at) * D + d;
                            v0 = fmaf(__ldcg(from), j.shared[p], v0), v1 = fmaf(__ldcg(from + 8), j.shared[p], v1);
                        }
                    store_out(a.out, to, v0, a.out_f32);
                    store_out(a.out, to + 8, v1, a.out_f32);
                    if (a.lse && d == 0) a.lse[at] = j.lse;
                    continue;
                }
                store_out(a.out, to, (e ? x.s.y : x.s.x) * inv, a.out_f32);
                store_out(a.out, to + 8, (e ? x.s.w : x.s.z) * inv, a.out_f32);
                if (a.lse && d == 0)
                    a.lse[row * a.q_heads + head] = l == 0.f ? -CUDART_INF_F : (m + log2f(l) - 2.f) * 0.69314718055994530942f;
            }
        }
    };
    // COOP: the sums of the CTA's warps joined into warp 0's, through shared memory (over the rings).
    auto join_warps = [&]() {
        float* buf = reinterpret_cast<float*>(smem);  // [NW][8][PAD]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (g == 0) {
                    sm_m[warp * ROWS + 8 * nt + 2 * c + e] = M[nt][e];
                    sm_l[warp * ROWS + 8 * nt + 2 * c + e] = L[nt][e];
                }
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = 8 * nt + 2 * c + e;
                float m = -CUDART_INF_F;
                for (int w = g; w < NW; w += 8) m = fmaxf(m, sm_m[w * ROWS + col]);
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, w));
                const float f = M[nt][e] == -CUDART_INF_F ? 0.f : exp2_fast(M[nt][e] - m);
                if (warp == 0) {
                    float l = 0.f;
                    for (int w = g; w < NW; w += 8) {
                        const float mw = sm_m[w * ROWS + col];
                        l = fmaf(mw == -CUDART_INF_F ? 0.f : exp2_fast(mw - m), sm_l[w * ROWS + col], l);
                    }
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, w);
                    M[nt][e] = m, L[nt][e] = l;
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    buf[(warp * 8 + 2 * c + e) * S::PAD + 16 * i + g] = o[nt][i][e] * f;
                    buf[(warp * 8 + 2 * c + e) * S::PAD + 16 * i + g + 8] = o[nt][i][2 + e] * f;
                }
            }
            __syncthreads();
            // the sum over the warps into warp 0's place, every thread some of it
            for (int i = tid; i < 2 * D; i += THREADS) {
                float* to = buf + i / (D / 4) * S::PAD + i % (D / 4) * 4;
                float4 s = *reinterpret_cast<const float4*>(to);
#pragma unroll
                for (int w = 1; w < NW; ++w) {
                    const float4 v = *reinterpret_cast<const float4*>(to + w * 8 * S::PAD);
                    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
                }
                *reinterpret_cast<float4*>(to) = s;
            }
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][i][e] = buf[(2 * c + (e & 1)) * S::PAD + 16 * i + g + 8 * (e >> 1)];
            }
            if (NT > 1) __syncthreads();
        }
    };

    for (;;) {
    const bool there = pos < end;
    if (there) {
        // ---- the item at pos, and what of it is this worker's ----
        int b;
        uint32_t base;
        Request rq;
        {   // the thread whose requests hold it, by two ballots over the prefixes
            const uint32_t hi = __ballot_sync(0xFFFFFFFFu, prefix[lane * NW].x <= pos);
            const int t0 = (31 - __clz(hi)) * NW;
            const uint32_t lo = __ballot_sync(0xFFFFFFFFu, lane < NW && prefix[t0 + (lane < NW ? lane : 0)].x <= pos);
            const int t = t0 + 31 - __clz(lo);
            const uint4 at_t = prefix[t];
            base = at_t.x, b = t * stride;
            if (stride == 1) rq = sized((int)at_t.y, (int)at_t.z, (int)at_t.w);
            if (stride > 1) {  // 32 of its requests at a time
                for (;; b += 32) {
                    uint32_t n = 0;
                    if (b + lane < a.B && b + lane < (t + 1) * stride) {
                        const Request q = request(b + lane);
                        n = q.tiles * places_of(q);
                    }
                    uint32_t sum = n;
#pragma unroll
                    for (int w = 1; w < 32; w <<= 1) {
                        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, sum, w);
                        if (lane >= w) sum += y;
                    }
                    const uint32_t past = __ballot_sync(0xFFFFFFFFu, base + sum > pos);
                    if (past) {
                        const int l = __ffs(past) - 1;
                        base += __shfl_sync(0xFFFFFFFFu, sum - n, l), b += l;
                        break;
                    }
                    base += __shfl_sync(0xFFFFFFFFu, sum, 31);
                }
                rq = request(b);
            }
        }
        const uint32_t len = places_of(rq), item = (pos - base) / len, i0 = base + item * len, in = pos - i0;
        uint32_t u0, u1 = rq.units;
        if (COOP) {
            const uint32_t n = rq.units / len, more = rq.units - n * len;  // the first `more` pieces hold one unit more
            u0 = in * n + min(in, more), u1 = u0 + n + (in < more);
            pos += gridDim.x;
        } else {
            u0 = in > EXTRA ? in - EXTRA : 0;
            if (split)
                u1 = min(u1, max(end - i0, EXTRA) - EXTRA);
            else if (in > EXTRA)  // its first unit is another worker's, and so is the item
                u1 = 0;
            pos = i0 + len;
            if (u1 <= u0) continue;
        }
        const int q0 = rq.q0, nq = rq.nq, ctx = rq.ctx;
        h = (int)(item / (uint32_t)rq.qt);
        const int f0 = (int)(item - (uint32_t)h * rq.qt) * ROWS;
        const int pos_lo = ctx - nq + f0 / gq, pos_hi = ctx - nq + min(nq - 1, (f0 + ROWS - 1) / gq);
        {
            bs = max(rq.fb + (int)u0 * unit, kv4_first_seen(pos_lo, a.window) / 16);
            be = (int)min((long long)rq.fb + (long long)u1 * unit, (long long)max(pos_hi + 16, 0) / 16);
            be = max(bs, be);
            nsteps = be > bs + at * NB ? (be - bs - at * NB + S::STEP - 1) / S::STEP : 0;
            table = a.table + (long long)b * a.table_stride;
        }
        uint4 q_raw[NT == 1 ? J : 1];  // on their way while the block table is read
        if (NT == 1) {
            const int f = f0 + g, i = f / gq;
            const uint16_t* src = a.q + (long long)(q0 + i) * a.q_stride + (long long)(h * gq + f - i * gq) * D + 8 * c;
#pragma unroll
            for (int j = 0; j < J; ++j) q_raw[j] = i < nq ? *reinterpret_cast<const uint4*>(src + 32 * j) : make_uint4(0, 0, 0, 0);
        }
        for (int k = 0; k < DEPTH - 1; ++k) issue(k);

        // ---- the queries as B operands, and their sums over each group ----
        // word pairs of dimensions 32 j + 8 c + (0, 4), (1, 5), (2, 6), (3, 7) of row 8 nt + g
        uint32_t qf[NT == 1 ? J : 1][4];
        float qsum[NT == 1 ? NG : 1][2], qscale[2];
        int posc[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) posc[nt][e] = ctx - nq + min(nq - 1, (f0 + 8 * nt + 2 * c + e) / gq);
        if (NT > 1) sync();  // the last item's readers
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (NT > 1 && COOP && warp != nt % NW) continue;
            const int f = f0 + 8 * nt + g, i = f / gq;
            const uint16_t* src = a.q + (long long)(q0 + i) * a.q_stride + (long long)(h * gq + f - i * gq) * D + 8 * c;
            float sum[NG];
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) sum[gr] = 0.f;
            uint4 v[J];
            uint32_t big = 0;  // the largest |q| of the row, as bf16 bits
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (NT == 1)
                    v[j] = q_raw[j];
                else
                    v[j] = i < nq ? *reinterpret_cast<const uint4*>(src + 32 * j) : make_uint4(0, 0, 0, 0);
                big = __vmaxu2(__vmaxu2(big, v[j].x & 0x7FFF7FFFu), __vmaxu2(v[j].y & 0x7FFF7FFFu,
                               __vmaxu2(v[j].z & 0x7FFF7FFFu, v[j].w & 0x7FFF7FFFu)));
            }
            big = __vmaxu2(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
            big = __vmaxu2(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
            const uint32_t ex = max(max(big >> 16, big & 0xFFFFu) >> 7, 20u);  // its biased exponent
            // to 2^14, and back with the codes' 2^24 (in two factors: either is a normal number)
            const float up = copysignf(__uint_as_float((268u - ex) << 23), a.scale), down =
                fmaxf(__uint_as_float((ex - 14u) << 23) * (sl2 * 16777216.f), 1.17549435e-38f);  // 0 times the minus infinity of an unseen key is not 0
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
        if (NT > 1) sync();

        clear();
        // scores are kept as s and m give them; col_scale (>= 0) takes those of a column to powers of two
        auto col_scale = [&](int nt, int e) { return NT == 1 ? qscale[e] : qsums[NG * ROWS + 8 * nt + 2 * c + e]; };

        bool far = false;  // some row's maximum is kFar or more from 0
        // weights are 2^up p; in the lower half of limit the largest scale that this has room for, as fp16 bits
        float up = 2.f;
        uint32_t limit = 0x7FFF8000u;
        // of each column, what a score's power of two is off its weight's, and the score from which on its reference moves
        float shift[NT][2], above[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) shift[nt][0] = shift[nt][1] = 0.f, above[nt][0] = above[nt][1] = -CUDART_INF_F;
        for (int k = 0; k < nsteps; ++k) {
            cp_async_wait<DEPTH - 2>();
            __syncwarp();  // the step's copies of every lane are there, and step k - 1 is read
            issue(k + DEPTH - 1);
            const uint8_t* stage = my_ring + (k % DEPTH) * NB * BB;
            const int blk0 = bs + (k * STRIDE + at) * NB;

            // Some key of this step may be unseen by some row, or lie past the segment.
            const bool edge = blk0 + NB > be || (blk0 + NB) * 16 - 1 > pos_lo ||
                              (a.window && blk0 * 16 <= pos_hi - a.window);
            // limit, or a larger scale of V of the lane's share of the tokens
            uint32_t most = limit, ms[NB * (NG > 2 ? NG / 2 : 1)];
            constexpr int SHARE = NG > 2 ? NG / 2 : 1;
#pragma unroll
            for (int sub = 0; sub < NB; ++sub) {
                const int first = NG > 1 ? lane * SHARE : lane & 15;
                uint32_t m[SHARE];
                load_meta<SHARE>(stage + sub * BB + kv4_meta(D, G, 0, 0, 1) + 4 * first, m);
#pragma unroll
                for (int i = 0; i < SHARE; ++i) {
                    if (edge) {  // not that of a token that no row sees
                        const int t = (blk0 + sub) * 16 + (first + i) / NG;
                        if (blk0 + sub >= be || t > pos_hi || (a.window && t <= pos_lo - a.window)) m[i] = 0x8000u;
                    }
                }
#pragma unroll
                for (int i = 0; i < SHARE; ++i) ms[sub * SHARE + i] = m[i];
            }
#pragma unroll
            for (int i = 0; i + 1 < NB * SHARE; i += 2) most = __vimax3_s16x2(ms[i], ms[i + 1], most);
            if (NB * SHARE % 2) most = __vmaxs2(most, ms[NB * SHARE - 1]);

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
            bool raise = most != limit;
#pragma unroll
            for (int sub = 0; sub < NB; ++sub)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) raise |= y[sub][nt][e] > above[nt][e & 1];
            if (__any_sync(0xFFFFFFFFu, raise)) {
                float less = 1.f;  // of 2^up
                const int top = __reduce_max_sync(0xFFFFFFFFu, (int)(most << 16)) >> 16;
                if (top > (int16_t)limit) {  // room for twice the scale
                    const int E = min(max(top >> 10, 0) + 2, 31);
                    less = __int_as_float((30 - kSlack - E - (int)up + 127) << 23);
                    up = (float)(30 - kSlack - E), limit = 0x7FFF0000u | (uint32_t)(E < 31 ? (E << 10) - 1 : 0x7FFF);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = M[nt][e];
#pragma unroll
                        for (int sub = 0; sub < NB; ++sub) m = fmaxf(m, fmaxf(y[sub][nt][e], y[sub][nt][2 + e]));
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, w));
                        const float f = M[nt][e] == -CUDART_INF_F ? 0.f : less * exp2_fast((M[nt][e] - m) * col_scale(nt, e));
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
                bool out = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) out |= M[nt][e] != -CUDART_INF_F && !(fabsf(M[nt][e] * col_scale(nt, e)) < kFar);
                far = __any_sync(0xFFFFFFFFu, out);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = col_scale(nt, e);
                        const bool none = M[nt][e] == -CUDART_INF_F;
                        shift[nt][e] = none ? 0.f : far ? up : fmaf(-M[nt][e], f, up);
                        above[nt][e] = none ? -CUDART_INF_F : M[nt][e] + __fdividef((float)kSlack, f);
                    }
            }
            if (far) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float base = M[nt][e] == -CUDART_INF_F ? 0.f : M[nt][e];
#pragma unroll
                        for (int sub = 0; sub < NB; ++sub) y[sub][nt][e] -= base, y[sub][nt][2 + e] -= base;
                    }
            }
            // weights 2^up p
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float f = col_scale(nt, e);
#pragma unroll
                    for (int sub = 0; sub < NB; ++sub) {
                        y[sub][nt][e] = exp2_fast(fmaf(y[sub][nt][e], f, shift[nt][e]));
                        y[sub][nt][2 + e] = exp2_fast(fmaf(y[sub][nt][2 + e], f, shift[nt][e]));
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

        // ---- the rows' sums complete, of 4 p again, then the item or the worker's part of it ----
        const float down = __int_as_float((2 - (int)up + 127) << 23);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (M[nt][e] != -CUDART_INF_F) M[nt][e] *= col_scale(nt, e);
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) {
                    L[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, L[nt][e], w);
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) r[nt][gr][e] += __shfl_xor_sync(0xFFFFFFFFu, r[nt][gr][e], w);
                }
                L[nt][e] *= down;
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) r[nt][gr][e] *= down;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const int gr = i * 16 / G;
                    if (RAW) {
                        o[nt][i][e] = fmaf(o[nt][i][e] - z[gr][e], 0x1p24f * down, r[nt][gr][e]);
                        o[nt][i][2 + e] = fmaf(o[nt][i][2 + e] - z[gr][2 + e], 0x1p20f * down, r[nt][gr][e]);
                    } else {
                        o[nt][i][e] = fmaf(o[nt][i][e], down, r[nt][gr][e]);
                        o[nt][i][2 + e] = fmaf(o[nt][i][2 + e], down, r[nt][gr][e]);
                    }
                }
            }
        if (COOP) join_warps();
        if (!COOP || warp == 0) {
            if (u0 == 0 && u1 == rq.units) {
                store(q0, nq, h, f0);
            } else {
                // A warp's two parts at most: of an item that began before its share, and of one whose other parts are
                // later workers'. A CTA's: one per piece.
                const int begins = !COOP && u0 == 0;
                put_part(COOP ? i0 + in : 2 * me + begins);
                if (lane == 0) {
                    Pending& p = sh_pend[own][begins];
                    p.q0 = q0, p.nq = nq, p.h = h, p.f0 = f0;
                    p.first = COOP ? i0 : owner_of(i0 + EXTRA);
                    p.n = COOP ? len : owner_of(i0 + len - 1) - p.first + 1;
                }
            }
        }
    }
    if (!COOP && there) continue;

    // ---- parts: the worker that arrives last at an item joins them. A CTA looks behind each piece, a warp at the end ----
    sync();
    if (sh_pend[own][0].n + sh_pend[own][1].n > 0) {
        if ((COOP ? tid : lane) == 0) {
            __threadfence();  // the worker's parts before their counts
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint32_t n = sh_pend[own][w].n;
                sh_last[own][w] = n && atomicInc(counters + sh_pend[own][w].first, n - 1) == n - 1;  // back to 0 behind the last
            }
            __threadfence();
        }
        sync();
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
            if (!sh_last[own][w]) continue;
            const Pending p = sh_pend[own][w];
            if (COOP) {
                join_parts(p);
            } else {
                clear();
                add_parts(p.first, p.n);
                store(p.q0, p.nq, p.h, p.f0);
            }
        }
        sync();
        if ((COOP ? tid : lane) < 2) sh_pend[own][COOP ? tid : lane].n = 0;
        sync();
    }
    if (!there) break;
    }
    if (SHARED) pdl_wait();  // no CTA ends before the shared part's kernel: who waits for this one waits for both
    if (bad) atomicExch(&g_kv4_attn_range, 1);
}

struct Entry {
    const void* fn;
    int threads, smem, occ, rows, part, workers, step;
};

template <int D, int G, int NT, int NW, int NB, int DEPTH, int OCC, bool COOP, bool SHARED = false>
Entry entry() {
    using S = Shape<D, G, NT, NW, NB, DEPTH, COOP>;
    static_assert(S::SMEM * OCC <= 225 * 1024, "shared memory of the CTAs of an SM");
    return {(const void*)kv4_attention_kernel<D, G, NT, NW, NB, DEPTH, OCC, COOP, SHARED>, NW * 32, S::SMEM, OCC, S::ROWS, S::PART,
            S::WORKERS, S::STEP};
}

// Query rows per KV head of an average request from which on they are many: tiles of 128 rows on tcgen05 where there are
// enough such tiles (kv4_attention_tc.cu) and the head has at most 128 dimensions, else tiles of 16 here, which unpack K
// and V half as often as tiles of 8, with more empty rows and fewer warps to an SM. Measured, tiles of 16 or 8 against 128
// rows: 16 requests of 32 queries x 4 heads and 4000 tokens 188 us, 50 us; 16 of 16 x 7 heads and 4000 tokens 92, 38; 4
// tiles of 112 rows, 16 of them of 128, 32 of 128: a geometric mean over contexts of 300 to 16000 tokens of 0.64, 1.35 and
// 1.60 of the time here, the join of what many CTAs share included. Below 96 rows the two are closer than 1.2 but where
// there are as many items as SMs. (12 requests of 2 to 5 queries x 7 heads: tiles of 16 take 37 us, of 8 27.)
constexpr int kWideRows = 96, kTensorItems = 16;

// rows: query rows per KV head of an average request; few: few items, each cut over several SMs.
template <int D, int G>
Entry pick(int rows, bool few) {
    if constexpr (D == 256) {
        if constexpr (G == 64)
            if (rows >= kWideRows) return few ? entry<D, G, 2, 8, 1, 4, 1, true>() : entry<D, G, 2, 4, 1, 4, 2, false>();
        return few ? entry<D, G, 1, 8, 1, 4, 1, true>() : entry<D, G, 1, 4, 1, 4, 2, false>();
    } else {
        if (rows < kWideRows) return few ? entry<D, G, 1, 16, 2, D == 64 ? 4 : 2, 1, true>() : entry<D, G, 1, 4, 2, D == 64 ? 4 : 3, D == 64 ? 4 : 3, false>();
        return few ? entry<D, G, 2, 8, 1, 4, 1, true>() : entry<D, G, 2, 4, 1, 4, D == 64 ? 3 : 2, false>();
    }
}

// Of the requests' own tokens behind shared ones: few rows, and at most 128 dimensions.
template <int D, int G>
Entry pick_shared(bool few) {
    return few ? entry<D, G, 1, 16, 2, D == 64 ? 4 : 2, 1, true, true>() : entry<D, G, 1, 4, 2, D == 64 ? 4 : 3, D == 64 ? 4 : 3, false, true>();
}

Entry pick_for(int head_dim, int group, int rows, bool few, bool shared = false) {
    if (shared) {
        if (group == 32) return head_dim == 64 ? pick_shared<64, 32>(few) : pick_shared<128, 32>(few);
        return head_dim == 64 ? pick_shared<64, 64>(few) : pick_shared<128, 64>(few);
    }
    if (group == 32)
        return head_dim == 64 ? pick<64, 32>(rows, few) : head_dim == 128 ? pick<128, 32>(rows, few) : pick<256, 32>(rows, few);
    return head_dim == 64 ? pick<64, 64>(rows, few) : head_dim == 128 ? pick<128, 64>(rows, few) : pick<256, 64>(rows, few);
}

// One wave; for each warp two parts and a counter, for each CTA and each of at most 4 items per CTA a part and a counter.
constexpr int kItemsPerCta = 4;
int grid_of(const Entry& e, int sms) {
    const int n = sms * e.occ, most = e.workers > 1 ? kCounters / e.workers : kCounters / (kItemsPerCta + 1);
    return n < most ? n : most;
}
size_t workspace_of(const Entry& e, int grid) {
    const size_t slots = (size_t)grid * (e.workers > 1 ? 2 * e.workers : kItemsPerCta + 1);
    return kCounters * sizeof(uint32_t) + slots * e.part * sizeof(float);
}

}  // namespace

cudaError_t kv4_allow_smem(const void* kernel, int bytes) {
    struct Done {
        std::atomic<const void*> fn;
        std::atomic<unsigned> devices;
    };
    static Done done[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    Done* slot = nullptr;
    for (Done& d : done) {
        const void* fn = d.fn.load(std::memory_order_acquire);
        if (!fn && d.fn.compare_exchange_strong(fn, kernel)) fn = kernel;
        if (fn == kernel) {
            slot = &d;
            break;
        }
    }
    const unsigned bit = dev < 32 ? 1u << dev : 0u;
    if (slot && (slot->devices.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess && slot) slot->devices.fetch_or(bit, std::memory_order_release);
    return err;
}

size_t kv4_attention_workspace(int head_dim) {
    size_t most = 0;
    for (int group : {32, 64})
        for (int rows : {8, kWideRows})
            for (bool few : {false, true}) {
                const Entry e = pick_for(head_dim, group, rows, few);
                const size_t n = workspace_of(e, grid_of(e, device_sm_count()));
                most = n > most ? n : most;
            }
    const size_t n = kv4_attention_tc_workspace(head_dim);
    return n > most ? n : most;
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, cudaStream_t s) {
    const int sms = device_sm_count();
    const int64_t gq = a.q_heads / a.kv_heads, rows = ((int64_t)a.T * gq + a.B - 1) / a.B;
    const int64_t with = a.B < a.T ? a.B : a.T;  // requests that have queries, at most
    if (a.head_dim <= 128 && rows >= kWideRows && a.kv_heads * with * ((rows + 127) / 128) >= kTensorItems) return launch_kv4_attention_tc(a, s);
    const int64_t tile = rows < kWideRows || (a.head_dim == 256 && a.group == 32) ? 8 : 16;
    // items of requests of average size, and the most that requests of any sizes have
    const int64_t items = a.kv_heads * with * ((rows + tile - 1) / tile);
    const int64_t most_items = a.kv_heads * (with + ((int64_t)a.T * gq + tile - 1) / tile);
    // CTAs as workers cut whole items among them, so there have to be more CTAs than items by enough (12 requests of 8
    // KV heads and 32768 tokens, 96 items: 123 us against 92 with warps; 64 items: 68 against 69; 8: 19.5 against 84).
    const bool few = 2 * items <= sms && most_items <= kItemsPerCta * sms;
    const Entry e = pick_for(a.head_dim, a.group, (int)(rows < kWideRows ? rows : kWideRows), few, a.shared_len > 0);
    if (e.smem > 48 * 1024) {
        const cudaError_t err = kv4_allow_smem(e.fn, e.smem);
        if (err != cudaSuccess) return err;
    }
    int grid = grid_of(e, sms);
    int split = a.ws_bytes >= workspace_of(e, grid) ? 1 : 0;
    // Units so large that the line of all items has places of 32 bits.
    const int64_t tiles = a.kv_heads * (((int64_t)a.T * gq + e.rows - 1) / e.rows + a.B);
    int shift = 0;
    while (tiles * (((int64_t)a.table_width * a.page_size / 16 + ((int64_t)e.step << shift)) / ((int64_t)e.step << shift) + 3) > 0x7FFFFFFFll &&
           shift < 20)
        ++shift;
    // No more CTAs than there can be work for.
    const int64_t most = tiles * (((int64_t)a.table_width * a.page_size / 16 + e.step - 1) / e.step + 3);
    if (most < grid) grid = (int)(most > 0 ? most : 1);
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
    void* params[3] = {&args, &split, &shift};
    return cudaLaunchKernelExC(&cfg, e.fn, params);
}

// Behind the plain call's workspace, the shared part's outputs and log sums of all rows.
size_t kv4_attention_shared_workspace(int head_dim, int64_t T, int64_t q_heads) {
    const size_t plain = (kv4_attention_workspace(head_dim) + 15) / 16 * 16;
    return head_dim == 256 ? plain : plain + kv4_attention_prefix_rows(T, q_heads) * (head_dim + 1) * sizeof(float);
}

cudaError_t launch_kv4_attention_shared(const Kv4AttnArgs& a, int shared_len, cudaStream_t s) {
    const int64_t gq = a.q_heads / a.kv_heads, rows = ((int64_t)a.T * gq + a.B - 1) / a.B;
    // From kWideRows on the call's own tokens are the tcgen05 kernel's, which joins no part that is there already; 256 dimensions
    // do not fit the shared part's kernel. Both take the plain call, which reads the shared pages for every request.
    if (a.head_dim == 256 || rows >= kWideRows || a.ws_bytes < kv4_attention_shared_workspace(a.head_dim, a.T, a.q_heads)) return launch_kv4_attention(a, s);
    const size_t plain = (kv4_attention_workspace(a.head_dim) + 15) / 16 * 16;
    Kv4AttnArgs b = a;
    b.ws_bytes = plain;
    b.shared_len = shared_len;
    b.shared_out = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + plain);
    b.shared_lse = b.shared_out + kv4_attention_prefix_rows(a.T, a.q_heads) * a.head_dim;
    Kv4SharedPlan plan;
    cudaError_t e = plan_kv4_attention_prefix(b, shared_len, &plan);
    if (e != cudaSuccess) return e;
    if (plan.parts == 0) return launch_kv4_attention(a, s);
    b.shared_parts = plan.parts;
    e = launch_kv4_attention_prefix(b, plan, s);
    return e == cudaSuccess ? launch_kv4_attention(b, s) : e;
}

int kv4_attn_take_range() {
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_kv4_attn_range, sizeof(int)) != cudaSuccess) return -1;
    if (v) cudaMemcpyToSymbol(g_kv4_attn_range, &z, sizeof(int));
    return v;
}

}  // namespace mbw
