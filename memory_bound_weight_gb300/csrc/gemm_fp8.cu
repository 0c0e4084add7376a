// gemm_fp8.cu -- Y = X . W^T of 8-bit floating point operands with a scale for
// each block of 128, on tcgen05 (kind::f8f6f4), plain or gated.
//
//   y[m][n] = sum over blocks kb of  xs[m][kb] ws[n / 128][kb] d,   d = sum over k in kb of X[m][k] W[n][k]
//
// d is a sum of 128 products of e4m3 codes in fp32, a fresh accumulator in TMEM
// for each block of 128 k (one swizzled 128-byte row of shared memory); the
// scales, which change with every block, are applied as the sums are read back:
// y is kept in registers, y += (xs ws) d. Two accumulators in turn, so that the
// products of a block run while the one before is added.
//
// Two orientations of one kernel. With few rows of X (ROWS_X = false) the 128
// lanes of the accumulator are rows of W, its columns the rows of X (16 to 128 of
// them): the call is a stream of W, and the factor changes by column. With many,
// lanes are rows of X and columns rows of W.
//
// Gated: a second matrix U of W's shape, two sums a tile, y = silu(W sum) (U sum).
//
// A CTA is 10 warps: one that issues the copies, one that issues the products, 8
// that add (two for each quarter of the lanes, half of the columns each).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>

#include "device.cuh"
#include "internal.h"

namespace mbw {

namespace {

__device__ int g_f8_fault;  // a bounded wait expired

__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void bar_init(uint64_t* bar, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_at(bar)), "r"(count));
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_at(bar)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_at(bar)), "r"(bytes) : "memory");
}
// A bounded wait by a warp. Who has given up once waits no more: every role then runs to its end.
__device__ __forceinline__ void bar_wait(uint64_t* bar, uint32_t parity, bool& ok) {
    bool got = !ok;
    for (int i = 0; i < MBW_WAIT_LIMIT && !got; ++i) {
        uint32_t r;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(r) : "r"(smem_at(bar)), "r"(parity) : "memory");
        got = r != 0;
    }
    got = __all_sync(0xFFFFFFFFu, got);
    if (!got) atomicExch(&g_f8_fault, 1), ok = false;
}
__device__ __forceinline__ bool elect() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_at(bar)) : "memory");
}
__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_at(dst)),
                 "l"(map), "r"(c0), "r"(c1), "r"(smem_at(bar))
                 : "memory");
}
// K-major operand in rows of 128 bytes (128 codes), 8-row atoms of 1024 bytes with 128-byte swizzle.
__device__ __forceinline__ uint64_t desc(uint32_t at) {
    return (uint64_t)((at >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::f8f6f4: A and B e4m3, D fp32, both K-major
__host__ __device__ constexpr uint32_t idesc(int m, int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24); }
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"((uint32_t)add)
                 : "memory");
}

// N columns of the thread's TMEM lane, N = 8, 16 or 32.
template <int N>
__device__ __forceinline__ void ld(uint32_t* v, uint32_t at) {
    if constexpr (N == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]) : "r"(at));
    else if constexpr (N == 16)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
                       "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                     : "r"(at));
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
            "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
              "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
              "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
              "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
            : "r"(at));
}
// The loads before this are there, those of v among them, which is not used before.
template <int N>
__device__ __forceinline__ void wait_ld(uint32_t* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile("" : "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]), "+r"(v[i + 6]), "+r"(v[i + 7]));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{.reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z;}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

constexpr int kAdders = 8, kThreads = (kAdders + 2) * 32;
constexpr int kCounters = 1024;  // of tiles cut between CTAs; every call leaves them at zero
__device__ __forceinline__ void bar_adders() { asm volatile("bar.sync 1, %0;" ::"n"(kAdders * 32) : "memory"); }

// Lanes are 128 rows of X (ROWS_X) or of W, columns BN rows of the other; GLU: two sums of BN columns.
template <bool ROWS_X, int BN, bool GLU>
struct Shape {
    static constexpr int SETS = GLU ? 2 : 1, HC = BN / 2;                       // columns a thread adds, of each set
    static constexpr int LANE_BOX = 128 * 128, COL_BOX = BN * 128;              // bytes
    static constexpr int LANE_BOXES = GLU && !ROWS_X ? 2 : 1, COL_BOXES = GLU && ROWS_X ? 2 : 1;
    static constexpr int STAGE = LANE_BOXES * LANE_BOX + COL_BOXES * COL_BOX;
    static constexpr int DEPTH = 196608 / STAGE < 12 ? 196608 / STAGE : 12;
    static constexpr int COLS = 2 * SETS * BN;                                  // of TMEM
    static constexpr int TABLE = ROWS_X ? 0 : kAdders * 4 * SETS * HC * 4;      // factors of 4 blocks by column, a warp's own
    static constexpr int OFF_TABLE = DEPTH * STAGE, OFF_BAR = OFF_TABLE + TABLE;
    static constexpr int SMEM = OFF_BAR + (2 * DEPTH + 5) * 8 + 16 + 1024;
    static constexpr int PART = SETS * BN * 128;                                // floats of a part
    static_assert(COLS >= 32 && COLS <= 512 && (COLS & (COLS - 1)) == 0 && DEPTH >= 3 && SMEM <= 227 * 1024, "");
};

template <bool ROWS_X, int BN, bool GLU>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                    const __grid_constant__ CUtensorMap map_u, const Fp8Args a, const int split) {
    using S = Shape<ROWS_X, BN, GLU>;
    constexpr int SETS = S::SETS, HC = S::HC, DEPTH = S::DEPTH;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-smem_at(smem_raw) & 1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);
    uint64_t *empty = full + DEPTH, *sfull = empty + DEPTH, *sempty = sfull + 2, *done = sempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    __shared__ uint32_t sh_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    bool ok = true;

    if (tid == 0) {
        for (int i = 0; i < DEPTH; ++i) bar_init(&full[i], 1), bar_init(&empty[i], 1);
        for (int i = 0; i < 2; ++i) bar_init(&sfull[i], 1), bar_init(&sempty[i], kAdders);
        bar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_at(tmem_slot)), "n"(S::COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();

    // ---- the line: the blocks of k of all tiles, cut into equal shares, or whole tiles in turn ----
    const int KB = a.K / 128;
    const int tiles_m = ROWS_X ? (a.M + 127) / 128 : (a.M + BN - 1) / BN, tiles_n = ROWS_X ? (a.N + BN - 1) / BN : (a.N + 127) / 128;
    const long long all = (long long)tiles_m * tiles_n * KB, each = all / gridDim.x, rest = all - each * gridDim.x;
    auto start_of = [&](long long i) { return i * each + (i < rest ? i : rest); };
    auto owner_of = [&](long long p) {
        const long long big = rest * (each + 1);
        return (int)(p < big ? p / (each + 1) : rest + (p - big) / each);
    };
    struct Piece {
        int m0, n0, kb0, kb1;
        long long tile;
    };
    struct Line {
        long long pos, end, stride;
    };
    auto line = [&]() {
        Line l;
        l.pos = split ? start_of(blockIdx.x) : (long long)blockIdx.x * KB;
        l.end = split ? start_of(blockIdx.x + 1) : all;
        l.stride = split ? 0 : (long long)(gridDim.x - 1) * KB;
        return l;
    };
    auto next = [&](Line& l, Piece& p) {
        if (l.pos >= l.end) return false;
        p.tile = l.pos / KB;
        p.kb0 = (int)(l.pos - p.tile * KB);
        p.kb1 = (int)min((long long)KB, p.kb0 + l.end - l.pos);
        l.pos += p.kb1 - p.kb0 + l.stride;
        const int tn = (int)(p.tile / tiles_m), tm = (int)(p.tile - (long long)tn * tiles_m);  // tiles of one W one behind the other
        p.m0 = tm * (ROWS_X ? 128 : BN), p.n0 = tn * (ROWS_X ? BN : 128);
        return true;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ copies ----
        const bool leader = elect();
        auto weights = [&](uint8_t* st, const Piece& p, int kb, uint64_t* bar) {
            uint8_t* to = ROWS_X ? st + S::LANE_BOX : st;
            tma_2d(to, &map_w, kb * 128, p.n0, bar);
            if (GLU) tma_2d(to + (ROWS_X ? S::COL_BOX : S::LANE_BOX), &map_u, kb * 128, p.n0, bar);
        };
        auto rows = [&](uint8_t* st, const Piece& p, int kb, uint64_t* bar) {
            tma_2d(ROWS_X ? st : st + S::LANE_BOXES * S::LANE_BOX, &map_x, kb * 128, p.m0, bar);
        };
        Line l = line();
        Piece p;
        uint32_t it = 0;
        bool first = true;
        while (next(l, p)) {
            int kb = p.kb0;
            if (first) {  // weights do not depend on the kernel before: the ring is filled with them, then X is waited for
                const int pre = min(DEPTH, p.kb1 - p.kb0);
                if (leader)
                    for (int i = 0; i < pre; ++i) {
                        bar_expect(&full[i], S::STAGE);
                        weights(smem + i * S::STAGE, p, p.kb0 + i, &full[i]);
                    }
                __syncwarp();
                pdl_wait();
                if (leader)
                    for (int i = 0; i < pre; ++i) rows(smem + i * S::STAGE, p, p.kb0 + i, &full[i]);
                __syncwarp();
                it = pre, kb += pre, first = false;
            }
            for (; kb < p.kb1 && ok; ++kb, ++it) {
                const uint32_t s = it % DEPTH;
                if (it >= DEPTH) bar_wait(&empty[s], (it / DEPTH - 1) & 1, ok);
                if (!ok) break;
                if (leader) {
                    bar_expect(&full[s], S::STAGE);
                    weights(smem + s * S::STAGE, p, kb, &full[s]);
                    rows(smem + s * S::STAGE, p, kb, &full[s]);
                }
                __syncwarp();
            }
            if (!ok) break;
        }
        if (!ok) {  // no copy lands behind the CTA's end
            const uint32_t stop = it;
            for (uint32_t j = stop > DEPTH ? stop - DEPTH : 0; j < stop; ++j) {
                bool o = true;
                bar_wait(&full[j % DEPTH], (j / DEPTH) & 1, o);
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------- products ----
        const bool leader = elect();
        constexpr uint32_t ID = idesc(128, GLU && ROWS_X ? 2 * BN : BN);
        Line l = line();
        Piece p;
        uint32_t it = 0;
        while (next(l, p))
            for (int kb = p.kb0; kb < p.kb1; ++kb, ++it) {
                const uint32_t s = it % DEPTH, b = it & 1;
                if (it >= 2) bar_wait(&sempty[b], (it / 2 - 1) & 1, ok);
                bar_wait(&full[s], (it / DEPTH) & 1, ok);
                fence_after();
                if (leader) {
                    if (ok) {
                        const uint32_t at = smem_at(smem + s * S::STAGE), d = tmem + b * SETS * BN;
                        const uint64_t da = desc(at), db = desc(at + S::LANE_BOXES * S::LANE_BOX);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {  // 32 codes each: 32 bytes further inside the swizzle atom
                            mma(d, da + 2 * k, db + 2 * k, ID, k > 0);
                            if (GLU && !ROWS_X) mma(d + BN, da + S::LANE_BOX / 16 + 2 * k, db + 2 * k, ID, k > 0);
                        }
                    }
                    commit(&empty[s]);
                    commit(&sfull[b]);
                }
                __syncwarp();
            }
        // every product issued has completed before TMEM is released
        if (leader) commit(done);
        __syncwarp();
        bool last = true;
        bar_wait(done, 0, last);
    } else {
        // ------------------------------------------------- sums by their scales ----
        const int aw = warp - 2, quarter = warp & 3, half = aw >> 2;  // lanes, columns
        const int r = quarter * 32 + lane;                            // the thread's row of the lanes' side
        const uint32_t my = tmem + ((uint32_t)(quarter * 32) << 16) + half * HC;
        float* table = reinterpret_cast<float*>(smem + S::OFF_TABLE) + aw * (4 * SETS * HC);
        constexpr int CH = HC < 32 ? HC : 32, PER = (HC + 31) / 32;
        float2 acc[SETS][HC / 2];
        float* parts = reinterpret_cast<float*>(static_cast<uint32_t*>(a.workspace) + kCounters);
        pdl_wait();

        auto write = [&](const Piece& p) {
#pragma unroll
            for (int c = 0; c < HC; ++c) {
                const int m = ROWS_X ? p.m0 + r : p.m0 + half * HC + c, n = ROWS_X ? p.n0 + half * HC + c : p.n0 + r;
                if (m >= a.M || n >= a.N) continue;
                float v = c & 1 ? acc[0][c / 2].y : acc[0][c / 2].x;
                if (GLU) v = silu_f32(v) * (c & 1 ? acc[SETS - 1][c / 2].y : acc[SETS - 1][c / 2].x);
                const int64_t at = (int64_t)m * a.N + n;
                if (a.residual) v += bf16lo_to_f32(a.residual[at]);
                store_out(a.y, at, v, a.out_f32);
            }
        };

        Line l = line();
        Piece p;
        uint32_t it = 0;
        while (next(l, p)) {
#pragma unroll
            for (int s = 0; s < SETS; ++s)
#pragma unroll
                for (int c = 0; c < HC / 2; ++c) acc[s][c] = make_float2(0.f, 0.f);
            // scales of 4 blocks at a time, the next ones on their way
            const int nb = ROWS_X ? (p.n0 + (GLU ? 0 : half * HC)) / 128 : p.n0 / 128;
            const bool nb_there = nb * 128 < a.N;
            const float* wsp = a.ws + (int64_t)nb * KB;
            const float* usp = a.us + (int64_t)nb * KB;
            constexpr int XR = ROWS_X ? 1 : PER;
            float xs[XR][4], ws[4], us[4];
            auto fetch = [&](int kb) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool there = kb + i < p.kb1;
                    ws[i] = there && nb_there ? __ldg(wsp + kb + i) : 0.f;
                    us[i] = GLU && there && nb_there ? __ldg(usp + kb + i) : 0.f;
#pragma unroll
                    for (int j = 0; j < XR; ++j) {
                        const int m = ROWS_X ? p.m0 + r : p.m0 + half * HC + lane + 32 * j;
                        const bool has = there && m < a.M && (ROWS_X || lane + 32 * j < HC);
                        xs[j][i] = has ? a.xs[(int64_t)m * KB + kb + i] : 0.f;
                    }
                }
            };
            fetch(p.kb0);
            float f4[4], g4[4];  // ROWS_X: the row's factors
            for (int kb = p.kb0; kb < p.kb1; ++kb, ++it) {
                const int i = (kb - p.kb0) & 3;
                if (i == 0) {
                    if (ROWS_X) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) f4[q] = xs[0][q] * ws[q], g4[q] = GLU ? xs[0][q] * us[q] : 0.f;
                    } else {
                        __syncwarp();  // the factors before are read
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int j = 0; j < XR; ++j)
                                if (HC >= 32 || lane < HC) {
                                    table[q * SETS * HC + lane + 32 * j] = xs[j][q] * ws[q];
                                    if (GLU) table[q * SETS * HC + HC + lane + 32 * j] = xs[j][q] * us[q];
                                }
                        __syncwarp();
                    }
                    fetch(kb + 4);
                }
                const float f = i & 2 ? (i & 1 ? f4[3] : f4[2]) : (i & 1 ? f4[1] : f4[0]);
                const float g = i & 2 ? (i & 1 ? g4[3] : g4[2]) : (i & 1 ? g4[1] : g4[0]);
                const uint32_t b = it & 1;
                bar_wait(&sfull[b], (it / 2) & 1, ok);
                fence_after();
#pragma unroll
                for (int s = 0; s < SETS; ++s)
#pragma unroll
                    for (int c0 = 0; c0 < HC; c0 += CH) {
                        uint32_t v[CH];
                        ld<CH>(v, my + b * SETS * BN + s * BN + c0);
                        wait_ld<CH>(v);
                        if (s == SETS - 1 && c0 + CH >= HC) {
                            fence_before();
                            __syncwarp();
                            if (lane == 0) bar_arrive(&sempty[b]);
                        }
#pragma unroll
                        for (int c = 0; c < CH; c += 4) {
                            float2 f0, f1;
                            if (ROWS_X) {
                                f0 = f1 = s ? make_float2(g, g) : make_float2(f, f);
                            } else {
                                const float4 t = *reinterpret_cast<const float4*>(table + (i * SETS + s) * HC + c0 + c);
                                f0 = make_float2(t.x, t.y), f1 = make_float2(t.z, t.w);
                            }
                            float2* to = &acc[s][(c0 + c) / 2];
                            to[0] = fma2(make_float2(__uint_as_float(v[c]), __uint_as_float(v[c + 1])), f0, to[0]);
                            to[1] = fma2(make_float2(__uint_as_float(v[c + 2]), __uint_as_float(v[c + 3])), f1, to[1]);
                        }
                    }
            }
            if (p.kb0 == 0 && p.kb1 == KB) {
                write(p);
                continue;
            }
            // ---- a part of a tile; the CTA that arrives last adds them in their order ----
            const long long t0 = p.tile * KB;
            const int from = owner_of(t0), to = owner_of(t0 + KB - 1);
            {
                float* part = parts + (size_t)(2 * blockIdx.x + (p.kb0 == 0)) * S::PART;
#pragma unroll
                for (int s = 0; s < SETS; ++s)
#pragma unroll
                    for (int c = 0; c < HC; ++c)
                        part[(s * BN + half * HC + c) * 128 + r] = c & 1 ? acc[s][c / 2].y : acc[s][c / 2].x;
            }
            __threadfence();
            bar_adders();
            if (tid == 64) {
                const uint32_t n = to - from;
                sh_last = atomicInc(static_cast<uint32_t*>(a.workspace) + from, n) == n;  // back to 0 behind the last
                __threadfence();
            }
            bar_adders();
            if (sh_last) {
#pragma unroll
                for (int s = 0; s < SETS; ++s)
#pragma unroll
                    for (int c = 0; c < HC / 2; ++c) acc[s][c] = make_float2(0.f, 0.f);
                for (int i = from; i <= to; ++i) {
                    const float* part = parts + (size_t)(2 * i + (i == from)) * S::PART;
#pragma unroll
                    for (int s = 0; s < SETS; ++s)
#pragma unroll
                        for (int c = 0; c < HC; ++c) {
                            const float v = __ldcg(part + (s * BN + half * HC + c) * 128 + r);
                            if (c & 1)
                                acc[s][c / 2].y += v;
                            else
                                acc[s][c / 2].x += v;
                        }
                }
                write(p);
            }
            bar_adders();  // sh_last is read
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::COLS));
}

// ------------------------------------------------------------ host side ----
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool got = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                         q == cudaDriverEntryPointSuccess;
        return got ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return fn;
}

// Codes [rows][K], boxes of 128 k x `box` rows with 128-byte swizzle; rows past the end read zeros.
bool encode(CUtensorMap* map, const uint8_t* base, int64_t K, int64_t rows, int box) {
    const auto enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)K};
    const cuuint32_t size[2] = {128, (cuuint32_t)box}, one[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, size, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool ROWS_X, int BN, bool GLU>
cudaError_t launch(const Fp8Args& a, cudaStream_t s) {
    using S = Shape<ROWS_X, BN, GLU>;
    CUtensorMap mx, mw, mu;
    if (!encode(&mx, a.X, a.K, a.M, ROWS_X ? 128 : BN) || !encode(&mw, a.W, a.K, a.N, ROWS_X ? BN : 128) ||
        !encode(&mu, GLU ? a.U : a.W, a.K, a.N, ROWS_X ? BN : 128))
        return cudaErrorInvalidValue;
    auto* fn = gemm_fp8_kernel<ROWS_X, BN, GLU>;
    const cudaError_t err = kv4_allow_smem((const void*)fn, S::SMEM);
    if (err != cudaSuccess) return err;
    const int64_t tiles = ROWS_X ? ((a.M + 127) / 128) * (((int64_t)a.N + BN - 1) / BN) : (((int64_t)a.M + BN - 1) / BN) * ((a.N + 127) / 128);
    const int sms = device_sm_count() < kCounters ? device_sm_count() : kCounters;
    const size_t need = kCounters * sizeof(uint32_t) + (size_t)2 * sms * S::PART * sizeof(float);
    int split = !ROWS_X && a.ws_bytes >= need ? 1 : 0;
    const int64_t most = split ? tiles * (a.K / 128) : tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(most < sms ? most : sms), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attrs[1];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, fn, mx, mw, mu, a, (const int)split);
}

template <bool GLU>
cudaError_t launch_for(const Fp8Args& a, cudaStream_t s) {
    if (a.M <= 16) return launch<false, 16, GLU>(a, s);
    if (a.M <= 32) return launch<false, 32, GLU>(a, s);
    if (a.M <= 64) return launch<false, 64, GLU>(a, s);
    if (a.M <= 128) return launch<false, 128, GLU>(a, s);
    return launch<true, 128, GLU>(a, s);
}

}  // namespace

size_t gemm_fp8_workspace() {
    const int sms = device_sm_count() < kCounters ? device_sm_count() : kCounters;
    return kCounters * sizeof(uint32_t) + (size_t)2 * sms * Shape<false, 128, true>::PART * sizeof(float);
}

cudaError_t launch_gemm_fp8(const Fp8Args& a, cudaStream_t s) { return a.U ? launch_for<true>(a, s) : launch_for<false>(a, s); }

int gemm_fp8_take_fault() {
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_f8_fault, sizeof(int)) != cudaSuccess) return -1;
    if (v) cudaMemcpyToSymbol(g_f8_fault, &z, sizeof(int));
    return v;
}

}  // namespace mbw
