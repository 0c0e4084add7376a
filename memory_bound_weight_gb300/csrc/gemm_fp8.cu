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
// Gated: a second matrix U of W's shape, two sums a tile, y = silu(W sum) (U sum).
//
// A pair of CTAs takes a tile of 256 rows of X by 256 rows of W (cta_group::2), or 128
// of W and the same 128 of U. Each stages its own 128 rows of X and half of the other
// side (gated: one W, the other U), 32 KB a block of k, where a CTA alone would need 48
// for as many products, adds its 128 lanes x 256 columns into registers, 128 a thread,
// and writes them. A CTA is 12 warps: one that issues the copies, two (the even CTA's)
// that issue the products of both, one that multiplies the scales, 8 that add. The
// columns are two halves, each with its accumulators, barriers, issuing warp and adders,
// so that one's products run while the other's sums are on their way (4096 x 3584 x
// 18944: 216 us as one, 212 as two).
//
// Where there are fewer tiles than pairs, k is cut between up to four pairs of a
// cluster, whose sums are joined in order through their shared memory.
//
// What bounds it: a block of k takes a pair some 0.36 us, 650 clocks of products and, as
// there are but two accumulators, a part of the way from a product's end to the adders
// and back (commit 380, reading 290, arrival 250). 4096 x 3584 x 18944 is 198 us, 2810
// TFLOP/s, of which the products alone would take 145. (As it was at 212 us, without the
// additions it took 202, without any reading of accumulators 188, and its copies alone 158,
// 13.8 TB/s from L2. Since then who has given up a wait leaves the loop of the products,
// which no longer asks for each block whether it has.)
//
// Up to 128 rows of X are a second kernel's (Few below), up to 8, or 16, gemv_fp8.cu's.
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
// An accumulator is read. Relaxed: what it orders, reads of TMEM before the next products, the tcgen05 fence does, and a
// release would wait for the warp's loads of scales (256 x 256 tiles: 1.28 us a block of k instead of 0.58).
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_at(bar)), "r"(bytes) : "memory");
}
// A bounded wait by a warp, whose lanes give up together (the last round of some may see what that of others did not). Who
// has given up once waits no more, and every role comes to its end: the issuers of copies and of products issue nothing
// more, and neither they nor the adders, who go on over what is there, give anything back: the others then give up by
// themselves, and nobody takes a barrier's phase for one that it is not.
__device__ __forceinline__ void bar_wait(uint64_t* bar, uint32_t parity, bool& ok) {
    bool got = !ok;
    for (int i = 0; i < MBW_WAIT_LIMIT && !got; ++i) {
        uint32_t r;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(r) : "r"(smem_at(bar)), "r"(parity) : "memory");
        got = r != 0;
    }
    if (!__all_sync(0xFFFFFFFFu, got)) atomicExch(&g_f8_fault, 1), ok = false;
}
// Whether a phase is over, without waiting; to be looked at later (all_of), when the answer is there.
__device__ __forceinline__ uint32_t bar_ask(uint64_t* bar, uint32_t parity) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r) : "r"(smem_at(bar)), "r"(parity) : "memory");
    return r;
}
__device__ __forceinline__ bool all_of(uint32_t r) { return __all_sync(0xFFFFFFFFu, r != 0); }
__device__ __forceinline__ bool elect() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
template <int CTAS = 1>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if (CTAS == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_at(bar)) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_at(bar)) : "memory");
}
// The end of a warp that issues products, whoever has given up: its own are complete before the TMEM they write is released.
template <int CTAS = 1>
__device__ __forceinline__ void drain_products(uint64_t* bar, bool leader) {
    if (leader) commit<CTAS>(bar);
    __syncwarp();
    bool ok = true;
    bar_wait(bar, 0, ok);
}
// The end of a warp that issues copies, likewise: the last turn of each stage, of `it` in all, is over on `bars`, so that no copy
// lands behind the CTA's end, or on the sums that take the ring's place.
__device__ __forceinline__ void drain_copies(uint64_t* bars, uint32_t it, uint32_t depth) {
    bool ok = true;
    for (uint32_t j = it > depth ? it - depth : 0; j < it; ++j) bar_wait(&bars[j % depth], (j / depth) & 1, ok);
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



// silu to some 2^-21: e^-v as a power of two whose exponent's rounding is put back, and an approximate quotient. (With expf and
// the exact quotient a gated tile of 61 rows took 9 us to write.)
__device__ __forceinline__ float silu(float v) {
    const float h = v * -1.44269504f, l = fmaf(v, -1.44269504f, -h) - v * 1.92596299e-8f;
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(h));
    if (fabsf(h) < 127.f) e = fmaf(e, l * 0.693147181f, e);  // beyond, it is zero or infinite beside 1
    return __fdividef(v, 1.f + e);
}

// Eight outputs of a row, `left` of them inside the matrix; wide: they and the residual's lie on 16 bytes as bf16, and `held`
// are the residual's.
__device__ __forceinline__ void put8(const Fp8Args& a, int64_t at, float* o, int left, bool wide, uint4 held) {
    if (wide && left >= 8) {
        if (a.residual) {
            const uint32_t w[4] = {held.x, held.y, held.z, held.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) o[2 * i] += bf16lo_to_f32(w[i]), o[2 * i + 1] += bf16hi_to_f32(w[i]);
        }
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + at) = make_uint4(w[0], w[1], w[2], w[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) {
            if (a.residual) o[i] += bf16lo_to_f32(a.residual[at + i]);
            store_out(a.y, at + i, o[i], a.out_f32);
        }
}

constexpr int kMaxSplit = 4;  // pairs that share a tile's k
constexpr int kFewSplit = 8;  // CTAs that share a tile's k, where a CTA takes all rows of X
constexpr int kAdders = 8, kThreads = (4 + kAdders) * 32;
// Registers: 168 a thread at launch; then by warpgroup 56 for the issuers and 2 x 224 for the adders, 504 = 3 x 168.
constexpr int kRegsLaunch = 168, kRegsIssuers = 56, kRegsAdders = 224;
static_assert(4 * kRegsIssuers + kAdders * kRegsAdders <= (4 + kAdders) * kRegsLaunch, "");
constexpr int kStage = 2 * 128 * 128, kDepth = 6;
// Factors of four blocks of k by [block][row], two each: of the columns of the even CTA's W and of the odd one's W or U.
constexpr int kGroups = 4, kGroup = 4 * 128 * 8;
constexpr int kOffFactor = kDepth * kStage, kOffBar = kOffFactor + kGroups * kGroup, kSmem = kOffBar + (2 * kDepth + 8 + 2 * kGroups + 2) * 8 + 16 + 1024;
constexpr int kPitch = 260;  // floats of a row that the CTAs of a cluster are joined in: 4 to spread the banks
static_assert(kSmem <= 227 * 1024, "");
static_assert(128 * kPitch * 4 <= kOffFactor, "over the ring, which is drained then");

template <int N>
__device__ __forceinline__ void registers(bool more) {
    if (more)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <bool GLU>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                    const __grid_constant__ CUtensorMap map_u, const Fp8Args a) {
    constexpr int OUT = GLU ? 128 : 256;  // columns of Y a tile has
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-smem_at(smem_raw) & 1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);  // the even CTA's count both of the pair
    uint64_t *empty = full + kDepth, *sfull = empty + kDepth, *sempty = sfull + 4;  // sempty: the even CTA's count both
    uint64_t *ffull = sempty + 4, *fempty = ffull + kGroups, *done = fempty + kGroups;  // of factors; of all products
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 2);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t crank, csize;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(crank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
    const int rank = crank & 1, split = csize / 2;  // of the pair; pairs that share a tile's k
    bool ok = true;

    if (tid == 0) {
        for (int i = 0; i < kDepth; ++i) bar_init(&full[i], 1), bar_init(&empty[i], 2);
        for (int i = 0; i < 4; ++i) bar_init(&sfull[i], 1), bar_init(&sempty[i], kAdders);
        for (int i = 0; i < kGroups; ++i) bar_init(&ffull[i], 1), bar_init(&fempty[i], kAdders);
        bar_init(&done[0], 1), bar_init(&done[1], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_at(tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    cluster_sync();  // the peer's barriers exist before any copy, arrival or commit reaches them
    fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();

    // ---- a pair takes whole tiles in turn, or of one tile its share of the blocks of k ----
    const int KB = a.K / 128, tiles_m = (a.M + 255) / 256, tiles_n = (a.N + OUT - 1) / OUT;
    const long long tiles = (long long)tiles_m * tiles_n, first = blockIdx.x / csize, stride = gridDim.x / csize;
    const int kb0 = (int)((long long)KB * (crank / 2) / split), kb1 = (int)((long long)KB * (crank / 2 + 1) / split);
    auto tile_n = [&](long long t) { return (int)(t / tiles_m); };  // tiles of one W one behind the other
    auto tile_m0 = [&](long long t) { return (int)(t % tiles_m) * 256 + rank * 128; };
    auto even = [&](const void* p) {  // its address in the pair's even CTA
        uint32_t r;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_at(p)), "r"(crank & ~1u));
        return r;
    };

    if (warp < 4) {
        registers<kRegsIssuers>(false);
        if (warp == 0) {
            // -------------------------------------------------------- copies ----
            const bool leader = elect();
            const uint32_t full0 = even(full);
            auto copy = [&](uint8_t* dst, const CUtensorMap* map, int c0, int c1, uint32_t s) {
                asm volatile(
                    "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(
                        smem_at(dst)),
                    "l"(map), "r"(c0), "r"(c1), "r"(full0 + 8 * s)
                    : "memory");
            };
            const CUtensorMap* w = GLU && rank ? &map_u : &map_w;
            uint32_t it = 0;
            for (long long t = first; t < tiles && ok; t += stride) {
                const int n0 = tile_n(t) * OUT + (GLU ? 0 : rank * 128), m0 = tile_m0(t);
                int kb = kb0;
                if (t == first) {  // weights do not depend on the kernel before: the ring is filled with them, then X is waited for
                    const int pre = min(kDepth, kb1 - kb0);
                    if (leader)
                        for (int i = 0; i < pre; ++i) {
                            if (rank == 0) bar_expect(&full[i], 2 * kStage);
                            copy(smem + i * kStage + 128 * 128, w, (kb + i) * 128, n0, i);
                        }
                    __syncwarp();
                    pdl_wait();
                    if (leader)
                        for (int i = 0; i < pre; ++i) copy(smem + i * kStage, &map_x, (kb + i) * 128, m0, i);
                    __syncwarp();
                    it = pre, kb += pre;
                }
                for (; kb < kb1; ++kb, ++it) {
                    const uint32_t s = it % kDepth;
                    if (it >= kDepth) bar_wait(&empty[s], (it / kDepth - 1) & 1, ok);
                    if (!ok) break;
                    if (leader) {
                        if (rank == 0) bar_expect(&full[s], 2 * kStage);
                        copy(smem + s * kStage + 128 * 128, w, kb * 128, n0, s);
                        copy(smem + s * kStage, &map_x, kb * 128, m0, s);
                    }
                    __syncwarp();
                }
            }
            // Both CTAs' copies complete on the even one's `full`; the odd one, which has none, waits for its stages' products.
            drain_copies(rank == 0 ? full : empty, it, kDepth);
        } else if (warp <= 2) {
            if (rank == 0) {
            const int h = warp - 1;
            // ------------------------------------------------------ products ----
            const bool leader = elect();
            constexpr uint32_t ID = idesc(256, 128);
            auto commit2 = [&](uint64_t* bar) {
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_at(bar)),
                             "h"((uint16_t)(3 << crank))
                             : "memory");
            };
            uint32_t it = 0, s = 0, turn = 0, there = 0;  // the stage, the ring's turns before it, and whether it is full
            for (long long t = first; t < tiles && ok; t += stride)
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const uint32_t b = it & 1;
                    const uint32_t free = it < 2 ? 1u : bar_ask(&sempty[2 * b + h], (it / 2 - 1) & 1);
                    if (!all_of(there)) bar_wait(&full[s], turn & 1, ok);
                    if (!all_of(free)) bar_wait(&sempty[2 * b + h], (it / 2 - 1) & 1, ok);
                    if (!ok) break;
                    fence_after();
                    const uint32_t cur = s;
                    if (++s == kDepth) s = 0, ++turn;
                    there = bar_ask(&full[s], turn & 1);  // the next one's answer comes under the products' issue
                    if (leader) {
                        const uint64_t da = desc(smem_at(smem + cur * kStage)), db = da + (128 + 64 * h) * 128 / 16;
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // 32 codes each: 32 bytes further inside the swizzle atom
                            asm volatile(
                                "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(
                                    tmem + b * 256 + h * 128),
                                "l"(da + 2 * k), "l"(db + 2 * k), "r"(ID), "r"(k > 0 ? 1u : 0u)
                                : "memory");
                        commit2(&sfull[2 * b + h]);
                        commit2(&empty[cur]);
                    }
                    __syncwarp();
                }
            drain_products<2>(&done[h], leader);
            }
        } else {
            // ------------------------------------------------------- factors ----
            // by a warp of its own: the loads, 32 rows apart, held the adders up by a fifth
            const bool by4 = KB % 4 == 0 && (((uintptr_t)a.xs | (uintptr_t)a.ws | (GLU ? (uintptr_t)a.us : 0)) & 15) == 0;
            auto fetch = [&](const float* from, int kb, bool there) {
                if (by4) return there ? *reinterpret_cast<const float4*>(from + kb) : make_float4(0.f, 0.f, 0.f, 0.f);
                return make_float4(there ? from[kb] : 0.f, there && kb + 1 < KB ? from[kb + 1] : 0.f, there && kb + 2 < KB ? from[kb + 2] : 0.f,
                                   there && kb + 3 < KB ? from[kb + 3] : 0.f);
            };
            pdl_wait();
            uint32_t turn = 0;
            for (long long t = first; t < tiles; t += stride) {
                const int m0 = tile_m0(t), nb = tile_n(t) * (OUT / 128);
                const bool cols = nb * 128 < a.N, cols2 = GLU ? cols : (nb + 1) * 128 < a.N;
                const float *wsp = a.ws + (int64_t)nb * KB, *usp = GLU ? a.us + (int64_t)nb * KB : wsp + KB;
                for (int kb = kb0 & ~3; kb < kb1; kb += 4, ++turn) {
                    const float4 ws = fetch(wsp, kb, cols), us = fetch(usp, kb, cols2);
                    float4 xs[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int m = m0 + i * 32 + lane;
                        xs[i] = fetch(a.xs + (int64_t)m * KB, kb, m < a.M);
                    }
                    const uint32_t slot = turn % kGroups;
                    if (turn >= kGroups) bar_wait(&fempty[slot], (turn / kGroups - 1) & 1, ok);
                    float2* to = reinterpret_cast<float2*>(smem + kOffFactor + slot * kGroup) + lane;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        to[i * 32] = make_float2(xs[i].x * ws.x, xs[i].x * us.x), to[i * 32 + 128] = make_float2(xs[i].y * ws.y, xs[i].y * us.y);
                        to[i * 32 + 256] = make_float2(xs[i].z * ws.z, xs[i].z * us.z), to[i * 32 + 384] = make_float2(xs[i].w * ws.w, xs[i].w * us.w);
                    }
                    __syncwarp();
                    if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_at(&ffull[slot])) : "memory");
                }
            }
        }
    } else {
        // ------------------------------------------------- sums by their scales ----
        registers<kRegsAdders>(true);
        const int quarter = warp & 3, half = (warp - 4) >> 2, r = quarter * 32 + lane;
        const uint32_t my = tmem + ((uint32_t)(quarter * 32) << 16) + half * 128;
        const uint32_t sempty0 = even(sempty + half);
        auto column = [](int j) { return 32 * j; };  // of the j-th 32 of the thread's columns
        float2 acc[64];  // 64 columns of the even CTA's W, 64 of the odd one's W or U
        uint32_t v[2][32];
        pdl_wait();
        const bool wide = a.N % 8 == 0 && !a.out_f32 && ((uintptr_t)a.residual & 15) == 0;
        uint32_t it = 0, group = 0;
        for (long long t = first; t < tiles; t += stride) {
            const int m = tile_m0(t) + r, n0 = tile_n(t) * OUT + half * 64;
            const bool row = m < a.M;
#pragma unroll
            for (int c = 0; c < 64; ++c) acc[c] = make_float2(0.f, 0.f);
            float2 fg[4];  // factors of four blocks
            bool begun = false;  // the first 32 columns of the next block are on their way
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const uint32_t b = it & 1, at = my + b * 256;
                if (!begun) {
                    bar_wait(&sfull[2 * b + half], (it / 2) & 1, ok);
                    fence_after();
                    ld<32>(v[0], at);
                }
                if ((kb & 3) == 0 || kb == kb0) {
                    const uint32_t slot = group % kGroups;
                    bar_wait(&ffull[slot], (group / kGroups) & 1, ok);
                    const float2* from = reinterpret_cast<const float2*>(smem + kOffFactor + slot * kGroup) + r;
#pragma unroll
                    for (int i = 0; i < 4; ++i) fg[i] = from[128 * i];
                    __syncwarp();
                    if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_at(&fempty[slot])) : "memory");
                    __syncwarp();  // the wait for loads below is the warp's
                    ++group;
                }
                const float2 now = kb & 2 ? (kb & 1 ? fg[3] : fg[2]) : (kb & 1 ? fg[1] : fg[0]);
                uint32_t ready = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    wait_ld<32>(v[j & 1]);
                    if (j < 3) {
                        ld<32>(v[(j + 1) & 1], at + column(j + 1));
                    } else {
                        fence_before();
                        __syncwarp();
                        if (lane == 0 && ok) bar_arrive(sempty0 + 16 * b);
                        if (kb + 1 < kb1) ready = bar_ask(&sfull[2 * (b ^ 1) + half], ((it + 1) / 2) & 1);
                    }
                    const float2 ff = j >= 2 ? make_float2(now.y, now.y) : make_float2(now.x, now.x);
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        acc[16 * j + c] = fma2(make_float2(__uint_as_float(v[j & 1][2 * c]), __uint_as_float(v[j & 1][2 * c + 1])), ff, acc[16 * j + c]);
                }
                begun = all_of(ready);
                if (begun) {
                    fence_after();
                    ld<32>(v[0], my + (b ^ 1) * 256);
                }
            }
            if (split > 1) {  // into shared memory, [row][column]
                asm volatile("bar.sync 1, %0;" ::"n"(kAdders * 32) : "memory");  // both halves' products have read the ring
                float* to = reinterpret_cast<float*>(smem) + r * kPitch + half * 64;
                if (ok)  // else copies may be on their way there
#pragma unroll
                    for (int c = 0; c < 128; c += 4)
                        *reinterpret_cast<float4*>(to + (c >= 64 ? 64 + c : c)) = make_float4(acc[c / 2].x, acc[c / 2].y, acc[c / 2 + 1].x, acc[c / 2 + 1].y);
            } else if (row) {
                const int64_t to = (int64_t)m * a.N + n0;
                constexpr int COLUMNS = GLU ? 64 : 128;
                // The residual's values are read some ahead: it may be the output, and no load is moved before a store by itself
                // (4096 x 3584 x 18944 with a residual, now 205 to 211 us: 228 one by one, 222 four ahead, 221 eight, 235 the whole row,
                // whose registers do not fit).
                constexpr int HELD = 8;
                uint4 held[HELD];
#pragma unroll
                for (int c = 0; c < COLUMNS; c += 8) {
                    if (c / 8 % HELD == 0) {
#pragma unroll
                        for (int i = 0; i < HELD; ++i) {
                            const int off = c + 8 * i >= 64 ? 64 + c + 8 * i : c + 8 * i;
                            held[i] = make_uint4(0, 0, 0, 0);
                            if (wide && a.residual && a.N - n0 - off >= 8) held[i] = *reinterpret_cast<const uint4*>(a.residual + to + off);
                        }
                    }
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 x = acc[(c + i) / 2];
                        o[i] = i & 1 ? x.y : x.x;
                        if (GLU) {
                            const float2 u = acc[32 + ((c + i) / 2) % 32];
                            o[i] = silu(o[i]) * (i & 1 ? u.y : u.x);
                        }
                    }
                    const int off = c >= 64 ? 64 + c : c;
                    put8(a, to + off, o, a.N - n0 - off, wide, held[c / 8 % HELD]);
                }
            }
        }
    }
    if (split > 1) {
        // ---- the pairs' sums in their order, each CTA a share of the columns of its rows ----
        fence_before();
        cluster_sync();
        fence_after();
        if (warp >= 4) {
            const int m0 = tile_m0(first), rows = min(128, a.M - m0), n0 = tile_n(first) * OUT;
            const int g0 = OUT / 4 * (int)(crank / 2) / split, groups = OUT / 4 * (int)(crank / 2 + 1) / split - g0;  // of 4 columns
            const bool four = a.N % 4 == 0 && !a.out_f32 && ((uintptr_t)a.residual & 7) == 0;
            for (int e = tid - 128; e < rows * groups; e += kAdders * 32) {
                const int row = e / groups, c = (g0 + e % groups) * 4;
                const uint32_t at = smem_at(reinterpret_cast<float*>(smem) + row * kPitch + c);
                float4 x[kMaxSplit][GLU ? 2 : 1];  // all on their way before the first is added
#pragma unroll
                for (int q = 0; q < kMaxSplit; ++q) {
                    if (q >= split) break;
                    uint32_t from;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(at), "r"(2 * q + rank));
#pragma unroll
                    for (int u = 0; u < (GLU ? 2 : 1); ++u)
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(x[q][u].x), "=f"(x[q][u].y), "=f"(x[q][u].z), "=f"(x[q][u].w) : "r"(from + u * 512) : "memory");
                }
                const int64_t to = (int64_t)(m0 + row) * a.N + n0 + c;
                const int left = a.N - n0 - c;
                float res[4] = {0.f, 0.f, 0.f, 0.f};
                if (a.residual) {
                    if (four && left > 0) {
                        const uint2 h = *reinterpret_cast<const uint2*>(a.residual + to);
                        res[0] = bf16lo_to_f32(h.x), res[1] = bf16hi_to_f32(h.x), res[2] = bf16lo_to_f32(h.y), res[3] = bf16hi_to_f32(h.y);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i < left) res[i] = bf16lo_to_f32(a.residual[to + i]);
                    }
                }
                float o[2][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) o[0][i] = o[1][i] = 0.f;
#pragma unroll
                for (int q = 0; q < kMaxSplit; ++q)
                    if (q < split)
#pragma unroll
                        for (int u = 0; u < (GLU ? 2 : 1); ++u) o[u][0] += x[q][u].x, o[u][1] += x[q][u].y, o[u][2] += x[q][u].z, o[u][3] += x[q][u].w;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (GLU) o[0][i] = silu(o[0][i]) * o[1][i];
                    if (a.residual) o[0][i] += res[i];
                }
                if (four && left > 0) {
                    const __nv_bfloat162 h0 = __floats2bfloat162_rn(o[0][0], o[0][1]), h1 = __floats2bfloat162_rn(o[0][2], o[0][3]);
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + to) = make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < left) store_out(a.y, to + i, o[0][i], a.out_f32);
                }
            }
        }
    }
    fence_before();
    __syncthreads();
    cluster_sync();  // all CTAs are done with each other's memory, barriers and copies, and the pair with its TMEM
    fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Up to NX = 32, 64 or 128 rows of X: the weights are the products' rows, 128 a CTA, and X their columns, so that no product is
// of rows that are not there; a column of Y is a lane of the accumulator, of one weight scale a block. No pairs: X is small,
// and a CTA has a tile of W (gated: and U's) for itself. Two or four accumulators are in turn. k is cut between up to eight
// CTAs of a cluster.
// What bounds it: where each SM has one tile, W's stream from HBM and the start before it (32 x 152064 x 3584 85 us, 6.4 TB/s;
// 64 x 4608 x 3584 7.7 us, most of them a start and a join); a block of k takes 0.26 us for 64 rows, the issue of products
// and the adders' way through waits, loads and factors, and 0.42 for 128, most of it the adders'. (32 rows as 64: 18944 x
// 3584 16.0 us in place of 13.9, gated 5632 x 2048 11.3 in place of 9.7.) The gated form spills, 204 to 264 bytes a thread
// stored at the 168 registers of its launch.
template <bool GLU, int NX>
struct Few {
    static constexpr int MATS = GLU ? 2 : 1, STAGE = MATS * 128 * 128 + NX * 128, DEPTH = 208 * 1024 / STAGE;
    static constexpr int COLS = MATS * NX, NACC = 512 / COLS < 4 ? 512 / COLS : 4;  // TMEM columns of an accumulator, accumulators
    static constexpr int GROUP = 4 * COLS * 4;                                      // factors of four blocks by [block][matrix][row of X]
    static constexpr int OFF_FACTOR = DEPTH * STAGE, OFF_BAR = OFF_FACTOR + kGroups * GROUP;
    static constexpr int SMEM = OFF_BAR + (2 * DEPTH + 2 * NACC + 2 * kGroups + 2) * 8 + 16 + 1024;
    static_assert(SMEM <= 227 * 1024, "");
    static_assert(COLS * 128 * 4 <= OFF_FACTOR, "sums lie over the ring, which is drained then");
};

template <bool GLU, int NX>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp8_few_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                        const __grid_constant__ CUtensorMap map_u, const Fp8Args a) {
    using L = Few<GLU, NX>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-smem_at(smem_raw) & 1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
    uint64_t *empty = full + L::DEPTH, *sfull = empty + L::DEPTH, *sempty = sfull + L::NACC, *ffull = sempty + L::NACC, *fempty = ffull + kGroups;
    uint64_t* done = fempty + kGroups;  // of all products
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 2);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t crank, csize;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(crank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(csize));
    const int split = csize;  // CTAs that share a tile's k
    bool ok = true;

    if (tid == 0) {
        for (int i = 0; i < L::DEPTH; ++i) bar_init(&full[i], 1), bar_init(&empty[i], 1);
        for (int i = 0; i < L::NACC; ++i) bar_init(&sfull[i], 1), bar_init(&sempty[i], kAdders);
        for (int i = 0; i < kGroups; ++i) bar_init(&ffull[i], 1), bar_init(&fempty[i], kAdders);
        bar_init(&done[0], 1), bar_init(&done[1], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_at(tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();

    // ---- a CTA takes whole tiles of 128 columns of Y in turn, or of one tile its share of the blocks of k ----
    const int KB = a.K / 128, tiles = (a.N + 127) / 128, first = blockIdx.x / csize, stride = gridDim.x / csize;
    const int kb0 = (int)((long long)KB * crank / split), kb1 = (int)((long long)KB * (crank + 1) / split);

    if (warp < 4) {
        registers<kRegsIssuers>(false);
        if (warp == 0) {
            // -------------------------------------------------------- copies ----
            const bool leader = elect();
            auto weights = [&](uint32_t s, int kb, int n0) {
                bar_expect(&full[s], L::STAGE);
                tma_2d(smem + s * L::STAGE, &map_w, kb * 128, n0, &full[s]);
                if (GLU) tma_2d(smem + s * L::STAGE + 128 * 128, &map_u, kb * 128, n0, &full[s]);
            };
            auto rows = [&](uint32_t s, int kb) { tma_2d(smem + s * L::STAGE + L::MATS * 128 * 128, &map_x, kb * 128, 0, &full[s]); };
            uint32_t it = 0, s = 0, turn = 0;
            for (int t = first; t < tiles && ok; t += stride) {
                int kb = kb0;
                if (t == first) {  // weights do not depend on the kernel before: the ring is filled with them, then X is waited for
                    const int pre = min(L::DEPTH, kb1 - kb0);
                    if (leader)
                        for (int i = 0; i < pre; ++i) weights(i, kb + i, t * 128);
                    __syncwarp();
                    pdl_wait();
                    if (leader)
                        for (int i = 0; i < pre; ++i) rows(i, kb + i);
                    __syncwarp();
                    it = pre, kb += pre, s = pre % L::DEPTH, turn = pre / L::DEPTH;
                }
                for (; kb < kb1; ++kb, ++it) {
                    if (turn) bar_wait(&empty[s], (turn - 1) & 1, ok);
                    if (!ok) break;
                    if (leader) weights(s, kb, t * 128), rows(s, kb);
                    __syncwarp();
                    if (++s == L::DEPTH) s = 0, ++turn;
                }
            }
            drain_copies(full, it, L::DEPTH);
        } else if (warp <= 2) {
            // ------------------------------------------------------ products ----
            // by two warps in turn, since the issue of a block's takes a warp longer than the tensor pipe (64 rows, blocks of one
            // CTA: one warp 0.34 us, two 0.27)
            const bool leader = elect();
            constexpr uint32_t ID = idesc(128, NX);
            const uint32_t blocks = (uint32_t)((tiles - first + stride - 1) / stride) * (uint32_t)(kb1 - kb0);
            uint32_t s = warp - 1, turn = 0;  // the stage, and the ring's turns before it
            for (uint32_t it = warp - 1; it < blocks; it += 2) {
                const uint32_t b = it % L::NACC;
                if (s >= L::DEPTH) s -= L::DEPTH, ++turn;
                // The accumulator first: where it is free, block it - NACC has been added, so that the stage's turn before,
                // which may have been the other warp's, is over, and the parity waited for next is this turn's.
                static_assert(L::NACC % 2 == 0 && L::DEPTH >= L::NACC, "");
                if (it >= L::NACC) bar_wait(&sempty[b], (it / L::NACC - 1) & 1, ok);
                bar_wait(&full[s], turn & 1, ok);
                if (!ok) break;
                fence_after();
                if (leader) {
                    const uint64_t dw = desc(smem_at(smem + s * L::STAGE)), dx = dw + L::MATS * 128 * 128 / 16;
#pragma unroll
                    for (int u = 0; u < L::MATS; ++u)
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // 32 codes each: 32 bytes further inside the swizzle atom
                            mma(tmem + b * L::COLS + u * NX, dw + u * 128 * 128 / 16 + 2 * k, dx + 2 * k, ID, k > 0);
                    commit(&sfull[b]);
                    commit(&empty[s]);
                }
                __syncwarp();
                s += 2;
            }
            drain_products(&done[warp - 1], leader);
        } else {
            // ------------------------------------------------------- factors ----
            const bool by4 = KB % 4 == 0 && (((uintptr_t)a.xs | (uintptr_t)a.ws | (GLU ? (uintptr_t)a.us : 0)) & 15) == 0;
            auto fetch = [&](const float* from, int kb, bool there) {
                if (by4) return there ? *reinterpret_cast<const float4*>(from + kb) : make_float4(0.f, 0.f, 0.f, 0.f);
                return make_float4(there ? from[kb] : 0.f, there && kb + 1 < KB ? from[kb + 1] : 0.f, there && kb + 2 < KB ? from[kb + 2] : 0.f,
                                   there && kb + 3 < KB ? from[kb + 3] : 0.f);
            };
            pdl_wait();
            uint32_t turn = 0;
            for (int t = first; t < tiles; t += stride) {
                const float *wsp = a.ws + (int64_t)t * KB, *usp = GLU ? a.us + (int64_t)t * KB : wsp;
                for (int kb = kb0 & ~3; kb < kb1; kb += 4, ++turn) {
                    const float4 ws = fetch(wsp, kb, true), us = GLU ? fetch(usp, kb, true) : ws;
                    float4 xs[NX / 32];
#pragma unroll
                    for (int i = 0; i < NX / 32; ++i) xs[i] = fetch(a.xs + (int64_t)(i * 32 + lane) * KB, kb, i * 32 + lane < a.M);
                    const uint32_t slot = turn % kGroups;
                    if (turn >= kGroups) bar_wait(&fempty[slot], (turn / kGroups - 1) & 1, ok);
                    float* to = reinterpret_cast<float*>(smem + L::OFF_FACTOR + slot * L::GROUP) + lane;
#pragma unroll
                    for (int i = 0; i < NX / 32; ++i)
#pragma unroll
                        for (int u = 0; u < L::MATS; ++u) {
                            const float4 f = u ? us : ws;
                            float* at = to + u * NX + 32 * i;
                            at[0] = xs[i].x * f.x, at[L::COLS] = xs[i].y * f.y, at[2 * L::COLS] = xs[i].z * f.z, at[3 * L::COLS] = xs[i].w * f.w;
                        }
                    __syncwarp();
                    if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_at(&ffull[slot])) : "memory");
                }
            }
        }
    } else {
        // ------------------------------------------------- sums by their scales ----
        registers<kRegsAdders>(true);
        // A thread's columns are read in pieces, the next on its way under the additions of the one before: whole blocks, or
        // of the gated form of 128 rows, whose sums leave no registers, a quarter of one.
        constexpr int C = NX / 2, U = C < 32 ? C : 32, CHUNKS = C / U, UNITS = L::MATS * CHUNKS;  // columns of a thread; units of up to 32 of them, in all
        constexpr int P = UNITS <= 2 ? UNITS : 1, PIECES = UNITS / P;                             // units of a piece
        const int quarter = warp & 3, half = (warp - 4) >> 2, r = quarter * 32 + lane;
        const uint32_t my = tmem + ((uint32_t)(quarter * 32) << 16) + half * C;
        auto column = [](int i) { return i / CHUNKS * NX + i % CHUNKS * U; };  // of the i-th unit, among an accumulator's
        float2 acc[UNITS * U / 2];
        uint32_t v[2][P * U];
        pdl_wait();
        uint32_t it = 0, group = 0;
        auto fetch = [&](uint32_t(&to)[P * U], uint32_t at, int j) {
#pragma unroll
            for (int h = 0; h < P; ++h) ld<U>(to + U * h, at + column(j * P + h));
        };
        bool begun;  // the next block's first piece is on its way
        auto block = [&](int kb, uint32_t(&v0)[P * U], uint32_t(&v1)[P * U]) {
            const uint32_t b = it % L::NACC, next = (it + 1) % L::NACC;
            if (!begun) {
                bar_wait(&sfull[b], (it / L::NACC) & 1, ok);
                fence_after();
                fetch(v0, my + b * L::COLS, 0);
            }
            const uint32_t slot = group % kGroups;
            if ((kb & 3) == 0 || kb == kb0) bar_wait(&ffull[slot], (group / kGroups) & 1, ok);
            const float* f = reinterpret_cast<const float*>(smem + L::OFF_FACTOR + slot * L::GROUP) + (kb & 3) * L::COLS + half * C;
#pragma unroll
            for (int j = 0; j < PIECES; ++j) {
                auto& now = j & 1 ? v1 : v0;
                auto& then = j & 1 ? v0 : v1;
                const uint32_t ready = j + 1 == PIECES && kb + 1 < kb1 ? bar_ask(&sfull[next], ((it + 1) / L::NACC) & 1) : 0;
                wait_ld<P * U>(now);
                if (j + 1 < PIECES) {
                    fetch(then, my + b * L::COLS, j + 1);
                } else {
                    fence_before();
                    __syncwarp();
                    if (lane == 0 && ok) bar_arrive(smem_at(&sempty[b]));
                    begun = all_of(ready);
                    if (begun) {
                        fence_after();
                        fetch(then, my + next * L::COLS, 0);
                    }
                }
#pragma unroll
                for (int c = 0; c < P * U; c += 4) {
                    const float4 ff = *reinterpret_cast<const float4*>(f + column(j * P + c / U) + c % U);
                    float2* to = acc + (j * P * U + c) / 2;
                    to[0] = fma2(make_float2(__uint_as_float(now[c]), __uint_as_float(now[c + 1])), make_float2(ff.x, ff.y), to[0]);
                    to[1] = fma2(make_float2(__uint_as_float(now[c + 2]), __uint_as_float(now[c + 3])), make_float2(ff.z, ff.w), to[1]);
                }
            }
            if ((kb & 3) == 3 || kb + 1 == kb1) {
                __syncwarp();
                if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_at(&fempty[slot])) : "memory");
                ++group;
            }
            ++it;
        };
        for (int t = first; t < tiles; t += stride) {
#pragma unroll
            for (int c = 0; c < UNITS * U / 2; ++c) acc[c] = make_float2(0.f, 0.f);
            begun = false;
            for (int kb = kb0; kb < kb1; ++kb) {
                block(kb, v[0], v[1]);
                if (PIECES % 2 == 0) continue;  // the next block's first piece lies in the first again
                if (++kb == kb1) break;
                block(kb, v[1], v[0]);
            }
            if (split > 1) {  // into shared memory, [matrix][row of X][column of Y]
                float* to = reinterpret_cast<float*>(smem) + half * C * 128 + r;
                if (ok)  // else copies may be on their way there
#pragma unroll
                    for (int j = 0; j < UNITS; ++j)
#pragma unroll
                        for (int c = 0; c < U; ++c) to[(column(j) + c) * 128] = c & 1 ? acc[(j * U + c) / 2].y : acc[(j * U + c) / 2].x;
            } else if (t * 128 + r < a.N) {
                constexpr int HELD = 16;  // of the residual, ahead of the stores
                uint16_t held[HELD];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int m = half * C + c;
                    const int64_t to = (int64_t)m * a.N + t * 128 + r;
                    if (c % HELD == 0)
#pragma unroll
                        for (int i = 0; i < HELD; ++i) held[i] = a.residual && m + i < a.M ? a.residual[to + (int64_t)i * a.N] : (uint16_t)0;
                    float o = c & 1 ? acc[c / 2].y : acc[c / 2].x;
                    if constexpr (GLU) o = silu(o) * (c & 1 ? acc[(C + c) / 2].y : acc[(C + c) / 2].x);
                    if (a.residual) o += bf16lo_to_f32(held[c % HELD]);
                    if (m < a.M) store_out(a.y, to, o, a.out_f32);
                }
            }
        }
    }
    if (split > 1) {
        // ---- the CTAs' sums in their order, each CTA a share of the rows of X ----
        fence_before();
        cluster_sync();
        fence_after();
        if (warp >= 4) {
            const int m0 = a.M * (int)crank / split, items = (a.M * (int)(crank + 1) / split - m0) * 32;
            const bool four = a.N % 4 == 0 && !a.out_f32 && ((uintptr_t)a.residual & 7) == 0;
            for (int e = tid - 128; e < items; e += kAdders * 32) {
                const int m = m0 + e / 32, c = e % 32 * 4, left = a.N - first * 128 - c;
                const int64_t to = (int64_t)m * a.N + first * 128 + c;
                const uint32_t at = smem_at(reinterpret_cast<float*>(smem) + m * 128 + c);
                float res[4] = {0.f, 0.f, 0.f, 0.f};
                if (a.residual) {
                    if (four && left > 0) {
                        const uint2 h = *reinterpret_cast<const uint2*>(a.residual + to);
                        res[0] = bf16lo_to_f32(h.x), res[1] = bf16hi_to_f32(h.x), res[2] = bf16lo_to_f32(h.y), res[3] = bf16hi_to_f32(h.y);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i < left) res[i] = bf16lo_to_f32(a.residual[to + i]);
                    }
                }
                float4 x[kFewSplit][L::MATS];  // all on their way before the first is added
#pragma unroll
                for (int q = 0; q < kFewSplit; ++q) {
                    if (q >= split) break;
                    uint32_t from;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(at), "r"(q));
#pragma unroll
                    for (int u = 0; u < L::MATS; ++u)
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(x[q][u].x), "=f"(x[q][u].y), "=f"(x[q][u].z), "=f"(x[q][u].w) : "r"(from + u * NX * 512) : "memory");
                }
                float o[2][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) o[0][i] = o[1][i] = 0.f;
#pragma unroll
                for (int q = 0; q < kFewSplit; ++q)
                    if (q < split)
#pragma unroll
                        for (int u = 0; u < L::MATS; ++u) o[u][0] += x[q][u].x, o[u][1] += x[q][u].y, o[u][2] += x[q][u].z, o[u][3] += x[q][u].w;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (GLU) o[0][i] = silu(o[0][i]) * o[1][i];
                    if (a.residual) o[0][i] += res[i];
                }
                if (four && left > 0) {
                    const __nv_bfloat162 h0 = __floats2bfloat162_rn(o[0][0], o[0][1]), h1 = __floats2bfloat162_rn(o[0][2], o[0][3]);
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + to) = make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < left) store_out(a.y, to + i, o[0][i], a.out_f32);
                }
            }
        }
        cluster_sync();  // no CTA ends while another reads its sums
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
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

// What a kernel's launches need to know of it, asked for once per device: whether it has the registers of its split, and how
// many clusters of 1, 2, ... shares of a tile's k the device holds at once.
using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const Fp8Args);
struct Known {
    std::atomic<int> regs{0};
    std::atomic<int> held[16][kFewSplit];
};

// What the parts of a launch take, in ns: a block of k, the start of a CTA, the join of a cluster, and of it each share. (Without
// a time for each share, 64 x 3584 x 3584 took 8.4 us in clusters of 5, now 7.3 of 4; 64 x 2048 x 2048 5.5 of 6, now 4.8 of 4.)
struct Times {
    int block, start, join, share;
};

// Tiles whose k is cut between up to `most` shares of `unit` CTAs each, where that takes less time.
cudaError_t launch_cut(Kernel fn, Known& known, int smem, int unit, int most, int64_t tiles, const Times& of, int x_rows, const Fp8Args& a, cudaStream_t s) {
    CUtensorMap mx, mw, mu;
    if (!encode(&mx, a.X, a.K, a.M, x_rows) || !encode(&mw, a.W, a.K, a.N, 128) || !encode(&mu, a.U ? a.U : a.W, a.K, a.N, 128))
        return cudaErrorInvalidValue;
    const cudaError_t err = kv4_allow_smem((const void*)fn, smem);
    if (err != cudaSuccess) return err;
    if (!known.regs.load(std::memory_order_relaxed)) {
        cudaFuncAttributes attr;
        const cudaError_t e = cudaFuncGetAttributes(&attr, fn);
        if (e != cudaSuccess) return e;
        known.regs.store(attr.numRegs, std::memory_order_relaxed);
    }
    if (known.regs.load(std::memory_order_relaxed) < kRegsLaunch) return cudaErrorLaunchOutOfResources;  // the split would wait forever
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeClusterDimension;
    attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
    attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attrs;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int64_t KB = a.K / 128;
    int split = 1, held = 1;
    int64_t best = INT64_MAX;
    for (int n = 1; n <= most && n <= KB; ++n) {
        int h = dev < 16 ? known.held[dev][n - 1].load(std::memory_order_relaxed) : 0;
        if (!h) {
            attrs[0].val.clusterDim.x = unit * n;
            cfg.gridDim = dim3(unit * n, 1, 1);
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&h, fn, &cfg);
            if (e != cudaSuccess) return e;
            if (h < 1) h = 1;
            if (dev < 16) known.held[dev][n - 1].store(h, std::memory_order_relaxed);
        }
        const int64_t waves = (tiles + h - 1) / h, blocks = (KB + n - 1) / n;
        const int64_t cost = n == 1 ? waves * blocks * of.block + of.start : waves * (blocks * of.block + of.start) + of.join + n * of.share;
        if (cost < best) best = cost, split = n, held = h;
    }
    const int64_t clusters = split > 1 || tiles < held ? tiles : held;
    attrs[0].val.clusterDim.x = unit * split;
    cfg.gridDim = dim3((unsigned)(unit * split * clusters), 1, 1);
    cfg.numAttrs = 2;
    count_launch();
    return cudaLaunchKernelEx(&cfg, fn, mx, mw, mu, a);
}

template <bool GLU>
cudaError_t launch_pairs(const Fp8Args& a, cudaStream_t s) {
    static Known known;
    const int64_t tiles = (((int64_t)a.M + 255) / 256) * (((int64_t)a.N + (GLU ? 127 : 255)) / (GLU ? 128 : 256));
    return launch_cut(gemm_fp8_kernel<GLU>, known, kSmem, 2, kMaxSplit, tiles, {375, 3000, 3000, 0}, 128, a, s);
}
template <bool GLU, int NX>
cudaError_t launch_few(const Fp8Args& a, cudaStream_t s) {
    static Known known;
    constexpr int BLOCK = (NX == 32 ? 230 : NX == 64 ? 260 : 420) * (GLU ? 8 : 5) / 5;
    return launch_cut(gemm_fp8_few_kernel<GLU, NX>, known, Few<GLU, NX>::SMEM, 1, kFewSplit, ((int64_t)a.N + 127) / 128, {BLOCK, 4000, 1000, 260}, NX,
                      a, s);
}

}  // namespace

cudaError_t launch_gemm_fp8(const Fp8Args& a, cudaStream_t s) {
    // Few rows as a stream of W on mma.sync, up to 8, whose products cost it no more than one row's (2048 x 2048 2.6 us, here
    // 4.5; 18944 x 3584 14.0, 14.0), and up to 16 of smaller weights (2048 x 2048 3.1, 4.5; 4608 x 3584 6.5, 8.0; gated 5632 x
    // 2048, 23 MB, 9.9, 9.7; 2560 x 9728, 25 MB, 12.2, 8.4; 3584 x 18944 19.7, 15.2; gated 18944 x 3584 39, 25.6).
    const int64_t weights = (int64_t)a.N * a.K * (a.U ? 2 : 1);
    if (a.M <= 8 || (a.M <= 16 && weights < 20000000)) return launch_gemv_fp8(a, s);
    // Up to 128 rows with the weights as the products' rows (128 x 3584 x 18944: 20.0 us, by pairs 26.7; 100 x 18944 x 3584
    // gated 33, 36).
    if (a.M <= 32) return a.U ? launch_few<true, 32>(a, s) : launch_few<false, 32>(a, s);
    if (a.M <= 64) return a.U ? launch_few<true, 64>(a, s) : launch_few<false, 64>(a, s);
    if (a.M <= 128) return a.U ? launch_few<true, 128>(a, s) : launch_few<false, 128>(a, s);
    return a.U ? launch_pairs<true>(a, s) : launch_pairs<false>(a, s);
}

int gemm_fp8_take_fault() {
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_f8_fault, sizeof(int)) != cudaSuccess) return -1;
    if (v) cudaMemcpyToSymbol(g_f8_fault, &z, sizeof(int));
    return v;
}

}  // namespace mbw
