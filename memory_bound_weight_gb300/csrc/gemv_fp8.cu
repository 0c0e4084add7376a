// gemv_fp8.cu -- Y = X . W^T of 8-bit floating point operands with a scale for
// each block of 128 (formula at gemm_fp8.cu), of up to 16 rows of X: a stream of W.
//
// m16n8k32 on e4m3 codes (which the compiler makes of conversions to fp16 and products
// of that, exact). A warp's step is a block of 16 rows of W by 128 k, 2 KB, loaded
// straight into registers some steps ahead of its use: lane 4 g + c holds bytes 32 c ..
// 32 c + 31 of rows g and g + 8, and the four products of a step take their k in that
// order (words 2 q and 2 q + 1 of the lane's eight); X's operand is the same 32 bytes
// of row g of X, read through L1. A block's sums come out of a fresh accumulator and go
// into the row's by xs ws, fp32.
// The steps of a CTA's tiles (16 rows of W; gated: of W and of U in turn) are one
// line, of which a warp takes every sixteenth, so that its warps end together whatever
// the sizes. A tile's sums of the warps meet in shared memory, some tiles at a
// time, in two buffers in turn: one barrier a round, with the loads of the next under
// way. Where there are too few tiles to go round, k is cut between the CTAs of a
// cluster and their sums joined through its shared memory in order.
#include <cuda_runtime.h>

#include <atomic>

#include "device.cuh"
#include "internal.h"

namespace mbw {

namespace {

// 16 warps, one CTA an SM: with 8, two CTAs of the same registers and a next launch that loads beside this one, one token
// took 17.4 us where this takes 13.2 (18944 x 3584), and 2.5 for 2.6 at 2048 x 2048.
constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;  // CTAs that share tiles

template <int NT>
struct Shape {
    static constexpr int AHEAD = NT == 1 ? 4 : 3;  // steps of a warp under way
    // Logical tiles whose sums meet at a time: a barrier every 2 tiles cost 15 to 30%, behind which no loads are issued.
    static constexpr int ROUND = 8 / NT;
    static constexpr int SUMS = NT * 128;  // of a tile: 16 rows of W x 8 NT of X
    static constexpr int OFF_JOIN = 2 * ROUND * kWarps * SUMS * 4, SMEM = OFF_JOIN + ROUND * SUMS * 4;
};

__device__ __forceinline__ void mma_e4m3(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 32 bytes, cached: X is read again for every tile.
__device__ __forceinline__ void ld32(uint32_t* v, const void* p) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]) : "l"(p));
}
// The same from 16-byte boundaries.
__device__ __forceinline__ void ld16x2(uint32_t* v, const void* p) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[4 * i]), "=r"(v[4 * i + 1]), "=r"(v[4 * i + 2]), "=r"(v[4 * i + 3]) : "l"(static_cast<const uint8_t*>(p) + 16 * i));
}

// WIDE: X lies on 32 bytes, which its rows and blocks then do too; else on 16.
template <int NT, bool GLU, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) gemv_fp8_kernel(const Fp8Args a, const int split) {
    using S = Shape<NT>;
    constexpr int SETS = GLU ? 2 : 1, ROUND = S::ROUND, SUMS = S::SUMS, AHEAD = S::AHEAD;
    extern __shared__ __align__(16) uint8_t smem[];
    float* sums = reinterpret_cast<float*>(smem);                  // [2][ROUND][kWarps][SUMS]
    float* joined = reinterpret_cast<float*>(smem + S::OFF_JOIN);  // [ROUND][SUMS], of a CTA that shares its tiles
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int rank = split > 1 ? (int)blockIdx.x % split : 0;
    pdl_launch_dependents();

    // ---- the CTA's tiles, and its blocks of k ----
    const int KB = a.K / 128, tiles = (a.N + 15) / 16, groups = gridDim.x / split, me = blockIdx.x / split;
    const int p0 = (int)((long long)tiles * me / groups), nt = ((int)((long long)tiles * (me + 1) / groups) - p0) * SETS;
    const int k0 = (int)((long long)KB * rank / split), kn = (int)((long long)KB * (rank + 1) / split) - k0;
    const long long steps = (long long)nt * kn;  // the warp's are warp, warp + 16, ...

    struct Place {  // a step's tile and block
        int lt, j;
    };
    auto forward = [&](Place& p) {
        p.j += kWarps;
        while (p.j >= kn && p.lt < nt) p.j -= kn, ++p.lt;
    };
    Place load = {0, warp - kWarps}, use;
    if (kn > 0) forward(load); else load.lt = nt;
    use = load;

    uint32_t w[AHEAD][2][8];
    auto fetch = [&](uint32_t (*to)[8], const Place& p) {
        const uint8_t* base = GLU && (p.lt & 1) ? a.U : a.W;
        const int row = (p0 + p.lt / SETS) * 16 + g;
        const uint8_t* at = base + (int64_t)(k0 + p.j) * 128 + 32 * c;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x8 x = ld_stream32(at + (int64_t)min(row + 8 * i, a.N - 1) * a.K);  // past the end: any row, whose sums are not written
#pragma unroll
            for (int q = 0; q < 8; ++q) to[i][q] = x.v[q];
        }
    };
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
        if (load.lt < nt) fetch(w[i], load);
        forward(load);
    }
    pdl_wait();

    uint32_t x[NT][8];
    float f[NT][2];
    auto fetch_x = [&](const Place& p) {  // X's block, and the factors of the lane's two columns
        const int kb = k0 + p.j;
        const float s = __ldg((GLU && (p.lt & 1) ? a.us : a.ws) + (int64_t)((p0 + p.lt / SETS) / 8) * KB + kb);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int m = 8 * i + g;
            if (m < a.M) {
                const uint8_t* at = a.X + (int64_t)m * a.K + kb * 128 + 32 * c;
                if (WIDE)
                    ld32(x[i], at);
                else
                    ld16x2(x[i], at);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) x[i][q] = 0;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = 8 * i + 2 * c + e;
                f[i][e] = col < a.M ? a.xs[(int64_t)col * KB + kb] * s : 0.f;
            }
        }
    };

    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

    auto store = [&](int m, int n, float v, float up) {
        if (GLU) v = silu_f32(v) * up;
        const int64_t at = (int64_t)m * a.N + n;
        if (a.residual) v += bf16lo_to_f32(a.residual[at]);
        store_out(a.y, at, v, a.out_f32);
    };
    // The sums of the round that ends with logical tile lt, whose place a thread has for 16 rows of W by a column.
    auto end_round = [&](int lt) {
        const float* from = sums + (lt / ROUND & 1) * ROUND * kWarps * SUMS;
        const int first = lt / ROUND * ROUND, n = lt - first + 1;
        __syncthreads();
        for (int e = tid; e < (split > 1 ? n : n / SETS) * SUMS; e += kThreads) {
            const int t = e / SUMS, i = e % SUMS;  // i: column * 16 + row
            float v[SETS];
#pragma unroll
            for (int s = 0; s < SETS; ++s) {
                const float* at = from + (split > 1 ? t : t * SETS + s) * kWarps * SUMS + i;
                v[s] = 0.f;
#pragma unroll
                for (int q = 0; q < kWarps; ++q) v[s] += at[q * SUMS];
                if (split > 1) break;
            }
            if (split > 1) {
                joined[e] = v[0];
            } else {
                const int m = i / 16, row = (p0 + first / SETS + t) * 16 + i % 16;
                if (m < a.M && row < a.N) store(m, row, v[0], v[SETS - 1]);
            }
        }
    };
    // The warp's sums of the tiles before `to` into shared memory; those of which it had no step are zeros.
    int done = 0;
    auto flush = [&](int to) {
        for (; done < to; ++done) {
            float* at = sums + ((done / ROUND & 1) * ROUND + done % ROUND) * kWarps * SUMS + warp * SUMS;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    at[(8 * i + 2 * c + (e & 1)) * 16 + g + 8 * (e >> 1)] = acc[i][e];
                    acc[i][e] = 0.f;
                }
            if (done % ROUND == ROUND - 1 || done == nt - 1) end_round(done);
        }
    };

    const int mine = (int)(steps > warp ? (steps - warp + kWarps - 1) / kWarps : 0);
    for (int s0 = 0; s0 < mine; s0 += AHEAD) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (s0 + u >= mine) break;
            if (use.lt != done) flush(use.lt);
            fetch_x(use);
            float t[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                t[i][0] = t[i][1] = t[i][2] = t[i][3] = 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) mma_e4m3(t[i], w[u][0][2 * q], w[u][1][2 * q], w[u][0][2 * q + 1], w[u][1][2 * q + 1], x[i][2 * q], x[i][2 * q + 1]);
            }
            if (load.lt < nt) fetch(w[u], load);
            forward(load);
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(t[i][e], f[i][e & 1], acc[i][e]);
            forward(use);
        }
    }
    flush(nt);

    if (split > 1) {
        cluster_sync();
        const int total = nt / SETS * SUMS, e0 = (int)((long long)total * rank / split), e1 = (int)((long long)total * (rank + 1) / split);
        for (int e = e0 + tid; e < e1; e += kThreads) {
            const int t = e / SUMS, i = e % SUMS, m = i / 16, row = (p0 + t) * 16 + i % 16;
            if (m >= a.M || row >= a.N) continue;
            float v[SETS];
#pragma unroll
            for (int s = 0; s < SETS; ++s) {
                const uint32_t at = (uint32_t)__cvta_generic_to_shared(joined + (t * SETS + s) * SUMS + i);
                v[s] = 0.f;
                for (int q = 0; q < split; ++q) {
                    uint32_t from;
                    float part;
                    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(at), "r"(q));
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(part) : "r"(from) : "memory");
                    v[s] += part;
                }
            }
            store(m, row, v[0], v[SETS - 1]);
        }
        // no CTA leaves while another reads its sums
        cluster_sync();
    }
}

template <int NT, bool GLU, bool WIDE>
cudaError_t launch(const Fp8Args& a, cudaStream_t s) {
    using S = Shape<NT>;
    constexpr int SETS = GLU ? 2 : 1;
    auto* fn = gemv_fp8_kernel<NT, GLU, WIDE>;
    const cudaError_t err = kv4_allow_smem((const void*)fn, S::SMEM);
    if (err != cudaSuccess) return err;
    const int sms = device_sm_count();
    const int64_t KB = a.K / 128, tiles = ((int64_t)a.N + 15) / 16;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeClusterDimension;
    attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
    attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attrs;
    // CTAs that share a tile's k: as the longest line of steps is shortest, a cluster's join taken for 16 steps. There are no
    // more groups than the device holds at once, which is asked for once per device (2560 x 9728: 15.4 us in 21 clusters
    // of 7, which are not all held, 9.4 so).
    static std::atomic<int> known[16][kMaxCluster];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int split = 1;
    int64_t best = INT64_MAX, groups = 1;
    for (int n = 1; n <= kMaxCluster && n <= KB && n <= sms; ++n) {
        int held = n == 1 ? sms : dev < 16 ? known[dev][n - 1].load(std::memory_order_relaxed) : 0;
        if (!held) {
            attrs[0].val.clusterDim.x = n;
            cfg.gridDim = dim3(n, 1, 1);
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&held, fn, &cfg);
            if (e != cudaSuccess) return e;
            if (held < 1) held = 1;
            if (dev < 16) known[dev][n - 1].store(held, std::memory_order_relaxed);
        }
        const int64_t g = tiles < held ? tiles : held, most = (tiles + g - 1) / g * SETS;
        if (n > 1 && most > S::ROUND) continue;
        const int64_t cost = most * ((KB + n - 1) / n) + (n > 1 ? 16 : 0);
        if (cost < best) best = cost, split = n, groups = g;
    }
    attrs[0].val.clusterDim.x = (unsigned)split;
    cfg.gridDim = dim3((unsigned)(groups * split), 1, 1);
    cfg.numAttrs = 2;
    count_launch();
    return cudaLaunchKernelEx(&cfg, fn, a, (const int)split);
}

template <int NT, bool WIDE>
cudaError_t launch(const Fp8Args& a, cudaStream_t s) {
    return a.U ? launch<NT, true, WIDE>(a, s) : launch<NT, false, WIDE>(a, s);
}

}  // namespace

cudaError_t launch_gemv_fp8(const Fp8Args& a, cudaStream_t s) {
    const bool wide = ((uintptr_t)a.X & 31) == 0;
    if (a.M <= 8) return wide ? launch<1, true>(a, s) : launch<1, false>(a, s);
    return wide ? launch<2, true>(a, s) : launch<2, false>(a, s);
}

}  // namespace mbw
