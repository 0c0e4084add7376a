// abi.cu -- the extern "C" entry points of libmbw.so (declared in mbw.h):
// argument checks on the host, plan lookup, launch, status reporting.
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include <atomic>
#include <cstring>
#include <string>

#include "internal.h"
#include "mbw.h"

namespace mbw {

static thread_local std::string g_last_error;
static thread_local int g_out_f32 = 0;
static thread_local uint64_t g_launches = 0;
static thread_local int g_injected_failures = 0;  // mbw_inject_launch_failures

void set_last_error(const std::string& msg) { g_last_error = msg; }
void count_launch() { ++g_launches; }

int device_sm_count() {
    static std::atomic<int> known[16];  // per device, once asked for
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    const bool keep = dev >= 0 && dev < 16;
    if (keep && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
    if (keep) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

static mbw_status fail(mbw_status st, const std::string& msg) {
    g_last_error = msg;
    return st;
}

static mbw_status cuda_fail(cudaError_t e, const char* where) {
    g_last_error = std::string(where) + ": " + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) + ")";
    return MBW_ERR_CUDA;
}

static bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// The test hook's failure, taken at the point where a call would launch.
static bool take_injected_failure(const char* where) {
    if (g_injected_failures <= 0) return false;
    --g_injected_failures;
    g_last_error = std::string(where) + ": injected launch failure (mbw_inject_launch_failures)";
    return true;
}

// Common size checks. Returns MBW_OK, or an error with the detail set.
static mbw_status check_sizes(const char* fn, int64_t M, int64_t N, int64_t K, int64_t kunit) {
    if (M < 0 || N < 0 || K < 0) return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": negative size");
    if (N > MBW_MAX_DIM || K > MBW_MAX_DIM || M > MBW_MAX_DIM)
        return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": N, K and M must be at most MBW_MAX_DIM (2^31 - 2^16)");
    if (K % kunit != 0)
        return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": K must be a multiple of " + std::to_string(kunit));
    return MBW_OK;
}

static mbw_status zero_output(void* y, int64_t M, int64_t N, cudaStream_t s) {
    const size_t bytes = (size_t)M * (size_t)N * (g_out_f32 ? 4 : 2);
    cudaError_t e = cudaMemsetAsync(y, 0, bytes, s);
    return e == cudaSuccess ? MBW_OK : cuda_fail(e, "cudaMemsetAsync");
}

// Run a CUDA-core streaming GEMV over M activation rows, in slices of the
// planned kernel's batch width.
// `op` may carry MBW_FUSE_* bits; `fz` then holds the fusion pointers.
static mbw_status run_simt(int fmt, int op, const uint8_t* W, const uint16_t* scales, const uint8_t* zeros,
                           const uint16_t* X, void* Y, int64_t M, int64_t N, int64_t K, cudaStream_t s,
                           const float* rscale = nullptr, const mbw_fusion* fz = nullptr) {
    if (take_injected_failure("GEMV launch")) return MBW_ERR_CUDA;
    const Plan p = plan_lookup(op, M, N, K, s);
    if (p.kind == PLAN_NONE)
        return fail(MBW_ERR_UNSUPPORTED, "no kernel fits this shape: the x of one CTA's k-range (split over the "
                                         "largest cluster) does not fit shared memory; see mbw_plan_candidates");
    const int width = plan_batch_width(fmt, p);
    GemvArgs a{};
    a.W = W;
    a.scales = scales;
    a.zeros = zeros;
    a.N = (int)N;
    a.K = (int)K;
    a.chunks = (int)(fmt == FMT_BF16 ? K / 8 : fmt == FMT_I8 ? K / 16 : K / 32);
    a.split_chunks = (a.chunks + p.split - 1) / p.split;
    a.groups = (int)(fmt == FMT_G64 ? K / 64 : fmt == FMT_AWQ ? K / 128 : 0);
    a.zstride = (a.groups + 1) / 2;
    a.out_f32 = g_out_f32;
    a.rscale = rscale;
    a.x_natural = (op & MBW_REPACKED) ? 1 : 0;
    if (fz) {
        a.norm_w = static_cast<const uint16_t*>(fz->norm_weight);
        a.norm_eps = fz->norm_eps;
        if (fz->up_weights) {
            a.glu = 1;
            a.W2 = static_cast<const uint8_t*>(fz->up_weights);
            a.scales2 = static_cast<const uint16_t*>(fz->up_scales);
            a.rscale2 = static_cast<const float*>(fz->up_scales);
            if (fmt == FMT_AWQ) a.zeros2 = static_cast<const uint8_t*>(fz->up_zeros);
        }
    }
    const size_t ybytes = g_out_f32 ? 4 : 2;
    for (int64_t m0 = 0; m0 < M; m0 += width) {
        a.x = X + m0 * K;
        a.y = static_cast<char*>(Y) + (size_t)m0 * (size_t)N * ybytes;
        if (fz && fz->residual) a.residual = static_cast<const uint16_t*>(fz->residual) + (size_t)m0 * (size_t)N;
        a.M = (int)((M - m0) < width ? (M - m0) : width);
        cudaError_t e = launch_plan(fmt, p, a, s);
        if (e != cudaSuccess) return cuda_fail(e, "gemv launch");
    }
    return MBW_OK;
}

// AWQ-style INT4 call (`op` may carry MBW_REPACKED): checks, then the planned launch.
static mbw_status awq_call(const char* fn, int op, const uint8_t* Wq, const void* scales, const uint8_t* zeros,
                           const void* X, void* Y, int64_t M, int64_t N, int64_t K, cudaStream_t stream) {
    mbw_status st = check_sizes(fn, M, N, K, 128);
    if (st != MBW_OK) return st;
    if (N == 0 || M == 0) return MBW_OK;
    if (!Y || (K > 0 && (!Wq || !scales || !zeros || !X)))
        return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": NULL pointer");
    if (!aligned(Wq, 32) || !aligned(X, 16) || !aligned(Y, 16) || !aligned(scales, 2))
        return fail(MBW_ERR_MISALIGNED,
                    std::string(fn) + ": Wq must be 32-byte aligned, X and Y 16-byte, scales 2-byte");
    if (K == 0) return zero_output(Y, M, N, stream);
    return run_simt(FMT_AWQ, op, Wq, (const uint16_t*)scales, zeros, (const uint16_t*)X, Y, M, N, K, stream);
}

// The sizes of a 4-bit cache (its pages' pointer is checked by the calls that use it).
static mbw_status check_cache(const char* fn, const mbw_kv4_cache* c) {
    if (!c) return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": NULL cache");
    if (mbw_kv4_page_bytes(c->page_size, c->kv_heads, c->head_dim, c->group) == 0)
        return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": page_size must be a multiple of 16 up to 1024, head_dim 64, "
                                                         "128 or 256, group 32 or 64, kv_heads 1 to 1024");
    if (c->num_pages < 1) return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": num_pages must be positive");
    if (c->num_pages > MBW_MAX_DIM) return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": at most MBW_MAX_DIM pages");
    return MBW_OK;
}

}  // namespace mbw

using namespace mbw;

extern "C" {

mbw_status gemv_bf16(const void* W, const void* x, void* y, int64_t N, int64_t K, void* workspace,
                     size_t ws_bytes, mbw_stream_t stream) {
    (void)workspace;
    (void)ws_bytes;
    mbw_status st = check_sizes("gemv_bf16", 1, N, K, 8);
    if (st != MBW_OK) return st;
    if (N == 0) return MBW_OK;
    if (!y || (K > 0 && (!W || !x))) return fail(MBW_ERR_INVALID_ARG, "gemv_bf16: NULL pointer");
    if (!aligned(W, 32) || !aligned(x, 16) || !aligned(y, 16))
        return fail(MBW_ERR_MISALIGNED, "gemv_bf16: W must be 32-byte aligned, x and y 16-byte");
    if (K == 0) return zero_output(y, 1, N, (cudaStream_t)stream);
    return run_simt(FMT_BF16, MBW_OP_GEMV_BF16, (const uint8_t*)W, nullptr, nullptr, (const uint16_t*)x, y, 1, N,
                    K, (cudaStream_t)stream);
}

mbw_status gemv_int4_g64(const uint8_t* Wq, const void* scales, const void* x, void* y, int64_t N, int64_t K,
                         void* workspace, size_t ws_bytes, mbw_stream_t stream) {
    (void)workspace;
    (void)ws_bytes;
    mbw_status st = check_sizes("gemv_int4_g64", 1, N, K, 64);
    if (st != MBW_OK) return st;
    if (N == 0) return MBW_OK;
    if (!y || (K > 0 && (!Wq || !scales || !x))) return fail(MBW_ERR_INVALID_ARG, "gemv_int4_g64: NULL pointer");
    if (!aligned(Wq, 32) || !aligned(x, 16) || !aligned(y, 16) || !aligned(scales, 2))
        return fail(MBW_ERR_MISALIGNED, "gemv_int4_g64: Wq must be 32-byte aligned, x and y 16-byte, scales 2-byte");
    if (K == 0) return zero_output(y, 1, N, (cudaStream_t)stream);
    return run_simt(FMT_G64, MBW_OP_GEMV_INT4_G64, Wq, (const uint16_t*)scales, nullptr, (const uint16_t*)x, y, 1,
                    N, K, (cudaStream_t)stream);
}

mbw_status gemv_int4_awq_g128(const uint8_t* Wq, const void* scales, const uint8_t* zeros, const void* X, void* Y,
                              int64_t M, int64_t N, int64_t K, void* workspace, size_t ws_bytes,
                              mbw_stream_t stream) {
    (void)workspace;
    (void)ws_bytes;
    return awq_call("gemv_int4_awq_g128", MBW_OP_GEMV_INT4_AWQ_G128, Wq, scales, zeros, X, Y, M, N, K,
                    (cudaStream_t)stream);
}

mbw_status gemv_int4_awq_g128_repacked(const uint8_t* Wr, const void* scales, const uint8_t* zeros, const void* X,
                                       void* Y, int64_t M, int64_t N, int64_t K, void* workspace, size_t ws_bytes,
                                       mbw_stream_t stream) {
    (void)workspace;
    (void)ws_bytes;
    return awq_call("gemv_int4_awq_g128_repacked", MBW_OP_GEMV_INT4_AWQ_G128 | MBW_REPACKED, Wr, scales, zeros, X,
                    Y, M, N, K, (cudaStream_t)stream);
}

mbw_status mbw_repack_int4(const uint8_t* Wq, uint8_t* Wr, int64_t N, int64_t K, mbw_stream_t stream) {
    mbw_status st = check_sizes("mbw_repack_int4", 1, N, K, 8);
    if (st != MBW_OK) return st;
    if (N == 0 || K == 0) return MBW_OK;
    if (!Wq || !Wr) return fail(MBW_ERR_INVALID_ARG, "mbw_repack_int4: NULL pointer");
    if (!aligned(Wq, 4) || !aligned(Wr, 4))
        return fail(MBW_ERR_MISALIGNED, "mbw_repack_int4: Wq and Wr must be 4-byte aligned");
    if (take_injected_failure("repack launch")) return MBW_ERR_CUDA;
    cudaError_t e = launch_repack_int4(Wq, Wr, N, K, (cudaStream_t)stream);
    return e == cudaSuccess ? MBW_OK : cuda_fail(e, "repack launch");
}

mbw_status gemv_int8_pc(const int8_t* Wq, const float* scales, const void* X, void* Y, int64_t M, int64_t N,
                        int64_t K, void* workspace, size_t ws_bytes, mbw_stream_t stream) {
    (void)workspace;
    (void)ws_bytes;
    mbw_status st = check_sizes("gemv_int8_pc", M, N, K, 128);
    if (st != MBW_OK) return st;
    if (N == 0 || M == 0) return MBW_OK;
    if (!Y || (K > 0 && (!Wq || !scales || !X))) return fail(MBW_ERR_INVALID_ARG, "gemv_int8_pc: NULL pointer");
    if (!aligned(Wq, 32) || !aligned(X, 16) || !aligned(Y, 16) || !aligned(scales, 4))
        return fail(MBW_ERR_MISALIGNED, "gemv_int8_pc: Wq must be 32-byte aligned, X and Y 16-byte, scales 4-byte");
    if (K == 0) return zero_output(Y, M, N, (cudaStream_t)stream);
    return run_simt(FMT_I8, MBW_OP_GEMV_INT8_PC, (const uint8_t*)Wq, nullptr, nullptr, (const uint16_t*)X, Y, M, N,
                    K, (cudaStream_t)stream, scales);
}

mbw_status mbw_quantize_int8_pc(const void* W, int8_t* Wq, float* scales, int64_t N, int64_t K,
                                mbw_stream_t stream) {
    mbw_status st = check_sizes("mbw_quantize_int8_pc", 1, N, K, 1);
    if (st != MBW_OK) return st;
    if (N == 0) return MBW_OK;
    if (!scales || (K > 0 && (!W || !Wq))) return fail(MBW_ERR_INVALID_ARG, "mbw_quantize_int8_pc: NULL pointer");
    if (!aligned(W, 2) || !aligned(scales, 4))
        return fail(MBW_ERR_MISALIGNED, "mbw_quantize_int8_pc: W must be 2-byte aligned, scales 4-byte");
    if (take_injected_failure("quantize launch")) return MBW_ERR_CUDA;
    cudaError_t e = launch_quantize_int8_pc((const uint16_t*)W, Wq, scales, N, K, (cudaStream_t)stream);
    return e == cudaSuccess ? MBW_OK : cuda_fail(e, "quantize launch");
}

mbw_status gemv_fused(int op, const void* W, const void* scales, const void* X, void* Y, int64_t M, int64_t N,
                      int64_t K, const mbw_fusion* fusion, void* workspace, size_t ws_bytes, mbw_stream_t stream) {
    (void)workspace;
    (void)ws_bytes;
    int fmt;
    switch (op) {
        case MBW_OP_GEMV_BF16: fmt = FMT_BF16; break;
        case MBW_OP_GEMV_INT4_G64: fmt = FMT_G64; break;
        case MBW_OP_GEMV_INT8_PC: fmt = FMT_I8; break;
        default: return fail(MBW_ERR_INVALID_ARG, "gemv_fused: op must be MBW_OP_GEMV_BF16, _INT4_G64 or _INT8_PC");
    }
    const int64_t kmul = (fmt == FMT_BF16) ? 8 : (fmt == FMT_G64) ? 64 : 128;
    mbw_status st = check_sizes("gemv_fused", M, N, K, kmul);
    if (st != MBW_OK) return st;
    if (N == 0 || M == 0) return MBW_OK;
    if (K == 0) return fail(MBW_ERR_BAD_SHAPE, "gemv_fused: K must be positive");
    if (fmt == FMT_G64 && M != 1) return fail(MBW_ERR_BAD_SHAPE, "gemv_fused: INT4 g64 takes M = 1");
    if (!W || !X || !Y || (fmt != FMT_BF16 && !scales)) return fail(MBW_ERR_INVALID_ARG, "gemv_fused: NULL pointer");
    const size_t salign = (fmt == FMT_I8) ? 4 : 2;
    if (!aligned(W, 32) || !aligned(X, 16) || !aligned(Y, 16) || (scales && !aligned(scales, salign)))
        return fail(MBW_ERR_MISALIGNED, "gemv_fused: W must be 32-byte aligned, X and Y 16-byte, scales 2 or 4 bytes");
    int fop = op;
    if (fusion) {
        if (fusion->norm_weight) {
            if (!aligned(fusion->norm_weight, 16))
                return fail(MBW_ERR_MISALIGNED, "gemv_fused: norm_weight must be 16-byte aligned");
            if (!(fusion->norm_eps >= 0.0f)) return fail(MBW_ERR_INVALID_ARG, "gemv_fused: norm_eps must be >= 0");
            fop |= MBW_FUSE_NORM;
        }
        if (fusion->up_weights) {
            if (!aligned(fusion->up_weights, 32))
                return fail(MBW_ERR_MISALIGNED, "gemv_fused: up_weights must be 32-byte aligned");
            if (fmt != FMT_BF16 && (!fusion->up_scales || !aligned(fusion->up_scales, salign)))
                return fail(MBW_ERR_INVALID_ARG, "gemv_fused: up_scales missing or misaligned");
            fop |= MBW_FUSE_GLU;
        }
        if (fusion->residual) {
            if (!aligned(fusion->residual, 2))
                return fail(MBW_ERR_MISALIGNED, "gemv_fused: residual must be 2-byte aligned");
            fop |= MBW_FUSE_RESIDUAL;
        }
    }
    if (fmt == FMT_G64 || fmt == FMT_I8) {
        if (fmt == FMT_G64 && K % 256 != 0 && (fop & MBW_FUSE_MASK))
            return fail(MBW_ERR_BAD_SHAPE, "gemv_fused: fused INT4 g64 needs K % 256 == 0");
    } else if ((fop & MBW_FUSE_MASK) && K % 64 != 0) {
        return fail(MBW_ERR_BAD_SHAPE, "gemv_fused: fused BF16 needs K % 64 == 0");
    }
    if (mbw_plan_candidates(fop, M, N, K) == 0)
        return fail(MBW_ERR_UNSUPPORTED, "gemv_fused: no kernel for this shape and fusion");
    return run_simt(fmt, fop, (const uint8_t*)W, (const uint16_t*)scales, nullptr, (const uint16_t*)X, Y, M, N, K,
                    (cudaStream_t)stream, fmt == FMT_I8 ? (const float*)scales : nullptr,
                    (fop & MBW_FUSE_MASK) ? fusion : nullptr);
}

mbw_status gemv_fused_awq_g128(const uint8_t* Wq, const void* scales, const uint8_t* zeros, const void* X, void* Y,
                               int64_t M, int64_t N, int64_t K, int repacked, const mbw_fusion* fusion,
                               void* workspace, size_t ws_bytes, mbw_stream_t stream) {
    (void)workspace;
    (void)ws_bytes;
    if (repacked != 0 && repacked != 1) return fail(MBW_ERR_INVALID_ARG, "gemv_fused_awq_g128: repacked must be 0 or 1");
    const int op = MBW_OP_GEMV_INT4_AWQ_G128 | (repacked ? MBW_REPACKED : 0);
    int fop = op;
    if (fusion) {
        if (fusion->norm_weight) {
            if (!aligned(fusion->norm_weight, 16))
                return fail(MBW_ERR_MISALIGNED, "gemv_fused_awq_g128: norm_weight must be 16-byte aligned");
            if (!(fusion->norm_eps >= 0.0f))
                return fail(MBW_ERR_INVALID_ARG, "gemv_fused_awq_g128: norm_eps must be >= 0");
            fop |= MBW_FUSE_NORM;
        }
        if (fusion->up_weights) {
            if (!aligned(fusion->up_weights, 32))
                return fail(MBW_ERR_MISALIGNED, "gemv_fused_awq_g128: up_weights must be 32-byte aligned");
            if (!fusion->up_scales || !aligned(fusion->up_scales, 2) || !fusion->up_zeros)
                return fail(MBW_ERR_INVALID_ARG, "gemv_fused_awq_g128: up_scales or up_zeros missing or misaligned");
            fop |= MBW_FUSE_GLU;
        }
        if (fusion->residual) {
            if (!aligned(fusion->residual, 2))
                return fail(MBW_ERR_MISALIGNED, "gemv_fused_awq_g128: residual must be 2-byte aligned");
            fop |= MBW_FUSE_RESIDUAL;
        }
    }
    if (!(fop & MBW_FUSE_MASK))
        return awq_call("gemv_fused_awq_g128", op, Wq, scales, zeros, X, Y, M, N, K, (cudaStream_t)stream);
    mbw_status st = check_sizes("gemv_fused_awq_g128", M, N, K, 256);
    if (st != MBW_OK) return st;
    if (N == 0 || M == 0) return MBW_OK;
    if (K == 0) return fail(MBW_ERR_BAD_SHAPE, "gemv_fused_awq_g128: K must be positive");
    if (!Wq || !scales || !zeros || !X || !Y) return fail(MBW_ERR_INVALID_ARG, "gemv_fused_awq_g128: NULL pointer");
    if (!aligned(Wq, 32) || !aligned(X, 16) || !aligned(Y, 16) || !aligned(scales, 2))
        return fail(MBW_ERR_MISALIGNED,
                    "gemv_fused_awq_g128: Wq must be 32-byte aligned, X and Y 16-byte, scales 2-byte");
    if (mbw_plan_candidates(fop, M, N, K) == 0)
        return fail(MBW_ERR_UNSUPPORTED, "gemv_fused_awq_g128: no kernel for this shape and fusion");
    return run_simt(FMT_AWQ, fop, Wq, (const uint16_t*)scales, zeros, (const uint16_t*)X, Y, M, N, K,
                    (cudaStream_t)stream, nullptr, fusion);
}

mbw_status gemm_skinny_bf16(const void* X, const void* W, void* Y, int64_t M, int64_t N, int64_t K,
                            void* workspace, size_t ws_bytes, mbw_stream_t stream) {
    (void)workspace;
    (void)ws_bytes;
    mbw_status st = check_sizes("gemm_skinny_bf16", M, N, K, 8);
    if (st != MBW_OK) return st;
    if (N == 0 || M == 0) return MBW_OK;
    if (!Y || (K > 0 && (!W || !X))) return fail(MBW_ERR_INVALID_ARG, "gemm_skinny_bf16: NULL pointer");
    if (!aligned(W, 32) || !aligned(X, 16) || !aligned(Y, 16))
        return fail(MBW_ERR_MISALIGNED, "gemm_skinny_bf16: W must be 32-byte aligned, X and Y 16-byte");
    if (K == 0) return zero_output(Y, M, N, (cudaStream_t)stream);
    return run_simt(FMT_BF16, MBW_OP_GEMM_SKINNY_BF16, (const uint8_t*)W, nullptr, nullptr, (const uint16_t*)X, Y,
                    M, N, K, (cudaStream_t)stream);
}

size_t mbw_kv4_page_bytes(int32_t page_size, int32_t kv_heads, int32_t head_dim, int32_t group) {
    if (page_size < 16 || page_size > 1024 || page_size % 16 != 0 || kv_heads < 1 || kv_heads > 1024) return 0;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || (group != 32 && group != 64)) return 0;
    return (size_t)kv_heads * (size_t)(page_size / 16) * (size_t)(16 * head_dim + 128 * (head_dim / group));
}

mbw_status mbw_kv4_append(const mbw_kv4_cache* cache, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, const int64_t* slots, const void* q, int64_t q_stride, void* q_out,
                          int64_t q_out_stride, int64_t q_heads, const mbw_rope* rope, int64_t T,
                          mbw_stream_t stream) {
    const char* fn = "mbw_kv4_append";
    mbw_status st = check_cache(fn, cache);
    if (st != MBW_OK) return st;
    if (T < 0 || q_heads < 0) return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": negative size");
    if (T > MBW_MAX_DIM || q_heads > 65536)
        return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": at most MBW_MAX_DIM tokens and 65536 query heads");
    if (T == 0) return MBW_OK;
    if (!cache->pages || !k || !v || !slots || (q_heads > 0 && (!q || !q_out)))
        return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": NULL pointer");
    const int64_t kvw = (int64_t)cache->kv_heads * cache->head_dim, qw = q_heads * cache->head_dim;
    if (k_stride < kvw || v_stride < kvw || (q_heads > 0 && (q_stride < qw || q_out_stride < qw)))
        return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": a row stride is shorter than the row");
    if (!aligned(cache->pages, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8) || k_stride % 8 ||
        v_stride % 8 || (q_heads > 0 && (!aligned(q, 16) || !aligned(q_out, 16) || q_stride % 8 || q_out_stride % 8)))
        return fail(MBW_ERR_MISALIGNED, std::string(fn) + ": pages, k, v, q and q_out must be 16-byte aligned, slots "
                                                          "8-byte, strides multiples of 8 elements");
    Kv4AppendArgs a{};
    if (rope) {
        if (!rope->cos_sin || !rope->positions)
            return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": rope without cos_sin or positions");
        if (rope->interleaved != 0 && rope->interleaved != 1)
            return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": interleaved must be 0 or 1");
        if (rope->max_pos < 1) return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": max_pos must be positive");
        if (rope->rotary_dim < 16 || rope->rotary_dim % 16 != 0 || rope->rotary_dim > cache->head_dim)
            return fail(MBW_ERR_BAD_SHAPE,
                        std::string(fn) + ": rotary_dim must be a multiple of 16, at most head_dim");
        if (!aligned(rope->cos_sin, 16) || !aligned(rope->positions, 4))
            return fail(MBW_ERR_MISALIGNED, std::string(fn) + ": cos_sin must be 16-byte aligned, positions 4-byte");
        a.cos_sin = rope->cos_sin;
        a.positions = rope->positions;
        a.max_pos = rope->max_pos;
        a.rotary = rope->rotary_dim;
        a.interleaved = rope->interleaved;
    }
    a.pages = static_cast<uint8_t*>(cache->pages);
    a.num_slots = cache->num_pages * cache->page_size;
    a.page_size = cache->page_size;
    a.kv_heads = cache->kv_heads;
    a.head_dim = cache->head_dim;
    a.group = cache->group;
    a.k = static_cast<const uint16_t*>(k);
    a.v = static_cast<const uint16_t*>(v);
    a.q = static_cast<const uint16_t*>(q);
    a.q_out = static_cast<uint16_t*>(q_out);
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_stride = q_stride;
    a.q_out_stride = q_out_stride;
    a.q_heads = (int)q_heads;
    a.slots = slots;
    a.T = T;
    if (take_injected_failure("append launch")) return MBW_ERR_CUDA;
    cudaError_t e = launch_kv4_append(a, (cudaStream_t)stream);
    return e == cudaSuccess ? MBW_OK : cuda_fail(e, "append launch");
}

mbw_status mbw_kv4_gather(const mbw_kv4_cache* cache, const int64_t* slots, void* k, void* v, int64_t T,
                          mbw_stream_t stream) {
    const char* fn = "mbw_kv4_gather";
    mbw_status st = check_cache(fn, cache);
    if (st != MBW_OK) return st;
    if (T < 0) return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": negative size");
    if (T > MBW_MAX_DIM) return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": at most MBW_MAX_DIM tokens");
    if (T == 0) return MBW_OK;
    if (!cache->pages || !slots || !k || !v) return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": NULL pointer");
    if (!aligned(cache->pages, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
        return fail(MBW_ERR_MISALIGNED, std::string(fn) + ": pages, k and v must be 16-byte aligned, slots 8-byte");
    Kv4GatherArgs a{};
    a.pages = static_cast<const uint8_t*>(cache->pages);
    a.num_slots = cache->num_pages * cache->page_size;
    a.page_size = cache->page_size;
    a.kv_heads = cache->kv_heads;
    a.head_dim = cache->head_dim;
    a.group = cache->group;
    a.slots = slots;
    a.k = static_cast<uint16_t*>(k);
    a.v = static_cast<uint16_t*>(v);
    a.T = T;
    if (take_injected_failure("gather launch")) return MBW_ERR_CUDA;
    cudaError_t e = launch_kv4_gather(a, (cudaStream_t)stream);
    return e == cudaSuccess ? MBW_OK : cuda_fail(e, "gather launch");
}

size_t mbw_kv4_attention_workspace_bytes(int32_t head_dim) {
    return (head_dim == 64 || head_dim == 128 || head_dim == 256) ? kv4_attention_workspace(head_dim) : 0;
}

mbw_status mbw_kv4_attention(const mbw_kv4_cache* cache, const void* q, int64_t q_stride, void* out,
                             int64_t out_stride, float* lse, const int32_t* block_table, int64_t table_stride,
                             int64_t table_width, const int32_t* ctx_lens, const int32_t* q_starts, int64_t B,
                             int64_t T, int64_t q_heads, float scale, int64_t window, void* workspace,
                             size_t ws_bytes, mbw_stream_t stream) {
    const char* fn = "mbw_kv4_attention";
    mbw_status st = check_cache(fn, cache);
    if (st != MBW_OK) return st;
    if (B < 0 || T < 0 || table_stride < 0 || table_width < 0 || window < 0)
        return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": negative size");
    if (q_heads < 1 || q_heads % cache->kv_heads != 0)
        return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": q_heads must be a positive multiple of kv_heads");
    if (B > (1 << 20) || T > MBW_MAX_DIM || q_heads > 65536 || T * q_heads > MBW_MAX_DIM)
        return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": at most 2^20 requests and MBW_MAX_DIM query rows");
    if (table_width * cache->page_size > MBW_MAX_DIM)
        return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": at most MBW_MAX_DIM tokens per request");
    if (T == 0) return MBW_OK;
    if (B == 0) return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": queries of no request");
    if (!q_starts && T % B != 0)
        return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": without q_starts T must be a multiple of B");
    if (!cache->pages || !q || !out || !ctx_lens || (table_width > 0 && !block_table))
        return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": NULL pointer");
    if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f)
        return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": scale must be finite");
    const int64_t qw = q_heads * cache->head_dim;
    if (q_stride < qw || out_stride < qw)
        return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": a row stride is shorter than the row");
    if (B > 1 && table_stride < table_width)
        return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": table_stride is shorter than table_width");
    if (!aligned(cache->pages, 16) || !aligned(q, 16) || !aligned(out, 16) || q_stride % 8 || out_stride % 8 ||
        !aligned(block_table, 4) || !aligned(ctx_lens, 4) || !aligned(q_starts, 4) || !aligned(lse, 4) ||
        !aligned(workspace, 16))
        return fail(MBW_ERR_MISALIGNED, std::string(fn) + ": pages, q, out and workspace must be 16-byte aligned, "
                                                          "strides multiples of 8 elements, the rest 4-byte");
    Kv4AttnArgs a{};
    a.pages = static_cast<const uint8_t*>(cache->pages);
    a.num_pages = cache->num_pages;
    a.page_size = cache->page_size;
    a.kv_heads = cache->kv_heads;
    a.head_dim = cache->head_dim;
    a.group = cache->group;
    a.q = static_cast<const uint16_t*>(q);
    a.q_stride = q_stride;
    a.out = out;
    a.out_stride = out_stride;
    a.lse = lse;
    a.table = block_table;
    a.table_stride = table_stride;
    a.table_width = (int)table_width;
    a.ctx_lens = ctx_lens;
    a.q_starts = q_starts;
    a.B = (int)B;
    a.T = (int)T;
    a.q_heads = (int)q_heads;
    a.scale = scale;
    a.window = (int)(window < MBW_MAX_DIM ? window : 0);  // no context is longer
    a.out_f32 = g_out_f32;
    a.workspace = workspace;
    a.ws_bytes = workspace ? ws_bytes : 0;
    if (take_injected_failure("attention launch")) return MBW_ERR_CUDA;
    cudaError_t e = launch_kv4_attention(a, (cudaStream_t)stream);
    return e == cudaSuccess ? MBW_OK : cuda_fail(e, "attention launch");
}

size_t mbw_token_logprobs_workspace_bytes(void) { return token_logprobs_workspace(); }

mbw_status mbw_token_logprobs(const void* logits, int fp32, int64_t row_stride, const int32_t* targets, int64_t M,
                              int64_t V, float scale, int32_t top_k, float* logprob, int32_t* rank, float* entropy,
                              int32_t* top_ids, float* top_logprobs, void* workspace, size_t ws_bytes,
                              mbw_stream_t stream) {
    const char* fn = "mbw_token_logprobs";
    if (M < 0 || V < 0 || top_k < 0) return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": negative size");
    if (fp32 != 0 && fp32 != 1) return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": fp32 must be 0 or 1");
    if (M > MBW_MAX_DIM || V > MBW_MAX_DIM)
        return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": M and V must be at most MBW_MAX_DIM");
    if (top_k > 32) return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": top_k must be at most 32");
    if (!(scale > 0.f) || scale > 3.0e38f)
        return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": scale must be positive and finite");
    if (M == 0) return MBW_OK;
    if (V == 0) return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": V must be positive");
    if (row_stride < V) return fail(MBW_ERR_BAD_SHAPE, std::string(fn) + ": row_stride is shorter than the row");
    if (!logits) return fail(MBW_ERR_INVALID_ARG, std::string(fn) + ": NULL pointer");
    if (!aligned(logits, fp32 ? 4 : 2) || !aligned(targets, 4) || !aligned(logprob, 4) || !aligned(rank, 4) ||
        !aligned(entropy, 4) || !aligned(top_ids, 4) || !aligned(top_logprobs, 4) || !aligned(workspace, 16))
        return fail(MBW_ERR_MISALIGNED, std::string(fn) + ": workspace must be 16-byte aligned, the rest element-wise");
    LogprobArgs a{};
    a.logits = logits;
    a.fp32 = fp32;
    a.row_stride = row_stride;
    a.targets = targets;
    a.M = M;
    a.V = V;
    a.scale = scale;
    a.top_k = (top_ids || top_logprobs) ? top_k : 0;
    a.logprob = logprob;
    a.rank = rank;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.workspace = workspace;
    a.ws_bytes = workspace ? ws_bytes : 0;
    if (take_injected_failure("logprobs launch")) return MBW_ERR_CUDA;
    cudaError_t e = launch_token_logprobs(a, (cudaStream_t)stream);
    return e == cudaSuccess ? MBW_OK : cuda_fail(e, "logprobs launch");
}

size_t mbw_workspace_bytes(int op, int64_t M, int64_t N, int64_t K) {
    (void)op;
    (void)M;
    (void)N;
    (void)K;
    return 0;
}

mbw_status mbw_dequant_int4_g64(const uint8_t* Wq, const void* scales, float* out, int64_t N, int64_t K,
                                mbw_stream_t stream) {
    mbw_status st = check_sizes("mbw_dequant_int4_g64", 1, N, K, 64);
    if (st != MBW_OK) return st;
    if (N == 0 || K == 0) return MBW_OK;
    if (!Wq || !scales || !out) return fail(MBW_ERR_INVALID_ARG, "mbw_dequant_int4_g64: NULL pointer");
    if (!aligned(scales, 2) || !aligned(out, 4)) return fail(MBW_ERR_MISALIGNED, "mbw_dequant_int4_g64: alignment");
    if (take_injected_failure("dequant launch")) return MBW_ERR_CUDA;
    cudaError_t e = launch_dequant(FMT_G64, Wq, (const uint16_t*)scales, nullptr, out, N, K, (cudaStream_t)stream);
    return e == cudaSuccess ? MBW_OK : cuda_fail(e, "dequant launch");
}

mbw_status mbw_dequant_int4_awq_g128(const uint8_t* Wq, const void* scales, const uint8_t* zeros, float* out,
                                     int64_t N, int64_t K, mbw_stream_t stream) {
    mbw_status st = check_sizes("mbw_dequant_int4_awq_g128", 1, N, K, 128);
    if (st != MBW_OK) return st;
    if (N == 0 || K == 0) return MBW_OK;
    if (!Wq || !scales || !zeros || !out)
        return fail(MBW_ERR_INVALID_ARG, "mbw_dequant_int4_awq_g128: NULL pointer");
    if (!aligned(scales, 2) || !aligned(out, 4))
        return fail(MBW_ERR_MISALIGNED, "mbw_dequant_int4_awq_g128: alignment");
    if (take_injected_failure("dequant launch")) return MBW_ERR_CUDA;
    cudaError_t e = launch_dequant(FMT_AWQ, Wq, (const uint16_t*)scales, zeros, out, N, K, (cudaStream_t)stream);
    return e == cudaSuccess ? MBW_OK : cuda_fail(e, "dequant launch");
}

mbw_status mbw_set_output_fp32(int enable) {
    if (enable != 0 && enable != 1) return fail(MBW_ERR_INVALID_ARG, "mbw_set_output_fp32: 0 or 1");
    g_out_f32 = enable;
    return MBW_OK;
}

mbw_status mbw_check_device_error(void) {
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize");
    const int f = tma_take_fault();
    const int f2 = tc_take_fault(), f3 = kv4_attn_tc_take(true);
    const int r = kv4_cache_take_range(), r2 = kv4_attn_take_range(), r3 = logprobs_take_range();
    const int r4 = kv4_attn_tc_take(false);
    if (f < 0 || f2 < 0 || f3 < 0 || r < 0 || r2 < 0 || r3 < 0 || r4 < 0)
        return cuda_fail(cudaGetLastError(), "reading the device fault flag");
    // Every flag is cleared, so every one is named; the status is that of the gravest.
    std::string what;
    auto name = [&](bool set, const char* text) {
        if (set) what += (what.empty() ? "" : "; ") + std::string(text);
    };
    name(f || f2 || f3, "a bounded wait inside a kernel expired");
    name(r, "a cache slot or position was out of range");
    name(r2 || r4, "a page id, context length or query offset was out of range");
    name(r3, "a target token id was out of range");
    if (what.empty()) return MBW_OK;
    return fail(f || f2 || f3 ? MBW_ERR_DEVICE_TIMEOUT : MBW_ERR_DEVICE_RANGE, what);
}

mbw_status mbw_selftest_wait_expiry(int64_t tries, mbw_stream_t stream) {
    if (tries < 1 || tries > MBW_WAIT_LIMIT)
        return fail(MBW_ERR_INVALID_ARG, "mbw_selftest_wait_expiry: tries must be in [1, MBW_WAIT_LIMIT]");
    cudaError_t e = launch_tma_wait_expiry((long long)tries, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "wait-expiry launch");
    e = launch_tc_wait_expiry((long long)tries, (cudaStream_t)stream);
    return e == cudaSuccess ? MBW_OK : cuda_fail(e, "wait-expiry launch");
}

mbw_status mbw_inject_launch_failures(int count) {
    if (count < 0) return fail(MBW_ERR_INVALID_ARG, "mbw_inject_launch_failures: count must be >= 0");
    g_injected_failures = count;
    return MBW_OK;
}

uint64_t mbw_launch_count(void) { return g_launches; }

const char* mbw_status_string(mbw_status s) {
    switch (s) {
        case MBW_OK: return "MBW_OK";
        case MBW_ERR_INVALID_ARG: return "MBW_ERR_INVALID_ARG";
        case MBW_ERR_MISALIGNED: return "MBW_ERR_MISALIGNED";
        case MBW_ERR_BAD_SHAPE: return "MBW_ERR_BAD_SHAPE";
        case MBW_ERR_WORKSPACE_TOO_SMALL: return "MBW_ERR_WORKSPACE_TOO_SMALL";
        case MBW_ERR_UNSUPPORTED: return "MBW_ERR_UNSUPPORTED";
        case MBW_ERR_CUDA: return "MBW_ERR_CUDA";
        case MBW_ERR_DEVICE_TIMEOUT: return "MBW_ERR_DEVICE_TIMEOUT";
        case MBW_ERR_DEVICE_RANGE: return "MBW_ERR_DEVICE_RANGE";
        default: return "MBW_ERR_UNKNOWN";
    }
}

const char* mbw_last_error(void) { return g_last_error.c_str(); }

}  // extern "C"
