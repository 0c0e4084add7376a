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
// One read of the logits. A row is cut into pieces, one CTA each, where there
// are few rows. A warp keeps one reference for all its lanes, so that its common
// path is the sums and, for four 16-byte loads at a time, one comparison with the
// gate: 74 instructions per 16-byte load of 8 logits. That bounds 2000 rows of 152064
// 16-bit logits, 608 MB: 124 us, 4.9 TB/s, and 6.1 TB/s for a further row.
//   The rare path, taken when a logit passes the gate, moves the reference and takes
// in candidates for the top tokens: into a buffer of the CTA, or in long pieces into
// the warp's list, one entry per lane, in order. The first gate is the K-th largest
// of the warps' best lanes' largest logits, which is little below the K-th best of
// the first loads; the lists' K-th entries raise it. At the end the better ones of
// each candidate are counted. Pieces of a row meet in the workspace; the CTA that
// arrives last joins them in their order, and of their lists only what can still be
// among the K best. (The 20 best of 1 row: 10.6 us, 6.6 without any; of 50 rows of
// 4-byte logits 20.5 and 11.0; 32 with a list per warp and a gate that was the least
// of the warps'.)
#include <cuda_runtime.h>

#include <math_constants.h>

#include "device.cuh"
#include "internal.h"

namespace mbw {

namespace {

__device__ int g_logprobs_range;  // a target was not below V

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTop = 32;        // a warp's list is one entry per lane
constexpr int kBuffer = kMaxTop * kMaxTop - kWarps * kMaxTop;  // candidates of a CTA, besides its warps' lists
constexpr int kPieces = 8192;      // pieces that the workspace holds
constexpr int kMaxSplit = 256;     // pieces of a row, one per thread of the CTA that joins them
constexpr int kNoTau = (int)0x807FFFFF;  // minus infinity as an ordered whole number
constexpr float kFar = 1e8f;       // |shift| from which on terms are taken plainly; below it |lag| <= 4
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct Cand {  // a logit and its index; better: larger, then the lower index
    float x;
    int i;
};
__device__ __forceinline__ bool better(float x, int i, float y, int j) { return x > y || (x == y && i < j); }

struct Stats {  // of some of a row's logits, in powers of two of (x - ref) * scale
    float ref;   // the largest, or one larger than all of them; minus infinity where there is none
    int own;     // the index of the logit that is ref and is not in the sums; none: ref belongs to others
    float s, t;  // sum of e and of e log2 e
    int before;  // logits ahead of the target
};
struct __align__(16) Piece {
    Stats st;
    Cand top[kMaxTop];
};

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// Pairs of fp32 in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{.reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 z, x, y;\n mov.b64 {%0, %1}, z;}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{.reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z;}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

__device__ __forceinline__ float logit(const uint16_t* p, int64_t i) { return bf16lo_to_f32(p[i]); }
__device__ __forceinline__ float logit(const float* p, int64_t i) { return p[i]; }

// What the kernel does with the 16 bytes of a load, by type: the logits, the largest (a NaN is passed over), how many
// are above a threshold, and bits of all minus infinity.
struct Bf16Load {
    static constexpr int E = 8;
    static constexpr uint32_t kNone = 0xFF80FF80u;
    static __device__ __forceinline__ void spread(uint4 v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = bf16lo_to_f32(w[i]), x[2 * i + 1] = bf16hi_to_f32(w[i]);
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t largest2(uint4 v) { return max2(max2(v.x, v.y), max2(v.z, v.w)); }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max2(a, b); }
    static __device__ __forceinline__ float value(uint32_t m) { return fmaxf(bf16lo_to_f32(m), bf16hi_to_f32(m)); }
    // not below `low`, a pair (a NaN stays one)
    static __device__ __forceinline__ uint4 at_least(uint4 v, uint32_t low) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(w[i]) : "r"(w[i]), "r"(low));
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // the next bf16 pair below a finite x
    static __device__ __forceinline__ uint32_t below(float x) {
        const uint32_t b = __float_as_uint(x) >> 16;
        return threshold((uint16_t)(x > 0.f ? (b == 0 ? 0x8001 : b - 1) : (b | 0x8000) + 1));
    }
    static __device__ __forceinline__ uint32_t above2(uint32_t a, uint32_t b) {  // 1 or 0 in bf16
        uint32_t r;
        asm("set.gt.bf16x2.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ float half(uint32_t w, int j) { return j & 1 ? bf16hi_to_f32(w) : bf16lo_to_f32(w); }
    // `low` in the place of logit j, where the load has it
    static __device__ __forceinline__ uint4 put(uint4 v, int j, uint32_t low) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (j >> 1 == i) w[i] = __byte_perm(w[i], low, j & 1 ? 0x5410 : 0x3254);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // Counts of the logits above a threshold, a pair; at most 4 each per load, exact up to 256.
    static __device__ __forceinline__ uint32_t above(uint4 v, uint32_t thr, uint32_t n) {
        return add(n, add(add(above2(v.x, thr), above2(v.y, thr)), add(above2(v.z, thr), above2(v.w, thr))));
    }
    static __device__ __forceinline__ float count(uint32_t n) { return bf16lo_to_f32(n) + bf16hi_to_f32(n); }
    static __device__ __forceinline__ uint32_t threshold(uint16_t x) { return x | (uint32_t)x << 16; }
    // the threshold that everything not below x is above (x finite or plus infinity)
    static __device__ __forceinline__ uint32_t threshold_below(uint16_t x) {
        return threshold((x & 0x7FFF) == 0 ? 0x8001 : x & 0x8000 ? x + 1 : x - 1);
    }
};
struct F32Load {
    static constexpr int E = 4;
    static constexpr uint32_t kNone = 0xFF800000u;
    static __device__ __forceinline__ void spread(uint4 v, float* x) {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ uint32_t largest2(uint4 v) {
        return __float_as_uint(fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w))));
    }
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    static __device__ __forceinline__ float value(uint32_t m) { return __uint_as_float(m); }
    static __device__ __forceinline__ uint4 at_least(uint4 v, uint32_t low) {
        const float l = __uint_as_float(low);
        return make_uint4(__float_as_uint(max_nan(__uint_as_float(v.x), l)), __float_as_uint(max_nan(__uint_as_float(v.y), l)),
                          __float_as_uint(max_nan(__uint_as_float(v.z), l)), __float_as_uint(max_nan(__uint_as_float(v.w), l)));
    }
    static __device__ __forceinline__ uint32_t below(float x) { return __float_as_uint(x); }
    static __device__ __forceinline__ float half(uint32_t w, int) { return __uint_as_float(w); }
    static __device__ __forceinline__ uint4 put(uint4 v, int j, uint32_t low) {
        return make_uint4(j == 0 ? low : v.x, j == 1 ? low : v.y, j == 2 ? low : v.z, j == 3 ? low : v.w);
    }
    static __device__ __forceinline__ float above1(uint32_t a, uint32_t b) {
        float r;
        asm("set.gt.f32.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
        return r;
    }
    static __device__ __forceinline__ uint32_t above(uint4 v, uint32_t thr, uint32_t n) {
        return __float_as_uint(__uint_as_float(n) + ((above1(v.x, thr) + above1(v.y, thr)) + (above1(v.z, thr) + above1(v.w, thr))));
    }
    static __device__ __forceinline__ float count(uint32_t n) { return __uint_as_float(n); }
    static __device__ __forceinline__ uint32_t threshold(float x) { return __float_as_uint(x); }
    static __device__ __forceinline__ uint32_t threshold_below(float x) {
        const uint32_t b = __float_as_uint(x);
        return x == 0.f ? 0x80000001u : b >> 31 ? b + 1 : b - 1;
    }
};
template <typename T>
struct LoadOf;
template <>
struct LoadOf<uint16_t> { using type = Bf16Load; };
template <>
struct LoadOf<float> { using type = F32Load; };

// b joined to a: the sums taken to the larger ref, the term of a smaller one that was left out added.
__device__ __forceinline__ void merge(Stats& a, const Stats& b, float c2) {
    const bool swap = better(b.ref, b.own, a.ref, a.own);
    const float hi = swap ? b.ref : a.ref, lo = swap ? a.ref : b.ref;
    const float s_hi = swap ? b.s : a.s, t_hi = swap ? b.t : a.t, s_lo = swap ? a.s : b.s, t_lo = swap ? a.t : b.t;
    const bool none = lo == -CUDART_INF_F;
    const float one = (swap ? a.own : b.own) != INT_MAX ? 1.f : 0.f;
    const float d = none ? 0.f : max_nan((lo - hi) * c2, -1000.f), f = none ? 0.f : exp2_fast(d);
    if (swap) a.ref = b.ref, a.own = b.own;
    a.s = s_hi + f * (s_lo + one);
    a.t = t_hi + f * (t_lo + d * (s_lo + one));
    a.before += b.before;
}

// How many of n candidates in shared memory (a multiple of 2, the rest of the last pair no candidate) are better.
__device__ __forceinline__ int place(const Cand* c, int n, Cand x) {
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 2) {
        const int4 v = *reinterpret_cast<const int4*>(c + j);
        r += better(__int_as_float(v.x), v.y, x.x, x.i);
        r += better(__int_as_float(v.z), v.w, x.x, x.i);
    }
    return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) token_logprobs_kernel(LogprobArgs a, int split) {
    using L = typename LoadOf<T>::type;
    constexpr int E = L::E, AHEAD = 4;  // loads of a thread in flight
    __shared__ Stats sm_stats[kWarps];
    __shared__ __align__(16) Cand sm_cand[kMaxTop * kMaxTop + 2];  // the warps' lists; later the entries of a row's pieces that can win
    __shared__ Cand sm_top[kMaxTop];
    __shared__ int sm_tau;  // k-th best logit of some warp of the CTA, as an ordered whole number
    __shared__ Cand sm_bound;    // the K-th best head of a row's pieces
    __shared__ int sm_seeds[kWarps * (kMaxTop / kWarps + 3)];
    __shared__ int sm_ref, sm_n, sm_lists, sm_last, sm_list[kMaxTop];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, K = a.top_k;
    const unsigned row = blockIdx.x / (unsigned)split, piece = blockIdx.x - row * split;
    const T* x = static_cast<const T*>(a.logits) + (int64_t)row * a.row_stride;
    const int V = (int)a.V;
    const float c2 = a.scale * kLog2e;

    // Loads are of 16 aligned bytes: load v holds the logits v * E - skew ...; those of [full0, full1) lie in the row
    const int skew = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    const uint4* xv = reinterpret_cast<const uint4*>(x - skew);
    const unsigned loads = ((unsigned)V + skew + E - 1) / E, each = loads / split, rest = loads - each * split;
    const int v0 = (int)(piece * each + min(piece, rest)), v1 = v0 + (int)(each + (piece < rest));
    // A row's first and last 16 bytes may not all be its own: such loads are made logit by logit, by one thread in a
    // turn of their own before and behind the others, minus infinity in the place of what is not the row's.
    const int full0 = skew ? 1 : 0, full1 = (int)(((unsigned)V + skew) / E), first = max(v0, full0), last = min(v1, full1);
    const uint4 none4 = make_uint4(L::kNone, L::kNone, L::kNone, L::kNone);
    auto load = [&](int v) {
        uint4 raw = none4;
        if (v < last) raw = ld_stream16(xv + v);
        return raw;
    };
    auto load_part = [&](int v) {
        uint32_t w[4] = {none4.x, none4.y, none4.z, none4.w};
        if (tid == 0) {
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int64_t i = (int64_t)v * E - skew + j;
                if (i < 0 || i >= V) continue;
                if (sizeof(T) == 4)
                    w[j & 3] = __float_as_uint(logit(x, i));
                else
                    w[j >> 1] = __byte_perm(w[j >> 1], __float_as_uint(logit(x, i)) >> 16, j & 1 ? 0x5410 : 0x3254);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    const bool head_part = v0 < first, tail_part = v1 > max(first, last);  // a row of one load is all head
    uint4 ring[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) ring[u] = load(first + u * kThreads + tid);
    if (tid == 0) sm_tau = sm_ref = kNoTau, sm_n = 0;
    __syncthreads();

    int target = a.targets ? a.targets[row] : -1;
    if (target >= V) {
        if (tid == 0) atomicExch(&g_logprobs_range, 1);
        target = -1;
    }
    const int tv = target < 0 ? INT_MAX : (int)(((unsigned)target + skew) / E);
    const float xt = target < 0 ? CUDART_INF_F : logit(x, target);
    const bool dead = xt == -CUDART_INF_F;  // a masked target: behind all logits of lower index
    // Ahead of the target are, at lower indexes, the logits not below it, at higher ones those above it; the load that
    // holds the target counts as one of higher indexes, and is put right at the end. (Of a dead target's lower ones
    // none is counted: minus infinity plus one bit is a NaN.)
    const uint32_t after = L::threshold(target < 0 ? T(L::kNone) : x[target]);
    const uint32_t until = target < 0 ? after : L::threshold_below(x[target]);

    Stats st = {-CUDART_INF_F, INT_MAX, 0.f, 0.f, 0};
    float2 s2 = make_float2(0.f, 0.f), t2 = s2;
    float counted = 0.f;
    // y = (x - best) * c2 as x c2 + shift in one operation. shift is off by -lag, for all logits alike, which is put
    // right when best moves and at the end. Logits are first raised to `low`, where y is below -150 and finite: their
    // e is 0, and 0 times it. Where best is kFar away or more (a mask of finite numbers over a whole row), plainly: lag
    // would not stay small beside fp32's range, nor 160 / c2 beside best's own last place.
    float shift = 0.f, lag = 0.f;
    uint32_t low = 0;
    bool plain = true;
    Cand mine = {-CUDART_INF_F, INT_MAX};  // the warp's list, in order: entry `lane`
    float gate = -CUDART_INF_F;  // no logit up to this one moves the maximum or enters the list
    // Where the first loads, which make the gate, are a fair share of the piece, few pass it: they go into a buffer of the
    // CTA, ranked at the end. In long pieces the lists let the gate rise. (50 rows in 9 pieces each, the 32 best: 44 us with
    // lists; 2000 rows of one piece with a buffer would rank some 30 times the tokens asked for.)
    const bool append = v1 - v0 <= 6 * kThreads * AHEAD;

    // Logits as ordered whole numbers (a NaN below all), and back.
    auto tau_of = [](float v) {  // an ordered whole number, and back
        const int b = __float_as_int(fmaxf(v, -CUDART_INF_F) + 0.f);  // zeros of both signs tie
        return b < 0 ? b ^ 0x7FFFFFFF : b;
    };

    auto value_of = [](int t) { return __int_as_float(t < 0 ? t ^ 0x7FFFFFFF : t); };

    auto before_of = [](float v) {  // the number below
        const int b = __float_as_int(v);
        return v == -CUDART_INF_F ? v : v == 0.f ? -1.4012985e-45f : __int_as_float(b > 0 ? b - 1 : b + 1);
    };

    auto moved = [&](float by) {  // the sums as if every y had been so much larger
        const float f = exp2_fast(by);
        t2 = make_float2(f * fmaf(by, s2.x, t2.x), f * fmaf(by, s2.y, t2.y));
        s2 = make_float2(f * s2.x, f * s2.y);
    };
    auto settle = [&]() { moved(lag); };  // as if y had been exact
    auto sum_fast = [&](const float* e) {
        const float2 sh = make_float2(shift, shift), cc = make_float2(c2, c2);
#pragma unroll
        for (int j = 0; j < E; j += 2) {
            const float2 y = fma2(make_float2(e[j], e[j + 1]), cc, sh), p = make_float2(exp2_fast(y.x), exp2_fast(y.y));
            s2 = add2(s2, p);
            t2 = fma2(p, y, t2);
        }
    };

    // Logit j (0 .. AHEAD * E - 1) of the thread's loads in hand.
    auto pick = [&](int j) {
        uint32_t w = ring[0].x;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const uint32_t r[4] = {ring[u].x, ring[u].y, ring[u].z, ring[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (j / (E / 4) == 4 * u + i) w = r[i];
        }
        return L::half(w, j);
    };
    auto refer = [&](float x) {
        st.ref = x;
        shift = -x * c2, lag = fmaf(-x, c2, -shift);
        const float cut = x - 160.f / c2;
        plain = !(fabsf(shift) < kFar) || !(cut > -1e37f) || !(x < 1e37f);
        low = L::below(cut);
    };
    // Where the largest of the loads in hand is, among equals the first: its number in them, and its index.
    auto where = [&](int base, float x, int& own, int& at) {
        own = -1, at = INT_MAX;
#pragma unroll
        for (int u = AHEAD - 1; u >= 0; --u) {
            float e[E];
            L::spread(ring[u], e);
#pragma unroll
            for (int j = E - 1; j >= 0; --j)
                if (e[j] == x) own = u * E + j;
        }
        if (own >= 0) at = (base + own / E * kThreads) * E - skew + own % E;
    };
    // Some of the loads in hand holds a logit past the gate. `base`: the first one's number, the others kThreads apart.
    auto past_gate = [&](int base, float big, int& excluded) {
        if (__any_sync(0xFFFFFFFFu, big > st.ref)) {  // ---- the maximum ----
            const float wm = value_of(__reduce_max_sync(0xFFFFFFFFu, tau_of(big)));
            int at = INT_MAX, own = -1;
            if (big == wm) where(base, wm, own, at);
            const int first_at = __reduce_min_sync(0xFFFFFFFFu, at);
            if (at != first_at) own = -1;
            const bool none = st.ref == -CUDART_INF_F;
            const float d = none ? 0.f : max_nan((st.ref - wm) * c2, -1000.f), f = none ? 0.f : exp2_fast(d);
            if (!plain) settle();
            if (lane == 0 && st.own != INT_MAX) s2.x += 1.f;
            // f = 0 keeps a NaN that the sums hold
            t2 = make_float2(f * (t2.x + d * s2.x), f * (t2.y + d * s2.y));
            s2 = make_float2(f * s2.x, f * s2.y);
            st.own = first_at;
            refer(wm);
            if (!plain) moved(-lag);  // as the terms to come are
            excluded = own;
        }
        gate = st.ref;
        if (K > 0) {  // ---- the list ----
            const float kth = __shfl_sync(0xFFFFFFFFu, mine.x, K - 1);
            const float floor = value_of(*reinterpret_cast<volatile int*>(&sm_tau));
            // behind this warp's K-th, or below the gate of all: not among the K best
            uint32_t has = 0;
            if (big > kth && big >= floor) {
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    float e[E];
                    L::spread(ring[u], e);
#pragma unroll
                    for (int j = 0; j < E; ++j) has |= (uint32_t)(e[j] > kth && e[j] >= floor) << (u * E + j);
                }
            }
            if (append && __any_sync(0xFFFFFFFFu, has != 0)) {
                int n = __popc(has), at = n;  // the lanes' places in the CTA's buffer
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xFFFFFFFFu, at, o);
                    if (lane >= o) at += y;
                }
                int start = 0;
                if (lane == 31) start = atomicAdd(&sm_n, at);
                at += __shfl_sync(0xFFFFFFFFu, start, 31) - n;
                for (; __any_sync(0xFFFFFFFFu, has != 0 && at < kBuffer); ++at) {
                    const int b = __ffs(has) - 1;
                    const float v = pick(b);
                    if (has && at < kBuffer) {
                        sm_cand[at] = {v, (base + b / E * kThreads) * E - skew + b % E};
                        has &= has - 1;
                    }
                }
            }
            uint32_t lanes = __ballot_sync(0xFFFFFFFFu, has != 0);  // with no place there: into the warp's list
            float now = kth;
            if (lanes) {
                do {
                    const int from = __ffs(lanes) - 1, b = __ffs(has) - 1;
                    const int ci = __shfl_sync(0xFFFFFFFFu, (base + b / E * kThreads) * E - skew + b % E, from);
                    const float cx = __shfl_sync(0xFFFFFFFFu, pick(b), from);
                    if (lane == from) has &= has - 1;
                    const int pos = __popc(__ballot_sync(0xFFFFFFFFu, better(mine.x, mine.i, cx, ci)));
                    const float ux = __shfl_up_sync(0xFFFFFFFFu, mine.x, 1);
                    const int ui = __shfl_up_sync(0xFFFFFFFFu, mine.i, 1);
                    if (lane > pos) mine.x = ux, mine.i = ui;
                    if (lane == pos) mine.x = cx, mine.i = ci;
                    lanes = __ballot_sync(0xFFFFFFFFu, has != 0);
                } while (lanes);
                now = __shfl_sync(0xFFFFFFFFu, mine.x, K - 1);
                if (lane == 0 && now > floor) atomicMax(&sm_tau, tau_of(now));
            }
            // a logit equal to another warp's K-th may still be ahead of it, one equal to this warp's not
            gate = fminf(fmaxf(now, before_of(floor)), st.ref);
        }
    };

#pragma unroll 1
    for (int phase = head_part ? 0 : 1; phase < (tail_part ? 3 : 2); ++phase) {
        int base = first + tid, end = last;
        if (phase != 1) {  // one load, of thread 0
            base = phase == 0 ? v0 : v1 - 1;
            end = base + 1;
            ring[0] = load_part(base);
#pragma unroll
            for (int u = 1; u < AHEAD; ++u) ring[u] = none4;
        } else {
            if (head_part) {
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) ring[u] = load(base + u * kThreads);
            }
            // The CTA's largest logit so far is what its other warps refer to at first: each with its own largest, they
            // would have to move it some three times more. And a first gate for the lists: of the largest logits of
            // each warp's best `seeds` lanes the K-th largest, which is not above the K-th best logit of the CTA.
            uint32_t most = L::largest2(ring[0]);
#pragma unroll
            for (int u = 1; u < AHEAD; ++u) most = L::larger(most, L::largest2(ring[u]));
            const float big = L::value(most);
            int o = tau_of(big), t = __reduce_max_sync(0xFFFFFFFFu, o);
            const int top = t, seeds = min(K, (K + kWarps - 1) / kWarps + 3);
            for (int r = 0; r < seeds; ++r) {
                const uint32_t who = __ballot_sync(0xFFFFFFFFu, o == t);
                if (lane == __ffs(who) - 1) sm_seeds[warp * seeds + r] = t, o = kNoTau;
                t = __reduce_max_sync(0xFFFFFFFFu, o);
            }
            if (lane == 0) atomicMax(&sm_ref, top);
            __syncthreads();
            const int ref = sm_ref;
            if (tid < kWarps * seeds) {
                const int own = sm_seeds[tid];
                int ahead = 0;
                for (int j = 0; j < kWarps * seeds; ++j) {
                    const int v = sm_seeds[j];
                    ahead += v > own || (v == own && j < tid);
                }
                if (ahead == K - 1) atomicMax(&sm_tau, own);
            }
            if (top != ref && st.ref == -CUDART_INF_F) {
                refer(value_of(ref));
                if (K == 0) gate = st.ref;
            }
            if (K > 0) __syncthreads();
            if (K > 0 && st.ref != -CUDART_INF_F) gate = fminf(before_of(value_of(sm_tau)), st.ref);
            __syncthreads();
        }
        const int step = phase == 1 ? tid : 0;
#pragma unroll 1
        for (; base - step < end; base += kThreads * AHEAD) {
            uint4 next[AHEAD];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) next[u] = phase == 1 ? load(base + (AHEAD + u) * kThreads) : none4;
            uint32_t most = L::largest2(ring[0]), n = 0;
#pragma unroll
            for (int u = 1; u < AHEAD; ++u) most = L::larger(most, L::largest2(ring[u]));
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) n = L::above(ring[u], base + u * kThreads < tv ? until : after, n);
            counted += L::count(n);
            int excluded = -1;  // the maximum itself is not summed
            if (__any_sync(0xFFFFFFFFu, L::value(most) > gate)) past_gate(base, L::value(most), excluded);
            if (plain) {
                for (int j = 0; j < AHEAD * E; ++j) {
                    const float ref = st.ref == -CUDART_INF_F ? 0.f : st.ref;
                    const float y = j == excluded ? -1000.f : max_nan((pick(j) - ref) * c2, -1000.f), p = exp2_fast(y);
                    s2.x += p, t2.x = fmaf(p, y, t2.x);
                }
            } else {
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    uint4 v = L::at_least(ring[u], low);
                    if (excluded >= 0) v = L::put(v, excluded - u * E, low);
                    float e[E];
                    L::spread(v, e);
                    sum_fast(e);
                }
            }
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) ring[u] = next[u];
        }
    }
    if (!plain) settle();
    int before = (int)counted;
    if (tid == 0 && tv >= v0 && tv < v1)  // the target's own load
        for (int i = max(tv * E - skew, 0); i < target; ++i) {
            const float v = logit(x, i);
            before += dead ? -(v > xt) : v == xt;
        }

    // ---- the warps' numbers and lists ----
    st.s = warp_sum(s2.x + s2.y);
    st.t = warp_sum(t2.x + t2.y);
    st.before = __reduce_add_sync(0xFFFFFFFFu, before);
    if (lane == 0) sm_stats[warp] = st;
    __syncthreads();
    // The lanes' numbers joined over n lanes, a power of two.
    auto joined = [&](Stats sum, int n) {
        for (int o = n / 2; o > 0; o >>= 1) {
            Stats q;
            q.ref = __shfl_xor_sync(0xFFFFFFFFu, sum.ref, o), q.own = __shfl_xor_sync(0xFFFFFFFFu, sum.own, o);
            q.s = __shfl_xor_sync(0xFFFFFFFFu, sum.s, o), q.t = __shfl_xor_sync(0xFFFFFFFFu, sum.t, o);
            q.before = __shfl_xor_sync(0xFFFFFFFFu, sum.before, o);
            merge(sum, q, c2);
        }
        return sum;
    };
    Stats all = {-CUDART_INF_F, INT_MAX, 0.f, 0.f, 0};
    if (warp == 0) all = joined(sm_stats[lane % kWarps], kWarps);
    // The first K of what is in sm_cand, by rank, into sm_top; the rest of it empty.
    auto rank = [&]() {
        const int n = sm_n;
        if (tid == 0 && (n & 1)) sm_cand[n] = {-CUDART_INF_F, INT_MAX};
        __syncthreads();
        for (int j = tid; j < n; j += kThreads) {
            const Cand c = sm_cand[j];
            const int r = place(sm_cand, n, c);
            if (r < K) sm_top[r] = c;
        }
        if (tid >= n && tid < K) sm_top[tid] = {-CUDART_INF_F, INT_MAX};
        __syncthreads();
    };
    if (K > 0) {
        if (tid == 0) sm_n = min(sm_n, kBuffer);
        __syncthreads();
        const int tau = sm_tau;  // entries below it are not among the K best; the order of the others does not matter
        if (lane < K && mine.i != INT_MAX && tau_of(mine.x) >= tau) sm_cand[atomicAdd(&sm_n, 1)] = mine;
        __syncthreads();
        rank();
    }

    if (split > 1) {
        uint32_t* counters = static_cast<uint32_t*>(a.workspace);
        Piece* pieces = reinterpret_cast<Piece*>(counters + kPieces);
        Piece* own = pieces + blockIdx.x;
        if (tid == 0) own->st = all;
        if (tid < K) own->top[tid] = sm_top[tid];
        __syncthreads();
        if (tid == 0) {
            __threadfence();  // the piece before its count
            sm_last = atomicInc(counters + row, split - 1) == (unsigned)split - 1;  // back to 0 behind the last
            __threadfence();
            sm_n = sm_lists = 0;
            sm_bound = {-CUDART_INF_F, INT_MAX};
        }
        __syncthreads();
        if (!sm_last) return;
        const Piece* of = pieces + (int64_t)row * split;
        // Where there are fewer pieces than K, each holds `deep` entries that are not behind the worst of the deep-th ones:
        // K in all, so that what is behind that is not among the K best.
        const int deep = split < K ? (K + split - 1) / split : 1;
        Cand head = {-CUDART_INF_F, INT_MAX};
        if (K > 0) {
            if (tid < split) head = {__ldcg(&of[tid].top[deep - 1].x), __ldcg(&of[tid].top[deep - 1].i)};
            sm_cand[tid] = head;  // those past split are no candidates
        }
        if (warp == 0) {  // the pieces in their order, 32 at a time to the warp's lanes, then those
            Stats sum = {-CUDART_INF_F, INT_MAX, 0.f, 0.f, 0};
            for (int p = lane; p < split; p += 32) {
                Stats q;
                q.ref = __ldcg(&of[p].st.ref), q.own = __ldcg(&of[p].st.own), q.s = __ldcg(&of[p].st.s);
                q.t = __ldcg(&of[p].st.t), q.before = __ldcg(&of[p].st.before);
                merge(sum, q, c2);
            }
            all = joined(sum, 32);
        }
        __syncthreads();
        if (K > 0) {
            // Else only the pieces with the K best heads can hold one of the row's K best, in entries not behind the K-th.
            if (head.i != INT_MAX) {
                const int r = place(sm_cand, split, head);
                if (split >= K && r < K) sm_list[atomicAdd(&sm_lists, 1)] = tid;
                if (r == min(split, K) - 1) sm_bound = head;
            }
            if (split < K && tid < split) sm_list[atomicAdd(&sm_lists, 1)] = tid;
            __syncthreads();
            const int entries = sm_lists * K;
            const Cand bound = sm_bound;
            for (int j = tid; j < entries; j += kThreads) {
                const Cand* at = &of[sm_list[j / K]].top[j % K];
                const Cand e = {__ldcg(&at->x), __ldcg(&at->i)};
                if (e.i != INT_MAX && !better(bound.x, bound.i, e.x, e.i)) sm_cand[atomicAdd(&sm_n, 1)] = e;
            }
            __syncthreads();
            rank();
        }
    }

    if (warp != 0) return;
    const bool none = all.ref == -CUDART_INF_F;
    const float s = all.s + (none ? 0.f : all.ref - all.ref);  // plus infinity gives NaN
    const float lse = log1pf(s);
    if (tid == 0) {
        if (a.logprob) a.logprob[row] = target < 0 ? 0.f : none ? -CUDART_INF_F + s : (xt - all.ref) * a.scale - lse;
        if (a.rank) a.rank[row] = target < 0 ? 0 : 1 + all.before + (dead ? target : 0);
        if (a.entropy) a.entropy[row] = none ? s : lse - kLn2 * all.t / (1.f + s);
    }
    if (tid < K) {
        const Cand c = sm_top[tid];
        const bool no = c.i == INT_MAX;
        if (a.top_ids) a.top_ids[(int64_t)row * K + tid] = no ? -1 : c.i;
        if (a.top_logprobs) a.top_logprobs[(int64_t)row * K + tid] = no ? -CUDART_INF_F + s : (c.x - all.ref) * a.scale - lse;
    }
}

}  // namespace

size_t token_logprobs_workspace() { return kPieces * sizeof(uint32_t) + (size_t)kPieces * sizeof(Piece); }

cudaError_t launch_token_logprobs(const LogprobArgs& a, cudaStream_t s) {
    // Pieces of at least 2048 logits, in whole waves of three CTAs per SM as far as that goes: a piece costs what its
    // logits do and as much as some 20,000 more.
    int64_t split = 1;
    if (a.ws_bytes >= token_logprobs_workspace()) {
        const int64_t slots = 3 * (int64_t)device_sm_count();
        int64_t most = a.V / 2048, best = -1;
        if (most > kMaxSplit) most = kMaxSplit;
        for (int64_t n = 1; n <= most && (n == 1 || n * a.M <= kPieces); ++n) {
            const int64_t cost = (a.M * n + slots - 1) / slots * (a.V / n + 20000);
            if (best < 0 || cost < best) best = cost, split = n;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.M * split), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attrs[1];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, a.fp32 ? token_logprobs_kernel<float> : token_logprobs_kernel<uint16_t>, a, (int)split);
}

int logprobs_take_range() {
    int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_logprobs_range, sizeof(int)) != cudaSuccess) return -1;
    if (v) cudaMemcpyToSymbol(g_logprobs_range, &z, sizeof(int));
    return v;
}

}  // namespace mbw
