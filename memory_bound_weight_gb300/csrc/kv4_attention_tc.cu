// kv4_attention_tc.cu -- attention over the 4-bit paged cache for chunks of a
// prompt: many query rows per KV head, on tcgen05 with the scores, the weights,
// the queries and the outputs in TMEM. The formulas are those of
// kv4_attention.cu; that kernel takes few rows per request.
//
// An item is a tile of 128 query rows (query tokens x heads of the group) of
// one KV head of one request; its keys come 128 at a time.
//
// Mathematics. With 128 rows the codes are worth unpacking into operands:
//   k = s n + m = s (n - 8) + (m + 8 s)
// The first part, at most 8 s, is rounded to fp16, which moves it by at most
// 2^-11 of itself, 2^-8 of a step of the quantization; the offset m + 8 s enters
// unrounded, as two fp16 numbers (value and remainder) in columns of their own
// beside the sums of q, also two fp16 numbers, so that a channel far from zero
// costs no precision:
//   q . k = sum q k' + sum over groups (m + 8 s) sum q
// (Where 8 s would pass fp16, s > 8188, 7.5 takes the place of 8: n - 7.5 times
// s then fits.) V likewise: v' are the columns of the second product's B operand,
// the offsets' two parts more columns, and a column of ones sums the weights as
// they were rounded, so that a weight's rounding acts on the distance of v from
// the result alone. The weights are fp16 of 2^7 p; p refers to a maximum that
// follows the true one only when it has grown by 2^8 (2^7 p <= 2^15 then), which
// spares the outputs in TMEM most rescalings. q is scaled per row by a power of
// two to at most 2^8, so that sums of 64 of them stay in fp16's range and bf16
// entries down to 2^-24 of the largest stay exact.
//
// Work. A CTA has 8 warps of softmax (two threads per row, each half its scores and
// outputs, in its TMEM lane), 16 that unpack K and V of a block of 16 keys each, of
// even or of odd tiles, from copies on their way under the tiles before to operands
// with 128-byte swizzle in shared memory, and one that issues the products. Scores
// are double-buffered, so that Q K of a tile runs under the softmax of the one
// before; the weights take the place of the scores. Q is an operand in TMEM: from
// shared memory the first product would read twice as much there. Items are cut
// along the keys between CTAs where there are at most half as many as SMs, and
// joined by the CTA that arrives last, in order.
//
// What bounds it: instructions. A tile of 128 keys takes some 2600 cycles, in which
// an SM issues about 8000 instructions, three quarters of what it can, two thirds of
// them to unpack; the tensor pipe is busy for 40% of them. On the way there, for 3
// requests of 90 to 200 queries of 32 heads that see 2048 keys each (15 GFLOP): 101
// us with m16n8k16 in kv4_attention.cu; 46 with 8 warps that unpack from registers,
// in the order of which a fence waits for the loads behind it; 39 with copies and
// offsets one a lane; 38 with the constants of the unpacking kept in registers; 35
// with shared memory addressed as such, not through generic pointers; 31 with the
// maximum taken in the pass of the weights, the first item found by one warp, halves
// of Q read by halves of the softmax, and joins at the roles' ends (33 with a join
// behind each piece, whose registers the loops paid for): 500 TFLOP/s. 16 requests of
// 32 queries of 32 heads and 4000 tokens take 50 us, 665 TFLOP/s.
//
// Tokens that some rows do not see may hold no numbers, or bytes that no append
// wrote, whose products pass fp16; and 0 times NaN is not 0: V's groups of either
// kind become zeros, and where there was one in an item, its rows look at the tokens
// that they see once more at the end.
#include <cuda_runtime.h>

#include <math_constants.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "kv4.cuh"

namespace mbw {

namespace {

__device__ int g_kv4_tc_range;  // a page id, length or query offset was out of range
__device__ int g_kv4_tc_fault;  // a bounded wait expired

__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void bar_init(uint64_t* bar, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_at(bar)), "r"(count));
}
__device__ __forceinline__ void bar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_at(bar)) : "memory");
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
    if (!got) atomicExch(&g_kv4_tc_fault, 1), ok = false;
    __syncwarp();
}
// The warpgroup's registers a thread from here on.
template <int N>
__device__ __forceinline__ void registers(bool more) {
    if (more)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ bool elect() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_at(bar)) : "memory");
}

// 32 or 16 columns of the thread's TMEM lane.
__device__ __forceinline__ void ld32(uint32_t* v, uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(at));
}
__device__ __forceinline__ void ld16(uint32_t* v, uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(at));
}
__device__ __forceinline__ void st16(uint32_t at, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void st8(uint32_t at, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// The loads before this are there, those of v among them, which is not used before.
__device__ __forceinline__ void wait_ld16(uint32_t* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void wait_ld(uint32_t* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]),
                   "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                   "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29])
                 :
                 : "memory");
    asm volatile("" : "+r"(v[30]), "+r"(v[31]));
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{.reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z;}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Whether x holds for any of the 64 threads of two warps.
__device__ __forceinline__ bool bar_any(int bar, bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbarrier.cta.red.or.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(bar), "r"((uint32_t)x) : "memory");
    return r != 0;
}

// K-major operand in rows of 128 bytes (64 fp16), 8-row atoms of 1024 bytes with 128-byte swizzle.
__device__ __forceinline__ uint64_t desc(uint32_t at) {
    return (uint64_t)((at >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// kind::f16: A and B fp16, D fp32, both K-major
__host__ __device__ constexpr uint32_t idesc(int m, int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24); }

__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool add) {  // A in TMEM
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(id), "r"((uint32_t)add)
                 : "memory");
}

__device__ __forceinline__ uint32_t h2(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }
__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }
__device__ __forceinline__ uint32_t pack(float a, float b) { return h2(__floats2half2_rn(a, b)); }
// The same, the largest finite number in the place of what is beyond it (a NaN stays one).
__device__ __forceinline__ uint32_t pack_finite(float a, float b) {
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Nibbles 0 and 4, 1 and 5, 2 and 6, 3 and 7 of a word, less 8 each, times s and plus d: the codes ORed into the bits of
// 1024 and of 64, an exact subtraction, one rounding. The constants are held in registers, opaque to the compiler, which
// else puts a move beside every use.
struct Unpack {
    uint32_t one, two, c1, c2;  // 1024 and 64, twice; 1032 and 72
    __device__ __forceinline__ Unpack() {
        asm volatile("mov.b32 %0, 0x64006400;" : "=r"(one));
        asm volatile("mov.b32 %0, 0x54005400;" : "=r"(two));
        asm volatile("mov.b32 %0, 0x64086408;" : "=r"(c1));
        asm volatile("mov.b32 %0, 0x54805480;" : "=r"(c2));
    }
    template <int I>
    __device__ __forceinline__ uint32_t pair(uint32_t w, uint32_t s, uint32_t d) const {
        uint32_t x, y;
        if (I & 1)
            asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0xEA;" : "=r"(x) : "r"(w), "r"(two));
        else
            asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(x) : "r"(w), "r"(one));
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(I & 1 ? c2 : c1));
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(x) : "r"(y), "r"(s), "r"(d));
        return x;
    }
    __device__ __forceinline__ void operator()(uint32_t w, uint32_t s, uint32_t d, uint32_t* o) const {
        const uint32_t v = w >> 8;
        o[0] = pair<0>(w, s, d), o[1] = pair<1>(w, s, d), o[2] = pair<2>(v, s, d), o[3] = pair<3>(v, s, d);
    }
};

// Half a step where the centre is 7.5 codes, in place of 8, whose product with the scale would pass fp16; else 0.
__device__ __forceinline__ uint32_t half_step(uint32_t s2) {
    return h2(__hmul2(as_h2(s2), as_h2(0x38003800u))) & __hgt2_mask(as_h2(s2), as_h2(0x6FFF6FFFu));  // 0.5; 8188
}
// The centre's value of a (scale, minimum) pair, in two fp16 parts: value, remainder.
__device__ __forceinline__ uint32_t offset_of(uint32_t m) {
    const float2 sm = kv4_pair(m);
    const float c = fmaf(sm.x > 8188.f ? 7.5f : 8.f, sm.x, sm.y);
    const uint32_t hi = pack(c, 0.f);
    return pack(__half2float(__ushort_as_half((unsigned short)hi)), c - __half2float(__ushort_as_half((unsigned short)hi)));
}
// Whether a pair, whose offset is given, makes operands that are no numbers: one that is none itself, or that an append
// does not write (of finite values its scale is at most 8704, whose 7.5 steps are 65280, or minus zero, and its centre lies
// between them), as a place that was never written may hold.
__device__ __forceinline__ bool no_number(uint32_t m, uint32_t offset) {
    const uint32_t s = m & 0xFFFFu;
    return (s > 0x7040u && s != 0x8000u) || (offset & 0x7C00u) == 0x7C00u;
}

constexpr int kRows = 128, kKeys = 128, kStages = 2;
// Warps: softmax, 8 that unpack even tiles, 8 odd ones, one that issues the products, and 3 that only fill its warpgroup.
constexpr int kSoftmax = 8, kUnpack = 8, kIssuer = kSoftmax + 2 * kUnpack, kWarps = kIssuer + 4, kThreads = kWarps * 32;
// Registers: 72 a thread at launch, 64512 in all; then by warpgroup 2 x 104 + 4 x 64 + 40 = 504, times 128 the same. A
// build with fewer at launch could not hand them out, and is not launched.
constexpr int kRegsSoftmax = 104, kRegsUnpack = 64, kRegsIssuer = 40, kRegsLaunch = 72;
static_assert(kSoftmax * kRegsSoftmax + 2 * kUnpack * kRegsUnpack + 4 * kRegsIssuer <= kWarps * kRegsLaunch, "");
constexpr int kCounters = 4096;  // of items cut between CTAs, as the other kernel's: both leave them at zero
constexpr int kUp = 7;           // weights are 2^kUp p
constexpr int kPieces = 8;       // of an item: the CTA that joins them reads 64 KB a piece, some 0.5 us
constexpr float kGrow = 8.f;     // growth of the maximum, in powers of two, that is let pass

// All warps but those that have nothing to do.
__device__ __forceinline__ void bar_joiners() { asm volatile("bar.sync 1, %0;" ::"n"((kIssuer + 1) * 32) : "memory"); }

template <int D>
struct Layout {
    static constexpr int N = D + 16;                                  // columns of the outputs: D, the offsets' parts, the weights' sum
    static constexpr int K_BOX = kKeys * 128, V_BOX = N * 128;        // 64 dimensions of 128 keys; 64 keys of N columns
    static constexpr int K_BYTES = (D / 64 + 1) * K_BOX, V_BYTES = (kKeys / 64) * V_BOX;
    static constexpr int OFF_V = kStages * K_BYTES, OFF_BAR = OFF_V + kStages * V_BYTES;
    static constexpr int OFF_RING = OFF_BAR + 256;                    // [2 kUnpack] blocks
    static constexpr int OFF_PREFIX = OFF_RING + 2 * kUnpack * kv4_block_bytes(D, 32);
    static constexpr int SMEM = OFF_PREFIX + kThreads * 16 + 1024;
    static constexpr int S_COL = 0, O_COL = 256, Q_COL = 416;         // TMEM columns
    static constexpr int PART = kRows * (D + 2);                      // floats of a part: [row][column], then maxima and sums of the rows
};

// SHARED: the items are those of one request, of all the call's queries, whose keys are the shared tokens; a row's position
// is that of its query in its own request. (The items of different requests have their rows in one tile then.) An item's
// keys are cut into a.shared_parts parts of `slots` pieces, each a CTA's of a cluster, which join theirs through shared memory;
// the parts are left to the kernel of the other tokens. (With pieces in the workspace, as elsewhere, one CTA read them all for
// 15 of a call's 40 us: 16 items of 9 pieces of 7 tiles.)
template <int D, int G, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1) kv4_attention_tc_kernel(Kv4AttnArgs a, int slots) {
    using L = Layout<D>;
    constexpr int NG = D / G, KS = D / 16;  // groups; steps of 16 in Q K, the offsets' one not counted
    static_assert(4 * NG <= 16 && 2 * NG <= 8 && kStages == 2, "the offsets' columns; a stage per set of unpacking warps");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-smem_at(smem_raw) & 1023);  // an offset, so that accesses stay known to be shared memory's
    uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
    uint64_t *kempty = kfull + kStages, *vfull = kempty + kStages, *vempty = vfull + kStages;
    uint64_t *sfull = vempty + kStages, *pfull = sfull + 2, *odone = pfull + 2, *qfull = odone + 2, *done = qfull + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    // the places before each thread's requests, and q0, nq and ctx of the one where a thread has no more
    uint4* prefix = reinterpret_cast<uint4*>(smem + L::OFF_PREFIX);
    __shared__ float sh_units[kWarps];
    __shared__ uint32_t sh_sum[kWarps], sh_items[kWarps];
    __shared__ float sh_max[2][kRows], sh_sums[2][kRows];
    __shared__ uint32_t sh_bad;  // the last key tile in which a group of V was no number, from 1

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gq = a.q_heads / a.kv_heads, bpp = a.page_size / 16;
    bool bad = false, ok = true;

    if (tid == 0) {
        sh_bad = 0;
        for (int i = 0; i < kStages; ++i) bar_init(&kfull[i], kUnpack), bar_init(&kempty[i], 1), bar_init(&vfull[i], kUnpack), bar_init(&vempty[i], 1);
        for (int i = 0; i < 2; ++i) bar_init(&sfull[i], 1), bar_init(&pfull[i], kSoftmax), bar_init(&odone[i], 1);
        bar_init(qfull, kSoftmax), bar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_at(tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    // What no tile changes: of the offsets' columns of K those past the groups', zeros; of V's last rows one of ones, for
    // the weights' sum, and zeros.
    for (int i = tid; i < kStages * L::K_BOX / 16; i += kThreads)
        *reinterpret_cast<uint4*>(smem + i / (L::K_BOX / 16) * L::K_BYTES + (D / 64) * L::K_BOX + i % (L::K_BOX / 16) * 16) = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < kStages * (kKeys / 64) * 16 * 32; i += kThreads) {
        const int word = i & 31, row = (i >> 5) & 15, box = i >> 9;
        *reinterpret_cast<uint32_t*>(smem + L::OFF_V + box * L::V_BOX + (D + row) * 128 + word * 4) = row == 2 * NG ? 0x3C003C00u : 0u;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    fence_before();
    __syncthreads();
    fence_after();

    // SHARED: the other tokens' kernel may start only where what came before this one is complete, since it waits for this one's
    // results alone, and not before it joins them.
    if (!SHARED) pdl_launch_dependents();
    pdl_wait();
    if (SHARED) pdl_launch_dependents();

    // ---- places: per request, its items times the pieces each is cut into ----
    struct Request {
        int q0, nq, ctx, tiles, units;  // row tiles per KV head; key tiles of the longest item
    };
    const int cap = a.table_width * a.page_size;
    auto sized = [&](int q0, int nq, int ctx) {
        Request r;
        r.q0 = q0, r.nq = nq, r.ctx = ctx;
        r.tiles = (int)(((uint32_t)nq * gq + kRows - 1) / kRows);
        r.units = (a.window ? min(ctx, a.window + kRows) : ctx) / kKeys + 1;
        return r;
    };
    auto request = [&](int b) {
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
        int ctx = max(a.ctx_lens[b], 0);
        if (ctx > cap) bad = true, ctx = cap;
        return sized(q0, q1 - q0, ctx);
    };
    // Offsets that fall make ranges that overlap: then there is no work, as in kv4_attention.cu. Looked for once, at the start.
    auto offsets_fall = [&](int b) { return a.q_starts && a.q_starts[b + 1] < a.q_starts[b]; };
    // Up to 32 requests are a lane's each, and every warp finds its items by itself; more are shared out over the threads.
    const bool lanes = !SHARED && a.B <= 32;
    struct Batch {  // SHARED: of the requests that have queries and tokens, the first and last query's position, and the longest
        int lo, hi, b, keys;  // with its shared tokens
    };
    __shared__ Batch sh_batch;
    const int stride = (a.B + kThreads - 1) / kThreads;  // requests per thread
    uint32_t W = 0;
    float per_unit = 0.f;
    auto pieces_of = [&](const Request& r) { return min((uint32_t)min(max(1, r.units / 2), kPieces), max(1u, (uint32_t)((float)r.units * per_unit))); };
    auto set_per_unit = [&](float units, uint32_t items) {
        per_unit = 2 * items <= (uint32_t)gridDim.x && items + gridDim.x <= (uint32_t)slots ? (float)gridDim.x / (units * a.kv_heads) : 0.f;
    };
    auto scan = [&](uint32_t n) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, n, o);
            if (lane >= o) n += y;
        }
        return n;
    };
    if (!SHARED && !lanes) {
        float units = 0.f;
        uint32_t items = 0, n = 0;
        bool falls = false;
        uint4 mine = make_uint4(0, 0, 0, 0);
        for (int i = 0; i < stride; ++i) {
            const int b = tid * stride + i;
            if (b < a.B) {
                const Request r = request(b);
                falls |= offsets_fall(b);
                mine.y = r.q0, mine.z = r.nq, mine.w = r.ctx;
                units += (float)r.tiles * (float)r.units, items += r.tiles;
            }
        }
        units = warp_sum(units), items = __reduce_add_sync(0xFFFFFFFFu, items);
        if (lane == 0) sh_units[warp] = units, sh_items[warp] = items;
        __syncthreads();
        units = 0.f, items = 0;
#pragma unroll 4
        for (int w = 0; w < kWarps; ++w) units += sh_units[w], items += sh_items[w];
        set_per_unit(units, items * a.kv_heads);
        for (int i = 0; i < stride; ++i) {
            const int b = tid * stride + i;
            if (b < a.B) {
                const Request r = stride == 1 ? sized(mine.y, mine.z, mine.w) : request(b);
                n += (uint32_t)r.tiles * a.kv_heads * pieces_of(r);
            }
        }
        const uint32_t sum = scan(n);
        if (lane == 31) sh_sum[warp] = sum;
        __syncthreads();
        uint32_t before = 0;
#pragma unroll 4
        for (int w = 0; w < kWarps; ++w) before += w < warp ? sh_sum[w] : 0, W += sh_sum[w];
        mine.x = before + sum - n;
        prefix[tid] = mine;
        if (__syncthreads_or(falls)) W = 0;
    }
    const uint32_t tmem = *tmem_slot;

    struct Item {
        int b, q0, nq, ctx, h, f0, bs, n;  // first block of its piece, key tiles of it; n < 0: past the last
        int pos_lo, pos_hi;
        uint32_t first, piece, pieces;
    };
    auto item_at = [&](uint32_t place) {
        Item it;
        Request r;
        uint32_t base;
        int b0, b1;
        if constexpr (SHARED) {
            const Batch all = sh_batch;
            b0 = kv4_first_seen(all.lo, a.window) / 16, b1 = (all.keys + 15) / 16;
            r = sized(0, a.T, 0);
            r.units = max(0, b1 - b0 + 7) / 8;
            W = (uint32_t)r.tiles * a.kv_heads * a.shared_parts * slots;
            it.n = -1, it.b = all.b, base = 0;
            if (place >= W) return it;
        } else if (lanes) {
            Request mine = {0, 0, 0, 0, 0};
            if (lane < a.B) mine = request(lane);
            set_per_unit(warp_sum((float)mine.tiles * (float)mine.units), __reduce_add_sync(0xFFFFFFFFu, (uint32_t)mine.tiles) * a.kv_heads);
            const uint32_t n = (uint32_t)mine.tiles * a.kv_heads * pieces_of(mine), sum = scan(n);
            W = __shfl_sync(0xFFFFFFFFu, sum, 31);
            it.n = -1;
            if (place >= W) return it;
            it.b = __ffs(__ballot_sync(0xFFFFFFFFu, sum > place)) - 1;
            base = __shfl_sync(0xFFFFFFFFu, sum - n, it.b);
            r = sized(__shfl_sync(0xFFFFFFFFu, mine.q0, it.b), __shfl_sync(0xFFFFFFFFu, mine.nq, it.b), __shfl_sync(0xFFFFFFFFu, mine.ctx, it.b));
        } else {
            it.n = -1;
            if (place >= W) return it;
            int lo = 0, hi = kThreads;  // the last thread whose prefix is at most place
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (prefix[mid].x <= place)
                    lo = mid;
                else
                    hi = mid;
            }
            const uint4 at_lo = prefix[lo];
            base = at_lo.x;
            it.b = lo * stride;
            r = stride == 1 ? sized((int)at_lo.y, (int)at_lo.z, (int)at_lo.w) : request(it.b);
            while (stride > 1 && it.b + 1 < a.B) {
                const uint32_t n = (uint32_t)r.tiles * a.kv_heads * pieces_of(r);
                if (base + n > place) break;
                base += n, r = request(++it.b);
            }
        }
        it.pieces = SHARED ? (uint32_t)(a.shared_parts * slots) : pieces_of(r);
        const uint32_t at = (place - base) / it.pieces;
        it.piece = place - base - at * it.pieces, it.first = base + at * it.pieces;
        it.h = (int)(at / (uint32_t)r.tiles);
        it.f0 = (r.tiles - 1 - (int)(at - (uint32_t)it.h * r.tiles)) * kRows;  // those of most keys first
        it.q0 = r.q0, it.nq = r.nq, it.ctx = r.ctx;
        if constexpr (SHARED) {
            it.pos_hi = sh_batch.keys - 1, it.pos_lo = min(sh_batch.lo, it.pos_hi);  // keys past pos_hi are not the item's
        } else {
            it.pos_lo = r.ctx - r.nq + it.f0 / gq;
            it.pos_hi = r.ctx - r.nq + min(r.nq - 1, (it.f0 + kRows - 1) / gq);
            b0 = kv4_first_seen(it.pos_lo, a.window) / 16, b1 = max(it.pos_hi + 16, 0) / 16;
        }
        const int total = max(0, b1 - b0 + 7) / 8;
        const int each = total / (int)it.pieces, rest = total - each * (int)it.pieces, p = (int)it.piece;
        it.bs = b0 + (p * each + min(p, rest)) * 8;
        it.n = each + (p < rest);
        return it;
    };
    // The first item is found by one warp: all of them at it take as long as the unpacking of a tile.
    __shared__ Item sh_first;
    __shared__ uint32_t sh_places;
    __shared__ Item sh_items_cut[2];  // of which the CTA has a part: there are fewer places than two per CTA where items are cut
    __shared__ int sh_cut, sh_last[2];
    __shared__ float sh_per_unit;
    if (warp == kIssuer) {
        bool falls = false;
        if constexpr (SHARED) {
            Batch all = {0x7FFFFFFF, -1, 0, 0};
            for (int b = lane; b < a.B; b += 32) {
                const Request r = request(b);
                falls |= offsets_fall(b);
                if (r.nq == 0 || r.ctx == 0) continue;
                all.lo = min(all.lo, r.ctx - r.nq), all.hi = max(all.hi, r.ctx - 1);
                if (r.ctx > all.keys) all.keys = r.ctx, all.b = b;
            }
            const int keys = __reduce_max_sync(0xFFFFFFFFu, all.keys);
            all.b = __reduce_min_sync(0xFFFFFFFFu, all.keys == keys ? all.b : 0x7FFFFFFF);
            all.lo = __reduce_min_sync(0xFFFFFFFFu, all.lo), all.hi = __reduce_max_sync(0xFFFFFFFFu, all.hi);
            all.keys = min(keys, a.shared_len);
            if (keys == 0) all.lo = 0, all.b = 0;
            if (lane == 0) sh_batch = all;
            __syncwarp();
        }
        Item it = item_at(blockIdx.x);
        if (SHARED && __any_sync(0xFFFFFFFFu, falls)) it.n = -1, W = 0;
        if (lanes && __any_sync(0xFFFFFFFFu, lane < a.B && offsets_fall(lane))) it.n = -1, W = 0;
        if (lane == 0) sh_first = it, sh_places = W, sh_per_unit = per_unit, sh_cut = 0;
    }
    __syncthreads();
    W = sh_places, per_unit = sh_per_unit;
    auto next_item = [&](uint32_t place) {
        Item it = sh_first;
        if (place >= W)
            it.n = -1;
        else if (place != blockIdx.x)
            it = item_at(place);
        return it;
    };
    float* parts = reinterpret_cast<float*>(static_cast<uint32_t*>(a.workspace) + kCounters);
    // An item's parts joined, in order, by the warps of softmax and unpacking.
    auto join = [&](const Item& it) {
        const float* part = parts + (size_t)it.first * L::PART;
        constexpr int LPR = D / 4, BATCH = 4;  // lanes of a row, four columns each; parts on their way at a time
        for (int r = warp * (32 / LPR) + lane / LPR; r < kRows; r += kIssuer * (32 / LPR)) {
            const int f = it.f0 + r, qi = f / gq, d = lane % LPR * 4;
            if (f >= it.nq * gq) break;
            float m = -CUDART_INF_F, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (uint32_t j = 0; j < it.pieces; j += BATCH) {
                float4 v[BATCH];
                float mj[BATCH], lj[BATCH];
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    mj[i] = -CUDART_INF_F, lj[i] = 0.f;
                    if (j + i < it.pieces) {
                        const float* p = part + (size_t)(j + i) * L::PART;
                        mj[i] = __ldcg(p + kRows * D + r), lj[i] = __ldcg(p + kRows * (D + 1) + r);
                        v[i] = __ldcg(reinterpret_cast<const float4*>(p + r * D + d));
                    }
                }
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    if (mj[i] == -CUDART_INF_F && lj[i] == 0.f) continue;  // no key, or none that is a number: then l is none
                    const float top = fmaxf(m, mj[i]), e = m == top ? 1.f : exp2_fast(m - top), x = mj[i] == top ? 1.f : exp2_fast(mj[i] - top);
                    m = top, l = fmaf(l, e, lj[i] * x);
                    o = make_float4(fmaf(o.x, e, v[i].x * x), fmaf(o.y, e, v[i].y * x), fmaf(o.z, e, v[i].z * x), fmaf(o.w, e, v[i].w * x));
                }
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const long long to = (long long)(it.q0 + qi) * a.out_stride + (long long)(it.h * gq + f - qi * gq) * D + d;
            store_out(a.out, to, o.x * inv, a.out_f32), store_out(a.out, to + 1, o.y * inv, a.out_f32);
            store_out(a.out, to + 2, o.z * inv, a.out_f32), store_out(a.out, to + 3, o.w * inv, a.out_f32);
            if (a.lse && d == 0)
                a.lse[(long long)(it.q0 + qi) * a.q_heads + it.h * gq + f - qi * gq] =
                    l == 0.f ? -CUDART_INF_F : (m + log2f(l) - kUp) * 0.69314718055994530942f;
        }
    };

    // At the end of a role: the CTA's parts are counted, and the items whose last part was among them joined. (At the end
    // of each piece the roles' registers would be spilled around it.)
    auto finish = [&](bool joins) {
        if (per_unit == 0.f) return;
        bar_joiners();
        if (tid == 0) {
            __threadfence();
            for (int i = 0; i < sh_cut; ++i)
                sh_last[i] = atomicInc(static_cast<uint32_t*>(a.workspace) + sh_items_cut[i].first, sh_items_cut[i].pieces - 1) == sh_items_cut[i].pieces - 1;
            __threadfence();
        }
        bar_joiners();
        if (!joins) return;
#pragma unroll 1
        for (int i = 0; i < sh_cut; ++i)
            if (sh_last[i]) join(sh_items_cut[i]);
    };

    // SHARED, items of several pieces: behind the first cluster_sync the pieces' sums lie in the CTAs' shared memory, behind the
    // second no CTA reads another's. Every thread of the cluster comes to both.
    constexpr int PITCH = D + 4;  // floats of a row there, over K's stages
    static_assert(kRows * PITCH * 4 <= kStages * L::K_BYTES, "");
    float* sums = reinterpret_cast<float*>(smem);

    uint32_t tile = 0, count = 0;  // key tiles, and items with any, before this one: the phases of every barrier
    if (warp < kSoftmax) {
        // ------------------------------------------------------------ softmax: two threads per row ----
        registers<kRegsSoftmax>(true);
        const int half = warp >> 2, r = tid & (kRows - 1);  // of the keys, and of the outputs' columns; the row
        const uint32_t my = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float sl2 = fabsf(a.scale) * 1.44269504088896340736f;
        for (uint32_t place = blockIdx.x;; place += gridDim.x) {
            const Item it = next_item(place);
            if (it.n < 0) break;
            const int f = it.f0 + r, qi = min(f / gq, it.nq - 1);
            int pos = it.ctx - it.nq + qi, last = pos;  // the query's, and the last key's that it sees here
            if constexpr (SHARED) {
                int b = qi / max(1, a.T / a.B), first = b * (a.T / a.B), n = a.T / a.B;
                if (a.q_starts) {  // the last request that begins with the query or before it
                    int lo = 0, hi = a.B - 1;
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) / 2;
                        if (a.q_starts[mid] <= qi)
                            lo = mid;
                        else
                            hi = mid - 1;
                    }
                    b = lo, first = a.q_starts[lo], n = a.q_starts[lo + 1] - first;
                }
                const int ctx = min(max(a.ctx_lens[b], 0), cap);
                pos = ctx == 0 || qi < first || qi - first >= n ? -1 : ctx - n + qi - first;
                last = min(pos, it.pos_hi);
            }
            const bool there = f < it.nq * gq;
            const long long row = it.q0 + qi;
            const int head = it.h * gq + f - (f / gq) * gq;
            float scale_row = 0.f;
            if (it.n > 0) {  // ---- half of the row of Q, its dimensions in the codes' order, and the sums of its groups, in two parts ----
                constexpr int LH = D / 16, GH = NG > 1 ? NG / 2 : 1;  // 16-byte words, groups
                const uint16_t* src = a.q + row * a.q_stride + (long long)head * D + D / 2 * half;
                uint4 v[LH];
                uint32_t big = 0;
#pragma unroll
                for (int l = 0; l < LH; ++l) v[l] = there ? reinterpret_cast<const uint4*>(src)[l] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int l = 0; l < LH; ++l)
                    big = __vmaxu2(__vmaxu2(big, v[l].x & 0x7FFF7FFFu), __vmaxu2(v[l].y & 0x7FFF7FFFu, __vmaxu2(v[l].z & 0x7FFF7FFFu, v[l].w & 0x7FFF7FFFu)));
                big = max(big >> 16, big & 0xFFFFu);
                sh_max[half][r] = __uint_as_float(big);
                bar_any(2 + (warp & 3), false);
                big = max(big, __float_as_uint(sh_max[half ^ 1][r]));
                const uint32_t ex = max(big >> 7, 20u);  // the largest entry's biased exponent
                const float up = copysignf(__uint_as_float((261u - ex) << 23), a.scale);  // to [2^7, 2^8)
                scale_row = __uint_as_float((ex - 7u) << 23) * sl2;
                float sum[GH];
#pragma unroll
                for (int gr = 0; gr < GH; ++gr) sum[gr] = 0.f;
#pragma unroll
                for (int l0 = 0; l0 < LH; l0 += 4) {
                    uint32_t out[16];
#pragma unroll
                    for (int l = 0; l < 4; ++l) {
                        const uint32_t x[4] = {v[l0 + l].x, v[l0 + l].y, v[l0 + l].z, v[l0 + l].w};
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float q0 = bf16lo_to_f32(x[i]) * up, q1 = bf16hi_to_f32(x[i]) * up;
                            sum[(l0 + l) * 8 / G] += q0 + q1;
                            w[i] = pack(q0, q1);
                        }
                        out[4 * l] = __byte_perm(w[0], w[2], 0x5410), out[4 * l + 1] = __byte_perm(w[0], w[2], 0x7632);
                        out[4 * l + 2] = __byte_perm(w[1], w[3], 0x5410), out[4 * l + 3] = __byte_perm(w[1], w[3], 0x7632);
                    }
                    st16(my + L::Q_COL + D / 4 * half + 4 * l0, out);
                }
                // the sums of the other half's groups, or, of one group, its other part
                if (half)
#pragma unroll
                    for (int gr = 0; gr < GH; ++gr) sh_sums[gr][r] = sum[gr];
                bar_any(2 + (warp & 3), false);
                if (half == 0) {
                    uint32_t ext[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) ext[i] = 0;
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) {  // (hi, hi, lo, 0) beside (hi, lo, hi, 0) of the offset
                        const float x = NG == 1 ? sum[0] + sh_sums[0][r] : gr < GH ? sum[gr % GH] : sh_sums[gr % GH][r];
                        const __half hi = __float2half_rn(x), lo = __float2half_rn(x - __half2float(hi));
                        ext[2 * gr] = (uint32_t)__half_as_ushort(hi) * 0x10001u, ext[2 * gr + 1] = __half_as_ushort(lo);
                    }
                    st8(my + L::Q_COL + D / 2, ext);
                }
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(qfull);
            }
            float M = -CUDART_INF_F;
            // What a score's power of two is off its weight's. Rounded up, so that the maximum's weight is at least 2^kUp however
            // large the scores are; beyond 2^24, where the rounding passes a power of two, a weight may pass fp16, and its
            // largest number takes its place: the keys that have it are as near to each other as scores of 32 bits are.
            auto offset_to = [&](float m) { return m == -CUDART_INF_F ? 0.f : __fmaf_ru(-m, scale_row, (float)kUp); };
            const uint32_t tile0 = tile;
            for (int k = 0; k < it.n; ++k, ++tile) {
                const uint32_t sb = tile & 1, s_at = my + L::S_COL + sb * 128 + 64 * half;
                const int t0 = (it.bs + 8 * k) * 16;
                const bool edge = t0 + kKeys - 1 > it.pos_lo || (a.window && t0 <= (SHARED ? sh_batch.hi : it.pos_hi) - a.window);
                // the columns that the row sees: lo .. lo + span
                int c_lo = a.window ? max(0, pos - a.window + 1 - t0) : 0, span = min(last - t0, kKeys - 1) - c_lo;
                if (span < 0) c_lo = 1 << 20, span = 0;
                c_lo -= 64 * half;
                bar_wait(&sfull[sb], (tile >> 1) & 1, ok);
                fence_after();
                // One pass for the weights against the maximum so far and for the tile's own; another where that has
                // grown too far, which is rare behind the first tile.
                uint32_t w[32];
                float m, off = offset_to(M);
                auto pass = [&](auto edge_tile, auto maximum_alone) {
                    constexpr bool EDGE = decltype(edge_tile)::value, ALONE = decltype(maximum_alone)::value;
                    float m2[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t v[32];
                        ld32(v, s_at + 32 * c);
                        wait_ld(v);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int col = 32 * c + 2 * i;
                            const float x = __uint_as_float(v[2 * i]), y = __uint_as_float(v[2 * i + 1]);
                            const bool see_x = !EDGE || (uint32_t)(col - c_lo) <= (uint32_t)span, see_y = !EDGE || (uint32_t)(col + 1 - c_lo) <= (uint32_t)span;
                            m2[i & 1] = max3(m2[i & 1], see_x ? x : -CUDART_INF_F, see_y ? y : -CUDART_INF_F);
                            if (ALONE) continue;
                            const float2 e = fma2(make_float2(x, y), make_float2(scale_row, scale_row), make_float2(off, off));
                            w[16 * c + i] = pack_finite(see_x ? exp2_fast(e.x) : 0.f, see_y ? exp2_fast(e.y) : 0.f);
                        }
                    }
                    m = fmaxf(m2[0], m2[1]);
                };
                if (k == 0)
                    pass(std::true_type(), std::true_type());
                else if (edge)
                    pass(std::true_type(), std::false_type());
                else
                    pass(std::false_type(), std::false_type());
                bool raise = m > M && (M == -CUDART_INF_F || (m - M) * scale_row > kGrow);
                if (bar_any(2 + (warp & 3), raise || k == 0)) {
                    sh_max[half][r] = m;
                    bar_any(2 + (warp & 3), false);
                    m = fmaxf(m, sh_max[half ^ 1][r]);
                    raise = m > M && (M == -CUDART_INF_F || (m - M) * scale_row > kGrow);
                    if (k > 0) {
                        const float e = raise && M != -CUDART_INF_F ? exp2_fast(offset_to(m) - off) : 1.f;
                        bar_wait(&odone[(tile - 1) & 1], ((tile - 1) >> 1) & 1, ok);  // the products into the outputs so far
                        fence_after();
#pragma unroll 1
                        for (int c = 16 * half; c < L::N; c += 32) {
                            uint32_t v[16];
                            ld16(v, my + L::O_COL + c);
                            wait_ld16(v);
#pragma unroll
                            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * e);
                            st16(my + L::O_COL + c, v);
                        }
                    }
                    if (raise) M = m;
                    off = offset_to(M);
                    pass(std::true_type(), std::false_type());
                    bar_any(2 + (warp & 3), false);  // sh_max is read
                }
                st16(s_at, w), st16(s_at + 16, w + 16);  // over columns that are read
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&pfull[sb]);
            }
            // ---- outputs, or the item's part ----
            float l = 0.f, off[NG];
            uint32_t poison = 0;  // groups in which a key that the row sees is no number
            if (it.n > 0) {
                // The last product is issued behind V's arrival in every tile, of the even set's warps and of the odd set's:
                // behind this wait sh_bad is all that they found in the item.
                bar_wait(&odone[(tile - 1) & 1], ((tile - 1) >> 1) & 1, ok);
                fence_after();
                if (*reinterpret_cast<volatile uint32_t*>(&sh_bad) > tile0) {
                    const int end = min(last + 1, (it.bs + 8 * it.n) * 16);
                    for (int t = max(it.bs * 16, a.window ? pos - a.window + 1 : 0); t < end; ++t) {
                        const int p = t / a.page_size, page = a.table[(long long)it.b * a.table_stride + p];
                        const long long blk = ((long long)(page < 0 || page >= a.num_pages ? 0 : page) * a.kv_heads + it.h) * bpp + (t - p * a.page_size) / 16;
                        const uint32_t* meta = reinterpret_cast<const uint32_t*>(a.pages + blk * kv4_block_bytes(D, G) + kv4_meta(D, G, t & 15, 0, 1));
#pragma unroll
                        for (int gr = 0; gr < NG; ++gr) poison |= (uint32_t)no_number(meta[gr], offset_of(meta[gr])) << gr;
                    }
                    __syncwarp();
                }
                uint32_t v[16];
                ld16(v, my + L::O_COL + D);
                wait_ld16(v);
                l = __uint_as_float(v[2 * NG]);
#pragma unroll
                for (int gr = 0; gr < NG; ++gr)
                    off[gr] = poison >> gr & 1 ? CUDART_NAN_F : __uint_as_float(v[2 * gr]) + __uint_as_float(v[2 * gr + 1]);
            }
            const bool none = SHARED && pos < 0;  // a query of no request or before its first token: its tiles were not looked at key by key
            if (none) M = -CUDART_INF_F, l = 0.f;
            const float m2 = M == -CUDART_INF_F ? M : kUp - offset_to(M);  // what the weights refer to
            const float inv = (SHARED ? slots : (int)it.pieces) > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;
            const long long shared_row = SHARED ? ((long long)(it.piece / (uint32_t)slots) * a.T + row) * a.q_heads + head : 0;  // in its part
            float* part = parts + (size_t)place * L::PART;
            const long long to = row * a.out_stride + (long long)head * D;
#pragma unroll 1
            for (int c = D / 2 * half; c < D / 2 * (half + 1); c += 32) {
                uint32_t v[32];
                if (it.n > 0) {
                    ld32(v, my + L::O_COL + c);
                    wait_ld(v);
                    float o = 0.f;  // of the 32 columns' group
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) o = c / G == gr ? off[gr] : o;
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = none ? 0u : __float_as_uint((__uint_as_float(v[i]) + o) * inv);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0;
                }
                if (SHARED && slots > 1) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) reinterpret_cast<uint4*>(sums + r * PITCH + c)[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                } else if (!SHARED && it.pieces > 1) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) reinterpret_cast<uint4*>(part + r * D + c)[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                } else if (SHARED) {
                    if (there)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            reinterpret_cast<uint4*>(a.shared_out + shared_row * D + c)[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                } else if (there) {
                    if (a.out_f32) {
                        float* p = static_cast<float*>(a.out) + to + c;
#pragma unroll
                        for (int i = 0; i < 32; ++i) p[i] = __uint_as_float(v[i]);
                    } else {
                        uint16_t* p = static_cast<uint16_t*>(a.out) + to + c;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(v[8 * i + 2 * j]), __uint_as_float(v[8 * i + 2 * j + 1]));
                                w[j] = *reinterpret_cast<const uint32_t*>(&x);
                            }
                            reinterpret_cast<uint4*>(p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
            }
            if (half) {
            } else if (SHARED && slots > 1)
                sh_sums[0][r] = m2, sh_sums[1][r] = l;
            else if (!SHARED && it.pieces > 1)
                part[D * kRows + r] = m2, part[(D + 1) * kRows + r] = l;
            else if (SHARED) {
                if (there) a.shared_lse[shared_row] = l == 0.f ? -CUDART_INF_F : m2 + log2f(l) - kUp;
            } else if (there && a.lse)
                a.lse[row * a.q_heads + head] = l == 0.f ? -CUDART_INF_F : (m2 + log2f(l) - kUp) * 0.69314718055994530942f;
            fence_before();
            if (!SHARED && it.pieces > 1 && tid == 0) sh_items_cut[sh_cut++] = it;
        }
        if (SHARED && slots > 1) {
            // A cluster's CTAs have one item, of which each joins some rows, the pieces in order.
            cluster_sync();
            const int rank = blockIdx.x % slots, r1 = kRows * (rank + 1) / slots;
            constexpr int LPR = D / 4;  // lanes of a row, four columns each
            for (int r = kRows * rank / slots + warp * (32 / LPR) + lane / LPR; r < r1 && W > 0; r += kSoftmax * (32 / LPR)) {
                const int f = sh_first.f0 + r, d = lane % LPR * 4;
                if (f >= a.T * gq) break;
                float m = -CUDART_INF_F, l = 0.f;
                float4 v[kPieces], o = make_float4(0.f, 0.f, 0.f, 0.f);
                float mj[kPieces], lj[kPieces];
#pragma unroll
                for (int j = 0; j < kPieces; ++j) {
                    mj[j] = -CUDART_INF_F, lj[j] = 0.f, v[j] = o;
                    if (j < slots) {
                        uint32_t at;
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_at(sums + r * PITCH + d)), "r"(j));
                        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[j].x), "=f"(v[j].y), "=f"(v[j].z), "=f"(v[j].w) : "r"(at) : "memory");
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_at(&sh_sums[0][r])), "r"(j));
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(mj[j]) : "r"(at) : "memory");
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(lj[j]) : "r"(at + kRows * 4) : "memory");
                    }
                }
#pragma unroll
                for (int j = 0; j < kPieces; ++j) {
                    if (mj[j] == -CUDART_INF_F && lj[j] == 0.f) continue;  // no key, or none that is a number: then l is none
                    const float top = fmaxf(m, mj[j]), e = m == top ? 1.f : exp2_fast(m - top), x = mj[j] == top ? 1.f : exp2_fast(mj[j] - top);
                    m = top, l = fmaf(l, e, lj[j] * x);
                    o = make_float4(fmaf(o.x, e, v[j].x * x), fmaf(o.y, e, v[j].y * x), fmaf(o.z, e, v[j].z * x), fmaf(o.w, e, v[j].w * x));
                }
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const int qi = f / gq;
                const long long at = ((long long)(sh_first.piece / (uint32_t)slots) * a.T + qi) * a.q_heads + sh_first.h * gq + f - qi * gq;
                *reinterpret_cast<float4*>(a.shared_out + at * D + d) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
                if (d == 0) a.shared_lse[at] = l == 0.f ? -CUDART_INF_F : m + log2f(l) - kUp;
            }
            cluster_sync();
        }
        finish(true);
    } else if (warp < kIssuer) {
        // ------------------ unpack: a warp takes K, or V, of a block of 16 keys of each tile ----
        registers<kRegsUnpack>(false);
        const int u = (warp - kSoftmax) % kUnpack, set = (warp - kSoftmax) / kUnpack, g = lane >> 2, c = lane & 3;
        constexpr int BB = kv4_block_bytes(D, G), J = D / 32, NV = D / 64;
        constexpr int PER = (16 * NG + 31) / 32;  // (token, group) pairs of a lane
        uint8_t* blk = smem + L::OFF_RING + (warp - kSoftmax) * BB;
        uint32_t* kmeta = reinterpret_cast<uint32_t*>(blk + kv4_meta(D, G, 0, 0, 0));  // [token][group]
        uint32_t* vmeta = reinterpret_cast<uint32_t*>(blk + kv4_meta(D, G, 0, 0, 1));
        const uint32_t ring_at = smem_at(blk) + lane * 16;
        const uint8_t* pages = a.pages + lane * 16;
        // the set's stage, and this warp's place in it
        uint8_t* ks = smem + set * L::K_BYTES + 16 * u * 128;
        uint8_t* vs = smem + L::OFF_V + set * L::V_BYTES + (u >> 2) * L::V_BOX;
        const int k_at = g * 128 + (((c ^ g) << 4) ^ ((g & 1) << 6));
        const int v_at = g * 128 + (((2 * (u & 3)) ^ g) << 4) + 4 * c;
        uint32_t turn = 0;  // tiles of the set so far
        const Unpack unpack;
        for (uint32_t place = blockIdx.x;; place += gridDim.x) {
            const Item it = next_item(place);
            if (it.n < 0) break;
            const int b1 = max(it.pos_hi + 16, 0) / 16;
            const int32_t* table = a.table + (long long)it.b * a.table_stride;
            const int k0 = (tile ^ set) & 1;  // the set's first tile of the item
            auto offset = [&](int k) -> long long {  // of the warp's block of tile k, -1 past the end
                const int blk = it.bs + 8 * k + u;
                if (k >= it.n || blk >= b1) return -1;
                const int p = blk / bpp;
                int page = table[p];
                if (page < 0 || page >= a.num_pages) bad = true, page = 0;
                return (((long long)page * a.kv_heads + it.h) * bpp + (blk - p * bpp)) * BB;
            };
            long long offs = offset(k0 + 2 * lane);  // of the lane's tile among 32 of the set
            auto copy = [&](long long o, int v) {    // K or V of a block, a group of copies
                if (o >= 0) {
                    const uint32_t at = v * 8 * D, meta = 16 * D + v * 64 * NG;
#pragma unroll
                    for (int i = 0; i < D / 64; ++i)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring_at + at + i * 512), "l"(pages + o + at + i * 512) : "memory");
                    if (lane < 4 * NG) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring_at + meta), "l"(pages + o + meta) : "memory");
                }
                cp_async_commit();
            };
            {
                const long long o = __shfl_sync(0xFFFFFFFFu, offs, 0);
                copy(o, 0);
                copy(o, 1);
            }
            for (int k = k0; k < it.n; k += 2, ++turn) {
                const int next = (k - k0) / 2 + 1;
                if (next % 32 == 0) offs = offset(k + 2 + 2 * lane);
                const long long o_next = __shfl_sync(0xFFFFFFFFu, offs, next % 32);
                uint32_t off[PER];  // the offsets of a (token, group) a lane
                // ---- K: rows of keys ----
                cp_async_wait<1>();
                __syncwarp();
#pragma unroll
                for (int i = 0; i < PER; ++i) off[i] = 16 * NG % 32 == 0 || lane < 16 * NG ? offset_of(kmeta[lane + 32 * i]) : 0;
                if (turn) bar_wait(&kempty[set], (turn - 1) & 1, ok);
#pragma unroll
                for (int i = 0; i < PER; ++i) {  // (hi, lo, hi, 0) of a group
                    const int j = lane + 32 * i, t = j / NG, gr = j % NG;
                    if (16 * NG % 32 == 0 || lane < 16 * NG)
                        *reinterpret_cast<uint2*>(ks + (D / 64) * L::K_BOX + t * 128 + (((gr >> 1) ^ (t & 7)) << 4) + (gr & 1) * 8) = make_uint2(off[i], off[i] & 0xFFFFu);
                }
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {  // rolled: the warps' code streams through small instruction caches
                    uint32_t kw[J], sk[NG], dk[NG];
                    if constexpr (D == 64) {
                        const uint2 v = *reinterpret_cast<const uint2*>(blk + (g + 8 * t) * 32 + c * 8);
                        kw[0] = v.x, kw[1] = v.y;
                    } else {
                        const uint4 v = *reinterpret_cast<const uint4*>(blk + (g + 8 * t) * 64 + c * 16);
                        kw[0] = v.x, kw[1] = v.y, kw[2] = v.z, kw[3] = v.w;
                    }
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) sk[gr] = __byte_perm(kmeta[(g + 8 * t) * NG + gr], 0, 0x1010), dk[gr] = half_step(sk[gr]);
                    uint8_t *to0 = ks + k_at + t * 1024, *to1 = ks + (k_at ^ 64) + t * 1024;
#pragma unroll
                    for (int j0 = 0; j0 < J; j0 += 2)
                        // lanes of odd rows write the other of two words first: 8 lanes then write 8 chunks of 16 bytes apart
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const bool odd = (g & 1) ^ e;
                            const uint32_t w = odd ? kw[j0 + 1] : kw[j0];  // dimensions 32 (j0 + odd) + 8 c ...
                            uint32_t s, d;
                            if (G == 64)
                                s = sk[j0 / 2 % NG], d = dk[j0 / 2 % NG];
                            else
                                s = odd ? sk[(j0 + 1) % NG] : sk[j0 % NG], d = odd ? dk[(j0 + 1) % NG] : dk[j0 % NG];
                            uint32_t o[4];
                            unpack(w, s, d, o);
                            *reinterpret_cast<uint4*>((e ? to1 : to0) + (j0 / 2) * L::K_BOX) = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) bar_arrive(&kfull[set]);
                copy(o_next, 0);  // over what was just read

                // ---- V: rows of dimensions, pairs of tokens. What is no number, or unseen by every row, becomes zeros ----
                cp_async_wait<1>();
                __syncwarp();
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int j = lane + 32 * i;
                    if (16 * NG % 32 && lane >= 16 * NG) break;
                    const uint32_t y = vmeta[j];
                    const bool unseen = (it.bs + 8 * k + u) * 16 + j / NG > it.pos_hi;
                    off[i] = offset_of(y);
                    if (unseen || no_number(y, off[i])) {
                        if (!unseen) atomicMax(&sh_bad, tile + k + 1);
                        vmeta[j] = off[i] = 0;
                    }
                }
                __syncwarp();
                if (turn) bar_wait(&vempty[set], (turn - 1) & 1, ok);
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int j = lane + 32 * i, t = j / NG, row = 2 * (j % NG);
                    if (16 * NG % 32 && lane >= 16 * NG) break;
                    uint8_t* to = vs + (D + row) * 128 + (((2 * (u & 3) + (t >> 3)) ^ row) << 4) + (t & 7) * 2;
                    *reinterpret_cast<uint16_t*>(to) = (uint16_t)off[i];
                    *reinterpret_cast<uint16_t*>(vs + (to - vs + 128 ^ 16)) = (uint16_t)(off[i] >> 16);  // the next row
                }
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t vw[2 * NV], s2[NG], d2[NG];  // words (b, w)
                    if constexpr (NV == 1) {
                        const uint2 v = *reinterpret_cast<const uint2*>(blk + 8 * D + lane * 16 + h * 8);
                        vw[0] = v.x, vw[1] = v.y;
                    } else {
                        const uint4 v = *reinterpret_cast<const uint4*>(blk + 8 * D + h * 512 + lane * 16);
                        vw[0] = v.x, vw[1] = v.y, vw[2] = v.z, vw[3] = v.w;
                    }
                    const uint32_t* vm = vmeta + (8 * h + 2 * c) * NG;  // two tokens
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) s2[gr] = __byte_perm(vm[gr], vm[NG + gr], 0x5410), d2[gr] = half_step(s2[gr]);
                    uint8_t* to = vs + (v_at ^ (h << 4));
#pragma unroll
                    for (int w = 0; w < NV; ++w)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {  // slots 0 .. 3, 4 .. 7
                            const int gr = (64 * w + 32 * half) / G;
                            uint32_t o[4];
                            unpack(__byte_perm(vw[w], vw[NV + w], half ? 0x7632 : 0x5410), s2[gr], d2[gr], o);
#pragma unroll
                            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t*>(to + (64 * w + 8 * (4 * half + i)) * 128) = o[i];
                        }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) bar_arrive(&vfull[set]);
                copy(o_next, 1);
            }
            tile += it.n;
        }
        if (SHARED && slots > 1) cluster_sync(), cluster_sync();
        finish(true);
    } else if (warp >= kIssuer) {
        registers<kRegsIssuer>(false);
        if (warp == kIssuer) {
        // ------------------------------------------------------------ products ----
        const bool leader = elect();
        constexpr uint32_t ID_S = idesc(kRows, kKeys), ID_O = idesc(kRows, L::N);
        auto outputs = [&](uint32_t t, bool first) {  // the weights of tile t times V
            const uint32_t st = t % kStages, sb = t & 1;
            bar_wait(&pfull[sb], (t >> 1) & 1, ok);
            bar_wait(&vfull[st], (t / kStages) & 1, ok);
            fence_after();
            if (leader) {
                if (ok) {
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)
                        mma(tmem + L::O_COL, tmem + L::S_COL + sb * 128 + (k / 4) * 64 + (k % 4) * 8,
                            desc(smem_at(smem + L::OFF_V + st * L::V_BYTES + (k / 4) * L::V_BOX)) + 2 * (k % 4), ID_O, !first || k > 0);
                }
                commit(&vempty[st]);
                commit(&odone[sb]);
            }
            __syncwarp();
        };
        for (uint32_t place = blockIdx.x;; place += gridDim.x) {
            const Item it = next_item(place);
            if (it.n < 0) break;
            if (it.n > 0) bar_wait(qfull, count++ & 1, ok);
            for (int k = 0; k < it.n; ++k, ++tile) {
                const uint32_t st = tile % kStages, sb = tile & 1;
                bar_wait(&kfull[st], (tile / kStages) & 1, ok);
                fence_after();
                if (leader) {
                    if (ok) {
#pragma unroll
                        for (int i = 0; i <= KS; ++i)
                            mma(tmem + L::S_COL + sb * 128, tmem + L::Q_COL + i * 8,
                                desc(smem_at(smem + st * L::K_BYTES + (i / 4) * L::K_BOX)) + 2 * (i % 4), ID_S, i > 0);
                    }
                    commit(&kempty[st]);
                    commit(&sfull[sb]);
                }
                __syncwarp();
                if (k > 0) outputs(tile - 1, k == 1);
            }
            if (it.n > 0) outputs(tile - 1, it.n == 1);
        }
        finish(false);
        // every product issued has completed before TMEM is released
        if (leader) commit(done);
        __syncwarp();
        bool last = true;
        bar_wait(done, 0, last);
        }
        if (SHARED && slots > 1) cluster_sync(), cluster_sync();
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kIssuer) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    if (bad) atomicExch(&g_kv4_tc_range, 1);
}

// pieces: CTAs of a cluster that share an item (SHARED), else 1.
template <int D, int G, bool SHARED>
cudaError_t launch(const Kv4AttnArgs& a, int slots, int grid, int pieces, cudaStream_t s) {
    constexpr int smem = Layout<D>::SMEM;
    static_assert(smem <= 227 * 1024, "");
    const cudaError_t err = kv4_allow_smem((const void*)kv4_attention_tc_kernel<D, G, SHARED>, smem);
    if (err != cudaSuccess) return err;
    static std::atomic<int> regs{0};
    if (!regs.load(std::memory_order_relaxed)) {
        cudaFuncAttributes attr;
        const cudaError_t e = cudaFuncGetAttributes(&attr, kv4_attention_tc_kernel<D, G, SHARED>);
        if (e != cudaSuccess) return e;
        regs.store(attr.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) < kRegsLaunch) return cudaErrorLaunchOutOfResources;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)kThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = (unsigned)pieces;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = pieces > 1 ? 2 : 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, kv4_attention_tc_kernel<D, G, SHARED>, a, slots);
}

template <bool SHARED>
cudaError_t launch_for(const Kv4AttnArgs& a, int slots, int grid, int pieces, cudaStream_t s) {
    if (a.head_dim == 64) return a.group == 32 ? launch<64, 32, SHARED>(a, slots, grid, pieces, s) : launch<64, 64, SHARED>(a, slots, grid, pieces, s);
    return a.group == 32 ? launch<128, 32, SHARED>(a, slots, grid, pieces, s) : launch<128, 64, SHARED>(a, slots, grid, pieces, s);
}

}  // namespace

size_t kv4_attention_tc_workspace(int head_dim) {
    if (head_dim == 256) return 0;
    return kCounters * sizeof(uint32_t) + (size_t)(2 * device_sm_count()) * (kRows * (head_dim + 2)) * sizeof(float);
}

cudaError_t launch_kv4_attention_tc(const Kv4AttnArgs& a, cudaStream_t s) {
    const size_t part = (size_t)kRows * (a.head_dim + 2) * sizeof(float), counters = kCounters * sizeof(uint32_t);
    const size_t room = a.ws_bytes > counters ? (a.ws_bytes - counters) / part : 0;
    const int slots = (int)(room < (size_t)kCounters ? room : (size_t)kCounters);
    return launch_for<false>(a, slots, device_sm_count(), 1, s);
}

namespace {

// Clusters of n CTAs of the kernel that the device holds at once (a GPC's SMs hold them or not), asked for once per device.
template <int D, int G>
cudaError_t held(int n, int* out) {
    static std::atomic<int> known[16][kPieces];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    *out = dev < 16 ? known[dev][n - 1].load(std::memory_order_relaxed) : 0;
    if (*out) return cudaSuccess;
    e = kv4_allow_smem((const void*)kv4_attention_tc_kernel<D, G, true>, Layout<D>::SMEM);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)n, 1, 1);
    cfg.blockDim = dim3((unsigned)kThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)Layout<D>::SMEM;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)n;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(out, kv4_attention_tc_kernel<D, G, true>, &cfg);
    if (e != cudaSuccess) return e;
    if (*out < 1) *out = 1;
    if (dev < 16) known[dev][n - 1].store(*out, std::memory_order_relaxed);
    return cudaSuccess;
}

cudaError_t held_for(const Kv4AttnArgs& a, int n, int* out) {
    if (a.head_dim == 64) return a.group == 32 ? held<64, 32>(n, out) : held<64, 64>(n, out);
    return a.group == 32 ? held<128, 32>(n, out) : held<128, 64>(n, out);
}

int64_t prefix_items(const Kv4AttnArgs& a) { return ((int64_t)a.T * (a.q_heads / a.kv_heads) + kRows - 1) / kRows * a.kv_heads; }

}  // namespace

// An item is 128 rows or fewer of a KV head, so that there are q_heads T / 128 or more; more than one part only where the
// CTAs have one of them each.
size_t kv4_attention_prefix_rows(int64_t T, int64_t q_heads) {
    const int64_t rows = T * q_heads, most = (int64_t)device_sm_count() * kRows;
    return (size_t)(rows > most ? rows : most);
}

cudaError_t plan_kv4_attention_prefix(const Kv4AttnArgs& a, int shared_len, Kv4SharedPlan* plan) {
    const int64_t sms = device_sm_count(), items = prefix_items(a), units = (shared_len + kKeys - 1) / kKeys;
    // Pieces of two key tiles or more, as many as find an SM each.
    int64_t best = 1;
    *plan = {1, 1};
    for (int c = 1; c <= kPieces; ++c) {
        int n = 0;
        const cudaError_t e = held_for(a, c, &n);
        if (e != cudaSuccess) return e;
        for (int g = 1; g <= kKv4SharedParts; ++g) {
            const int64_t pieces = c * g;
            if (pieces > 1 && (items * g > n || items * pieces > sms || 2 * pieces > units)) continue;
            if (pieces > best || (pieces == best && g < plan->parts)) best = pieces, *plan = {g, c};
        }
    }
    // Worth it where reading the shared tokens for every request, once for each 8 rows, at 4.9 TB/s (the rate of 64 requests)
    // would take longer than this kernel, 12 us and 1.25 a tile of keys, and what its SMs leave undone of the other's start
    // where that one has many items. Measured, plain and shared, us: Qwen3-4B's heads, 8192 tokens, 2, 4, 8 and 64 requests:
    // 13.8 19.0, 18.7 26.7, 26.0 31.4, 114.9 42.5; Qwen2.5-7B's, 12 of 2 to 5 queries, 30000 tokens: 132 53; 64, 512: 14.5 31.3.
    // A window is not looked at: 64 requests behind 8192 tokens, windows of 64, 256, 1024, 2048, 4096 and none: 9.2 21.0, 13.5 28.7,
    // 23.0 30.5, 35.8 32.0, 61.1 34.1, 112.8 38.8.
    const int64_t with = a.B < a.T ? a.B : a.T, gq = a.q_heads / a.kv_heads, rows = ((int64_t)a.T * gq + a.B - 1) / a.B;
    const double read = (double)with * ((rows + 7) / 8) * a.kv_heads * shared_len * (a.head_dim + 8 * (a.head_dim / a.group)) / 4900.0;
    const int64_t waves = (items * best + sms - 1) / sms, tiles = (units + best - 1) / best * waves;
    if (read < 12000.0 + 1250.0 * tiles + (2 * with * a.kv_heads > sms ? 5000.0 : 0.0)) plan->parts = 0;
    return cudaSuccess;
}

cudaError_t launch_kv4_attention_prefix(const Kv4AttnArgs& a, const Kv4SharedPlan& plan, cudaStream_t s) {
    const int64_t sms = device_sm_count(), all = prefix_items(a) * plan.parts * plan.ctas;
    return launch_for<true>(a, plan.ctas, (int)(plan.parts * plan.ctas > 1 || all < sms ? all : sms), plan.ctas, s);
}

int kv4_attn_tc_take(bool fault) {
    int v = 0, z = 0;
    if (fault) {
        if (cudaMemcpyFromSymbol(&v, g_kv4_tc_fault, sizeof(int)) != cudaSuccess) return -1;
        if (v) cudaMemcpyToSymbol(g_kv4_tc_fault, &z, sizeof(int));
    } else {
        if (cudaMemcpyFromSymbol(&v, g_kv4_tc_range, sizeof(int)) != cudaSuccess) return -1;
        if (v) cudaMemcpyToSymbol(g_kv4_tc_range, &z, sizeof(int));
    }
    return v;
}

}  // namespace mbw
