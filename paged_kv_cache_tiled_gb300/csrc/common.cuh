// Device-side helpers shared by the libfattn kernels: error reporting,
// bounded waits, and thin inline-PTX wrappers for mbarrier, TMA (bulk tensor
// copies), tcgen05 (tensor-core MMA with TMEM accumulators) and warp-level MMA.
// Everything here targets sm_103a.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/fattn.h"

namespace fa {

// ------------------------------------------- paged tensor-core layout ---
// Chunks of the paged path that go to the tensor-core kernel are cut into
// work entries of consecutive query tokens; each entry is one unit per kv
// head (or per pair of query heads), two 128-row Q slots sharing every K/V
// tile.  When the GQA group size g = Hq/Hkv divides 128 (g = 2, 4, 8, 16) a
// slot packs 128/g tokens x the g heads of the group (row = token * g + head),
// so a short chunk does not pad a 128-row tile per head; otherwise a slot is
// 128 tokens of one head.
__host__ __device__ inline bool paged_tc_pack(int g) { return g == 2 || g == 4 || g == 8 || g == 16; }
// tokens of a query slot
__host__ __device__ inline int paged_tc_slot_tokens(int g) { return paged_tc_pack(g) ? 128 / g : 128; }
// query tokens of a work entry: two packed slots; a head pair's two slots over
// the same 128 tokens (g even); or two consecutive 128-token slots of one head
__host__ __device__ inline int paged_tc_entry_tokens(int g) {
    return paged_tc_pack(g) ? 2 * (128 / g) : (g % 2 == 0 ? 128 : 256);
}

// Do the rows [q0, q0 + q_len) of a sequence lie in a call's total_q?  (Neither q0 nor q_len negative.)
__host__ __device__ inline bool rows_fit(int q0, int q_len, int total_q) { return q_len <= total_q - q0; }

// ---------------------------------------------------------------- errors ---
// Bits of the per-device error word.
enum : unsigned { ERR_BOUNDS_BIT = 1u, ERR_TIMEOUT_BIT = 2u };

struct DevCtx {
    unsigned* err;              // device error word
    unsigned long long wait_ns; // bound on each pipeline wait
    int force_timeout;          // test hook: start every role with a wait that cannot complete (n > 1: the listed
                                // blocks' warps wait so before the n-th page instead)
};

__device__ __forceinline__ void raise_error(const DevCtx& c, unsigned bit) { atomicOr(c.err, bit); }

__device__ __forceinline__ uint64_t globaltimer_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ------------------------------------------------------------- mbarrier ---
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_fence_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Non-blocking probes of three barriers issued back to back, so that their
// shared-memory latencies overlap; r[i] is 1 when barrier i's phase with parity
// q[i] is complete (acquire, like a completed wait).
__device__ __forceinline__ void mbar_test3(uint64_t* b0, uint32_t q0, uint64_t* b1, uint32_t q1, uint64_t* b2,
                                           uint32_t q2, uint32_t (&r)[3]) {
    asm volatile(
        "{\n\t.reg .pred p0, p1, p2;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p0, [%3], %4;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p1, [%5], %6;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p2, [%7], %8;\n\t"
        "selp.u32 %0, 1, 0, p0;\n\t"
        "selp.u32 %1, 1, 0, p1;\n\t"
        "selp.u32 %2, 1, 0, p2;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2])
        : "r"(smem_u32(b0)), "r"(q0), "r"(smem_u32(b1)), "r"(q1), "r"(smem_u32(b2)), "r"(q2)
        : "memory");
}

// Waits for the phase of `bar` with the given parity to complete.  Gives up
// after `limit_ns` nanoseconds, or as soon as *abort is set by another role of
// the same CTA; returns false in both cases.
__device__ __forceinline__ bool mbar_wait_bounded(uint64_t* bar, uint32_t parity,
                                                  unsigned long long limit_ns,
                                                  volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (abort && *abort) return false;
        if (globaltimer_ns() - t0 > limit_ns) return false;
    }
}

// Warp-uniform form of mbar_wait_bounded: every lane of the (converged) warp
// polls, and the warp proceeds only if every lane saw the phase complete, so a
// time-out can never leave the warp diverged before a warp-collective
// instruction.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, unsigned long long limit_ns,
                                               volatile int* abort) {
    const bool ok = mbar_wait_bounded(bar, parity, limit_ns, abort);
    return __all_sync(0xffffffffu, ok);
}

// -------------------------------------------------------------------- TMA ---
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0,
                                            int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3, int c4) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_desc(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// Makes this thread's generic-proxy shared-memory writes visible to the async
// proxy (TMA, tensor cores).
__device__ __forceinline__ void fence_proxy_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// --------------------------------------------------------------- tcgen05 ---
__device__ __forceinline__ void tmem_alloc(uint32_t* dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on `bar` once every tcgen05 operation this thread issued so far has
// completed.
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

// 32 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor for tcgen05.mma (sm_100 family format):
//   bits  0-13 start address >> 4, 16-29 leading byte offset >> 4,
//   32-45 stride byte offset >> 4, 46-47 version (1), 61-63 swizzle mode
//   (2 = 128-byte swizzle).  The 128-byte swizzle atom is 8 rows x 128 bytes.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((lbo_bytes >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)((sbo_bytes >> 4) & 0x3FFFu) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// Instruction descriptor for tcgen05.mma kind::f16 with bf16 inputs and fp32
// accumulation: bits 4-5 D format (1 = f32), 7-9 A format (1 = bf16),
// 10-12 B format (1 = bf16), 15 A major (0 = K), 16 B major (1 = MN),
// 17-22 N >> 3, 24-28 M >> 4.
__host__ __device__ constexpr uint32_t idesc_bf16_f32(int M, int N, int a_mn_major, int b_mn_major) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn_major << 15) | ((uint32_t)b_mn_major << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// ---------------------------------------------------- warp-level MMA path ---
__device__ __forceinline__ void ldsm_x4(uint32_t saddr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(saddr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t saddr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                          uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(saddr));
}
// D = A(16x16 bf16, row) * B(16x8 bf16, col) + C, fp32 accumulate
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// --------------------------------------------------------------- numeric ---
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// max of three floats in one instruction (sm_100+); a NaN input is ignored like fmaxf
__device__ __forceinline__ float fmax3f(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// m16n8k16 warp MMA, f16 inputs, fp32 accumulation (D += A B).
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// tanh in fp32.  |u| <= 1: u times a degree-6 polynomial in u^2, a minimax fit of
// tanh(u) / u made for this file (relative error 5e-8, 1.6e-7 as evaluated);
// beyond, 1 - 2 / (1 + e^(2|u|)), whose cancellation is harmless there (absolute
// error below 3e-7).  The hardware's tanh.approx is off by up to 2^-11, which a
// cap of 50 would turn into 0.02 on a logit.
constexpr float kTanhC0 = 0.99999994f, kTanhC1 = -0.3333284f, kTanhC2 = 0.13325204f, kTanhC3 = -0.053457025f,
                kTanhC4 = 0.020289972f, kTanhC5 = -0.006203373f, kTanhC6 = 0.0010410206f;
__device__ __forceinline__ float tanh_f32(float u) {
    const float a = fabsf(u), w = u * u;
    float t = fmaf(kTanhC6, w, kTanhC5);
    t = fmaf(t, w, kTanhC4);
    t = fmaf(t, w, kTanhC3);
    t = fmaf(t, w, kTanhC2);
    t = fmaf(t, w, kTanhC1);
    t = fmaf(t, w, kTanhC0);
    const float e = fast_exp2(a * 2.885390081777927f);  // e^(2a); +inf gives 1
    const float big = copysignf(1.f - __fdividef(2.f, 1.f + e), u);
    return a <= 1.f ? u * t : big;
}

// tanh on |u| <= kTanhNear: u times a degree-4 polynomial in u^2 of the same kind
// (relative error 2.8e-07 as evaluated).  Both polynomials go on rising past
// the end of their range, so a score below it only gets a still lower logit.
constexpr float kTanhNear = 0.65f;
constexpr float kTanhD0 = 0.9999998f, kTanhD1 = -0.333315f, kTanhD2 = 0.13297874f, kTanhD3 = -0.051517908f,
                kTanhD4 = 0.014625075f;
// tanh with an absolute (not relative) error below 4e-7 anywhere:
// 1 - 2 / (1 + e^(2|u|)) with the hardware's exponential and reciprocal, about
// half of tanh_f32's instructions.  A logit is then off by 4e-7 of the cap, which
// is as much as its own rounding for the caps in use and more than all of its
// digits for very large ones: caps above kWideCap take tanh_f32.
__device__ __forceinline__ float tanh_abs(float u) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + fast_exp2(fabsf(u) * 2.885390081777927f)));
    return copysignf(fmaf(-2.f, r, 1.f), u);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// n / d for 0 <= n < 2^31 by a multiplication: with s = 31 + ceil(log2 d) and
// m = floor(2^s / d) + 1 the error n (m d - 2^s) / (d 2^s) stays below 1 / d.
struct FastDiv {
    uint32_t m = 0;
    int s = 0;
    FastDiv() = default;
    explicit FastDiv(int d) {
        int c = 0;
        while ((1ll << c) < d) ++c;
        s = 31 + c;
        m = (uint32_t)((1ull << s) / (uint64_t)d + 1);
    }
    __device__ __forceinline__ int operator()(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> s); }
};

// ------------------------------------------------------- score modifiers ---
// Logit of query position i and key position j for dot product s, in log2
// units:  f(s) - slope_h log2(e) |i - j|,  f(s) = s scale log2(e), or with a cap
// c log2(e) tanh(s scale / c).  Key j is visible when every mask given allows
// it: causal or prefix (j <= i, or j < prefix), window (j > i - window; without
// the causal flag also j < i + window), and the documents (dense only).
struct ScoreMod {
    float cap_in;           // scale / cap
    float cap_out;          // cap * log2(e); 0: no cap
    const float* slopes;    // fp32 [Hq], or null
    const int32_t* prefix;  // int32 per sequence, or null
    int window;             // 0: none
    float* lse;             // fp32 log-sum-exp per row ([rows, Hq] paged), or null
    float* logits;          // decode rows: logits kept for the weight sums (log2 units), or null
    int logit_rows;         // rows a page's logits take in that buffer
};

// A distance slope in log2 units.  Bounded, so that a slope near fp32's largest
// still times distance 0 is 0 (an infinite one gave NaN for the query's own key).
__device__ __forceinline__ float slope_log2(float slope) {
    constexpr float most = 3.4028235e38f;
    return fminf(fmaxf(slope * 1.4426950408889634f, -most), most);
}

// The capped logit as a polynomial of the raw dot product s, in pairs of equal
// coefficients: c log2(e) tanh(s scale / c) = s (a_0 + a_1 s^2 + ...) while the
// row's largest s scale / c is at most kTanhNear (near) or 1 (unit).  A score
// below minus that bound gets a wrong logit, which is harmless when its weight
// is below 2^-30 of the row's: `slack` plus the row's running max (log2 units)
// has to reach 30.  slack is -inf when a coefficient leaves fp32's range.
// Other rows take the exact tanh_abs, or tanh_f32 when the cap is `wide`: rows
// share a form with their warp, so that a row of ordinary logits meets it too.
constexpr float kWideCap = 256.f;  // c log2(e) up to which tanh_abs is exact enough: 1e-4 of a logit
struct CapPoly {
    float2 near[5], unit[7];
    float near_max, unit_max;      // largest s
    float near_slack, unit_slack;  // c log2(e) tanh(kTanhNear), c log2(e) tanh(1)
    int wide;
};

// Four E4M3 bytes (byte i = element i) to two f16x2 words: lo = elements
// 0, 1 and hi = elements 2, 3 (exact: every E4M3 value is an f16 value).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t x, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}
// Two fp32 values to E4M3 bytes (round to nearest even, saturating at +-448):
// bits 0-7 = lo, bits 8-15 = hi.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\n\t"
        "cvt.u32.u16 %0, t;\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// 32-byte global store (sm_100 family).
__device__ __forceinline__ void st_global_v8(void* p, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t a4,
                                             uint32_t a5, uint32_t a6, uint32_t a7) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a0), "r"(a1), "r"(a2),
                 "r"(a3), "r"(a4), "r"(a5), "r"(a6), "r"(a7)
                 : "memory");
}

// Byte offset of 16-byte chunk `chunk` (0..7) of row `row` inside a
// 128-byte-swizzled tile whose rows are 128 bytes and whose base is
// 1024-byte aligned.
__device__ __forceinline__ uint32_t sw128_offset(uint32_t row, uint32_t chunk) {
    return row * 128u + ((chunk ^ (row & 7u)) << 4);
}

}  // namespace fa
