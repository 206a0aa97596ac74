// Host-side helpers shared by the libfattn translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "common.cuh"

namespace fa {

// Device error word of the current device (a file-scope __device__ variable
// in api.cu; its device address is looked up once per device).
unsigned* error_word_ptr(fa_status* st);

// Per-launch device context: error word + current wait bound.
fa_status make_ctx(DevCtx* ctx);

// Number of SMs of the current device (cached per device).
int sm_count();

// Returns FA_OK when the current device is an sm_103 part.
fa_status check_device();

// Raises `kernel`'s dynamic shared-memory limit to at least `bytes` on the
// current device, once per (device, kernel); thread-safe.
fa_status raise_dynamic_smem(const void* kernel, int bytes);

// Dynamic shared memory that a kernel may be launched with without that: 48 KB less
// its static shared memory (the kernels whose lists grow with a call's sizes have
// at most 700 bytes of it).
constexpr size_t kUnraisedSmem = 48 * 1024 - 1024;

// Records how many kernels the current API call launched (per host thread).
void set_launch_count(int n);

// cuTensorMapEncodeTiled, resolved through the runtime's driver entry point.
fa_status encode_tmap_bf16_4d(CUtensorMap* map, const void* base, const uint64_t dims[4],
                              const uint64_t strides_bytes[3], const uint32_t box[4]);
// 5-D bf16 tensor map, 128-byte swizzle (strides for dims 1..4, in bytes; any order).
fa_status encode_tmap_bf16_5d(CUtensorMap* map, const void* base, const uint64_t dims[5], const uint64_t strides_bytes[4],
                              const uint32_t box[5]);
// The same for any element type and swizzle mode.
fa_status encode_tmap_4d(CUtensorMap* map, const void* base, const uint64_t dims[4], const uint64_t strides_bytes[3],
                         const uint32_t box[4], CUtensorMapDataType dtype, CUtensorMapSwizzle swizzle);

// Tensor maps of the paged tensor-core kernels (defined in attn_tc.cu).
fa_status paged_query_map(CUtensorMap* tq, const void* q, int Hq, int Hkv, int d, int total_q);
fa_status paged_cache_map(CUtensorMap* tk, const void* cache, int num_blocks, int Hkv, int d);

// Prefill of query rows [q0, q0 + Tq) of every sequence against keys [0, Tk)
// (defined in attn_tc.cu; used by the host-buffer pipeline).
fa_status launch_prefill_rows(const void* q, const void* k, const void* v, void* out, int B, int T, int Hq, int Hkv,
                              int d, int causal, float scale, int q0, int Tq, int Tk, cudaStream_t s);

// Checks and packs the score modifiers of a call (lse may be null).  A window
// beyond any length the library can hold is the same as a very long one.
inline fa_status make_score_mod(ScoreMod* m, float scale, float softcap, const float* slopes, int window,
                                const int32_t* prefix, float* lse) {
    if (!(softcap >= 0.f) || !(softcap < INFINITY) || window < 0) return FA_ERR_INVALID_ARG;
    *m = ScoreMod{};
    if (softcap > 0.f) {
        m->cap_in = scale / softcap;
        m->cap_out = softcap * 1.4426950408889634f;
        // both have to be normal numbers (a bad scale is refused with the other arguments)
        if (scale > 0.f && !(m->cap_in >= 1.17549435e-38f && m->cap_in < INFINITY && m->cap_out < INFINITY))
            return FA_ERR_INVALID_ARG;
    }
    m->slopes = slopes;
    m->prefix = prefix;
    m->window = window < (1 << 29) ? window : (1 << 29);
    m->lse = lse;
    return FA_OK;
}

// The polynomial forms of a call's cap (m.cap_out > 0).
inline CapPoly cap_poly(const ScoreMod& m) {
    CapPoly c{};
    const double in = m.cap_in, out = m.cap_out;
    const double near[5] = {kTanhD0, kTanhD1, kTanhD2, kTanhD3, kTanhD4};
    const double unit[7] = {kTanhC0, kTanhC1, kTanhC2, kTanhC3, kTanhC4, kTanhC5, kTanhC6};
    // the last coefficients may be subnormal: 1e-41 still carries 13 bits, more
    // than the 1e-3 that they add to the result needs
    auto fits = [](float x) { return std::fabs(x) > 1e-41f && std::fabs(x) < 1e30f; };
    bool near_fits = true, unit_fits = true;
    double f = out * in;
    for (int k = 0; k < 7; ++k, f *= in * in) {
        const float u = (float)(unit[k] * f);
        c.unit[k] = make_float2(u, u);
        unit_fits &= fits(u);
        if (k < 5) {
            const float n = (float)(near[k] * f);
            c.near[k] = make_float2(n, n);
            near_fits &= fits(n);
        }
    }
    c.wide = m.cap_out > kWideCap;
    c.near_max = (float)(kTanhNear / in);
    c.unit_max = (float)(1.0 / in);
    c.near_slack = near_fits ? (float)(out * std::tanh(kTanhNear)) : -INFINITY;
    c.unit_slack = unit_fits ? (float)(out * std::tanh(1.0)) : -INFINITY;
    return c;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

inline fa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

}  // namespace fa
