// Attention of up to 16 query rows over pages of 16 keys with warp MMAs: what the
// kernels that stream single pages of a paged cache share.
#pragma once

#include "cache_scaled.cuh"

namespace fa {

// KV8 false: bf16 pages, K and V [16 tokens][D], one 64-channel half (16 rows of 128
// bytes, 128-byte swizzle) after the other.
// KV8 true: pages of the 8-bit cache, K [16 tokens][D] bytes (rows of D bytes, swizzled
// over their length), V [D channels][16 tokens] bytes.  Both go to f16, which holds
// every E4M3 value; a row of queries is divided by a power of two of its own first, so
// that f16 holds it whatever its magnitude.  The MMA's K dimension is taken in a
// permuted order, so that a lane word of one ldmatrix (4 channels, or 4 tokens of V)
// gives both B registers: logical k (2t, 2t+1, 2t+8, 2t+9) = elements 4t .. 4t+3; K rows
// are loaded so that the score tile's columns come out in the order that P V takes.
//
// A block's scales 2^ks (keys) and 2^ev (values) are powers of two.  2^ks multiplies the
// scores; 2^ev goes into the exponent: with w = x + ev the weights are
// p = 2^(w - m), m the running maximum of w, so that f16 holds them whatever the
// scales; O = sum p code, l = sum 2^-ev p, and the result is O / l.  No weight passes 1,
// so they go to f16 times 2^15 (32768 of 65504): it keeps all its digits down to 2^-29 of
// the largest and something down to 2^-40, which without it would be 2^-14 and 2^-25.
// O is that much larger until the end (kDown); l and m are not.
template <int D, bool KV8>
struct PageMma {
    static constexpr int kPage = kScaledBlock * D * (KV8 ? 1 : 2);  // bytes of a K (or V) page
    static constexpr int kSlotRow = D + 8;                          // floats between rows of a partial result
    static constexpr float kUp = KV8 ? 15.f : 0.f, kDown = KV8 ? 0x1p-15f : 1.f;  // O is 2^kUp times the sum of p and values
    uint32_t qa[D / 16][4];
    float o[D / 8][4];
    float m[2], l[2];
    float mul[2];  // scale * log2(e) times what the row was divided by

    // Query rows gid and gid + 8 (null: zeros).
    __device__ __forceinline__ void load_q(const uint16_t* r0, const uint16_t* r1, float scale_log2) {
        const int tig = threadIdx.x & 3;
        const uint16_t* row[2] = {r0, r1};
        if constexpr (KV8) {
            uint2 w[2][D / 16];  // channels 4t .. 4t + 3 of each 16: the permuted order
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t top = 0;  // largest magnitude, as bf16 bits
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    w[i][ks] = row[i] ? __ldg(reinterpret_cast<const uint2*>(row[i] + ks * 16 + tig * 4)) : make_uint2(0u, 0u);
                    top = max(max(top, w[i][ks].x & 0x7fffu), (w[i][ks].x >> 16) & 0x7fffu);
                    top = max(max(top, w[i][ks].y & 0x7fffu), (w[i][ks].y >> 16) & 0x7fffu);
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // divided by 2^e, e the largest value's exponent: values below 2 (within fp32's normal powers)
                const int e = top == 0 ? 0 : min(126, max(-126, (int)(top >> 7) - 127));
                const float f = __uint_as_float((uint32_t)(127 - e) << 23);
                mul[i] = scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint2 u = w[i][ks];
                    qa[ks][i] = pack_f16x2(__uint_as_float(u.x << 16) * f, __uint_as_float(u.x & 0xFFFF0000u) * f);
                    qa[ks][i + 2] = pack_f16x2(__uint_as_float(u.y << 16) * f, __uint_as_float(u.y & 0xFFFF0000u) * f);
                }
            }
        } else {
            mul[0] = mul[1] = scale_log2;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = ks * 16 + tig * 2;
                    qa[ks][i] = row[i] ? __ldg(reinterpret_cast<const uint32_t*>(row[i] + c)) : 0u;
                    qa[ks][i + 2] = row[i] ? __ldg(reinterpret_cast<const uint32_t*>(row[i] + c + 8)) : 0u;
                }
        }
    }
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }
    // Token of this lane's column pair (nt, e) within a page.
    static __device__ __forceinline__ int token(int nt, int e) {
        const int tig = threadIdx.x & 3;
        return KV8 ? tig * 4 + nt * 2 + e : nt * 8 + tig * 2 + e;
    }
    // 16 rows x 16 tokens of Q K^T
    __device__ __forceinline__ void scores(uint32_t kbase, float (&sc)[2][4]) const {
        const int lane = threadIdx.x & 31, mi = lane >> 3, r8 = lane & 7;
        if constexpr (KV8) {
            // matrix mi: n-tile mi & 1, 16-byte chunk 2j + (mi >> 1)
            const int tok = (r8 >> 1) * 4 + 2 * (mi & 1) + (r8 & 1);
            const int sw = D == 128 ? tok & 7 : (tok >> 1) & 3;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                uint32_t w[4], b[8];
                ldsm_x4(kbase + tok * D + (((2 * j + (mi >> 1)) ^ sw) << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) e4m3x4_to_f16x4(w[i], b[2 * i], b[2 * i + 1]);
                mma_f16_16816(sc[0], qa[2 * j], b[0], b[1]);
                mma_f16_16816(sc[1], qa[2 * j], b[2], b[3]);
                mma_f16_16816(sc[0], qa[2 * j + 1], b[4], b[5]);
                mma_f16_16816(sc[1], qa[2 * j + 1], b[6], b[7]);
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const int tok = (mi >> 1) * 8 + r8, chunk = ks * 2 + (mi & 1);
                uint32_t b0, b1, b2, b3;
                ldsm_x4(kbase + (chunk >> 3) * 2048 + sw128_offset(tok, chunk & 7), b0, b1, b2, b3);
                mma_bf16_16816(sc[0], qa[ks], b0, b1);
                mma_bf16_16816(sc[1], qa[ks], b2, b3);
            }
        }
    }
    // Zeroes the values of tokens from nvalid on in a V page (whatever is stored there must not meet a weight of 0).
    static __device__ __forceinline__ void clear_tail(uint32_t vbase, int nvalid) {
        const int lane = threadIdx.x & 31;
        if constexpr (KV8) {
            for (int c = lane; c < D; c += 32)
                for (int w = 0; w < 4; ++w) {
                    const int left = nvalid - 4 * w;
                    if (left >= 4) continue;
                    uint32_t v;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(vbase + c * 16 + w * 4));
                    v &= left <= 0 ? 0u : (1u << (8 * left)) - 1;
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(vbase + c * 16 + w * 4), "r"(v) : "memory");
                }
        } else {
            for (int i = lane; i < (kScaledBlock - nvalid) * (D / 8); i += 32) {
                const int row = nvalid + i / (D / 8), c = i % (D / 8);
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vbase + (c >> 3) * 2048 + row * 128 + (c & 7) * 16), "r"(0)
                             : "memory");
            }
        }
        fence_proxy_async_smem();  // (the next copy to this place comes through the async proxy)
        __syncwarp();
    }
    // O += P V
    __device__ __forceinline__ void add_pv(uint32_t vbase, const float (&p)[2][4]) {
        const int lane = threadIdx.x & 31, mi = lane >> 3, r8 = lane & 7;
        if constexpr (KV8) {
            const uint32_t pa[4] = {pack_f16x2(p[0][0], p[0][1]), pack_f16x2(p[0][2], p[0][3]), pack_f16x2(p[1][0], p[1][1]),
                                    pack_f16x2(p[1][2], p[1][3])};
#pragma unroll
            for (int q4 = 0; q4 < D / 32; ++q4) {
                uint32_t w[4];
                ldsm_x4(vbase + ((4 * q4 + mi) * 8 + r8) * 16, w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t b0, b1;
                    e4m3x4_to_f16x4(w[i], b0, b1);
                    mma_f16_16816(o[4 * q4 + i], pa, b0, b1);
                }
            }
        } else {
            const uint32_t pa[4] = {pack_bf16x2(p[0][0], p[0][1]), pack_bf16x2(p[0][2], p[0][3]),
                                    pack_bf16x2(p[1][0], p[1][1]), pack_bf16x2(p[1][2], p[1][3])};
#pragma unroll
            for (int dn = 0; dn < D / 16; ++dn) {
                const int tok = (mi & 1) * 8 + r8, chunk = dn * 2 + (mi >> 1);
                uint32_t b0, b1, b2, b3;
                ldsm_x4_t(vbase + (chunk >> 3) * 2048 + sw128_offset(tok, chunk & 7), b0, b1, b2, b3);
                mma_bf16_16816(o[2 * dn], pa, b0, b1);
                mma_bf16_16816(o[2 * dn + 1], pa, b2, b3);
            }
        }
    }
    // One pass of the softmax over n <= NP pages at once (their chains of MMAs overlap).
    // Page i: K at kv[i], V kPage behind it, its first token at position tok[i], its scale
    // codes ks[i], ev[i] (KV8).  Row gid (gid + 8) sees the keys up to position lim0 (lim1);
    // values at positions from `len` on count as zeros.
    template <int NP>
    __device__ __forceinline__ void step(int n, const uint32_t (&kv)[NP], const int (&tok)[NP], const int (&ks)[NP],
                                         const int (&ev)[NP], int lim0, int lim1, int len) {
        float x[NP][2][4], mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < NP; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][0][e] = x[i][1][e] = 0.f;
            if (i < n) scores(kv[i], x[i]);
        }
        bool all = n == NP;  // every key of every page visible to every row
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const float f0 = KV8 ? mul[0] * scale_of(ks[i]) : mul[0], f1 = KV8 ? mul[1] * scale_of(ks[i]) : mul[1];
            const float add = KV8 ? (float)(ev[i] - kExpBias) : 0.f;
            all = all && min(lim0, lim1) - tok[i] >= kScaledBlock - 1;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[i][nt][e] = KV8 ? fmaf(x[i][nt][e], e < 2 ? f0 : f1, add) : x[i][nt][e] * (e < 2 ? f0 : f1);
        }
        if (!__all_sync(0xffffffffu, all)) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int a0 = i < n ? lim0 - tok[i] : -1, a1 = i < n ? lim1 - tok[i] : -1;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (token(nt, e & 1) > (e < 2 ? a0 : a1)) x[i][nt][e] = -INFINITY;
                if (i < n && len - tok[i] < kScaledBlock) clear_tail(kv[i] + kPage, max(0, len - tok[i]));
            }
        }
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], fmaxf(x[i][0][e], x[i][1][e]));
        float a[2], use[2];  // (use: what a weight's exponent is less than its w by)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
            const float mn = fmaxf(m[r], mx[r]);
            const float top = mn == -INFINITY ? 0.f : mn;
            a[r] = fast_exp2(m[r] - top);
            use[r] = top - kUp;
            m[r] = mn;
            l[r] *= a[r];
        }
        if (__any_sync(0xffffffffu, a[0] != 1.f || a[1] != 1.f)) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                o[c][0] *= a[0];
                o[c][1] *= a[0];
                o[c][2] *= a[1];
                o[c][3] *= a[1];
            }
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            if (i >= n) continue;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][nt][e] = fast_exp2(x[i][nt][e] - use[e >> 1]);
            const float back = KV8 ? scale_of(2 * kExpBias - ev[i]) * kDown : 1.f;  // 2^-ev, of sums 2^kUp times too large
            l[0] = fmaf(back, (x[i][0][0] + x[i][0][1]) + (x[i][1][0] + x[i][1][1]), l[0]);
            l[1] = fmaf(back, (x[i][0][2] + x[i][0][3]) + (x[i][1][2] + x[i][1][3]), l[1]);
            add_pv(kv[i] + kPage, x[i]);
        }
    }
    // The rows' sums over the four lanes that share them.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        }
    }
    // Rows below nrows to a partial result in shared memory: O, then (max, sum) per row.
    __device__ __forceinline__ void store_partial(float* slot, int nrows) const {
        const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = gid + 8 * i;
            if (r >= nrows) continue;
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<float2*>(slot + r * kSlotRow + c * 8 + tig * 2) = make_float2(o[c][2 * i], o[c][2 * i + 1]);
            if (tig == 0) reinterpret_cast<float2*>(slot + 16 * kSlotRow)[r] = make_float2(m[i], l[i]);
        }
    }
    static constexpr int kSlotFloats = 16 * kSlotRow + 32;
};

// Warps of the kernel for listed blocks that an SM holds, by their registers and rings.
constexpr int kListSmWarps = 12;

// Tensor maps of the caches as these kernels take them (one box a page; bf16: a half of one).
template <int D, bool KV8>
inline fa_status page_maps(const void* k_cache, const void* v_cache, int num_blocks, int Hkv, CUtensorMap* tk, CUtensorMap* tv) {
    constexpr uint64_t B = kScaledBlock, size = KV8 ? 1 : 2;
    const uint64_t kd[4] = {(uint64_t)D, B, (uint64_t)Hkv, (uint64_t)num_blocks};
    const uint64_t ks[3] = {D * size, B * D * size, Hkv * B * D * size};
    fa_status st;
    if constexpr (KV8) {
        // (a V page lands as it is: in rows of 128 bytes, since TMA takes rows of 16 bytes at a fraction of the rate)
        const uint32_t kb[4] = {D, (uint32_t)B, 1, 1}, vb[4] = {128, D / 8, 1, 1};
        const uint64_t vd[4] = {128, (uint64_t)D / 8, (uint64_t)Hkv, (uint64_t)num_blocks};
        const uint64_t vs[3] = {128, B * D, Hkv * B * D};
        st = encode_tmap_4d(tk, k_cache, kd, ks, kb, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                            D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
        if (st == FA_OK) st = encode_tmap_4d(tv, v_cache, vd, vs, vb, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE);
    } else {
        const uint32_t box[4] = {64, (uint32_t)B, 1, 1};
        st = encode_tmap_bf16_4d(tk, k_cache, kd, ks, box);
        if (st == FA_OK) st = encode_tmap_bf16_4d(tv, v_cache, kd, ks, box);
    }
    return st;
}

// One thread requests a page: K at dst, V behind it (2 * kPage bytes on `bar`).  A block
// outside the map fills zeros.
template <int D, bool KV8>
__device__ __forceinline__ void load_page(uint8_t* dst, const CUtensorMap* tk, const CUtensorMap* tv, uint64_t* bar, int hk,
                                          int blk) {
    constexpr int kPage = PageMma<D, KV8>::kPage;
    mbar_arrive_expect_tx(bar, 2 * kPage);
    if constexpr (KV8) {
        tma_load_4d(dst, tk, bar, 0, 0, hk, blk);
        tma_load_4d(dst + kPage, tv, bar, 0, 0, hk, blk);
    } else {
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
            tma_load_4d(dst + h * 2048, tk, bar, h * 64, 0, hk, blk);
            tma_load_4d(dst + kPage + h * 2048, tv, bar, h * 64, 0, hk, blk);
        }
    }
}

}  // namespace fa
