// Device helpers of the cache in 8 bits with a scale per block and kv head, and of
// kernels whose warps find their place in a batch from its lengths.
#pragma once

#include <algorithm>

#include "host_common.cuh"

namespace fa {

constexpr int kScaledBlock = 16;  // tokens per block
constexpr int kExpBias = 127;     // scale code e stands for 2^(e - 127)
// The smallest code written, 2^-40: a softmax that folds a block's value scale into its
// exponents keeps all digits while the codes of a context lie within 100 of each other.
constexpr int kExpLeast = 87;

// 2^(code - 127) for a scale code (0: 2^-127; 255: +inf, as the power of two it is not).
__device__ __forceinline__ float scale_of(int code) { return __uint_as_float(code > 0 ? (uint32_t)code << 23 : 0x00400000u); }

// Do a chunk of ql tokens and a context of cl of them (the chunk included) fit the table?
__device__ __forceinline__ bool lens_ok(int ql, int cl, int mbps) {
    return ql >= 0 && ql <= cl && cl <= (long long)mbps * kScaledBlock;
}

// Where items of a batch lie when sequence s has count(q_len, ctx_len) of them (negative:
// none).  Made and asked by whole warps.
struct SeqItem {
    int s, ql, cl;   // sequence and its lengths
    long long off;   // item within the sequence
    int q0;          // first packed query row of the sequence
};
struct SeqScan {
    long long items, rows;  // of the batch
    bool bad;               // some sequence's lengths are inconsistent, with queries or without
    long long n, in, iq, q; // this lane's items and rows, and those up to its end
    int lo, hi;             // its sequences

    template <class Count>
    __device__ __forceinline__ SeqScan(const int32_t* __restrict__ q_lens, const int32_t* __restrict__ ctx_lens, int num_seqs,
                                       int mbps, Count count) {
        const int lane = threadIdx.x & 31, per = (num_seqs + 31) >> 5;
        lo = min(num_seqs, lane * per);
        hi = min(num_seqs, lo + per);
        n = q = 0;
        bool b = false;
#pragma unroll 4
        for (int s = lo; s < hi; ++s) {
            const int ql = __ldg(q_lens + s), cl = __ldg(ctx_lens + s);
            const long long c = count(ql, cl);
            n += max(0ll, c);
            q += max(0, ql);
            b |= !lens_ok(ql, cl, mbps);
        }
        if (!__any_sync(0xffffffffu, n >= 1 << 26 || q >= 1 << 26)) {  // 32 bits hold every sum
            int x = (int)n, y = (int)q;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) {
                    x += u;
                    y += v;
                }
            }
            in = x;
            iq = y;
        } else {
            in = n;
            iq = q;
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, in, o), v = __shfl_up_sync(0xffffffffu, iq, o);
                if (lane >= o) {
                    in += u;
                    iq += v;
                }
            }
        }
        items = __shfl_sync(0xffffffffu, in, 31);
        rows = __shfl_sync(0xffffffffu, iq, 31);
        bad = __any_sync(0xffffffffu, b);
    }
    template <class Count>
    __device__ __forceinline__ bool find(const int32_t* __restrict__ q_lens, const int32_t* __restrict__ ctx_lens, long long idx,
                                         Count count, SeqItem& it) const {
        const int lane = threadIdx.x & 31;
        const unsigned hit = __ballot_sync(0xffffffffu, n > 0 && idx >= in - n && idx < in);
        if (!hit) return false;
        const int src = __ffs(hit) - 1;
        int s_ = 0, ql_ = 0, cl_ = 0, q0_ = 0;
        long long off_ = 0;
        if (lane == src) {
            long long off = idx - (in - n), q0 = iq - q;
            for (int s = lo; s < hi; ++s) {
                const int ql = __ldg(q_lens + s), cl = __ldg(ctx_lens + s);
                const long long c = max(0ll, (long long)count(ql, cl));
                if (off < c) {
                    s_ = s;
                    ql_ = ql;
                    cl_ = cl;
                    off_ = off;
                    q0_ = (int)min(q0, 0x7fffffffLL);  // (past any row when the lengths are nonsense)
                    break;
                }
                off -= c;
                q0 += max(0, ql);
            }
        }
        it.s = __shfl_sync(0xffffffffu, s_, src);
        it.ql = __shfl_sync(0xffffffffu, ql_, src);
        it.cl = __shfl_sync(0xffffffffu, cl_, src);
        it.off = __shfl_sync(0xffffffffu, off_, src);
        it.q0 = __shfl_sync(0xffffffffu, q0_, src);
        return true;
    }
};

// Blocks that a chunk's tokens lie in (-1: inconsistent lengths).
__device__ __forceinline__ int chunk_blocks(int ql, int cl, int mbps) {
    if (!lens_ok(ql, cl, mbps)) return -1;
    return ql == 0 ? 0 : (cl - 1) / kScaledBlock - (cl - ql) / kScaledBlock + 1;
}
// What that can be for all sequences together: n tokens lie in at most (n + 14) / 16 + 1 blocks.
inline long chunk_blocks_bound(int num_seqs, int total_q) {
    return std::min<long>(total_q, total_q / kScaledBlock + 2L * num_seqs);
}

// Four E4M3 bytes times a factor.
__device__ __forceinline__ void e4m3x4_to_f32x4(uint32_t w, float f, float (&x)[4]) {
    uint32_t lo, hi;
    e4m3x4_to_f16x4(w, lo, hi);
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo)), b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    x[0] = a.x * f;
    x[1] = a.y * f;
    x[2] = b.x * f;
    x[3] = b.y * f;
}
__device__ __forceinline__ uint32_t f32x4_to_e4m3x4(float a, float b, float c, float d) {
    return f32x2_to_e4m3x2(a, b) | f32x2_to_e4m3x2(c, d) << 16;
}

}  // namespace fa
