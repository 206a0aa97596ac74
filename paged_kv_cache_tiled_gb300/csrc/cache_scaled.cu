// The paged cache in 8 bits with a scale per block and kv head, and the blocks'
// channel bounds.
//
// fa_cache_append_fp8_scaled: a (block, kv head) holds E4M3 codes and one scale
// 2^(e - 127) for its keys, one for its values.  The scale is a power of two: E4M3
// is a floating format, so a finer scale would not make its values any finer, and
// with powers of two a block whose scale grows keeps its codes' values exactly (only
// what falls below 2^-6 of the new scale is rounded again).  The call knows its
// tokens by sequence (block table and lengths), so a warp owns the codes of a (block,
// head) of K or of V: it loads the block's new tokens (at most 16, a lane D / 32
// channels of each, all loads in flight), turns the keys by rows of cos_sin that its CTA
// has in shared memory for all heads, finds the largest magnitude, and writes codes; no
// atomics, nothing that depends on an order.  V is channel-major: a lane's codes are whole
// 16-byte rows.  Queries are turned by further CTAs of the same launch.  Memory bound on
// prompts, latency bound on single tokens.
//
// fa_block_bounds: smallest and largest value of every channel over a block's tokens,
// recomputed for the blocks that a chunk's tokens lie in; a warp a (block, head).
#include <algorithm>
#include <type_traits>

#include "cache_scaled.cuh"

namespace fa {

struct AppendArgs {
    const void *q, *k, *v;
    const int32_t* positions;  // null: the cache positions
    const float* cos_sin;      // null: no rotation
    uint16_t* q_out;
    uint8_t *kc, *vc, *ke, *ve;
    const int32_t *bt, *ctx_lens, *q_lens;
    int max_pos, num_seqs, mbps, num_blocks, total_q, Hq, Hkv;
    int pairs, parts, block_ctas;  // (head, K or V) pairs a CTA, CTAs a block, and of all blocks; those of the queries follow
    DevCtx ctx;
};

// N consecutive values (N = 2 or 4) as fp32.
template <bool kF32, int N>
struct Raw {
    uint32_t w[kF32 ? N : N / 2];
    __device__ __forceinline__ void load(const void* base, long at) {
        if constexpr (kF32) {
            const float* p = static_cast<const float*>(base) + at;
            if constexpr (N == 4) {
                const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
                w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
            } else {
                const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
                w[0] = u.x; w[1] = u.y;
            }
        } else {
            const uint16_t* p = static_cast<const uint16_t*>(base) + at;
            if constexpr (N == 4) {
                const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
                w[0] = u.x; w[1] = u.y;
            } else {
                w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
            }
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (kF32) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
};

// Eight of them.
template <bool kF32>
struct Raw8 {
    uint4 w[kF32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* base, long at) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + at * (kF32 ? 4 : 2));
#pragma unroll
        for (int i = 0; i < (kF32 ? 2 : 1); ++i) w[i] = __ldg(p + i);
    }
    __device__ __forceinline__ float get(int i) const {
        const uint4& u = w[kF32 ? i / 4 : 0];
        const int k = kF32 ? i % 4 : i / 2;
        const uint32_t v = k == 0 ? u.x : (k == 1 ? u.y : (k == 2 ? u.z : u.w));
        if constexpr (kF32) return __uint_as_float(v);
        else return __uint_as_float(i & 1 ? v & 0xFFFF0000u : v << 16);
    }
};

// E4M3 codes times `ratio` (a power of two), rounded again.
__device__ __forceinline__ uint32_t rescale_codes(uint32_t w, float ratio) {
    float x[4];
    e4m3x4_to_f32x4(w, ratio, x);
    return f32x4_to_e4m3x4(x[0], x[1], x[2], x[3]);
}

// A CTA takes a block that new tokens go to, or a part of its heads: one (head, K or V) pair a warp, two when there
// are many blocks; even warps keys, odd warps values.  Prompts need bytes in flight, so no register holds a value that
// can be worked out again and an SM has seven CTAs (with four and all values kept 5123 tokens of 8 heads took 32.9 us, now
// 26.6; 1117 tokens with two pairs a warp 14.4, with one 10.3).
constexpr int kAppendWarps = 4;

template <int D, bool kF32>
__global__ void __launch_bounds__(kAppendWarps * 32, kF32 ? 4 : 7) append_scaled_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int N = D / 32, B = kScaledBlock;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    SeqItem it;
    if ((int)blockIdx.x < a.block_ctas) {
        __shared__ __align__(16) float turns[B][D];  // the tokens' rows of cos_sin
        const int part = blockIdx.x % a.parts, place = blockIdx.x / a.parts;
        auto count = [&](int ql, int cl) { return chunk_blocks(ql, cl, a.mbps); };
        const SeqScan scan(a.q_lens, a.ctx_lens, a.num_seqs, a.mbps, count);
        if (blockIdx.x == 0 && threadIdx.x == 0 && (scan.bad || scan.rows > a.total_q)) raise_error(a.ctx, ERR_BOUNDS_BIT);
        // (the same for the whole CTA from here on, but for the pairs)
        if (!scan.find(a.q_lens, a.ctx_lens, place, count, it) || (long long)it.q0 + it.ql > a.total_q) return;
        const int first = it.cl - it.ql, blk = first / B + (int)it.off;
        const int lo = max(0, first - blk * B), hi = min(B, it.cl - blk * B);  // the block's new tokens
        const int phys = __ldg(a.bt + (long)it.s * a.mbps + blk);
        const long row0 = (long)it.q0 + blk * B - first;  // packed row of the block's token 0
        Raw<kF32, N> raw[B];
        const bool is_v = warp & 1;
        auto load = [&](int pair) {
            const long at = (row0 * a.Hkv + pair / 2) * D + lane * N;
#pragma unroll
            for (int i = 0; i < B; ++i)
                if (i >= lo && i < hi) raw[i].load(is_v ? a.v : a.k, at + (long)i * a.Hkv * D);
        };
        const int end = min(2 * a.Hkv, (part + 1) * a.pairs);
        int pair = part * a.pairs + warp;
        if (pair < end) load(pair);
        unsigned live = ((1u << hi) - 1) & ~((1u << lo) - 1);
        if (a.cos_sin) {
            // lane i: token i's position
            const int i = lane & 15;
            const bool in = lane < B && i >= lo && i < hi;
            const int pos = !in ? 0 : (a.positions ? __ldg(a.positions + row0 + i) : blk * B + i);
            const unsigned out = __ballot_sync(0xffffffffu, in && (pos < 0 || pos >= a.max_pos));
            if (out && threadIdx.x == 0) raise_error(a.ctx, ERR_BOUNDS_BIT);
            live &= ~out;
            constexpr int kQuads = D / 4;
            for (int x = threadIdx.x; x < B * kQuads; x += kAppendWarps * 32) {  // (whole warps)
                const int tok = x / kQuads, p = __shfl_sync(0xffffffffu, pos, tok);
                if ((live >> tok) & 1u)
                    *reinterpret_cast<float4*>(&turns[tok][x % kQuads * 4]) =
                        __ldg(reinterpret_cast<const float4*>(a.cos_sin + (long)p * D) + x % kQuads);
            }
            __syncthreads();
        }
        if (phys < 0 || phys >= a.num_blocks) {
            if (threadIdx.x == 0) raise_error(a.ctx, ERR_BOUNDS_BIT);
            return;
        }
        const bool turned = !is_v && a.cos_sin;
        const int at_pair = (lane & 15) * N;  // channel j < D/2 (lanes 0 .. 15) pairs with j + D/2 (lanes 16 .. 31)
        for (; pair < end; pair += kAppendWarps) {
            const long head = (long)phys * a.Hkv + pair / 2;
            uint8_t* page = (is_v ? a.vc : a.kc) + head * B * D;
            uint8_t* exps = is_v ? a.ve : a.ke;
            const int e_old = lo > 0 ? (int)exps[head] : 0;
            // token i's values, turned (worked out twice: registers for all of them would halve the loads in flight)
            auto values = [&](int i, float (&x)[N]) {
#pragma unroll
                for (int c = 0; c < N; ++c) x[c] = raw[i].get(c);
                if (turned) {
#pragma unroll
                    for (int c = 0; c < N; ++c) {
                        const float y = __shfl_xor_sync(0xffffffffu, x[c], 16);
                        const float co = turns[i][at_pair + c], ys = y * turns[i][D / 2 + at_pair + c];
                        x[c] = fmaf(x[c], co, lane < 16 ? -ys : ys);
                    }
                }
            };
            float m = 0.f;  // the largest finite magnitude
#pragma unroll
            for (int i = 0; i < B; ++i) {
                if (!((live >> i) & 1u)) continue;  // (the same for the whole warp)
                float x[N];
                values(i, x);
#pragma unroll
                for (int c = 0; c < N; ++c) m = fabsf(x[c]) < INFINITY ? fmaxf(m, fabsf(x[c])) : m;
            }
            // the smallest code whose 448 (1.75 * 2^8) times the scale reaches it
            const uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
            const int e = max(max(e_old, kExpLeast), (int)(mb >> 23) - 8 + ((mb & 0x7FFFFFu) > 0x600000u ? 1 : 0));
            const float inv = __uint_as_float((uint32_t)max(0, 254 - e) << 23);                 // 2^(127 - e)
            const float ratio = __uint_as_float((uint32_t)max(0, kExpBias + e_old - e) << 23);  // of the older tokens' codes
            const bool moved = lo > 0 && e != e_old;
            if (!is_v) {
                uint8_t* at = page + lane * N;
                if (moved) {
                    for (int i = 0; i < lo; ++i) {
                        if constexpr (N == 4)
                            *reinterpret_cast<uint32_t*>(at + i * D) = rescale_codes(*reinterpret_cast<uint32_t*>(at + i * D), ratio);
                        else
                            *reinterpret_cast<uint16_t*>(at + i * D) =
                                (uint16_t)rescale_codes(*reinterpret_cast<uint16_t*>(at + i * D), ratio);
                    }
                }
#pragma unroll
                for (int i = 0; i < B; ++i) {
                    if (!((live >> i) & 1u)) continue;
                    float x[N];
                    values(i, x);
                    const uint32_t lo2 = f32x2_to_e4m3x2(x[0] * inv, x[1] * inv);
                    if constexpr (N == 4)
                        *reinterpret_cast<uint32_t*>(at + i * D) = lo2 | f32x2_to_e4m3x2(x[2] * inv, x[3] * inv) << 16;
                    else
                        *reinterpret_cast<uint16_t*>(at + i * D) = (uint16_t)lo2;
                }
            } else {
                uint4* at = reinterpret_cast<uint4*>(page) + lane * N;  // a channel's 16 tokens
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    const uint4 old = live == 0xffffu ? make_uint4(0, 0, 0, 0) : at[c];
                    uint32_t o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        auto bytes = [](unsigned b) {
                            return ((b & 1u) | (b & 2u) << 7 | (b & 4u) << 14 | (b & 8u) << 21) * 255u;
                        };
                        if (moved) {
                            const uint32_t mask = bytes((((1u << lo) - 1) >> (4 * w)) & 15u);
                            o[w] = (o[w] & ~mask) | (rescale_codes(o[w], ratio) & mask);
                        }
                        const uint32_t mask = bytes((live >> (4 * w)) & 15u);
                        o[w] = (o[w] & ~mask) | (f32x4_to_e4m3x4(raw[4 * w].get(c) * inv, raw[4 * w + 1].get(c) * inv,
                                                                 raw[4 * w + 2].get(c) * inv, raw[4 * w + 3].get(c) * inv) & mask);
                    }
                    at[c] = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            if (lane == 0) exps[head] = (uint8_t)e;
            if (pair + kAppendWarps < end) load(pair + kAppendWarps);
        }
        return;
    }
    // a query token a warp: D / 16 lanes a head, 8 channel pairs each
    const int row = ((int)blockIdx.x - a.block_ctas) * kAppendWarps + warp;
    if (row >= a.total_q || !a.q) return;
    constexpr int kLanes = D / 16, kHeads = 32 / kLanes, kAhead = 4;
    const int c = (lane % kLanes) * 8, h0 = lane / kLanes;
    Raw8<kF32> x[kAhead], y[kAhead];
    auto load = [&](int h) {
        const long base = (long)row * a.Hq * D + c;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (h + k * kHeads < a.Hq) {
                x[k].load(a.q, base + (long)(h + k * kHeads) * D);
                y[k].load(a.q, base + (long)(h + k * kHeads) * D + D / 2);
            }
    };
    load(h0);  // on their way while the token's sequence is found
    auto count = [](int ql, int) { return max(0, ql); };
    const SeqScan scan(a.q_lens, a.ctx_lens, a.num_seqs, a.mbps, count);
    if (!scan.find(a.q_lens, a.ctx_lens, row, count, it)) return;
    const int pos = a.positions ? __ldg(a.positions + row) : it.cl - it.ql + (row - it.q0);
    const bool fits = lens_ok(it.ql, it.cl, a.mbps) && rows_fit(it.q0, it.ql, a.total_q);  // (reported above)
    const bool in = pos >= 0 && pos < a.max_pos;
    if (fits && !in && lane == 0) raise_error(a.ctx, ERR_BOUNDS_BIT);
    if (fits && in) {
        Raw8<true> co, si;
        co.load(a.cos_sin, (long)pos * D + c);
        si.load(a.cos_sin, (long)pos * D + D / 2 + c);
        for (int h = h0; h < a.Hq; h += kAhead * kHeads) {
            if (h != h0) load(h);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (h + k * kHeads >= a.Hq) break;
                const long at = ((long)row * a.Hq + h + k * kHeads) * D + c;
                float u[8], v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    u[i] = fmaf(x[k].get(i), co.get(i), -(y[k].get(i) * si.get(i)));
                    v[i] = fmaf(y[k].get(i), co.get(i), x[k].get(i) * si.get(i));
                }
                *reinterpret_cast<uint4*>(a.q_out + at) =
                    make_uint4(pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]), pack_bf16x2(u[4], u[5]), pack_bf16x2(u[6], u[7]));
                *reinterpret_cast<uint4*>(a.q_out + at + D / 2) =
                    make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
            }
        }
    }
}

// ------------------------------------------------------------------ bounds --
// (40 registers, so that an SM holds 48 warps: 8080 blocks and heads 11.2 us; with values as fp32 one by one, 48 registers
// and 40 warps, 12.3)
template <int D, bool KV8>
__global__ void __launch_bounds__(128, 12) block_bounds_kernel(const void* __restrict__ kc, const uint8_t* __restrict__ ke,
                                                           const int32_t* __restrict__ bt,
                                                           const int32_t* __restrict__ ctx_lens,
                                                           const int32_t* __restrict__ q_lens, uint16_t* __restrict__ bounds,
                                                           int num_seqs, int mbps, int num_blocks, int total_q, int Hkv,
                                                           DevCtx ctx) {
    constexpr int N = D / 32, B = kScaledBlock;
    const int w = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31, hk = w % Hkv;
    SeqItem it;
    auto count = [&](int ql, int cl) { return chunk_blocks(ql, cl, mbps); };
    const SeqScan scan(q_lens, ctx_lens, num_seqs, mbps, count);
    if (w == 0 && lane == 0 && (scan.bad || scan.rows > total_q)) raise_error(ctx, ERR_BOUNDS_BIT);
    if (!scan.find(q_lens, ctx_lens, w / Hkv, count, it)) return;
    const int blk = (it.cl - it.ql) / B + (int)it.off, n = min(B, it.cl - blk * B);
    const int phys = __ldg(bt + (long)it.s * mbps + blk);
    if (phys < 0 || phys >= num_blocks) {
        if (lane == 0) raise_error(ctx, ERR_BOUNDS_BIT);
        return;
    }
    const long head = (long)phys * Hkv + hk;
    uint32_t raw[B][KV8 ? 1 : N / 2];
#pragma unroll
    for (int i = 0; i < B; ++i) {
        const long at = head * B * D + i * D + lane * N;
        if (i >= n) continue;
        if constexpr (KV8) {
            if constexpr (N == 4) raw[i][0] = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(kc) + at));
            else raw[i][0] = __ldg(reinterpret_cast<const uint16_t*>(static_cast<const uint8_t*>(kc) + at));
        } else {
            Raw<false, N> r;
            r.load(kc, at);
#pragma unroll
            for (int c = 0; c < N / 2; ++c) raw[i][c] = r.w[c];
        }
    }
    const float f = KV8 ? scale_of(ke[head]) : 1.f;
    // two channels at a time, codes as f16 (which holds them; their scale follows at the end); a NaN gives way to a number
    using Two = std::conditional_t<KV8, __half2, __nv_bfloat162>;
    auto two = [](uint32_t w) { return *reinterpret_cast<const Two*>(&w); };
    Two lo[N / 2], hi[N / 2];
#pragma unroll
    for (int c = 0; c < N / 2; ++c) {
        lo[c] = two(KV8 ? 0x7C007C00u : 0x7F807F80u);  // +inf
        hi[c] = two(KV8 ? 0xFC00FC00u : 0xFF80FF80u);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
        if (i >= n) continue;
        uint32_t x[2];
        if constexpr (KV8) {
            e4m3x4_to_f16x4(raw[i][0], x[0], x[1]);
        } else {
#pragma unroll
            for (int c = 0; c < N / 2; ++c) x[c] = raw[i][c];
        }
#pragma unroll
        for (int c = 0; c < N / 2; ++c) {
            lo[c] = __hmin2(lo[c], two(x[c]));
            hi[c] = __hmax2(hi[c], two(x[c]));
        }
    }
    // a channel without a number (its keys are NaN) is 0 to 0, so that bounds are finite
#pragma unroll
    for (int c = 0; c < N / 2; ++c) {
        const uint32_t some = ~__hgt2_mask(lo[c], hi[c]);
        const uint32_t l = *reinterpret_cast<const uint32_t*>(&lo[c]) & some, h = *reinterpret_cast<const uint32_t*>(&hi[c]) & some;
        lo[c] = two(l);
        hi[c] = two(h);
    }
    auto word = [&](const Two& v) -> uint32_t {
        if constexpr (KV8) {
            const float2 x = __half22float2(v);
            return pack_bf16x2(x.x * f, x.y * f);  // (E4M3 values times a power of two: exact)
        } else {
            return *reinterpret_cast<const uint32_t*>(&v);
        }
    };
    uint16_t* dst = bounds + head * 2 * D + lane * N;
    if constexpr (N == 4) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(word(lo[0]), word(lo[1]));
        *reinterpret_cast<uint2*>(dst + D) = make_uint2(word(hi[0]), word(hi[1]));
    } else {
        *reinterpret_cast<uint32_t*>(dst) = word(lo[0]);
        *reinterpret_cast<uint32_t*>(dst + D) = word(hi[0]);
    }
}

}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_cache_append_fp8_scaled(const void* q, const void* k, const void* v, const int32_t* positions,
                                     const float* cos_sin, int max_pos, void* q_out, void* k_cache, void* v_cache,
                                     uint8_t* k_exp, uint8_t* v_exp, const int32_t* block_table, const int32_t* ctx_lens,
                                     const int32_t* q_lens, int num_seqs, int max_blocks_per_seq, int num_blocks,
                                     int total_q, int Hq, int Hkv, int d, int block_size, fa_dtype in_dtype,
                                     fa_stream_t stream) {
    set_launch_count(0);
    if (num_seqs < 0 || max_blocks_per_seq < 0 || num_blocks < 0 || total_q < 0 || Hkv <= 0 || max_pos < 0 ||
        (q && Hq <= 0) || (in_dtype != FA_BF16 && in_dtype != FA_F32))
        return FA_ERR_INVALID_ARG;
    if (block_size != kScaledBlock || (d != 64 && d != 128)) return FA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0) return FA_OK;
    if (!k || !v || !k_cache || !v_cache || !k_exp || !v_exp || !block_table || !ctx_lens || !q_lens) return FA_ERR_INVALID_ARG;
    if ((q && (!q_out || !cos_sin)) || (positions && !cos_sin)) return FA_ERR_INVALID_ARG;  // queries are only turned
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(q) || !aligned16(q_out) ||
        !aligned16(cos_sin))
        return FA_ERR_INVALID_ARG;
    if (num_blocks == 0 || max_blocks_per_seq == 0) return FA_ERR_INVALID_ARG;
    fa_status st = check_device();
    if (st != FA_OK) return st;
    AppendArgs a{q, k, v, positions, cos_sin, static_cast<uint16_t*>(q_out), static_cast<uint8_t*>(k_cache),
                 static_cast<uint8_t*>(v_cache), k_exp, v_exp, block_table, ctx_lens, q_lens, max_pos, num_seqs,
                 max_blocks_per_seq, num_blocks, total_q, Hq, Hkv, kAppendWarps, 1, 0, {}};
    if ((st = make_ctx(&a.ctx)) != FA_OK) return st;
    const long blocks = chunk_blocks_bound(num_seqs, total_q);
    // (more CTAs than the GPU holds at once: two pairs a warp, which share a CTA's search and its rows of cos_sin)
    if (blocks * ((2 * Hkv + kAppendWarps - 1) / kAppendWarps) > 7L * sm_count()) a.pairs = 2 * kAppendWarps;
    a.parts = (2 * Hkv + a.pairs - 1) / a.pairs;
    const long block_ctas = blocks * a.parts, ctas = block_ctas + (q ? (total_q + kAppendWarps - 1) / kAppendWarps : 0);
    if (ctas > 0x7fffffffL) return FA_ERR_UNSUPPORTED;
    a.block_ctas = (int)block_ctas;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto kernel = d == 128 ? (in_dtype == FA_F32 ? append_scaled_kernel<128, true> : append_scaled_kernel<128, false>)
                           : (in_dtype == FA_F32 ? append_scaled_kernel<64, true> : append_scaled_kernel<64, false>);
    kernel<<<(unsigned)ctas, kAppendWarps * 32, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    set_launch_count(1);
    return FA_OK;
}

fa_status fa_block_bounds(const void* k_cache, const uint8_t* k_exp, const int32_t* block_table, const int32_t* ctx_lens,
                          const int32_t* q_lens, void* bounds, int num_seqs, int max_blocks_per_seq, int num_blocks,
                          int total_q, int Hkv, int d, int block_size, fa_stream_t stream) {
    set_launch_count(0);
    if (num_seqs < 0 || max_blocks_per_seq < 0 || num_blocks < 0 || total_q < 0 || Hkv <= 0) return FA_ERR_INVALID_ARG;
    if (block_size != kScaledBlock || (d != 64 && d != 128)) return FA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0) return FA_OK;
    if (!k_cache || !block_table || !ctx_lens || !q_lens || !bounds) return FA_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(bounds)) return FA_ERR_INVALID_ARG;
    if (num_blocks == 0 || max_blocks_per_seq == 0) return FA_ERR_INVALID_ARG;
    fa_status st = check_device();
    if (st != FA_OK) return st;
    DevCtx ctx;
    if ((st = make_ctx(&ctx)) != FA_OK) return st;
    const long ctas = (chunk_blocks_bound(num_seqs, total_q) * Hkv + 3) / 4;
    if (ctas > 0x1fffffffL) return FA_ERR_UNSUPPORTED;
    auto kernel = d == 128 ? (k_exp ? block_bounds_kernel<128, true> : block_bounds_kernel<128, false>)
                           : (k_exp ? block_bounds_kernel<64, true> : block_bounds_kernel<64, false>);
    kernel<<<(unsigned)ctas, 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        k_cache, k_exp, block_table, ctx_lens, q_lens, static_cast<uint16_t*>(bounds), num_seqs, max_blocks_per_seq,
        num_blocks, total_q, Hkv, ctx);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    set_launch_count(1);
    return FA_OK;
}

}  // extern "C"
