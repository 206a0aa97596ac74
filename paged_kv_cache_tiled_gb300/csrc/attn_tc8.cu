// Chunks of queries over the paged cache in 8 bits with block scales, on tcgen05
// tensor cores (fa_paged_attn_fp8_scaled; single tokens take paged.cu's decode kernel).
//
// The algorithm and the division into work units are attn_tc.cu's: a unit is two
// 128-row query tiles ("slots") that share every K/V tile of 128 keys; S = Q K^T and
// O += P V in TMEM; the softmax threads own a row each and write P over S.  What is
// different is how the operands come about.  MMAs take operands of one type, and f16
// holds every E4M3 value exactly, so the codes are widened to f16 on their way:
//   warps 0-7   softmax; at a unit's start each thread turns its query row from bf16 to
//               f16 in place, divided by a power of two so that any magnitude fits;
//   warp 8      producer: TMA of a tile's eight pages into a staging buffer, a byte a value;
//   warp 9      tcgen05.mma issuer and TMEM owner;
//   warps 10-11 converters: 16 codes at a time from the staging buffer to f16 in the
//               128-byte swizzled tiles that the MMAs read.  V pages are channel-major, so
//               V is a K-major operand; tokens past the context become zeros here.
// The block scales never touch the operands.  Both are powers of two: a key block's
// multiplies its 16 columns of scores (one factor per 16 columns in the softmax's
// multiply-add), a value block's goes into the exponent, w = x + ev: P = 2^(w - m) with
// m the running maximum of w, and the row sum takes 2^-ev times each group's sum.
#include <algorithm>

#include "cache_scaled.cuh"

namespace fa {

constexpr int kT8Threads = 384;
constexpr int kT8Producer = 8, kT8Mma = 9, kT8Convert = 10, kT8Converters = 2;
constexpr int kT8Rows = 128;
constexpr int kT8Units = 4;                     // mailboxes
constexpr int kT8Readers = 9 + kT8Converters;   // their readers
constexpr int kT8Scales = 4;                    // tiles whose block scales are kept
constexpr float kT8Rescale = 14.f;  // growth of a maximum that moves it: weights up to 2^14 still fit f16

template <int D>
struct T8Cfg {
    static constexpr int kAtoms = D / 64;
    static constexpr int kAtomBytes = kT8Rows * 128;
    static constexpr int kTileBytes = kAtoms * kAtomBytes;  // f16 tile of Q, K or V
    static constexpr int kStageBytes = kT8Rows * D;         // the same as codes
    static constexpr int kStages = 4, kStaging = 2;
    static constexpr int kBars = 2 * kStages + 2 * kStaging + 2 * 7 + 2 + 2 * kT8Units;
    static constexpr int kSmem = 1024 + 2 * kTileBytes + kStages * kTileBytes + kStaging * kStageBytes +
                                 kT8Scales * 24 * 4 + kBars * 8 + 16 + 4 * kT8Units;
    static constexpr uint32_t kS0 = 0, kS1 = 128, kO0 = 256, kO1 = 256 + D;
};
static_assert(T8Cfg<128>::kSmem <= 227 * 1024, "shared memory of a CTA");

struct T8Params {
    int Hq, Hkv, g, causal, pair_heads, pack, pack_shift, per_rank, per_head, mbps, num_blocks, total_q;
    FastDiv div_rank, div_head;
    float scale_log2;
    uint16_t* out;
    float* lse;
    const uint8_t *ke, *ve;
    const int32_t *bt, *ctx_lens, *q_lens, *q_start;
    const int32_t* work_count;
    const int4* pieces;  // (sequence, first query token, first | end << 16 of its KV tiles, place of its partial results or -1)
    float4* part_o;      // partial results: [d / 4][256 rows] each
    float2* part_ml;
    DevCtx ctx;
};

struct T8Unit {
    int seq, hk, head[2], row0[2], nrows[2], qtok[2];
    int kv_len, pos_off, kt0, n_kt, slot;
};
__device__ __forceinline__ int pick(const int (&a)[2], int s) { return s ? a[1] : a[0]; }

__device__ __forceinline__ T8Unit t8_unit(const T8Params& p, int u) {
    T8Unit U;
    const int e = p.div_rank(u), rest = u - e * p.per_rank;
    const int4 piece = __ldg(p.pieces + e);
    const int ql = __ldg(p.q_lens + piece.x), cl = __ldg(p.ctx_lens + piece.x);
    int qs = __ldg(p.q_start + piece.x), rows = ql;
    if (!rows_fit(qs, ql, p.total_q)) qs = rows = 0;  // (reported by the metadata kernel; nothing is written)
    U.seq = piece.x;
    int tokens = kT8Rows;
    if (p.pack) {  // 128 / g tokens x the heads of kv head `rest`'s group
        tokens = kT8Rows >> p.pack_shift;
        U.hk = rest;
        U.head[0] = U.head[1] = rest * p.g;
        U.row0[0] = piece.y;
        U.row0[1] = piece.y + tokens;
    } else if (p.pair_heads) {
        U.hk = p.div_head(rest);
        U.head[0] = U.hk * p.g + 2 * (rest - U.hk * p.per_head);
        U.head[1] = U.head[0] + 1;
        U.row0[0] = U.row0[1] = piece.y;
    } else {
        U.head[0] = U.head[1] = rest;
        U.hk = p.div_head(rest);
        U.row0[0] = piece.y;
        U.row0[1] = piece.y + kT8Rows;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        U.nrows[s] = max(0, min(tokens, rows - U.row0[s]));
        U.qtok[s] = qs + U.row0[s];
    }
    U.kv_len = cl;
    U.pos_off = cl - ql;
    U.kt0 = piece.z & 0xffff;
    U.n_kt = (int)((unsigned)piece.z >> 16);
    U.slot = piece.w < 0 ? -1 : piece.w + rest;
    return U;
}

// Instruction descriptor, f16 operands (both K-major), fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// This thread's TMEM row of D fp32 columns times alpha.
template <int D>
__device__ __noinline__ void t8_scale_row(uint32_t taddr, float alpha) {
    __syncwarp();  // warp-collective TMEM accesses follow
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(taddr + c * 32, o);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
        tmem_st32(taddr + c * 32, o);
    }
    tmem_wait_st();
}

// A piece's row for the join kernel: O / l, four channels of 256 rows side by side, and (max, sum).
template <int D>
__device__ __noinline__ void t8_partial_row(uint32_t taddr, float4* o, float2* ml, float m, float l) {
    const float inv = l > 0.f ? 1.f / l : 0.f;
    __syncwarp();
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
        uint32_t raw[32];
        tmem_ld32(taddr + c * 32, raw);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j)
            o[(c * 8 + j) * 2 * kT8Rows] =
                make_float4(__uint_as_float(raw[4 * j]) * inv, __uint_as_float(raw[4 * j + 1]) * inv,
                            __uint_as_float(raw[4 * j + 2]) * inv, __uint_as_float(raw[4 * j + 3]) * inv);
    }
    *ml = make_float2(m, l);
}

__device__ __forceinline__ void st_shared(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Turns row r of a query tile (128-byte swizzled atoms of 64 channels) from bf16 to f16 in
// place, divided by a power of two that brings its largest magnitude below 2; returns
// that power.
template <int D>
__device__ __forceinline__ float t8_turn_row(uint8_t* tile, int r) {
    using C = T8Cfg<D>;
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        const uint4 w = *reinterpret_cast<const uint4*>(tile + (c >> 3) * C::kAtomBytes + sw128_offset(r, c & 7));
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(v[i] & 0x7fffu, (v[i] >> 16) & 0x7fffu));
    }
    const int e = top == 0 ? 0 : min(126, max(-126, (int)(top >> 7) - 127));
    const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
        uint4* at = reinterpret_cast<uint4*>(tile + (c >> 3) * C::kAtomBytes + sw128_offset(r, c & 7));
        const uint4 w = *at;
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = pack_f16x2(__uint_as_float(v[i] << 16) * f, __uint_as_float(v[i] & 0xFFFF0000u) * f);
        *at = make_uint4(h[0], h[1], h[2], h[3]);
    }
    return __uint_as_float((uint32_t)(127 + e) << 23);
}

__device__ __forceinline__ bool t8_wait_sleepy(uint64_t* bar, uint32_t parity, unsigned long long limit_ns, volatile int* abort) {
    bool done = mbar_try_wait(bar, parity);
    if (!done) {
        const uint64_t t0 = globaltimer_ns();
        while (!done) {
            if (*abort || globaltimer_ns() - t0 > limit_ns) break;
            __nanosleep(100);
            done = mbar_try_wait(bar, parity);
        }
    }
    return __all_sync(0xffffffffu, done);
}

template <int D>
__global__ void __launch_bounds__(kT8Threads, 1)
    attn_tc8_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ T8Params p) {
    using C = T8Cfg<D>;
    constexpr int S = C::kStages, G8 = C::kStaging;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* qbuf = smem;
    uint8_t* ring = qbuf + 2 * C::kTileBytes;
    uint8_t* staging = ring + S * C::kTileBytes;
    float* scales = reinterpret_cast<float*>(staging + G8 * C::kStageBytes);  // [kT8Scales][8 key factors, 8 value exponents, 8 times 2^-exponent]
    uint64_t* full = reinterpret_cast<uint64_t*>(scales + kT8Scales * 24);
    uint64_t* empty = full + S;
    uint64_t* sfill = empty + S;      // [2] staging: codes have landed
    uint64_t* sfree = sfill + G8;     // [2] and are converted
    uint64_t* qfull = sfree + G8;     // [2]
    uint64_t* qready = qfull + 2;     // [2] turned to f16
    uint64_t* qempty = qready + 2;    // [2]
    uint64_t* sfull = qempty + 2;     // [2]
    uint64_t* pfull = sfull + 2;      // [slot * 2 + half]; the MMA warp waits on half 1, signalled after half 0
    uint64_t* ofull = pfull + 4;      // [2]
    uint64_t* drain = ofull + 2;
    uint64_t* never = drain + 1;  // nothing arrives on it (forced time-out test hook)
    uint64_t* ufull = never + 1;
    uint64_t* uempty = ufull + kT8Units;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(uempty + kT8Units);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* umbox = abort_flag + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], kT8Converters);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < G8; ++i) {
            mbar_init(&sfill[i], 1);
            mbar_init(&sfree[i], kT8Converters);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&qfull[s], 1);
            mbar_init(&qready[s], kT8Rows);
            mbar_init(&qempty[s], 1);
            mbar_init(&sfull[s], 1);
            mbar_init(&pfull[2 * s], kT8Rows);
            mbar_init(&pfull[2 * s + 1], kT8Rows);
            mbar_init(&ofull[s], 1);
        }
        mbar_init(drain, 1);
        mbar_init(never, 1);
        for (int k = 0; k < kT8Units; ++k) {
            mbar_init(&ufull[k], 1);
            mbar_init(&uempty[k], kT8Readers);
        }
        *abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
    }
    // (the join kernel that may follow waits for this grid's end before it reads)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == kT8Mma) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    const int num_units = __ldg(p.work_count) * p.per_rank;
    const int G = gridDim.x;
    const unsigned long long lim_ns = p.ctx.wait_ns;
    bool ok = !p.ctx.force_timeout || mbar_wait_warp(never, 0, lim_ns, abort_flag);
    // the i-th unit of this CTA as the readers see it (false: the wait gave up)
    auto read_unit = [&](int i, int& u) -> bool {
        const int k = i % kT8Units;
        if (!mbar_wait_warp(&ufull[k], (i / kT8Units) & 1, lim_ns, abort_flag)) return false;
        int v = 0;
        if (lane == 0) {
            v = umbox[k];
            mbar_arrive(&uempty[k]);
        }
        u = __shfl_sync(0xffffffffu, v, 0);
        return true;
    };

    if (warp == kT8Producer) {
        // ================================================== TMA producer ====
        int fill = 0, q_loads = 0, tiles = 0;  // (query loads: slots by turns)
        for (int i = 0; ok; ++i) {
            // the first unit is this CTA's own, then the next in the longest-first order that no CTA has taken
            int v = -1;
            if (lane == 0) {
                if (i == 0) {
                    v = (int)blockIdx.x < num_units ? (int)blockIdx.x : -1;
                } else {
                    const int t = atomicAdd(const_cast<int32_t*>(p.work_count) + 1, 1);
                    v = t < num_units - G ? G + t : -1;
                }
            }
            const int u = __shfl_sync(0xffffffffu, v, 0), k = i % kT8Units;
            if (i >= kT8Units && !mbar_wait_warp(&uempty[k], ((i / kT8Units) - 1) & 1, lim_ns, abort_flag)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                umbox[k] = u;
                mbar_arrive(&ufull[k]);
            }
            __syncwarp();
            if (u < 0) break;
            const T8Unit U = t8_unit(p, u);
            if (U.kt0 >= U.n_kt) continue;
            for (int s = 0; s < 2 && ok; ++s) {
                if (!t8_wait_sleepy(&qempty[s], ((q_loads >> 1) & 1) ^ 1, lim_ns, abort_flag)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&qfull[s], C::kTileBytes);
#pragma unroll
                    for (int a = 0; a < C::kAtoms; ++a)
                        tma_load_4d(qbuf + s * C::kTileBytes + a * C::kAtomBytes, &tm_q, &qfull[s], a * 64, pick(U.head, s),
                                    pick(U.qtok, s), 0);
                }
                __syncwarp();
                ++q_loads;
            }
            if (!ok) break;
            // lane j < 8: the tile's j-th block.  Blocks are looked up two tiles ahead, scales one.
            auto load_blk = [&](int kt) -> int {
                const int lb = kt * 8 + lane;
                if (lane >= 8 || kt >= U.n_kt || lb * kScaledBlock >= U.kv_len) return p.num_blocks;  // the copy fills zeros
                const int b = __ldg(p.bt + (long)U.seq * p.mbps + lb);
                return b;
            };
            auto load_exps = [&](int blk) -> int {
                if (blk < 0 || blk >= p.num_blocks) return kExpBias | kExpBias << 8;
                const long at = (long)blk * p.Hkv + U.hk;
                return __ldg(p.ke + at) | __ldg(p.ve + at) << 8;
            };
            int blk = load_blk(U.kt0), blk_next = load_blk(U.kt0 + 1);
            int exps = load_exps(blk);
            for (int kt = U.kt0; kt < U.n_kt && ok; ++kt) {
                const int blk_after = load_blk(kt + 2), exps_next = load_exps(blk_next);
                int at = blk;
                if (at < 0 || at > p.num_blocks || (at == p.num_blocks && lane < 8 && (kt * 8 + lane) * kScaledBlock < U.kv_len)) {
                    raise_error(p.ctx, ERR_BOUNDS_BIT);
                    at = p.num_blocks;
                }
                for (int which = 0; which < 2; ++which) {  // 0: K tile, 1: V tile
                    const int st = fill % G8;
                    if (!t8_wait_sleepy(&sfree[st], ((fill / G8) & 1) ^ 1, lim_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (which == 0 && lane < 8) {
                        // (this tile's place held scales of four tiles ago, whose softmax is done: its K tile's
                        // place in the ring was taken again since)
                        float* sc = scales + (tiles % kT8Scales) * 24;
                        sc[lane] = scale_of(exps & 255);
                        sc[8 + lane] = (float)((exps >> 8) - kExpBias);
                        sc[16 + lane] = scale_of(2 * kExpBias - (exps >> 8));
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive_expect_tx(&sfill[st], C::kStageBytes);
                    __syncwarp();
                    if (lane < 8)
                        tma_load_4d(staging + st * C::kStageBytes + lane * kScaledBlock * D, which ? &tm_v : &tm_k, &sfill[st], 0,
                                    0, U.hk, at);
                    __syncwarp();
                    ++fill;
                }
                ++tiles;
                blk = blk_next;
                blk_next = blk_after;
                exps = exps_next;
            }
        }
        if (!ok) {
            if (lane == 0) {
                raise_error(p.ctx, ERR_TIMEOUT_BIT);
                *abort_flag = 1;
            }
            // let every copy already issued land before the CTA can exit
            for (int f = max(0, fill - G8); f < fill; ++f)
                (void)mbar_wait_warp(&sfill[f % G8], (f / G8) & 1, 1000000000ull, nullptr);
            for (int f = max(0, q_loads - 2); f < q_loads; ++f)
                (void)mbar_wait_warp(&qfull[f & 1], (f >> 1) & 1, 1000000000ull, nullptr);
        }
    } else if (warp >= kT8Convert) {
        // ===================================================== converters ===
        const int t = threadIdx.x - kT8Convert * 32;
        constexpr int kThreads = kT8Converters * 32;
        int n = 0;  // tiles (K and V) converted
        auto widen = [](const uint4& w, uint4& a, uint4& b) {
            e4m3x4_to_f16x4(w.x, a.x, a.y);
            e4m3x4_to_f16x4(w.y, a.z, a.w);
            e4m3x4_to_f16x4(w.z, b.x, b.y);
            e4m3x4_to_f16x4(w.w, b.z, b.w);
        };
        for (int i = 0; ok; ++i) {
            int u;
            if (!read_unit(i, u)) {
                ok = false;
                break;
            }
            if (u < 0) break;
            const T8Unit U = t8_unit(p, u);
            for (int kt = U.kt0; kt < U.n_kt && ok; ++kt) {
                for (int which = 0; which < 2; ++which, ++n) {
                    const int st = n % G8, stage = n % S;
                    if (!mbar_wait_warp(&sfill[st], (n / G8) & 1, lim_ns, abort_flag) ||
                        !mbar_wait_warp(&empty[stage], ((n / S) & 1) ^ 1, lim_ns, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint8_t* src = staging + st * C::kStageBytes;
                    uint8_t* dst = ring + stage * C::kTileBytes;
                    // Piece k of 16 codes is this thread's x = t + 64 k.  Eight are loaded before the first is stored (the
                    // compiler cannot tell the two buffers apart); every address is a base plus a constant.
                    constexpr int kPieces = kT8Rows * D / 16 / kThreads, kAhead = 8;
                    const int left = U.kv_len - kt * kT8Rows;  // tokens of the tile that exist
                    const uint8_t* from = src + t * 16;
#pragma unroll
                    for (int k0 = 0; k0 < kPieces; k0 += kAhead) {
                        uint4 w[kAhead];
#pragma unroll
                        for (int k = 0; k < kAhead; ++k) w[k] = *reinterpret_cast<const uint4*>(from + (k0 + k) * kThreads * 16);
                        if (which == 0) {
                            // token t / kPer + k * kStep, piece t % kPer of its row (k moves whole groups of eight rows).  The
                            // second atom's pieces store their halves in the other order: eight lanes, eight bank groups.
                            constexpr uint32_t kPer = D / 16, kStep = kThreads / kPer;
                            static_assert(kStep % 8 == 0, "the swizzle is the same for every k");
                            const uint32_t tok = (uint32_t)t / kPer, c = (uint32_t)t % kPer, c0 = 2 * (c & 3), swap = c >> 2;
                            uint8_t* atom = dst + swap * C::kAtomBytes;
                            uint8_t *to0 = atom + sw128_offset(tok, c0 + swap), *to1 = atom + sw128_offset(tok, c0 + 1 - swap);
#pragma unroll
                            for (int k = 0; k < kAhead; ++k) {
                                uint4 a, b;
                                widen(w[k], a, b);
                                *reinterpret_cast<uint4*>(to0 + (k0 + k) * kStep * 128) = swap ? b : a;
                                *reinterpret_cast<uint4*>(to1 + (k0 + k) * kStep * 128) = swap ? a : b;
                            }
                        } else {
                            constexpr int kPerPage = D / kThreads;  // a thread's pieces of a page: channels t, t + 64
                            if (left < kT8Rows) {                   // whatever is stored behind the last token counts as zeros
#pragma unroll
                                for (int k = 0; k < kAhead; ++k) {
                                    const int have = left - (k0 + k) / kPerPage * kScaledBlock;
                                    auto cut = [&](uint32_t v, int q) {
                                        const int h = have - 4 * q;
                                        return h >= 4 ? v : (h <= 0 ? 0u : v & ((1u << (8 * h)) - 1));
                                    };
                                    w[k] = make_uint4(cut(w[k].x, 0), cut(w[k].y, 1), cut(w[k].z, 2), cut(w[k].w, 3));
                                }
                            }
                            const uint32_t row = smem_u32(dst) + t * 128 + ((t & 7) << 4);  // chunk 0 of channel t, swizzled
#pragma unroll
                            for (int k = 0; k < kAhead; ++k) {
                                const int page = (k0 + k) / kPerPage, far = (k0 + k) % kPerPage;
                                uint4 a, b;
                                widen(w[k], a, b);
                                const uint32_t at = row + (page >> 2) * (D * 128) + far * kThreads * 128;
                                st_shared(at ^ (2 * (page & 3)) << 4, a);
                                st_shared(at ^ (2 * (page & 3) + 1) << 4, b);
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&full[stage]);
                        mbar_arrive(&sfree[st]);
                    }
                    __syncwarp();
                }
            }
        }
        if (!ok && lane == 0) {
            raise_error(p.ctx, ERR_TIMEOUT_BIT);
            *abort_flag = 1;
        }
    } else if (warp == kT8Mma) {
        // ===================================================== MMA issuer ===
        constexpr uint32_t kIdescQK = idesc_f16_f32(128, 128), kIdescPV = idesc_f16_f32(128, D);
        const uint32_t q_addr = smem_u32(qbuf), ring_addr = smem_u32(ring);
        int cons = 0, ucnt = 0, pc[2] = {0, 0};
        auto issue_qk = [&](int s, int kidx) {
            const uint64_t kd = smem_desc_sw128(ring_addr + (kidx % S) * C::kTileBytes, 16, 1024);
            const uint64_t qd = smem_desc_sw128(q_addr + s * C::kTileBytes, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * C::kAtomBytes + (kk & 3) * 32) >> 4;
                umma_ss(tbase + (s ? C::kS1 : C::kS0), qd + off, kd + off, kIdescQK, kk > 0);
            }
        };
        auto pv = [&](int s, int vidx, bool acc_first) -> bool {
            if (!mbar_wait_warp(&pfull[2 * s + 1], (s ? pc[1] : pc[0]) & 1, lim_ns, abort_flag)) return false;
            tc_fence_after();
            if (lane == 0) {
                const uint64_t vd = smem_desc_sw128(ring_addr + (vidx % S) * C::kTileBytes, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {  // 16 keys each; a half of 64 keys is D rows of 128 bytes
                    const uint32_t off = ((kk >> 2) * (D * 128) + (kk & 3) * 32) >> 4;
                    umma_ts(tbase + (s ? C::kO1 : C::kO0), tbase + (s ? C::kS1 : C::kS0) + kk * 8, vd + off, kIdescPV,
                            acc_first || kk > 0);
                }
            }
            __syncwarp();
            if (s) ++pc[1];
            else ++pc[0];
            return true;
        };
        for (int i = 0; ok; ++i) {
            int u;
            if (!read_unit(i, u)) {
                ok = false;
                break;
            }
            if (u < 0) break;
            const T8Unit U = t8_unit(p, u);
            if (U.kt0 >= U.n_kt) continue;
            for (int s = 0; s < 2; ++s)
                if (!t8_wait_sleepy(&qready[s], ucnt & 1, lim_ns, abort_flag)) ok = false;
            if (!ok) break;
            ++ucnt;
            tc_fence_after();
            const int n = U.n_kt - U.kt0;
            for (int it = 0; it < n && ok; ++it) {
                const int kidx = cons + 2 * it, prev_v = kidx - 1;
                for (int s = 0; s < 2 && ok; ++s) {
                    if (it > 0) {
                        if (s == 0 && !mbar_wait_warp(&full[prev_v % S], (prev_v / S) & 1, lim_ns, abort_flag)) ok = false;
                        if (!ok || !pv(s, prev_v, it > 1)) {
                            ok = false;
                            break;
                        }
                    }
                    if (s == 0) {
                        if (!mbar_wait_warp(&full[kidx % S], (kidx / S) & 1, lim_ns, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                    }
                    if (lane == 0) {
                        issue_qk(s, kidx);
                        umma_commit(&sfull[s]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (lane == 0) {
                    umma_commit(&empty[kidx % S]);
                    if (it > 0) umma_commit(&empty[prev_v % S]);
                }
                __syncwarp();
            }
            if (!ok) break;
            const int last_v = cons + 2 * n - 1;
            if (lane == 0) {
                umma_commit(&qempty[0]);
                umma_commit(&qempty[1]);
            }
            if (!mbar_wait_warp(&full[last_v % S], (last_v / S) & 1, lim_ns, abort_flag)) {
                ok = false;
                break;
            }
            for (int s = 0; s < 2 && ok; ++s) {
                if (!pv(s, last_v, n > 1)) {
                    ok = false;
                    break;
                }
                if (lane == 0) umma_commit(&ofull[s]);
                __syncwarp();
            }
            if (!ok) break;
            if (lane == 0) umma_commit(&empty[last_v % S]);
            __syncwarp();
            cons += 2 * n;
        }
        if (!ok && lane == 0) {
            raise_error(p.ctx, ERR_TIMEOUT_BIT);
            *abort_flag = 1;
        }
        // every MMA issued above completes before TMEM is released
        if (lane == 0) umma_commit(drain);
        __syncwarp();
        (void)mbar_wait_bounded(drain, 0, 1000000000ull, nullptr);
    } else {
        // ======================================================== softmax ===
        const int s = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t trow = tbase + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_col = s ? C::kS1 : C::kS0, o_col = s ? C::kO1 : C::kO0;
        int sc = 0, uc = 0, tiles = 0;
        for (int i = 0; ok; ++i) {
            int u;
            if (!read_unit(i, u)) {
                ok = false;
                break;
            }
            if (u < 0) break;
            const T8Unit U = t8_unit(p, u);
            if (U.kt0 >= U.n_kt) continue;
            // query token of this thread's row, and its head within a packed slot
            const int tok = p.pack ? r >> p.pack_shift : r, hl = p.pack ? r & (p.g - 1) : 0;
            const int row = pick(U.row0, s) + tok;
            const int vis_end = p.causal ? min(U.kv_len, row + U.pos_off + 1) : U.kv_len;
            if (!mbar_wait_warp(&qfull[s], uc & 1, lim_ns, abort_flag)) {
                ok = false;
                break;
            }
            const float mul = p.scale_log2 * t8_turn_row<D>(qbuf + s * C::kTileBytes, r);
            fence_proxy_async_smem();
            mbar_arrive(&qready[s]);
            float m = -INFINITY, l = 0.f;
            for (int kt = U.kt0; kt < U.n_kt; ++kt, ++tiles) {
                if (!mbar_wait_warp(&sfull[s], sc & 1, lim_ns, abort_flag)) {
                    ok = false;
                    break;
                }
                ++sc;
                tc_fence_after();
                const int vlim = vis_end - kt * kT8Rows;  // visible columns: [0, vlim)
                const bool plain = __all_sync(0xffffffffu, vlim >= kT8Rows);
                const float4* sv = reinterpret_cast<const float4*>(scales + (tiles % kT8Scales) * 24);
                // pass 1: the largest w = s mul 2^ks + ev, a block's 16 columns at a time
                float mx = -INFINITY;
                {
                    uint32_t raw[kT8Rows];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32(trow + s_col + c * 32, *reinterpret_cast<uint32_t(*)[32]>(raw + 32 * c));
                    tmem_wait_ld();
                    float gm[8];
#pragma unroll
                    for (int b = 0; b < 8; ++b) gm[b] = -INFINITY;
                    // (group after group in turn: eight independent chains)
                    if (plain) {
#pragma unroll
                        for (int j = 0; j < kT8Rows / 2; ++j) {
                            const int b = j & 7, c = 16 * b + 2 * (j >> 3);
                            gm[b] = fmax3f(gm[b], __uint_as_float(raw[c]), __uint_as_float(raw[c + 1]));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < kT8Rows / 2; ++j) {
                            const int b = j & 7, c = 16 * b + 2 * (j >> 3);
                            gm[b] = fmax3f(gm[b], c < vlim ? __uint_as_float(raw[c]) : -INFINITY,
                                           c + 1 < vlim ? __uint_as_float(raw[c + 1]) : -INFINITY);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float4 kf = sv[h], va = sv[2 + h];
                        const float k4[4] = {kf.x, kf.y, kf.z, kf.w}, v4[4] = {va.x, va.y, va.z, va.w};
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const float x = gm[4 * h + b];
                            mx = fmaxf(mx, x == -INFINITY ? x : fmaf(x, mul * k4[b], v4[b]));
                        }
                    }
                }
                const float m_new = fmaxf(m, mx);
                const bool warp_rescale = __any_sync(0xffffffffu, m_new > m + kT8Rescale);
                float alpha = 1.f;
                if (warp_rescale) {
                    alpha = m == -INFINITY ? 0.f : fast_exp2(m - m_new);
                    l *= alpha;
                    m = m_new;
                }
                const float m_use = m == -INFINITY ? 0.f : m;
                const bool rescale_o = warp_rescale && kt > U.kt0;
                // pass 2: P = 2^(w - m) as f16, each half of the columns signalled as soon as it is stored
                // (with a rescale of O, both behind it)
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t raw[64];
                    tmem_ld32(trow + s_col + h * 64, *reinterpret_cast<uint32_t(*)[32]>(raw));
                    tmem_ld32(trow + s_col + h * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(raw + 32));
                    const float4 kf = sv[h], va = sv[2 + h], vb = sv[4 + h];
                    const float k4[4] = {kf.x, kf.y, kf.z, kf.w}, v4[4] = {va.x, va.y, va.z, va.w}, b4[4] = {vb.x, vb.y, vb.z, vb.w};
                    float2 f2[4], add2[4], sum[4];
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        f2[b] = both(mul * k4[b]);
                        add2[b] = both(v4[b] - m_use);
                        sum[b] = make_float2(0.f, 0.f);
                    }
                    tmem_wait_ld();
                    uint32_t pk[32];
                    if (plain) {
#pragma unroll
                        for (int j0 = 0; j0 < 32; ++j0) {
                            const int b = j0 & 3, j = 8 * b + (j0 >> 2);
                            const float2 x =
                                __ffma2_rn(make_float2(__uint_as_float(raw[2 * j]), __uint_as_float(raw[2 * j + 1])), f2[b], add2[b]);
                            const float2 pp = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                            sum[b] = __fadd2_rn(sum[b], pp);
                            pk[j] = pack_f16x2(pp.x, pp.y);
                        }
                    } else {
#pragma unroll
                        for (int j0 = 0; j0 < 32; ++j0) {
                            const int b = j0 & 3, j = 8 * b + (j0 >> 2), c = h * 64 + 2 * j;
                            const float2 x =
                                __ffma2_rn(make_float2(__uint_as_float(raw[2 * j]), __uint_as_float(raw[2 * j + 1])), f2[b], add2[b]);
                            const float2 pp = make_float2(c < vlim ? fast_exp2(x.x) : 0.f, c + 1 < vlim ? fast_exp2(x.y) : 0.f);
                            sum[b] = __fadd2_rn(sum[b], pp);
                            pk[j] = pack_f16x2(pp.x, pp.y);
                        }
                    }
#pragma unroll
                    for (int b = 0; b < 4; ++b) l = fmaf(sum[b].x + sum[b].y, b4[b], l);  // 2^-ev
                    tmem_st32(trow + s_col + h * 32, pk);
                    if (!rescale_o) {
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(&pfull[2 * s + h]);
                    }
                }
                if (rescale_o) {
                    t8_scale_row<D>(trow + o_col, alpha);
                    tc_fence_before();
                    mbar_arrive(&pfull[2 * s]);
                    mbar_arrive(&pfull[2 * s + 1]);
                }
            }
            if (!ok) break;
            const T8Unit E = t8_unit(p, u);  // derived again: its fields are not live across the tile loop
            if (!mbar_wait_warp(&ofull[s], uc & 1, lim_ns, abort_flag)) {
                ok = false;
                break;
            }
            ++uc;
            tc_fence_after();
            if (E.slot >= 0) {  // a piece of the keys: the join kernel puts the pieces together
                const int at = s * kT8Rows + r;
                t8_partial_row<D>(trow + o_col, p.part_o + (long)E.slot * (D / 4) * 2 * kT8Rows + at,
                                  p.part_ml + (long)E.slot * 2 * kT8Rows + at, m, l);
                tc_fence_before();  // (the next unit's MMAs write O again)
                continue;
            }
            const bool valid = tok < pick(E.nrows, s);
            const long orow = ((long)pick(E.qtok, s) + tok) * p.Hq + pick(E.head, s) + hl;
            const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                uint32_t raw[64];
                tmem_ld32(trow + o_col + c * 64, *reinterpret_cast<uint32_t(*)[32]>(raw));
                tmem_ld32(trow + o_col + c * 64 + 32, *reinterpret_cast<uint32_t(*)[32]>(raw + 32));
                tmem_wait_ld();
                uint32_t pk[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    pk[j] = pack_bf16x2(__uint_as_float(raw[2 * j]) * inv, __uint_as_float(raw[2 * j + 1]) * inv);
                if (valid) {
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4)
                        st_global_v8(p.out + orow * D + c * 64 + q4 * 16, pk[8 * q4], pk[8 * q4 + 1], pk[8 * q4 + 2],
                                     pk[8 * q4 + 3], pk[8 * q4 + 4], pk[8 * q4 + 5], pk[8 * q4 + 6], pk[8 * q4 + 7]);
                }
            }
            if (p.lse && valid) p.lse[orow] = l > 0.f ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
            tc_fence_before();
        }
        if (!ok && lane == 0) {
            raise_error(p.ctx, ERR_TIMEOUT_BIT);
            *abort_flag = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kT8Mma) tmem_dealloc(tbase, 512);
}

template <int D>
static fa_status launch_tc8(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const T8Params& p, cudaStream_t s) {
    auto kernel = attn_tc8_kernel<D>;
    const fa_status st = raise_dynamic_smem(reinterpret_cast<const void*>(kernel), T8Cfg<D>::kSmem);
    if (st != FA_OK) return st;
    kernel<<<sm_count(), kT8Threads, T8Cfg<D>::kSmem, s>>>(tq, tk, tv, p);
    return cuda_status(cudaGetLastError());
}

fa_status launch_paged_prefill_fp8(const void* q, const void* k_cache, const void* v_cache, const uint8_t* k_exp,
                                   const uint8_t* v_exp, const int32_t* block_table, const int32_t* ctx_lens,
                                   const int32_t* q_lens, const int32_t* q_start, const int32_t* work_count, void* out,
                                   float* lse, int mbps, int num_blocks, int Hq, int Hkv, int d, int causal, float scale,
                                   int total_q, const int4* pieces, float4* part_o, float2* part_ml, cudaStream_t s,
                                   const DevCtx& ctx) {
    CUtensorMap tq, tk, tv;
    fa_status st = paged_query_map(&tq, q, Hq, Hkv, d, total_q);
    if (st != FA_OK) return st;
    // a box a page of 16 d bytes, landing as it is, in rows of 128 bytes
    const uint64_t page = (uint64_t)kScaledBlock * d;
    const uint64_t dims[4] = {128, page / 128, (uint64_t)Hkv, (uint64_t)num_blocks}, strides[3] = {128, page, Hkv * page};
    const uint32_t box[4] = {128, (uint32_t)(page / 128), 1, 1};
    st = encode_tmap_4d(&tk, k_cache, dims, strides, box, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (st == FA_OK)
        st = encode_tmap_4d(&tv, v_cache, dims, strides, box, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (st != FA_OK) return st;
    T8Params p{};
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.g = Hq / Hkv;
    p.causal = causal ? 1 : 0;
    p.pair_heads = p.g % 2 == 0 ? 1 : 0;
    p.pack = paged_tc_pack(p.g) ? 1 : 0;
    p.pack_shift = p.pack ? __builtin_ctz((unsigned)p.g) : 0;
    p.per_head = p.pair_heads ? p.g / 2 : p.g;
    p.per_rank = Hkv * (p.pack ? 1 : p.per_head);
    p.div_rank = FastDiv(p.per_rank);
    p.div_head = FastDiv(p.per_head);
    p.mbps = mbps;
    p.num_blocks = num_blocks;
    p.total_q = total_q;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.ke = k_exp;
    p.ve = v_exp;
    p.bt = block_table;
    p.ctx_lens = ctx_lens;
    p.q_lens = q_lens;
    p.q_start = q_start;
    p.work_count = work_count;
    p.pieces = pieces;
    p.part_o = part_o;
    p.part_ml = part_ml;
    p.ctx = ctx;
    return d == 128 ? launch_tc8<128>(tq, tk, tv, p, s) : launch_tc8<64>(tq, tk, tv, p, s);
}

}  // namespace fa
