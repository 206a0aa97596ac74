// For each query and kv head the cache blocks whose keys can matter most to it
// (fa_block_select).
//
// A block's keys lie in the box of its channel bounds [lo, hi], so the largest score
// that any of them can have with query q is
//     u = sum_c max(q_c lo_c, q_c hi_c) = q+ . hi + q- . lo,
// q+ = max(q, 0), q- = min(q, 0): two dot products, of which a score kernel makes
// m16n8k16 warp MMAs (rows: the queries' heads, columns: 8 blocks).  A block counts as
// much as it does for the head of the group that wants it most.
//
// block_score_kernel lays the steps of 32 blocks of all (sequence, kv head, set of query
// tiles) end to end and gives each CTA of one wave an equal run of them, so that contexts
// of any mix of lengths fill the GPU.  A producer warp looks a step's blocks up, a lane
// each, and copies their bounds (4 d bytes a block) into a ring in shared memory; four
// warps take eight of its blocks each for one tile, or, when a sequence has four tiles or
// more, all of them for a tile each, so that they are read once for four tiles.  The MMA's
// K dimension is taken in an order in which a lane's B operands are 16 consecutive
// bytes of a block's row.  Memory bound for single tokens.
//
// block_top_kernel, a CTA a row, finds the border with a histogram over the scores' own
// range (again within the bin that holds the border, if that is full).  An MMA's sum is off
// by its roundings, which must not decide: blocks whose score lies within the
// rounding bound of the border are summed again in twice fp32's digits and ordered by
// that, equal ones by their number, so that the choice is that of exact
// arithmetic.  Few blocks are that close (a handful of thousands), unless many are equal.
#include <algorithm>
#include <type_traits>

#include "cache_scaled.cuh"

namespace fa {

constexpr int kScWarps = 4, kScCtasPerSm = 3;  // warps beside the producer
constexpr int kScBlocks = 32, kScStages = 4;   // blocks of a step, steps of the ring

constexpr int kTopItems = 16;     // scores per thread that stay in registers
constexpr int kTopBins = 1024;
constexpr int kTopNear = 256;     // blocks near the border that are ranked in shared memory, by counting
constexpr int kTopCtas = 8 * 160;   // grid of the top kernel at most, and its scratch
constexpr int kTopFew = 512, kTopMany = 128;  // threads of a row's CTA when there are few rows (latency), and many

struct SelectArgs {
    const uint16_t *q, *bounds;
    const int32_t *bt, *ctx_lens, *q_lens;
    float* scores;   // [total_q][Hkv][mbps]
    float* largest;  // [num_seqs][Hkv][mbps]: a block's largest |bound|
    int32_t* near_b;   // per CTA of the top kernel: blocks near the border
    unsigned long long* near_key;  // and their keys
    int32_t* sel;
    int num_seqs, mbps, num_blocks, total_q, Hq, Hkv, keep, recent, sink;
    int g2_log, per;  // rows that a token's heads take in a tile (log2), tokens a tile
    int many;         // some sequence may have kScWarps tiles or more
    DevCtx ctx;
};

__device__ __forceinline__ uint32_t min0_bf16x2(uint32_t x) {
    const __nv_bfloat162 z = __floats2bfloat162_rn(0.f, 0.f);
    const __nv_bfloat162 v = __hmin2(*reinterpret_cast<const __nv_bfloat162*>(&x), z);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t max0_bf16x2(uint32_t x) {
    const __nv_bfloat162 z = __floats2bfloat162_rn(0.f, 0.f);
    const __nv_bfloat162 v = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&x), z);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int D>
struct ScoreSmem {
    static constexpr int kRow = 4 * D + 64;  // bytes between blocks: two neighbours' 64 bytes lie in different banks
    static constexpr int kStage = kScBlocks * kRow;
    static constexpr int kBytes = kScStages * kStage + (2 * kScStages + 1) * 8 + 16;
};

// A tile's rows: `per` tokens, each with its g heads in 2^g2_log rows (the least such number, at
// most 16; the rows behind the g-th repeat the first head, which changes no maximum); with
// g > 16 one token, whose heads come 16 at a time.
//
// A place in the run: sequence, kv head, set of tiles, step.  A sequence of four tiles or
// more has sets of four, each warp a tile; otherwise (and in a call whose bound on the
// chunks' lengths leaves room for none) a set is a tile.
struct ScorePlace {
    SeqItem it;
    int tiles, sets, steps;
    int hk, set, step;
};
__device__ __forceinline__ int score_tiles(const SelectArgs& a, int ql) { return (ql + a.per - 1) >> (4 - a.g2_log); }
__device__ __forceinline__ int score_sets(const SelectArgs& a, int tiles) {
    return a.many && tiles >= kScWarps ? (tiles + kScWarps - 1) / kScWarps : tiles;
}
__device__ __forceinline__ int score_steps(int cl) { return ((cl - 1) / kScaledBlock + kScBlocks) / kScBlocks; }
__device__ __forceinline__ long long score_items(const SelectArgs& a, int ql, int cl) {
    if (!lens_ok(ql, cl, a.mbps) || ql == 0 || (cl - 1) / kScaledBlock + 1 <= a.keep) return 0;
    return (long long)a.Hkv * score_sets(a, score_tiles(a, ql)) * score_steps(cl);
}
__device__ __forceinline__ void score_enter(const SelectArgs& a, ScorePlace& p) {
    p.tiles = score_tiles(a, p.it.ql);
    p.sets = score_sets(a, p.tiles);
    p.steps = score_steps(p.it.cl);
}
// (only called while there are items left)
__device__ __forceinline__ void score_advance(const SelectArgs& a, ScorePlace& p) {
    if (++p.step < p.steps) return;
    p.step = 0;
    if (++p.set < p.sets) return;
    p.set = 0;
    if (++p.hk < a.Hkv) return;
    p.hk = 0;
    long long q0 = p.it.q0;
    do {
        q0 += max(0, p.it.ql);
        ++p.it.s;
        p.it.ql = __ldg(a.q_lens + p.it.s);
        p.it.cl = __ldg(a.ctx_lens + p.it.s);
    } while (score_items(a, p.it.ql, p.it.cl) == 0);
    p.it.q0 = (int)min(q0, 0x7fffffffll);
    score_enter(a, p);
}

// BIG: groups of more than 16 heads.  MANY: some sequence may have four tiles.
template <int D, bool BIG, bool MANY>
__global__ void __launch_bounds__((kScWarps + 1) * 32, kScCtasPerSm) block_score_kernel(const __grid_constant__ SelectArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    using L = ScoreSmem<D>;
    constexpr int CH = D / 32;  // 16-byte chunks of a bound row per lane
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kScStages * L::kStage);
    uint64_t* empty = full + kScStages;
    uint64_t* never = empty + kScStages;  // nothing arrives on it (time-out test hook)
    volatile int* abort_flag = reinterpret_cast<volatile int*>(never + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = a.Hq / a.Hkv;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kScStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kScWarps);
        }
        mbar_init(never, 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    // this CTA's run of items, and where its first one is
    ScorePlace p;
    long long n_items;
    {
        auto count = [&](int ql, int cl) { return score_items(a, ql, cl); };
        const SeqScan scan(a.q_lens, a.ctx_lens, a.num_seqs, a.mbps, count);
        const long long W = gridDim.x, w = blockIdx.x;
        const long long each = scan.items < 1ll << 31 ? (int)scan.items / (int)gridDim.x : scan.items / W, more = scan.items - each * W;
        n_items = each + (w < more ? 1 : 0);
        if (n_items > 0) {  // (else there is no such item)
            scan.find(a.q_lens, a.ctx_lens, w * each + min(w, more), count, p.it);
            score_enter(a, p);
            const long long of_set = p.it.off < 1ll << 31 ? (int)p.it.off / p.steps : p.it.off / p.steps;
            p.step = (int)(p.it.off - of_set * p.steps);
            p.hk = (int)(of_set < 1ll << 31 ? (int)of_set / p.sets : of_set / p.sets);
            p.set = (int)(of_set - (long long)p.hk * p.sets);
        }
    }
    __syncthreads();
    if (n_items <= 0) return;
    bool ok = !a.ctx.force_timeout || mbar_wait_warp(never, 0, a.ctx.wait_ns, abort_flag);
    if (warp == kScWarps) {
        // producer: lane j copies the bounds of the step's j-th block
        auto block_of = [&](const ScorePlace& x) {
            const int b = x.step * kScBlocks + lane;
            return b <= (x.it.cl - 1) / kScaledBlock ? __ldg(a.bt + (long)x.it.s * a.mbps + b) : -2;  // (-2: behind the last)
        };
        long long i = 0;
        int phys = block_of(p), hk = p.hk;
        for (; i < n_items && ok; ++i) {
            const int cur = phys, cur_hk = hk;
            if (i + 1 < n_items) {
                score_advance(a, p);
                phys = block_of(p);
                hk = p.hk;
            }
            const int st = (int)(i % kScStages);
            if (!mbar_wait_warp(&empty[st], (((int)(i / kScStages)) & 1) ^ 1, a.ctx.wait_ns, abort_flag)) {
                ok = false;
                break;
            }
            uint8_t* row = smem + st * L::kStage + lane * L::kRow;
            const bool in = cur >= 0 && cur < a.num_blocks;
            const int rows = __popc(__ballot_sync(0xffffffffu, in));
            if (!in && cur != -2) {  // counts as a block of bounds 0
                raise_error(a.ctx, ERR_BOUNDS_BIT);
                for (int c = 0; c < 4 * D; c += 16) *reinterpret_cast<uint4*>(row + c) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&full[st], rows * 4 * D);
            __syncwarp();
            if (in)
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                 smem_u32(row)),
                             "l"(a.bounds + ((long)cur * a.Hkv + cur_hk) * 2 * D), "r"(4 * D), "r"(smem_u32(&full[st]))
                             : "memory");
        }
        if (!ok) {
            if (lane == 0) {
                raise_error(a.ctx, ERR_TIMEOUT_BIT);
                *abort_flag = 1;
            }
            // let every copy already issued land before the CTA can exit
            for (long long f = max(0ll, i - kScStages); f < i; ++f)
                (void)mbar_wait_warp(&full[f % kScStages], (int)(f / kScStages) & 1, 1000000000ull, nullptr);
        }
        return;
    }
    const int gid = lane >> 2, tig = lane & 3;
    const int rows_log = a.g2_log, row_mask = (1 << rows_log) - 1;
    uint32_t lo[2 * CH][4], hi[2 * CH][4];  // q- and q+: [chunk][half of it] channels 32 i + 8 tig + 4 j + {0, 1}, {2, 3}
    int ti = 0, t0 = 0, nt = 0, blocks = 0;  // the warp's tile, its first token, its tokens, the blocks that its last token sees
    float *dst[2] = {nullptr, nullptr}, *most = nullptr;
    auto load_q = [&](int h0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int rr = gid + 8 * r, h = h0 + (rr & row_mask), tok = rr >> rows_log;
            const uint16_t* src = a.q + (((long)p.it.q0 + t0 + tok) * a.Hq + p.hk * g + (h < g ? h : 0)) * D + 8 * tig;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                const uint4 w = tok < nt ? __ldg(reinterpret_cast<const uint4*>(src + 32 * i)) : make_uint4(0, 0, 0, 0);
                const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    lo[2 * i + k / 2][r + 2 * (k & 1)] = min0_bf16x2(v[k]);
                    hi[2 * i + k / 2][r + 2 * (k & 1)] = max0_bf16x2(v[k]);
                }
            }
        }
    };
    for (long long i = 0; i < n_items && ok; ++i) {
        const bool many = MANY && p.tiles >= kScWarps;
        if (i == 0 || p.step == 0) {  // another set
            ti = many ? p.set * kScWarps + warp : p.set;
            t0 = ti * a.per;
            nt = min(a.per, p.it.ql - t0);
            blocks = (p.it.cl - p.it.ql + t0 + nt - 1) / kScaledBlock + 1;
            if (ti >= p.tiles || blocks <= a.keep || (long long)p.it.q0 + p.it.ql > a.total_q) blocks = 0;  // nothing to do
            if (blocks > 0) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {  // scores of rows gid, gid + 8 (null: not a token's first row)
                    const int rr = gid + 8 * r, tok = rr >> rows_log;
                    dst[r] = (rr & row_mask) == 0 && tok < nt
                                 ? a.scores + (((long)p.it.q0 + t0 + tok) * a.Hkv + p.hk) * a.mbps + 2 * tig : nullptr;
                }
                // the tile that sees every block writes their largest |bound|
                most = ti == p.tiles - 1 ? a.largest + ((long)p.it.s * a.Hkv + p.hk) * a.mbps + gid : nullptr;
                load_q(0);
            }
        }
        const int st = (int)(i % kScStages);
        if (!mbar_wait_warp(&full[st], ((int)(i / kScStages)) & 1, a.ctx.wait_ns, abort_flag)) {
            ok = false;
            break;
        }
        const int b0 = p.step * kScBlocks;
        // NG groups of 8 blocks from bg on at once, so that their chains of MMAs overlap
        auto groups = [&](auto ng, int bg) {
            constexpr int NG = decltype(ng)::value;
            const uint8_t* row = smem + st * L::kStage + (bg - b0 + gid) * L::kRow + tig * 16;
            float m[NG][4];  // rows gid, gid + 8; blocks 2 tig, 2 tig + 1
#pragma unroll
            for (int u = 0; u < NG; ++u) m[u][0] = m[u][1] = m[u][2] = m[u][3] = -INFINITY;
            for (int h0 = 0; h0 < (BIG ? g : 1); h0 += 16) {
                if (BIG) load_q(h0);
                float c[NG][2][4];
#pragma unroll
                for (int u = 0; u < NG; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k) c[u][k][0] = c[u][k][1] = c[u][k][2] = c[u][k][3] = 0.f;
#pragma unroll
                for (int ch = 0; ch < CH; ++ch)
#pragma unroll
                    for (int u = 0; u < NG; ++u) {
                        const uint4 bl = *reinterpret_cast<const uint4*>(row + u * 8 * L::kRow + ch * 64);
                        const uint4 bh = *reinterpret_cast<const uint4*>(row + u * 8 * L::kRow + 2 * D + ch * 64);
                        mma_bf16_16816(c[u][0], lo[2 * ch], bl.x, bl.y);
                        mma_bf16_16816(c[u][1], hi[2 * ch], bh.x, bh.y);
                        mma_bf16_16816(c[u][0], lo[2 * ch + 1], bl.z, bl.w);
                        mma_bf16_16816(c[u][1], hi[2 * ch + 1], bh.z, bh.w);
                    }
#pragma unroll
                for (int u = 0; u < NG; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) m[u][e] = fmaxf(m[u][e], c[u][0][e] + c[u][1][e]);
            }
            // the maximum over a token's rows
            if (rows_log == 4) {
#pragma unroll
                for (int u = 0; u < NG; ++u) {
                    m[u][0] = fmaxf(m[u][0], m[u][2]);
                    m[u][1] = fmaxf(m[u][1], m[u][3]);
                }
            }
#pragma unroll
            for (int o = 0; o < 3; ++o)
                if (o < rows_log) {
#pragma unroll
                    for (int u = 0; u < NG; ++u)
#pragma unroll
                        for (int e = 0; e < 4; ++e) m[u][e] = fmaxf(m[u][e], __shfl_xor_sync(0xffffffffu, m[u][e], 4 << o));
                }
            const int last = blocks - 2 * tig;  // this lane's columns from `last` on do not exist
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (dst[r]) {
#pragma unroll
                    for (int u = 0; u < NG; ++u) {
                        if (bg + 8 * u < last) dst[r][bg + 8 * u] = m[u][2 * r];
                        if (bg + 8 * u + 1 < last) dst[r][bg + 8 * u + 1] = m[u][2 * r + 1];
                    }
                }
            if (most) {
#pragma unroll 1
                for (int u = 0; u < NG; ++u) {
                    uint32_t top = 0;
#pragma unroll
                    for (int i2 = 0; i2 < 2 * CH; ++i2) {
                        const uint4 w = *reinterpret_cast<const uint4*>(row + u * 8 * L::kRow + i2 * 64);
                        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) top = max(top, max(v[k] & 0x7fffu, (v[k] >> 16) & 0x7fffu));
                    }
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    if (tig == 0 && bg + 8 * u + gid < blocks) most[bg + 8 * u] = __uint_as_float(top << 16);
                }
            }
        };
        if (MANY && many) {
#pragma unroll 1
            for (int bg = b0; bg < min(blocks, b0 + kScBlocks); bg += 16) groups(std::integral_constant<int, 2>{}, bg);
        } else if (b0 + 8 * warp < blocks) {
            groups(std::integral_constant<int, 1>{}, b0 + 8 * warp);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        if (i + 1 < n_items) score_advance(a, p);
    }
    if (!ok && lane == 0) {
        raise_error(a.ctx, ERR_TIMEOUT_BIT);
        *abort_flag = 1;
    }
}

__device__ __forceinline__ uint32_t float_key(float x) {  // order-preserving, of a number
    const uint32_t b = __float_as_uint(x);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k); }

// An MMA sum differs from the exact one by at most this times sum |products|.  q-'s and q+'s
// products are summed apart, in d / 16 steps each and one addition.  In a step 16 exact products
// and the sum so far (or 8 and the sum, twice: 18 terms) are aligned to the largest and may each
// lose what lies below its 24 bits, 2^-23 of the magnitudes that meet in it; the addition rounds once.
__device__ __forceinline__ float sum_slack(int d) { return (float)(d / 16 * 18 + 1) * 1.1920929e-7f; }

// A number in two fp32 parts, sums of such (Knuth's error-free addition of the first parts), and their order as
// integers: larger number, larger key; NaN below everything.
struct TwoFloat {
    float hi, lo;
    __device__ __forceinline__ void add(float bh, float bl) {
        const float s = __fadd_rn(hi, bh), t = __fsub_rn(s, hi);
        const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(bh, t));
        hi = s;
        lo = __fadd_rn(lo, __fadd_rn(bl, e));
    }
    __device__ __forceinline__ unsigned long long key() const {
        const float h = __fadd_rn(hi, lo), l = __fsub_rn(lo, __fsub_rn(h, hi));  // (h is the nearest to the number)
        if (!(h == h)) return 0ull;
        return (unsigned long long)float_key(h + 0.f) << 32 | float_key(l == l ? l + 0.f : 0.f);
    }
};

// The exact score of block `phys` for a token's heads (q: the first head's channels): a warp.
template <int D>
__device__ __forceinline__ unsigned long long exact_key(const uint16_t* __restrict__ q, int g, const uint16_t* __restrict__ box) {
    constexpr int N = D / 32;  // channels per lane
    const int lane = threadIdx.x & 31;
    uint32_t l[N / 2], h[N / 2];
    auto load = [&](const uint16_t* p, uint32_t (&x)[N / 2]) {
        if constexpr (N == 4) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(p + lane * 4));
            x[0] = u.x;
            x[1] = u.y;
        } else {
            x[0] = __ldg(reinterpret_cast<const uint32_t*>(p + lane * 2));
        }
    };
    auto get = [](const uint32_t (&x)[N / 2], int c) { return __uint_as_float(c & 1 ? x[c / 2] & 0xFFFF0000u : x[c / 2] << 16); };
    load(box, l);
    load(box + D, h);
    unsigned long long best = 0;
    for (int h0 = 0; h0 < g; h0 += 4) {  // four heads' sums side by side
        TwoFloat s[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t x[N / 2];
            load(q + (long)min(h0 + k, g - 1) * D, x);
            s[k] = TwoFloat{0.f, 0.f};
#pragma unroll
            for (int c = 0; c < N; ++c) {  // (a product of two bf16 numbers is exact in fp32)
                const float v = get(x, c);
                s[k].add(__fmul_rn(v, v < 0.f ? get(l, c) : get(h, c)), 0.f);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float bh = __shfl_xor_sync(0xffffffffu, s[k].hi, o), bl = __shfl_xor_sync(0xffffffffu, s[k].lo, o);
                s[k].add(bh, bl);
            }
#pragma unroll
        for (int k = 0; k < 4; ++k) best = max(best, s[k].key());
    }
    return best;
}

template <int D, int kTopThreads>
__global__ void __launch_bounds__(kTopThreads, 1024 / kTopThreads) block_top_kernel(const __grid_constant__ SelectArgs a) {
    extern __shared__ uint32_t taken[];  // a bit for each block
    __shared__ __align__(16) int hist[kTopBins];
    __shared__ unsigned long long near_key_sh[kTopNear];
    __shared__ int near_b_sh[kTopNear];
    __shared__ int warp_sums[kTopThreads / 32], bin_sel, above_sel, count_sel, near_n, sure_n;
    __shared__ uint32_t lo_sh, hi_sh, big_sh, sum_sh;  // keys of the range's ends; bits of the largest |bound| and sum of |q|
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = a.Hq / a.Hkv;
    constexpr int kBinsPer = kTopBins / kTopThreads;
    bool waited = false;
    const long rows = (long)a.total_q * a.Hkv;
    for (long row = blockIdx.x; row < rows; row += gridDim.x) {
        const long at_row = row < 1l << 31 ? (int)row / a.Hkv : row / a.Hkv;
        const int hk = (int)(row - at_row * a.Hkv);
        // the largest sum of |q| of a head
        float sum_q = 0.f;
        for (int h = warp; h < g; h += kTopThreads / 32) {
            const uint16_t* q = a.q + (at_row * a.Hq + hk * g + h) * D;
            float x = 0.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) x += fabsf(__uint_as_float((uint32_t)__ldg(q + c * 32 + lane) << 16));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            sum_q = fmaxf(sum_q, x);
        }
        SeqItem it;
        auto count = [](int ql, int) { return ql; };
        const SeqScan scan(a.q_lens, a.ctx_lens, a.num_seqs, a.mbps, count);
        const bool some = scan.find(a.q_lens, a.ctx_lens, at_row, count, it);
        const bool fits = some && lens_ok(it.ql, it.cl, a.mbps) && (long long)it.q0 + it.ql <= a.total_q;
        if (hk == 0 && tid == 0 && (some != fits || scan.bad || scan.rows > a.total_q)) raise_error(a.ctx, ERR_BOUNDS_BIT);
        if (!fits) continue;  // (or a row behind the last sequence)
        int32_t* out = a.sel + row * a.keep;
        const int n = (it.cl - it.ql + (int)it.off) / kScaledBlock + 1;  // blocks that the query sees
        if (n <= a.keep) {
            for (int i = tid; i < a.keep; i += kTopThreads) out[i] = i < n ? i : -1;
            continue;
        }
        const int mid0 = a.sink, mid1 = n - a.recent;  // the scores decide about blocks [mid0, mid1)
        const int want = a.keep - a.sink - a.recent;
        const int words = (n + 31) / 32;
        __syncthreads();  // what the row before left in shared memory is read
        for (int w = tid; w < words; w += kTopThreads) {
            uint32_t bits = 0;  // the first and the last blocks
            const int b0 = w * 32;
            if (mid0 > b0) bits |= mid0 - b0 >= 32 ? 0xffffffffu : (1u << (mid0 - b0)) - 1;
            if (mid1 < b0 + 32) bits |= mid1 <= b0 ? 0xffffffffu : ~((1u << (mid1 - b0)) - 1);
            if (n < b0 + 32) bits &= (1u << (n - b0)) - 1;
            taken[w] = bits;
        }
        auto clear_bins = [&]() {
#pragma unroll
            for (int k = 0; k < kTopBins / 2 / kTopThreads; ++k)
                reinterpret_cast<int2*>(hist)[k * kTopThreads + tid] = make_int2(0, 0);
        };
        clear_bins();
        if (tid == 0) {
            near_n = sure_n = 0;
            lo_sh = 0xffffffffu;
            hi_sh = big_sh = sum_sh = 0u;
        }
        if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // the scores are complete
        waited = true;
        const float* sc = a.scores + row * a.mbps;
        const float* largest = a.largest + ((long)it.s * a.Hkv + hk) * a.mbps;
        constexpr int kPass = kTopThreads * kTopItems;
        const bool once = n <= kPass;
        float v[kTopItems];
        auto load = [&](int base) {  // scores of blocks base + kTopThreads k + tid (finite: the largest numbers stand for infinities, NaN last)
#pragma unroll
            for (int k = 0; k < kTopItems; ++k) {
                if (base + k * kTopThreads >= mid1) break;  // (the same for the whole CTA)
                const int b = base + k * kTopThreads + tid;
                const float x = b >= mid0 && b < mid1 ? __ldcg(sc + b) : 0.f;
                v[k] = x == x ? fminf(fmaxf(x, -1e38f), 1e38f) : -1e38f;
            }
        };
        // f(block, its score, whether the scores decide about it) for all of them, whole warps
        auto for_scores = [&](auto f) {
            for (int base = 0; base < mid1; base += kPass) {
                if (!once) load(base);
#pragma unroll
                for (int k = 0; k < kTopItems; ++k) {
                    if (base + k * kTopThreads >= mid1) break;
                    const int b = base + k * kTopThreads + tid;
                    f(b, v[k], b >= mid0 && b < mid1);
                }
            }
        };
        float big = 0.f;
        for (int b = mid0 + tid; b < mid1; b += kTopThreads) {
            const float x = __ldcg(largest + b);
            if (x < INFINITY) big = fmaxf(big, x);  // (an infinite bound says nothing about the others' roundings)
        }
        load(0);
        __syncthreads();
        if (want > 0) {
            uint32_t klo = 0xffffffffu, khi = 0u;
            for_scores([&](int, float x, bool in) {
                if (in) {
                    klo = min(klo, float_key(x));
                    khi = max(khi, float_key(x));
                }
            });
            klo = __reduce_min_sync(0xffffffffu, klo);
            khi = __reduce_max_sync(0xffffffffu, khi);
            const uint32_t kbig = __reduce_max_sync(0xffffffffu, __float_as_uint(big));  // (not negative: in order as integers)
            if (lane == 0) {
                atomicMin(&lo_sh, klo);
                atomicMax(&hi_sh, khi);
                atomicMax(&big_sh, kbig);
                atomicMax(&sum_sh, __float_as_uint(sum_q));
            }
            __syncthreads();
            float lo = key_float(lo_sh), hi = key_float(hi_sh);
            float slack = 2.f * __uint_as_float(big_sh) * __uint_as_float(sum_sh) * sum_slack(D);
            if (!(slack < 1e37f)) slack = 0.f;  // queries that are not finite, or products that fp32 cannot hold: as they come
            // Bins of the range [lo, hi]; the range becomes that of the bin with the last block taken while it holds
            // many blocks and is wider than what the roundings blur anyway.
            int need = want, sel = 0;  // blocks to take of the range
            float inv;
            auto bin = [&](float x) { return min(kTopBins - 1, max(0, (int)((x - lo) * inv))); };
            for (int pass = 0;; ++pass) {
                inv = fminf((kTopBins - 1) / fmaxf(hi - lo, 1e-37f), 1e37f);
                for_scores([&](int, float x, bool in) {
                    if (in && x >= lo && x <= hi) atomicAdd(&hist[bin(x)], 1);
                });
                __syncthreads();
                const int top = kTopBins - kBinsPer * (tid + 1);  // this thread's bins, highest first
                int cnt[kBinsPer], own = 0;
#pragma unroll
                for (int b = 0; b < kBinsPer; b += 2) {
                    const int2 c = *reinterpret_cast<const int2*>(&hist[top + b]);
                    cnt[b] = c.x;
                    cnt[b + 1] = c.y;
                    own += c.x + c.y;
                }
                int x = own;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                if (lane == 31) warp_sums[warp] = x;
                __syncthreads();
                int above = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane & (kTopThreads / 32 - 1)] : 0) + x - own;
                if (above < need && above + own >= need) {
#pragma unroll
                    for (int b = kBinsPer - 1; b >= 0; --b) {
                        if (above < need && above + cnt[b] >= need) {
                            bin_sel = top + b;
                            above_sel = above;
                            count_sel = cnt[b];
                        }
                        above += cnt[b];
                    }
                }
                if (tid == 0) {
                    lo_sh = 0xffffffffu;
                    hi_sh = 0u;
                }
                clear_bins();
                __syncthreads();
                sel = bin_sel;
                if (count_sel <= 32 || pass == 5 || !(1.f > slack * inv)) break;
                need -= above_sel;
                klo = 0xffffffffu;
                khi = 0u;
                for_scores([&](int, float y, bool in) {
                    if (in && y >= lo && y <= hi && bin(y) == sel) {
                        klo = min(klo, float_key(y));
                        khi = max(khi, float_key(y));
                    }
                });
                klo = __reduce_min_sync(0xffffffffu, klo);
                khi = __reduce_max_sync(0xffffffffu, khi);
                if (lane == 0) {
                    atomicMin(&lo_sh, klo);
                    atomicMax(&hi_sh, khi);
                }
                __syncthreads();
                lo = key_float(lo_sh);
                hi = key_float(hi_sh);
                if (lo == hi) break;  // (all alike)
            }
            // The border lies in bin `sel` of [lo, hi], or at lo = hi.  Sure: above it by more than both sums' errors;
            // near: within them (a bin more, for the rounding of the bins themselves).
            const int blur = lo == hi ? 0 : (int)fminf(slack * inv, (float)kTopBins) + 2;
            int32_t* near_far = a.near_b + (long)blockIdx.x * a.mbps;
            int sure = 0;
            for_scores([&](int b, float x, bool in) {
                bool is_sure = x > hi + slack, is_near = x >= lo - slack && !is_sure;
                if (lo != hi && x >= lo && x <= hi) {
                    is_sure = bin(x) > sel + blur;
                    is_near = !is_sure && bin(x) >= sel - blur;
                } else if (lo != hi) {  // outside the last range: near if within the slack of the border's bin
                    is_near = is_near && (x > hi ? kTopBins - 1 - sel <= blur : sel <= blur);
                    is_sure = x > hi && !is_near;
                }
                is_sure = is_sure && in;
                is_near = is_near && in;
                const unsigned ms = __ballot_sync(0xffffffffu, is_sure), mn = __ballot_sync(0xffffffffu, is_near);
                sure += __popc(ms);
                if (lane == 0 && ms) atomicOr(&taken[b >> 5], ms);  // (a warp's 32 blocks are one word)
                if (mn) {
                    int at = 0;
                    if (lane == 0) at = atomicAdd(&near_n, __popc(mn));
                    at = __shfl_sync(0xffffffffu, at, 0) + __popc(mn & ((1u << lane) - 1));
                    if (is_near) {
                        if (at < kTopNear) near_b_sh[at] = b;
                        near_far[at] = b;
                    }
                }
            });
            if (lane == 0 && sure) atomicAdd(&sure_n, sure);
            __syncthreads();
            const int cand = near_n, rest0 = want - sure_n;
            const bool far = cand > kTopNear;
            const int32_t* near_b = far ? near_far : near_b_sh;
            unsigned long long* near_key = far ? a.near_key + (long)blockIdx.x * a.mbps : near_key_sh;
            if (cand <= rest0) {
                for (int i = tid; i < cand; i += kTopThreads) atomicOr(&taken[near_b[i] >> 5], 1u << (near_b[i] & 31));
            } else {
                // exact keys of the blocks near the border (without a bound on the roundings, all alike)
                const uint16_t* q = a.q + (at_row * a.Hq + hk * g) * D;
                for (int i = warp; i < cand; i += kTopThreads / 32) {
                    const int phys = __ldg(a.bt + (long)it.s * a.mbps + near_b[i]);
                    unsigned long long key = 1ull << 63 | 1ull << 31;  // a score of 0
                    if (slack > 0.f && phys >= 0 && phys < a.num_blocks)
                        key = exact_key<D>(q, g, a.bounds + ((long)phys * a.Hkv + hk) * 2 * D);
                    if (lane == 0) near_key[i] = key;
                }
                __syncthreads();
                // the `rest0` largest, equal ones by block number
                if (!far) {
                    for (int i = tid; i < cand; i += kTopThreads) {
                        const unsigned long long k = near_key_sh[i];
                        const int b = near_b_sh[i];
                        int before = 0;
                        for (int j = 0; j < cand; ++j) before += near_key_sh[j] > k || (near_key_sh[j] == k && near_b_sh[j] < b);
                        if (before < rest0) atomicOr(&taken[b >> 5], 1u << (b & 31));
                    }
                } else {
                    // radix select over (key, ~block number), 8 bits at a time: distinct, so it ends with one
                    unsigned long long p0 = 0;
                    uint32_t p1 = 0;
                    int rest = rest0;
                    for (int pass = 0; pass < 12; ++pass) {
                        const int sh = 56 - 8 * pass, sh1 = 24 - 8 * (pass - 8);
                        for (int i = tid; i < cand; i += kTopThreads) {
                            const unsigned long long k = near_key[i];
                            const uint32_t nb = ~(uint32_t)near_b[i];
                            bool in;
                            int dg;
                            if (pass < 8) {
                                in = pass == 0 || (k ^ p0) >> (sh + 8) == 0;
                                dg = (int)(k >> sh) & 255;
                            } else {
                                in = k == p0 && (pass == 8 || (nb ^ p1) >> (sh1 + 8) == 0);
                                dg = (int)(nb >> sh1) & 255;
                            }
                            if (in) atomicAdd(&hist[dg], 1);
                        }
                        __syncthreads();
                        if (warp == 0) {  // 8 bins a lane, highest first
                            int own = 0;
                            for (int b = 0; b < 8; ++b) own += hist[255 - 8 * lane - b];
                            int x = own;
#pragma unroll
                            for (int o = 1; o < 32; o <<= 1) {
                                const int y = __shfl_up_sync(0xffffffffu, x, o);
                                if (lane >= o) x += y;
                            }
                            int above = x - own;
                            if (above < rest && above + own >= rest)
                                for (int b = 0; b < 8; ++b) {
                                    const int c = hist[255 - 8 * lane - b];
                                    if (above < rest && above + c >= rest) {
                                        bin_sel = 255 - 8 * lane - b;
                                        above_sel = above;
                                    }
                                    above += c;
                                }
                        }
                        __syncthreads();
                        for (int i = tid; i < 256; i += kTopThreads) hist[i] = 0;
                        if (pass < 8) p0 |= (unsigned long long)bin_sel << sh;
                        else p1 |= (uint32_t)bin_sel << sh1;
                        rest -= above_sel;
                        __syncthreads();
                    }
                    for (int i = tid; i < cand; i += kTopThreads) {
                        const unsigned long long k = near_key[i];
                        const int b = near_b[i];
                        if (k > p0 || (k == p0 && ~(uint32_t)b >= p1)) atomicOr(&taken[b >> 5], 1u << (b & 31));
                    }
                }
            }
        }
        __syncthreads();
        // the taken blocks in order
        int before = 0;
        for (int base = 0; base < words; base += kTopThreads) {
            const int w = base + tid;
            uint32_t bits = w < words ? taken[w] : 0u;
            const int own = __popc(bits);
            int x = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (base > 0) __syncthreads();  // warp_sums is read
            if (lane == 31) warp_sums[warp] = x;
            __syncthreads();
            const int ws = lane < kTopThreads / 32 ? warp_sums[lane] : 0;
            int at = before + __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0) + x - own;
            before += __reduce_add_sync(0xffffffffu, ws);
            for (; bits; bits &= bits - 1, ++at)
                if (at < a.keep) out[at] = w * 32 + __ffs(bits) - 1;
        }
    }
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // never complete ahead of the grid before
}

struct SelectWs {
    size_t scores, largest, near_b, near_key, total;
};
static SelectWs select_ws_layout(int num_seqs, int mbps, int Hkv, int total_q) {
    SelectWs w{};
    w.scores = 0;
    w.largest = align256(sizeof(float) * (size_t)total_q * Hkv * mbps);
    w.near_key = align256(w.largest + sizeof(float) * (size_t)num_seqs * Hkv * mbps);
    const size_t ctas = std::min<size_t>((size_t)total_q * Hkv, kTopCtas);  // (a CTA a row while they last)
    w.near_b = align256(w.near_key + sizeof(unsigned long long) * ctas * mbps);
    w.total = align256(w.near_b + sizeof(int32_t) * ctas * mbps);
    return w;
}

}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_block_select_workspace_size(int num_seqs, int max_blocks_per_seq, int Hq, int Hkv, int d, int total_q) {
    if (num_seqs <= 0 || max_blocks_per_seq <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || total_q <= 0) return 0;
    return select_ws_layout(num_seqs, max_blocks_per_seq, Hkv, total_q).total;
}

fa_status fa_block_select(const void* q, const void* bounds, const int32_t* block_table, const int32_t* ctx_lens,
                          const int32_t* q_lens, int32_t* sel, int num_seqs, int max_blocks_per_seq, int num_blocks, int Hq,
                          int Hkv, int d, int block_size, int keep, int recent, int sink, int total_q, int max_q_len, void* ws,
                          size_t ws_bytes, fa_stream_t stream) {
    set_launch_count(0);
    if (num_seqs < 0 || max_blocks_per_seq < 0 || num_blocks < 0 || Hq <= 0 || Hkv <= 0 || total_q < 0 || max_q_len < 0 ||
        keep <= 0 || recent < 0 || sink < 0 || recent > keep || sink > keep - recent)
        return FA_ERR_INVALID_ARG;
    if (block_size != kScaledBlock || (d != 64 && d != 128) || Hq % Hkv != 0) return FA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0 || max_q_len == 0) return FA_OK;
    if (!q || !bounds || !block_table || !ctx_lens || !q_lens || !sel) return FA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(bounds)) return FA_ERR_INVALID_ARG;
    if (num_blocks == 0 || max_blocks_per_seq == 0) return FA_ERR_INVALID_ARG;
    const SelectWs w = select_ws_layout(num_seqs, max_blocks_per_seq, Hkv, total_q);
    if (!ws || ws_bytes < w.total || (reinterpret_cast<uintptr_t>(ws) & 255)) return FA_ERR_WORKSPACE;
    const size_t bitmap = sizeof(uint32_t) * (((size_t)max_blocks_per_seq + 31) / 32);
    if (bitmap > 160 * 1024 || (long)num_seqs * Hkv > 0x7fffffffL) return FA_ERR_UNSUPPORTED;
    fa_status st = check_device();
    if (st != FA_OK) return st;
    uint8_t* wsb = static_cast<uint8_t*>(ws);
    SelectArgs a{static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(bounds), block_table, ctx_lens, q_lens,
                 reinterpret_cast<float*>(wsb + w.scores), reinterpret_cast<float*>(wsb + w.largest),
                 reinterpret_cast<int32_t*>(wsb + w.near_b), reinterpret_cast<unsigned long long*>(wsb + w.near_key), sel,
                 num_seqs, max_blocks_per_seq, num_blocks, total_q, Hq, Hkv, keep, recent, sink, 0, 1, 0, {}};
    while (1 << a.g2_log < Hq / Hkv && a.g2_log < 4) ++a.g2_log;
    a.per = 16 >> a.g2_log;
    a.many = max_q_len > (kScWarps - 1) * a.per;
    if ((st = make_ctx(&a.ctx)) != FA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int launches = 0;
    if (max_blocks_per_seq > keep) {  // else every block is taken
        const unsigned grid = (unsigned)(kScCtasPerSm * sm_count());
        auto variant = [&](auto big, auto many) {
            constexpr bool BIG = decltype(big)::value, MANY = decltype(many)::value;
            return d == 128 ? block_score_kernel<128, BIG, MANY> : block_score_kernel<64, BIG, MANY>;
        };
        const std::true_type yes;
        const std::false_type no;
        auto score = Hq / Hkv > 16 ? (a.many ? variant(yes, yes) : variant(yes, no)) : (a.many ? variant(no, yes) : variant(no, no));
        const int smem = d == 128 ? ScoreSmem<128>::kBytes : ScoreSmem<64>::kBytes;
        if ((st = raise_dynamic_smem(reinterpret_cast<const void*>(score), smem)) != FA_OK) return st;
        score<<<grid, (kScWarps + 1) * 32, smem, s>>>(a);
        if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
        ++launches;
    }
    // few rows: more threads each (the call with 128 rows of up to 2048 scores 35.0 us, with 256 threads 37.1; with 1140
    // rows of up to 500 36.7, with 256 threads 41.2)
    const long rows = (long)total_q * Hkv;
    const int threads = rows <= 2L * sm_count() ? kTopFew : kTopMany;
    auto top = threads == kTopFew ? (d == 128 ? block_top_kernel<128, kTopFew> : block_top_kernel<64, kTopFew>)
                                  : (d == 128 ? block_top_kernel<128, kTopMany> : block_top_kernel<64, kTopMany>);
    if (bitmap + 16 * 1024 > kUnraisedSmem &&
        (st = raise_dynamic_smem(reinterpret_cast<const void*>(top), (int)bitmap)) != FA_OK)
        return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<long>(rows, std::min<long>(kTopCtas, 1024L / threads * sm_count())));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = bitmap;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = launches > 0 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, top, a) != cudaSuccess) return FA_ERR_CUDA;
    set_launch_count(launches + 1);
    return FA_OK;
}

}  // extern "C"
