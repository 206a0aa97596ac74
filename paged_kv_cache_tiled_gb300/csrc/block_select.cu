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
// block_score_kernel reads each block's bounds once for all rows of a tile (4 d bytes,
// straight to registers: the MMA's K dimension is taken in an order in which a lane's B
// operands are 16 consecutive bytes).  Memory bound for single tokens.
// block_top_kernel finds the score of the last block taken with a radix select over
// order-preserving integer keys.  An MMA's sum is off by its roundings, which must not
// decide: blocks whose score lies within the rounding bound of that border are summed
// again in 64 bits and ordered by that, equal ones by their number, so that the
// choice is that of exact arithmetic.  Few blocks are that close (a handful of
// thousands), unless many are equal.
#include <algorithm>

#include "cache_scaled.cuh"

namespace fa {

constexpr int kScWarps = 8;
constexpr int kTopThreads = 256;
constexpr int kTopItems = 16;    // scores per thread that stay in registers
constexpr int kTopBins = 2048;
constexpr int kTopCount = 256;   // blocks near the border that are ranked by counting
constexpr int kTopCtasPerSm = 4;  // grid of the top kernel, and its scratch

struct SelectArgs {
    const uint16_t *q, *bounds;
    const int32_t *bt, *ctx_lens, *q_lens;
    float* scores;   // [total_q][Hkv][mbps]
    float* largest;  // [num_seqs][Hkv][mbps]: a block's largest |bound|
    int32_t* near_b;   // per CTA of the top kernel: blocks near the border
    unsigned long long* near_key;  // and their keys
    int32_t* sel;
    int num_seqs, mbps, num_blocks, total_q, Hq, Hkv, keep, recent, sink;
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

// CTA (sequence and kv head; share of its blocks; share of its tokens).  A warp takes
// groups of 8 blocks and tiles of 16 / g tokens (one token and its heads in turns of 16
// when g > 16); with many tokens the warps of a CTA take different tokens of the
// same blocks, whose bounds they then find in L1.
template <int D>
__global__ void __launch_bounds__(kScWarps * 32, 2) block_score_kernel(const __grid_constant__ SelectArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int CH = D / 32;  // 16-byte chunks of a bound row per lane
    __shared__ float tile[kScWarps][16][8 + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
    const int s = blockIdx.x / a.Hkv, hk = blockIdx.x % a.Hkv, g = a.Hq / a.Hkv;
    const int ql = __ldg(a.q_lens + s), cl = __ldg(a.ctx_lens + s);
    if (!lens_ok(ql, cl, a.mbps) || ql == 0 || (cl - 1) / kScaledBlock + 1 <= a.keep) return;
    long long q0 = 0;
    for (int i = lane; i < s; i += 32) q0 += max(0, __ldg(a.q_lens + i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) q0 += __shfl_xor_sync(0xffffffffu, q0, o);
    if (q0 + ql > a.total_q) return;
    const int per = g <= 16 ? 16 / g : 1, tiles = (ql + per - 1) / per;  // tokens a tile, tiles
    int side = 1;  // warps side by side along the tokens
    while (side < kScWarps && side < tiles) side *= 2;
    const int my_tile = blockIdx.z * side + warp % side, my_group = blockIdx.y * (kScWarps / side) + warp / side;
    const int tile_step = gridDim.z * side, group_step = gridDim.y * (kScWarps / side);
    for (int ti = my_tile; ti < tiles; ti += tile_step) {
        const int t0 = ti * per, nt = min(per, ql - t0);
        const int blocks = (cl - ql + t0 + nt - 1) / kScaledBlock + 1;  // that the tile's last token sees
        if (blocks <= a.keep) continue;
        const int groups = (blocks + 7) / 8;
        for (int h0 = 0; h0 < g; h0 += 16) {
            // A rows: token t0 + r / g, head r % g of the group (g > 16: head h0 + r of one token)
            const int nr = g <= 16 ? nt * g : min(16, g - h0);
            uint32_t qa[2 * CH][4];  // [chunk][half of it]: channels 32 i + 8 tig + 4 j + {0, 1}, {2, 3} of rows gid, gid + 8
#pragma unroll
            for (int i = 0; i < CH; ++i)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int rr = gid + 8 * r;
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (rr < nr) {
                        const int tok = g <= 16 ? t0 + rr / g : t0, head = g <= 16 ? rr % g : h0 + rr;
                        w = __ldg(reinterpret_cast<const uint4*>(a.q + ((q0 + tok) * a.Hq + hk * g + head) * D + 32 * i + 8 * tig));
                    }
                    qa[2 * i][r] = w.x;
                    qa[2 * i][r + 2] = w.y;
                    qa[2 * i + 1][r] = w.z;
                    qa[2 * i + 1][r + 2] = w.w;
                }
            auto block_of = [&](int grp) {
                const int b = grp * 8 + gid;
                int phys = grp < groups && b < blocks ? __ldg(a.bt + (long)s * a.mbps + b) : -1;
                if (phys >= a.num_blocks) phys = -1;
                return phys;
            };
            uint4 w[2 * CH], next[2 * CH];  // lo's chunks, then hi's
            auto load = [&](int phys, uint4 (&x)[2 * CH]) {
                const uint4* src = reinterpret_cast<const uint4*>(a.bounds + ((long)phys * a.Hkv + hk) * 2 * D) + tig;
#pragma unroll
                for (int i = 0; i < 2 * CH; ++i) x[i] = phys >= 0 ? __ldg(src + 4 * i) : make_uint4(0, 0, 0, 0);
            };
            int phys = block_of(my_group), phys_next = block_of(my_group + group_step);
            load(phys, w);
            for (int grp = my_group; grp < groups; grp += group_step) {
                load(phys_next, next);
                const int phys_after = block_of(grp + 2 * group_step);
                if (phys < 0 && grp * 8 + gid < blocks) raise_error(a.ctx, ERR_BOUNDS_BIT);
                float c[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < CH; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t lo[4], hi[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            lo[r] = min0_bf16x2(qa[2 * i + j][r]);
                            hi[r] = max0_bf16x2(qa[2 * i + j][r]);
                        }
                        const uint4 &bl = w[i], &bh = w[CH + i];
                        mma_bf16_16816(c, lo, j ? bl.z : bl.x, j ? bl.w : bl.y);
                        mma_bf16_16816(c2, hi, j ? bh.z : bh.x, j ? bh.w : bh.y);
                    }
                const bool last = ti == tiles - 1 && h0 == 0;  // the tile that sees every block
                if (last) {  // the block's largest |bound|
#pragma unroll
                    for (int i = 0; i < 2 * CH; ++i) {
                        const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) top = max(top, max(v[k] & 0x7fffu, (v[k] >> 16) & 0x7fffu));
                    }
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                }
                __syncwarp();  // the tile's values of the group before are read
                tile[warp][gid][2 * tig] = c[0] + c2[0];
                tile[warp][gid][2 * tig + 1] = c[1] + c2[1];
                tile[warp][gid + 8][2 * tig] = c[2] + c2[2];
                tile[warp][gid + 8][2 * tig + 1] = c[3] + c2[3];
                __syncwarp();
                for (int x = lane; x < nt * 8; x += 32) {
                    const int tok = x >> 3, b = grp * 8 + (x & 7);
                    const int r0 = g <= 16 ? tok * g : 0, r1 = g <= 16 ? r0 + g : nr;
                    float m = -INFINITY;
                    for (int r = r0; r < r1; ++r) m = fmaxf(m, tile[warp][r][x & 7]);
                    if (b >= blocks) continue;
                    float* dst = a.scores + ((q0 + t0 + tok) * a.Hkv + hk) * a.mbps + b;
                    *dst = h0 > 0 ? fmaxf(m, *dst) : m;
                }
                if (last && tig == 0 && grp * 8 + gid < blocks)
                    a.largest[((long)s * a.Hkv + hk) * a.mbps + grp * 8 + gid] = __uint_as_float(top << 16);
#pragma unroll
                for (int i = 0; i < 2 * CH; ++i) w[i] = next[i];
                phys = phys_next;
                phys_next = phys_after;
            }
        }
    }
}

// Larger score, larger key; NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t score_key(float x) {
    if (!(x == x)) return 0u;
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_score(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long score_key64(double x) {
    if (!(x == x)) return 0ull;
    const unsigned long long b = (unsigned long long)__double_as_longlong(x + 0.0);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// An MMA sum differs from the exact one by at most this times sum |products|: 2 (d / 16)
// steps and the final addition; in a step 16 exact products and the accumulator are
// aligned to the largest and may each lose what lies below its 24 bits, 17 * 2^-23 < 2^-18
// of the magnitudes that meet in it.
__device__ __forceinline__ float sum_slack(int d) { return (float)(d / 8 + 1) * 3.814697265625e-6f; }

template <int D>
__global__ void __launch_bounds__(kTopThreads, kTopCtasPerSm) block_top_kernel(const __grid_constant__ SelectArgs a) {
    extern __shared__ uint32_t taken[];  // a bit for each block
    __shared__ __align__(16) int hist[kTopBins];
    __shared__ int warp_sums[kTopThreads / 32], digit_sel, above_sel, near_n, sure_n;
    __shared__ float slack_sh[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = a.Hq / a.Hkv;
    constexpr int kBinsPer = kTopBins / kTopThreads;
    int32_t* near_b = a.near_b + (long)blockIdx.x * a.mbps;
    unsigned long long* near_key = a.near_key + (long)blockIdx.x * a.mbps;
    bool waited = false;
    const long rows = (long)a.total_q * a.Hkv;
    for (long row = blockIdx.x; row < rows; row += gridDim.x) {
        const int hk = (int)(row % a.Hkv);
        SeqItem it;
        const bool some = find_item(a.q_lens, a.ctx_lens, a.num_seqs, row / a.Hkv,
                                    [&](int ql, int cl) { return lens_ok(ql, cl, a.mbps) ? ql : -1; }, it);
        if (row == 0 && tid == 0 && (it.bad || it.rows != a.total_q)) raise_error(a.ctx, ERR_BOUNDS_BIT);
        if (!some || (long long)it.q0 + it.ql > a.total_q) continue;
        const long at_row = (long)it.q0 + it.off;
        int32_t* out = a.sel + (at_row * a.Hkv + hk) * a.keep;
        const int n = (it.cl - it.ql + it.off) / kScaledBlock + 1;  // blocks that the query sees
        if (n <= a.keep) {
            for (int i = tid; i < a.keep; i += kTopThreads) out[i] = i < n ? i : -1;
            continue;
        }
        if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");  // the scores are complete
        waited = true;
        const float* sc = a.scores + (at_row * a.Hkv + hk) * a.mbps;
        const int mid0 = a.sink, mid1 = n - a.recent;  // the scores decide about blocks [mid0, mid1)
        const int want = a.keep - a.sink - a.recent;
        const bool once = n <= kTopThreads * kTopItems;
        uint32_t key[kTopItems];
        unsigned middle;
        auto load = [&](int base) {
            middle = 0;
#pragma unroll
            for (int k = 0; k < kTopItems; ++k) {
                const int b = base + k * kTopThreads + tid;
                key[k] = 0;
                if (b >= mid0 && b < mid1) {
                    key[k] = score_key(__ldcg(sc + b));
                    middle |= 1u << k;
                }
            }
        };
        load(0);
        const int words = (n + 31) / 32;
        __syncthreads();  // `taken` of the row before is read
        for (int w = tid; w < words; w += kTopThreads) {
            uint32_t bits = 0;  // the first and the last blocks
            const int b0 = w * 32;
            if (mid0 > b0) bits |= mid0 - b0 >= 32 ? 0xffffffffu : (1u << (mid0 - b0)) - 1;
            if (mid1 < b0 + 32) bits |= mid1 <= b0 ? 0xffffffffu : ~((1u << (mid1 - b0)) - 1);
            if (n < b0 + 32) bits &= (1u << (n - b0)) - 1;
            taken[w] = bits;
        }
        for (int i = tid; i < kTopBins; i += kTopThreads) hist[i] = 0;
        if (tid == 0) near_n = sure_n = 0;
        // the rounding bound: the largest bound of the blocks, times the largest sum of |q| of a head
        float big = 0.f;
        for (int b = mid0 + tid; b < mid1; b += kTopThreads)
            big = fmaxf(big, __ldcg(a.largest + ((long)it.s * a.Hkv + hk) * a.mbps + b));
        if (tid < 2) slack_sh[tid] = 0.f;
        __syncthreads();
        big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
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
        if (lane == 0) {  // (not negative: as integers in order)
            atomicMax(reinterpret_cast<int*>(&slack_sh[0]), __float_as_int(big));
            atomicMax(reinterpret_cast<int*>(&slack_sh[1]), __float_as_int(sum_q));
        }
        uint32_t prefix = 0;
        int need = want;
        for (int pass = 0; pass < 3 && want > 0; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
            for (int base = 0; base < n; base += kTopThreads * kTopItems) {
                if (!once) load(base);
#pragma unroll
                for (int k = 0; k < kTopItems; ++k) {
                    const bool in = ((middle >> k) & 1u) && (pass == 0 || ((key[k] ^ prefix) >> (shift + bits)) == 0);
                    if (in) atomicAdd(&hist[(key[k] >> shift) & ((1u << bits) - 1)], 1);
                }
            }
            __syncthreads();
            const int top = kTopBins - kBinsPer * (tid + 1);  // this thread's bins, highest first
            int cnt[kBinsPer], own = 0;
#pragma unroll
            for (int b = 0; b < kBinsPer; ++b) {
                cnt[b] = hist[top + b];
                hist[top + b] = 0;
                own += cnt[b];
            }
            int x = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) warp_sums[warp] = x;
            __syncthreads();
            int above = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane & 7] : 0) + x - own;
            if (above < need && above + own >= need) {
#pragma unroll
                for (int b = kBinsPer - 1; b >= 0; --b) {
                    if (above < need && above + cnt[b] >= need) {
                        digit_sel = top + b;
                        above_sel = above;
                    }
                    above += cnt[b];
                }
            }
            __syncthreads();
            prefix |= (uint32_t)digit_sel << shift;
            need -= above_sel;
        }
        if (want > 0) {
            // sure: above the border by more than both sums' errors; near: within them
            const float t = key_score(prefix);
            float slack = 2.f * slack_sh[0] * slack_sh[1] * sum_slack(D);
            if (!(slack < INFINITY)) slack = 0.f;  // bounds or queries that are not finite: as they come
            const uint32_t hi = prefix == 0u ? 0u : score_key(t + slack), lo = prefix == 0u ? 0u : score_key(t - slack);
            for (int base = 0; base < n; base += kTopThreads * kTopItems) {
                if (!once) load(base);
                int sure = 0;
#pragma unroll
                for (int k = 0; k < kTopItems; ++k) {
                    const int b = base + k * kTopThreads + tid;
                    const bool in = (middle >> k) & 1u, is_sure = in && key[k] > hi, is_near = in && key[k] >= lo && key[k] <= hi;
                    const unsigned ms = __ballot_sync(0xffffffffu, is_sure), mn = __ballot_sync(0xffffffffu, is_near);
                    sure += __popc(ms);
                    if (lane == 0 && ms) atomicOr(&taken[b >> 5], ms);  // (a warp's 32 blocks are one word)
                    if (mn) {
                        int at = 0;
                        if (lane == 0) at = atomicAdd(&near_n, __popc(mn));
                        at = __shfl_sync(0xffffffffu, at, 0);
                        if (is_near) near_b[at + __popc(mn & ((1u << lane) - 1))] = b;
                    }
                }
                if (lane == 0 && sure) atomicAdd(&sure_n, sure);
            }
            __syncthreads();
            const int cand = near_n, left = want - sure_n;
            if (cand <= left) {
                for (int i = tid; i < cand; i += kTopThreads) atomicOr(&taken[near_b[i] >> 5], 1u << (near_b[i] & 31));
            } else {
                // exact keys of the blocks near the border (equal scores for sure: all alike)
                for (int i = warp; i < cand; i += kTopThreads / 32) {
                    const int phys = __ldg(a.bt + (long)it.s * a.mbps + near_b[i]);
                    double best = 0.0;
                    if (slack > 0.f && phys >= 0 && phys < a.num_blocks) {
                        const uint16_t* box = a.bounds + ((long)phys * a.Hkv + hk) * 2 * D;
                        for (int h = 0; h < g; ++h) {
                            const uint16_t* q = a.q + (at_row * a.Hq + hk * g + h) * D;
                            double sum = 0.0;
#pragma unroll
                            for (int c = lane; c < D; c += 32) {
                                const float x = __uint_as_float((uint32_t)__ldg(q + c) << 16);
                                // (a product of two bf16 numbers is exact in fp32, unless it leaves its range)
                                sum += (double)x * (double)__uint_as_float((uint32_t)__ldg(box + (x < 0.f ? c : D + c)) << 16);
                            }
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                            best = h == 0 || sum > best ? sum : best;
                        }
                    }
                    if (lane == 0) near_key[i] = score_key64(best);
                }
                __syncthreads();
                // the `left` largest, equal ones by block number
                if (cand <= kTopCount) {
                    for (int i = tid; i < cand; i += kTopThreads) {
                        const unsigned long long k = near_key[i];
                        const int b = near_b[i];
                        int before = 0;
                        for (int j = 0; j < cand; ++j) before += near_key[j] > k || (near_key[j] == k && near_b[j] < b);
                        if (before < left) atomicOr(&taken[b >> 5], 1u << (b & 31));
                    }
                } else {
                    // radix select over (key, ~block number), 8 bits at a time: distinct, so it ends with one
                    unsigned long long p0 = 0;
                    uint32_t p1 = 0;
                    int rest = left;
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
                                        digit_sel = 255 - 8 * lane - b;
                                        above_sel = above;
                                    }
                                    above += c;
                                }
                        }
                        __syncthreads();
                        for (int i = tid; i < 256; i += kTopThreads) hist[i] = 0;
                        if (pass < 8) p0 |= (unsigned long long)digit_sel << sh;
                        else p1 |= (uint32_t)digit_sel << sh1;
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
            __syncthreads();  // warp_sums is read
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
    const size_t ctas = (size_t)kTopCtasPerSm * 160;
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
                 num_seqs, max_blocks_per_seq, num_blocks, total_q, Hq, Hkv, keep, recent, sink, {}};
    if ((st = make_ctx(&a.ctx)) != FA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int launches = 0;
    if (max_blocks_per_seq > keep) {  // else every block is taken
        const int g = Hq / Hkv, per = g <= 16 ? 16 / g : 1;
        const long tiles = (std::min(max_q_len, total_q) + per - 1) / per;
        const long seg = (long)num_seqs * Hkv, groups = (max_blocks_per_seq + 7) / 8;
        const long z = std::min<long>((tiles + kScWarps - 1) / kScWarps, 64);
        const long side = tiles >= kScWarps ? 1 : kScWarps;  // about how many of a CTA's warps take groups of their own
        const long y = std::max<long>(1, std::min((groups + side - 1) / side, 8L * sm_count() / std::max<long>(1, seg * z)));
        const dim3 grid((unsigned)seg, (unsigned)std::min<long>(y, 65535), (unsigned)z);
        if (d == 128) block_score_kernel<128><<<grid, kScWarps * 32, 0, s>>>(a);
        else block_score_kernel<64><<<grid, kScWarps * 32, 0, s>>>(a);
        if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
        ++launches;
    }
    auto top = d == 128 ? block_top_kernel<128> : block_top_kernel<64>;
    if (bitmap + sizeof(int) * kTopBins > kUnraisedSmem &&
        (st = raise_dynamic_smem(reinterpret_cast<const void*>(top), (int)bitmap)) != FA_OK)
        return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<long>((long)total_q * Hkv, (long)kTopCtasPerSm * std::min(sm_count(), 160)));
    cfg.blockDim = dim3(kTopThreads);
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
