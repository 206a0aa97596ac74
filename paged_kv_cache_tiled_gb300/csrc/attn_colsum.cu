// Weight sums of chunks over the paged cache, on the tensor cores: for every
// key t of a sequence the softmax weight that the chunk's queries gave it,
//   acc_out[s][hk][t] = decay acc_in[s][hk][t] + sum_{rows r of the group} 2^(x_rt - lse_r),
// x the (modified) logits in log2 units and lse the final log-sum-exp of the
// attention that ran before.  acc_in counts as 0 for the chunk's own keys.
//
// The transposed product S^T = K Q^T puts a key in each TMEM lane and the query
// rows in the columns, so the sum over queries is a sum along a thread's own
// columns: no shuffles, no atomics, a fixed order.  Persistent CTAs (608 threads,
// one per SM) take units of 256 keys of one (sequence, kv head) from a ticket
// counter, chunks with many query tiles first.  A unit's two K tiles stay in
// shared memory while the query tiles that see it pass through a ring of two
// pairs; each pair (256 query rows), loaded once, meets both K tiles in two
// 128x256xd products.  Warps:
//   0-15  four summing warpgroups: warpgroup w = 2 kt + side owns TMEM columns
//         [128 w, 128 w + 128) and sums the products of K tile kt with query
//         tile `side` of every pair, while the tensor core works for the other K
//         tile; side 1 hands its sums to side 0 at the end of a unit;
//   16    TMA producer and ticket taker;  17  MMA issuer and TMEM owner;
//   18    looks up what the sums need of the query rows (-lse, slope, run of keys)
//         a pair or two ahead.
// Per logit the sum costs half a packed multiply-add, an exponential and half a
// packed add, against two passes over the scores in the attention itself.  The
// pace is the MMA warp's: 256 query rows per product, because eight MMAs of 128
// columns took 950 cycles to issue and each commit and barrier check 100 to 200.
// Eight chunks of up to 512 queries over up to 4600 keys (32 heads in 8 groups,
// d = 128): 59 us, the tensor pipe 42 % busy, the exponential unit 41 % (one CTA
// per 128 keys took 82 us, 128-row products in a persistent kernel 77).
#include <cmath>
#include <type_traits>

#include "host_common.cuh"

namespace fa {

constexpr int kCsThreads = 608;
constexpr int kCsProducer = 16, kCsMma = 17, kCsStats = 18;
constexpr int kCsReaders = 18;  // of a unit's mailbox: every warp but the producer
constexpr int kCsRows = 128;    // keys of a K tile, and query rows of a tile
constexpr int kCsPairs = 2, kCsUnitSlots = 4;  // query pairs in flight, unit mailboxes
constexpr float kCsLog2e = 1.4426950408889634f;
// CS_BIAS also caps when asked.  kWide variants: the cap is wider than kWideCap (the
// other form of tanh beside the first cost ordinary caps 3 % and caps with a bias 22 %).
enum { CS_PLAIN = 0, CS_CAP = 1, CS_BIAS = 2 };

struct ColsumParams {
    const int32_t* bt;
    const int32_t* ctx_lens;
    const int32_t* q_lens;
    const int32_t* q_start;
    const int32_t* k_start;  // [rank] first unit row (256 keys each) of the sequence k_seq[rank], then their number
    const int32_t* k_seq;    // sequences by decreasing number of query tiles
    int32_t* tickets;
    const float* lse;
    const float* acc_in;
    float* acc_out;
    int acc_len;
    float decay;
    int num_seqs, Hq, Hkv, g, pack, pack_shift, mbps, num_blocks, causal;
    float scale_log2;
    ScoreMod mod;
    CapPoly cap;
    DevCtx ctx;
};

template <int D>
struct CsCfg {
    static constexpr int kAtoms = D / 64;
    static constexpr int kAtomBytes = kCsRows * 128;
    static constexpr int kTileBytes = kAtoms * kAtomBytes;
    static constexpr uint32_t kGroup = kAtoms * 1024;  // 8-row groups of the K tile (halves side by side)
    static constexpr int kBars = 3 + 2 * kCsPairs + 4 + 4 + 2 * kCsUnitSlots + 2 + 2 * kCsPairs;
    // per query row of a pair: -lse, distance slope, end and first of the keys
    // seen, position from the unit's first key; then the largest -lse of each tile
    static constexpr int kColArrays = 5;
    static constexpr int kColBytes = kCsPairs * (kColArrays * 2 * kCsRows + 4) * 4;
    static constexpr int kPartBytes = 2 * kCsRows * 4;
    static constexpr int kSmem = 1024 + (2 + 2 * kCsPairs) * kTileBytes + kColBytes + kPartBytes + kBars * 8 +
                                 kCsUnitSlots * 16 + 16;
};

// Keys [lo, hi) that a query at `pos` sees.
__device__ __forceinline__ int2 cs_range(const ColsumParams& p, int pos, int prefix, int cl) {
    int lo = 0, hi = cl;
    if (p.causal)
        hi = max(pos + 1, prefix);
    else if (p.mod.window > 0)
        hi = pos + p.mod.window;
    if (p.mod.window > 0) lo = max(0, pos - p.mod.window + 1);
    return make_int2(lo, min(hi, cl));
}

// A unit as every role sees it: 256 keys from kv0 of (seq, hk), and the query
// tiles that see one of them.
struct CsUnit {
    int seq, hk, kv0, ql, cl, qs, pos0, prefix;
    int t_lo, n;   // first query tile, number of query tiles (times the heads when not packed)
    int nk;        // K tiles with keys: 1 or 2
};

__device__ __forceinline__ CsUnit cs_unit(const ColsumParams& p, int seq, int hk, int y, int tt, int heads) {
    CsUnit U;
    U.seq = seq;
    U.hk = hk;
    U.kv0 = y * 2 * kCsRows;
    U.ql = __ldg(p.q_lens + seq);
    U.cl = __ldg(p.ctx_lens + seq);
    U.qs = __ldg(p.q_start + seq);
    U.pos0 = U.cl - U.ql;
    U.prefix = p.causal && p.mod.prefix ? __ldg(p.mod.prefix + seq) : 0;
    U.nk = U.kv0 + kCsRows < U.cl ? 2 : 1;
    // Both ends of a row's run never decrease along the rows, so the tiles that
    // see a key of the unit are one run: from the first token whose run ends
    // behind the first key to the last whose run begins before the last one.
    const int kv_last = min(U.cl, U.kv0 + 2 * kCsRows) - 1, w = p.mod.window;
    const int tok_lo = p.causal ? (U.prefix > U.kv0 ? 0 : max(0, U.kv0 - U.pos0))
                                : (w > 0 ? max(0, U.kv0 - w + 1 - U.pos0) : 0);
    const int tok_hi = w > 0 ? min(U.ql - 1, kv_last + w - 1 - U.pos0) : U.ql - 1;
    const int ntok = (U.ql + tt - 1) / tt;
    U.t_lo = min(ntok, tok_lo / tt);
    U.n = (max(U.t_lo, tok_hi < 0 ? 0 : tok_hi / tt + 1) - U.t_lo) * heads;
    return U;
}

template <int D, int MOD, bool kWide>
__global__ void __launch_bounds__(kCsThreads, 1)
    attn_colsum_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const ColsumParams p) {
    using C = CsCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* kbuf = smem;
    uint8_t* qring = smem + 2 * C::kTileBytes;
    float* cols = reinterpret_cast<float*>(qring + 2 * kCsPairs * C::kTileBytes);
    float* part = cols + C::kColBytes / 4;  // [K tile][key]: side 1's sums
    uint64_t* kfull = reinterpret_cast<uint64_t*>(part + 2 * kCsRows);  // [2] K tile kt in
    uint64_t* kempty = kfull + 2;                                       // both read by the unit's last product
    uint64_t* qfull = kempty + 1;
    uint64_t* qempty = qfull + kCsPairs;
    uint64_t* sfull = qempty + kCsPairs;  // [2] a pair's product with K tile kt is complete
    uint64_t* sempty = sfull + 2;         // [2] its columns are in registers
    uint64_t* pfull = sempty + 2;         // [2] K tile kt's sums of side 1 are in `part`
    uint64_t* pempty = pfull + 2;         // [2] and read
    uint64_t* ufull = pempty + 2;
    uint64_t* uempty = ufull + kCsUnitSlots;
    uint64_t* cfull = uempty + kCsUnitSlots;  // [kCsPairs] a pair's row statistics are in
    uint64_t* cempty = cfull + kCsPairs;      // and read by every summing warp
    uint64_t* drain = cempty + kCsPairs;
    uint64_t* never = drain + 1;
    volatile int4* umbox = reinterpret_cast<volatile int4*>((reinterpret_cast<uintptr_t>(never + 1) + 15) & ~uintptr_t(15));
    uint32_t* tmem_slot = const_cast<uint32_t*>(reinterpret_cast<volatile uint32_t*>(umbox + kCsUnitSlots));
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(kempty, 1);
        for (int i = 0; i < kCsPairs; ++i) {
            mbar_init(&qfull[i], 1);
            mbar_init(&qempty[i], 1);
            mbar_init(&cfull[i], 1);
            mbar_init(&cempty[i], 16);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(&kfull[k], 1);
            mbar_init(&sfull[k], 1);
            mbar_init(&sempty[k], 2 * kCsRows);
            mbar_init(&pfull[k], kCsRows);
            mbar_init(&pempty[k], kCsRows);
        }
        for (int k = 0; k < kCsUnitSlots; ++k) {
            mbar_init(&ufull[k], 1);
            mbar_init(&uempty[k], kCsReaders);
        }
        mbar_init(drain, 1);
        mbar_init(never, 1);
        *abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
    }
    if (warp == kCsMma) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_slot;
    const unsigned long long lim_ns = p.ctx.wait_ns;
    // query tiles: `tt` tokens of all heads of the group (packed) or of one head
    const int tt = p.pack ? kCsRows >> p.pack_shift : kCsRows;
    const int heads = p.pack ? 1 : p.g;
    auto fail = [&]() {
        raise_error(p.ctx, ERR_TIMEOUT_BIT);
        *abort_flag = 1;
    };
    // the i-th unit of this CTA, as the producer published it; seq < 0: no more
    auto next_unit = [&](int i, int4& u) -> bool {
        const int k = i % kCsUnitSlots;
        if (!mbar_wait_warp(&ufull[k], (i / kCsUnitSlots) & 1, lim_ns, abort_flag)) return false;
        u.x = umbox[k].x;
        u.y = umbox[k].y;
        u.z = umbox[k].z;
        __syncwarp();
        if (lane == 0) mbar_arrive(&uempty[k]);
        return true;
    };

    bool ok = !p.ctx.force_timeout || mbar_wait_warp(never, 0, lim_ns, abort_flag);
    if (warp == kCsProducer) {
        int kf[2] = {0, 0}, ku = 0, qf = 0;  // K tiles, units with products and query pairs requested
        const int rows = __ldg(p.k_start + p.num_seqs);
        int ticket = 0;
        if (lane == 0) ticket = atomicAdd(p.tickets, 1);
        for (int i = 0; ok; ++i) {
            // unit t: kv head t % Hkv of unit row t / Hkv (the heads of a row side by side);
            // the ticket was asked for before the last unit's query tiles
            const int t = __shfl_sync(0xffffffffu, ticket, 0);
            int seq = -1, y = 0;
            if ((long)t < (long)rows * p.Hkv) {
                const int row = t / p.Hkv;
                int lo = 0, hi = p.num_seqs - 1;  // last sequence whose first row is not behind `row`
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (__ldg(p.k_start + mid) <= row) lo = mid;
                    else hi = mid - 1;
                }
                seq = __ldg(p.k_seq + lo);
                y = row - __ldg(p.k_start + lo);
            }
            const int k = i % kCsUnitSlots;
            if (i >= kCsUnitSlots && !mbar_wait_warp(&uempty[k], ((i / kCsUnitSlots) - 1) & 1, lim_ns, abort_flag)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                umbox[k].x = seq;
                umbox[k].y = t % p.Hkv;
                umbox[k].z = y;
                mbar_arrive(&ufull[k]);
            }
            __syncwarp();
            if (seq < 0) break;
            if (lane == 0) ticket = atomicAdd(p.tickets, 1);
            const CsUnit U = cs_unit(p, seq, t % p.Hkv, y, tt, heads);
            if (U.n == 0) continue;
            // lane j < 16: the unit's j-th block (blocks that no query of the chunk sees are not read)
            int blk = p.num_blocks;  // outside the map: zeros
            const int tok = U.kv0 + lane * 16;
            if (lane < 16 && tok < U.cl && (p.mod.window == 0 || tok + 16 > U.pos0 - p.mod.window + 1)) {
                const int b = __ldg(p.bt + (long)seq * p.mbps + tok / 16);
                if (b < 0 || b >= p.num_blocks) raise_error(p.ctx, ERR_BOUNDS_BIT);
                else blk = b;
            }
            // pair jj: tiles 2 jj and 2 jj + 1, laid out [64-channel half][256 rows][128 B]
            auto request_pair = [&](int jj) {
                const int st = qf % kCsPairs, tiles = min(2, U.n - 2 * jj);
                if (!mbar_wait_warp(&qempty[st], ((qf / kCsPairs) & 1) ^ 1, lim_ns, abort_flag)) {
                    ok = false;
                    return;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&qfull[st], tiles * C::kTileBytes);
                    for (int e = 0; e < tiles; ++e) {
                        const int j = 2 * jj + e;
#pragma unroll
                        for (int a = 0; a < C::kAtoms; ++a)
                            tma_load_4d(qring + st * 2 * C::kTileBytes + (2 * a + e) * C::kAtomBytes, &tm_q, &qfull[st],
                                        a * 64, U.hk * p.g + j % heads, U.qs + (U.t_lo + j / heads) * tt, 0);
                    }
                }
                __syncwarp();
                ++qf;
            };
            request_pair(0);  // before the K tiles, whose places are free only when the unit before is done
            if (!ok || !mbar_wait_warp(kempty, (ku & 1) ^ 1, lim_ns, abort_flag)) {
                ok = false;
                break;
            }
            ++ku;
#pragma unroll
            for (int kt = 0; kt < 2; ++kt) {
                if (kt >= U.nk) continue;
                if (lane == 0) mbar_arrive_expect_tx(&kfull[kt], C::kTileBytes);
                __syncwarp();
                if (lane >= 8 * kt && lane < 8 * kt + 8) {
                    uint8_t* dst = kbuf + kt * C::kTileBytes;
                    if constexpr (D == 128)
                        tma_load_5d(dst + (lane & 7) * 4096, &tm_k, &kfull[kt], 0, 0, 0, 0, blk * p.Hkv + U.hk);
                    else
                        tma_load_4d(dst + (lane & 7) * 2048, &tm_k, &kfull[kt], 0, 0, U.hk, blk);
                }
                __syncwarp();
                ++kf[kt];
            }
            for (int jj = 1; 2 * jj < U.n && ok; ++jj) request_pair(jj);
        }
        if (!ok) {
            if (lane == 0) fail();
            // the copies already issued land before the CTA exits
            for (int kt = 0; kt < 2; ++kt)
                if (kf[kt] > 0) (void)mbar_wait_warp(&kfull[kt], (kf[kt] - 1) & 1, 1000000000ull, nullptr);
            for (int f = max(0, qf - kCsPairs); f < qf; ++f)
                (void)mbar_wait_warp(&qfull[f % kCsPairs], (f / kCsPairs) & 1, 1000000000ull, nullptr);
        }
    } else if (warp == kCsMma) {
        constexpr uint32_t kIdesc1 = idesc_bf16_f32(128, 128, 0, 0), kIdesc2 = idesc_bf16_f32(128, 256, 0, 0);
        const uint32_t k_addr = smem_u32(kbuf), q_addr = smem_u32(qring);
        int kc[2] = {0, 0}, qc = 0, sc[2] = {0, 0};  // K tiles and pairs consumed, products issued per K tile
        for (int i = 0; ok; ++i) {
            int4 u;
            if (!next_unit(i, u)) {
                ok = false;
                break;
            }
            if (u.x < 0) break;
            const CsUnit U = cs_unit(p, u.x, u.y, u.z, tt, heads);
            if (U.n == 0) continue;
            for (int j = 0; j < U.n && ok; j += 2) {
                const int st = qc % kCsPairs;
                // the pair and both products' buffers are probed together: three checks in
                // flight cost about one
                uint32_t rdy[3];
                mbar_test3(&qfull[st], (qc / kCsPairs) & 1, &sempty[0], (sc[0] & 1) ^ 1, &sempty[1], (sc[1] & 1) ^ 1, rdy);
                if (!__all_sync(0xffffffffu, rdy[0]) &&
                    !mbar_wait_warp(&qfull[st], (qc / kCsPairs) & 1, lim_ns, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint64_t qd = smem_desc_sw128(q_addr + st * 2 * C::kTileBytes, 16, 1024);
                const uint32_t idesc = j + 1 < U.n ? kIdesc2 : kIdesc1;
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) {
                    if (kt >= U.nk || !ok) continue;
                    if (j == 0 && !mbar_wait_warp(&kfull[kt], kc[kt] & 1, lim_ns, abort_flag)) {
                        ok = false;
                        continue;
                    }
                    const bool free_buf = __all_sync(0xffffffffu, rdy[1 + kt]);
                    if (!free_buf && !mbar_wait_warp(&sempty[kt], (sc[kt] & 1) ^ 1, lim_ns, abort_flag)) {
                        ok = false;
                        continue;
                    }
                    tc_fence_after();
                    if (lane == 0) {
                        const uint64_t kd = smem_desc_sw128(k_addr + kt * C::kTileBytes, 16, C::kGroup);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t koff = ((kk >> 2) * 1024 + (kk & 3) * 32) >> 4;
                            const uint32_t qoff = ((kk >> 2) * 2 * C::kAtomBytes + (kk & 3) * 32) >> 4;
                            umma_ss(tbase + kt * 256, kd + koff, qd + qoff, idesc, kk > 0);
                        }
                        umma_commit(&sfull[kt]);
                    }
                    __syncwarp();
                    ++sc[kt];
                }
                if (!ok) break;
                if (lane == 0) {
                    umma_commit(&qempty[st]);
                    if (j + 2 >= U.n) umma_commit(kempty);
                }
                __syncwarp();
                ++qc;
            }
            if (!ok) break;
            ++kc[0];
            if (U.nk > 1) ++kc[1];
        }
        if (!ok && lane == 0) fail();
        // every product issued above completes before TMEM is released
        if (lane == 0) umma_commit(drain);
        __syncwarp();
        (void)mbar_wait_bounded(drain, 0, 1000000000ull, nullptr);
    } else if (warp == kCsStats) {
        int cc = 0;  // pairs described
        for (int i = 0; ok; ++i) {
            int4 u;
            if (!next_unit(i, u)) {
                ok = false;
                break;
            }
            if (u.x < 0) break;
            const CsUnit U = cs_unit(p, u.x, u.y, u.z, tt, heads);
            int tile = U.t_lo, head = 0;  // of the pair's first tile
            for (int j = 0; j < U.n; j += 2, ++cc) {
                const int slot = cc % kCsPairs;
                float lse[8], sl[8], at[8];
                int2 seen[8];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const int c = b * 32 + lane;
                        const int tok = tile * tt + (p.pack ? c >> p.pack_shift : c);
                        const int hd = U.hk * p.g + head + (p.pack ? c & (p.g - 1) : 0);
                        const bool real = j + e < U.n && tok < U.ql;
                        lse[4 * e + b] = real ? __ldg(p.lse + (long)(U.qs + tok) * p.Hq + hd) : 0.f;
                        if constexpr (MOD == CS_BIAS) {
                            sl[4 * e + b] = -slope_log2(__ldg(p.mod.slopes + hd));
                            at[4 * e + b] = (float)(U.pos0 + tok - U.kv0);
                        }
                        seen[4 * e + b] = real ? cs_range(p, U.pos0 + tok, U.prefix, U.cl) : make_int2(0, 0);
                    }
                    if (++head == heads) {
                        head = 0;
                        ++tile;
                    }
                }
                if (!mbar_wait_warp(&cempty[slot], ((cc / kCsPairs) & 1) ^ 1, lim_ns, abort_flag)) {
                    ok = false;
                    break;
                }
                float* nlse = cols + slot * (C::kColArrays * 2 * kCsRows + 4);
                float* slope = nlse + 2 * kCsRows;
                int* end = reinterpret_cast<int*>(slope + 2 * kCsRows);
                int* first = end + 2 * kCsRows;
                float* rel = reinterpret_cast<float*>(first + 2 * kCsRows);
                float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int c = k * 32 + lane;
                    const float nl = lse[k] == -INFINITY ? 0.f : -lse[k] * kCsLog2e;
                    nlse[c] = nl;
                    if (seen[k].y > 0) most[k >> 2] = fmaxf(most[k >> 2], nl);  // (rows that exist)
                    if constexpr (MOD == CS_BIAS) {
                        slope[c] = sl[k];
                        rel[c] = at[k];
                    }
                    end[c] = seen[k].y;
                    first[c] = seen[k].x;
                }
                if constexpr (MOD == CS_CAP) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) most[e] = fmaxf(most[e], __shfl_xor_sync(0xffffffffu, most[e], o));
                        if (lane == 0) rel[2 * kCsRows + e] = most[e];
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&cfull[slot]);
            }
        }
        if (!ok && lane == 0) fail();
    } else {
        const int w = warp >> 2, kt = w >> 1, side = w & 1, quarter = warp & 3;
        const uint32_t trow = tbase + ((uint32_t)(quarter * 32) << 16) + w * 128;
        int sc = 0, cc = 0, handed = 0;  // products seen, pairs seen, sums handed over
        for (int i = 0; ok; ++i) {
            int4 u;
            if (!next_unit(i, u)) {
                ok = false;
                break;
            }
            if (u.x < 0) break;
            const CsUnit U = cs_unit(p, u.x, u.y, u.z, tt, heads);
            const int k_rel = kt * kCsRows + quarter * 32;  // this warp's keys within the unit
            const int k_lo = U.kv0 + k_rel, k_hi = min(U.cl, k_lo + 32), key = k_lo + lane;
            [[maybe_unused]] const float key_rel = (float)(k_rel + lane);  // from the unit's first key
            float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            int tile = U.t_lo + side / heads, head = side % heads;
            for (int j = side; j - side < U.n; j += 2, ++cc) {
                const int slot = cc % kCsPairs;
                if (!mbar_wait_warp(&cfull[slot], (cc / kCsPairs) & 1, lim_ns, abort_flag)) {
                    ok = false;
                    break;
                }
                auto done = [&]() {  // the pair's statistics are read
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&cempty[slot]);
                };
                if (kt >= U.nk) {  // no such K tile
                    done();
                    continue;
                }
                const int tok0 = tile * tt;
                // Warp-uniform: does every row of the tile exist and see every key of this warp
                // (plain), or no row any of them (none)?
                const int2 rf = cs_range(p, U.pos0 + tok0, U.prefix, U.cl);
                const int2 rl = cs_range(p, U.pos0 + min(U.ql, tok0 + tt) - 1, U.prefix, U.cl);
                const bool plain = tok0 + tt <= U.ql && k_lo >= rl.x && k_hi <= rf.y;
                const bool none = j >= U.n || k_lo >= rl.y || k_hi <= rf.x;  // (a last pair may have one tile)
                const float* nlse = cols + slot * (C::kColArrays * 2 * kCsRows + 4) + side * kCsRows;
                const float* slope = nlse + 2 * kCsRows;
                const int* end = reinterpret_cast<const int*>(slope + 2 * kCsRows);
                const int* first = end + 2 * kCsRows;
                const float* rel = reinterpret_cast<const float*>(first + 2 * kCsRows);
                // CapPoly's slack: the smallest lse of the tile stands for the running max
                [[maybe_unused]] float low = 0.f;
                if constexpr (MOD == CS_CAP) low = -rel[2 * kCsRows - side * (kCsRows - 1)];
                if (!mbar_wait_warp(&sfull[kt], sc & 1, lim_ns, abort_flag)) {
                    ok = false;
                    break;
                }
                ++sc;
                tc_fence_after();
                // 32 columns at a time, the next ones on their way while these are summed;
                // `masked`: 1 some row of the tile is not real or does not see some key, 2 and runs may begin
                // behind the first key.  Row ends come four at a time: packed into one word per row
                // their unpacking took a masked tile from 1800 cycles to 8000.
                auto columns = [&](auto masked) {
                    constexpr int kAhead = MOD == CS_PLAIN ? 1 : 0;  // (registers: 96 a thread)
                    uint32_t raw[1 + kAhead][32];
                    if constexpr (kAhead) tmem_ld32(trow, raw[0]);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if constexpr (!kAhead) tmem_ld32(trow + b * 32, raw[0]);
                        tmem_wait_ld();
                        if (b < 3) {
                            if constexpr (kAhead) tmem_ld32(trow + (b + 1) * 32, raw[(b + 1) & kAhead]);
                        } else {  // every column is in registers: the buffer is free
                            tc_fence_before();
                            mbar_arrive(&sempty[kt]);
                        }
                        [[maybe_unused]] int tier = 2;
                        if constexpr (MOD == CS_CAP) {
                            float mz[2] = {0.f, 0.f};
#pragma unroll
                            for (int jj = 0; jj < 32; jj += 2)
                                mz[(jj >> 1) & 1] = fmax3f(mz[(jj >> 1) & 1], __uint_as_float(raw[0][jj]),
                                                           __uint_as_float(raw[0][jj + 1]));
                            const float z = fmaxf(mz[0], mz[1]);
                            if (__all_sync(0xffffffffu, z <= p.cap.near_max && low + p.cap.near_slack >= 30.f)) tier = 0;
                            else if (__all_sync(0xffffffffu, z <= p.cap.unit_max && low + p.cap.unit_slack >= 30.f)) tier = 1;
                        }
                        auto sum_block = [&](auto form) {
#pragma unroll
                            for (int jj = 0; jj < 32; jj += 4) {
                                const float4 nl = *reinterpret_cast<const float4*>(nlse + b * 32 + jj);
                                const float nls[4] = {nl.x, nl.y, nl.z, nl.w};
                                [[maybe_unused]] int4 he = make_int4(0, 0, 0, 0), fe = he;
                                if constexpr (decltype(masked)::value >= 1) he = *reinterpret_cast<const int4*>(end + b * 32 + jj);
                                if constexpr (decltype(masked)::value == 2)
                                    fe = *reinterpret_cast<const int4*>(first + b * 32 + jj);
#pragma unroll
                                for (int e = 0; e < 4; e += 2) {
                                    const int c = b * 32 + jj + e;
                                    float2 x = make_float2(__uint_as_float(raw[b & kAhead][jj + e]),
                                                           __uint_as_float(raw[b & kAhead][jj + e + 1]));
                                    const float2 l2 = make_float2(nls[e], nls[e + 1]);
                                    if constexpr (MOD == CS_CAP && decltype(form)::value < 2) {
                                        constexpr int top = decltype(form)::value == 0 ? 4 : 6;
                                        const float2* co = decltype(form)::value == 0 ? p.cap.near : p.cap.unit;
                                        const float2 q2 = __fmul2_rn(x, x);
                                        float2 t = __ffma2_rn(co[top], q2, co[top - 1]);
#pragma unroll
                                        for (int k = top - 2; k >= 0; --k) t = __ffma2_rn(t, q2, co[k]);
                                        x = __ffma2_rn(x, t, l2);
                                    } else if (MOD == CS_CAP || (MOD == CS_BIAS && p.mod.cap_out > 0.f)) {
                                        auto tanh_of = [](float u) { return kWide ? tanh_f32(u) : tanh_abs(u); };
                                        x.x = fmaf(p.mod.cap_out, tanh_of(x.x * p.mod.cap_in), l2.x);
                                        x.y = fmaf(p.mod.cap_out, tanh_of(x.y * p.mod.cap_in), l2.y);
                                    } else {
                                        x = __ffma2_rn(x, make_float2(p.scale_log2, p.scale_log2), l2);
                                    }
                                    if constexpr (MOD == CS_BIAS) {
                                        const float2 sl = *reinterpret_cast<const float2*>(slope + c);
                                        const float2 at = *reinterpret_cast<const float2*>(rel + c);
                                        x.x = fmaf(sl.x, fabsf(key_rel - at.x), x.x);
                                        x.y = fmaf(sl.y, fabsf(key_rel - at.y), x.y);
                                    }
                                    float2 pr = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                                    if constexpr (decltype(masked)::value >= 1) {
                                        pr.x = key < (e ? he.z : he.x) ? pr.x : 0.f;
                                        pr.y = key < (e ? he.w : he.y) ? pr.y : 0.f;
                                    }
                                    if constexpr (decltype(masked)::value == 2) {
                                        pr.x = key >= (e ? fe.z : fe.x) ? pr.x : 0.f;
                                        pr.y = key >= (e ? fe.w : fe.y) ? pr.y : 0.f;
                                    }
                                    sum[(c >> 1) & 3] = __fadd2_rn(sum[(c >> 1) & 3], pr);
                                }
                            }
                        };
                        if constexpr (MOD == CS_CAP) {
                            if (tier == 0) sum_block(std::integral_constant<int, 0>{});
                            else if (tier == 1) sum_block(std::integral_constant<int, 1>{});
                            else sum_block(std::integral_constant<int, 2>{});
                        } else {
                            sum_block(std::integral_constant<int, 2>{});
                        }
                    }
                };
                if (none) {
                    mbar_arrive(&sempty[kt]);
                } else if (plain) {
                    columns(std::integral_constant<int, 0>{});
                } else if (p.mod.window == 0) {
                    columns(std::integral_constant<int, 1>{});
                } else {
                    columns(std::integral_constant<int, 2>{});
                }
                done();
                for (head += 2; head >= heads; head -= heads) ++tile;
            }
            if (!ok) break;
            if (kt >= U.nk) continue;
            const float mine =
                ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) + ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y));
            float* at = part + kt * kCsRows + quarter * 32 + lane;
            if (side == 1) {
                if (!mbar_wait_warp(&pempty[kt], (handed & 1) ^ 1, lim_ns, abort_flag)) {
                    ok = false;
                    break;
                }
                *at = mine;
                mbar_arrive(&pfull[kt]);
            } else {
                if (!mbar_wait_warp(&pfull[kt], handed & 1, lim_ns, abort_flag)) {
                    ok = false;
                    break;
                }
                const float odd = *at;
                mbar_arrive(&pempty[kt]);
                if (key < U.cl) {
                    const long o = ((long)U.seq * p.Hkv + U.hk) * p.acc_len + key;
                    const float old = p.acc_in && key < U.pos0 ? p.decay * p.acc_in[o] : 0.f;
                    p.acc_out[o] = old + (mine + odd);
                }
            }
            ++handed;
        }
        if (!ok && lane == 0) fail();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kCsMma) tmem_dealloc(tbase, 512);
}

template <int D, int MOD, bool kWide = false>
static fa_status launch_colsum(const CUtensorMap& tq, const CUtensorMap& tk, const ColsumParams& p, int grid,
                               cudaStream_t s) {
    const fa_status st =
        raise_dynamic_smem(reinterpret_cast<const void*>(attn_colsum_kernel<D, MOD, kWide>), CsCfg<D>::kSmem);
    if (st != FA_OK) return st;
    attn_colsum_kernel<D, MOD, kWide><<<grid, kCsThreads, CsCfg<D>::kSmem, s>>>(tq, tk, p);
    return cuda_status(cudaGetLastError());
}

// Weight sums of the sequences whose chunks took the tensor-core path.
fa_status launch_accum_chunk(const void* q, const void* k_cache, const int32_t* block_table, const int32_t* ctx_lens,
                             const int32_t* q_lens, const int32_t* q_start, const int32_t* k_start,
                             const int32_t* k_seq, int32_t* tickets, const float* lse, const float* acc_in,
                             float* acc_out, int acc_len, float decay, int num_seqs, int mbps, int num_blocks, int Hq,
                             int Hkv, int d, int causal, float scale, int total_q, const ScoreMod& mod, cudaStream_t s,
                             const DevCtx& ctx) {
    CUtensorMap tq, tk;
    fa_status st = paged_query_map(&tq, q, Hq, Hkv, d, total_q);
    if (st == FA_OK) st = paged_cache_map(&tk, k_cache, num_blocks, Hkv, d);
    if (st != FA_OK) return st;
    ColsumParams p{};
    p.bt = block_table;
    p.ctx_lens = ctx_lens;
    p.q_lens = q_lens;
    p.q_start = q_start;
    p.k_start = k_start;
    p.k_seq = k_seq;
    p.tickets = tickets;
    p.num_seqs = num_seqs;
    p.lse = lse;
    p.acc_in = acc_in;
    p.acc_out = acc_out;
    p.acc_len = acc_len;
    p.decay = decay;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.g = Hq / Hkv;
    p.pack = paged_tc_pack(p.g) ? 1 : 0;
    p.pack_shift = p.pack ? __builtin_ctz((unsigned)p.g) : 0;
    p.mbps = mbps;
    p.num_blocks = num_blocks;
    p.causal = causal;
    p.scale_log2 = scale * kCsLog2e;
    p.mod = mod;
    if (mod.cap_out > 0.f) p.cap = cap_poly(mod);
    p.ctx = ctx;
    const int grid = sm_count();
    auto go = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        if (mod.slopes)
            return p.cap.wide ? launch_colsum<D, CS_BIAS, true>(tq, tk, p, grid, s) : launch_colsum<D, CS_BIAS>(tq, tk, p, grid, s);
        if (mod.cap_out > 0.f)
            return p.cap.wide ? launch_colsum<D, CS_CAP, true>(tq, tk, p, grid, s) : launch_colsum<D, CS_CAP>(tq, tk, p, grid, s);
        return launch_colsum<D, CS_PLAIN>(tq, tk, p, grid, s);
    };
    return d == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 64>{});
}

}  // namespace fa
