// Weight sums of chunks over the paged cache, on the tensor cores: for every
// key t of a sequence the softmax weight that the chunk's queries gave it,
//   acc_out[s][hk][t] = decay acc_in[s][hk][t] + sum_{rows r of the group} 2^(x_rt - lse_r),
// x the (modified) logits in log2 units and lse the final log-sum-exp of the
// attention that ran before.  acc_in counts as 0 for the chunk's own keys.
//
// The transposed product S^T = K Q^T puts a key in each TMEM lane and the query
// rows in the columns, so the sum over queries is a sum along a thread's own
// columns: no shuffles, no atomics, a fixed order.  A CTA owns 128 keys of one
// (sequence, kv head): its K tile stays in shared memory while the group's
// query tiles pass through a ring of two stages, each answered by one
// 128x128xd product into one of two TMEM buffers; warpgroup w sums the tiles of
// parity w while the tensor core fills the other buffer.  Two CTAs share an SM
// (96 KB of tiles and half of the TMEM each), so one's set-up hides behind the
// other's work.  Per logit the sum costs one multiply-add, one exponential and
// one add, against two passes over the scores in the attention itself.
#include <cmath>
#include <type_traits>

#include "host_common.cuh"

namespace fa {

constexpr int kCsThreads = 320;  // two summing warpgroups, the TMA producer, the MMA issuer
constexpr int kCsProducer = 8, kCsMma = 9;
constexpr int kCsRows = 128;  // keys of a CTA, and query rows of a tile
constexpr int kCsStages = 2;
constexpr float kCsLog2e = 1.4426950408889634f;
enum { CS_PLAIN = 0, CS_CAP = 1, CS_BIAS = 2 };  // CS_BIAS also caps when asked

struct ColsumParams {
    const int32_t* bt;
    const int32_t* ctx_lens;
    const int32_t* q_lens;
    const int32_t* q_start;
    const float* lse;
    const float* acc_in;
    float* acc_out;
    int acc_len;
    float decay;
    int Hq, Hkv, g, pack, pack_shift, mbps, num_blocks, causal;
    float scale_log2;
    ScoreMod mod;
    DevCtx ctx;
};

template <int D>
struct CsCfg {
    static constexpr int kAtoms = D / 64;
    static constexpr int kAtomBytes = kCsRows * 128;
    static constexpr int kTileBytes = kAtoms * kAtomBytes;
    static constexpr uint32_t kGroup = kAtoms * 1024;  // 8-row groups of the K tile (halves side by side)
    static constexpr int kBars = 1 + 2 * kCsStages + 4 + 2;
    // per summing warp and column: -lse, distance slope, run of keys seen (each warp keeps its own, so no barrier across
    // warps is needed in the loop)
    static constexpr int kColBytes = 8 * 3 * kCsRows * 4;
    static constexpr int kSmem = 1024 + (1 + kCsStages) * kTileBytes + kColBytes + kCsRows * 4 + kBars * 8 + 16;
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

template <int D, int MOD>
__global__ void __launch_bounds__(kCsThreads, 2)
    attn_colsum_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const ColsumParams p) {
    using C = CsCfg<D>;
    const int seq = blockIdx.x / p.Hkv, hk = blockIdx.x % p.Hkv, kv0 = blockIdx.y * kCsRows;
    const int ql = __ldg(p.q_lens + seq), cl = __ldg(p.ctx_lens + seq);
    // decode rows (at most 16 packed rows) are summed from their kept logits
    if (ql <= 0 || p.g * ql <= 16 || ql > cl || cl > p.mbps * 16 || kv0 >= cl) return;
    if (cl > p.acc_len) {
        if (threadIdx.x == 0) raise_error(p.ctx, ERR_BOUNDS_BIT);
        return;
    }
    const int qs = __ldg(p.q_start + seq), pos0 = cl - ql;
    const int prefix = p.causal && p.mod.prefix ? __ldg(p.mod.prefix + seq) : 0;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* kbuf = smem;
    uint8_t* qring = smem + C::kTileBytes;
    float* cols = reinterpret_cast<float*>(qring + kCsStages * C::kTileBytes);
    float* part = cols + C::kColBytes / 4;
    uint64_t* kfull = reinterpret_cast<uint64_t*>(part + kCsRows);
    uint64_t* qfull = kfull + 1;
    uint64_t* qempty = qfull + kCsStages;
    uint64_t* sfull = qempty + kCsStages;  // [2] product of parity w complete
    uint64_t* sempty = sfull + 2;          // [2] its columns read
    uint64_t* drain = sempty + 2;
    uint64_t* never = drain + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(kfull, 1);
        for (int i = 0; i < kCsStages; ++i) {
            mbar_init(&qfull[i], 1);
            mbar_init(&qempty[i], 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(&sfull[w], 1);
            mbar_init(&sempty[w], kCsRows);
        }
        mbar_init(drain, 1);
        mbar_init(never, 1);
        *abort_flag = 0;
        mbar_fence_init();
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
    }
    if (warp == kCsMma) {
        tmem_alloc(tmem_slot, 256);
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
    const int ntok = (ql + tt - 1) / tt;
    const int kv_last = min(cl, kv0 + kCsRows) - 1;
    // token tiles that see a key of this CTA: both ends of a row's run never
    // decrease along the rows, so they are one run [t_lo, t_hi).  First token
    // whose run ends behind the first key, last token whose run begins before
    // the last one:
    const int w_ = p.mod.window;
    const int tok_lo = p.causal ? (prefix > kv0 ? 0 : max(0, kv0 - pos0)) : (w_ > 0 ? max(0, kv0 - w_ + 1 - pos0) : 0);
    const int tok_hi = w_ > 0 ? min(ql - 1, kv_last + w_ - 1 - pos0) : ql - 1;
    const int t_lo = min(ntok, tok_lo / tt), t_hi = max(t_lo, tok_hi < 0 ? 0 : tok_hi / tt + 1);
    const int n = (t_hi - t_lo) * heads;
    auto fail = [&]() {
        raise_error(p.ctx, ERR_TIMEOUT_BIT);
        *abort_flag = 1;
    };

    float mine = 0.f;  // summing warps: this thread's key over its warpgroup's tiles
    bool ok = !p.ctx.force_timeout || mbar_wait_warp(never, 0, lim_ns, abort_flag);
    if (warp == kCsProducer) {
        int issued = 0;
        bool k_out = false;
        if (ok && n > 0) {
            int blk = p.num_blocks;  // outside the map: zeros
            if (lane < 8 && kv0 + lane * 16 < cl) {
                const int b = __ldg(p.bt + (long)seq * p.mbps + kv0 / 16 + lane);
                const int tok = kv0 + lane * 16;
                // blocks that no query of the chunk sees are not read
                const bool seen = p.mod.window == 0 || tok + 16 > pos0 - p.mod.window + 1;
                if (seen) {
                    if (b < 0 || b >= p.num_blocks)
                        raise_error(p.ctx, ERR_BOUNDS_BIT);
                    else
                        blk = b;
                }
            }
            if (lane == 0) mbar_arrive_expect_tx(kfull, C::kTileBytes);
            __syncwarp();
            if (lane < 8) {
                if constexpr (D == 128)
                    tma_load_5d(kbuf + lane * 4096, &tm_k, kfull, 0, 0, 0, 0, blk * p.Hkv + hk);
                else
                    tma_load_4d(kbuf + lane * 2048, &tm_k, kfull, 0, 0, hk, blk);
            }
            __syncwarp();
            k_out = true;
            for (; issued < n; ++issued) {
                const int st = issued % kCsStages;
                if (!mbar_wait_warp(&qempty[st], ((issued / kCsStages) & 1) ^ 1, lim_ns, abort_flag)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const int tile = t_lo + issued / heads, h = hk * p.g + issued % heads;
                    mbar_arrive_expect_tx(&qfull[st], C::kTileBytes);
#pragma unroll
                    for (int a = 0; a < C::kAtoms; ++a)
                        tma_load_4d(qring + st * C::kTileBytes + a * C::kAtomBytes, &tm_q, &qfull[st], a * 64, h,
                                    qs + tile * tt, 0);
                }
                __syncwarp();
            }
        }
        if (!ok) {
            if (lane == 0) fail();
            // the copies already issued land before the CTA exits
            if (k_out) (void)mbar_wait_warp(kfull, 0, 1000000000ull, nullptr);
            for (int f = max(0, issued - kCsStages); f < issued; ++f)
                (void)mbar_wait_warp(&qfull[f % kCsStages], (f / kCsStages) & 1, 1000000000ull, nullptr);
        }
    } else if (warp == kCsMma) {
        constexpr uint32_t kIdesc = idesc_bf16_f32(128, 128, 0, 0);
        const uint32_t k_addr = smem_u32(kbuf), q_addr = smem_u32(qring);
        if (ok && n > 0 && !mbar_wait_warp(kfull, 0, lim_ns, abort_flag)) ok = false;
        for (int i = 0; ok && i < n; ++i) {
            const int st = i % kCsStages, w = i & 1;
            if (!mbar_wait_warp(&qfull[st], (i / kCsStages) & 1, lim_ns, abort_flag) ||
                !mbar_wait_warp(&sempty[w], ((i >> 1) & 1) ^ 1, lim_ns, abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (lane == 0) {
                const uint64_t kd = smem_desc_sw128(k_addr, 16, C::kGroup);
                const uint64_t qd = smem_desc_sw128(q_addr + st * C::kTileBytes, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t koff = ((kk >> 2) * 1024 + (kk & 3) * 32) >> 4;
                    const uint32_t qoff = ((kk >> 2) * C::kAtomBytes + (kk & 3) * 32) >> 4;
                    umma_ss(tbase + w * 128, kd + koff, qd + qoff, kIdesc, kk > 0);
                }
                umma_commit(&qempty[st]);
                umma_commit(&sfull[w]);
            }
            __syncwarp();
        }
        if (!ok && lane == 0) fail();
        // every product issued above completes before TMEM is released
        if (lane == 0) umma_commit(drain);
        __syncwarp();
        (void)mbar_wait_bounded(drain, 0, 1000000000ull, nullptr);
    } else {
        const int w = warp >> 2, quarter = warp & 3;
        const uint32_t trow = tbase + ((uint32_t)(quarter * 32) << 16) + w * 128;
        float* nlse = cols + warp * 3 * kCsRows;
        float* slope = nlse + kCsRows;
        short2* run = reinterpret_cast<short2*>(slope + kCsRows);  // from this warp's first key
        float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const int k_lo = kv0 + quarter * 32, k_hi = min(cl, k_lo + 32);  // this warp's keys
        for (int i = w; ok && i < n; i += 2) {
            const int tile = t_lo + i / heads, h0 = hk * p.g + i % heads, tok0 = tile * tt;
            // statistics of the tile's columns (query rows): four per lane
            __syncwarp();
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int c = b * 32 + lane;
                const int tok = tok0 + (p.pack ? c >> p.pack_shift : c);
                const int head = h0 + (p.pack ? c & (p.g - 1) : 0);
                float L = 0.f;
                if (tok < ql) {
                    L = __ldg(p.lse + (long)(qs + tok) * p.Hq + head);
                    L = L == -INFINITY ? 0.f : -L * kCsLog2e;
                }
                nlse[c] = L;
                const int2 seen = tok < ql ? cs_range(p, pos0 + tok, prefix, cl) : make_int2(0, 0);
                run[c] = make_short2((short)min(32, max(0, seen.x - k_lo)), (short)min(32, max(0, seen.y - k_lo)));
                if constexpr (MOD == CS_BIAS) slope[c] = -__ldg(p.mod.slopes + head) * kCsLog2e;
            }
            __syncwarp();
            // every row of the tile is real and sees every key of this warp (warp-uniform)
            const int2 rf = cs_range(p, pos0 + tok0, prefix, cl);
            const int2 rl = cs_range(p, pos0 + min(ql, tok0 + tt) - 1, prefix, cl);
            const bool plain = tok0 + tt <= ql && k_lo >= rl.x && k_hi <= rf.y;
            if (!mbar_wait_warp(&sfull[w], (i >> 1) & 1, lim_ns, abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // four columns at a time; `masked`: some row of the tile is not real or does not see some key
            auto columns = [&](auto masked) {
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    uint32_t raw[32];
                    tmem_ld32(trow + b * 32, raw);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 nl = *reinterpret_cast<const float4*>(nlse + b * 32 + j);
                        const float nls[4] = {nl.x, nl.y, nl.z, nl.w};
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            float2 x = make_float2(__uint_as_float(raw[j + e]), __uint_as_float(raw[j + e + 1]));
                            const float2 l2 = make_float2(nls[e], nls[e + 1]);
                            if (MOD == CS_CAP || (MOD == CS_BIAS && p.mod.cap_out > 0.f)) {
                                x.x = fmaf(p.mod.cap_out, tanh_f32(x.x * p.mod.cap_in), l2.x);
                                x.y = fmaf(p.mod.cap_out, tanh_f32(x.y * p.mod.cap_in), l2.y);
                            } else {
                                x = __ffma2_rn(x, make_float2(p.scale_log2, p.scale_log2), l2);
                            }
                            if constexpr (MOD == CS_BIAS) {
                                const float2 sl = *reinterpret_cast<const float2*>(slope + b * 32 + j + e);
                                const int c = b * 32 + j + e, d0 = k_lo + lane - pos0 - tok0;
                                x.x = fmaf(sl.x, fabsf((float)(d0 - (p.pack ? c >> p.pack_shift : c))), x.x);
                                x.y = fmaf(sl.y, fabsf((float)(d0 - (p.pack ? (c + 1) >> p.pack_shift : c + 1))), x.y);
                            }
                            float2 pr = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                            if constexpr (decltype(masked)::value) {
                                const short2 ra = run[b * 32 + j + e], rb = run[b * 32 + j + e + 1];
                                pr.x = lane >= ra.x && lane < ra.y ? pr.x : 0.f;
                                pr.y = lane >= rb.x && lane < rb.y ? pr.y : 0.f;
                            }
                            sum[(j + e) >> 1 & 3] = __fadd2_rn(sum[(j + e) >> 1 & 3], pr);
                        }
                    }
                }
            };
            if (plain) columns(std::false_type{});
            else columns(std::true_type{});
            tc_fence_before();
            mbar_arrive(&sempty[w]);
        }
        if (!ok && lane == 0) fail();
        mine = ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) + ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y));
        if (w == 1) part[quarter * 32 + lane] = mine;
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kCsMma) tmem_dealloc(tbase, 256);
    const int key = kv0 + threadIdx.x;
    if (threadIdx.x < kCsRows && key < cl && !*abort_flag) {
        const long at = ((long)seq * p.Hkv + hk) * p.acc_len + key;
        const float old = p.acc_in && key < pos0 ? p.decay * p.acc_in[at] : 0.f;
        p.acc_out[at] = old + (mine + part[threadIdx.x]);
    }
}

template <int D, int MOD>
static fa_status launch_colsum(const CUtensorMap& tq, const CUtensorMap& tk, const ColsumParams& p, dim3 grid,
                               cudaStream_t s) {
    const fa_status st =
        raise_dynamic_smem(reinterpret_cast<const void*>(attn_colsum_kernel<D, MOD>), CsCfg<D>::kSmem);
    if (st != FA_OK) return st;
    attn_colsum_kernel<D, MOD><<<grid, kCsThreads, CsCfg<D>::kSmem, s>>>(tq, tk, p);
    return cuda_status(cudaGetLastError());
}

// Weight sums of the sequences whose chunks took the tensor-core path.
fa_status launch_accum_chunk(const void* q, const void* k_cache, const int32_t* block_table, const int32_t* ctx_lens,
                             const int32_t* q_lens, const int32_t* q_start, const float* lse, const float* acc_in,
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
    p.ctx = ctx;
    const dim3 grid(num_seqs * Hkv, (mbps * 16 + kCsRows - 1) / kCsRows);
    auto go = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        if (mod.slopes) return launch_colsum<D, CS_BIAS>(tq, tk, p, grid, s);
        if (mod.cap_out > 0.f) return launch_colsum<D, CS_CAP>(tq, tk, p, grid, s);
        return launch_colsum<D, CS_PLAIN>(tq, tk, p, grid, s);
    };
    return d == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 64>{});
}

}  // namespace fa
