// Attention of each query over the cache blocks listed for it (fa_paged_attn_blocks), and
// of single tokens over every block of short contexts in the 8-bit cache.
//
// One list per (query token, kv head): the Hq / Hkv heads of the group are the rows
// of m16n8k16 warp MMAs, so that a listed block is read once for all of them.  A CTA
// of two to four warps, or a cluster of up to eight of them when there are few lists,
// takes one list: warp w of W takes entries w, w + W, ..., streams their pages through a
// ring of its own in shared memory (TMA, the block looked up in the sequence's table)
// and keeps a softmax of its own; at the end the warps' results are joined with
// log-sum-exp weights in shared memory, across a cluster through distributed shared
// memory.  Nothing passes through device memory and one launch does it all.  Memory
// bound: 2 * 16 d values a block.
#include <algorithm>
#include <climits>

#include "page_mma.cuh"

namespace fa {

constexpr int kBlBatch = 32;  // list entries that a warp looks up at a time

struct BlocksArgs {
    const uint16_t* q;
    const int32_t *bt, *ctx_lens, *q_lens, *sel;
    const uint8_t *ke, *ve;
    uint16_t* out;
    float* lse;
    int num_seqs, mbps, num_blocks, total_q, Hq, Hkv, keep, head_tiles;
    int max_q_len;  // longer chunks are reported
    float scale_log2;
    DevCtx ctx;
};

template <int D, bool KV8, int NW>
struct BlocksSmem {
    using M = PageMma<D, KV8>;
    static constexpr int kStage = 2 * M::kPage;
    static constexpr int kStages = KV8 ? (D == 128 ? 4 : 8) : (D == 128 ? 2 : 4);
    static constexpr int kPages = KV8 ? (D == 128 ? 2 : 4) : (D == 128 ? 1 : 2);  // pages of one pass
    static constexpr int kRing = NW * kStages * kStage;
    // a warp's partial result takes its ring's place when its pages are read, four of the CTA's joined rows lie behind each
    static constexpr int kJoined = (M::kSlotFloats * 4 + 127) / 128 * 128;
    static constexpr int kBytes = 1024 + kRing + NW * kBlBatch * 16 + (NW * kStages + 1) * 8 + 16;
    static_assert(kStages > kPages, "copies in flight while a pass runs");
    static_assert(NW < 4 || kJoined + 16 / NW * D * 4 <= kStages * kStage, "a ring holds a partial result and the joined rows");
};

__device__ __forceinline__ void blocks_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The floats at p (an address of this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ float4 remote_f4(const float* p, unsigned rank) {
    uint32_t a;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 remote_f2(const float2* p, unsigned rank) {
    uint32_t a;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}

template <int D, bool KV8, int NW>
__global__ void __launch_bounds__(NW * 32, kListSmWarps / NW)
    blocks_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ BlocksArgs a) {
    using L = BlocksSmem<D, KV8, NW>;
    using M = PageMma<D, KV8>;
    constexpr int NP = L::kPages, ST = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    int4* lists = reinterpret_cast<int4*>(smem + L::kRing);
    uint64_t* bars = reinterpret_cast<uint64_t*>(lists + NW * kBlBatch);
    uint64_t* never = bars + NW * ST;  // nothing arrives on it (time-out test hook)
    volatile int* abort_flag = reinterpret_cast<volatile int*>(never + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned rank, C;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        for (int i = 0; i < NW * ST + 1; ++i) mbar_init(&bars[i], 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    // list: (query token, kv head), heads in tiles of 16
    const int unit = blockIdx.x / C, ht = unit % a.head_tiles, list = unit / a.head_tiles;
    const int hk = list % a.Hkv, row = list / a.Hkv, g = a.Hq / a.Hkv;
    const int nrows = min(16, g - ht * 16);
    // the first entries and the queries are on their way while the row's sequence is found
    const int gid = lane >> 2;
    const long out_row = (long)row * a.Hq + hk * g + ht * 16;  // of the tile's first head
    const int32_t* sel = a.sel ? a.sel + ((long)row * a.Hkv + hk) * a.keep : nullptr;  // null: every block of the table
    const int W = NW * (int)C, w0 = (int)rank * NW + warp;
    auto entry = [&](int i) { return i >= a.keep ? -1 : (sel ? __ldg(sel + i) : i); };
    int b_next = entry(w0 + lane * W);
    M t;
    {
        const uint16_t* q = a.q + out_row * D;
        t.load_q(gid < nrows ? q + gid * D : nullptr, gid + 8 < nrows ? q + (gid + 8) * D : nullptr, a.scale_log2);
    }
    t.reset();
    SeqItem it;
    auto count = [](int ql, int) { return ql; };
    const SeqScan scan(a.q_lens, a.ctx_lens, a.num_seqs, a.mbps, count);
    const bool some = scan.find(a.q_lens, a.ctx_lens, row, count, it);
    // (the whole cluster takes the same way)
    const bool fits = some && lens_ok(it.ql, it.cl, a.mbps) && (long long)it.q0 + it.ql <= a.total_q;
    if (blockIdx.x % C == 0 && threadIdx.x == 0 && (some != fits || scan.bad || scan.rows > a.total_q || (some && it.ql > a.max_q_len)))
        raise_error(a.ctx, ERR_BOUNDS_BIT);
    __syncthreads();
    if (!fits) return;
    const int pos = it.cl - it.ql + (int)it.off;
    uint8_t* ring = smem + warp * ST * L::kStage;
    uint64_t* wbar = bars + warp * ST;
    int4* entries = lists + warp * kBlBatch;
    bool ok = a.ctx.force_timeout != 1 || mbar_wait_warp(never, 0, a.ctx.wait_ns, abort_flag);
    int done = 0;  // pages taken from the ring so far
    for (int base = w0; base < a.keep && ok; base += W * kBlBatch) {
        // the next 32 entries of this warp: table and scales looked up by a lane each
        int n, place, ks_new = kExpBias, ev_new = kExpBias;
        {
            const int b = b_next;
            b_next = entry(base + (lane + kBlBatch) * W);
            bool use = b >= 0;
            int phys = -1;
            if (use) {
                if (b > (it.cl - 1) / kScaledBlock) {
                    if (sel) raise_error(a.ctx, ERR_BOUNDS_BIT);
                    use = false;
                } else if (b * kScaledBlock > pos) {
                    use = false;  // nothing of it is visible
                }
            }
            if (use) {
                phys = __ldg(a.bt + (long)it.s * a.mbps + b);
                if (phys < 0 || phys >= a.num_blocks) {
                    raise_error(a.ctx, ERR_BOUNDS_BIT);
                    phys = a.num_blocks;  // outside the tensor map: the copy fills zeros, at scale 1
                }
            }
            const unsigned live = __ballot_sync(0xffffffffu, use);
            n = __popc(live);
            place = __popc(live & ((1u << lane) - 1));
            if (use) {
                entries[place].x = phys;
                entries[place].y = b * kScaledBlock;
            } else {
                place = -1;
            }
            if (KV8 && use && phys < a.num_blocks) {  // (on their way while the first pages are asked for)
                ks_new = __ldg(a.ke + (long)phys * a.Hkv + hk);
                ev_new = __ldg(a.ve + (long)phys * a.Hkv + hk);
            }
            __syncwarp();
        }
        int issued = 0, i = 0;  // pages of these entries asked for, and taken from the ring
        auto issue = [&]() {
            const int stage = (done + issued) % ST;
            load_page<D, KV8>(ring + stage * L::kStage, &tm_k, &tm_v, &wbar[stage], hk, entries[issued].x);
            ++issued;
        };
        if (lane == 0)
            while (issued < n && issued < ST) issue();
        if (KV8 && place >= 0) {
            entries[place].z = ks_new;
            entries[place].w = ev_new;
        }
        __syncwarp();
        // (the test hook that gives up later, with copies in flight, ends the loop before: a test in it cost 2 %)
        const int stop = a.ctx.force_timeout > 1 ? min(n, max(0, a.ctx.force_timeout - 1 - done)) : n;
        while (i < stop && ok) {
            const int np = min(NP, stop - i);
            uint32_t kv[NP];
            int tok[NP], ks[NP], ev[NP];
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const int stage = (done + i + j) % ST;
                kv[j] = smem_u32(ring + stage * L::kStage);
                const int4 e = entries[min(i + j, kBlBatch - 1)];
                tok[j] = e.y;
                ks[j] = e.z;
                ev[j] = e.w;
                if (j < np && ok) ok = mbar_wait_warp(&wbar[stage], ((done + i + j) / ST) & 1, a.ctx.wait_ns, abort_flag);
            }
            if (!ok) break;
            t.template step<NP>(np, kv, tok, ks, ev, pos, pos, pos + 1);
            __syncwarp();
            i += np;
            if (lane == 0)
                while (issued < n && issued < i + ST) issue();
        }
        if (stop < n && ok) ok = mbar_wait_warp(never, 0, a.ctx.wait_ns, abort_flag);
        if (!ok && lane == 0) {  // let the copies in flight land before the CTA may end (earlier phases are over)
            for (; i < issued; ++i)
                (void)mbar_wait_bounded(&wbar[(done + i) % ST], ((done + i) / ST) & 1, 1000000000ull, nullptr);
        }
        done += n;
        __syncwarp();
    }
    if (!ok && lane == 0) {
        raise_error(a.ctx, ERR_TIMEOUT_BIT);
        *abort_flag = 1;
    }
    // join the warps, then the cluster's CTAs: row by row M = max m, weights 2^(m - M)
    t.finish();
    t.store_partial(reinterpret_cast<float*>(ring), nrows);
    __syncthreads();
    constexpr int kCols = D / 4;
    auto write = [&](int r, int c, float4 v, float mx, float sum) {
        const float inv = sum > 0.f ? M::kDown / sum : 0.f;
        *reinterpret_cast<uint2*>(a.out + (out_row + r) * D + c * 4) =
            make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
        if (a.lse && c == 0)
            a.lse[out_row + r] = sum > 0.f ? (mx + __log2f(sum)) * 0.6931471805599453f : -INFINITY;
    };
    auto join = [&](int r, int c, int parts, auto ml_of, auto o_of, float4& v, float& mx, float& sum) {
        mx = -INFINITY;
        sum = 0.f;
        v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < parts; ++i) mx = fmaxf(mx, ml_of(i, r).x);
        for (int i = 0; i < parts; ++i) {
            const float2 ml = ml_of(i, r);
            const float4 x = o_of(i, r, c);
            const float f = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - mx);
            sum = fmaf(f, ml.y, sum);
            v.x = fmaf(f, x.x, v.x);
            v.y = fmaf(f, x.y, v.y);
            v.z = fmaf(f, x.z, v.z);
            v.w = fmaf(f, x.w, v.w);
        }
    };
    auto slot = [&](int i) { return reinterpret_cast<const float*>(smem + i * ST * L::kStage); };
    auto warp_ml = [&](int i, int r) { return reinterpret_cast<const float2*>(slot(i) + 16 * M::kSlotRow)[r]; };
    auto warp_o = [&](int i, int r, int c) { return *reinterpret_cast<const float4*>(slot(i) + r * M::kSlotRow + c * 4); };
    constexpr int kRowsEach = (16 + NW - 1) / NW;  // of the CTA's joined rows behind each warp's partial result
    auto mine = [&](int r) {
        return reinterpret_cast<float*>(smem + r / kRowsEach * ST * L::kStage + L::kJoined) + r % kRowsEach * D;
    };
    float2* mine_ml = reinterpret_cast<float2*>(lists);  // (the lists are read)
    for (int i = threadIdx.x; i < nrows * kCols; i += blockDim.x) {
        const int r = i / kCols, c = i % kCols;
        float4 v;
        float mx, sum;
        join(r, c, NW, warp_ml, warp_o, v, mx, sum);
        if (C == 1) {
            if (!*abort_flag) write(r, c, v, mx, sum);
        } else {
            *reinterpret_cast<float4*>(mine(r) + c * 4) = v;
            // (a CTA whose waits gave up says so with a negative sum: no CTA of the cluster writes its share of the rows)
            if (c == 0) mine_ml[r] = *abort_flag ? make_float2(-INFINITY, -1.f) : make_float2(mx, sum);
        }
    }
    if (C == 1) return;
    blocks_cluster_sync();
    for (int i = (int)rank * blockDim.x + threadIdx.x; i < nrows * kCols; i += (int)C * blockDim.x) {
        const int r = i / kCols, c = i % kCols;
        float4 v;
        float mx, sum;
        bool whole = true;  // (else a part of the row's keys is missing)
        auto cta_ml = [&](int k, int rr) {
            const float2 ml = remote_f2(mine_ml + rr, k);
            whole = whole && !(ml.y < 0.f);
            return ml;
        };
        join(r, c, (int)C, cta_ml,
             [&](int k, int rr, int cc) { return remote_f4(mine(rr) + cc * 4, k); }, v, mx, sum);
        if (whole) write(r, c, v, mx, sum);
    }
    blocks_cluster_sync();  // no CTA leaves while another reads its rows
}

template <int D, bool KV8, int NW>
static fa_status launch_blocks_warps(const CUtensorMap& tk, const CUtensorMap& tv, const BlocksArgs& a, long units, int cluster,
                                     cudaStream_t s) {
    using L = BlocksSmem<D, KV8, NW>;
    auto kernel = blocks_attn_kernel<D, KV8, NW>;
    const fa_status st = raise_dynamic_smem(reinterpret_cast<const void*>(kernel), L::kBytes);
    if (st != FA_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * cluster));
    cfg.blockDim = dim3(NW * 32);
    cfg.dynamicSmemBytes = L::kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, tk, tv, a));
}

template <int D, bool KV8>
static fa_status launch_blocks(const void* k_cache, const void* v_cache, const BlocksArgs& a, cudaStream_t s) {
    CUtensorMap tk, tv;
    const fa_status st = page_maps<D, KV8>(k_cache, v_cache, a.num_blocks, a.Hkv, &tk, &tv);
    if (st != FA_OK) return st;
    const long units = (long)a.total_q * a.Hkv * a.head_tiles;
    const long slots = (long)kListSmWarps * sm_count();
    // Few lists: four warps and clusters of such CTAs, while they all fit the GPU at once and each warp still gets
    // pages for a pass (160 lists of 256: 41 us, with two warps 56).  More: three warps while all lists fit at once
    // (518 bf16 lists of 48 22.7 us, with two 26.7; 512 8-bit ones of 64 32.8, with two 34.3, with four 41, with one 49).
    // Many: two warps, so that fewer wait for their list's others (8352 lists of 48 230 us, with one 250, with four 266).
    int cluster = 1;
    while (cluster < 8 && units * cluster * 8 <= slots && a.keep >= 8 * cluster * BlocksSmem<D, KV8, 4>::kPages) cluster *= 2;
    if (units * cluster > 0x7fffffffL) return FA_ERR_UNSUPPORTED;
    if (units * 3 > slots) return launch_blocks_warps<D, KV8, 2>(tk, tv, a, units, 1, s);
    if (units * 4 > slots) return launch_blocks_warps<D, KV8, 3>(tk, tv, a, units, 1, s);
    return launch_blocks_warps<D, KV8, 4>(tk, tv, a, units, cluster, s);
}

// Single tokens over every block of short tables (fa_paged_attn_fp8_scaled).
fa_status launch_whole_lists(const void* q, const void* k_cache, const void* v_cache, const uint8_t* k_exp, const uint8_t* v_exp,
                             const int32_t* block_table, const int32_t* ctx_lens, const int32_t* q_lens, void* out, float* lse,
                             int num_seqs, int mbps, int num_blocks, int Hq, int Hkv, int d, float scale, int total_q,
                             int max_q_len, cudaStream_t s, const DevCtx& ctx) {
    const BlocksArgs a{static_cast<const uint16_t*>(q), block_table, ctx_lens, q_lens, nullptr, k_exp, v_exp,
                       static_cast<uint16_t*>(out), lse, num_seqs, mbps, num_blocks, total_q, Hq, Hkv, mbps,
                       (Hq / Hkv + 15) / 16, max_q_len, scale * 1.4426950408889634f, ctx};
    return d == 128 ? launch_blocks<128, true>(k_cache, v_cache, a, s) : launch_blocks<64, true>(k_cache, v_cache, a, s);
}

}  // namespace fa

using namespace fa;

extern "C" fa_status fa_paged_attn_blocks(const void* q, const void* k_cache, const void* v_cache, const uint8_t* k_exp,
                                          const uint8_t* v_exp, const int32_t* block_table, const int32_t* ctx_lens,
                                          const int32_t* q_lens, const int32_t* sel, int keep, void* out, float* lse,
                                          int num_seqs, int max_blocks_per_seq, int num_blocks, int Hq, int Hkv, int d,
                                          int block_size, float scale, int total_q, fa_stream_t stream) {
    set_launch_count(0);
    if (num_seqs < 0 || max_blocks_per_seq < 0 || num_blocks < 0 || Hq <= 0 || Hkv <= 0 || total_q < 0 || keep < 0 ||
        !(scale > 0.f) || !(scale < INFINITY) || !k_exp != !v_exp)
        return FA_ERR_INVALID_ARG;
    if (block_size != kScaledBlock || (d != 64 && d != 128) || Hq % Hkv != 0) return FA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0) return FA_OK;
    if (!q || !k_cache || !v_cache || !block_table || !ctx_lens || !q_lens || (!sel && keep > 0) || !out)
        return FA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return FA_ERR_INVALID_ARG;
    if (num_blocks == 0 || max_blocks_per_seq == 0) return FA_ERR_INVALID_ARG;
    fa_status st = check_device();
    if (st != FA_OK) return st;
    BlocksArgs a{static_cast<const uint16_t*>(q), block_table, ctx_lens, q_lens, sel, k_exp, v_exp, static_cast<uint16_t*>(out),
                 lse, num_seqs, max_blocks_per_seq, num_blocks, total_q, Hq, Hkv, keep, (Hq / Hkv + 15) / 16,
                 INT_MAX, scale * 1.4426950408889634f, {}};
    if ((st = make_ctx(&a.ctx)) != FA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (d == 128) st = k_exp ? launch_blocks<128, true>(k_cache, v_cache, a, s) : launch_blocks<128, false>(k_cache, v_cache, a, s);
    else st = k_exp ? launch_blocks<64, true>(k_cache, v_cache, a, s) : launch_blocks<64, false>(k_cache, v_cache, a, s);
    if (st == FA_OK) set_launch_count(1);
    return st;
}
