// Eviction from the paged cache by accumulated attention weight: per sequence
// and kv head the first `sink` tokens, the last `recent` ones and, of the rest,
// those with the largest accumulated weights (equal weights: the earlier token)
// are kept, `keep` in all, and copied in order of position from the blocks of
// one table to those of another.
//
// evict_select_kernel finds the weight of the last token kept with a radix
// select over order-preserving integer keys (three passes of 11, 11 and 10
// bits), then lists the kept tokens with one scan.  A sequence and kv head is one
// CTA, or a cluster of up to eight when its row is long: each CTA histograms
// its part (kept in registers when it has at most 4096 tokens), the parts are
// added through distributed shared memory, and every CTA takes the same
// decision.  evict_move_kernel gathers the kept rows.  Memory bound: the weights
// are read once, each kept row once.  Two sequences of 32768 tokens to 8192 (8
// heads, d = 128): 39 us, 25 of them the copy (5.4 TB/s); 64 sequences of up to
// 4096 to 512 (2 heads): 20.5.
#include <algorithm>

#include "host_common.cuh"

namespace fa {

constexpr int kEvBlock = 16;
constexpr int kEvThreads = 512;
constexpr int kEvBins = 2048;
constexpr int kEvItems = 8;  // consecutive tokens per thread and scan pass

// Larger weight, larger key; NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float x) {
    if (!(x == x)) return 0u;
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ unsigned cluster_rank() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ unsigned cluster_size() {
    unsigned r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The int at p (an address of this CTA's shared memory) in CTA `rank` of the cluster.
__device__ __forceinline__ int cluster_load(const int* p, unsigned rank) {
    uint32_t a;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// Adds v to the int at p (as above) in CTA `rank` of the cluster.
__device__ __forceinline__ void cluster_add(int* p, unsigned rank, int v) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("red.relaxed.cluster.shared::cluster.add.s32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Do a context of cl tokens and the n kept ones fit the tables and the row of weights?
__device__ __forceinline__ bool lens_fit(int cl, int n, int mbps, int dst_mbps, int acc_len) {
    return cl >= 0 && cl <= mbps * kEvBlock && cl <= acc_len && n <= dst_mbps * kEvBlock;
}

constexpr int kEvPass = kEvThreads * kEvItems;  // tokens of a scan pass
__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const float* acc, int acc_len,
                                                                  const int32_t* __restrict__ ctx_lens, float* acc_out,
                                                                  int out_len, int32_t* __restrict__ list, int Hkv,
                                                                  int mbps, int dst_mbps, int keep, int recent,
                                                                  int sink, DevCtx ctx) {
    static_assert(kEvBins == 4 * kEvThreads, "a thread owns four bins");
    __shared__ __align__(16) int hist[kEvBins];  // this CTA's counts
    // the cluster's counts, by turns, so that one cluster barrier per pass is enough (a single CTA uses hist)
    __shared__ __align__(16) int total[2][kEvBins];
    __shared__ int2 warp_sums[32];
    __shared__ int sel_digit, sel_above, sel_count, totals[2];
    // the rows' copy may be scheduled; it waits for this grid's end before it reads the list
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int CL = (int)cluster_size(), rank = (int)cluster_rank();
    const int sh = blockIdx.x / CL, s = sh / Hkv;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int cl = __ldg(ctx_lens + s);
    int32_t* out = list + (long)sh * keep;
    const int n = min(cl, keep);
    const int gtid = rank * kEvThreads + tid, gthreads = CL * kEvThreads;
    if (!lens_fit(cl, n, mbps, dst_mbps, acc_len)) {  // the same for the whole cluster
        if (rank == 0 && tid == 0) raise_error(ctx, ERR_BOUNDS_BIT);
        for (int i = gtid; i < keep; i += gthreads) out[i] = -1;
        return;
    }
    for (int i = n + gtid; i < keep; i += gthreads) out[i] = -1;
    const float* a = acc + (long)sh * acc_len;
    float* ao = acc_out ? acc_out + (long)sh * out_len : nullptr;
    if (cl <= keep) {
        for (int i = gtid; i < cl; i += gthreads) {
            out[i] = i;
            if (ao) ao[i] = a[i];
        }
        return;
    }
    // this CTA's tokens [p0, p1), a multiple of the scan's items except at the end
    const int part = ((cl + CL - 1) / CL + kEvItems - 1) / kEvItems * kEvItems;
    const int p0 = min(cl, rank * part), p1 = min(cl, p0 + part);
    const bool vec = (acc_len & 3) == 0 && (reinterpret_cast<uintptr_t>(acc) & 15) == 0;
    const int mid_end = cl - recent;
    float v[kEvItems];
    uint32_t key[kEvItems];
    unsigned middle = 0;  // which of the thread's tokens the weights decide about
    auto load = [&](int t0) {
        if (vec && t0 + kEvItems <= p1) {
            const float4 x = *reinterpret_cast<const float4*>(a + t0), y = *reinterpret_cast<const float4*>(a + t0 + 4);
            v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w; v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
        } else {
#pragma unroll
            for (int k = 0; k < kEvItems; ++k) v[k] = t0 + k < p1 ? a[t0 + k] : 0.f;
        }
        middle = 0;
#pragma unroll
        for (int k = 0; k < kEvItems; ++k) {
            key[k] = weight_key(v[k]);
            if (t0 + k < p1 && t0 + k >= sink && t0 + k < mid_end) middle |= 1u << k;
        }
    };
    const bool once = p1 - p0 <= kEvPass;  // the part stays in registers
    load(p0 + tid * kEvItems);
    // the `want` largest keys of the tokens [sink, mid_end)
    const int want = keep - sink - recent;
    uint32_t prefix = 0;  // digits fixed so far
    int need = want;      // tokens still to take among those that match the prefix
    const int top = kEvBins - 4 * (tid + 1);  // this thread's bins [top, top + 4): highest bins first
    const int4 zero4 = make_int4(0, 0, 0, 0);
    *reinterpret_cast<int4*>(&hist[top]) = zero4;
    *reinterpret_cast<int4*>(&total[0][top]) = zero4;
    if (CL > 1) cluster_sync_all();  // every CTA's counts are clear before another adds to them
    else __syncthreads();
    for (int pass = 0; pass < 3 && want > 0; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
        for (int base = p0; base < p1; base += kEvPass) {
            if (!once) load(base + tid * kEvItems);
            if (!__any_sync(0xffffffffu, middle)) continue;
#pragma unroll
            for (int k = 0; k < kEvItems; ++k) {
                const bool in = ((middle >> k) & 1u) && (pass == 0 || ((key[k] ^ prefix) >> (shift + bits)) == 0);
                const uint32_t digit = in ? (key[k] >> shift) & ((1u << bits) - 1) : 0xffffffffu;
                // many tokens may hold the same weight (0): one add for the warp then
                const bool same = __all_sync(0xffffffffu, digit == __shfl_sync(0xffffffffu, digit, 0));
                if (in && (!same || lane == 0)) atomicAdd(&hist[digit], same ? 32 : 1);
            }
        }
        __syncthreads();
        int4 c = *reinterpret_cast<const int4*>(&hist[top]);
        *reinterpret_cast<int4*>(&hist[top]) = zero4;  // (next used behind the barriers below)
        if (CL > 1) {
            // Few of the bins hold anything, so the counts are added to every CTA's totals
            // (reading all bins of eight CTAs took 1.6 us a pass).
            int* sums = total[pass & 1];
            const int own[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (own[b])
                    for (int r = 0; r < CL; ++r) cluster_add(&sums[top + b], r, own[b]);
            *reinterpret_cast<int4*>(&total[(pass + 1) & 1][top]) = zero4;  // read last before the barrier of the pass before
            cluster_sync_all();
            c = *reinterpret_cast<const int4*>(&sums[top]);
        }
        // the digit where the count from the top reaches `need`
        const int own_c = c.x + c.y + c.z + c.w;
        int x = own_c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_sums[wid].x = x;
        __syncthreads();
        int above = __reduce_add_sync(0xffffffffu, lane < wid ? warp_sums[lane].x : 0) + x - own_c;
        if (above < need && above + own_c >= need) {  // in one of this thread's bins
            const int cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int b = 3; b >= 0; --b) {
                if (above < need && above + cs[b] >= need) {
                    sel_digit = top + b;
                    sel_above = above;
                    sel_count = cs[b];
                }
                above += cs[b];
            }
        }
        __syncthreads();
        prefix |= (uint32_t)sel_digit << shift;
        need -= sel_above;
        // Every token that matches the digits so far is kept: no need to tell them apart (22 bits
        // mostly single one token out).  Keys above prefix - 1 are kept then.
        if (sel_count == need && prefix > 0) {
            --prefix;
            need = 0;
            break;
        }
        // (sel_* is written again only behind the next pass's barriers)
    }
    // tokens above the threshold key, the forced ones, and the first `need` equal to it
    auto classify = [&](int t0, unsigned& sure, unsigned& eq) {
        sure = eq = 0;
#pragma unroll
        for (int k = 0; k < kEvItems; ++k) {
            const int t = t0 + k;
            if (t >= p1) continue;
            if (!((middle >> k) & 1u) || (want > 0 && key[k] > prefix))
                sure |= 1u << k;
            else if (want > 0 && key[k] == prefix)
                eq |= 1u << k;
        }
    };
    int kept_before = 0, eq_before = 0;
    if (CL > 1) {  // what the CTAs before this one hold
        if (tid < 2) totals[tid] = 0;
        __syncthreads();
        for (int base = p0; base < p1; base += kEvPass) {
            unsigned sure, eq;
            if (!once) load(base + tid * kEvItems);
            classify(base + tid * kEvItems, sure, eq);
            const int ns = __reduce_add_sync(0xffffffffu, __popc(sure)), ne = __reduce_add_sync(0xffffffffu, __popc(eq));
            if (lane == 0) {
                atomicAdd(&totals[0], ns);
                atomicAdd(&totals[1], ne);
            }
        }
        cluster_sync_all();
        for (int r = 0; r < rank; ++r) {
            kept_before += cluster_load(&totals[0], r);
            eq_before += cluster_load(&totals[1], r);
        }
        cluster_sync_all();  // no CTA leaves while another still reads its totals
    }
    for (int base = p0; base < p1; base += kEvPass) {
        const int t0 = base + tid * kEvItems;
        if (!once) load(t0);
        unsigned sure, eq;
        classify(t0, sure, eq);
        int2 x = make_int2(__popc(sure), __popc(eq));
        const int2 own = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y0 = __shfl_up_sync(0xffffffffu, x.x, o), y1 = __shfl_up_sync(0xffffffffu, x.y, o);
            if (lane >= o) {
                x.x += y0;
                x.y += y1;
            }
        }
        __syncthreads();  // warp_sums of the pass before is read
        if (lane == 31) warp_sums[wid] = x;
        __syncthreads();
        const int2 ws = lane < kEvThreads / 32 ? warp_sums[lane] : make_int2(0, 0);
        int ns = kept_before + x.x - own.x + __reduce_add_sync(0xffffffffu, lane < wid ? ws.x : 0);
        int ne = eq_before + x.y - own.y + __reduce_add_sync(0xffffffffu, lane < wid ? ws.y : 0);
        kept_before += __reduce_add_sync(0xffffffffu, ws.x);
        eq_before += __reduce_add_sync(0xffffffffu, ws.y);
        // (every weight of this pass is in registers: acc_out may be acc itself, no write lands on a later token)
#pragma unroll
        for (int k = 0; k < kEvItems; ++k) {
            const bool is_eq = (eq >> k) & 1u;
            const bool take = ((sure >> k) & 1u) || (is_eq && ne < need);
            const int pos = ns + min(ne, need);
            if (take && pos < keep) {
                out[pos] = t0 + k;
                if (ao) ao[pos] = v[k];
            }
            ns += (sure >> k) & 1u;
            ne += is_eq ? 1 : 0;
        }
    }
}

// Row i of (sequence, kv head): kept token list[i] from its block of `src` to
// token i of `dst`, K and V, 16 bytes per thread; kEvRows rows per thread whose
// loads are in flight together, and full occupancy behind the three dependent
// loads (token, blocks, values) of a row.
// CTA (sequence and head, group of rows).  The first of a sequence writes its new
// length, here and not in the select: new_lens may be ctx_lens itself, which every
// CTA of the select reads.
constexpr int kEvRows = 2;
template <int D>
__global__ void __launch_bounds__(256, 8) evict_move_kernel(uint16_t* kc, uint16_t* vc, const int32_t* __restrict__ src,
                                                            const int32_t* __restrict__ dst, const int32_t* list,
                                                            const int32_t* ctx_lens, int32_t* new_lens, int acc_len,
                                                            int Hkv, int mbps, int dst_mbps, int keep, int num_blocks,
                                                            DevCtx ctx) {
    constexpr int d = D, cpr = D / 8;      // chunks per row
    constexpr int lanes = 2 * cpr;         // threads per row pair (K and V)
    constexpr int rows_cta = 256 / lanes;  // rows side by side
    const int c = threadIdx.x % lanes, rr = threadIdx.x / lanes;
    uint16_t* cache = c < cpr ? kc : vc;
    const int off = (c < cpr ? c : c - cpr) * 8;
    const int sh = blockIdx.x, s = sh / Hkv, h = sh % Hkv;
    const bool first = blockIdx.y == 0 && h == 0 && threadIdx.x == 0;
    const int cl = first ? ctx_lens[s] : 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the list is complete
    if (first) {
        const int n = min(cl, keep);
        new_lens[s] = lens_fit(cl, n, mbps, dst_mbps, acc_len) ? n : 0;
    }
    const int i0 = blockIdx.y * rows_cta * kEvRows + rr;
    const int32_t* tokens = list + (long)sh * keep;
    int t[kEvRows];
#pragma unroll
    for (int k = 0; k < kEvRows; ++k) t[k] = i0 + k * rows_cta < keep ? __ldcg(tokens + i0 + k * rows_cta) : -1;
    long to[kEvRows];
    uint4 v[kEvRows];
#pragma unroll
    for (int k = 0; k < kEvRows; ++k) {
        const int i = i0 + k * rows_cta;
        to[k] = -1;
        if (t[k] < 0) continue;
        const int sb = __ldg(src + (long)s * mbps + t[k] / kEvBlock);
        const int db = __ldg(dst + (long)s * dst_mbps + i / kEvBlock);
        if (sb < 0 || sb >= num_blocks || db < 0 || db >= num_blocks) {
            raise_error(ctx, ERR_BOUNDS_BIT);
            continue;
        }
        v[k] = *reinterpret_cast<const uint4*>(cache + (((long)sb * Hkv + h) * kEvBlock + t[k] % kEvBlock) * d + off);
        to[k] = (((long)db * Hkv + h) * kEvBlock + i % kEvBlock) * d + off;
    }
#pragma unroll
    for (int k = 0; k < kEvRows; ++k)
        if (to[k] >= 0) *reinterpret_cast<uint4*>(cache + to[k]) = v[k];
}

}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_cache_evict_workspace_size(int num_seqs, int max_blocks_per_seq, int Hkv, int keep) {
    if (num_seqs <= 0 || max_blocks_per_seq < 0 || Hkv <= 0 || keep <= 0) return 0;
    return align256((size_t)num_seqs * Hkv * keep * sizeof(int32_t));
}

fa_status fa_cache_evict(void* k_cache, void* v_cache, const float* acc, int acc_len, const int32_t* block_table,
                         const int32_t* ctx_lens, const int32_t* dst_table, float* acc_out, int acc_out_len,
                         int32_t* new_lens, int32_t* kept, int num_seqs, int max_blocks_per_seq,
                         int dst_blocks_per_seq, int num_blocks, int Hkv, int d, int block_size, int keep, int recent,
                         int sink, void* ws, size_t ws_bytes, fa_stream_t stream) {
    set_launch_count(0);
    if (num_seqs < 0 || max_blocks_per_seq < 0 || dst_blocks_per_seq < 0 || num_blocks < 0 || Hkv <= 0 || keep <= 0 ||
        recent < 0 || sink < 0 || recent > keep || sink > keep - recent || acc_len < 0 || acc_out_len < 0)
        return FA_ERR_INVALID_ARG;
    if (block_size != kEvBlock || (d != 64 && d != 128)) return FA_ERR_UNSUPPORTED;
    if ((long)num_seqs * Hkv >= 1L << 27 || keep > 16 * 65535) return FA_ERR_UNSUPPORTED;  // grid limits
    if (num_seqs == 0) return FA_OK;
    if (!k_cache || !v_cache || !acc || !block_table || !ctx_lens || !dst_table || !new_lens)
        return FA_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache) || dst_table == block_table) return FA_ERR_INVALID_ARG;
    // weights moved within their own rows (fine) or into rows of another length (they would overlap)
    if (acc_out && (acc_out_len < keep || (acc_out == acc && acc_out_len != acc_len))) return FA_ERR_INVALID_ARG;
    if (num_blocks == 0 || max_blocks_per_seq == 0 || dst_blocks_per_seq == 0) return FA_ERR_INVALID_ARG;
    int32_t* list = kept;
    if (!list) {
        if (!ws || ws_bytes < fa_cache_evict_workspace_size(num_seqs, max_blocks_per_seq, Hkv, keep) ||
            (reinterpret_cast<uintptr_t>(ws) & 255))
            return FA_ERR_WORKSPACE;
        list = static_cast<int32_t*>(ws);
    }
    fa_status st = check_device();
    if (st != FA_OK) return st;
    DevCtx ctx;
    if ((st = make_ctx(&ctx)) != FA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // CTAs per sequence and head: as few as keep the row in registers (a cluster's
    // barriers and remote counts cost more than half the tokens save: rows of 4096
    // tokens took 13 us in pairs of CTAs), while they all fit the GPU at once; one
    // when the weights move inside rows too long for the registers of a cluster
    // (a CTA must not overwrite what another has yet to read)
    const long rows = (long)num_seqs * Hkv, longest = std::min<long>((long)max_blocks_per_seq * kEvBlock, acc_len);
    int cluster = 1;
    while (cluster < 8 && longest > (long)kEvPass * cluster && rows * cluster * 2 <= 2L * sm_count()) cluster *= 2;
    if (acc_out == acc && longest > (long)cluster * (kEvPass - kEvItems)) cluster = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * cluster));
    cfg.blockDim = dim3(kEvThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, evict_select_kernel, acc, acc_len, ctx_lens, acc_out, acc_out_len, list, Hkv,
                           max_blocks_per_seq, dst_blocks_per_seq, keep, recent, sink, ctx) != cudaSuccess)
        return FA_ERR_CUDA;
    const int rows_item = 256 / (2 * (d / 8)) * kEvRows;
    const int per = (keep + rows_item - 1) / rows_item;  // CTAs per sequence and head
    cfg.gridDim = dim3((unsigned)rows, (unsigned)per);
    cfg.blockDim = dim3(256);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    auto move = d == 128 ? evict_move_kernel<128> : evict_move_kernel<64>;
    if (cudaLaunchKernelEx(&cfg, move, static_cast<uint16_t*>(k_cache), static_cast<uint16_t*>(v_cache), block_table,
                           dst_table, static_cast<const int32_t*>(list), ctx_lens, new_lens, acc_len, Hkv, max_blocks_per_seq,
                           dst_blocks_per_seq, keep, num_blocks, ctx) != cudaSuccess)
        return FA_ERR_CUDA;
    set_launch_count(2);
    return FA_OK;
}

}  // extern "C"
