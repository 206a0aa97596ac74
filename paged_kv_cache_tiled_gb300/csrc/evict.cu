// Eviction from the paged cache by accumulated attention weight: per sequence
// and kv head the first `sink` tokens, the last `recent` ones and, of the rest,
// those with the largest accumulated weights (equal weights: the earlier token)
// are kept, `keep` in all, and copied in order of position from the blocks of
// one table to those of another.
//
// evict_select_kernel (one CTA per sequence and kv head) finds the weight of
// the last token kept with a radix select over order-preserving integer keys
// (three passes of 11, 11 and 10 bits), then lists the kept tokens with one
// scan; evict_move_kernel gathers their rows.  Memory bound: the weights are read
// once from HBM (the passes after the first hit L2), each kept row once.
#include "host_common.cuh"

namespace fa {

constexpr int kEvBlock = 16;
constexpr int kEvThreads = 1024;
constexpr int kEvBins = 2048;
constexpr int kEvItems = 8;  // consecutive tokens per thread and scan pass

// Larger weight, larger key; NaN below everything, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float x) {
    if (!(x == x)) return 0u;
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const float* acc, int acc_len,
                                                                  const int32_t* __restrict__ ctx_lens, float* acc_out,
                                                                  int out_len, int32_t* __restrict__ list,
                                                                  int32_t* __restrict__ new_lens, int Hkv, int mbps,
                                                                  int dst_mbps, int keep, int recent, int sink,
                                                                  DevCtx ctx) {
    __shared__ int hist[kEvBins];
    __shared__ int2 warp_sums[32];
    __shared__ int sel_digit, sel_above;
    const int s = blockIdx.x / Hkv, h = blockIdx.x % Hkv, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int cl = __ldg(ctx_lens + s);
    int32_t* out = list + (long)blockIdx.x * keep;
    const int n = min(cl, keep);
    if (cl < 0 || cl > mbps * kEvBlock || cl > acc_len || n > dst_mbps * kEvBlock) {
        if (tid == 0) raise_error(ctx, ERR_BOUNDS_BIT);
        for (int i = tid; i < keep; i += kEvThreads) out[i] = -1;
        if (h == 0 && tid == 0) new_lens[s] = 0;
        return;
    }
    if (h == 0 && tid == 0) new_lens[s] = n;
    for (int i = n + tid; i < keep; i += kEvThreads) out[i] = -1;
    const float* a = acc + (long)blockIdx.x * acc_len;
    float* ao = acc_out ? acc_out + (long)blockIdx.x * out_len : nullptr;
    if (cl <= keep) {
        for (int i = tid; i < cl; i += kEvThreads) {
            out[i] = i;
            if (ao) ao[i] = a[i];
        }
        return;
    }
    // the `want` largest keys of the tokens [sink, mid_end)
    const int mid_end = cl - recent;
    int want = keep - sink - recent;
    uint32_t prefix = 0;  // digits fixed so far
    int need = want;      // tokens still to take among those that match the prefix
    for (int pass = 0; pass < 3 && want > 0; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
        for (int i = tid; i < kEvBins; i += kEvThreads) hist[i] = 0;
        __syncthreads();
        for (int t0 = sink + wid * 32; t0 < mid_end; t0 += kEvThreads) {
            const int t = t0 + lane;
            const uint32_t key = t < mid_end ? weight_key(a[t]) : 0u;
            const bool in = t < mid_end && (pass == 0 || (key >> (shift + bits)) == (prefix >> (shift + bits)));
            const uint32_t digit = in ? (key >> shift) & ((1u << bits) - 1) : 0xffffffffu;
            int same;
            __match_all_sync(0xffffffffu, digit, &same);
            if (same) {  // many tokens may hold the same weight (0): one add for the warp
                if (in && lane == 0) atomicAdd(&hist[digit], 32);
            } else if (in) {
                atomicAdd(&hist[digit], 1);
            }
        }
        __syncthreads();
        // the digit where the count from the top reaches `need`: each thread owns two bins
        const int b1 = kEvBins - 1 - 2 * tid, b0 = b1 - 1;  // highest bins first
        const int c1 = hist[b1], c0 = hist[b0];
        int x = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_sums[wid].x = x;
        __syncthreads();
        int before = 0;
        for (int k = 0; k < wid; ++k) before += warp_sums[k].x;
        const int above = before + x - c0 - c1;  // keys in higher bins than b1
        if (above < need && above + c1 >= need) {
            sel_digit = b1;
            sel_above = above;
        } else if (above + c1 < need && above + c1 + c0 >= need) {
            sel_digit = b0;
            sel_above = above + c1;
        }
        __syncthreads();
        prefix |= (uint32_t)sel_digit << shift;
        need -= sel_above;
        __syncthreads();
    }
    // tokens above the threshold key, the forced ones, and the first `need` equal to it
    int kept_before = 0, eq_before = 0;
    for (int base = 0; base < cl; base += kEvThreads * kEvItems) {
        const int t0 = base + tid * kEvItems;
        float v[kEvItems];
        unsigned sure = 0, eq = 0;
#pragma unroll
        for (int k = 0; k < kEvItems; ++k) {
            const int t = t0 + k;
            v[k] = t < cl ? a[t] : 0.f;
            if (t >= cl) continue;
            const uint32_t key = weight_key(v[k]);
            if (t < sink || t >= mid_end || (want > 0 && key > prefix))
                sure |= 1u << k;
            else if (want > 0 && key == prefix)
                eq |= 1u << k;
        }
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
        if (lane == 31) warp_sums[wid] = x;
        __syncthreads();
        int2 pre = make_int2(0, 0), tot = make_int2(0, 0);
        for (int k = 0; k < 32; ++k) {
            const int2 t = warp_sums[k];
            if (k < wid) {
                pre.x += t.x;
                pre.y += t.y;
            }
            tot.x += t.x;
            tot.y += t.y;
        }
        int ns = kept_before + pre.x + x.x - own.x, ne = eq_before + pre.y + x.y - own.y;
        // (every weight of this pass is read: acc_out may be acc itself, no write lands on a later token)
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
        kept_before += tot.x;
        eq_before += tot.y;
        __syncthreads();
    }
}

// Row i of (sequence, kv head): kept token list[i] from its block of `src` to
// token i of `dst`, K and V, 16 bytes per thread; kEvRows rows per thread so
// that their loads are in flight together.
constexpr int kEvRows = 4;
__global__ void __launch_bounds__(256) evict_move_kernel(uint16_t* kc, uint16_t* vc, const int32_t* __restrict__ src,
                                                         const int32_t* __restrict__ dst,
                                                         const int32_t* __restrict__ list, int num_seqs, int Hkv, int d,
                                                         int mbps, int dst_mbps, int keep, int num_blocks, DevCtx ctx) {
    const int cpr = d >> 3;             // chunks per row
    const int lanes = 2 * cpr;          // threads per row pair (K and V)
    const int rows_cta = 256 / lanes;   // rows side by side
    const long per = (keep + rows_cta * kEvRows - 1) / (rows_cta * kEvRows);  // CTA items per (sequence, head)
    const long total = (long)num_seqs * Hkv * per;
    const int c = threadIdx.x % lanes, rr = threadIdx.x / lanes;
    uint16_t* cache = c < cpr ? kc : vc;
    const int off = (c < cpr ? c : c - cpr) * 8;
    for (long item = blockIdx.x; item < total; item += gridDim.x) {
        const long sh = item / per;
        const int s = (int)(sh / Hkv), h = (int)(sh % Hkv), i0 = (int)(item % per) * rows_cta * kEvRows + rr;
        long to[kEvRows];
        uint4 v[kEvRows];
#pragma unroll
        for (int k = 0; k < kEvRows; ++k) {
            const int i = i0 + k * rows_cta;
            to[k] = -1;
            const int t = i < keep ? __ldg(list + sh * keep + i) : -1;
            if (t < 0) continue;
            const int sb = __ldg(src + (long)s * mbps + t / kEvBlock);
            const int db = __ldg(dst + (long)s * dst_mbps + i / kEvBlock);
            if (sb < 0 || sb >= num_blocks || db < 0 || db >= num_blocks) {
                raise_error(ctx, ERR_BOUNDS_BIT);
                continue;
            }
            v[k] = *reinterpret_cast<const uint4*>(cache + (((long)sb * Hkv + h) * kEvBlock + t % kEvBlock) * d + off);
            to[k] = (((long)db * Hkv + h) * kEvBlock + i % kEvBlock) * d + off;
        }
#pragma unroll
        for (int k = 0; k < kEvRows; ++k)
            if (to[k] >= 0) *reinterpret_cast<uint4*>(cache + to[k]) = v[k];
    }
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
    if ((long)num_seqs * Hkv >= 1L << 31) return FA_ERR_UNSUPPORTED;
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
    evict_select_kernel<<<num_seqs * Hkv, kEvThreads, 0, s>>>(acc, acc_len, ctx_lens, acc_out, acc_out_len, list,
                                                              new_lens, Hkv, max_blocks_per_seq, dst_blocks_per_seq,
                                                              keep, recent, sink, ctx);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    const int rows_item = 256 / (2 * (d / 8)) * kEvRows;
    const long items = (long)num_seqs * Hkv * ((keep + rows_item - 1) / rows_item);
    const long cap = (long)sm_count() * 8;
    evict_move_kernel<<<(int)(items < cap ? items : cap), 256, 0, s>>>(
        static_cast<uint16_t*>(k_cache), static_cast<uint16_t*>(v_cache), block_table, dst_table, list, num_seqs, Hkv, d,
        max_blocks_per_seq, dst_blocks_per_seq, keep, num_blocks, ctx);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    set_launch_count(2);
    return FA_OK;
}

}  // extern "C"
