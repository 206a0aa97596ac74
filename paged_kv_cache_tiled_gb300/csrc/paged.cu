// Paged attention ("Fast Attention Kernels and Operator Fusion", section
// "Paged Attention Kernels"): keys and values sit in 16-token blocks of a
// shared pool, [num_blocks, Hkv, 16, d] bf16, and every access goes through
// the per-sequence block table ("the kernel cannot assume that K[t+1] is
// adjacent to K[t]").
//
// Decode rows (the section "FlashAttention-Style Kernels" notes that decode
// has one or a few queries and is dominated by reading the growing cache)
// take a bandwidth-bound kernel that streams the cache in balanced ranges:
//   * the (sequence, kv head) segments are laid end to end as one stream of
//     16-token pages; each of the grid's warps (one CTA of eight warps per SM)
//     takes an equal contiguous range of pages, so every SM moves the same
//     number of bytes whatever the mix of context lengths;
//   * each warp streams its pages through a private ring of shared memory
//     with TMA (one 2 KB box per 64 channels of K and of V, 128-byte swizzled
//     so the fragment loads below are bank-conflict free); the physical block
//     id is read from the block table just before the copy;
//   * all Hq/Hkv query heads of the kv head (times the chunk's query tokens,
//     at most 16 rows) share each K/V load: they form the M dimension of
//     m16n8k16 warp MMAs, so K and V are read from HBM exactly once;
//   * the running row max / row sum are kept in fp32 (online softmax with
//     base-2 exponentials, scale * log2(e) folded into the scores); P is rounded
//     to V's type for the P V product (an MMA's operands have one type);
//   * a segment inside one warp's range is written as final bf16 output; a
//     segment cut by a range boundary leaves fp32 partials (unnormalised O,
//     running max, running sum) in shared memory, which the CTA combines with
//     log-sum-exp weights once its warps are done: into the final rows when
//     the segment lies inside the CTA's range, otherwise into one partial per
//     CTA that a second kernel merges the same way.
// Longer chunks take the tensor-core kernel (attn_tc.cu) through a work list
// built on the device by `paged_meta_kernel`.
// With modified scores (MOD variants) the stream holds only the blocks that a
// window leaves, and the weight sums' variant keeps its logits for
// `accum_decode_kernel`: 64 sequences of up to 8192 tokens with a window of 4096
// and a cap 41 us (the stream alone 4.8 TB/s), up to 4096 tokens with the sums 39
// us (33 without).
#include <algorithm>
#include <climits>
#include <mutex>
#include <type_traits>

#include "page_mma.cuh"

namespace fa {

constexpr int kBS = 16;            // tokens per block
constexpr int kDecodeRows = 16;    // M of the warp MMA

// Launched from attn_tc.cu.
fa_status launch_paged_prefill(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                               const int32_t* ctx_lens, const int32_t* q_lens, const int32_t* q_start,
                               const int32_t* work_list, const int32_t* work_count, void* out, int num_seqs,
                               int mbps, int num_blocks, int Hq, int Hkv, int d, int causal, float scale,
                               int total_q, cudaStream_t s, const DevCtx& ctx, const ScoreMod* mod,
                               const int4* pieces, float4* part_o, float2* part_ml);
// The same over the 8-bit cache with block scales, launched from attn_tc8.cu.
fa_status launch_paged_prefill_fp8(const void* q, const void* k_cache, const void* v_cache, const uint8_t* k_exp,
                                   const uint8_t* v_exp, const int32_t* block_table, const int32_t* ctx_lens,
                                   const int32_t* q_lens, const int32_t* q_start, const int32_t* work_count, void* out,
                                   float* lse, int mbps, int num_blocks, int Hq, int Hkv, int d, int causal, float scale,
                                   int total_q, const int4* pieces, float4* part_o, float2* part_ml, cudaStream_t s,
                                   const DevCtx& ctx);
// Single tokens over every block of short tables in one launch (blocks_attn.cu).
fa_status launch_whole_lists(const void* q, const void* k_cache, const void* v_cache, const uint8_t* k_exp, const uint8_t* v_exp,
                             const int32_t* block_table, const int32_t* ctx_lens, const int32_t* q_lens, void* out, float* lse,
                             int num_seqs, int mbps, int num_blocks, int Hq, int Hkv, int d, float scale, int total_q,
                             int max_q_len, cudaStream_t s, const DevCtx& ctx);
// Weight sums of the sequences that take the tensor-core path (attn_colsum.cu).
fa_status launch_accum_chunk(const void* q, const void* k_cache, const int32_t* block_table, const int32_t* ctx_lens,
                             const int32_t* q_lens, const int32_t* q_start, const int32_t* k_start,
                             const int32_t* k_seq, int32_t* tickets, const float* lse, const float* acc_in,
                             float* acc_out, int acc_len, float decay, int num_seqs, int mbps, int num_blocks, int Hq,
                             int Hkv, int d, int causal, float scale, int total_q, const ScoreMod& mod, cudaStream_t s,
                             const DevCtx& ctx);

__host__ __device__ inline bool is_decode_row(int q_len, int g) { return q_len >= 1 && g * q_len <= kDecodeRows; }

// Rows of a batch: sequence s has max(0, q_lens[s]) of them behind those of the sequences
// before it (q0, at most INT_MAX).  A sequence whose rows do not all lie in the call's
// total_q, as after lengths that are wrong, is reported (with the negative lengths) by the
// merge or the metadata kernel, and nothing of it is read from q or written.

// ------------------------------------------------------------------ layout --
constexpr int kStreamWarps = 8;      // page streams per decode CTA
constexpr int kMaxStreamCtas = 160;  // decode grid cap (one CTA per SM); sizes the partial slots

struct PagedWs {
    size_t q_start, work_count, work_list, part_o, part_ml, total;
    int max_entries;
};

// Workspace: scheduling lists of the tensor-core path, then two partial slots
// per decode CTA (16 rows of fp32 O, plus (max, sum) per row).
inline PagedWs paged_ws_layout(int num_seqs, int mbps, int Hq, int Hkv, int d, int total_q) {
    (void)Hq;
    (void)Hkv;
    (void)mbps;
    PagedWs w{};
    w.max_entries = total_q / 16 + num_seqs + 1;  // entries hold at least 16 tokens (paged_tc_entry_tokens)
    size_t off = 0;
    w.q_start = off;
    off = align256(off + sizeof(int32_t) * (size_t)(num_seqs + 1));
    w.work_count = off;
    off = align256(off + sizeof(int32_t) * 4);
    w.work_list = off;
    off = align256(off + sizeof(int32_t) * 2 * (size_t)w.max_entries);
    w.part_o = off;
    off = align256(off + sizeof(float) * (size_t)2 * kMaxStreamCtas * kDecodeRows * d);
    w.part_ml = off;
    off = align256(off + sizeof(float2) * (size_t)2 * kMaxStreamCtas * kDecodeRows);
    w.total = off;
    return w;
}

// -------------------------------------------------------------- decode -----
// Work is balanced by pages: the decode segments (sequence, kv head) are laid
// end to end, sequence-major, as one stream of 16-token pages; warp w of the
// grid takes pages [w*P/W, (w+1)*P/W), so CTA c holds pages [8c*P/W,
// (8c+8)*P/W).  A segment that lies inside one warp's range is finished by
// that warp (bf16 output); a segment cut by a warp's range boundary leaves
// that warp's partial (running max, row sum, unnormalised O) in shared memory,
// and the CTA combines the pieces of its warps: final rows for a segment inside
// the CTA's range, else the CTA's partial in slot 2c (the CTA's first segment)
// or 2c+1 (its last) for the merge kernel.  Every page is read once; every warp
// streams the same number of bytes, so no SM waits on a long sequence.

// First block of a context that a query of its chunk can see through a sliding
// window (0: no window): the chunk's first query sits at cl - ql.
__device__ __forceinline__ int first_block(int cl, int ql, int window) {
    return window > 0 ? max(0, cl - ql - window + 1) / kBS : 0;
}

// Pages one kv head of sequence s contributes to the decode stream (0 when the
// sequence takes the tensor-core path or its lengths are inconsistent).
__device__ __forceinline__ int decode_blocks(const int32_t* __restrict__ q_lens, const int32_t* __restrict__ ctx_lens,
                                             int s, int g, int mbps, int window) {
    const int ql = __ldg(q_lens + s), cl = __ldg(ctx_lens + s);
    if (!is_decode_row(ql, g) || ql > cl || cl > mbps * kBS) return 0;
    return (cl + kBS - 1) / kBS - first_block(cl, ql, window);
}

// The stream partition: warp w of W starts at page floor(w * P / W).  With
// P = qt * W + rm this is w * qt + (w * rm) / W, where (w * rm) < W * W fits
// 32 bits: one 64-bit division per kernel instead of one per lookup.
struct StreamSplit {
    long long P, qt;
    int rm, W;
    __device__ StreamSplit(long long P_, int W_) : P(P_), qt(P_ / W_), rm((int)(P_ - P_ / W_ * W_)), W(W_) {}
    __device__ __forceinline__ long long begin(int w) const {
        return (long long)w * qt + (int)((unsigned)w * (unsigned)rm / (unsigned)W);
    }
    // warp whose range holds page x (0 <= x < P): the last w with floor(w P / W) <= x,
    // that is w P < (x + 1) W
    __device__ __forceinline__ int owner(long long x) const { return (int)(((x + 1) * W - 1) / P); }
};

// Warps that share a modified call's stream: at most one per `pages` pages, in whole CTAs.
// (Spread over every CTA of the grid, a short context leaves one piece per page
// to the merge kernel: 90 pages took 22 us, in twelve CTAs they take half.)
__device__ __forceinline__ int stream_warps(int W, long long P, int pages) {
    const int cta = pages * kStreamWarps;
    return (int)min((long long)W, (P + cta - 1) / cta * kStreamWarps);
}

// The cache that a decode kernel reads: bf16, E4M3 with a scale for the whole cache, or
// E4M3 with a power of two for every block and kv head (PageMma's form).
enum { KV_BF16 = 0, KV_FP8 = 1, KV_FP8_SCALED = 2 };
constexpr int kPageBatch = 32;  // KV_FP8_SCALED: pages that a warp looks up at a time, a lane each

// Shared memory of a decode CTA: each warp's TMA ring, then each warp's slot
// for the partial of its first segment (ROWS query rows).  The ring has three
// stages (8 KB each at d = 128, 4 KB at d = 64) except at d = 128 with slots of
// 16 rows, which leave room for two; the 8-bit (E4M3) cache's pages are half
// the bytes, so its ring is twice as deep to keep the same bytes in flight.
template <int D, int KV, int ROWS>
struct StreamSmem {
    static constexpr bool KV8 = KV != KV_BF16;
    static constexpr int kPage = kBS * D * (KV8 ? 1 : 2);  // bytes of one K (or V) page
    static constexpr int kStage = 2 * kPage;              // K page + V page
    static constexpr int kStages = (KV8 ? 2 : 1) * (D == 128 && ROWS > 6 ? 2 : 3);
    static constexpr int kRing = kStreamWarps * kStages * kStage;
    // a partial: ROWS rows of unnormalised O (fp32, rows kSlotRow floats
    // apart), then (max, sum) per row
    static constexpr int kSlotRow = D + 8;
    static constexpr int kSlotBytes = ROWS * kSlotRow * 4 + ROWS * 8;
    static constexpr int kSlots = kStreamWarps * kSlotBytes;
    static constexpr int kBars = kStreamWarps * kStages + 1;
    static constexpr int kCutEntries = 2 * kStreamWarps;  // segments cut between the CTA's warps, at most
    static constexpr int kLists = KV == KV_FP8_SCALED ? kStreamWarps * 2 * kPageBatch * 8 : 0;  // pages looked up
    static constexpr int kBytes = 1024 /*align slack*/ + kRing + kSlots + kBars * 8 + 64 + kCutEntries * 32 + kLists;
    static_assert(kSlotBytes <= kStages * kStage, "a warp's ring holds the partial of its last segment");
    static_assert(kSlots % 64 == 0 && kSlotBytes % 16 == 0, "slots keep 16-byte alignment");
    static_assert((kStreamWarps * kStages * 8) % 64 == 0, "the barrier after the ring barriers is 64-byte aligned");
};

// Position of a stream cursor: sequence, kv head, block within the sequence.
struct Cursor {
    int s, hk, blk, nblk;  // nblk: pages per kv head of sequence s
    int blk0;              // block of the sequence that page 0 is (0 without a window)
    int q0;                // first packed query row of sequence s
};

// KV8 reads the 8-bit cache: K pages [16 tokens][D] bytes (128-byte swizzled
// rows), V pages [D channels][16 tokens] bytes; the warp MMAs run in f16
// (every E4M3 value is an f16 value; bf16 queries are converted to f16),
// k_scale is folded into scale_log2 by the host and v_scale multiplies the
// output.  The MMA's K dimension is taken in a permuted order so that one
// ldmatrix lane word (4 consecutive bytes = 4 channels, or 4 tokens of V)
// gives both B registers: logical k (2t, 2t+1, 2t+8, 2t+9) of a 16-wide step
// = elements (4t .. 4t+3); queries are loaded in the same order for Q K^T,
// and for P V the S tile's columns (tokens) are produced in that order by
// loading K rows 4t+2nt+e into n-tile nt, column 2t+e.
// MOD 1 applies the score modifiers `mod` (cap, distance slopes, window, prefix)
// and writes the rows' log-sum-exp; a window drops whole blocks from the
// stream.  MOD 2 also keeps every logit (log2 units, -inf where masked) at
// [page of the stream][row][token] for the weight sums that need the final
// log-sum-exp: logit_rows * 64 bytes beside the page's 64 d.
constexpr int kLensPerLane = 8;  // sequences per lane whose lengths are loaded in one batch
constexpr float kLn2f = 0.6931471805599453f, kLog2ef = 1.4426950408889634f;
// KV_FP8_SCALED takes the warps' pages two (d = 64: four) at a time, and block numbers
// and scales ahead in batches of 32.
template <int D, int KV, int ROWS, int MOD>
__global__ void __launch_bounds__(kStreamWarps * 32, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const uint16_t* __restrict__ q, const int32_t* __restrict__ bt,
                        const int32_t* __restrict__ ctx_lens, const int32_t* __restrict__ q_lens,
                        uint16_t* __restrict__ out, float* __restrict__ part_o, float2* __restrict__ part_ml,
                        int num_seqs, int mbps, int num_blocks, int Hq, int Hkv, int q_prefetch_rows, int causal,
                        float scale_log2, float v_scale, int total_q, DevCtx ctx, ScoreMod mod,
                        const uint8_t* __restrict__ k_exp, const uint8_t* __restrict__ v_exp) {
    constexpr bool KV8 = KV != KV_BF16, SCALED = KV == KV_FP8_SCALED;
    static_assert(MOD == 0 || !KV8, "score modifiers are built for the bf16 cache");
    const int window = MOD ? mod.window : 0;
    // the merge kernel that follows may be scheduled now; it waits for this
    // grid's completion before reading anything
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    using L = StreamSmem<D, KV, ROWS>;
    constexpr int kStreamStages = L::kStages;  // ring depth of this variant
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kRing + L::kSlots);
    uint64_t* never = bars + kStreamWarps * kStreamStages;  // nothing arrives on it (time-out test hook)
    volatile int* abort_flag = reinterpret_cast<volatile int*>(never + 1);
    int* cut_count = const_cast<int*>(abort_flag) + 1;  // entries in cut_table
    // 2 int4 per entry, see the end; `never` is 64-byte aligned (the ring, the
    // slots and the barriers before it are multiples of 64 bytes), so this is 16
    int4* cut_table = reinterpret_cast<int4*>(never + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = Hq / Hkv;
    int W = gridDim.x * kStreamWarps;
    const int gw = blockIdx.x * kStreamWarps + warp;
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        for (int i = 0; i < L::kBars; ++i) mbar_init(&bars[i], 1);
        *abort_flag = 0;
        *cut_count = 0;
        mbar_fence_init();
    }
    {
        // warm L2 with this CTA's share of the block table and (when every
        // query row is a decode row) of the queries, read right after the lengths
        constexpr long kMaxPrefetchLines = (4L << 20) / 128;  // 4 MB each at most
        const long tb_lines = min(kMaxPrefetchLines, ((long)num_seqs * mbps * 4 + 127) / 128);
        const long q_lines = min(kMaxPrefetchLines, ((long)q_prefetch_rows * Hq * D * 2 + 127) / 128);
        const long tb_lo = tb_lines * blockIdx.x / gridDim.x, tb_hi = tb_lines * (blockIdx.x + 1) / gridDim.x;
        const long q_lo = q_lines * blockIdx.x / gridDim.x, q_hi = q_lines * (blockIdx.x + 1) / gridDim.x;
        for (long i = tb_lo + threadIdx.x; i < tb_hi; i += blockDim.x)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(bt) + i * 128));
        for (long i = q_lo + threadIdx.x; i < q_hi; i += blockDim.x)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(q) + i * 128));
    }

    // Where this warp's pages start.  Every warp finds out on its own (no
    // CTA-wide step on the path to the first copy): lane j sums the decode
    // pages and the query rows of sequences [j*per, (j+1)*per), and a warp
    // scan gives each lane's offsets and the total P.
    const int per = (num_seqs + 31) >> 5;
    const int s_lo = min(num_seqs, lane * per), s_hi = min(num_seqs, s_lo + per);
    long long my_p = 0, my_q = 0;
    bool bad = false;
    auto count = [&](int ql, int cl) {
        my_q += max(0, ql);
        if (!is_decode_row(ql, g)) return;
        if (ql > cl || cl > mbps * kBS) {
            bad = true;
            return;
        }
        my_p += (long long)Hkv * ((cl + kBS - 1) / kBS - first_block(cl, ql, window));
    };
    if (per <= kLensPerLane) {
        int qv[kLensPerLane], cv[kLensPerLane];
#pragma unroll
        for (int i = 0; i < kLensPerLane; ++i) {  // all loads issued before any is used
            const bool in = s_lo + i < s_hi;
            qv[i] = in ? __ldg(q_lens + s_lo + i) : 0;
            cv[i] = in ? __ldg(ctx_lens + s_lo + i) : 0;
        }
        __syncthreads();  // barrier initialisation visible to every warp (the loads are in flight)
#pragma unroll
        for (int i = 0; i < kLensPerLane; ++i)
            if (s_lo + i < s_hi) count(qv[i], cv[i]);
    } else {
        __syncthreads();
#pragma unroll 4
        for (int s = s_lo; s < s_hi; ++s) count(__ldg(q_lens + s), __ldg(ctx_lens + s));
    }
    if (bad && gw == 0) raise_error(ctx, ERR_BOUNDS_BIT);
    long long inc_p = my_p, inc_q = my_q;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long yp = __shfl_up_sync(0xffffffffu, inc_p, o), yq = __shfl_up_sync(0xffffffffu, inc_q, o);
        if (lane >= o) {
            inc_p += yp;
            inc_q += yq;
        }
    }
    const long long P = __shfl_sync(0xffffffffu, inc_p, 31);
    if (P == 0) return;
    if constexpr (MOD != 0 || SCALED) {
        W = stream_warps(W, P, SCALED ? 2 : 1);
        if (gw >= W) return;  // a whole CTA
    }
    const StreamSplit split(P, W);
    const long long b0 = split.begin(gw), b1 = split.begin(gw + 1);
    const int n_pages = (int)(b1 - b0);
    if (n_pages <= 0) return;  // not among the warps of the CTA barrier at the end
    // the lane whose sequences hold page b0 walks them (lengths are L1 hits now)
    Cursor start;
    {
        const unsigned hit = __ballot_sync(0xffffffffu, my_p > 0 && b0 >= inc_p - my_p && b0 < inc_p);
        const int src = __ffs(hit) - 1;  // exactly one lane: 0 <= b0 < P
        int a_s = 0, a_off = 0, a_q0 = 0;
        if (lane == src) {
            long long off = b0 - (inc_p - my_p), q0 = inc_q - my_q;
            for (int s = s_lo; s < s_hi; ++s) {
                const int ql = __ldg(q_lens + s), cl = __ldg(ctx_lens + s);
                const long long n =
                    (is_decode_row(ql, g) && ql <= cl && cl <= mbps * kBS)
                        ? (long long)Hkv * ((cl + kBS - 1) / kBS - first_block(cl, ql, window))
                        : 0;
                if (off < n) {
                    a_s = s;
                    a_off = (int)off;
                    a_q0 = (int)min(q0, 0x7fffffffll);
                    break;
                }
                off -= n;
                q0 += max(0, ql);
            }
        }
        start.s = __shfl_sync(0xffffffffu, a_s, src);
        a_off = __shfl_sync(0xffffffffu, a_off, src);
        start.q0 = __shfl_sync(0xffffffffu, a_q0, src);
        start.nblk = decode_blocks(q_lens, ctx_lens, start.s, g, mbps, window);
        start.blk0 = MOD ? first_block(__ldg(ctx_lens + start.s), __ldg(q_lens + start.s), window) : 0;
        start.hk = a_off / start.nblk;
        start.blk = a_off % start.nblk;
    }

    uint8_t* ring = smem + warp * kStreamStages * L::kStage;
    uint64_t* wbar = bars + warp * kStreamStages;
    // Partials of segments cut by a range boundary stay in shared memory:
    // the first segment's in this warp's slot, the last one's (when it is
    // another segment) in this warp's ring, free once its last page is read.
    float* slot_first = reinterpret_cast<float*>(smem + L::kRing + warp * L::kSlotBytes);
    float* slot_last = reinterpret_cast<float*>(ring);
    // advances a cursor by one page; entering a new sequence skips the ones
    // with no decode pages and carries the packed query offset along
    auto advance = [&](Cursor& c) {
        if (++c.blk < c.nblk) return;
        c.blk = 0;
        if (++c.hk < Hkv) return;
        c.hk = 0;
        do {
            c.q0 = (int)min((unsigned)c.q0 + (unsigned)max(0, __ldg(q_lens + c.s)), 0x7fffffffu);
            ++c.s;
            c.nblk = c.s < num_seqs ? decode_blocks(q_lens, ctx_lens, c.s, g, mbps, window) : 0;
        } while (c.s < num_seqs && c.nblk == 0);
        if constexpr (MOD != 0)
            if (c.s < num_seqs) c.blk0 = first_block(__ldg(ctx_lens + c.s), __ldg(q_lens + c.s), window);
    };

    Cursor ci = start;  // issue cursor (lane 0 only; SCALED: of the next batch's first page)
    // SCALED: (block, kv head << 16 | v scale << 8 | k scale) of the warp's pages, two batches by turns.  Lane j
    // looks up page j of the batch at `ci`: its place, its block (into `found`), and later its scales.
    [[maybe_unused]] int2* list = reinterpret_cast<int2*>(cut_table + 2 * L::kCutEntries) + warp * 2 * kPageBatch;
    [[maybe_unused]] int found = -1, found_hk = 0, found_scales = 0;
    [[maybe_unused]] auto look_up_blocks = [&](int first) {  // pages first .. first + 31 of the warp
        found = -1;
        const bool in = first + lane < n_pages;
        Cursor c = ci;
        int off = lane;  // pages from `ci` on
        while (in) {
            const int left = c.nblk - c.blk;
            if (off < left) break;
            off -= left;
            c.blk = c.nblk - 1;
            advance(c);
        }
        if (in) {
            c.blk += off;
            found = __ldg(bt + (long)c.s * mbps + c.blk);
            found_hk = c.hk;
            if (lane == kPageBatch - 1) advance(c);
        }
        // the next batch begins behind the last lane's page (if there is one)
        ci.s = __shfl_sync(0xffffffffu, c.s, kPageBatch - 1);
        ci.hk = __shfl_sync(0xffffffffu, c.hk, kPageBatch - 1);
        ci.blk = __shfl_sync(0xffffffffu, c.blk, kPageBatch - 1);
        ci.nblk = __shfl_sync(0xffffffffu, c.nblk, kPageBatch - 1);
    };
    [[maybe_unused]] auto look_up_scales = [&]() {
        found_scales = kExpBias | kExpBias << 8;  // (outside the pool: zeros at scale 1, as the chunks' kernel)
        if (found >= 0 && found < num_blocks) {
            const long at = (long)found * Hkv + found_hk;
            found_scales = __ldg(k_exp + at) | __ldg(v_exp + at) << 8;
        }
    };
    [[maybe_unused]] auto keep_blocks = [&](int first) {
        int phys = found;
        if (first + lane < n_pages && (phys < 0 || phys >= num_blocks)) {
            raise_error(ctx, ERR_BOUNDS_BIT);
            phys = num_blocks;  // outside the tensor map: the copy fills zeros
        }
        list[(first / kPageBatch & 1) * kPageBatch + lane] = make_int2(phys, (int)((unsigned)found_hk << 16));
        __syncwarp();
    };
    [[maybe_unused]] auto keep_scales = [&](int first) {
        list[(first / kPageBatch & 1) * kPageBatch + lane].y = (int)((unsigned)found_hk << 16 | (unsigned)found_scales);
        __syncwarp();
    };
    // lane 0 reads the block-table entry of the next page one issue ahead, so
    // that load's latency is not on the copy's path
    int next_phys = !SCALED && lane == 0 ? __ldg(bt + (long)ci.s * mbps + ci.blk0 + ci.blk) : 0;
    auto issue = [&](int i) {
        const int stage = i % kStreamStages;
        if constexpr (SCALED) {
            const int2 e = list[i % (2 * kPageBatch)];
            load_page<D, true>(ring + stage * L::kStage, &tm_k, &tm_v, &wbar[stage], (int)((unsigned)e.y >> 16), e.x);
            return;
        }
        int phys = next_phys;
        if (phys < 0 || phys >= num_blocks) {
            raise_error(ctx, ERR_BOUNDS_BIT);
            phys = num_blocks;  // outside the tensor map: the copy fills zeros
        }
        uint8_t* kp = ring + stage * L::kStage;
        uint8_t* vp = kp + L::kPage;
        mbar_arrive_expect_tx(&wbar[stage], L::kStage);
        if constexpr (KV8) {  // one box per page: K rows, V channel rows
            tma_load_4d(kp, &tm_k, &wbar[stage], 0, 0, ci.hk, phys);
            tma_load_4d(vp, &tm_v, &wbar[stage], 0, 0, ci.hk, phys);
        } else {
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                tma_load_4d(kp + h * 2048, &tm_k, &wbar[stage], h * 64, 0, ci.hk, phys);
                tma_load_4d(vp + h * 2048, &tm_v, &wbar[stage], h * 64, 0, ci.hk, phys);
            }
        }
        advance(ci);
        if (i + 1 < n_pages) next_phys = __ldg(bt + (long)ci.s * mbps + ci.blk0 + ci.blk);
    };
    bool ok = !ctx.force_timeout || mbar_wait_warp(never, 0, ctx.wait_ns, abort_flag);
    if (!ok && lane == 0) {
        raise_error(ctx, ERR_TIMEOUT_BIT);
        *abort_flag = 1;
    }
    int issued = 0;  // lane 0's count of copies issued
    if constexpr (SCALED) {
        look_up_blocks(0);
        keep_blocks(0);
        look_up_scales();  // (on their way while the first pages are asked for)
    }
    if (lane == 0 && ok)
        for (; issued < n_pages && issued < kStreamStages; ++issued) issue(issued);
    if constexpr (SCALED) {
        __syncwarp();
        keep_scales(0);
    }

    const int gid = lane >> 2, tig = lane & 3, mi = lane >> 3, r8 = lane & 7;
    Cursor cc = start;            // compute cursor (all lanes)
    long long seg_first = b0 - start.blk;  // global index of the current segment's first page
    Cursor seg_last = start;               // the segment begun last, its first page and query rows
    long long seg_last_first = seg_first;
    int seg_last_rows = 0, first_rows = -1;  // and the first segment's query rows
    int ctx_len = 0, q_len = 0, nrows = 0, pos_r0 = 0, pos_r1 = 0;
    int qpos[2] = {0, 0}, lo_r[2] = {0, 0};  // MOD: position and first visible key of rows gid, gid + 8
    float slope[2] = {0.f, 0.f};             // MOD: their distance slopes (log2 units)
    PageMma<D, KV8> acc;  // the segment's queries, running max and sum, and O
    auto& qa = acc.qa;
    auto& o = acc.o;
    float &m0 = acc.m[0], &m1 = acc.m[1], &l0 = acc.l[0], &l1 = acc.l[1];
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;

    // starts segment (cc.s, cc.hk): loads its query rows as MMA A fragments
    // (rows r = token * g + head-in-group) and resets the softmax state
    auto begin_segment = [&]() {
        seg_last = cc;
        seg_last_first = seg_first;
        ctx_len = __ldg(ctx_lens + cc.s);
        q_len = __ldg(q_lens + cc.s);
        nrows = rows_fit(cc.q0, q_len, total_q) ? g * q_len : 0;  // (else none is read or written)
        seg_last_rows = nrows;
        if (first_rows < 0) first_rows = nrows;
        const int rr[2] = {gid, gid + 8};
        const uint16_t* qrow[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            qrow[i] = rr[i] < nrows ? q + ((long)(cc.q0 + rr[i] / g) * Hq + cc.hk * g + rr[i] % g) * D : nullptr;
        if constexpr (SCALED) {
            acc.load_q(qrow[0], qrow[1], scale_log2);
        } else if constexpr (KV8) {
            // f16, channels 4t .. 4t+3 of each 16-channel step (the permuted K order)
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint2 w = qrow[i] ? __ldg(reinterpret_cast<const uint2*>(qrow[i] + ks * 16 + tig * 4))
                                            : make_uint2(0u, 0u);
                    qa[ks][i] = pack_f16x2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u));
                    qa[ks][i + 2] = pack_f16x2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
                }
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const int c = ks * 16 + tig * 2;
                qa[ks][0] = qrow[0] ? __ldg(reinterpret_cast<const uint32_t*>(qrow[0] + c)) : 0u;
                qa[ks][1] = qrow[1] ? __ldg(reinterpret_cast<const uint32_t*>(qrow[1] + c)) : 0u;
                qa[ks][2] = qrow[0] ? __ldg(reinterpret_cast<const uint32_t*>(qrow[0] + c + 8)) : 0u;
                qa[ks][3] = qrow[1] ? __ldg(reinterpret_cast<const uint32_t*>(qrow[1] + c + 8)) : 0u;
            }
        }
        // keys <= pos(row) are visible
        pos_r0 = causal ? ctx_len - q_len + gid / g : ctx_len - 1;
        pos_r1 = causal ? ctx_len - q_len + (gid + 8) / g : ctx_len - 1;
        if constexpr (MOD != 0) {
            const int prefix = causal && mod.prefix ? max(0, __ldg(mod.prefix + cc.s)) : 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                qpos[i] = ctx_len - q_len + rr[i] / g;
                lo_r[i] = window > 0 ? qpos[i] - window + 1 : 0;
                slope[i] = mod.slopes && rr[i] < nrows ? slope_log2(__ldg(mod.slopes + cc.hk * g + rr[i] % g)) : 0.f;
            }
            pos_r0 = max(pos_r0, prefix - 1);
            pos_r1 = max(pos_r1, prefix - 1);
            if (!causal && window > 0) {
                pos_r0 = min(pos_r0, qpos[0] + window - 1);
                pos_r1 = min(pos_r1, qpos[1] + window - 1);
            }
        }
#pragma unroll
        for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
    };
    // finishes the current segment: final bf16 rows when the whole segment
    // was in this warp's range, otherwise a partial in shared memory
    auto end_segment = [&]() {
        float la = l0 + __shfl_xor_sync(0xffffffffu, l0, 1);
        la += __shfl_xor_sync(0xffffffffu, la, 2);
        float lb = l1 + __shfl_xor_sync(0xffffffffu, l1, 1);
        lb += __shfl_xor_sync(0xffffffffu, lb, 2);
        const bool whole = seg_first >= b0 && seg_first + cc.nblk <= b1;
        const int rr[2] = {gid, gid + 8};
        const float ml[2] = {m0, m1}, ls[2] = {la, lb};
        if (whole) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = rr[i];
                if (r >= nrows) continue;
                const float inv = ls[i] > 0.f ? v_scale / ls[i] : 0.f;
                uint16_t* dst = out + ((long)(cc.q0 + r / g) * Hq + cc.hk * g + r % g) * D;
                if constexpr (MOD != 0 || SCALED)
                    if (mod.lse && tig == 0)
                        mod.lse[(long)(cc.q0 + r / g) * Hq + cc.hk * g + r % g] =
                            ls[i] > 0.f ? (ml[i] + __log2f(ls[i])) * kLn2f : -INFINITY;
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<uint32_t*>(dst + n * 8 + tig * 2) =
                        pack_bf16x2(o[n][2 * i] * inv, o[n][2 * i + 1] * inv);
            }
        } else {
            // a slot holds ROWS rows: more means max_q_len was below a chunk's length
            if (nrows > ROWS && lane == 0) raise_error(ctx, ERR_BOUNDS_BIT);
            float* so = seg_first <= b0 ? slot_first : slot_last;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = rr[i];
                if (r >= nrows || r >= ROWS) continue;
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2*>(so + r * L::kSlotRow + n * 8 + tig * 2) =
                        make_float2(o[n][2 * i] * v_scale, o[n][2 * i + 1] * v_scale);
                if (tig == 0) reinterpret_cast<float2*>(so + ROWS * L::kSlotRow)[r] = make_float2(ml[i], ls[i]);
            }
        }
    };

    int consumed = 0;
    if (ok) begin_segment();
    if constexpr (SCALED) {
        constexpr int NP = D == 64 ? 4 : 2;  // pages at a time
        static_assert(NP < kStreamStages && kStreamStages + NP <= kPageBatch, "copies in flight during a pass");
        int ready = kPageBatch;  // pages whose list entries are kept
        int step = 0;            // of the next batch: 0 nothing, 1 blocks asked for, 2 scales asked for
        for (int i = 0; ok && i < n_pages;) {
            if (i > 0 && cc.blk == 0) {  // the cursor entered a new segment
                seg_first = b0 + i;
                begin_segment();
            }
            const int np = min(NP, min(n_pages - i, cc.nblk - cc.blk));
            uint32_t kv[NP];
            int tok[NP], ks[NP], ev[NP];
#pragma unroll
            for (int j = 0; j < NP; ++j) {
                const int stage = (i + j) % kStreamStages;
                kv[j] = smem_u32(ring + stage * L::kStage);
                const unsigned e = (unsigned)list[(i + j) % (2 * kPageBatch)].y;
                ks[j] = (int)(e & 255u);
                ev[j] = (int)(e >> 8 & 255u);
                tok[j] = (cc.blk + j) * kBS;
                if (j < np && ok && !mbar_wait_warp(&wbar[stage], ((i + j) / kStreamStages) & 1, ctx.wait_ns, abort_flag)) {
                    if (lane == 0) {
                        raise_error(ctx, ERR_TIMEOUT_BIT);
                        *abort_flag = 1;
                    }
                    ok = false;
                }
            }
            if (!ok) break;
            acc.template step<NP>(np, kv, tok, ks, ev, pos_r0, pos_r1, ctx_len);
            __syncwarp();
            if (i + np == n_pages || cc.blk + np == cc.nblk) end_segment();
            cc.blk += np - 1;
            advance(cc);
            i += np;
            consumed = i;
            // The next batch: its blocks as early as can be, its scales 16 pages ahead, its list when the next
            // copy needs it.  (The half that it takes held pages below i by then: the ring is shorter than a batch.)
            if (ready < n_pages) {
                const bool now = i + kStreamStages > ready;
                if (step == 0) {
                    look_up_blocks(ready);
                    step = 1;
                } else if (step == 1 && i + kStreamStages + kPageBatch / 2 > ready) {
                    look_up_scales();
                    step = 2;
                }
                if (now) {
                    if (step == 1) look_up_scales();
                    keep_blocks(ready);
                    keep_scales(ready);
                    ready += kPageBatch;
                    step = 0;
                }
            }
            if (lane == 0)
                while (issued < n_pages && issued < i + kStreamStages) issue(issued++);
        }
    } else
    for (int i = 0; ok && i < n_pages; ++i, consumed = i) {
        if (i > 0 && cc.blk == 0) {  // the cursor entered a new segment
            seg_first = b0 + i;
            begin_segment();
        }
        const int stage = i % kStreamStages;
        if (!mbar_wait_warp(&wbar[stage], (i / kStreamStages) & 1, ctx.wait_ns, abort_flag)) {
            if (lane == 0) {
                raise_error(ctx, ERR_TIMEOUT_BIT);
                *abort_flag = 1;
            }
            ok = false;
            break;
        }
        const uint32_t kbase = smem_u32(ring + stage * L::kStage);
        const uint32_t vbase = kbase + L::kPage;
        const int tok0 = (cc.blk0 + cc.blk) * kBS;

        // S = Q K^T : 16 rows x 16 tokens
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        if constexpr (KV8) {
            // matrix mi: n-tile mi & 1, 16-byte chunk 2j + (mi >> 1); its row r8
            // is token 4 (r8 / 2) + 2 (mi & 1) + r8 % 2 (the S column order P V uses)
            const int tok = (r8 >> 1) * 4 + 2 * (mi & 1) + (r8 & 1);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const int chunk = 2 * j + (mi >> 1);
                uint32_t w[4], b[8];
                ldsm_x4(kbase + tok * D + ((chunk ^ (tok & 7)) << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int m = 0; m < 4; ++m) e4m3x4_to_f16x4(w[m], b[2 * m], b[2 * m + 1]);
                mma_f16_16816(sc[0], qa[2 * j], b[0], b[1]);
                mma_f16_16816(sc[1], qa[2 * j], b[2], b[3]);
                mma_f16_16816(sc[0], qa[2 * j + 1], b[4], b[5]);
                mma_f16_16816(sc[1], qa[2 * j + 1], b[6], b[7]);
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                const int tok = (mi >> 1) * 8 + r8;
                const int chunk = ks * 2 + (mi & 1);
                uint32_t b0r, b1r, b2r, b3r;
                ldsm_x4(kbase + (chunk >> 3) * 2048 + sw128_offset(tok, chunk & 7), b0r, b1r, b2r, b3r);
                mma_bf16_16816(sc[0], qa[ks], b0r, b1r);
                mma_bf16_16816(sc[1], qa[ks], b2r, b3r);
            }
        }
        // mask + online softmax (base 2)
        float x[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = KV8 ? tok0 + tig * 4 + nt * 2 + (e & 1) : tok0 + nt * 8 + tig * 2 + (e & 1);
                const int lim = (e < 2) ? pos_r0 : pos_r1;
                if constexpr (MOD != 0) {
                    float z = mod.cap_out > 0.f ? mod.cap_out * tanh_f32(sc[nt][e] * mod.cap_in) : sc[nt][e] * scale_log2;
                    z = fmaf(-slope[e >> 1], fabsf((float)(t - qpos[e >> 1])), z);
                    x[nt][e] = (t <= lim && t < ctx_len && t >= lo_r[e >> 1]) ? z : -INFINITY;
                } else {
                    x[nt][e] = (t <= lim && t < ctx_len) ? sc[nt][e] * scale_log2 : -INFINITY;
                }
            }
        if constexpr (MOD == 2) {
            float* lg = mod.logits + (long)(b0 + i) * mod.logit_rows * kBS + tig * 2;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int rr = 0; rr < 2; ++rr)
                    if (gid + 8 * rr < min(nrows, mod.logit_rows))
                        *reinterpret_cast<float2*>(lg + (gid + 8 * rr) * kBS + nt * 8) =
                            make_float2(x[nt][2 * rr], x[nt][2 * rr + 1]);
        }
        float mx0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
        float mx1 = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
        const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
        const float mu0 = mn0 == -INFINITY ? 0.f : mn0, mu1 = mn1 == -INFINITY ? 0.f : mn1;
        const float a0 = fast_exp2(m0 - mu0), a1 = fast_exp2(m1 - mu1);
        m0 = mn0;
        m1 = mn1;
        float pr[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            pr[nt][0] = fast_exp2(x[nt][0] - mu0);
            pr[nt][1] = fast_exp2(x[nt][1] - mu0);
            pr[nt][2] = fast_exp2(x[nt][2] - mu1);
            pr[nt][3] = fast_exp2(x[nt][3] - mu1);
        }
        l0 = l0 * a0 + (pr[0][0] + pr[0][1] + pr[1][0] + pr[1][1]);
        l1 = l1 * a1 + (pr[0][2] + pr[0][3] + pr[1][2] + pr[1][3]);
        if (__any_sync(0xffffffffu, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                o[n][0] *= a0;
                o[n][1] *= a0;
                o[n][2] *= a1;
                o[n][3] *= a1;
            }
        }
        uint32_t pa[4];
        if constexpr (KV8) {
            pa[0] = pack_f16x2(pr[0][0], pr[0][1]);
            pa[1] = pack_f16x2(pr[0][2], pr[0][3]);
            pa[2] = pack_f16x2(pr[1][0], pr[1][1]);
            pa[3] = pack_f16x2(pr[1][2], pr[1][3]);
        } else {
            pa[0] = pack_bf16x2(pr[0][0], pr[0][1]);
            pa[1] = pack_bf16x2(pr[0][2], pr[0][3]);
            pa[2] = pack_bf16x2(pr[1][0], pr[1][1]);
            pa[3] = pack_bf16x2(pr[1][2], pr[1][3]);
        }
        // O += P V : V rows past the context are zeroed so stale cache words
        // (possibly NaN) cannot reach the accumulator through a zero weight
        const int nvalid = ctx_len - tok0;  // >= 1
        if constexpr (KV8) {
            // V page rows are channels (16 token bytes each); matrix mi of
            // step q4 is n-tile 4 q4 + mi; a lane word holds tokens 4t .. 4t+3
            const uint32_t zb = (tig * 4 < nvalid ? 0x000000ffu : 0u) | (tig * 4 + 1 < nvalid ? 0x0000ff00u : 0u) |
                                (tig * 4 + 2 < nvalid ? 0x00ff0000u : 0u) | (tig * 4 + 3 < nvalid ? 0xff000000u : 0u);
#pragma unroll
            for (int q4 = 0; q4 < D / 32; ++q4) {
                uint32_t w[4];
                ldsm_x4(vbase + ((4 * q4 + mi) * 8 + r8) * 16, w[0], w[1], w[2], w[3]);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    uint32_t b0r, b1r;
                    e4m3x4_to_f16x4(w[m] & zb, b0r, b1r);
                    mma_f16_16816(o[4 * q4 + m], pa, b0r, b1r);
                }
            }
        } else {
            const uint32_t zlo =
                (tig * 2 < nvalid ? 0x0000ffffu : 0u) | (tig * 2 + 1 < nvalid ? 0xffff0000u : 0u);
            const uint32_t zhi =
                (tig * 2 + 8 < nvalid ? 0x0000ffffu : 0u) | (tig * 2 + 9 < nvalid ? 0xffff0000u : 0u);
#pragma unroll
            for (int dn = 0; dn < D / 16; ++dn) {
                const int tok = (mi & 1) * 8 + r8;
                const int chunk = dn * 2 + (mi >> 1);
                uint32_t b0r, b1r, b2r, b3r;
                ldsm_x4_t(vbase + (chunk >> 3) * 2048 + sw128_offset(tok, chunk & 7), b0r, b1r, b2r, b3r);
                b0r &= zlo;
                b2r &= zlo;
                b1r &= zhi;
                b3r &= zhi;
                mma_bf16_16816(o[2 * dn], pa, b0r, b1r);
                mma_bf16_16816(o[2 * dn + 1], pa, b2r, b3r);
            }
        }
        __syncwarp();
        if (lane == 0 && issued < n_pages) issue(issued++);
        // leaving the segment: last page of the range or of the segment
        const bool last_here = (i + 1 == n_pages) || (cc.blk + 1 == cc.nblk);
        if (last_here) end_segment();
        advance(cc);
    }
    if (!ok && lane == 0) {
        // drain: let the copies this warp issued but did not consume land
        // before the CTA can exit
        for (int i = consumed; i < issued; ++i)
            (void)mbar_wait_bounded(&wbar[i % kStreamStages], (i / kStreamStages) & 1, 1000000000ull, nullptr);
    }

    // Segments cut between this CTA's warps (or by the CTA's range boundaries).
    // The warp holding a segment's first page within the CTA's range lists it;
    // then the CTA's warps share out the listed rows and combine the pieces of
    // the CTA's warps, from shared memory, with log-sum-exp weights: into the
    // final bf16 rows when the segment lies inside the CTA's range, otherwise
    // into the CTA's partial (slot 2c for the segment holding the CTA's first
    // page, 2c+1 for the one holding its last) for the merge kernel.  Warps
    // without pages have left; the barriers count the others.
    const int cw0 = blockIdx.x * kStreamWarps;
    long long wb[kStreamWarps + 1];  // first page of each warp of this CTA, then the CTA's end
#pragma unroll
    for (int w = 0; w <= kStreamWarps; ++w) wb[w] = split.begin(cw0 + w);
    unsigned busy = 0;  // warps of this CTA with pages
#pragma unroll
    for (int w = 0; w < kStreamWarps; ++w) busy |= (wb[w + 1] > wb[w] ? 1u : 0u) << w;
    const int nbusy = __popc(busy);
    asm volatile("bar.sync 1, %0;" ::"r"(32 * nbusy) : "memory");
    if (*abort_flag) return;
    const long long c0 = wb[0], c1 = wb[kStreamWarps];
    // 1. the warp holding a cut segment's first page within the CTA lists it:
    //    (first query row, kv head, rows, pieces) and (output kind, slot, source slot of its own piece)
    for (int which = 0; which < 2; ++which) {
        const Cursor X = which ? seg_last : start;
        const long long sf = which ? seg_last_first : b0 - start.blk;
        if (which == 1 && sf == b0 - start.blk) break;  // one segment only
        const long long se = sf + X.nblk;
        if (sf >= b0 && se <= b1) continue;  // finished by this warp
        if (sf < b0 && b0 > c0) continue;    // an earlier warp of the CTA holds its first piece here
        // pieces: this warp and the later warps of the CTA whose pages start
        // before the segment's end (warps without pages wrote nothing)
        const long long lim = min(se, c1);
        unsigned mask = 0;
#pragma unroll
        for (int w = 0; w < kStreamWarps; ++w)
            if (w >= warp && wb[w] < lim && ((busy >> w) & 1u)) mask |= 1u << w;
        if (lane == 0) {
            const int e = atomicAdd(cut_count, 1);  // < kCutEntries: at most two per warp
            const bool final_rows = sf >= c0 && se <= c1;
            cut_table[2 * e] = make_int4(X.q0, X.hk, min(ROWS, which ? seg_last_rows : first_rows), (int)mask);
            cut_table[2 * e + 1] = make_int4(final_rows ? -1 : 2 * (int)blockIdx.x + (sf <= c0 ? 0 : 1), warp, which, 0);
        }
    }
    asm volatile("bar.sync 1, %0;" ::"r"(32 * nbusy) : "memory");
    // 2. the CTA's warps share out the listed segments' rows: per row, the
    //    pieces are combined with log-sum-exp weights into the final bf16 row
    //    (segment inside the CTA's range) or the CTA's partial for the merge kernel
    const int n_cut = *cut_count;
    const int rank = __popc(busy & ((1u << warp) - 1u));
    constexpr int kPer = D / 32;  // channels per lane
    int e = 0, e_row0 = 0;        // entry of the current item, and its first item index
    for (int it = rank;; it += nbusy) {
        int4 h = make_int4(0, 0, 0, 0);
        while (e < n_cut) {
            h = cut_table[2 * e];
            if (it < e_row0 + h.z) break;
            e_row0 += h.z;
            ++e;
        }
        if (e >= n_cut) break;
        const int4 t = cut_table[2 * e + 1];
        const int r = it - e_row0;
        const unsigned mask = (unsigned)h.w;
        // piece of warp w: the listing warp's own slot (first or last segment), else warp w's first-segment slot
        auto piece = [&](int w) -> const float* {
            if (w == t.y && t.z) return reinterpret_cast<const float*>(smem + w * kStreamStages * L::kStage);
            return reinterpret_cast<const float*>(smem + L::kRing + w * L::kSlotBytes);
        };
        float2 ml[kStreamWarps];
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kStreamWarps; ++w) {
            ml[w] = ((mask >> w) & 1u) ? reinterpret_cast<const float2*>(piece(w) + ROWS * L::kSlotRow)[r]
                                       : make_float2(-INFINITY, 0.f);
            M = fmaxf(M, ml[w].x);
        }
        float lsum = 0.f, acc[kPer];
#pragma unroll
        for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
#pragma unroll
        for (int w = 0; w < kStreamWarps; ++w) {
            if (!((mask >> w) & 1u)) continue;
            const float wt = ml[w].x == -INFINITY ? 0.f : fast_exp2(ml[w].x - M);
            lsum += wt * ml[w].y;
            const float* src = piece(w) + r * L::kSlotRow + lane * kPer;
            if constexpr (kPer == 4) {
                const float4 v = *reinterpret_cast<const float4*>(src);
                acc[0] += wt * v.x;
                acc[1] += wt * v.y;
                acc[2] += wt * v.z;
                acc[3] += wt * v.w;
            } else {
                const float2 v = *reinterpret_cast<const float2*>(src);
                acc[0] += wt * v.x;
                acc[1] += wt * v.y;
            }
        }
        if (t.x < 0) {
            const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
            uint16_t* dst = out + ((long)(h.x + r / g) * Hq + h.y * g + r % g) * D + lane * kPer;
            if constexpr (MOD != 0 || SCALED)
                if (mod.lse && lane == 0)
                    mod.lse[(long)(h.x + r / g) * Hq + h.y * g + r % g] =
                        lsum > 0.f ? (M + __log2f(lsum)) * kLn2f : -INFINITY;
            if constexpr (kPer == 4)
                *reinterpret_cast<uint2*>(dst) =
                    make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
            else
                *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
        } else {
            float* dst = part_o + ((long)t.x * kDecodeRows + r) * D + lane * kPer;
            if constexpr (kPer == 4)
                *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            else
                *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
            if (lane == 0) part_ml[(long)t.x * kDecodeRows + r] = make_float2(M, lsum);
        }
    }
}

// Merges the partials of segments cut by the decode CTAs' range boundaries (one
// piece per CTA, the CTA having combined its warps' pieces already): for row
// r, m = max_p m_p, l = sum_p 2^(m_p - m) l_p, O = sum_p 2^(m_p - m) O_p / l
// (base 2, O_p unnormalised).  One CTA per (sequence, kv head) with one warp
// per output row (as many warps as the batch's longest decode chunk has rows):
// lane j owns channels 4j..4j+3 and piece j's statistics.  The first four
// pieces' O rows are requested together with the statistics, the rest eight
// (then four) at a time, so a segment cut into few pieces costs one round
// trip.  The programmatic launch lets the CTAs compute their offsets as decode
// CTAs exit; they read partials only after griddepcontrol.wait.
// max_q_len: the call's bound on the chunks' lengths when it has no other kernel for
// longer ones.  It sizes the slots, these CTAs and the logits, so a chunk above
// it is an error, reported here (in the decode kernel the comparison cost 0.1 to
// 0.4 us).
constexpr int kMergeMaxThreads = 32 * kDecodeRows;
// PAGES: as in the decode kernel's stream_warps (0: every warp of the grid).
template <int D, bool MOD, int PAGES = MOD ? 1 : 0>
__global__ void __launch_bounds__(kMergeMaxThreads, 1) paged_merge_kernel(const int32_t* __restrict__ ctx_lens,
                                                                    const int32_t* __restrict__ q_lens,
                                                                    const float* part_o, const float2* part_ml,
                                                                    uint16_t* __restrict__ out, int num_seqs,
                                                                    int Hq, int Hkv, int mbps, int W, int max_q_len,
                                                                    int total_q, DevCtx ctx, ScoreMod mod) {
    // (the weight sums that may follow wait for this grid's end before they read)
    if constexpr (MOD) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int window = MOD ? mod.window : 0;
    // one warp per output row: warp w of CTA (s, hk) merges row w
    const int s = blockIdx.x, hk = blockIdx.y, r = threadIdx.x >> 5, g = Hq / Hkv;
    const int lane = threadIdx.x & 31;
    const int ql_s = __ldg(q_lens + s), cl_s = __ldg(ctx_lens + s);
    // (PAGES 2, the 8-bit cache with block scales: also the lengths of sequences without queries, as its other forms)
    if ((ql_s > max_q_len || ql_s < 0 || (PAGES == 2 && !lens_ok(ql_s, cl_s, mbps))) && hk == 0 && threadIdx.x == 0)
        raise_error(ctx, ERR_BOUNDS_BIT);
    const bool mine = is_decode_row(ql_s, g) && ql_s <= cl_s && cl_s <= mbps * kBS && r < g * ql_s;
    if (!mine) {
        // every CTA waits for the decode grid, so this grid never completes ahead of it
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const int nblk = (cl_s + kBS - 1) / kBS - first_block(cl_s, ql_s, window);
    // inputs only so far: total pages, this sequence's first page and query row
    long long tot = 0, pre = 0, q0 = 0;
    for (int i = lane; i < num_seqs; i += 32) {
        const int ql = __ldg(q_lens + i), cl = __ldg(ctx_lens + i);
        const long long n = (is_decode_row(ql, g) && ql <= cl && cl <= mbps * kBS)
                                ? (cl + kBS - 1) / kBS - first_block(cl, ql, window)
                                : 0;
        tot += n;
        if (i < s) {
            pre += n;
            q0 += max(0, ql);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        tot += __shfl_xor_sync(0xffffffffu, tot, o);
        pre += __shfl_xor_sync(0xffffffffu, pre, o);
        q0 += __shfl_xor_sync(0xffffffffu, q0, o);
    }
    const bool fits = q0 + ql_s <= total_q;
    if (!fits && hk == 0 && threadIdx.x == 0) raise_error(ctx, ERR_BOUNDS_BIT);
    const long long P = (long long)Hkv * tot;
    const long long seg_first = (long long)Hkv * pre + (long long)hk * nblk;
    if constexpr (PAGES > 0) W = stream_warps(W, P, PAGES);
    const StreamSplit split(P, W);  // W: the decode grid's warps
    const int c_lo = split.owner(seg_first) / kStreamWarps, c_hi = split.owner(seg_first + nblk - 1) / kStreamWarps;
    const int npieces = c_hi - c_lo + 1;
    // slot of piece k: 2c, or 2c+1 when the segment starts after CTA c's first
    // page; -1 when CTA c's range is empty (fewer pages than warps: it wrote nothing)
    auto slot_of = [&](int k) -> long {
        const int c = c_lo + k;
        const long long cb = split.begin(c * kStreamWarps);
        if (split.begin((c + 1) * kStreamWarps) == cb) return -1;
        return 2L * c + (seg_first <= cb ? 0 : 1);
    };
    const long lane_slot = lane < npieces ? slot_of(lane) : -1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c_lo == c_hi || !fits) return;  // the whole segment was finished inside one decode CTA

    constexpr int kPer = D / 32;  // channels per lane
    float acc[kPer];
#pragma unroll
    for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
    float lsum = 0.f, M = -INFINITY;
    // pieces in groups of 32: lane j holds piece j's (max, sum); the running
    // max of earlier groups rescales the accumulators
    for (int c0 = 0; c0 < npieces; c0 += 32) {
        const long myslot = c0 + lane < npieces ? (c0 == 0 ? lane_slot : slot_of(c0 + lane)) : -1;
        const int n = min(32, npieces - c0);
        // partials are read through L2 (ld.global.cg): the decode grid wrote them
        // while this grid was already resident, so the read-only path is not valid.
        // The first four pieces' O rows do not depend on the statistics: requested with them.
        float v0[4][kPer];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const long sj = __shfl_sync(0xffffffffu, myslot, u);
            if (u < n && sj >= 0) {
                const float* src = part_o + (sj * kDecodeRows + r) * D + lane * kPer;
                if constexpr (kPer == 4) {
                    const float4 t4 = __ldcg(reinterpret_cast<const float4*>(src));
                    v0[u][0] = t4.x; v0[u][1] = t4.y; v0[u][2] = t4.z; v0[u][3] = t4.w;
                } else {
                    const float2 t2 = __ldcg(reinterpret_cast<const float2*>(src));
                    v0[u][0] = t2.x; v0[u][1] = t2.y;
                }
            } else {
#pragma unroll
                for (int c = 0; c < kPer; ++c) v0[u][c] = 0.f;
            }
        }
        const float2 ml = myslot >= 0 ? __ldcg(part_ml + myslot * kDecodeRows + r) : make_float2(-INFINITY, 0.f);
        float gm = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
        const float Mn = fmaxf(M, gm);
        if (Mn == -INFINITY) continue;  // nothing visible yet (uniform)
        const float rescale = M == -INFINITY ? 0.f : fast_exp2(M - Mn);
#pragma unroll
        for (int c = 0; c < kPer; ++c) acc[c] *= rescale;
        lsum *= rescale;
        M = Mn;
        const float w = myslot >= 0 ? fast_exp2(ml.x - M) : 0.f;
        lsum += w * ml.y;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float wu = __shfl_sync(0xffffffffu, w, u);  // 0 past the group or for an empty range
#pragma unroll
            for (int c = 0; c < kPer; ++c) acc[c] += wu * v0[u][c];
        }
        int j = 4;
        for (; j + 8 <= n; j += 8) {  // eight pieces' loads in flight at once
            float v[8][kPer];
            float wj[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                wj[u] = __shfl_sync(0xffffffffu, w, j + u);
                const long sj = __shfl_sync(0xffffffffu, myslot, j + u);
                const float* src = part_o + ((sj < 0 ? 0 : sj) * kDecodeRows + r) * D + lane * kPer;
                if constexpr (kPer == 4) {
                    const float4 t = __ldcg(reinterpret_cast<const float4*>(src));
                    v[u][0] = t.x; v[u][1] = t.y; v[u][2] = t.z; v[u][3] = t.w;
                } else {
                    const float2 t = __ldcg(reinterpret_cast<const float2*>(src));
                    v[u][0] = t.x; v[u][1] = t.y;
                }
                if (sj < 0)  // an empty range wrote no partial: ignore whatever the slot holds
#pragma unroll
                    for (int c = 0; c < kPer; ++c) v[u][c] = 0.f;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int c = 0; c < kPer; ++c) acc[c] += wj[u] * v[u][c];
        }
        for (; j < n; j += 4) {  // the rest, four pieces' loads in flight at once
            float v[4][kPer];
            float wj[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = j + u;
                wj[u] = __shfl_sync(0xffffffffu, w, k & 31);
                const long sj = __shfl_sync(0xffffffffu, myslot, k & 31);
                if (k < n && sj >= 0) {
                    const float* src = part_o + (sj * kDecodeRows + r) * D + lane * kPer;
                    if constexpr (kPer == 4) {
                        const float4 t4 = __ldcg(reinterpret_cast<const float4*>(src));
                        v[u][0] = t4.x; v[u][1] = t4.y; v[u][2] = t4.z; v[u][3] = t4.w;
                    } else {
                        const float2 t2 = __ldcg(reinterpret_cast<const float2*>(src));
                        v[u][0] = t2.x; v[u][1] = t2.y;
                    }
                } else {
                    wj[u] = 0.f;
#pragma unroll
                    for (int c = 0; c < kPer; ++c) v[u][c] = 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int c = 0; c < kPer; ++c) acc[c] += wj[u] * v[u][c];
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, o);
    const float inv = lsum > 0.f ? 1.f / lsum : 0.f;
    if constexpr (MOD != 0)
        if (mod.lse && lane == 0)
            mod.lse[(long)(q0 + r / g) * Hq + hk * g + r % g] = lsum > 0.f ? (M + __log2f(lsum)) * kLn2f : -INFINITY;
    uint16_t* dst = out + ((long)(q0 + r / g) * Hq + hk * g + r % g) * D + lane * kPer;
    if constexpr (kPer == 4)
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
    else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
}

// --------------------------------------------------------- weight sums -----
// acc_out[s][hk][t] = decay acc_in[s][hk][t] (0 for the chunk's own tokens, and
// without acc_in) + sum over the sequence's query rows r of the group of
// 2^(x_rt - lse_r), from the logits x that the decode kernel kept and the
// final log-sum-exp: sequences that took the decode kernel, and those without
// queries.  Memory bound: rows * 4 bytes a key read, 8 bytes of sums.  The sum
// over rows runs in a fixed order.  CTA (s, hk, split): every gridDim.z-th group
// of kAccumPages pages of the context, a half-warp per page.  The
// programmatic launch lets the CTAs find their places while the attention's
// last kernel runs.
constexpr int kAccumPages = 16;  // pages per CTA
__global__ void __launch_bounds__(256) accum_decode_kernel(const int32_t* __restrict__ ctx_lens,
                                                           const int32_t* __restrict__ q_lens,
                                                           const float* lse, const float* logits, int logit_rows,
                                                           const float* acc_in, float* acc_out, int acc_len,
                                                           float decay, int num_seqs, int mbps, int Hq, int Hkv,
                                                           int window, int total_q, DevCtx ctx) {
    const int s = blockIdx.x, hk = blockIdx.y, g = Hq / Hkv, lane = threadIdx.x & 31;
    const int ql = __ldg(q_lens + s), cl = __ldg(ctx_lens + s);
    int p0 = blockIdx.z * kAccumPages;
    const int npages = (cl + kBS - 1) / kBS;
    const bool mine = ql <= cl && ql >= 0 && cl <= mbps * kBS && (ql == 0 || is_decode_row(ql, g)) && p0 < npages;
    if (!mine || cl > acc_len) {
        if (mine && threadIdx.x == 0) raise_error(ctx, ERR_BOUNDS_BIT);
        // every CTA waits for the grid before, so this one never completes ahead of it
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    __shared__ float neg_lse2[kDecodeRows];
    long long pre = 0, q0 = 0;  // pages and query rows of the sequences before s (every warp)
    if (ql > 0) {
        for (int i = lane; i < s; i += 32) {
            const int qi = __ldg(q_lens + i), ci = __ldg(ctx_lens + i);
            if (is_decode_row(qi, g) && qi <= ci && ci <= mbps * kBS)
                pre += (ci + kBS - 1) / kBS - first_block(ci, qi, window);
            q0 += max(0, qi);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            pre += __shfl_xor_sync(0xffffffffu, pre, o);
            q0 += __shfl_xor_sync(0xffffffffu, q0, o);
        }
    }
    if (q0 + ql > total_q) {  // (the same for the whole CTA; reported by the merge kernel)
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const int nrows = ql > 0 ? min(g * ql, logit_rows) : 0;
    const int blk0 = ql > 0 ? first_block(cl, ql, window) : 0;
    const long long seg = pre * Hkv + (long long)hk * (npages - blk0);  // the segment's first page of the stream
    const long row = ((long)s * Hkv + hk) * acc_len;
    const int i = threadIdx.x & 15;
    float x[kDecodeRows];  // this token's logits: all loads in flight with the statistics'
    float a = 0.f;
    auto load_sum = [&]() {
        const int t = (p0 + (threadIdx.x >> 4)) * kBS + i;
        a = t < cl && acc_in && t < cl - ql ? decay * acc_in[row + t] : 0.f;
    };
    auto load_logits = [&]() {
        const int p = p0 + (threadIdx.x >> 4), t = p * kBS + i;
        if (t >= cl || p < blk0) return;
        const float* src = logits + (seg + p - blk0) * logit_rows * kBS + i;
#pragma unroll
        for (int r = 0; r < kDecodeRows; ++r) x[r] = r < nrows ? __ldcg(src + r * kBS) : -INFINITY;
    };
    // inputs only so far, the old sums among them: the call's first kernel began
    // behind everything that could have written them
    load_sum();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    load_logits();
    if (threadIdx.x < nrows) {
        const int r = threadIdx.x;
        const float L = __ldcg(lse + (q0 + r / g) * Hq + hk * g + r % g);
        neg_lse2[r] = L == -INFINITY ? 0.f : -L * kLog2ef;
    }
    __syncthreads();
    while (true) {
        const int p = p0 + (threadIdx.x >> 4), t = p * kBS + i;
        if (t < cl) {
            float w = 0.f;
            if (p >= blk0) {
#pragma unroll
                for (int r = 0; r < kDecodeRows; ++r)
                    if (r < nrows) w += fast_exp2(x[r] + neg_lse2[r]);
            }
            acc_out[row + t] = a + w;
        }
        p0 += gridDim.z * kAccumPages;
        if (p0 >= npages) return;
        load_sum();
        load_logits();
    }
}

// ------------------------------------------------------------ metadata -----
// Two CTAs side by side, since every chunked call waits for them.  The second:
// q_start (exclusive prefix sum of q_lens), and the weight sums' units.  The
// first: the list of work entries (entry_tokens consecutive query tokens,
// paged_tc_entry_tokens) of the sequences that take the tensor-core kernel,
// ordered by decreasing number of KV tiles (longest first) with a counting sort.
// Entry = (sequence, first query token of the entry within the chunk).
//
// Calls with modified scores get `pieces` instead: an entry whose KV tiles are
// many for the work there is (few chunks over long contexts) is cut along its
// keys, so that the call still fills the GPU; its pieces leave partial results
// that paged_join_kernel puts together.  With `share` the tiles of all units for
// each SM, a piece has at least four tiles (a unit's fixed cost is that of
// three), the share up to six of them (a GPU that is nearly full gains nothing
// from pieces of four: 4 chunks of 300 over 1000 keys 44 us, whole 33), and half
// the share beyond.  Measured, 32 heads in 8 groups, d = 128: a chunk of 128
// over 4000 keys 88 us whole, 32 in pieces; one of 512 over 30000 376 and 140;
// 16 chunks of 64 over up to 8000 (12 heads in 2 groups) 107 and 74.
constexpr int kSplitTiles = 4, kSplitShare = 6;
constexpr int kSplitMost = 32;  // pieces of an entry (a warp lists them, the join takes 0.3 us for each)
constexpr int kSplitSlots = 2 * kMaxStreamCtas;  // total / least, at most
// (Cutting is a variant of its own: its divisions and counters in the kernel that
// every chunked call waits for cost 5 us of 225.)
enum { META_LIST = 0, META_PIECES = 1, META_CUT = 2 };
template <int KIND>
__global__ void __launch_bounds__(1024) paged_meta_kernel(const int32_t* __restrict__ ctx_lens,
                                                          const int32_t* __restrict__ q_lens, int num_seqs, int mbps,
                                                          int g, int causal, int entry_tokens,
                                                          int32_t* __restrict__ q_start, int32_t* __restrict__ count,
                                                          int32_t* __restrict__ list, int max_entries,
                                                          int window, const int32_t* __restrict__ prefix,
                                                          int32_t* __restrict__ k_start, int acc_len,
                                                          int4* __restrict__ pieces, int4* __restrict__ split,
                                                          int max_slots, int per_rank, int total_q, int all_lens, DevCtx ctx) {
    extern __shared__ int hist[];  // [nbins + 1]
    __shared__ int warp_sums[32];
    __shared__ long long row_sums[32], rows_before;
    __shared__ int carry, n_slots, n_split;
    __shared__ unsigned long long all_tiles;
    const int nbins = (mbps * kBS + 127) / 128 + 1;
    // This thread's sequences are mine, mine + 1024, ...; the lengths of the first stay in registers, every
    // step below asks for them.  (Neighbours go to different warps when a warp works on one entry at a time.)
    const int mine = KIND == META_CUT ? (threadIdx.x & 31) * 32 + (threadIdx.x >> 5) : threadIdx.x;
    const int ql0 = mine < num_seqs ? __ldg(q_lens + mine) : 0, cl0 = mine < num_seqs ? __ldg(ctx_lens + mine) : 0;
    auto q_len = [&](int s) { return s == mine ? ql0 : __ldg(q_lens + s); };
    auto ctx_len = [&](int s) { return s == mine ? cl0 : __ldg(ctx_lens + s); };
    for (int i = threadIdx.x; i <= nbins; i += blockDim.x) hist[i] = 0;
    if (threadIdx.x == 0) {
        carry = n_slots = n_split = 0;
        rows_before = 0;
        all_tiles = 0;
    }
    __syncthreads();
    if (blockIdx.x == 1) {
        // prefix sum of q_lens, 1024 sequences per pass
        for (int base = 0; base < num_seqs; base += blockDim.x) {
            const int s = base + threadIdx.x;
            const int v = s < num_seqs ? max(0, q_len(s)) : 0;
            long long x = v;
            const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) row_sums[w] = x;
            __syncthreads();
            if (w == 0) {
                long long t = row_sums[lane];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, t, o);
                    if (lane >= o) t += y;
                }
                row_sums[lane] = t;
            }
            __syncthreads();
            const long long excl = rows_before + (w ? row_sums[w - 1] : 0) + x - v;
            if (s < num_seqs) q_start[s] = (int)min(excl, 0x7fffffffll);
            if (v > 0 && excl + v > total_q) raise_error(ctx, ERR_BOUNDS_BIT);
            __syncthreads();
            if (threadIdx.x == blockDim.x - 1) rows_before = excl + v;
            __syncthreads();
        }
        // weight sums: sequences by decreasing chunk length (a counting sort over 64
        // lengths; the order only decides who goes first), then their units of 256
        // keys in that order (none for a sequence whose sums do not fit, which is
        // reported, and for those without a chunk)
        if (KIND != META_LIST && k_start) {
            __shared__ int order[64];
            int32_t* k_seq = k_start + num_seqs + 1;
            auto rank_bin = [&](int s) { return 63 - min(63, max(0, q_len(s)) / 32); };
            __syncthreads();
            if (threadIdx.x < 64) order[threadIdx.x] = 0;
            if (threadIdx.x == 0) carry = 0;
            __syncthreads();
            for (int s = threadIdx.x; s < num_seqs; s += blockDim.x) atomicAdd(&order[rank_bin(s)], 1);
            __syncthreads();
            if (threadIdx.x == 0) {
                int run = 0;
                for (int b = 0; b < 64; ++b) {
                    const int c = order[b];
                    order[b] = run;
                    run += c;
                }
            }
            __syncthreads();
            for (int s = threadIdx.x; s < num_seqs; s += blockDim.x) k_seq[atomicAdd(&order[rank_bin(s)], 1)] = s;
            __syncthreads();
            for (int base = 0; base < num_seqs; base += blockDim.x) {
                const int r = base + threadIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
                const int s = r < num_seqs ? k_seq[r] : 0;
                const int ql = r < num_seqs ? q_lens[s] : 0, cl = r < num_seqs ? ctx_lens[s] : 0;
                const bool chunk = ql > 0 && !is_decode_row(ql, g) && ql <= cl && cl <= mbps * kBS &&
                                   rows_fit(q_start[s], ql, total_q);
                if (chunk && cl > acc_len) raise_error(ctx, ERR_BOUNDS_BIT);
                const int v = chunk && cl <= acc_len ? (cl + 255) / 256 : 0;
                int x = v;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, x, o);
                    if (lane >= o) x += y;
                }
                if (lane == 31) warp_sums[w] = x;
                __syncthreads();
                const int t = warp_sums[lane];
                const int before = carry + __reduce_add_sync(0xffffffffu, lane < w ? t : 0) + x - v;
                if (r < num_seqs) k_start[r] = before;
                __syncthreads();
                if (threadIdx.x == blockDim.x - 1) carry = before + v;
                __syncthreads();
            }
            if (threadIdx.x == 0) k_start[num_seqs] = carry;
        }
        return;
    }
    // an entry's KV tiles [x, y): from the first key its first row sees to the last its last row sees
    auto entry_tiles = [&](int s, int ql, int cl, int t0) {
        const int first = cl - ql + t0, last = cl - ql + min(ql, t0 + entry_tokens) - 1;  // positions
        int hi = causal ? last + 1 : (window > 0 ? last + window : cl);
        if (causal && prefix) hi = max(hi, prefix[s]);
        const int lo = window > 0 ? max(0, first - window + 1) : 0;
        return make_int2(lo / 128, (min(hi, cl) + 127) / 128);
    };
    auto is_chunk = [&](int ql, int cl) { return ql > 0 && !is_decode_row(ql, g) && ql <= cl && cl <= mbps * kBS; };
    [[maybe_unused]] int least = 1;  // tiles of a piece, at least
    if constexpr (KIND == META_CUT) {
        unsigned long long tiles = 0;
        for (int s = mine; s < num_seqs; s += blockDim.x) {
            const int ql = q_len(s), cl = ctx_len(s);
            if (!is_chunk(ql, cl)) continue;
            for (int t0 = 0; t0 < ql; t0 += entry_tokens) {
                const int2 t = entry_tiles(s, ql, cl, t0);
                tiles += t.y - t.x;
            }
        }
        if (tiles) atomicAdd(&all_tiles, tiles);
        __syncthreads();
        const unsigned long long total = all_tiles * per_rank, share = (total + kMaxStreamCtas - 1) / kMaxStreamCtas;
        unsigned long long t = max((unsigned long long)kSplitTiles, max(min(share, (unsigned long long)kSplitShare), (share + 1) / 2));
        t = max(t, (total + max_slots - 1) / max_slots);  // their partial results fit
        least = (int)min(t, 1ull << 30);
    }
    auto cuts = [&](int tiles) { return KIND == META_CUT && tiles >= 2 * least ? min(kSplitMost, tiles / least) : 1; };
    auto cut = [](int i, int n, int tiles) {  // end of piece i
        return i + 1 == n ? tiles : (KIND == META_CUT ? (i + 1) * tiles / n : 0);
    };
    // f(sequence, its lengths, first token, piece) for every entry: a thread per sequence, or, when entries
    // are cut, a warp for 32 sequences whose lanes are the pieces of one entry after another
    auto for_entries = [&](auto f) {
        const int lane = threadIdx.x & 31;
        for (int s = mine; s < num_seqs + (KIND == META_CUT ? lane * 32 : 0); s += blockDim.x) {
            const int ql = s < num_seqs ? q_len(s) : 0, cl = s < num_seqs ? ctx_len(s) : 0;
            if constexpr (KIND == META_CUT) {
                for (unsigned m = __ballot_sync(0xffffffffu, is_chunk(ql, cl)); m; m &= m - 1) {
                    const int b = __ffs(m) - 1, ql_b = __shfl_sync(0xffffffffu, ql, b), cl_b = __shfl_sync(0xffffffffu, cl, b);
                    for (int t0 = 0; t0 < ql_b; t0 += entry_tokens) f(s + (b - lane) * 32, ql_b, cl_b, t0, lane);
                }
            } else if (is_chunk(ql, cl)) {
                for (int t0 = 0; t0 < ql; t0 += entry_tokens) f(s, ql, cl, t0, 0);
            }
        }
    };
    for (int s = mine; s < num_seqs; s += blockDim.x) {
        const int ql = q_len(s), cl = ctx_len(s);
        if (ql < 0 || (ql > 0 && !is_decode_row(ql, g) && !is_chunk(ql, cl)) || (all_lens && !lens_ok(ql, cl, mbps)))
            raise_error(ctx, ERR_BOUNDS_BIT);
    }
    // histogram of the costs
    for_entries([&](int s, int ql, int cl, int t0, int i) {
        const int2 t = entry_tiles(s, ql, cl, t0);
        const int tiles = t.y - t.x, n = cuts(tiles);
        if (i < n) atomicAdd(&hist[cut(i, n, tiles) - cut(i - 1, n, tiles)], 1);
    });
    __syncthreads();
    if (threadIdx.x < 32) {  // bucket starts, highest cost first (a warp: a wide table has thousands of buckets)
        const int lane = threadIdx.x;
        int run = 0;
        for (int b0 = nbins - 1; b0 >= 0; b0 -= 32) {
            const int b = b0 - lane, c = b >= 0 ? hist[b] : 0;
            int x = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (b >= 0) hist[b] = run + x - c;
            run += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) {
            *count = run < max_entries ? run : max_entries;
            count[1] = 0;  // the tensor-core kernel's unit tickets
            count[2] = 0;  // and the weight sums'
        }
    }
    __syncthreads();
    for_entries([&](int s, int ql, int cl, int t0, int i) {
        const int2 t = entry_tiles(s, ql, cl, t0);
        const int tiles = t.y - t.x, n = cuts(tiles);
        [[maybe_unused]] int slot = -1;
        if (KIND == META_CUT && n > 1) {
            if (i == 0) {
                slot = atomicAdd(&n_slots, n * per_rank);
                split[atomicAdd(&n_split, 1)] = make_int4(s, t0, slot, n);
            }
            slot = __shfl_sync(0xffffffffu, slot, 0) + i * per_rank;
        }
        if (i >= n) return;
        const int a = cut(i - 1, n, tiles), b = cut(i, n, tiles), pos = atomicAdd(&hist[b - a], 1);
        if (pos >= max_entries) return;
        if constexpr (KIND != META_LIST) {
            pieces[pos] = make_int4(s, t0, (t.x + a) | (t.x + b) << 16, slot);
        } else {
            list[2 * pos] = s;
            list[2 * pos + 1] = t0;
        }
    });
    if constexpr (KIND == META_CUT) {
        __syncthreads();
        if (threadIdx.x == 0) count[3] = n_split;
    }
}

// Rows of the entries that were cut along their keys: the pieces' partial
// results weighed by their sums 2^(m_i - M) l_i and added in order, and the
// log-sum-exp.  A warp takes 16 channels of 32 rows, a row a lane; what it reads
// is mostly in the L2 that it was just written to.
template <int D>
__global__ void __launch_bounds__(256) paged_join_kernel(const int4* split, const int32_t* count, const float4* part_o,
                                                         const float2* part_ml, const int32_t* __restrict__ q_lens,
                                                         const int32_t* __restrict__ q_start, uint16_t* __restrict__ out,
                                                         float* __restrict__ lse, int per_rank, int Hq, int g, int total_q) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kSlices = D / 16;
    const int lane = threadIdx.x & 31;
    const long items = (long)__ldcg(count + 3) * per_rank * 8 * kSlices;
    const bool pack = paged_tc_pack(g);
    for (long idx = (long)blockIdx.x * 8 + (threadIdx.x >> 5); idx < items; idx += (long)gridDim.x * 8) {
        const int slice = (int)(idx % kSlices), row = (int)(idx / kSlices % 8) * 32 + lane;
        const int unit = (int)(idx / (8 * kSlices)), rest = unit % per_rank;
        const int4 e = __ldcg(split + unit / per_rank);
        const int ql = __ldg(q_lens + e.x), qs = __ldg(q_start + e.x);
        const float2* ml = part_ml + (long)(e.z + rest) * 256 + row;
        const float4* src = part_o + ((long)(e.z + rest) * (D / 4) + slice * 4) * 256 + row;
        float M = -INFINITY, sum = 0.f;
#pragma unroll 8
        for (int i = 0; i < e.w; ++i) {
            const float2 x = __ldcg(ml + (long)i * per_rank * 256);
            if (x.y > 0.f) M = fmaxf(M, x.x);
        }
        float acc[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) acc[c] = 0.f;
#pragma unroll 4
        for (int i = 0; i < e.w; ++i) {
            const float2 x = __ldcg(ml + (long)i * per_rank * 256);
            float4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __ldcg(src + ((long)i * per_rank * (D / 4) + j) * 256);
            const float f = x.y > 0.f ? x.y * fast_exp2(x.x - M) : 0.f;  // (a piece without a visible key has no share)
            sum += f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[4 * j] = f > 0.f ? fmaf(f, v[j].x, acc[4 * j]) : acc[4 * j];
                acc[4 * j + 1] = f > 0.f ? fmaf(f, v[j].y, acc[4 * j + 1]) : acc[4 * j + 1];
                acc[4 * j + 2] = f > 0.f ? fmaf(f, v[j].z, acc[4 * j + 2]) : acc[4 * j + 2];
                acc[4 * j + 3] = f > 0.f ? fmaf(f, v[j].w, acc[4 * j + 3]) : acc[4 * j + 3];
            }
        }
        // as the attention lays a unit's two slots out
        int tok, head;
        if (pack) {
            tok = e.y + row / g;
            head = rest * g + row % g;
        } else if (g % 2 == 0) {
            tok = e.y + (row & 127);
            head = rest / (g / 2) * g + 2 * (rest % (g / 2)) + (row >> 7);
        } else {
            tok = e.y + row;
            head = rest;
        }
        if (tok >= ql || !rows_fit(qs, ql, total_q)) continue;
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const long at = ((long)qs + tok) * Hq + head;
        if (lse && slice == 0) lse[at] = sum > 0.f ? (M + __log2f(sum)) * kLn2f : -INFINITY;
        uint4* dst = reinterpret_cast<uint4*>(out + at * D + slice * 16);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            dst[j] = make_uint4(pack_bf16x2(acc[8 * j] * inv, acc[8 * j + 1] * inv),
                                pack_bf16x2(acc[8 * j + 2] * inv, acc[8 * j + 3] * inv),
                                pack_bf16x2(acc[8 * j + 4] * inv, acc[8 * j + 5] * inv),
                                pack_bf16x2(acc[8 * j + 6] * inv, acc[8 * j + 7] * inv));
    }
}

// A library-owned side stream per device: the chunked-prefill metadata pass (two
// CTAs) runs there beside the split-KV decode kernel and its merge, which do
// not depend on it; two events fork it from and join it back to the caller's
// stream (both capturable, so the call may be recorded into a CUDA graph).
constexpr int kMaxSideDevices = 64;
struct SideStream {
    std::mutex mu;
    cudaStream_t s = nullptr;
    cudaEvent_t fork = nullptr, join = nullptr;
};
SideStream g_side[kMaxSideDevices];

static fa_status side_stream(SideStream** out) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxSideDevices) return FA_ERR_CUDA;
    SideStream& ss = g_side[dev];
    if (!ss.s && cudaStreamCreateWithFlags(&ss.s, cudaStreamNonBlocking) != cudaSuccess) return FA_ERR_CUDA;
    if (!ss.fork && cudaEventCreateWithFlags(&ss.fork, cudaEventDisableTiming) != cudaSuccess) return FA_ERR_CUDA;
    if (!ss.join && cudaEventCreateWithFlags(&ss.join, cudaEventDisableTiming) != cudaSuccess) return FA_ERR_CUDA;
    *out = &ss;
    return FA_OK;
}

template <int D, int KV = KV_BF16, int MOD = 0>
static fa_status launch_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* bt,
                               const int32_t* ctx_lens, const int32_t* q_lens, void* out, const PagedWs& w,
                               uint8_t* ws, int num_seqs, int mbps, int num_blocks, int Hq, int Hkv,
                               int max_q_len, int total_q, int q_prefetch_rows, int causal, float scale, int merge_rows,
                               cudaStream_t s, const DevCtx& ctx, int* launches,
                               float k_scale = 1.f, float v_scale = 1.f, const ScoreMod& mod = ScoreMod{},
                               const uint8_t* k_exp = nullptr, const uint8_t* v_exp = nullptr) {
    CUtensorMap tk, tv;
    fa_status st;
    if constexpr (KV == KV_FP8_SCALED) {
        v_scale = PageMma<D, true>::kDown;
        st = page_maps<D, true>(k_cache, v_cache, num_blocks, Hkv, &tk, &tv);
        if (st != FA_OK) return st;
    } else if constexpr (KV == KV_FP8) {
        // K [blocks][Hkv][16][D] bytes, rows of D bytes, 128-byte swizzle;
        // V [blocks][Hkv][D][16] bytes, one 16-byte row per channel
        const uint64_t kd[4] = {(uint64_t)D, (uint64_t)kBS, (uint64_t)Hkv, (uint64_t)num_blocks};
        const uint64_t vd[4] = {(uint64_t)kBS, (uint64_t)D, (uint64_t)Hkv, (uint64_t)num_blocks};
        const uint64_t ks[3] = {(uint64_t)D, (uint64_t)kBS * D, (uint64_t)Hkv * kBS * D};
        const uint64_t vs[3] = {(uint64_t)kBS, (uint64_t)kBS * D, (uint64_t)Hkv * kBS * D};
        const uint32_t kb[4] = {(uint32_t)D, (uint32_t)kBS, 1, 1};
        const uint32_t vb[4] = {(uint32_t)kBS, (uint32_t)D, 1, 1};
        st = encode_tmap_4d(&tk, k_cache, kd, ks, kb, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != FA_OK) return st;
        st = encode_tmap_4d(&tv, v_cache, vd, vs, vb, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_NONE);
        if (st != FA_OK) return st;
    } else {
        const uint64_t dims[4] = {(uint64_t)D, (uint64_t)kBS, (uint64_t)Hkv, (uint64_t)num_blocks};
        const uint64_t strides[3] = {(uint64_t)D * 2, (uint64_t)kBS * D * 2, (uint64_t)Hkv * kBS * D * 2};
        const uint32_t box[4] = {64, (uint32_t)kBS, 1, 1};
        st = encode_tmap_bf16_4d(&tk, k_cache, dims, strides, box);
        if (st != FA_OK) return st;
        if ((st = encode_tmap_bf16_4d(&tv, v_cache, dims, strides, box)) != FA_OK) return st;
    }
    float* part_o = reinterpret_cast<float*>(ws + w.part_o);
    float2* part_ml = reinterpret_cast<float2*>(ws + w.part_ml);
    const float scale_log2 = scale * k_scale * 1.4426950408889634f;
    const int grid = std::min(sm_count(), kMaxStreamCtas);
    // partial slots of 6 rows when no decode chunk has more (then the ring keeps
    // three stages at d = 128), else of 16
    auto launch = [&](auto rows) -> fa_status {
        constexpr int R = decltype(rows)::value;
        using L = StreamSmem<D, KV, R>;
        const fa_status st2 = raise_dynamic_smem(reinterpret_cast<const void*>(paged_decode_kernel<D, KV, R, MOD>), L::kBytes);
        if (st2 != FA_OK) return st2;
        paged_decode_kernel<D, KV, R, MOD><<<grid, kStreamWarps * 32, L::kBytes, s>>>(
            tk, tv, static_cast<const uint16_t*>(q), bt, ctx_lens, q_lens, static_cast<uint16_t*>(out), part_o, part_ml,
            num_seqs, mbps, num_blocks, Hq, Hkv, q_prefetch_rows, causal, scale_log2, v_scale, total_q, ctx,
            mod, k_exp, v_exp);
        return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
    };
    st = merge_rows <= 6 ? launch(std::integral_constant<int, 6>{}) : launch(std::integral_constant<int, kDecodeRows>{});
    if (st != FA_OK) return st;
    ++*launches;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_seqs, Hkv, 1);
    cfg.blockDim = dim3(32 * merge_rows);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    constexpr bool kScaled = KV == KV_FP8_SCALED;
    if (cudaLaunchKernelEx(&cfg, paged_merge_kernel<D, (MOD != 0 || kScaled), kScaled ? 2 : (MOD != 0 ? 1 : 0)>, ctx_lens, q_lens,
                           static_cast<const float*>(part_o), static_cast<const float2*>(part_ml),
                           static_cast<uint16_t*>(out), num_seqs, Hq, Hkv, mbps, grid * kStreamWarps, max_q_len, total_q, ctx, mod) !=
        cudaSuccess)
        return FA_ERR_CUDA;
    ++*launches;
    return FA_OK;
}

// Behind the attention's own workspace, calls with modified scores keep their
// pieces and the partial results of those that do not have all of their keys:
// as many as the tables' tiles and the queries could ask for, at most kSplitSlots.
struct PiecesWs {
    int slots, per_rank, max_pieces;
    size_t list, split, ml, o, total;
};
// `smaller`: room for every problem of no larger sizes too (those of few queries
// need more than this one may), which is what the size queries give.
static PiecesWs pieces_ws_layout(const PagedWs& w, int num_seqs, int mbps, int Hq, int Hkv, int d, int total_q,
                                 int max_q_len, bool smaller) {
    PiecesWs x{};
    const int g = Hq / Hkv;
    x.per_rank = paged_tc_pack(g) ? Hkv : (g % 2 == 0 ? Hkv * (g / 2) : Hq);
    const long tiles = ((long)mbps * kBS + 127) / 128, entries = total_q / paged_tc_entry_tokens(g) + (long)num_seqs;
    // (an entry is cut into tiles / kSplitTiles pieces at most, and only when that is two or more)
    // (none for queries that make a unit for every SM anyway: the join's launch would cost 3 us)
    const bool few = max_q_len > 0 && !is_decode_row(max_q_len, g) &&
                     (smaller || total_q / paged_tc_entry_tokens(g) * (long)x.per_rank < kMaxStreamCtas);
    // (rounded up, so that the places never limit the cuts below kSplitSlots: the shares go by the lengths alone)
    const long cuts = !few || tiles / kSplitTiles < 2 ? 0 : std::min<long>((tiles + kSplitTiles - 1) / kSplitTiles, kSplitSlots);
    x.slots = (int)std::min<long>(kSplitSlots, std::min<long>(entries, kSplitSlots) * x.per_rank * cuts);
    x.max_pieces = w.max_entries + x.slots;
    x.list = align256(w.total);
    x.split = align256(x.list + sizeof(int4) * (size_t)x.max_pieces);
    x.ml = align256(x.split + sizeof(int4) * (size_t)(x.slots / 2 + 1));
    x.o = align256(x.ml + sizeof(float2) * 256 * (size_t)x.slots);
    x.total = align256(x.o + sizeof(float) * 256 * (size_t)x.slots * d);
    return x;
}

// Weight sums wanted by a call (fa_paged_attn_accum), and where its workspace
// keeps, behind the attention's own, the first unit of every chunk and the
// decode rows' logits: min(16, g * max_q_len) rows of 16 for every page that the
// tables can hold.
struct AccumArgs {
    const float* in;
    float* out;
    int len;
    float decay;
};
struct AccumWs {
    size_t k_start, logits, total;
};
static AccumWs accum_ws_layout(size_t base, int num_seqs, int mbps, int Hq, int Hkv, int max_q_len) {
    const int g = Hq / Hkv;
    const long rows = g <= kDecodeRows ? std::min<long>(kDecodeRows, (long)g * max_q_len) : 0;
    AccumWs a{};
    a.k_start = align256(base);
    a.logits = align256(a.k_start + sizeof(int32_t) * (2 * (size_t)num_seqs + 1));
    a.total = align256(a.logits + (size_t)num_seqs * mbps * Hkv * rows * kBS * sizeof(float));
    return a;
}

// The scale codes of a cache in 8 bits (such a call comes with a `mod` that modifies nothing).
struct ScaledKv {
    const uint8_t *k_exp, *v_exp;
};

// Does a call over the 8-bit cache take a CTA or a cluster for each (sequence, kv head), in one launch
// (blocks_attn.cu), instead of the stream and its merge?  Only single tokens, by the longest context that the tables
// can hold.  Measured at d = 128 (lists and stream, us; tables as long as the longest context; all sequences that long,
// a quarter of it and more, one that long and the others an eighth of it at most):
//   8 pairs, 4000 tokens     12.3 14.9   12.3 15.3   12.3 14.5
//   128 pairs, 2000          20.5 23.0   20.5 22.5   16.4 16.4;  4000  34.6 38.9   30.7 30.7   26.6 18.4
//   512 pairs, 1000          31.1 41.0   24.6 28.8   20.5 16.4;  2000  50.0 62.8   46.5 47.2   32.8 20.5
//   2400 pairs, 2000          201 239     151 168    61.7 51.2;  4000   380 445     290 300     108 72
// The lists win by a fifth at most while contexts are about as long, and lose when one long context lies among short
// ones: by a fifth over 1000 and 2000 tokens (20.5 16.4, 61.7 51.2), by half over 4000 (108 72).  The lengths are on the
// device, so the rule goes by the longest context there can be, and takes the lists while that is short.
static bool whole_lists(int num_seqs, int mbps, int Hkv, int g, int max_q_len) {
    if (max_q_len != 1) return false;
    const long lists = (long)num_seqs * Hkv * ((g + 15) / 16), warps = (long)kListSmWarps * sm_count();
    if (mbps <= 64) return true;
    if (mbps <= 128) return lists * 8 <= warps || lists >= warps;
    return mbps <= 256 && (lists * 32 <= warps || lists >= warps);
}

static fa_status paged_attn_run(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                        const int32_t* ctx_lens, const int32_t* q_lens, void* out, int num_seqs,
                        int max_blocks_per_seq, int num_blocks, int Hq, int Hkv, int d, int block_size, int causal,
                        float scale, int total_q, int max_q_len, void* ws, size_t ws_bytes, fa_stream_t stream,
                                ScoreMod* mod, const AccumArgs* acc, const ScaledKv* kv8 = nullptr) {
    set_launch_count(0);
    if (num_seqs < 0 || max_blocks_per_seq < 0 || num_blocks < 0 || Hq <= 0 || Hkv <= 0 || total_q < 0 ||
        max_q_len < 0 || !(scale > 0.f) || !(scale < INFINITY))
        return FA_ERR_INVALID_ARG;
    if (block_size != kBS || (d != 64 && d != 128) || Hq % Hkv != 0) return FA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0 || max_q_len == 0) return FA_OK;
    if (!q || !k_cache || !v_cache || !block_table || !ctx_lens || !q_lens || !out) return FA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned32(out)) return FA_ERR_INVALID_ARG;
    if (num_blocks == 0 || max_blocks_per_seq == 0) return FA_ERR_INVALID_ARG;
    const PagedWs w = paged_ws_layout(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q);
    const PiecesWs pw =
        mod ? pieces_ws_layout(w, num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q, max_q_len, false) : PiecesWs{};
    const AccumWs aw = acc ? accum_ws_layout(pw.total, num_seqs, max_blocks_per_seq, Hq, Hkv, max_q_len) : AccumWs{};
    if (!ws || ws_bytes < (acc ? aw.total : mod ? pw.total : w.total) || (reinterpret_cast<uintptr_t>(ws) & 255)) return FA_ERR_WORKSPACE;
    fa_status st = check_device();
    if (st != FA_OK) return st;
    DevCtx ctx;
    if ((st = make_ctx(&ctx)) != FA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* wsb = static_cast<uint8_t*>(ws);
    const int g = Hq / Hkv;
    if (kv8 && whole_lists(num_seqs, max_blocks_per_seq, Hkv, g, max_q_len)) {
        st = launch_whole_lists(q, k_cache, v_cache, kv8->k_exp, kv8->v_exp, block_table, ctx_lens, q_lens, out, mod->lse, num_seqs,
                                max_blocks_per_seq, num_blocks, Hq, Hkv, d, scale, total_q, max_q_len, s, ctx);
        if (st == FA_OK) set_launch_count(1);
        return st;
    }
    int launches = 0;
    const bool decode_path = g <= kDecodeRows;  // some sequences may be decode rows
    const bool tc_path = !is_decode_row(max_q_len, g);
    // the tensor-core path's work list: on the side stream when the decode
    // kernel also runs (they are independent), else in line
    SideStream* ss = nullptr;
    std::unique_lock<std::mutex> side_lock;
    if (tc_path) {
        const int entry_tokens = paged_tc_entry_tokens(g);
        int32_t* q_start = reinterpret_cast<int32_t*>(wsb + w.q_start);
        int32_t* count = reinterpret_cast<int32_t*>(wsb + w.work_count);
        int32_t* list = reinterpret_cast<int32_t*>(wsb + w.work_list);
        const int nbins = (max_blocks_per_seq * kBS + 127) / 128 + 1;
        const size_t hist_bytes = sizeof(int) * (size_t)(nbins + 1);
        if (hist_bytes > 200 * 1024) return FA_ERR_UNSUPPORTED;
        auto meta = pw.slots > 0 ? paged_meta_kernel<META_CUT>
                                 : (mod ? paged_meta_kernel<META_PIECES> : paged_meta_kernel<META_LIST>);
        if (hist_bytes > kUnraisedSmem &&
            (st = raise_dynamic_smem(reinterpret_cast<const void*>(meta), (int)hist_bytes)) != FA_OK)
            return st;
        cudaStream_t ms = s;
        if (decode_path) {
            if ((st = side_stream(&ss)) != FA_OK) return st;
            side_lock = std::unique_lock<std::mutex>(ss->mu);
            if (cudaEventRecord(ss->fork, s) != cudaSuccess || cudaStreamWaitEvent(ss->s, ss->fork, 0) != cudaSuccess)
                return FA_ERR_CUDA;
            ms = ss->s;
        }
        meta<<<2, 1024, hist_bytes, ms>>>(ctx_lens, q_lens, num_seqs, max_blocks_per_seq, g, causal,
                                                       entry_tokens, q_start, count, list,
                                                       mod ? pw.max_pieces : w.max_entries,
                                                       mod ? mod->window : 0, mod ? mod->prefix : nullptr,
                                                       acc ? reinterpret_cast<int32_t*>(wsb + aw.k_start) : nullptr,
                                                       acc ? acc->len : 0,
                                                       mod ? reinterpret_cast<int4*>(wsb + pw.list) : nullptr,
                                                       mod ? reinterpret_cast<int4*>(wsb + pw.split) : nullptr,
                                                       pw.slots, pw.per_rank, total_q, kv8 != nullptr, ctx);
        const bool launched = cudaGetLastError() == cudaSuccess;
        if (ss && (cudaEventRecord(ss->join, ss->s) != cudaSuccess || !launched)) {
            (void)cudaStreamWaitEvent(s, ss->join, 0);  // leave the side stream joined
            return FA_ERR_CUDA;
        }
        if (!launched) return FA_ERR_CUDA;
        ++launches;
    }
    if (decode_path) {
        const int merge_rows = (int)std::min<long>(kDecodeRows, (long)g * max_q_len);
        const int qpf = is_decode_row(max_q_len, g) ? total_q : 0;  // every query row is a decode row
        if (acc) {
            mod->logits = reinterpret_cast<float*>(wsb + aw.logits);
            mod->logit_rows = merge_rows;
        }
        auto go = [&](auto dim, auto variant, auto cache) {
            return launch_decode<decltype(dim)::value, decltype(cache)::value, decltype(variant)::value>(
                q, k_cache, v_cache, block_table, ctx_lens, q_lens, out, w, wsb, num_seqs, max_blocks_per_seq,
                num_blocks, Hq, Hkv, tc_path ? INT_MAX : max_q_len, total_q, qpf, causal, scale, merge_rows, s, ctx, &launches, 1.f, 1.f,
                mod ? *mod : ScoreMod{}, kv8 ? kv8->k_exp : nullptr, kv8 ? kv8->v_exp : nullptr);
        };
        auto go_d = [&](auto variant, auto cache) {
            return d == 128 ? go(std::integral_constant<int, 128>{}, variant, cache)
                            : go(std::integral_constant<int, 64>{}, variant, cache);
        };
        const std::integral_constant<int, KV_BF16> bf16{};
        st = kv8   ? go_d(std::integral_constant<int, 0>{}, std::integral_constant<int, KV_FP8_SCALED>{})
             : acc ? go_d(std::integral_constant<int, 2>{}, bf16)
             : mod ? go_d(std::integral_constant<int, 1>{}, bf16)
                   : go_d(std::integral_constant<int, 0>{}, bf16);
        if (st != FA_OK) {
            if (ss) (void)cudaStreamWaitEvent(s, ss->join, 0);  // keep the side stream joined
            return st;
        }
    }
    if (tc_path) {
        if (ss && cudaStreamWaitEvent(s, ss->join, 0) != cudaSuccess) return FA_ERR_CUDA;
        int32_t* q_start = reinterpret_cast<int32_t*>(wsb + w.q_start);
        int32_t* count = reinterpret_cast<int32_t*>(wsb + w.work_count);
        int32_t* list = reinterpret_cast<int32_t*>(wsb + w.work_list);
        if (kv8)
            st = launch_paged_prefill_fp8(q, k_cache, v_cache, kv8->k_exp, kv8->v_exp, block_table, ctx_lens, q_lens, q_start,
                                          count, out, mod->lse, max_blocks_per_seq, num_blocks, Hq, Hkv, d, causal, scale,
                                          total_q, reinterpret_cast<const int4*>(wsb + pw.list),
                                          reinterpret_cast<float4*>(wsb + pw.o), reinterpret_cast<float2*>(wsb + pw.ml), s, ctx);
        else
            st = launch_paged_prefill(q, k_cache, v_cache, block_table, ctx_lens, q_lens, q_start, list, count, out,
                                      num_seqs, max_blocks_per_seq, num_blocks, Hq, Hkv, d, causal, scale, total_q, s,
                                      ctx, mod, mod ? reinterpret_cast<const int4*>(wsb + pw.list) : nullptr,
                                      reinterpret_cast<float4*>(wsb + pw.o), reinterpret_cast<float2*>(wsb + pw.ml));
        if (st != FA_OK) return st;
        ++launches;
        if (pw.slots > 0) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(4 * sm_count());
            cfg.blockDim = dim3(256);
            cfg.stream = s;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            auto join = d == 128 ? paged_join_kernel<128> : paged_join_kernel<64>;
            if (cudaLaunchKernelEx(&cfg, join, reinterpret_cast<const int4*>(wsb + pw.split),
                                   static_cast<const int32_t*>(count), reinterpret_cast<const float4*>(wsb + pw.o),
                                   reinterpret_cast<const float2*>(wsb + pw.ml), q_lens,
                                   static_cast<const int32_t*>(q_start), static_cast<uint16_t*>(out), mod->lse, pw.per_rank, Hq,
                                   g, total_q) != cudaSuccess)
                return FA_ERR_CUDA;
            ++launches;
        }
    }
    if (acc) {
        // rows whose queries took the decode kernel (and sequences without
        // queries), then the chunks: each sequence is one or the other
        // (about one wave of CTAs: a wide table says little about the contexts)
        const long want = std::max<long>(1, 8L * sm_count() / ((long)num_seqs * Hkv));
        const dim3 grid(num_seqs, Hkv, (unsigned)std::min<long>(want, (max_blocks_per_seq + kAccumPages - 1) / kAccumPages));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = grid;
        cfg.blockDim = dim3(kAccumPages * kBS);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, accum_decode_kernel, ctx_lens, q_lens, static_cast<const float*>(mod->lse),
                               static_cast<const float*>(mod->logits), mod->logit_rows, acc->in, acc->out, acc->len,
                               acc->decay, num_seqs, max_blocks_per_seq, Hq, Hkv, mod->window, total_q, ctx) !=
            cudaSuccess)
            return FA_ERR_CUDA;
        ++launches;
        if (tc_path) {
            st = launch_accum_chunk(q, k_cache, block_table, ctx_lens, q_lens,
                                    reinterpret_cast<int32_t*>(wsb + w.q_start),
                                    reinterpret_cast<int32_t*>(wsb + aw.k_start),
                                    reinterpret_cast<int32_t*>(wsb + aw.k_start) + num_seqs + 1,
                                    reinterpret_cast<int32_t*>(wsb + w.work_count) + 2, mod->lse, acc->in, acc->out, acc->len,
                                    acc->decay, num_seqs, max_blocks_per_seq, num_blocks, Hq, Hkv, d, causal, scale,
                                    total_q, *mod, s, ctx);
            if (st != FA_OK) return st;
            ++launches;
        }
    }
    set_launch_count(launches);
    return FA_OK;
}

}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_paged_attn_workspace_size(int num_seqs, int max_blocks_per_seq, int Hq, int Hkv, int d, int total_q) {
    if (num_seqs < 0 || max_blocks_per_seq < 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || total_q < 0) return 0;
    return paged_ws_layout(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q).total;
}

fa_status fa_paged_attn(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                        const int32_t* ctx_lens, const int32_t* q_lens, void* out, int num_seqs,
                        int max_blocks_per_seq, int num_blocks, int Hq, int Hkv, int d, int block_size, int causal,
                        float scale, int total_q, int max_q_len, void* ws, size_t ws_bytes, fa_stream_t stream) {
    return paged_attn_run(q, k_cache, v_cache, block_table, ctx_lens, q_lens, out, num_seqs, max_blocks_per_seq,
                          num_blocks, Hq, Hkv, d, block_size, causal, scale, total_q, max_q_len, ws, ws_bytes, stream,
                          nullptr, nullptr);
}

size_t fa_paged_attn_mod_workspace_size(int num_seqs, int max_blocks_per_seq, int Hq, int Hkv, int d, int total_q,
                                        int max_q_len) {
    if (max_q_len < 0) return 0;
    if (fa_paged_attn_workspace_size(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q) == 0 || Hq % Hkv != 0) return 0;
    const PagedWs w = paged_ws_layout(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q);
    return pieces_ws_layout(w, num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q, max_q_len, true).total;
}

fa_status fa_paged_attn_mod(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                            const int32_t* ctx_lens, const int32_t* q_lens, void* out, float* lse, int num_seqs,
                            int max_blocks_per_seq, int num_blocks, int Hq, int Hkv, int d, int block_size, int causal,
                            float scale, float softcap, const float* alibi_slopes, int window,
                            const int32_t* prefix_lens, int total_q, int max_q_len, void* ws, size_t ws_bytes,
                            fa_stream_t stream) {
    set_launch_count(0);
    ScoreMod mod;
    const fa_status st = make_score_mod(&mod, scale, softcap, alibi_slopes, window, prefix_lens, lse);
    if (st != FA_OK) return st;
    return paged_attn_run(q, k_cache, v_cache, block_table, ctx_lens, q_lens, out, num_seqs, max_blocks_per_seq,
                          num_blocks, Hq, Hkv, d, block_size, causal, scale, total_q, max_q_len, ws, ws_bytes, stream,
                          &mod, nullptr);
}

size_t fa_paged_attn_accum_workspace_size(int num_seqs, int max_blocks_per_seq, int Hq, int Hkv, int d, int total_q,
                                          int max_q_len) {
    const size_t base = fa_paged_attn_mod_workspace_size(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q, max_q_len);
    return base == 0 ? 0 : accum_ws_layout(base, num_seqs, max_blocks_per_seq, Hq, Hkv, max_q_len).total;
}

fa_status fa_paged_attn_accum(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                              const int32_t* ctx_lens, const int32_t* q_lens, void* out, float* lse,
                              const float* acc_in, float* acc_out, int acc_len, float decay, int num_seqs,
                              int max_blocks_per_seq, int num_blocks, int Hq, int Hkv, int d, int block_size,
                              int causal, float scale, float softcap, const float* alibi_slopes, int window,
                              const int32_t* prefix_lens, int total_q, int max_q_len, void* ws, size_t ws_bytes,
                              fa_stream_t stream) {
    set_launch_count(0);
    if (acc_len < 0 || !(decay >= 0.f) || !(decay < INFINITY)) return FA_ERR_INVALID_ARG;
    ScoreMod mod;
    const fa_status st = make_score_mod(&mod, scale, softcap, alibi_slopes, window, prefix_lens, lse);
    if (st != FA_OK) return st;
    if (num_seqs > 0 && total_q > 0 && max_q_len > 0 && (!lse || !acc_out)) return FA_ERR_INVALID_ARG;
    const AccumArgs acc{acc_in, acc_out, acc_len, decay};
    return paged_attn_run(q, k_cache, v_cache, block_table, ctx_lens, q_lens, out, num_seqs, max_blocks_per_seq,
                          num_blocks, Hq, Hkv, d, block_size, causal, scale, total_q, max_q_len, ws, ws_bytes, stream,
                          &mod, &acc);
}

fa_status fa_paged_attn_fp8(const void* q, const void* k_cache, const void* v_cache, float k_scale, float v_scale,
                            const int32_t* block_table, const int32_t* ctx_lens, const int32_t* q_lens, void* out,
                            int num_seqs, int max_blocks_per_seq, int num_blocks, int Hq, int Hkv, int d,
                            int block_size, int causal, float scale, int total_q, int max_q_len, void* ws,
                            size_t ws_bytes, fa_stream_t stream) {
    set_launch_count(0);
    if (num_seqs < 0 || max_blocks_per_seq < 0 || num_blocks < 0 || Hq <= 0 || Hkv <= 0 || total_q < 0 ||
        max_q_len < 0 || !(scale > 0.f) || !(scale < INFINITY) || !(k_scale > 0.f) || !(k_scale < INFINITY) ||
        !(v_scale > 0.f) || !(v_scale < INFINITY))
        return FA_ERR_INVALID_ARG;
    if (block_size != kBS || d != 128 || Hq % Hkv != 0) return FA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q == 0 || max_q_len == 0) return FA_OK;
    if (!is_decode_row(max_q_len, Hq / Hkv)) return FA_ERR_UNSUPPORTED;  // decode rows only
    if (!q || !k_cache || !v_cache || !block_table || !ctx_lens || !q_lens || !out) return FA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned32(out)) return FA_ERR_INVALID_ARG;
    if (num_blocks == 0 || max_blocks_per_seq == 0) return FA_ERR_INVALID_ARG;
    const PagedWs w = paged_ws_layout(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q);
    if (!ws || ws_bytes < w.total || (reinterpret_cast<uintptr_t>(ws) & 255)) return FA_ERR_WORKSPACE;
    fa_status st = check_device();
    if (st != FA_OK) return st;
    DevCtx ctx;
    if ((st = make_ctx(&ctx)) != FA_OK) return st;
    int launches = 0;
    st = launch_decode<128, KV_FP8>(q, k_cache, v_cache, block_table, ctx_lens, q_lens, out, w,
                                  static_cast<uint8_t*>(ws), num_seqs, max_blocks_per_seq, num_blocks, Hq, Hkv,
                                  max_q_len, total_q, total_q, causal, scale, (Hq / Hkv) * max_q_len,
                                  reinterpret_cast<cudaStream_t>(stream), ctx, &launches, k_scale, v_scale);
    if (st != FA_OK) return st;
    set_launch_count(launches);
    return FA_OK;
}

}  // extern "C"

extern "C" {

size_t fa_paged_attn_fp8_scaled_workspace_size(int num_seqs, int max_blocks_per_seq, int Hq, int Hkv, int d, int total_q,
                                               int max_q_len) {
    return fa_paged_attn_mod_workspace_size(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q, max_q_len);
}

fa_status fa_paged_attn_fp8_scaled(const void* q, const void* k_cache, const void* v_cache, const uint8_t* k_exp,
                                   const uint8_t* v_exp, const int32_t* block_table, const int32_t* ctx_lens,
                                   const int32_t* q_lens, void* out, float* lse, int num_seqs, int max_blocks_per_seq,
                                   int num_blocks, int Hq, int Hkv, int d, int block_size, int causal, float scale, int total_q,
                                   int max_q_len, void* ws, size_t ws_bytes, fa_stream_t stream) {
    set_launch_count(0);
    if (num_seqs > 0 && total_q > 0 && max_q_len > 0 && (!k_exp || !v_exp)) return FA_ERR_INVALID_ARG;
    if (Hkv > 0xffff) return FA_ERR_UNSUPPORTED;  // (a page's list entry has 16 bits for its head)
    ScoreMod mod{};  // nothing modified: its path keeps the log-sum-exp and shares chunks along their keys
    mod.lse = lse;
    const ScaledKv kv{k_exp, v_exp};
    return paged_attn_run(q, k_cache, v_cache, block_table, ctx_lens, q_lens, out, num_seqs, max_blocks_per_seq, num_blocks,
                          Hq, Hkv, d, block_size, causal, scale, total_q, max_q_len, ws, ws_bytes, stream, &mod, nullptr, &kv);
}

}  // extern "C"

// ------------------------------------------------------ allocation-free ---
// Scratch for fa_paged_attn_noalloc: a fixed device array that every GPU
// loading this library holds until the process exits.  Host code only sees a
// stand-in for its name, so its device address is looked up per device with
// cudaGetSymbolAddress (with that device current) and handed to the kernels.
namespace fa {
namespace {
static __device__ __align__(256) uint8_t g_noalloc_scratch[FA_NOALLOC_SCRATCH_BYTES];
std::mutex g_noalloc_mu;
void* g_noalloc_ptr[64] = {};

fa_status noalloc_scratch(void** out) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FA_ERR_CUDA;
    std::lock_guard<std::mutex> lk(g_noalloc_mu);
    if (!g_noalloc_ptr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || !p) return FA_ERR_CUDA;
        g_noalloc_ptr[dev] = p;
    }
    *out = g_noalloc_ptr[dev];
    return FA_OK;
}
}  // namespace
}  // namespace fa

extern "C" fa_status fa_paged_attn_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                           const int32_t* block_table, const int32_t* ctx_lens,
                                           const int32_t* q_lens, void* out, int num_seqs, int max_blocks_per_seq,
                                           int num_blocks, int Hq, int Hkv, int d, int block_size, int causal,
                                           float scale, int total_q, int max_q_len, fa_stream_t stream) {
    const size_t need = fa_paged_attn_workspace_size(num_seqs, max_blocks_per_seq, Hq, Hkv, d, total_q);
    if (need > FA_NOALLOC_SCRATCH_BYTES) return FA_ERR_WORKSPACE;  // problem too large for the fixed scratch
    void* scratch = nullptr;
    fa_status st = fa::noalloc_scratch(&scratch);
    if (st != FA_OK) return st;
    return fa_paged_attn(q, k_cache, v_cache, block_table, ctx_lens, q_lens, out, num_seqs, max_blocks_per_seq,
                         num_blocks, Hq, Hkv, d, block_size, causal, scale, total_q, max_q_len, scratch,
                         FA_NOALLOC_SCRATCH_BYTES, stream);
}
