// nvfp4kv_tree_attention_tc.cu -- attention of a drafted tree's nodes over the
// NVFP4 KV cache on the sm_100a tensor cores (tcgen05).
//
// Node i of sequence b (its K/V already appended at slot start[b] + i) sees
// every token t < start[b], and slot start[b] + j iff bit j of its mask row is
// set (without a mask: j <= i, a chain).  With g query heads per KV head the
// nodes make rows = nodes * g rows of one (sequence, KV head), all of which
// read the same keys and values:
//     S = Q . K^T     M = 128 rows, N = 128 tokens, K = head_dim
//     O += P . V      M = 128 rows, N = head_dim,   K = 128 tokens
// over the cache's FP8 values, exact in f16 (kind::f16 MMAs, fp32
// accumulators in tensor memory).  A bf16 query is exact in f16 after a
// power-of-two row scaling.
//
// Work split: the (sequence, KV head, row unit, 128-token tile) list is cut
// into one equal contiguous range per CTA, one CTA per SM.  A unit is up to RB x
// 128 rows, which share every dequantized tile.  Units cut by a range's end
// leave partial (O, m, l) in the workspace; a second small kernel merges them.
//
// Two softmax groups of 128 threads work on alternate items, each with its own
// scores S and accumulator O in tensor memory, so that one group's waits are the
// other's work.  An item is one tile of the unit's rows (alternate tiles go to
// alternate groups, whose (m, l, O) are merged when the unit ends); a unit of
// more than 128 rows makes two items of every tile, a row block to each group.
// Thread r of a group owns row r.  With 64 rows or fewer the rows stand 2 or 4 times
// among the 128, and each copy takes its part of the tile's tokens: the softmax's time
// falls with the rows, at no cost to the MMAs, which multiply 128 rows anyway.  P . V of
// a copy's tokens writes its lanes of O only (the others are disabled), so that nothing
// needs zeroing.
//
// A query row with a NaN or an infinity enters as NaN throughout: all of its scores are
// NaN then, and the row's m and l carry it to the output wherever a token is seen.
//
// Warp roles:
//   warps 0-7    softmax, groups 0 and 1; they also load the queries
//   warps 8-9    bulk copies of raw codes and scales into the ring: keys, values
//   warp 10      MMA issue (one elected lane): O += P(i) . V, then S(i + 2)
//   warps 12-    dequant, DG groups of eight warps; group i takes tiles i mod DG:
//                thread t of its first four warps owns token t's keys, of the
//                others its values
//   warp 11      prefetch of the segments' queries into L2
// P overwrites S in tensor memory, as the A operand of P . V: it takes no
// shared memory.
//
// What only the hardware signals (copies and MMAs that have ended) is an
// mbarrier; what warps signal is a named barrier.  A wait that gives up sets
// the CTA's abort flag; every role then runs through its loop without work, so
// that all named barriers are met.
//
// Measured (B200, head_dim 128; a tile's raw bytes take 774 clocks of an SM's share
// of 6.55 TB/s, its MMAs 512 with one row block and 1,024 with two):
//   128 sequences x 8 KV heads, up to 8 nodes x 4 heads, 1,024 to 8,192 tokens:
//     361 us, 1,870 clocks a tile within a unit.  A loop of waits paces it, for each of two
//     buffers: dequant 2,300 to 2,900 (the SM issues 0.59 instructions a clock and
//     scheduler, the integer pipe is 58% busy), then 1,000 of MMA issue and completion.
//     Between two units of a CTA lie 9,000 to 12,000 clocks: the unit's end, the next
//     one's queries and first scores.
//   8 KV heads, 32 nodes x 8 heads (two row blocks), 64K tokens: 101 us, 4,480 clocks
//     a tile; the softmax paces it: 3,300 of arithmetic (256 x 128 exponentials are
//     2,048 at the SM's 16 a clock) and 1,200 between P and the next scores
//   DRAM bytes read are the cache's (172.3 MB for 172.6 with queries and outputs, 32
//     ragged sequences); the tensor pipe is 42% busy there, 38% at 64K tokens and 51% at
//     128K with the second term.
// Tried and slower on the first, each against its day's figure: rows on N, with one
// exchange of maxima per tile (394 us); 8 dequant warps in place of 16 (451 us, 433);
// all 16 on each tile (438, 370); e4m3 keys with queries in two e4m3/e5m2 terms and a
// third value buffer (377, 370: 10% fewer integer instructions, but more code than
// the instruction cache holds).  On the second: the next scores read ahead (107, 102).
#include <cuda_bf16.h>

#include <algorithm>

#include "nvfp4kv_device.cuh"
#include "nvfp4kv_internal.h"
#include "nvfp4kv_pipeline.cuh"
#include "nvfp4kv_tcgen05.cuh"

namespace nvfp4kv {

namespace {

constexpr int T = 128;                                // tokens per tile, rows per row block
constexpr int kLoadWarp = 8, kMmaWarp = 10, kDqWarp0 = 12;
// named barriers (0: __syncthreads)
constexpr int kBarSoftmax = 1, kBarK = 2, kBarV = 4, kBarP = 6, kBarDq = 8, kBarMeet = 12;
constexpr uint32_t kTmemCols = 512;
// O is rescaled only when a row's running max grows by more than 2^kSlack;
// P = 2^(s - m + kBias) <= 2^14 stays inside f16, and weights down to 2^-30
// of the row's largest keep a bit of it
constexpr float kSlack = 8.0f, kBias = 6.0f;
constexpr int kLutCopies = 2;
// fp32 outputs: the tensor core truncates its accumulator at every 16-token
// step, a bias that grows with the context (1.6e-5 of the output at 128K
// tokens).  After this many of a group's items O is added, with rounding, to an
// fp32 sum in the workspace, and started again.
constexpr int kFlush = 16;

struct Params {
    const void* q;                                    // [B][N][Hq][D] bf16
    const uint8_t *kc, *ks, *vc, *vs;
    const float *st_k, *st_v;
    const int32_t *start, *n_nodes, *mask, *block_table;
    int64_t mask_stride;
    void* out;                                        // [B][N][Hq][D]
    float* partials;                                  // [2 * grid] slots
    float* sums;                                      // [2 * grid][D][128]: flushed O of each group (fp32 outputs)
    int4* desc;                                       // [grid] units cut by a range's start
    int32_t* status;
    int32_t B, N, Hq, Hkv, g, S_max, W;               // W mask words per node
    int32_t page_tokens, max_pages, num_pages;
    int32_t out_bf16;
    float scale_log2;                                 // softmax scale * log2(e)
    uint32_t wait_polls;
    FastDiv fd_g;
};

template <int D_, int RB_>
struct Cfg {
    static constexpr int D = D_, RB = RB_;
    // Dequant groups of eight warps.  One takes 1,900 to 2,450 clocks a tile: less than
    // two row blocks' softmax (3,400), whose threads the registers of a second group
    // would be taken from; more than one block's (1,700 over two groups), where the
    // second gains 4%.
    static constexpr int DG = RB == 2 ? 1 : 2;
    static constexpr int kThreads = 32 * (kDqWarp0 + 8 * DG);
    // registers after the prologue: 256 x softmax + 128 x misc + 256 DG x dequant, of
    // 640 x 96 = 61,440 or 896 x 72 = 64,512
    static constexpr uint32_t kRegsSoftmax = DG == 1 ? 136 : 112, kRegsMisc = DG == 1 ? 64 : 56,
                              kRegsDequant = DG == 1 ? 72 : 56;
    static constexpr int kCB = D / 2, kSB = D / 16;   // code / scale bytes per token
    static constexpr int kStage = T * (2 * kCB + 2 * kSB);
    static constexpr int kOffVC = T * kCB, kOffKS = 2 * T * kCB, kOffVS = 2 * T * kCB + T * kSB;
    static constexpr int kRing = RB == 2 && D == 128 ? 1 : 3;
    static constexpr int kTileBytes = T * D * 2;
    static constexpr uint32_t kColO = 0, kColS = 2 * D;   // of each group
    static constexpr int kSlot = RB * T * (D + 2);    // floats of a partial: O [D/4][row][4], (m, l) [row]
};

// Canonical non-swizzled layouts (8 rows x 16 bytes per core matrix): K-major
// (r/8) * 16D + (k/8) * 128 + (r%8) * 16, MN-major (d/8) * 2048 + (t/8) * 128 +
// (t%8) * 16 (bytes).
template <class C>
struct __align__(1024) Smem {
    uint8_t q[C::RB][C::kTileBytes];
    uint8_t k[2][C::kTileBytes];
    uint8_t v[2][C::kTileBytes];
    uint8_t ring[C::kRing][C::kStage];
    uint2 lut[2][128][kLutCopies];
    float cs[C::RB][T];                               // score factor of a row
    float ml[2][2][T];                                // m and l of each group's rows
    int32_t prefix[kMaxBatchPerLaunch + 1];
    int32_t warp_tot[16];
    uint64_t full[2][C::kRing], empty[2][C::kRing];   // keys, values
    uint64_t kfree[2], vfree[2], sready[2], pdone[2], qready, oread, mma_done;
    uint32_t tmem_base;
    int32_t abort_flag;
};

__device__ __forceinline__ void tmem_st_x16(uint32_t addr, const uint32_t* v) {
    tc::tmem_st_x8(addr, v);
    tc::tmem_st_x8(addr + 8, v + 8);
}

// STEPS kind::f16 MMAs (K = 16 each) with A and B in shared memory, the
// descriptors advancing 256 bytes a step; the first accumulates when acc != 0.
template <int STEPS>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
#define NVFP4_SS_STEP "add.s64 %1, %1, 16;\n\tadd.s64 %2, %2, 16;\n\t" \
                      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p1;\n\t"
    if (STEPS == 8)
        asm volatile("{\n\t.reg .pred p0, p1;\n\tsetp.ne.b32 p0, %3, %3;\n\tsetp.eq.b32 p1, %3, %3;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p0;\n\t"
                     NVFP4_SS_STEP NVFP4_SS_STEP NVFP4_SS_STEP NVFP4_SS_STEP NVFP4_SS_STEP NVFP4_SS_STEP
                     NVFP4_SS_STEP "}"
                     : "+r"(d), "+l"(a), "+l"(b) : "r"(idesc) : "memory");
    else
        asm volatile("{\n\t.reg .pred p0, p1;\n\tsetp.ne.b32 p0, %3, %3;\n\tsetp.eq.b32 p1, %3, %3;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p0;\n\t"
                     NVFP4_SS_STEP NVFP4_SS_STEP NVFP4_SS_STEP "}"
                     : "+r"(d), "+l"(a), "+l"(b) : "r"(idesc) : "memory");
#undef NVFP4_SS_STEP
}

// Two kind::f16 MMAs over 32 tokens with A = P in tensor memory, columns a .. a + 15,
// into the lanes that off[] does not name (a bit per lane of D).
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc,
                                       const uint32_t (&off)[4]) {
    asm volatile("{\n\t.reg .pred p0, p1;\n\tsetp.ne.b32 p0, %4, 0;\n\tsetp.eq.b32 p1, %4, %4;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p0;\n\t"
                 "add.u32 %1, %1, 8;\n\tadd.s64 %2, %2, 16;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p1;\n\t}"
                 : "+r"(d), "+r"(a), "+l"(b)
                 : "r"(idesc), "r"(acc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3])
                 : "memory");
}

template <uint32_t N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Named barriers of n threads.  What a warp did before (fenced for the async proxy
// where the tensor cores read it) comes before what the others do after.  Producers
// and the MMA warp both wait: if a producer's warp only arrived, one that came again
// early (as the roles do once a wait has given up) would stand for another warp.
// (Arriving only was no faster: 371 us for 368 then on the ragged batch above.)
__device__ __forceinline__ void bar_sync(int id, int n) {
    asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ void softmax_sync() { bar_sync(kBarSoftmax, 256); }

__device__ __forceinline__ uint4 dequant8(uint32_t x, uint2 l) {
    uint32_t lo, hi;
    dequant_word(x, l.x, l.y, lo, hi);
    uint4 o;
    e4m3x4_to_f16x2x2(lo, o.x, o.y);
    e4m3x4_to_f16x2x2(hi, o.z, o.w);
    return o;
}

// nodes of sequence b that attend; 0 for a padding row or one that is refused
__device__ __forceinline__ int live_nodes(const Params& p, int b, int start, int& err) {
    const int n = p.n_nodes != nullptr ? p.n_nodes[b] : p.N;
    err = 0;
    if (n < 0 || n > p.N) {
        err = NVFP4_ERR_INVALID_ARG;
        return 0;
    }
    if (start < 0 || (int64_t)start + n > p.S_max) {
        err = NVFP4_ERR_CAPACITY;
        return 0;
    }
    return n;
}

// One contiguous run of tiles of one unit inside a CTA's range.
struct Segment {
    int b, hk, ru;                                    // sequence, KV head, row unit
    int start, nodes, rows;                           // rows of this unit
    int tile0, tiles, unit_tiles;
};

// log2 of the copies of a unit's rows
__device__ __forceinline__ int lg_copies(int rows) { return rows > 64 ? 0 : (rows > 32 ? 1 : 2); }

template <class C>
struct Walker {
    int pos, end, b;
    __device__ __forceinline__ Walker(int lo, int hi) : pos(lo), end(hi), b(0) {}
    __device__ __forceinline__ bool next(const Params& p, const int32_t* prefix, Segment& s) {
        if (pos >= end) return false;
        if (pos >= prefix[b + 1]) {                   // the last b with prefix[b] <= pos
            int lo = b + 1, hi = p.B - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (prefix[mid] <= pos) lo = mid;
                else hi = mid - 1;
            }
            b = lo;
        }
        s.b = b;
        s.start = p.start[b];
        int err;
        s.nodes = live_nodes(p, b, s.start, err);
        const int all_rows = s.nodes * p.g;
        const int nru = (all_rows + C::RB * T - 1) / (C::RB * T);
        s.unit_tiles = (s.start + s.nodes + T - 1) / T;
        const int rem = pos - prefix[b];
        const int u = rem / s.unit_tiles;
        s.tile0 = rem - u * s.unit_tiles;
        s.hk = u / nru;
        s.ru = u - s.hk * nru;
        s.rows = min(C::RB * T, all_rows - s.ru * C::RB * T);
        s.tiles = min(s.unit_tiles - s.tile0, end - pos);
        pos += s.tiles;
        return true;
    }
};

// 64 bits from bit `o` of a mask row of W words (bits past the row: 0)
__device__ __forceinline__ uint64_t mask_bits(const int32_t* row, int W, int o) {
    const int w = o >> 5, sh = o & 31;
    const uint32_t a = w < W ? (uint32_t)__ldg(row + w) : 0u;
    const uint32_t b = w + 1 < W ? (uint32_t)__ldg(row + w + 1) : 0u;
    const uint32_t c = w + 2 < W ? (uint32_t)__ldg(row + w + 2) : 0u;
    return (uint64_t)__funnelshift_r(a, b, sh) | ((uint64_t)__funnelshift_r(b, c, sh) << 32);
}

__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1); }

// which of tokens t0 .. t0 + 63 node i sees
__device__ __forceinline__ uint64_t visible64(const Params& p, const Segment& s, int i, int t0) {
    const int rel = s.start - t0;                     // prefix tokens of the window
    const int j0 = rel > 0 ? 0 : -rel;                // first node of the window
    uint64_t tree;
    if (p.mask == nullptr)
        tree = low_bits(i + 1 - j0);
    else
        tree = mask_bits(p.mask + (int64_t)s.b * p.mask_stride + (int64_t)i * p.W, p.W, j0) & low_bits(s.nodes - j0);
    if (rel <= 0) return tree;
    return low_bits(rel) | (rel < 64 ? tree << rel : 0ull);
}

template <class C, bool TWO>
__global__ void __launch_bounds__(C::kThreads, 1) tree_attention_tc_kernel(const __grid_constant__ Params p) {
    constexpr int D = C::D, RB = C::RB;
    extern __shared__ uint8_t smem_raw[];
    Smem<C>& sm = *reinterpret_cast<Smem<C>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- prologue: barriers, lookup tables, the split ----
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&sm.tmem_base, kTmemCols);
        tc::tmem_relinquish();
    }
    if (warp == kLoadWarp && lane == 0) {
        for (int s = 0; s < C::kRing; ++s) {
            for (int kv = 0; kv < 2; ++kv) {
                mbar_init(&sm.full[kv][s], 1);
                mbar_init(&sm.empty[kv][s], 4);
            }
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.kfree[s], 1);
            mbar_init(&sm.vfree[s], 1);
            mbar_init(&sm.sready[s], 1);
            mbar_init(&sm.pdone[s], 1);
        }
        mbar_init(&sm.qready, 1);
        mbar_init(&sm.oread, 1);
        mbar_init(&sm.mma_done, 1);
        fence_mbar_init();
        sm.abort_flag = 0;
    }
    const float st_k = *p.st_k, st_v = *p.st_v;
    if (tid < 256) {
        const int plane = tid >> 7;
        const uint2 w = lut_words((uint32_t)(tid & 127), plane ? st_v : st_k);
#pragma unroll
        for (int c = 0; c < kLutCopies; ++c)          // lanes rotated over the banks
            sm.lut[plane][tid & 127][(c + lane) & (kLutCopies - 1)] = w;
    }
    if (tid == 0 && blockIdx.x == 0) {
        const bool ok = st_k > 0.f && st_k <= 3.4028234663852886e38f && st_v > 0.f && st_v <= 3.4028234663852886e38f;
        if (!ok) report(p.status, NVFP4_ERR_NONFINITE);
    }
    {
        int tiles = 0;
        if (tid < p.B) {
            const int start = p.start[tid];
            int err;
            const int n = live_nodes(p, tid, start, err);
            if (err && blockIdx.x == 0) report(p.status, err);
            if (n > 0) tiles = p.Hkv * ((n * p.g + RB * T - 1) / (RB * T)) * ((start + n + T - 1) / T);
        }
        int incl = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += up;
        }
        if (warp < 16 && lane == 31) sm.warp_tot[warp] = incl;
        __syncthreads();
        if (warp < 16) {
            int before = 0;
            for (int w = 0; w < warp; ++w) before += sm.warp_tot[w];
            sm.prefix[tid + 1] = before + incl;
            if (tid == 0) sm.prefix[0] = 0;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tbase = sm.tmem_base;
    int32_t* const abort_flag = &sm.abort_flag;
    const uint32_t polls = p.wait_polls;
    // as many ranges as there are tiles at most, so that none is empty between others
    const int total = sm.prefix[p.B];
    const int nr = total < (int)gridDim.x ? (total > 0 ? total : 1) : (int)gridDim.x;
    auto range_start = [&](int c) -> int { return (int)((int64_t)total * (c < nr ? c : nr) / nr); };
    const int lo = range_start((int)blockIdx.x), hi = range_start((int)blockIdx.x + 1);

    if (warp >= kLoadWarp && warp < kDqWarp0) {
        regs_dec<C::kRegsMisc>();
        if (warp < kLoadWarp + 2 && lane == 0) {
            // ================= bulk copies, one stage per tile: keys or values =================
            const int which = warp - kLoadWarp;
            uint64_t* const full = sm.full[which];
            uint64_t* const empty = sm.empty[which];
            const uint8_t* const codes = which ? p.vc : p.kc;
            const uint8_t* const scales = which ? p.vs : p.ks;
            uint32_t n = 0;                           // tiles issued
            bool ok = true;
            Walker<C> w(lo, hi);
            Segment s;
            while (ok && w.next(p, sm.prefix, s)) {
#pragma unroll 1
                for (int k = 0; k < s.tiles; ++k, ++n) {
                    const int st = n % C::kRing;
                    if (n >= C::kRing && !wait_one(&empty[st], (n / C::kRing - 1) & 1, abort_flag, p.status, polls)) {
                        ok = false;
                        break;
                    }
                    const int t0 = (s.tile0 + k) * T;
                    const int live = min(T, s.start + s.nodes - t0);
                    const int ncopy = (live + 3) & ~3;  // every copy a multiple of 16 bytes
                    int64_t tok;
                    if (p.block_table == nullptr) {
                        tok = ((int64_t)s.b * p.Hkv + s.hk) * p.S_max + t0;
                    } else {
                        const int lp = t0 / p.page_tokens;
                        int32_t page = p.block_table[(int64_t)s.b * p.max_pages + lp];
                        if (page < 0 || page >= p.num_pages) {
                            report(p.status, NVFP4_ERR_INVALID_ARG);
                            page = 0;
                        }
                        tok = ((int64_t)page * p.Hkv + s.hk) * p.page_tokens + (t0 - lp * p.page_tokens);
                    }
                    const uint32_t cb = (uint32_t)ncopy * C::kCB, sb = (uint32_t)ncopy * C::kSB;
                    mbar_arrive_expect_tx(&full[st], cb + sb);
                    bulk_g2s(sm.ring[st] + (which ? C::kOffVC : 0), codes + tok * C::kCB, cb, &full[st]);
                    bulk_g2s(sm.ring[st] + (which ? C::kOffVS : C::kOffKS), scales + tok * C::kSB, sb, &full[st]);
                }
            }
            // ---- the unit that this range's start cuts first is merged by block
            // blockIdx.x: contributors and rows, sequence, KV head, row unit ----
            if (which == 0) {
                int4 d = make_int4(0, 0, 0, 0);
                Walker<C> w0(lo, hi);
                if (w0.next(p, sm.prefix, s) && s.tile0 > 0 && lo - s.tile0 >= range_start((int)blockIdx.x - 1)) {
                    int c = (int)blockIdx.x + 1;      // ranges blockIdx.x - 1 .. c - 1 hold tiles of it
#pragma unroll 1
                    while (c < nr && range_start(c) < lo - s.tile0 + s.unit_tiles) ++c;
                    d = make_int4((c - (int)blockIdx.x + 1) | s.rows << 16, s.b, s.hk, s.ru);
                }
                p.desc[blockIdx.x] = d;
            }
            // every issued copy lands before the CTA exits
            for (uint32_t i = n > C::kRing ? n - C::kRing : 0; i < n; ++i)
                if (!mbar_wait_sleep(&full[i % C::kRing], (i / C::kRing) & 1, 1u << 16)) {
                    report(p.status, NVFP4_ERR_TIMEOUT);
                    break;
                }
        } else if (warp == kMmaWarp) {
            // ================= MMA issue =================
            const uint32_t idesc_qk = tc::idesc_e4m3(128, 128, false, false, false);
            const uint32_t idesc_pv = tc::idesc_e4m3(128, D, false, true, false);   // B = V, MN-major
            uint32_t gi = 0, gt = 0, seg = 0;         // items, tiles, segments
            bool ok = true;
            Walker<C> w(lo, hi);
            Segment s;
            for (; w.next(p, sm.prefix, s); ++seg) {
                const int dual = RB == 2 && s.rows > T ? 1 : 0;
                const int items = s.tiles << dual;
                const int lg_parts = lg_copies(s.rows);
                ok = wait_warp(&sm.qready, seg & 1, abort_flag, p.status, polls) && ok;
                // S(i) = Q . K^T of group (gi + i) % 2.  (P(i - 2), which lay there, has been
                // read by an MMA issued before.)
                auto issue_qk = [&](int i) {
                    const uint32_t grp = (gi + i) & 1, kt = gt + (i >> dual), kb = kt & 1;
                    if (!dual || !(i & 1)) bar_sync(kBarK + kb, 160);
                    tc::fence_after_sync();
                    if (ok && tc::elect_one()) {
                        mma_ss<D / 16>(tbase + C::kColS + T * grp,
                                       tc::smem_desc(tc::smem_addr(sm.q[dual ? grp : 0]), 128, 16 * D),
                                       tc::smem_desc(tc::smem_addr(sm.k[kb]), 128, 16 * D), idesc_qk);
                        tc::mma_commit(&sm.sready[grp]);
                        if (!dual || (i & 1)) tc::mma_commit(&sm.kfree[kb]);
                    }
                    __syncwarp();
                };
                issue_qk(0);
                if (items > 1) issue_qk(1);
#pragma unroll 1
                for (int i = 0; i < items; ++i) {
                    const uint32_t grp = (gi + i) & 1, vt = gt + (i >> dual), vb = vt & 1;
                    if (!dual || !(i & 1)) bar_sync(kBarV + vb, 160);
                    if (i == 0 && seg > 0)            // the previous segment's O has been read
                        ok = wait_warp(&sm.oread, (seg - 1) & 1, abort_flag, p.status, polls) && ok;
                    bar_sync(kBarP + grp, 160);
                    tc::fence_after_sync();
                    if (ok && tc::elect_one()) {
                        const uint64_t dv = tc::smem_desc(tc::smem_addr(sm.v[vb]), 128, 2048);
                        const uint32_t a = tbase + C::kColS + T * grp, o = tbase + C::kColO + D * grp;
                        const int j = i >> 1;         // the group's items of this segment before
                        const uint32_t acc = (TWO ? j % kFlush : j) > 0 ? 1u : 0u;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            // the lanes of the copy that takes these 32 tokens
                            const int lg_cpp = 2 - lg_parts;   // chunks of a copy
                            uint32_t off[4];
#pragma unroll
                            for (int l = 0; l < 4; ++l) off[l] = l >> lg_cpp == c >> lg_cpp ? 0u : 0xFFFFFFFFu;
                            const uint32_t first = c & ((1 << lg_cpp) - 1);
                            mma_pv(o, a + 32 * c, dv + 32 * c, idesc_pv, first > 0 ? 1u : acc, off);
                            if (TWO) mma_pv(o, a + 32 * c + 16, dv + 32 * c, idesc_pv, 1u, off);
                        }
                        tc::mma_commit(&sm.pdone[grp]);
                        if (!dual || (i & 1)) tc::mma_commit(&sm.vfree[vb]);
                    }
                    __syncwarp();
                    if (i + 2 < items) issue_qk(i + 2);
                }
                gi += items;
                gt += s.tiles;
            }
            if (tc::elect_one()) tc::mma_commit(&sm.mma_done);
            __syncwarp();
        }
        else if (warp == kMmaWarp + 1) {
            // ================= the segments' queries, node by node, into L2 =================
            Walker<C> w(lo, hi);
            Segment s;
            while (w.next(p, sm.prefix, s)) {
                const int gr0 = s.ru * RB * T, nd0 = (int)p.fd_g.div((uint32_t)gr0),
                          nd1 = (int)p.fd_g.div((uint32_t)(gr0 + s.rows - 1));
                for (int nd = nd0 + lane; nd <= nd1; nd += 32) {
                    const int first = max(gr0 - nd * p.g, 0), end = min(p.g, gr0 + s.rows - nd * p.g);
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                                     reinterpret_cast<const uint16_t*>(p.q) +
                                     (((int64_t)s.b * p.N + nd) * p.Hq + (int64_t)s.hk * p.g + first) * D),
                                 "r"((end - first) * D * 2)
                                 : "memory");
                }
            }
        }
    } else if (warp >= kDqWarp0) {
        // ================= dequant: token t of each tile, keys or values =================
        regs_dec<C::kRegsDequant>();
        const int which = ((warp - kDqWarp0) >> 2) & 1;   // 0: keys, 1: values
        const int group = (warp - kDqWarp0) >> 3, bar = kBarDq + ((warp - kDqWarp0) >> 2);
        const int t = tid & (T - 1);
        const uint2* lut = &sm.lut[which][0][lane & (kLutCopies - 1)];
        const bool poller = (warp & 3) == 0;
        constexpr int NCH = D / 32;                   // 16-byte code chunks of a token
        const uint32_t ntiles = (uint32_t)(hi - lo);  // every tile of the range once, in order
#pragma unroll 1
        for (uint32_t n = group; n < ntiles; n += C::DG) {
            const uint32_t st = n % C::kRing, buf = n & 1;
            if (poller) {
                wait_warp(&sm.full[which][st], (n / C::kRing) & 1, abort_flag, p.status, polls);
                // the MMAs of the buffer's last tile have read it
                if (n >= 2)
                    wait_warp(which ? &sm.vfree[buf] : &sm.kfree[buf], ((n >> 1) - 1) & 1, abort_flag, p.status, polls);
            }
            bar_sync(bar, 128);
            const uint8_t* raw = sm.ring[st] + (which ? C::kOffVC : 0) + t * C::kCB;
            const uint8_t* sraw = sm.ring[st] + (which ? C::kOffVS : C::kOffKS) + t * C::kSB;
            uint8_t* dst = which ? sm.v[buf] + (t / 8) * 128 + (t % 8) * 16 : sm.k[buf] + (t / 8) * (16 * D) + (t % 8) * 16;
            const int step = which ? 2048 : 128;      // between 8-element groups of the head dimension
            // chunk order rotated per thread: eight lanes read eight different 16-byte
            // banks.  The loop stays rolled: the roles' loops together have to fit the
            // instruction cache.
            const int rot = D == 128 ? (t >> 1) : (t >> 2);
#pragma unroll 1
            for (int j = 0; j < NCH; ++j) {
                const int c = (j + rot) & (NCH - 1);
                const uint4 code = *reinterpret_cast<const uint4*>(raw + 16 * c);
                const uint32_t two = *reinterpret_cast<const uint16_t*>(sraw + 2 * c);
                const uint2 la = lut[(two & 0x7F) * kLutCopies];
                const uint2 lb = lut[(two >> 8 & 0x7F) * kLutCopies];
                uint8_t* const d8 = dst + 4 * c * step;
                *reinterpret_cast<uint4*>(d8) = dequant8(code.x, la);
                *reinterpret_cast<uint4*>(d8 + step) = dequant8(code.y, la);
                *reinterpret_cast<uint4*>(d8 + 2 * step) = dequant8(code.z, lb);
                *reinterpret_cast<uint4*>(d8 + 3 * step) = dequant8(code.w, lb);
            }
            fence_proxy_async_smem();
            // this warp has read (and used) what it needs of the stage
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.empty[which][st]);
            bar_sync((which ? kBarV : kBarK) + (int)buf, 160);
        }
    } else {
        // ================= softmax: row r (or its copy) of the group's items =================
        regs_inc<C::kRegsSoftmax>();
        const int h = warp >> 2, r = tid & (T - 1);
        const uint32_t trow = tbase + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t scol = trow + C::kColS + T * h, ocol = trow + C::kColO + D * h;
        float* const sums = TWO ? p.sums + (int64_t)(2 * blockIdx.x + h) * D * T + r : nullptr;
        uint32_t gi = 0, seg = 0;
        Walker<C> w(lo, hi);
        Segment s;
#pragma unroll 1
        for (; w.next(p, sm.prefix, s); ++seg) {
            const int dual = RB == 2 && s.rows > T ? 1 : 0;
            // copies of the rows, and tokens of a tile each takes: 128, 64 or 32
            const int lg_parts = lg_copies(s.rows);
            const int rows_per = T >> lg_parts, part = r >> (7 - lg_parts), lr = r & (rows_per - 1);
            const int gr0 = s.ru * RB * T;
            // ---- query operand: q * 2^e rounded to f16, e from the row's amax ----
            {
                // Lanes: 8 rows x 4 quarters of every 32 columns, so that eight lanes write
                // 128 contiguous bytes of the operand; all of a row's loads are in flight.
                constexpr int NP = D / 32;
                const int quarter = lane >> 3;
                const int rows = dual ? 2 * T : rows_per, copies = dual ? 1 : 1 << lg_parts;
                const uint16_t* qh = reinterpret_cast<const uint16_t*>(p.q) +
                                     ((int64_t)s.b * p.N * p.Hq + (int64_t)s.hk * p.g) * D + 8 * quarter;
#pragma unroll 1
                for (int row = 8 * warp + (lane & 7); row < rows; row += 64) {   // (a warp's rows: all or none)
                    uint32_t x[4 * NP];
                    const int gr = gr0 + row, qn = (int)p.fd_g.div((uint32_t)gr);
#pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        uint4 u = make_uint4(0, 0, 0, 0);
                        if (row < s.rows)
                            u = __ldg(reinterpret_cast<const uint4*>(qh + ((int64_t)qn * p.Hq + (gr - qn * p.g)) * D + 32 * k));
                        x[4 * k] = u.x; x[4 * k + 1] = u.y; x[4 * k + 2] = u.z; x[4 * k + 3] = u.w;
                    }
                    uint32_t amax = 0;
#pragma unroll
                    for (int j = 0; j < 4 * NP; ++j) amax = max(amax, max((x[j] & 0x7FFFu) << 16, x[j] & 0x7FFF0000u));
                    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 8));
                    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 16));
                    int e = 0;
                    if (amax > 0u && amax < 0x7F800000u) {
                        // amax < 2^(ex + 1); a subnormal takes the largest shift
                        e = 14 - ((int)(amax >> 23) - 127);
                        e = e < -126 ? -126 : (e > 126 ? 126 : e);
                    }
                    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
                    const float cs = fmaxf(p.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23), 1.17549435e-38f);
#pragma unroll
                    for (int j = 0; j < 4 * NP; ++j)
                        x[j] = amax < 0x7F800000u
                                   ? pack_f16x2(__uint_as_float(x[j] << 16) * up, __uint_as_float(x[j] & 0xFFFF0000u) * up)
                                   : 0x7FFF7FFFu;     // an infinity or a NaN in the row: all of its scores are NaN
#pragma unroll 1
                    for (int c = 0; c < copies; ++c) {
                        const int at = row + c * rows, rb = at >> 7;
                        uint8_t* d8 = sm.q[rb] + ((at & 127) / 8) * (16 * D) + quarter * 128 + (at % 8) * 16;
#pragma unroll
                        for (int k = 0; k < NP; ++k)
                            *reinterpret_cast<uint4*>(d8 + 512 * k) = make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                        if (quarter == 0) sm.cs[rb][at & 127] = cs;
                    }
                }
            }
            fence_proxy_async_smem();
            softmax_sync();
            if (tid == 0) mbar_arrive(&sm.qready);

            const int row = dual ? T * h + r : lr;    // of the unit
            const bool live = row < s.rows;
            // a warp without live rows leaves P as it is: it only reaches its own rows of O
            const bool idle = dual ? T * h + 32 * (warp & 3) >= s.rows : ((32 * (warp & 3)) & (rows_per - 1)) >= s.rows;
            const int nd = live ? (int)p.fd_g.div((uint32_t)(gr0 + row)) : 0;
            const float cs = sm.cs[dual ? h : 0][r];
            const int c_lo = part << (2 - lg_parts), c_hi = c_lo + (4 >> lg_parts);   // 32-token chunks
            float m_run = -INFINITY, l_run = 0.0f;
            float m_sum = -INFINITY;                  // m of the flushed O
            int own = 0;                              // this group's items of the segment so far
#pragma unroll 1
            for (int i = (int)((gi ^ h) & 1); i < s.tiles << dual; i += 2, ++own) {
                const uint32_t x = gi + i;
                const int t0 = (s.tile0 + (i >> dual)) * T;
                wait_warp(&sm.sready[h], (x >> 1) & 1, abort_flag, p.status, polls);
                tc::fence_after_sync();
                if (!idle) {
                    const bool tail = t0 + T > s.start;
                    // ---- the row's max over its tokens ----
                    uint32_t v[32];
                    float mt = -INFINITY;
#pragma unroll 1
                    for (int c = c_lo; c < c_hi; ++c) {
                        tc::tmem_ld_x16(scol + 32 * c, v);
                        tc::tmem_ld_x16(scol + 32 * c + 16, v + 16);
                        tc::tmem_wait_ld();
                        if (tail) {
                            const uint32_t vis = (uint32_t)visible64(p, s, nd, t0 + 32 * c);
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!((vis >> j) & 1)) v[j] = 0xFF800000u;
                        }
                        float m4[4] = {__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3])};
#pragma unroll
                        for (int j = 4; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], __uint_as_float(v[j]));
                        mt = fmaxf(mt, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
                    }
                    mt *= cs;
                    float f = 1.0f;
                    if (mt > m_run + kSlack || m_run == -INFINITY) {
                        const float m_new = fmaxf(m_run, mt);
                        f = m_new == m_run ? 1.0f : (m_run == -INFINITY ? 0.0f : fast_exp2(m_run - m_new));
                        l_run *= f;
                        m_run = m_new;
                    }
                    // The group's O is complete: its last P . V was issued before this S.
                    // (tcgen05.ld/st are warp-wide: all rows rescale when any must.)
                    const bool flush = TWO && own > 0 && own % kFlush == 0;
                    if (own > 0 && (flush || __any_sync(0xFFFFFFFFu, f != 1.0f))) {
                        const float fs = m_sum == -INFINITY ? 0.0f : fast_exp2(m_sum - m_run);
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tc::tmem_ld_x16(ocol + c, o);
                            tc::tmem_wait_ld();
                            if (flush) {
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    float y = __uint_as_float(o[j]) * f;
                                    if (own > kFlush) y = __fmaf_rn(sums[(c + j) * T], fs, y);
                                    sums[(c + j) * T] = y;
                                }
                            } else {
#pragma unroll
                                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tc::tmem_st_x8(ocol + c, o);
                                tc::tmem_st_x8(ocol + c + 8, o + 8);
                            }
                        }
                        if (flush) m_sum = m_run;
                    }
                    // ---- weights: chunk c to columns 32c .. 32c + 15 (second terms: + 16) ----
                    const float base = (m_run == -INFINITY ? 0.0f : m_run) - kBias;
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
                    for (int c = c_lo; c < c_hi; ++c) {
                        if (lg_parts < 2) {           // else the one chunk is still here
                            tc::tmem_ld_x16(scol + 32 * c, v);
                            tc::tmem_ld_x16(scol + 32 * c + 16, v + 16);
                            tc::tmem_wait_ld();
                            if (tail) {
                                const uint32_t vis = (uint32_t)visible64(p, s, nd, t0 + 32 * c);
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    if (!((vis >> j) & 1)) v[j] = 0xFF800000u;
                            }
                        }
                        uint32_t lo16[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float a = fast_exp2(__fmaf_rn(__uint_as_float(v[2 * j]), cs, -base));
                            const float b = fast_exp2(__fmaf_rn(__uint_as_float(v[2 * j + 1]), cs, -base));
                            sum[2 * (j & 1)] += a;
                            sum[2 * (j & 1) + 1] += b;
                            v[j] = pack_f16x2(a, b);
                            if (TWO) lo16[j] = pack_f16x2(a - f16_lo_to_float(v[j]), b - f16_hi_to_float(v[j]));
                        }
                        tmem_st_x16(scol + 32 * c, v);
                        if (TWO) tmem_st_x16(scol + 32 * c + 16, lo16);
                    }
                    l_run += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tc::tmem_wait_st();
                }
                tc::fence_before_sync();
                bar_sync(kBarP + h, 160);
            }
            gi += (uint32_t)s.tiles << dual;

            // ---- both groups' O are complete: their shares of a row ----
            // (the last two items' P . V: one of each group, or there was one item)
            for (uint32_t x = gi >= 2 ? gi - 2 : 0; x < gi; ++x)
                wait_warp(&sm.pdone[x & 1], (x >> 1) & 1, abort_flag, p.status, polls);
            // A NaN among the row's weights (all of its scores, then) is carried in m: the
            // running maximum passes NaN by, and -infinity says that nothing was seen.
            sm.ml[h][0][r] = live ? (l_run == l_run ? m_run : l_run) : -INFINITY;
            sm.ml[h][1][r] = live ? l_run : 0.0f;
            softmax_sync();
            tc::fence_after_sync();
            const bool whole = s.tiles == s.unit_tiles;
            float* const slot = p.partials + (int64_t)(2 * blockIdx.x + (s.tile0 > 0 ? 0 : 1)) * C::kSlot;
            // m and l of the row over its copies and, unless each group has its own rows, groups
            float m8[8], m_all = -INFINITY, l_all = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int g = i >> 2, q = i & 3;
                m8[i] = (!dual || g == h) && q < 1 << lg_parts ? sm.ml[g][0][lr + q * rows_per] : -INFINITY;
                m_all = fmaxf(m_all, m8[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (m8[i] != -INFINITY)
                    l_all = __fmaf_rn(sm.ml[i >> 2][1][lr + (i & 3) * rows_per], fast_exp2(m8[i] - m_all), l_all);
            const float inv = whole ? (l_all == 0.0f ? 0.0f : 1.0f / l_all) : 1.0f;
            // factors of the groups' O (of this copy); 0 where a group saw nothing: O is anything then
            float fo[2], ff[2];                       // of O, and of what was flushed of it
            int flushed[2];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const float mg = dual && g != h ? -INFINITY : sm.ml[g][0][r];
                fo[g] = mg == -INFINITY ? 0.0f : fast_exp2(mg - m_all) * inv;
                ff[g] = 0.0f;
                flushed[g] = 0;
            }
            if (TWO) {
                // the groups exchange the m of their flushed sums
                const int mine = own > 0 ? (own - 1) / kFlush : 0;
                softmax_sync();
                sm.ml[h][0][r] = mine > 0 ? m_sum : -INFINITY;
                softmax_sync();
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const float mg = dual && g != h ? -INFINITY : sm.ml[g][0][r];
                    ff[g] = mg == -INFINITY ? 0.0f : fast_exp2(mg - m_all) * inv;
                    flushed[g] = !dual || g == h;
                }
            }
            const int64_t at =
                (((int64_t)s.b * p.N + nd) * p.Hq + (int64_t)s.hk * p.g + (gr0 + row - nd * p.g)) * D;
            // four columns of the row: fp32 to the partial (or the output), or bf16
            float* const dst = whole && TWO ? reinterpret_cast<float*>(p.out) + at : slot + 4 * row;
            const int dst_step = whole && TWO ? 4 : 4 * RB * T;
            auto store4 = [&](int col, float4 z) {
                if (!live) return;
                if (!TWO && whole) {
                    const __nv_bfloat162 e = __floats2bfloat162_rn(z.x, z.y), f = __floats2bfloat162_rn(z.z, z.w);
                    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + at + col) =
                        make_uint2(*reinterpret_cast<const uint32_t*>(&e), *reinterpret_cast<const uint32_t*>(&f));
                } else {
                    *reinterpret_cast<float4*>(dst + (col / 4) * dst_step) = z;
                }
            };
            // Columns 16 at a time: group h takes every other 16 (all of them when the rows
            // are its own).  The copies' sums meet in the query buffer, 64 bytes a row, its
            // 16-byte pieces permuted so that eight rows' fill all banks; each copy sums
            // its share of the pieces over the copies.  (Two buffers where the query buffer
            // holds them: one barrier less.)
            constexpr bool TWOBUF = sizeof(sm.q[0]) >= 4 * T * 16 * sizeof(float);
            float4* const meet0 = reinterpret_cast<float4*>(sm.q[0]) + h * (T * 4);
            const int turn = (r >> 1) & 3;
#pragma unroll 1
            for (int c = dual ? 0 : 16 * h; c < D; c += dual ? 16 : 32) {
                float y[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) y[j] = 0.0f;
                if (!idle) {
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (dual && g != h) continue;
                        uint32_t o[16];
                        tc::tmem_ld_x16(trow + C::kColO + D * g + c, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            if (fo[g] != 0.0f) y[j] = __fmaf_rn(__uint_as_float(o[j]), fo[g], y[j]);
                            if (TWO && flushed[g] && ff[g] != 0.0f)
                                y[j] = __fmaf_rn(p.sums[((int64_t)(2 * blockIdx.x + g) * D + c + j) * T + r], ff[g], y[j]);
                        }
                    }
                }
                if (lg_parts == 0) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4) store4(c + j, make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]));
                } else {
                    float4* const meet = meet0 + (TWOBUF && (c & 32) ? 2 * T * 4 : 0);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        meet[4 * r + (j ^ turn)] = make_float4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
                    bar_sync(kBarMeet + h, 128);
                    // piece 2 part + i / 2 of copy i % 2, or piece part of copy i
                    float4 z[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int from = lr + (lg_parts == 1 ? (i & 1) * 64 : i * 32);
                        const int piece = lg_parts == 1 ? 2 * part + (i >> 1) : part;
                        z[i] = meet[4 * from + (piece ^ turn)];
                    }
                    auto add4 = [](float4 u, float4 v) { return make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w); };
                    const float4 lo = add4(z[0], z[1]), hi2 = add4(z[2], z[3]);
                    if (lg_parts == 1) {
                        store4(c + 8 * part, lo);
                        store4(c + 8 * part + 4, hi2);
                    } else {
                        store4(c + 4 * part, add4(lo, hi2));
                    }
                    if (!TWOBUF) bar_sync(kBarMeet + h, 128);   // read before it is written again
                }
            }
            if (!whole && live && part == 0 && (dual || h == 0)) {
                reinterpret_cast<float2*>(slot + (int64_t)RB * T * D)[row] = make_float2(l_all == l_all ? m_all : l_all, l_all);
            }
            tc::fence_before_sync();
            softmax_sync();                           // O, the query buffer and the exchanges have been read
            if (tid == 0) mbar_arrive(&sm.oread);
        }
    }

    // ---- release tensor memory once every MMA has completed ----
    if (warp == kMmaWarp) {
        if (!mbar_wait_sleep(&sm.mma_done, 0, 1u << 16)) report(p.status, NVFP4_ERR_TIMEOUT);
        __syncwarp();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kMmaWarp) tc::tmem_dealloc(tbase, kTmemCols);
}

// ---------------------------------------------------------------------------
// Merge of the units that ranges cut: block (c, y) takes rows y * R .. of the
// unit described by desc[c], whose contributors are range c - 1 (its last
// segment) and ranges c, c + 1, .. (their first).  A programmatic dependent of
// the attention grid.
// ---------------------------------------------------------------------------
constexpr int kMergeThreads = 256;

template <int D, int RB>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ Params p) {
    constexpr int kSlot = RB * T * (D + 2);
    constexpr int RPB = kMergeThreads / (D / 4);      // rows of a block
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 d = p.desc[blockIdx.x];
    const int parts = d.x & 0xFFFF, rows = d.x >> 16, gr0 = d.w * RB * T;
    const int row = blockIdx.y * RPB + threadIdx.x % RPB, col = 4 * (threadIdx.x / RPB);
    if (row >= rows) return;
    const int c0 = (int)blockIdx.x - 1;
    float M = -INFINITY, L = 0.0f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // four contributors' loads in flight, joined under a running maximum
#pragma unroll 1
    for (int j0 = 0; j0 < parts; j0 += 4) {
        float2 ml[4];
        float4 o[4];
        float Mn = M;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = min(j0 + k, parts - 1);
            const float* sp = p.partials + (int64_t)(2 * (c0 + j) + (j == 0 ? 1 : 0)) * kSlot;
            ml[k] = __ldcg(reinterpret_cast<const float2*>(sp + RB * T * D) + row);
            o[k] = __ldcg(reinterpret_cast<const float4*>(sp) + (col / 4) * (RB * T) + row);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) Mn = fmaxf(Mn, ml[k].x);
        const float f = M == -INFINITY ? 0.0f : fast_exp2(M - Mn);
        L *= f; acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
        M = Mn;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // a contributor that saw nothing left its O undefined; a NaN maximum stays one
            const float w = j0 + k >= parts || ml[k].x == -INFINITY ? 0.0f : fast_exp2(ml[k].x - M);
            if (w != 0.0f) {
                L = __fmaf_rn(ml[k].y, w, L);
                acc.x = __fmaf_rn(o[k].x, w, acc.x);
                acc.y = __fmaf_rn(o[k].y, w, acc.y);
                acc.z = __fmaf_rn(o[k].z, w, acc.z);
                acc.w = __fmaf_rn(o[k].w, w, acc.w);
            }
        }
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const int nd = (int)p.fd_g.div((uint32_t)(gr0 + row));
    const int64_t at =
        (((int64_t)d.y * p.N + nd) * p.Hq + (int64_t)d.z * p.g + (gr0 + row - nd * p.g)) * D + col;
    if (p.out_bf16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
        const __nv_bfloat162 b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + at) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
}

template <class C, bool TWO>
cudaError_t launch(const Params& p, int grid, cudaStream_t stream) {
    const int smem = (int)sizeof(Smem<C>) + 1024;
    static_assert(sizeof(Smem<C>) + 1024 <= 227 * 1024, "shared memory");
    static int configured[kMaxDevices] = {};
    cudaError_t e =
        ensure_smem_attribute(reinterpret_cast<const void*>(tree_attention_tc_kernel<C, TWO>), smem, configured);
    if (e != cudaSuccess) return e;
    tree_attention_tc_kernel<C, TWO><<<(unsigned)grid, C::kThreads, smem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int most_rows = (int)std::min<int64_t>((int64_t)p.N * p.g, C::RB * T);
    constexpr int kRows = kMergeThreads / (C::D / 4);
    cfg.gridDim = dim3((unsigned)grid, (unsigned)((most_rows + kRows - 1) / kRows));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_merge_kernel<C::D, C::RB>, p);
}

// row blocks of a unit: two when some sequence can have more than 128 rows
int row_blocks(int N, int g) { return (int64_t)N * g > T ? 2 : 1; }

size_t desc_bytes(size_t sms) { return (sms * sizeof(int4) + 255) / 256 * 256; }
size_t partial_bytes(size_t sms, int rb, int D) { return 2 * sms * (size_t)rb * T * (D + 2) * sizeof(float); }

}  // namespace

size_t tree_attention_workspace(int B, int N, int Hq, int Hkv, int D) {
    (void)B;
    const size_t sms = (size_t)device_sm_count();
    // units cut by the ranges, their partials, and the flushed sums of fp32 outputs
    return desc_bytes(sms) + partial_bytes(sms, row_blocks(N, Hq / Hkv), D) + 2 * sms * (size_t)T * D * sizeof(float);
}

cudaError_t launch_tree_attention(const TreeLaunch& a, cudaStream_t stream) {
    Params p = {};
    const int sms = device_sm_count();
    p.st_k = a.st_k; p.st_v = a.st_v;
    p.mask_stride = a.mask_stride;
    const int rb = row_blocks(a.N, a.Hq / a.Hkv);
    uint8_t* const ws = reinterpret_cast<uint8_t*>(a.partials);
    p.desc = reinterpret_cast<int4*>(ws);
    p.partials = reinterpret_cast<float*>(ws + desc_bytes(sms));
    p.sums = reinterpret_cast<float*>(ws + desc_bytes(sms) + partial_bytes(sms, rb, a.D));
    p.status = a.status;
    p.N = a.N; p.Hq = a.Hq; p.Hkv = a.Hkv; p.g = a.Hq / a.Hkv; p.S_max = a.S_max;
    p.W = (a.N + 31) / 32;
    p.page_tokens = a.page_tokens; p.max_pages = a.max_pages; p.num_pages = a.num_pages;
    p.out_bf16 = a.out_bf16 ? 1 : 0;
    const float scale = a.softmax_scale > 0.0f ? a.softmax_scale : 1.0f / sqrtf((float)a.D);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.wait_polls = a.wait_polls;
    p.fd_g = FastDiv((uint32_t)p.g);
    for (int b0 = 0; b0 < a.B; b0 += kMaxBatchPerLaunch) {
        p.B = a.B - b0 < kMaxBatchPerLaunch ? a.B - b0 : kMaxBatchPerLaunch;
        p.q = reinterpret_cast<const uint16_t*>(a.q) + (int64_t)b0 * a.N * a.Hq * a.D;
        p.out = static_cast<uint8_t*>(a.out) + (int64_t)b0 * a.N * a.Hq * a.D * (a.out_bf16 ? 2 : 4);
        const int64_t seq = a.block_table != nullptr ? 0 : (int64_t)b0 * a.Hkv * a.S_max;
        p.kc = a.kc + seq * (a.D / 2); p.ks = a.ks + seq * (a.D / 16);
        p.vc = a.vc + seq * (a.D / 2); p.vs = a.vs + seq * (a.D / 16);
        p.block_table = a.block_table != nullptr ? a.block_table + (int64_t)b0 * a.max_pages : nullptr;
        p.start = a.start + b0;
        p.n_nodes = a.n_nodes != nullptr ? a.n_nodes + b0 : nullptr;
        p.mask = a.mask != nullptr ? a.mask + (int64_t)b0 * a.mask_stride : nullptr;
        // no more CTAs than tiles there can be
        const int64_t units = (int64_t)p.B * a.Hkv * (((int64_t)a.N * p.g + rb * T - 1) / (rb * T));
        const int64_t most = units * ((a.S_max + T - 1) / T);
        const int grid = (int)(most < sms ? most : sms);
        cudaError_t e;
        if (a.D == 128)
            e = rb == 2 ? (a.out_bf16 ? launch<Cfg<128, 2>, false>(p, grid, stream) : launch<Cfg<128, 2>, true>(p, grid, stream))
                        : (a.out_bf16 ? launch<Cfg<128, 1>, false>(p, grid, stream) : launch<Cfg<128, 1>, true>(p, grid, stream));
        else
            e = rb == 2 ? (a.out_bf16 ? launch<Cfg<64, 2>, false>(p, grid, stream) : launch<Cfg<64, 2>, true>(p, grid, stream))
                        : (a.out_bf16 ? launch<Cfg<64, 1>, false>(p, grid, stream) : launch<Cfg<64, 1>, true>(p, grid, stream));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace nvfp4kv
