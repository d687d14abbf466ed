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
// Warp roles:
//   warps 0-7    softmax: thread (h, r) owns tokens 64h .. 64h + 63 of score
//                row r of a tile; the two halves exchange their maxima through shared
//                memory (one 64-thread barrier per tile)
//   warps 8-15   dequant: thread t of the first four warps owns token t's keys, of
//                the others its values
//   warp 16      bulk copies of raw codes and scales into the ring
//   warp 17      MMA issue (one elected lane)
//   warp 18      describes the unit this range cuts to the merge kernel
// P overwrites S in tensor memory, as the A operand of P . V: it takes no
// shared memory.  S(i + 1) is issued before O += P(i) . V, so the scores of
// the next item are ready when the softmax finishes one.
#include <cuda_bf16.h>

#include "nvfp4kv_device.cuh"
#include "nvfp4kv_internal.h"
#include "nvfp4kv_pipeline.cuh"
#include "nvfp4kv_tcgen05.cuh"

namespace nvfp4kv {

namespace {

constexpr int T = 128;                                // tokens per tile, rows per row block
constexpr int kThreads = 20 * 32;
constexpr int kDqWarp0 = 8, kLoadWarp = 16, kMmaWarp = 17, kDescWarp = 18;
// registers after the prologue: 256 x 136 + 256 x 72 + 128 x 64 = 61,440 = 640 x 96
constexpr uint32_t kRegsSoftmax = 136, kRegsDequant = 72, kRegsMisc = 64;
constexpr uint32_t kTmemCols = 512;
// O is rescaled only when a row's running max grows by more than 2^kSlack;
// P = 2^(s - m + kBias) <= 2^14 stays inside f16, and weights down to 2^-30
// of the row's largest keep a bit of it
constexpr float kSlack = 8.0f, kBias = 6.0f;
constexpr int kLutCopies = 2;
// fp32 outputs: the tensor core truncates its accumulator at every 16-token
// step, a bias that grows with the context (1.6e-5 of the output at 128K
// tokens); after this many tiles O is added, with rounding, to a second accumulator
constexpr int kFlush = 8;

struct Params {
    const void* q;                                    // [B][N][Hq][D] bf16
    const uint8_t *kc, *ks, *vc, *vs;
    const float *st_k, *st_v;
    const int32_t *start, *n_nodes, *mask, *block_table;
    int64_t mask_stride;
    void* out;                                        // [B][N][Hq][D]
    float* partials;                                  // [2 * grid] slots
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
    static constexpr int kCB = D / 2, kSB = D / 16;   // code / scale bytes per token
    static constexpr int kStage = T * (2 * kCB + 2 * kSB);
    static constexpr int kOffVC = T * kCB, kOffKS = 2 * T * kCB, kOffVS = 2 * T * kCB + T * kSB;
    static constexpr int kRing = RB == 2 && D == 128 ? 1 : 3;
    static constexpr int kTileBytes = T * D * 2;
    static constexpr uint32_t kColO = 0, kColS = RB * D;
    static constexpr uint32_t kColM = kColS + 2 * T;  // fp32 outputs (RB = 1): the sum of flushed O
    static constexpr int kSlot = RB * T * (D + 2);    // floats of a partial: O, m, l
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
    float mx[2][2][T];                                // row maxima (and sums) of the two halves
    int32_t prefix[kMaxBatchPerLaunch + 1];
    int32_t warp_tot[16];
    uint64_t full[C::kRing], empty[C::kRing];
    uint64_t kready[2], kfree[2], vready[2], vfree[2], sready[2], pready[2];
    uint64_t qready, oread, mma_done;
    uint32_t tmem_base;
    int32_t abort_flag;
};

__device__ __forceinline__ void tmem_ld64(uint32_t addr, uint32_t (&v)[64]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) tc::tmem_ld_x16(addr + 16 * c, v + 16 * c);
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

// Eight kind::f16 MMAs over 128 tokens with A = P in tensor memory: tokens
// 0-63 in columns a .. a + 31, tokens 64-127 in a + 64 .. a + 95.
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
#define NVFP4_TS_STEP(INC) "add.u32 %1, %1, " INC ";\n\tadd.s64 %2, %2, 16;\n\t" \
                           "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p1;\n\t"
    asm volatile("{\n\t.reg .pred p0, p1;\n\tsetp.ne.b32 p0, %4, 0;\n\tsetp.eq.b32 p1, %4, %4;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p0;\n\t"
                 NVFP4_TS_STEP("8") NVFP4_TS_STEP("8") NVFP4_TS_STEP("8") NVFP4_TS_STEP("40")
                 NVFP4_TS_STEP("8") NVFP4_TS_STEP("8") NVFP4_TS_STEP("8") "}"
                 : "+r"(d), "+r"(a), "+l"(b) : "r"(idesc), "r"(acc) : "memory");
#undef NVFP4_TS_STEP
}

template <uint32_t N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Barrier of the two warps that share 32 rows; true when both pass true.  They
// meet once per item whatever their waits gave, so that neither is left alone.
__device__ __forceinline__ bool pair_and(int id, bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\t"
        "barrier.cta.red.and.aligned.pred b, %2, 64, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r)
        : "r"(ok ? 1u : 0u), "r"(id)
        : "memory");
    return r != 0;
}

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
__global__ void __launch_bounds__(kThreads, 1) tree_attention_tc_kernel(const __grid_constant__ Params p) {
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
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 256);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.kready[s], 128);
            mbar_init(&sm.kfree[s], 1);
            mbar_init(&sm.vready[s], 128);
            mbar_init(&sm.vfree[s], 1);
            mbar_init(&sm.sready[s], 1);
            mbar_init(&sm.pready[s], 256);
        }
        mbar_init(&sm.qready, 256);
        mbar_init(&sm.oread, 256);
        mbar_init(&sm.mma_done, 1);
        fence_mbar_init();
        sm.abort_flag = 0;
    }
    const float st_k = *p.st_k, st_v = *p.st_v;
    if (tid < 256) {
        const int plane = tid >> 7;
        const uint2 w = lut_words((uint32_t)(tid & 127), plane ? st_v : st_k);
#pragma unroll
        for (int c = 0; c < kLutCopies; ++c) sm.lut[plane][tid & 127][c] = w;
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

    if (warp >= kLoadWarp) {
        regs_dec<kRegsMisc>();
        if (warp == kLoadWarp && lane == 0) {
            // ================= bulk copies, one stage per tile =================
            uint32_t n = 0;                           // tiles issued
            bool ok = true;
            Walker<C> w(lo, hi);
            Segment s;
            while (ok && w.next(p, sm.prefix, s)) {
                for (int k = 0; k < s.tiles; ++k, ++n) {
                    const int st = n % C::kRing;
                    if (n >= C::kRing && !wait_one(&sm.empty[st], (n / C::kRing - 1) & 1, abort_flag, p.status, polls)) {
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
                    mbar_arrive_expect_tx(&sm.full[st], 2 * (cb + sb));
                    uint8_t* dst = sm.ring[st];
                    bulk_g2s(dst, p.kc + tok * C::kCB, cb, &sm.full[st]);
                    bulk_g2s(dst + C::kOffKS, p.ks + tok * C::kSB, sb, &sm.full[st]);
                    bulk_g2s(dst + C::kOffVC, p.vc + tok * C::kCB, cb, &sm.full[st]);
                    bulk_g2s(dst + C::kOffVS, p.vs + tok * C::kSB, sb, &sm.full[st]);
                }
            }
            // every issued copy lands before the CTA exits
            for (uint32_t i = n > C::kRing ? n - C::kRing : 0; i < n; ++i)
                if (!mbar_wait_sleep(&sm.full[i % C::kRing], (i / C::kRing) & 1, 1u << 16)) {
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
            while (ok && w.next(p, sm.prefix, s)) {
                const int nrb = RB == 2 && s.rows > T ? 2 : 1;
                const int items = s.tiles * nrb;
                ok = wait_warp(&sm.qready, seg & 1, abort_flag, p.status, polls);
                // S(i) = Q . K^T into buffer (gi + i) % 2
                auto issue_qk = [&](int i) -> bool {
                    const int tile = RB == 2 && nrb == 2 ? i >> 1 : i, rb = RB == 2 && nrb == 2 ? i & 1 : 0;
                    const uint32_t kt = gt + tile, kb = kt & 1;
                    if (rb == 0 && !wait_warp(&sm.kready[kb], (kt >> 1) & 1, abort_flag, p.status, polls)) return false;
                    tc::fence_after_sync();
                    if (tc::elect_one()) {
                        mma_ss<D / 16>(tbase + C::kColS + T * ((gi + i) & 1),
                                       tc::smem_desc(tc::smem_addr(sm.q[rb]), 128, 16 * D),
                                       tc::smem_desc(tc::smem_addr(sm.k[kb]), 128, 16 * D), idesc_qk);
                        tc::mma_commit(&sm.sready[(gi + i) & 1]);
                        if (rb == nrb - 1) tc::mma_commit(&sm.kfree[kb]);
                    }
                    __syncwarp();
                    return true;
                };
                if (ok) ok = issue_qk(0);
                for (int i = 0; ok && i < items; ++i) {
                    if (i + 1 < items && !issue_qk(i + 1)) {
                        ok = false;
                        break;
                    }
                    const int tile = RB == 2 && nrb == 2 ? i >> 1 : i, rb = RB == 2 && nrb == 2 ? i & 1 : 0;
                    const uint32_t x = gi + i, vt = gt + tile, vb = vt & 1;
                    if (!wait_warp(&sm.pready[x & 1], (x >> 1) & 1, abort_flag, p.status, polls) ||
                        (rb == 0 && !wait_warp(&sm.vready[vb], (vt >> 1) & 1, abort_flag, p.status, polls)) ||
                        // the previous segment's O has been read
                        (i == 0 && seg > 0 && !wait_warp(&sm.oread, (seg - 1) & 1, abort_flag, p.status, polls))) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    if (tc::elect_one()) {
                        const uint64_t dv = tc::smem_desc(tc::smem_addr(sm.v[vb]), 128, 2048);
                        const uint32_t a = tbase + C::kColS + T * (x & 1), o = tbase + C::kColO + D * rb;
                        mma_pv(o, a, dv, idesc_pv, (TWO ? tile % kFlush : tile) > 0 ? 1u : 0u);
                        if (TWO) mma_pv(o, a + 32, dv, idesc_pv, 1u);
                        if (rb == nrb - 1) tc::mma_commit(&sm.vfree[vb]);
                    }
                    __syncwarp();
                }
                gi += items;
                gt += s.tiles;
                ++seg;
            }
            if (tc::elect_one()) tc::mma_commit(&sm.mma_done);
            __syncwarp();
        } else if (warp == kDescWarp && lane == 0) {
            // ================= the unit that this range's start cuts first =================
            // is merged by block blockIdx.x: contributors, sequence, KV head, row unit
            int4 d = make_int4(0, 0, 0, 0);
            Walker<C> w(lo, hi);
            Segment s;
            if (w.next(p, sm.prefix, s) && s.tile0 > 0 && lo - s.tile0 >= range_start((int)blockIdx.x - 1)) {
                int c = (int)blockIdx.x + 1;          // ranges blockIdx.x - 1 .. c - 1 hold tiles of it
                while (c < nr && range_start(c) < lo - s.tile0 + s.unit_tiles) ++c;
                d = make_int4(c - (int)blockIdx.x + 1, s.b, s.hk, s.ru);
            }
            p.desc[blockIdx.x] = d;
        }
    } else if (warp >= kDqWarp0) {
        // ================= dequant: token t of each tile, keys or values =================
        regs_dec<kRegsDequant>();
        const int which = (warp - kDqWarp0) >> 2;     // 0: keys, 1: values
        const int t = tid & (T - 1);
        const uint2* lut = &sm.lut[which][0][lane & (kLutCopies - 1)];
        uint64_t* const ready = which ? sm.vready : sm.kready;
        uint64_t* const free_ = which ? sm.vfree : sm.kfree;
        uint32_t n = 0;
        constexpr int NCH = D / 32;                   // 16-byte code chunks of a token
        const uint32_t ntiles = (uint32_t)(hi - lo);  // every tile of the range once, in order
        for (; n < ntiles; ++n) {
            const int st = n % C::kRing;
            if (!wait_warp(&sm.full[st], (n / C::kRing) & 1, abort_flag, p.status, polls)) break;
            const uint8_t* raw = sm.ring[st] + (which ? C::kOffVC : 0) + t * C::kCB;
            // chunk order rotated per thread: eight lanes read eight different 16-byte banks
            uint4 code[NCH];
            const int rot = D == 128 ? (t >> 1) : (t >> 2);
#pragma unroll
            for (int j = 0; j < NCH; ++j)
                code[j] = *reinterpret_cast<const uint4*>(raw + 16 * ((j + rot) & (NCH - 1)));
            uint32_t sb[2];
            const uint8_t* sraw = sm.ring[st] + (which ? C::kOffVS : C::kOffKS) + t * C::kSB;
            if (D == 128) {
                const uint2 u = *reinterpret_cast<const uint2*>(sraw);
                sb[0] = u.x;
                sb[1] = u.y;
            } else {
                sb[0] = sb[1] = *reinterpret_cast<const uint32_t*>(sraw);
            }
            fence_proxy_async_smem();                 // the next copy into this stage comes after these reads
            mbar_arrive(&sm.empty[st]);
            const uint32_t buf = n & 1;
            if (n >= 2 && !wait_warp(&free_[buf], ((n >> 1) - 1) & 1, abort_flag, p.status, polls)) break;
            uint8_t* dst = which ? sm.v[buf] + (t / 8) * 128 + (t % 8) * 16 : sm.k[buf] + (t / 8) * (16 * D) + (t % 8) * 16;
            const int step = which ? 2048 : 128;      // between 8-element groups of the head dimension
#pragma unroll
            for (int j = 0; j < NCH; ++j) {
                const int c = (j + rot) & (NCH - 1);
                const uint32_t two = (D == 128 && (c & 2) ? sb[1] : sb[0]) >> (16 * (c & 1));
                const uint2 la = lut[(two & 0x7F) * kLutCopies];
                const uint2 lb = lut[((two >> 8) & 0x7F) * kLutCopies];
                uint8_t* d8 = dst + 4 * c * step;
                *reinterpret_cast<uint4*>(d8) = dequant8(code[j].x, la);
                *reinterpret_cast<uint4*>(d8 + step) = dequant8(code[j].y, la);
                *reinterpret_cast<uint4*>(d8 + 2 * step) = dequant8(code[j].z, lb);
                *reinterpret_cast<uint4*>(d8 + 3 * step) = dequant8(code[j].w, lb);
            }
            fence_proxy_async_smem();
            mbar_arrive(&ready[buf]);
        }
    } else {
        // ================= softmax: tokens 64h .. 64h + 63 of row r =================
        regs_inc<kRegsSoftmax>();
        const int h = warp >> 2, r = tid & (T - 1);
        const uint32_t trow = tbase + ((uint32_t)(32 * (warp & 3)) << 16);
        const int bar = 1 + (warp & 3);
        constexpr int DH = D / 2;                     // columns of O this thread rescales and stores
        uint32_t gi = 0, gt = 0;
        bool ok = true;
        Walker<C> w(lo, hi);
        Segment s;
        while (ok && w.next(p, sm.prefix, s)) {
            const int nrb = RB == 2 && s.rows > T ? 2 : 1;
            float cs[RB], m_run[RB], l_run[RB];
            int node[RB];
            // query operand: q * 2^e rounded to f16, e from the row's amax
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                m_run[rb] = -INFINITY;
                l_run[rb] = 0.0f;
                cs[rb] = 0.0f;
                node[rb] = 0;
                if (rb >= nrb) continue;
                const int row = rb * T + r;
                const bool live = row < s.rows;
                const int gr = s.ru * RB * T + row;
                const int nd = live ? (int)p.fd_g.div((uint32_t)gr) : 0;
                node[rb] = nd;
                const uint4* src = reinterpret_cast<const uint4*>(
                    reinterpret_cast<const uint16_t*>(p.q) +
                    (((int64_t)s.b * p.N + nd) * p.Hq + (int64_t)s.hk * p.g + (gr - nd * p.g)) * D);
                uint32_t amax = 0;
                if (live)
                    for (int c = 0; c < D / 8; ++c) {
                        const uint4 u = __ldg(src + c);
                        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            amax = max(amax, max((x[j] & 0x7FFFu) << 16, x[j] & 0x7FFF0000u));
                    }
                int e = 0;
                if (amax > 0u && amax < 0x7F800000u) {
                    int ex;
                    frexpf(__uint_as_float(amax), &ex);
                    e = 15 - ex;
                    e = e < -126 ? -126 : (e > 126 ? 126 : e);
                }
                const float up = __uint_as_float((uint32_t)(127 + e) << 23);
                uint8_t* qd = sm.q[rb] + (r / 8) * (16 * D) + (r % 8) * 16;
                for (int c = h * (D / 16); c < (h + 1) * (D / 16); ++c) {
                    uint4 u = live ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
                    uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[j] = pack_f16x2(__uint_as_float(x[j] << 16) * up, __uint_as_float(x[j] & 0xFFFF0000u) * up);
                    *reinterpret_cast<uint4*>(qd + c * 128) = make_uint4(x[0], x[1], x[2], x[3]);
                }
                cs[rb] = fmaxf(p.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23), 1.17549435e-38f);
            }
            fence_proxy_async_smem();
            mbar_arrive(&sm.qready);

            for (int k = 0; ok && k < s.tiles; ++k) {
                const int t0 = (s.tile0 + k) * T;
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) {
                    if (rb >= nrb) break;
                    const uint32_t sb = gi & 1;
                    ok = ok && wait_warp(&sm.sready[sb], (gi >> 1) & 1, abort_flag, p.status, polls);
                    tc::fence_after_sync();
                    // a warp without live rows leaves P as it is: it only reaches its own rows of O
                    if (rb * T + 32 * (warp & 3) >= s.rows) {
                        if (!ok) break;
                    } else {
                        uint32_t v[64];
                        const uint32_t scol = trow + C::kColS + T * sb + 64 * h;
                        tmem_ld64(scol, v);
                        tc::tmem_wait_ld();
                        if (t0 + T > s.start) {
                            const uint64_t vis = visible64(p, s, node[rb], t0 + 64 * h);
#pragma unroll
                            for (int j = 0; j < 64; ++j)
                                if (!((vis >> j) & 1)) v[j] = 0xFF800000u;
                        }
                        float mt = __uint_as_float(v[0]);
#pragma unroll
                        for (int j = 1; j < 64; ++j) mt = fmaxf(mt, __uint_as_float(v[j]));
                        mt *= cs[rb];
                        sm.mx[sb][h][r] = mt;
                        ok = pair_and(bar, ok);
                        if (!ok) break;
                        mt = fmaxf(mt, sm.mx[sb][h ^ 1][r]);
                        float m_new = m_run[rb];
                        if (mt > m_new + kSlack || m_new == -INFINITY) m_new = fmaxf(m_new, mt);
                        float f = 1.0f;
                        if (m_new != m_run[rb]) {
                            f = m_run[rb] == -INFINITY ? 0.0f : fast_exp2(m_run[rb] - m_new);
                            l_run[rb] *= f;
                            m_run[rb] = m_new;
                        }
                        // tcgen05.ld/st are warp-wide: the warp rescales when any of its rows must
                        const bool flush = TWO && k > 0 && k % kFlush == 0;
                        if (k > 0 && (flush || __any_sync(0xFFFFFFFFu, f != 1.0f))) {
                            // P . V of this row block's previous tile has ended (with two row
                            // blocks it was issued before this S, so it has)
                            const uint32_t pt = gt + k - 1;
                            if (nrb == 1) ok = wait_warp(&sm.vfree[pt & 1], (pt >> 1) & 1, abort_flag, p.status, polls);
                            tc::fence_after_sync();
#pragma unroll 1
                            for (int c = 0; c < DH / 16; ++c) {
                                uint32_t o[16];
                                const uint32_t col = DH * h + 16 * c;
                                const uint32_t oc = trow + C::kColO + D * rb + col, mc = trow + C::kColM + col;
                                tc::tmem_ld_x16(oc, o);
                                tc::tmem_wait_ld();
                                if (TWO && k > kFlush) {
                                    uint32_t m[16];
                                    tc::tmem_ld_x16(mc, m);
                                    tc::tmem_wait_ld();
#pragma unroll
                                    for (int j = 0; j < 16; ++j)
                                        m[j] = __float_as_uint(
                                            (__uint_as_float(m[j]) + (flush ? __uint_as_float(o[j]) : 0.0f)) * f);
                                    tc::tmem_st_x8(mc, m);
                                    tc::tmem_st_x8(mc + 8, m + 8);
                                }
#pragma unroll
                                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                if (!flush) {
                                    tc::tmem_st_x8(oc, o);
                                    tc::tmem_st_x8(oc + 8, o + 8);
                                } else if (k == kFlush) {
                                    tc::tmem_st_x8(mc, o);
                                    tc::tmem_st_x8(mc + 8, o + 8);
                                }
                            }
                        }
                        const float base = (m_run[rb] == -INFINITY ? 0.0f : m_run[rb]) - kBias;
                        uint32_t ph[32];
                        float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float a = fast_exp2(__fmaf_rn(__uint_as_float(v[2 * j]), cs[rb], -base));
                            const float b = fast_exp2(__fmaf_rn(__uint_as_float(v[2 * j + 1]), cs[rb], -base));
                            sum0 += a;
                            sum1 += b;
                            ph[j] = pack_f16x2(a, b);
                            if (TWO) v[j] = pack_f16x2(a - f16_lo_to_float(ph[j]), b - f16_hi_to_float(ph[j]));
                        }
                        l_run[rb] += sum0 + sum1;
                        tc::tmem_st_x32(scol, ph);
                        if (TWO) {
                            uint32_t pl[32];
#pragma unroll
                            for (int j = 0; j < 32; ++j) pl[j] = v[j];
                            tc::tmem_st_x32(scol + 32, pl);
                        }
                        tc::tmem_wait_st();
                    }
                    tc::fence_before_sync();
                    mbar_arrive(&sm.pready[sb]);
                    ++gi;
                }
            }
            gt += s.tiles;
            // ---- the segment's O: the output when it is a whole unit, else a partial ----
            const uint32_t last = gt - 1;
            ok = ok && wait_warp(&sm.vfree[last & 1], (last >> 1) & 1, abort_flag, p.status, polls);
            if (32 * (warp & 3) < s.rows) ok = pair_and(bar, ok);
            if (!ok) break;
            tc::fence_after_sync();
            const bool whole = s.tiles == s.unit_tiles;
            float* const slot = p.partials + (int64_t)(2 * blockIdx.x + (s.tile0 > 0 ? 0 : 1)) * C::kSlot;
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                if (rb >= nrb || rb * T + 32 * (warp & 3) >= s.rows) continue;
                const int row = rb * T + r;
                const bool live = row < s.rows;
                sm.mx[rb][h][r] = l_run[rb];
                pair_and(bar, true);
                const float l = l_run[rb] + sm.mx[rb][h ^ 1][r];
                pair_and(bar, true);                  // the exchange is read before the next one writes
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                const int gr = s.ru * RB * T + row;
                const int64_t orow =
                    (((int64_t)s.b * p.N + node[rb]) * p.Hq + (int64_t)s.hk * p.g + (gr - node[rb] * p.g)) * D + DH * h;
#pragma unroll 1
                for (int c = 0; c < DH / 16; ++c) {
                    uint32_t o[16];
                    tc::tmem_ld_x16(trow + C::kColO + D * rb + DH * h + 16 * c, o);
                    tc::tmem_wait_ld();
                    if (TWO && s.tiles > kFlush) {
                        uint32_t m[16];
                        tc::tmem_ld_x16(trow + C::kColM + DH * h + 16 * c, m);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            o[j] = __float_as_uint(__uint_as_float(o[j]) + __uint_as_float(m[j]));
                    }
                    if (!live) continue;
                    if (!whole) {
                        float4* dst = reinterpret_cast<float4*>(slot + (int64_t)row * D + DH * h + 16 * c);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            dst[j] = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                                 __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
                    } else if (TWO) {
                        float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + orow + 16 * c);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            dst[j] = make_float4(__uint_as_float(o[4 * j]) * inv, __uint_as_float(o[4 * j + 1]) * inv,
                                                 __uint_as_float(o[4 * j + 2]) * inv, __uint_as_float(o[4 * j + 3]) * inv);
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.out) + orow + 16 * c);
                        uint32_t x[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(o[2 * j]) * inv,
                                                                           __uint_as_float(o[2 * j + 1]) * inv);
                            x[j] = *reinterpret_cast<const uint32_t*>(&y);
                        }
                        dst[0] = make_uint4(x[0], x[1], x[2], x[3]);
                        dst[1] = make_uint4(x[4], x[5], x[6], x[7]);
                    }
                }
                if (!whole && live && h == 0) {
                    slot[(int64_t)RB * T * D + row] = m_run[rb];
                    slot[(int64_t)RB * T * (D + 1) + row] = l;
                }
            }
            tc::fence_before_sync();
            mbar_arrive(&sm.oread);
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
    if (d.x == 0) return;
    int err;
    const int nodes = live_nodes(p, d.y, p.start[d.y], err);
    const int gr0 = d.w * RB * T;
    const int row = blockIdx.y * RPB + threadIdx.x / (D / 4), col = 4 * (threadIdx.x % (D / 4));
    if (row >= min(RB * T, nodes * p.g - gr0)) return;
    const int c0 = (int)blockIdx.x - 1;
    auto slot = [&](int j) -> const float* { return p.partials + (int64_t)(2 * (c0 + j) + (j == 0 ? 1 : 0)) * kSlot; };
    float M = -INFINITY;
    for (int j = 0; j < d.x; ++j) M = fmaxf(M, __ldcg(slot(j) + RB * T * D + row));
    float L = 0.0f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int j = 0; j < d.x; ++j) {
        const float* sp = slot(j);
        const float m = __ldcg(sp + RB * T * D + row);
        const float w = m == -INFINITY ? 0.0f : fast_exp2(m - M);
        const float l = __ldcg(sp + RB * T * (D + 1) + row);
        const float4 o = __ldcg(reinterpret_cast<const float4*>(sp + (int64_t)row * D + col));
        if (w > 0.0f) {                               // a contributor that saw nothing left its O undefined
            L = __fmaf_rn(l, w, L);
            acc.x = __fmaf_rn(o.x, w, acc.x);
            acc.y = __fmaf_rn(o.y, w, acc.y);
            acc.z = __fmaf_rn(o.z, w, acc.z);
            acc.w = __fmaf_rn(o.w, w, acc.w);
        }
    }
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
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
    tree_attention_tc_kernel<C, TWO><<<(unsigned)grid, kThreads, smem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, (unsigned)(C::RB * T / (kMergeThreads / (C::D / 4))));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_merge_kernel<C::D, C::RB>, p);
}

// Row blocks of a unit: two when some sequence can have more than 128 rows and
// the output is bf16 (with fp32 outputs the second accumulator takes the tensor
// memory of the second row block).
int row_blocks(int N, int g, bool out_bf16) { return out_bf16 && (int64_t)N * g > T ? 2 : 1; }

}  // namespace

size_t tree_attention_workspace(int B, int N, int Hq, int Hkv, int D) {
    (void)B;
    const size_t sms = (size_t)device_sm_count();
    const size_t slot = (size_t)row_blocks(N, Hq / Hkv, true) * T * (D + 2) * sizeof(float);
    return ((sms * sizeof(int4) + 255) / 256 * 256) + 2 * sms * slot;
}

cudaError_t launch_tree_attention(const TreeLaunch& a, cudaStream_t stream) {
    Params p = {};
    const int sms = device_sm_count();
    p.st_k = a.st_k; p.st_v = a.st_v;
    p.mask_stride = a.mask_stride;
    p.desc = reinterpret_cast<int4*>(a.partials);
    p.partials = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.partials) +
                                          (((size_t)sms * sizeof(int4) + 255) / 256 * 256));
    p.status = a.status;
    p.N = a.N; p.Hq = a.Hq; p.Hkv = a.Hkv; p.g = a.Hq / a.Hkv; p.S_max = a.S_max;
    p.W = (a.N + 31) / 32;
    p.page_tokens = a.page_tokens; p.max_pages = a.max_pages; p.num_pages = a.num_pages;
    p.out_bf16 = a.out_bf16 ? 1 : 0;
    const float scale = a.softmax_scale > 0.0f ? a.softmax_scale : 1.0f / sqrtf((float)a.D);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.wait_polls = a.wait_polls;
    p.fd_g = FastDiv((uint32_t)p.g);
    const int rb = row_blocks(a.N, p.g, a.out_bf16);
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
            e = !a.out_bf16 ? launch<Cfg<128, 1>, true>(p, grid, stream)
                            : (rb == 2 ? launch<Cfg<128, 2>, false>(p, grid, stream) : launch<Cfg<128, 1>, false>(p, grid, stream));
        else
            e = !a.out_bf16 ? launch<Cfg<64, 1>, true>(p, grid, stream)
                            : (rb == 2 ? launch<Cfg<64, 2>, false>(p, grid, stream) : launch<Cfg<64, 1>, false>(p, grid, stream));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace nvfp4kv
