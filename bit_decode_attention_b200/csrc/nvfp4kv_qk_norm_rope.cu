// nvfp4kv_qk_norm_rope.cu -- what stands between a layer's Q/K/V projection
// and attention over the NVFP4 cache, in one pass: RMS norm of each query and
// key head, rotary position embedding, and the quantize-append of K and V.
//
//   y = x * r * w,  r = 1 / sqrt(mean(x^2) + eps)            (queries, keys)
//   (y_i, y_j) -> (y_i c - y_j s, y_j c + y_i s)             c, s of the token's position
//   q_out = y rounded once; K and V blocks -> E2M1 codes and E4M3 scales
//
// Every step is one fp32 rounding; the keys are quantized from their fp32
// values.  A head's row is held by D / 16 lanes, each with 8 elements of the
// rotated part's first half and the 8 elements R / 2 further on (or, behind the
// rotated part, with 16 neighbours): the rotation's pairs (i, i + R/2) and
// (2i, 2i + 1) then sit in one lane, and a 16-element block in one or two
// neighbours (one shuffle for its amax).  A warp keeps one token's cos and sin
// in registers and walks the token's heads, the next row's loads in flight.
// Where R / 16 is odd a block would straddle the halves, and the pairs are
// exchanged by shuffles instead (R = 64 that way: 53 us for 31 below).
//
// Measured (B200, bf16, head_dim 128): 2,048 tokens of 96 + 2 x 8 heads 28.4 us,
// 3.9 TB/s of the 112 MB it has to move (17 us at 6.55 TB/s); the instructions
// take as long (two elements each in the norm and the rotation, one at a time:
// 37 us).  8 tokens of 32 + 2 x 8 heads: 4.4 us, launch and memory latency.
// Blocks an SM for bf16: 6 without spills 30.6 us and 20.6 for 4 x 512 tokens, 7
// with up to 32 bytes of them 28.4 and 16.7, 8 31.0 and 18.2.  fp32: 41 us for 34.
#include <cuda_bf16.h>

#include "nvfp4kv_device.cuh"
#include "nvfp4kv_internal.h"

namespace nvfp4kv {

namespace {

constexpr int kThreads = 128;

enum RotKind { kRotNone = 0, kRotHalf = 1, kRotInterleaved = 2, kRotHalfPartial = 3 };

// resident blocks of an SM, which the registers are cut for
__host__ __device__ constexpr int blocks_per_sm(bool f32, int rot) { return rot == kRotHalfPartial ? 4 : (f32 ? 5 : 7); }

struct NormRopeParams {
    const void *xq, *xk, *xv;
    int64_t sq, sk, sv;                               // elements between tokens
    const void *wq, *wk;                              // [D] or nullptr
    const float* table;                               // [P][R]: R/2 cos, R/2 sin
    const int32_t* positions;                         // [B][n] or nullptr
    const int32_t* start;
    const int32_t* n_valid;                           // [B] or nullptr
    int32_t* new_lens;
    const float *st_k, *st_v;
    void* q_out;                                      // [B][n][Hq][D]
    uint8_t *kc, *ks, *vc, *vs;
    const int32_t* block_table;
    int32_t* status;
    int32_t B, n, Hq, Hkv, S_max, R, P;
    int32_t page_tokens, max_pages, num_pages;
    float eps;                                        // negative: no norm
    int32_t heads_per_task, tasks_per_token;
    uint32_t tasks;
    FastDiv fd_tasks, fd_n;
};

// 8 codes (one 32-bit word) and the scale byte of a 16-element block whose
// other 8 elements the neighbouring lane holds: the arithmetic of
// quantize_block, to be kept like it (a test compares the bytes of the two
// appends).  amax, nan: over the whole block.
__device__ __forceinline__ uint32_t quantize_half(const float (&v)[8], float amax, bool nan, float st, uint32_t& sb) {
    const float r = __fdiv_rn(amax, __fmul_rn(6.0f, st));
    sb = e4m3_from_float(r);
    const float den = __fmul_rn(e4m3_to_float(sb), st);
    uint32_t word = 0;
    if (!nan && r <= 448.0f && den >= kCorrectionMinDivisor && den <= kCorrectionMaxDivisor) {
        const float y = __frcp_rn(den);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            word |= e2m1x2_from_floats(copysignf(div_rn_by_correction(v[2 * k], den, y), v[2 * k]),
                                       copysignf(div_rn_by_correction(v[2 * k + 1], den, y), v[2 * k + 1]))
                    << (8 * k);
    } else if (den == 0.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) word |= ((__float_as_uint(v[i]) >> 28) & 0x8u) << (4 * i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) word |= e2m1_from_float(__fdiv_rn(v[i], den)) << (4 * i);
    }
    return word;
}

// eight elements as they lie in memory
template <bool F32>
struct Raw { uint4 w[F32 ? 2 : 1]; };
template <bool F32>
__device__ __forceinline__ Raw<F32> fetch8(const void* base, int64_t i) {
    Raw<F32> r;
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + i * (F32 ? 4 : 2));
    r.w[0] = __ldg(p);
    if (F32) r.w[F32 ? 1 : 0] = __ldg(p + 1);
    return r;
}
template <bool F32>
__device__ __forceinline__ void unpack8(const Raw<F32>& r, float (&v)[8]) {
    if (F32) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint4 u = r.w[F32 ? j : 0];
            v[4 * j] = __uint_as_float(u.x); v[4 * j + 1] = __uint_as_float(u.y);
            v[4 * j + 2] = __uint_as_float(u.z); v[4 * j + 3] = __uint_as_float(u.w);
        }
    } else {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
}

template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t i, float (&v)[8]) {
    unpack8<F32>(fetch8<F32>(base, i), v);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t i, const float (&v)[8]) {
    if (F32) {
        float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + i);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + i) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
    }
}

// Two fp32 operations at once, each rounded as alone.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// (a, b) -> (a c - b s, b c + a s) for two pairs, one rounding a step
__device__ __forceinline__ void rotate2(float& a0, float& a1, float& b0, float& b1, float2 c, float2 s) {
    const float2 a = make_float2(a0, a1), b = make_float2(b0, b1);
    const float2 x = fma2(mul2(b, s), make_float2(-1.0f, -1.0f), mul2(a, c));
    const float2 y = fma2(mul2(a, s), make_float2(1.0f, 1.0f), mul2(b, c));
    a0 = x.x; a1 = x.y; b0 = y.x; b1 = y.y;
}

// (a, b) -> (a c - b s, b c + a s), one rounding a step
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
    const float x = a, y = b;
    a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

template <bool F32, int D, int ROT>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(F32, ROT)) qk_norm_rope_append_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int LPR = D / 16;                       // lanes per row
    constexpr int RPW = 32 / LPR;                     // rows per warp pass
    const int lane = threadIdx.x & 31;
    const int t = lane % LPR, sub = lane / LPR;
    // The lane's chunks of 8 elements: rotated ones with their partners, R / 2 further
    // on; behind them whole blocks of 16.
    const int hc = ROT == kRotHalf ? p.R / 16 : LPR;
    const bool whole = t >= hc;
    const int ca = whole ? 2 * t : t, cc = whole ? 2 * t + 1 : t + hc;
    const float st_k = *p.st_k, st_v = *p.st_v;
    const bool ok_k = st_k > 0.0f && st_k <= 3.4028234663852886e38f;
    const bool ok_v = st_v > 0.0f && st_v <= 3.4028234663852886e38f;
    if (!ok_k || !ok_v) {                             // a bad tensor scale skips everything
        if (blockIdx.x == 0 && threadIdx.x == 0) report(p.status, NVFP4_ERR_NONFINITE);
        return;
    }
    const int Ht = p.Hq + 2 * p.Hkv;
    for (uint32_t task = (blockIdx.x * kThreads + threadIdx.x) >> 5; task < p.tasks;
         task += gridDim.x * (kThreads / 32)) {
        const uint32_t tok = p.fd_tasks.div(task);    // token b * n + i
        const int part = (int)(task - tok * (uint32_t)p.tasks_per_token);
        const int b = (int)p.fd_n.div(tok);
        const int i = (int)tok - b * p.n;
        const int start = p.start[b];
        const int cnt = p.n_valid != nullptr ? p.n_valid[b] : p.n;
        if (cnt < 0 || cnt > p.n || start < 0 || (int64_t)start + cnt > p.S_max) {
            if (lane == 0 && part == 0 && i == 0)
                report(p.status, cnt < 0 || cnt > p.n ? NVFP4_ERR_INVALID_ARG : NVFP4_ERR_CAPACITY);
            continue;
        }
        if (part == 0 && i == 0 && lane == 0 && p.new_lens != nullptr) p.new_lens[b] = start + cnt;
        if (i >= cnt) continue;                       // padding: left as it was

        // the position's cos and sin
        float cs[ROT == kRotHalfPartial ? 16 : 8], sn[ROT == kRotHalfPartial ? 16 : 8];
        if (ROT != kRotNone) {
            const int pos = p.positions != nullptr ? p.positions[tok] : start + i;
            if (pos < 0 || pos >= p.P) {
                if (lane == 0 && part == 0) report(p.status, NVFP4_ERR_INVALID_ARG);
                continue;
            }
            const float* row = p.table + (int64_t)pos * p.R;
            const int half = p.R / 2;
            if (ROT == kRotHalf) {
#pragma unroll
                for (int e = 0; !whole && e < 8; e += 4) {
                    *reinterpret_cast<float4*>(cs + e) = __ldg(reinterpret_cast<const float4*>(row + 8 * t + e));
                    *reinterpret_cast<float4*>(sn + e) = __ldg(reinterpret_cast<const float4*>(row + half + 8 * t + e));
                }
            } else if (ROT == kRotInterleaved) {
                // chunk c rotates pairs 4c .. 4c + 3; past R: the identity
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = t + h * LPR;
                    const bool in = 8 * c < p.R;
                    const float4 a = in ? __ldg(reinterpret_cast<const float4*>(row + 4 * c)) : make_float4(1, 1, 1, 1);
                    const float4 z =
                        in ? __ldg(reinterpret_cast<const float4*>(row + half + 4 * c)) : make_float4(0, 0, 0, 0);
                    *reinterpret_cast<float4*>(cs + 4 * h) = a;
                    *reinterpret_cast<float4*>(sn + 4 * h) = z;
                }
            } else {
                // chunk c of the first half pairs with chunk c + R/16 of the second
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = t + h * LPR, hc = p.R / 16;
                    const int f = c < hc ? c : c - hc;
                    const bool in = c < 2 * hc;
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        *reinterpret_cast<float4*>(cs + 8 * h + e) =
                            in ? __ldg(reinterpret_cast<const float4*>(row + 8 * f + e)) : make_float4(1, 1, 1, 1);
                        *reinterpret_cast<float4*>(sn + 8 * h + e) =
                            in ? __ldg(reinterpret_cast<const float4*>(row + half + 8 * f + e))
                               : make_float4(0, 0, 0, 0);
                    }
                }
            }
        }
        // the cache slot
        int64_t slot0 = 0, slot_step = 0;             // token slot of head 0, slots between heads
        bool slot_ok = true;
        {
            const int s = start + i;
            if (p.block_table == nullptr) {
                slot_step = p.S_max;
                slot0 = (int64_t)b * p.Hkv * p.S_max + s;
            } else {
                const int lp = s / p.page_tokens;
                const int32_t page = p.block_table[(int64_t)b * p.max_pages + lp];
                slot_ok = page >= 0 && page < p.num_pages;
                if (!slot_ok && lane == 0 && part == 0) report(p.status, NVFP4_ERR_INVALID_ARG);
                slot_step = p.page_tokens;
                slot0 = (int64_t)(slot_ok ? page : 0) * p.Hkv * p.page_tokens + (s - lp * p.page_tokens);
            }
        }

        const int h_end = min(Ht, (part + 1) * p.heads_per_task);
        // a row's two pieces are fetched while the row before is worked on
        Raw<F32> ra = {}, rc = {};
        auto fetch = [&](int h) {
            if (h >= h_end) return;
            const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
            const void* x = is_q ? p.xq : (is_k ? p.xk : p.xv);
            const int64_t at = (int64_t)tok * (is_q ? p.sq : (is_k ? p.sk : p.sv)) +
                               (int64_t)(is_q ? h : (is_k ? h - p.Hq : h - p.Hq - p.Hkv)) * D;
            ra = fetch8<F32>(x, at + 8 * ca);
            rc = fetch8<F32>(x, at + 8 * cc);
        };
        fetch(part * p.heads_per_task + sub);
#pragma unroll 1
        for (int h0 = part * p.heads_per_task; h0 < h_end; h0 += RPW) {
            const int h = h0 + sub;
            const bool live = h < h_end;
            const bool is_q = h < p.Hq, is_k = !is_q && h < p.Hq + p.Hkv;
            const int hk = is_k ? h - p.Hq : h - p.Hq - p.Hkv;
            float a[8], c[8];                         // the lane's two chunks
            unpack8<F32>(ra, a);
            unpack8<F32>(rc, c);
            fetch(h + RPW);
            // elements taken two at a time: the neighbours, or of two interleaved pairs
            // the first ones and the second ones
            constexpr int S = ROT == kRotInterleaved ? 2 : 1;
            auto first = [](int i) { return S == 2 ? 4 * (i >> 1) + (i & 1) : 2 * i; };
            const bool normed = is_q || is_k;         // values are left as they are
            if (p.eps >= 0.0f && h0 < p.Hq + p.Hkv) {
                float2 s2 = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = first(i);
                    s2 = fma2(make_float2(a[e], a[e + S]), make_float2(a[e], a[e + S]), s2);
                    s2 = fma2(make_float2(c[e], c[e + S]), make_float2(c[e], c[e + S]), s2);
                }
                float ss = s2.x + s2.y;
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                if (live && normed) {
                    const float r = __frsqrt_rn(__fadd_rn(ss * (1.0f / D), p.eps));
                    const void* w = is_q ? p.wq : p.wk;
                    float wa[8], wc[8];
                    if (w != nullptr) {
                        load8<F32>(w, 8 * ca, wa);
                        load8<F32>(w, 8 * cc, wc);
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) wa[e] = wc[e] = 1.0f;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int e = first(i);
                        const float2 r2 = make_float2(r, r);
                        const float2 y = mul2(mul2(make_float2(a[e], a[e + S]), r2), make_float2(wa[e], wa[e + S]));
                        const float2 z = mul2(mul2(make_float2(c[e], c[e + S]), r2), make_float2(wc[e], wc[e + S]));
                        a[e] = y.x; a[e + S] = y.y;
                        c[e] = z.x; c[e + S] = z.y;
                    }
                }
            }
            if (ROT == kRotHalf) {
                if (normed && !whole) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        rotate2(a[e], a[e + 1], c[e], c[e + 1], make_float2(cs[e], cs[e + 1]), make_float2(sn[e], sn[e + 1]));
                }
            } else if (ROT == kRotInterleaved) {
                if (normed) {
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        if (8 * t < p.R)
                            rotate2(a[2 * e], a[2 * e + 2], a[2 * e + 1], a[2 * e + 3], make_float2(cs[e], cs[e + 1]),
                                    make_float2(sn[e], sn[e + 1]));
                        if (8 * (t + LPR) < p.R)
                            rotate2(c[2 * e], c[2 * e + 2], c[2 * e + 1], c[2 * e + 3], make_float2(cs[4 + e], cs[5 + e]),
                                    make_float2(sn[4 + e], sn[5 + e]));
                    }
                }
            } else if (ROT == kRotHalfPartial) {
                // the partner chunk sits in another lane, in its first or second slot
                const int rc = p.R / 16;
                float pa[8], pc[8];
                const int qa = ca < rc ? ca + rc : ca - rc, qc = cc < rc ? cc + rc : cc - rc;
                const int base = lane - t;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a0 = __shfl_sync(0xFFFFFFFFu, a[e], base + (qa & (LPR - 1)));
                    const float a1 = __shfl_sync(0xFFFFFFFFu, c[e], base + (qa & (LPR - 1)));
                    const float c0 = __shfl_sync(0xFFFFFFFFu, a[e], base + (qc & (LPR - 1)));
                    const float c1 = __shfl_sync(0xFFFFFFFFu, c[e], base + (qc & (LPR - 1)));
                    pa[e] = qa < LPR ? a0 : a1;
                    pc[e] = qc < LPR ? c0 : c1;
                }
                if (normed) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (ca < 2 * rc) {
                            if (ca < rc) rotate(a[e], pa[e], cs[e], sn[e]);
                            else { rotate(pa[e], a[e], cs[e], sn[e]); }
                        }
                        if (cc < 2 * rc) {
                            if (cc < rc) rotate(c[e], pc[e], cs[8 + e], sn[8 + e]);
                            else { rotate(pc[e], c[e], cs[8 + e], sn[8 + e]); }
                        }
                    }
                }
            }
            if (live && is_q) {
                const int64_t at = ((int64_t)tok * p.Hq + h) * D;
                store8<F32>(p.q_out, at + 8 * ca, a);
                store8<F32>(p.q_out, at + 8 * cc, c);
            }
            if (h0 + RPW > p.Hq) {                    // some row of this pass is a key or a value
                float ma = 0.0f, mc = 0.0f;
                bool na = false, nc = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ma = fmaxf(ma, fabsf(a[e]));
                    mc = fmaxf(mc, fabsf(c[e]));
                    na |= a[e] != a[e];
                    nc |= c[e] != c[e];
                }
                // the other chunk of the block: the neighbouring lane's, or this lane's
                const float oa = __shfl_xor_sync(0xFFFFFFFFu, ma, 1), oc = __shfl_xor_sync(0xFFFFFFFFu, mc, 1);
                const int flags = (na ? 1 : 0) | (nc ? 2 : 0), other = __shfl_xor_sync(0xFFFFFFFFu, flags, 1);
                if (whole) {
                    ma = mc = fmaxf(ma, mc);
                    na = nc = flags != 0;
                } else {
                    ma = fmaxf(ma, oa);
                    mc = fmaxf(mc, oc);
                    na |= (other & 1) != 0;
                    nc |= (other & 2) != 0;
                }
                if (live && !is_q && slot_ok) {
                    const float st = is_k ? st_k : st_v;
                    uint32_t sa, sc;
                    const uint32_t wa = quantize_half(a, ma, na, st, sa);
                    const uint32_t wc = quantize_half(c, mc, nc, st, sc);
                    const int64_t slot = slot0 + (int64_t)hk * slot_step;
                    uint8_t* codes = (is_k ? p.kc : p.vc) + slot * (D / 2);
                    uint8_t* scales = (is_k ? p.ks : p.vs) + slot * (D / 16);
                    *reinterpret_cast<uint32_t*>(codes + 4 * ca) = wa;
                    *reinterpret_cast<uint32_t*>(codes + 4 * cc) = wc;
                    if ((ca & 1) == 0) scales[ca / 2] = (uint8_t)sa;
                    if ((cc & 1) == 0) scales[cc / 2] = (uint8_t)sc;
                }
            }
        }
    }
}

template <bool F32, int D>
cudaError_t launch(const NormRopeParams& p, int rot, cudaStream_t stream) {
    const int64_t warps = p.tasks;
    int64_t grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t cap = blocks_per_sm(F32, rot) * (int64_t)device_sm_count();
    if (grid > cap) grid = cap;
    switch (rot) {
        case kRotNone: qk_norm_rope_append_kernel<F32, D, kRotNone><<<(unsigned)grid, kThreads, 0, stream>>>(p); break;
        case kRotHalf: qk_norm_rope_append_kernel<F32, D, kRotHalf><<<(unsigned)grid, kThreads, 0, stream>>>(p); break;
        case kRotInterleaved:
            qk_norm_rope_append_kernel<F32, D, kRotInterleaved><<<(unsigned)grid, kThreads, 0, stream>>>(p);
            break;
        default:
            qk_norm_rope_append_kernel<F32, D, kRotHalfPartial><<<(unsigned)grid, kThreads, 0, stream>>>(p);
            break;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope_append(const NormRopeLaunch& a, cudaStream_t stream) {
    NormRopeParams p = {};
    p.xq = a.xq; p.xk = a.xk; p.xv = a.xv;
    p.sq = a.sq; p.sk = a.sk; p.sv = a.sv;
    p.wq = a.wq; p.wk = a.wk;
    p.table = a.table; p.positions = a.positions;
    p.start = a.start; p.n_valid = a.n_valid; p.new_lens = a.new_lens;
    p.st_k = a.st_k; p.st_v = a.st_v;
    p.q_out = a.q_out;
    p.kc = a.kc; p.ks = a.ks; p.vc = a.vc; p.vs = a.vs;
    p.block_table = a.block_table;
    p.status = a.status;
    p.B = a.B; p.n = a.n; p.Hq = a.Hq; p.Hkv = a.Hkv; p.S_max = a.S_max; p.R = a.R; p.P = a.P;
    p.page_tokens = a.page_tokens; p.max_pages = a.max_pages; p.num_pages = a.num_pages;
    p.eps = a.eps;
    const int rpw = 32 / (a.D / 16);
    const int Ht = a.Hq + 2 * a.Hkv;
    const int passes = (Ht + rpw - 1) / rpw;
    const int rot = a.R == 0 ? kRotNone : (a.interleaved ? kRotInterleaved : (a.R % 32 == 0 ? kRotHalf : kRotHalfPartial));
    // Passes of one task: the split of the tokens' passes that the resident warps
    // finish first, a task costing about two passes of its own (position, slot).
    const int64_t tokens = (int64_t)a.B * a.n, warps = (int64_t)blocks_per_sm(a.f32, rot) * (kThreads / 32) * device_sm_count();
    int64_t per = 1, best = INT64_MAX;
    for (int parts = 1; parts <= passes; ++parts) {
        const int64_t len = (passes + parts - 1) / parts, rounds = (tokens * parts + warps - 1) / warps;
        if (rounds * (len + 2) < best) {
            best = rounds * (len + 2);
            per = len;
        }
    }
    p.heads_per_task = (int)per * rpw;
    p.tasks_per_token = (Ht + p.heads_per_task - 1) / p.heads_per_task;
    p.tasks = (uint32_t)(tokens * p.tasks_per_token);
    p.fd_tasks = FastDiv((uint32_t)p.tasks_per_token);
    p.fd_n = FastDiv((uint32_t)a.n);
    if (a.f32) return a.D == 128 ? launch<true, 128>(p, rot, stream) : launch<true, 64>(p, rot, stream);
    return a.D == 128 ? launch<false, 128>(p, rot, stream) : launch<false, 64>(p, rot, stream);
}

}  // namespace nvfp4kv
