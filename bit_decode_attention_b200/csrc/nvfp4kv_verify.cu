// nvfp4kv_verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers (speculative sampling over a tree).
//
// The walk starts at node 0.  At node a the weights are w = p_a with Z = 1; a
// child c (token x) is accepted when u_c * d_a(x) * Z < w(x), else
// w <- max(w - Z d_a, 0) and Z <- sum w (both kept when that sum is 0), with
// d_a the draft's distribution, or the point mass at x without one.  The next
// token is the least i with w(0) + .. + w(i) > u * sum w.
//
// All of it in 64 bits: a token's border moves with the rounding of a sum
// over the whole vocabulary, which 32 bits would shift by whole tokens.
//
// One cluster of CTAs per sequence.  Every CTA walks the tree on its own from
// the tested tokens' probabilities (gathered first, in parallel: one memory
// latency for all nodes); only a rejection, or the end of the walk, needs a
// pass over the vocabulary, of which each CTA takes a slice and each warp a
// contiguous chunk.  The chunks' sums are kept, so that the last pass also
// says which warp's chunk holds the sampled token; that warp alone reads its
// chunk again (from L2).
//
// Measured (B200): one sequence, 6 nodes over 32,000 tokens: 8.4 us, a chain of
// memory latencies and cluster barriers.  64 sequences, up to 16 nodes over
// 131,072: 41 to 48 us by the walks, where 59 MB of rows take 9 at 6.55 TB/s (26.7
// without draft rows, 34.9 with bf16 ones): a sequence waits for
// two or three passes in turn, of 10 us each; 12 of the 41 are the 64-bit weights
// (conversions run at 16 a clock and SM).  Loops over elements unrolled further,
// or the loop over rejections inside them, make the code larger than the
// instruction cache holds: 72 us and 18.5.
#include <cooperative_groups.h>

#include "nvfp4kv_device.cuh"
#include "nvfp4kv_internal.h"

namespace nvfp4kv {

namespace {

namespace cg = cooperative_groups;

// Of 4 CTAs an SM.  512 threads (2 an SM): 42 us as here for 64 sequences of 16 nodes
// over 131,072 tokens, 10.3 for 8.4 for one of 6 over 32,000, 26 for 16 for 64 of
// those, but 12.4 for 15.0 for one over 131,072.
constexpr int kCluster = 8, kThreads = 256, kWarps = kThreads / 32;

struct VerifyParams {
    const void* p;                                    // [B][N][V]
    const void* d;                                    // [B][N][V] or nullptr: point masses
    const int32_t* tokens;                            // [B][N]
    const int32_t* parents;                           // [N], or [B][N] with parent_stride N
    const float* u_accept;                            // [B][N]
    const float* u_sample;                            // [B]
    const int32_t* n_nodes;                           // [B] or nullptr
    int32_t* path;                                    // [B][N]
    int32_t* n_acc;                                   // [B]
    int32_t* next;                                    // [B]
    int32_t* status;
    int64_t parent_stride;
    int32_t N, V, chunk;                              // chunk: elements of a warp, a multiple of 32 * kWarps
};

template <bool F32>
__device__ __forceinline__ float load1(const void* base, int64_t i) {
    if (F32) return __ldg(reinterpret_cast<const float*>(base) + i);
    return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t*>(base) + i) << 16);
}

// VEC consecutive elements at i (VEC > 1: 16-byte aligned)
template <bool F32, int VEC>
__device__ __forceinline__ void load_vec(const void* base, int64_t i, float (&v)[VEC]) {
    if (VEC == 1) {
        v[0] = load1<F32>(base, i);
    } else if (F32) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + i));
        v[0] = f.x; v[1 % VEC] = f.y; v[2 % VEC] = f.z; v[3 % VEC] = f.w;
    } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + i));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[(2 * j) % VEC] = __uint_as_float(w[j] << 16);
            v[(2 * j + 1) % VEC] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
}

// 16-byte aligned, a multiple of 16 bytes
__device__ __forceinline__ void prefetch_l2(const void* from, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
}

// NaN and negative weights count as 0
__device__ __forceinline__ double positive(double x) { return x > 0.0 ? x : 0.0; }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

struct Shared {
    double z[kTreeMaxNodes];                          // Z subtracted by each rejection of the current node
    float pp[kTreeMaxNodes], dd[kTreeMaxNodes];       // p and d of a node's token at its parent
    float ua[kTreeMaxNodes];
    int32_t token[kTreeMaxNodes], parent[kTreeMaxNodes];
    int32_t rejected[kTreeMaxNodes];                  // the tokens of the current node's rejections
    double warp_sum[kWarps];
    double total[2][kCluster];                        // the CTAs' sums of the last two passes
};

// DRAFT: with the draft's distribution; else point masses
template <bool F32, int VEC, bool DRAFT>
__global__ void __launch_bounds__(kThreads, 4) verify_drafts_kernel(const VerifyParams q) {
    __shared__ Shared sm;
    cg::cluster_group cluster = cg::this_cluster();
    cluster_arrive();
    const int rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = (int)(blockIdx.x / (unsigned)kCluster);
    const int N = q.N, V = q.V;
    const int64_t row0 = (int64_t)b * N;
    const int n = q.n_nodes != nullptr ? q.n_nodes[b] : N;
    const float us = q.u_sample[b];

    // the tested tokens' probabilities; a node with a bad parent or token is never tested
#pragma unroll 1
    for (int i = tid; i < N; i += kThreads) {
        const int32_t par = q.parents[(int64_t)b * q.parent_stride + i];
        const int32_t tok = q.tokens[row0 + i];
        const float ua = q.u_accept[row0 + i];
        const bool ok = i > 0 && par >= 0 && par < i && tok >= 0 && tok < V;
        if (i > 0 && i < n && n <= N && !ok && rank == 0) report(q.status, NVFP4_ERR_INVALID_ARG);
        sm.parent[i] = ok ? par : -1;
        sm.token[i] = tok;
        sm.ua[i] = ua;
        sm.pp[i] = ok && i < n ? load1<F32>(q.p, (row0 + par) * V + tok) : 0.0f;
        sm.dd[i] = DRAFT && ok && i < n ? fmaxf(load1<F32>(q.d, (row0 + par) * V + tok), 0.0f) : 1.0f;
    }
    if (n < 1 || n > N) {                             // 0: a padding row, left as it was
        if (n != 0 && rank == 0 && tid == 0) report(q.status, NVFP4_ERR_INVALID_ARG);
        return;                                       // the whole cluster
    }
    __syncthreads();
    cluster_wait();                                   // every CTA has started: its memory may be written

    int at = 0, nrej = 0, passes = 0, n_acc = 1;
    double Z = 1.0;
    bool sums_valid = false;                          // warp_sum and total hold the current weights' sums

    // E weights at once, of tokens x, x + 1, .. (probability pv, draft dv >= 0), after the
    // first k rejections.  NaN counts as 0.  (The loop over rejections stays rolled:
    // unrolled over elements too, the code would be the kernel's time.)
    auto weights = [&](auto& w, const auto& pv, const auto& dv, int x, int k) {
        constexpr int E = (int)(sizeof(pv) / sizeof(float));
#pragma unroll
        for (int e = 0; e < E; ++e) w[e] = (double)fmaxf(pv[e], 0.0f);
#pragma unroll 1
        for (int j = 0; j < k; ++j) {
            const double z = sm.z[j];
            if (DRAFT) {
#pragma unroll
                for (int e = 0; e < E; ++e) w[e] = positive(w[e] - z * (double)dv[e]);
            } else {
                const uint32_t at_e = (uint32_t)(sm.rejected[j] - x);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (at_e == (uint32_t)e) w[e] = positive(w[e] - z);
            }
        }
    };
    const int slice = q.chunk * kWarps;
    const int64_t lo = (int64_t)rank * slice + (int64_t)warp * q.chunk;
    const int64_t hi = lo + q.chunk < V ? lo + q.chunk : V;
    // sum of the weights after k rejections of node `at`, over the cluster
    auto pass = [&](int k) -> double {
        const int64_t base = (row0 + at) * V;
        double s = 0.0;
        if (VEC > 1 && lane == 0 && lo < hi) {        // the chunk to L2 at once: its loads then wait for no DRAM
            constexpr int ES = F32 ? 4 : 2;
            const uint32_t bytes = (uint32_t)(hi - lo) * ES;
            prefetch_l2(static_cast<const uint8_t*>(q.p) + (base + lo) * ES, bytes);
            if (DRAFT && k > 0) prefetch_l2(static_cast<const uint8_t*>(q.d) + (base + lo) * ES, bytes);
        }
        constexpr int U = VEC == 8 ? 1 : 2;          // loads of each row in flight
#pragma unroll 1
        for (int64_t i0 = lo + lane * VEC; i0 < hi; i0 += 32 * VEC * U) {
            float pv[U][VEC], dv[U][VEC];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = i0 + u * 32 * VEC;
#pragma unroll
                for (int e = 0; e < VEC; ++e) pv[u][e] = dv[u][e] = 0.0f;
                if (i < hi) {
                    load_vec<F32, VEC>(q.p, base + i, pv[u]);
                    if (DRAFT && k > 0) {
                        load_vec<F32, VEC>(q.d, base + i, dv[u]);
#pragma unroll
                        for (int e = 0; e < VEC; ++e) dv[u][e] = fmaxf(dv[u][e], 0.0f);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                double w[VEC];
                weights(w, pv[u], dv[u], (int)(i0 + u * 32 * VEC), k);
#pragma unroll
                for (int e = 0; e < VEC; ++e) s += w[e];
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0) sm.warp_sum[warp] = s;
        __syncthreads();
        // Every CTA gives its sum to all of them.  (The slot's last readers came to the
        // barrier of the pass between.)
        double* const slot = sm.total[passes & 1];
        if (warp == 0) {
            double t = lane < kWarps ? sm.warp_sum[lane] : 0.0;
#pragma unroll
            for (int o = kWarps / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
            if (lane < kCluster) *cluster.map_shared_rank(slot + rank, lane) = t;
        }
        cluster.sync();
        double t = 0.0;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) t += slot[r];
        ++passes;
        return t;
    };

    if (rank == 0 && tid == 0) q.path[row0] = 0;
#pragma unroll 1
    for (int i = 1; i < n; ++i) {
        if (sm.parent[i] != at) continue;             // uniform over the cluster
        const float pv[1] = {sm.pp[i]}, dv[1] = {sm.dd[i]};
        double w[1];
        weights(w, pv, dv, sm.token[i], nrej);
        if ((double)sm.ua[i] * (double)dv[0] * Z < w[0]) {
            if (rank == 0 && tid == 0) q.path[row0 + n_acc] = i;
            ++n_acc;
            at = i;
            nrej = 0;
            Z = 1.0;
            sums_valid = false;
            continue;
        }
        __syncthreads();                              // readers of the previous list are done
        if (tid == 0) {
            sm.z[nrej] = Z;
            sm.rejected[nrej] = sm.token[i];
        }
        __syncthreads();
        const double total = pass(nrej + 1);
        sums_valid = total > 0.0;
        if (sums_valid) {
            ++nrej;
            Z = total;
        }
    }
    for (int j = n_acc + tid; rank == 0 && j < N; j += kThreads) q.path[row0 + j] = -1;
    const double total = sums_valid ? Z : pass(nrej);
    if (rank == 0 && tid == 0) {
        q.n_acc[b] = n_acc;
        if (!(total > 0.0) || total > 1.7e308) {
            q.next[b] = -1;
            report(q.status, NVFP4_ERR_NONFINITE);
        }
    }
    if (total > 0.0 && total <= 1.7e308) {
        // the slice, then the warp's chunk, then the 1/16 of that chunk, then the
        // element whose inclusive sum is the first past the target; should
        // rounding pass the end, the last one that holds any weight
        const double target = us > 0.0f ? (double)us * total : 0.0;
        double before = 0.0, mine = 0.0;
        bool last = true;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) {
            const double t = sm.total[(passes - 1) & 1][r];
            if (r < rank) before += t;
            if (r == rank) mine = t;
            if (r > rank && t > 0.0) last = false;
        }
        if (mine > 0.0 && before <= target && (target < before + mine || last)) {
            // (uniform over the CTA from here)
            auto first_past = [&](double& acc) -> int {
                int hit = 0;
                double at_hit = acc;
#pragma unroll 1
                for (int w = 0; w < kWarps; ++w) {
                    const double s = sm.warp_sum[w];
                    if (s > 0.0) {
                        hit = w;
                        at_hit = acc;
                        if (acc + s > target) break;
                        acc += s;
                    }
                }
                acc = at_hit;
                return hit;
            };
            double acc = before;
            const int hit = first_past(acc);
            const int64_t base = (row0 + at) * V;
            const int sub = q.chunk / kWarps;          // a multiple of 32
            const int64_t s0 = (int64_t)rank * slice + (int64_t)hit * q.chunk + (int64_t)warp * sub;
            const int64_t s1 = s0 + sub < V ? s0 + sub : V;
            auto weight_at = [&](int64_t i) -> double {
                float pv[1] = {0.0f}, dv[1] = {0.0f};
                if (i < s1) {
                    pv[0] = load1<F32>(q.p, base + i);
                    if (DRAFT && nrej > 0) dv[0] = fmaxf(load1<F32>(q.d, base + i), 0.0f);
                }
                double w[1];
                weights(w, pv, dv, (int)i, nrej);
                return w[0];
            };
            double s = 0.0;
#pragma unroll 1
            for (int64_t i0 = s0; i0 < s1; i0 += 32) s += weight_at(i0 + lane);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            __syncthreads();                          // the chunks' sums are consumed
            if (lane == 0) sm.warp_sum[warp] = s;
            __syncthreads();
            if (warp == first_past(acc)) {
                int answer = -1, best = 0;
#pragma unroll 1
                for (int64_t i0 = s0; i0 < s1 && answer < 0; i0 += 32) {
                    const double w = weight_at(i0 + lane);
                    double c = w;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const double up = __shfl_up_sync(0xFFFFFFFFu, c, o);
                        if (lane >= o) c += up;
                    }
                    const uint32_t over = __ballot_sync(0xFFFFFFFFu, w > 0.0 && acc + c > target);
                    const uint32_t some = __ballot_sync(0xFFFFFFFFu, w > 0.0);
                    if (over) answer = (int)i0 + __ffs(over) - 1;
                    if (some) best = (int)i0 + 31 - __clz(some);
                    acc += __shfl_sync(0xFFFFFFFFu, c, 31);
                }
                if (lane == 0) q.next[b] = answer >= 0 ? answer : best;
            }
        }
    }
    // (After the last pass's barrier no CTA touches another's memory.)
}

template <bool F32, int VEC, bool DRAFT>
cudaError_t launch(VerifyParams& q, int B, cudaStream_t stream) {
    constexpr int align = 32 * kWarps;                 // whole 32-element rows for each warp's share of a chunk
    const int64_t chunk = ((int64_t)q.V + kCluster * kWarps - 1) / (kCluster * kWarps);
    q.chunk = (int32_t)((chunk + align - 1) / align * align);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * kCluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)kCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<F32, VEC, DRAFT>, q);
}

template <bool F32, int VEC>
cudaError_t launch(VerifyParams& q, int B, cudaStream_t stream) {
    return q.d != nullptr ? launch<F32, VEC, true>(q, B, stream) : launch<F32, VEC, false>(q, B, stream);
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyLaunch& a, cudaStream_t stream) {
    VerifyParams q = {};
    q.p = a.p;
    q.d = a.d;
    q.tokens = a.tokens;
    q.parents = a.parents;
    q.parent_stride = a.parents_shared ? 0 : a.N;
    q.u_accept = a.u_accept;
    q.u_sample = a.u_sample;
    q.n_nodes = a.n_nodes;
    q.path = a.path;
    q.n_acc = a.n_acc;
    q.next = a.next;
    q.status = a.status;
    q.N = a.N;
    q.V = a.V;
    const int per16 = a.f32 ? 4 : 8;
    const bool vec = a.V % per16 == 0 && reinterpret_cast<uintptr_t>(a.p) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.d) % 16 == 0;
    if (a.f32) return vec ? launch<true, 4>(q, a.B, stream) : launch<true, 1>(q, a.B, stream);
    return vec ? launch<false, 8>(q, a.B, stream) : launch<false, 1>(q, a.B, stream);
}

}  // namespace nvfp4kv
