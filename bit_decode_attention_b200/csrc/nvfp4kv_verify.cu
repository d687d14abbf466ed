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
// chunk again (from L2).  Bound by HBM for large batches, by the chain of
// memory latencies and cluster barriers for one sequence.
#include <cooperative_groups.h>

#include "nvfp4kv_device.cuh"
#include "nvfp4kv_internal.h"

namespace nvfp4kv {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

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
    int32_t N, V, chunk;                              // chunk: elements of a warp, a multiple of 512
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

// NaN and negative weights count as 0
__device__ __forceinline__ double positive(double x) { return x > 0.0 ? x : 0.0; }

struct Shared {
    double z[kTreeMaxNodes];                          // Z subtracted by each rejection of the current node
    float pp[kTreeMaxNodes], dd[kTreeMaxNodes];       // p and d of a node's token at its parent
    float ua[kTreeMaxNodes];
    int32_t token[kTreeMaxNodes], parent[kTreeMaxNodes];
    int32_t rejected[kTreeMaxNodes];                  // the rejected nodes of the current node
    double warp_sum[kWarps];
    double total[2];                                  // this CTA's slice sum, two passes' worth
};

template <bool F32, int VEC>
__global__ void __launch_bounds__(kThreads) verify_drafts_kernel(const VerifyParams q) {
    __shared__ Shared sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), nranks = (int)cluster.num_blocks();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = (int)(blockIdx.x / (unsigned)nranks);
    const int N = q.N, V = q.V;
    const int n = q.n_nodes != nullptr ? q.n_nodes[b] : N;
    if (n < 1 || n > N) {                             // 0: a padding row, left as it was
        if (n != 0 && rank == 0 && tid == 0) report(q.status, NVFP4_ERR_INVALID_ARG);
        return;                                       // the whole cluster
    }
    const int64_t row0 = (int64_t)b * N;

    // the tested tokens' probabilities; a node with a bad parent or token is never tested
    for (int i = tid; i < n; i += kThreads) {
        const int32_t par = q.parents[(int64_t)b * q.parent_stride + i];
        const int32_t tok = q.tokens[row0 + i];
        const bool ok = i > 0 && par >= 0 && par < i && tok >= 0 && tok < V;
        if (i > 0 && !ok && rank == 0) report(q.status, NVFP4_ERR_INVALID_ARG);
        sm.parent[i] = ok ? par : -1;
        sm.token[i] = tok;
        sm.ua[i] = q.u_accept[row0 + i];
        sm.pp[i] = ok ? load1<F32>(q.p, (row0 + par) * V + tok) : 0.0f;
        sm.dd[i] = ok && q.d != nullptr ? load1<F32>(q.d, (row0 + par) * V + tok) : 1.0f;
    }
    __syncthreads();

    int at = 0, nrej = 0, passes = 0, n_acc = 1;
    double Z = 1.0;
    bool sums_valid = false;                          // warp_sum and total hold the current weights' sums

    // w of token x (probability pv, draft dv) after the first k rejections
    auto weight = [&](float pv, double dv, int x, int k) -> double {
        double w = (double)fmaxf(pv, 0.0f);           // NaN gives 0
        if (q.d != nullptr) {
            for (int j = 0; j < k; ++j) w = positive(w - sm.z[j] * dv);
        } else {
            for (int j = 0; j < k; ++j)
                if (sm.token[sm.rejected[j]] == x) w = positive(w - sm.z[j]);
        }
        return w;
    };
    const int slice = q.chunk * kWarps;
    const int64_t lo = (int64_t)rank * slice + (int64_t)warp * q.chunk;
    const int64_t hi = lo + q.chunk < V ? lo + q.chunk : V;
    // sum of the weights after k rejections of node `at`, over the cluster
    auto pass = [&](int k) -> double {
        const int64_t base = (row0 + at) * V;
        const bool use_d = q.d != nullptr && k > 0;
        double s = 0.0;
        constexpr int U = 4;
        for (int64_t i0 = lo + lane * VEC; i0 < hi; i0 += 32 * VEC * U) {
            float pv[U][VEC], dv[U][VEC];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = i0 + u * 32 * VEC;
                if (i < hi) {
                    load_vec<F32, VEC>(q.p, base + i, pv[u]);
                    if (use_d) load_vec<F32, VEC>(q.d, base + i, dv[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = i0 + u * 32 * VEC;
                if (i < hi) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        s += weight(pv[u][e], use_d ? (double)dv[u][e] : 0.0, (int)i + e, k);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0) sm.warp_sum[warp] = s;
        __syncthreads();
        double* slot = &sm.total[passes & 1];
        if (tid == 0) {
            double t = 0.0;
            for (int w = 0; w < kWarps; ++w) t += sm.warp_sum[w];
            *slot = t;
        }
        cluster.sync();
        double t = 0.0;
        for (int r = 0; r < nranks; ++r) t += *cluster.map_shared_rank(slot, r);
        ++passes;
        return t;
    };

    if (rank == 0 && tid == 0) q.path[row0] = 0;
    for (int i = 1; i < n; ++i) {
        if (sm.parent[i] != at) continue;             // uniform over the cluster
        const double w = weight(sm.pp[i], (double)sm.dd[i], sm.token[i], nrej);
        if ((double)sm.ua[i] * (double)sm.dd[i] * Z < w) {
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
            sm.rejected[nrej] = i;
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
        const float us = q.u_sample[b];
        const double target = us > 0.0f ? (double)us * total : 0.0;
        double before = 0.0, mine = 0.0;
        bool last = true;
        for (int r = 0; r < nranks; ++r) {
            const double t = *cluster.map_shared_rank(&sm.total[(passes - 1) & 1], r);
            if (r < rank) before += t;
            if (r == rank) mine = t;
            if (r > rank && t > 0.0) last = false;
        }
        if (mine > 0.0 && before <= target && (target < before + mine || last)) {
            // (uniform over the CTA from here)
            auto first_past = [&](double& acc) -> int {
                int hit = 0;
                double at_hit = acc;
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
            const int sub = q.chunk / kWarps;         // a multiple of 32
            const int64_t s0 = (int64_t)rank * slice + (int64_t)hit * q.chunk + (int64_t)warp * sub;
            const int64_t s1 = s0 + sub < V ? s0 + sub : V;
            auto weight_at = [&](int64_t i) -> double {
                return i < s1 ? weight(load1<F32>(q.p, base + i),
                                       q.d != nullptr && nrej > 0 ? (double)load1<F32>(q.d, base + i) : 0.0, (int)i,
                                       nrej)
                              : 0.0;
            };
            double s = 0.0;
#pragma unroll 4
            for (int64_t i0 = s0; i0 < s1; i0 += 32) s += weight_at(i0 + lane);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            __syncthreads();                          // the chunks' sums are consumed
            if (lane == 0) sm.warp_sum[warp] = s;
            __syncthreads();
            if (warp == first_past(acc)) {
                int answer = -1, best = 0;
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
    cluster.sync();                                   // no CTA leaves while others read its sums
}

template <bool F32, int VEC>
cudaError_t launch(const VerifyParams& q, int B, int cluster, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<F32, VEC>, q);
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
    const int cluster = kMaxCluster;
    const int per16 = a.f32 ? 4 : 8;
    const bool vec = a.V % per16 == 0 && reinterpret_cast<uintptr_t>(a.p) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.d) % 16 == 0;
    const int align = 32 * kWarps;                    // whole 32-element rows for each sixteenth of a chunk
    const int64_t chunk = ((int64_t)a.V + cluster * kWarps - 1) / (cluster * kWarps);
    q.chunk = (int32_t)((chunk + align - 1) / align * align);
    if (a.f32) return vec ? launch<true, 4>(q, a.B, cluster, stream) : launch<true, 1>(q, a.B, cluster, stream);
    return vec ? launch<false, 8>(q, a.B, cluster, stream) : launch<false, 1>(q, a.B, cluster, stream);
}

}  // namespace nvfp4kv
