// nvfp4kv_commit_path.cu -- keeping the accepted path of a drafted tree: the
// cache slots start + path[j] of the accepted nodes move to start + j, for
// every KV head and any number of planes (all layers' K and V) in one launch.
//
// Bytes are moved, nothing is computed: path[0] < path[1] < ..., so
// path[j] >= j, and a slot is overwritten only by nodes that come after the
// one it held.  A block loads a chunk of rows j .. j + n - 1, waits, and
// stores them; later chunks read slots path[j'] >= j' >= j + n only, which no
// earlier chunk wrote.
#include "nvfp4kv_device.cuh"
#include "nvfp4kv_internal.h"

namespace nvfp4kv {

namespace {

constexpr int kThreads = 256;

struct CommitParams {
    uint8_t* codes[kCommitPlanes];
    uint8_t* scales[kCommitPlanes];
    const int32_t* start;
    const int32_t* path;
    const int32_t* n_acc;
    int32_t* new_lens;
    int32_t* status;
    const int32_t* block_table;                       // nullptr: contiguous planes
    int32_t num_pages, page_tokens, max_pages;
    int32_t Hkv, S_max, N;
    int32_t code_cols, cols;                          // 16-byte code columns, and all columns, of a token's heads
    int32_t lg_code;                                  // log2 of the 16-byte code columns a head
    int32_t scale_bytes;                              // scale bytes of a token and head: 8 or 4
    int32_t rows;                                     // path rows a block moves at once
    int32_t first;                                    // this launch holds the call's first plane
};

// grid (planes, sequences).  Thread (row, column): column c < code_cols is 16
// code bytes of head c >> lg_code, the others one head's scale bytes.
__global__ void __launch_bounds__(kThreads) commit_path_kernel(const __grid_constant__ CommitParams p) {
    __shared__ int32_t s_path[kTreeMaxNodes];
    const int b = blockIdx.y, plane = blockIdx.x, tid = threadIdx.x;
    const int32_t start = p.start[b];
    const int32_t n = p.n_acc[b];
    const int32_t* row = p.path + (int64_t)b * p.N;
    // every block checks its sequence: increasing nodes inside the tree and the cache
    int bad = n < 0 || n > p.N || start < 0 || (int64_t)start + n > p.S_max ? 1 : 0;
    const bool over = n >= 0 && n <= p.N && start >= 0 && (int64_t)start + n > p.S_max;
    int past = over ? 1 : 0;
    if (!bad) {
        for (int j = tid; j < n; j += kThreads) {
            const int32_t v = row[j];
            const int32_t prev = j > 0 ? row[j - 1] : -1;
            s_path[j] = v;
            if (v <= prev || v >= p.N) bad = 1;
            else if ((int64_t)start + v >= p.S_max) bad = past = 1;
        }
    }
    bad = __syncthreads_or(bad);
    past = __syncthreads_or(past);
    if (bad) {
        if (tid == 0 && plane == 0) report(p.status, past ? NVFP4_ERR_CAPACITY : NVFP4_ERR_INVALID_ARG);
        return;
    }
    if (tid == 0 && plane == 0 && p.first && p.new_lens != nullptr) p.new_lens[b] = start + n;

    uint8_t* const codes = p.codes[plane];
    uint8_t* const scales = p.scales[plane];
    // bytes of token t's first head, in units of a token slot; -1: a page outside the pool
    auto slot_of = [&](int32_t t, int h) -> int64_t {
        if (p.block_table == nullptr) return ((int64_t)b * p.Hkv + h) * p.S_max + t;
        const int lp = t / p.page_tokens;
        const int32_t page = p.block_table[(int64_t)b * p.max_pages + lp];
        if (page < 0 || page >= p.num_pages) return -1;
        return ((int64_t)page * p.Hkv + h) * p.page_tokens + (t - lp * p.page_tokens);
    };
    const int r = tid / p.cols, c0 = tid - r * p.cols;
    // columns past a block's threads (cols > kThreads) are taken in further passes
    for (int cb = 0; cb < p.cols; cb += kThreads) {
        const int c = p.cols > kThreads ? cb + tid : c0;
        const int rr = p.cols > kThreads ? 0 : r;
        const bool code = c < p.code_cols;
        const int h = code ? c >> p.lg_code : c - p.code_cols;
        for (int j0 = 0; j0 < n; j0 += p.rows) {
            const int j = j0 + rr;
            const bool mine = rr < p.rows && c < p.cols && j < n && s_path[min(j, n - 1)] != j;
            int64_t src = -1, dst = -1;
            if (mine) {
                src = slot_of(start + s_path[j], h);
                dst = slot_of(start + j, h);
                if (src < 0 || dst < 0) report(p.status, NVFP4_ERR_INVALID_ARG);
            }
            const bool go = src >= 0 && dst >= 0;
            uint4 w = make_uint4(0, 0, 0, 0);
            const int col = c & ((1 << p.lg_code) - 1);
            if (go) {
                if (code)
                    w = *reinterpret_cast<const uint4*>(codes + (((src << p.lg_code) + col) << 4));
                else if (p.scale_bytes == 8)
                    *reinterpret_cast<uint2*>(&w) = *reinterpret_cast<const uint2*>(scales + src * 8);
                else
                    w.x = *reinterpret_cast<const uint32_t*>(scales + src * 4);
            }
            __syncthreads();
            if (go) {
                if (code)
                    *reinterpret_cast<uint4*>(codes + (((dst << p.lg_code) + col) << 4)) = w;
                else if (p.scale_bytes == 8)
                    *reinterpret_cast<uint2*>(scales + dst * 8) = make_uint2(w.x, w.y);
                else
                    *reinterpret_cast<uint32_t*>(scales + dst * 4) = w.x;
            }
        }
    }
}

}  // namespace

cudaError_t launch_commit_path(const CommitLaunch& a, cudaStream_t stream) {
    CommitParams p = {};
    p.start = a.start;
    p.path = a.path;
    p.n_acc = a.n_acc;
    p.new_lens = a.new_lens;
    p.status = a.status;
    p.block_table = a.block_table;
    p.num_pages = a.num_pages;
    p.page_tokens = a.page_tokens;
    p.max_pages = a.max_pages;
    p.Hkv = a.Hkv;
    p.S_max = a.S_max;
    p.N = a.N;
    p.lg_code = a.D == 128 ? 2 : 1;
    p.code_cols = a.Hkv << p.lg_code;
    p.cols = p.code_cols + a.Hkv;
    p.scale_bytes = a.D / 16;
    p.rows = p.cols >= kThreads ? 1 : kThreads / p.cols;
    for (int first = 0; first < a.n_planes; first += kCommitPlanes) {
        const int np = a.n_planes - first < kCommitPlanes ? a.n_planes - first : kCommitPlanes;
        for (int i = 0; i < np; ++i) {
            p.codes[i] = a.codes(a.planes, first + i);
            p.scales[i] = a.scales(a.planes, first + i);
        }
        p.first = first == 0;
        for (int b0 = 0; b0 < a.B; b0 += 65535) {         // the grid's second axis
            CommitParams q = p;
            q.start += b0;
            q.path += (int64_t)b0 * a.N;
            q.n_acc += b0;
            if (q.new_lens != nullptr) q.new_lens += b0;
            if (q.block_table != nullptr) {
                q.block_table += (int64_t)b0 * a.max_pages;
            } else {
                for (int i = 0; i < np; ++i) {
                    q.codes[i] += (int64_t)b0 * a.Hkv * a.S_max * (a.D / 2);
                    q.scales[i] += (int64_t)b0 * a.Hkv * a.S_max * (a.D / 16);
                }
            }
            const int nb = a.B - b0 < 65535 ? a.B - b0 : 65535;
            commit_path_kernel<<<dim3((unsigned)np, (unsigned)nb), kThreads, 0, stream>>>(q);
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace nvfp4kv
