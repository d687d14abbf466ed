// nvfp4kv_api.cu -- the extern "C" entry points of libnvfp4kv.so declared in
// include/nvfp4kv.h: argument validation, workspace layout and launches.
// Every call is asynchronous on the caller's stream and allocates nothing.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <atomic>
#include <mutex>

#include <cuda_runtime.h>

#include "../../include/nvfp4kv.h"
#include "nvfp4kv_internal.h"

namespace nvfp4kv {

namespace {
std::mutex g_dev_mutex;
int g_sm_count[kMaxDevices] = {};   // 0 = not looked up yet
}  // namespace

int device_sm_count() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 148;
    if (dev >= kMaxDevices) {
        int n = 0;
        return (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && n > 0) ? n : 148;
    }
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    if (g_sm_count[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
            n = 148;
        g_sm_count[dev] = n;
    }
    return g_sm_count[dev];
}

cudaError_t ensure_smem_attribute(const void* kernel, int bytes, int* done_flags) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    std::lock_guard<std::mutex> lock(g_dev_mutex);
    if (!done_flags[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        done_flags[dev] = 1;
    }
    return cudaSuccess;
}

AttnWorkspace attention_workspace(int B, int Hq, int Hkv, int D) {
    AttnWorkspace w{};
    const int g = Hq / Hkv;
    w.grid = kMaxCtasPerSm * device_sm_count();
    w.counters_bytes = ((size_t)B * Hkv * sizeof(int32_t) + 255) / 256 * 256;
    w.partial_floats = (size_t)2 * w.grid * (size_t)partial_slot_floats(g, D);
    w.total_bytes = w.counters_bytes + w.partial_floats * sizeof(float);
    return w;
}

}  // namespace nvfp4kv

namespace {

using namespace nvfp4kv;

// Give-up limit of the tensor-core attention kernel's pipeline waits, in
// sleeping polls of up to 20 us each (2^16: about a second or more);
// nvfp4_set_wait_limit changes it (a testing hook).
constexpr uint32_t kDefaultWaitPolls = 1u << 16;
std::atomic<uint32_t> g_wait_polls{kDefaultWaitPolls};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool plane_ok(const nvfp4_kv_plane* pl) {
    if (pl == nullptr || pl->codes == nullptr || pl->scales == nullptr) return false;
    if (pl->B < 0 || pl->H_kv <= 0 || pl->S_max <= 0 || (pl->S_max % 16) != 0) return false;
    if (pl->D != 64 && pl->D != 128) return false;
    if (!aligned16(pl->codes) || !aligned16(pl->scales)) return false;
    return true;
}

nvfp4_status from_cuda(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

bool paged_ok(const nvfp4_kv_paged_plane* pl) {
    if (pl == nullptr || pl->codes == nullptr || pl->scales == nullptr || pl->block_table == nullptr)
        return false;
    if (pl->B < 0 || pl->H_kv <= 0 || pl->num_pages <= 0 || pl->max_pages <= 0) return false;
    if (pl->page_tokens <= 0 || (pl->page_tokens % 128) != 0) return false;
    if ((int64_t)pl->max_pages * pl->page_tokens > (int64_t)INT32_MAX) return false;
    if (pl->D != 64 && pl->D != 128) return false;
    if (!aligned16(pl->codes) || !aligned16(pl->scales)) return false;
    return true;
}

// What a launch over sequences b0.. reads: contiguous planes advance by a
// sequence stride; paged planes keep their pools and advance the block table.
struct CacheView {
    const uint8_t *kc, *ks, *vc, *vs;
    size_t seq_code_bytes, seq_scale_bytes;
    const int32_t* block_table;
    int page_tokens, max_pages, num_pages;
};

// Validation and batch-chunked launches shared by the contiguous and the
// paged attention entry points (the planes are already validated).
// Argument checks shared by every attention entry point (the planes are
// already validated): dtype, group size, pointers, alignment, softmax scale,
// and the 32-bit tile count of one launch.
nvfp4_status check_attention_args(const void* q, nvfp4_dtype q_dtype, int H_q, int B, int H_kv, int S_max,
                                  const float* d_s_tensor_k, const float* d_s_tensor_v,
                                  const int32_t* d_seq_lens, float softmax_scale, const float* out) {
    if (q_dtype != NVFP4_IN_BF16 && q_dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
    if (H_q <= 0 || (H_q % H_kv) != 0) return NVFP4_ERR_INVALID_ARG;
    if (H_q / H_kv > 16) return NVFP4_ERR_UNSUPPORTED;
    if (d_s_tensor_k == nullptr || d_s_tensor_v == nullptr || d_seq_lens == nullptr)
        return NVFP4_ERR_INVALID_ARG;
    if (!(std::isfinite(softmax_scale)) || softmax_scale < 0.0f) return NVFP4_ERR_INVALID_ARG;
    if (B == 0) return NVFP4_OK;
    if (q == nullptr || out == nullptr || !aligned16(q) || !aligned16(out)) return NVFP4_ERR_INVALID_ARG;
    // the kernels split a launch's tiles (32 tokens at the smallest) of every
    // (sequence, KV head) with 32-bit prefix sums
    const int64_t launch_tiles = (int64_t)(B < kMaxBatchPerLaunch ? B : kMaxBatchPerLaunch) * H_kv *
                                 (((int64_t)S_max + 31) / 32);
    if (launch_tiles > (int64_t)INT32_MAX) return NVFP4_ERR_UNSUPPORTED;
    return NVFP4_OK;
}

// The new tokens of an append + attention call (nullptr: attention only).
struct AppendArgs {
    const void* x_k;
    const void* x_v;
    bool f32;
    const int32_t* start_pos;
    int32_t* new_lens;
};

nvfp4_status run_attention(const void* q, nvfp4_dtype q_dtype, int H_q, int B, int H_kv, int D,
                           int S_max, const CacheView& c, const float* d_s_tensor_k,
                           const float* d_s_tensor_v, const int32_t* d_seq_lens, float softmax_scale,
                           float* out, void* workspace, size_t workspace_bytes, int32_t* d_status,
                           nvfp4_stream_t stream, const AppendArgs* app = nullptr) {
    const nvfp4_status pre = check_attention_args(q, q_dtype, H_q, B, H_kv, S_max, d_s_tensor_k,
                                                  d_s_tensor_v, d_seq_lens, softmax_scale, out);
    if (pre != NVFP4_OK || B == 0) return pre;
    const AttnWorkspace ws = attention_workspace(B, H_q, H_kv, D);
    if (workspace == nullptr || workspace_bytes < ws.total_bytes || !aligned16(workspace))
        return NVFP4_ERR_WORKSPACE;

    const size_t esz = q_dtype == NVFP4_IN_F32 ? 4 : 2;
    AttnLaunch a{};
    a.q_f32 = q_dtype == NVFP4_IN_F32;
    a.Hq = H_q;
    a.Hkv = H_kv;
    a.S_max = S_max;
    a.D = D;
    a.st_k = d_s_tensor_k;
    a.st_v = d_s_tensor_v;
    a.softmax_scale = softmax_scale > 0.0f ? softmax_scale : 1.0f / std::sqrt((float)D);
    a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ws.counters_bytes);
    a.status = d_status;
    a.grid = ws.grid;
    a.block_table = c.block_table;
    a.page_tokens = c.page_tokens;
    a.max_pages = c.max_pages;
    a.num_pages = c.num_pages;
    a.wait_polls = g_wait_polls.load();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    for (int b0 = 0; b0 < B; b0 += kMaxBatchPerLaunch) {
        const int nb = (B - b0) < kMaxBatchPerLaunch ? (B - b0) : kMaxBatchPerLaunch;
        a.B = nb;
        a.q = static_cast<const uint8_t*>(q) + (size_t)b0 * H_q * D * esz;
        a.kc = c.kc + (size_t)b0 * c.seq_code_bytes;    // paged: offsets 0, the table moves
        a.ks = c.ks + (size_t)b0 * c.seq_scale_bytes;
        a.vc = c.vc + (size_t)b0 * c.seq_code_bytes;
        a.vs = c.vs + (size_t)b0 * c.seq_scale_bytes;
        if (c.block_table != nullptr) a.block_table = c.block_table + (size_t)b0 * c.max_pages;
        a.seq_lens = d_seq_lens + b0;
        a.out = out + (size_t)b0 * H_q * D;
        a.counters = static_cast<int32_t*>(workspace) + (size_t)b0 * H_kv;
        if (app != nullptr) {
            const size_t xsz = app->f32 ? 4 : 2;
            a.x_k_new = static_cast<const uint8_t*>(app->x_k) + (size_t)b0 * H_kv * D * xsz;
            a.x_v_new = static_cast<const uint8_t*>(app->x_v) + (size_t)b0 * H_kv * D * xsz;
            a.x_f32 = app->f32;
            a.start_pos = app->start_pos + b0;
            a.new_lens = app->new_lens != nullptr ? app->new_lens + b0 : nullptr;
        }
        cudaError_t e = launch_decode_attention(a, s);
        if (e != cudaSuccess) return NVFP4_ERR_CUDA;
    }
    return NVFP4_OK;
}


}  // namespace

namespace nvfp4kv {

nvfp4_status attention_precheck(const void* q, nvfp4_dtype q_dtype, int H_q, const nvfp4_kv_plane* k,
                                const nvfp4_kv_plane* v, const float* d_s_tensor_k,
                                const float* d_s_tensor_v, const int32_t* d_seq_lens,
                                float softmax_scale, const float* out) {
    if (!plane_ok(k) || !plane_ok(v)) return NVFP4_ERR_INVALID_ARG;
    if (k->B != v->B || k->H_kv != v->H_kv || k->S_max != v->S_max || k->D != v->D)
        return NVFP4_ERR_INVALID_ARG;
    return check_attention_args(q, q_dtype, H_q, k->B, k->H_kv, k->S_max, d_s_tensor_k, d_s_tensor_v,
                                d_seq_lens, softmax_scale, out);
}

}  // namespace nvfp4kv

extern "C" {

const char* nvfp4_status_string(int status) {
    switch (status) {
        case NVFP4_OK: return "ok";
        case NVFP4_ERR_INVALID_ARG: return "invalid argument";
        case NVFP4_ERR_UNSUPPORTED: return "unsupported";
        case NVFP4_ERR_CAPACITY: return "sequence past cache capacity";
        case NVFP4_ERR_NONFINITE: return "non-finite value or scale";
        case NVFP4_ERR_CUDA: return "CUDA error";
        case NVFP4_ERR_TIMEOUT: return "device wait timed out";
        case NVFP4_ERR_WORKSPACE: return "workspace missing or too small";
        default: return "unknown status";
    }
}

const char* nvfp4_version(void) { return "nvfp4kv 0.1.0 (sm_100a)"; }

void nvfp4_set_wait_limit(int64_t polls) {
    g_wait_polls.store(polls < 0 ? kDefaultWaitPolls
                                 : (polls > (int64_t)UINT32_MAX ? UINT32_MAX : (uint32_t)polls));
}

size_t nvfp4_cache_bytes(int B, int H_kv, int S_max, int D) {
    if (B < 0 || H_kv <= 0 || S_max < 0 || D <= 0 || (D % 16) != 0) return 0;
    return (size_t)B * H_kv * S_max * (size_t)(D / 2 + D / 16);
}

nvfp4_status nvfp4_calib_tensor_scale(const void* x, nvfp4_dtype dtype, int64_t n,
                                      float* d_s_tensor, int32_t* d_status, nvfp4_stream_t stream) {
    if (d_s_tensor == nullptr || n < 0 || (n > 0 && x == nullptr)) return NVFP4_ERR_INVALID_ARG;
    if (dtype != NVFP4_IN_BF16 && dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
    const size_t esz = dtype == NVFP4_IN_F32 ? 4 : 2;
    if ((reinterpret_cast<uintptr_t>(x) % esz) != 0) return NVFP4_ERR_INVALID_ARG;
    return from_cuda(launch_calib(x, dtype == NVFP4_IN_F32, n, d_s_tensor, d_status,
                                  reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_kv_quantize_append(const void* x_new, nvfp4_dtype dtype, int n_new,
                                      const int32_t* d_start_pos, int32_t* d_new_lens,
                                      const float* d_s_tensor, const nvfp4_kv_plane* plane,
                                      int32_t* d_status, nvfp4_stream_t stream) {
    if (!plane_ok(plane) || n_new < 0 || d_s_tensor == nullptr || d_start_pos == nullptr)
        return NVFP4_ERR_INVALID_ARG;
    if (dtype != NVFP4_IN_BF16 && dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
    if (d_new_lens != nullptr && d_new_lens == d_start_pos) return NVFP4_ERR_INVALID_ARG;
    if (n_new == 0 || plane->B == 0) return NVFP4_OK;
    if (x_new == nullptr || !aligned16(x_new)) return NVFP4_ERR_INVALID_ARG;
    return from_cuda(launch_quantize_append(x_new, dtype == NVFP4_IN_F32, n_new, d_start_pos,
                                            d_new_lens, d_s_tensor, *plane, d_status,
                                            reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_kv_quantize_append_paged(const void* x_new, nvfp4_dtype dtype, int n_new,
                                            const int32_t* d_start_pos, int32_t* d_new_lens,
                                            const float* d_s_tensor,
                                            const nvfp4_kv_paged_plane* plane, int32_t* d_status,
                                            nvfp4_stream_t stream) {
    if (!paged_ok(plane) || n_new < 0 || d_s_tensor == nullptr || d_start_pos == nullptr)
        return NVFP4_ERR_INVALID_ARG;
    if (dtype != NVFP4_IN_BF16 && dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
    if (d_new_lens != nullptr && d_new_lens == d_start_pos) return NVFP4_ERR_INVALID_ARG;
    if (n_new == 0 || plane->B == 0) return NVFP4_OK;
    if (x_new == nullptr || !aligned16(x_new)) return NVFP4_ERR_INVALID_ARG;
    return from_cuda(launch_quantize_append_paged(x_new, dtype == NVFP4_IN_F32, n_new, d_start_pos,
                                                  d_new_lens, d_s_tensor, *plane, d_status,
                                                  reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_kv_quantize_append_kv(const void* x_k, const void* x_v, nvfp4_dtype dtype,
                                         int n_new, const int32_t* d_start_pos, int32_t* d_new_lens,
                                         const float* d_s_tensor_k, const float* d_s_tensor_v,
                                         const nvfp4_kv_plane* k, const nvfp4_kv_plane* v,
                                         int32_t* d_status, nvfp4_stream_t stream) {
    if (!plane_ok(k) || !plane_ok(v) || n_new < 0 || d_s_tensor_k == nullptr ||
        d_s_tensor_v == nullptr || d_start_pos == nullptr)
        return NVFP4_ERR_INVALID_ARG;
    if (k->B != v->B || k->H_kv != v->H_kv || k->S_max != v->S_max || k->D != v->D)
        return NVFP4_ERR_INVALID_ARG;
    if (dtype != NVFP4_IN_BF16 && dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
    if (d_new_lens != nullptr && d_new_lens == d_start_pos) return NVFP4_ERR_INVALID_ARG;
    if (n_new == 0 || k->B == 0) return NVFP4_OK;
    if (x_k == nullptr || x_v == nullptr || !aligned16(x_k) || !aligned16(x_v)) return NVFP4_ERR_INVALID_ARG;
    return from_cuda(launch_quantize_append_kv(x_k, x_v, dtype == NVFP4_IN_F32, n_new, d_start_pos,
                                               d_new_lens, d_s_tensor_k, d_s_tensor_v, *k, *v,
                                               d_status, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mxfp4_cache_bytes(int B, int H_kv, int S_max, int D) {
    if (B < 0 || H_kv <= 0 || S_max < 0 || D <= 0 || (D % 32) != 0) return 0;
    return (size_t)B * H_kv * S_max * (size_t)(D / 2 + D / 32);
}

nvfp4_status mxfp4_kv_quantize_append(const void* x_new, nvfp4_dtype dtype, int n_new,
                                      const int32_t* d_start_pos, int32_t* d_new_lens,
                                      const nvfp4_kv_plane* plane, int32_t* d_status,
                                      nvfp4_stream_t stream) {
    if (!plane_ok(plane) || n_new < 0 || d_start_pos == nullptr) return NVFP4_ERR_INVALID_ARG;
    if (dtype != NVFP4_IN_BF16 && dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
    if (d_new_lens != nullptr && d_new_lens == d_start_pos) return NVFP4_ERR_INVALID_ARG;
    if (n_new == 0 || plane->B == 0) return NVFP4_OK;
    if (x_new == nullptr || !aligned16(x_new)) return NVFP4_ERR_INVALID_ARG;
    return from_cuda(launch_mxfp4_quantize_append(x_new, dtype == NVFP4_IN_F32, n_new, d_start_pos,
                                                  d_new_lens, *plane, d_status,
                                                  reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_kv_dequant_fp8(const nvfp4_kv_plane* plane, const float* d_s_tensor,
                                  const int32_t* d_seq_lens, uint8_t* out_e4m3, int32_t* d_status,
                                  nvfp4_stream_t stream) {
    if (!plane_ok(plane) || d_s_tensor == nullptr || d_seq_lens == nullptr)
        return NVFP4_ERR_INVALID_ARG;
    if (plane->B == 0) return NVFP4_OK;
    if (out_e4m3 == nullptr || !aligned16(out_e4m3)) return NVFP4_ERR_INVALID_ARG;
    return from_cuda(launch_dequant_fp8(*plane, d_s_tensor, d_seq_lens, out_e4m3, d_status,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

size_t nvfp4_decode_attention_workspace(int B, int H_q, int H_kv, int D) {
    if (B < 0 || H_kv <= 0 || H_q <= 0 || (H_q % H_kv) != 0 || H_q / H_kv > 16) return 0;
    if (D != 64 && D != 128) return 0;
    return attention_workspace(B, H_q, H_kv, D).total_bytes;
}

nvfp4_status nvfp4_decode_attention(const void* q, nvfp4_dtype q_dtype, int H_q,
                                    const nvfp4_kv_plane* k, const nvfp4_kv_plane* v,
                                    const float* d_s_tensor_k, const float* d_s_tensor_v,
                                    const int32_t* d_seq_lens, float softmax_scale, float* out,
                                    void* workspace, size_t workspace_bytes, int32_t* d_status,
                                    nvfp4_stream_t stream) {
    if (!plane_ok(k) || !plane_ok(v)) return NVFP4_ERR_INVALID_ARG;
    if (k->B != v->B || k->H_kv != v->H_kv || k->S_max != v->S_max || k->D != v->D)
        return NVFP4_ERR_INVALID_ARG;
    CacheView c{};
    c.kc = k->codes; c.ks = k->scales; c.vc = v->codes; c.vs = v->scales;
    const size_t plane_tok = (size_t)k->H_kv * k->S_max;  // token slots per sequence
    c.seq_code_bytes = plane_tok * (k->D / 2);
    c.seq_scale_bytes = plane_tok * (k->D / 16);
    return run_attention(q, q_dtype, H_q, k->B, k->H_kv, k->D, k->S_max, c, d_s_tensor_k, d_s_tensor_v,
                         d_seq_lens, softmax_scale, out, workspace, workspace_bytes, d_status, stream);
}

nvfp4_status nvfp4_decode_attention_append(const void* q, nvfp4_dtype q_dtype, int H_q,
                                           const void* x_k_new, const void* x_v_new, nvfp4_dtype x_dtype,
                                           const int32_t* d_start_pos, int32_t* d_new_lens,
                                           const nvfp4_kv_plane* k, const nvfp4_kv_plane* v,
                                           const float* d_s_tensor_k, const float* d_s_tensor_v,
                                           float softmax_scale, float* out, void* workspace,
                                           size_t workspace_bytes, int32_t* d_status,
                                           nvfp4_stream_t stream) {
    if (!plane_ok(k) || !plane_ok(v)) return NVFP4_ERR_INVALID_ARG;
    if (k->B != v->B || k->H_kv != v->H_kv || k->S_max != v->S_max || k->D != v->D)
        return NVFP4_ERR_INVALID_ARG;
    if (x_dtype != NVFP4_IN_BF16 && x_dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
    if (d_start_pos == nullptr || (d_new_lens != nullptr && d_new_lens == d_start_pos))
        return NVFP4_ERR_INVALID_ARG;
    if (k->B > 0 && (x_k_new == nullptr || x_v_new == nullptr || !aligned16(x_k_new) || !aligned16(x_v_new)))
        return NVFP4_ERR_INVALID_ARG;
    CacheView c{};
    c.kc = k->codes; c.ks = k->scales; c.vc = v->codes; c.vs = v->scales;
    const size_t plane_tok = (size_t)k->H_kv * k->S_max;
    c.seq_code_bytes = plane_tok * (k->D / 2);
    c.seq_scale_bytes = plane_tok * (k->D / 16);
    AppendArgs app{x_k_new, x_v_new, x_dtype == NVFP4_IN_F32, d_start_pos, d_new_lens};
    // the lengths come from d_start_pos (start + 1); it stands in for seq_lens in the checks
    return run_attention(q, q_dtype, H_q, k->B, k->H_kv, k->D, k->S_max, c, d_s_tensor_k, d_s_tensor_v,
                         d_start_pos, softmax_scale, out, workspace, workspace_bytes, d_status, stream, &app);
}

nvfp4_status nvfp4_decode_attention_paged(const void* q, nvfp4_dtype q_dtype, int H_q,
                                          const nvfp4_kv_paged_plane* k,
                                          const nvfp4_kv_paged_plane* v,
                                          const float* d_s_tensor_k, const float* d_s_tensor_v,
                                          const int32_t* d_seq_lens, float softmax_scale,
                                          float* out, void* workspace, size_t workspace_bytes,
                                          int32_t* d_status, nvfp4_stream_t stream) {
    if (!paged_ok(k) || !paged_ok(v)) return NVFP4_ERR_INVALID_ARG;
    if (k->block_table != v->block_table || k->B != v->B || k->H_kv != v->H_kv ||
        k->page_tokens != v->page_tokens || k->max_pages != v->max_pages || k->D != v->D)
        return NVFP4_ERR_INVALID_ARG;
    CacheView c{};
    c.kc = k->codes; c.ks = k->scales; c.vc = v->codes; c.vs = v->scales;
    c.block_table = k->block_table;
    c.page_tokens = k->page_tokens;
    c.max_pages = k->max_pages;
    c.num_pages = k->num_pages < v->num_pages ? k->num_pages : v->num_pages;
    return run_attention(q, q_dtype, H_q, k->B, k->H_kv, k->D, k->max_pages * k->page_tokens, c,
                         d_s_tensor_k, d_s_tensor_v, d_seq_lens, softmax_scale, out, workspace,
                         workspace_bytes, d_status, stream);
}

nvfp4_status nvfp4_prefill_attention(const void* q, nvfp4_dtype q_dtype, int C, int H_q,
                                     const nvfp4_kv_plane* k, const nvfp4_kv_plane* v,
                                     const float* d_s_tensor_k, const float* d_s_tensor_v,
                                     const int32_t* d_start_pos, float softmax_scale, float* out,
                                     int32_t* d_status, nvfp4_stream_t stream) {
    if (!plane_ok(k) || !plane_ok(v)) return NVFP4_ERR_INVALID_ARG;
    if (k->B != v->B || k->H_kv != v->H_kv || k->S_max != v->S_max || k->D != v->D)
        return NVFP4_ERR_INVALID_ARG;
    if (q_dtype != NVFP4_IN_BF16 && q_dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
    if (C < 0 || H_q <= 0 || (H_q % k->H_kv) != 0) return NVFP4_ERR_INVALID_ARG;
    if (d_s_tensor_k == nullptr || d_s_tensor_v == nullptr || d_start_pos == nullptr)
        return NVFP4_ERR_INVALID_ARG;
    if (!(std::isfinite(softmax_scale)) || softmax_scale < 0.0f) return NVFP4_ERR_INVALID_ARG;
    // the tensor-core prefill takes bf16 queries (exact in its f16 operand
    // after a power-of-two row scaling, down to 2^-31 of the row maximum); an
    // fp32 query would need a second f16 term and its shared memory
    if (k->D != 128 || H_q / k->H_kv > 128 || q_dtype != NVFP4_IN_BF16) return NVFP4_ERR_UNSUPPORTED;
    if (k->B == 0 || C == 0) return NVFP4_OK;
    if (q == nullptr || out == nullptr || !aligned16(q) || !aligned16(out)) return NVFP4_ERR_INVALID_ARG;
    const int g = H_q / k->H_kv, cq = 128 / g;
    if ((int64_t)k->B * k->H_kv * ((C + cq - 1) / cq) > (int64_t)INT32_MAX) return NVFP4_ERR_UNSUPPORTED;
    return from_cuda(launch_prefill_tc(q, q_dtype == NVFP4_IN_F32, C, H_q, *k, *v, d_s_tensor_k, d_s_tensor_v,
                                       d_start_pos, softmax_scale, out, d_status,
                                       g_wait_polls.load(std::memory_order_relaxed),
                                       reinterpret_cast<cudaStream_t>(stream)));
}


// ---------------------------------------------------------------------------
// A step of tree-drafted decoding.  The contiguous and the paged entry points
// differ in the addressing only.
// ---------------------------------------------------------------------------
}  // extern "C"

namespace {

// The shape and addressing that a call's K and V planes share.
struct CachePair {
    uint8_t *kc, *ks, *vc, *vs;
    int B, H_kv, S_max, D;
    const int32_t* block_table;
    int page_tokens, max_pages, num_pages;
};

bool cache_pair(const nvfp4_kv_plane* k, const nvfp4_kv_plane* v, CachePair& c) {
    if (!plane_ok(k) || !plane_ok(v)) return false;
    if (k->B != v->B || k->H_kv != v->H_kv || k->S_max != v->S_max || k->D != v->D) return false;
    c = CachePair{k->codes, k->scales, v->codes, v->scales, k->B, k->H_kv, k->S_max, k->D, nullptr, 0, 0, 0};
    return true;
}

bool cache_pair(const nvfp4_kv_paged_plane* k, const nvfp4_kv_paged_plane* v, CachePair& c) {
    if (!paged_ok(k) || !paged_ok(v)) return false;
    if (k->block_table != v->block_table || k->B != v->B || k->H_kv != v->H_kv ||
        k->page_tokens != v->page_tokens || k->max_pages != v->max_pages || k->D != v->D)
        return false;
    c = CachePair{k->codes, k->scales, v->codes, v->scales, k->B, k->H_kv, k->max_pages * k->page_tokens, k->D,
                  k->block_table, k->page_tokens, k->max_pages,
                  k->num_pages < v->num_pages ? k->num_pages : v->num_pages};
    return true;
}

// A plane's memory: bytes_per_slot for every token slot of every KV head.
struct Range {
    uintptr_t lo, hi;
};
int64_t plane_slots(const nvfp4_kv_plane& p) { return (int64_t)p.B * p.H_kv * p.S_max; }
int64_t plane_slots(const nvfp4_kv_paged_plane& p) { return (int64_t)p.num_pages * p.H_kv * p.page_tokens; }
template <class Plane>
Range plane_range(const Plane& p, const uint8_t* at, int bytes_per_slot) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(at);
    return {lo, lo + (uintptr_t)(plane_slots(p) * bytes_per_slot)};
}
bool share(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// Whether two planes (already validated) that a launch writes share memory.
template <class Plane>
bool planes_share(const Plane& a, const Plane& b) {
    return share(plane_range(a, a.codes, a.D / 2), plane_range(b, b.codes, b.D / 2)) ||
           share(plane_range(a, a.scales, a.D / 16), plane_range(b, b.scales, b.D / 16));
}

// Whether na and nb 32-bit values share memory (nullptr: none).
bool overlap32(const void* a, int64_t na, const void* b, int64_t nb) {
    if (a == nullptr || b == nullptr) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + 4 * (uintptr_t)nb && y < x + 4 * (uintptr_t)na;
}

nvfp4_status run_qk_norm_rope_append(const void* x_q, const void* x_k, const void* x_v, nvfp4_dtype dtype, int n_new,
                                     int H_q, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                     const void* w_q, const void* w_k, float eps, const float* rope_table,
                                     int rope_positions, int rope_dims, int rope_interleaved,
                                     const int32_t* d_positions, const int32_t* d_start_pos,
                                     const int32_t* d_n_valid, int32_t* d_new_lens, const float* d_s_tensor_k,
                                     const float* d_s_tensor_v, const CachePair& c, bool shared, void* q_out,
                                     int32_t* d_status, nvfp4_stream_t stream) {
    if (dtype != NVFP4_IN_BF16 && dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
    if (n_new < 0 || H_q <= 0 || d_s_tensor_k == nullptr || d_s_tensor_v == nullptr || d_start_pos == nullptr)
        return NVFP4_ERR_INVALID_ARG;
    // a block writes its sequence's length while others still read these
    if (overlap32(d_new_lens, c.B, d_start_pos, c.B) || overlap32(d_new_lens, c.B, d_n_valid, c.B) ||
        overlap32(d_new_lens, c.B, d_positions, (int64_t)c.B * n_new))
        return NVFP4_ERR_INVALID_ARG;
    if (!std::isfinite(eps)) return NVFP4_ERR_INVALID_ARG;
    if (rope_table == nullptr ? rope_dims != 0 : (rope_dims <= 0 || rope_dims > c.D || rope_dims % 16 != 0 ||
                                                  rope_positions <= 0 || !aligned16(rope_table)))
        return NVFP4_ERR_INVALID_ARG;
    const int per16 = dtype == NVFP4_IN_F32 ? 4 : 8;
    const int64_t dq = (int64_t)H_q * c.D, dk = (int64_t)c.H_kv * c.D;
    NormRopeLaunch a{};
    a.sq = q_stride == 0 ? dq : q_stride;
    a.sk = k_stride == 0 ? dk : k_stride;
    a.sv = v_stride == 0 ? dk : v_stride;
    if (a.sq < dq || a.sk < dk || a.sv < dk || a.sq % per16 != 0 || a.sk % per16 != 0 || a.sv % per16 != 0)
        return NVFP4_ERR_INVALID_ARG;
    if (n_new == 0 || c.B == 0) return NVFP4_OK;
    if (x_q == nullptr || x_k == nullptr || x_v == nullptr || q_out == nullptr || !aligned16(x_q) || !aligned16(x_k) ||
        !aligned16(x_v) || !aligned16(q_out) || !aligned16(w_q) || !aligned16(w_k))
        return NVFP4_ERR_INVALID_ARG;
    // the kernel counts (token, group of four heads) tasks in 31 bits
    if ((int64_t)c.B * n_new > (int64_t)INT32_MAX / ((H_q + 2 * (int64_t)c.H_kv + 3) / 4 + 1))
        return NVFP4_ERR_UNSUPPORTED;
    if (shared) return NVFP4_ERR_INVALID_ARG;          // K's and V's blocks are written at the same time
    a.xq = x_q; a.xk = x_k; a.xv = x_v;
    a.f32 = dtype == NVFP4_IN_F32;
    a.wq = w_q; a.wk = w_k;
    a.table = rope_table;
    a.positions = d_positions; a.start = d_start_pos; a.n_valid = d_n_valid; a.new_lens = d_new_lens;
    a.st_k = d_s_tensor_k; a.st_v = d_s_tensor_v;
    a.q_out = q_out;
    a.kc = c.kc; a.ks = c.ks; a.vc = c.vc; a.vs = c.vs;
    a.block_table = c.block_table;
    a.status = d_status;
    a.B = c.B; a.n = n_new; a.Hq = H_q; a.Hkv = c.H_kv; a.D = c.D; a.S_max = c.S_max;
    a.R = rope_dims; a.P = rope_positions;
    a.page_tokens = c.page_tokens; a.max_pages = c.max_pages; a.num_pages = c.num_pages;
    a.eps = eps;
    a.interleaved = rope_interleaved != 0;
    return from_cuda(launch_qk_norm_rope_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status run_tree_attention(const void* q, nvfp4_dtype q_dtype, int N, int H_q, const CachePair& c,
                                const float* d_s_tensor_k, const float* d_s_tensor_v, const int32_t* d_start_pos,
                                const int32_t* d_n_nodes, const int32_t* d_tree_mask, int64_t mask_stride,
                                float softmax_scale, void* out, nvfp4_dtype out_dtype, void* workspace,
                                size_t workspace_bytes, int32_t* d_status, nvfp4_stream_t stream) {
    if (q_dtype != NVFP4_IN_BF16 && q_dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
    if (out_dtype != NVFP4_IN_BF16 && out_dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
    if (N < 0 || H_q <= 0 || (H_q % c.H_kv) != 0) return NVFP4_ERR_INVALID_ARG;
    if (d_s_tensor_k == nullptr || d_s_tensor_v == nullptr || d_start_pos == nullptr) return NVFP4_ERR_INVALID_ARG;
    if (!(std::isfinite(softmax_scale)) || softmax_scale < 0.0f) return NVFP4_ERR_INVALID_ARG;
    const int64_t words = ((int64_t)N + 31) / 32;
    if (d_tree_mask != nullptr && mask_stride != 0 && mask_stride < N * words) return NVFP4_ERR_INVALID_ARG;
    if (q_dtype != NVFP4_IN_BF16 || N > kTreeMaxNodes || H_q / c.H_kv > 128) return NVFP4_ERR_UNSUPPORTED;
    if (c.B == 0 || N == 0) return NVFP4_OK;
    if (q == nullptr || out == nullptr || !aligned16(q) || !aligned16(out)) return NVFP4_ERR_INVALID_ARG;
    // the kernel numbers a launch's (unit, 128-token tile) pairs in 32 bits
    const int64_t units = (int64_t)(c.B < kMaxBatchPerLaunch ? c.B : kMaxBatchPerLaunch) * c.H_kv *
                          (((int64_t)N * (H_q / c.H_kv) + 127) / 128);
    const int64_t tiles = ((int64_t)c.S_max + 127) / 128;
    if (units > (int64_t)INT32_MAX / tiles) return NVFP4_ERR_UNSUPPORTED;
    if (tiles * 128 > (int64_t)INT32_MAX) return NVFP4_ERR_UNSUPPORTED;   // and their tokens
    if (workspace == nullptr || !aligned16(workspace) ||
        workspace_bytes < tree_attention_workspace(c.B, N, H_q, c.H_kv, c.D))
        return NVFP4_ERR_WORKSPACE;
    // A unit writes the rows whose queries it has read, and no others: bf16 outputs may lie
    // over the queries exactly, any other overlap reaches queries that are still to be read.
    const int64_t elements = (int64_t)c.B * N * H_q * c.D;
    if (!(q == out && out_dtype == NVFP4_IN_BF16) &&
        overlap32(q, elements / 2, out, out_dtype == NVFP4_IN_BF16 ? elements / 2 : elements))
        return NVFP4_ERR_INVALID_ARG;
    TreeLaunch a{};
    a.q = q;
    a.out_bf16 = out_dtype == NVFP4_IN_BF16;
    a.B = c.B; a.N = N; a.Hq = H_q; a.Hkv = c.H_kv; a.D = c.D; a.S_max = c.S_max;
    a.kc = c.kc; a.ks = c.ks; a.vc = c.vc; a.vs = c.vs;
    a.st_k = d_s_tensor_k; a.st_v = d_s_tensor_v;
    a.start = d_start_pos; a.n_nodes = d_n_nodes;
    a.mask = d_tree_mask; a.mask_stride = mask_stride;
    a.softmax_scale = softmax_scale;
    a.out = out;
    a.partials = static_cast<float*>(workspace);
    a.status = d_status;
    a.block_table = c.block_table;
    a.page_tokens = c.page_tokens; a.max_pages = c.max_pages; a.num_pages = c.num_pages;
    a.wait_polls = g_wait_polls.load();
    return from_cuda(launch_tree_attention(a, reinterpret_cast<cudaStream_t>(stream)));
}

// Whether two of n ranges share a byte.  No memory is allocated: more than 256 are
// compared pair by pair.
template <class F>
bool any_overlap(int n, F range) {
    bool rising = true;                               // as the slices of one tensor are
    for (int i = 1; rising && i < n; ++i) rising = range(i - 1).hi <= range(i).lo;
    if (rising) return false;
    constexpr int kMost = 256;
    if (n > kMost) {
        for (int i = 1; i < n; ++i) {
            const Range a = range(i);
            for (int j = 0; j < i; ++j) {
                const Range b = range(j);
                if (share(a, b)) return true;
            }
        }
        return false;
    }
    Range r[kMost];
    for (int i = 0; i < n; ++i) r[i] = range(i);
    std::sort(r, r + n, [](const Range& a, const Range& b) { return a.lo < b.lo; });
    for (int i = 1; i < n; ++i)
        if (r[i - 1].hi > r[i].lo) return true;
    return false;
}

template <class Plane>
nvfp4_status run_commit_path(const Plane* planes, int n_planes, int N, const int32_t* d_start_pos,
                             const int32_t* d_path, const int32_t* d_n_accepted, int32_t* d_new_lens,
                             int32_t* d_status, nvfp4_stream_t stream) {
    if (n_planes < 0 || N < 0 || (n_planes > 0 && planes == nullptr)) return NVFP4_ERR_INVALID_ARG;
    if (d_start_pos == nullptr || (d_path == nullptr && N > 0) || d_n_accepted == nullptr) return NVFP4_ERR_INVALID_ARG;
    const int64_t B = n_planes > 0 ? planes[0].B : 1;
    // a block writes its sequence's length while others still read these
    if (overlap32(d_new_lens, B, d_start_pos, B) || overlap32(d_new_lens, B, d_n_accepted, B) ||
        overlap32(d_new_lens, B, d_path, B * N))
        return NVFP4_ERR_INVALID_ARG;
    if (N > kTreeMaxNodes) return NVFP4_ERR_UNSUPPORTED;
    if (n_planes == 0) return NVFP4_OK;
    CommitLaunch a{};
    CachePair c{};
    a.num_pages = INT32_MAX;
    for (int i = 0; i < n_planes; ++i) {
        if (!cache_pair(&planes[0], &planes[i], c)) return NVFP4_ERR_INVALID_ARG;
        if (c.num_pages < a.num_pages) a.num_pages = c.num_pages;
    }
    // planes are moved at the same time: none may be given twice
    if (any_overlap(n_planes, [&](int i) { return plane_range(planes[i], planes[i].codes, c.D / 2); }) ||
        any_overlap(n_planes, [&](int i) { return plane_range(planes[i], planes[i].scales, c.D / 16); }))
        return NVFP4_ERR_INVALID_ARG;
    if (c.B == 0 || N == 0) return NVFP4_OK;
    a.planes = planes;
    a.codes = [](const void* p, int i) { return static_cast<const Plane*>(p)[i].codes; };
    a.scales = [](const void* p, int i) { return static_cast<const Plane*>(p)[i].scales; };
    a.n_planes = n_planes;
    a.start = d_start_pos; a.path = d_path; a.n_acc = d_n_accepted;
    a.new_lens = d_new_lens; a.status = d_status;
    a.block_table = c.block_table;
    a.page_tokens = c.page_tokens; a.max_pages = c.max_pages;
    a.B = c.B; a.Hkv = c.H_kv; a.S_max = c.S_max; a.D = c.D; a.N = N;
    return from_cuda(launch_commit_path(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

#define NVFP4_NORM_ROPE_ENTRY(NAME, PLANE)                                                                            \
    nvfp4_status NAME(const void* x_q, const void* x_k, const void* x_v, nvfp4_dtype dtype, int n_new, int H_q,       \
                      int64_t q_stride, int64_t k_stride, int64_t v_stride, const void* w_q, const void* w_k,         \
                      float eps, const float* rope_table, int rope_positions, int rope_dims, int rope_interleaved,    \
                      const int32_t* d_positions, const int32_t* d_start_pos, const int32_t* d_n_valid,               \
                      int32_t* d_new_lens, const float* d_s_tensor_k, const float* d_s_tensor_v, const PLANE* k,      \
                      const PLANE* v, void* q_out, int32_t* d_status, nvfp4_stream_t stream) {                        \
        CachePair c{};                                                                                                \
        if (!cache_pair(k, v, c)) return NVFP4_ERR_INVALID_ARG;                                                       \
        return run_qk_norm_rope_append(x_q, x_k, x_v, dtype, n_new, H_q, q_stride, k_stride, v_stride, w_q, w_k, eps, \
                                       rope_table, rope_positions, rope_dims, rope_interleaved, d_positions,          \
                                       d_start_pos, d_n_valid, d_new_lens, d_s_tensor_k, d_s_tensor_v, c,             \
                                       planes_share(*k, *v), q_out, d_status, stream);                                \
    }
NVFP4_NORM_ROPE_ENTRY(nvfp4_qk_norm_rope_append, nvfp4_kv_plane)
NVFP4_NORM_ROPE_ENTRY(nvfp4_qk_norm_rope_append_paged, nvfp4_kv_paged_plane)
#undef NVFP4_NORM_ROPE_ENTRY

size_t nvfp4_tree_attention_workspace(int B, int N, int H_q, int H_kv, int D) {
    if (B < 0 || N < 0 || N > kTreeMaxNodes || H_kv <= 0 || H_q <= 0 || (H_q % H_kv) != 0 || H_q / H_kv > 128) return 0;
    if (D != 64 && D != 128) return 0;
    return tree_attention_workspace(B, N, H_q, H_kv, D);
}

#define NVFP4_TREE_ENTRY(NAME, PLANE)                                                                                \
    nvfp4_status NAME(const void* q, nvfp4_dtype q_dtype, int N, int H_q, const PLANE* k, const PLANE* v,            \
                      const float* d_s_tensor_k, const float* d_s_tensor_v, const int32_t* d_start_pos,              \
                      const int32_t* d_n_nodes, const int32_t* d_tree_mask, int64_t mask_stride,                     \
                      float softmax_scale, void* out, nvfp4_dtype out_dtype, void* workspace,                        \
                      size_t workspace_bytes, int32_t* d_status, nvfp4_stream_t stream) {                            \
        CachePair c{};                                                                                               \
        if (!cache_pair(k, v, c)) return NVFP4_ERR_INVALID_ARG;                                                      \
        return run_tree_attention(q, q_dtype, N, H_q, c, d_s_tensor_k, d_s_tensor_v, d_start_pos, d_n_nodes,         \
                                  d_tree_mask, mask_stride, softmax_scale, out, out_dtype, workspace,                \
                                  workspace_bytes, d_status, stream);                                                \
    }
NVFP4_TREE_ENTRY(nvfp4_tree_attention, nvfp4_kv_plane)
NVFP4_TREE_ENTRY(nvfp4_tree_attention_paged, nvfp4_kv_paged_plane)
#undef NVFP4_TREE_ENTRY

nvfp4_status nvfp4_verify_drafts(const void* target_probs, const void* draft_probs, nvfp4_dtype dtype, int B, int N,
                                 int V, const int32_t* d_tokens, const int32_t* d_parents, int parents_shared,
                                 const float* d_u_accept, const float* d_u_sample, const int32_t* d_n_nodes,
                                 int32_t* d_path, int32_t* d_n_accepted, int32_t* d_next_token, int32_t* d_status,
                                 nvfp4_stream_t stream) {
    if (dtype != NVFP4_IN_BF16 && dtype != NVFP4_IN_F32) return NVFP4_ERR_INVALID_ARG;
    if (B < 0 || N <= 0 || V <= 0) return NVFP4_ERR_INVALID_ARG;
    if (N > kTreeMaxNodes || B > (1 << 24)) return NVFP4_ERR_UNSUPPORTED;
    if (B == 0) return NVFP4_OK;
    if (target_probs == nullptr || d_tokens == nullptr || d_parents == nullptr || d_u_accept == nullptr ||
        d_u_sample == nullptr || d_path == nullptr || d_n_accepted == nullptr || d_next_token == nullptr)
        return NVFP4_ERR_INVALID_ARG;
    // A path is written while other blocks still read the inputs; the other outputs after
    // a sequence's last pass, when its n_nodes has been read (the accepted counts may
    // take its place).
    const int64_t nodes = (int64_t)B * N, np = parents_shared ? N : nodes;
    const struct { const void* at; int64_t n; } out[3] = {{d_path, nodes}, {d_n_accepted, B}, {d_next_token, B}},
        in[4] = {{d_tokens, nodes}, {d_parents, np}, {d_u_accept, nodes}, {d_u_sample, B}};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 4; ++j)
            if (overlap32(out[i].at, out[i].n, in[j].at, in[j].n)) return NVFP4_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap32(out[i].at, out[i].n, out[j].at, out[j].n)) return NVFP4_ERR_INVALID_ARG;
    }
    if (overlap32(d_path, nodes, d_n_nodes, B)) return NVFP4_ERR_INVALID_ARG;
    const uintptr_t esz = dtype == NVFP4_IN_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(target_probs) % esz != 0 || reinterpret_cast<uintptr_t>(draft_probs) % esz != 0)
        return NVFP4_ERR_INVALID_ARG;
    VerifyLaunch a{};
    a.p = target_probs; a.d = draft_probs;
    a.f32 = dtype == NVFP4_IN_F32;
    a.tokens = d_tokens; a.parents = d_parents;
    a.parents_shared = parents_shared != 0;
    a.u_accept = d_u_accept; a.u_sample = d_u_sample;
    a.n_nodes = d_n_nodes;
    a.path = d_path; a.n_acc = d_n_accepted; a.next = d_next_token; a.status = d_status;
    a.B = B; a.N = N; a.V = V;
    return from_cuda(launch_verify_drafts(a, reinterpret_cast<cudaStream_t>(stream)));
}

nvfp4_status nvfp4_kv_commit_path(const nvfp4_kv_plane* planes, int n_planes, int N, const int32_t* d_start_pos,
                                  const int32_t* d_path, const int32_t* d_n_accepted, int32_t* d_new_lens,
                                  int32_t* d_status, nvfp4_stream_t stream) {
    return run_commit_path(planes, n_planes, N, d_start_pos, d_path, d_n_accepted, d_new_lens, d_status, stream);
}

nvfp4_status nvfp4_kv_commit_path_paged(const nvfp4_kv_paged_plane* planes, int n_planes, int N,
                                        const int32_t* d_start_pos, const int32_t* d_path,
                                        const int32_t* d_n_accepted, int32_t* d_new_lens, int32_t* d_status,
                                        nvfp4_stream_t stream) {
    return run_commit_path(planes, n_planes, N, d_start_pos, d_path, d_n_accepted, d_new_lens, d_status, stream);
}

}  // extern "C"
