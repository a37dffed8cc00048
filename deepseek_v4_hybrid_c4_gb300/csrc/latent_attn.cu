// Dense attention over ranges of the paged latent cache (K = V = the bf16 row):
//   csa_prefix_attn   one token per request, the batch's first rows shared
//   csa_window_attn   causal, a sliding window and the first tokens of the sequence
//
//   l_j = scale * q . K_j,  o = sum_j softmax(l)_j V_j,  lse = ln sum_j exp(l_j)
//
// One warp per query row: a lane holds 16 of the row's 512 dims, a key's dot product is a warp
// reduction, and the softmax is the running one (maximum m, sum l, O rescaled when m moves).
#include "common.cuh"
#include "internal.h"

namespace csa {

struct LatArgs {
    const uint16_t* q;
    int H;
    float scale;
    DPaged kv;
    int64_t table_pages;       // entries of a request's page table
    // prefix: request b = row / H sees rows [0, n_rows[b]); rows below n_shared through table row 0
    const int64_t* n_rows;
    int64_t n_shared, max_rows;
    // window (q_offsets set): B sequences
    const int64_t* q_offsets;
    const int64_t* n_tokens;
    int64_t total_q, max_q;
    int window, n_sink;
    int B;
    uint16_t* out;
    float* lse;
    int32_t* status;
};

__device__ __forceinline__ const uint8_t* lat_row(const LatArgs& a, int b, int64_t r) {
    if (r / a.kv.rpp >= a.table_pages) {
        raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
        return nullptr;
    }
    return row_addr(a.kv, b, r, ROW_BYTES, a.status);
}

__global__ void __launch_bounds__(256) lat_rows_kernel(LatArgs a, int64_t rows) {
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (row >= rows) return;
    int b = 0;
    int64_t sink_hi = 0, lo = 0, hi = 0;
    if (a.q_offsets) {
        const int64_t t = row / a.H;
        int l = 0, r = a.B;  // the last sequence that starts at or before t
        while (r - l > 1) {
            const int m = (l + r) / 2;
            if (__ldg(a.q_offsets + m) <= t) l = m;
            else r = m;
        }
        b = l;
        const int64_t q0 = __ldg(a.q_offsets + b), q1 = __ldg(a.q_offsets + b + 1);
        if (t < q0 || t >= q1) return;
        if (q1 > a.total_q || q1 - q0 > a.max_q) {
            raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
            return;
        }
        const int64_t pos = __ldg(a.n_tokens + b) - (q1 - t);
        hi = pos + 1 > 0 ? pos + 1 : 0;
        lo = hi > a.window ? hi - a.window : 0;
        sink_hi = a.n_sink < lo ? a.n_sink : lo;
    } else {
        b = (int)(row / a.H);
        hi = __ldg(a.n_rows + b);
        if (hi > a.max_rows || hi < 0) {
            raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
            hi = hi < 0 ? 0 : a.max_rows;
        }
    }
    float q[16], o[16];
    const uint4* qp = reinterpret_cast<const uint4*>(a.q + row * D + lane * 16);
    const uint4 q0 = qp[0], q1 = qp[1];
    const uint32_t qw[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        q[2 * e] = bf16lo(qw[e]) * a.scale;
        q[2 * e + 1] = bf16hi(qw[e]) * a.scale;
        o[2 * e] = o[2 * e + 1] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    auto attend = [&](int64_t j) {
        const uint8_t* p = lat_row(a, j < a.n_shared ? 0 : b, j);
        if (!p) return;
        const uint4* kp = reinterpret_cast<const uint4*>(p) + lane * 2;
        const uint4 k0 = __ldg(kp), k1 = __ldg(kp + 1);
        const uint32_t kw[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x = fmaf(q[2 * e + 1], bf16hi(kw[e]), fmaf(q[2 * e], bf16lo(kw[e]), x));
        for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
        const float mn = fmaxf(m, x);
        const float alpha = m == -INFINITY ? 0.f : expf(m - mn), w = expf(x - mn);
        m = mn;
        l = l * alpha + w;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            o[2 * e] = fmaf(w, bf16lo(kw[e]), o[2 * e] * alpha);
            o[2 * e + 1] = fmaf(w, bf16hi(kw[e]), o[2 * e + 1] * alpha);
        }
    };
    for (int64_t j = 0; j < sink_hi; ++j) attend(j);
    for (int64_t j = lo; j < hi; ++j) attend(j);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
    uint4* op = reinterpret_cast<uint4*>(a.out + row * D + lane * 16);
    op[0] = make_uint4(w[0], w[1], w[2], w[3]);
    op[1] = make_uint4(w[4], w[5], w[6], w[7]);
    if (lane == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

// What both calls ask of the cache: a page table, pages of whole 1,024-byte rows, row ids below 2^31.
static csa_status check_cache(const csa_paged& kv, int64_t page_table_stride) {
    const csa_status rc = check_paged(kv, kLatentRowBytes);
    if (rc) return rc;
    if (!kv.page_table || !al4(kv.page_table) || page_table_stride < 1) return CSA_ERR_INVALID_ARG;
    if (kv.page_stride_bytes % kLatentRowBytes) return CSA_ERR_UNSUPPORTED;
    const int64_t per_page = kv.page_stride_bytes / kLatentRowBytes;
    if (per_page > 0x7FFFFFFFLL || kv.n_pages > 0x7FFFFFFFLL / per_page) return CSA_ERR_UNSUPPORTED;
    return CSA_OK;
}

static DPaged cache_of(const csa_paged& kv, int64_t page_table_stride) {
    DPaged d;
    d.base = static_cast<const uint8_t*>(kv.base);
    d.pt = kv.page_table;
    d.pt_stride = page_table_stride;
    d.page_stride = kv.page_stride_bytes;
    d.n_pages = kv.n_pages;
    d.rpp = kv.rows_per_page;
    d.qpr = 1;
    return d;
}

static csa_status check_prefix(int32_t B, int32_t H, int64_t n_shared, int64_t max_rows) {
    if (H < 1 || H > 128 || B < 1 || B > 65535 || max_rows > 0x7FFFFFFFLL) return CSA_ERR_UNSUPPORTED;
    if (n_shared < 0 || max_rows < n_shared) return CSA_ERR_INVALID_ARG;
    return CSA_OK;
}

static csa_status check_window(int32_t B, int32_t H, int64_t total_q, int64_t max_q, int32_t window, int32_t n_sink) {
    if (H < 1 || H > 128 || B < 1 || B > 65535 || window > (1 << 30) || n_sink > (1 << 30)) return CSA_ERR_UNSUPPORTED;
    if (window < 1 || n_sink < 0 || total_q < 0 || max_q < 1) return CSA_ERR_INVALID_ARG;
    if (total_q > 0x7FFFFFFFLL / H || max_q > 0x7FFFFFFFLL) return CSA_ERR_UNSUPPORTED;
    return CSA_OK;
}

static cudaError_t launch_rows(const LatArgs& a, int64_t rows, cudaStream_t s) {
    lat_rows_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(a, rows);
    return cudaGetLastError();
}

}  // namespace csa

using namespace csa;

extern "C" {

size_t csa_prefix_attn_workspace_size(int32_t B, int32_t H, int64_t n_shared, int64_t max_rows) {
    return check_prefix(B, H, n_shared, max_rows) ? 0 : 256;
}

csa_status csa_prefix_attn(const void* q, int32_t B, int32_t H, float scale, csa_paged kv, int64_t page_table_stride,
                           int64_t n_shared, const int64_t* n_rows, int64_t max_rows, void* out, float* lse,
                           void* workspace, size_t ws_bytes, void* stream) {
    csa_status rc = check_prefix(B, H, n_shared, max_rows);
    if (rc) return rc;
    if (!q || !al16(q) || !out || !al16(out) || (lse && !al4(lse)) || !n_rows || !al8(n_rows))
        return CSA_ERR_INVALID_ARG;
    if ((rc = check_cache(kv, page_table_stride))) return rc;
    if (page_table_stride < (max_rows + kv.rows_per_page - 1) / kv.rows_per_page) return CSA_ERR_INVALID_ARG;
    if (!workspace || !al16(workspace) || ws_bytes < csa_prefix_attn_workspace_size(B, H, n_shared, max_rows))
        return CSA_ERR_WORKSPACE;
    LatArgs a = {};
    a.status = device_status_ptr();
    if (!a.status) return CSA_ERR_CUDA;
    a.q = static_cast<const uint16_t*>(q);
    a.H = H;
    a.scale = scale;
    a.kv = cache_of(kv, page_table_stride);
    a.table_pages = page_table_stride;
    a.n_rows = n_rows;
    a.n_shared = n_shared;
    a.max_rows = max_rows;
    a.B = B;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    return from_cuda(launch_rows(a, (int64_t)B * H, static_cast<cudaStream_t>(stream)));
}

size_t csa_window_attn_workspace_size(int32_t B, int32_t H, int64_t total_q, int64_t max_q, int32_t window,
                                      int32_t n_sink) {
    (void)B, (void)H, (void)total_q, (void)max_q, (void)window, (void)n_sink;
    return 0;
}

csa_status csa_window_attn(const void* q, int32_t H, float scale, csa_paged kv_raw, int64_t page_table_stride,
                           int32_t B, const int64_t* q_offsets, const int64_t* n_tokens, int64_t total_q,
                           int64_t max_q, int32_t window, int32_t n_sink, void* out, float* lse, void* workspace,
                           size_t ws_bytes, void* stream) {
    csa_status rc = check_window(B, H, total_q, max_q, window, n_sink);
    if (rc) return rc;
    if (!q || !al16(q) || !out || !al16(out) || (lse && !al4(lse)) || !q_offsets || !al8(q_offsets) || !n_tokens ||
        !al8(n_tokens))
        return CSA_ERR_INVALID_ARG;
    if ((rc = check_cache(kv_raw, page_table_stride))) return rc;
    const size_t need = csa_window_attn_workspace_size(B, H, total_q, max_q, window, n_sink);
    if (need && (!workspace || !al16(workspace) || ws_bytes < need)) return CSA_ERR_WORKSPACE;
    if (total_q == 0) return CSA_OK;
    LatArgs a = {};
    a.status = device_status_ptr();
    if (!a.status) return CSA_ERR_CUDA;
    a.q = static_cast<const uint16_t*>(q);
    a.H = H;
    a.scale = scale;
    a.kv = cache_of(kv_raw, page_table_stride);
    a.table_pages = page_table_stride;
    a.q_offsets = q_offsets;
    a.n_tokens = n_tokens;
    a.total_q = total_q;
    a.max_q = max_q;
    a.window = window;
    a.n_sink = n_sink;
    a.B = B;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    return from_cuda(launch_rows(a, total_q * H, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
