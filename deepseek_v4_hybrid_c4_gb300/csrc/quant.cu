// The quantised latent cache: rows written (csa_quant_write) and read back (csa_quant_read).
//
//   k = max(-117, the least k with max |x_i| <= 448 2^k) over the 128 dims of a block,  c_i = e4m3(x_i 2^-k)
//
// Both are bound by memory: 1,024 bytes of bf16 and 516 of codes and scales a row.  A warp takes four rows (one, where
// there are few), with their loads in flight together; a row's sequence is found by a search over the offsets 32 at a
// time, beside the loads of the new rows.  261K rows written: 65 us, 6.2 TB/s, 93 percent of the copy rate; 279K
// read back: 68 us, 6.3 TB/s, 94 percent (110 and 82 us before a warp took four rows and a lane 16 dims of each).
#include <cuda_fp8.h>

#include <algorithm>

#include "internal.h"
#include "quant.cuh"

namespace csa {

constexpr int QC_T = 256;
// Rows of a warp where there are many.  One and four: writes of 12K, 25K, 49K and 98K rows 5.1 and 4.9 us, 9.7 and 10.5, 16.9
// and 17.1, 30.6 and 27.5; reads 5.5 and 5.4, 9.2 and 8.5, 16.9 and 15.3, 30.6 and 26.5.
constexpr int QC_W = 4, QC_R = 4;
constexpr int64_t QC_MANY = 16384;

struct QuantArgs {
    const uint8_t* rows;        // write: bf16 [total][512]
    uint8_t* out;               // read: bf16 [total][512]
    DPaged kv;
    int64_t table_pages;
    int B;
    const int64_t* offsets;
    const int64_t* n_tokens;
    int64_t total, max_rows;
    bool wide_out;              // read: out is 32-byte aligned
    int32_t* status;
};

constexpr int64_t QC_MAX_TOKENS = 0x7FFFFFFF - 127;

// Page and slot of rows [row0, row0 + R) of the batch, lane i with row i's (a warp): page -1 where a row has no place in
// the pool, -2 where no sequence covers it.
template <int R>
CSA_DEV int2 places(const QuantArgs& a, int64_t row0, int lane) {
    int page = -2, pos = -1, seq = 0, b = 0;
    int64_t end = -1, q0 = 0, q1 = 0, nt = 0;
#pragma unroll 1
    for (int i = 0; i < R && row0 + i < a.total; ++i) {
        const int64_t row = row0 + i;
        if (row >= end) {
            b = warp_seq_of(a.offsets, a.B, row, lane);
            q0 = __ldg(a.offsets + b), q1 = __ldg(a.offsets + b + 1), nt = __ldg(a.n_tokens + b);
            const bool valid = q0 >= 0 && q1 >= q0 && q1 <= a.total && q1 - q0 <= a.max_rows && nt <= QC_MAX_TOKENS;
            if (!valid && lane == 0) raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
            if (!valid) q1 = q0;  // covers nothing
            end = row < q1 ? q1 : row + 1;
        }
        if (lane == i && row >= q0 && row < q1) {
            page = -1;
            pos = nt >= q1 - row ? (int)(nt - (q1 - row)) : -1;
            seq = b;
        }
    }
    int slot = 0;
    if (pos >= 0) {
        const int lp = pos / a.kv.rpp;
        slot = pos - lp * a.kv.rpp;
        if (lp < a.table_pages) page = __ldg(a.kv.pt + (int64_t)seq * a.kv.pt_stride + lp);
        if (page < 0 || page >= a.kv.n_pages) {
            page = -1;
            raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
        }
    }
    return make_int2(page, slot);
}

// Sequences that lie outside the batch's rows are reported by a thread each, as the rows that look them up may be none
// (by one warp for all of them, one row of each of 4,096 sequences took 44 us, and of 65,535 1.1 ms).
CSA_DEV void report_sequences(const QuantArgs& a) {
    const int b = (int)blockIdx.x * QC_T + threadIdx.x;  // (a grid has B threads at least)
    if (b < a.B) {
        const int64_t q0 = __ldg(a.offsets + b), q1 = __ldg(a.offsets + b + 1);
        if (q0 < 0 || q1 < q0 || q1 > a.total || q1 - q0 > a.max_rows || __ldg(a.n_tokens + b) > QC_MAX_TOKENS)
            raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
    }
}

// Lane l has dims [16 l, 16 l + 16): a block of 128 dims is a quarter of a warp.  WIDE: rows are 32-byte aligned.
template <int R, bool WIDE>
__global__ void __launch_bounds__(QC_T) quant_write_kernel(QuantArgs a) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * (QC_T / 32) + (threadIdx.x >> 5), row0 = warp * R;
    if (row0 >= a.total) return report_sequences(a);
    uint32_t v[R][8];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const uint8_t* p = a.rows + min(row0 + i, a.total - 1) * ROW_BYTES + lane * 32;
        if (WIDE) {
            ldg_nc_v8(p, v[i]);
        } else {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(p)), y = __ldg(reinterpret_cast<const uint4*>(p) + 1);
            v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
            v[i][4] = y.x, v[i][5] = y.y, v[i][6] = y.z, v[i][7] = y.w;
        }
    }
    const int2 at = places<R>(a, row0, lane);
    report_sequences(a);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int page = __shfl_sync(0xffffffffu, at.x, i), slot = __shfl_sync(0xffffffffu, at.y, i);
        if (page < 0) continue;
        // the block's largest magnitude, as bits: infinities and NaN are above all others
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = __vmaxu2(m, v[i][e] & 0x7FFF7FFFu);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t t = max(m & 0xFFFFu, m >> 16);
        const bool fine = t < 0x7F80u;
        // (fp32 bits of the largest) 1.75 2^e is 448 2^(e - 8); anything above calls for the next power
        uint32_t s = max((int)(((t << 16) + 0x1FFFFFu) >> 23) - 8, 10);
        const float f = __uint_as_float((254u - s) << 23);  // 2^(127 - s)
        uint32_t c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float2 y = f32x2_split(f32x2_mul(f32x2(bf16lo(v[i][e]), bf16hi(v[i][e])), f32x2(f, f)));
            c[e] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
        }
        uint4 w = make_uint4(c[0] | c[1] << 16, c[2] | c[3] << 16, c[4] | c[5] << 16, c[6] | c[7] << 16);
        if (s >= 247u) {
            if (!fine) {
                s = 255u;
                w = make_uint4(0, 0, 0, 0);
            } else {  // 256 2^120 would read back as infinity: codes end at 240 (0x77)
                uint32_t* x = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = (x[e] & 0x80808080u) | __vminu4(x[e] & 0x7F7F7F7Fu, 0x77777777u);
            }
        }
        *reinterpret_cast<uint4*>(q_codes(a.kv.base, a.kv.page_stride, page, slot) + lane * 16) = w;
        // lanes 0, 8, 16 and 24 have the row's scales
        s |= __shfl_down_sync(0xffffffffu, s, 8) << 8;
        s |= __shfl_down_sync(0xffffffffu, s, 16) << 16;
        if (lane == 0)
            *reinterpret_cast<uint32_t*>(q_scales(a.kv.base, a.kv.page_stride, a.kv.rpp, page, slot)) = s;
    }
}

// Lane l has dims [16 l, 16 l + 16).
template <int R>
__global__ void __launch_bounds__(QC_T) quant_read_kernel(QuantArgs a) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * (QC_T / 32) + (threadIdx.x >> 5), row0 = warp * R;
    if (row0 >= a.total) return report_sequences(a);
    const int2 at = places<R>(a, row0, lane);
    report_sequences(a);
    uint4 c[R];
    uint32_t s[R];
    int page[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        page[i] = __shfl_sync(0xffffffffu, at.x, i);
        const int slot = __shfl_sync(0xffffffffu, at.y, i);
        c[i] = make_uint4(0, 0, 0, 0);
        s[i] = 127;
        if (page[i] >= 0) {
            c[i] = ldg_nc_v4(q_codes(a.kv.base, a.kv.page_stride, page[i], slot) + lane * 16);
            s[i] = __ldg(q_scales(a.kv.base, a.kv.page_stride, a.kv.rpp, page[i], slot) + (lane >> 3));
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (page[i] == -2) continue;
        uint4 x, y;
        q_values(c[i], q_factor(s[i]), x, y);
        const uint32_t rest = q_factor_rest(s[i]);
        if (rest != 0x3F803F80u) q_times(x, rest), q_times(y, rest);
        uint8_t* p = a.out + (row0 + i) * ROW_BYTES + lane * 32;
        const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        if (a.wide_out) {
            stg_v8(p, w);
        } else {
            reinterpret_cast<uint4*>(p)[0] = x;
            reinterpret_cast<uint4*>(p)[1] = y;
        }
    }
}

csa_status check_quant_cache(const csa_paged& kv, int64_t page_table_stride) {
    const csa_status rc = check_paged(kv, Q_ROW_BYTES);
    if (rc) return rc;
    if (!kv.page_table || !al4(kv.page_table) || page_table_stride < 1) return CSA_ERR_INVALID_ARG;
    if (kv.n_pages > 0x7FFFFFFFLL || kv.n_pages > (1LL << 32) / (kv.page_stride_bytes / 16)) return CSA_ERR_UNSUPPORTED;
    return CSA_OK;
}

static csa_status quant_args(QuantArgs& a, const void* data, const csa_paged& kv, int64_t page_table_stride, int32_t B,
                             const int64_t* offsets, const int64_t* n_tokens, int64_t total, int64_t max_rows) {
    if (B < 1 || B > 65535 || total > 0x7FFFFFFFLL) return CSA_ERR_UNSUPPORTED;
    if (total < 0 || max_rows < 1 || (total > 0 && !data) || !al16(data) || !offsets || !al8(offsets) || !n_tokens ||
        !al8(n_tokens))
        return CSA_ERR_INVALID_ARG;
    const csa_status rc = check_quant_cache(kv, page_table_stride);
    if (rc || total == 0) return rc;
    a.kv.base = static_cast<const uint8_t*>(kv.base);
    a.kv.pt = kv.page_table;
    a.kv.pt_stride = page_table_stride;
    a.kv.page_stride = kv.page_stride_bytes;
    a.kv.n_pages = kv.n_pages;
    a.kv.rpp = kv.rows_per_page;
    a.kv.qpr = 1;
    a.table_pages = page_table_stride;
    a.B = B;
    a.offsets = offsets;
    a.n_tokens = n_tokens;
    a.total = total;
    a.max_rows = max_rows;
    a.status = device_status_ptr();
    return a.status ? CSA_OK : CSA_ERR_CUDA;
}

// CTAs for the rows, and a thread for each sequence.
static dim3 quant_grid(const QuantArgs& a, int R) {
    const int64_t rows = R * (QC_T / 32);
    return dim3((unsigned)std::max((a.total + rows - 1) / rows, ((int64_t)a.B + QC_T - 1) / QC_T));
}

}  // namespace csa

using namespace csa;

extern "C" {

csa_status csa_quant_write(const void* rows, csa_paged cache, int64_t page_table_stride, int32_t B,
                           const int64_t* offsets, const int64_t* n_tokens, int64_t total, int64_t max_rows,
                           void* stream) {
    QuantArgs a = {};
    const csa_status rc = quant_args(a, rows, cache, page_table_stride, B, offsets, n_tokens, total, max_rows);
    if (rc || total == 0) return rc;
    a.rows = static_cast<const uint8_t*>(rows);
    const bool many = total >= QC_MANY;
    const bool wide = (reinterpret_cast<uintptr_t>(rows) & 31u) == 0;
    return from_cuda(launch_after(many ? (wide ? quant_write_kernel<QC_W, true> : quant_write_kernel<QC_W, false>)
                                       : (wide ? quant_write_kernel<1, true> : quant_write_kernel<1, false>),
                                  quant_grid(a, many ? QC_W : 1), QC_T, 0, static_cast<cudaStream_t>(stream), a));
}

csa_status csa_quant_read(csa_paged cache, int64_t page_table_stride, int32_t B, const int64_t* offsets,
                          const int64_t* n_tokens, int64_t total, int64_t max_rows, void* out, void* stream) {
    QuantArgs a = {};
    const csa_status rc = quant_args(a, out, cache, page_table_stride, B, offsets, n_tokens, total, max_rows);
    if (rc || total == 0) return rc;
    a.out = static_cast<uint8_t*>(out);
    a.wide_out = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
    const bool many = total >= QC_MANY;
    return from_cuda(launch_after(many ? quant_read_kernel<QC_R> : quant_read_kernel<1>, quant_grid(a, many ? QC_R : 1),
                                  QC_T, 0, static_cast<cudaStream_t>(stream), a));
}

}  // extern "C"
