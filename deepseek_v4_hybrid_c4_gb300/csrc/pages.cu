// The pages that page tables name: reference counts, new pages, forks, moves to the front ("SGLang 如何为
// DeepSeek V4 打造「Day-0」推理加速", sec. "创新 1：ShadowRadix": one virtual slot space projected onto the
// physical pools, a page id standing for a page in every pool).
//
// refs[p] counts the table entries that name page p; a page is free where it is 0.  Every call that needs
// free or used pages in order scans refs in chunks of 4,096 pages: a chunk's CTA counts the pages in use before
// it (up to 32,768 pages all of them by itself, beyond from counts that a kernel before it left), adds its own
// prefix sums and writes the pages' ranks and lists.  The lists make the
// results independent of timing: new pages are the lowest free ids, moved pages go in the order of
// their ids.  Reference counts move by integer atomics, whose order does not show.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace csa {

constexpr int PG_T = 1024;                  // threads of a scan CTA
constexpr int PG_V = 4;                     // pages of a thread
constexpr int PG_CHUNK = PG_T * PG_V;

struct PoolArgs {
    int n_pools;
    int64_t n_pages;
    uint8_t* base[CSA_POOLS_MAX];
    int64_t bytes[CSA_POOLS_MAX];
    int64_t stride[CSA_POOLS_MAX];
};

// Workspace: the chunk counts, a header {pages counted, entries of list a below it}, three lists.
struct PagesWs {
    int32_t* cnt;
    int64_t* hdr;        // [0] free pages (alloc, fork) or used pages U (compact); [1] used pages below U
    int32_t* list;       // free page of rank r (alloc, fork); used page of rank r, r >= hdr[1] (compact)
    int32_t* hole;       // compact: free page of rank r below U
    int32_t* rank;       // compact: rank of a used page among the used ones, -1 of a free page
};
static int64_t pages_chunks(int64_t n_pages) { return (n_pages + PG_CHUNK - 1) / PG_CHUNK; }
static PagesWs pages_ws(void* ws, int64_t n_pages, size_t* total) {
    PagesWs w;
    uint8_t* b = static_cast<uint8_t*>(ws);
    size_t off = 0;
    w.hdr = reinterpret_cast<int64_t*>(b + off);
    off += 256;
    w.cnt = reinterpret_cast<int32_t*>(b + off);
    off += align_up((size_t)pages_chunks(n_pages) * 4, 256);
    const size_t l = align_up((size_t)n_pages * 4, 256);
    w.list = reinterpret_cast<int32_t*>(b + off);
    w.hole = reinterpret_cast<int32_t*>(b + off + l);
    w.rank = reinterpret_cast<int32_t*>(b + off + 2 * l);
    if (total) *total = off + 3 * l;
    return w;
}

// Sums of a and b over the CTA's warps, to every thread.  red: 2 x 32 words of shared memory.
__device__ __forceinline__ void block_sum2(int& a, int& b, int32_t* red) {
    for (int o = 16; o; o >>= 1) {
        a += __shfl_down_sync(0xffffffffu, a, o);
        b += __shfl_down_sync(0xffffffffu, b, o);
    }
    const int lane = threadIdx.x & 31, warps = (int)blockDim.x >> 5;
    __syncthreads();
    if (lane == 0) {
        red[threadIdx.x >> 5] = a;
        red[32 + (threadIdx.x >> 5)] = b;
    }
    __syncthreads();
    a = lane < warps ? red[lane] : 0;
    b = lane < warps ? red[32 + lane] : 0;
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
}

// Pages of chunk blockIdx.x that are used (free: the rest).
__global__ void __launch_bounds__(PG_T) pages_count_kernel(const int32_t* refs, int64_t n, int32_t* cnt) {
    __shared__ int32_t red[64];
    pdl_wait();
    const int64_t base = (int64_t)blockIdx.x * PG_CHUNK;
    int c = 0, none = 0;
#pragma unroll
    for (int v = 0; v < PG_V; ++v) {
        const int64_t i = base + v * PG_T + threadIdx.x;
        if (i < n) c += refs[i] > 0;
    }
    block_sum2(c, none, red);
    if (threadIdx.x == 0) cnt[blockIdx.x] = c;
    pdl_launch_dependents();
}

// Pools up to this size are counted by every scan CTA: a launch less (3 us), for up to 32 loads of a thread.
constexpr int64_t kSelfCount = 8 * PG_CHUNK;

// Ranks of chunk blockIdx.x.  COMPACT false: the free pages into list, hdr[0] = their number.
// COMPACT true: U = used pages -> hdr[0]; used pages' ranks; free pages below U into hole; used pages of
// id >= U into list at their rank; hdr[1] = used pages below U; refs copied to refs_out where they differ.
template <bool COMPACT>
__global__ void __launch_bounds__(PG_T) pages_scan_kernel(const int32_t* refs, int32_t* refs_out, int64_t n, PagesWs w,
                                                          int64_t* n_used) {
    __shared__ int32_t red[64];
    __shared__ int32_t wsum[PG_V * 32];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int chunks = (int)gridDim.x;
    const int64_t base = (int64_t)blockIdx.x * PG_CHUNK;
    // this thread's pages: base + 1024 v + tid; pre: used ones before it in its warp
    int32_t r[PG_V];
    int pre[PG_V];
#pragma unroll
    for (int v = 0; v < PG_V; ++v) {
        const int64_t i = base + v * PG_T + tid;
        r[v] = i < n ? __ldcg(refs + i) : 0;
    }
    int before = 0, all = 0;  // used pages before this chunk, and in all
    if (n <= kSelfCount) {
        const int last = (int)n;
#pragma unroll 8
        for (int i = tid; i < last; i += PG_T) {
            const int u = __ldcg(refs + i) > 0;
            all += u;
            if (i < (int)base) before += u;
        }
    } else {
        for (int c = tid; c < chunks; c += PG_T) {
            const int32_t x = w.cnt[c];
            all += x;
            if (c < (int)blockIdx.x) before += x;
        }
    }
#pragma unroll
    for (int v = 0; v < PG_V; ++v) {
        const unsigned m = __ballot_sync(0xffffffffu, r[v] > 0);
        pre[v] = __popc(m & ((1u << lane) - 1u));
        if (lane == 0) wsum[v * 32 + warp] = __popc(m);
    }
    block_sum2(before, all, red);  // (its barriers publish wsum)
    if (warp == 0) {  // exclusive prefix over the 128 (round, warp) counts, four a lane
        int c[4], t = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            c[e] = wsum[lane * 4 + e];
            t += c[e];
        }
        int x = t;
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        x -= t;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            wsum[lane * 4 + e] = x;
            x += c[e];
        }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < PG_V; ++v) {
        const int64_t i = base + v * PG_T + tid;
        const int rk = before + wsum[v * 32 + warp] + pre[v];  // used pages of smaller id
        if (i < n) {
            if (COMPACT) {
                w.rank[i] = r[v] > 0 ? rk : -1;
                if (r[v] > 0 && i >= all) w.list[rk] = (int32_t)i;
                if (r[v] <= 0 && i < all) w.hole[i - rk] = (int32_t)i;
                if (i == all) w.hdr[1] = rk;
                if (refs_out != refs) refs_out[i] = r[v];
            } else if (r[v] <= 0) {
                w.list[i - rk] = (int32_t)i;
            }
        }
    }
    if (blockIdx.x == 0 && tid == 0) {
        w.hdr[0] = COMPACT ? all : n - all;
        if (COMPACT) {
            if (all == n) w.hdr[1] = n;
            if (n_used) *n_used = all;
        }
    }
}

// Request blockIdx.x's new pages.
__global__ void __launch_bounds__(256) pages_alloc_kernel(int32_t* refs, int32_t* table, int64_t stride, int B,
                                                          const int32_t* first, const int32_t* count, PagesWs w,
                                                          int32_t* status) {
    __shared__ int32_t red[64];
    pdl_wait();
    const int b = blockIdx.x;
    auto valid = [&](int g) {
        const int64_t f = first[g], c = count[g];
        return f >= 0 && c >= 0 && f + c <= stride;
    };
    // entries of the requests before: in halves, as up to 4,096 rows of 2^31 - 1 entries do not fit 32 bits
    int64_t s = 0;
    for (int g = threadIdx.x; g < b; g += blockDim.x)
        if (valid(g)) s += count[g];
    int lo = (int)(s & 0xFFFFF), mid = (int)((s >> 20) & 0xFFFFF), hi = (int)(s >> 40), none = 0;
    block_sum2(lo, mid, red);
    block_sum2(hi, none, red);
    s = (int64_t)lo + ((int64_t)mid << 20) + ((int64_t)hi << 40);
    if (!valid(b)) {
        if (threadIdx.x == 0) raise_status(status, CSA_ERR_DEVICE_BOUNDS);
        return;
    }
    const int64_t n_free = w.hdr[0];
    int32_t* row = table + (int64_t)b * stride + first[b];
    const int64_t n = count[b];  // (up to 2^31 - 1: a 32-bit index would pass it by wrapping)
    for (int64_t j = threadIdx.x; j < n; j += blockDim.x) {
        int32_t p = -1;
        if (s + j < n_free) {
            p = w.list[s + j];
            refs[p] = 1;
        } else {
            raise_status(status, CSA_ERR_NO_PAGES);
        }
        row[j] = p;
    }
}

// An entry gives its page back.  The exchange makes a row that is listed twice count once.
__global__ void __launch_bounds__(256) pages_free_kernel(int32_t* refs, int64_t n_pages, int32_t* table, int64_t stride,
                                                         int B, const int32_t* rows, int32_t* status) {
    pdl_wait();
    const int32_t b = rows[blockIdx.y];
    if (b < 0 || b >= B) {
        if (threadIdx.x == 0 && blockIdx.x == 0) raise_status(status, CSA_ERR_DEVICE_BOUNDS);
        return;
    }
    int32_t* row = table + (int64_t)b * stride;
    for (int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; j < stride; j += (int64_t)gridDim.x * blockDim.x) {
        if (row[j] == -1) continue;
        const int32_t p = atomicExch(row + j, -1);
        if (p < 0) continue;
        if (p >= n_pages) {
            raise_status(status, CSA_ERR_DEVICE_BOUNDS);
        } else if (atomicSub(refs + p, 1) <= 0) {
            atomicAdd(refs + p, 1);
            raise_status(status, CSA_ERR_DEVICE_BOUNDS);
        }
    }
}

// A page is copied in pieces of 8 KB (of one pool; the last one of a pool may be shorter), each by a CTA
// of 256 threads with two 16-byte loads in flight per thread.
constexpr int PG_PIECE = 512;  // in 16 bytes
static int pieces_of(const PoolArgs& a) {
    int64_t n = 0;
    for (int p = 0; p < a.n_pools; ++p) n += (a.bytes[p] / 16 + PG_PIECE - 1) / PG_PIECE;
    return n > 0x7FFFFFFF ? 0x7FFFFFFF : (int)n;
}
__device__ __forceinline__ void copy_piece(const PoolArgs& a, int64_t src, int64_t dst, int64_t piece) {
#pragma unroll
    for (int p = 0; p < CSA_POOLS_MAX; ++p) {
        if (p >= a.n_pools) return;
        const int64_t n16 = a.bytes[p] / 16, n = (n16 + PG_PIECE - 1) / PG_PIECE;
        if (piece < n) {
            const int64_t i = piece * PG_PIECE + threadIdx.x;
            const uint4* s = reinterpret_cast<const uint4*>(a.base[p] + src * a.stride[p]) + i;
            uint4* d = reinterpret_cast<uint4*>(a.base[p] + dst * a.stride[p]) + i;
            uint4 v0, v1;
            if (i < n16) v0 = __ldcs(s);
            if (i + 256 < n16) v1 = __ldcs(s + 256);
            if (i < n16) __stcs(d, v0);
            if (i + 256 < n16) __stcs(d + 256, v1);
            return;
        }
        piece -= n;
    }
}

// Child blockIdx.y of a fork; the blocks of a child share its row and its page's copy.
struct ForkArgs {
    PoolArgs pools;
    int32_t* refs;
    int32_t* table;
    int64_t stride;
    int B, F, rpp, pieces;
    const int32_t* src;
    const int32_t* dst;
    int64_t* n_tokens;
    PagesWs w;
    int32_t* status;
};

__global__ void __launch_bounds__(256) pages_fork_kernel(ForkArgs a) {
    __shared__ int32_t red[64];
    pdl_wait();
    const int f = blockIdx.y, tid = threadIdx.x;
    const bool lead = blockIdx.x == 0 && tid == 0;
    // the parent's last page where it is to be copied, -1 where there is none; tokens to *n
    auto last_page = [&](int g, int64_t* n) -> int64_t {
        const int32_t b = a.src[g];
        if (b < 0 || b >= a.B) return -1;
        *n = a.n_tokens[b];
        if (*n <= 0 || *n % a.rpp == 0 || *n / a.rpp >= a.stride) return -1;
        const int32_t p = a.table[b * a.stride + *n / a.rpp];
        return p >= 0 && p < a.pools.n_pages ? p : -1;
    };
    const int32_t b = a.src[f], d = a.dst[f];
    int clash = 0, before = 0;
    for (int g = tid; g < a.F; g += blockDim.x) {
        clash += d == a.src[g] || (g != f && d == a.dst[g]);
        int64_t n;
        if (g < f && last_page(g, &n) >= 0) ++before;
    }
    block_sum2(clash, before, red);
    int64_t n = -1;
    const int64_t last = last_page(f, &n);
    if (b < 0 || b >= a.B || d < 0 || d >= a.B || clash || n < 0 || n / a.rpp + (n % a.rpp != 0) > a.stride) {
        if (lead) raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
        return;
    }
    const int64_t full = n / a.rpp;
    const bool part = n % a.rpp != 0;
    int64_t fresh = -1;
    if (last >= 0) {
        if (before < a.w.hdr[0]) fresh = a.w.list[before];
        else if (lead) raise_status(a.status, CSA_ERR_NO_PAGES);
    }
    if (lead) {
        a.n_tokens[d] = last >= 0 && fresh < 0 ? full * a.rpp : n;
        if (fresh >= 0) a.refs[fresh] = 1;
        // a last page without a page behind it was given back before, or its id is outside the pool
        if (part && last < 0 && a.table[b * a.stride + full] >= 0) raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
    }
    const int64_t t = (int64_t)blockIdx.x * blockDim.x + tid, nt = (int64_t)gridDim.x * blockDim.x;
    if (fresh >= 0)
        for (int p = blockIdx.x; p < a.pieces; p += gridDim.x) copy_piece(a.pools, last, fresh, p);
    const int32_t* from = a.table + b * a.stride;
    int32_t* to = a.table + d * a.stride;
    for (int64_t j = t; j < a.stride; j += nt) {
        int32_t p = -1;
        if (j < full) {
            p = from[j];
            if (p >= a.pools.n_pages) {
                raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
                p = -1;
            }
            if (p >= 0) atomicAdd(a.refs + p, 1);
            else p = -1;
        } else if (j == full) {
            p = (int32_t)fresh;
        }
        to[j] = p;
    }
}

struct MoveArgs {
    PoolArgs pools;
    const int32_t* refs;
    int32_t* refs_out;
    const int32_t* table;
    int32_t* table_out;
    int64_t entries;
    PagesWs w;
    int pieces;
    int32_t* status;
};

// Tables, counts and pages of a compaction: move k takes used page list[hdr[1] + k] to hole[k].
__global__ void __launch_bounds__(256) pages_move_kernel(MoveArgs a) {
    pdl_wait();
    const int64_t U = a.w.hdr[0], low = a.w.hdr[1], moves = U - low;
    const int64_t t = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, nt = (int64_t)gridDim.x * blockDim.x;
    for (int64_t k = t; k < moves; k += nt) {
        const int32_t s = a.w.list[low + k], d = a.w.hole[k];
        const int32_t r = a.refs[s];
        a.refs_out[d] = r;
        a.refs_out[s] = 0;
    }
    for (int64_t e = t; e < a.entries; e += nt) {
        int32_t p = a.table[e];
        if (p >= 0) {
            const int32_t r = p < a.pools.n_pages ? a.w.rank[p] : -1;
            if (r < 0) raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
            else if (p >= U) p = a.w.hole[r - low];
        }
        a.table_out[e] = p;
    }
    for (int64_t u = blockIdx.x; u < moves * a.pieces; u += gridDim.x) {
        const int64_t k = u / a.pieces;
        copy_piece(a.pools, a.w.list[low + k], a.w.hole[k], u - k * a.pieces);
    }
}

__global__ void __launch_bounds__(256) pages_copy_kernel(PoolArgs a, int pieces, const int32_t* src, const int32_t* dst,
                                                         int n, int32_t* status) {
    pdl_wait();
    for (int64_t u = blockIdx.x; u < (int64_t)n * pieces; u += gridDim.x) {
        const int64_t k = u / pieces;
        const int32_t s = src[k], d = dst[k];
        if (s < 0 || d < 0 || s >= a.n_pages || d >= a.n_pages) {
            if (threadIdx.x == 0) raise_status(status, CSA_ERR_DEVICE_BOUNDS);
            continue;
        }
        copy_piece(a, s, d, u - k * pieces);
    }
}

constexpr int64_t kMaxPoolPages = 1 << 28;

static csa_status check_pools(const csa_page_pools* p, PoolArgs* a) {
    if (!p) return CSA_ERR_INVALID_ARG;
    if (p->n_pools < 1 || p->n_pools > CSA_POOLS_MAX || p->n_pages < 1) return CSA_ERR_INVALID_ARG;
    if (p->n_pages > kMaxPoolPages) return CSA_ERR_UNSUPPORTED;
    a->n_pools = p->n_pools;
    a->n_pages = p->n_pages;
    for (int i = 0; i < p->n_pools; ++i) {
        if (!p->base[i] || !al16(p->base[i]) || p->page_bytes[i] < 16 || p->page_bytes[i] % 16 ||
            p->page_stride[i] % 16 || p->page_stride[i] < p->page_bytes[i])
            return CSA_ERR_INVALID_ARG;
        a->base[i] = static_cast<uint8_t*>(p->base[i]);
        a->bytes[i] = p->page_bytes[i];
        a->stride[i] = p->page_stride[i];
    }
    return CSA_OK;
}

static csa_status check_table(const void* refs, int64_t n_pages, const void* table, int64_t stride, int32_t B) {
    if (!refs || !al4(refs) || !table || !al4(table) || n_pages < 1 || B < 1 || stride < 1) return CSA_ERR_INVALID_ARG;
    if (n_pages > kMaxPoolPages || B > 65535 || stride > 0x7FFFFFFFLL || stride * B > (1LL << 40))
        return CSA_ERR_UNSUPPORTED;
    return CSA_OK;
}

static csa_status check_ws(const void* ws, size_t bytes, int64_t n_pages) {
    size_t need;
    pages_ws(nullptr, n_pages, &need);
    return ws && al16(ws) && bytes >= need ? CSA_OK : CSA_ERR_WORKSPACE;
}

static cudaError_t launch_scan(bool compact, const int32_t* refs, int32_t* refs_out, int64_t n, const PagesWs& w,
                               int64_t* n_used, cudaStream_t s) {
    const unsigned c = (unsigned)pages_chunks(n);
    if (n > kSelfCount) {
        cudaError_t e = launch_after(pages_count_kernel, dim3(c), PG_T, 0, s, refs, n, w.cnt);
        if (e != cudaSuccess) return e;
    }
    return compact ? launch_after(pages_scan_kernel<true>, dim3(c), PG_T, 0, s, refs, refs_out, n, w, n_used)
                   : launch_after(pages_scan_kernel<false>, dim3(c), PG_T, 0, s, refs, refs_out, n, w, n_used);
}

}  // namespace csa

using namespace csa;

extern "C" {

size_t csa_pages_workspace_size(int64_t n_pages) {
    if (n_pages < 1 || n_pages > kMaxPoolPages) return 0;
    size_t need;
    pages_ws(nullptr, n_pages, &need);
    return need;
}

csa_status csa_pages_alloc(int32_t* refs, int64_t n_pages, int32_t* page_table, int64_t table_stride, int32_t B,
                           const int32_t* first, const int32_t* count, void* workspace, size_t ws_bytes,
                           void* stream) {
    csa_status rc = check_table(refs, n_pages, page_table, table_stride, B);
    if (rc) return rc;
    if (!first || !al4(first) || !count || !al4(count)) return CSA_ERR_INVALID_ARG;
    if (B > 4096) return CSA_ERR_UNSUPPORTED;
    if ((rc = check_ws(workspace, ws_bytes, n_pages))) return rc;
    int32_t* st = device_status_ptr();
    if (!st) return CSA_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const PagesWs w = pages_ws(workspace, n_pages, nullptr);
    cudaError_t e = launch_scan(false, refs, refs, n_pages, w, nullptr, s);
    if (e == cudaSuccess)
        e = launch_after(pages_alloc_kernel, dim3(B), 256, 0, s, refs, page_table, table_stride, B, first, count, w, st);
    return from_cuda(e);
}

csa_status csa_pages_free(int32_t* refs, int64_t n_pages, int32_t* page_table, int64_t table_stride, int32_t B,
                          const int32_t* rows, int32_t R, void* stream) {
    csa_status rc = check_table(refs, n_pages, page_table, table_stride, B);
    if (rc) return rc;
    if (R < 0 || (R > 0 && !rows) || !al4(rows)) return CSA_ERR_INVALID_ARG;
    if (R > 65535) return CSA_ERR_UNSUPPORTED;
    if (R == 0) return CSA_OK;
    int32_t* st = device_status_ptr();
    if (!st) return CSA_ERR_CUDA;
    // one entry a thread where the rows are not endless: an entry is a chain of a load and two atomics (16 rows of
    // 8,188 entries at four a thread: 10.4 us; one atomic for equal pages of 16 rows, in longer chains: 12.0 us)
    int64_t x = (table_stride + 255) / 256;
    if (x * R > 4096) x = std::max<int64_t>(4096 / R, 1);
    return from_cuda(launch_after(pages_free_kernel, dim3((unsigned)x, (unsigned)R), 256, 0,
                                  static_cast<cudaStream_t>(stream), refs, n_pages, page_table, table_stride, B, rows, st));
}

csa_status csa_pages_fork(const csa_page_pools* pools, int32_t* refs, int32_t* page_table, int64_t table_stride,
                          int32_t B, const int32_t* src, const int32_t* dst, int32_t F, int64_t* n_tokens,
                          int32_t rows_per_page, void* workspace, size_t ws_bytes, void* stream) {
    ForkArgs a;
    csa_status rc = check_pools(pools, &a.pools);
    if (rc) return rc;
    if ((rc = check_table(refs, pools->n_pages, page_table, table_stride, B))) return rc;
    if (F < 0 || (F > 0 && (!src || !dst)) || !al4(src) || !al4(dst) || !n_tokens || !al8(n_tokens) || rows_per_page < 1)
        return CSA_ERR_INVALID_ARG;
    if (F > 1024) return CSA_ERR_UNSUPPORTED;
    if ((rc = check_ws(workspace, ws_bytes, pools->n_pages))) return rc;
    if (F == 0) return CSA_OK;
    int32_t* st = device_status_ptr();
    if (!st) return CSA_ERR_CUDA;
    a.refs = refs;
    a.table = page_table;
    a.stride = table_stride;
    a.B = B;
    a.F = F;
    a.rpp = rows_per_page;
    a.src = src;
    a.dst = dst;
    a.n_tokens = n_tokens;
    a.w = pages_ws(workspace, pools->n_pages, nullptr);
    a.pieces = pieces_of(a.pools);
    a.status = st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_scan(false, refs, refs, pools->n_pages, a.w, nullptr, s);
    // CTAs of a child: one for each 256 entries of its row, and one for each piece of its page's copy
    int64_t x = std::max<int64_t>((table_stride + 255) / 256, a.pieces);
    if (x * F > 4096) x = std::max<int64_t>(4096 / F, 1);
    if (e == cudaSuccess) e = launch_after(pages_fork_kernel, dim3((unsigned)x, (unsigned)F), 256, 0, s, a);
    return from_cuda(e);
}

csa_status csa_pages_compact(const csa_page_pools* pools, const int32_t* refs, int32_t* refs_out,
                             const int32_t* page_table, int32_t* page_table_out, int64_t table_stride, int32_t B,
                             int64_t* n_used, void* workspace, size_t ws_bytes, void* stream) {
    MoveArgs a;
    csa_status rc = check_pools(pools, &a.pools);
    if (rc) return rc;
    if ((rc = check_table(refs, pools->n_pages, page_table, table_stride, B))) return rc;
    if (!refs_out || !al4(refs_out) || !page_table_out || !al4(page_table_out) || (n_used && !al8(n_used)))
        return CSA_ERR_INVALID_ARG;
    if ((rc = check_ws(workspace, ws_bytes, pools->n_pages))) return rc;
    int32_t* st = device_status_ptr();
    const int sms = device_sm_count();
    if (!st || !sms) return CSA_ERR_CUDA;
    a.refs = refs;
    a.refs_out = refs_out;
    a.table = page_table;
    a.table_out = page_table_out;
    a.entries = table_stride * B;
    a.w = pages_ws(workspace, pools->n_pages, nullptr);
    a.pieces = pieces_of(a.pools);
    a.status = st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_scan(true, refs, refs_out, pools->n_pages, a.w, n_used, s);
    if (e == cudaSuccess) e = launch_after(pages_move_kernel, dim3((unsigned)sms * 8), 256, 0, s, a);
    return from_cuda(e);
}

csa_status csa_pages_copy(const csa_page_pools* pools, const int32_t* src, const int32_t* dst, int32_t n,
                          void* stream) {
    PoolArgs a;
    csa_status rc = check_pools(pools, &a);
    if (rc) return rc;
    if (n < 0 || (n > 0 && (!src || !al4(src) || !dst || !al4(dst)))) return CSA_ERR_INVALID_ARG;
    if (n == 0) return CSA_OK;
    int32_t* st = device_status_ptr();
    const int sms = device_sm_count();
    if (!st || !sms) return CSA_ERR_CUDA;
    const int pieces = pieces_of(a);
    const int64_t g = std::min<int64_t>((int64_t)n * pieces, (int64_t)sms * 8);
    return from_cuda(launch_after(pages_copy_kernel, dim3((unsigned)g), 256, 0, static_cast<cudaStream_t>(stream), a, pieces,
                                  src, dst, n, st));
}

}  // extern "C"
