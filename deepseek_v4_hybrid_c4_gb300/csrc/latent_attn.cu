// Dense attention over ranges of the paged latent cache (K = V = the bf16 row):
//   csa_prefix_attn   one token per request, the batch's first rows shared
//   csa_window_attn   causal, a sliding window and the first tokens of the sequence
//   csa_quant_attn    the same over quantised rows (codes and scales, quant.cuh)
//
//   l_j = scale * q . K_j,  o = sum_j softmax(l)_j V_j,  lse = ln sum_j exp(l_j)
//
// Both are the same work: 128 query rows (heads of one or several tokens or requests) against a list of
// key rows.  A pair of CTAs (one cluster, one CTA per SM) takes an item: 128 query rows and the
// key rows of one or more tiles of 128.  The tensor-core products run over the pair (tcgen05, cta_group::2,
// M = 128): each CTA holds 64 of the query rows, and
//   S = Q K^T   N = 128 keys, K = 512: each CTA stages half of the tile's keys, all dims
//   O += P V    N = 256 twice, K = 128: each CTA stages all of the tile's keys, half of the dims
// so that the 128 x 512 fp32 accumulator takes 256 of the pair's TMEM columns and S another 64 (two
// buffers), where a single CTA would need all of its TMEM for O alone (and with O cut in two along its
// dims would have to compute S twice).  Measured on GB300 with nothing but these products in flight: 2,056 cycles
// a tile against 2,048 at the nominal rate.
//
// What bounds it.  Many query rows over a long prefix: the tensor cores under the power limit (4,096 rows over
// 32K keys, 276 GFLOP: 161 us with the same inputs again, 183 us with others, 1.51 PFLOP/s).  A prompt under a
// short window: the softmax warps' chain through an item (8,192 tokens of 128 heads, window 128: 461 us, 4.7 TB/s
// of queries and outputs; 40 percent of an item is its output).  Single tokens: one chain of dependent loads,
// products and stores, 9 to 11 us.
//
// Roles (16 warps a CTA): warps 0-7 own the TMEM lanes, two to a lane quarter (softmax, output); warp 8 of
// the even CTA issues the products; warp 9 works the items out for the others, looks up the tiles' pages, up to
// four tiles ahead, and loads Q; warps 10-15 load key rows.  Both CTAs' copies report to the even CTA's
// barriers.  The code is kept small and, for the products, free of branches: with the items worked out in
// every role and a wait before each slot's products, the kernel was 175 KB of code, every step of a role
// cost some 200 cycles (the waits themselves were over at once), and a tile took 4,400 cycles.  Windows and
// prefixes are separate kernels (a shared one: prefixes 2 to 5 percent slower), 64 to 68 KB each, and 14 KB
// (lat_not_finite) that only infinities call.
// Key rows come through a ring of 8 slots of 16 KB in the order in which the products take them: S of a tile
// in four slots (128 dims each of the CTA's own keys), P V in four (32 keys each, the CTA's half of the
// dims; empty ones in a short tile).  The order is S(0), then S(i+1), PV(i): the softmax of tile i runs beside S(i+1).
// Key rows are copied by TMA in the products' swizzle: where 16 rows always share a page (rows_per_page a
// multiple of 16) in boxes of 64, 32 or 16 rows, as many as lie one behind the other in their page (issuing
// a copy costs a warp some 60 cycles whatever its size); otherwise in boxes of 16 rows where a unit's rows lie one
// behind the other, and in four-row gathers where they do not.  The list of
// key rows is made of 16-row units; rows of a unit that no query sees are masked.
//
// Softmax: a thread holds one row's logits of a quarter of a tile; the row's four threads exchange their
// maxima.  The running maximum moves only when a tile exceeds it by 2^8 (O is then rescaled in TMEM);
// P is rounded to bf16 for the product, its sum is taken in fp32 before the rounding.  P and O wait for the
// product before; the last tile of a window item, when it is short, has a place of its own for P and waits only to
// rescale O (a prompt of 8K tokens: 524 -> 503 us).  So a weight is off by up to half a bf16 step, also a dominant one whose
// tile did not move the maximum, and an output by as much of its weighted absolute values; a second sum, of the rounded
// weights, would cancel the dominant one's share and cost 2 percent (a prompt of 8K tokens: 462 -> 470 us; mean errors against
// 64 bits stay 1.7 to 2.1e-3, where the output's own rounding alone is 1.65e-3).
//
// A masked weight is exactly 0, but 0 * NaN is NaN, and the products see every row of a unit.  In
// a tile with masked rows a NaN or an infinity in any row makes that row's logits of all 128 query rows
// non-finite; where a thread finds one, its CTA replaces the non-finite values of the tile's V rows by 0 before the
// product, once the products' thread has told it that they are there (waiting for them in every tile with masked rows
// cost a prompt 6 percent).  Query rows that do attend such a key get what the formula gives: a logit of NaN or +inf makes
// them NaN; one of -inf is a weight of 0, and 0 times what V holds is NaN in the dims that are not finite.  In tiles without
// masked rows the product says so itself; for the others, and where every logit of a tile is -inf, the query's row is
// noted (LP_SM_LOST), and its output mended behind the item (lat_not_finite).
//
// Quantised rows.  The loading warps turn codes into fp16 on their way to the ring, each value over the largest scale of its
// tile (times 2^Q_UP, as far as fp16 reaches): a conversion and a product for two values, where bf16, which has no conversion from e4m3, takes five
// operations; S and P V are then fp16 products.  That scale, 2^T, comes back in the softmax: logits are multiplied by
// it, and O and the weights (fp16, at most 2^15) are kept over a running maximum of weight times scale, while
// the sum of the weights has one of the weights alone.  Rows more than 2^15 apart keep scales of their own, which the
// softmax then looks up for each.  Q becomes fp16 in shared memory, each row with a power of two of its own.
// 20 warps: 8 loading warps, two for Q (it is ready beside the item before), and 104 registers for the softmax, 88 for
// the others.  Work is dealt out in runs of one length cut anywhere (quant_item).
// What bounds it (a chunk of 1,024 tokens of 128 heads over 24K rows: 6.6 ms, 1.02 PFLOP/s, 4,900 cycles a tile where the
// products take 2,056): the L1's data pipe, 80 percent of its peak with the products' operands, the rows on their way in
// and out of registers and what is looked up, and instruction fetch (85 percent of what the cache beyond an SM's
// delivers).  Every row is turned into fp16 twice in a pair, as a key by one CTA and as a value by the CTA that has its
// dims.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <limits>

#include "common.cuh"
#include "internal.h"
#include "quant.cuh"

namespace csa {

constexpr int LP_T = 512;
constexpr int LP_SOFT = 8;                                // softmax warps
constexpr int LP_PROD = 6;                                // loading warps
constexpr int LP_SLOTS = 8;
constexpr int LP_PAIRS = 76;                              // pairs of SMs: sizes the splits (and so the workspace)
constexpr uint32_t LP_SLOT = 16384;
constexpr uint32_t LP_QSLAB = 64 * 128;                   // 64 dims of the CTA's 64 query rows
constexpr uint32_t LP_SM_RING = 8 * LP_QSLAB;             // behind Q
constexpr uint32_t LP_SM_P = LP_SM_RING + LP_SLOTS * LP_SLOT;  // slabs of 64 keys x 64 rows: two, and
                                                          // one for tiles of up to 4 units (the last of an item)
constexpr uint32_t LP_SM_BAR = LP_SM_P + 3 * LP_QSLAB;
constexpr uint32_t LP_FULL = LP_SM_BAR, LP_EMPTY = LP_FULL + 64, LP_LOOK = LP_EMPTY + 64, LP_USED = LP_LOOK + 64;
constexpr uint32_t LP_QFULL = LP_USED + 64, LP_QEMPTY = LP_QFULL + 8, LP_SFULL = LP_QEMPTY + 8;
constexpr uint32_t LP_PREADY = LP_SFULL + 16, LP_PVDONE = LP_PREADY + 16, LP_ITEM = LP_PVDONE + 16;
constexpr uint32_t LP_TAKEN = LP_ITEM + 32;
static_assert(LP_TAKEN + 32 <= LP_SM_BAR + 512, "barriers");
constexpr uint32_t LP_SM_TMEM = LP_SM_BAR + 512, LP_SM_DEAD = LP_SM_TMEM + 8;
constexpr uint32_t LP_SM_WANT = LP_SM_TMEM + 16, LP_SM_LAND = LP_SM_TMEM + 20;  // the last tile whose V rows a softmax
                                                          // warp asked for (even CTA), and that are there (both)
constexpr uint32_t LP_SM_CLOSED = LP_SM_TMEM + 24;        // the first item that warp 9 will not bring
constexpr uint32_t LP_SM_VALID = LP_SM_TMEM + 64;         // [8 tiles][128 keys] bits of the rows that are there
constexpr uint32_t LP_SM_LOOK = LP_SM_VALID + 128;        // [8 tiles][128] row ids, or [8] units {page, row}, runs
constexpr uint32_t LP_SM_MAX = LP_SM_LOOK + 8 * 512;      // [2][256] row maxima of the threads
constexpr uint32_t LP_SM_SUM = LP_SM_MAX + 2048;          // [256] row sums of the threads
constexpr uint32_t LP_SM_ITEM = LP_SM_SUM + 1024;         // [4] items
constexpr uint32_t LP_SM_PLAIN = LP_SM_ITEM + 4 * 128;    // [8 tiles] plain (tile_plain)
constexpr uint32_t LP_SM_NEXT = LP_SM_PLAIN + 32;         // [8 tiles] gathers: which quads' rows follow each other
constexpr uint32_t LP_SM_LOST = LP_SM_NEXT + 128;         // [64] the last item in which the row's query saw a logit of
                                                          // -inf that calls for a look at its output; [64]: any row
constexpr uint32_t LP_SM_MORE = LP_SM_LOST + 272;         // [256] a second kind of maxima (quantised rows)
constexpr uint32_t LP_SMEM = LP_SM_MORE + 1024 + 1024;    // + alignment slack
static_assert(LP_SMEM <= 227 * 1024, "latent attention shared memory");
// Quantised rows, in the place of the slab for short tiles: what a row's logits are to be multiplied by (2^s of its largest
// scale s, or of the tile's), and its four scales over that, in fp16.
constexpr uint32_t LP_SM_FACTOR = LP_SM_P + 2 * LP_QSLAB;  // [8 tiles][128] fp32
constexpr uint32_t LP_SM_RATIO = LP_SM_FACTOR + 8 * 512;   // [4 tiles][128][4] fp16
constexpr uint32_t LP_QREADY = LP_TAKEN + 32;              // Q is there as fp16 (even CTA: of both)
constexpr uint32_t LP_QTOP = LP_QREADY + 8;                // and its rows' exponents: [2 items][64] bytes, a barrier each
                                                           // (the queries may be one item ahead of the softmax, not two)
constexpr uint32_t LP_SM_QTOP = LP_SM_NEXT;
static_assert(LP_SM_RATIO + 4 * 1024 <= LP_SM_BAR && LP_QTOP + 16 <= LP_SM_BAR + 512, "places of quantised rows");
// Of a tile: plain; one factor for all rows; values of 2^128; from bit 8 on the largest scale code of its rows.
constexpr uint32_t LQ_PLAIN = 1, LQ_EVEN = 2, LQ_HUGE = 4;
constexpr int LQ_TOP = 8;
constexpr float LQ_ROOM = 7.f;                             // weights are at most 2^(LP_RESCALE + LQ_ROOM) in fp16
constexpr int LQ_APART = 60;                              // log2: how far sums may lie below their weights
constexpr int64_t LP_MAX_ROWS = 0x7FFFFFFF - 127;         // of a request: a row id behind its last tile is an int too
// Tiles of a split at most: O takes eight additions a tile in the tensor cores, each of which may lose 2^-23 of the
// sum so far, in all no more than the 2^-8 that a rounded weight may be off.
constexpr int LP_MAX_TILES = 4096;
#define LAT_RARE(x) __builtin_expect(!!(x), 0)
constexpr float LP_LOG2E = 1.4426950408889634f;
constexpr float LP_LN2 = 0.6931471805599453f;
constexpr float LP_RESCALE = 8.0f;                        // log2 units
constexpr float LP_LSE_LOST = -3.4028235e38f;             // lse of a partial result whose rows all have logits of -inf: a
                                                          // weight of 0 in the merge, times NaN where they are not finite

// n / d for 0 <= n < 2^31 by a multiplication: with s = ceil(log2 d) and m = ceil(2^(31+s) / d) < 2^32,
// m n / 2^(31+s) exceeds n / d by less than n / 2^31 / d < 1 / d.
struct FastDiv {
    uint32_t m, s;
};
static FastDiv fast_div(uint32_t d) {
    FastDiv f = {0, 0};
    while ((1u << f.s) < d) ++f.s;
    f.m = (uint32_t)(((1ull << (31 + f.s)) + d - 1) / d);
    return f;
}
__device__ __forceinline__ int div_by(int n, FastDiv f) { return (int)(((uint64_t)(uint32_t)n * f.m) >> (31 + f.s)); }

struct QuantRun;
struct LatArgs {
    int H;
    FastDiv by_H;
    float sl2;                 // |scale| * log2(e); the sign is in the products
    int sl2_power;             // quantised rows: its power of two, and sl2 is in [1, 2)
    uint32_t negate;           // instruction-descriptor bit that negates Q
    DPaged kv;
    int64_t table_pages;       // entries of a request's page table
    FastDiv by_rpp;
    int B;
    // prefix: request b = row / H sees rows [0, n_rows[b]); rows below n_shared through table row 0
    const int64_t* n_rows;     // nullptr: window
    int n_shared, max_rows;
    int RT, SP, OS;            // row tiles over the batch; splits of the shared rows, of a request's own rows
    FastDiv by_RT, by_SP, by_OS, by_WS;
    // prefix, in runs (run > 0): the row tiles' shared tiles, the first tS of every gS places, and the requests' own ones,
    // tO of every gO, are each laid end to end and cut every `run` places: NS runs of the first, then those of the second
    int run, NS, tS, gS, tO, gO;
    FastDiv by_run, by_gS, by_gO;
    // window: B sequences
    const int64_t* q_offsets;
    const int64_t* n_tokens;
    int64_t total_q, max_q;
    int window, n_sink;
    int WS;                    // splits of a row tile's keys
    int items;                 // runs, or items (window: at most, where the sequences do not overlap)
    int rows;                  // query rows in all (B * H, total_q * H)
    int parts;                 // partial results of a row (1: written to out directly)
    float* part_o;             // [parts][rows][512] normalised
    float* part_lse;           // [parts][rows]
    uint16_t* out;
    // quantised rows: runs of `cut` places or more (QR runs at most), or, with cut = 0, items that are row tiles
    int cut;
    int slot_rows;             // rows of a partial result: [3 QR][slot_rows] of them
    QuantRun* runs;            // [QR + 1]
    bool wide_out;             // out is 32-byte aligned
    float* lse;
    int32_t* status;
};

// Of a run of a call over quantised rows: the row tile that begins in it and ends in run `last` (none: last is the run
// itself).  Behind the last of them, row0 is the number of runs.  A pair writes all of its runs before its first wait, so
// that after a wait that ran out none of them is what the workspace held; and the merge takes nothing from the list
// that would lead it out of the rows or of the partial results.
struct QuantRun {
    int row0, nrows, last;
};
constexpr int QR = LP_PAIRS;
constexpr int QUANT_DIRECT = 1, QUANT_MORE = 2;  // LatItem::shared: the output itself, joined with what the slot holds
constexpr int QUANT_ITEM = 3;                    // places of an item beside its tiles

// An item: query rows [row0, row0 + nrows) against tiles [t0, t0 + T) of a list of 16-row units: units
// [0, uA) of the request (sinks), then units uB, uB + 1, ..., nU in all.  T < 0: behind the last item.
struct LatItem {
    int T, t0, nU, uA, uB;
    int row0, nrows;
    int trow;                  // page-table row
    int part;
    int a1, lo, hi;            // rows that a query of the item may see: [0, a1) and [lo, hi)
    int full_lo, full_hi;      // rows that every query of the item sees
    int rr0;                   // window: first query row within its sequence
    int shared;                // prefix: the shared rows (else request trow's own)
    int64_t pos0;              // window: position of the sequence's first new token
};
static_assert(sizeof(LatItem) == 72, "an item's place in shared memory is read in 16-byte pieces");
__device__ __forceinline__ LatItem load_item(uint32_t at) {
    union {
        LatItem x;
        uint4 v[5];
    } u;
#pragma unroll
    for (int i = 0; i < 5; ++i) u.v[i] = ld_shared_v4(at + 16 * i);
    return u.x;
}

// Sequences by row tiles, 32 at a time, one per lane; item indices ascend.
struct SeqCursor {
    int c0 = -32, base = 0, total = 0;
    int incl = 0, tiles = 0, ql = 0;
    int64_t q0 = 0, nt = 0;
    int pos = -1, end = 0, run = 0;  // a run: the next place, the end, its number among the runs of its kind
};

__device__ __forceinline__ bool seq_valid(const LatArgs& a, int64_t q0, int64_t q1, int64_t nt) {
    return q0 >= 0 && q1 >= q0 && q1 <= a.total_q && q1 - q0 <= a.max_q && nt <= LP_MAX_ROWS;
}

// The last sequence that starts at or before token tok.
__device__ __forceinline__ int seq_of(const LatArgs& a, int64_t tok) {
    int l = 0, r = a.B;
    while (r - l > 1) {
        const int m = (l + r) / 2;
        if (__ldg(a.q_offsets + m) <= tok) l = m;
        else r = m;
    }
    return l;
}

__device__ __forceinline__ int ceil_div(int x, int y) { return (int)(((uint32_t)x + (uint32_t)y - 1u) / (uint32_t)y); }

// Row tile `tile` of a sequence: its rows and the units that they see.
__device__ __forceinline__ void window_item(const LatArgs& a, LatItem& x, int tile, int ql, int64_t q0, int64_t nt,
                                            int trow) {
    x.rr0 = tile * 128;
    x.nrows = min(128, ql * a.H - x.rr0);
    x.row0 = (int)q0 * a.H + x.rr0;
    x.trow = trow;
    x.shared = 0;
    x.pos0 = (nt > 0 ? nt : 0) - ql;
    const int64_t p0 = x.pos0 + div_by(x.rr0, a.by_H), p1 = x.pos0 + div_by(x.rr0 + x.nrows - 1, a.by_H);
    x.hi = p1 >= 0 ? (int)p1 + 1 : 0;
    x.lo = p0 >= a.window ? (int)p0 - a.window + 1 : 0;
    x.a1 = min(a.n_sink, x.hi);
    x.uA = min(ceil_div(x.a1, 16), ceil_div(x.hi, 16));
    x.uB = max(x.lo / 16, x.uA);
    x.nU = x.uA + max(0, ceil_div(x.hi, 16) - x.uB);
    x.full_lo = p1 >= a.window ? (int)p1 - a.window + 1 : 0;
    x.full_hi = p0 >= 0 ? (int)p0 + 1 : 0;
}

// The pair's next item (warp-collective), or false behind its last one.  `it`: the item's number, or, in runs, that of
// the run that the pair is in; a pair takes every `pairs`-th, whatever number of pairs the device has room for.
template <bool WINDOW>
__device__ __forceinline__ bool lat_item(const LatArgs& a, SeqCursor& cur, int& it, int pairs, int lane, bool report,
                                         LatItem& x) {
    int split, splits;
    FastDiv by;
    int first = 0, last = 0;  // tiles of a run's item
    if (!WINDOW) {
        int kb0, kb1, seg;
        if (a.run) {
            int g, t;
            for (;; it += pairs, cur.pos = -1) {
                if (cur.pos < 0) {
                    if (it >= a.items) return false;
                    cur.run = it < a.NS ? it : it - a.NS;
                    cur.pos = cur.run * a.run;
                    cur.end = min(cur.pos + a.run, it < a.NS ? a.RT * a.gS : a.B * a.gO);
                    cur.total = it < a.NS;
                }
                x.shared = cur.total;
                g = x.shared ? a.gS : a.gO, t = x.shared ? a.tS : a.tO;
                seg = div_by(cur.pos, x.shared ? a.by_gS : a.by_gO);
                if (cur.pos - seg * g >= t) cur.pos = ++seg * g;
                if (cur.pos < cur.end) break;  // (else the run ends, in places behind a segment's tiles)
            }
            first = cur.pos - seg * g;
            last = min(first + cur.end - cur.pos, t);
            cur.pos += last - first;
            split = cur.run - div_by(seg * g, a.by_run);
            splits = 0;
            by = a.by_run;
        } else {
            if (it >= a.items) return false;
            x.shared = it < a.RT * a.SP;
            if (x.shared) {  // neighbouring items read the same keys
                split = div_by(it, a.by_RT);
                splits = a.SP;
                by = a.by_SP;
                seg = it - split * a.RT;
            } else {
                const int j = it - a.RT * a.SP;
                seg = div_by(j, a.by_OS);
                split = j - seg * a.OS;
                splits = a.OS;
                by = a.by_OS;
            }
            first = split;  // (0 once a request)
        }
        x.a1 = x.uA = x.rr0 = 0;
        x.pos0 = 0;
        if (x.shared) {
            x.row0 = seg * 128;
            x.nrows = min(128, a.rows - x.row0);
            x.trow = 0;
            x.part = split;
            // the shortest and the longest of the rows' requests
            const int b0 = div_by(x.row0, a.by_H), b1 = div_by(x.row0 + x.nrows - 1, a.by_H);
            int mn = 0x7FFFFFFF, mx = 0;
            const bool look = report && first == 0 && a.OS == 0;  // (with rows of their own: reported there)
            for (int b = b0 + lane; b <= b1; b += 32) {
                const int64_t n = __ldg(a.n_rows + b);
                if (look && (n < 0 || n > a.max_rows)) raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
                const int c = n < 0 ? 0 : (n > a.n_shared ? a.n_shared : (int)n);
                mn = min(mn, c);
                mx = max(mx, c);
            }
            for (int o = 16; o; o >>= 1) {
                mn = min(mn, __shfl_xor_sync(0xffffffffu, mn, o));
                mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            }
            kb0 = 0;
            kb1 = mx;
            x.full_lo = 0;
            x.full_hi = mn;
            x.nU = ceil_div(a.n_shared, 16);  // the same split of the keys for every row tile
        } else {
            const int b = seg;
            x.row0 = b * a.H;
            x.nrows = a.H;
            x.trow = b;
            x.part = a.SP + split;
            const int64_t n = __ldg(a.n_rows + b);
            if (report && lane == 0 && first == 0 && (n < 0 || n > a.max_rows))
                raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
            kb0 = a.n_shared;
            kb1 = n < 0 ? 0 : (n > a.max_rows ? a.max_rows : (int)n);
            x.full_lo = kb0;
            x.full_hi = kb1;
            x.nU = kb1 > kb0 ? ceil_div(kb1, 16) - kb0 / 16 : 0;
        }
        x.uB = kb0 / 16;
        x.lo = kb0;
        x.hi = kb1;
    } else {
        if (it >= a.items) return false;  // (only offsets that fall and rise again would have more)
        while (it >= cur.base + cur.total) {
            cur.base += cur.total;
            cur.c0 += 32;
            if (cur.c0 >= a.B) return false;
            const int b = cur.c0 + lane;
            cur.tiles = 0;
            if (b < a.B) {
                cur.q0 = __ldg(a.q_offsets + b);
                const int64_t q1 = __ldg(a.q_offsets + b + 1);
                cur.nt = __ldg(a.n_tokens + b);
                if (seq_valid(a, cur.q0, q1, cur.nt)) {
                    cur.ql = (int)(q1 - cur.q0);
                    cur.tiles = ceil_div(cur.ql * a.H, 128) * a.WS;
                } else if (report) {
                    raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
                }
            }
            cur.incl = cur.tiles;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, cur.incl, o);
                if (lane >= o) cur.incl += v;
            }
            cur.total = __shfl_sync(0xffffffffu, cur.incl, 31);
        }
        const int at = it - cur.base;
        const int src = __ffs(__ballot_sync(0xffffffffu, cur.incl > at)) - 1;
        const int d = at - __shfl_sync(0xffffffffu, cur.incl - cur.tiles, src);
        const int ql = __shfl_sync(0xffffffffu, cur.ql, src);
        const int64_t q0 = __shfl_sync(0xffffffffu, cur.q0, src), nt = __shfl_sync(0xffffffffu, cur.nt, src);
        const int tile = div_by(d, a.by_WS);
        splits = a.WS;
        by = a.by_WS;
        split = d - tile * a.WS;
        window_item(a, x, tile, ql, q0, nt, cur.c0 + src);
        x.part = split;
    }
    const int tiles = ceil_div(x.nU, 8);
    if (!WINDOW && a.run) {
        x.t0 = first;
        x.T = max(min(last, tiles) - first, 0);
    } else {
        const int each = div_by(tiles, by), more = tiles - each * splits;  // the first `more` splits take one more
        x.t0 = split * each + min(split, more);
        x.T = each + (split < more ? 1 : 0);
    }
    if (x.shared && x.t0 * 128 >= x.hi) x.T = 0;
    return true;
}

// Calls over quantised rows.  Where there are few row tiles, every row tile of a sequence has as many places as its last
// one has key tiles, and QUANT_ITEM more; the places of all sequences are laid end to end and cut into at most QR runs of
// one length.  A row tile that lies in one run is an item whose output is written directly; of one that is cut, each run
// has a partial result: slot 2 r + 1 of the run r that it begins in, 2 r of those that it goes on in.  So there are three
// slots a run at most (the third for items of more than LP_MAX_TILES tiles, which are worked off in pieces, each joined
// with those before it in its slot), whatever the batch.
struct QuantCursor {
    int c0 = -32, tiles = 0, ql = 0, g = 0;
    int64_t base = 0, sum = 0, incl = 0;  // of the 32 sequences: places before them, in them, up to the lane's
    int64_t q0 = 0, nt = 0;
    int64_t total = 0, cut = 1, pos = -1, end = 0;
    int run = 0, left = 0, slot = 0;
    bool direct = false;
};

// The next 32 sequences, one per lane.
__device__ __forceinline__ void quant_load(const LatArgs& a, QuantCursor& c, int lane, bool report) {
    c.base += c.sum;
    c.c0 += 32;
    const int b = c.c0 + lane;
    c.tiles = c.g = 0;
    if (b < a.B) {
        c.q0 = __ldg(a.q_offsets + b);
        const int64_t q1 = __ldg(a.q_offsets + b + 1);
        c.nt = __ldg(a.n_tokens + b);
        if (seq_valid(a, c.q0, q1, c.nt)) {
            c.ql = (int)(q1 - c.q0);
            c.tiles = ceil_div(c.ql * a.H, 128);
            // key tiles of a row tile at most: its tokens' windows and the sinks, or all that there is
            const int64_t reach = min((int64_t)a.window + a.n_sink + 127 / a.H + 32, max(c.nt, (int64_t)0));
            c.g = ceil_div((int)reach, 128) + QUANT_ITEM;
        } else if (report) {
            raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
        }
    }
    const int64_t mine = a.cut ? (int64_t)c.tiles * c.g : c.tiles;
    c.incl = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, c.incl, o);
        if (lane >= o) c.incl += v;
    }
    c.sum = __shfl_sync(0xffffffffu, c.incl, 31);
    c.incl -= mine;  // (up to the lane's, without it)
}

__device__ __forceinline__ bool quant_item(const LatArgs& a, QuantCursor& c, int pair, int pairs, int lane, bool report,
                                           LatItem& x) {
    if (c.left > 0) {  // the rest of an item of very many tiles
        x.t0 += x.T;
        x.T = min(c.left, LP_MAX_TILES);
        c.left -= x.T;
        x.shared = (c.left == 0 && c.direct ? QUANT_DIRECT : 0) | QUANT_MORE;
        return true;
    }
    if (c.pos < 0) {  // the first call
        if (a.cut) {
            while (c.c0 + 32 < a.B) {
                quant_load(a, c, lane, report);
                c.total += c.sum;
            }
            c.cut = max((c.total + QR - 1) / QR, (int64_t)a.cut);
            c.c0 = -32;
            c.base = c.sum = 0;
            if (report && pair == 0 && lane == 0) a.runs[QR].row0 = (int)((c.total + c.cut - 1) / c.cut);
            if (report && lane == 0)
#pragma unroll 1
                for (int r = pair; r < QR; r += pairs) a.runs[r] = {0, 0, r};
        }
        c.pos = c.end = 0;
        c.run = pair - pairs;
    }
    for (;;) {
        if (c.pos >= c.end) {
            c.run += pairs;
            if (a.cut) {
                c.pos = c.run * c.cut;
                c.end = min(c.pos + c.cut, c.total);
                if (c.pos >= c.total) return false;
            } else {
                c.pos = c.run;
                c.end = c.pos + 1;
            }
        }
        while (c.pos >= c.base + c.sum) {
            if (c.c0 + 32 >= a.B) return false;
            quant_load(a, c, lane, report && !a.cut);
        }
        const int64_t at = c.pos - c.base;
        const int src = 31 - __clz((int)__ballot_sync(0xffffffffu, c.tiles > 0 && c.incl <= at));
        const int ql = __shfl_sync(0xffffffffu, c.ql, src), g = __shfl_sync(0xffffffffu, c.g, src);
        const int64_t q0 = __shfl_sync(0xffffffffu, c.q0, src), nt = __shfl_sync(0xffffffffu, c.nt, src);
        const int64_t d = at - __shfl_sync(0xffffffffu, c.incl, src);
        const int tile = a.cut ? (int)(d / g) : (int)d;
        window_item(a, x, tile, ql, q0, nt, c.c0 + src);
        const int T = ceil_div(x.nU, 8);
        int last = T;
        x.t0 = 0;
        c.direct = true;
        c.slot = a.cut ? 2 * QR + c.run : pair;
        if (a.cut) {
            x.t0 = (int)(d - (int64_t)tile * g);
            const int64_t first = c.pos - x.t0, left = min(c.end, first + g) - c.pos;
            c.pos += left;
            if (x.t0 >= max(T, 1)) continue;  // places behind the row tile's tiles
            last = (int)min((int64_t)T, x.t0 + left);
            const int r1 = (int)((first + max(T, 1) - 1) / c.cut);
            if (x.t0 > 0 || r1 > c.run) {
                c.direct = false;
                c.slot = 2 * c.run + (x.t0 == 0 ? 1 : 0);
                if (x.t0 == 0 && report && lane == 0) a.runs[c.run] = {x.row0, x.nrows, r1};
            }
        } else {
            ++c.pos;
        }
        x.part = c.slot;
        c.left = last - x.t0;
        x.T = min(c.left, LP_MAX_TILES);
        c.left -= x.T;
        x.shared = c.left == 0 && c.direct ? QUANT_DIRECT : 0;
        return true;
    }
}

__device__ __forceinline__ int item_units(const LatItem& x, int i) { return min(8, x.nU - (x.t0 + i) * 8); }
template <bool WINDOW>
__device__ __forceinline__ int unit_row(const LatItem& x, int u) {
    return (!WINDOW ? u + x.uB : u < x.uA ? u : u - x.uA + x.uB) * 16;
}

// Tile i of the item: every row seen by every query of the item, and every page there (vw: the rows that are).
template <bool WINDOW>
__device__ __forceinline__ bool tile_plain(const LatItem& x, int i, uint4 vw) {
    const int u0 = (x.t0 + i) * 8;
    return x.nU - u0 >= 8 && (vw.x & vw.y & vw.z & vw.w) == 0xffffffffu && (!WINDOW || u0 >= x.uA) &&
           unit_row<WINDOW>(x, u0) >= x.full_lo && unit_row<WINDOW>(x, u0 + 7) + 16 <= x.full_hi;
}

// Bounded wait; false once any wait of this CTA has run out.  The loads, the products and the passing on
// stop there; the softmax warps run on to the end of their item (their barriers count on one another), each
// further wait returning at once, and to the next one if there is one: that is for warp 9 alone to say (lat_wait_item),
// as a warp that found its item just there would wait for ever for one that had looked before and given up.
// Lane i waits on the barrier at its own address: a warp can wait on several at once.  A wait that is not over at
// the first look goes on out of line (the code of all roles goes through one instruction cache).
// (Quantised rows: in line, as a kernel whose warps share out its registers has no room for calls that return to
// several roles.)
__device__ __forceinline__ bool lat_wait_loop(uint32_t bar, uint32_t parity, volatile uint32_t* dead) {
#pragma unroll 1
    for (uint32_t i = 0; i < CSA_SPIN_LIMIT; ++i) {
        if (mbar_try_wait_for(bar, parity, 4000)) return true;
        if (*dead) return false;
    }
    *dead = 1;
    return false;
}
__device__ __noinline__ bool lat_wait_on(uint32_t bar, uint32_t parity, volatile uint32_t* dead) {
#pragma unroll 1
    for (uint32_t i = 0; i < CSA_SPIN_LIMIT; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*dead) return false;
        if (i >= 32) __nanosleep(64);
    }
    *dead = 1;
    return false;
}
template <bool QUANT>
__device__ __forceinline__ bool lat_wait(uint32_t bar, uint32_t parity, volatile uint32_t* dead) {
    if (QUANT) return lat_wait_loop(bar, parity, dead);
    return mbar_try_wait(bar, parity) || lat_wait_on(bar, parity, dead);
}

// Item number `it`, or false where warp 9 has ended before it (the first item that never comes: closed).  Warp 9's own
// waits are bounded, and none of them is for a warp that waits here, so that the limit is only the last resort.
__device__ __forceinline__ bool lat_wait_item_loop(uint32_t bar, uint32_t parity, int it, volatile int* closed) {
#pragma unroll 1
    for (uint32_t i = 0; i < 4 * CSA_SPIN_LIMIT; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*closed <= it) return false;
        if (i >= 32) __nanosleep(64);
    }
    return false;
}
__device__ __noinline__ bool lat_wait_item_on(uint32_t bar, uint32_t parity, int it, volatile int* closed) {
    return lat_wait_item_loop(bar, parity, it, closed);
}
template <bool QUANT>
__device__ __forceinline__ bool lat_wait_item(uint32_t bar, uint32_t parity, int it, volatile int* closed) {
    if (QUANT) return lat_wait_item_loop(bar, parity, it, closed);
    return mbar_try_wait(bar, parity) || lat_wait_item_on(bar, parity, it, closed);
}

// The same as lat_wait for a word of shared memory.
__device__ __forceinline__ bool lat_word(uint32_t at, uint32_t want, volatile uint32_t* dead) {
#pragma unroll 1
    for (uint32_t i = 0; i < CSA_SPIN_LIMIT; ++i) {
        if (ld_shared_u32(at) == want) return true;
        if (*dead) return false;
        if (i >= 32) __nanosleep(64);
    }
    *dead = 1;
    return false;
}

// The products' thread: a bounded wait for P of tile t.  A softmax warp that has to look into the tile's V rows
// (full, par: their barriers) asks for them meanwhile: both CTAs are told when they are there.
template <bool QUANT>
__device__ __forceinline__ bool lat_wait_p(uint32_t sb, uint32_t full, uint32_t par, uint32_t t,
                                            volatile uint32_t* dead) {
    bool ok = true;
#pragma unroll 1
    for (uint32_t i = 0; i < CSA_SPIN_LIMIT; ++i) {
        if (mbar_try_wait(sb + LP_PREADY + 8 * (t & 1), (t >> 1) & 1)) return true;
        if (ld_shared_u32(sb + LP_SM_WANT) == t + 1 && ld_shared_u32(sb + LP_SM_LAND) != t + 1) {
#pragma unroll 1
            for (int v = 0; v < 4; ++v) ok = ok && lat_wait<QUANT>(full + 8 * v, par, dead);
            fence_cluster();
#pragma unroll 1
            for (int c = 0; ok && c < 2; ++c) st_dsmem_u32(mapa(sb + LP_SM_LAND, c), t + 1);
        }
        if (*dead || !ok) break;
    }
    *dead = 1;
    return false;
}

__device__ __forceinline__ float lat_ex2(float x) {  // ex2.approx.ftz: relative error below 2^-22
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 32 bytes to global memory; narrow: only 16-byte aligned.
__device__ __forceinline__ void store_sector(uint8_t* p, const uint32_t* w, bool wide) {
    if (wide) {
        stg_v8(p, w);
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Page-table entry of logical row j of the item's request (-1 behind the table) and j's row in its page.
__device__ __forceinline__ int lat_entry(const LatArgs& a, const int32_t* pt, int j, int& slot) {
    const int lp = div_by(j, a.by_rpp);
    slot = j - lp * a.kv.rpp;
    return lp < a.table_pages ? __ldg(pt + lp) : -1;
}

// The cache's tensor maps: boxes of 64 dims and [0] 16, [1] 32, [2] 64 rows of a page, or, over all rows of the
// pool, [0] one row (gathers) and [1] 8, [2] 16, [3] 32 rows.
struct KeyMaps {
    CUtensorMap m[4];
};

// Caches read by gathers, quad q (rows 4q .. 4q+3 of a tile): the map of its copy, -1 where another quad's copy takes
// its rows along.  Boxes of 32, 16 and 8 rows where two units, a unit or half of one lie row behind row in memory, a
// gather for any four rows.  Bits at the run's first quad (LP_SM_NEXT); q0: the copying warp's first quad; two: it
// copies both units of the pair.
struct QuadRuns {
    uint32_t half, unit, pair;
};
__device__ __forceinline__ int quad_map(QuadRuns n, int q, int q0, bool two) {
    const int u = q & ~3, p = q0 + ((q - q0) & ~7);  // the quad's unit, and pair of units
    if (two && (n.pair >> p) & 1u) return q == p ? 3 : -1;
    if ((n.unit >> u) & 1u) return q == u ? 2 : -1;
    if ((n.half >> (q & ~1)) & 1u) return q & 1 ? -1 : 1;
    return 0;
}

// 0 times a value that is not finite (a warp; lanes with `go` have a row each): dims [at, at + 128) of an output row (of
// out, or of partial result `part`) whose query saw a logit of -inf become NaN where one of the rows that it sees holds no
// finite value; all of them where it saw no other logit (l_run 0).  Rare: the warp reads all rows that its queries see,
// two at a time, eight in flight, and each lane gathers the dims of those that its own query sees.
template <bool QUANT>
__device__ __noinline__ void lat_not_finite(const LatArgs& a, int row, int part, int64_t prow, bool direct, int at,
                                            float l_run, bool go) {
    if (!QUANT) direct = a.parts == 1, prow = (int64_t)part * a.rows + row;
    const int64_t to = (direct ? (int64_t)row : prow) * D + at;
    auto put = [&](int d) {
        if (direct) a.out[to + d] = 0x7FFFu;
        else a.part_o[to + d] = __int_as_float(0x7FFFFFFF);
    };
    if (l_run != l_run) go = false;  // all NaN already
    if (go && l_run == 0.f) {
        if (direct) {
#pragma unroll 1
            for (int d = 0; d < 128; ++d) put(d);
            go = false;
        } else if (at == 0) {
            a.part_lse[prow] = LP_LSE_LOST;
        }
    }
    int lo = 0, hi = 0, sinks = 0, b = 0;
    if (go) {
        b = div_by(row, a.by_H);
        if (a.n_rows) {
            const int64_t n = __ldg(a.n_rows + b);
            lo = part < a.SP ? 0 : a.n_shared;
            hi = (int)max(min(n, (int64_t)(part < a.SP ? a.n_shared : a.max_rows)), (int64_t)0);
            if (part < a.SP) b = 0;
        } else {
            const int64_t tok = b;
            b = seq_of(a, tok);
            const int64_t q0 = __ldg(a.q_offsets + b), q1 = __ldg(a.q_offsets + b + 1), nt = __ldg(a.n_tokens + b);
            hi = seq_valid(a, q0, q1, nt) ? (int)max(nt - (q1 - tok) + 1, (int64_t)0) : 0;
            lo = max(0, hi - a.window);
            sinks = min(a.n_sink, lo);
        }
    }
    const unsigned all = 0xffffffffu, who = __ballot_sync(all, go);
    if (!who) return;
    // the rows of an item come through one row of the table: sinks, then what any of the queries sees
    const int32_t* pt = a.kv.pt + (int64_t)__shfl_sync(all, b, __ffs(who) - 1) * a.kv.pt_stride;
    const int s1 = __reduce_max_sync(all, sinks);
    const int l1 = max(__reduce_min_sync(all, go ? lo : 0x7FFFFFFF), s1), h1 = __reduce_max_sync(all, hi);
    const uint32_t total = (uint32_t)s1 + (uint32_t)max(h1 - l1, 0);
    auto key = [&](uint32_t k) { return k < (uint32_t)s1 ? (int)k : (int)(k - (uint32_t)s1) + l1; };
    const int lane = threadIdx.x & 31, half = lane >> 4, c = lane & 15;
    uint32_t acc[4] = {0, 0, 0, 0};  // [x / 2], 16 bits for each x: bit c is dim 8 c + x
#pragma unroll 1
    for (uint32_t k0 = 0; k0 < total; k0 += 8) {
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t k = k0 + 2 * e + half;
            v[e] = make_uint4(0, 0, 0, 0);
            if (k >= total) continue;
            int slot;
            const int pg = lat_entry(a, pt, key(k), slot);
            if (pg < 0 || pg >= a.kv.n_pages) continue;
            if (QUANT) {
                const uint8_t* row = q_codes(a.kv.base, a.kv.page_stride, pg, slot);
                const uint2 w = __ldg(reinterpret_cast<const uint2*>(row + at) + c);
                const uint32_t s = __ldg(q_scales(a.kv.base, a.kv.page_stride, a.kv.rpp, pg, slot) + at / 128);
                uint4 none;
                q_values(make_uint4(w.x, w.y, 0, 0), q_factor(s), v[e], none);
                q_times(v[e], q_factor_rest(s));
                const uint2 x = e4m3x4_nan(w.x), y = e4m3x4_nan(w.y);
                v[e].x |= x.x, v[e].y |= x.y, v[e].z |= y.x, v[e].w |= y.y;
            } else {
                v[e] = __ldg(reinterpret_cast<const uint4*>(a.kv.base + (int64_t)pg * a.kv.page_stride +
                                                            (int64_t)slot * ROW_BYTES + at * 2) + c);
            }
        }
#pragma unroll 1
        for (int e = 0; e < 4; ++e) {
            const uint4 u = e == 0 ? v[0] : e == 1 ? v[1] : e == 2 ? v[2] : v[3];
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
            uint32_t bad = 0;
#pragma unroll
            for (int x = 0; x < 8; ++x)
                if (((w[x >> 1] >> (16 * (x & 1))) & 0x7F80u) == 0x7F80u) bad |= 1u << x;
            if (!__any_sync(all, bad != 0)) continue;
            uint32_t sees = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t k = k0 + 2 * e + h;
                const int j = key(k);
                if (go && k < total && (j < sinks || (j >= lo && j < hi))) sees |= 0xFFFFu << (16 * h);
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint32_t m = __ballot_sync(all, (bad >> x) & 1u) & sees;
                acc[x >> 1] |= ((m | (m >> 16)) & 0xFFFFu) << (16 * (x & 1));
            }
        }
    }
#pragma unroll 1
    for (int d = 0; d < 16; ++d)
#pragma unroll
        for (int x = 0; x < 8; ++x)
            if ((acc[x >> 1] >> (16 * (x & 1) + d)) & 1u) put(8 * d + x);
}

// Quantised rows: log2 units of a logit, sl2 2^e with sl2 in [1, 2): the scale's, the query's and the row's powers of two are
// added up in e, before any of them could pass fp32's range.  At least the least number above 0 (a masked logit stays
// -inf), and finite (one of 0 stays 0).
__device__ __forceinline__ float lat_unit(float sl2, int e) {
    e = min(max(e, -252), 254);
    const int h = e >> 1;
    const float u = sl2 * __uint_as_float((uint32_t)(h + 127) << 23) * __uint_as_float((uint32_t)(e - h + 127) << 23);
    return fminf(fmaxf(u, __int_as_float(1)), 3.4028235e38f);
}
// The part of e of a query whose largest value has the exponent E and is now in [2^14, 2^15), for rows that are 2^Q_UP as
// large as they should be.
__device__ __forceinline__ int lat_q_power(uint32_t E) { return (int)E - 141 - Q_UP; }

// The larger of top and v's magnitudes, as the bits of two bf16.
__device__ __forceinline__ uint32_t max_magnitude(uint32_t top, const uint4& v) {
    constexpr uint32_t m = 0x7FFF7FFFu;
    return __vmaxu2(__vmaxu2(top, v.x & m), __vmaxu2(v.y & m, __vmaxu2(v.z & m, v.w & m)));
}

// The CTA's 64 rows of Q in place from bf16 to fp16, each with its largest value in [2^14, 2^15) (the softmax
// warps).  Returns the row's lat_q_power().  A value 2^29 below its row's largest still has all
// its bits, and what is lost of smaller ones is 2^-39 of the largest.
__device__ __noinline__ int lat_q_to_f16(uint32_t sb, float* shared, int tid, bool wanted) {
    const int r = tid & 63;
    const uint32_t row = sb + (uint32_t)(tid >> 6) * 2 * LP_QSLAB + (uint32_t)r * 128;
    uint4 v[16];
    uint32_t top = 0;
    if (wanted) {
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            v[c] = ld_shared_v4(row + (c >> 3) * LP_QSLAB + (((c & 7) ^ (r & 7)) << 4));
            top = max_magnitude(top, v[c]);
        }
        if (LAT_RARE((top & 0x7FFFu) >= 0x7F80u || (top >> 16) >= 0x7F80u)) {  // infinities and NaN do not count
            top = 0;
#pragma unroll 1
            for (int c = 0; c < 64; ++c) {
                const uint32_t w = ld_shared_u32(row + (c >> 5) * LP_QSLAB + (c & 31) * 4);  // (in whatever order)
                if ((w & 0x7F80u) != 0x7F80u) top = max(top, w & 0x7FFFu);
                if ((w & 0x7F800000u) != 0x7F800000u) top = max(top, (w >> 16) & 0x7FFFu);
            }
        }
        top = max(top & 0xFFFFu, top >> 16);
    }
    shared[tid] = __uint_as_float(top);
    named_bar_sync(1, 32 * LP_SOFT);
    top = max(max(top, __float_as_uint(shared[tid ^ 64])),
              max(__float_as_uint(shared[tid ^ 128]), __float_as_uint(shared[tid ^ 192])));
    const uint32_t E = max(top >> 7, 15u);
    const float f = __uint_as_float((268u - E) << 23);
    if (wanted) {
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&v[c]);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = pack_f16x2(bf16lo(w[e]) * f, bf16hi(w[e]) * f);
            st_shared_v4(row + (c >> 3) * LP_QSLAB + (((c & 7) ^ (r & 7)) << 4), v[c]);
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if ((tid & 31) == 0) mbar_arrive_rank(sb + LP_QREADY, 0);
    return lat_q_power(E);
}

// The same by the two warps that do nothing else, of all items but the first, a lane a row: beside the softmax and the
// output of the item before (a prompt of 4K under a window of 128, two tiles an item: 610 -> 486 us).
__device__ __forceinline__ void lat_q_row(uint32_t sb, uint32_t top_at, int r) {
    const uint32_t row = sb + (uint32_t)r * 128;
    uint32_t top = 0;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint4 v = ld_shared_v4(row + c * LP_QSLAB + (uint32_t)((e ^ r) & 7) * 16);
            top = max_magnitude(top, v);
        }
    }
    if (LAT_RARE((top & 0x7FFFu) >= 0x7F80u || (top >> 16) >= 0x7F80u)) {
        top = 0;
#pragma unroll 1
        for (int c = 0; c < 256; ++c) {
            const uint32_t w = ld_shared_u32(row + (c >> 5) * LP_QSLAB + (c & 31) * 4);
            if ((w & 0x7F80u) != 0x7F80u) top = max(top, w & 0x7FFFu);
            if ((w & 0x7F800000u) != 0x7F800000u) top = max(top, (w >> 16) & 0x7FFFu);
        }
    }
    const uint32_t E = max(max(top & 0xFFFFu, top >> 16) >> 7, 15u);
    const uint64_t f = f32x2_bits((268u - E) << 23, (268u - E) << 23);
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t at = row + c * LP_QSLAB + (uint32_t)((e ^ r) & 7) * 16;
            uint4 v = ld_shared_v4(at);
            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float2 y = f32x2_split(f32x2_mul(f32x2(bf16lo(w[x]), bf16hi(w[x])), f));
                w[x] = pack_f16x2(y.x, y.y);
            }
            st_shared_v4(at, v);
        }
    }
    st_shared_u8(top_at, E);
}

// The pieces that a warp of the loading warps has stored at `to`: values of 2^128 and more become infinities (limit: of
// row `lane` of 16, in fp16 and its row's unit).  Rows that csa_quant_write made have none.
__device__ __noinline__ void lat_infinities(uint32_t to, uint32_t limit, int r0) {
#pragma unroll 1
    for (int e = 0; e < 16; ++e) {
        const uint32_t most = __shfl_sync(0xffffffffu, limit, (e & 14) + r0);
        const uint32_t ad = ((to ^ ((e & 6) << 4)) + (e >> 1) * 256) ^ ((e & 1) << 4);
        uint4 v = ld_shared_v4(ad);
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t lo = w[x] & 0x7FFFu, hi = (w[x] >> 16) & 0x7FFFu;
            if (lo >= most && lo < 0x7C00u) w[x] = (w[x] & 0xFFFF8000u) | 0x7C00u;
            if (hi >= most && hi < 0x7C00u) w[x] = (w[x] & 0x8000FFFFu) | 0x7C000000u;
        }
        st_shared_v4(ad, v);
    }
}

// Whether any of n logits is not finite (a warp).
__device__ __noinline__ bool lat_infinite(uint32_t ts, int n) {
    uint32_t v = 0;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
        v = max(v, tc_ld1(ts + j) & 0x7FFFFFFFu);
        __syncwarp();
    }
    return v >= 0x7F800000u;
}

// How a kernel's key rows are laid out and copied: bf16 rows by gathers or in boxes, or quantised rows, which the loading
// warps turn into fp16.
// (LK_QUANT4: four rows always share a page; LK_QUANT1: pages of any number of rows.)
enum LatKeys { LK_GATHER, LK_BOX, LK_QUANT4, LK_QUANT1 };
__host__ __device__ constexpr bool lat_quant(LatKeys keys) { return keys == LK_QUANT4 || keys == LK_QUANT1; }

__host__ __device__ constexpr int lat_loaders(LatKeys keys) { return lat_quant(keys) ? 8 : LP_PROD; }
constexpr int LQ_WARPS = 2;  // quantised rows: warps for the queries
__host__ __device__ constexpr int lat_threads(LatKeys keys) {
    return 32 * (LP_SOFT + 2 + lat_loaders(keys) + (lat_quant(keys) ? LQ_WARPS : 0));
}
static_assert(lat_threads(LK_QUANT4) == 640, "five warpgroups: 2 x 104 + 3 x 88 registers of 5 x 96 at the start");
static_assert(lat_threads(LK_BOX) == LP_T, "the bf16 kernels' warps");

// Ratios and factors of a tile whose rows each keep a scale of their own (lane l with rows 4 l ..., those of v there).
__device__ __noinline__ uint32_t quant_uneven(uint32_t ratios, uint32_t factors, uint4 scales, uint32_t v) {
    const uint32_t sc[4] = {scales.x, scales.y, scales.z, scales.w};
    uint32_t f[4], r[8], most = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t top = (v >> e) & 1u ? q_top(sc[e]) : 127u;
        most = max(most, top);
        f[e] = q_power(top);
        const uint2 w = (v >> e) & 1u ? q_ratios_any(sc[e], top) : make_uint2(0, 0);
        r[2 * e] = w.x, r[2 * e + 1] = w.y;
    }
    st_shared_v4(factors, make_uint4(f[0], f[1], f[2], f[3]));
    st_shared_v4(ratios, make_uint4(r[0], r[1], r[2], r[3]));
    st_shared_v4(ratios + 16, make_uint4(r[4], r[5], r[6], r[7]));
    most = __reduce_max_sync(0xffffffffu, most);
    return most << LQ_TOP | (most >= 247u ? LQ_HUGE : 0u);
}

template <LatKeys KEYS, bool WINDOW>
__device__ __forceinline__ void lat_pair(const CUtensorMap& qmap, const KeyMaps& km, const LatArgs& a) {
    constexpr bool QUANT = lat_quant(KEYS);
    extern __shared__ uint8_t lp_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(lp_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = (smem_u32(lp_raw) + 1023u) & ~1023u;  // (the same address, without a detour over generic ones)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    volatile uint32_t* dead = reinterpret_cast<volatile uint32_t*>(sm + LP_SM_DEAD);
    volatile int* closed = reinterpret_cast<volatile int*>(sm + LP_SM_CLOSED);

    if (warp == 0) {
        tmem_alloc_pair(sb + LP_SM_TMEM, 512);
        tmem_relinquish_pair();
    }
    if (tid == 64) {
        prefetch_tensormap(&qmap);
        if (!QUANT) prefetch_tensormap(&km.m[0]);
    }
    if (tid >= 96 && tid < 96 + 65) reinterpret_cast<volatile int*>(sm + LP_SM_LOST)[tid - 96] = 0;
    if (tid == 32) {
        for (int i = 0; i < LP_SLOTS; ++i) {
            mbar_init(sb + LP_FULL + 8 * i, QUANT ? 8 : 1);  // even CTA: both CTAs' rows
            mbar_init(sb + LP_EMPTY + 8 * i, 1);
            mbar_init(sb + LP_LOOK + 8 * i, 1);
            mbar_init(sb + LP_USED + 8 * i, lat_loaders(KEYS));
        }
        mbar_init(sb + LP_QFULL, 1);
        mbar_init(sb + LP_QEMPTY, 1);
        if (QUANT) mbar_init(sb + LP_QREADY, 2 * LP_SOFT);
        if (QUANT) mbar_init(sb + LP_QTOP, LQ_WARPS), mbar_init(sb + LP_QTOP + 8, LQ_WARPS);
        mbar_init(sb + LP_SFULL, 1);
        mbar_init(sb + LP_SFULL + 8, 1);
        mbar_init(sb + LP_PREADY, 2 * LP_SOFT);  // the softmax warps of both CTAs
        mbar_init(sb + LP_PREADY + 8, 2 * LP_SOFT);
        mbar_init(sb + LP_PVDONE, 1);
        mbar_init(sb + LP_PVDONE + 8, 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(sb + LP_ITEM + 8 * i, 1);
            mbar_init(sb + LP_TAKEN + 8 * i, LP_SOFT + lat_loaders(KEYS) + (QUANT ? LQ_WARPS : 0) + (rank == 0 ? 1 : 0));
        }
        *dead = 0;
        *closed = 0x7FFFFFFF;
        *reinterpret_cast<uint32_t*>(sm + LP_SM_WANT) = *reinterpret_cast<uint32_t*>(sm + LP_SM_LAND) = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    pdl_wait();
    const uint32_t tmem = 0;  // an allocation of all 512 columns
    LatItem x;
    int sidx = 0, g = 0, n = 0, q = 0;  // ring slots, tiles, items with tiles and items so far
    bool ok = true;
    // The next item as warp 9 left it; false behind the last one, and when a wait has run out.
    auto next_item = [&]() -> bool {
        const bool in = lat_wait_item<QUANT>(sb + LP_ITEM + 8 * (q & 3), (q >> 2) & 1, q, closed);
        x = load_item(sb + LP_SM_ITEM + (q & 3) * 128);
        __syncwarp();
        if (lane == 0) mbar_arrive(sb + LP_TAKEN + 8 * (q & 3));
        ++q;
        ok = ok && in;
        return in && x.T >= 0;
    };

    if (QUANT && warp >= LP_SOFT) setmaxnreg_dec<88>();
    if (warp < LP_SOFT) {
        // ---------------------------------------------------------------- softmax and output
        if (QUANT) setmaxnreg_inc<104>();
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const int r = tid & 63, half = (warp >> 1) & 1, ch = warp >> 2;
        float* mx = reinterpret_cast<float*>(sm + LP_SM_MAX);
        float* ls = reinterpret_cast<float*>(sm + LP_SM_SUM);
        volatile int* lost = reinterpret_cast<volatile int*>(sm + LP_SM_LOST);  // (items are counted from 1)
        while (next_item()) {
            const int row = x.row0 + (int)rank * 64 + r;  // this thread's query row
            const bool mine = (int)rank * 64 + r < x.nrows;
            const bool some = !QUANT || __any_sync(0xffffffffu, mine);  // (warps without a row only wait, as a rule)
            // rows that this query sees: [vlo, vhi) and [0, vs)
            int vlo = 0, vhi = 0, vs = 0;
            if (mine) {
                if (WINDOW) {
                    const int64_t pos = x.pos0 + div_by(x.rr0 + (int)rank * 64 + r, a.by_H);
                    vhi = pos >= 0 ? (int)pos + 1 : 0;
                    vlo = max(0, vhi - a.window);
                    vs = min(a.n_sink, vhi);
                } else if (x.shared) {
                    const int64_t nr = __ldg(a.n_rows + div_by(row, a.by_H));
                    vhi = nr < 0 ? 0 : (nr > x.hi ? x.hi : (int)nr);
                } else {
                    vlo = x.lo;
                    vhi = x.hi;
                }
            }
            int qe = 0;  // quantised: the query's and the scale's power of two in its logits
            if (QUANT && x.T > 0) {  // (the first item's queries have nobody else to wait for)
                ok = lat_wait<QUANT>(sb + (n ? LP_QTOP + 8 * (n & 1) : LP_QFULL), (n ? (n - 1) >> 1 : 0) & 1, dead) && ok;
                qe = n ? lat_q_power(ld_shared_u8(sb + LP_SM_QTOP + (n & 1) * 64 + r))
                       : lat_q_to_f16(sb, mx + (g & 1) * 256, tid, some);
                qe += a.sl2_power;
                ++n;
            }
            float m_run = -INFINITY, y_run = -INFINITY, l_run = 0.f;
            int most = 0;
            for (int i = 0; i < x.T; ++i, ++g) {
                const int nu = item_units(x, i), mu = (nu + 1) >> 1;  // units in all, and per half
                const int c0 = ch ? (mu + 1) >> 1 : 0, nc = ch ? mu - c0 : (mu + 1) >> 1;  // this thread's
                const int ub = half * mu + c0, u0 = (x.t0 + i) * 8;
                // the tile's lookups and its S, waited for together (even and odd lanes)
                ok = __all_sync(0xffffffffu, lane & 1 ? lat_wait<QUANT>(sb + LP_LOOK + 8 * (g & 7), (g >> 3) & 1, dead)
                                                      : lat_wait<QUANT>(sb + LP_SFULL + 8 * (g & 1), (g >> 1) & 1, dead)) && ok;
                tc_fence_after();
                uint32_t sr[32];
                const uint32_t ts = tmem + 256 + (uint32_t)((g & 1) * 64 + 16 * c0) + lane_off;
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (c < nc && some) tc_ld16(ts + 16 * c, sr + 16 * c);
                const uint32_t kind = ld_shared_u32(sb + LP_SM_PLAIN + (g & 7) * 4);
                const bool plain = QUANT ? (kind & LQ_PLAIN) != 0 : kind != 0;
                // quantised: one scale for all rows; the largest one, of the item's tiles too
                const bool even = QUANT && (kind & LQ_EVEN);
                const int top = (int)(kind >> LQ_TOP);
                most = max(most, top);
                tc_wait_ld();
                float mt = -INFINITY;  // of the logits before scaling
                bool bad = false;
                float* xs = reinterpret_cast<float*>(sr);
                // the unit of a logit; quantised: the largest weight times its row's scale, in log2 units; log2 of the tile's
                // scale
                float yt = -INFINITY, tsl2 = QUANT ? 1.f : a.sl2, tpow = 0.f;
                const uint32_t fa = sb + LP_SM_FACTOR + (uint32_t)(g & 7) * 512 + (uint32_t)ub * 64;
                if (QUANT) {
                    if (even) {
                        const int e = qe + top;  // (biased by 127)
                        tpow = (float)(top - 127);
                        tsl2 = a.sl2 * __uint_as_float((uint32_t)e << 23);
                        if (LAT_RARE(__any_sync(0xffffffffu, (uint32_t)(e - 1) >= 254u))) tsl2 = lat_unit(a.sl2, e - 127);
                    } else if (LAT_RARE(some)) {
                        // the logits themselves, in log2 units: times what makes them small before the rows' scales, times
                        // what makes them large behind them
                        const float u = lat_unit(a.sl2, qe);
                        const uint64_t u0 = qe < 0 ? f32x2(u, u) : f32x2(1.f, 1.f);
                        const uint64_t u1 = qe < 0 ? f32x2(1.f, 1.f) : f32x2(u, u);
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (c < nc) {
#pragma unroll
                                for (int j = 0; j < 16; j += 2) {
                                    const uint2 f = ld_shared_v2(fa + 64 * c + 4 * j);
                                    float* y = xs + 16 * c + j;
                                    const uint64_t v = f32x2_mul(f32x2_mul(f32x2(y[0], y[1]), u0), f32x2_bits(f.x, f.y));
                                    const float2 p = f32x2_split(f32x2_mul(v, u1));
                                    y[0] = p.x, y[1] = p.y;
                                }
                            }
                    }
                }
                if (!some) {
                    // (a CTA without any row has half of the values' dims all the same: it looks at the logits of the rows
                    // that it does not have, which are not finite where a key is not)
                    if (LAT_RARE(!plain && (int)rank * 64 >= x.nrows)) {
                        bad = lat_infinite(ts, 16 * min(nc, nu - ub));
                    }
                } else if (plain) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) mt = fmaxf(mt, xs[j]);
                } else {
                    const uint4 vw = ld_shared_v4(sb + LP_SM_VALID + (g & 7) * 16);
                    uint64_t z = 0;  // NaN where a logit of the tile is not finite
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int u = ub + c;
                        if (c < nc) {
                            uint32_t bits = 0;
                            if (u < nu) {
                                const int jb = unit_row<WINDOW>(x, u0 + u);
                                const int e0 = min(max(vlo - jb, 0), 16), e1 = min(max(vhi - jb, 0), 16);
                                const int e2 = min(max(vs - jb, 0), 16);
                                bits = (((1u << e1) - 1u) & ~((1u << e0) - 1u)) | ((1u << e2) - 1u);
                                const uint32_t vv = u < 4 ? (u < 2 ? vw.x : vw.y) : (u < 6 ? vw.z : vw.w);
                                bits &= vv >> ((u & 1) * 16);
#pragma unroll
                                for (int j = 0; j < 16; j += 2)
                                    z = f32x2_fma(f32x2(xs[16 * c + j], xs[16 * c + j + 1]), 0ull, z);
                            }
                            if (!__all_sync(0xffffffffu, bits == 0xFFFFu)) {
#pragma unroll
                                for (int j = 0; j < 16; ++j)
                                    if (!((bits >> j) & 1u)) xs[16 * c + j] = -INFINITY;
                            }
#pragma unroll
                            for (int j = 0; j < 16; ++j) mt = fmaxf(mt, xs[16 * c + j]);
                        }
                    }
                    const float2 zz = f32x2_split(z);
                    bad = !(zz.x == 0.f) || !(zz.y == 0.f);
                }
                mt *= tsl2;
                if (QUANT && LAT_RARE(!even && some)) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        if (c < nc) {
#pragma unroll
                            for (int j = 0; j < 16; j += 2) {
                                const uint2 f = ld_shared_v2(fa + 64 * c + 4 * j);
                                yt = fmaxf(yt, fmaxf(xs[16 * c + j] + q_log(f.x), xs[16 * c + j + 1] + q_log(f.y)));
                            }
                        }
                }
                // the row's other quarters, and whether any logit of the tile is not finite
                float* mb = mx + (g & 1) * 256;
                float* yb = reinterpret_cast<float*>(sm + (g & 1 ? LP_SM_SUM : LP_SM_MORE));
                mb[tid] = mt;
                if (QUANT && !even) yb[tid] = yt;
                const bool any_bad = named_bar_any(1, 32 * LP_SOFT, bad);
                mt = fmaxf(fmaxf(mt, mb[tid ^ 64]), fmaxf(mb[tid ^ 128], mb[tid ^ 192]));
                float alpha = 1.f;  // of O; of the sum, quantised: alpha_l
                if (QUANT) {
                    if (even) yt = mt + tpow;
                    else yt = fmaxf(fmaxf(yt, yb[tid ^ 64]), fmaxf(yb[tid ^ 128], yb[tid ^ 192]));
                    if (yt > -INFINITY) {
                        if (y_run == -INFINITY) {
                            y_run = yt;
                        } else if (yt > y_run + LP_RESCALE) {
                            alpha = lat_ex2(y_run - yt);
                            y_run = yt;
                        }
                    }
                }
                float alpha_l = 1.f;
                if (mt > -INFINITY) {
                    if (m_run == -INFINITY) {
                        m_run = mt;
                    } else if (mt > m_run + LP_RESCALE) {
                        alpha_l = lat_ex2(m_run - mt);
                        m_run = mt;
                    }
                    if (!QUANT) alpha = alpha_l;
                } else if (plain && some) {  // every logit is -inf or NaN
                    lost[r] = lost[64] = q;
                }
                const float mref = m_run == -INFINITY ? 0.f : m_run;
                const float yref = QUANT && y_run != -INFINITY ? y_run : 0.f;
                // Quantised and one scale: the weight in fp16 times that scale at once, and the sum without it.  Rows with
                // scales of their own, and a scale so far below another's that the sum's terms could be lost under 2^-126
                // (the two references are at most LP_RESCALE - LQ_ROOM further apart than the scales): a weight times its
                // scale has an exponential of its own (a weight, a scale and the largest product may each be next to
                // nothing).
                const bool two = QUANT && some && LAT_RARE(!even || most - top > LQ_APART);
                const float ref = even && !two ? yref - tpow - LQ_ROOM : mref;
                const uint64_t sl2 = f32x2(tsl2, tsl2), mneg = f32x2(-ref, -ref);
                uint64_t sum = 0;
                if (LAT_RARE(two)) {
                    const float shift = LQ_ROOM - yref;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        if (c < nc) {
#pragma unroll
                            for (int j = 0; j < 16; j += 2) {
                                const uint2 f = ld_shared_v2(fa + 64 * c + 4 * j);
                                const uint64_t y = f32x2(xs[16 * c + j], xs[16 * c + j + 1]);
                                const float2 e = f32x2_split(f32x2_fma(y, sl2, mneg));
                                const uint64_t with = f32x2(q_log(f.x) + shift, q_log(f.y) + shift);
                                const float2 t = f32x2_split(f32x2_fma(y, sl2, with));
                                sum = f32x2_add(sum, f32x2(lat_ex2(e.x), lat_ex2(e.y)));
                                xs[16 * c + j] = lat_ex2(t.x), xs[16 * c + j + 1] = lat_ex2(t.y);
                            }
                        }
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if (c < nc && some) {
#pragma unroll
                            for (int j = 0; j < 16; j += 2) {
                                const uint64_t y = f32x2(xs[16 * c + j], xs[16 * c + j + 1]);
                                const float2 e = f32x2_split(f32x2_fma(y, sl2, mneg));
                                const float p0 = lat_ex2(e.x), p1 = lat_ex2(e.y);
                                sum = f32x2_add(sum, f32x2(p0, p1));
                                if (!QUANT) sr[8 * c + (j >> 1)] = pack_bf16x2(p0, p1);
                                else xs[16 * c + j] = p0, xs[16 * c + j + 1] = p1;
                            }
                        }
                    }
                }
                const float2 ss = f32x2_split(sum);
                l_run = l_run * alpha_l + (even ? lat_ex2(ref - mref) * (ss.x + ss.y) : ss.x + ss.y);
                if (QUANT && some) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        if (c < nc) {
#pragma unroll
                            for (int j = 0; j < 16; j += 2)
                                sr[8 * c + (j >> 1)] = pack_f16x2(xs[16 * c + j], xs[16 * c + j + 1]);
                        }
                }
                // P and O are free once the product before this one is done; a short tile, the item's last, has a
                // slab of its own for P, and as a rule leaves O alone
                const bool tail = WINDOW && !QUANT && nu <= 4;
                if (i > 0 && (!tail || any_bad || __any_sync(0xffffffffu, alpha != 1.f))) {
                    ok = lat_wait<QUANT>(sb + LP_PVDONE + 8 * ((g - 1) & 1), ((g - 1) >> 1) & 1, dead) && ok;
                    tc_fence_after();
                    if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                        for (int c = 128 * ch; c < 128 * ch + 128; c += 32) {
                            uint32_t o[32];
                            tc_ld32(tmem + lane_off + c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tc_st32(tmem + lane_off + c, o);
                        }
                        tc_wait_st();
                    }
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (c < nc && some) {
                        const int u = ub + c;
                        const uint32_t pb = sb + LP_SM_P + (uint32_t)(tail ? 2 : u >> 2) * LP_QSLAB + (uint32_t)r * 128;
#pragma unroll
                        for (int h2 = 0; h2 < 2; ++h2)
                            st_shared_v4(pb + ((uint32_t)(((u & 3) * 2 + h2) ^ (r & 7)) << 4),
                                         make_uint4(sr[8 * c + 4 * h2], sr[8 * c + 4 * h2 + 1], sr[8 * c + 4 * h2 + 2],
                                                    sr[8 * c + 4 * h2 + 3]));
                    }
                }
                if (QUANT ? LAT_RARE(any_bad) : any_bad) {  // non-finite values of this CTA's V rows -> 0
#pragma unroll 1
                    for (int j = 0; j < 16 * nc; ++j) {
                        __syncwarp();
                        const uint32_t w = tc_ld1(ts + j);  // (S stays until this warp reports P)
                        const int u = ub + (j >> 4), k = unit_row<WINDOW>(x, u0 + u) + (j & 15);
                        if (w != 0xFF800000u || u >= nu || !(k < vs || (k >= vlo && k < vhi))) continue;
                        const uint32_t vv = ld_shared_u32(sb + LP_SM_VALID + (g & 7) * 16 + (u >> 1) * 4);
                        if ((vv >> ((u & 1) * 16 + (j & 15))) & 1u) lost[r] = lost[64] = q;
                    }
                    // (the products' thread, waiting for P, answers; a warp that gave up lets its own wait run out)
                    if (lane == 0) st_dsmem_u32(mapa(sb + LP_SM_WANT, 0), (uint32_t)g + 1);
                    ok = lat_word(sb + LP_SM_LAND, (uint32_t)g + 1, dead) && ok;
                    fence_cluster();
                    const int vs0 = sidx + 4 * min(i + 2, x.T) + 4 * i;  // the tile's first V slot
#pragma unroll 1
                    for (int s = 0; s < (nu + 1) >> 1; ++s) {
                        const int sl = QUANT ? 4 + s : (vs0 + s) & (LP_SLOTS - 1);
                        const uint32_t bytes = (uint32_t)min(2, nu - 2 * s) * 2048u;  // of each 4,096-byte slab
#pragma unroll 1
                        for (uint32_t c = tid * 16; c < LP_SLOT; c += 32 * LP_SOFT * 16) {
                            if ((c & 4095u) >= bytes) continue;
                            const uint32_t ad = sb + LP_SM_RING + (uint32_t)sl * LP_SLOT + c;
                            uint4 v = ld_shared_v4(ad);
                            uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                constexpr uint32_t top = QUANT ? 0x7C00u : 0x7F80u;  // exponent: no number
                                if ((w[e] & top) == top) w[e] &= 0xFFFF0000u;
                                if ((w[e] & (top << 16)) == top << 16) w[e] &= 0xFFFFu;
                            }
                            st_shared_v4(ad, v);
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_rank(sb + LP_PREADY + 8 * (g & 1), 0);
            }
            // while the last product runs: the row's sum, its lse and where its output goes
            if (x.T > 0) {
                sidx += 8 * x.T;
                if (QUANT) ls = reinterpret_cast<float*>(sm + (g & 1 ? LP_SM_SUM : LP_SM_MORE));
                ls[tid] = l_run;
                named_bar_sync(1, 32 * LP_SOFT);
                l_run = (ls[r] + ls[r + 64]) + (ls[r + 128] + ls[r + 192]);
                if (QUANT) named_bar_sync(1, 32 * LP_SOFT);  // (the next tile's maxima go there)
            }
            float inv = l_run == 0.f ? 0.f : 1.f / l_run, old = 0.f;  // what was there counts `old`
            // quantised: O's unit too; one next to nothing would leave inv no bits, so that its root comes in twice
            float root = 1.f;
            if (QUANT && l_run != 0.f) {
                const float unit = y_run - m_run - LQ_ROOM - Q_UP;
                if (LAT_RARE(unit < -64.f)) root = lat_ex2(0.5f * unit);
                else inv *= lat_ex2(unit);
            }
            const bool direct = QUANT ? (x.shared & QUANT_DIRECT) != 0 : a.parts == 1;
            const bool more = QUANT && (x.shared & QUANT_MORE) != 0;
            // this row of the partial results
            const int64_t prow = QUANT ? (int64_t)x.part * a.slot_rows + (int)rank * 64 + r : 0;
            bool had = false;
            float e = 0.f;  // (bf16 rows: of the threads that store it; with that and a place of the partial results in
                            // every thread a prompt of 8K tokens took 1 percent more)
            if (QUANT || (tid < 64 && mine)) e = l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * LP_LN2;
            if (more) {
                const float before = mine ? __ldcg(a.part_lse + prow) : -INFINITY;
                had = before != -INFINITY;
                if (before != before) e = before;  // (fmaxf would leave a NaN out)
                const float top = fmaxf(e, before);
                if (top > -INFINITY) {
                    const float w0 = had ? lat_ex2((before - top) * LP_LOG2E) : 0.f;
                    const float w1 = e == -INFINITY ? 0.f : lat_ex2((e - top) * LP_LOG2E);
                    inv *= w1 / (w0 + w1);
                    old = w0 / (w0 + w1);
                    if (had) l_run = 1.f;
                    e = top == LP_LSE_LOST ? top : top + log2f(w0 + w1) * LP_LN2;
                    if (direct && top == LP_LSE_LOST) e = -INFINITY, inv = __int_as_float(0x7FFFFFFF);
                }
                named_bar_sync(1, 32 * LP_SOFT);  // (a row's threads have all read what one of them replaces)
            }
            if (tid < 64 && mine) {
                if (!direct) a.part_lse[QUANT ? prow : (int64_t)x.part * a.rows + row] = e;
                else if (a.lse) a.lse[row] = e;
            }
            // ---- row r of the CTA, dims [256 half + 128 ch, + 128), normalised.  Four lanes exchange their rows'
            //      sectors, so that a store covers 128 bytes of each of 8 rows: an SM's stores leave at 43 bytes a
            //      cycle so, and at 17 with a sector of each of 32 rows (a 64 KB item: 1,520 and 3,250 cycles).
            if (direct || x.T > 0) {
                const int at = half * 256 + ch * 128, j = lane & 3;
                const int64_t gr = row - j;  // the group's first row
                const int left = x.nrows - ((int)rank * 64 + r - j);
                uint8_t* dst = (direct ? reinterpret_cast<uint8_t*>(a.out + gr * D + at)
                                       : reinterpret_cast<uint8_t*>(
                                             a.part_o + (QUANT ? prow - j : (int64_t)x.part * a.rows + gr) * D + at)) +
                               j * 32;
                const float* was = a.part_o + prow * D + at;  // (more)
                const int64_t pitch = direct ? D * 2 : D * 4;
                if (x.T > 0) {
                    ok = lat_wait<QUANT>(sb + LP_PVDONE + 8 * ((g - 1) & 1), ((g - 1) >> 1) & 1, dead) && ok;
                    tc_fence_after();
                }
                if (LAT_RARE(more || (QUANT && __any_sync(0xffffffffu, root != 1.f)))) {
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        uint32_t o[32];
                        tc_ld32(tmem + lane_off + 128 * ch + c, o);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float there = had ? old * __ldcg(was + c + e) : 0.f;
                            o[e] = __float_as_uint(fmaf(__uint_as_float(o[e]) * inv * root, root, there));
                        }
                        tc_st32(tmem + lane_off + 128 * ch + c, o);
                    }
                    tc_wait_st();
                    inv = 1.f;
                    __syncwarp();  // (the row's lanes have read what the group is about to write)
                }
#pragma unroll 1
                for (int c = 0; c < (!some ? 0 : direct ? 2 : 4); ++c) {
                    uint32_t v[32];  // 128 bytes of this lane's row
                    if (x.T == 0) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = 0;
                    } else if (direct) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t o[32];
                            const uint64_t inv2 = f32x2(inv, inv);
                            tc_ld32(tmem + lane_off + 128 * ch + 64 * c + 32 * h, o);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float2 f = f32x2_split(
                                    f32x2_mul(f32x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), inv2));
                                v[16 * h + e] = pack_bf16x2(f.x, f.y);
                            }
                        }
                    } else {
                        tc_ld32(tmem + lane_off + 128 * ch + 32 * c, v);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * inv);
                    }
                    // 4 x 4 transpose of sectors: lane j of a group ends with sector j of the group's rows 0 .. 3
                    auto exchange = [&](int p, int s) {
                        const bool up = (lane & s) != 0;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t lo = v[8 * p + e], hi = v[8 * (p | s) + e];
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, s);
                            v[8 * p + e] = up ? got : lo;
                            v[8 * (p | s) + e] = up ? hi : got;
                        }
                    };
                    exchange(0, 2);
                    exchange(1, 2);
#pragma unroll
                    for (int p = 0; p < 4; p += 2) {
                        exchange(p, 1);
#pragma unroll
                        for (int k = p; k < p + 2; ++k)
                            if (k < left) store_sector(dst + k * pitch + c * 128, v + 8 * k, a.wide_out || !direct);
                    }
                }
                tc_fence_before();
                if (QUANT ? LAT_RARE(lost[64] == q) : lost[64] == q) {
                    __syncwarp();  // (behind the other lanes' stores to this lane's row)
                    lat_not_finite<QUANT>(a, row, x.part, QUANT ? prow : 0, direct, half * 256 + ch * 128, l_run,
                                                     mine && lost[r] == q);
                }
            }
        }
    } else if (warp == LP_SOFT && rank == 0) {
        // ---------------------------------------------------------------- the products (one thread)
        if (elect_one()) {
            const uint64_t dk = sdesc_sw128(sb, 16, 1024), dv = sdesc_sw128(sb, 4096, 1024);
            const uint32_t klo = (uint32_t)dk, khi = (uint32_t)(dk >> 32), vlo = (uint32_t)dv, vhi = (uint32_t)(dv >> 32);
            auto desc = [](uint32_t lo, uint32_t hi, uint32_t off) -> uint64_t {
                return ((uint64_t)hi << 32) | (uint64_t)(lo + (off >> 4));
            };
            int T = 0, units = 0;
            auto take = [&]() {  // the next item that has tiles, or T < 0
                do {
                    ok = ok && lat_wait<QUANT>(sb + LP_ITEM + 8 * (q & 3), (q >> 2) & 1, dead);
                    const uint32_t at = sb + LP_SM_ITEM + (q & 3) * 128;
                    const uint2 tt = ld_shared_v2(at);  // T, t0
                    T = ok ? (int)tt.x : -1;
                    units = (int)ld_shared_u32(at + 8) - (int)tt.y * 8;
                    mbar_arrive(sb + LP_TAKEN + 8 * (q & 3));
                    ++q;
                } while (T == 0);
            };
            take();
            while (ok && T > 0) {
                const int T0 = T;
                ok = lat_wait<QUANT>(sb + (QUANT ? LP_QREADY : LP_QFULL), n & 1, dead);
                ++n;
                // S of tile i, then P V of tile i - 1.  Each slot's barrier is tested while the products of the slot
                // before it are issued: beside the copies and the products, a look at a barrier takes 150 cycles
                // and more.
#pragma unroll 1
                for (int i = 0; ok && i <= T0; ++i) {
                    if (i < T0) {
                        const int mu = (min(8, units - 8 * i) + 1) >> 1;
                        const uint32_t ids =  // N = 32 mu
                            (idesc_bf16_f32(128, 32, false) & ~(0x3Fu << 17) & ~(QUANT ? 0x480u : 0u)) |
                            ((uint32_t)(4 * mu) << 17) | a.negate;  // (quantised: both are fp16)
                        const uint32_t d = tmem + 256 + (uint32_t)((g + i) & 1) * 64;
                        const uint32_t reg = QUANT ? 0u : (uint32_t)(sidx >> 2) & 1;
                        const uint32_t bl = klo + ((LP_SM_RING + reg * 4 * LP_SLOT) >> 4);
                        const uint32_t par = (uint32_t)(QUANT ? g + i : sidx >> 3) & 1;
                        const uint32_t full = sb + LP_FULL + 32 * reg;
                        bool there = mbar_test_wait(full, par);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            if (!QUANT || !(kk & 1)) {  // (quantised: two slots at a time)
                                if (!there) ok = ok && lat_wait<QUANT>(full + 8 * kk, par, dead);
                                if (!ok) break;
                                if (QUANT ? kk < 2 : kk < 3) there = mbar_test_wait(full + 8 * kk + (QUANT ? 16 : 8), par);
                                tc_fence_after();
                            }
#pragma unroll
                            for (int s = 0; s < 2; ++s)
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    tc_mma_f16_pair(d, desc(klo, khi, (2 * kk + s) * LP_QSLAB + k * 32),
                                                    desc(bl, khi, kk * LP_SLOT + s * 8192 + k * 32), ids, (kk | s | k) ? 1u : 0u);
                            if (!QUANT || (kk & 1)) tc_commit_pair(sb + LP_EMPTY + 32 * reg + 8 * (QUANT ? kk - 1 : kk));
                        }
                        tc_commit_pair(sb + LP_SFULL + 8 * ((g + i) & 1));
                        if (i + 1 == T0) tc_commit_pair(sb + LP_QEMPTY);
                        sidx += 4;
                    }
                    if (i > 0 && ok) {
                        const int nu = min(8, units - 8 * (i - 1)), gt = g + i - 1;
                        const uint32_t reg = QUANT ? 1u : (uint32_t)(sidx >> 2) & 1;
                        const uint32_t par = (uint32_t)(QUANT ? gt : sidx >> 3) & 1;
                        const uint32_t bl = vlo + ((LP_SM_RING + reg * 4 * LP_SLOT) >> 4);
                        const uint32_t full = sb + LP_FULL + 32 * reg;
                        constexpr uint32_t idv = idesc_bf16_f32(128, 256, true) & ~(QUANT ? 0x480u : 0u);
                        bool there = mbar_test_wait(full, par);
                        const bool ready = mbar_test_wait(sb + LP_PREADY + 8 * (gt & 1), (gt >> 1) & 1);
                        if (!ready)
                            ok = ok && lat_wait_p<QUANT>(sb, full, par, (uint32_t)gt, dead);
                        tc_fence_after();
                        // (an operand whose place is no constant costs the products 5 percent: prefixes have one P)
                        const uint32_t pl = klo + ((LP_SM_P + (WINDOW && !QUANT && nu <= 4 ? 2 * LP_QSLAB : 0u)) >> 4);
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            if (!there) ok = ok && lat_wait<QUANT>(full + 8 * v, par, dead);
                            if (!ok) break;
                            if (v < 3) there = mbar_test_wait(full + 8 * v + 8, par);
                            tc_fence_after();
#pragma unroll
                            for (int u = 2 * v; u < 2 * v + 2; ++u) {
                                if (u >= nu) continue;
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    tc_mma_f16_pair(tmem + c * 128, desc(pl, khi, (u >> 2) * LP_QSLAB + (u & 3) * 32),
                                                    desc(bl, vhi, v * LP_SLOT + c * 8192 + (u & 1) * 2048), idv,
                                                    i == 1 && u == 0 ? 0u : 1u);
                            }
                            tc_commit_pair(sb + LP_EMPTY + 32 * reg + 8 * v);
                        }
                        tc_commit_pair(sb + LP_PVDONE + 8 * (gt & 1));
                        sidx += 4;
                    }
                }
                g += T0;
                take();
            }
        }
    } else if (warp == LP_SOFT + 1) {
        // ---------------------------------------------------------------- the tiles' pages, and Q
        const uint32_t qfull = mapa(sb + LP_QFULL, QUANT ? rank : 0);
        uint32_t* plain = reinterpret_cast<uint32_t*>(sm + LP_SM_PLAIN);
        SeqCursor cur;
        QuantCursor qc;
        for (int it = pair; ok; it += !WINDOW && a.run ? 0 : pairs, ++q) {
            bool there;
            if constexpr (QUANT) there = quant_item(a, qc, pair, pairs, lane, rank == 0, x);
            else there = lat_item<WINDOW>(a, cur, it, pairs, lane, rank == 0, x);
            if (!there) x.T = -1;
            if (q >= 4) ok = __all_sync(0xffffffffu, lat_wait<QUANT>(sb + LP_TAKEN + 8 * (q & 3), ((q >> 2) - 1) & 1, dead));
            if (!ok) break;  // (the item that is there may be in use)
            if (lane == 0) {
                *reinterpret_cast<LatItem*>(sm + LP_SM_ITEM + (q & 3) * 128) = x;
                mbar_arrive(sb + LP_ITEM + 8 * (q & 3));
            }
            __syncwarp();
            if (!there) break;
            const int32_t* pt = a.kv.pt + (int64_t)x.trow * a.kv.pt_stride;
            auto load_q = [&](int k) {
                if (k > 0) ok = __all_sync(0xffffffffu, lat_wait<QUANT>(sb + LP_QEMPTY, (k - 1) & 1, dead)) && ok;
                if (ok && (QUANT || rank == 0) && lane == 0)
                    mbar_arrive_expect_tx(sb + LP_QFULL, (QUANT ? 1 : 2) * 8 * LP_QSLAB);
                __syncwarp();
                if (ok && lane < 8)
                    tma_load_2d_pair(sb + lane * LP_QSLAB, &qmap, lane * 64, x.row0 + (int)rank * 64, qfull);
                __syncwarp();
            };
            if (!QUANT && x.T > 0 && n == 0) load_q(0);
            for (int i = 0; ok && i < x.T; ++i, ++g) {
                const int u0 = (x.t0 + i) * 8, slot = g & 7;
                // the tile's place in the ring: read by the loading warps eight tiles ago, and no further than
                // four tiles ahead of them
                if (g >= 4)
                    ok = ok && __all_sync(0xffffffffu, lat_wait<QUANT>(sb + LP_USED + 8 * ((g - 4) & 7), ((g - 4) >> 3) & 1, dead));
                uint32_t* vw = reinterpret_cast<uint32_t*>(sm + LP_SM_VALID) + slot * 4;
                uint32_t kind = 0;
                int* look = reinterpret_cast<int*>(sm + LP_SM_LOOK) + slot * 128;
                if (QUANT) {
                    // Where each of the tile's rows is, in 16 bytes from the pool's start (in a ring of four tiles), and its
                    // scales: lane l has rows 4 l .. 4 l + 3.
                    uint32_t* at = reinterpret_cast<uint32_t*>(sm + LP_SM_LOOK) + (g & 3) * 128;
                    const int u = u0 + (lane >> 2), j0 = u < x.nU ? unit_row<WINDOW>(x, u) + 4 * (lane & 3) : x.hi;
                    const int e0 = min(max(x.lo - j0, 0), 4), e1 = min(max(x.hi - j0, 0), 4);
                    const int e2 = min(max(min(x.a1, x.hi) - j0, 0), 4);
                    uint32_t seen = (((1u << e1) - 1u) & ~((1u << e0) - 1u)) | ((1u << e2) - 1u);  // by any query
                    uint32_t id[4], sc[4], v = 0;
                    bool bad = false;
                    if (KEYS == LK_QUANT4) {
                        const int lp = div_by(j0, a.by_rpp), rw = j0 - lp * a.kv.rpp;
                        int pg = -1;
                        if (seen && lp < a.table_pages) pg = __ldg(pt + lp);
                        const bool there = pg >= 0 && pg < a.kv.n_pages;
                        bad = seen && !there;
                        uint4 w = make_uint4(0, 0, 0, 0);
                        id[0] = 0;
                        if (there) {
                            v = seen;
                            id[0] = (uint32_t)pg * (uint32_t)(a.kv.page_stride / 16) + (uint32_t)rw * (Q_CODES / 16);
                            // (into L2, each CTA half of the tile, three tiles before the loading warps come for them)
                            if (lane >> 4 == (int)rank)
                                prefetch_l2(q_codes(a.kv.base, a.kv.page_stride, pg, rw), 4 * Q_CODES);
                            w = __ldg(reinterpret_cast<const uint4*>(
                                q_scales(a.kv.base, a.kv.page_stride, a.kv.rpp, pg, rw)));
                        }
                        sc[0] = w.x, sc[1] = w.y, sc[2] = w.z, sc[3] = w.w;
#pragma unroll
                        for (int e = 1; e < 4; ++e) id[e] = id[0] + e * (Q_CODES / 16);
                    } else {
                        int pg[4], rw[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int lp = div_by(j0 + e, a.by_rpp);
                            rw[e] = j0 + e - lp * a.kv.rpp;
                            pg[e] = (seen >> e) & 1u && lp < a.table_pages ? __ldg(pt + lp) : -1;
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bool there = pg[e] >= 0 && pg[e] < a.kv.n_pages;
                            bad = bad || (!there && ((seen >> e) & 1u));
                            id[e] = sc[e] = 0;
                            if (there) {
                                id[e] = (uint32_t)pg[e] * (uint32_t)(a.kv.page_stride / 16) +
                                        (uint32_t)rw[e] * (Q_CODES / 16);
                                sc[e] = __ldg(reinterpret_cast<const uint32_t*>(
                                    q_scales(a.kv.base, a.kv.page_stride, a.kv.rpp, pg[e], rw[e])));
                                v |= 1u << e;
                            }
                        }
                    }
                    if (bad) raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
                    // for rows that are not there another row of the tile is read, and counts 0
                    const uint32_t have = __ballot_sync(0xffffffffu, v != 0);
                    const uint32_t some = v & 1u ? id[0] : v & 2u ? id[1] : v & 4u ? id[2] : id[3];
                    const uint32_t other = __shfl_sync(0xffffffffu, some, have ? __ffs(have) - 1 : 0);
                    const uint32_t fill = v ? some : have ? other : 0u;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!((v >> e) & 1u)) id[e] = fill;
                    *reinterpret_cast<uint4*>(at + 4 * lane) = make_uint4(id[0], id[1], id[2], id[3]);
                    // Each row's largest scale; where they are within 2^15 of one another (or of rows of next to nothing),
                    // the largest of all serves every row, and the softmax has no scales of single rows to reckon with.
                    uint32_t least = 255u, most = 0u;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t m = __vmaxu2(sc[e] & 0x00FF00FFu, (sc[e] >> 8) & 0x00FF00FFu);
                        const uint32_t top = (v >> e) & 1u ? max(m & 255u, m >> 16) : 0u;
                        most = max(most, top);
                        if (top > 10u) least = min(least, top);
                    }
                    least = __reduce_min_sync(0xffffffffu, least);
                    most = __reduce_max_sync(0xffffffffu, most);
                    const uint32_t ratios = sb + LP_SM_RATIO + (uint32_t)(g & 3) * 1024 + 32 * lane;
                    const uint32_t factors = sb + LP_SM_FACTOR + (uint32_t)(g & 7) * 512 + 16 * lane;
                    if (most - 11u < 236u && most - least <= 15u) {  // (and no NaN)
                        kind = LQ_EVEN | most << LQ_TOP;
                        const uint32_t f = most << 23;
                        st_shared_v4(factors, make_uint4(f, f, f, f));
                        uint32_t r[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint2 w = q_ratios(sc[e], most, (v >> e) & 1u);
                            r[2 * e] = w.x, r[2 * e + 1] = w.y;
                        }
                        st_shared_v4(ratios, make_uint4(r[0], r[1], r[2], r[3]));
                        st_shared_v4(ratios + 16, make_uint4(r[4], r[5], r[6], r[7]));
                    } else {
                        kind = quant_uneven(ratios, factors, make_uint4(sc[0], sc[1], sc[2], sc[3]), v);
                    }
                    v <<= 4 * (lane & 7);
                    v |= __shfl_xor_sync(0xffffffffu, v, 1);
                    v |= __shfl_xor_sync(0xffffffffu, v, 2);
                    v |= __shfl_xor_sync(0xffffffffu, v, 4);
                    if ((lane & 7) == 0) vw[lane >> 3] = v;
                } else if (KEYS == LK_BOX) {
                    int pg = -1, rw = 0;
                    const int j = u0 + lane < x.nU && lane < 8 ? unit_row<WINDOW>(x, u0 + lane) : x.hi;
                    if (j < x.hi) {  // (a unit behind the last row that is seen: none)
                        pg = lat_entry(a, pt, j, rw);
                        if (pg < 0 || pg >= a.kv.n_pages) raise_status(a.status, CSA_ERR_DEVICE_BOUNDS), pg = -1;
                    }
                    const uint32_t b = __ballot_sync(0xffffffffu, pg >= 0);
                    const uint32_t b2 = b >> (2 * lane);
                    if (lane < 4) vw[lane] = (b2 & 1 ? 0xFFFFu : 0u) | (b2 & 2 ? 0xFFFF0000u : 0u);
                    if (pg < 0) pg = rw = 0;
                    // bit u: unit u + 1 lies right behind unit u
                    const int pn = __shfl_down_sync(0xffffffffu, pg, 1), rn = __shfl_down_sync(0xffffffffu, rw, 1);
                    const uint32_t runs = __ballot_sync(0xffffffffu, lane < 7 && pn == pg && rn == rw + 16);
                    if (lane < 8) {
                        look[2 * lane] = pg;
                        look[2 * lane + 1] = rw;
                    }
                    if (lane == 0) look[16] = (int)runs;
                } else {
                    int id[4], pg[4], rw[4];
                    uint32_t v = 0, seen = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {  // pages without a row that a query sees are not looked up
                        const int k = lane * 4 + e, u = u0 + (k >> 4);
                        const int j = u < x.nU ? unit_row<WINDOW>(x, u) + (k & 15) : x.hi;
                        const int lp = div_by(j, a.by_rpp), p0 = lp * a.kv.rpp;
                        rw[e] = j - p0;
                        if (j < x.hi && ((WINDOW && p0 < x.a1) || p0 > x.lo - a.kv.rpp)) seen |= 1u << e;
                        pg[e] = (seen >> e) & 1u && lp < a.table_pages ? __ldg(pt + lp) : -1;
                    }
                    bool bad = false;
                    int some = -1;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {  // (after all four loads)
                        const bool there = pg[e] >= 0 && pg[e] < a.kv.n_pages;
                        bad = bad || (!there && ((seen >> e) & 1u));
                        id[e] = there ? pg[e] * (int)(a.kv.page_stride / ROW_BYTES) + rw[e] : 0;
                        if (there) v |= 1u << (4 * (lane & 7) + e), some = id[e];
                    }
                    // for rows that are not looked up another row of the tile stands in: with one and the same for all
                    // items, read by every SM from a few L2 slices, ragged chunks took 90 us and not 78
                    const uint32_t have = __ballot_sync(0xffffffffu, some >= 0);
                    const int other = __shfl_sync(0xffffffffu, some, have ? __ffs(have) - 1 : 0);
                    const int fill = some >= 0 ? some : max(other, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!((v >> (4 * (lane & 7) + e)) & 1u)) id[e] = fill;
                    if (bad) raise_status(a.status, CSA_ERR_DEVICE_BOUNDS);
                    *reinterpret_cast<int4*>(look + 4 * lane) = make_int4(id[0], id[1], id[2], id[3]);
                    // bit q: quad q's rows follow each other; the next quad's follow them
                    const int behind = __shfl_down_sync(0xffffffffu, id[0], 1);
                    const bool all4 = ((v >> (4 * (lane & 7))) & 15u) == 15u;
                    const uint32_t in = __ballot_sync(0xffffffffu, all4 && id[1] == id[0] + 1 && id[2] == id[0] + 2 &&
                                                                       id[3] == id[0] + 3);
                    const uint32_t to = __ballot_sync(0xffffffffu, lane < 31 && behind == id[0] + 4);
                    const uint32_t half = in & (in >> 1) & to, unit = half & (to >> 1) & (half >> 2);
                    if (lane == 0)
                        *reinterpret_cast<uint4*>(sm + LP_SM_NEXT + slot * 16) =
                            make_uint4(half, unit, unit & (to >> 3) & (unit >> 4), 0);
                    v |= __shfl_xor_sync(0xffffffffu, v, 1);
                    v |= __shfl_xor_sync(0xffffffffu, v, 2);
                    v |= __shfl_xor_sync(0xffffffffu, v, 4);
                    if ((lane & 7) == 0) vw[lane >> 3] = v;
                }
                __syncwarp();
                if (lane == 0) {
                    plain[slot] = tile_plain<WINDOW>(x, i, *reinterpret_cast<const uint4*>(vw)) ? 1u | kind : kind;
                    mbar_arrive(sb + LP_LOOK + 8 * slot);
                }
                if (i == 0 && (QUANT || n > 0)) load_q(n);  // behind the first tile's lookups, as it may have to wait
                if (i == 0) ++n;
            }
        }
        if (!ok && lane == 0) *closed = q;
    } else if (QUANT && warp >= LP_SOFT + 2 && warp < LP_SOFT + 2 + lat_loaders(KEYS)) {
        // ---------------------------------------------------------------- quantised key rows
        // All eight warps bring the K rows of a tile, then the V rows of the one before, a step each: 16 rows and 256 dims
        // (a quarter of two slots of K, or half of a slot of V).  (With warps for K and warps for V: 6.60 against 6.54 ms for a
        // chunk of 1K over 24K.)  The code is the same for both and as
        // short as it can be: what the warps of an SM run does not fit the instruction caches, and a warp whose next
        // instructions are not there waits for them (a tile took 15,000 cycles when K and V had loops of their own
        // and every wait was in line).  As each of a step's eight pieces is
        // stored, a piece of the next step is fetched in its place.
        const int w = warp - (LP_SOFT + 2);
        // A lane's pieces: 16 dims of rows 2 e + r0.  The eight lanes of a pass of a store have four pieces of two
        // rows each, which the swizzle lays to eight different banks.
        const int r0 = (lane >> 2) & 1, p0 = (lane & 3) + 4 * (lane >> 3);
        const uint32_t in_slot = (uint32_t)(r0 * 128 + (((lane & 3) * 2 ^ r0) << 4));
        const uint32_t k_slot = 2 * (w >> 2), v_slot = 4 + (w >> 1);
        const uint32_t ring = sb + LP_SM_RING + in_slot, slab = (uint32_t)lane >> 3;
        const uint32_t k_to = ring + k_slot * LP_SLOT + slab * 8192 + (uint32_t)(w & 3) * 2048;
        const uint32_t v_to = ring + v_slot * LP_SLOT + slab * 4096 + (uint32_t)(w & 1) * 2048;
        const uint8_t* base = a.kv.base + p0 * 16;
        // K rows have the ring's first four slots, V rows the others: each part of them is one warp's alone, tile
        // after tile, so that a wait for it to be free cannot be two uses behind.
        struct Tile {
            int g, units;
        };
        // The next tile, of this item or of the next one that has any.  A warp that has rows to store must not wait for an
        // item: warp 9 may be waiting for an item's place (wait: false), which the softmax warps hold that wait for
        // those rows.
        bool looked = false;               // a first look at the next tile's lookups found them there
        bool ended = false, soon = false;  // behind the last item; the next item is not there yet
        int i = -1, T = 0, units = 0;      // in the item: the tile, its tiles, its units from the first tile on
        auto advance = [&](Tile& t, bool wait) -> bool {
            if (ended) return false;
            if (!soon) ++i;
            soon = false;
            while (i >= T) {
                if (!wait && !__all_sync(0xffffffffu, mbar_test_wait(sb + LP_ITEM + 8 * (q & 3), (q >> 2) & 1))) {
                    soon = true;
                    return false;
                }
                const bool in = lat_wait_item<QUANT>(sb + LP_ITEM + 8 * (q & 3), (q >> 2) & 1, q, closed);
                const uint32_t at = sb + LP_SM_ITEM + (q & 3) * 128;
                const uint2 tt = ld_shared_v2(at);  // T, t0
                T = (int)tt.x;
                units = (int)ld_shared_u32(at + 8) - (int)tt.y * 8;
                __syncwarp();
                if (lane == 0) mbar_arrive(sb + LP_TAKEN + 8 * (q & 3));
                ++q;
                i = 0;
                ok = ok && in;
                if (!in || T < 0) {
                    ended = true;
                    return false;
                }
            }
            t.units = min(8, units - 8 * i);
            t.g = g++;
            if (!__all_sync(0xffffffffu, looked))
                ok = ok && __all_sync(0xffffffffu, lat_wait<QUANT>(sb + LP_LOOK + 8 * (t.g & 7), (t.g >> 3) & 1, dead));
            return ok;
        };
        uint4 c[8];
        // A step's first row in its tile; where its rows, and what their codes are to be multiplied by, are looked up; its half
        // of the dims.
        auto row_of = [&](const Tile& t, bool k) {
            return r0 + (k ? (int)rank * ((t.units + 1) >> 1) * 16 + 16 * (w & 3) : 16 * w);
        };
        auto half_of = [&](bool k) { return k ? (uint32_t)w >> 2 : rank; };
        auto rows_at = [&](const Tile& t, bool k) {
            return sb + LP_SM_LOOK + (uint32_t)(t.g & 3) * 512 + (uint32_t)row_of(t, k) * 4;
        };
        auto ratios_at = [&](const Tile& t, bool k) {
            return sb + LP_SM_RATIO + (uint32_t)(t.g & 3) * 1024 + (uint32_t)row_of(t, k) * 8 + half_of(k) * 4 +
                   (uint32_t)(p0 >> 3) * 2;
        };
        Tile cur = {0, 0}, next = {0, 0}, v_first = {0, 0}, v_last = {0, 0};  // tiles whose V rows are still to come
        int pending = 0;
        bool is_k = true;
        bool have = false;   // this step's pieces have been fetched
        bool free = true;    // a first look at this step's slots found them free
#pragma unroll 1
        for (;;) {
            // the step behind this one: the K rows of a tile lead its V rows by a tile, where there is one
            if (have) {
                if (!is_k) {
                    v_first = v_last;
                    --pending;
                } else if (pending++) {
                    v_last = cur;
                } else {
                    v_first = cur;
                }
            }
            const bool next_k = pending < 2 && advance(next, !have && pending == 0);
            const bool there = next_k || pending > 0;
            if (!ok || !(have || there)) break;
            if (!next_k) next = v_first;
            const uint32_t slot = is_k ? k_slot : v_slot;
            if (have && cur.g > 0 && !__all_sync(0xffffffffu, free)) {
                ok = __all_sync(0xffffffffu, lat_wait<QUANT>(sb + LP_EMPTY + 8 * slot, (cur.g - 1) & 1, dead));
                if (!ok) break;
            }
            const int mu = (cur.units + 1) >> 1;
            const bool full = have && (is_k ? (w & 3) < min(max(cur.units - (int)rank * mu, 0), mu) : w < cur.units);
            const uint32_t to = is_k ? k_to : v_to;
            // (no branches from here to the last piece: stores that are not wanted are predicated off, and where there is no next
            // step the last rows are fetched once more; what is looked up is so two pieces ahead: later would hold the stores
            // up, earlier takes registers)
            const uint32_t fa = ratios_at(cur, is_k), ia = there ? rows_at(next, next_k) : rows_at(cur, is_k);
            const uint8_t* from = base + half_of(there ? next_k : is_k) * 256;
            uint32_t f[8], id[8];
#pragma unroll
            for (int e = 0; e < 2; ++e) f[e] = ld_shared_u16(fa + 16 * e), id[e] = ld_shared_u32(ia + 8 * e);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (e < 6) f[e + 2] = ld_shared_u16(fa + 16 * (e + 2)), id[e + 2] = ld_shared_u32(ia + 8 * (e + 2));
                uint4 lo, hi;
                q_halves(c[e], f[e], lo, hi);
                const uint32_t ad = (to ^ ((e & 3) << 5)) + e * 256;
                st_shared_v4_if(full, ad, lo);
                st_shared_v4_if(full, ad ^ 16, hi);
                c[e] = ldg_nc_v4(from + ((uint64_t)id[e] << 4));
                if (e == 5) {  // a first look at the barriers that the next step waits for, answered meanwhile
                    free = mbar_test_wait(sb + LP_EMPTY + 8 * (next_k ? k_slot : v_slot), (next.g - 1) & 1);
                    looked = mbar_test_wait(sb + LP_LOOK + 8 * (g & 7), (g >> 3) & 1);
                }
            }
            if (have) {
                if (LAT_RARE(full && (ld_shared_u32(sb + LP_SM_PLAIN + (cur.g & 7) * 4) & LQ_HUGE))) {
                    const uint32_t at = sb + LP_SM_FACTOR + (uint32_t)(cur.g & 7) * 512 +
                                        (uint32_t)(row_of(cur, is_k) - r0 + (lane & 15)) * 4;
                    lat_infinities(to, q_limit(ld_shared_u32(at) >> 23), r0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_rank_n(sb + LP_FULL + 8 * slot, 0, is_k ? 1 : 2);
                    if (!is_k) mbar_arrive(sb + LP_USED + 8 * (cur.g & 7));  // done with the tile's lookups
                }
            }
            have = there;
            cur = next;
            is_k = next_k;
        }
    } else if (QUANT && warp >= LP_SOFT + 2) {
        // ---------------------------------------------------------------- queries, quantised rows
        const int r = tid - 32 * (LP_SOFT + 2 + lat_loaders(KEYS));
        while (next_item()) {
            if (x.T == 0) continue;
            // The first item's queries are the softmax warps'.  A wait tells a phase from the one before it only: the first
            // wait is over once the item before's queries came and were used (which no later item's can be before these
            // are turned into fp16 here), the second once this one's are there.
            if (n > 0) {
                ok = lat_wait<QUANT>(sb + LP_QEMPTY, (n - 1) & 1, dead) && ok;
                ok = lat_wait<QUANT>(sb + LP_QFULL, n & 1, dead) && ok;
                if ((int)rank * 64 + r < x.nrows) lat_q_row(sb, sb + LP_SM_QTOP + (n & 1) * 64 + r, r);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(sb + LP_QTOP + 8 * (n & 1));
                    mbar_arrive_rank_n(sb + LP_QREADY, 0, LP_SOFT / LQ_WARPS);
                }
            }
            ++n;
        }
    } else if (!QUANT && warp >= LP_SOFT + 2) {
        // ---------------------------------------------------------------- key rows
        const uint32_t full0 = mapa(sb + LP_FULL, 0);  // the even CTA's barriers
        int turn = warp - (LP_SOFT + 2);               // slots until this warp's next one
        auto claim = [&](uint32_t pair_bytes) -> bool {  // slot sidx: free, and both CTAs' bytes announced
            const int sl = sidx & (LP_SLOTS - 1);
            if (sidx >= LP_SLOTS &&
                !__all_sync(0xffffffffu, lat_wait<QUANT>(sb + LP_EMPTY + 8 * sl, ((sidx / LP_SLOTS) - 1) & 1, dead)))
                return false;
            if (rank == 0 && lane == 0) {
                if (pair_bytes) mbar_arrive_expect_tx(sb + LP_FULL + 8 * sl, pair_bytes);
                else mbar_arrive(sb + LP_FULL + 8 * sl);
            }
            __syncwarp();
            return true;
        };
        while (next_item()) {
            const int units = x.nU - x.t0 * 8;
            // K rows of tile i, then V rows of tile i - 1
#pragma unroll 1
            for (int i = 0; ok && i <= x.T && x.T > 0; ++i) {
                if (i < x.T) {
                    if (turn < 4) {  // (six warps: one slot of the four at most)
                        const int kk = turn, gt = g + i, nu = min(8, units - 8 * i);
                        const int mu = (nu + 1) >> 1, ku = min(max(nu - (int)rank * mu, 0), mu), first = (int)rank * mu;
                        ok = __all_sync(0xffffffffu, lat_wait<QUANT>(sb + LP_LOOK + 8 * (gt & 7), (gt >> 3) & 1, dead));
                        const uint32_t look = sb + LP_SM_LOOK + (gt & 7) * 512;
                        sidx += kk;
                        const int sl = sidx & (LP_SLOTS - 1);
                        const uint32_t dst = sb + LP_SM_RING + (uint32_t)sl * LP_SLOT, bar = full0 + 8 * sl;
                        if (KEYS == LK_BOX) {
                            // lane: unit e of the CTA's own (at most 4), slab; the first unit of a run takes all of it
                            const int slab = lane & 1, e = (lane >> 1) & 3;
                            const uint2 at = ld_shared_v2(look + 8 * ((first + e) & 7));
                            uint32_t runs = ld_shared_u32(look + 64);
                            runs = (runs >> first) & ((1u << max(ku - 1, 0)) - 1u);  // bit e: unit e + 1 follows e
                            // rows of this lane's copy: 0 where another unit's covers it
                            const int big = runs == 7u ? (e == 0 ? 2 : -1) : ((runs >> (e & 2)) & 1u ? ((e & 1) ? -1 : 1) : 0);
                            ok = ok && claim((uint32_t)nu * 4096u);
                            if (ok && lane < 2 * ku && big >= 0)
                                tma_load_3d_pair(dst + slab * 8192 + e * 2048, &km.m[big], (2 * kk + slab) * 64, (int)at.y,
                                                 (int)at.x, bar);
                        } else {
                            const int slab = lane >> 4, qd = lane & 15;
                            const uint4 id = ld_shared_v4(look + 16 * ((first * 4 + qd) & 31));
                            const uint4 nx = ld_shared_v4(sb + LP_SM_NEXT + (gt & 7) * 16);
                            const int how = quad_map({nx.x, nx.y, nx.z}, first * 4 + qd, first * 4, (qd >> 2 | 1) < ku);
                            ok = ok && claim((uint32_t)nu * 4096u);
                            if (ok && qd < 4 * ku && how > 0)
                                tma_load_2d_pair(dst + slab * 8192 + qd * 512, &km.m[how], (2 * kk + slab) * 64, (int)id.x,
                                                 bar);
                            if (ok && qd < 4 * ku && how == 0)
                                tma_gather4_pair(dst + slab * 8192 + qd * 512, &km.m[0], (2 * kk + slab) * 64,
                                                 make_int4((int)id.x, (int)id.y, (int)id.z, (int)id.w), bar);
                        }
                        __syncwarp();
                        sidx += 4 - kk;
                        turn += LP_PROD - 4;
                    } else {
                        sidx += 4;
                        turn -= 4;
                    }
                }
                if (i > 0) {
                    const int gt = g + i - 1;
                    if (turn < 4) {
                        const int v = turn, nu = min(8, units - 8 * (i - 1));
                        ok = ok && __all_sync(0xffffffffu, lat_wait<QUANT>(sb + LP_LOOK + 8 * (gt & 7), (gt >> 3) & 1, dead));
                        const uint32_t look = sb + LP_SM_LOOK + (gt & 7) * 512;
                        sidx += v;
                        const int vu = min(max(nu - 2 * v, 0), 2), sl = sidx & (LP_SLOTS - 1);
                        const uint32_t dst = sb + LP_SM_RING + (uint32_t)sl * LP_SLOT, bar = full0 + 8 * sl;
                        if (KEYS == LK_BOX) {
                            const int s = lane & 3, e = (lane >> 2) & 1;
                            const uint2 at = ld_shared_v2(look + 8 * (2 * v + e));
                            uint32_t runs = ld_shared_u32(look + 64);
                            const int big = vu == 2 && ((runs >> (2 * v)) & 1u) ? (e ? -1 : 1) : 0;
                            ok = ok && claim((uint32_t)vu * 16384u);
                            if (ok && lane < 4 * vu && big >= 0)
                                tma_load_3d_pair(dst + s * 4096 + e * 2048, &km.m[big], (int)rank * 256 + s * 64, (int)at.y,
                                                 (int)at.x, bar);
                        } else {
                            const int s = lane >> 3, qd = lane & 7;
                            const uint4 id = ld_shared_v4(look + 16 * ((v * 8 + qd) & 31));
                            const uint4 nx = ld_shared_v4(sb + LP_SM_NEXT + (gt & 7) * 16);
                            const int how = quad_map({nx.x, nx.y, nx.z}, v * 8 + qd, v * 8, vu == 2);
                            ok = ok && claim((uint32_t)vu * 16384u);
                            if (ok && qd < 4 * vu && how > 0)
                                tma_load_2d_pair(dst + s * 4096 + qd * 512, &km.m[how], (int)rank * 256 + s * 64, (int)id.x,
                                                 bar);
                            if (ok && qd < 4 * vu && how == 0)
                                tma_gather4_pair(dst + s * 4096 + qd * 512, &km.m[0], (int)rank * 256 + s * 64,
                                                 make_int4((int)id.x, (int)id.y, (int)id.z, (int)id.w), bar);
                        }
                        __syncwarp();
                        sidx += 4 - v;
                        turn += LP_PROD - 4;
                    } else {
                        sidx += 4;
                        turn -= 4;
                    }
                    if (lane == 0) mbar_arrive(sb + LP_USED + 8 * (gt & 7));  // done with the tile's lookups
                }
            }
            g += x.T;
        }
    }
    ok = __all_sync(0xffffffffu, ok);  // (the products' thread is any lane)
    pdl_launch_dependents();
    if (!ok) {  // a wait ran out: leave the copies and products in flight some time to end
        if (lane == 0) raise_status(a.status, CSA_ERR_TIMEOUT);
#pragma unroll 1
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 0) tmem_dealloc_pair(tmem, 512);
}

template <LatKeys KEYS, bool WINDOW>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(lat_threads(KEYS), 1)
    lat_pair_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ KeyMaps km,
                    const __grid_constant__ LatArgs a) {
    lat_pair<KEYS, WINDOW>(qmap, km, a);
}

// Log-sum-exp merge of a row's partial results, in their order: one CTA per row, thread t columns
// 4t .. 4t+3, IN partial rows in flight: 8, or 16 where there may be more (32 requests of 16 heads, 30 partial results
// of a row: 70.1 -> 66.0 us in all; 16 for everyone costs 4,096 rows of 8 partial results 3 percent, as fewer CTAs
// fit an SM).  Window: rows that no sequence covers are left alone.
template <int IN>
__global__ void __launch_bounds__(128, IN > 8 ? 4 : 8) lat_merge_kernel(LatArgs a) {
    pdl_wait();
    const int row = blockIdx.x, t = threadIdx.x;
    if (!a.n_rows) {
        const int64_t q = row / a.H;
        const int l = seq_of(a, q);
        const int64_t q0 = __ldg(a.q_offsets + l), q1 = __ldg(a.q_offsets + l + 1);
        if (q < q0 || q >= q1 || !seq_valid(a, q0, q1, __ldg(a.n_tokens + l))) return;
    }
    // the row's partial results: all, or those of the runs that its row tile and its request lie in
    int n = a.parts, n_first = a.parts, skip = 0;
    if (a.run) {
        const int p = (row >> 7) * a.gS, o = div_by(row, a.by_H) * a.gO;
        n_first = a.tS ? div_by(p + a.tS - 1, a.by_run) - div_by(p, a.by_run) + 1 : 0;
        n = n_first + (a.tO ? div_by(o + a.tO - 1, a.by_run) - div_by(o, a.by_run) + 1 : 0);
        skip = a.SP - n_first;
    }
    // (the maximum so far is kept as a running one)
    const float* lp = a.part_lse + row;
    const float4* op = reinterpret_cast<const float4*>(a.part_o + (int64_t)row * D) + t;
    const int64_t step = (int64_t)a.rows;
    float M = -INFINITY, L = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
    bool nan = false;
    for (int s0 = 0; s0 < n; s0 += IN) {
        float v[IN];
        float4 f[IN];
#pragma unroll
        for (int s = 0; s < IN; ++s) {
            const int64_t at = (s0 + s < n_first ? s0 + s : s0 + s + skip) * step;
            v[s] = s0 + s < n ? __ldcg(lp + at) : -INFINITY;
            if (s0 + s < n) f[s] = __ldcg(op + at * (D / 4));
        }
        float m = M;
#pragma unroll
        for (int s = 0; s < IN; ++s) {
            m = fmaxf(m, v[s]);
            nan = nan || v[s] != v[s];
        }
        if (m > M) {
            const float w = M == -INFINITY ? 0.f : lat_ex2((M - m) * LP_LOG2E);
            L *= w, o0 *= w, o1 *= w, o2 *= w, o3 *= w;
            M = m;
        }
#pragma unroll
        for (int s = 0; s < IN; ++s) {
            if (v[s] == -INFINITY) continue;  // (no keys: its row may hold anything)
            const float w = lat_ex2((v[s] - M) * LP_LOG2E);
            L += w;
            o0 = fmaf(w, f[s].x, o0);
            o1 = fmaf(w, f[s].y, o1);
            o2 = fmaf(w, f[s].z, o2);
            o3 = fmaf(w, f[s].w, o3);
        }
    }
    const bool lost = M == LP_LSE_LOST;  // rows, and every logit -inf
    const float inv = lost ? __int_as_float(0x7FFFFFFF) : L == 0.f ? 0.f : 1.f / L;
    uint2 w;
    w.x = pack_bf16x2(o0 * inv, o1 * inv);
    w.y = pack_bf16x2(o2 * inv, o3 * inv);
    *reinterpret_cast<uint2*>(a.out + (int64_t)row * D + t * 4) = w;
    if (t == 0 && a.lse) a.lse[row] = nan ? __int_as_float(0x7FFFFFFF) : (L == 0.f || lost ? -INFINITY : M + log2f(L) * LP_LN2);
}

// The rows of row tiles that are cut, from their runs' partial results in the order of the runs: a warp a row, lane l
// columns 4 l + 128 k.
constexpr int QM_IN = 4;                         // partial rows in flight
constexpr int QM_CTAS = 2 * 2 * LP_PAIRS;
constexpr float QM_MOST = 128.f;                 // more than a row has partial results; a power of two: the same bits
static_assert(QR < QM_MOST, "partial results of a row");
__global__ void __launch_bounds__(256, 2) quant_merge_kernel(LatArgs a) {
    // (each CTA reads the runs once: warps that all read them for themselves took 24 us and more at the few L2 lines that
    // they are in)
    __shared__ int listed[3 * (QR + 1)];
    pdl_wait();
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 3 * (QR + 1)) listed[threadIdx.x] = __ldcg(reinterpret_cast<const int*>(a.runs) + threadIdx.x);
    __syncthreads();
    const int runs = (uint32_t)listed[3 * QR] <= QR ? listed[3 * QR] : 0;
    // runs 3 lane .. 3 lane + 2: the rows of the row tile that begins in each, added up
    static_assert(QR <= 96, "a warp holds all runs");
    QuantRun run[3];
    int rows[3], before = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int r = 3 * lane + k;
        run[k] = {0, 0, 0};
        if (r < runs) run[k] = {listed[3 * r], listed[3 * r + 1], listed[3 * r + 2]};
        const bool fine = run[k].last > r && run[k].last < runs && run[k].nrows > 0 && run[k].nrows <= a.slot_rows &&
                          run[k].row0 >= 0 && run[k].row0 <= a.rows - run[k].nrows;
        rows[k] = fine ? run[k].nrows : 0;
        before += rows[k];
    }
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    const int total = __shfl_sync(0xffffffffu, before, 31);
    before -= rows[0] + rows[1] + rows[2];
    for (int at = blockIdx.x * 8 + (threadIdx.x >> 5); at < total; at += 8 * gridDim.x) {
        // the last lane whose rows begin at or before this one
        const int src = 31 - __clz((int)__ballot_sync(0xffffffffu, before <= at && rows[0] + rows[1] + rows[2] > 0));
        int i = at - before, k = 0;
        if (i >= rows[0]) i -= rows[0], k = 1;
        if (k == 1 && i >= rows[1]) i -= rows[1], k = 2;
        i = __shfl_sync(0xffffffffu, i, src);
        const int r0 = 3 * src + __shfl_sync(0xffffffffu, k, src);
        const int row = __shfl_sync(0xffffffffu, k == 0 ? run[0].row0 : k == 1 ? run[1].row0 : run[2].row0, src) + i;
        const int last = __shfl_sync(0xffffffffu, k == 0 ? run[0].last : k == 1 ? run[1].last : run[2].last, src);
        float M = -INFINITY, L = 0.f, o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = 0.f;
        bool nan = false;
        for (int s0 = r0; s0 <= last; s0 += QM_IN) {
            float v[QM_IN];
            float4 f[QM_IN][4];
#pragma unroll
            for (int s = 0; s < QM_IN; ++s) {
                const int r = s0 + s;
                const int64_t prow = (int64_t)(2 * r + (r == r0 ? 1 : 0)) * a.slot_rows + i;
                v[s] = r <= last ? __ldcg(a.part_lse + prow) : -INFINITY;
                if (r <= last) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        f[s][c] = __ldcg(reinterpret_cast<const float4*>(a.part_o + prow * D) + lane + 32 * c);
                }
            }
            float m = M;
#pragma unroll
            for (int s = 0; s < QM_IN; ++s) {
                m = fmaxf(m, v[s]);
                nan = nan || v[s] != v[s];
            }
            if (m > M) {
                const float w = M == -INFINITY ? 0.f : lat_ex2((M - m) * LP_LOG2E);
                L *= w;
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] *= w;
                M = m;
            }
#pragma unroll
            for (int s = 0; s < QM_IN; ++s) {
                if (v[s] == -INFINITY) continue;  // (no keys that its rows see)
                const float w = lat_ex2((v[s] - M) * LP_LOG2E) * (1.f / QM_MOST);  // (sums of large values stay finite)
                L += w;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    o[4 * c] = fmaf(w, f[s][c].x, o[4 * c]);
                    o[4 * c + 1] = fmaf(w, f[s][c].y, o[4 * c + 1]);
                    o[4 * c + 2] = fmaf(w, f[s][c].z, o[4 * c + 2]);
                    o[4 * c + 3] = fmaf(w, f[s][c].w, o[4 * c + 3]);
                }
            }
        }
        const bool lost = M == LP_LSE_LOST;  // rows, and every logit -inf
        const float inv = lost ? __int_as_float(0x7FFFFFFF) : L == 0.f ? 0.f : 1.f / L;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            reinterpret_cast<uint2*>(a.out + (int64_t)row * D)[lane + 32 * c] =
                make_uint2(pack_bf16x2(o[4 * c] * inv, o[4 * c + 1] * inv),
                           pack_bf16x2(o[4 * c + 2] * inv, o[4 * c + 3] * inv));
        if (lane == 0 && a.lse)
            a.lse[row] = nan ? __int_as_float(0x7FFFFFFF) : (L == 0.f || lost ? -INFINITY : M + log2f(L * QM_MOST) * LP_LN2);
    }
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
    if (H < 1 || H > 128 || B < 1 || B > 65535 || max_rows > LP_MAX_ROWS) return CSA_ERR_UNSUPPORTED;
    if (n_shared < 0 || max_rows < n_shared) return CSA_ERR_INVALID_ARG;
    return CSA_OK;
}

static csa_status check_window(int32_t B, int32_t H, int64_t total_q, int64_t max_q, int32_t window, int32_t n_sink) {
    if (H < 1 || H > 128 || B < 1 || B > 65535 || window > (1 << 30) || n_sink > (1 << 30)) return CSA_ERR_UNSUPPORTED;
    if (window < 1 || n_sink < 0 || total_q < 0 || max_q < 1) return CSA_ERR_INVALID_ARG;
    if (total_q > 0x7FFFFFFFLL / H) return CSA_ERR_UNSUPPORTED;
    return CSA_OK;
}

static void set_scale(LatArgs& a, float scale, bool quant = false) {
    a.sl2 = (scale < 0.f ? -scale : scale) * LP_LOG2E;
    // every weight 1 (whatever the logits: at most 3.4e38 times the least number above 0), and a masked logit still -inf
    if (a.sl2 == 0.f) a.sl2 = std::numeric_limits<float>::denorm_min();
    if (quant && std::isfinite(a.sl2)) {
        a.sl2 = 2.f * std::frexp(a.sl2, &a.sl2_power);
        --a.sl2_power;
    }
    a.negate = scale < 0.f ? 1u << 13 : 0u;
}

// How long the slowest of LP_PAIRS pairs takes, in tiles of 128 keys, for n1 items of t1 tiles and n2 of t2 behind
// them, dealt out in turn; an item costs about three tiles more (its Q, its first and last product, its output).
static int64_t deal_cost(int64_t n1, int64_t t1, int64_t n2, int64_t t2) {
    const int64_t P = LP_PAIRS, c1 = t1 + 3, c2 = t2 + 3;
    int64_t worst = 0;
    // pairs differ by whether they get one more of the first kind, and one more in all
    const int64_t edges[3] = {0, n1 % P, (n1 + n2) % P};
    for (int64_t p : edges) {
        const int64_t a = n1 / P + (p < n1 % P), all = (n1 + n2) / P + (p < (n1 + n2) % P);
        worst = std::max(worst, a * c1 + (all - a) * c2);
    }
    return worst;
}

// How the tiles are dealt to the pairs: the splits of the shared rows (SP) and of a request's own (OS) that end
// soonest, or runs (then SP and OS are the most partial results that a row has of each); a partial result of every row,
// written and read again, is taken to cost 1.4 tiles for each 4,096 rows (16 MB through L2 beside the products) and 0.02
// for its place in the merge: estimates, which the shapes below bear out.
static void plan_prefix(int B, int H, int64_t n_shared, int64_t max_rows, LatArgs* a) {
    a->rows = B * H;
    a->RT = (a->rows + 127) / 128;
    const int tiles = (int)((n_shared + 127) / 128);
    const int own = max_rows > n_shared ? (int)((max_rows + 15) / 16 - n_shared / 16 + 7) / 8 : 0;
    a->SP = 0;
    a->OS = 0;
    double best = 1e30;
    const int os_least = (own + LP_MAX_TILES - 1) / LP_MAX_TILES, sp_least = (tiles + LP_MAX_TILES - 1) / LP_MAX_TILES;
    const int os_most = own ? std::min(own, std::max(1, 4 * LP_PAIRS / B)) : 0;
    const int sp_most = std::max(sp_least, std::min(tiles, LP_PAIRS));
    for (int sp = sp_least; sp <= sp_most; ++sp) {
        // a request's own rows: whole, or in pieces as long as the shared ones
        const int piece = sp ? std::max(4, (tiles + sp - 1) / sp)
                             : (int)std::max<int64_t>(2, ((int64_t)own * B + LP_PAIRS - 1) / LP_PAIRS);
        const int os = std::max(os_least, own ? std::min((own + piece - 1) / piece, os_most) : 0);
        const double c = (double)deal_cost((int64_t)a->RT * sp, sp ? (tiles + sp - 1) / sp : 0, (int64_t)B * os,
                                           os ? (own + os - 1) / os : 0) +
                         (sp + os > 1 ? 1.4 * (sp + os) * a->rows / 4096.0 + 0.02 * (sp + os) : 0.0);
        if (c < best) best = c, a->SP = sp, a->OS = os;
    }
    // Or in runs, one for each pair: all of one length and with fewer partial results a row, at the price of items that
    // end in a run's midst and of row tiles that read the same keys at different times.  Behind each row tile's or
    // request's tiles are places that stand for an item's cost beside its tiles (three and two: 158 and 60.6 us for
    // the two cases below; three and three 158 and 62.4, two and two 159 and 61.3, one and one 171 and 62.3).
    // 32 requests of 128 heads over 32K rows + 300: 174.7 us in splits, 160.7 in runs; of 16 heads over 64K + 2K: 65.4
    // and 61.3; where the splits come out even (8 x 128 over 8K + 512, one item a pair) they are the faster, 23.3 to 24.4.
    // Over 18 shapes (1 to 100 requests, 3 to 128 heads, 1 to 131K shared rows) runs alone were up to 7 percent slower
    // and splits alone up to 12; this choice was never more than 2 percent behind the better of the two.
    const int64_t gS = tiles ? tiles + 3 : 0, gO = own ? own + 2 : 0, inS = a->RT * gS, inO = B * gO;
    if (inS + inO >= 4 * LP_PAIRS && std::max(inS, inO) < 1 << 30) {
        int64_t C = (inS + inO + LP_PAIRS - 1) / LP_PAIRS;
        while ((inS + C - 1) / C + (inO + C - 1) / C > LP_PAIRS) C += 1 + C / 256;
        const int PS = tiles ? (int)((tiles + C - 2) / C) + 1 : 0, PO = own ? (int)((own + C - 2) / C) + 1 : 0;
        const double c = C + 3 + 1.4 * ((tiles + own) / (double)C + (tiles > 0) + (own > 0)) * a->rows / 4096.0 +
                         0.02 * (PS + PO);
        if (C <= LP_MAX_TILES && c < best) {
            a->SP = PS;
            a->OS = PO;
            a->run = (int)C;
            a->NS = (int)((inS + C - 1) / C);
            a->tS = tiles;
            a->gS = (int)gS;
            a->tO = own;
            a->gO = (int)gO;
        }
    }
    if (a->SP + a->OS == 0) a->OS = 1;  // no rows at all: every request is empty
    a->parts = a->SP + a->OS;
}

// positions: those that a row of the page table has pages for.  A window beyond them counts as one of them, down to
// 2^18 (half of what a split takes at most): wide ones are split because of LP_MAX_TILES, with a partial result of
// every row for each split, and one that is only meant to reach over everything needs none.
constexpr int64_t kLeastReach = 1 << 18;
static_assert(kLeastReach + 256 <= (int64_t)LP_MAX_TILES * 128, "a window of kLeastReach is one split");
static void plan_window(int B, int H, int64_t total_q, int64_t max_q, int window, int n_sink, int64_t positions,
                        LatArgs* a, int64_t* items) {
    a->rows = (int)(total_q * H);
    const int64_t per_seq = (std::min<int64_t>(max_q, 0x7FFFFFFF) * H + 127) / 128;
    const int64_t tiles_q = std::min((int64_t)B * per_seq, (total_q * H + 127) / 128 + B);
    // key tiles of a row tile: its tokens' windows and the sinks
    const int64_t reach = std::min((int64_t)window + n_sink, std::max(positions, kLeastReach));
    const int64_t keys = reach + 127 / H + 32;
    const int64_t tiles = (keys + 127) / 128;
    int64_t s = 1;
    if (tiles >= 4 && tiles_q <= LP_PAIRS / 2) s = std::min(tiles / 2, LP_PAIRS / std::max<int64_t>(tiles_q, 1));
    a->WS = (int)std::max(s, (tiles + LP_MAX_TILES - 1) / LP_MAX_TILES);
    a->parts = a->WS;
    if (items) *items = tiles_q * a->WS;
}

static size_t parts_bytes(const LatArgs& a) {
    if (a.parts <= 1) return 0;
    // (the partial rows start at a 256-byte boundary inside a workspace that is 16-byte aligned)
    return 256 + align_up((size_t)a.parts * a.rows * D * sizeof(float), 256) +
           align_up((size_t)a.parts * a.rows * sizeof(float), 256);
}

// Quantised rows: runs where there are few row tiles (QUANT_FEW at most, and QUANT_SEQS sequences, whose lengths every
// CTA adds up before it begins); else whole row tiles are dealt out in turn.  Both sides, whole row tiles and runs: chunks of
// 100, 152, 200, 304, 320, 400, 700 and 1,024 tokens of 128 heads (as many row tiles) over 8K rows 325 and 238 us, 330 and
// 333, 487 and 452, 654 and 663, 810 and 714, 974 and 894, 1,644 and 1,588, 2,338 and 2,377; 400 and 1,024 over 1K 180 and
// 194, 483 and 590; 400 and 1,000 under a window of 128 63 and 68, 130 and 138.  (So row tiles that come out unevenly gain
// up to a thousand of them, short ones lose.)  Single tokens of 16 heads, ragged: 128 over 8K rows 324 and 184 us, 256
// 532 and 340; beyond QUANT_SEQS runs would be the faster too, 300 over 8K 566 and 394, 1,000 over 2K 455 and 407, and 300
// of which one has 128K rows 2,579 and 132.
constexpr int QUANT_FEW = 4 * LP_PAIRS, QUANT_SEQS = 256;
constexpr int QUANT_CUT = 2;                     // places of a run at least (6: one token of 16 heads over 4K 29 us
                                                 // instead of 20, without the merge)
static void plan_quant(int B, int H, int64_t total_q, int64_t max_q, int window, int n_sink, LatArgs* a, int64_t* items) {
    a->rows = (int)(total_q * H);
    const int64_t per_seq = (std::min<int64_t>(max_q, 0x7FFFFFFF) * H + 127) / 128;
    const int64_t tiles_q = std::min((int64_t)B * per_seq, (total_q * H + 127) / 128 + B);
    a->cut = total_q > 0 && tiles_q <= QUANT_FEW && B <= QUANT_SEQS ? QUANT_CUT : 0;
    a->slot_rows = std::min(128, std::max(a->rows, 1));
    // (items of more than LP_MAX_TILES tiles need a slot each)
    a->parts = a->cut ? 3 * QR : total_q > 0 && (int64_t)window + n_sink + 256 > (int64_t)LP_MAX_TILES * 128 ? QR : 0;
    if (items) *items = a->cut ? QR : std::min<int64_t>(tiles_q, QR);
}

static size_t quant_bytes(const LatArgs& a) {
    if (a.parts == 0) return 0;
    const size_t rows = (size_t)a.parts * a.slot_rows;
    return 256 + align_up((QR + 1) * sizeof(QuantRun), 256) + align_up(rows * D * sizeof(float), 256) +
           align_up(rows * sizeof(float), 256);
}

// The places of the workspace: the list of runs, then the partial results.
static void quant_places(LatArgs& a, void* ws) {
    uint8_t* base = reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<uintptr_t>(ws), 256));
    a.runs = reinterpret_cast<QuantRun*>(base);
    base += align_up((QR + 1) * sizeof(QuantRun), 256);
    a.part_o = reinterpret_cast<float*>(base);
    a.part_lse = reinterpret_cast<float*>(base + align_up((size_t)a.parts * a.slot_rows * D * sizeof(float), 256));
}

// Pairs in a grid at most, as a device of fewer SMs has them (csa_selftest_pairs); 0: as many as the device has.
static std::atomic<int> g_pairs_most{0};

static cudaError_t launch_pair(LatArgs& a, const void* q, const csa_paged& kv, int64_t items, void* ws, cudaStream_t s,
                               bool quant = false) {
    if (quant) {
        if (a.parts > 0) quant_places(a, ws);
    } else if (a.parts > 1) {
        uint8_t* base = reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<uintptr_t>(ws), 256));
        a.part_o = reinterpret_cast<float*>(base);
        a.part_lse = reinterpret_cast<float*>(base + align_up((size_t)a.parts * a.rows * D * sizeof(float), 256));
    }
    a.wide_out = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
    a.by_H = fast_div(a.H);
    a.by_rpp = fast_div((uint32_t)kv.rows_per_page);
    a.by_RT = fast_div(std::max(a.RT, 1));
    a.by_SP = fast_div(std::max(a.SP, 1));
    a.by_OS = fast_div(std::max(a.OS, 1));
    a.by_WS = fast_div(std::max(a.WS, 1));
    a.by_run = fast_div(std::max(a.run, 1));
    a.by_gS = fast_div(std::max(a.gS, 1));
    a.by_gO = fast_div(std::max(a.gO, 1));
    const int sms = device_sm_count();
    if (sms < 2) return cudaErrorInvalidDevice;
    CUtensorMap qm;
    KeyMaps km = {};
    const uint64_t qd[2] = {(uint64_t)D, (uint64_t)a.rows}, qs[1] = {ROW_BYTES};
    const uint32_t qb[2] = {64, 64};
    if (!make_bf16_map(&qm, q, 2, qd, qs, qb)) return cudaErrorInvalidValue;
    const bool box = kv.rows_per_page % 16 == 0;
    if (quant) {  // read by plain loads
    } else if (box) {  // a box never reaches behind its page: only runs of units are copied in larger ones
        const uint64_t d[3] = {(uint64_t)D, (uint64_t)kv.rows_per_page, (uint64_t)kv.n_pages};
        const uint64_t st[2] = {ROW_BYTES, (uint64_t)kv.page_stride_bytes};
        for (int i = 0; i < 3 && kv.rows_per_page >= 16 << i; ++i) {
            const uint32_t b[3] = {64, 16u << i, 1};
            if (!make_bf16_map(&km.m[i], kv.base, 3, d, st, b)) return cudaErrorInvalidValue;
        }
    } else {  // the extent ends with the last page's own rows
        const uint64_t per_page = (uint64_t)(kv.page_stride_bytes / ROW_BYTES);
        const uint64_t d[2] = {(uint64_t)D, (uint64_t)(kv.n_pages - 1) * per_page + (uint64_t)kv.rows_per_page};
        const uint64_t st[1] = {ROW_BYTES};
        for (int i = 0; i < 4 && (i == 0 || d[1] >= 4u << i); ++i) {  // (a pool of fewer rows has no such run)
            const uint32_t b[2] = {64, i == 0 ? 1u : 4u << i};
            if (!make_bf16_map(&km.m[i], kv.base, 2, d, st, b)) return cudaErrorInvalidValue;
        }
    }
    void (*kernel)(CUtensorMap, KeyMaps, LatArgs) =
        quant      ? (kv.rows_per_page % 4 == 0 ? lat_pair_kernel<LK_QUANT4, true> : lat_pair_kernel<LK_QUANT1, true>)
        : a.n_rows ? (box ? lat_pair_kernel<LK_BOX, false> : lat_pair_kernel<LK_GATHER, false>)
                   : (box ? lat_pair_kernel<LK_BOX, true> : lat_pair_kernel<LK_GATHER, true>);
    cudaError_t e = set_func_attr_once((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)LP_SMEM);
    if (e != cudaSuccess) return e;
    const int cap = g_pairs_most.load(std::memory_order_relaxed);
    const int64_t most = cap > 0 ? std::min(cap, sms / 2) : sms / 2;
    const unsigned pairs = (unsigned)std::max<int64_t>(1, std::min(items, most));
    e = launch_after(kernel, dim3(2 * pairs), quant ? lat_threads(LK_QUANT4) : LP_T, LP_SMEM, s, qm, km, a);
    if (e == cudaSuccess && quant && a.cut)
        return launch_after(quant_merge_kernel, dim3(QM_CTAS), 256, 0, s, a);
    if (e != cudaSuccess || quant || a.parts == 1) return e;
    return launch_after(a.parts <= 8 ? lat_merge_kernel<8> : lat_merge_kernel<16>, dim3((unsigned)a.rows), 128, 0, s,
                        a);
}

// csa_window_attn and, over quantised rows, csa_quant_attn.
static csa_status window_attn(bool quant, const void* q, int32_t H, float scale, const csa_paged& kv_raw,
                              int64_t page_table_stride, int32_t B, const int64_t* q_offsets, const int64_t* n_tokens,
                              int64_t total_q, int64_t max_q, int32_t window, int32_t n_sink, void* out, float* lse,
                              void* workspace, size_t ws_bytes, void* stream) {
    csa_status rc = check_window(B, H, total_q, max_q, window, n_sink);
    if (rc) return rc;
    if ((total_q > 0 && (!q || !out)) || !al16(q) || !al16(out) || (lse && !al4(lse)) || !q_offsets || !al8(q_offsets) ||
        !n_tokens || !al8(n_tokens))
        return CSA_ERR_INVALID_ARG;
    if ((rc = quant ? check_quant_cache(kv_raw, page_table_stride) : check_cache(kv_raw, page_table_stride))) return rc;
    LatArgs a = {};
    int64_t items;
    const int64_t positions = std::min(page_table_stride, LP_MAX_ROWS) * kv_raw.rows_per_page;
    if (quant) plan_quant(B, H, total_q, max_q, window, n_sink, &a, &items);
    else plan_window(B, H, total_q, max_q, window, n_sink, positions, &a, &items);
    const size_t need = quant ? quant_bytes(a) : parts_bytes(a);
    if (need && (!workspace || !al16(workspace) || ws_bytes < need)) return CSA_ERR_WORKSPACE;
    if (total_q == 0) return CSA_OK;
    if (items > 0x7FFFFFFF) return CSA_ERR_UNSUPPORTED;
    a.status = device_status_ptr();
    if (!a.status) return CSA_ERR_CUDA;
    a.H = H;
    set_scale(a, scale, quant);
    a.kv = cache_of(kv_raw, page_table_stride);
    a.table_pages = page_table_stride;
    a.B = B;
    a.q_offsets = q_offsets;
    a.n_tokens = n_tokens;
    a.total_q = total_q;
    a.items = (int)items;
    a.max_q = max_q;
    a.window = window;
    a.n_sink = n_sink;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    return from_cuda(launch_pair(a, q, kv_raw, items, workspace, static_cast<cudaStream_t>(stream), quant));
}


}  // namespace csa

using namespace csa;

extern "C" {

csa_status csa_selftest_pairs(int32_t pairs) {
    if (pairs < 0) return CSA_ERR_INVALID_ARG;
    g_pairs_most.store(pairs, std::memory_order_relaxed);
    return CSA_OK;
}

csa_status csa_selftest_quant_merge(const void* workspace, size_t ws_bytes, int32_t rows, void* out, float* lse,
                                    void* stream) {
    LatArgs a = {};
    if (rows < 1 || !workspace || !al16(workspace) || !out || !al16(out) || (lse && !al4(lse))) return CSA_ERR_INVALID_ARG;
    a.rows = rows;
    a.slot_rows = std::min(128, rows);
    a.parts = 3 * QR;
    if (ws_bytes < quant_bytes(a)) return CSA_ERR_WORKSPACE;
    quant_places(a, const_cast<void*>(workspace));
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    return from_cuda(launch_after(quant_merge_kernel, dim3(QM_CTAS), 256, 0, static_cast<cudaStream_t>(stream), a));
}

size_t csa_prefix_attn_workspace_size(int32_t B, int32_t H, int64_t n_shared, int64_t max_rows) {
    if (check_prefix(B, H, n_shared, max_rows)) return 0;
    LatArgs a = {};
    plan_prefix(B, H, n_shared, max_rows, &a);
    return parts_bytes(a);
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
    LatArgs a = {};
    plan_prefix(B, H, n_shared, max_rows, &a);
    const size_t need = parts_bytes(a);
    if (need && (!workspace || !al16(workspace) || ws_bytes < need)) return CSA_ERR_WORKSPACE;
    int64_t items = (int64_t)a.RT * a.SP + (int64_t)B * a.OS;
    if (a.run) items = a.NS + ((int64_t)B * a.gO + a.run - 1) / a.run;
    if (items > 0x7FFFFFFF) return CSA_ERR_UNSUPPORTED;
    a.status = device_status_ptr();
    if (!a.status) return CSA_ERR_CUDA;
    a.H = H;
    set_scale(a, scale);
    a.kv = cache_of(kv, page_table_stride);
    a.table_pages = page_table_stride;
    a.B = B;
    a.n_rows = n_rows;
    a.items = (int)items;
    a.n_shared = (int)n_shared;
    a.max_rows = (int)max_rows;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    return from_cuda(launch_pair(a, q, kv, items, workspace, static_cast<cudaStream_t>(stream)));
}

size_t csa_window_attn_workspace_size(int32_t B, int32_t H, int64_t total_q, int64_t max_q, int32_t window,
                                      int32_t n_sink) {
    if (check_window(B, H, total_q, max_q, window, n_sink)) return 0;
    LatArgs a = {};
    plan_window(B, H, total_q, max_q, window, n_sink, INT64_MAX, &a, nullptr);
    return parts_bytes(a);
}

csa_status csa_window_attn(const void* q, int32_t H, float scale, csa_paged kv_raw, int64_t page_table_stride,
                           int32_t B, const int64_t* q_offsets, const int64_t* n_tokens, int64_t total_q,
                           int64_t max_q, int32_t window, int32_t n_sink, void* out, float* lse, void* workspace,
                           size_t ws_bytes, void* stream) {
    return window_attn(false, q, H, scale, kv_raw, page_table_stride, B, q_offsets, n_tokens, total_q, max_q, window,
                       n_sink, out, lse, workspace, ws_bytes, stream);
}

size_t csa_quant_attn_workspace_size(int32_t B, int32_t H, int64_t total_q, int64_t max_q, int32_t window,
                                     int32_t n_sink) {
    if (check_window(B, H, total_q, max_q, window, n_sink)) return 0;
    LatArgs a = {};
    plan_quant(B, H, total_q, max_q, window, n_sink, &a, nullptr);
    return quant_bytes(a);
}

csa_status csa_quant_attn(const void* q, int32_t H, float scale, csa_paged cache, int64_t page_table_stride,
                          int32_t B, const int64_t* q_offsets, const int64_t* n_tokens, int64_t total_q,
                          int64_t max_q, int32_t window, int32_t n_sink, void* out, float* lse, void* workspace,
                          size_t ws_bytes, void* stream) {
    return window_attn(true, q, H, scale, cache, page_table_stride, B, q_offsets, n_tokens, total_q, max_q, window,
                       n_sink, out, lse, workspace, ws_bytes, stream);
}

}  // extern "C"
