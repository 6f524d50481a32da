// The page table of a batch: pages handed out (extend) and taken back
// (rollback, truncate) on the GPU from device counts, with the slot and the
// position of every new token.
//
// Both are one exclusive scan over the requests (pages per request) followed by
// work on the scan's items (tokens, or pages going back). The order of the pages
// is that of the requests whatever the launch.
//
// A decode step (the same few tokens for every request; step_takes) is a single block, a
// thread a request: bound by latency, of which a scan is one barrier. Prompts and
// ended requests take a block per 1024 items, up to two per SM: every block makes
// the whole scan for itself, which costs it one pass over 8 bytes a request from L2,
// and then takes an equal share of the items. So one launch does it without any
// block waiting for another; the last block to have read the lengths (a ticket)
// writes the new ones and the free count. There the slot and position stores
// (8 bytes a token) are the floor.
#include <cstring>
#include <new>

#include "overlap.cuh"

namespace rssm {
namespace {

constexpr int kPagesThreads = 1024;     // most of the kernels that share items out; 512 where a round holds the batch
constexpr int kItemsPerBlock = 1024;
// Unused shared memory of the kernels that share items out, so that no SM takes more
// than two of their blocks: beside the end of the kernel before, early blocks would
// crowd onto the SMs that are free (256 prompts after as many leave: 39 us; plain
// launches 26; this 21.5).
constexpr int kSpread = 88 * 1024;
constexpr int kRun = 8;                 // tokens that a thread takes in a row
constexpr int kStepThreads = 1024;      // most of the single-block kernels
constexpr int kStepTokens = 16;         // most tokens a request that those take

struct PagesArgs {
    int32_t* lens;
    int32_t* table;
    int32_t* free_list;
    int32_t* free_count;
    int32_t* err;
    int32_t* refused;     // [batch]: the request's last extend was refused
    uint32_t* ticket;
    int32_t batch, page_size, num_pages, max_pages;
    int32_t shift;        // log2(page_size), or -1: a division costs 20 instructions
    // extend
    const int32_t* d_new;
    int32_t T;
    int32_t* slots;
    int32_t* positions;
    int32_t max_tokens;
    int32_t wide;         // slots and positions are 16-byte aligned
    // rollback (T > 0) or truncate (T = 0)
    const int32_t* keep;
};

// Inclusive scans of one int32 and one int64 a thread over the block, added to
// the totals so far, which the block's totals then join. One barrier: consecutive
// scans use the two halves of the buffers in turn.
struct ScanBuf {
    int32_t x[2][32];
    int64_t y[2][32];
};
struct Scan {
    int32_t cx = 0;
    int64_t cy = 0;
    int turn = 0;
    __device__ __forceinline__ void reset() { cx = 0, cy = 0; }
    template <bool kBoth>
    __device__ __forceinline__ void run(ScanBuf& s, int32_t& x, int64_t& y) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t n = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += n;
            if (kBoth) {
                const int64_t m = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) y += m;
            }
        }
        if (lane == 31) {
            s.x[turn][warp] = x;
            if (kBoth) s.y[turn][warp] = y;
        }
        __syncthreads();
        int32_t w = lane < warps ? s.x[turn][lane] : 0;
        int64_t v = kBoth && lane < warps ? s.y[turn][lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t n = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += n;
            if (kBoth) {
                const int64_t m = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += m;
            }
        }
        const int32_t bx = __shfl_sync(0xffffffffu, w, max(warp - 1, 0)), tx = __shfl_sync(0xffffffffu, w, 31);
        x += cx + (warp ? bx : 0);
        cx += tx;
        if (kBoth) {
            const int64_t by = __shfl_sync(0xffffffffu, v, max(warp - 1, 0)), ty = __shfl_sync(0xffffffffu, v, 31);
            y += cy + (warp ? by : 0);
            cy += ty;
        }
        turn ^= 1;
    }
};

// What one request asks for.
struct Ask {
    int32_t len, count;   // length; new tokens (extend) or pages that go back
    int32_t need;         // pages wanted (extend)
    int32_t bad;          // device error code, 0 if none
    int32_t newlen;
};

// Tokens to whole pages, for 0 <= n < 2^31 and a page more.
__device__ __forceinline__ int32_t whole_pages(const PagesArgs& a, uint32_t n) {
    return static_cast<int32_t>(a.shift >= 0 ? n >> a.shift : n / static_cast<uint32_t>(a.page_size));
}
__device__ __forceinline__ int32_t pages_of(const PagesArgs& a, uint32_t tokens) {
    return whole_pages(a, tokens + static_cast<uint32_t>(a.page_size) - 1);
}

// The tokens of request b as they count for the slots' offsets: at least 0.
__device__ __forceinline__ Ask ask_extend(const PagesArgs& a, int b) {
    Ask r{};
    if (b >= a.batch) return r;
    const int32_t n = a.d_new ? a.d_new[b] : a.T;
    r.len = a.lens[b];
    r.count = max(n, 0);
    const int64_t most = static_cast<int64_t>(a.max_pages) * a.page_size;
    if (n < 0 || r.len < 0 || r.len > most) r.bad = RSSM_DEV_PAGES_COUNT;
    else if (static_cast<int64_t>(r.len) + n > most) r.bad = RSSM_DEV_PAGES_ROW;
    r.newlen = r.len;
    if (r.bad == 0) r.need = pages_of(a, r.len + n) - pages_of(a, r.len);
    return r;
}

__device__ __forceinline__ Ask ask_shrink(const PagesArgs& a, int b) {
    Ask r{};
    if (b >= a.batch) return r;
    const int32_t k = a.keep[b];
    r.len = r.newlen = a.lens[b];
    const int64_t most = static_cast<int64_t>(a.max_pages) * a.page_size;
    if (r.len < 0 || r.len > most) r.bad = RSSM_DEV_PAGES_COUNT;
    else if (a.T > 0) {
        // drafts that were never let in are not there to be taken back
        const bool none = a.refused[b] != 0;
        if (k < 0 || k > a.T || a.T > r.len) r.bad = RSSM_DEV_PAGES_COUNT;
        else if (!none) r.newlen = r.len - a.T + k;
    } else {
        if (k < 0) r.bad = RSSM_DEV_PAGES_COUNT;
        else r.newlen = min(r.len, k);
    }
    if (r.newlen != r.len) r.count = pages_of(a, r.len) - pages_of(a, r.newlen);
    return r;
}

// One round of the scan as a table to find items in: entry i is request
// `base + i`. Entries of no items share their first item with the next entry
// that has some.
struct Round {
    int32_t first[kPagesThreads];   // the request's first item (2^31 - 1: past every list)
    int32_t len[kPagesThreads];     // extend: tokens before
    int32_t held[kPagesThreads];    // pages before (extend) or left (shrink)
    int32_t page[kPagesThreads];    // extend: pages handed out before the request's; -1: refused
};

// The last entry whose first item is <= it.
__device__ __forceinline__ int find_item(const Round& R, int n, int32_t it) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (R.first[m] <= it) lo = m;
        else hi = m - 1;
    }
    return lo;
}

// Whether this block is the last to get here; every thread of the block has
// finished its reads of what the last block then writes.
__device__ __forceinline__ bool last_block(uint32_t* ticket) {
    if (gridDim.x == 1) return true;
    __shared__ bool last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(ticket, 1u) == gridDim.x - 1;
        if (last) *ticket = 0;
    }
    __syncthreads();
    return last;
}

// One round of an extend's scan. On return `upto` and `tok_end` are the scan's
// values past the request; a request that the slot list cannot hold is refused
// before its pages are counted.
__device__ __forceinline__ void extend_round(const PagesArgs& a, int b, ScanBuf& buf, Scan& scan, Ask& r, int32_t& upto,
                                             int64_t& tok_end) {
    r = ask_extend(a, b);
    tok_end = r.count;
    upto = r.need;
    const Scan before = scan;
    scan.run<true>(buf, upto, tok_end);
    if (scan.cy <= a.max_tokens) return;                       // uniform: the lists hold every token so far
    if (r.bad == 0 && r.count > 0 && tok_end > a.max_tokens) {
        r.bad = RSSM_DEV_PAGES_SLOTS;
        r.need = 0;
    }
    int64_t unused = 0;
    upto = r.need;
    scan.cx = before.cx;
    scan.run<false>(buf, upto, unused);
}

__global__ void __launch_bounds__(kPagesThreads) pages_extend_kernel(const PagesArgs a) {
    __shared__ ScanBuf buf;
    __shared__ int32_t s_fit;
    __shared__ Round R;
    after_predecessor();
    const int tid = threadIdx.x, nthr = blockDim.x;
    const int32_t nfree = *a.free_count;
    const int rounds = (a.batch + nthr - 1) / nthr;

    // Total tokens, and the pages that go out: all that are asked for, or else
    // the largest scan value that the pool covers (the scan grows, so the requests
    // past it get none).
    if (tid == 0) s_fit = 0;
    Scan scan;
    Ask r{};
    int32_t upto = 0;
    int64_t tok_end = 0;
    for (int i = 0; i < rounds; ++i) {
        extend_round(a, i * nthr + tid, buf, scan, r, upto, tok_end);
        if (scan.cx > nfree && r.need > 0 && upto <= nfree) atomicMax(&s_fit, upto);
        else if (scan.cx <= nfree && tid == 0) atomicMax(&s_fit, scan.cx);
    }
    __syncthreads();
    const int32_t out = s_fit, base = nfree - out;
    const int64_t total = min(scan.cy, static_cast<int64_t>(a.max_tokens));
    const int64_t per = ((total + gridDim.x - 1) / gridDim.x + kRun - 1) / kRun * kRun;
    const int32_t t0 = static_cast<int32_t>(min(total, per * blockIdx.x)), t1 = static_cast<int32_t>(min(total, t0 + per));

    // The requests again, in order, now with what each one gets (with one round
    // the values are still in registers).
    scan.reset();
    for (int i = 0; i < rounds; ++i) {
        if (rounds > 1) {
            __syncthreads();                                   // the round before is used up
            extend_round(a, i * nthr + tid, buf, scan, r, upto, tok_end);
        }
        if (r.bad == 0 && r.need > 0 && upto > out) r.bad = RSSM_DEV_PAGES_EMPTY;
        R.first[tid] = static_cast<int32_t>(min(tok_end - r.count, static_cast<int64_t>(0x7FFFFFFF)));
        R.len[tid] = r.len;
        R.held[tid] = pages_of(a, max(r.len, 0));
        R.page[tid] = r.bad ? -1 : upto - r.need;
        __syncthreads();
        const int32_t g0 = max(t0, R.first[0]), g1 = static_cast<int32_t>(min(static_cast<int64_t>(t1), rounds > 1 ? scan.cy : total));
        int e = -1;
        int32_t next = 0;
        for (int64_t q8 = g0 / kRun * kRun + kRun * tid; q8 < g1; q8 += kRun * nthr) {
            const int32_t q = static_cast<int32_t>(q8);
            if (max(q, g0) >= next || e < 0) {
                e = find_item(R, nthr, max(q, g0));
                next = e + 1 < nthr ? R.first[e + 1] : 0x7FFFFFFF;
            }
            // In a long prompt the next kRun tokens are the same request's, of one page or
            // of two. (Every warp meets a page's end: the path must take it.)
            if (a.wide && q >= g0 && q <= g1 - kRun && q >= R.first[e] && q <= next - kRun && R.page[e] >= 0 &&
                a.page_size >= kRun) {
                const int32_t pos = R.len[e] + (q - R.first[e]), p = whole_pages(a, pos), off = pos - p * a.page_size;
                const int32_t left = a.page_size - off;          // tokens to the page's end
                const int32_t held = R.held[e], fresh = base + R.page[e] - held;
                int32_t* row = a.table + static_cast<int64_t>(i * nthr + e) * a.max_pages + p;
                const int32_t p1 = left < kRun ? p + 1 : p;
                const int32_t id0 = p < held ? row[0] : a.free_list[fresh + p];
                const int32_t id1 = p1 < held ? row[p1 - p] : a.free_list[fresh + p1];
                // a fresh page's first token is a new one, so the page is entered with it
                if (p >= held && off == 0) row[0] = id0;
                if (p1 > p && p1 >= held) row[1] = id1;
                const int32_t s0 = id0 * a.page_size + off, s1 = id1 * a.page_size - left;
#pragma unroll
                for (int j = 0; j < kRun; j += 4) {
                    *reinterpret_cast<int4*>(a.slots + q + j) =
                        make_int4((j < left ? s0 : s1) + j, (j + 1 < left ? s0 : s1) + j + 1, (j + 2 < left ? s0 : s1) + j + 2,
                                  (j + 3 < left ? s0 : s1) + j + 3);
                    if (a.positions)
                        *reinterpret_cast<int4*>(a.positions + q + j) = make_int4(pos + j, pos + j + 1, pos + j + 2, pos + j + 3);
                }
                continue;
            }
            // token by token
            int cur = e;
            int32_t upto_next = next;
#pragma unroll 1
            for (int32_t it = max(q, g0); it < g1 && it < q8 + kRun; ++it) {
                while (upto_next <= it && cur + 1 < nthr) {
                    ++cur;
                    upto_next = cur + 1 < nthr ? R.first[cur + 1] : 0x7FFFFFFF;
                }
                int32_t slot = -1, pos = -1;
                if (R.page[cur] >= 0) {
                    pos = R.len[cur] + (it - R.first[cur]);
                    const int32_t p = whole_pages(a, pos), off = pos - p * a.page_size, held = R.held[cur];
                    int32_t* at = a.table + static_cast<int64_t>(i * nthr + cur) * a.max_pages + p;
                    const int32_t page = p < held ? *at : a.free_list[base + R.page[cur] + (p - held)];
                    if (p >= held && off == 0) *at = page;
                    slot = page * a.page_size + off;
                }
                a.slots[it] = slot;
                if (a.positions) a.positions[it] = pos;
            }
        }
    }
    if (!last_block(a.ticket)) return;
    // The new lengths and the free count, by the last block.
    scan.reset();
    for (int i = 0; i < rounds; ++i) {
        const int b = i * nthr + tid;
        if (rounds > 1) {
            extend_round(a, b, buf, scan, r, upto, tok_end);
            if (r.bad == 0 && r.need > 0 && upto > out) r.bad = RSSM_DEV_PAGES_EMPTY;
        }
        if (b < a.batch) {
            if (r.bad) report_error(a.err, r.bad, b, a.d_new ? a.d_new[b] : a.T);
            else if (r.count > 0) a.lens[b] = r.len + r.count;
            if (r.bad || r.count > 0) a.refused[b] = r.bad != 0;
        }
    }
    if (tid == 0) *a.free_count = base;
}

__global__ void __launch_bounds__(kPagesThreads) pages_shrink_kernel(const PagesArgs a) {
    __shared__ ScanBuf buf;
    __shared__ Round R;
    after_predecessor();
    const int tid = threadIdx.x, nthr = blockDim.x;
    const int32_t nfree = *a.free_count;
    const int rounds = (a.batch + nthr - 1) / nthr;
    Scan scan;
    Ask r{};
    int32_t upto = 0;
    int64_t unused = 0;
    for (int i = 0; i < rounds; ++i) {
        r = ask_shrink(a, i * nthr + tid);
        upto = r.count;
        scan.run<false>(buf, upto, unused);
    }
    // never past the stack's end, whatever the lengths say
    const int32_t total = min(scan.cx, a.num_pages - nfree);
    const int32_t per = (total + gridDim.x - 1) / gridDim.x;
    const int32_t t0 = min(total, per * static_cast<int32_t>(blockIdx.x)), t1 = min(total, t0 + per);
    if (rounds > 1) scan.reset();
    for (int i = 0; i < rounds; ++i) {
        if (rounds > 1) {
            __syncthreads();                                   // the round before is used up
            r = ask_shrink(a, i * nthr + tid);
            upto = r.count;
            scan.run<false>(buf, upto, unused);
        }
        R.first[tid] = upto - r.count;
        R.held[tid] = pages_of(a, max(r.newlen, 0));
        __syncthreads();
        const int32_t g0 = max(t0, R.first[0]), g1 = min(t1, scan.cx);
        for (int32_t it = g0 + tid; it < g1; it += nthr) {
            const int e = find_item(R, nthr, it);
            int32_t* p = a.table + static_cast<int64_t>(i * nthr + e) * a.max_pages + R.held[e] + (it - R.first[e]);
            a.free_list[nfree + it] = *p;
            *p = -1;
        }
    }
    if (!last_block(a.ticket)) return;
    for (int i = 0; i < rounds; ++i) {
        const int b = i * nthr + tid;
        if (rounds > 1) r = ask_shrink(a, b);
        if (b >= a.batch) continue;
        if (r.bad) report_error(a.err, r.bad, b, a.keep[b]);
        else a.lens[b] = r.newlen;
    }
    if (tid == 0) *a.free_count = nfree + total;
}

// A decode step's extend: T tokens (at most kStepTokens) for every request, a
// thread a request, one block.
__global__ void __launch_bounds__(kStepThreads) pages_step_kernel(const PagesArgs a) {
    __shared__ ScanBuf buf;
    __shared__ int32_t s_fit;
    after_predecessor();
    const int tid = threadIdx.x, n = blockDim.x;
    const int32_t nfree = *a.free_count;
    const int rounds = (a.batch + n - 1) / n;
    if (tid == 0) s_fit = 0;
    Scan scan;
    Ask r{};
    int32_t upto = 0;
    int64_t unused = 0;
    for (int i = 0; i < rounds; ++i) {
        r = ask_extend(a, i * n + tid);
        upto = r.need;
        scan.run<false>(buf, upto, unused);
        if (scan.cx > nfree && r.need > 0 && upto <= nfree) atomicMax(&s_fit, upto);
        else if (scan.cx <= nfree && tid == 0) atomicMax(&s_fit, scan.cx);
    }
    int32_t out = scan.cx;
    if (scan.cx > nfree) {                                     // uniform
        __syncthreads();
        out = s_fit;
    }
    const int32_t base = nfree - out;
    scan.reset();
    for (int i = 0; i < rounds; ++i) {
        const int b = i * n + tid;
        if (rounds > 1) {
            r = ask_extend(a, b);
            upto = r.need;
            scan.run<false>(buf, upto, unused);
        }
        if (b >= a.batch) continue;
        if (r.bad == 0 && r.need > 0 && upto > out) r.bad = RSSM_DEV_PAGES_EMPTY;
        const int32_t held = pages_of(a, max(r.len, 0));
        int32_t* row = a.table + static_cast<int64_t>(b) * a.max_pages;
        int32_t* slots = a.slots + static_cast<int64_t>(b) * a.T;
        int32_t p = whole_pages(a, max(r.len, 0)), off = r.len - p * a.page_size, page = -1;
        if (r.bad == 0 && off > 0) page = row[p];
        for (int t = 0; t < a.T; ++t) {
            if (r.bad == 0 && off == 0) {
                page = a.free_list[base + upto - r.need + (p - held)];
                row[p] = page;
            }
            slots[t] = r.bad || page < 0 ? -1 : page * a.page_size + off;
            if (a.positions) a.positions[static_cast<int64_t>(b) * a.T + t] = r.bad ? -1 : r.len + t;
            if (++off == a.page_size) {
                off = 0;
                ++p;
            }
        }
        if (r.bad) report_error(a.err, r.bad, b, a.T);
        else a.lens[b] = r.len + a.T;
        a.refused[b] = r.bad != 0;
    }
    if (tid == 0) *a.free_count = base;                        // every thread read it before the scan's barrier
}

// A decode step's rollback: at most a few pages a request, one block.
__global__ void __launch_bounds__(kStepThreads) pages_step_back_kernel(const PagesArgs a) {
    __shared__ ScanBuf buf;
    after_predecessor();
    const int tid = threadIdx.x, n = blockDim.x;
    const int32_t nfree = *a.free_count;
    Scan scan;
    int64_t unused = 0;
    for (int i = 0; i * n < a.batch; ++i) {
        const int b = i * n + tid;
        const Ask r = ask_shrink(a, b);
        int32_t upto = r.count;
        scan.run<false>(buf, upto, unused);
        if (b >= a.batch) continue;
        int32_t* row = a.table + static_cast<int64_t>(b) * a.max_pages + pages_of(a, max(r.newlen, 0));
        for (int j = 0; j < r.count; ++j) {
            const int32_t at = nfree + upto - r.count + j;
            if (at < a.num_pages) a.free_list[at] = row[j];    // never past the stack's end
            row[j] = -1;
        }
        if (r.bad) report_error(a.err, r.bad, b, a.keep[b]);
        else a.lens[b] = r.newlen;
    }
    if (tid == 0) *a.free_count = min(nfree + scan.cx, a.num_pages);
}

__global__ void pages_init_kernel(int32_t* lens, int batch, int32_t* table, int64_t entries, int32_t* free_list,
                                  const int32_t* free0, int num_pages, int32_t* free_count, int32_t* err,
                                  int32_t* refused, uint32_t* ticket) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int64_t n = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = t; i < entries; i += n) table[i] = -1;
    for (int64_t i = t; i < num_pages; i += n) free_list[i] = free0 ? free0[i] : static_cast<int32_t>(i);
    for (int64_t i = t; i < batch; i += n) lens[i] = refused[i] = 0;
    if (t == 0) {
        *free_count = num_pages;
        *ticket = 0;
        for (int i = 0; i < 4; ++i) err[i] = 0;
    }
}

constexpr size_t kPagesAlign = 256;
size_t up(size_t v) { return (v + kPagesAlign - 1) / kPagesAlign * kPagesAlign; }

rssm_status pages_layout(const rssm_pages_config* c, rssm_pages_layout* L) {
    if (c == nullptr || c->batch < 1 || c->page_size < 1 || c->num_pages < 1 || c->max_pages < 1)
        return RSSM_ERR_INVALID_ARG;
    if (static_cast<int64_t>(c->num_pages) * c->page_size > 0x7FFFFFFF ||
        static_cast<int64_t>(c->max_pages) * c->page_size > 0x7FFFFFFF ||
        static_cast<int64_t>(c->batch) * c->max_pages > 0x7FFFFFFF)
        return RSSM_ERR_INVALID_ARG;
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t o = off; off += up(bytes); return o; };
    L->lens = take(4 * static_cast<size_t>(c->batch));
    L->table = take(4 * static_cast<size_t>(c->batch) * c->max_pages);
    L->free = take(4 * static_cast<size_t>(c->num_pages));
    L->free_count = take(kPagesAlign);    // the count, and the ticket 128 bytes on
    L->err = take(16);
    L->refused = take(4 * static_cast<size_t>(c->batch));
    L->total_bytes = off;
    return RSSM_OK;
}

}  // namespace
}  // namespace rssm

using namespace rssm;

struct rssm_pages {
    rssm_pages_config cfg;
    rssm_pages_layout lay;
    char* base;
};

namespace {

PagesArgs pages_args(const rssm_pages* h) {
    PagesArgs a{};
    a.lens = reinterpret_cast<int32_t*>(h->base + h->lay.lens);
    a.table = reinterpret_cast<int32_t*>(h->base + h->lay.table);
    a.free_list = reinterpret_cast<int32_t*>(h->base + h->lay.free);
    a.free_count = reinterpret_cast<int32_t*>(h->base + h->lay.free_count);
    a.ticket = reinterpret_cast<uint32_t*>(h->base + h->lay.free_count + 128);
    a.err = reinterpret_cast<int32_t*>(h->base + h->lay.err);
    a.refused = reinterpret_cast<int32_t*>(h->base + h->lay.refused);
    a.batch = h->cfg.batch;
    a.page_size = h->cfg.page_size;
    a.num_pages = h->cfg.num_pages;
    a.max_pages = h->cfg.max_pages;
    a.shift = -1;
    if ((a.page_size & (a.page_size - 1)) == 0)
        for (a.shift = 0; (1 << a.shift) < a.page_size; ++a.shift) {}
    return a;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Blocks for `items` items at most: one per kItemsPerBlock, two per SM at most.
cudaError_t pages_grid(int64_t items, int* blocks) {
    int sms = 0, smem = 0;
    const cudaError_t e = device_limits(&sms, &smem);
    if (e != cudaSuccess) return e;
    const int64_t want = (items + kItemsPerBlock - 1) / kItemsPerBlock;
    *blocks = static_cast<int>(want < 1 ? 1 : want > 2 * sms ? 2 * sms : want);
    return cudaSuccess;
}

int pages_threads(int batch) { return batch <= kPagesThreads / 2 ? kPagesThreads / 2 : kPagesThreads; }

// Threads of a single-block kernel: one a request, in whole warps.
int step_threads(int batch) { return batch >= kStepThreads ? kStepThreads : (batch + 31) / 32 * 32; }

// Whether the single-block kernels take T tokens for every request: an extend and a
// rollback take them about 2.8 + 1.2 T us for every 1024 requests, and the
// others 7 to 8 us (1024 requests: T = 1 4.0 against 9.0, T = 8 11.8 against
// 7.6; 8192: T = 1 23 against 55; 64: T = 16 4.8 against 5.9).
bool step_takes(int32_t T, int32_t batch) {
    return T <= kStepTokens && T * (batch < kStepThreads ? batch : kStepThreads) <= 4 * kStepThreads;
}

rssm_status pages_shrink(rssm_pages* h, int32_t T, const int32_t* keep, void* stream) {
    PagesArgs a = pages_args(h);
    a.T = T;
    a.keep = keep;
    if (T > 0 && step_takes(T, a.batch)) {
        return launch_overlapped(pages_step_back_kernel, 1, step_threads(a.batch), 0, static_cast<cudaStream_t>(stream), a) == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
    }
    // a rollback returns at most ceil(T / page_size) pages a request
    const int64_t per = T > 0 ? (static_cast<int64_t>(T) + h->cfg.page_size - 1) / h->cfg.page_size : h->cfg.max_pages;
    const int64_t items = per * h->cfg.batch;
    int blocks = 1;
    cudaError_t e = pages_grid(items < h->cfg.num_pages ? items : h->cfg.num_pages, &blocks);
    if (e == cudaSuccess) {
        static LaunchCache lc;
        e = cached_dyn_smem(lc, pages_shrink_kernel, kSpread);
        if (e == cudaSuccess) e = launch_overlapped(pages_shrink_kernel, blocks, pages_threads(a.batch), kSpread, static_cast<cudaStream_t>(stream), a);
    }
    return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}

}  // namespace

extern "C" {

rssm_status rssm_pages_layout_for(const rssm_pages_config* cfg, rssm_pages_layout* out) {
    if (out == nullptr) return RSSM_ERR_INVALID_ARG;
    return pages_layout(cfg, out);
}

rssm_status rssm_pages_create(const rssm_pages_config* cfg, void* d_workspace, size_t workspace_bytes,
                              const int32_t* d_free0, void* stream, rssm_pages** out) {
    if (out == nullptr) return RSSM_ERR_INVALID_ARG;
    *out = nullptr;
    rssm_pages_layout L;
    const rssm_status st = pages_layout(cfg, &L);
    if (st != RSSM_OK) return st;
    if (d_workspace == nullptr || (reinterpret_cast<uintptr_t>(d_workspace) % kPagesAlign) != 0 || !aligned4(d_free0))
        return RSSM_ERR_INVALID_ARG;
    if (workspace_bytes < L.total_bytes) return RSSM_ERR_CAPACITY;
    rssm_pages* h = new (std::nothrow) rssm_pages;
    if (h == nullptr) return RSSM_ERR_CAPACITY;
    h->cfg = *cfg;
    h->lay = L;
    h->base = static_cast<char*>(d_workspace);
    const PagesArgs a = pages_args(h);
    pages_init_kernel<<<256, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        a.lens, a.batch, a.table, static_cast<int64_t>(a.batch) * a.max_pages, a.free_list, d_free0, a.num_pages,
        a.free_count, a.err, a.refused, a.ticket);
    if (cudaGetLastError() != cudaSuccess) {
        delete h;
        return RSSM_ERR_CUDA;
    }
    *out = h;
    return RSSM_OK;
}

rssm_status rssm_pages_extend(rssm_pages* h, int32_t T, const int32_t* d_new, int32_t* d_slots,
                              int32_t* d_positions, int32_t max_tokens, void* stream) {
    if (h == nullptr || max_tokens < 0 || (d_slots == nullptr && max_tokens > 0)) return RSSM_ERR_INVALID_ARG;
    if (!aligned4(d_slots) || !aligned4(d_positions) || !aligned4(d_new)) return RSSM_ERR_INVALID_ARG;
    if (d_new == nullptr ? (T < 1 || static_cast<int64_t>(T) * h->cfg.batch > max_tokens) : T != 0)
        return RSSM_ERR_INVALID_ARG;
    PagesArgs a = pages_args(h);
    a.d_new = d_new;
    a.T = T;
    a.slots = d_slots;
    a.positions = d_positions;
    a.max_tokens = max_tokens;
    a.wide = ((reinterpret_cast<uintptr_t>(d_slots) | reinterpret_cast<uintptr_t>(d_positions)) & 15u) == 0;
    if (d_new == nullptr && step_takes(T, a.batch)) {
        return launch_overlapped(pages_step_kernel, 1, step_threads(a.batch), 0, static_cast<cudaStream_t>(stream), a) == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
    }
    int blocks = 1;
    cudaError_t e = pages_grid(d_new ? max_tokens : static_cast<int64_t>(T) * h->cfg.batch, &blocks);
    if (e == cudaSuccess) {
        static LaunchCache lc;
        e = cached_dyn_smem(lc, pages_extend_kernel, kSpread);
        if (e == cudaSuccess) e = launch_overlapped(pages_extend_kernel, blocks, pages_threads(a.batch), kSpread, static_cast<cudaStream_t>(stream), a);
    }
    return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}

rssm_status rssm_pages_rollback(rssm_pages* h, int32_t T, const int32_t* d_accepted, void* stream) {
    if (h == nullptr || d_accepted == nullptr || !aligned4(d_accepted) || T < 1) return RSSM_ERR_INVALID_ARG;
    return pages_shrink(h, T, d_accepted, stream);
}

rssm_status rssm_pages_truncate(rssm_pages* h, const int32_t* d_keep, void* stream) {
    if (h == nullptr || d_keep == nullptr || !aligned4(d_keep)) return RSSM_ERR_INVALID_ARG;
    return pages_shrink(h, 0, d_keep, stream);
}

rssm_status rssm_pages_get_error(rssm_pages* h, int32_t* err4, void* stream) {
    if (h == nullptr || err4 == nullptr) return RSSM_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    void* dev = h->base + h->lay.err;
    cudaError_t e = cudaMemcpyAsync(err4, dev, 16, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) e = cudaMemsetAsync(dev, 0, 16, s);
    return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}

rssm_status rssm_pages_destroy(rssm_pages* h) {
    if (h == nullptr) return RSSM_ERR_INVALID_ARG;
    delete h;
    return RSSM_OK;
}

}  // extern "C"
