// The page table of a batch: pages handed out (extend) and taken back
// (rollback, truncate) on the GPU from device counts, with the slot and the
// position of every new token.
//
// Both are one exclusive scan over the requests (pages per request) followed by
// work on the scan's items (tokens, or pages going back). Every block makes
// the whole scan for itself, which costs it one pass over 8 bytes a request
// from L2, and then takes an equal share of the items. So one launch does it
// without any block waiting for another; the last block to have read the
// lengths (a ticket) writes the new ones and the free count. The order of the
// pages is that of the requests whatever the launch.
//
// Bound by latency for a decode step (a block, two barriers a scan), and by the
// slot and position stores (8 bytes a token) for prompts.
#include <cstring>
#include <new>

#include "common.cuh"

namespace rssm {
namespace {

constexpr int kPagesThreads = 1024;
constexpr int kTokensPerBlock = 4096;   // at least; more blocks than this gives cost more scans than they save

struct PagesArgs {
    int32_t* lens;
    int32_t* table;
    int32_t* free_list;
    int32_t* free_count;
    int32_t* err;
    uint32_t* ticket;
    int32_t batch, page_size, num_pages, max_pages;
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

// Inclusive scan of one value a thread over the block, added to *carry (the
// total so far, the same in every thread), which the block's total then grows by.
template <class V>
__device__ __forceinline__ V block_scan(V v, V* s_warp, V* carry) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V n = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += n;
    }
    __syncthreads();                      // s_warp may hold an earlier scan
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    V w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V n = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += n;
    }
    const V before = warp == 0 ? V(0) : __shfl_sync(0xffffffffu, w, warp - 1);
    const V total = __shfl_sync(0xffffffffu, w, 31);
    v += *carry + before;
    *carry += total;
    return v;
}

// What one request asks for.
struct Ask {
    int32_t len, count;   // length; new tokens (extend) or pages that go back
    int32_t need;         // pages wanted (extend)
    int32_t bad;          // device error code, 0 if none
    int32_t newlen;
};

__device__ __forceinline__ int32_t pages_of(int64_t tokens, int32_t ps) {
    return static_cast<int32_t>((tokens + ps - 1) / ps);
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
    if (r.bad == 0) r.need = pages_of(static_cast<int64_t>(r.len) + n, a.page_size) - pages_of(r.len, a.page_size);
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
        if (k < 0 || k > a.T || a.T > r.len) r.bad = RSSM_DEV_PAGES_COUNT;
        else r.newlen = r.len - a.T + k;
    } else {
        if (k < 0) r.bad = RSSM_DEV_PAGES_COUNT;
        else r.newlen = min(r.len, k);
    }
    r.count = pages_of(r.len, a.page_size) - pages_of(r.newlen, a.page_size);
    return r;
}

// The requests of one batch of the scan that own items of this block, in order.
struct Listed {
    int64_t first[kPagesThreads];   // the request's first item
    int32_t request[kPagesThreads];
    int32_t len[kPagesThreads];     // extend: tokens before; shrink: pages left
    int32_t page[kPagesThreads];    // extend: the scan of its pages; -1: refused
    int32_t n;
};

// The list entry that item `it` belongs to: the last whose first item is <= it.
__device__ __forceinline__ int find_item(const Listed& L, int64_t it) {
    int lo = 0, hi = L.n - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (L.first[m] <= it) lo = m;
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

__global__ void __launch_bounds__(kPagesThreads) pages_extend_kernel(const PagesArgs a) {
    __shared__ int32_t s_need[32];
    __shared__ int64_t s_tok[32];
    __shared__ int32_t s_fit;
    __shared__ Listed L;
    const int tid = threadIdx.x;
    const int32_t nfree = *a.free_count;
    const int rounds = (a.batch + kPagesThreads - 1) / kPagesThreads;

    // total tokens, and the pages that go out: the largest scan value that the
    // pool still covers (the scan grows, so the requests past it get none)
    if (tid == 0) s_fit = 0;
    __syncthreads();
    int32_t c_need = 0;
    int64_t c_tok = 0;
    Ask r{};
    int32_t upto = 0;
    int64_t tok_end = 0;
    for (int i = 0; i < rounds; ++i) {
        r = ask_extend(a, i * kPagesThreads + tid);
        tok_end = block_scan<int64_t>(r.count, s_tok, &c_tok);
        if (r.bad == 0 && tok_end > a.max_tokens) {
            r.bad = RSSM_DEV_PAGES_SLOTS;
            r.need = 0;
        }
        upto = block_scan<int32_t>(r.need, s_need, &c_need);
        if (r.need > 0 && upto <= nfree) atomicMax(&s_fit, upto);
    }
    __syncthreads();
    const int32_t out = s_fit;               // pages handed out
    const int32_t base = nfree - out;
    const int64_t total = min(c_tok, static_cast<int64_t>(a.max_tokens));
    const int64_t per = ((total + gridDim.x - 1) / gridDim.x + 3) / 4 * 4;
    const int64_t t0 = min(total, per * blockIdx.x), t1 = min(total, t0 + per);

    // The requests again, in order, now with what each one gets (with one round
    // the values are still in registers).
    c_need = 0;
    c_tok = 0;
    for (int i = 0; i < rounds; ++i) {
        const int b = i * kPagesThreads + tid;
        if (rounds > 1) {
            r = ask_extend(a, b);
            tok_end = block_scan<int64_t>(r.count, s_tok, &c_tok);
            if (r.bad == 0 && tok_end > a.max_tokens) {
                r.bad = RSSM_DEV_PAGES_SLOTS;
                r.need = 0;
            }
            upto = block_scan<int32_t>(r.need, s_need, &c_need);
        }
        if (r.bad == 0 && r.need > 0 && upto > out) r.bad = RSSM_DEV_PAGES_EMPTY;
        const int64_t tok0 = tok_end - r.count;
        const bool mine = r.count > 0 && tok0 < t1 && tok_end > t0;
        // positions in the list, by a count over the block
        int32_t zero = 0;
        const int32_t at = block_scan<int32_t>(mine ? 1 : 0, s_need, &zero) - 1;
        if (mine) {
            L.first[at] = tok0;
            L.request[at] = b;
            L.len[at] = r.len;
            L.page[at] = r.bad ? -1 : upto - r.need;
        }
        if (tid == 0) L.n = zero;
        __syncthreads();
        if (zero > 0) {
            const int64_t g0 = max(t0, L.first[0]);
            // the list's last token: of the last request, or the block's last
            const int64_t g1 = min(t1, rounds > 1 ? c_tok : total);
            for (int64_t q = g0 / 4 * 4 + 4 * tid; q < g1; q += 4 * kPagesThreads) {
                int e = find_item(L, max(q, g0));
                int4 sl, po;
                int32_t* slv = &sl.x;
                int32_t* pov = &po.x;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t it = q + j;
                    slv[j] = pov[j] = -1;
                    if (it < g0 || it >= g1) continue;
                    while (e + 1 < L.n && L.first[e + 1] <= it) ++e;
                    if (L.page[e] < 0) continue;
                    const int32_t pos = L.len[e] + static_cast<int32_t>(it - L.first[e]);
                    const int32_t p = pos / a.page_size, off = pos - p * a.page_size;
                    const int32_t held = pages_of(L.len[e], a.page_size);
                    int32_t* row = a.table + static_cast<int64_t>(L.request[e]) * a.max_pages;
                    int32_t page;
                    if (p < held) {
                        page = row[p];
                    } else {
                        page = a.free_list[base + L.page[e] + (p - held)];
                        if (off == 0) row[p] = page;   // a fresh page's first token is a new one
                    }
                    slv[j] = page < 0 ? -1 : page * a.page_size + off;
                    pov[j] = pos;
                }
                if (a.wide && q >= g0 && q + 4 <= g1) {
                    *reinterpret_cast<int4*>(a.slots + q) = sl;
                    if (a.positions) *reinterpret_cast<int4*>(a.positions + q) = po;
                } else {
                    for (int j = 0; j < 4; ++j) {
                        if (q + j < g0 || q + j >= g1) continue;
                        a.slots[q + j] = slv[j];
                        if (a.positions) a.positions[q + j] = pov[j];
                    }
                }
            }
            __syncthreads();
        }
    }
    if (!last_block(a.ticket)) return;
    // The new lengths and the free count, by the last block.
    c_need = 0;
    c_tok = 0;
    for (int i = 0; i < rounds; ++i) {
        const int b = i * kPagesThreads + tid;
        if (rounds > 1) {
            r = ask_extend(a, b);
            tok_end = block_scan<int64_t>(r.count, s_tok, &c_tok);
            if (r.bad == 0 && tok_end > a.max_tokens) {
                r.bad = RSSM_DEV_PAGES_SLOTS;
                r.need = 0;
            }
            upto = block_scan<int32_t>(r.need, s_need, &c_need);
            if (r.bad == 0 && r.need > 0 && upto > out) r.bad = RSSM_DEV_PAGES_EMPTY;
        }
        if (b < a.batch) {
            if (r.bad) report_error(a.err, r.bad, b, a.d_new ? a.d_new[b] : a.T);
            else if (r.count > 0) a.lens[b] = r.len + r.count;
        }
    }
    if (tid == 0) *a.free_count = base;
}

__global__ void __launch_bounds__(kPagesThreads) pages_shrink_kernel(const PagesArgs a) {
    __shared__ int32_t s_back[32];
    __shared__ Listed L;
    const int tid = threadIdx.x;
    const int32_t nfree = *a.free_count;
    const int rounds = (a.batch + kPagesThreads - 1) / kPagesThreads;
    int32_t c_back = 0;
    Ask r{};
    int32_t upto = 0;
    for (int i = 0; i < rounds; ++i) {
        r = ask_shrink(a, i * kPagesThreads + tid);
        upto = block_scan<int32_t>(r.count, s_back, &c_back);
    }
    // never past the stack's end, whatever the lengths say
    const int32_t total = min(c_back, a.num_pages - nfree);
    const int32_t per = (total + gridDim.x - 1) / gridDim.x;
    const int32_t t0 = min(total, per * static_cast<int32_t>(blockIdx.x)), t1 = min(total, t0 + per);
    int32_t c2 = 0;
    for (int i = 0; i < rounds; ++i) {
        const int b = i * kPagesThreads + tid;
        if (rounds > 1) {
            r = ask_shrink(a, b);
            upto = block_scan<int32_t>(r.count, s_back, &c2);
        }
        const bool mine = r.count > 0 && upto - r.count < t1 && upto > t0;
        int32_t zero = 0;
        const int32_t at = block_scan<int32_t>(mine ? 1 : 0, s_back, &zero) - 1;
        if (mine) {
            L.first[at] = upto - r.count;
            L.request[at] = b;
            L.len[at] = pages_of(r.newlen, a.page_size);
        }
        if (tid == 0) L.n = zero;
        __syncthreads();
        if (zero > 0) {
            const int32_t g0 = max(t0, static_cast<int32_t>(L.first[0]));
            const int32_t g1 = min(t1, rounds > 1 ? c2 : c_back);
            for (int32_t it = g0 + tid; it < g1; it += kPagesThreads) {
                const int e = find_item(L, it);
                int32_t* p = a.table + static_cast<int64_t>(L.request[e]) * a.max_pages + L.len[e] +
                             (it - static_cast<int32_t>(L.first[e]));
                a.free_list[nfree + it] = *p;
                *p = -1;
            }
            __syncthreads();
        }
    }
    if (!last_block(a.ticket)) return;
    for (int i = 0; i < rounds; ++i) {
        const int b = i * kPagesThreads + tid;
        if (rounds > 1) r = ask_shrink(a, b);
        if (b >= a.batch) continue;
        if (r.bad) report_error(a.err, r.bad, b, a.keep[b]);
        else a.lens[b] = r.newlen;
    }
    if (tid == 0) *a.free_count = nfree + total;
}

__global__ void pages_init_kernel(int32_t* lens, int batch, int32_t* table, int64_t entries, int32_t* free_list,
                                  const int32_t* free0, int num_pages, int32_t* free_count, int32_t* err,
                                  uint32_t* ticket) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int64_t n = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t i = t; i < entries; i += n) table[i] = -1;
    for (int64_t i = t; i < num_pages; i += n) free_list[i] = free0 ? free0[i] : static_cast<int32_t>(i);
    for (int64_t i = t; i < batch; i += n) lens[i] = 0;
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
    a.batch = h->cfg.batch;
    a.page_size = h->cfg.page_size;
    a.num_pages = h->cfg.num_pages;
    a.max_pages = h->cfg.max_pages;
    return a;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Blocks for `items` items at most: one per kTokensPerBlock, two per SM at most.
cudaError_t pages_grid(int64_t items, int* blocks) {
    int sms = 0, smem = 0;
    const cudaError_t e = device_limits(&sms, &smem);
    if (e != cudaSuccess) return e;
    const int64_t want = (items + kTokensPerBlock - 1) / kTokensPerBlock;
    *blocks = static_cast<int>(want < 1 ? 1 : want > 2 * sms ? 2 * sms : want);
    return cudaSuccess;
}

rssm_status pages_shrink(rssm_pages* h, int32_t T, const int32_t* keep, void* stream) {
    PagesArgs a = pages_args(h);
    a.T = T;
    a.keep = keep;
    // a rollback returns at most ceil(T / page_size) pages a request
    const int64_t per = T > 0 ? (T + h->cfg.page_size - 1) / h->cfg.page_size : h->cfg.max_pages;
    const int64_t items = per * h->cfg.batch;
    int blocks = 1;
    cudaError_t e = pages_grid(items < h->cfg.num_pages ? items : h->cfg.num_pages, &blocks);
    if (e == cudaSuccess) {
        pages_shrink_kernel<<<blocks, kPagesThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
        e = cudaGetLastError();
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
        a.free_count, a.err, a.ticket);
    if (cudaGetLastError() != cudaSuccess) {
        delete h;
        return RSSM_ERR_CUDA;
    }
    *out = h;
    return RSSM_OK;
}

rssm_status rssm_pages_extend(rssm_pages* h, int32_t T, const int32_t* d_new, int32_t* d_slots,
                              int32_t* d_positions, int32_t max_tokens, void* stream) {
    if (h == nullptr || d_slots == nullptr || max_tokens < 0) return RSSM_ERR_INVALID_ARG;
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
    int blocks = 1;
    cudaError_t e = pages_grid(d_new ? max_tokens : static_cast<int64_t>(T) * h->cfg.batch, &blocks);
    if (e == cudaSuccess) {
        pages_extend_kernel<<<blocks, kPagesThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
        e = cudaGetLastError();
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
