// Entry points of the attention over a paged cache, and the cache's writer.
#include <cstring>
#include <new>

#include "attn.h"
#include "overlap.cuh"

namespace rssm {
namespace {

// New tokens' keys and values to their slots: one thread per VEC elements of K or V.
template <class TI, class TO, int VEC>
__global__ void __launch_bounds__(256) attn_append_kernel(const TI* k, const TI* v, int64_t k_stride,
                                                          int64_t v_stride, const int32_t* slots, TO* kc, TO* vc,
                                                          const float* k_scale, const float* v_scale, int tokens,
                                                          int heads, int dim, int page_size, int num_pages, int64_t page_stride, int32_t* err) {
    after_predecessor();
    const int per_head = dim / VEC, per_token = heads * per_head;
    const int64_t n = static_cast<int64_t>(tokens) * per_token;
    const bool is_v = blockIdx.y == 1;
    const TI* src = is_v ? v : k;
    TO* dst = is_v ? vc : kc;
    const float* scale = is_v ? v_scale : k_scale;
    const int64_t stride = is_v ? v_stride : k_stride;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int tok = static_cast<int>(i / per_token), e = static_cast<int>(i - static_cast<int64_t>(tok) * per_token);
        const int head = e / per_head, d = (e - head * per_head) * VEC;
        const int32_t slot = slots[tok];
        if (slot < 0) continue;
        const int page = slot / page_size;
        if (page >= num_pages) {
            if (e == 0 && !is_v) report_error(err, RSSM_DEV_ATTN_SLOT, tok, slot);
            continue;
        }
        const TI* from = src + tok * stride + head * dim + d;
        TO* to = dst + page * page_stride + (static_cast<int64_t>(head) * page_size + (slot - page * page_size)) * dim + d;
        if constexpr (sizeof(TO) == sizeof(TI)) {
            if constexpr (VEC == 1) *to = *reinterpret_cast<const TO*>(from);
            else *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
        } else {
            const float s = scale[head];
            if constexpr (VEC == 1) {
                *to = static_cast<TO>(e4m3x2(__fdiv_rn(to_f(*from), s), 0.f) & 0xFF);
            } else {
                const float4 a = load4(from), b = load4(from + 4);
                uint2 c;
                c.x = e4m3x2(__fdiv_rn(a.x, s), __fdiv_rn(a.y, s)) |
                      (static_cast<uint32_t>(e4m3x2(__fdiv_rn(a.z, s), __fdiv_rn(a.w, s))) << 16);
                c.y = e4m3x2(__fdiv_rn(b.x, s), __fdiv_rn(b.y, s)) |
                      (static_cast<uint32_t>(e4m3x2(__fdiv_rn(b.z, s), __fdiv_rn(b.w, s))) << 16);
                *reinterpret_cast<uint2*>(to) = c;
            }
        }
    }
}

constexpr size_t kAttnAlign = 256;
size_t up256(size_t v) { return (v + kAttnAlign - 1) / kAttnAlign * kAttnAlign; }

// Regions of the workspace. The error word and the counters, which every call leaves at
// zero, have one size and one place whatever the configuration, and the parts, which a
// call leaves as they fall, lie behind them: layers of any shapes may share a workspace.
struct AttnLayout {
    size_t err, arrived, arrived_round, part_ml, part_o, total;
};

int elem_size(int kv_dtype) { return kv_dtype == RSSM_F32 ? 4 : kv_dtype == RSSM_BF16 ? 2 : 1; }

rssm_status attn_check(const rssm_attn_config* c) {
    if (c == nullptr || c->batch < 1 || c->q_heads < 1 || c->kv_heads < 1 || c->head_dim < 1 || c->page_size < 1 ||
        c->num_pages < 1 || c->max_pages < 1 || c->max_draft < 1 || c->window < 0)
        return RSSM_ERR_INVALID_ARG;
    if (c->q_heads % c->kv_heads != 0) return RSSM_ERR_INVALID_ARG;
    if (c->in_dtype != RSSM_F32 && c->in_dtype != RSSM_BF16) return RSSM_ERR_INVALID_ARG;
    if (c->kv_dtype != RSSM_F32 && c->kv_dtype != RSSM_BF16 && c->kv_dtype != RSSM_KV_FP8) return RSSM_ERR_INVALID_ARG;
    if (!(c->scale == c->scale) || c->scale - c->scale != 0.f) return RSSM_ERR_INVALID_ARG;   // NaN, infinite
    if (static_cast<int64_t>(c->num_pages) * c->page_size > 0x7FFFFFFF ||
        static_cast<int64_t>(c->max_pages) * c->page_size > 0x7FFFFFFF ||
        static_cast<int64_t>(c->batch) * c->max_pages > 0x7FFFFFFF ||
        static_cast<int64_t>(c->batch) * c->q_heads * c->max_draft > 0x7FFFFFFF)
        return RSSM_ERR_INVALID_ARG;
    const int64_t page = static_cast<int64_t>(c->kv_heads) * c->page_size * c->head_dim;
    if (c->page_stride != 0 && (c->page_stride < page || (c->page_stride * elem_size(c->kv_dtype)) % 16 != 0 ||
                                c->page_stride >= (1ll << 38)))
        return RSSM_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return RSSM_ERR_UNSUPPORTED;
    if (c->page_size % kAttnGroup != 0 || c->max_draft > kMaxDraft) return RSSM_ERR_UNSUPPORTED;
    if ((c->in_dtype == RSSM_F32) != (c->kv_dtype == RSSM_F32)) return RSSM_ERR_UNSUPPORTED;
    return RSSM_OK;
}

// Blocks' worth of query rows per cache head.
int attn_chunks(int rows, const rssm_attn_config& c) {
    const int per = attn_block_rows(rows, c.kv_dtype, c.head_dim);
    return (rows + per - 1) / per;
}

AttnLayout attn_layout(const rssm_attn_config& c) {
    AttnLayout L{};
    const int rows = c.max_draft * (c.q_heads / c.kv_heads);
    const size_t parts = 2 * static_cast<size_t>(kAttnMaxGrid) * attn_block_rows(rows, c.kv_dtype, c.head_dim);
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t o = off; off += up256(bytes); return o; };
    L.err = take(20);                     // the error word, and whether any wait ran out
    L.arrived = take(4 * static_cast<size_t>(kAttnMaxGrid));
    L.arrived_round = take(4 * 2 * static_cast<size_t>(kAttnMaxGrid));
    L.part_ml = take(parts * 8);
    L.part_o = take(parts * c.head_dim * 4);
    L.total = off;
    return L;
}

// cuTensorMapEncodeTiled of the driver, or null where there is none.
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult st;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &st) != cudaSuccess ||
            st != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// A cache as bytes [page][head][128-byte chunk of a token][token of the page][byte],
// boxes of 16 tokens of one head: a slot's rows are 128 bytes (64 for FP8 heads
// of 64) under the swizzle of that width.
bool encode_cache(CUtensorMap* m, void* base, const rssm_attn_config& c) {
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t es = elem_size(c.kv_dtype), rb = es * c.head_dim, cb = rb < 128 ? rb : 128;
    const cuuint64_t page = c.page_stride ? c.page_stride * es : rb * c.page_size * c.kv_heads;
    const cuuint64_t dims[5] = {cb, static_cast<cuuint64_t>(c.page_size), rb / cb, static_cast<cuuint64_t>(c.kv_heads),
                                static_cast<cuuint64_t>(c.num_pages)};
    const cuuint64_t strides[4] = {rb, cb, rb * c.page_size, page};
    const cuuint32_t box[5] = {static_cast<cuuint32_t>(cb), kAttnGroup, static_cast<cuuint32_t>(rb / cb), 1, 1};
    const cuuint32_t step[5] = {1, 1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, base, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              cb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace rssm

using namespace rssm;

struct rssm_attn {
    CUtensorMap kmap, vmap;       // first: 64-byte aligned
    rssm_attn_config cfg;
    AttnLayout lay;
    char* base;
    void *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int64_t page_stride;
};

namespace {

template <class TI, class TO>
cudaError_t launch_append(const rssm_attn* h, int tokens, const void* k, int64_t ks, const void* v, int64_t vs,
                          const int32_t* slots, cudaStream_t s) {
    const rssm_attn_config& c = h->cfg;
    constexpr int kWide = 16 / sizeof(TI);
    const bool wide = aligned(k, 16) && aligned(v, 16) && (ks * sizeof(TI)) % 16 == 0 && (vs * sizeof(TI)) % 16 == 0;
    const int64_t n = static_cast<int64_t>(tokens) * c.kv_heads * (c.head_dim / (wide ? kWide : 1));
    const int64_t want = (n + 255) / 256;
    const dim3 grid(static_cast<unsigned>(want < 8 * 152 ? want : 8 * 152), 2);
    int32_t* err = reinterpret_cast<int32_t*>(h->base + h->lay.err);
    auto go = [&](auto kernel) {
        return launch_overlapped(kernel, grid, 256, 0, s, static_cast<const TI*>(k), static_cast<const TI*>(v), ks, vs, slots,
                                    static_cast<TO*>(h->k_cache), static_cast<TO*>(h->v_cache), h->k_scale, h->v_scale,
                                    tokens, c.kv_heads, c.head_dim, c.page_size, c.num_pages, h->page_stride, err);
    };
    return wide ? go(attn_append_kernel<TI, TO, kWide>) : go(attn_append_kernel<TI, TO, 1>);
}

}  // namespace

extern "C" {

rssm_status rssm_attn_workspace_size(const rssm_attn_config* cfg, size_t* bytes) {
    if (bytes == nullptr) return RSSM_ERR_INVALID_ARG;
    const rssm_status st = attn_check(cfg);
    if (st != RSSM_OK) return st;
    *bytes = attn_layout(*cfg).total;
    return RSSM_OK;
}

rssm_status rssm_attn_create(const rssm_attn_config* cfg, void* d_k_cache, void* d_v_cache, const float* d_k_scale,
                             const float* d_v_scale, void* d_workspace, size_t workspace_bytes, void* stream,
                             rssm_attn** out) {
    if (out == nullptr) return RSSM_ERR_INVALID_ARG;
    *out = nullptr;
    const rssm_status st = attn_check(cfg);
    if (st != RSSM_OK) return st;
    if (d_k_cache == nullptr || d_v_cache == nullptr || !aligned(d_k_cache, 16) || !aligned(d_v_cache, 16) ||
        d_workspace == nullptr || !aligned(d_workspace, kAttnAlign))
        return RSSM_ERR_INVALID_ARG;
    const bool fp8 = cfg->kv_dtype == RSSM_KV_FP8;
    if ((d_k_scale != nullptr) != fp8 || (d_v_scale != nullptr) != fp8 || !aligned(d_k_scale, 4) || !aligned(d_v_scale, 4))
        return RSSM_ERR_INVALID_ARG;
    const AttnLayout L = attn_layout(*cfg);
    if (workspace_bytes < L.total) return RSSM_ERR_CAPACITY;
    rssm_attn* h = new (std::nothrow) rssm_attn;
    if (h == nullptr) return RSSM_ERR_CAPACITY;
    h->cfg = *cfg;
    h->lay = L;
    h->base = static_cast<char*>(d_workspace);
    h->k_cache = d_k_cache;
    h->v_cache = d_v_cache;
    h->k_scale = d_k_scale;
    h->v_scale = d_v_scale;
    h->page_stride = cfg->page_stride ? cfg->page_stride
                                      : static_cast<int64_t>(cfg->kv_heads) * cfg->page_size * cfg->head_dim;
    if (h->cfg.scale == 0.f) h->cfg.scale = cfg->head_dim == 64 ? 0.125f : cfg->head_dim == 128 ? 0.08838834764831845f : 0.0625f;
    bool ok = encode_cache(&h->kmap, d_k_cache, *cfg) && encode_cache(&h->vmap, d_v_cache, *cfg);
    ok = ok && cudaMemsetAsync(h->base, 0, L.part_ml, static_cast<cudaStream_t>(stream)) == cudaSuccess;
    if (!ok) {
        delete h;
        return RSSM_ERR_CUDA;
    }
    *out = h;
    return RSSM_OK;
}

rssm_status rssm_attn_append(rssm_attn* h, int32_t tokens, const void* d_k, int64_t k_stride, const void* d_v,
                             int64_t v_stride, const int32_t* d_slots, void* stream) {
    if (h == nullptr || tokens < 0) return RSSM_ERR_INVALID_ARG;
    const rssm_attn_config& c = h->cfg;
    const int64_t row = static_cast<int64_t>(c.kv_heads) * c.head_dim;
    if (k_stride == 0) k_stride = row;
    if (v_stride == 0) v_stride = row;
    if (k_stride < row || v_stride < row) return RSSM_ERR_INVALID_ARG;
    if (tokens == 0) return RSSM_OK;
    const uintptr_t es = c.in_dtype == RSSM_F32 ? 4 : 2;
    if (d_k == nullptr || d_v == nullptr || d_slots == nullptr || !aligned(d_slots, 4) || !aligned(d_k, es) || !aligned(d_v, es))
        return RSSM_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (c.kv_dtype == RSSM_F32) e = launch_append<float, float>(h, tokens, d_k, k_stride, d_v, v_stride, d_slots, s);
    else if (c.kv_dtype == RSSM_BF16)
        e = launch_append<__nv_bfloat16, __nv_bfloat16>(h, tokens, d_k, k_stride, d_v, v_stride, d_slots, s);
    else e = launch_append<__nv_bfloat16, uint8_t>(h, tokens, d_k, k_stride, d_v, v_stride, d_slots, s);
    return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}

rssm_status rssm_attn_decode(rssm_attn* h, int32_t T, const void* d_q, int64_t q_stride, const int32_t* d_lens,
                             const int32_t* d_table, void* d_out, float* d_lse, void* stream) {
    if (h == nullptr || T < 1) return RSSM_ERR_INVALID_ARG;
    const rssm_attn_config& c = h->cfg;
    const int64_t row = static_cast<int64_t>(c.q_heads) * c.head_dim;
    const int es = c.in_dtype == RSSM_F32 ? 4 : 2;
    if (q_stride == 0) q_stride = row;
    if (q_stride < row || (q_stride * es) % 16 != 0) return RSSM_ERR_INVALID_ARG;
    if (d_q == nullptr || d_lens == nullptr || d_table == nullptr || d_out == nullptr || !aligned(d_q, 16) ||
        !aligned(d_out, 16) || !aligned(d_lens, 4) || !aligned(d_table, 4) || !aligned(d_lse, 4))
        return RSSM_ERR_INVALID_ARG;
    if (T > c.max_draft) return RSSM_ERR_CAPACITY;
    AttnArgs a{};
    a.q = d_q;
    a.q_stride = q_stride;
    a.lens = d_lens;
    a.table = d_table;
    a.out = d_out;
    a.lse = d_lse;
    a.k_scale = h->k_scale;
    a.v_scale = h->v_scale;
    a.err = reinterpret_cast<int32_t*>(h->base + h->lay.err);
    a.arrived = reinterpret_cast<uint32_t*>(h->base + h->lay.arrived);
    a.arrived_round = reinterpret_cast<uint32_t*>(h->base + h->lay.arrived_round);
    a.part_ml = reinterpret_cast<float2*>(h->base + h->lay.part_ml);
    a.part_o = reinterpret_cast<float*>(h->base + h->lay.part_o);
    a.B = c.batch;
    a.q_heads = c.q_heads;
    a.kv_heads = c.kv_heads;
    a.group = c.q_heads / c.kv_heads;
    a.T = T;
    const int rows = T * a.group;
    a.chunks = attn_chunks(rows, c);
    a.page_size = c.page_size;
    a.num_pages = c.num_pages;
    a.max_pages = c.max_pages;
    a.window = c.window;
    a.scale_log2 = c.scale * 1.4426950408889634f;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const auto launch = c.kv_dtype == RSSM_F32 ? attn_launch_f32 : c.kv_dtype == RSSM_BF16 ? attn_launch_bf16 : attn_launch_fp8;
    return launch(a, c.head_dim, attn_block_rows(rows, c.kv_dtype, c.head_dim), h->kmap, h->vmap, s) == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}

rssm_status rssm_attn_get_error(rssm_attn* h, int32_t* err4, void* stream) {
    if (h == nullptr || err4 == nullptr) return RSSM_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    void* dev = h->base + h->lay.err;
    int32_t word[5];
    cudaError_t e = cudaMemcpyAsync(word, dev, sizeof(word), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess) {
        std::memcpy(err4, word, 16);
        // a call that gave up has not counted all its parts: the counters too go back to zero
        e = cudaMemsetAsync(dev, 0, word[4] != 0 ? h->lay.part_ml : sizeof(word), s);
    }
    return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}

rssm_status rssm_attn_destroy(rssm_attn* h) {
    if (h == nullptr) return RSSM_ERR_INVALID_ARG;
    delete h;
    return RSSM_OK;
}

}  // extern "C"
