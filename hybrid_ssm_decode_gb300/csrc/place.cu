// Rotary positions, and keys and values on their way into and out of a paged cache:
// what stands between an attention layer's projection and its attention.
//
// Rotary positions. Pair i of a head at position p turns by p w_i; for far positions
// that product needs more bits than FP32 or FP64 keep behind the point. Only its
// fraction of a whole turn matters, so w_i / 2 pi is held as a 64-bit fraction and
// the product taken in 64-bit integers, where whole turns drop out by themselves: exact
// to p 2^-64 turns for every 32-bit position, at the cost of one integer product. The
// angle, reduced to an eighth of a turn, then goes through sincospif. A block makes
// the sines of its tokens once, in shared memory, for all their heads.
//
// The cache's writer rotates keys on the way into the cache and queries beside them, so
// that a decode step makes one launch where it made two or three, and neither keys nor
// their rotation pass through memory in between. A thread takes 16 channels of a key or
// a value, one block of an NVFP4 cache; a key's other halves of its pairs are
// read once more, from L1. Bound by HBM for many tokens and by latency for few.
#include <cmath>
#include <initializer_list>
#include <type_traits>

#include "attn.h"
#include "attn_nvfp4.cuh"
#include "overlap.cuh"

namespace rssm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRotary = 1024;    // rotated channels of a head at most

// cos and sin of position p's angle for a frequency of `turn` 2^-64 turns a position.
__device__ __forceinline__ float2 turn_of(int32_t p, uint64_t turn) {
    const uint64_t a = static_cast<uint64_t>(static_cast<int64_t>(p)) * turn + 0x80000000u;
    const uint32_t t = static_cast<uint32_t>(a >> 32);                  // 2^-32 turns
    const uint32_t k = (t + 0x20000000u) >> 30;                         // nearest quarter
    const int32_t rest = static_cast<int32_t>(t - (k << 30));           // an eighth of a turn at most
    float s, c;
    sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
    const float x = (k & 1) ? -s : c, y = (k & 1) ? c : s;
    return (k & 2) ? make_float2(-x, -y) : make_float2(x, y);
}

// The sines of `n` tokens from `first` on, [n][half].
__device__ __forceinline__ void make_turns(float2* cs, const int32_t* positions, const uint64_t* turns, int64_t first, int n,
                                           int half, float gain) {
    for (int i = threadIdx.x; i < n * half; i += kThreads) {
        const int t = i / half;
        const float2 v = turn_of(positions[first + t], turns[i - t * half]);
        cs[i] = make_float2(v.x * gain, v.y * gain);
    }
    __syncthreads();
}

// N consecutive elements, aligned to their size or 16 bytes.
template <class T, int N>
struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Pack {
    T v[N];
};
template <class T, int N>
__device__ __forceinline__ void load_n(float* x, const T* p) {
    const Pack<T, N> a = *reinterpret_cast<const Pack<T, N>*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f(a.v[i]);
}
template <class T, int N>
__device__ __forceinline__ void store_n(T* p, const float* x) {
    Pack<T, N> a;
#pragma unroll
    for (int i = 0; i < N; ++i) a.v[i] = from_f<T>(x[i]);
    *reinterpret_cast<Pack<T, N>*>(p) = a;
}

// u cos - v sin, and with -v in the place of v the other half's v cos + u sin: spelt out,
// so that every kernel rounds alike.
__device__ __forceinline__ float turned(float u, float v, float2 t) { return __fmaf_rn(u, t.x, -__fmul_rn(v, t.y)); }

// Pairs of one head, VEC at a time: item e of R/2/VEC, then copies of what is not rotated.
template <class T, int VEC>
__device__ __forceinline__ void rotate_item(const T* x, T* out, const float2* cs, int e, int R, bool inter) {
    const int half = R / 2;
    const int i = e * VEC;
    if (i >= half) {
        const int d = R + (i - half);
        *reinterpret_cast<Pack<T, VEC>*>(out + d) = *reinterpret_cast<const Pack<T, VEC>*>(x + d);
        return;
    }
    float a[2 * VEC];
    const int d0 = inter ? 2 * i : i, d1 = inter ? 2 * i + VEC : half + i;
    load_n<T, VEC>(a, x + d0);
    load_n<T, VEC>(a + VEC, x + d1);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const float2 t = cs[i + j];
        float& u = inter ? a[2 * j] : a[j];
        float& v = inter ? a[2 * j + 1] : a[VEC + j];
        const float y = turned(u, v, t), z = turned(v, -u, t);
        u = y;
        v = z;
    }
    store_n<T, VEC>(out + d0, a);
    store_n<T, VEC>(out + d1, a + VEC);
}

struct RotaryArgs {
    const void* x;
    void* out;
    const int32_t* positions;
    const uint64_t* turns;
    int64_t tokens, x_stride, out_stride;
    int heads, dim, rotary_dim, interleaved;
    float gain;
};

template <class T, int VEC>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, int nt) {
    extern __shared__ float2 cs[];
    after_predecessor();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * nt;
    const int n = static_cast<int>(min(static_cast<int64_t>(nt), a.tokens - first)), half = a.rotary_dim / 2;
    make_turns(cs, a.positions, a.turns, first, n, half, a.gain);
    const uint32_t per_head = (half + (a.out == a.x ? 0 : a.dim - a.rotary_dim)) / VEC, per_token = a.heads * per_head;
    for (uint32_t i = blockIdx.y * kThreads + threadIdx.x; i < n * per_token; i += gridDim.y * kThreads) {
        const uint32_t t = i / per_token, r = i - t * per_token, h = r / per_head;
        const T* x = static_cast<const T*>(a.x) + (first + t) * a.x_stride + static_cast<int64_t>(h) * a.dim;
        T* out = static_cast<T*>(a.out) + (first + t) * a.out_stride + static_cast<int64_t>(h) * a.dim;
        rotate_item<T, VEC>(x, out, cs + t * half, r - h * per_head, a.rotary_dim, a.interleaved != 0);
    }
}

// Channels d0..d0 + 15 of a row, rotated.
template <class T, int VEC, bool ROPE>
__device__ __forceinline__ void load_block(float (&x)[16], const T* row, int d0, const float2* cs, int R, bool inter) {
#pragma unroll
    for (int q = 0; q < 16; q += VEC) load_n<T, VEC>(x + q, row + d0 + q);
    if (!ROPE) return;
    const int half = R / 2;
#pragma unroll
    for (int q = 0; q < 16; q += VEC) {
        const int d = d0 + q;
        if (d >= R) continue;
        if (!inter) {
            // the other halves of the pairs
            const bool low = d < half;
            float y[VEC];
            load_n<T, VEC>(y, row + (low ? d + half : d - half));
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float2 t = cs[(low ? d : d - half) + j];
                x[q + j] = turned(x[q + j], low ? y[j] : -y[j], t);
            }
        } else if constexpr (VEC > 1) {
#pragma unroll
            for (int j = 0; j < VEC; j += 2) {
                const float2 t = cs[(d + j) / 2];
                const float u = x[q + j], v = x[q + j + 1];
                x[q + j] = turned(u, v, t);
                x[q + j + 1] = turned(v, -u, t);
            }
        } else {
            if (q & 1) continue;                             // d0 is even: q, q + 1 are a pair
            const float2 t = cs[d / 2];
            const float u = x[q], v = x[q + 1];
            x[q] = turned(u, v, t);
            x[q + 1] = turned(v, -u, t);
        }
    }
}

__device__ __forceinline__ bool any_nan(const float (&x)[16]) {
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) nan = nan || x[i] != x[i];
    return nan;
}

// A block of 16 as NVFP4 under the head's scale s: its codes and its scale. The products
// and quotients are those of the definition, rounded one by one, so that codes next to
// a border come out as it says. A NaN makes the block's scale NaN, and with it every
// value; infinities are held as the largest value.
__device__ __forceinline__ uint8_t quantise16(const float (&x)[16], float s, uint32_t (&codes)[2]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(x[i]));
    const uint32_t b = e4m3x2(__fmul_rn(m, __fdiv_rn(1.f, __fmul_rn(6.f, s))), 0.f) & 0xFF;
    const float inv = b == 0 ? 0.f : fminf(__fdiv_rn(1.f, __fmul_rn(e4m3_to_f(b), s)), 3.402823466e38f);
    codes[0] = codes[1] = 0;
    if (any_nan(x)) return 0x7F;
    if (b == 0) return 0;
#pragma unroll
    for (int i = 0; i < 16; i += 2)
        codes[i / 8] |= e2m1x2(__fmul_rn(x[i], inv), __fmul_rn(x[i + 1], inv)) << (4 * (i % 8));
    return static_cast<uint8_t>(b);
}

// Where a token's 16 channels from d0 = 16 b on lie in a cache.
template <bool V>
__device__ __forceinline__ char* group_of(char* cache, const PlaceArgs& a, int page, int head, int in_page) {
    return cache + page * a.page_stride + static_cast<int64_t>(head * (a.page_size / kAttnGroup) + in_page / kAttnGroup) * (9 * a.dim);
}

// Channels 16 b.. of token `in_page` of a page and head into the cache.
template <class T, int KV, bool V>
__device__ __forceinline__ void store_block(const PlaceArgs& a, const float (&x)[16], int page, int head, int in_page, int b) {
    char* cache = V ? a.v_cache : a.k_cache;
    const float* scales = V ? a.v_scale : a.k_scale;
    if constexpr (KV == RSSM_KV_NVFP4) {
        char* at = group_of<V>(cache, a, page, head, in_page);
        const int t = in_page % kAttnGroup;
        uint32_t c[2];
        const uint8_t s = quantise16(x, scales[head], c);
        char* to = at + nvfp4_codes_at<V>(a.dim, t, b);
        if (V && a.dim == 64) {
            *reinterpret_cast<uint32_t*>(to) = c[0];
            *reinterpret_cast<uint32_t*>(to + 32) = c[1];
        } else {
            *reinterpret_cast<uint2*>(to) = make_uint2(c[0], c[1]);
        }
        *reinterpret_cast<uint8_t*>(at + nvfp4_scale_at<V>(a.dim, t, b)) = s;
    } else {
        const int64_t at = (static_cast<int64_t>(head) * a.page_size + in_page) * a.dim + 16 * b;
        if constexpr (KV == RSSM_KV_FP8) {
            const float s = scales[head];
            uint32_t c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c[i] = e4m3x2(__fdiv_rn(x[4 * i], s), __fdiv_rn(x[4 * i + 1], s)) |
                       (static_cast<uint32_t>(e4m3x2(__fdiv_rn(x[4 * i + 2], s), __fdiv_rn(x[4 * i + 3], s))) << 16);
            *reinterpret_cast<uint4*>(cache + page * a.page_stride + at) = make_uint4(c[0], c[1], c[2], c[3]);
        } else {
            store_n<T, 16>(reinterpret_cast<T*>(cache + page * a.page_stride) + at, x);
        }
    }
}

// Channels 16 b.. of a token from the cache.
template <class T, int KV, bool V>
__device__ __forceinline__ void fetch_block(const PlaceArgs& a, float (&x)[16], int page, int head, int in_page, int b) {
    char* cache = V ? a.v_cache : a.k_cache;
    const float* scales = V ? a.v_scale : a.k_scale;
    if constexpr (KV == RSSM_KV_NVFP4) {
        const char* at = group_of<V>(cache, a, page, head, in_page);
        const int t = in_page % kAttnGroup;
        const char* from = at + nvfp4_codes_at<V>(a.dim, t, b);
        uint2 c;
        if (V && a.dim == 64) {
            c.x = *reinterpret_cast<const uint32_t*>(from);
            c.y = *reinterpret_cast<const uint32_t*>(from + 32);
        } else {
            c = *reinterpret_cast<const uint2*>(from);
        }
        const float s = __fmul_rn(e4m3_to_f(*reinterpret_cast<const uint8_t*>(at + nvfp4_scale_at<V>(a.dim, t, b))), scales[head]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = e2m1x2_to_f2(((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xFF);
            x[2 * i] = __fmul_rn(v.x, s);
            x[2 * i + 1] = __fmul_rn(v.y, s);
        }
    } else {
        const int64_t at = (static_cast<int64_t>(head) * a.page_size + in_page) * a.dim + 16 * b;
        if constexpr (KV == RSSM_KV_FP8) {
            const float s = scales[head];
            const uint4 c = *reinterpret_cast<const uint4*>(cache + page * a.page_stride + at);
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 v = e4m3x2_to_f2(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))));
                x[2 * i] = __fmul_rn(v.x, s);
                x[2 * i + 1] = __fmul_rn(v.y, s);
            }
        } else {
            load_n<T, 16>(x, reinterpret_cast<const T*>(cache + page * a.page_stride) + at);
        }
    }
}

// Unit i of a tile's blocks of keys and values. Blocks run fastest, then up to four
// tokens, whose V codes share a sector, then heads (keys before values), then fours
// of tokens.
struct Unit {
    int t, head, b;
    bool v;
};
__device__ __forceinline__ Unit unit_of(uint32_t i, const PlaceArgs& a, int tq_log2) {
    const uint32_t nb = a.dim / 16;
    Unit u;
    u.b = i & (nb - 1);
    i /= nb;
    const uint32_t t = i & ((1u << tq_log2) - 1);
    i >>= tq_log2;
    const uint32_t heads = 2 * a.heads, four = i / heads, h = i - four * heads;
    u.t = static_cast<int>((four << tq_log2) + t);
    u.v = h >= static_cast<uint32_t>(a.heads);
    u.head = static_cast<int>(u.v ? h - a.heads : h);
    return u;
}

// A slot's page and place, or false where it is to be skipped (and one past the cache is reported).
__device__ __forceinline__ bool slot_of(const PlaceArgs& a, int64_t tok, const Unit& u, int& page, int& in_page) {
    const int32_t slot = a.slots[tok];
    if (slot < 0) return false;
    page = slot / a.page_size;
    in_page = slot - page * a.page_size;
    if (page < a.num_pages) return true;
    if (u.b == 0 && u.head == 0 && !u.v) report_error(a.err, RSSM_DEV_ATTN_SLOT, static_cast<int>(tok), slot);
    return false;
}

template <class T, int KV, int VEC, bool ROPE>
__global__ void __launch_bounds__(kThreads) place_kernel(const PlaceArgs a, int nt, int tq_log2) {
    extern __shared__ float2 cs[];
    after_predecessor();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * nt;
    const int n = static_cast<int>(min(static_cast<int64_t>(nt), a.tokens - first)), half = a.rotary_dim / 2;
    const bool inter = ROPE && a.interleaved != 0;
    uint32_t nq = 0, per_head = 1, per_token = 1;
    if (ROPE) {
        make_turns(cs, a.positions, a.turns, first, n, half, a.gain);
        if (a.q != nullptr) {
            per_head = (half + (a.q_out == a.q ? 0 : a.dim - a.rotary_dim)) / VEC;
            per_token = a.q_heads * per_head;
            nq = n * per_token;
        }
    }
    const uint32_t units = static_cast<uint32_t>(nt) * 2 * a.heads * (a.dim / 16);
    for (uint32_t i = blockIdx.y * kThreads + threadIdx.x; i < nq + units; i += gridDim.y * kThreads) {
        if (ROPE && i < nq) {
            const uint32_t t = i / per_token, r = i - t * per_token, h = r / per_head;
            const T* x = static_cast<const T*>(a.q) + (first + t) * a.q_stride + static_cast<int64_t>(h) * a.dim;
            T* out = static_cast<T*>(a.q_out) + (first + t) * a.qo_stride + static_cast<int64_t>(h) * a.dim;
            rotate_item<T, VEC>(x, out, cs + t * half, r - h * per_head, a.rotary_dim, inter);
            continue;
        }
        const Unit u = unit_of(i - nq, a, tq_log2);
        int page, in_page;
        if (u.t >= n || !slot_of(a, first + u.t, u, page, in_page)) continue;
        float x[16];
        if (u.v) {
            load_block<T, VEC, false>(x, static_cast<const T*>(a.v) + (first + u.t) * a.v_stride + static_cast<int64_t>(u.head) * a.dim,
                                      16 * u.b, cs, 0, false);
            store_block<T, KV, true>(a, x, page, u.head, in_page, u.b);
        } else {
            load_block<T, VEC, ROPE>(x, static_cast<const T*>(a.k) + (first + u.t) * a.k_stride + static_cast<int64_t>(u.head) * a.dim,
                                     16 * u.b, cs + u.t * half, a.rotary_dim, inter);
            store_block<T, KV, false>(a, x, page, u.head, in_page, u.b);
        }
    }
}

template <class T, int KV, int VEC>
__global__ void __launch_bounds__(kThreads) read_kernel(const PlaceArgs a, int nt, int tq_log2) {
    after_predecessor();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * nt;
    const int n = static_cast<int>(min(static_cast<int64_t>(nt), a.tokens - first));
    const uint32_t units = static_cast<uint32_t>(nt) * 2 * a.heads * (a.dim / 16);
    for (uint32_t i = blockIdx.y * kThreads + threadIdx.x; i < units; i += gridDim.y * kThreads) {
        const Unit u = unit_of(i, a, tq_log2);
        int page, in_page;
        if (u.t >= n || !slot_of(a, first + u.t, u, page, in_page)) continue;
        float x[16];
        if (u.v) fetch_block<T, KV, true>(a, x, page, u.head, in_page, u.b);
        else fetch_block<T, KV, false>(a, x, page, u.head, in_page, u.b);
        T* out = static_cast<T*>(const_cast<void*>(u.v ? a.v : a.k)) + (first + u.t) * (u.v ? a.v_stride : a.k_stride) +
                 static_cast<int64_t>(u.head) * a.dim + 16 * u.b;
#pragma unroll
        for (int q = 0; q < 16; q += VEC) store_n<T, VEC>(out + q, x + q);
    }
}

// The widest of 8, 4, 2 and 1 elements by which all of `steps` (strides and channel counts,
// 0 for none) and the pointers, in elements of es bytes, can be taken.
int vec_of(std::initializer_list<int64_t> steps, std::initializer_list<const void*> ptrs, int es) {
    int vec = 8;
    const auto fits = [&] {
        for (const int64_t s : steps)
            if (s % vec != 0) return false;
        const uintptr_t bytes = vec * es < 16 ? vec * es : 16;
        for (const void* p : ptrs)
            if (reinterpret_cast<uintptr_t>(p) % bytes != 0) return false;
        return true;
    };
    while (vec > 1 && !fits()) vec /= 2;
    return vec;
}

struct Tiling {
    int nt, tq_log2;
    dim3 grid;
};

// Tokens of a block's tile: four, whose sines 256 threads make at once for 128 rotated
// channels, where that still leaves four blocks an SM; else one, with its units spread
// over several blocks while those are few.
cudaError_t tiling(int64_t tokens, int64_t units_per_token, Tiling* t) {
    int sms = 0, smem = 0;
    const cudaError_t e = device_limits(&sms, &smem);
    if (e != cudaSuccess) return e;
    t->nt = tokens >= 16 * static_cast<int64_t>(sms) ? 4 : 1;
    t->tq_log2 = t->nt == 4 ? 2 : 0;
    const int64_t blocks = (tokens + t->nt - 1) / t->nt, per = (units_per_token * t->nt + kThreads - 1) / kThreads;
    const int64_t room = (4 * static_cast<int64_t>(sms) + blocks - 1) / blocks;
    t->grid = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(per < room ? per : room));
    return cudaSuccess;
}

template <class F>
cudaError_t by_vec(int vec, F f) {
    switch (vec) {
        case 8: return f(std::integral_constant<int, 8>{});
        case 4: return f(std::integral_constant<int, 4>{});
        case 2: return f(std::integral_constant<int, 2>{});
        default: return f(std::integral_constant<int, 1>{});
    }
}

// Calls f with the input type and the cache type, as types.
template <class F>
cudaError_t by_cache(const PlaceArgs& a, F f) {
    switch (a.kv_dtype) {
        case RSSM_F32: return f(float{}, std::integral_constant<int, RSSM_F32>{});
        case RSSM_BF16: return f(__nv_bfloat16{}, std::integral_constant<int, RSSM_BF16>{});
        case RSSM_KV_FP8: return f(__nv_bfloat16{}, std::integral_constant<int, RSSM_KV_FP8>{});
        default: return f(__nv_bfloat16{}, std::integral_constant<int, RSSM_KV_NVFP4>{});
    }
}

}  // namespace

cudaError_t place_launch(const PlaceArgs& a, cudaStream_t s) {
    const int es = a.in_dtype == RSSM_F32 ? 4 : 2, half = a.rotary_dim / 2;
    const bool rope = a.positions != nullptr;
    // a vector lies in one half of the rotated channels, or beside them
    const int vec = vec_of({a.k_stride, a.v_stride, a.q ? a.q_stride : 0, a.q ? a.qo_stride : 0, a.interleaved ? 0 : half, a.rotary_dim / (a.interleaved ? 2 : 1)},
                           {a.k, a.v, a.q, a.q_out}, es);
    Tiling t;
    const int64_t q_units = rope && a.q ? static_cast<int64_t>(a.q_heads) * ((half + a.dim - a.rotary_dim) / vec) : 0;
    const cudaError_t e = tiling(a.tokens, q_units + 2 * static_cast<int64_t>(a.heads) * (a.dim / 16), &t);
    if (e != cudaSuccess) return e;
    const size_t smem = static_cast<size_t>(t.nt) * half * sizeof(float2);
    return by_cache(a, [&](auto in, auto kv) {
        return by_vec(vec, [&](auto v) {
            using T = decltype(in);
            if (rope) return launch_overlapped(place_kernel<T, decltype(kv)::value, decltype(v)::value, true>, t.grid, kThreads, smem, s, a, t.nt, t.tq_log2);
            return launch_overlapped(place_kernel<T, decltype(kv)::value, decltype(v)::value, false>, t.grid, kThreads, 0, s, a, t.nt, t.tq_log2);
        });
    });
}

cudaError_t read_launch(const PlaceArgs& a, cudaStream_t s) {
    const int vec = vec_of({a.k_stride, a.v_stride}, {a.k, a.v}, a.in_dtype == RSSM_F32 ? 4 : 2);
    Tiling t;
    const cudaError_t e = tiling(a.tokens, 2 * static_cast<int64_t>(a.heads) * (a.dim / 16), &t);
    if (e != cudaSuccess) return e;
    return by_cache(a, [&](auto in, auto kv) {
        return by_vec(vec, [&](auto v) {
            return launch_overlapped(read_kernel<decltype(in), decltype(kv)::value, decltype(v)::value>, t.grid, kThreads, 0, s, a, t.nt, t.tq_log2);
        });
    });
}

}  // namespace rssm

using namespace rssm;

namespace {

bool is_finite(double x) { return x - x == 0.0; }

template <class T>
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s) {
    const int half = a.rotary_dim / 2;
    const int vec = vec_of({a.heads > 1 ? a.dim : 0, a.tokens > 1 ? a.x_stride : 0, a.tokens > 1 ? a.out_stride : 0, half,
                            a.out == a.x ? 0 : a.dim - a.rotary_dim},
                           {a.x, a.out}, sizeof(T));
    Tiling t;
    const int64_t units = static_cast<int64_t>(a.heads) * ((half + (a.out == a.x ? 0 : a.dim - a.rotary_dim)) / vec);
    const cudaError_t e = tiling(a.tokens, units, &t);
    if (e != cudaSuccess) return e;
    return by_vec(vec, [&](auto v) {
        return launch_overlapped(rotary_kernel<T, decltype(v)::value>, t.grid, kThreads, static_cast<size_t>(t.nt) * half * sizeof(float2), s, a, t.nt);
    });
}

}  // namespace

extern "C" {

rssm_status rssm_rope_frequencies(const rssm_rope_config* c, double* freq, float* gain) {
    if (c == nullptr || freq == nullptr || gain == nullptr) return RSSM_ERR_INVALID_ARG;
    if (c->rotary_dim < 2 || c->rotary_dim % 2 != 0 || c->rotary_dim > kMaxRotary) return RSSM_ERR_INVALID_ARG;
    if (c->scaling < RSSM_ROPE_PLAIN || c->scaling > RSSM_ROPE_WAVELENGTH || !(c->base > 1.0) || !is_finite(c->base) || !is_finite(c->gain))
        return RSSM_ERR_INVALID_ARG;
    if (c->scaling != RSSM_ROPE_PLAIN && (!(c->factor > 0.0) || !is_finite(c->factor))) return RSSM_ERR_INVALID_ARG;
    const bool bands = c->scaling == RSSM_ROPE_YARN || c->scaling == RSSM_ROPE_WAVELENGTH;
    const double fast = c->fast != 0.0 ? c->fast : c->scaling == RSSM_ROPE_YARN ? 32.0 : 4.0, slow = c->slow != 0.0 ? c->slow : 1.0;
    if (bands && (!(c->original >= 1.0) || !is_finite(c->original) || !(slow > 0.0) || !(fast > slow) || !is_finite(fast)))
        return RSSM_ERR_INVALID_ARG;
    if (c->scaling == RSSM_ROPE_NTK && c->rotary_dim == 2) return RSSM_ERR_INVALID_ARG;
    constexpr double kTwoPi = 6.283185307179586476925;
    const double R = c->rotary_dim, f = c->factor;
    const double base = c->scaling == RSSM_ROPE_NTK ? c->base * std::pow(f, R / (R - 2.0)) : c->base;
    double lo = 0.0, hi = 0.0;
    if (c->scaling == RSSM_ROPE_YARN) {
        // the channels that turn `fast` and `slow` times over the original positions
        const auto channel = [&](double turns) { return R * std::log(c->original / (turns * kTwoPi)) / (2.0 * std::log(base)); };
        lo = std::fmax(std::floor(channel(fast)), 0.0);
        hi = std::fmin(std::ceil(channel(slow)), R - 1.0);
    }
    for (int i = 0; i < c->rotary_dim / 2; ++i) {
        const double w = std::pow(base, -2.0 * i / R);
        double stretched = 0.0;                              // how much of the channel is scaled
        if (c->scaling == RSSM_ROPE_LINEAR) stretched = 1.0;
        if (c->scaling == RSSM_ROPE_YARN) stretched = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
        if (c->scaling == RSSM_ROPE_WAVELENGTH)
            stretched = 1.0 - std::fmin(std::fmax((c->original * w / kTwoPi - slow) / (fast - slow), 0.0), 1.0);
        freq[i] = stretched == 0.0 ? w : w / f * stretched + w * (1.0 - stretched);
    }
    *gain = static_cast<float>(c->gain != 0.0 ? c->gain : c->scaling == RSSM_ROPE_YARN ? 0.1 * std::log(f) + 1.0 : 1.0);
    return RSSM_OK;
}

rssm_status rssm_rope_turns(int32_t n, const double* freq, uint64_t* turns) {
    if (n < 1 || freq == nullptr || turns == nullptr) return RSSM_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (!is_finite(freq[i])) return RSSM_ERR_INVALID_ARG;
    // freq / 2 pi in two terms, so that all 64 bits behind the point are there
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;      // 1 / 2 pi
    const auto fixed = [](double t) {                        // modulo 1, in 2^-64
        const double whole = std::fabs(t), part = whole - std::floor(whole);      // exact, below 1
        const uint64_t u = static_cast<uint64_t>(std::ldexp(part, 64));
        return t < 0.0 ? 0 - u : u;
    };
    for (int i = 0; i < n; ++i) {
        const double hi = freq[i] * kHi;
        turns[i] = fixed(hi) + fixed(std::fma(freq[i], kHi, -hi) + freq[i] * kLo);
    }
    return RSSM_OK;
}

rssm_status rssm_rotary(const rssm_rotary_config* c, const void* d_x, const int32_t* d_positions, const uint64_t* d_turns,
                        void* d_out, void* stream) {
    if (c == nullptr || c->tokens < 0 || c->tokens > 0x7FFFFFFF || c->heads < 1 || c->dim < 1) return RSSM_ERR_INVALID_ARG;
    if (c->dtype != RSSM_F32 && c->dtype != RSSM_BF16) return RSSM_ERR_INVALID_ARG;
    if (c->rotary_dim < 2 || c->rotary_dim % 2 != 0 || c->rotary_dim > c->dim || c->interleaved < 0 || c->interleaved > 1 ||
        !is_finite(c->gain))
        return RSSM_ERR_INVALID_ARG;
    const int64_t row = static_cast<int64_t>(c->heads) * c->dim;
    if (row > (1 << 24)) return RSSM_ERR_INVALID_ARG;         // a tile's units are counted in 32 bits
    if (c->rotary_dim > kMaxRotary) return RSSM_ERR_UNSUPPORTED;
    RotaryArgs a{};
    a.x_stride = c->x_stride ? c->x_stride : row;
    a.out_stride = c->out_stride ? c->out_stride : row;
    if (a.x_stride < row || a.out_stride < row) return RSSM_ERR_INVALID_ARG;
    if (c->tokens == 0) return RSSM_OK;
    const uintptr_t es = c->dtype == RSSM_F32 ? 4 : 2;
    const auto off = [](const void* p, uintptr_t n) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % n != 0; };
    if (off(d_x, es) || off(d_out, es) || off(d_positions, 4) || off(d_turns, 8) || (d_out == d_x && a.out_stride != a.x_stride))
        return RSSM_ERR_INVALID_ARG;
    a.x = d_x; a.out = d_out; a.positions = d_positions; a.turns = d_turns;
    a.tokens = c->tokens; a.heads = c->heads; a.dim = c->dim; a.rotary_dim = c->rotary_dim;
    a.interleaved = c->interleaved; a.gain = c->gain;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = c->dtype == RSSM_F32 ? launch_rotary<float>(a, s) : launch_rotary<__nv_bfloat16>(a, s);
    return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}

}  // extern "C"
