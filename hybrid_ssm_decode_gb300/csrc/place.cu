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
// read once more, from L1.
//
// Bound by HBM for many tokens: 16384 tokens of 40 heads of 128 rotated in 53 us
// (6.4 TB/s), FP32 with a quarter of 256 channels 30 us (6.1 TB/s), 32,750 tokens of 8
// heads to a 4-bit cache in 33 us and back in 33 (5.2 TB/s; instructions, 65 % of the
// issue slots), 12,003 tokens with 32 query heads to an FP8 cache 58 us (4.7 TB/s: as it
// is arranged, 121 registers leave two blocks an SM; BF16 and 4-bit caches, 114 and 112,
// take as long, and FP32 ones, twice the bytes, 100). By latency for few: one token's rotation 2.1 us
// and a step of 256 tokens into the cache 4.1 us from a CUDA graph.
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

enum { kNone = 0, kHalves = 1, kInterleaved = 2 };      // how a head's pairs lie

// The sines of `n` tokens from `first` on. Those of pair i lie at (i % step) * (half / step)
// + i / step of their token, so that threads that take `step` pairs each read side by side.
__device__ __forceinline__ void make_turns(float2* cs, const int32_t* positions, const uint64_t* turns, int64_t first, int n,
                                           int half, int step, float gain) {
    const int rows = half / step;
    for (int i = threadIdx.x; i < n * half; i += kThreads) {
        const int t = i / half, pair = i - t * half, q = pair / step;
        const float2 v = turn_of(positions[first + t], turns[pair]);
        cs[t * half + (pair - q * step) * rows + q] = make_float2(v.x * gain, v.y * gain);
    }
    __syncthreads();
}

// N consecutive elements as they are stored (in words, so that BF16 widens by one
// instruction an element and is rounded two at a time), aligned to their size.
template <class T, int N>
struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Pack {
    static constexpr int kWords = N * sizeof(T) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* p) { *this = *reinterpret_cast<const Pack*>(p); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Pack*>(p) = *this; }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float((i & 1) ? (w[i / 2] & 0xFFFF0000u) : (w[i / 2] << 16));
    }
    __device__ __forceinline__ void set(const float* x) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 4) {
                w[i] = __float_as_uint(x[i]);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
    }
};
template <>
struct Pack<__nv_bfloat16, 1> {
    __nv_bfloat16 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *p; }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *p = v; }
    __device__ __forceinline__ float at(int) const { return __bfloat162float(v); }
    __device__ __forceinline__ void set(const float* x) { v = __float2bfloat16_rn(*x); }
};
template <class T, int N>
__device__ __forceinline__ void store_n(T* p, const float* x) {
    constexpr int kStep = N * sizeof(T) <= 16 ? N : 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < N; i += kStep) {
        Pack<T, kStep> a;
        a.set(x + i);
        a.store(p + i);
    }
}

// u cos - v sin, and with -v in the place of v the other half's v cos + u sin: spelt out,
// so that every kernel rounds alike.
__device__ __forceinline__ float turned(float u, float v, float2 t) { return __fmaf_rn(u, t.x, -__fmul_rn(v, t.y)); }

// Threads that a head of `half` pairs and `beside` channels more takes.
__host__ __device__ __forceinline__ int head_threads(int half, int beside, int vec) {
    return (half + beside / (beside % (2 * vec) == 0 ? 2 : 1)) / vec;
}

// The heads of a tile's tokens, rotated. A thread keeps to VEC pairs of one token (or to
// as many of the channels beside them, which are copied, half as many where they cannot
// be halved), so that their sines stay in
// registers, and goes through the token's heads by twos, the next two's channels under
// way while it turns these; the first are on their way before the sines are made.
template <class T, int VEC, int PAIRS>
struct Rotator {
    const T* x;                              // the thread's channels of the head under way
    T* out;                                  // and of the one before
    const T* x0;
    T* out0;
    int64_t x_stride, out_stride;
    int heads, dim, R, half, per_head;       // per_head: threads of a head
    int work, groups, per_token, part, parts;   // groups of threads; a token's heads in `parts` parts, per_token of them here
    static constexpr int kAhead = 2;
    struct Raw {
        Pack<T, VEC> a, b;
    };
    Raw raw[kAhead];
    int slot, e, h;

    int apart;                               // of a copying thread's two vectors; 0: it has one
    __device__ __forceinline__ bool pairs() const { return e * VEC < half; }
    __device__ __forceinline__ int d0() const { return !pairs() ? R - half + e * VEC : PAIRS == kInterleaved ? 2 * e * VEC : e * VEC; }
    __device__ __forceinline__ int d1() const { return !pairs() ? apart : PAIRS == kInterleaved ? VEC : half; }   // from d0; 0: none

    // x, out: the tile's first token. The block takes part `y` of `ny` of every token's heads.
    __device__ __forceinline__ void start(const T* x_, T* out_, int64_t xs, int64_t os, int heads_, int dim_, int R_, int tile, int n,
                                          int y, int ny) {
        x0 = x_; out0 = out_; x_stride = xs; out_stride = os; heads = heads_; dim = dim_; R = R_; half = R / 2;
        const int beside = static_cast<const void*>(out_) == x_ ? 0 : dim - R;
        per_head = head_threads(half, beside, VEC);
        apart = beside % (2 * VEC) == 0 ? beside / 2 : 0;
        groups = max(1, kThreads / per_head);                // heads of more threads: one after another
        per_token = max(1, groups / tile);
        parts = per_token * ny;
        part = y * per_token;
        slot = threadIdx.x / per_head;                       // 0 for heads of more threads than there are
        e = threadIdx.x - slot * per_head;
        work = slot < groups ? n * per_token : 0;
        begin();
    }
    // The first head of the slot.
    __device__ __forceinline__ void begin() {
        h = heads;
        if (slot >= work) return;
        const int t = slot / per_token;
        h = part + slot - t * per_token;
        x = x0 + t * x_stride + static_cast<int64_t>(h) * dim + d0();
        out = out0 + t * out_stride + static_cast<int64_t>(h) * dim + d0();
        fetch();
    }
    // The heads from h on, as they are stored.
    __device__ __forceinline__ void fetch() {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (h + k * parts < heads) {
                raw[k].a.load(x);
                if (d1()) raw[k].b.load(x + d1());
            }
            x += parts * static_cast<int64_t>(dim);
        }
    }
    __device__ __forceinline__ void put(const Raw& p, const float2 (&cs)[VEC]) const {
        if (!pairs()) {
            p.a.store(out);
            if (apart) p.b.store(out + apart);
            return;
        }
        float r[2 * VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) r[j] = p.a.at(j), r[VEC + j] = p.b.at(j);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            constexpr bool kInter = PAIRS == kInterleaved;
            const float u = r[kInter ? 2 * j : j], v = r[kInter ? 2 * j + 1 : VEC + j];
            r[kInter ? 2 * j : j] = turned(u, v, cs[j]);
            r[kInter ? 2 * j + 1 : VEC + j] = turned(v, -u, cs[j]);
        }
        store_n<T, VEC>(out, r);
        store_n<T, VEC>(out + d1(), r + VEC);
    }
    // After the sines are made.
    __device__ __forceinline__ void run(const float2* cs) {
        const int rows = half / VEC;
        for (;;) {
            if (slot < work) {
                float2 t[VEC];
                const int tok = slot / per_token;
                if (pairs()) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) t[j] = cs[tok * half + j * rows + e];
                }
                while (h < heads) {
                    Raw now[kAhead];
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) now[k] = raw[k];
                    const int first = h;
                    h += kAhead * parts;
                    fetch();
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) {
                        if (first + k * parts < heads) put(now[k], t);
                        out += parts * static_cast<int64_t>(dim);
                    }
                }
            }
            // the next slot; heads of more channels than threads: the next channels first
            if (per_head > kThreads && (e += kThreads) < per_head) {
                begin();
                continue;
            }
            e = per_head > kThreads ? static_cast<int>(threadIdx.x) : e;
            slot += groups;
            if (slot >= work) return;
            begin();
        }
    }
};

struct RotaryArgs {
    const void* x;
    void* out;
    const int32_t* positions;
    const uint64_t* turns;
    int64_t tokens, x_stride, out_stride;
    int heads, dim, rotary_dim, interleaved;
    float gain;
};

template <class T, int VEC, int PAIRS>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, int nt) {
    extern __shared__ float2 cs[];
    after_predecessor();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * nt;
    const int n = static_cast<int>(min(static_cast<int64_t>(nt), a.tokens - first));
    Rotator<T, VEC, PAIRS> r;
    r.start(static_cast<const T*>(a.x) + first * a.x_stride, static_cast<T*>(a.out) + first * a.out_stride, a.x_stride, a.out_stride,
            a.heads, a.dim, a.rotary_dim, nt, n, blockIdx.y, gridDim.y);
    make_turns(cs, a.positions, a.turns, first, n, a.rotary_dim / 2, VEC, a.gain);
    r.run(cs);
}

// 16 channels of a key (or, not rotated, of a value): as stored, with the other halves of
// their pairs, and rotated.
template <class T, int VEC, int PAIRS>
struct Key {
    static constexpr int kSines = PAIRS == kHalves ? 16 : PAIRS == kInterleaved ? 8 : 1;
    Pack<T, VEC> own[16 / VEC], other[PAIRS == kHalves ? 16 / VEC : 1];

    __device__ __forceinline__ void load(const T* row, int d0, int R) {
#pragma unroll
        for (int q = 0; q < 16 / VEC; ++q) own[q].load(row + d0 + q * VEC);
        if constexpr (PAIRS == kHalves) {
            const int half = R / 2;
#pragma unroll
            for (int q = 0; q < 16 / VEC; ++q) {
                const int d = d0 + q * VEC;
                if (d < R) other[q].load(row + (d < half ? d + half : d - half));
            }
        }
    }
    // Sines of the 16 channels from their token's, of which a rotator's step is VEC pairs.
    __device__ __forceinline__ static void sines(float2 (&t)[kSines], const float2* cs, int d0, int R) {
        const int half = R / 2, rows = half / VEC;
        if constexpr (PAIRS == kHalves) {
#pragma unroll
            for (int q = 0; q < 16; q += VEC) {
                const int d = d0 + q, i = d < half ? d : d - half;       // a multiple of VEC
                if (d < R) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        t[q + j] = cs[j * rows + i / VEC];
                        if (d < half) t[q + j].y = -t[q + j].y;          // low halves: u cos - v sin
                    }
                }
            }
        } else if constexpr (PAIRS == kInterleaved) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = d0 / 2 + j;
                if (2 * i < R) t[j] = cs[(i % VEC) * rows + i / VEC];
            }
        }
    }
    __device__ __forceinline__ void rotate(float (&x)[16], const float2 (&t)[kSines], int d0, int R) const {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = own[i / VEC].at(i % VEC);
        if constexpr (PAIRS == kHalves) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                // x cos + y sin, the sine's sign turned for low halves: as turned() rounds it
                const float y = other[i / VEC].at(i % VEC);
                if (d0 + i / VEC * VEC < R) x[i] = __fmaf_rn(x[i], t[i].x, __fmul_rn(y, t[i].y));
            }
        } else if constexpr (PAIRS == kInterleaved) {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float u = x[i], v = x[i + 1];
                if (d0 + i >= R) continue;
                x[i] = turned(u, v, t[i / 2]);
                x[i + 1] = turned(v, -u, t[i / 2]);
            }
        }
    }
};

// The larger one, NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A block of 16 as NVFP4 under the head's scale s: its codes and its scale. The products
// and quotients are those of the definition, rounded one by one, so that codes next to
// a border come out as it says. A NaN makes the block's scale NaN, and with it every
// value; infinities are held as the largest value.
__device__ __forceinline__ uint8_t quantise16(const float (&x)[16], float s, uint32_t (&codes)[2]) {
    float m = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) m = max_nan(m, fabsf(x[i]));
    const uint32_t b = e4m3x2(__fmul_rn(m, __frcp_rn(__fmul_rn(6.f, s))), 0.f) & 0xFF;      // NaN: 0x7F
    codes[0] = codes[1] = 0;
    // (1 / (6 s) is infinite for the smallest s, and 0 times it NaN: zeros stay zeros)
    if (b == 0 || b == 0x7F) return static_cast<uint8_t>(m == 0.f ? 0 : b);
    const float inv = fminf(__frcp_rn(__fmul_rn(e4m3_to_f(b), s)), 3.402823466e38f);
#pragma unroll
    for (int i = 0; i < 16; i += 2)
        codes[i / 8] |= e2m1x2(__fmul_rn(x[i], inv), __fmul_rn(x[i + 1], inv)) << (4 * (i % 8));
    return static_cast<uint8_t>(b);
}

// E4M3(x / s) of 16 values, as the rounded quotient gives it. x (1 / s) is within 2.5
// steps of that (5 below a power of two), so the code is the same unless a border between
// codes, a number of five significant bits, lies that near: then, of numbers that are
// not zero or exact one in 30,000, the quotients are taken. Where s is a power of two
// the product is the quotient.
__device__ __forceinline__ void divide16(const float (&x)[16], float s, uint32_t (&c)[4]) {
    const float r = __frcp_rn(s);
    float y[16];
    uint32_t near = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        y[i] = __fmul_rn(x[i], r);
        near = min(near, (__float_as_uint(y[i]) + 8) & 0x7FFFFu);
    }
    const bool plain = s > 1e-30f && s < 1e30f;
    if (!plain || (near <= 16 && (__float_as_uint(s) & 0x7FFFFFu) != 0)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = __fdiv_rn(x[i], s);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = e4m3x2(y[4 * i], y[4 * i + 1]) | (static_cast<uint32_t>(e4m3x2(y[4 * i + 2], y[4 * i + 3])) << 16);
}

// Where a token's 16 channels from d0 = 16 b on lie in a cache.
template <bool V>
__device__ __forceinline__ char* group_of(char* cache, const PlaceArgs& a, int page, int head, int in_page) {
    return cache + page * a.page_stride + static_cast<int64_t>(head * (a.page_size / kAttnGroup) + in_page / kAttnGroup) * (9 * a.dim);
}

// Channels 16 b.. of token `in_page` of a page and head, whose scale is s, into the cache.
template <class T, int KV, bool V>
__device__ __forceinline__ void store_block(const PlaceArgs& a, const float (&x)[16], int page, int head, int in_page, int b, float s) {
    char* cache = V ? a.v_cache : a.k_cache;
    if constexpr (KV == RSSM_KV_NVFP4) {
        char* at = group_of<V>(cache, a, page, head, in_page);
        const int t = in_page % kAttnGroup;
        uint32_t c[2];
        const uint8_t scale = quantise16(x, s, c);
        if (V) c[0] = nvfp4_exchanged(c[0], t), c[1] = nvfp4_exchanged(c[1], t);
        char* to = at + nvfp4_codes_at<V>(a.dim, t, b);
        if (V && a.dim == 64) {
            *reinterpret_cast<uint32_t*>(to) = c[0];
            *reinterpret_cast<uint32_t*>(to + 32) = c[1];
        } else {
            *reinterpret_cast<uint2*>(to) = make_uint2(c[0], c[1]);
        }
        *reinterpret_cast<uint8_t*>(at + nvfp4_scale_at<V>(a.dim, t, b)) = scale;
    } else {
        const int64_t at = (static_cast<int64_t>(head) * a.page_size + in_page) * a.dim + 16 * b;
        if constexpr (KV == RSSM_KV_FP8) {
            uint32_t c[4];
            divide16(x, s, c);
            *reinterpret_cast<uint4*>(cache + page * a.page_stride + at) = make_uint4(c[0], c[1], c[2], c[3]);
        } else {
            store_n<T, 16>(reinterpret_cast<T*>(cache + page * a.page_stride) + at, x);
        }
    }
}

// Channels 16 b.. of a token of the cache: as they are stored, and their values.
template <class T, int KV, bool V>
struct Held {
    static constexpr int kWords = KV == RSSM_KV_NVFP4 ? 2 : KV == RSSM_KV_FP8 ? 4 : 4 * sizeof(T);
    uint32_t w[kWords];
    uint32_t block;              // NVFP4: the block's scale
    float s;                     // the head's

    __device__ __forceinline__ void load(const PlaceArgs& a, int page, int head, int in_page, int b) {
        const char* cache = V ? a.v_cache : a.k_cache;
        if constexpr (KV == RSSM_KV_NVFP4 || KV == RSSM_KV_FP8) s = (V ? a.v_scale : a.k_scale)[head];
        if constexpr (KV == RSSM_KV_NVFP4) {
            const char* at = group_of<V>(const_cast<char*>(cache), a, page, head, in_page);
            const int t = in_page % kAttnGroup;
            const char* from = at + nvfp4_codes_at<V>(a.dim, t, b);
            block = *reinterpret_cast<const uint8_t*>(at + nvfp4_scale_at<V>(a.dim, t, b));
            if (V && a.dim == 64) {
                w[0] = *reinterpret_cast<const uint32_t*>(from);
                w[1] = *reinterpret_cast<const uint32_t*>(from + 32);
            } else {
                const uint2 c = *reinterpret_cast<const uint2*>(from);
                w[0] = c.x, w[1] = c.y;
            }
        } else {
            constexpr int kSize = KV == RSSM_KV_FP8 ? 1 : sizeof(T);
            const uint4* from = reinterpret_cast<const uint4*>(
                cache + page * a.page_stride + ((static_cast<int64_t>(head) * a.page_size + in_page) * a.dim + 16 * b) * kSize);
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 c = from[i];
                w[4 * i] = c.x, w[4 * i + 1] = c.y, w[4 * i + 2] = c.z, w[4 * i + 3] = c.w;
            }
        }
    }
    __device__ __forceinline__ void get(float (&x)[16], int in_page) const {
        if constexpr (KV == RSSM_KV_NVFP4) {
            const float f = __fmul_rn(e4m3_to_f(block), s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t c = V ? nvfp4_exchanged(w[i / 4], in_page) : w[i / 4];
                const float2 v = e2m1x2_to_f2((c >> (8 * (i & 3))) & 0xFF);
                x[2 * i] = __fmul_rn(v.x, f);
                x[2 * i + 1] = __fmul_rn(v.y, f);
            }
        } else if constexpr (KV == RSSM_KV_FP8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 v = e4m3x2_to_f2(static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1))));
                x[2 * i] = __fmul_rn(v.x, s);
                x[2 * i + 1] = __fmul_rn(v.y, s);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                x[i] = __uint_as_float(sizeof(T) == 4 ? w[i * sizeof(T) / 4] : (i & 1) ? (w[i / 2] & 0xFFFF0000u) : (w[i / 2] << 16));
        }
    }
};

// A thread's share of a tile's blocks of 16 channels: one block of one token in every
// `step`-th head. Blocks run fastest, then tokens (four share a sector of V codes), then heads.
struct Share {
    int b, t, head, step;
};
__device__ __forceinline__ Share share_of(const PlaceArgs& a, int nt_log2) {
    const int nb = a.dim / 16, nb_log2 = nb == 4 ? 2 : nb == 8 ? 3 : 4;
    Share s;
    s.b = threadIdx.x & (nb - 1);
    s.t = (threadIdx.x >> nb_log2) & ((1 << nt_log2) - 1);
    const int per = kThreads >> (nb_log2 + nt_log2);
    s.head = threadIdx.x >> (nb_log2 + nt_log2);
    s.step = per;
    return s;
}

// A token's page and place, or false where it is to be skipped (and, `tell`, one past the cache is reported).
__device__ __forceinline__ bool slot_of(const PlaceArgs& a, int64_t tok, bool tell, int& page, int& in_page) {
    const int32_t slot = a.slots[tok];
    if (slot < 0) return false;
    page = slot / a.page_size;
    in_page = slot - page * a.page_size;
    if (page < a.num_pages) return true;
    if (tell) report_error(a.err, RSSM_DEV_ATTN_SLOT, static_cast<int>(tok), slot);
    return false;
}

// A thread's blocks of one token's keys or values, the next head's on its way while this
// one's is written. (Two heads ahead cost occupancy: 32,750 tokens to a 4-bit cache 36
// -> 43 us.)
template <class T, int KV, int VEC, int PAIRS, bool V>
__device__ __forceinline__ void write_heads(const PlaceArgs& a, const T* row, const Share& u, int page, int in_page,
                                            const float2 (&t)[Key<T, VEC, PAIRS>::kSines]) {
    constexpr bool kScaled = KV == RSSM_KV_FP8 || KV == RSSM_KV_NVFP4;
    const float* scales = V ? a.v_scale : a.k_scale;
    const int64_t next = u.step * static_cast<int64_t>(a.dim);
    Key<T, VEC, PAIRS> raw;
    float s = 0.f;
    row += u.head * static_cast<int64_t>(a.dim);
    if (u.head < a.heads) {
        raw.load(row, 16 * u.b, a.rotary_dim);
        if (kScaled) s = scales[u.head];
    }
    for (int h = u.head; h < a.heads; h += u.step) {
        const Key<T, VEC, PAIRS> now = raw;
        const float scale = s;
        row += next;
        if (h + u.step < a.heads) {
            raw.load(row, 16 * u.b, a.rotary_dim);
            if (kScaled) s = scales[h + u.step];
        }
        float x[16];
        now.rotate(x, t, 16 * u.b, a.rotary_dim);
        store_block<T, KV, V>(a, x, page, h, in_page, u.b, scale);
    }
}

// grid.y: 1, and a block takes its tile's queries, keys and values; or one block for the
// keys, one for the values and the others for the queries (none where there are none).
// Without rotation five blocks an SM leave 48 registers: 24 bytes of spills a thread, up to
// 118 where rows do not begin on 16 bytes.
template <class T, int KV, int VEC, int PAIRS>
__global__ void __launch_bounds__(kThreads, PAIRS == kNone ? 5 : 1) place_kernel(const PlaceArgs a, int nt_log2) {
    extern __shared__ float2 cs[];
    after_predecessor();
    const int nt = 1 << nt_log2, half = a.rotary_dim / 2;
    const int64_t first = static_cast<int64_t>(blockIdx.x) << nt_log2;
    const int n = static_cast<int>(min(static_cast<int64_t>(nt), a.tokens - first));
    const bool all = gridDim.y == 1, keys = all || blockIdx.y == 0, values = all || blockIdx.y == 1;
    const Share u = share_of(a, nt_log2);
    int page = 0, in_page = 0;
    bool live = false;
    if (keys || values) live = u.t < n && slot_of(a, first + u.t, keys && u.b == 0 && u.head == 0, page, in_page);
    if constexpr (PAIRS != kNone) {
        Rotator<T, VEC, PAIRS> r;
        const bool queries = a.q != nullptr && (all || blockIdx.y > 1);
        if (queries)
            r.start(static_cast<const T*>(a.q) + first * a.q_stride, static_cast<T*>(a.q_out) + first * a.qo_stride, a.q_stride, a.qo_stride,
                    a.q_heads, a.dim, a.rotary_dim, nt, n, all ? 0 : blockIdx.y - 2, all ? 1 : gridDim.y - 2);
        if (all || !values) make_turns(cs, a.positions, a.turns, first, n, half, VEC, a.gain);
        if (queries) r.run(cs);
    }
    if (!live) return;
    if (keys) {
        float2 t[Key<T, VEC, PAIRS>::kSines];
        Key<T, VEC, PAIRS>::sines(t, cs + u.t * half, 16 * u.b, a.rotary_dim);
        write_heads<T, KV, VEC, PAIRS, false>(a, static_cast<const T*>(a.k) + (first + u.t) * a.k_stride, u, page, in_page, t);
    }
    if (values) {
        const float2 t[1] = {};
        write_heads<T, KV, VEC, kNone, true>(a, static_cast<const T*>(a.v) + (first + u.t) * a.v_stride, u, page, in_page, t);
    }
}

// A thread's blocks of one token, the next head's on its way.
template <class T, int KV, int VEC, bool V>
__device__ __forceinline__ void read_heads(const PlaceArgs& a, int64_t tok, const Share& u, int page, int in_page) {
    T* row = static_cast<T*>(const_cast<void*>(V ? a.v : a.k)) + tok * (V ? a.v_stride : a.k_stride) + 16 * u.b;
    Held<T, KV, V> raw;
    if (u.head < a.heads) raw.load(a, page, u.head, in_page, u.b);
    for (int h = u.head; h < a.heads; h += u.step) {
        const Held<T, KV, V> now = raw;
        if (h + u.step < a.heads) raw.load(a, page, h + u.step, in_page, u.b);
        float x[16];
        now.get(x, in_page);
#pragma unroll
        for (int q = 0; q < 16; q += VEC) store_n<T, VEC>(row + static_cast<int64_t>(h) * a.dim + q, x + q);
    }
}

// grid.y: 0 the keys, 1 the values.
template <class T, int KV, int VEC>
__global__ void __launch_bounds__(kThreads) read_kernel(const PlaceArgs a, int nt_log2) {
    after_predecessor();
    const int64_t first = static_cast<int64_t>(blockIdx.x) << nt_log2;
    const Share u = share_of(a, nt_log2);
    int page, in_page;
    if (first + u.t >= a.tokens || !slot_of(a, first + u.t, blockIdx.y == 0 && u.b == 0 && u.head == 0, page, in_page)) return;
    if (blockIdx.y == 0) read_heads<T, KV, VEC, false>(a, first + u.t, u, page, in_page);
    else read_heads<T, KV, VEC, true>(a, first + u.t, u, page, in_page);
}

// The widest of 16 bytes, 4, 2 and 1 elements by which all of `steps` (strides and channel
// counts, 0 for none) and the pointers, in elements of es bytes, can be taken.
int vec_of(std::initializer_list<int64_t> steps, std::initializer_list<const void*> ptrs, int es) {
    int vec = 16 / es;
    const auto fits = [&] {
        for (const int64_t s : steps)
            if (s % vec != 0) return false;
        for (const void* p : ptrs)
            if (reinterpret_cast<uintptr_t>(p) % (vec * es) != 0) return false;
        return true;
    };
    while (vec > 1 && !fits()) vec /= 2;
    return vec;
}

// Tokens of a block's tile, as a power of two: up to 16, so that what a thread finds out
// about its token and channels serves several heads, while eight blocks an SM are left
// and the sines (half a token) fit 32 KB.
cudaError_t tile_log2(int64_t tokens, int half, int* sms, int* out) {
    int smem = 0;
    const cudaError_t e = device_limits(sms, &smem);
    *out = 0;
    while (*out < 4 && tokens >> (*out + 1) >= 8 * static_cast<int64_t>(*sms) && static_cast<size_t>(half) << (*out + 1) <= 32768 / sizeof(float2)) ++*out;
    return e;
}

// Blocks that share the heads of one token's tile: as many as have a row of threads each
// to work on, while that leaves four blocks an SM at most.
int split(int64_t blocks, int64_t items, int sms) {
    const int64_t per = (items + kThreads - 1) / kThreads, room = (4 * static_cast<int64_t>(sms) + blocks - 1) / blocks;
    return static_cast<int>(per < 1 ? 1 : per < room ? per : room);
}

template <class T, class F>
cudaError_t by_vec(int vec, F f) {
    if constexpr (sizeof(T) == 2)
        if (vec == 8) return f(std::integral_constant<int, 8>{});
    switch (vec) {
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
    const int vec = vec_of({a.k_stride, a.v_stride, a.q ? a.q_stride : 0, a.q ? a.qo_stride : 0, half}, {a.k, a.v, a.q, a.q_out}, es);
    int nt = 0, sms = 0;
    const cudaError_t e = tile_log2(a.tokens, half, &sms, &nt);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (a.tokens + (1 << nt) - 1) >> nt;
    dim3 grid(static_cast<unsigned>(blocks));
    if (nt == 0 && 3 * blocks <= 4 * static_cast<int64_t>(sms)) {
        // few tokens: keys, values and queries in blocks of their own
        const int per_head = rope && a.q ? head_threads(half, a.q_out == a.q ? 0 : a.dim - a.rotary_dim, vec) : 0;
        grid.y = 2 + (per_head ? split(3 * blocks, static_cast<int64_t>(a.q_heads) * per_head, sms) : 0);
    }
    const size_t smem = (static_cast<size_t>(half) << nt) * sizeof(float2);
    return by_cache(a, [&](auto in, auto kv) {
        using T = decltype(in);
        return by_vec<T>(vec, [&](auto v) {
            constexpr int KV = decltype(kv)::value, VEC = decltype(v)::value;
            if (rope && a.interleaved) return launch_overlapped(place_kernel<T, KV, VEC, kInterleaved>, grid, kThreads, smem, s, a, nt);
            if (rope) return launch_overlapped(place_kernel<T, KV, VEC, kHalves>, grid, kThreads, smem, s, a, nt);
            if constexpr (KV == RSSM_KV_NVFP4) return launch_overlapped(place_kernel<T, KV, VEC, kNone>, grid, kThreads, 0, s, a, nt);
            return cudaErrorInvalidValue;                    // the others have a writer of their own (attn.cu)
        });
    });
}

cudaError_t read_launch(const PlaceArgs& a, cudaStream_t s) {
    const int vec = vec_of({a.k_stride, a.v_stride}, {a.k, a.v}, a.in_dtype == RSSM_F32 ? 4 : 2);
    int nt = 0, sms = 0;
    const cudaError_t e = tile_log2(a.tokens, 0, &sms, &nt);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>((a.tokens + (1ll << nt) - 1) >> nt), 2);
    return by_cache(a, [&](auto in, auto kv) {
        using T = decltype(in);
        return by_vec<T>(vec, [&](auto v) {
            return launch_overlapped(read_kernel<T, decltype(kv)::value, decltype(v)::value>, grid, kThreads, 0, s, a, nt);
        });
    });
}

}  // namespace rssm

using namespace rssm;

namespace {

bool is_finite(double x) { return x - x == 0.0; }

template <class T>
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s) {
    const int half = a.rotary_dim / 2, beside = a.out == a.x ? 0 : a.dim - a.rotary_dim;
    const int vec = vec_of({a.heads > 1 ? a.dim : 0, a.tokens > 1 ? a.x_stride : 0, a.tokens > 1 ? a.out_stride : 0, half, beside},
                           {a.x, a.out}, sizeof(T));
    int nt = 0, sms = 0;
    const cudaError_t e = tile_log2(a.tokens, half, &sms, &nt);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (a.tokens + (1 << nt) - 1) >> nt;
    const dim3 grid(static_cast<unsigned>(blocks), nt == 0 ? split(blocks, static_cast<int64_t>(a.heads) * head_threads(half, beside, vec), sms) : 1);
    const size_t smem = (static_cast<size_t>(half) << nt) * sizeof(float2);
    return by_vec<T>(vec, [&](auto v) {
        constexpr int VEC = decltype(v)::value;
        if (a.interleaved) return launch_overlapped(rotary_kernel<T, VEC, kInterleaved>, grid, kThreads, smem, s, a, 1 << nt);
        return launch_overlapped(rotary_kernel<T, VEC, kHalves>, grid, kThreads, smem, s, a, 1 << nt);
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
