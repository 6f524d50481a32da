// Attention over a 4-bit (NVFP4) cache: the layout of the cache, and the products of
// one warp. The split over blocks, the ring and the joins are attn_decode.cuh's.
//
// The layout. Sixteen tokens of one cache head (a group) are 9 D bytes in one piece,
// 8 D of codes and D of block scales, ordered so that each lane of a warp finds the
// codes of its matrix fragments side by side, and a warp's loads fill whole rows of
// banks. Of token t = 0..15 of the group and block b = 0..D/16 - 1 (16 channels, two
// codes a byte, the even channel in the low half):
//   K  codes at 8 b + (D/2) t (heads of 256: the upper and lower 64 bytes of odd tokens
//      exchanged); the scale at 8 D + (t%8) D/8 + (b/2%4) D/32 + (t/8) D/64 + (b%2) + 2 (b/8),
//      heads of 64: 8 D + (t%8) 8 + 2 b + t/8.
//   V  codes at 4 D (t/8) + 64 b + 8 (t%8), heads of 64: 4 D (t/8) + 64 b + 4 (t%8), the
//      second half of the block 32 further on, a byte's two codes exchanged for odd t; the
//      scale at 8 D + 16 b + 4 (t%8/2) + 2 (t/8) + t%2.
//
// The products. Scores are made as K Q^T and outputs as V^T P^T, 16 tokens or 16
// channels by 8 query rows: with few rows (8 or less is the common case) the matrix
// instructions and the softmax then cost half of what 16 rows cost. The codes widen to
// FP16 (cvt), and their block scales multiply them there, exactly: 2 by 4 significant
// bits, between 2^-10 and 2688. Q and the weights are FP16, scaled as for FP8 caches.
//
// What bounds it. A group of 16 tokens of 128 channels takes 98 cycles of an SM at the
// bandwidth of a copy; its 512 words of codes take 51 at the rate measured for a conversion
// and a multiplication a pair (10 words of 8 codes a cycle), and in all a warp issues 260
// instructions for it, 65 cycles if the SM never waited. Neither bound is reached (80 % of
// the bandwidth, 55 % of the issue slots): three warps a scheduler do not cover each
// other's waits for fixed latencies and for shared memory. So what a widened fragment costs beside its
// conversion is kept low: the interleaving of two tokens' V codes is two instructions for
// 16 codes, a lane's channels of V all belong to one block, so that a pair of scales
// serves 16 fragments, and the running maximum is looked at by a vote. Small blocks of two
// consumer warps and a producer, four an SM at 168 registers, do best: more warps at 128
// registers lose their interleaving, and fewer producers refill too late.
//
// Measured: 8 requests of 128k, 1.07 GB: 199 us, 5.4 TB/s; 256 ragged requests, 1.33 GB:
// 265 us, 5.0 TB/s; 4 drafts of 8 heads of 256, 64 requests: 141 us; windows of 1000 over
// 16 heads of 64, 128 requests: 67 us; one request of 777 tokens: 11 us. 64 requests of 4096
// tokens over 4 heads of 128: 42 us for 8 rows, 68 for 16, whose 64 outputs and 32 queries
// a thread do not fit 168 registers (340 bytes of spills; 32 and 64 rows, and heads of
// 256 at 32: 92 to 116), 97 for 32.
#pragma once

#include "attn_decode.cuh"

namespace rssm {

// Bytes from a group's start to the codes (8 bytes; heads of 64, V: 4 and 4, 32 apart)
// and to the scale of block b of token t.
template <bool V>
__host__ __device__ __forceinline__ int nvfp4_codes_at(int D, int t, int b) {
    if (V) return 4 * D * (t >> 3) + 64 * b + (D == 64 ? 4 : 8) * (t & 7);
    return (D / 2) * t + ((8 * b) ^ (D == 256 ? (t & 1) << 6 : 0));
}
template <bool V>
__host__ __device__ __forceinline__ int nvfp4_scale_at(int D, int t, int b) {
    if (V) return 8 * D + 16 * b + 4 * ((t & 7) >> 1) + 2 * (t >> 3) + (t & 1);
    if (D == 64) return 8 * D + 8 * (t & 7) + 2 * b + (t >> 3);
    return 8 * D + (t & 7) * (D / 8) + ((b >> 1) & 3) * (D / 32) + (t >> 3) * (D / 64) + (b & 1) + 2 * (b >> 3);
}

// A token's V codes as they are stored, and back.
__device__ __forceinline__ uint32_t nvfp4_exchanged(uint32_t c, int t) {
    return (t & 1) ? ((c & 0x0F0F0F0Fu) << 4) | ((c >> 4) & 0x0F0F0F0Fu) : c;
}

namespace attn {

// NR: tiles of 8 query rows that one warp takes. DS: warps that share the channels of a
// slot's tokens. Heads of 256 are shared by two: each makes the scores of its half of
// the channels, they exchange and add them, and each then takes its half of the
// outputs. One warp alone has 64 registers of outputs and 32 of queries for 8 rows,
// and twice that for 16, which spilled.
template <int D_, int NR_, int WM_>
struct Shape4 {
    static constexpr int D = D_, NR = NR_, WM = WM_, DS = D == 256 ? 2 : 1;
    // Consumer warps per row group, and as many blocks an SM as their registers allow. These
    // are shared out per quarter of an SM: 8 warps leave 255 a thread, 12 leave 168 and 16
    // 128, producers included.
    static constexpr int kMinBlocks = attn4_blocks(8 * NR * WM, D);
    static constexpr int NT = D == 256 ? (NR == 1 ? 2 : WM == 1 ? 3 : 2)
                            : D == 128 ? (NR == 1 ? 2 : WM == 4 ? 2 : 5)
                                       : (NR == 1 ? 2 : WM == 4 ? 2 : WM == 2 ? 3 : 5);
    static constexpr int kJoin = 32;
    static constexpr int kWarpRows = 8 * NR;
    // 32 and 64 rows: queries are read from shared memory at each product. In registers, beside
    // the outputs, they leave an SM five to seven warps, and those a third of its issue slots.
    static constexpr bool kQShared = WM > 1 && D >= 128;
    static constexpr int kQueries = NR * (D / DS / 16) * 2 * 32 * 4;           // bytes of a warp's queries
    static constexpr int kSlotScores = 2 * NR * 4 * 32 * 4;   // bytes of a slot's scores, as one warp holds them
    static constexpr int kRows = kWarpRows * WM;
    static constexpr int kConsumers = WM * NT * DS;
    static constexpr int kExchange = DS == 1 ? 0 : WM * NT * 2 * 2 * kSlotScores;   // [pair][turn][half]
    static constexpr int kShared = kExchange + (kQShared ? kConsumers * kQueries : 0);
    static constexpr int kThreads = (kConsumers + 1) * 32;
    static constexpr int kQsz = 2;
    // A slot holds two groups, which a warp takes together.
    static constexpr int kSlotGroups = 2;
    static constexpr int kHalf = (9 * D + 127) / 128 * 128;   // copies begin on 128 bytes
    static constexpr int kSlot = 2 * kSlotGroups * kHalf;
    static constexpr int kCopied = 2 * 9 * D;
    static constexpr int QS = D * kQsz + 16;
    static constexpr int OS = D + 8;
    static constexpr int kBudget = (kMinBlocks == 4 ? 56 : kMinBlocks == 2 ? 113 : 226) * 1024 - 1024;
    static constexpr int fixed_bytes(int nb) {
        return 2 * kRows * QS + nb * kRows * OS * 4 + NT * kRows * 8 + kRows * 8 + 1024 + kShared;
    }
    static constexpr int NB = (kBudget - fixed_bytes(NT)) / kSlot >= 8 ? NT : 1;
    static constexpr int kFixed = fixed_bytes(NB);
    static constexpr int kSlotsFit = (kBudget - kFixed) / kSlot;
    static constexpr int NS = (kSlotsFit > 24 ? 24 : kSlotsFit) / NT * NT;
    static constexpr bool kPair = false;
    static constexpr bool kTogether = D / DS * NR <= 128 || kQShared;     // the scores of a slot's groups, product by product
    static constexpr int PB = 8;
    static constexpr int kSmem = 1024 + NS * kSlot + kFixed;
    static_assert(NS >= NT && NS % NT == 0 && NS >= PB / kSlotGroups, "ring too small");
    static_assert(16 * NS + 32 + 8 + 2 * 48 <= 1024, "barriers and parts");
};

__device__ __forceinline__ uint32_t lds32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
template <int N>
__device__ __forceinline__ void lds(uint32_t (&v)[N], uint32_t at) {
    static_assert(N == 2 || N == 4, "8 or 16 bytes");
    if constexpr (N == 2) asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(at));
    else asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at));
}
// The eight E2M1 codes of a word, a byte's two to one register of two FP16.
__device__ __forceinline__ void widen(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// The 8x8 matrix of 16-bit values of which a lane holds two of row lane/4, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

template <class S>
struct Warp<kNVFP4, S> {
    static constexpr int D = S::D, NR = S::NR;
    static constexpr int kWords = D / S::DS / 32;   // of K codes, per lane and token
    static constexpr int kTiles = D / S::DS / 16;   // of 16 channels, in the order in which V's words hold them
    static constexpr int kLaneRows = 2 * NR;     // row x is 8 (x/2) + 2 c + x%2
    // Weights, and l and o with them, are 2^kUp times as large, and relative to a score
    // that the row's largest may pass by kSlack before all is rescaled: they stay
    // below 2^16. Rescaling at every new maximum took a rescale in two of three steps
    // where 16 rows run over some thousands of tokens. Weights below 2^-26 of that
    // score lose some of FP16's bits, and those below 2^-37 vanish.
    static constexpr float kUp = 12.f, kSlack = 3.f, kOver = kUp;
    float o[NR][kTiles][4];      // of a tile's two channels of this lane: the rows' pair in [0..1] and in [2..3]
    float base[kLaneRows];       // the score, before its multiplier, that weights are relative to; the same in all lanes of a row
    float most[kLaneRows];       // scores up to here need no other; -inf before the first
    float l[kLaneRows];          // this lane's tokens only
    uint32_t qf[S::kQShared ? 1 : NR][2 * kWords][2];
    uint32_t qs = 0;             // or in shared memory, [NR][2 kWords][lane] pairs of words
    float mul[kLaneRows];        // score multiplier, > 0
    int lane, g, c;
    int half = 0, pair = 0, turn = 0;   // of a pair's two warps; the pair; of its two exchange buffers
    char* shared = nullptr;

    // The warp's place in its pair, where the two exchange their scores, and where its
    // queries are.
    __device__ __forceinline__ void settle(int warp, char* buffers) {
        if constexpr (S::DS == 2) {
            half = warp & 1;
            pair = warp >> 1;
            shared = buffers + pair * 4 * S::kSlotScores;
        }
        if constexpr (S::kQShared) qs = smem_u32(buffers + S::kExchange + warp * S::kQueries) + lane * 8;
    }
    // The sum of both warps' scores. A buffer is written again two exchanges later, behind
    // the barrier of the one between them, which the other warp passes after its reads.
    template <int NG>
    __device__ __forceinline__ void exchange(float (&s)[NG][NR][4]) {
        if constexpr (S::DS == 2) {
            float4* mine = reinterpret_cast<float4*>(shared + (2 * turn + half) * S::kSlotScores) + lane;
            const float4* other = reinterpret_cast<const float4*>(shared + (2 * turn + 1 - half) * S::kSlotScores) + lane;
            turn ^= 1;
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int n = 0; n < NR; ++n) mine[(i * NR + n) * 32] = make_float4(s[i][n][0], s[i][n][1], s[i][n][2], s[i][n][3]);
            named_sync(3 + pair, 64);
#pragma unroll
            for (int i = 0; i < NG; ++i)
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    const float4 v = other[(i * NR + n) * 32];
                    s[i][n][0] += v.x, s[i][n][1] += v.y, s[i][n][2] += v.z, s[i][n][3] += v.w;
                }
        }
    }

    __device__ __forceinline__ int row(int x) const { return 8 * (x >> 1) + 2 * c + (x & 1); }
    __device__ __forceinline__ void join_columns(int x) {
#pragma unroll
        for (int d = 4; d < 32; d *= 2) l[x] += __shfl_xor_sync(0xffffffffu, l[x], d);
    }
    __device__ __forceinline__ bool speaks() const { return g == 0; }
    // The maximum under which row x's sums stand: rounded, the same wherever it is taken.
    __device__ __forceinline__ float top(int x) const { return most[x] == -INFINITY ? -INFINITY : __fmul_rn(base[x], mul[x]); }

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < kTiles; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
#pragma unroll
        for (int x = 0; x < kLaneRows; ++x) {
            most[x] = -INFINITY;
            base[x] = 0.f;
            l[x] = 0.f;
        }
    }

    // The lane's channels of a K row: word j holds 8 from here on.
    __device__ __forceinline__ int channel(int j) const { return D == 64 ? 16 * c + 8 * j : 32 * c + 8 * j + 128 * half; }

    // Query rows as the B operand, scaled as for FP8 caches: each by a power of two so
    // that its largest finite value lies in [2^14, 2^15).
    __device__ __forceinline__ void load_q(const char* rows, float scale_log2, float kscale) {
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const char* q = rows + (8 * n + g) * S::QS;
            float mx = 0.f;
#pragma unroll
            for (int j = 0; j < kWords * S::DS; ++j)          // both halves: the row has one factor
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 v = load4(reinterpret_cast<const __nv_bfloat16*>(q) + (channel(j % kWords) ^ (j / kWords * 128)) + 4 * h);
                    for (const float x : {v.x, v.y, v.z, v.w}) mx = fabsf(x) < INFINITY ? fmaxf(mx, fabsf(x)) : mx;
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            int e = static_cast<int>((__float_as_uint(mx) >> 23) & 0xFF) - 127;
            if (e < -126) e = 14;                             // no normal number: as it stands
            const int up = 14 - e, half = up / 2;            // 2^up may pass FP32: two factors
            const float f1 = scale_log2 < 0.f ? -pow2(half) : pow2(half), f2 = pow2(up - half);
            // positive and normal, so that the largest product is the largest score, and -inf stays
            const float mu = fmaxf(fabsf(scale_log2) * kscale * pow2(-half) * pow2(half - up), 1.17549435e-38f);
#pragma unroll
            for (int x = 0; x < 2; ++x) mul[2 * n + x] = __shfl_sync(0xffffffffu, mu, 4 * (2 * c + x));
#pragma unroll
            for (int j = 0; j < kWords; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 v = load4(reinterpret_cast<const __nv_bfloat16*>(q) + channel(j) + 4 * h);
                    const uint32_t q0 = pack_f16(v.x * f1 * f2, v.y * f1 * f2), q1 = pack_f16(v.z * f1 * f2, v.w * f1 * f2);
                    if constexpr (S::kQShared) {
                        asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(qs + ((n * 2 * kWords) + 2 * j + h) * 256), "r"(q0), "r"(q1) : "memory");
                    } else {
                        qf[n][2 * j + h][0] = q0;
                        qf[n][2 * j + h][1] = q1;
                    }
                }
        }
    }

    // K's block scales of tokens g and g + 8, as two FP16 each.
    __device__ __forceinline__ void key_scales(uint32_t k, uint32_t (&s)[2][2]) const {
        const uint32_t at = k + 8 * D + lane * (D / 32);
        if constexpr (D == 64) {
            uint16_t b;
            asm volatile("ld.shared.b16 %0, [%1];" : "=h"(b) : "r"(at));
            const uint32_t h = e4m3x2_to_h2(b);
            s[0][0] = __byte_perm(h, h, 0x1010);
            s[1][0] = __byte_perm(h, h, 0x3232);
        } else {
            uint32_t b[2];
            if constexpr (D == 128) {
                b[0] = lds32(at);
                b[1] = b[0] >> 16;
            } else {
                lds<2>(b, at);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t h = e4m3x2_to_h2(b[t] >> (16 * half));
                s[t][0] = __byte_perm(h, h, 0x1010);
                s[t][1] = __byte_perm(h, h, 0x3232);
            }
        }
    }

    // Scores of 16 tokens a group: s[i][n][..] holds tokens g (0, 1) and g + 8 (2, 3) of
    // group i, rows 8 n + 2 c, +1; before their multiplier.
    template <int NG>
    __device__ __forceinline__ void scores(const uint32_t (&kb)[NG], float (&s)[NG][NR][4]) const {
        uint32_t w[NG][2][kWords], b[NG][2][2];
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            key_scales(kb[i], b[i]);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                lds<kWords>(w[i][t], kb[i] + (g + 8 * t) * (D / 2) + ((4 * kWords * c) ^ (D == 256 ? ((g & 1) ^ half) << 6 : 0)));
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][n][j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            uint32_t q[2][NR][2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    if constexpr (S::kQShared) lds<2>(q[h][n], qs + (n * 2 * kWords + 2 * j + h) * 256);
                    else q[h][n][0] = qf[n][2 * j + h][0], q[h][n][1] = qf[n][2 * j + h][1];
                }
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                uint32_t x[4], y[4];
                widen(w[i][0][j], x);
                widen(w[i][1][j], y);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    x[h] = mul_h2(x[h], b[i][0][j / 2]);
                    y[h] = mul_h2(y[h], b[i][1][j / 2]);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t a[4] = {x[2 * h], y[2 * h], x[2 * h + 1], y[2 * h + 1]};
#pragma unroll
                    for (int n = 0; n < NR; ++n) mma_f16(s[i][n], a, q[h][n][0], q[h][n][1]);
                }
            }
        }
    }

    // Running sum under a maximum; the scores become weights. A row's lanes exchange their
    // maxima, and all is rescaled, only where some lane's score passes what is allowed.
    template <int NG>
    __device__ __forceinline__ void softmax(float (&s)[NG][NR][4]) {
        float mx[kLaneRows];
        bool more = false;
#pragma unroll
        for (int x = 0; x < kLaneRows; ++x) {
            mx[x] = fmaxf(s[0][x >> 1][x & 1], s[0][x >> 1][2 + (x & 1)]);
#pragma unroll
            for (int i = 1; i < NG; ++i) mx[x] = fmaxf(mx[x], fmaxf(s[i][x >> 1][x & 1], s[i][x >> 1][2 + (x & 1)]));
            more = more || mx[x] > most[x];
        }
        if (__any_sync(0xffffffffu, more)) {
#pragma unroll
            for (int x = 0; x < kLaneRows; ++x) {
#pragma unroll
                for (int d = 4; d < 32; d *= 2) mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], d));
                const bool up = mx[x] > most[x];
                const float to = up ? mx[x] : base[x];
                const float f = most[x] == -INFINITY ? 0.f : ex2((base[x] - to) * mul[x]);
                // rounded down: where scores are so large that kSlack is less than the step to the
                // next one, none passes without a rescale. (The quotient's own rounding is
                // worth 2^-24 of kSlack; rounded down too, it took a call: 265 -> 280 us over
                // 256 ragged requests.)
                if (up) most[x] = __fadd_rd(to, kSlack / mul[x]);
                base[x] = to;
                l[x] *= f;
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    o[x >> 1][i][x & 1] *= f;
                    o[x >> 1][i][2 + (x & 1)] *= f;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int x = 2 * n + (j & 1);
                    // the difference first: it is exact near the reference, however large that is
                    s[i][n][j] = ex2(fmaf(s[i][n][j] - base[x], mul[x], kUp));
                    l[x] += s[i][n][j];
                }
    }

    // The weights of 16 tokens as the B operand; [1]: with neighbouring tokens exchanged.
    struct Weights {
        uint32_t b[2][NR][2];
    };
    __device__ __forceinline__ Weights weights(const float (&p)[NR][4]) const {
        Weights w;
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                w.b[0][n][t] = transposed(pack_f16(p[n][2 * t], p[n][2 * t + 1]));
                w.b[1][n][t] = __byte_perm(w.b[0][n][t], 0, 0x1032);
            }
        return w;
    }

    // V as the A operand, tile after tile, through f(tile, a): registers 0 and 1 hold
    // tokens 2 c, +1 of the tile's two channels of this lane, 2 and 3 tokens 2 c + 8, +9.
    // A byte of the interleaved words is one channel of two tokens: even channels of even
    // tokens and (exchanged as they are stored) of odd ones share a nibble's place with
    // each other's, so that one selection interleaves eight codes. Odd channels then come
    // with their tokens exchanged: odd tiles, for the weights' second form.
    template <class F>
    __device__ __forceinline__ void each_value(uint32_t v, F f) const {
        constexpr int kW = D == 64 ? 1 : 2;                  // words of a token's block
        constexpr uint32_t kLow = 0x0F0F0F0Fu;
        {
            uint32_t w[2][2 * kW], s[2][2];
            const uint32_t b = lds32(v + 8 * D + (D == 64 ? (lane >> 3) * 16 + c * 4 : half * 128 + lane * 4));
            s[0][0] = e4m3x2_to_h2(b);
            s[0][1] = e4m3x2_to_h2(b >> 16);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                s[1][h] = __byte_perm(s[0][h], 0, 0x1032);
                lds<2 * kW>(w[h], v + 4 * D * h + 512 * half + lane * (8 * kW));
            }
#pragma unroll
            for (int k = 0; k < kW; ++k) {
                uint32_t r[2][2][4];                             // [odd channels][half][channel of four]
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x = w[h][k], y = w[h][kW + k];     // tokens 2 c and 2 c + 1
                    widen((x & kLow) | (y & ~kLow), r[0][h]);
                    widen((x & ~kLow) | (y & kLow), r[1][h]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        r[0][h][i] = mul_h2(r[0][h][i], s[0][h]);
                        r[1][h][i] = mul_h2(r[1][h][i], s[1][h]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int odd = i & 1, e = 2 * (i >> 1);
                    const uint32_t a[4] = {r[odd][0][e], r[odd][0][e + 1], r[odd][1][e], r[odd][1][e + 1]};
                    f(4 * k + i, a);
                }
            }
        }
    }
    // The lane's channels of tiles i (even) and i + 1: from here on, tile i's first, tile
    // i + 1's first, and their second ones.
    __device__ __forceinline__ int chan(int i) const { return D == 64 ? 8 * g + 2 * i : 16 * (g + 8 * half) + 2 * i; }

    __device__ __forceinline__ void accumulate(uint32_t vb, const Weights& w) {
        each_value(vb, [&](int i, const uint32_t (&a)[4]) {
#pragma unroll
            for (int n = 0; n < NR; ++n) mma_f16(o[n][i], a, w.b[i & 1][n][0], w.b[i & 1][n][1]);
        });
    }

    // NG groups whose tokens all rows see.
    template <int NG>
    __device__ __forceinline__ void step(const uint32_t (&kb)[NG], const uint32_t (&vb)[NG]) {
        float s[NG][NR][4];
        if constexpr (S::kTogether) {
            scores(kb, s);
        } else {
            // one after the other: their codes and scales side by side do not fit the registers
#pragma unroll
            for (int i = 0; i < NG; ++i) scores(*reinterpret_cast<const uint32_t(*)[1]>(&kb[i]), *reinterpret_cast<float(*)[1][NR][4]>(&s[i]));
        }
        exchange(s);
        softmax(s);
#pragma unroll
        for (int i = 0; i < NG; ++i) accumulate(vb[i], weights(s[i]));
    }

    // A register of two tokens' values with the tokens outside [lo, hi] set to zero bits.
    __device__ __forceinline__ uint32_t cut(uint32_t v, int tile, int half, int lo, int hi) const {
        const int t = half * 8 + 2 * c, u = t + (tile & 1);
        const int w = t + 1 - (tile & 1);
        return v & ((u >= lo && u <= hi ? 0x0000FFFFu : 0u) | (w >= lo && w <= hi ? 0xFFFF0000u : 0u));
    }

    // One group of which row x of the lane sees the tokens lo[x]..hi[x] (0..15) and some
    // row of the block any_lo..any_hi, all of them all_lo..all_hi; tok0 is its first
    // token's position.
    __device__ __forceinline__ void step_masked(uint32_t kb, uint32_t vb, const int (&lo)[kLaneRows], const int (&hi)[kLaneRows],
                                                int any_lo, int any_hi, int all_lo, int all_hi, int T, int tok0, int len,
                                                int window, const int (&draft)[kLaneRows]) {
        float s[1][NR][4];
        const uint32_t k1[1] = {kb};
        scores(k1, s);
        exchange(s);
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int x = 2 * n + (j & 1), t = g + 8 * (j >> 1);
                if (t < lo[x] || t > hi[x]) s[0][n][j] = -INFINITY;
            }
        softmax(s);
        const Weights w = weights(s[0]);
        bool bad = false;
        if (T > 1 && (max(any_lo, 0) < all_lo || min(any_hi, kAttnGroup - 1) > all_hi)) {
            // the tokens that some drafts see and others do not: a value is finite unless
            // its block's scale is NaN
            for (int i = lane; i < kAttnGroup * (D / 16); i += 32) {
                const int t = i / (D / 16), b = i % (D / 16);
                if (t < any_lo || t > any_hi || (t >= all_lo && t <= all_hi)) continue;
                uint16_t v;
                asm volatile("{\n\t.reg .b8 x;\n\tld.shared.b8 x, [%1];\n\tcvt.u16.u8 %0, x;\n\t}" : "=h"(v) : "r"(vb + nvfp4_scale_at<true>(D, t, b)));
                bad = bad || (v & 0x7F) == 0x7F;
            }
            bad = __any_sync(0xffffffffu, bad);
        }
        if (!bad) {
            each_value(vb, [&](int i, const uint32_t (&a)[4]) {
                const uint32_t x[4] = {cut(a[0], i, 0, any_lo, any_hi), cut(a[1], i, 0, any_lo, any_hi),
                                       cut(a[2], i, 1, any_lo, any_hi), cut(a[3], i, 1, any_lo, any_hi)};
#pragma unroll
                for (int n = 0; n < NR; ++n) mma_f16(o[n][i], x, w.b[i & 1][n][0], w.b[i & 1][n][1]);
            });
            return;
        }
        // 0 * NaN must not reach a row that does not see the token: draft by draft, with
        // only that draft's tokens in place, into its rows alone
        for (int t = 0; t < T; ++t) {
            const int p = len - T + t;
            const int a0 = window_start(p, window) - tok0, a1 = p - tok0;
            each_value(vb, [&](int i, const uint32_t (&a)[4]) {
                const uint32_t x[4] = {cut(a[0], i, 0, a0, a1), cut(a[1], i, 0, a0, a1), cut(a[2], i, 1, a0, a1), cut(a[3], i, 1, a0, a1)};
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_f16(acc, x, w.b[i & 1][n][0], w.b[i & 1][n][1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (draft[2 * n + (j & 1)] == t) o[n][i][j] += acc[j];
                }
            });
        }
    }

    // The outputs times f[row] to the warp's rows of a buffer, or added to what is there.
    __device__ __forceinline__ int first_row() const { return 0; }
    template <bool kAdd>
    __device__ __forceinline__ void leave(float* to, const float (&f)[kLaneRows]) const {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < kTiles; i += 2) {
                    float4* p = reinterpret_cast<float4*>(to + (8 * n + 2 * c + e) * S::OS + chan(i));
                    const float fx = f[2 * n + e];
                    float4 v = make_float4(o[n][i][e] * fx, o[n][i + 1][e] * fx, o[n][i][2 + e] * fx, o[n][i + 1][2 + e] * fx);
                    if (kAdd) v.x += p->x, v.y += p->y, v.z += p->z, v.w += p->w;
                    *p = v;
                }
    }
};

}  // namespace attn
}  // namespace rssm
