// Attention of T new tokens a request over a paged cache.
//
// The mathematics. The queries that read one cache head, T drafts times
// q_heads/kv_heads, are the rows of one small matrix Q; the scores of a group of
// 16 cached tokens are Q K^T, and the outputs a running sum. A softmax needs
// one pass over the tokens: with m the running maximum of the scores (in units
// of log2) and l, O the running sums,
//   m' = max(m, max s);  l' = l 2^(m-m') + sum 2^(s-m');  O' = O 2^(m-m') + 2^(s-m') V
// and parts (m, l, O) of one row made apart join by the same rule.
//
// The split. A cached token costs its bytes once and 4 D flops a row, so for up
// to 64 rows the cache's bytes bound it, and the question is only that every SM
// streams all the time, whatever the requests' lengths. The work of the launch is
// laid out as one line of units (request, cache head, 64 tokens) and cut into
// equal shares, one per block. A share may begin and end inside a request; those
// at most two parts go to the workspace, and the last of a request's parts to
// arrive joins them in the order of the tokens (no float atomics: reruns give the
// same bits). More than kJoin parts are joined in two steps, by rounds of kJoin
// neighbours and then the rounds, so that few long requests do not wait for one
// block to read hundreds of parts (FP8, 2 requests of 14k and 24k tokens, 15 rows
// of 64: 46 -> 28 us; BF16, one request of 100k, 8 rows of 128: 81 -> 25 us). SMs do
// not all see the same bandwidth: with equal shares the blocks of a launch end
// within 5 to 14 % of their mean. Small shares taken in turn from the last sixth of
// the line lost more to the joins than they evened out (BF16, 64 requests of 1000
// to 9999 tokens, 32 rows of 256: 194 -> 258 us; FP8, 8 requests of 128k: 318 ->
// 362 us).
//
// Measured, with the append in front (6.77 TB/s is a plain copy): BF16, 256 ragged
// requests, 2.37 GB: 354 us, 6.7 TB/s; FP8, 8 requests of 128k, 1.91 GB: 292 us,
// 6.5 TB/s; one request of 777 tokens: 11 us, latency.
//
// The block. One producer warp walks the shares, looks pages up and copies groups
// of 16 tokens (K and V, one 5-D TMA box each, swizzled so that fragment loads
// meet no bank twice) into a ring of slots; a box never leaves a page, because a
// page is a multiple of 16 tokens. With a part's query rows it leaves a
// description of the part in shared memory, two parts ahead. The consumer warps take groups in turn, each with its
// own running (m, l, O) in registers, so that they meet only at the end of a
// part. Groups whose tokens not all rows see (the request's end, the drafts, the
// window's start) take a masked path: scores by selection, values of unseen
// tokens replaced by zero bits, and where a value that some rows see and others do
// not is not finite, the rows' products are made draft by draft.
//
// Matrix instructions. m16n8k16 on BF16 caches, with 2^(s-m) split into two
// BF16 terms, so that the outputs carry only their own rounding; on FP8 caches the codes
// widen exactly to FP16 (Q scaled per row by a power of two into FP16's range;
// 2^(s-m+15) rounded to FP16's 11 bits, so that only weights below 2^-29 of the largest
// lose some of them and only those below 2^-40 vanish: a long tail under one large
// score counts), and on FP32 caches m16n8k8 on TF32 with both
// operands split in two (three products; what is left out is below 2^-21).
#pragma once

#include "attn.h"
#include "overlap.cuh"

namespace rssm {
namespace attn {

enum { kF32 = 0, kBF16 = 1, kFP8 = 2 };

template <int KV, int D_, int WM_>
struct Shape {
    static constexpr int D = D_;
    static constexpr int WM = WM_;                       // row groups of 16
    // Consumer warps per row group. Registers are shared out per quarter of an
    // SM: nine warps put three on one of them and leave 168 a thread, which
    // heads of 256 do not fit (128 of them are the outputs); up to eight leave 255.
    static constexpr int NT = D == 256 ? (WM == 1 ? 4 : WM == 2 ? 3 : 1) : WM == 4 ? 2 : 4;
    static constexpr int kRows = 16 * WM;
    static constexpr int kConsumers = WM * NT;
    static constexpr int kThreads = (kConsumers + 1) * 32;
    static constexpr int kEsz = KV == kF32 ? 4 : KV == kBF16 ? 2 : 1;
    static constexpr int kQsz = KV == kF32 ? 4 : 2;
    static constexpr int RB = D * kEsz;                  // bytes of a cached token
    static constexpr int CB = RB < 128 ? RB : 128;       // swizzled row
    static constexpr int CH = RB / CB;
    static constexpr int kHalf = kAttnGroup * RB;        // K (or V) of a slot
    static constexpr int kSlot = 2 * kHalf;
    static constexpr int QS = D * kQsz + 16;             // bytes from one query row to the next
    static constexpr int OS = D + 8;                     // floats from one merged row to the next
    // Two blocks per SM where the registers allow it: one block's joins then
    // overlap the other's stream.
    static constexpr int kMinBlocks = (WM == 1 && D <= 128) ? 2 : 1;
    static constexpr int kBudget = (kMinBlocks == 2 ? 113 : 226) * 1024 - 1024;
    // Buffers in which the warps of a row leave their outputs at the end of a
    // part: one each where the ring keeps eight slots beside them, else one that
    // they add to in turn.
    static constexpr int fixed_bytes(int nb) {
        return 2 * kRows * QS + nb * kRows * OS * 4 + NT * kRows * 8 + kRows * 8 + 512;
    }
    static constexpr int NB = (kBudget - fixed_bytes(NT)) / kSlot >= 8 ? NT : 1;
    static constexpr int kFixed = fixed_bytes(NB);
    static constexpr int kSlotsFit = (kBudget - kFixed) / kSlot;
    // A multiple of NT, so that a slot always belongs to the same warp of each
    // row group: a warp then never waits for a turn of a slot before it has seen
    // the turn before, which the parity of the slot's barrier could not tell apart.
    static constexpr int NS = (kSlotsFit > 24 ? 24 : kSlotsFit) / NT * NT;
    // Consumers take two groups at a time: heads of 64, whose products are few
    // beside the softmax. (At 128 the second group's scores cost registers that the
    // loop needs: 392 -> 422 us over 256 BF16 requests of up to 4500 tokens.)
    static constexpr bool kPair = KV != kF32 && D == 64;
    static constexpr int PB = NS >= 16 ? 8 : NS >= 8 ? 4 : NS >= 4 ? 2 : 1;   // groups the producer copies at a time
    // A warp with a pair's first group in hand waits for the one NT further on,
    // which must not be in a batch that waits for the first one's slot.
    static_assert(!kPair || NS - NT >= PB, "a pair of groups must fit the ring");
    static constexpr int kSmem = 1024 + NS * kSlot + kFixed;
    static_assert(NS >= NT && NS % NT == 0, "ring too small");
};

template <int N> struct Int { static constexpr int value = N; };

// ---- instructions -----------------------------------------------------------
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// Two E4M3 codes -> two FP16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
    return h;
}
__device__ __forceinline__ uint32_t tf32(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
// x = hi + lo to 22 bits: hi rounded, so that lo has either sign and cutting it
// off at TF32's bits leaves no bias. Above (1 - 2^-12) 2^128 hi is infinite and lo
// NaN or infinite: scores are then retaken. (The conversion that saturates costs 7 to
// 20 % of a pass.)
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    hi = tf32(x);
    lo = __float_as_uint(x - __uint_as_float(hi)) & 0xFFFFE000u;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int row, int head, int page, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2,%3,%4,%5,%6}], [%7];"
        ::"r"(dst), "l"(map), "r"(0), "r"(row), "r"(0), "r"(head), "r"(page), "r"(smem_u32(bar)) : "memory");
}

// 2^n for n in [-126, 127].
__device__ __forceinline__ float pow2(int n) { return __uint_as_float(static_cast<uint32_t>(n + 127) << 23); }

// Count one arrival; orders the block's writes before it (they are behind a block
// barrier) and the reads that follow the last arrival after it.
__device__ __forceinline__ uint32_t arrive_gpu(uint32_t* n) {
    uint32_t old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(n) : "memory");
    return old;
}

// Whether this arrival is the last, after `others` before it; then the counter is
// back at zero.
__device__ __forceinline__ bool arrive_last(uint32_t* n, int others) {
    if (arrive_gpu(n) != static_cast<uint32_t>(others)) return false;
    *n = 0;
    return true;
}

// Whether `ok` holds for every thread at the named barrier.
__device__ __forceinline__ bool all_of(bool ok, int id, int nthreads) {
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.s32 p, %1, 0;\n\t"
        "barrier.cta.red.and.aligned.pred q, %2, %3, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"(static_cast<int>(ok)), "r"(id), "r"(nthreads) : "memory");
    return r != 0;
}

// Wait for a phase, for at most kWaitLimitNs; false once any warp of the block
// has given up (the block then only runs its loops out).
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* dead, int32_t* err) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*dead) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *dead = 1;
            report_error(err, RSSM_DEV_TIMEOUT, -1, 0);
            err[4] = 1;
            return false;
        }
    }
    return true;
}

// ---- the share of a block ----------------------------------------------------
// Tokens of a request that any draft sees, as groups [g0, g1), and its units.
struct Span {
    int len, g0, g1, units;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b) {
    Span s;
    const int most = a.max_pages * a.page_size;
    const int len = __ldcg(a.lens + b);
    s.len = min(max(len, 0), most);
    const int64_t start = a.window > 0 ? static_cast<int64_t>(s.len) - a.T - a.window + 1 : 0;
    s.g0 = start > 0 ? static_cast<int>(start / kAttnGroup) : 0;
    s.g1 = (s.len + kAttnGroup - 1) / kAttnGroup;
    s.units = max(1, (s.g1 - s.g0 + kAttnUnit - 1) / kAttnUnit);   // an empty request still writes its zeros
    return s;
}

// The first position that a token at position p sees (window 0: from the start).
__device__ __forceinline__ int window_start(int p, int window) { return window > 0 && p >= window ? p - window + 1 : 0; }

// Walks the parts of the block's share; one warp.
struct Cursor {
    int64_t total, w, w1, base;  // units: in all, next, end, before request b
    int grid, b;
    Span sp;
    int pair, u0, u1;            // the current part
    bool fresh;
    bool even, only;             // requests cut evenly; the block's one part is not taken yet
    int first, others;           // then: the block of its request's first part, the parts beside it

    // False for a block without a share.
    __device__ __forceinline__ bool start(const AttnArgs& a, int lane) {
        const int heads = a.kv_heads * a.chunks, per = (a.B + 31) / 32;
        int64_t mine = 0;                     // units of this lane's requests, of one cache head
#pragma unroll 4
        for (int i = 0; i < per; ++i) {
            const int r = lane * per + i;
            if (r < a.B) mine += span_of(a, r).units;
        }
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t n = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += n;
        }
        total = __shfl_sync(0xffffffffu, incl, 31) * heads;
        const int c = blockIdx.x, blocks = gridDim.x;
        even = only = false;
        // Little work for few requests: a share that ends inside one request and begins
        // the next costs a second part, so every request and head is cut into even
        // parts of its own, a block each. (FP32, 4 requests of 8 heads of up to 2047
        // tokens: 18.2 -> 15.7 us; BF16, 4 of up to 4000: 17.6 -> 14.6. With more
        // units a block the parts' unevenness costs more than the second part: 8
        // requests of 128k over 8 heads would take parts of 455 units against 383.)
        if (a.B <= 32 && 2 * a.B * heads <= blocks && total < kEvenUnits * blocks) {
            const int units = static_cast<int>(mine);
            int size = static_cast<int>((total + blocks - 1) / blocks);   // units of a part
            // at most twice that and one: parts <= total / size + requests and heads <= blocks
            int n = (units + size - 1) / size;
            while (__reduce_add_sync(0xffffffffu, n) * heads > blocks) {
                ++size;
                n = (units + size - 1) / size;
            }
            int upto = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            const unsigned has = __ballot_sync(0xffffffffu, n > 0 && (upto - n) * heads <= c);
            const int src = 31 - __clz(has);
            const int parts = __shfl_sync(0xffffffffu, n, src), r = c - __shfl_sync(0xffffffffu, upto - n, src) * heads;
            if (c >= __shfl_sync(0xffffffffu, upto, 31) * heads) return false;
            b = src;
            sp = span_of(a, b);
            pair = r / parts;
            const int i = r - pair * parts;
            first = c - i;
            others = parts - 1;
            u0 = i * size;
            u1 = min(sp.units, u0 + size);
            w = w1 = 0;
            even = only = true;
            return true;
        }
        grid = static_cast<int>(min(static_cast<int64_t>(blocks), total));
        if (c >= grid) return false;
        w = total * c / grid;
        w1 = total * (c + 1) / grid;
        // the lane whose requests hold the first unit, then the request
        const int64_t excl = (incl - mine) * heads;
        const int src = 31 - __clz(__ballot_sync(0xffffffffu, mine > 0 && excl <= w));
        base = __shfl_sync(0xffffffffu, excl, src);
        b = src * per;
        for (int i0 = 0; i0 < per; i0 += 32) {
            const int r = src * per + i0 + lane;
            const int64_t n = (i0 + lane < per && r < a.B) ? static_cast<int64_t>(span_of(a, r).units) * heads : 0;
            int64_t upto = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            const unsigned past = __ballot_sync(0xffffffffu, base + upto > w);
            if (past) {
                const int l = __ffs(past) - 1;
                b = src * per + i0 + l;
                base += __shfl_sync(0xffffffffu, upto - n, l);
                break;
            }
            base += __shfl_sync(0xffffffffu, upto, 31);
        }
        sp = span_of(a, b);
        fresh = true;
        return true;
    }
    // The block whose share holds unit x: the last c with total c / grid <= x.
    __device__ __forceinline__ int owner(int64_t x) const { return static_cast<int>(((x + 1) * grid - 1) / total); }
    // The next part of the share; false at its end. Parts after the first begin
    // with a request's first unit.
    __device__ __forceinline__ bool next(const AttnArgs& a) {
        if (only) {
            only = false;
            return true;
        }
        if (w >= w1) return false;
        if (fresh) {
            const int64_t r = w - base;
            pair = static_cast<int>(r / sp.units);
            u0 = static_cast<int>(r - static_cast<int64_t>(pair) * sp.units);
            fresh = false;
        } else {
            u0 = 0;
            if (++pair == a.kv_heads * a.chunks) {
                pair = 0;
                base += static_cast<int64_t>(sp.units) * a.kv_heads * a.chunks;
                sp = span_of(a, ++b);
            }
        }
        u1 = static_cast<int>(min(static_cast<int64_t>(sp.units), u0 + (w1 - w)));
        w += u1 - u0;
        return true;
    }
    __device__ __forceinline__ int first_group() const { return sp.g0 + u0 * kAttnUnit; }
    __device__ __forceinline__ int end_group() const { return min(sp.g1, sp.g0 + u1 * kAttnUnit); }
};

// A part as the producer describes it to the consumers.
struct Part {
    int b, len, head, row0;      // request, its length, cache head, first query row
    int g0, ng;                  // groups of 16 tokens
    int pair;                    // -1: no more parts
    int first;                   // block of the request's first part
    int others;                  // parts of the request and head beside this one
    int at_start;                // the part begins with the request's first unit
};

// ---- one warp's products -----------------------------------------------------
// The byte of a slot's K or V at (token r, 16-byte chunk c) under the TMA swizzle.
template <class S>
__device__ __forceinline__ uint32_t swz(int r, int c) {
    if (S::CB == 128) return (c >> 3) * (kAttnGroup * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    return r * 64 + (((c & 3) ^ ((r >> 1) & 3)) << 4);
}

template <int KV, class S>
struct Warp {
    static constexpr int D = S::D;
    static constexpr int kQRegs = KV == kF32 ? 1 : D / 16;
    static constexpr int kTiles = D / 8;
    static constexpr float kUp = KV == kFP8 ? 15.f : 0.f;   // weights, and l and o with them, are 2^kUp times as large
    float o[kTiles][4];
    float m[2], l[2];            // rows lane/4 and lane/4 + 8; l is this lane's columns only
    uint32_t qf[kQRegs][4];
    const float* qs;             // FP32: the query rows in shared memory
    float mul[2];                // score multiplier of the two rows
    int lane, g, c;

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }

    // Query rows (16 of them, QS bytes apart) as the A operand.
    __device__ __forceinline__ void load_q(const char* rows, float scale_log2, float kscale) {
        mul[0] = mul[1] = scale_log2;
        if constexpr (KV == kF32) {
            qs = reinterpret_cast<const float*>(rows);
        } else if constexpr (KV == kBF16) {
            const uint32_t at = smem_u32(rows) + (lane & 15) * S::QS + (lane >> 4) * 16;
#pragma unroll
            for (int k = 0; k < kQRegs; ++k) ldsm4(qf[k], at + k * 32);
        } else {
            // columns permuted within 16 so that a lane's four K codes are its
            // own; each row scaled by a power of two so that its largest finite value
            // lies in [2^14, 2^15)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const char* row = rows + (g + 8 * h) * S::QS;
                float mx = 0.f;
#pragma unroll
                for (int k = 0; k < kQRegs; ++k) {
                    const float4 v = load4(reinterpret_cast<const __nv_bfloat16*>(row + k * 32 + c * 8));
                    for (const float x : {v.x, v.y, v.z, v.w}) mx = fabsf(x) < INFINITY ? fmaxf(mx, fabsf(x)) : mx;
                }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                // e with mx in [2^e, 2^(e+1)); rows without a normal number stay as they are
                int e = static_cast<int>((__float_as_uint(mx) >> 23) & 0xFF) - 127;
                if (e < -126) e = 14;
                const int up = 14 - e, half = up / 2;        // 2^up may pass FP32: two factors
                const float f1 = pow2(half), f2 = pow2(up - half);
                mul[h] = scale_log2 * kscale * pow2(-half) * pow2(half - up);
#pragma unroll
                for (int k = 0; k < kQRegs; ++k) {
                    const float4 v = load4(reinterpret_cast<const __nv_bfloat16*>(row + k * 32 + c * 8));
                    qf[k][h] = pack_f16(v.x * f1 * f2, v.y * f1 * f2);
                    qf[k][2 + h] = pack_f16(v.z * f1 * f2, v.w * f1 * f2);
                }
            }
        }
    }

    // Scores of 16 tokens: s[i][..] holds tokens 8 i + 2 c, +1 of rows g and g + 8.
    __device__ __forceinline__ void scores(uint32_t k, float (&s)[2][4]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
        uint32_t b[4];
        if constexpr (KV == kBF16) {
            const int r = (lane & 7) + ((lane >> 4) << 3), ch = (lane >> 3) & 1;
            float s2[2][4] = {};                               // two chains a score: half the latency
#pragma unroll
            for (int i = 0; i < kQRegs; i += 2) {
                uint32_t b2[4];
                ldsm4(b, k + swz<S>(r, 2 * i + ch));
                ldsm4(b2, k + swz<S>(r, 2 * i + 2 + ch));
                mma_bf16(s[0], qf[i], b[0], b[1]);
                mma_bf16(s[1], qf[i], b[2], b[3]);
                mma_bf16(s2[0], qf[i + 1], b2[0], b2[1]);
                mma_bf16(s2[1], qf[i + 1], b2[2], b2[3]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s[0][j] += s2[0][j], s[1][j] += s2[1][j];
        } else if constexpr (KV == kFP8) {
            const int r = lane & 15, ch = lane >> 4;         // tokens 0-7, 8-15 of one chunk, then of the next
            float s2[2][4] = {};
#pragma unroll
            for (int i = 0; i < kQRegs; i += 2) {
                ldsm4(b, k + swz<S>(r, i + ch));
                mma_f16(s[0], qf[i], e4m3x2_to_h2(b[0]), e4m3x2_to_h2(b[0] >> 16));
                mma_f16(s[1], qf[i], e4m3x2_to_h2(b[1]), e4m3x2_to_h2(b[1] >> 16));
                mma_f16(s2[0], qf[i + 1], e4m3x2_to_h2(b[2]), e4m3x2_to_h2(b[2] >> 16));
                mma_f16(s2[1], qf[i + 1], e4m3x2_to_h2(b[3]), e4m3x2_to_h2(b[3] >> 16));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) s[0][j] += s2[0][j], s[1][j] += s2[1][j];
        } else {
            // The tensor cores cut their sums off below FP32's last bit, always
            // towards zero, so chains are kept short: the leading products of 32
            // columns at a time, rounded into s by FP32 adds, and the two small
            // products apart from them.
            const int r = (lane & 7) + ((lane >> 4) << 3), ch = (lane >> 3) & 1;
            float small[2][2][4] = {};
#pragma unroll 1
            for (int i0 = 0; i0 < D / 8; i0 += 4) {
                float lead[2][4] = {};
#pragma unroll
                for (int i = i0; i < i0 + 4; ++i) {
                    uint32_t ah[4], al[4], bh[4], bl[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        split_tf32(qs[(g + 8 * (j & 1)) * (S::QS / 4) + i * 8 + c + 4 * (j >> 1)], ah[j], al[j]);
                    ldsm4(b, k + swz<S>(r, 2 * i + ch));
#pragma unroll
                    for (int j = 0; j < 4; ++j) split_tf32(__uint_as_float(b[j]), bh[j], bl[j]);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        mma_tf32(small[0][j], al, bh[2 * j], bh[2 * j + 1]);
                        mma_tf32(small[1][j], ah, bl[2 * j], bl[2 * j + 1]);
                        mma_tf32(lead[j], ah, bh[2 * j], bh[2 * j + 1]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x) s[j][x] += lead[j][x];
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[j][x] += small[0][j][x] + small[1][j][x];
        }
    }

    // The weights as the A operand: P[x][..] of the tokens' two halves (TF32: of
    // 8 tokens each) or of all 16, with the part that the first rounding left.
    struct Weights {
        uint32_t hi[KV == kF32 ? 2 : 1][4];
        uint32_t lo[KV == kF32 ? 2 : 1][4];
    };
    __device__ __forceinline__ Weights weights(const float (&p)[2][4]) const {
        Weights w;
        if constexpr (KV == kF32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float v[4] = {p[i][0], p[i][2], p[i][1], p[i][3]};
#pragma unroll
                for (int j = 0; j < 4; ++j) split_tf32(v[j], w.hi[i][j], w.lo[i][j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = p[j >> 1][2 * (j & 1)], y = p[j >> 1][2 * (j & 1) + 1];
                if constexpr (KV == kBF16) {
                    w.hi[0][j] = pack_bf16(x, y);
                    w.lo[0][j] = pack_bf16(x - __uint_as_float(w.hi[0][j] << 16),
                                           y - __uint_as_float(w.hi[0][j] & 0xFFFF0000u));
                } else {
                    w.hi[0][j] = pack_f16(x, y);
                    w.lo[0][j] = 0;
                }
            }
        }
        return w;
    }

    // B fragments of V for output tiles 2 i and 2 i + 1: v[0..1] and v[2..3], as
    // stored (BF16, widened FP8) or FP32 bits; FP32 for the 8 tokens of half h.
    __device__ __forceinline__ void values(uint32_t vb, int i, int h, uint32_t (&v)[4]) const {
        if constexpr (KV == kBF16) {
            ldsm4t(v, vb + swz<S>(lane & 15, 2 * i + (lane >> 4)));
        }
        if constexpr (KV == kF32) {
            const int d0 = i * 16 + g, r0 = h * 8 + 2 * c;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = d0 + 8 * (j >> 1), r = r0 + (j & 1);
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[j]) : "r"(vb + swz<S>(r, d >> 2) + (d & 3) * 4));
            }
        }
    }
    // FP8: one load covers 32 columns (two pairs of tiles); tile 2 i holds the
    // even columns of chunk i, tile 2 i + 1 the odd ones.
    __device__ __forceinline__ void values_fp8(uint32_t vb, int i, uint32_t (&v)[2][4]) const {
        uint32_t r[4];
        ldsm4t(r, vb + swz<S>(lane & 15, i + (lane >> 4)));
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {                     // tokens 0-7, 8-15
                v[j][k] = e4m3x2_to_h2(__byte_perm(r[2 * j + k], 0, 0x4420));
                v[j][2 + k] = e4m3x2_to_h2(__byte_perm(r[2 * j + k], 0, 0x4431));
            }
    }

    __device__ __forceinline__ void product(float (&acc)[4], const Weights& w, int h, uint32_t b0, uint32_t b1) const {
        if constexpr (KV == kBF16) {
            mma_bf16(acc, w.hi[0], b0, b1);
            mma_bf16(acc, w.lo[0], b0, b1);
        } else if constexpr (KV == kFP8) {
            mma_f16(acc, w.hi[0], b0, b1);
        } else {
            uint32_t h0, l0, h1, l1;
            split_tf32(__uint_as_float(b0), h0, l0);
            split_tf32(__uint_as_float(b1), h1, l1);
            float p[4] = {};                                   // a short chain, as in scores()
            mma_tf32(p, w.lo[h], h0, h1);
            mma_tf32(p, w.hi[h], l0, l1);
            mma_tf32(p, w.hi[h], h0, h1);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] += p[j];
        }
    }

    // Every (tile, half) fragment of V through f(tile, half, b0, b1); half is 0
    // but for FP32, where 0 and 1 are tokens 0-7 and 8-15.
    template <class F>
    __device__ __forceinline__ void each_value(uint32_t vb, F f) const {
        if constexpr (KV == kFP8) {
#pragma unroll
            for (int i = 0; i < D / 16; i += 2) {
                uint32_t v[2][4];
                values_fp8(vb, i, v);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    f(2 * (i + j), 0, v[j][0], v[j][1]);
                    f(2 * (i + j) + 1, 0, v[j][2], v[j][3]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kTiles / 2; ++i)
#pragma unroll
                for (int h = 0; h < (KV == kF32 ? 2 : 1); ++h) {
                    uint32_t v[4];
                    values(vb, i, h, v);
                    f(2 * i, h, v[0], v[1]);
                    f(2 * i + 1, h, v[2], v[3]);
                }
        }
    }

    // A fragment with the tokens outside [lo, hi] (of the group: 0..15) set to zero bits.
    __device__ __forceinline__ uint32_t cut(uint32_t v, int half, int which, int lo, int hi) const {
        if constexpr (KV == kF32) {
            const int t = half * 8 + 2 * c + which;
            return (t >= lo && t <= hi) ? v : 0u;
        } else {
            const int t = which * 8 + 2 * c;
            return v & ((t >= lo && t <= hi ? 0x0000FFFFu : 0u) | (t + 1 >= lo && t + 1 <= hi ? 0xFFFF0000u : 0u));
        }
    }
    // Of a word of the cache.
    __device__ __forceinline__ static bool stored_not_finite(uint32_t v) {
        if constexpr (KV == kF32) return (v & 0x7F800000u) == 0x7F800000u;
        if constexpr (KV == kBF16) return (((v & 0x7F807F80u) + 0x00800080u) & 0x80008000u) != 0;
        return (((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;       // E4M3: 0x7F alone
    }

    // FP32: an infinity, or a number near the largest, makes a split product NaN.
    // Scores that are NaN are taken once more as they stand: -inf then is -inf (and
    // weighs nothing), and NaN is NaN. (16 requests of 1000 to 2000 tokens, 8 cache heads
    // of 128: 1 row 75.1 -> 74.0 us, 64 rows 217 -> 221.)
    __device__ __forceinline__ void retake(uint32_t kb, float (&s)[2][4]) const {
        if constexpr (KV == kF32) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += s[j >> 2][j & 3];
            if (sum == sum) return;
            float plain[8] = {};
#pragma unroll 1
            for (int d = 0; d < D; ++d) {
                const float q[2] = {qs[g * (S::QS / 4) + d], qs[(g + 8) * (S::QS / 4) + d]};
#pragma unroll
                for (int t = 0; t < 4; ++t) {                 // tokens 2 c, +1, of either half
                    float k;
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(k) : "r"(kb + swz<S>(8 * (t >> 1) + 2 * c + (t & 1), d >> 2) + (d & 3) * 4));
                    plain[t] = fmaf(q[0], k, plain[t]);
                    plain[4 + t] = fmaf(q[1], k, plain[4 + t]);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float& x = s[j >> 2][j & 3];
                const int row = (j >> 1) & 1, t = 2 * (j >> 2) + (j & 1);
                if (x != x) x = plain[4 * row + t] * mul[row];
            }
        }
    }

    // Running maximum and sum over the scores of 8 N tokens, which become their
    // weights; the outputs so far are rescaled where the maximum grew.
    template <int N>
    __device__ __forceinline__ void softmax(float (&s)[N][4]) {
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) mx[j >> 1] = fmaxf(mx[j >> 1], s[i][j]);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 1));
            mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], 2));
        }
        if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
            float f[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                f[x] = ex2(m[x] - (mx[x] == -INFINITY ? 0.f : mx[x]));
                m[x] = mx[x];
                l[x] *= f[x];
            }
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                o[i][0] *= f[0];
                o[i][1] *= f[0];
                o[i][2] *= f[1];
                o[i][3] *= f[1];
            }
        }
        const float ref[2] = {(m[0] == -INFINITY ? 0.f : m[0]) - kUp, (m[1] == -INFINITY ? 0.f : m[1]) - kUp};
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = ex2(s[i][j] - ref[j >> 1]);
                sum[j >> 1] += s[i][j];
            }
        l[0] += sum[0];
        l[1] += sum[1];
    }

    // o += weights V of one group.
    __device__ __forceinline__ void accumulate(uint32_t vb, const Weights& w) {
        if constexpr (KV == kBF16) {
            // four tiles' first terms, then their second ones: no product waits for its neighbour
#pragma unroll
            for (int i = 0; i < kTiles; i += 4) {
                uint32_t v[2][4];
                values(vb, i / 2, 0, v[0]);
                values(vb, i / 2 + 1, 0, v[1]);
#pragma unroll
                for (int j = 0; j < 4; ++j) mma_bf16(o[i + j], w.hi[0], v[j >> 1][2 * (j & 1)], v[j >> 1][2 * (j & 1) + 1]);
#pragma unroll
                for (int j = 0; j < 4; ++j) mma_bf16(o[i + j], w.lo[0], v[j >> 1][2 * (j & 1)], v[j >> 1][2 * (j & 1) + 1]);
            }
        } else if constexpr (KV == kF32) {
            // short chains, as in scores(), four tiles beside each other
#pragma unroll
            for (int i = 0; i < kTiles; i += 4) {
                float p[4][4] = {};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t v[2][4], vh[2][4], vl[2][4];
                    values(vb, i / 2, h, v[0]);
                    values(vb, i / 2 + 1, h, v[1]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) split_tf32(__uint_as_float(v[j >> 2][j & 3]), vh[j >> 2][j & 3], vl[j >> 2][j & 3]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma_tf32(p[j], w.lo[h], vh[j >> 1][2 * (j & 1)], vh[j >> 1][2 * (j & 1) + 1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma_tf32(p[j], w.hi[h], vl[j >> 1][2 * (j & 1)], vl[j >> 1][2 * (j & 1) + 1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma_tf32(p[j], w.hi[h], vh[j >> 1][2 * (j & 1)], vh[j >> 1][2 * (j & 1) + 1]);
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) o[i + (j >> 2)][j & 3] += p[j >> 2][j & 3];
            }
        } else {
            each_value(vb, [&](int t, int h, uint32_t b0, uint32_t b1) { product(o[t], w, h, b0, b1); });
        }
    }

    // NG groups whose tokens all rows see.
    template <int NG>
    __device__ __forceinline__ void step(const uint32_t (&kb)[NG], const uint32_t (&vb)[NG]) {
        float s[2 * NG][4];
#pragma unroll
        for (int n = 0; n < NG; ++n) scores(kb[n], *reinterpret_cast<float(*)[2][4]>(&s[2 * n]));
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] *= mul[j >> 1];
#pragma unroll
        for (int n = 0; n < NG; ++n) retake(kb[n], *reinterpret_cast<float(*)[2][4]>(&s[2 * n]));
        softmax(s);
#pragma unroll
        for (int n = 0; n < NG; ++n) accumulate(vb[n], weights(*reinterpret_cast<float(*)[2][4]>(&s[2 * n])));
    }

    // One group of which rows g and g + 8 see the tokens lo[x]..hi[x] (0..15) and
    // some row of the block any_lo..any_hi, all of them all_lo..all_hi; tok0 is its
    // first token's position.
    __device__ __forceinline__ void step_masked(uint32_t kb, uint32_t vb, const int (&lo)[2], const int (&hi)[2], int any_lo,
                                                int any_hi, int all_lo, int all_hi, int T, int tok0, int len, int window, const int (&draft)[2]) {
        float s[2][4];
        scores(kb, s);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int x = j >> 1, t = 8 * i + 2 * c + (j & 1);
                s[i][j] = (t < lo[x] || t > hi[x]) ? -INFINITY : s[i][j] * mul[x];
            }
        retake(kb, s);
        softmax(s);
        const Weights w = weights(s);
        bool bad = false;
        if (T > 1) {
            // the tokens that some drafts see and others do not, at most T - 1 at either end
            constexpr int kChunks = S::RB / 16;
            const int a0 = max(any_lo, 0), na = max(0, min(all_lo, kAttnGroup) - a0);
            const int b0 = max(max(all_hi + 1, 0), a0 + na), nb = max(0, min(any_hi, kAttnGroup - 1) + 1 - b0);
            for (int i = lane; i < (na + nb) * kChunks; i += 32) {
                const int n = i / kChunks, r = n < na ? a0 + n : b0 + n - na;
                uint32_t v[4];
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(vb + swz<S>(r, i % kChunks)));
                bad = bad || stored_not_finite(v[0]) || stored_not_finite(v[1]) || stored_not_finite(v[2]) || stored_not_finite(v[3]);
            }
            bad = __any_sync(0xffffffffu, bad);
        }
        if (!bad) {
            each_value(vb, [&](int t, int h, uint32_t b0, uint32_t b1) {
                product(o[t], w, h, cut(b0, h, 0, any_lo, any_hi), cut(b1, h, 1, any_lo, any_hi));
            });
            return;
        }
        // 0 * infinity must not reach a row that does not see the token: draft
        // by draft, with only that draft's tokens in place, into its rows alone
        for (int t = 0; t < T; ++t) {
            const int p = len - T + t;
            const int a0 = window_start(p, window) - tok0, a1 = p - tok0;
            each_value(vb, [&](int tile, int h, uint32_t b0, uint32_t b1) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                product(acc, w, h, cut(b0, h, 0, a0, a1), cut(b1, h, 1, a0, a1));
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (draft[j >> 1] == t) o[tile][j] += acc[j];
            });
        }
    }

    // The outputs times f[row] to rows g and g + 8 of a buffer (`to`: row g), or
    // added to what is there.
    template <bool kAdd>
    __device__ __forceinline__ void leave(float* to, const float (&f)[2]) const {
#pragma unroll
        for (int i = 0; i < kTiles; i += 2)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float* d = to + 8 * x * S::OS;
                const float a0 = o[i][2 * x] * f[x], a1 = o[i][2 * x + 1] * f[x];
                const float b0 = o[i + 1][2 * x] * f[x], b1 = o[i + 1][2 * x + 1] * f[x];
                if constexpr (KV == kFP8) {                   // tiles of even and of odd columns
                    float4* p = reinterpret_cast<float4*>(d + 8 * i + 4 * c);
                    float4 v = make_float4(a0, b0, a1, b1);
                    if (kAdd) v.x += p->x, v.y += p->y, v.z += p->z, v.w += p->w;
                    *p = v;
                } else {
                    float2 *p = reinterpret_cast<float2*>(d + 8 * i + 2 * c), *q = p + 4;
                    float2 v = make_float2(a0, a1), u = make_float2(b0, b1);
                    if (kAdd) v.x += p->x, v.y += p->y, u.x += q->x, u.y += q->y;
                    *p = v;
                    *q = u;
                }
            }
    }
};

// Outputs of row r of a part, columns col..col + 3, from the sums v under maximum
// M and total L; vs: FP8, the scale of the head's values.
template <int KV, class S>
__device__ __forceinline__ void put(const AttnArgs& a, const Part& part, int r, int col, float4 v, float M, float L, float vs) {
    const int t = (part.row0 + r) / a.group, j = (part.row0 + r) % a.group;
    const int64_t at = (static_cast<int64_t>(part.b) * a.T + t) * a.q_heads + part.head * a.group + j;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    v.x *= inv; v.y *= inv; v.z *= inv; v.w *= inv;
    if (KV == kFP8) {
        v.x *= vs; v.y *= vs; v.z *= vs; v.w *= vs;
    }
    if (KV == kF32) {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at * S::D + col) = v;
    } else {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at * S::D + col) =
            make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    }
    if (a.lse != nullptr && col == 0) a.lse[at] = L == 0.f ? -INFINITY : (M + (log2f(L) - Warp<KV, S>::kUp)) * 0.69314718055994531f;
}

// Join the parts of a request and head: the consumer warps, once all have
// arrived. Not inlined: it runs once or twice a block, and its registers are
// not the stream's.
constexpr int kJoin = 16;      // parts joined at a time

template <int KV, class S>
__device__ __noinline__ void join_parts(const AttnArgs& a, const Part part, float* fw, float2* s_row, volatile int* s_last) {
    const int rows = min(S::kRows, a.T * a.group - part.row0);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int D = S::D, kThreads = S::kConsumers * 32;
    static_assert((kAttnMaxGrid + kJoin - 1) / kJoin <= 32 && 32 <= S::OS, "a round of parts must fit a warp and the buffer");
    const int np = part.others + 1;
    const float vs = KV == kFP8 ? __ldcg(a.v_scale + part.head) : 1.f;
    // this block's kJoin neighbours, and then one part for each such round; or all at once
    int p0 = 0, step = 1, n = np;
    bool final = np <= kJoin;
    if (!final) {
        p0 = (static_cast<int>(blockIdx.x) - part.first) / kJoin * kJoin;
        n = min(kJoin, np - p0);
    }
    for (;;) {
        const auto part_at = [&](int i, int r) {              // part p0 + i step
            const int p = p0 + i * step;
            return (2 * static_cast<int64_t>(part.first + p) + (p == 0 ? 1 : 0)) * S::kRows + r;
        };
        // Weights of the parts first (parts across the lanes, a warp a row at a
        // time), then the outputs, with no product waiting for another.
        for (int r = warp; r < rows; r += S::kConsumers) {
            float2 ml = make_float2(-INFINITY, 0.f);
            if (lane < n) ml = __ldcg(a.part_ml + part_at(lane, r));
            const float M = warp_max(ml.x);
            const float f = ex2(ml.x - (M == -INFINITY ? 0.f : M));
            if (lane < n) fw[lane * rows + r] = f;            // [n][rows]
            const float L = warp_sum(ml.y * f);
            if (lane == 0) s_row[r] = make_float2(M, L);
        }
        named_sync(1, kThreads);
        // 16 loads ahead: of one output where there is one a thread, else of four
        const auto sums = [&](auto items_c, auto ahead_c) {
            constexpr int kItems = decltype(items_c)::value, kAhead = decltype(ahead_c)::value;
            const int items = rows * (D / 4);
            for (int x0 = tid; x0 < items; x0 += kItems * kThreads) {
                float4 acc[kItems];
#pragma unroll
                for (int i = 0; i < kItems; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int q = 0; q < n; q += kAhead) {
                    float4 v[kItems][kAhead];
                    float fp[kItems][kAhead];
#pragma unroll
                    for (int i = 0; i < kItems; ++i)
#pragma unroll
                        for (int k = 0; k < kAhead; ++k) {
                            const int x = x0 + i * kThreads;
                            v[i][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                            fp[i][k] = 0.f;
                            if (x >= items || q + k >= n) continue;
                            const int r = x / (D / 4), col = (x % (D / 4)) * 4;
                            v[i][k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + part_at(q + k, r) * D + col));
                            fp[i][k] = fw[(q + k) * rows + r];
                        }
#pragma unroll
                    for (int k = 0; k < kAhead; ++k)
#pragma unroll
                        for (int i = 0; i < kItems; ++i) {
                            acc[i].x = fmaf(v[i][k].x, fp[i][k], acc[i].x);
                            acc[i].y = fmaf(v[i][k].y, fp[i][k], acc[i].y);
                            acc[i].z = fmaf(v[i][k].z, fp[i][k], acc[i].z);
                            acc[i].w = fmaf(v[i][k].w, fp[i][k], acc[i].w);
                        }
                }
#pragma unroll
                for (int i = 0; i < kItems; ++i) {
                    const int x = x0 + i * kThreads;
                    if (x >= items) break;
                    const int r = x / (D / 4), col = (x % (D / 4)) * 4;
                    if (final) {
                        put<KV, S>(a, part, r, col, acc[i], s_row[r].x, s_row[r].y, vs);
                    } else {
                        // into the round's first part, which only this thread still reads here
                        __stcg(reinterpret_cast<float4*>(a.part_o + part_at(0, r) * D + col), acc[i]);
                        if (col == 0) __stcg(a.part_ml + part_at(0, r), s_row[r]);
                    }
                }
            }
        };
        if (rows * (D / 4) <= kThreads) sums(Int<1>{}, Int<16>{});
        else sums(Int<4>{}, Int<4>{});
        if (final) return;
        named_sync(1, kThreads);
        if (tid == 0) *s_last = arrive_last(a.arrived + part.first, (np - 1) / kJoin);
        named_sync(1, kThreads);
        if (!*s_last) return;
        p0 = 0;
        step = kJoin;
        n = (np + kJoin - 1) / kJoin;
        final = true;
    }
}

// ---- the kernel --------------------------------------------------------------
template <int KV, class S>
__global__ void __launch_bounds__(S::kThreads, S::kMinBlocks)
attn_decode_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    constexpr int D = S::D, NS = S::NS;
    extern __shared__ char smem_raw[];
    char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    char* slots = smem;
    char* qbuf = slots + NS * S::kSlot;                                  // [2][kRows][QS]
    float* merged = reinterpret_cast<float*>(qbuf + 2 * S::kRows * S::QS);   // [NB][kRows][OS]
    float2* s_ml = reinterpret_cast<float2*>(merged + S::NB * S::kRows * S::OS);   // [NT][kRows]
    float2* s_row = s_ml + S::NT * S::kRows;                             // [kRows]
    uint64_t* full = reinterpret_cast<uint64_t*>(s_row + S::kRows);      // [NS]
    uint64_t* empty = full + NS;
    uint64_t* qfull = empty + NS;                                        // [2]
    uint64_t* qempty = qfull + 2;
    volatile int* dead = reinterpret_cast<volatile int*>(qempty + 2);
    volatile int* s_last = dead + 1;
    Part* s_part = reinterpret_cast<Part*>(const_cast<int*>(dead + 2));  // [2]

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, S::WM);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(qfull + i, 1);
            mbar_init(qempty + i, S::kConsumers);
        }
        *dead = 0;
        fence_mbar_init();
    }
    if constexpr (KV == kF32) {
        // rows beyond a part's take part in the products: zeros, so that what they
        // find in shared memory never makes retake() work
        for (int i = tid; i < 2 * S::kRows * S::QS / 16; i += S::kThreads) reinterpret_cast<float4*>(qbuf)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    after_predecessor();

    const int rows_all = a.T * a.group;
    int pos = 0, turn = 0;     // ring: the next group's slot, and how often the ring went round
    int parts = 0;

    if (warp == S::kConsumers) {
        // ---- producer ----
        // what earlier kernels stored is read by copies, another proxy, from here on
        asm volatile("fence.proxy.async.global;" ::: "memory");
        const uint32_t q_bytes = D * S::kQsz;
        Cursor cur;
        // The next part is found, and its first pages are looked up, before the
        // current one's copies go out: a part's start then costs no round trip.
        Part d, nd;
        int g1 = 0, ng1 = 0, next_page = 0, next_row = 0;
        const auto look_up = [&](int b, int base, int end, int& page, int& row) {
            page = a.num_pages;                          // outside the map: read as zeros
            row = 0;
            if (base + lane >= end) return;
            const int tok = (base + lane) * kAttnGroup;
            const int at = tok / a.page_size;
            row = tok - at * a.page_size;
            page = __ldcg(a.table + static_cast<int64_t>(b) * a.max_pages + at);
        };
        const auto find = [&]() -> bool {
            if (!cur.next(a)) return false;
            nd.b = cur.b;
            nd.len = cur.sp.len;
            nd.head = cur.pair / a.chunks;
            nd.row0 = (cur.pair - nd.head * a.chunks) * S::kRows;
            nd.g0 = cur.first_group();
            ng1 = cur.end_group();
            nd.ng = ng1 - nd.g0;
            nd.pair = cur.pair;
            nd.first = nd.others = 0;
            nd.at_start = cur.u0 == 0;
            if (cur.even) {
                nd.first = cur.first;
                nd.others = cur.others;
            } else if (cur.u1 - cur.u0 < cur.sp.units) {
                const int64_t first = cur.base + static_cast<int64_t>(cur.pair) * cur.sp.units;
                nd.first = cur.owner(first);
                nd.others = cur.owner(first + cur.sp.units - 1) - nd.first;
            }
            look_up(nd.b, nd.g0, ng1, next_page, next_row);
            return true;
        };
        bool more = cur.start(a, lane) && find();
        while (more) {
            d = nd;
            g1 = ng1;
            int page = next_page, row = next_row;
            const int rows = min(S::kRows, rows_all - d.row0);
            const int pq = parts & 1;
            if ((parts < 2 || wait_phase(qempty + pq, ((parts >> 1) - 1) & 1, dead, a.err)) && !*dead) {
                if (lane == 0) {
                    s_part[pq] = d;
                    if (d.at_start && d.pair == 0) {
                        const int given = __ldcg(a.lens + d.b);
                        if (given != d.len) report_error(a.err, RSSM_DEV_ATTN_LEN, d.b, given);
                    }
                    mbar_arrive_expect_tx(qfull + pq, rows * q_bytes);
                }
                __syncwarp();
                for (int r = lane; r < rows; r += 32) {
                    const int t = (d.row0 + r) / a.group, j = (d.row0 + r) - t * a.group;
                    const char* src = static_cast<const char*>(a.q) +
                                      ((static_cast<int64_t>(d.b) * a.T + t) * a.q_stride +
                                       static_cast<int64_t>(d.head * a.group + j) * D) * S::kQsz;
                    bulk_g2s(qbuf + (pq * S::kRows + r) * S::QS, src, q_bytes, qfull + pq);
                }
            }
            ++parts;
            // pages of 32 groups at a time, a step ahead; copies of PB groups at a time, a lane each
            more = find();
            int page2 = 0, row2 = 0;
            for (int base = d.g0; base < g1; base += 32, page = page2, row = row2) {
                look_up(d.b, base + 32, g1, page2, row2);
                if (base + lane < g1 && (page < 0 || page >= a.num_pages)) {
                    report_error(a.err, RSSM_DEV_ATTN_PAGE, d.b, page);
                    page = a.num_pages;
                }
                const int n = min(32, g1 - base);
                for (int i = 0; i < n; i += S::PB) {
                    const int m = min(S::PB, n - i);
                    const int pg = __shfl_sync(0xffffffffu, page, (i + lane) & 31), rw = __shfl_sync(0xffffffffu, row, (i + lane) & 31);
                    if (lane < m) {
                        const bool wrap = pos + lane >= NS;
                        const int s = pos + lane - (wrap ? NS : 0), tn = turn + (wrap ? 1 : 0);
                        if ((tn == 0 || wait_phase(empty + s, (tn - 1) & 1, dead, a.err)) && !*dead) {
                            const uint32_t dst = smem_u32(slots + s * S::kSlot);
                            mbar_arrive_expect_tx(full + s, S::kSlot);
                            tma_load_5d(dst, &kmap, rw, d.head, pg, full + s);
                            tma_load_5d(dst + S::kHalf, &vmap, rw, d.head, pg, full + s);
                        }
                    }
                    __syncwarp();
                    pos += m;
                    if (pos >= NS) {
                        pos -= NS;
                        ++turn;
                    }
                }
            }
        }
        // no more parts
        const int pq = parts & 1;
        if ((parts < 2 || wait_phase(qempty + pq, ((parts >> 1) - 1) & 1, dead, a.err)) && !*dead && lane == 0) {
            s_part[pq].pair = -1;
            mbar_arrive(qfull + pq);
        }
        if (*dead && lane == 0) {
            // let the copies in flight land before the block's memory goes
            for (int s = 0; s < NS; ++s) {
                const int tn = s < pos ? turn : turn - 1;   // the slot's last turn, if it had one
                if (tn >= 0) mbar_wait_bounded(full + s, tn & 1, kWaitLimitNs / 16);
            }
            for (int i = max(0, parts - 2); i < parts; ++i)
                mbar_wait_bounded(qfull + (i & 1), (i >> 1) & 1, kWaitLimitNs / 16);
        }
        return;
    }

    // ---- consumers ----
    constexpr int kThreads = S::kConsumers * 32;
    const int wm = warp / S::NT, wt = warp % S::NT;
    Warp<KV, S> wp;
    wp.lane = lane;
    wp.g = lane >> 2;
    wp.c = lane & 3;
    // The part that went to the workspace last: its arrival is counted while the
    // next part runs (one thread waits for the writes and the count, not the
    // block), and if it was the request's last, it is joined after that part.
    Part left;
    left.pair = -1;
    // A split request and head is known by the block of its first part: that part ends
    // its block's share, so no block has two such.
    const auto count_left = [&] {                            // thread 0, after a block barrier
        if (left.others < kJoin) {
            *s_last = arrive_last(a.arrived + left.first, left.others);
        } else {
            const int p = static_cast<int>(blockIdx.x) - left.first, p0 = p / kJoin * kJoin;
            *s_last = arrive_last(a.arrived_round + 2 * (left.first + p0) + (p0 == 0 ? 1 : 0),
                                  min(kJoin, left.others + 1 - p0) - 1);
        }
    };
    for (;;) {
        const int pq = parts & 1;
        // all consumer warps go on, or none: one that gave up must not leave the
        // others at a barrier
        if (!all_of(wait_phase(qfull + pq, (parts >> 1) & 1, dead, a.err), 2, kThreads)) break;
        const Part part = s_part[pq];
        if (part.pair < 0) break;
        if (left.pair >= 0 && tid == 0) count_left();
        const int head = part.head, row0 = part.row0, len = part.len;
        const int rows = min(S::kRows, rows_all - row0);
        // what the warp's two rows see: [see_lo, see_hi]
        int draft[2], see_lo[2], see_hi[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = min(row0 + wm * 16 + wp.g + 8 * x, rows_all - 1);
            draft[x] = r / a.group;
            see_hi[x] = len - a.T + draft[x];
            see_lo[x] = window_start(see_hi[x], a.window);
        }
        const int all_hi = len - a.T;                             // the last token that all drafts see
        const int all_lo = window_start(len - 1, a.window);         // and the first
        const int some_lo = window_start(len - a.T, a.window);
        wp.reset();
        wp.load_q(qbuf + (pq * S::kRows + wm * 16) * S::QS, a.scale_log2, KV == kFP8 ? __ldcg(a.k_scale + head) : 1.f);
        if (KV != kF32) {
            __syncwarp();
            if (lane == 0) mbar_arrive(qempty + pq);
        }
        // this warp's groups: those whose slot is wt modulo NT; those that all rows
        // see whole, [f0, f1), two at a time where the registers allow it
        const int g0 = part.g0, ng = part.ng;
        const int f0 = (all_lo + kAttnGroup - 1) / kAttnGroup - g0, f1 = (all_hi + 1) / kAttnGroup - g0;
        constexpr int NG = S::kPair ? 2 : 1;
        int k = (wt + S::NT - pos % S::NT) % S::NT;
        int s = pos + k, tn = turn;
        const auto forward = [&] {                            // to this warp's next group
            k += S::NT;
            s += S::NT;
            if (s >= NS) {
                s -= NS;
                ++tn;
            }
        };
        if (s >= NS) {
            s -= NS;
            ++tn;
        }
        while (k < ng) {
            const uint32_t kb = smem_u32(slots + s * S::kSlot), vb = kb + S::kHalf;
            uint64_t* const done = empty + s;
            bool ok = wait_phase(full + s, tn & 1, dead, a.err);
            if (k >= f0 && k < f1) {
                if (NG == 2 && k + S::NT < min(f1, ng)) {
                    forward();
                    const uint32_t kb2 = smem_u32(slots + s * S::kSlot), vb2 = kb2 + S::kHalf;
                    ok = wait_phase(full + s, tn & 1, dead, a.err) && ok;
                    const uint32_t ks[2] = {kb, kb2}, vs[2] = {vb, vb2};
                    if (ok) wp.step(ks, vs);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(empty + s);
                } else {
                    const uint32_t ks[1] = {kb}, vs[1] = {vb};
                    if (ok) wp.step(ks, vs);
                }
            } else if (ok) {
                const int tok = (g0 + k) * kAttnGroup;
                const int lo[2] = {see_lo[0] - tok, see_lo[1] - tok}, hi[2] = {see_hi[0] - tok, see_hi[1] - tok};
                wp.step_masked(kb, vb, lo, hi, some_lo - tok, len - 1 - tok, all_lo - tok, all_hi - tok, a.T, tok, len, a.window, draft);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(done);
            forward();
        }
        pos += ng;
        turn += pos / NS;
        pos %= NS;
        if (KV == kF32) {
            __syncwarp();
            if (lane == 0) mbar_arrive(qempty + pq);
        }
        ++parts;
        const float vs = KV == kFP8 ? __ldcg(a.v_scale + head) : 1.f;   // there once the warps are joined

        // ---- join the warps of each row ----
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            wp.l[x] += __shfl_xor_sync(0xffffffffu, wp.l[x], 1);
            wp.l[x] += __shfl_xor_sync(0xffffffffu, wp.l[x], 2);
            if (wp.c == 0) s_ml[wt * S::kRows + wm * 16 + wp.g + 8 * x] = make_float2(wp.m[x], wp.l[x]);
        }
        named_sync(1, kThreads);
        float f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = wm * 16 + wp.g + 8 * x;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < S::NT; ++w) M = fmaxf(M, s_ml[w * S::kRows + r].x);
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < S::NT; ++w) L += s_ml[w * S::kRows + r].y * ex2(s_ml[w * S::kRows + r].x - ref);
            f[x] = ex2(wp.m[x] - ref);
            if (wt == 0 && wp.c == 0) s_row[r] = make_float2(M, L);
        }
        // warp w into buffer w % NB, those of later rounds adding to it
#pragma unroll 1
        for (int w = 0; w < S::NT; w += S::NB) {
            if (wt >= w && wt < w + S::NB) {
                float* to = merged + ((wt - w) * S::kRows + wm * 16 + wp.g) * S::OS;
                if (w == 0) wp.template leave<false>(to, f);
                else wp.template leave<true>(to, f);
            }
            named_sync(1, kThreads);
        }
        const auto sum_of = [&](int r, int col) {
            float4 v = *reinterpret_cast<const float4*>(merged + r * S::OS + col);
#pragma unroll
            for (int w = 1; w < S::NB; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(merged + (w * S::kRows + r) * S::OS + col);
                v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w;
            }
            return v;
        };
        if (part.others == 0) {
            for (int x = tid; x < rows * (D / 4); x += kThreads) {
                const int r = x / (D / 4), col = (x % (D / 4)) * 4;
                put<KV, S>(a, part, r, col, sum_of(r, col), s_row[r].x, s_row[r].y, vs);
            }
        } else {
            const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + part.at_start;
            for (int x = tid; x < rows * (D / 4); x += kThreads) {
                const int r = x / (D / 4), col = (x % (D / 4)) * 4;
                __stcg(reinterpret_cast<float4*>(a.part_o + (slot * S::kRows + r) * D + col), sum_of(r, col));
                if (col == 0) __stcg(a.part_ml + slot * S::kRows + r, s_row[r]);
            }
        }
        if (left.pair >= 0) {
            named_sync(1, kThreads);                          // the buffers are read
            if (*s_last) join_parts<KV, S>(a, left, merged, s_row, s_last);
        }
        left = part;
        if (part.others == 0) left.pair = -1;
    }
    if (left.pair >= 0) {
        if (tid == 0) count_left();
        named_sync(1, kThreads);
        if (*s_last) join_parts<KV, S>(a, left, merged, s_row, s_last);
    }
}

// Launch of one shape: as many blocks as the GPU holds at once, at most kAttnMaxGrid.
template <int KV, class S>
cudaError_t launch_shape(const AttnArgs& a, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
    static LaunchCache lc;
    int sms = 0, optin = 0;
    cudaError_t e = device_limits(&sms, &optin);
    if (e != cudaSuccess) return e;
    auto kernel = attn_decode_kernel<KV, S>;
    e = cached_dyn_smem(lc, kernel, S::kSmem);
    if (e != cudaSuccess) return e;
    const int want = sms * S::kMinBlocks;
    return launch_overlapped(kernel, want < kAttnMaxGrid ? want : kAttnMaxGrid, S::kThreads, S::kSmem, s, a, k, v);
}

template <int KV, int D>
cudaError_t launch_rows(const AttnArgs& a, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
    switch (rows) {
        case 16: return launch_shape<KV, Shape<KV, D, 1>>(a, k, v, s);
        case 32: return launch_shape<KV, Shape<KV, D, 2>>(a, k, v, s);
        default:
            if constexpr (KV == kF32 && D == 256) return cudaErrorInvalidValue;
            else return launch_shape<KV, Shape<KV, D, 4>>(a, k, v, s);
    }
}

template <int KV>
cudaError_t launch_dim(const AttnArgs& a, int D, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s) {
    switch (D) {
        case 64: return launch_rows<KV, 64>(a, rows, k, v, s);
        case 128: return launch_rows<KV, 128>(a, rows, k, v, s);
        default: return launch_rows<KV, 256>(a, rows, k, v, s);
    }
}

}  // namespace attn
}  // namespace rssm
