// What the attention kernels and the entry points (attn.cu) share.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace rssm {

constexpr int kAttnMaxGrid = 304;    // blocks of one launch at most: two per SM
constexpr int kAttnGroup = 16;       // tokens that one warp takes at a time
constexpr int kAttnUnit = 4;         // groups in the unit by which work is shared out
constexpr int kEvenUnits = 8;        // units a block below which few requests are cut evenly (attn_decode.cuh)

struct AttnArgs {
    const void* q;
    int64_t q_stride;           // elements between tokens
    const int32_t* lens;        // [B]
    const int32_t* table;       // [B][max_pages]
    void* out;                  // [B][T][q_heads][D]
    float* lse;                 // [B][T][q_heads] or null
    const float* k_scale;       // [kv_heads], FP8 caches
    const float* v_scale;
    int32_t* err;               // error word [4]; [4]: a wait ran out, and the counters are not at zero
    uint32_t* arrived;          // [blocks], by the block of the request and head's first part, 0 between launches
    uint32_t* arrived_round;    // [2 blocks], by the slot of a round's first part, 0 between launches
    float2* part_ml;            // [2 blocks][rows]: maximum and sum of a part
    float* part_o;              // [2 blocks][rows][D]
    int B, q_heads, kv_heads, group, T, chunks;   // chunks: of the T*group query rows, per cache head
    int page_size, num_pages, max_pages, window;
    float scale_log2;           // softmax scale times log2(e)
};

// Query rows (drafts x heads of a cache head) that one block takes, for `rows` in
// all: 16, 32 or 64. FP32 heads of 256 stop at 32: the ring's slots are 32 KB there.
inline int attn_block_rows(int rows, int kv_dtype, int D) {
    return rows <= 16 ? 16 : rows <= 32 || (kv_dtype == RSSM_F32 && D == 256) ? 32 : 64;
}

// The kernels by cache type (attn_f32.cu, attn_bf16.cu, attn_fp8.cu).
cudaError_t attn_launch_f32(const AttnArgs& a, int D, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s);
cudaError_t attn_launch_bf16(const AttnArgs& a, int D, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s);
cudaError_t attn_launch_fp8(const AttnArgs& a, int D, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s);

}  // namespace rssm
