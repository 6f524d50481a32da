// What the attention kernels and the entry points (attn.cu) share.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace rssm {

constexpr int kAttnMaxGrid = 608;    // blocks of one launch at most: four per SM
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
    const float* k_scale;       // [kv_heads], FP8 and NVFP4 caches
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
// all: 16, 32 or 64, and 8 over NVFP4 caches, whose kernel takes rows by eights. Heads of
// 256 stop at 32 over FP32 caches (the ring's slots are 32 KB there) and over NVFP4 ones
// (64 requests of 4096 tokens, 64 rows: 231 us in one block, 183 in two of 32).
inline int attn_block_rows(int rows, int kv_dtype, int D) {
    if (kv_dtype == RSSM_KV_NVFP4 && rows <= 8) return 8;
    const bool most32 = D == 256 && (kv_dtype == RSSM_F32 || kv_dtype == RSSM_KV_NVFP4);
    return rows <= 16 ? 16 : rows <= 32 || most32 ? 32 : 64;
}

// Blocks an SM for which an NVFP4 launch of that shape is made (attn_nvfp4.cuh), and the
// blocks of a launch at most; never below two an SM, what the parts' room is made for.
__host__ __device__ constexpr int attn4_blocks(int rows, int D) { return rows == 8 ? (D == 256 ? 2 : 4) : rows == 16 && D < 256 ? 2 : 1; }
__host__ __device__ constexpr int attn_max_grid(int blocks_per_sm) { return 152 * (blocks_per_sm < 2 ? 2 : blocks_per_sm); }

// The kernels by cache type (attn_f32.cu, attn_bf16.cu, attn_fp8.cu, attn_nvfp4.cu).
cudaError_t attn_launch_f32(const AttnArgs& a, int D, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s);
cudaError_t attn_launch_bf16(const AttnArgs& a, int D, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s);
cudaError_t attn_launch_fp8(const AttnArgs& a, int D, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s);
cudaError_t attn_launch_nvfp4(const AttnArgs& a, int D, int rows, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t s);

// Rotary positions of q and k, and keys and values to and from a cache (place.cu).
struct PlaceArgs {
    const void *k, *v;          // new tokens [tokens][heads][dim]
    const void* q;              // with rotary positions: null, or queries [tokens][q_heads][dim] to rotate
    void* q_out;
    int64_t k_stride, v_stride, q_stride, qo_stride;
    const int32_t* slots;
    const int32_t* positions;   // rotary positions, one a token; null: none
    const uint64_t* turns;      // [rotary_dim / 2]
    float gain;
    int rotary_dim, interleaved;
    char *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int64_t page_stride;        // bytes
    int tokens, q_heads, heads, dim, page_size, num_pages;
    int in_dtype, kv_dtype;
    int32_t* err;
};
cudaError_t place_launch(const PlaceArgs& a, cudaStream_t s);

// Tokens of a cache to k and v, which are written there.
cudaError_t read_launch(const PlaceArgs& a, cudaStream_t s);

inline int64_t kv_row_bytes(int kv_dtype, int64_t dim) {      // of a token and head
    return kv_dtype == RSSM_F32 ? 4 * dim : kv_dtype == RSSM_BF16 ? 2 * dim : kv_dtype == RSSM_KV_FP8 ? dim : dim / 16 * 9;
}

}  // namespace rssm
