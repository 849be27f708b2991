// Prompt attention: what the host layer (mac_prompt.cu) and the kernels
// (mac_prompt_attention.cu) share.
#pragma once
#include "mac_internal.cuh"

namespace macgpu {

constexpr int kPMaxBatch = 1024;        // sequences per call (their item counts stand in shared memory)
constexpr int kPMaxGroup = 128;         // query heads per KV head: a tile has at least one token
constexpr int kPLevels = 2048;          // levels by which items are ordered: of a block each up to 262016 keys
constexpr int kPMaxCtas = 256;          // upper bound of the grid (one CTA per SM)
constexpr int kPRows = 256;             // query rows of an item: two tiles of 128
// Items per CTA, at least, in the line of blocks that is cut.  us with one and two: chunks of 2048 and 509 tokens 674, 707;
// 24 ragged prompts 415, 418; 5 with 28 / 4 heads 222, 227.
constexpr int kPLineRows = 1;
// Blocks that an item counts besides its own in the split of the work: a piece costs 7000 to 10000 cycles whatever its
// length, a block 2400 to 2700.  us with 0, 2, 4 and 6: 6001 tokens of 32 / 8 heads 252, 216, 212, 216, of 28 / 4 heads
// 220, 194, 193, 193; ten prompts of 958 tokens 90, 88.5, 88, 91; 1024 prompts of 16 tokens 293, 287, 288, 288.
constexpr int kPExtra = 4;

// bits of the device error word
enum : uint32_t { kPErrStarts = 1u, kPErrTimeout = 2u };

// An item that begins in CTA first's share of the line and ends in last's: the
// first holds its part in its slot 1, the others in their slots 0.  seq < 0: none.
struct PromptMeta {
    int seq, head, tile, first, last, pad[3];
};

struct PromptArgs {
    int heads, kv_heads, G, tile_tokens;    // tile_tokens: 128 / G query tokens to a tile of 128 rows
    uint32_t pair_inverse;                  // 2^32 / (2 tile_tokens), rounded up
    int batch, lag;
    int n_q, n_kv;                          // tokens of q and of k, v
    int most_tiles;                         // pairs of tiles that `batch` sequences of n_q tokens together can have
    const int32_t *starts, *k_starts;
    void *out;                              // bf16, or fp32 where wide
    int wide;
    float *lse;
    float scale_log2;                       // score scale x log2(e)
    float *part_o;                          // [CTA][2][kPRows][128] unnormalised partial outputs
    float2 *part_ml;                        // [CTA][2][kPRows] reference (log2) and sum
    float4 *carry;                          // [CTA][2 tiles][32][128 rows] sums of runs of products
    PromptMeta *meta;                       // [CTA]
    uint32_t *err;
};

struct PromptMaps {
    CUtensorMap q, k, v;
};

cudaError_t prompt_attention_config(int sm_count);
cudaError_t prompt_maps(const PromptArgs &a, const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                        int64_t v_stride, PromptMaps &maps);
cudaError_t launch_prompt_attention(const PromptArgs &a, const PromptMaps &maps, int sm_count, cudaStream_t s);

}  // namespace macgpu
