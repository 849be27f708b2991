// The 4-bit KV store: its layout, shared by the kernels that write it, read it
// back and attend over it.
//
// Values.  16 consecutive elements of a head share a scale s, an e4m3 value:
// s = max|x| / 6 rounded to nearest even, at most 448; an element is s times an
// e2m1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).  An e2m1 value
// times an e4m3 scale has at most six significant bits and lies in
// [2^-10, 2688] (or is 0), so every stored value is exact in bf16 and in f16.
// A scale is never negative, so bit 7 of its byte is free: shifted to bits 7
// .. 14 of an f16 the byte is the f16 of 2^-8 times the scale, subnormals
// included, and 0xff is an f16 NaN.  That byte marks a block that holds a NaN or
// an infinity, which then reads back as NaN.
//
// Layout.  One 16-token page of one KV head is 2304 contiguous bytes (144 per
// token against 512 in bf16), [num_pages][kv_heads][2304], so a page is one
// bulk copy.  Inside a page the bytes stand where the attention kernel's
// threads want them: its warp reads a page with 16-byte shared-memory loads and
// no bank conflict, and each thread's words are matrix fragments once
// converted (g = lane / 4, c = lane % 4):
//   K codes   [token 16][64 B]: byte i of a token = elements 2 i, 2 i + 1
//   K scales  [c 4][block 8][tt 4]: token 4 c + tt
//   V codes   [w 2][block 8][c 4][tt 4][i 4]: token 4 c + tt, elements 8 w + 2 i
//             and 8 w + 2 i + 1 of the block
//   V scales  [c 4][block 8][4]: tokens 4 c, 4 c + 2, 4 c + 1, 4 c + 3 (two
//             masks then leave the f16 pairs of tokens 0, 1 and 2, 3)
// The four scales, and the sixteen bytes of value codes, of an aligned quad of
// tokens stand together, so a writer of whole quads stores words and vectors.
// In a byte the lower element stands in the low four bits.
#pragma once
#include "mac_internal.cuh"

namespace macgpu {

constexpr int kQBlock = 16;                             // elements per scale
constexpr int kQBlocks = kD / kQBlock;                  // scales per token and head
constexpr int kQPageBytes = 2 * kPage * (kD / 2 + kQBlocks);
constexpr int kQKScale = kPage * kD / 2;                // offsets in a page
constexpr int kQV = kQKScale + kPage * kQBlocks;
constexpr int kQVScale = kQV + kPage * kD / 2;
static_assert(kQPageBytes == 2304 && kQV % 128 == 0 && kQVScale % 128 == 0, "page layout");

// bits of the device error word
enum : uint32_t { kQErrPage = 1u, kQErrSlot = 2u, kQErrLen = 4u, kQErrTimeout = 8u, kQErrRow = 16u };

// the byte of token t % 4 among a block's four V scales
__host__ __device__ inline int q_scale_byte(int tt) { return (tt >> 1) | (tt & 1) << 1; }

__host__ __device__ inline int q_kscale_at(int tok, int block) { return kQKScale + (tok >> 2) * 32 + block * 4 + (tok & 3); }
__host__ __device__ inline int q_vscale_at(int tok, int block)
{
    return kQVScale + (tok >> 2) * 32 + block * 4 + q_scale_byte(tok & 3);
}
// word w of a token's two words of value codes in a block
__host__ __device__ inline int q_v_at(int tok, int block, int w)
{
    return kQV + w * 512 + (block * 4 + (tok >> 2)) * 16 + (tok & 3) * 4;
}

constexpr int kQMaxBatch = 1024;        // requests per attention call (one prefix in shared memory)
constexpr int kQMaxRows = 32;           // query rows per KV head and request: group x query tokens
constexpr int kQPartRows = 49152;       // rows of partial summaries the scratch holds (25 MB)

struct QuantStore {
    uint8_t *pages;
    int num_pages, kv_heads;
    float k_scale, v_scale, k_inv, v_inv;   // powers of two
    uint32_t *err;
};

struct QuantAttnArgs {
    QuantStore st;
    int heads, G, n_query, rows;        // rows = G * n_query
    int batch;
    const __nv_bfloat16 *q;
    const int32_t *table;
    int64_t table_stride;
    int table_cols;
    const int32_t *lens;
    __nv_bfloat16 *out;
    float *lse;
    float scale_log2;                   // score scale x log2(e) x k_scale x 2^8
    float v_out_scale;                  // v_scale x 2^8
    float *part_o;                      // [kQPartRows][128]
    float2 *part_ml;                    // [kQPartRows]
    int4 *meta;                         // groups that cross blocks: {group or -1, last block, first block, 0}
};

// A step's packed new tokens as rows (mac_quant_step_rows): arguments as in
// include/mac.h.
struct StepRowArgs {
    int batch, n_query, n_packed, table_cols;
    int64_t table_stride;
    const int32_t *starts, *pos, *slots, *table, *lens;
    int32_t *pos_out, *slots_out, *lens_out;
    uint32_t *err;
};

bool step_row_args_good(const StepRowArgs &a);
cudaError_t launch_step_rows(const StepRowArgs &a, cudaStream_t s);
void quant_error_text(uint32_t bits, char *text, size_t n);    // the error word in words

cudaError_t quant_attention_config(int sm_count);
cudaError_t launch_quant_attention(const QuantAttnArgs &a, int sm_count, cudaStream_t s);

}  // namespace macgpu
