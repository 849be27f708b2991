// The 8-bit KV store: its layout, shared by the kernels that write it, read it
// back and attend over it.
//
// Values.  The 16 tokens of a page share, per KV head and for keys and values
// apart, a scale 2^e with e in -60 .. 60; an element is an e4m3 value times it
// (the code 0x7f / 0xff is NaN; it stands for infinities too).  An e4m3 value
// has four significant bits and lies in [2^-9, 448] (or is 0): stored values are
// exact in bf16, codes are exact in f16.  With powers of two a page whose scale
// grows loses nothing but what falls below 2^-9 of the new scale's range.
//
// Layout.  A page of one KV head is 4128 bytes, of which 4112 are read, as one
// bulk copy (257 B per token against 512 in bf16; 4128 keeps pages on 32-byte
// sectors).  Inside, the bytes stand where the attention kernel's threads want
// them: lane (g, c) = (lane / 4, lane % 4) reads 16 bytes at lane * 16, which
// is free of bank conflicts, and they are matrix fragments once converted:
//   K codes   [r 2][i 2][lane][16]: token 4 (g / 2) + g % 2 + 2 r, elements
//             32 c + 16 i .. + 15
//   V codes   [i 4][lane][4][4]: elements 16 g + 4 i .. + 3, for each the tokens
//             4 c .. 4 c + 3
//   tail      e + 60 of K, e + 60 of V, as 32-bit words
// A writer's lane l with elements 4 l .. 4 l + 3 of all tokens has a word of
// each token's K codes and, for each quad of tokens, 16 bytes of V codes.
#pragma once
#include "mac_quant.cuh"

namespace macgpu {

constexpr int kBKBytes = kPage * kD;
constexpr int kBTail = 2 * kBKBytes;
constexpr int kBCopyBytes = kBTail + 16;
constexpr int kBPageBytes = kBTail + 32;
constexpr int kBExpBias = 60, kBExpTop = 120;           // exponents are held as e + 60
static_assert(kBPageBytes % 32 == 0 && kBCopyBytes % 16 == 0, "page layout");

// the four K codes 4 l .. 4 l + 3 of a token
__host__ __device__ inline int b_k_at(int tok, int l)
{
    return ((tok >> 1 & 1) * 2 + (l >> 2 & 1)) * 512 + ((2 * (tok >> 2) + (tok & 1)) * 4 + (l >> 3)) * 16 + (l & 3) * 4;
}
// the V codes 4 l .. 4 l + 3 of the tokens 4 c .. 4 c + 3: byte 4 (element % 4) + token % 4
__host__ __device__ inline int b_v_at(int c, int l) { return kBKBytes + (l & 3) * 512 + ((l >> 2) * 4 + c) * 16; }

// What an append knows of a page it stores to: the mask of the stored offsets
// and, by offset, the token (plus one) that comes there.  All zero between calls.
struct BlockMark {
    uint32_t mask;
    uint32_t token[kPage];
};

cudaError_t block_attention_config(int sm_count);
cudaError_t launch_block_attention(const QuantAttnArgs &a, int sm_count, cudaStream_t s);

}  // namespace macgpu
