// The 8-bit KV store (layout and format: mac_block.cuh): its handle, the append
// that quantises new tokens into it by their slots, and the gather that reads
// tokens back.
//
// Append.  Per page that a call stores to, KV head, and keys or values, with x
// the call's tokens of that page (a NaN or an infinity does not count):
//   need = min { e in -60 .. 60 : max|x| <= 448 2^e }
//   e    = need                       if the call stores the page's slot 0,
//          max(e before, need)        otherwise
//   codes = e4m3(x 2^-e); where e has grown, the codes of the page's other slots
//   become e4m3(code 2^(e before - e)); where slot 0 is stored, zeros.
// So a page's tokens have to come together, wherever they stand in the call.  Up
// to kScanTokens tokens the block of a token looks through all slots of the
// call; beyond, a first kernel notes them in the pages' marks.  Either way the
// block that has the page's lowest slot stores the whole page, head by head, a
// warp to keys or values: lane l has elements 4 l .. 4 l + 3 of all 16 tokens, so
// a token is one coalesced 256-byte load and the page's largest element one warp
// maximum.  Nothing is read twice, but for the tokens of pages that get few of them
// or some that are not finite: those are loaded for the maximum and again for the
// codes.
#include "../../include/mac.h"
#include "mac_block.cuh"
#include "mac_device.cuh"

#include <cuda_fp16.h>

#include <cmath>
#include <cstdio>
#include <mutex>
#include <new>

using namespace macgpu;

namespace macgpu {

namespace {

constexpr int kThreads = 256;
// Tokens of a call up to which every token's block looks through all slots.  Both
// sides, us, 8 heads, scan against marks: 256 requests' tokens 3.6 / 8.8, 1000
// requests' 10.4 / 17; 1024 tokens in whole pages 6.2 / 10; 2048 10.5 / 11.3, but
// of 2000 requests on one head 10.5 / 6.9.
constexpr int kScanTokens = 1024;
// Beyond: blocks that fit an SM at once, so that a call is one wave of them, and at
// most so many tokens to a block (32768 tokens, us: 16 to a block 42.8, 64 41, of
// one head 13.7 and 8.4; with registers for three blocks 50, for five 80).
constexpr int kBlocksPerSm = 4, kMostTokens = 64;
// Tokens of a page up to which they are stored one after another (1024 tokens in
// whole pages so 13 us against 6.2 at once, 1000 requests' tokens 7.7 against 10.4
// where the kernel has both; 8 of them 2.8 either way).
constexpr int kFewTokens = 4;
// (token, head) pairs below which a gather's warp takes 4 tokens instead of 16
// (us: 8 tokens 2.6 against 4.1, 1024 2.7 / 3.7, 8192 10.4 / 10.1, 32768 41 / 37).
constexpr int kSmallGather = 16384;

// Two bf16 elements' magnitude patterns, 0 for a NaN or an infinity.
__device__ __forceinline__ uint32_t finite_magnitudes(uint32_t two)
{
    const uint32_t m = two & 0x7fff7fffu;
    return m & ~__vcmpgeu2(m, 0x7f807f80u);
}

// e + 60 that a largest magnitude pattern (bf16) needs: 448 = 1.75 x 2^8.
__device__ __forceinline__ int needed_exponent(uint32_t top)
{
    const int e = (int)(top >> 7) - 127 - 8 + ((top & 127u) > 96u) + kBExpBias;
    return min(max(e, 0), kBExpTop);
}

// Four bf16 elements -> e4m3 codes; inv is the scale's inverse.  The added x * 0
// makes an infinity NaN.
__device__ __forceinline__ uint32_t to_codes(uint2 u, float inv)
{
    float x[4] = {__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                  __uint_as_float(u.y & 0xffff0000u)};
#pragma unroll
    for (int i = 0; i < 4; i++) x[i] = __fmaf_rn(x[i], inv, __fmul_rn(x[i], 0.f));
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(x[3]), "f"(x[2]));
    return lo | (uint32_t)hi << 16;
}

// The same for finite elements.
__device__ __forceinline__ uint32_t finite_codes(uint2 u, float inv)
{
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n"
        : "=h"(lo) : "f"(__uint_as_float(u.x & 0xffff0000u) * inv), "f"(__uint_as_float(u.x << 16) * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n"
        : "=h"(hi) : "f"(__uint_as_float(u.y & 0xffff0000u) * inv), "f"(__uint_as_float(u.y << 16) * inv));
    return lo | (uint32_t)hi << 16;
}

__device__ __forceinline__ void from_codes(uint32_t w, float (&x)[4])
{
    uint32_t lo, hi;
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo)), b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}

// Codes rounded again at a scale 1 / f times theirs.
__device__ __forceinline__ uint32_t requantise(uint32_t w, float f)
{
    float x[4];
    from_codes(w, x);
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(x[1] * f), "f"(x[0] * f));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(x[3] * f), "f"(x[2] * f));
    return lo | (uint32_t)hi << 16;
}

// A 4 x 4 matrix of bytes (a word per row) transposed.
__device__ __forceinline__ void transpose4(uint32_t (&w)[4])
{
    const uint32_t a = __byte_perm(w[0], w[1], 0x5140), b = __byte_perm(w[2], w[3], 0x5140);
    const uint32_t c = __byte_perm(w[0], w[1], 0x7362), d = __byte_perm(w[2], w[3], 0x7362);
    w[0] = __byte_perm(a, b, 0x5410);
    w[1] = __byte_perm(a, b, 0x7632);
    w[2] = __byte_perm(c, d, 0x5410);
    w[3] = __byte_perm(c, d, 0x7632);
}

__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((127 + e) << 23); }

struct BlockMoveArgs {
    QuantStore st;
    BlockMark *marks;
    const __nv_bfloat16 *k, *v;         // append: sources with a token stride
    int64_t k_stride, v_stride;
    __nv_bfloat16 *k_out, *v_out;       // gather: dense destinations
    const int32_t *slots;
    int n_tokens;
};

// The slot as it stands if it is inside the store, else -1.
__device__ __forceinline__ int slot_inside(const BlockMoveArgs &a, int t, bool report)
{
    const int slot = a.slots[t];
    if (slot >= 0 && slot / kPage >= a.st.num_pages) {
        if (report) atomicOr(a.st.err, kQErrSlot);
        return -1;
    }
    return slot < 0 ? -1 : slot;
}

__global__ void __launch_bounds__(kThreads) block_mark_kernel(const __grid_constant__ BlockMoveArgs a)
{
    pdl_wait();
    pdl_launch_dependents();
    const int t = blockIdx.x * kThreads + threadIdx.x;
    if (t >= a.n_tokens) return;
    const int slot = slot_inside(a, t, true);
    if (slot < 0) return;
    BlockMark &m = a.marks[slot / kPage];
    atomicOr(&m.mask, 1u << slot % kPage);
    atomicMax(&m.token[slot % kPage], (uint32_t)t + 1u);    // of tokens that share a slot the last one counts
}

// One page of one KV head, keys or values, by a warp.  token[i], in shared memory:
// which token comes to offset i, for the offsets of mask.  One token after
// another: little code to fetch, which is what bounds a small call.
__device__ __noinline__ void store_tokens(const BlockMoveArgs &a, const int *token, uint32_t mask, uint8_t *page, bool is_v, int h)
{
    const int lane = threadIdx.x & 31;
    const __nv_bfloat16 *src = (is_v ? a.v : a.k) + h * kD + 4 * lane;
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    auto load = [&](int i) { return *reinterpret_cast<const uint2 *>(src + token[i] * stride); };
    uint32_t *tail = reinterpret_cast<uint32_t *>(page + kBTail) + is_v;
    const bool fresh = mask & 1;
    const int before = fresh ? 0 : min((int)*tail, kBExpTop);
    uint32_t two = 0;
#pragma unroll 1
    for (uint32_t m = mask; m; m &= m - 1) {
        const uint2 u = load(__ffs(m) - 1);
        two = __vmaxu2(two, __vmaxu2(finite_magnitudes(u.x), finite_magnitudes(u.y)));
    }
    const int need = needed_exponent(__reduce_max_sync(0xffffffffu, max(two & 0xffffu, two >> 16)));
    const int now = max(before, need);
    const bool grows = !fresh && now > before, others = fresh || grows;
    const float inv = power_of_two(kBExpBias - now), down = power_of_two(max(before - now, -60));
    __syncwarp();                       // every lane has read the page's exponent
    if (lane == 0 && others) *tail = now;
    if (!is_v) {
#pragma unroll 1
        for (uint32_t m = others ? 0xffffu : mask; m; m &= m - 1) {
            const int i = __ffs(m) - 1;
            uint32_t *at = reinterpret_cast<uint32_t *>(page + b_k_at(i, lane));
            *at = mask >> i & 1 ? to_codes(load(i), inv) : fresh ? 0u : requantise(*at, down);
        }
    } else {
#pragma unroll 1
        for (int c = 0; c < kPage / 4; c++) {
            const uint32_t mine = mask >> 4 * c & 15;
            if (!mine && !others) continue;
            uint4 *at = reinterpret_cast<uint4 *>(page + b_v_at(c, lane));
            uint32_t w[4] = {0, 0, 0, 0};
            if (mine != 15 && !fresh) {
                const uint4 old = *at;
                w[0] = old.x, w[1] = old.y, w[2] = old.z, w[3] = old.w;
                transpose4(w);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if (mine >> i & 1) w[i] = to_codes(load(4 * c + i), inv);
                else if (grows) w[i] = requantise(w[i], down);
            }
            transpose4(w);
            *at = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// The same for many tokens at once, all loads in flight together.  Elements that
// are not finite, which do not count towards the scale and become NaN, are left
// to the function above, so that nobody else pays for them.
__device__ __forceinline__ void store_page(const BlockMoveArgs &a, const int *tokens, uint32_t mask, uint8_t *page, bool is_v, int h)
{
    const int lane = threadIdx.x & 31;
    int token[kPage];
#pragma unroll
    for (int i = 0; i < kPage; i++) token[i] = tokens[i];
    const __nv_bfloat16 *src = (is_v ? a.v : a.k) + h * kD + 4 * lane;
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    uint2 u[kPage];
    uint32_t *tail = reinterpret_cast<uint32_t *>(page + kBTail) + is_v;
    const bool fresh = token[0] >= 0;
    const int before = fresh ? 0 : min((int)*tail, kBExpTop);
#pragma unroll
    for (int i = 0; i < kPage; i++) {
        u[i] = make_uint2(0, 0);
        if (token[i] >= 0) u[i] = *reinterpret_cast<const uint2 *>(src + token[i] * stride);
    }
    uint32_t two = 0;
#pragma unroll
    for (int i = 0; i < kPage; i++) two = __vimax3_u16x2(two, u[i].x & 0x7fff7fffu, u[i].y & 0x7fff7fffu);
    const uint32_t top = __reduce_max_sync(0xffffffffu, max(two & 0xffffu, two >> 16));
    if (top >= 0x7f80u) {
        store_tokens(a, tokens, mask, page, is_v, h);
        return;
    }
    const int need = needed_exponent(top);
    const int now = max(before, need);
    const bool grows = !fresh && now > before;
    const float inv = power_of_two(kBExpBias - now), down = power_of_two(max(before - now, -60));
    __syncwarp();                       // every lane has read the page's exponent
    if (lane == 0 && (fresh || grows)) *tail = now;
    if (!is_v) {
#pragma unroll
        for (int i = 0; i < kPage; i++) {
            uint32_t *at = reinterpret_cast<uint32_t *>(page + b_k_at(i, lane));
            if (token[i] >= 0) *at = finite_codes(u[i], inv);
            else if (fresh) *at = 0;
            else if (grows) *at = requantise(*at, down);
        }
    } else {
#pragma unroll
        for (int c = 0; c < kPage / 4; c += 2) {
            // two quads of tokens are 32 bytes, one whole sector
            uint32_t w[8];
            bool any = false;
#pragma unroll
            for (int q = 0; q < 2; q++) {
                const int t = 4 * (c + q);
                const bool some = token[t] >= 0 || token[t + 1] >= 0 || token[t + 2] >= 0 || token[t + 3] >= 0;
                const bool all = token[t] >= 0 && token[t + 1] >= 0 && token[t + 2] >= 0 && token[t + 3] >= 0;
                any |= some;
                uint32_t x[4] = {0, 0, 0, 0};
                if (!all && !fresh) {
                    const uint4 old = *reinterpret_cast<const uint4 *>(page + b_v_at(c + q, lane));
                    x[0] = old.x, x[1] = old.y, x[2] = old.z, x[3] = old.w;
                    transpose4(x);      // a word per token
                }
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (token[t + i] >= 0) x[i] = finite_codes(u[t + i], inv);
                    else if (grows) x[i] = requantise(x[i], down);
                }
                transpose4(x);          // a word per element
#pragma unroll
                for (int i = 0; i < 4; i++) w[4 * q + i] = x[i];
            }
            if (any || fresh || grows)
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n"
                             :: "l"(page + b_v_at(c, lane)), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]),
                                "r"(w[6]), "r"(w[7])
                             : "memory");
        }
    }
}

__device__ __forceinline__ void store(const BlockMoveArgs &a, const int *tokens, uint32_t mask, uint8_t *page, bool is_v, int h)
{
    if (__popc(mask) <= kFewTokens) store_tokens(a, tokens, mask, page, is_v, h);
    else store_page(a, tokens, mask, page, is_v, h);
}

// Up to kScanTokens tokens: a block per token and eight (head, keys or values),
// a warp each, which looks through the slots for the others of its page.
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) block_append_scan_kernel(const __grid_constant__ BlockMoveArgs a)
{
    __shared__ int s_token[kPage];
    __shared__ uint32_t s_mask;
    const int tid = threadIdx.x, Hkv = a.st.kv_heads, item = blockIdx.y * (kThreads / 32) + (tid >> 5);
    pdl_wait();
    const int slot = slot_inside(a, blockIdx.x, tid == 0 && blockIdx.y == 0);
    if (slot < 0) return;
    const int page = slot / kPage;
    if (tid < kPage) s_token[tid] = -1;
    if (tid == kPage) s_mask = 0;
    __syncthreads();
    for (int t = tid; t < a.n_tokens; t += kThreads) {
        const int other = a.slots[t];
        if (other >= 0 && other / kPage == page) {
            atomicMax(&s_token[other % kPage], t);          // of tokens that share a slot the last one counts
            atomicOr(&s_mask, 1u << other % kPage);
        }
    }
    __syncthreads();
    // the block that has the page's lowest slot stores the page
    if (__ffs(s_mask) - 1 != slot % kPage || s_token[slot % kPage] != (int)blockIdx.x || item >= 2 * Hkv) return;
    store(a, s_token, s_mask, a.st.pages + ((size_t)page * Hkv + (item >> 1)) * kBPageBytes, item & 1, item >> 1);
}

// More tokens: a block takes the pages whose lowest slot is among its `tokens`
// consecutive tokens (kept in the marks), and its warps go through their heads'
// keys and values.
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) block_append_kernel(const __grid_constant__ BlockMoveArgs a, int tokens)
{
    __shared__ int s_page[kMostTokens], s_token[kMostTokens][kPage], s_pages;
    const int tid = threadIdx.x, Hkv = a.st.kv_heads;
    if (tid == 0) s_pages = 0;
    __syncthreads();
    pdl_wait();
    if (tid < tokens) {
        const int64_t t = (int64_t)blockIdx.x * tokens + tid;
        const int slot = t < a.n_tokens ? slot_inside(a, (int)t, false) : -1;
        if (slot >= 0) {
            // a page that another block has stored already has an empty mark
            const volatile BlockMark *m = a.marks + slot / kPage;
            const uint32_t mask = m->mask;
            if (mask && __ffs(mask) - 1 == slot % kPage && m->token[slot % kPage] == (uint32_t)t + 1u)
                s_page[atomicAdd(&s_pages, 1)] = slot / kPage;
        }
    }
    __syncthreads();
    const int pages = s_pages;
    for (int i = tid; i < pages * kPage; i += kThreads) {
        BlockMark &m = a.marks[s_page[i / kPage]];
        s_token[i / kPage][i % kPage] = (int)m.token[i % kPage] - 1;
        m.token[i % kPage] = 0;
        if (i % kPage == 0) m.mask = 0;
    }
    __syncthreads();
    for (int w = tid >> 5; w < pages * 2 * Hkv; w += kThreads / 32) {
        const int i = w / (2 * Hkv), item = w - i * 2 * Hkv, h = item >> 1, lane = tid & 31;
        uint8_t *page = a.st.pages + ((size_t)s_page[i] * Hkv + h) * kBPageBytes;
        const uint32_t mask = __ballot_sync(0xffffffffu, lane < kPage && s_token[i][lane & (kPage - 1)] >= 0);
        store(a, s_token[i], mask, page, item & 1, h);
    }
}

// A warp reads 4 kQuads consecutive tokens' keys or values of one head, lane l
// the elements 4 l .. 4 l + 3.  The values of four tokens that are an aligned quad
// of a page, as a prefill's are, come with one load.
template <int kQuads>
__global__ void __launch_bounds__(kThreads) block_gather_kernel(const __grid_constant__ BlockMoveArgs a)
{
    pdl_wait();
    const int lane = threadIdx.x & 31, Hkv = a.st.kv_heads;
    const int64_t warp = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;   // [4 kQuads tokens][head][K or V]
    const bool is_v = warp & 1;
    const int h = (int)((warp >> 1) % Hkv);
    const int64_t t0 = (warp >> 1) / Hkv * (4 * kQuads);
    if (t0 >= a.n_tokens) return;
    const int own = lane < 4 * kQuads && t0 + lane < a.n_tokens ? slot_inside(a, (int)t0 + lane, h == 0 && !is_v) : -1;
    __nv_bfloat16 *out = (is_v ? a.v_out : a.k_out) + (t0 * Hkv + h) * kD + 4 * lane;
#pragma unroll
    for (int c = 0; c < kQuads; c++) {
        int slot[4];
        uint32_t w[4] = {0, 0, 0, 0}, e[4] = {kBExpBias, kBExpBias, kBExpBias, kBExpBias};
#pragma unroll
        for (int i = 0; i < 4; i++) slot[i] = __shfl_sync(0xffffffffu, own, 4 * c + i);
        const bool quad = slot[0] >= 0 && (slot[0] & 3) == 0 && slot[1] == slot[0] + 1 && slot[2] == slot[0] + 2 &&
                          slot[3] == slot[0] + 3;
        if (is_v && quad) {
            const uint8_t *page = a.st.pages + ((size_t)(slot[0] / kPage) * Hkv + h) * kBPageBytes;
            const uint4 x = *reinterpret_cast<const uint4 *>(page + b_v_at(slot[0] % kPage / 4, lane));
            e[0] = e[1] = e[2] = e[3] = *reinterpret_cast<const uint32_t *>(page + kBTail + 4);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
            transpose4(w);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                if (slot[i] < 0) continue;
                const uint8_t *page = a.st.pages + ((size_t)(slot[i] / kPage) * Hkv + h) * kBPageBytes;
                const int off = slot[i] % kPage;
                e[i] = *reinterpret_cast<const uint32_t *>(page + kBTail + 4 * is_v);
                if (!is_v) {
                    w[i] = *reinterpret_cast<const uint32_t *>(page + b_k_at(off, lane));
                } else {
                    const uint8_t *b = page + b_v_at(off >> 2, lane) + (off & 3);
                    w[i] = b[0] | (uint32_t)b[4] << 8 | (uint32_t)b[8] << 16 | (uint32_t)b[12] << 24;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (t0 + 4 * c + i >= a.n_tokens) break;
            const float s = power_of_two((int)min(e[i], (uint32_t)kBExpTop) - kBExpBias);
            float x[4];
            from_codes(w[i], x);
            *reinterpret_cast<uint2 *>(out + (int64_t)(4 * c + i) * Hkv * kD) = make_uint2(
                bf16x2_bits(__floats2bfloat162_rn(x[0] * s, x[1] * s)), bf16x2_bits(__floats2bfloat162_rn(x[2] * s, x[3] * s)));
        }
    }
}

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

mac_status check_config(const mac_block_config *c)
{
    if (!c) return MAC_ERR_INVALID_ARG;
    if (c->heads < 1 || c->kv_heads < 1 || c->heads % c->kv_heads || c->heads > 4096) return MAC_ERR_INVALID_ARG;
    if (c->head_dim != kD || c->page_size != kPage) return MAC_ERR_INVALID_ARG;
    if (c->max_query < 1 || (int64_t)(c->heads / c->kv_heads) * c->max_query > kQMaxRows) return MAC_ERR_INVALID_ARG;
    if (c->max_batch < 1 || c->max_batch > kQMaxBatch) return MAC_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->num_pages > (1 << 27) - 1) return MAC_ERR_INVALID_ARG;   // slots are int32
    if (!(c->sm_scale >= 0.f) || !std::isfinite(c->sm_scale)) return MAC_ERR_INVALID_ARG;
    return MAC_OK;
}

// The marks come last and have one size per page, so that handles of different
// num_pages can share a scratch.
struct Sizes {
    size_t store, part_o, part_ml, meta, err, marks, scratch;
};

Sizes sizes_of(const mac_block_config *c)
{
    Sizes z;
    z.store = (size_t)c->num_pages * c->kv_heads * kBPageBytes;
    z.part_o = 0;
    z.part_ml = align_up((size_t)kQPartRows * kD * 4);
    z.meta = z.part_ml + align_up((size_t)kQPartRows * 8);
    z.err = z.meta + align_up((size_t)kMaxCtas * sizeof(int4));
    z.marks = z.err + 256;
    z.scratch = z.marks + align_up((size_t)c->num_pages * sizeof(BlockMark));
    return z;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

}  // namespace macgpu

struct mac_block_ctx {
    mac_block_config cfg;
    QuantAttnArgs attn;     // what does not change from call to call
    BlockMark *marks = nullptr;
    int device = 0, sm_count = 0;
    const char *scratch = nullptr;
    size_t scratch_bytes = 0;
    mac_block_ctx *next = nullptr;      // live handles, under g_live_mutex
    mac_status sticky = MAC_OK;
    char errbuf[256] = {0};
};

namespace macgpu {

namespace {

// The live handles: one made on another's scratch must not clear the error
// word that they share, which may hold what nobody has read yet.
std::mutex g_live_mutex;
mac_block_ctx *g_live = nullptr;

mac_status fail_cuda(mac_block_ctx *h, cudaError_t e, const char *where)
{
    h->sticky = MAC_ERR_CUDA;
    std::snprintf(h->errbuf, sizeof h->errbuf, "%s: %s", where, cudaGetErrorString(e));
    return MAC_ERR_CUDA;
}

// A refused argument: no text of an earlier error stands for it.
mac_status refuse(mac_block_ctx *h)
{
    h->errbuf[0] = 0;
    return MAC_ERR_INVALID_ARG;
}

// The handle is usable and its device is the current one.
mac_status check_handle(mac_block_ctx *h)
{
    if (!h) return MAC_ERR_INVALID_ARG;
    if (h->sticky != MAC_OK) return h->sticky;
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail_cuda(h, e, "cudaGetDevice");
    if (dev != h->device) {
        std::snprintf(h->errbuf, sizeof h->errbuf, "the handle lives on device %d, the current device is %d", h->device, dev);
        return MAC_ERR_INVALID_ARG;
    }
    return MAC_OK;
}

BlockMoveArgs move_args(const mac_block_ctx *h, int n_tokens, const int32_t *slots)
{
    BlockMoveArgs a{};
    a.st = h->attn.st;
    a.marks = h->marks;
    a.slots = slots;
    a.n_tokens = n_tokens;
    return a;
}

}  // namespace

}  // namespace macgpu

extern "C" {

mac_status mac_block_query_sizes(const mac_block_config *cfg, size_t *store_bytes, size_t *scratch_bytes)
{
    const mac_status st = check_config(cfg);
    if (st != MAC_OK) return st;
    const Sizes z = sizes_of(cfg);
    if (store_bytes) *store_bytes = z.store;
    if (scratch_bytes) *scratch_bytes = z.scratch;
    return MAC_OK;
}

mac_status mac_block_create(const mac_block_config *cfg, void *dev_store, size_t store_bytes, void *dev_scratch,
                            size_t scratch_bytes, mac_block_handle *out)
{
    if (!out) return MAC_ERR_INVALID_ARG;
    *out = nullptr;
    const mac_status st = check_config(cfg);
    if (st != MAC_OK) return st;
    if (!dev_store || !dev_scratch) return MAC_ERR_INVALID_ARG;
    const Sizes z = sizes_of(cfg);
    if (((uintptr_t)dev_store | (uintptr_t)dev_scratch) & 255) return MAC_ERR_OOM;
    if (store_bytes < z.store || scratch_bytes < z.scratch) return MAC_ERR_OOM;
    mac_block_ctx *h = new (std::nothrow) mac_block_ctx();
    if (!h) return MAC_ERR_OOM;
    h->cfg = *cfg;
    char *sc = (char *)dev_scratch;
    QuantAttnArgs &a = h->attn;
    a = QuantAttnArgs{};
    a.st.pages = (uint8_t *)dev_store;
    a.st.num_pages = cfg->num_pages;
    a.st.kv_heads = cfg->kv_heads;
    a.st.k_scale = a.st.v_scale = a.st.k_inv = a.st.v_inv = 1.f;
    a.st.err = (uint32_t *)(sc + z.err);
    a.heads = cfg->heads;
    a.G = cfg->heads / cfg->kv_heads;
    const double scale = cfg->sm_scale > 0.f ? (double)cfg->sm_scale : 1.0 / std::sqrt((double)kD);
    a.scale_log2 = (float)(scale * 1.4426950408889634);
    a.v_out_scale = 1.f;
    a.part_o = (float *)(sc + z.part_o);
    a.part_ml = (float2 *)(sc + z.part_ml);
    a.meta = (int4 *)(sc + z.meta);
    h->marks = (BlockMark *)(sc + z.marks);

    cudaDeviceProp prop;
    bool good = cudaGetDevice(&h->device) == cudaSuccess && cudaGetDeviceProperties(&prop, h->device) == cudaSuccess;
    good = good && prop.major * 10 + prop.minor == 103;
    if (good) {
        h->sm_count = prop.multiProcessorCount;
        h->scratch = sc;
        h->scratch_bytes = z.scratch;
        std::lock_guard<std::mutex> lock(g_live_mutex);
        size_t shared = 0;              // bytes of the scratch that a live handle keeps in order
        for (const mac_block_ctx *o = g_live; o; o = o->next)
            if (o->scratch == sc && o->device == h->device && o->scratch_bytes > shared) shared = o->scratch_bytes;
        // an unwritten slot reads back as zeros; work in flight may still use a shared scratch or a recycled buffer
        good = block_attention_config(h->sm_count) == cudaSuccess && cudaDeviceSynchronize() == cudaSuccess &&
               cudaMemset(dev_store, 0, z.store) == cudaSuccess &&
               (shared >= z.scratch || cudaMemset(sc + shared, 0, z.scratch - shared) == cudaSuccess) &&
               cudaDeviceSynchronize() == cudaSuccess;
        if (good) {
            h->next = g_live;
            g_live = h;
        }
    }
    if (!good) {
        delete h;
        return MAC_ERR_CUDA;
    }
    *out = h;
    return MAC_OK;
}

mac_status mac_block_destroy(mac_block_handle h)
{
    if (!h) return MAC_ERR_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(h->device) == cudaSuccess) {
        cudaDeviceSynchronize();
        if (dev != h->device) cudaSetDevice(dev);
    }
    {
        std::lock_guard<std::mutex> lock(g_live_mutex);
        for (mac_block_ctx **p = &g_live; *p; p = &(*p)->next)
            if (*p == h) {
                *p = h->next;
                break;
            }
    }
    delete h;
    return MAC_OK;
}

const char *mac_block_last_error(mac_block_handle h) { return h ? h->errbuf : ""; }

mac_status mac_block_append(mac_block_handle h, int n_tokens, const void *dev_k, int64_t k_stride, const void *dev_v,
                            int64_t v_stride, const int32_t *dev_slots, void *stream)
{
    const mac_status st = check_handle(h);
    if (st != MAC_OK) return st;
    if (n_tokens < 0) return refuse(h);
    if (n_tokens == 0) return MAC_OK;
    const int64_t row = (int64_t)h->cfg.kv_heads * kD;
    if (!dev_k || !dev_v || !dev_slots || !aligned16(dev_k) || !aligned16(dev_v) || ((uintptr_t)dev_slots & 3))
        return refuse(h);
    if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8) return refuse(h);
    if ((int64_t)n_tokens * h->cfg.kv_heads > (1 << 30)) return refuse(h);
    BlockMoveArgs a = move_args(h, n_tokens, dev_slots);
    a.k = (const __nv_bfloat16 *)dev_k;
    a.v = (const __nv_bfloat16 *)dev_v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    cudaError_t e;
    if (n_tokens <= kScanTokens) {
        e = launch_maybe_pdl(block_append_scan_kernel, dim3(n_tokens, (2 * h->cfg.kv_heads * 32 + kThreads - 1) / kThreads), dim3(kThreads), 0,
                             (cudaStream_t)stream, true, a);
    } else {
        e = launch_maybe_pdl(block_mark_kernel, dim3((n_tokens + kThreads - 1) / kThreads), dim3(kThreads), 0,
                             (cudaStream_t)stream, true, a);
        int tokens = 1;
        while (tokens < kMostTokens && n_tokens / tokens > kBlocksPerSm * h->sm_count) tokens *= 2;
        if (e == cudaSuccess)
            e = launch_maybe_pdl(block_append_kernel, dim3((n_tokens + tokens - 1) / tokens), dim3(kThreads), 0,
                                 (cudaStream_t)stream, true, a, tokens);
    }
    return e == cudaSuccess ? MAC_OK : fail_cuda(h, e, "append launch");
}

mac_status mac_block_gather(mac_block_handle h, int n_tokens, const int32_t *dev_slots, void *dev_k, void *dev_v,
                            void *stream)
{
    const mac_status st = check_handle(h);
    if (st != MAC_OK) return st;
    if (n_tokens < 0) return refuse(h);
    if (n_tokens == 0) return MAC_OK;
    if (!dev_k || !dev_v || !dev_slots || !aligned16(dev_k) || !aligned16(dev_v) || ((uintptr_t)dev_slots & 3))
        return refuse(h);
    if ((int64_t)n_tokens * h->cfg.kv_heads > (1 << 30)) return refuse(h);
    BlockMoveArgs a = move_args(h, n_tokens, dev_slots);
    a.k_out = (__nv_bfloat16 *)dev_k;
    a.v_out = (__nv_bfloat16 *)dev_v;
    const bool small = (int64_t)n_tokens * h->cfg.kv_heads < kSmallGather;
    const int tokens = small ? 4 : 16;
    const int64_t warps = 2 * (((int64_t)n_tokens + tokens - 1) / tokens) * h->cfg.kv_heads;
    const cudaError_t e = launch_maybe_pdl(small ? block_gather_kernel<1> : block_gather_kernel<4>,
                                           dim3((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32))), dim3(kThreads), 0,
                                           (cudaStream_t)stream, true, a);
    return e == cudaSuccess ? MAC_OK : fail_cuda(h, e, "gather launch");
}

mac_status mac_block_attention(mac_block_handle h, int batch, int n_query, const void *dev_q, const int32_t *dev_table,
                               int64_t table_stride, int table_cols, const int32_t *dev_lens, void *dev_out,
                               float *dev_lse, void *stream)
{
    const mac_status st = check_handle(h);
    if (st != MAC_OK) return st;
    if (batch < 0 || batch > h->cfg.max_batch || n_query < 1 || n_query > h->cfg.max_query) return refuse(h);
    if (batch == 0) return MAC_OK;
    if (!dev_q || !dev_table || !dev_lens || !dev_out || !aligned16(dev_q) || !aligned16(dev_out) ||
        (((uintptr_t)dev_table | (uintptr_t)dev_lens | (uintptr_t)dev_lse) & 3))
        return refuse(h);
    if (table_cols < 1 || table_cols > (1 << 26) || table_stride < table_cols) return refuse(h);
    QuantAttnArgs a = h->attn;
    a.n_query = n_query;
    a.rows = a.G * n_query;
    a.batch = batch;
    a.q = (const __nv_bfloat16 *)dev_q;
    a.table = dev_table;
    a.table_stride = table_stride;
    a.table_cols = table_cols;
    a.lens = dev_lens;
    a.out = (__nv_bfloat16 *)dev_out;
    a.lse = dev_lse;
    const cudaError_t e = launch_block_attention(a, h->sm_count, (cudaStream_t)stream);
    return e == cudaSuccess ? MAC_OK : fail_cuda(h, e, "attention launch");
}

mac_status mac_block_step_rows(mac_block_handle h, int batch, int n_query, int n_packed, const int32_t *dev_starts,
                               const int32_t *dev_pos, const int32_t *dev_slots, const int32_t *dev_table,
                               int64_t table_stride, int table_cols, const int32_t *dev_lens, int32_t *dev_pos_out,
                               int32_t *dev_slots_out, int32_t *dev_lens_out, void *stream)
{
    const mac_status st = check_handle(h);
    if (st != MAC_OK) return st;
    if (batch < 0 || batch > h->cfg.max_batch || n_query < 1 || n_query > h->cfg.max_query || n_packed < 0) return refuse(h);
    if (batch == 0) return MAC_OK;
    const StepRowArgs a{batch,    n_query,  n_packed, table_cols,  table_stride,  dev_starts,   dev_pos,  dev_slots,
                        dev_table, dev_lens, dev_pos_out, dev_slots_out, dev_lens_out, h->attn.st.err};
    if (!step_row_args_good(a)) return refuse(h);
    const cudaError_t e = launch_step_rows(a, (cudaStream_t)stream);
    return e == cudaSuccess ? MAC_OK : fail_cuda(h, e, "step rows launch");
}

mac_status mac_block_sync(mac_block_handle h)
{
    const mac_status st = check_handle(h);
    if (st != MAC_OK) return st;
    cudaError_t e = cudaDeviceSynchronize();
    uint32_t bits = 0;
    if (e == cudaSuccess) e = cudaMemcpy(&bits, h->attn.st.err, 4, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && bits) e = cudaMemset(h->attn.st.err, 0, 4);
    if (e != cudaSuccess) return fail_cuda(h, e, "mac_block_sync");
    h->errbuf[0] = 0;
    if (!bits) return MAC_OK;
    quant_error_text(bits, h->errbuf, sizeof h->errbuf);
    return MAC_ERR_STATE;
}

}  // extern "C"
