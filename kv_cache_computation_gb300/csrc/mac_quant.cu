// The 4-bit KV store (layout and format: mac_quant.cuh): its handle, the
// append that quantises new tokens into it by their slots, the gather that
// reads tokens back, and the layout of a step's packed tokens as rows.
//
// Append, per block of 16 elements x of a head (all exact in fp32 but the two
// roundings the format itself makes):
//   s = e4m3(max|x| / 6), code_i = e2m1(x_i / s)
// The quotient is formed as x * (1 / s), rounded to a multiple of 2^-13 before
// the conversion.  A tie between two e2m1 values is x = t s with t in {0.25,
// ..., 5}; x has 8 significant bits and t s at most 7, so a quotient that is no
// tie is off it by at least 2^-9 of it (2^-11), while x * (1 / s) is within
// 2^-22 of it: the rounding puts ties back on the tie and moves nothing across
// one.  A division per element would cost more than the rest of the kernel.
//
// What bounds them, 32768 tokens of 8 heads: the append (134 MB in, 38 MB out)
// 32 us, 5.4 TB/s, the loads' latency at half occupancy (four tokens' blocks
// per lane; three or six blocks per SM instead of four: 36 and 40 us); the gather
// (38 MB in, 134 MB out) 34 us, 4.0 TB/s of writes, which is what a plain fill
// reaches (4.03).  8 tokens: 1.7 and 1.5 us in a captured graph, launch and latency.
#include "../../include/mac.h"
#include "mac_device.cuh"
#include "mac_quant.cuh"

#include <cuda_fp16.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <new>

using namespace macgpu;

namespace macgpu {

namespace {

constexpr int kThreads = 256;
// From this many (token, head) pairs on a lane takes four tokens; below, one
// block per lane spreads further.  Both sides, us, append of 8 heads: 512 tokens
// 2.3 (one block) against 3.0, 1024 2.7 / 3.0, 2048 4.1 / 3.9, 8192 9.8 / 7.8,
// 32768 38 / 32 (gather: 512 3.0 / 3.4, 8192 11.3 / 11.4, 32768 36 / 34).
constexpr int64_t kQuadPairs = 16384;

// two e2m1 codes (lo in the low four bits) of two floats, ties to even, at most 6
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n.reg .b8 t;\ncvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\ncvt.u32.u8 %0, t;\n}\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// the e4m3 byte of one float, ties to even, at most 448
__device__ __forceinline__ uint32_t to_e4m3(float x)
{
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xff;
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two)
{
    uint32_t r;
    const unsigned short h = (unsigned short)two;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(r) : "h"(h));
    return r;
}

// The sixteen elements (as two 16-byte loads) of one block -> scale byte and
// eight bytes of codes.  inv: 1 / the store's global scale.
__device__ __forceinline__ void quantise(const uint4 (&u)[2], float inv, uint32_t &scale, uint2 &codes)
{
    uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
    // largest magnitude pattern: its order is that of the magnitudes, NaN above infinity
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; i++) m[i] = w[i] & 0x7fff7fffu;
    const uint32_t two = __vimax3_s16x2(__vimax3_s16x2(m[0], m[1], m[2]), __vimax3_s16x2(m[3], m[4], m[5]),
                                        __vmaxs2(m[6], m[7]));
    const uint32_t top = max(two & 0xffffu, two >> 16);
    scale = 0xff;       // NaN
    codes = make_uint2(0, 0);
    if (top >= 0x7f80u) return;
    const float want = __uint_as_float(top << 16) * inv / 6.f;
    scale = to_e4m3(want);
    if (scale == 0) return;
    const uint32_t sh = e4m3x2_to_f16x2(scale);
    const float s = __low2float(*reinterpret_cast<const __half2 *>(&sh));
    const float r = inv / s;
    if (want > 500.f) {
        // the scale has saturated: what lies beyond 8 s, and ends as 6 s, could leave the range of the rounding below
        const __nv_bfloat162 lim = __float2bfloat162_rn(8.f * s / inv);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(&w[i]);
            w[i] = bf16x2_bits(__hmax2(__hmin2(x, lim), __hneg2(lim)));
        }
    }
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        // x / s to a multiple of 2^-13: an fma onto 1.5 x 2^10, whose last bit that is, and back (|x / s| is at most 12:
        // s is at least 15/16 of max / 6, or half of it among the smallest scales)
        const float lo = __fsub_rn(__fmaf_rn(__uint_as_float(w[i] << 16), r, 1536.f), 1536.f);
        const float hi = __fsub_rn(__fmaf_rn(__uint_as_float(w[i] & 0xffff0000u), r, 1536.f), 1536.f);
        b[i] = to_e2m1x2(lo, hi);
    }
    codes.x = b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
    codes.y = b[4] | b[5] << 8 | b[6] << 16 | b[7] << 24;
}

struct MoveArgs {
    QuantStore st;
    const __nv_bfloat16 *k, *v;         // append: sources with a token stride
    int64_t k_stride, v_stride;
    __nv_bfloat16 *k_out, *v_out;       // gather: dense destinations
    const int32_t *slots;
    int64_t rows;                       // 2 x tokens x kv_heads
    int n_tokens;
};

// Writes one block of one token: eight bytes of codes and the scale byte.
__device__ __forceinline__ void put_block(uint8_t *page, bool is_v, int tok, int j, uint2 codes, uint32_t scale)
{
    if (!is_v) {
        *reinterpret_cast<uint2 *>(page + tok * (kD / 2) + j * 8) = codes;
        page[q_kscale_at(tok, j)] = (uint8_t)scale;
    } else {
        *reinterpret_cast<uint32_t *>(page + q_v_at(tok, j, 0)) = codes.x;
        *reinterpret_cast<uint32_t *>(page + q_v_at(tok, j, 1)) = codes.y;
        page[q_vscale_at(tok, j)] = (uint8_t)scale;
    }
}

__device__ __forceinline__ void get_block(const uint8_t *page, bool is_v, int tok, int j, uint2 &codes, uint32_t &scale)
{
    if (!is_v) {
        codes = *reinterpret_cast<const uint2 *>(page + tok * (kD / 2) + j * 8);
        scale = page[q_kscale_at(tok, j)];
    } else {
        codes = make_uint2(*reinterpret_cast<const uint32_t *>(page + q_v_at(tok, j, 0)),
                           *reinterpret_cast<const uint32_t *>(page + q_v_at(tok, j, 1)));
        scale = page[q_vscale_at(tok, j)];
    }
}

__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n.reg .b8 a, b, c, d;\nmov.b32 {a, b, c, d}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, a;\ncvt.rn.f16x2.e2m1x2 %1, b;\ncvt.rn.f16x2.e2m1x2 %2, c;\ncvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// four codes' bf16 values, times the block's scale (exact in both)
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t h, float s)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return bf16x2_bits(__floats2bfloat162_rn(f.x * s, f.y * s));
}

// A block's sixteen values as bf16.
__device__ __forceinline__ void write_block(__nv_bfloat16 *out, uint2 codes, uint32_t scale, float global)
{
    const uint32_t sh = e4m3x2_to_f16x2(scale);
    const float s = __low2float(*reinterpret_cast<const __half2 *>(&sh)) * global;
    uint32_t x[4], y[4];
    e2m1x8_to_f16(codes.x, x);
    e2m1x8_to_f16(codes.y, y);
    reinterpret_cast<uint4 *>(out)[0] = make_uint4(scaled_bf16x2(x[0], s), scaled_bf16x2(x[1], s),
                                                   scaled_bf16x2(x[2], s), scaled_bf16x2(x[3], s));
    reinterpret_cast<uint4 *>(out)[1] = make_uint4(scaled_bf16x2(y[0], s), scaled_bf16x2(y[1], s),
                                                   scaled_bf16x2(y[2], s), scaled_bf16x2(y[3], s));
}

// The token's slot, or -1 where it has none or one outside the store.
__device__ __forceinline__ int slot_of(const MoveArgs &a, int t, bool report)
{
    const int slot = a.slots[t];
    if (slot >= 0 && slot / kPage >= a.st.num_pages) {
        if (report) atomicOr(a.st.err, kQErrSlot);
        return -1;
    }
    return slot < 0 ? -1 : slot;
}

__device__ __forceinline__ uint8_t *page_at(const MoveArgs &a, int slot, int h)
{
    return a.st.pages + ((size_t)(slot / kPage) * a.st.kv_heads + h) * kQPageBytes;
}

// Few tokens: a row (token, K or V, head) per eight lanes, a block per lane.
template <bool kGather>
__global__ void __launch_bounds__(kThreads) quant_rows_kernel(const __grid_constant__ MoveArgs a)
{
    pdl_wait();
    const int j = threadIdx.x & 7, Hkv = a.st.kv_heads;
    const int64_t row = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 3;
    if (row >= a.rows) return;
    const int h = (int)(row % Hkv);
    const int64_t r2 = row / Hkv;
    const bool is_v = r2 & 1;
    const int t = (int)(r2 >> 1);
    const int slot = slot_of(a, t, j == 0);
    uint32_t scale = 0;
    uint2 codes = make_uint2(0, 0);
    if (kGather) {
        if (slot >= 0) get_block(page_at(a, slot, h), is_v, slot % kPage, j, codes, scale);
        write_block((is_v ? a.v_out : a.k_out) + ((int64_t)t * Hkv + h) * kD + j * kQBlock, codes, scale,
                    is_v ? a.st.v_scale : a.st.k_scale);
    } else if (slot >= 0) {
        const __nv_bfloat16 *x = (is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + h * kD + j * kQBlock;
        const uint4 u[2] = {reinterpret_cast<const uint4 *>(x)[0], reinterpret_cast<const uint4 *>(x)[1]};
        quantise(u, is_v ? a.st.v_inv : a.st.k_inv, scale, codes);
        put_block(page_at(a, slot, h), is_v, slot % kPage, j, codes, scale);
    }
}

// Many tokens: a warp takes 16 consecutive tokens of one head and K or V, lane
// (c, j) block j of the tokens 4 c .. 4 c + 3.  Where those four are an aligned
// quad of a page (as a prefill's are), their scales are one word and their
// value codes two 16-byte vectors, and a warp's stores cover whole sectors;
// elsewhere each token goes by itself, as above.
template <bool kGather>
__global__ void __launch_bounds__(kThreads, 4) quant_quads_kernel(const __grid_constant__ MoveArgs a)
{
    pdl_wait();
    const int lane = threadIdx.x & 31, j = lane & 7, c = lane >> 3, Hkv = a.st.kv_heads;
    const int64_t warp = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;   // [16 tokens][K or V][head]
    const int h = (int)(warp % Hkv);
    const int64_t r2 = warp / Hkv;
    const bool is_v = r2 & 1;
    const int t0 = (int)(r2 >> 1) * kPage + 4 * c;
    if (t0 >= a.n_tokens) return;
    int slot[4];
#pragma unroll
    for (int i = 0; i < 4; i++) slot[i] = t0 + i < a.n_tokens ? slot_of(a, t0 + i, j == 0) : -1;
    const bool quad = slot[0] >= 0 && (slot[0] & 3) == 0 && slot[1] == slot[0] + 1 && slot[2] == slot[0] + 2 &&
                      slot[3] == slot[0] + 3;
    const float global = is_v ? a.st.v_scale : a.st.k_scale, inv = is_v ? a.st.v_inv : a.st.k_inv;
    uint2 codes[4];
    uint32_t scale[4];
    if (kGather) {
        __nv_bfloat16 *out = (is_v ? a.v_out : a.k_out) + ((int64_t)t0 * Hkv + h) * kD + j * kQBlock;
        if (quad) {
            const uint8_t *page = page_at(a, slot[0], h);
            const int tok = slot[0] % kPage;
            const uint32_t sw = *reinterpret_cast<const uint32_t *>(page + (is_v ? q_vscale_at(tok, j) : q_kscale_at(tok, j)));
            if (is_v) {
                const uint4 x = *reinterpret_cast<const uint4 *>(page + q_v_at(tok, j, 0));
                const uint4 y = *reinterpret_cast<const uint4 *>(page + q_v_at(tok, j, 1));
                codes[0] = make_uint2(x.x, y.x);
                codes[1] = make_uint2(x.y, y.y);
                codes[2] = make_uint2(x.z, y.z);
                codes[3] = make_uint2(x.w, y.w);
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++) codes[i] = *reinterpret_cast<const uint2 *>(page + (tok + i) * (kD / 2) + j * 8);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) scale[i] = sw >> 8 * (is_v ? q_scale_byte(i) : i) & 0xff;
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                codes[i] = make_uint2(0, 0);
                scale[i] = 0;
                if (slot[i] >= 0) get_block(page_at(a, slot[i], h), is_v, slot[i] % kPage, j, codes[i], scale[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (t0 + i < a.n_tokens) write_block(out + (int64_t)i * Hkv * kD, codes[i], scale[i], global);
    } else {
        const __nv_bfloat16 *src = is_v ? a.v : a.k;
        const int64_t stride = is_v ? a.v_stride : a.k_stride;
        uint4 u[4][2];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint4 *x = reinterpret_cast<const uint4 *>(src + (t0 + i) * stride + h * kD + j * kQBlock);
            if (slot[i] >= 0) {
                u[i][0] = x[0];
                u[i][1] = x[1];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (slot[i] >= 0) quantise(u[i], inv, scale[i], codes[i]);
        if (quad) {
            uint8_t *page = page_at(a, slot[0], h);
            const int tok = slot[0] % kPage;
            if (is_v) {
                *reinterpret_cast<uint4 *>(page + q_v_at(tok, j, 0)) = make_uint4(codes[0].x, codes[1].x, codes[2].x, codes[3].x);
                *reinterpret_cast<uint4 *>(page + q_v_at(tok, j, 1)) = make_uint4(codes[0].y, codes[1].y, codes[2].y, codes[3].y);
                *reinterpret_cast<uint32_t *>(page + q_vscale_at(tok, j)) =
                    scale[0] | scale[2] << 8 | scale[1] << 16 | scale[3] << 24;
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++) *reinterpret_cast<uint2 *>(page + (tok + i) * (kD / 2) + j * 8) = codes[i];
                *reinterpret_cast<uint32_t *>(page + q_kscale_at(tok, j)) =
                    scale[0] | scale[1] << 8 | scale[2] << 16 | scale[3] << 24;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (slot[i] >= 0) put_block(page_at(a, slot[i], h), is_v, slot[i] % kPage, j, codes[i], scale[i]);
        }
    }
}

struct RowArgs {
    int batch, n_query, n_packed, table_cols;
    int64_t table_stride;
    const int32_t *starts, *pos, *slots, *table, *lens;
    int32_t *pos_out, *slots_out, *lens_out;
    uint32_t *err;
};

// Packed new tokens laid out as n_query rows per request, a warp per request
// and a lane per row.  A request's rows count only if it has exactly n_query
// packed tokens and each of their slots is the one that its own table gives the
// last n_query tokens of its length, which is where the attention reads them.
// Three dependent reads behind the launch: 1.5 us (1 request) to 1.8 (1024) in a
// captured graph.
__global__ void __launch_bounds__(kThreads) step_rows_kernel(const __grid_constant__ RowArgs a)
{
    pdl_wait();
    const int lane = threadIdx.x & 31, b = (int)((blockIdx.x * kThreads + threadIdx.x) >> 5), nq = a.n_query;
    if (b >= a.batch) return;
    const long long len = a.lens[b], first = a.starts ? a.starts[b] : (long long)b * nq;
    const long long n = a.starts ? a.starts[b + 1] - first : nq;
    const bool inside = n == nq && first >= 0 && first + nq <= a.n_packed;
    const bool row = lane < nq;
    const int slot = inside && row ? a.slots[first + lane] : -1;
    const long long p = len - nq + lane;
    bool own = false;
    if (slot >= 0 && p >= 0 && p < (long long)a.table_cols * kPage)
        own = slot == (long long)a.table[b * a.table_stride + p / kPage] * kPage + p % kPage;
    const bool keep = __popc(__ballot_sync(0xffffffffu, own)) == nq;
    const bool some = __any_sync(0xffffffffu, slot >= 0);
    if (row) {
        a.pos_out[b * nq + lane] = keep ? a.pos[first + lane] : 0;
        a.slots_out[b * nq + lane] = keep ? slot : -1;
    }
    if (lane == 0) {
        a.lens_out[b] = keep ? (int)len : 0;
        // no token at all is an idle request, no slot at all one that got no page
        if (!keep && (some || (n != 0 && !inside))) atomicOr(a.err, kQErrRow);
    }
}

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

bool power_of_two(float x)
{
    int e;
    return std::isfinite(x) && x > 0.f && std::frexp(x, &e) == 0.5f && e > -60 && e <= 60;
}

mac_status check_config(const mac_quant_config *c)
{
    if (!c) return MAC_ERR_INVALID_ARG;
    if (c->heads < 1 || c->kv_heads < 1 || c->heads % c->kv_heads || c->heads > 4096) return MAC_ERR_INVALID_ARG;
    if (c->head_dim != kD || c->page_size != kPage) return MAC_ERR_INVALID_ARG;
    if (c->max_query < 1 || (int64_t)(c->heads / c->kv_heads) * c->max_query > kQMaxRows) return MAC_ERR_INVALID_ARG;
    if (c->max_batch < 1 || c->max_batch > kQMaxBatch) return MAC_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->num_pages > (1 << 27) - 1) return MAC_ERR_INVALID_ARG;   // slots are int32
    if (!(c->sm_scale >= 0.f) || !std::isfinite(c->sm_scale)) return MAC_ERR_INVALID_ARG;
    if (!power_of_two(c->k_scale) || !power_of_two(c->v_scale)) return MAC_ERR_INVALID_ARG;
    return MAC_OK;
}

struct Sizes {
    size_t store, part_o, part_ml, meta, err, scratch;
};

Sizes sizes_of(const mac_quant_config *c)
{
    Sizes z;
    z.store = (size_t)c->num_pages * c->kv_heads * kQPageBytes;
    z.part_o = 0;
    z.part_ml = align_up((size_t)kQPartRows * kD * 4);
    z.meta = z.part_ml + align_up((size_t)kQPartRows * 8);
    z.err = z.meta + align_up((size_t)kMaxCtas * sizeof(int4));
    z.scratch = z.err + 256;
    return z;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

}  // namespace macgpu

struct mac_quant_ctx {
    mac_quant_config cfg;
    QuantStore st;
    QuantAttnArgs attn;     // what does not change from call to call
    int device = 0, sm_count = 0;
    const void *scratch = nullptr;
    mac_quant_ctx *next = nullptr;      // live handles, under g_live_mutex
    mac_status sticky = MAC_OK;
    char errbuf[256] = {0};
};

namespace macgpu {

namespace {

// The live handles: one made on another's scratch must not clear the error
// word that they share, which may hold what nobody has read yet.
std::mutex g_live_mutex;
mac_quant_ctx *g_live = nullptr;

mac_status fail_cuda(mac_quant_ctx *h, cudaError_t e, const char *where)
{
    h->sticky = MAC_ERR_CUDA;
    std::snprintf(h->errbuf, sizeof h->errbuf, "%s: %s", where, cudaGetErrorString(e));
    return MAC_ERR_CUDA;
}

// A refused argument: no text of an earlier error stands for it.
mac_status refuse(mac_quant_ctx *h)
{
    h->errbuf[0] = 0;
    return MAC_ERR_INVALID_ARG;
}

// The handle is usable and its device is the current one.
mac_status check_handle(mac_quant_ctx *h)
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

mac_status launch_move(mac_quant_ctx *h, bool gather, MoveArgs a, void *stream)
{
    a.st = h->st;
    const int Hkv = h->cfg.kv_heads;
    a.rows = 2 * (int64_t)a.n_tokens * Hkv;
    const bool quads = (int64_t)a.n_tokens * Hkv >= kQuadPairs;
    const int64_t threads = quads ? 2 * ((int64_t)(a.n_tokens + kPage - 1) / kPage) * Hkv * 32 : a.rows * 8;
    const auto kernel = quads ? (gather ? quant_quads_kernel<true> : quant_quads_kernel<false>)
                              : (gather ? quant_rows_kernel<true> : quant_rows_kernel<false>);
    const cudaError_t e = launch_maybe_pdl(kernel, dim3((unsigned)((threads + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                                           (cudaStream_t)stream, true, a);
    return e == cudaSuccess ? MAC_OK : fail_cuda(h, e, gather ? "gather launch" : "append launch");
}

}  // namespace

}  // namespace macgpu

extern "C" {

mac_status mac_quant_query_sizes(const mac_quant_config *cfg, size_t *store_bytes, size_t *scratch_bytes)
{
    const mac_status st = check_config(cfg);
    if (st != MAC_OK) return st;
    const Sizes z = sizes_of(cfg);
    if (store_bytes) *store_bytes = z.store;
    if (scratch_bytes) *scratch_bytes = z.scratch;
    return MAC_OK;
}

mac_status mac_quant_create(const mac_quant_config *cfg, void *dev_store, size_t store_bytes, void *dev_scratch,
                            size_t scratch_bytes, mac_quant_handle *out)
{
    if (!out) return MAC_ERR_INVALID_ARG;
    *out = nullptr;
    const mac_status st = check_config(cfg);
    if (st != MAC_OK) return st;
    if (!dev_store || !dev_scratch) return MAC_ERR_INVALID_ARG;
    const Sizes z = sizes_of(cfg);
    if (((uintptr_t)dev_store | (uintptr_t)dev_scratch) & 255) return MAC_ERR_OOM;
    if (store_bytes < z.store || scratch_bytes < z.scratch) return MAC_ERR_OOM;
    mac_quant_ctx *h = new (std::nothrow) mac_quant_ctx();
    if (!h) return MAC_ERR_OOM;
    h->cfg = *cfg;
    char *sc = (char *)dev_scratch;
    h->st.pages = (uint8_t *)dev_store;
    h->st.num_pages = cfg->num_pages;
    h->st.kv_heads = cfg->kv_heads;
    h->st.k_scale = cfg->k_scale;
    h->st.v_scale = cfg->v_scale;
    h->st.k_inv = 1.f / cfg->k_scale;
    h->st.v_inv = 1.f / cfg->v_scale;
    h->st.err = (uint32_t *)(sc + z.err);
    QuantAttnArgs &a = h->attn;
    a = QuantAttnArgs{};
    a.st = h->st;
    a.heads = cfg->heads;
    a.G = cfg->heads / cfg->kv_heads;
    const double scale = cfg->sm_scale > 0.f ? (double)cfg->sm_scale : 1.0 / std::sqrt((double)kD);
    a.scale_log2 = (float)(scale * 1.4426950408889634 * cfg->k_scale * 256.0);
    a.v_out_scale = cfg->v_scale * 256.f;
    a.part_o = (float *)(sc + z.part_o);
    a.part_ml = (float2 *)(sc + z.part_ml);
    a.meta = (int4 *)(sc + z.meta);

    cudaDeviceProp prop;
    bool good = cudaGetDevice(&h->device) == cudaSuccess && cudaGetDeviceProperties(&prop, h->device) == cudaSuccess;
    good = good && prop.major * 10 + prop.minor == 103;
    if (good) {
        h->sm_count = prop.multiProcessorCount;
        h->scratch = dev_scratch;
        std::lock_guard<std::mutex> lock(g_live_mutex);
        bool shared = false;
        for (const mac_quant_ctx *o = g_live; o; o = o->next) shared |= o->scratch == dev_scratch && o->device == h->device;
        // an unwritten slot reads back as zeros; work in flight may still use a shared scratch or a recycled buffer
        good = quant_attention_config(h->sm_count) == cudaSuccess && cudaDeviceSynchronize() == cudaSuccess &&
               cudaMemset(dev_store, 0, z.store) == cudaSuccess &&
               (shared || cudaMemset(dev_scratch, 0, z.scratch) == cudaSuccess) && cudaDeviceSynchronize() == cudaSuccess;
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

mac_status mac_quant_destroy(mac_quant_handle h)
{
    if (!h) return MAC_ERR_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(h->device) == cudaSuccess) {
        cudaDeviceSynchronize();
        if (dev != h->device) cudaSetDevice(dev);
    }
    {
        std::lock_guard<std::mutex> lock(g_live_mutex);
        for (mac_quant_ctx **p = &g_live; *p; p = &(*p)->next)
            if (*p == h) {
                *p = h->next;
                break;
            }
    }
    delete h;
    return MAC_OK;
}

const char *mac_quant_last_error(mac_quant_handle h) { return h ? h->errbuf : ""; }

mac_status mac_quant_append(mac_quant_handle h, int n_tokens, const void *dev_k, int64_t k_stride, const void *dev_v,
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
    MoveArgs a{};
    a.k = (const __nv_bfloat16 *)dev_k;
    a.v = (const __nv_bfloat16 *)dev_v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.slots = dev_slots;
    a.n_tokens = n_tokens;
    return launch_move(h, false, a, stream);
}

mac_status mac_quant_gather(mac_quant_handle h, int n_tokens, const int32_t *dev_slots, void *dev_k, void *dev_v,
                            void *stream)
{
    const mac_status st = check_handle(h);
    if (st != MAC_OK) return st;
    if (n_tokens < 0) return refuse(h);
    if (n_tokens == 0) return MAC_OK;
    if (!dev_k || !dev_v || !dev_slots || !aligned16(dev_k) || !aligned16(dev_v) || ((uintptr_t)dev_slots & 3))
        return refuse(h);
    if ((int64_t)n_tokens * h->cfg.kv_heads > (1 << 30)) return refuse(h);
    MoveArgs a{};
    a.k_out = (__nv_bfloat16 *)dev_k;
    a.v_out = (__nv_bfloat16 *)dev_v;
    a.slots = dev_slots;
    a.n_tokens = n_tokens;
    return launch_move(h, true, a, stream);
}

mac_status mac_quant_attention(mac_quant_handle h, int batch, int n_query, const void *dev_q, const int32_t *dev_table,
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
    const cudaError_t e = launch_quant_attention(a, h->sm_count, (cudaStream_t)stream);
    return e == cudaSuccess ? MAC_OK : fail_cuda(h, e, "attention launch");
}

mac_status mac_quant_step_rows(mac_quant_handle h, int batch, int n_query, int n_packed, const int32_t *dev_starts,
                               const int32_t *dev_pos, const int32_t *dev_slots, const int32_t *dev_table,
                               int64_t table_stride, int table_cols, const int32_t *dev_lens, int32_t *dev_pos_out,
                               int32_t *dev_slots_out, int32_t *dev_lens_out, void *stream)
{
    const mac_status st = check_handle(h);
    if (st != MAC_OK) return st;
    if (batch < 0 || batch > h->cfg.max_batch || n_query < 1 || n_query > h->cfg.max_query || n_packed < 0) return refuse(h);
    if (batch == 0) return MAC_OK;
    const void *need[] = {dev_pos, dev_slots, dev_table, dev_lens, dev_pos_out, dev_slots_out, dev_lens_out};
    for (const void *x : need)
        if (!x || ((uintptr_t)x & 3)) return refuse(h);
    if ((uintptr_t)dev_starts & 3) return refuse(h);
    if (!dev_starts && n_packed < batch * n_query) return refuse(h);
    if (table_cols < 1 || table_cols > (1 << 26) || table_stride < table_cols) return refuse(h);
    const RowArgs a{batch,    n_query,  n_packed, table_cols,  table_stride,  dev_starts,   dev_pos,  dev_slots,
                    dev_table, dev_lens, dev_pos_out, dev_slots_out, dev_lens_out, h->st.err};
    const cudaError_t e = launch_maybe_pdl(step_rows_kernel, dim3((batch * 32 + kThreads - 1) / kThreads), dim3(kThreads), 0,
                                           (cudaStream_t)stream, true, a);
    return e == cudaSuccess ? MAC_OK : fail_cuda(h, e, "step rows launch");
}

mac_status mac_quant_sync(mac_quant_handle h)
{
    mac_status st = check_handle(h);
    if (st != MAC_OK) return st;
    cudaError_t e = cudaDeviceSynchronize();
    uint32_t bits = 0;
    if (e == cudaSuccess) e = cudaMemcpy(&bits, h->st.err, 4, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && bits) e = cudaMemset(h->st.err, 0, 4);
    if (e != cudaSuccess) return fail_cuda(h, e, "mac_quant_sync");
    h->errbuf[0] = 0;
    if (!bits) return MAC_OK;
    std::snprintf(h->errbuf, sizeof h->errbuf, "device checks met:%s%s%s%s%s", bits & kQErrPage ? " a page outside the pool" : "",
                  bits & kQErrSlot ? " a slot outside the pool" : "",
                  bits & kQErrLen ? " a length outside the page table" : "",
                  bits & kQErrTimeout ? " a copy that did not arrive" : "",
                  bits & kQErrRow ? " a request whose new tokens are not its rows of the step" : "");
    return MAC_ERR_STATE;
}

}  // extern "C"
