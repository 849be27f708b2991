// A QKV projection's rows made ready for a decode step, in one pass: per-head
// RMS norm of queries and keys, the rotary embedding, and the split into the
// dense tensors the attention entry points take.
//
// Per token and head (x the head's 128 elements, w the norm's weight):
//   y      = x / sqrt(mean(x^2) + eps) * w          (y = x without a weight)
//   q_pre  = y                                      (what Match compares)
//   q_post = R(pos) y,  k_out = R(pos) y,  v_out = x
// with R the rotation of the pairs (a, b) of the first r elements by
// t = pos * base^(-2 i / r): (a cos t - b sin t, b cos t + a sin t).  All of it
// is held in fp32 and each output is rounded to bf16 once, from fp32 (q_post
// is rotated from the unrounded y, not from q_pre).
//
// Angles: a float product pos * freq is off by up to 2^-24 of the angle, which
// is 0.008 rad at position 131072, so the angle is formed in whole turns as a
// 64-bit fixed-point fraction: turns[i] = 2^64 base^(-2 i / r) / 2 pi, and
// pos * turns[i] mod 2^64 drops the whole turns exactly for any position.
//
// What bounds it: many tokens, the memory (256 B in and 256 to 512 B out per
// row, nothing read twice); few tokens, the launch and one round trip.  A row
// belongs to 8 (or 16) lanes: a lane holds the two chunks whose elements
// rotate with each other, so the rotation needs no shuffle and the mean of
// squares three or four.  A block takes four tokens and first makes their
// sines and cosines (one sincospi per thread), which all their heads share; a
// thread stays with one token and keeps its part in registers.  Few tokens
// spread over more blocks (gridDim.y splits a token's rows), so that each row of
// lanes has one to three rows and one token's latency is a single row's.
// Measured, 32 over 8 heads with norms and pre-rotation queries: 1 token 2.1 us,
// 37 tokens 2.2, 600 tokens 4.0 (in a captured graph); 32768 tokens 176 us, 6.1
// TB/s, of which 671 MB are writes at 3.8 TB/s (a plain fill reaches 4.03).  8-byte chunks with the sines read from shared memory per row took 195 us;
// two rows in flight per lane at three blocks per SM beat one (190 us), three
// (182, two blocks) and six (245).
#include "../../include/mac.h"
#include "mac_device.cuh"

#include <cmath>

using namespace macgpu;

namespace macgpu {

namespace {

constexpr int kThreads = 256;
constexpr int kPairs = kD / 2;
// A block takes four tokens from kTileRows tokens per row of a token on.  Both
// sides, us: 48 rows: 608 tokens 4.7 (one token per block) against 5.5, 2048
// 13.9 / 15.2, 3000 20.3 / 20.4, 8192 53 / 49, 32768 203 / 176; 10 rows: 1024
// 4.9 / 4.0, 32768 124 / 73.
constexpr int kTileRows = 60;
constexpr int kSpreadBlocks = 608;                  // four blocks per SM

struct QkvArgs {
    const __nv_bfloat16 *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const __nv_bfloat16 *wq, *wk;
    const int32_t *pos;
    __nv_bfloat16 *q_pre, *q_post, *k_out, *v_out;
    int n_tokens, H, Hkv, rows;                     // rows per token: H + Hkv (+ Hkv with values)
    int rotary, interleaved;
    float eps;
};

struct Turns {
    uint64_t t[kPairs];
};

// W (4 or 8) bf16 elements as W / 2 words
template <int W>
struct Chunk {
    uint32_t w[W / 2];
};

template <int W>
__device__ __forceinline__ Chunk<W> load(const __nv_bfloat16 *p)
{
    Chunk<W> c;
    if (W == 8) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        c.w[0] = u.x, c.w[1] = u.y, c.w[W / 2 - 2] = u.z, c.w[W / 2 - 1] = u.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        c.w[0] = u.x, c.w[1] = u.y;
    }
    return c;
}

template <int W>
__device__ __forceinline__ void store(__nv_bfloat16 *p, const Chunk<W> &c)
{
    if (W == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(c.w[0], c.w[1], c.w[W / 2 - 2], c.w[W / 2 - 1]);
    else *reinterpret_cast<uint2 *>(p) = make_uint2(c.w[0], c.w[1]);
}

template <int W>
__device__ __forceinline__ void unpack(const Chunk<W> &c, float (&x)[W])
{
#pragma unroll
    for (int i = 0; i < W / 2; i++) {
        x[2 * i] = __uint_as_float(c.w[i] << 16);
        x[2 * i + 1] = __uint_as_float(c.w[i] & 0xffff0000u);
    }
}

template <int W>
__device__ __forceinline__ void put(__nv_bfloat16 *p, const float (&x)[W])
{
    Chunk<W> c;
#pragma unroll
    for (int i = 0; i < W / 2; i++) c.w[i] = bf16x2_bits(__floats2bfloat162_rn(x[2 * i], x[2 * i + 1]));
    store<W>(p, c);
}

// LANES lanes own a row, a lane two chunks of W = 64 / LANES elements.  The
// block's kTile tokens share its rows of lanes evenly, so a thread stays with
// one token and keeps its sines and cosines in registers.  kBatch rows are
// loaded together before the first is used.
template <int LANES, int kTile, int kBatch, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks) qkv_norm_rope_kernel(const __grid_constant__ QkvArgs a,
                                                                 const __grid_constant__ Turns turns)
{
    constexpr int W = kPairs / LANES, kPer = kThreads / LANES / kTile;   // kPer: rows of a token worked on at once
    __shared__ float2 cs[kTile][kPairs];
    pdl_wait();
    const int lane = threadIdx.x % LANES, unit = threadIdx.x / LANES;
    const int t0 = blockIdx.x * kTile;
    const int pairs = a.rotary >> 1;
    for (int i = threadIdx.x; i < kTile * kPairs; i += kThreads) {
        const int t = i / kPairs, j = i % kPairs;
        float s = 0.f, c = 1.f;
        if (j < pairs && t0 + t < a.n_tokens) {
            const uint64_t turn = (uint64_t)(int64_t)a.pos[t0 + t] * turns.t[j];
            // the nearest whole turn is dropped: a signed fraction in [-1/2, 1/2)
            sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
        }
        cs[t][j] = make_float2(c, s);
    }
    // the lane's two chunks of a row, and whether they rotate
    const int turning = a.rotary / (2 * W);       // lanes that rotate
    const bool turn = lane < turning;
    const int da = a.interleaved ? 2 * W * lane : turn ? W * lane : a.rotary + W * (lane - turning);
    const int db = da + (a.interleaved ? W : turn ? pairs : (kD - a.rotary) >> 1);
    Chunk<W> wqa{}, wqb{}, wka{}, wkb{};
    if (a.wq) wqa = load<W>(a.wq + da), wqb = load<W>(a.wq + db);
    if (a.wk) wka = load<W>(a.wk + da), wkb = load<W>(a.wk + db);
    __syncthreads();

    const int t = unit / kPer, tok = t0 + t;
    float2 rot[W];
#pragma unroll
    for (int j = 0; j < W; j++) rot[j] = turn ? cs[t][W * lane + j] : make_float2(1.f, 0.f);
    const int total = tok < a.n_tokens ? a.rows : 0;
    const int step = kPer * gridDim.y, first = blockIdx.y * kPer + unit % kPer;
    // every lane of a warp takes part in every turn of the loop (the shuffles): it runs for the block's first row
    for (int base = 0; base + blockIdx.y * kPer < a.rows; base += step * kBatch) {
        Chunk<W> ra[kBatch], rb[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; i++) {
            const int r = first + base + i * step;
            ra[i] = rb[i] = Chunk<W>{};
            if (r < total) {
                const __nv_bfloat16 *p = r < a.H           ? a.q + tok * a.q_stride + (int64_t)r * kD
                                         : r < a.H + a.Hkv ? a.k + tok * a.k_stride + (int64_t)(r - a.H) * kD
                                                           : a.v + tok * a.v_stride + (int64_t)(r - a.H - a.Hkv) * kD;
                ra[i] = load<W>(p + da);
                rb[i] = load<W>(p + db);
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; i++) {
            const int r = first + base + i * step;
            const bool live = r < total;
            float x[W], y[W];
            unpack<W>(ra[i], x);
            unpack<W>(rb[i], y);
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < W; j++) ss = fmaf(x[j], x[j], fmaf(y[j], y[j], ss));
#pragma unroll
            for (int o = LANES / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (live && r >= a.H + a.Hkv) {
                __nv_bfloat16 *o = a.v_out + ((int64_t)tok * a.Hkv + (r - a.H - a.Hkv)) * kD;
                store<W>(o + da, ra[i]);
                store<W>(o + db, rb[i]);
            } else if (live) {
                const bool is_q = r < a.H;
                if (is_q ? a.wq != nullptr : a.wk != nullptr) {
                    const float inv = rsqrtf(ss * (1.f / kD) + a.eps);
                    float wa[W], wb[W];
                    unpack<W>(is_q ? wqa : wka, wa);
                    unpack<W>(is_q ? wqb : wkb, wb);
#pragma unroll
                    for (int j = 0; j < W; j++) {
                        x[j] *= inv * wa[j];
                        y[j] *= inv * wb[j];
                    }
                }
                const int64_t at =
                    is_q ? ((int64_t)tok * a.H + r) * kD : ((int64_t)tok * a.Hkv + (r - a.H)) * kD;
                if (is_q && a.q_pre) {
                    put<W>(a.q_pre + at + da, x);
                    put<W>(a.q_pre + at + db, y);
                }
                if (!turn) {
                    // these elements stay: a product with the sine's 0 would bring a neighbour's infinity or NaN in
                } else if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < W / 2; j++) {
                        const float2 c0 = rot[j], c1 = rot[j + W / 2];
                        const float x0 = x[2 * j], x1 = x[2 * j + 1], y0 = y[2 * j], y1 = y[2 * j + 1];
                        x[2 * j] = x0 * c0.x - x1 * c0.y;
                        x[2 * j + 1] = x1 * c0.x + x0 * c0.y;
                        y[2 * j] = y0 * c1.x - y1 * c1.y;
                        y[2 * j + 1] = y1 * c1.x + y0 * c1.y;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < W; j++) {
                        const float x0 = x[j], y0 = y[j];
                        x[j] = x0 * rot[j].x - y0 * rot[j].y;
                        y[j] = y0 * rot[j].x + x0 * rot[j].y;
                    }
                }
                __nv_bfloat16 *o = (is_q ? a.q_post : a.k_out) + at;
                put<W>(o + da, x);
                put<W>(o + db, y);
            }
        }
    }
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace

}  // namespace macgpu

extern "C" mac_status mac_rope_init(const mac_rope_config *cfg, mac_rope *out)
{
    if (!cfg || !out) return MAC_ERR_INVALID_ARG;
    if (cfg->heads < 1 || cfg->kv_heads < 1 || cfg->heads % cfg->kv_heads || cfg->heads > 1024) return MAC_ERR_INVALID_ARG;
    if (cfg->head_dim != kD) return MAC_ERR_INVALID_ARG;
    if (cfg->rotary_dim < 0 || cfg->rotary_dim > kD || cfg->rotary_dim % 8) return MAC_ERR_INVALID_ARG;
    if (cfg->interleaved != 0 && cfg->interleaved != 1) return MAC_ERR_INVALID_ARG;
    if (!(cfg->eps >= 0.f) || !std::isfinite(cfg->eps)) return MAC_ERR_INVALID_ARG;
    if (!(cfg->rope_base >= 1.0) || !std::isfinite(cfg->rope_base)) return MAC_ERR_INVALID_ARG;
    *out = mac_rope{};
    out->cfg = *cfg;
    for (int i = 0; i < cfg->rotary_dim / 2; i++) {
        // at most 1 / 2 pi of a turn per position, so the product is below 2^62
        const double t = std::pow(cfg->rope_base, -2.0 * i / cfg->rotary_dim) / 6.283185307179586476925287;
        out->turns[i] = (uint64_t)std::llround(std::ldexp(t, 64));
    }
    return MAC_OK;
}

extern "C" mac_status mac_qkv_norm_rope(const mac_rope *rope, int n_tokens, const void *dev_q, int64_t q_stride,
                                        const void *dev_k, int64_t k_stride, const void *dev_v, int64_t v_stride,
                                        const void *dev_w_q, const void *dev_w_k, const int32_t *dev_pos,
                                        void *dev_q_pre, void *dev_q_post, void *dev_k_out, void *dev_v_out,
                                        void *stream)
{
    if (!rope || rope->cfg.head_dim != kD || rope->cfg.heads < 1 || rope->cfg.heads > 1024 || rope->cfg.kv_heads < 1 ||
        rope->cfg.kv_heads > rope->cfg.heads || rope->cfg.rotary_dim < 0 || rope->cfg.rotary_dim > kD ||
        rope->cfg.rotary_dim % 8)
        return MAC_ERR_INVALID_ARG;
    if (n_tokens < 0) return MAC_ERR_INVALID_ARG;
    if (n_tokens == 0) return MAC_OK;
    const int H = rope->cfg.heads, Hkv = rope->cfg.kv_heads;
    if (!dev_q || !dev_k || !dev_pos || !dev_q_post || !dev_k_out) return MAC_ERR_INVALID_ARG;
    if ((dev_v == nullptr) != (dev_v_out == nullptr)) return MAC_ERR_INVALID_ARG;
    if (!aligned16(dev_q) || !aligned16(dev_k) || !aligned16(dev_v) || !aligned16(dev_w_q) || !aligned16(dev_w_k) ||
        !aligned16(dev_q_pre) || !aligned16(dev_q_post) || !aligned16(dev_k_out) || !aligned16(dev_v_out) ||
        ((uintptr_t)dev_pos & 3))
        return MAC_ERR_INVALID_ARG;
    if (q_stride < (int64_t)H * kD || k_stride < (int64_t)Hkv * kD || (dev_v && v_stride < (int64_t)Hkv * kD))
        return MAC_ERR_INVALID_ARG;
    if (q_stride % 8 || k_stride % 8 || (dev_v && v_stride % 8)) return MAC_ERR_INVALID_ARG;

    QkvArgs a{};
    a.q = (const __nv_bfloat16 *)dev_q;
    a.k = (const __nv_bfloat16 *)dev_k;
    a.v = (const __nv_bfloat16 *)dev_v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.wq = (const __nv_bfloat16 *)dev_w_q;
    a.wk = (const __nv_bfloat16 *)dev_w_k;
    a.pos = dev_pos;
    a.q_pre = (__nv_bfloat16 *)dev_q_pre;
    a.q_post = (__nv_bfloat16 *)dev_q_post;
    a.k_out = (__nv_bfloat16 *)dev_k_out;
    a.v_out = (__nv_bfloat16 *)dev_v_out;
    a.n_tokens = n_tokens;
    a.H = H;
    a.Hkv = Hkv;
    a.rows = H + Hkv + (dev_v ? Hkv : 0);
    a.rotary = rope->cfg.rotary_dim;
    a.interleaved = rope->cfg.interleaved;
    a.eps = rope->cfg.eps;
    Turns t;
    for (int i = 0; i < kPairs; i++) t.t[i] = rope->turns[i];
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (n_tokens < kTileRows * a.rows) {
        // few tokens: one to a block, its rows over as many blocks as keep the grid near four blocks per SM
        int split = kSpreadBlocks / n_tokens;
        const int most = (a.rows + 15) / 16;
        split = split < 1 ? 1 : split > most ? most : split;
        e = launch_maybe_pdl(qkv_norm_rope_kernel<16, 1, 3, 4>, dim3(n_tokens, split), dim3(kThreads), 0, s, true, a, t);
    } else if (a.rotary % 16 == 0) {
        e = launch_maybe_pdl(qkv_norm_rope_kernel<8, 4, 2, 3>, dim3((n_tokens + 3) / 4), dim3(kThreads), 0, s, true, a, t);
    } else {
        // 16-byte chunks would hold elements that rotate and elements that do not
        e = launch_maybe_pdl(qkv_norm_rope_kernel<16, 4, 2, 3>, dim3((n_tokens + 3) / 4), dim3(kThreads), 0, s, true, a, t);
    }
    return e == cudaSuccess ? MAC_OK : MAC_ERR_CUDA;
}
