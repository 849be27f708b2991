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
// row, nothing read twice); few tokens, the launch and one round trip.  A
// half-warp owns a row: lane l holds the two 4-element chunks whose elements
// rotate with each other, so the rotation needs no shuffle and the mean of
// squares four.  A block takes kTile tokens and first makes their sines and
// cosines (one sincospi per thread for four tokens), which all their heads
// share.  Few tokens spread over more blocks (gridDim.y splits a token's
// rows), so that each half-warp has one to three rows and one token's latency
// is a single row's.
#include "../../include/mac.h"
#include "mac_device.cuh"

#include <cmath>

using namespace macgpu;

namespace macgpu {

namespace {

constexpr int kThreads = 256;
constexpr int kRowLanes = 16;                       // lanes per row
constexpr int kRows = kThreads / kRowLanes;         // rows a block works on at once
constexpr int kPairs = kD / 2;

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

__device__ __forceinline__ uint2 load8(const __nv_bfloat16 *p) { return *reinterpret_cast<const uint2 *>(p); }

__device__ __forceinline__ void unpack4(uint2 u, float (&x)[4])
{
    x[0] = __uint_as_float(u.x << 16);
    x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16);
    x[3] = __uint_as_float(u.y & 0xffff0000u);
}

__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float (&x)[4])
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(bf16x2_bits(__floats2bfloat162_rn(x[0], x[1])),
                                               bf16x2_bits(__floats2bfloat162_rn(x[2], x[3])));
}

// Rows of kBatch half-warp turns are loaded together before the first is used.
template <int kTile, int kBatch>
__global__ void __launch_bounds__(kThreads) qkv_norm_rope_kernel(const __grid_constant__ QkvArgs a,
                                                                 const __grid_constant__ Turns turns)
{
    __shared__ float2 cs[kTile][kPairs];
    pdl_wait();
    const int lane = threadIdx.x % kRowLanes, unit = threadIdx.x / kRowLanes;
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
    int da, db;
    const bool turn = lane < (a.rotary >> 3);
    if (a.interleaved) {
        da = 8 * lane;
        db = da + 4;
    } else if (turn) {
        da = 4 * lane;
        db = da + pairs;
    } else {
        da = a.rotary + 4 * (lane - (a.rotary >> 3));
        db = da + ((kD - a.rotary) >> 1);
    }
    float wqa[4], wqb[4], wka[4], wkb[4];
    if (a.wq) {
        unpack4(load8(a.wq + da), wqa);
        unpack4(load8(a.wq + db), wqb);
    }
    if (a.wk) {
        unpack4(load8(a.wk + da), wka);
        unpack4(load8(a.wk + db), wkb);
    }
    __syncthreads();

    const int tokens = min(kTile, a.n_tokens - t0);
    const int total = tokens * a.rows;
    const int step = kRows * gridDim.y;
    for (int base = blockIdx.y * kRows + unit; base - unit < total; base += step * kBatch) {
        uint2 ra[kBatch], rb[kBatch];
        int tok[kBatch], row[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; i++) {
            const int it = base + i * step;
            tok[i] = -1;
            ra[i] = rb[i] = make_uint2(0, 0);
            if (it < total) {
                const int t = kTile == 1 ? 0 : it / a.rows;
                tok[i] = t0 + t;
                row[i] = it - t * a.rows;
                const int r = row[i];
                const __nv_bfloat16 *p = r < a.H           ? a.q + tok[i] * a.q_stride + (int64_t)r * kD
                                         : r < a.H + a.Hkv ? a.k + tok[i] * a.k_stride + (int64_t)(r - a.H) * kD
                                                           : a.v + tok[i] * a.v_stride + (int64_t)(r - a.H - a.Hkv) * kD;
                ra[i] = load8(p + da);
                rb[i] = load8(p + db);
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; i++) {
            const int r = row[i];
            const bool live = tok[i] >= 0;
            float x[4], y[4];
            unpack4(ra[i], x);
            unpack4(rb[i], y);
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 4; j++) ss = fmaf(x[j], x[j], fmaf(y[j], y[j], ss));
#pragma unroll
            for (int o = kRowLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (!live) continue;
            if (r >= a.H + a.Hkv) {
                __nv_bfloat16 *o = a.v_out + ((int64_t)tok[i] * a.Hkv + (r - a.H - a.Hkv)) * kD;
                *reinterpret_cast<uint2 *>(o + da) = ra[i];
                *reinterpret_cast<uint2 *>(o + db) = rb[i];
                continue;
            }
            const bool is_q = r < a.H;
            const __nv_bfloat16 *w = is_q ? a.wq : a.wk;
            if (w) {
                const float inv = rsqrtf(ss * (1.f / kD) + a.eps);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    x[j] *= inv * (is_q ? wqa[j] : wka[j]);
                    y[j] *= inv * (is_q ? wqb[j] : wkb[j]);
                }
            }
            const int64_t at = is_q ? ((int64_t)tok[i] * a.H + r) * kD : ((int64_t)tok[i] * a.Hkv + (r - a.H)) * kD;
            if (is_q && a.q_pre) {
                store4(a.q_pre + at + da, x);
                store4(a.q_pre + at + db, y);
            }
            if (turn) {
                const float2 *c = &cs[kTile == 1 ? 0 : tok[i] - t0][4 * lane];
                if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        const float2 c0 = c[j], c1 = c[j + 2];
                        const float x0 = x[2 * j], x1 = x[2 * j + 1], y0 = y[2 * j], y1 = y[2 * j + 1];
                        x[2 * j] = x0 * c0.x - x1 * c0.y;
                        x[2 * j + 1] = x1 * c0.x + x0 * c0.y;
                        y[2 * j] = y0 * c1.x - y1 * c1.y;
                        y[2 * j + 1] = y1 * c1.x + y0 * c1.y;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float2 c0 = c[j];
                        const float x0 = x[j], y0 = y[j];
                        x[j] = x0 * c0.x - y0 * c0.y;
                        y[j] = y0 * c0.x + x0 * c0.y;
                    }
                }
            }
            __nv_bfloat16 *o = (is_q ? a.q_post : a.k_out) + at;
            store4(o + da, x);
            store4(o + db, y);
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
    if (n_tokens < 608) {
        // few tokens: one to a block, its rows over as many blocks as keep the grid near four blocks per SM
        int split = 608 / n_tokens;
        const int most = (a.rows + kRows - 1) / kRows;
        split = split < 1 ? 1 : split > most ? most : split;
        e = launch_maybe_pdl(qkv_norm_rope_kernel<1, 3>, dim3(n_tokens, split), dim3(kThreads), 0, s, true, a, t);
    } else {
        e = launch_maybe_pdl(qkv_norm_rope_kernel<4, 4>, dim3((n_tokens + 3) / 4), dim3(kThreads), 0, s, true, a, t);
    }
    return e == cudaSuccess ? MAC_OK : MAC_ERR_CUDA;
}
