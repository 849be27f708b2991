// Parts that the attentions over the quantised stores share behind their long
// loops: a piece of a group that is not finished by one warp is parked, the
// pieces of a block are merged, and a second kernel merges the groups that
// cross blocks.
#pragma once
#include "mac_quant_line.cuh"

namespace macgpu {

namespace {

constexpr uint32_t kSpinLimit = 1u << 22;
constexpr int kMaxPieces = 32;
constexpr int kParkRow = kD + 4;                        // floats per parked row: its output and summary, padded

__device__ __forceinline__ bool mbar_wait(uint32_t mbar, uint32_t parity)
{
    for (uint32_t i = 0; i < kSpinLimit; i++) {
        uint32_t ok;
        asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                     : "=r"(ok)
                     : "r"(mbar), "r"(parity)
                     : "memory");
        if (ok) return true;
    }
    return false;
}

// D += A (16 x 16 f16) B (16 x 8 f16), fp32 accumulators
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A sum of weights, l, at a reference -d log2 units higher: l 2^d, with w = 2^d.  kFar, for the 8-bit store: its references
// are those of products, in whose units a token's weight may be 2^69, so that l 2^d counts where 2^d alone is 0 already.
template <bool kFar>
__device__ __forceinline__ float sum_at(float l, float w, float d)
{
    if (kFar && d < -120.f) return l * 0x1p-120f * ex2_approx(d + 120.f);
    return l * w;
}

// What the merge needs of a block: the line, the block's units of it, and the
// group of each parked piece, in order (-1: none).
struct MergeState {
    Line line;
    long long lo, hi;
    int piece_group[kMaxPieces];
};

// Writes a row's finished output (four elements at d0) and its lse.
__device__ __forceinline__ void finish4(const QuantAttnArgs &a, int b, int g, int r, int d0, float4 o, float m, float l,
                                        bool write_lse)
{
    const int qt = r / a.G, head = g * a.G + (r - qt * a.G);
    const int64_t row = ((int64_t)b * a.n_query + qt) * a.heads + head;
    const float inv = l == 0.f ? 0.f : a.v_out_scale / l;
    if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<uint2 *>(a.out + row * kD + d0) = make_uint2(
        bf16x2_bits(__floats2bfloat162_rn(o.x * inv, o.y * inv)), bf16x2_bits(__floats2bfloat162_rn(o.z * inv, o.w * inv)));
    if (write_lse && a.lse) a.lse[row] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
}

// The lane's 32 elements from 32 c on of row r of a group's queries (zeros past
// the rows).
__device__ __forceinline__ void load_q(const QuantAttnArgs &a, int b, int g, int r, int c, uint32_t (&w)[16])
{
#pragma unroll
    for (int i = 0; i < 16; i++) w[i] = 0;
    if (r < a.rows) {
        const int qt = r / a.G;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            a.q + (((int64_t)b * a.n_query + qt) * a.heads + g * a.G + (r - qt * a.G)) * kD + 32 * c);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint4 v = src[i];
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    }
}

// The largest bit pattern of the finite magnitudes in w.
__device__ __forceinline__ uint32_t finite_top(const uint32_t (&w)[16])
{
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
        top = max(top, lo < 0x7f80u ? lo : 0u);
        top = max(top, hi < 0x7f80u ? hi : 0u);
    }
    return top;
}

// Partial rows in the scratch: every block's two crossing groups, then every
// team's first piece.  A team's last piece is parked in its own shared memory,
// which it has read to the end by then.
struct Parking {
    unsigned char *smem;
    int team_bytes, teams, padrows;
    __device__ __forceinline__ int64_t crossing_row(int which, int r) const
    {
        return ((int64_t)blockIdx.x * 2 + which) * padrows + r;
    }
    __device__ __forceinline__ int64_t first_row(int t, int r) const
    {
        return ((int64_t)gridDim.x * 2 + (int64_t)blockIdx.x * teams + t) * padrows + r;
    }
    __device__ __forceinline__ float *last_o(int t, int r) const
    {
        return reinterpret_cast<float *>(smem + (size_t)t * team_bytes) + r * kParkRow;
    }
    __device__ __forceinline__ float2 *last_ml(int t, int r) const { return reinterpret_cast<float2 *>(last_o(t, r) + kD); }
};

// Behind the long loop: all warps of the block (WARPS, in TEAMS teams).
template <int TEAMS, int WARPS, bool FAR>
__device__ __forceinline__ void merge_pieces(const QuantAttnArgs &a, const MergeState &sm, const Parking &park)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, Hkv = a.st.kv_heads;
    __threadfence_block();
    __syncthreads();

    // Merge the parked pieces group by group; the rows of all groups go round the
    // warps.  Lane i looks at piece i; a run of pieces of one group starts where the group differs
    // from the piece before it.
    const int mine = lane < 2 * TEAMS ? sm.piece_group[lane] : -1;
    const uint32_t parked = __ballot_sync(0xffffffffu, mine >= 0);
    const uint32_t below = parked & ((1u << lane) - 1u);
    const int before = __shfl_sync(0xffffffffu, mine, below ? 31 - __clz(below) : 0);
    uint32_t starts = __ballot_sync(0xffffffffu, mine >= 0 && (!below || before != mine));
    int turn = warp;        // the warp's next row of the run
    while (starts) {
        const int first = __ffs(starts) - 1;
        starts &= starts - 1;
        const uint32_t run = parked & ~((1u << first) - 1u) & (starts ? (1u << (__ffs(starts) - 1)) - 1u : 0xffffffffu);
        const int grp = __shfl_sync(0xffffffffu, mine, first);
        const int b = grp / Hkv, g = grp - b * Hkv;
        const long long n_units = sm.line.pre[b + 1] - sm.line.pre[b];
        const long long start = sm.line.pre[b] * Hkv + g * n_units;
        const bool whole = start >= sm.lo && start + n_units <= sm.hi;
        if (whole && tid == 0 && meta_by_group(a, gridDim.x)) a.meta[grp] = make_int4(-1, 0, 0, 0);
        int r = turn;
        for (; r < a.rows; r += WARPS) {
            float2 ml = make_float2(-CUDART_INF_F, 0.f);
            if (run >> lane & 1) ml = lane & 1 ? *park.last_ml(lane >> 1, r) : a.part_ml[park.first_row(lane >> 1, r)];
            const bool none = ml.y == 0.f;      // saw no token
            const float m = warp_max(none ? -CUDART_INF_F : ml.x);
            // a NaN sum survives: its weight is a number or NaN, and the product NaN
            const float d = ml.x - m, w = none ? 0.f : exp2f(d);
            const float l = warp_sum(none ? 0.f : sum_at<FAR>(ml.y, w, d));
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            uint32_t rest_of = __ballot_sync(0xffffffffu, !none);
            while (rest_of) {
                const int i = __ffs(rest_of) - 1;
                rest_of &= rest_of - 1;
                const float wi = __shfl_sync(0xffffffffu, w, i);
                const float *src = i & 1 ? park.last_o(i >> 1, r) : a.part_o + park.first_row(i >> 1, r) * kD;
                const float4 x = reinterpret_cast<const float4 *>(src)[lane];
                o.x += x.x * wi;
                o.y += x.y * wi;
                o.z += x.z * wi;
                o.w += x.w * wi;
            }
            if (whole) {
                finish4(a, b, g, r, lane * 4, o, m, l, lane == 0);
            } else {
                const int64_t at = park.crossing_row(start < sm.lo ? 0 : 1, r);
                reinterpret_cast<float4 *>(a.part_o + at * kD)[lane] = o;
                if (lane == 0) a.part_ml[at] = make_float2(m, l);
            }
        }
        turn = r - a.rows;
    }
}

// The groups that cross blocks, merged: block (x, y) has the group of meta[x],
// which spans the attention kernel's blocks meta.z .. meta.y, and the rows
// y rpb .. of it, 8 / rpb warps to a row, a lane with four elements.  A warp
// takes eight partials at a time, and its loads are independent of one another.
// The body runs twice: first without partials while the attention kernel still
// works, which brings its instructions into the caches (1 to 1.5 us of the 3.6
// that the merge took without), then with them.
constexpr int kCombineWarps = 8, kCombineBatch = 8;

template <bool FAR>
__global__ void __launch_bounds__(kCombineWarps * 32) quant_combine_kernel(const __grid_constant__ QuantAttnArgs a,
                                                                          int padrows, int rpb)
{
    __shared__ float4 so[kCombineWarps][32];
    __shared__ float2 sml[kCombineWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wpr = kCombineWarps / rpb, sub = warp % wpr, r = blockIdx.y * rpb + warp / wpr;
#pragma unroll 1
    for (int pass = 0; pass < 2; pass++) {
        int n = 0, group = 0, cta0 = 0;
        if (pass) {
            pdl_wait();
            const int4 meta = __ldcg(a.meta + blockIdx.x);
            if (meta.x < 0) return;
            group = meta.x;
            cta0 = meta.z;
            n = r < a.rows ? meta.y - cta0 + 1 : 0;
        }
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float m = -CUDART_INF_F, l = 0.f;
        int k0 = sub * kCombineBatch;
        do {
            // partial k: the group's part of block cta0 + k
            float2 ml[kCombineBatch];
            float4 x[kCombineBatch];
#pragma unroll
            for (int i = 0; i < kCombineBatch; i++) {
                const int k = k0 + i;
                const int64_t row = ((int64_t)(cta0 + k) * 2 + (k == 0 ? 1 : 0)) * padrows + r;
                ml[i] = make_float2(-CUDART_INF_F, 0.f);
                x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k < n) {
                    ml[i] = __ldcg(a.part_ml + row);
                    x[i] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + row * kD) + lane);
                }
            }
            float top = m;
#pragma unroll
            for (int i = 0; i < kCombineBatch; i++)
                if (ml[i].y != 0.f) top = fmaxf(top, ml[i].x);      // a sum of 0 saw no token
            const float wo = l == 0.f ? 0.f : ex2_approx(m - top);
            o = make_float4(o.x * wo, o.y * wo, o.z * wo, o.w * wo);
            l = sum_at<FAR>(l, wo, m - top);
#pragma unroll
            for (int i = 0; i < kCombineBatch; i++) {
                // a NaN sum survives: its weight is a number or NaN, and the product NaN
                const bool some = ml[i].y != 0.f;
                const float d = ml[i].x - top, w = some ? ex2_approx(d) : 0.f;
                l += some ? sum_at<FAR>(ml[i].y, w, d) : 0.f;
                o.x += some ? x[i].x * w : 0.f;
                o.y += some ? x[i].y * w : 0.f;
                o.z += some ? x[i].z * w : 0.f;
                o.w += some ? x[i].w * w : 0.f;
            }
            m = top;
            k0 += wpr * kCombineBatch;
        } while (k0 < n);
        so[warp][lane] = o;
        if (lane == 0) sml[warp] = make_float2(m, l);
        __syncthreads();
        if (sub == 0) {
            float top = -CUDART_INF_F;
#pragma unroll 1
            for (int w = 0; w < wpr; w++)
                if (sml[warp + w].y != 0.f) top = fmaxf(top, sml[warp + w].x);
            o = make_float4(0.f, 0.f, 0.f, 0.f);
            l = 0.f;
#pragma unroll 1
            for (int w = 0; w < wpr; w++) {
                const float2 ml = sml[warp + w];
                const float4 x = so[warp + w][lane];
                if (ml.y == 0.f) continue;
                const float d = ml.x - top, f = ex2_approx(d);
                l += sum_at<FAR>(ml.y, f, d);
                o = make_float4(o.x + x.x * f, o.y + x.y * f, o.z + x.z * f, o.w + x.w * f);
            }
            const int b = group / a.st.kv_heads;
            if (n > 0) finish4(a, b, group - b * a.st.kv_heads, r, lane * 4, o, top, l, lane == 0);
        }
        __syncthreads();
    }
}

}  // namespace

// Blocks of the attention kernel: as many as fit the SMs, and as have room for
// their partial rows in the scratch.
inline int quant_grid(int sm_count, int blocks_per_sm, int teams, int padrows)
{
    int grid = sm_count * blocks_per_sm;
    const int fit = kQPartRows / ((teams + 2) * padrows);
    grid = grid < fit ? grid : fit;
    return grid < kMaxCtas ? grid : kMaxCtas;
}

template <bool FAR>
static inline cudaError_t launch_quant_combine(const QuantAttnArgs &a, int grid, int padrows, int sm_count, cudaStream_t s)
{
    // as many warps to a row as keep the blocks, most of which find nothing to merge, near one wave
    const int items = meta_by_group(a, grid) ? a.batch * a.st.kv_heads : grid;
    int rpb = 1;
    while (rpb < kCombineWarps && rpb < a.rows && (int64_t)items * ((a.rows + rpb - 1) / rpb) > 4 * sm_count) rpb *= 2;
    return launch_maybe_pdl(quant_combine_kernel<FAR>, dim3(items, (a.rows + rpb - 1) / rpb), dim3(kCombineWarps * 32), 0, s, true,
                            a, padrows, rpb);
}

}  // namespace macgpu
