// Parts of the attentions over the quantised stores: the line of work units and
// its cut into equal ranges, and the unpacking of 4-bit codes.
//
// A unit is a fixed number of tokens of one (request, KV head) group; a request
// without tokens has one unit, so that its output gets written.  The units of
// all groups form one line, request by request and head by head, which is cut
// into equal ranges; every block derives both from the lengths.
#pragma once
#include "mac_device.cuh"
#include "mac_quant.cuh"

namespace macgpu {

namespace {

constexpr float kMargin = 6.f;      // log2: how far a score may pass the softmax reference
constexpr float kPShift = 9.f;      // P is held times 2^kPShift: 2^(6 + 9) is below the f16 maximum
constexpr float kLowest = -3e38f;   // the reference before the first token: finite, so that masked scores give weight 0

struct Line {
    long long pre[kQMaxBatch + 1];  // units of the requests before b (per KV head)
    int len[kQMaxBatch];
    long long scan[32];
};

// Fills the line from the lengths; all threads of the block (kWarps warps).
// kExtra: units that each group counts besides its own, in front of them, for
// what a piece costs whatever its length.
template <int kWarps, int kTok, int kExtra = 0>
__device__ __forceinline__ void make_line(const QuantAttnArgs &a, Line &line)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long cap = (long long)a.table_cols * kPage;
    long long carry = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kWarps * 32) {
        const int b = b0 + tid;
        int len = 0;
        if (b < a.batch) {
            len = a.lens[b];
            if (len < 0 || len > cap) {
                if (blockIdx.x == 0) atomicOr(a.st.err, kQErrLen);
                len = len < 0 ? 0 : (int)cap;
            }
            line.len[b] = len;
        }
        const long long own = b < a.batch ? (len > kTok ? (len - 1) / kTok + 1 : 1) + kExtra : 0;
        long long x = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) line.scan[warp] = x;
        __syncthreads();
        long long before = carry, all = carry;
#pragma unroll
        for (int w = 0; w < kWarps; w++) {
            if (w < warp) before += line.scan[w];
            all += line.scan[w];
        }
        if (b < a.batch) line.pre[b] = before + x - own;
        carry = all;
        __syncthreads();
    }
    if (tid == 0) line.pre[a.batch] = carry;
    __syncthreads();
}

// The cut of `units` units into `parts` equal ranges: part i starts at
// floor(units i / parts).  The remainder's share fits 32 bits, and so do the
// units almost always.
struct Cut {
    long long per;
    uint32_t rest;
    int parts;
    __device__ __forceinline__ Cut(long long units, int n) : parts(n)
    {
        per = units >> 32 ? units / n : (long long)((uint32_t)units / (uint32_t)n);
        rest = (uint32_t)(units - per * n);
    }
    __device__ __forceinline__ long long first(int i) const
    {
        return per * i + (long long)(rest * (uint32_t)i / (uint32_t)parts);
    }
};

// The group (b, g) that holds a unit of the line, the unit's place in it and
// the group's units.
__device__ __forceinline__ void locate(const QuantAttnArgs &a, const Line &line, long long unit, int &b, int &g, int &u, int &n)
{
    const int Hkv = a.st.kv_heads;
    int lo = 0, hi = a.batch;           // the last b with pre[b] * Hkv <= unit
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (line.pre[mid] * Hkv <= unit) lo = mid;
        else hi = mid;
    }
    b = lo;
    n = (int)(line.pre[lo + 1] - line.pre[lo]);
    const long long in = unit - line.pre[lo] * Hkv;
    g = in >> 32 ? (int)(in / n) : (int)((uint32_t)in / (uint32_t)n);
    u = (int)(in - (long long)g * n);
}

// Where the second kernel finds its groups: with no more groups than blocks in
// meta[group], else in meta[the block in which the group starts].
__host__ __device__ inline bool meta_by_group(const QuantAttnArgs &a, int grid) { return (int64_t)a.batch * a.st.kv_heads <= grid; }

// Leaves the group that starts in this block (units [lo, hi), `parts` parts of
// the cut per block) and runs on behind it to the second kernel.
__device__ __forceinline__ void write_meta(const QuantAttnArgs &a, const Line &line, const Cut &cut, long long units, int grid,
                                           int parts, long long lo, long long hi)
{
    const int cta = blockIdx.x;
    const bool by_group = meta_by_group(a, gridDim.x);
    int b, g, u, n;
    locate(a, line, hi - 1, b, g, u, n);
    const long long start = hi - 1 - u, end = start + n;
    int owner = -1, last = 0;
    if (start >= lo && end > hi) {
        owner = b * a.st.kv_heads + g;
        // the block that holds the group's last unit: a float guess, put right by the exact ranges
        last = min(grid - 1, (int)((float)(end - 1) / (float)units * (float)grid));
        while (cut.first(last * parts) >= end) last--;
        while (cut.first((last + 1) * parts) < end) last++;
    }
    if (owner >= 0 || !by_group) a.meta[by_group ? owner : cta] = make_int4(owner, last, cta, 0);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t mbar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(mbar)
                 : "memory");
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;\n" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// two floats as f16x2, x in the low half
__device__ __forceinline__ uint32_t f16x2(float x, float y)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(y), "f"(x));
    return r;
}

// eight codes -> four f16x2, one per byte
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t (&h)[4])
{
    asm("{\n.reg .b8 a, b, c, d;\nmov.b32 {a, b, c, d}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, a;\ncvt.rn.f16x2.e2m1x2 %1, b;\ncvt.rn.f16x2.e2m1x2 %2, c;\ncvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void sts16(uint32_t addr, const uint32_t (&v)[4])
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};\n" :: "r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

__device__ __forceinline__ uint32_t lds4(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void lds8(uint32_t addr, float (&v)[2])
{
    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];\n" : "=f"(v[0]), "=f"(v[1]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void sts4(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared.u32 [%0], %1;\n" :: "r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t lds1(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];\n" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Two bf16 times up as f16x2.  The added x * 0 makes an infinity NaN: scores of
// minus infinity alone would read as a row that sees nothing.
__device__ __forceinline__ uint32_t scaled_f16x2(uint32_t two, float up)
{
    const float x = __uint_as_float(two << 16), y = __uint_as_float(two & 0xffff0000u);
    return f16x2(__fmaf_rn(x, up, __fmul_rn(x, 0.f)), __fmaf_rn(y, up, __fmul_rn(y, 0.f)));
}

}  // namespace

}  // namespace macgpu
