// Decode attention over the 4-bit store (format and layout: mac_quant.cuh).
//
// Per request (len tokens) and KV head, the group's heads times the request's
// n_query new tokens are `rows` rows (at most 32); row r is head r % G of
// query token r / G and sees the first len - (n_query - 1) + r / G tokens:
//   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q . k_t),
//   lse = log sum_t p_t;  a row that sees nothing gives out 0, lse -inf.
//
// What bounds it.  The stream is 144 B per (token, KV head), 3.6 times less than
// in bf16, so at the memory's rate an SM has 100 cycles for a page of 16 tokens:
// the 4096 codes of a page have to be unpacked, scaled and multiplied in 400
// issue slots.  Everything is laid out for that count:
//  - a warp takes whole pages (bulk copies of 2304 B into a ring of its own, so
//    no warp waits for another), and its lanes' 16-byte loads are matrix
//    fragments once converted: two codes per cvt.e2m1x2, one f16x2 multiply by
//    the scale (exact), no shuffle;
//  - scores are S^T[tokens x rows] = K Q^T and the output O^T[dims x rows] +=
//    V^T P^T, both mma.m16n8k16 in f16 with fp32 accumulators: tokens (then
//    dims) fill M, and 1 to 8 rows cost one N tile.  tcgen05 would need the
//    unpacked page written to shared memory and read back, 512 B per token
//    against the 144 that are read here, which alone is 60 % of the budget;
//  - the order of the contraction index is free, so a thread's K words are 32
//    consecutive elements of a token, and its V words the same 16 elements of
//    four consecutive tokens, whose codes are paired by token with two logic
//    operations per eight codes.
// Roundings: Q is bf16 and becomes f16 with a power of two per row (exact
// unless an element is 2^-28 of the row's largest); stored values are exact in
// f16; the weights P, at most 2^15, are rounded to f16 (2^-11 of each) and
// summed unrounded in fp32; sums, the maximum and the output stay in fp32.
// P's factor 2^9 keeps weights down to 2^-33 of the largest.
//
// Work split.  The units (two pages) of all (request, KV head) groups form one
// line, which is cut into equal ranges, one per warp team, whatever the
// lengths; the cut is derived in every block from the lengths on the device, so
// a captured call serves any lengths.  A group inside one team's range is
// finished by it.  The pieces of the others are parked, merged per block, and,
// where a group crosses blocks, merged again by a second kernel (one block per
// crossing group and row).  No block waits for another.
#include "mac_device.cuh"
#include "mac_quant.cuh"

#include <cuda_fp16.h>

namespace macgpu {

namespace {

constexpr int kPP = 2;                                  // pages per unit
constexpr int kUnitTok = kPP * kPage;
constexpr int kUnitBytes = kPP * kQPageBytes;
constexpr float kMargin = 6.f;                          // log2: how far a score may pass the softmax reference
constexpr float kPShift = 9.f;                          // P is held times 2^kPShift: 2^(6 + 9) is below the f16 maximum
constexpr uint32_t kSpinLimit = 1u << 22;
constexpr int kMaxPieces = 32;
constexpr int kParkRow = kD + 4;                        // floats per parked row: its output and summary, padded

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t mbar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(mbar)
                 : "memory");
}

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
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

__device__ __forceinline__ uint32_t scales2(uint32_t two)
{
    uint32_t r;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(r) : "r"(two));
    return r;
}

__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t lds2(uint32_t addr)
{
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(addr) : "memory");
    return v;
}

// Units of request b: two pages each, one for an empty request (its output
// still has to be written).
__device__ __forceinline__ int units_of(int len) { return len > kUnitTok ? (len - 1) / kUnitTok + 1 : 1; }

// A position on the line of units: request, KV head, unit of the group.
struct Cursor {
    int b, g, u, n;     // n: units of the request
};

struct Smem {
    long long pre[kQMaxBatch + 1];      // units of the requests before b (per KV head)
    int len[kQMaxBatch];
    long long scan[32];
    // parked pieces of the block, in order: their group (-1: none)
    int piece_group[kMaxPieces];
    float2 nothing;                     // the summary of a piece that is not there
    unsigned long long bar[64];
};

__device__ __forceinline__ Cursor cursor_at(const Smem &sm, int batch, int Hkv, long long unit)
{
    int lo = 0, hi = batch;             // last b with pre[b] * Hkv <= unit
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sm.pre[mid] * Hkv <= unit) lo = mid;
        else hi = mid;
    }
    Cursor c;
    c.b = lo;
    c.n = (int)(sm.pre[lo + 1] - sm.pre[lo]);
    const long long in = unit - sm.pre[lo] * Hkv;
    c.g = (int)(in / c.n);
    c.u = (int)(in - (long long)c.g * c.n);
    return c;
}

__device__ __forceinline__ void step(Cursor &c, const Smem &sm, int batch, int Hkv)
{
    if (++c.u < c.n) return;
    c.u = 0;
    if (++c.g < Hkv) return;
    c.g = 0;
    if (++c.b < batch) c.n = (int)(sm.pre[c.b + 1] - sm.pre[c.b]);
}

// Writes a row's finished output (four elements at d0) and its lse.
__device__ __forceinline__ void finish4(const QuantAttnArgs &a, int b, int g, int r, int d0, float4 o, float m, float l,
                                        bool write_lse)
{
    const int qt = r / a.G, head = g * a.G + (r - qt * a.G);
    const int64_t row = ((int64_t)b * a.n_query + qt) * a.heads + head;
    const float inv = l == 0.f ? 0.f : a.st.v_scale / l;
    if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<uint2 *>(a.out + row * kD + d0) = make_uint2(
        bf16x2_bits(__floats2bfloat162_rn(o.x * inv, o.y * inv)), bf16x2_bits(__floats2bfloat162_rn(o.z * inv, o.w * inv)));
    if (write_lse && a.lse) a.lse[row] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
}

// Adds n partial rows to (o, m, l), a warp per call: lanes hold four elements
// of o each.  at(i) gives partial i's summary (max, sum) and its 128 floats;
// the summaries are read first, one lane each, so the rows' loads depend on
// nothing and run together.
// With kOthers the rows come from other blocks: they are read past the L1.
template <bool kOthers, typename F>
__device__ __forceinline__ void merge_rows(int n, F at, int lane, float4 &o, float &m, float &l)
{
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int k = min(32, n - i0);
        float2 ml = make_float2(-CUDART_INF_F, 0.f);
        const float4 *src = nullptr;
        if (lane < k) {
            const float2 *summary;
            at(i0 + lane, summary, src);
            ml = kOthers ? __ldcg(summary) : *summary;
        }
        const bool none = ml.y == 0.f;      // saw no token
        const float top = fmaxf(m, warp_max(none ? -CUDART_INF_F : ml.x));
        // a NaN sum survives: its weight is a number or NaN, and the product NaN
        const float w = none ? 0.f : exp2f(ml.x - top), wo = l == 0.f ? 0.f : exp2f(m - top);
        l = l * wo + warp_sum(none ? 0.f : ml.y * w);
        o = make_float4(o.x * wo, o.y * wo, o.z * wo, o.w * wo);
        m = top;
#pragma unroll 8
        for (int i = 0; i < k; i++) {
            const float4 *p = reinterpret_cast<const float4 *>(__shfl_sync(0xffffffffu, (unsigned long long)src, i));
            const float wi = __shfl_sync(0xffffffffu, w, i);
            const int skip = __shfl_sync(0xffffffffu, (int)none, i);
            const float4 x = skip ? make_float4(0.f, 0.f, 0.f, 0.f) : kOthers ? __ldcg(p + lane) : p[lane];
            o.x += x.x * wi;
            o.y += x.y * wi;
            o.z += x.z * wi;
            o.w += x.w * wi;
        }
    }
}

// NT: N tiles (8 rows each) per warp; RW: warps that share a page and split
// the rows; WARPS per block; STAGES units in a team's ring.
template <int NT, int RW, int WARPS, int STAGES, int MINB>
__global__ void __launch_bounds__(WARPS * 32, MINB) quant_attention_kernel(const __grid_constant__ QuantAttnArgs a)
{
    constexpr int TEAMS = WARPS / RW;
    constexpr int PADROWS = NT * 8 * RW;
    static_assert(2 * TEAMS <= kMaxPieces && TEAMS * STAGES <= 64, "block shape");
    static_assert(PADROWS * kParkRow * 4 <= STAGES * kUnitBytes, "a parked piece fits the team's ring");
    extern __shared__ __align__(128) unsigned char dyn[];
    __shared__ Smem sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int team = warp / RW, part = warp % RW;   // part: which rows of the group
    const int g8 = lane >> 2, c4 = lane & 3;
    const int Hkv = a.st.kv_heads;
    pdl_wait();
    pdl_launch_dependents();

    // lengths, and the prefix of the requests' units
    {
        const long long cap = (long long)a.table_cols * kPage;
        long long carry = 0;
        for (int b0 = 0; b0 < a.batch; b0 += WARPS * 32) {
            const int b = b0 + tid;
            int len = 0;
            if (b < a.batch) {
                len = a.lens[b];
                if (len < 0 || len > cap) {
                    if (blockIdx.x == 0) atomicOr(a.st.err, kQErrLen);
                    len = len < 0 ? 0 : (int)cap;
                }
                sm.len[b] = len;
            }
            long long x = b < a.batch ? units_of(len) : 0;
            const long long own = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) sm.scan[warp] = x;
            __syncthreads();
            long long before = carry, all = carry;
#pragma unroll
            for (int w = 0; w < WARPS; w++) {
                if (w < warp) before += sm.scan[w];
                all += sm.scan[w];
            }
            if (b < a.batch) sm.pre[b] = before + x - own;
            carry = all;
            __syncthreads();
        }
        if (tid == 0) sm.pre[a.batch] = carry;
    }
    const uint32_t bar0 = smem_u32(&sm.bar[team * STAGES]);
    const uint32_t ring = smem_u32(dyn) + (uint32_t)team * STAGES * kUnitBytes;
    if (tid == 0) {
        for (int i = 0; i < TEAMS * STAGES; i++)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" :: "r"(smem_u32(&sm.bar[i])) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (tid < 2 * TEAMS) sm.piece_group[tid] = -1;
    if (tid == 0) sm.nothing = make_float2(-CUDART_INF_F, 0.f);
    __syncthreads();

    // the block's and the team's range of units
    const long long U = sm.pre[a.batch] * Hkv;
    // every team of an active block has work: blocks beyond that stay idle
    const long long most = U / TEAMS > 0 ? U / TEAMS : 1;
    const int grid = most < (long long)gridDim.x ? (int)most : (int)gridDim.x;
    const int cta = blockIdx.x;
    if (cta >= grid) {
        if (tid == 0) a.meta[cta] = make_int4(-1, 0, 0, 0);
        return;
    }
    const long long teams = (long long)grid * TEAMS, me = (long long)cta * TEAMS + team;
    const long long lo = U * me / teams, hi = U * (me + 1) / teams;
    const long long cta_lo = U * cta / grid, cta_hi = U * (cta + 1) / grid;
    // partial rows: the block's two crossing groups, then its teams' first pieces.  A team's last piece is parked in
    // its own ring, which it has read to the end by then.
    const int64_t crossing = (int64_t)cta * 2 * PADROWS;
    const int64_t park = ((int64_t)gridDim.x * 2 + (int64_t)cta * TEAMS) * PADROWS;

    auto parked_o = [&](int t, int r) { return reinterpret_cast<float *>(dyn + (size_t)t * STAGES * kUnitBytes) + r * kParkRow; };
    auto parked_ml = [&](int t, int r) { return reinterpret_cast<float2 *>(parked_o(t, r) + kD); };

    if (lo < hi) {
        Cursor at = cursor_at(sm, a.batch, Hkv, lo);
        Cursor ld = at;                 // the next unit to copy
        long long ld_pos = lo;
        // page of the unit `ld` stands at (lane i < kPP: its i-th page; -1: none)
        auto page_of = [&](const Cursor &c) {
            int id = -1;
            const int p = c.u * kPP + lane;
            if (lane < kPP && p * (long long)kPage < sm.len[c.b]) {
                id = a.table[c.b * a.table_stride + p];
                if ((unsigned)id >= (unsigned)a.st.num_pages) {
                    atomicOr(a.st.err, kQErrPage);
                    id = 0;             // stays inside the store; the request's output is wrong
                }
            }
            return id;
        };
        int next_id = page_of(ld);
        // copies the unit at `ld` into stage s and moves on; the page after it is looked up a step ahead
        auto issue = [&](int s) {
            if (ld_pos >= hi) return;
            const uint32_t bar = bar0 + 8 * s, dst = ring + (uint32_t)s * kUnitBytes;
            const int id = next_id, head = ld.g;
            const uint32_t have = __ballot_sync(0xffffffffu, id >= 0);
            step(ld, sm, a.batch, Hkv);
            ld_pos++;
            if (ld_pos < hi) next_id = page_of(ld);
            if (part == 0) {
                if (lane == 0)
                    asm volatile("{\n.reg .b64 st;\nmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n}\n"
                                 :: "r"(bar), "r"((uint32_t)__popc(have) * kQPageBytes)
                                 : "memory");
                __syncwarp();
                if (id >= 0)
                    bulk_load(dst + lane * kQPageBytes, a.st.pages + ((size_t)id * Hkv + head) * kQPageBytes, kQPageBytes, bar);
            }
        };
#pragma unroll
        for (int s = 0; s < STAGES; s++) issue(s);

        int stage = 0;
        uint32_t phase = 0;
        long long pos = lo;
        while (pos < hi) {
            // one piece: units [at.u, at.u + n) of group (at.b, at.g)
            const int b = at.b, g = at.g, n_units = at.n, u0 = at.u;
            const int n = (int)(hi - pos < n_units - u0 ? hi - pos : n_units - u0);
            const int len = sm.len[b];
            const int full = len - (a.n_query - 1) > 0 ? len - (a.n_query - 1) : 0;   // tokens every row sees
            const int row0 = part * NT * 8;
            uint32_t qf[NT][16];
            float sc[NT][2], ref[NT][2], sum[NT][2], o[NT][8][4];
            int lim[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                const int r = row0 + nt * 8 + g8;
                float rs = 0.f;
                uint4 w[4];
#pragma unroll
                for (int i = 0; i < 4; i++) w[i] = make_uint4(0, 0, 0, 0);
                if (r < a.rows) {
                    const int qt = r / a.G;
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        a.q + (((int64_t)b * a.n_query + qt) * a.heads + g * a.G + (r - qt * a.G)) * kD + 32 * c4);
#pragma unroll
                    for (int i = 0; i < 4; i++) w[i] = src[i];
                }
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        top = max(top, x[k] & 0x7fffu);
                        top = max(top, (x[k] >> 16) & 0x7fffu);
                    }
                }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^shift brings the row's largest element into [2^14, 2^15)
                int shift = 14 - ((int)(top >> 7) - 127);
                if (top == 0 || top >= 0x7f80u) shift = 0;
                shift = shift > 126 ? 126 : shift;
                const float up = __int_as_float((shift + 127) << 23);
                rs = fmaxf(a.scale_log2 * __int_as_float((127 - shift) << 23), 1e-37f);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        qf[nt][4 * i + k] = f16x2(__uint_as_float(x[k] << 16) * up, __uint_as_float(x[k] & 0xffff0000u) * up);
                }
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int col = 2 * c4 + h, rr = row0 + nt * 8 + col;
                    sc[nt][h] = __shfl_sync(0xffffffffu, rs, col * 4);
                    const int l = len - (a.n_query - 1) + rr / a.G;
                    lim[nt][h] = rr < a.rows && l > 0 ? l : 0;
                    ref[nt][h] = -CUDART_INF_F;
                    sum[nt][h] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 8; j++)
#pragma unroll
                    for (int k = 0; k < 4; k++) o[nt][j][k] = 0.f;
            }

            for (int i = 0; i < n; i++) {
                if (!mbar_wait(bar0 + 8 * stage, phase)) atomicOr(a.st.err, kQErrTimeout);
                const uint32_t unit = ring + (uint32_t)stage * kUnitBytes;
                const int tok0 = (u0 + i) * kUnitTok;
                const bool tail = tok0 + kUnitTok > full;

                // scores
                float s[kPP][NT][4];
#pragma unroll
                for (int pp = 0; pp < kPP; pp++) {
                    const uint32_t page = unit + pp * kQPageBytes;
                    const int tk = 4 * (g8 >> 1) + (g8 & 1);     // token of matrix row g; row g + 8 is token tk + 2
                    const uint4 ka = lds16(page + tk * 64 + c4 * 16), kb = lds16(page + (tk + 2) * 64 + c4 * 16);
                    const uint32_t sa = scales2(lds2(page + kQKScale + tk * 8 + 2 * c4));
                    const uint32_t sb = scales2(lds2(page + kQKScale + (tk + 2) * 8 + 2 * c4));
                    const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int k = 0; k < 4; k++) s[pp][nt][k] = 0.f;
#pragma unroll
                    for (int w = 0; w < 4; w++) {
                        uint32_t ha[4], hb[4];
                        unpack8(wa[w], ha);
                        unpack8(wb[w], hb);
                        const uint32_t xa = __byte_perm(sa, sa, w < 2 ? 0x1010 : 0x3232);
                        const uint32_t xb = __byte_perm(sb, sb, w < 2 ? 0x1010 : 0x3232);
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            ha[k] = hmul2(ha[k], xa);
                            hb[k] = hmul2(hb[k], xb);
                        }
#pragma unroll
                        for (int k = 0; k < 2; k++)
#pragma unroll
                            for (int nt = 0; nt < NT; nt++)
                                mma_f16(s[pp][nt], ha[2 * k], hb[2 * k], ha[2 * k + 1], hb[2 * k + 1], qf[nt][4 * w + 2 * k],
                                        qf[nt][4 * w + 2 * k + 1]);
                    }
                }
                if (tail) {
#pragma unroll
                    for (int pp = 0; pp < kPP; pp++)
#pragma unroll
                        for (int nt = 0; nt < NT; nt++)
#pragma unroll
                            for (int k = 0; k < 4; k++) {
                                const int tok = tok0 + pp * kPage + 4 * (g8 >> 1) + (g8 & 1) + (k & 2);
                                if (tok >= lim[nt][k & 1]) s[pp][nt][k] = -CUDART_INF_F;
                            }
                }
                // softmax: the reference moves only when a score passes it by more than the margin
                bool moves = false;
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        float x = fmaxf(s[0][nt][h], s[0][nt][2 + h]);
#pragma unroll
                        for (int pp = 1; pp < kPP; pp++) x = fmaxf(x, fmaxf(s[pp][nt][h], s[pp][nt][2 + h]));
                        moves |= x * sc[nt][h] > ref[nt][h] + kMargin;
                    }
                if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            float x = fmaxf(s[0][nt][h], s[0][nt][2 + h]);
#pragma unroll
                            for (int pp = 1; pp < kPP; pp++) x = fmaxf(x, fmaxf(s[pp][nt][h], s[pp][nt][2 + h]));
                            x *= sc[nt][h];
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
                            const float top = fmaxf(ref[nt][h], x);
                            const float f = ref[nt][h] == -CUDART_INF_F ? 0.f : ex2_approx(ref[nt][h] - top);
                            ref[nt][h] = top;
                            sum[nt][h] *= f;
#pragma unroll
                            for (int j = 0; j < 8; j++) {
                                o[nt][j][h] *= f;
                                o[nt][j][2 + h] *= f;
                            }
                        }
                }
                uint32_t pb[kPP][NT][2];    // P^T fragments: tokens 4 c .. 4 c + 3, row g
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    float base[2];
#pragma unroll
                    for (int h = 0; h < 2; h++) base[h] = kPShift - (ref[nt][h] == -CUDART_INF_F ? 0.f : ref[nt][h]);
#pragma unroll
                    for (int pp = 0; pp < kPP; pp++) {
                        float p[4];
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            p[k] = ex2_approx(fmaf(s[pp][nt][k], sc[nt][k & 1], base[k & 1]));
                            sum[nt][k & 1] += p[k];
                        }
                        pb[pp][nt][0] = movmatrix_t(f16x2(p[0], p[1]));
                        pb[pp][nt][1] = movmatrix_t(f16x2(p[2], p[3]));
                    }
                }
                // output
#pragma unroll
                for (int pp = 0; pp < kPP; pp++) {
                    const uint32_t page = unit + pp * kQPageBytes;
                    uint32_t keep01 = 0xffffffffu, keep23 = 0xffffffffu;
                    if (tail) {
                        // tokens nobody sees: their scales may be NaN
                        const int left = len - (tok0 + pp * kPage + 4 * c4);
                        keep01 = (left > 0 ? 0xffffu : 0u) | (left > 1 ? 0xffff0000u : 0u);
                        keep23 = (left > 2 ? 0xffffu : 0u) | (left > 3 ? 0xffff0000u : 0u);
                    }
#pragma unroll
                    for (int w = 0; w < 2; w++) {
                        const uint4 t = lds16(page + kQV + w * 512 + lane * 16);
                        const uint4 sv = lds16(page + kQVScale + c4 * 32 + w * 16);
                        const uint32_t sw[4] = {sv.x, sv.y, sv.z, sv.w};
                        uint32_t a0[4], a1[4], a2[4], a3[4];
                        unpack8((t.x & 0x0f0f0f0fu) | ((t.y << 4) & 0xf0f0f0f0u), a0);
                        unpack8(((t.x >> 4) & 0x0f0f0f0fu) | (t.y & 0xf0f0f0f0u), a1);
                        unpack8((t.z & 0x0f0f0f0fu) | ((t.w << 4) & 0xf0f0f0f0u), a2);
                        unpack8(((t.z >> 4) & 0x0f0f0f0fu) | (t.w & 0xf0f0f0f0u), a3);
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const uint32_t s01 = scales2(sw[j]) & keep01, s23 = scales2(sw[j] >> 16) & keep23;
                            const uint32_t v0 = hmul2(a0[j], s01), v1 = hmul2(a1[j], s01), v2 = hmul2(a2[j], s23),
                                           v3 = hmul2(a3[j], s23);
#pragma unroll
                            for (int nt = 0; nt < NT; nt++)
                                mma_f16(o[nt][4 * w + j], v0, v1, v2, v3, pb[pp][nt][0], pb[pp][nt][1]);
                        }
                    }
                }
                // the stage is free once the team has read it
                if (RW > 1) named_bar(1 + team, RW * 32);
                else __syncwarp();
                issue(stage);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            pos += n;
            at.u = u0 + n - 1;
            step(at, sm, a.batch, Hkv);

            // the piece's sums over its tokens
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) sum[nt][h] += __shfl_xor_sync(0xffffffffu, sum[nt][h], off);
                }
            const bool whole = u0 == 0 && n == n_units;
            const int which = u0 + n == n_units ? 0 : 1;    // continues to the next team: the team's last piece
            if (!whole && part == 0 && lane == 0) sm.piece_group[2 * team + which] = b * Hkv + g;
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int r = row0 + nt * 8 + 2 * c4 + h;
                    if (r >= a.rows) continue;
                    const float l = sum[nt][h];
                    if (whole) {
                        const int qt = r / a.G;
                        const int64_t row = ((int64_t)b * a.n_query + qt) * a.heads + g * a.G + (r - qt * a.G);
                        const float inv = l == 0.f ? 0.f : a.st.v_scale / l;
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            const float x = l == 0.f ? 0.f : o[nt][j][h] * inv, y = l == 0.f ? 0.f : o[nt][j][2 + h] * inv;
                            *reinterpret_cast<uint32_t *>(a.out + row * kD + 16 * j + 2 * g8) =
                                bf16x2_bits(__floats2bfloat162_rn(x, y));
                        }
                        if (a.lse && g8 == 0)
                            a.lse[row] = l == 0.f ? -CUDART_INF_F : (ref[nt][h] - kPShift + log2f(l)) * kLn2;
                    } else {
                        const int64_t row = park + (int64_t)team * PADROWS + r;
                        float *dst = which ? parked_o(team, r) : a.part_o + row * kD;
#pragma unroll
                        for (int j = 0; j < 8; j++)
                            *reinterpret_cast<float2 *>(dst + 16 * j + 2 * g8) = make_float2(o[nt][j][h], o[nt][j][2 + h]);
                        if (g8 == 0) *(which ? parked_ml(team, r) : a.part_ml + row) = make_float2(ref[nt][h] - kPShift, l);
                    }
                }
        }
    }
    __threadfence_block();
    __syncthreads();

    // merge the parked pieces group by group
    int owner = -1, owner_last = 0;
    for (int i = 0; i < 2 * TEAMS;) {
        const int grp = sm.piece_group[i];
        if (grp < 0) {
            i++;
            continue;
        }
        int j = i + 1;
        while (j < 2 * TEAMS && (sm.piece_group[j] == grp || sm.piece_group[j] < 0)) j++;
        const int b = grp / Hkv, g = grp - b * Hkv;
        const long long n_units = sm.pre[b + 1] - sm.pre[b];
        const long long start = sm.pre[b] * Hkv + g * n_units, end = start + n_units;
        const bool whole = start >= cta_lo && end <= cta_hi;
        const int slot = start < cta_lo ? 0 : 1;
        if (!whole && slot == 1) {
            owner = grp;
            owner_last = (int)((end * grid - 1) / U);
        }
        for (int r = warp; r < a.rows; r += WARPS) {
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            float m = -CUDART_INF_F, l = 0.f;
            merge_rows<false>(j - i, [&](int k, const float2 *&ml, const float4 *&src) {
                const int t = (i + k) >> 1;
                const int64_t row = park + (int64_t)t * PADROWS + r;
                const bool last = (i + k) & 1;
                ml = sm.piece_group[i + k] < 0 ? &sm.nothing : last ? parked_ml(t, r) : a.part_ml + row;
                src = reinterpret_cast<const float4 *>(last ? parked_o(t, r) : a.part_o + row * kD);
            }, lane, o, m, l);
            if (whole) {
                finish4(a, b, g, r, lane * 4, o, m, l, lane == 0);
            } else {
                const int64_t row = crossing + slot * PADROWS + r;
                reinterpret_cast<float4 *>(a.part_o + row * kD)[lane] = o;
                if (lane == 0) a.part_ml[row] = make_float2(m, l);
            }
        }
        i = j;
    }
    if (tid == 0) a.meta[cta] = make_int4(owner, owner_last, 0, 0);
}

// Block (i, r): row r of the group that starts in block i of the attention
// grid and runs on into the blocks up to meta.y.
constexpr int kCombineWarps = 4;

__global__ void __launch_bounds__(kCombineWarps * 32) quant_combine_kernel(const __grid_constant__ QuantAttnArgs a,
                                                                          int padrows)
{
    __shared__ float4 so[kCombineWarps][32];
    __shared__ float2 sml[kCombineWarps];
    pdl_wait();
    const int4 meta = a.meta[blockIdx.x];
    if (meta.x < 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.y;
    const int n = meta.y - (int)blockIdx.x + 1;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -CUDART_INF_F, l = 0.f;
    // warp w takes partials w, w + 4, ...; then lane w of warp 0 the four warps' results
    merge_rows<true>((n - warp + kCombineWarps - 1) / kCombineWarps, [&](int i, const float2 *&ml, const float4 *&src) {
        const int k = i * kCombineWarps + warp;
        const int64_t row = ((int64_t)(blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * padrows + r;
        ml = a.part_ml + row;
        src = reinterpret_cast<const float4 *>(a.part_o + row * kD);
    }, lane, o, m, l);
    so[warp][lane] = o;
    if (lane == 0) sml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp) return;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    m = -CUDART_INF_F;
    l = 0.f;
    merge_rows<false>(kCombineWarps, [&](int i, const float2 *&ml, const float4 *&src) {
        ml = &sml[i];
        src = so[i];
    }, lane, o, m, l);
    const int b = meta.x / a.st.kv_heads;
    finish4(a, b, meta.x - b * a.st.kv_heads, r, lane * 4, o, m, l, lane == 0);
}

struct Variant {
    void (*kernel)(QuantAttnArgs);
    int teams, padrows, threads, blocks_per_sm;
    size_t smem;
};

// rows 1..8, 9..16, 17..32
template <int NT, int RW, int WARPS, int STAGES, int MINB>
Variant variant()
{
    return {quant_attention_kernel<NT, RW, WARPS, STAGES, MINB>, WARPS / RW, NT * 8 * RW, WARPS * 32, MINB,
            (size_t)(WARPS / RW) * STAGES * kUnitBytes};
}

Variant variant_for(int rows)
{
    if (rows <= 8) return variant<1, 1, 8, 2, 2>();
    if (rows <= 16) return variant<2, 1, 12, 3, 1>();
    return variant<2, 2, 12, 4, 1>();
}

int grid_of(const Variant &v, int sm_count)
{
    int grid = sm_count * v.blocks_per_sm;
    const int fit = kQPartRows / ((v.teams + 2) * v.padrows);     // blocks whose partial rows the scratch holds
    grid = grid < fit ? grid : fit;
    return grid < kMaxCtas ? grid : kMaxCtas;
}

}  // namespace

cudaError_t quant_attention_config(int sm_count)
{
    const int rows[3] = {8, 16, 32};
    for (int r : rows) {
        const Variant v = variant_for(r);
        const cudaError_t e = cudaFuncSetAttribute(v.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)v.smem);
        if (e != cudaSuccess) return e;
        if (grid_of(v, sm_count) < 1) return cudaErrorInvalidConfiguration;
    }
    return cudaSuccess;
}

cudaError_t launch_quant_attention(const QuantAttnArgs &a, int sm_count, cudaStream_t s)
{
    const Variant v = variant_for(a.rows);
    const int grid = grid_of(v, sm_count);
    cudaError_t e = launch_maybe_pdl(v.kernel, dim3(grid), dim3(v.threads), v.smem, s, true, a);
    if (e != cudaSuccess) return e;
    return launch_maybe_pdl(quant_combine_kernel, dim3(grid, a.rows), dim3(kCombineWarps * 32), 0, s, true, a, v.padrows);
}

}  // namespace macgpu
