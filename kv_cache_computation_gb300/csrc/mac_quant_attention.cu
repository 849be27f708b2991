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
//  - the orders of the contraction index and of the output's rows are free, so a
//    thread's K words are 32 consecutive elements of a token (two scales), and
//    its V words one 16-element block of four consecutive tokens (four scales),
//    whose codes are paired by token with two logic operations per eight codes.
// Roundings: Q is bf16 and becomes f16 with a power of two per row (exact but
// for elements below 2^-28 of the row's largest, which keep 2^-39 of it);
// stored values are exact in f16; the weights P, at most 2^15, are rounded to
// f16 (2^-11 of each, an eighth of the bf16 output's own rounding; P's factor 2^9
// keeps weights down to 2^-33 of the largest; a second product for their low
// halves would add half again to the tensor work) and summed unrounded in fp32;
// scores, sums, the reference and the output stay in fp32.
//
// Work split.  The units (two pages) of all (request, KV head) groups form one
// line, which is cut into equal ranges, one per warp, whatever the lengths; the
// cut is derived in every block from the lengths on the device, so a captured
// call serves any lengths, and it is fixed by them, so a call repeats bit for
// bit.  A group inside one warp's range is finished by it.  The pieces of the
// others are parked, merged per block, and, where a group crosses blocks, merged
// again by a second kernel.  No block waits for another.
//
// Measured (GB300, in a captured graph; stream against the copy peak of 6.7 TB/s):
//   rows  8 KV heads x 8 x 128K (1208 MB) 205 us, 5.9 TB/s   288 instructions a page
//         8 KV heads x 1 x 128K (151 MB)   37 us, 4.1
//         8 KV heads x 1 x 4K              12 us
//    16   1 KV head  x 8 x 128K (151 MB)   51 us, 3.0        392
//    24                                    61 us, 2.5
//    32                                    77 us, 2.0        477
// (One power of two for a whole group instead of one per row: 204, 37, 12, 51, 61
// and 74 us, but one row's size then costs the others their bits.)
// At 8 rows the stream runs at 6.2 TB/s while it lasts (the ALU, where a
// conversion takes two cycles, 56 % busy, the half-rate f16 multiplies 42 %); a
// single request pays the fixed chain besides: prologue 1.5 us, first page 1,
// merge 2, second kernel 4.  Beyond 8 rows a warp's 64 to 128 output registers
// leave 12 and 8 warps per SM, whose dependent instructions are not hidden
// (1.9 and 1.5 instructions a cycle, tensor pipe 31 % and 40 % busy).
// Tried and slower, us: at 8 rows (then 204) units of one page with 16 or 20 warps
// 248 and 263, 20 warps with spills 246, the next unit's scores in one block
// with this unit's output 212, value scales for every element block in every lane
// 240; at 16 / 32 rows (then 50 / 74) two warps per page with 16 rows each (84 at 32),
// pairs of warps that split scores by page and output by element 57 / 83, a unit's
// pages one after the other 52 / 80 and, with more warps, 58 / 170, keys
// and accumulators in tensor memory on tcgen05 71 / 98 (four barrier round trips
// per 128 tokens take longer than their stream).
#include "mac_device.cuh"
#include "mac_quant_merge.cuh"

namespace macgpu {

namespace {

constexpr int kPP = 2;                                  // pages per unit
constexpr int kUnitTok = kPP * kPage;
constexpr int kUnitBytes = kPP * kQPageBytes;

// The bytes of the first n of a word of four V scales (tokens 0, 2, 1, 3).
__device__ __forceinline__ uint32_t scales_of_first(int n)
{
    return (n > 0 ? 0xffu : 0u) | (n > 2 ? 0xff00u : 0u) | (n > 1 ? 0xff0000u : 0u) | (n > 3 ? 0xff000000u : 0u);
}

// A warp's shared memory: its ring and, where Q does not stay in registers, Q;
// at the end the piece it parks.
__host__ __device__ constexpr int team_bytes(int nt, int stages, bool qreg)
{
    const int run = stages * kUnitBytes + (qreg ? 0 : nt * 2048), parked = (nt * 8 * kParkRow * 4 + 127) / 128 * 128;
    return run > parked ? run : parked;
}

struct Smem : MergeState {
    unsigned long long bar[64];
    // several queries: the first token with a NaN scale that only some of them see, per warp and element block
    int bad[kMaxPieces / 2][kQBlocks];
    float row_sc[kMaxPieces / 2][kQMaxRows];    // log2 units of a row's raw scores, per warp
};

// NT: N tiles (8 rows each), TEAMS warps per block, STAGES units in a warp's
// ring.  Up to 16 rows a lane keeps its part of Q in registers, beyond that in
// shared memory (one 16-byte load per tile serves both pages of a unit).
template <int NT, int TEAMS, int STAGES, int MINB, bool QREG>
__global__ void __launch_bounds__(TEAMS * 32, MINB) quant_attention_kernel(const __grid_constant__ QuantAttnArgs a)
{
    constexpr int PADROWS = NT * 8;
    constexpr int PG = NT <= 2 ? kPP : 1;       // pages whose scores are made together, as registers allow
    constexpr int TEAM_BYTES = team_bytes(NT, STAGES, QREG);
    static_assert(2 * TEAMS <= kMaxPieces && TEAMS * STAGES <= 64, "block shape");
    extern __shared__ __align__(128) unsigned char dyn[];
    __shared__ Smem sm;
    const int tid = threadIdx.x, lane = tid & 31, team = tid >> 5;
    const int g8 = lane >> 2, c4 = lane & 3;
    const int Hkv = a.st.kv_heads;
    pdl_wait();
    pdl_launch_dependents();

    make_line<TEAMS, kUnitTok>(a, sm.line);
    const uint32_t bar0 = smem_u32(&sm.bar[team * STAGES]);
    const uint32_t ring = smem_u32(dyn) + (uint32_t)team * TEAM_BYTES;
    if (tid == 0) {
        for (int i = 0; i < TEAMS * STAGES; i++)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;\n" :: "r"(smem_u32(&sm.bar[i])) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (tid < 2 * TEAMS) sm.piece_group[tid] = -1;
    __syncthreads();

    // the block's and the warp's range of units
    const long long U = sm.line.pre[a.batch] * Hkv;
    // every warp of an active block has work: blocks beyond that stay idle
    const long long most = U >= TEAMS ? U / TEAMS : 1;
    const int grid = most < (long long)gridDim.x ? (int)most : (int)gridDim.x;
    const int cta = blockIdx.x;
    const bool by_group = meta_by_group(a, gridDim.x);
    if (cta >= grid) {
        if (tid == 0 && !by_group) a.meta[cta] = make_int4(-1, 0, 0, 0);
        return;
    }
    const Cut cut(U, grid * TEAMS);
    const long long lo = cut.first(cta * TEAMS + team), hi = cut.first(cta * TEAMS + team + 1);
    const long long cta_lo = cut.first(cta * TEAMS), cta_hi = cut.first((cta + 1) * TEAMS);
    if (tid == 0) {
        sm.lo = cta_lo;     // for the merge behind the long loop
        sm.hi = cta_hi;
    }
    const Parking park{dyn, TEAM_BYTES, TEAMS, PADROWS};

    if (lo < hi) {
        int left = (int)(hi - lo);      // units to go
        int b, g, u0, n_units;
        locate(a, sm.line, lo, b, g, u0, n_units);

        // The copies run ahead of the reading over the same units: ld_group units of (ld_b, ld_g) to go, tokens from
        // the next unit on in the request, and the lane's page id of that unit, read one unit ahead.
        const size_t page_stride = (size_t)Hkv * kQPageBytes;
        int ld_left = left, ld_b = b, ld_g = g, ld_group = n_units - u0, ld_tok = sm.line.len[b] - u0 * kUnitTok;
        const int32_t *ld_ids = a.table + (int64_t)b * a.table_stride + u0 * kPP + lane;
        int next_id = 0;
        auto fetch = [&]() {
            next_id = 0;
            if (lane < kPP && lane * kPage < ld_tok) next_id = *ld_ids;     // checked where it is used, when it has arrived
        };
        auto issue = [&](int s) {
            if (ld_left == 0) return;
            const uint32_t bar = bar0 + 8 * s;
            if ((unsigned)next_id >= (unsigned)a.st.num_pages) {
                atomicOr(a.st.err, kQErrPage);
                next_id = 0;            // stays inside the store; the request's output is wrong
            }
            const int pages = ld_tok > kPage ? 2 : ld_tok > 0 ? 1 : 0;
            if (lane == 0)
                asm volatile("{\n.reg .b64 st;\nmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n}\n"
                             :: "r"(bar), "r"((uint32_t)pages * kQPageBytes)
                             : "memory");
            __syncwarp();
            if (lane < pages)
                bulk_load(ring + (uint32_t)s * kUnitBytes + lane * kQPageBytes,
                          a.st.pages + (size_t)(unsigned)next_id * page_stride + (size_t)ld_g * kQPageBytes, kQPageBytes, bar);
            if (--ld_left == 0) return;
            if (--ld_group == 0) {
                if (++ld_g == Hkv) {
                    ld_g = 0;
                    ld_b++;
                }
                ld_group = (int)(sm.line.pre[ld_b + 1] - sm.line.pre[ld_b]);
                ld_tok = sm.line.len[ld_b];
                ld_ids = a.table + (int64_t)ld_b * a.table_stride + lane;
            } else {
                ld_tok -= kUnitTok;
                ld_ids += kPP;
            }
            fetch();
        };
        static_assert(kPP == 2, "a unit has one or two pages");
        fetch();
#pragma unroll
        for (int s = 0; s < STAGES; s++) issue(s);

        // while the first pages arrive: the group that starts in this block and runs on behind it, for the second kernel
        // (the last warp of a block always has a unit)
        if (team == TEAMS - 1 && lane == 0) write_meta(a, sm.line, cut, U, grid, TEAMS, cta_lo, cta_hi);

        int stage = 0;
        uint32_t phase = 0;
        const int tk = 4 * (g8 >> 1) + (g8 & 1);    // token of matrix row g; row g + 8 is token tk + 2
        while (left > 0) {
            // one piece: units [u0, u0 + n) of group (b, g)
            const int n = min(left, n_units - u0);
            const int len = sm.line.len[b];
            const int full = max(len - (a.n_query - 1), 0);     // tokens every row sees
            uint32_t qf[QREG ? NT : 1][16];
            // low: the row's reference less kPShift, weights are 2^(score - low)
            float low[NT][2], sum[NT][2], o[NT][8][4];
            // Q in f16, each row times the power of two that brings its largest finite element into [2^14, 2^15), so that
            // no row depends on another's size; row_sc takes a row's raw scores to log2 units
            uint32_t w[16];
            auto load_row = [&](int nt) {
                load_q(a, b, g, nt * 8 + g8, c4, w);
                uint32_t top = finite_top(w);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const int shift = top ? min(14 - ((int)(top >> 7) - 127), 126) : 0;
                if (c4 == 0)
                    sm.row_sc[team][nt * 8 + g8] = fmaxf(a.scale_log2 * __int_as_float((127 - shift) << 23), 1e-37f);
                return __int_as_float((shift + 127) << 23);
            };
            if (QREG) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    const float up = load_row(nt);
#pragma unroll
                    for (int i = 0; i < 16; i++) qf[nt][i] = scaled_f16x2(w[i], up);
                }
            } else {
                const uint32_t q0 = ring + STAGES * kUnitBytes + lane * 16;
#pragma unroll 1
                for (int nt = 0; nt < NT; nt++) {
                    const float up = load_row(nt);
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        uint32_t f[4];
#pragma unroll
                        for (int k = 0; k < 4; k++) f[k] = scaled_f16x2(w[4 * i + k], up);
                        sts16(q0 + (nt * 4 + i) * 512, f);
                    }
                }
            }
            const uint32_t sc0 = smem_u32(&sm.row_sc[team][2 * c4]);
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    low[nt][h] = kLowest;
                    sum[nt][h] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 8; j++)
#pragma unroll
                    for (int k = 0; k < 4; k++) o[nt][j][k] = 0.f;
            }

            __syncwarp();
            if (lane < kQBlocks) sm.bad[team][lane] = 0x7fffffff;
            __syncwarp();
            for (int i = 0; i < n; i++) {
                if (!mbar_wait(bar0 + 8 * stage, phase)) atomicOr(a.st.err, kQErrTimeout);
                const uint32_t unit = ring + (uint32_t)stage * kUnitBytes;
                const int tok0 = (u0 + i) * kUnitTok;
                const bool tail = tok0 + kUnitTok > full;

                // scores of both pages
                float s[kPP][NT][4];
#pragma unroll
                for (int pp = 0; pp < kPP; pp++)
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int k = 0; k < 4; k++) s[pp][nt][k] = 0.f;
#pragma unroll
                for (int p0 = 0; p0 < kPP; p0 += PG) {
                    uint32_t wa[PG][4], wb[PG][4], xa[PG][2], xb[PG][2];
#pragma unroll
                    for (int pp = 0; pp < PG; pp++) {
                        const uint32_t page = unit + (p0 + pp) * kQPageBytes;
                        const uint4 ka = lds16(page + tk * 64 + c4 * 16), kb = lds16(page + (tk + 2) * 64 + c4 * 16);
                        wa[pp][0] = ka.x, wa[pp][1] = ka.y, wa[pp][2] = ka.z, wa[pp][3] = ka.w;
                        wb[pp][0] = kb.x, wb[pp][1] = kb.y, wb[pp][2] = kb.z, wb[pp][3] = kb.w;
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            // the scale's f16 (times 2^-8) in both halves
                            const uint32_t at = page + kQKScale + (g8 >> 1) * 32 + (2 * c4 + h) * 4 + (g8 & 1);
                            xa[pp][h] = lds1(at) * 0x00800080u;
                            xb[pp][h] = lds1(at + 2) * 0x00800080u;
                        }
                    }
#pragma unroll
                    for (int w = 0; w < 4; w++) {
                        uint32_t ha[PG][4], hb[PG][4];
#pragma unroll
                        for (int pp = 0; pp < PG; pp++) {
                            unpack8(wa[pp][w], ha[pp]);
                            unpack8(wb[pp][w], hb[pp]);
#pragma unroll
                            for (int k = 0; k < 4; k++) {
                                ha[pp][k] = hmul2(ha[pp][k], xa[pp][w >> 1]);
                                hb[pp][k] = hmul2(hb[pp][k], xb[pp][w >> 1]);
                            }
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; nt++) {
                            uint32_t f[4];
                            if (QREG) {
#pragma unroll
                                for (int k = 0; k < 4; k++) f[k] = qf[nt][4 * w + k];
                            } else {
                                const uint4 v = lds16(ring + STAGES * kUnitBytes + ((nt * 4 + w) * 32 + lane) * 16);
                                f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
                            }
#pragma unroll
                            for (int k = 0; k < 2; k++)
#pragma unroll
                                for (int pp = 0; pp < PG; pp++)
                                    mma_f16(s[p0 + pp][nt], ha[pp][2 * k], hb[pp][2 * k], ha[pp][2 * k + 1],
                                            hb[pp][2 * k + 1], f[2 * k], f[2 * k + 1]);
                        }
                    }
                }
                if (tail) {
                    // Value scales that may be NaN, whose product with a weight of 0 would be NaN: those of tokens nobody
                    // sees, and the NaN scales of tokens that some of several queries see, are made zero in the ring.
                    // (lane: word (page, c, block) of the unit's scales, bytes of tokens 0, 2, 1, 3)
#pragma unroll 1
                    for (int k = lane; k < kPP * 32; k += 32) {
                        const int first = tok0 + (k >> 5) * kPage + 4 * ((k >> 3) & 3);
                        const uint32_t at = unit + (k >> 5) * kQPageBytes + kQVScale + (k & 31) * 4;
                        uint32_t sv = lds4(at) & scales_of_first(len - first);
                        const uint32_t nan = __vcmpeq4(sv, 0xffffffffu) & ~scales_of_first(full - first);
                        if (nan)
                            atomicMin(&sm.bad[team][k & 7],
                                      first + (nan & 0xffu ? 0 : nan & 0xff0000u ? 1 : nan & 0xff00u ? 2 : 3));
                        sts4(at, sv & ~nan);
                    }
                    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");   // a later copy writes the same bytes
                    __syncwarp();
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const int r = nt * 8 + 2 * c4 + h, lim = r < a.rows ? len - (a.n_query - 1) + r / a.G : 0;
#pragma unroll
                            for (int pp = 0; pp < kPP; pp++)
#pragma unroll
                                for (int k = 0; k < 2; k++)
                                    if (tok0 + pp * kPage + tk + 2 * k >= lim) s[pp][nt][2 * k + h] = -CUDART_INF_F;
                        }
                }
                // softmax: the reference moves only when a score passes it by more than the margin.  Scores are rounded
                // before the reference is taken off, as the reference was: a fused product would be off by its rounding,
                // which passes any margin for scores beyond 2^27.
                float x[NT][2];
                bool moves = false;
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    float sc[2];
                    lds8(sc0 + nt * 32, sc);
#pragma unroll
                    for (int h = 0; h < 2; h++) {
#pragma unroll
                        for (int pp = 0; pp < kPP; pp++) {
                            s[pp][nt][h] = __fmul_rn(s[pp][nt][h], sc[h]);
                            s[pp][nt][2 + h] = __fmul_rn(s[pp][nt][2 + h], sc[h]);
                        }
                        x[nt][h] = fmaxf(s[0][nt][h], s[0][nt][2 + h]);
#pragma unroll
                        for (int pp = 1; pp < kPP; pp++) x[nt][h] = fmaxf(x[nt][h], fmaxf(s[pp][nt][h], s[pp][nt][2 + h]));
                        moves |= x[nt][h] - low[nt][h] > kMargin + kPShift;
                    }
                }
                if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            float y = x[nt][h];
#pragma unroll
                            for (int off = 4; off < 32; off <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, off));
                            // a row moves by its own scores alone; those of 2^23 and more are whole numbers too coarse to
                            // take the shift from
                            y = y - low[nt][h] > kMargin + kPShift ? (fabsf(y) < 0x1p23f ? y - kPShift : y) : low[nt][h];
                            const float f = ex2_approx(low[nt][h] - y);
                            low[nt][h] = y;
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
#pragma unroll
                    for (int pp = 0; pp < kPP; pp++) {
                        float p[4];
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            p[k] = ex2_approx(s[pp][nt][k] - low[nt][k & 1]);
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
                    const uint32_t sv = lds4(page + kQVScale + c4 * 32 + g8 * 4);
                    // f16 pairs of the scales of tokens 0, 1 and 2, 3, times 2^-8
                    const uint32_t s01 = (sv & 0x00ff00ffu) << 7, s23 = (sv & 0xff00ff00u) >> 1;
#pragma unroll
                    for (int w = 0; w < 2; w++) {
                        const uint4 t = lds16(page + kQV + w * 512 + lane * 16);
                        uint32_t a0[4], a1[4], a2[4], a3[4];
                        unpack8((t.x & 0x0f0f0f0fu) | ((t.y << 4) & 0xf0f0f0f0u), a0);
                        unpack8(((t.x >> 4) & 0x0f0f0f0fu) | (t.y & 0xf0f0f0f0u), a1);
                        unpack8((t.z & 0x0f0f0f0fu) | ((t.w << 4) & 0xf0f0f0f0u), a2);
                        unpack8(((t.z >> 4) & 0x0f0f0f0fu) | (t.w & 0xf0f0f0f0u), a3);
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const uint32_t v0 = hmul2(a0[j], s01), v1 = hmul2(a1[j], s01), v2 = hmul2(a2[j], s23),
                                           v3 = hmul2(a3[j], s23);
#pragma unroll
                            for (int nt = 0; nt < NT; nt++)
                                mma_f16(o[nt][4 * w + j], v0, v1, v2, v3, pb[pp][nt][0], pb[pp][nt][1]);
                        }
                    }
                }
                __syncwarp();       // the stage is free once the warp has read it
                issue(stage);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            left -= n;

            const int bad = sm.bad[team][g8];
            if (__any_sync(0xffffffffu, bad != 0x7fffffff)) {
                // the queries that see a token whose scale was made zero get its NaN here (the lane's outputs are of block g)
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const int r = nt * 8 + 2 * c4 + h;
                        if (r >= a.rows || len - (a.n_query - 1) + r / a.G <= bad) continue;
#pragma unroll
                        for (int j = 0; j < 8; j++) o[nt][j][h] = o[nt][j][2 + h] = CUDART_NAN_F;
                    }
            }

            // the piece's sums over its tokens
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) sum[nt][h] += __shfl_xor_sync(0xffffffffu, sum[nt][h], off);
                }
            const bool ends = u0 + n == n_units, whole = u0 == 0 && ends;
            const int which = ends ? 0 : 1;     // 1: the group runs on into the next warp's range
            if (lane == 0) {
                if (!whole) sm.piece_group[2 * team + which] = b * Hkv + g;
                else if (meta_by_group(a, gridDim.x)) a.meta[b * Hkv + g] = make_int4(-1, 0, 0, 0);
            }
            if (which) __syncwarp();            // the parked piece takes the place of what the warp has read
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int r = nt * 8 + 2 * c4 + h;
                    if (r >= a.rows) continue;
                    const float l = sum[nt][h];
                    if (whole) {
                        const int qt = r / a.G;
                        const int64_t row = ((int64_t)b * a.n_query + qt) * a.heads + g * a.G + (r - qt * a.G);
                        const float inv = l == 0.f ? 0.f : a.v_out_scale / l;
                        uint32_t y[8];
#pragma unroll
                        for (int j = 0; j < 8; j++)
                            y[j] = l == 0.f ? 0u : bf16x2_bits(__floats2bfloat162_rn(o[nt][j][h] * inv, o[nt][j][2 + h] * inv));
                        uint4 *dst = reinterpret_cast<uint4 *>(a.out + row * kD + 16 * g8);
                        dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
                        dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
                        if (a.lse && g8 == 0)
                            a.lse[row] = l == 0.f ? -CUDART_INF_F : (low[nt][h] + log2f(l)) * kLn2;
                    } else {
                        const int64_t row = park.first_row(team, r);
                        float *dst = which ? park.last_o(team, r) : a.part_o + row * kD;
#pragma unroll
                        for (int j = 0; j < 8; j += 2)
                            *reinterpret_cast<float4 *>(dst + 16 * g8 + 2 * j) =
                                make_float4(o[nt][j][h], o[nt][j][2 + h], o[nt][j + 1][h], o[nt][j + 1][2 + h]);
                        if (g8 == 0) *(which ? park.last_ml(team, r) : a.part_ml + row) = make_float2(low[nt][h], l);
                    }
                }
            // the next group
            u0 = 0;
            if (++g == Hkv) {
                g = 0;
                if (++b < a.batch) n_units = (int)(sm.line.pre[b + 1] - sm.line.pre[b]);
            }
        }
    }
    merge_pieces<TEAMS, TEAMS, false>(a, sm, park);
}

struct Variant {
    void (*kernel)(QuantAttnArgs);
    int teams, padrows, blocks_per_sm;
    size_t smem;
};

template <int NT, int TEAMS, int STAGES, int MINB, bool QREG>
Variant variant()
{
    return {quant_attention_kernel<NT, TEAMS, STAGES, MINB, QREG>, TEAMS, NT * 8, MINB,
            (size_t)TEAMS * team_bytes(NT, STAGES, QREG)};
}

// As many warps as the registers of an output tile of 8 NT rows leave room for.
Variant variant_for(int rows)
{
    if (rows <= 8) return variant<1, 8, 2, 2, true>();
    if (rows <= 16) return variant<2, 12, 2, 1, true>();
    if (rows <= 24) return variant<3, 8, 3, 1, false>();
    return variant<4, 8, 3, 1, false>();
}

int grid_of(const Variant &v, int sm_count) { return quant_grid(sm_count, v.blocks_per_sm, v.teams, v.padrows); }

}  // namespace

cudaError_t quant_attention_config(int sm_count)
{
    const int rows[4] = {8, 16, 24, 32};
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
    cudaError_t e = launch_maybe_pdl(v.kernel, dim3(grid), dim3(v.teams * 32), v.smem, s, true, a);
    if (e != cudaSuccess) return e;
    return launch_quant_combine<false>(a, grid, v.padrows, sm_count, s);
}

}  // namespace macgpu
