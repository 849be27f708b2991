// Decode attention over the 8-bit store (format and layout: mac_block.cuh).
//
// Per request (len tokens) and KV head, the group's heads times the request's
// n_query new tokens are `rows` rows (at most 32); row r is head r % G of
// query token r / G and sees the first len - (n_query - 1) + r / G tokens:
//   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q . k_t),
//   lse = log sum_t p_t;  a row that sees nothing gives out 0, lse -inf.
// With s_t the scores in log2 units, keys 2^ek and values 2^ev times their codes
// (ek, ev of t's page), and any reference low:
//   w_t = 2^(s_t + ev - low),  out = sum_t w_t code_t / l,  l = sum_t w_t 2^-ev,
//   lse = ln 2 (low + log2 l)
// so that a page's value scale costs one subtraction per row and page: it goes
// into the exponent, the reference is that of the products, and the codes need
// no scaling at all.  A w below fp32's range adds nothing to out, but w 2^-ev may
// still count in l: there it is taken as one power, 2^(s_t - low), and so are the
// factors that bring sums to a later reference (sum_at).  Scores of 2^23 and more,
// which exponents cannot be added to, are held less a whole number per row.
//
// Rows, products, fragments' free orders, the split into equal ranges of a line
// of units and the merge of pieces are those of the 4-bit store's attention
// (mac_quant_attention.cu, mac_quant_line.cuh, mac_quant_merge.cuh), but that a
// piece's own cost counts in the line: a warp takes whole pages from a ring of its own, scores are S^T = K Q^T, the output O^T +=
// V^T P^T, both mma.m16n8k16 in f16 with fp32 accumulators.
// Roundings: Q is bf16 and becomes f16 with a power of two per row (exact but
// for elements below 2^-28 of the row's largest); codes are exact in f16;
// the weights w, at most 2^15, are rounded to f16 (2^-11 of each) and summed
// unrounded in fp32; everything else stays in fp32.
//
// Measured (graph replays, 258 bytes per token and KV head): 8 x 131072, 32 / 8
// heads 321 us (6.7 TB/s, the copy rate); 1 x 4096 14 us; 4 ragged requests to
// 122880, 21 rows for each of 4 heads 64 us (3.7 TB/s); 32 ragged ones to 65536,
// 32 rows on one head 81 us (2.7 TB/s).  8 x 65536 with 8 heads at 4, 8, 12, 16,
// 24, 32 rows: 169, 174, 175, 178, 202, 258 us.
// What bounds it.  Up to 16 rows the stream, around which a call pays about 12 us:
// launch, lengths and line, the first page, the merges and the second kernel.  With
// more rows the registers leave two warps to a scheduler, whose dependent
// instructions' latencies nothing covers (issue slots 36 % used, tensor pipe 40 %
// at 32 rows).
#include "mac_block.cuh"
#include "mac_quant_merge.cuh"

namespace macgpu {

namespace {

// two e4m3 codes (low, high byte) -> f16x2, exact
__device__ __forceinline__ void unpack4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Value scales below this one can make a token whose weight w is under fp32's range (2^-126 of the row's reference) count in
// l, by w 2^-ev: l is at least 2^9 2^-60, and as many tokens as a length can hold, each 2^-126 2^-ev, stay below 2^-24 of
// that for ev >= -21.
constexpr int kSmallExp = -21, kAlways = 1000;

__host__ __device__ constexpr int block_team_bytes(int nt, int pp, int stages, bool qreg)
{
    const int run = stages * pp * kBCopyBytes + (qreg ? 0 : nt * 2048), parked = nt * 8 * kParkRow * 4;
    return ((run > parked ? run : parked) + 127) / 128 * 128;
}

template <int TEAMS>
struct BlockSmem : MergeState {
    unsigned long long bar[64];
    // several queries: the first token with a NaN that only some of them see, per warp and element
    int bad[TEAMS][kD];
    float row_sc[TEAMS][kQMaxRows];     // log2 units of a row's raw scores, per warp
    // what is taken off a row's scores where they are too coarse, in all and by the last step, per warp
    float row_base[TEAMS][kQMaxRows], row_off[TEAMS][kQMaxRows];
};

// A quad of tokens' value codes (4 elements x 4 tokens) of which the request has
// `live` tokens, the first `sure` of them seen by every row: codes of others
// become 0, and so do NaN codes behind `sure`, whose tokens are noted in bad.
__device__ __forceinline__ uint32_t clean_values(uint32_t w, int live, int sure, int first, int *bad)
{
    const uint32_t keep = live >= 4 ? 0xffffffffu : live <= 0 ? 0u : (1u << 8 * live) - 1u;
    const uint32_t known = sure >= 4 ? 0xffffffffu : sure <= 0 ? 0u : (1u << 8 * sure) - 1u;
    w &= keep;
    const uint32_t nan = __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) & ~known;
    if (nan) atomicMin(bad, first + ((__ffs(nan) - 1) >> 3));
    return w & ~nan;
}

// NT: N tiles (8 rows each), TEAMS warps per block, STAGES units of PP pages in
// a warp's ring.  Up to 16 rows a lane keeps its part of Q in registers, beyond
// that in shared memory.
template <int NT, int PP, int TEAMS, int STAGES, int MINB, bool QREG>
__global__ void __launch_bounds__(TEAMS * 32, MINB) block_attention_kernel(const __grid_constant__ QuantAttnArgs a)
{
    constexpr int PADROWS = NT * 8, UNIT_TOK = PP * kPage, UNIT_BYTES = PP * kBCopyBytes;
    // What a piece costs besides its units, in units: Q, the first scores, the rows on their way out.  By the clock 1 to
    // 2 units at 8 rows, 2.4 at 16, 3.2 at 24, 4 to 5 at 32.  us with 0, NT, NT + 2 (and 2 NT) units: 4 ragged requests of
    // 21 rows for each of 4 KV heads 92, 77.8, 60.2 (60.3), the same of 28 rows 64.6 / 59.6 / 51.7; 32 ragged requests of
    // 32 rows on one head 92.7 / 81.5 / 78.2 (78.9), of 8 rows 48.9 / 46.6 / 46.1; long uniform ones and one of 4096 tokens
    // are the same with all.
    constexpr int EXTRA = NT + 2;
    constexpr int TEAM_BYTES = block_team_bytes(NT, PP, STAGES, QREG);
    static_assert(kQMaxRows == 32 && 2 * TEAMS <= kMaxPieces && TEAMS * STAGES <= 64, "block shape");
    extern __shared__ __align__(128) unsigned char dyn[];
    __shared__ BlockSmem<TEAMS> sm;
    const int tid = threadIdx.x, lane = tid & 31, team = tid >> 5;
    const int g8 = lane >> 2, c4 = lane & 3;
    const int Hkv = a.st.kv_heads;
    pdl_wait();
    pdl_launch_dependents();

    make_line<TEAMS, UNIT_TOK, EXTRA>(a, sm.line);
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
    const long long most = U >= TEAMS ? U / TEAMS : 1;      // every warp of an active block has work
    const int grid = most < (long long)gridDim.x ? (int)most : (int)gridDim.x;
    const int cta = blockIdx.x;
    const bool by_group = meta_by_group(a, gridDim.x);
    if (cta >= grid) {
        if (tid == 0 && !by_group) a.meta[cta] = make_int4(-1, 0, 0, 0);
        return;
    }
    // The warp's range and the block's.  A bound that would leave a piece with extra units alone moves to its group's
    // beginning.  A warp's range may be empty then; the block's, of TEAMS units and more, is not.
    static_assert(EXTRA + 1 < TEAMS, "a block has a piece");
    const Cut cut(U, grid * TEAMS);
    long long bound = U;
    {
        const int at = lane & 1 ? team + 1 : team, i = cta * TEAMS + (lane & 2 ? (lane & 1 ? TEAMS : 0) : at);
        const long long p = cut.first(i);
        if (p < U) {
            int b, g, u, n;
            locate(a, sm.line, p, b, g, u, n);
            bound = u <= EXTRA ? p - u : p;
        }
    }
    const long long lo = __shfl_sync(0xffffffffu, bound, 0), hi = __shfl_sync(0xffffffffu, bound, 1),
                    cta_lo = __shfl_sync(0xffffffffu, bound, 2), cta_hi = __shfl_sync(0xffffffffu, bound, 3);
    if (tid == 0) {
        sm.lo = cta_lo;     // for the merge behind the long loop
        sm.hi = cta_hi;
    }
    const Parking park{dyn, TEAM_BYTES, TEAMS, PADROWS};
    // the group that starts in this block and runs on behind it, for the second kernel
    auto leave_meta = [&] {
        if (team == TEAMS - 1 && lane == 0) write_meta(a, sm.line, cut, U, grid, TEAMS, cta_lo, cta_hi);
    };
    if (lo >= hi) leave_meta();

    if (lo < hi) {
        int left = (int)(hi - lo);      // units to go, extra ones among them
        int b, g, u0, n_units;
        locate(a, sm.line, lo, b, g, u0, n_units);
        // a group's own units: from its beginning EXTRA fewer
        int n = min(left, n_units - u0) - (u0 == 0 ? EXTRA : 0);
        if (u0) u0 -= EXTRA;

        // The copies run ahead of the reading over the same units: ld_group units of (ld_b, ld_g) to go and ld_left behind
        // them, tokens from the next unit on in the request, and the lane's page id of that unit, read one unit ahead.
        const size_t page_stride = (size_t)Hkv * kBPageBytes;
        int ld_b = b, ld_g = g, ld_group = n, ld_left = left - n - (u0 ? 0 : EXTRA), ld_tok = sm.line.len[b] - u0 * UNIT_TOK;
        const int32_t *ld_ids = a.table + (int64_t)b * a.table_stride + u0 * PP + lane;
        int next_id = 0;
        auto fetch = [&]() {
            next_id = 0;
            if (lane < PP && lane * kPage < ld_tok) next_id = *ld_ids;      // checked where it is used, when it has arrived
        };
        auto issue = [&](int s) {
            if (ld_group == 0) return;
            const uint32_t bar = bar0 + 8 * s;
            if ((unsigned)next_id >= (unsigned)a.st.num_pages) {
                atomicOr(a.st.err, kQErrPage);
                next_id = 0;            // stays inside the store; the request's output is wrong
            }
            int pages = 0;
#pragma unroll
            for (int p = 0; p < PP; p++) pages += ld_tok > p * kPage;
            if (lane == 0)
                asm volatile("{\n.reg .b64 st;\nmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n}\n"
                             :: "r"(bar), "r"((uint32_t)pages * kBCopyBytes)
                             : "memory");
            __syncwarp();
            if (lane < pages)
                bulk_load(ring + (uint32_t)s * UNIT_BYTES + lane * kBCopyBytes,
                          a.st.pages + (size_t)(unsigned)next_id * page_stride + (size_t)ld_g * kBPageBytes, kBCopyBytes, bar);
            if (--ld_group == 0) {
                if (ld_left == 0) return;
                if (++ld_g == Hkv) {
                    ld_g = 0;
                    ld_b++;
                }
                const int all = min(ld_left, (int)(sm.line.pre[ld_b + 1] - sm.line.pre[ld_b]));
                ld_left -= all;
                ld_group = all - EXTRA;
                ld_tok = sm.line.len[ld_b];
                ld_ids = a.table + (int64_t)ld_b * a.table_stride + lane;
            } else {
                ld_tok -= UNIT_TOK;
                ld_ids += PP;
            }
            fetch();
        };
        fetch();
#pragma unroll
        for (int s = 0; s < STAGES; s++) issue(s);

        leave_meta();                   // while the first pages arrive

        int stage = 0;
        uint32_t phase = 0;
        const int tk = 4 * (g8 >> 1) + (g8 & 1);    // token of matrix row g; row g + 8 is token tk + 2
        while (left > 0) {
            // one piece: units [u0, u0 + n) of group (b, g)
            const int len = sm.line.len[b];
            const int full = max(len - (a.n_query - 1), 0);     // tokens every row sees
            uint32_t qf[QREG ? NT : 1][16];
            // low: the row's reference less kPShift, weights are 2^(score + ev - low)
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
                const uint32_t q0 = ring + STAGES * UNIT_BYTES + lane * 16;
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
            const uint32_t sc0 = smem_u32(&sm.row_sc[team][2 * c4]), base0 = smem_u32(&sm.row_base[team][2 * c4]);
            int small = kSmallExp;      // kAlways where some row's base is not 0
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
            sm.row_base[team][lane] = 0.f;
            if (a.n_query > 1) {
#pragma unroll
                for (int i = 0; i < kD / 32; i++) sm.bad[team][lane + 32 * i] = 0x7fffffff;
            }
            bool met = false;       // a NaN was noted in bad
            __syncwarp();
            for (int i = 0; i < n; i++) {
                if (!mbar_wait(bar0 + 8 * stage, phase)) atomicOr(a.st.err, kQErrTimeout);
                const uint32_t unit = ring + (uint32_t)stage * UNIT_BYTES;
                const int tok0 = (u0 + i) * UNIT_TOK;
                const bool tail = tok0 + UNIT_TOK > full;

                // scores of the unit's pages
                float s[PP][NT][4];
                int ek[PP], ev[PP];
#pragma unroll
                for (int pp = 0; pp < PP; pp++) {
                    const uint32_t e0 = lds4(unit + pp * kBCopyBytes + kBTail), e1 = lds4(unit + pp * kBCopyBytes + kBTail + 4);
                    // a page behind the request's last was not copied: any bytes
                    ek[pp] = (int)min(e0, (uint32_t)kBExpTop) - kBExpBias;
                    ev[pp] = (int)min(e1, (uint32_t)kBExpTop) - kBExpBias;
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int k = 0; k < 4; k++) s[pp][nt][k] = 0.f;
                }
#pragma unroll
                for (int i2 = 0; i2 < 2; i2++) {
                    // Q of the lane's elements 16 i2 .. 16 i2 + 15, two 16-byte words of fragments
                    uint32_t f[NT][8];
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) {
                        if (QREG) {
#pragma unroll
                            for (int k = 0; k < 8; k++) f[nt][k] = qf[nt][8 * i2 + k];
                        } else {
#pragma unroll
                            for (int k = 0; k < 2; k++) {
                                const uint4 v = lds16(ring + STAGES * UNIT_BYTES + ((nt * 4 + 2 * i2 + k) * 32 + lane) * 16);
                                f[nt][4 * k] = v.x, f[nt][4 * k + 1] = v.y, f[nt][4 * k + 2] = v.z, f[nt][4 * k + 3] = v.w;
                            }
                        }
                    }
#pragma unroll
                    for (int pp = 0; pp < PP; pp++) {
                        const uint32_t page = unit + pp * kBCopyBytes;
                        const uint4 ka = lds16(page + i2 * 512 + lane * 16), kb = lds16(page + (2 + i2) * 512 + lane * 16);
                        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            uint32_t a0, a1, a2, a3;
                            unpack4(wa[k], a0, a2);
                            unpack4(wb[k], a1, a3);
#pragma unroll
                            for (int nt = 0; nt < NT; nt++) mma_f16(s[pp][nt], a0, a1, a2, a3, f[nt][2 * k], f[nt][2 * k + 1]);
                        }
                    }
                }
                // softmax: the reference moves only when a product's exponent passes it by more than the margin.  Scores
                // are rounded before the reference is taken off, as the reference was.
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    float sc[2];
                    lds8(sc0 + nt * 32, sc);
#pragma unroll
                    for (int h = 0; h < 2; h++)
#pragma unroll
                        for (int pp = 0; pp < PP; pp++) {
                            const float f = __fmul_rn(sc[h], __int_as_float((ek[pp] + 127) << 23));
                            s[pp][nt][h] = __fmul_rn(s[pp][nt][h], f);
                            s[pp][nt][2 + h] = __fmul_rn(s[pp][nt][2 + h], f);
                        }
                }
                if (tail) {
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            const int r = nt * 8 + 2 * c4 + h, lim = r < a.rows ? len - (a.n_query - 1) + r / a.G : 0;
#pragma unroll
                            for (int pp = 0; pp < PP; pp++)
#pragma unroll
                                for (int k = 0; k < 2; k++)
                                    if (tok0 + pp * kPage + tk + 2 * k >= lim) s[pp][nt][2 * k + h] = -CUDART_INF_F;
                        }
                }
                auto top_products = [&](float (&x)[NT][2]) {
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            x[nt][h] = -CUDART_INF_F;
#pragma unroll
                            for (int pp = 0; pp < PP; pp++)
                                x[nt][h] = fmaxf(x[nt][h], fmaxf(s[pp][nt][h], s[pp][nt][2 + h]) + (float)ev[pp]);
                        }
                };
                float x[NT][2];
                top_products(x);
                bool moves = false;
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int h = 0; h < 2; h++) moves |= x[nt][h] - low[nt][h] > kMargin + kPShift;
                int least = ev[0];
#pragma unroll
                for (int pp = 1; pp < PP; pp++) least = min(least, ev[pp]);
                // What small scales and coarse scores need stands behind the branch of references that move (8 x 65536, us at 24
                // and 32 rows: 208 and 262 beside it, 202 and 258 in it).
                moves |= least < small;
                if (__any_sync(0xffffffffu, moves)) {
                    // Scores of 2^23 and more are too coarse to add exponents to and to take the shift from: such a row's are from
                    // here on those above its largest product now, and the second pass takes that off this unit's.
                    uint32_t off = base0;
#pragma unroll 1
                    for (int pass = 0; pass < 2; pass++) {
                        if (small == kAlways) {
#pragma unroll
                            for (int nt = 0; nt < NT; nt++) {
                                float base[2];
                                lds8(off + nt * 32, base);
#pragma unroll
                                for (int pp = 0; pp < PP; pp++)
#pragma unroll
                                    for (int k = 0; k < 4; k++) s[pp][nt][k] -= base[k & 1];
                            }
                            top_products(x);
                        }
                        bool far = false;
#pragma unroll
                        for (int nt = 0; nt < NT; nt++)
#pragma unroll
                            for (int h = 0; h < 2; h++) {
#pragma unroll
                                for (int o = 4; o < 32; o <<= 1)
                                    x[nt][h] = fmaxf(x[nt][h], __shfl_xor_sync(0xffffffffu, x[nt][h], o));
                                far |= x[nt][h] - low[nt][h] > kMargin + kPShift && fabsf(x[nt][h]) >= 0x1p23f;
                            }
                        if (!__any_sync(0xffffffffu, far)) break;
#pragma unroll
                        for (int nt = 0; nt < NT; nt++)
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                const bool it = x[nt][h] - low[nt][h] > kMargin + kPShift && fabsf(x[nt][h]) >= 0x1p23f;
                                const float base = it ? x[nt][h] : 0.f;
                                low[nt][h] -= base;
                                if (g8 == 0) {
                                    sm.row_off[team][nt * 8 + 2 * c4 + h] = base;
                                    sm.row_base[team][nt * 8 + 2 * c4 + h] += base;
                                }
                            }
                        small = kAlways;
                        off = smem_u32(&sm.row_off[team][2 * c4]);
                        __syncwarp();
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            // a row moves by its own scores alone
                            const float y = x[nt][h] - low[nt][h] > kMargin + kPShift ? x[nt][h] - kPShift : low[nt][h];
                            const float d = low[nt][h] - y, f = ex2_approx(d);
                            low[nt][h] = y;
                            sum[nt][h] = sum_at<true>(sum[nt][h], f, d);
#pragma unroll
                            for (int j = 0; j < 8; j++) {
                                o[nt][j][h] *= f;
                                o[nt][j][2 + h] *= f;
                            }
                        }
                    // a weight below 2^-126 becomes 0 further down; with a small value scale its part of the sum still counts
                    if (least < kSmallExp) {
#pragma unroll
                        for (int pp = 0; pp < PP; pp++)
#pragma unroll
                            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                                for (int k = 0; k < 4; k++) {
                                    const float w = s[pp][nt][k] - (low[nt][k & 1] - (float)ev[pp]);
                                    if (w < -126.f) sum[nt][k & 1] += ex2_approx(w - (float)ev[pp]);
                                }
                    }
                }
                uint32_t pb[PP][NT][2];     // P^T fragments: tokens 4 c .. 4 c + 3, row g
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
#pragma unroll
                    for (int pp = 0; pp < PP; pp++) {
                        const float down = __int_as_float((127 - ev[pp]) << 23);
                        float p[4];
#pragma unroll
                        for (int k = 0; k < 4; k++) p[k] = ex2_approx(s[pp][nt][k] - (low[nt][k & 1] - (float)ev[pp]));
#pragma unroll
                        for (int h = 0; h < 2; h++) sum[nt][h] = fmaf(p[h] + p[2 + h], down, sum[nt][h]);
                        pb[pp][nt][0] = movmatrix_t(f16x2(p[0], p[1]));
                        pb[pp][nt][1] = movmatrix_t(f16x2(p[2], p[3]));
                    }
                }
                // output
#pragma unroll
                for (int pp = 0; pp < PP; pp++) {
                    const uint32_t page = unit + pp * kBCopyBytes + kBKBytes;
#pragma unroll
                    for (int i4 = 0; i4 < 4; i4++) {
                        const uint4 t = lds16(page + i4 * 512 + lane * 16);
                        uint32_t v[4] = {t.x, t.y, t.z, t.w};
                        if (tail) {
                            const int first = tok0 + pp * kPage + 4 * c4;
#pragma unroll
                            for (int k = 0; k < 4; k++)
                                v[k] = clean_values(v[k], len - first, full - first, first, &sm.bad[team][16 * g8 + 4 * i4 + k]);
                        }
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            // elements 16 g + 4 i4 + 2 k (matrix row g) and the next (row g + 8)
                            uint32_t a0, a1, a2, a3;
                            unpack4(v[2 * k], a0, a2);
                            unpack4(v[2 * k + 1], a1, a3);
#pragma unroll
                            for (int nt = 0; nt < NT; nt++)
                                mma_f16(o[nt][2 * i4 + k], a0, a1, a2, a3, pb[pp][nt][0], pb[pp][nt][1]);
                        }
                    }
                }
                met |= tail;
                __syncwarp();       // the stage is free once the warp has read it
                issue(stage);
                if (++stage == STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            left -= n + (u0 ? 0 : EXTRA);

            if (met && a.n_query > 1) {
                // the queries that see a token whose NaN was taken out get it here
#pragma unroll
                for (int j = 0; j < 8; j++)
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        const int first = sm.bad[team][16 * g8 + 2 * j + k];
                        if (first == 0x7fffffff) continue;
#pragma unroll
                        for (int nt = 0; nt < NT; nt++)
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                const int r = nt * 8 + 2 * c4 + h;
                                if (r < a.rows && len - (a.n_query - 1) + r / a.G > first) o[nt][j][2 * k + h] = CUDART_NAN_F;
                            }
                    }
            }

            // the piece's sums over its tokens
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) sum[nt][h] += __shfl_xor_sync(0xffffffffu, sum[nt][h], off);
                    if (small == kAlways) low[nt][h] += sm.row_base[team][nt * 8 + 2 * c4 + h];
                }
            const bool ends = u0 + n + EXTRA == n_units, whole = u0 == 0 && ends;
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
                        const float inv = l == 0.f ? 0.f : 1.f / l;
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
            n = min(left, n_units) - EXTRA;
        }
    }
    merge_pieces<TEAMS, TEAMS, true>(a, sm, park);
}

struct Variant {
    void (*kernel)(QuantAttnArgs);
    int teams, padrows, blocks_per_sm;
    size_t smem;
};

template <int NT, int PP, int TEAMS, int STAGES, int MINB, bool QREG>
Variant variant()
{
    return {block_attention_kernel<NT, PP, TEAMS, STAGES, MINB, QREG>, TEAMS, NT * 8, MINB,
            (size_t)TEAMS * block_team_bytes(NT, PP, STAGES, QREG)};
}

// As many warps as the registers of an output tile of 8 NT rows, and the rings, leave room for.
Variant variant_for(int rows)
{
    // N tiles as the rows need: a tile more costs (8 x 65536, 8 heads) 4 rows 178 -> 185 us, 16 rows 194 -> 202, 24 rows
    // 202 -> 249.  8 warps, two to a scheduler, where 12 would fit as well: 4 rows 178 -> 169, 16 rows 194 -> 179, 1 x
    // 4096 16.5 -> 14.5 (figures of the time); 6 warps 184 and 222, 16 of one-page units 182 and 316.  Two pages to a unit: one page 189 and 208
    // (32 rows: 254 -> 296), four 184 and 198; a third stage 184 and 179.  Q in registers where they suffice.
    if (rows <= 8) return variant<1, 2, 8, 2, 1, true>();
    if (rows <= 16) return variant<2, 2, 8, 2, 1, true>();
    if (rows <= 24) return variant<3, 2, 8, 2, 1, false>();
    return variant<4, 2, 8, 2, 1, false>();
}

int grid_of(const Variant &v, int sm_count) { return quant_grid(sm_count, v.blocks_per_sm, v.teams, v.padrows); }

}  // namespace

cudaError_t block_attention_config(int sm_count)
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

cudaError_t launch_block_attention(const QuantAttnArgs &a, int sm_count, cudaStream_t s)
{
    const Variant v = variant_for(a.rows);
    const int grid = grid_of(v, sm_count);
    const cudaError_t e = launch_maybe_pdl(v.kernel, dim3(grid), dim3(v.teams * 32), v.smem, s, true, a);
    if (e != cudaSuccess) return e;
    return launch_quant_combine<true>(a, grid, v.padrows, sm_count, s);
}

}  // namespace macgpu
