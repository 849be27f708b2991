// Causal attention of whole prompts, packed behind one another, on the
// 5th-generation tensor cores.
//
// Sequence b has n query tokens (rows starts[b] .. starts[b + 1] of q) and m
// keys (k_starts[b] .. of k and v); query i sees the first
//   seen(i) = clip(m - n + i + 1 - lag, 0, m)
// of them: out_i = sum_{j < seen} p_j v_j / sum_{j < seen} p_j,
// p_j = exp(scale q_i . k_j), lse_i = log sum p_j; out 0 and lse -inf where
// nothing is seen.
//
// Rows.  The G query heads of a KV head times 128 / G consecutive tokens are the
// 128 rows of a tile (row r: token r / G, head r % G), so any group fills the M of
// the products and a tile's causal edge is 128 / G tokens wide.  An item is two
// tiles, A and B, of consecutive tokens and one KV head; its keys come in blocks
// of 128, and both tiles use a block while it is in shared memory.
//
// Per block and tile: S = Q K^T (8 tcgen05.mma of 128 x 128 x 16, operands in
// shared memory, S in tensor memory), softmax by one thread per row, P in bf16
// back into tensor memory over S, O += P V (8 more, P read from tensor memory).
// The tensor pipe needs 512 cycles for each of the two products, and while it
// works for one tile the other tile's four warps do their softmax.
// Roundings: scores, references, sums and O in fp32; P to bf16 (2^-8 of each
// weight, as the bf16 output's own rounding; the sums take P unrounded).  Where
// the output is fp32, P is a bf16 pair hi + lo (2^-16) and O += P_hi V + P_lo V.
//
// Work split.  Items are numbered sequence by sequence, tile by tile from the
// last (longest) on, head by head.  With R + 1 or more items per CTA, a CTA takes
// R whole items, one from each row of `grid` items (back and forth, so that lengths
// even out), and what is left, one to two rows, is one line of blocks that is cut
// so that all CTAs end together; an item that is cut is merged by a second kernel.
// Everything follows from the lengths on the device, in each CTA's prologue: a
// captured call serves other lengths, and a call repeats bit for bit.
//
// Warps 0-3 softmax of tile A, 4-7 of tile B; warp 8 issues the products; warp 9
// loads keys and values by TMA into a ring of four blocks; warp 10 loads Q and
// looks through the value blocks on the causal edge (or a sequence's end): a NaN
// or an infinity there would reach rows that do not see it, as 0 * NaN, so it is
// taken out of the block and put back into the rows that do see it at the end.
// Every wait on an mbarrier has an iteration limit; on expiry the kernel sets
// kPErrTimeout, lets its copies and products land, frees its tensor memory and
// returns.  Completion k of a barrier is awaited with parity k & 1; every role
// waits each completion in order, and none can be two ahead of a waiter: a stage,
// a tile's Q, S, P and O are filled again only after their reader has passed on.
#include "mac_device.cuh"
#include "mac_prompt.cuh"

#include <climits>
#include <cudaTypedefs.h>

namespace macgpu {

namespace {

constexpr int kTok = 128;                           // keys per block
constexpr int kBlockBytes = 2 * kTok * 128;         // two column halves of 128 rows x 128 bytes
constexpr int kStages = 4;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kCheckWarp = 10;
constexpr int kThreads = 12 * 32;                   // three warpgroups; warp 11 has no role
// registers: 168 per thread at launch (three warpgroups: 504), then 208 for the
// softmax's two and 88 for the others'
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kTmemCols = 512;                      // S of A, B at 0, 128; O at 256, 384
constexpr int kDynBytes = 1024 + (2 + kStages) * kBlockBytes;
constexpr uint32_t kSpin = 1u << 22;
constexpr float kMargin = 8.f;                      // log2: how far a score may pass its row's reference
constexpr float kLowest = -3e38f;                   // the reference before the first key: finite, so that masked scores weigh 0

// kind::f16: D f32, A and B bf16; N >> 3 at bit 17, M >> 4 at bit 24; bit 16: B MN-major
constexpr uint32_t kIdescS = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescO = kIdescS | (1u << 16);

// Shared-memory matrix descriptors, 128-byte swizzle, rows of 8 every 1024
// bytes: the high word is the same for all, the low word holds the address and
// the leading offset, both / 16, so that a step through a tile is one addition.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) { return addr >> 4 | (lbo >> 4) << 16; }

// D (tensor memory) = or += A B; A in shared memory (ss) or in tensor memory (ts).
template <bool kAdd>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc)
{
    asm volatile("{\n.reg .pred p;\n.reg .b64 x, y;\nsetp.ne.b32 p, %4, 0;\nmov.b64 x, {%1, %5};\nmov.b64 y, {%2, %5};\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n"
                 :: "r"(d), "r"(a), "r"(b), "r"(idesc), "n"(kAdd ? 1 : 0), "n"(kDescHigh)
                 : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add)
{
    asm volatile("{\n.reg .pred p;\n.reg .b64 y;\nsetp.ne.b32 p, %4, 0;\nmov.b64 y, {%2, %5};\n"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n"
                 :: "r"(d), "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kDescHigh)
                 : "memory");
}

__device__ __forceinline__ void commit(uint32_t mbar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" :: "r"(mbar) : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }

__device__ __forceinline__ void mbar_init(uint32_t mbar, int count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" :: "r"(mbar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t mbar)
{
    asm volatile("{\n.reg .b64 st;\nmbarrier.arrive.shared::cta.b64 st, [%0];\n}\n" :: "r"(mbar) : "memory");
}

__device__ __forceinline__ void mbar_expect(uint32_t mbar, uint32_t bytes)
{
    asm volatile("{\n.reg .b64 st;\nmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n}\n" :: "r"(mbar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t mbar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(mbar)
                 : "memory");
}

// Bounded wait for a phase; gives up once another role has failed.  The lanes
// of a warp run it in step on the same word and the same flag and leave it with
// one outcome.
__device__ __forceinline__ bool wait_or_fail(uint32_t mbar, uint32_t parity, volatile int *fail)
{
    for (uint32_t i = 0; i < kSpin; i++) {
        uint32_t ok;
        asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                     : "=r"(ok)
                     : "r"(mbar), "r"(parity)
                     : "memory");
        if (ok) return true;
        if ((i & 255) == 255 && *fail) return false;
    }
    *fail = 1;
    return false;
}

// Bounded wait for copies and products in flight when the CTA winds down.
__device__ __forceinline__ void wait_bounded(uint32_t mbar, uint32_t parity)
{
    for (uint32_t i = 0; i < kSpin; i++) {
        uint32_t ok;
        asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                     : "=r"(ok)
                     : "r"(mbar), "r"(parity)
                     : "memory");
        if (ok) return;
    }
}

// 32 consecutive columns of the thread's tensor-memory lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float *v)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
                 "%29,%30,%31}, [%32];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
                   "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
                   "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, float *v)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n"
                 :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                    "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) { return bf16x2_bits(__floats2bfloat162_rn(lo, hi)); }

// ---- the work split -----------------------------------------------------------

// A sequence's query tokens, keys, and the keys that query 0 sees less one
// (before clipping).
struct Seq {
    int q0, n, k0, m;
    __device__ __forceinline__ int seen(const PromptArgs &a, int i) const
    {
        const long long s = (long long)m - n - a.lag + i + 1;
        return s <= 0 ? 0 : s < m ? (int)s : m;
    }
};

__device__ __forceinline__ Seq sequence(const PromptArgs &a, int b, bool report)
{
    const int q0 = a.starts[b], q1 = a.starts[b + 1], k0 = a.k_starts[b], k1 = a.k_starts[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.n_q || k0 < 0 || k1 < k0 || k1 > a.n_kv) {
        if (report) atomicOr(a.err, kPErrStarts);
        return Seq{0, 0, 0, 0};
    }
    return Seq{q0, q1 - q0, k0, k1 - k0};
}

// One item, or the part of it that a CTA does: blocks j0 .. j1 - 1 of its keys.
// (Scalars and selections, no arrays: an index that varies would put it in memory.)
struct Piece {
    Seq s;
    int seq, head, tile;
    int tok0;                   // first query token of tile A; tile B's come behind its tile_tokens
    int rows_a, rows_b;         // valid rows
    int nblk_a, nblk_b;         // key blocks each tile sees
    int edge;                   // first block that not every row sees whole
    int j0, j1;
    int slot;                   // -1: the whole item, else the partial slot
    __device__ __forceinline__ int tok(const PromptArgs &a, int x) const { return tok0 + (x ? a.tile_tokens : 0); }
    __device__ __forceinline__ int rows(int x) const { return x ? rows_b : rows_a; }
    // tile x does blocks j0 .. last - 1
    __device__ __forceinline__ int last(int x) const { return min(j1, x ? nblk_b : nblk_a); }
    __device__ __forceinline__ bool uses(int x) const { return last(x) > j0; }
};

struct Split {
    int pre[kPMaxBatch + 1];    // items of the sequences before b
    int scan[kThreads / 32];
    int cost[2 * kPMaxCtas];    // prefix of the blocks of the items of the line
    int load[kPMaxCtas];        // blocks that the CTAs do in whole items
    int quota[kPMaxCtas + 1];   // where the CTAs' shares of the line begin
    int rounds, line_items;
};

// Item `i` of the call.
__device__ __forceinline__ Piece item_at(const PromptArgs &a, const Split &sp, int i)
{
    int lo = 0, hi = a.batch;           // the last b with pre[b] <= i
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sp.pre[mid] <= i) lo = mid;
        else hi = mid;
    }
    Piece p;
    p.seq = lo;
    p.s = sequence(a, lo, false);
    const int in = i - sp.pre[lo], tiles = (sp.pre[lo + 1] - sp.pre[lo]) / a.kv_heads;
    const int down = in / a.kv_heads, T = a.tile_tokens;
    p.head = in - down * a.kv_heads;
    p.tile = tiles - 1 - down;
    p.tok0 = 2 * p.tile * T;
    const int ta = min(T, p.s.n - p.tok0), tb = min(T, p.s.n - p.tok0 - T);     // the item exists: ta >= 1
    p.rows_a = ta * a.G;
    p.rows_b = max(tb, 0) * a.G;
    p.nblk_a = (p.s.seen(a, p.tok0 + ta - 1) + kTok - 1) / kTok;
    p.nblk_b = tb > 0 ? (p.s.seen(a, p.tok0 + T + tb - 1) + kTok - 1) / kTok : 0;
    p.edge = p.s.seen(a, p.tok0) / kTok;
    p.j0 = 0;
    p.j1 = max(p.nblk_a, p.nblk_b);
    p.slot = -1;
    return p;
}

// Work of an item in blocks; one that sees no key still has its output to write.
__device__ __forceinline__ int item_cost(const Piece &p) { return max(p.j1, 1); }

__device__ __forceinline__ int block_scan(Split &sp, int v, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sp.scan[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w++) {
        if (w < warp) before += sp.scan[w];
        all += sp.scan[w];
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

// The whole split, by all threads of the CTA.
__device__ __forceinline__ void make_split(const PromptArgs &a, Split &sp)
{
    const int tid = threadIdx.x, grid = gridDim.x;
    int items = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
        const int b = b0 + tid;
        int own = 0, all;
        if (b < a.batch) {
            const Seq s = sequence(a, b, blockIdx.x == 0);
            own = (s.n + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens) * a.kv_heads;
        }
        const int at = block_scan(sp, own, &all);
        if (b < a.batch) sp.pre[b] = items + at;
        items += all;
    }
    if (tid == 0) sp.pre[a.batch] = items;
    __syncthreads();
    const int rounds = max(items / grid - 1, 0), first = rounds * grid, line = items - first;
    // blocks of the whole items
    for (int c = tid; c < grid; c += kThreads) {
        int load = 0;
        for (int r = 0; r < rounds; r++)
            load = min(load + item_cost(item_at(a, sp, r * grid + (r & 1 ? grid - 1 - c : c))), 1 << 29);
        sp.load[c] = load;
    }
    // blocks of the line
    int total = 0;
    for (int i0 = 0; i0 < line; i0 += kThreads) {
        const int i = i0 + tid;
        int all;
        const int own = i < line ? item_cost(item_at(a, sp, first + i)) : 0;
        const int at = block_scan(sp, own, &all);
        if (i < line) sp.cost[i] = total + at;
        total += all;
    }
    __syncthreads();
    if (tid < 32) {
        // the level at which the CTAs' shares, level - load, add up to the line
        int top = 0;
        for (int c = tid; c < grid; c += 32) top = max(top, sp.load[c]);
        top = __reduce_max_sync(0xffffffffu, top);
        int lo = 0, hi = top + (total + grid - 1) / grid;       // hi is enough
        while (lo < hi) {
            const int mid = lo + (hi - lo) / 2;
            long long sum = 0;
            for (int c = tid; c < grid; c += 32) sum += max(mid - sp.load[c], 0);
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (sum >= total) hi = mid;
            else lo = mid + 1;
        }
        int at = 0;
        for (int c0 = 0; c0 < grid; c0 += 32) {
            const int c = c0 + tid, own = c < grid ? max(hi - sp.load[c], 0) : 0;
            int x = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (tid >= o) x += y;
            }
            if (c < grid) sp.quota[c] = min(at + x - own, total);
            at = min(at + __shfl_sync(0xffffffffu, x, 31), total);
        }
        if (tid == 0) {
            sp.quota[grid] = total;
            sp.rounds = rounds;
            sp.line_items = line;
        }
    }
    __syncthreads();
}

// A CTA's pieces, one after another: first its whole items, then its share of
// the line.
struct Walk {
    int round, item, at, end;
    __device__ __forceinline__ Walk(const Split &sp)
    {
        round = 0;
        at = sp.quota[blockIdx.x];
        end = sp.quota[blockIdx.x + 1];
        int lo = 0, hi = sp.line_items;         // the line's item that holds block `at`
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sp.cost[mid] <= at) lo = mid;
            else hi = mid;
        }
        item = lo;
    }
    __device__ __forceinline__ bool next(const PromptArgs &a, const Split &sp, Piece &p)
    {
        const int grid = gridDim.x;
        if (round < sp.rounds) {
            p = item_at(a, sp, round * grid + (round & 1 ? grid - 1 - blockIdx.x : blockIdx.x));
            round++;
            return true;
        }
        if (at >= end) return false;
        p = item_at(a, sp, sp.rounds * grid + item);
        const int start = sp.cost[item], stop = start + item_cost(p);
        const bool begins = start >= at, ends = stop <= end;
        if (!begins || !ends) {
            p.slot = begins ? 1 : 0;
            p.j0 = at - start;
            p.j1 = min(p.j1, end - start);
        }
        at = min(stop, end);
        item++;
        return true;
    }
};

template <int N>
__device__ __forceinline__ void more_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" :: "n"(N));
}

template <int N>
__device__ __forceinline__ void fewer_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" :: "n"(N));
}

// ---- the attention --------------------------------------------------------------

// O of the row times f, in tensor memory.
__device__ __forceinline__ void rescale(uint32_t tO, float f)
{
#pragma unroll
    for (int c = 0; c < 8; c++) {
        float o[16];
        tmem_ld16(tO + 16 * c, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; i++) o[i] *= f;
        tmem_st16(tO + 16 * c, reinterpret_cast<const uint32_t *>(o));
    }
}

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// two fp32 operations in one instruction
__device__ __forceinline__ void fma2(float &x, float &y, float scale, float add)
{
    asm("{\n.reg .b64 a, b, c;\nmov.b64 a, {%0, %1};\nmov.b64 b, {%2, %2};\nmov.b64 c, {%3, %3};\n"
        "fma.rn.f32x2 a, a, b, c;\nmov.b64 {%0, %1}, a;\n}\n"
        : "+f"(x), "+f"(y)
        : "f"(scale), "f"(add));
}

__device__ __forceinline__ void add2(float &x, float &y, float a, float b)
{
    asm("{\n.reg .b64 a, b;\nmov.b64 a, {%0, %1};\nmov.b64 b, {%2, %3};\nadd.rn.f32x2 a, a, b;\nmov.b64 {%0, %1}, a;\n}\n"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}

// The scores of a chunk of 32 keys whose first `live` the row sees.
__device__ __forceinline__ void hide(float *s, int live)
{
#pragma unroll
    for (int i = 0; i < 32; i++)
        if (i >= live) s[i] = -CUDART_INF_F;
}

__device__ __forceinline__ float chunk_max(const float *s, float top)
{
    float m[4] = {fmaxf(top, s[0]), s[1], s[2], s[3]};
#pragma unroll
    for (int i = 4; i < 28; i += 8)
#pragma unroll
        for (int k = 0; k < 4; k++) m[k] = max3(m[k], s[i + k], s[i + k + 4]);
#pragma unroll
    for (int k = 0; k < 4; k++) m[k] = fmaxf(m[k], s[28 + k]);
    return fmaxf(max3(m[0], m[1], m[2]), m[3]);
}

// One block of one row: its scores in tensor memory become weights, in bf16, or
// (kWide) as bf16 pairs hi + lo, which take the place of all 128 scores.
template <bool kWide>
__device__ __forceinline__ void softmax_block(uint32_t tS, uint32_t tO, float sc, int live, bool edge, bool later, float &ref,
                                              float &sum)
{
    float s[128], top = -CUDART_INF_F, part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; c++) tmem_ld32(tS + 32 * c, s + 32 * c);
    tmem_wait_ld();
    if (edge) {
#pragma unroll
        for (int c = 0; c < 4; c++) hide(s + 32 * c, live - 32 * c);
    }
#pragma unroll
    for (int c = 0; c < 4; c++) top = chunk_max(s + 32 * c, top);
    top *= sc;
    if (__any_sync(0xffffffffu, top - ref > kMargin)) {
        const float now = top - ref > kMargin ? top : ref, f = ex2_approx(ref - now);
        ref = now;
        sum *= f;
        // the product of the block before is complete: these scores were issued behind it
        if (later) rescale(tO, f);
    }
    // 2^(s sc - ref), the exponent fused; that is off by the reference's rounding, which could pass any weight's range
    // for references beyond 2^28: those rows take the product first
    const bool far = fabsf(ref) >= 0x1p28f;
    if (__any_sync(0xffffffffu, far)) {
#pragma unroll
        for (int i = 0; i < 128; i++) s[i] = far ? __fmul_rn(s[i], sc) : s[i];
        if (far) sc = 1.f;
    }
#pragma unroll
    for (int c = 0; c < 4; c++) {
        float *v = s + 32 * c;
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) fma2(v[i], v[i + 1], sc, -ref);
#pragma unroll
        for (int i = 0; i < 32; i++) v[i] = ex2_approx(v[i]);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            add2(part[0], part[1], v[i], v[i + 1]);
            add2(part[2], part[3], v[i + 2], v[i + 3]);
        }
#pragma unroll
        for (int i = 0; i < 16; i++) w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
        tmem_st16(tS + 16 * c, w);
        if (kWide) {
#pragma unroll
            for (int i = 0; i < 16; i++)
                w[i] = bf16_pair(v[2 * i] - __uint_as_float(w[i] << 16), v[2 * i + 1] - __uint_as_float(w[i] & 0xffff0000u));
            tmem_st16(tS + 64 + 16 * c, w);
        }
    }
    sum += (part[0] + part[1]) + (part[2] + part[3]);
}

struct Bars {
    unsigned long long full[kStages], empty[kStages];   // ring of key and value blocks
    unsigned long long q_full[2], q_empty[2];           // Q of a tile
    unsigned long long s_full[2], p_full[2], o_full[2]; // scores made, weights written, output complete
    unsigned long long v_ok[2], done;                   // values of an odd stage looked through
};

template <bool kWide>
__global__ void __launch_bounds__(kThreads, 1) prompt_attention_kernel(const __grid_constant__ PromptArgs a,
                                                                      const __grid_constant__ PromptMaps maps)
{
    extern __shared__ __align__(1024) uint8_t dyn_raw[];
    __shared__ Split sp;
    __shared__ __align__(8) Bars bars;
    __shared__ int s_bad[2][kD], s_dirty[2];            // first token whose value is not finite, by element; two items in turn
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail, s_written[8];                // pieces that each softmax warp is done with
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    volatile int *fail = &s_fail;
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(dyn_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sQ = smem_u32(base), sKV = sQ + 2 * kBlockBytes;
    auto B_ = [](unsigned long long &b) { return smem_u32(&b); };

    pdl_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < kStages; i++) {
            mbar_init(B_(bars.full[i]), 1);
            mbar_init(B_(bars.empty[i]), i & 1 ? 2 : 1);        // value blocks stand in odd stages: warp 10 reads them too
        }
        for (int x = 0; x < 2; x++) {
            mbar_init(B_(bars.q_full[x]), 1);
            mbar_init(B_(bars.q_empty[x]), 1);
            mbar_init(B_(bars.s_full[x]), 1);
            mbar_init(B_(bars.p_full[x]), 128);
            mbar_init(B_(bars.o_full[x]), 1);
            mbar_init(B_(bars.v_ok[x]), 1);
        }
        mbar_init(B_(bars.done), 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        s_fail = 0;
    }
    if (tid < 2 * kD) s_bad[tid / kD][tid % kD] = INT_MAX;
    if (tid < 2) s_dirty[tid] = 0;
    if (tid < 8) s_written[tid] = 0;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n"
                     :: "r"(smem_u32(&s_tmem)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = s_tmem;
    pdl_wait();
    make_split(a, sp);

    Piece p;
    Walk walk(sp);
    if (warp < 8) {
        more_registers<kSoftmaxRegs>();
        // softmax and output: a thread per row of its tile
        const int x = warp >> 2, row = tid & 127;
        const int row_tok = row / a.G, row_head = row - row_tok * a.G;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + 128 * x + lanes, tO = tmem + 256 + 128 * x + lanes;
        const float sc = a.scale_log2;
        uint32_t ns = 0, no = 0;
        bool ok = true;
        // a CTA without a share of the line has no part in the items that span it
        if (sp.quota[blockIdx.x] == sp.quota[blockIdx.x + 1])
            a.part_ml[(int64_t)blockIdx.x * 2 * kPRows + tid] = make_float2(0.f, 0.f);
        for (int k = 0; ok && walk.next(a, sp, p); k++) {
            const bool valid = row < p.rows(x);
            const int lim = valid ? p.s.seen(a, p.tok(a, x) + row_tok) : 0;       // keys the row sees
            float ref = kLowest, sum = 0.f;
            const int last = p.last(x);
            for (int j = p.j0; j < last; j++) {
                if (!wait_or_fail(B_(bars.s_full[x]), ns & 1, fail)) {
                    ok = false;
                    break;
                }
                ns++;
                fence_after();
                const int live = lim - j * kTok;        // of the block's keys, those that the row sees
                softmax_block<kWide>(tS, tO, sc, live, j >= p.edge, j > p.j0, ref, sum);
                tmem_wait_st();
                fence_before();
                mbar_arrive(B_(bars.p_full[x]));
            }
            if (!ok) break;

            // the row's output, or its part of one
            const bool some = last > p.j0;
            if (some) {
                if (!wait_or_fail(B_(bars.o_full[x]), no & 1, fail)) break;
                no++;
                fence_after();
            }
            const bool dirty = some && *(volatile int *)&s_dirty[k & 1];
            const bool part = p.slot >= 0;
            const float inv = part ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
            const int64_t at = (int64_t)(p.s.q0 + p.tok(a, x) + row_tok) * a.heads + p.head * a.G + row_head;
            const int64_t prow = ((int64_t)blockIdx.x * 2 + p.slot) * kPRows + 128 * x + row;
#pragma unroll
            for (int c = 0; c < 4; c++) {
                float o[32];
                __syncwarp();
                if (some) {
                    tmem_ld32(tO + 32 * c, o);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int i = 0; i < 32; i++) {
                    o[i] = some && sum != 0.f ? o[i] * inv : 0.f;
                    if (dirty && s_bad[k & 1][32 * c + i] < lim) o[i] = CUDART_NAN_F;
                }
                if (!valid) continue;
                if (part || kWide) {
                    float *dst = part ? a.part_o + prow * kD + 32 * c : reinterpret_cast<float *>(a.out) + at * kD + 32 * c;
#pragma unroll
                    for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4 *>(dst + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                } else {
                    __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(a.out) + at * kD + 32 * c;
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        *reinterpret_cast<uint4 *>(dst + i) = make_uint4(bf16_pair(o[i], o[i + 1]), bf16_pair(o[i + 2], o[i + 3]),
                                                                         bf16_pair(o[i + 4], o[i + 5]), bf16_pair(o[i + 6], o[i + 7]));
                }
            }
            if (valid) {
                if (part) a.part_ml[prow] = make_float2(ref, sum);
                else if (a.lse) a.lse[at] = sum == 0.f ? -CUDART_INF_F : (ref + log2f(sum)) * kLn2;
            }
            fence_before();
            __syncwarp();
            if (lane == 0) *(volatile int *)&s_written[warp] = k + 1;
        }
    } else {
        fewer_registers<kOtherRegs>();
        if (warp == kLoadWarp) {
            if (lane == 0) {
                uint32_t n = 0;             // blocks issued: use n of the ring is in stage n % kStages
                bool ok = true;
                while (ok && walk.next(a, sp, p)) {
                    for (int j = p.j0; j < p.j1 && ok; j++)
                        for (int kv = 0; kv < 2; kv++, n++) {
                            const uint32_t st = n % kStages, turn = n / kStages;
                            if (turn && !wait_or_fail(B_(bars.empty[st]), (turn - 1) & 1, fail)) {
                                ok = false;
                                break;
                            }
                            const uint32_t full = B_(bars.full[st]), dst = sKV + st * kBlockBytes;
                            const CUtensorMap *map = kv ? &maps.v : &maps.k;
                            mbar_expect(full, kBlockBytes);
                            for (int h = 0; h < 2; h++)
                                tma_load(dst + h * (kBlockBytes / 2), map, 64 * h, p.head, p.s.k0 + j * kTok, full);
                        }
                }
                // before the CTA exits, the copies that it issued have landed
                for (uint32_t s = 0; s < kStages; s++) {
                    const uint32_t uses = (n + kStages - 1 - s) / kStages;
                    if (uses) wait_bounded(B_(bars.full[s]), (uses - 1) & 1);
                }
            }
        } else if (warp == kMmaWarp) {
            // The whole warp walks and waits, so that addresses stay uniform, and one lane issues.  A wait that gives up is
            // noted and the walk goes on: every later wait then gives up soon, and nothing is read out of bounds.
            uint32_t n = 0;             // ring uses of the pieces before
            uint32_t nq[2] = {0, 0}, np[2] = {0, 0};
            const uint32_t q_low = desc_low(sQ, 16), key_low = desc_low(sKV, 16), value_low = desc_low(sKV, kBlockBytes / 2);
            auto wait = [&](unsigned long long &bar, uint32_t k) { wait_or_fail(B_(bar), k & 1, fail); };
            auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
            // scores of tile x against the key block in stage st
            auto score = [&](int x, uint32_t st, bool final) {
                const uint32_t d = tmem + 128 * x, q = q_low + x * (kBlockBytes >> 4), b = key_low + st * (kBlockBytes >> 4);
                fence_after();
                if (lane == 0) {
                    mma_ss<false>(d, q, b, kIdescS);
#pragma unroll
                    for (int k = 1; k < 8; k++) {
                        const uint32_t off = ((k >> 2) * (kBlockBytes / 2) + (k & 3) * 32) >> 4;
                        mma_ss<true>(d, q + off, b + off, kIdescS);
                    }
                    commit(B_(bars.s_full[x]));
                    if (final) commit(B_(bars.q_empty[x]));
                }
            };
            // weights of tile x times the value block in stage st
            auto output = [&](int x, uint32_t st, bool first, bool final) {
                const uint32_t d = tmem + 256 + 128 * x, w = tmem + 128 * x, b = value_low + st * (kBlockBytes >> 4);
                fence_after();
                if (lane == 0) {
                    mma_ts(d, w, b, kIdescO, !first);
#pragma unroll
                    for (int k = 1; k < 8; k++) mma_ts(d, w + 8 * k, b + k * (2048 >> 4), kIdescO, 1);
                    if (kWide) {
#pragma unroll
                        for (int k = 0; k < 8; k++) mma_ts(d, w + 64 + 8 * k, b + k * (2048 >> 4), kIdescO, 1);
                    }
                    if (final) commit(B_(bars.o_full[x]));
                }
            };
            auto release = [&](uint32_t use) {
                if (lane == 0) commit(B_(bars.empty[use % kStages]));
            };
            while (walk.next(a, sp, p)) {
                const int j0 = same(p.j0), j1 = same(p.j1), edge = same(p.edge), last[2] = {same(p.last(0)), same(p.last(1))};
                if (j1 > j0) {
                    wait(bars.full[n % kStages], n / kStages);
#pragma unroll
                    for (int x = 0; x < 2; x++)
                        if (last[x] > j0) {
                            wait(bars.q_full[x], nq[x]++);
                            score(x, n % kStages, j0 + 1 == last[x]);
                        }
                    release(n);
                }
                for (int j = j0; j < j1; j++, n += 2) {
                    // uses of the ring: n keys of j, n + 1 values of j, n + 2 keys of j + 1
                    const uint32_t vst = (n + 1) % kStages, kst = (n + 2) % kStages;
                    bool next_keys = j + 1 == j1;
                    wait(bars.full[vst], (n + 1) / kStages);
                    if (j >= edge) wait(bars.v_ok[vst >> 1], (n + 1) / kStages);
#pragma unroll
                    for (int x = 0; x < 2; x++) {
                        if (j < last[x]) {
                            wait(bars.p_full[x], np[x]++);
                            output(x, vst, j == j0, j + 1 == last[x]);
                        }
                        if (x == 1) release(n + 1);
                        if (j + 1 < last[x]) {
                            if (!next_keys) wait(bars.full[kst], (n + 2) / kStages);
                            next_keys = true;
                            score(x, kst, j + 2 == last[x]);
                        }
                    }
                    if (j + 1 < j1) release(n + 2);
                }
            }
            // every product issued is complete before the CTA frees its tensor memory
            if (lane == 0) {
                commit(B_(bars.done));
                wait_bounded(B_(bars.done), 0);
            }
            __syncwarp();
        } else if (warp == kCheckWarp) {
            uint32_t n = 0, nq[2] = {0, 0}, q_bytes = (uint32_t)a.tile_tokens * a.G * 256;
            bool ok = true;
            for (int k = 0; ok && walk.next(a, sp, p); k++) {
                // marks of the item two before this one: taken back once that item is written
                if (*(volatile int *)&s_dirty[k & 1]) {
                    for (uint32_t i = 0; ok && !__all_sync(0xffffffffu, *(volatile int *)&s_written[lane & 7] >= k - 1); i++)
                        if (i > kSpin || *fail) {
                            *fail = 1;
                            ok = false;
                        }
                    ok = __all_sync(0xffffffffu, ok);
                    for (int d = lane; d < kD; d += 32) s_bad[k & 1][d] = INT_MAX;
                    __syncwarp();
                    if (lane == 0) s_dirty[k & 1] = 0;
                    __threadfence_block();
                    __syncwarp();
                }
                for (int x = 0; x < 2 && ok; x++)
                    if (p.uses(x)) {
                        if (nq[x] && !wait_or_fail(B_(bars.q_empty[x]), (nq[x] - 1) & 1, fail)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) {
                            mbar_expect(B_(bars.q_full[x]), q_bytes);
                            for (int h = 0; h < 2; h++)
                                tma_load(sQ + x * kBlockBytes + h * (kBlockBytes / 2), &maps.q, 64 * h, p.head * a.G,
                                         p.s.q0 + p.tok(a, x), B_(bars.q_full[x]));
                        }
                        nq[x]++;
                    }
                for (int j = p.j0; j < p.j1 && ok; j++) {
                    const uint32_t use = n + 2 * (j - p.j0) + 1, st = use % kStages;
                    if (!wait_or_fail(B_(bars.full[st]), use / kStages & 1, fail)) {
                        ok = false;
                        break;
                    }
                    if (j >= p.edge) {
                        uint8_t *v = base + (2 + st) * kBlockBytes;
                        // 0 * x is 0 but for a NaN or an infinity
                        const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
                        __nv_bfloat162 acc[4] = {zero, zero, zero, zero};
#pragma unroll 8
                        for (int i = lane; i < kBlockBytes / 16; i += 32) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(v + i * 16);
                            acc[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&w.x), zero, acc[0]);
                            acc[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&w.y), zero, acc[1]);
                            acc[2] = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&w.z), zero, acc[2]);
                            acc[3] = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&w.w), zero, acc[3]);
                        }
                        uint32_t any = 0;
#pragma unroll
                        for (int i = 0; i < 4; i++) any |= bf16x2_bits(acc[i]) & 0x7fff7fffu;
                        if (__any_sync(0xffffffffu, any != 0)) {
#pragma unroll 1
                            for (int i = lane; i < kBlockBytes / 2; i += 32) {
                                uint16_t *e = reinterpret_cast<uint16_t *>(v) + i;
                                if ((*e & 0x7f80) != 0x7f80) continue;
                                // element i of the swizzled tile: half, row (token), 16-byte chunk
                                const int half = i >> 13, row = i >> 6 & 127, chunk = (i >> 3 & 7) ^ (row & 7);
                                *e = 0;
                                atomicMin(&s_bad[k & 1][half * 64 + chunk * 8 + (i & 7)], j * kTok + row);
                            }
                            __syncwarp();
                            if (lane == 0) s_dirty[k & 1] = 1;
                            asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                            __threadfence_block();
                            __syncwarp();
                        }
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(B_(bars.v_ok[st >> 1]));
                        mbar_arrive(B_(bars.empty[st]));
                    }
                }
                n += 2 * (p.j1 - p.j0);
            }
            // before the CTA exits, the copies that it issued have landed
            if (lane == 0)
                for (int x = 0; x < 2; x++)
                    if (nq[x]) wait_bounded(B_(bars.q_full[x]), (nq[x] - 1) & 1);
        }
    }

    // the items of the line that begin in this CTA's share: which CTAs the second kernel finds them in
    if (warp == kLoadWarp) {
        const int lo = sp.quota[blockIdx.x], hi = sp.quota[blockIdx.x + 1], grid = gridDim.x;
        for (int i = lane; i < sp.line_items; i += 32) {
            const int start = sp.cost[i];
            if (start < lo || start >= hi) continue;
            const int stop = i + 1 < sp.line_items ? sp.cost[i + 1] : sp.quota[grid];
            PromptMeta m{-1, 0, 0, 0, 0, {0, 0, 0}};
            if (stop > hi) {
                const Piece q = item_at(a, sp, sp.rounds * grid + i);
                int c = blockIdx.x;
                while (sp.quota[c + 1] < stop) c++;
                m = PromptMeta{q.seq, q.head, q.tile, (int)blockIdx.x, c, {0, 0, 0}};
            }
            a.meta[i] = m;
        }
        if (blockIdx.x == 0)
            for (int i = sp.line_items + lane; i < 2 * grid; i += 32) a.meta[i] = PromptMeta{-1, 0, 0, 0, 0, {0, 0, 0}};
    }
    __syncthreads();
    if (*fail && tid == 0) atomicOr(a.err, kPErrTimeout);
    fence_before();
    __syncthreads();
    if (warp == 0) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" :: "r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// The items that several CTAs worked on: block (i, y) merges rows of item i of
// the line, a warp per row, a lane with four elements.
constexpr int kMergeWarps = 8, kMergeRows = 32;

template <bool kWide>
__global__ void __launch_bounds__(kMergeWarps * 32) prompt_merge_kernel(const __grid_constant__ PromptArgs a)
{
    pdl_wait();
    const PromptMeta meta = a.meta[blockIdx.x];
    if (meta.seq < 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, T = a.tile_tokens;
    const Seq s = sequence(a, meta.seq, false);
    for (int r = blockIdx.y * kMergeRows + warp; r < (int)(blockIdx.y + 1) * kMergeRows; r += kMergeWarps) {
        const int row = r & 127, tok = (2 * meta.tile + (r >> 7)) * T + row / a.G;
        if (row >= T * a.G || tok >= s.n) continue;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float m = -CUDART_INF_F, l = 0.f;
        for (int c = meta.first; c <= meta.last; c++) {
            const int64_t at = ((int64_t)c * 2 + (c == meta.first)) * kPRows + r;
            const float2 ml = a.part_ml[at];
            const float4 x = reinterpret_cast<const float4 *>(a.part_o + at * kD)[lane];
            if (ml.y == 0.f) continue;          // saw no key
            const float top = fmaxf(m, ml.x), f = ex2_approx(m - top), g = ex2_approx(ml.x - top);
            o = make_float4(o.x * f + x.x * g, o.y * f + x.y * g, o.z * f + x.z * g, o.w * f + x.w * g);
            l = l * f + ml.y * g;
            m = top;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
        const int64_t at = (int64_t)(s.q0 + tok) * a.heads + meta.head * a.G + row % a.G;
        if (kWide) {
            reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + at * kD)[lane] =
                make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        } else {
            reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + at * kD)[lane] =
                make_uint2(bf16_pair(o.x * inv, o.y * inv), bf16_pair(o.z * inv, o.w * inv));
        }
        if (lane == 0 && a.lse) a.lse[at] = l == 0.f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
    }
}

using EncodeTiled = PFN_cuTensorMapEncodeTiled_v12000;

}  // namespace

cudaError_t prompt_attention_config(int sm_count)
{
    if (sm_count > kPMaxCtas) return cudaErrorInvalidConfiguration;
    const cudaError_t e = cudaFuncSetAttribute(prompt_attention_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynBytes);
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(prompt_attention_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynBytes);
}

// Maps over [token][head][128] tensors: boxes of 64 elements (a 128-byte swizzle
// row) by the group's heads and a tile's tokens of q, by 128 keys of one head.
cudaError_t prompt_maps(const PromptArgs &a, const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                        int64_t v_stride, PromptMaps &maps)
{
    static const EncodeTiled encode = [] {      // the driver's tensor-map encoder, looked up once
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult r = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<EncodeTiled>(fn);
    }();
    if (!encode) return cudaErrorNotSupported;
    struct {
        CUtensorMap *map;
        const void *base;
        int64_t heads, tokens, stride;
        int box_heads, box_tokens;
    } each[3] = {{&maps.q, q, a.heads, a.n_q, q_stride, a.G, a.tile_tokens},
                 {&maps.k, k, a.kv_heads, a.n_kv, k_stride, 1, kTok},
                 {&maps.v, v, a.kv_heads, a.n_kv, v_stride, 1, kTok}};
    for (auto &t : each) {
        if (t.tokens == 0) {            // no keys at all: the map is not used
            t.base = q;
            t.tokens = 1;
        }
        const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)t.heads, (cuuint64_t)t.tokens};
        const cuuint64_t strides[2] = {(cuuint64_t)kD * 2, (cuuint64_t)t.stride * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)t.box_heads, (cuuint32_t)t.box_tokens};
        const cuuint32_t each_one[3] = {1, 1, 1};
        const CUresult r = encode(t.map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(t.base), dims, strides, box, each_one,
                                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) return cudaErrorInvalidValue;
    }
    return cudaSuccess;
}

cudaError_t launch_prompt_attention(const PromptArgs &a, const PromptMaps &maps, int sm_count, cudaStream_t s)
{
    // items at most: no sequence has more than a partly filled one per head besides
    const int64_t most = ((int64_t)a.n_q / (2 * a.tile_tokens) + a.batch) * a.kv_heads;
    const int64_t line = most < 2 * sm_count ? most : 2 * sm_count;
    const auto kernel = a.wide ? prompt_attention_kernel<true> : prompt_attention_kernel<false>;
    const cudaError_t e = launch_maybe_pdl(kernel, dim3(sm_count), dim3(kThreads), kDynBytes, s, true, a, maps);
    if (e != cudaSuccess) return e;
    const auto merge = a.wide ? prompt_merge_kernel<true> : prompt_merge_kernel<false>;
    return launch_maybe_pdl(merge, dim3((unsigned)line, kPRows / kMergeRows), dim3(kMergeWarps * 32), 0, s, true, a);
}

}  // namespace macgpu
