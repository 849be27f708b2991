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
// The tensor pipe needs 512 cycles for each of the two products (64 for each of
// the 8, whichever memory A comes from, and whatever the softmax does beside it:
// measured), and while it works for one tile the other tile's four warps do their
// softmax.  S, P and O of two tiles fill the 512 columns of tensor memory, and two
// tiles of Q and four blocks of keys and values 192 KB of shared memory.
// Roundings: scores, references, sums and O in fp32; P to bf16 (2^-8 of each
// weight, as the bf16 output's own rounding; the sums take P unrounded).  Where
// the output is fp32, P is a bf16 pair hi + lo (2^-17 of each weight) and O += P_hi
// V + P_lo V, in runs of eight blocks (kWideRun).
//
// Work split.  Items are numbered from those of the most key blocks down, over all
// sequences.  With R + 1 or more items per CTA, a CTA takes R whole items, one from
// each row of `grid` items (back and forth, so that lengths even out), and what is
// left, one to two rows, is one line of blocks that is cut so that all CTAs end
// together (an item counts kPExtra blocks besides its own); an item that is cut is
// merged by a second kernel (there is none where no sequence has more than a block of
// keys).  Numbered sequence by sequence, 24 ragged prompts took 452 us instead of 427,
// 5 with 28 / 4 heads 257 instead of 240: the whole items' loads differed by up to 13 %.
// Everything follows from the lengths on the device, in each CTA's prologue: a
// captured call serves other lengths, and a call repeats bit for bit.
//
// Warps 0-3 softmax and output of tile A, 4-7 of tile B; warp 8 issues the
// products; warp 11 finds the CTA's pieces (items, or parts of them), which takes
// longer than a block of keys, and announces them up to four ahead; warp 9 loads
// keys and values by TMA into a ring of four blocks; warp 10 loads Q and
// looks through the value blocks on the causal edge (or a sequence's end): a NaN
// or an infinity there would reach rows that do not see it, as 0 * NaN, so it is
// taken out of the block and put back into the rows that do see it at the end.
// Every wait on an mbarrier has an iteration limit; on expiry the kernel sets
// kPErrTimeout, lets its copies and products land, frees its tensor memory and
// returns.  Completion k of a barrier is awaited with parity k & 1; every role
// waits each completion in order, and none can be two ahead of a waiter: a stage,
// a tile's Q, S, P and O are filled again only after their reader has passed on.
//
// Measured (graph replays; 32 / 8 heads but where noted; 1965 TFLOP/s is the
// library's largest product's rate): 32768 tokens 4.95 ms with rests between calls,
// 5.3 to 5.5 on end (1775 and 1600 to 1650 TFLOP/s of the products that the causal
// edge leaves), 6001 tokens 212 us (1390), 2048 and 509 tokens behind 30720 and 8191
// 675 us (1680), 24 ragged prompts of 1 .. 4096 tokens 409 us (1330), 5 of 1 .. 6001
// with 28 / 4 heads 219 us (1365), 512 fp32 rows behind 32256 288 to 324 us (840 to
// 945; with the second P V 1260 to 1415), 16 tokens 8.6 us on end, 12.4 a replay by
// itself; 100 prompts of 1000 tokens 860 us (955), 256 of 64 tokens 94, 1024 of 16
// 276 (their bytes take 50).
// What bounds it.  A steady block takes 2450 to 2600 cycles of the pipe's 2048:
// from scores to weights a tile takes 1240 (880 of them the softmax itself: 512 of
// ex2 at 32 a cycle and SM, loads and stores of tensor memory, maximum and packing;
// the rest barriers), its products 1024 and 190 until they are seen, and the other
// tile fills 2048 of that.  In long calls the card then holds its power limit at
// 1.7 to 1.85 GHz, and fewer cycles give little.  A piece costs 7000 to 10000 cycles
// besides its blocks (first scores, first softmax, the output, code that was not
// near), which with the edge blocks' hidden halves is what ragged prompts lose; a
// prompt of at most 128 / G tokens is a piece per KV head with an empty tile B, and
// many of those run one after another.  The prologue (lengths, split, first loads)
// takes 8000 to 16000 a call.
// Tried and slower (32768 tokens, ms, against the form of the time): softmax
// warps of half a row each 5.79 / 5.45; a second warp to issue 7.05 / 6.0; P V
// issued for the first keys before the last weights are there 5.70 / 5.33; waits
// that spin 5.5 / 5.33; weights against the old reference, which the row's sum
// then confirms, instead of a maximum first: no faster, chunks 677 / 685 us; every
// eighth ex2 as a polynomial 5.43 / 5.28 (packed products run at
// half rate); outputs through shared memory, in whole lines, slower than 32 bytes a
// thread from the registers.  A third part of the weights for fp32 outputs, in the
// first one's place after its products: error 7e-7 instead of 2e-6 at 2048 keys, 512
// rows behind 32256 476 us instead of 298.  Only where a sequence has few keys: error
// 4e-7 to 1.2e-6 instead of 1.6e-6 to 2.2e-6 up to 2048 keys (fp32 products 2e-7 to
// 8e-7), 64 keys 7.6 -> 8.3 us, 256 18.6 -> 23, 2048 41 -> 61, and the choice alone
// took the rows behind 32256 keys from 287 to 353 us.
#include "mac_device.cuh"
#include "mac_prompt.cuh"

#include <climits>
#include <cudaTypedefs.h>

namespace macgpu {

namespace {

constexpr int kTok = 128;                           // keys per block
constexpr int kBlockBytes = 2 * kTok * 128;         // two column halves of 128 rows x 128 bytes
constexpr int kStages = 4;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kCheckWarp = 10;       // warp 11 announces the pieces
constexpr int kPieces = 4;                          // pieces announced ahead
constexpr int kThreads = 12 * 32;                   // three warpgroups
// registers: 168 per thread at launch (three warpgroups: 504), then 208 for the
// softmax's two and 88 for the others'
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kTmemCols = 512;                      // S of A, B at 0, 128; O at 256, 384
constexpr int kDynBytes = 1024 + (2 + kStages) * kBlockBytes;
constexpr uint32_t kSpin = 1u << 22;
// Blocks of a run, a power of two.  The tensor cores cut a sum off towards 0 where
// a product is added to it: 1.4e-8 of it on average, always the same way, so that it
// grows with the number of products (16 per block in the wide form, 8 in the other).
// So a sum of a run's products goes to memory, in fp32, and the next run starts anew.
// 512 fp32 rows behind 32256 keys, error and us with runs of 4, 8, 16 blocks and with
// one: 2.8e-6 326, 3.4e-6 298, 5.2e-6 283, 2.9e-5 256 (fp32 products 3.2e-6).  Beside
// outputs of 2^-9 512 blocks' 2^-14 are enough, which calls of at most 65536 keys do
// not reach: they take the form without runs (24 ragged prompts 455 -> 448 us).
constexpr int kWideRun = 8, kRun = 512;
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

// One lane of the warp, the same every time.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}

// Whether a phase is complete; does not wait.
__device__ __forceinline__ uint32_t phase_done(uint32_t mbar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(mbar), "r"(parity)
                 : "memory");
    return ok;
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

// A sequence: its first query row and number of queries, its first key row and
// number of keys.
struct Seq {
    int q0, n, k0, m;
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
    int seq, head, tile;        // seq < 0: no more pieces
    int row0;                   // row of q and out of tile A's first token; tile B's come behind its tile_tokens
    int key0, keys;             // the sequence's first key row, its keys
    int first_seen;             // keys that tile A's first token sees, before clipping to 0 .. keys; one more for each token behind
    int rows_a, rows_b;         // valid rows
    int nblk_a, nblk_b;         // key blocks each tile sees
    int edge;                   // first block that not every row sees whole
    int j0, j1;
    int slot;                   // -1: the whole item, else the partial slot
    __device__ __forceinline__ int rows(int x) const { return x ? rows_b : rows_a; }
    // tile x does blocks j0 .. last - 1
    __device__ __forceinline__ int last(int x) const { return min(j1, x ? nblk_b : nblk_a); }
    __device__ __forceinline__ bool uses(int x) const { return last(x) > j0; }
    __device__ __forceinline__ int seen(int token) const { return min(max(first_seen + token, 0), keys); }
};

struct Split {
    int2 seq[kPMaxBatch];       // of a sequence its queries n, and m - n - lag
    int above[kPLevels + 1];    // items of level k and more; a level is 2^shift blocks of an item
    int before[kPMaxBatch + 1]; // items of one level of the sequences before b: of the level that item_at met last
    int scan[2][kThreads / 32];
    int cost[(kPLineRows + 1) * kPMaxCtas];     // prefix of the blocks of the items of the line
    int load[kPMaxCtas];        // blocks that the CTAs do in whole items
    int quota[kPMaxCtas + 1];   // where the CTAs' shares of the line begin
    unsigned long long tiles;   // of all sequences
    int top, shift, levels;
    int rounds, line_items, line_blocks;
};

// x / (2 tile_tokens), x up to 2^24 and a tile more.
__device__ __forceinline__ int pairs_of(const PromptArgs &a, int x) { return (int)__umulhi((uint32_t)x, a.pair_inverse); }

// The following take of a sequence its queries n (x) and m - n - lag (y).
__device__ __forceinline__ int tiles_of(const PromptArgs &a, int2 s) { return pairs_of(a, s.x + 2 * a.tile_tokens - 1); }

// Key blocks that the tokens up to `token` (inclusive) of a sequence see.
__device__ __forceinline__ int blocks_seen(int2 s, int token) { return (max(s.y + token + 1, 0) + kTok - 1) / kTok; }

// Blocks of keys of an item, of its longer tile; one that sees no key still has its output to write.
__device__ __forceinline__ int item_blocks(const PromptArgs &a, int2 s, int tile)
{
    return max(blocks_seen(s, min((tile + 1) * 2 * a.tile_tokens, s.x) - 1), 1);
}

// Tiles of a sequence whose items have at least so many blocks: its last ones.
__device__ __forceinline__ int tiles_from(const PromptArgs &a, int2 s, int blocks)
{
    const int tiles = tiles_of(a, s);
    if (blocks <= 1) return tiles;
    const int need = (blocks - 1) * kTok + 1 - s.y;     // tokens up to the first whose block that is
    if (need > s.x) return 0;
    return need <= 0 ? tiles : tiles - pairs_of(a, need - 1);
}

// The level of item `i`: the last one with more than i items of it and above.
__device__ __forceinline__ int level_of(const Split &sp, int i)
{
    int lo = 0, hi = sp.levels;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sp.above[mid] > i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Item `i` of the call, by a whole warp: items go by levels from the highest down, in a level by sequences, tiles from the
// last down, and heads.  met: the level of sp.before, or -1.
__device__ __forceinline__ Piece item_at(const PromptArgs &a, Split &sp, int i, int &met)
{
    const int lane = threadIdx.x & 31, level = level_of(sp, i), low = level << sp.shift, high = (level + 1) << sp.shift;
    if (level != met) {
        met = level;
        int all = 0;
        __syncwarp();
        for (int b0 = 0; b0 < a.batch; b0 += 32) {
            const int2 q = b0 + lane < a.batch ? sp.seq[b0 + lane] : make_int2(0, 0);
            const int own = (tiles_from(a, q, low) - tiles_from(a, q, high)) * a.kv_heads;
            int x = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (b0 + lane < a.batch) sp.before[b0 + lane] = all + x - own;
            all += __shfl_sync(0xffffffffu, x, 31);
        }
        __syncwarp();
    }
    const int place = i - sp.above[level + 1];
    int b = 0, end = a.batch;           // the last b with before[b] <= place
    while (end - b > 1) {
        const int mid = (b + end) >> 1;
        if (sp.before[mid] <= place) b = mid;
        else end = mid;
    }
    const Seq s = sequence(a, b, false);
    const int2 q = sp.seq[b];
    const uint32_t in = place - sp.before[b], down = in / (uint32_t)a.kv_heads;
    const int T = a.tile_tokens;
    Piece p;
    p.seq = b;
    p.head = in - down * a.kv_heads;
    p.tile = tiles_of(a, q) - 1 - tiles_from(a, q, high) - down;
    const int tok0 = 2 * p.tile * T, ta = min(T, s.n - tok0), tb = max(min(T, s.n - tok0 - T), 0);  // the item exists: ta >= 1
    p.row0 = s.q0 + tok0;
    p.key0 = s.k0;
    p.keys = s.m;
    p.first_seen = s.m - s.n - a.lag + tok0 + 1;
    p.rows_a = ta * a.G;
    p.rows_b = tb * a.G;
    p.nblk_a = blocks_seen(q, tok0 + ta - 1);
    p.nblk_b = tb > 0 ? blocks_seen(q, tok0 + T + tb - 1) : 0;
    p.edge = p.seen(0) / kTok;
    p.j0 = 0;
    p.j1 = max(p.nblk_a, p.nblk_b);
    p.slot = -1;
    return p;
}

// Sum of v over the threads before this one, and over all; calls take turns with the two halves of sp.scan.
__device__ __forceinline__ int block_scan(Split &sp, int v, int *total, int &turn)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int *sums = sp.scan[turn];
    turn ^= 1;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w++) {
        if (w < warp) before += sums[w];
        all += sums[w];
    }
    *total = all;
    return before + x - v;
}

// The last item of the line with cost[item] <= at: the one that holds block `at`.
__device__ __forceinline__ int item_of(const Split &sp, int at)
{
    int lo = 0, hi = sp.line_items;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sp.cost[mid] <= at) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Blocks of item `i`, for one thread.
__device__ __forceinline__ int blocks_at(const PromptArgs &a, const Split &sp, int i)
{
    const int level = level_of(sp, i);
    if (sp.shift == 0) return level;
    int in = i - sp.above[level + 1];
    for (int b = 0;; b++) {
        const int above = tiles_from(a, sp.seq[b], (level + 1) << sp.shift);
        const int own = (tiles_from(a, sp.seq[b], level << sp.shift) - above) * a.kv_heads;
        if (in < own) return item_blocks(a, sp.seq[b], tiles_of(a, sp.seq[b]) - 1 - above - in / a.kv_heads);
        in -= own;
    }
}

// The whole split, by all threads of the CTA.
__device__ __forceinline__ void make_split(const PromptArgs &a, Split &sp)
{
    const int tid = threadIdx.x, grid = gridDim.x;
    int turn = 0;
    if (tid == 0) {
        sp.top = 0;
        sp.tiles = 0;
    }
    __syncthreads();
    for (int b = tid; b < a.batch; b += kThreads) {
        const Seq s = sequence(a, b, blockIdx.x == 0);
        const int2 q = make_int2(s.n, s.m - s.n - a.lag);
        sp.seq[b] = q;
        if (s.n > 0) {
            atomicMax(&sp.top, item_blocks(a, q, tiles_of(a, q) - 1));
            atomicAdd(&sp.tiles, (unsigned long long)tiles_of(a, q));
        }
    }
    __syncthreads();
    // More tiles than sequences behind one another can have: starts that go back, with other sequences on the same rows.
    // Nothing is done then; counts that fit 32 bits would not be sure.
    const bool none = sp.tiles > (unsigned long long)a.most_tiles;
    if (none && tid == 0 && blockIdx.x == 0) atomicOr(a.err, kPErrStarts);
    const int top = none ? 0 : sp.top;
    int shift = 0;
    while (top >> shift >= kPLevels) shift++;
    const int levels = (top >> shift) + 1;
    if (levels > 4 * a.batch) {         // a thread to a level, or, with many sequences, a warp (1024 of 16 tokens: 302 -> 262 us)
        for (int k = tid; k <= levels; k += kThreads) {
            int tiles = 0;
            for (int b = 0; b < a.batch; b++) tiles += tiles_from(a, sp.seq[b], k << shift);
            sp.above[k] = none ? 0 : tiles * a.kv_heads;
        }
    } else {
        for (int k = tid >> 5; k <= levels; k += kThreads / 32) {
            int tiles = 0;
            for (int b = tid & 31; b < a.batch; b += 32) tiles += tiles_from(a, sp.seq[b], k << shift);
            tiles = __reduce_add_sync(0xffffffffu, tiles);
            if ((tid & 31) == 0) sp.above[k] = none ? 0 : tiles * a.kv_heads;
        }
    }
    if (tid == 0) {
        sp.shift = shift;
        sp.levels = levels;
    }
    __syncthreads();
    const int items = sp.above[0], rounds = max(items / grid - kPLineRows, 0), first = rounds * grid, line = items - first;
    // blocks of the whole items (where levels are coarse: about)
    if (tid < kPMaxCtas) {
        int load = 0;
        if (tid < grid)
            for (int r = 0, k = levels - 1; r < rounds; r++) {
                const int i = r * grid + (r & 1 ? grid - 1 - tid : tid);
                while (sp.above[k] <= i) k--;
                load += (k << shift) + kPExtra;
            }
        sp.load[tid] = load;
    }
    // blocks of the line
    int total = 0;
    for (int i0 = 0; i0 < line; i0 += kThreads) {
        const int i = i0 + tid;
        int all;
        const int own = i < line ? blocks_at(a, sp, first + i) + kPExtra : 0, at = block_scan(sp, own, &all, turn);
        if (i < line) sp.cost[i] = total + at;
        total += all;
    }
    __syncthreads();
    if (tid < 32) {
        // The level at which the CTAs' shares, level - load, add up to the line: the mean over all, or, where some CTAs are
        // past that already, over the others, until none is left out any more.  A lane has kPer consecutive CTAs.
        constexpr int kPer = kPMaxCtas / 32;
        const int per = (grid + 31) / 32;
        int load[kPer];
#pragma unroll
        for (int i = 0; i < kPer; i++) load[i] = i < per && tid * per + i < grid ? sp.load[tid * per + i] : INT_MAX;
        int level = INT_MAX, in = 0;
        if (rounds == 0) level = (total + grid - 1) / grid;
        else for (;;) {
            int n = 0;
            long long sum = 0;
#pragma unroll
            for (int i = 0; i < kPer; i++)
                if (load[i] < level) {
                    n++;
                    sum += load[i];
                }
            n = __reduce_add_sync(0xffffffffu, n);
            if (n == in || n == 0) break;
            in = n;
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            level = (int)((sum + total + n - 1) / n);
        }
        int share = 0;
#pragma unroll
        for (int i = 0; i < kPer; i++) share += max(level - load[i], 0);
        int at = share;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, at, o);
            if (tid >= o) at += y;
        }
        at -= share;
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (i < per && tid * per + i < grid) {
                sp.quota[tid * per + i] = min(at, total);
                at += max(level - load[i], 0);
            }
        if (tid == 0) {
            sp.quota[grid] = total;
            sp.rounds = rounds;
            sp.line_items = line;
            sp.line_blocks = total;
        }
    }
    __syncthreads();
    // The extra blocks of an item stand in front.  A bound that would leave a piece with them alone moves to the item's
    // beginning, which may leave a CTA without a share.
    if (tid < grid) {
        const int at = sp.quota[tid];
        if (at < total) {
            const int start = sp.cost[item_of(sp, at)];
            if (at - start <= kPExtra) sp.quota[tid] = start;
        }
    }
    __syncthreads();
}

// A CTA's pieces, one after another: first its whole items, then its share of
// the line.
struct Walk {
    int round, item, at, end, met = -1;
    PromptMeta meta{-1, 0, 0, 0, 0, {0, 0, 0}};     // the item that begins in this CTA's share and runs on behind it
    __device__ __forceinline__ Walk(const Split &sp)
    {
        round = 0;
        at = sp.quota[blockIdx.x];
        end = sp.quota[blockIdx.x + 1];
        item = item_of(sp, at);
    }
    __device__ __forceinline__ Piece next(const PromptArgs &a, Split &sp)
    {
        const int grid = gridDim.x;
        Piece p;
        p.seq = -1;
        if (round < sp.rounds) {
            p = item_at(a, sp, round * grid + (round & 1 ? grid - 1 - blockIdx.x : blockIdx.x), met);
            round++;
        } else if (at < end) {
            p = item_at(a, sp, sp.rounds * grid + item, met);
            const int start = sp.cost[item], stop = start + kPExtra + max(p.j1, 1);
            const bool begins = start >= at, ends = stop <= end;
            if (!begins || !ends) {
                p.slot = begins ? 1 : 0;
                if (begins) {
                    int c = blockIdx.x;
                    while (sp.quota[c + 1] < stop) c++;
                    meta = PromptMeta{p.seq, p.head, p.tile, (int)blockIdx.x, c, {0, 0, 0}};
                }
                p.j0 = max(at - start - kPExtra, 0);
                p.j1 = min(p.j1, end - start - kPExtra);
            }
            at = min(stop, end);
            item++;
        }
        return p;
    }
};

// An infinity becomes NaN, as the values on an edge become (x * 0 is NaN for it, else a zero of x's sign).
__device__ __forceinline__ float finite_or_nan(float x) { return __fmaf_rn(x, 0.f, x); }

// 32 bytes of a row.
__device__ __forceinline__ void store32(void *to, const uint32_t *w)
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n"
                 :: "l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

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

// A row's sum of the runs before, in memory: element 4 i .. 4 i + 3 at carry[128 i],
// so that a warp's rows are one line.  leave_run adds O of the row to it (or starts
// it; f brings it to O's reference), take_run adds it, times f, to O.
__device__ __noinline__ void leave_run(uint32_t tO, float4 *carry, bool starts, float f)
{
    if (!starts && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
        for (int i = 0; i < kD / 4; i++) {
            const float4 v = __ldcg(carry + 128 * i);
            __stcg(carry + 128 * i, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
        }
    }
#pragma unroll 1
    for (int c = 0; c < 4; c++) {
        float o[32];
        tmem_ld32(tO + 32 * c, o);
        tmem_wait_ld();
        float4 *to = carry + 1024 * c;
        if (starts) {
#pragma unroll
            for (int i = 0; i < 8; i++) __stcg(to + 128 * i, make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};\n"
                             :: "l"(to + 128 * i), "f"(o[4 * i]), "f"(o[4 * i + 1]), "f"(o[4 * i + 2]), "f"(o[4 * i + 3])
                             : "memory");
        }
    }
}

__device__ __noinline__ void take_run(uint32_t tO, const float4 *carry, float f)
{
#pragma unroll 1
    for (int c = 0; c < 8; c++) {
        float o[16];
        tmem_ld16(tO + 16 * c, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float4 v = __ldcg(carry + 512 * c + 128 * i);
            o[4 * i] = fmaf(v.x, f, o[4 * i]), o[4 * i + 1] = fmaf(v.y, f, o[4 * i + 1]);
            o[4 * i + 2] = fmaf(v.z, f, o[4 * i + 2]), o[4 * i + 3] = fmaf(v.w, f, o[4 * i + 3]);
        }
        tmem_st16(tO + 16 * c, reinterpret_cast<const uint32_t *>(o));
    }
    tmem_wait_st();
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
    if (edge && __any_sync(0xffffffffu, live < kTok)) {
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

// Does a run of blocks, whose products add up in tensor memory, begin with block j of a piece?
template <bool kWide, bool kRuns>
__device__ __forceinline__ bool run_begins(int j, int j0)
{
    return kRuns ? ((j - j0) & ((kWide ? kWideRun : kRun) - 1)) == 0 : j == j0;
}

struct Bars {
    unsigned long long full[kStages], empty[kStages];   // ring of key and value blocks
    unsigned long long q_full[2], q_empty[2];           // Q of a tile
    unsigned long long s_full[2], p_full[2], o_full[2]; // scores made, weights written, output complete
    unsigned long long v_ok[2], done;                   // values of an odd stage looked through
    unsigned long long next[kPieces], free[kPieces];    // pieces announced, and taken back by all that follow them
};

// The pieces ahead, and for each the first token whose value is not finite, by
// element.
struct Queue {
    Piece piece[kPieces];
    int bad[kPieces][kD], dirty[kPieces];
};

// Follows the queue: take(p) waits for the next piece (false: none, or a wait
// gave up), done() gives its place back.
struct Follow {
    Queue &q;
    Bars &bars;
    volatile int *fail;
    uint32_t k = 0;
    __device__ __forceinline__ int place() const { return k % kPieces; }
    __device__ __forceinline__ const Piece *take()
    {
        if (!wait_or_fail(smem_u32(&bars.next[place()]), k / kPieces & 1, fail)) return nullptr;
        const Piece *p = &q.piece[place()];
        return p->seq < 0 ? nullptr : p;
    }
    __device__ __forceinline__ void done(bool one)
    {
        if (one) mbar_arrive(smem_u32(&bars.free[place()]));
        k++;
    }
};

// kWide: fp32 outputs.  kRuns: pieces may be longer than a run.
template <bool kWide, bool kRuns>
__global__ void __launch_bounds__(kThreads, 1) prompt_attention_kernel(const __grid_constant__ PromptArgs a,
                                                                      const __grid_constant__ PromptMaps maps)
{
    extern __shared__ __align__(1024) uint8_t dyn_raw[];
    __shared__ Split sp;
    __shared__ __align__(8) Bars bars;
    __shared__ Queue queue;
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;
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
            mbar_init(B_(bars.p_full[x]), 4);                  // one arrival per warp
            mbar_init(B_(bars.o_full[x]), 1);
            mbar_init(B_(bars.v_ok[x]), 1);
        }
        mbar_init(B_(bars.done), 1);
        for (int i = 0; i < kPieces; i++) {
            mbar_init(B_(bars.next[i]), 1);
            mbar_init(B_(bars.free[i]), 11);                    // the softmax warps, the products', the loader and warp 10
        }
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        s_fail = 0;
    }
    // Rows of the tiles that no token fills, where 128 is no multiple of the group: zeros, which no copy overwrites.  Scores
    // from whatever stood there could take the paths for references that move or are huge (5 prompts with 28 / 4 heads 233 -> 222 us).
    const int used = a.tile_tokens * a.G, spare = (128 - used) * 8;
    for (int i = tid; i < 4 * spare; i += kThreads)
        *reinterpret_cast<uint4 *>(base + i / spare * (kBlockBytes / 2) + used * 128 + i % spare * 16) = make_uint4(0, 0, 0, 0);
    if (spare) asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    for (int i = tid; i < kPieces * kD; i += kThreads) queue.bad[i / kD][i % kD] = INT_MAX;
    if (tid < kPieces) queue.dirty[tid] = 0;
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n"
                     :: "r"(smem_u32(&s_tmem)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = 0;            // all 512 columns: the allocation starts at column 0
    if (tid == 0 && s_tmem != 0) s_fail = 1;
    pdl_wait();
    make_split(a, sp);

    Follow follow{queue, bars, fail};
    if (warp < 8) {
        more_registers<kSoftmaxRegs>();
        // softmax and output: a thread per row of its tile
        const int x = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + 128 * x + lanes, tO = tmem + 256 + 128 * x + lanes;
        const float sc = a.scale_log2;
        uint32_t ns = 0, no = 0;
        bool ok = true;
        // a CTA without a share of the line has no part in the items that span it
        if (sp.quota[blockIdx.x] == sp.quota[blockIdx.x + 1])
            a.part_ml[(int64_t)blockIdx.x * 2 * kPRows + tid] = make_float2(0.f, 0.f);
        while (const Piece *p = follow.take()) {
            const int j0 = p->j0, last = p->last(x), edge = p->edge;
            const bool valid = row < p->rows(x);
            const int lim = valid ? p->seen(x * a.tile_tokens + row / a.G) : 0;       // keys the row sees
            float ref = kLowest, sum = 0.f, carry_ref = kLowest;
            bool carried = false;
            float4 *carry = a.carry + ((int64_t)blockIdx.x * 2 + x) * (kD / 4) * 128 + row;
            for (int j = j0; j < last; j++) {
                if (!wait_or_fail(B_(bars.s_full[x]), ns & 1, fail)) {
                    ok = false;
                    break;
                }
                ns++;
                fence_after();
                const bool starts = run_begins<kWide, kRuns>(j, j0);
                if (kRuns && starts && j > j0) {
                    // the products before are complete: these scores were issued behind them
                    leave_run(tO, carry, !carried, ex2_approx(carry_ref - ref));
                    carried = true;
                    carry_ref = ref;
                }
                const int live = lim - j * kTok;        // of the block's keys, those that the row sees
                softmax_block<kWide>(tS, tO, sc, live, j >= edge, !starts, ref, sum);
                tmem_wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(B_(bars.p_full[x]));
            }
            if (!ok) break;

            // The row's output, or its part of one.  What needs no product comes while the last one runs.
            const bool some = last > j0;
            const int slot = p->slot;
            const bool part = slot >= 0;
            // a row that sees keys and has no weight, its scores being minus infinity, is 0 / 0
            const float none = lim > 0 && !part ? CUDART_NAN_F : 0.f;
            const float scale = !some || sum == 0.f ? none : part ? 1.f : 1.f / sum;
            const int row_tok = row / a.G;
            const int64_t out_row = (int64_t)(p->row0 + x * a.tile_tokens + row_tok) * a.heads + p->head * a.G + row - row_tok * a.G;
            const int64_t part_row = ((int64_t)blockIdx.x * 2 + slot) * kPRows + 128 * x + row;
            const bool fp32 = part || kWide;
            char *to = fp32 ? reinterpret_cast<char *>(part ? a.part_o + part_row * kD : reinterpret_cast<float *>(a.out) + out_row * kD)
                            : reinterpret_cast<char *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + out_row * kD);
            if (valid) {
                if (part) a.part_ml[part_row] = make_float2(ref, sum);
                else if (a.lse) a.lse[out_row] = sum == 0.f ? none - CUDART_INF_F : (ref + log2f(sum)) * kLn2;
            }
            const bool every = __all_sync(0xffffffffu, scale != 0.f);       // else some rows' O was never written, or is to be 0
            if (some) {
                if (!wait_or_fail(B_(bars.o_full[x]), no & 1, fail)) break;
                no++;
                fence_after();
            }
            if (kRuns && carried) take_run(tO, carry, ex2_approx(carry_ref - ref));
            const bool dirty = some && *(volatile int *)&queue.dirty[follow.place()];
            const int *bad = queue.bad[follow.place()];
            // (rolled up: once per piece, its instructions come from far away; with a body of 32 columns for bf16 24 ragged
            // prompts 412 us instead of 407, 1024 of 16 tokens 291 instead of 278)
#pragma unroll 1
            for (int c = 0; c < 8; c++) {
                float o[16];
                tmem_ld16(tO + 16 * c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i++) o[i] = finite_or_nan(o[i] * scale);
                if (!every || dirty) {
#pragma unroll
                    for (int i = 0; i < 16; i++) {
                        if (scale == 0.f) o[i] = 0.f;
                        if (dirty && bad[16 * c + i] < lim) o[i] = CUDART_NAN_F;
                    }
                }
                if (!valid) continue;
                uint32_t w[16];
                if (fp32) {
#pragma unroll
                    for (int i = 0; i < 16; i++) w[i] = __float_as_uint(o[i]);
                    store32(to + 64 * c, w);
                    store32(to + 64 * c + 32, w + 8);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++) w[i] = bf16_pair(o[2 * i], o[2 * i + 1]);
                    store32(to + 32 * c, w);
                }
            }
            fence_before();
            __syncwarp();
            follow.done(lane == 0);
        }
    } else {
        fewer_registers<kOtherRegs>();
        if (warp == kLoadWarp) {
            if (lane == 0) {
                uint32_t n = 0;             // blocks issued: use n of the ring is in stage n % kStages
                bool ok = true;
                while (const Piece *p = follow.take()) {
                    const int j1 = p->j1, head = p->head, key0 = p->key0;
                    for (int j = p->j0; j < j1 && ok; j++)
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
                                tma_load(dst + h * (kBlockBytes / 2), map, 64 * h, head, key0 + j * kTok, full);
                        }
                    if (!ok) break;
                    follow.done(true);
                }
                // before the CTA exits, the copies that it issued have landed
                for (uint32_t s = 0; s < kStages; s++) {
                    const uint32_t uses = (n + kStages - 1 - s) / kStages;
                    if (uses) wait_bounded(B_(bars.full[s]), (uses - 1) & 1);
                }
            }
        } else if (warp == kMmaWarp) {
            // The whole warp walks and waits, so that addresses stay uniform, and one lane issues.  The pipe takes one product
            // ahead of the one that it works on, so what stands between two products must be short, and a wait behind the last
            // of eight would leave the pipe idle for the 100 to 200 cycles that even a completed barrier costs here: the next
            // eight's barriers are tested before the last.  A wait that gives up is noted and the piece goes on: every later wait then gives up
            // soon, and nothing is read out of bounds.
            constexpr int kAhead = 7;
            constexpr uint32_t kStep = kBlockBytes >> 4;        // a stage, or a tile of Q, in descriptor units
            uint32_t m = 0;             // blocks so far: block m's keys are use 2 m of the ring, its values use 2 m + 1
            uint32_t nq[2] = {0, 0}, np[2] = {0, 0};
            const uint32_t q_low = desc_low(sQ, 16), key_low = desc_low(sKV, 16), value_low = desc_low(sKV, kBlockBytes / 2);
            auto wait = [&](unsigned long long &bar, uint32_t k) { wait_or_fail(B_(bar), k & 1, fail); };
            auto test = [&](unsigned long long &bar, uint32_t k) { return phase_done(B_(bar), k & 1); };
            auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
            // scores of tile x against the key block at `keys`; `ahead` is called before the last products
            auto score = [&](uint32_t x, uint32_t keys, bool final, auto &&ahead) {
                auto product = [&](int k) {
                    const uint32_t off = ((k >> 2) * (kBlockBytes / 2) + (k & 3) * 32) >> 4;
                    if (k == 0) mma_ss<false>(128 * x, q_low + x * kStep + off, keys + off, kIdescS);
                    else mma_ss<true>(128 * x, q_low + x * kStep + off, keys + off, kIdescS);
                };
                fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kAhead; k++) product(k);
                }
                ahead();
                if (elect_one()) {
#pragma unroll
                    for (int k = kAhead; k < 8; k++) product(k);
                    commit(B_(bars.s_full[x]));
                    if (final) commit(B_(bars.q_empty[x]));
                }
            };
            // weights of tile x times the value block at `values`
            auto output = [&](uint32_t x, uint32_t values, bool first, bool final, auto &&ahead) {
                auto product = [&](int part, int k, uint32_t add) {
                    mma_ts(256 + 128 * x, 128 * x + 64 * part + 8 * k, values + k * (2048 >> 4), kIdescO, add);
                };
                fence_after();
                if (elect_one()) {
                    product(0, 0, !first);
                    if (kWide) {
#pragma unroll
                        for (int k = 0; k < 8; k++) product(1, k, 1);
                    }
#pragma unroll
                    for (int k = 1; k < kAhead; k++) product(0, k, 1);
                }
                ahead();
                if (elect_one()) {
#pragma unroll
                    for (int k = kAhead; k < 8; k++) product(0, k, 1);
                    if (final) commit(B_(bars.o_full[x]));
                }
            };
            auto release = [&](int st) {
                if (elect_one()) commit(B_(bars.empty[st]));
            };
            while (const Piece *p = follow.take()) {
                const int j0 = same(p->j0), j1 = same(p->j1), edge = same(p->edge), last_a = same(p->last(0)), last_b = same(p->last(1));
                __syncwarp();
                follow.done(lane == 0);
                if (j1 == j0) continue;
                // Outputs of block j, and the scores of j + 1 (m: its keys are use 2 m of the ring, block j's values use
                // 2 m - 1), tile after tile.  Steady blocks: both tiles go on, no run begins and no row is at its edge.  The others,
                // with the piece's first scores (j = j0 - 1) among them, have a body of their own.  One of each, for both tiles and
                // both halves of the ring: code that comes only now and then has to be fetched from far away.  With bodies for
                // every tile and half, of constants, 24 ragged prompts took 431 us instead of 414, chunks 697 instead of 685, 32768
                // tokens 5.07 ms instead of 4.95; all blocks through the general body 449, 780 and 5.82.
                uint32_t ready_v = 0, ready_p[2] = {0, 0};
                auto steady = [&] {
                    const uint32_t k = 2 * (m & 1), v = 3 - k, keys = key_low + k * kStep, values = value_low + v * kStep;
                    uint32_t ready_k = 0;
                    if (!ready_v) wait(bars.full[v], (m - 1) >> 1);
#pragma unroll 1
                    for (uint32_t x = 0; x < 2; x++) {
                        if (!(x ? ready_p[1] : ready_p[0])) wait(bars.p_full[x], x ? np[1] : np[0]);
                        if (x) np[1]++;
                        else np[0]++;
                        output(x, values, false, false, [&] {
                            if (!x) ready_k = test(bars.full[k], m >> 1);
                        });
                        if (x) release(v);
                        else if (!ready_k) wait(bars.full[k], m >> 1);
                        score(x, keys, false, [&] {
                            if (x) ready_v = test(bars.full[k + 1], m >> 1);
                            const uint32_t other = test(bars.p_full[1 - x], x ? np[0] : np[1]);
                            if (x) ready_p[0] = other;
                            else ready_p[1] = other;
                        });
                    }
                    release(k);
                };
                auto block = [&](int j) {
                    const bool now = j >= j0, more = j + 1 < j1;
                    const uint32_t half = m & 1, v = 3 - 2 * half, k = 2 * half;
                    const uint32_t keys = key_low + k * kStep, values = value_low + v * kStep;
                    uint32_t ready_k = !more;
                    if (now) {
                        if (!ready_v) wait(bars.full[v], (m - 1) >> 1);
                        if (j >= edge) wait(bars.v_ok[1 - half], (m - 1) >> 1);
                    }
#pragma unroll 1
                    for (uint32_t x = 0; x < 2; x++) {
                        const int last = x ? last_b : last_a;
                        if (now && j < last) {
                            if (!(x ? ready_p[1] : ready_p[0])) wait(bars.p_full[x], x ? np[1] : np[0]);
                            if (x) np[1]++;
                            else np[0]++;
                            output(x, values, run_begins<kWide, kRuns>(j, j0), j + 1 == last, [&] {
                                if (!x && more) ready_k = test(bars.full[k], m >> 1);
                            });
                        }
                        if (x) {
                            if (now) release(v);
                            ready_v = ready_p[0] = 0;
                        } else {
                            if (!ready_k) wait(bars.full[k], m >> 1);
                            ready_p[1] = 0;
                        }
                        if (j + 1 < last) {
                            if (!now) wait(bars.q_full[x], x ? nq[1]++ : nq[0]++);
                            score(x, keys, j + 2 == last, [&] {
                                if (x) ready_v = test(bars.full[k + 1], m >> 1);
                                else if (now && j < last_b) ready_p[1] = test(bars.p_full[1], np[1]);
                                if (x && now && j + 1 < last_a) ready_p[0] = test(bars.p_full[0], np[0]);
                            });
                        }
                    }
                    if (more) release(k);
                };
                const int steady_end = min(min(last_a, last_b) - 2, edge);
#pragma unroll 1
                for (int j = j0 - 1; j < j1; j++, m++) {
                    if (j < j0 || j >= steady_end || run_begins<kWide, kRuns>(j, j0)) block(j);
                    else steady();
                }
                m--;
            }
            // every product issued is complete before the CTA frees its tensor memory
            if (elect_one()) commit(B_(bars.done));
            wait_bounded(B_(bars.done), 0);
        } else if (warp == kCheckWarp) {
            uint32_t n = 0, nq[2] = {0, 0};
            const uint32_t q_bytes = (uint32_t)a.tile_tokens * a.G * 256;
            bool ok = true;
            while (const Piece *p = follow.take()) {
                const int j0 = p->j0, j1 = p->j1, edge = p->edge;
#pragma unroll
                for (int x = 0; x < 2; x++)
                    if (ok && p->uses(x)) {
                        if (nq[x] && !wait_or_fail(B_(bars.q_empty[x]), (nq[x] - 1) & 1, fail)) {
                            ok = false;
                        } else if (lane == 0) {
                            mbar_expect(B_(bars.q_full[x]), q_bytes);
                            for (int h = 0; h < 2; h++)
                                tma_load(sQ + x * kBlockBytes + h * (kBlockBytes / 2), &maps.q, 64 * h, p->head * a.G,
                                         p->row0 + x * a.tile_tokens, B_(bars.q_full[x]));
                        }
                        if (ok) nq[x]++;
                    }
                for (int j = j0; j < j1 && ok; j++) {
                    const uint32_t use = n + 2 * (j - j0) + 1, st = use % kStages;
                    if (!wait_or_fail(B_(bars.full[st]), use / kStages & 1, fail)) {
                        ok = false;
                        break;
                    }
                    if (j >= edge) {
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
                            const int at = follow.place();
#pragma unroll 1
                            for (int i = lane; i < kBlockBytes / 2; i += 32) {
                                uint16_t *e = reinterpret_cast<uint16_t *>(v) + i;
                                if ((*e & 0x7f80) != 0x7f80) continue;
                                // element i of the swizzled tile: half, row (token), 16-byte chunk
                                const int half = i >> 13, row = i >> 6 & 127, chunk = (i >> 3 & 7) ^ (row & 7);
                                *e = 0;
                                atomicMin(&queue.bad[at][half * 64 + chunk * 8 + (i & 7)], j * kTok + row);
                            }
                            __syncwarp();
                            if (lane == 0) queue.dirty[at] = 1;
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
                if (!ok) break;
                n += 2 * (j1 - j0);
                __syncwarp();
                follow.done(lane == 0);
            }
            // before the CTA exits, the copies that it issued have landed
            if (lane == 0)
                for (int x = 0; x < 2; x++)
                    if (nq[x]) wait_bounded(B_(bars.q_full[x]), (nq[x] - 1) & 1);
        } else {
            // announces the pieces, a few ahead: finding one takes more time than a block of keys
            Walk walk(sp);
            for (uint32_t k = 0;; k++) {
                const int at = k % kPieces;
                const Piece p = walk.next(a, sp);
                if (k >= kPieces) {
                    if (!wait_or_fail(B_(bars.free[at]), (k / kPieces - 1) & 1, fail)) break;
                    if (queue.dirty[at]) {
                        for (int d = lane; d < kD; d += 32) queue.bad[at][d] = INT_MAX;
                        __syncwarp();
                        if (lane == 0) queue.dirty[at] = 0;
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    queue.piece[at] = p;
                    mbar_arrive(B_(bars.next[at]));
                }
                if (p.seq < 0) break;
            }
            if (lane == 0) a.meta[blockIdx.x] = walk.meta;      // for the second kernel
        }
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

// The items that several CTAs worked on: block (c, y) merges rows of the one that
// begins in CTA c's share, a warp two rows (one of tile A, one of B), a lane four
// elements; the parts' loads are four ahead of one another.
constexpr int kMergeWarps = 8, kMergeAhead = 4;

template <bool kWide>
__global__ void __launch_bounds__(kMergeWarps * 32) prompt_merge_kernel(const __grid_constant__ PromptArgs a)
{
    pdl_wait();
    const PromptMeta meta = a.meta[blockIdx.x];
    if (meta.seq < 0) return;
    const int lane = threadIdx.x & 31, row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5), T = a.tile_tokens;
    if (row >= T * a.G) return;
    const Seq s = sequence(a, meta.seq, false);
    const int row_tok = row / a.G, row_head = row - row_tok * a.G, tok[2] = {2 * meta.tile * T + row_tok, (2 * meta.tile + 1) * T + row_tok};
    float4 o[2] = {};
    float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};
    for (int c0 = meta.first; c0 <= meta.last; c0 += kMergeAhead) {
        float2 ml[2][kMergeAhead];
        float4 part[2][kMergeAhead];
#pragma unroll
        for (int x = 0; x < 2; x++)
#pragma unroll
            for (int i = 0; i < kMergeAhead; i++) {
                const int c = c0 + i;
                ml[x][i] = make_float2(-CUDART_INF_F, 0.f);
                part[x][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c <= meta.last && tok[x] < s.n) {
                    const int64_t at = ((int64_t)c * 2 + (c == meta.first)) * kPRows + 128 * x + row;
                    ml[x][i] = __ldcg(a.part_ml + at);
                    part[x][i] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * kD) + lane);
                }
            }
#pragma unroll
        for (int x = 0; x < 2; x++)
#pragma unroll
            for (int i = 0; i < kMergeAhead; i++) {
                if (ml[x][i].y == 0.f) continue;        // saw no key
                const float top = fmaxf(m[x], ml[x][i].x), f = ex2_approx(m[x] - top), g = ex2_approx(ml[x][i].x - top);
                const float4 v = part[x][i];
                o[x] = make_float4(o[x].x * f + v.x * g, o[x].y * f + v.y * g, o[x].z * f + v.z * g, o[x].w * f + v.w * g);
                l[x] = l[x] * f + ml[x][i].y * g;
                m[x] = top;
            }
    }
#pragma unroll
    for (int x = 0; x < 2; x++) {
        if (tok[x] >= s.n) continue;
        const float inv = l[x] == 0.f ? 0.f : 1.f / l[x];
        const float none = s.m > 0 && s.m - s.n - a.lag + tok[x] + 1 > 0 ? CUDART_NAN_F : 0.f;      // as in a whole item
        const float4 v = l[x] == 0.f ? make_float4(none, none, none, none)
                                     : make_float4(o[x].x * inv, o[x].y * inv, o[x].z * inv, o[x].w * inv);
        const int64_t at = (int64_t)(s.q0 + tok[x]) * a.heads + meta.head * a.G + row_head;
        if (kWide) reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.out) + at * kD)[lane] = v;
        else
            reinterpret_cast<uint2 *>(reinterpret_cast<__nv_bfloat16 *>(a.out) + at * kD)[lane] =
                make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
        if (lane == 0 && a.lse) a.lse[at] = l[x] == 0.f ? none - CUDART_INF_F : (m[x] + log2f(l[x])) * kLn2;
    }
}

using EncodeTiled = PFN_cuTensorMapEncodeTiled_v12000;

}  // namespace

cudaError_t prompt_attention_config(int sm_count)
{
    if (sm_count > kPMaxCtas) return cudaErrorInvalidConfiguration;
    for (const auto kernel : {prompt_attention_kernel<false, false>, prompt_attention_kernel<false, true>, prompt_attention_kernel<true, true>}) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDynBytes);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
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
    const auto kernel = a.wide ? prompt_attention_kernel<true, true>
                        : a.n_kv > kRun * kTok ? prompt_attention_kernel<false, true> : prompt_attention_kernel<false, false>;
    const cudaError_t e = launch_maybe_pdl(kernel, dim3(sm_count), dim3(kThreads), kDynBytes, s, true, a, maps);
    if (e != cudaSuccess || a.n_kv <= kTok) return e;       // items of one block are not cut
    const auto merge = a.wide ? prompt_merge_kernel<true> : prompt_merge_kernel<false>;
    return launch_maybe_pdl(merge, dim3(sm_count, 128 / kMergeWarps), dim3(kMergeWarps * 32), 0, s, true, a);
}

}  // namespace macgpu
