// The page bookkeeping of one serving step, on the GPU from the requests'
// lengths: pages for the new tokens, the finished requests' pages back to the
// free list, the new lengths, and the packed tokens' positions and slots.
//
// Per request b with len tokens, of which `back` are taken back (rejected
// drafts), and n new ones (n < 0: finished), in order:
//   held   = ceil(len / 16), kept = len - back, after = ceil((kept + n) / 16)
//   need   = max(after - held, 0)                    (0 where the request is denied)
//   rel    = held of a finished request, else held less what it keeps
//   begin  = sum of n over earlier requests          (packed tokens)
//   first  = sum of need over earlier requests       (pages taken from the ring)
// Free page ids stand in a ring of num_pages entries; `head` is the next one
// out and `count` how many there are.  Page j of the step's pages is
// ring[head + j]; released pages, the last `rel` of a request's row, go to
// ring[head + count ...].
//
// All of it is integers, a few hundred KB at most, so the launch and the chain
// of dependent steps bound it: load, three block scans, one write phase.  One
// block, or for many tokens or pages one cluster of blocks, does the whole step
// in a single launch: every block makes the scans of the (at most 1024)
// requests for itself, one request per thread, and the cluster barrier behind
// the scans separates all reads of the old state from all writes of the new, so
// a caller may update in place.
// Tokens, new pages and freed pages are then spread over all threads, each
// finding its request by a binary search in shared memory.
// Released pages are read twice: their ids are looked at before anything is
// written, since one outside the pool must not get into the ring.
// Measured in a captured graph: 1 request 5.0 us, 32 requests 5.0, 250 requests
// 5.6; 65536 packed tokens 8.7 us (1 request) to 12.5 (250); 16 requests of
// 131072 tokens released 15 us.
#include "../../include/mac.h"
#include "mac_device.cuh"

using namespace macgpu;

namespace macgpu {

namespace {

constexpr int kThreads = 1024;          // one request per thread in the scans
constexpr int kCluster = 8;             // blocks (a portable cluster size)
// Up to this many packed tokens, and pages that could be released, one block
// does the step.  Both sides, us: 512 tokens 5.3 and 5.3, 1024 5.7 / 5.8 (a
// cluster), 2048 6.4 / 5.7, 16384 16 / 6.4; 512 released pages 7.0 and 7.0, 2048
// 7.2 / 7.2, 8192 10.4 / 8.1, 131072 75 / 14.
constexpr int kOneBlockTokens = 1024;
constexpr int kOneBlockPages = 4096;

struct PageArgs {
    int batch, table_cols, num_pages, max_tokens;
    int64_t table_stride;
    const int32_t *len_in, *new_tokens, *rejected, *state_in;
    int32_t *len_out, *state_out, *table, *ring, *starts, *pos, *slot, *status, *unreleased;
};

template <typename T>
__device__ __forceinline__ T warp_scan(T v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// Inclusive block scan; *total gets the sum.  Ends with a barrier.
template <typename T>
__device__ T block_scan(T v, T *buf, T *total)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const T x = warp_scan(v, lane);
    if (lane == 31) buf[w] = x;
    __syncthreads();
    const T t = warp_scan(buf[lane], lane);
    *total = __shfl_sync(0xffffffffu, t, 31);
    const T before = __shfl_sync(0xffffffffu, t, (w + 31) & 31);
    __syncthreads();
    return x + (w ? before : 0);
}

// The last index with v[i] <= x among n non-decreasing values, v[0] <= x.
__device__ __forceinline__ int last_at_most(const int *v, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int wrap(long long i, int n) { return (int)(i >= n ? i - n : i); }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }

// *p = x in the shared memory of the cluster's block k.
__device__ __forceinline__ void store_in_block(int *p, unsigned k, int x)
{
    uint32_t addr;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(addr) : "r"(smem_u32(p)), "r"(k));
    asm volatile("st.shared::cluster.u32 [%0], %1;\n" :: "r"(addr), "r"(x) : "memory");
}

__global__ void __launch_bounds__(kThreads) page_step_kernel(const __grid_constant__ PageArgs a)
{
    __shared__ long long buf[32];
    __shared__ int ibuf[32];
    __shared__ int s_begin[kThreads], s_first[kThreads], s_rel[kThreads], s_len[kThreads];
    __shared__ int s_held[kThreads], s_from[kThreads];
    __shared__ unsigned char s_ok[kThreads];
    __shared__ int s_stuck[kThreads];       // the request's pages stay: an id among them lies outside the pool
    __shared__ int s_status, s_popped, s_any_stuck;
    const int tid = threadIdx.x, b = tid;
    if (tid == 0) s_status = s_popped = s_any_stuck = 0;
    s_stuck[tid] = 0;
    cluster_arrive();                       // every block may mark requests in every other from the wait on
    pdl_wait();
    const int N = a.num_pages;
    int head = a.state_in[0], count = a.state_in[1];
    const bool bad_state = head < 0 || head >= N || count < 0 || count > N;
    if (bad_state) head = count = 0;
    const bool live = b < a.batch;
    const int len = live ? a.len_in[b] : 0, asked = live ? a.new_tokens[b] : 0;
    const int back = live && asked >= 0 && a.rejected ? a.rejected[b] : 0;
    const bool bad = len < 0 || (long long)len > (long long)a.table_cols * kPage || back < 0 || back > len;
    const long long n = asked > 0 ? asked : 0;
    const int kept = bad ? 0 : len - back, held = bad ? 0 : (len + kPage - 1) / kPage;
    const long long after = bad ? 0 : (kept + n + kPage - 1) / kPage;
    __syncthreads();

    // tokens are counted in 64 bits; pages, at most batch x table_cols of them, fit 32
    long long total;
    int total_rel, ignored;
    const long long end = block_scan(n, buf, &total);
    const bool gone = live && asked < 0 && !bad;
    const bool wide = after > a.table_cols, late = end > a.max_tokens;
    const bool can = live && asked >= 0 && !bad && !wide && !late;
    const int need = can && after > held ? (int)(after - held) : 0;
    const int cum = block_scan(need, ibuf, &ignored);
    const bool dry = can && need > 0 && cum > count;
    bool ok = can && !dry;
    // pages the request gives back: the last of its row
    const long long keeps = gone ? 0 : ok ? after : (kept + kPage - 1) / kPage;
    const int rel = live && keeps < held ? held - (int)keeps : 0;
    const int rel_end = block_scan(rel, ibuf, &total_rel);
    int bits = (dry ? 1 : 0) | (live && bad ? 4 : 0);
    if (live && asked >= 0 && !bad) bits |= wide ? 2 : late ? 8 : 0;
    if (bits) atomicOr(&s_status, bits);
    if (ok && need > 0) atomicMax(&s_popped, cum);
    const long long cap = a.max_tokens;
    const int begin = (int)(end - n < cap ? end - n : cap);
    s_begin[tid] = begin;
    s_first[tid] = cum - need;
    s_rel[tid] = rel_end - rel;
    s_from[tid] = held - rel;
    s_held[tid] = held;
    s_len[tid] = kept;
    s_ok[tid] = ok;
    __syncthreads();
    const int popped = s_popped;
    const bool give_back = !bad_state && (long long)count + total_rel <= N;
    const int rank = blockIdx.x, stride = gridDim.x * kThreads, gid = rank * kThreads + tid;
    int found = 0;   // status bits met in the table and ring
    cluster_wait();
    // freed pages j0, j0 + 32, ...: their requests and ids (0 past the last), the loads in flight together.  A warp takes
    // kFlight x 32 pages in a row, so a lane's are seldom of two requests and one search serves them.
    constexpr int kFlight = 4;
    const long long first_freed = (long long)(gid - (tid & 31)) * kFlight + (tid & 31);
    auto freed = [&](long long j0, int (&r)[kFlight], int (&id)[kFlight]) {
        int at = 0, next = 0;       // the request and where the one behind it starts
#pragma unroll
        for (int i = 0; i < kFlight; i++) {
            const long long j = j0 + 32 * i;
            id[i] = 0;
            if (j >= total_rel) continue;
            if ((int)j >= next) {
                at = last_at_most(s_rel, a.batch, (int)j);
                next = at + 1 < a.batch ? s_rel[at + 1] : 0x7fffffff;
            }
            r[i] = at;
            id[i] = a.table[at * a.table_stride + s_from[at] + (j - s_rel[at])];
        }
    };
    // an id outside the pool must not reach the ring: its request gives nothing back
    if (give_back) {
        for (long long j0 = first_freed; j0 < total_rel; j0 += (long long)kFlight * stride) {
            int r[kFlight], id[kFlight];
            freed(j0, r, id);
#pragma unroll
            for (int i = 0; i < kFlight; i++) {
                if ((unsigned)id[i] < (unsigned)N) continue;
                found |= 4;
                for (unsigned k = 0; k < gridDim.x; k++) {
                    store_in_block(&s_stuck[r[i]], k, 1);
                    store_in_block(&s_any_stuck, k, 1);
                }
            }
        }
    }

    // every block has read the old lengths and state by now
    cluster_arrive();
    cluster_wait();
    // a request whose pages cannot be given back keeps them all, and its length (it takes none from the ring, either)
    const bool stuck = rel > 0 && (!give_back || s_stuck[tid]);
    if (s_any_stuck || (total_rel && !give_back)) {      // the same in all blocks
        const int mine = stuck ? 0 : rel;
        s_rel[tid] = block_scan(mine, ibuf, &total_rel) - mine;
        if (stuck) {
            ok = false;
            s_ok[tid] = 0;
            s_len[tid] = len;
        }
        if (!give_back) found |= 16;
        __syncthreads();
    }
    if (rank == 0) {
        if (live) {
            a.len_out[b] = gone ? 0 : bad || stuck ? len : ok ? (int)(kept + n) : kept;
            if (a.unreleased) a.unreleased[b] = gone && stuck ? len : 0;
            a.starts[b] = begin;
        }
        if (tid == 0) {
            a.starts[a.batch] = (int)(total < cap ? total : cap);
            if (bad_state) {
                a.state_out[0] = a.state_in[0];
                a.state_out[1] = a.state_in[1];
            } else {
                a.state_out[0] = wrap((long long)head + popped, N);
                a.state_out[1] = count - popped + (give_back ? total_rel : 0);
            }
            found |= s_status | (bad_state ? 4 : 0);
        }
    }
    // block table: the new pages' entries
    for (int j = gid; j < popped; j += stride) {
        const int r = last_at_most(s_first, a.batch, j);
        const int id = a.ring[wrap((long long)head + j, N)];
        if ((unsigned)id >= (unsigned)N) found |= 4;
        a.table[r * a.table_stride + s_held[r] + (j - s_first[r])] = id;
    }
    // released pages behind the ring's last free one
    if (give_back) {
        for (long long j0 = first_freed; j0 < total_rel; j0 += (long long)kFlight * stride) {
            int r[kFlight], id[kFlight];
            freed(j0, r, id);
#pragma unroll
            for (int i = 0; i < kFlight; i++) {
                const long long j = j0 + 32 * i;
                if (j < total_rel) a.ring[wrap(wrap((long long)head + count, N) + j, N)] = id[i];
            }
        }
    }
    // positions and slots of the packed tokens
    const int tokens = (int)(total < cap ? total : cap);
    for (int t = gid; t < a.max_tokens; t += stride) {
        int pos = 0, slot = -1;
        if (t < tokens) {
            const int r = last_at_most(s_begin, a.batch, t), l = s_len[r];
            pos = l + (t - s_begin[r]);
            if (s_ok[r]) {
                const int c = pos / kPage, had = s_held[r];
                const int id = c < had ? a.table[r * a.table_stride + c]
                                       : a.ring[wrap((long long)head + s_first[r] + (c - had), N)];
                if ((unsigned)id < (unsigned)N) slot = id * kPage + pos % kPage;
                else found |= 4;
            }
        }
        a.pos[t] = pos;
        a.slot[t] = slot;
    }
    // status: the bits of the scans (block 0) and those met while writing,
    // gathered in block 0's shared memory of the cluster
    if (found) {
        uint32_t addr;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(addr) : "r"(smem_u32(&s_status)), "r"(0));
        asm volatile("atom.shared::cluster.or.b32 %0, [%0], %1;\n" : "+r"(addr) : "r"(found) : "memory");
    }
    cluster_arrive();
    cluster_wait();
    if (rank == 0 && tid == 0) *a.status = *(volatile int *)&s_status;
}

bool aligned4(const void *p) { return ((uintptr_t)p & 3) == 0; }

}  // namespace

}  // namespace macgpu

extern "C" {

mac_status mac_page_step(int batch, int max_tokens, int num_pages, const int32_t *dev_len_in, const int32_t *dev_new,
                         int32_t *dev_len_out, int32_t *dev_table, int64_t table_stride, int table_cols, int32_t *dev_ring,
                         const int32_t *dev_state_in, int32_t *dev_state_out, int32_t *dev_starts, int32_t *dev_pos,
                         int32_t *dev_slot, int32_t *dev_status, void *stream)
{
    return mac_page_step_ex(batch, max_tokens, num_pages, dev_len_in, dev_new, dev_len_out, dev_table, table_stride,
                            table_cols, dev_ring, dev_state_in, dev_state_out, dev_starts, dev_pos, dev_slot, dev_status,
                            nullptr, nullptr, stream);
}

mac_status mac_page_step_ex(int batch, int max_tokens, int num_pages, const int32_t *dev_len_in, const int32_t *dev_new,
                            int32_t *dev_len_out, int32_t *dev_table, int64_t table_stride, int table_cols,
                            int32_t *dev_ring, const int32_t *dev_state_in, int32_t *dev_state_out, int32_t *dev_starts,
                            int32_t *dev_pos, int32_t *dev_slot, int32_t *dev_status, const int32_t *dev_rejected,
                            int32_t *dev_unreleased, void *stream)
{
    if (batch < 1 || batch > kThreads || max_tokens < 1 || max_tokens > (1 << 30)) return MAC_ERR_INVALID_ARG;
    if (num_pages < 1 || num_pages > (1 << 27) - 1) return MAC_ERR_INVALID_ARG;   // slots are int32
    if (table_cols < 1 || table_cols > (1 << 26) || table_stride < table_cols) return MAC_ERR_INVALID_ARG;
    if ((int64_t)batch * table_cols > 0x7fffffff) return MAC_ERR_INVALID_ARG;
    const void *p[] = {dev_len_in, dev_new, dev_len_out, dev_table, dev_ring, dev_state_in, dev_state_out, dev_starts,
                       dev_pos, dev_slot, dev_status};
    for (const void *x : p)
        if (!x || !aligned4(x)) return MAC_ERR_INVALID_ARG;
    if (!aligned4(dev_rejected) || !aligned4(dev_unreleased)) return MAC_ERR_INVALID_ARG;
    PageArgs a{batch, table_cols, num_pages, max_tokens, table_stride, dev_len_in, dev_new, dev_rejected, dev_state_in,
               dev_len_out, dev_state_out, dev_table, dev_ring, dev_starts, dev_pos, dev_slot, dev_status,
               dev_unreleased};
    const bool small = max_tokens <= kOneBlockTokens && (int64_t)batch * table_cols <= kOneBlockPages;
    const int blocks = small ? 1 : kCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, page_step_kernel, a) == cudaSuccess ? MAC_OK : MAC_ERR_CUDA;
}

}  // extern "C"
