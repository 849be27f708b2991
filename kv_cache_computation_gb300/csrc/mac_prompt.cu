// Host layer of prompt attention: its handle, argument checks and launch.
#include "../../include/mac.h"
#include "mac_prompt.cuh"

#include <cmath>
#include <cstdio>
#include <mutex>
#include <new>

using namespace macgpu;

struct mac_prompt_ctx {
    mac_prompt_config cfg;
    PromptArgs args;        // what does not change from call to call
    int device = 0, sm_count = 0;
    const char *scratch = nullptr;
    mac_prompt_ctx *next = nullptr;     // live handles, under g_live_mutex
    mac_status sticky = MAC_OK;
    char errbuf[256] = {0};
};

namespace macgpu {

namespace {

// The live handles: one made on another's scratch must not clear the error
// word that they share, which may hold what nobody has read yet.
std::mutex g_live_mutex;
mac_prompt_ctx *g_live = nullptr;

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

// The error word comes first, at one place for all handles that share a scratch.
struct Sizes {
    size_t err, meta, part_ml, part_o, carry, scratch;
};

Sizes scratch_sizes()
{
    Sizes z;
    z.err = 0;
    z.meta = 256;
    z.part_ml = z.meta + align_up(kPMaxCtas * sizeof(PromptMeta));
    z.part_o = z.part_ml + align_up((size_t)kPMaxCtas * 2 * kPRows * sizeof(float2));
    z.carry = z.part_o + (size_t)kPMaxCtas * 2 * kPRows * kD * sizeof(float);
    z.scratch = z.carry + (size_t)kPMaxCtas * kPRows * kD * sizeof(float);
    return z;
}

mac_status check_config(const mac_prompt_config *c)
{
    if (!c) return MAC_ERR_INVALID_ARG;
    if (c->heads < 1 || c->kv_heads < 1 || c->heads % c->kv_heads || c->heads > 4096) return MAC_ERR_INVALID_ARG;
    if (c->heads / c->kv_heads > kPMaxGroup || c->head_dim != kD) return MAC_ERR_INVALID_ARG;
    if (c->max_batch < 1 || c->max_batch > kPMaxBatch) return MAC_ERR_INVALID_ARG;
    if (c->max_tokens < 1 || c->max_tokens > (1 << 24)) return MAC_ERR_INVALID_ARG;
    if (!(c->sm_scale >= 0.f) || !std::isfinite(c->sm_scale)) return MAC_ERR_INVALID_ARG;
    return MAC_OK;
}

mac_status fail_cuda(mac_prompt_ctx *h, cudaError_t e, const char *where)
{
    h->sticky = MAC_ERR_CUDA;
    std::snprintf(h->errbuf, sizeof h->errbuf, "%s: %s", where, cudaGetErrorString(e));
    return MAC_ERR_CUDA;
}

// A refused argument: no text of an earlier error stands for it.
mac_status refuse(mac_prompt_ctx *h, const char *text = "")
{
    std::snprintf(h->errbuf, sizeof h->errbuf, "%s", text);
    return MAC_ERR_INVALID_ARG;
}

// The handle is usable and its device is the current one.
mac_status check_handle(mac_prompt_ctx *h)
{
    if (!h) return MAC_ERR_INVALID_ARG;
    if (h->sticky != MAC_OK) return h->sticky;
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail_cuda(h, e, "cudaGetDevice");
    if (dev != h->device) {
        std::snprintf(h->errbuf, sizeof h->errbuf, "the handle lives on device %d, the current device is %d", h->device, dev);
        return MAC_ERR_INVALID_ARG;
    }
    return MAC_OK;
}

bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace

}  // namespace macgpu

extern "C" {

mac_status mac_prompt_query_sizes(const mac_prompt_config *cfg, size_t *scratch_bytes)
{
    const mac_status st = check_config(cfg);
    if (st != MAC_OK) return st;
    if (scratch_bytes) *scratch_bytes = scratch_sizes().scratch;
    return MAC_OK;
}

mac_status mac_prompt_create(const mac_prompt_config *cfg, void *dev_scratch, size_t scratch_bytes, mac_prompt_handle *out)
{
    if (!out) return MAC_ERR_INVALID_ARG;
    *out = nullptr;
    const mac_status st = check_config(cfg);
    if (st != MAC_OK) return st;
    if (!dev_scratch) return MAC_ERR_INVALID_ARG;
    const Sizes z = scratch_sizes();
    if (!aligned(dev_scratch, 256) || scratch_bytes < z.scratch) return MAC_ERR_OOM;
    mac_prompt_ctx *h = new (std::nothrow) mac_prompt_ctx();
    if (!h) return MAC_ERR_OOM;
    h->cfg = *cfg;
    char *sc = (char *)dev_scratch;
    h->scratch = sc;
    PromptArgs &a = h->args;
    a = PromptArgs{};
    a.heads = cfg->heads;
    a.kv_heads = cfg->kv_heads;
    a.G = cfg->heads / cfg->kv_heads;
    a.tile_tokens = 128 / a.G;
    a.pair_inverse = (uint32_t)(((1ull << 32) + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens));
    const double scale = cfg->sm_scale > 0.f ? (double)cfg->sm_scale : 1.0 / std::sqrt((double)kD);
    a.scale_log2 = (float)(scale * 1.4426950408889634);
    a.err = (uint32_t *)(sc + z.err);
    a.meta = (PromptMeta *)(sc + z.meta);
    a.part_ml = (float2 *)(sc + z.part_ml);
    a.part_o = (float *)(sc + z.part_o);
    a.carry = (float4 *)(sc + z.carry);

    cudaDeviceProp prop;
    bool good = cudaGetDevice(&h->device) == cudaSuccess && cudaGetDeviceProperties(&prop, h->device) == cudaSuccess;
    good = good && prop.major * 10 + prop.minor == 103;
    if (good) {
        h->sm_count = prop.multiProcessorCount;
        std::lock_guard<std::mutex> lock(g_live_mutex);
        bool shared = false;
        for (const mac_prompt_ctx *o = g_live; o; o = o->next) shared |= o->scratch == sc && o->device == h->device;
        good = prompt_attention_config(h->sm_count) == cudaSuccess;
        // work in flight may still use a recycled buffer
        if (good && !shared)
            good = cudaDeviceSynchronize() == cudaSuccess && cudaMemset(sc + z.err, 0, 4) == cudaSuccess &&
                   cudaDeviceSynchronize() == cudaSuccess;
        if (good) {
            h->next = g_live;
            g_live = h;
        }
    }
    if (!good) {
        delete h;
        return MAC_ERR_CUDA;
    }
    *out = h;
    return MAC_OK;
}

mac_status mac_prompt_destroy(mac_prompt_handle h)
{
    if (!h) return MAC_ERR_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(h->device) == cudaSuccess) {
        cudaDeviceSynchronize();
        if (dev != h->device) cudaSetDevice(dev);
    }
    {
        std::lock_guard<std::mutex> lock(g_live_mutex);
        for (mac_prompt_ctx **p = &g_live; *p; p = &(*p)->next)
            if (*p == h) {
                *p = h->next;
                break;
            }
    }
    delete h;
    return MAC_OK;
}

const char *mac_prompt_last_error(mac_prompt_handle h) { return h ? h->errbuf : ""; }

mac_status mac_prompt_attention(mac_prompt_handle h, int batch, int n_q, int n_kv, int lag, const void *dev_q, int64_t q_stride,
                                const void *dev_k, int64_t k_stride, const void *dev_v, int64_t v_stride,
                                const int32_t *dev_starts, const int32_t *dev_k_starts, void *dev_out, int out_fp32,
                                float *dev_lse, void *stream)
{
    const mac_status st = check_handle(h);
    if (st != MAC_OK) return st;
    const mac_prompt_config &c = h->cfg;
    if (batch < 0 || batch > c.max_batch) return refuse(h, "more sequences than the handle was made for");
    if (n_q < 0 || n_q > c.max_tokens) return refuse(h, "more query tokens than the handle was made for");
    if (n_kv < 0 || n_kv > (1 << 26) || lag < 0 || lag > (1 << 30) || (out_fp32 != 0 && out_fp32 != 1)) return refuse(h);
    if (!dev_starts || !aligned(dev_starts, 4) || !aligned(dev_k_starts, 4) || !aligned(dev_lse, 4)) return refuse(h);
    if (batch == 0 || n_q == 0) return MAC_OK;
    if (!dev_q || !dev_out || !aligned(dev_q, 16) || !aligned(dev_out, 32)) return refuse(h);   // outputs go out 32 bytes at a time
    if (n_kv > 0 && (!dev_k || !dev_v || !aligned(dev_k, 16) || !aligned(dev_v, 16))) return refuse(h);
    const int64_t q_row = (int64_t)c.heads * kD, kv_row = (int64_t)c.kv_heads * kD, most = (int64_t)1 << 38;
    if (q_stride < q_row || k_stride < kv_row || v_stride < kv_row || q_stride > most || k_stride > most || v_stride > most)
        return refuse(h);
    if (q_stride % 8 || k_stride % 8 || v_stride % 8) return refuse(h);
    // blocks of keys per SM, at most: the split of the work counts them in 32 bits
    const int most_tiles = n_q / (2 * h->args.tile_tokens) + batch;
    const int64_t items = (int64_t)most_tiles * c.kv_heads;
    if ((items / h->sm_count + 1) * ((int64_t)n_kv / 128 + 1 + kPExtra) > (1ll << 30)) return refuse(h, "more work than a call may hold");
    PromptArgs a = h->args;
    a.batch = batch;
    a.lag = lag;
    a.n_q = n_q;
    a.n_kv = n_kv;
    a.most_tiles = most_tiles;
    a.starts = dev_starts;
    a.k_starts = dev_k_starts ? dev_k_starts : dev_starts;
    a.out = dev_out;
    a.wide = out_fp32;
    a.lse = dev_lse;
    PromptMaps maps;
    cudaError_t e = prompt_maps(a, dev_q, q_stride, dev_k, k_stride, dev_v, v_stride, maps);
    if (e != cudaSuccess) return fail_cuda(h, e, "tensor maps");
    e = launch_prompt_attention(a, maps, h->sm_count, (cudaStream_t)stream);
    return e == cudaSuccess ? MAC_OK : fail_cuda(h, e, "prompt attention launch");
}

mac_status mac_prompt_sync(mac_prompt_handle h)
{
    const mac_status st = check_handle(h);
    if (st != MAC_OK) return st;
    cudaError_t e = cudaDeviceSynchronize();
    uint32_t bits = 0;
    if (e == cudaSuccess) e = cudaMemcpy(&bits, h->args.err, 4, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && bits) e = cudaMemset(h->args.err, 0, 4);
    if (e != cudaSuccess) return fail_cuda(h, e, "mac_prompt_sync");
    h->errbuf[0] = 0;
    if (!bits) return MAC_OK;
    std::snprintf(h->errbuf, sizeof h->errbuf, "device checks met:%s%s",
                  bits & kPErrStarts ? " a sequence whose starts decrease or lie outside the tensors" : "",
                  bits & kPErrTimeout ? " a wait that gave up" : "");
    return MAC_ERR_STATE;
}

}  // extern "C"
