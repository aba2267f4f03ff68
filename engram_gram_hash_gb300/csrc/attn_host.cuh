// Host helpers shared by the attention step's translation units: argument
// checks, the batch as the kernels see it, launches.  Functions over a cache
// take either structure of engram.h (the 16-bit one, the 8-bit one).
#pragma once

#include <algorithm>
#include <cmath>
#include <cstring>
#include <initializer_list>

#include "common.cuh"
#include "host.cuh"

#include "attn_common.cuh"
#include "qk_rope.cuh"

namespace engram {
namespace attn {

static bool finite_pos(float x) { return x > 0.f && x < INFINITY; }

static engram_status check_attn_config(const engram_attn_config *c) {
    if (!c) return ENGRAM_EINVAL;
    if (c->n_kv_heads < 1 || c->n_heads < 1 || c->n_heads % c->n_kv_heads) return ENGRAM_EINVAL;
    if (c->n_heads / c->n_kv_heads > 128 || c->n_heads > 65536) return ENGRAM_EINVAL;
    if (c->head_dim < 8 || c->head_dim > 128 || c->head_dim % 8) return ENGRAM_EINVAL;
    if (c->rope_dim < 0 || c->rope_dim > c->head_dim || c->rope_dim % 16) return ENGRAM_EINVAL;
    if (c->rope_layout > ENGRAM_ROPE_INTERLEAVED || c->dtype > ENGRAM_FP16) return ENGRAM_EINVAL;
    if (!(c->norm_eps >= 0.f) || !finite_pos(c->scale) || c->window < 0) return ENGRAM_EINVAL;
    return ENGRAM_OK;
}

static bool view_ok(const engram_heads *h) {
    return h && h->data && aligned(h->data, 16) && h->token_stride % 8 == 0 && h->head_stride % 8 == 0;
}
static HeadView view(const engram_heads *h) {
    return h ? HeadView{static_cast<uint16_t *>(h->data), h->token_stride, h->head_stride} : HeadView{nullptr, 0, 0};
}

static engram_status check_batch(const engram_kv_batch *b) {
    if (!b || b->n_query < 0 || b->n_seqs < 0) return ENGRAM_EINVAL;
    if (b->n_query > INT32_MAX || b->n_seqs > INT32_MAX || b->table_stride < 0) return ENGRAM_EINVAL;
    if (b->n_query == 0) return ENGRAM_OK;
    if (b->n_seqs < 1 || b->table_stride < 1 || b->table_stride > INT32_MAX) return ENGRAM_EINVAL;
    if (b->table_width < 0 || b->table_width > b->table_stride) return ENGRAM_EINVAL;
    if (!b->seq_offsets || !b->kv_len || !b->block_table) return ENGRAM_EINVAL;
    if (!aligned(b->seq_offsets, 8) || !aligned(b->kv_len, 4) || !aligned(b->block_table, 4)) return ENGRAM_EINVAL;
    return ENGRAM_OK;
}

// Entries of a sequence's row of the block table.
static int64_t table_width(const engram_kv_batch *b) { return b->table_width > 0 ? b->table_width : b->table_stride; }

template <typename Cache>
static Batch device_batch(const engram_kv_batch *b, const Cache *c) {
    Batch d;
    d.offs = b->seq_offsets;
    d.kv_len = b->kv_len;
    d.block_table = b->block_table;
    d.table_stride = b->table_stride;
    d.table_width = table_width(b);
    d.n_seqs = b->n_seqs;
    d.n_query = b->n_query;
    d.n_pages = c->n_pages;
    d.page_size = c->page_size;
    return d;
}

// An ordinary launch that may start while the kernel before it drains: every
// kernel here waits for that kernel's completion before its first global
// access, so this only hides launch latency.
template <typename... P, typename... A>
static engram_status launch_after(void (*kern)(P...), dim3 grid, int threads, int smem, int cluster, cudaStream_t st,
                                  const char *what, const A &...args) {
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr[2];
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.gridDim = grid;
    lc.blockDim = dim3(threads);
    lc.dynamicSmemBytes = smem;
    lc.stream = st;
    lc.attrs = attr;
    lc.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&lc, kern, args...);
    return e == cudaSuccess ? ENGRAM_OK : cuda_fail(e, what);
}

// Norm and rotation of heads, with the append to the 16-bit cache or without.
template <typename E, int LPH, int U, bool APPEND>
static engram_status head_launch_u(const engram_attn_config *cfg, HeadParams &p, cudaStream_t st) {
    constexpr int per = 32 / LPH * U;  // heads per warp; a block takes 8 tokens
    const int64_t blocks = (p.n_tokens + 7) / 8;
    const dim3 grid((unsigned)blocks, (p.n_q + per - 1) / per + (p.n_k + p.n_v + per - 1) / per);
    if (grid.y > 65535) return ENGRAM_EINVAL;
    if (cfg->rope_layout == ENGRAM_ROPE_INTERLEAVED)
        return launch_after(head_kernel<E, LPH, U, true, APPEND>, grid, 256, 0, 1, st, "head_kernel", p);
    return launch_after(head_kernel<E, LPH, U, false, APPEND>, grid, 256, 0, 1, st, "head_kernel", p);
}

static bool many_heads(const HeadParams &p) {
    return p.n_tokens * ((p.n_q + p.n_k + p.n_v + 3) / 4) >= (int64_t)num_sms() * 64;
}
template <typename E, bool APPEND>
static engram_status head_launch(const engram_attn_config *cfg, HeadParams &p, cudaStream_t st) {
    p.head_dim = cfg->head_dim;
    p.rope_dim = cfg->rope_dim;
    p.eps = cfg->norm_eps;
    p.inv_dim = 1.f / (float)cfg->head_dim;
    // One head per lane while the batch leaves SMs idle (a shorter chain per warp), two once there are
    // 64 warps per SM without it: 32,768 tokens of 32 + 8 heads of 128 take 120 us with two, 140 with
    // one, 117 to 145 with four (more registers, fewer warps); 64 tokens 1.8 us with one or two.
    const bool wide = many_heads(p);
    if (cfg->head_dim <= 64)
        return wide ? head_launch_u<E, 4, 2, APPEND>(cfg, p, st) : head_launch_u<E, 4, 1, APPEND>(cfg, p, st);
    return wide ? head_launch_u<E, 8, 2, APPEND>(cfg, p, st) : head_launch_u<E, 8, 1, APPEND>(cfg, p, st);
}

static int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }
static size_t up256(size_t x) { return (x + 255) / 256 * 256; }
static int padded_dim(const engram_attn_config *cfg) { return cfg->head_dim <= 64 ? 64 : 128; }

// Keys that the block table has room for (in a window's reach).
template <typename Cache>
static int64_t keys_most(const engram_attn_config *cfg, const Cache *cache, const engram_kv_batch *batch) {
    const int64_t room = table_width(batch) * cache->page_size;
    return cfg->window > 0 ? std::min<int64_t>(room, (int64_t)cfg->window + 256) : room;
}
// The configuration with a window that hides nothing taken for plain causal attention (0): no position
// reaches the block table's room or 2^31 - 1, so a window of that many tokens ends before every sequence.
template <typename Cache>
static engram_attn_config effective(const engram_attn_config *cfg, const Cache *cache, const engram_kv_batch *batch) {
    engram_attn_config c = *cfg;
    if (c.window >= std::min<int64_t>(table_width(batch) * cache->page_size, INT32_MAX)) c.window = 0;
    return c;
}

}  // namespace attn
}  // namespace engram
