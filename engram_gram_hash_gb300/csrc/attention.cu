// The attention step (head norm + rotation, cache append, paged attention): C
// entry points, argument checks, tensor maps, launches.  A translation unit of
// its own: it shares no device code with the Engram read but the helpers of
// common.cuh, and the two compile side by side.
#include <type_traits>

#include "attn_host.cuh"
#include "attn_rows.cuh"
#include "attn_tile.cuh"

namespace engram {
namespace attn {

cudaError_t take_error(unsigned int *w) { return take_error_word(w); }

static engram_status check_cache(const engram_attn_config *cfg, const engram_kv_cache *c) {
    if (!c || !c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return ENGRAM_EINVAL;
    if (c->n_pages < 1 || c->n_pages > INT32_MAX) return ENGRAM_EINVAL;
    if (c->page_size < 16 || c->page_size > 65536 || c->page_size % 16) return ENGRAM_EINVAL;
    // strides positive (a size of one may still name any), so no value lies before the base
    for (int64_t s : {c->page_stride, c->token_stride, c->head_stride})
        if (s < 8 || s % 8 || s >= (INT64_C(1) << 39)) return ENGRAM_EINVAL;
    if (c->token_stride < cfg->head_dim || c->page_stride < cfg->head_dim) return ENGRAM_EINVAL;
    if (cfg->n_kv_heads > 1 && c->head_stride < cfg->head_dim) return ENGRAM_EINVAL;
    return ENGRAM_OK;
}

// ---------------------------------------------------------------- attention --

// A [page][head][token][D] view of K or V pages for TMA: boxes of 64 values x
// `rows` tokens in 128-byte swizzled rows; values past head_dim read as zeros.
static bool page_map(CUtensorMap *m, const engram_attn_config *cfg, const engram_kv_cache *c, void *base, int rows) {
    auto enc = tensormap_encoder();
    if (!enc) return false;
    cuuint64_t dims[4] = {(cuuint64_t)cfg->head_dim, (cuuint64_t)c->page_size, (cuuint64_t)cfg->n_kv_heads,
                          (cuuint64_t)c->n_pages};
    cuuint64_t strides[3] = {(cuuint64_t)c->token_stride * 2, (cuuint64_t)c->head_stride * 2,
                             (cuuint64_t)c->page_stride * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type =
        cfg->dtype == ENGRAM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return enc(m, type, 4, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static size_t rows_part_o_bytes(const engram_attn_config *cfg) {
    return up256((size_t)num_sms() * 2 * rows::ROWS * padded_dim(cfg) * sizeof(float));
}
static size_t rows_workspace_bytes(const engram_attn_config *cfg) {
    return rows_part_o_bytes(cfg) + up256((size_t)num_sms() * 2 * 2 * rows::ROWS * sizeof(float));
}

// Segments of the rows kernel (row tile x kv head) at most, and the 32 KB key tiles that the block table
// has room for (in a window's reach).
static int64_t rows_segs_most(const engram_attn_config *cfg, const engram_kv_batch *batch) {
    const int64_t group = cfg->n_heads / cfg->n_kv_heads, seqs = std::min(batch->n_seqs, batch->n_query);
    return cfg->n_kv_heads * std::min(batch->n_query * ((group + rows::ROWS - 1) / rows::ROWS),
                                      (batch->n_query * group + (rows::ROWS - 1) * seqs) / rows::ROWS);
}
static int64_t rows_tiles_most(const engram_attn_config *cfg, const engram_kv_cache *cache, const engram_kv_batch *batch) {
    return (keys_most(cfg, cache, batch) * padded_dim(cfg) + 8191) / 8192;
}

// How a segment's tiles are shared out.  The lengths are on the device; what is known here is the room
// of the block tables (tiles at most) and how many segments there are at most.
//   cluster of 8 or 4: few segments and short tables, one launch.  15 clusters of 8 and 36 of 4 fit the
//     GPU at once.
//   whole: no cut, no join; about one segment an SM, or so short that a cut cannot pay.
//   cut: equal runs of tiles for every SM, then the join (a launch and about 5 us).
// Measured, 8 key/value heads of 128, us a call in a CUDA graph, cluster of 8 / of 4 / whole / cut:
//   1 sequence of 500 tokens 7.0 / 7.3 / 9.2 / 9.1, 2,000: 8.4 / 10.4 / 21.7 / 11.0, 4,000: 10.4 / 14.5 / 38 / 14.2,
//     8,000: 14.7 / 22.9 / 70 / 14.2;  2 of 2,000: 16.1 / 10.5 / 21.9 / 10.9;
//   4 of 2,000: 24.2 / 10.7 / 21.9 / 15.2, 4,000: 30.3 / 14.9 / 38 / 18.0;  16 of 500: - / 29 / 9.8 / 15.0,
//     2,000: - / 48 / 25.2 / 31.0;  64 of 1,000: whole 50.7, cut 53.6 with equal lengths, but unequal ones would
//     wait for the longest.
struct RowsShares {
    int32_t cluster, whole, runs;
    bool cut() const { return whole == 0 && runs > 1; }
};
static RowsShares rows_shares(const engram_attn_config *cfg, const engram_kv_cache *cache, const engram_kv_batch *batch) {
    const int64_t tiles = rows_tiles_most(cfg, cache, batch), segs = rows_segs_most(cfg, batch);
    const int sms = num_sms();
    RowsShares p = {1, 0, sms};
    if (tiles > 2 && tiles <= 64 && segs * 12 <= sms) {
        p.cluster = 8;
    } else if (tiles > 2 && tiles <= (segs >= 24 ? 64 : 32) && segs * 4 <= sms - 8) {
        p.cluster = 4;
    } else if (tiles <= 8 || (tiles <= 32 && segs * 2 >= sms && segs <= sms)) {
        p.whole = (int32_t)tiles;
    }
    if (p.cluster > 1) {
        p.whole = 1;
        p.runs = (int32_t)segs;
    }
    return p;
}

template <typename E, int DP>
static engram_status rows_launch(const engram_attn_config *cfg, const engram_kv_cache *cache,
                                 const engram_kv_batch *batch, const engram_heads *q, const engram_heads *out,
                                 float *lse, void *workspace, cudaStream_t st) {
    rows::Params p;
    memset(&p, 0, sizeof(p));
    p.b = device_batch(batch, cache);
    p.q = static_cast<const uint16_t *>(q->data);
    p.q_token_stride = q->token_stride;
    p.q_head_stride = q->head_stride;
    p.out = static_cast<uint16_t *>(out->data);
    p.out_token_stride = out->token_stride;
    p.out_head_stride = out->head_stride;
    p.lse = lse;
    p.values = ValuePages{static_cast<const uint16_t *>(cache->v), cache->page_stride, cache->token_stride, cache->head_stride};
    p.part_o = static_cast<float *>(workspace);
    p.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + rows_part_o_bytes(cfg));
    p.n_heads = cfg->n_heads;
    p.n_kv_heads = cfg->n_kv_heads;
    p.group = cfg->n_heads / cfg->n_kv_heads;
    p.by_group = Divisor(p.group);
    p.by_heads = Divisor(cfg->n_kv_heads);
    p.side = 1;
    p.line_heads = cfg->n_kv_heads;
    p.head_dim = cfg->head_dim;
    p.window = cfg->window;
    p.kt_log2 = rows::Cfg<DP>::KT_LOG2;
    p.box = gcd(cache->page_size, rows::Cfg<DP>::KT);
    const RowsShares shares = rows_shares(cfg, cache, batch);
    p.cluster = shares.cluster;
    p.whole = shares.whole;
    p.runs = shares.runs;
    p.scale_log2 = cfg->scale * 1.4426950408889634f;
    CUtensorMap km, vm;
    if (!page_map(&km, cfg, cache, cache->k, p.box) || !page_map(&vm, cfg, cache, cache->v, p.box)) return ENGRAM_ECUDA;
    constexpr int smem = rows::smem_bytes<DP>();
    static std::atomic<bool> attr_done[64];
    const auto kern = rows::rows_kernel<E, DP>;
    engram_status s = ensure_smem((const void *)kern, smem, attr_done);
    if (s != ENGRAM_OK) return s;
    s = launch_after(kern, dim3(p.runs * p.cluster), rows::NUM_THREADS, smem, p.cluster, st, "rows_kernel", km, vm, p);
    if (s != ENGRAM_OK || !shares.cut()) return s;
    return launch_after(rows::rows_join_kernel<E, DP, rows::ROWS>, dim3(p.runs - 1, rows::ROWS / 4), 128, 0, 1, st, "rows_join_kernel", p);
}

// Row blocks x kv heads of a batch at most.
static int64_t tile_items_most(const engram_attn_config *cfg, int64_t n_seqs, int64_t n_query) {
    const int64_t rows = n_query * (cfg->n_heads / cfg->n_kv_heads);
    const int64_t seqs = n_seqs < n_query ? n_seqs : n_query;
    return (rows / tile::ROWS + seqs) * cfg->n_kv_heads;
}
// Slots for partial results.  Nothing is split, none are needed and no join follows with six items a SM
// or more (the last round is at most a sixth of the time, and the parts cost about as much) or with at
// most six tiles of keys (a part costs about six).
static int64_t tile_slots(const engram_attn_config *cfg, const engram_kv_cache *cache, const engram_kv_batch *batch) {
    const int64_t n_seqs = batch->n_seqs, n_query = batch->n_query;
    if (keys_most(cfg, cache, batch) <= 6 * tile::KT) return 0;
    const int64_t least = (n_query * (cfg->n_heads / cfg->n_kv_heads) + tile::ROWS - 1) / tile::ROWS * cfg->n_kv_heads;
    if (least >= (int64_t)num_sms() * 6) return 0;
    return std::min<int64_t>((int64_t)num_sms() * tile::SLOTS_PER_SM,
                             tile_items_most(cfg, n_seqs, n_query) * tile::MAX_SPLIT);
}
static size_t tile_part_o_bytes(const engram_attn_config *cfg, int64_t slots) {
    return up256((size_t)slots * tile::ROWS * padded_dim(cfg) * sizeof(float));
}
static size_t tile_workspace_bytes(const engram_attn_config *cfg, const engram_kv_cache *cache, const engram_kv_batch *batch) {
    const int64_t slots = tile_slots(cfg, cache, batch);
    if (slots == 0) return 0;
    return tile_part_o_bytes(cfg, slots) + up256((size_t)slots * 2 * tile::ROWS * sizeof(float)) + 256;  // the plan's cut last
}

// Rows kernel or tile kernel: the one whose estimate, in us on this GPU, is less.  Both count the parts of
// sequences of the mean number of rows (the lengths are on the device): a segment of 16 rows costs 2.5 and
// 0.6 a 32 KB tile of keys, an item of 256 rows 3.7 and 1.6 a tile of 128 keys; whole rounds of them, or
// equal shares after a later start (split and joined).  Fitted to 197 measured pairs (8, 4 and 32 key/value
// heads, 1 to 40 sequences of 2 to 256 new tokens over 1 to 16,000): the choice costs 0.2 % over the better
// kernel in the mean and 15 % at worst.  Of them, 32 heads of 128 with 8 key/value heads, us rows kernel /
// tile kernel, new tokens over cached ones: 8 over 16,000 27 / 32, 16 42 / 33; 64 over 4,000 42 / 28; prompts
// of 64 7.4 / 9.0, 128 12.4 / 11.4, 256 25 / 13; 8 sequences of 4 over 16,000 90 / 119, of 8 over 2,000
// 28 / 32, of 16 44 / 32; 40 of 4 over 2,000 64 / 98, of 16 182 / 100.
static bool use_tiles(const engram_attn_config *cfg, const engram_kv_cache *cache, const engram_kv_batch *batch) {
    const double sms = num_sms();
    const int64_t seqs = std::min(batch->n_seqs, batch->n_query), rows = batch->n_query * (cfg->n_heads / cfg->n_kv_heads);
    const double mean = (double)rows / (double)seqs, parts = (double)seqs * cfg->n_kv_heads;
    const double segs = parts * ceil(mean / rows::ROWS), items = parts * ceil(mean / tile::ROWS);
    const double seg_us = 2.5 + 0.6 * (double)rows_tiles_most(cfg, cache, batch);
    const double item_us = 3.7 + 1.6 * (double)((keys_most(cfg, cache, batch) + tile::KT - 1) / tile::KT);
    const double rows_us = std::min(9.0 + segs * seg_us / sms, 3.5 + ceil(segs / sms) * seg_us);
    const double tile_us = tile_slots(cfg, cache, batch) > 0 ? 24.0 + items * item_us / sms : 4.0 + ceil(items / sms) * item_us;
    return tile_us < rows_us;
}

template <typename E, int DP>
static engram_status tile_launch(const engram_attn_config *cfg, const engram_kv_cache *cache,
                                 const engram_kv_batch *batch, const engram_heads *q, const engram_heads *out,
                                 float *lse, void *workspace, cudaStream_t st) {
    tile::Params p;
    memset(&p, 0, sizeof(p));
    const int64_t slots = tile_slots(cfg, cache, batch);
    p.b = device_batch(batch, cache);
    p.q = static_cast<const uint16_t *>(q->data);
    p.q_token_stride = q->token_stride;
    p.q_head_stride = q->head_stride;
    p.out = static_cast<uint16_t *>(out->data);
    p.out_token_stride = out->token_stride;
    p.out_head_stride = out->head_stride;
    p.lse = lse;
    p.values = ValuePages{static_cast<const uint16_t *>(cache->v), cache->page_stride, cache->token_stride, cache->head_stride};
    p.part_o = static_cast<float *>(workspace);
    p.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + tile_part_o_bytes(cfg, slots));
    p.n_heads = cfg->n_heads;
    p.n_kv_heads = cfg->n_kv_heads;
    p.group = cfg->n_heads / cfg->n_kv_heads;
    p.by_group = Divisor(p.group);
    p.by_heads = Divisor(cfg->n_kv_heads);
    p.head_dim = cfg->head_dim;
    p.window = cfg->window;
    p.box = gcd(cache->page_size, tile::KT);
    p.ctas = num_sms();
    p.max_slots = (int32_t)slots;
    p.cut = slots == 0 ? nullptr
                       : reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) +
                                                     tile_workspace_bytes(cfg, cache, batch) - 256);
    p.scale_log2 = cfg->scale * 1.4426950408889634f;
    CUtensorMap km, vm;
    if (!page_map(&km, cfg, cache, cache->k, p.box) || !page_map(&vm, cfg, cache, cache->v, p.box)) return ENGRAM_ECUDA;
    constexpr int smem = tile::smem_bytes<DP>();
    static std::atomic<bool> attr_done[64];
    const auto kern = tile::tile_kernel<E, DP, std::is_same<E, Bf16>::value>;
    engram_status s = ensure_smem((const void *)kern, smem, attr_done);
    if (s != ENGRAM_OK) return s;
    s = launch_after(kern, dim3(p.ctas), tile::NUM_THREADS, smem, 1, st, "tile_kernel", km, vm, p);
    if (s != ENGRAM_OK || slots == 0) return s;
    return launch_after(tile::tile_join_kernel<E, DP>, dim3(p.ctas * tile::JOIN_PER_SM), 128, 0, 1, st, "tile_join_kernel", p);
}

}  // namespace attn
}  // namespace engram

using namespace engram;

extern "C" engram_status engram_qk_norm_rope(const engram_attn_config *cfg, int64_t n_tokens, const engram_heads *q,
                                             const engram_heads *k, const int32_t *positions, const float *table,
                                             int64_t table_rows, const void *w_q, const void *w_k,
                                             const engram_heads *q_out, const engram_heads *k_out, void *stream) {
    using namespace engram::attn;
    if (check_attn_config(cfg) != ENGRAM_OK || n_tokens < 0 || n_tokens > INT32_MAX) return ENGRAM_EINVAL;
    if (n_tokens == 0 || (!q && !k)) return ENGRAM_OK;
    if ((q && (!view_ok(q) || !view_ok(q_out))) || (k && (!view_ok(k) || !view_ok(k_out)))) return ENGRAM_EINVAL;
    if (!aligned(w_q, 16) || !aligned(w_k, 16) || table_rows < 0) return ENGRAM_EINVAL;
    if (cfg->rope_dim > 0 && (!positions || !table || !aligned(positions, 4) || !aligned(table, 16))) return ENGRAM_EINVAL;
    HeadParams p;
    memset(&p, 0, sizeof(p));
    p.q = view(q);
    p.k = view(k);
    p.q_out = view(q ? q_out : nullptr);
    p.k_out = view(k ? k_out : nullptr);
    p.n_q = q ? cfg->n_heads : 0;
    p.n_k = k ? cfg->n_kv_heads : 0;
    p.w_q = static_cast<const uint16_t *>(w_q);
    p.w_k = static_cast<const uint16_t *>(w_k);
    p.positions = cfg->rope_dim > 0 ? positions : nullptr;
    p.table = table;
    p.table_rows = table_rows;
    p.n_tokens = n_tokens;
    return cfg->dtype == ENGRAM_BF16 ? head_launch<Bf16, false>(cfg, p, (cudaStream_t)stream)
                                     : head_launch<Fp16, false>(cfg, p, (cudaStream_t)stream);
}

extern "C" engram_status engram_kv_append(const engram_attn_config *cfg, const engram_kv_cache *cache,
                                          const engram_kv_batch *batch, const engram_heads *k, const engram_heads *v,
                                          const void *w_k, const float *table, int64_t table_rows,
                                          const engram_heads *q, const void *w_q, const engram_heads *q_out,
                                          void *stream) {
    using namespace engram::attn;
    if (check_attn_config(cfg) != ENGRAM_OK || check_batch(batch) != ENGRAM_OK) return ENGRAM_EINVAL;
    if (batch->n_query == 0) return ENGRAM_OK;
    if (check_cache(cfg, cache) != ENGRAM_OK || !view_ok(k) || !view_ok(v)) return ENGRAM_EINVAL;
    if (q && (!view_ok(q) || !view_ok(q_out))) return ENGRAM_EINVAL;
    if (!aligned(w_q, 16) || !aligned(w_k, 16) || table_rows < 0) return ENGRAM_EINVAL;
    if (cfg->rope_dim > 0 && (!table || !aligned(table, 16))) return ENGRAM_EINVAL;
    HeadParams p;
    memset(&p, 0, sizeof(p));
    p.q = view(q);
    p.k = view(k);
    p.v = view(v);
    p.q_out = view(q ? q_out : nullptr);
    p.n_q = q ? cfg->n_heads : 0;
    p.n_k = p.n_v = cfg->n_kv_heads;
    p.w_q = static_cast<const uint16_t *>(w_q);
    p.w_k = static_cast<const uint16_t *>(w_k);
    p.table = table;
    p.table_rows = table_rows;
    p.n_tokens = batch->n_query;
    p.k_pages = static_cast<uint16_t *>(cache->k);
    p.v_pages = static_cast<uint16_t *>(cache->v);
    p.page_stride = cache->page_stride;
    p.slot_stride = cache->token_stride;
    p.page_head_stride = cache->head_stride;
    p.batch = device_batch(batch, cache);
    p.by_page = Divisor(cache->page_size);
    return cfg->dtype == ENGRAM_BF16 ? head_launch<Bf16, true>(cfg, p, (cudaStream_t)stream)
                                     : head_launch<Fp16, true>(cfg, p, (cudaStream_t)stream);
}

namespace engram {
namespace attn {
static size_t workspace_bytes(const engram_attn_config *cfg, const engram_kv_cache *cache, const engram_kv_batch *batch) {
    if (use_tiles(cfg, cache, batch)) return tile_workspace_bytes(cfg, cache, batch);
    return rows_shares(cfg, cache, batch).cut() ? rows_workspace_bytes(cfg) : 0;
}
}  // namespace attn
}  // namespace engram

extern "C" size_t engram_paged_attention_workspace_bytes(const engram_attn_config *cfg, const engram_kv_cache *cache,
                                                         const engram_kv_batch *batch) {
    using namespace engram::attn;
    if (check_attn_config(cfg) != ENGRAM_OK || check_batch(batch) != ENGRAM_OK || batch->n_query == 0) return 0;
    if (check_cache(cfg, cache) != ENGRAM_OK) return 0;
    const engram_attn_config eff = effective(cfg, cache, batch);
    return workspace_bytes(&eff, cache, batch);
}

extern "C" engram_status engram_paged_attention(const engram_attn_config *cfg, const engram_kv_cache *cache,
                                                const engram_kv_batch *batch, const engram_heads *q,
                                                const engram_heads *out, float *lse, void *workspace,
                                                size_t workspace_bytes, void *stream) {
    using namespace engram::attn;
    if (check_attn_config(cfg) != ENGRAM_OK || check_batch(batch) != ENGRAM_OK) return ENGRAM_EINVAL;
    if (batch->n_query == 0) return ENGRAM_OK;
    if (check_cache(cfg, cache) != ENGRAM_OK || !view_ok(q) || !view_ok(out) || !aligned(lse, 4)) return ENGRAM_EINVAL;
    if (batch->n_query > INT32_MAX / cfg->n_heads) return ENGRAM_EINVAL;
    const engram_attn_config eff = effective(cfg, cache, batch);
    cfg = &eff;
    const size_t need = engram::attn::workspace_bytes(cfg, cache, batch);
    if (need > 0 && (!workspace || !aligned(workspace, 256))) return ENGRAM_EINVAL;
    if (workspace_bytes < need) return ENGRAM_ENOMEM;
    cudaStream_t st = (cudaStream_t)stream;
    const bool bf16 = cfg->dtype == ENGRAM_BF16;
    if (use_tiles(cfg, cache, batch)) {
        if (padded_dim(cfg) == 64)
            return bf16 ? tile_launch<Bf16, 64>(cfg, cache, batch, q, out, lse, workspace, st)
                        : tile_launch<Fp16, 64>(cfg, cache, batch, q, out, lse, workspace, st);
        return bf16 ? tile_launch<Bf16, 128>(cfg, cache, batch, q, out, lse, workspace, st)
                    : tile_launch<Fp16, 128>(cfg, cache, batch, q, out, lse, workspace, st);
    }
    if (padded_dim(cfg) == 64)
        return bf16 ? rows_launch<Bf16, 64>(cfg, cache, batch, q, out, lse, workspace, st)
                    : rows_launch<Fp16, 64>(cfg, cache, batch, q, out, lse, workspace, st);
    return bf16 ? rows_launch<Bf16, 128>(cfg, cache, batch, q, out, lse, workspace, st)
                : rows_launch<Fp16, 128>(cfg, cache, batch, q, out, lse, workspace, st);
}
