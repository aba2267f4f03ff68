// The serving step over the 8-bit cache (block tables from request lengths, the
// quantising append, attention over codes): C entry points, argument checks,
// tensor maps, launches.  A translation unit of its own beside the 16-bit
// step's, whose plans and joins it instantiates again.
#include "attn_host.cuh"
#include "attn_rows.cuh"
#include "attn_tile.cuh"

#include "append8.cuh"
#include "attn8_common.cuh"
#include "attn_rows8.cuh"
#include "attn_tile8.cuh"
#include "kv_plan.cuh"

namespace engram {
namespace attn {

cudaError_t take_error8(unsigned int *w) { return take_error_word(w); }

// What both calls over the 8-bit cache ask of the configuration and the cache.
static engram_status check_cache8(const engram_attn_config *cfg, const engram_kv_cache_q8 *c) {
    if (cfg->head_dim % 16) return ENGRAM_EINVAL;
    if (!c || !c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return ENGRAM_EINVAL;
    if (!c->k_scales || !c->v_scales || !aligned(c->k_scales, 4) || !aligned(c->v_scales, 4)) return ENGRAM_EINVAL;
    if (c->n_pages < 1 || c->n_pages > INT32_MAX) return ENGRAM_EINVAL;
    if (c->page_size < 16 || c->page_size > 65536 || c->page_size % 16) return ENGRAM_EINVAL;
    const int32_t b = c->block_tokens;
    if ((b != 16 && b != 32 && b != 64 && b != 128) || c->page_size % b) return ENGRAM_EINVAL;
    // strides positive (a size of one may still name any), so no value lies before the base
    for (int64_t s : {c->page_stride, c->token_stride, c->head_stride})
        if (s < 16 || s % 16 || s >= (INT64_C(1) << 40)) return ENGRAM_EINVAL;
    if (c->token_stride < cfg->head_dim || c->page_stride < cfg->head_dim) return ENGRAM_EINVAL;
    if (cfg->n_kv_heads > 1 && c->head_stride < cfg->head_dim) return ENGRAM_EINVAL;
    return ENGRAM_OK;
}

// --------------------------------------------------------------------- plan --

static engram_status check_plan(const engram_kv_plan_args *a) {
    if (!a || a->n_seqs < 0 || a->n_seqs > INT32_MAX || a->max_tokens < 0 || a->max_tokens > INT32_MAX) return ENGRAM_EINVAL;
    if (a->n_pages < 1 || a->n_pages > INT32_MAX) return ENGRAM_EINVAL;
    if (a->page_size < 16 || a->page_size > 65536 || a->page_size % 16) return ENGRAM_EINVAL;
    if (!a->seq_offsets || !aligned(a->seq_offsets, 8) || !a->counts || !aligned(a->counts, 4)) return ENGRAM_EINVAL;
    if (!a->free_pages || !aligned(a->free_pages, 4) || !a->n_free || !aligned(a->n_free, 4) || !a->n_free_out ||
        !aligned(a->n_free_out, 4))
        return ENGRAM_EINVAL;
    if (!aligned(a->positions, 4) || !aligned(a->slots, 8)) return ENGRAM_EINVAL;
    if (a->n_seqs == 0) return ENGRAM_OK;
    if (a->table_stride < 1 || a->table_stride > INT32_MAX || a->table_width < 0 || a->table_width > a->table_stride)
        return ENGRAM_EINVAL;
    if (!a->new_len || !aligned(a->new_len, 4) || !aligned(a->keep_len, 4) || !a->kv_len || !aligned(a->kv_len, 4) ||
        !a->kv_len_out || !aligned(a->kv_len_out, 4) || !a->block_table || !aligned(a->block_table, 4))
        return ENGRAM_EINVAL;
    return ENGRAM_OK;
}

// ------------------------------------------------------------------- append --

template <typename E, int LPH, bool INTERLEAVED, int THREADS>
static engram_status append8_launch_t(const Append8 &a, int64_t blocks, int threads, cudaStream_t st) {
    const int smem = a.block * a.h.rope_dim * (int)sizeof(float);
    const auto kern = append8_kernel<E, LPH, INTERLEAVED, THREADS>;
    static std::atomic<bool> attr_done[64];
    const engram_status s = ensure_smem((const void *)kern, THREADS / 32 * TOKENS_PER_WARP * 128 * (int)sizeof(float), attr_done);
    if (s != ENGRAM_OK) return s;
    return launch_after(kern, dim3((unsigned)blocks), threads, smem, 1, st, "append8_kernel", a);
}
template <typename E, int LPH>
static engram_status append8_launch(const engram_attn_config *cfg, Append8 &a, cudaStream_t st) {
    constexpr int per = 32 / LPH;
    const int warps = a.block / TOKENS_PER_WARP;
    const int64_t kv_blocks = a.units * 2 * ((a.n_kv + per - 1) / per);
    // The queries of many tokens go in a launch of their own: beside the keys' registers half as many of their warps
    // run (32,768 tokens of 32 + 8 heads 297 us in one launch).
    const bool apart = a.h.n_tokens * ((a.h.n_q + 3) / 4) >= (int64_t)num_sms() * 256;
    a.q_groups = apart ? 0 : (a.h.n_q + per - 1) / per;
    const int64_t blocks = kv_blocks + (a.h.n_tokens + warps - 1) / warps * a.q_groups;
    if (blocks > INT32_MAX) return ENGRAM_EINVAL;  // before the first launch
    if (apart) {
        HeadParams q = a.h;
        a.h.n_q = 0;
        const engram_status s = head_launch<E, true>(cfg, q, st);
        if (s != ENGRAM_OK) return s;
    }
    a.kv_blocks = (int32_t)kv_blocks;
    const bool pairs = cfg->rope_layout == ENGRAM_ROPE_INTERLEAVED;
    if (warps <= 8)
        return pairs ? append8_launch_t<E, LPH, true, 256>(a, blocks, warps * 32, st) : append8_launch_t<E, LPH, false, 256>(a, blocks, warps * 32, st);
    return pairs ? append8_launch_t<E, LPH, true, 512>(a, blocks, warps * 32, st) : append8_launch_t<E, LPH, false, 512>(a, blocks, warps * 32, st);
}

// ---------------------------------------------------------------- attention --

// A [page][head][token][D] view of K or V codes for TMA: boxes of the padded head (rows of 128 bytes, or 64) x
// `rows` tokens, swizzled over the row where asked; codes past head_dim read as zeros.
static bool page_map8(CUtensorMap *m, const engram_attn_config *cfg, const engram_kv_cache_q8 *c, void *base, int rows, bool swizzle) {
    auto enc = tensormap_encoder();
    if (!enc) return false;
    cuuint64_t dims[4] = {(cuuint64_t)cfg->head_dim, (cuuint64_t)c->page_size, (cuuint64_t)cfg->n_kv_heads,
                          (cuuint64_t)c->n_pages};
    cuuint64_t strides[3] = {(cuuint64_t)c->token_stride, (cuuint64_t)c->head_stride, (cuuint64_t)c->page_stride};
    cuuint32_t box[4] = {(cuuint32_t)padded_dim(cfg), (cuuint32_t)rows, 1, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : padded_dim(cfg) == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static Scales scales_of(const engram_kv_cache_q8 *c) {
    int log2 = 4;
    while ((1 << log2) < c->block_tokens) ++log2;
    return Scales{c->k_scales, c->v_scales, c->page_size / c->block_tokens, log2};
}

static size_t rows8_part_o_bytes(const engram_attn_config *cfg) {
    return up256((size_t)num_sms() * 2 * rows::ROWS8 * padded_dim(cfg) * sizeof(float));
}
static size_t rows8_workspace_bytes(const engram_attn_config *cfg) {
    return rows8_part_o_bytes(cfg) + up256((size_t)num_sms() * 2 * 2 * rows::ROWS8 * sizeof(float));
}

// Segments of the rows kernel (row tile x kv head) at most, and the tiles of 128 keys that the block table has
// room for (in a window's reach).
static int64_t rows8_segs_most(const engram_attn_config *cfg, const engram_kv_batch *batch) {
    const int64_t group = cfg->n_heads / cfg->n_kv_heads, seqs = std::min(batch->n_seqs, batch->n_query);
    return cfg->n_kv_heads * std::min(batch->n_query * ((group + rows::ROWS8 - 1) / rows::ROWS8),
                                      (batch->n_query * group + (rows::ROWS8 - 1) * seqs) / rows::ROWS8);
}
static int64_t rows8_tiles_most(const engram_attn_config *cfg, const engram_kv_cache_q8 *cache, const engram_kv_batch *batch) {
    return (keys_most(cfg, cache, batch) + rows::KT8 - 1) / rows::KT8;
}

// How a segment's tiles are shared out, and about how long that takes (us on this GPU): the least of
//   whole: no cut, no join; a round of segments over the SMs costs 2.9 and 0.61 a tile (64 values: 0.54), the first 2.4 more;
//   cluster of 8 or 4: a segment's tiles over that many CTAs, joined through distributed shared memory, one launch;
//     15 clusters of 8 and 36 of 4 run at once on this GPU's 152 SMs, as observed; beyond that some wait, so more
//     segments than sms / 10 and sms / 4 - 2 do not go this way;
//   cut: equal runs of tiles for every SM, then the join: 9.5, and 0.78 a tile.  Several sequences seldom have the room
//     that their tables give them; here alone that shortens the work, so it counts for less (unequal lengths make the
//     others wait for the longest).
// Measured, 32 / 8 heads of 128, us a call in a CUDA graph, cluster of 8 / of 4 / whole / cut:
//   1 sequence of 100 tokens 7.3 / 7.1 / 5.8 / 6.8, 1,000 7.3 / 7.7 / 9.8 / 9.1, 8,000 11.1 / 15.5 / 41 / 12.5, 32,000
//   25 / 43 / 153 / 18.8;  4 of 2,000 - / 9.1 / 14.7 / 11.3;  8 of 500 - / - / 8.0 / 9.9, 8,000 43 / 31;  64 of 100
//   16.5 / 19.4, 2,000 53 / 55, 8,000 169 / 164.
// Cut, the heads lie side by side (as many as divide them and leave hardly an SM out): the CTAs that share a page
// read it at the same time, which DRAM likes better than 128 bytes of every 1,024 (64 sequences of up to 16,384 tokens
// 173 us instead of 197).
struct Rows8Shares {
    int32_t cluster, whole, runs, side;
    double us;
    bool cut() const { return whole == 0 && runs > 1; }
};
static int32_t heads_aside(int n_kv_heads, int sms) {
    int32_t side = 1;
    for (int d = 2; d <= n_kv_heads && d <= 16; ++d)
        if (n_kv_heads % d == 0 && sms / d * d * 32 >= sms * 31) side = d;
    return side;
}
static Rows8Shares rows8_shares(const engram_attn_config *cfg, const engram_kv_cache_q8 *cache, const engram_kv_batch *batch) {
    const int64_t tiles = std::max<int64_t>(rows8_tiles_most(cfg, cache, batch), 1), segs = rows8_segs_most(cfg, batch);
    const int sms = num_sms();
    const double tile_us = padded_dim(cfg) == 64 ? 0.54 : 0.61, t = (double)tiles, g = (double)segs;
    Rows8Shares p = {1, (int32_t)std::min<int64_t>(tiles, INT32_MAX), sms, 1, 2.4 + ceil(g / sms) * (2.9 + tile_us * t)};
    for (int c = 8; c >= 4; c -= 4) {
        const double us = 6.7 + tile_us * t / c;
        if (segs <= (c == 8 ? sms / 10 : sms / 4 - 2) && us < p.us) p = {c, 1, (int32_t)segs, 1, us};
    }
    const double cut = 9.5 + (batch->n_seqs > 1 ? 0.85 : 1.0) * 0.78 * g * std::max(t, 1.5) / sms;
    if (cut < p.us) {
        p = {1, 0, sms, heads_aside(cfg->n_kv_heads, sms), cut};
        p.runs = sms / p.side;
    }
    return p;
}

template <typename E, int DP>
static engram_status rows8_launch(const engram_attn_config *cfg, const engram_kv_cache_q8 *cache,
                                  const engram_kv_batch *batch, const engram_heads *q, const engram_heads *out,
                                  float *lse, void *workspace, cudaStream_t st) {
    rows::Params8 a;
    memset(&a, 0, sizeof(a));
    rows::Params &p = a.r;
    p.b = device_batch(batch, cache);
    p.q = static_cast<const uint16_t *>(q->data);
    p.q_token_stride = q->token_stride;
    p.q_head_stride = q->head_stride;
    p.out = static_cast<uint16_t *>(out->data);
    p.out_token_stride = out->token_stride;
    p.out_head_stride = out->head_stride;
    p.lse = lse;
    p.part_o = static_cast<float *>(workspace);
    p.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + rows8_part_o_bytes(cfg));
    p.n_heads = cfg->n_heads;
    p.n_kv_heads = cfg->n_kv_heads;
    p.group = cfg->n_heads / cfg->n_kv_heads;
    p.by_group = Divisor(p.group);
    p.head_dim = cfg->head_dim;
    p.window = cfg->window;
    p.kt_log2 = rows::Cfg8<DP>::KT_LOG2;
    p.box = gcd(cache->page_size, rows::KT8);
    const Rows8Shares shares = rows8_shares(cfg, cache, batch);
    p.cluster = shares.cluster;
    p.whole = shares.whole;
    p.runs = shares.runs;
    p.side = shares.side;
    p.line_heads = cfg->n_kv_heads / shares.side;
    p.by_heads = Divisor(p.line_heads);
    p.scale_log2 = cfg->scale * 1.4426950408889634f;
    a.scales = scales_of(cache);
    a.by_page = Divisor(cache->page_size);
    a.codes = CodePages{static_cast<const uint8_t *>(cache->v), cache->page_stride, cache->token_stride, cache->head_stride};
    CUtensorMap km, vm;
    if (!page_map8(&km, cfg, cache, cache->k, p.box, true) || !page_map8(&vm, cfg, cache, cache->v, p.box, true)) return ENGRAM_ECUDA;
    constexpr int smem = rows::smem8_bytes<DP>();
    static std::atomic<bool> attr_done[64];
    const auto kern = rows::rows8_kernel<E, DP>;
    engram_status s = ensure_smem((const void *)kern, smem, attr_done);
    if (s != ENGRAM_OK) return s;
    s = launch_after(kern, dim3(p.runs * p.side * p.cluster), rows::NUM_THREADS8, smem, p.cluster, st, "rows8_kernel", km, vm, a);
    if (s != ENGRAM_OK || !shares.cut()) return s;
    return launch_after(rows::rows_join_kernel<E, DP, rows::ROWS8>, dim3((p.runs - 1) * p.side, rows::ROWS8 / 4), 128, 0, 1, st, "rows_join_kernel", p);
}

// Row blocks x kv heads of a batch at most, and the slots for partial results, as for the 16-bit cache.
static int64_t tile8_items_most(const engram_attn_config *cfg, int64_t n_seqs, int64_t n_query) {
    const int64_t rows = n_query * (cfg->n_heads / cfg->n_kv_heads);
    const int64_t seqs = n_seqs < n_query ? n_seqs : n_query;
    return (rows / tile::ROWS + seqs) * cfg->n_kv_heads;
}
static int64_t tile8_slots(const engram_attn_config *cfg, const engram_kv_cache_q8 *cache, const engram_kv_batch *batch) {
    const int64_t n_seqs = batch->n_seqs, n_query = batch->n_query;
    if (keys_most(cfg, cache, batch) <= 6 * tile::KT) return 0;
    const int64_t least = (n_query * (cfg->n_heads / cfg->n_kv_heads) + tile::ROWS - 1) / tile::ROWS * cfg->n_kv_heads;
    if (least >= (int64_t)num_sms() * 6) return 0;
    return std::min<int64_t>((int64_t)num_sms() * tile::SLOTS_PER_SM, tile8_items_most(cfg, n_seqs, n_query) * tile::MAX_SPLIT);
}
static size_t tile8_part_o_bytes(const engram_attn_config *cfg, int64_t slots) {
    return up256((size_t)slots * tile::ROWS * padded_dim(cfg) * sizeof(float));
}
// The parts' results and the plan's cut, the latter at the end.
static size_t tile8_parts_bytes(const engram_attn_config *cfg, int64_t slots) {
    return slots == 0 ? 0 : tile8_part_o_bytes(cfg, slots) + up256((size_t)slots * 2 * tile::ROWS * sizeof(float)) + 256;
}

// Items of the tile kernel at most, about.
static double tile8_items(const engram_attn_config *cfg, const engram_kv_batch *batch) {
    const double seqs = (double)std::min(batch->n_seqs, batch->n_query), rows = (double)batch->n_query * (cfg->n_heads / cfg->n_kv_heads);
    return seqs * cfg->n_kv_heads * ceil(rows / seqs / tile::ROWS);
}

// Bytes for the sequences' codes as 16-bit tiles, made before the tile kernel; 0: its own warps convert each tile that it
// meets.  Opened, a tile of an item takes 0.7 us less (64 values: 0.45); opening costs 8 us and 0.16 (0.08) a thousand
// keys and heads.  Measured, us opened / not, 32 / 8 heads of 128, new tokens over cached ones: a prompt of 8,192 415 / 541,
// 1,024 33 / 32; 2,048 over 63,488 1,515 / 2,078; 512 over 16,000 157 / 167, 64 74 / 46; 8 sequences of 256 over 4,000
// 186 / 178; 8 prompts of up to 4,096, a window of 1,000 304 / 351, of 128 184 / 172; 64 values, a prompt of 8,192 335 / 430.
// Keys are counted by the table's width: a prompt of 1,024 in a table with room for 131,072 opens (45 us, 34 in a tight one).
// Up to 1 GiB: 4 bytes a key's value for the table's room of every sequence.
constexpr int64_t OPEN_MOST = 1ll << 30;
static int64_t opened_keys(const engram_kv_cache_q8 *cache, const engram_kv_batch *batch) {
    return (table_width(batch) * cache->page_size + tile::KT - 1) / tile::KT * tile::KT + tile::KT;
}
static size_t opened_bytes(const engram_attn_config *cfg, const engram_kv_cache_q8 *cache, const engram_kv_batch *batch) {
    const int64_t keys = opened_keys(cache, batch);
    if (keys > OPEN_MOST / 256) return 0;
    const bool narrow = padded_dim(cfg) == 64;
    const int64_t one = (narrow ? tile::opened_bytes<64>(keys) : tile::opened_bytes<128>(keys)) * cfg->n_kv_heads;
    if (one > OPEN_MOST || batch->n_seqs > OPEN_MOST / one) return 0;
    const double seqs = (double)std::min(batch->n_seqs, batch->n_query), thousands = (double)keys * seqs * cfg->n_kv_heads / 1000;
    const double reach = std::min((double)keys_most(cfg, cache, batch),
                                  std::max((double)(table_width(batch) * cache->page_size) - batch->n_query / seqs / 2, 1.0));
    const double saved = tile8_items(cfg, batch) * reach / tile::KT * (narrow ? 0.45 : 0.7) / num_sms();
    return saved > 8 + thousands * (narrow ? 0.08 : 0.16) ? up256((size_t)(one * batch->n_seqs)) : 0;
}
static size_t tile8_workspace_bytes(const engram_attn_config *cfg, const engram_kv_cache_q8 *cache, const engram_kv_batch *batch) {
    return tile8_parts_bytes(cfg, tile8_slots(cfg, cache, batch)) + opened_bytes(cfg, cache, batch);
}

// Rows kernel or tile kernel: the one whose estimate is less.  An item of 256 rows costs 3.2 us and 2.2 a tile of 128
// keys; whole rounds of them, or equal shares after a later start (split and joined).  Fitted to 545 measured pairs
// (32 / 8 and 16 / 16 heads of 128, 32 / 4 of 64; 1 to 40 sequences of 1 to 256 new tokens over 1 to 16,000): the
// choice costs 0.2 % over the better kernel in the mean and 25 % at worst.  Of them, 32 / 8 heads of 128, us rows kernel /
// tile kernel, new tokens over cached ones: 8 sequences of 8 over 8,000 78 / 98; 40 of 16 prompts 61 / 21, 8 over 2,000
// 107 / 128.
static bool use_tiles8(const engram_attn_config *cfg, const engram_kv_cache_q8 *cache, const engram_kv_batch *batch) {
    const double sms = num_sms(), items = tile8_items(cfg, batch);
    const double item_us = 3.2 + 2.2 * (double)((keys_most(cfg, cache, batch) + tile::KT - 1) / tile::KT);
    const double tile_us = tile8_slots(cfg, cache, batch) > 0 ? 28.8 + items * item_us / sms : 5.2 + ceil(items / sms) * item_us;
    return tile_us < rows8_shares(cfg, cache, batch).us;
}

template <typename E, int DP, bool OPEN>
static engram_status tile8_run(const CUtensorMap &km, const CUtensorMap &vm, const tile::Params8 &a, cudaStream_t st) {
    constexpr int smem = tile::smem8_bytes<DP, OPEN>();
    static std::atomic<bool> attr_done[64];
    const auto kern = tile::tile8_kernel<E, DP, OPEN>;
    const engram_status s = ensure_smem((const void *)kern, smem, attr_done);
    if (s != ENGRAM_OK) return s;
    return launch_after(kern, dim3(a.t.ctas), OPEN ? tile::NUM_THREADS : tile::NUM_THREADS8, smem, 1, st, "tile8_kernel", km, vm, a);
}

template <typename E, int DP>
static engram_status tile8_launch(const engram_attn_config *cfg, const engram_kv_cache_q8 *cache,
                                  const engram_kv_batch *batch, const engram_heads *q, const engram_heads *out,
                                  float *lse, void *workspace, cudaStream_t st) {
    tile::Params8 a;
    memset(&a, 0, sizeof(a));
    tile::Params &p = a.t;
    const int64_t slots = tile8_slots(cfg, cache, batch);
    p.b = device_batch(batch, cache);
    p.q = static_cast<const uint16_t *>(q->data);
    p.q_token_stride = q->token_stride;
    p.q_head_stride = q->head_stride;
    p.out = static_cast<uint16_t *>(out->data);
    p.out_token_stride = out->token_stride;
    p.out_head_stride = out->head_stride;
    p.lse = lse;
    p.part_o = static_cast<float *>(workspace);
    p.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + tile8_part_o_bytes(cfg, slots));
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
                       : reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) + tile8_parts_bytes(cfg, slots) - 256);
    p.scale_log2 = cfg->scale * 1.4426950408889634f;
    a.scales = scales_of(cache);
    a.by_page = Divisor(cache->page_size);
    a.codes = CodePages{static_cast<const uint8_t *>(cache->v), cache->page_stride, cache->token_stride, cache->head_stride};
    CUtensorMap km, vm;
    if (!page_map8(&km, cfg, cache, cache->k, p.box, false) || !page_map8(&vm, cfg, cache, cache->v, p.box, false))
        return ENGRAM_ECUDA;
    engram_status s;
    if (opened_bytes(cfg, cache, batch) > 0) {
        tile::OpenParams o;
        memset(&o, 0, sizeof(o));
        o.b = p.b;
        o.k = static_cast<const uint8_t *>(cache->k);
        o.v = static_cast<const uint8_t *>(cache->v);
        o.page_stride = cache->page_stride;
        o.slot_stride = cache->token_stride;
        o.head_stride = cache->head_stride;
        o.scales = a.scales;
        o.by_page = a.by_page;
        o.opened = a.opened = tile::Opened{static_cast<uint8_t *>(workspace) + tile8_parts_bytes(cfg, slots), opened_keys(cache, batch)};
        o.tiles = (int32_t)(o.opened.keys / tile::KT);
        o.units = batch->n_seqs * o.tiles * cfg->n_kv_heads * 2;
        o.n_kv_heads = cfg->n_kv_heads;
        o.head_dim = cfg->head_dim;
        o.window = cfg->window;
        o.scale_log2 = p.scale_log2;
        s = launch_after(tile::open_kernel<E, DP>, dim3((unsigned)std::min<int64_t>(o.units, (int64_t)num_sms() * tile::OPEN_PER_SM)),
                         tile::OPEN_THREADS, 0, 1, st, "open_kernel", o);
        if (s == ENGRAM_OK) s = tile8_run<E, DP, true>(km, vm, a, st);
    } else {
        s = tile8_run<E, DP, false>(km, vm, a, st);
    }
    if (s != ENGRAM_OK || slots == 0) return s;
    return launch_after(tile::tile_join_kernel<E, DP>, dim3(p.ctas * tile::JOIN_PER_SM), 128, 0, 1, st, "tile_join_kernel", p);
}

static size_t workspace_bytes8(const engram_attn_config *cfg, const engram_kv_cache_q8 *cache, const engram_kv_batch *batch) {
    if (use_tiles8(cfg, cache, batch)) return tile8_workspace_bytes(cfg, cache, batch);
    return rows8_shares(cfg, cache, batch).cut() ? rows8_workspace_bytes(cfg) : 0;
}

}  // namespace attn
}  // namespace engram

using namespace engram;

extern "C" engram_status engram_kv_plan(const engram_kv_plan_args *a, void *stream) {
    using namespace engram::attn;
    if (check_plan(a) != ENGRAM_OK) return ENGRAM_EINVAL;
    plan::Params p;
    memset(&p, 0, sizeof(p));
    p.new_len = a->new_len;
    p.keep_len = a->keep_len;
    p.kv_len = a->kv_len;
    p.kv_len_out = a->kv_len_out;
    p.table = a->block_table;
    p.table_stride = a->table_stride;
    p.table_width = a->table_width > 0 ? a->table_width : a->table_stride;
    p.free_pages = a->free_pages;
    p.n_free = a->n_free;
    p.n_free_out = a->n_free_out;
    p.offs = a->seq_offsets;
    p.positions = a->positions;
    p.slots = a->slots;
    p.counts = a->counts;
    p.n_seqs = a->n_seqs;
    p.max_tokens = a->max_tokens;
    p.n_pages = a->n_pages;
    p.page_size = a->page_size;
    p.by_page = Divisor(a->page_size);
    p.maps = a->max_tokens <= 4096;
    cudaStream_t st = (cudaStream_t)stream;
    // 256 threads where requests and pages to take are few (a decode step 2.9 us, 4.2 with 1,024), else 1,024
    const engram_status s = p.n_seqs <= 256 && p.max_tokens / p.page_size <= 1024 ? launch_after(plan::plan_kernel<256>, dim3(1), 256, 0, 1, st, "plan_kernel", p)
                                            : launch_after(plan::plan_kernel<plan::MOST>, dim3(1), plan::MOST, 0, 1, st, "plan_kernel", p);
    if (s != ENGRAM_OK || p.maps || (!p.positions && !p.slots)) return s;
    const int64_t warps = p.max_tokens / plan::SPAN + p.n_seqs + 1;
    return launch_after(plan::map_kernel, dim3((unsigned)((warps + 7) / 8)), 256, 0, 1, st, "map_kernel", p);
}

extern "C" engram_status engram_kv_append_q8(const engram_attn_config *cfg, const engram_kv_cache_q8 *cache,
                                             const engram_kv_batch *batch, const engram_heads *k, const engram_heads *v,
                                             const void *w_k, const float *table, int64_t table_rows,
                                             const engram_heads *q, const void *w_q, const engram_heads *q_out,
                                             void *stream) {
    using namespace engram::attn;
    if (check_attn_config(cfg) != ENGRAM_OK || check_batch(batch) != ENGRAM_OK) return ENGRAM_EINVAL;
    if (batch->n_query == 0) return ENGRAM_OK;
    if (check_cache8(cfg, cache) != ENGRAM_OK || !view_ok(k) || !view_ok(v)) return ENGRAM_EINVAL;
    if (q && (!view_ok(q) || !view_ok(q_out))) return ENGRAM_EINVAL;
    if (!aligned(w_q, 16) || !aligned(w_k, 16) || table_rows < 0) return ENGRAM_EINVAL;
    if (cfg->rope_dim > 0 && (!table || !aligned(table, 16))) return ENGRAM_EINVAL;
    Append8 a;
    memset(&a, 0, sizeof(a));
    HeadParams &p = a.h;
    p.q = view(q);
    p.k = view(k);
    p.v = view(v);
    p.q_out = view(q ? q_out : nullptr);
    p.n_q = q ? cfg->n_heads : 0;  // keys and values go their own way
    p.w_q = static_cast<const uint16_t *>(w_q);
    p.w_k = static_cast<const uint16_t *>(w_k);
    p.table = table;
    p.table_rows = table_rows;
    p.n_tokens = batch->n_query;
    p.head_dim = cfg->head_dim;
    p.rope_dim = cfg->rope_dim;
    p.eps = cfg->norm_eps;
    p.inv_dim = 1.f / (float)cfg->head_dim;
    p.batch = device_batch(batch, cache);
    p.by_page = Divisor(cache->page_size);
    a.k_pages = static_cast<uint8_t *>(cache->k);
    a.v_pages = static_cast<uint8_t *>(cache->v);
    a.k_scales = cache->k_scales;
    a.v_scales = cache->v_scales;
    a.page_stride = cache->page_stride;
    a.slot_stride = cache->token_stride;
    a.head_stride = cache->head_stride;
    a.n_kv = cfg->n_kv_heads;
    a.block = cache->block_tokens;
    a.per_page = cache->page_size / cache->block_tokens;
    a.units = std::min(batch->n_query / a.block + 2 * batch->n_seqs, batch->n_query);
    cudaStream_t st = (cudaStream_t)stream;
    if (cfg->head_dim <= 64)
        return cfg->dtype == ENGRAM_BF16 ? append8_launch<Bf16, 4>(cfg, a, st) : append8_launch<Fp16, 4>(cfg, a, st);
    return cfg->dtype == ENGRAM_BF16 ? append8_launch<Bf16, 8>(cfg, a, st) : append8_launch<Fp16, 8>(cfg, a, st);
}

extern "C" size_t engram_paged_attention_q8_workspace_bytes(const engram_attn_config *cfg, const engram_kv_cache_q8 *cache,
                                                            const engram_kv_batch *batch) {
    using namespace engram::attn;
    if (check_attn_config(cfg) != ENGRAM_OK || check_batch(batch) != ENGRAM_OK || batch->n_query == 0) return 0;
    if (check_cache8(cfg, cache) != ENGRAM_OK) return 0;
    const engram_attn_config eff = effective(cfg, cache, batch);
    return workspace_bytes8(&eff, cache, batch);
}

extern "C" engram_status engram_paged_attention_q8(const engram_attn_config *cfg, const engram_kv_cache_q8 *cache,
                                                   const engram_kv_batch *batch, const engram_heads *q,
                                                   const engram_heads *out, float *lse, void *workspace,
                                                   size_t workspace_bytes, void *stream) {
    using namespace engram::attn;
    if (check_attn_config(cfg) != ENGRAM_OK || check_batch(batch) != ENGRAM_OK) return ENGRAM_EINVAL;
    if (batch->n_query == 0) return ENGRAM_OK;
    if (check_cache8(cfg, cache) != ENGRAM_OK || !view_ok(q) || !view_ok(out) || !aligned(lse, 4)) return ENGRAM_EINVAL;
    if (batch->n_query > INT32_MAX / cfg->n_heads) return ENGRAM_EINVAL;
    const engram_attn_config eff = effective(cfg, cache, batch);
    cfg = &eff;
    const size_t need = workspace_bytes8(cfg, cache, batch);
    if (need > 0 && (!workspace || !aligned(workspace, 256))) return ENGRAM_EINVAL;
    if (workspace_bytes < need) return ENGRAM_ENOMEM;
    cudaStream_t st = (cudaStream_t)stream;
    const bool bf16 = cfg->dtype == ENGRAM_BF16;
    if (use_tiles8(cfg, cache, batch)) {
        if (padded_dim(cfg) == 64)
            return bf16 ? tile8_launch<Bf16, 64>(cfg, cache, batch, q, out, lse, workspace, st)
                        : tile8_launch<Fp16, 64>(cfg, cache, batch, q, out, lse, workspace, st);
        return bf16 ? tile8_launch<Bf16, 128>(cfg, cache, batch, q, out, lse, workspace, st)
                    : tile8_launch<Fp16, 128>(cfg, cache, batch, q, out, lse, workspace, st);
    }
    if (padded_dim(cfg) == 64)
        return bf16 ? rows8_launch<Bf16, 64>(cfg, cache, batch, q, out, lse, workspace, st)
                    : rows8_launch<Fp16, 64>(cfg, cache, batch, q, out, lse, workspace, st);
    return bf16 ? rows8_launch<Bf16, 128>(cfg, cache, batch, q, out, lse, workspace, st)
                : rows8_launch<Fp16, 128>(cfg, cache, batch, q, out, lse, workspace, st);
}
