// Paged attention for many query rows per key/value head (prompts, chunks):
// the same sum as the rows kernel,
//   out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),  s_j = scale * q.k_j,
// with both products on the tcgen05 tensor cores.
//
// Bound: by the count of operations the tensor pipe (4 * 128 * 128 * D flop per
// 128 x 128 tile); measured, the softmax's instructions beside it: a pair of row
// tiles takes about 3,400 cycles of an SM at 128 values and 3,000 at 64, its
// products 2,048 and 1,290.  A prompt of 8,192 tokens, 32 / 8 heads: 359 us at
// 128 values (1,530 TFLOP/s, 79 % of the burst rate; 384 us in a long run, at
// 1,945 instead of 2,070 MHz under the power cap), 318 us at 64 (866 TFLOP/s).
//
// An item is 256 query rows (the pairs (token, query head of the group),
// consecutive: all heads that share a key/value head share its tiles) as two
// 128-row tiles, against a run of 128-key tiles.  Per CTA (one per SM,
// persistent over items):
//   warps 0-3, 4-7  one softmax warpgroup per row tile, a row per thread: the
//                   row's 128 scores come from TMEM into registers, its
//                   maximum and sum need no exchange; weights go back to
//                   TMEM as 16-bit pairs over the scores they came from (up
//                   to 64 values: beside them).  At an item's end the rows
//                   change hands in shared memory and leave in 128-byte pieces.
//   warps 8, 11     issue the products of a row tile each: S = Q K^T (shared x
//                   shared memory), O += P V (TMEM x shared memory).  While one tile's
//                   softmax runs, the other tile's products do.
//   warp 9          TMA: K and V tiles in turn into a ring (4 stages of 32 KB,
//                   8 of 16 KB up to 64 values).
//   warp 10         finds the CTA's next items and hands them to the others.
// TMEM: S0 | S1 | O0 | O1, 128 columns each (512 in all at 128 values).
// What runs once an item or less is kept in loops and 32 bits: with few tiles
// an item the instruction cache binds (kernel code of 216 KB: a window of 128
// keys over 8 prompts 152 us; 169 KB: 135; 150 KB: 132).
//
// The running maximum moves only when a row's new maximum exceeds it by
// 2^E::RESCALE (then O and the sum are scaled): weights stay below 2^8 in bf16
// and, lifted, 2^15 in fp16, inside the types, and most tiles need no pass over
// O.  O is complete up to the tile before whenever new scores arrive (one
// in-order MMA queue; APART: when pv_done says so), so the softmax warps scale
// it themselves.  (A lagging maximum and two row tiles in turn are published
// techniques; the latter: Shah et al., 2024, arXiv 2407.08608.)
//
// Few items are split along the keys (by the plan below) and leave partial
// (m, l, O) for tile_join_kernel.
#pragma once

namespace engram {
namespace attn {
namespace tile {

constexpr int MT = 128;               // rows per tile (TMEM lanes)
constexpr int ROWS = 2 * MT;          // rows per item
constexpr int KT = 128;               // keys per tile
constexpr int NUM_THREADS = 384;
constexpr int CHUNKS = 64;            // the plan's prefix sums: sequences in this many chunks
constexpr int P_PARTS = 2;            // a tile's weights are handed over in this many parts
constexpr int MAX_SPLIT = 152;
constexpr int SLOTS_PER_SM = 8;       // workspace for partial results
// The join's blocks of an SM, all resident at 80 registers: 8 came in two waves (69 us instead of 70.5 for
// a mixed step), 8 at 64 registers spill (78).
constexpr int JOIN_PER_SM = 6;

// How many parts the longest item is cut into at most; the plan picks one.
constexpr int N_CAND = 16;
__device__ const int kSplits[N_CAND] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 16, 24, 38, 64, 96, 152};

template <int DP>
struct Cfg {
    static constexpr int STAGE_BYTES = KT * DP * 2;  // K or V of a tile
    // 128 values: 4 leave room for the rows on their way out; a fifth stage was worth nothing (a chunk of
    // 2,048 over 63,488 tokens 1,550 us with either).
    static constexpr int STAGES = DP == 128 ? 4 : 8;
    static constexpr int Q_BYTES = MT * DP * 2;      // one row tile
    static constexpr int SWAP_BYTES = 8 * 32 * 128;  // the softmax warps' rows on their way out, 128 bytes of each
    static constexpr int O_COL = 256;                // TMEM: scores in columns 0..255, then the outputs
    static constexpr int TMEM_COLS = 512;
    // Up to 64 values TMEM has room for the weights beside the scores: the next scores are then
    // computed while a tile's weights are.  Weights over the scores there: 7 sequences of 440 new
    // tokens over 8,001 294 us instead of 283, one of 4,096 over 28,672 1,294 instead of 1,234 (32/4
    // heads of 64).  With 128 values O takes the columns that this needs.
    static constexpr bool APART = DP == 64;
    static constexpr int P_COL = APART ? O_COL + 2 * DP : 0;  // weights: 64 columns a row tile, or over the scores
};

struct PlanShared {
    int64_t items[CHUNKS + 1];   // items before each chunk of sequences
    int64_t parts[CHUNKS + 1];   // ... and among them the parts of split ones (workspace slots)
    unsigned long long cand_items[N_CAND], cand_parts[N_CAND];
    unsigned long long work;
    int max_tiles;
    int cut;                     // tiles per part at most
};

struct Item {
    int64_t s;           // sequence
    int64_t slot;        // workspace slot of this part (split items)
    Seq q;
    int32_t head, r0, n_rows, pos0;  // n_rows 0: no more items
    int32_t lo, hi;      // keys in reach of any row
    int32_t key0, n;     // this part's first key and tiles
    int32_t part, splits;
    int32_t full_lo, full_hi;  // keys in reach of every row
    int32_t bad_lo, bad_hi;    // this part's tiles in which infinities or NaN were cleared
};
constexpr int ITEMS = 4;  // items found ahead

template <int DP>
struct Shared {
    uint64_t kv_full[Cfg<DP>::STAGES];
    uint64_t kv_empty[Cfg<DP>::STAGES];
    uint64_t q_full[2];
    uint64_t s_full[2];
    uint64_t p_ready[2][P_PARTS];
    uint64_t s_free[2];   // APART: the scores have been read
    uint64_t pv_done[2];  // APART: the weights have been used, O is up to date
    uint64_t o_full[2];
    uint64_t turn[2];
    uint64_t drained[2];
    uint64_t item_full[ITEMS];
    uint64_t item_empty[ITEMS];
    Item items[ITEMS];
    uint32_t tmem_base;
    int abort;
    PlanShared plan;
};

template <int DP>
constexpr int smem_bytes() {
    return 2 * Cfg<DP>::Q_BYTES + Cfg<DP>::STAGES * Cfg<DP>::STAGE_BYTES + Cfg<DP>::SWAP_BYTES + (int)sizeof(Shared<DP>);
}
static_assert(smem_bytes<128>() <= 232448, "tile kernel shared memory over the per-CTA limit");

struct Params {
    Batch b;
    const uint16_t *q;
    int64_t q_token_stride, q_head_stride;
    uint16_t *out;
    int64_t out_token_stride, out_head_stride;
    float *lse;
    ValuePages values;
    float *part_o;      // [slots][ROWS][DP]
    float *part_ml;     // [slots][2][ROWS]
    int32_t n_heads, n_kv_heads, group, head_dim;
    Divisor by_group, by_heads;  // the query heads of a kv head; the kv heads
    int32_t window;
    int32_t box;        // tokens per TMA box: gcd(page_size, KT)
    int32_t ctas;
    int32_t max_slots;  // 0: nothing is split
    int32_t *cut;       // the plan's cut, for the join
    float scale_log2;
};

// ------------------------------------------------------------------- plan ----

// A sequence's share: row blocks, the most key tiles any of them reaches, and
// about how many they reach on average.
struct Share {
    int64_t segs;    // row blocks x kv heads
    int32_t blocks;
    int32_t tiles;
    int32_t mean;
};
__device__ __forceinline__ Share share(const Params &p, const Seq &q) {
    Share r;
    r.blocks = (int32_t)(((int64_t)q.q_len * p.group + ROWS - 1) / ROWS);
    r.segs = (int64_t)r.blocks * p.n_kv_heads;
    int32_t n = (q.kv + KT - 1) / KT;
    if (p.window > 0) {
        const int64_t reach = (int64_t)p.window + p.by_group.quotient(ROWS - 2) + 1;
        const int64_t w = (reach + p.box + KT - 2) / KT;
        if (w < n) n = (int32_t)w;
    }
    const int32_t first = q.kv - q.q_len > 0 ? q.kv - q.q_len : 0;
    const int32_t mean = (int32_t)(((int64_t)q.kv + first) / 2 / KT) + 1;
    r.tiles = n;
    r.mean = mean < n ? mean : n;
    return r;
}
__device__ __forceinline__ int32_t splits_of(int32_t tiles, int32_t cut) {
    return tiles > cut ? (tiles + cut - 1) / cut : 1;
}

// The candidate that takes the least time, by a warp: lane c < N_CAND with the
// items and parts of candidate c and its cut.  Times are in tiles: equal items
// go in rounds; items of unequal size fill each other's gaps (half the longest
// is left over).  An item costs about two tiles beside its own, a part about
// six (its partial result is written, read again and joined; taken for five,
// a mixed step of 9 sequences was split: 69 us instead of 60).
__device__ __forceinline__ int32_t best_cut(const Params &p, float items, float parts, float work, int32_t cut_c) {
    const int lane = threadIdx.x & 31;
    float best = INFINITY;
    int32_t cut = INT32_MAX;
    if (lane < N_CAND) {
        const float g = (float)p.ctas, rounds = ceilf(items / g);
        const float span = items <= g ? (float)cut_c : (work > 0.85f * items * cut_c ? rounds * cut_c : work / g + 0.5f * cut_c);
        const bool whole = kSplits[lane] == 1;
        if (whole || parts <= (float)p.max_slots) best = span + rounds * (whole ? 2.f : 6.f);
        cut = whole ? INT32_MAX : cut_c;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {  // of equals the first candidate (lower lane)
        const float ob = __shfl_down_sync(0xffffffffu, best, o);
        const int32_t oc = __shfl_down_sync(0xffffffffu, cut, o);
        if (ob < best) {
            best = ob;
            cut = oc;
        }
    }
    return __shfl_sync(0xffffffffu, cut, 0);
}

// The sums over the chunks of sequences, by all threads of a block of at least
// CHUNKS threads: a[c + 1] and b[c + 1] from per(s), a pair of counts.
template <typename F>
__device__ __forceinline__ void chunk_sums(const Params &p, int64_t *a, int64_t *b, const F &per) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t size = (p.b.n_seqs + CHUNKS - 1) / CHUNKS;
    if (tid < CHUNKS) {
        const int64_t s0 = tid * size, s1 = s0 + size < p.b.n_seqs ? s0 + size : p.b.n_seqs;
        int64_t x = 0, y = 0;
        for (int64_t s = s0; s < s1; ++s) per(s, x, y);
        a[tid + 1] = x;
        b[tid + 1] = y;
        if (tid == 0) a[0] = b[0] = 0;
    }
    __syncthreads();
    if (tid < 64) {  // inclusive, 32 at a time; a warp for each array
        int64_t *v = tid < 32 ? a : b;
        int64_t run = 0;
        for (int c = 0; c < CHUNKS; c += 32) {
            int64_t x = v[c + lane + 1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t u = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += u;
            }
            v[c + lane + 1] = run + x;
            run += __shfl_sync(0xffffffffu, x, 31);
        }
    }
    __syncthreads();
}

// The chunk whose range of v (sums over the chunks) holds x.
__device__ __forceinline__ int find_chunk(const int64_t *v, int64_t x) {
    int lo = 0, hi = CHUNKS;  // v[lo] <= x < v[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// All threads of a block of NT threads, into sh: the cut, and the items before
// each chunk of sequences.
template <int NT>
__device__ void make_plan(const Params &p, int64_t base, PlanShared *sh) {
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid < N_CAND) sh->cand_items[tid] = sh->cand_parts[tid] = 0;
    if (tid == 0) {
        sh->work = 0;
        sh->max_tiles = 1;
        sh->cut = INT32_MAX;
    }
    __syncthreads();
    if (p.max_slots > 0) {
        int64_t work = 0;
        int32_t most = 1;
        for (int64_t s = tid; s < p.b.n_seqs; s += NT) {
            const Share h = share(p, load_seq(p.b, s, base));
            work += h.segs * h.mean;
            if (h.segs > 0 && h.tiles > most) most = h.tiles;
        }
        if (work) {
            atomicAdd(&sh->work, (unsigned long long)work);
            atomicMax(&sh->max_tiles, most);
        }
        __syncthreads();
        // a candidate per lane, two sequences per warp and round
        static_assert(N_CAND == 16, "a half warp of candidates");
        const int c = lane & 15;
        const int32_t max_tiles = sh->max_tiles, cut_c = (max_tiles + kSplits[c] - 1) / kSplits[c];
        unsigned long long items = 0, parts = 0;
        for (int64_t s = (tid >> 4); s < p.b.n_seqs; s += NT / 16) {
            const Share h = share(p, load_seq(p.b, s, base));
            const int32_t n = splits_of(h.tiles, cut_c);
            items += h.segs * n;
            if (n > 1) parts += h.segs * n;
        }
        if (items) {
            atomicAdd(&sh->cand_items[c], items);
            atomicAdd(&sh->cand_parts[c], parts);
        }
        __syncthreads();
        if (tid < 32) {
            const int32_t cut = best_cut(p, (float)sh->cand_items[c], (float)sh->cand_parts[c], (float)sh->work, cut_c);
            if (lane == 0) sh->cut = cut;
        }
        __syncthreads();
    }
    const int32_t cut = sh->cut;
    chunk_sums(p, sh->items, sh->parts, [&](int64_t s, int64_t &n, int64_t &parts) {
        const Share h = share(p, load_seq(p.b, s, base));
        const int32_t k = splits_of(h.tiles, cut);
        n += h.segs * k;
        if (k > 1) parts += h.segs * k;
    });
}

// Rows and keys of segment seg = block * n_kv_heads + head of sequence it.q;
// part it.part of it.splits.
__device__ __forceinline__ void place(const Params &p, Item &it, int32_t seg) {
    const int32_t block = p.by_heads.quotient(seg);
    it.head = seg - block * p.n_kv_heads;
    it.r0 = block * ROWS;
    const int32_t left = it.q.q_len * p.group - it.r0;
    it.n_rows = left < ROWS ? left : ROWS;
    it.pos0 = it.q.kv - it.q.q_len;
    const int32_t first = it.pos0 + p.by_group.quotient(it.r0), last = it.pos0 + p.by_group.quotient(it.r0 + it.n_rows - 1);
    it.hi = last + 1 > 0 ? last + 1 : 0;
    it.lo = first_seen(first, p.window);
    it.full_hi = first + 1;
    it.full_lo = first_seen(last, p.window);
    it.bad_lo = INT32_MAX;
    it.bad_hi = -1;
    // Tiles start at the box of the first key: with a window, on multiples of KT an item would meet half a
    // tile more (128 keys, groups of 4: 2.5 tiles an item instead of 2).
    const int32_t k0 = it.lo - it.lo % p.box, nt = it.hi > it.lo ? (it.hi - k0 + KT - 1) / KT : 0;
    // nt * (splits + 1) stays under 2^32: 2^24 tiles, 152 parts
    const int32_t a = (int32_t)((uint32_t)nt * it.part / (uint32_t)it.splits),
                  b = (int32_t)((uint32_t)nt * (it.part + 1) / (uint32_t)it.splits);
    it.key0 = k0 + a * KT;
    it.n = b - a;
}

// Item `at` of sequence it.s, of segs x it.splits (it.q, it.splits and it.slot,
// the parts before the sequence, are set).
template <typename I>
__device__ __forceinline__ void locate(const Params &p, Item &it, I at, int32_t segs, int32_t blocks) {
    it.part = (int32_t)(at < INT32_MAX ? (int32_t)at / segs : at / segs);
    const int32_t k = (int32_t)(at - (I)it.part * segs);  // < segs, an int32 (n_query * n_heads < 2^31)
    const int32_t block = p.by_heads.quotient(k);
    const int32_t seg = (blocks - 1 - block) * p.n_kv_heads + k - block * p.n_kv_heads;
    it.slot += (int64_t)seg * it.splits + it.part;
    place(p, it, seg);
}

// Item number `index` of the plan (every thread of the caller alike).
// Parts outermost (all heads and blocks go over the same keys at about the
// same time and share them through L2), the longest blocks first, heads
// innermost.
__device__ __forceinline__ Item find_item(const Params &p, int64_t base, const PlanShared *sh, int64_t index) {
    const int lo = find_chunk(sh->items, index);
    const int64_t per = (p.b.n_seqs + CHUNKS - 1) / CHUNKS;
    Item it;
    int64_t at = index - sh->items[lo];
    it.slot = sh->parts[lo];
    for (it.s = lo * per;; ++it.s) {
        it.q = load_seq(p.b, it.s, base);
        const Share h = share(p, it.q);
        it.splits = splits_of(h.tiles, sh->cut);
        const int64_t n = h.segs * it.splits;
        if (at < n) {
            locate(p, it, at, (int32_t)h.segs, h.blocks);
            return it;
        }
        at -= n;
        if (it.splits > 1) it.slot += n;
    }
}

// The same plan for at most 32 sequences, by one warp (the one that finds the
// items: no block barrier, and no other role waits for it).  Here the sequences
// go longest parts first, too.
// Counts fit 32 bits: a row block has 256 of fewer than 2^31 rows x heads, and parts beyond those are
// bounded by the workspace.  (64-bit divisions here were most of the 10 us before the first item.)
struct WarpPlan {
    int32_t total;   // items in all
    int32_t cut;
    // of this lane's sequence: the items before it and its own, the parts before it
    int32_t before, items, slots;
    int32_t segs, blocks, splits;
};
__device__ __forceinline__ WarpPlan plan_warp(const Params &p, int64_t base) {
    const int lane = threadIdx.x & 31, n = (int)p.b.n_seqs;
    WarpPlan w;
    Share h = {0, 0, 0, 0};
    if (lane < n) h = share(p, load_seq(p.b, lane, base));
    w.segs = (int32_t)h.segs;
    w.blocks = h.blocks;
    w.cut = INT32_MAX;
    if (p.max_slots > 0) {
        float work = (float)w.segs * (float)h.mean;
        int32_t most = w.segs > 0 && h.tiles > 1 ? h.tiles : 1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            work += __shfl_xor_sync(0xffffffffu, work, o);
            most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        }
        const int32_t cut_c = (most + kSplits[lane & 15] - 1) / kSplits[lane & 15];
        float items = 0.f, parts = 0.f;
#pragma unroll 1
        for (int i = 0; 2 * i < n; ++i) {  // a candidate per lane, the sequences by halves of the warp
            const int s = 2 * i + (lane >> 4);
            const int32_t segs = __shfl_sync(0xffffffffu, w.segs, s & 31), tiles = __shfl_sync(0xffffffffu, h.tiles, s & 31);
            if (s >= n) continue;
            const int32_t k = splits_of(tiles, cut_c);
            items += (float)segs * (float)k;
            if (k > 1) parts += (float)segs * (float)k;
        }
        items += __shfl_xor_sync(0xffffffffu, items, 16);
        parts += __shfl_xor_sync(0xffffffffu, parts, 16);
        w.cut = best_cut(p, items, parts, work, cut_c);
    }
    w.splits = splits_of(h.tiles, w.cut);
    w.items = w.segs * w.splits;
    const int32_t size = (h.tiles + w.splits - 1) / w.splits;  // tiles of a part
    w.total = w.before = w.slots = 0;
#pragma unroll 1
    for (int s = 0; s < n; ++s) {
        const int32_t items = __shfl_sync(0xffffffffu, w.items, s);
        const int32_t other = __shfl_sync(0xffffffffu, size, s), k = __shfl_sync(0xffffffffu, w.splits, s);
        w.total += items;
        if (other > size || (other == size && s < lane)) w.before += items;
        if (s < lane && k > 1) w.slots += items;
    }
    return w;
}
// Item number `index` < total of the plan, each lane its own (the whole warp calls).
__device__ __forceinline__ Item find_item_warp(const Params &p, int64_t base, const WarpPlan &w, int64_t index64) {
    const int32_t index = index64 < w.total ? (int32_t)index64 : w.total;
    int cur = 0;
#pragma unroll 1
    for (int s = 0; s < (int)p.b.n_seqs; ++s) {
        const int32_t b = __shfl_sync(0xffffffffu, w.before, s), n = __shfl_sync(0xffffffffu, w.items, s);
        if (index >= b && index < b + n) cur = s;
    }
    Item it;
    it.s = cur;
    it.slot = __shfl_sync(0xffffffffu, w.slots, cur);
    it.splits = __shfl_sync(0xffffffffu, w.splits, cur);
    const int32_t at = index - __shfl_sync(0xffffffffu, w.before, cur);
    const int32_t segs = __shfl_sync(0xffffffffu, w.segs, cur), blocks = __shfl_sync(0xffffffffu, w.blocks, cur);
    it.n_rows = 0;
    if (index < w.total) {
        it.q = load_seq(p.b, cur, base);
        locate(p, it, at, segs, blocks);
    }
    return it;
}

// ---------------------------------------------------------------- helpers ----

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    mma_bf16(d, a, b, idesc, accumulate);  // kind::f16: the descriptor names the type
}
// A from TMEM (16-bit pairs, a row per lane), B from shared memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The bits x, x + 1, ..., 31 (all for x <= 0, none for x > 31).
__device__ __forceinline__ uint32_t bits_from(int32_t x) { return x <= 0 ? ~0u : x > 31 ? 0u : ~0u << x; }
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(is));
    return is != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}

// kind::f16 instruction descriptor, fp32 accumulator, A K-major.
__host__ __device__ constexpr uint32_t idesc_16(bool bf16, int M, int N, bool b_mn_major) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_mn_major ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// ----------------------------------------------------------------- kernel ----

template <typename E, int DP, bool BF16>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    tile_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                const __grid_constant__ Params p) {
    using C = Cfg<DP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *q_smem = smem;
    uint8_t *kv_smem = smem + 2 * C::Q_BYTES;
    uint8_t *swap_smem = kv_smem + C::STAGES * C::STAGE_BYTES;
    Shared<DP> *sh = reinterpret_cast<Shared<DP> *>(swap_smem + C::SWAP_BYTES);
    volatile int *abort = &sh->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((smem_u32(smem) & 1023u) != 0) {  // the same for every CTA
        grid_dependency_wait();
        if (threadIdx.x == 0) raise_error(ENGRAM_EUNSUPPORTED);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&sh->kv_full[i], 1);
            mbar_init(&sh->kv_empty[i], 2);  // both row tiles' products
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->q_full[i], 4);
            mbar_init(&sh->s_full[i], 1);
            for (int c = 0; c < P_PARTS; ++c) mbar_init(&sh->p_ready[i][c], 4);
            mbar_init(&sh->s_free[i], 4);
            mbar_init(&sh->pv_done[i], 1);
            mbar_init(&sh->turn[i], 1);
            mbar_init(&sh->drained[i], 1);
            mbar_init(&sh->o_full[i], 1);
        }
        for (int i = 0; i < ITEMS; ++i) {
            mbar_init(&sh->item_full[i], 1);
            mbar_init(&sh->item_empty[i], 11);  // eight softmax warps, two MMA warps and the load warp
        }
        sh->abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&k_map);
        prefetch_tensormap(&v_map);
    }
    if (warp == 8) {
        tmem_alloc(&sh->tmem_base, C::TMEM_COLS);
        tmem_relinquish();
    }
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t base = __ldg(p.b.offs);
    if (blockIdx.x == 0 && threadIdx.x == 0 && __ldg(p.b.offs + p.b.n_seqs) - base != p.b.n_query)
        raise_error(ENGRAM_ERANGE);
    tc_fence_before();
    const bool few = p.b.n_seqs <= 32;  // then the items' warp plans alone, below
    if (few) {
        __syncthreads();
    } else {
        make_plan<NUM_THREADS>(p, base, &sh->plan);  // synchronises the block
        if (blockIdx.x == 0 && threadIdx.x == 0 && p.cut) *p.cut = sh->plan.cut;
    }
    tc_fence_after();
    const uint32_t tmem = sh->tmem_base;

    // Item number i of this CTA, for a whole warp: every role takes all of them in order (null after a time-out).
    const auto take = [&](uint32_t i) -> const Item * {
        return warp_wait(&sh->item_full[i % ITEMS], (i / ITEMS) & 1, abort) ? &sh->items[i % ITEMS] : nullptr;
    };

    // Registers move from the load and MMA warps to the softmax warps, which hold a row of 128
    // scores each: 256 x 208 + 128 x 88 = the launch's 384 x 168.
    if (warp < 8) {  // ------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = warp >> 2;                  // row tile
        const int row = (warp & 3) * 32 + lane;   // row of the tile: this thread's TMEM lane
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tm = tmem + lanes + t * KT, o_tm = tmem + lanes + C::O_COL + t * DP;
        const uint32_t p_tm = C::APART ? tmem + lanes + C::P_COL + t * 64 : s_tm;
        constexpr float LIFT = E::LIFT > 0.f ? E::LIFT - E::RESCALE : 0.f;  // of a weight at the running maximum
        uint32_t s_ph = 0, o_ph = 0, it = 0, pv_ph = 0;
        bool ok = true;

        // The tile's query rows into shared memory by asynchronous copies, 16 bytes a lane and round
        // (rows past the item's are zero): fetch_q starts them, hand_q waits for them and tells the
        // MMA warp.
        constexpr int PIECES = DP / 8, PER = 32 / PIECES;  // 16-byte pieces of a row, rows a warp loads at once
        const auto fetch_q = [&](const Item &w) {
            const int ch = lane % PIECES;
            const int32_t rr = w.r0 + t * MT + row, tok = p.by_group.quotient(rr), n_rows = w.n_rows;
            const int64_t mine = ((int64_t)w.q.row0 + tok) * p.q_token_stride +
                                 (int64_t)(w.head * p.group + rr - tok * p.group) * p.q_head_stride;
            const uint32_t dst = smem_u32(q_smem) + t * C::Q_BYTES + (ch >> 3) * (MT * 128);
#pragma unroll 4
            for (int i = 0; i < 32; i += PER) {
                const int r = (warp & 3) * 32 + i + lane / PIECES;
                const int64_t at = __shfl_sync(0xffffffffu, mine, r & 31);
                const bool in = t * MT + r < n_rows && ch * 8 < p.head_dim;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + r * 128 + (((ch & 7) ^ (r & 7)) << 4)),
                             "l"(p.q + (in ? at + ch * 8 : 0)), "r"(in ? 16 : 0)
                             : "memory");
            }
        };
        const auto hand_q = [&] {
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->q_full[t]);
        };

        const Item *w = take(0);
        if (w && w->n > 0 && w->n_rows > t * MT) {
            fetch_q(*w);
            hand_q();
        }
        for (uint32_t k = 0; w && w->n_rows > 0 && ok; ++k) {
            const bool mine = w->n_rows > t * MT;
            const int32_t n = w->n;
            const Item *next = nullptr;
            float m = -INFINITY, l = 0.f;  // m: the maximum that the weights refer to, in scores
            if (mine && n > 0) {
                const int32_t item_key0 = w->key0;
                const int32_t pos = w->pos0 + p.by_group.quotient(w->r0 + t * MT + row);
                const int32_t row_lo = first_seen(pos, p.window);
                // keys in reach of every row of the tile
                const int32_t last = (w->n_rows < (t + 1) * MT ? w->n_rows : (t + 1) * MT) - 1;
                const int32_t full_hi = w->pos0 + p.by_group.quotient(w->r0 + t * MT) + 1;
                const int32_t full_lo = first_seen(w->pos0 + p.by_group.quotient(w->r0 + last), p.window);
                for (int32_t j = 0; j < n; ++j) {
                    const int32_t key0 = item_key0 + j * KT;
                    ok = warp_wait(&sh->s_full[t], s_ph++ & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    // Values that must not meet a weight of zero leave the tile before the products: those
                    // of keys that no row reaches (they may be anything), infinities and NaN of keys that
                    // some row does not see.  Both row tiles do it, each before its own products; who clears
                    // one first notes it, so either's epilogue adds it to the rows that see it.
                    if (key0 < w->full_lo || key0 + KT > w->full_hi) {
                        const uint32_t vi = it + 2 * j + 1;
                        ok = warp_wait(&sh->kv_full[vi % C::STAGES], (vi / C::STAGES) & 1, abort);
                        if (!ok) break;
                        const uint32_t vrow = smem_u32(kv_smem) + (vi % C::STAGES) * C::STAGE_BYTES + row * 128;
                        const auto at = [&](int i) { return vrow + (i >> 3) * (KT * 128) + (((i ^ row) & 7) << 4); };
                        const bool keep = key0 + row >= w->lo && key0 + row < w->hi;
                        if (holds_nonfinite<E, DP / 8>(keep, at)) {
                            Item *const note = const_cast<Item *>(w);
                            atomicMin(&note->bad_lo, j);
                            atomicMax(&note->bad_hi, j);
                            __threadfence_block();
                            clear_nonfinite<E, DP / 8>(true, at);
                        } else if (!keep) {
                            clear_nonfinite<E, DP / 8>(false, at);
                        }
                        fence_proxy_async_smem();
                    }
                    // the second half of the scores arrives under the first half's maximum
                    uint32_t raw[4][32];
                    tmem_ld_32x32b_x32(s_tm, raw[0]);
                    tmem_ld_32x32b_x32(s_tm + 32, raw[1]);
                    tmem_ld_wait();
                    tmem_ld_32x32b_x32(s_tm + 64, raw[2]);
                    tmem_ld_32x32b_x32(s_tm + 96, raw[3]);
                    const bool edge = key0 < full_lo || key0 + KT > full_hi;
                    const int32_t a = row_lo - key0, b = pos - key0;  // this row's keys: [a, b] of the tile
                    float s[KT];
                    float part[4];  // independent chains: one alone would wait out each maximum's latency
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h) {
                            tmem_ld_wait();
                            if (C::APART) {
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&sh->s_free[t]);
                            }
                        }
#pragma unroll
                        for (int i = h * 64; i < h * 64 + 64; ++i) s[i] = __uint_as_float(raw[i >> 5][i & 31]);
                        if (edge) {
#pragma unroll
                            for (int c = h * 2; c < h * 2 + 2; ++c) {
                                const uint32_t in = bits_from(a - c * 32) & ~bits_from(b - c * 32 + 1);
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (!(in & (1u << i))) s[c * 32 + i] = -INFINITY;
                            }
                        }
#pragma unroll
                        for (int i = h * 64; i < h * 64 + 64; i += 2)
                            part[(i >> 1) & 3] = i < 8 ? fmaxf(s[i], s[i + 1]) : max3(part[(i >> 1) & 3], s[i], s[i + 1]);
                    }
                    const float mx = fmaxf(max3(part[0], part[1], part[2]), part[3]);
                    if (C::APART) {  // the tile before is in O, its weights are used (before the first there is none)
                        ok = warp_wait(&sh->pv_done[t], pv_ph ^ 1, abort);
                        pv_ph ^= 1;
                        if (!ok) break;
                        tc_fence_after();
                    }
                    float up = 1.f;
                    if ((mx - m) * p.scale_log2 > E::RESCALE) {  // also from -inf
                        up = rows::exp2_approx((m - mx) * p.scale_log2);
                        m = mx;
                    }
                    if (j > 0 && __any_sync(0xffffffffu, up != 1.f)) {
                        l *= up;
#pragma unroll
                        for (int c = 0; c < DP / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16(o_tm + c * 16, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * up);
                            tmem_st_32x32b_x16(o_tm + c * 16, o);
                        }
                    }
                    const float mref = m == -INFINITY ? 0.f : fmaf(m, p.scale_log2, -LIFT);
                    const float2 sc = make_float2(p.scale_log2, p.scale_log2), off = make_float2(-mref, -mref);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 x = fma2(make_float2(s[c * 32 + 2 * i], s[c * 32 + 2 * i + 1]), sc, off);
                            x.x = rows::exp2_approx(x.x);
                            x.y = rows::exp2_approx(x.y);
                            sum[i & 1] = add2(sum[i & 1], x);
                            pk[i] = E::pack(x.x, x.y);  // 16-bit operands of the second product
                        }
                        tmem_st_32x32b_x16(p_tm + c * 16, pk);
                        if ((c + 1) % (4 / P_PARTS) == 0) {  // the second product may start on these keys
                            tmem_st_wait();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sh->p_ready[t][c * P_PARTS / 4]);
                        }
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                }
                if (!ok) break;
            }
            it += 2 * n;
            if (mine && n > 0) {
                // The last scores were there, so the queries' memory is free: the next item's are fetched
                // under this item's last product, and its scores computed under this item's epilogue.
                next = take(k + 1);
                const bool next_mine = next && next->n > 0 && next->n_rows > t * MT;
                if (next_mine) fetch_q(*next);
                ok = warp_wait(&sh->o_full[t], o_ph++ & 1, abort);
                if (!ok) break;
                if (next_mine) hand_q();
                tc_fence_after();
            } else {
                next = take(k + 1);
                if (next && next->n > 0 && next->n_rows > t * MT) {
                    fetch_q(*next);
                    hand_q();
                }
            }
            if (mine) {
                const bool whole = w->splits == 1, live = t * MT + row < w->n_rows;
                const int64_t slot = whole ? 0 : w->slot;
                const int32_t rr = w->r0 + t * MT + row, tok = p.by_group.quotient(rr), head = w->head * p.group + rr - tok * p.group;
                const int64_t out_row = (int64_t)w->q.row0 + tok;
                const float inv = whole ? inverse(l, w->pos0 + tok) : 1.f;
                // A lane has a row in TMEM, but lanes that store to 32 rows at once cost an access to L1 each:
                // the rows change hands in shared memory, 128 bytes of each at a time (the pieces permuted,
                // so neither way meets a bank twice), and eight lanes store a row's piece.
                const uint32_t swap = smem_u32(swap_smem) + warp * (32 * 128);
                const int64_t dst = out_row * p.out_token_stride + (int64_t)head * p.out_head_stride;
                float *part = p.part_o + (slot * ROWS + t * MT + row - lane) * DP;
                const int32_t warp_rows = w->n_rows - (t * MT + row - lane);  // this warp's rows of the item
                const auto read_o = [&](int c, uint32_t (&o)[32]) {  // 32 columns of this lane's row
                    if (n > 0) {
                        tmem_ld_32x32b_x32(o_tm + c, o);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0;
                    }
                    if (w->bad_hi >= 0 && live) {
                        const int32_t pos = w->pos0 + tok;
                        float x[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(o[i]);
                        add_nonfinite<E, 32>(p.b, p.values, w->s, w->head, max(first_seen(pos, p.window), w->key0 + w->bad_lo * KT),
                                             min(pos + 1, w->key0 + (w->bad_hi + 1) * KT), c, p.head_dim, x);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(x[i]);
                    }
                };
                const auto put = [&](int i, const uint32_t *v) {
                    sts16(swap + lane * 128 + (((i ^ lane) & 7) << 4), make_uint4(v[0], v[1], v[2], v[3]));
                };
                const auto get = [&](int r) { return lds16(swap + r * 128 + (((lane ^ r) & 7) << 4)); };
                if (whole) {
#pragma unroll 1
                    for (int c = 0; c < DP; c += 64) {
#pragma unroll 1
                        for (int half = 0; half < 2; ++half) {
                            uint32_t o[32], u[16];
                            read_o(c + half * 32, o);
#pragma unroll
                            for (int h = 0; h < 16; ++h)
                                u[h] = E::pack(__uint_as_float(o[2 * h]) * inv, __uint_as_float(o[2 * h + 1]) * inv);
#pragma unroll
                            for (int i = 0; i < 4; ++i) put(half * 4 + i, u + 4 * i);
                        }
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int r = k * 4 + (lane >> 3), at = c + (lane & 7) * 8;
                            const int64_t to = __shfl_sync(0xffffffffu, dst, r);
                            if (r < warp_rows && at < p.head_dim) *reinterpret_cast<uint4 *>(p.out + to + at) = get(r);
                        }
                        __syncwarp();
                    }
                } else if (n > 0) {
#pragma unroll 1
                    for (int c = 0; c < DP; c += 32) {
                        uint32_t o[32];
                        read_o(c, o);
#pragma unroll
                        for (int i = 0; i < 8; ++i) put(i, o + 4 * i);
                        __syncwarp();
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int r = k * 4 + (lane >> 3);
                            if (r < warp_rows) *reinterpret_cast<uint4 *>(part + r * DP + c + (lane & 7) * 4) = get(r);
                        }
                        __syncwarp();
                    }
                }
                tc_fence_before();  // O has been read before the next item's first product is allowed
                if (live) {
                    const float m2 = m == -INFINITY ? -INFINITY : fmaf(m, p.scale_log2, -LIFT);
                    if (!whole) {
                        p.part_ml[slot * (2 * ROWS) + t * MT + row] = m2;
                        p.part_ml[slot * (2 * ROWS) + ROWS + t * MT + row] = l;
                    } else if (p.lse) {
                        p.lse[out_row * p.n_heads + head] = rows::lse_of(m2, l);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->item_empty[k % ITEMS]);
            w = next;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");  // after a time-out queries may still be on their way
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 10) {  // --------------------------------------------- items
            // Rounds of one item per CTA, every other one in reverse: the items come longest first, and
            // the CTAs at one end would get the longer one of every round.  A lane finds one of the
            // next 32 items (several divisions each), then they are handed out in order.
            const auto prefetch_q = [&](const Item &w) {  // an item's queries on their way into L2
                const int64_t row0 = w.q.row0;
                const int32_t r0 = w.r0, n_rows = w.n > 0 ? w.n_rows : 0, head0 = w.head * p.group;
                for (int r = lane; r < n_rows; r += 32) {
                    const int32_t tok = p.by_group.quotient(r0 + r), hh = r0 + r - tok * p.group;
                    const uint16_t *q = p.q + (row0 + tok) * p.q_token_stride + (int64_t)(head0 + hh) * p.q_head_stride;
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
                    if (p.head_dim > 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64));
                }
            };
            WarpPlan plan;
            if (few) {
                plan = plan_warp(p, base);
                if (blockIdx.x == 0 && lane == 0 && p.cut) *p.cut = plan.cut;
            } else {
                plan.total = sh->plan.items[CHUNKS];
            }
            bool ok = true, more = true;
            for (uint32_t i0 = 0; ok && more; i0 += 32) {
                const uint32_t i = i0 + lane;
                const int64_t index = (int64_t)i * gridDim.x + (i & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
                Item mine;
                mine.n_rows = 0;
                if (few)
                    mine = find_item_warp(p, base, plan, index);
                else if (index < plan.total)
                    mine = find_item(p, base, &sh->plan, index);
                for (int k = 0; ok && more && k < 32; ++k) {
                    if (lane == k) {
                        if (i >= ITEMS) ok = mbar_wait(&sh->item_empty[i % ITEMS], ((i / ITEMS) - 1) & 1, abort);
                        if (ok) {
                            sh->items[i % ITEMS] = mine;
                            mbar_arrive(&sh->item_full[i % ITEMS]);
                        }
                        more = mine.n_rows != 0;
                    }
                    ok = __shfl_sync(0xffffffffu, ok, k);
                    more = __shfl_sync(0xffffffffu, more, k);
                    if (ok && more) prefetch_q(sh->items[(i0 + k) % ITEMS]);
                }
            }
        } else if (warp == 9) {  // --------------------------------------- K, V loads
            const int boxes = KT / p.box;
            const uint32_t box_bytes = (uint32_t)p.box * 128u * (DP / 64);
            uint32_t it = 0;
            bool ok = true;
            for (uint32_t i = 0; ok; ++i) {
                const Item *const item = take(i);
                if (!item || item->n_rows == 0) break;
                const struct {
                    int64_t s;
                    int32_t head, key0, n, lo, hi;
                } w = {item->s, item->head, item->key0, item->n, item->lo, item->hi};
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->item_empty[i % ITEMS]);
                int64_t window0 = -1;
                int32_t page = -1;
                for (int32_t j = 0; ok && j < w.n; ++j) {
                    const int64_t b0 = w.key0 / p.box + (int64_t)j * boxes;
                    if (window0 < 0 || b0 + boxes > window0 + 32) {  // the pages of the next 32 boxes, a lane each
                        window0 = b0;
                        const int64_t key = (b0 + lane) * p.box;
                        page = -1;
                        if (key < w.hi) {
                            page = __ldg(p.b.block_table + w.s * p.b.table_stride + (uint32_t)key / (uint32_t)p.b.page_size);
                            if (page < 0 || page >= p.b.n_pages) {
                                if (key + p.box > w.lo) raise_error(ENGRAM_ERANGE);
                                page = -1;  // out of range: the copy fills zeros
                            }
                        }
                    }
                    const int32_t mine = __shfl_sync(0xffffffffu, page, (int)(b0 - window0) + (lane < boxes ? lane : 0));
                    const int64_t key = (b0 + lane) * p.box;
                    const bool load = lane < boxes && key < w.hi && key + p.box > w.lo;
                    const uint32_t loads = __popc(__ballot_sync(0xffffffffu, load));
                    const int y = (int)((uint32_t)key % (uint32_t)p.b.page_size);
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++it) {
                        const int st = it % C::STAGES;
                        if (lane == 0) {
                            if (it >= C::STAGES) ok = mbar_wait(&sh->kv_empty[st], ((it / C::STAGES) - 1) & 1, abort);
                            if (ok) mbar_arrive_expect_tx(&sh->kv_full[st], loads * box_bytes);
                        }
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (!ok) break;
                        if (load) {
                            uint8_t *dst = kv_smem + st * C::STAGE_BYTES + lane * p.box * 128;
#pragma unroll
                            for (int c = 0; c < DP / 64; ++c)
                                rows::tma_load_4d(dst + c * KT * 128, kv ? &v_map : &k_map, &sh->kv_full[st], c * 64, y, w.head,
                                                  mine);
                        }
                    }
                }
            }
            if (lane == 0) {  // never leave with a copy still landing (also after an abort elsewhere)
                int no_abort = 0;
                for (uint32_t i = it < C::STAGES ? 0 : it - C::STAGES; i < it; ++i)
                    mbar_wait(&sh->kv_full[i % C::STAGES], (i / C::STAGES) & 1, &no_abort, 200000000ull);
            }
        } else {  // warps 8, 11 ---------------------------------- MMAs of row tile t
            // The whole warp walks the tiles with warp-uniform values (the instruction takes its
            // descriptors from uniform registers) and one elected lane issues.  Issuing blocks while
            // the tensor pipe has a few products waiting, so each row tile has a warp of its own that
            // waits for weights and keys meanwhile; the two take strict turns (turn[t]).  Without the
            // turns their products interleave, both softmaxes then run at once and both wait for the
            // tensor pipe at once (65,536-token chunk: 1.99 ms; one warp for both tiles 1.64 ms).
            const int t = warp == 8 ? 0 : 1;
            constexpr uint32_t ID_S = idesc_16(BF16, MT, KT, false), ID_O = idesc_16(BF16, MT, DP, true);
            const bool leader = elect_one();
            const uint32_t kva = smem_u32(kv_smem);
            const uint64_t q_desc = smem_desc(smem_u32(q_smem) + t * C::Q_BYTES, 16, 1024, kSwizzle128B);
            const uint64_t k_desc = smem_desc(kva, 16, 1024, kSwizzle128B);
            const uint64_t v_desc = smem_desc(kva, KT * 128, 1024, kSwizzle128B);
            const uint32_t s_tm = __shfl_sync(0xffffffffu, tmem, 0) + t * KT;
            const uint32_t o_tm = __shfl_sync(0xffffffffu, tmem, 0) + C::O_COL + t * DP;
            const uint32_t p_tm = C::APART ? __shfl_sync(0xffffffffu, tmem, 0) + C::P_COL + t * 64 : s_tm;
            uint32_t st = 0, st_ph = 0;  // ring entry to consume next, and its phase
            uint32_t q_ph = 0, p_ph = 0, turn_ph = 0, s_ph = 0;
            bool ok = true;
            const auto advance = [&] {
                if (++st == C::STAGES) st = 0, st_ph ^= 1;
            };
            const auto scores = [&] {  // S = Q K^T, K in ring entry st
                const uint64_t k0 = k_desc + st * (C::STAGE_BYTES >> 4);
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const uint32_t off = ((k >> 2) * (KT * 128) + (k & 3) * 32) >> 4;
                    mma_ss(s_tm, q_desc + off, k0 + off, ID_S, k != 0);
                }
                mma_commit(&sh->s_full[t]);
                mma_commit(&sh->kv_empty[st]);
            };
            // Row tile 0 has the first turn: its first wait finds the phase before the first complete.
            const auto my_turn = [&](bool both) {
                if (C::APART || !both) return true;
                const bool r = warp_wait(&sh->turn[t], turn_ph ^ (t == 0), abort);
                turn_ph ^= 1;
                return r;
            };
            // APART: the scores before have been read (before the first there are none).
            const auto scores_free = [&] {
                if (!C::APART) return true;
                const bool r = warp_wait(&sh->s_free[t], s_ph ^ 1, abort);
                s_ph ^= 1;
                return r;
            };
            for (uint32_t i = 0; ok; ++i) {
                const Item *const item = take(i);
                ok = item != nullptr;
                if (!ok) break;
                const int32_t n_rows = __shfl_sync(0xffffffffu, item->n_rows, 0);
                const int32_t n = __shfl_sync(0xffffffffu, item->n, 0);
                if (n_rows == 0) break;
                __syncwarp();
                if (leader) mbar_arrive(&sh->item_empty[i % ITEMS]);
                if (n == 0) continue;
                const bool both = n_rows > MT;
                if (!both && t == 1) {  // no rows here: give every ring entry back as it fills
                    for (int32_t j = 0; ok && j < 2 * n; ++j) {
                        ok = warp_wait(&sh->kv_full[st], st_ph, abort);
                        if (leader) mbar_arrive(&sh->kv_empty[st]);
                        advance();
                    }
                    continue;
                }
                ok = warp_wait(&sh->q_full[t], q_ph, abort) && warp_wait(&sh->kv_full[st], st_ph, abort) && scores_free() &&
                     my_turn(both);
                if (!ok) break;
                q_ph ^= 1;
                tc_fence_after();
                if (leader) {
                    scores();
                    if (!C::APART && both) mbar_arrive(&sh->turn[t ^ 1]);
                }
                advance();
                for (int32_t j = 0; j < n; ++j) {
                    const bool more = j + 1 < n;
                    const uint32_t v = st;
                    const uint64_t v0 = v_desc + v * (C::STAGE_BYTES >> 4);
                    ok = warp_wait(&sh->kv_full[v], st_ph, abort);
                    advance();
                    ok = ok && (!more || warp_wait(&sh->kv_full[st], st_ph, abort));
                    if (C::APART && more && ok) {
                        ok = scores_free();
                        tc_fence_after();
                        if (ok && leader) scores();
                    }
                    ok = ok && warp_wait(&sh->p_ready[t][0], p_ph, abort) && my_turn(both);
#pragma unroll
                    for (int c = 0; c < P_PARTS; ++c) {
                        if (c) ok = ok && warp_wait(&sh->p_ready[t][c], p_ph, abort);
                        if (!ok) break;
                        tc_fence_after();
                        if (leader) {
#pragma unroll
                            for (int k = c * (KT / 16 / P_PARTS); k < (c + 1) * (KT / 16 / P_PARTS); ++k)
                                mma_ts(o_tm, p_tm + k * 8, v0 + k * (2048 >> 4), ID_O, (j | k) != 0);
                        }
                    }
                    if (!ok) break;
                    p_ph ^= 1;
                    if (leader) {
                        if (C::APART) mma_commit(&sh->pv_done[t]);
                        if (!more)
                            mma_commit(&sh->o_full[t]);
                        else if (!C::APART)
                            scores();
                        if (!C::APART && both) mbar_arrive(&sh->turn[t ^ 1]);
                        mma_commit(&sh->kv_empty[v]);
                    }
                    if (more) advance();
                }
            }
            // Leave only when every MMA and the arrivals that follow them are done: one more commit of the
            // issuing lane, on a barrier that nothing else uses.
            if (leader) {
                int no_abort = 0;
                mma_commit(&sh->drained[t]);
                mbar_wait(&sh->drained[t], 0, &no_abort, 200000000ull);
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// Adds up the parts of split items, in order.  A block takes 16 rows of a
// segment at a time, a warp 4 of them (their loads together), its lanes 4
// values of each.
template <typename E, int DP>
__global__ void __launch_bounds__(128, JOIN_PER_SM) tile_join_kernel(const __grid_constant__ Params p) {
    constexpr int R = 4;
    __shared__ int64_t segs[CHUNKS + 1], parts[CHUNKS + 1];
    grid_dependency_wait();
    allow_dependent_launch();
    const int32_t cut = __ldcg(p.cut);
    if (cut == INT32_MAX) return;
    const int64_t base = __ldg(p.b.offs);
    chunk_sums(p, segs, parts, [&](int64_t s, int64_t &n, int64_t &k_sum) {
        const Share h = share(p, load_seq(p.b, s, base));
        const int32_t k = splits_of(h.tiles, cut);
        if (k > 1) {
            n += h.segs;
            k_sum += h.segs * k;
        }
    });
    const int lane = threadIdx.x & 31;
    const bool on = lane * 4 < DP;
    const int64_t per = (p.b.n_seqs + CHUNKS - 1) / CHUNKS;
    for (int64_t x = blockIdx.x; x < segs[CHUNKS] * (ROWS / 16); x += gridDim.x) {
        // the segment: the sequence whose split segments hold number x / 16
        const int c = find_chunk(segs, x / (ROWS / 16));
        int64_t at = x / (ROWS / 16) - segs[c], slot = parts[c];
        Item it;
        for (it.s = c * per;; ++it.s) {
            it.q = load_seq(p.b, it.s, base);
            const Share h = share(p, it.q);
            it.splits = splits_of(h.tiles, cut);
            if (it.splits == 1) continue;
            if (at < h.segs) break;
            at -= h.segs;
            slot += h.segs * it.splits;
        }
        it.part = 0;
        place(p, it, (int32_t)at);
        slot += at * it.splits;
        const int r0 = (int)(x % (ROWS / 16)) * 16 + (threadIdx.x >> 5) * R;
        if (r0 >= it.n_rows) continue;

        float m[R], l[R];
        float4 acc[R];
#pragma unroll
        for (int q = 0; q < R; ++q) {
            m[q] = -INFINITY;
            l[q] = 0.f;
            acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const float *ml = p.part_ml + slot * (2 * ROWS) + r0;  // 4 rows: one 16-byte load
        for (int k = lane; k < it.splits; k += 32) {
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(ml + (int64_t)k * (2 * ROWS)));
            m[0] = fmaxf(m[0], v.x);
            m[1] = fmaxf(m[1], v.y);
            m[2] = fmaxf(m[2], v.z);
            m[3] = fmaxf(m[3], v.w);
        }
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m[q] = fmaxf(m[q], __shfl_xor_sync(0xffffffffu, m[q], o));
        for (int k0 = 0; k0 < it.splits; k0 += 32) {
            float mk[R], wk[R];
#pragma unroll
            for (int q = 0; q < R; ++q) mk[q] = -INFINITY, wk[q] = 0.f;
            if (k0 + lane < it.splits) {
                const float *a = ml + (int64_t)(k0 + lane) * (2 * ROWS);
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(a)), u = __ldcg(reinterpret_cast<const float4 *>(a + ROWS));
                mk[0] = v.x, mk[1] = v.y, mk[2] = v.z, mk[3] = v.w;
                const float lk[R] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int q = 0; q < R; ++q)
                    if (r0 + q < it.n_rows) {
                        wk[q] = rows::weight(mk[q], m[q]);
                        l[q] += wk[q] * lk[q];
                    }
            }
            const int n = it.splits - k0 < 32 ? it.splits - k0 : 32;
#pragma unroll 2
            for (int k = 0; k < n; ++k) {
                float4 v[R];
                const float *o = p.part_o + ((slot + k0 + k) * ROWS + r0) * DP + lane * 4;
#pragma unroll
                for (int q = 0; q < R; ++q)
                    v[q] = on ? __ldcg(reinterpret_cast<const float4 *>(o + q * DP)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int q = 0; q < R; ++q) {
                    const float f = __shfl_sync(0xffffffffu, wk[q], k);
                    // a part without keys for this row left no sum (and, without any tile, no O)
                    if (__shfl_sync(0xffffffffu, mk[q], k) != -INFINITY) {
                        acc[q].x = fmaf(f, v[q].x, acc[q].x);
                        acc[q].y = fmaf(f, v[q].y, acc[q].y);
                        acc[q].z = fmaf(f, v[q].z, acc[q].z);
                        acc[q].w = fmaf(f, v[q].w, acc[q].w);
                    }
                }
            }
        }
#pragma unroll
        for (int q = 0; q < R; ++q) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l[q] += __shfl_xor_sync(0xffffffffu, l[q], o);
            const int r = r0 + q;
            if (r >= it.n_rows) continue;
            const int32_t tok = p.by_group.quotient(it.r0 + r), head = it.head * p.group + it.r0 + r - tok * p.group;
            const float inv = inverse(l[q], it.pos0 + tok);
            const int64_t row = (int64_t)it.q.row0 + tok;
            if (lane * 4 < p.head_dim)
                *reinterpret_cast<uint2 *>(p.out + row * p.out_token_stride + (int64_t)head * p.out_head_stride + lane * 4) =
                    make_uint2(E::pack(acc[q].x * inv, acc[q].y * inv), E::pack(acc[q].z * inv, acc[q].w * inv));
            if (p.lse && lane == 0) p.lse[row * p.n_heads + head] = rows::lse_of(m[q], l[q]);
        }
    }
}

}  // namespace tile
}  // namespace attn
}  // namespace engram
