// Paged attention for few query rows per key/value head (single tokens and
// short chunks): one pass over the keys with a running maximum and sum.
//
//   s_j = scale * q.k_j;  m = max s_j;  out = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),
//   carried per row as (m, l = sum, O = weighted sum); two parts of a row join
//   as m = max(m1, m2), l = l1 e^(m1-m) + l2 e^(m2-m), O likewise (Milakov and
//   Gimelshein, "Online normalizer calculation for softmax", 2018).
//
// Bound: the bytes of K and V (each is read once, for all the query heads that
// share it): one token of each of 64 sequences of up to 16,385 takes 341-354
// us, 6.4-6.7 TB/s, 95-98 % of the copy rate.  A "segment" is one 16-row tile
// (rows are the pairs (token, query head of the group), consecutive) of one
// sequence and one key/value head, its work the key tiles in its reach.  The
// tiles of all segments form one line that is cut into equal runs, one per CTA
// (one CTA per SM): the load is even whatever the lengths are.  A segment
// inside one run is finished there; a cut one leaves partial (m, l, O) in the
// workspace, which rows_join_kernel adds up in order.  With few segments and
// short tables the join's launch would cost as much as the attention: then a
// cluster of CTAs takes a segment, a share of its tiles each, and they join
// through distributed shared memory.
//
// Per CTA: two TMA producer warps (K, V) fill a ring of 32 KB tiles (64 keys of
// 128 values or 128 of 64, 128-byte swizzle; the ring holds what HBM latency
// needs in flight per SM) and run ahead across segments; two groups of four
// warps take tiles in turn, each warp a quarter of its tile's keys with mma.sync
// m16n8k16 (16 rows need no larger instruction, and the tensor time is a
// fifth of the tile's memory time), its own m, l and O in registers; the
// eight warps join through shared memory at the end of the segment.
#pragma once

namespace engram {
namespace attn {
namespace rows {

constexpr int ROWS = 16;            // query rows per segment
constexpr int CONSUMERS = 8;        // two groups of four warps
constexpr int MAX_CLUSTER = 8;      // CTAs that share a segment
constexpr int NUM_THREADS = 384;    // the consumers, and the producer's warpgroup (three idle warps)

template <int DP>
struct Cfg {
    static constexpr int KT_LOG2 = DP == 64 ? 7 : 6;
    static constexpr int KT = 1 << KT_LOG2;       // keys per tile: 32 KB of K and V
    static constexpr int KPW = KT / 4;            // keys per warp
    static constexpr int KV_BYTES = KT * DP * 2;  // K (or V) of a tile
    static constexpr int STAGE_BYTES = 2 * KV_BYTES;
    // Even: the two consumer groups take tiles in turn, so a stage then belongs to one group.
    // (A parity wait tells only neighbouring phases apart: a group that had not consumed a
    // stage's last phase itself could pass a wait for the next one before either had landed.)
    static constexpr int STAGES = 196608 / STAGE_BYTES;
    static_assert(STAGES % 2 == 0, "each ring stage must belong to one consumer group");
    static constexpr int JOIN_FLOATS = 4 * ROWS * DP;
};

// Float c of row r in a join buffer: the rows' eight-float groups are rotated, so
// that the accumulators' layout (8 rows x 4 pairs of columns a store) meets
// different banks.
template <int DP>
__device__ __forceinline__ int join_at(int r, int c) { return r * DP + (c ^ ((r & 3) * 8)); }

template <int DP>
struct Shared {
    uint64_t full[Cfg<DP>::STAGES];
    uint64_t empty[Cfg<DP>::STAGES];
    float m[CONSUMERS][ROWS];
    float l[CONSUMERS][ROWS];
    int64_t scan[NUM_THREADS / 32];
    int64_t find_s;       // plan_find's answer
    int64_t find_before;
    uint64_t ready, done;  // cluster: every CTA's share is in its shared memory; every CTA has read the others'
    float tm[ROWS], tl[ROWS];      // cluster: this CTA's maximum and sum of each row
    int32_t bad_lo[2], bad_hi[2];  // tiles in which infinities or NaN were cleared; two segments in turn
    int abort;
};

static_assert(196608 + Cfg<128>::JOIN_FLOATS * 4 + sizeof(Shared<128>) <= 232448, "rows kernel shared memory");

template <int DP>
constexpr int smem_bytes() {
    return Cfg<DP>::STAGES * Cfg<DP>::STAGE_BYTES + Cfg<DP>::JOIN_FLOATS * 4 + (int)sizeof(Shared<DP>);
}

struct Params {
    Batch b;
    const uint16_t *q;
    int64_t q_token_stride, q_head_stride;
    uint16_t *out;
    int64_t out_token_stride, out_head_stride;
    float *lse;         // [n_query][n_heads] or null
    ValuePages values;
    float *part_o;      // [grid][2][rows of a segment][DP]
    float *part_ml;     // [grid][2][2][rows of a segment]
    int32_t n_heads, n_kv_heads, group, head_dim;
    // The kv heads lie on `side` lines beside each other (head h on line h % side), each cut at the same places: CTAs
    // on different lines then read the same pages at about the same time.
    int32_t side, line_heads;    // side * line_heads = n_kv_heads
    Divisor by_group, by_heads;  // the query heads of a kv head; a line's heads
    int32_t window;
    int32_t kt_log2;    // Cfg<DP>::KT_LOG2
    int32_t box;        // tokens per TMA box: gcd(page_size, KT)
    int32_t runs;       // CTAs of a line (all CTAs of the attention launch: times side, times cluster)
    int32_t cluster;    // CTAs that share a segment through distributed shared memory (1: none; then whole = 1)
    int32_t whole;      // > 0: every segment is given this many tiles and none is cut (no join follows)
    float scale_log2;   // scale * log2(e)
};

// ------------------------------------------------------------------- plan ----

// Key tiles that a segment (R rows) of sequence q is given on the line (at
// least one, so that rows without keys are written too), and its segments per
// kv head.
template <int R>
__device__ __forceinline__ int32_t seg_tiles(const Params &p, const Seq &q) {
    if (p.whole > 0) return p.whole;
    const int32_t kt = 1 << p.kt_log2;
    int32_t n = (q.kv + kt - 1) >> p.kt_log2;
    if (p.window > 0) {
        const int32_t tokens = (R - 2) / p.group + 2;  // most tokens that R consecutive rows touch
        const int64_t reach = (int64_t)p.window + tokens - 1;
        const int64_t w = ((reach + kt - 2) >> p.kt_log2) + 1;
        if (w < n) n = (int32_t)w;
    }
    return n > 0 ? n : 1;
}
template <int R>
__device__ __forceinline__ int32_t seg_rows(const Params &p, const Seq &q) {
    return (int32_t)(((int64_t)q.q_len * p.group + R - 1) / R);
}

struct Plan {
    int64_t total;  // tiles on the line
    int64_t run;    // tiles per CTA
};

__device__ __forceinline__ int64_t run_of(const Params &p, int64_t total) {
    int64_t run = total < INT32_MAX - p.runs ? ((int32_t)total + p.runs - 1) / p.runs : (total + p.runs - 1) / p.runs;
    if (p.whole > 1) run = (run + p.whole - 1) / p.whole * p.whole;
    return run < 1 ? 1 : run;
}

// All threads of a block of NT: the length of the line, the tiles per CTA,
// and for f(run) = the place asked for the sequence it lies in (sh_s, with
// the tiles before that sequence in sh_before; sh_s = -1 past the end).
template <int NT, int R>
__device__ Plan plan_find(const Params &p, int64_t base, int64_t index, int64_t *scan, int64_t *sh_s, int64_t *sh_before) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t per = (p.b.n_seqs + NT - 1) / NT;
    const int64_t s0 = tid * per, s1 = s0 + per < p.b.n_seqs ? s0 + per : p.b.n_seqs;
    int64_t sum = 0;
    for (int64_t s = s0; s < s1; ++s) {
        const Seq q = load_seq(p.b, s, base);
        sum += (int64_t)seg_rows<R>(p, q) * p.line_heads * seg_tiles<R>(p, q);
    }
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    if (tid == 0) *sh_s = -1;
    __syncthreads();
    Plan r;
    int64_t before = incl - sum;
    r.total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += scan[w];
        r.total += scan[w];
    }
    r.run = run_of(p, r.total);
    const int64_t f = index * r.run;
    if (f >= before && f < before + sum) {
        int64_t at = before;
        for (int64_t s = s0; s < s1; ++s) {
            const Seq q = load_seq(p.b, s, base);
            const int64_t c = (int64_t)seg_rows<R>(p, q) * p.line_heads * seg_tiles<R>(p, q);
            if (f < at + c) {
                *sh_s = s;
                *sh_before = at;
                break;
            }
            at += c;
        }
    }
    __syncthreads();
    return r;
}

// The same for at most 32 sequences, by every warp for itself: one round of
// loads and no block barrier.
template <int R>
__device__ __forceinline__ Plan plan_find_small(const Params &p, int64_t base, int64_t index, int64_t &s, int64_t &before) {
    const int lane = threadIdx.x & 31;
    int64_t cost = 0;
    if (lane < p.b.n_seqs) {
        const Seq q = load_seq(p.b, lane, base);
        cost = (int64_t)seg_rows<R>(p, q) * p.line_heads * seg_tiles<R>(p, q);
    }
    int64_t incl = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    Plan r;
    r.total = __shfl_sync(0xffffffffu, incl, 31);
    r.run = run_of(p, r.total);
    const int64_t f = index * r.run;
    const uint32_t in = __ballot_sync(0xffffffffu, f >= incl - cost && f < incl);
    s = __ffs(in) - 1;  // -1 past the end
    before = __shfl_sync(0xffffffffu, incl - cost, in ? (int)s : 0);
    return r;
}

// A place on the line: the segment and the tile within it.
template <int R>
struct Walk {
    int64_t s;       // sequence
    int32_t line;    // the line: heads line, line + side, ...
    int32_t seg;     // segment within the sequence: row tile * line_heads + head of the line
    int32_t n_segs;  // (n_query * n_heads < 2^31)
    int32_t tiles;   // tiles per segment of this sequence
    int32_t j;       // tile within the segment
    Seq q;

    __device__ __forceinline__ void enter(const Params &p, int64_t base, int64_t s_) {
        s = s_;
        q = load_seq(p.b, s, base);
        tiles = seg_tiles<R>(p, q);
        n_segs = seg_rows<R>(p, q) * p.line_heads;
    }
    __device__ __forceinline__ void start(const Params &p, int64_t base, int64_t s_, int64_t offset, int32_t line_) {
        line = line_;
        enter(p, base, s_);
        seg = (int32_t)(offset < INT32_MAX ? (int32_t)offset / tiles : offset / tiles);
        j = (int32_t)(offset - (int64_t)seg * tiles);
    }
    // to the first tile of the next segment (the line has one)
    __device__ __forceinline__ void next(const Params &p, int64_t base) {
        j = 0;
        if (++seg < n_segs) return;
        seg = 0;
        do {
            if (s + 1 >= p.b.n_seqs) return;
            enter(p, base, s + 1);
        } while (n_segs == 0);
    }
};

// What a segment covers.
struct Segment {
    int32_t head;       // kv head
    int32_t r0;         // first row (token * group + query head within the group)
    int32_t n_rows;     // 1..R
    int32_t pos0;       // position of the sequence's first new token
    int32_t lo, hi;     // keys in reach of any row: [lo, hi)
    int32_t full_lo, full_hi;  // keys in reach of every row
    int32_t tile0, n_tiles;
};

template <int R>
__device__ __forceinline__ Segment segment(const Params &p, const Walk<R> &w) {
    Segment g;
    const int32_t block = p.by_heads.quotient(w.seg);
    g.head = (w.seg - block * p.line_heads) * p.side + w.line;
    g.r0 = block * R;
    const int32_t left = w.q.q_len * p.group - g.r0;
    g.n_rows = left < R ? left : R;
    g.pos0 = w.q.kv - w.q.q_len;
    const int32_t first = g.pos0 + p.by_group.quotient(g.r0), last = g.pos0 + p.by_group.quotient(g.r0 + g.n_rows - 1);
    g.hi = last + 1;  // <= kv
    g.full_hi = first + 1;
    g.lo = first_seen(first, p.window);
    g.full_lo = first_seen(last, p.window);
    if (g.hi < 0) g.hi = 0;
    g.tile0 = g.lo >> p.kt_log2;
    g.n_tiles = g.hi > g.lo ? ((g.hi + (1 << p.kt_log2) - 1) >> p.kt_log2) - g.tile0 : 0;
    return g;
}

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
        "[%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// e^(x - m) in base 2, 0 where nothing was seen (m = -inf only with x = -inf)
__device__ __forceinline__ float weight(float x, float m) { return exp2_approx(x - (m == -INFINITY ? 0.f : m)); }

template <int R>
__device__ __forceinline__ int64_t w_row(const Walk<R> &w, int32_t token) { return (int64_t)w.q.row0 + token; }
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * CONSUMERS) : "memory"); }
// (m, l) in base 2 -> ln sum; -inf where nothing was seen
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f; }
// A row's maximum and sum over the consumer warps, in warp order.
template <typename S>
__device__ __forceinline__ void row_total(const S *sh, int r, float &m, float &l) {
    constexpr int WARPS = sizeof(sh->m) / sizeof(sh->m[0]);
    m = sh->m[0][r];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) m = fmaxf(m, sh->m[w][r]);
    l = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) l += sh->l[w][r] * weight(sh->m[w][r], m);
}

// One arrival on this barrier's counterpart in CTA `rank` of the cluster,
// after this thread's earlier accesses (and those it has synchronised with).
__device__ __forceinline__ void arrive_at(uint64_t *bar, uint32_t rank) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(mapa_shared(smem_u32(bar), rank))
                 : "memory");
}
__device__ __forceinline__ float ld_shared_cluster_f1(uint32_t cluster_saddr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_saddr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_shared_cluster_f4(uint32_t cluster_saddr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_saddr)
                 : "memory");
    return v;
}

// ---------------------------------------------------------------- kernel ----

// Values c .. c + 3 of row r of the segment, v / l, and the row's lse.
template <typename E, int R>
__device__ __forceinline__ void write_out(const Params &p, const Walk<R> &w, const Segment &g, int r, int c, float4 v, float l) {
    if (c >= p.head_dim) return;
    const int32_t tok = p.by_group.quotient(g.r0 + r), hh = (g.r0 + r) - tok * p.group;
    const float inv = inverse(l, g.pos0 + tok);
    uint16_t *dst = p.out + (int64_t)w_row(w, tok) * p.out_token_stride + (int64_t)(g.head * p.group + hh) * p.out_head_stride + c;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(E::pack(v.x * inv, v.y * inv), E::pack(v.z * inv, v.w * inv));
}
template <int R>
__device__ __forceinline__ void write_lse(const Params &p, const Walk<R> &w, const Segment &g, int r, float m, float l) {
    const int32_t tok = p.by_group.quotient(g.r0 + r), hh = (g.r0 + r) - tok * p.group;
    p.lse[(int64_t)w_row(w, tok) * p.n_heads + g.head * p.group + hh] = lse_of(m, l);
}

template <typename E, int DP>
__global__ void __launch_bounds__(NUM_THREADS, 1)
    rows_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                const __grid_constant__ Params p) {
    using C = Cfg<DP>;
    constexpr int KT = C::KT, KPW = C::KPW;
    extern __shared__ __align__(1024) uint8_t smem[];
    float *join = reinterpret_cast<float *>(smem + C::STAGES * C::STAGE_BYTES);
    Shared<DP> *sh = reinterpret_cast<Shared<DP> *>(join + C::JOIN_FLOATS);
    volatile int *abort = &sh->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&sh->full[i], 2);  // K and V
            mbar_init(&sh->empty[i], 4);
        }
        sh->abort = 0;
        sh->bad_lo[0] = sh->bad_lo[1] = INT32_MAX;
        sh->bad_hi[0] = sh->bad_hi[1] = -1;
        mbar_init(&sh->ready, p.cluster);
        mbar_init(&sh->done, p.cluster);
        fence_mbar_init();
        prefetch_tensormap(&k_map);
        prefetch_tensormap(&v_map);
    }
    if (p.cluster > 1) cluster_sync_all();  // the others' barriers are there before anyone arrives on them
    grid_dependency_wait();
    allow_dependent_launch();
    if ((smem_u32(smem) & 1023u) != 0) {  // the same for every CTA
        if (threadIdx.x == 0) raise_error(ENGRAM_EUNSUPPORTED);
        return;
    }
    const int64_t base = __ldg(p.b.offs);
    if (blockIdx.x == 0 && threadIdx.x == 0 && __ldg(p.b.offs + p.b.n_seqs) - base != p.b.n_query)
        raise_error(ENGRAM_ERANGE);
    const int64_t index = blockIdx.x / p.cluster;
    const int rank = p.cluster > 1 ? (int)cluster_ctarank() : 0;
    Plan plan;
    int64_t at_s, at_before;
    if (p.b.n_seqs <= 32) {
        plan = plan_find_small<ROWS>(p, base, index, at_s, at_before);
        __syncthreads();  // the barriers are initialised
    } else {
        plan = plan_find<NUM_THREADS, ROWS>(p, base, index, sh->scan, &sh->find_s, &sh->find_before);
        at_s = sh->find_s;
        at_before = sh->find_before;
    }
    const int64_t f0 = index * plan.run;
    const int64_t f1 = f0 + plan.run < plan.total ? f0 + plan.run : plan.total;
    if (f0 >= f1) return;
    Walk<ROWS> walk;
    walk.start(p, base, at_s, f0 - at_before, 0);
    uint32_t it = 0;  // tiles through the ring
    // This CTA's tiles [first, end) of a segment, and the places on the line that it covers.
    const auto tiles_of = [&](const Segment &g, int64_t f, int32_t &first, int32_t &end) -> int32_t {
        if (p.cluster > 1) {
            first = (int32_t)((int64_t)g.n_tiles * rank / p.cluster);
            end = (int32_t)((int64_t)g.n_tiles * (rank + 1) / p.cluster);
            return 1;
        }
        const int32_t n = (int32_t)(f1 - f < walk.tiles - walk.j ? f1 - f : walk.tiles - walk.j);
        first = walk.j;
        end = walk.j + n < g.n_tiles ? walk.j + n : g.n_tiles;
        return n;
    };

    // Registers move to the consumers, which hold 16 rows' queries and outputs: 256 x 192 + 128 x 120 =
    // the launch's 384 x 168.
    if (warp >= CONSUMERS) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
        if (warp < CONSUMERS + 2) {  // ---------------------- producers: one warp loads K, the next V
            const bool is_v = warp == CONSUMERS + 1;
            const CUtensorMap *const map = is_v ? &v_map : &k_map;
            const int boxes = KT / p.box;
            const uint32_t box_bytes = (uint32_t)p.box * 128u * (DP / 64);
            for (int64_t f = f0; f < f1;) {
                const Segment g = segment(p, walk);
                int32_t first, end;
                const int32_t n = tiles_of(g, f, first, end);
                int64_t window0 = -1;  // first box whose page lane 0 holds
                int32_t page = -1;
                for (int32_t j = first; j < end; ++j, ++it) {
                    const int32_t tile = g.tile0 + j;
                    const int64_t b0 = (int64_t)tile * boxes;
                    if (window0 < 0 || b0 + boxes > window0 + 32) {  // the pages of the next 32 boxes, a lane each
                        window0 = b0;
                        const int64_t key = (b0 + lane) * p.box;
                        page = -1;
                        if (key < g.hi) {
                            page = __ldg(p.b.block_table + walk.s * p.b.table_stride + key / p.b.page_size);
                            if (page < 0 || page >= p.b.n_pages) {
                                if (key + p.box > g.lo) raise_error(ENGRAM_ERANGE);
                                page = -1;  // out of range: the copy fills zeros
                            }
                        }
                    }
                    const int32_t mine = __shfl_sync(0xffffffffu, page, (int)(b0 - window0) + (lane < boxes ? lane : 0));
                    const int64_t key = (b0 + lane) * p.box;
                    const bool load = lane < boxes && key < g.hi && key + p.box > g.lo;
                    const uint32_t loads = __popc(__ballot_sync(0xffffffffu, load));
                    const int st = it % C::STAGES;
                    bool ok = true;
                    if (lane == 0) {
                        if (it >= C::STAGES) ok = mbar_wait(&sh->empty[st], ((it / C::STAGES) - 1) & 1, abort);
                        if (ok) mbar_arrive_expect_tx(&sh->full[st], loads * box_bytes);
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (ok && load) {
                        uint8_t *dst = smem + st * C::STAGE_BYTES + (is_v ? C::KV_BYTES : 0) + lane * p.box * 128;
                        const int y = (int)(key % p.b.page_size);
#pragma unroll
                        for (int c = 0; c < DP / 64; ++c)
                            tma_load_4d(dst + c * KT * 128, map, &sh->full[st], c * 64, y, g.head, mine);
                    }
                }
                f += n;
                if (f < f1) walk.next(p, base);
            }
            // never leave with a copy still landing (also after an abort elsewhere)
            if (lane == 0) {
                int no_abort = 0;
                for (uint32_t i = it < C::STAGES ? 0 : it - C::STAGES; i < it; ++i)
                    mbar_wait(&sh->full[i % C::STAGES], (i / C::STAGES) & 1, &no_abort, 200000000ull);
            }
        }
    } else {  // ------------------------------------------------------ consumers
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        const int grp = warp >> 2, wq = warp & 3;
        const int qr = lane >> 2, qc = (lane & 3) * 2;  // this lane's rows qr, qr + 8 and first column
        int turn = 0;  // segments alternate
        uint32_t exchange_ph = 0;
        for (int64_t f = f0; f < f1; turn ^= 1) {
            const Segment g = segment(p, walk);
            int32_t first, end;
            const int32_t n = tiles_of(g, f, first, end);

            // the 16 query rows as A fragments, and each row's reach
            uint32_t qf[DP / 16][4];
            int32_t row_lo[2], row_hi[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = qr + i * 8;
                const bool live = r < g.n_rows;
                const int32_t tok = p.by_group.quotient(g.r0 + r), hh = (g.r0 + r) - tok * p.group;
                const int32_t pos = g.pos0 + tok;
                row_hi[i] = live ? pos : -1;
                row_lo[i] = first_seen(pos, p.window);
                const uint16_t *src = p.q + (int64_t)(w_row(walk, tok)) * p.q_token_stride +
                                      (int64_t)(g.head * p.group + hh) * p.q_head_stride;
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int c = kk * 16 + h * 8 + qc;
                        qf[kk][h * 2 + i] =
                            live && c < p.head_dim ? __ldg(reinterpret_cast<const uint32_t *>(src + c)) : 0u;
                    }
            }

            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
            float o[DP / 8][4];
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

            for (int32_t j = first; j < end; ++j, ++it) {
                if ((int)(it & 1) != grp) continue;
                const int st = it % C::STAGES;
                const bool ok = warp_wait(&sh->full[st], (it / C::STAGES) & 1, abort);
                const int32_t key0 = (g.tile0 + j) * KT + wq * KPW;
                if (ok && key0 < g.hi && key0 + KPW > g.lo) {
                    const uint32_t kb = smem_u32(smem + st * C::STAGE_BYTES) + wq * KPW * 128;
                    // keys outside [full_lo, full_hi) are hidden from some row; keys outside
                    // [lo, hi) may hold anything
                    const bool edge = key0 < g.full_lo || key0 + KPW > g.full_hi;
                    if (edge) {  // this warp's keys are read by no other
                        constexpr int LANES = 32 / KPW, PIECES = DP / 8 / LANES;  // lanes per key, 16-byte pieces per lane
                        const int key = lane / LANES, c0 = (lane % LANES) * PIECES;
                        const uint32_t vrow = kb + C::KV_BYTES + key * 128;
                        const auto at = [&](int i) {
                            const int ch = c0 + i;
                            return vrow + (ch >> 3) * (KT * 128) + (((ch & 7) ^ (key & 7)) << 4);
                        };
                        const bool keep = key0 + key >= g.lo && key0 + key < g.hi, bad = holds_nonfinite<E, PIECES>(keep, at);
                        if (bad) {
                            atomicMin(&sh->bad_lo[turn], g.tile0 + j);
                            atomicMax(&sh->bad_hi[turn], g.tile0 + j);
                        }
                        if (bad || !keep) clear_nonfinite<E, PIECES>(keep, at);
                        fence_proxy_async_smem();  // before the ring's next copy over it
                        __syncwarp();
                    }
                    float s[KPW / 8][4];  // rows qr (0, 1) and qr + 8 (2, 3), keys 8 t + qc, + 1
#pragma unroll
                    for (int t = 0; t < KPW / 8; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
                    {
                        const int key = ((lane >> 4) << 3) + (lane & 7);
                        const uint32_t krow = kb + key * 128;
#pragma unroll
                        for (int kk = 0; kk < DP / 16; ++kk) {
                            const int ch = kk * 2 + ((lane >> 3) & 1);  // 16-byte piece of the key's row
#pragma unroll
                            for (int b16 = 0; b16 < KPW / 16; ++b16) {
                                uint32_t b[4];
                                ldmatrix_x4(b, krow + b16 * 16 * 128 + (ch >> 3) * (KT * 128) + (((ch & 7) ^ (key & 7)) << 4));
                                E::mma(s[2 * b16], qf[kk], b[0], b[1]);
                                E::mma(s[2 * b16 + 1], qf[kk], b[2], b[3]);
                            }
                        }
                    }
#pragma unroll
                    for (int t = 0; t < KPW / 8; ++t)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            s[t][c] *= p.scale_log2;
                            if (edge) {
                                const int32_t key = key0 + t * 8 + qc + (c & 1);
                                if (key > row_hi[c >> 1] || key < row_lo[c >> 1]) s[t][c] = -INFINITY;
                            }
                        }
                    float up[2], ref[2];
                    bool same = true;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float mx = fmaxf(s[0][2 * i], s[0][2 * i + 1]);
#pragma unroll
                        for (int t = 1; t < KPW / 8; ++t) mx = fmaxf(mx, fmaxf(s[t][2 * i], s[t][2 * i + 1]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        mx = fmaxf(mx, m[i]);
                        up[i] = weight(m[i], mx);
                        same = same && mx == m[i];
                        m[i] = mx;
                        ref[i] = mx - E::LIFT;
                    }
                    if (!__all_sync(0xffffffffu, same)) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) l[i] *= up[i];
#pragma unroll
                        for (int i = 0; i < DP / 8; ++i) {
                            o[i][0] *= up[0];
                            o[i][1] *= up[0];
                            o[i][2] *= up[1];
                            o[i][3] *= up[1];
                        }
                    }
#pragma unroll
                    for (int t = 0; t < KPW / 8; ++t)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            s[t][c] = weight(s[t][c], ref[c >> 1]);
                            l[c >> 1] += s[t][c];
                        }
                    const int key = (((lane >> 3) & 1) << 3) + (lane & 7);
#pragma unroll
                    for (int b16 = 0; b16 < KPW / 16; ++b16) {
                        // the weights rounded to the values' type: the matrix instruction takes 16-bit
                        // operands, and a weight's relative error there is the output's own rounding (LIFT)
                        const float(&u)[4] = s[2 * b16], (&v)[4] = s[2 * b16 + 1];
                        const uint32_t pa[4] = {E::pack(u[0], u[1]), E::pack(u[2], u[3]), E::pack(v[0], v[1]), E::pack(v[2], v[3])};
                        const uint32_t vrow = kb + C::KV_BYTES + (b16 * 16 + key) * 128;
#pragma unroll
                        for (int nn = 0; nn < DP / 16; ++nn) {
                            const int ch = nn * 2 + (lane >> 4);
                            uint32_t b[4];
                            ldmatrix_x4_trans(b, vrow + (ch >> 3) * (KT * 128) + (((ch & 7) ^ (key & 7)) << 4));
                            E::mma(o[nn * 2], pa, b[0], b[1]);
                            E::mma(o[nn * 2 + 1], pa, b[2], b[3]);
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->empty[st]);
            }

            // the eight warps' parts of the segment, joined in warp order; from here on m is what the weights refer to
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[i] -= E::LIFT;
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
                if ((lane & 3) == 0) {
                    sh->m[warp][qr + i * 8] = m[i];
                    sh->l[warp][qr + i * 8] = l[i];
                }
            }
            consumers_sync();
            if (threadIdx.x == 0) {  // the segment before is done with its turn
                sh->bad_lo[turn ^ 1] = INT32_MAX;
                sh->bad_hi[turn ^ 1] = -1;
            }
            float all[2], fac[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                all[i] = sh->m[0][qr + i * 8];
#pragma unroll
                for (int w = 1; w < CONSUMERS; ++w) all[i] = fmaxf(all[i], sh->m[w][qr + i * 8]);
                fac[i] = weight(m[i], all[i]);
            }
            float *mine = join + wq * (ROWS * DP);
#pragma unroll
            for (int half = 1; half >= 0; --half) {
                if (grp == half) {
#pragma unroll
                    for (int nn = 0; nn < DP / 8; ++nn)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float2 *at = reinterpret_cast<float2 *>(mine + join_at<DP>(qr + i * 8, nn * 8 + qc));
                            float2 v = make_float2(o[nn][2 * i] * fac[i], o[nn][2 * i + 1] * fac[i]);
                            if (half == 0) {
                                v.x += at->x;
                                v.y += at->y;
                            }
                            *at = v;
                        }
                }
                consumers_sync();
            }
            const bool whole = walk.j == 0 && n == walk.tiles;
            const int slot = (int)blockIdx.x * 2 + (f == f0 ? 0 : 1);
            // a thread takes 4 values of a row at a time
            for (int e = threadIdx.x * 4; e < ROWS * DP; e += 32 * CONSUMERS * 4) {
                const int r = e / DP, c = e - r * DP;
                if (r >= g.n_rows) continue;
                const int at = join_at<DP>(r, c);
                float4 v = *reinterpret_cast<const float4 *>(join + at);
#pragma unroll
                for (int w = 1; w < 4; ++w) {
                    const float4 t = *reinterpret_cast<const float4 *>(join + w * (ROWS * DP) + at);
                    v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
                }
                if (sh->bad_hi[turn] >= 0 && c < p.head_dim) {
                    const int32_t pos = g.pos0 + p.by_group.quotient(g.r0 + r);
                    float x[4] = {v.x, v.y, v.z, v.w};
                    add_nonfinite<E, 4>(p.b, p.values, walk.s, g.head, max(first_seen(pos, p.window), sh->bad_lo[turn] * KT),
                                        min(pos + 1, (sh->bad_hi[turn] + 1) * KT), c, p.head_dim, x);
                    v = make_float4(x[0], x[1], x[2], x[3]);
                }
                if (p.cluster > 1) {
                    *reinterpret_cast<float4 *>(join + at) = v;  // read by this thread alone so far
                    continue;
                }
                if (!whole) {
                    *reinterpret_cast<float4 *>(p.part_o + (int64_t)slot * (ROWS * DP) + e) = v;
                    continue;
                }
                float mm, ll;
                row_total(sh, r, mm, ll);
                write_out<E>(p, walk, g, r, c, v, ll);
            }
            if (threadIdx.x < g.n_rows) {
                const int r = threadIdx.x;
                float mm, ll;
                row_total(sh, r, mm, ll);
                if (p.cluster > 1) {
                    sh->tm[r] = mm;
                    sh->tl[r] = ll;
                } else if (!whole) {
                    p.part_ml[slot * (2 * ROWS) + r] = mm;
                    p.part_ml[slot * (2 * ROWS) + ROWS + r] = ll;
                } else if (p.lse) {
                    write_lse(p, walk, g, r, mm, ll);
                }
            }
            if (p.cluster > 1) {  // each CTA joins its share of the values from all shares of the keys, in rank order
                consumers_sync();
                if (threadIdx.x < p.cluster) arrive_at(&sh->ready, threadIdx.x);
                const bool ok = mbar_wait_cluster(&sh->ready, exchange_ph, abort);
                const int share = ROWS * DP / p.cluster;
                for (int e = rank * share + threadIdx.x * 4; ok && e < (rank + 1) * share; e += 32 * CONSUMERS * 4) {
                    const int r = e / DP, c = e - r * DP;
                    if (r >= g.n_rows) continue;
                    float mk[MAX_CLUSTER], lk[MAX_CLUSTER], mm = -INFINITY, ll = 0.f;
                    float4 x[MAX_CLUSTER], v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < MAX_CLUSTER; ++k) {
                        mk[k] = -INFINITY;
                        lk[k] = 0.f;
                        x[k] = v;
                        if (k < p.cluster) {
                            mk[k] = ld_shared_cluster_f1(mapa_shared(smem_u32(&sh->tm[r]), k));
                            lk[k] = ld_shared_cluster_f1(mapa_shared(smem_u32(&sh->tl[r]), k));
                            x[k] = ld_shared_cluster_f4(mapa_shared(smem_u32(join + join_at<DP>(r, c)), k));
                        }
                    }
#pragma unroll
                    for (int k = 0; k < MAX_CLUSTER; ++k) mm = fmaxf(mm, mk[k]);
#pragma unroll
                    for (int k = 0; k < MAX_CLUSTER; ++k) {
                        const float w = weight(mk[k], mm);
                        ll = fmaf(w, lk[k], ll);
                        v.x = fmaf(w, x[k].x, v.x);
                        v.y = fmaf(w, x[k].y, v.y);
                        v.z = fmaf(w, x[k].z, v.z);
                        v.w = fmaf(w, x[k].w, v.w);
                    }
                    write_out<E>(p, walk, g, r, c, v, ll);
                    if (p.lse && c == 0) write_lse(p, walk, g, r, mm, ll);
                }
                if (f + n < f1) {  // (more segments than clusters only with offsets that overlap)
                    consumers_sync();
                    if (threadIdx.x < p.cluster) arrive_at(&sh->done, threadIdx.x);
                    mbar_wait_cluster(&sh->done, exchange_ph, abort);  // nobody reads this CTA's memory any more
                }
                exchange_ph ^= 1;
            }
            consumers_sync();  // the join's memory is free again
            f += n;
            if (f < f1) walk.next(p, base);
        }
    }
    if (p.cluster > 1) {  // no CTA leaves while another may read its memory or arrive on its barriers, after a time-out either
        __syncwarp();
        cluster_sync_all();
    }
}

// Adds up the parts of the segments that the line's cuts went through.  Block
// x looks at a cut of a line and acts on it if it is the
// first inside its segment; a warp takes one row, its lanes 4 values each.
template <typename E, int DP, int R>
__global__ void __launch_bounds__(128) rows_join_kernel(const __grid_constant__ Params p) {
    __shared__ int64_t scan[4], find_s, find_before;
    // The plan reads the batch only, which was final before the attention kernel let this one start
    // (it does so after its own wait); the partial results need the wait below.
    const int64_t base = __ldg(p.b.offs);
    const int32_t line = blockIdx.x % p.side;
    const int64_t cut = (int64_t)(blockIdx.x / p.side) + 1;
    Plan plan;
    int64_t at_s, at_before;
    if (p.b.n_seqs <= 32) {
        plan = plan_find_small<R>(p, base, cut, at_s, at_before);
    } else {
        plan = plan_find<128, R>(p, base, cut, scan, &find_s, &find_before);
        at_s = find_s;
        at_before = find_before;
    }
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t f = cut * plan.run;
    if (f >= plan.total) return;
    Walk<R> w;
    w.start(p, base, at_s, f - at_before, line);
    const int64_t first = f - w.j;  // the segment's first tile on the line
    if (w.j == 0 || (cut - 1) * plan.run > first) return;
    const Segment g = segment(p, w);
    const int r = (int)blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (r >= g.n_rows) return;
    const int64_t end = first + w.tiles;
    const int parts = (int)((end - 1) / plan.run - (cut - 1)) + 1;
    const int after = (cut - 1) * plan.run == first ? 0 : 1;  // the first part's slot of its CTA
    const auto slot_of = [&](int k) { return ((cut - 1 + k) * p.side + line) * 2 + (k == 0 ? after : 0); };

    float m = -INFINITY;
    for (int k = lane; k < parts; k += 32) m = fmaxf(m, __ldcg(p.part_ml + slot_of(k) * (2 * R) + r));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool on = lane * 4 < DP;
    for (int k0 = 0; k0 < parts; k0 += 32) {
        float wk = 0.f;
        if (k0 + lane < parts) {
            const float *ml = p.part_ml + slot_of(k0 + lane) * (2 * R) + r;
            wk = weight(__ldcg(ml), m);
            l += wk * __ldcg(ml + R);
        }
        const int n = parts - k0 < 32 ? parts - k0 : 32;
#pragma unroll 8
        for (int k = 0; k < n; ++k) {
            const float x = __shfl_sync(0xffffffffu, wk, k);
            if (on) {
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.part_o + slot_of(k0 + k) * (R * DP) + r * DP) + lane);
                acc.x = fmaf(x, v.x, acc.x);
                acc.y = fmaf(x, v.y, acc.y);
                acc.z = fmaf(x, v.z, acc.z);
                acc.w = fmaf(x, v.w, acc.w);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const int32_t tok = p.by_group.quotient(g.r0 + r), hh = (g.r0 + r) - tok * p.group, head = g.head * p.group + hh;
    const float inv = inverse(l, g.pos0 + tok);
    const int64_t row = w_row(w, tok);
    if (lane * 4 < p.head_dim)
        *reinterpret_cast<uint2 *>(p.out + row * p.out_token_stride + head * p.out_head_stride + lane * 4) =
            make_uint2(E::pack(acc.x * inv, acc.y * inv), E::pack(acc.z * inv, acc.w * inv));
    if (p.lse && lane == 0) p.lse[row * p.n_heads + head] = lse_of(m, l);
}

}  // namespace rows
}  // namespace attn
}  // namespace engram
