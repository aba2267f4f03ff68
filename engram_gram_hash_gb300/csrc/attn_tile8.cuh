// Attention over the 8-bit cache for many query rows per key/value head
// (prompts, chunks): the tile kernel's items, plan, products and join, on tiles
// that four more warps make from the codes.
//
// The products run on 16-bit tiles (codes are exact in both types), so a tile's codes are converted first: the fp8 matrix
// instruction wants both operands in 8 bits, and queries and weights would have to be split into two or three
// pieces each.  Two forms:
//   opened   for work with many row blocks over the same keys a kernel makes the tiles of every sequence and head
//            once, in the workspace, in the order of the ring's stages, and a stage is two plain bulk copies (a prompt
//            of 8,192 tokens has 128 row blocks a head: its tiles are converted once instead of 65 times in the mean);
//   in place for fewer, four more warps convert each tile that the CTA meets.
// Opened, bound as the 16-bit kernel by the softmax's chain beside the tensor pipe, longer by the strips' factors:
// a prompt of 8,192 tokens, 32 / 8 heads of 128, 415 us (1,325 TFLOP/s, 70 % of the burst rate; about 12 are the
// opening), 2,048 more over 63,488 cached 1,515-1,580 (1,430-1,370 TFLOP/s, the clock falls in long runs), 64 values 335; the 16-bit kernel takes 360, 1,400 and
// 317.  Keys are opened in the queries' type, values as fp16: with keys in fp16 too, bf16 queries had to be converted
// between items (434 us).  Tried and left: half of a tile's factors in registers 422-427, codes brought to one
// scale a tile and a second form of the softmax for such tiles 465 (then 440).
// In place, bound by the converters and the softmax beside them: 541 and 2,090 us; a pair of row tiles takes 4,600
// cycles of an SM, 3,000 on 16-bit tiles.  By a clock trace the converters are busy all that time (1,500 cycles a
// tile of keys or values, most of it the latency of one load and store after another); loading eight pieces ahead
// takes them to 950, but both softmaxes then fall into step, share the issue slots and the period grows to 5,400.
// Tried and left: codes from global memory straight into the converters' registers (649 us: too few bytes in
// flight), two threads a row in the softmax (732), scores read twice from TMEM in rolled loops (572), factors kept in
// registers (575), strips brought to one scale while converting (546, and inexact), row tile 1 held half a period
// behind (592).
//
// Beside the roles of the 16-bit kernel (softmax, products, loads, items), in place:
//   warps 12-15   wait for a tile of codes (a stage of keys and one of values, 16 KB
//                 each), convert a quarter of its keys each and store them as
//                 the products read them (four stages of 32 KB; three: 565 us).
//                 They also clear what the products must not meet: values of
//                 keys that no row reaches, NaN in tiles that some row sees
//                 only part of.
//   Scales come with their tile of keys (asynchronous copies, counted by its
//   barrier); a converter turns them into the factor, log2 and inverse that the
//   softmax reads, a strip of 16 keys at a time.
// The memory through which the 16-bit kernel's rows change hands on their way
// out went to the ring: a lane stores its own row, 32 bytes at a time.
#pragma once

#include <type_traits>

namespace engram {
namespace attn {
namespace tile {

constexpr int NUM_THREADS8 = 512;
constexpr int CONVERTERS = 4;
constexpr int STRIPS = KT / STRIP;  // scales of a tile
template <int DP>
struct Cfg8 : Cfg<DP> {
    static constexpr int RAW_BYTES = KT * DP;  // codes of K or V of a tile
    static constexpr int RAW_STAGES = DP == 128 ? 2 : 4;
    static_assert(RAW_STAGES % 2 == 0, "keys and values by turns");
    // Tiles whose factors are kept.  Tile f's are written when the ring has room for its keys: the values up to tile
    // f - (STAGES + 2) / 2 have then been used by both row tiles, so their softmaxes are done with the factors.
    static constexpr int FACTORS = DP == 128 ? 4 : 8;
    static_assert(FACTORS >= (Cfg<DP>::STAGES + 2) / 2, "factors' ring");
};

template <int DP>
struct Shared8 {
    uint64_t kv_full[Cfg8<DP>::STAGES];
    uint64_t kv_empty[Cfg8<DP>::STAGES];
    uint64_t raw_full[Cfg8<DP>::RAW_STAGES];
    uint64_t raw_empty[Cfg8<DP>::RAW_STAGES];
    uint64_t fac_full[Cfg8<DP>::FACTORS];
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
    float4 fac[Cfg8<DP>::FACTORS][STRIPS];  // of a strip: the scores' factor, log2 of the value scale, its inverse
    float scales[Cfg8<DP>::RAW_STAGES / 2][2][STRIPS];
    Item items[ITEMS];
    uint32_t tmem_base;
    int abort;
    PlanShared plan;
};

template <int DP, bool OPEN>
constexpr int smem8_bytes() {
    return 2 * Cfg8<DP>::Q_BYTES + Cfg8<DP>::STAGES * Cfg8<DP>::STAGE_BYTES +
           (OPEN ? 0 : Cfg8<DP>::RAW_STAGES * Cfg8<DP>::RAW_BYTES) + (int)sizeof(Shared8<DP>);
}
static_assert(smem8_bytes<128, false>() <= 232448 && smem8_bytes<64, false>() <= 232448, "tile kernel shared memory over the per-CTA limit");

// The sequences' keys (in the queries' type) and values (fp16), in the order of the ring's stages: for each sequence and head the keys' 64
// values at a time (rows of 128 bytes, swizzled over 8 keys), the values' likewise, then the strips' factors.
struct Opened {
    uint8_t *at;
    int64_t keys;  // of a sequence and head: the block table's room, rounded up to tiles, and a tile of zeros
};
template <int DP>
__host__ __device__ constexpr int64_t opened_bytes(int64_t keys) { return keys * (4 * DP + (int)sizeof(float4) / STRIP); }

struct Params8 {
    Params t;  // values: unused
    Scales scales;
    CodePages codes;
    Divisor by_page;
    Opened opened;  // at null: none
};

__device__ __forceinline__ uint2 lds8(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
// 32 bytes to global memory, as one piece (32-byte aligned) or two.
__device__ __forceinline__ void store32(void *to, const uint32_t *v, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}
// A strip's factor for a row.  Not 0 (a key scale may be): a hidden score, -inf, must stay that.
__device__ __forceinline__ float factor(float strip, float row) { return fmaxf(strip * row, 7.5231638452626401e-37f); }

// 16-byte aligned global memory into shared memory, asynchronously, counted in bytes by the barrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

struct OpenParams {
    Batch b;
    const uint8_t *k, *v;
    int64_t page_stride, slot_stride, head_stride;
    Scales scales;
    Divisor by_page;
    Opened opened;
    int64_t units;  // sequences x tiles x kv heads x 2
    int32_t tiles, n_kv_heads, head_dim, window;
    float scale_log2;
};
constexpr int OPEN_THREADS = 256;
constexpr int OPEN_PER_SM = 6;
// A tile of keys (in the queries' type), or of values (fp16), of one sequence and head into the opened memory; with the values the strips'
// factors, log2 and inverse, and whether a value was NaN.  Keys that no token of the sequence sees become zeros, NaN
// values too.  Bound: memory (1 byte in, 2 out a code).
template <typename E, int DP>
__global__ void __launch_bounds__(OPEN_THREADS, OPEN_PER_SM) open_kernel(const OpenParams p) {
    __shared__ int bad[STRIPS];
    grid_dependency_wait();
    allow_dependent_launch();
    const int64_t base = __ldg(p.b.offs);
    constexpr int PIECES = DP / 16;                   // 16 codes each, of a key
    constexpr int EACH = KT * PIECES / OPEN_THREADS;  // a thread's
    const int ch = threadIdx.x % PIECES;
    for (int64_t u = blockIdx.x; u < p.units; u += gridDim.x) {
        const int kv = (int)(u & 1);
        const int64_t tile_of = (u >> 1) / p.n_kv_heads, s = tile_of / p.tiles;
        const int32_t head = (int32_t)((u >> 1) - tile_of * p.n_kv_heads), key0 = (int32_t)(tile_of - s * p.tiles) * KT;
        const Seq q = load_seq(p.b, s, base);
        const int32_t lo = first_seen(q.kv - q.q_len, p.window), hi = q.kv;
        // With a window an item's tiles begin on any box of a page, so its last one may end in the tile after the last key.
        if (q.q_len == 0 || hi <= 0 || key0 >= hi + (p.window > 0 ? KT : 0) || key0 + KT <= lo) continue;
        const auto page_of = [&](int32_t entry) { return __ldg(p.b.block_table + s * p.b.table_stride + entry); };
        uint8_t *const to = p.opened.at + (s * p.n_kv_heads + head) * opened_bytes<DP>(p.opened.keys);
        const uint8_t *const codes = (kv ? p.v : p.k) + head * p.head_stride + ch * 16;
        uint4 c[EACH];
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int32_t key = key0 + (i * OPEN_THREADS + threadIdx.x) / PIECES;
            c[i] = make_uint4(0, 0, 0, 0);
            if (key >= lo && key < hi) {
                const int32_t entry = p.by_page.quotient(key), page = page_of(entry);
                if (page < 0 || page >= p.b.n_pages)
                    raise_error(ENGRAM_ERANGE);
                else if (ch * 16 < p.head_dim)
                    c[i] = *reinterpret_cast<const uint4 *>(codes + page * p.page_stride + (key - entry * p.b.page_size) * p.slot_stride);
            }
        }
        float ks = 0.f, vs = 0.f;
        if (kv) {  // the same for the block
            if (threadIdx.x < STRIPS) {
                const int32_t key = key0 + threadIdx.x * STRIP;
                if (key < hi && key + STRIP > lo) {
                    const int32_t entry = p.by_page.quotient(key), page = page_of(entry);
                    if (page >= 0 && page < p.b.n_pages) {
                        const int64_t at = ((int64_t)page * p.n_kv_heads + head) * p.scales.per_page +
                                           ((key - entry * p.b.page_size) >> p.scales.block_log2);
                        ks = p.scales.k[at];
                        vs = p.scales.v[at];
                    }
                }
                bad[threadIdx.x] = 0;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                if (nan_codes(c[i].x) | nan_codes(c[i].y) | nan_codes(c[i].z) | nan_codes(c[i].w))
                    bad[(i * OPEN_THREADS + threadIdx.x) / PIECES / STRIP] = 1;
                c[i] = make_uint4(without_nan(c[i].x), without_nan(c[i].y), without_nan(c[i].z), without_nan(c[i].w));
            }
        }
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int32_t key = key0 + (i * OPEN_THREADS + threadIdx.x) / PIECES;
            uint8_t *const row = to + ((int64_t)(kv * (DP / 64) + (ch >> 2)) * p.opened.keys + key) * 128;
            const int at = (ch & 3) * 2, swizzle = key & 7;
            uint32_t x[8] = {codes_lo(c[i].x), codes_hi(c[i].x), codes_lo(c[i].y), codes_hi(c[i].y),
                             codes_lo(c[i].z), codes_hi(c[i].z), codes_lo(c[i].w), codes_hi(c[i].w)};
            if (std::is_same<E, Bf16>::value && !kv) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 f = Fp16::unpack(x[k]);
                    x[k] = E::pack(f.x, f.y);
                }
            }
            *reinterpret_cast<uint4 *>(row + ((at ^ swizzle) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<uint4 *>(row + (((at + 1) ^ swizzle) << 4)) = make_uint4(x[4], x[5], x[6], x[7]);
        }
        if (kv) {
            __syncthreads();
            if (threadIdx.x < STRIPS) {
                const float2 f = value_scale(vs);
                reinterpret_cast<float4 *>(to + p.opened.keys * 4 * DP)[key0 / STRIP + threadIdx.x] =
                    make_float4(factor(ks, p.scale_log2), f.x, f.y, bad[threadIdx.x] ? 1.f : 0.f);
            }
            // (a thread clears its own mark next)
        }
    }
}

template <typename E, int DP, bool OPEN>
__global__ void __launch_bounds__(OPEN ? NUM_THREADS : NUM_THREADS8, 1)
    tile8_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                const __grid_constant__ Params8 p8) {
    using C = Cfg8<DP>;
    using H = Fp16;  // of the second product (in place, of both)
    constexpr int FACTORS = C::FACTORS, MAKERS = OPEN ? 0 : CONVERTERS;
    const Params &p = p8.t;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *q_smem = smem;
    uint8_t *kv_smem = smem + 2 * C::Q_BYTES;
    uint8_t *raw_smem = kv_smem + C::STAGES * C::STAGE_BYTES;
    Shared8<DP> *sh = reinterpret_cast<Shared8<DP> *>(raw_smem + (OPEN ? 0 : C::RAW_STAGES * C::RAW_BYTES));
    volatile int *abort = &sh->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if ((smem_u32(smem) & 1023u) != 0) {  // the same for every CTA
        grid_dependency_wait();
        if (threadIdx.x == 0) raise_error(ENGRAM_EUNSUPPORTED);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&sh->kv_full[i], OPEN ? 1 : CONVERTERS);
            mbar_init(&sh->kv_empty[i], 2);  // both row tiles' products
        }
        for (int i = 0; i < C::RAW_STAGES; ++i) {
            mbar_init(&sh->raw_full[i], i % 2 == 0 ? 1 + 2 * STRIPS : 1);  // keys bring both scales
            mbar_init(&sh->raw_empty[i], CONVERTERS);
        }
        for (int i = 0; i < FACTORS; ++i) mbar_init(&sh->fac_full[i], 1);
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
            mbar_init(&sh->item_empty[i], 11 + MAKERS);  // eight softmax warps, two MMA warps, the load warp and the converters
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
        make_plan<OPEN ? NUM_THREADS : NUM_THREADS8>(p, base, &sh->plan);  // synchronises the block
        if (blockIdx.x == 0 && threadIdx.x == 0 && p.cut) *p.cut = sh->plan.cut;
    }
    tc_fence_after();
    const uint32_t tmem = sh->tmem_base;

    // Item number i of this CTA, for a whole warp: every role takes all of them in order (null after a time-out).
    const auto take = [&](uint32_t i) -> const Item * {
        return warp_wait(&sh->item_full[i % ITEMS], (i / ITEMS) & 1, abort) ? &sh->items[i % ITEMS] : nullptr;
    };

    // Registers move from the other warps to the softmax warps, which hold a row of 128 scores each:
    // 256 x 192 + 128 x 72 + 128 x 56 = the launch's 512 x 128, 256 x 208 + 128 x 88 = 384 x 168.
    if (warp < 8) {  // ------------------------------------------------- softmax
        if (OPEN)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        const int t = warp >> 2;                  // row tile
        const int row = (warp & 3) * 32 + lane;   // row of the tile: this thread's TMEM lane
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tm = tmem + lanes + t * KT, o_tm = tmem + lanes + C::O_COL + t * DP;
        const uint32_t p_tm = C::APART ? tmem + lanes + C::P_COL + t * 64 : s_tm;
        constexpr float LIFT = H::LIFT - H::RESCALE;  // of a weight at the running maximum
        uint32_t s_ph = 0, o_ph = 0, it = 0, pv_ph = 0;  // it: tiles before the item
        // Factors in registers: 853 -> 817 us (2,048 new over 30,720); at 64 values, beside the second score buffer's
        // registers, 336 -> 364 (a prompt of 8,192).
        constexpr bool AHEAD = OPEN && !C::APART;
        float rf = 1.f;  // what this thread's row of queries was divided by
        const auto of_row = [&](float strip) { return OPEN ? strip : factor(strip, rf); };
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
            if (!OPEN && std::is_same<E, Bf16>::value) {  // this thread's row as fp16: exact but for values below 2^-28 of its largest
                __syncwarp();  // the warp's lanes have copied each other's rows
                const uint32_t at = smem_u32(q_smem) + t * C::Q_BYTES + row * 128;
                const auto piece = [&](int i) { return at + (i >> 3) * (MT * 128) + (((i ^ row) & 7) << 4); };
                // Pieces loaded together: one after another each waits out its load (5,000 cycles an item).  All at
                // once is best at 128 values (a prompt of 8,192 tokens, in place, 541 us; four 548); at 64 it costs the
                // softmax registers (470 us; four 428).
                constexpr int BATCH = C::APART ? 4 : DP / 8;
                float most = 0.f;
#pragma unroll 1
                for (int i = 0; i < DP / 8; i += BATCH) {
                    uint4 v[BATCH];
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) v[k] = lds16(piece(i + k));
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const uint32_t x[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                        for (int c = 0; c < 4; ++c) most = max3(most, fabsf(bf16_lo(x[c])), fabsf(bf16_hi(x[c])));
                    }
                }
                const int e = row_exponent<14>(most);
                const float up = exp2i(e);
                rf = exp2i(-e);
                const auto half = [&](uint32_t x) { return H::pack(bf16_lo(x) * up, bf16_hi(x) * up); };
#pragma unroll 1
                for (int i = 0; i < DP / 8; i += BATCH) {
                    uint4 v[BATCH];
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) v[k] = lds16(piece(i + k));
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) sts16(piece(i + k), make_uint4(half(v[k].x), half(v[k].y), half(v[k].z), half(v[k].w)));
                }
            }
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
            float m = -INFINITY, l = 0.f;  // m: the exponent that the weights refer to
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
                    const uint32_t f = it + j;
                    const float4 *const fac = sh->fac[f % FACTORS];
                    float nan_in = 0.f;  // OPEN: whether values of the tile were NaN
                    // AHEAD: the strips' factors come into registers before the scores are waited for.  (Not an item's
                    // first: a row tile that passed items over may be phases behind the factors' barriers until its
                    // scores are there.)
                    float kf[STRIPS], yf[STRIPS];
                    const auto fetch = [&] {
                        ok = warp_wait(&sh->fac_full[f % FACTORS], (f / FACTORS) & 1, abort);
                        if constexpr (AHEAD) {
#pragma unroll
                            for (int c = 0; c < STRIPS; ++c) {
                                const float4 g = fac[c];
                                kf[c] = g.x, yf[c] = g.y;
                                nan_in += g.w;
                            }
                        }
                    };
                    if (AHEAD && j > 0) {
                        fetch();
                        if (!ok) break;
                    }
                    ok = warp_wait(&sh->s_full[t], s_ph++ & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    if (!AHEAD || j == 0) {
                        fetch();
                        if (!ok) break;
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
                    float mx = -INFINITY;  // of the exponents u = s F + log2 vs
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
                        float part[4];  // a strip each: independent chains
#pragma unroll
                        for (int i = 0; i < STRIP; i += 2)
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const float u = s[h * 64 + c * STRIP + i], v = s[h * 64 + c * STRIP + i + 1];
                                part[c] = i == 0 ? fmaxf(u, v) : max3(part[c], u, v);
                            }
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if constexpr (AHEAD) {
                                part[c] = fmaf(part[c], kf[h * 4 + c], yf[h * 4 + c]);
                            } else {
                                const float4 g = fac[h * 4 + c];
                                part[c] = fmaf(part[c], of_row(g.x), g.y);
                                if (OPEN) nan_in += g.w;
                            }
                        }
                        mx = max3(mx, part[0], part[1]);
                        mx = max3(mx, part[2], part[3]);
                    }
                    if (C::APART) {  // the tile before is in O, its weights are used (before the first there is none)
                        ok = warp_wait(&sh->pv_done[t], pv_ph ^ 1, abort);
                        pv_ph ^= 1;
                        if (!ok) break;
                        tc_fence_after();
                    }
                    float up = 1.f;
                    if (mx - m > H::RESCALE) {  // also from -inf
                        up = rows::exp2_approx(m - mx);
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
                    if (OPEN && nan_in != 0.f) {  // the same in every lane
                        if (lane == 0) {
                            Item *const note = const_cast<Item *>(w);
                            atomicMin(&note->bad_lo, j);
                            atomicMax(&note->bad_hi, j);
                            __threadfence_block();
                        }
                        __syncwarp();
                    }
                    const float mref = m == -INFINITY ? 0.f : m - LIFT;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t pk[16];
#pragma unroll
                        for (int g = 0; g < 2; ++g) {  // a strip: one factor, one scale
                            const float4 fa = fac[2 * c + g];
                            const float k = AHEAD ? kf[2 * c + g] : of_row(fa.x), at = (AHEAD ? yf[2 * c + g] : fa.y) - mref;
                            const float2 sc = make_float2(k, k), off = make_float2(at, at);
                            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                            for (int i = 8 * g; i < 8 * g + 8; ++i) {
                                float2 x = fma2(make_float2(s[c * 32 + 2 * i], s[c * 32 + 2 * i + 1]), sc, off);
                                x.x = rows::exp2_approx(x.x);
                                x.y = rows::exp2_approx(x.y);
                                sum = i == 8 * g ? x : add2(sum, x);
                                pk[i] = H::pack(x.x, x.y);  // 16-bit operands of the second product
                            }
                            l = fmaf(sum.x + sum.y, fa.z, l);
                        }
                        tmem_st_32x32b_x16(p_tm + c * 16, pk);
                        if ((c + 1) % (4 / P_PARTS) == 0) {  // the second product may start on these keys
                            tmem_st_wait();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&sh->p_ready[t][c * P_PARTS / 4]);
                        }
                    }
                }
                if (!ok) break;
            }
            it += n;
            if (mine && n > 0) {
                // The last scores were there, so the queries' memory is free: the next item's are fetched
                // under this item's last product, and its scores computed under this item's epilogue.  (Handed over before
                // that product too they were worth 1 % of a long prompt and cost 9 % of a window of 128 tokens.)
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
                const int64_t dst = out_row * p.out_token_stride + (int64_t)head * p.out_head_stride;
                float *part = p.part_o + (slot * ROWS + t * MT + row) * DP;
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
                        const int32_t key_lo = max(first_seen(pos, p.window), w->key0 + w->bad_lo * KT);
                        const int32_t key_hi = min(pos + 1, w->key0 + (w->bad_hi + 1) * KT);
                        if (OPEN) {
                            const float4 *const strips = reinterpret_cast<const float4 *>(
                                p8.opened.at + (w->s * p.n_kv_heads + w->head) * opened_bytes<DP>(p8.opened.keys) + p8.opened.keys * 4 * DP);
                            for (int32_t k0 = key_lo & ~(STRIP - 1); k0 < key_hi; k0 += STRIP)
                                if (strips[k0 / STRIP].w != 0.f)
                                    add_nan<32>(p.b, p8.codes, w->s, w->head, max(key_lo, k0), min(key_hi, k0 + STRIP), c, p.head_dim, x);
                        } else {
                            add_nan<32>(p.b, p8.codes, w->s, w->head, key_lo, key_hi, c, p.head_dim, x);
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(x[i]);
                    }
                };
                // A lane stores its row's values itself, 32 bytes at a time where the rows begin on such a boundary: the
                // ring takes the memory through which the 16-bit kernel's rows change hands.
                if (whole) {
                    const bool wide = ((reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.out_token_stride * 2) |
                                        (uintptr_t)(p.out_head_stride * 2)) & 31) == 0;
#pragma unroll 1
                    for (int c = 0; c < DP; c += 32) {
                        uint32_t o[32];
                        read_o(c, o);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t u[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                u[i] = E::pack(__uint_as_float(o[h * 16 + 2 * i]) * inv, __uint_as_float(o[h * 16 + 2 * i + 1]) * inv);
                            if (live && c + h * 16 < p.head_dim) store32(p.out + dst + c + h * 16, u, wide);  // head_dim % 16 == 0
                        }
                    }
                } else if (n > 0) {
#pragma unroll 1
                    for (int c = 0; c < DP; c += 32) {
                        uint32_t o[32];
                        read_o(c, o);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (live) store32(part + c + i * 8, o + i * 8, true);
                    }
                }
                tc_fence_before();  // O has been read before the next item's first product is allowed
                if (live) {
                    const float m2 = m == -INFINITY ? -INFINITY : m - LIFT;
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
    } else if (!OPEN && warp >= 12) {  // ----------------------- codes to fp16 tiles
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const int part = warp - 12;  // a quarter of each tile's keys
        constexpr int LPK = DP / 8, KEYS = 32 / LPK;  // lanes a key (8 codes each), keys at a time
        const int ch = lane % LPK, key = part * 32 + lane / LPK;
        const uint32_t src = smem_u32(raw_smem) + key * DP + ch * 8;
        const uint32_t dst = smem_u32(kv_smem) + (ch >> 3) * (KT * 128) + key * 128;
        uint32_t it = 0;  // tiles of keys and values by turns
        bool ok = true;
        for (uint32_t i = 0; ok; ++i) {
            const Item *const item = take(i);
            if (!item || item->n_rows == 0) break;
            const int32_t n = item->n, lo = item->lo, hi = item->hi, full_lo = item->full_lo, full_hi = item->full_hi;
            for (int32_t j = 0; ok && j < n; ++j) {
                const int32_t key0 = item->key0 + j * KT;
                const bool edge = key0 < full_lo || key0 + KT > full_hi;
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++it) {
                    const uint32_t r = it % C::RAW_STAGES, st = it % C::STAGES;
                    ok = warp_wait(&sh->raw_full[r], (it / C::RAW_STAGES) & 1, abort);
                    if (!ok) break;
                    ok = it < C::STAGES || warp_wait(&sh->kv_empty[st], ((it / C::STAGES) - 1) & 1, abort);
                    if (!ok) break;
                    if (kv == 0 && part == 0) {  // the tile's factors
                        const uint32_t f = it / 2;
                        if (lane < STRIPS) {
                            const float2 vs = value_scale(sh->scales[r / 2][1][lane]);
                            sh->fac[f % FACTORS][lane] = make_float4(sh->scales[r / 2][0][lane] * p.scale_log2, vs.x, vs.y, 0.f);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh->fac_full[f % FACTORS]);
                    }
                    const uint32_t from = src + r * C::RAW_BYTES, to = dst + st * C::STAGE_BYTES;
                    uint32_t bad = 0;
#pragma unroll 8
                    for (int g = 0; g < 32; g += KEYS) {
                        uint2 c = lds8(from + g * DP);
                        // Values that must not meet a weight of zero: those of keys that no row reaches (they may be
                        // anything), NaN of keys that some row does not see (the epilogue adds it to the rows that do).
                        if (kv && edge) {
                            if (key0 + key + g < lo || key0 + key + g >= hi) c = make_uint2(0, 0);
                            bad |= nan_codes(c.x) | nan_codes(c.y);
                            c = make_uint2(without_nan(c.x), without_nan(c.y));
                        }
                        sts16(to + g * 128 + (((ch ^ (key + g)) & 7) << 4),
                              make_uint4(codes_lo(c.x), codes_hi(c.x), codes_lo(c.y), codes_hi(c.y)));
                    }
                    if (bad) {
                        Item *const note = const_cast<Item *>(item);
                        atomicMin(&note->bad_lo, j);
                        atomicMax(&note->bad_hi, j);
                        __threadfence_block();
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh->kv_full[st]);
                        mbar_arrive(&sh->raw_empty[r]);
                    }
                }
            }
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&sh->item_empty[i % ITEMS]);
        }
    } else {
        if (OPEN)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
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
        } else if (OPEN && warp == 9) {  // ------------------------------- opened K, V, factors
            uint32_t it = 0;
            bool ok = true;
            for (uint32_t i = 0; ok; ++i) {
                const Item *const item = take(i);
                if (!item || item->n_rows == 0) break;
                const int32_t n = item->n;
                const uint8_t *const from = p8.opened.at + (item->s * p.n_kv_heads + item->head) * opened_bytes<DP>(p8.opened.keys);
                const int64_t key0 = item->key0;  // on a strip: boxes are whole strips
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->item_empty[i % ITEMS]);
                for (int32_t j = 0; ok && j < n; ++j) {
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv, ++it) {
                        const int st = it % C::STAGES;
                        if (lane == 0) {
                            if (it >= C::STAGES) ok = mbar_wait(&sh->kv_empty[st], ((it / C::STAGES) - 1) & 1, abort);
                            if (ok) {
                                mbar_arrive_expect_tx(&sh->kv_full[st], C::STAGE_BYTES);
#pragma unroll
                                for (int c = 0; c < DP / 64; ++c)
                                    bulk_load(smem_u32(kv_smem) + st * C::STAGE_BYTES + c * KT * 128,
                                              from + ((kv * (DP / 64) + c) * p8.opened.keys + key0 + j * KT) * 128, KT * 128, &sh->kv_full[st]);
                                if (kv == 0) {
                                    const uint32_t f = it / 2 % FACTORS;
                                    mbar_arrive_expect_tx(&sh->fac_full[f], STRIPS * (int)sizeof(float4));
                                    bulk_load(smem_u32(sh->fac[f]), from + p8.opened.keys * 4 * DP + (key0 + j * KT) / STRIP * (int)sizeof(float4),
                                              STRIPS * (int)sizeof(float4), &sh->fac_full[f]);
                                }
                            }
                        }
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (!ok) break;
                    }
                }
            }
            if (lane == 0) {  // never leave with a copy still landing (also after an abort elsewhere)
                int no_abort = 0;
                for (uint32_t i = it < C::STAGES ? 0 : it - C::STAGES; i < it; ++i) {
                    mbar_wait(&sh->kv_full[i % C::STAGES], (i / C::STAGES) & 1, &no_abort, 200000000ull);
                    if (i % 2 == 0) mbar_wait(&sh->fac_full[i / 2 % FACTORS], (i / 2 / FACTORS) & 1, &no_abort, 200000000ull);
                }
            }
        } else if (warp == 9) {  // --------------------------------------- codes of K, V
            const int box_log2 = 31 - __clz(p.box), boxes = KT >> box_log2;  // the box divides 128
            const uint32_t box_bytes = (uint32_t)p.box * DP;
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
                // keys in 32 bits without sign: the boxes looked up ahead may lie past 2^31
                int32_t window0 = -1;
                int32_t page = -1;
                for (int32_t j = 0; ok && j < w.n; ++j) {
                    const int32_t b0 = (w.key0 >> box_log2) + j * boxes;
                    if (window0 < 0 || b0 + boxes > window0 + 32) {  // the pages of the next 32 boxes, a lane each
                        window0 = b0;
                        const uint32_t ahead = (uint32_t)(b0 + lane) << box_log2;
                        page = -1;
                        if (ahead < (uint32_t)w.hi) {
                            page = __ldg(p.b.block_table + w.s * p.b.table_stride + p8.by_page.quotient((int32_t)ahead));
                            if (page < 0 || page >= p.b.n_pages) {
                                if (ahead + p.box > (uint32_t)w.lo) raise_error(ENGRAM_ERANGE);
                                page = -1;  // out of range: the copy fills zeros
                            }
                        }
                    }
                    const int32_t mine = __shfl_sync(0xffffffffu, page, (b0 - window0) + (lane < boxes ? lane : 0));
                    const uint32_t key = (uint32_t)(b0 + lane) << box_log2;
                    const bool load = lane < boxes && key < (uint32_t)w.hi && key + p.box > (uint32_t)w.lo;
                    const uint32_t loads = __popc(__ballot_sync(0xffffffffu, load));
                    const int y = load ? (int)key - p8.by_page.quotient((int32_t)key) * p.b.page_size : 0;
                    // lanes 0..7 copy the strips' key scales, 8..15 their value scales
                    const int sl = lane & (STRIPS - 1);
                    const int32_t strip_page = __shfl_sync(0xffffffffu, page, (b0 - window0) + ((sl * STRIP) >> box_log2));
                    const uint32_t strip = ((uint32_t)b0 << box_log2) + sl * STRIP;
                    const bool has_scale = strip < (uint32_t)w.hi && strip + STRIP > (uint32_t)w.lo && strip_page >= 0;
                    const int32_t block = ((int32_t)strip - p8.by_page.quotient((int32_t)strip) * p.b.page_size) >> p8.scales.block_log2;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++it) {
                        const int st = it % C::RAW_STAGES;
                        if (lane == 0) {
                            if (it >= C::RAW_STAGES) ok = mbar_wait(&sh->raw_empty[st], ((it / C::RAW_STAGES) - 1) & 1, abort);
                            if (ok) mbar_arrive_expect_tx(&sh->raw_full[st], loads * box_bytes);
                        }
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (!ok) break;
                        if (load)
                            rows::tma_load_4d(raw_smem + st * C::RAW_BYTES + lane * p.box * DP, kv ? &v_map : &k_map,
                                              &sh->raw_full[st], 0, y, w.head, mine);
                        if (kv == 0 && lane < 2 * STRIPS) {
                            copy4_async(smem_u32(&sh->scales[st / 2][lane / STRIPS][sl]),
                                        (lane < STRIPS ? p8.scales.k : p8.scales.v) +
                                            (has_scale ? ((int64_t)strip_page * p.n_kv_heads + w.head) * p8.scales.per_page + block : 0),
                                        has_scale);
                            arrive_when_copied(&sh->raw_full[st]);
                        }
                    }
                }
            }
            if (lane == 0) {  // never leave with a copy still landing (also after an abort elsewhere)
                int no_abort = 0;
                for (uint32_t i = it < C::RAW_STAGES ? 0 : it - C::RAW_STAGES; i < it; ++i)
                    mbar_wait(&sh->raw_full[i % C::RAW_STAGES], (i / C::RAW_STAGES) & 1, &no_abort, 200000000ull);
            }
        } else {  // warps 8, 11 ---------------------------------- MMAs of row tile t
            // The whole warp walks the tiles with warp-uniform values (the instruction takes its
            // descriptors from uniform registers) and one elected lane issues.  Issuing blocks while
            // the tensor pipe has a few products waiting, so each row tile has a warp of its own that
            // waits for weights and keys meanwhile; the two take strict turns (turn[t]).  Without the
            // turns their products interleave, both softmaxes then run at once and both wait for the
            // tensor pipe at once (65,536-token chunk: 1.99 ms; one warp for both tiles 1.64 ms).
            const int t = warp == 8 ? 0 : 1;
            constexpr uint32_t ID_S = idesc_16(OPEN && std::is_same<E, Bf16>::value, MT, KT, false), ID_O = idesc_16(false, MT, DP, true);
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
                        mma_commit(&sh->kv_empty[v]);  // before the scores: the keys after next wait for it
                        if (!more)
                            mma_commit(&sh->o_full[t]);
                        else if (!C::APART)
                            scores();
                        if (!C::APART && both) mbar_arrive(&sh->turn[t ^ 1]);
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

}  // namespace tile
}  // namespace attn
}  // namespace engram
