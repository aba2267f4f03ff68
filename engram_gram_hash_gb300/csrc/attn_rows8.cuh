// Attention over the 8-bit cache for few query rows per key/value head (single
// tokens and short chunks): the rows kernel's plan, ring and joins over tiles
// of codes, 8 rows a segment.
//
// Bound: the bytes of the codes, half the 16-bit cache's, if a tile costs the
// warps few enough instructions: the conversion of the codes is most of them.
// Both products therefore have the cache as the matrix instruction's first
// operand (mma.sync m16n8k16 on fp16), S^T = K Q^T and O^T = V^T P^T, whose 16 rows
// are all keys or values, and the 8 query rows as the second: 8 rows instead of
// 16 in the accumulators of the softmax, and no row of an instruction is empty.
// (mma.sync on e4m3 itself is no way around it: it took as long as two fp16
// ones and the conversions of both operands.)  Between the products the
// weights change from keys by lanes to rows by lanes, 8 x 8 at a time, by
// movmatrix.  Queries are exact in fp16: a row is multiplied by the power of two
// that brings its largest value to 2^14 .. 2^15 (below 2^-28 of it values lose
// bits).
// A warp has a quarter of a tile (128 keys, 32 KB of K and V at 128 values) and
// every value's order within the products is free, so a lane's four codes are
// neighbours in memory: two conversions for them, and for V, whose pairs lie
// across keys, a byte permutation.  The strips' scales travel with their tile:
// 4-byte asynchronous copies that the tile's barrier counts.
// 64 sequences of up to 16,384 tokens, 32 / 8 heads of 128: 173-176 us, 96-97 % of
// the copy rate; 131,072 tokens of one 51 us, 77 % (launch, first loads and the
// join take 11); 512 tokens, 4 / 2 heads of 64, 5.9 us in a CUDA graph.
#pragma once

namespace engram {
namespace attn {
namespace rows {

constexpr int ROWS8 = 8;               // query rows per segment
constexpr int GROUPS = 2;              // groups of four consumer warps, which take tiles in turn
constexpr int CONSUMERS8 = 4 * GROUPS;
constexpr int NUM_THREADS8 = 32 * (CONSUMERS8 + 4);
constexpr int KT8 = 128;               // keys per tile
constexpr int STRIPS = KT8 / STRIP;    // scales of a tile

template <int DP>
struct Cfg8 {
    static constexpr int KT_LOG2 = 7, KT = KT8;
    static constexpr int KPW = KT / 4;          // keys per warp
    static constexpr int KV_BYTES = KT * DP;    // K (or V) of a tile
    static constexpr int STAGE_BYTES = 2 * KV_BYTES;
    static constexpr int STAGES = 196608 / STAGE_BYTES;
    static_assert(STAGES % GROUPS == 0, "each ring stage must belong to one consumer group");
    static constexpr int JOIN_FLOATS = 4 * ROWS8 * DP;
};

// Shared memory of piece ch (16 codes) of a tile's key, swizzled by TMA: rows of 128 bytes, or two of 64.
template <int DP>
__device__ __forceinline__ uint32_t piece_at(int key, int ch) {
    return DP == 128 ? key * 128 + (((ch ^ key) & 7) << 4) : key * 64 + (((ch ^ (key >> 1)) & 3) << 4);
}
// Float c of row r in a join buffer: the rows' 32-byte pieces are rotated, so that the accumulators' layout (4
// rows x 4 pairs of values a half warp) meets different banks.
template <int DP>
__device__ __forceinline__ int join8_at(int r, int c) { return r * DP + (c ^ (((r >> 1) & 3) * 8)); }

// An 8 x 8 matrix of 16-bit values, two neighbours of row lane / 4 a lane: transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int DP>
struct Shared8 {
    uint64_t full[Cfg8<DP>::STAGES];
    uint64_t empty[Cfg8<DP>::STAGES];
    float scales[Cfg8<DP>::STAGES][2][STRIPS];
    float m[CONSUMERS8][ROWS8];
    float l[CONSUMERS8][ROWS8];
    int64_t scan[NUM_THREADS8 / 32];
    int64_t find_s;
    int64_t find_before;
    uint64_t ready, done;
    float tm[ROWS8], tl[ROWS8];
    int32_t bad_lo[2], bad_hi[2];  // tiles in which NaN was cleared; two segments in turn
    int abort;
};
__device__ __forceinline__ void consumers8_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * CONSUMERS8) : "memory"); }

template <int DP>
constexpr int smem8_bytes() {
    return Cfg8<DP>::STAGES * Cfg8<DP>::STAGE_BYTES + Cfg8<DP>::JOIN_FLOATS * 4 + (int)sizeof(Shared8<DP>);
}
static_assert(smem8_bytes<128>() <= 232448 && smem8_bytes<64>() <= 232448, "rows kernel shared memory");

struct Params8 {
    Params r;  // values: unused
    Scales scales;
    CodePages codes;
    Divisor by_page;
};

template <typename E, int DP>
__global__ void __launch_bounds__(NUM_THREADS8, 1)
    rows8_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                const __grid_constant__ Params8 p8) {
    const Params &p = p8.r;
    using C = Cfg8<DP>;
    constexpr int KT = C::KT, KPW = C::KPW;
    extern __shared__ __align__(1024) uint8_t smem[];
    float *join = reinterpret_cast<float *>(smem + C::STAGES * C::STAGE_BYTES);
    Shared8<DP> *sh = reinterpret_cast<Shared8<DP> *>(join + C::JOIN_FLOATS);
    volatile int *abort = &sh->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&sh->full[i], 2 + 2 * STRIPS);  // K and V, and their scales
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
    const int32_t line = blockIdx.x / p.cluster % p.side;
    const int64_t index = blockIdx.x / p.cluster / p.side;
    const int rank = p.cluster > 1 ? (int)cluster_ctarank() : 0;
    Plan plan;
    int64_t at_s, at_before;
    if (p.b.n_seqs <= 32) {
        plan = plan_find_small<ROWS8>(p, base, index, at_s, at_before);
        __syncthreads();  // the barriers are initialised
    } else {
        plan = plan_find<NUM_THREADS8, ROWS8>(p, base, index, sh->scan, &sh->find_s, &sh->find_before);
        at_s = sh->find_s;
        at_before = sh->find_before;
    }
    const int64_t f0 = index * plan.run;
    const int64_t f1 = f0 + plan.run < plan.total ? f0 + plan.run : plan.total;
    if (f0 >= f1) return;
    Walk<ROWS8> walk;
    walk.start(p, base, at_s, f0 - at_before, line);
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

    // Registers move to the consumers: 256 x 192 + 128 x 120 = the launch's 384 x 168.
    if (warp >= CONSUMERS8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
        if (warp < CONSUMERS8 + 2) {  // ---------------------- producers: one warp loads K, the next V
            const bool is_v = warp == CONSUMERS8 + 1;
            const CUtensorMap *const map = is_v ? &v_map : &k_map;
            const int box_log2 = 31 - __clz(p.box), boxes = KT >> box_log2;  // the box divides 128
            const uint32_t box_bytes = (uint32_t)p.box * DP;
            const float *const scales = is_v ? p8.scales.v : p8.scales.k;
            for (int64_t f = f0; f < f1;) {
                const Segment g = segment(p, walk);
                int32_t first, end;
                const int32_t n = tiles_of(g, f, first, end);
                // keys in 32 bits without sign: the boxes looked up ahead may lie past 2^31
                int32_t window0 = -1;  // first box whose page lane 0 holds
                int32_t page = -1;
                for (int32_t j = first; j < end; ++j, ++it) {
                    const int32_t tile = g.tile0 + j, b0 = tile * boxes;
                    if (window0 < 0 || b0 + boxes > window0 + 32) {  // the pages of the next 32 boxes, a lane each
                        window0 = b0;
                        const uint32_t ahead = (uint32_t)(b0 + lane) * p.box;
                        page = -1;
                        if (ahead < (uint32_t)g.hi) {
                            page = __ldg(p.b.block_table + walk.s * p.b.table_stride + p8.by_page.quotient((int32_t)ahead));
                            if (page < 0 || page >= p.b.n_pages) {
                                if (ahead + p.box > (uint32_t)g.lo) raise_error(ENGRAM_ERANGE);
                                page = -1;  // out of range: the copy fills zeros
                            }
                        }
                    }
                    const int32_t mine = __shfl_sync(0xffffffffu, page, (b0 - window0) + (lane < boxes ? lane : 0));
                    const uint32_t key = (uint32_t)(b0 + lane) * p.box;
                    const bool load = lane < boxes && key < (uint32_t)g.hi && key + p.box > (uint32_t)g.lo;
                    const uint32_t loads = __popc(__ballot_sync(0xffffffffu, load));
                    // this lane's strip of keys, whose scale it copies
                    const int32_t strip_page = __shfl_sync(0xffffffffu, page, (b0 - window0) + (((lane & (STRIPS - 1)) * STRIP) >> box_log2));
                    const uint32_t strip = (uint32_t)tile * KT + lane * STRIP;
                    const bool has_scale = strip < (uint32_t)g.hi && strip + STRIP > (uint32_t)g.lo && strip_page >= 0;
                    const int st = it % C::STAGES;
                    bool ok = true;
                    if (lane == 0) {
                        if (it >= C::STAGES) ok = mbar_wait(&sh->empty[st], ((it / C::STAGES) - 1) & 1, abort);
                        if (ok) mbar_arrive_expect_tx(&sh->full[st], loads * box_bytes);
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (ok && load) {
                        uint8_t *dst = smem + st * C::STAGE_BYTES + (is_v ? C::KV_BYTES : 0) + lane * p.box * DP;
                        const int y = load ? (int)key - p8.by_page.quotient((int32_t)key) * p.b.page_size : 0;
                        tma_load_4d(dst, map, &sh->full[st], 0, y, g.head, mine);
                    }
                    if (ok && lane < STRIPS) {
                        const int32_t at = (int32_t)strip - p8.by_page.quotient((int32_t)strip) * p.b.page_size;
                        copy4_async(smem_u32(&sh->scales[st][is_v][lane]),
                                    scales + (has_scale ? ((int64_t)strip_page * p.n_kv_heads + g.head) * p8.scales.per_page + (at >> p8.scales.block_log2) : 0),
                                    has_scale);
                        arrive_when_copied(&sh->full[st]);
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
        const int qr = lane >> 2, qc = (lane & 3) * 2;  // this lane's key of each 8; the rows qc and qc + 1 are its own
        int turn = 0;  // segments alternate
        uint32_t exchange_ph = 0;
        for (int64_t f = f0; f < f1; turn ^= 1) {
            const Segment g = segment(p, walk);
            int32_t first, end;
            const int32_t n = tiles_of(g, f, first, end);

            // Query row qr in fp16, of every 16 values the four neighbours that the lane gets of a key.
            uint32_t qf[DP / 16][2];
            // The lane's own rows: what they were divided by, times the scores' factor, and their reach.
            float rf[2];
            int32_t row_lo[2], row_hi[2];
            {
                const int32_t tok = p.by_group.quotient(g.r0 + qr), hh = (g.r0 + qr) - tok * p.group;
                const uint16_t *src = p.q + (int64_t)(w_row(walk, tok)) * p.q_token_stride +
                                      (int64_t)(g.head * p.group + hh) * p.q_head_stride;
                uint2 x[DP / 16];
#pragma unroll
                for (int c = 0; c < DP / 16; ++c) {
                    const int at = c * 16 + (lane & 3) * 4;
                    x[c] = qr < g.n_rows && at < p.head_dim ? __ldg(reinterpret_cast<const uint2 *>(src + at)) : make_uint2(0, 0);
                }
                float most = 0.f;
#pragma unroll
                for (int c = 0; c < DP / 16; ++c) {
                    const float2 u = E::unpack(x[c].x), v = E::unpack(x[c].y);
                    // (an infinity stays; NaN may be lost here, but the row's own NaN remains)
                    most = fmaxf(fmaxf(fmaxf(most, fabsf(u.x)), fabsf(u.y)), fmaxf(fabsf(v.x), fabsf(v.y)));
                }
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
                const int k = row_exponent<14>(most);
                const float up = exp2i(k);
#pragma unroll
                for (int c = 0; c < DP / 16; ++c) {
                    const float2 u = E::unpack(x[c].x), v = E::unpack(x[c].y);
                    qf[c][0] = Fp16::pack(u.x * up, u.y * up);
                    qf[c][1] = Fp16::pack(v.x * up, v.y * up);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    rf[i] = exp2i(-__shfl_sync(0xffffffffu, k, (qc + i) * 4)) * p.scale_log2;
                    const int32_t pos = g.pos0 + p.by_group.quotient(g.r0 + qc + i);
                    row_hi[i] = qc + i < g.n_rows ? pos : -1;
                    row_lo[i] = first_seen(pos, p.window);
                }
            }

            // m, l: of the lane's rows (l its own keys').  O^T: values 16 c + 2 qr (0, 1) and + 1 (2, 3) of these rows.
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
            float o[DP / 16][4];
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

            for (int32_t j = first; j < end; ++j, ++it) {
                if ((int)(it % GROUPS) != grp) continue;
                const int st = it % C::STAGES;
                const bool ok = warp_wait(&sh->full[st], (it / C::STAGES) & 1, abort);
                const int32_t key0 = (g.tile0 + j) * KT + wq * KPW;
                if (ok && key0 < g.hi && key0 + KPW > g.lo) {
                    const uint32_t kb = smem_u32(smem + st * C::STAGE_BYTES) + wq * KPW * DP;
                    // keys outside [full_lo, full_hi) are hidden from some row; keys outside
                    // [lo, hi) may hold anything
                    const bool edge = key0 < g.full_lo || key0 + KPW > g.full_hi;
                    if (edge) {  // this warp's keys are read by no other; a lane looks at one
                        static_assert(KPW == 32, "a key per lane");
                        const uint32_t vrow = kb + C::KV_BYTES;
                        const bool keep = key0 + lane >= g.lo && key0 + lane < g.hi;
                        uint32_t bad = 0;
#pragma unroll
                        for (int c = 0; c < DP / 16; ++c) {
                            const uint4 v = lds16(vrow + piece_at<DP>(lane, c));
                            bad |= nan_codes(v.x) | nan_codes(v.y) | nan_codes(v.z) | nan_codes(v.w);
                        }
                        if (!keep || bad) {
#pragma unroll 1
                            for (int c = 0; c < DP / 16; ++c) {
                                const uint32_t at = vrow + piece_at<DP>(lane, c);
                                const uint4 v = lds16(at);
                                sts16(at, keep ? make_uint4(without_nan(v.x), without_nan(v.y), without_nan(v.z), without_nan(v.w))
                                               : make_uint4(0, 0, 0, 0));
                            }
                            if (keep) {
                                atomicMin(&sh->bad_lo[turn], g.tile0 + j);
                                atomicMax(&sh->bad_hi[turn], g.tile0 + j);
                            }
                        }
                        fence_proxy_async_smem();  // before the ring's next copy over it
                        __syncwarp();
                    }
                    float s[KPW / 16][4];  // keys 16 t + qr (0, 1) and + 8 (2, 3) of rows qc (0, 2) and qc + 1
#pragma unroll
                    for (int t = 0; t < KPW / 16; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
                    {
                        const int key = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
#pragma unroll
                        for (int c = 0; c < DP / 16; c += 2) {
#pragma unroll
                            for (int t = 0; t < KPW / 16; ++t) {
                                uint32_t b[4];  // 8 keys x 16 codes: keys 0..7 and 8..15 of pieces c and c + 1
                                ldmatrix_x4(b, kb + piece_at<DP>(t * 16 + key, c + half));
                                const uint32_t k0[4] = {codes_lo(b[0]), codes_lo(b[2]), codes_hi(b[0]), codes_hi(b[2])};
                                const uint32_t k1[4] = {codes_lo(b[1]), codes_lo(b[3]), codes_hi(b[1]), codes_hi(b[3])};
                                Fp16::mma(s[t], k0, qf[c][0], qf[c][1]);
                                Fp16::mma(s[t], k1, qf[c + 1][0], qf[c + 1][1]);
                            }
                        }
                    }
                    // The tile's values and scales into registers, and its stage back to the ring before the softmax: what
                    // is in flight decides the rate.
                    uint32_t vr[KPW / 16][DP / 32][4];  // pairs of values of keys 0..7 and 8..15, pieces 2 c and 2 c + 1
                    const int vkey = (((lane >> 3) & 1) << 3) + (lane & 7);
#pragma unroll
                    for (int t = 0; t < KPW / 16; ++t)
#pragma unroll
                        for (int c = 0; c < DP / 32; ++c)
                            ldmatrix_x4_trans(vr[t][c], kb + C::KV_BYTES + piece_at<DP>(t * 16 + vkey, 2 * c + (lane >> 4)));
                    float ks[KPW / STRIP], vs[KPW / STRIP];
#pragma unroll
                    for (int t = 0; t < KPW / STRIP; ++t) {
                        ks[t] = sh->scales[st][0][wq * (KPW / STRIP) + t];
                        vs[t] = sh->scales[st][1][wq * (KPW / STRIP) + t];
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->empty[st]);
                    float rs[KPW / STRIP];  // 1 / value scale of a strip
                    float mx[2] = {m[0], m[1]};
#pragma unroll
                    for (int t = 0; t < KPW / STRIP; ++t) {
                        const float2 v = value_scale(vs[t]);
                        rs[t] = v.y;
                        const float f[2] = {rf[0] * ks[t], rf[1] * ks[t]};
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            s[t][c] = fmaf(s[t][c], f[c & 1], v.x);
                            if (edge) {
                                const int32_t key = key0 + t * 16 + (c >> 1) * 8 + qr;
                                if (key > row_hi[c & 1] || key < row_lo[c & 1]) s[t][c] = -INFINITY;
                            }
                            mx[c & 1] = fmaxf(mx[c & 1], s[t][c]);
                        }
                    }
#pragma unroll
                    for (int w = 4; w < 32; w *= 2) {
                        mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], w));
                        mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], w));
                    }
                    if (!__all_sync(0xffffffffu, mx[0] == m[0] && mx[1] == m[1])) {
                        const float up[2] = {weight(m[0], mx[0]), weight(m[1], mx[1])};
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            l[i] *= up[i];
                            m[i] = mx[i];
                        }
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i)
#pragma unroll
                            for (int c = 0; c < 4; ++c) o[i][c] *= up[c & 1];
                    }
                    const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0] - Fp16::LIFT, m[1] == -INFINITY ? 0.f : m[1] - Fp16::LIFT};
#pragma unroll
                    for (int t = 0; t < KPW / 16; ++t) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[t][c] = exp2_approx(s[t][c] - ref[c & 1]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) l[i] = fmaf(s[t][i] + s[t][2 + i], rs[t], l[i]);
                        // the weights rounded to fp16 (the matrix instruction takes 16-bit operands): at most 2^-11
                        // of each, an eighth of a bf16 output's own rounding and as much as an fp16 one's
                        const uint32_t p0 = transpose8(Fp16::pack(s[t][0], s[t][1])), p1 = transpose8(Fp16::pack(s[t][2], s[t][3]));
#pragma unroll
                        for (int c = 0; c < DP / 16; c += 2) {
                            uint32_t(&b)[4] = vr[t][c / 2];
#pragma unroll
                            for (int i = 0; i < 4; ++i) b[i] = __byte_perm(b[i], 0, 0x3120);  // even values of two keys, then odd ones
                            const uint32_t v0[4] = {codes_lo(b[0]), codes_hi(b[0]), codes_lo(b[1]), codes_hi(b[1])};
                            const uint32_t v1[4] = {codes_lo(b[2]), codes_hi(b[2]), codes_lo(b[3]), codes_hi(b[3])};
                            Fp16::mma(o[c], v0, p0, p1);
                            Fp16::mma(o[c + 1], v1, p0, p1);
                        }
                    }
                } else if (lane == 0) {
                    mbar_arrive(&sh->empty[st]);
                }
            }

            // the warps' parts of the segment, joined in warp order; from here on m is what the weights refer to
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[i] -= Fp16::LIFT;
#pragma unroll
                for (int w = 4; w < 32; w *= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
                if (qr == 0) {
                    sh->m[warp][qc + i] = m[i];
                    sh->l[warp][qc + i] = l[i];
                }
            }
            consumers8_sync();
            if (threadIdx.x == 0) {  // the segment before is done with its turn
                sh->bad_lo[turn ^ 1] = INT32_MAX;
                sh->bad_hi[turn ^ 1] = -1;
            }
            float fac[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float all = sh->m[0][qc + i];
#pragma unroll
                for (int w = 1; w < CONSUMERS8; ++w) all = fmaxf(all, sh->m[w][qc + i]);
                fac[i] = weight(m[i], all);
            }
            float *mine = join + wq * (ROWS8 * DP);
#pragma unroll
            for (int turns = GROUPS - 1; turns >= 0; --turns) {  // the last group's first
                if (grp == turns) {
#pragma unroll
                    for (int c = 0; c < DP / 16; ++c)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float2 *at = reinterpret_cast<float2 *>(mine + join8_at<DP>(qc + i, c * 16 + qr * 2));
                            float2 v = make_float2(o[c][i] * fac[i], o[c][2 + i] * fac[i]);
                            if (turns != GROUPS - 1) {
                                const float2 w = *at;
                                v.x += w.x, v.y += w.y;
                            }
                            *at = v;
                        }
                }
                consumers8_sync();
            }
            const bool whole = walk.j == 0 && n == walk.tiles;
            const int slot = (int)blockIdx.x * 2 + (f == f0 ? 0 : 1);
            // a thread takes 4 values of a row at a time
            for (int e = threadIdx.x * 4; e < ROWS8 * DP; e += 32 * CONSUMERS8 * 4) {
                const int r = e / DP, c = e - r * DP;
                if (r >= g.n_rows) continue;
                const int at = join8_at<DP>(r, c);
                float4 v = *reinterpret_cast<const float4 *>(join + at);
#pragma unroll
                for (int w = 1; w < 4; ++w) {
                    const float4 t = *reinterpret_cast<const float4 *>(join + w * (ROWS8 * DP) + at);
                    v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
                }
                if (sh->bad_hi[turn] >= 0 && c < p.head_dim) {
                    const int32_t pos = g.pos0 + p.by_group.quotient(g.r0 + r);
                    float x[4] = {v.x, v.y, v.z, v.w};
                    add_nan<4>(p.b, p8.codes, walk.s, g.head, max(first_seen(pos, p.window), sh->bad_lo[turn] * KT),
                               min(pos + 1, (sh->bad_hi[turn] + 1) * KT), c, p.head_dim, x);
                    v = make_float4(x[0], x[1], x[2], x[3]);
                }
                if (p.cluster > 1) {
                    *reinterpret_cast<float4 *>(join + at) = v;  // read by this thread alone so far
                    continue;
                }
                if (!whole) {
                    *reinterpret_cast<float4 *>(p.part_o + (int64_t)slot * (ROWS8 * DP) + e) = v;
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
                    p.part_ml[slot * (2 * ROWS8) + r] = mm;
                    p.part_ml[slot * (2 * ROWS8) + ROWS8 + r] = ll;
                } else if (p.lse) {
                    write_lse(p, walk, g, r, mm, ll);
                }
            }
            if (p.cluster > 1) {  // each CTA joins its share of the values from all shares of the keys, in rank order
                consumers8_sync();
                if (threadIdx.x < p.cluster) arrive_at(&sh->ready, threadIdx.x);
                const bool ok = mbar_wait_cluster(&sh->ready, exchange_ph, abort);
                const int share = ROWS8 * DP / p.cluster;
                for (int e = rank * share + threadIdx.x * 4; ok && e < (rank + 1) * share; e += 32 * CONSUMERS8 * 4) {
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
                            x[k] = ld_shared_cluster_f4(mapa_shared(smem_u32(join + join8_at<DP>(r, c)), k));
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
                    consumers8_sync();
                    if (threadIdx.x < p.cluster) arrive_at(&sh->done, threadIdx.x);
                    mbar_wait_cluster(&sh->done, exchange_ph, abort);  // nobody reads this CTA's memory any more
                }
                exchange_ph ^= 1;
            }
            consumers8_sync();  // the join's memory is free again
            f += n;
            if (f < f1) walk.next(p, base);
        }
    }
    if (p.cluster > 1) {  // no CTA leaves while another may read its memory or arrive on its barriers, after a time-out either
        __syncwarp();
        cluster_sync_all();
    }
}

}  // namespace rows
}  // namespace attn
}  // namespace engram
