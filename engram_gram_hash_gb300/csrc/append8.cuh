// The append of keys and values to a paged cache of 8-bit codes (e4m3) with a
// scale for each block of B tokens and head.
//
//   s = 2^e, the least with max |x| <= 448 s over the block's finite values
//   (-48 <= e <= 48), no smaller than before where the block holds earlier
//   tokens; code = e4m3(x / s).  Powers of two: codes are floating-point, so
//   within their range a finer scale would buy nothing, x / s is exact, and
//   when a later token makes a block's scale grow, its earlier codes stay exact
//   but for those that leave the normal range (below 2^-6 s).
// Keys are normed, rotated and rounded to the 16-bit type first, as the 16-bit
// cache holds them: one more half step of 2^-9 (bf16) beside the code's 2^-4,
// for which a block's values wait for its scale in half the registers.
//
// Bound: memory, for a prompt (2 bytes in, 1 out a value); a decode step by the
// chain offsets -> length -> page -> scale.  A CTA has one block of tokens, the
// keys or the values of the 4 or 8 heads that a warp holds side by side, and a
// warp for every 8 tokens: each value is read once, stays in registers while
// the block's maximum is found, and is written once.  The angles of a block's
// tokens come into shared memory beside the keys (from the table token by
// token, each waited for, 32,768 tokens took 62 us instead of 56).  56 us are
// 57 % of the copy rate, 15,026 tokens of 8 sequences 27-28 us (53-55 %): by the
// counters instructions (262 a warp and token) at the 16 warps an SM that 128
// registers leave; the maxima are packed 16-bit ones already.  64 tokens with
// their queries 5.4-6.1 us in a CUDA graph.
// The queries' CTAs of the same launch have as many warps as those of the
// blocks, at the same 128 registers: two for blocks of 16.  2,407 tokens of 24
// + 4 heads of 96 in blocks of 16 take 14.7 us, 7.7 without the queries, whose
// rotation alone takes 5.4: 7,224 such CTAs run in about six waves.
#pragma once

namespace engram {
namespace attn {

constexpr int TOKENS_PER_WARP = 8;
constexpr int MAX_EXP = 48;     // of a scale: 2^-48 .. 2^48

struct Append8 {
    HeadParams h;  // the heads in; with queries, their outputs
    uint8_t *k_pages, *v_pages;
    float *k_scales, *v_scales;  // [page][kv head][block]
    int64_t page_stride, slot_stride, head_stride;
    int64_t units;               // blocks of tokens that the batch can touch
    int32_t n_kv, block, per_page;
    int32_t kv_blocks;           // CTAs for keys and values; those for the queries follow
    int32_t q_groups;            // warps' shares of a token's query heads
};

// The unbiased exponent of the least power of two >= x, cut to -48 .. 48; -48 unless x > 0.
__device__ __forceinline__ int exponent_over(float x) {
    if (!(x > 0.f)) return -MAX_EXP;
    const uint32_t b = __float_as_uint(x);
    const int e = (int)(b >> 23) - 127 + ((b & 0x7FFFFFu) != 0u);
    return e < -MAX_EXP ? -MAX_EXP : (e > MAX_EXP ? MAX_EXP : e);
}
// ... of the least one whose 448-fold holds x (448 = 1.75 * 2^8).
__device__ __forceinline__ int exponent_for(float x) {
    const uint32_t b = __float_as_uint(x);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u);
    return e < -MAX_EXP ? -MAX_EXP : (e > MAX_EXP ? MAX_EXP : e);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint32_t to_codes(float2 lo, float2 hi) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3) << 16;
}
// 8 values times f as codes (NaN stays NaN).
template <typename E>
__device__ __forceinline__ uint2 quantise(uint4 x, float f) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = mul2(E::unpack(w[i]), make_float2(f, f));
    return make_uint2(to_codes(v[0], v[1]), to_codes(v[2], v[3]));
}
// 4 codes that stood for multiples of `was` as codes for multiples of 1 / inv.
__device__ __forceinline__ uint32_t requantise(uint32_t c, float was, float inv) {
    float2 a = e4m3x2_to_float2((uint16_t)c), b = e4m3x2_to_float2((uint16_t)(c >> 16));
    a = mul2(mul2(a, make_float2(was, was)), make_float2(inv, inv));
    b = mul2(mul2(b, make_float2(was, was)), make_float2(inv, inv));
    return to_codes(a, b);
}
// The two values' larger magnitude pattern onto m, each half for itself.
__device__ __forceinline__ uint32_t max_abs(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }
// Infinities become NaN (the codes have none).
template <typename E>
__device__ __forceinline__ uint32_t nan_for_inf(uint32_t w) {
    if ((w & E::EXPONENT) == E::EXPONENT) w |= 0x7FFFu;
    if (((w >> 16) & E::EXPONENT) == E::EXPONENT) w |= 0x7FFF0000u;
    return w;
}

template <typename E, int LPH, bool INTERLEAVED, int THREADS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) append8_kernel(const __grid_constant__ Append8 a) {
    constexpr int GPW = 32 / LPH, N = TOKENS_PER_WARP;
    __shared__ uint32_t most[THREADS / 32][GPW];
    extern __shared__ __align__(16) float rows[];  // the table's rows of the block's tokens, for keys
    grid_dependency_wait();
    allow_dependent_launch();
    const HeadParams &p = a.h;
    const Batch &b = p.batch;
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % LPH, grp = lane / LPH, groups = (a.n_kv + GPW - 1) / GPW;
    if ((int)blockIdx.x >= a.kv_blocks) {  // queries
        const int at = (int)blockIdx.x - a.kv_blocks;
        head_rows<E, LPH, 1, INTERLEAVED, true>(p, (int64_t)(at / a.q_groups) * warps + warp, at % a.q_groups);
        return;
    }
    const int part = (int)blockIdx.x / (int)a.units;
    const int64_t u = (int)blockIdx.x - part * (int)a.units;
    const bool is_v = part >= groups;
    const int h = (is_v ? part - groups : part) * GPW + grp;
    const bool live = h < a.n_kv;

    // Sequence s has the units from min(row0 / B + 2 s, row0) on: its rows touch at most one block more than they fill,
    // and no more blocks than there are rows.
    const int32_t B = a.block;
    const int64_t base = __ldg(b.offs);
    if (blockIdx.x == 0 && threadIdx.x == 0 && __ldg(b.offs + b.n_seqs) - base != p.n_tokens) raise_error(ENGRAM_ERANGE);
    const auto first_unit = [&](int64_t i, int64_t row) { return min(row / B + 2 * i, row); };
    const int64_t s = warp_find(b.n_seqs, [&](int64_t i) { return first_unit(i, __ldg(b.offs + i) - base) <= u; });
    const int64_t r0 = __ldg(b.offs + s) - base, r1 = __ldg(b.offs + s + 1) - base;
    if (r0 < 0 || r1 < r0 || r1 > p.n_tokens) {
        if (threadIdx.x == 0) raise_error(ENGRAM_ERANGE);
        return;
    }
    const int64_t kv = __ldg(b.kv_len + s), first = kv - (r1 - r0);  // the first new token's position; before 0: padding
    const int64_t begin = first > 0 ? first : 0;
    const int64_t block0 = (begin / B + (u - first_unit(s, r0))) * B;
    const int64_t lo = begin > block0 ? begin : block0;
    int64_t hi = kv < block0 + B ? kv : block0 + B;
    if (lo >= hi) return;
    if (p.rope_dim > 0 && hi > p.table_rows) {  // for values too: the token is left out
        if (threadIdx.x == 0) raise_error(ENGRAM_ERANGE);
        hi = p.table_rows;
        if (lo >= hi) return;
    }
    const int32_t entry = p.by_page.quotient((int32_t)block0), slot0 = (int32_t)block0 - entry * b.page_size;
    int32_t page = -1;
    if (entry < b.table_width) page = __ldg(b.block_table + s * b.table_stride + entry);
    const int32_t n_old = (int32_t)(lo - block0), n_end = (int32_t)(hi - block0);  // new tokens: [n_old, n_end) of the block

    if (page < 0 || page >= b.n_pages) {
        if (threadIdx.x == 0) raise_error(ENGRAM_ERANGE);
        return;
    }
    float *scale = (is_v ? a.v_scales : a.k_scales) + ((int64_t)page * a.n_kv + h) * a.per_page + slot0 / B;
    const float was = live && n_old > 0 ? *scale : 0.f;
    if (!is_v && p.rope_dim > 0) {
        const float *from = p.table + block0 * p.rope_dim;
        for (int i = n_old * p.rope_dim + threadIdx.x * 4; i < n_end * p.rope_dim; i += blockDim.x * 4)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(rows + i)), "l"(from + i) : "memory");
    }
    HeadLane k;
    if (is_v) {  // any pieces do
        k.c0 = 2 * l;
        k.c1 = 2 * l + 1;
        k.has0 = k.c0 < (p.head_dim >> 3);
        k.has1 = k.c1 < (p.head_dim >> 3);
    } else {
        k = head_lane<LPH, INTERLEAVED>(p, l);
    }
    k.has0 = k.has0 && live;
    k.has1 = k.has1 && live;
    const HeadView in = is_v ? p.v : p.k;
    const uint16_t *src = in.data + (r0 + block0 - first) * in.token_stride + (int64_t)h * in.head_stride;
    uint4 x0[N], x1[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {  // token i * warps + warp of the block
        const int t = i * warps + warp;
        const bool on = t >= n_old && t < n_end;
        x0[i] = on && k.has0 ? *reinterpret_cast<const uint4 *>(src + t * in.token_stride + k.c0 * 8) : make_uint4(0, 0, 0, 0);
        x1[i] = on && k.has1 ? *reinterpret_cast<const uint4 *>(src + t * in.token_stride + k.c1 * 8) : make_uint4(0, 0, 0, 0);
    }
    if (!is_v) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int t = i * warps + warp;
            if (t < n_old || t >= n_end) continue;
            Turn turn;
            turn_weights<E, INTERLEAVED>(k, p.w_k, turn);
            const float *row = rows + t * p.rope_dim;
            turn_angles<INTERLEAVED>(p, k, [&](int j) { return *reinterpret_cast<const float4 *>(row + j); }, turn);
            float2 f[4], g[4];
            turn_head<E, LPH, INTERLEAVED>(p, k, turn, p.w_k != nullptr, x0[i], x1[i], f, g);
            from_pairs<E, INTERLEAVED>(f, g, x0[i], x1[i]);
        }
    }
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        m2 = max_abs(max_abs(max_abs(max_abs(m2, x0[i].x), x0[i].y), x0[i].z), x0[i].w);
        m2 = max_abs(max_abs(max_abs(max_abs(m2, x1[i].x), x1[i].y), x1[i].z), x1[i].w);
    }
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    if (m >= E::EXPONENT) {  // an infinity or NaN among them: the maximum is the finite values'
        m = 0;
        const auto take = [&](uint32_t &w) {
            w = nan_for_inf<E>(w);
            if ((w & E::EXPONENT) != E::EXPONENT) m = max(m, w & 0x7FFFu);
            if (((w >> 16) & E::EXPONENT) != E::EXPONENT) m = max(m, (w >> 16) & 0x7FFFu);
        };
#pragma unroll
        for (int i = 0; i < N; ++i) {
            take(x0[i].x), take(x0[i].y), take(x0[i].z), take(x0[i].w);
            take(x1[i].x), take(x1[i].y), take(x1[i].z), take(x1[i].w);
        }
    }
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (l == 0) most[warp][grp] = m;
    __syncthreads();
    m = 0;
    for (int w = 0; w < warps; ++w) m = max(m, most[w][grp]);
    if (!live) return;
    int e = exponent_for(E::unpack(m).x);
    if (n_old > 0) e = max(e, exponent_over(was));
    const float now = power_of_two(e), inv = power_of_two(-e);

    uint8_t *dst = (is_v ? a.v_pages : a.k_pages) + (int64_t)page * a.page_stride + (int64_t)slot0 * a.slot_stride + (int64_t)h * a.head_stride;
    if (n_old > 0 && now != was) {  // the earlier tokens' codes stand for multiples of the new scale from here on
        for (int t = warp; t < n_old; t += warps) {
            uint8_t *at = dst + t * a.slot_stride;
            const auto again = [&](uint8_t *c) {
                uint2 v = *reinterpret_cast<uint2 *>(c);
                *reinterpret_cast<uint2 *>(c) = make_uint2(requantise(v.x, was, inv), requantise(v.y, was, inv));
            };
            if (k.has0) again(at + k.c0 * 8);
            if (k.has1) again(at + k.c1 * 8);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int t = i * warps + warp;
        if (t < n_old || t >= n_end) continue;
        uint8_t *at = dst + t * a.slot_stride;
        const uint2 y0 = quantise<E>(x0[i], inv), y1 = quantise<E>(x1[i], inv);
        if (is_v) {  // head_dim is a multiple of 16: both pieces or none
            if (k.has0) *reinterpret_cast<uint4 *>(at + k.c0 * 8) = make_uint4(y0.x, y0.y, y1.x, y1.y);
        } else {
            if (k.has0) *reinterpret_cast<uint2 *>(at + k.c0 * 8) = y0;
            if (k.has1) *reinterpret_cast<uint2 *>(at + k.c1 * 8) = y1;
        }
    }
    if (warp == 0 && l == 0) *scale = now;  // (read by all before the barrier)
}

}  // namespace attn
}  // namespace engram
