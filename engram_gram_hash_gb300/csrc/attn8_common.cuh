// Attention over a cache of 8-bit codes with a scale for each block of tokens
// and head: what its two kernels share.
//
//   With key j's codes kc_j, vc_j and its blocks' scales ks_j, vs_j,
//     u_j = log2(e) scale ks_j (q.kc_j) + log2 vs_j,   R = max u_j,
//     O = sum_j 2^(u_j - R) vc_j,   l = sum_j 2^(u_j - R) / vs_j,
//     out = O / l,   lse = ln 2 (R + log2 l).
// So both scales come into the exponent, one multiply-add a score as without
// them, and nothing is multiplied per value.  R follows what a row's result is
// made of (weight times scale), so weights rounded to fp16 keep their bits
// whatever the scales are; l, in fp32, takes the scale out again, a block at a
// time.  (m, l, O) of two parts join as in the 16-bit kernels, with R for m.
// Codes are exact in fp16 and weights keep 11 bits there, so the second product
// runs on fp16 whatever the type of the queries.
#pragma once

namespace engram {
namespace attn {

constexpr int STRIP = 16;  // keys that always share their scales: blocks and pages hold whole strips

// The scales' cached memory: [page][kv head][block of tokens].
struct Scales {
    const float *k, *v;
    int32_t per_page;    // blocks in a page
    int32_t block_log2;  // tokens in a block
};

// log2 vs and 1 / vs of a strip's value scale.  Below 2^-48 it counts as 2^-48, so a block of zeros may have
// scale 0; above 2^48 as that.  The logarithm is the exponent, exact, and that of the mantissa, off by 2^-22 at
// most; the same number weighs a key's values and, taken out of l by the inverse, hardly its weight.
__device__ __forceinline__ float2 value_scale(float vs) {
    const float x = fminf(fmaxf(vs, 3.5527136788005009e-15f), 281474976710656.f);
    const uint32_t b = __float_as_uint(x);
    float lg, inv;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg) : "f"(__uint_as_float((b & 0x7FFFFFu) | 0x3F800000u)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(x));
    return make_float2(lg + (float)((int)(b >> 23) - 127), inv);
}

// Two codes (the low or high half of w) as an fp16 pair.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
    uint32_t d;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(d) : "r"(w));
    return d;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
    uint32_t d;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(d) : "r"(w));
    return d;
}

// Whether any of four codes is NaN (0x7F or 0xFF), and the codes with those set to zero.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t without_nan(uint32_t w) { return w & ~((nan_codes(w) >> 7) * 0xFFu); }

// The power of two that brings a row's largest magnitude to 2^TO .. 2^(TO + 1), as its exponent (at most 124); 0 for
// a row of zeros or with an infinity or NaN.
template <int TO>
__device__ __forceinline__ int row_exponent(float most) {
    if (!(most > 0.f) || !(most < INFINITY)) return 0;
    const int e = TO + 127 - (int)(__float_as_uint(most) >> 23);
    return e > 124 ? 124 : e;
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The cached codes of values as plain memory.
struct CodePages {
    const uint8_t *v;
    int64_t page_stride, slot_stride, head_stride;
};
// o[i] becomes NaN where value c + i < dim, i < N, of a key in [key_lo, key_hi) of sequence s is NaN: the codes
// that were taken out of the products of tiles that some row sees only part of.
template <int N>
__device__ __forceinline__ void add_nan(const Batch &b, const CodePages &pages, int64_t s, int32_t head, int32_t key_lo,
                                        int32_t key_hi, int c, int dim, float (&o)[N]) {
#pragma unroll 1
    for (int32_t key = key_lo; key < key_hi; ++key) {
        const int32_t page = __ldg(b.block_table + s * b.table_stride + key / b.page_size);
        if (page < 0 || page >= b.n_pages) continue;
        const uint8_t *v = pages.v + page * pages.page_stride + (key % b.page_size) * pages.slot_stride + head * pages.head_stride + c;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            if (c + i >= dim) break;
            const uint32_t bad = nan_codes(*reinterpret_cast<const uint32_t *>(v + i));
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (bad & (0x80u << (8 * k))) o[i + k] = NAN;
        }
    }
}

// 4 bytes into shared memory (zero without `in`), asynchronously.
__device__ __forceinline__ void copy4_async(uint32_t dst, const float *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
// One arrival on the barrier once this thread's asynchronous copies so far have landed.
__device__ __forceinline__ void arrive_when_copied(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

}  // namespace attn
}  // namespace engram
