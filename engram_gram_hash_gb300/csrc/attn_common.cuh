// Shared pieces of the attention kernels: the two 16-bit types, the step's
// batch as the kernels see it, and the warp's search for a token's sequence.
#pragma once

namespace engram {
namespace attn {

// LIFT: the softmax weights are kept times 2^LIFT at most (numerator and sum alike, so it cancels) before
// they are rounded to the type for the second product.  bf16 has fp32's exponents and needs none.  fp16
// loses bits below 2^-14: with its weights up to 2^15 only those under 2^-29 of the row's largest do, 2^-25
// in the tile kernel (without, those under 2^-14: a key 14 nats above the others, whose value is zero, left
// 1.6e-2 relative error).
// RESCALE: the tile kernel's running maximum may lag the true one by 2^RESCALE.  fp16, a prompt of 8,192
// tokens with 1 / 2 / 4 / 8: 405, 398, 363, 364 us.
struct Bf16 {
    static constexpr float LIFT = 0.f, RESCALE = 8.f;
    // two values times zero onto acc: NaN from then on if either is an infinity or NaN
    static __device__ __forceinline__ void spot(uint32_t &acc, uint32_t w) {
        asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w), "r"(0u));
    }
    static constexpr uint32_t EXPONENT = 0x7F80u;
    static __device__ __forceinline__ float2 unpack(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

struct Fp16 {
    static constexpr float LIFT = 15.f, RESCALE = 4.f;
    static __device__ __forceinline__ void spot(uint32_t &acc, uint32_t w) {
        asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(w), "r"(0u));
    }
    static constexpr uint32_t EXPONENT = 0x7C00u;
    static __device__ __forceinline__ float2 unpack(uint32_t w) {
        return __half22float2(*reinterpret_cast<__half2 *>(&w));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&v);
    }
    static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// Division of 0 <= n < 2^31 by a fixed d >= 1 as a multiplication (Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994):
// with 2^l >= d and m = floor(2^(31+l) / d) + 1, m d - 2^(31+l) <= 2^l, so
// floor(n m / 2^(31+l)) = floor(n / d).
struct Divisor {
    uint32_t d, m, l;
    Divisor() = default;
    explicit Divisor(uint32_t d_) : d(d_), l(0) {
        while ((1u << l) < d) ++l;
        m = (uint32_t)((UINT64_C(1) << (31 + l)) / d + 1);
    }
    __device__ __forceinline__ int32_t quotient(int32_t n) const {
        return d == 1 ? n : (int32_t)(__umulhi((uint32_t)n, m) >> (l - 1));
    }
};

// engram_kv_batch with the cache's page geometry.
struct Batch {
    const int64_t *offs;
    const int32_t *kv_len;
    const int32_t *block_table;
    int64_t table_stride, table_width;
    int64_t n_seqs;
    int64_t n_query;
    int64_t n_pages;
    int32_t page_size;
};

constexpr int64_t MAX_KV = INT32_MAX - 1023;

// Sequence s of a step: its first row among the step's tokens, its new
// tokens and its length with them.  Offsets that descend or leave the step's
// rows, and lengths past the block table, are cut to what is there (rows and
// table entries stay in bounds) and flagged; so are lengths past MAX_KV, which
// a tile's end, rounded up, would take out of 32 bits.
struct Seq {
    int32_t row0;
    int32_t q_len;
    int32_t kv;
};

__device__ __forceinline__ Seq load_seq(const Batch &b, int64_t s, int64_t base) {
    int64_t a = __ldg(b.offs + s) - base, e = __ldg(b.offs + s + 1) - base;
    int64_t kv = __ldg(b.kv_len + s);
    const int64_t room = b.table_width * b.page_size, cap = room < MAX_KV ? room : MAX_KV;
    const bool bad = a < 0 || e < a || e > b.n_query || kv > cap;
    if (bad) {
        raise_error(ENGRAM_ERANGE);
        a = a < 0 ? 0 : (a > b.n_query ? b.n_query : a);
        e = e < a ? a : (e > b.n_query ? b.n_query : e);
        kv = kv > cap ? cap : kv;
    }
    return Seq{(int32_t)a, (int32_t)(e - a), kv < 0 ? 0 : (int32_t)kv};
}

// The first position that a token at `pos` sees (0: plain causal).  Compared
// before subtracted: with a padded token (pos < 0) and a window near 2^31 the
// difference would leave 32 bits.
__device__ __forceinline__ int32_t first_seen(int32_t pos, int32_t window) {
    return window > 0 && pos >= window ? pos - window + 1 : 0;
}

// What the weighted sum of the row at `pos` is multiplied by: 1 / l.  l is 0 (no
// weight was above zero) for a row before the sequence's start, which has no
// key and gets 0, and for one whose scores are all -inf, whose softmax is NaN.
__device__ __forceinline__ float inverse(float l, int32_t pos) {
    return l > 0.f ? 1.f / l : (l == 0.f ? (pos < 0 ? 0.f : NAN) : l);
}

// mbar_wait by a whole warp, with one answer for all its lanes (near the time
// limit the lanes could differ, and the warp-wide steps that follow must not).
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

// Infinities and NaN among the values.  A key that is hidden from a row has
// weight 0 there, but 0 times an infinity is NaN, and the products run over
// whole tiles.  So in tiles that some row sees only part of ("edge" tiles) such
// values are cleared before the product (clear_nonfinite) and, where any was
// found, added to the rows that do see their key afterwards (add_nonfinite).
// No hidden value reaches a row; a row that sees one that is not finite has no
// finite result either, but it may be NaN where the sum is an infinity: in the
// other tiles, or when parts are joined, a weight that underflows to 0 meets it.

// The infinities and NaN of the two values in w are set to zero.
template <typename E>
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
    if ((w & E::EXPONENT) == E::EXPONENT) w &= 0xFFFF0000u;
    if (((w >> 16) & E::EXPONENT) == E::EXPONENT) w &= 0x0000FFFFu;
    return w;
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// N 16-byte pieces of shared memory, `at(i)` the address of the i-th: whether
// they hold an infinity or NaN (false if !keep), and their clearing: all of
// them if !keep, else the infinities and NaN.
template <typename E, int N, typename F>
__device__ __forceinline__ bool holds_nonfinite(bool keep, const F &at) {
    uint32_t acc = 0;
    if (keep) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint4 v = lds16(at(i));
            E::spot(acc, v.x);
            E::spot(acc, v.y);
            E::spot(acc, v.z);
            E::spot(acc, v.w);
        }
    }
    return acc != 0u;
}
template <typename E, int N, typename F>
__device__ __forceinline__ void clear_nonfinite(bool keep, const F &at) {
    if (!keep) {
#pragma unroll
        for (int i = 0; i < N; ++i) sts16(at(i), make_uint4(0, 0, 0, 0));
        return;
    }
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
        const uint4 v = lds16(at(i));
        sts16(at(i), make_uint4(finite_only<E>(v.x), finite_only<E>(v.y), finite_only<E>(v.z), finite_only<E>(v.w)));
    }
}

// The cached values as plain memory.
struct ValuePages {
    const uint16_t *v;
    int64_t page_stride, slot_stride, head_stride;
};
// o[i] += the infinities and NaN among values c + i < dim, i < N, of keys
// [key_lo, key_hi) of sequence s.
template <typename E, int N>
__device__ __forceinline__ void add_nonfinite(const Batch &b, const ValuePages &pages, int64_t s, int32_t head, int32_t key_lo,
                                              int32_t key_hi, int c, int dim, float (&o)[N]) {
#pragma unroll 1
    for (int32_t key = key_lo; key < key_hi; ++key) {
        const int32_t page = __ldg(b.block_table + s * b.table_stride + key / b.page_size);
        if (page < 0 || page >= b.n_pages) continue;
        const uint16_t *v = pages.v + page * pages.page_stride + (key % b.page_size) * pages.slot_stride +
                            head * pages.head_stride + c;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            if (c + i >= dim) break;
            const uint32_t w = *reinterpret_cast<const uint32_t *>(v + i);
            const float2 f = E::unpack(w);
            if ((w & E::EXPONENT) == E::EXPONENT) o[i] += f.x;
            if (((w >> 16) & E::EXPONENT) == E::EXPONENT) o[i + 1] += f.y;
        }
    }
}

// The last sequence s with offs[s] <= base + t (a whole warp looks at 32
// offsets at a time, so up to 32 sequences take one load and 1,024 take two).
__device__ __forceinline__ int64_t warp_find_seq(const int64_t *offs, int64_t n_seqs, int64_t p) {
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, n = n_seqs;  // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int64_t step = (n + 31) / 32;
        const int64_t at = lo + lane * step;
        const bool le = lane == 0 || (lane * step < n && __ldg(offs + at) <= p);
        const int k = 31 - __clz(__ballot_sync(0xffffffffu, le));  // offsets ascend: the last lane that holds
        lo += k * step;
        n = n - k * step < step ? n - k * step : step;
    }
    return lo;
}

}  // namespace attn
}  // namespace engram
