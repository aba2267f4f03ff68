// Shared pieces of the attention kernels: the two 16-bit types, the step's
// batch as the kernels see it, and the warp's search for a token's sequence.
#pragma once

namespace engram {
namespace attn {

struct Bf16 {
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
    int64_t table_stride;
    int64_t n_seqs;
    int64_t n_query;
    int64_t n_pages;
    int32_t page_size;
};

// Sequence s of a step: its first row among the step's tokens, its new
// tokens and its length with them.  Offsets that descend or leave the step's
// rows, and lengths past the block table, are cut to what is there (rows and
// table entries stay in bounds) and flagged.
struct Seq {
    int32_t row0;
    int32_t q_len;
    int32_t kv;
};

__device__ __forceinline__ Seq load_seq(const Batch &b, int64_t s, int64_t base) {
    int64_t a = __ldg(b.offs + s) - base, e = __ldg(b.offs + s + 1) - base;
    int64_t kv = __ldg(b.kv_len + s);
    const int64_t cap = b.table_stride * b.page_size;
    const bool bad = a < 0 || e < a || e > b.n_query || kv > cap;
    if (bad) {
        raise_error(ENGRAM_ERANGE);
        a = a < 0 ? 0 : (a > b.n_query ? b.n_query : a);
        e = e < a ? a : (e > b.n_query ? b.n_query : e);
        kv = kv > cap ? cap : kv;
    }
    return Seq{(int32_t)a, (int32_t)(e - a), kv < 0 ? 0 : (int32_t)kv};
}

// mbar_wait by a whole warp, with one answer for all its lanes (near the time
// limit the lanes could differ, and the warp-wide steps that follow must not).
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
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
