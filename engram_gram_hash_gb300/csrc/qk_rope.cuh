// Head norm + rotation, and the append of keys and values to a paged cache:
// one kernel, since both do the same to a head on its way from the packed
// projection to where it is kept.
//
//   n = x / sqrt(mean(x^2) + eps) * w;  y_a = n_a cos - n_b sin,
//   y_b = n_b cos + n_a sin for the pair (a, b) of each angle.
//
// Bound: memory.  Every value is read once and written once in 16-byte pieces;
// the fp32 table row of a token (rope_dim * 4 bytes) is read once per warp and
// serves all its heads.  32,768 tokens of 32 + 8 heads of 128: 120 us, 5.7 TB/s
// (84 % of the copy rate); 15,026 tokens' keys and values into pages 27 us,
// 4.8 TB/s (bound by the chain offsets -> length -> page -> slot of every token;
// this form also spills, 72 bytes a thread at the 64 registers that four blocks
// an SM leave).
// Layout: a lane holds two 8-value pieces of a head, chosen so that both
// values of every pair are in the same lane (HALVES: piece l and the piece
// rope_dim/2 further on; INTERLEAVED: any two), so the rotation needs no
// exchange and the norm one butterfly over the LPH lanes of the head.  What
// limits it then is instructions, so the arithmetic is done on pairs
// (f32x2), weights and angles are multiplied together once per token, and
// nothing is divided.
#pragma once

namespace engram {
namespace attn {

struct HeadView {
    uint16_t *data;
    int64_t token_stride;
    int64_t head_stride;
};

struct HeadParams {
    HeadView q, k, v, q_out, k_out;  // data null: left out
    const uint16_t *w_q, *w_k;       // null: no norm
    const int32_t *positions;        // engram_qk_norm_rope; the append derives them from the batch
    const float *table;
    int64_t table_rows;
    int64_t n_tokens;
    int32_t n_q, n_k, n_v;           // heads of each kind in this launch
    int32_t head_dim, rope_dim;
    float eps, inv_dim;
    // append: the cache (k_out / v_out are its pages) and the batch
    uint16_t *k_pages, *v_pages;
    int64_t page_stride, slot_stride, page_head_stride;
    Batch batch;
    Divisor by_page;
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}

// The 16 values of two pieces as 8 pairs (f, s), two pairs to a float2.
// HALVES: f from piece 0, s from piece 1 at the same place.  INTERLEAVED: f the
// even, s the odd values, piece 0 in pairs 0..3 and piece 1 in pairs 4..7.
template <typename E, bool INTERLEAVED>
__device__ __forceinline__ void to_pairs(uint4 p0, uint4 p1, float2 (&f)[4], float2 (&s)[4]) {
    const uint32_t a[4] = {p0.x, p0.y, p0.z, p0.w}, b[4] = {p1.x, p1.y, p1.z, p1.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (INTERLEAVED) {
            const float2 u = E::unpack(i < 2 ? a[2 * i] : b[2 * i - 4]), v = E::unpack(i < 2 ? a[2 * i + 1] : b[2 * i - 3]);
            f[i] = make_float2(u.x, v.x);
            s[i] = make_float2(u.y, v.y);
        } else {
            f[i] = E::unpack(a[i]);
            s[i] = E::unpack(b[i]);
        }
    }
}
template <typename E, bool INTERLEAVED>
__device__ __forceinline__ void from_pairs(const float2 (&f)[4], const float2 (&s)[4], uint4 &p0, uint4 &p1) {
    uint32_t a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (INTERLEAVED) {
            (i < 2 ? a[2 * i] : b[2 * i - 4]) = E::pack(f[i].x, s[i].x);
            (i < 2 ? a[2 * i + 1] : b[2 * i - 3]) = E::pack(f[i].y, s[i].y);
        } else {
            a[i] = E::pack(f[i].x, f[i].y);
            b[i] = E::pack(s[i].x, s[i].y);
        }
    }
    p0 = make_uint4(a[0], a[1], a[2], a[3]);
    p1 = make_uint4(b[0], b[1], b[2], b[3]);
}

// A lane's two 8-value pieces of a head, and which of them turn.
struct HeadLane {
    int c0, c1;
    bool rot0, rot1, has0, has1;
};
template <int LPH, bool INTERLEAVED>
__device__ __forceinline__ HeadLane head_lane(const HeadParams &p, int l) {
    const int n_pieces = p.head_dim >> 3, rot_pieces = p.rope_dim >> 3;
    HeadLane k;
    if (INTERLEAVED) {
        k.c0 = l;
        k.c1 = l + LPH;
        k.rot0 = k.c0 < rot_pieces;
        k.rot1 = k.c1 < rot_pieces;
    } else {
        const int half = rot_pieces >> 1;
        k.rot0 = k.rot1 = l < half;
        k.c0 = k.rot0 ? l : rot_pieces + 2 * (l - half);
        k.c1 = k.rot0 ? l + half : k.c0 + 1;
    }
    k.has0 = k.c0 < n_pieces;
    k.has1 = k.c1 < n_pieces;
    return k;
}

// The lane's 8 pairs (f, s) turn as f' = f A + s B, s' = s C + f D with the weights in the factors,
// A = w_f cos, B = -w_s sin, C = w_s cos, D = w_f sin, made once for all its heads of a token.
struct Turn {
    float2 A[4], B[4], C[4], D[4];
};
// A and C to start from: the weights (1 without).
template <typename E, bool INTERLEAVED>
__device__ __forceinline__ void turn_weights(const HeadLane &k, const uint16_t *w, Turn &t) {
    if (w)
        to_pairs<E, INTERLEAVED>(k.has0 ? __ldg(reinterpret_cast<const uint4 *>(w + k.c0 * 8)) : make_uint4(0, 0, 0, 0),
                                 k.has1 ? __ldg(reinterpret_cast<const uint4 *>(w + k.c1 * 8)) : make_uint4(0, 0, 0, 0), t.A, t.C);
    else
#pragma unroll
        for (int i = 0; i < 4; ++i) t.A[i] = t.C[i] = make_float2(1.f, 1.f);
}
// `angles(i)`: four numbers of the position's table row from the i-th on.
template <bool INTERLEAVED, typename F>
__device__ __forceinline__ void turn_angles(const HeadParams &p, const HeadLane &k, const F &angles, Turn &t) {
    const int hr = p.rope_dim >> 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // pairs 4i .. 4i + 3
        t.B[2 * i] = t.B[2 * i + 1] = t.D[2 * i] = t.D[2 * i + 1] = make_float2(0.f, 0.f);
        if (i ? k.rot1 : k.rot0) {
            const int at = INTERLEAVED ? (i ? k.c1 : k.c0) * 4 : k.c0 * 8 + i * 4;
            const float4 c4 = angles(at), s4 = angles(hr + at);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int q = 2 * i + j;
                const float2 cs = j ? make_float2(c4.z, c4.w) : make_float2(c4.x, c4.y);
                const float2 sn = j ? make_float2(s4.z, s4.w) : make_float2(s4.x, s4.y);
                t.B[q] = mul2(t.C[q], make_float2(-sn.x, -sn.y));
                t.D[q] = mul2(t.A[q], sn);
                t.A[q] = mul2(t.A[q], cs);
                t.C[q] = mul2(t.C[q], cs);
            }
        }
    }
}
// The lane's pieces of one head: normed (norm, over the LPH lanes of the head; the whole warp calls) and turned.
template <typename E, int LPH, bool INTERLEAVED>
__device__ __forceinline__ void turn_head(const HeadParams &p, const HeadLane &k, const Turn &t, bool norm, uint4 x0, uint4 x1,
                                          float2 (&f)[4], float2 (&s)[4]) {
    to_pairs<E, INTERLEAVED>(x0, x1, f, s);
    float rinv = 1.f;
    if (norm) {
        float2 ss = mul2(f[0], f[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) ss = fma2(f[i], f[i], ss);
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma2(s[i], s[i], ss);
        float sum = ss.x + ss.y;
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        rinv = rsqrtf(fmaf(sum, p.inv_dim, p.eps));
    }
    const float2 r2 = make_float2(rinv, rinv);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 a = mul2(f[i], t.A[i]), b = mul2(s[i], t.C[i]);
        if (i < 2 ? k.rot0 : k.rot1) {  // values that do not turn never meet their neighbours'
            a = fma2(s[i], t.B[i], a);
            b = fma2(f[i], t.D[i], b);
        }
        f[i] = mul2(a, r2);
        s[i] = mul2(b, r2);
    }
}

// LPH lanes per head (4 up to 64 values, 8 up to 128), U heads per lane: a
// warp takes up to U * 32 / LPH heads of token t, either queries or, in one
// row, keys and values (the values are only copied).  `block` counts the
// warps' shares of a token's heads, the queries' first.
template <typename E, int LPH, int U, bool INTERLEAVED, bool APPEND>
__device__ __forceinline__ void head_rows(const HeadParams &p, int64_t t, int block) {
    constexpr int GPW = 32 / LPH, PER = GPW * U;
    const int lane = threadIdx.x & 31;
    const int l = lane % LPH, grp = lane / LPH;
    if (t >= p.n_tokens) return;
    const bool first = t == 0 && block == 0;
    // the warp's kind and its first head
    const int q_blocks = (p.n_q + PER - 1) / PER;
    const bool is_q = block < q_blocks;
    if (!is_q) block -= q_blocks;
    const int n_rot = is_q ? p.n_q : p.n_k, n_heads = is_q ? p.n_q : p.n_k + p.n_v;
    const HeadView in = is_q ? p.q : p.k;
    const int h0 = block * PER + grp;
    const bool turns = block * PER < n_rot;  // any of the warp's heads
    const HeadLane k = head_lane<LPH, INTERLEAVED>(p, l);

    // all of this lane's heads: loads first, the position's chain behind them
    uint4 x0[U], x1[U];
    const uint16_t *src = in.data + t * in.token_stride;
    const uint16_t *src_v = APPEND ? p.v.data + t * p.v.token_stride : nullptr;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * GPW;
        const uint16_t *a = APPEND && h >= n_rot ? src_v + (int64_t)(h - n_rot) * p.v.head_stride : src + (int64_t)h * in.head_stride;
        x0[u] = h < n_heads && k.has0 ? *reinterpret_cast<const uint4 *>(a + k.c0 * 8) : make_uint4(0, 0, 0, 0);
        x1[u] = h < n_heads && k.has1 ? *reinterpret_cast<const uint4 *>(a + k.c1 * 8) : make_uint4(0, 0, 0, 0);
    }

    int64_t pos = 0;
    int64_t slot = 0;  // element offset of the token's slot in the pages
    if (APPEND) {
        const int64_t base = __ldg(p.batch.offs);
        if (first && lane == 0 && __ldg(p.batch.offs + p.batch.n_seqs) - base != p.n_tokens)
            raise_error(ENGRAM_ERANGE);
        const int64_t s = warp_find_seq(p.batch.offs, p.batch.n_seqs, base + t);
        const int64_t after = __ldg(p.batch.offs + s + 1) - (base + t);  // new tokens from this one on
        if (after <= 0) return;                                          // offsets that stop short, flagged above
        pos = __ldg(p.batch.kv_len + s) - after;
        if (pos < 0) return;  // padding
        const int32_t entry = p.by_page.quotient((int32_t)pos);  // pos < kv_len, an int32
        int32_t page = -1;
        if (entry < p.batch.table_width) page = __ldg(p.batch.block_table + s * p.batch.table_stride + entry);
        if (page < 0 || page >= p.batch.n_pages) {
            if (lane == 0) raise_error(ENGRAM_ERANGE);
            return;
        }
        slot = page * p.page_stride + ((int32_t)pos - entry * p.batch.page_size) * p.slot_stride;
    } else if (p.positions) {
        pos = __ldg(p.positions + t);
    }
    if (p.rope_dim > 0 && (pos < 0 || pos >= p.table_rows)) {  // for a copied head too: the token is left out
        if (lane == 0) raise_error(ENGRAM_ERANGE);
        return;
    }

    if (turns) {
        const uint16_t *w = is_q ? p.w_q : p.w_k;
        Turn turn;
        turn_weights<E, INTERLEAVED>(k, w, turn);
        const float *row = p.table + pos * p.rope_dim;
        turn_angles<INTERLEAVED>(p, k, [&](int i) { return __ldg(reinterpret_cast<const float4 *>(row + i)); }, turn);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 f[4], s[4];
            turn_head<E, LPH, INTERLEAVED>(p, k, turn, w != nullptr, x0[u], x1[u], f, s);
            if (!APPEND || h0 + u * GPW < n_rot) from_pairs<E, INTERLEAVED>(f, s, x0[u], x1[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * GPW;
        if (h >= n_heads) continue;
        uint16_t *a;
        if (is_q)
            a = p.q_out.data + t * p.q_out.token_stride + (int64_t)h * p.q_out.head_stride;
        else if (!APPEND)
            a = p.k_out.data + t * p.k_out.token_stride + (int64_t)h * p.k_out.head_stride;
        else
            a = (h < n_rot ? p.k_pages + (int64_t)h * p.page_head_stride : p.v_pages + (int64_t)(h - n_rot) * p.page_head_stride) + slot;
        if (k.has0) *reinterpret_cast<uint4 *>(a + k.c0 * 8) = x0[u];
        if (k.has1) *reinterpret_cast<uint4 *>(a + k.c1 * 8) = x1[u];
    }
}

template <typename E, int LPH, int U, bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(256, 4) head_kernel(const __grid_constant__ HeadParams p) {
    grid_dependency_wait();
    allow_dependent_launch();
    head_rows<E, LPH, U, INTERLEAVED, APPEND>(p, (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5), blockIdx.y);
}

}  // namespace attn
}  // namespace engram
