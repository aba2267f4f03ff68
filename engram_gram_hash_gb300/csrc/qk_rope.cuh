// Head norm + rotation, and the append of keys and values to a paged cache:
// one kernel, since both do the same to a head on its way from the packed
// projection to where it is kept.
//
//   n = x / sqrt(mean(x^2) + eps) * w;  y_a = n_a cos - n_b sin,
//   y_b = n_b cos + n_a sin for the pair (a, b) of each angle.
//
// Bound: memory.  Every value is read once and written once (16-byte pieces,
// 128 bytes per lane and round in flight); the fp32 table row of a token
// (rope_dim * 4 bytes) is read once per warp and serves all its heads.
// Layout: a lane holds two 8-value pieces of a head, chosen so that both
// values of every pair are in the same lane (HALVES: piece l and the piece
// rope_dim/2 further on; INTERLEAVED: any two), so the rotation needs no
// exchange and the norm one butterfly over the LPH lanes of the head.
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
    int32_t head_blocks;             // warps per token
    int32_t head_dim, rope_dim;
    float eps;
    // append: the cache (k_out / v_out are its pages) and the batch
    uint16_t *k_pages, *v_pages;
    int64_t page_stride, slot_stride, page_head_stride;
    Batch batch;
};

template <typename E>
__device__ __forceinline__ void unpack8(uint4 w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 t = E::unpack(u[i]);
        f[2 * i] = t.x;
        f[2 * i + 1] = t.y;
    }
}
template <typename E>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(E::pack(f[0], f[1]), E::pack(f[2], f[3]), E::pack(f[4], f[5]), E::pack(f[6], f[7]));
}

// LPH lanes per head (4 up to 64 values, 8 up to 128), U heads per lane: a
// warp takes U * 32 / LPH heads of one token.
template <typename E, int LPH, int U, bool INTERLEAVED, bool APPEND>
__global__ void __launch_bounds__(256) head_kernel(const __grid_constant__ HeadParams p) {
    constexpr int GPW = 32 / LPH;
    grid_dependency_wait();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const int l = lane % LPH, grp = lane / LPH;
    const int64_t wid = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t t = wid / p.head_blocks;
    if (t >= p.n_tokens) return;
    const int h0 = (int)(wid - t * p.head_blocks) * (GPW * U) + grp;
    const int n_pieces = p.head_dim >> 3, rot_pieces = p.rope_dim >> 3;

    int c0, c1;
    bool rot0, rot1;
    if (INTERLEAVED) {
        c0 = l;
        c1 = l + LPH;
        rot0 = c0 < rot_pieces;
        rot1 = c1 < rot_pieces;
    } else {
        const int half = rot_pieces >> 1;
        rot0 = rot1 = l < half;
        c0 = rot0 ? l : rot_pieces + 2 * (l - half);
        c1 = rot0 ? l + half : c0 + 1;
    }
    const bool has0 = c0 < n_pieces, has1 = c1 < n_pieces;

    // all of this lane's heads: loads first, the position's chain behind them
    uint4 x0[U], x1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * GPW;
        x0[u] = x1[u] = make_uint4(0, 0, 0, 0);
        const uint16_t *src = nullptr;
        if (h < p.n_q)
            src = p.q.data + t * p.q.token_stride + h * p.q.head_stride;
        else if (h < p.n_q + p.n_k)
            src = p.k.data + t * p.k.token_stride + (h - p.n_q) * p.k.head_stride;
        else if (APPEND && h < p.n_q + p.n_k + p.n_v)
            src = p.v.data + t * p.v.token_stride + (h - p.n_q - p.n_k) * p.v.head_stride;
        if (src) {
            if (has0) x0[u] = *reinterpret_cast<const uint4 *>(src + c0 * 8);
            if (has1) x1[u] = *reinterpret_cast<const uint4 *>(src + c1 * 8);
        }
    }

    int64_t pos = 0;
    int64_t slot = 0;  // element offset of the token's slot in the pages
    if (APPEND) {
        const int64_t base = __ldg(p.batch.offs);
        if (wid == 0 && lane == 0 && __ldg(p.batch.offs + p.batch.n_seqs) - base != p.n_tokens)
            raise_error(ENGRAM_ERANGE);
        const int64_t s = warp_find_seq(p.batch.offs, p.batch.n_seqs, base + t);
        const int64_t after = __ldg(p.batch.offs + s + 1) - (base + t);  // new tokens from this one on
        if (after <= 0) return;                                          // offsets that stop short, flagged above
        pos = __ldg(p.batch.kv_len + s) - after;
        if (pos < 0) return;  // padding
        const int64_t entry = pos / p.batch.page_size;
        int32_t page = -1;
        if (entry < p.batch.table_stride) page = __ldg(p.batch.block_table + s * p.batch.table_stride + entry);
        if (page < 0 || page >= p.batch.n_pages) {
            if (lane == 0) raise_error(ENGRAM_ERANGE);
            return;
        }
        slot = page * p.page_stride + (pos - entry * p.batch.page_size) * p.slot_stride;
    } else if (p.positions) {
        pos = __ldg(p.positions + t);
    }
    if (p.rope_dim > 0 && (pos < 0 || pos >= p.table_rows)) {
        if (lane == 0) raise_error(ENGRAM_ERANGE);
        return;
    }

    // angles of the lane's pairs: HALVES pair i of piece c0 in slot i;
    // INTERLEAVED pairs of c0 in slots 0..3, of c1 in slots 4..7
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
    }
    const float *row = p.table + pos * p.rope_dim;
    const int hr = p.rope_dim >> 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool on = INTERLEAVED ? (i ? rot1 : rot0) : rot0;
        const int at = INTERLEAVED ? (i ? c1 : c0) * 4 : c0 * 8 + i * 4;
        if (on) {
            const float4 c4 = __ldg(reinterpret_cast<const float4 *>(row + at));
            const float4 s4 = __ldg(reinterpret_cast<const float4 *>(row + hr + at));
            cs[4 * i] = c4.x, cs[4 * i + 1] = c4.y, cs[4 * i + 2] = c4.z, cs[4 * i + 3] = c4.w;
            sn[4 * i] = s4.x, sn[4 * i + 1] = s4.y, sn[4 * i + 2] = s4.z, sn[4 * i + 3] = s4.w;
        }
    }

#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * GPW;
        const bool is_q = h < p.n_q;
        const bool live = h < p.n_q + p.n_k;  // normed and rotated; the values' heads are copied
        const uint16_t *w = is_q ? p.w_q : p.w_k;
        float a[8], b[8];
        unpack8<E>(x0[u], a);
        unpack8<E>(x1[u], b);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (live) {
            if (w) {
                const float rinv = rsqrtf(ss / (float)p.head_dim + p.eps);
                float wa[8], wb[8];
                unpack8<E>(has0 ? __ldg(reinterpret_cast<const uint4 *>(w + c0 * 8)) : make_uint4(0, 0, 0, 0), wa);
                unpack8<E>(has1 ? __ldg(reinterpret_cast<const uint4 *>(w + c1 * 8)) : make_uint4(0, 0, 0, 0), wb);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a[i] *= rinv * wa[i];
                    b[i] *= rinv * wb[i];
                }
            }
            if (INTERLEAVED) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
                    a[2 * i] = a0 * cs[i] - a1 * sn[i];
                    a[2 * i + 1] = a1 * cs[i] + a0 * sn[i];
                    b[2 * i] = b0 * cs[4 + i] - b1 * sn[4 + i];
                    b[2 * i + 1] = b1 * cs[4 + i] + b0 * sn[4 + i];
                }
            } else if (rot0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float av = a[i], bv = b[i];
                    a[i] = av * cs[i] - bv * sn[i];
                    b[i] = bv * cs[i] + av * sn[i];
                }
            }
            x0[u] = pack8<E>(a);
            x1[u] = pack8<E>(b);
        }
        uint16_t *dst = nullptr;
        if (is_q)
            dst = p.q_out.data + t * p.q_out.token_stride + h * p.q_out.head_stride;
        else if (h < p.n_q + p.n_k)
            dst = APPEND ? p.k_pages + slot + (h - p.n_q) * p.page_head_stride
                         : p.k_out.data + t * p.k_out.token_stride + (h - p.n_q) * p.k_out.head_stride;
        else if (APPEND && h < p.n_q + p.n_k + p.n_v)
            dst = p.v_pages + slot + (h - p.n_q - p.n_k) * p.page_head_stride;
        if (dst) {
            if (has0) *reinterpret_cast<uint4 *>(dst + c0 * 8) = x0[u];
            if (has1) *reinterpret_cast<uint4 *>(dst + c1 * 8) = x1[u];
        }
    }
}

}  // namespace attn
}  // namespace engram
