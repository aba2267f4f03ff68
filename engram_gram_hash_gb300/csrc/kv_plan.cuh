// Block tables, slot maps and the batch's offsets from the requests' lengths.
//
//   had = ceil(old / P), need = ceil((keep + new) / P) pages of a request;
//   had > need: entries need .. had - 1 of its row go back on the free stack,
//   had < need: entries had .. need - 1 come off its top, both in the order of
//   (request, entry); offsets are the new tokens' running sum, token i of a
//   request has position keep + i and slot table[pos / P] * P + pos % P.
//
// Bound: a decode step's plan by latency (a chain of loads, a scan, the page
// moves), a prompt's by the 12 bytes written for each token.  One block scans
// the requests (1,024 at a time, 256 where that is all) and moves the pages, so
// the whole step is checked before anything changes and the stack's order does
// not depend on timing.  Pages and tokens go to the block's threads one each,
// whosever they are (a search in the scan's sums finds the request): a warp a
// request, its 16 requests' loads one after another, took 19 us for 512 mixed
// requests.  The maps of many tokens are a second kernel over the whole GPU.
#pragma once

namespace engram {
namespace attn {
namespace plan {

constexpr int MOST = 1024;  // requests at a time
constexpr int SPAN = 256;   // tokens of a warp of the map kernel

struct Params {
    const int32_t *new_len, *keep_len, *kv_len;  // keep_len null: all is kept
    int32_t *kv_len_out;
    int32_t *table;
    int64_t table_stride, table_width;
    int32_t *free_pages;
    const int32_t *n_free;
    int32_t *n_free_out;
    int64_t *offs;
    int32_t *positions;  // null: left out
    int64_t *slots;      // null: left out
    int32_t *counts;     // tokens, pages taken, pages given back, pages missing
    int64_t n_seqs, max_tokens, n_pages;
    int32_t page_size;
    int32_t maps;        // the plan's block writes positions and slots itself
    Divisor by_page;
};

struct Request {
    int32_t keep, fresh, had, need;
    bool ok;
};
__device__ __forceinline__ int32_t pages_of(const Params &p, int32_t n) { return n > 0 ? p.by_page.quotient(n - 1) + 1 : 0; }
__device__ __forceinline__ Request load_request(const Params &p, int64_t s) {
    const int32_t old = p.kv_len[s], fresh = p.new_len[s], keep = p.keep_len ? p.keep_len[s] : old;
    Request r = {keep, fresh, 0, 0, old >= 0 && keep >= 0 && keep <= old && fresh >= 0 && (int64_t)keep + fresh <= MAX_KV};
    if (r.ok) {
        r.had = pages_of(p, old);
        r.need = pages_of(p, keep + fresh);
        r.ok = r.had <= p.table_width && r.need <= p.table_width;
    }
    if (!r.ok) r.keep = r.fresh = r.had = r.need = 0;
    return r;
}

struct Sums {
    int64_t tokens, back, take;
};
__device__ __forceinline__ Sums operator+(const Sums &a, const Sums &b) {
    return Sums{a.tokens + b.tokens, a.back + b.back, a.take + b.take};
}

template <int NT>
struct Shared {
    Sums warp[NT / 32];
    // before each request of the chunk and after the last; pages: in a plan that is carried out the sums are at most n_pages
    int64_t tokens[NT + 1];
    int32_t back[NT + 1], take[NT + 1];
    int32_t had[NT], need[NT], keep[NT];
};

// Exclusive sums over the block's threads, and their total.
template <int NT>
__device__ __forceinline__ Sums block_scan(Sums v, Sums *warps, Sums &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const auto scan = [&](Sums x, int n) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            if (o >= n) break;
            const Sums u = {__shfl_up_sync(0xffffffffu, x.tokens, o), __shfl_up_sync(0xffffffffu, x.back, o),
                            __shfl_up_sync(0xffffffffu, x.take, o)};
            if (lane >= o) x = x + u;
        }
        return x;
    };
    const Sums x = scan(v, 32);
    __syncthreads();  // the last call's sums have been read
    if (lane == 31) warps[warp] = x;
    __syncthreads();
    const Sums y = scan(lane < NT / 32 ? warps[lane] : Sums{0, 0, 0}, NT / 32);
    const auto at = [&](int w) {
        return Sums{__shfl_sync(0xffffffffu, y.tokens, w), __shfl_sync(0xffffffffu, y.back, w), __shfl_sync(0xffffffffu, y.take, w)};
    };
    total = at(NT / 32 - 1);
    const Sums before = warp > 0 ? at(warp - 1) : Sums{0, 0, 0};
    return Sums{before.tokens + x.tokens - v.tokens, before.back + x.back - v.back, before.take + x.take - v.take};
}

// The request of the chunk that holds place x: the last i < n with v[i] <= x.
template <typename T>
__device__ __forceinline__ int request_of(const T *v, int n, T x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void write_token(const Params &p, int64_t s, int64_t t, int32_t pos) {
    if (p.positions) p.positions[t] = pos;
    if (p.slots) {
        const int32_t entry = p.by_page.quotient(pos);
        p.slots[t] = (int64_t)p.table[s * p.table_stride + entry] * p.page_size + (pos - entry * p.page_size);
    }
}
__device__ __forceinline__ void write_none(const Params &p, int64_t t) {
    if (p.positions) p.positions[t] = -1;
    if (p.slots) p.slots[t] = -1;
}

template <int NT>
__global__ void __launch_bounds__(NT) plan_kernel(const __grid_constant__ Params p) {
    __shared__ Shared<NT> sh;
    grid_dependency_wait();
    allow_dependent_launch();
    const int tid = threadIdx.x;
    const bool single = p.n_seqs <= NT;
    const int64_t n_free = *p.n_free;
    Sums done = {0, 0, 0};  // before the chunk
    bool bad = false;
    // The chunk of requests at c0: its counts in shared memory, with what lies before each.
    const auto enter = [&](int64_t c0) {
        Request r = {0, 0, 0, 0, true};
        if (c0 + tid < p.n_seqs) r = load_request(p, c0 + tid);
        bad = bad || !r.ok;
        const Sums mine = {r.fresh, r.had > r.need ? r.had - r.need : 0, r.need > r.had ? r.need - r.had : 0};
        Sums total;
        const Sums at = done + block_scan<NT>(mine, sh.warp, total);
        sh.tokens[tid] = at.tokens;
        sh.back[tid] = (int32_t)at.back;
        sh.take[tid] = (int32_t)at.take;
        sh.had[tid] = r.had;
        sh.need[tid] = r.need;
        sh.keep[tid] = r.keep;
        done = done + total;
        if (tid == NT - 1) {
            sh.tokens[NT] = done.tokens;
            sh.back[NT] = (int32_t)done.back;
            sh.take[NT] = (int32_t)done.take;
        }
        __syncthreads();
    };
    for (int64_t c0 = 0; c0 < p.n_seqs; c0 += NT) enter(c0);
    const Sums all = done;
    bad = __syncthreads_or(bad) || n_free < 0 || n_free + all.back > p.n_pages;
    const int64_t missing = bad ? 0 : all.take - (n_free + all.back);
    if (bad || missing > 0 || all.tokens > p.max_tokens) {  // nothing changes, and the step has no tokens
        if (tid == 0) raise_error(bad ? ENGRAM_ERANGE : ENGRAM_ECAPACITY);
        for (int64_t s = tid; s < p.n_seqs; s += NT) {
            p.kv_len_out[s] = p.kv_len[s];
            p.offs[s] = 0;
        }
        if (p.maps)
            for (int64_t t = tid; t < p.max_tokens; t += NT) write_none(p, t);
        if (tid == 0) {
            p.offs[p.n_seqs] = 0;
            *p.n_free_out = (int32_t)n_free;
            p.counts[0] = p.counts[1] = p.counts[2] = 0;
            p.counts[3] = (int32_t)(missing > 0 ? (missing < INT32_MAX ? missing : INT32_MAX) : 0);
        }
        return;
    }

    // pages given back, all of them before the first is taken
    if (all.back > 0) {
        done = Sums{0, 0, 0};
        for (int64_t c0 = 0; c0 < p.n_seqs; c0 += NT) {
            if (!single) enter(c0);
            const int n = (int)(p.n_seqs - c0 < NT ? p.n_seqs - c0 : NT);
#pragma unroll 4
            for (int32_t k = sh.back[0] + tid; k < sh.back[NT]; k += NT) {
                const int i = request_of(sh.back, n, k);
                p.free_pages[n_free + k] = p.table[(c0 + i) * p.table_stride + sh.need[i] + k - sh.back[i]];
            }
        }
        __syncthreads();
    }
    const int64_t top = n_free + all.back - 1;
    done = Sums{0, 0, 0};
    for (int64_t c0 = 0; c0 < p.n_seqs; c0 += NT) {
        if (!single) enter(c0);
        const int n = (int)(p.n_seqs - c0 < NT ? p.n_seqs - c0 : NT);
        if (all.take > 0) {
#pragma unroll 4
            for (int32_t k = sh.take[0] + tid; k < sh.take[NT]; k += NT) {
                const int i = request_of(sh.take, n, k);
                p.table[(c0 + i) * p.table_stride + sh.had[i] + k - sh.take[i]] = p.free_pages[top - k];
            }
        }
        if (tid < n) {
            p.kv_len_out[c0 + tid] = sh.keep[tid] + (int32_t)(sh.tokens[tid + 1] - sh.tokens[tid]);
            p.offs[c0 + tid] = sh.tokens[tid];
        }
        if (p.maps) {
            __syncthreads();  // the pages are in the table
            for (int64_t t = sh.tokens[0] + tid; t < sh.tokens[NT]; t += NT) {
                const int i = request_of(sh.tokens, n, t);
                write_token(p, c0 + i, t, sh.keep[i] + (int32_t)(t - sh.tokens[i]));
            }
        }
    }
    if (p.maps)
        for (int64_t t = all.tokens + tid; t < p.max_tokens; t += NT) write_none(p, t);
    if (tid == 0) {
        p.offs[p.n_seqs] = all.tokens;
        *p.n_free_out = (int32_t)(n_free + all.back - all.take);
        p.counts[0] = (int32_t)all.tokens;
        p.counts[1] = (int32_t)all.take;
        p.counts[2] = (int32_t)all.back;
        p.counts[3] = 0;
    }
}

// Positions and slots, a warp for up to SPAN tokens of one request.  Request s
// has the warps from offs[s] / SPAN + s on: as many as it can need, found
// without another scan.
__global__ void __launch_bounds__(256) map_kernel(const __grid_constant__ Params p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int lane = threadIdx.x & 31;
    const int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (p.n_seqs > 0) {  // without requests there are no lengths, no rows of the table and one offset
        const int64_t s = warp_find(p.n_seqs, [&](int64_t i) { return p.offs[i] / SPAN + i <= u; });
        const int64_t t0 = p.offs[s], t1 = p.offs[s + 1], j0 = (u - t0 / SPAN - s) * SPAN;
        const int64_t end = t1 - t0 < j0 + SPAN ? t1 - t0 : j0 + SPAN;
        const int32_t keep = p.kv_len_out[s] - (int32_t)(t1 - t0);
#pragma unroll 4
        for (int64_t j = j0 + lane; j < end; j += 32) write_token(p, s, t0 + j, keep + (int32_t)j);
    }
    for (int64_t t = p.offs[p.n_seqs] + u * 32 + lane; t < p.max_tokens; t += (int64_t)gridDim.x * 256) write_none(p, t);
}

}  // namespace plan
}  // namespace attn
}  // namespace engram
