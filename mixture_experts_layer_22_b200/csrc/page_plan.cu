// page_plan.cu - block table and slot map of a batch from its request lengths
// (moe_page_plan).
//
// Two exclusive sums over the requests, of new tokens and of new pages, decide
// everything: request b's new tokens are the rows from the first, its new
// pages the entries of the free list from the second.  A token row finds its
// request by a binary search in the sums.
//
// Latency-bound: at 1024 requests and 33,000 rows it touches 0.3 MB.  So it is
// one launch, in which every block forms both sums for itself in shared memory
// (two loads and one block scan, cheaper than a second launch or a grid
// barrier) and then takes its share of the token rows and of the new pages.  A
// token's slot comes from the free list where its page is new and from the
// table where its page was held before, so no block reads what another writes.
#include "common.cuh"
#include "overlap.cuh"

namespace moe {

constexpr int kPlanThreads = 512;
constexpr int kPlanMaxB = 4096;

// The last request whose start is <= i, given start[0] = 0 <= i < start[B]:
// requests with nothing of their own (start[b] == start[b+1]) are passed over.
__device__ __forceinline__ int owner_of(const int32_t *start, int B, int32_t i)
{
    int lo = 0, hi = B;                          // start[lo] <= i < start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Exclusive sums over the block of (x, y), both at once; totals in sx, sy.
__device__ __forceinline__ void block_scan2(long long &x, long long &y, long long &sx, long long &sy)
{
    __shared__ long long wx[kPlanThreads / 32], wy[kPlanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long ix = x, iy = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long vx = __shfl_up_sync(0xffffffffu, ix, o), vy = __shfl_up_sync(0xffffffffu, iy, o);
        if (lane >= o) {
            ix += vx;
            iy += vy;
        }
    }
    if (lane == 31) {
        wx[warp] = ix;
        wy[warp] = iy;
    }
    __syncthreads();
    long long bx = 0, by = 0;
    sx = sy = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) {
            bx += wx[w];
            by += wy[w];
        }
        sx += wx[w];
        sy += wy[w];
    }
    x = bx + ix - x;
    y = by + iy - y;
}

__device__ __forceinline__ int32_t clamp_i32(long long v)
{
    return static_cast<int32_t>(v < 0x7fffffffll ? v : 0x7fffffffll);
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(moe_page_shape_t s, const int32_t *__restrict__ cached,
                                                                 const int32_t *__restrict__ fresh,
                                                                 const int32_t *__restrict__ free_pages,
                                                                 const int32_t *__restrict__ free_pos,
                                                                 int32_t *block_table, int32_t *q_start, int32_t *kv_len,
                                                                 int32_t *positions, int32_t *slots, int32_t *free_next,
                                                                 int32_t *status)
{
    __shared__ int32_t s_tok[kPlanMaxB + 1], s_page[kPlanMaxB + 1];   // exclusive sums
    const int tid = threadIdx.x;
    const int ps = s.page_size;
    const long long room = static_cast<long long>(s.max_pages) * ps;
    bool bad = false;

    const int per = (s.B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(s.B, tid * per), b1 = min(s.B, b0 + per);
    long long tok = 0, pages = 0;
    for (int b = b0; b < b1; ++b) {
        long long c = __ldg(cached + b), f = __ldg(fresh + b);
        if (c < 0 || f < 0 || c + f > room) {
            bad = true;
            c = f = 0;
        }
        // the loop's own counts wait in shared memory for the block's sums
        const int32_t np = static_cast<int32_t>((c + f + ps - 1) / ps - (c + ps - 1) / ps);
        s_tok[b] = static_cast<int32_t>(f);
        s_page[b] = np;
        tok += f;
        pages += np;
        if (blockIdx.x == 0) kv_len[b] = static_cast<int32_t>(c + f);
    }
    long long n_tok, n_page;
    block_scan2(tok, pages, n_tok, n_page);
    for (int b = b0; b < b1; ++b) {
        const int32_t f = s_tok[b], np = s_page[b];
        s_tok[b] = clamp_i32(tok);
        s_page[b] = clamp_i32(pages);
        if (blockIdx.x == 0) q_start[b] = s_tok[b];
        tok += f;
        pages += np;
    }
    if (tid == 0) {
        s_tok[s.B] = clamp_i32(n_tok);
        s_page[s.B] = clamp_i32(n_page);
    }
    long long from = free_pos ? __ldg(free_pos) : 0;
    if (from < 0 || from > s.n_free) {
        bad = true;
        from = s.n_free;
    }
    if (blockIdx.x == 0 && tid == 0) {
        q_start[s.B] = clamp_i32(n_tok);
        const long long next = from + n_page;
        if (free_next) *free_next = static_cast<int32_t>(next < s.n_free ? next : s.n_free);
        bad = bad || n_tok > s.max_tokens;
    }
    __syncthreads();

    // the id at entry i of the new pages, -1 where there is none
    auto new_page = [&](long long i) -> int32_t {
        const int32_t id = from + i < s.n_free ? __ldg(free_pages + from + i) : -1;
        const bool ok = id >= 0 && id < s.num_pages;
        bad = bad || !ok;
        return ok ? id : -1;
    };

    auto held_pages = [&](int b) { return static_cast<int>((__ldg(cached + b) + static_cast<long long>(ps) - 1) / ps); };

    const int stride = gridDim.x * kPlanThreads;
    const int first = blockIdx.x * kPlanThreads + tid;
    const int total = s_tok[s.B];
    for (int t = first; t < s.max_tokens; t += stride) {
        int32_t pos = 0, slot = -1;
        if (t < total) {
            const int b = owner_of(s_tok, s.B, t);
            pos = __ldg(cached + b) + (t - s_tok[b]);
            const int held = held_pages(b), col = pos / ps;
            int32_t id;
            if (col >= held) {
                id = new_page(static_cast<long long>(s_page[b]) + (col - held));
            } else {
                id = block_table[static_cast<long long>(b) * s.max_pages + col];
                if (id < 0 || id >= s.num_pages) {
                    bad = true;
                    id = -1;
                }
            }
            if (id >= 0) slot = id * ps + pos % ps;
        }
        positions[t] = pos;
        slots[t] = slot;
    }
    const int n_new = s_page[s.B];
    for (long long i = first; i < n_new; i += stride) {
        const int b = owner_of(s_page, s.B, static_cast<int32_t>(i));
        block_table[static_cast<long long>(b) * s.max_pages + held_pages(b) + (i - s_page[b])] = new_page(i);
    }
    if (bad && status) set_status(status, MOE_ERR_DEVICE_CHECK);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_page_plan(const moe_page_shape_t *shape, const int32_t *cached, const int32_t *fresh,
                             const int32_t *free_pages, const int32_t *free_pos, int32_t *block_table,
                             int32_t *q_start, int32_t *kv_len, int32_t *positions, int32_t *slots, int32_t *free_next,
                             int32_t *status, moe_stream_t stream)
{
    int &launches = launch_counter();
    launches = 0;
    if (!shape) return MOE_ERR_INVALID_ARG;
    const moe_page_shape_t &s = *shape;
    if (s.B < 1 || s.B > kPlanMaxB || s.max_tokens < 0 || s.max_tokens > (1 << 30) || s.max_pages < 1 || s.page_size < 1 ||
        s.num_pages < 1 || s.n_free < 0)
        return MOE_ERR_INVALID_ARG;
    if (static_cast<int64_t>(s.num_pages) * s.page_size > 0x7fffffffll) return MOE_ERR_INVALID_ARG;
    if (static_cast<int64_t>(s.max_pages) * s.page_size > 0x7fffffffll) return MOE_ERR_INVALID_ARG;
    if (!cached || !fresh || !block_table || !q_start || !kv_len) return MOE_ERR_INVALID_ARG;
    if (s.max_tokens > 0 && (!positions || !slots)) return MOE_ERR_INVALID_ARG;
    if (s.n_free > 0 && !free_pages) return MOE_ERR_INVALID_ARG;
    // Blocks read the inputs while others write: no output may lie over an input, nor over
    // another output.
    const Extent in[] = {{cached, s.B * 4ll}, {fresh, s.B * 4ll}, {free_pages, s.n_free * 4ll}, {free_pos, 4}};
    const Extent out[] = {{block_table, static_cast<int64_t>(s.B) * s.max_pages * 4}, {q_start, (s.B + 1) * 4ll}, {kv_len, s.B * 4ll},
                          {positions, s.max_tokens * 4ll}, {slots, s.max_tokens * 4ll}, {free_next, 4}, {status, 4}};
    for (int i = 0; i < 7; ++i) {
        for (const Extent &e : in)
            if (overlap(out[i], e)) return MOE_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return MOE_ERR_INVALID_ARG;
    }
    // One row per thread up to a block per SM.  New pages are at most a page
    // per token plus the rows that max_tokens cuts off; the loops stride.
    const int want = (s.max_tokens + kPlanThreads - 1) / kPlanThreads;
    const int blocks = want < 1 ? 1 : want < 148 ? want : 148;
    page_plan_kernel<<<blocks, kPlanThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        s, cached, fresh, free_pages, free_pos, block_table, q_start, kv_len, positions, slots, free_next, status);
    launches = 1;
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
