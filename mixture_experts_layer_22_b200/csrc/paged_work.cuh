// paged_work.cuh - how the paged-attention kernels divide a batch among CTAs.
//
// An item is one tile of query rows of one request and key/value head: row r of
// a request is token r / group, query head kv_head * group + r % group, so that
// the heads that share a key/value head share its loads.  An item has as many
// blocks of keys as its last row sees.  The blocks of all items, in the order
// request, key/value head, tile, block, are numbered through and cut into G equal
// ranges, range c being the numbers [W c / G, W (c + 1) / G): one for each CTA, or
// for each warp.  All thus have the same work however ragged the lengths are, a
// long sequence is split over many and neighbours read the same keys at the same
// time.  An item that lies whole in one range is written by its owner; of an item
// over several ranges each owner writes a partial result (unnormalised sums, their
// maximum and total), and a second kernel joins them in order.  A range has at
// most two partial items: the one it continues (slot 0) and the one it starts and
// does not finish (slot 1).  The division depends on lengths and G alone, so
// results are reproducible.
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kAttnMaxB = 4096;
constexpr int kAttnMaxSms = 160;
constexpr int kAttnMaxUnits = kAttnMaxSms * 8;   // ranges of one kernel: up to 8 warps or 4 CTAs per SM

// Where element d of row r lies in the partial result of an item of many rows: four
// elements of all rows side by side, since the writers have a row a lane.
__device__ __forceinline__ int many_at(int rows, int r, int d) { return ((d >> 2) * rows + r) * 4 + (d & 3); }

// What a combine block needs to know of the item that range c starts and does not
// finish: its parts are (c, slot 1), (c + 1, slot 0), ... (c + parts - 1, slot 0).
struct AttnDesc {
    int32_t parts;        // 0: none
    int32_t qs, kvh, row0, rows;
};

// Bounded wait for the phase of the given parity, as mbar_wait, but the wall
// clock is read only every 256 tries: a wait here is on the critical path of
// every block, and reading the clock takes longer than the phase.
__device__ __forceinline__ bool attn_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 255u) == 0) {
            if (*abort_flag) return false;
            const uint64_t now = globaltimer();
            if (t0 == 0) t0 = now;
            if (now - t0 > kTimeoutNs) {
                *abort_flag = 1;
                return false;
            }
        }
    }
}

// Division of 0 <= n < 2^31 by a divisor fixed on the host: with 2^s at least the
// divisor times 2^32 and m = ceil(2^s / d), n m / 2^s exceeds n / d by less than
// n / 2^s < 1 / d, so the whole part is that of n / d.
struct FastDiv {
    unsigned long long m;
    int s;

    void set(int d)
    {
        int log = 0;
        while ((1ll << log) < d) ++log;
        s = 32 + log - (log > 31 ? 1 : 0);
        m = ((1ull << s) - 1) / d + 1;
    }
    __device__ __forceinline__ int div(int n) const { return static_cast<int>(static_cast<unsigned long long>(n) * m >> s); }
};

struct AttnParams {
    const void *q, *k_cache, *v_cache;
    const int32_t *table, *q_start, *kv_len;
    void *out;
    int32_t *status;
    float *part;          // [G][2][rows * (D + 2)]: sums, then maxima, then totals, of items
    AttnDesc *desc;       // [G]
    long long q_stride, page_stride;
    int B, T, n_heads, n_kv, group, page_size, num_pages, max_pages, causal;
    int min_rows, max_rows;   // this kernel's requests: rows in [min_rows, max_rows]
    int tile_rows;            // query rows of an item
    int tile_tokens;          // whole tokens of an item, 0 where tokens are cut
    int team_log, n_teams;    // 2^team_log heads side by side, n_kv / 2^team_log times
    FastDiv by_group, by_page, by_tile;
    int wait_at_end;          // launched while the kernel before it runs
    float scale_log2, v_scale;
};

// One request as the kernels see it: n new tokens from row qs on, kv keys.
// n is 0 for requests that are empty, malformed or another kernel's.
struct Req {
    int n, kv, qs;
};

__device__ __forceinline__ Req attn_request(const AttnParams &p, int b, bool &bad)
{
    Req r;
    const int s = __ldg(p.q_start + b), e = __ldg(p.q_start + b + 1);
    int kv = __ldg(p.kv_len + b);
    const long long room = static_cast<long long>(p.max_pages) * p.page_size;
    if (s < 0 || e < s || e > p.T) {
        bad = true;
        r.n = r.kv = r.qs = 0;
        return r;
    }
    if (kv < 0 || kv > room) {
        bad = true;
        kv = kv < 0 ? 0 : static_cast<int>(room);
    }
    const int rows = (e - s) * p.group;
    r.n = rows >= p.min_rows && rows <= p.max_rows ? e - s : 0;
    r.kv = kv;
    r.qs = s;
    return r;
}

// Keys that row `row` of the request sees.
__device__ __forceinline__ int row_limit(const AttnParams &p, const Req &r, int row)
{
    if (!p.causal) return r.kv;
    const int hi = r.kv - r.n + 1 + p.by_group.div(row);
    return hi < 0 ? 0 : hi;
}

// Blocks of the tile whose last row is `last`; a row that sees nothing still has
// its zeros written, so there is at least one.
template <int kBlk>
__device__ __forceinline__ int tile_blocks(const AttnParams &p, const Req &r, int last)
{
    const int nb = (row_limit(p, r, last) + kBlk - 1) / kBlk;
    return nb < 1 ? 1 : nb;
}

// a / b for a >= 0, b > 0.  Nearly always both fit 32 bits, where a division costs
// a fifth of a 64-bit one, and a CTA's first load waits for several.
__device__ __forceinline__ long long div_ll(long long a, long long b)
{
    return ((a | b) >> 32) == 0 ? static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// sum over i < m of floor((a i + b) / c), a, b >= 0, c > 0, by the Euclid-like
// reduction that swaps the roles of a and c.
__device__ __forceinline__ long long floor_sum(long long m, long long c, long long a, long long b)
{
    long long s = 0;
    for (;;) {
        if (a >= c) {
            const long long x = div_ll(a, c);
            s += (m - 1) * m / 2 * x;
            a -= x * c;
        }
        if (b >= c) {
            const long long x = div_ll(b, c);
            s += m * x;
            b -= x * c;
        }
        const long long y = a * m + b;
        if (y < c) return s;
        m = div_ll(y, c);
        b = y - m * c;
        const long long t = c;
        c = a;
        a = t;
    }
}

// Query rows of an item: the kernel's constant, or p.tile_rows where kRows is 0.
template <int kRows>
__device__ __forceinline__ int item_rows(const AttnParams &p)
{
    return kRows > 0 ? kRows : p.tile_rows;
}

// Blocks of one request and key/value head, all tiles.
template <int kRows, int kBlk>
__device__ __forceinline__ long long request_blocks(const AttnParams &p, const Req &r)
{
    if (r.n == 0) return 0;
    const int per = item_rows<kRows>(p), rows = r.n * p.group, tiles = p.by_tile.div(rows + per - 1);
    if (!p.causal) return static_cast<long long>(tiles) * tile_blocks<kBlk>(p, r, rows - 1);
    long long s = tile_blocks<kBlk>(p, r, rows - 1);
    if (p.tile_tokens && r.kv >= r.n) {
        // the full tiles see kv - n + (i + 1) tile_tokens keys
        const int step = p.tile_tokens;
        if (tiles > 1) s += floor_sum(tiles - 1, kBlk, step, r.kv - r.n + step + kBlk - 1);
    } else {
        for (int i = 0; i < tiles - 1; ++i) s += tile_blocks<kBlk>(p, r, (i + 1) * per - 1);
    }
    return s;
}

// A position in the numbering, held by every lane of a warp.  kvh counts teams of
// heads (see Split).
template <int kRows, int kBlk>
struct Cursor {
    Req r;
    int b, kvh, tile, blk, nblk, tiles;

    __device__ __forceinline__ int row0(const AttnParams &p) const { return tile * item_rows<kRows>(p); }
    __device__ __forceinline__ int rows(const AttnParams &p) const { return min(item_rows<kRows>(p), r.n * p.group - row0(p)); }
    __device__ __forceinline__ void enter(const AttnParams &p)
    {
        nblk = tile_blocks<kBlk>(p, r, row0(p) + rows(p) - 1);
    }
    __device__ __forceinline__ void enter_request(const AttnParams &p)
    {
        tiles = p.by_tile.div(r.n * p.group + item_rows<kRows>(p) - 1);
    }
    // On to the next item (warp-collective).  There must be one.
    __device__ __forceinline__ void next_item(const AttnParams &p)
    {
        blk = 0;
        if (++tile == tiles) {
            tile = 0;
            if (++kvh == p.n_teams) {
                kvh = 0;
                bool bad = false;
                const int lane = threadIdx.x & 31;
                for (int base = b + 1; base < p.B; base += 32) {
                    const int mine = base + lane;
                    const bool some = mine < p.B && attn_request(p, mine, bad).n > 0;
                    const unsigned any = __ballot_sync(0xffffffffu, some);
                    if (any) {
                        b = base + __ffs(any) - 1;
                        break;
                    }
                }
                r = attn_request(p, b, bad);
                enter_request(p);
            }
        }
        enter(p);
    }
};

// The division itself.  A CTA has one range for all, or its first kUnits warps have
// ranges of their own.  Then 2^team_log warps side by side are a team with one range,
// in which each takes another head of the same keys, and teams are what is numbered
// where it says head (few ranges spread over all SMs).  init() finds where the calling thread's range starts (cur)
// and returns how many blocks it has; block-collective over kThreads threads, with
// kThreads words of shared memory to itself meanwhile.
template <int kThreads, int kRows, int kBlk, int kUnits = 1>
struct Split {
    long long W;          // blocks in all
    int G;                // ranges that share them

    __device__ __forceinline__ long long start(int c) const { return div_ll(W * c, G); }
    // the range of warp k
    static __device__ __forceinline__ int range(const AttnParams &p, int k)
    {
        return (kUnits > 1 ? k >> p.team_log : k) * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    }
    static __device__ __forceinline__ int ranges(const AttnParams &p)
    {
        return (kUnits > 1 ? kUnits >> p.team_log : 1) * static_cast<int>(gridDim.x);
    }

    __device__ __forceinline__ long long init(const AttnParams &p, Cursor<kRows, kBlk> &cur, long long *s_before)
    {
        __shared__ long long s_warp[kThreads / 32];
        __shared__ int s_at[kUnits][4];
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        const int chunk = (p.B + kThreads - 1) / kThreads;
        const int b0 = min(p.B, tid * chunk), b1 = min(p.B, b0 + chunk);
        bool bad = false;
        long long sum = 0;
        for (int b = b0; b < b1; ++b) sum += p.n_teams * request_blocks<kRows, kBlk>(p, attn_request(p, b, bad));
        if (bad && p.status && blockIdx.x == 0) set_status(p.status, MOE_ERR_DEVICE_CHECK);
        long long inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) s_warp[warp] = inc;
        __syncthreads();
        long long before = inc - sum;
        W = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += s_warp[w];
            W += s_warp[w];
        }
        s_before[tid] = before;
        const int most = ranges(p);
        G = W < most ? static_cast<int>(W) : most;
        if (range(p, 0) >= G) return 0;                          // none of the CTA's ranges
        __syncthreads();
        if (warp < kUnits && range(p, warp) < G) {
            long long at = start(range(p, warp));
            // the thread in whose requests it lies: the last one with before <= at
            int lo = 0, hi = kThreads;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_before[mid] <= at) lo = mid;
                else hi = mid;
            }
            at -= s_before[lo];
            int b = min(p.B, lo * chunk);
            Req r;
            long long per_head;
            for (;; ++b) {
                r = attn_request(p, b, bad);
                per_head = request_blocks<kRows, kBlk>(p, r);
                if (at < per_head * p.n_teams) break;
                at -= per_head * p.n_teams;
            }
            const int kvh = static_cast<int>(div_ll(at, per_head));
            at -= per_head * kvh;
            const int per = item_rows<kRows>(p), rows = r.n * p.group, tiles = p.by_tile.div(rows + per - 1);
            int tile = 0;
            if (!p.causal) {
                const int nb = tile_blocks<kBlk>(p, r, rows - 1);
                tile = static_cast<int>(div_ll(at, nb));
                at -= static_cast<long long>(tile) * nb;
            } else if (p.tile_tokens && r.kv >= r.n) {
                // the last tile with no more than `at` blocks before it, 32 tries at once
                const long long base = r.kv - r.n + p.tile_tokens + kBlk - 1;
                int behind = tiles;
                while (behind - tile > 1) {
                    const int step = (behind - tile + 31) / 32, probe = tile + lane * step;
                    const bool fits = lane == 0 || (probe < behind && floor_sum(probe, kBlk, p.tile_tokens, base) <= at);
                    const int last = 31 - __clz(__ballot_sync(0xffffffffu, fits));
                    tile += last * step;
                    behind = min(behind, tile + step);
                }
                if (tile > 0) at -= floor_sum(tile, kBlk, p.tile_tokens, base);
            } else {
                for (;; ++tile) {
                    const int nb = tile_blocks<kBlk>(p, r, min((tile + 1) * per, rows) - 1);
                    if (at < nb) break;
                    at -= nb;
                }
            }
            if (lane == 0) {
                s_at[warp][0] = b;
                s_at[warp][1] = kvh;
                s_at[warp][2] = tile;
                s_at[warp][3] = static_cast<int>(at);
            }
        }
        __syncthreads();
        const int k = kUnits > 1 ? warp : 0;
        if (k >= kUnits || range(p, k) >= G) return 0;
        cur.b = s_at[k][0];
        cur.kvh = s_at[k][1];
        cur.tile = s_at[k][2];
        cur.blk = s_at[k][3];
        cur.r = attn_request(p, cur.b, bad);
        cur.enter_request(p);
        cur.enter(p);
        return start(range(p, k) + 1) - start(range(p, k));
    }

    // Ranges over which the item extends that range c starts at `from_start`
    // blocks into it and that has `blocks` blocks.
    __device__ __forceinline__ int parts(int c, long long from_start, int blocks) const
    {
        // the first range x with W x / G >= its end is the first one behind it
        const long long end = start(c) + from_start + blocks;
        return static_cast<int>(div_ll(end * G + W - 1, W)) - c;
    }
};

// What q.k, or q times a code, is multiplied by to be an exponent of 2.
inline float attn_scale_log2(const moe_attn_shape_t &s)
{
    return s.scale * (s.cache_dtype == MOE_E4M3 ? s.k_scale : 1.0f) * 1.4426950408889634f;
}

// The tensor-memory kernel: whether it takes a shape, the query rows of its items,
// its launch with one CTA (and range) per SM.
bool attn_tc_takes(const moe_attn_shape_t &s);
int attn_tc_rows(const moe_attn_shape_t &s);
cudaError_t launch_attn_tc(const AttnParams &p, int head_dim, bool e4m3, int sms, bool chained, cudaStream_t st);

// The decode kernel (head_dim 64 and 128), one CTA of kDecodeWarps ranges per SM.
constexpr int kDecodeWarps = 8;
cudaError_t launch_attn_decode(const AttnParams &p, int head_dim, bool e4m3, int sms, cudaStream_t st);

}  // namespace moe
