// paged_attention_tc.cu - attention over a paged cache for requests with many
// query rows, on tcgen05 with the scores and the output in tensor memory.
//
// Same mathematics and same division of the work as the kernel in
// paged_attention.cu, with items of 256 query rows in two tiles of 128 and
// blocks of 128 keys.  Per tile and block: S = Q K^T (128 x 128 x D), a softmax
// step on S, O += P V (128 x D x 128).  At D = 128 a tensor pipe takes 1024
// cycles for the two products of a tile, and the 16384 exponentials of a tile
// take the special-function units of an SM 1024 cycles as well, so both have to
// run all the time.  Hence
//   - two tiles in turn: while the softmax of one runs, the tensor pipe does the
//     products of the other;
//   - one thread per query row: a warpgroup owns a tile, a thread reads its row
//     of S from tensor memory, and no value crosses threads;
//   - P (bf16) takes the place of S in tensor memory and is the A operand of the
//     second product from there: it never goes through shared memory;
//   - O stays in tensor memory.  Its rows are rescaled only when their maximum
//     has grown by more than 2^8 since the last time (until then p may exceed 1,
//     which costs nothing in bf16 and in fp32 sums).
// Warp roles: 0-3 and 4-7 softmax of tile 0 and 1 (they also bring Q into shared
// memory and write the output), 8 issues the MMAs, 9 the TMA loads, 10 and 11 fill
// their warpgroup up, which hands registers to the softmax: a thread there holds
// its row's 128 scores.  K and V
// blocks share one ring of slots in the order K0 V0 K1 V1 ...; a block is put
// together from one TMA box per page and 64 columns, whose page ids the 32 lanes
// of the load warp read side by side.
#include <atomic>
#include <mutex>

#include <cuda_bf16.h>

#include "paged_work.cuh"
#include "ptx.cuh"

namespace moe {

template <int kD>
struct TcCfg {
    static constexpr int kThreads = 384, kRows = 256, kBlk = 128;
    static constexpr int kHalf = 128 * 128;                  // bytes of 128 rows x 64 columns
    static constexpr int kHalves = kD / 64;
    static constexpr int kTile = kHalves * kHalf;            // 128 rows x D
    static constexpr int kSlots = kD == 128 ? 5 : 8;
    static constexpr int kSmem = 2 * kTile + kSlots * kTile + 1024;   // + alignment
    static constexpr int kColS = 0, kColO = 256;             // tensor-memory columns, tile t at + 128 t
};

constexpr float kRescale = 8.0f;                             // log2 of the growth that is let stand

// Shared-memory descriptor of an operand stored with its M or N dimension
// contiguous, 128-byte swizzle: 64-element blocks `lead` bytes apart along that
// dimension, groups of 8 along K 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t lead)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(lead >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// D += A B with A in tensor memory (two 16-bit K elements per 32-bit column).
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 32 lanes x 32 columns of 32 bits: thread i gets lane (quarter * 32 + i).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
        "%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
        "%30,%31};" ::"f"(r[0]),
        "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]), "f"(r[10]),
        "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]), "f"(r[16]), "f"(r[17]), "f"(r[18]), "f"(r[19]),
        "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]), "f"(r[26]), "f"(r[27]), "f"(r[28]),
        "f"(r[29]), "f"(r[30]), "f"(r[31]), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float tc_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t tc_bf16x2(float a, float b)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Geometry of the cache's tensor maps: box_rows rows of a page per TMA box.
struct TcMaps {
    int box_rows;
};

template <int kD>
__global__ void __launch_bounds__(TcCfg<kD>::kThreads, 1)
    paged_attention_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                              const AttnParams p, const TcMaps maps)
{
    using C = TcCfg<kD>;
    constexpr int kRows = C::kRows, kBlk = C::kBlk, kSlots = C::kSlots;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t s_full[kSlots], s_empty[kSlots], s_qfull[2], s_sfull[2], s_pfull[2], s_ofull[2], s_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *s_q = smem;
    const uint32_t ring = smem_u32(smem + 2 * C::kTile);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&s_empty[i]), 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&s_qfull[t]), 4);
            mbar_init(smem_u32(&s_sfull[t]), 1);
            mbar_init(smem_u32(&s_pfull[t]), 4);
            mbar_init(smem_u32(&s_ofull[t]), 1);
        }
        mbar_init(smem_u32(&s_drain), 1);
        s_abort = 0;
        fence_mbar_init();
    }
    Split<C::kThreads, kRows, kBlk> split;
    Cursor<kRows, kBlk> cur;
    const long long n_blocks = split.init(p, cur);           // ends with a block barrier
    grid_dep_launch();
    if (n_blocks == 0) {
        if (tid == 0) p.desc[blockIdx.x].parts = 0;
        if (p.wait_at_end) grid_dep_wait();
        return;
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    // a wait's answer is the whole warp's
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, &s_abort));
    };
    long long left = n_blocks;
    // 12 warps x 168 registers at launch = 8 x 216 + 4 x 72
    if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 9) {
        // ---------------------------------------------------------- TMA loads
        // lane: box of rows row .. row + box_rows - 1 of the block, columns 64 h ..
        const int boxes = kBlk / maps.box_rows;
        const int h = lane / boxes, row = lane % boxes * maps.box_rows;
        const bool mine = h < C::kHalves;
        const uint64_t policy = policy_evict_normal();
        bool bad = false;
        int slot = 0;
        uint32_t phase = 0, n_fill = 0;
        auto page_of = [&](const Cursor<kRows, kBlk> &at) {  // -1: no such key
            const int key = at.blk * kBlk + row;
            if (!mine || key >= at.r.kv) return -1;
            int id = __ldg(p.table + static_cast<long long>(at.b) * p.max_pages + key / p.page_size);
            if (id < 0 || id >= p.num_pages) {
                bad = true;
                id = p.num_pages;                            // outside the map: zeros
            }
            return id;
        };
        int id = page_of(cur);
        bool ok = true;
        while (ok) {
            const int key = cur.blk * kBlk + row, off = key % p.page_size, kvh = cur.kvh;
            const int n_box = __popc(__ballot_sync(0xffffffffu, id >= 0));
            int next = -1;
            const bool more = --left > 0;
            if (more) {
                if (++cur.blk == cur.nblk) cur.next_item(p);
                next = page_of(cur);
            }
#pragma unroll
            for (int kv = 0; kv < 2 && ok; ++kv) {
                ok = wait(&s_empty[slot], phase ^ 1u);
                if (!ok) break;
                const uint32_t bar = smem_u32(&s_full[slot]);
                if (lane == 0) mbar_arrive_expect_tx(bar, n_box * maps.box_rows * 128);
                __syncwarp();
                if (id >= 0)
                    tma_load_4d(ring + slot * C::kTile + h * C::kHalf + row * 128, kv ? &tm_v : &tm_k, bar, 64 * h, kvh, off, id,
                                policy);
                ++n_fill;
                if (++slot == kSlots) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
            if (!more) break;
            id = next;
        }
        if (bad && p.status) set_status(p.status, MOE_ERR_DEVICE_CHECK);
        if (!ok) {
            // copies that were issued have to land before the CTA leaves
            volatile int no_abort = 0;
            for (uint32_t i = n_fill > kSlots ? n_fill - kSlots : 0; i < n_fill; ++i)
                mbar_wait(smem_u32(&s_full[i % kSlots]), (i / kSlots) & 1u, &no_abort);
        }
    } else if (warp == 8) {
        // --------------------------------------------------------------- MMAs
        const uint32_t idesc_s = idesc_make(1, 128, 128), idesc_o = idesc_make(1, 128, kD) | (1u << 16);
        const uint32_t q0 = smem_u32(s_q);
        int slot = 0;
        uint32_t phase = 0, qphase[2] = {0, 0}, pphase[2] = {0, 0};
        bool ok = true;
        auto scores = [&](int t, int kslot) {
            if (lane == 0) {
                const uint32_t a = q0 + t * C::kTile, b = ring + kslot * C::kTile;
#pragma unroll
                for (int ks = 0; ks < kD / 16; ++ks) {
                    const uint32_t at = (ks >> 2) * C::kHalf + (ks & 3) * 32;
                    mma_bf16(tmem + C::kColS + 128 * t, sdesc_k_sw128(a + at), sdesc_k_sw128(b + at), idesc_s, ks > 0);
                }
                mma_commit(smem_u32(&s_sfull[t]));
            }
        };
        auto next_slot = [&]() {
            if (++slot == kSlots) {
                slot = 0;
                phase ^= 1u;
            }
        };
        while (left > 0 && ok) {
            const int n = static_cast<int>(min(left, static_cast<long long>(cur.nblk - cur.blk)));
            const int tiles = cur.rows(p) > 128 ? 2 : 1;
            ok = wait(&s_full[slot], phase);
            for (int t = 0; t < tiles && ok; ++t) {
                ok = wait(&s_qfull[t], qphase[t]);
                if (!ok) break;
                qphase[t] ^= 1u;
                tc_fence_after();
                scores(t, slot);
            }
            if (!ok) break;
            if (lane == 0) mma_commit(smem_u32(&s_empty[slot]));
            next_slot();
            for (int j = 0; j < n && ok; ++j) {
                const int vslot = slot;
                ok = wait(&s_full[slot], phase);
                if (!ok) break;
                next_slot();
                // values behind the last key must not reach the product: 0 x NaN
                const int valid = cur.r.kv - (cur.blk + j) * kBlk;
                if (valid < kBlk) {
                    uint8_t *v = smem + 2 * C::kTile + vslot * C::kTile;
                    const int from = valid < 0 ? 0 : valid;
                    for (int x = from * 8 + lane; x < kBlk * 8; x += 32)
#pragma unroll
                        for (int h = 0; h < C::kHalves; ++h)
                            *reinterpret_cast<uint4 *>(v + h * C::kHalf + x * 16) = make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                    __syncwarp();
                }
                const int kslot = slot;
                for (int t = 0; t < tiles && ok; ++t) {
                    ok = wait(&s_pfull[t], pphase[t]);
                    if (!ok) break;
                    pphase[t] ^= 1u;
                    tc_fence_after();
                    if (lane == 0) {
                        const uint32_t b = ring + vslot * C::kTile;
#pragma unroll
                        for (int ks = 0; ks < kBlk / 16; ++ks)
                            mma_f16_ta(tmem + C::kColO + 128 * t, tmem + C::kColS + 128 * t + 8 * ks,
                                       sdesc_mn_sw128(b + ks * 2048, C::kHalf), idesc_o, j > 0 || ks > 0);
                    }
                    if (j + 1 < n) {
                        if (t == 0) {
                            ok = wait(&s_full[slot], phase);
                            if (!ok) break;
                        }
                        scores(t, kslot);
                    } else if (lane == 0) {
                        mma_commit(smem_u32(&s_ofull[t]));
                    }
                }
                if (!ok) break;
                if (lane == 0) {
                    mma_commit(smem_u32(&s_empty[vslot]));
                    if (j + 1 < n) mma_commit(smem_u32(&s_empty[kslot]));
                }
                if (j + 1 < n) next_slot();
            }
            left -= n;
            if (left > 0) cur.next_item(p);
        }
        if (!ok) {
            if (lane == 0) {
                volatile int no_abort = 0;
                mma_commit(smem_u32(&s_drain));
                mbar_wait(smem_u32(&s_drain), 0, &no_abort);
            }
            __syncwarp();
        }
    }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ------------------------------------------- softmax of tile t, a row each
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;      // lane 32 (warp mod 4) in bits 16..
        const uint32_t ts = tmem + C::kColS + 128 * t + lanes, to = tmem + C::kColO + 128 * t + lanes;
        const uint32_t flip = p.scale_log2 < 0.0f ? 0x80008000u : 0u;      // a negative scale: -q and its magnitude
        const float mult = fmaxf(fabsf(p.scale_log2), 1e-30f);             // 0 times a masked -inf must stay -inf
        uint32_t sphase = 0, ophase = 0;
        bool ok = true, continued = cur.blk > 0;
        long long item_from = 0;
        while (left > 0 && ok) {
            const int n = static_cast<int>(min(left, static_cast<long long>(cur.nblk - cur.blk)));
            const bool last = cur.blk + n == cur.nblk;
            const int rows = cur.rows(p);
            if (128 * t < rows) {
                const int row = 128 * t + r, grow = cur.row0() + row;
                const bool real = row < rows;
                const long long tok = cur.r.qs + grow / p.group;
                const int head = cur.kvh * p.group + grow % p.group;
                const int lim = real ? row_limit(p, cur.r, grow) : 0;
                {
                    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + tok * p.q_stride +
                                                                       static_cast<long long>(head) * kD);
                    uint8_t *dst = s_q + t * C::kTile + r * 128;
#pragma unroll
                    for (int c = 0; c < kD / 8; ++c) {
                        uint4 w = real ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
                        w.x ^= flip;
                        w.y ^= flip;
                        w.z ^= flip;
                        w.w ^= flip;
                        *reinterpret_cast<uint4 *>(dst + (c >> 3) * C::kHalf + ((c & 7) ^ (r & 7)) * 16) = w;
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&s_qfull[t]));
                }
                float m = -INFINITY, l = 0.0f;               // m: largest q.k that O is relative to
                for (int j = 0; j < n; ++j) {
                    ok = wait(&s_sfull[t], sphase);
                    if (!ok) break;
                    sphase ^= 1u;
                    tc_fence_after();
                    float s[kBlk];
#pragma unroll
                    for (int c = 0; c < kBlk; c += 32) tmem_ld32(ts + c, s + c);
                    tmem_wait_ld();
                    const int seen = lim - (cur.blk + j) * kBlk;
                    if (__any_sync(0xffffffffu, seen < kBlk)) {
#pragma unroll
                        for (int i = 0; i < kBlk; ++i) s[i] = i < seen ? s[i] : -INFINITY;
                    }
                    float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int i = 4; i < kBlk; i += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            top[e] = i + 4 + e < kBlk ? fmaxf(fmaxf(top[e], s[i + e]), s[i + 4 + e]) : fmaxf(top[e], s[i + e]);
                    const float mn = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
                    if (__any_sync(0xffffffffu, (mn - m) * mult > kRescale)) {
                        // (mn = m = -inf gives NaN above and does not count)
                        const float f = m == -INFINITY ? 0.0f : tc_exp2((m - mn) * mult);
                        m = mn;
                        l *= f;
                        if (j > 0) {
#pragma unroll
                            for (int c = 0; c < kD; c += 32) {
                                float o[32];
                                tmem_ld32(to + c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] *= f;
                                tmem_st32(to + c, o);
                            }
                        }
                    }
                    const float base = m == -INFINITY ? 0.0f : m * mult;
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int c = 0; c < kBlk; c += 32) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float a = tc_exp2(fmaf(s[c + i], mult, -base)), b = tc_exp2(fmaf(s[c + i + 1], mult, -base));
                            sum[i & 2] += a;
                            sum[(i & 2) + 1] += b;
                            w[i >> 1] = tc_bf16x2(a, b);
                        }
                        tmem_st16(ts + (c >> 1), w);
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&s_pfull[t]));
                }
                if (ok) ok = wait(&s_ofull[t], ophase);
                if (!ok) break;
                ophase ^= 1u;
                tc_fence_after();
                if (last && !continued) {
                    const float inv = l > 0.0f ? p.v_scale / l : l == 0.0f ? 0.0f : l;
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + (tok * p.n_heads + head) * kD;
#pragma unroll
                    for (int c = 0; c < kD; c += 32) {
                        float o[32];
                        tmem_ld32(to + c, o);
                        tmem_wait_ld();
                        if (real) {
#pragma unroll
                            for (int i = 0; i < 32; i += 8)
                                *reinterpret_cast<uint4 *>(dst + c + i) =
                                    make_uint4(tc_bf16x2(o[i] * inv, o[i + 1] * inv), tc_bf16x2(o[i + 2] * inv, o[i + 3] * inv),
                                               tc_bf16x2(o[i + 4] * inv, o[i + 5] * inv), tc_bf16x2(o[i + 6] * inv, o[i + 7] * inv));
                        }
                    }
                } else {
                    float *part = p.part + (2LL * blockIdx.x + (continued ? 0 : 1)) * (kRows * (kD + 2));
#pragma unroll
                    for (int c = 0; c < kD; c += 32) {
                        float o[32];
                        tmem_ld32(to + c, o);
                        tmem_wait_ld();
                        if (real) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                *reinterpret_cast<float4 *>(part + row * kD + c + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        }
                    }
                    if (real) {
                        part[kRows * kD + row] = m == -INFINITY ? m : m * mult;
                        part[kRows * kD + kRows + row] = l;
                    }
                }
                tc_fence_before();
            }
            left -= n;
            if (left == 0) {
                if (tid == 0) {
                    AttnDesc d;
                    d.parts = 0;
                    d.qs = cur.r.qs;
                    d.kvh = cur.kvh;
                    d.row0 = cur.row0();
                    d.rows = rows;
                    if (!last && !continued) d.parts = split.parts(blockIdx.x, item_from, cur.nblk);
                    p.desc[blockIdx.x] = d;
                }
            } else {
                item_from = n_blocks - left;
                cur.next_item(p);
                continued = false;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && s_abort) {
        p.desc[blockIdx.x].parts = 0;
        if (p.status) set_status(p.status, MOE_ERR_TIMEOUT);
    }
    if (warp == 8) tmem_dealloc(tmem, 512);
    if (p.wait_at_end) grid_dep_wait();
}

// ------------------------------------------------------------------ host side
typedef CUresult (*AttnEncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static AttnEncodeFn attn_encode_fn()
{
    static AttnEncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<AttnEncodeFn>(ptr);
    });
    return fn;
}

// A cache as [num_pages][page_size][n_kv][D] with boxes of box_rows tokens of one
// head and 64 columns.
static bool cache_map(CUtensorMap *m, const void *base, const AttnParams &p, int kD, int box_rows)
{
    AttnEncodeFn fn = attn_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(p.n_kv), static_cast<cuuint64_t>(p.page_size),
                                static_cast<cuuint64_t>(p.num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(kD) * 2, static_cast<cuuint64_t>(kD) * 2 * p.n_kv,
                                   static_cast<cuuint64_t>(p.page_stride) * 2};
    const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(box_rows), 1}, one[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool attn_tc_takes(const moe_attn_shape_t &s)
{
    // a block of 128 keys is made of whole boxes: pages that divide it (the
    // 1024-byte swizzle pattern wants at least 8 rows), or that it divides.  A
    // tensor map's stride is below 2^40 bytes.
    if (s.head_dim != 64 && s.head_dim != 128) return false;
    if (s.cache_dtype != MOE_BF16) return false;
    return (s.page_size >= 8 && 128 % s.page_size == 0) || s.page_size % 128 == 0;
}

int attn_tc_ctas()
{
    static std::atomic<int> cache[64];
    int dev = 0;
    cudaGetDevice(&dev);
    int n = dev >= 0 && dev < 64 ? cache[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (cudaFuncSetAttribute(paged_attention_tc_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcCfg<64>::kSmem) !=
                cudaSuccess ||
            cudaFuncSetAttribute(paged_attention_tc_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcCfg<128>::kSmem) !=
                cudaSuccess)
            return 0;
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (n > kAttnTcMaxCtas) n = kAttnTcMaxCtas;
        if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

cudaError_t launch_attn_tc(const AttnParams &p, int head_dim, int ctas, bool chained, cudaStream_t st)
{
    TcMaps maps;
    maps.box_rows = p.page_size < 128 ? p.page_size : 128;
    CUtensorMap k, v;
    if (!cache_map(&k, p.k_cache, p, head_dim, maps.box_rows) || !cache_map(&v, p.v_cache, p, head_dim, maps.box_rows))
        return cudaErrorInvalidValue;
    if (head_dim == 64)
        return launch_kernel(paged_attention_tc_kernel<64>, dim3(ctas), dim3(TcCfg<64>::kThreads), TcCfg<64>::kSmem, st, chained, k, v, p,
                             maps);
    return launch_kernel(paged_attention_tc_kernel<128>, dim3(ctas), dim3(TcCfg<128>::kThreads), TcCfg<128>::kSmem, st, chained, k, v, p,
                         maps);
}

}  // namespace moe
