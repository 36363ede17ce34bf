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
//   - a block is worked on in two halves of 64 keys with their own columns of S:
//     the scores of one half are made while the softmax of the other runs, so the
//     softmax never waits for its own products;
//   - P takes the place of S in tensor memory and is the A operand of the second
//     product from there: it never goes through shared memory.  It has the type of V,
//     as one MMA's operands must: bf16, or with codes fp16.  A second bf16 part, as
//     decode has, would double the second product; without it the error against 64 bits is
//     0.0021 to 0.0023 of the output's norm where the output's own rounding gives 0.0017;
//   - O stays in tensor memory.  Its rows are rescaled only when their maximum
//     has grown by more than 2^8 since the last time (until then p may exceed 1,
//     which costs nothing in 16 bits and in fp32 sums);
//   - an item's Q is loaded when the last scores of the item before are done, and
//     its first scores are issued behind that item's last products, so that they
//     run while its output is written.
// Measured: 1024 tokens over 32768 keys, 32 and 8 heads of 128, bf16: 525 us, 1030
// TFLOP/s, in ten replays of a graph, 605 us in a long run, where the power limit
// brings the SMs from 1.97 to 1.54 GHz (a library product of the same length reaches
// 1391); every form of the softmax tried gave the burst figure within 1%: turns at
// the exponentials, part of them as polynomials on the fp32 pipe, other orders, the
// next scores fetched early.  4 prompts of 2048 tokens: 182 and 196 us, of which the ends
// of items (5000 cycles each for the output) and their first blocks are a third; both
// are on the softmax warps, as O's rescaling is.
// A tile holds whole tokens: tile_rows / 2 = group * floor(128 / group) rows.
// Warp roles: 0-3 and 4-7 softmax of tile 0 and 1 and the output, 8 and 9 issue the
// MMAs of tile 0 and 1 (apart, because a wait of one must not hold up the other)
// and load its Q.  K and V blocks share one ring of slots in the order K0 V0 K1 V1
// ...  Three ways to fill it:
//   kLoadTma    bf16 cache whose pages a block is made of, or that are made of
//               blocks: warp 10 issues one TMA box per page and 64 columns, whose
//               page ids its lanes read side by side;
//   kLoadCopy   any other page size: warps 12-15 copy rows with cp.async, and hand a
//               block over once its copies have landed;
//   kLoadCodes  E4M3 cache: warps 12-15 copy codes ahead and convert them, K to bf16
//               and V to fp16, into the ring.
#include <mutex>

#include "paged_mma.cuh"
#include "paged_work.cuh"

namespace moe {

// How K and V get into shared memory.
enum { kLoadTma = 0, kLoadCopy = 1, kLoadCodes = 2 };

template <int kD, int kLoad>
struct TcCfg {
    static constexpr int kThreads = kLoad == kLoadTma ? 384 : 512, kBlk = 128;
    static constexpr int kHalf = 128 * 128;                  // bytes of 128 rows x 64 columns
    static constexpr int kHalves = kD / 64;
    static constexpr int kTile = kHalves * kHalf;            // 128 rows x D
    static constexpr int kSlots = kD == 64 ? 8 : kLoad == kLoadCodes ? 4 : 5;
    // codes on their way: kDepth blocks of K or V
    static constexpr int kDepth = kD == 64 ? 4 : 2, kRaw = kLoad == kLoadCodes ? kDepth * 128 * kD : 0;
    static constexpr int kSmem = 2 * kTile + kSlots * kTile + kRaw + 1024;   // + alignment
    static constexpr int kColS = 0, kColO = 256;             // tensor-memory columns, tile t at + 128 t
};

constexpr float kRescale = 8.0f;                             // log2 of the growth that is let stand

// One lane of a converged warp.  Code under it is known to the compiler to run in
// one thread, which tcgen05 instructions want (their operands are uniform
// registers): under a plain test of the lane each MMA took some 100 cycles to issue.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

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

// The loads before it have landed.  The operands tie the values to it, so that
// nothing computed from them moves before it.
__device__ __forceinline__ void tmem_landed(float *r)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                   "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]),
                   "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]),
                   "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two fp16 values that came from E4M3 codes as bf16, exactly.
__device__ __forceinline__ uint32_t bf16x2_of_f16x2(uint32_t h)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return bf16x2_of(f.x, f.y);
}

// 32 bytes of a lane's own row: one store of a whole sector where the buffer allows
// it.  A warp's store touches 32 rows, and takes as long whatever it brings to each.
__device__ __forceinline__ void put_32b(void *dst, const uint32_t (&y)[8], bool wide)
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]),
                     "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
}

// 16-code chunk `chunk` of rows row, row + kStep, ... into an operand tile, as bf16
// or fp16, both exactly.  Lanes of the second half of the columns start with their
// odd 16 bytes, so that the 8 lanes of a row hit 8 different bank groups.
template <int kHalf, int kStep, bool kBf16, int kN>
__device__ __forceinline__ void put_codes(uint8_t *tile, int row, int chunk, const uint4 (&from)[kN])
{
    uint8_t *dst = tile + (chunk >> 2) * kHalf;
    const int k = 2 * (chunk & 3), e0 = chunk >> 2 & 1;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int r = row + i * kStep;
        const uint32_t ww[4] = {from[i].x, from[i].y, from[i].z, from[i].w};
        uint32_t x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f16x4_of_e4m3(ww[j], x[2 * j], x[2 * j + 1]);
            if (kBf16) {
                x[2 * j] = bf16x2_of_f16x2(x[2 * j]);
                x[2 * j + 1] = bf16x2_of_f16x2(x[2 * j + 1]);
            }
        }
        const uint4 even = make_uint4(x[0], x[1], x[2], x[3]), odd = make_uint4(x[4], x[5], x[6], x[7]);
        *reinterpret_cast<uint4 *>(dst + r * 128 + ((k + e0) ^ (r & 7)) * 16) = e0 ? odd : even;
        *reinterpret_cast<uint4 *>(dst + r * 128 + ((k + 1 - e0) ^ (r & 7)) * 16) = e0 ? even : odd;
    }
}

template <int kD, int kLoad>
__global__ void __launch_bounds__(TcCfg<kD, kLoad>::kThreads, 1)
    paged_attention_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                              const __grid_constant__ CUtensorMap tm_v, const AttnParams p, int box_rows)
{
    using C = TcCfg<kD, kLoad>;
    constexpr int kBlk = C::kBlk, kSlots = C::kSlots;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t s_full[kSlots], s_empty[kSlots], s_qfull[2], s_sfull[2][2], s_pfull[2][2],
        s_pv[2][2], s_drain[2];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t *s_q = smem;
    const uint32_t ring = smem_u32(smem + 2 * C::kTile);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_u32(&s_full[i]), kLoad == kLoadTma ? 1 : 4);     // the load warps
            mbar_init(smem_u32(&s_empty[i]), 2);             // both tiles
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&s_qfull[t]), 1);
            for (int x = 0; x < 2; ++x) {
                mbar_init(smem_u32(&s_sfull[t][x]), 1);
                mbar_init(smem_u32(&s_pfull[t][x]), 4);
                mbar_init(smem_u32(&s_pv[t][x]), 1);
            }
            mbar_init(smem_u32(&s_drain[t]), 1);
        }
        s_abort = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
    }
    if (tid == 32) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    tc_fence_before();
    __shared__ Split<C::kThreads, 0, kBlk> s_split;          // wanted once more, at the end
    Split<C::kThreads, 0, kBlk> split;
    Cursor<0, kBlk> cur;
    const int n_blocks = static_cast<int>(split.init(p, cur, reinterpret_cast<long long *>(smem)));      // has block barriers
    tc_fence_after();
    if (tid == 0) s_split = split;
    fence_async_smem();                                      // its shared memory is TMA's now
    __syncthreads();
    grid_dep_launch();
    if (n_blocks == 0) {
        if (tid == 0) p.desc[blockIdx.x].parts = 0;
        if (warp == 8) tmem_dealloc(s_tmem, 512);
        if (p.wait_at_end) grid_dep_wait();
        return;
    }
    const uint32_t tmem = s_tmem;
    // a wait's answer is the whole warp's
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, attn_wait(smem_u32(bar), parity, &s_abort));
    };
    const int tile = p.tile_rows >> 1;                       // rows of a tile, at most 128
    int left = n_blocks;
    // 16 warps x 128 registers at launch = 8 x 160 + 8 x 96: a softmax thread holds
    // 64 scores
    if (kLoad != kLoadTma && warp >= 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (kLoad == kLoadTma && warp == 10) {
        // ------------------------------------------------ K and V loads by TMA
        // lane: box of rows row .. row + box_rows - 1 of the block, columns 64 h ..
        const int boxes = kBlk / box_rows;
        const int h = lane / boxes, row = lane % boxes * box_rows;
        const bool mine = h < C::kHalves;
        const uint64_t policy = policy_evict_normal();
        bool bad = false;
        int slot = 0;
        uint32_t phase = 0, n_fill = 0;
        auto page_of = [&](const Cursor<0, kBlk> &at) {  // -1: no such key
            const int key = at.blk * kBlk + row;
            if (!mine || key >= at.r.kv) return -1;
            int id = __ldg(p.table + static_cast<long long>(at.b) * p.max_pages + p.by_page.div(key));
            if (id < 0 || id >= p.num_pages) {
                bad = true;
                id = p.num_pages;                            // outside the map: zeros
            }
            return id;
        };
        int id = page_of(cur);
        bool ok = true;
        while (ok) {
            const int key = cur.blk * kBlk + row, off = key - p.by_page.div(key) * p.page_size, kvh = cur.kvh;
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
                if (lane == 0) mbar_arrive_expect_tx(bar, n_box * box_rows * 128);
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
    } else if (kLoad != kLoadTma && warp >= 12) {
        // ---------------------------- K and V loads, 32 rows of a block a warp
        // Lane r looks up row r's page: any page size; keys behind the last one, or
        // on a page outside the cache, become zeros.
        constexpr int esz = kLoad == kLoadCodes ? 1 : 2, kPerRow = kD * esz / 16, kAtOnce = 32 / kPerRow, kCopies = 32 / kAtOnce;
        const int first = 32 * (warp - 12), sub = lane / kPerRow, chunk = lane % kPerRow;
        bool bad = false, ok = true;
        int slot = 0;
        uint32_t phase = 0;
        auto look_up = [&]() -> long long {                  // the row's place in bytes, -1: none
            const int key = cur.blk * kBlk + first + lane;
            if (key >= cur.r.kv) return -1;
            const int col = p.by_page.div(key);
            const int id = __ldg(p.table + static_cast<long long>(cur.b) * p.max_pages + col);
            if (id < 0 || id >= p.num_pages) {
                bad = true;
                return -1;
            }
            return (id * p.page_stride + (static_cast<long long>(key - col * p.page_size) * p.n_kv + cur.kvh) * kD) * esz;
        };
        auto landed = [&](int at) {                          // a slot's rows are written: hand them over
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s_full[at]));
        };
        auto step = [&]() {
            if (++slot == kSlots) {
                slot = 0;
                phase ^= 1u;
            }
        };
        long long off = look_up();
        auto advance = [&]() -> long long {                  // the next block's place
            if (left == 0 || --left == 0) return -1;
            if (++cur.blk == cur.nblk) cur.next_item(p);
            return look_up();
        };
        if constexpr (kLoad == kLoadCopy) {
            int open0 = -1, open1 = -1;                      // slots whose copies are under way, oldest first
            auto flush = [&]() {
                copies_wait<0>();
                if (open0 >= 0) landed(open0);
                if (open1 >= 0) landed(open1);
                open0 = open1 = -1;
            };
            while (left > 0 && ok) {
                const long long next = advance();
#pragma unroll
                for (int kv = 0; kv < 2 && ok; ++kv) {
                    // a slot that is not free yet may be waiting for copies not handed over
                    if (!__all_sync(0xffffffffu, mbar_try_wait(smem_u32(&s_empty[slot]), phase ^ 1u))) {
                        flush();
                        ok = wait(&s_empty[slot], phase ^ 1u);
                        if (!ok) break;
                    }
                    const uint8_t *cache = static_cast<const uint8_t *>(kv ? p.v_cache : p.k_cache);
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) {
                        const long long o = __shfl_sync(0xffffffffu, off, i * kAtOnce + sub);
                        const int r = first + i * kAtOnce + sub;
                        copy16(ring + slot * C::kTile + (chunk >> 3) * C::kHalf + r * 128 + ((chunk & 7) ^ (r & 7)) * 16,
                               cache + (o < 0 ? 0 : o) + chunk * 16, o >= 0);
                    }
                    copies_commit();
                    if (open1 >= 0) {
                        copies_wait<2>();
                        landed(open0);
                        open0 = open1;
                        open1 = slot;
                    } else if (open0 >= 0) {
                        open1 = slot;
                    } else {
                        open0 = slot;
                    }
                    step();
                }
                off = next;
            }
            flush();
        } else if constexpr (kLoad == kLoadCodes) {
            // The codes of K or V blocks are copied kDepth ahead; K becomes bf16
            // (like q), V fp16 (like p), both exactly.  A lane converts what it
            // copied itself.
            const uint32_t raw = ring + kSlots * C::kTile + first * kD + lane * 16;
            int todo = 2 * left;                       // K and V blocks to convert
            int fill = 0;                                    // of the one to copy next, mod kDepth
            bool v_next = false;
            auto copy = [&]() {
                const uint8_t *cache = static_cast<const uint8_t *>(v_next ? p.v_cache : p.k_cache);
#pragma unroll
                for (int i = 0; i < kCopies; ++i) {
                    const long long o = __shfl_sync(0xffffffffu, off, i * kAtOnce + sub);
                    copy16(raw + fill * (128 * kD) + i * 512, cache + (o < 0 ? 0 : o) + chunk * 16, o >= 0);
                }
                copies_commit();
                if (++fill == C::kDepth) fill = 0;
                if (v_next) off = advance();
                v_next = !v_next;
            };
#pragma unroll
            for (int i = 0; i < C::kDepth; ++i) copy();
            for (bool v_now = false; todo > 0; --todo, v_now = !v_now) {
                copies_wait<C::kDepth - 1>();
                uint4 w[kCopies];
#pragma unroll
                for (int i = 0; i < kCopies; ++i)
                    w[i] = *reinterpret_cast<const uint4 *>(smem + (raw - smem_u32(smem)) + fill * (128 * kD) + i * 512);
                ok = wait(&s_empty[slot], phase ^ 1u);
                if (!ok) break;
                copy();
                uint8_t *to = smem + 2 * C::kTile + slot * C::kTile;
                if (!v_now) put_codes<C::kHalf, kAtOnce, true>(to, first + sub, chunk, w);
                else put_codes<C::kHalf, kAtOnce, false>(to, first + sub, chunk, w);
                landed(slot);
                step();
            }
            copies_wait<0>();
        }
        if (bad && p.status) set_status(p.status, MOE_ERR_DEVICE_CHECK);
    } else if (warp == 8 || warp == 9) {
        // ------------------------------------- MMAs of tile t, and its Q
        const int t = warp - 8;
        // P and V are bf16, with a cache of codes fp16; V's rows are the second product's K
        const uint32_t idesc_s = idesc_make(1, 128, 64), idesc_o = idesc_make(kLoad == kLoadCodes ? 0 : 1, 128, kD) | (1u << 16);
        const uint32_t q0 = smem_u32(s_q) + t * C::kTile;
        const uint32_t ts = tmem + C::kColS + 128 * t, to = tmem + C::kColO + 128 * t;
        int slot = 0;                                        // the next fill to wait for
        uint32_t phase = 0, qphase = 0, pphase = 0;
        bool ok = true;
        auto next_fill = [&]() {                             // its slot, once it has landed
            ok = wait(&s_full[slot], phase);
            const int x = slot;
            if (++slot == kSlots) {
                slot = 0;
                phase ^= 1u;
            }
            return x;
        };
        auto scores = [&](int kslot, int half) {             // S half = Q K[64 half ..]^T, by the elected lane
            const uint32_t b = ring + kslot * C::kTile + half * 8192;
#pragma unroll
            for (int ks = 0; ks < kD / 16; ++ks) {
                const uint32_t at = (ks >> 2) * C::kHalf + (ks & 3) * 32;
                mma_bf16(ts + 64 * half, sdesc_k_sw128(q0 + at), sdesc_k_sw128(b + at), idesc_s, ks > 0);
            }
            mma_commit(smem_u32(&s_sfull[t][half]));
        };
        uint32_t q_under_way = 0;
        const uint64_t policy = policy_evict_normal();
        auto load_q = [&](const Cursor<0, kBlk> &at) {       // the tile's rows of an item
            if (t * tile >= at.rows(p)) return;
            if (elect_one()) {
                const uint32_t bar = smem_u32(&s_qfull[t]);
                mbar_arrive_expect_tx(bar, C::kHalves * tile * 128);
                for (int h = 0; h < C::kHalves; ++h)
                    tma_load_3d(q0 + h * C::kHalf, &tm_q, bar, 64 * h, at.kvh * p.group,
                                at.r.qs + p.by_group.div(at.row0(p) + t * tile), policy);
            }
            __syncwarp();
            q_under_way = 1;
        };
        load_q(cur);
        while (left > 0 && ok) {
            const int n = min(left, cur.nblk - cur.blk);
            Cursor<0, kBlk> nxt = cur;
            if (left > n) nxt.next_item(p);
            if (t * tile < cur.rows(p)) {
                int kslot = next_fill();
                if (!ok) break;
                ok = wait(&s_qfull[t], qphase);
                if (!ok) break;
                qphase ^= 1u;
                q_under_way = 0;
                tc_fence_after();
                if (elect_one()) {
                    scores(kslot, 0);
                    scores(kslot, 1);
                    mma_commit(smem_u32(&s_empty[kslot]));
                }
                for (int j = 0; j < n && ok; ++j) {
                    const int vslot = next_fill();
                    if (!ok) break;
                    // values behind the last key must not reach the product: 0 x NaN
                    // (both tiles' warps write the same zeros)
                    const int valid = cur.r.kv - (cur.blk + j) * kBlk;
                    if (kLoad == kLoadTma && valid < kBlk) {
                        uint8_t *v = smem + 2 * C::kTile + vslot * C::kTile;
                        const int from = valid < 0 ? 0 : valid;
                        for (int x = from * 8 + lane; x < kBlk * 8; x += 32)
#pragma unroll
                            for (int h = 0; h < C::kHalves; ++h)
                                *reinterpret_cast<uint4 *>(v + h * C::kHalf + x * 16) = make_uint4(0, 0, 0, 0);
                        fence_async_smem();
                        __syncwarp();
                    }
                    if (j + 1 < n) {
                        kslot = next_fill();
                        if (!ok) break;
                    }
                    // From P's arrival to the next scores' is what a tile waits for, so
                    // nothing stands between: the product, the scores behind it in the
                    // half's columns, and only then who else is told.
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        ok = wait(&s_pfull[t][half], pphase);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t b = ring + vslot * C::kTile + half * 8192;
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                mma_f16_ta(to, ts + 64 * half + 8 * ks, sdesc_mn_sw128(b + ks * 2048, C::kHalf), idesc_o,
                                           j > 0 || half > 0 || ks > 0);
                            if (j + 1 < n) scores(kslot, half);
                            mma_commit(smem_u32(&s_pv[t][half]));
                            if (half == 1) {
                                mma_commit(smem_u32(&s_empty[vslot]));
                                if (j + 1 < n) mma_commit(smem_u32(&s_empty[kslot]));
                            }
                        }
                        __syncwarp();
                    }
                    // the item's last scores are done: its Q may go
                    if (ok && j + 1 == n && left > n) load_q(nxt);
                    pphase ^= 1u;
                }
            } else {
                // no rows for this tile: only give the slots back
                for (int x = 0; x < 2 * n && ok; ++x) {
                    const int f = next_fill();
                    if (ok && lane == 0) mbar_arrive(smem_u32(&s_empty[f]));
                }
                if (ok && left > n) load_q(nxt);
            }
            if (!ok) break;
            left -= n;
            cur = nxt;
        }
        if (!ok) {
            if (elect_one()) {
                volatile int no_abort = 0;
                if (q_under_way) mbar_wait(smem_u32(&s_qfull[t]), qphase, &no_abort);
                mma_commit(smem_u32(&s_drain[t]));
                mbar_wait(smem_u32(&s_drain[t]), 0, &no_abort);
            }
            __syncwarp();
        }
    } else if (warp < 8) {
        // ------------------------------------------- softmax of tile t, a row each
        if (kLoad != kLoadTma) asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;      // lane 32 (warp mod 4) in bits 16..
        const uint32_t ts = tmem + C::kColS + 128 * t + lanes, to = tmem + C::kColO + 128 * t + lanes;
        const float mult = p.scale_log2;                                   // > 0: a masked -inf stays one
        uint32_t ph = 0;                                     // of the barriers of the block's two halves
        bool ok = true, continued = cur.blk > 0;
        int item_from = 0;
        while (left > 0 && ok) {
            const int n = min(left, cur.nblk - cur.blk);
            const bool last = cur.blk + n == cur.nblk;
            const int rows = cur.rows(p);
            if (t * tile < rows) {
                const int row = t * tile + r;
                const bool real = r < tile && row < rows;
                const int lim = real ? row_limit(p, cur.r, cur.row0(p) + row) : 0;
                float m = -INFINITY, l = 0.0f;               // m: largest q.k that O is relative to
                for (int x = 0; x < 2 * n; ++x) {            // blocks of 64 keys
                    const int half = x & 1;
                    ok = wait(&s_sfull[t][half], ph);
                    if (!ok) break;
                    tc_fence_after();
                    float s[64];
                    tmem_ld32(ts + 64 * half, s);
                    tmem_ld32(ts + 64 * half + 32, s + 32);
                    tmem_landed(s);
                    tmem_landed(s + 32);
                    const int seen = lim - (cur.blk * kBlk + 64 * x);
                    if (__any_sync(0xffffffffu, seen < 64)) {
#pragma unroll
                        for (int i = 0; i < 64; ++i) s[i] = i < seen ? s[i] : -INFINITY;
                    }
                    float top[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) top[e] = max3(s[e], s[8 + e], s[16 + e]);
#pragma unroll
                    for (int i = 24; i < 56; i += 16)
#pragma unroll
                        for (int e = 0; e < 8; ++e) top[e] = max3(top[e], s[i + e], s[i + 8 + e]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) top[e] = fmaxf(top[e], s[56 + e]);
                    const float mn = max3(max3(m, top[0], top[1]), max3(top[2], top[3], top[4]), max3(top[5], top[6], top[7]));
                    if (__any_sync(0xffffffffu, (mn - m) * mult > kRescale)) {
                        // (mn = m = -inf gives NaN above and does not count)
                        const float f = m == -INFINITY ? 0.0f : exp2_fast((m - mn) * mult);
                        m = mn;
                        l *= f;
                        if (x > 0) {
                            ok = wait(&s_pv[t][half ^ 1], half ? ph : ph ^ 1u);      // O at rest
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int c = 0; c < kD; c += 32) {
                                float o[32];
                                tmem_ld32(to + c, o);
                                tmem_landed(o);
#pragma unroll
                                for (int i = 0; i < 32; ++i) o[i] *= f;
                                tmem_st32(to + c, o);
                            }
                        }
                    }
                    const float base = m == -INFINITY ? 0.0f : kLoad == kLoadCodes ? __fmaf_rn(m, mult, -kF16UpLag) : m * mult;
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                    const float2 mult2 = make_float2(mult, mult), base2 = make_float2(-base, -base);
#pragma unroll
                    for (int c = 0; c < 64; c += 32) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 v = __ffma2_rn(make_float2(s[c + i], s[c + i + 1]), mult2, base2);
                            const float2 e = make_float2(exp2_fast(v.x), exp2_fast(v.y));
                            sum[(i >> 1) & 1] = __fadd2_rn(sum[(i >> 1) & 1], e);
                            w[i >> 1] = kLoad == kLoadCodes ? f16x2_of(e.x, e.y) : bf16x2_of(e.x, e.y);
                        }
                        tmem_st16(ts + 64 * half + c / 2, w);
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&s_pfull[t][half]));
                    ph ^= half;
                }
                if (ok) ok = wait(&s_pv[t][1], ph ^ 1u);
                if (!ok) break;
                tc_fence_after();
                if (last && !continued) {
                    const float inv = row_inverse(l), vs = kLoad == kLoadCodes ? p.v_scale : 1.0f;
                    const int grow = cur.row0(p) + row, tok = p.by_group.div(grow);
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) +
                                         (static_cast<long long>(cur.r.qs + tok) * p.n_heads + cur.kvh * p.group + (grow - tok * p.group)) * kD;
                    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
#pragma unroll
                    for (int c = 0; c < kD; c += 32) {
                        float o[32];
                        tmem_ld32(to + c, o);
                        tmem_landed(o);
                        if (real) {
#pragma unroll
                            for (int i = 0; i < 32; i += 16) {
                                uint32_t y[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e) y[e] = bf16x2_of(o[i + 2 * e] * inv * vs, o[i + 2 * e + 1] * inv * vs);
                                put_32b(dst + c + i, y, wide);
                            }
                        }
                    }
                } else {
                    float *part = p.part + (2LL * blockIdx.x + (continued ? 0 : 1)) * (static_cast<long long>(p.tile_rows) * (kD + 2));
#pragma unroll
                    for (int c = 0; c < kD; c += 32) {
                        float o[32];
                        tmem_ld32(to + c, o);
                        tmem_landed(o);
                        if (real) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                *reinterpret_cast<float4 *>(part + many_at(p.tile_rows, row, c + i)) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        }
                    }
                    if (real) {
                        part[p.tile_rows * kD + row] = m == -INFINITY ? m : m * mult;
                        part[p.tile_rows * (kD + 1) + row] = l;
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
                    d.row0 = cur.row0(p);
                    d.rows = rows;
                    if (!last && !continued) d.parts = s_split.parts(blockIdx.x, item_from, cur.nblk);
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

static bool encode(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                   const cuuint32_t *box)
{
    AttnEncodeFn fn = attn_encode_fn();
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void *>(base), dims, strides, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A cache as [num_pages][page_size][n_kv][D] with boxes of box_rows tokens of one
// head and 64 columns.
static bool cache_map(CUtensorMap *m, const void *base, const AttnParams &p, int kD, int box_rows)
{
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(p.n_kv), static_cast<cuuint64_t>(p.page_size),
                                static_cast<cuuint64_t>(p.num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(kD) * 2, static_cast<cuuint64_t>(kD) * 2 * p.n_kv,
                                   static_cast<cuuint64_t>(p.page_stride) * 2};
    const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(box_rows), 1};
    return encode(m, base, 4, dims, strides, box);
}

// Queries as [T][n_heads][D] with boxes of a tile's tokens, one group's heads and
// 64 columns: a tile's rows in their order.
static bool query_map(CUtensorMap *m, const AttnParams &p, int kD)
{
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(p.n_heads), static_cast<cuuint64_t>(p.T)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kD) * 2, static_cast<cuuint64_t>(p.q_stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(128 / p.group)};
    return encode(m, p.q, 3, dims, strides, box);
}

bool attn_tc_takes(const moe_attn_shape_t &s)
{
    // a tile of 128 rows holds whole tokens, the maximum of q.k is that of the scores
    // (and times the scale still -inf where it is); the query map's stride is below
    // 2^40 bytes
    if (s.head_dim != 64 && s.head_dim != 128) return false;
    return s.n_heads / s.n_kv_heads <= 128 && attn_scale_log2(s) >= 1e-37f && s.q_stride < 1ll << 39;
}

int attn_tc_rows(const moe_attn_shape_t &s)
{
    const int group = s.n_heads / s.n_kv_heads;
    return 2 * group * (128 / group);
}

template <int kD, int kLoad>
static cudaError_t launch_tc(const AttnParams &p, int sms, bool chained, cudaStream_t st)
{
    using C = TcCfg<kD, kLoad>;
    static PerDeviceOnce once;
    once([] { cudaFuncSetAttribute(paged_attention_tc_kernel<kD, kLoad>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem); });
    const int box_rows = p.page_size < 128 ? p.page_size : 128;
    CUtensorMap q, k, v;
    if (!query_map(&q, p, kD)) return cudaErrorInvalidValue;
    k = v = q;
    if (kLoad == kLoadTma && (!cache_map(&k, p.k_cache, p, kD, box_rows) || !cache_map(&v, p.v_cache, p, kD, box_rows)))
        return cudaErrorInvalidValue;
    return launch_kernel(paged_attention_tc_kernel<kD, kLoad>, dim3(sms), dim3(C::kThreads), C::kSmem, st, chained, q, k, v, p, box_rows);
}

cudaError_t launch_attn_tc(const AttnParams &p, int head_dim, bool e4m3, int sms, bool chained, cudaStream_t st)
{
    // TMA takes a block as whole boxes: pages that divide it (8 rows at least, the
    // swizzle's pattern), or that it divides.  Against row copies, in replays of a graph:
    // 4 prompts of 2048 tokens 183 to 222 us, a mixed batch with 16-token pages 137 to 172.
    const bool boxes = ((p.page_size >= 8 && 128 % p.page_size == 0) || p.page_size % 128 == 0) && p.page_stride < 1ll << 39;
    if (head_dim == 64)
        return e4m3    ? launch_tc<64, kLoadCodes>(p, sms, chained, st)
               : boxes ? launch_tc<64, kLoadTma>(p, sms, chained, st)
                       : launch_tc<64, kLoadCopy>(p, sms, chained, st);
    return e4m3    ? launch_tc<128, kLoadCodes>(p, sms, chained, st)
           : boxes ? launch_tc<128, kLoadTma>(p, sms, chained, st)
                   : launch_tc<128, kLoadCopy>(p, sms, chained, st);
}

}  // namespace moe
