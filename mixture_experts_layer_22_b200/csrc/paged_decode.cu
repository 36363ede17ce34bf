// paged_decode.cu - attention over a paged cache for requests with at most 16
// query rows (the heads of a group, times a few tokens): decode.
//
// A decode step reads every key and value of its requests once and does 4 group
// operations per element, so HBM bounds it: at 64 requests of up to 8192 keys
// 1.08 GB, 165 us at the measured copy rate.  What that takes is bytes in flight
// from the first moment to the last on every SM, and few instructions per byte:
//   - one CTA per SM with a ring of blocks of keys and values, nearly all of the
//     shared memory.  Four warps fill it with cp.async, 16 bytes a lane, a page
//     lookup per row (any page size; keys behind the last one, or on a page
//     outside the cache, become zeros).  They run ahead of the others over the
//     borders of items, so that short sequences keep the ring full too.  (TMA
//     boxes of a page each were slower: 4.0 TB/s with 16-token pages, 5.7 with
//     128-token pages.)
//   - the other warps take the blocks in turn, each on its own: a warp multiplies
//     its block with the item's rows, keeps its own running maximum, sum and
//     output, and gives the slot back.  Nothing synchronises them until the end
//     of an item, where their results are put together in warp order; an item of
//     one block is written by its warp alone.  The number of slots is a multiple
//     of the warps of either kind, so a slot is always the same warp's: copies land
//     out of order, and a warp that waited for a slot's next filling without having seen
//     the one before would take that one's parity for its own.
//
// Products run on mma.sync m16n8k16, whose 16 rows the heads of a group fill;
// tcgen05's 128 would be nearly empty, and the tensor pipe is idle most of the
// time either way.
#include "paged_mma.cuh"
#include "paged_work.cuh"

namespace moe {

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
// Arrive on `bar` when every earlier copy of this thread has landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <int kD, bool kE4m3>
struct DecCfg {
    // codes take half the bytes, and their conversion as many instructions again:
    // twice the warps
    static constexpr int kWarps = kE4m3 ? 8 : 4, kLoaders = 4, kThreads = 32 * (kWarps + kLoaders);
    static constexpr int kRowBytes = kD * (kE4m3 ? 1 : 2), kChunks = kRowBytes / 16;
    static constexpr int kRows = 16, kBlk = kRowBytes == 256 ? 32 : 64;
    static constexpr int kMat = kBlk * kRowBytes, kStage = 2 * kMat;     // K, then V
    static constexpr int kMerge = kWarps * kRows * kD * 4;
    static constexpr int kFit = (229376 - kMerge) / kStage / kWarps * kWarps;
    static constexpr int kStages = kFit < 16 ? kFit : 16;
    static_assert(kStages % kWarps == 0 && kStages % kLoaders == 0, "a slot belongs to one warp of either kind");
    static constexpr int kSmem = kStages * kStage + kMerge;
};

template <int kD, bool kE4m3>
__global__ void __launch_bounds__(DecCfg<kD, kE4m3>::kThreads, 1) paged_decode_kernel(const AttnParams p)
{
    using C = DecCfg<kD, kE4m3>;
    constexpr int kBlk = C::kBlk, kRows = C::kRows, kWarps = C::kWarps, kStages = C::kStages, kChunks = C::kChunks;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t s_full[kStages], s_empty[kStages];
    __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
    __shared__ volatile int s_abort;
    float *s_merge = reinterpret_cast<float *>(smem + kStages * C::kStage);
    const uint32_t ring = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&s_full[i]), 32);
            mbar_init(smem_u32(&s_empty[i]), 1);
        }
        s_abort = 0;
        fence_mbar_init();
    }
    Split<C::kThreads, kRows, kBlk> split;
    Cursor<kRows, kBlk> cur;
    const int n_blocks = static_cast<int>(split.init(p, cur));           // has block barriers
    grid_dep_launch();
    if (n_blocks == 0) {
        if (tid == 0) p.desc[blockIdx.x].parts = 0;
        return;
    }

    if (warp >= kWarps) {
        // -------------------------------------------------------------- loads
        // The load warps take the blocks in turn.  Lane r looks up the page of row r
        // (and of row r + 32), one of its blocks ahead; a copy takes 32 / kChunks rows.
        constexpr int kLook = (kBlk + 31) / 32, kAtOnce = 32 / kChunks;
        constexpr int esz = kE4m3 ? 1 : 2;
        const int sub = lane / kChunks, chunk = lane % kChunks;
        bool bad = false, ok = true;
        int slot = warp - kWarps;
        uint32_t phase = 0;
        auto look_up = [&](long long (&off)[kLook]) {        // byte offsets of this lane's rows, -1: none
#pragma unroll
            for (int j = 0; j < kLook; ++j) {
                const int key = cur.blk * kBlk + 32 * j + lane;
                off[j] = -1;
                if (key >= cur.r.kv) continue;
                const int col = key / p.page_size;
                const int id = __ldg(p.table + static_cast<long long>(cur.b) * p.max_pages + col);
                if (id < 0 || id >= p.num_pages) bad = true;
                else off[j] = (id * p.page_stride + (static_cast<long long>(key - col * p.page_size) * p.n_kv + cur.kvh) * kD) * esz;
            }
        };
        auto advance = [&](int blocks) {
            for (int x = 0; x < blocks; ++x)
                if (++cur.blk == cur.nblk) cur.next_item(p);
        };
        long long off[kLook], next[kLook];
        if (slot < n_blocks) {
            advance(slot);
            look_up(off);
        }
        for (int i = slot; i < n_blocks; i += C::kLoaders) {
            if (i + C::kLoaders < n_blocks) {
                advance(C::kLoaders);
                look_up(next);
            }
            ok = __all_sync(0xffffffffu, attn_wait(smem_u32(&s_empty[slot]), phase ^ 1u, &s_abort));
            if (!ok) break;
            const uint32_t dst = ring + slot * C::kStage;
#pragma unroll
            for (int r0 = 0; r0 < kBlk; r0 += kAtOnce) {
                const long long o = __shfl_sync(0xffffffffu, off[r0 / 32], r0 % 32 + sub);
                const int r = r0 + sub;
                const long long at = (o < 0 ? 0 : o) + chunk * 16;
                const uint32_t d = dst + r * C::kRowBytes + chunk_of<kChunks>(r, chunk) * 16;
                copy16(d, static_cast<const uint8_t *>(p.k_cache) + at, o >= 0);
                copy16(d + C::kMat, static_cast<const uint8_t *>(p.v_cache) + at, o >= 0);
            }
            copies_arrive(smem_u32(&s_full[slot]));
            if ((slot += C::kLoaders) >= kStages) {
                slot -= kStages;
                phase ^= 1u;
            }
#pragma unroll
            for (int j = 0; j < kLook; ++j) off[j] = next[j];
        }
        copies_wait();
        if (bad && p.status) set_status(p.status, MOE_ERR_DEVICE_CHECK);
        if (!ok && lane == 0 && p.status) set_status(p.status, MOE_ERR_TIMEOUT);
        return;
    }

    // ------------------------------------------------------------- products
    // After a wait that ran out nothing is left out but the waiting: the results
    // are void, and every warp still meets the others at the end of an item.
    const int cq = lane & 3, r_lo = lane >> 2;
    uint32_t qf[kD / 16][4];
    float o[kD / 8][4], m[2], l[2], mult[2];
    int lim[2];
    int slot = warp;
    uint32_t phase = 0;
    int mine = warp, begin = 0;                              // my next block; the item's first one
    bool continued = cur.blk > 0;
    // column of element e of the accumulator's tile i
    auto col = [&](int i, int e) { return kE4m3 ? 16 * (i >> 1) + 4 * cq + 2 * e + (i & 1) : 8 * i + 2 * cq + e; };
    auto out_row = [&](int grow) {
        return static_cast<__nv_bfloat16 *>(p.out) + (static_cast<long long>(cur.r.qs + grow / p.group) * p.n_heads +
                                                      cur.kvh * p.group + grow % p.group) * kD;
    };
    for (;;) {
        const int n = min(n_blocks - begin, cur.nblk - cur.blk);
        const bool last = cur.blk + n == cur.nblk, whole = last && !continued;
        const int rows = cur.rows(p), row0 = cur.row0(p);
        float *part = p.part + (2LL * blockIdx.x + (continued ? 0 : 1)) * (kRows * (kD + 2));
#pragma unroll
        for (int i = 0; i < kD / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.0f;
        if (mine < begin + n) {
            // the item's query rows as A fragments.  For an E4M3 cache in fp16 (see
            // row_power), and a lane takes 4 adjacent elements of 16 where the plain
            // fragment has two pairs: the order in which ldmatrix delivers codes.
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = r_lo + 8 * h, grow = row0 + r;
                const bool real = r < rows;
                const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.q) +
                                           static_cast<long long>(cur.r.qs + grow / p.group) * p.q_stride +
                                           static_cast<long long>(cur.kvh * p.group + grow % p.group) * kD;
                lim[h] = real ? row_limit(p, cur.r, grow) : 0;
                mult[h] = p.scale_log2;
#pragma unroll
                for (int ks = 0; ks < kD / 16; ++ks) {
                    if constexpr (kE4m3) {
                        const uint2 w = real ? __ldg(reinterpret_cast<const uint2 *>(src + 16 * ks + 4 * cq)) : make_uint2(0, 0);
                        qf[ks][h] = w.x;
                        qf[ks][2 + h] = w.y;
                    } else {
                        qf[ks][h] = real ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * ks + 2 * cq)) : 0;
                        qf[ks][2 + h] = real ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * ks + 8 + 2 * cq)) : 0;
                    }
                }
                if constexpr (kE4m3) {
                    float amax = 0.0f;
#pragma unroll
                    for (int ks = 0; ks < kD / 16; ++ks)
#pragma unroll
                        for (int e = h; e < 4; e += 2) amax = fmaxf(amax, fmaxf(fabsf(lo_of(qf[ks][e])), fabsf(hi_of(qf[ks][e]))));
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                    const int up = row_power(amax);
                    const float f = power_of_two(up);
                    mult[h] *= power_of_two(-up);
#pragma unroll
                    for (int ks = 0; ks < kD / 16; ++ks)
#pragma unroll
                        for (int e = h; e < 4; e += 2) qf[ks][e] = f16x2_of(lo_of(qf[ks][e]) * f, hi_of(qf[ks][e]) * f);
                }
            }
        }
        for (; mine < begin + n; mine += kWarps) {
            const int key0 = (cur.blk + mine - begin) * kBlk;
            attn_wait(smem_u32(&s_full[slot]), phase, &s_abort);
            __syncwarp();
            const uint32_t kst = ring + slot * C::kStage, vst = kst + C::kMat;
            // chunk c of row r
            auto at = [&](uint32_t base, int r, int c) { return base + r * C::kRowBytes + chunk_of<kChunks>(r, c) * 16; };
            // scores
            float s[kBlk / 8][4];
#pragma unroll
            for (int i = 0; i < kBlk / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
            if constexpr (!kE4m3) {
#pragma unroll
                for (int ks = 0; ks < kD / 16; ++ks)
#pragma unroll
                    for (int np = 0; np < kBlk / 16; ++np) {
                        uint32_t b[4];
                        ldsm4(b, at(kst, np * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)));
                        mma16816<false>(s[2 * np], qf[ks], b[0], b[1]);
                        mma16816<false>(s[2 * np + 1], qf[ks], b[2], b[3]);
                    }
            } else {
#pragma unroll
                for (int k2 = 0; k2 < kD / 32; ++k2) {
                    uint32_t b[kBlk / 16][4];
#pragma unroll
                    for (int np = 0; np < kBlk / 16; ++np) {
                        // matrices: keys 0-7 and 8-15 at chunk 2 k2, then at 2 k2 + 1
                        ldsm4(b[np], at(kst, np * 16 + (lane & 15), 2 * k2 + (lane >> 4)));
                    }
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                        for (int np = 0; np < kBlk / 16; ++np)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t b0, b1;
                                f16x4_of_e4m3(b[np][2 * kk + h], b0, b1);
                                mma16816<true>(s[2 * np + h], qf[2 * k2 + kk], b0, b1);
                            }
                }
            }
            // mask where the block reaches behind a row's last key, maximum, p
            if (__any_sync(0xffffffffu, key0 + kBlk > min(lim[0], lim[1]))) {
#pragma unroll
                for (int i = 0; i < kBlk / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[i][e] = key0 + 8 * i + 2 * cq + (e & 1) < lim[e >> 1] ? s[i][e] * mult[e >> 1] : -INFINITY;
            } else {
#pragma unroll
                for (int i = 0; i < kBlk / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i][e] *= mult[e >> 1];
            }
            float alpha[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = m[h];
#pragma unroll
                for (int i = 0; i < kBlk / 8; ++i) top = fmaxf(top, fmaxf(s[i][2 * h], s[i][2 * h + 1]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float base = top == -INFINITY ? 0.0f : top;        // a row that has seen nothing yet
                alpha[h] = exp2_fast(m[h] - base);
                m[h] = top;
                l[h] *= alpha[h];
#pragma unroll
                for (int i = 0; i < kBlk / 8; ++i)
#pragma unroll
                    for (int e = 2 * h; e < 2 * h + 2; ++e) {
                        s[i][e] = exp2_fast(s[i][e] - base);
                        l[h] += s[i][e];
                    }
            }
            if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
                for (int i = 0; i < kD / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][e] *= alpha[e >> 1];
            }
            // o += p v.  With a bf16 cache p goes in as two bf16, high and low
            // part: tensor work that is idle here, and the output's own rounding
            // stays the only one of 8 bits.  With codes p is fp16 (11 bits).
#pragma unroll
            for (int kt = 0; kt < kBlk / 16; ++kt) {
                uint32_t ph[4], pl[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = s[2 * kt + (j >> 1)][2 * (j & 1)], b = s[2 * kt + (j >> 1)][2 * (j & 1) + 1];
                    if constexpr (kE4m3) {
                        ph[j] = f16x2_of(a, b);
                    } else {
                        ph[j] = bf16x2_of(a, b);
                        pl[j] = bf16x2_of(a - lo_of(ph[j]), b - hi_of(ph[j]));
                    }
                }
                // the products of one accumulator are kept apart
                if constexpr (!kE4m3) {
#pragma unroll
                    for (int d4 = 0; d4 < kChunks / 2; d4 += 4) {
                        uint32_t b[4][4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) ldsm4_t(b[x], at(vst, kt * 16 + (lane & 15), 2 * (d4 + x) + (lane >> 4)));
#pragma unroll
                        for (int part_p = 0; part_p < 2; ++part_p)
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                mma16816<false>(o[2 * (d4 + x)], part_p ? pl : ph, b[x][0], b[x][1]);
                                mma16816<false>(o[2 * (d4 + x) + 1], part_p ? pl : ph, b[x][2], b[x][3]);
                            }
                    }
                } else {
#pragma unroll
                    for (int dp = 0; dp < kChunks / 2; ++dp) {
                        uint32_t b[4];
                        ldsm4_t(b, at(vst, kt * 16 + (lane & 15), 2 * dp + (lane >> 4)));
                        // a 16-bit unit holds elements 2n and 2n + 1 of one key: tile
                        // 2 ch takes the even ones of chunk ch, 2 ch + 1 the odd ones
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t x0, x1, y0, y1;
                            f16x4_of_e4m3(__byte_perm(b[2 * h], 0, 0x3120), x0, x1);
                            f16x4_of_e4m3(__byte_perm(b[2 * h + 1], 0, 0x3120), y0, y1);
                            const int ch = 2 * dp + h;
                            mma16816<true>(o[2 * ch], ph, x0, y0);
                            mma16816<true>(o[2 * ch + 1], ph, x1, y1);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s_empty[slot]));
            if ((slot += kWarps) >= kStages) {
                slot -= kStages;
                phase ^= 1u;
            }
            if (n == 1) {
                // the item's only block here: no other warp has to do with it
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                    const int r = r_lo + 8 * h;
                    if (r >= rows) continue;
                    if (whole) {
                        const float inv = l[h] > 0.0f ? p.v_scale / l[h] : l[h] == 0.0f ? 0.0f : l[h];
                        __nv_bfloat16 *dst = out_row(row0 + r);
#pragma unroll
                        for (int i = 0; i < kD / 8; i += 2) {
                            const float a = o[i][2 * h] * inv, b = o[i][2 * h + 1] * inv, c = o[i + 1][2 * h] * inv, d = o[i + 1][2 * h + 1] * inv;
                            if constexpr (kE4m3) {
                                *reinterpret_cast<uint2 *>(dst + col(i, 0)) = make_uint2(bf16x2_of(a, c), bf16x2_of(b, d));
                            } else {
                                *reinterpret_cast<uint32_t *>(dst + col(i, 0)) = bf16x2_of(a, b);
                                *reinterpret_cast<uint32_t *>(dst + col(i + 1, 0)) = bf16x2_of(c, d);
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < kD / 8; ++i) {
                            part[r * kD + col(i, 0)] = o[i][2 * h];
                            part[r * kD + col(i, 1)] = o[i][2 * h + 1];
                        }
                        if (cq == 0) {
                            part[kRows * kD + r] = m[h];
                            part[kRows * (kD + 1) + r] = l[h];
                        }
                    }
                }
            }
        }
        if (n > 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                const int r = r_lo + 8 * h;
                if (cq == 0) {
                    s_m[warp][r] = m[h];
                    s_l[warp][r] = l[h];
                }
                float *dst = s_merge + (warp * kRows + r) * kD;
#pragma unroll
                for (int i = 0; i < kD / 8; i += 2) {
                    if constexpr (kE4m3) {
                        *reinterpret_cast<float4 *>(dst + col(i, 0)) =
                            make_float4(o[i][2 * h], o[i + 1][2 * h], o[i][2 * h + 1], o[i + 1][2 * h + 1]);
                    } else {
                        *reinterpret_cast<float2 *>(dst + col(i, 0)) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
                        *reinterpret_cast<float2 *>(dst + col(i + 1, 0)) = make_float2(o[i + 1][2 * h], o[i + 1][2 * h + 1]);
                    }
                }
            }
            named_bar_sync(1, 32 * kWarps);
            for (int x = tid; x < rows * (kD / 4); x += 32 * kWarps) {
                const int r = x / (kD / 4), c = x % (kD / 4) * 4;
                float mx = s_m[0][r];
#pragma unroll
                for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][r]);
                const float base = mx == -INFINITY ? 0.0f : mx;
                float lt = 0.0f;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = exp2_fast(s_m[w][r] - base);
                    const float4 y = *reinterpret_cast<const float4 *>(s_merge + (w * kRows + r) * kD + c);
                    lt += f * s_l[w][r];
                    v.x += f * y.x;
                    v.y += f * y.y;
                    v.z += f * y.z;
                    v.w += f * y.w;
                }
                if (whole) {
                    const float inv = lt > 0.0f ? p.v_scale / lt : lt == 0.0f ? 0.0f : lt;
                    *reinterpret_cast<uint2 *>(out_row(row0 + r) + c) =
                        make_uint2(bf16x2_of(v.x * inv, v.y * inv), bf16x2_of(v.z * inv, v.w * inv));
                } else {
                    *reinterpret_cast<float4 *>(part + r * kD + c) = v;
                    if (c == 0) {
                        part[kRows * kD + r] = mx;
                        part[kRows * (kD + 1) + r] = lt;
                    }
                }
            }
            named_bar_sync(1, 32 * kWarps);                  // the merge area may be written again
        }
        begin += n;
        if (begin == n_blocks) {
            if (tid == 0) {
                AttnDesc d;
                d.parts = 0;
                d.qs = cur.r.qs;
                d.kvh = cur.kvh;
                d.row0 = row0;
                d.rows = rows;
                if (!last && !continued) d.parts = split.parts(blockIdx.x, begin - n, cur.nblk);
                p.desc[blockIdx.x] = d;
            }
            break;
        }
        cur.next_item(p);
        continued = false;
    }
}

bool attn_decode_takes(const moe_attn_shape_t &s) { return s.head_dim == 64 || s.head_dim == 128; }

template <int kD, bool kE4m3>
static cudaError_t launch_decode(const AttnParams &p, int ctas, cudaStream_t st)
{
    using C = DecCfg<kD, kE4m3>;
    static PerDeviceOnce once;
    once([] { cudaFuncSetAttribute(paged_decode_kernel<kD, kE4m3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem); });
    return launch_kernel(paged_decode_kernel<kD, kE4m3>, dim3(ctas), dim3(C::kThreads), C::kSmem, st, false, p);
}

cudaError_t launch_attn_decode(const AttnParams &p, int head_dim, bool e4m3, int ctas, cudaStream_t st)
{
    if (head_dim == 64) return e4m3 ? launch_decode<64, true>(p, ctas, st) : launch_decode<64, false>(p, ctas, st);
    return e4m3 ? launch_decode<128, true>(p, ctas, st) : launch_decode<128, false>(p, ctas, st);
}

}  // namespace moe
