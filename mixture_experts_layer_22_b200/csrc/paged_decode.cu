// paged_decode.cu - attention over a paged cache for requests with at most 16
// query rows (the heads of a group, times a few tokens): decode.
//
// A decode step reads every key and value of its requests once and does 4 group
// operations per element, so HBM bounds it: at 64 requests of up to 8192 keys
// 1.08 GB, 165 us at the measured copy rate.  What that takes is bytes in flight
// from the first moment to the last on every SM, and few instructions per byte:
//   - every warp is on its own: it has a range of blocks, a ring of kSlots blocks
//     in shared memory that it fills with cp.async, 16 bytes a lane, and its own
//     running maximum, sum and output.  Nothing synchronises warps, so a warp that
//     begins or ends an item holds up no other, and short sequences cost little;
//   - its load side runs kSlots - 1 blocks ahead, over the borders of items; a lane
//     looks up a row's page one block before the row is copied.  Any page size; keys
//     behind the last one, or on a page outside the cache, become zeros.
//   - heads with short rows are read side by side: two or four warps take the same
//     keys of heads next to one another, so that lines and DRAM pages are used whole.
// Forms that were slower: the block's keys split among four warps with a block
// barrier per block (4.1 TB/s on the case above), TMA boxes of a page each (4.0 TB/s
// with 16-token pages, 5.7 with 128-token pages), and load warps filling one ring
// for compute warps that take its blocks in turn and join their results at the end
// of every item (5.8 TB/s, but 1.3 with 128 requests of up to 1000 keys of codes).
//
// Products run on mma.sync m16n8k16, whose 16 rows the heads of a group fill;
// tcgen05's 128 would be nearly empty, and the tensor pipe is idle most of the
// time either way.
#include "paged_mma.cuh"
#include "paged_work.cuh"

namespace moe {

template <int kD, bool kE4m3>
struct DecCfg {
    static constexpr int kWarps = kDecodeWarps, kThreads = 32 * kWarps;
    static constexpr int kRowBytes = kD * (kE4m3 ? 1 : 2), kChunks = kRowBytes / 16;
    // 4 or 6 KB of K and as many of V: 16, 48 or 96 keys.  Against blocks of 32 and 64
    // in three slots, those of shorter rows gain 1 to 3% (128 requests, E4M3: 183 to 178 us).
    static constexpr int kRows = 16, kBlk = kRowBytes == 256 ? 16 : 6144 / kRowBytes, kSlots = kRowBytes == 256 ? 3 : 2;
    static constexpr int kMat = kBlk * kRowBytes, kStage = 2 * kMat;
    static constexpr int kSmem = kWarps * kSlots * kStage;
};

template <int kD, bool kE4m3>
__global__ void __launch_bounds__(DecCfg<kD, kE4m3>::kThreads, 1) paged_decode_kernel(const AttnParams p)
{
    using C = DecCfg<kD, kE4m3>;
    constexpr int kBlk = C::kBlk, kRows = C::kRows, kChunks = C::kChunks, kSlots = C::kSlots;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t ring = smem_u32(smem) + warp * (kSlots * C::kStage);

    Split<C::kThreads, kRows, kBlk, C::kWarps> split;
    // the warp's range, its head of a team's, and its place among the partial results:
    // one head's ranges lie side by side
    const int range = split.range(p, warp), in_team = warp & ((1 << p.team_log) - 1), unit = in_team * split.ranges(p) + range;
    Cursor<kRows, kBlk> cur;
    const long long n_blocks = split.init(p, cur, reinterpret_cast<long long *>(smem));
    grid_dep_launch();
    if (n_blocks == 0) {
        if (lane == 0) p.desc[unit].parts = 0;
        return;
    }

    auto head_of = [&](const Cursor<kRows, kBlk> &at) { return (at.kvh << p.team_log) + in_team; };

    // ------------------------------------------------------------------ loads
    // Lane r has row r of a block (and rows r + 32, r + 64); a copy takes 32 / kChunks rows.
    constexpr int kLook = (kBlk + 31) / 32, kAtOnce = 32 / kChunks;
    constexpr int esz = kE4m3 ? 1 : 2;
    Cursor<kRows, kBlk> ld = cur;
    long long ld_left = n_blocks;                            // blocks not yet looked up
    long long off[kLook];                                    // the next block's rows in bytes, -1: none
    bool bad = false;
    auto look_up = [&]() {
#pragma unroll
        for (int j = 0; j < kLook; ++j) off[j] = -1;
        if (ld_left == 0) return;
#pragma unroll
        for (int j = 0; j < kLook; ++j) {
            const int row = 32 * j + lane, key = ld.blk * kBlk + row;
            if (row >= kBlk || key >= ld.r.kv) continue;
            const int col = p.by_page.div(key);
            const int id = __ldg(p.table + static_cast<long long>(ld.b) * p.max_pages + col);
            if (id < 0 || id >= p.num_pages) bad = true;
            else off[j] = (id * p.page_stride + (static_cast<long long>(key - col * p.page_size) * p.n_kv + head_of(ld)) * kD) * esz;
        }
        if (--ld_left > 0 && ++ld.blk == ld.nblk) ld.next_item(p);
    };
    const int sub = lane / kChunks, chunk = lane % kChunks;
    auto copy_block = [&](int slot) {
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
    };
    look_up();
#pragma unroll
    for (int i = 0; i < kSlots - 1; ++i) {
        if (i < n_blocks) copy_block(i);
        copies_commit();
        look_up();
    }

    // ------------------------------------------------------------- products
    const int cq = lane & 3, r_lo = lane >> 2;
    uint32_t qf[kD / 16][4];
    float o[kD / 8][4], m[2], l[2], mult[2];
    int lim[2];
    int slot = 0;
    long long begin = 0;                                     // the item's first block in the range
    bool continued = cur.blk > 0;
    // column of element e of the accumulator's tile i
    auto col = [&](int i, int e) { return kE4m3 ? 16 * (i >> 1) + 4 * cq + 2 * e + (i & 1) : 8 * i + 2 * cq + e; };
    auto out_row = [&](int grow) {
        return static_cast<__nv_bfloat16 *>(p.out) + (static_cast<long long>(cur.r.qs + p.by_group.div(grow)) * p.n_heads +
                                                      head_of(cur) * p.group + (grow - p.by_group.div(grow) * p.group)) * kD;
    };
    for (;;) {
        const int n = static_cast<int>(min(n_blocks - begin, static_cast<long long>(cur.nblk - cur.blk)));
        const bool last = cur.blk + n == cur.nblk, whole = last && !continued;
        const int rows = cur.rows(p), row0 = cur.row0(p);
        float *part = p.part + (2LL * unit + (continued ? 0 : 1)) * (kRows * (kD + 2));
#pragma unroll
        for (int i = 0; i < kD / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.0f;
        {
            // the item's query rows as A fragments.  For an E4M3 cache in fp16 (see
            // row_power), and a lane takes 4 adjacent elements of 16 where the plain
            // fragment has two pairs: the order in which ldmatrix delivers codes.
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = r_lo + 8 * h, grow = row0 + r;
                const bool real = r < rows;
                const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.q) +
                                           static_cast<long long>(cur.r.qs + p.by_group.div(grow)) * p.q_stride +
                                           static_cast<long long>(head_of(cur) * p.group + (grow - p.by_group.div(grow) * p.group)) * kD;
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
        for (int j = 0; j < n; ++j) {
            const int key0 = (cur.blk + j) * kBlk;
            // the block kSlots - 1 ahead goes where the last one was
            if (begin + j + kSlots - 1 < n_blocks) copy_block(slot == 0 ? kSlots - 1 : slot - 1);
            copies_commit();
            look_up();
            copies_wait<kSlots - 1>();
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
                const float from = kE4m3 ? base - kF16Up : base;
#pragma unroll
                for (int i = 0; i < kBlk / 8; ++i)
#pragma unroll
                    for (int e = 2 * h; e < 2 * h + 2; ++e) {
                        s[i][e] = exp2_fast(s[i][e] - from);
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
            __syncwarp();                                    // the slot is read
            if (++slot == kSlots) slot = 0;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            const int r = r_lo + 8 * h;
            if (r >= rows) continue;
            if (whole) {
                const float inv = row_inverse(l[h]), vs = kE4m3 ? p.v_scale : 1.0f;
                __nv_bfloat16 *dst = out_row(row0 + r);
#pragma unroll
                for (int i = 0; i < kD / 8; i += 2) {
                    const float a = o[i][2 * h] * inv * vs, b = o[i][2 * h + 1] * inv * vs, c = o[i + 1][2 * h] * inv * vs,
                                d = o[i + 1][2 * h + 1] * inv * vs;
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
        begin += n;
        if (begin == n_blocks) {
            if (lane == 0) {
                AttnDesc d;
                d.parts = 0;
                d.qs = cur.r.qs;
                d.kvh = head_of(cur);
                d.row0 = row0;
                d.rows = rows;
                if (!last && !continued) d.parts = split.parts(range, begin - n, cur.nblk);
                p.desc[unit] = d;
            }
            break;
        }
        cur.next_item(p);
        continued = false;
    }
    copies_wait<0>();
    if (bad && p.status) set_status(p.status, MOE_ERR_DEVICE_CHECK);
}

template <int kD, bool kE4m3>
static cudaError_t launch_decode(const AttnParams &p, int sms, cudaStream_t st)
{
    using C = DecCfg<kD, kE4m3>;
    static PerDeviceOnce once;
    once([] { cudaFuncSetAttribute(paged_decode_kernel<kD, kE4m3>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem); });
    return launch_kernel(paged_decode_kernel<kD, kE4m3>, dim3(sms), dim3(C::kThreads), C::kSmem, st, false, p);
}

cudaError_t launch_attn_decode(const AttnParams &p, int head_dim, bool e4m3, int sms, cudaStream_t st)
{
    if (head_dim == 64) return e4m3 ? launch_decode<64, true>(p, sms, st) : launch_decode<64, false>(p, sms, st);
    return e4m3 ? launch_decode<128, true>(p, sms, st) : launch_decode<128, false>(p, sms, st);
}

}  // namespace moe
