// paged_attention.cu - attention of a batch's new tokens over a paged cache
// (moe_paged_attention): the entry point with its choice of kernels, the kernel
// that joins partial results, and the kernel for the shapes the other two do not
// take.
//
// o_i = sum_j p_ij v_j / sum_j p_ij with p_ij = 2^(s_ij - m_i), s = q.k scale
// log2(e), in one pass over the keys with the running maximum m_i and sum: when
// a block of keys raises m_i, what was summed so far is scaled by 2^(old - new).
//
// Requests with at most 16 query rows a key/value head are bound by reading the
// cache and go to paged_decode.cu, those with more by the products and exponentials
// and go to paged_attention_tc.cu.  The kernel here takes head_dim 256 for both
// (kWM = 1 and 4): a decode warp's output alone would be 128 registers a thread, and two
// 128-row tiles with their scores more than tensor memory's 512 columns.  With many rows
// it also takes a scale whose log2 form is below 1e-37 (zero and negative ones with
// it), a group of more than 128 heads and a token stride of 2^39 elements or more.  It is
// mma.sync with 64-key blocks in a ring that all four warps fill by cp.async and
// read behind a block barrier; the warps lie down the rows, or with few rows along the
// keys of a block.  At head_dim 256 (32 and 8 heads): 32 requests of 8192 keys 455 us (4.7
// TB/s) in bf16, 360 us (3.0 TB/s) in E4M3, whose codes are converted in the chain; 4 prompts
// of 2048 tokens 1465 us (190 TFLOP/s) and 1890 us, the E4M3 form with 764 bytes spilled;
// 1024 tokens over 8192 keys 1160 us.  mma.sync's rate bounds the many rows.
#include <atomic>

#include "overlap.cuh"
#include "paged_mma.cuh"
#include "paged_work.cuh"

namespace moe {

// Geometry of one kernel: kWM warps down the query rows (16 each), 4 / kWM
// along the keys of a block.
template <int kD, bool kE4m3, int kWM>
struct AttnCfg {
    static constexpr int kThreads = 128, kBlk = 64;
    static constexpr int kWN = 4 / kWM, kRows = 16 * kWM, kKeys = kBlk / kWN;
    static constexpr int kRowBytes = kD * (kE4m3 ? 1 : 2), kChunks = kRowBytes / 16;
    static constexpr int kStage = 2 * kBlk * kRowBytes;
    static constexpr int kStages = kRowBytes <= 128 ? 4 : 3;
    static constexpr int kQ = kRows * kD * 2;
    static constexpr int kMerge = kWN > 1 ? kRows * kD * 4 : 0;
    static constexpr int kSmem = kStages * kStage + kQ + kMerge;
    // bf16 cache, few rows: p goes into its product as two bf16 (high and
    // low part), which costs tensor work that is idle here and leaves the
    // output's own rounding the only one of 8 bits.  With many rows that work
    // counts, and p is rounded once; for an E4M3 cache it is fp16 (11 bits).
    static constexpr bool kSplitP = !kE4m3 && kWM == 1;
    static constexpr bool kQReg = kD <= 128;
};

template <int kD, bool kE4m3, int kWM>
__global__ void __launch_bounds__(128) paged_attention_kernel(const AttnParams p)
{
    using C = AttnCfg<kD, kE4m3, kWM>;
    constexpr int kBlk = C::kBlk, kRows = C::kRows, kChunks = C::kChunks, kRowBytes = C::kRowBytes, kStages = C::kStages;
    constexpr int kKeys = C::kKeys, kWN = C::kWN;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_off[2][kBlk];         // element offset of each key's row, -1: none
    __shared__ float s_inv[kRows];               // 1 / the row's factor in q (E4M3 cache)
    __shared__ float s_m[4][16], s_l[4][16];
    const uint32_t ring = smem_u32(smem);
    uint8_t *s_q = smem + kStages * C::kStage;
    float *s_merge = reinterpret_cast<float *>(s_q + C::kQ);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wm = warp / kWN, wn = warp % kWN;

    Split<128, kRows, kBlk> split;
    Cursor<kRows, kBlk> cur;                     // the compute side
    const long long n_blocks = split.init(p, cur, reinterpret_cast<long long *>(smem));
    if (n_blocks == 0) {
        if (tid == 0) p.desc[blockIdx.x].parts = 0;
        grid_dep_launch();
        if (p.wait_at_end) grid_dep_wait();
        return;
    }
    grid_dep_launch();

    // ---- load side: warps 0 and 1, a lane per key of a block ----
    Cursor<kRows, kBlk> ld = cur;
    long long ld_left = n_blocks;                // blocks whose page id is still to be read
    int id_key = 0, id_page = 0, id_kvh = 0;     // the last id read: its key, page and head
    bool id_in = false;
    bool bad = false;
    auto read_id = [&]() {                       // page id of the next block's key
        if (ld_left > 0) {
            id_key = ld.blk * kBlk + tid;
            id_in = id_key < ld.r.kv;
            id_kvh = ld.kvh;
            id_page = id_in ? __ldg(p.table + static_cast<long long>(ld.b) * p.max_pages + p.by_page.div(id_key)) : 0;
            if (--ld_left > 0 && ++ld.blk == ld.nblk) ld.next_item(p);
        } else {
            id_in = false;
        }
    };
    auto put_off = [&](int buf) {                // the id just read becomes an offset
        long long off = -1;
        if (id_in) {
            if (id_page >= 0 && id_page < p.num_pages)
                off = id_page * p.page_stride + (static_cast<long long>(id_key - p.by_page.div(id_key) * p.page_size) * p.n_kv + id_kvh) * kD;
            else
                bad = true;
        }
        s_off[buf][tid] = off;
    };
    constexpr int esz = kE4m3 ? 1 : 2;
    auto issue = [&](int stage, int buf) {       // all threads: copy one block's rows
        const uint32_t dst = ring + stage * C::kStage;
        constexpr int kPer = kBlk * kChunks / 128;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int x = tid + i * 128, r = x / kChunks, c = x % kChunks;
            const long long off = s_off[buf][r];
            const long long at = (off < 0 ? 0 : off * esz) + c * 16;
            const uint32_t d = dst + r * kRowBytes + chunk_of<kChunks>(r, c) * 16;
            copy16(d, static_cast<const uint8_t *>(p.k_cache) + at, off >= 0);
            copy16(d + kBlk * kRowBytes, static_cast<const uint8_t *>(p.v_cache) + at, off >= 0);
        }
    };

    if (warp < 2) {
        read_id();
        put_off(0);
        read_id();
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {      // block i's offsets are in buffer i & 1
        if (i < n_blocks) issue(i, i & 1);
        copies_commit();
        if (warp < 2) {
            put_off((i + 1) & 1);
            read_id();
        }
        __syncthreads();
    }

    // ---- compute side ----
    float o[kD / 8][4];
    float m[2], l[2];
    uint32_t qf[C::kQReg ? kD / 16 : 1][4];
    int lim[2];
    float mult[2];
    const int r_lo = 16 * wm + (lane >> 2), cq = lane & 3;
    bool fresh_item = true;
    long long item_from = 0;                     // where in this CTA's range the item starts
    bool continued = cur.blk > 0;
    const uint32_t sq = smem_u32(s_q);
    auto load_qf = [&](uint32_t (&f)[4], int ks) {
        const int r = 16 * wm + (lane & 15), c = 2 * ks + (lane >> 4);
        ldsm4(f, sq + r * (kD * 2) + (c ^ (r & 7)) * 16);
    };

    for (long long it = 0; it < n_blocks; ++it) {
        copies_wait<kStages - 2>();
        if (fresh_item) {
            // the item's query rows into shared memory; for an E4M3 cache in fp16
            // (see row_power), the columns permuted within 16 to the order in
            // which ldmatrix delivers a row of bytes
            constexpr int kTpr = 128 / kRows, kCpt = kD / 8 / kTpr;   // threads per row, chunks per thread
            const int r = tid / kTpr, part = tid % kTpr;
            const int rows = cur.rows(p);
            const int grow = cur.row0(p) + r;
            const int tok = p.by_group.div(grow);
            const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(p.q) +
                                       static_cast<long long>(cur.r.qs + tok) * p.q_stride +
                                       static_cast<long long>(cur.kvh * p.group + (grow - p.by_group.div(grow) * p.group)) * kD;
            uint4 w[kCpt];
#pragma unroll
            for (int i = 0; i < kCpt; ++i)
                w[i] = r < rows ? __ldg(reinterpret_cast<const uint4 *>(src) + part + i * kTpr) : make_uint4(0, 0, 0, 0);
            if constexpr (kE4m3) {
                float amax = 0.0f;
#pragma unroll
                for (int i = 0; i < kCpt; ++i) {
                    const uint32_t ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(ww[j] << 16)), fabsf(__uint_as_float(ww[j] & 0xFFFF0000u))));
                }
#pragma unroll
                for (int o2 = kTpr / 2; o2 > 0; o2 >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o2));
                const int up = row_power(amax);
                const float f = power_of_two(up);
                if (part == 0) s_inv[r] = power_of_two(-up);
#pragma unroll
                for (int i = 0; i < kCpt; ++i) {
                    const uint32_t ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                    const int c8 = part + i * kTpr;       // elements 8 c8 .. 8 c8 + 7
                    // d = 16 ks + 4 c + {0, 1} -> column 2 c + {0, 1}, + {2, 3} -> 8 + 2 c + {0, 1}
                    const int ks = c8 >> 1, c0 = (c8 & 1) * 2;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t h = f16x2_of(__uint_as_float(ww[j] << 16) * f, __uint_as_float(ww[j] & 0xFFFF0000u) * f);
                        const int col = 2 * (c0 + (j >> 1)), chunk = 2 * ks + (j & 1);
                        *reinterpret_cast<uint32_t *>(s_q + r * (kD * 2) + (chunk ^ (r & 7)) * 16 + col * 2) = h;
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < kCpt; ++i) {
                    const int c = part + i * kTpr;
                    *reinterpret_cast<uint4 *>(s_q + r * (kD * 2) + (c ^ (r & 7)) * 16) = w[i];
                }
            }
        }
        __syncthreads();
        // block it has landed, block it - 1 has been read by every warp
        {
            const long long nx = it + kStages - 1;
            if (nx < n_blocks) issue(static_cast<int>(nx % kStages), static_cast<int>(nx & 1));
            copies_commit();
            if (warp < 2) {
                put_off(static_cast<int>((nx + 1) & 1));
                read_id();
            }
        }
        if (fresh_item) {
#pragma unroll
            for (int i = 0; i < kD / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
            m[0] = m[1] = -INFINITY;
            l[0] = l[1] = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = r_lo + 8 * h;
                lim[h] = r < cur.rows(p) ? row_limit(p, cur.r, cur.row0(p) + r) : 0;
                mult[h] = p.scale_log2 * (kE4m3 ? s_inv[r] : 1.0f);
            }
            if constexpr (C::kQReg) {
#pragma unroll
                for (int ks = 0; ks < kD / 16; ++ks) load_qf(qf[ks], ks);
            }
            fresh_item = false;
        }
        const uint32_t kst = ring + static_cast<int>(it % kStages) * C::kStage, vst = kst + kBlk * kRowBytes;

        // scores of the warp's rows and keys
        float s[kKeys / 8][4];
#pragma unroll
        for (int i = 0; i < kKeys / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
        if constexpr (!kE4m3) {
#pragma unroll
            for (int ks = 0; ks < kD / 16; ++ks) {
                if constexpr (!C::kQReg) load_qf(qf[0], ks);
                const uint32_t (&a)[4] = qf[C::kQReg ? ks : 0];
#pragma unroll
                for (int np = 0; np < kKeys / 16; ++np) {
                    const int r = wn * kKeys + np * 16 + (lane & 7) + ((lane >> 4) << 3), c = 2 * ks + ((lane >> 3) & 1);
                    uint32_t b[4];
                    ldsm4(b, kst + r * kRowBytes + chunk_of<kChunks>(r, c) * 16);
                    mma16816<false>(s[2 * np], a, b[0], b[1]);
                    mma16816<false>(s[2 * np + 1], a, b[2], b[3]);
                }
            }
        } else {
#pragma unroll
            for (int k2 = 0; k2 < kD / 32; ++k2) {
#pragma unroll
                for (int np = 0; np < kKeys / 16; ++np) {
                    // matrices: keys 0-7 and 8-15 at chunk 2 k2, then at 2 k2 + 1
                    const int r = wn * kKeys + np * 16 + (lane & 15), c = 2 * k2 + (lane >> 4);
                    uint32_t b[4];
                    ldsm4(b, kst + r * kRowBytes + chunk_of<kChunks>(r, c) * 16);
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        if constexpr (!C::kQReg) load_qf(qf[0], 2 * k2 + kk);
                        const uint32_t (&a)[4] = qf[C::kQReg ? 2 * k2 + kk : 0];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t x = b[2 * kk + h];
                            uint32_t b0, b1;
                            f16x4_of_e4m3(x, b0, b1);
                            mma16816<true>(s[2 * np + h], a, b0, b1);
                        }
                    }
                }
            }
        }
        // mask, running maximum, p
        const int key0 = cur.blk * kBlk + wn * kKeys + 2 * cq;
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < kKeys / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float t = key0 + 8 * i + (e & 1) < lim[e >> 1] ? s[i][e] * mult[e >> 1] : -INFINITY;
                s[i][e] = t;
                top[e >> 1] = fmaxf(top[e >> 1], t);
            }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
            const float mn = fmaxf(m[h], top[h]);
            const float base = mn == -INFINITY ? 0.0f : mn;      // a row that has seen nothing yet
            const float alpha = exp2_fast(m[h] - base);
            m[h] = mn;
            l[h] *= alpha;
            const float from = kE4m3 ? base - kF16Up : base;
#pragma unroll
            for (int i = 0; i < kKeys / 8; ++i)
#pragma unroll
                for (int e = 2 * h; e < 2 * h + 2; ++e) {
                    s[i][e] = exp2_fast(s[i][e] - from);
                    l[h] += s[i][e];
                }
            if (alpha != 1.0f) {
#pragma unroll
                for (int i = 0; i < kD / 8; ++i) {
                    o[i][2 * h] *= alpha;
                    o[i][2 * h + 1] *= alpha;
                }
            }
        }
        // o += p v
#pragma unroll
        for (int kt = 0; kt < kKeys / 16; ++kt) {
            uint32_t ph[4], pl[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float a = s[2 * kt + (j >> 1)][2 * (j & 1)], b = s[2 * kt + (j >> 1)][2 * (j & 1) + 1];
                if constexpr (kE4m3) {
                    ph[j] = f16x2_of(a, b);
                } else {
                    ph[j] = bf16x2_of(a, b);
                    if constexpr (C::kSplitP)
                        pl[j] = bf16x2_of(a - __uint_as_float(ph[j] << 16), b - __uint_as_float(ph[j] & 0xFFFF0000u));
                }
            }
            const int r = wn * kKeys + kt * 16 + (lane & 15);
#pragma unroll
            for (int dp = 0; dp < kChunks / 2; ++dp) {
                const int c = 2 * dp + (lane >> 4);
                uint32_t b[4];
                ldsm4_t(b, vst + r * kRowBytes + chunk_of<kChunks>(r, c) * 16);
                if constexpr (!kE4m3) {
                    mma16816<false>(o[2 * dp], ph, b[0], b[1]);
                    mma16816<false>(o[2 * dp + 1], ph, b[2], b[3]);
                    if constexpr (C::kSplitP) {
                        mma16816<false>(o[2 * dp], pl, b[0], b[1]);
                        mma16816<false>(o[2 * dp + 1], pl, b[2], b[3]);
                    }
                } else {
                    // a 16-bit unit holds elements 2n and 2n + 1 of one key: tile
                    // 2 ch takes the even ones of chunk ch, 2 ch + 1 the odd ones
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t x = __byte_perm(b[2 * h], 0, 0x3120), y = __byte_perm(b[2 * h + 1], 0, 0x3120);
                        const int ch = 2 * dp + h;
                        uint32_t x0, x1, y0, y1;
                        f16x4_of_e4m3(x, x0, x1);
                        f16x4_of_e4m3(y, y0, y1);
                        mma16816<true>(o[2 * ch], ph, x0, y0);
                        mma16816<true>(o[2 * ch + 1], ph, x1, y1);
                    }
                }
            }
        }

        // ---- the item's end, in this CTA ----
        const bool last = cur.blk + 1 == cur.nblk;
        if (last || it + 1 == n_blocks) {
            const bool whole = last && !continued;
            const int rows = cur.rows(p);
            const long long slot = 2LL * blockIdx.x + (continued ? 0 : 1);
            float *part = p.part + slot * (kRows * (kD + 2));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            }
            // column of element e of the accumulator's tile i
            auto col = [&](int i, int e) { return kE4m3 ? 16 * (i >> 1) + 4 * cq + 2 * e + (i & 1) : 8 * i + 2 * cq + e; };
            if constexpr (kWN == 1) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = r_lo + 8 * h;
                    if (r < rows) {
                        const int grow = cur.row0(p) + r;
                        if (whole) {
                            const float inv = row_inverse(l[h]), vs = p.v_scale;
                            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) +
                                                 (static_cast<long long>(cur.r.qs + p.by_group.div(grow)) * p.n_heads +
                                                  cur.kvh * p.group + (grow - p.by_group.div(grow) * p.group)) * kD;
#pragma unroll
                            for (int i = 0; i < kD / 8; ++i) {
                                if constexpr (kE4m3) {
                                    dst[col(i, 0)] = __float2bfloat16_rn(o[i][2 * h] * inv * vs);
                                    dst[col(i, 1)] = __float2bfloat16_rn(o[i][2 * h + 1] * inv * vs);
                                } else {
                                    *reinterpret_cast<uint32_t *>(dst + col(i, 0)) = bf16x2_of(o[i][2 * h] * inv * vs, o[i][2 * h + 1] * inv * vs);
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < kD / 8; ++i) {
                                part[many_at(kRows, r, col(i, 0))] = o[i][2 * h];
                                part[many_at(kRows, r, col(i, 1))] = o[i][2 * h + 1];
                            }
                            if (cq == 0) {
                                part[kRows * kD + r] = m[h];
                                part[kRows * kD + kRows + r] = l[h];
                            }
                        }
                    }
                }
            } else {
                // the warps hold different keys of the same rows: to one maximum,
                // then summed in warp order
                if (cq == 0) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        s_m[warp][r_lo + 8 * h] = m[h];
                        s_l[warp][r_lo + 8 * h] = l[h];
                    }
                }
                __syncthreads();
                float f[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = r_lo + 8 * h;
                    const float mx = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
                    f[h] = exp2_fast(m[h] - (mx == -INFINITY ? 0.0f : mx));
                }
#pragma unroll
                for (int w = 0; w < kWN; ++w) {
                    if (warp == w) {
#pragma unroll
                        for (int i = 0; i < kD / 8; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float *d = s_merge + (r_lo + 8 * (e >> 1)) * kD + col(i, e & 1);
                                const float v = o[i][e] * f[e >> 1];
                                *d = w == 0 ? v : *d + v;
                            }
                    }
                    __syncthreads();
                }
                for (int x = tid; x < rows * (kD / 8); x += 128) {
                    const int r = x / (kD / 8), c = x % (kD / 8) * 8;
                    const float mx = fmaxf(fmaxf(s_m[0][r], s_m[1][r]), fmaxf(s_m[2][r], s_m[3][r]));
                    const float base = mx == -INFINITY ? 0.0f : mx;
                    float lt = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWN; ++w) lt += s_l[w][r] * exp2_fast(s_m[w][r] - base);
                    const float *v = s_merge + r * kD + c;
                    if (whole) {
                        const float inv = row_inverse(lt), vs = p.v_scale;
                        const int grow = cur.row0(p) + r;
                        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) +
                                             (static_cast<long long>(cur.r.qs + p.by_group.div(grow)) * p.n_heads +
                                              cur.kvh * p.group + (grow - p.by_group.div(grow) * p.group)) * kD + c;
                        *reinterpret_cast<uint4 *>(dst) =
                            make_uint4(bf16x2_of(v[0] * inv * vs, v[1] * inv * vs), bf16x2_of(v[2] * inv * vs, v[3] * inv * vs),
                                       bf16x2_of(v[4] * inv * vs, v[5] * inv * vs), bf16x2_of(v[6] * inv * vs, v[7] * inv * vs));
                    } else {
                        float4 *d = reinterpret_cast<float4 *>(part + r * kD + c);
                        d[0] = make_float4(v[0], v[1], v[2], v[3]);
                        d[1] = make_float4(v[4], v[5], v[6], v[7]);
                        if (c == 0) {
                            part[kRows * kD + r] = mx;
                            part[kRows * kD + kRows + r] = lt;
                        }
                    }
                }
            }
            if (it + 1 == n_blocks && tid == 0) {
                AttnDesc d;
                d.parts = 0;
                d.qs = cur.r.qs;
                d.kvh = cur.kvh;
                d.row0 = cur.row0(p);
                d.rows = rows;
                if (!last && !continued) d.parts = split.parts(blockIdx.x, item_from, cur.nblk);
                p.desc[blockIdx.x] = d;
            }
            if (it + 1 < n_blocks) {
                cur.next_item(p);
                fresh_item = true;
                continued = false;
                item_from = it + 1;
                __syncthreads();                 // s_q, s_m and the merge area are read
            }
        } else {
            ++cur.blk;
        }
    }
    copies_wait<0>();
    if (bad && p.status) set_status(p.status, MOE_ERR_DEVICE_CHECK);
    if (p.wait_at_end) grid_dep_wait();
}

// The partial results of one kernel.
struct AttnParts {
    const float *part;
    const AttnDesc *desc;
    int units, rows;          // ranges, and query rows of an item
};

// One row of an item in several ranges: its sums over parts first .. behind - 1,
// relative to the largest maximum of all its parts, kD / 32 elements a lane; l is
// the total over those parts, in every lane.
template <int kD>
__device__ __forceinline__ void join_row(const AttnParts &from, int c, int parts, int r, int first, int behind, float (&acc)[kD / 32], float &l)
{
    constexpr int kE = kD / 32;
    const int lane = threadIdx.x & 31;
    const long long stride = static_cast<long long>(from.rows) * (kD + 2);
    // part k of the item
    auto part = [&](int k) { return from.part + (k == 0 ? 2LL * c + 1 : 2LL * (c + k)) * stride; };
    const int at_m = from.rows * kD + r, at_l = at_m + from.rows;
    float base = -INFINITY;
#pragma unroll 4
    for (int k = lane; k < parts; k += 32) base = fmaxf(base, part(k)[at_m]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) base = fmaxf(base, __shfl_xor_sync(0xffffffffu, base, o));
    if (base == -INFINITY) base = 0.0f;
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] = 0.0f;
    for (int k0 = first; k0 < behind; k0 += 32) {
        float f = 0.0f;
        if (k0 + lane < behind) {
            const float *q = part(k0 + lane);
            f = exp2_fast(q[at_m] - base);
            l += f * q[at_l];
        }
        const int n = min(32, behind - k0);
#pragma unroll 8
        for (int k = 0; k < n; ++k) {
            const float *q = part(k0 + k) + r * kD + lane * kE;
            const float fk = __shfl_sync(0xffffffffu, f, k);
            float v[kE];
            if constexpr (kE == 2) {
                *reinterpret_cast<float2 *>(v) = *reinterpret_cast<const float2 *>(q);
            } else {
#pragma unroll
                for (int e = 0; e < kE; e += 4) *reinterpret_cast<float4 *>(v + e) = *reinterpret_cast<const float4 *>(q + e);
            }
#pragma unroll
            for (int e = 0; e < kE; ++e) acc[e] += fk * v[e];
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
}

template <int kD>
__device__ __forceinline__ void put_row(const AttnParams &p, const AttnDesc &d, int r, const float (&acc)[kD / 32], float l)
{
    constexpr int kE = kD / 32;
    const float inv = row_inverse(l), vs = p.v_scale;
    const int grow = d.row0 + r;
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) +
                         (static_cast<long long>(d.qs + p.by_group.div(grow)) * p.n_heads + d.kvh * p.group + (grow - p.by_group.div(grow) * p.group)) * kD +
                         (threadIdx.x & 31) * kE;
#pragma unroll
    for (int e = 0; e < kE; e += 2) *reinterpret_cast<uint32_t *>(dst + e) = bf16x2_of(acc[e] * inv * vs, acc[e + 1] * inv * vs);
}

// The same for items of many rows (see many_at): two adjacent rows a lane, kD / 4
// lanes across them where that is less than a warp.
template <int kD>
__device__ __forceinline__ void join_rows(const AttnParams &p, const AttnParts &from, int c, int row0, int behind)
{
    constexpr int kAcross = kD / 4 < 32 ? kD / 4 : 32, kC = kD / 4 / kAcross, kStep = 2 * (32 / kAcross);
    const AttnDesc d = from.desc[c];
    if (d.parts < 2) return;
    const int lane = threadIdx.x & 31, x = lane % kAcross;
    const long long stride = static_cast<long long>(from.rows) * (kD + 2);
    auto part = [&](int k) { return from.part + (k == 0 ? 2LL * c + 1 : 2LL * (c + k)) * stride; };
    for (int r0 = row0 + (threadIdx.x >> 5) * kStep; r0 < min(d.rows, behind); r0 += 8 * kStep) {
        const int r = r0 + 2 * (lane / kAcross), at_m = from.rows * kD + r, at_l = at_m + from.rows;
        if (r >= d.rows) continue;               // no lane waits for another here
        float base[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
        float4 acc[2][kC];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < kC; ++i) acc[j][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        // from.rows and r are even and r is a row of the item's: the second has a place in
        // the part even where it is none of the item's
#pragma unroll 4
        for (int k = 0; k < d.parts; ++k) {
            base[0] = fmaxf(base[0], part(k)[at_m]);
            base[1] = fmaxf(base[1], part(k)[at_m + 1]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (base[j] == -INFINITY) base[j] = 0.0f;
#pragma unroll 4
        for (int k = 0; k < d.parts; ++k) {
            const float *q = part(k);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float f = exp2_fast(q[at_m + j] - base[j]);
                l[j] += f * q[at_l + j];
#pragma unroll
                for (int i = 0; i < kC; ++i) {
                    const float4 v = *reinterpret_cast<const float4 *>(q + many_at(from.rows, r + j, 4 * (x + i * kAcross)));
                    acc[j][i] = make_float4(acc[j][i].x + f * v.x, acc[j][i].y + f * v.y, acc[j][i].z + f * v.z, acc[j][i].w + f * v.w);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (r + j >= d.rows) continue;
            const float inv = row_inverse(l[j]), vs = p.v_scale;
            const int grow = d.row0 + r + j, tok = p.by_group.div(grow);
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) +
                                 (static_cast<long long>(d.qs + tok) * p.n_heads + d.kvh * p.group + (grow - tok * p.group)) * kD;
#pragma unroll
            for (int i = 0; i < kC; ++i)
                *reinterpret_cast<uint2 *>(dst + 4 * (x + i * kAcross)) =
                    make_uint2(bf16x2_of(acc[j][i].x * inv * vs, acc[j][i].y * inv * vs), bf16x2_of(acc[j][i].z * inv * vs, acc[j][i].w * inv * vs));
        }
    }
}

// Joins the parts of the items that lie in several ranges, of one or two kernels.
// First kernel (items of up to 16 rows, up to 8 ranges per SM): a block has 8
// ranges and every fourth row of the items that they start; a warp joins its
// item's row alone, and where an item has many parts (few requests, long
// sequences) the 8 warps share them.  Second kernel (items of many rows): a block
// has one range and 32 rows of its item.
constexpr int kManyParts = 16;

template <int kD>
__global__ void __launch_bounds__(256) attention_combine_kernel(const AttnParams p, const AttnParts few, const AttnParts many)
{
    constexpr int kE = kD / 32;
    __shared__ float s_acc[8][kD], s_l[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int few_blocks = (few.units + 7) / 8 * 4;
    float acc[kE], l;
    grid_dep_wait();
    if (static_cast<int>(blockIdx.x) >= few_blocks) {
        const int per = (many.rows + 31) / 32, x = blockIdx.x - few_blocks, row0 = x % per * 32;
        join_rows<kD>(p, many, x / per, row0, row0 + 32);
        return;
    }
    const int c0 = blockIdx.x / 4 * 8, y = blockIdx.x % 4;
    const int parts = lane < 8 && c0 + lane < few.units ? few.desc[c0 + lane].parts : 0;      // the same in every warp
    const int own = __shfl_sync(0xffffffffu, parts, warp);
    if (own >= 2 && own <= kManyParts) {
        const AttnDesc d = few.desc[c0 + warp];
        for (int r = y; r < d.rows; r += 4) {
            join_row<kD>(few, c0 + warp, own, r, 0, own, acc, l);
            put_row<kD>(p, d, r, acc, l);
        }
    }
    for (unsigned left = __ballot_sync(0xffffffffu, parts > kManyParts); left; left &= left - 1) {
        const int i = __ffs(left) - 1, n = __shfl_sync(0xffffffffu, parts, i);
        const AttnDesc d = few.desc[c0 + i];
        for (int r = y; r < d.rows; r += 4) {
            join_row<kD>(few, c0 + i, n, r, n * warp / 8, n * (warp + 1) / 8, acc, l);
#pragma unroll
            for (int e = 0; e < kE; ++e) s_acc[warp][lane * kE + e] = acc[e];
            if (lane == 0) s_l[warp] = l;
            __syncthreads();
            if (warp == 0) {
                for (int w = 1; w < 8; ++w) {
                    l += s_l[w];
#pragma unroll
                    for (int e = 0; e < kE; ++e) acc[e] += s_acc[w][lane * kE + e];
                }
                put_row<kD>(p, d, r, acc, l);
            }
            __syncthreads();
        }
    }
}

// SMs of the current device (0 on an error), up to what the workspace holds.
static int sm_count()
{
    static std::atomic<int> cache[64];
    int dev = 0;
    cudaGetDevice(&dev);
    int n = dev >= 0 && dev < 64 ? cache[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        if (n > kAttnMaxSms) n = kAttnMaxSms;
        if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// CTAs of a kernel that are resident on the GPU at once, found once per kernel
// and device together with the shared-memory limit.
template <int kD, bool kE4m3, int kWM>
static int resident_ctas()
{
    using C = AttnCfg<kD, kE4m3, kWM>;
    static std::atomic<int> cache[64];
    int dev = 0;
    cudaGetDevice(&dev);
    int n = dev >= 0 && dev < 64 ? cache[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        auto kern = paged_attention_kernel<kD, kE4m3, kWM>;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess) return 0;
        int sms = 0, per = 0;
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, 128, C::kSmem) != cudaSuccess || per < 1) return 0;
        n = sms * per;
        if (n > kAttnMaxUnits) n = kAttnMaxUnits;
        if (dev >= 0 && dev < 64) cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

template <int kD, bool kE4m3, int kWM>
static int launch_mma(const AttnParams &p, AttnParts &parts, bool chained, cudaStream_t st)
{
    using C = AttnCfg<kD, kE4m3, kWM>;
    parts = AttnParts{p.part, p.desc, resident_ctas<kD, kE4m3, kWM>(), C::kRows};
    if (parts.units == 0) return MOE_ERR_CUDA;
    return launch_kernel(paged_attention_kernel<kD, kE4m3, kWM>, dim3(parts.units), dim3(128), C::kSmem, st, chained, p) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

// Requests of up to 16 rows go to the kernel whose tile is 16 rows, the others to
// the tensor-memory kernel, or where that does not take the shape, to 64-row
// tiles.  A batch that by its hint has only the former is one kernel's.  The
// second kernel starts while the first one ends.
constexpr int kFewRows = 16;

static bool only_few(const moe_attn_shape_t &s)
{
    return s.max_q > 0 && static_cast<int64_t>(s.max_q) * (s.n_heads / s.n_kv_heads) <= kFewRows;
}

// Workspace: descriptors and partial results of either kernel.
struct AttnWs {
    size_t few_desc, many_desc, few_part, many_part, total;
};

static AttnWs attn_ws(const moe_attn_shape_t &s)
{
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    auto parts = [&](int units, int rows) { return up(static_cast<size_t>(units) * 2 * rows * (s.head_dim + 2) * 4); };
    AttnWs w;
    w.few_desc = 0;
    w.many_desc = up(sizeof(AttnDesc) * kAttnMaxUnits);
    w.few_part = 2 * w.many_desc;
    w.many_part = w.few_part + parts(kAttnMaxUnits, kFewRows);
    w.total = w.many_part;
    if (!only_few(s)) w.total += attn_tc_takes(s) ? parts(kAttnMaxSms, attn_tc_rows(s)) : parts(kAttnMaxUnits, 64);
    return w;
}

template <int kD>
static int launch_attention(const moe_attn_shape_t &s, AttnParams p, char *ws, cudaStream_t st, int &launches)
{
    const AttnWs w = attn_ws(s);
    const bool e4m3 = s.cache_dtype == MOE_E4M3;
    AttnParts few, many = {nullptr, nullptr, 0, 0};
    const int sms = sm_count();
    if (sms == 0) return MOE_ERR_CUDA;
    p.desc = reinterpret_cast<AttnDesc *>(ws + w.few_desc);
    p.part = reinterpret_cast<float *>(ws + w.few_part);
    p.min_rows = 1;
    p.max_rows = only_few(s) ? 0x7fffffff : kFewRows;
    p.wait_at_end = 0;
    auto items_of = [&](int rows) {
        p.tile_rows = rows;
        p.tile_tokens = rows % p.group ? 0 : rows / p.group;
        p.by_tile.set(rows);
    };
    items_of(kFewRows);
    p.team_log = 0;
    int r;
    if constexpr (kD <= 128) {
        // Heads side by side until a team reads 256 bytes of a key.  Rows of 64 bytes
        // alone had every 128-byte line fetched twice (128 requests, E4M3, D = 64: 165 to
        // 110 us; D = 128: 208 to 183; bf16, D = 64: 104 to 97).  Teams of 512 and
        // 1024 bytes: 115, 181, 96 and 115, 186, 99, and slower with few keys.
        const int row_bytes = kD * (e4m3 ? 1 : 2);
        while (s.n_kv_heads % (2 << p.team_log) == 0 && row_bytes << p.team_log < 256) ++p.team_log;
        p.n_teams = s.n_kv_heads >> p.team_log;
        few = AttnParts{p.part, p.desc, sms * kDecodeWarps, kFewRows};
        if (launch_attn_decode(p, kD, e4m3, sms, st) != cudaSuccess) return MOE_ERR_CUDA;
    } else {
        p.n_teams = s.n_kv_heads;
        r = e4m3 ? launch_mma<kD, true, 1>(p, few, false, st) : launch_mma<kD, false, 1>(p, few, false, st);
        if (r != MOE_OK) return r;
    }
    launches += 1;
    if (!only_few(s)) {
        p.desc = reinterpret_cast<AttnDesc *>(ws + w.many_desc);
        p.part = reinterpret_cast<float *>(ws + w.many_part);
        p.min_rows = kFewRows + 1;
        p.max_rows = 0x7fffffff;
        p.wait_at_end = 1;
        p.team_log = 0;
        p.n_teams = s.n_kv_heads;
        if (attn_tc_takes(s)) {
            items_of(attn_tc_rows(s));
            many = AttnParts{p.part, p.desc, sms, p.tile_rows};
            if (launch_attn_tc(p, kD, e4m3, sms, true, st) != cudaSuccess) return MOE_ERR_CUDA;
        } else {
            items_of(64);
            r = e4m3 ? launch_mma<kD, true, 4>(p, many, true, st) : launch_mma<kD, false, 4>(p, many, true, st);
            if (r != MOE_OK) return r;
        }
        launches += 1;
    }
    if (launch_kernel(attention_combine_kernel<kD>, dim3((few.units + 7) / 8 * 4 + many.units * ((many.rows + 31) / 32)), dim3(256), 0, st, true, p, few, many) !=
        cudaSuccess)
        return MOE_ERR_CUDA;
    launches += 1;
    return MOE_OK;
}

static bool attn_misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

static int check_attn(const moe_attn_shape_t *shape)
{
    if (!shape) return MOE_ERR_INVALID_ARG;
    const moe_attn_shape_t &s = *shape;
    if (s.B < 1 || s.B > kAttnMaxB || s.num_tokens < 0 || s.n_heads < 1 || s.n_kv_heads < 1 || s.n_heads > 65536 ||
        s.n_heads % s.n_kv_heads || s.page_size < 1 || s.num_pages < 1 || s.max_pages < 1 ||
        (s.causal != 0 && s.causal != 1) || s.max_q < 0 || (s.cache_dtype != MOE_BF16 && s.cache_dtype != MOE_E4M3))
        return MOE_ERR_INVALID_ARG;
    if (s.head_dim != 64 && s.head_dim != 128 && s.head_dim != 256) return MOE_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(s.num_pages) * s.page_size > 0x7fffffffll || static_cast<int64_t>(s.num_tokens) * s.n_heads > 0x40000000ll ||
        static_cast<int64_t>(s.max_pages) * s.page_size > 0x40000000ll)
        return MOE_ERR_INVALID_ARG;
    if (s.q_stride && (s.q_stride < static_cast<int64_t>(s.n_heads) * s.head_dim || s.q_stride % 8)) return MOE_ERR_INVALID_ARG;
    if (s.page_stride && (s.page_stride < static_cast<int64_t>(s.page_size) * s.n_kv_heads * s.head_dim || s.page_stride % 16))
        return MOE_ERR_INVALID_ARG;
    // no address computed from a stride may leave 63 bits
    if (s.q_stride > (1ll << 60) / (s.num_tokens + 1ll) || s.page_stride > (1ll << 60) / s.num_pages) return MOE_ERR_INVALID_ARG;
    auto finite = [](float x) { return x - x == 0.0f; };
    if (!finite(s.scale)) return MOE_ERR_INVALID_ARG;
    if (s.cache_dtype == MOE_E4M3 && !(s.k_scale > 0.0f && s.v_scale > 0.0f && finite(s.k_scale) && finite(s.v_scale)))
        return MOE_ERR_INVALID_ARG;
    // the kernels multiply q . k, which may be 0, by this
    if (!finite(attn_scale_log2(s))) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_attn_workspace_size(const moe_attn_shape_t *shape, size_t *bytes)
{
    const int st = check_attn(shape);
    if (st != MOE_OK) return st;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = attn_ws(*shape).total;
    return MOE_OK;
}

extern "C" int moe_paged_attention(const moe_attn_shape_t *shape, const void *q, const void *k_cache, const void *v_cache,
                                   const int32_t *block_table, const int32_t *q_start, const int32_t *kv_len, void *out,
                                   int32_t *status, void *ws, size_t ws_bytes, moe_stream_t stream)
{
    int &launches = launch_counter();
    launches = 0;
    const int st = check_attn(shape);
    if (st != MOE_OK) return st;
    const moe_attn_shape_t &s = *shape;
    if (s.num_tokens == 0) return MOE_OK;
    if (!q || !k_cache || !v_cache || !block_table || !q_start || !kv_len || !out || !ws) return MOE_ERR_INVALID_ARG;
    if (attn_misaligned(q) || attn_misaligned(k_cache) || attn_misaligned(v_cache) || attn_misaligned(out) ||
        (reinterpret_cast<uintptr_t>(ws) & 255))
        return MOE_ERR_INVALID_ARG;
    if (ws_bytes < attn_ws(s).total) return MOE_ERR_WORKSPACE_TOO_SMALL;
    const int64_t q_row = static_cast<int64_t>(s.n_heads) * s.head_dim, page_row = static_cast<int64_t>(s.page_size) * s.n_kv_heads * s.head_dim;
    const int64_t q_stride = s.q_stride ? s.q_stride : q_row, page_stride = s.page_stride ? s.page_stride : page_row;
    {
        // What the kernels write lies over nothing that they read, and over nothing else
        // that they write: other CTAs still read a request's queries when its first rows
        // are stored.
        const int64_t esz = s.cache_dtype == MOE_E4M3 ? 1 : 2;
        const Extent read[] = {{q, q_row * 2, q_stride * 2, s.num_tokens},
                               {k_cache, page_row * esz, page_stride * esz, s.num_pages},
                               {v_cache, page_row * esz, page_stride * esz, s.num_pages},
                               {block_table, static_cast<int64_t>(s.B) * s.max_pages * 4},
                               {q_start, (s.B + 1) * 4ll},
                               {kv_len, s.B * 4ll}};
        const Extent written[] = {{out, q_row * 2 * s.num_tokens}, {ws, static_cast<int64_t>(attn_ws(s).total)}, {status, 4}};
        for (int i = 0; i < 3; ++i) {
            for (const Extent &r : read)
                if (overlap(written[i], r)) return MOE_ERR_INVALID_ARG;
            for (int j = 0; j < i; ++j)
                if (overlap(written[i], written[j])) return MOE_ERR_INVALID_ARG;
        }
    }
    AttnParams p;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.table = block_table;
    p.q_start = q_start;
    p.kv_len = kv_len;
    p.out = out;
    p.status = status;
    p.q_stride = q_stride;
    p.page_stride = page_stride;
    p.B = s.B;
    p.T = s.num_tokens;
    p.n_heads = s.n_heads;
    p.n_kv = s.n_kv_heads;
    p.group = s.n_heads / s.n_kv_heads;
    p.page_size = s.page_size;
    p.by_group.set(p.group);
    p.by_page.set(p.page_size);
    p.num_pages = s.num_pages;
    p.max_pages = s.max_pages;
    p.causal = s.causal;
    p.scale_log2 = attn_scale_log2(s);
    p.v_scale = s.cache_dtype == MOE_E4M3 ? s.v_scale : 1.0f;
    cudaStream_t sm = reinterpret_cast<cudaStream_t>(stream);
    char *wb = static_cast<char *>(ws);
    if (s.head_dim == 64) return launch_attention<64>(s, p, wb, sm, launches);
    if (s.head_dim == 128) return launch_attention<128>(s, p, wb, sm, launches);
    return launch_attention<256>(s, p, wb, sm, launches);
}
