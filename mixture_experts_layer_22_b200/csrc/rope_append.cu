// rope_append.cu - rotary embedding of q and k fused with the write of k and v
// into a paged cache (moe_rope_append); of q and k the rotation that the inverse
// rotary step takes back.
//
// Each pair of a q or k head of token t, (i, i + rot_dim/2) or (2i, 2i + 1),
// becomes a' = a c - b s, b' = b c + a s with c, s from row positions[t] of the
// table; elements beyond rot_dim and all of v pass through.  fp32 arithmetic,
// one rounding at the store: to bf16, or to E4M3 of the IEEE quotient by the
// cache's scale.
//
// HBM-bound: a token's bytes are read once and written once and the rotation is
// a few instructions per element.  A token is n_heads + 2 n_kv_heads head
// vectors; head_dim / 16 lanes take one, 16 elements a lane in two 16-byte
// chunks chosen so that both elements of a pair sit in one lane (the layout of
// the inverse step).  A warp takes a run of a token's heads as one item, so that
// the position, the slot and the lane's coefficients are read once for the run;
// the first heads' loads go out before them.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "overlap.cuh"

namespace moe {

struct AppendParams {
    const __nv_bfloat16 *q, *k, *v;
    const int32_t *positions, *slots;
    const float *cos_sin;
    __nv_bfloat16 *q_out;
    void *k_cache, *v_cache;
    int32_t *status;
    long long qs, ks, vs, page_stride;
    int T, n_q, n_kv, rot_dim, max_pos, page_size, n_slots, hc;
    float k_scale, v_scale, k_rs, v_rs;   // scales and their reciprocals (0: not to be used)
};

__device__ __forceinline__ float append_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float append_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t append_bf16x2(float a, float b)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
}

// RN(a / scale) as far as its E4M3 code goes, from rs = RN(1 / scale): q = RN(a rs)
// is within an ulp, its residual is exact in one fused multiply-add, and RN(q +
// residual rs) is the correctly rounded quotient (Markstein's theorem on division by
// reciprocal refinement, "IA-64 and Elementary Functions", 2000), for scales within
// 2^-60 .. 2^60.  A q below 2^-11 has the code 0 with its sign, one of 2^10 or more
// (infinity included) saturates, and a NaN stays one: they are taken as they are.
// (An IEEE division each cost 3 us of 40 with 8192 tokens of 2 x 8 heads of 128.)
__device__ __forceinline__ float quotient(float a, float scale, float rs)
{
    const float q = __fmul_rn(a, rs);
    const float t = __fmaf_rn(__fmaf_rn(-q, scale, a), rs, q);
    constexpr uint32_t lo = 0x3A000000u, hi = 0x44800000u;              // 2^-11, 2^10
    return (__float_as_uint(q) & 0x7FFFFFFFu) - lo < hi - lo ? t : q;
}

__device__ __forceinline__ uint32_t append_e4m3x4(float a, float b, float c, float d, float scale, float rs)
{
    // rs is 0 for scales outside the range
    const float x = rs != 0.0f ? quotient(a, scale, rs) : __fdiv_rn(a, scale), y = rs != 0.0f ? quotient(b, scale, rs) : __fdiv_rn(b, scale);
    const float z = rs != 0.0f ? quotient(c, scale, rs) : __fdiv_rn(c, scale), w = rs != 0.0f ? quotient(d, scale, rs) : __fdiv_rn(d, scale);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(z, w), __NV_SATFINITE, __NV_E4M3);
    return (lo & 0xFFFFu) | (hi << 16);
}

// kL lanes per head, kP passes of 32 / kL heads whose loads are in flight
// together.
template <int kL, bool kInterleaved, bool kE4m3>
__global__ void __launch_bounds__(256) rope_append_kernel(const AppendParams p)
{
    constexpr int kHd = 16 * kL, kHpw = 32 / kL, kP = 4;
    const int lane = threadIdx.x & 31;
    const int sub = lane / kL, li = lane % kL;
    const int half = p.rot_dim >> 1;
    // the lane's two chunks of 8 elements, its first pair and how many of its
    // eight pairs rotate
    int off0 = 16 * li, off1 = off0 + 8, pair = 8 * li, n_rot;
    if (kInterleaved) {
        n_rot = min(8, max(0, half - pair));
    } else {
        const int rotating = half >> 3;
        n_rot = li < rotating ? 8 : 0;
        if (li < rotating) {
            off0 = 8 * li;
            off1 = half + 8 * li;
        } else {
            off0 = p.rot_dim + 16 * (li - rotating);
            off1 = off0 + 8;
        }
    }
    const int n_all = p.n_q + 2 * p.n_kv;
    const int n_chunks = (n_all + p.hc - 1) / p.hc;
    const long long n_items = static_cast<long long>(p.T) * n_chunks;
    const long long n_warps = static_cast<long long>(gridDim.x) * (blockDim.x >> 5);
    for (long long item = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; item < n_items;
         item += n_warps) {
        const int t = static_cast<int>(item / n_chunks);
        const int h_begin = static_cast<int>(item % n_chunks) * p.hc, h_end = min(n_all, h_begin + p.hc);
        const int slot = __ldg(p.slots + t);
        const int pos = p.rot_dim ? __ldg(p.positions + t) : 0;
        float C[8], S[8];
        long long cache_row = 0;
        for (int h0 = h_begin; h0 < h_end; h0 += kP * kHpw) {
            uint4 w[kP][2];
#pragma unroll
            for (int u = 0; u < kP; ++u) {
                const int h = h0 + u * kHpw + sub;
                if (h < h_end) {
                    const __nv_bfloat16 *src = h < p.n_q ? p.q + t * p.qs + static_cast<long long>(h) * kHd
                                             : h < p.n_q + p.n_kv ? p.k + t * p.ks + static_cast<long long>(h - p.n_q) * kHd
                                             : p.v + t * p.vs + static_cast<long long>(h - p.n_q - p.n_kv) * kHd;
                    // plain loads: q may be q_out
                    w[u][0] = *reinterpret_cast<const uint4 *>(src + off0);
                    w[u][1] = *reinterpret_cast<const uint4 *>(src + off1);
                }
            }
            if (h0 == h_begin) {
                const bool bad = slot < -1 || slot >= p.n_slots || (p.rot_dim && (pos < 0 || pos >= p.max_pos));
                if (slot == -1 || bad) {                  // the same for the whole warp
                    if (slot != -1 && lane == 0 && p.status) set_status(p.status, MOE_ERR_DEVICE_CHECK);
                    break;
                }
                cache_row = static_cast<long long>(slot / p.page_size) * p.page_stride +
                            static_cast<long long>(slot % p.page_size) * p.n_kv * kHd;
                const float *cs = p.cos_sin + static_cast<long long>(pos) * p.rot_dim;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    C[i] = i < n_rot ? __ldg(cs + pair + i) : 1.0f;
                    S[i] = i < n_rot ? __ldg(cs + half + pair + i) : 0.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < kP; ++u) {
                const int h = h0 + u * kHpw + sub;
                if (h >= h_end) continue;
                uint32_t ww[8] = {w[u][0].x, w[u][0].y, w[u][0].z, w[u][0].w, w[u][1].x, w[u][1].y, w[u][1].z, w[u][1].w};
                const bool is_q = h < p.n_q, is_v = h >= p.n_q + p.n_kv;
                float x[16];                              // in element order
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[2 * i] = append_lo(ww[i]);
                    x[2 * i + 1] = append_hi(ww[i]);
                }
                if (!is_v) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int ia = kInterleaved ? 2 * i : i, ib = kInterleaved ? 2 * i + 1 : 8 + i;
                        const float a = x[ia], b = x[ib];
                        if (i < n_rot) {
                            x[ia] = a * C[i] - b * S[i];
                            x[ib] = b * C[i] + a * S[i];
                        }
                    }
                }
                if (kE4m3 && !is_q) {
                    const float sc = is_v ? p.v_scale : p.k_scale, rs = is_v ? p.v_rs : p.k_rs;
                    uint8_t *dst = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) + cache_row +
                                   static_cast<long long>(h - p.n_q - (is_v ? p.n_kv : 0)) * kHd;
                    *reinterpret_cast<uint2 *>(dst + off0) = make_uint2(append_e4m3x4(x[0], x[1], x[2], x[3], sc, rs),
                                                                        append_e4m3x4(x[4], x[5], x[6], x[7], sc, rs));
                    *reinterpret_cast<uint2 *>(dst + off1) = make_uint2(append_e4m3x4(x[8], x[9], x[10], x[11], sc, rs),
                                                                        append_e4m3x4(x[12], x[13], x[14], x[15], sc, rs));
                    continue;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (!is_v) ww[i] = append_bf16x2(x[2 * i], x[2 * i + 1]);
                __nv_bfloat16 *dst =
                    is_q ? p.q_out + (static_cast<long long>(t) * p.n_q + h) * kHd
                         : static_cast<__nv_bfloat16 *>(is_v ? p.v_cache : p.k_cache) + cache_row +
                               static_cast<long long>(h - p.n_q - (is_v ? p.n_kv : 0)) * kHd;
                *reinterpret_cast<uint4 *>(dst + off0) = make_uint4(ww[0], ww[1], ww[2], ww[3]);
                *reinterpret_cast<uint4 *>(dst + off1) = make_uint4(ww[4], ww[5], ww[6], ww[7]);
            }
        }
    }
}

template <int kL, bool kInterleaved, bool kE4m3>
static void launch_append(const AppendParams &p, long long items, cudaStream_t st)
{
    const long long want = (items + 7) / 8;
    const long long cap = 148LL * 2;                          // the blocks that are resident at once
    rope_append_kernel<kL, kInterleaved, kE4m3><<<static_cast<int>(want < cap ? want : cap), 256, 0, st>>>(p);
}

}  // namespace moe

using namespace moe;

static bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

extern "C" int moe_rope_append(const moe_append_shape_t *shape, const void *q, const void *k, const void *v,
                               const int32_t *positions, const int32_t *slots, const float *cos_sin, void *q_out,
                               void *k_cache, void *v_cache, int32_t *status, moe_stream_t stream)
{
    int &launches = launch_counter();
    launches = 0;
    if (!shape) return MOE_ERR_INVALID_ARG;
    const moe_append_shape_t &s = *shape;
    if (s.num_tokens < 0 || s.n_heads < 1 || s.n_kv_heads < 1 || s.n_heads > 65536 || s.n_kv_heads > 65536 || s.rot_dim < 0 ||
        (s.rot_dim & 1) || s.rot_dim > s.head_dim || (s.rot_dim > 0 && s.max_pos < 1) ||
        (s.interleaved != 0 && s.interleaved != 1) || s.page_size < 1 || s.num_pages < 1 ||
        (s.cache_dtype != MOE_BF16 && s.cache_dtype != MOE_E4M3))
        return MOE_ERR_INVALID_ARG;
    if (s.head_dim != 64 && s.head_dim != 128 && s.head_dim != 256) return MOE_ERR_UNSUPPORTED;
    if (!s.interleaved && s.rot_dim % 16 != 0) return MOE_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(s.num_pages) * s.page_size > 0x7fffffffll) return MOE_ERR_INVALID_ARG;
    AppendParams p;
    const int64_t q_row = static_cast<int64_t>(s.n_heads) * s.head_dim, kv_row = static_cast<int64_t>(s.n_kv_heads) * s.head_dim;
    p.qs = s.q_stride ? s.q_stride : q_row;
    p.ks = s.k_stride ? s.k_stride : kv_row;
    p.vs = s.v_stride ? s.v_stride : kv_row;
    p.page_stride = s.page_stride ? s.page_stride : kv_row * s.page_size;
    if (p.qs < q_row || p.ks < kv_row || p.vs < kv_row || p.page_stride < kv_row * s.page_size || p.qs % 8 || p.ks % 8 ||
        p.vs % 8 || p.page_stride % 16)
        return MOE_ERR_INVALID_ARG;
    // no address computed from a stride may leave 63 bits
    const int64_t most = (1ll << 60) / (s.num_tokens + 1ll);
    if (p.qs > most || p.ks > most || p.vs > most || p.page_stride > (1ll << 60) / s.num_pages) return MOE_ERR_INVALID_ARG;
    auto finite = [](float x) { return x - x == 0.0f; };
    if (s.cache_dtype == MOE_E4M3 && !(s.k_scale > 0.0f && s.v_scale > 0.0f && finite(s.k_scale) && finite(s.v_scale)))
        return MOE_ERR_INVALID_ARG;
    if (s.num_tokens == 0) return MOE_OK;
    if (!q || !k || !v || !slots || !q_out || !k_cache || !v_cache) return MOE_ERR_INVALID_ARG;
    if (s.rot_dim > 0 && (!positions || !cos_sin)) return MOE_ERR_INVALID_ARG;
    if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(q_out, 16) || misaligned(k_cache, 16) ||
        misaligned(v_cache, 16) || misaligned(cos_sin, 4))
        return MOE_ERR_INVALID_ARG;
    if (q == q_out && p.qs != q_row) return MOE_ERR_INVALID_ARG;
    {
        // What the kernel writes lies over nothing else: the warps read and write tokens
        // and heads in any order.  In place, a lane writes only what it has read itself;
        // one cache for both is the caller's statement that k and v are the same.
        const int64_t esz = s.cache_dtype == MOE_E4M3 ? 1 : 2, n = s.num_tokens, rot = s.rot_dim > 0;
        const Extent written[] = {{q_out, q_row * 2 * n},
                                  {k_cache, kv_row * s.page_size * esz, p.page_stride * esz, s.num_pages},
                                  {v_cache, kv_row * s.page_size * esz, p.page_stride * esz, s.num_pages},
                                  {status, 4}};
        const Extent read[] = {{q, q_row * 2, p.qs * 2, n},
                               {k, kv_row * 2, p.ks * 2, n},
                               {v, kv_row * 2, p.vs * 2, n},
                               {slots, 4 * n},
                               {positions, 4 * n * rot},
                               {cos_sin, 4ll * s.max_pos * s.rot_dim * rot}};
        for (int i = 0; i < 4; ++i) {
            for (int j = 0; j < 6; ++j)
                if (overlap(written[i], read[j]) && !(i == 0 && j == 0 && q_out == q)) return MOE_ERR_INVALID_ARG;
            for (int j = 0; j < i; ++j)
                if (overlap(written[i], written[j]) && !(i == 2 && j == 1 && v_cache == k_cache)) return MOE_ERR_INVALID_ARG;
        }
    }
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.positions = positions;
    p.slots = slots;
    p.cos_sin = cos_sin;
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.status = status;
    p.T = s.num_tokens;
    p.n_q = s.n_heads;
    p.n_kv = s.n_kv_heads;
    p.rot_dim = s.rot_dim;
    p.max_pos = s.max_pos;
    p.page_size = s.page_size;
    p.n_slots = s.num_pages * s.page_size;
    p.k_scale = s.k_scale;
    p.v_scale = s.v_scale;
    auto reciprocal = [](float x) { return x >= 0x1p-60f && x <= 0x1p60f ? 1.0f / x : 0.0f; };
    p.k_rs = reciprocal(s.k_scale);
    p.v_rs = reciprocal(s.v_scale);
    const int L = s.head_dim / 16, hpw = 32 / L, n_all = s.n_heads + 2 * s.n_kv_heads;
    // heads per item: all of a token's heads when there are tokens enough to
    // give every SM 32 warps, else fewer so that small batches spread over the GPU
    int hc = (n_all + hpw - 1) / hpw * hpw;
    while (hc > hpw && static_cast<long long>(s.num_tokens) * ((n_all + hc - 1) / hc) < 148LL * 32)
        hc = ((hc / 2) + hpw - 1) / hpw * hpw;
    p.hc = hc;
    const long long items = static_cast<long long>(s.num_tokens) * ((n_all + hc - 1) / hc);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool e4m3 = s.cache_dtype == MOE_E4M3;
#define MOE_APPEND(LL)                                                                                     \
    do {                                                                                                   \
        if (s.interleaved && e4m3) launch_append<LL, true, true>(p, items, st);                            \
        else if (s.interleaved) launch_append<LL, true, false>(p, items, st);                              \
        else if (e4m3) launch_append<LL, false, true>(p, items, st);                                       \
        else launch_append<LL, false, false>(p, items, st);                                                \
    } while (0)
    if (L == 4) MOE_APPEND(4);
    else if (L == 8) MOE_APPEND(8);
    else MOE_APPEND(16);
#undef MOE_APPEND
    launches = 1;
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
