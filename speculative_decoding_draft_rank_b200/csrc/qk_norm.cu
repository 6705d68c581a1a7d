// qk_norm.cu -- the pass between a target layer's projections and its
// attention: RMS norm of every query and key head, position rotation, and the
// write of keys and values into the paged 4-bit cache; and the gather that
// reads cached tokens back.
//
//   y = x / sqrt(mean(x^2) + eps) * w          (no w: y = x)
//   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t),
//     t = pos * inv_freq[i], pairs (i, i + rot/2) or interleaved (2i, 2i + 1)
//   scale = e4m3(max |y| over 16 dims / (6 g)), code = e2m1(y / (scale g)),
//     both to nearest, ties to even (g = k_scale or v_scale).
//
// A CTA takes one token.  A row (head) belongs to D / 16 neighbouring lanes;
// lane i holds two octets of dims that rotate with each other: dims 8i.. and
// rot/2 + 8i.. of the rotated part, or two octets of the rest.  So a rotation
// needs no exchange, the 16 dims of a scale are two neighbouring lanes, and
// loads and stores are 16 bytes.  The angles are reduced to a turn in fp64 (a
// position of 2^20 times a frequency has 44 bits), then sine and cosine run in
// fp32 once per token and frequency, shared by all heads.
// Measured (bf16, D = 128, with the cache write): 1184 tokens of 64 query and 8
// key heads (45 MB) 14 us, 5200 tokens of 32 and 8 (113 MB) 39 us with the rows
// in L2 and 45 from HBM, one token 3 to 4 us in a graph; HBM alone would need 7
// and 17 us.  Reading the same tokens back takes 3.1, 6.4 and 2 us (0.9 and 4.2).
// What bounds the large ones: four CTAs of 128 threads fit an SM (104 to 124
// registers), and a token's positions, angles and first rows are waited for
// before its arithmetic begins, so time goes up by waves of 592 tokens (592
// tokens 8.0 us, 740 12.7, 1184 14.3); inside a wave the schedulers issue in
// 53 % of the cycles (hence two-lane fp32 arithmetic and several rows a
// thread), at 20 % of DRAM's rate.
#include "cache.cuh"

namespace dspark {

namespace {

constexpr int kMaxThreads = 512;
constexpr int kOnePerSm = 148;   // tokens that get an SM each

struct Oct {
    float2 v[4];
};
// Eight elements as loaded (widened when they are used, so that rows under
// way take few registers).
template <typename T> struct Raw;
template <> struct Raw<float> { float4 a, b; };
template <> struct Raw<__nv_bfloat16> { uint4 x; };
__device__ __forceinline__ void load8(Raw<float> &r, const float *p) {
    r.a = __ldcs(reinterpret_cast<const float4 *>(p));
    r.b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
}
__device__ __forceinline__ void load8(Raw<__nv_bfloat16> &r, const __nv_bfloat16 *p) {
    r.x = __ldcs(reinterpret_cast<const uint4 *>(p));
}
__device__ __forceinline__ Oct widen(const Raw<float> &r) {
    return {{make_float2(r.a.x, r.a.y), make_float2(r.a.z, r.a.w), make_float2(r.b.x, r.b.y), make_float2(r.b.z, r.b.w)}};
}
__device__ __forceinline__ Oct widen(const Raw<__nv_bfloat16> &r) {
    return {{make_float2(bf16lo(r.x.x), bf16hi(r.x.x)), make_float2(bf16lo(r.x.y), bf16hi(r.x.y)),
             make_float2(bf16lo(r.x.z), bf16hi(r.x.z)), make_float2(bf16lo(r.x.w), bf16hi(r.x.w))}};
}
__device__ __forceinline__ void store8(float *p, const Oct &q) {
    *reinterpret_cast<float4 *>(p) = make_float4(q.v[0].x, q.v[0].y, q.v[1].x, q.v[1].y);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(q.v[2].x, q.v[2].y, q.v[3].x, q.v[3].y);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const Oct &q) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 x = __float22bfloat162_rn(q.v[i]);
        w[i] = *reinterpret_cast<const uint32_t *>(&x);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 pa, pb, pd;\n\tmov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
        "mul.rn.f32x2 pd, pa, pb;\n\tmov.b64 {%0, %1}, pd;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// x / y correctly rounded, from r = 1 / y correctly rounded: the remainder of
// the first product is exact in an fma, and one step with it rounds the
// quotient as a division would (P. Markstein, IBM J. Res. Dev. 34, 1990).
// Finite operands, no overflow of x * r.
__device__ __forceinline__ float quotient(float x, float y, float r) {
    const float q = x * r;
    return fmaf(fmaf(-q, y, x), r, q);
}

// Where a lane stores an octet of a row: offsets in a half record.
struct Place {
    int codes, scale;
};

// An octet of a group of 16 (this lane and its neighbour) to `half`.  NaN
// goes to 0 and infinities to the largest value; both are reported.  g6 = 6 g,
// r6 its reciprocal.  Values are clamped to where they saturate before they
// are divided, so no quotient overflows.
__device__ __forceinline__ bool quantise8(const Oct &q, float g, float g6, float r6, uint8_t *half, const Place &at,
                                          bool lead, bool live) {
    float x[8], m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = i & 1 ? q.v[i / 2].y : q.v[i / 2].x;
        m = fmaxf(m, fabsf(x[i]));           // passes NaN by
    }
    // A sum with 0 * x is 0 unless an x is infinite or NaN.
    float odd = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) odd = fmaf(0.f, x[i], odd);
    const bool bad = odd != 0.f;             // also for NaN
    if (bad) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] == x[i] ? x[i] : 0.f;
    }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    uint16_t s8;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(s8)
        : "f"(0.f), "f"(quotient(fminf(m, 512.f * g6), g6, r6)));
    const float s = __half2float(__ushort_as_half((unsigned short)((s8 & 0x7f) << 7))) * 256.f * g;
    uint32_t codes = 0;
    if (s > 0.f) {
        const float r = __frcp_rn(s), top = 8.f * s;
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = quotient(fminf(fmaxf(x[2 * i], -top), top), s, r);
            const float hi = quotient(fminf(fmaxf(x[2 * i + 1], -top), top), s, r);
            asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}"
                : "=r"(c[i])
                : "f"(lo), "f"(hi));
        }
        codes = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
    }
    if (live) {
        *reinterpret_cast<uint32_t *>(half + at.codes) = codes;
        if (lead) half[at.scale] = (uint8_t)(s8 & 0x7f);
    }
    return bad && live;
}

template <typename T, int D, bool WRITE>
__global__ void __launch_bounds__(kMaxThreads, 1) qk_norm_rope_kernel(const NormArgs a) {
    constexpr int kLanes = D / 16;
    constexpr int kUnder = sizeof(T) == 2 ? 3 : 2;     // rows under way per thread
    __shared__ __align__(16) float2 cs[D / 2];
    const int t = blockIdx.x;
    const int i = threadIdx.x % kLanes;
    const int rows = a.Hq + (WRITE ? 2 : 1) * a.Hkv;
    const int n_rot = a.rot / 16;
    const bool rotated = i < n_rot;
    // First dims of this lane's octets.
    const int da = 8 * (rotated ? i : a.rot / 8 + (i - n_rot));
    const int db = 8 * (rotated ? i + n_rot : a.rot / 8 + (D - a.rot) / 16 + (i - n_rot));
    // Row r is at q_row + r * D, or the k_row or v_row that makes it so.
    const T *q_row = static_cast<const T *>(a.q) + (long long)t * a.q_stride;
    const T *k_row = static_cast<const T *>(a.k) + (long long)t * a.k_stride - a.Hq * D;
    const T *v_row = WRITE ? static_cast<const T *>(a.v) + (long long)t * a.v_stride - (a.Hq + a.Hkv) * D : nullptr;
    const int step = blockDim.x / kLanes, first = threadIdx.x / kLanes;
    Raw<T> ra[kUnder], rb[kUnder];
    auto fetch = [&](int r0) {
#pragma unroll
        for (int u = 0; u < kUnder; ++u)
            if (r0 + u * step < rows) {
                const int r = r0 + u * step;
                const T *p = (r < a.Hq ? q_row : r < a.Hq + a.Hkv ? k_row : v_row) + r * D;
                load8(ra[u], p + da);
                load8(rb[u], p + db);
            }
    };
    // Everything the token needs is asked for before anything is waited for.
    const int n_rows = a.n_rows != nullptr ? __ldg(a.n_rows) : a.T;
    const int pos = a.rot > 0 ? __ldg(a.pos + t) : 0;
    int slot = WRITE ? __ldg(a.slot + t) : -1;
    if (t >= n_rows) return;
    fetch(first);
    // This lane's norm weights, as loaded.
    Raw<T> wqa = {}, wqb = {}, wka = {}, wkb = {};
    if (a.wq != nullptr) {
        load8(wqa, static_cast<const T *>(a.wq) + da);
        load8(wqb, static_cast<const T *>(a.wq) + db);
    }
    if (a.wk != nullptr) {
        load8(wka, static_cast<const T *>(a.wk) + da);
        load8(wkb, static_cast<const T *>(a.wk) + db);
    }
    for (int f = threadIdx.x; f < a.rot / 2; f += blockDim.x) {
        // The angle in half turns, less whole turns, in fp64.
        const double x = (double)pos * (double)__ldg(a.inv_freq + f) * 0.15915494309189533577;
        float s, c;
        sincospif((float)(2.0 * (x - rint(x))), &s, &c);
        cs[f] = make_float2(c, s);
    }
    uint8_t *record = nullptr;   // the token's page, head 0
    Place pa = {}, pb = {};
    const bool lead = (i & 1) == 0;
    const int rec = record_bytes(a.P, D), kv_half = half_bytes(a.P, D);
    if (WRITE) {
        if (slot >= a.n_pages * a.P) {
            if (threadIdx.x == 0) flag_status(a.hdr, DSPARK_DEV_PAGE_RANGE);
            slot = -1;
        }
        const int page = slot >= 0 ? slot / a.P : 0, off = slot >= 0 ? slot - page * a.P : 0;
        record = a.cache + (size_t)page * a.Hkv * rec;
        const int scales = half_scales_off(a.P, D) + off * (D / 16);
        pa = {(da / 32 * a.P + off) * 16 + da % 32 / 2, scales + da / 16};
        pb = {(db / 32 * a.P + off) * 16 + db % 32 / 2, scales + db / 16};
    }
    __syncthreads();
    // Whole warps stay in the loops together (the shuffles name all lanes).
    bool bad = false;
    const float rk = WRITE ? __frcp_rn(6.f * a.k_scale) : 0.f, rv = WRITE ? __frcp_rn(6.f * a.v_scale) : 0.f;
    for (int r0 = first, k0 = 0; k0 < rows; r0 += kUnder * step, k0 += kUnder * step) {
        if (k0 > 0) fetch(r0);
#pragma unroll
        for (int u = 0; u < kUnder; ++u) {
            if (k0 + u * step >= rows) break;          // the whole block
            const int r = r0 + u * step;
            const bool live = r < rows;
            const bool is_v = r >= a.Hq + a.Hkv, is_k = !is_v && r >= a.Hq;
            Oct xa = {}, xb = {};
            if (live) {
                xa = widen(ra[u]);
                xb = widen(rb[u]);
            }
            if (__any_sync(0xffffffffu, !is_v) && (a.wq != nullptr || a.wk != nullptr)) {
                float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < 4; ++e) s2 = fma2(xa.v[e], xa.v[e], fma2(xb.v[e], xb.v[e], s2));
                float ss = s2.x + s2.y;
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (!is_v && (is_k ? a.wk : a.wq) != nullptr) {
                    const float inv = __frsqrt_rn(ss * (1.f / D) + a.eps);
                    const float2 inv2 = make_float2(inv, inv);
                    const Oct wa = widen(is_k ? wka : wqa), wb = widen(is_k ? wkb : wqb);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        xa.v[e] = mul2(mul2(xa.v[e], inv2), wa.v[e]);
                        xb.v[e] = mul2(mul2(xb.v[e], inv2), wb.v[e]);
                    }
                }
            }
            if (!is_v && rotated) {
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 ca = cs[da / 2 + e], cb = cs[db / 2 + e];
                        xa.v[e] = make_float2(xa.v[e].x * ca.x - xa.v[e].y * ca.y, xa.v[e].y * ca.x + xa.v[e].x * ca.y);
                        xb.v[e] = make_float2(xb.v[e].x * cb.x - xb.v[e].y * cb.y, xb.v[e].y * cb.x + xb.v[e].x * cb.y);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 c4 = *reinterpret_cast<const float4 *>(&cs[da + 2 * e]);   // two dims' (cos, sin)
                        const float2 c = make_float2(c4.x, c4.z), s = make_float2(c4.y, c4.w);
                        const float2 p = xa.v[e], q = xb.v[e];
                        xa.v[e] = fma2(p, c, mul2(q, make_float2(-s.x, -s.y)));
                        xb.v[e] = fma2(q, c, mul2(p, s));
                    }
                }
            }
            if (live && r < a.Hq) {
                T *o = static_cast<T *>(a.q_out) + ((long long)t * a.Hq + r) * D;
                store8(o + da, xa);
                store8(o + db, xb);
            }
            if (live && is_k && a.k_out != nullptr) {
                T *o = static_cast<T *>(a.k_out) + ((long long)t * a.Hkv + r - a.Hq) * D;
                store8(o + da, xa);
                store8(o + db, xb);
            }
            if (WRITE) {
                // A warp whose rows are all queries has nothing to quantise.
                if (__any_sync(0xffffffffu, live && r >= a.Hq)) {
                    const bool put = live && r >= a.Hq && slot >= 0;
                    const int h = is_v ? r - a.Hq - a.Hkv : r - a.Hq;
                    uint8_t *half = record + (put ? h * rec + (is_v ? kv_half : 0) : 0);
                    const float g = is_v ? a.v_scale : a.k_scale, g6 = 6.f * g, r6 = is_v ? rv : rk;
                    bad |= quantise8(xa, g, g6, r6, half, pa, lead, put);
                    bad |= quantise8(xb, g, g6, r6, half, pb, lead, put);
                }
            }
        }
    }
    if (WRITE && bad) flag_status(a.hdr, DSPARK_DEV_BAD_VALUE);
}

template <typename T, int D>
cudaError_t launch_norm_d(const NormArgs &a, cudaStream_t st) {
    constexpr int kLanes = D / 16;
    const bool write = a.cache != nullptr;
    const int rows = a.Hq + (write ? 2 : 1) * a.Hkv;
    // Up to a token per SM: all rows at once, for the latency.  More: 128
    // threads with several rows each, so that what a thread sets up serves them
    // all.  Measured with 64 query and 8 key heads, all at once against 128
    // threads: 1 token 4.3 and 5.3 us, 148 tokens 4.5 and 5.5, 296 8.2 and 6.4,
    // 592 15.0 and 8.0.
    int threads = round_up(rows * kLanes, 32);
    const int most = a.T > kOnePerSm ? 128 : kMaxThreads;
    if (threads > most) threads = most;
    if (write)
        qk_norm_rope_kernel<T, D, true><<<a.T, threads, 0, st>>>(a);
    else
        qk_norm_rope_kernel<T, D, false><<<a.T, threads, 0, st>>>(a);
    return cudaGetLastError();
}

// A CTA per token, eight dims a thread and step: four bytes of codes and one scale.
constexpr int kReadThreads = 128;
template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const ReadArgs a) {
    constexpr int kPer = D / 8;
    const int t = blockIdx.x, slot = __ldg(a.slot + t);
    if (slot < 0) return;
    if (slot >= a.n_pages * a.P) {
        if (threadIdx.x == 0) flag_status(a.hdr, DSPARK_DEV_PAGE_RANGE);
        return;
    }
    const int page = slot / a.P, off = slot - page * a.P, rec = record_bytes(a.P, D), hb = half_bytes(a.P, D);
    const uint8_t *record = a.cache + (size_t)page * a.Hkv * rec;
    const int e = threadIdx.x % kPer;              // the same octet of every row
    const int codes_at = (e / 4 * a.P + off) * 16 + e % 4 * 4, scale_at = half_scales_off(a.P, D) + off * (D / 16) + e / 2;
    for (int row = threadIdx.x / kPer; row < 2 * a.Hkv; row += kReadThreads / kPer) {   // K heads, then V heads
        const bool is_v = row >= a.Hkv;
        const int h = is_v ? row - a.Hkv : row;
        const uint8_t *half = record + h * rec + (is_v ? hb : 0);
        const uint32_t codes = __ldg(reinterpret_cast<const uint32_t *>(half + codes_at));
        const uint32_t s = __ldg(half + scale_at);
        uint32_t r[4];
        e2m1x8_to_f16(codes, r[0], r[1], r[2], r[3]);
        const uint32_t sf = scale_f16x2<0>(s);
        const float g = is_v ? a.v_scale : a.k_scale;
        Oct v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t m = mul_f16x2(r[i], sf);
            v.v[i] = mul2(__half22float2(*reinterpret_cast<const __half2 *>(&m)), make_float2(g, g));
        }
        store8(static_cast<T *>(is_v ? a.v_out : a.k_out) + ((size_t)t * a.Hkv + h) * D + e * 8, v);
    }
}

template <typename T>
cudaError_t launch_read(const ReadArgs &a, cudaStream_t st) {
    if (a.D == 128)
        cache_read_kernel<T, 128><<<a.T, kReadThreads, 0, st>>>(a);
    else
        cache_read_kernel<T, 64><<<a.T, kReadThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormArgs &a, cudaStream_t st) {
    if (a.dtype == DSPARK_BF16)
        return a.D == 128 ? launch_norm_d<__nv_bfloat16, 128>(a, st) : launch_norm_d<__nv_bfloat16, 64>(a, st);
    return a.D == 128 ? launch_norm_d<float, 128>(a, st) : launch_norm_d<float, 64>(a, st);
}

cudaError_t launch_cache_read(const ReadArgs &a, cudaStream_t st) {
    return a.dtype == DSPARK_BF16 ? launch_read<__nv_bfloat16>(a, st) : launch_read<float>(a, st);
}

}  // namespace dspark
