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
// A CTA takes one token.  A row (head) belongs to D / 8 neighbouring lanes;
// lane i holds two groups of four dims that rotate with each other: dims
// 4i.. and rot/2 + 4i.. of the rotated part, or two groups of the rest.  So a
// rotation needs no exchange, 16 dims of a scale are four neighbouring lanes,
// and loads and stores stay contiguous.  The angles are reduced modulo 2 pi in
// fp64 (a position of 2^20 times a frequency has 44 bits), then sine and
// cosine run in fp32 once per token and frequency, shared by all heads.
// Bytes bound it: each row is read and written once.
#include "cache.cuh"

namespace dspark {

namespace {

constexpr int kMaxThreads = 512;

struct Quad {
    float v[4];
};
__device__ __forceinline__ Quad load4(const float *p) {
    const float4 x = __ldcs(reinterpret_cast<const float4 *>(p));
    return {{x.x, x.y, x.z, x.w}};
}
__device__ __forceinline__ Quad load4(const __nv_bfloat16 *p) {
    const uint2 x = __ldcs(reinterpret_cast<const uint2 *>(p));
    return {{bf16lo(x.x), bf16hi(x.x), bf16lo(x.y), bf16hi(x.y)}};
}
__device__ __forceinline__ Quad weight4(const float *p) {
    const float4 x = __ldg(reinterpret_cast<const float4 *>(p));
    return {{x.x, x.y, x.z, x.w}};
}
__device__ __forceinline__ Quad weight4(const __nv_bfloat16 *p) {
    const uint2 x = __ldg(reinterpret_cast<const uint2 *>(p));
    return {{bf16lo(x.x), bf16hi(x.x), bf16lo(x.y), bf16hi(x.y)}};
}
__device__ __forceinline__ void store4(float *p, const Quad &q) {
    *reinterpret_cast<float4 *>(p) = make_float4(q.v[0], q.v[1], q.v[2], q.v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const Quad &q) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(q.v[0], q.v[1]), b = __floats2bfloat162_rn(q.v[2], q.v[3]);
    *reinterpret_cast<uint2 *>(p) =
        make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// Four dims of a group of 16 (four neighbouring lanes) into the half record
// at `half`: quad u of the token at page offset `off`.  NaN goes to 0 and
// infinities to the largest value; both are reported.
__device__ __forceinline__ bool quantise4(const Quad &q, float g, uint8_t *half, int u, int off, int P, int D,
                                          bool live) {
    bool bad = false;
    float x[4], m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bad |= !(fabsf(q.v[i]) <= 3.402823466e38f);
        x[i] = q.v[i] == q.v[i] ? q.v[i] : 0.f;
        m = fmaxf(m, fabsf(x[i]));
    }
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    uint16_t s8;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(s8) : "f"(0.f), "f"(__fdiv_rn(m, 6.f * g)));
    const float s = __half2float(__ushort_as_half((unsigned short)((s8 & 0x7f) << 7))) * 256.f * g;
    uint32_t codes = 0;
    if (s > 0.f) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            uint32_t c;
            asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}"
                : "=r"(c)
                : "f"(__fdiv_rn(x[i], s)), "f"(__fdiv_rn(x[i + 1], s)));
            codes |= c << (4 * i);
        }
    }
    if (live) {
        *reinterpret_cast<uint16_t *>(half + (u / 8) * (P * 16) + off * 16 + (u % 8) * 2) = (uint16_t)codes;
        if ((u & 3) == 0) half[half_scales_off(P, D) + off * (D / 16) + u / 4] = (uint8_t)(s8 & 0x7f);
    }
    return bad && live;
}

template <typename T, int D, bool WRITE>
__global__ void __launch_bounds__(kMaxThreads) qk_norm_rope_kernel(const NormArgs a) {
    constexpr int kLanes = D / 8;
    __shared__ float2 cs[D / 2];
    const int t = blockIdx.x;
    if (a.n_rows != nullptr && t >= __ldg(a.n_rows)) return;
    const int i = threadIdx.x % kLanes;
    const int rows = a.Hq + (WRITE ? 2 : 1) * a.Hkv;
    const int n_rot = a.rot / 8;
    const bool rotated = i < n_rot;
    // Quads of this lane, in units of four dims.
    const int ua = rotated ? i : a.rot / 4 + (i - n_rot);
    const int ub = rotated ? i + n_rot : a.rot / 4 + (D - a.rot) / 8 + (i - n_rot);
    auto source = [&](int r) -> const T * {
        if (r < a.Hq) return static_cast<const T *>(a.q) + (long long)t * a.q_stride + r * D;
        if (r < a.Hq + a.Hkv) return static_cast<const T *>(a.k) + (long long)t * a.k_stride + (r - a.Hq) * D;
        return static_cast<const T *>(a.v) + (long long)t * a.v_stride + (r - a.Hq - a.Hkv) * D;
    };
    int r = threadIdx.x / kLanes;
    const int step = blockDim.x / kLanes;
    Quad xa, xb;
    if (r < rows) {
        const T *p = source(r);
        xa = load4(p + 4 * ua);
        xb = load4(p + 4 * ub);
    }
    if ((int)threadIdx.x < a.rot / 2) {
        // t = pos * f exactly in fp64, less the nearest multiple of 2 pi.
        const double x = (double)__ldg(a.pos + t) * (double)__ldg(a.inv_freq + threadIdx.x);
        const double k = rint(x * 0.15915494309189533577);
        const float y = (float)fma(-k, 2.4492935982947064e-16, fma(-k, 6.283185307179586232, x));
        float s, c;
        sincosf(y, &s, &c);
        cs[threadIdx.x] = make_float2(c, s);
    }
    int slot = -1, page = 0, off = 0;
    if (WRITE) {
        slot = __ldg(a.slot + t);
        if (slot >= a.n_pages * a.P) {
            if (threadIdx.x == 0) flag_status(a.hdr, DSPARK_DEV_PAGE_RANGE);
            slot = -1;
        }
        if (slot >= 0) {
            page = slot / a.P;
            off = slot % a.P;
        }
    }
    __syncthreads();
    // Whole warps stay in the loop together (the shuffles name all lanes).
    const int rounds = (rows + step - 1) / step;
    bool bad = false;
    for (int k = 0; k < rounds; ++k, r += step) {
        const bool live = r < rows;
        Quad na, nb;
        if (r + step < rows) {   // the next row is in flight while this one is worked on
            const T *p = source(r + step);
            na = load4(p + 4 * ua);
            nb = load4(p + 4 * ub);
        }
        const bool is_v = r >= a.Hq + a.Hkv, is_k = !is_v && r >= a.Hq;
        if (!live) {
#pragma unroll
            for (int e = 0; e < 4; ++e) xa.v[e] = xb.v[e] = 0.f;
        }
        const void *w = is_k ? a.wk : a.wq;
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fmaf(xa.v[e], xa.v[e], fmaf(xb.v[e], xb.v[e], ss));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (!is_v && w != nullptr) {
            const float inv = __frsqrt_rn(ss * (1.f / D) + a.eps);
            const Quad wa = weight4(static_cast<const T *>(w) + 4 * ua), wb = weight4(static_cast<const T *>(w) + 4 * ub);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                xa.v[e] = xa.v[e] * inv * wa.v[e];
                xb.v[e] = xb.v[e] * inv * wb.v[e];
            }
        }
        if (!is_v && rotated) {
            if (a.interleaved) {
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float2 ca = cs[2 * ua + e / 2], cb = cs[2 * ub + e / 2];
                    const float a0 = xa.v[e], a1 = xa.v[e + 1], c0 = xb.v[e], c1 = xb.v[e + 1];
                    xa.v[e] = a0 * ca.x - a1 * ca.y;
                    xa.v[e + 1] = a1 * ca.x + a0 * ca.y;
                    xb.v[e] = c0 * cb.x - c1 * cb.y;
                    xb.v[e + 1] = c1 * cb.x + c0 * cb.y;
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 c = cs[4 * ua + e];
                    const float p = xa.v[e], q = xb.v[e];
                    xa.v[e] = p * c.x - q * c.y;
                    xb.v[e] = q * c.x + p * c.y;
                }
            }
        }
        if (live && r < a.Hq) {
            T *o = static_cast<T *>(a.q_out) + ((long long)t * a.Hq + r) * D;
            store4(o + 4 * ua, xa);
            store4(o + 4 * ub, xb);
        }
        if (live && is_k && a.k_out != nullptr) {
            T *o = static_cast<T *>(a.k_out) + ((long long)t * a.Hkv + r - a.Hq) * D;
            store4(o + 4 * ua, xa);
            store4(o + 4 * ub, xb);
        }
        if (WRITE) {
            // A warp whose rows are all queries has nothing to quantise.
            if (__any_sync(0xffffffffu, live && r >= a.Hq)) {
                const bool put = live && r >= a.Hq && slot >= 0;
                const int h = is_v ? r - a.Hq - a.Hkv : (r >= a.Hq ? r - a.Hq : 0);
                uint8_t *half = a.cache + ((size_t)page * a.Hkv + (put ? h : 0)) * record_bytes(a.P, D) +
                                (is_v ? half_bytes(a.P, D) : 0);
                const float g = is_v ? a.v_scale : a.k_scale;
                bad |= quantise4(xa, g, half, ua, off, a.P, D, put);
                bad |= quantise4(xb, g, half, ub, off, a.P, D, put);
            }
        }
        xa = na;
        xb = nb;
    }
    if (WRITE && bad) flag_status(a.hdr, DSPARK_DEV_BAD_VALUE);
}

template <typename T, int D>
cudaError_t launch_norm_d(const NormArgs &a, cudaStream_t st) {
    constexpr int kLanes = D / 8;
    const bool write = a.cache != nullptr;
    const int rows = a.Hq + (write ? 2 : 1) * a.Hkv;
    // As few rounds over the rows as 512 threads allow, the rows dealt evenly.
    const int rounds = (rows * kLanes + kMaxThreads - 1) / kMaxThreads;
    int threads = round_up((rows + rounds - 1) / rounds * kLanes, 32);
    if (threads < D / 2) threads = D / 2;   // one thread per frequency
    if (write)
        qk_norm_rope_kernel<T, D, true><<<a.T, threads, 0, st>>>(a);
    else
        qk_norm_rope_kernel<T, D, false><<<a.T, threads, 0, st>>>(a);
    return cudaGetLastError();
}

__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&x);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight dims a thread: four bytes of codes and one scale.
template <typename T, int D>
__global__ void __launch_bounds__(256) cache_read_kernel(const ReadArgs a) {
    constexpr int kPer = D / 8;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const int e = (int)(id % kPer);
    const long long row = id / kPer;               // (token, K or V, head)
    const int h = (int)(row % a.Hkv), part = (int)(row / a.Hkv % 2);
    const long long t = row / (2 * a.Hkv);
    if (t >= a.T) return;
    const int slot = __ldg(a.slot + t);
    if (slot < 0) return;
    if (slot >= a.n_pages * a.P) {
        if (e == 0 && h == 0 && part == 0) flag_status(a.hdr, DSPARK_DEV_PAGE_RANGE);
        return;
    }
    const uint8_t *half = a.cache + ((size_t)(slot / a.P) * a.Hkv + h) * record_bytes(a.P, D) +
                          part * half_bytes(a.P, D);
    const int off = slot % a.P;
    const uint32_t codes = *reinterpret_cast<const uint32_t *>(half + (e / 4) * (a.P * 16) + off * 16 + e % 4 * 4);
    const uint32_t s = half[half_scales_off(a.P, D) + off * (D / 16) + e / 2];
    uint32_t r[4];
    e2m1x8_to_f16(codes, r[0], r[1], r[2], r[3]);
    const uint32_t sf = scale_f16x2<0>(s);
    const float g = part ? a.v_scale : a.k_scale;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t m = mul_f16x2(r[i], sf);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&m));
        v[2 * i] = f.x * g;
        v[2 * i + 1] = f.y * g;
    }
    store8(static_cast<T *>(part ? a.v_out : a.k_out) + ((size_t)t * a.Hkv + h) * D + e * 8, v);
}

template <typename T>
cudaError_t launch_read(const ReadArgs &a, cudaStream_t st) {
    const long long n = (long long)a.T * a.Hkv * 2 * (a.D / 8);
    const unsigned grid = (unsigned)((n + 255) / 256);
    if (a.D == 128)
        cache_read_kernel<T, 128><<<grid, 256, 0, st>>>(a);
    else
        cache_read_kernel<T, 64><<<grid, 256, 0, st>>>(a);
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
