// cache.cuh -- the paged 4-bit key/value cache of the target pass: record
// layout, the two number formats, and the launchers of its kernels.
//
// A page holds P consecutive tokens of one request.  The record of a page and
// head is one contiguous run of R = P * D * 9 / 8 bytes, so a single bulk copy
// brings all that attention needs of it:
//   K codes [D/32][P][16 B] | K scales [P][D/16 B] | V codes | V scales.
// A 16-byte piece of codes is 32 dims of one token (byte j: dims 2j and 2j+1,
// low nibble first, e2m1); pieces of one 32-dim chunk lie token after token,
// so the 32 lanes of a warp, one token each, read 512 consecutive bytes.  A
// scale byte is the e4m3 scale of 16 dims.  A value is code * scale * g with
// the caller's g (k_scale or v_scale); code * scale has at most 6 significant
// bits and lies in [2^-10, 2880], so f16 holds it exactly.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "kernels.cuh"

namespace dspark {

inline bool page_ok(int P) { return P == 16 || P == 32 || P == 64 || P == 128; }
inline bool cache_dim_ok(int D) { return D == 64 || D == 128; }
__host__ __device__ inline int record_bytes(int P, int D) { return P * D / 8 * 9; }

// Offsets inside one half (K or V) of a record.
__host__ __device__ inline int half_scales_off(int P, int D) { return P * D / 2; }
__host__ __device__ inline int half_bytes(int P, int D) { return P * D / 16 * 9; }

// Four bytes of codes -> eight f16 values (each pair: low nibble, high nibble).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t codes, uint32_t &r0, uint32_t &r1, uint32_t &r2,
                                              uint32_t &r3) {
    asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\tmov.b32 {t0, t1, t2, t3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, t0;\n\tcvt.rn.f16x2.e2m1x2 %1, t1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, t2;\n\tcvt.rn.f16x2.e2m1x2 %3, t3;\n\t}"
        : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
        : "r"(codes));
}
// Byte i (0..3) of a word of scales -> the scale in both halves of an f16x2.
// The seven bits of an e4m3 magnitude, moved up by 7, are the f16 of
// scale * 2^-8 (subnormals included); every bit pattern gives a finite value
// (0x7f, e4m3's NaN, reads as 480), so bytes of tokens that were never
// written cannot bring a NaN into a masked place.
template <int I>
__device__ __forceinline__ uint32_t scale_f16x2(uint32_t scales) {
    const uint32_t b = __byte_perm(scales, 0, I | 4 << 4 | I << 8 | 4 << 12);
    const uint32_t h = (b & 0x007f007fu) << 7;
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&h), __half2half2(__ushort_as_half(0x5c00)));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// The dynamic shared memory limit of a kernel, set once per device (the call
// costs about as much as a launch).  `done`: one word per kernel, a bit per
// device; setting it twice does no harm.
inline cudaError_t allow_smem(const void *kernel, size_t bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// ------------------------------------------------------------------ plan
struct PlanArgs {
    const int32_t *ctx, *ell;
    int B, G, P, max_pages, n_pages;
    int32_t *table, *held;
    const int32_t *free_list;
    int32_t *free_count;
    WsHeader *hdr;
    int32_t *q_start, *kv_len, *slot, *pos;
    int T;              // rows of slot and pos
    int32_t *ell_out;   // may be ell, or null
};
struct CommitArgs {
    const int32_t *ctx, *q_start, *nout, *done;
    int B, P, max_pages, n_pages;
    int32_t *table, *held, *free_list, *free_count;
    WsHeader *hdr;
    int32_t *ctx_out;
    // A round's results, cleared where a request has no rows (null: left alone).
    int32_t *nout_rw, *acc, *tokens;
    int G;
};
cudaError_t launch_cache_plan(const PlanArgs &a, cudaStream_t st);
cudaError_t launch_cache_commit(const CommitArgs &a, cudaStream_t st);

// -------------------------------------------------- norm, rotation, write
struct NormArgs {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;   // elements between tokens
    const void *wq, *wk;
    float eps;
    const int32_t *pos;
    const float *inv_freq;
    int rot, interleaved;
    const int32_t *n_rows;
    int T, Hq, Hkv, D, dtype;
    void *q_out, *k_out;
    uint8_t *cache;
    const int32_t *slot;
    int P, n_pages;
    float k_scale, v_scale;
    WsHeader *hdr;
};
cudaError_t launch_qk_norm_rope(const NormArgs &a, cudaStream_t st);

struct ReadArgs {
    const uint8_t *cache;
    const int32_t *slot;
    int T, Hkv, D, P, n_pages, dtype;
    float k_scale, v_scale;
    void *k_out, *v_out;
    WsHeader *hdr;
};
cudaError_t launch_cache_read(const ReadArgs &a, cudaStream_t st);

// -------------------------------------------------------------- attention
struct AttnArgs {
    const __nv_bfloat16 *q;
    long long q_stride;
    const uint8_t *cache;
    const int32_t *table, *q_start, *kv_len;
    int B, T, Hq, Hkv, group, D, P, max_pages, n_pages, window;
    float qk_mul;    // softmax scale * k_scale * log2(e)
    float v_mul;     // v_scale
    __nv_bfloat16 *out;
    WsHeader *hdr;
    int32_t *desc;   // per CTA: the item it leaves unfinished
    float2 *part_ml;
    float *part_o;
    uint32_t polls;   // bound of every wait
};
size_t attention_ws_bytes(int D);
// The most work a call may bring, in the kernel's units (at most 16 a tile of
// 128 keys, 70 an item of up to 48 rows): positions inside a CTA's share are
// 32 bits, and a share is 1/148 of this.  (About two minutes of a GPU.)
inline bool attention_work_fits(int B, int T, int Hkv, int group, int P, int max_pages) {
    const double items = (double)Hkv * ((double)B + (double)T * group / 48.0 + 1.0);
    return items * (16.0 * ((double)max_pages * P / 128.0 + 2.0) + 70.0) < 0x1p38;
}
cudaError_t launch_cache_attention(AttnArgs a, void *ws, cudaStream_t st);

}  // namespace dspark
