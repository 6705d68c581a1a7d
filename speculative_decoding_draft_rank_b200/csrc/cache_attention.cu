// cache_attention.cu -- attention of the target pass over the paged 4-bit
// cache (tcgen05 / TMEM / cp.async).
//
// For query row r (token j of request b, head hq; its key head h = hq / group)
// at position p_r = kv_len[b] - n_b + j, over the keys i it may see
// (max(0, p_r - window + 1) <= i <= p_r):
//   x_i = qk_mul * <q_r, k_i>,  o_r = sum_i 2^(x_i - m) v_i / sum_i 2^(x_i - m).
//
// All rows of one request and key head (n_b * group, in equal blocks of at
// most 48) share one pass over its keys: an item.  Items are cut into tiles of
// 128 keys, the costs of all tiles are laid end to end, and every CTA takes an
// equal run of them, so ragged lengths and single long requests load the
// machine evenly.  An item that a CTA does not finish leaves (m, sum, o) in
// the workspace, and a second kernel joins its parts in a fixed order.
//
// Keys are the M = 128 side of both products, so that a tile costs little
// more for 48 query rows than for one (measured: an MMA with M = 128 and both
// operands in shared memory takes 39 cycles for 16 columns and 48 for 64; with
// A in TMEM 9 and 32):
//   S^T [keys x rows] = K Q^T      A = K in TMEM, B = Q in shared memory
//   O^T [D x rows]   += V^T P^T    A = V in shared memory, B = P
//   L   [.. x rows]  += 1 P^T      A = ones in TMEM: the softmax sums, of the
//                                  rounded P that the products use
// Three groups of four warps take the tiles in turn, and a group does all of
// a tile's arithmetic, a thread per key: its K codes into f16 in TMEM (a tile
// of its own ahead, so that the scores are there when it needs them), the
// probabilities of all rows, its V codes into f16 in shared memory; the group
// that ends an item writes its result.  So a tile costs a warp six waits, and
// while one group waits the others work.  (With a role per step -- keys,
// values, softmax in 24 warps -- waits and hand-overs were half of all
// instructions.)  Four more warps:
//   12  pages: the tiles' record addresses from the block table, ahead of use
//   13  issues the score MMAs
//   14  issues the MMAs with the values and the ones
//   15  queries of the next item, while this one runs
// An issuing thread stands still while its MMAs queue, and a wait costs it
// some hundred cycles, so the two products have a thread each.
// A thread copies the codes of its own key with cp.async, one own tile ahead,
// so no barrier stands between copy and use.  (A producer warp with two bulk
// copies per page took 2200 cycles a tile: it was what bounded the kernel.)
// P is 2^7 times exp2 of the scaled score minus a running maximum that is only
// raised (and O, L rescaled) when a score passes it by more than 8.  So P is at
// most 2^15; f16 keeps 11 bits of it down to 2^-21 of the maximum, then steps
// of 2^-31, and drops a key below 2^-32 (half a step) from both sums: n such
// keys lose less than n * 2^-32 of the row.  K and V are exact in f16.  Q is
// scaled by a power of two per row to [2^14, 2^15) (rows above 2^-86); its
// elements are exact down to 2^-31 of the row's largest, and smaller ones off
// by 2^-39 of it at most.  So P's rounding is the only one that counts before
// the output's.
//
// Measured: 256 requests of up to 6 tokens over 4096, 64 heads over 8, 350 us;
// 4 requests over 131072, 32 heads over 8, 136 to 170 (by the lengths drawn);
// 128 requests of up to 17 tokens, window 128, 55; one token 16.
// From a capture of the first (44 thousand tiles of 18 KB): 2150 cycles a CTA
// and tile, changes of items among them, where HBM would need 800; 4200 warp
// instructions and 820 wavefronts of shared-memory loads and stores a tile
// (the tensor core's reads of V, P and Q come on top).  Schedulers issue in
// 54 % of the cycles, the tensor pipe is busy in 22 %, DRAM 27 %: sixteen warps
// of 128 registers are all that an SM holds, and they wait for memory, shared
// memory and instructions in turn.  With a window the changes of items are
// most of the time: two tiles of 13 units an item against 70 for the change.
// The code has to stay small: with slow paths and unrolled loops laid out
// differently, and nothing else changed, the same case took 347 to 511 us.
// Every wait is bounded: on expiry the roles run on without waiting, nothing
// more is copied or multiplied, and the status word says so.
#include <climits>

#include "cache.cuh"
#include "tc.cuh"

namespace dspark {

namespace {

using namespace tc;

constexpr int kTile = 128;        // keys per tile
constexpr int kRows = 48;         // query rows per item (six tokens of groups of eight)
constexpr int kGroups = 3;        // groups of four warps: tiles under way
constexpr int kRing = 4;          // buffers of scores and of probabilities: one more, so that a group need not
                                  // wait for its last tile's products
constexpr int kAhead = 16;        // tiles whose pages are known
constexpr int kWarpLoad = 4 * kGroups, kWarpQk = kWarpLoad + 1, kWarpPv = kWarpLoad + 2;   // the last warp: queries
constexpr int kThreads = (kWarpLoad + 4) * 32;
constexpr int kMaxCtas = 160;
constexpr long long kWaitBudget = 4000000000LL;
constexpr float kLift = 7.f;      // log2 of P at the running maximum
constexpr float kRaise = 15.f;    // and of the largest P before the maximum is raised
constexpr int kDescInts = 8;      // CTAs that go on with the item, q0, r0, nr, h

// TMEM columns.
constexpr int kColK = 0, kColS = 192, kColO = 384, kColL = 432, kColOne = 480;

template <int D>
struct Lay {
    static constexpr int kVBytes = kTile * D * 2;
    static constexpr int kPBytes = kTile * 128;         // a 128-byte row per key
    static constexpr int kQBytes = kRows * D * 2;
    static constexpr int kHalf = kTile * D / 16 * 9;     // one tile's K (or V) codes [D/32][128][16], then scales
    static constexpr int v = 0;
    static constexpr int p = v + 2 * kVBytes;
    static constexpr int q = p + kRing * kPBytes;
    static constexpr int raw = q + 2 * kQBytes;           // per group: K half, V half
    static constexpr int misc = raw + kGroups * 2 * kHalf;
};

// What the softmax knows of an item's rows, two rows to an entry of `mul_m`:
// the multipliers of their raw scores and their negated running maxima, which
// are kept kLift low throughout, in the parts for the join too.
struct Rows {
    float4 mul_m[kRows / 2];
    int2 lim[kRows];         // visible keys [x, y)
    int orow[kRows];         // output row (token * Hq + head)
    int nr, base, t0, t1, nt, q0, r0, h, last;   // the piece: rows, first key, its tiles of the item's nt, where it
                                                // belongs; the CTA of the item's last tile
    int version;             // times the maxima were raised
    __device__ __forceinline__ float &mul(int r) { return reinterpret_cast<float *>(&mul_m[r / 2])[r & 1]; }
    __device__ __forceinline__ float &neg_max(int r) { return reinterpret_cast<float *>(&mul_m[r / 2])[2 + (r & 1)]; }
};
struct Misc {
    Rows rows[2];
    float fac[kGroups][kRows];
    float wmax[kGroups][4][kRows];
    unsigned long long rec[kAhead][8];   // a tile's page records (0: no keys there)
    uint64_t rec_full[kAhead], rec_empty[kAhead];
    // Per group: its keys are in TMEM; its scores are there; it has had its turn at the maxima and O.
    uint64_t k_full[kGroups], s_full[kGroups], turn[kGroups];
    // Per tile of the ring: P and V are in shared memory; the products are done.
    uint64_t vp_full[kRing], pv_done[kRing];
    uint64_t q_full[2], q_empty[2], m_full[2], drain[2];   // m_full: the piece's first maxima are set
    uint32_t tmem;
    int abort;
    long long scan[16];
    int scan_t[16];
};

struct Req {
    int q0, n, L;
};

__device__ __forceinline__ Req load_req(const AttnArgs &a, int b) {
    Req r;
    const int s0 = min(max(__ldg(a.q_start + b), 0), a.T), s1 = min(max(__ldg(a.q_start + b + 1), s0), a.T);
    r.q0 = s0;
    r.n = s1 - s0;
    r.L = min(max(__ldg(a.kv_len + b), 0), a.max_pages * a.P);
    return r;
}

// Row block rb of a request: its rows in equal blocks of at most kRows; rows
// [r0, r0 + nr), keys [base, hi) in tiles.
struct Block {
    int r0, nr, base, hi, nt;
};
__device__ __forceinline__ int row_blocks(const AttnArgs &a, const Req &q) { return (q.n * a.group + kRows - 1) / kRows; }
__device__ __forceinline__ Block row_block(const AttnArgs &a, const Req &q, int rb) {
    Block k;
    const int rows = q.n * a.group, nb = max(1, row_blocks(a, q));
    k.r0 = (int)((long long)rows * rb / nb);
    k.nr = (int)((long long)rows * (rb + 1) / nb) - k.r0;
    const int jf = k.r0 / a.group, jl = (k.r0 + k.nr - 1) / a.group;
    k.hi = max(0, q.L - q.n + jl + 1);
    const int lo = a.window > 0 ? max(0, q.L - q.n + jf - a.window + 1) : 0;
    k.base = lo / a.P * a.P;
    k.nt = max(1, (k.hi - k.base + kTile - 1) / kTile);   // a row block without keys still writes zeros
    return k;
}

// What a tile costs, and what changing to another item does (its last
// products and result; the first maxima), in units of about 125 cycles:
// measured 1600 cycles a tile up to 32 rows, 2000 for 48 rows, 9000 an item
// in a run of some 20 tiles each.  CTAs get equal costs rather than equal tiles.
__device__ __forceinline__ int tile_cost(const Block &k) { return k.nr <= 32 ? 13 : 16; }
constexpr int kItemCost = 70, kMinQuota = 16;   // a quota holds the start of at least one tile
constexpr long long kRefused = 1LL << 50;
__device__ __forceinline__ int item_cost(const Block &k) { return k.nt * tile_cost(k) + kItemCost; }

// x / d, short where x is: 64-bit divisions take some two hundred cycles.
__device__ __forceinline__ unsigned long long divide(unsigned long long x, uint32_t d) {
    return x >> 32 == 0 ? (uint32_t)x / d : x / d;
}

// The item in which position `pos` of the batch's costs lies, its first tile
// that starts there or later (nt: none), and the tiles of the batch before that.
struct Spot {
    int b, rb, h, t, tiles;
    uint32_t start;                  // position of the item, from `pos`
    Req q;
    Block k;
};
__device__ __forceinline__ Spot spot_at(const AttnArgs &a, const long long *cost, const int *tiles, long long pos) {
    Spot p;
    int lo = 0, hi = a.B;                // the request: cost[b] <= pos < cost[b + 1]
#pragma unroll 1
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cost[mid] <= pos) lo = mid; else hi = mid;
    }
    p.b = lo;
    p.q = load_req(a, lo);
    unsigned long long rest = pos - cost[lo];
    int c = 0;
    p.tiles = tiles[lo];
#pragma unroll 1
    for (p.rb = 0;; ++p.rb) {
        p.k = row_block(a, p.q, p.rb);
        c = item_cost(p.k);
        const unsigned long long all = (unsigned long long)c * a.Hkv;
        if (rest < all) break;
        rest -= all;
        p.tiles += p.k.nt * a.Hkv;
    }
    p.h = (int)divide(rest, c);
    const int off = (int)(rest - (unsigned long long)p.h * c);
    p.start = 0u - off;
    const int w = tile_cost(p.k);
    p.t = min(p.k.nt, (off + w - 1) / w);
    p.tiles += p.h * p.k.nt + p.t;
    return p;
}

// This CTA's run of tiles, piece by piece (a piece: consecutive tiles of one item).
struct Walk {
    const AttnArgs &a;
    int left;                // tiles left in the run
    int b, rb, h, t0, t1;
    uint32_t start;          // position of the item, from that of the run (below 2^31 + 2^28 at its last tile)
    Req q;
    Block k;
    __device__ __forceinline__ void next_item() {
        start += item_cost(k);
        if (++h == a.Hkv) {
            h = 0;
            if (rb + 1 < row_blocks(a, q)) {
                ++rb;
            } else {
                rb = 0;
#pragma unroll 1
                do q = load_req(a, b = min(b + 1, a.B - 1)); while (q.n == 0 && b + 1 < a.B);
            }
            k = row_block(a, q, rb);
        }
        t0 = 0;
    }
    __device__ __forceinline__ Walk(const AttnArgs &args, const Spot &p, int tiles) : a(args), left(tiles) {
        b = p.b;
        rb = p.rb;
        h = p.h;
        t0 = p.t;
        start = p.start;
        q = p.q;
        k = p.k;
        if (t0 == k.nt) next_item();
        t1 = min(k.nt, t0 + left);
    }
    __device__ __forceinline__ bool next() {   // false: the run is done
        left -= t1 - t0;
        if (left <= 0) return false;
        next_item();
        t1 = min(k.nt, left);
        return true;
    }
};

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// 16 columns of this thread's lane; the values are there after tmem_ld_wait().
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ float rcp(float x) {   // within 1 ulp
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float warp_max_f32(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// Bounded waits.  The roles' code together has to fit the instruction cache,
// so a wait is one short polling loop, and its bound a number of polls: an
// unsatisfied try_wait suspends its warp and returns after some 7800 cycles
// (measured; with or without a hint), so the default budget ends a wait in
// about four seconds.  Returns false when it ran out, here or in another role.
constexpr int kPollCycles = 4000;
__device__ __forceinline__ bool wait1(uint64_t *bar, uint32_t parity, volatile int *abort, uint32_t polls) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n, a;\n\tmov.u32 n, %4;\nPOLL%=:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE%=;\n\t"
        "ld.volatile.shared.u32 a, [%3];\n\tsub.u32 n, n, 1;\n\tsetp.ne.u32 q, n, 0;\n\t"
        "setp.eq.and.u32 q, a, 0, q;\n\t@q bra POLL%=;\n\tst.volatile.shared.u32 [%3], 1;\nDONE%=:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(smem_u32(const_cast<int *>(abort))), "r"(polls)
        : "memory");
    return ok != 0;
}
// The same for a whole warp, converged again afterwards.
__device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity, volatile int *abort, uint32_t polls) {
    wait1(bar, parity, abort, polls);
    __syncwarp();
}
// The 128 threads of softmax group sg.
__device__ __forceinline__ void soft_sync(int sg) {
    __syncwarp();
    asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(sg + 1) : "memory");
}
__device__ __forceinline__ bool soft_any(int sg, bool v) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbarrier.cta.red.or.aligned.pred p, %2, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(sg + 1)
        : "memory");
    return r != 0;
}
// Shared-memory operands in 128-byte swizzled rows, eight rows 1024 bytes
// apart.  The descriptor's upper word is the same for all of them; the lower
// word is the address and, for operands whose 64-element blocks of the row
// dimension lie `lbo` bytes apart (D-major values, row-major probabilities),
// that distance.  Adding bytes / 16 to the lower word moves the address.
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
    return (saddr >> 4 & 0x3FFF) | (lbo >> 4) << 16;
}
template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(kDescHi), "r"(idesc), "n"(ACC ? 1 : 0)
        : "memory");
}
template <bool ACC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(kDescHi), "r"(idesc), "n"(ACC ? 1 : 0)
        : "memory");
}
// The products of one tile with the values and the ones.
template <bool FIRST>
__device__ __forceinline__ void mma_values(uint32_t tm, uint32_t v_lo, uint32_t p_lo, uint32_t id_o, uint32_t id_l) {
    mma_ss<!FIRST>(tm + kColO, v_lo, p_lo, id_o);
    mma_ts<!FIRST>(tm + kColL, tm + kColOne, p_lo, id_l);
#pragma unroll
    for (int kk = 1; kk < kTile / 16; ++kk) {
        mma_ss<true>(tm + kColO, v_lo + kk * 128, p_lo + kk * 128, id_o);
        mma_ts<true>(tm + kColL, tm + kColOne, p_lo + kk * 128, id_l);
    }
}
// kind::f16 with f16 operands and fp32 sums, M = 128.
__device__ __forceinline__ uint32_t idesc_f16(int N, bool a_mn, bool b_mn) {
    return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void cp_async16(uint8_t *dst, const uint8_t *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
template <int BYTES>   // 4 or 8
__device__ __forceinline__ void cp_async_scales(uint8_t *dst, const uint8_t *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}
// 16 bytes of codes and two scales -> 16 f16x2.
__device__ __forceinline__ void unpack32(const uint4 c, uint32_t s0, uint32_t s1, uint32_t (&r)[16]) {
    e2m1x8_to_f16(c.x, r[0], r[1], r[2], r[3]);
    e2m1x8_to_f16(c.y, r[4], r[5], r[6], r[7]);
    e2m1x8_to_f16(c.z, r[8], r[9], r[10], r[11]);
    e2m1x8_to_f16(c.w, r[12], r[13], r[14], r[15]);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = mul_f16x2(r[i], s0);
#pragma unroll
    for (int i = 8; i < 16; ++i) r[i] = mul_f16x2(r[i], s1);
}

// The tile's probabilities of 16 * C rows from r0 for this thread's key: scores from
// TMEM, 2^(score - maximum) in f16 to the P operand's row of the key.  Returns
// the largest exponent.
template <int C, bool MASKED>
__device__ __forceinline__ float probs(uint32_t ts, const Rows &rw, uint8_t *prow, int r0, int key, int me) {
    uint32_t s[C][16];
#pragma unroll
    for (int c = 0; c < C; ++c) tmem_ld16(ts + r0 + 16 * c, s[c]);
    tmem_ld_wait();
    float top = -INFINITY;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        uint32_t ph[8];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float4 mm = rw.mul_m[r0 / 2 + 8 * c + i / 2];
            float2 x = fma2(make_float2(__uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1])),
                            make_float2(mm.x, mm.y), make_float2(mm.z, mm.w));
            if (MASKED) {
                const int4 l = *reinterpret_cast<const int4 *>(&rw.lim[r0 + 16 * c + i]);
                if (me < l.x || me >= l.y) x.x = -INFINITY;
                if (me < l.z || me >= l.w) x.y = -INFINITY;
            }
            top = max3(top, x.x, x.y);
            const __half2 h2 = __floats2half2_rn(fast_exp2(x.x), fast_exp2(x.y));
            ph[i / 2] = *reinterpret_cast<const uint32_t *>(&h2);
        }
        *reinterpret_cast<uint4 *>(prow + (((r0 / 8 + 2 * c) ^ (key & 7)) * 16)) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
        *reinterpret_cast<uint4 *>(prow + (((r0 / 8 + 2 * c + 1) ^ (key & 7)) * 16)) = make_uint4(ph[4], ph[5], ph[6], ph[7]);
    }
    return top;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cache_attention_kernel(const AttnArgs a) {
    using Y = Lay<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);   // still known to be shared memory
    Misc &ms = *reinterpret_cast<Misc *>(sm + Y::misc);
    // In the probabilities' place: read for the last time before the roles begin.
    long long *prefix = reinterpret_cast<long long *>(sm + Y::p);   // costs and tiles before a request
    int *before_t = reinterpret_cast<int *>(prefix + 4096);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // Tiles of every request, and their prefix: thread t sums a run of requests.
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    long long sum = 0;
    int sum_t = 0;   // the batch's tiles may pass 32 bits; only differences within a CTA's run are used
    bool bad = false;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        const Req q = load_req(a, b);
        bad |= __ldg(a.kv_len + b) != q.L || __ldg(a.q_start + b) != q.q0 || __ldg(a.q_start + b + 1) != q.q0 + q.n;
        prefix[b] = sum;
        before_t[b] = sum_t;
#pragma unroll 1
        for (int rb = 0; rb < row_blocks(a, q); ++rb) {
            const Block k = row_block(a, q, rb);
            sum += (long long)item_cost(k) * a.Hkv;
            sum_t += k.nt * a.Hkv;
        }
        if (__ldg(a.q_start + b + 1) < __ldg(a.q_start + b)) sum = kRefused;
    }
    if (bad && blockIdx.x == 0) flag_status(a.hdr, DSPARK_DEV_LENGTH_RANGE);
    long long inc = sum;
    int inc_t = sum_t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        const int z = __shfl_up_sync(0xffffffffu, inc_t, o);
        if (lane >= o) {
            inc += y;
            inc_t += z;
        }
    }
    if (lane == 31) {
        ms.scan[warp] = inc;
        ms.scan_t[warp] = inc_t;
    }
    if (tid == 0) {
        ms.abort = 0;
#pragma unroll 1
        for (int i = 0; i < kAhead; ++i) {
            mbar_init(&ms.rec_full[i], 1);
            mbar_init(&ms.rec_empty[i], 4);
        }
        for (int i = 0; i < kGroups; ++i) {
            mbar_init(&ms.k_full[i], 4);
            mbar_init(&ms.s_full[i], 1);
            mbar_init(&ms.turn[i], 4);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&ms.vp_full[i], 4);
            mbar_init(&ms.pv_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms.q_full[i], 1);
            mbar_init(&ms.q_empty[i], 4 * kGroups);
            mbar_init(&ms.m_full[i], 4);
            mbar_init(&ms.drain[i], 1);
        }
        fence_barrier_init();
    }
    __syncthreads();
    long long before = inc - sum, total = 0;
    int before_tiles = inc_t - sum_t, all_tiles = 0;
#pragma unroll 1
    for (int w = 0; w < kThreads / 32; ++w) {
        const long long x = ms.scan[w];
        const int y = ms.scan_t[w];
        if (w < warp) {
            before += x;
            before_tiles += y;
        }
        total += x;
        all_tiles += y;
    }
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        prefix[b] += before;
        before_t[b] += before_tiles;
    }
    __syncthreads();
    // Offsets that fall (requests would share rows), or more work than the
    // positions of a run can count: nothing is done.
    const bool refused = total > (long long)gridDim.x * INT_MAX;
    if (refused && tid == 0 && blockIdx.x == 0) flag_status(a.hdr, DSPARK_DEV_LENGTH_RANGE);
    const int quota = refused ? INT_MAX : max(kMinQuota, (int)divide(total + gridDim.x - 1, gridDim.x));
    const long long w0 = (long long)blockIdx.x * quota, w1 = w0 + quota;
    Spot spot = {};
    int tiles = 0;
    if (w0 < total && !refused) {
        spot = spot_at(a, prefix, before_t, w0);
        tiles = (w1 < total ? spot_at(a, prefix, before_t, w1).tiles : all_tiles) - spot.tiles;
    }
    if (tiles <= 0) {   // the whole CTA: no work, nothing left unfinished
        if (tid == 0) a.desc[blockIdx.x * kDescInts] = 0;
        return;
    }
    if (tid == 0) a.desc[blockIdx.x * kDescInts] = 0;   // an unfinished last item replaces it below
    if (warp == 0) {
        tmem_alloc(&ms.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = ms.tmem;
    volatile int *abort = &ms.abort;
    int g = 0;   // tiles done by this role

    if (warp < 4 * kGroups) {
        // ----------------------------------------------- keys, softmax, values
        // Group sg takes the tiles g with g % kGroups == sg.  The groups share
        // the rows' maxima and O: tile g's probabilities are given to the
        // products only after tile g - 1 had its turn, and computed anew in the
        // rare case that its turn raised a maximum.
        const int key = tid & 127, sw = warp & 3, sg = warp >> 2;
        const uint32_t lane_base = (uint32_t)(sw * 32) << 16;
        // A thread copies the codes and scales of its own key, one own tile
        // ahead, so it waits for its own copies only.
        uint8_t *kraw = sm + Y::raw + sg * 2 * Y::kHalf + key * 16, *vraw = kraw + Y::kHalf;
        constexpr int kScaleAt = kTile * D / 2;
        uint8_t *kscale = kraw + kScaleAt - key * 16 + key * (D / 16), *vscale = kscale + Y::kHalf;
        const int off = key % a.P, hb = half_bytes(a.P, D), soff = half_scales_off(a.P, D) + off * (D / 16);
        auto find = [&](int x) -> unsigned long long {      // this key's record in tile x
            unsigned long long r = 0;
            if (x < tiles) {
                // Only what the producer has published is an address.
                if (wait1(&ms.rec_full[x % kAhead], (x / kAhead) & 1, abort, a.polls)) r = ms.rec[x % kAhead][key / a.P];
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.rec_empty[x % kAhead]);
            }
            return r;
        };
        auto copy = [&](unsigned long long from, uint8_t *codes, uint8_t *scales) {
            if (from != 0) {
                const uint8_t *p = reinterpret_cast<const uint8_t *>(from) + off * 16;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) cp_async16(codes + c * (kTile * 16), p + c * a.P * 16);
                cp_async_scales<D / 16>(scales, reinterpret_cast<const uint8_t *>(from) + soff);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            __syncwarp();   // lanes whose pages end differ: whole warps for the tensor-memory instructions behind
        };
        // The keys go into the group's TMEM buffer one own tile ahead, so the
        // scores are there when the tile's turn comes.
        auto unpack_keys = [&]() {
#pragma unroll 1
            for (int c = 0; c < D / 32; c += 2) {   // 64 dims: two pieces of codes, one word of scales
                const uint32_t sc = *reinterpret_cast<const uint32_t *>(kscale + c * 2);
                const uint4 c0 = *reinterpret_cast<const uint4 *>(kraw + c * (kTile * 16));
                const uint4 c1 = *reinterpret_cast<const uint4 *>(kraw + (c + 1) * (kTile * 16));
                uint32_t r[16];
                unpack32(c0, scale_f16x2<0>(sc), scale_f16x2<1>(sc), r);
                tmem_st16(tm + lane_base + kColK + sg * 64 + c * 16, r);
                unpack32(c1, scale_f16x2<2>(sc), scale_f16x2<3>(sc), r);
                tmem_st16(tm + lane_base + kColK + sg * 64 + c * 16 + 16, r);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.k_full[sg]);
        };
        unsigned long long rec = find(sg), next = 0;   // records of this tile; of the own tile behind it
        copy(rec, kraw, kscale);
        copy(rec ? rec + hb : 0, vraw, vscale);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        if (sg == 0) {   // the ones: before this group's first keys, whose wait for stores covers them
            uint32_t one[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) one[i] = 0x3c003c00u;
            __syncwarp();
            tmem_st16(tm + lane_base + kColOne, one);
        }
        if (sg < tiles) unpack_keys();
        next = find(sg + kGroups);
        copy(next, kraw, kscale);
        // The group of tile g - 1, and its parity when this group's is even.
        const int p1 = (sg + kGroups - 1) % kGroups;
        const uint32_t x1 = sg < 1;
        uint32_t ph = 0;       // parity of this group's barriers for its current tile
        int end = 0;           // the piece's tiles are [.., end) of the run
        g = sg;
#pragma unroll 1
        for (int piece = 0; end < tiles; ++piece) {
            Rows &rw = ms.rows[piece & 1];
            wait(&ms.q_full[piece & 1], (piece >> 1) & 1, abort, a.polls);
            if (soft_any(sg, *abort != 0)) break;   // the piece may not be there: the four warps leave together
            const int nr = rw.nr, N = (nr + 15) / 16 * 16, t0 = rw.t0, t1 = rw.t1, g0 = end;
            // Tiles that every row sees whole need no mask.
            const int all_hi = rw.lim[0].y, all_lo = rw.lim[nr - 1].x;
            int version = 0;
            end += t1 - t0;
#pragma unroll 1
            for (; g < end; g += kGroups) {
                const int t = t0 + g - g0;
                const int ri = g % kRing, kpos = rw.base + t * kTile, me = kpos + key;
                const uint32_t rp = (g / kRing) & 1;           // parity of the ring's barriers for this tile
                const uint32_t ts = tm + lane_base + kColS + ri * kRows;
                uint8_t *prow = sm + Y::p + ri * Y::kPBytes + key * 128;
                const bool masked = kpos + kTile > all_hi || kpos < all_lo;
                // Probabilities.
                wait(&ms.pv_done[ri], rp ^ 1, abort, a.polls);      // of tile g - kRing: it read this P buffer
                wait(&ms.s_full[sg], ph, abort, a.polls);
                tc_fence_after();
                if (t == t0) {
                    // The rows' first maxima: a quarter of the rows a warp, over
                    // its own 32 keys.  Any key's score will do -- P of the key
                    // that set it is 1, and a tile that passes it by too much raises it.
#pragma unroll 1
                    for (int r0 = sw * (N / 4); r0 < (sw + 1) * (N / 4); r0 += 4) {
                        __syncwarp();
                        uint32_t s[4];
                        tmem_ld4(ts + r0, s);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float x = __uint_as_float(s[i]) * rw.mul(r0 + i);
                            if (masked) {
                                const int2 l = rw.lim[r0 + i];
                                if (me < l.x || me >= l.y) x = -INFINITY;
                            }
                            x = warp_max_f32(x);
                            if (lane == 0) rw.neg_max(r0 + i) = x == x ? kLift - x : INFINITY;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.m_full[piece & 1]);
                }
                if (t < t0 + kGroups) wait(&ms.m_full[piece & 1], (piece >> 1) & 1, abort, a.polls);
                bool raise = false, mine = t == t0, have_v = false;   // mine: tile g - 1 had its turn (or is another item's)
                for (;;) {
                    if (raise) {
                        // New maxima over the tile: a warp's 32 keys, then the four warps.
#pragma unroll 1
                        for (int r0 = 0; r0 < N; r0 += 4) {
                            __syncwarp();
                            uint32_t s[4];
                            tmem_ld4(ts + r0, s);
                            tmem_ld_wait();
                            float x[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                x[i] = __uint_as_float(s[i]) * rw.mul(r0 + i);
                                if (masked) {
                                    const int2 l = rw.lim[r0 + i];
                                    if (me < l.x || me >= l.y) x[i] = -INFINITY;
                                }
                                x[i] = warp_max_f32(x[i]);
                            }
                            if (lane == 0)
                                *reinterpret_cast<float4 *>(&ms.wmax[sg][sw][r0]) = make_float4(x[0], x[1], x[2], x[3]);
                        }
                        soft_sync(sg);
                        if (key < N) {
                            float &neg = rw.neg_max(key);
                            const float old = -neg;
                            const float top = fmaxf(fmaxf(ms.wmax[sg][0][key], ms.wmax[sg][1][key]),
                                                    fmaxf(ms.wmax[sg][2][key], ms.wmax[sg][3][key]));
                            const float nm = fmaxf(top - kLift, old);
                            ms.fac[sg][key] = nm == old ? 1.f : fast_exp2(old - nm);
                            neg = -nm;
                        }
                        if (key == 0) ++rw.version;
                        ++version;
                        soft_sync(sg);
                        if (t > t0) {
                            wait(&ms.pv_done[(g - 1) % kRing], ((g - 1) / kRing) & 1, abort, a.polls);
                            tc_fence_after();
#pragma unroll 1
                            for (int r0 = 0; r0 < N; r0 += 4) {
                                uint32_t o[4], l[4];
                                tmem_ld4(tm + lane_base + kColO + r0, o);
                                tmem_ld4(tm + lane_base + kColL + r0, l);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float f = ms.fac[sg][r0 + i];
                                    o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                    l[i] = __float_as_uint(__uint_as_float(l[i]) * f);
                                }
                                tmem_st4(tm + lane_base + kColO + r0, o);
                                tmem_st4(tm + lane_base + kColL + r0, l);
                            }
                            tmem_st_wait();
                        }
                    }
                    float top = -INFINITY;
                    if (masked) {   // a piece's last tile, with a window nearly all: one code for every number of rows
#pragma unroll 1
                        for (int c = 0; c < N; c += 16)
                            top = fmaxf(top, probs<1, true>(ts, rw, prow, c, key, me));
                    } else {
                        if (N == 16) top = probs<1, false>(ts, rw, prow, 0, key, me);
                        else if (N == 32) top = probs<2, false>(ts, rw, prow, 0, key, me);
                        else top = probs<3, false>(ts, rw, prow, 0, key, me);
                    }
                    if (!have_v) {
                        have_v = true;
                        // The next own tile's keys: the scores of this tile have read the buffer.
                        // (Both copies were asked for an own tile ago.)
                        asm volatile("cp.async.wait_group 0;" ::: "memory");
                        if (g + kGroups < tiles) unpack_keys();
                        const unsigned long long after = find(g + 2 * kGroups);
                        copy(after, kraw, kscale);
                        // Values.  Their buffer was last read by the products of tile g - 2.
                        uint8_t *vrow = sm + Y::v + (g & 1) * Y::kVBytes + key * 128;
                        uint4 codes[D / 32];
                        uint32_t sc[D / 64];
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) sc[c] = *reinterpret_cast<const uint32_t *>(vscale + c * 4);
#pragma unroll
                        for (int c = 0; c < D / 32; ++c)
                            codes[c] = *reinterpret_cast<const uint4 *>(vraw + c * (kTile * 16));
                        if (g >= 2) wait(&ms.pv_done[(g - 2) % kRing], ((g - 2) / kRing) & 1, abort, a.polls);
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t r[16];
                            if (c & 1) unpack32(codes[c], scale_f16x2<2>(sc[c / 2]), scale_f16x2<3>(sc[c / 2]), r);
                            else unpack32(codes[c], scale_f16x2<0>(sc[c / 2]), scale_f16x2<1>(sc[c / 2]), r);
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                *reinterpret_cast<uint4 *>(vrow + (c / 2) * (kTile * 128) +
                                                           (((c & 1) * 4 + u) ^ (key & 7)) * 16) =
                                    make_uint4(r[4 * u], r[4 * u + 1], r[4 * u + 2], r[4 * u + 3]);
                        }
                        rec = next;
                        next = after;
                        copy(rec ? rec + hb : 0, vraw, vscale);
                    }
                    if (!mine) {
                        mine = true;
                        wait(&ms.turn[p1], ph ^ x1, abort, a.polls);
                        const int v = __shfl_sync(0xffffffffu, rw.version, 0);
                        if (v != version) {
                            version = v;
                            continue;
                        }
                    }
                    if (raise) break;                  // at most one raise a tile
                    raise = soft_any(sg, top > kRaise);
                    if (!raise) break;
                }
                if (t == t0 && g > 0) wait(&ms.turn[p1], ph ^ x1, abort, a.polls);   // the last item's O was read
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.vp_full[ri]);
                if (t + 1 == t1) {
                    // The piece's result: this thread's dim of every row.
                    wait(&ms.pv_done[ri], rp, abort, a.polls);
                    tc_fence_after();
                    const bool whole = t0 == 0 && t1 == rw.nt;
                    const int slot = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
                    if (whole) {
                        // O is read and its place given back before the results are stored.
                        uint32_t y[kRows / 2];
#pragma unroll
                        for (int c = 0; c < kRows / 16; ++c) {
                            if (c * 16 < nr) {
                                __syncwarp();
                                uint32_t o[16], l[16];
                                tmem_ld16(tm + lane_base + kColO + c * 16, o);
                                tmem_ld16(tm + lane_base + kColL + c * 16, l);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 16; i += 2) {
                                    // No visible key: the sum is 0 and so is O.
                                    const float l0 = __uint_as_float(l[i]), l1 = __uint_as_float(l[i + 1]);
                                    const float v0 = l0 == 0.f ? 0.f : rcp(l0) * a.v_mul;
                                    const float v1 = l1 == 0.f ? 0.f : rcp(l1) * a.v_mul;
                                    const __nv_bfloat162 z = __floats2bfloat162_rn(__uint_as_float(o[i]) * v0,
                                                                                   __uint_as_float(o[i + 1]) * v1);
                                    y[c * 8 + i / 2] = *reinterpret_cast<const uint32_t *>(&z);
                                }
                            }
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ms.turn[sg]);
                        if (key < D) {
                            uint16_t *out = reinterpret_cast<uint16_t *>(a.out) + key;
#pragma unroll
                            for (int r = 0; r < kRows; r += 4) {
                                if (r < nr) {
                                    const int4 w = *reinterpret_cast<const int4 *>(&rw.orow[r]);
                                    out[(long long)w.x * D] = (uint16_t)y[r / 2];
                                    if (r + 1 < nr) out[(long long)w.y * D] = (uint16_t)(y[r / 2] >> 16);
                                    if (r + 2 < nr) out[(long long)w.z * D] = (uint16_t)y[r / 2 + 1];
                                    if (r + 3 < nr) out[(long long)w.w * D] = (uint16_t)(y[r / 2 + 1] >> 16);
                                }
                            }
                        }
                    } else {
                        float *po = a.part_o + (size_t)slot * kRows * D + key;
#pragma unroll 1
                        for (int r0 = 0; r0 < nr; r0 += 4) {
                            __syncwarp();
                            uint32_t o[4], l[4];
                            tmem_ld4(tm + lane_base + kColO + r0, o);
                            tmem_ld4(tm + lane_base + kColL + r0, l);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int r = r0 + i;
                                if (r < nr && key < D) po[r * D] = __uint_as_float(o[i]);
                                if (r < nr && key == i)
                                    a.part_ml[slot * kRows + r] = make_float2(-rw.neg_max(r), __uint_as_float(l[i]));
                            }
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ms.turn[sg]);
                    }
                    if (!whole && t0 == 0 && key == 0) {
                        int32_t *d = a.desc + blockIdx.x * kDescInts;
                        d[1] = rw.q0;
                        d[2] = rw.r0;
                        d[3] = nr;
                        d[4] = rw.h;
                        d[0] = rw.last - (int)blockIdx.x;   // CTAs that go on with it
                    }
                } else {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ms.turn[sg]);
                }
                ph ^= 1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.q_empty[piece & 1]);
        }
    } else if (warp == kWarpLoad) {
        // --------------------------------------------------------- pages
        // A lane per page of a tile: its record's address, up to kAhead tiles
        // before they are used.
        const int ppt = kTile / a.P;
        const unsigned long long rec_bytes = record_bytes(a.P, D);
        Walk wk(a, spot, tiles);
#pragma unroll 1
        for (int t = wk.t0; g < tiles; ++g) {
            const int key0 = wk.k.base + t * kTile, np = min(ppt, max(0, (wk.k.hi - key0 + a.P - 1) / a.P));
            unsigned long long rec = 0;
            if (lane < np) {
                int page = __ldg(a.table + (long long)wk.b * a.max_pages + key0 / a.P + lane);
                if (page < 0 || page >= a.n_pages) {
                    flag_status(a.hdr, DSPARK_DEV_PAGE_RANGE);
                    page = 0;
                }
                rec = reinterpret_cast<unsigned long long>(a.cache) +
                      ((unsigned long long)page * a.Hkv + wk.h) * rec_bytes;
            }
            const int st = g % kAhead;
            if (!__all_sync(0xffffffffu, wait1(&ms.rec_empty[st], ((g / kAhead) & 1) ^ 1, abort, a.polls))) break;
            if (lane < 8) ms.rec[st][lane] = rec;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.rec_full[st]);
            if (++t == wk.t1 && wk.next()) t = wk.t0;
        }
    } else if (warp == kWarpQk) {
        // -------------------------------------------------------- scores
        if (elect_one()) {
            const uint32_t q0 = desc_lo(smem_u32(sm + Y::q), 16);
#pragma unroll 1
            for (int piece = 0; g < tiles; ++piece) {
                if (!wait1(&ms.q_full[piece & 1], (piece >> 1) & 1, abort, a.polls)) break;
                const Rows &rw = ms.rows[piece & 1];
                const int g_end = g + rw.t1 - rw.t0;
                const uint32_t id = idesc_f16((rw.nr + 15) / 16 * 16, false, false);
                const uint32_t q_lo = q0 + (piece & 1) * (Y::kQBytes / 16);
                bool ok = true;
#pragma unroll 1
                for (; g < g_end; ++g) {
                    const int sg = g % kGroups, ri = g % kRing;
                    // The keys are there, and the scores of tile g - kRing are done with.
                    ok = wait1(&ms.k_full[sg], (g / kGroups) & 1, abort, a.polls) &&
                         wait1(&ms.vp_full[ri], ((g / kRing) & 1) ^ 1, abort, a.polls);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t ds = tm + kColS + ri * kRows, dk = tm + kColK + sg * 64;
                    mma_ts<false>(ds, dk, q_lo, id);
#pragma unroll
                    for (int kk = 1; kk < D / 16; ++kk)
                        mma_ts<true>(ds, dk + kk * 8, q_lo + (kk / 4) * (kRows * 8) + (kk & 3) * 2, id);
                    mma_commit(&ms.s_full[sg]);
                }
                if (!ok) break;
            }
        }
    } else if (warp == kWarpPv) {
        // -------------------------------------------------------- values
        // D = 64: the second 64 rows of the value operand repeat the first (their lanes are not read).
        if (elect_one()) {
            const uint32_t v0 = desc_lo(smem_u32(sm + Y::v), D == 128 ? kTile * 128 : 0);
            const uint32_t p0 = desc_lo(smem_u32(sm + Y::p), 0);
#pragma unroll 1
            for (int piece = 0; g < tiles; ++piece) {
                if (!wait1(&ms.q_full[piece & 1], (piece >> 1) & 1, abort, a.polls)) break;
                const Rows &rw = ms.rows[piece & 1];
                const int N = (rw.nr + 15) / 16 * 16, g0 = g, g_end = g + rw.t1 - rw.t0;
                const uint32_t id_o = idesc_f16(N, true, true), id_l = idesc_f16(N, false, true);
                bool ok = true;
#pragma unroll 1
                for (; g < g_end; ++g) {
                    const int ri = g % kRing;
                    ok = wait1(&ms.vp_full[ri], (g / kRing) & 1, abort, a.polls);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t v_lo = v0 + (g & 1) * (Y::kVBytes / 16), p_lo = p0 + ri * (Y::kPBytes / 16);
                    if (g == g0)
                        mma_values<true>(tm, v_lo, p_lo, id_o, id_l);
                    else
                        mma_values<false>(tm, v_lo, p_lo, id_o, id_l);
                    mma_commit(&ms.pv_done[ri]);
                }
                if (!ok) break;
            }
        }
    } else {
        // ------------------------------------------------------- queries
        // A lane works out where rows lane and lane + 32 come from and what they
        // see; then D / 16 lanes a row, 16 dims each, scale it by a power of two
        // so that f16 holds it exactly.
        constexpr int kLanes = D / 16, kPass = 32 / kLanes, kBatch = 2;
        const int part = lane % kLanes, rsub = lane / kLanes;
        int piece = 0;
        Walk wk(a, spot, tiles);
        do {
            Rows &rw = ms.rows[piece & 1];
            uint8_t *qs = sm + Y::q + (piece & 1) * Y::kQBytes;
            const int nr = wk.k.nr, N = (nr + 15) / 16 * 16;
            wait(&ms.q_empty[piece & 1], ((piece >> 1) & 1) ^ 1, abort, a.polls);
            const __nv_bfloat16 *src[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int r = lane + 32 * u, gr = wk.k.r0 + min(r, nr - 1), j = gr / a.group;
                const int hd = wk.h * a.group + gr - j * a.group, pos = wk.q.L - wk.q.n + j;
                src[u] = a.q + (long long)(wk.q.q0 + j) * a.q_stride + hd * D;
                if (r >= kRows) continue;
                rw.lim[r] = r < nr ? make_int2(a.window > 0 ? max(0, pos - a.window + 1) : 0, pos + 1)
                                   : make_int2(0, 0);
                rw.orow[r] = (wk.q.q0 + j) * a.Hq + hd;
            }
            if (lane == 0) {
                rw.nr = nr;
                rw.base = wk.k.base;
                rw.t0 = wk.t0;
                rw.t1 = wk.t1;
                rw.nt = wk.k.nt;
                rw.q0 = wk.q.q0;
                rw.r0 = wk.k.r0;
                rw.h = wk.h;
                rw.last = blockIdx.x + (wk.start + (uint32_t)((wk.k.nt - 1) * tile_cost(wk.k))) / (uint32_t)quota;
                rw.version = 0;
            }
#pragma unroll 1
            for (int rr = 0; rr < N; rr += kPass * kBatch) {   // N is a multiple of 16, as is the step (or half of it)
                uint4 w[kBatch][2];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int r = rr + u * kPass + rsub;
                    const unsigned long long p0 = __shfl_sync(0xffffffffu, (unsigned long long)src[0], r & 31);
                    const unsigned long long p1 = __shfl_sync(0xffffffffu, (unsigned long long)src[1], r & 31);
                    const uint4 *p = reinterpret_cast<const uint4 *>(r < 32 ? p0 : p1) + part * 2;
                    w[u][0] = w[u][1] = make_uint4(0, 0, 0, 0);
                    if (r < nr) {
                        w[u][0] = __ldg(p);
                        w[u][1] = __ldg(p + 1);
                    }
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int r = rr + u * kPass + rsub;
                    const uint32_t v[8] = {w[u][0].x, w[u][0].y, w[u][0].z, w[u][0].w,
                                           w[u][1].x, w[u][1].y, w[u][1].z, w[u][1].w};
                    uint32_t top = 0;   // magnitudes of bf16 pairs as integers: order as the values
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = __vmaxu2(top, v[i] & 0x7fff7fffu);
                    top = max(top & 0xffffu, top >> 16);
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    // 2^e * max in [2^14, 2^15); e within fp32's exponents; infinities and NaN stay.
                    const int ex = (int)(top >> 7) - 127;
                    const int e = (top > 0 && ex < 128) ? min(14 - ex, 100) : 0;
                    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
                    uint32_t hh[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const __half2 x = __floats2half2_rn(bf16lo(v[i]) * up, bf16hi(v[i]) * up);
                        hh[i] = *reinterpret_cast<const uint32_t *>(&x);
                    }
                    if (r < N) {
                        uint8_t *row = qs + (part / 4) * (kRows * 128) + r * 128;
                        const int c = part % 4 * 2;
                        *reinterpret_cast<uint4 *>(row + (c ^ (r & 7)) * 16) = make_uint4(hh[0], hh[1], hh[2], hh[3]);
                        *reinterpret_cast<uint4 *>(row + ((c + 1) ^ (r & 7)) * 16) = make_uint4(hh[4], hh[5], hh[6], hh[7]);
                        if (part == 0) {
                            rw.mul(r) = r < nr ? a.qk_mul * __uint_as_float((uint32_t)(127 - e) << 23) : 0.f;
                            rw.neg_max(r) = r < nr ? INFINITY : 0.f;
                        }
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.q_full[piece & 1]);
            ++piece;
        } while (wk.next());
    }
    // Tear-down.  Without a timeout every copy and product has been waited
    // for; after one, what is in flight is (the drain has its own budget).
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*abort) {
        int own = 0;
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (tid == 0) flag_status(a.hdr, DSPARK_DEV_TIMEOUT);
        if (warp == kWarpQk || warp == kWarpPv) {
            uint64_t *bar = &ms.drain[warp - kWarpQk];
            if (elect_one()) mma_commit(bar);
            __syncwarp();
            mbar_wait_bounded(bar, 0, &own, kWaitBudget);
        }
        __syncthreads();
    }
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tm, 512);
}

// Joins the parts of the item that CTA blockIdx.x left unfinished: a warp per row.
template <int D>
__global__ void __launch_bounds__(256) cache_attention_join(const AttnArgs a) {
    const int32_t *d = a.desc + blockIdx.x * kDescInts;
    const int more = d[0];
    if (more <= 0) return;
    const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (r >= d[3]) return;
    const int parts = 1 + more;
    // Part 0 is this CTA's second slot, part i > 0 the first slot of CTA blockIdx.x + i.
    auto slot = [&](int i) { return i == 0 ? 2 * (int)blockIdx.x + 1 : 2 * ((int)blockIdx.x + i); };
    float m = -INFINITY;
    for (int i = lane; i < parts; i += 32) {
        const float2 v = a.part_ml[slot(i) * kRows + r];
        m = fmaxf(m, v.x);
    }
    m = warp_max_f32(m);
    constexpr int kPer = D / 32;
    float o[kPer], l = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) o[k] = 0.f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const size_t at = (size_t)slot(i) * kRows + r;
        const float2 v = a.part_ml[at];
        const float w = v.x == -INFINITY ? (v.y == 0.f ? 0.f : v.y) : fast_exp2(v.x - m);   // y != 0 here is NaN
        l = fmaf(w, v.y, l);
#pragma unroll
        for (int k = 0; k < kPer; ++k) o[k] = fmaf(w, a.part_o[at * D + k * 32 + lane], o[k]);
    }
    const int gr = d[2] + r;
    const long long row = (long long)(d[1] + gr / a.group) * a.Hq + d[4] * a.group + gr % a.group;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        a.out[row * D + k * 32 + lane] = __float2bfloat16_rn(l == 0.f ? 0.f : o[k] / l * a.v_mul);
}

template <int D>
cudaError_t launch_d(const AttnArgs &a, int grid, cudaStream_t st) {
    const size_t bytes = Lay<D>::misc + sizeof(Misc) + 1024;
    static_assert(Lay<D>::misc + sizeof(Misc) + 1024 <= 227 * 1024, "shared memory of an SM");
    static_assert(4096 * (sizeof(long long) + sizeof(int)) <= kRing * Lay<D>::kPBytes, "the prefix of the largest batch");
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(cache_attention_kernel<D>), bytes, done);
    if (e != cudaSuccess) return e;
    cache_attention_kernel<D><<<grid, kThreads, bytes, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cache_attention_join<D><<<dim3(grid, kRows / 8), 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t attention_ws_bytes(int D) {
    return sizeof(WsHeader) + align256((size_t)kMaxCtas * kDescInts * 4) +
           align256((size_t)2 * kMaxCtas * kRows * sizeof(float2)) + align256((size_t)2 * kMaxCtas * kRows * D * 4);
}

cudaError_t launch_cache_attention(AttnArgs a, void *ws, cudaStream_t st) {
    uint8_t *p = static_cast<uint8_t *>(ws);
    a.hdr = reinterpret_cast<WsHeader *>(p);
    p += sizeof(WsHeader);
    a.desc = reinterpret_cast<int32_t *>(p);
    p += align256((size_t)kMaxCtas * kDescInts * 4);
    a.part_ml = reinterpret_cast<float2 *>(p);
    p += align256((size_t)2 * kMaxCtas * kRows * sizeof(float2));
    a.part_o = reinterpret_cast<float *>(p);
    a.polls = (uint32_t)(wait_budget(kWaitBudget) / kPollCycles) + 1;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int grid = sms < kMaxCtas ? sms : kMaxCtas;
    return a.D == 128 ? launch_d<128>(a, grid, st) : launch_d<64>(a, grid, st);
}

}  // namespace dspark
