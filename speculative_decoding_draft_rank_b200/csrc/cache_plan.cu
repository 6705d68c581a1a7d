// cache_plan.cu -- a round's block tables, slot map and positions from the
// admitted lengths, and after verification the pages behind the accepted
// tokens given back; all on the device, so no round trip to the host stands
// between the scheduler and the target pass.
//
// Prefix sums over the requests give every new token its row and every new
// page its place on the free list, so the result does not depend on the order
// in which threads run.  The work is a third of a megabyte at the largest
// batch: what bounds it is latency (the dependent steps lengths, prefix,
// owner, page), so each is one launch.  Measured in a graph, plan and commit
// together: 4 requests 9 us, 256 requests 12 us, 4096 requests 25 us.
#include "cache.cuh"
#include "tc.cuh"

namespace dspark {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kCommitThreads = 1024;
// Pages (below 2^27) and rows (4096 requests of 2^20 + 1, below 2^33) in one sum.
constexpr int kRowBits = 34;
constexpr long long kRowMask = (1LL << kRowBits) - 1;

__device__ __forceinline__ int pages_of(int tokens, int P) { return (tokens + P - 1) / P; }

// Exclusive prefix of one value per thread over the block, and the total.
template <int N>
__device__ __forceinline__ long long block_scan(long long v, long long &total, long long *sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = inc;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < N / 32; ++w) {
        const long long x = sh[w];
        if (w < warp) before += x;
        total += x;
    }
    return before + inc - v;
}

// Largest b in [0, B) with first[b] <= i (first is non-decreasing, first[0] <= i).
__device__ __forceinline__ int owner(const int *first, int B, int i) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

// One request's wish: its tokens, and the pages it lacks.
struct Wish {
    int ctx, held, n, need;
};
__device__ __forceinline__ Wish wish_of(const PlanArgs &a, int b, uint32_t &flags) {
    Wish w;
    w.ctx = __ldg(a.ctx + b);
    w.held = a.held[b];
    if (w.held < 0 || w.held > a.max_pages) {
        flags |= DSPARK_DEV_LENGTH_RANGE;
        w.held = min(max(w.held, 0), a.max_pages);
    }
    if (w.ctx < 0) {                       // an empty seat
        w.n = w.need = 0;
        return w;
    }
    int e = a.ell[b];   // ell_out may be ell
    if (e < 0 || e > a.G) {
        flags |= DSPARK_DEV_ELL_RANGE;
        e = min(max(e, 0), a.G);
    }
    const int cap = a.max_pages * a.P;
    if (w.ctx > cap) {
        flags |= DSPARK_DEV_LENGTH_RANGE;
        w.ctx = cap;
    }
    w.n = min(e + 1, cap - w.ctx);
    if (w.n < e + 1) flags |= DSPARK_DEV_CACHE_FULL;
    w.need = max(0, pages_of(w.ctx + w.n, a.P) - w.held);
    return w;
}

// A cluster of up to 8 CTAs: each repeats the prefix sums (a few reads per
// thread), then they share the tokens and pages.  The cluster barrier stands
// between the last read of held and free_count and their update.
__global__ void __launch_bounds__(kPlanThreads) cache_plan_kernel(const PlanArgs a) {
    extern __shared__ int sh[];
    __shared__ long long part[kPlanThreads / 32];
    int *start = sh;                  // first row of a request
    int *first = sh + a.B + 1;        // its first new page, counted from the top of the free list
    int *old = first + a.B + 1;       // pages held before
    const int tid = threadIdx.x, rank = blockIdx.x, ranks = gridDim.x;
    const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    uint32_t flags = 0;
    int count = *a.free_count;
    if (count < 0 || count > a.n_pages) {
        flags |= DSPARK_DEV_LENGTH_RANGE;
        count = min(max(count, 0), a.n_pages);
    }
    long long need = 0, total;
    for (int b = b0; b < b1; ++b) need += wish_of(a, b, flags).need;
    const long long e0 = block_scan<kPlanThreads>(need, total, part);
    // Granted: a request that needs pages gets all of them or none, in order.
    long long e = e0, both = 0;
    for (int b = b0; b < b1; ++b) {
        Wish w = wish_of(a, b, flags);
        const bool ok = w.need == 0 || e + w.need <= count;
        e += w.need;
        if (!ok) {
            flags |= DSPARK_DEV_CACHE_FULL;
            w.n = max(0, min(w.n, w.held * a.P - w.ctx));
            w.need = 0;
        }
        both += (long long)w.need << kRowBits | w.n;
        old[b] = w.held;
        start[b] = w.n;
        first[b] = w.need;
    }
    long long sums;
    long long run = block_scan<kPlanThreads>(both, sums, part);
    for (int b = b0; b < b1; ++b) {
        const int n = start[b], nd = first[b];
        start[b] = (int)min(run & kRowMask, (long long)a.T);
        first[b] = (int)(run >> kRowBits);
        run += (long long)nd << kRowBits | n;
    }
    if ((sums & kRowMask) > a.T) flags |= DSPARK_DEV_CACHE_FULL;
    const int rows = (int)min(sums & kRowMask, (long long)a.T), pages = (int)(sums >> kRowBits);
    if (tid == 0) {
        start[a.B] = rows;
        first[a.B] = pages;
    }
    __syncthreads();
    if (ranks > 1) tc::cluster_sync();
    const int stride = ranks * kPlanThreads, id = rank * kPlanThreads + tid;
    for (int b = id; b < a.B; b += stride) {
        const int n = start[b + 1] - start[b], c = __ldg(a.ctx + b);
        a.q_start[b] = start[b];
        a.kv_len[b] = c < 0 ? 0 : min(c, a.max_pages * a.P) + n;
        a.held[b] = old[b] + first[b + 1] - first[b];
        if (a.ell_out != nullptr) a.ell_out[b] = max(n - 1, 0);
    }
    if (id == 0) {
        a.q_start[a.B] = rows;
        *a.free_count = count - pages;
    }
    if (rank == 0 && flags) atomicOr(&a.hdr->status, flags);
    for (int t = id; t < a.T; t += stride) {
        int slot = -1, pos = -1;
        if (t < rows) {
            const int b = owner(start, a.B, t);
            pos = min(__ldg(a.ctx + b), a.max_pages * a.P) + t - start[b];
            const int pg = pos / a.P;
            const int page = pg < old[b] ? a.table[(size_t)b * a.max_pages + pg]
                                         : __ldg(a.free_list + (count - 1 - (first[b] + pg - old[b])));
            if (page >= 0 && page < a.n_pages)
                slot = page * a.P + pos % a.P;
            else
                flag_status(a.hdr, DSPARK_DEV_PAGE_RANGE);
        }
        a.slot[t] = slot;
        a.pos[t] = pos;
    }
    for (int i = id; i < pages; i += stride) {
        const int b = owner(first, a.B, i);
        a.table[(size_t)b * a.max_pages + old[b] + i - first[b]] = __ldg(a.free_list + (count - 1 - i));
    }
}

__global__ void __launch_bounds__(kCommitThreads) cache_commit_kernel(const CommitArgs a) {
    extern __shared__ int sh[];
    __shared__ long long part[kCommitThreads / 32];
    int *first = sh;               // released pages of the requests before
    int *keep = sh + a.B + 1;      // pages a request keeps
    const int tid = threadIdx.x;
    const int per = (a.B + kCommitThreads - 1) / kCommitThreads;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    uint32_t flags = 0;
    int count = *a.free_count;
    if (count < 0 || count > a.n_pages) {
        flags |= DSPARK_DEV_LENGTH_RANGE;
        count = min(max(count, 0), a.n_pages);
    }
    long long sum = 0, total;
    for (int b = b0; b < b1; ++b) {
        const int c = a.ctx[b];              // ctx_out may be ctx
        int held = a.held[b];
        if (held < 0 || held > a.max_pages) {
            flags |= DSPARK_DEV_LENGTH_RANGE;
            held = min(max(held, 0), a.max_pages);
        }
        int out = -1;
        // Nothing of a request without rows went through the target.
        if (a.nout_rw != nullptr && __ldg(a.q_start + b + 1) <= __ldg(a.q_start + b)) {
            a.nout_rw[b] = 0;
            if (a.acc != nullptr) a.acc[b] = 0;
            if (a.tokens != nullptr)
                for (int j = 0; j <= a.G; ++j) a.tokens[(size_t)b * (a.G + 1) + j] = -1;
        }
        if (c >= 0 && (a.done == nullptr || __ldg(a.done + b) == 0)) {
            const int s0 = max(0, __ldg(a.q_start + b)), s1 = max(s0, __ldg(a.q_start + b + 1));
            const int n = min(s1 - s0, a.max_pages * a.P);
            const int k = a.nout[b];
            if (k < 0 || k > n) flags |= DSPARK_DEV_LENGTH_RANGE;
            out = min(c, a.max_pages * a.P) + min(max(k, 0), n);
            out = min(out, a.max_pages * a.P);
        }
        const int kp = min(held, pages_of(max(out, 0), a.P));
        a.ctx_out[b] = out;
        a.held[b] = kp;
        keep[b] = kp;
        first[b] = held - kp;
        sum += held - kp;
    }
    long long run = block_scan<kCommitThreads>(sum, total, part);
    for (int b = b0; b < b1; ++b) {
        const int n = first[b];
        first[b] = (int)run;
        run += n;
    }
    if (tid == 0) first[a.B] = (int)total;
    __syncthreads();
    const int back = (int)total;
    // More pages than the pool has: the tables do not belong to it.
    if (back > a.n_pages - count) flags |= DSPARK_DEV_LENGTH_RANGE;
    // The first page released goes on top, so undoing a plan restores the list.
    for (int i = tid; i < back; i += kCommitThreads) {
        const int b = owner(first, a.B, i);
        int32_t *cell = a.table + (size_t)b * a.max_pages + keep[b] + i - first[b];
        const int at = count + back - 1 - i;
        if (at < a.n_pages) a.free_list[at] = *cell;
        *cell = -1;
    }
    if (tid == 0) *a.free_count = min(a.n_pages, count + back);
    if (flags) atomicOr(&a.hdr->status, flags);
}

}  // namespace

cudaError_t launch_cache_plan(const PlanArgs &a, cudaStream_t st) {
    // One CTA for up to 1024 tokens, else a cluster of 8.  Measured, one CTA
    // against the cluster: 24 tokens 3.9 and 4.5 us, 384 4.3 and 4.9, 1152 5.1
    // and 4.9, 2400 6.6 and 5.3.
    const int ranks = a.T <= 2 * kPlanThreads ? 1 : 8;
    const size_t bytes = (size_t)(3 * a.B + 3) * sizeof(int);
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void *>(cache_plan_kernel), (3 * 4096 + 3) * sizeof(int), done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ranks);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, cache_plan_kernel, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_cache_commit(const CommitArgs &a, cudaStream_t st) {
    const size_t bytes = (size_t)(2 * a.B + 2) * sizeof(int);
    cache_commit_kernel<<<1, kCommitThreads, bytes, st>>>(a);
    return cudaGetLastError();
}

}  // namespace dspark
