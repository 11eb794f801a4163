// kvd_paged_plan.cu -- one scheduling step of the paged cache on the device:
// block tables, the free-page stack, and the slot and position of every new row.
//
// With held_b = ceil(len_b / P) and after_b = ceil((keep_b + new_b) / P), a
// request gives up pages after_b .. held_b or takes pages held_b .. after_b,
// never both, so the step is three prefix sums over the requests (new rows,
// pages given, pages taken) and three independent fills: push, pop, slots.
//
// Bound by latency: a few tens of KB in all.  One cluster of CTAs does the
// step in one launch.  Every CTA takes the prefix sums itself (8192 requests
// at most, in shared memory), so nothing but the two orderings between the
// fills crosses CTAs, and the cluster's hardware barrier carries those.  The
// fills walk flat ranges of pages and rows with a binary search over the
// prefix sums, so one long prompt spreads over all threads like many short ones.
// Pages that are to change hands are looked at before the first barrier, which
// carries the verdict too: one outside the pool stops the step while nothing that
// counts is written (the stack above its old height is nobody's).
//
// Measured: one token for each of 256 requests 6.8 us, 500 requests with up to 256
// new rows each 12.1 us, 8000 requests of one row 20 us.  An empty launch takes 2;
// the rest is a chain of dependent steps (lengths, three block scans, two cluster
// barriers, table, slots).  Separate kernels would pay a launch for each barrier.

#include "kvd_internal.cuh"

namespace kvd {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxSeq = 8192;
constexpr int kPlanCtas = 8;  // the portable cluster size

struct PlanArgs {
    const int32_t *seq_len, *keep_len, *new_len, *n_free;
    int32_t n_seq, page_log2, max_pages;
    int32_t n_pages, n_tokens;
    int32_t *block_table, *free_pages, *seq_len_out, *n_free_out, *cu_new, *positions, *slots;
    uint32_t *err;
};

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// A word of the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_word(const uint32_t *word, uint32_t rank) {
    uint32_t at, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(word)), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// Largest i in [0, n) with pre[i] <= x, for pre[0] = 0 <= x (the last of equal
// entries, so an empty request is passed over).
__device__ __forceinline__ int owner_of(const int32_t *pre, int n, int32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Exclusive prefix sum over the block of one value per thread; *total gets the sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *warp_sums, int64_t *total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp_sums[w] = x;
    __syncthreads();
    if (w == 0) {
        int64_t y = warp_sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t z = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) y += z;
        }
        warp_sums[lane] = y;
    }
    __syncthreads();
    const int64_t before = w == 0 ? 0 : warp_sums[w - 1];
    *total = warp_sums[31];
    __syncthreads();
    return before + x - v;
}

template <int RUN>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ int32_t sm[];
    __shared__ int64_t warp_sums[32];
    __shared__ uint32_t strange;  // this CTA has met a page outside the pool
    const int n = a.n_seq;
    int32_t *cu = sm, *keep = cu + n + 1, *held = keep + n, *gone = held + n, *take = gone + n + 1;
    if (threadIdx.x == 0) strange = 0;
    pdl_wait();

    // Prefix sums.  A thread takes a run of consecutive requests.
    const int per = (n + kPlanThreads - 1) / kPlanThreads;
    const int b0 = threadIdx.x * per < n ? threadIdx.x * per : n, b1 = b0 + per < n ? b0 + per : n;
    int64_t rows = 0, given = 0, taken = 0;
    uint32_t bad = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t len = a.seq_len[b], kept = a.keep_len != nullptr ? a.keep_len[b] : len, fresh = a.new_len[b];
        const int64_t room = int64_t(a.max_pages) << a.page_log2, total = kept + fresh;
        if (len < 0 || kept < 0 || kept > len || fresh < 0 || len > room) bad |= kErrBounds;
        else if (total > room) bad |= kErrPages;
        const int64_t h = (len + (int64_t(1) << a.page_log2) - 1) >> a.page_log2;
        const int64_t f = (total + (int64_t(1) << a.page_log2) - 1) >> a.page_log2;
        keep[b] = int32_t(kept);
        held[b] = int32_t(h);
        rows += fresh;
        given += h > f ? h - f : 0;
        taken += f > h ? f - h : 0;
    }
    const int any_bounds = __syncthreads_or(bad & kErrBounds), any_full = __syncthreads_or(bad & kErrPages);
    int64_t n_rows, n_given, n_taken;
    int64_t r0 = block_scan(rows, warp_sums, &n_rows);
    int64_t g0 = block_scan(given, warp_sums, &n_given);
    int64_t t0 = block_scan(taken, warp_sums, &n_taken);
    const int64_t free0 = a.n_free[0];
    bool malformed = any_bounds || free0 < 0 || free0 > a.n_pages || free0 + n_given > a.n_pages;
    const bool full = any_full || n_taken > free0 + n_given || n_rows > a.n_tokens;
    const int tid = blockIdx.x * kPlanThreads + threadIdx.x, n_thr = gridDim.x * kPlanThreads;
    const int64_t top = free0 + n_given;  // height once everything given is pushed

    if (!malformed && !full) {
        for (int b = b0; b < b1; ++b) {
            const int32_t fresh = a.new_len[b];
            const int32_t f = int32_t((int64_t(keep[b]) + fresh + (1 << a.page_log2) - 1) >> a.page_log2);
            cu[b] = int32_t(r0);
            gone[b] = int32_t(g0);
            take[b] = int32_t(t0);
            r0 += fresh;
            g0 += held[b] > f ? held[b] - f : 0;
            t0 += f > held[b] ? f - held[b] : 0;
        }
        if (threadIdx.x == 0) {
            cu[n] = int32_t(n_rows);
            gone[n] = int32_t(n_given);
            take[n] = int32_t(n_taken);
        }
        __syncthreads();
        const auto in_pool = [&](int32_t page) { return page >= 0 && page < a.n_pages; };
        // push: j-th page given, counted over requests and then pages
        for (int j = tid; j < n_given; j += n_thr) {
            const int b = owner_of(gone, n, j);
            const int count = gone[b + 1] - gone[b];
            const int32_t page = a.block_table[int64_t(b) * a.max_pages + held[b] - count + (j - gone[b])];
            if (!in_pool(page)) strange = 1;
            a.free_pages[free0 + j] = page;
        }
        // what lay on the stack and is taken; the thread's first is kept at hand
        int32_t first = -1;
        for (int64_t j = n_given + tid; j < n_taken; j += n_thr) {
            const int32_t page = a.free_pages[top - 1 - j];
            if (!in_pool(page)) strange = 1;
            if (j == n_given + tid) first = page;
        }
        // every thread of every CTA has also read its inputs by now, so the
        // outputs that may alias them are written only after this barrier
        cluster_barrier();
        const uint32_t lane = threadIdx.x & 31;
        malformed = __any_sync(0xffffffffu, lane < kPlanCtas && peer_word(&strange, lane) != 0);
        if (!malformed) {
            const auto pop = [&](int64_t j, int32_t page) {
                const int b = owner_of(take, n, int32_t(j));
                a.block_table[int64_t(b) * a.max_pages + held[b] + (j - take[b])] = page;
            };
            for (int64_t j = n_given + tid; j < n_taken; j += n_thr) pop(j, j == n_given + tid ? first : a.free_pages[top - 1 - j]);
            for (int64_t j = tid; j < n_given && j < n_taken; j += n_thr) pop(j, a.free_pages[top - 1 - j]);
        }
        cluster_barrier();
    } else {
        cluster_barrier();
        cluster_barrier();
    }

    const bool ok = !malformed && !full;
    if (tid == 0) {
        if (!ok) set_error(a.err, malformed ? kErrBounds : kErrPages);
        a.n_free_out[0] = int32_t(ok ? top - n_taken : free0);
    }
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b < n; b += kPlanThreads) {
            if (ok) a.seq_len_out[b] = keep[b] + (cu[b + 1] - cu[b]);
            else if (a.seq_len_out != a.seq_len) a.seq_len_out[b] = a.seq_len[b];
        }
        for (int b = threadIdx.x; b <= n; b += kPlanThreads) a.cu_new[b] = ok ? cu[b] : 0;
    }
    // slots: a thread takes the rows t .. t + RUN - 1, one after another
    const int32_t mask = (1 << a.page_log2) - 1;
    for (int64_t t = int64_t(tid) * RUN; t < a.n_tokens; t += int64_t(n_thr) * RUN) {
        int32_t pos[RUN], slot[RUN], b = 0, end = 0;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            pos[i] = slot[i] = -1;
            if (!ok || t + i >= n_rows) continue;
            if (t + i >= end) {
                b = owner_of(cu, n, int32_t(t) + i);
                end = cu[b + 1];
            }
            pos[i] = keep[b] + (int32_t(t) + i - cu[b]);
            const int32_t page = a.block_table[int64_t(b) * a.max_pages + (pos[i] >> a.page_log2)];
            if (page < 0 || page >= a.n_pages) set_error(a.err, kErrBounds);
            else slot[i] = (page << a.page_log2) + (pos[i] & mask);
        }
        if (RUN == 4 && t + RUN <= a.n_tokens) {
            *reinterpret_cast<int4 *>(a.positions + t) = *reinterpret_cast<int4 *>(pos);
            *reinterpret_cast<int4 *>(a.slots + t) = *reinterpret_cast<int4 *>(slot);
        } else {
#pragma unroll
            for (int i = 0; i < RUN; ++i) {
                if (t + i >= a.n_tokens) break;
                a.positions[t + i] = pos[i];
                a.slots[t + i] = slot[i];
            }
        }
    }
}

}  // namespace
}  // namespace kvd

using namespace kvd;

extern "C" kvd_status kv_paged_plan(const int32_t *seq_len, const int32_t *keep_len, const int32_t *new_len,
                                    int32_t n_seq, int64_t n_pages, int32_t page_size, int32_t *block_table,
                                    int32_t max_pages, int32_t *free_pages, const int32_t *n_free,
                                    int32_t *seq_len_out, int32_t *n_free_out, int32_t *cu_new,
                                    int32_t *positions, int32_t *slots, int64_t n_tokens, uint32_t *err,
                                    void *stream) {
    KVD_NVTX_RANGE("kv_paged_plan");
    if (seq_len == nullptr || new_len == nullptr || block_table == nullptr || free_pages == nullptr ||
        n_free == nullptr || seq_len_out == nullptr || n_free_out == nullptr || cu_new == nullptr || err == nullptr)
        return KVD_EINVAL;
    if (n_seq < 1 || n_seq > kPlanMaxSeq || max_pages < 1 || n_tokens < 0 || n_tokens > (int64_t(1) << 30)) return KVD_EINVAL;
    if (n_tokens > 0 && (positions == nullptr || slots == nullptr)) return KVD_EINVAL;
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return KVD_EINVAL;
    if (n_pages < 1 || n_pages >= (int64_t(1) << 31) || n_pages * page_size >= (int64_t(1) << 31)) return KVD_EINVAL;
    if (int64_t(max_pages) * page_size > (int64_t(1) << 31) - 1024) return KVD_EINVAL;
    PlanArgs a = {};
    a.seq_len = seq_len;
    a.keep_len = keep_len;
    a.new_len = new_len;
    a.n_free = n_free;
    a.n_seq = n_seq;
    a.page_log2 = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
    a.max_pages = max_pages;
    a.n_pages = int32_t(n_pages);
    a.n_tokens = int32_t(n_tokens);
    a.block_table = block_table;
    a.free_pages = free_pages;
    a.seq_len_out = seq_len_out;
    a.n_free_out = n_free_out;
    a.cu_new = cu_new;
    a.positions = positions;
    a.slots = slots;
    a.err = err;
    // With more rows than threads and runs of rows that one request owns, a thread
    // takes four neighbours at a time: one search and one wide store for them.
    // (500 requests of some 128 new rows: 11.8 us, one by one 13.8; 8000 of three:
    // 23.7 and 21.2.)
    const bool four = n_tokens > kPlanCtas * kPlanThreads && n_tokens >= 8 * int64_t(n_seq) &&
                      ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(slots)) & 15) == 0;
    const auto kern = four ? plan_kernel<4> : plan_kernel<1>;
    const size_t smem = (5 * size_t(n_seq) + 3) * 4;
    if (smem > 40 * 1024 && set_smem_once(reinterpret_cast<const void *>(kern), (5 * kPlanMaxSeq + 3) * 4) != cudaSuccess)
        return KVD_ECUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kPlanCtas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = as_stream(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kPlanCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    return e == cudaSuccess && !fault_fires() ? KVD_OK : KVD_ECUDA;
}

extern "C" kvd_status kv_paged_device_error(uint32_t *err, int32_t clear, uint32_t *word_out) {
    if (err == nullptr) return KVD_EINVAL;
    uint32_t w = 0;
    if (cudaMemcpy(&w, err, 4, cudaMemcpyDeviceToHost) != cudaSuccess) return KVD_ECUDA;
    // (cleared when this returns: a call on another stream may follow at once)
    if (clear && (cudaMemset(err, 0, 4) != cudaSuccess || cudaStreamSynchronize(nullptr) != cudaSuccess)) return KVD_ECUDA;
    if (word_out) *word_out = w;
    return w ? KVD_EDEVICE : KVD_OK;
}
