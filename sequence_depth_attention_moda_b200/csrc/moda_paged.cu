// moda_paged.cu -- the paged KV cache behind the attention of drafted tokens:
// pages and slots from request lengths (moda_page_plan), new keys and values
// into their slots (moda_cache_append), ancestor bits of drafted trees
// (moda_tree_mask), and the C entry points of these and of moda_tree_decode.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <utility>

#include "moda.h"
#include "moda_internal.h"
#include "moda_tree.cuh"

namespace moda {
namespace {

// ------------------------------------------------------------------ plan ----
// Page lists from lengths.  Request b holds have_b = ceil(held/P) pages and is
// to hold need_b = ceil(want/P).  With exclusive prefixes over the requests,
// drop_b of the pages given back (have - need where positive) and take_b of
// those asked for, and top = count + sum of drops, released page r of the call
// goes to place top-1-r of the free list and asked-for page q comes from place
// top-1-q: a stack, the first request's pages on top, so that giving back what
// a call took restores the list.  A request is served whole or not at all: if it
// needs no page, or take_b + its own pages <= top; those that are served pages
// come before those that are refused some, so pages 0 .. granted-1 are theirs.
// Released entries that name no page (a held length beyond the pages a request has)
// are counted while they are moved and taken out again: they do not count in top.
//
// Bound by latency, not by bytes.  Every CTA adds up all requests (8 KB for 1024
// of them) and keeps the prefixes in shared memory; then a thread finds its
// page's or token's request by bisection, so few long requests spread over the
// threads as many short ones do.  Released pages are written before any is
// taken, and table entries before slots read them: CTA barriers where one CTA
// does it all, else barriers of a cluster of 8 (see launch_plan for the choice).
// The slots of many tokens are a grid of their own.  Measured inside a graph, a call that
// takes pages and the one that gives them back together: 256 requests of 8 new tokens
// 12.7 us, 64 prompts of up to 8192 tokens 17.0 us.
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMaxPlanRequests = 16384;
constexpr int kSlotThreads = 256;
constexpr int kSlotsPerLane = 4;

struct PlanArgs {
    const int *held, *want;
    int *table, *free_pages, *free_count, *cu, *granted;
    long long* slots;
    unsigned int* status;
    int B, N, page_shift, n_pages, max_pages;
    int slots_here;                  // the plan kernel writes the slots itself
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
template <int CTAS>
__device__ __forceinline__ void plan_barrier() {
    if (CTAS == 1) {
        __syncthreads();
    } else {
        cluster_arrive();
        cluster_wait();
    }
}

// Exclusive prefixes of x and y over the CTA's threads; tx and ty get the sums.
__device__ __forceinline__ void block_prefix(long long& x, long long& y, longlong2* warp_sum, long long* tx,
                                             long long* ty) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long ix = x, iy = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long ux = __shfl_up_sync(0xffffffffu, ix, o), uy = __shfl_up_sync(0xffffffffu, iy, o);
        if (lane >= o) {
            ix += ux;
            iy += uy;
        }
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = make_longlong2(ix, iy);
    __syncthreads();
    long long wx = 0, wy = 0;            // lane w: the sum of warp w
    if (lane < kPlanWarps) {
        wx = warp_sum[lane].x;
        wy = warp_sum[lane].y;
    }
    long long px = wx, py = wy;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long ux = __shfl_up_sync(0xffffffffu, px, o), uy = __shfl_up_sync(0xffffffffu, py, o);
        if (lane >= o) {
            px += ux;
            py += uy;
        }
    }
    *tx = __shfl_sync(0xffffffffu, px, 31);
    *ty = __shfl_sync(0xffffffffu, py, 31);
    x = __shfl_sync(0xffffffffu, px - wx, warp) + ix - x;
    y = __shfl_sync(0xffffffffu, py - wy, warp) + iy - y;
}

struct PlanRequest {
    int held, want, have, need;      // clamped; need = have where the request cannot fit its row
    bool fits;
};
__device__ __forceinline__ PlanRequest plan_request(const PlanArgs& a, int b) {
    PlanRequest r;
    const int P1 = (1 << a.page_shift) - 1;
    const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
    const int h = a.held[b], w = a.want[b];
    r.held = static_cast<int>(min(static_cast<long long>(max(h, 0)), cap));
    r.want = max(w, 0);
    if (r.held != h || r.want != w) atomicOr(a.status, kStatusBadIndex);
    r.fits = r.want <= cap;
    r.have = static_cast<int>((static_cast<long long>(r.held) + P1) >> a.page_shift);
    r.need = r.fits ? static_cast<int>((static_cast<long long>(r.want) + P1) >> a.page_shift) : r.have;
    return r;
}

__device__ __forceinline__ bool is_page(const PlanArgs& a, int page) {
    return static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages);
}

// The last of n entries of an ascending list that is <= x (the first is 0).
__device__ __forceinline__ int last_at_most(const int* list, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (list[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Slots of tokens t0 + 32u + lane, u < kSlotsPerLane (whole warp); s_cu: cu in shared memory.
__device__ __forceinline__ void write_slots(const PlanArgs& a, const int* s_cu, long long t0, int lane) {
    const int n_in = min(s_cu[a.B], a.N);
    long long slot[kSlotsPerLane];
    int b = a.B > 0 && t0 < n_in ? last_at_most(s_cu, a.B, static_cast<int>(t0)) : 0;
#pragma unroll
    for (int u = 0; u < kSlotsPerLane; ++u) {
        const long long t = t0 + 32 * u + lane;
        slot[u] = -1;
        if (t < n_in) {
            while (s_cu[b + 1] <= t) ++b;
            const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
            const int held = static_cast<int>(min(static_cast<long long>(max(a.held[b], 0)), cap));
            const int key = held + static_cast<int>(t - s_cu[b]);
            const int page = __ldcg(a.table + static_cast<size_t>(b) * a.max_pages + (key >> a.page_shift));
            if (is_page(a, page))
                slot[u] = (static_cast<long long>(page) << a.page_shift) + (key & ((1 << a.page_shift) - 1));
            else
                atomicOr(a.status, kStatusBadIndex);
        }
    }
#pragma unroll
    for (int u = 0; u < kSlotsPerLane; ++u) {
        const long long t = t0 + 32 * u + lane;
        if (t < a.N) a.slots[t] = slot[u];
    }
}

// Adds n to *x in the shared memory of every CTA.  (Rare, where a sum read from the
// others costs every call 0.7 us.)
template <int CTAS>
__device__ __forceinline__ void add_everywhere(int* x, int n) {
    if (CTAS == 1) {
        atomicAdd(x, n);
        return;
    }
#pragma unroll 1
    for (int r = 0; r < CTAS; ++r) {
        uint32_t at;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(x)), "r"(r));
        asm volatile("red.shared::cluster.add.s32 [%0], %1;" ::"r"(at), "r"(n) : "memory");
    }
}

// The table's entry for released page x of the call; s_drop: prefixes of those pages.
__device__ __forceinline__ int* released_entry(const PlanArgs& a, const int* s_drop, unsigned x) {
    const int b = last_at_most(s_drop, a.B, static_cast<int>(x));
    return a.table + static_cast<size_t>(b) * a.max_pages + plan_request(a, b).need + (static_cast<int>(x) - s_drop[b]);
}

// (Rare; one CTA.)  Of `drops` released entries the pages alone go to places count, count + 1, ..
// of the list: taken from its places count .., or, if they are not there, from the table.
__device__ __noinline__ void pack_released(const PlanArgs& a, const int* s_drop, longlong2* warp_sum, int count,
                                           long long drops, bool listed) {
    long long place = count;
    for (long long i0 = 0; i0 < drops; i0 += kPlanThreads) {
        const long long i = i0 + threadIdx.x;
        int* entry = nullptr;
        if (i < drops)
            entry = listed ? a.free_pages + count + i : released_entry(a, s_drop, static_cast<unsigned>(drops - 1 - i));
        const int page = entry ? __ldcg(entry) : -1;
        long long at = is_page(a, page), none = 0, n, n_none;
        block_prefix(at, none, warp_sum, &n, &n_none);       // (all have read before any writes)
        if (is_page(a, page) && place + at < a.n_pages) a.free_pages[place + at] = page;
        if (entry && !listed) *entry = -1;
        place += n;
    }
}

template <int CTAS>
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ int plan_smem[];
    __shared__ longlong2 warp_sum[kPlanWarps];
    __shared__ int s_lost;
    int* s_cu = plan_smem;               // [B+1] prefixes of tokens,
    int* s_take = s_cu + a.B + 1;        // [B]   of pages asked for,
    int* s_drop = s_take + a.B;          // [B]   of pages given back
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = CTAS == 1 ? 0 : static_cast<int>(blockIdx.x);     // one cluster
    const int all = rank * kPlanThreads + tid;                          // thread of the grid
    const int ch = (a.B + kPlanThreads - 1) / kPlanThreads;
    const int b0 = min(a.B, tid * ch), b1 = min(a.B, b0 + ch);
    if (tid == 0) s_lost = 0;
    if (CTAS > 1) cluster_arrive();
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();

    const int count0 = __ldcg(a.free_count);
    PlanRequest r0 = {};                 // up to 1024 requests have a thread each
    if (b0 < b1) r0 = plan_request(a, b0);
    long long take = 0, drop = 0, takes, drops;
    for (int b = b0; b < b1; ++b) {
        const PlanRequest r = b == b0 ? r0 : plan_request(a, b);
        take += max(r.need - r.have, 0);
        drop += max(r.have - r.need, 0);
    }
    block_prefix(take, drop, warp_sum, &takes, &drops);
    if (CTAS > 1) cluster_wait();        // every CTA has begun, with its s_lost at 0
    // released pages onto the list
    const int count = min(max(count0, 0), a.n_pages);
    const bool room = count + drops <= a.n_pages;      // else some of them cannot be pages, or the list is wrong
    int lost = 0;                        // entries that name no page
    if (drops > 0) {
        for (int b = b0; b < b1; ++b) {
            const PlanRequest r = b == b0 ? r0 : plan_request(a, b);
            s_drop[b] = static_cast<int>(drop);
            drop += max(r.have - r.need, 0);
        }
        __syncthreads();
        int mine = 0;
        for (unsigned x = all; x < static_cast<unsigned>(drops); x += CTAS * kPlanThreads) {
            int* entry = released_entry(a, s_drop, x);
            const int page = __ldcg(entry);
            mine += !is_page(a, page);
            if (!room) continue;
            a.free_pages[count + static_cast<int>(drops) - 1 - static_cast<int>(x)] = page;
            *entry = -1;
        }
        if (mine > 0) add_everywhere<CTAS>(&s_lost, mine);
        plan_barrier<CTAS>();
        lost = s_lost;
        if (lost > 0 || !room) {         // (rare) one CTA moves the pages together, from the list's bottom
            if (rank == 0) pack_released(a, s_drop, warp_sum, count, drops, room);
            plan_barrier<CTAS>();
        }
    }
    const long long top = count + drops - lost;
    if (count != count0 || lost > 0 || top > a.n_pages) atomicOr(a.status, kStatusBadIndex);
    // what is served: its tokens and pages
    long long tokens = 0, pages = 0, n_tokens, granted;
    {
        long long at = take;
        for (int b = b0; b < b1; ++b) {
            const PlanRequest r = b == b0 ? r0 : plan_request(a, b);
            const int t = max(r.need - r.have, 0);
            s_take[b] = static_cast<int>(at);
            at += t;
            if (r.fits && (t == 0 || at <= top)) {
                tokens += max(r.want - r.held, 0);
                pages += t;
            }
        }
    }
    block_prefix(tokens, pages, warp_sum, &n_tokens, &granted);
    long long c = tokens, at = take;
    for (int b = b0; b < b1; ++b) {
        const PlanRequest r = b == b0 ? r0 : plan_request(a, b);
        const int t = max(r.need - r.have, 0);
        at += t;
        const bool served = r.fits && (t == 0 || at <= top);
        s_cu[b] = static_cast<int>(min(c, 0x7fffffffll));
        if (rank == 0) {
            a.cu[b] = s_cu[b];
            a.granted[b] = served ? r.want : r.held;
        }
        if (served) c += max(r.want - r.held, 0);
    }
    if (tid == 0) {
        s_cu[a.B] = static_cast<int>(min(n_tokens, 0x7fffffffll));
        if (rank == 0) {
            a.cu[a.B] = s_cu[a.B];
            if (n_tokens > a.N) atomicOr(a.status, kStatusBadIndex);
        }
    }
    __syncthreads();

    // asked-for pages off it
    for (unsigned x = all; x < static_cast<unsigned>(granted); x += CTAS * kPlanThreads) {
        const int b = last_at_most(s_take, a.B, static_cast<int>(x));
        const long long place = top - 1 - x;
        int page = place < a.n_pages ? __ldcg(a.free_pages + place) : -1;
        if (!is_page(a, page)) {
            page = -1;
            atomicOr(a.status, kStatusBadIndex);
        }
        a.table[static_cast<size_t>(b) * a.max_pages + plan_request(a, b).have + (static_cast<int>(x) - s_take[b])] = page;
    }
    if (rank == 0 && tid == 0) *a.free_count = static_cast<int>(min(top - granted, static_cast<long long>(a.n_pages)));
    if (!a.slots_here) return;
    plan_barrier<CTAS>();
    for (long long t0 = (all >> 5) * 32ll * kSlotsPerLane; t0 < a.N; t0 += CTAS * kPlanThreads * kSlotsPerLane)
        write_slots(a, s_cu, t0, lane);
}

// The slots of many tokens, after the plan.
__global__ void __launch_bounds__(kSlotThreads) plan_slots_kernel(const __grid_constant__ PlanArgs a) {
    extern __shared__ int plan_smem[];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    for (int b = threadIdx.x; b <= a.B; b += kSlotThreads) plan_smem[b] = __ldcg(a.cu + b);
    __syncthreads();
    const int per = kSlotThreads * kSlotsPerLane;
    for (long long t0 = static_cast<long long>(blockIdx.x) * per + (threadIdx.x >> 5) * 32 * kSlotsPerLane; t0 < a.N;
         t0 += static_cast<long long>(gridDim.x) * per)
        write_slots(a, plan_smem, t0, threadIdx.x & 31);
}

// A launch that may be set up while the grid before it in the stream ends (the
// kernels wait for it themselves).
template <typename A>
cudaError_t launch_dependent(void (*kernel)(A), dim3 grid, unsigned block, int smem, int cluster, cudaStream_t s,
                             const A& a) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

cudaError_t launch_plan(PlanArgs& a, cudaStream_t s) {
    // One CTA while its 1024 threads need few turns for the pages that may be taken (at most
    // N / page + B), else a cluster of 8; and slots in a grid of their own from where its
    // SMs gain more than the second launch costs.  Measured inside a graph, one CTA
    // against the cluster: 256 requests, 2048 tokens (pages of 64) 7.6, 8.4 us; with the
    // slots apart 2048 requests, 16384 tokens 11.1, 11.3; 64, 32768 (pages of 16) 8.8, 7.9;
    // 1024, 65536 (16) 12.8, 9.5.  Slots by the plan's one CTA against apart: 4096 tokens
    // 8.3, 8.9; 8192 12.1, 9.6; 16384 20.0, 11.1.
    // N does not bound the pages that are given back, and what does, B * max_pages, is large
    // for every server: the host cannot tell a call that ends many long requests from a step
    // that moves a few pages.  With a small N it gets the one CTA, which then is the slower
    // choice (2048 pages given back 5.9 us against 6.5, 4096 7.4, 6.7; 8192 11.9, 6.8;
    // 131072, 256 requests of 8192 tokens in pages of 16, 122, 22).
    const bool small = static_cast<long long>(a.N >> a.page_shift) + a.B <= 4 * kPlanThreads;
    a.slots_here = a.N <= kPlanThreads * kSlotsPerLane;
    const int list = (a.B + 1) * static_cast<int>(sizeof(int)), smem = 3 * list;
    const int most = 3 * (kMaxPlanRequests + 1) * static_cast<int>(sizeof(int));
    auto kernel = small ? page_plan_kernel<1> : page_plan_kernel<8>;
    cudaError_t e = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), most);
    if (e == cudaSuccess) e = launch_dependent(kernel, small ? 1 : 8, kPlanThreads, smem, small ? 1 : 8, s, a);
    if (e != cudaSuccess || a.slots_here || a.N == 0) return e;
    e = set_max_dynamic_smem(reinterpret_cast<const void*>(plan_slots_kernel), most / 3);
    if (e != cudaSuccess) return e;
    const long long per = kSlotThreads * kSlotsPerLane, want = (a.N + per - 1) / per, cap = 8ll * device_sm_count();
    return launch_dependent(plan_slots_kernel, static_cast<unsigned>(want < cap ? want : cap), kSlotThreads, list, 1, s, a);
}

// ---------------------------------------------------------------- append ----
// A copy of N rows of Hk*d elements for K and for V, 16 bytes a thread and
// access; a head's d elements are contiguous on both sides (128 to 512 bytes).
// Bound by HBM: every byte is read once and written once.  Measured: 32768 tokens of
// 8 heads (268 MB moved) 43.5 us, 94% of a plain copy's bandwidth; 128 tokens 3.2 us
// inside a graph, 6.5 to 6.9 through the Python binding.
constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 4;

struct AppendArgs {
    const uint4 *k, *v;
    uint4 *kc, *vc;
    const long long* slots;
    unsigned int* status;
    long long n_slots, n_chunks;     // cache slots; N * row_chunks
    int Hk, head_chunks, row_chunks, page_shift;
};

__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const __grid_constant__ AppendArgs a) {
    const long long first = static_cast<long long>(blockIdx.x) * (kAppendThreads * kAppendUnroll);
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const long long tok0 = first / a.row_chunks;
    const unsigned c0 = static_cast<unsigned>(first - tok0 * a.row_chunks);
    uint4 kv[kAppendUnroll], vv[kAppendUnroll];
    long long dst[kAppendUnroll];
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u) {
        const unsigned i = c0 + u * kAppendThreads + threadIdx.x;
        const unsigned dt = i / static_cast<unsigned>(a.row_chunks);
        const unsigned c = i - dt * a.row_chunks;
        const long long tok = tok0 + dt;
        const long long src = tok * a.row_chunks + c;
        dst[u] = -1;
        if (src >= a.n_chunks) continue;
        const long long slot = a.slots[tok];
        if (slot >= 0 && slot < a.n_slots) {
            const unsigned hk = c / static_cast<unsigned>(a.head_chunks);
            const long long page = slot >> a.page_shift;
            const long long off = slot & ((1ll << a.page_shift) - 1);
            dst[u] = (((page * a.Hk + hk) << a.page_shift) + off) * a.head_chunks + (c - hk * a.head_chunks);
            kv[u] = __ldcs(a.k + src);
            vv[u] = __ldcs(a.v + src);
        } else if (slot != -1) {
            atomicOr(a.status, kStatusBadIndex);
        }
    }
#pragma unroll
    for (int u = 0; u < kAppendUnroll; ++u)
        if (dst[u] >= 0) {
            a.kc[dst[u]] = kv[u];
            a.vc[dst[u]] = vv[u];
        }
}

// ------------------------------------------------------------------ mask ----
// mask[i] = bit i | mask[parent[i]]: a thread a token walks its ancestors through
// the parents in shared memory.  Parents are earlier tokens, so the walk ends, and
// meets the words from the last to the first: it collects four at a time and
// stores them when it leaves them behind.  A CTA has 256 tokens of a request.
// Bound by the launch and by latency: random trees are shallow, a chain of n costs
// its last token n steps of about 60 cycles.  Measured inside a graph: 8 requests of
// 32 tokens 1.5 us, 256 of 256 3.0 us (both 11 through the Python binding), 8 of 2048 13 us,
// a chain of 2048 73 us.
constexpr int kMaskThreads = 256;
constexpr int kMaskGroup = 4;        // words a walk collects
constexpr int kMaxMaskWords = 64;

struct MaskArgs {
    const int *parent, *cu, *held;   // held: NULL counts positions from 0
    uint32_t* mask;
    int* position;
    unsigned int* status;
    int B, N, words;
};

__global__ void __launch_bounds__(kMaskThreads) tree_mask_kernel(const __grid_constant__ MaskArgs a) {
    __shared__ int up[32 * kMaxMaskWords];
    const int b = blockIdx.x;
    const int i0 = blockIdx.y * kMaskThreads;        // the CTA's first token
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int c0 = a.cu[b], c1 = a.cu[b + 1];
    const int h = a.held ? a.held[b] : 0;
    const int first = min(max(c0, 0), a.N);
    const int n = max(0, min(min(max(c1, 0), a.N) - first, 32 * a.words));
    bool bad = first != c0 || n != static_cast<long long>(c1) - c0;
    if (i0 >= n && i0 > 0) return;
    for (int i = threadIdx.x; i < min(n, i0 + kMaskThreads); i += kMaskThreads) {
        int p = a.parent[first + i];
        if (p < -1 || p >= i) {          // no earlier token: taken as the root's child
            bad = true;
            p = -1;
        }
        up[i] = p;
    }
    if (bad) atomicOr(a.status, kStatusBadIndex);
    __syncthreads();
    const int i = i0 + threadIdx.x;
    if (i >= n) return;
    uint32_t* row = a.mask + static_cast<size_t>(first + i) * a.words;
    int t = i, depth = -1;
    for (int w0 = (a.words - 1) / kMaskGroup * kMaskGroup; w0 >= 0; w0 -= kMaskGroup) {
        uint32_t w[kMaskGroup] = {};
        for (; t >= 32 * w0; t = up[t]) {
            const int at = (t >> 5) - w0;
            const uint32_t bit = 1u << (t & 31);
#pragma unroll
            for (int k = 0; k < kMaskGroup; ++k) w[k] |= at == k ? bit : 0u;
            ++depth;
        }
#pragma unroll
        for (int k = 0; k < kMaskGroup; ++k)
            if (w0 + k < a.words) row[w0 + k] = w[k];
    }
    a.position[first + i] = h + depth;
}

// ------------------------------------------------------------------- host ---
bool power_of_two(int x) { return x > 0 && (x & (x - 1)) == 0; }

moda_status failf(moda_status s, const char* fmt, long long x = 0, long long y = 0, long long z = 0) {
    char msg[240];
    snprintf(msg, sizeof(msg), fmt, x, y, z);
    return api_fail(s, msg);
}

// What every paged call checks: sizes of the batch and of the pages.
moda_status check_pages(const moda_paged_shape* s, Paged* p) {
    if (!s) return failf(MODA_ERR_INVALID_ARG, "shape is NULL");
    if (s->B < 0 || s->N < 0) return failf(MODA_ERR_INVALID_ARG, "B=%lld N=%lld must be >= 0", s->B, s->N);
    if (!power_of_two(s->page_size) || s->page_size < 8 || s->page_size > 1024)
        return failf(MODA_ERR_INVALID_ARG, "page_size=%lld must be a power of two in 8..1024", s->page_size);
    // (a thread's share of the requests is rounded up in 32 bits)
    if (s->B > 2147483647 - 1024) return failf(MODA_ERR_UNSUPPORTED, "B=%lld requests are too many", s->B);
    if (s->n_pages < 1 || s->max_pages < 1)
        return failf(MODA_ERR_INVALID_ARG, "n_pages=%lld and max_pages=%lld must be >= 1", s->n_pages, s->max_pages);
    // positions and table entries are indexed with 32 bits, and so are the rows behind the last
    // position of the tiles that are asked for ahead (fewer than 256)
    if (static_cast<double>(s->max_pages) * s->page_size > 2147483648.0 - 1024.0 ||
        static_cast<double>(s->B) * s->max_pages > 2147483647.0)
        return failf(MODA_ERR_UNSUPPORTED, "max_pages=%lld too large for B=%lld requests of pages of %lld tokens",
                     s->max_pages, s->B, s->page_size);
    p->B = s->B; p->N = s->N; p->page = s->page_size; p->n_pages = s->n_pages; p->max_pages = s->max_pages;
    p->page_shift = 0;
    while ((1 << p->page_shift) < s->page_size) ++p->page_shift;
    return MODA_OK;
}

moda_status check_words(const moda_paged_shape* s, Paged* p, bool needed) {
    if (s->mask_words < (needed ? 1 : 0) || s->mask_words > kMaxMaskWords)
        return failf(MODA_ERR_INVALID_ARG, "mask_words=%lld must be in %lld..%lld", s->mask_words, needed ? 1 : 0,
                     kMaxMaskWords);
    p->words = s->mask_words;
    return MODA_OK;
}

// The cache's element type, heads and head dimension.
moda_status check_cache(const moda_paged_shape* s, Paged* p) {
    if (s->dtype != MODA_BF16 && s->dtype != MODA_FP32)
        return failf(MODA_ERR_INVALID_ARG, "unknown dtype %lld", s->dtype);
    if (s->Hk < 1) return failf(MODA_ERR_INVALID_ARG, "need Hk >= 1 (Hk=%lld)", s->Hk);
    if (s->d != 64 && s->d != 128) return failf(MODA_ERR_UNSUPPORTED, "the paged calls support d in {64, 128} (d=%lld)", s->d);
    if (static_cast<double>(s->n_pages) * s->Hk > 2147483647.0)
        return failf(MODA_ERR_UNSUPPORTED, "n_pages=%lld of Hk=%lld heads pass 32-bit page indices", s->n_pages, s->Hk);
    p->Hk = s->Hk; p->d = s->d;
    p->elem_bytes = s->dtype == MODA_BF16 ? 2 : 4;
    return MODA_OK;
}

moda_status check_tree(const moda_paged_shape* s, Paged* p) {
    moda_status st;
    if ((st = check_pages(s, p)) != MODA_OK || (st = check_words(s, p, false)) != MODA_OK ||
        (st = check_cache(s, p)) != MODA_OK)
        return st;
    if (s->Hq < 1 || s->Hq % s->Hk != 0)
        return failf(MODA_ERR_INVALID_ARG, "need Hq >= 1 and Hq %% Hk == 0 (Hq=%lld Hk=%lld)", s->Hq, s->Hk);
    if (s->Hq / s->Hk > 64)
        return failf(MODA_ERR_UNSUPPORTED, "moda_tree_decode supports G <= 64 (G=%lld)", s->Hq / s->Hk);
    if (s->L < 0) return failf(MODA_ERR_INVALID_ARG, "L=%lld must be >= 0", s->L);
    if (s->depth_window < 0 || s->depth_window > s->L)
        return failf(MODA_ERR_INVALID_ARG, "depth_window=%lld must be in 0..L (L=%lld)", s->depth_window, s->L);
    if (!(s->softmax_scale >= 0.0f) || std::isinf(s->softmax_scale))
        return failf(MODA_ERR_INVALID_ARG, "softmax_scale must be >= 0 and finite (0 selects 1/sqrt(d))");
    if (static_cast<double>(s->N) * s->Hq > 2147483647.0 || static_cast<double>(s->N) * s->Hk > 2147483647.0)
        return failf(MODA_ERR_UNSUPPORTED, "N=%lld tokens of Hq=%lld heads pass 32-bit row indices", s->N, s->Hq);
    p->Hq = s->Hq; p->G = s->Hq / s->Hk; p->L = s->L;
    p->win_lo = s->depth_window > 0 ? s->L - s->depth_window : 0;
    p->Lw = p->L - p->win_lo;
    p->scale_log2 = (s->softmax_scale > 0.0f ? s->softmax_scale : 1.0f / std::sqrt(float(s->d))) * 1.4426950408889634f;
    return MODA_OK;
}

moda_status check_ptrs(std::initializer_list<std::pair<const void*, const char*>> ptrs) {
    char msg[120];
    for (const auto& pr : ptrs) {
        if (!pr.first) {
            snprintf(msg, sizeof(msg), "%s is NULL", pr.second);
            return api_fail(MODA_ERR_INVALID_ARG, msg);
        }
        if ((reinterpret_cast<uintptr_t>(pr.first) & 15u) != 0) {
            snprintf(msg, sizeof(msg), "%s is not 16-byte aligned", pr.second);
            return api_fail(MODA_ERR_MISALIGNED, msg);
        }
    }
    return MODA_OK;
}

moda_status launched(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return MODA_OK;
    char msg[200];
    snprintf(msg, sizeof(msg), "%s: %s", what, cudaGetErrorString(e));
    return api_fail(MODA_ERR_CUDA, msg);
}

moda_status too_many_tiles() {
    return failf(MODA_ERR_UNSUPPORTED, "the block table's length times N passes 2^31 tiles");
}

moda_status no_device() { return api_fail(MODA_ERR_CUDA, "no usable CUDA device"); }

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Nothing may be thrown across the C ABI (a full host heap, a broken mutex).
template <typename F>
moda_status guarded(F&& f) noexcept {
    try {
        return f();
    } catch (...) {
        return MODA_ERR_CUDA;
    }
}

}  // namespace

// The most the schedule's costs can add up to: every request at the table's
// length, every new token's depth rows in a tile of their own.
static double most_cost(const Paged& p, const TreePlan& t) {
    const double groups = p.B + double(p.N) / t.Tg;
    return p.Hk * (groups * ((double(p.max_pages) * p.page / t.KT + 1) * t.tiles + t.job_cost) +
                   double(p.N) * t.dsplit);
}

TreePlan tree_plan(const Paged& p) {
    TreePlan t;
    // tokens of a request, on average
    const int per = p.B > 0 ? static_cast<int>((static_cast<long long>(p.N) + p.B - 1) / p.B) : p.N;
    const int Lw = p.Lw > 0 ? p.Lw : 1;
    t.tiles = 1;
    if (p.elem_bytes == 2) {           // tensor cores: 128-row tiles, one CTA an SM
        t.rows = t.KT = 128;
        t.Tq = t.rows / p.G;
        // Two row tiles a job read the keys once for 256 rows, but leave two score
        // buffers instead of three, and a job's blocks run one after the other on one
        // SM.  Where requests fill more than one tile and the cache (as far as the
        // shape tells) is more than L2 keeps, the bytes win, the sooner the more tiles
        // read them again.  G = 4, d = 128, 8 heads, 8 requests, one tile against two:
        // n = 64 over 4096 keys (cache of 137 MB) 65, 71 us; 8192 (270 MB) 98, 103; 9000
        // (297 MB) 108, 106; 10500 127, 118; 32768 362, 301.  n = 128 over 4096 101, 113;
        // 8192 196, 176.  n = 256 over 4096 (143 MB) 185, 191; 8192 347, 326.  n = 1000 over
        // 4096 (167 MB) 818, 789.  With d = 64 a tile's bytes are half and its exponentials
        // the same: n = 64 over 32768 257, 272.
        // The lengths are on the device: what counts here is the pool and the table, and all N
        // rows.  Where those are much larger than what the requests hold, two tiles are taken
        // for short requests too (n = 64 over 4096 keys: 75 us in a pool of 4 GB and a table of
        // 128K tokens, 65 in a tight one; n = 128 123, 113).
        const double pages = double(p.B) * p.max_pages < p.n_pages ? double(p.B) * p.max_pages : p.n_pages;
        const double cache = pages * p.page * p.Hk * p.d * 2 * p.elem_bytes;
        t.tiles = per > t.Tq && p.d == 128 && cache > (per > 2 * t.Tq ? 160e6 : 280e6) ? 2 : 1;
        t.Lp = (Lw + 7) / 8 * 8;       // a token's depth rows begin on a swizzle atom
        t.n_cta = device_sm_count();
    } else {
        t.KT = 32;
        const long long rows = static_cast<long long>(per) * p.G;     // of a request and KV head
        // (a block of more rows than there are costs their arithmetic: 8 requests, G = 4, d = 128,
        // T = 8192: n = 1 in blocks of 4, 16, 64 rows 143, 228, 524 us; n = 4 in 16, 64 232, 526.
        // N counts padding rows: 8 requests of one token padded to 64 rows take blocks of 64,
        // 269 us: warps without a row skip the work)
        t.rows = p.G <= 4 && rows <= 4 ? 4 : (p.G <= 16 && rows <= 16 ? 16 : 64);
        t.Tq = t.rows / p.G;
        t.Lp = Lw;
        t.n_cta = 2 * device_sm_count();
    }
    // A job's beginning in tiles.  Uneven requests, job_cost = 0, 1, 2, 3, 4: bf16, 48 of up
    // to 64 tokens over 4096 keys 98, 92, 88, 87, 87 us; 32 of up to 200 161, 154, 143, 141,
    // 138; fp32, 64 of one token over 1000 keys 70, 64, 57, 56, 58; even ones: no change.
    t.job_cost = 3;
    t.Tg = t.Tq * t.tiles;
    t.dtok = Lw <= t.KT ? t.KT / t.Lp : 1;
    t.dsplit = (Lw + t.KT - 1) / t.KT;
    const long long rows = static_cast<long long>(p.N) * p.G;
    t.rec_rows = rows < static_cast<long long>(t.Tg) * p.G ? static_cast<int>(rows) : t.Tg * p.G;
    t.off_ml = round256(sizeof(tree::CtaHeader) * t.n_cta);
    t.off_po = t.off_ml + round256(sizeof(float2) * 2 * t.n_cta * t.rec_rows);
    t.bytes = 256 + t.off_po + round256(sizeof(float) * 2 * t.n_cta * t.rec_rows * p.d);
    return t;
}

}  // namespace moda

using namespace moda;

extern "C" {

moda_status moda_page_plan(const moda_paged_shape* shape, const int* held_len, const int* want_len,
                           int* block_table, int* free_pages, int* free_count, int* cu_new,
                           int* granted_len, long long* slot_map, moda_stream_t stream) {
    return guarded([&]() -> moda_status {
        Paged p{};
        moda_status st = check_pages(shape, &p);
        if (st != MODA_OK) return st;
        if (p.B > kMaxPlanRequests)
            return failf(MODA_ERR_UNSUPPORTED, "moda_page_plan supports B <= %lld (B=%lld)", kMaxPlanRequests, p.B);
        if ((st = check_ptrs({{free_pages, "free_pages"}, {free_count, "free_count"}, {cu_new, "cu_new"}})) != MODA_OK)
            return st;
        if (p.B > 0 && (st = check_ptrs({{held_len, "held_len"}, {want_len, "want_len"}, {block_table, "block_table"},
                                         {granted_len, "granted_len"}})) != MODA_OK)
            return st;
        if (p.N > 0 && (st = check_ptrs({{slot_map, "slot_map"}})) != MODA_OK) return st;
        if (p.B > 0 && (granted_len == held_len || granted_len == want_len))
            return failf(MODA_ERR_INVALID_ARG, "granted_len must not alias held_len or want_len");
        PlanArgs a;
        a.held = held_len; a.want = want_len; a.table = block_table; a.free_pages = free_pages;
        a.free_count = free_count; a.cu = cu_new; a.granted = granted_len; a.slots = slot_map;
        a.status = device_status_word();
        if (!a.status) return no_device();
        a.B = p.B; a.N = p.N; a.page_shift = p.page_shift; a.n_pages = p.n_pages; a.max_pages = p.max_pages;
        const cudaError_t e = launch_plan(a, reinterpret_cast<cudaStream_t>(stream));
        return launched(e, "page plan launch");
    });
}

moda_status moda_cache_append(const moda_paged_shape* shape, const void* k_new, const void* v_new,
                              const long long* slot_map, void* k_cache, void* v_cache,
                              moda_stream_t stream) {
    return guarded([&]() -> moda_status {
        Paged p{};
        moda_status st;
        if ((st = check_pages(shape, &p)) != MODA_OK || (st = check_cache(shape, &p)) != MODA_OK) return st;
        if (p.N == 0) return MODA_OK;
        if ((st = check_ptrs({{k_new, "k_new"}, {v_new, "v_new"}, {slot_map, "slot_map"}, {k_cache, "k_cache"},
                              {v_cache, "v_cache"}})) != MODA_OK)
            return st;
        AppendArgs a;
        a.k = static_cast<const uint4*>(k_new); a.v = static_cast<const uint4*>(v_new);
        a.kc = static_cast<uint4*>(k_cache); a.vc = static_cast<uint4*>(v_cache);
        a.slots = slot_map;
        a.status = device_status_word();
        if (!a.status) return no_device();
        const long long row_chunks = static_cast<long long>(p.Hk) * (p.d * p.elem_bytes / 16);
        if (row_chunks > (1 << 24)) return failf(MODA_ERR_UNSUPPORTED, "Hk=%lld too large", p.Hk);
        a.Hk = p.Hk;
        a.head_chunks = p.d * p.elem_bytes / 16;
        a.row_chunks = static_cast<int>(row_chunks);
        a.page_shift = p.page_shift;
        a.n_slots = static_cast<long long>(p.n_pages) << p.page_shift;
        a.n_chunks = row_chunks * p.N;
        const long long per = kAppendThreads * kAppendUnroll;
        const long long grid = (a.n_chunks + per - 1) / per;
        if (grid > 0x7fffffffll) return failf(MODA_ERR_UNSUPPORTED, "N=%lld tokens are too many for one call", p.N);
        return launched(launch_dependent(cache_append_kernel, static_cast<unsigned>(grid), kAppendThreads, 0, 1,
                                         reinterpret_cast<cudaStream_t>(stream), a),
                        "cache append launch");
    });
}

moda_status moda_tree_mask(const moda_paged_shape* shape, const int* parent, const int* cu_new,
                           const int* held_len, unsigned int* mask, int* position,
                           moda_stream_t stream) {
    return guarded([&]() -> moda_status {
        Paged p{};
        moda_status st;
        if ((st = check_pages(shape, &p)) != MODA_OK || (st = check_words(shape, &p, true)) != MODA_OK) return st;
        if (p.B == 0 || p.N == 0) return MODA_OK;
        if ((st = check_ptrs({{parent, "parent"}, {cu_new, "cu_new"}, {mask, "mask"}, {position, "position"}})) != MODA_OK)
            return st;
        if (held_len && (st = check_ptrs({{held_len, "held_len"}})) != MODA_OK) return st;
        MaskArgs a;
        a.parent = parent; a.cu = cu_new; a.held = held_len; a.mask = mask; a.position = position;
        a.status = device_status_word();
        if (!a.status) return no_device();
        a.B = p.B; a.N = p.N; a.words = p.words;
        return launched(launch_dependent(tree_mask_kernel,
                                         dim3(p.B, (32 * p.words + kMaskThreads - 1) / kMaskThreads), kMaskThreads, 0, 1,
                                         reinterpret_cast<cudaStream_t>(stream), a),
                        "tree mask launch");
    });
}

size_t moda_tree_decode_workspace_size(const moda_paged_shape* shape) {
    size_t bytes = static_cast<size_t>(-1);
    guarded([&]() -> moda_status {
        Paged p{};
        const moda_status st = check_tree(shape, &p);
        if (st != MODA_OK) return st;
        const TreePlan t = tree_plan(p);
        if (p.B > 0 && p.N > 0 && most_cost(p, t) > 2147483647.0) return too_many_tiles();
        bytes = p.B == 0 || p.N == 0 ? 0 : t.bytes;
        return st;
    });
    return bytes;
}

moda_status moda_tree_decode(const moda_paged_shape* shape, const void* q, const void* k_cache,
                             const void* v_cache, const void* Kd, const void* Vd,
                             const int* block_table, const int* held_len, const int* cu_new,
                             const unsigned int* mask, void* o, float* lse, void* ws,
                             size_t ws_bytes, moda_stream_t stream) {
    return guarded([&]() -> moda_status {
        Paged p{};
        moda_status st = check_tree(shape, &p);
        if (st != MODA_OK) return st;
        if (p.B == 0 || p.N == 0) return MODA_OK;
        if ((st = check_ptrs({{q, "q"}, {k_cache, "k_cache"}, {v_cache, "v_cache"}, {block_table, "block_table"},
                              {held_len, "held_len"}, {cu_new, "cu_new"}, {o, "o"}, {lse, "lse"}, {ws, "ws"}})) != MODA_OK)
            return st;
        if (p.L > 0 && (st = check_ptrs({{Kd, "Kd"}, {Vd, "Vd"}})) != MODA_OK) return st;
        if ((mask != nullptr) != (p.words > 0))
            return failf(MODA_ERR_INVALID_ARG, "a mask needs mask_words >= 1, and mask_words = 0 (a chain) no mask "
                         "(mask_words=%lld)", p.words);
        if (mask && (st = check_ptrs({{mask, "mask"}})) != MODA_OK) return st;
        unsigned int* status = device_status_word();
        if (!status) return no_device();
        const TreePlan t = tree_plan(p);
        if (most_cost(p, t) > 2147483647.0) return too_many_tiles();
        if (ws_bytes < t.bytes)
            return failf(MODA_ERR_WORKSPACE, "moda_tree_decode needs %lld bytes of workspace (got %lld)",
                         static_cast<long long>(t.bytes), static_cast<long long>(ws_bytes));
        tree::TreeArgs a;
        std::memset(&a, 0, sizeof(a));
        a.q = q; a.kc = k_cache; a.vc = v_cache; a.kd = Kd; a.vd = Vd;
        a.table = block_table; a.held = held_len; a.cu = cu_new; a.mask = mask;
        a.o = o; a.lse = lse;
        // (whole 256-byte lines of a workspace that need only be 16-byte aligned)
        unsigned char* base =
            reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(ws) + 255) & ~uintptr_t(255));
        a.hdr = reinterpret_cast<tree::CtaHeader*>(base);
        a.ml = reinterpret_cast<float2*>(base + t.off_ml);
        a.po = reinterpret_cast<float*>(base + t.off_po);
        a.status = status;
        a.B = p.B; a.N = p.N; a.Hq = p.Hq; a.Hk = p.Hk; a.G = p.G; a.L = p.L; a.Lw = p.Lw; a.win_lo = p.win_lo;
        a.page_shift = p.page_shift; a.n_pages = p.n_pages; a.max_pages = p.max_pages; a.words = p.words;
        a.Tq = t.Tq; a.Tg = t.Tg; a.KT = t.KT; a.Lp = t.Lp; a.dtok = t.dtok; a.dsplit = t.dsplit;
        a.two_cost = t.tiles;
        a.job_cost = t.job_cost;
        while ((1 << a.kt_shift) < t.KT) ++a.kt_shift;
        a.rec_rows = t.rec_rows; a.n_cta = t.n_cta; a.scale_log2 = p.scale_log2;
        cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
        phase_mark(0, s);
        cudaError_t e = p.elem_bytes == 2 ? launch_tree_sm100(p, t, a, s) : launch_tree_simt(p, t, a, s);
        if (e == cudaSuccess) e = launch_tree_combine(p, t, a, s);
        if (e == cudaSuccess) phase_mark(1, s);
        return launched(e, "tree decode launch");
    });
}

}  // extern "C"
