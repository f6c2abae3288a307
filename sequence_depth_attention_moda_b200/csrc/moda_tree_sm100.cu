// moda_tree_sm100.cu -- attention of drafted tokens over a paged cache on the
// tensor cores, bf16 (the operator, the schedule and the masks: moda_tree.cuh;
// the formulas: moda_tree_simt.cu).
//
// Bound: HBM.  A cached key and value row (4 d bytes) is read once and costs
// 4 d R operations for the R rows of a job, so up to R = 128 rows the tensor
// cores need less than half of the time the bytes take, and they do not mind
// that few of their 128 rows are real; at R = 256 the two are about even.
//
// One CTA per SM over a contiguous range of the flattened list of 128-key
// tiles, which it streams through a K ring and a V ring.  A job has one or two
// query tiles of 128 rows; a block is one key tile against one query tile, and
// a sequence tile is loaded once for both of a job's query tiles (two blocks),
// a depth tile holds one query tile's tokens (one block).  Two instances: jobs
// of one query tile (NQ = 1), and of up to two, where those of one use the two
// query slots (shared memory) and O accumulators (TMEM) in turn.  tree_plan
// chooses and has the figures.
//
// Warps: 0 TMA producer (Q, K; a lane a page or a token, so pages as small
// as 8 rows cost one issue each); 1 TMA producer of V; 2 issues S = Q K^T, up to
// the number of S buffers ahead; 3 issues O += P V; 4..11 softmax, 16 rows a warp
// and two threads a row (columns [0,64) and [64,128)): O and l are rescaled only
// when the maximum passes the reference by more than 2^8 (exact: any reference
// gives the same quotient), P in bf16 over the score columns.  Warps without a
// real row, and in depth tiles those whose tokens are not in the tile, skip the
// work.
// TMEM columns: S buffers from 0 (three, or two where jobs may have two query
// tiles), then an O accumulator of d for each slot.
//
// A tile that ends a request's keys leaves rows of the V stage unwritten (pages
// behind the last key are not loaded) or with what the page held; P is 0 there,
// but 0 * NaN is not, so the softmax warps store zeros (16 rows each), before P
// of the tile's first block is announced.  In rows that only some of the query
// rows see (new keys, depth rows) they replace infinities and NaN and mark the
// segment (add_not_finite).  Tiles of held keys pass untouched.
//
// Measured (32 query heads over 8, d 128, 48 depth rows, 8 requests of 32768 keys):
// 1 token 168 to 174 us inside a graph, 6.2 TB/s, where the bytes alone take 164, and 181
// to 186 among calls on changing inputs through the Python binding; 32 tokens 190 to 205,
// and 224 to 230 once the power cap has brought the clock to 1.4 GHz: a tile's block then
// takes the softmax warps as long as HBM its bytes.  A block takes about 2000 cycles, of
// which 1024 are exponentials (16 a cycle) and 1024 tensor work; the rest is latency
// of two warps a sub-partition.  48 ragged requests of up to 64 tokens over 4096 keys
// 82 to 89 us inside a graph, 92 on changing inputs (the bytes 41), 11 of them before the
// first block.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "moda_tree.cuh"

namespace moda {
namespace {

using namespace ptx;
using namespace tree;

constexpr int kTile = 128;                   // keys per tile, rows per query tile
constexpr int kThreads = 384;
constexpr int kSoftmaxWarps = 8;
constexpr uint32_t kSlab = 128 * 128;        // 128 rows x 64 bf16
constexpr uint32_t kTmemCols = 512;
constexpr float kLazy = 8.0f;                // log2 by which a maximum may pass the reference
constexpr int kMarks = 2;                    // segments whose marks are told apart: a warp marks segment k+1
                                             // only when all have begun to write out segment k

// A segment: the tiles of one job that this CTA owns.  Warp 0 walks the jobs and
// publishes their segments in a ring in shared memory, so that the walk's code
// and its reads of lengths exist once.  Warp 0 is ahead of the slowest role by at
// most a K ring and the S buffers in tiles, each of which may be a segment: the
// ring is longer than that, and no one has to say that a segment is done with.
struct Seg {
    Request r;
    int b, hk, tok0, ntok, nseq, ndep0, keys;
    int i0, i1;          // its tiles; i1 < 0: there are no more segments
    int whole, slot;     // see Walk
    int pad[2];
};
constexpr int kSegs = 16;

// NQ: query tiles of a job, and O accumulators.
template <int D, int NQ>
struct Lay {
    static constexpr int kSlabs = D / 64;
    static constexpr uint32_t kTileBytes = kSlabs * kSlab;
    // all of shared memory: V stages are held until P V is done, K stages only until S is
    static constexpr int kKS = D == 64 ? 6 : (NQ == 1 ? 3 : 2);
    static constexpr int kVS = D == 64 ? 7 : 3;
    static constexpr int kNS = NQ == 2 ? 2 : 3;             // S buffers
    static constexpr uint32_t kColO = kNS * 128;            // O of slot s: + s * D
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = NQ * kTileBytes;
    static constexpr uint32_t kV = kK + kKS * kTileBytes;
    static constexpr uint32_t kBar = kV + kVS * kTileBytes;
    // barrier indexes; from kPReady on they take an arrival of each softmax warp
    static constexpr int kQFull = 0, kQFree = NQ, kKFull = 2 * NQ, kKEmpty = kKFull + kKS, kVFull = kKEmpty + kKS,
                         kVEmpty = kVFull + kVS, kSFull = kVEmpty + kVS, kSFree = kSFull + kNS,
                         kOFull = kSFree + kNS, kSegFull = kOFull + NQ, kPReady = kSegFull + kSegs,
                         kOFree = kPReady + kNS, kNumBars = kOFree + NQ;
    static constexpr uint32_t kStart = kBar + (kNumBars * 8 + 15) / 16 * 16;
    static constexpr uint32_t kSeg = kStart + (sizeof(Start) + 15) / 16 * 16;
    static constexpr uint32_t kMisc = kSeg + kSegs * sizeof(Seg);       // tmem base, abort flag, marks
    static constexpr uint32_t kBytes = kMisc + 16 + kMarks * 4;
    static_assert(kColO + NQ * D <= kTmemCols, "TMEM columns");
    static_assert(kBytes <= 232448, "shared memory of one CTA");
    static_assert(kKS + kNS + 2 < kSegs && kVS + 2 < kSegs, "segments in flight");
};

struct SmArgs {
    TreeArgs t;
    TmaMap tq, tk, tv, tkd, tvd;
    int box_rows;        // rows of a cache box: min(page, 128)
    int wide;            // o is 32-byte aligned: rows are stored by whole sectors (else by
                         // halves: 105 us instead of 100 for 48 ragged requests)
};

// What the MMA and softmax roles derive alike while they go through the CTA's tiles.
// A slot is a query tile's place: shared memory for Q, TMEM for O.  Jobs of one
// query tile take the slots in turn.
template <int NQ>
struct Roles {
    int j = 0;           // tiles so far: ring stages, barrier phases
    int b = 0;           // blocks so far: S buffers, barrier phases
    int turn = 0;        // slot of the next job of one query tile
    int used0 = 0, used1 = 0;   // segments that used each slot so far
    bool two;            // two query tiles
    int first;           // slots first .. last
    int last;
    __device__ __forceinline__ void segment(const TreeArgs& a, const Seg& g) {
        two = NQ == 2 && g.ntok > a.Tq;
        first = two ? 0 : turn;
        last = two ? 1 : turn;
    }
    __device__ __forceinline__ int used(int s) const { return NQ == 2 && s ? used1 : used0; }
    // Query tile of slot s.
    __device__ __forceinline__ int sub(int s) const { return two ? s : 0; }
    // Whether slot s takes the job's tile i.
    __device__ __forceinline__ bool takes(const Seg& g, int i, int s) const {
        return !two || i < g.nseq || (i >= g.nseq + g.ndep0) == (s == 1);
    }
    __device__ __forceinline__ void end_segment() {
        used0 += first == 0;
        if (NQ == 2) {
            used1 += last == 1;
            if (!two) turn ^= 1;
        }
    }
};

// A depth tile's query tile, its index there, and a query tile's tokens.
__device__ __forceinline__ int dep_sub(const Seg& g, int i) { return i >= g.nseq + g.ndep0 ? 1 : 0; }
__device__ __forceinline__ int dep_index(const Seg& g, int i) {
    const int dt = i - g.nseq;
    return dt < g.ndep0 ? dt : dt - g.ndep0;
}
__device__ __forceinline__ int sub_tokens(const TreeArgs& a, const Seg& g, int sub) {
    return sub == 0 ? min(g.ntok, a.Tq) : g.ntok - a.Tq;
}

// Rows of tile i from its first on that its products have to cover.
__device__ __forceinline__ int tile_rows(const TreeArgs& a, const Seg& g, int i) {
    if (i < g.nseq) return min(kTile, g.keys - i * kTile);
    const int dt = dep_index(g, i);
    if (a.Lw <= kTile) return min(a.dtok, sub_tokens(a, g, dep_sub(g, i)) - dt * a.dtok) * a.Lp;
    return min(kTile, a.Lw - dt % a.dsplit * kTile);
}

// A lane's share of a tile's load: one box of a page, or of a token's depth rows.
struct Box {
    bool mine, dep, once;
    int c1, c2;          // coordinates (c0 is the slab)
    int row;             // first row in the tile
    uint32_t bytes;      // of the whole tile
};
// Table entry for this lane's box of tile i (0 where it has none).
__device__ __forceinline__ int box_entry(const TreeArgs& a, int box_rows, const Seg& g, int i, int lane) {
    if (i >= min(g.i1, g.nseq) || lane * box_rows >= min(kTile, g.keys - i * kTile)) return 0;
    return table_entry(a, g.b, i * kTile + lane * box_rows);
}
__device__ __forceinline__ Box tile_box(const TreeArgs& a, int box_rows, int slabs, const Seg& g, int i, int entry,
                                        int lane) {
    Box x;
    x.dep = i >= g.nseq;
    x.once = x.dep || g.r.n <= a.Tg;   // one group: no other job reads these keys
    x.mine = false;
    x.c1 = x.c2 = x.row = 0;
    if (!x.dep) {
        const int key = i * kTile + lane * box_rows;
        const int left = min(kTile, g.keys - i * kTile);
        x.mine = lane * box_rows < left;
        x.bytes = ((left + box_rows - 1) / box_rows) * box_rows * 128u * slabs;
        if (x.mine) {
            const int p = checked_page(a, entry);
            x.row = lane * box_rows;
            x.c1 = key & ((1 << a.page_shift) - 1);
            x.c2 = p < 0 ? -1 : p * a.Hk + g.hk;      // outside: the box reads as zeros
        }
        return x;
    }
    const int sub = dep_sub(g, i), dt = dep_index(g, i);
    const int tok = g.r.cu0 + g.tok0 + sub * a.Tq;
    if (a.Lw <= kTile) {
        const int cnt = min(a.dtok, sub_tokens(a, g, sub) - dt * a.dtok);
        x.mine = lane < cnt;
        x.bytes = cnt * a.Lw * 128u * slabs;
        x.row = lane * a.Lp;
        x.c1 = a.win_lo;
        x.c2 = (tok + dt * a.dtok + lane) * a.Hk + g.hk;
    } else {
        x.mine = lane == 0;
        x.bytes = kTile * 128u * slabs;                 // rows behind the last depth row read as zeros
        x.c1 = a.win_lo + dt % a.dsplit * kTile;
        x.c2 = (tok + dt / a.dsplit) * a.Hk + g.hk;
    }
    return x;
}

// Rows r0 .. r0+15 of a V stage (whole warp): clears those that P V covers but
// that are not there (from `rows` on; of every `pitch` rows those behind the
// first `used`), and takes infinities and NaN out of those from row `from` on,
// which are masked for some query row.  True if it found any.
template <int D>
__device__ __forceinline__ bool clean_values(unsigned char* stage, int r0, int rows, int from, int pitch, int used) {
    const int lane = threadIdx.x & 31;
    if (r0 >= rows || r0 + 16 <= from) return false;
    uint4* p = reinterpret_cast<uint4*>(stage) + r0 * 8 + lane;      // row r0 + 4u + lane/8, chunk lane%8 of a slab
    uint4 v[4 * (D / 64)];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int x = 0; x < D / 64; ++x) v[u * (D / 64) + x] = p[x * (kSlab / 16) + 32 * u];
    uint32_t acc[4] = {0u, 0u, 0u, 0u};
    if (r0 >= from && r0 + 16 <= rows && pitch == used) {            // all there, all masked for somebody
#pragma unroll
        for (int u = 0; u < 4 * (D / 64); ++u) {
            acc[0] = not_finite_acc(v[u].x, acc[0]);
            acc[1] = not_finite_acc(v[u].y, acc[1]);
            acc[2] = not_finite_acc(v[u].z, acc[2]);
            acc[3] = not_finite_acc(v[u].w, acc[3]);
        }
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int row = r0 + 4 * u + (lane >> 3);
            const bool there = row < rows && row % pitch < used;
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
                const uint4 y = v[u * (D / 64) + x];
                if (!there) {
                    p[x * (kSlab / 16) + 32 * u] = make_uint4(0, 0, 0, 0);
                } else if (row >= from) {
                    acc[0] = not_finite_acc(y.x, acc[0]);
                    acc[1] = not_finite_acc(y.y, acc[1]);
                    acc[2] = not_finite_acc(y.z, acc[2]);
                    acc[3] = not_finite_acc(y.w, acc[3]);
                }
            }
        }
        fence_proxy_async_smem();
    }
    const bool bad = __any_sync(0xffffffffu, ((acc[0] | acc[1] | acc[2] | acc[3]) & 0x7fff7fffu) != 0u);
    if (bad) {
#pragma unroll 1
        for (int y = 0; y < D / 16; ++y) {
            const int row = r0 + 4 * (y & 3) + (lane >> 3);
            if (row < from || row >= rows) continue;      // (a hole is zeros by now)
            uint4* q = p + (y >> 2) * (kSlab / 16) + 32 * (y & 3);
            uint4 v = *q;
            uint32_t* e = &v.x;
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                if ((e[z] & 0x7f80u) == 0x7f80u) e[z] &= 0xffff0000u;
                if ((e[z] & 0x7f800000u) == 0x7f800000u) e[z] &= 0x0000ffffu;
            }
            *q = v;
        }
    }
    if (bad) fence_proxy_async_smem();
    return bad;
}

// mask_visible of 64 keys.  (Its arguments are values: a reference to the kernel's
// parameters was read through memory.)
__device__ __forceinline__ uint2 mask_visible64(const uint32_t* row, int words, int n, int rel) {
    return make_uint2(mask_visible(row, words, n, rel), mask_visible(row, words, n, rel + 32));
}

template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, 1) tree_sm100_kernel(const __grid_constant__ SmArgs g) {
    using L = Lay<D, NQ>;
    const TreeArgs& a = g.t;
    extern __shared__ __align__(1024) unsigned char smem[];      // (TMA's and the descriptors' 128-byte swizzle)
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
    Start* start = reinterpret_cast<Start*>(smem + L::kStart);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    volatile int* marks = reinterpret_cast<volatile int*>(tmem_holder + 4);
    const int lane = threadIdx.x & 31;
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);    // known to be uniform

    // the combine kernel may be set up now; it waits for this grid on the device
    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kNumBars; ++i) mbar_init(&bars[i], i >= L::kPReady ? kSoftmaxWarps : 1);
        *abort_flag = 0;
        for (int i = 0; i < kMarks; ++i) marks[i] = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, kTmemCols);
        tmem_relinquish();
    }
    if (threadIdx.x == 64) {
        prefetch_tmap(&g.tq);
        prefetch_tmap(&g.tk);
        prefetch_tmap(&g.tv);
    }
    // Launched while the grid before it ends: nothing of it is read, and nothing
    // in memory written, before this.
    griddep_wait();
    tc_fence_before();
    schedule(a, start);        // ends with a CTA barrier
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    auto wait = [&](int bar, uint32_t phase) -> bool { return mbar_wait(&bars[bar], phase & 1, a.status, abort_flag); };
    auto wait_all = [&](int bar, uint32_t phase) -> bool { return __all_sync(0xffffffffu, wait(bar, phase)); };
    // Tiles that this call reads once leave L2 first: what else lives there (the
    // kernel's own code, tables, records) then survives a cache of many GB.
    const uint64_t once = policy_evict_first();
    // one box a lane: arms the stage's barrier for the whole tile, then loads
    auto load_tile = [&](const Box& x, int full, unsigned char* stage, const TmaMap* seq, const TmaMap* depth) {
        if (lane == 0) mbar_arrive_expect_tx(&bars[full], x.bytes);
        __syncwarp();
        if (x.mine) {
            unsigned char* dst = stage + x.row * 128;
#pragma unroll
            for (int y = 0; y < L::kSlabs; ++y) {
                if (x.once) tma_load_3d_hint(dst + y * kSlab, x.dep ? depth : seq, &bars[full], y * 64, x.c1, x.c2, once);
                else tma_load_3d(dst + y * kSlab, seq, &bars[full], y * 64, x.c1, x.c2);
            }
        }
    };
    // Every load lands before the CTA retires (bounded by time only: these
    // waits ignore the abort flag).
    auto drain = [&](int full, int stages, int issued) {
        int no_abort = 0;
        for (int x = max(0, issued - stages); x < issued; ++x)
            mbar_wait(&bars[full + x % stages], (x / stages) & 1, a.status, &no_abort);
    };

    Seg* segs = reinterpret_cast<Seg*>(smem + L::kSeg);
    Seg sg;
    int k = -1;              // segment
    // the next segment, or false; for a whole warp, and for one thread
    auto next_seg_all = [&]() -> bool {
        ++k;
        if (!wait_all(L::kSegFull + k % kSegs, k / kSegs)) return false;
        sg = segs[k % kSegs];
        return sg.i1 >= 0;
    };
    auto next_seg_one = [&]() -> bool {
        ++k;
        if (!wait(L::kSegFull + k % kSegs, k / kSegs)) return false;
        sg = segs[k % kSegs];
        return sg.i1 >= 0;
    };
    Roles<NQ> r;
    // 384 threads of 168 registers: 128 x 104 + 256 x 200, or 128 x 88 + 256 x 208
    // (two query tiles' statistics); local memory has next to no L1 beside this
    // much shared memory, so a spill in the block loop costs thousands of cycles
    if (warp < 4) {
        regs_dec<NQ == 1 ? 104 : 88>();
        if (warp == 0) {
            // ------------------------------------------------- producer of Q, K --
            const uint32_t q_bytes = L::kSlabs * 128u * a.Tq * a.G;
            bool ok = true;
            Walk w;
            for (bool more = w.begin(a, *start); ok; more = w.next(a)) {
                ++k;
                sg.r = w.j.r;
                sg.b = w.j.b;
                sg.hk = w.j.hk;
                sg.tok0 = w.j.tok0;
                sg.ntok = w.j.ntok;
                sg.nseq = w.j.nseq;
                sg.ndep0 = w.j.ndep0;
                sg.keys = w.j.r.held + (a.mask ? w.j.r.n : w.j.tok0 + w.j.ntok);
                sg.i0 = w.i0;
                sg.i1 = more ? w.i1 : -1;
                sg.whole = w.whole();
                sg.slot = w.slot();
                if (lane == 0) {
                    segs[k % kSegs] = sg;
                    mbar_arrive(&bars[L::kSegFull + k % kSegs]);
                }
                __syncwarp();
                if (!more) break;
                r.segment(a, sg);
                // table entries two tiles ahead: under load a read takes as long as a tile
                int e0 = box_entry(a, g.box_rows, sg, sg.i0, lane), e1 = box_entry(a, g.box_rows, sg, sg.i0 + 1, lane);
                for (int s = r.first; s <= r.last; ++s) {
                    if (r.used(s) > 0 && !wait_all(L::kQFree + s, r.used(s) - 1)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bars[L::kQFull + s], q_bytes);
                        for (int x = 0; x < L::kSlabs; ++x)
                            tma_load_3d(smem + L::kQ + s * L::kTileBytes + x * kSlab, &g.tq, &bars[L::kQFull + s], x * 64,
                                        sg.hk * a.G, sg.r.cu0 + sg.tok0 + r.sub(s) * a.Tq);
                    }
                }
                if (!ok) break;
                for (int i = sg.i0; i < sg.i1; ++i, ++r.j) {
                    const Box x = tile_box(a, g.box_rows, L::kSlabs, sg, i, e0, lane);
                    e0 = e1;
                    e1 = box_entry(a, g.box_rows, sg, i + 2, lane);
                    const int st = r.j % L::kKS;
                    if (r.j >= L::kKS && !wait_all(L::kKEmpty + st, r.j / L::kKS - 1)) {
                        ok = false;
                        break;
                    }
                    load_tile(x, L::kKFull + st, smem + L::kK + st * L::kTileBytes, &g.tk, &g.tkd);
                }
                r.end_segment();
            }
            if (lane == 0) {
                for (int s = 0; s < NQ; ++s)
                    if (r.used(s) > 0) drain(L::kQFull + s, 1, r.used(s));
                drain(L::kKFull, L::kKS, r.j);
            }
        } else if (warp == 1) {
            // ------------------------------------------------- producer of V -----
            bool ok = true;
            while (ok && next_seg_all()) {
                int e0 = box_entry(a, g.box_rows, sg, sg.i0, lane), e1 = box_entry(a, g.box_rows, sg, sg.i0 + 1, lane);
                for (int i = sg.i0; i < sg.i1; ++i, ++r.j) {
                    const Box x = tile_box(a, g.box_rows, L::kSlabs, sg, i, e0, lane);
                    e0 = e1;
                    e1 = box_entry(a, g.box_rows, sg, i + 2, lane);
                    const int st = r.j % L::kVS;
                    if (r.j >= L::kVS && !wait_all(L::kVEmpty + st, r.j / L::kVS - 1)) {
                        ok = false;
                        break;
                    }
                    load_tile(x, L::kVFull + st, smem + L::kV + st * L::kTileBytes, &g.tv, &g.tvd);
                }
            }
            if (lane == 0) drain(L::kVFull, L::kVS, r.j);
        } else if (warp == 2) {
            // ------------------------------------------------------ S = Q K^T -----
            if (elect_one()) {
                const uint32_t id = idesc_bf16(128, kTile, false, false);
                const uint64_t qd = desc_kmajor_sw128(smem_u32(smem + L::kQ));
                const uint64_t kd = desc_kmajor_sw128(smem_u32(smem + L::kK));
                bool ok = true;
                while (ok && next_seg_one()) {
                    r.segment(a, sg);
                    for (int s = r.first; ok && s <= r.last; ++s) ok = wait(L::kQFull + s, r.used(s));
                    for (int i = sg.i0; ok && i < sg.i1; ++i, ++r.j) {
                        const int st = r.j % L::kKS;
                        if (!(ok = wait(L::kKFull + st, r.j / L::kKS))) break;
                        for (int s = r.first; s <= r.last; ++s) {
                            if (!r.takes(sg, i, s)) continue;
                            // the buffer holds P of block b - kNS until its P V is done
                            const int sb = r.b % L::kNS;
                            if (r.b >= L::kNS && !(ok = wait(L::kSFree + sb, r.b / L::kNS - 1))) break;
                            tc_fence_after();
                            const uint64_t q0 = qd + ((s * L::kTileBytes) >> 4);
                            const uint64_t k0 = kd + ((st * L::kTileBytes) >> 4);
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint64_t off = ((kk >> 2) * kSlab + (kk & 3) * 32) >> 4;
                                umma_ss(tmem + sb * 128, q0 + off, k0 + off, id, kk > 0 ? 1u : 0u);
                            }
                            umma_commit(&bars[L::kSFull + sb]);
                            ++r.b;
                        }
                        if (ok) umma_commit(&bars[L::kKEmpty + st]);
                    }
                    if (ok)
                        for (int s = r.first; s <= r.last; ++s) umma_commit(&bars[L::kQFree + s]);
                    r.end_segment();
                }
            }
            __syncwarp();
        } else if (warp == 3) {
            // ------------------------------------------------------ O += P V ------
            if (elect_one()) {
                const uint32_t id = idesc_bf16(128, D, false, true);
                const uint64_t vd = desc_mnmajor_sw128(smem_u32(smem + L::kV), kSlab);
                bool ok = true;
                while (ok && next_seg_one()) {
                    r.segment(a, sg);
                    // the slots' accumulators must have been read out
                    for (int s = r.first; ok && s <= r.last; ++s)
                        if (r.used(s) > 0) ok = wait(L::kOFree + s, r.used(s) - 1);
                    int begun = 0;                        // slots with a product in this segment (bits)
                    for (int i = sg.i0; ok && i < sg.i1; ++i, ++r.j) {
                        const int st = r.j % L::kVS;
                        const int steps = (tile_rows(a, sg, i) + 15) / 16;     // 16 keys each
                        if (!(ok = wait(L::kVFull + st, r.j / L::kVS))) break;
                        for (int s = r.first; s <= r.last; ++s) {
                            if (!r.takes(sg, i, s)) continue;
                            const int sb = r.b % L::kNS;
                            if (!(ok = wait(L::kPReady + sb, r.b / L::kNS))) break;
                            tc_fence_after();
                            const uint64_t v0 = vd + ((st * L::kTileBytes) >> 4);
                            if (steps == kTile / 16) {
#pragma unroll
                                for (int kk = 0; kk < kTile / 16; ++kk)
                                    umma_ts(tmem + L::kColO + s * D, tmem + sb * 128 + kk * 8, v0 + kk * (2048 >> 4), id,
                                            (begun >> s & 1) || kk > 0 ? 1u : 0u);
                            } else {
#pragma unroll 1
                                for (int kk = 0; kk < steps; ++kk)
                                    umma_ts(tmem + L::kColO + s * D, tmem + sb * 128 + kk * 8, v0 + kk * (2048 >> 4), id,
                                            (begun >> s & 1) || kk > 0 ? 1u : 0u);
                            }
                            umma_commit(&bars[L::kSFree + sb]);
                            begun |= 1 << s;
                            ++r.b;
                        }
                        if (ok) umma_commit(&bars[L::kVEmpty + st]);
                    }
                    if (ok)
                        for (int s = r.first; s <= r.last; ++s) umma_commit(&bars[L::kOFull + s]);
                    r.end_segment();
                }
            }
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------ softmax -------
        regs_inc<NQ == 1 ? 200 : 208>();
        const int quarter = warp & 3;                 // TMEM lanes 32*quarter ..
        const int half = lane >> 4;                   // column half of the row
        const int row0 = quarter * 32 + ((warp - 4) >> 2) * 16;     // the warp's 16 rows
        const int row = row0 + (lane & 15);
        const int t_off = row / a.G;                  // token within the query tile
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(row0) << 16);
        const float sl2 = a.scale_log2;
        bool ok = true;
        while (ok && next_seg_all()) {
            r.segment(a, sg);
            float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;   // per slot; l: this half's share
            int prev0 = -1, prev1 = -1;               // the slot's last block in this segment
            const int n_tok0 = sub_tokens(a, sg, 0), n_tok1 = r.two ? sub_tokens(a, sg, 1) : n_tok0;
            // One block: slot s, tile i; `masks`: some key of the tile is hidden from some row.
            // `clean`: the tile's values are looked over here (a tile's first block does).
            // (One instance, in one loop: short jobs pay for every line of code they touch.)
            auto block = [&](bool masks, int i, int s, int n_tok, float& m, float& l, int& prev, bool clean) -> bool {
                const int sb = r.b % L::kNS;
                if (!wait_all(L::kSFull + sb, r.b / L::kNS)) return false;
                tc_fence_after();
                uint32_t pk[32];
                const bool active = row0 < n_tok * a.G;    // some row of the warp is real
                const uint32_t s_addr = lane_base + sb * 128;
                if (active) {
                    const bool real = t_off < n_tok && t_off < a.Tq;
                    uint32_t vis0 = 0xffffffffu, vis1 = 0xffffffffu;   // of this thread's 64 columns
                    bool blind = false;               // none of the warp's tokens is in this depth tile
                    if (masks) {
                        const bool dep = i >= sg.nseq;
                        if (real) {
                            const int c = half * 64;
                            if (dep) {
                                const int dt = dep_index(sg, i);
                                vis0 = dep_visible(a, t_off, dt, c);
                                vis1 = dep_visible(a, t_off, dt, c + 32);
                            } else {
                                const int token = sg.tok0 + r.sub(s) * a.Tq + t_off;
                                const int rel = i * kTile + c - sg.r.held;
                                if (a.mask) {
                                    const uint2 v = mask_visible64(
                                        a.mask + static_cast<size_t>(sg.r.cu0 + token) * a.words, a.words, sg.r.n, rel);
                                    vis0 = v.x;
                                    vis1 = v.y;
                                } else {
                                    vis0 = chain_visible(sg.r.n, token, rel);
                                    vis1 = chain_visible(sg.r.n, token, rel + 32);
                                }
                            }
                        }
                        blind = dep && !__any_sync(0xffffffffu, real && (vis0 | vis1));
                    }
                    if (blind) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) pk[e] = 0u;
                    } else {
                        uint32_t x[64];
                        tmem_ld16x2_32<64>(s_addr, x);
                        tmem_ld16x2_32<64>(s_addr + 32, x + 32);
                        tmem_wait_ld();
                        reg_fence<64>(x);
                        if (masks) {
#pragma unroll
                            for (int e = 0; e < 64; ++e)
                                if (!((e < 32 ? vis0 : vis1) >> (e & 31) & 1)) x[e] = __float_as_uint(-INFINITY);
                        }
                        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < 64; e += 8)
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                mx[u] = fmax3(mx[u], __uint_as_float(x[e + 2 * u]), __uint_as_float(x[e + 2 * u + 1]));
                        // this half row's maximum: whether it passes the reference needs no
                        // word from the other half (a row's first key: m = -inf)
                        float mn = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
                        if (__any_sync(0xffffffffu, real && mn > m + kLazy)) {
                            mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 16));
                            mn = fmaxf(m, mn);
                            // o and l are 0 until a key is seen
                            const float alpha = m == -INFINITY ? 1.0f : ex2(m - mn);
                            l *= alpha;
                            m = mn;
                            if (prev >= 0) {
                                // O must hold the sum up to the slot's last block.  Blocks up to b - kNS are
                                // done (their buffer's reuse waited for them); a later one's barrier can
                                // not have moved on, since the next use of its buffer needs a later P.
                                if (prev > r.b - L::kNS && !wait_all(L::kSFree + prev % L::kNS, prev / L::kNS)) return false;
                                tc_fence_after();
#pragma unroll 1
                                for (int c = 0; c < D / 2; c += 32) {
                                    uint32_t o[32];
                                    const uint32_t at = lane_base + L::kColO + s * D + c;
                                    tmem_ld16x2_32<D / 2>(at, o);
                                    tmem_wait_ld();
                                    reg_fence<32>(o);
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                    tmem_st16x2_32<D / 2>(at, o);
                                }
                                tmem_wait_st();
                            }
                        }
                        // p = 2^(s sl2 - m), packed
                        const float ref = m == -INFINITY ? 0.0f : m;     // a row that sees nothing yet: p = 0
                        // (multiply-adds and sums two at a time: 3% of the whole where blocks bound it)
                        const uint64_t sl22 = pack2(sl2, sl2), ref2 = pack2(-ref, -ref);
                        uint64_t rs[2] = {0, 0};
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float p0, p1;
                            unpack2(fma2(pack2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), sl22, ref2),
                                    p0, p1);
                            p0 = ex2(p0);
                            p1 = ex2(p1);
                            rs[e & 1] = add2(rs[e & 1], pack2(p0, p1));
                            pk[e] = pack_bf16(p0, p1);
                        }
                        float l0, l1;
                        unpack2(add2(rs[0], rs[1]), l0, l1);
                        l += l0 + l1;
                    }
                }
                if (active) {
                    __syncwarp();
                    tmem_st16x2_32<32>(s_addr, pk);
                    tmem_wait_st();
                }
                if (masks) {
                    // S of this tile is done, so P V of tile j - kVS is, and the stage's phase is this tile's
                    if (clean) {
                        const int st = r.j % L::kVS;
                        if (!wait_all(L::kVFull + st, r.j / L::kVS)) return false;
                        const bool dep = i >= sg.nseq;
                        const bool bad = clean_values<D>(smem + L::kV + st * L::kTileBytes, (warp - 4) * 16,
                                                         tile_rows(a, sg, i), dep ? 0 : sg.r.held - i * kTile,
                                                         dep && a.Lw <= kTile ? a.Lp : kTile,
                                                         dep && a.Lw <= kTile ? a.Lw : kTile);
                        if (bad && lane == 0) marks[k % kMarks] = k + 1;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[L::kPReady + sb]);
                prev = r.b++;
                return true;
            };
            const int open = sg.r.held / kTile;       // tiles of held keys alone come first
            // the mask rows are wanted only then, and from L1
            if (a.mask && row0 + (lane & 15) < min(sg.ntok, a.Tg) * a.G) {
                const uint32_t* m = a.mask + static_cast<size_t>(sg.r.cu0 + sg.tok0 + t_off) * a.words;
                for (int x = half * 32; x < a.words; x += 64) prefetch_l1(m + x);
            }
            for (int i = sg.i0; ok && i < sg.i1; ++i, ++r.j) {
                const bool masks = i >= open;
                bool clean = masks;
#pragma unroll 1
                for (int s = r.first; ok && s <= r.last; ++s) {
                    if (masks && !r.takes(sg, i, s)) continue;
                    if (NQ == 1) {
                        ok = block(masks, i, 0, n_tok0, m0, l0, prev0, clean);
                    } else {
                        float m = s ? m1 : m0, l = s ? l1 : l0;
                        int prev = s ? prev1 : prev0;
                        ok = block(masks, i, s, s ? n_tok1 : n_tok0, m, l, prev, clean);
                        if (s) m1 = m, l1 = l, prev1 = prev;
                        else m0 = m, l0 = l, prev0 = prev;
                    }
                    clean = false;
                }
            }
            // ------------------------------------------------ end of segment --
            const bool whole = sg.whole != 0;
#pragma unroll 1
            for (int s = r.first; ok && s <= r.last; ++s) {
                if (!wait_all(L::kOFull + s, r.used(s))) {
                    ok = false;
                    break;
                }
                const float m = s ? m1 : m0, l = s ? l1 : l0;
                tc_fence_after();
                const int n_tok = sub_tokens(a, sg, r.sub(s));
                const bool real = t_off < n_tok && t_off < a.Tq;
                const bool poison = marks[k % kMarks] == k + 1;
                const float lt = l + __shfl_xor_sync(0xffffffffu, l, 16);
                const int token = sg.tok0 + r.sub(s) * a.Tq + t_off;
                const size_t orow = static_cast<size_t>(sg.r.cu0 + token) * a.Hq + sg.hk * a.G + (row - t_off * a.G);
                const size_t rec = static_cast<size_t>(sg.slot) * a.rec_rows + r.sub(s) * a.Tq * a.G + row;
                const bool some = row0 < n_tok * a.G && (s ? prev1 : prev0) >= 0;    // O of these rows was written
                uint32_t o[D / 2];
                if (some) {
#pragma unroll
                    for (int c = 0; c < D / 2; c += 32) tmem_ld16x2_32<D / 2>(lane_base + L::kColO + s * D + c, o + c);
                    tmem_wait_ld();
                    reg_fence<D / 2>(o);
                }
                // O is in registers: the slot's next job may overwrite it
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[L::kOFree + s]);
                if (real && whole) {
                    const float inv = lt == 0.0f ? 0.0f : 1.0f / lt;
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + orow * D + half * (D / 2);
#pragma unroll
                    for (int c = 0; c < D / 2; c += 16) {
                        uint32_t v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[e] = pack_bf16(__uint_as_float(o[c + 2 * e]) * inv, __uint_as_float(o[c + 2 * e + 1]) * inv);
                        if (g.wide) {
                            store32(dst + c, v);
                        } else {
                            *reinterpret_cast<uint4*>(dst + c) = make_uint4(v[0], v[1], v[2], v[3]);
                            *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(v[4], v[5], v[6], v[7]);
                        }
                    }
                    if (half == 0) a.lse[orow] = row_lse(m, lt);
                } else if (real) {
                    if (some) {
                        float* dst = a.po + rec * D + half * (D / 2);
#pragma unroll
                        for (int c = 0; c < D / 2; c += 8) store32(dst + c, o + c);
                    }
                    // a slot without a block here (only depth tiles of the other one): an empty record
                    if (half == 0) a.ml[rec] = make_float2(m, poison ? -lt : lt);
                }
                if (poison && whole && row0 < n_tok * a.G) {
                    __syncwarp();
                    add_not_finite<__nv_bfloat16, D, 8>(a, sg.r, sg.b, sg.hk, sg.tok0 + r.sub(s) * a.Tq, row0, 1,
                                                         min(16, n_tok * a.G - row0));
                }
            }
            r.end_segment();
        }
    }
    __syncwarp();        // a barrier counts a warp when the first of its lanes arrives
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D, int NQ>
cudaError_t launch_d(const Paged& p, const TreePlan& t, const TreeArgs& a, cudaStream_t s) {
    SmArgs g;
    g.t = a;
    g.box_rows = p.page < kTile ? p.page : kTile;
    g.wide = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
    cudaError_t e;
    // A query tile: Tq tokens of the group's G heads, rows token * G + head.
    if ((e = make_tma_3d_bf16(&g.tq, a.q, D, p.Hq, p.N, p.G, t.Tq)) != cudaSuccess) return e;
    const uint64_t pages = static_cast<uint64_t>(p.n_pages) * p.Hk;
    if ((e = make_tma_3d_bf16(&g.tk, a.kc, D, p.page, pages, g.box_rows, 1)) != cudaSuccess) return e;
    if ((e = make_tma_3d_bf16(&g.tv, a.vc, D, p.page, pages, g.box_rows, 1)) != cudaSuccess) return e;
    if (p.Lw > 0) {
        // one token's depth rows a box, so that tokens start on 8-row boundaries
        // of the tile and no box reaches into tokens the job does not have
        const uint32_t rows = static_cast<uint32_t>(p.Lw < kTile ? p.Lw : kTile);
        const uint64_t slots = static_cast<uint64_t>(p.N) * p.Hk;
        if ((e = make_tma_3d_bf16(&g.tkd, a.kd, D, p.L, slots, rows, 1)) != cudaSuccess) return e;
        if ((e = make_tma_3d_bf16(&g.tvd, a.vd, D, p.L, slots, rows, 1)) != cudaSuccess) return e;
    } else {
        g.tkd = g.tk;
        g.tvd = g.tv;
    }
    const void* f = reinterpret_cast<const void*>(tree_sm100_kernel<D, NQ>);
    if ((e = set_max_dynamic_smem(f, Lay<D, NQ>::kBytes)) != cudaSuccess) return e;
    // set up (barriers, TMEM) while the grid before it in the stream ends
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(t.n_cta);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Lay<D, NQ>::kBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_sm100_kernel<D, NQ>, g);
}

}  // namespace

cudaError_t launch_tree_sm100(const Paged& p, const TreePlan& t, const TreeArgs& a, cudaStream_t s) {
    if (p.d == 64) return launch_d<64, 1>(p, t, a, s);
    return t.tiles == 1 ? launch_d<128, 1>(p, t, a, s) : launch_d<128, 2>(p, t, a, s);
}

}  // namespace moda
