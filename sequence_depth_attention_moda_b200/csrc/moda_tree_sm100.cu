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
// tiles, which it streams through a K ring and a V ring.  Two softmax
// warpgroups ("streams") each own an S tile and an O accumulator in TMEM:
//   a job of at most 128 rows   both streams hold the same query tile and take
//                               the tiles alternately; their (m, l, O) are
//                               merged at the end of the segment;
//   a job of up to 256 rows     stream s holds query tile s and takes every
//                               sequence tile, and its own tokens' depth tiles.
// Either way each stream's chain scores -> softmax -> values of one tile runs
// beside the other's, and a tile is loaded once for all rows of the job.
//
// Warps: 0 TMA producer (Q, K, V; a lane a page or a token, so pages as small
// as 8 rows cost one issue each); 1 clears the V rows that are not there and
// the values that are not finite (below); 2 issues S = Q K^T; 3 issues
// O += P V; 4..7 and 8..11 the streams' softmax, one thread a row: exponentials
// against the running reference without a maximum, which is taken only when a
// row sum passes 2^11 or a row has seen no key yet (exact: any reference gives
// the same quotient), P in bf16 over the score columns.
// TMEM columns: S0 [0,128), S1 [128,256), O0 [256,256+d), O1 [384,384+d).
//
// Warp 1: a tile that ends a request's keys leaves rows of the V stage unwritten
// (pages behind the last key are not loaded) or with what the page held; P is
// 0 there, but 0 * NaN is not, so it stores zeros.  In rows that only some of the
// query rows see (new keys, depth rows) it replaces infinities and NaN and
// marks the segment (not_finite_sum).  Tiles of held keys pass untouched.
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
constexpr uint32_t kSlab = 128 * 128;        // 128 rows x 64 bf16
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;
constexpr float kSumLimit = 2048.0f;         // largest row sum of a tile kept without a new reference
constexpr int kMarks = 8;                    // segments whose marks are told apart

template <int D>
struct Lay {
    static constexpr int kSlabs = D / 64;
    static constexpr uint32_t kTileBytes = kSlabs * kSlab;
    // V stages are held until P V is done, K stages only until S is
    static constexpr int kKS = D == 128 ? 2 : 5;
    static constexpr int kVS = D == 128 ? 3 : 6;
    static constexpr uint32_t kQ = 0;                       // two query tiles
    static constexpr uint32_t kK = 2 * kTileBytes;
    static constexpr uint32_t kV = kK + kKS * kTileBytes;
    static constexpr uint32_t kBar = kV + kVS * kTileBytes;
    // barrier indexes
    static constexpr int kQFull = 0, kQFree = 2, kKFull = 4, kKEmpty = kKFull + kKS, kVFull = kKEmpty + kKS,
                         kVFix = kVFull + kVS, kVEmpty = kVFix + kVS, kSFull = kVEmpty + kVS, kPReady = kSFull + 2,
                         kPVDone = kPReady + 2, kOFree = kPVDone + 2, kXDone = kOFree + 2, kNumBars = kXDone + 2;
    static constexpr uint32_t kExch = kBar + (kNumBars * 8 + 15) / 16 * 16;   // float2 [128]
    static constexpr uint32_t kStart = kExch + 128 * 8;
    static constexpr uint32_t kMisc = kStart + (sizeof(Start) + 15) / 16 * 16;  // tmem base, abort flag, marks
    static constexpr uint32_t kBytes = kMisc + 16 + kMarks * 4;
    static constexpr uint32_t kDynSmem = kBytes + 1024;     // alignment slack
    static_assert(kDynSmem <= 232448, "shared memory of one CTA");
    // warp 1 runs at most a V ring ahead of a segment's last tile, of which the
    // two streams may still hold two
    static_assert(kVS + 2 <= kMarks, "marks of segments in flight must differ");
};

struct SmArgs {
    TreeArgs t;
    TmaMap tq, tk, tv, tkd, tvd;
    int box_rows;        // rows of a cache box: min(page, 128)
};

// What every role derives alike while it walks the CTA's tiles.
struct Roles {
    int j = 0;           // tiles so far: ring stages, barrier phases
    int qtog = 0;        // query slot of the next one-tile job
    int qn[2] = {0, 0};  // uses of each query slot so far
    int primary;         // stream of the segment's first tile (one-tile jobs)
    int slot;            // query slot (one-tile jobs)
    bool two;            // two query tiles
    __device__ __forceinline__ void segment(const TreeArgs& a, const Walk& w) {
        two = w.j.ntok > a.Tq;
        primary = j & 1;
        slot = qtog;
    }
    // Streams (bit mask) that take the job's tile i, which is tile j of the CTA.
    __device__ __forceinline__ int streams(const Walk& w, int i) const {
        if (!two) return 1 << (j & 1);
        return i < w.j.nseq ? 3 : (i < w.j.nseq + w.j.ndep0 ? 1 : 2);
    }
    __device__ __forceinline__ int query_slot(int s) const { return two ? s : slot; }
    __device__ __forceinline__ void end_segment() {
        if (two) {
            ++qn[0];
            ++qn[1];
        } else {
            ++qn[slot];
            qtog ^= 1;
        }
    }
};

// Sequence keys of a job, and whether a tile has rows that are masked for
// somebody or are not there.
__device__ __forceinline__ int job_keys(const TreeArgs& a, const Job& j) {
    return j.r.held + (a.mask ? j.r.n : j.tok0 + j.ntok);
}
// Depth tile index within its query tile, and that tile's tokens.
__device__ __forceinline__ int dep_index(const Walk& w, int i) {
    const int dt = i - w.j.nseq;
    return dt < w.j.ndep0 ? dt : dt - w.j.ndep0;
}
__device__ __forceinline__ int sub_tokens(const TreeArgs& a, const Job& j, int sub) {
    return sub == 0 ? min(j.ntok, a.Tq) : j.ntok - a.Tq;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) tree_sm100_kernel(const __grid_constant__ SmArgs g) {
    using L = Lay<D>;
    const TreeArgs& a = g.t;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
    float2* exch = reinterpret_cast<float2*>(smem + L::kExch);
    Start* start = reinterpret_cast<Start*>(smem + L::kStart);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    volatile int* marks = reinterpret_cast<volatile int*>(tmem_holder + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < L::kNumBars; ++i)
            mbar_init(&bars[i], (i >= L::kPReady && i < L::kPVDone) || i >= L::kOFree ? 4 : 1);
        *abort_flag = 0;
        for (int i = 0; i < kMarks; ++i) marks[i] = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    schedule(a, start);        // ends with a CTA barrier
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    auto wait = [&](int bar, uint32_t phase) -> bool { return mbar_wait(&bars[bar], phase & 1, a.status, abort_flag); };
    auto wait_all = [&](int bar, uint32_t phase) -> bool { return __all_sync(0xffffffffu, wait(bar, phase)); };

    Walk w;
    Roles r;
    if (warp == 0) {
        // ---------------------------------------------------------- producer --
        if (lane == 0) {
            prefetch_tmap(&g.tq);
            prefetch_tmap(&g.tk);
            prefetch_tmap(&g.tv);
            if (a.Lw > 0) {
                prefetch_tmap(&g.tkd);
                prefetch_tmap(&g.tvd);
            }
        }
        const uint32_t q_bytes = L::kSlabs * 128u * a.Tq * a.G;
        int issued_k = 0, issued_v = 0;
        bool ok = true;
        for (bool more = w.begin(a, *start); ok && more; more = w.next(a)) {
            r.segment(a, w);
            for (int sub = 0; sub < (r.two ? 2 : 1); ++sub) {
                const int sl = r.query_slot(sub);
                if (r.qn[sl] > 0 && !wait_all(L::kQFree + sl, r.qn[sl] - 1)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars[L::kQFull + sl], q_bytes);
                    for (int s = 0; s < L::kSlabs; ++s)
                        tma_load_3d(smem + L::kQ + sl * L::kTileBytes + s * kSlab, &g.tq, &bars[L::kQFull + sl], s * 64,
                                    w.j.hk * a.G, w.j.r.cu0 + w.j.tok0 + sub * a.Tq);
                }
            }
            for (int i = w.i0; ok && i < w.i1; ++i, ++r.j) {
                // this lane's box: coordinates, first row of the tile, rows
                bool mine = false;
                int c1 = 0, c2 = 0, c3 = 0, row = 0;
                uint32_t bytes;
                const bool dep = i >= w.j.nseq;
                if (!dep) {
                    const int key = i * kTile + lane * g.box_rows;
                    const int boxes = kTile / g.box_rows;
                    const int left = min(kTile, job_keys(a, w.j) - i * kTile);
                    mine = lane < boxes && lane * g.box_rows < left;
                    bytes = ((left + g.box_rows - 1) / g.box_rows) * g.box_rows * 128u * L::kSlabs;
                    if (mine) {
                        const int p = page_of(a, w.j.b, key);
                        row = lane * g.box_rows;
                        c1 = key & ((1 << a.page_shift) - 1);
                        c2 = p < 0 ? -1 : p * a.Hk + w.j.hk;      // outside: the box reads as zeros
                    }
                } else {
                    const int sub = r.two && i >= w.j.nseq + w.j.ndep0 ? 1 : 0;
                    const int dt = dep_index(w, i);
                    const int tok = w.j.r.cu0 + w.j.tok0 + sub * a.Tq;
                    c2 = w.j.hk;
                    if (a.Lw <= kTile) {
                        const int cnt = min(a.dtok, sub_tokens(a, w.j, sub) - dt * a.dtok);
                        mine = lane < cnt;
                        bytes = cnt * a.Lw * 128u * L::kSlabs;
                        row = lane * a.Lp;
                        c1 = a.win_lo;
                        c3 = tok + dt * a.dtok + lane;
                    } else {
                        mine = lane == 0;
                        bytes = kTile * 128u * L::kSlabs;         // rows behind the last depth row read as zeros
                        c1 = a.win_lo + dt % a.dsplit * kTile;
                        c3 = tok + dt / a.dsplit;
                    }
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int ns = kv ? L::kVS : L::kKS;
                    const int st = r.j % ns;
                    const int full = (kv ? L::kVFull : L::kKFull) + st;
                    if (r.j >= ns && !wait_all((kv ? L::kVEmpty : L::kKEmpty) + st, r.j / ns - 1)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&bars[full], bytes);
                    __syncwarp();
                    if (kv) issued_v = r.j + 1;
                    else issued_k = r.j + 1;
                    if (mine) {
                        unsigned char* dst = smem + (kv ? L::kV : L::kK) + st * L::kTileBytes + row * 128;
#pragma unroll
                        for (int s = 0; s < L::kSlabs; ++s) {
                            if (dep)
                                tma_load_4d(dst + s * kSlab, kv ? &g.tvd : &g.tkd, &bars[full], s * 64, c1, c2, c3);
                            else
                                tma_load_3d(dst + s * kSlab, kv ? &g.tv : &g.tk, &bars[full], s * 64, c1, c2);
                        }
                    }
                }
            }
            r.end_segment();
        }
        // every load lands before the CTA retires (bounded by time only: these
        // waits ignore the abort flag)
        if (lane == 0) {
            int no_abort = 0;
            for (int s = 0; s < 2; ++s)
                if (r.qn[s] > 0) mbar_wait(&bars[L::kQFull + s], (r.qn[s] - 1) & 1, a.status, &no_abort);
            for (int x = max(0, issued_k - L::kKS); x < issued_k; ++x)
                mbar_wait(&bars[L::kKFull + x % L::kKS], (x / L::kKS) & 1, a.status, &no_abort);
            for (int x = max(0, issued_v - L::kVS); x < issued_v; ++x)
                mbar_wait(&bars[L::kVFull + x % L::kVS], (x / L::kVS) & 1, a.status, &no_abort);
        }
    } else if (warp == 1) {
        // ------------------------------------- rows of V that are not there --
        bool ok = true;
        for (bool more = w.begin(a, *start); ok && more; more = w.next(a)) {
            r.segment(a, w);
            for (int i = w.i0; i < w.i1; ++i, ++r.j) {
                const int st = r.j % L::kVS;
                if (!wait_all(L::kVFull + st, r.j / L::kVS)) {
                    ok = false;
                    break;
                }
                const bool dep = i >= w.j.nseq;
                const int from = dep ? 0 : max(0, w.j.r.held - i * kTile);
                if (from < kTile) {
                    const int there = job_keys(a, w.j) - i * kTile;   // sequence rows of the tile that exist
                    int cnt = 0, last = 0;                            // depth: tokens, or rows of one token
                    if (dep) {
                        const int sub = r.two && i >= w.j.nseq + w.j.ndep0 ? 1 : 0;
                        const int dt = dep_index(w, i);
                        cnt = min(a.dtok, sub_tokens(a, w.j, sub) - dt * a.dtok);
                        last = a.Lw - dt % a.dsplit * kTile;
                    }
                    bool bad = false;
#pragma unroll
                    for (int s = 0; s < L::kSlabs; ++s) {
                        uint4* base = reinterpret_cast<uint4*>(smem + L::kV + st * L::kTileBytes + s * kSlab);
#pragma unroll 4
                        for (int x = from * 8 + lane; x < kTile * 8; x += 32) {
                            const int row = x >> 3;
                            bool real;
                            if (!dep) real = row < there;
                            else if (a.Lw <= kTile) real = row / a.Lp < cnt && row % a.Lp < a.Lw;
                            else real = row < last;
                            if (!real) {
                                base[x] = make_uint4(0, 0, 0, 0);
                                continue;
                            }
                            const uint4 v = base[x];
                            uint32_t e[4] = {v.x, v.y, v.z, v.w};
                            bool hit = false;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if ((e[k] & 0x7f80u) == 0x7f80u) e[k] &= 0xffff0000u, hit = true;
                                if ((e[k] & 0x7f800000u) == 0x7f800000u) e[k] &= 0x0000ffffu, hit = true;
                            }
                            if (hit) {
                                base[x] = make_uint4(e[0], e[1], e[2], e[3]);
                                bad = true;
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    if (__any_sync(0xffffffffu, bad) && lane == 0) marks[w.seg % kMarks] = w.seg + 1;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[L::kVFix + st]);
            }
            r.end_segment();
        }
    } else if (warp == 2) {
        // ------------------------------------------------------ S = Q K^T -----
        if (elect_one()) {
            const uint32_t id = idesc_bf16(128, kTile, false, false);
            const uint64_t qd = desc_kmajor_sw128(smem_u32(smem + L::kQ));
            const uint64_t kd = desc_kmajor_sw128(smem_u32(smem + L::kK));
            int js[2] = {0, 0};
            bool ok = true;
            for (bool more = w.begin(a, *start); ok && more; more = w.next(a)) {
                r.segment(a, w);
                for (int sub = 0; ok && sub < (r.two ? 2 : 1); ++sub)
                    ok = wait(L::kQFull + r.query_slot(sub), r.qn[r.query_slot(sub)]);
                for (int i = w.i0; ok && i < w.i1; ++i, ++r.j) {
                    const int st = r.j % L::kKS;
                    if (!(ok = wait(L::kKFull + st, r.j / L::kKS))) break;
                    const int set = r.streams(w, i);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (!(set >> s & 1)) continue;
                        // S_s holds P of the stream's last tile until its P V is done
                        if (js[s] > 0 && !(ok = wait(L::kPVDone + s, js[s] - 1))) break;
                        tc_fence_after();
                        const uint64_t q0 = qd + ((r.query_slot(s) * L::kTileBytes) >> 4);
                        const uint64_t k0 = kd + ((st * L::kTileBytes) >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t off = ((kk >> 2) * kSlab + (kk & 3) * 32) >> 4;
                            umma_ss(tmem + s * 128, q0 + off, k0 + off, id, kk > 0 ? 1u : 0u);
                        }
                        umma_commit(&bars[L::kSFull + s]);
                        ++js[s];
                    }
                    if (ok) umma_commit(&bars[L::kKEmpty + st]);
                }
                if (ok)
                    for (int sub = 0; sub < (r.two ? 2 : 1); ++sub) umma_commit(&bars[L::kQFree + r.query_slot(sub)]);
                r.end_segment();
            }
        }
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------------------ O += P V ------
        if (elect_one()) {
            const uint32_t id = idesc_bf16(128, D, false, true);
            const uint64_t vd = desc_mnmajor_sw128(smem_u32(smem + L::kV), kSlab);
            int js[2] = {0, 0}, segs[2] = {0, 0};
            bool ok = true;
            for (bool more = w.begin(a, *start); ok && more; more = w.next(a)) {
                r.segment(a, w);
                int in_seg[2] = {0, 0};
                for (int i = w.i0; ok && i < w.i1; ++i, ++r.j) {
                    const int st = r.j % L::kVS;
                    if (!(ok = wait(L::kVFix + st, r.j / L::kVS))) break;
                    const int set = r.streams(w, i);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (!(set >> s & 1)) continue;
                        // the first product of a segment overwrites O, which must have been read out
                        if (in_seg[s] == 0 && segs[s] > 0 && !(ok = wait(L::kOFree + s, segs[s] - 1))) break;
                        if (!(ok = wait(L::kPReady + s, js[s]))) break;
                        tc_fence_after();
                        const uint64_t v0 = vd + ((st * L::kTileBytes) >> 4);
#pragma unroll
                        for (int kk = 0; kk < kTile / 16; ++kk)
                            umma_ts(tmem + kColO + s * 128, tmem + s * 128 + kk * 8, v0 + kk * (2048 >> 4), id,
                                    in_seg[s] > 0 || kk > 0 ? 1u : 0u);
                        umma_commit(&bars[L::kPVDone + s]);
                        ++js[s];
                        ++in_seg[s];
                    }
                    if (ok) umma_commit(&bars[L::kVEmpty + st]);
                }
                segs[0] += in_seg[0] > 0;
                segs[1] += in_seg[1] > 0;
                r.end_segment();
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ softmax -------
        const int s = (warp - 4) >> 2;               // stream
        const int quarter = warp & 3;                // TMEM lanes 32*quarter ..
        const int row = quarter * 32 + lane;
        const int t_off = row / a.G;                 // token within the query tile
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t s_col = lane_base + s * 128;
        const float sl2 = a.scale_log2;
        int js = 0, merges[2] = {0, 0};              // tiles of this stream; merges with each secondary stream
        bool ok = true;
        for (bool more = w.begin(a, *start); ok && more; more = w.next(a)) {
            r.segment(a, w);
            const int sub = r.two ? s : 0;
            const int n_tok = sub_tokens(a, w.j, sub);
            const bool real = t_off < n_tok && t_off < a.Tq;
            const bool active = quarter * 32 < n_tok * a.G;     // some row of the warp is real
            const int token = w.j.tok0 + sub * a.Tq + t_off;    // relative to the request
            float m = -INFINITY, l = 0.0f;
            int in_seg = 0;
            for (int i = w.i0; i < w.i1; ++i, ++r.j) {
                if (!(r.streams(w, i) >> s & 1)) continue;
                if (!wait_all(L::kSFull + s, js)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (active) {
                    const bool dep = i >= w.j.nseq;
                    const bool masked = dep || (i + 1) * kTile > w.j.r.held;
                    const int dt = dep ? dep_index(w, i) : 0;
                    // 32 scores from column 32c on; those the row does not see become -inf
                    auto hide = [&](uint32_t* x, int c) {
                        const uint32_t vis = !real ? 0xffffffffu
                                                   : (dep ? dep_visible(a, t_off, dt, 32 * c)
                                                          : seq_visible(a, w.j.r, token, i * kTile + 32 * c));
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(vis >> e & 1)) x[e] = __float_as_uint(-INFINITY);
                    };
                    uint32_t pk[64];
                    // p = 2^(s sl2 - ref), packed; returns the row sum
                    auto exps = [&](float ref) -> float {
                        float rs[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        uint32_t x[2][32];
                        tmem_ld32(s_col, x[0]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            tmem_wait_ld();
                            reg_fence<32>(x[c & 1]);
                            if (c < 3) tmem_ld32(s_col + 32 * (c + 1), x[(c + 1) & 1]);
                            if (masked) hide(x[c & 1], c);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float p0 = ex2(fmaf(__uint_as_float(x[c & 1][2 * e]), sl2, -ref));
                                const float p1 = ex2(fmaf(__uint_as_float(x[c & 1][2 * e + 1]), sl2, -ref));
                                rs[e & 3] += p0 + p1;
                                pk[16 * c + e] = pack_bf16(p0, p1);
                            }
                        }
                        return (rs[0] + rs[1]) + (rs[2] + rs[3]);
                    };
                    float rs = 0.0f;
                    bool anew = __any_sync(0xffffffffu, real && m == -INFINITY);   // a row without a reference
                    if (!anew) {
                        rs = exps(real ? m : 0.0f);
                        anew = __any_sync(0xffffffffu, real && !(rs <= kSumLimit));
                    }
                    if (anew) {
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[32];
                            tmem_ld32(s_col + 32 * c, x);
                            tmem_wait_ld();
                            reg_fence<32>(x);
                            if (masked) hide(x, c);
#pragma unroll
                            for (int e = 0; e < 32; e += 2)
                                mx = fmax3(mx, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                        }
                        const float mn = fmaxf(m, mx * sl2);
                        const float alpha = m == -INFINITY ? 1.0f : ex2(m - mn);   // o and l are 0 until a key is seen
                        l *= alpha;
                        m = mn;
                        if (in_seg > 0) {
                            // O holds the sum up to the last tile: its product was done before these scores began
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t o[32];
                                tmem_ld32(lane_base + kColO + s * 128 + c, o);
                                tmem_wait_ld();
                                reg_fence<32>(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st32(lane_base + kColO + s * 128 + c, o);
                            }
                            tmem_wait_st();
                        }
                        rs = exps(real && m != -INFINITY ? m : 0.0f);
                    }
                    l += rs;
                    __syncwarp();
                    tmem_st32(s_col, pk);
                    tmem_st32(s_col + 32, pk + 32);
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[L::kPReady + s]);
                ++js;
                ++in_seg;
            }
            if (!ok) break;
            // ------------------------------------------------ end of segment --
            // One query tile and two tiles or more: the other stream has a share.
            const bool both = !r.two && w.i1 - w.i0 >= 2;
            const bool second = both && s != r.primary;
            if (in_seg > 0) {
                if (!wait_all(L::kPVDone + s, js - 1)) {
                    ok = false;
                    break;
                }
                if (second) {
                    exch[row] = make_float2(m, l);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[L::kXDone + s]);
                } else {
                    float m2 = -INFINITY, l2 = 0.0f;
                    if (both) {
                        if (!wait_all(L::kXDone + (s ^ 1), merges[s ^ 1])) {
                            ok = false;
                            break;
                        }
                        const float2 x = exch[row];
                        m2 = x.x;
                        l2 = x.y;
                    }
                    tc_fence_after();
                    const float M = fmaxf(m, m2);
                    const float w1 = m == -INFINITY ? 0.0f : ex2(m - M), w2 = m2 == -INFINITY ? 0.0f : ex2(m2 - M);
                    const float lt = l * w1 + l2 * w2;
                    const bool poison = marks[w.seg % kMarks] == w.seg + 1;
                    const bool whole = w.whole();
                    const float inv = !whole ? 1.0f : (lt == 0.0f ? 0.0f : 1.0f / lt);
                    const float f1 = w1 * inv, f2 = w2 * inv;
                    const size_t orow =
                        static_cast<size_t>(w.j.r.cu0 + token) * a.Hq + w.j.hk * a.G + (row - t_off * a.G);
                    const size_t rec = static_cast<size_t>(w.slot(a)) * a.rec_rows + sub * a.Tq * a.G + row;
                    if (active) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tmem_ld32(lane_base + kColO + s * 128 + c, o);
                            tmem_wait_ld();
                            reg_fence<32>(o);
                            if (both) {
                                uint32_t o2[32];
                                tmem_ld32(lane_base + kColO + (s ^ 1) * 128 + c, o2);
                                tmem_wait_ld();
                                reg_fence<32>(o2);
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * f1 + __uint_as_float(o2[e]) * f2);
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f1);
                            }
                            if (!real) continue;
                            if (whole) {
                                if (poison) {
#pragma unroll 1
                                    for (int e = 0; e < 32; ++e) {
                                        const float add = not_finite_sum<__nv_bfloat16, D>(a, w.j, token, c + e);
                                        // o stays in registers: a select per element
#pragma unroll
                                        for (int k = 0; k < 32; ++k)
                                            if (k == e) o[k] = __float_as_uint(__uint_as_float(o[k]) + add);
                                    }
                                }
                                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + orow * D + c);
#pragma unroll
                                for (int e = 0; e < 32; e += 8)
                                    dst[e / 8] = make_uint4(
                                        pack_bf16(__uint_as_float(o[e]), __uint_as_float(o[e + 1])),
                                        pack_bf16(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3])),
                                        pack_bf16(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5])),
                                        pack_bf16(__uint_as_float(o[e + 6]), __uint_as_float(o[e + 7])));
                            } else {
                                uint4* dst = reinterpret_cast<uint4*>(a.po + rec * D + c);
#pragma unroll
                                for (int e = 0; e < 32; e += 4) dst[e / 4] = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                            }
                        }
                        if (real) {
                            if (whole) a.lse[orow] = row_lse(M, lt);
                            else a.ml[rec] = make_float2(M, poison ? -lt : lt);
                        }
                    }
                    // O (of both streams) may be overwritten
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bars[L::kOFree + s]);
                        if (both) mbar_arrive(&bars[L::kOFree + (s ^ 1)]);
                    }
                }
            }
            if (in_seg == 0 && r.two && real)    // two query tiles, and only depth tiles of the other one here
                a.ml[static_cast<size_t>(w.slot(a)) * a.rec_rows + sub * a.Tq * a.G + row] = make_float2(-INFINITY, 0.0f);
            if (both) ++merges[r.primary ^ 1];
            r.end_segment();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
cudaError_t launch_d(const Paged& p, const TreePlan& t, const TreeArgs& a, cudaStream_t s) {
    SmArgs g;
    g.t = a;
    g.box_rows = p.page < kTile ? p.page : kTile;
    cudaError_t e;
    // A query tile: Tq tokens of the group's G heads, rows token * G + head.
    if ((e = make_tma_3d_bf16(&g.tq, a.q, D, p.Hq, p.N, p.G, t.Tq)) != cudaSuccess) return e;
    const uint64_t pages = static_cast<uint64_t>(p.n_pages) * p.Hk;
    if ((e = make_tma_3d_bf16(&g.tk, a.kc, D, p.page, pages, g.box_rows, 1)) != cudaSuccess) return e;
    if ((e = make_tma_3d_bf16(&g.tv, a.vc, D, p.page, pages, g.box_rows, 1)) != cudaSuccess) return e;
    if (p.Lw > 0) {
        // one token's depth rows a box, so that tokens start on 8-row boundaries
        // of the tile and no box reaches into tokens the job does not have
        const uint64_t row = D * 2;
        const uint64_t dims[4] = {D, static_cast<uint64_t>(p.L), static_cast<uint64_t>(p.Hk), static_cast<uint64_t>(p.N)};
        const uint64_t strides[3] = {row, row * p.L, row * p.L * p.Hk};
        const uint32_t box[4] = {64, static_cast<uint32_t>(p.Lw < kTile ? p.Lw : kTile), 1, 1};
        if ((e = make_tma_4d_bf16(&g.tkd, a.kd, dims, strides, box)) != cudaSuccess) return e;
        if ((e = make_tma_4d_bf16(&g.tvd, a.vd, dims, strides, box)) != cudaSuccess) return e;
    } else {
        g.tkd = g.tk;
        g.tvd = g.tv;
    }
    const void* f = reinterpret_cast<const void*>(tree_sm100_kernel<D>);
    if ((e = set_max_dynamic_smem(f, Lay<D>::kDynSmem)) != cudaSuccess) return e;
    tree_sm100_kernel<D><<<t.n_cta, kThreads, Lay<D>::kDynSmem, s>>>(g);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_sm100(const Paged& p, const TreePlan& t, const TreeArgs& a, cudaStream_t s) {
    return p.d == 128 ? launch_d<128>(p, t, a, s) : launch_d<64>(p, t, a, s);
}

}  // namespace moda
