// moda_tree.cuh -- what the two paths of the attention of drafted tokens over
// a paged cache share: the arguments, the schedule, the visible sets and the
// partial records (moda_tree_simt.cu: CUDA cores, fp32, and the merging of split
// jobs; moda_tree_sm100.cu: tensor cores, bf16).
//
// Work.  A job is (request b, KV head hk, group of Tg consecutive new tokens);
// its rows are the G query heads of each token, row = token * G + head.  A job
// reads tiles of KT key rows: first its sequence tiles (keys 0 .. held+n-1 of
// the request, through the block table), then the depth tiles of its tokens.
// Only the keys from `held` on and the depth rows are masked.  The jobs' tiles
// form one list, in the order request, KV head, group, tile; each has a cost (a
// sequence tile that two row tiles take costs more than one that a single one
// takes, and a job's beginning costs job_cost: the pipeline drains and fills, Q is
// fetched and O written), and CTA c of P owns the tiles that begin in the c-th of
// P equal parts of the total cost X (X < 2^31, which the host checks, so 32 bits
// and no long division; X / P is at least the largest tile's cost, so that a part
// between two of a job's tiles has one of them itself).  Lengths live on the
// device (a captured graph replays with other ones), so every CTA adds up the
// list itself.  Where cu_new descends the requests share rows and the host's bound
// does not hold: then the list is empty.  A job that one CTA owns whole is
// written out by it; of a job cut at a range's end every CTA leaves one (m, l, o)
// record a row, and the combine kernel merges them in CTA order.  At most two of
// a CTA's jobs can be cut (its first and its last), so the records take 2 slots a
// CTA whatever the lengths.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "moda_internal.h"
#include "moda_ptx.cuh"

namespace moda {
namespace tree {

// A request's clamped lengths.
struct Request {
    int held, n, cu0;
};

// The job that holds a CTA's first tile, left for the combine kernel.
struct CtaHeader {
    int x_total;           // cost of the whole call
    int n_ranges;          // parts it is cut into
    int job_start;         // where the job begins
    int b, hk, group;
    Request r;
    int pad[3];
};

struct TreeArgs {
    const void *q, *kc, *vc, *kd, *vd;   // [N,Hq,D], cache [n_pages,Hk,page,D], [N,Hk,L,D]
    const int *table, *held, *cu;        // [B,max_pages], [B], [B+1]
    const uint32_t* mask;                // [N,words] or NULL (chain)
    void* o;                             // [N,Hq,D]
    float* lse;                          // [N,Hq]
    CtaHeader* hdr;                      // [n_cta]
    float2* ml;                          // [2*n_cta][rec_rows]: m (base 2), l (negative: see row_poisoned)
    float* po;                           // [2*n_cta][rec_rows][D]
    unsigned int* status;
    int B, N, Hq, Hk, G, L, Lw, win_lo;  // Lw: depth rows in the window
    int page_shift, n_pages, max_pages, words;
    int Tq, Tg;                          // tokens per row tile, per job (Tg = Tq or 2*Tq)
    int kt_shift, KT;                    // key rows per tile, a power of two
    int Lp, dtok, dsplit;                // depth tiles: rows a token takes, tokens per tile (Lw <= KT),
                                         // tiles per token (Lw > KT)
    int two_cost;                        // cost of a sequence tile that two row tiles take: 1 or 2 (others: 1)
    int job_cost;                        // of a job's beginning, before its first tile
    int rec_rows, n_cta;
    float scale_log2;
};

// A request's lengths as the caller has them, and clamped: what lies outside
// the tables' bounds is cut off, so that no index below leaves its array, and
// reported.
struct RawRequest {
    int held, c0, c1;
};
__device__ __forceinline__ RawRequest load_raw(const TreeArgs& a, int b) {
    return RawRequest{a.held[b], a.cu[b], a.cu[b + 1]};
}
__device__ __forceinline__ Request clamp_request(const TreeArgs& a, const RawRequest& x) {
    Request r;
    const long long cap = static_cast<long long>(a.max_pages) << a.page_shift;
    r.held = static_cast<int>(min(static_cast<long long>(max(x.held, 0)), cap));
    r.cu0 = min(max(x.c0, 0), a.N);
    long long n = min(max(x.c1, 0), a.N) - r.cu0;
    n = min(n, cap - r.held);
    if (a.mask) n = min(n, 32ll * a.words);
    r.n = static_cast<int>(max(n, 0ll));
    if (r.held != x.held || r.cu0 != x.c0 || r.n != static_cast<long long>(x.c1) - x.c0)
        atomicOr(a.status, kStatusBadIndex);
    return r;
}
__device__ __forceinline__ Request load_request(const TreeArgs& a, int b) { return clamp_request(a, load_raw(a, b)); }

__device__ __forceinline__ int dep_tiles_of(const TreeArgs& a, int tokens) {
    if (a.Lw == 0 || tokens <= 0) return 0;
    if (a.Lw > a.KT) return tokens * a.dsplit;
    return tokens <= a.dtok ? 1 : (tokens + a.dtok - 1) / a.dtok;
}

struct Job {
    int b, hk, group;
    Request r;
    int tok0, ntok;      // the group's tokens, relative to the request's first
    int nseq, ndep0, nt; // sequence tiles, depth tiles of the first Tq tokens, all tiles
    int cseq, cost;      // cost of a sequence tile (1 or 2), of the job
};
// Where tile i of a job begins, and the first tile that begins at x or behind.
__device__ __forceinline__ int tile_begin(const TreeArgs& a, const Job& j, int i) {
    return a.job_cost + i + min(i, j.nseq) * (j.cseq - 1);
}
__device__ __forceinline__ int tile_from(const TreeArgs& a, const Job& j, int x) {
    x -= a.job_cost;
    if (x <= 0) return 0;
    if (x <= j.nseq * j.cseq) return (x + j.cseq - 1) >> (j.cseq - 1);
    return min(j.nt, x - j.nseq * (j.cseq - 1));
}

__device__ __forceinline__ int groups_of(const TreeArgs& a, const Request& r) {
    return r.n <= a.Tg ? (r.n > 0) : (r.n + a.Tg - 1) / a.Tg;
}

__device__ __forceinline__ void set_group(const TreeArgs& a, Job& j, int group) {
    j.group = group;
    j.tok0 = group * a.Tg;
    j.ntok = min(a.Tg, j.r.n - j.tok0);
    // a chain's group sees no key behind its last token
    const int keys = j.r.held + (a.mask ? j.r.n : j.tok0 + j.ntok);
    j.nseq = (keys + a.KT - 1) >> a.kt_shift;
    j.ndep0 = dep_tiles_of(a, min(j.ntok, a.Tq));
    j.nt = j.nseq + j.ndep0 + dep_tiles_of(a, j.ntok - a.Tq);
    j.cseq = j.ntok > a.Tq ? a.two_cost : 1;
    j.cost = a.job_cost + j.nt + j.nseq * (j.cseq - 1);
}

// Cost of one KV head of a request.
__device__ __forceinline__ int head_cost(const TreeArgs& a, const Request& r) {
    Job j;
    j.r = r;
    const int ng = groups_of(a, r);
    if (ng == 0) return 0;
    set_group(a, j, ng - 1);
    int t = j.cost;
    if (ng > 1) {                       // all groups but the last are alike, but for a chain's keys
        set_group(a, j, 0);
        t += j.cost * (ng - 1);
        if (!a.mask)
            for (int g = 1; g < ng - 1; ++g)
                t += (((r.held + (g + 1) * a.Tg + a.KT - 1) >> a.kt_shift) - j.nseq) * j.cseq;
    }
    return t;
}

// Where a CTA starts, in shared memory; written by schedule().
struct Start {
    int warp_sum[32];
    int max_cost[32];        // of a warp's sequence tiles, or kNoSchedule
    Job j;                   // the job in which the CTA's part begins,
    int lo;                  // and where in it
    int length;              // of the part; 0: none
};

// Where part c of P begins in a total of x.
__device__ __forceinline__ int range_begin(int c, int x, int P) {
    const int q = x / P, rem = x - q * P;
    return c * q + min(c, rem);
}
// The part that holds x = t.
__device__ __forceinline__ int range_of(int t, int x, int P) {
    const int q = x / P, rem = x - q * P;
    return t < rem * (q + 1) ? t / (q + 1) : rem + (t - rem * (q + 1)) / q;
}

constexpr int kNoSchedule = 0x7fffffff;

// Called by all threads of the CTA: finds the CTA's part and writes its header.
// Ends with a __syncthreads.
__device__ __forceinline__ void schedule(const TreeArgs& a, Start* s) {
    const int nth = static_cast<int>(blockDim.x), tid = static_cast<int>(threadIdx.x);
    const int lane = tid & 31, warp = tid >> 5;
    const int ch = (a.B + nth - 1) / nth;
    const int b0 = min(a.B, tid * ch), b1 = min(a.B, b0 + ch);
    Request r = {};
    int hc = 0, mine = 0, most = 1;
    bool down = false;                   // cu_new descends
    for (int b = b0; b < b1; ++b) {
        const RawRequest raw = load_raw(a, b);
        down |= raw.c1 < raw.c0;
        r = clamp_request(a, raw);
        hc = head_cost(a, r);
        mine += hc * a.Hk;
        if (r.n > a.Tq) most = a.two_cost;
    }
    int inc = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    most = 1 + __any_sync(0xffffffffu, most > 1);
    if (__any_sync(0xffffffffu, down)) most = kNoSchedule;
    if (lane == 31) {
        s->warp_sum[warp] = inc;
        s->max_cost[warp] = most;
    }
    if (tid == 0) s->length = 0;
    __syncthreads();
    int at = inc - mine, total = 0;
#pragma unroll 1
    for (int w = 0; w < (nth >> 5); ++w) {
        if (w < warp) at += s->warp_sum[w];
        total += s->warp_sum[w];
        most = max(most, s->max_cost[w]);
    }
    const int P = most == kNoSchedule ? 0 : min(a.n_cta, total / most), c = static_cast<int>(blockIdx.x);
    if (c < P) {
        const int lo = range_begin(c, total, P);
        if (at <= lo && lo < at + mine) {
            int b = b0;
            if (ch > 1) {                // which of this thread's requests
                for (;; ++b) {
                    r = load_request(a, b);
                    hc = head_cost(a, r);
                    if (lo < at + hc * a.Hk) break;
                    at += hc * a.Hk;
                }
            }
            const int hk = (lo - at) / hc;
            at += hc * hk;
            Job j;
            j.r = r;
            j.b = b;
            j.hk = hk;
            int g = 0;
            for (;; ++g) {
                set_group(a, j, g);
                if (lo < at + j.cost) break;
                at += j.cost;
            }
            s->j = j;
            s->lo = lo - at;
            s->length = range_begin(c + 1, total, P) - lo;
            a.hdr[c] = CtaHeader{total, P, at, b, hk, g, r, {}};
        }
    } else if (tid == 0) {
        a.hdr[c] = CtaHeader{total, P, 0, 0, 0, 0, {}, {}};
    }
    __syncthreads();
}

// Walks a CTA's jobs.  The next request's lengths are asked for when a request
// begins: under load such a read takes as long as a tile or two.
struct Walk {
    Job j;
    RawRequest ahead;    // of request j.b + 1
    int i0, i1;          // this CTA's tiles of the job
    int end;             // where the CTA's part ends, from the job's beginning
    __device__ __forceinline__ bool begin(const TreeArgs& a, const Start& s) {
        if (s.length == 0) return false;
        j = s.j;
        look_ahead(a);
        end = s.lo + s.length;
        take(a, tile_from(a, j, s.lo));
        // the part may begin behind the job's last tile's beginning, or end before the
        // first one's: then it has none of this job (nor does the combine kernel look for it)
        return i0 < i1 || next(a);
    }
    __device__ __forceinline__ bool next(const TreeArgs& a) {
        end -= j.cost;
        if (end <= a.job_cost) return false;
        int g = j.group + 1;
        if (g * a.Tg >= j.r.n) {
            g = 0;
            if (++j.hk == a.Hk) {
                j.hk = 0;
                do {
                    if (++j.b >= a.B) return false;
                    j.r = clamp_request(a, ahead);
                    look_ahead(a);
                } while (j.r.n == 0);
            }
        }
        set_group(a, j, g);
        take(a, 0);
        return true;
    }
    // Whether this CTA owns the job whole (then it writes the outputs itself).
    __device__ __forceinline__ bool whole() const { return i0 == 0 && i1 == j.nt; }
    // Where its record of a cut job goes: a job that began before the part is the
    // part's first, one that begins in it and goes on is its last.
    __device__ __forceinline__ int slot() const { return 2 * static_cast<int>(blockIdx.x) + (i0 == 0); }

   private:
    __device__ __forceinline__ void look_ahead(const TreeArgs& a) {
        if (j.b + 1 < a.B) ahead = load_raw(a, j.b + 1);
    }
    __device__ __forceinline__ void take(const TreeArgs& a, int first) {
        i0 = first;
        i1 = tile_from(a, j, end);
    }
};

// ------------------------------------------------------------ visible sets --
// Bit c set for lo <= c < hi, 0 <= c < 32.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
    lo = max(lo, 0);
    hi = min(hi, 32);
    if (lo >= hi) return 0u;
    return (0xffffffffu >> (32 - (hi - lo))) << lo;
}

// Which of the 32 new keys rel .. rel+31 (below 0: held keys) of a request's n a
// token sees by its mask row: every held key, and those whose bit the row has.
__device__ __forceinline__ uint32_t mask_visible(const uint32_t* row, int words, int n, int rel) {
    if (rel <= -32) return 0xffffffffu;
    const int w = rel >> 5;             // floor
    auto word = [&](int x) -> uint32_t { return x < 0 ? 0xffffffffu : (x < words ? row[x] : 0u); };
    return __funnelshift_r(word(w), word(w + 1), rel & 31) & bits_between(0, n - rel);
}
// The same without a mask (a chain): the new keys up to the token itself.
__device__ __forceinline__ uint32_t chain_visible(int n, int token, int rel) {
    return rel <= -32 ? 0xffffffffu : bits_between(0, min(token + 1, n) - rel);
}
// Which of the 32 sequence keys from key `k0` on the token sees.
__device__ __forceinline__ uint32_t seq_visible(const TreeArgs& a, const Request& r, int token, int k0) {
    return a.mask ? mask_visible(a.mask + static_cast<size_t>(r.cu0 + token) * a.words, a.words, r.n, k0 - r.held)
                  : chain_visible(r.n, token, k0 - r.held);
}

// Which of 32 rows from row `c0` on of depth tile `dt` (of the row tile's
// tokens) are the depth rows of the row tile's token `t`.
__device__ __forceinline__ uint32_t dep_visible(const TreeArgs& a, int t, int dt, int c0) {
    if (a.Lw <= a.KT) {
        const int at = (t - dt * a.dtok) * a.Lp - c0;
        return (t >= dt * a.dtok && t < (dt + 1) * a.dtok) ? bits_between(at, at + a.Lw) : 0u;
    }
    const int tok = dt / a.dsplit;
    return tok == t ? bits_between(0, a.Lw - (dt - tok * a.dsplit) * a.KT - c0) : 0u;
}

// The block table's entry for a request's key `key`; the page an entry names, -1
// (and a status) if it names none of the cache.
__device__ __forceinline__ int table_entry(const TreeArgs& a, int b, int key) {
    return a.table[static_cast<size_t>(b) * a.max_pages + (key >> a.page_shift)];
}
__device__ __forceinline__ int checked_page(const TreeArgs& a, int p) {
    if (static_cast<unsigned>(p) < static_cast<unsigned>(a.n_pages)) return p;
    atomicOr(a.status, kStatusBadIndex);
    return -1;
}

__device__ __forceinline__ int page_of(const TreeArgs& a, int b, int key) {
    return checked_page(a, table_entry(a, b, key));
}

// ------------------------------------------------- values that are not finite --
// P V sums over all rows of a tile, and 0 * Inf is NaN: an infinity or a NaN
// in a value that only some of a tile's query rows see would reach the others.
// So in the rows of V that are masked for anybody (new keys, depth rows) such
// elements are replaced by 0 before the product and the record is marked; the
// (rare) marked rows add them here, to the outputs just stored and each from
// the keys it sees.  Added without its weight: p > 0 does not change an
// infinity or a NaN.
//
// A warp goes once over the keys and depth rows that any of its rows sees, whole rows
// of V at a time, and notes for each column which of its rows see a +Inf and which a
// -Inf (a NaN counts as both): the time is that of reading V.  A chain of 4096 tokens
// with an infinity or NaN in three of 8 heads' values (32 query heads, d = 128): 2.3 ms
// against 0.30 without, in fp32 6.4 against 4.3.  A walk over the keys for every column
// of every row took 560 and 950 ms.
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_float(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Rows row0, row0 + step, ... (n <= 16 of them; row = token * G + head, from the
// request's token tok0 on) of a KV head's outputs, which the warp's lanes stored before
// (or others, and a barrier).  Whole warp.  kAhead: rows of V in flight, which bound the
// time and the registers (a callee's count is its kernel's too).
template <typename E, int D, int kAhead>
__device__ __noinline__ void add_not_finite(const TreeArgs& a, const Request r, int b, int hk, int tok0, int row0,
                                            int step, int n) {
    constexpr int C = D / 32;            // columns C * lane .. of a row are the lane's
    constexpr int kWords = C * static_cast<int>(sizeof(E)) / 4;
    constexpr uint32_t kAll = 0xffffffffu;
    union alignas(4 * kWords) Piece {
        uint32_t w[kWords];
        E e[C];
        __device__ Piece() {}
    };
    const int lane = threadIdx.x & 31, page = 1 << a.page_shift;
    const int token = tok0 + (row0 + min(lane, n - 1) * step) / a.G;     // of the lane's output row
    const int last = tok0 + (row0 + (n - 1) * step) / a.G;
    uint32_t seen[C] = {};               // bit i: output row i sees a +Inf, bit 16 + i: a -Inf
    const int keys = a.mask ? r.n : last + 1;
    int k = 0, t = tok0 + row0 / a.G, l = a.win_lo;      // next key; then next depth row
#pragma unroll 1
    while (k < keys || (l < a.L && t <= last)) {
        // 32 rows of V: lane i's `off` says where row i begins (-1: nowhere), bit i of
        // `vis` whether the lane's output row sees it
        const bool dep = k >= keys;
        const E* base = static_cast<const E*>(dep ? a.vd : a.vc);
        long long off = -1;
        uint32_t vis = 0;
        if (!dep) {
            if (lane < n) vis = seq_visible(a, r, token, r.held + k);
            if (k + lane < keys) {
                const int key = r.held + k + lane, p = page_of(a, b, key);
                if (p >= 0) off = ((static_cast<long long>(p) * a.Hk + hk) * page + (key & (page - 1))) * D;
            }
            k += 32;
        } else {
            if (lane < n && token == t) vis = kAll;
            if (l + lane < a.L) off = ((static_cast<long long>(r.cu0 + t) * a.Hk + hk) * a.L + l + lane) * D;
            l += 32;
            if (l >= a.L) {
                l = a.win_lo;
                ++t;
            }
        }
        const uint32_t any = __reduce_or_sync(kAll, vis) & __ballot_sync(kAll, off >= 0);
#pragma unroll 1
        for (int k0 = 0; k0 < 32; k0 += kAhead) {
            if ((any >> k0 & (kAll >> (32 - kAhead))) == 0u) continue;
            Piece v[kAhead];
            uint32_t acc = 0;            // zeros (of any sign) while all is finite
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const long long at = __shfl_sync(kAll, off, k0 + u);
#pragma unroll
                for (int w = 0; w < kWords; ++w) v[u].w[w] = 0u;
                if (any >> (k0 + u) & 1u) v[u] = *reinterpret_cast<const Piece*>(base + at + C * lane);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
#pragma unroll
                for (int w = 0; w < kWords; ++w)
                    acc = sizeof(E) == 2 ? ptx::not_finite_acc(v[u].w[w], acc)
                                         : __float_as_uint(fmaf(__uint_as_float(v[u].w[w]), 0.0f, __uint_as_float(acc)));
            if (!__any_sync(kAll, acc & (sizeof(E) == 2 ? 0x7fff7fffu : 0x7fffffffu))) continue;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const uint32_t rows = __ballot_sync(kAll, vis >> (k0 + u) & 1u);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float x = to_float(v[u].e[c]);
                    if (!(x < INFINITY)) seen[c] |= rows;
                    if (!(x > -INFINITY)) seen[c] |= rows << 16;
                }
            }
        }
    }
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const int row = row0 + i * step;
        E* out = static_cast<E*>(a.o) +
                 (static_cast<size_t>(r.cu0 + tok0 + row / a.G) * a.Hq + hk * a.G + row % a.G) * D + C * lane;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const uint32_t is = seen[c] >> i & 0x10001u;
            if (is == 0u) continue;
            float x = to_float(out[c]);
            if (is & 1u) x += INFINITY;
            if (is >> 16) x -= INFINITY;
            from_float(out + c, x);
        }
    }
}

// A record's l is a sum of exponentials, never negative: its sign carries the
// mark.  (-0 for a marked row that saw no key.)
__device__ __forceinline__ bool row_poisoned(float l) { return signbit(l); }

__device__ __forceinline__ float row_lse(float m, float l) {
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;   // an empty row: log 0
}

}  // namespace tree

// One path's plan for a shape: row tile and tile sizes, CTAs, workspace.
struct TreePlan {
    int rows, KT;            // query rows per row tile, keys per tile
    int tiles;               // row tiles per job (1 or 2)
    int Tq, Tg, Lp, dtok, dsplit, rec_rows, n_cta, job_cost;
    size_t off_ml, off_po, bytes;
};
TreePlan tree_plan(const Paged& p);
cudaError_t launch_tree_simt(const Paged& p, const TreePlan& t, const tree::TreeArgs& a, cudaStream_t s);
cudaError_t launch_tree_sm100(const Paged& p, const TreePlan& t, const tree::TreeArgs& a, cudaStream_t s);
cudaError_t launch_tree_combine(const Paged& p, const TreePlan& t, const tree::TreeArgs& a, cudaStream_t s);

}  // namespace moda
