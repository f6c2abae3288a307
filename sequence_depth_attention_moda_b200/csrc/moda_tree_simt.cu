// moda_tree_simt.cu -- attention of drafted tokens over a paged cache on the
// CUDA cores, fp32 (the operator, the schedule and the masks: moda_tree.cuh),
// and the merging of jobs that several CTAs share (both types).
//
// For one row (new token i of request b, query head h, KV head hk = h / G):
//   s_k = scale <q, K_k>   over the keys k < held and the new keys the token sees
//   s_l = scale <q, Kd_l>  over the token's own depth rows in the window
//   o = (sum p V + sum p Vd) / l,  p = 2^(s log2 e - m),  l = sum p,
// by the online form: a running maximum m and sum l, o rescaled by
// 2^(m_old - m_new) when the maximum grows.  Everything in fp32.
//
// CTA: 256 threads, R query rows, tiles of 32 keys; two CTAs an SM.  Key and value
// rows come by cp.async, kStages tiles ahead (a row that is not there is filled
// with zeros), so the loads of a tile run under the arithmetic of those before.
// A thread computes 4 rows x 4 keys of S and 4 rows x D/8 columns of O; DS = 128/R
// lanes of a warp share such a block and split the head dimension of S and the
// keys of P V, so that all threads have work whatever R is (the parts of S are
// joined by halving exchanges, those of O once a job).  R = 4, 16 or 64, the least
// that holds a request's rows on average: padded rows cost as much arithmetic as
// real ones.  Shared memory rows are padded by 16 bytes, and the lanes are laid out
// so that the eight of a quarter warp read different banks (with the lanes that
// share a block always adjacent, R = 64 took 680 us where it then took 533).
//
// Measured inside a graph (8 requests, 32 query heads over 8, d 128, 8192 keys each): 1
// token 139 us (R = 4; keys and values of 0.54 GB at 3.9 TB/s), 4 tokens 235 (R = 16),
// 16 tokens 517 (R = 64; 17 GFLOP, half of what the FMA pipes can do: shared memory
// reads 8 vectors for 64 multiply-adds, and larger blocks do not fit the registers of
// two CTAs an SM).  One tile in flight and plain loads: 359, 363 and 743 us.
#include "moda_tree.cuh"

namespace moda {
namespace {

using namespace tree;
using ptx::ex2;

constexpr int kThreads = 256;
constexpr int kKeys = 32;

template <int D, int R>
struct Lay {
    static constexpr int kPitch = D + 4;                       // floats of a row
    static constexpr int kStages = D == 128 ? (R == 64 ? 2 : 3) : (R == 64 ? 4 : 5);
    static constexpr int kTile = kKeys * kPitch * 4;           // bytes of a K (or V) tile
    static constexpr int kQ = 0;                               // float [R][kPitch]
    static constexpr int kKV = kQ + R * kPitch * 4;            // [kStages][K, V][32][kPitch]
    static constexpr int kP = kKV + kStages * 2 * kTile;       // float [R][32+4]
    static constexpr int kStat = kP + R * (kKeys + 4) * 4;     // float [3][R]: alpha, m, l
    static constexpr int kStart = (kStat + 3 * R * 4 + 15) / 16 * 16;
    static constexpr int kWalk = kStart + (static_cast<int>(sizeof(Start)) + 15) / 16 * 16;
    static constexpr int kBytes = kWalk + static_cast<int>(sizeof(Walk)) + 16;
    static_assert(2 * (kBytes + 1024) <= 228 * 1024, "two CTAs an SM");
};

__device__ __forceinline__ void copy16(float* dst, const float* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}

// Sums v[0..N) over the DS lanes of a group (lane % DS = ds); lane ds ends with
// the N/DS sums v[ds * N/DS ..] in place (DS <= N), or, for more lanes than
// values, each with the sum it shares with DS/N - 1 others.  Adjacent parts are
// kStep lanes apart.
template <int N, int DS, int kStep>
__device__ __forceinline__ void group_sum(float* v, int ds) {
    if constexpr (DS > 1) {
        constexpr int H = DS / 2;
        if constexpr (N > 1) {
            const bool up = ds & H;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float give = up ? v[i] : v[i + N / 2], keep = up ? v[i + N / 2] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, H * kStep);
            }
            group_sum<N / 2, H, kStep>(v, ds & (H - 1));
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], H * kStep);
            group_sum<1, H, kStep>(v, ds & (H - 1));
        }
    }
}

// The infinities and NaN of a marked job's values (add_not_finite).  A call between the
// jobs, where next to nothing is in registers: elsewhere it cost the tile loop some.
template <int D, int R>
__device__ __noinline__ void finish_job(const TreeArgs& a, const Job& j) {
    constexpr int n = R < 8 ? 1 : R / 8;
    const int rows = j.ntok * a.G, row0 = static_cast<int>(threadIdx.x >> 5) * n;
    if (row0 < rows) add_not_finite<float, D, 4>(a, j.r, j.b, j.hk, j.tok0, row0, 1, min(n, rows - row0));
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 2) tree_simt_kernel(const __grid_constant__ TreeArgs a) {
    using L = Lay<D, R>;
    constexpr int DS = 128 / R;           // lanes sharing a block
    constexpr int TPR = kThreads / R;     // softmax threads per row
    constexpr int KPT = kKeys / TPR > 0 ? kKeys / TPR : 1;    // keys each has
    constexpr int NC = D / 32;            // float4 columns of O per thread
    constexpr int CH = D / 4;             // 16-byte chunks of a row
    constexpr int CPT = kKeys * CH / kThreads;    // chunks of a K (and V) tile a thread copies
    extern __shared__ __align__(16) unsigned char smem[];
    float* sq = reinterpret_cast<float*>(smem + L::kQ);
    float* skv = reinterpret_cast<float*>(smem + L::kKV);
    float* sp = reinterpret_cast<float*>(smem + L::kP);
    float* salpha = reinterpret_cast<float*>(smem + L::kStat);
    float* sm = salpha + R;
    float* sl = sm + R;
    Start* st = reinterpret_cast<Start*>(smem + L::kStart);
    // the walk over the jobs, advanced by thread 0: in registers it would crowd out the accumulators
    Walk& w = *reinterpret_cast<Walk*>(smem + L::kWalk);
    int* spoison = reinterpret_cast<int*>(&w + 1);
    int* smore = spoison + 1;
    int* sfinish = smore + 1;             // the last job's outputs lack its infinities and NaN

    const int tid = threadIdx.x;
    if (tid == 0) *sfinish = 0;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    schedule(a, st);
    // A quarter warp reads eight 16-byte pieces at a time, free of bank conflicts if
    // it is eight parts of a block or eight blocks' same part.
    constexpr int kStep = DS < 8 ? 8 : 1;
    const int ds = tid / kStep % DS;
    const int cg = kStep == 1 ? tid / DS % 8 : tid % 8;       // keys cg + 8c of S, columns 4cg + 32j of O
    const int rg = tid / DS / 8;          // rows 4rg .. 4rg+3
    const int page = 1 << a.page_shift;
    const int wr0 = 4 * ((tid & ~31) / DS / 8), wr1 = 4 * ((tid | 31) / DS / 8) + 4;      // the warp's rows

    for (bool first = true;; first = false) {
        __syncthreads();                  // the previous job is done with shared memory, its outputs are stored
        if (*sfinish) {
            finish_job<D, R>(a, w.j);
            __syncthreads();
        }
        if (tid == 0) {
            *sfinish = 0;
            *smore = first ? w.begin(a, *st) : w.next(a);
            *spoison = 0;
        }
        __syncthreads();
        if (!*smore) break;
        const Job& j = w.j;
        const int rows = j.ntok * a.G;
        // This thread's chunks of a tile: column tid % CH of rows tid / CH, + kThreads / CH, ...
        // Table entries of the rows, asked for a tile before they are used.
        int entry[CPT];
        auto ask = [&](int t) {
#pragma unroll
            for (int u = 0; u < CPT; ++u) {
                const int key = t * kKeys + tid / CH + u * (kThreads / CH);
                entry[u] = t < min(w.i1, j.nseq) && key < j.r.held + j.r.n ? table_entry(a, j.b, key) : -1;
            }
        };
        auto load = [&](int t, int stage) {
            const bool seq = t < j.nseq;
            const float* kb = static_cast<const float*>(seq ? a.kc : a.kd);
            const float* vb = static_cast<const float*>(seq ? a.vc : a.vd);
            float* dst = skv + stage * (2 * L::kTile / 4);
#pragma unroll
            for (int u = 0; u < CPT; ++u) {
                const int r = tid / CH + u * (kThreads / CH), c = tid % CH * 4;
                long long off = -1;       // the row's first element, -1: not there
                if (seq) {
                    const int key = t * kKeys + r;
                    if (key < j.r.held + j.r.n) {
                        const int p = checked_page(a, entry[u]);
                        if (p >= 0) off = ((static_cast<long long>(p) * a.Hk + j.hk) * page + (key & (page - 1))) * D;
                    }
                } else {
                    const int dt = t - j.nseq;
                    int tok, d;
                    if (a.Lw <= a.KT) {
                        const int at = r / a.Lp;
                        tok = at < a.dtok ? dt * a.dtok + at : j.ntok;
                        d = r - at * a.Lp;
                    } else {
                        tok = dt / a.dsplit;
                        d = (dt - tok * a.dsplit) * a.KT + r;
                    }
                    if (d < a.Lw && tok < j.ntok)
                        off = ((static_cast<long long>(j.r.cu0 + j.tok0 + tok) * a.Hk + j.hk) * a.L + a.win_lo + d) * D;
                }
                const bool there = off >= 0;
                const long long from = there ? off + c : 0;
                copy16(dst + r * L::kPitch + c, kb + from, there);
                copy16(dst + L::kTile / 4 + r * L::kPitch + c, vb + from, there);
            }
        };
        ask(w.i0);
#pragma unroll 1
        for (int s = 0; s < L::kStages - 1; ++s) {
            if (w.i0 + s < w.i1) {
                load(w.i0 + s, s);
                ask(w.i0 + s + 1);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        for (int i = tid; i < R * CH; i += kThreads) {
            const int r = i / CH, c = i % CH * 4;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r < rows) {
                const size_t row = static_cast<size_t>(j.r.cu0 + j.tok0 + r / a.G) * a.Hq + j.hk * a.G + r % a.G;
                v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + row * D + c);
            }
            *reinterpret_cast<float4*>(&sq[r * L::kPitch + c]) =
                make_float4(v.x * a.scale_log2, v.y * a.scale_log2, v.z * a.scale_log2, v.w * a.scale_log2);
        }
        float o[4][NC][4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < NC; ++c) o[r][c][0] = o[r][c][1] = o[r][c][2] = o[r][c][3] = 0.0f;
        // softmax state of row tid / TPR, the same in its threads
        const int srw = tid / TPR, sub = tid % TPR;
        float m = -INFINITY, l = 0.0f;
        const int token = j.tok0 + srw / a.G;        // relative to the request
        const bool real = srw < rows;

        int stage = 0;
        for (int t = w.i0; t < w.i1; ++t) {
            const bool dep = t >= j.nseq;
            const int dt = t - j.nseq;
            // rows of V from key row `from` on are masked for some query row
            const int from = dep ? 0 : j.r.held - t * kKeys;
            float* sk = skv + stage * (2 * L::kTile / 4);
            float* sv = sk + L::kTile / 4;
            asm volatile("cp.async.wait_group %0;" ::"n"(L::kStages - 2) : "memory");
            if (from < kKeys) {           // each thread looks over the chunks it copied
#pragma unroll
                for (int u = 0; u < CPT; ++u) {
                    const int r = tid / CH + u * (kThreads / CH), c = tid % CH * 4;
                    if (r < from) continue;
                    float4 v = *reinterpret_cast<float4*>(sv + r * L::kPitch + c);
                    if (isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w)) continue;
                    v.x = isfinite(v.x) ? v.x : 0.0f;
                    v.y = isfinite(v.y) ? v.y : 0.0f;
                    v.z = isfinite(v.z) ? v.z : 0.0f;
                    v.w = isfinite(v.w) ? v.w : 0.0f;
                    *reinterpret_cast<float4*>(sv + r * L::kPitch + c) = v;
                    *spoison = 1;
                }
            }
            __syncthreads();              // the tile is there, and the one before done with
            {
                const int next = t + L::kStages - 1;
                if (next < w.i1) {
                    load(next, stage == 0 ? L::kStages - 1 : stage - 1);
                    ask(next + 1);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
            // Whether any of the warp's rows sees any of the tile's: not those behind the last
            // token, nor, in a depth tile, other tokens' rows (their p will be 0).  22 requests of
            // up to 78 tokens over 221 keys: 103 us without, 97 with it.
            bool mine = true;
            if (R > 4 && wr0 >= rows) mine = false;
            if (R > 4 && dep) {
                const int tok = a.Lw <= a.KT ? dt * a.dtok : dt / a.dsplit, n = a.Lw <= a.KT ? a.dtok : 1;
                mine = mine && wr0 < (tok + n) * a.G && wr1 > tok * a.G;
            }
            // S: 4 rows x 4 keys over this lane's share of the head dimension
            if (mine) {
                float s[16] = {};             // [row][key]
#pragma unroll 4
                for (int d = ds * 4; d < D; d += 4 * DS) {
                    float4 qv[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(&sq[(4 * rg + i) * L::kPitch + d]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float4 kv = *reinterpret_cast<const float4*>(&sk[(cg + 8 * c) * L::kPitch + d]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            float x = s[4 * r + c];
                            x = fmaf(qv[r].x, kv.x, x);
                            x = fmaf(qv[r].y, kv.y, x);
                            x = fmaf(qv[r].z, kv.z, x);
                            s[4 * r + c] = fmaf(qv[r].w, kv.w, x);
                        }
                    }
                }
                group_sum<16, DS, kStep>(s, ds);
                {
                    constexpr int part = DS <= 16 ? 16 / DS : 1;
                    const int first = DS <= 16 ? ds * part : ds / (DS / 16);
                    if (DS <= 16 || ds % (DS / 16) == 0) {
#pragma unroll
                        for (int i = 0; i < part; ++i) {
                            const int x = first + i;             // row x / 4, key x % 4 of the block
                            sp[(4 * rg + x / 4) * (kKeys + 4) + cg + 8 * (x % 4)] = s[i];
                        }
                    }
                }
            }
            __syncthreads();
            // online softmax: this row's keys sub, sub + TPR, ... (a row's spare threads repeat the last keys)
            {
                const uint32_t vis = !real ? 0u
                                           : (dep ? dep_visible(a, token - j.tok0, dt, 0)
                                                  : seq_visible(a, j.r, token, t * kKeys));
                float x[KPT], mx = -INFINITY;
                float* row = &sp[srw * (kKeys + 4)];
#pragma unroll
                for (int i = 0; i < KPT; ++i) {
                    const int c = (sub + i * TPR) & (kKeys - 1);
                    x[i] = vis >> c & 1u ? row[c] : -INFINITY;
                    mx = fmaxf(mx, x[i]);
                }
                constexpr int W = TPR < 32 ? TPR : 32;       // the row's threads within a warp
#pragma unroll
                for (int y = 1; y < W; y <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
                const float mn = fmaxf(m, mx);
                const float ref = mn == -INFINITY ? 0.0f : mn;       // a row that saw no key yet
                const float alpha = m == -INFINITY ? 1.0f : ex2(m - mn);   // its o and l are 0
                float ps = 0.0f;
                if (TPR > kKeys) __syncthreads();            // two warps read the row
#pragma unroll
                for (int i = 0; i < KPT; ++i) {
                    const float p = ex2(x[i] - ref);
                    ps += p;
                    row[(sub + i * TPR) & (kKeys - 1)] = p;
                }
#pragma unroll
                for (int y = 1; y < W; y <<= 1) ps += __shfl_xor_sync(0xffffffffu, ps, y);
                l = fmaf(l, alpha, ps);
                m = mn;
                if (sub == 0) salpha[srw] = alpha;
            }
            __syncthreads();
            // O = O alpha + P V over this lane's share of the keys (alpha is 1 where p is 0)
            if (mine) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float al = salpha[4 * rg + r];
#pragma unroll
                    for (int c = 0; c < NC; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[r][c][e] *= al;
                }
#pragma unroll 8
                for (int k = ds; k < kKeys; k += DS) {
                    float p[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) p[r] = sp[(4 * rg + r) * (kKeys + 4) + k];
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const float4 v = *reinterpret_cast<const float4*>(&sv[k * L::kPitch + 4 * cg + 32 * c]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            o[r][c][0] = fmaf(p[r], v.x, o[r][c][0]);
                            o[r][c][1] = fmaf(p[r], v.y, o[r][c][1]);
                            o[r][c][2] = fmaf(p[r], v.z, o[r][c][2]);
                            o[r][c][3] = fmaf(p[r], v.w, o[r][c][3]);
                        }
                    }
                }
            }
            if (++stage == L::kStages) stage = 0;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (sub == 0) {
            sm[srw] = m;
            sl[srw] = l;
        }
        __syncthreads();
        const bool poison = *spoison != 0;
        const bool whole = w.whole();
        const size_t slot = w.slot();
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int y = 1; y < DS; y <<= 1)
                        o[r][c][e] += __shfl_xor_sync(0xffffffffu, o[r][c][e], y * kStep);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 4 * rg + r;
            if (row >= rows || ds != 0) continue;
            const float lr = sl[row], mr = sm[row];
            if (whole) {
                const int tk = j.tok0 + row / a.G;
                const size_t orow = static_cast<size_t>(j.r.cu0 + tk) * a.Hq + j.hk * a.G + row % a.G;
                const float inv = lr == 0.0f ? 0.0f : 1.0f / lr;
                float* out = static_cast<float*>(a.o) + orow * D;
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int col = 4 * cg + 32 * c;
                    *reinterpret_cast<float4*>(out + col) =
                        make_float4(o[r][c][0] * inv, o[r][c][1] * inv, o[r][c][2] * inv, o[r][c][3] * inv);
                }
                if (poison) *sfinish = 1;
                if (cg == 0) a.lse[orow] = row_lse(mr, lr);
            } else {
                const size_t rec = slot * a.rec_rows + row;
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    *reinterpret_cast<float4*>(a.po + rec * D + 4 * cg + 32 * c) =
                        make_float4(o[r][c][0], o[r][c][1], o[r][c][2], o[r][c][3]);
                if (cg == 0) a.ml[rec] = make_float2(mr, poison ? -lr : lr);
            }
        }
    }
}

template <int D, int R>
cudaError_t launch_r(const TreePlan& t, const TreeArgs& a, cudaStream_t s) {
    const void* f = reinterpret_cast<const void*>(tree_simt_kernel<D, R>);
    const cudaError_t e = set_max_dynamic_smem(f, Lay<D, R>::kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(t.n_cta);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Lay<D, R>::kBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_simt_kernel<D, R>, a);
}

template <int D>
cudaError_t launch_d(const TreePlan& t, const TreeArgs& a, cudaStream_t s) {
    if (t.rows == 4) return launch_r<D, 4>(t, a, s);
    return t.rows == 16 ? launch_r<D, 16>(t, a, s) : launch_r<D, 64>(t, a, s);
}

// Merges the records of a job that range ends cut: o = sum_i o_i 2^(m_i - M) / sum_i l_i 2^(m_i - M).
// CTA (c, y) looks at the job in which part c begins, and works if the part before
// holds the job's first tile and some other its last one; a warp takes one row.
// Bound by latency (headers, records, outputs: three dependent accesses, about 3 us
// behind the grid it waits for); up to kBatch records of a row are in flight.
constexpr int kCombineWarps = 8;
constexpr int kBatch = 8;

template <typename E, int D>
__global__ void __launch_bounds__(32 * kCombineWarps) tree_combine_kernel(const __grid_constant__ TreeArgs a) {
    constexpr int C = D / 32;
    const int c = static_cast<int>(blockIdx.x) + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const CtaHeader h = a.hdr[c];
    const int P = h.n_ranges;
    if (c >= P) return;
    Job j;
    j.b = h.b;
    j.hk = h.hk;
    j.r = h.r;
    set_group(a, j, h.group);
    // The parts that hold the beginnings of the job's first and last tile.  Part c
    // is the one to work if it is the second of several.
    const int first = range_of(h.job_start + tile_begin(a, j, 0), h.x_total, P);
    const int last = range_of(h.job_start + tile_begin(a, j, j.nt - 1), h.x_total, P);
    if (c != first + 1 || last == first) return;
    const int n = last - first + 1;
    auto slot_of = [&](int i) -> size_t { return 2 * static_cast<size_t>(first + i) + (i == 0); };   // see Walk::slot
    bool poison = false;
    for (int row = blockIdx.y * kCombineWarps + warp; row < j.ntok * a.G; row += gridDim.y * kCombineWarps) {
        // online over the records, kBatch of them in flight at a time
        float M = -INFINITY, l = 0.0f, acc[C] = {};
        for (int i0 = 0; i0 < n; i0 += kBatch) {
            float2 ml[kBatch];
            float v[kBatch][C];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                ml[u] = make_float2(-INFINITY, 0.0f);
                if (i0 + u >= n) continue;
                const size_t rec = slot_of(i0 + u) * a.rec_rows + row;
                ml[u] = a.ml[rec];
#pragma unroll
                for (int e = 0; e < C; ++e) v[u][e] = a.po[rec * D + lane + 32 * e];
            }
            float mn = M;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) mn = fmaxf(mn, ml[u].x);
            const float ref = mn == -INFINITY ? 0.0f : mn;
            const float alpha = M == -INFINITY ? 1.0f : ex2(M - mn);     // l and acc are 0 until a key was seen
            l *= alpha;
#pragma unroll
            for (int e = 0; e < C; ++e) acc[e] *= alpha;
            M = mn;
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                poison |= row_poisoned(ml[u].y);
                if (ml[u].x == -INFINITY && ml[u].y == 0.0f) continue;    // a record without keys: no O was written
                const float wt = ex2(ml[u].x - ref);
                l = fmaf(fabsf(ml[u].y), wt, l);
#pragma unroll
                for (int e = 0; e < C; ++e) acc[e] = fmaf(v[u][e], wt, acc[e]);
            }
        }
        const float ref = M == -INFINITY ? 0.0f : M;
        const int tk = j.tok0 + row / a.G;
        const size_t orow = static_cast<size_t>(j.r.cu0 + tk) * a.Hq + j.hk * a.G + row % a.G;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int e = 0; e < C; ++e) from_float(static_cast<E*>(a.o) + orow * D + lane + 32 * e, acc[e] * inv);
        if (lane == 0) a.lse[orow] = row_lse(ref, l);
    }
    if (poison) {                        // a record's mark is that of all its rows
        __syncwarp();
        const int step = gridDim.y * kCombineWarps, row0 = blockIdx.y * kCombineWarps + warp;
        const int n = (j.ntok * a.G - row0 + step - 1) / step;           // (> 0: some row was marked)
        for (int i = 0; i < n; i += 16)
            add_not_finite<E, D, 4>(a, j.r, j.b, j.hk, j.tok0, row0 + i * step, step, min(16, n - i));
    }
}

template <typename E, int D>
cudaError_t launch_combine(const TreePlan& t, const TreeArgs& a, cudaStream_t s) {
    if (t.n_cta < 2) return cudaSuccess;
    // launched before the split kernel ends (it waits for it on the device)
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int y = (t.rec_rows + kCombineWarps - 1) / kCombineWarps;
    cfg.gridDim = dim3(t.n_cta - 1, y < 8 ? y : 8);
    cfg.blockDim = dim3(32 * kCombineWarps);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_combine_kernel<E, D>, a);
}

}  // namespace

cudaError_t launch_tree_simt(const Paged& p, const TreePlan& t, const TreeArgs& a, cudaStream_t s) {
    return p.d == 128 ? launch_d<128>(t, a, s) : launch_d<64>(t, a, s);
}

cudaError_t launch_tree_combine(const Paged& p, const TreePlan& t, const TreeArgs& a, cudaStream_t s) {
    if (p.elem_bytes == 4)
        return p.d == 128 ? launch_combine<float, 128>(t, a, s) : launch_combine<float, 64>(t, a, s);
    return p.d == 128 ? launch_combine<__nv_bfloat16, 128>(t, a, s) : launch_combine<__nv_bfloat16, 64>(t, a, s);
}

}  // namespace moda
