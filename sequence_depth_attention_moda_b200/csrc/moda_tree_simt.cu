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
// CTA: 256 threads, R query rows, tiles of 64 keys in shared memory.  A thread
// computes 4 rows x 4 keys of S and 4 rows x D/16 columns of O; with R < 64 the
// 256 threads exceed the 4x4 blocks, and DS = 64/R adjacent lanes split the
// head dimension of S and the keys of P V, so all of them have work (shuffles
// join the parts).  R = 16 is taken when the requests' rows fit in it on
// average (G * tokens <= 16): a 64-row tile would do four times the work on
// rows that are not there.
#include "moda_tree.cuh"

namespace moda {
namespace {

using namespace tree;
using ptx::ex2;

constexpr int kThreads = 256;
constexpr int kKeys = 64;

template <int D, int R>
struct Lay {
    static constexpr int kQ = 0;                              // float [R][D+4]
    static constexpr int kK = kQ + R * (D + 4) * 4;           // float [64][D+4]
    static constexpr int kV = kK + kKeys * (D + 4) * 4;       // float [64][D]
    static constexpr int kP = kV + kKeys * D * 4;             // float [R][64+4]
    static constexpr int kRow = kP + R * (kKeys + 4) * 4;     // long long [64]: element offset, -1: no row
    static constexpr int kStat = kRow + kKeys * 8;            // float [3][R]: alpha, m, l
    static constexpr int kStart = (kStat + 3 * R * 4 + 15) / 16 * 16;
    static constexpr int kBytes = kStart + static_cast<int>(sizeof(Start)) + 16;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <int D, int R>
__global__ void __launch_bounds__(kThreads) tree_simt_kernel(const __grid_constant__ TreeArgs a) {
    using L = Lay<D, R>;
    constexpr int DS = 64 / R;            // lanes sharing a 4x4 block
    constexpr int TPR = kThreads / R;     // softmax threads per row
    extern __shared__ __align__(16) unsigned char smem[];
    float* sq = reinterpret_cast<float*>(smem + L::kQ);
    float* sk = reinterpret_cast<float*>(smem + L::kK);
    float* sv = reinterpret_cast<float*>(smem + L::kV);
    float* sp = reinterpret_cast<float*>(smem + L::kP);
    long long* srow = reinterpret_cast<long long*>(smem + L::kRow);
    float* salpha = reinterpret_cast<float*>(smem + L::kStat);
    float* sm = salpha + R;
    float* sl = sm + R;
    Start* st = reinterpret_cast<Start*>(smem + L::kStart);
    int* spoison = reinterpret_cast<int*>(st + 1);

    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    schedule(a, st);
    const int tid = threadIdx.x;
    const int ds = tid % DS;
    const int cg = (tid / DS) % 16;       // keys cg + 16c of S, columns 4cg + 64j of O
    const int rg = tid / DS / 16;         // rows 4rg .. 4rg+3
    const int page = 1 << a.page_shift;

    Walk w;
    for (bool more = w.begin(a, *st); more; more = w.next(a)) {
        const Job& j = w.j;
        const int rows = j.ntok * a.G;
        __syncthreads();                  // the previous job is done with shared memory
        if (tid == 0) *spoison = 0;
        for (int i = tid; i < R * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = i % (D / 4) * 4;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r < rows) {
                const size_t row = static_cast<size_t>(j.r.cu0 + j.tok0 + r / a.G) * a.Hq + j.hk * a.G + r % a.G;
                v = load4(static_cast<const float*>(a.q) + row * D + c);
            }
            *reinterpret_cast<float4*>(&sq[r * (D + 4) + c]) =
                make_float4(v.x * a.scale_log2, v.y * a.scale_log2, v.z * a.scale_log2, v.w * a.scale_log2);
        }
        float o[4][D / 64][4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < D / 64; ++c) o[r][c][0] = o[r][c][1] = o[r][c][2] = o[r][c][3] = 0.0f;
        // softmax state of row tid / TPR, the same in its TPR threads
        const int srw = tid / TPR, sub = tid % TPR;
        float m = -INFINITY, l = 0.0f;
        const int token = j.tok0 + srw / a.G;        // relative to the request
        const bool real = srw < rows;

        for (int t = w.i0; t < w.i1; ++t) {
            const bool dep = t >= j.nseq;
            const int dt = t - j.nseq;
            // rows of V from key row `from` on are masked for some query row
            const int from = dep ? 0 : j.r.held - t * kKeys;
            __syncthreads();
            if (tid < kKeys) {
                long long off = -1;
                if (!dep) {
                    const int key = t * kKeys + tid;
                    if (key < j.r.held + j.r.n) {
                        const int p = page_of(a, j.b, key);
                        if (p >= 0)
                            off = ((static_cast<long long>(p) * a.Hk + j.hk) * page + (key & (page - 1))) * D;
                    }
                } else {
                    int tok, d;
                    if (a.Lw <= a.KT) {
                        tok = dt * a.dtok + tid / a.Lp;
                        d = tid % a.Lp;
                        if (tid / a.Lp >= a.dtok || d >= a.Lw) tok = j.ntok;
                    } else {
                        tok = dt / a.dsplit;
                        d = dt % a.dsplit * a.KT + tid;
                        if (d >= a.Lw) tok = j.ntok;
                    }
                    if (tok < j.ntok)
                        off = ((static_cast<long long>(j.r.cu0 + j.tok0 + tok) * a.Hk + j.hk) * a.L + a.win_lo + d) * D;
                }
                srow[tid] = off;
            }
            __syncthreads();
            const float* kb = static_cast<const float*>(dep ? a.kd : a.kc);
            const float* vb = static_cast<const float*>(dep ? a.vd : a.vc);
#pragma unroll 8
            for (int i = tid; i < kKeys * (D / 4); i += kThreads) {
                const int r = i / (D / 4), c = i % (D / 4) * 4;
                const long long off = srow[r];
                float4 kv = make_float4(0.0f, 0.0f, 0.0f, 0.0f), vv = kv;
                if (off >= 0) {
                    kv = load4(kb + off + c);
                    vv = load4(vb + off + c);
                }
                if (r >= from) {
                    float* e = &vv.x;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (!isfinite(e[k])) {
                            e[k] = 0.0f;
                            *spoison = 1;
                        }
                }
                *reinterpret_cast<float4*>(&sk[r * (D + 4) + c]) = kv;
                *reinterpret_cast<float4*>(&sv[r * D + c]) = vv;
            }
            __syncthreads();
            // S: 4 rows x 4 keys over this lane's share of the head dimension
            float s[4][4] = {};
#pragma unroll 4
            for (int d = ds * 4; d < D; d += 4 * DS) {
                float4 qv[4], kv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    qv[i] = *reinterpret_cast<const float4*>(&sq[(4 * rg + i) * (D + 4) + d]);
                    kv[i] = *reinterpret_cast<const float4*>(&sk[(cg + 16 * i) * (D + 4) + d]);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        s[r][c] = fmaf(qv[r].x, kv[c].x, s[r][c]);
                        s[r][c] = fmaf(qv[r].y, kv[c].y, s[r][c]);
                        s[r][c] = fmaf(qv[r].z, kv[c].z, s[r][c]);
                        s[r][c] = fmaf(qv[r].w, kv[c].w, s[r][c]);
                    }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
#pragma unroll
                    for (int x = 1; x < DS; x <<= 1) s[r][c] += __shfl_xor_sync(0xffffffffu, s[r][c], x);
                    if (ds == 0) sp[(4 * rg + r) * (kKeys + 4) + cg + 16 * c] = s[r][c];
                }
            __syncthreads();
            // online softmax: this row's keys sub, sub + TPR, ...
            {
                uint32_t vis[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    vis[h] = !real ? 0u
                                   : (dep ? dep_visible(a, token - j.tok0, dt, 32 * h)
                                          : seq_visible(a, j.r, token, t * kKeys + 32 * h));
                float x[kKeys / TPR], mx = -INFINITY;
#pragma unroll
                for (int k = 0; k < kKeys / TPR; ++k) {
                    const int c = sub + k * TPR;
                    x[k] = ((c < 32 ? vis[0] : vis[1]) >> (c & 31)) & 1u ? sp[srw * (kKeys + 4) + c] : -INFINITY;
                    mx = fmaxf(mx, x[k]);
                }
#pragma unroll
                for (int y = 1; y < TPR; y <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
                const float mn = fmaxf(m, mx);
                const float ref = mn == -INFINITY ? 0.0f : mn;       // a row that saw no key yet
                const float alpha = m == -INFINITY ? 1.0f : ex2(m - mn);   // its o and l are 0
                float ps = 0.0f;
#pragma unroll
                for (int k = 0; k < kKeys / TPR; ++k) {
                    const float p = ex2(x[k] - ref);
                    ps += p;
                    sp[srw * (kKeys + 4) + sub + k * TPR] = p;
                }
#pragma unroll
                for (int y = 1; y < TPR; y <<= 1) ps += __shfl_xor_sync(0xffffffffu, ps, y);
                l = fmaf(l, alpha, ps);
                m = mn;
                if (sub == 0) salpha[srw] = alpha;
            }
            __syncthreads();
            // O = O alpha + P V over this lane's share of the keys
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float al = salpha[4 * rg + r];
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[r][c][e] *= al;
            }
#pragma unroll 4
            for (int k = ds; k < kKeys; k += DS) {
                float4 vv[D / 64];
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    vv[c] = *reinterpret_cast<const float4*>(&sv[k * D + 4 * cg + 64 * c]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float p = sp[(4 * rg + r) * (kKeys + 4) + k];
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        o[r][c][0] = fmaf(p, vv[c].x, o[r][c][0]);
                        o[r][c][1] = fmaf(p, vv[c].y, o[r][c][1]);
                        o[r][c][2] = fmaf(p, vv[c].z, o[r][c][2]);
                        o[r][c][3] = fmaf(p, vv[c].w, o[r][c][3]);
                    }
                }
            }
        }
        if (sub == 0) {
            sm[srw] = m;
            sl[srw] = l;
        }
        __syncthreads();
        const bool poison = *spoison != 0;
        const bool whole = w.whole();
        const size_t slot = w.slot();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 4 * rg + r;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int x = 1; x < DS; x <<= 1)
                        o[r][c][e] += __shfl_xor_sync(0xffffffffu, o[r][c][e], x);
            if (row >= rows || ds != 0) continue;
            const float lr = sl[row], mr = sm[row];
            if (whole) {
                const int tk = j.tok0 + row / a.G;
                const size_t orow = static_cast<size_t>(j.r.cu0 + tk) * a.Hq + j.hk * a.G + row % a.G;
                const float inv = lr == 0.0f ? 0.0f : 1.0f / lr;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const int col = 4 * cg + 64 * c;
                    float* out = static_cast<float*>(a.o) + orow * D;
                    *reinterpret_cast<float4*>(out + col) =
                        make_float4(o[r][c][0] * inv, o[r][c][1] * inv, o[r][c][2] * inv, o[r][c][3] * inv);
                    if (poison) add_not_finite<float, D>(a, j.r, j.b, j.hk, tk, out, col, 1, 4);
                }
                if (cg == 0) a.lse[orow] = row_lse(mr, lr);
            } else {
                const size_t rec = slot * a.rec_rows + row;
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    *reinterpret_cast<float4*>(a.po + rec * D + 4 * cg + 64 * c) =
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

// Merges the records of a job that range ends cut: o = sum_i o_i 2^(m_i - M) / sum_i l_i 2^(m_i - M).
// CTA (c, y) looks at the job that holds range c's first tile, and works if c
// is the first range end inside that job; a warp takes one row.
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
    const int first = range_of(h.job_start, h.x_total, P);
    const int last = range_of(h.job_start + tile_begin(j, j.nt - 1), h.x_total, P);
    if (c != first + 1 || last == first) return;
    const int n = last - first + 1;
    auto slot_of = [&](int i) -> size_t { return 2 * static_cast<size_t>(first + i) + (i == 0); };   // see Walk::slot
    for (int row = blockIdx.y * kCombineWarps + warp; row < j.ntok * a.G; row += gridDim.y * kCombineWarps) {
        // online over the records, kBatch of them in flight at a time
        float M = -INFINITY, l = 0.0f, acc[C] = {};
        bool poison = false;
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
        if (poison) add_not_finite<E, D>(a, j.r, j.b, j.hk, tk, static_cast<E*>(a.o) + orow * D, lane, 32, C);
        if (lane == 0) a.lse[orow] = row_lse(ref, l);
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
    if (p.d == 128) return t.rows == 16 ? launch_r<128, 16>(t, a, s) : launch_r<128, 64>(t, a, s);
    return t.rows == 16 ? launch_r<64, 16>(t, a, s) : launch_r<64, 64>(t, a, s);
}

cudaError_t launch_tree_combine(const Paged& p, const TreePlan& t, const TreeArgs& a, cudaStream_t s) {
    if (p.elem_bytes == 4)
        return p.d == 128 ? launch_combine<float, 128>(t, a, s) : launch_combine<float, 64>(t, a, s);
    return p.d == 128 ? launch_combine<__nv_bfloat16, 128>(t, a, s) : launch_combine<__nv_bfloat16, 64>(t, a, s);
}

}  // namespace moda
