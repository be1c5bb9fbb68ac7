// adapters.cu -- the router projection with a low-rank adapter per request, forward and backward:
// the fp32 FMA kernels (fp32 activations, and the parts that both types share).
//
// "Switch Transformers paper review" (tildalice.io/?p=118), Switch Routing Step 1, h = x W_r, with
// the selective-precision recipe (logits in fp32). Row i of the batch belongs to a request whose
// adapter is a = adapter_idx[i] (-1: none):
//   u_i = A_a x_i  (r values, "hidden"),   h_i = x_i W_r + s_a B_a u_i.
// Backward, dh = dL/dh:
//   du_i = s_a B_a^T dh_i,  dx_i = W_r dh_i + A_a^T du_i,
//   dA_a = sum_{i in a} du_i x_i^T,  dB_a = s_a sum_{i in a} dh_i u_i^T,  dW_r = sum_i x_i dh_i^T.
#include "common.cuh"

namespace moe {

namespace adp {
constexpr int kThreads = 256;
constexpr int kPad = 64;        // a group's rows are padded to this many in the grouped order
constexpr int kSeg = 512;       // rows of one partial sum of the row contractions
constexpr int kPlanThreads = 1024;
}  // namespace adp

// Rows grouped by adapter (group na: rows without one), in row order inside a group, each group
// padded to a multiple of kPad with -1.
struct AdapterPlan {
    int32_t *perm;   // [m_pad] row of each grouped position, or -1
    int32_t *goff;   // [na + 2] first grouped position of each group
    int32_t *gcnt;   // [na + 1] rows of each group
    int32_t *sseg;   // [na + 2] first segment (kSeg grouped positions) of each group
};

static int64_t adapter_padded_rows(int64_t m, int na) { return m + (int64_t)adp::kPad * (na + 1); }
static int64_t adapter_segments(int64_t rows, int groups) { return (rows + adp::kSeg - 1) / adp::kSeg + groups; }

struct AdapterWs {
    AdapterPlan plan;
    float *du;       // [m, r]
    float *part;     // [segments, q, p] partial sums of the row contractions
};

static size_t adapter_ws_layout(int64_t m, int d, int n, int r, int na, AdapterWs* w, char* base) {
    size_t off = 0;
    auto take = [&](size_t bytes) { char* p = base + off; off += (bytes + 255) & ~size_t(255); return p; };
    char* p;
    const int64_t mp = adapter_padded_rows(m, na);
    p = take(4 * (size_t)mp);          if (w) w->plan.perm = (int32_t*)p;
    p = take(4 * (size_t)(na + 2));    if (w) w->plan.goff = (int32_t*)p;
    p = take(4 * (size_t)(na + 1));    if (w) w->plan.gcnt = (int32_t*)p;
    p = take(4 * (size_t)(na + 2));    if (w) w->plan.sseg = (int32_t*)p;
    p = take(4 * (size_t)m * r);       if (w) w->du = (float*)p;
    const size_t by_group = (size_t)adapter_segments(mp, na + 1) * r * (size_t)(d > n ? d : n);
    const size_t all = (size_t)adapter_segments(m, 1) * d * n;
    p = take(4 * (by_group > all ? by_group : all)); if (w) w->part = (float*)p;
    return off;
}

// Stable grouping of the rows by adapter in one CTA. Warp w takes a run of consecutive rows; a
// histogram per warp, their scan over (group, warp), then each warp places its rows: within 32 rows
// the lanes of one group rank themselves by a match.
__global__ void __launch_bounds__(adp::kPlanThreads)
adapter_plan_kernel(const int32_t* __restrict__ idx, int64_t m, int na, AdapterPlan p) {
    using namespace adp;
    extern __shared__ int hist[];  // [32][na + 1]
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, G = na + 1;
    pdl_trigger();
    pdl_wait();
    for (int i = tid; i < 32 * G; i += kPlanThreads) hist[i] = 0;
    __syncthreads();
    const int64_t per = ((m + 31) / 32 + 31) / 32 * 32;  // rows per warp, a multiple of 32
    const int64_t r0 = min(wid * per, m), r1 = min(r0 + per, m);
    for (int64_t b = r0; b < r1; b += 32) {
        const int64_t r = b + lane;
        int g = -1;
        if (r < r1) {
            g = idx[r];
            if (g < -1 || g >= na) record_error(kErrAdapterIndex);
            if (g < 0 || g >= na) g = na;
        }
        const unsigned same = __match_any_sync(0xffffffffu, g);
        if (g >= 0 && lane == __ffs(same) - 1) hist[wid * G + g] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // group totals, then offsets by one warp
    for (int g = tid; g < G; g += kPlanThreads) {
        int c = 0;
        for (int w = 0; w < 32; ++w) c += hist[w * G + g];
        p.gcnt[g] = c;
    }
    __syncthreads();
    if (wid == 0) {
        int base = 0, seg = 0;
        for (int g0 = 0; g0 < G; g0 += 32) {
            const int g = g0 + lane;
            const int c = g < G ? p.gcnt[g] : 0;
            const int pc = (c + kPad - 1) / kPad * kPad, sc = (pc + kSeg - 1) / kSeg;
            int a = pc, s = sc;
            for (int o = 1; o < 32; o <<= 1) {
                const int ta = __shfl_up_sync(0xffffffffu, a, o), ts = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) { a += ta; s += ts; }
            }
            if (g < G) { p.goff[g] = base + a - pc; p.sseg[g] = seg + s - sc; }
            base += __shfl_sync(0xffffffffu, a, 31);
            seg += __shfl_sync(0xffffffffu, s, 31);
        }
        if (lane == 0) { p.goff[G] = base; p.sseg[G] = seg; }
    }
    __syncthreads();
    for (int g = tid; g < G; g += kPlanThreads) {
        int at = p.goff[g];
        for (int w = 0; w < 32; ++w) { const int c = hist[w * G + g]; hist[w * G + g] = at; at += c; }
        for (; at < p.goff[g + 1]; ++at) p.perm[at] = -1;
    }
    __syncthreads();
    for (int64_t b = r0; b < r1; b += 32) {
        const int64_t r = b + lane;
        int g = -1;
        if (r < r1) {
            g = idx[r];
            if (g < 0 || g >= na) g = na;
        }
        const unsigned same = __match_any_sync(0xffffffffu, g);
        const int rank = __popc(same & ((1u << lane) - 1u));
        const int at = g >= 0 ? hist[wid * G + g] : 0;
        __syncwarp();
        if (g >= 0) {
            p.perm[at + rank] = (int32_t)r;
            if (rank == 0) hist[wid * G + g] = at + __popc(same);
        }
        __syncwarp();
    }
}

static cudaError_t launch_adapter_plan(const int32_t* idx, int64_t m, int na, const AdapterPlan& p,
                                       cudaStream_t stream) {
    const size_t smem = sizeof(int) * 32 * (size_t)(na + 1);
    cudaError_t e = cudaFuncSetAttribute(adapter_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(sizeof(int) * 32 * (kMaxAdapters + 1)));
    if (e != cudaSuccess) return e;
    return launch_pdl(adapter_plan_kernel, dim3(1), dim3(adp::kPlanThreads), smem, stream, idx, m, na, p);
}

// ---- forward: R rows per CTA, thread (column, row group); 32 input columns at a time through
// shared memory. The products of 32 columns are summed first and then added to the row's sum, so the
// rounding errors grow with the number of blocks, not of columns.
template <typename T, int NPAD>
__global__ void __launch_bounds__(adp::kThreads)
adapters_rows_kernel(const T* __restrict__ x, const float* __restrict__ w_r, const T* __restrict__ a,
                     const T* __restrict__ bmat, const int32_t* __restrict__ idx, const float* __restrict__ scale,
                     int64_t m, int d, int n, int r, int na, float* __restrict__ logits, float* __restrict__ hidden) {
    using namespace adp;
    constexpr int KC = 32, RG = kThreads / NPAD, R = RG > 16 ? RG : 16, RPT = R / RG, V = Vec16<T>::N;
    __shared__ float xs[R][KC + 1];
    __shared__ float ws[KC][NPAD + 1];
    __shared__ float us[R][kMaxRank + 1];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int col = tid % NPAD, rg = tid / NPAD;
    pdl_trigger();
    pdl_wait();
    const int64_t row0 = (int64_t)blockIdx.x * R;
    float acc[RPT];
#pragma unroll
    for (int q = 0; q < RPT; ++q) acc[q] = 0.f;
    for (int k0 = 0; k0 < d; k0 += KC) {
        for (int i = tid; i < R * KC; i += kThreads) {
            const int rr = i / KC, kk = i % KC;
            xs[rr][kk] = (row0 + rr < m && k0 + kk < d) ? Elem<T>::load(x + (row0 + rr) * d + k0 + kk) : 0.f;
        }
        for (int i = tid; i < KC * n; i += kThreads) {
            const int kk = i / n, j = i % n;
            ws[kk][j] = k0 + kk < d ? w_r[(int64_t)(k0 + kk) * n + j] : 0.f;
        }
        __syncthreads();
        float blk[RPT];
#pragma unroll
        for (int q = 0; q < RPT; ++q) blk[q] = 0.f;
        if (col < n) {
#pragma unroll 8
            for (int kk = 0; kk < KC; ++kk) {
                const float wv = ws[kk][col];
#pragma unroll
                for (int q = 0; q < RPT; ++q) blk[q] = fmaf(xs[rg + RG * q][kk], wv, blk[q]);
            }
        }
#pragma unroll
        for (int q = 0; q < RPT; ++q) acc[q] += blk[q];
        __syncthreads();
    }
    // u: a warp per row, four of the adapter's rows at a time, lanes along d
    for (int rr = wid; rr < R; rr += kThreads / 32) {
        const int64_t row = row0 + rr;
        if (row >= m) break;
        int ad = idx[row];
        if (ad < -1 || ad >= na) { if (lane == 0) record_error(kErrAdapterIndex); ad = -1; }
        if (ad < 0) {
            for (int j = lane; j < r; j += 32) { us[rr][j] = 0.f; if (hidden) hidden[row * r + j] = 0.f; }
            continue;
        }
        const float sc = scale[ad];
        for (int j0 = 0; j0 < r; j0 += 4) {
            float s[4] = {0.f, 0.f, 0.f, 0.f};
            for (int c = lane * V; c < d; c += 32 * V) {
                float xv[V], av[V];
                Vec16<T>::load(x + row * d + c, xv);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (j0 + q >= r) continue;
                    Vec16<T>::load(a + ((int64_t)ad * r + j0 + q) * d + c, av);
                    float t = 0.f;
#pragma unroll
                    for (int i = 0; i < V; ++i) t = fmaf(xv[i], av[i], t);
                    s[q] += t;
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float t = warp_sum(s[q]);
                if (lane == q && j0 + q < r) {
                    us[rr][j0 + q] = sc * t;
                    if (hidden) hidden[row * r + j0 + q] = t;
                }
            }
        }
    }
    __syncthreads();
    if (col < n) {
#pragma unroll
        for (int q = 0; q < RPT; ++q) {
            const int rr = rg + RG * q;
            const int64_t row = row0 + rr;
            if (row >= m) continue;
            const int ad = idx[row];
            float t = 0.f;
            if (ad >= 0 && ad < na) {
                const T* bp = bmat + ((int64_t)ad * n + col) * r;
                for (int j = 0; j < r; ++j) t = fmaf(us[rr][j], Elem<T>::load(bp + j), t);
            }
            logits[row * n + col] = acc[q] + t;
        }
    }
}

// ---- du_ij = s_a sum_e dh_ie B_a[e, j]: a warp per row, lanes along j
template <typename T>
__global__ void __launch_bounds__(adp::kThreads)
adapters_du_kernel(const float* __restrict__ dh, const T* __restrict__ bmat, const int32_t* __restrict__ idx,
                   const float* __restrict__ scale, int64_t m, int n, int r, int na, float* __restrict__ du) {
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    const int64_t row = (int64_t)blockIdx.x * (adp::kThreads / 32) + (threadIdx.x >> 5);
    if (row >= m) return;
    const int ad = idx[row];
    const bool has = ad >= 0 && ad < na;
    for (int j = lane; j < r; j += 32) {
        float t = 0.f;
        if (has) {
            const T* bp = bmat + (int64_t)ad * n * r + j;
            for (int e = 0; e < n; ++e) t = fmaf(dh[row * n + e], Elem<T>::load(bp + (int64_t)e * r), t);
            t *= scale[ad];
        }
        du[row * r + j] = t;
    }
}

// ---- dx: 16 rows x 128 columns of d per CTA
template <typename T>
__global__ void __launch_bounds__(adp::kThreads)
adapters_dx_kernel(const float* __restrict__ dh, const float* __restrict__ w_r, const T* __restrict__ a,
                   const int32_t* __restrict__ idx, const float* __restrict__ du, int64_t m, int d, int n, int r,
                   int na, T* __restrict__ dx) {
    using namespace adp;
    constexpr int R = 16, DC = 128, EC = 32;
    __shared__ float hs[R][kMaxExperts + 1];
    __shared__ float us[R][kMaxRank + 1];
    __shared__ float ws[EC][DC + 1];
    const int tid = threadIdx.x;
    pdl_trigger();
    pdl_wait();
    const int64_t row0 = (int64_t)blockIdx.x * R;
    const int c0 = blockIdx.y * DC, col = tid % DC, rg = tid / DC;  // two row groups of eight
    for (int i = tid; i < R * n; i += kThreads) {
        const int64_t row = row0 + i / n;
        hs[i / n][i % n] = row < m ? dh[row * n + i % n] : 0.f;
    }
    for (int i = tid; i < R * r; i += kThreads) {
        const int64_t row = row0 + i / r;
        us[i / r][i % r] = row < m ? du[row * r + i % r] : 0.f;
    }
    float acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = 0.f;
    for (int e0 = 0; e0 < n; e0 += EC) {
        __syncthreads();
        for (int i = tid; i < EC * DC; i += kThreads) {
            const int kk = i / EC, e = i % EC;
            ws[e][kk] = (c0 + kk < d && e0 + e < n) ? w_r[(int64_t)(c0 + kk) * n + e0 + e] : 0.f;
        }
        __syncthreads();
        const int top = min(EC, n - e0);
        for (int e = 0; e < top; ++e) {
            const float wv = ws[e][col];
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] = fmaf(hs[rg * 8 + q][e0 + e], wv, acc[q]);
        }
    }
    if (c0 + col >= d) return;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const int64_t row = row0 + rg * 8 + q;
        if (row >= m) continue;
        const int ad = idx[row];
        float t = 0.f;
        if (ad >= 0 && ad < na) {
            const T* ap = a + (int64_t)ad * r * d + c0 + col;
            for (int j = 0; j < r; ++j) t = fmaf(us[rg * 8 + q][j], Elem<T>::load(ap + (int64_t)j * d), t);
        }
        Elem<T>::store(dx + row * d + c0 + col, acc[q] + t);
    }
}

// ---- row contractions: part[seg][q][p] = sum over the segment's rows of X[row][p] Y[row][q].
// 64 x 64 tiles, 4 x 4 per thread, 16 rows at a time (summed first, then added). perm == NULL: the
// rows in order, one group.
template <typename TX, typename TY>
__global__ void __launch_bounds__(adp::kThreads)
rows_outer_kernel(const TX* __restrict__ X, int np, const TY* __restrict__ Y, int nq, int64_t m, int groups,
                  AdapterPlan plan, float* __restrict__ part) {
    using namespace adp;
    constexpr int RB = 16;
    __shared__ float xs[RB][65], ys[RB][65];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    pdl_trigger();
    pdl_wait();
    const int seg = blockIdx.z;
    int64_t b = (int64_t)seg * kSeg, end = min(b + kSeg, m);
    if (plan.perm) {
        if (seg >= plan.sseg[groups]) return;
        int lo = 0, hi = groups;  // largest group with sseg <= seg
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (plan.sseg[mid] <= seg) lo = mid; else hi = mid;
        }
        b = plan.goff[lo] + (int64_t)(seg - plan.sseg[lo]) * kSeg;
        end = min(b + kSeg, (int64_t)plan.goff[lo + 1]);
    } else if (b >= m) {
        return;
    }
    const int p0 = blockIdx.x * 64, q0 = blockIdx.y * 64;
    float acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    for (int64_t at = b; at < end; at += RB) {
        for (int i = tid; i < RB * 64; i += kThreads) {
            const int rr = i >> 6, c = i & 63;
            int64_t row = -1;
            if (at + rr < end) row = plan.perm ? plan.perm[at + rr] : at + rr;
            xs[rr][c] = (row >= 0 && p0 + c < np) ? Elem<TX>::load(X + row * np + p0 + c) : 0.f;
            ys[rr][c] = (row >= 0 && q0 + c < nq) ? Elem<TY>::load(Y + row * nq + q0 + c) : 0.f;
        }
        __syncthreads();
        float blk[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) blk[i][j] = 0.f;
#pragma unroll
        for (int rr = 0; rr < RB; ++rr) {
            float xv[4], yv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) { xv[i] = xs[rr][tx + 16 * i]; yv[i] = ys[rr][ty + 16 * i]; }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) blk[i][j] = fmaf(xv[j], yv[i], blk[i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] += blk[i][j];
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int p = p0 + tx + 16 * j, q = q0 + ty + 16 * i;
            if (p < np && q < nq) part[((int64_t)seg * nq + q) * np + p] = acc[i][j];
        }
}

// out[g][i] = s_g * sum over the group's segments, in order, of part[seg][i] (zero for no rows)
__global__ void __launch_bounds__(adp::kThreads)
rows_fold_kernel(const float* __restrict__ part, int64_t per, int64_t segs, AdapterPlan plan,
                 const float* __restrict__ scale, float* __restrict__ out) {
    pdl_trigger();
    pdl_wait();
    const int g = blockIdx.y;
    const int64_t i = (int64_t)blockIdx.x * adp::kThreads + threadIdx.x;
    if (i >= per) return;
    const int64_t s0 = plan.perm ? plan.sseg[g] : 0, s1 = plan.perm ? plan.sseg[g + 1] : segs;
    float t = 0.f;
    for (int64_t s = s0; s < s1; ++s) t += part[s * per + i];
    out[g * per + i] = scale ? scale[g] * t : t;
}

template <typename TX, typename TY>
static cudaError_t launch_rows_contract(const TX* X, int np, const TY* Y, int nq, int64_t m, int na,
                                        const AdapterPlan& plan, const float* scale, float* part, float* out,
                                        cudaStream_t stream) {
    const bool grouped = plan.perm != nullptr;
    const int64_t segs = grouped ? adapter_segments(adapter_padded_rows(m, na), na + 1)
                                 : (m + adp::kSeg - 1) / adp::kSeg;
    cudaError_t e = cudaSuccess;
    if (segs > 0)
        e = launch_pdl(rows_outer_kernel<TX, TY>, dim3((unsigned)((np + 63) / 64), (unsigned)((nq + 63) / 64), (unsigned)segs),
                       dim3(adp::kThreads), 0, stream, X, np, Y, nq, m, na + 1, plan, part);
    if (e != cudaSuccess) return e;
    const int64_t per = (int64_t)np * nq;
    return launch_pdl(rows_fold_kernel, dim3((unsigned)((per + adp::kThreads - 1) / adp::kThreads), grouped ? na : 1),
                      dim3(adp::kThreads), 0, stream, part, per, segs, plan, scale, out);
}

size_t router_adapters_workspace_bytes(int64_t m, int32_t d, int32_t n, int32_t r, int32_t na, moe_dtype dt) {
    (void)m; (void)d; (void)n; (void)r; (void)na; (void)dt;
    return 0;
}

size_t router_adapters_grad_workspace_bytes(int64_t m, int32_t d, int32_t n, int32_t r, int32_t na, moe_dtype dt) {
    (void)dt;
    if (m < 0 || d < 1 || n < 1 || r < 1 || na < 1) return 0;
    return adapter_ws_layout(m, d, n, r, na, nullptr, nullptr);
}

template <typename T>
static cudaError_t launch_adapters_rows(const T* x, const float* w_r, const T* a, const T* b, const int32_t* idx,
                                        const float* scale, int64_t m, int d, int n, int r, int na, float* logits,
                                        float* hidden, cudaStream_t stream) {
#define MOE_ADAPTER_ROWS(NP)                                                                                       \
    do {                                                                                                           \
        constexpr int RG = adp::kThreads / NP, R = RG > 16 ? RG : 16;                                              \
        return launch_pdl(adapters_rows_kernel<T, NP>, dim3((unsigned)((m + R - 1) / R)), dim3(adp::kThreads), 0,  \
                          stream, x, w_r, a, b, idx, scale, m, d, n, r, na, logits, hidden);                       \
    } while (0)
    if (n <= 8) MOE_ADAPTER_ROWS(8);
    if (n <= 16) MOE_ADAPTER_ROWS(16);
    if (n <= 32) MOE_ADAPTER_ROWS(32);
    if (n <= 64) MOE_ADAPTER_ROWS(64);
    if (n <= 128) MOE_ADAPTER_ROWS(128);
    MOE_ADAPTER_ROWS(256);
#undef MOE_ADAPTER_ROWS
}

cudaError_t launch_router_adapters(const void* x, moe_dtype dt, const float* w_r, const void* a, const void* b,
                                   const int32_t* idx, const float* scale, int64_t m, int d, int n, int r, int na,
                                   float* logits, float* hidden, void* workspace, cudaStream_t stream) {
    (void)workspace;
    if (m == 0) return cudaSuccess;
    if (dt == MOE_BF16)
        return launch_adapters_rows(static_cast<const __nv_bfloat16*>(x), w_r, static_cast<const __nv_bfloat16*>(a),
                                    static_cast<const __nv_bfloat16*>(b), idx, scale, m, d, n, r, na, logits, hidden,
                                    stream);
    return launch_adapters_rows(static_cast<const float*>(x), w_r, static_cast<const float*>(a),
                                static_cast<const float*>(b), idx, scale, m, d, n, r, na, logits, hidden, stream);
}

template <typename T>
static cudaError_t launch_adapters_grad_t(const float* dh, const T* x, const float* w_r, const T* a, const T* b,
                                          const int32_t* idx, const float* scale, const float* hidden, int64_t m,
                                          int d, int n, int r, int na, T* dx, float* da, float* db, float* dw_r,
                                          void* workspace, cudaStream_t stream) {
    AdapterWs w;
    adapter_ws_layout(m, d, n, r, na, &w, static_cast<char*>(workspace));
    cudaError_t e = launch_adapter_plan(idx, m, na, w.plan, stream);
    if (e != cudaSuccess) return e;
    if (m > 0) {
        const int rows = adp::kThreads / 32;
        e = launch_pdl(adapters_du_kernel<T>, dim3((unsigned)((m + rows - 1) / rows)), dim3(adp::kThreads), 0, stream,
                       dh, b, idx, scale, m, n, r, na, w.du);
        if (e != cudaSuccess) return e;
        if (dx) {
            e = launch_pdl(adapters_dx_kernel<T>, dim3((unsigned)((m + 15) / 16), (unsigned)((d + 127) / 128)),
                           dim3(adp::kThreads), 0, stream, dh, w_r, a, idx, w.du, m, d, n, r, na, dx);
            if (e != cudaSuccess) return e;
        }
    }
    e = launch_rows_contract(x, d, w.du, r, m, na, w.plan, nullptr, w.part, da, stream);
    if (e != cudaSuccess) return e;
    e = launch_rows_contract(hidden, r, dh, n, m, na, w.plan, scale, w.part, db, stream);
    if (e != cudaSuccess || !dw_r) return e;
    AdapterPlan none = {};
    return launch_rows_contract(dh, n, x, d, m, na, none, nullptr, w.part, dw_r, stream);
}

cudaError_t launch_router_adapters_grad(const float* dh, const void* x, moe_dtype dt, const float* w_r, const void* a,
                                        const void* b, const int32_t* idx, const float* scale, const float* hidden,
                                        int64_t m, int d, int n, int r, int na, void* dx, float* da, float* db,
                                        float* dw_r, void* workspace, cudaStream_t stream) {
    if (dt == MOE_BF16)
        return launch_adapters_grad_t(dh, static_cast<const __nv_bfloat16*>(x), w_r,
                                      static_cast<const __nv_bfloat16*>(a), static_cast<const __nv_bfloat16*>(b), idx,
                                      scale, hidden, m, d, n, r, na, static_cast<__nv_bfloat16*>(dx), da, db, dw_r,
                                      workspace, stream);
    return launch_adapters_grad_t(dh, static_cast<const float*>(x), w_r, static_cast<const float*>(a),
                                  static_cast<const float*>(b), idx, scale, hidden, m, d, n, r, na,
                                  static_cast<float*>(dx), da, db, dw_r, workspace, stream);
}

}  // namespace moe
