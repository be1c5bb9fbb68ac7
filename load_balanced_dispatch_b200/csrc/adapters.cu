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
constexpr int kTile = 256;      // rows of a tensor-core row tile
constexpr int kPlanThreads = 1024;
}  // namespace adp

// Rows grouped by adapter (group na: rows without one), in row order inside a group, each group
// padded to a multiple of kPad with -1.
struct AdapterPlan {
    int32_t *perm;   // [m_pad] row of each grouped position, or -1
    int32_t *goff;   // [na + 2] first grouped position of each group
    int32_t *gcnt;   // [na + 1] rows of each group
    int32_t *sseg;   // [na + 2] first segment (kSeg grouped positions) of each group
    int32_t *tstart; // [na + 2] first row tile (kTile grouped positions) of each group
};

static int64_t adapter_padded_rows(int64_t m, int na) { return m + (int64_t)adp::kPad * (na + 1); }
static int64_t adapter_segments(int64_t rows, int groups) { return (rows + adp::kSeg - 1) / adp::kSeg + groups; }

static size_t adapter_plan_layout(int64_t m, int na, AdapterPlan* plan, char* base) {
    size_t off = 0;
    auto take = [&](size_t ints) { char* p = base + off; off += (4 * ints + 255) & ~size_t(255); return (int32_t*)p; };
    int32_t* p;
    p = take((size_t)adapter_padded_rows(m, na)); if (plan) plan->perm = p;
    p = take((size_t)na + 2);                     if (plan) plan->goff = p;
    p = take((size_t)na + 1);                     if (plan) plan->gcnt = p;
    p = take((size_t)na + 2);                     if (plan) plan->sseg = p;
    p = take((size_t)na + 2);                     if (plan) plan->tstart = p;
    return off;
}

struct AdapterWs {
    AdapterPlan plan;
    float *du;       // [m, r]
    float *part;     // [segments, q, p] partial sums of the row contractions
};

static size_t adapter_ws_layout(int64_t m, int d, int n, int r, int na, AdapterWs* w, char* base) {
    size_t off = adapter_plan_layout(m, na, w ? &w->plan : nullptr, base);
    auto take = [&](size_t bytes) { char* p = base + off; off += (bytes + 255) & ~size_t(255); return p; };
    char* p;
    const int64_t mp = adapter_padded_rows(m, na);
    p = take(4 * (size_t)m * r);       if (w) w->du = (float*)p;
    const size_t by_group = (size_t)adapter_segments(mp, na + 1) * r * (size_t)(d > n ? d : n);
    const size_t all = (size_t)adapter_segments(m, 1) * d * n;
    p = take(4 * (by_group > all ? by_group : all)); if (w) w->part = (float*)p;
    return off;
}

// Stable grouping of the rows by adapter in one CTA (block 0). Warp w takes a run of consecutive rows; a
// histogram per warp, their scan over (group, warp), then each warp places its rows: within 32 rows
// the lanes of one group rank themselves by a match. Block 0 also clears the tickets.
// The other blocks, where the tensor cores need it, write W_r [d, n] fp32 in bf16 parts that add up to it:
// three parts as wparts [3, n, d] (transposed, for x W_r), or two as wparts [2, d, nk], nk >= n with zeros
// behind n (for dh W_r^T).
__global__ void __launch_bounds__(adp::kPlanThreads)
adapter_prep_kernel(const int32_t* __restrict__ idx, int64_t m, int na, AdapterPlan p, int32_t* __restrict__ tickets,
                    int64_t ntickets, const float* __restrict__ w_r, int d, int n, int nk, int parts,
                    __nv_bfloat16* __restrict__ wparts) {
    using namespace adp;
    extern __shared__ int hist[];  // [32][na + 1]
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, G = na + 1;
    pdl_trigger();
    pdl_wait();
    if (blockIdx.x > 0) {
        __shared__ float tile[32][33];
        const int nb = (n + 31) / 32, b = (int)blockIdx.x - 1;
        const int t0 = b / nb * 32, j0 = b % nb * 32;
        float v = (t0 + wid < d && j0 + lane < n) ? w_r[(int64_t)(t0 + wid) * n + j0 + lane] : 0.f;
        int j = j0 + lane, t = t0 + wid;
        if (parts == 3) {
            tile[wid][lane] = v;
            __syncthreads();
            j = j0 + wid;
            t = t0 + lane;
            v = tile[lane][wid];
        }
        if (j >= (parts == 3 ? n : nk) || t >= d) return;
        const __nv_bfloat16 p0 = __float2bfloat16_rn(v);
        const float r1 = v - __bfloat162float(p0);
        const __nv_bfloat16 p1 = __float2bfloat16_rn(r1);
        const int64_t o = parts == 3 ? (int64_t)j * d + t : (int64_t)t * nk + j;
        const int64_t plane = parts == 3 ? (int64_t)n * d : (int64_t)d * nk;
        wparts[o] = p0;
        wparts[plane + o] = p1;
        if (parts == 3) wparts[2 * plane + o] = __float2bfloat16_rn(r1 - __bfloat162float(p1));
        return;
    }
    for (int64_t i = tid; i < ntickets; i += kPlanThreads) tickets[i] = 0;
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
        int base = 0, seg = 0, til = 0;
        for (int g0 = 0; g0 < G; g0 += 32) {
            const int g = g0 + lane;
            const int c = g < G ? p.gcnt[g] : 0;
            const int pc = (c + kPad - 1) / kPad * kPad, sc = (pc + kSeg - 1) / kSeg, tc = (pc + kTile - 1) / kTile;
            int a = pc, s = sc, t = tc;
            for (int o = 1; o < 32; o <<= 1) {
                const int ua = __shfl_up_sync(0xffffffffu, a, o), us = __shfl_up_sync(0xffffffffu, s, o);
                const int ut = __shfl_up_sync(0xffffffffu, t, o);
                if (lane >= o) { a += ua; s += us; t += ut; }
            }
            if (g < G) { p.goff[g] = base + a - pc; p.sseg[g] = seg + s - sc; p.tstart[g] = til + t - tc; }
            base += __shfl_sync(0xffffffffu, a, 31);
            seg += __shfl_sync(0xffffffffu, s, 31);
            til += __shfl_sync(0xffffffffu, t, 31);
        }
        if (lane == 0) { p.goff[G] = base; p.sseg[G] = seg; p.tstart[G] = til; }
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

// wparts == NULL: the plan alone.
static cudaError_t launch_adapter_prep(const int32_t* idx, int64_t m, int na, const AdapterPlan& p, int32_t* tickets,
                                       int64_t ntickets, const float* w_r, int d, int n, int nk, int parts,
                                       __nv_bfloat16* wparts, cudaStream_t stream) {
    const size_t smem = sizeof(int) * 32 * (size_t)(na + 1);
    // set on every call: the attribute belongs to the current device
    cudaError_t e = cudaFuncSetAttribute(adapter_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(sizeof(int) * 32 * (kMaxAdapters + 1)));
    if (e != cudaSuccess) return e;
    const unsigned blocks = 1 + (wparts ? (unsigned)((d + 31) / 32) * (unsigned)((n + 31) / 32) : 0);
    return launch_pdl(adapter_prep_kernel, dim3(blocks), dim3(adp::kPlanThreads), smem, stream, idx, m, na, p, tickets,
                      ntickets, w_r, d, n, nk, parts, wparts);
}

// ---- forward: R rows per CTA, thread (column, row group); 32 input columns at a time through
// shared memory. The products of 32 columns are summed first and then added to the row's sum, so the
// rounding errors grow with the number of blocks, not of columns.
template <int NPAD>
__global__ void __launch_bounds__(adp::kThreads)
adapters_rows_kernel(const float* __restrict__ x, const float* __restrict__ w_r, const float* __restrict__ a,
                     const float* __restrict__ bmat, const int32_t* __restrict__ idx, const float* __restrict__ scale,
                     int64_t m, int d, int n, int r, int na, float* __restrict__ logits, float* __restrict__ hidden) {
    using namespace adp;
    constexpr int KC = 32, RG = kThreads / NPAD, R = RG > 16 ? RG : 16, RPT = R / RG, V = Vec16<float>::N;
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
            xs[rr][kk] = (row0 + rr < m && k0 + kk < d) ? x[(row0 + rr) * d + k0 + kk] : 0.f;
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
                Vec16<float>::load(x + row * d + c, xv);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (j0 + q >= r) continue;
                    Vec16<float>::load(a + ((int64_t)ad * r + j0 + q) * d + c, av);
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
                const float* bp = bmat + ((int64_t)ad * n + col) * r;
                for (int j = 0; j < r; ++j) t = fmaf(us[rr][j], bp[j], t);
            }
            logits[row * n + col] = acc[q] + t;
        }
    }
}

// ---- du_ij = s_a sum_e dh_ie B_a[e, j]: a warp per row, lanes along j
__global__ void __launch_bounds__(adp::kThreads)
adapters_du_kernel(const float* __restrict__ dh, const float* __restrict__ bmat, const int32_t* __restrict__ idx,
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
            const float* bp = bmat + (int64_t)ad * n * r + j;
            for (int e = 0; e < n; ++e) t = fmaf(dh[row * n + e], bp[(int64_t)e * r], t);
            t *= scale[ad];
        }
        du[row * r + j] = t;
    }
}

// ---- dx: 16 rows x 128 columns of d per CTA
__global__ void __launch_bounds__(adp::kThreads)
adapters_dx_kernel(const float* __restrict__ dh, const float* __restrict__ w_r, const float* __restrict__ a,
                   const int32_t* __restrict__ idx, const float* __restrict__ du, int64_t m, int d, int n, int r,
                   int na, float* __restrict__ dx) {
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
            const float* ap = a + (int64_t)ad * r * d + c0 + col;
            for (int j = 0; j < r; ++j) t = fmaf(us[rg * 8 + q][j], ap[(int64_t)j * d], t);
        }
        dx[row * d + c0 + col] = acc[q] + t;
    }
}

// ---- row contractions: part[seg][q][p] = sum over the segment's rows of X[row][p] Y[row][q].
// 64 x 64 tiles, 4 x 4 per thread, 16 rows at a time (summed first, then added). perm == NULL: the
// rows in order, one group.
__global__ void __launch_bounds__(adp::kThreads)
rows_outer_kernel(const float* __restrict__ X, int np, const float* __restrict__ Y, int nq, int64_t m, int groups,
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
            xs[rr][c] = (row >= 0 && p0 + c < np) ? X[row * np + p0 + c] : 0.f;
            ys[rr][c] = (row >= 0 && q0 + c < nq) ? Y[row * nq + q0 + c] : 0.f;
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

static cudaError_t launch_rows_contract(const float* X, int np, const float* Y, int nq, int64_t m, int na,
                                        const AdapterPlan& plan, const float* scale, float* part, float* out,
                                        cudaStream_t stream) {
    const bool grouped = plan.perm != nullptr;
    const int64_t segs = grouped ? adapter_segments(adapter_padded_rows(m, na), na + 1)
                                 : (m + adp::kSeg - 1) / adp::kSeg;
    cudaError_t e = cudaSuccess;
    if (segs > 0)
        e = launch_pdl(rows_outer_kernel, dim3((unsigned)((np + 63) / 64), (unsigned)((nq + 63) / 64), (unsigned)segs),
                       dim3(adp::kThreads), 0, stream, X, np, Y, nq, m, na + 1, plan, part);
    if (e != cudaSuccess) return e;
    const int64_t per = (int64_t)np * nq;
    return launch_pdl(rows_fold_kernel, dim3((unsigned)((per + adp::kThreads - 1) / adp::kThreads), grouped ? na : 1),
                      dim3(adp::kThreads), 0, stream, part, per, segs, plan, scale, out);
}

}  // namespace moe
