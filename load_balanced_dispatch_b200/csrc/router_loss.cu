// router_loss.cu -- the router's losses over a ragged batch and their gradient with respect to
// the router logits.
//
// "Switch Transformers paper review" (tildalice.io/?p=118), auxiliary load balancing loss
// L = alpha N sum_i f_i P_i (f_i fixed by the routing decision, the gradient through P_i);
// "Qwen global-batch load balance" (agentlenshq.com): the same loss on separate parts of the
// batch, averaged. Here the parts are the sequences of a ragged batch. The z-loss (mean squared
// log-sum-exp of a token's logits) and the gates' own gradient share the pass over the logits.
//
//   router_loss_chunk_kernel  one CTA per kRows consecutive rows. A row belongs to L lanes (four
//     or eight logits each, 16-byte loads), so a warp holds 32 / L rows; the scores are summed in
//     fp64 per sequence run of the chunk, the picks counted with integer atomics in shared memory.
//     Partial sums go to slot (chunk + sequence): walking the rows, each new slot advances the
//     chunk or the sequence, so the index is unique and nchunk + nseq slots are enough.
//   router_loss_fold_kernel   one CTA per (sequence, 32 experts) and per (whole batch, 32 experts)
//     folds its chunks in order; the last CTA (a ticket) adds the sequences' losses in order.
//   router_loss_grad_kernel   one pass: logits in, gradient out.
//
// No floating-point atomics, every fold in a fixed order: the results are bit-reproducible.
// Bound by reading the logits (and writing the gradient): 4 m n bytes each.
#include "common.cuh"

namespace moe {

namespace rloss {
constexpr int kRows = 128;     // rows per CTA of the chunk pass
constexpr int kThreads = 256;
constexpr int kFoldCols = 32;  // experts per CTA of the fold
}  // namespace rloss

struct RouterLossWs {
    double *psum, *tsum;       // [nchunk + nseq, n] per run; [nchunk, n] per chunk, all its runs
    double *zsum, *part;       // [nchunk] sum of squared log-sum-exp; [nseq + 1, col blocks] sum_i f_i P_i
    int32_t *pcnt, *tcnt;      // picks, as psum and tsum
    int32_t *ptok, *ttok;      // valid tokens, [nchunk + nseq] and [nchunk]
    int32_t* ticket;
};

static size_t router_loss_layout(int64_t m, int n, int64_t nseq, RouterLossWs* w, char* base) {
    const size_t nch = (size_t)((m + rloss::kRows - 1) / rloss::kRows), runs = nch + (size_t)nseq;
    const size_t ncb = (size_t)(n + rloss::kFoldCols - 1) / rloss::kFoldCols;
    size_t off = 0;
    auto take = [&](size_t bytes) { char* p = base + off; off += (bytes + 255) & ~size_t(255); return p; };
    char* p;
    p = take(8 * runs * n);             if (w) w->psum = (double*)p;
    p = take(8 * nch * n);              if (w) w->tsum = (double*)p;
    p = take(8 * nch);                  if (w) w->zsum = (double*)p;
    p = take(8 * ((size_t)nseq + 1) * ncb); if (w) w->part = (double*)p;
    p = take(4 * runs * n);             if (w) w->pcnt = (int32_t*)p;
    p = take(4 * nch * n);              if (w) w->tcnt = (int32_t*)p;
    p = take(4 * runs);                 if (w) w->ptok = (int32_t*)p;
    p = take(4 * nch);                  if (w) w->ttok = (int32_t*)p;
    p = take(4);                        if (w) w->ticket = (int32_t*)p;
    return off;
}

size_t router_loss_workspace_bytes(int64_t m, int32_t n, int64_t nseq) {
    if (m < 0 || n < 1 || nseq < 1) return 0;
    return router_loss_layout(m, n, nseq, nullptr, nullptr);
}

// Index of the sequence that holds row r: the last s in [-1, nseq] with off[s] <= r (nseq: the
// row lies behind the last sequence). Empty sequences in between are passed over.
__device__ __forceinline__ int seq_of_row(const int32_t* __restrict__ off, int nseq, int64_t r) {
    int lo = 0, hi = nseq + 1;  // first index with off > r
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)off[mid] <= r) lo = mid + 1; else hi = mid;
    }
    return lo - 1;
}

// The 4 V logits that lane `sub` of the row's L lanes owns: columns 4 (sub + L v) .. + 3, v < V.
// Columns past n read as -inf (no score, no weight).
template <int L, int V>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int n, bool vec, int sub, float (&h)[4 * V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int j = 4 * (sub + L * v);
        if (vec) {
            if (j < n) {
                const float4 t = *reinterpret_cast<const float4*>(row + j);
                h[4 * v] = t.x; h[4 * v + 1] = t.y; h[4 * v + 2] = t.z; h[4 * v + 3] = t.w;
            } else {
                h[4 * v] = h[4 * v + 1] = h[4 * v + 2] = h[4 * v + 3] = -INFINITY;
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) h[4 * v + q] = j + q < n ? row[j + q] : -INFINITY;
        }
    }
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// h_j <- exp(h_j - top) / sum, and the log-sum-exp of a row held by L lanes. A row whose logits are
// all -inf has no scores: 0 throughout and lse = 0. NaN and +inf give NaN.
template <int L, int V>
__device__ __forceinline__ float row_softmax(float (&h)[4 * V]) {
    float top = h[0];
#pragma unroll
    for (int q = 1; q < 4 * V; ++q) top = fmaxf(top, h[q]);
    top = lanes_max<L>(top);
    float s = 0.f;
    if (top == -INFINITY) {  // fmaxf passes over NaN: keep it in the sum
#pragma unroll
        for (int q = 0; q < 4 * V; ++q) { h[q] = h[q] == -INFINITY ? 0.f : h[q]; s += h[q]; }
    } else {
#pragma unroll
        for (int q = 0; q < 4 * V; ++q) { h[q] = expf(h[q] - top); s += h[q]; }
    }
    s = lanes_sum<L>(s);
    if (top == -INFINITY) return s;
    const float inv = 1.f / s;
#pragma unroll
    for (int q = 0; q < 4 * V; ++q) h[q] *= inv;
    return top + logf(s);
}

__device__ __forceinline__ float logistic(float h) { return 1.f / (1.f + expf(-h)); }

template <int L, int V>
__global__ void __launch_bounds__(rloss::kThreads)
router_loss_chunk_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx, int64_t m, int n, int k,
                         const int32_t* __restrict__ off, int nseq, const uint8_t* __restrict__ mask, int fn,
                         int want_z, RouterLossWs w) {
    using namespace rloss;
    constexpr int RW = 32 / L;                      // rows a warp holds
    constexpr int GROUPS = (kThreads / 32) * RW;    // rows the CTA holds at a time
    constexpr int U = GROUPS >= 64 ? 1 : 4;         // rows in flight per lane group
    constexpr int FS = 4 * V * L + 1;
    extern __shared__ double fold[];                // [GROUPS][FS] a row group's sums
    __shared__ double tot_p[kMaxExperts];
    __shared__ int cnt[kMaxExperts], tot_c[kMaxExperts];
    __shared__ double zpart[GROUPS];
    __shared__ int ntok;
    const int tid = threadIdx.x, lane = tid & 31, sub = lane % L, grp = (tid >> 5) * RW + lane / L;
    const bool vec = (n & 3) == 0;
    pdl_trigger();
    pdl_wait();
    const int64_t c = blockIdx.x, r0 = c * kRows, r1 = min(r0 + (int64_t)kRows, m);
    if (c == 0 && tid == 0) *w.ticket = 0;
    if (tid < n) { tot_p[tid] = 0.0; tot_c[tid] = 0; }
    double z = 0.0;
    int total = 0;
    for (int64_t at = r0; at < r1;) {
        const int s = seq_of_row(off, nseq, at);
        if (s >= nseq) break;                                        // behind the last sequence
        const int64_t next = min((int64_t)off[s + 1], r1);           // > at: off[s + 1] is the first offset above it
        if (s < 0) { at = next; continue; }                          // before the first
        if (tid < n) cnt[tid] = 0;
        if (tid == 0) ntok = 0;
        __syncthreads();
        double acc[4 * V];
#pragma unroll
        for (int q = 0; q < 4 * V; ++q) acc[q] = 0.0;
        // every lane of a warp runs the same number of rounds: the row's lanes reduce together
        for (int64_t base = at; base < next; base += GROUPS * U) {
            bool live[U];
            int pick[U];
            float h[U][4 * V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = base + grp + GROUPS * u;
                live[u] = r < next && (!mask || mask[r]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t r = base + grp + GROUPS * u;
#pragma unroll
                for (int q = 0; q < 4 * V; ++q) h[u][q] = -INFINITY;
                if (live[u]) load_row<L, V>(logits + r * n, n, vec, sub, h[u]);
                pick[u] = live[u] && sub < k ? idx[r * k + sub] : 0;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (fn == MOE_SIGMOID) {
                    float e[4 * V];
#pragma unroll
                    for (int q = 0; q < 4 * V; ++q) e[q] = h[u][q];
                    if (want_z) {
                        const float lse = row_softmax<L, V>(e);
                        if (sub == 0) z += (double)lse * (double)lse;
                    }
#pragma unroll
                    for (int q = 0; q < 4 * V; ++q) h[u][q] = live[u] ? logistic(h[u][q]) : 0.f;
                } else {
                    const float lse = row_softmax<L, V>(h[u]);
                    if (sub == 0) z += (double)lse * (double)lse;
                }
                if (live[u]) {
                    const int64_t r = base + grp + GROUPS * u;
                    if (sub == 0) atomicAdd(&ntok, 1);
                    int e = pick[u];
                    for (int t = sub; t < k;) {
                        if (e < 0 || e >= n) record_error(kErrExpertIndex);
                        else atomicAdd(&cnt[e], 1);
                        t += L;
                        if (t < k) e = idx[r * k + t];
                    }
                }
            }
            // U scores are added in fp32, the sums over the rounds in fp64
#pragma unroll
            for (int q = 0; q < 4 * V; ++q) {
                float t = h[0][q];
                if constexpr (U == 4) t = (h[0][q] + h[1][q]) + (h[2][q] + h[3][q]);
                acc[q] += (double)t;
            }
        }
        // column 4 (sub + L v) + q of row group g sits at fold[g][4 (sub + L v) + q]
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int q = 0; q < 4; ++q) fold[grp * FS + 4 * (sub + L * v) + q] = acc[4 * v + q];
        __syncthreads();
        const int64_t slot = c + s;
        if (tid < n) {
            double t = 0.0;
#pragma unroll 8
            for (int g = 0; g < GROUPS; ++g) t += fold[g * FS + tid];
            w.psum[slot * n + tid] = t;
            w.pcnt[slot * n + tid] = cnt[tid];
            tot_p[tid] += t;
            tot_c[tid] += cnt[tid];
        }
        if (tid == 0) { w.ptok[slot] = ntok; total += ntok; }
        __syncthreads();
        at = next;
    }
    if (sub == 0) zpart[grp] = z;
    if (tid < n) { w.tsum[c * n + tid] = tot_p[tid]; w.tcnt[c * n + tid] = tot_c[tid]; }
    __syncthreads();
    if (tid == 0) {
        double t = 0.0;
        for (int g = 0; g < GROUPS; ++g) t += zpart[g];
        w.zsum[c] = t;
        w.ttok[c] = total;
    }
}

// blockIdx.x = sequence (nseq: the whole batch), blockIdx.y = 32 experts; 8 rows of 32 lanes.
__global__ void __launch_bounds__(rloss::kThreads)
router_loss_fold_kernel(int64_t m, int n, int k, const int32_t* __restrict__ off, int nseq, double alpha,
                        double alpha_seq, double z_coef, float* __restrict__ loss, int32_t* __restrict__ counts,
                        int32_t* __restrict__ tokens, float* __restrict__ f, float* __restrict__ P, RouterLossWs w) {
    using namespace rloss;
    constexpr int W = kThreads / 32;
    __shared__ double ps[W][kFoldCols];
    __shared__ int cs[W][kFoldCols];
    __shared__ int ts[W];
    __shared__ double red[kThreads];
    __shared__ int redi[kThreads];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.x, e = blockIdx.y * kFoldCols + lane;
    const bool whole = s == nseq;
    const int64_t nch = (m + kRows - 1) / kRows;
    int64_t c0 = 0, c1 = nch;  // the chunks that hold rows of the sequence
    if (!whole) {
        int64_t b = off[s], t = off[s + 1];
        if (tid == 0 && (b < 0 || t < b || t > m)) record_error(kErrSeqOffsets);
        b = max((int64_t)0, min(b, m));
        t = max(b, min(t, m));
        c0 = b / kRows;
        c1 = t > b ? (t - 1) / kRows + 1 : c0;
    }
    const double* psum = whole ? w.tsum : w.psum + (int64_t)s * n;
    const int32_t* pcnt = whole ? w.tcnt : w.pcnt + (int64_t)s * n;
    const int32_t* ptok = whole ? w.ttok : w.ptok + s;
    double a = 0.0;
    int cn = 0, tk = 0;
    for (int64_t c = c0 + wid; c < c1; c += W) {
        if (e < n) { a += psum[c * n + e]; cn += pcnt[c * n + e]; }
        tk += ptok[c];
    }
    ps[wid][lane] = a;
    cs[wid][lane] = cn;
    if (lane == 0) ts[wid] = tk;
    __syncthreads();
    if (wid == 0) {
        double p = 0.0;
        int cc = 0, T = 0;
        for (int q = 0; q < W; ++q) { p += ps[q][lane]; cc += cs[q][lane]; T += ts[q]; }
        double prod = 0.0;
        if (e < n) {
            const double fe = T > 0 ? (double)cc / ((double)k * (double)T) : 0.0;
            const double pe = T > 0 ? p / (double)T : 0.0;
            counts[(int64_t)s * n + e] = cc;
            f[(int64_t)s * n + e] = (float)fe;
            P[(int64_t)s * n + e] = (float)pe;
            prod = fe * pe;
        }
        prod = warp_sum_d(prod);
        if (lane == 0) {
            w.part[(int64_t)s * gridDim.y + blockIdx.y] = prod;
            if (blockIdx.y == 0) tokens[s] = T;
        }
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(w.ticket, 1) == (int)(gridDim.x * gridDim.y) - 1;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    // the last CTA: the sequences' losses in order (thread t takes sequences t, t + 256, ...)
    const int ncb = gridDim.y;
    double seq = 0.0;
    int full = 0;
    for (int q = tid; q < nseq; q += kThreads) {
        for (int b = 0; b < ncb; ++b) seq += __ldcg(w.part + (int64_t)q * ncb + b);
        full += __ldcg(tokens + q) > 0;
    }
    double z = 0.0;
    for (int64_t c = tid; c < nch; c += kThreads) z += __ldcg(w.zsum + c);
    red[tid] = seq;
    redi[tid] = full;
    __syncthreads();
    if (tid == 0) {
        for (int q = 1; q < kThreads; ++q) { seq += red[q]; full += redi[q]; }
    }
    __syncthreads();
    red[tid] = z;
    __syncthreads();
    if (tid == 0) {
        for (int q = 1; q < kThreads; ++q) z += red[q];
        const int T = __ldcg(tokens + nseq);
        double batch = 0.0;
        for (int b = 0; b < ncb; ++b) batch += __ldcg(w.part + (int64_t)nseq * ncb + b);
        batch *= alpha * (double)n;
        seq = full > 0 ? alpha_seq * (double)n * seq / (double)full : 0.0;
        z = T > 0 ? z_coef * z / (double)T : 0.0;
        loss[0] = (float)(batch + seq + z);
        loss[1] = (float)batch;
        loss[2] = (float)seq;
        loss[3] = (float)z;
    }
}

// dL/dp_j of a token of sequence s, f held fixed: g_j = up (alpha n f^G_j / T + alpha_seq n f^s_j / (S' T_s)).
// For softmax, p_j (g_j - sum_i p_i g_i) does not change when a constant is taken from every g, so
// f - 1/n = (count n - k T) / (k T n) stands for f (an exact whole number over a constant): near balance the
// difference keeps its digits. A lane group takes consecutive rows, two in flight.
template <int L, int V>
__global__ void __launch_bounds__(rloss::kThreads)
router_loss_grad_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx, int64_t m, int n, int k,
                        const int32_t* __restrict__ off, int nseq, const uint8_t* __restrict__ mask, int fn,
                        double alpha, double alpha_seq, double z_coef, const int32_t* __restrict__ counts,
                        const int32_t* __restrict__ tokens, const float* __restrict__ dloss,
                        const float* __restrict__ dgate, int renorm, float* __restrict__ dlogits) {
    using namespace rloss;
    constexpr int RW = 32 / L, GROUPS = (kThreads / 32) * RW, U = 2;
    constexpr int CW = 4 * V * L;
    extern __shared__ float scat[];  // [GROUPS][CW]: a row's logits for its picks, then what the gates add to each column
    __shared__ int s_full;
    const int tid = threadIdx.x, lane = tid & 31, sub = lane % L, grp = (tid >> 5) * RW + lane / L;
    const bool vec = (n & 3) == 0;
    pdl_trigger();
    pdl_wait();
    if (alpha_seq != 0.0) {
        if (tid == 0) s_full = 0;
        __syncthreads();
        int full = 0;
        for (int q = tid; q < nseq; q += kThreads) full += tokens[q] > 0;
        if (full) atomicAdd(&s_full, full);
        __syncthreads();
    }
    float* mine = scat + grp * CW;
    if (dgate)
        for (int j = sub; j < CW; j += L) mine[j] = 0.f;
    __syncwarp();
    const double up = dloss ? (double)*dloss : 1.0;
    const int T = max(tokens[nseq], 1);
    const bool soft = fn == MOE_SOFTMAX;
    const float cz = (float)(2.0 * z_coef * up / T);
    const bool chosen = soft && renorm && k > 1;  // gate = softmax over the picks
    const double full = alpha_seq != 0.0 ? (double)max(s_full, 1) : 1.0;
    // a table row's part of g for the owned columns: coef / T * (count n - k T) / (k T), or coef / T * count n / (k T)
    auto table = [&](const int32_t* row, int64_t t, double coef, float (&g)[4 * V]) {
        const float scale = (float)(coef / ((double)t * (double)t * (double)k));
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int j = 4 * (sub + L * v) + q;
                g[4 * v + q] = j < n ? scale * (float)((int64_t)row[j] * n - (soft ? (int64_t)k * t : 0)) : 0.f;
            }
    };
    float gG[4 * V], gt[4 * V];  // the whole batch's part; with the row's sequence
    table(counts + (int64_t)nseq * n, T, up * alpha, gG);
#pragma unroll
    for (int q = 0; q < 4 * V; ++q) gt[q] = gG[q];
    const int64_t groups = (int64_t)gridDim.x * GROUPS, per = (m + groups - 1) / groups;
    const int64_t r0 = ((int64_t)blockIdx.x * GROUPS + grp) * per, r1 = min(r0 + per, m);
    int seq = -2;
    int64_t seq_end = -1;  // the rows below it that follow the current one belong to `seq`
    // every lane of a warp runs the same number of rounds: the row's lanes reduce together
    for (int64_t i = 0; i < per; i += U) {
        float h[U][4 * V], dg[U];
        int pick[U];
        bool live[U];
        bool ok[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + i + u;
            ok[u] = i + u < per && r < r1 && (!mask || mask[r]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + i + u;
#pragma unroll
            for (int q = 0; q < 4 * V; ++q) h[u][q] = -INFINITY;
            if (ok[u]) load_row<L, V>(logits + r * n, n, vec, sub, h[u]);
            const bool has = ok[u] && dgate && sub < k;
            pick[u] = has ? idx[r * k + sub] : -1;
            dg[u] = has ? dgate[r * k + sub] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + i + u;
            const bool in = i + u < per && r < r1;
            if (in && r >= seq_end) {
                seq = seq_of_row(off, nseq, r);
                seq_end = seq >= nseq ? m : (int64_t)off[seq + 1];
                if (alpha_seq != 0.0 && seq >= 0 && seq < nseq) {
                    table(counts + (int64_t)seq * n, max(tokens[seq], 1), up * alpha_seq / full, gt);
#pragma unroll
                    for (int q = 0; q < 4 * V; ++q) gt[q] += gG[q];
                }
            }
            live[u] = ok[u] && seq >= 0 && seq < nseq;
            float add[4 * V];
#pragma unroll
            for (int q = 0; q < 4 * V; ++q) add[q] = 0.f;
            if (dgate) {
                if (chosen) {
                    // q_r = softmax over the picks' logits; dL/dh = q_r (dg_r - sum q dg)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        *reinterpret_cast<float4*>(mine + 4 * (sub + L * v)) =
                            make_float4(h[u][4 * v], h[u][4 * v + 1], h[u][4 * v + 2], h[u][4 * v + 3]);
                    __syncwarp();
                    const int e0 = live[u] && pick[u] >= 0 && pick[u] < n ? pick[u] : -1;
                    const float x0 = e0 >= 0 ? mine[e0] : -INFINITY;
                    float top = x0;
                    for (int t = sub + L; t < k; t += L) {
                        const int e = live[u] ? idx[r * k + t] : -1;
                        if (e >= 0 && e < n) top = fmaxf(top, mine[e]);
                    }
                    top = lanes_max<L>(top);
                    if (top == -INFINITY) top = 0.f;  // no pick has a score: every weight is 0
                    const float w0 = expf(x0 - top);
                    float sum = w0, dot = w0 * dg[u];
                    for (int t = sub + L; t < k; t += L) {
                        const int e = live[u] ? idx[r * k + t] : -1;
                        if (e >= 0 && e < n) {
                            const float x = expf(mine[e] - top);
                            sum += x;
                            dot = fmaf(x, dgate[r * k + t], dot);
                        }
                    }
                    sum = lanes_sum<L>(sum);
                    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
                    dot = lanes_sum<L>(dot) * inv;
                    // further picks (k > L): their terms wait in registers of the second pass over the row's logits
                    float keep[4 * V];
#pragma unroll
                    for (int q = 0; q < 4 * V; ++q) keep[q] = 0.f;
                    if (k > L) {
                        // column j's term, from the picks that name it: each lane looks at every pick
                        for (int t = 0; t < k; ++t) {
                            const int e = live[u] ? idx[r * k + t] : -1;
#pragma unroll
                            for (int v = 0; v < V; ++v)
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    if (e == 4 * (sub + L * v) + q && e < n)
                                        keep[4 * v + q] += expf(h[u][4 * v + q] - top) * inv * (dgate[r * k + t] - dot);
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        *reinterpret_cast<float4*>(mine + 4 * (sub + L * v)) = make_float4(keep[4 * v], keep[4 * v + 1], keep[4 * v + 2], keep[4 * v + 3]);
                    __syncwarp();
                    if (k <= L && e0 >= 0) atomicAdd(&mine[e0], w0 * inv * (dg[u] - dot));
                } else {
                    if (live[u] && pick[u] >= 0 && pick[u] < n) atomicAdd(&mine[pick[u]], dg[u]);
                    for (int t = sub + L; t < k; t += L) {
                        const int e = live[u] ? idx[r * k + t] : -1;
                        if (e >= 0 && e < n) atomicAdd(&mine[e], dgate[r * k + t]);
                    }
                }
                __syncwarp();
                // read the row's columns and clear them for the next row
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float4* at = reinterpret_cast<float4*>(mine + 4 * (sub + L * v));
                    const float4 t = *at;
                    *at = make_float4(0.f, 0.f, 0.f, 0.f);
                    add[4 * v] = t.x; add[4 * v + 1] = t.y; add[4 * v + 2] = t.z; add[4 * v + 3] = t.w;
                }
                __syncwarp();
            }
            float out[4 * V];
            if (soft) {
                const float lse = row_softmax<L, V>(h[u]);  // h is the score now
                float c = 0.f;
                float g[4 * V];
#pragma unroll
                for (int q = 0; q < 4 * V; ++q) {
                    g[q] = gt[q] + (chosen ? 0.f : add[q]);
                    c = fmaf(h[u][q], g[q], c);
                }
                c = lanes_sum<L>(c);
#pragma unroll
                for (int q = 0; q < 4 * V; ++q) out[q] = fmaf(h[u][q], g[q] - c + cz * lse, chosen ? add[q] : 0.f);
            } else {
#pragma unroll
                for (int q = 0; q < 4 * V; ++q)  // 1 - rho from its own exponential: exact for large h
                    out[q] = (gt[q] + add[q]) * logistic(h[u][q]) * logistic(-h[u][q]);
                if (cz != 0.f) {
                    const float lse = row_softmax<L, V>(h[u]);
#pragma unroll
                    for (int q = 0; q < 4 * V; ++q) out[q] = fmaf(cz * lse, h[u][q], out[q]);
                }
            }
            if (in) {
                float* row = dlogits + r * n;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int j = 4 * (sub + L * v);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (!live[u]) out[4 * v + q] = 0.f;
                    if (vec) {
                        if (j < n)
                            *reinterpret_cast<float4*>(row + j) =
                                make_float4(out[4 * v], out[4 * v + 1], out[4 * v + 2], out[4 * v + 3]);
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (j + q < n) row[j + q] = out[4 * v + q];
                    }
                }
            }
        }
    }
}

// Lanes per row L and 16-byte loads per lane V that hold n logits.
#define MOE_ROUTER_LOSS_DISPATCH(n, CALL)  \
    do {                                   \
        if ((n) <= 8) { CALL(2, 1); }      \
        else if ((n) <= 16) { CALL(4, 1); }  \
        else if ((n) <= 32) { CALL(8, 1); }  \
        else if ((n) <= 64) { CALL(16, 1); } \
        else if ((n) <= 128) { CALL(32, 1); } \
        else { CALL(32, 2); }              \
    } while (0)

cudaError_t launch_router_loss(const float* logits, const int32_t* idx, int64_t m, int n, int k, const int32_t* off,
                               int nseq, const uint8_t* mask, int fn, float alpha, float alpha_seq, float z_coef,
                               float* loss, int32_t* counts, int32_t* tokens, float* f, float* P, void* workspace,
                               cudaStream_t stream) {
    RouterLossWs w;
    router_loss_layout(m, n, nseq, &w, static_cast<char*>(workspace));
    const int64_t nch = (m + rloss::kRows - 1) / rloss::kRows;
    if (nch > 0) {
        cudaError_t e = cudaSuccess;
#define CALL(L, V)                                                                                                  \
    e = launch_pdl(router_loss_chunk_kernel<L, V>, dim3((unsigned)nch), dim3(rloss::kThreads),                      \
                   sizeof(double) * (rloss::kThreads / 32) * (32 / L) * (4 * V * L + 1), stream, logits, idx, m, n, \
                   k, off, nseq, mask, fn, z_coef != 0.f ? 1 : 0, w)
        MOE_ROUTER_LOSS_DISPATCH(n, CALL);
#undef CALL
        if (e != cudaSuccess) return e;
    } else {
        const cudaError_t e = cudaMemsetAsync(w.ticket, 0, sizeof(int32_t), stream);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(router_loss_fold_kernel, dim3((unsigned)nseq + 1, (unsigned)((n + rloss::kFoldCols - 1) / rloss::kFoldCols)),
                      dim3(rloss::kThreads), 0, stream, m, n, k, off, nseq, (double)alpha, (double)alpha_seq,
                      (double)z_coef, loss, counts, tokens, f, P, w);
}

cudaError_t launch_router_loss_grad(const float* logits, const int32_t* idx, int64_t m, int n, int k,
                                    const int32_t* off, int nseq, const uint8_t* mask, int fn, float alpha,
                                    float alpha_seq, float z_coef, const int32_t* counts, const int32_t* tokens,
                                    const float* dloss, const float* dgate, int renorm, float* dlogits,
                                    cudaStream_t stream) {
    if (m == 0) return cudaSuccess;
    cudaError_t e = cudaSuccess;
#define CALL(L, V)                                                                                                   \
    do {                                                                                                             \
        constexpr int G = (rloss::kThreads / 32) * (32 / L);                                                         \
        int64_t blocks = (m + G - 1) / G;                                                                            \
        if (blocks > (int64_t)kNumSMs * 6) blocks = (int64_t)kNumSMs * 6;                                            \
        e = launch_pdl(router_loss_grad_kernel<L, V>, dim3((unsigned)blocks), dim3(rloss::kThreads),                 \
                       sizeof(float) * G * 4 * V * L, stream, logits, idx, m, n, k, off, nseq, mask, fn, (double)alpha, \
                       (double)alpha_seq, (double)z_coef, counts, tokens, dloss, dgate, renorm, dlogits);            \
    } while (0)
    MOE_ROUTER_LOSS_DISPATCH(n, CALL);
#undef CALL
    return e;
}

}  // namespace moe
