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
// Reading the logits (and writing the gradient) is 4 m n bytes each; both passes wait for instruction issue before
// that (65536 x 256, k 8: 36 and 53 us). The exponentials are expf, as the router's are: __expf is off by 1.2 |x| ulp,
// which is many in the scores of experts far below a row's best, and with scores added in fp32 by twos and fours
// before the fp64 sums it saved 3 and 4 of these microseconds.
#include "common.cuh"

namespace moe {

namespace rloss {
constexpr int kRows = 128;     // rows per CTA of the chunk pass
constexpr int kThreads = 256;
constexpr int kFoldCols = 32;  // experts per CTA of the fold
constexpr int kFoldThreads = 512;
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

// The same by the whole block, in one read where the offsets are few (a binary search is a chain of reads).
__device__ __forceinline__ int seq_of_row_block(const int32_t* __restrict__ off, int nseq, int64_t r) {
    if (nseq >= rloss::kThreads) return seq_of_row(off, nseq, r);
    const int tid = threadIdx.x;
    return __syncthreads_count(tid <= nseq && (int64_t)off[min(tid, nseq)] <= r) - 1;
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
    if (top == -INFINITY) top = 0.f;
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < 4 * V; ++q) { h[q] = expf(h[q] - top); s += h[q]; }
    s = lanes_sum<L>(s);
    const float inv = s == 0.f ? 0.f : 1.f / (s == 0.f ? 1.f : s);
#pragma unroll
    for (int q = 0; q < 4 * V; ++q) h[q] *= inv;
    return s == 0.f ? 0.f : top + logf(s);
}

// By t = exp(-|h|), so that what is inverted lies in [1, 2]: the quotient of an infinity (the columns behind n) is slow.
__device__ __forceinline__ float logistic(float h) {
    const float t = expf(-fabsf(h)), w = 1.f / (1.f + t);
    return h >= 0.f ? w : t * w;
}

template <int L, int V>
__global__ void __launch_bounds__(rloss::kThreads, 4)
router_loss_chunk_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx, int64_t m, int n, int k,
                         const int32_t* __restrict__ off, int nseq, const uint8_t* __restrict__ mask, int fn,
                         int want_z, RouterLossWs w) {
    using namespace rloss;
    constexpr int RW = 32 / L;                      // rows a warp holds
    constexpr int GROUPS = (kThreads / 32) * RW;    // rows the CTA holds at a time
    constexpr int U = GROUPS >= 64 ? 1 : V == 2 ? 2 : 4;  // rows in flight per lane group
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
        const int s = seq_of_row_block(off, nseq, at);
        if (s >= nseq) break;                                        // behind the last sequence
        // off[s + 1] is the first offset above `at`; offsets that do not ascend (an error) may not be: step on all the same
        const int64_t next = max(at + 1, min((int64_t)off[s + 1], r1));
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
                if (!__any_sync(0xffffffffu, live[u])) {  // short sequences leave most of a round's rows empty
#pragma unroll
                    for (int q = 0; q < 4 * V; ++q) h[u][q] = 0.f;
                    continue;
                }
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
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int q = 0; q < 4 * V; ++q) acc[q] += (double)h[u][q];
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
    if (tid < 32) {
        double t = 0.0;
        for (int g = tid; g < GROUPS; g += 32) t += zpart[g];
        t = warp_sum_d(t);
        if (tid == 0) { w.zsum[c] = t; w.ttok[c] = total; }
    }
}

// blockIdx.x = sequence (nseq: the whole batch), blockIdx.y = 32 experts; a warp takes every 16th chunk.
__global__ void __launch_bounds__(rloss::kFoldThreads)
router_loss_fold_kernel(int64_t m, int n, int k, const int32_t* __restrict__ off, int nseq, double alpha,
                        double alpha_seq, double z_coef, float* __restrict__ loss, int32_t* __restrict__ counts,
                        int32_t* __restrict__ tokens, float* __restrict__ f, float* __restrict__ P, RouterLossWs w) {
    using namespace rloss;
    constexpr int W = kFoldThreads / 32;
    __shared__ double ps[W][kFoldCols];
    __shared__ int cs[W][kFoldCols];
    __shared__ int ts[W];
    __shared__ double red[W], redz[W];
    __shared__ int redi[W];
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
    const int ec = min(e, n - 1);
#pragma unroll 8
    for (int64_t c = c0 + wid; c < c1; c += W) {
        a += psum[c * n + ec];
        cn += pcnt[c * n + ec];
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
    // the last CTA: the sequences' losses in order (thread t takes sequences t, t + 512, ...)
    const int ncb = gridDim.y;
    double seq = 0.0;
    int full = 0;
    for (int q = tid; q < nseq; q += kFoldThreads) {
        for (int b = 0; b < ncb; ++b) seq += __ldcg(w.part + (int64_t)q * ncb + b);
        full += __ldcg(tokens + q) > 0;
    }
    double z = 0.0;
    for (int64_t c = tid; c < nch; c += kFoldThreads) z += __ldcg(w.zsum + c);
    seq = warp_sum_d(seq);
    z = warp_sum_d(z);
    full = __reduce_add_sync(0xffffffffu, full);
    if (lane == 0) { red[wid] = seq; redz[wid] = z; redi[wid] = full; }
    __syncthreads();
    if (tid == 0) {
        for (int q = 1; q < W; ++q) { seq += red[q]; z += redz[q]; full += redi[q]; }
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
    extern __shared__ float bufs[];  // [GROUPS][U][2][CW]: a row's logits for its picks; what the gates add to each column
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
    float* mine = bufs + grp * U * 2 * CW;
    if (dgate)
        for (int j = sub; j < U * 2 * CW; j += L) mine[j] = 0.f;
    __syncwarp();
    const double up = dloss ? (double)*dloss : 1.0;
    const int T = max(tokens[nseq], 1);
    const bool soft = fn == MOE_SOFTMAX;
    const float cz = (float)(2.0 * z_coef * up / T);
    const bool chosen = soft && renorm && k > 1 && dgate;  // gate = softmax over the picks
    const double full = alpha_seq != 0.0 ? (double)max(s_full, 1) : 1.0;
    // g for the owned columns, rounded once: a table row's part is coef / T * (count n - k T) / (k T), without the k T
    // above for a logistic; the whole batch's row and (s < nseq) sequence s's
    float gt[4 * V];
    auto table = [&](int s) {
        const int t = s < nseq ? max(tokens[s], 1) : 1;
        const double cG = up * alpha / ((double)T * T * k), cs = s < nseq ? up * alpha_seq / (full * t * t * k) : 0.0;
        const double zG = soft ? (double)k * T : 0.0, zs = soft ? (double)k * t : 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int j = 4 * (sub + L * v) + q;
                double g = 0.0;
                if (j < n) g = cG * ((double)counts[(int64_t)nseq * n + j] * n - zG);
                if (j < n && s < nseq) g += cs * ((double)counts[(int64_t)s * n + j] * n - zs);
                gt[4 * v + q] = (float)g;
            }
    };
    table(nseq);
    const int64_t groups = (int64_t)gridDim.x * GROUPS, per = (m + groups - 1) / groups;
    const int64_t r0 = ((int64_t)blockIdx.x * GROUPS + grp) * per, r1 = min(r0 + per, m);
    int seq = -2;
    int64_t seq_end = -1;  // the rows below it that follow the current one belong to `seq`
    // every lane of a warp runs the same number of rounds (the row's lanes reduce together), and the rows of a round
    // go through each step together, so that one's shuffles hide the other's
    for (int64_t i = 0; i < per; i += U) {
        float h[U][4 * V], g[U][4 * V], dg[U], x0[U];
        int pick[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + i + u;
            live[u] = i + u < per && r < r1 && (!mask || mask[r]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + i + u;
#pragma unroll
            for (int q = 0; q < 4 * V; ++q) h[u][q] = -INFINITY;
            if (live[u]) load_row<L, V>(logits + r * n, n, vec, sub, h[u]);
            const bool has = live[u] && dgate && sub < k;
            pick[u] = has ? idx[r * k + sub] : -1;
            dg[u] = has ? dgate[r * k + sub] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + i + u;
            if (i + u < per && r < r1 && r >= seq_end) {
                seq = seq_of_row(off, nseq, r);
                seq_end = seq >= nseq ? m : (int64_t)off[seq + 1];
                if (alpha_seq != 0.0 && seq >= 0 && seq < nseq) table(seq);
            }
            live[u] = live[u] && seq >= 0 && seq < nseq;
            if (!live[u] || pick[u] < 0 || pick[u] >= n) pick[u] = -1;
#pragma unroll
            for (int q = 0; q < 4 * V; ++q) g[u][q] = gt[q];
        }
        // the picks: their logits, or what their gates add to g
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float* logit = mine + u * 2 * CW;
            float* add = logit + CW;
            if (chosen) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    *reinterpret_cast<float4*>(logit + 4 * (sub + L * v)) = make_float4(h[u][4 * v], h[u][4 * v + 1], h[u][4 * v + 2], h[u][4 * v + 3]);
            } else if (dgate) {
                if (pick[u] >= 0) atomicAdd(&add[pick[u]], dg[u]);
                for (int t = sub + L; t < k; t += L) {
                    const int e = live[u] ? idx[(r0 + i + u) * k + t] : -1;
                    if (e >= 0 && e < n) atomicAdd(&add[e], dgate[(r0 + i + u) * k + t]);
                }
            }
        }
        __syncwarp();
        float top[U], ptop[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float* logit = mine + u * 2 * CW;
            float* add = mine + u * 2 * CW + CW;
            x0[u] = -INFINITY;
            if (chosen) {
                if (pick[u] >= 0) x0[u] = logit[pick[u]];
            } else if (dgate) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float4* at = reinterpret_cast<float4*>(add + 4 * (sub + L * v));
                    const float4 t = *at;
                    *at = make_float4(0.f, 0.f, 0.f, 0.f);
                    g[u][4 * v] += t.x; g[u][4 * v + 1] += t.y; g[u][4 * v + 2] += t.z; g[u][4 * v + 3] += t.w;
                }
            }
            ptop[u] = x0[u];
            if (chosen)
                for (int t = sub + L; t < k; t += L) {
                    const int e = live[u] ? idx[(r0 + i + u) * k + t] : -1;
                    if (e >= 0 && e < n) ptop[u] = fmaxf(ptop[u], logit[e]);
                }
            top[u] = h[u][0];
#pragma unroll
            for (int q = 1; q < 4 * V; ++q) top[u] = fmaxf(top[u], h[u][q]);
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
                if (chosen) ptop[u] = fmaxf(ptop[u], __shfl_xor_sync(0xffffffffu, ptop[u], o));
            }
        float s[U], eg[U], sq[U], dq[U], w0[U];
        float e[U][4 * V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[u] = eg[u] = 0.f;
            if (top[u] == -INFINITY) top[u] = 0.f;  // a row without scores
            if (soft || cz != 0.f) {
#pragma unroll
                for (int q = 0; q < 4 * V; ++q) {
                    e[u][q] = expf(h[u][q] - top[u]);
                    s[u] += e[u][q];
                    eg[u] = fmaf(e[u][q], g[u][q], eg[u]);
                }
            }
            if (ptop[u] == -INFINITY) ptop[u] = 0.f;  // no pick has a score: every weight is 0
            w0[u] = chosen ? expf(x0[u] - ptop[u]) : 0.f;
            sq[u] = w0[u];
            dq[u] = w0[u] * dg[u];
            if (chosen)
                for (int t = sub + L; t < k; t += L) {
                    const int p = live[u] ? idx[(r0 + i + u) * k + t] : -1;
                    if (p >= 0 && p < n) {
                        const float x = expf(mine[u * 2 * CW + p] - ptop[u]);
                        sq[u] += x;
                        dq[u] = fmaf(x, dgate[(r0 + i + u) * k + t], dq[u]);
                    }
                }
        }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
                if (soft) eg[u] += __shfl_xor_sync(0xffffffffu, eg[u], o);
                if (chosen) {
                    sq[u] += __shfl_xor_sync(0xffffffffu, sq[u], o);
                    dq[u] += __shfl_xor_sync(0xffffffffu, dq[u], o);
                }
            }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float inv = s[u] == 0.f ? 0.f : 1.f / (s[u] == 0.f ? 1.f : s[u]);
            const float lse = s[u] == 0.f ? 0.f : top[u] + logf(s[u]);
            if (soft) {
                const float c = eg[u] * inv - cz * lse;
#pragma unroll
                for (int q = 0; q < 4 * V; ++q) e[u][q] *= inv * (g[u][q] - c);
            } else {
#pragma unroll
                for (int q = 0; q < 4 * V; ++q) {  // rho (1 - rho) = t / (1 + t)^2, t = exp(-|h|): exact for large h
                    const float z = cz != 0.f ? cz * lse * inv * e[u][q] : 0.f;
                    const float t = expf(-fabsf(h[u][q])), s1 = 1.f + t, lost = t - (s1 - 1.f);  // 1 + t = s1 + lost
                    e[u][q] = fmaf(g[u][q], t * __frcp_rn(fmaf(s1, s1, 2.f * s1 * lost)), z);
                }
            }
            if (chosen) {  // dL/dh of a pick: q_r (dg_r - sum q dg)
                const float iq = sq[u] != 0.f ? 1.f / sq[u] : 0.f, dot = dq[u] * iq;
                float* add = mine + u * 2 * CW + CW;
                if (pick[u] >= 0) atomicAdd(&add[pick[u]], w0[u] * iq * (dg[u] - dot));
                for (int t = sub + L; t < k; t += L) {
                    const int p = live[u] ? idx[(r0 + i + u) * k + t] : -1;
                    if (p >= 0 && p < n)
                        atomicAdd(&add[p], expf(mine[u * 2 * CW + p] - ptop[u]) * iq * (dgate[(r0 + i + u) * k + t] - dot));
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = r0 + i + u;
            const bool in = i + u < per && r < r1;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int j = 4 * (sub + L * v);
                float4 o = make_float4(e[u][4 * v], e[u][4 * v + 1], e[u][4 * v + 2], e[u][4 * v + 3]);
                if (chosen) {
                    float4* at = reinterpret_cast<float4*>(mine + u * 2 * CW + CW + j);
                    const float4 t = *at;
                    *at = make_float4(0.f, 0.f, 0.f, 0.f);
                    o.x += t.x; o.y += t.y; o.z += t.z; o.w += t.w;
                }
                if (!live[u]) o = make_float4(0.f, 0.f, 0.f, 0.f);
                if (!in) continue;
                float* row = dlogits + r * n + j;
                if (vec) {
                    if (j < n) *reinterpret_cast<float4*>(row) = o;
                } else {
                    if (j < n) row[0] = o.x;
                    if (j + 1 < n) row[1] = o.y;
                    if (j + 2 < n) row[2] = o.z;
                    if (j + 3 < n) row[3] = o.w;
                }
            }
        }
        __syncwarp();
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
                      dim3(rloss::kFoldThreads), 0, stream, m, n, k, off, nseq, (double)alpha, (double)alpha_seq,
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
        constexpr int G = (rloss::kThreads / 32) * (32 / L), most = kNumSMs * (V == 2 ? 2 : 4);                      \
        int64_t blocks = (m + G - 1) / G;                                                                            \
        if (blocks > most) blocks = most;  /* one wave */                                                            \
        e = launch_pdl(router_loss_grad_kernel<L, V>, dim3((unsigned)blocks), dim3(rloss::kThreads),                 \
                       sizeof(float) * G * 2 * 2 * 4 * V * L, stream, logits, idx, m, n, k, off, nseq, mask, fn, (double)alpha, \
                       (double)alpha_seq, (double)z_coef, counts, tokens, dloss, dgate, renorm, dlogits);            \
    } while (0)
    MOE_ROUTER_LOSS_DISPATCH(n, CALL);
#undef CALL
    return e;
}

}  // namespace moe
