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

// e_j = exp(h_j - top) / sum and the log-sum-exp of a row held by L lanes. A row whose logits are
// all -inf has no scores: e = 0 and lse = 0. NaN and +inf give NaN.
template <int L, int V>
__device__ __forceinline__ void row_softmax(const float (&h)[4 * V], float (&e)[4 * V], float& lse) {
    float top = h[0];
#pragma unroll
    for (int q = 1; q < 4 * V; ++q) top = fmaxf(top, h[q]);
    top = lanes_max<L>(top);
    float s = 0.f;
    if (top == -INFINITY) {  // fmaxf passes over NaN: keep it in the sum
#pragma unroll
        for (int q = 0; q < 4 * V; ++q) { e[q] = h[q] == -INFINITY ? 0.f : h[q]; s += e[q]; }
        s = lanes_sum<L>(s);
        lse = s;
        return;
    }
#pragma unroll
    for (int q = 0; q < 4 * V; ++q) { e[q] = expf(h[q] - top); s += e[q]; }
    s = lanes_sum<L>(s);
    const float inv = 1.f / s;
#pragma unroll
    for (int q = 0; q < 4 * V; ++q) e[q] *= inv;
    lse = top + logf(s);
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
    extern __shared__ double fold[];                // [GROUPS][4 V L + 1] a row group's sums
    __shared__ int cnt[kMaxExperts];
    __shared__ double zpart[GROUPS];
    __shared__ int ntok;
    const int tid = threadIdx.x, lane = tid & 31, sub = lane % L, grp = (tid >> 5) * RW + lane / L;
    constexpr int FS = 4 * V * L + 1;
    const bool vec = (n & 3) == 0;
    pdl_trigger();
    pdl_wait();
    const int64_t c = blockIdx.x, r0 = c * kRows, r1 = min(r0 + (int64_t)kRows, m);
    if (c == 0 && tid == 0) *w.ticket = 0;
    for (int e = tid; e < n; e += kThreads) { w.tsum[c * n + e] = 0.0; w.tcnt[c * n + e] = 0; }
    double z = 0.0;
    int total = 0;
    for (int64_t at = r0; at < r1;) {
        const int s = seq_of_row(off, nseq, at);
        if (s >= nseq) break;                                        // behind the last sequence
        const int64_t next = min((int64_t)off[s + 1], r1);           // > at: off[s + 1] is the first offset above it
        if (s < 0) { at = next; continue; }                          // before the first
        for (int e = tid; e < n; e += kThreads) cnt[e] = 0;
        if (tid == 0) ntok = 0;
        __syncthreads();
        double acc[4 * V];
#pragma unroll
        for (int q = 0; q < 4 * V; ++q) acc[q] = 0.0;
        // every lane of a warp runs the same number of rounds: the row's lanes reduce together
        for (int64_t base = at; base < next; base += GROUPS) {
            const int64_t r = base + grp;
            const bool live = r < next && (!mask || mask[r]);
            float h[4 * V], p[4 * V];
#pragma unroll
            for (int q = 0; q < 4 * V; ++q) h[q] = -INFINITY;
            if (live) load_row<L, V>(logits + r * n, n, vec, sub, h);
            float lse = 0.f;
            if (fn == MOE_SOFTMAX || want_z) row_softmax<L, V>(h, p, lse);
            if (fn == MOE_SIGMOID) {
#pragma unroll
                for (int q = 0; q < 4 * V; ++q) p[q] = logistic(h[q]);
            }
            if (live) {
#pragma unroll
                for (int q = 0; q < 4 * V; ++q) acc[q] += (double)p[q];
                if (sub == 0) { z += (double)lse * (double)lse; atomicAdd(&ntok, 1); }
                for (int t = sub; t < k; t += L) {
                    const int e = idx[r * k + t];
                    if (e < 0 || e >= n) record_error(kErrExpertIndex);
                    else atomicAdd(&cnt[e], 1);
                }
            }
        }
        // column 4 (sub + L v) + q of row group g sits at fold[g][4 (sub + L v) + q]
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int q = 0; q < 4; ++q) fold[grp * FS + 4 * (sub + L * v) + q] = acc[4 * v + q];
        __syncthreads();
        const int64_t slot = c + s;
        for (int e = tid; e < n; e += kThreads) {
            double t = 0.0;
            for (int g = 0; g < GROUPS; ++g) t += fold[g * FS + e];
            w.psum[slot * n + e] = t;
            w.pcnt[slot * n + e] = cnt[e];
            w.tsum[c * n + e] += t;
            w.tcnt[c * n + e] += cnt[e];
        }
        if (tid == 0) { w.ptok[slot] = ntok; total += ntok; }
        __syncthreads();
        at = next;
    }
    if (sub == 0) zpart[grp] = z;
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
// f - 1/n stands for f: near balance the difference keeps its digits.
template <int L, int V>
__global__ void __launch_bounds__(rloss::kThreads)
router_loss_grad_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx, int64_t m, int n, int k,
                        const int32_t* __restrict__ off, int nseq, const uint8_t* __restrict__ mask, int fn,
                        double alpha, double alpha_seq, double z_coef, const int32_t* __restrict__ counts,
                        const int32_t* __restrict__ tokens, const float* __restrict__ dloss,
                        const float* __restrict__ dgate, int renorm, float* __restrict__ dlogits) {
    using namespace rloss;
    constexpr int RW = 32 / L, GROUPS = (kThreads / 32) * RW;
    extern __shared__ float scat[];  // [GROUPS][4 V L]: what the gates add to each column of the row
    __shared__ int s_full;
    const int tid = threadIdx.x, lane = tid & 31, sub = lane % L, grp = (tid >> 5) * RW + lane / L;
    constexpr int CW = 4 * V * L;
    const bool vec = (n & 3) == 0;
    pdl_trigger();
    pdl_wait();
    if (tid == 0) s_full = 0;
    __syncthreads();
    if (alpha_seq != 0.0) {
        int full = 0;
        for (int q = tid; q < nseq; q += kThreads) full += tokens[q] > 0;
        if (full) atomicAdd(&s_full, full);
    }
    float* mine = scat + grp * CW;
    if (dgate)
        for (int j = sub; j < CW; j += L) mine[j] = 0.f;
    __syncthreads();
    const double up = dloss ? (double)*dloss : 1.0;
    const double T = (double)max(tokens[nseq], 1);
    const double shift = fn == MOE_SOFTMAX ? 1.0 / (double)n : 0.0;
    const float cz = (float)(2.0 * z_coef * up / T);
    const bool chosen = fn == MOE_SOFTMAX && renorm && k > 1;  // gate = softmax over the picks
    // g's constants: the whole batch's part of each owned column
    float gG[4 * V], gs[4 * V];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int j = 4 * (sub + L * v) + q;
            gG[4 * v + q] = 0.f;
            gs[4 * v + q] = 0.f;
            if (j < n)
                gG[4 * v + q] = (float)(up * alpha * n / T * ((double)counts[(int64_t)nseq * n + j] / (k * T) - shift));
        }
    const int64_t per = (m + gridDim.x - 1) / gridDim.x;  // rows of this CTA, consecutive
    const int64_t r0 = blockIdx.x * per, r1 = min(r0 + per, m);
    int seq = -2;
    int64_t seq_end = -1;  // the rows below it that follow the current one belong to `seq`
    for (int64_t base = r0; base < r1; base += GROUPS) {
        const int64_t r = base + grp;
        const bool in = r < r1;
        if (in && r >= seq_end) {
            seq = seq_of_row(off, nseq, r);
            seq_end = seq >= nseq ? m : (int64_t)off[seq + 1];
            if (alpha_seq != 0.0 && seq >= 0 && seq < nseq) {
                const double Ts = (double)max(tokens[seq], 1);
                const double cs = up * alpha_seq * n / ((double)max(s_full, 1) * Ts);
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int j = 4 * (sub + L * v) + q;
                        if (j < n) gs[4 * v + q] = (float)(cs * ((double)counts[(int64_t)seq * n + j] / (k * Ts) - shift));
                    }
            }
        }
        const bool live = in && seq >= 0 && seq < nseq && (!mask || mask[r]);
        float h[4 * V], p[4 * V], soft[4 * V], out[4 * V];
#pragma unroll
        for (int q = 0; q < 4 * V; ++q) h[q] = -INFINITY;
        if (live) load_row<L, V>(logits + r * n, n, vec, sub, h);
        float lse = 0.f;
        if (fn == MOE_SOFTMAX || cz != 0.f) row_softmax<L, V>(h, soft, lse);
        float g[4 * V];
#pragma unroll
        for (int q = 0; q < 4 * V; ++q) g[q] = gG[q] + gs[q];
        if (dgate) {
            if (chosen) {
                // q_r = softmax over the picks' logits; dL/dh = q_r (dg_r - sum q dg)
                float top = -INFINITY, sum = 0.f, dot = 0.f;
                for (int t = sub; t < k; t += L) {
                    const int e = live ? idx[r * k + t] : -1;
                    if (e >= 0 && e < n) top = fmaxf(top, logits[r * n + e]);
                }
                top = lanes_max<L>(top);
                for (int t = sub; t < k; t += L) {
                    const int e = live ? idx[r * k + t] : -1;
                    if (e >= 0 && e < n && top != -INFINITY) {
                        const float x = expf(logits[r * n + e] - top);
                        sum += x;
                        dot = fmaf(x, dgate[r * k + t], dot);
                    }
                }
                sum = lanes_sum<L>(sum);
                dot = lanes_sum<L>(dot) / sum;
                for (int t = sub; t < k; t += L) {
                    const int e = live ? idx[r * k + t] : -1;
                    if (e >= 0 && e < n && top != -INFINITY)
                        atomicAdd(&mine[e], expf(logits[r * n + e] - top) / sum * (dgate[r * k + t] - dot));
                }
            } else {
                for (int t = sub; t < k; t += L) {
                    const int e = live ? idx[r * k + t] : -1;
                    if (e >= 0 && e < n) atomicAdd(&mine[e], dgate[r * k + t]);
                }
            }
            __syncwarp();
            // read the row's columns and clear them for the next row
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int j = 4 * (sub + L * v) + q;
                    out[4 * v + q] = mine[j];
                    mine[j] = 0.f;
                }
            __syncwarp();
        } else {
#pragma unroll
            for (int q = 0; q < 4 * V; ++q) out[q] = 0.f;
        }
        if (!chosen) {
#pragma unroll
            for (int q = 0; q < 4 * V; ++q) { g[q] += out[q]; out[q] = 0.f; }
        }
        if (fn == MOE_SOFTMAX) {
            float c = 0.f;
#pragma unroll
            for (int q = 0; q < 4 * V; ++q) c = fmaf(soft[q], g[q], c);
            c = lanes_sum<L>(c);
#pragma unroll
            for (int q = 0; q < 4 * V; ++q) out[q] = fmaf(soft[q], g[q] - c, out[q]);
        } else {
#pragma unroll
            for (int q = 0; q < 4 * V; ++q) {
                p[q] = logistic(h[q]);
                out[q] = g[q] * p[q] * logistic(-h[q]);  // 1 - rho from its own exponential: exact for large h
            }
        }
        if (cz != 0.f) {
#pragma unroll
            for (int q = 0; q < 4 * V; ++q) out[q] = fmaf(cz * lse, soft[q], out[q]);
        }
        if (in) {
            float* row = dlogits + r * n;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int j = 4 * (sub + L * v);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (!live) out[4 * v + q] = 0.f;
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
        if (blocks > (int64_t)kNumSMs * 4) blocks = (int64_t)kNumSMs * 4;                                            \
        e = launch_pdl(router_loss_grad_kernel<L, V>, dim3((unsigned)blocks), dim3(rloss::kThreads),                 \
                       sizeof(float) * G * 4 * V * L, stream, logits, idx, m, n, k, off, nseq, mask, fn, (double)alpha, \
                       (double)alpha_seq, (double)z_coef, counts, tokens, dloss, dgate, renorm, dlogits);            \
    } while (0)
    MOE_ROUTER_LOSS_DISPATCH(n, CALL);
#undef CALL
    return e;
}

}  // namespace moe
