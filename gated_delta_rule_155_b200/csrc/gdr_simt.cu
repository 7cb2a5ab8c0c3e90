// gdr_simt.cu — the head-gated delta rule in chunks of 64 tokens, exact fp32 on CUDA cores: every
// dtype and head size (bf16 at dk = dv = 128 has its own tensor-core kernels).
//
// One value head, one chunk, with G the running sum of the log-decays, gamma = e^G,
// lam_s = e^(G_C - G_s), D_ts = e^(G_t - G_s) for s <= t (all differences are <= 0 for g <= 0, so no
// factor overflows) and S the state at the chunk's start:
//
//   A_ts = beta_t D_ts k_t.k_s (s < t)   M = (I + A)^-1   P_ts = D_ts q_t.k_s (s <= t)
//   X = K S    R = beta (V - gamma X)    U = M R    O = gamma (Q S) + (P M) R
//   S <- gamma_C S + K^T (lam U)
//
// and for the gradients, with dS the gradient of the state at the chunk's end:
//
//   H = M^T (lam (K dS)) + (P M)^T dO    dV = W = beta H
//   dS <- gamma_C dS + Q^T (gamma dO) - K^T (gamma W)
//   dQ = gamma (dO S^T) + (dP.D) K       dP = dO U^T (s <= t)
//   dK = lam (U dS^T) - gamma (W S^T) + (dP.D)^T Q + N K + N^T K     N = -(W U^T).D (s < t)
//   dbeta_t = H_t.(V_t - gamma_t X_t) - sum_s (H U^T)_ts D_ts k_t.k_s
//   dg_t = gamma_C <dS, S> + sum_{s < t} k_s.(lam U dS^T)_s
//       + sum_{t' >= t} [q.(gamma dO S^T) - k.(gamma W S^T) + rowsum(E) - colsum(E)]_t',
//       E = dP.P + (N/D).(D K K^T)
//   (what crosses token t's gate; the writes enter by a sum over the tokens before t, not as
//   <dS, S_end> less those from t on, which would cancel where a gate forgets nearly all).
//
// M and P M are the same products in both directions, so one kernel makes them for every chunk at
// once (prep); what is left between chunks is three products a chunk, walked in order by one block
// per (sequence, value head, 32 state columns) — the columns of S never mix.  The gradients of
// q, k, g, beta need only their own chunk's S and dS, which the two walks leave in the workspace.
#include "gdr.cuh"

namespace kda {
namespace {

using namespace gdr;

constexpr int NT = 256;
constexpr int NS = 32;          // state columns of a chain block
constexpr int LM = 68;          // row stride of 64 x 64 fp32 tiles
constexpr int LS = NS + 4;      // row stride of state slices

struct Ws {                     // fp32 workspace, items = slots * Hv
    float *M, *PM;              // [items, 64, 64]
    float *S, *dS;              // [items, dk, dv]   (backward)
    float *U, *H;               // [items, 64, dv]   (backward)
};

Ws carve(void *ws, long long items, int dk, int dv, bool backward)
{
    float *p = (float *)ws;
    Ws w{};
    w.M = p; p += items * CH * CH;
    w.PM = p; p += items * CH * CH;
    if (backward) {
        w.S = p; p += items * dk * dv;
        w.dS = p; p += items * dk * dv;
        w.U = p; p += items * CH * dv;
        w.H = p; p += items * CH * dv;
    }
    return w;
}

struct P {
    GdrArgs a;
    Ws w;
};

// rows [row0, row0 + valid) of head h of [T, H, D] as fp32 rows of LD floats; rows behind `valid` are zeros
template <typename IO, int D, int LD>
KDA_DEVICE void load_rows(float *dst, const IO *src, size_t row0, int H, int h, int valid, int tid, int col0 = 0, int ld = D)
{
    for (int u = tid; u < CH * (D / 4); u += NT) {
        const int t = u / (D / 4), c = 4 * (u % (D / 4));
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (t < valid) ld4(src + ((row0 + t) * H + h) * ld + col0 + c, x);
        st4(dst + t * LD + c, x);
    }
}

// gates of a chunk: G (hi + lo), gamma, lam, beta; zeros (no decay, no write) behind `valid`.  One barrier inside.
struct Gates {
    float raw[CH], hi[CH], lo[CH], gam[CH], lam[CH], beta[CH];
};
template <typename IO>
KDA_DEVICE void load_gates(Gates &s, const IO *g, const IO *beta, size_t row0, int Hv, int hv, int valid, int tid)
{
    if (tid < CH) {
        s.raw[tid] = tid < valid ? clamp_gate(ld_f32(g + (row0 + tid) * Hv + hv)) : 0.0f;
        s.beta[tid] = tid < valid ? ld_f32(beta + (row0 + tid) * Hv + hv) : 0.0f;
    }
    __syncthreads();
    if (tid < 32) {
        gate_sums(s.raw, s.hi, s.lo, tid);
        __syncwarp();
        for (int t = tid; t < CH; t += 32) {
            s.gam[t] = __expf(s.hi[t]);
            s.lam[t] = __expf((s.hi[CH - 1] - s.hi[t]) + (s.lo[CH - 1] - s.lo[t]));
        }
    }
}
KDA_DEVICE float decay(const Gates &s, int t, int u) { return __expf((s.hi[t] - s.hi[u]) + (s.lo[t] - s.lo[u])); }

// acc[i][j] += sum_k A[ra + i][k] B[rb + 16 j][k]   (both rows along k, K a multiple of 4)
template <int K, int NI, int NJ>
KDA_DEVICE void mm_nt(float (&acc)[NI][NJ], const float *A, int lda, const float *B, int ldb)
{
#pragma unroll 4
    for (int k = 0; k < K; k += 4) {
        float4 a[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) a[i] = *(const float4 *)(A + i * lda + k);
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const float4 b = *(const float4 *)(B + 16 * j * ldb + k);
#pragma unroll
            for (int i = 0; i < NI; ++i)
                acc[i][j] += a[i].x * b.x + a[i].y * b.y + a[i].z * b.z + a[i].w * b.w;
        }
    }
}
// acc[i][j] += sum_k A[i][k] B[k][j]   (A rows along k, B rows of 4 consecutive columns)
template <int K>
KDA_DEVICE void mm_nn(float (&acc)[4][4], const float *A, int lda, const float *B, int ldb)
{
#pragma unroll 4
    for (int k = 0; k < K; k += 4) {
        float a[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) ld4(A + i * lda + k, a[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float b[4];
            ld4(B + (k + e) * ldb, b);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += a[i][e] * b[j];
        }
    }
}
// acc[i][j] += sum_k A[k][i] B[k][j]   (4 consecutive columns of both)
template <int K>
KDA_DEVICE void mm_tn(float (&acc)[4][4], const float *A, int lda, const float *B, int ldb)
{
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        float a[4], b[4];
        ld4(A + k * lda, a);
        ld4(B + k * ldb, b);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] += a[i] * b[j];
    }
}

// ---------------------------------------------------------------- prep: M and P M of every chunk
template <typename IO, int DK>
__global__ void __launch_bounds__(NT) gdr_prep_simt_kernel(P p)
{
    const GdrArgs &a = p.a;
    int n, c;
    SeqSpan span;
    if (!find_slot(a.cu, a.N, a.T, blockIdx.x, n, c, span)) return;
    extern __shared__ float sm[];
    constexpr int LK = DK + 4;
    float *K = sm, *Q = K + CH * LK, *A = Q + CH * LK, *Pm = A + CH * LM;
    float *M = K;             // K and Q are read only by the Gram products
    __shared__ Gates gs;
    const int tid = threadIdx.x, hv = blockIdx.y, hk = hv / (a.Hv / a.Hk);
    const size_t row0 = (size_t)span.row0 + c * CH;
    const int valid = min(CH, span.len - c * CH);
    load_rows<IO, DK, LK>(K, (const IO *)a.k, row0, a.Hk, hk, valid, tid);
    load_rows<IO, DK, LK>(Q, (const IO *)a.q, row0, a.Hk, hk, valid, tid);
    load_gates<IO>(gs, (const IO *)a.g, (const IO *)a.beta, row0, a.Hv, hv, valid, tid);
    __syncthreads();
    const int ty = tid >> 4, tx = tid & 15;
    float kk[4][4] = {}, qk[4][4] = {};
    mm_nt<DK>(kk, K + 4 * ty * LK, LK, K + tx * LK, LK);
    mm_nt<DK>(qk, Q + 4 * ty * LK, LK, K + tx * LK, LK);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = 4 * ty + i, s = tx + 16 * j;
            const float d = s <= t ? decay(gs, t, s) : 0.0f;
            A[t * LM + s] = s < t ? gs.beta[t] * d * kk[i][j] : 0.0f;
            Pm[t * LM + s] = s <= t ? d * qk[i][j] : 0.0f;
        }
    __syncthreads();
    unit_lower_inverse<LM>(A, M, tid);
    const size_t item = (size_t)blockIdx.x * a.Hv + hv;
    float pm[4][4] = {};
    mm_nn<CH>(pm, Pm + 4 * ty * LM, LM, M + 4 * tx, LM);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        st4(p.w.PM + item * CH * CH + (4 * ty + i) * CH + 4 * tx, pm[i]);
        st4(p.w.M + item * CH * CH + (4 * ty + i) * CH + 4 * tx, *(const float(*)[4])(M + (4 * ty + i) * LM + 4 * tx));
    }
}

// ---------------------------------------------------------------- the walk along a sequence
template <int D>
KDA_DEVICE void load_item(float *dst, int ld, const float *src, int tid)   // 64 rows of D floats
{
    for (int u = tid; u < CH * (D / 4); u += NT) {
        const int t = u / (D / 4), c = 4 * (u % (D / 4));
        *(float4 *)(dst + t * ld + c) = *(const float4 *)(src + t * D + c);
    }
}

// KEEP: leaves each chunk's start state and U in the workspace for the gradients, and writes no output
template <typename IO, int DK, int DV, bool KEEP>
__global__ void __launch_bounds__(NT) gdr_forward_simt_kernel(P p)
{
    const GdrArgs &a = p.a;
    extern __shared__ float sm[];
    constexpr int LK = DK + 4;
    float *KQ = sm, *MM = KQ + 2 * CH * LK, *S = MM + 2 * CH * LM, *R = S + DK * LS, *Y = R + CH * LS;
    __shared__ Gates gs;
    const int tid = threadIdx.x, col0 = blockIdx.x % (DV / NS) * NS, hv = blockIdx.y, n = blockIdx.x / (DV / NS), hk = hv / (a.Hv / a.Hk);
    const SeqSpan span = span_of(a.cu, n, a.N, a.T);
    const int nchunks = (span.len + CH - 1) / CH;
    const int page0 = a.s0 ? page_of(a.s0_index, n, a.pages, a.err) : -1;
    const float *s0 = page0 >= 0 ? a.s0 + ((size_t)page0 * a.Hv + hv) * DK * DV + col0 : nullptr;
    for (int u = tid; u < DK * NS; u += NT) {
        const int r = u / NS, c = u % NS;
        S[r * LS + c] = s0 ? s0[(size_t)r * DV + c] : 0.0f;
    }
    const int rg = tid >> 3, cg = 4 * (tid & 7);   // rows 4 rg .. + 3, columns cg .. + 3
    for (int ch = 0; ch < nchunks; ++ch) {
        const size_t row0 = (size_t)span.row0 + ch * CH;
        const int valid = min(CH, span.len - ch * CH);
        const size_t item = (size_t)(slot_base(span.row0, n) + ch) * a.Hv + hv;
        __syncthreads();
        load_rows<IO, DK, LK>(KQ, (const IO *)a.k, row0, a.Hk, hk, valid, tid);
        load_rows<IO, DK, LK>(KQ + CH * LK, (const IO *)a.q, row0, a.Hk, hk, valid, tid);
        load_item<CH>(MM, LM, p.w.M + item * CH * CH, tid);
        load_item<CH>(MM + CH * LM, LM, p.w.PM + item * CH * CH, tid);
        load_rows<IO, NS, LS>(R, (const IO *)a.v, row0, a.Hv, hv, valid, tid, col0, DV);
        load_gates<IO>(gs, (const IO *)a.g, (const IO *)a.beta, row0, a.Hv, hv, valid, tid);
        if (KEEP)
            for (int u = tid; u < DK * NS; u += NT)
                p.w.S[(item * DK + u / NS) * DV + col0 + u % NS] = S[(u / NS) * LS + u % NS];
        __syncthreads();
        float d1[4][4] = {};
        mm_nn<DK>(d1, KQ + 4 * rg * LK, LK, S + cg, LS);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * rg + i;
            if (t < CH) {   // X = K S -> R
                float v[4];
                ld4(R + t * LS + cg, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = gs.beta[t] * (v[j] - gs.gam[t] * d1[i][j]);
                st4(R + t * LS + cg, v);
            } else {        // Q S
#pragma unroll
                for (int j = 0; j < 4; ++j) d1[i][j] *= gs.gam[t - CH];
                st4(Y + (t - CH) * LS + cg, d1[i]);
            }
        }
        __syncthreads();
        float d2[4][4] = {};
        mm_nn<CH>(d2, MM + 4 * rg * LM, LM, R + cg, LS);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * rg + i;
            if (t < CH) {
                if (KEEP) st4(p.w.U + (item * CH + t) * DV + col0 + cg, d2[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) d2[i][j] *= gs.lam[t];
                st4(R + t * LS + cg, d2[i]);
            } else if (!KEEP && t - CH < valid) {
                float y[4];
                ld4(Y + (t - CH) * LS + cg, y);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] += d2[i][j];
                st4((IO *)a.out + ((row0 + t - CH) * a.Hv + hv) * DV + col0 + cg, y);
            }
        }
        __syncthreads();
        if (rg < DK / 4) {
            float s[4][4];
            const float gc = gs.gam[CH - 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ld4(S + (4 * rg + i) * LS + cg, s[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] *= gc;
            }
            mm_tn<CH>(s, KQ + 4 * rg, LK, R + cg, LS);
#pragma unroll
            for (int i = 0; i < 4; ++i) st4(S + (4 * rg + i) * LS + cg, s[i]);
        }
    }
    __syncthreads();
    if (KEEP || !a.sT) return;
    const int page = page_of(a.sT_index, n, a.pages, a.err);
    if (page < 0) return;
    if ((a.sT_index || (a.s0_index && a.sT == a.s0)) &&
        !page_is_free(a.sT_index, a.s0_index, a.sT == a.s0, n, a.N, page, tid, NT)) {
        if (tid == 0) raise_error(a.err, ERR_PAGE_INDEX);
        return;
    }
    float *sT = a.sT + ((size_t)page * a.Hv + hv) * DK * DV + col0;
    for (int u = tid; u < DK * NS; u += NT) sT[(size_t)(u / NS) * DV + u % NS] = S[(u / NS) * LS + u % NS];
}

template <typename IO, int DK, int DV>
__global__ void __launch_bounds__(NT) gdr_reverse_simt_kernel(P p)
{
    const GdrArgs &a = p.a;
    extern __shared__ float sm[];
    constexpr int LK = DK + 4;
    float *KQ = sm, *MM = KQ + 2 * CH * LK, *S = MM + 2 * CH * LM, *R = S + DK * LS;   // R: 128 rows
    __shared__ Gates gs;
    const int tid = threadIdx.x, col0 = blockIdx.x % (DV / NS) * NS, hv = blockIdx.y, n = blockIdx.x / (DV / NS), hk = hv / (a.Hv / a.Hk);
    const SeqSpan span = span_of(a.cu, n, a.N, a.T);
    const int nchunks = (span.len + CH - 1) / CH;
    const size_t st = ((size_t)n * a.Hv + hv) * DK * DV + col0;
    for (int u = tid; u < DK * NS; u += NT)
        S[(u / NS) * LS + u % NS] = a.dST ? a.dST[st + (size_t)(u / NS) * DV + u % NS] : 0.0f;
    const int rg = tid >> 3, cg = 4 * (tid & 7);
    for (int ch = nchunks - 1; ch >= 0; --ch) {
        const size_t row0 = (size_t)span.row0 + ch * CH;
        const int valid = min(CH, span.len - ch * CH);
        const size_t item = (size_t)(slot_base(span.row0, n) + ch) * a.Hv + hv;
        __syncthreads();
        load_rows<IO, DK, LK>(KQ, (const IO *)a.k, row0, a.Hk, hk, valid, tid);
        load_rows<IO, DK, LK>(KQ + CH * LK, (const IO *)a.q, row0, a.Hk, hk, valid, tid);
        load_item<CH>(MM, LM, p.w.M + item * CH * CH, tid);
        load_item<CH>(MM + CH * LM, LM, p.w.PM + item * CH * CH, tid);
        load_rows<IO, NS, LS>(R + CH * LS, (const IO *)a.dO, row0, a.Hv, hv, valid, tid, col0, DV);
        load_gates<IO>(gs, (const IO *)a.g, (const IO *)a.beta, row0, a.Hv, hv, valid, tid);
        for (int u = tid; u < DK * NS; u += NT)
            p.w.dS[(item * DK + u / NS) * DV + col0 + u % NS] = S[(u / NS) * LS + u % NS];
        __syncthreads();
        const int t0 = 4 * rg;   // rows of the 64-row products: the first 128 threads
        if (t0 < CH) {
            float d1[4][4] = {};
            mm_nn<DK>(d1, KQ + t0 * LK, LK, S + cg, LS);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) d1[i][j] *= gs.lam[t0 + i];
                st4(R + (t0 + i) * LS + cg, d1[i]);
            }
        }
        __syncthreads();
        float h[4][4] = {};
        if (t0 < CH) mm_tn<2 * CH>(h, MM + t0, LM, R + cg, LS);
        __syncthreads();
        if (t0 < CH) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = t0 + i;
                st4(p.w.H + (item * CH + t) * DV + col0 + cg, h[i]);
                float w[4], x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = gs.beta[t] * h[i][j];
                if (t < valid) st4((IO *)a.dv_ + ((row0 + t) * a.Hv + hv) * DV + col0 + cg, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] *= -gs.gam[t];
                st4(R + t * LS + cg, w);
                ld4(R + (CH + t) * LS + cg, x);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] *= gs.gam[t];
                st4(R + (CH + t) * LS + cg, x);
            }
        }
        __syncthreads();
        if (rg < DK / 4) {
            float s[4][4];
            const float gc = gs.gam[CH - 1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ld4(S + (4 * rg + i) * LS + cg, s[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] *= gc;
            }
            mm_tn<2 * CH>(s, KQ + 4 * rg, LK, R + cg, LS);
#pragma unroll
            for (int i = 0; i < 4; ++i) st4(S + (4 * rg + i) * LS + cg, s[i]);
        }
    }
    __syncthreads();
    if (!a.ds0) return;
    for (int u = tid; u < DK * NS; u += NT) a.ds0[st + (size_t)(u / NS) * DV + u % NS] = S[(u / NS) * LS + u % NS];
}

// ---------------------------------------------------------------- gradients of q, k, g, beta, a chunk and key head a block
template <typename IO, int DK, int DV>
__global__ void __launch_bounds__(NT) gdr_grads_simt_kernel(P p)
{
    const GdrArgs &a = p.a;
    int n, c;
    SeqSpan span;
    if (!find_slot(a.cu, a.N, a.T, blockIdx.x, n, c, span)) return;
    extern __shared__ float sm[];
    constexpr int LK = DK + 4, LV = DV + 4, NJ = DK / 16;
    float *K = sm, *Q = K + CH * LK, *dO = Q + CH * LK, *U = dO + CH * LV, *H = U + CH * LV;
    float *DP = dO, *NM = U;                 // after their last use: dP.D and N, 64 x LM
    static_assert(LV >= LM, "the 64 x 64 tiles fit over dO and U");
    __shared__ Gates gs;
    __shared__ float s_row[CH], s_col[4][CH], s_db[CH], s_red[NT / 32];
    const int tid = threadIdx.x, hk = blockIdx.y, rep = a.Hv / a.Hk;
    const int ty = tid >> 4, tx = tid & 15;
    const size_t row0 = (size_t)span.row0 + c * CH;
    const int valid = min(CH, span.len - c * CH);
    load_rows<IO, DK, LK>(K, (const IO *)a.k, row0, a.Hk, hk, valid, tid);
    load_rows<IO, DK, LK>(Q, (const IO *)a.q, row0, a.Hk, hk, valid, tid);
    float dq[4][NJ] = {}, dk[4][NJ] = {};    // rows 4 ty + i, columns tx + 16 j
    auto sum16 = [](float v) {               // over the 16 threads of a row
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    for (int r = 0; r < rep; ++r) {
        const int hv = hk * rep + r;
        const size_t item = (size_t)blockIdx.x * a.Hv + hv;
        const float *S = p.w.S + item * DK * DV, *dS = p.w.dS + item * DK * DV;
        __syncthreads();
        load_rows<IO, DV, LV>(dO, (const IO *)a.dO, row0, a.Hv, hv, valid, tid);
        load_item<DV>(U, LV, p.w.U + item * CH * DV, tid);
        load_item<DV>(H, LV, p.w.H + item * CH * DV, tid);
        load_gates<IO>(gs, (const IO *)a.g, (const IO *)a.beta, row0, a.Hv, hv, valid, tid);
        // <dS, S> of the start state
        float ss = 0.0f;
        for (int u = tid; u < DK * DV / 4; u += NT) {
            const float4 x = *(const float4 *)(S + 4 * u), y = *(const float4 *)(dS + 4 * u);
            ss += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
        }
        ss = warp_sum(ss);
        if ((tid & 31) == 0) s_red[tid >> 5] = ss;
        __syncthreads();
        float row[4], kud[4], db[4];         // per row: the part of dG, k.(lam U dS^T), dbeta
        {
            float x[4][NJ] = {};
            mm_nt<DV>(x, dO + 4 * ty * LV, LV, S + (size_t)tx * DV, DV);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float gm = gs.gam[4 * ty + i];
                float s = 0.0f;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    x[i][j] *= gm;
                    dq[i][j] += x[i][j];
                    s += x[i][j] * Q[(4 * ty + i) * LK + tx + 16 * j];
                }
                row[i] = sum16(s);
            }
        }
        {
            float x[4][NJ] = {};
            mm_nt<DV>(x, H + 4 * ty * LV, LV, S + (size_t)tx * DV, DV);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 4 * ty + i;
                const float gm = gs.gam[t], bt = gs.beta[t];
                float s = 0.0f, hvv = 0.0f;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    x[i][j] *= gm;
                    dk[i][j] -= bt * x[i][j];
                    s += x[i][j] * K[t * LK + tx + 16 * j];
                }
                if (t < valid)
                    for (int e = tx; e < DV; e += 16)
                        hvv += H[t * LV + e] * ld_f32((const IO *)a.v + ((row0 + t) * a.Hv + hv) * DV + e);
                s = sum16(s);
                row[i] -= bt * s;
                db[i] = sum16(hvv) - s;
            }
        }
        {
            float x[4][NJ] = {};
            mm_nt<DV>(x, U + 4 * ty * LV, LV, dS + (size_t)tx * DV, DV);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lm = gs.lam[4 * ty + i];
                float s = 0.0f;
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    x[i][j] *= lm;
                    dk[i][j] += x[i][j];
                    s += x[i][j] * K[(4 * ty + i) * LK + tx + 16 * j];
                }
                kud[i] = sum16(s);
            }
        }
        // 64 x 64 products: rows 4 ty + i, columns tx + 16 j
        float dp[4][4] = {}, hu[4][4] = {}, qk[4][4] = {}, kk[4][4] = {};
        mm_nt<DV>(dp, dO + 4 * ty * LV, LV, U + tx * LV, LV);
        mm_nt<DV>(hu, H + 4 * ty * LV, LV, U + tx * LV, LV);
        mm_nt<DK>(qk, Q + 4 * ty * LK, LK, K + tx * LK, LK);
        mm_nt<DK>(kk, K + 4 * ty * LK, LK, K + tx * LK, LK);
        __syncthreads();                     // dO and U are consumed
        float ecol[4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * ty + i;
            float er = 0.0f, dbs = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int s = tx + 16 * j;
                const float d = s <= t ? decay(gs, t, s) : 0.0f;
                const float dpd = s <= t ? dp[i][j] * d : 0.0f;
                const float hud = s < t ? hu[i][j] * d : 0.0f;
                const float nm = -gs.beta[t] * hud;
                DP[t * LM + s] = dpd;
                NM[t * LM + s] = nm;
                const float e = s < t ? dpd * qk[i][j] + nm * kk[i][j] : 0.0f;   // s == t cancels in rowsum - colsum
                er += e;
                ecol[j] += e;
                dbs += hud * kk[i][j];
            }
            row[i] += sum16(er);
            db[i] -= sum16(dbs);
        }
        // column sums over the 16 row groups: two per warp, eight warps
#pragma unroll
        for (int j = 0; j < 4; ++j) ecol[j] += __shfl_xor_sync(0xffffffffu, ecol[j], 16);
        if (tx == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s_row[4 * ty + i] = row[i];
                s_db[4 * ty + i] = db[i];
                s_col[0][4 * ty + i] = kud[i];
            }
        }
        __syncthreads();
        float *cs = H;                       // H's last use was hu; 8 rows of partial column sums
        if ((tid & 16) == 0)
#pragma unroll
            for (int j = 0; j < 4; ++j) cs[(tid >> 5) * CH + tx + 16 * j] = ecol[j];
        __syncthreads();
        if (tid < CH) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < NT / 32; ++w) s += cs[w * CH + tid];
            s_col[1][tid] = s_row[tid] - s;
        }
        __syncthreads();
        if (tid < 32) {
            float base = 0.0f;
            for (int w = 0; w < NT / 32; ++w) base += s_red[w];
            base *= gs.gam[CH - 1];
            float lo, hi, wl, wh;
            sums_across(s_col[1][tid], s_col[1][tid + 32], s_col[0][tid], s_col[0][tid + 32], lo, hi, wl, wh, tid);
            if (tid < valid) ((IO *)a.dg)[(row0 + tid) * a.Hv + hv] = from_f32<IO>(base + wl + lo);
            if (tid + 32 < valid) ((IO *)a.dg)[(row0 + tid + 32) * a.Hv + hv] = from_f32<IO>(base + wh + hi);
        } else if (tid >= 64 && tid - 64 < valid) {
            if (tid < 128) ((IO *)a.dbeta)[(row0 + tid - 64) * a.Hv + hv] = from_f32<IO>(s_db[tid - 64]);
        }
        // dQ += dPD K;  dK += N K + dPD^T Q + N^T K
        for (int s = 0; s < CH; ++s) {
            float kv[NJ], qv[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                kv[j] = K[s * LK + tx + 16 * j];
                qv[j] = Q[s * LK + tx + 16 * j];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 4 * ty + i;
                const float x = DP[t * LM + s], y = NM[t * LM + s] + NM[s * LM + t], z = DP[s * LM + t];
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    dq[i][j] += x * kv[j];
                    dk[i][j] += y * kv[j] + z * qv[j];
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = 4 * ty + i;
        if (t >= valid) continue;
        const size_t o = ((row0 + t) * a.Hk + hk) * DK;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            ((IO *)a.dq)[o + tx + 16 * j] = from_f32<IO>(dq[i][j]);
            ((IO *)a.dk_)[o + tx + 16 * j] = from_f32<IO>(dk[i][j]);
        }
    }
}

template <int DK>
constexpr int prep_bytes() { return (2 * CH * (DK + 4) + 2 * CH * LM) * 4; }
template <int DK>
constexpr int chain_bytes() { return (2 * CH * (DK + 4) + 2 * CH * LM + DK * LS + 2 * CH * LS) * 4; }
template <int DK, int DV>
constexpr int grads_bytes() { return (2 * CH * (DK + 4) + 3 * CH * (DV + 4)) * 4; }
static_assert(chain_bytes<128>() <= 227 * 1024 && grads_bytes<128, 128>() <= 227 * 1024, "shared memory per block");

template <typename IO, int DK, int DV>
cudaError_t launch_all(const GdrArgs &a, bool backward, cudaStream_t s)
{
    struct TagP; struct TagF; struct TagK; struct TagR; struct TagG;
    const long long slots = gdr_slots(a.N, a.T);
    P p{a, carve(a.ws, slots * a.Hv, DK, DV, backward)};
    cudaError_t e;
    if (a.T > 0) {
        if ((e = smem_opt_in<TagP>((const void *)gdr_prep_simt_kernel<IO, DK>, prep_bytes<DK>())) != cudaSuccess) return e;
        gdr_prep_simt_kernel<IO, DK><<<dim3((unsigned)slots, a.Hv), NT, prep_bytes<DK>(), s>>>(p);
    }
    const dim3 chain((unsigned)a.N * (DV / NS), a.Hv);
    if (!backward) {
        auto fn = gdr_forward_simt_kernel<IO, DK, DV, false>;
        if ((e = smem_opt_in<TagF>((const void *)fn, chain_bytes<DK>())) != cudaSuccess) return e;
        fn<<<chain, NT, chain_bytes<DK>(), s>>>(p);
        return cudaGetLastError();
    }
    if (a.T > 0) {
        auto fn = gdr_forward_simt_kernel<IO, DK, DV, true>;
        if ((e = smem_opt_in<TagK>((const void *)fn, chain_bytes<DK>())) != cudaSuccess) return e;
        fn<<<chain, NT, chain_bytes<DK>(), s>>>(p);
    }
    auto rv = gdr_reverse_simt_kernel<IO, DK, DV>;
    if ((e = smem_opt_in<TagR>((const void *)rv, chain_bytes<DK>())) != cudaSuccess) return e;
    rv<<<chain, NT, chain_bytes<DK>(), s>>>(p);
    if (a.T > 0) {
        auto gr = gdr_grads_simt_kernel<IO, DK, DV>;
        if ((e = smem_opt_in<TagG>((const void *)gr, grads_bytes<DK, DV>())) != cudaSuccess) return e;
        gr<<<dim3((unsigned)slots, a.Hk), NT, grads_bytes<DK, DV>(), s>>>(p);
    }
    return cudaGetLastError();
}

template <typename IO>
cudaError_t launch_dims(const GdrArgs &a, bool backward, cudaStream_t s)
{
    if (a.dk == 64) return a.dv == 64 ? launch_all<IO, 64, 64>(a, backward, s) : launch_all<IO, 64, 128>(a, backward, s);
    return a.dv == 64 ? launch_all<IO, 128, 64>(a, backward, s) : launch_all<IO, 128, 128>(a, backward, s);
}

}  // namespace

size_t gdr_simt_workspace(int N, int T, int Hk, int Hv, int dk, int dv, bool backward)
{
    (void)Hk;
    const size_t items = (size_t)gdr_slots(N, T) * Hv;
    return 4 * items * (2 * gdr::CH * gdr::CH + (backward ? 2 * (size_t)dk * dv + 2 * gdr::CH * dv : 0));
}

cudaError_t launch_gdr_forward_simt(const GdrArgs &a, cudaStream_t s)
{
    return a.io == IO_BF16 ? launch_dims<__nv_bfloat16>(a, false, s) : launch_dims<float>(a, false, s);
}
cudaError_t launch_gdr_backward_simt(const GdrArgs &a, cudaStream_t s)
{
    return a.io == IO_BF16 ? launch_dims<__nv_bfloat16>(a, true, s) : launch_dims<float>(a, true, s);
}

}  // namespace kda
