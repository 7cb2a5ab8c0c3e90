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
// per (sequence, value head, 16 state columns) — the columns of S never mix.  The gradients of
// q, k, g, beta need only their own chunk's S and dS, which the two walks leave in the workspace.
#include "gdr.cuh"

namespace kda {
namespace {

using namespace gdr;

constexpr int NT = 256;         // threads of prep and of the gradients
constexpr int WT = 128;         // threads of a walk
constexpr int NS = 16;          // state columns of a walk's block
constexpr int LM = 68;          // row stride of 64 x 64 fp32 tiles
constexpr int LS = NS + 4;      // row stride of state slices
constexpr int ITEM = 2 * CH * CH + 256;   // floats of a chunk and value head: M, P M, then gamma, lam, beta (64 each)

struct Ws {                     // fp32 workspace, items = slots * Hv
    float *I;                   // [items, ITEM]
    float *S, *dS;              // [items, dk, dv]   (backward)
    float *U, *H;               // [items, 64, dv]   (backward)
    float *dq, *dk;             // [items, 64, dk]   (backward, grouped heads): each value head's part
};

Ws carve(void *ws, long long items, int dk, int dv, bool backward, bool grouped)
{
    float *p = (float *)ws;
    Ws w{};
    w.I = p; p += items * ITEM;
    if (backward) {
        w.S = p; p += items * dk * dv;
        w.dS = p; p += items * dk * dv;
        w.U = p; p += items * CH * dv;
        w.H = p; p += items * CH * dv;
        if (grouped) {
            w.dq = p; p += items * CH * dk;
            w.dk = p; p += items * CH * dk;
        }
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
        st4(p.w.I + item * ITEM + CH * CH + (4 * ty + i) * CH + 4 * tx, pm[i]);
        st4(p.w.I + item * ITEM + (4 * ty + i) * CH + 4 * tx, *(const float(*)[4])(M + (4 * ty + i) * LM + 4 * tx));
    }
    if (tid < CH) {
        float *g = p.w.I + item * ITEM + 2 * CH * CH + tid;
        g[0] = gs.gam[tid];
        g[CH] = gs.lam[tid];
        g[2 * CH] = gs.beta[tid];
    }
}

// ---------------------------------------------------------------- the walks along a sequence
// A block has 16 columns of a head's state, its rows in registers (and as an operand in shared memory).
// Thread (rg, cg): tokens rg and rg + 32 of the chunk's products, or dk / 32 state rows, of columns
// cg .. cg + 3, so a product's step of four k is 4 + 4 16-byte loads for 64 FMAs and what a token's rows
// of one product give stays in registers for the next.  The next chunk's tiles come by cp.async (bf16:
// through registers) under this chunk's products.
KDA_DEVICE void cp_async16(void *dst, const void *src, bool take)
{
    const int n = take ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(n)
                 : "memory");
}
KDA_DEVICE void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
KDA_DEVICE void cp_async_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

template <typename IO, int DK>
struct Tiles {
    static constexpr int LK = DK + 4;
    static constexpr int KQ = 2 * CH * LK, MM = 2 * CH * LM, STAGE = KQ + MM + 256;   // floats
    static constexpr bool DIRECT = sizeof(IO) == 4;
    static constexpr int U = DIRECT ? 1 : CH * DK * 2 * 2 / 16 / WT;   // 16-byte pieces of bf16 K and Q rows a thread
    uint4 hold[U];
    // starts the copies of a chunk into the stage `b`; K, Q rows behind `valid` are zeros
    KDA_DEVICE void fetch(float *b, const GdrArgs &a, const float *item, size_t row0, int hk, int valid, int tid)
    {
        if (DIRECT) {
            for (int u = tid; u < 2 * CH * (DK / 4); u += WT) {
                const int r = u / (DK / 4), c = 4 * (u % (DK / 4)), t = r & (CH - 1);
                const float *src = (const float *)(r < CH ? a.k : a.q) + ((row0 + min(t, valid - 1)) * a.Hk + hk) * DK + c;
                cp_async16(b + r * LK + c, src, t < valid);
            }
        } else {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int u = tid + i * WT, r = u / (DK / 8), c = 8 * (u % (DK / 8)), t = r & (CH - 1);
                hold[i] = t < valid ? *(const uint4 *)((const IO *)(r < CH ? a.k : a.q) + ((row0 + t) * a.Hk + hk) * DK + c)
                                    : make_uint4(0u, 0u, 0u, 0u);
            }
        }
        for (int u = tid; u < 2 * CH * (CH / 4); u += WT)
            cp_async16(b + KQ + (u / (CH / 4)) * LM + 4 * (u % (CH / 4)), item + 4 * u, true);
        if (tid < 48) cp_async16(b + KQ + MM + 4 * tid, item + 2 * CH * CH + 4 * tid, true);
        cp_async_commit();
    }
    KDA_DEVICE void put(float *b, int tid)   // bf16: the rows that fetch has read
    {
        if (DIRECT) return;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int u = tid + i * WT, r = u / (DK / 8), c = 8 * (u % (DK / 8));
            const uint32_t w[4] = {hold[i].x, hold[i].y, hold[i].z, hold[i].w};
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = __uint_as_float(w[e] << 16);
                x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
            }
            st4(b + r * LK + c, *(const float(*)[4])x);
            st4(b + r * LK + c + 4, *(const float(*)[4])(x + 4));
        }
    }
};

// acc[i][j] += sum_{k < K} A[32 i ld + k] B[k][j]: NI rows 32 apart, four columns
template <int K, int NI>
KDA_DEVICE void mm_rows(float (&acc)[NI][4], const float *A, int lda, int step, const float *B)
{
#pragma unroll 4
    for (int k = 0; k < K; k += 4) {
        float a[NI][4];
#pragma unroll
        for (int i = 0; i < NI; ++i) ld4(A + i * step * lda + k, a[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float b[4];
            ld4(B + (k + e) * LS, b);
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += a[i][e] * b[j];
        }
    }
}
// SR consecutive floats
template <int SR>
KDA_DEVICE void ld_row(const float *p, float (&x)[SR])
{
    if constexpr (SR == 4) ld4(p, x);
    else { const float2 t = *(const float2 *)p; x[0] = t.x; x[1] = t.y; }
}

// KEEP: leaves each chunk's start state and U in the workspace for the gradients, and writes no output
template <typename IO, int DK, int DV, bool KEEP>
__global__ void __launch_bounds__(WT) gdr_forward_simt_kernel(P p)
{
    const GdrArgs &a = p.a;
    extern __shared__ float sm[];
    using T = Tiles<IO, DK>;
    constexpr int LK = T::LK, SR = DK / 32;
    float *S = sm + 2 * T::STAGE, *R = S + DK * LS, *Ub = R + CH * LS;
    const int tid = threadIdx.x, col0 = blockIdx.x % (DV / NS) * NS, hv = blockIdx.y, n = blockIdx.x / (DV / NS), hk = hv / (a.Hv / a.Hk);
    const SeqSpan span = span_of(a.cu, n, a.N, a.T);
    const int nchunks = (span.len + CH - 1) / CH;
    const int rg = tid >> 2, cg = 4 * (tid & 3), r0 = rg * SR, col = col0 + cg;
    const int page0 = a.s0 ? page_of(a.s0_index, n, a.pages, a.err) : -1;
    float s[SR][4];
#pragma unroll
    for (int i = 0; i < SR; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
        if (page0 >= 0) ld4(a.s0 + (((size_t)page0 * a.Hv + hv) * DK + r0 + i) * DV + col, s[i]);
        st4(S + (r0 + i) * LS + cg, s[i]);
    }
    T tiles;
    float v[2][4], vn[2][4];
    const size_t item0 = (size_t)slot_base(span.row0, n);
    auto fetch = [&](int ch) {
        const size_t row0 = (size_t)span.row0 + ch * CH;
        const int valid = min(CH, span.len - ch * CH);
        tiles.fetch(sm + (ch & 1) * T::STAGE, a, p.w.I + ((item0 + ch) * a.Hv + hv) * ITEM, row0, hk, valid, tid);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) vn[i][j] = 0.0f;
            if (rg + 32 * i < valid) ld4((const IO *)a.v + ((row0 + rg + 32 * i) * a.Hv + hv) * DV + col, vn[i]);
        }
    };
    if (nchunks > 0) {
        fetch(0);
        tiles.put(sm, tid);
    }
    for (int ch = 0; ch < nchunks; ++ch) {
        const size_t row0 = (size_t)span.row0 + ch * CH, item = (item0 + ch) * a.Hv + hv;
        const int valid = min(CH, span.len - ch * CH);
        const float *KQ = sm + (ch & 1) * T::STAGE, *MM = KQ + T::KQ, *g = MM + T::MM;
        cp_async_wait();
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = vn[i][j];
        if (ch + 1 < nchunks) fetch(ch + 1);
        if (KEEP)
#pragma unroll
            for (int i = 0; i < SR; ++i) st4(p.w.S + (item * DK + r0 + i) * DV + col, s[i]);
        float x[4][4] = {};                          // rows: X of the two tokens, Q S of the two tokens
        if (KEEP) mm_rows<DK, 2>(*(float(*)[2][4])x, KQ + rg * LK, LK, 32, S + cg);
        else mm_rows<DK, 4>(x, KQ + rg * LK, LK, 32, S + cg);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = rg + 32 * i;
            const float gam = g[t], beta = g[2 * CH + t];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i][j] = beta * (v[i][j] - gam * x[i][j]);
                x[2 + i][j] *= gam;
            }
            st4(R + t * LS + cg, x[i]);
        }
        __syncthreads();
        float u[4][4] = {};                          // U of the two tokens, P U of the two tokens; M, P M are lower
        if (KEEP) {
            mm_rows<32, 2>(*(float(*)[2][4])u, MM + rg * LM, LM, 32, R + cg);
            mm_rows<32, 1>(*(float(*)[1][4])u[1], MM + (rg + 32) * LM + 32, LM, 0, R + 32 * LS + cg);
        } else {
            mm_rows<32, 4>(u, MM + rg * LM, LM, 32, R + cg);
            float w[2][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) { w[0][j] = u[1][j]; w[1][j] = u[3][j]; }
            mm_rows<32, 2>(w, MM + (rg + 32) * LM + 32, LM, 64, R + 32 * LS + cg);
#pragma unroll
            for (int j = 0; j < 4; ++j) { u[1][j] = w[0][j]; u[3][j] = w[1][j]; }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = rg + 32 * i;
            if (KEEP) st4(p.w.U + (item * CH + t) * DV + col, u[i]);
            const float lam = g[CH + t];
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = lam * u[i][j];
            st4(Ub + t * LS + cg, y);
            if (!KEEP && t < valid) {
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = x[2 + i][j] + u[2 + i][j];
                st4((IO *)a.out + ((row0 + t) * a.Hv + hv) * DV + col, y);
            }
        }
        __syncthreads();
        const float gc = g[CH - 1];
#pragma unroll
        for (int i = 0; i < SR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] *= gc;
#pragma unroll 8
        for (int t = 0; t < CH; ++t) {
            float kr[SR], b[4];
            ld_row<SR>(KQ + t * LK + r0, kr);
            ld4(Ub + t * LS + cg, b);
#pragma unroll
            for (int i = 0; i < SR; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] += kr[i] * b[j];
        }
#pragma unroll
        for (int i = 0; i < SR; ++i) st4(S + (r0 + i) * LS + cg, s[i]);
        if (ch + 1 < nchunks) tiles.put(sm + ((ch + 1) & 1) * T::STAGE, tid);
    }
    if (KEEP || !a.sT) return;
    const int page = page_of(a.sT_index, n, a.pages, a.err);
    if (page < 0) return;
    if ((a.sT_index || (a.s0_index && a.sT == a.s0)) &&
        !page_is_free(a.sT_index, a.s0_index, a.sT == a.s0, n, a.N, page, tid, WT)) {
        if (tid == 0) raise_error(a.err, ERR_PAGE_INDEX);
        return;
    }
#pragma unroll
    for (int i = 0; i < SR; ++i) st4(a.sT + (((size_t)page * a.Hv + hv) * DK + r0 + i) * DV + col, s[i]);
}

template <typename IO, int DK, int DV>
__global__ void __launch_bounds__(WT) gdr_reverse_simt_kernel(P p)
{
    const GdrArgs &a = p.a;
    extern __shared__ float sm[];
    using T = Tiles<IO, DK>;
    constexpr int LK = T::LK, SR = DK / 32;
    float *S = sm + 2 * T::STAGE, *Yb = S + DK * LS, *dO = Yb + CH * LS, *W = dO + CH * LS;
    const int tid = threadIdx.x, col0 = blockIdx.x % (DV / NS) * NS, hv = blockIdx.y, n = blockIdx.x / (DV / NS), hk = hv / (a.Hv / a.Hk);
    const SeqSpan span = span_of(a.cu, n, a.N, a.T);
    const int nchunks = (span.len + CH - 1) / CH;
    const int rg = tid >> 2, cg = 4 * (tid & 3), r0 = rg * SR, col = col0 + cg;
    const size_t st = (((size_t)n * a.Hv + hv) * DK + r0) * DV + col;
    float s[SR][4];
#pragma unroll
    for (int i = 0; i < SR; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
        if (a.dST) ld4(a.dST + st + (size_t)i * DV, s[i]);
        st4(S + (r0 + i) * LS + cg, s[i]);
    }
    T tiles;
    float y[2][4];
    const size_t item0 = (size_t)slot_base(span.row0, n);
    auto fetch = [&](int ch) {
        const size_t row0 = (size_t)span.row0 + ch * CH;
        const int valid = min(CH, span.len - ch * CH);
        tiles.fetch(sm + (ch & 1) * T::STAGE, a, p.w.I + ((item0 + ch) * a.Hv + hv) * ITEM, row0, hk, valid, tid);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[i][j] = 0.0f;
            if (rg + 32 * i < valid) ld4((const IO *)a.dO + ((row0 + rg + 32 * i) * a.Hv + hv) * DV + col, y[i]);
        }
    };
    if (nchunks > 0) {
        fetch(nchunks - 1);
        tiles.put(sm + ((nchunks - 1) & 1) * T::STAGE, tid);
    }
    for (int ch = nchunks - 1; ch >= 0; --ch) {
        const size_t row0 = (size_t)span.row0 + ch * CH, item = (item0 + ch) * a.Hv + hv;
        const int valid = min(CH, span.len - ch * CH);
        const float *KQ = sm + (ch & 1) * T::STAGE, *MM = KQ + T::KQ, *g = MM + T::MM;
        cp_async_wait();
        __syncthreads();
        st4(dO + rg * LS + cg, y[0]);
        st4(dO + (rg + 32) * LS + cg, y[1]);
        if (ch > 0) fetch(ch - 1);
#pragma unroll
        for (int i = 0; i < SR; ++i) st4(p.w.dS + (item * DK + r0 + i) * DV + col, s[i]);
        float x[2][4] = {};
        mm_rows<DK, 2>(x, KQ + rg * LK, LK, 32, S + cg);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float lam = g[CH + rg + 32 * i];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i][j] *= lam;
            st4(Yb + (rg + 32 * i) * LS + cg, x[i]);
        }
        __syncthreads();
        float h[2][4] = {};                          // H of tokens 2 rg, 2 rg + 1: rows from the warp's first token on
#pragma unroll 4
        for (int t = 16 * (tid >> 5); t < CH; ++t) {
            const float2 m = *(const float2 *)(MM + t * LM + 2 * rg), pm = *(const float2 *)(MM + (CH + t) * LM + 2 * rg);
            float b[4], c[4];
            ld4(Yb + t * LS + cg, b);
            ld4(dO + t * LS + cg, c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[0][j] += m.x * b[j] + pm.x * c[j];
                h[1][j] += m.y * b[j] + pm.y * c[j];
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * rg + i;
            const float gam = g[t], beta = g[2 * CH + t];
            st4(p.w.H + (item * CH + t) * DV + col, h[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[i][j] *= beta;
            if (t < valid) st4((IO *)a.dv_ + ((row0 + t) * a.Hv + hv) * DV + col, h[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[i][j] *= -gam;
            st4(W + t * LS + cg, h[i]);
        }
        __syncthreads();
        const float gc = g[CH - 1];
#pragma unroll
        for (int i = 0; i < SR; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] *= gc;
#pragma unroll 4
        for (int t = 0; t < CH; ++t) {
            float kr[SR], qr[SR], b[4], c[4];
            ld_row<SR>(KQ + t * LK + r0, kr);
            ld_row<SR>(KQ + (CH + t) * LK + r0, qr);
            ld4(W + t * LS + cg, b);
            ld4(dO + t * LS + cg, c);
            const float gam = g[t];
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] *= gam;
#pragma unroll
            for (int i = 0; i < SR; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] += kr[i] * b[j] + qr[i] * c[j];
        }
#pragma unroll
        for (int i = 0; i < SR; ++i) st4(S + (r0 + i) * LS + cg, s[i]);
        if (ch > 0) tiles.put(sm + ((ch - 1) & 1) * T::STAGE, tid);
    }
    if (!a.ds0) return;
#pragma unroll
    for (int i = 0; i < SR; ++i) st4(a.ds0 + st + (size_t)i * DV, s[i]);
}

// ---------------------------------------------------------------- gradients of q, k, g, beta, a chunk and value head a block
template <int D>
KDA_DEVICE void load_item(float *dst, int ld, const float *src, int tid)   // 64 rows of D floats
{
    for (int u = tid; u < CH * (D / 4); u += NT) {
        const int t = u / (D / 4), c = 4 * (u % (D / 4));
        *(float4 *)(dst + t * ld + c) = *(const float4 *)(src + t * D + c);
    }
}

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
    const int tid = threadIdx.x, hv = blockIdx.y, rep = a.Hv / a.Hk, hk = hv / rep;
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
    const size_t item = (size_t)blockIdx.x * a.Hv + hv;
    {
        const float *S = p.w.S + item * DK * DV, *dS = p.w.dS + item * DK * DV;
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
        if (rep > 1) {                       // a part of the group's sum
            const size_t o = (item * CH + t) * DK;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                p.w.dq[o + tx + 16 * j] = dq[i][j];
                p.w.dk[o + tx + 16 * j] = dk[i][j];
            }
            continue;
        }
        const size_t o = ((row0 + t) * a.Hk + hk) * DK;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            ((IO *)a.dq)[o + tx + 16 * j] = from_f32<IO>(dq[i][j]);
            ((IO *)a.dk_)[o + tx + 16 * j] = from_f32<IO>(dk[i][j]);
        }
    }
}

// dq, dk of a chunk and key head: the sum of its value heads' parts, in order
template <typename IO, int DK>
__global__ void __launch_bounds__(NT) gdr_group_sum_kernel(P p)
{
    const GdrArgs &a = p.a;
    int n, c;
    SeqSpan span;
    if (!find_slot(a.cu, a.N, a.T, blockIdx.x, n, c, span)) return;
    const int hk = blockIdx.y, rep = a.Hv / a.Hk, valid = min(CH, span.len - c * CH);
    const size_t row0 = (size_t)span.row0 + c * CH, item = (size_t)blockIdx.x * a.Hv + hk * rep;
    for (int u = threadIdx.x; u < valid * (DK / 4); u += NT) {
        const int t = u / (DK / 4), col = 4 * (u % (DK / 4));
        float x[4] = {}, y[4] = {};
        for (int r = 0; r < rep; ++r) {
            float e[4], f[4];
            ld4(p.w.dq + ((item + r) * CH + t) * DK + col, e);
            ld4(p.w.dk + ((item + r) * CH + t) * DK + col, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] += e[j];
                y[j] += f[j];
            }
        }
        const size_t o = ((row0 + t) * a.Hk + hk) * DK + col;
        st4((IO *)a.dq + o, x);
        st4((IO *)a.dk_ + o, y);
    }
}

template <int DK>
constexpr int prep_bytes() { return (2 * CH * (DK + 4) + 2 * CH * LM) * 4; }
template <int DK>
constexpr int walk_bytes(int buffers) { return (2 * (2 * CH * (DK + 4) + 2 * CH * LM + 256) + DK * LS + buffers * CH * LS) * 4; }
template <int DK, int DV>
constexpr int grads_bytes() { return (2 * CH * (DK + 4) + 3 * CH * (DV + 4)) * 4; }
static_assert(walk_bytes<128>(3) <= 227 * 1024 && grads_bytes<128, 128>() <= 227 * 1024, "shared memory per block");

template <typename IO, int DK, int DV>
cudaError_t launch_all(const GdrArgs &a, bool backward, cudaStream_t s)
{
    struct TagP; struct TagF; struct TagK; struct TagR; struct TagG;
    constexpr int FB = walk_bytes<DK>(2), RB = walk_bytes<DK>(3);
    const long long slots = gdr_slots(a.N, a.T);
    P p{a, carve(a.ws, slots * a.Hv, DK, DV, backward, a.Hv > a.Hk)};
    cudaError_t e;
    if (a.T > 0) {
        if ((e = smem_opt_in<TagP>((const void *)gdr_prep_simt_kernel<IO, DK>, prep_bytes<DK>())) != cudaSuccess) return e;
        gdr_prep_simt_kernel<IO, DK><<<dim3((unsigned)slots, a.Hv), NT, prep_bytes<DK>(), s>>>(p);
    }
    const dim3 chain((unsigned)a.N * (DV / NS), a.Hv);
    if (!backward) {
        auto fn = gdr_forward_simt_kernel<IO, DK, DV, false>;
        if ((e = smem_opt_in<TagF>((const void *)fn, FB)) != cudaSuccess) return e;
        fn<<<chain, WT, FB, s>>>(p);
        return cudaGetLastError();
    }
    if (a.T > 0) {
        auto fn = gdr_forward_simt_kernel<IO, DK, DV, true>;
        if ((e = smem_opt_in<TagK>((const void *)fn, FB)) != cudaSuccess) return e;
        fn<<<chain, WT, FB, s>>>(p);
    }
    auto rv = gdr_reverse_simt_kernel<IO, DK, DV>;
    if ((e = smem_opt_in<TagR>((const void *)rv, RB)) != cudaSuccess) return e;
    rv<<<chain, WT, RB, s>>>(p);
    if (a.T > 0) {
        auto gr = gdr_grads_simt_kernel<IO, DK, DV>;
        if ((e = smem_opt_in<TagG>((const void *)gr, grads_bytes<DK, DV>())) != cudaSuccess) return e;
        gr<<<dim3((unsigned)slots, a.Hv), NT, grads_bytes<DK, DV>(), s>>>(p);
        if (a.Hv > a.Hk) gdr_group_sum_kernel<IO, DK><<<dim3((unsigned)slots, a.Hk), NT, 0, s>>>(p);
    }
    return cudaGetLastError();
}

template <typename IO>
cudaError_t launch_dims(const GdrArgs &a, bool backward, cudaStream_t s)
{
    if (a.dk == 64) return a.dv == 64 ? launch_all<IO, 64, 64>(a, backward, s) : launch_all<IO, 64, 128>(a, backward, s);
    if (a.dv == 64) return launch_all<IO, 128, 64>(a, backward, s);
    if constexpr (sizeof(IO) == 4) return launch_all<IO, 128, 128>(a, backward, s);
    else return cudaErrorInvalidValue;   // the tensor-core kernels' shape
}

}  // namespace

size_t gdr_simt_workspace(int N, int T, int Hk, int Hv, int dk, int dv, bool backward)
{
    const size_t items = (size_t)gdr_slots(N, T) * Hv;
    return 4 * items * (ITEM + (backward ? 2 * (size_t)dk * dv + 2 * gdr::CH * dv + (Hv > Hk ? 2 * gdr::CH * dk : 0) : 0));
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
