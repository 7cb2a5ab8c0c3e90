// gdr_simt.cu — the head-gated delta rule in chunks of 64 tokens, to fp32 accuracy: every dtype and
// head size (bf16 at dk = dv = 128 has its own tensor-core kernels).
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
// fp32, d = 64: 1278 tokens of 12 heads in 15 + 52 us (4 us a chunk of the longest sequence), the gradients of 429
// tokens of 4 heads in 12 + 25 + 28 + 4 us; both wait on the latency of their own products.
#include "gdr.cuh"

namespace kda {
namespace {

using namespace gdr;

constexpr int NT = 256;         // threads of prep and of the gradients
constexpr int WT = 256;         // threads of a walk
constexpr int NS = 16;          // state columns of a walk's block
constexpr int LM = 68;          // row stride of 64 x 64 fp32 tiles
// Row stride of 16-column operands: 24 spreads the four rows and eight columns of a fragment over all banks
// (at dk = 128 there is room for 20 only, where two of the rows share eight banks)
template <int DK> constexpr int LS = DK == 64 ? 24 : 20;
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

// Products of shared-memory operands by warps, to fp32 accuracy on tf32 MMAs: x = hi + lo with hi rounded to
// tf32's 11 bits and lo the exact rest (read to 11 bits: x is off by 2^-23), products lo hi, hi lo, hi hi;
// lo lo is left out (2^-24).  Eight products at a time are summed by the MMA, which truncates, and added to
// the result with a rounded addition, so that long sums do not drift.
//   acc[i] += A[16 rows, k0 .. k1) B[k0 .. k1, columns 8 i ..), row r and k of A at A[r ar + k ak], k and
//   column n of B at B[k bk + n bn]; SCALED: row k of B times scale[k].
// Lane l has rows l / 4 (elements 0, 1) and l / 4 + 8 (2, 3), columns 2 (l % 4) and the next.
KDA_DEVICE void split_tf32(float x, uint32_t &hi, uint32_t &lo)
{
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(hi) : "f"(x));
    lo = __float_as_uint(x - __uint_as_float(hi));
}
KDA_DEVICE void mma_tf32(float (&c)[4], const uint32_t (&p)[4], const uint32_t (&q)[2])
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3]), "r"(q[0]), "r"(q[1]));
}
template <int NTL, bool SCALED = false>
KDA_DEVICE void mm(float (&acc)[NTL][4], int k0, int k1, const float *A, int ar, int ak, const float *B, int bk, int bn, int lane,
                   const float *scale = nullptr)
{
    const float *a = A + (lane >> 2) * ar + (lane & 3) * ak, *b = B + (lane & 3) * bk + (lane >> 2) * bn;
    // a narrow product has little independent work: the small products run on along k in accumulators of their own
    constexpr bool NARROW = NTL < 4;
    constexpr int AHEAD = NARROW ? 4 : 1;
    float s1[NARROW ? NTL : 1][4] = {}, s2[NARROW ? NTL : 1][4] = {};
#pragma unroll AHEAD
    for (int k = k0; k < k1; k += 8) {
        uint32_t ah[4], al[4];
        split_tf32(a[k * ak], ah[0], al[0]);
        split_tf32(a[8 * ar + k * ak], ah[1], al[1]);
        split_tf32(a[(k + 4) * ak], ah[2], al[2]);
        split_tf32(a[8 * ar + (k + 4) * ak], ah[3], al[3]);
        float f0 = 1.0f, f1 = 1.0f;
        if (SCALED) {
            f0 = scale[k + (lane & 3)];
            f1 = scale[k + 4 + (lane & 3)];
        }
#pragma unroll
        for (int i = 0; i < NTL; ++i) {
            uint32_t bh[2], bl[2];
            split_tf32(SCALED ? f0 * b[k * bk + 8 * i * bn] : b[k * bk + 8 * i * bn], bh[0], bl[0]);
            split_tf32(SCALED ? f1 * b[(k + 4) * bk + 8 * i * bn] : b[(k + 4) * bk + 8 * i * bn], bh[1], bl[1]);
            float c[4] = {};
            if constexpr (NARROW) {
                mma_tf32(s1[i], al, bh);
                mma_tf32(s2[i], ah, bl);
            } else {
                mma_tf32(c, al, bh);
                mma_tf32(c, ah, bl);
            }
            mma_tf32(c, ah, bh);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] += c[e];
        }
    }
    if constexpr (NARROW)
#pragma unroll
        for (int i = 0; i < NTL; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] += s1[i][e] + s2[i][e];
}

// ---------------------------------------------------------------- prep: M and P M of every chunk
template <typename IO, int DK>
__global__ void __launch_bounds__(NT) gdr_prep_simt_kernel(P p)
{
    follow();
    const GdrArgs &a = p.a;
    int n, c;
    SeqSpan span;
    if (!find_slot(a.cu, a.N, a.T, blockIdx.x, n, c, span)) return;
    extern __shared__ float sm[];
    constexpr int LK = DK + 4;
    float *K = sm, *Q = K + CH * LK, *A = Q + CH * LK, *Pm = A + CH * LM;
    float *M = A;             // the inverse takes A's place
    __shared__ Gates gs;
    const int tid = threadIdx.x, hv = blockIdx.y, hk = hv / (a.Hv / a.Hk);
    const size_t row0 = (size_t)span.row0 + c * CH;
    const int valid = min(CH, span.len - c * CH);
    load_rows<IO, DK, LK>(K, (const IO *)a.k, row0, a.Hk, hk, valid, tid);
    load_rows<IO, DK, LK>(Q, (const IO *)a.q, row0, a.Hk, hk, valid, tid);
    load_gates<IO>(gs, (const IO *)a.g, (const IO *)a.beta, row0, a.Hv, hv, valid, tid);
    __syncthreads();
    // rows 16 m .. of the warp, columns 32 h ..
    const int w = tid >> 5, lane = tid & 31, m = 16 * (w >> 1), h = 32 * (w & 1), g4 = lane >> 2, c2 = 2 * (lane & 3);
    {
        float kk[4][4] = {}, qk[4][4] = {};
        if (h <= m) {
            mm<4>(kk, 0, DK, K + m * LK, LK, 1, K + h * LK, 1, LK, lane);
            mm<4>(qk, 0, DK, Q + m * LK, LK, 1, K + h * LK, 1, LK, lane);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const int t = m + g4 + 4 * e, s = h + 8 * i + c2;
                float2 x, y;
                const float d0 = s <= t ? decay(gs, t, s) : 0.0f, d1 = s + 1 <= t ? decay(gs, t, s + 1) : 0.0f;
                x.x = s < t ? gs.beta[t] * d0 * kk[i][e] : 0.0f;
                x.y = s + 1 < t ? gs.beta[t] * d1 * kk[i][e + 1] : 0.0f;
                y.x = s <= t ? d0 * qk[i][e] : 0.0f;
                y.y = s + 1 <= t ? d1 * qk[i][e + 1] : 0.0f;
                *(float2 *)(A + t * LM + s) = x;
                *(float2 *)(Pm + t * LM + s) = y;
            }
    }
    __syncthreads();
    unit_lower_inverse<LM, NT / 32>(A, tid);
    const size_t item = (size_t)blockIdx.x * a.Hv + hv;
    float *dst = p.w.I + item * ITEM;
    float pm[4][4] = {};
    if (h <= m) mm<4>(pm, h, m + 16, Pm + m * LM, LM, 1, M + h, LM, 1, lane);   // both lower
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; e += 2)
            *(float2 *)(dst + CH * CH + (m + g4 + 4 * e) * CH + h + 8 * i + c2) = make_float2(pm[i][e], pm[i][e + 1]);
    for (int u = tid; u < CH * CH / 4; u += NT) {
        const int t = u >> 4, s = 4 * (u & 15);
        *(float4 *)(dst + 4 * u) = t < 32 && s >= 32 ? make_float4(0.f, 0.f, 0.f, 0.f) : *(const float4 *)(M + t * LM + s);
    }
    if (tid < CH) {
        float *g = p.w.I + item * ITEM + 2 * CH * CH + tid;
        g[0] = gs.gam[tid];
        g[CH] = gs.lam[tid];
        g[2 * CH] = gs.beta[tid];
    }
}

// ---------------------------------------------------------------- the walks along a sequence
// A block has 16 columns of a head's state, in registers as the MMAs' results lie (and as an operand in shared
// memory).  What a warp has of one product's rows stays in its registers for the next, three barriers a chunk;
// the next chunk's tiles come by cp.async (bf16: through registers) under this chunk's products.
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
            constexpr int STEP = WT / (DK / 4);      // rows between a thread's pieces
            const int t0 = tid / (DK / 4), c = 4 * (tid % (DK / 4));
            const size_t at = ((row0 + t0) * a.Hk + hk) * DK + c, step = (size_t)STEP * a.Hk * DK;
            const float *k = (const float *)a.k + at, *q = (const float *)a.q + at;
            float *d = b + t0 * LK + c;
#pragma unroll
            for (int i = 0; i < CH / STEP; ++i) {
                const bool in = t0 + i * STEP < valid;   // behind the end: 16 zero bytes, and an address that exists
                cp_async16(d + i * STEP * LK, in ? k + i * step : (const float *)a.k, in);
                cp_async16(d + (CH + i * STEP) * LK, in ? q + i * step : (const float *)a.q, in);
            }
        } else {
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int u = tid + i * WT, r = u / (DK / 8), c = 8 * (u % (DK / 8)), t = r & (CH - 1);
                hold[i] = t < valid ? *(const uint4 *)((const IO *)(r < CH ? a.k : a.q) + ((row0 + t) * a.Hk + hk) * DK + c)
                                    : make_uint4(0u, 0u, 0u, 0u);
            }
        }
        {
            const float *src = item + 4 * tid;
            float *d = b + KQ + (tid / (CH / 4)) * LM + 4 * (tid % (CH / 4));
#pragma unroll
            for (int i = 0; i < 2 * CH * (CH / 4) / WT; ++i) cp_async16(d + i * (WT / (CH / 4)) * LM, src + i * 4 * WT, true);
        }
        if (tid < 48) cp_async16(b + KQ + MM + 4 * tid, item + 2 * CH * CH + 4 * tid, true);
        cp_async_commit();
    }
    KDA_DEVICE void put(float *b, int tid)   // bf16: the rows that fetch has read
    {
        if constexpr (!DIRECT)
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

// two neighbouring elements
KDA_DEVICE float2 ld2(const float *p) { return *(const float2 *)p; }
KDA_DEVICE float2 ld2(const __nv_bfloat16 *p) { return __bfloat1622float2(*(const __nv_bfloat162 *)p); }
KDA_DEVICE void st2(float *p, float x, float y) { *(float2 *)p = make_float2(x, y); }
KDA_DEVICE void st2(__nv_bfloat16 *p, float x, float y) { *(__nv_bfloat162 *)p = __floats2bfloat162_rn(x, y); }

// KEEP: leaves each chunk's start state and U in the workspace for the gradients, and writes no output
template <typename IO, int DK, int DV, bool KEEP>
KDA_DEVICE void walk_forward(const P &p, unsigned block)
{
    const GdrArgs &a = p.a;
    extern __shared__ float sm[];
    using T = Tiles<IO, DK>;
    constexpr int LK = T::LK, L = LS<DK>;
    constexpr int NSR = DK == 64 ? 1 : 2;            // state tiles (16 rows, 8 columns) of a warp
    constexpr int NT1 = KEEP ? 1 : 2;                // token tiles: KEEP X's, a warp 16 tokens and 8 columns; else X's and Q S's, 16 columns
    float *S = sm + 2 * T::STAGE, *R = S + DK * L, *Ub = R + CH * L;
    const int tid = threadIdx.x, col0 = block % (DV / NS) * NS, hv = blockIdx.y, n = block / (DV / NS), hk = hv / (a.Hv / a.Hk);
    const SeqSpan span = span_of(a.cu, n, a.N, a.T);
    const int nchunks = (span.len + CH - 1) / CH;
    const int w = tid >> 5, lane = tid & 31, g4 = lane >> 2, c2 = 2 * (lane & 3);
    const int rs = DK == 64 ? 16 * (w >> 1) : 16 * w, ns = DK == 64 ? 8 * (w & 1) : 0;   // state tile
    const int m = KEEP ? 16 * (w >> 1) : 16 * (w & 3), nt = KEEP ? 8 * (w & 1) : 0;       // token tile
    const bool xrow = KEEP || w < 4;                 // of X and U; else of Q S and P U
    const int arow = m + (xrow ? 0 : CH);            // its rows in [K; Q] and [M; P M]
    const int page0 = a.s0 ? page_of(a.s0_index, n, a.pages, a.err) : -1;
    float s[NSR][4];
    auto each_state = [&](auto f) {                  // f(tile, element pair, row, column)
#pragma unroll
        for (int i = 0; i < NSR; ++i)
#pragma unroll
            for (int e = 0; e < 4; e += 2) f(i, e, rs + g4 + 4 * e, ns + 8 * i + c2);
    };
    auto each_token = [&](auto f) {
#pragma unroll
        for (int i = 0; i < NT1; ++i)
#pragma unroll
            for (int e = 0; e < 4; e += 2) f(i, e, m + g4 + 4 * e, nt + 8 * i + c2);
    };
    each_state([&](int i, int e, int row, int c) {
        float2 x = make_float2(0.0f, 0.0f);
        if (page0 >= 0) x = ld2(a.s0 + (((size_t)page0 * a.Hv + hv) * DK + row) * DV + col0 + c);
        s[i][e] = x.x;
        s[i][e + 1] = x.y;
        st2(S + row * L + c, x.x, x.y);
    });
    T tiles;
    float vn[NT1][4];
    const size_t item0 = (size_t)slot_base(span.row0, n);
    auto fetch = [&](int ch) {
        const size_t row0 = (size_t)span.row0 + ch * CH;
        const int valid = min(CH, span.len - ch * CH);
        tiles.fetch(sm + (ch & 1) * T::STAGE, a, p.w.I + ((item0 + ch) * a.Hv + hv) * ITEM, row0, hk, valid, tid);
        if (xrow)
            each_token([&](int i, int e, int t, int c) {
                float2 x = make_float2(0.0f, 0.0f);
                if (t < valid) x = ld2((const IO *)a.v + ((row0 + t) * a.Hv + hv) * DV + col0 + c);
                vn[i][e] = x.x;
                vn[i][e + 1] = x.y;
            });
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
        float v[NT1][4];
#pragma unroll
        for (int i = 0; i < NT1; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i][e] = vn[i][e];
        if (ch + 1 < nchunks) fetch(ch + 1);
        if (KEEP)
            each_state([&](int i, int e, int row, int c) { st2(p.w.S + (item * DK + row) * DV + col0 + c, s[i][e], s[i][e + 1]); });
        float x[NT1][4] = {};                        // X, or gamma Q S
        mm<NT1>(x, 0, DK, KQ + arow * LK, LK, 1, S + nt, L, 1, lane);
        each_token([&](int i, int e, int t, int c) {
            const float gam = g[t], beta = g[2 * CH + t];
            if (xrow) {
                st2(R + t * L + c, beta * (v[i][e] - gam * x[i][e]), beta * (v[i][e + 1] - gam * x[i][e + 1]));
            } else {
                x[i][e] *= gam;
                x[i][e + 1] *= gam;
            }
        });
        __syncthreads();
        float u[NT1][4] = {};                        // U, or P U; M and P M are lower
        mm<NT1>(u, 0, m + 16, MM + arow * LM, LM, 1, R + nt, L, 1, lane);
        each_token([&](int i, int e, int t, int c) {
            if (xrow) {
                const float lam = g[CH + t];
                st2(Ub + t * L + c, lam * u[i][e], lam * u[i][e + 1]);
                if (KEEP) st2(p.w.U + (item * CH + t) * DV + col0 + c, u[i][e], u[i][e + 1]);
            } else if (t < valid) {
                st2((IO *)a.out + ((row0 + t) * a.Hv + hv) * DV + col0 + c, x[i][e] + u[i][e], x[i][e + 1] + u[i][e + 1]);
            }
        });
        __syncthreads();
        const float gc = g[CH - 1];
#pragma unroll
        for (int i = 0; i < NSR; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][e] *= gc;
        mm<NSR>(s, 0, CH, KQ + rs, 1, LK, Ub + ns, L, 1, lane);
        each_state([&](int i, int e, int row, int c) { st2(S + row * L + c, s[i][e], s[i][e + 1]); });
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
    each_state([&](int i, int e, int row, int c) {
        st2(a.sT + (((size_t)page * a.Hv + hv) * DK + row) * DV + col0 + c, s[i][e], s[i][e + 1]);
    });
}

template <typename IO, int DK, int DV>
KDA_DEVICE void walk_reverse(const P &p, unsigned block)
{
    const GdrArgs &a = p.a;
    extern __shared__ float sm[];
    using T = Tiles<IO, DK>;
    constexpr int LK = T::LK, L = LS<DK>, NSR = DK == 64 ? 1 : 2;
    float *S = sm + 2 * T::STAGE, *Yb = S + DK * L, *dO = Yb + CH * L, *W = dO + CH * L;
    const int tid = threadIdx.x, col0 = block % (DV / NS) * NS, hv = blockIdx.y, n = block / (DV / NS), hk = hv / (a.Hv / a.Hk);
    const SeqSpan span = span_of(a.cu, n, a.N, a.T);
    const int nchunks = (span.len + CH - 1) / CH;
    const int w = tid >> 5, lane = tid & 31, g4 = lane >> 2, c2 = 2 * (lane & 3);
    const int rs = DK == 64 ? 16 * (w >> 1) : 16 * w, ns = DK == 64 ? 8 * (w & 1) : 0;   // state tile
    const int m = 16 * (w >> 1), nt = 8 * (w & 1);                                        // token tile
    const size_t st = ((size_t)n * a.Hv + hv) * DK * DV + col0;
    float s[NSR][4];
    auto each_state = [&](auto f) {
#pragma unroll
        for (int i = 0; i < NSR; ++i)
#pragma unroll
            for (int e = 0; e < 4; e += 2) f(i, e, rs + g4 + 4 * e, ns + 8 * i + c2);
    };
    auto each_token = [&](auto f) {
#pragma unroll
        for (int e = 0; e < 4; e += 2) f(e, m + g4 + 4 * e, nt + c2);
    };
    each_state([&](int i, int e, int row, int c) {
        float2 x = make_float2(0.0f, 0.0f);
        if (a.dST) x = ld2(a.dST + st + (size_t)row * DV + c);
        s[i][e] = x.x;
        s[i][e + 1] = x.y;
        st2(S + row * L + c, x.x, x.y);
    });
    T tiles;
    float y[4];
    const size_t item0 = (size_t)slot_base(span.row0, n);
    auto fetch = [&](int ch) {
        const size_t row0 = (size_t)span.row0 + ch * CH;
        const int valid = min(CH, span.len - ch * CH);
        tiles.fetch(sm + (ch & 1) * T::STAGE, a, p.w.I + ((item0 + ch) * a.Hv + hv) * ITEM, row0, hk, valid, tid);
        each_token([&](int e, int t, int c) {
            float2 x = make_float2(0.0f, 0.0f);
            if (t < valid) x = ld2((const IO *)a.dO + ((row0 + t) * a.Hv + hv) * DV + col0 + c);
            y[e] = x.x;
            y[e + 1] = x.y;
        });
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
        each_token([&](int e, int t, int c) { st2(dO + t * L + c, y[e], y[e + 1]); });
        if (ch > 0) fetch(ch - 1);
        each_state([&](int i, int e, int row, int c) { st2(p.w.dS + (item * DK + row) * DV + col0 + c, s[i][e], s[i][e + 1]); });
        float x[1][4] = {};
        mm<1>(x, 0, DK, KQ + m * LK, LK, 1, S + nt, L, 1, lane);
        each_token([&](int e, int t, int c) {
            const float lam = g[CH + t];
            st2(Yb + t * L + c, lam * x[0][e], lam * x[0][e + 1]);
        });
        __syncthreads();
        float h[1][4] = {};                          // H: rows of M and P M from the tile's first token on
        mm<1>(h, m, CH, MM + m, 1, LM, Yb + nt, L, 1, lane);
        mm<1>(h, m, CH, MM + CH * LM + m, 1, LM, dO + nt, L, 1, lane);
        each_token([&](int e, int t, int c) {
            const float gam = g[t], beta = g[2 * CH + t];
            st2(p.w.H + (item * CH + t) * DV + col0 + c, h[0][e], h[0][e + 1]);
            const float d0 = beta * h[0][e], d1 = beta * h[0][e + 1];
            if (t < valid) st2((IO *)a.dv_ + ((row0 + t) * a.Hv + hv) * DV + col0 + c, d0, d1);
            st2(W + t * L + c, -gam * d0, -gam * d1);
        });
        __syncthreads();
        const float gc = g[CH - 1];
#pragma unroll
        for (int i = 0; i < NSR; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][e] *= gc;
        mm<NSR>(s, 0, CH, KQ + rs, 1, LK, W + ns, L, 1, lane);
        mm<NSR, true>(s, 0, CH, KQ + CH * LK + rs, 1, LK, dO + ns, L, 1, lane, g);
        each_state([&](int i, int e, int row, int c) { st2(S + row * L + c, s[i][e], s[i][e + 1]); });
        if (ch > 0) tiles.put(sm + ((ch - 1) & 1) * T::STAGE, tid);
    }
    if (!a.ds0) return;
    each_state([&](int i, int e, int row, int c) { st2(a.ds0 + st + (size_t)row * DV + c, s[i][e], s[i][e + 1]); });
}

template <typename IO, int DK, int DV>
__global__ void __launch_bounds__(WT) gdr_forward_simt_kernel(P p)
{
    follow();
    walk_forward<IO, DK, DV, false>(p, blockIdx.x);
}
// Both walks of the backward pass at once: neither reads what the other leaves.
template <typename IO, int DK, int DV>
__global__ void __launch_bounds__(WT) gdr_walks_simt_kernel(P p)
{
    follow();
    const unsigned half = gridDim.x / 2;
    if (blockIdx.x >= half) walk_forward<IO, DK, DV, true>(p, blockIdx.x - half);
    else walk_reverse<IO, DK, DV>(p, blockIdx.x);
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
    follow();
    const GdrArgs &a = p.a;
    int n, c;
    SeqSpan span;
    if (!find_slot(a.cu, a.N, a.T, blockIdx.x, n, c, span)) return;
    extern __shared__ float sm[];
    constexpr int LK = DK + 4, LV = DV + 4, NTL = DK / 16;   // column tiles of a warp: half the channels
    constexpr bool STAGED = DK == 64 && DV == 64;            // S and dS fit in shared memory beside the rest
    float *K = sm, *Q = K + CH * LK, *dO = Q + CH * LK, *U = dO + CH * LV, *H = U + CH * LV;
    float *S = H + CH * LV, *dS = S + DK * LV;               // (STAGED)
    float *DP = dO, *NM = U;                 // after their last use: dP.D and N, 64 x LM
    static_assert(LV >= LM, "the 64 x 64 tiles fit over dO and U");
    __shared__ Gates gs;
    __shared__ float s_row[2][CH], s_kud[2][CH], s_db[2][CH], s_col[4][CH], s_red[NT / 32];
    const int tid = threadIdx.x, hv = blockIdx.y, rep = a.Hv / a.Hk, hk = hv / rep;
    // the warp: tokens 16 m .., channels (or columns) of half h
    const int w = tid >> 5, lane = tid & 31, m = 16 * (w >> 1), h = w & 1, g4 = lane >> 2, c2 = 2 * (lane & 3);
    const size_t row0 = (size_t)span.row0 + c * CH;
    const int valid = min(CH, span.len - c * CH);
    const size_t item = (size_t)blockIdx.x * a.Hv + hv;
    load_rows<IO, DK, LK>(K, (const IO *)a.k, row0, a.Hk, hk, valid, tid);
    load_rows<IO, DK, LK>(Q, (const IO *)a.q, row0, a.Hk, hk, valid, tid);
    load_rows<IO, DV, LV>(dO, (const IO *)a.dO, row0, a.Hv, hv, valid, tid);
    load_item<DV>(U, LV, p.w.U + item * CH * DV, tid);
    load_item<DV>(H, LV, p.w.H + item * CH * DV, tid);
    load_gates<IO>(gs, (const IO *)a.g, (const IO *)a.beta, row0, a.Hv, hv, valid, tid);
    const float *Sg = p.w.S + item * DK * DV, *dSg = p.w.dS + item * DK * DV;
    int ls = DV;
    {   // <dS, S>
        float ss = 0.0f;
        for (int u = tid; u < DK * DV / 4; u += NT) {
            const float4 x = *(const float4 *)(Sg + 4 * u), y = *(const float4 *)(dSg + 4 * u);
            ss += x.x * y.x + x.y * y.y + x.z * y.z + x.w * y.w;
            if (STAGED) {
                *(float4 *)(S + (u / (DV / 4)) * LV + 4 * (u % (DV / 4))) = x;
                *(float4 *)(dS + (u / (DV / 4)) * LV + 4 * (u % (DV / 4))) = y;
            }
        }
        ss = warp_sum(ss);
        if (lane == 0) s_red[w] = ss;
    }
    if (STAGED) {
        Sg = S;
        dSg = dS;
        ls = LV;
    }
    __syncthreads();
    // sums over a row: of the four lanes that share it (its other half is another warp's)
    auto row_sum = [](float v) {
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        return v + __shfl_xor_sync(0xffffffffu, v, 2);
    };
    const int t2[2] = {m + g4, m + g4 + 8};
    const float gm[2] = {gs.gam[t2[0]], gs.gam[t2[1]]}, bt[2] = {gs.beta[t2[0]], gs.beta[t2[1]]};
    float dq[NTL][4], dk[NTL][4], row[2] = {}, kud[2] = {}, db[2] = {};
    const int c0 = h * (DK / 2) + c2;        // the lane's channels: c0 + 8 i and the next
    auto dot_row = [&](const float(&x)[NTL][4], const float *R, float (&d)[2]) {
        d[0] = d[1] = 0.0f;
#pragma unroll
        for (int i = 0; i < NTL; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float2 r = *(const float2 *)(R + t2[e] * LK + c0 + 8 * i);
                d[e] += x[i][2 * e] * r.x + x[i][2 * e + 1] * r.y;
            }
    };
    {   // gamma (dO S^T)
        float d[2];
#pragma unroll
        for (int i = 0; i < NTL; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) dq[i][e] = 0.0f;
        mm<NTL>(dq, 0, DV, dO + m * LV, LV, 1, Sg + h * (DK / 2) * ls, 1, ls, lane);
#pragma unroll
        for (int i = 0; i < NTL; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) dq[i][e] *= gm[e >> 1];
        dot_row(dq, Q, d);
        row[0] += d[0];
        row[1] += d[1];
    }
    {   // - beta gamma (H S^T)
        float d[2];
#pragma unroll
        for (int i = 0; i < NTL; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) dk[i][e] = 0.0f;
        mm<NTL>(dk, 0, DV, H + m * LV, LV, 1, Sg + h * (DK / 2) * ls, 1, ls, lane);
#pragma unroll
        for (int i = 0; i < NTL; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) dk[i][e] *= gm[e >> 1];
        dot_row(dk, K, d);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            row[e] -= bt[e] * d[e];
            db[e] -= d[e];
            if (t2[e] < valid)               // H.V, a quarter of a half row a lane
                for (int x = h * (DV / 2) + 4 * (lane & 3); x < (h + 1) * (DV / 2); x += 16) {
                    float v[4], y[4];
                    ld4((const IO *)a.v + ((row0 + t2[e]) * a.Hv + hv) * DV + x, v);
                    ld4(H + t2[e] * LV + x, y);
                    db[e] += (v[0] * y[0] + v[1] * y[1]) + (v[2] * y[2] + v[3] * y[3]);
                }
        }
#pragma unroll
        for (int i = 0; i < NTL; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) dk[i][e] *= -bt[e >> 1];
    }
    {   // lam (U dS^T)
        float x[NTL][4] = {};
        mm<NTL>(x, 0, DV, U + m * LV, LV, 1, dSg + h * (DK / 2) * ls, 1, ls, lane);
#pragma unroll
        for (int i = 0; i < NTL; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[i][e] *= gs.lam[t2[e >> 1]];
                dk[i][e] += x[i][e];
            }
        dot_row(x, K, kud);
    }
    // the pairwise products: rows 16 m .., columns s = 32 h .., zero above the diagonal
    float dp[4][4] = {}, nm[4][4] = {};
    {
        float qk[4][4] = {}, kk[4][4] = {};
        if (32 * h <= m) {
            mm<4>(dp, 0, DV, dO + m * LV, LV, 1, U + 32 * h * LV, 1, LV, lane);
            mm<4>(nm, 0, DV, H + m * LV, LV, 1, U + 32 * h * LV, 1, LV, lane);
            mm<4>(qk, 0, DK, Q + m * LK, LK, 1, K + 32 * h * LK, 1, LK, lane);
            mm<4>(kk, 0, DK, K + m * LK, LK, 1, K + 32 * h * LK, 1, LK, lane);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float col[2] = {};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = t2[e >> 1], s = 32 * h + 8 * i + c2 + (e & 1);
                const float d = s <= t ? decay(gs, t, s) : 0.0f;
                const float dpd = s <= t ? dp[i][e] * d : 0.0f, hud = s < t ? nm[i][e] * d : 0.0f;
                dp[i][e] = dpd;
                nm[i][e] = -bt[e >> 1] * hud;
                const float x = s < t ? dpd * qk[i][e] + nm[i][e] * kk[i][e] : 0.0f;   // s == t cancels in rowsum - colsum
                row[e >> 1] += x;
                col[e & 1] += x;
                db[e >> 1] -= hud * kk[i][e];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {    // over the warp's 16 rows
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) col[e] += __shfl_xor_sync(0xffffffffu, col[e], o);
                if (g4 == 0) s_col[w >> 1][32 * h + 8 * i + c2 + e] = col[e];
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float x = row_sum(row[e]), y = row_sum(kud[e]), z = row_sum(db[e]);
        if ((lane & 3) == 0) {
            s_row[h][t2[e]] = x;
            s_kud[h][t2[e]] = y;
            s_db[h][t2[e]] = z;
        }
    }
    __syncthreads();                         // dO, U are consumed
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            st2(DP + t2[e] * LM + 32 * h + 8 * i + c2, dp[i][2 * e], dp[i][2 * e + 1]);
            st2(NM + t2[e] * LM + 32 * h + 8 * i + c2, nm[i][2 * e], nm[i][2 * e + 1]);
        }
    if (w == 0) {
        const float base = gs.gam[CH - 1] * warp_sum(lane < NT / 32 ? s_red[lane] : 0.0f);
        float x[2], y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = lane + 32 * i;
            x[i] = (s_row[0][t] + s_row[1][t]) - ((s_col[0][t] + s_col[1][t]) + (s_col[2][t] + s_col[3][t]));
            y[i] = s_kud[0][t] + s_kud[1][t];
        }
        float lo, hi, wl, wh;
        sums_across(x[0], x[1], y[0], y[1], lo, hi, wl, wh, lane);
        if (lane < valid) ((IO *)a.dg)[(row0 + lane) * a.Hv + hv] = from_f32<IO>(base + wl + lo);
        if (lane + 32 < valid) ((IO *)a.dg)[(row0 + lane + 32) * a.Hv + hv] = from_f32<IO>(base + wh + hi);
    } else if (w < 3) {
        const int t = 32 * (w - 1) + lane;
        if (t < valid) ((IO *)a.dbeta)[(row0 + t) * a.Hv + hv] = from_f32<IO>(s_db[0][t] + s_db[1][t]);
    }
    __syncthreads();
    // dQ += (dP.D) K;  dK += N K + N^T K + (dP.D)^T Q
    const float *Kh = K + h * (DK / 2), *Qh = Q + h * (DK / 2);
    mm<NTL>(dq, 0, m + 16, DP + m * LM, LM, 1, Kh, LK, 1, lane);
    mm<NTL>(dk, 0, m + 16, NM + m * LM, LM, 1, Kh, LK, 1, lane);
    mm<NTL>(dk, m, CH, NM + m, 1, LM, Kh, LK, 1, lane);
    mm<NTL>(dk, m, CH, DP + m, 1, LM, Qh, LK, 1, lane);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int t = t2[e];
        if (t >= valid) continue;
        if (rep > 1) {                       // a part of the group's sum
            const size_t o = (item * CH + t) * DK + c0;
#pragma unroll
            for (int i = 0; i < NTL; ++i) {
                st2(p.w.dq + o + 8 * i, dq[i][2 * e], dq[i][2 * e + 1]);
                st2(p.w.dk + o + 8 * i, dk[i][2 * e], dk[i][2 * e + 1]);
            }
        } else {
            const size_t o = ((row0 + t) * a.Hk + hk) * DK + c0;
#pragma unroll
            for (int i = 0; i < NTL; ++i) {
                st2((IO *)a.dq + o + 8 * i, dq[i][2 * e], dq[i][2 * e + 1]);
                st2((IO *)a.dk_ + o + 8 * i, dk[i][2 * e], dk[i][2 * e + 1]);
            }
        }
    }
}

// dq, dk of a chunk and key head: the sum of its value heads' parts, in order
template <typename IO, int DK>
__global__ void __launch_bounds__(NT) gdr_group_sum_kernel(P p)
{
    follow();
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
constexpr int walk_bytes(int buffers) { return (2 * (2 * CH * (DK + 4) + 2 * CH * LM + 256) + (DK + buffers * CH) * LS<DK>) * 4; }
template <int DK, int DV>
constexpr int grads_bytes() { return (2 * CH * (DK + 4) + 3 * CH * (DV + 4) + (DK == 64 && DV == 64 ? 2 * DK * (DV + 4) : 0)) * 4; }
static_assert(walk_bytes<128>(3) <= 227 * 1024 && grads_bytes<128, 128>() <= 227 * 1024, "shared memory per block");

template <typename IO, int DK, int DV>
cudaError_t launch_all(const GdrArgs &a, bool backward, cudaStream_t s)
{
    struct TagP; struct TagF; struct TagR; struct TagG;
    constexpr int FB = walk_bytes<DK>(2), RB = walk_bytes<DK>(3);
    const long long slots = gdr_slots(a.N, a.T);
    P p{a, carve(a.ws, slots * a.Hv, DK, DV, backward, a.Hv > a.Hk)};
    cudaError_t e;
    if (a.T > 0) {
        if ((e = smem_opt_in<TagP>((const void *)gdr_prep_simt_kernel<IO, DK>, prep_bytes<DK>())) != cudaSuccess) return e;
        e = launch_after(gdr_prep_simt_kernel<IO, DK>, dim3((unsigned)slots, a.Hv), NT, prep_bytes<DK>(), s, p);
        if (e != cudaSuccess) return e;
    }
    const dim3 chain((unsigned)a.N * (DV / NS), a.Hv);
    if (!backward) {
        auto fn = gdr_forward_simt_kernel<IO, DK, DV>;
        if ((e = smem_opt_in<TagF>((const void *)fn, FB)) != cudaSuccess) return e;
        return launch_after(fn, chain, WT, FB, s, p);
    }
    auto fn = gdr_walks_simt_kernel<IO, DK, DV>;
    if ((e = smem_opt_in<TagR>((const void *)fn, RB)) != cudaSuccess) return e;
    if ((e = launch_after(fn, dim3(2 * chain.x, chain.y), WT, RB, s, p)) != cudaSuccess) return e;
    if (a.T > 0) {
        auto gr = gdr_grads_simt_kernel<IO, DK, DV>;
        if ((e = smem_opt_in<TagG>((const void *)gr, grads_bytes<DK, DV>())) != cudaSuccess) return e;
        if ((e = launch_after(gr, dim3((unsigned)slots, a.Hv), NT, grads_bytes<DK, DV>(), s, p)) != cudaSuccess) return e;
        if (a.Hv > a.Hk) return launch_after(gdr_group_sum_kernel<IO, DK>, dim3((unsigned)slots, a.Hk), NT, 0, s, p);
    }
    return cudaSuccess;
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
