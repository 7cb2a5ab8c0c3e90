// gdr_tc_bwd.cu — gradients of the head-gated delta rule on tcgen05 tensor cores (bf16, dk = dv = 128).
// The formulas are those of gdr_simt.cu, the operand layouts and the forward sweep those of gdr_tc.cu.
//
// Three launches: prep; the forward walk, which leaves each chunk's start state S and U, together with the
// reverse walk (below), which leaves the gradient dS of each chunk's end state and H, and writes dv; then the
// gradients of q, k, g and beta, a block per chunk and key head, which need only their own chunk's S, dS, U and H.
// S, dS, U and H are left as bf16 operand tiles, rounded once: they meet only products whose result is
// stored in bf16 (the recurrences themselves keep fp32 and hi + lo operands).
//
// Reverse walk, transposed as the forward one (lanes of tensor memory = value columns):
//     Y^T = dS^T K^T     H^T = (lam Y)^T M + dO^T (P M)     dv = beta H
//     dS^T <- gamma_C dS^T + (gamma dO)^T Q - (beta gamma H)^T K
// dO enters the second product as it is; lam Y, gamma dO, beta gamma H, dS, M and P M as hi + lo pairs.
#include "gdr_tc_walk.cuh"

namespace kda {
namespace {

using namespace gdr;

// tensor memory columns: dS (fp32), dS as an operand (hi, lo), Y then lam Y then beta gamma H, H, gamma dO
KDA_DEVICE void walk_reverse(const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_do, const TcP &p, unsigned block)
{
    constexpr int TM_S = 0, TM_SHL = 128, TM_Y = 256, TM_H = 320, TM_G = 384;
    const GdrArgs &a = p.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t *full = (uint64_t *)(sm + W_BAR), *empty = full + STAGES;
    uint64_t *b_s = empty + STAGES, *b_y = b_s + 1, *b_w = b_s + 2;    // vector phases done
    uint64_t *m_y = b_s + 3, *m_h = b_s + 4, *m_s = b_s + 5;           // products done
    uint64_t *drain = b_s + 6;
    uint32_t *tslot = (uint32_t *)(drain + 1);
    volatile int *abort_flag = (volatile int *)(tslot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hv = (int)(block % a.Hv), hk = hv / (a.Hv / a.Hk);
    const int n = p.order ? p.order[block / a.Hv] : (int)(block / a.Hv);
    const SeqSpan span = span_of(a.cu, n, a.N, a.T);
    const int nchunks = (span.len + CH - 1) / CH;
    const size_t item0 = (size_t)slot_base(span.row0, n);

    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1 + 16);
        }
        mbar_init(b_s, 16);
        mbar_init(b_y, 16);
        mbar_init(b_w, 16);
        mbar_init(m_y, 1);
        mbar_init(m_h, 1);
        mbar_init(m_s, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    // step i works on chunk nchunks - 1 - i
    auto wait = [&](uint64_t *bar, int i) { return mbar_wait_bounded(bar, (uint32_t)(i & 1), abort_flag, a.err, p.wait_ns); };
    auto wait_all = [&](uint64_t *bar, int i) { return __all_sync(0xffffffffu, wait(bar, i)) != 0; };
    auto wait_full = [&](int i) { return wait_all(&full[i % STAGES], i / STAGES); };

    if (warp == 16) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            int issued = 0;
            if (nchunks > 0) {
                prefetch_tmap(&tm_q);
                prefetch_tmap(&tm_k);
                prefetch_tmap(&tm_do);
            }
            for (int i = 0; i < nchunks && !*abort_flag; ++i) {
                const int st = i % STAGES, ch = nchunks - 1 - i;
                if (i >= STAGES && !wait(&empty[st], i / STAGES - 1)) break;
                if (i == p.skip_load_chunk) continue;    // injected failure: the wait for it runs out
                uint8_t *s = sm + st * ST_BYTES;
                mbar_arrive_expect_tx(&full[st], 3 * TILE + IT_WALK);
                const int row = span.row0 + ch * CH;
                for (int cb = 0; cb < 2; ++cb) {
                    tma_load_4d(s + ST_KQ + cb * TILE, &tm_k, cb * 64, hk, row, 0, &full[st]);
                    tma_load_4d(s + ST_KQ + cb * TILE + TILE / 2, &tm_q, cb * 64, hk, row, 0, &full[st]);
                    tma_load_4d(s + ST_V + cb * (TILE / 2), &tm_do, cb * 64, hv, row, 0, &full[st]);
                }
                const uint8_t *item = p.items + ((item0 + ch) * a.Hv + hv) * IT_BYTES;
                bulk_load(s + ST_MM, item, IT_WALK, &full[st]);
                issued = i + 1;
                // prep has given up on this chunk: so does the block (found here, where nothing waits for the answer: as a
                // branch of the chain's or the MMAs' warps it took 1 to 2 % of a walk)
                if (((const float *)(item + IT_GATES))[GA_GAM + CH - 1] < 0.0f) *abort_flag = 1;
            }
            for (int seen = issued > STAGES ? issued - STAGES : 0; seen < issued && *abort_flag; ++seen)
                if (seen != p.skip_load_chunk)
                    mbar_wait_timed(&full[seen % STAGES], (uint32_t)((seen / STAGES) & 1), DRAIN_NS);
        }
        __syncwarp();
        if (a.ds0) named_bar_arrive(1, 544);             // every chunk's mark has been looked at
    } else if (warp == 17) {
        // ------------------------------------------------------------ MMAs
        constexpr uint32_t id_y = idesc_bf16(128, 64, false, false), id_h = idesc_bf16(128, 64, false, true),
                           id_p = idesc_bf16(128, 64, true, true), id_s = idesc_bf16(128, 128, false, true);
        auto keep_h = [&](int i) {
            bulk_store(p.H + ((item0 + nchunks - 1 - i) * a.Hv + hv) * TILE, sm + W_KEEP_U, TILE);
            bulk_commit();
        };
        bool ok = true;
        for (int i = 0; i < nchunks && ok; ++i) {
            uint8_t *s = sm + (i % STAGES) * ST_BYTES;
            ok = wait_full(i);
            const int valid = min(CH, span.len - (nchunks - 1 - i) * CH);
            if (valid < CH) {     // rows behind the end (the next sequence's, or NaN) meet zeros of the other operand
                for (int u = lane; u < (CH - valid) * 48; u += 32) {
                    const int t = valid + u / 48, b = u % 48 >> 3;   // b: K, Q of both channel blocks, dO of both
                    const int at = b < 4 ? ST_KQ + (b >> 1) * TILE + (b & 1) * (TILE / 2) : ST_V + (b & 1) * (TILE / 2);
                    *(uint4 *)(s + at + swz(t, u & 7)) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async();
                __syncwarp();
            }
            if (lane == 0) {
                const uint32_t kq = smem_u32(s + ST_KQ), mm = smem_u32(s + ST_MM), dy = smem_u32(s + ST_V);
                if (ok && (ok = wait(b_s, i))) {                 // dS^T K^T, then dO^T (P M)
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                        for (int hl = 0; hl < 2; ++hl)
                            mma_ts(tmem + TM_Y, tmem + TM_SHL + 64 * hl + 8 * kk,
                                   sdesc(kq + (kk >> 2) * TILE + (kk & 3) * 32, 16, 1024), id_y, kk | hl);
                    mma_commit(m_y);
                    if (i > 0) keep_h(i - 1);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int hl = 0; hl < 2; ++hl)
                            mma_ss(tmem + TM_H, sdesc(dy + kk * 2048, TILE / 2, 1024),
                                   sdesc(mm + hl * IT_LO + TILE / 2 + kk * 2048, TILE / 2, 1024), id_p, kk | hl);
                }
                if (ok && (ok = wait(b_y, i))) {                 // (lam Y)^T M, then (gamma dO)^T Q
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t yh = tmem + TM_Y + 16 * kk, yl = yh + 8;
                        const uint64_t bh = sdesc(mm + kk * 2048, TILE / 2, 1024), bl = sdesc(mm + IT_LO + kk * 2048, TILE / 2, 1024);
                        mma_ts(tmem + TM_H, yh, bh, id_h, 1);
                        mma_ts(tmem + TM_H, yl, bh, id_h, 1);
                        mma_ts(tmem + TM_H, yh, bl, id_h, 1);
                    }
                    bulk_wait_read_all();                        // H's tile may be written again
                    mma_commit(m_h);
                    bulk_store(p.dS + ((item0 + nchunks - 1 - i) * a.Hv + hv) * 2 * TILE, sm + W_KEEP_S, 2 * TILE);
                    bulk_commit();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int hl = 0; hl < 2; ++hl)
                            mma_ts(tmem + TM_S, tmem + TM_G + 16 * kk + 8 * hl, sdesc(kq + TILE / 2 + kk * 2048, TILE, 1024), id_s, 1);
                }
                if (ok && (ok = wait(b_w, i))) {                 // - (beta gamma H)^T K
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int hl = 0; hl < 2; ++hl)
                            mma_ts(tmem + TM_S, tmem + TM_Y + 16 * kk + 8 * hl, sdesc(kq + kk * 2048, TILE, 1024), id_s, 1);
                    bulk_wait_read_all();                        // and dS's
                    mma_commit(m_s);
                    mma_commit(&empty[i % STAGES]);
                }
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0);
        }
        if (lane == 0) {
            if (ok && nchunks > 0 && wait(b_s, nchunks)) keep_h(nchunks - 1);
            bulk_wait_read_all();
        }
        if (lane == 0 && *abort_flag) {
            mma_commit(drain);
            mbar_wait_timed(drain, 0u, DRAIN_NS);
        }
    } else {
        // ------------------------------------------------------------ the chain, and dv
        const int grp = warp >> 2, lq = warp & 3, dv = 32 * lq + lane;
        const uint32_t at = tmem + ((uint32_t)(32 * lq) << 16);
        const int r0 = 32 * grp, t0 = 16 * grp;      // the thread's state rows r0 .. + 31 and tokens t0 .. + 15 of column dv
        auto arrive = [&](uint64_t *bar) {           // after the writes to tensor memory
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        const size_t st0 = (((size_t)n * a.Hv + hv) * D + r0) * D + dv;
        {
            uint32_t x[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = a.dST ? __float_as_uint(a.dST[st0 + (size_t)e * D]) : 0u;
            tmem_st32(at + TM_S + r0, x);
            tmem_wait_st();                          // each thread reads back what it wrote itself
        }
        bool ok = true;
        for (int i = 0; i < nchunks; ++i) {
            const int ch = nchunks - 1 - i, st = i % STAGES, valid = min(CH, span.len - ch * CH);
            uint8_t *s = sm + st * ST_BYTES;
            const float *gates = (const float *)(s + ST_G);
            if (i > 0) {
                if (!(ok = wait_all(m_s, i - 1))) break;
                tc_fence_after();
            }
            uint32_t S[32];
            tmem_ld32(at + TM_S + r0, S);
            tmem_wait_ld();
            {
                uint32_t h[16], l[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) split2(__uint_as_float(S[2 * e]), __uint_as_float(S[2 * e + 1]), h[e], l[e]);
                tmem_st16(at + TM_SHL + (r0 >> 1), h);
                tmem_st16(at + TM_SHL + 64 + (r0 >> 1), l);
                arrive(b_s);
                uint8_t *dst = sm + W_KEEP_S + (grp >> 1) * TILE;        // [dv][state row]
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *(uint4 *)(dst + swz(dv, 4 * (grp & 1) + j)) = make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
                fence_proxy_async();
            }
            if (!(ok = wait_full(i))) break;
            {                                        // dS decayed, in the shadow of the product
                const float gC = gates[GA_GAM + CH - 1];
                float *x = (float *)S;
#pragma unroll
                for (int e = 0; e < 32; e += 2) mul2(x[e], x[e + 1], x[e], x[e + 1], gC, gC);
                tmem_st32(at + TM_S + r0, S);
            }
            float r[16], w[16];
            {                                        // gamma dO^T, column dv of the thread's tokens
                const uint8_t *dy = s + ST_V + (dv >> 6) * (TILE / 2) + t0 * 128 + 2 * (dv & 7);
                const int j = (dv & 63) >> 3;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    float g4[4];
                    ld4(gates + GA_GAM + t0 + e, g4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        r[e + k] = __bfloat162float(*(const __nv_bfloat16 *)(dy + (e + k) * 128 + ((j ^ ((e + k) & 7)) << 4)));
                    mul2(r[e], r[e + 1], r[e], r[e + 1], g4[0], g4[1]);
                    mul2(r[e + 2], r[e + 3], r[e + 2], r[e + 3], g4[2], g4[3]);
                }
                if (valid < CH)                      // rows behind the end may hold NaN
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (t0 + e >= valid) r[e] = 0.0f;
                put_tokens(at + TM_G + t0, r);
            }
#pragma unroll
            for (int e = 0; e < 16; e += 4) ld4(gates + GA_LAM + t0 + e, *(float(*)[4])(w + e));
            if (!(ok = wait_all(m_y, i))) break;
            tc_fence_after();
            {
                uint32_t x[16];
                tmem_ld16(at + TM_Y + t0, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 2)
                    mul2(r[e], r[e + 1], w[e], w[e + 1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                put_tokens(at + TM_Y + t0, r);
            }
            arrive(b_y);
#pragma unroll
            for (int e = 0; e < 16; e += 4) ld4(gates + GA_BG + t0 + e, *(float(*)[4])(w + e));
            if (!(ok = wait_all(m_h, i))) break;
            tc_fence_after();
            {
                uint32_t x[16];
                tmem_ld16(at + TM_H + t0, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 2)
                    mul2(r[e], r[e + 1], -w[e], -w[e + 1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                put_tokens(at + TM_Y + t0, r);       // lam Y has been read: H's product is done
                arrive(b_w);
                // H as an operand tile [token][dv], and dv = beta H
                uint8_t *hd = sm + W_KEEP_U + (dv >> 6) * (TILE / 2) + t0 * 128 + 2 * (dv & 7);
                const int j = (dv & 63) >> 3;
                __nv_bfloat16 *vd = (__nv_bfloat16 *)a.dv_ + (((size_t)span.row0 + ch * CH + t0) * a.Hv + hv) * D + dv;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    float b4[4];
                    ld4(gates + GA_BETA + t0 + e, b4);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float h = __uint_as_float(x[e + k]);
                        *(__nv_bfloat16 *)(hd + (e + k) * 128 + ((j ^ ((e + k) & 7)) << 4)) = __float2bfloat16_rn(h);
                        if (t0 + e + k < valid) vd[(size_t)((e + k) * a.Hv) * D] = __float2bfloat16_rn(b4[k] * h);
                    }
                }
                fence_proxy_async();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
        }
        if (ok && nchunks > 0) arrive(b_s);          // the last H's tile is written
        if (a.ds0) {
            if (nchunks > 0 && ok && (ok = wait_all(m_s, nchunks - 1))) tc_fence_after();
            named_bar_sync(1, 544);                  // all warps or none
            if (ok && !*abort_flag) {
                uint32_t x[32];
                tmem_ld32(at + TM_S + r0, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) a.ds0[st0 + (size_t)e * D] = __uint_as_float(x[e]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Both walks at once: neither reads what the other leaves, and where there are few sequences and heads each
// alone leaves SMs without work (64 + 64 blocks at 2 sequences of 32 heads: 243 us instead of 201 + 247).
// The halves of the grid, not neighbouring blocks, take the two: neighbours share an instruction cache, and
// with a reverse and a forward walk side by side the same call took 348 us.
__global__ void __launch_bounds__(W_THREADS, 1)
gdr_walks_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, TcP p)
{
    follow();
    const unsigned half = gridDim.x / 2;
    if (blockIdx.x >= half) walk_forward<true>(tm_q, tm_k, tm_v, p, blockIdx.x - half);
    else walk_reverse(tm_q, tm_k, tm_do, p, blockIdx.x);
}

// ---------------------------------------------------------------- gradients of q, k, g, beta
// A block per chunk and key head; per value head of the group, with lane t of tensor memory = token t of
// the k rows, lane 64 + t = token t of the q rows (A operands of 128 rows, stacked):
//     [K; Q] K^T                 (once)       D = e^(G_t - G_s)
//     [H; dO] U^T                -> N = -beta D (H U^T) below the diagonal, dPD = D (dO U^T)
//     [H; dO] S^T                -> dk -= beta gamma (H S^T), dq += gamma (dO S^T)
//     U dS^T                     -> dk += lam (U dS^T)
//     [N; dPD] K, N^T K + dPD^T Q -> dk, dq: sums of all the group's heads in tensor memory
// and the row sums and column sums that dg and dbeta need, in fp32 registers.  A thread has one token and
// half the channels (64) of the sums of dk or dq in registers.
// A block stays on its SM and takes every gridDim-th (chunk, key head); the tiles of the next value head come
// as soon as this one's have been read (the MMAs' and the dot products'), under the rest of its vector work.
// 2 x 4096 tokens of 32 heads (610 MB of tiles): 169 us, 3.9 TB/s.  Code size rules its loops: at 112 KB, above
// the 64 KB of the instruction cache, the same work took 326 us; with sixteen vector warps it takes 199 us.
constexpr int G_VT = 256;                        // vector threads: warps 0..7; warp 8: copies and MMAs
constexpr int G_THREADS = G_VT + 32;
constexpr int GS_KQ = 0, GS_HO = 4 * TILE, GS_S = 6 * TILE, GS_DS = 8 * TILE, GS_U = 10 * TILE, GS_V = 11 * TILE,
              GS_N = 12 * TILE, GS_ZERO = 13 * TILE;   // K, Q twice, as are the gates
constexpr int GS_GATES = GS_ZERO + TILE / 2;     // one head's gates (all six)
constexpr int GS_ROW = GS_GATES + 2 * 1536;      // floats [2 heads][2 halves][128]: row sums of the lanes
constexpr int GS_KUD = GS_ROW + 2 * 1024, GS_DB = GS_KUD + 2 * 512, GS_COL = GS_DB + 2 * 512;   // [2][2][64], [2][2][64], [2][4][64]
constexpr int GS_SUM = GS_COL + 2 * 1024;        // [2][8]
constexpr int GS_BAR = GS_SUM + 64, GS_BYTES = GS_BAR + 128 + 1024;
static_assert(GS_BYTES <= 232448, "shared memory per block");
constexpr int TG_GRAM = 0, TG_DP = 64, TG_ST = 128, TG_UD = 256, TG_ACC = 384;

KDA_DEVICE float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
KDA_DEVICE float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// d0 + d1 += the products of eight pairs of bf16
KDA_DEVICE void dot8(float &d0, float &d1, const uint4 &a, const uint4 &b)
{
    fma2(d0, d1, bf_lo(a.x), bf_hi(a.x), bf_lo(b.x), bf_hi(b.x), d0, d1);
    fma2(d0, d1, bf_lo(a.y), bf_hi(a.y), bf_lo(b.y), bf_hi(b.y), d0, d1);
    fma2(d0, d1, bf_lo(a.z), bf_hi(a.z), bf_lo(b.z), bf_hi(b.z), d0, d1);
    fma2(d0, d1, bf_lo(a.w), bf_hi(a.w), bf_lo(b.w), bf_hi(b.w), d0, d1);
}

__global__ void __launch_bounds__(G_THREADS, 1)
gdr_grads_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do, TcP p)
{
    follow();
    const GdrArgs &a = p.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t *full = (uint64_t *)(sm + GS_BAR);                      // a head's tiles
    uint64_t *m_p = full + 1, *m_st = full + 2, *m_ud = full + 3, *m_acc = full + 4;   // products done
    uint64_t *b_n = full + 5, *b_d = full + 6;                       // [N; dPD] written; TG_ST and TG_UD read
    uint64_t *b_dot = full + 7, *b_out = full + 8;                   // S, dS, H, V read; TG_ACC read
    uint64_t *drain = full + 9;
    uint32_t *tslot = (uint32_t *)(full + 10);
    volatile int *abort_flag = (volatile int *)(tslot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rep = a.Hv / a.Hk;
    const long long nwork = gdr_slots(a.N, a.T) * a.Hk;
    // the block's value heads in order: (slot, key head, head r of the group), i of them and wi groups before it
    struct Unit {
        long long w;
        int slot, hk, r, row0, valid, i, wi;
    };
    auto seek = [&](Unit &u) {               // the first (slot, key head) from u.w on whose slot is a chunk
        for (; u.w < nwork; u.w += gridDim.x) {
            u.slot = (int)(u.w / a.Hk);
            u.hk = (int)(u.w % a.Hk);
            const int2 rows = slot_rows(a.cu, a.N, a.T, u.slot);
            u.row0 = rows.x;
            u.valid = rows.y;
            if (rows.y) return;
        }
    };
    auto first = [&]() {
        Unit u{(long long)blockIdx.x, 0, 0, 0, 0, 0, 0, 0};
        seek(u);
        return u;
    };
    auto next = [&](Unit u) {
        ++u.i;
        if (++u.r == rep) {
            u.r = 0;
            ++u.wi;
            u.w += gridDim.x;
            seek(u);
        }
        return u;
    };

    if (tid == 0) {
        mbar_init(full, 1);
        mbar_init(m_p, 1);
        mbar_init(m_st, 1);
        mbar_init(m_ud, 1);
        mbar_init(m_acc, 1);
        mbar_init(b_n, G_VT / 32);
        mbar_init(b_d, G_VT / 32);
        mbar_init(b_dot, G_VT / 32);
        mbar_init(b_out, G_VT / 32);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    for (int u = tid; u < TILE / 2 / 16; u += G_THREADS) *(uint4 *)(sm + GS_ZERO + 16 * u) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    auto wait = [&](uint64_t *bar, int i) { return mbar_wait_bounded(bar, (uint32_t)(i & 1), abort_flag, a.err, p.wait_ns); };
    auto wait_all = [&](uint64_t *bar, int i) { return __all_sync(0xffffffffu, wait(bar, i)) != 0; };

    if (warp == 8) {
        // ------------------------------------------------------------ copies and MMAs
        int issued = 0;
        auto load = [&](const Unit &u) {
            const int hv = u.hk * rep + u.r;
            const size_t item = (size_t)u.slot * a.Hv + hv;
            uint8_t *kq = sm + GS_KQ + (u.wi & 1) * 2 * TILE;
            mbar_arrive_expect_tx(full, (u.r == 0 ? 2 * TILE : 0) + 8 * TILE + 1536);
            for (int cb = 0; cb < 2; ++cb) {
                if (u.r == 0) {
                    tma_load_4d(kq + cb * TILE, &tm_k, cb * 64, u.hk, u.row0, 0, full);
                    tma_load_4d(kq + cb * TILE + TILE / 2, &tm_q, cb * 64, u.hk, u.row0, 0, full);
                }
                bulk_load(sm + GS_HO + cb * TILE, p.H + item * TILE + cb * (TILE / 2), TILE / 2, full);
                tma_load_4d(sm + GS_HO + cb * TILE + TILE / 2, &tm_do, cb * 64, hv, u.row0, 0, full);
                tma_load_4d(sm + GS_V + cb * (TILE / 2), &tm_v, cb * 64, hv, u.row0, 0, full);
            }
            bulk_load(sm + GS_U, p.U + item * TILE, TILE, full);
            bulk_load(sm + GS_GATES + (u.i & 1) * 1536, p.items + item * IT_BYTES + IT_GATES, 1536, full);
            bulk_load(sm + GS_S, p.S + item * 2 * TILE, 2 * TILE, full);
            bulk_load(sm + GS_DS, p.dS + item * 2 * TILE, 2 * TILE, full);
            issued = u.i + 1;
        };
        const uint32_t ho = smem_u32(sm + GS_HO), ss = smem_u32(sm + GS_S), ds = smem_u32(sm + GS_DS),
                       uu = smem_u32(sm + GS_U), nn = smem_u32(sm + GS_N), zero = smem_u32(sm + GS_ZERO);
        constexpr uint32_t id_gram = idesc_bf16(128, 64, false, false), id_dp = idesc_bf16(128, 64, false, true),
                           id_st = idesc_bf16(128, 128, false, true), id_ud = idesc_bf16(128, 128, true, true);
        bool ok = true;
        Unit u = first();
        if (lane == 0 && u.w < nwork) load(u);
        while (u.w < nwork && ok) {
            const Unit v = next(u);
            uint8_t *kqt = sm + GS_KQ + (u.wi & 1) * 2 * TILE;
            const uint32_t kq = smem_u32(kqt);
            ok = wait_all(full, u.i);
            if (u.r == 0 && u.valid < CH) {   // K and Q rows behind the end meet the zeros of N and dPD
                for (int x = lane; x < (CH - u.valid) * 32; x += 32) {
                    const int t = u.valid + (x >> 5), b = (x >> 3) & 3;
                    *(uint4 *)(kqt + (b >> 1) * TILE + (b & 1) * (TILE / 2) + swz(t, x & 7)) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async();
                __syncwarp();
            }
            if (lane == 0 && ok) {
                if (u.i > 0) ok = wait(b_d, u.i - 1);
                if (ok) {
                    tc_fence_after();
                    if (u.r == 0)
#pragma unroll 2
                        for (int kk = 0; kk < 8; ++kk) {
                            const uint32_t x = kq + (kk >> 2) * TILE + (kk & 3) * 32;
                            mma_ss(tmem + TG_GRAM, sdesc(x, 16, 1024), sdesc(x, 16, 1024), id_gram, kk);
                        }
#pragma unroll 2
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ss(tmem + TG_DP, sdesc(ho + (kk >> 2) * TILE + (kk & 3) * 32, 16, 1024),
                               sdesc(uu + kk * 2048, TILE / 2, 1024), id_dp, kk);
                    mma_commit(m_p);
#pragma unroll 2
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ss(tmem + TG_ST, sdesc(ho + (kk >> 2) * TILE + (kk & 3) * 32, 16, 1024),
                               sdesc(ss + kk * 2048, TILE, 1024), id_st, kk);
                    mma_commit(m_st);
#pragma unroll 2
                    for (int kk = 0; kk < 8; ++kk)   // rows 64.. of A are whatever follows U: their lanes are not read
                        mma_ss(tmem + TG_UD, sdesc(uu + kk * 2048, TILE, 1024), sdesc(ds + kk * 2048, TILE, 1024), id_ud, kk);
                    mma_commit(m_ud);
                }
                // everything but K, Q and the gates has been read: the next head's tiles may come
                if (ok && (ok = wait(b_dot, u.i)) && (ok = wait(m_ud, u.i)) && v.w < nwork) load(v);
                if (ok && (ok = wait(b_n, u.i)) && (u.r > 0 || u.wi == 0 || (ok = wait(b_out, u.wi - 1)))) {
                    tc_fence_after();
#pragma unroll 2
                    for (int kk = 0; kk < 4; ++kk)   // [N; dPD] K
                        mma_ss(tmem + TG_ACC, sdesc(nn + kk * 32, 16, 1024), sdesc(kq + kk * 2048, TILE, 1024), id_st, u.r | kk);
#pragma unroll 2
                    for (int kk = 0; kk < 8; ++kk)   // rows 0..63 += N^T K, dPD^T Q; rows 64..: zeros
                        mma_ss(tmem + TG_ACC, sdesc(nn + kk * 2048, zero - nn - (kk >> 2) * (TILE / 2), 1024),
                               sdesc(kq + (kk >> 2) * (TILE / 2) + (kk & 3) * 2048, TILE, 1024), id_ud, 1);
                    mma_commit(m_acc);
                }
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0);
            u = v;
        }
        if (lane == 0 && *abort_flag) {
            if (issued > 0) mbar_wait_timed(full, (uint32_t)((issued - 1) & 1), DRAIN_NS);
            mma_commit(drain);
            mbar_wait_timed(drain, 0u, DRAIN_NS);
        }
    } else {
        // ------------------------------------------------------------ vector work
        const int lq = warp & 3, half = warp >> 2;
        const int L = 32 * lq + lane, t = L & 63;        // lane of tensor memory, token
        const bool krow = lq < 2;                        // a warp of k rows; else of q rows
        const uint32_t at = tmem + ((uint32_t)(32 * lq) << 16);
        float acc[64];                                   // channels 64 half ..: sums of dk or dq of row t
        bool ok = true;
        float gC = 0.0f;
        float *s_row, *s_kud, *s_db, *s_col, *s_sum;     // of even and odd heads in turn
        auto head = [&](const Unit &u) {                 // false: a wait has given up
            const int valid = u.valid;
            const float *gates = (const float *)(sm + GS_GATES + (u.i & 1) * 1536);
            const uint8_t *own = sm + GS_KQ + ((u.wi & 1) * 2 + half) * TILE;   // K, Q rows as the tiles have them: row L, block `half`
            if (u.r == 0)
#pragma unroll
                for (int e = 0; e < 64; ++e) acc[e] = 0.0f;
            if (!wait_all(full, u.i)) return false;
            gC = gates[GA_GAM + CH - 1];
            const float gm = gates[GA_GAM + t], lm = gates[GA_LAM + t], bt = gates[GA_BETA + t];
            const float ghi = gates[GA_HI + t], glo = gates[GA_LO + t];
            // <S, dS> of the block, H.V of the row
            {
                float x = 0.0f, y = 0.0f;
#pragma unroll 2
                for (int i = 0; i < 8; ++i)
                    dot8(x, y, *(const uint4 *)(sm + GS_S + 16 * (tid + i * G_VT)), *(const uint4 *)(sm + GS_DS + 16 * (tid + i * G_VT)));
                x = warp_sum(x + y);
                if (lane == 0) s_sum[warp] = x;
            }
            float db = 0.0f, row = 0.0f;
            if (krow) {
                float x = 0.0f;
#pragma unroll 2
                for (int j = 0; j < 8; ++j)
                    dot8(db, x, *(const uint4 *)(sm + GS_HO + half * TILE + swz(t, j)), *(const uint4 *)(sm + GS_V + half * (TILE / 2) + swz(t, j)));
                db += x;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(b_dot);
            // [K; Q] K^T and [H; dO] U^T, columns s = 32 half ..
            if (!wait_all(m_p, u.i)) return false;
            tc_fence_after();
            const int s0 = 32 * half;
            if (u.i > 0 && !wait_all(m_acc, u.i - 1)) return false;      // the head before has been read
            const float sc = krow ? -bt : 1.0f;
            const int last = t >= valid ? -1 : krow ? t - 1 : t;         // N is strictly lower, dPD has the diagonal
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {                // eight columns at a time: code that stays in the instruction cache
                const int c0 = s0 + 8 * c;
                float e8[8];
                uint32_t w[4] = {};
                if (c0 > 32 * (lq & 1) + 31) {           // the warp's rows all end before these columns
#pragma unroll
                    for (int e = 0; e < 8; ++e) e8[e] = 0.0f;
                } else {
                    uint32_t g8[8], x8[8];
                    tmem_ld8(at + TG_GRAM + c0, g8);
                    tmem_ld8(at + TG_DP + c0, x8);
                    float h[8], l[8];
                    ld4(gates + GA_HI + c0, *(float(*)[4])h);
                    ld4(gates + GA_HI + c0 + 4, *(float(*)[4])(h + 4));
                    ld4(gates + GA_LO + c0, *(float(*)[4])l);
                    ld4(gates + GA_LO + c0 + 4, *(float(*)[4])(l + 4));
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {     // e^((ghi - h) + (glo - l))
                        fma2(h[e], h[e + 1], h[e], h[e + 1], -1.0f, -1.0f, ghi, ghi);
                        fma2(l[e], l[e + 1], l[e], l[e + 1], -1.0f, -1.0f, glo, glo);
                        fma2(h[e], h[e + 1], h[e], h[e + 1], 1.0f, 1.0f, l[e], l[e + 1]);
                        h[e] = __expf(h[e]);
                        h[e + 1] = __expf(h[e + 1]);
                    }
                    tmem_wait_ld();
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float z = h[e] * __uint_as_float(x8[e]), zg = z * __uint_as_float(g8[e]);
                        const bool in = c0 + e <= last, off = in && c0 + e < t;      // s == t cancels in rows - columns
                        y[e] = in ? sc * z : 0.0f;
                        e8[e] = off ? sc * zg : 0.0f;
                        row += e8[e];
                        if (krow) db -= off ? zg : 0.0f;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(y[2 * e], y[2 * e + 1]);
                }
                *(uint4 *)(sm + GS_N + swz(L, 4 * half + c)) = make_uint4(w[0], w[1], w[2], w[3]);
                // column sums over the warp's 32 rows: lane l gets column c0 + l / 4
#pragma unroll
                for (int o = 4; o > 0; o >>= 1)
#pragma unroll
                    for (int e = 0; e < o; ++e) {
                        const bool up = lane & (4 * o);
                        const float mine = up ? e8[e + o] : e8[e], give = up ? e8[e] : e8[e + o];
                        e8[e] = mine + __shfl_xor_sync(0xffffffffu, give, 4 * o);
                    }
                e8[0] += __shfl_xor_sync(0xffffffffu, e8[0], 2);
                e8[0] += __shfl_xor_sync(0xffffffffu, e8[0], 1);
                if ((lane & 3) == 0) s_col[lq * 64 + c0 + (lane >> 2)] = e8[0];
            }
            fence_proxy_async();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_n);
            // [H; dO] S^T, then U dS^T (k rows): one piece of code for the two
#pragma unroll 1
            for (int ud = 0; ud < 2; ++ud) {
                if (!wait_all(ud ? m_ud : m_st, u.i)) return false;
                if (ud && !krow) break;
                tc_fence_after();
                const float sc = ud ? lm : krow ? -bt * gm : gm;
                float d = 0.0f, d1 = 0.0f;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t x[32];
                    tmem_ld32(at + (ud ? TG_UD : TG_ST) + 64 * half + 32 * hf, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 k4 = *(const uint4 *)(own + swz(L, 4 * hf + j));
                        const uint32_t kw[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float x0 = __uint_as_float(x[8 * j + 2 * i]), x1 = __uint_as_float(x[8 * j + 2 * i + 1]);
                            float *c = acc + 32 * hf + 8 * j + 2 * i;
                            fma2(d, d1, x0, x1, bf_lo(kw[i]), bf_hi(kw[i]), d, d1);
                            fma2(c[0], c[1], x0, x1, sc, sc, c[0], c[1]);
                        }
                    }
                }
                d += d1;
                if (ud) {
                    s_kud[half * 64 + t] = lm * d;
                    s_db[half * 64 + t] = db;
                } else {
                    row += sc * d;
                    if (krow) db -= gm * d;
                }
            }
            s_row[half * 128 + L] = row;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_d);
            return true;
        };
        for (Unit u = first(); u.w < nwork; u = next(u)) {
            const int hv = u.hk * rep + u.r, par = u.i & 1, row0 = u.row0, valid = u.valid;
            s_row = (float *)(sm + GS_ROW) + par * 256;
            s_kud = (float *)(sm + GS_KUD) + par * 128;
            s_db = (float *)(sm + GS_DB) + par * 128;
            s_col = (float *)(sm + GS_COL) + par * 256;
            s_sum = (float *)(sm + GS_SUM) + par * 8;
            ok = ok && head(u);
            named_bar_sync(1, G_VT);                     // by all warps, whatever their waits said
            if (!ok) continue;
            if (warp == 0) {
                float base = 0.0f, x[2], w[2];
                for (int i = 0; i < 8; ++i) base += s_sum[i];
                base *= gC;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = lane + 32 * i;
                    x[i] = (s_row[t] + s_row[128 + t]) + (s_row[64 + t] + s_row[192 + t]);
                    x[i] -= (s_col[t] + s_col[64 + t]) + (s_col[128 + t] + s_col[192 + t]);
                    w[i] = s_kud[t] + s_kud[64 + t];
                    if (t >= valid) x[i] = w[i] = 0.0f;
                }
                float lo, hi, wl, wh;
                sums_across(x[0], x[1], w[0], w[1], lo, hi, wl, wh, lane);
                __nv_bfloat16 *dg = (__nv_bfloat16 *)a.dg + (size_t)row0 * a.Hv + hv;
                if (lane < valid) dg[(size_t)lane * a.Hv] = __float2bfloat16_rn(base + wl + lo);
                if (lane + 32 < valid) dg[(size_t)(lane + 32) * a.Hv] = __float2bfloat16_rn(base + wh + hi);
            } else if (warp < 3) {
                const int t = 32 * (warp - 1) + lane;
                if (t < valid) ((__nv_bfloat16 *)a.dbeta)[(size_t)(row0 + t) * a.Hv + hv] = __float2bfloat16_rn(s_db[t] + s_db[64 + t]);
            }
            if (u.r + 1 < rep) continue;
            if (!(ok = wait_all(m_acc, u.i))) continue;
            tc_fence_after();
            __nv_bfloat16 *dst = (__nv_bfloat16 *)(krow ? a.dk_ : a.dq) + ((size_t)(row0 + t) * a.Hk + u.hk) * D + 64 * half;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t x[32];
                tmem_ld32(at + TG_ACC + 64 * half + 32 * hf, x);
                tmem_wait_ld();
                if (t < valid)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[i] = pack_bf16x2(acc[32 * hf + 8 * j + 2 * i] + __uint_as_float(x[8 * j + 2 * i]),
                                               acc[32 * hf + 8 * j + 2 * i + 1] + __uint_as_float(x[8 * j + 2 * i + 1]));
                        *(uint4 *)(dst + 32 * hf + 8 * j) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_out);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

cudaError_t launch_gdr_backward_tc(const GdrArgs &a, cudaStream_t s)
{
    struct TagR; struct TagG;
    TcP p;
    gdr_tc_plan(a, true, p);
    CUtensorMap mq{}, mk{}, mv{}, mo{};
    cudaError_t e = launch_gdr_prep_tc(p, mq, mk, mv, s);
    if (e != cudaSuccess) return e;
    if (a.T > 0 && !make_tile_map(&mo, a.dO, 1, a.T, a.Hv, CH)) return cudaErrorInvalidValue;
    if ((e = smem_opt_in<TagR>((const void *)gdr_walks_tc_kernel, W_KEEP_BYTES)) != cudaSuccess) return e;
    if ((e = launch_after(gdr_walks_tc_kernel, (unsigned)(a.N * a.Hv) * 2, W_THREADS, W_KEEP_BYTES, s, mq, mk, mv, mo, p)) != cudaSuccess)
        return e;
    if (a.T > 0) {
        if ((e = smem_opt_in<TagG>((const void *)gdr_grads_tc_kernel, GS_BYTES)) != cudaSuccess) return e;
        int dev = 0, sms = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        const long long work = gdr_slots(a.N, a.T) * a.Hk;
        return launch_after(gdr_grads_tc_kernel, (unsigned)(work < sms ? work : sms), G_THREADS, GS_BYTES, s, mq, mk, mv, mo, p);
    }
    return cudaSuccess;
}

}  // namespace kda
