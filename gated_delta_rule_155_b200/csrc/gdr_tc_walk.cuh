// gdr_tc_walk.cuh — the walk along a sequence on tcgen05 tensor cores (bf16, dk = dv = 128): the forward
// pass's, and, leaving states and corrections instead of outputs, the backward pass's.
//
// A block per sequence and value head, everything transposed: the lanes of tensor memory are the
// 128 value columns, so what a chunk computes from the state is the A operand of the next product and
// never leaves tensor memory, and K, Q and [M; P M] are B operands as the copies brought them:
//   X^T  = S^T K^T       R^T = beta (V^T - gamma X^T)
//   U^T  = R^T M^T       S^T <- gamma_C S^T + (lam U)^T K
//   QS^T = S^T Q^T       O^T = gamma QS^T + R^T (P M)^T
// K, Q enter as they are.  S, R, lam U and [M; P M] enter as bf16 hi + lo pairs (lo x lo left out),
// so what one chunk hands to the next is good to about 2^-16; S itself stays in fp32.
// The chain S -> X -> R -> U -> S bounds a sequence: three products, three reads of tensor memory with a
// few operations a value, three writes.  Sixteen warps do that, a quarter of the columns each, and write
// the outputs under the state's product; one thread issues the MMAs, one the copies of the chunks to
// come.  An M = 128 MMA takes about max(54, N / 2) cycles, so X and Q S, and U and P U, are one product
// of N = 128 each: 36 MMAs a chunk.
// A chunk takes about 5900 cycles: the MMAs 3560, the vector phases 1500, six hand-offs 850.  4 x 8192 tokens of
// 96 heads (384 chains on 148 SMs): 1.20 ms; 8192 packed tokens of 32 heads, the longest 3001: 155 us.  A product
// of two narrower halves that overlapped the state's split, with 60 MMAs a chunk, took 1.42 ms against 1.29.
#pragma once

#include "gdr_tc.cuh"

namespace kda {
namespace gdr {

// Tensor memory columns: S (fp32), S as an operand (hi, lo), X then R, Q S, U, P U.
// KEEP: leaves each chunk's start state and U for the gradients, and writes no output and no final state
template <bool KEEP>
KDA_DEVICE void walk_forward(const CUtensorMap &tm_q, const CUtensorMap &tm_k, const CUtensorMap &tm_v, const TcP &p, unsigned block)
{
    constexpr int TM_S = 0, TM_SHL = 128, TM_X = 256, TM_QS = 320, TM_U = 384, TM_PU = 448;
    const GdrArgs &a = p.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t *full = (uint64_t *)(sm + W_BAR), *empty = full + STAGES;
    uint64_t *b_s = empty + STAGES, *b_r = b_s + 1, *b_u = b_s + 2;    // vector phases done
    uint64_t *m_x = b_s + 3, *m_u = b_s + 4, *m_s = b_s + 5;           // products done
    uint64_t *drain = b_s + 6;
    uint32_t *tslot = (uint32_t *)(drain + 1);
    volatile int *abort_flag = (volatile int *)(tslot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hv = p.head0 + (int)(block % p.heads), hk = hv / (a.Hv / a.Hk);
    const int n = p.order ? p.order[block / p.heads] : (int)(block / p.heads);
    SeqSpan span = span_of(a.cu, n, a.N, a.T);
    // a second walk has nothing to go on where the first has given up: no chunks, and no state to keep
    auto carried = [&]() -> int & { return p.carried[(size_t)n * a.Hv + hv]; };
    auto begun = [&]() { return p.chunk0 == 0 || carried(); };
    const int all = (span.len + CH - 1) / CH, first = min(p.chunk0, all), nchunks = begun() ? min(p.chunk1, all) - first : 0;
    const size_t item0 = (size_t)slot_base(span.row0, n) + first;
    span.row0 += first * CH;
    span.len -= first * CH;

    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1 + 16);
        }
        mbar_init(b_s, 16);
        mbar_init(b_r, 16);
        mbar_init(b_u, 16);
        mbar_init(m_x, 1);
        mbar_init(m_u, 1);
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
    auto wait = [&](uint64_t *bar, int i) { return mbar_wait_bounded(bar, (uint32_t)(i & 1), abort_flag, a.err, p.wait_ns); };
    // by a whole warp: one answer for all its lanes
    auto wait_all = [&](uint64_t *bar, int i) { return __all_sync(0xffffffffu, wait(bar, i)) != 0; };
    auto wait_full = [&](int ch) { return wait_all(&full[ch % STAGES], ch / STAGES); };

    if (warp == 16) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            int issued = 0;
            if (nchunks > 0) {
                prefetch_tmap(&tm_q);
                prefetch_tmap(&tm_k);
                prefetch_tmap(&tm_v);
            }
            for (int ch = 0; ch < nchunks && !*abort_flag; ++ch) {
                const int st = ch % STAGES;
                if (ch >= STAGES && !wait(&empty[st], ch / STAGES - 1)) break;
                if (first + ch == p.skip_load_chunk) continue;   // injected failure: the wait for it runs out
                uint8_t *s = sm + st * ST_BYTES;
                mbar_arrive_expect_tx(&full[st], 3 * TILE + IT_WALK);
                const int row = span.row0 + ch * CH;
                for (int cb = 0; cb < 2; ++cb) {
                    tma_load_4d(s + ST_KQ + cb * TILE, &tm_k, cb * 64, hk, row, 0, &full[st]);
                    tma_load_4d(s + ST_KQ + cb * TILE + TILE / 2, &tm_q, cb * 64, hk, row, 0, &full[st]);
                    tma_load_4d(s + ST_V + cb * (TILE / 2), &tm_v, cb * 64, hv, row, 0, &full[st]);
                }
                const uint8_t *item = p.items + ((item0 + ch) * a.Hv + hv) * IT_BYTES;
                bulk_load(s + ST_MM, item, IT_WALK, &full[st]);
                issued = ch + 1;
                // prep has given up on this chunk: so does the block (found here, where nothing waits for the answer: as a
                // branch of the chain's or the MMAs' warps it took 1 to 2 % of a walk)
                if (((const float *)(item + IT_GATES))[GA_GAM + CH - 1] < 0.0f) *abort_flag = 1;
            }
            // after an abort the loads of the last stages may still be on their way
            for (int seen = issued > STAGES ? issued - STAGES : 0; seen < issued && *abort_flag; ++seen)
                if (first + seen != p.skip_load_chunk)
                    mbar_wait_timed(&full[seen % STAGES], (uint32_t)((seen / STAGES) & 1), DRAIN_NS);
        }
        __syncwarp();
        if (!KEEP && a.sT) named_bar_arrive(1, 544);     // every chunk's mark has been looked at
    } else if (warp == 17) {
        // ------------------------------------------------------------ MMAs
        constexpr int NX = KEEP ? 64 : 128;      // X (and Q S), U (and P U)
        constexpr uint32_t id_x = idesc_bf16(128, NX, false, false), id_s = idesc_bf16(128, 128, false, true);
        auto keep_u = [&](int ch) {
            bulk_store(p.U + ((item0 + ch) * a.Hv + hv) * TILE, sm + W_KEEP_U, TILE);
            bulk_commit();
        };
        bool ok = true;
        for (int ch = 0; ch < nchunks && ok; ++ch) {
            uint8_t *s = sm + (ch % STAGES) * ST_BYTES;
            ok = wait_full(ch);
            const int valid = min(CH, span.len - ch * CH);
            if (valid < CH) {     // K rows behind the end (the next sequence's, or NaN) meet the zeros of U: zero
                for (int u = lane; u < (CH - valid) * 16; u += 32)
                    *(uint4 *)(s + ST_KQ + ((u >> 3) & 1) * TILE + swz(valid + (u >> 4), u & 7)) = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async();
                __syncwarp();
            }
            if (lane == 0) {
                const uint32_t kq = smem_u32(s + ST_KQ), mm = smem_u32(s + ST_MM);
                if (ok && (ok = wait(b_s, ch))) {                // S^T [K; Q]^T
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                        for (int hl = 0; hl < 2; ++hl)
                            mma_ts(tmem + TM_X, tmem + TM_SHL + 64 * hl + 8 * kk,
                                   sdesc(kq + (kk >> 2) * TILE + (kk & 3) * 32, 16, 1024), id_x, kk | hl);
                    mma_commit(m_x);
                    if (KEEP && ch > 0) keep_u(ch - 1);
                }
                if (ok && (ok = wait(b_r, ch))) {                // R^T [M; P M]^T
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t rh = tmem + TM_X + 16 * kk, rl = rh + 8;
                        const uint64_t bh = sdesc(mm + kk * 32, 16, 1024), bl = sdesc(mm + IT_LO + kk * 32, 16, 1024);
                        mma_ts(tmem + TM_U, rh, bh, id_x, kk);
                        mma_ts(tmem + TM_U, rl, bh, id_x, 1);
                        mma_ts(tmem + TM_U, rh, bl, id_x, 1);
                    }
                    if (KEEP) bulk_wait_read_all();              // U's tile may be written again
                    mma_commit(m_u);
                    if (KEEP) {
                        bulk_store(p.S + ((item0 + ch) * a.Hv + hv) * 2 * TILE, sm + W_KEEP_S, 2 * TILE);
                        bulk_commit();
                    }
                }
                if (ok && (ok = wait(b_u, ch))) {                // (lam U)^T K
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int hl = 0; hl < 2; ++hl)
                            mma_ts(tmem + TM_S, tmem + TM_X + 16 * kk + 8 * hl, sdesc(kq + kk * 2048, TILE, 1024), id_s, 1);
                    if (KEEP) bulk_wait_read_all();              // and S's
                    mma_commit(m_s);
                    mma_commit(&empty[ch % STAGES]);
                }
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0);
        }
        if (KEEP && lane == 0) {
            if (ok && nchunks > 0 && wait(b_s, nchunks)) keep_u(nchunks - 1);
            bulk_wait_read_all();
        }
        if (lane == 0 && *abort_flag) {
            mma_commit(drain);
            mbar_wait_timed(drain, 0u, DRAIN_NS);
        }
    } else {
        // ------------------------------------------------------------ the chain, and the outputs
        const int grp = warp >> 2, lq = warp & 3, dv = 32 * lq + lane;
        const uint32_t at = tmem + ((uint32_t)(32 * lq) << 16);
        const int r0 = 32 * grp, t0 = 16 * grp;      // the thread's state rows r0 .. + 31 and tokens t0 .. + 15 of column dv
        auto arrive = [&](uint64_t *bar) {           // after the writes to tensor memory
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        {
            const int page = a.s0 ? page_of(a.s0_index, n, a.pages, a.err) : -1;
            const float *src = a.s0 + (((size_t)max(page, 0) * a.Hv + hv) * D + r0) * D + dv;
            uint32_t x[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = page >= 0 ? __float_as_uint(src[(size_t)e * D]) : 0u;
            tmem_st32(at + TM_S + r0, x);
            tmem_wait_st();                          // each thread reads back what it wrote itself
        }
        bool ok = true;
        for (int ch = 0; ch < nchunks; ++ch) {
            const int st = ch % STAGES, valid = min(CH, span.len - ch * CH);
            uint8_t *s = sm + st * ST_BYTES;
            const float *gates = (const float *)(s + ST_G);
            if (ch > 0) {
                if (!(ok = wait_all(m_s, ch - 1))) break;
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
                if (KEEP) {                          // [dv][state row]
                    uint8_t *dst = sm + W_KEEP_S + (grp >> 1) * TILE;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *(uint4 *)(dst + swz(dv, 4 * (grp & 1) + j)) = make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]);
                    fence_proxy_async();
                }
            }
            if (!(ok = wait_full(ch))) break;
            {                                        // the state decayed, in the shadow of the product
                const float gC = gates[GA_GAM + CH - 1];
                float *x = (float *)S;
#pragma unroll
                for (int e = 0; e < 32; e += 2) mul2(x[e], x[e + 1], x[e], x[e + 1], gC, gC);
                tmem_st32(at + TM_S + r0, S);
            }
            // beta V^T: column dv of the thread's tokens
            float r[16], w[16];
            {
                const uint8_t *vt = s + ST_V + (dv >> 6) * (TILE / 2) + t0 * 128 + 2 * (dv & 7);
                const int j = (dv & 63) >> 3;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    float b4[4], c4[4];
                    ld4(gates + GA_BETA + t0 + e, b4);
                    ld4(gates + GA_BG + t0 + e, c4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        r[e + i] = __bfloat162float(*(const __nv_bfloat16 *)(vt + (e + i) * 128 + ((j ^ ((e + i) & 7)) << 4)));
                        w[e + i] = -c4[i];
                    }
                    mul2(r[e], r[e + 1], r[e], r[e + 1], b4[0], b4[1]);
                    mul2(r[e + 2], r[e + 3], r[e + 2], r[e + 3], b4[2], b4[3]);
                }
                if (valid < CH)                      // rows behind the end may hold NaN
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (t0 + e >= valid) r[e] = 0.0f;
            }
            if (!(ok = wait_all(m_x, ch))) break;
            tc_fence_after();
            {
                uint32_t x[16];
                tmem_ld16(at + TM_X + t0, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 2)
                    fma2(r[e], r[e + 1], w[e], w[e + 1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]), r[e], r[e + 1]);
                put_tokens(at + TM_X + t0, r);
            }
            arrive(b_r);
#pragma unroll
            for (int e = 0; e < 16; e += 4) ld4(gates + GA_LAM + t0 + e, *(float(*)[4])(w + e));
            if (!(ok = wait_all(m_u, ch))) break;
            tc_fence_after();
            {
                uint32_t x[16];
                tmem_ld16(at + TM_U + t0, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 2)
                    mul2(r[e], r[e + 1], w[e], w[e + 1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                put_tokens(at + TM_X + t0, r);       // R has been read: U's product is done
                arrive(b_u);
                if (KEEP) {                          // [dv][token]
                    uint8_t *dst = sm + W_KEEP_U;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t u[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            u[e] = pack_bf16x2(__uint_as_float(x[8 * j + 2 * e]), __uint_as_float(x[8 * j + 2 * e + 1]));
                        *(uint4 *)(dst + swz(dv, 2 * grp + j)) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                    fence_proxy_async();
                }
            }
            if (!KEEP) {                             // outputs, under the state's product
                uint32_t x[16], y[16];
                tmem_ld16(at + TM_QS + t0, x);
                tmem_ld16(at + TM_PU + t0, y);
                tmem_wait_ld();
                __nv_bfloat16 *dst = (__nv_bfloat16 *)a.out + (((size_t)span.row0 + ch * CH + t0) * a.Hv + hv) * D + dv;
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    float g4[4];
                    ld4(gates + GA_GAM + t0 + e, g4);
                    float o[4];
#pragma unroll
                    for (int i = 0; i < 4; i += 2)
                        fma2(o[i], o[i + 1], g4[i], g4[i + 1], __uint_as_float(x[e + i]), __uint_as_float(x[e + i + 1]),
                             __uint_as_float(y[e + i]), __uint_as_float(y[e + i + 1]));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (t0 + e + i < valid) dst[(size_t)((e + i) * a.Hv) * D] = __float2bfloat16_rn(o[i]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
        }
        if (KEEP && ok && nchunks > 0) arrive(b_s);  // the last U's tile is written
        if (!KEEP && a.sT) {
            if (nchunks > 0 && ok && (ok = wait_all(m_s, nchunks - 1))) tc_fence_after();
            const int page = page_of(a.sT_index, n, a.pages, a.err);
            named_bar_sync(1, 544);                  // all warps or none: a state is kept whole
            bool keep = page >= 0 && ok && begun() && !*abort_flag;
            if (page >= 0 && (a.sT_index || (p.start_index && a.sT == p.start))) {
                bool clash = false;       // as page_is_free, a warp at a time
                for (int j = lane; j < a.N; j += 32) {
                    if (a.sT_index && j < n && a.sT_index[j] == page) clash = true;
                    if (a.sT == p.start && j != n && (p.start_index ? p.start_index[j] : j) == page) clash = true;
                }
                if (__any_sync(0xffffffffu, clash)) {
                    keep = false;
                    raise_error(a.err, ERR_PAGE_INDEX);
                }
            }
            if (p.carried && p.chunk0 == 0 && tid == 0) carried() = keep;
            if (keep) {
                float *dst = a.sT + (((size_t)page * a.Hv + hv) * D + r0) * D + dv;
                uint32_t x[32];
                tmem_ld32(at + TM_S + r0, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) dst[(size_t)e * D] = __uint_as_float(x[e]);
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

}  // namespace gdr
}  // namespace kda
