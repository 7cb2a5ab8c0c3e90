// gdr_tc.cu — the head-gated delta rule in chunks of 64 tokens on tcgen05 tensor cores (bf16,
// dk = dv = 128): the forward pass.  The formulas are those of gdr_simt.cu.
//
// prep, a block per chunk and value head: [K; Q] K^T in one M = 128 MMA (exact bf16 operands, fp32
//   sums), the decays, M = (I + A)^-1 and P M in fp32 on CUDA cores; M and P M go to the workspace as
//   one 128 x 64 operand [M; P M], split into bf16 hi + lo, in the 128-byte swizzle of the MMA's
//   operand tiles, so the walk brings it in with one bulk copy.
// walk, a block per sequence and value head, everything transposed: the lanes of tensor memory are the
//   128 value columns, so what a chunk computes from the state is the A operand of the next product and
//   never leaves tensor memory, and K, Q and [M; P M] are B operands as the copies brought them:
//     X^T  = S^T K^T       R^T = beta (V^T - gamma X^T)
//     U^T  = R^T M^T       S^T <- gamma_C S^T + (lam U)^T K
//     QS^T = S^T Q^T       O^T = gamma QS^T + R^T (P M)^T
//   K, Q enter as they are.  S, R, lam U and [M; P M] enter as bf16 hi + lo pairs (lo x lo left out),
//   so what one chunk hands to the next is good to about 2^-16; S itself stays in fp32.
// The chain S -> X -> R -> U -> S bounds a sequence: three products, three reads of tensor memory with a
// few operations a value, three writes.  Sixteen warps do that, a quarter of the columns each, and write
// the outputs under the state's product; one thread issues the MMAs, one the copies of the chunks to
// come.  An M = 128 MMA takes about max(54, N / 2) cycles, so X and Q S, and U and P U, are one product
// of N = 128 each: 36 MMAs a chunk.
#include "gdr_tc.cuh"

namespace kda {
namespace {

using namespace gdr;

// ---------------------------------------------------------------- prep
// Shared memory: K; Q tiles; once their product is done, P (hi, lo; later P M) and M (fp32) in their
// place.  A (fp32), later M (hi, lo).  53 KB, so that four blocks share an SM.
constexpr int LM = 68;
constexpr int PR_KQ = 0, PR_P = 0, PR_M = TILE, PR_A = 33 * 1024, PR_MHL = PR_A, PR_G = PR_A + 64 * LM * 4;
constexpr int PR_BYTES = PR_G + 4 * 256 + 64 + 1024;
static_assert(PR_M + 64 * LM * 4 <= PR_A && PR_MHL + TILE <= PR_G && PR_BYTES <= 57344, "regions");

// order[r] <- the sequence whose length is the r-th longest: the walks start with the longest.  A warp a sequence.
KDA_DEVICE void order_sequences(const TcP &p, int first, int step, int lane)
{
    const GdrArgs &a = p.a;
    for (int n = first; n < a.N; n += step) {
        const int len = span_of(a.cu, n, a.N, a.T).len;
        int before = 0;
        for (int j = lane; j < a.N; j += 32) {
            const int l = span_of(a.cu, j, a.N, a.T).len;
            before += l > len || (l == len && j < n);
        }
        before = __reduce_add_sync(0xffffffffu, before);
        if (lane == 0) p.order[before] = n;
    }
}

__global__ void __launch_bounds__(256, 4)
gdr_prep_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, TcP p)
{
    const GdrArgs &a = p.a;
    if (p.order && blockIdx.y == gridDim.y - 1) {       // the blocks behind the heads: the sequences' order
        order_sequences(p, blockIdx.x * (256 / 32) + (threadIdx.x >> 5), gridDim.x * (256 / 32), threadIdx.x & 31);
        return;
    }
    int n, c;
    SeqSpan span;
    if (!find_slot(a.cu, a.N, a.T, blockIdx.x, n, c, span)) return;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    float *A = (float *)(sm + PR_A), *M = (float *)(sm + PR_M);
    float *graw = (float *)(sm + PR_G), *ghi = graw + 64, *glo = ghi + 64, *beta = glo + 64;
    uint64_t *bars = (uint64_t *)(sm + PR_G + 4 * 256);   // tiles, [K; Q] K^T, P M
    uint32_t *tslot = (uint32_t *)(bars + 3);
    volatile int *abort_flag = (volatile int *)(tslot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hv = blockIdx.y, hk = hv / (a.Hv / a.Hk);
    const int row0 = span.row0 + c * CH, valid = min(CH, span.len - c * CH);
    if (tid == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        mbar_init(&bars[2], 1);
        *abort_flag = 0;
        fence_mbar_init();
        mbar_arrive_expect_tx(&bars[0], 2 * TILE);
        for (int cb = 0; cb < 2; ++cb) {
            tma_load_4d(sm + PR_KQ + cb * TILE, &tm_k, cb * 64, hk, row0, 0, &bars[0]);
            tma_load_4d(sm + PR_KQ + cb * TILE + TILE / 2, &tm_q, cb * 64, hk, row0, 0, &bars[0]);
        }
    }
    if (warp == 0) {
        tmem_alloc(tslot, 64);
        tmem_relinquish();
    }
    if (tid >= 64 && tid < 128) {
        const int t = tid - 64;
        const size_t at = (size_t)(row0 + t) * a.Hv + hv;
        graw[t] = t < valid ? clamp_gate(__bfloat162float(((const __nv_bfloat16 *)a.g)[at])) : 0.0f;
        beta[t] = t < valid ? __bfloat162float(((const __nv_bfloat16 *)a.beta)[at]) : 0.0f;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    if (tid == 0) {
        if (mbar_wait_bounded(&bars[0], 0, abort_flag, a.err, p.wait_ns)) {
            const uint32_t kq = smem_u32(sm + PR_KQ);
            constexpr uint32_t id = idesc_bf16(128, 64, false, false);
#pragma unroll 2
            for (int kk = 0; kk < 8; ++kk) {
                const uint32_t at = kq + (kk >> 2) * TILE + (kk & 3) * 32;
                mma_ss(tmem, sdesc(at, 16, 1024), sdesc(at, 16, 1024), id, kk > 0);
            }
            mma_commit(&bars[1]);
        }
    }
    uint8_t *item = p.items + ((size_t)blockIdx.x * a.Hv + hv) * IT_BYTES;
    float *gates = (float *)(item + IT_GATES);
    if (warp == 1) {
        gate_sums(graw, ghi, glo, lane);
        __syncwarp();
        for (int t = lane; t < CH; t += 32) {
            const float gm = __expf(ghi[t]);
            gates[GA_GAM + t] = gm;
            gates[GA_LAM + t] = __expf((ghi[63] - ghi[t]) + (glo[63] - glo[t]));
            gates[GA_BETA + t] = beta[t];
            gates[GA_BG + t] = beta[t] * gm;
            gates[GA_HI + t] = ghi[t];
            gates[GA_LO + t] = glo[t];
        }
    }
    if (tid == 0 && !*abort_flag) mbar_wait_bounded(&bars[1], 0, abort_flag, a.err, p.wait_ns);
    __syncthreads();
    bool ok = !*abort_flag;
    const int lq = warp & 3, r = 32 * lq + lane, half = warp >> 2, s0 = 32 * half;   // lane of tensor memory, 32 of its columns
    const uint32_t at = tmem + ((uint32_t)(32 * lq) << 16) + s0;
    if (ok) {
        tc_fence_after();
        const int t = r & 63;
        const int last = t >= valid ? -1 : r < 64 ? t - 1 : t;   // A is strictly lower; rows behind the end may hold NaN
        const float gh = ghi[t], gl = glo[t], scale = r < 64 ? beta[t] : 1.0f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {          // eight columns at a time: the instruction cache bounds this kernel
            const int c0 = s0 + 8 * c;
            float y[8] = {};
            if (c0 <= 32 * (lq & 1) + 31) {    // else the warp's rows all end before these columns
                uint32_t x[8];
                tmem_ld8(at + 8 * c, x);
                float h[8], l[8];
                ld4(ghi + c0, *(float(*)[4])h);
                ld4(ghi + c0 + 4, *(float(*)[4])(h + 4));
                ld4(glo + c0, *(float(*)[4])l);
                ld4(glo + c0 + 4, *(float(*)[4])(l + 4));
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = scale * __expf((gh - h[e]) + (gl - l[e]));
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = c0 + e <= last ? h[e] * __uint_as_float(x[e]) : 0.0f;
            }
            if (r < 64) {
                st4(A + t * LM + c0, *(const float(*)[4])y);
                st4(A + t * LM + c0 + 4, *(const float(*)[4])(y + 4));
            } else {
                put_split(sm + PR_P, sm + PR_P + TILE / 2, t, c0 / 8, y);
            }
        }
        fence_proxy_async();
        tc_fence_before();
    }
    __syncthreads();
    if (ok) {
        unit_lower_inverse<LM>(A, M, tid);
        {                                      // M as hi + lo
            const int t = tid >> 2;
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
                float y[8];
                const int q8 = (tid & 3) + 4 * j;      // a quarter of a warp reads 8 different bank groups
                ld4(M + t * LM + 8 * q8, *(float(*)[4])y);
                ld4(M + t * LM + 8 * q8 + 4, *(float(*)[4])(y + 4));
                put_split(sm + PR_MHL, sm + PR_MHL + TILE / 2, t, q8, y);
            }
        }
        fence_proxy_async();
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && ok) {                      // P M, rows 64.. of A (M) give lanes that are not read
        tc_fence_after();
        const uint32_t pp = smem_u32(sm + PR_P), mm = smem_u32(sm + PR_MHL);
        constexpr uint32_t id = idesc_bf16(128, 64, false, true);
#pragma unroll 1
        for (int kk = 0; kk < 4; ++kk) {
            const uint64_t ph = sdesc(pp + kk * 32, 16, 1024), pl = sdesc(pp + TILE / 2 + kk * 32, 16, 1024);
            const uint64_t mh = sdesc(mm + kk * 2048, TILE / 2, 1024), ml = sdesc(mm + TILE / 2 + kk * 2048, TILE / 2, 1024);
            mma_ss(tmem, ph, mh, id, kk > 0);
            mma_ss(tmem, pl, mh, id, 1);
            mma_ss(tmem, ph, ml, id, 1);
        }
        mma_commit(&bars[2]);
        mbar_wait_bounded(&bars[2], 0, abort_flag, a.err, p.wait_ns);
    }
    __syncthreads();
    ok = ok && !*abort_flag;
    if (ok) {
        tc_fence_after();
        if (r < 64) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {      // over P, which has been read
                uint32_t x[8];
                tmem_ld8(at + 8 * c, x);
                tmem_wait_ld();
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(x[e]);
                put_split(sm + PR_P, sm + PR_P + TILE / 2, r, 4 * half + c, y);
            }
            fence_proxy_async();
        }
    } else if (tid == 0) {
        mbar_wait_timed(&bars[0], 0, DRAIN_NS);   // the tiles, if they are still on their way
        mma_commit(&bars[1]);
        mbar_wait_timed(&bars[1], 0, DRAIN_NS);
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 32 && ok) {
        bulk_store(item, sm + PR_MHL, TILE / 2);
        bulk_store(item + TILE / 2, sm + PR_P, TILE / 2);
        bulk_store(item + IT_LO, sm + PR_MHL + TILE / 2, TILE / 2);
        bulk_store(item + IT_LO + TILE / 2, sm + PR_P + TILE / 2, TILE / 2);
        bulk_commit();
        bulk_wait_read_all();
    }
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 64);
    }
}

// ---------------------------------------------------------------- the walk
// tensor memory columns: S (fp32), S as an operand (hi, lo), X then R, Q S, U, P U
constexpr int TM_S = 0, TM_SHL = 128, TM_X = 256, TM_QS = 320, TM_U = 384, TM_PU = 448;

// KEEP: leaves each chunk's start state and U for the gradients, and writes no output and no final state
template <bool KEEP>
__global__ void __launch_bounds__(W_THREADS, 1)
gdr_walk_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, TcP p)
{
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
    const int hv = blockIdx.x % a.Hv, hk = hv / (a.Hv / a.Hk);
    const int n = p.order ? p.order[blockIdx.x / a.Hv] : blockIdx.x / a.Hv;
    const SeqSpan span = span_of(a.cu, n, a.N, a.T);
    const int nchunks = (span.len + CH - 1) / CH;
    const size_t item0 = (size_t)slot_base(span.row0, n);

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
                if (ch == p.skip_load_chunk) continue;   // injected failure: the wait for it runs out
                uint8_t *s = sm + st * ST_BYTES;
                mbar_arrive_expect_tx(&full[st], 3 * TILE + IT_WALK);
                const int row = span.row0 + ch * CH;
                for (int cb = 0; cb < 2; ++cb) {
                    tma_load_4d(s + ST_KQ + cb * TILE, &tm_k, cb * 64, hk, row, 0, &full[st]);
                    tma_load_4d(s + ST_KQ + cb * TILE + TILE / 2, &tm_q, cb * 64, hk, row, 0, &full[st]);
                    tma_load_4d(s + ST_V + cb * (TILE / 2), &tm_v, cb * 64, hv, row, 0, &full[st]);
                }
                bulk_load(s + ST_MM, p.items + ((item0 + ch) * a.Hv + hv) * IT_BYTES, IT_WALK, &full[st]);
                issued = ch + 1;
            }
            // after an abort the loads of the last stages may still be on their way
            for (int seen = issued > STAGES ? issued - STAGES : 0; seen < issued && *abort_flag; ++seen)
                if (seen != p.skip_load_chunk)
                    mbar_wait_timed(&full[seen % STAGES], (uint32_t)((seen / STAGES) & 1), DRAIN_NS);
        }
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
#pragma unroll
                for (int e = 0; e < 32; ++e) S[e] = __float_as_uint(gC * __uint_as_float(S[e]));
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
                        const float f = __bfloat162float(*(const __nv_bfloat16 *)(vt + (e + i) * 128 + ((j ^ ((e + i) & 7)) << 4)));
                        r[e + i] = t0 + e + i < valid ? b4[i] * f : 0.0f;
                        w[e + i] = c4[i];
                    }
                }
            }
            if (!(ok = wait_all(m_x, ch))) break;
            tc_fence_after();
            {
                uint32_t x[16];
                tmem_ld16(at + TM_X + t0, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) r[e] -= w[e] * __uint_as_float(x[e]);
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
                for (int e = 0; e < 16; ++e) r[e] = w[e] * __uint_as_float(x[e]);
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
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (t0 + e + i < valid)
                            dst[(size_t)((e + i) * a.Hv) * D] =
                                __float2bfloat16_rn(g4[i] * __uint_as_float(x[e + i]) + __uint_as_float(y[e + i]));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
        }
        if (KEEP && ok && nchunks > 0) arrive(b_s);  // the last U's tile is written
        if (!KEEP && a.sT) {
            if (nchunks > 0 && ok && (ok = wait_all(m_s, nchunks - 1))) tc_fence_after();
            const int page = page_of(a.sT_index, n, a.pages, a.err);
            bool keep = page >= 0 && ok;
            if (page >= 0 && (a.sT_index || (a.s0_index && a.sT == a.s0))) {
                bool clash = false;       // as page_is_free, a warp at a time
                for (int j = lane; j < a.N; j += 32) {
                    if (a.sT_index && j < n && a.sT_index[j] == page) clash = true;
                    if (a.sT == a.s0 && j != n && (a.s0_index ? a.s0_index[j] : j) == page) clash = true;
                }
                if (__any_sync(0xffffffffu, clash)) {
                    keep = false;
                    raise_error(a.err, ERR_PAGE_INDEX);
                }
            }
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

}  // namespace

bool gdr_tc_shape(int dk, int dv, IoType io) { return io == IO_BF16 && dk == D && dv == D; }
bool gdr_tc_available() { return device_is_sm100() && tensor_maps_available(); }

// items; then 1 KB aligned: for the gradients S, U, dS, H; the sequences' order
size_t gdr_tc_workspace(int N, int T, int Hk, int Hv, bool backward)
{
    (void)Hk;
    const size_t items = (size_t)gdr_slots(N, T) * Hv;
    return items * (IT_BYTES + (backward ? 6 * TILE : 0)) + 4 * (size_t)N;
}

void gdr_tc_plan(const GdrArgs &a, bool backward, TcP &p)
{
    const WaitHooks hk = wait_hooks();
    const size_t items = (size_t)gdr_slots(a.N, a.T) * a.Hv;
    p = TcP{};
    p.a = a;
    p.items = (uint8_t *)a.ws;
    uint8_t *at = p.items + items * IT_BYTES;
    if (backward) {
        p.S = at; at += items * 2 * TILE;
        p.dS = at; at += items * 2 * TILE;
        p.U = at; at += items * TILE;
        p.H = at; at += items * TILE;
    }
    if (a.T > 0 && a.cu && a.N > 1) p.order = (int *)at;
    p.wait_ns = hk.wait_ns;
    p.skip_load_chunk = hk.skip_load_chunk;
}

cudaError_t launch_gdr_prep_walk_tc(const TcP &p, bool keep, cudaStream_t s)
{
    struct TagP; struct TagW; struct TagK;
    const GdrArgs &a = p.a;
    CUtensorMap mq{}, mk{}, mv{};
    cudaError_t e;
    if (a.T > 0) {
        if (!make_tile_map(&mq, a.q, 1, a.T, a.Hk, CH) || !make_tile_map(&mk, a.k, 1, a.T, a.Hk, CH) ||
            !make_tile_map(&mv, a.v, 1, a.T, a.Hv, CH))
            return cudaErrorInvalidValue;
        if ((e = smem_opt_in<TagP>((const void *)gdr_prep_tc_kernel, PR_BYTES)) != cudaSuccess) return e;
        gdr_prep_tc_kernel<<<dim3((unsigned)gdr_slots(a.N, a.T), a.Hv + (p.order ? 1 : 0)), 256, PR_BYTES, s>>>(mq, mk, p);
    }
    const unsigned blocks = (unsigned)(a.N * a.Hv);
    if (keep) {
        if ((e = smem_opt_in<TagK>((const void *)gdr_walk_tc_kernel<true>, W_KEEP_BYTES)) != cudaSuccess) return e;
        gdr_walk_tc_kernel<true><<<blocks, W_THREADS, W_KEEP_BYTES, s>>>(mq, mk, mv, p);
    } else {
        if ((e = smem_opt_in<TagW>((const void *)gdr_walk_tc_kernel<false>, W_BYTES)) != cudaSuccess) return e;
        gdr_walk_tc_kernel<false><<<blocks, W_THREADS, W_BYTES, s>>>(mq, mk, mv, p);
    }
    return cudaGetLastError();
}

cudaError_t launch_gdr_forward_tc(const GdrArgs &a, cudaStream_t s)
{
    TcP p;
    gdr_tc_plan(a, false, p);
    return launch_gdr_prep_walk_tc(p, false, s);
}

}  // namespace kda
