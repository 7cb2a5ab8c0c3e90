// gdr_tc.cu — the head-gated delta rule in chunks of 64 tokens on tcgen05 tensor cores (bf16,
// dk = dv = 128).  The formulas are those of gdr_simt.cu.
//
// prep, a block per chunk and value head: [K; Q] K^T in one M = 128 MMA (exact bf16 operands, fp32
//   sums), the decays, M = (I + A)^-1 and P M in fp32 on CUDA cores; M and P M go to the workspace as
//   one 128 x 64 operand [M; P M], split into bf16 hi + lo, in the 128-byte swizzle of the MMA's
//   operand tiles, so the walk brings it in with one bulk copy.
// walk, a block per sequence, value head and 64 or 128 state columns: three products a chunk, each
//   an M = 128 MMA with the 64 columns of a warpgroup as N:
//     D1 = [K; Q] S         rows 0..63: X = K S, rows 64..127: Q S
//     D2 = [M; P M] R       rows 0..63: U, rows 64..127: P U        (R = beta (V - gamma X))
//     D3 = K^T (lam U)      S <- gamma_C S + D3
//   K, Q enter as they are.  S, R, U and [M; P M] enter as bf16 hi + lo pairs (lo x lo left out), so
//   what one chunk hands to the next is good to about 2^-16.  S stays in fp32 registers (a thread has
//   one row of it); TMEM holds only the three products.  The B operands (S, R, U: k rows x 64 columns,
//   MN-major) share one 32 KB buffer, since each is written after the MMA that read the one before.
// A chunk is a chain: three MMAs, each between a read of TMEM, a few operations a value and a
// write of shared memory; what it costs is that chain's latency, so two warpgroups with 64 columns
// each work on the same tiles of K, Q and [M; P M] and fill each other's waits.
#include <cuda.h>

#include "gdr.cuh"
#include "tc_common.cuh"

namespace kda {
namespace {

using namespace gdr;
using namespace tc;

constexpr int D = 128;               // dk = dv
constexpr int N = 64;                // state columns of a warpgroup
constexpr int TILE = 128 * 128;      // bytes of 128 rows x 64 bf16

// workspace item of a chunk and value head
constexpr int IT_LO = TILE;          // [M; P M] hi at 0, lo here
constexpr int IT_GATES = 2 * TILE;   // floats: gamma, lam, beta, then G hi, G lo (64 each)
constexpr int IT_BYTES = IT_GATES + 2048;
constexpr int IT_WALK = IT_GATES + 768;   // what the walk reads

KDA_DEVICE void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// x -> bf16 hi and lo, two values a word
KDA_DEVICE void split2(float x0, float x1, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(x0, x1);
    const float2 h = unpack_bf16x2(hi);
    lo = pack_bf16x2(x0 - h.x, x1 - h.y);
}

struct TcP {
    GdrArgs a;
    uint8_t *items;
    __nv_bfloat16 *S, *U;    // kept for the gradients: [items, 128, 128], [items, 64, 128]
    unsigned long long wait_ns;
    int skip_load_chunk;
};

// What a block has in flight when a bounded wait has given up: every MMA of the issuing threads
// (one commit each on `drain`) and the loads that were issued but not waited for are let finish
// before shared and tensor memory are released.
constexpr unsigned long long DRAIN_NS = 2000000000ull;

// ---------------------------------------------------------------- prep
constexpr int LM = 68;
constexpr int PR_KQ = 0, PR_M = 0, PR_TMP = 64 * LM * 4;
constexpr int PR_A = 2 * TILE, PR_P = PR_A + 64 * LM * 4, PR_G = PR_P + 64 * LM * 4;
constexpr int PR_BYTES = PR_G + 6 * 256 + 64 + 1024;
static_assert(PR_TMP + 48 * LM * 4 <= 2 * TILE, "M and its scratch take K's and Q's place");

__global__ void __launch_bounds__(256, 3)
gdr_prep_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, TcP p)
{
    const GdrArgs &a = p.a;
    int n, c;
    SeqSpan span;
    if (!find_slot(a.cu, a.N, a.T, blockIdx.x, n, c, span)) return;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    float *A = (float *)(sm + PR_A), *Pm = (float *)(sm + PR_P), *M = (float *)(sm + PR_M), *tmp = (float *)(sm + PR_TMP);
    float *graw = (float *)(sm + PR_G), *ghi = graw + 64, *glo = ghi + 64, *beta = glo + 64;
    uint64_t *bars = (uint64_t *)(sm + PR_G + 6 * 256);   // tiles, MMA
    uint32_t *tslot = (uint32_t *)(bars + 2);
    volatile int *abort_flag = (volatile int *)(tslot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hv = blockIdx.y, hk = hv / (a.Hv / a.Hk);
    const int row0 = span.row0 + c * CH, valid = min(CH, span.len - c * CH);
    if (tid == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
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
    bool ok = true;
    if (tid == 0) {
        if (mbar_wait_bounded(&bars[0], 0, abort_flag, a.err, p.wait_ns)) {
            const uint32_t kq = smem_u32(sm + PR_KQ);
            constexpr uint32_t id = idesc_bf16(128, 64, false, false);
            for (int kk = 0; kk < 8; ++kk) {
                const uint32_t at = kq + (kk >> 2) * TILE + (kk & 3) * 32;
                mma_ss(tmem, sdesc(at, 16, 1024), sdesc(at, 16, 1024), id, kk > 0);
            }
            mma_commit(&bars[1]);
        }
    }
    float *gates = nullptr;
    uint8_t *item = p.items + ((size_t)blockIdx.x * a.Hv + hv) * IT_BYTES;
    gates = (float *)(item + IT_GATES);
    if (warp == 1) {
        gate_sums(graw, ghi, glo, lane);
        __syncwarp();
        for (int t = lane; t < CH; t += 32) {
            gates[t] = __expf(ghi[t]);
            gates[64 + t] = __expf((ghi[63] - ghi[t]) + (glo[63] - glo[t]));
            gates[128 + t] = beta[t];
            gates[192 + t] = ghi[t];
            gates[256 + t] = glo[t];
        }
    }
    if (tid == 0 && !*abort_flag) mbar_wait_bounded(&bars[1], 0, abort_flag, a.err, p.wait_ns);
    __syncthreads();
    ok = !*abort_flag;
    if (ok) {
        tc_fence_after();
        // thread: row r of [K; Q] K^T, 32 of its columns
        const int r = 32 * (warp & 3) + lane, t = r & 63, half = warp >> 2, s0 = 32 * half;
        float *dst = (r < 64 ? A : Pm) + t * LM + s0;
        const int last = t >= valid ? -1 : r < 64 ? t - 1 : t;   // A is strictly lower; rows behind the end may hold NaN
        if (s0 > 32 * (warp & 1) + 31) {       // the warp's rows all end before its columns
#pragma unroll
            for (int e = 0; e < 32; e += 4) *(float4 *)(dst + e) = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
            uint32_t x[32];
            tmem_ld32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + s0, x);
            tmem_wait_ld();
            const float gh = ghi[t], gl = glo[t], scale = r < 64 ? beta[t] : 1.0f;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                float y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int s = s0 + e + i;
                    const float d = __expf((gh - ghi[s]) + (gl - glo[s]));
                    y[i] = s <= last ? scale * d * __uint_as_float(x[e + i]) : 0.0f;
                }
                st4(dst + e, y);
            }
        }
        tc_fence_before();
    }
    __syncthreads();   // K and Q are consumed (the MMA is done)
    if (ok) {
        unit_lower_inverse<LM>(A, M, tmp, tid);
        // [M; P M] as hi + lo; P M's lower triangle: k runs from its column to its row
        const int ty = tid >> 4, tx = tid & 15;
        float pm[4][4] = {};
        if (tx <= ty)
            for (int k = 4 * tx; k < 4 * ty + 4; k += 4) {
                float x[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) ld4(Pm + (4 * ty + i) * LM + k, x[i]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float y[4];
                    ld4(M + (k + e) * LM + 4 * tx, y);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) pm[i][j] += x[i][e] * y[j];
                }
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * ty + i;
            const uint32_t off = swz(t, tx >> 1) + 8 * (tx & 1);
            float m[4];
            ld4(M + t * LM + 4 * tx, m);
            uint2 hi, lo;
            split2(m[0], m[1], hi.x, lo.x);
            split2(m[2], m[3], hi.y, lo.y);
            *(uint2 *)(item + off) = hi;
            *(uint2 *)(item + IT_LO + off) = lo;
            split2(pm[i][0], pm[i][1], hi.x, lo.x);
            split2(pm[i][2], pm[i][3], hi.y, lo.y);
            *(uint2 *)(item + TILE / 2 + off) = hi;
            *(uint2 *)(item + IT_LO + TILE / 2 + off) = lo;
        }
    } else if (tid == 0) {
        mbar_wait_timed(&bars[0], 0, DRAIN_NS);   // the tiles, if they are still on their way
        mma_commit(&bars[1]);
        mbar_wait_timed(&bars[1], 0, DRAIN_NS);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 64);
    }
}

// ---------------------------------------------------------------- the walk
// shared memory: two stages of {K; Q tiles 32 KB, [M; P M] hi + lo 32 KB, gates}, then a B operand
// buffer a warpgroup
constexpr int ST_KQ = 0, ST_MM = 2 * TILE, ST_BYTES = ST_MM + IT_GATES + 1024;
constexpr int STAGES = 2;
constexpr int OFF_B = STAGES * ST_BYTES, B_BYTES = 2 * TILE;   // 128 rows x 64 columns, hi then lo
template <int NWG> constexpr int walk_bar() { return OFF_B + NWG * B_BYTES; }
template <int NWG> constexpr int walk_bytes() { return walk_bar<NWG>() + 128 + 1024; }
static_assert(walk_bytes<2>() <= 232448, "shared memory per block");

// 8 values of a row -> the row's 16-byte pieces of a hi and a lo tile
KDA_DEVICE void put_split(uint8_t *hi, uint8_t *lo, int row, int j, const float (&x)[8])
{
    uint4 h, l;
    split2(x[0], x[1], h.x, l.x);
    split2(x[2], x[3], h.y, l.y);
    split2(x[4], x[5], h.z, l.z);
    split2(x[6], x[7], h.w, l.w);
    const uint32_t off = swz(row, j);
    *(uint4 *)(hi + off) = h;
    *(uint4 *)(lo + off) = l;
}
KDA_DEVICE uint4 pack8(const float (&x)[8])
{
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// K and Q rows behind a sequence's end (the next sequence's, or NaN) are zeroed before they meet the
// zeros of the other operand: the product of a zero and a NaN is not zero.
KDA_DEVICE void zero_tail(uint8_t *kq, int valid, int tid, int nthreads)
{
    for (int u = tid; u < (CH - valid) * 32; u += nthreads) {
        const int t = valid + (u >> 5), b = (u >> 3) & 3;   // b: channel block, then K or Q
        *(uint4 *)(kq + (b >> 1) * TILE + (b & 1) * (TILE / 2) + swz(t, u & 7)) = make_uint4(0u, 0u, 0u, 0u);
    }
}

template <int NWG, bool KEEP>
__global__ void __launch_bounds__(128 * NWG + 32, 1)
gdr_walk_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, TcP p)
{
    const GdrArgs &a = p.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint64_t *bars = (uint64_t *)(sm + walk_bar<NWG>());
    uint64_t *full = bars, *empty = bars + STAGES, *done = bars + 2 * STAGES, *drain = done + 3 * NWG;
    uint32_t *tslot = (uint32_t *)(drain + 1);
    volatile int *abort_flag = (volatile int *)(tslot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int GROUPS = 2 / NWG;      // blocks of a head
    const int n = blockIdx.x / GROUPS, hv = blockIdx.y, hk = hv / (a.Hv / a.Hk);
    const SeqSpan span = span_of(a.cu, n, a.N, a.T);
    const int nchunks = (span.len + CH - 1) / CH;
    const size_t item0 = (size_t)slot_base(span.row0, n);

    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], NWG + 4 * NWG);   // a commit a warpgroup, and its warps' reads of the gates
        }
        for (int i = 0; i < 3 * NWG; ++i) mbar_init(&done[i], 1);
        mbar_init(drain, NWG);
        *abort_flag = 0;
        fence_mbar_init();
        if (nchunks > 0) {
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
        }
    }
    if (warp == 0) {
        tmem_alloc(tslot, NWG == 2 ? 512 : 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;

    if (warp == 4 * NWG) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            int issued = 0, seen = 0;
            for (int ch = 0; ch < nchunks && !*abort_flag; ++ch) {
                const int st = ch % STAGES;
                if (ch >= STAGES && !mbar_wait_bounded(&empty[st], (uint32_t)((ch / STAGES - 1) & 1), abort_flag, a.err, p.wait_ns))
                    break;
                if (ch == p.skip_load_chunk) continue;   // injected failure: the wait for it runs out
                uint8_t *s = sm + st * ST_BYTES;
                mbar_arrive_expect_tx(&full[st], 2 * TILE + IT_WALK);
                const int row = span.row0 + ch * CH;
                for (int cb = 0; cb < 2; ++cb) {
                    tma_load_4d(s + ST_KQ + cb * TILE, &tm_k, cb * 64, hk, row, 0, &full[st]);
                    tma_load_4d(s + ST_KQ + cb * TILE + TILE / 2, &tm_q, cb * 64, hk, row, 0, &full[st]);
                }
                bulk_load(s + ST_MM, p.items + ((item0 + ch) * a.Hv + hv) * IT_BYTES, IT_WALK, &full[st]);
                issued = ch + 1;
            }
            // after an abort the loads of the last stages may still be on their way
            for (seen = issued > STAGES ? issued - STAGES : 0; seen < issued && *abort_flag; ++seen)
                if (seen != p.skip_load_chunk)
                    mbar_wait_timed(&full[seen % STAGES], (uint32_t)((seen / STAGES) & 1), DRAIN_NS);
        }
    } else {
        // ------------------------------------------------------------ a warpgroup and its 64 columns
        const int wg = warp >> 2, wt = tid & 127, lq = warp & 3;
        const int col0 = (NWG == 2 ? wg : (int)blockIdx.x % GROUPS) * N;
        const uint32_t lane_q = (uint32_t)(32 * lq) << 16;
        const uint32_t d1 = tmem + 192 * wg, d2 = d1 + 64, d3 = d1 + 128;
        uint8_t *B = sm + OFF_B + wg * B_BYTES;
        // one barrier a product: a warp that comes late must not find the phase it waits for gone by
        uint64_t *bar = &done[3 * wg];
        const bool leader = wt == 0;
        auto wait_mma = [&](int i, int ch) {
            mbar_wait_bounded(bar + i, (uint32_t)(ch & 1), abort_flag, a.err, p.wait_ns);
            tc_fence_after();
        };
        constexpr uint32_t id_b = idesc_bf16(128, N, false, true), id_tb = idesc_bf16(128, N, true, true);

        float S[N];                       // row wt of the state, this warpgroup's columns
        {
            const int page = a.s0 ? page_of(a.s0_index, n, a.pages, a.err) : -1;
            if (page >= 0) {
                const float *src = a.s0 + (((size_t)page * a.Hv + hv) * D + wt) * D + col0;
#pragma unroll
                for (int e = 0; e < N; e += 4) ld4(src + e, *(float(*)[4])(S + e));
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) S[e] = 0.0f;
            }
        }
        auto put_state = [&](int ch) {    // S -> hi + lo operand (and the copy kept for the gradients)
#pragma unroll
            for (int j = 0; j < N / 8; ++j) {
                const float(&x)[8] = *(const float(*)[8])(S + 8 * j);
                put_split(B, B + TILE, wt, j, x);
                if (KEEP && ch < nchunks)
                    *(uint4 *)(p.S + (((item0 + ch) * a.Hv + hv) * D + wt) * D + col0 + 8 * j) = pack8(x);
            }
            fence_proxy_async();
            tc_fence_before();
            named_bar_sync(1 + wg, 128);
        };
        if (nchunks > 0) put_state(0);

        for (int ch = 0; ch < nchunks; ++ch) {
            const int st = ch % STAGES;
            uint8_t *s = sm + st * ST_BYTES;
            const int valid = min(CH, span.len - ch * CH);
            const int t = wt & 63;        // rows 0..63 (warps 0, 1): X and U; 64..127 (warps 2, 3): the outputs
            const size_t tok = (size_t)span.row0 + ch * CH + t;
            mbar_wait_bounded(&full[st], (uint32_t)((ch / STAGES) & 1), abort_flag, a.err, p.wait_ns);
            const float *gates = (const float *)(s + ST_MM + IT_GATES);
            const float gam = gates[t], lam = gates[64 + t], bet = gates[128 + t], gC = gates[63];
            __syncwarp();
            if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(&empty[st])) : "memory");
            if (valid < CH) {             // uniform for the block
                zero_tail(s + ST_KQ, valid, tid, 128 * NWG);
                fence_proxy_async();
                named_bar_sync(3, 128 * NWG);
            }
            const uint32_t kq = smem_u32(s + ST_KQ), mm = smem_u32(s + ST_MM), b = smem_u32(B);
            if (leader && !*abort_flag) {
                tc_fence_after();
#pragma unroll
                for (int hl = 0; hl < 2; ++hl)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ss(d1, sdesc(kq + (kk >> 2) * TILE + (kk & 3) * 32, 16, 1024),
                               sdesc(b + hl * TILE + kk * 2048, 8192, 1024), id_b, hl | kk);
                mma_commit(bar + 0);
            }
            uint4 v[8];                   // V row, under the MMA
            if (lq < 2) {
                const uint4 *src = (const uint4 *)((const __nv_bfloat16 *)a.v + (tok * a.Hv + hv) * D + col0);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = t < valid ? src[j] : make_uint4(0u, 0u, 0u, 0u);
            }
            wait_mma(0, ch);
            if (lq < 2) {                 // R = beta (V - gamma X), zero behind the end
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t x[32];
                    tmem_ld32(d1 + lane_q + 32 * hf, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t w[4] = {v[4 * hf + j].x, v[4 * hf + j].y, v[4 * hf + j].z, v[4 * hf + j].w};
                        float r[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = unpack_bf16x2(w[e]);
                            r[2 * e] = t < valid ? bet * (f.x - gam * __uint_as_float(x[8 * j + 2 * e])) : 0.0f;
                            r[2 * e + 1] = t < valid ? bet * (f.y - gam * __uint_as_float(x[8 * j + 2 * e + 1])) : 0.0f;
                        }
                        put_split(B, B + TILE / 2, t, 4 * hf + j, r);
                    }
                }
                fence_proxy_async();
                tc_fence_before();
                named_bar_sync(4 + wg, 64);
                if (leader && !*abort_flag) {
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t ah = sdesc(mm + kk * 32, 16, 1024), al = sdesc(mm + IT_LO + kk * 32, 16, 1024);
                        const uint64_t bh = sdesc(b + kk * 2048, 8192, 1024), bl = sdesc(b + TILE / 2 + kk * 2048, 8192, 1024);
                        mma_ss(d2, ah, bh, id_b, kk);
                        mma_ss(d2, ah, bl, id_b, 1);
                        mma_ss(d2, al, bh, id_b, 1);
                    }
                    mma_commit(bar + 1);
                }
            }
            wait_mma(1, ch);
            if (lq < 2) {                 // lam U -> operand
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t x[32];
                    tmem_ld32(d2 + lane_q + 32 * hf, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float r[8];
                        if (KEEP) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) r[e] = __uint_as_float(x[8 * j + e]);
                            *(uint4 *)(p.U + (((item0 + ch) * a.Hv + hv) * CH + t) * D + col0 + 32 * hf + 8 * j) = pack8(r);
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) r[e] = lam * __uint_as_float(x[8 * j + e]);
                        put_split(B, B + TILE / 2, t, 4 * hf + j, r);
                    }
                }
                fence_proxy_async();
                tc_fence_before();
                named_bar_sync(4 + wg, 64);
                if (leader && !*abort_flag) {
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                        for (int hl = 0; hl < 2; ++hl)
                            mma_ss(d3, sdesc(kq + kk * 2048, TILE, 1024), sdesc(b + hl * (TILE / 2) + kk * 2048, 8192, 1024),
                                   id_tb, kk | hl);
                    mma_commit(bar + 2);
                    mma_commit(&empty[st]);
                }
            } else if (!KEEP) {           // outputs: gamma (Q S) + P U
                __nv_bfloat16 *dst = (__nv_bfloat16 *)a.out + (tok * a.Hv + hv) * D + col0;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t x[32], y[32];
                    tmem_ld32(d1 + lane_q + 32 * hf, y);
                    tmem_ld32(d2 + lane_q + 32 * hf, x);
                    tmem_wait_ld();
                    if (t < valid) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float r[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                r[e] = gam * __uint_as_float(y[8 * j + e]) + __uint_as_float(x[8 * j + e]);
                            *(uint4 *)(dst + 32 * hf + 8 * j) = pack8(r);
                        }
                    }
                }
            }
            wait_mma(2, ch);
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t x[32];
                tmem_ld32(d3 + lane_q + 32 * hf, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) S[32 * hf + e] = gC * S[32 * hf + e] + __uint_as_float(x[e]);
            }
            if (ch + 1 < nchunks) put_state(ch + 1);
        }

        if (!KEEP && a.sT) {
            const int page = page_of(a.sT_index, n, a.pages, a.err);
            bool keep = page >= 0 && !*abort_flag;
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
                float *dst = a.sT + (((size_t)page * a.Hv + hv) * D + wt) * D + col0;
#pragma unroll
                for (int e = 0; e < N; e += 4) st4(dst + e, *(const float(*)[4])(S + e));
            }
        }
        if (leader && *abort_flag) {
            mma_commit(drain);
            mbar_wait_timed(drain, 0u, DRAIN_NS);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, NWG == 2 ? 512 : 256);
    }
}

}  // namespace

bool gdr_tc_shape(int dk, int dv, IoType io) { return io == IO_BF16 && dk == D && dv == D; }
bool gdr_tc_available() { return device_is_sm100() && tensor_maps_available(); }

size_t gdr_tc_workspace(int N_, int T, int Hk, int Hv, bool backward)
{
    (void)Hk;
    const size_t items = (size_t)gdr_slots(N_, T) * Hv;
    return backward ? 0 : items * IT_BYTES;
}

cudaError_t launch_gdr_forward_tc(const GdrArgs &a, cudaStream_t s)
{
    struct TagP; struct Tag1; struct Tag2;
    const WaitHooks hk = wait_hooks();
    TcP p{a, (uint8_t *)a.ws, nullptr, nullptr, hk.wait_ns, hk.skip_load_chunk};
    CUtensorMap mq{}, mk{};
    cudaError_t e;
    if (a.T > 0) {
        if (!make_tile_map(&mq, a.q, 1, a.T, a.Hk, CH) || !make_tile_map(&mk, a.k, 1, a.T, a.Hk, CH)) return cudaErrorInvalidValue;
        if ((e = smem_opt_in<TagP>((const void *)gdr_prep_tc_kernel, PR_BYTES)) != cudaSuccess) return e;
        gdr_prep_tc_kernel<<<dim3((unsigned)gdr_slots(a.N, a.T), a.Hv), 256, PR_BYTES, s>>>(mq, mk, p);
    }
    // few heads: a block per 64 columns, so that twice as many SMs work
    if ((long long)a.N * a.Hv <= 74) {
        if ((e = smem_opt_in<Tag1>((const void *)gdr_walk_tc_kernel<1, false>, walk_bytes<1>())) != cudaSuccess) return e;
        gdr_walk_tc_kernel<1, false><<<dim3((unsigned)a.N * 2, a.Hv), 160, walk_bytes<1>(), s>>>(mq, mk, p);
    } else {
        if ((e = smem_opt_in<Tag2>((const void *)gdr_walk_tc_kernel<2, false>, walk_bytes<2>())) != cudaSuccess) return e;
        gdr_walk_tc_kernel<2, false><<<dim3((unsigned)a.N, a.Hv), 288, walk_bytes<2>(), s>>>(mq, mk, p);
    }
    return cudaGetLastError();
}

}  // namespace kda
