// gdr_tc.cu — the head-gated delta rule in chunks of 64 tokens on tcgen05 tensor cores (bf16,
// dk = dv = 128): the forward pass.  The formulas are those of gdr_simt.cu.
//
// prep, a block per chunk and value head: [K; Q] K^T in one M = 128 MMA (exact bf16 operands, fp32
//   sums), the decays in fp32, M = (I + A)^-1 by substitution in blocks of 16 (fp32) and split tf32 products of
//   the blocks (2^-21), P M on tcgen05 from bf16 hi + lo pairs (lo x lo left out: 2^-16); M and P M go to the
//   workspace as one 128 x 64 operand [M; P M], split into bf16 hi + lo, in the 128-byte swizzle of the MMA's
//   operand tiles, so the walk brings it in with one bulk copy.  765 us for 49152 chunks and heads (4 x 8192
//   tokens of 96 heads), 75 us for 4224; shared memory bounds it (its data pipe is busy 78 % of the time).
// walk, a block per sequence and value head: gdr_tc_walk.cuh.
#include <algorithm>
#include <atomic>
#include <climits>

#include "gdr_tc_walk.cuh"

namespace kda {
namespace {

using namespace gdr;

// ---------------------------------------------------------------- prep
// Shared memory: K; Q tiles; once their product is done, P (hi, lo; later P M) and A (fp32; its inverse M in
// place; later M's hi, lo) in their place.  36 KB and 128 threads, so that six blocks share an SM: a block is a
// chain of short steps with a barrier behind each, and what one leaves idle the others use.
constexpr int LM = 68, PR_T = 128;
constexpr int SMS = 148;                   // of a B200; the plans of launches depend on it, no result does
constexpr int PR_KQ = 0, PR_P = 0, PR_A = TILE, PR_MHL = PR_A, PR_G = 33 * 1024 + 512;
constexpr int PR_BYTES = PR_G + 4 * 256 + 64 + 1024;
static_assert(PR_A + 64 * LM * 4 <= PR_G && PR_MHL + TILE <= PR_G && 2 * TILE <= PR_G && PR_BYTES + 1024 <= 228 * 1024 / 6, "regions");
static_assert(W_ALONE_BYTES + PR_BYTES > 228 * 1024 && W_ALONE_BYTES >= W_BYTES, "no prep beside a leading walk");

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

__global__ void __launch_bounds__(PR_T, 6)
gdr_prep_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, TcP p)
{
    if (!p.beside) follow();
    const GdrArgs &a = p.a;
    if (p.beside && blockIdx.y == gridDim.y - 1) {      // the end of this kernel is the end of all before it
        if (blockIdx.x == 0) follow();
        return;
    }
    if (p.order && blockIdx.y == gridDim.y - 1) {       // the blocks behind the heads: the sequences' order
        order_sequences(p, blockIdx.x * (PR_T / 32) + (threadIdx.x >> 5), gridDim.x * (PR_T / 32), threadIdx.x & 31);
        return;
    }
    int n, c, slot = blockIdx.x;
    SeqSpan span;
    if (!a.cu || a.N == 1) {                            // a sequence's chunks side by side
        const int per = gridDim.x / a.N;
        n = blockIdx.x / per;
        c = p.chunk0 + (int)(blockIdx.x % per);
        span = span_of(a.cu, n, a.N, a.T);
        slot = slot_base(span.row0, n) + c;
        if (c * CH >= span.len) return;
    } else if (!find_slot(a.cu, a.N, a.T, slot, n, c, span) || c < p.chunk0 || c >= p.chunk1) {
        return;
    }
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    float *A = (float *)(sm + PR_A);
    float *graw = (float *)(sm + PR_G), *ghi = graw + 64, *glo = ghi + 64, *beta = glo + 64;
    uint64_t *bars = (uint64_t *)(sm + PR_G + 4 * 256);   // tiles, [K; Q] K^T, P M
    uint32_t *tslot = (uint32_t *)(bars + 3);
    volatile int *abort_flag = (volatile int *)(tslot + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hv = p.head0 + blockIdx.y, hk = hv / (a.Hv / a.Hk);
    const int row0 = span.row0 + c * CH, valid = min(CH, span.len - c * CH);
    if (tid == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        mbar_init(&bars[2], 1);
        *abort_flag = 0;
        fence_mbar_init();
        if (c != p.skip_prep_chunk) {                  // else an injected failure: the wait for them runs out
            mbar_arrive_expect_tx(&bars[0], 2 * TILE);
            for (int cb = 0; cb < 2; ++cb) {
                tma_load_4d(sm + PR_KQ + cb * TILE, &tm_k, cb * 64, hk, row0, 0, &bars[0]);
                tma_load_4d(sm + PR_KQ + cb * TILE + TILE / 2, &tm_q, cb * 64, hk, row0, 0, &bars[0]);
            }
        }
    }
    if (warp == 0) {
        tmem_alloc(tslot, 64);
        tmem_relinquish();
    }
    if (tid >= 64) {
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
    uint8_t *item = p.items + ((size_t)slot * a.Hv + hv) * IT_BYTES;
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
    const int t = tid & 63;                    // row of [K; Q] K^T in the thread's lane of tensor memory
    const uint32_t at = tmem + ((uint32_t)(32 * warp) << 16);
    if (ok) {
        tc_fence_after();
        const bool krow = tid < 64;
        const int last = t >= valid ? -1 : krow ? t - 1 : t;     // A is strictly lower; rows behind the end may hold NaN
        const float gh = ghi[t], gl = glo[t], scale = krow ? beta[t] : 1.0f;
#pragma unroll 1
        for (int c0 = 0; c0 < 64; c0 += 8) {   // eight columns at a time: the instruction cache bounds this kernel
            float y[8] = {};
            if (c0 <= 32 * (warp & 1) + 31) {  // else the warp's rows all end before these columns
                uint32_t x[8];
                tmem_ld8(at + c0, x);
                float h[8], l[8];
                ld4(ghi + c0, *(float(*)[4])h);
                ld4(ghi + c0 + 4, *(float(*)[4])(h + 4));
                ld4(glo + c0, *(float(*)[4])l);
                ld4(glo + c0 + 4, *(float(*)[4])(l + 4));
#pragma unroll
                for (int e = 0; e < 8; e += 2) {       // e^((gh - h) + (gl - l))
                    fma2(h[e], h[e + 1], h[e], h[e + 1], -1.0f, -1.0f, gh, gh);
                    fma2(l[e], l[e + 1], l[e], l[e + 1], -1.0f, -1.0f, gl, gl);
                    fma2(h[e], h[e + 1], h[e], h[e + 1], 1.0f, 1.0f, l[e], l[e + 1]);
                    h[e] = __expf(h[e]);
                    h[e + 1] = __expf(h[e + 1]);
                    mul2(h[e], h[e + 1], h[e], h[e + 1], scale, scale);
                }
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    mul2(y[e], y[e + 1], h[e], h[e + 1], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                    if (c0 + e > last) y[e] = 0.0f;
                    if (c0 + e + 1 > last) y[e + 1] = 0.0f;
                }
            }
            if (krow) {
                st4(A + t * LM + c0, *(const float(*)[4])y);
                st4(A + t * LM + c0 + 4, *(const float(*)[4])(y + 4));
            } else {
                put_split(sm + PR_P, sm + PR_P + TILE / 2, t, c0 / 8, y);
            }
        }
        fence_proxy_async();
        tc_fence_before();
        if (krow) named_bar_sync(1, 64);       // A is there: the inverse's diagonal blocks (these warps) need no P
        unit_lower_inverse<LM, PR_T / 32>(A, tid);
        // M as hi + lo over itself: a thread has half a row
        const int q = 4 * (tid >> 6);
        float y[4][8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            ld4(A + t * LM + 8 * (q + j), *(float(*)[4])y[j]);
            ld4(A + t * LM + 8 * (q + j) + 4, *(float(*)[4])(y[j] + 4));
        }
        __syncthreads();
        if (t < 32 && q)                       // scratch of the inverse
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) y[j][e] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) put_split(sm + PR_MHL, sm + PR_MHL + TILE / 2, t, q + j, y[j]);
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
        if (tid < 64) {
#pragma unroll 1
            for (int c0 = 0; c0 < 64; c0 += 8) {      // over P, which has been read
                uint32_t x[8];
                tmem_ld8(at + c0, x);
                tmem_wait_ld();
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(x[e]);
                put_split(sm + PR_P, sm + PR_P + TILE / 2, t, c0 / 8, y);
            }
            fence_proxy_async();
        }
    } else if (tid == 0) {
        gates[GA_GAM + CH - 1] = -1.0f;           // no decay is negative: the walks stop at this chunk
        if (c != p.skip_prep_chunk) mbar_wait_timed(&bars[0], 0, DRAIN_NS);   // the tiles, if they are still on their way
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
template <bool LEADS>
__global__ void __launch_bounds__(W_THREADS, 1)
gdr_walk_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, TcP p)
{
    follow();
    if (LEADS) come();                       // the next prep's blocks may
    walk_forward<false>(tm_q, tm_k, tm_v, p, blockIdx.x);
}

}  // namespace

bool gdr_tc_shape(int dk, int dv, IoType io) { return io == IO_BF16 && dk == D && dv == D; }
bool gdr_tc_available() { return device_is_sm100() && tensor_maps_available(); }

// Walks that leave SMs idle: how many chunks of every sequence (of the mean length) to walk before the others are
// prepared, which then runs beside them on the idle SMs; that takes about as long as those walks if prep costs
// 1 / 205 of a walk's step a chunk and head on all SMs (15.6 ns, 3.2 us).  2 x 4096 tokens of 32 heads 233 us (263
// in one prep and one walk), 32768 of 32 heads 1587 (1773), 4096 of 16 heads 210 (216); fewer than 600 chunks and
// heads to prepare beside are not worth two launches more (512 tokens of 64 heads, 320: 51 us against 44; 1024 of 32
// heads, 416: 71 against 67).  The states in between are fp32, so the parts give the bits of the whole.  0: all
// chunks in one prep and one walk.
static int early_chunks(int N, int T, int Hv)
{
    const long long walks = (long long)N * Hv, idle = SMS - walks, chunks = (T / N + CH - 1) / CH;
    if (idle <= 0) return 0;
    const long long early = (chunks * walks * SMS) / (205 * idle + walks * SMS) + 1;
    return (chunks - early) * walks >= 600 ? (int)early : 0;
}

// items; then 1 KB aligned: for the gradients S, U, dS, H, or the states between two walks and their marks; the
// sequences' order
size_t gdr_tc_workspace(int N, int T, int Hk, int Hv, bool backward)
{
    (void)Hk;
    const size_t items = (size_t)gdr_slots(N, T) * Hv;
    // whether they are used or not, so that a workspace of the most sequences and tokens does for fewer
    const size_t carry = backward ? 0 : (size_t)std::min<long long>((long long)N * Hv, SMS) * (D * D + 1) * 4;
    return items * (IT_BYTES + (backward ? 6 * TILE : 0)) + carry + 4 * (size_t)N;
}

static std::atomic<int> g_skip_prep_chunk{-1};
void set_gdr_prep_hook(int skip_chunk) { g_skip_prep_chunk.store(skip_chunk); }

void gdr_tc_plan(const GdrArgs &a, bool backward, TcP &p)
{
    const WaitHooks hk = wait_hooks();
    const size_t items = (size_t)gdr_slots(a.N, a.T) * a.Hv;
    p = TcP{};
    p.a = a;
    p.heads = a.Hv;
    p.chunk1 = INT_MAX;
    p.start = a.s0;
    p.start_index = a.s0_index;
    p.items = (uint8_t *)a.ws;
    uint8_t *at = p.items + items * IT_BYTES;
    if (backward) {
        p.S = at; at += items * 2 * TILE;
        p.dS = at; at += items * 2 * TILE;
        p.U = at; at += items * TILE;
        p.H = at; at += items * TILE;
    } else if (early_chunks(a.N, a.T, a.Hv)) {
        p.carry = (float *)at;
        at += (size_t)a.N * a.Hv * D * D * 4;
        p.carried = (int *)at;
        at += (size_t)a.N * a.Hv * 4;
    }
    if (a.T > 0 && a.cu && a.N > 1) p.order = (int *)at;
    p.wait_ns = hk.wait_ns;
    p.skip_load_chunk = hk.skip_load_chunk;
    p.skip_prep_chunk = g_skip_prep_chunk.load();
}

cudaError_t launch_gdr_prep_tc(const TcP &p, CUtensorMap &mq, CUtensorMap &mk, CUtensorMap &mv, cudaStream_t s)
{
    struct TagP;
    const GdrArgs &a = p.a;
    cudaError_t e;
    if (a.T > 0) {
        if (!make_tile_map(&mq, a.q, 1, a.T, a.Hk, CH) || !make_tile_map(&mk, a.k, 1, a.T, a.Hk, CH) ||
            !make_tile_map(&mv, a.v, 1, a.T, a.Hv, CH))
            return cudaErrorInvalidValue;
        if ((e = smem_opt_in<TagP>((const void *)gdr_prep_tc_kernel, PR_BYTES)) != cudaSuccess) return e;
        const long long per = std::min<long long>(p.chunk1, ((a.cu ? a.T : a.T / a.N) + CH - 1) / CH) - p.chunk0;
        const unsigned slots = (unsigned)(!a.cu || a.N == 1 ? a.N * per : gdr_slots(a.N, a.T));
        return launch_after(gdr_prep_tc_kernel, dim3(slots, p.heads + (p.order || p.beside ? 1 : 0)), PR_T, PR_BYTES, s, mq, mk, p);
    }
    return cudaSuccess;
}

// Sequences of one length whose walks fill the SMs more than once but not evenly: the value heads that walk first,
// few enough to leave SMs idle, so many that the others' walks fill the SMs evenly.  The others' prep runs beside them
// on the idle SMs (not before, and not on the idle SMs of the last round, when nothing is left to do).  4 x 8192
// tokens of 96 heads 2000 us (2090 in one prep and one walk), 2 x 4096 of 96 heads 500 (577), 2 x 512 of 96 heads 79
// (88); where the idle SMs have fewer than 400 chunks' time, two launches more cost what it gives (2 x 128 of 96
// heads 34.5 against 33.6).  Packed sequences: their lengths are on the device only; launches that decide there which
// of them has work gave 4 x 8192 packed tokens of 96 heads 1 % and cost lengths that differ 5 %.  0: all heads in
// one prep and one walk, as in the backward pass, whose longer reverse and shorter forward walks fill the SMs better
// (2 x 4096 tokens of 48 heads 775 us, 813 in two parts).
static int leading_heads(const GdrArgs &a)
{
    const long long walks = (long long)a.N * a.Hv;
    if ((a.cu && a.N > 1) || walks <= SMS || walks % SMS == 0) return 0;
    const long long lead = (walks % SMS + a.N - 1) / a.N, idle = SMS - lead * a.N, chunks = (a.T / a.N + CH - 1) / CH;
    return lead < a.Hv && idle > 0 && chunks * idle >= 400 ? (int)lead : 0;
}

cudaError_t launch_gdr_forward_tc(const GdrArgs &a, cudaStream_t s)
{
    struct TagW; struct TagL;
    TcP p;
    CUtensorMap mq{}, mk{}, mv{};
    gdr_tc_plan(a, false, p);
    cudaError_t e;
    const int lead = leading_heads(a), early = early_chunks(a.N, a.T, a.Hv);
    if (lead || early) {
        if (lead) p.heads = lead;
        if (early) {
            p.chunk1 = early;
            p.a.sT = p.carry;
            p.a.sT_index = nullptr;
            p.start = nullptr;
        }
        if ((e = launch_gdr_prep_tc(p, mq, mk, mv, s)) != cudaSuccess) return e;
        if ((e = smem_opt_in<TagL>((const void *)gdr_walk_tc_kernel<true>, W_ALONE_BYTES)) != cudaSuccess) return e;
        e = launch_after(gdr_walk_tc_kernel<true>, (unsigned)(a.N * p.heads), W_THREADS, W_ALONE_BYTES, s, mq, mk, mv, p);
        if (e != cudaSuccess) return e;
        if (lead) {
            p.head0 = lead;
            p.heads = a.Hv - lead;
        }
        if (early) {
            p.a = a;
            p.a.s0 = p.carry;
            p.a.s0_index = nullptr;
            p.start = a.s0;
            p.chunk0 = early;
            p.chunk1 = INT_MAX;
        }
        p.beside = true;
    }
    if ((e = launch_gdr_prep_tc(p, mq, mk, mv, s)) != cudaSuccess) return e;
    if ((e = smem_opt_in<TagW>((const void *)gdr_walk_tc_kernel<false>, W_BYTES)) != cudaSuccess) return e;
    return launch_after(gdr_walk_tc_kernel<false>, (unsigned)(a.N * p.heads), W_THREADS, W_BYTES, s, mq, mk, mv, p);
}

}  // namespace kda
