// gdr_tc.cuh — layouts and helpers shared by the tensor-core kernels of the head-gated delta rule.
#pragma once

#include <cuda.h>

#include "gdr.cuh"
#include "tc_common.cuh"

namespace kda {
namespace gdr {

using namespace tc;

constexpr int D = 128;               // dk = dv
constexpr int TILE = 128 * 128;      // bytes of 128 rows x 64 bf16

// workspace item of a chunk and value head: [M; P M] as a 128-row operand tile, hi at 0, lo at IT_LO,
// then gates, 64 floats each: gamma, lam, beta, beta gamma, G hi, G lo
constexpr int IT_LO = TILE;
constexpr int IT_GATES = 2 * TILE;
constexpr int IT_BYTES = IT_GATES + 2048;
constexpr int IT_WALK = IT_GATES + 1024;   // what the walks read
enum { GA_GAM = 0, GA_LAM = 64, GA_BETA = 128, GA_BG = 192, GA_HI = 256, GA_LO = 320 };

struct TcP {
    GdrArgs a;
    uint8_t *items;
    int *order;              // sequences by length, longest first (null: as they are)
    float *carry;            // the states between two walks of the forward pass
    int *carried;            // whether the first of them left one: [N, Hv] (null: no two walks)
    uint8_t *S, *U, *dS, *H; // kept for the gradients, operand tiles of 2, 1, 2 and 1 TILE bytes an item
    int head0, heads;        // the value heads of a launch of prep and forward walk
    int chunk0, chunk1;      // and its chunks of every sequence
    const float *start;      // what the caller's sequences start from, for a walk that starts from another's states
    const int *start_index;
    bool beside;             // prep: beside the walk before it in the stream
    unsigned long long wait_ns;
    int skip_load_chunk, skip_prep_chunk;   // injected failures: of the walks, of prep (-1: none)
};

KDA_DEVICE void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
KDA_DEVICE void bulk_store(void *dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}
KDA_DEVICE void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// named_bar_sync for warps that need not wait
KDA_DEVICE void named_bar_arrive(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// x -> bf16 hi and lo, two values a word
KDA_DEVICE void split2(float x0, float x1, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(x0, x1);
    float l0, l1;
    fma2(l0, l1, __uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u), -1.0f, -1.0f, x0, x1);
    lo = pack_bf16x2(l0, l1);
}

// find_slot for a chunk's first row and its rows: {row, rows}, rows 0 for a slot that no chunk has (out of
// line: where it is called from four places, the instruction cache bounds the kernel)
static __device__ __noinline__ int2 slot_rows(const int *cu, int N, int T, int slot)
{
    int n, c;
    SeqSpan span;
    if (!find_slot(cu, N, T, slot, n, c, span)) return make_int2(0, 0);
    return make_int2(span.row0 + c * CH, min(CH, span.len - c * CH));
}

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

// What a block has in flight when a bounded wait has given up (MMAs, by one commit of the thread that
// issues them; loads that were issued but not waited for) is let finish before its memory is released.
constexpr unsigned long long DRAIN_NS = 2000000000ull;

// The walks' shared memory: stages of {K; Q tiles 32 KB, V (backward: dO) tiles 16 KB, [M; P M] hi + lo
// 32 KB, gates 1 KB}.
constexpr int ST_KQ = 0, ST_V = 2 * TILE, ST_MM = ST_V + TILE, ST_G = ST_MM + IT_GATES, ST_BYTES = ST_G + 1024;
constexpr int STAGES = 2;
constexpr int W_BAR = STAGES * ST_BYTES, W_BYTES = W_BAR + 256 + 1024;
constexpr int W_ALONE_BYTES = 200 * 1024;   // of a walk that no block of prep fits beside (it would wait for tensor memory)
// and, in the backward pass, what goes to the workspace: the state's tile (32 KB) and U's or H's (16 KB), each
// stored by one bulk copy (as 16-byte pieces of 128-byte rows from the registers the walks took a fifth longer)
constexpr int W_KEEP_S = W_BAR + 1024, W_KEEP_U = W_KEEP_S + 2 * TILE, W_KEEP_BYTES = W_KEEP_U + TILE + 1024;
static_assert(W_KEEP_BYTES <= 232448, "shared memory per block");
// Their warps: 4 g .. 4 g + 3, g < 4: tokens 16 g .. and state rows 32 g .. of the chain; 16 the copies, 17 the MMAs.
constexpr int W_THREADS = 576;

// 16 values of a lane (tokens of an A operand's step) as hi + lo words at `to`
KDA_DEVICE void put_tokens(uint32_t to, const float (&x)[16])
{
    uint32_t h[8], l[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) split2(x[2 * e], x[2 * e + 1], h[e], l[e]);
    tmem_st8(to, h);
    tmem_st8(to + 8, l);
}

}  // namespace gdr

// Lays out a call's workspace; makes the maps of q, k and v, and launches prep (nothing of both at T = 0).
void gdr_tc_plan(const GdrArgs &a, bool backward, gdr::TcP &p);
cudaError_t launch_gdr_prep_tc(const gdr::TcP &p, CUtensorMap &mq, CUtensorMap &mk, CUtensorMap &mv, cudaStream_t s);

}  // namespace kda
