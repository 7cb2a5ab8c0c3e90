// gdr.cuh — device helpers of the head-gated delta rule's kernels.
#pragma once

#include "common.cuh"
#include "gdr.h"

namespace kda {
namespace gdr {

constexpr int CH = 64;              // chunk length
constexpr int ERR_PAGE_INDEX = kErrPageIndex;

// Log-decays are clamped at -128 per token before they are summed: e^-128 is 0 in fp32, and so is
// every decay that contains it, so the clamp changes no result; it keeps differences of sums finite
// where a gate is -inf.  NaN stays NaN.
KDA_DEVICE float clamp_gate(float g) { return g < -128.0f ? -128.0f : g; }

// Rows of sequence n (offsets clamped into [0, T]; cu == null: N sequences of T / N tokens).
KDA_DEVICE SeqSpan span_of(const int *cu, int n, int N, int T)
{
    if (!cu) return SeqSpan{n * (T / N), T / N};
    return seq_span(cu, n, T);
}
// The first chunk slot of a sequence.
KDA_DEVICE int slot_base(int row0, int n) { return row0 / CH + n; }

// The sequence and chunk of a slot; false for a slot that no chunk has.  By whole warps: 32 sequences are
// looked at a time, so that a search is one round of loads for 32 sequences, two for 1024.
KDA_DEVICE bool find_slot(const int *cu, int N, int T, int slot, int &n, int &c, SeqSpan &span)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, len = N, step, k;    // the last sequence with slot_base <= slot is in [lo, lo + len)
    SeqSpan mine;
    do {
        step = (len + 31) / 32;
        const int i = lane * step;
        mine = span_of(cu, lo + min(i, len - 1), N, T);
        k = 31 - __clz(__ballot_sync(0xffffffffu, i < len && slot_base(mine.row0, lo + i) <= slot) | 1u);
        lo += k * step;
        len = min(step, len - k * step);
    } while (len > 1);
    n = lo;
    span.row0 = __shfl_sync(0xffffffffu, mine.row0, k);
    span.len = __shfl_sync(0xffffffffu, mine.len, k);
    c = slot - slot_base(span.row0, n);
    return c >= 0 && c * CH < span.len;
}

// Running sums of a chunk's 64 log-decays, by the first warp: G as hi + lo floats (the sum is
// formed in 64 bits, so a difference of two far sums keeps the bits of the gates between them).
KDA_DEVICE void gate_sums(const float *g, float *hi, float *lo, int lane)
{
    double a = (double)g[lane], b = (double)g[lane + 32];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double ya = __shfl_up_sync(0xffffffffu, a, o), yb = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) { a += ya; b += yb; }
    }
    b += __shfl_sync(0xffffffffu, a, 31);
    const float ah = (float)a, bh = (float)b;
    hi[lane] = ah;
    lo[lane] = (float)(a - (double)ah);
    hi[lane + 32] = bh;
    lo[lane + 32] = (float)(b - (double)bh);
}

// Of 64 rows (lane and lane + 32): inclusive suffix sums of r, exclusive prefix sums of w.  One warp.
KDA_DEVICE void sums_across(float r0, float r1, float w0, float w1, float &s0, float &s1, float &p0, float &p1, int lane)
{
    float a = w0, b = w1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float d0 = __shfl_down_sync(0xffffffffu, r0, o), d1 = __shfl_down_sync(0xffffffffu, r1, o);
        const float u0 = __shfl_up_sync(0xffffffffu, a, o), u1 = __shfl_up_sync(0xffffffffu, b, o);
        if (lane + o < 32) { r0 += d0; r1 += d1; }
        if (lane >= o) { a += u0; b += u1; }
    }
    s1 = r1;
    s0 = r0 + __shfl_sync(0xffffffffu, r1, 0);
    // exclusive: the sum up to the lane before (not a - w0, which would cancel where w0 is large)
    const float total = __shfl_sync(0xffffffffu, a, 31);
    const float x0 = __shfl_up_sync(0xffffffffu, a, 1), x1 = __shfl_up_sync(0xffffffffu, b, 1);
    p0 = lane ? x0 : 0.0f;
    p1 = total + (lane ? x1 : 0.0f);
}

// Page of sequence n: -1 where it has none (or the index is out of range, which sets the error word).
KDA_DEVICE int page_of(const int *index, int n, int pages, int *err)
{
    if (!index) return n;
    const int p = index[n];
    if (p >= pages) {
        raise_error(err, ERR_PAGE_INDEX);
        return -1;
    }
    return p < 0 ? -1 : p;
}

// Whether sequence n may write its final state to `page`: no earlier sequence writes there and, in
// the same buffer, no other sequence starts from there.  Called by all threads of a block.
KDA_DEVICE bool page_is_free(const int *sT_index, const int *s0_index, bool same_buffer, int n, int N, int page, int tid,
                             int nthreads)
{
    bool clash = false;
    for (int j = tid; j < N; j += nthreads) {
        if (sT_index && j < n && sT_index[j] == page) clash = true;
        if (same_buffer && j != n && (s0_index ? s0_index[j] : j) == page) clash = true;
    }
    return !__syncthreads_or(clash);
}

// M <- (I + A)^-1 for the strictly lower A, 64 x 64 in rows of LD floats: the 16 x 16 diagonal blocks
// by forward substitution (one column a thread: a product form such as (I - A)(I + A^2)... would cancel
// where keys repeat), then twice [[X, 0], [B, Y]]^-1 = [[X^-1, 0], [-Y^-1 B X^-1, Y^-1]] (16 -> 32 -> 64),
// every product in fp32.  A's upper right quarter is scratch.  256 threads; M's upper triangle is written
// as zeros.  Ends with a barrier.
template <int LD>
KDA_DEVICE void unit_lower_inverse(float *A, float *M, int tid)
{
    float *tmp = A + 32;   // rows 0..31, columns 32..63
    if (tid < 64) {
        const int b = tid >> 4, c = tid & 15;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float s[4] = {r == c ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = 0; m < r; m += 4) {
                float a[4];
                ld4(A + (16 * b + r) * LD + 16 * b + m, a);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (m + e < r) s[e] -= a[e] * x[m + e];
            }
            x[r] = (s[0] + s[1]) + (s[2] + s[3]);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) M[(16 * b + r) * LD + 16 * b + c] = x[r];
    } else {
        const float z[4] = {};
        for (int u = tid - 64; u < 6 * 64; u += 192) {   // blocks (0,1) (0,2) (0,3) (1,2) (1,3) (2,3)
            const int b = u >> 6, I = b < 3 ? 0 : b < 5 ? 1 : 2, J = b < 3 ? b + 1 : b < 5 ? b - 1 : 3;
            st4(M + (16 * I + ((u & 63) >> 2)) * LD + 16 * J + 4 * (u & 3), z);
        }
    }
    __syncthreads();
    {   // 16 -> 32, two pairs of blocks: two columns a thread
        const int o = 32 * (tid >> 7), r = (tid & 127) >> 3, c = 2 * (tid & 7);
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int m = 0; m < 16; m += 4) {
            float a[4];
            ld4(A + (o + 16 + r) * LD + o + m, a);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 b = *(const float2 *)(M + (o + m + e) * LD + o + c);
                s0 += a[e] * b.x;
                s1 += a[e] * b.y;
            }
        }
        float *t = tmp + (o >> 1) * LD;
        *(float2 *)(t + r * LD + c) = make_float2(s0, s1);
        __syncthreads();
        s0 = s1 = 0.0f;
#pragma unroll
        for (int m = 0; m < 16; m += 4) {
            float a[4];
            ld4(M + (o + 16 + r) * LD + o + 16 + m, a);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 b = *(const float2 *)(t + (m + e) * LD + c);
                s0 -= a[e] * b.x;
                s1 -= a[e] * b.y;
            }
        }
        *(float2 *)(M + (o + 16 + r) * LD + o + c) = make_float2(s0, s1);
    }
    __syncthreads();
    {   // 32 -> 64: four columns a thread
        const int r = tid >> 3, c = 4 * (tid & 7);
        float s[4] = {};
#pragma unroll 2
        for (int m = 0; m < 32; m += 4) {        // every lane at the same row of M: one wavefront a load, zeros included
            float a[4];
            ld4(A + (32 + r) * LD + m, a);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float b[4];
                ld4(M + (m + e) * LD + c, b);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] += a[e] * b[j];
            }
        }
        st4(tmp + r * LD + c, s);
        __syncthreads();
        float x[4] = {};
#pragma unroll 1
        for (int m = 0; m <= (r | 3); m += 4) {  // a warp has four rows
            float a[4];
            ld4(M + (32 + r) * LD + 32 + m, a);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float b[4];
                ld4(tmp + (m + e) * LD + c, b);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] -= a[e] * b[j];
            }
        }
        st4(M + (32 + r) * LD + c, x);
    }
    __syncthreads();
}

}  // namespace gdr
}  // namespace kda
