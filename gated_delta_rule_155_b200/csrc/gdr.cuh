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

// The sequence and chunk of a slot; false for a slot that no chunk has.
KDA_DEVICE bool find_slot(const int *cu, int N, int T, int slot, int &n, int &c, SeqSpan &span)
{
    int lo = 0, hi = N - 1;
    while (lo < hi) {   // last n with slot_base <= slot
        const int mid = (lo + hi + 1) >> 1;
        if (slot_base(span_of(cu, mid, N, T).row0, mid) <= slot) lo = mid;
        else hi = mid - 1;
    }
    n = lo;
    span = span_of(cu, n, N, T);
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

// M <- (I + A)^-1 for the strictly lower A, 64 x 64 in rows of LD floats, by 16 x 16 blocks:
// the diagonal blocks by forward substitution (one column a thread), then block row by block row
// M_IJ = -M_II sum_{J <= K < I} A_IK M_KJ, every product in fp32, four columns of one row a thread
// (one 16-byte load of A feeds four of M, 16 FMAs).  `tmp`: 48 rows of LD floats.  256 threads; M's
// upper triangle is written as zeros.  Ends with a barrier.
template <int LD>
KDA_DEVICE void unit_lower_inverse(const float *A, float *M, float *tmp, int tid)
{
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
    }
    {
        const int r = tid >> 4, c = tid & 15;
#pragma unroll
        for (int I = 0; I < 4; ++I)
#pragma unroll
            for (int J = I + 1; J < 4; ++J) M[(16 * I + r) * LD + 16 * J + c] = 0.0f;
    }
    __syncthreads();
    const int J = tid >> 6, r = (tid & 63) >> 2, c = 4 * (tid & 3);
#pragma unroll
    for (int I = 1; I < 4; ++I) {
        if (J < I) {
            float s[4] = {};
            for (int m = 16 * J; m < 16 * I; m += 4) {
                float a[4];
                ld4(A + (16 * I + r) * LD + m, a);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float b[4];
                    ld4(M + (m + e) * LD + 16 * J + c, b);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[j] += a[e] * b[j];
                }
            }
            st4(tmp + (16 * J + r) * LD + c, s);
        }
        __syncthreads();
        if (J < I) {
            float s[4] = {};
#pragma unroll
            for (int m = 0; m < 16; m += 4) {
                float a[4];
                ld4(M + (16 * I + r) * LD + 16 * I + m, a);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float b[4];
                    ld4(tmp + (16 * J + m + e) * LD + c, b);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[j] -= a[e] * b[j];
                }
            }
            st4(M + (16 * I + r) * LD + 16 * J + c, s);
        }
        __syncthreads();
    }
}

}  // namespace gdr
}  // namespace kda
