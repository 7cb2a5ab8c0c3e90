// gdr.cuh — device helpers of the head-gated delta rule's kernels.
#pragma once

#include "common.cuh"
#include "gdr.h"

namespace kda {
namespace gdr {

// Launches fn behind what is on the stream, its blocks brought up while that ends (see follow).
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*fn)(Params...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, const Args &...args)
{
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

constexpr int CH = 64;              // chunk length
constexpr int ERR_PAGE_INDEX = kErrPageIndex;

// Log-decays are clamped at -128 per token before they are summed: e^-128 is 0 in fp32, and so is
// every decay that contains it, so the clamp changes no result; it keeps differences of sums finite
// where a gate is -inf.  NaN stays NaN.
KDA_DEVICE float clamp_gate(float g) { return g < -128.0f ? -128.0f : g; }

// The first words of every kernel here, launched by launch_after: it may be on the GPU before the kernel it follows
// has ended, and goes no further until that one's writes can be seen.  Every block waits, those with nothing
// to do too, so that the end of a kernel is the end of all before it.
KDA_DEVICE void follow() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel come before this one's end; only for work that is to run beside it: blocks placed among those
// of a running kernel end up unevenly, and the walks lost more by that than an earlier start gave (8192 tokens
// backward 529 us against 513).
KDA_DEVICE void come() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Two fp32 operations an instruction (kernels that are short of issue slots, not of arithmetic).
KDA_DEVICE void fma2(float &d0, float &d1, float a0, float a1, float b0, float b1, float c0, float c1)
{
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
KDA_DEVICE void mul2(float &d0, float &d1, float a0, float a1, float b0, float b1)
{
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

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
    if (p >= pages || p < -1) {
        raise_error(err, ERR_PAGE_INDEX);
        return -1;
    }
    return p;
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

// c += A B, k in [k0, k1), for an A of 16 rows (of lda floats) and a B of 8 columns (rows of ldb), one warp: tf32 products
// of hi and lo parts (hi: the upper 11 bits, exact; lo x lo left out), so good to about 2^-21 of the terms.
// Lane l has rows l / 4 and l / 4 + 8 of columns 2 (l % 4) and the next.  A 16-byte load from shared memory
// costs four cycles however many lanes share its address, so products of 16 x 16 blocks on CUDA cores (20
// loads for 64 FMAs) spent four times the cycles that these fragments do.
KDA_DEVICE void mma_block(float (&c)[4], int k0, int k1, const float *A, int lda, const float *B, int ldb, int lane)
{
    const float *a = A + (lane >> 2) * lda + (lane & 3), *b = B + (lane & 3) * ldb + (lane >> 2);
#pragma unroll 2
    for (int k = k0; k < k1; k += 8) {
        const float x[4] = {a[k], a[8 * lda + k], a[k + 4], a[8 * lda + k + 4]}, y[2] = {b[k * ldb], b[(k + 4) * ldb]};
        uint32_t xh[4], xl[4], yh[2], yl[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            xh[i] = __float_as_uint(x[i]) & 0xffffe000u;
            xl[i] = __float_as_uint(x[i] - __uint_as_float(xh[i]));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            yh[i] = __float_as_uint(y[i]) & 0xffffe000u;
            yl[i] = __float_as_uint(y[i] - __uint_as_float(yh[i]));
        }
        auto mma = [&](const uint32_t (&p)[4], const uint32_t (&q)[2]) {
            asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                : "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3]), "r"(q[0]), "r"(q[1]));
        };
        mma(xl, yh);
        mma(xh, yl);
        mma(xh, yh);
    }
}
KDA_DEVICE void put_block(float *dst, int ld, const float (&c)[4], float sign, int lane)
{
    float *d = dst + (lane >> 2) * ld + 2 * (lane & 3);
    *(float2 *)d = make_float2(sign * c[0], sign * c[1]);
    *(float2 *)(d + 8 * ld) = make_float2(sign * c[2], sign * c[3]);
}

// A <- (I + A)^-1 for the strictly lower A, 64 x 64 in rows of LD floats, in place: the 16 x 16 diagonal
// blocks by forward substitution (one column a thread: a product form such as (I - A)(I + A^2)... would
// cancel where keys repeat), then twice [[X, 0], [B, Y]]^-1 = [[X^-1, 0], [-Y^-1 B X^-1, Y^-1]] (16 -> 32 -> 64)
// with mma_block's products.  Rows 0..31 of columns 32.. are scratch, and hold no zeros behind it.  W warps,
// at least four.  Ends with a barrier.
template <int LD, int W>
KDA_DEVICE void unit_lower_inverse(float *A, int tid)
{
    const int w = tid >> 5, lane = tid & 31;
    float *tmp = A + 32;   // rows 0..31, columns 32..63
    if (tid < 64) {
        const int b = tid >> 4, c = tid & 15;
        float *D = A + 16 * b * (LD + 1);
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float s[4] = {r == c ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = 0; m < r; m += 4) {
                float a[4];
                ld4(D + r * LD + m, a);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (m + e < r) s[e] -= a[e] * x[m + e];
            }
            x[r] = (s[0] + s[1]) + (s[2] + s[3]);
        }
        __syncwarp();      // both blocks of the warp have been read
#pragma unroll
        for (int r = 0; r < 16; ++r) D[r * LD + c] = x[r];
    }
    __syncthreads();
    {   // 16 -> 32: two pairs of blocks, eight columns a warp
        const int o = 32 * (w >> 1), n = 8 * (w & 1);
        if (w < 4) {
            float c[4] = {};
            mma_block(c, n, 16, A + (o + 16) * LD + o, LD, A + o * LD + o + n, LD, lane);
            put_block(tmp + (o >> 1) * LD + n, LD, c, 1.0f, lane);
        }
        __syncthreads();
        if (w < 4) {
            float c[4] = {};
            mma_block(c, 0, 16, A + (o + 16) * LD + o + 16, LD, tmp + (o >> 1) * LD + n, LD, lane);
            put_block(A + (o + 16) * LD + o + n, LD, c, -1.0f, lane);
        }
    }
    __syncthreads();
    // 32 -> 64: eight tiles of sixteen rows and eight columns
#pragma unroll
    for (int i = w; i < 8; i += W) {
        const int m = 16 * (i >> 2), n = 8 * (i & 3);
        float c[4] = {};
        mma_block(c, n, 32, A + (32 + m) * LD, LD, A + n, LD, lane);            // lower
        put_block(tmp + m * LD + n, LD, c, 1.0f, lane);
    }
    __syncthreads();
#pragma unroll
    for (int i = w; i < 8; i += W) {
        const int m = 16 * (i >> 2), n = 8 * (i & 3);
        float x[4] = {};
        mma_block(x, 0, m + 16, A + (32 + m) * LD + 32, LD, tmp + n, LD, lane);
        put_block(A + (32 + m) * LD + n, LD, x, -1.0f, lane);
    }
    __syncthreads();
}

}  // namespace gdr
}  // namespace kda
