// gdr_decode.cu — the head-gated delta rule token by token, on pages of a state cache
// (memory-bound: one read and one write of each state, however many tokens it takes).
//
// Per sequence, value head and token, with S the dk x dv fp32 state and alpha = e^g:
//     a = alpha S^T k;   b = alpha S^T q;   u = beta (v - a);   S <- alpha S + k u^T;   o = b + (q.k) u
// so both column sums come from one pass over the state before its update.
// The columns of S never mix: a warp has sixteen of them and needs no other.  Four lanes take a row's 64
// bytes, lane l the dk / 8 consecutive rows from (l / 4) dk / 8 on, so its k and q are vector loads; all
// the state's loads go out before anything is waited for (8 KB a warp, 128 KB an SM), and the column sums
// are shuffles.  A block is four warps (64 columns).  Bound by HBM: 250 sequences of 32 heads (1.05 GB)
// in 164 us, 6.4 TB/s; five drafted tokens of 37 sequences (158 MB) 43.5 us.
// When it was chosen, against its own 162 and 39 us in the same measurement: a block per head with sums over
// its warps in shared memory, three barriers a token: 276 and 82 us; eight columns a warp (32-byte pieces of
// rows): 211 and 63 us; three blocks an SM instead of four: 171 and 47 us; the next token's vectors loaded
// ahead into registers: 170 and 49 us.
#include "gdr.cuh"

namespace kda {
namespace {

using namespace gdr;

constexpr int NT = 128, LPR = 4, MINB = 4, COLS = NT / 32 * 4 * LPR;   // threads, lanes of a row, columns of a block

// R consecutive elements
template <int R>
KDA_DEVICE void load_vec(const float *p, float (&x)[R])
{
#pragma unroll
    for (int e = 0; e < R; e += 4) ld4(p + e, *(float(*)[4])(x + e));
}
template <int R>
KDA_DEVICE void load_vec(const __nv_bfloat16 *p, float (&x)[R])
{
    static_assert(R % 8 == 0, "16-byte loads");
    uint32_t w[R / 2];
#pragma unroll
    for (int e = 0; e < R / 2; e += 4) *(uint4 *)(w + e) = *(const uint4 *)(p + 2 * e);
#pragma unroll
    for (int e = 0; e < R / 2; ++e) {
        x[2 * e] = __uint_as_float(w[e] << 16);
        x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
}

template <typename IO, int DK>
__global__ void __launch_bounds__(NT, MINB)
gdr_decode_kernel(GdrDecodeArgs a)
{
    follow();
    constexpr int R = DK * LPR / 32;                // rows of a lane
    const int slices = a.dv / COLS;
    const int n = blockIdx.x / slices, hv = blockIdx.y, hk = hv / (a.Hv / a.Hk);
    const int tid = threadIdx.x, lane = tid & 31;
    const int page = page_of(a.index, n, a.pages, a.err);
    if (page < 0) return;

    const int col = blockIdx.x % slices * COLS + (tid >> 5) * 4 * LPR + 4 * (lane % LPR), r0 = lane / LPR * R;
    float *S = a.state + (((size_t)page * a.Hv + hv) * DK + r0) * a.dv + col;
    float s[R][4];
#pragma unroll
    for (int p = 0; p < R; ++p) ld4(S + (size_t)p * a.dv, s[p]);
    float k[R], q[R], v[4], g, beta;
    auto load_token = [&](int t) {
        const size_t tok = (size_t)n * a.T + t, kat = (tok * a.Hk + hk) * DK + r0, vat = tok * a.Hv + hv;
        load_vec<R>((const IO *)a.k + kat, k);
        load_vec<R>((const IO *)a.q + kat, q);
        ld4((const IO *)a.v + vat * a.dv + col, v);
        g = to_f32(((const IO *)a.g)[vat]);
        beta = to_f32(((const IO *)a.beta)[vat]);
    };
    load_token(0);
    if (a.index) {   // a page belongs to the first row that names it; later ones are refused
        bool clash = false;
        for (int j = tid; j < n; j += NT) clash |= a.index[j] == page;
        if (__syncthreads_or(clash)) {
            if (tid == 0) raise_error(a.err, ERR_PAGE_INDEX);
            return;
        }
    }
    for (int t = 0;;) {
        const float alpha = __expf(clamp_gate(g));
        float x[9] = {}, kq = 0.0f;           // S^T k, S^T q of four columns, q.k
#pragma unroll
        for (int p = 0; p < R; ++p)
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                fma2(x[j], x[j + 1], k[p], k[p], s[p][j], s[p][j + 1], x[j], x[j + 1]);
                fma2(x[4 + j], x[5 + j], q[p], q[p], s[p][j], s[p][j + 1], x[4 + j], x[5 + j]);
            }
#pragma unroll
        for (int p = 0; p < R; p += 2) fma2(x[8], kq, k[p], k[p + 1], q[p], q[p + 1], x[8], kq);
        x[8] += kq;
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
            for (int j = 0; j < 9; ++j) x[j] += __shfl_xor_sync(0xffffffffu, x[j], o);
        float u[4], y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            u[j] = beta * (v[j] - alpha * x[j]);
            y[j] = alpha * x[4 + j] + x[8] * u[j];
        }
        if (lane < LPR) st4((IO *)a.out + (((size_t)n * a.T + t) * a.Hv + hv) * a.dv + col, y);
#pragma unroll
        for (int p = 0; p < R; ++p)
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                mul2(s[p][j], s[p][j + 1], alpha, alpha, s[p][j], s[p][j + 1]);
                fma2(s[p][j], s[p][j + 1], k[p], k[p], u[j], u[j + 1], s[p][j], s[p][j + 1]);
            }
        if (++t == a.T) break;
        load_token(t);
    }
#pragma unroll
    for (int p = 0; p < R; ++p) st4(S + (size_t)p * a.dv, s[p]);
}

}  // namespace

cudaError_t launch_gdr_decode(const GdrDecodeArgs &a, cudaStream_t s)
{
    const dim3 grid((unsigned)a.N * (a.dv / COLS), a.Hv);
    const auto fn = a.io == IO_BF16 ? (a.dk == 128 ? gdr_decode_kernel<__nv_bfloat16, 128> : gdr_decode_kernel<__nv_bfloat16, 64>)
                                    : (a.dk == 128 ? gdr_decode_kernel<float, 128> : gdr_decode_kernel<float, 64>);
    return launch_after(fn, grid, NT, 0, s, a);
}

}  // namespace kda
