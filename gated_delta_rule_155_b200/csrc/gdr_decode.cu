// gdr_decode.cu — the head-gated delta rule token by token, on pages of a state cache
// (memory-bound: one read and one write of each state, however many tokens it takes).
//
// Per sequence, value head and token, with S the dk x dv fp32 state:
//     S' = e^g S;   a = S'^T k;   b = S'^T q;   u = beta (v - a);   S <- S' + k u^T;   o = b + (q.k) u
// so both column sums come from one pass over the decayed state and a token costs one reduction.
// A block holds a slice of the state's columns in registers for all its tokens: a warp reads whole
// rows of the slice (a float4 a lane), so 64 KB of loads of a 128-column block are in flight before
// anything else is waited for.  Column sums reduce over the rows of a warp by shuffles and over the
// warps in shared memory.
#include "gdr.cuh"

namespace kda {
namespace {

using namespace gdr;

template <typename IO, int DK, int SLICE, int NTH>
__global__ void __launch_bounds__(NTH)
gdr_decode_kernel(GdrDecodeArgs a)
{
    constexpr int LPR = SLICE / 4;            // lanes of a row
    constexpr int ROWS = NTH / LPR;           // rows of a pass
    constexpr int NP = DK / ROWS;
    constexpr int NW = NTH / 32;
    static_assert(LPR <= 32 && NTH >= DK && NTH >= SLICE && NP >= 1, "block shape");
    __shared__ float s_k[2][DK], s_q[2][DK];
    __shared__ float s_a[NW][SLICE], s_b[NW][SLICE], s_u[SLICE];
    __shared__ float s_qk[NW];

    const int slices = a.dv / SLICE;
    const int n = blockIdx.x / slices, col0 = blockIdx.x % slices * SLICE, hv = blockIdx.y, hk = hv / (a.Hv / a.Hk);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int page = page_of(a.index, n, a.pages, a.err);
    if (page < 0) return;

    const int col = 4 * (tid % LPR), r0 = tid / LPR;
    float *S = a.state + ((size_t)page * a.Hv + hv) * DK * a.dv + col0 + col;
    float4 s[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) s[p] = *reinterpret_cast<const float4 *>(S + (size_t)(r0 + p * ROWS) * a.dv);
    if (a.index) {   // a page belongs to the first row that names it; later ones are refused
        bool clash = false;
        for (int j = tid; j < n; j += NTH) clash |= a.index[j] == page;
        if (__syncthreads_or(clash)) {
            if (tid == 0) raise_error(a.err, ERR_PAGE_INDEX);
            return;
        }
    }
    const IO *q = (const IO *)a.q, *k = (const IO *)a.k, *v = (const IO *)a.v;
    for (int t = 0; t < a.T; ++t) {
        const size_t tok = (size_t)n * a.T + t;
        const int x = t & 1;
        float qk = 0.0f;
        if (tid < DK) {
            const float kr = to_f32(k[(tok * a.Hk + hk) * DK + tid]), qr = to_f32(q[(tok * a.Hk + hk) * DK + tid]);
            s_k[x][tid] = kr;
            s_q[x][tid] = qr;
            qk = kr * qr;
        }
        const float alpha = __expf(clamp_gate(to_f32(((const IO *)a.g)[tok * a.Hv + hv])));
        const float beta = to_f32(((const IO *)a.beta)[tok * a.Hv + hv]);
        const float vv = tid < SLICE ? to_f32(v[(tok * a.Hv + hv) * a.dv + col0 + tid]) : 0.0f;
        qk = warp_sum(qk);
        if (lane == 0) s_qk[warp] = qk;
        __syncthreads();
        float sa[4] = {}, sb[4] = {};
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const float kr = s_k[x][r0 + p * ROWS], qr = s_q[x][r0 + p * ROWS];
            s[p].x *= alpha; s[p].y *= alpha; s[p].z *= alpha; s[p].w *= alpha;
            sa[0] += kr * s[p].x; sa[1] += kr * s[p].y; sa[2] += kr * s[p].z; sa[3] += kr * s[p].w;
            sb[0] += qr * s[p].x; sb[1] += qr * s[p].y; sb[2] += qr * s[p].z; sb[3] += qr * s[p].w;
        }
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sa[j] += __shfl_xor_sync(0xffffffffu, sa[j], o);
                sb[j] += __shfl_xor_sync(0xffffffffu, sb[j], o);
            }
        if (lane < LPR) {
            st4(&s_a[warp][col], sa);
            st4(&s_b[warp][col], sb);
        }
        __syncthreads();
        if (tid < SLICE) {
            float xa = 0.0f, xb = 0.0f, xq = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                xa += s_a[w][tid];
                xb += s_b[w][tid];
                xq += s_qk[w];
            }
            const float u = beta * (vv - xa);
            s_u[tid] = u;
            ((IO *)a.out)[(tok * a.Hv + hv) * a.dv + col0 + tid] = from_f32<IO>(xb + xq * u);
        }
        __syncthreads();
        const float4 u = *(const float4 *)&s_u[col];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const float kr = s_k[x][r0 + p * ROWS];
            s[p].x += kr * u.x; s[p].y += kr * u.y; s[p].z += kr * u.z; s[p].w += kr * u.w;
        }
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) *reinterpret_cast<float4 *>(S + (size_t)(r0 + p * ROWS) * a.dv) = s[p];
}

template <typename IO, int DK>
void launch(const GdrDecodeArgs &a, cudaStream_t s)
{
    if (a.dv == 128)
        gdr_decode_kernel<IO, DK, 128, 512><<<dim3(a.N, a.Hv), 512, 0, s>>>(a);
    else
        gdr_decode_kernel<IO, DK, 64, 256><<<dim3(a.N, a.Hv), 256, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_gdr_decode(const GdrDecodeArgs &a, cudaStream_t s)
{
    if (a.io == IO_BF16) a.dk == 128 ? launch<__nv_bfloat16, 128>(a, s) : launch<__nv_bfloat16, 64>(a, s);
    else a.dk == 128 ? launch<float, 128>(a, s) : launch<float, 64>(a, s);
    return cudaGetLastError();
}

}  // namespace kda
