// pages.cu — pages of a state cache: fork (allocate and copy), copy, free, compact.
//
// The cache is [layers, pages, page_bytes]; refs[p] counts the holders of page p (0: free).  What
// is to be moved is decided by one block over refs (fork, compact), on the device, so that a call
// can be captured in a graph; the moves themselves are bandwidth-bound copies over (move, layer,
// piece of a page), 16 bytes a thread and load, as many loads in flight as a piece has.  HBM bounds them: 64
// pages of 2 MB in four layers (604 MB read and written) in 97 us, 6.2 TB/s; the plan takes 4 us.
#include "gdr.cuh"

namespace kda {
namespace {

using namespace gdr;

constexpr int PT = 1024;            // plan block
constexpr int CT = 256;             // copy block
constexpr int UNROLL = 8;
constexpr int PIECE = CT * 16 * UNROLL;   // bytes of a page that a block copies at a time: 32 KB

// Exclusive prefix of x over the block (PT threads), and the block's sum.
KDA_DEVICE int block_prefix(int x, int &sum, int tid)
{
    __shared__ int s_w[32];
    int y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if ((tid & 31) >= o) y += z;
    }
    __syncthreads();                // readers of the previous call's s_w
    if ((tid & 31) == 31) s_w[tid >> 5] = y;
    __syncthreads();
    int w = s_w[tid & 31], before = 0;
    sum = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const int v = __shfl_sync(0xffffffffu, w, i);
        if (i < (tid >> 5)) before += v;
        sum += v;
    }
    return before + y - x;
}

// children[i] <- the i-th free page (lowest first), -1 where there is none or parents[i] is no live
// page; refs of the pages handed out <- 1.  Parents are judged by refs as they are at the call.
__global__ void __launch_bounds__(PT) pages_fork_plan_kernel(int *refs, int pages, const int *parents, int *children, int n,
                                                             int *err)
{
    follow();
    const int tid = threadIdx.x;
    for (int i = tid; i < n; i += PT) {
        const int p = parents[i];
        const bool ok = p == -1 || (p >= 0 && p < pages && refs[p] > 0);
        if (!ok) raise_error(err, ERR_PAGE_INDEX);
        children[i] = ok ? 0 : -1;
    }
    __syncthreads();
    int done = 0;
    for (int base = 0; base < pages && done < n; base += 4 * PT) {
        const int p0 = base + 4 * tid;
        bool f[4];
        int mine = 0, sum;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[e] = p0 + e < pages && refs[p0 + e] == 0;
            mine += f[e];
        }
        int rank = done + block_prefix(mine, sum, tid);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (f[e]) {
                if (rank < n && children[rank] == 0) {
                    children[rank] = p0 + e;
                    refs[p0 + e] = 1;
                }
                ++rank;
            }
        done += sum;
    }
    for (int i = done + tid; i < n; i += PT) children[i] = -1;
}

// map[p]: the page that live page p moves to (itself if it stays).  The k-th live page at or above
// the number of live pages goes to the k-th free page below it; no page is both left and entered.
__global__ void __launch_bounds__(PT) pages_compact_plan_kernel(int *refs, int pages, int *table, int n, int *live, int *map,
                                                                int *from, int *to, int *count, int *err)
{
    follow();
    const int tid = threadIdx.x;
    int mine = 0, m;
    for (int p = tid; p < pages; p += PT) mine += refs[p] > 0;
    block_prefix(mine, m, tid);
    int holes = 0, movers = 0;
    for (int base = 0; base < pages; base += PT) {
        const int p = base + tid;
        const bool in = p < pages, used = in && refs[p] > 0;
        const bool hole = in && !used && p < m, mover = used && p >= m;
        int sh, sm;
        const int rh = holes + block_prefix(hole, sh, tid), rm = movers + block_prefix(mover, sm, tid);
        if (hole) to[rh] = p;
        if (mover) from[rm] = p;
        if (in) map[p] = used ? p : -1;
        holes += sh;
        movers += sm;
    }
    __syncthreads();
    for (int k = tid; k < movers; k += PT) {
        const int f = from[k], t = to[k];
        map[f] = t;
        refs[t] = refs[f];
        refs[f] = 0;
    }
    __syncthreads();
    for (int i = tid; i < n; i += PT) {
        const int p = table[i];
        if (p == -1) continue;
        const int t = p >= 0 && p < pages ? map[p] : -1;
        if (t < 0) raise_error(err, ERR_PAGE_INDEX);
        table[i] = t;
    }
    if (tid == 0) {
        *count = movers;
        if (live) *live = m;
    }
}

// Moves src[i] -> dst[i], i < n (count: n on the device, at most n), of every layer.  src -1: the
// page is zeroed; dst -1: nothing.  CHECK: the pairs are the caller's: a pair whose page is out of
// range, whose destination an earlier pair has, or whose source another pair writes, is left out.
// Pieces run slowest, pairs fastest, so that pairs with one source read it while it is in L2.
template <bool CHECK>
__global__ void __launch_bounds__(CT) pages_copy_kernel(PagesArgs a, const int *src, const int *dst, int n, const int *count)
{
    follow();
    const int tid = threadIdx.x;
    if (count) n = min(n, *count);
    const long long pieces = (long long)((a.page_bytes + PIECE - 1) / PIECE);
    const long long total = pieces * a.layers * n;
    for (long long w = blockIdx.x; w < total; w += gridDim.x) {
        const int i = (int)(w % n);
        const long long r = w / n;
        const size_t layer = (size_t)(r / pieces), off = (size_t)(r % pieces) * PIECE;
        const int d = dst[i], f = src[i];
        if (CHECK) {
            bool bad = d < -1 || d >= a.pages || f < -1 || f >= a.pages;
            if (!bad && d >= 0)
                for (int j = tid; j < n; j += CT) {
                    const int dj = dst[j];
                    if (dj < 0 || j == i) continue;
                    bad |= dj == d && j < i;
                    bad |= dj == f && src[j] != dj;
                }
            if (__syncthreads_or(bad)) {
                if (tid == 0) raise_error(a.err, ERR_PAGE_INDEX);
                continue;
            }
        }
        if (d < 0 || f == d) continue;
        uint4 *to = (uint4 *)((char *)a.cache + (layer * a.pages + d) * a.page_bytes + off);
        const uint4 *from = (const uint4 *)((const char *)a.cache + (layer * a.pages + (f < 0 ? 0 : f)) * a.page_bytes + off);
        const size_t left = a.page_bytes - off;
        const int vecs = (int)((left < (size_t)PIECE ? left : (size_t)PIECE) / 16);
        uint4 x[UNROLL];
#pragma unroll
        for (int e = 0; e < UNROLL; ++e)
            if (tid + e * CT < vecs) x[e] = f < 0 ? make_uint4(0u, 0u, 0u, 0u) : from[tid + e * CT];
#pragma unroll
        for (int e = 0; e < UNROLL; ++e)
            if (tid + e * CT < vecs) to[tid + e * CT] = x[e];
    }
}

__global__ void pages_free_kernel(int *refs, int pages, const int *ids, int n, int *err)
{
    follow();
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    const int p = ids[i];
    if (p == -1) return;
    if (p < 0 || p >= pages) {
        raise_error(err, ERR_PAGE_INDEX);
        return;
    }
    if (atomicSub(refs + p, 1) <= 0) {   // nobody held it
        atomicAdd(refs + p, 1);
        raise_error(err, ERR_PAGE_INDEX);
    }
}

unsigned copy_blocks(const PagesArgs &a, long long moves)
{
    const long long total = (long long)((a.page_bytes + PIECE - 1) / PIECE) * a.layers * moves;
    const long long most = 1 << 20;      // further pieces are looped over
    return (unsigned)(total < 1 ? 1 : total > most ? most : total);
}

}  // namespace

cudaError_t launch_pages_fork(const PagesArgs &a, int *refs, const int *parents, int *children, int n, cudaStream_t s)
{
    const cudaError_t e = launch_after(pages_fork_plan_kernel, 1, PT, 0, s, refs, a.pages, parents, children, n, a.err);
    if (e != cudaSuccess) return e;
    // every child is a page that was free, every parent one that was not: the pairs cannot meet
    return launch_after(pages_copy_kernel<false>, copy_blocks(a, n), CT, 0, s, a, parents, children, n, nullptr);
}

cudaError_t launch_pages_copy(const PagesArgs &a, const int *src, const int *dst, int n, cudaStream_t s)
{
    return launch_after(pages_copy_kernel<true>, copy_blocks(a, n), CT, 0, s, a, src, dst, n, nullptr);
}

cudaError_t launch_pages_free(int *refs, int pages, const int *ids, int n, int *err, cudaStream_t s)
{
    return launch_after(pages_free_kernel, (n + 255) / 256, 256, 0, s, refs, pages, ids, n, err);
}

// map [pages], from [pages / 2], to [pages / 2], count
size_t pages_compact_workspace(int pages) { return 4 * ((size_t)pages + 2 * (size_t)(pages / 2) + 1); }

cudaError_t launch_pages_compact(const PagesArgs &a, int *refs, int *table, int n, int *live, void *ws, cudaStream_t s)
{
    int *map = (int *)ws, *from = map + a.pages, *to = from + a.pages / 2, *count = to + a.pages / 2;
    const cudaError_t e = launch_after(pages_compact_plan_kernel, 1, PT, 0, s, refs, a.pages, table, n, live, map, from, to, count, a.err);
    if (e != cudaSuccess || a.pages < 2) return e;
    return launch_after(pages_copy_kernel<false>, copy_blocks(a, a.pages / 2), CT, 0, s, a, from, to, a.pages / 2, count);
}

}  // namespace kda
