// gdr.h — launchers of the head-gated delta rule (one gate per value head, grouped heads)
// and of the state cache's pages.  Launchers assume validated arguments.
#pragma once

#include "internal.h"

namespace kda {

// N sequences packed over a token axis of T rows (cu: their N + 1 offsets on the device, or
// null for N sequences of T / N tokens); Hv value heads in groups that share a key head.
struct GdrArgs {
    const void *q, *k, *v, *g, *beta;   // io: [T, Hk, dk], [T, Hk, dk], [T, Hv, dv], [T, Hv], [T, Hv]
    const float *s0;                    // [N or pages, Hv, dk, dv] or null (zeros)
    const int *s0_index;                // page of each sequence's initial state, -1: zeros; null: sequence n's is n
    void *out;                          // io [T, Hv, dv]
    float *sT;                          // [N or pages, Hv, dk, dv] or null
    const int *sT_index;                // page of each sequence's final state, -1: not kept; null: n
    int pages;                          // pages that the indices may name
    const int *cu;
    void *ws;
    int N, T, Hk, Hv, dk, dv;
    IoType io;
    int *err;
    // backward only
    const void *dO;
    const float *dST;
    void *dq, *dk_, *dv_, *dg, *dbeta;
    float *ds0;
};

// Chunk slots: sequence n's chunks start at slot first_row / 64 + n, so that no prefix sum over
// the sequences is needed; T / 64 + N slots in all.
__host__ __device__ inline long long gdr_slots(int N, int T) { return (long long)T / 64 + N; }

size_t gdr_simt_workspace(int N, int T, int Hk, int Hv, int dk, int dv, bool backward);
cudaError_t launch_gdr_forward_simt(const GdrArgs &a, cudaStream_t s);
cudaError_t launch_gdr_backward_simt(const GdrArgs &a, cudaStream_t s);

// tcgen05 kernels: bf16, dk = dv = 128.
bool gdr_tc_shape(int dk, int dv, IoType io);
bool gdr_tc_available();
// The chunk whose tiles prep never loads, for tests (-1: none).  Process-wide, as WaitHooks.
void set_gdr_prep_hook(int skip_chunk);
size_t gdr_tc_workspace(int N, int T, int Hk, int Hv, bool backward);
cudaError_t launch_gdr_forward_tc(const GdrArgs &a, cudaStream_t s);
cudaError_t launch_gdr_backward_tc(const GdrArgs &a, cudaStream_t s);

struct GdrDecodeArgs {
    const void *q, *k, *v, *g, *beta;   // io [N, T, Hk, dk], ..., [N, T, Hv]
    float *state;                       // [pages, Hv, dk, dv]
    const int *index;                   // [N] or null
    int pages;
    void *out;                          // io [N, T, Hv, dv]
    int N, T, Hk, Hv, dk, dv;
    IoType io;
    int *err;
};
cudaError_t launch_gdr_decode(const GdrDecodeArgs &a, cudaStream_t s);

struct PagesArgs {
    void *cache;                        // [layers, pages, page_bytes]
    size_t page_bytes;
    int layers, pages;
    int *err;
};
cudaError_t launch_pages_fork(const PagesArgs &a, int *refs, const int *parents, int *children, int n, cudaStream_t s);
cudaError_t launch_pages_copy(const PagesArgs &a, const int *src, const int *dst, int n, cudaStream_t s);
cudaError_t launch_pages_free(int *refs, int pages, const int *ids, int n, int *err, cudaStream_t s);
size_t pages_compact_workspace(int pages);
cudaError_t launch_pages_compact(const PagesArgs &a, int *refs, int *table, int n, int *live, void *ws, cudaStream_t s);

// Device error word: a page index out of range, not live, or named twice.
constexpr int kErrPageIndex = 3;

// The device error word of the current device (api.cu).
int *device_error_word();

}  // namespace kda
