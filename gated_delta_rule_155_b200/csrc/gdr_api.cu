// gdr_api.cu — C entry points of the head-gated delta rule and of the state cache's pages
// (declared in include/kda.h).  As in api.cu: all arguments are checked before any launch.
#include <climits>
#include <initializer_list>
#include <cstdint>

#include "../../include/kda.h"
#include "gdr.h"

namespace {

bool misaligned(std::initializer_list<const void *> ptrs)
{
    for (const void *p : ptrs)
        if (p && ((uintptr_t)p & 15u)) return true;
    return false;
}
bool any_null(std::initializer_list<const void *> ptrs)
{
    for (const void *p : ptrs)
        if (!p) return true;
    return false;
}
kda_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }
kda::IoType io_of(kda_dtype_t io) { return io == KDA_BF16 ? kda::IO_BF16 : kda::IO_F32; }

kda_status_t check_dims(int N, int T, int Hk, int Hv, int dk, int dv, kda_dtype_t io)
{
    if (N < 1 || T < 0 || Hk < 1 || Hv < 1 || Hv % Hk) return KDA_ERR_INVALID_ARG;
    if (io != KDA_F32 && io != KDA_BF16) return KDA_ERR_INVALID_ARG;
    if ((dk != 64 && dk != 128) || (dv != 64 && dv != 128)) return KDA_ERR_UNSUPPORTED;
    // grids have the value heads in y; token, chunk and block counts are 32-bit, element offsets 64-bit
    if (Hv > 65534 || (long long)T * Hv > INT_MAX / 2 || (long long)N * Hv > INT_MAX / 2) return KDA_ERR_UNSUPPORTED;
    if ((long long)N * 8 > INT_MAX / 2 || (long long)T + 64ll * N > INT_MAX / 2) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// bf16 at dk = dv = 128 runs on the tensor cores and nowhere else
bool on_tensor_cores(int dk, int dv, kda_dtype_t io) { return kda::gdr_tc_shape(dk, dv, io_of(io)); }

size_t workspace_bytes_of(int N, int T, int Hk, int Hv, int dk, int dv, kda_dtype_t io, bool backward)
{
    if (T == 0) return 0;
    return on_tensor_cores(dk, dv, io) ? kda::gdr_tc_workspace(N, T, Hk, Hv, backward)
                                                 : kda::gdr_simt_workspace(N, T, Hk, Hv, dk, dv, backward);
}

kda_status_t check_workspace(const void *ws, size_t have, size_t need)
{
    if (need == 0) return KDA_OK;
    if (!ws || have < need) return KDA_ERR_WORKSPACE;
    return ((uintptr_t)ws & 255u) ? KDA_ERR_MISALIGNED : KDA_OK;
}

kda_status_t check_pages(const void *cache, size_t page_bytes, int layers, int pages, int n)
{
    if (!cache || layers < 1 || pages < 1 || n < 0 || page_bytes == 0) return KDA_ERR_INVALID_ARG;
    if (page_bytes % 16) return KDA_ERR_UNSUPPORTED;
    if ((uintptr_t)cache & 15u) return KDA_ERR_MISALIGNED;
    return KDA_OK;
}
// whether a buffer that is written is also one that is read, or is written twice
bool shared(std::initializer_list<const void *> written, std::initializer_list<const void *> read)
{
    for (auto w = written.begin(); w != written.end(); ++w) {
        if (!*w) continue;
        for (const void *r : read)
            if (*w == r) return true;
        for (auto x = written.begin(); x != w; ++x)
            if (*w == *x) return true;
    }
    return false;
}
bool meet(const int *a, const int *b, int n) { return a < b + n && b < a + n; }
bool misaligned4(std::initializer_list<const void *> ptrs)
{
    for (const void *p : ptrs)
        if (p && ((uintptr_t)p & 3u)) return true;
    return false;
}

}  // namespace

extern "C" {

kda_status_t kda_gdr_workspace_size(int N, int T_total, int Hk, int Hv, int dk, int dv, kda_dtype_t io, int backward,
                                    size_t *bytes)
{
    if (!bytes) return KDA_ERR_INVALID_ARG;
    const kda_status_t st = check_dims(N, T_total, Hk, Hv, dk, dv, io);
    if (st != KDA_OK) return st;
    *bytes = workspace_bytes_of(N, T_total, Hk, Hv, dk, dv, io, backward != 0);
    return KDA_OK;
}

kda_status_t kda_gdr_forward(const void *q, const void *k, const void *v, const void *g, const void *beta,
                             const float *initial_state, const int *initial_index, void *out, float *final_state,
                             const int *final_index, int pages, const int *cu_seqlens, void *workspace,
                             size_t workspace_bytes, int N, int T_total, int Hk, int Hv, int dk, int dv, kda_dtype_t io,
                             kda_stream_t stream)
{
    kda_status_t st = check_dims(N, T_total, Hk, Hv, dk, dv, io);
    if (st != KDA_OK) return st;
    if (T_total > 0 && any_null({q, k, v, g, beta, out})) return KDA_ERR_INVALID_ARG;
    if ((initial_index && !initial_state) || (final_index && !final_state)) return KDA_ERR_INVALID_ARG;
    if ((initial_index || final_index) && pages < 1) return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens && T_total % N) return KDA_ERR_INVALID_ARG;
    if (misaligned({q, k, v, g, beta, initial_state, out, final_state}) ||
        misaligned4({initial_index, final_index, cu_seqlens}))
        return KDA_ERR_MISALIGNED;
    st = check_workspace(workspace, workspace_bytes, workspace_bytes_of(N, T_total, Hk, Hv, dk, dv, io, false));
    if (st != KDA_OK) return st;
    // what no kernel touches may be anything: at T_total = 0 the tensors of tokens and the workspace
    const bool tokens = T_total > 0;
    const void *o = tokens ? out : nullptr, *ws = tokens ? workspace : nullptr;
    if (shared({o, final_state, ws}, {initial_index, final_index, cu_seqlens}) || shared({o, ws}, {initial_state}) ||
        (tokens && shared({out, final_state, workspace}, {q, k, v, g, beta})))
        return KDA_ERR_INVALID_ARG;
    kda::GdrArgs a{q, k, v, g, beta, initial_state, initial_index, out, final_state, final_index, pages, cu_seqlens,
                   workspace, N, T_total, Hk, Hv, dk, dv, io_of(io), kda::device_error_word()};
    if (on_tensor_cores(dk, dv, io)) {
        if (!kda::gdr_tc_available()) return KDA_ERR_UNSUPPORTED;
        return cuda_status(kda::launch_gdr_forward_tc(a, (cudaStream_t)stream));
    }
    return cuda_status(kda::launch_gdr_forward_simt(a, (cudaStream_t)stream));
}

kda_status_t kda_gdr_backward(const void *q, const void *k, const void *v, const void *g, const void *beta,
                              const float *initial_state, const int *cu_seqlens, const void *d_out,
                              const float *d_final_state, void *d_q, void *d_k, void *d_v, void *d_g, void *d_beta,
                              float *d_initial_state, void *workspace, size_t workspace_bytes, int N, int T_total, int Hk,
                              int Hv, int dk, int dv, kda_dtype_t io, kda_stream_t stream)
{
    kda_status_t st = check_dims(N, T_total, Hk, Hv, dk, dv, io);
    if (st != KDA_OK) return st;
    if (T_total > 0 && any_null({q, k, v, g, beta, d_out, d_q, d_k, d_v, d_g, d_beta})) return KDA_ERR_INVALID_ARG;
    if (!cu_seqlens && T_total % N) return KDA_ERR_INVALID_ARG;
    if (misaligned({q, k, v, g, beta, initial_state, d_out, d_final_state, d_q, d_k, d_v, d_g, d_beta, d_initial_state}) ||
        misaligned4({cu_seqlens}))
        return KDA_ERR_MISALIGNED;
    st = check_workspace(workspace, workspace_bytes, workspace_bytes_of(N, T_total, Hk, Hv, dk, dv, io, true));
    if (st != KDA_OK) return st;
    // d_initial_state may be d_final_state: a block reads its columns of the one before it writes them to the other.
    // It may not be initial_state, which other blocks may not have read yet.
    if (shared({d_initial_state}, {initial_state, cu_seqlens})) return KDA_ERR_INVALID_ARG;
    if (T_total > 0 && (shared({d_q, d_k, d_v, d_g, d_beta, d_initial_state, workspace},
                               {q, k, v, g, beta, d_out, initial_state, cu_seqlens}) ||
                        shared({d_q, d_k, d_v, d_g, d_beta, workspace}, {d_final_state})))
        return KDA_ERR_INVALID_ARG;
    kda::GdrArgs a{q, k, v, g, beta, initial_state, nullptr, nullptr, nullptr, nullptr, 0, cu_seqlens,
                   workspace, N, T_total, Hk, Hv, dk, dv, io_of(io), kda::device_error_word(),
                   d_out, d_final_state, d_q, d_k, d_v, d_g, d_beta, d_initial_state};
    if (on_tensor_cores(dk, dv, io)) {
        if (!kda::gdr_tc_available()) return KDA_ERR_UNSUPPORTED;
        return cuda_status(kda::launch_gdr_backward_tc(a, (cudaStream_t)stream));
    }
    return cuda_status(kda::launch_gdr_backward_simt(a, (cudaStream_t)stream));
}

kda_status_t kda_gdr_decode(const void *q, const void *k, const void *v, const void *g, const void *beta, float *state,
                            const int *index, int pages, void *out, int N, int T, int Hk, int Hv, int dk, int dv,
                            kda_dtype_t io, kda_stream_t stream)
{
    if (N > 0 && T > INT_MAX / N) return KDA_ERR_UNSUPPORTED;
    kda_status_t st = check_dims(N, N > 0 ? N * T : T, Hk, Hv, dk, dv, io);
    if (st != KDA_OK) return st;
    if (T < 1 || any_null({q, k, v, g, beta, state, out})) return KDA_ERR_INVALID_ARG;
    if (index && pages < 1) return KDA_ERR_INVALID_ARG;
    if (misaligned({q, k, v, g, beta, state, out}) || misaligned4({index})) return KDA_ERR_MISALIGNED;
    if (shared({out, state}, {q, k, v, g, beta, index})) return KDA_ERR_INVALID_ARG;
    kda::GdrDecodeArgs a{q, k, v, g, beta, state, index, pages, out, N, T, Hk, Hv, dk, dv, io_of(io),
                         kda::device_error_word()};
    return cuda_status(kda::launch_gdr_decode(a, (cudaStream_t)stream));
}

kda_status_t kda_pages_fork(void *cache, size_t page_bytes, int layers, int pages, int *refs, const int *parents,
                            int *children, int n, kda_stream_t stream)
{
    const kda_status_t st = check_pages(cache, page_bytes, layers, pages, n);
    if (st != KDA_OK) return st;
    if (!refs || (n > 0 && any_null({parents, children}))) return KDA_ERR_INVALID_ARG;
    if (misaligned4({refs, parents, children})) return KDA_ERR_MISALIGNED;
    if (n == 0) return KDA_OK;
    if (shared({cache, refs, children}, {parents})) return KDA_ERR_INVALID_ARG;
    if (meet(children, parents, n)) return KDA_ERR_INVALID_ARG;   // written before the copies read the parents
    kda::PagesArgs a{cache, page_bytes, layers, pages, kda::device_error_word()};
    return cuda_status(kda::launch_pages_fork(a, refs, parents, children, n, (cudaStream_t)stream));
}

kda_status_t kda_pages_copy(void *cache, size_t page_bytes, int layers, int pages, const int *src, const int *dst, int n,
                            kda_stream_t stream)
{
    const kda_status_t st = check_pages(cache, page_bytes, layers, pages, n);
    if (st != KDA_OK) return st;
    if (n > 0 && any_null({src, dst})) return KDA_ERR_INVALID_ARG;
    if (misaligned4({src, dst})) return KDA_ERR_MISALIGNED;
    if (n == 0) return KDA_OK;
    if (shared({cache}, {src, dst})) return KDA_ERR_INVALID_ARG;
    kda::PagesArgs a{cache, page_bytes, layers, pages, kda::device_error_word()};
    return cuda_status(kda::launch_pages_copy(a, src, dst, n, (cudaStream_t)stream));
}

kda_status_t kda_pages_free(int *refs, int pages, const int *ids, int n, kda_stream_t stream)
{
    if (!refs || pages < 1 || n < 0 || (n > 0 && !ids)) return KDA_ERR_INVALID_ARG;
    if (misaligned4({refs, ids})) return KDA_ERR_MISALIGNED;
    if (n == 0) return KDA_OK;
    if (shared({refs}, {ids})) return KDA_ERR_INVALID_ARG;
    return cuda_status(kda::launch_pages_free(refs, pages, ids, n, kda::device_error_word(), (cudaStream_t)stream));
}

kda_status_t kda_pages_workspace_size(int pages, size_t *bytes)
{
    if (!bytes || pages < 1) return KDA_ERR_INVALID_ARG;
    *bytes = kda::pages_compact_workspace(pages);
    return KDA_OK;
}

kda_status_t kda_pages_compact(void *cache, size_t page_bytes, int layers, int pages, int *refs, int *table, int n, int *live,
                               void *workspace, size_t workspace_bytes, kda_stream_t stream)
{
    const kda_status_t st = check_pages(cache, page_bytes, layers, pages, n);
    if (st != KDA_OK) return st;
    if (!refs || (n > 0 && !table)) return KDA_ERR_INVALID_ARG;
    if (misaligned4({refs, table, live, workspace})) return KDA_ERR_MISALIGNED;
    if (!workspace || workspace_bytes < kda::pages_compact_workspace(pages)) return KDA_ERR_WORKSPACE;
    if (shared({cache, refs, n > 0 ? table : nullptr, live, workspace}, {})) return KDA_ERR_INVALID_ARG;
    kda::PagesArgs a{cache, page_bytes, layers, pages, kda::device_error_word()};
    return cuda_status(kda::launch_pages_compact(a, refs, table, n, live, workspace, (cudaStream_t)stream));
}

}  // extern "C"
