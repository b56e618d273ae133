// api_paged.cu -- the paged-cache calls of include/pisa.h: argument validation on
// the host and dispatch, by the same rules as api.cu (nothing is enqueued unless
// every check passes; no call allocates memory).
#include <math.h>
#include <stdint.h>

#include "pisa.h"
#include "pisa_internal.h"
#include "pisa_paged.cuh"

using namespace pisa;

namespace {

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? PISA_OK : PISA_E_CUDA; }
int64_t width(const pisa_cfg* c, const pisa_pages* g) { return ((int64_t)c->N + g->S - 1) / g->S; }

// limits of the kernels that address a paged cache (those of the decode calls, and the pages')
int check(const pisa_cfg* c, const pisa_pages* g) {
    if (!c || !g) return PISA_E_INVALID;
    const int s = check_gpu_cfg(c);
    if (s) return s;
    if (g->S < 1 || g->P < 1) return PISA_E_INVALID;
    if (g->S > 1024 || c->N > (1 << 30)) return PISA_E_UNSUPPORTED;
    if ((int64_t)g->P * c->Hkv * g->S >= ((int64_t)1 << 31)) return PISA_E_UNSUPPORTED;  // 32-bit pool rows
    if ((int64_t)c->B * width(c, g) >= ((int64_t)1 << 31)) return PISA_E_UNSUPPORTED;
    return PISA_OK;
}

PagedParams params(const pisa_cfg* c, const pisa_pages* g, const int32_t* table, const int32_t* len) {
    PagedParams p;
    p.B = c->B; p.Hq = c->Hq; p.Hkv = c->Hkv; p.N = c->N;
    p.S = g->S; p.P = g->P; p.W = (int)width(c, g);
    p.qscale = (float)(1.4426950408889634 / sqrt((double)c->d));
    p.table = table;
    p.len = len;
    return p;
}

PagedDecodeParams decode_params(const pisa_cfg* c, const pisa_pages* g, const int32_t* table) {
    PagedDecodeParams p;
    p.B = c->B; p.Hq = c->Hq; p.Hkv = c->Hkv; p.N = c->N; p.C = c->C; p.K = c->K;
    p.forced_mask = c->forced_mask;
    p.qscale = (float)(1.4426950408889634 / sqrt((double)c->d));
    make_geom(c->N, c->C, &p.geom);
    p.variant = c->score_variant;
    p.table = table; p.S = g->S; p.P = g->P; p.W = (int)width(c, g);
    return p;
}

int elem_bytes(const pisa_cfg* c) { return c->dtype == PISA_DTYPE_BF16 ? 2 : 4; }

}  // namespace

extern "C" {

int64_t pisa_pages_state_words(const pisa_pages* pages) {
    if (!pages || pages->S < 1 || pages->P < 1) return PISA_E_INVALID;
    return PageState(pages->P).words();
}

int pisa_pages_init(const pisa_cfg* cfg, const pisa_pages* pages, int32_t* state, int32_t* table, int32_t* len,
                    void* stream) {
    const int s = check(cfg, pages);
    if (s) return s;
    if (!state || !len || (cfg->N > 0 && !table)) return PISA_E_INVALID;
    if (!aligned(state, 16) || !aligned(table, 4) || !aligned(len, 4)) return PISA_E_ALIGNMENT;
    return cuda_status(launch_pages_init(state, table, len, cfg->B, pages->P, (int)width(cfg, pages), (cudaStream_t)stream));
}

int pisa_pages_reserve(const pisa_cfg* cfg, const pisa_pages* pages, const int32_t* add, int32_t* state, int32_t* table,
                       int32_t* len, int32_t* grant, int32_t* moves, int64_t moves_words, void* stream) {
    const int s = check(cfg, pages);
    if (s) return s;
    if (cfg->B > kReserveMaxSeqs) return PISA_E_UNSUPPORTED;
    if (!add || !state || !len || !grant || !moves || (cfg->N > 0 && !table)) return PISA_E_INVALID;
    if (grant == add || grant == len || add == len) return PISA_E_INVALID;
    if (moves_words < kMovesHead + 2 * (int64_t)cfg->B) return PISA_E_INVALID;
    if (!aligned(state, 16) || !aligned(add, 4) || !aligned(table, 4) || !aligned(len, 4) || !aligned(grant, 4) ||
        !aligned(moves, 4))
        return PISA_E_ALIGNMENT;
    return cuda_status(launch_pages_reserve(add, state, table, len, grant, moves, cfg->B, cfg->N, pages->S, pages->P,
                                            (int)width(cfg, pages), (cudaStream_t)stream));
}

int pisa_pages_fork(const pisa_cfg* cfg, const pisa_pages* pages, const int32_t* parent, int32_t* state,
                    const int32_t* table, const int32_t* len, int32_t* table_out, int32_t* len_out, void* stream) {
    const int s = check(cfg, pages);
    if (s) return s;
    if (cfg->N == 0) return PISA_OK;
    if (!parent || !state || !table || !len || !table_out || !len_out) return PISA_E_INVALID;
    if (table_out == table || len_out == len) return PISA_E_INVALID;
    if (!aligned(state, 16) || !aligned(parent, 4) || !aligned(table, 4) || !aligned(len, 4) || !aligned(table_out, 4) ||
        !aligned(len_out, 4))
        return PISA_E_ALIGNMENT;
    return cuda_status(launch_pages_fork(parent, state, table, len, table_out, len_out, cfg->B, pages->P,
                                         (int)width(cfg, pages), (cudaStream_t)stream));
}

int pisa_pages_free(const pisa_cfg* cfg, const pisa_pages* pages, const int32_t* seqs, int n, int32_t* state,
                    int32_t* table, int32_t* len, void* stream) {
    const int s = check(cfg, pages);
    if (s) return s;
    if (n < 0) return PISA_E_INVALID;
    if (n == 0 || cfg->N == 0) return PISA_OK;
    if (!seqs || !state || !table || !len) return PISA_E_INVALID;
    if (!aligned(state, 16) || !aligned(seqs, 4) || !aligned(table, 4) || !aligned(len, 4)) return PISA_E_ALIGNMENT;
    if ((int64_t)n * ((width(cfg, pages) + 255) / 256) >= ((int64_t)1 << 31)) return PISA_E_UNSUPPORTED;
    return cuda_status(launch_pages_free(seqs, n, state, table, len, cfg->B, pages->P, (int)width(cfg, pages),
                                         (cudaStream_t)stream));
}

int pisa_pages_compact(const pisa_cfg* cfg, const pisa_pages* pages, int32_t* state, int32_t* table, int32_t* moves,
                       int64_t moves_words, void* stream) {
    const int s = check(cfg, pages);
    if (s) return s;
    if (!state || !moves || (cfg->N > 0 && !table)) return PISA_E_INVALID;
    if (moves_words < kMovesHead + 2 * (int64_t)(pages->P / 2)) return PISA_E_INVALID;
    if (!aligned(state, 16) || !aligned(table, 4) || !aligned(moves, 4)) return PISA_E_ALIGNMENT;
    return cuda_status(launch_pages_compact(state, table, moves, pages->P / 2, cfg->B, pages->P,
                                            (int)width(cfg, pages), (cudaStream_t)stream));
}

int pisa_pages_copy(const pisa_cfg* cfg, const pisa_pages* pages, const int32_t* moves, int64_t moves_words, void* K,
                    void* V, void* stream) {
    const int s = check(cfg, pages);
    if (s) return s;
    if (!moves || !K || !V || K == V || moves_words < kMovesHead) return PISA_E_INVALID;
    if (!aligned(K, 16) || !aligned(V, 16) || !aligned(moves, 4)) return PISA_E_ALIGNMENT;
    int64_t most = (moves_words - kMovesHead) / 2;
    if (most > pages->P) most = pages->P;
    if (most == 0) return PISA_OK;
    const int64_t page_bytes = (int64_t)cfg->Hkv * pages->S * cfg->d * elem_bytes(cfg);
    return cuda_status(launch_pages_copy(moves, (int)most, K, V, page_bytes, pages->P, sm_count(), (cudaStream_t)stream));
}

int pisa_paged_append(const pisa_cfg* cfg, const pisa_pages* pages, const void* k_new, const void* v_new, int T,
                      const int32_t* len, const int32_t* count, const int32_t* table, void* K, void* V, void* stream) {
    const int s = check(cfg, pages);
    if (s) return s;
    if (T < 0) return PISA_E_INVALID;
    if (T == 0 || cfg->N == 0) return PISA_OK;
    if (!k_new || !v_new || !len || !count || !table || !K || !V || K == V) return PISA_E_INVALID;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(len, 4) ||
        !aligned(count, 4) || !aligned(table, 4))
        return PISA_E_ALIGNMENT;
    const int row_bytes = cfg->d * elem_bytes(cfg);
    const int64_t tiles = ((int64_t)cfg->Hkv * T * (row_bytes / 16) + 255) / 256;
    if (tiles * cfg->B >= ((int64_t)1 << 31)) return PISA_E_UNSUPPORTED;
    return cuda_status(launch_paged_append(row_bytes, k_new, v_new, T, count, K, V, params(cfg, pages, table, len),
                                           (cudaStream_t)stream));
}

int64_t pisa_paged_workspace_bytes(const pisa_cfg* cfg, const pisa_pages* pages) {
    const int s = check(cfg, pages);
    if (s) return s;
    // two parts a CTA: o, then maximum and sum, for each head of a group; and what there is to join
    return (int64_t)kPagedMaxCtas * (2 * (cfg->Hq / cfg->Hkv) * (cfg->d + 2) + 2) * (int64_t)sizeof(float);
}

int pisa_paged_attn(const pisa_cfg* cfg, const pisa_pages* pages, const void* q, const void* k_new, const void* v_new,
                    void* K, void* V, const int32_t* table, const int32_t* len, void* o, float* lse, void* workspace,
                    size_t workspace_bytes, void* stream) {
    const int s = check(cfg, pages);
    if (s) return s;
    if (cfg->causal != 1) return PISA_E_INVALID;  // the new token sees only the past
    if ((int64_t)cfg->B * cfg->Hkv * (cfg->N / 32 + 2) >= ((int64_t)1 << 31)) return PISA_E_UNSUPPORTED;  // 32-bit list of tiles
    if (cfg->N == 0) return PISA_OK;
    if (!q || !K || !V || K == V || !table || !len || !o || !workspace) return PISA_E_INVALID;
    if ((k_new == nullptr) != (v_new == nullptr)) return PISA_E_INVALID;
    if (workspace_bytes < (size_t)pisa_paged_workspace_bytes(cfg, pages)) return PISA_E_INVALID;
    if (!aligned(q, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(K, 16) || !aligned(V, 16) ||
        !aligned(o, 16) || !aligned(table, 4) || !aligned(len, 4) || !aligned(lse, 4) || !aligned(workspace, 16))
        return PISA_E_ALIGNMENT;
    return cuda_status(launch_paged_attn(cfg->dtype, cfg->d, q, k_new, v_new, K, V, o, lse, workspace,
                                         params(cfg, pages, table, len), sm_count(), (cudaStream_t)stream));
}

int pisa_paged_build_pyramid(const pisa_cfg* cfg, const pisa_pages* pages, const void* K, const int32_t* table,
                             const int32_t* len, float* pyr, void* stream) {
    const int s = check(cfg, pages);
    if (s) return s;
    if (pages->S % cfg->C != 0) return PISA_E_UNSUPPORTED;
    if (cfg->N == 0) return PISA_OK;
    if (!K || !table || !len || !pyr) return PISA_E_INVALID;
    if (!aligned(K, 16) || !aligned(pyr, 16) || !aligned(table, 4) || !aligned(len, 4)) return PISA_E_ALIGNMENT;
    if ((int64_t)cfg->B * cfg->Hkv > 65535) return PISA_E_UNSUPPORTED;  // one grid row per (b, kv-head)
    PagedPoolParams p;
    p.B = cfg->B; p.Hkv = cfg->Hkv; p.N = cfg->N; p.C = cfg->C;
    p.k_rows = cfg->N;
    p.len = len;
    make_geom(cfg->N, cfg->C, &p.geom);
    p.table = table; p.S = pages->S; p.P = pages->P; p.W = (int)width(cfg, pages);
    return cuda_status(launch_paged_pool(cfg->dtype, cfg->d, K, pyr, p, (cudaStream_t)stream));
}

int pisa_paged_pyramid_append(const pisa_cfg* cfg, const pisa_pages* pages, const void* k_new, const void* v_new, void* K,
                              void* V, const int32_t* table, const int32_t* len, float* pyr, void* stream) {
    const int s = check(cfg, pages);
    if (s) return s;
    if (pages->S % cfg->C != 0) return PISA_E_UNSUPPORTED;
    if (cfg->N == 0) return PISA_OK;
    if (!k_new || !v_new || !K || !V || K == V || !table || !len || !pyr) return PISA_E_INVALID;
    if (!aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(pyr, 16) ||
        !aligned(table, 4) || !aligned(len, 4))
        return PISA_E_ALIGNMENT;
    return cuda_status(launch_paged_pyramid_append(cfg->dtype, cfg->d, K, V, pyr, k_new, v_new, len,
                                                   decode_params(cfg, pages, table), (cudaStream_t)stream));
}

int pisa_paged_decode_step(const pisa_cfg* cfg, const pisa_pages* pages, const void* q_new, const void* k_new,
                           const void* v_new, void* K, void* V, const int32_t* table, const int32_t* len, float* pyr,
                           int32_t* idx, void* o, void* stream) {
    const int s = check(cfg, pages);
    if (s) return s;
    if (cfg->causal != 1) return PISA_E_INVALID;
    if (pages->S % cfg->C != 0) return PISA_E_UNSUPPORTED;
    if (cfg->N == 0) return PISA_OK;
    if (!q_new || !k_new || !v_new || !K || !V || K == V || !table || !len || !pyr || !idx || !o) return PISA_E_INVALID;
    if (!aligned(q_new, 16) || !aligned(k_new, 16) || !aligned(v_new, 16) || !aligned(K, 16) || !aligned(V, 16) ||
        !aligned(pyr, 16) || !aligned(o, 16) || !aligned(table, 4) || !aligned(len, 4) || !aligned(idx, 4))
        return PISA_E_ALIGNMENT;
    return cuda_status(launch_paged_step(cfg->dtype, cfg->d, q_new, k_new, v_new, K, V, len, pyr, idx, o,
                                         decode_params(cfg, pages, table), (cudaStream_t)stream));
}

}  // extern "C"
