// pisa_paged.cuh -- what the paged-cache kernels share: their parameter blocks and
// launchers, and the page state's layout.
#pragma once

#include <atomic>
#include <stdint.h>

#include "pisa_internal.h"

namespace pisa {

constexpr float kLn2 = 0.69314718055994531f;

// SMs of the current device (a fixed fact of it, looked up once)
inline int sm_count() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    int sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
        if (dev < 64) known[dev].store(sms, std::memory_order_relaxed);
    }
    return sms;
}

// shared memory above 48 KB: asked for once a device and kernel
template <class Kern>
inline cudaError_t allow_smem(Kern kern, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_relaxed) >> dev) & 1)) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
    return e;
}

// The attention's workspace holds two parts for each of at most this many CTAs.
constexpr int kPagedMaxCtas = 512;

// pages_reserve_kernel is one CTA that keeps its sequences in shared memory.
constexpr int kReserveMaxSeqs = 4096;

struct PageView {
    int S, P, W;           // tokens a page, pages in the pool, pages a sequence
    const int32_t* table;  // [B, W], -1 = no page
};

struct PagedParams : PageView {
    int B, Hq, Hkv, N;   // N: most tokens a sequence holds
    float qscale;        // log2(e) / sqrt(d)
    const int32_t* len;  // [B]
};

// the contiguous kernels' blocks, K and V being pools
struct PagedDecodeParams : DecodeParams, PageView {};
struct PagedPoolParams : PoolParams, PageView {};

// Page state, in int32 words (each part begins on a multiple of 4):
//   refs  [P]           sequences' entries that name the page; 0 = free
//   bits  [ceil(P/32)]  bit j of word i: page 32 i + j is free
//   then room for the calls themselves: old bits, live pages before each
//   word, and a page id for each page.
struct PageState {
    int64_t p4, b4;
    __host__ __device__ explicit PageState(int P) : p4(((int64_t)P + 3) / 4 * 4), b4((((int64_t)P + 31) / 32 + 3) / 4 * 4) {}
    __host__ __device__ int64_t bits() const { return p4; }
    __host__ __device__ int64_t old_bits() const { return p4 + b4; }
    __host__ __device__ int64_t before() const { return p4 + 2 * b4; }
    __host__ __device__ int64_t map() const { return p4 + 3 * b4 + 16; }
    __host__ __device__ int64_t words() const { return 2 * p4 + 3 * b4 + 16; }
};

// words in front of the (source, destination) pairs of a list of moves
constexpr int kMovesHead = 4;

// the GPU limits every call checks (api.cu): PISA_OK or the status to return
int check_gpu_cfg(const pisa_cfg* c);

cudaError_t launch_paged_attn(int dtype, int d, const void* q, const void* k_new, const void* v_new, void* K, void* V,
                              void* o, float* lse, void* ws, const PagedParams& p, int sms, cudaStream_t st);
cudaError_t launch_paged_append(int row_bytes, const void* k_new, const void* v_new, int T, const int32_t* count, void* K,
                                void* V, const PagedParams& p, cudaStream_t st);
cudaError_t launch_paged_pool(int dtype, int d, const void* K, float* pyr, const PagedPoolParams& p, cudaStream_t st);
// the sparse step: paged_step.cu's kernel, or decode.cu's (launch_paged_decode) where that does not fit
cudaError_t launch_paged_step(int dtype, int d, const void* q, const void* k_new, const void* v_new, void* K, void* V,
                              const int32_t* len, float* pyr, int32_t* idx, void* o, const PagedDecodeParams& p,
                              cudaStream_t st);
cudaError_t launch_paged_decode(int dtype, int d, const void* q, const void* k_new, const void* v_new, void* K, void* V,
                                const int32_t* len, float* pyr, int32_t* idx, void* o, const PagedDecodeParams& p,
                                cudaStream_t st);
cudaError_t launch_paged_pyramid_append(int dtype, int d, void* K, void* V, float* pyr, const void* k_new, const void* v_new,
                                        const int32_t* len, const PagedDecodeParams& p, cudaStream_t st);
cudaError_t launch_pages_init(int32_t* state, int32_t* table, int32_t* len, int B, int P, int W, cudaStream_t st);
cudaError_t launch_pages_reserve(const int32_t* add, int32_t* state, int32_t* table, int32_t* len, int32_t* grant,
                                 int32_t* moves, int B, int N, int S, int P, int W, cudaStream_t st);
cudaError_t launch_pages_fork(const int32_t* parent, int32_t* state, const int32_t* table, const int32_t* len,
                              int32_t* table_out, int32_t* len_out, int B, int P, int W, cudaStream_t st);
cudaError_t launch_pages_free(const int32_t* seqs, int n, int32_t* state, int32_t* table, int32_t* len, int B, int P,
                              int W, cudaStream_t st);
cudaError_t launch_pages_compact(int32_t* state, int32_t* table, int32_t* moves, int max_moves, int B, int P, int W,
                                 cudaStream_t st);
cudaError_t launch_pages_copy(const int32_t* moves, int max_moves, void* K, void* V, int64_t page_bytes, int P, int sms,
                              cudaStream_t st);

}  // namespace pisa
