// pisa_paged.cuh -- what the paged-cache kernels share: the parameter block of
// the attention, the page state's layout and the address of a token's row.
#pragma once

#include <atomic>
#include <stdint.h>

#include "pisa_device.cuh"

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

struct PagedParams {
    int B, Hq, Hkv, N;     // N: most tokens a sequence holds
    int S, P, W;           // tokens a page, pages in the pool, pages a sequence
    float qscale;          // log2(e) / sqrt(d)
    const int32_t* table;  // [B, W], -1 = no page
    const int32_t* len;    // [B]
};

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

}  // namespace pisa
