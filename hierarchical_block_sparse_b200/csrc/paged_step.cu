// paged_step.cu -- the sparse decode step (close reading §5.1, §5.3) over a paged cache.
//
// One CTA of 4 or 8 warps per (sequence, KV head), in four phases:
//   1. append and the walk of the internal levels, as in decode.cu (shared code);
//   2. the keys of every candidate leaf stream past the group's queries; the logits stay
//      in shared memory (32 leaves x C keys x G heads). The warps take tiles of KT keys in
//      turn, each through a ring of its own, with no barrier in between;
//   3. log-sum-exps from those logits, and the final choice;
//   4. the values of the kept leaves alone stream past 2^(z - Z).
// decode.cu sums a key's products on the CUDA cores with the queries read from
// shared memory, G times for every element, and merges softmax states a tile at a
// time: from G = 4 on that is what its time goes to. Here phases 2 and 4 cost 16
// tensor-core products a 16 keys (fp32: the queries stay in registers) and the
// softmax is taken once (8 KV heads, decode.cu's kernel over pages against this one): 64
// sequences of 16 K tokens 136 -> 83 us (84% of the HBM floor); 32 of 665 tokens with groups of
// 8 178 -> 33 us (fp32: 239 -> 66); 8 of 32 K with groups of 16 422 -> 71 us. What bounds it is the
// chain of dependent phases: about 13 us of walk, one level after another, in which HBM is idle.
#include "pisa_decode.cuh"
#include "pisa_paged.cuh"
#include "pisa_tiles.cuh"

namespace pisa {

namespace {

// floats a head's logits of one leaf take: whole tiles, and 4 so that heads fall into different banks
__host__ __device__ constexpr int logit_stride(int C, int kt) { return (C + kt - 1) / kt * kt + 4; }

template <class Tile, int kWarps, int kStages>
size_t step_smem(int C, int K) {
    const size_t ring = (size_t)kWarps * kStages * kTileBytes;
    const size_t slots = sizeof(float) * kWarps * Tile::G * (Tile::D + 1);
    const size_t scratch = (size_t)(kWarps - 1 + kMaxLevels) * Tile::D * sizeof(float);  // the append's
    size_t head = ring > slots ? ring : slots;
    if (scratch > head) head = scratch;
    return (head + 15) / 16 * 16 + sizeof(float) * ((size_t)2 * K * Tile::G * logit_stride(C, Tile::KT) + kWarps * Tile::kWeighFloats);
}

// CTAs of one SM that the registers are cut for
template <int G, int kWarps, int kStages>
constexpr int step_blocks() {
    return kWarps == 8 ? (kStages == 2 && G <= 4 ? 2 : 1) : G <= 4 ? 4 : G <= 8 ? 3 : 2;
}

template <class Tile, int kWarps, int kStages>
__global__ void __launch_bounds__(kWarps * 32, step_blocks<Tile::G, kWarps, kStages>()) paged_step_kernel(
    const typename Tile::T* __restrict__ q_new, const typename Tile::T* __restrict__ k_new,
    const typename Tile::T* __restrict__ v_new, typename Tile::T* __restrict__ K, typename Tile::T* __restrict__ V,
    const int32_t* __restrict__ len, float* __restrict__ pyr, int32_t* __restrict__ idx, typename Tile::T* __restrict__ out,
    int z_at, PagedDecodeParams p) {
    using T = typename Tile::T;
    constexpr int D = Tile::D, G = Tile::G, KT = Tile::KT, kThreads = kWarps * 32;
    constexpr int CPR = Tile::RowBytes / 16, RPI = 32 / CPR;
    extern __shared__ __align__(128) uint8_t dyn[];  // rings (append: scratch; at the end: slots), logits, scratch
    __shared__ __align__(16) float s_q[G][D];
    __shared__ WalkShared<G> s_walk;
    __shared__ float s_lse[32][G];
    __shared__ int s_sel[32], s_slot[32], s_row[32], s_kj[32];
    __shared__ int s_nlist;
    __shared__ float s_Z[G];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x, b = unit / p.Hkv, kvh = unit % p.Hkv;
    float* z = reinterpret_cast<float*>(dyn + z_at);
    const int zs = logit_stride(p.C, KT);
    float* scratch = z + 2 * p.K * G * zs + warp * Tile::kWeighFloats;
    const int t = len[b] - 1;
    auto leaf_row = [&](int leaf) -> int {  // its first row of the pool (pages hold whole leaves); -1: no page
        const int tok = leaf * p.C;
        const int page = __ldg(p.table + (size_t)b * p.W + tok / p.S);
        return (unsigned)page < (unsigned)p.P ? (page * p.Hkv + kvh) * p.S + tok % p.S : -1;
    };
    const int new_row = t >= 0 && t < p.N ? leaf_row(t / p.C) : -1;
    const size_t head0 = (size_t)b * p.Hq + (size_t)kvh * G;
    if (new_row < 0) {
        if (tid < p.K) idx[(size_t)unit * p.K + tid] = -1;
        for (int i = tid; i < G * D; i += kThreads) out[head0 * D + i] = (T)0.f;
        return;
    }
    const int n_keys = t + 1;
    float* P = pyr + (int64_t)unit * p.geom.rows * D;
    const Forced F(t, p.C, 1, p.forced_mask);
    for (int i = tid; i < G * D; i += kThreads) s_q[i / D][i % D] = (float)q_new[head0 * D + i] * p.qscale;
    __syncthreads();
    // the append runs on the other warps while warp 0 passes the first levels, which never read what it rewrites
    if (warp >= 1)
        append_unit<T, D, kWarps - 1>(K + (size_t)new_row * D, V + (size_t)new_row * D, P, k_new + (size_t)unit * D,
                                      v_new + (size_t)unit * D, t, p, warp - 1, lane, reinterpret_cast<float*>(dyn), 1);
    int cand = 0;  // warp 0's walk state
    walk_levels<D, G, kThreads>(P, s_q, s_walk, n_keys, t, F, p, tid, cand);
    if (warp == 0) {
        const LevelState s = level_state(cand, 1, p.C, n_keys, t, 1, F);
        if (s.valid) {
            const int j = __popc(s.vmask & ((1u << lane) - 1u));
            s_sel[j] = cand;
            s_slot[j] = lane;
            s_row[j] = leaf_row(cand);
        }
        if (lane == 0) s_nlist = s.n;
    }
    Tile tile;
    tile.load_q(q_new + head0 * D, p.qscale, lane);
    tile.reset();
    __syncthreads();

    const int tpl = (p.C + KT - 1) / KT;  // tiles a leaf
    const int nlist = s_nlist;
    const uint32_t ring = tc::smem_u32(dyn) + warp * kStages * kTileBytes;
    auto rows_of = [&](int j) { return s_row[j] < 0 ? 0 : min(p.C, n_keys - s_sel[j] * p.C); };  // keys of scored leaf j
    // streams every kWarps-th of `tiles` through this warp's ring; at(i, j, r0): tile i is rows r0.. of scored leaf j
    auto stream = [&](const T* pool, int tiles, auto at, auto use) {
        auto issue = [&](int i, int stage) {
            if (i < tiles) {
                int j, r0;
                at(i, j, r0);
                const int rows = rows_of(j) - r0, c = lane % CPR;
                const T* src = pool + (size_t)(max(s_row[j], 0) + r0) * D + c * (16 / sizeof(T));
                const uint32_t dst = ring + stage * kTileBytes;
#pragma unroll
                for (int u = 0; u < KT / RPI; ++u) {
                    const int r = u * RPI + lane / CPR;
                    cp_async16_if(dst + ring_off<KT>(r, c), r < rows ? src + (size_t)r * D : pool, r < rows);
                }
            }
            tc::cp_async_commit();
        };
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) issue(warp + s * kWarps, s);
        int stage = 0, fill = kStages - 1;
        for (int i = warp; i < tiles; i += kWarps) {
            issue(i + (kStages - 1) * kWarps, fill);
            tc::cp_async_wait_group<kStages - 1>();
            __syncwarp();
            int j, r0;
            at(i, j, r0);
            use(ring + stage * kTileBytes, j, r0);
            __syncwarp();  // the stage is refilled next
            stage = stage + 1 == kStages ? 0 : stage + 1;
            fill = fill + 1 == kStages ? 0 : fill + 1;
        }
    };

    stream(
        K, nlist * tpl, [&](int i, int& j, int& r0) { j = i / tpl; r0 = (i - j * tpl) * KT; },
        [&](uint32_t buf, int j, int r0) { tile.logits(buf, p.qscale, z + (size_t)j * G * zs + r0, zs, lane); });
    __syncthreads();

    // log-sum-exp of every (leaf, head), 8 lanes each
    for (int i0 = 0; i0 < nlist * G; i0 += kThreads / 8) {
        const int i = i0 + tid / 8, j = i / G, h = i - j * G;
        const bool mine = i < nlist * G;
        const int n = mine ? rows_of(j) : 0;
        const float* zr = z + ((size_t)j * G + h) * zs;
        float m = -INFINITY, e = 0.f;
        for (int k = lane % 8; k < n; k += 8) m = fmaxf(m, zr[k]);
#pragma unroll
        for (int w = 1; w < 8; w <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, w));
        const float from = m == -INFINITY ? 0.f : m;  // keys of -inf logits alone: a sum of 0
        for (int k = lane % 8; k < n; k += 8) e += exp2f(zr[k] - from);
#pragma unroll
        for (int w = 1; w < 8; w <<= 1) e += __shfl_xor_sync(kFull, e, w);
        if (mine && lane % 8 == 0) s_lse[s_slot[j]][h] = n > 0 ? m + log2f(e) : -INFINITY;
    }
    __syncthreads();
    if (warp == 0) keep_leaves<G>(cand, n_keys, t, F, p, lane, s_lse, s_lse, idx + (size_t)unit * p.K, s_walk.cand, s_kj, s_nlist, s_Z);
    __syncthreads();

    stream(
        V, s_nlist * tpl,
        [&](int i, int& j, int& r0) {
            const int k = i / tpl;
            j = s_kj[k];
            r0 = (i - k * tpl) * KT;
        },
        [&](uint32_t buf, int j, int r0) {
            tile.weigh(buf, z + (size_t)j * G * zs + r0, zs, s_Z, rows_of(j) - r0, lane, scratch);
        });
    tc::cp_async_wait_all();
    __syncthreads();  // the rings are free
    float* slots = reinterpret_cast<float*>(dyn);
    constexpr int kSlot = G * (D + 1);
    tile.put_sums(slots + warp * kSlot, lane);
    __syncthreads();
    for (int i = tid; i < G * D; i += kThreads) {
        float num = 0.f, den = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            num += slots[w * kSlot + i];
            den += slots[w * kSlot + G * D + i / D];
        }
        out[head0 * D + i] = (T)(den > 0.f || den != den ? num / den : 0.f);  // NaN stays NaN; no key counted: 0
    }
}

template <class Tile, int kWarps, int kStages>
cudaError_t launch_shape(const void* q, const void* k_new, const void* v_new, void* K, void* V, const int32_t* len,
                         float* pyr, int32_t* idx, void* o, const PagedDecodeParams& p, cudaStream_t st, bool* taken) {
    using T = typename Tile::T;
    const size_t smem = step_smem<Tile, kWarps, kStages>(p.C, p.K);
    // static: queries, dots, log-sum-exps; all of an SM's 227 KB at most
    const size_t fixed = sizeof(float) * (Tile::G * Tile::D + 97 * Tile::G) + 2048;
    *taken = smem + fixed <= (size_t)227 * 1024;
    if (!*taken) return cudaSuccess;
    auto kern = paged_step_kernel<Tile, kWarps, kStages>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(kern, 227 * 1024 - (int)fixed, done);
    if (e != cudaSuccess) return e;
    const int z_at = (int)(smem - sizeof(float) * ((size_t)2 * p.K * Tile::G * logit_stride(p.C, Tile::KT) + kWarps * Tile::kWeighFloats));
    kern<<<(unsigned)(p.B * p.Hkv), kWarps * 32, smem, st>>>((const T*)q, (const T*)k_new, (const T*)v_new, (T*)K, (T*)V, len,
                                                             pyr, idx, (T*)o, z_at, p);
    return cudaGetLastError();
}

// Up to one unit an SM: 8 warps and a longer ring each, for a CTA has its SM alone (64 units
// at 32 K tokens: 45 us with 4 warps, 31 with 8; groups of 4: 53 and 38, of 16: 92 and 71). Up to two: 8
// warps where two such CTAs fit (G <= 4; 256 units at 8 K tokens, groups of 4: 64 us with 4 warps, 52 with
// 8; with groups of 8, where one fits, 75 and 90). More: 4 warps, 4 CTAs (512 units at 16 K tokens: 83 us;
// 94 with 8 warps, 120 with rings of 3 stages, which let 3 CTAs share an SM).
template <class Tile>
cudaError_t launch_step(const void* q, const void* k_new, const void* v_new, void* K, void* V, const int32_t* len,
                        float* pyr, int32_t* idx, void* o, const PagedDecodeParams& p, cudaStream_t st, bool* taken) {
    const int64_t units = (int64_t)p.B * p.Hkv, sms = sm_count();
    *taken = false;
    cudaError_t e = cudaSuccess;
    if (units <= sms) e = launch_shape<Tile, 8, 3>(q, k_new, v_new, K, V, len, pyr, idx, o, p, st, taken);
    if (!*taken && e == cudaSuccess && units <= (Tile::G <= 4 ? 2 : 1) * sms)
        e = launch_shape<Tile, 8, 2>(q, k_new, v_new, K, V, len, pyr, idx, o, p, st, taken);
    if (!*taken && e == cudaSuccess) e = launch_shape<Tile, 4, 2>(q, k_new, v_new, K, V, len, pyr, idx, o, p, st, taken);
    return e;
}

template <int D, int G>
cudaError_t launch_dtype(int dtype, const void* q, const void* k_new, const void* v_new, void* K, void* V,
                         const int32_t* len, float* pyr, int32_t* idx, void* o, const PagedDecodeParams& p, cudaStream_t st,
                         bool* taken) {
    if (dtype == 1) return launch_step<MmaTile<D, G>>(q, k_new, v_new, K, V, len, pyr, idx, o, p, st, taken);
    return launch_step<FmaTile<D, G>>(q, k_new, v_new, K, V, len, pyr, idx, o, p, st, taken);
}

template <int D>
cudaError_t launch_group(int dtype, const void* q, const void* k_new, const void* v_new, void* K, void* V,
                         const int32_t* len, float* pyr, int32_t* idx, void* o, const PagedDecodeParams& p, cudaStream_t st,
                         bool* taken) {
    switch (p.Hq / p.Hkv) {
        case 1: return launch_dtype<D, 1>(dtype, q, k_new, v_new, K, V, len, pyr, idx, o, p, st, taken);
        case 2: return launch_dtype<D, 2>(dtype, q, k_new, v_new, K, V, len, pyr, idx, o, p, st, taken);
        case 4: return launch_dtype<D, 4>(dtype, q, k_new, v_new, K, V, len, pyr, idx, o, p, st, taken);
        case 8: return launch_dtype<D, 8>(dtype, q, k_new, v_new, K, V, len, pyr, idx, o, p, st, taken);
        case 16: return launch_dtype<D, 16>(dtype, q, k_new, v_new, K, V, len, pyr, idx, o, p, st, taken);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

// The step by this kernel where its logits fit in shared memory and leaves are ranked by
// their log-sum-exp, else by decode.cu's.
cudaError_t launch_paged_step(int dtype, int d, const void* q, const void* k_new, const void* v_new, void* K, void* V,
                              const int32_t* len, float* pyr, int32_t* idx, void* o, const PagedDecodeParams& p,
                              cudaStream_t st) {
    if (p.variant == PISA_SCORE_LSE) {
        bool taken = false;
        const cudaError_t e = d == 128 ? launch_group<128>(dtype, q, k_new, v_new, K, V, len, pyr, idx, o, p, st, &taken)
                                       : launch_group<64>(dtype, q, k_new, v_new, K, V, len, pyr, idx, o, p, st, &taken);
        if (taken || e != cudaSuccess) return e;
    }
    return launch_paged_decode(dtype, d, q, k_new, v_new, K, V, len, pyr, idx, o, p, st);
}

}  // namespace pisa
