// paged.cu -- attention of one new token a sequence over a paged cache.
//
//   z_j = q . k_j / sqrt(d) over the len[b] cached keys;  o = sum_j e^(z_j) v_j / sum_j e^(z_j)
//
// One pass over the keys and values with a running reference and sum (in log2
// units). The work is a list of tiles of TK keys, ordered by (sequence, KV head,
// position); CTA c takes the c-th equal share of that list, whatever the lengths, so
// one long sequence and many short ones load the GPU alike. Beginning and ending a
// (sequence, KV head) unit costs about as much as a tile, which the list counts in
// front of the unit's own (kUnitCost). A unit that falls into one share is finished by
// its CTA; one that is cut leaves (max, sum, unnormalised o) of each part in the
// workspace, which paged_join_kernel joins in share order (the result depends on the
// lengths alone, not on timing).
//
// Few and short units (see launch_tile) go without list and join: a cluster of up
// to 8 CTAs takes one unit and joins its parts through its shared memory.
//
// Inside a CTA each of the 4 warps takes KT keys of a tile and streams them
// through a ring of its own (kStages x 8 KB), with no barrier before the unit ends: a
// warp that waits for memory holds up no other. The rows come by TMA where a page
// holds whole groups of KT rows, else by cp.async, which takes any page size (and
// starts sooner: the clusters use it).
//
// Bound by HBM: every byte is read once (16 sequences of 16 K tokens, 8 KV heads: 1.071 GB
// of DRAM reads for 1.068 GB of keys and values; tensor pipe 15%, issue slots 31% busy).
// 64 such sequences take 660 to 690 us, 256 K tokens of one 168 to 173 us, back to back (98
// to 94% and 98 to 95% of a copy's bandwidth, by the GPU). Both run at the board's power
// limit, so instructions cost time: heads as the 8 columns of a product instead of its 16
// rows took 64 sequences from 729 to 696 us, TMA instead of cp.async to 640; all 24 bits of
// the probabilities and rounded sums over tiles (pisa_tiles.cuh) added 3% and 1%.
#include <cooperative_groups.h>
#include <cuda.h>  // CUtensorMap

#include "pisa_internal.h"
#include "pisa_paged.cuh"
#include "pisa_tiles.cuh"

namespace cg = cooperative_groups;

namespace pisa {

namespace {

constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr int kStageBytes = 2 * kTileBytes;  // KT key rows, then KT value rows
constexpr int kUnitCost = 1;  // 0: 103.5 us, 1: 80.1, 2: 81.1, 4: 83.9 for 64 sequences of 0..15 K tokens, 32 / 8 heads
constexpr int kClusterTiles = 4;  // most tiles for a cluster's CTA (1 K tokens, 8 heads: 6.3 us, by the list 7.9 and a second
                                  // launch; 2 K: 8.7 and 8.9; 4 K, with 8 tiles a CTA: 13.4, by the list 10.3)

// rows [y, y + box) x 128 bytes from x (elements) of a pool into shared memory
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(tc::smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(tc::smem_u32(bar)), "r"(bytes)
                 : "memory");
}

// ---- the list of tiles ------------------------------------------------------------------

struct Share {
    int pos0;          // position of the unit's first tile in the list
    int b, h, t;       // sequence (-1: none), KV head and tile inside the unit (< 0: in front of its tiles)
    int n, nt;         // keys and tiles of sequence b
};

__device__ __forceinline__ int keys_of(const PagedParams& p, int b) { return min(max(p.len[b], 0), p.N); }

// positions a unit takes
__device__ __forceinline__ int span(int n, int tk) { return n > 0 ? (n + tk - 1) / tk + kUnitCost : 0; }

// (the host refuses caches whose list could pass 2^31 positions)
__device__ __forceinline__ int list_length(const PagedParams& p, int tk, int lane) {
    int sum = 0;
    for (int b = lane; b < p.B; b += 32) sum += span(keys_of(p, b), tk);
    return __reduce_add_sync(kFull, sum) * p.Hkv;
}

// where position x of the list lies; called by whole warps
__device__ __forceinline__ void locate(const PagedParams& p, int tk, int x, int lane, Share& s) {
    s.b = -1;
    int base = 0;  // positions (of one head) before this round of 32 sequences
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        const int n = b < p.B ? keys_of(p, b) : 0;
        const int len = span(n, tk);
        int end = len;
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) {
            const int y = __shfl_up_sync(kFull, end, w);
            if (lane >= w) end += y;
        }
        const int first = (base + end - len) * p.Hkv;
        const unsigned hit = __ballot_sync(kFull, len > 0 && x >= first && x < (base + end) * p.Hkv);
        if (hit) {
            const int at = __ffs(hit) - 1;
            const int f = __shfl_sync(kFull, first, at), one = __shfl_sync(kFull, len, at);
            s.b = b0 + at;
            s.n = __shfl_sync(kFull, n, at);
            s.nt = one - kUnitCost;
            s.h = (x - f) / one;
            s.pos0 = f + s.h * one + kUnitCost;
            s.t = x - s.pos0;
            return;
        }
        base += __shfl_sync(kFull, end, 31);
    }
}

// first sequence from b on that has keys (B: none)
__device__ __forceinline__ int next_seq(const PagedParams& p, int b, int& n) {
    while (b < p.B && (n = keys_of(p, b)) == 0) ++b;
    return b;
}

// The list of `total` positions in `shares` parts (at most as many, so that none is empty),
// share c from floor(total * c / shares) on: the longer ones are spread out. (With all of
// them in front, CTAs run in step through memory: 165 us instead of 158 for 256 K tokens.)
struct Cut {
    int total, shares, each, rest;
    __device__ __forceinline__ Cut(int n, int s) : total(n), shares(s), each(n / s), rest(n - n / s * s) {}
    __device__ __forceinline__ int begin(int c) const { return c * each + c * rest / shares; }
    // the share that holds position x
    __device__ __forceinline__ int of(int x) const { return (int)((((int64_t)x + 1) * shares - 1) / total); }
};

// What the join has to do at the beginning of a CTA's share: `parts` (0: nothing) from
// the CTA before it on, for the heads from output row `row` on.
struct JoinItem {
    int parts, row;
};

template <class Tile>
struct Smem {
    static constexpr int kSlotFloats = Tile::G * (Tile::D + 2);
    // merge slots: one a warp where they fit beside the ring twice an SM, else warps take turns
    static constexpr int kRoom = 115712 - kWarps * kStages * kStageBytes - kWarps * (Tile::kScratchFloats + 4) * 4 - 256;
    static constexpr int kSlots = 4 * kSlotFloats * 4 <= kRoom ? 4 : 2 * kSlotFloats * 4 <= kRoom ? 2 : 1;
    alignas(1024) uint8_t ring[kWarps][kStages][kStageBytes];
    float slot[kSlots][kSlotFloats];
    alignas(16) float scratch[kWarps][Tile::kScratchFloats + 4];
    unsigned mask[kWarps][kStages];
    uint64_t full[kWarps][kStages];  // TMA: a stage's rows have landed
    // a cluster's CTA: its part of the unit ([G][D] o, then m[G], l[G]), over the ring
    __device__ __forceinline__ float* fin() { return reinterpret_cast<float*>(&ring[0][0][0]); }
};

// what a kernel is: the list fed by cp.async, a unit a cluster, the list fed by TMA
enum Mode { kList, kCluster, kListTma };

template <class Tile, Mode MODE>
__global__ void __launch_bounds__(kWarps * 32, 2) paged_attn_kernel(
    const typename Tile::T* __restrict__ q, const typename Tile::T* __restrict__ k_new,
    const typename Tile::T* __restrict__ v_new, typename Tile::T* __restrict__ K, typename Tile::T* __restrict__ V,
    typename Tile::T* __restrict__ out, float* __restrict__ lse, float* __restrict__ part, PagedParams p,
    const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    using T = typename Tile::T;
    constexpr bool CLUSTER = MODE == kCluster, TMA = MODE == kListTma;
    constexpr int D = Tile::D, G = Tile::G, KT = Tile::KT, TK = kWarps * KT;
    constexpr int CPR = Tile::RowBytes / 16, RPI = 32 / CPR;  // chunks a row, rows a warp copies at once
    extern __shared__ __align__(1024) uint8_t raw[];
    Smem<Tile>& sm = *reinterpret_cast<Smem<Tile>*>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int grid = gridDim.x, cta = blockIdx.x;
    if constexpr (TMA) {
        if (lane == 0) {
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(&k_map) : "memory");
            asm volatile("prefetch.tensormap [%0];\n" ::"l"(&v_map) : "memory");
            for (int i = 0; i < kStages; ++i) tc::mbar_init(&sm.full[warp][i], 1);
            tc::fence_mbar_init();
        }
        __syncwarp();  // a warp's barriers are its own
    }

    Share at;
    int x1;  // the end of this CTA's share
    if constexpr (CLUSTER) {
        const int size = (int)cg::this_cluster().num_blocks(), unit = cta / size, rank = cta % size;
        at.b = unit / p.Hkv;
        at.h = unit % p.Hkv;
        at.n = keys_of(p, at.b);
        at.nt = (at.n + TK - 1) / TK;
        at.pos0 = 0;
        at.t = at.nt * rank / size;
        x1 = at.nt * (rank + 1) / size;
    } else {
        asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
        // empty sequences: nothing to attend to
        for (int b = cta; b < p.B; b += grid)
            if (keys_of(p, b) == 0) {
                for (int i = tid; i < p.Hq * D; i += kWarps * 32) out[(size_t)b * p.Hq * D + i] = (T)0.f;
                if (lse)
                    for (int i = tid; i < p.Hq; i += kWarps * 32) lse[(size_t)b * p.Hq + i] = -INFINITY;
            }
        const int total = list_length(p, TK, lane), shares = min(grid, total);
        JoinItem item = {0, 0};
        if (cta < shares) {
            const Cut cut(total, shares);
            x1 = cut.begin(cta + 1);
            locate(p, TK, cut.begin(cta), lane, at);
            // a unit cut here for the first time: its parts are this share's, the one before and
            // those up to the one that holds its last tile
            if (at.b >= 0 && at.t > 0 && cut.begin(cta - 1) <= at.pos0) {
                item.parts = cut.of(at.pos0 + at.nt - 1) - cta + 2;
                item.row = at.b * p.Hq + at.h * G;
            }
        }
        if (tid == 0) reinterpret_cast<JoinItem*>(part + (size_t)grid * 2 * G * (D + 2))[cta] = item;
        if (cta >= shares) return;
        at.t = max(at.t, 0);
        if (at.b < 0 || at.pos0 + at.t >= x1) return;
    }

    // ---- the loading side: its own place in the list, kStages - 1 tiles ahead
    int lb = at.b, lh = at.h, lt = at.t, ln = at.n, lnt = at.nt;
    int left = x1 - (at.pos0 + at.t);  // positions up to the share's end
    int page = -1;                     // of this lane's row of the next tile (lanes < KT)
    auto fetch = [&]() {
        if constexpr (TMA) {  // one page for all rows
            const int pos = lt * TK + warp * KT;
            page = left > 0 && pos < ln ? __ldg(p.table + (size_t)lb * p.W + pos / p.S) : -1;
            return;
        }
        const int pos = lt * TK + warp * KT + lane;
        page = left > 0 && lane < KT && pos < ln ? __ldg(p.table + (size_t)lb * p.W + pos / p.S) : -1;
    };
    // the token in hand lies in this warp's rows of tile t of sequence b (n keys; a length past N has none)
    auto fresh_at = [&](int b, int t, int n) {
        return k_new != nullptr && (n - 1) / TK == t && ((n - 1) % TK) / KT == warp && p.len[b] == n;
    };
    auto issue_rows = [&](int stage) {
        const int pos = lt * TK + warp * KT + lane;
        const bool live = lane < KT && pos < ln && page >= 0 && page < p.P;
        const int row = live ? (page * p.Hkv + lh) * p.S + pos % p.S : -1;  // of the pool (< 2^31)
        const unsigned mask = __ballot_sync(kFull, live);
        if (lane == 0) sm.mask[warp][stage] = mask;
        const uint32_t kbuf = tc::smem_u32(sm.ring[warp][stage]), vbuf = kbuf + kStageBytes / 2;
        const int c = lane % CPR;
        const bool fresh = fresh_at(lb, lt, ln);
#pragma unroll
        for (int i = 0; i < KT / RPI; ++i) {
            const int r = i * RPI + lane / CPR;
            const int src = __shfl_sync(kFull, row, r);
            const size_t e = (size_t)max(src, 0) * D + c * (16 / sizeof(T));
            const T *ks = K + e, *vs = V + e;
            if (fresh && lt * TK + warp * KT + r == ln - 1) {  // the token in hand: from its rows, and into its page
                const size_t u = ((size_t)lb * p.Hkv + lh) * D + c * (16 / sizeof(T));
                ks = k_new + u;
                vs = v_new + u;
                if (src >= 0) {
                    *reinterpret_cast<uint4*>(K + e) = __ldg(reinterpret_cast<const uint4*>(ks));
                    *reinterpret_cast<uint4*>(V + e) = __ldg(reinterpret_cast<const uint4*>(vs));
                }
            }
            cp_async16_if(kbuf + ring_off<KT>(r, c), ks, src >= 0);
            cp_async16_if(vbuf + ring_off<KT>(r, c), vs, src >= 0);
        }
    };
    auto issue_tma = [&](int stage) {
        const int pos = lt * TK + warp * KT;
        const bool live = pos < ln && (unsigned)page < (unsigned)p.P;
        const int row = live ? (page * p.Hkv + lh) * p.S + pos % p.S : 0;
        if (lane == 0) {
            const int rows = live ? min(KT, ln - pos) : 0;
            sm.mask[warp][stage] = rows == 32 ? kFull : (1u << rows) - 1u;
            uint64_t* bar = &sm.full[warp][stage];
            const uint32_t kbuf = tc::smem_u32(sm.ring[warp][stage]);
            mbar_expect(bar, live ? kStageBytes : 0);
            if (live) {
#pragma unroll
                for (int i = 0; i < Tile::RowBytes / 128; ++i) {
                    tma_rows(kbuf + i * KT * 128, &k_map, i * (128 / (int)sizeof(T)), row, bar);
                    tma_rows(kbuf + kStageBytes / 2 + i * KT * 128, &v_map, i * (128 / (int)sizeof(T)), row, bar);
                }
            }
        }
        if (live && fresh_at(lb, lt, ln) && lane < CPR) {  // into its page; the ring gets it when the stage is used
            const size_t u = ((size_t)lb * p.Hkv + lh) * D + lane * (16 / sizeof(T));
            const size_t e = (size_t)(row + (ln - 1) % KT) * D + lane * (16 / sizeof(T));
            *reinterpret_cast<uint4*>(K + e) = __ldg(reinterpret_cast<const uint4*>(k_new + u));
            *reinterpret_cast<uint4*>(V + e) = __ldg(reinterpret_cast<const uint4*>(v_new + u));
        }
    };
    auto issue = [&](int stage) {
        if (left > 0) {
            if constexpr (TMA) issue_tma(stage);
            else issue_rows(stage);
            --left;
            if (++lt == lnt) {
                lt = 0;
                left -= kUnitCost;
                if (++lh == p.Hkv) {
                    lh = 0;
                    lb = next_seq(p, lb + 1, ln);
                    if (lb == p.B) left = 0;
                    lnt = (ln + TK - 1) / TK;
                }
            }
            fetch();
        }
        if constexpr (!TMA) tc::cp_async_commit();
    };
    fetch();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    // ---- the computing side
    Tile tile;
    tile.reset();
    int b = at.b, h = at.h, t = at.t, n = at.n, nt = at.nt, t_first = at.t;
    auto query = [&](int bb, int hh) { return q + ((size_t)bb * p.Hq + (size_t)hh * G) * D; };
    tile.load_q(query(b, h), p.qscale, lane);
    int stage = 0, fill = kStages - 1;
    uint32_t parity = 0;  // TMA: of the round of stages in use
    bool failed = false;
    for (int x = at.pos0 + at.t; x < x1; ++x) {
        // the unit that follows, if it is this share's: its queries are fetched behind the last tile
        const bool next = t + 1 == nt && x + 1 + kUnitCost < x1;
        int b2 = b, h2 = h, n2 = n;
        if (next) {
            if (++h2 == p.Hkv) {
                h2 = 0;
                b2 = min(next_seq(p, b + 1, n2), p.B - 1);  // positions are left, so there is one
            }
            tile.fetch_q(query(b2, h2), lane);
        }
        const uint32_t kbuf = tc::smem_u32(sm.ring[warp][stage]);
        if constexpr (TMA) {
            const bool gave_up = !failed && !tc::mbar_wait(&sm.full[warp][stage], parity, nullptr, 0);
            if (__any_sync(kFull, gave_up)) {  // after about a second: no more copies, and those under way
                failed = true;                 // get as long again
                left = 0;
                for (int i = 0; i < kStages; ++i)
                    tc::mbar_wait(&sm.full[warp][(stage + i) % kStages], parity ^ (stage + i >= kStages), nullptr, 0);
            }
            const unsigned mask = sm.mask[warp][stage];
            if (failed) {
                tile.poison();  // the result is NaN
            } else if (mask != 0) {
                const int rows = __popc(mask);
                const bool fresh = fresh_at(b, t, n);
                if (rows < KT || fresh) {
                    // rows past the end may hold anything: their values count as zeros. The token in hand
                    // comes from its rows (its page may have been read before they were there).
                    for (int i = lane; i < (KT - rows) * CPR; i += 32)
                        *reinterpret_cast<uint4*>(sm.ring[warp][stage] + kStageBytes / 2 + ring_off<KT>(rows + i / CPR, i % CPR)) =
                            make_uint4(0u, 0u, 0u, 0u);
                    if (fresh && lane < CPR) {
                        const size_t u = ((size_t)b * p.Hkv + h) * D + lane * (16 / sizeof(T));
                        uint8_t* at_row = sm.ring[warp][stage] + ring_off<KT>((n - 1) % KT, lane);
                        *reinterpret_cast<uint4*>(at_row) = __ldg(reinterpret_cast<const uint4*>(k_new + u));
                        *reinterpret_cast<uint4*>(at_row + kStageBytes / 2) = __ldg(reinterpret_cast<const uint4*>(v_new + u));
                    }
                    tc::fence_async_smem();  // before the next TMA write of this stage
                    __syncwarp();
                }
                tile.step(kbuf, kbuf + kStageBytes / 2, mask, p.qscale, lane, sm.scratch[warp]);
            }
        } else {
            tc::cp_async_wait_group<kStages - 2>();
            __syncwarp();
            tile.step(kbuf, kbuf + kStageBytes / 2, sm.mask[warp][stage], p.qscale, lane, sm.scratch[warp]);
        }
        __syncwarp();
        issue(fill);
        if (++stage == kStages) {
            stage = 0;
            parity ^= 1;
        }
        fill = fill + 1 == kStages ? 0 : fill + 1;
        ++t;
        if (t < nt && x + 1 < x1) continue;
        // the unit, or this CTA's part of it, is through: merge the warps
        const bool whole = t_first == 0 && t == nt;
        __syncthreads();  // the slots' last contents have been read
        constexpr int NS = Smem<Tile>::kSlots;
#pragma unroll
        for (int r = 0; r < kWarps / NS; ++r) {
            if (warp / NS == r) tile.put(sm.slot[warp % NS], r > 0, lane);
            __syncthreads();
        }
        const size_t unit = (size_t)b * p.Hq + (size_t)h * G;
        for (int i = tid; i < G * D / 4; i += kWarps * 32) {
            const int hh = i / (D / 4), e = (i % (D / 4)) * 4;
            float ms[NS], M = -INFINITY;
#pragma unroll
            for (int w = 0; w < NS; ++w) {
                ms[w] = sm.slot[w][G * D + hh];
                M = fmaxf(M, ms[w]);
            }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < NS; ++w) {
                const float a = ms[w] == -INFINITY ? 0.f : exp2f(ms[w] - M);
                const float* x4 = &sm.slot[w][hh * D + e];
                sum += a * sm.slot[w][G * D + G + hh];
                acc.x += a * x4[0];
                acc.y += a * x4[1];
                acc.z += a * x4[2];
                acc.w += a * x4[3];
            }
            if constexpr (CLUSTER) {  // this CTA's part, in the ring (all its loads have been used)
                *reinterpret_cast<float4*>(&sm.fin()[hh * D + e]) = acc;
                if (e == 0) {
                    sm.fin()[G * D + hh] = M;
                    sm.fin()[G * D + G + hh] = sum;
                }
            } else if (whole) {
                const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;  // no key counted: 0
                const float r[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
                store_vec<T, 4>(out + (unit + hh) * D + e, r);
                if (lse && e == 0) lse[unit + hh] = lse2(M, sum) * kLn2;
            } else {
                // slot 0: a part that begins inside its unit; 1: one that ends inside it
                const size_t at_part = ((size_t)cta * 2 + (t_first == 0 ? 1 : 0)) * G + hh;
                *reinterpret_cast<float4*>(part + at_part * D + e) = acc;
                if (e == 0) {
                    float* ml = part + (size_t)grid * 2 * G * D + at_part * 2;
                    ml[0] = M;
                    ml[1] = sum;
                }
            }
        }
        if (!next) break;
        tile.reset();
        tile.take_q(query(b2, h2), p.qscale, lane);
        b = b2;
        h = h2;
        n = n2;
        nt = (n + TK - 1) / TK;
        t = t_first = 0;
        x += kUnitCost;
    }
    tc::cp_async_wait_all();
    if constexpr (CLUSTER) {
        if (at.t == x1)  // more CTAs than tiles: no part
            for (int i = tid; i < G * (D + 2); i += kWarps * 32) sm.fin()[i] = i / G == D ? -INFINITY : 0.f;
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        const int size = (int)cluster.num_blocks(), rank = cta % size;
        const size_t unit = (size_t)at.b * p.Hq + (size_t)at.h * G;
        for (int i = rank * kWarps * 32 + tid; i < G * D / 4; i += size * kWarps * 32) {
            const int hh = i / (D / 4), e = (i % (D / 4)) * 4;
            float M = -INFINITY, sum = 0.f;
            for (int r = 0; r < size; ++r) M = fmaxf(M, cluster.map_shared_rank(sm.fin(), r)[G * D + hh]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r = 0; r < size; ++r) {
                const float* f = cluster.map_shared_rank(sm.fin(), r);
                const float m = f[G * D + hh], a = m == -INFINITY ? 0.f : exp2f(m - M);
                const float4 v = *reinterpret_cast<const float4*>(f + hh * D + e);
                sum += a * f[G * D + G + hh];
                acc.x += a * v.x;
                acc.y += a * v.y;
                acc.z += a * v.z;
                acc.w += a * v.w;
            }
            const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
            const float r4[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
            store_vec<T, 4>(out + (unit + hh) * D + e, r4);
            if (lse && e == 0) lse[unit + hh] = lse2(M, sum) * kLn2;
        }
        cluster.sync();  // the others have read this CTA's part
    }
}

// Joins the parts of the units that more than one CTA had a share of. CTA (c, head): where
// share c is the first to begin inside a unit, the unit's parts are slot 1 of c - 1 and
// slot 0 of c, c + 1, ...
template <int G>
constexpr int join_warps() { return G <= 2 ? 16 : G <= 4 ? 8 : 4; }  // few heads, few CTAs: more warps each

template <typename T, int D, int G>
__global__ void __launch_bounds__(join_warps<G>() * 32) paged_join_kernel(T* __restrict__ out, float* __restrict__ lse,
                                                         const float* __restrict__ part) {
    constexpr int NW = join_warps<G>();
    __shared__ float s_m[NW], s_l[NW];
    __shared__ float4 s_o[NW][D / 4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int grid = gridDim.x, c = blockIdx.x, hh = blockIdx.y;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const JoinItem item = reinterpret_cast<const JoinItem*>(part + (size_t)grid * 2 * G * (D + 2))[c];
    const int parts = item.parts;
    if (parts == 0) return;
    const float* ml = part + (size_t)grid * 2 * G * D;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = -INFINITY, sum = 0.f;
    auto merge = [&](float m, float l, const float4& v) {
        const float mn = fmaxf(M, m), a = M == -INFINITY ? 0.f : exp2f(M - mn), b = m == -INFINITY ? 0.f : exp2f(m - mn);
        M = mn;
        sum = a * sum + b * l;
        acc.x = a * acc.x + b * v.x;
        acc.y = a * acc.y + b * v.y;
        acc.z = a * acc.z + b * v.z;
        acc.w = a * acc.w + b * v.w;
    };
    // every NW-th part a warp, 4 at once; the order is fixed, so the result does not depend on timing
    for (int i0 = warp; i0 < parts; i0 += 4 * NW) {
        float4 v[4];
        float2 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + NW * u;
            w[u] = make_float2(-INFINITY, 0.f);
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i >= parts) continue;
            const size_t r = ((size_t)(c - 1 + i) * 2 + (i == 0 ? 1 : 0)) * G + hh;
            w[u] = *reinterpret_cast<const float2*>(ml + r * 2);
            if (lane < D / 4) v[u] = *reinterpret_cast<const float4*>(part + r * D + lane * 4);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) merge(w[u].x, w[u].y, v[u]);
    }
    if (lane < D / 4) s_o[warp][lane] = acc;
    if (lane == 0) {
        s_m[warp] = M;
        s_l[warp] = sum;
    }
    __syncthreads();
    if (warp == 0) {
        for (int w = 1; w < min(NW, parts); ++w) merge(s_m[w], s_l[w], lane < D / 4 ? s_o[w][lane] : make_float4(0.f, 0.f, 0.f, 0.f));
        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        const float r[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
        const size_t u = (size_t)item.row + hh;
        if (lane < D / 4) store_vec<T, 4>(out + u * D + lane * 4, r);
        if (lse && lane == 0) lse[u] = lse2(M, sum) * kLn2;
    }
}

using PFN_encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// TMA's view of a pool: all rows of all pages, in boxes of `rows` x 128 bytes
bool row_map(CUtensorMap* map, const void* pool, const PagedParams& p, int rows, int d, int elem) {
    static const PFN_encode encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
        return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_encode>(fn) : nullptr;
    }();
    if (!encode) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)p.P * p.Hkv * p.S};
    const cuuint64_t strides[1] = {(cuuint64_t)d * elem};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / elem), (cuuint32_t)rows}, step[2] = {1, 1};
    return encode(map, elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                  const_cast<void*>(pool), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class Tile>
cudaError_t launch_tile(const void* q, const void* k_new, const void* v_new, void* K, void* V, void* o, float* lse,
                        float* part, const PagedParams& p, int sms, cudaStream_t st) {
    using T = typename Tile::T;
    constexpr int TK = kWarps * Tile::KT, D = Tile::D;
    const int smem = (int)sizeof(Smem<Tile>);
    const int64_t per_unit = ((int64_t)p.N + TK - 1) / TK, units = (int64_t)p.B * p.Hkv;
    const int64_t room = 2 * (int64_t)sms < kPagedMaxCtas ? 2 * (int64_t)sms : kPagedMaxCtas;  // two CTAs an SM

    // One cluster a unit: saves the look at all lengths and the second launch, but
    // gives a unit at most 8 CTAs, whatever its length.
    int size = 8;
    while (size > 1 && units * size > room) size /= 2;
    if (units <= room && per_unit <= (int64_t)size * kClusterTiles) {
        static std::atomic<uint64_t> done{0};
        auto kern = paged_attn_kernel<Tile, kCluster>;
        const cudaError_t e = allow_smem(kern, smem, done);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(units * size));
        cfg.blockDim = dim3(kWarps * 32);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = size;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kern, (const T*)q, (const T*)k_new, (const T*)v_new, (T*)K, (T*)V, (T*)o, lse,
                                  part, p, CUtensorMap{}, CUtensorMap{});
    }

    int64_t grid = units * (per_unit + kUnitCost);
    if (grid > room) grid = room;  // all resident at once
    cudaError_t e;
    CUtensorMap k_map{}, v_map{};
    if (p.S % Tile::KT == 0 && row_map(&k_map, K, p, Tile::KT, D, sizeof(T)) && row_map(&v_map, V, p, Tile::KT, D, sizeof(T))) {
        static std::atomic<uint64_t> done{0};
        auto kern = paged_attn_kernel<Tile, kListTma>;
        e = allow_smem(kern, smem, done);
        if (e != cudaSuccess) return e;
        kern<<<(unsigned)grid, kWarps * 32, smem, st>>>((const T*)q, (const T*)k_new, (const T*)v_new, (T*)K, (T*)V, (T*)o,
                                                        lse, part, p, k_map, v_map);
    } else {
        static std::atomic<uint64_t> done{0};
        auto kern = paged_attn_kernel<Tile, kList>;
        e = allow_smem(kern, smem, done);
        if (e != cudaSuccess) return e;
        kern<<<(unsigned)grid, kWarps * 32, smem, st>>>((const T*)q, (const T*)k_new, (const T*)v_new, (T*)K, (T*)V, (T*)o,
                                                        lse, part, p, k_map, v_map);
    }
    e = cudaGetLastError();
    if (e != cudaSuccess || per_unit == 1 || grid == 1) return e;  // no unit can be cut
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, Tile::G);
    cfg.blockDim = dim3(join_warps<Tile::G>() * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr;  // the join's launch overlaps the kernel above
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_join_kernel<T, Tile::D, Tile::G>, (T*)o, lse, (const float*)part);
}

template <int D, int G>
cudaError_t launch_dtype(int dtype, const void* q, const void* k_new, const void* v_new, void* K, void* V, void* o,
                         float* lse, float* part, const PagedParams& p, int sms, cudaStream_t st) {
    if (dtype == 1) return launch_tile<MmaTile<D, G>>(q, k_new, v_new, K, V, o, lse, part, p, sms, st);
    return launch_tile<FmaTile<D, G>>(q, k_new, v_new, K, V, o, lse, part, p, sms, st);
}

template <int D>
cudaError_t launch_group(int dtype, const void* q, const void* k_new, const void* v_new, void* K, void* V, void* o,
                         float* lse, float* part, const PagedParams& p, int sms, cudaStream_t st) {
    switch (p.Hq / p.Hkv) {
        case 1: return launch_dtype<D, 1>(dtype, q, k_new, v_new, K, V, o, lse, part, p, sms, st);
        case 2: return launch_dtype<D, 2>(dtype, q, k_new, v_new, K, V, o, lse, part, p, sms, st);
        case 4: return launch_dtype<D, 4>(dtype, q, k_new, v_new, K, V, o, lse, part, p, sms, st);
        case 8: return launch_dtype<D, 8>(dtype, q, k_new, v_new, K, V, o, lse, part, p, sms, st);
        case 16: return launch_dtype<D, 16>(dtype, q, k_new, v_new, K, V, o, lse, part, p, sms, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_paged_attn(int dtype, int d, const void* q, const void* k_new, const void* v_new, void* K, void* V,
                              void* o, float* lse, void* ws, const PagedParams& p, int sms, cudaStream_t st) {
    float* part = (float*)ws;
    if (d == 128) return launch_group<128>(dtype, q, k_new, v_new, K, V, o, lse, part, p, sms, st);
    if (d == 64) return launch_group<64>(dtype, q, k_new, v_new, K, V, o, lse, part, p, sms, st);
    return cudaErrorInvalidValue;
}

}  // namespace pisa
