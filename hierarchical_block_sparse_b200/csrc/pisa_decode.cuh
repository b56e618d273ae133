// pisa_decode.cuh -- device code of the decode step that its kernels share: the
// append to one head's cache and pyramid, the walk of the internal levels, and the
// final choice of leaves.
#pragma once

#include "pisa_internal.h"
#include "pisa_walk.cuh"

namespace pisa {

// named barrier over `count` threads (a multiple of 32)
__device__ __forceinline__ void bar_sync(int id, int count) {
    asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(count) : "memory");
}

// Summaries' update of one (b, kv-head) for the row at n: NWA warps (wi =
// this warp's index among them) write the new key/value row, fetch the leaf's
// cached rows before n (Kl, Vl: the leaf's first rows; summed per warp,
// INFLIGHT loads in flight per lane)
// and the sibling of each ancestor into `scratch` ((NWA + kMaxLevels) x D
// floats of shared memory) -- none of which depends on the new row -- meet on
// named barrier `bar`, and warp 0 of them runs the chain leaf -> root.
template <typename T, int D, int NWA>
__device__ __forceinline__ void append_unit(T* Kl, T* Vl, float* P, const T* krow, const T* vrow, int64_t n,
                                            const DecodeParams& p, int wi, int lane, float* scratch, int bar) {
    constexpr int VD = D / 32;
    constexpr int INFLIGHT = 8;
    float* s_part = scratch;            // [NWA][D]
    float* s_sib = scratch + NWA * D;   // [kMaxLevels][D]
    float kn[VD];
    Ld<T, VD>::run(krow + lane * VD, kn);
    const int64_t leaf = n / p.C, lo = leaf * p.C;
    if (wi == 0) {
        float vn[VD];
        Ld<T, VD>::run(vrow + lane * VD, vn);
        store_vec<T, VD>(Kl + (n - lo) * D + lane * VD, kn);
        store_vec<T, VD>(Vl + (n - lo) * D + lane * VD, vn);
    }
    float acc[VD];
#pragma unroll
    for (int e = 0; e < VD; ++e) acc[e] = 0.f;
    for (int64_t r0 = lo + wi; r0 < n; r0 += NWA * INFLIGHT) {
        float x[INFLIGHT][VD];
#pragma unroll
        for (int i = 0; i < INFLIGHT; ++i) {
            const int64_t r = r0 + (int64_t)i * NWA;
            if (r < n) {
                Ld<T, VD>::run(Kl + (r - lo) * D + lane * VD, x[i]);
            } else {
#pragma unroll
                for (int e = 0; e < VD; ++e) x[i][e] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < INFLIGHT; ++i)
#pragma unroll
            for (int e = 0; e < VD; ++e) acc[e] += x[i][e];
    }
#pragma unroll
    for (int e = 0; e < VD; ++e) s_part[wi * D + lane * VD + e] = acc[e];
    const int64_t len = n + 1;
    for (int l = 1 + wi; l < p.geom.L; l += NWA) {
        const int64_t sib = (leaf >> (l - 1)) ^ 1;
        if (sib * ((int64_t)p.C << (l - 1)) < len) {
            float sv[VD];
            Ld<float, VD>::run(P + (p.geom.off[l] + sib) * D + lane * VD, sv);
#pragma unroll
            for (int e = 0; e < VD; ++e) s_sib[(l - 1) * D + lane * VD + e] = sv[e];
        }
    }
    bar_sync(bar, NWA * 32);
    if (wi != 0) return;
    // leaf mean over [leaf*C, n]
    float m[VD];
    const float inv = 1.f / (float)(n - lo + 1);
#pragma unroll
    for (int e = 0; e < VD; ++e) {
        float sum = kn[e];
#pragma unroll
        for (int w = 0; w < NWA; ++w) sum += s_part[w * D + lane * VD + e];
        m[e] = sum * inv;
    }
    store_vec<float, VD>(P + (p.geom.off[1] + leaf) * D + lane * VD, m);
    // ancestors: mean of the existing children at length n + 1
    int64_t node = leaf;
    for (int l = 1; l < p.geom.L; ++l) {
        const int64_t sib = node ^ 1;
        if (sib * ((int64_t)p.C << (l - 1)) < len) {
#pragma unroll
            for (int e = 0; e < VD; ++e) m[e] = (m[e] + s_sib[(l - 1) * D + lane * VD + e]) * 0.5f;
        }
        node >>= 1;
        store_vec<float, VD>(P + (p.geom.off[l + 1] + node) * D + lane * VD, m);
    }
}

template <int G>
struct WalkShared {
    int cand[32];
    float dot[64][G];
    unsigned need;
    int level;
};

// The internal levels for one query group, by a CTA of NT threads (s_q: the scaled
// queries). On return `cand` of warp 0's lanes holds the level-1 candidates.
template <int D, int G, int NT>
__device__ __forceinline__ void walk_levels(const float* P, const float (&s_q)[G][D], WalkShared<G>& sm, int64_t n_keys,
                                            int64_t t, const Forced& F, const DecodeParams& p, int tid, int& cand) {
    // ---- internal levels. Warp 0 carries the walk (lane c = candidate c,
    // valid candidates in ascending node order) and passes alone through the
    // levels that need no dot products; at a scored level all threads compute
    // the <= 64 child dots into sm.dot.
    constexpr int TPRW = D / 16;      // threads per fp32 pyramid row
    constexpr int RowsW = NT / TPRW;  // pyramid rows per pass
    const int lane = tid & 31, warp = tid >> 5;
    cand = lane == 0 ? 0 : -1;
    int l = p.geom.L;
    for (;;) {
        if (warp == 0) {
            unsigned need = 0;
            for (; l >= 2; --l) {
                const LevelState s = level_state(cand, l, p.C, n_keys, t, 1, F);
                if (s.n <= p.K) {
                    const int parent = compact_by_rank(cand, s.vmask, lane >> 1);
                    cand = lane < 2 * s.n ? 2 * parent + (lane & 1) : -1;
                    continue;
                }
                const unsigned fmask = __ballot_sync(kFull, s.forced);
                if (__popc(fmask) >= p.K) {  // the forced nodes fill the budget
                    int id = cand;
                    const int kept = keep_topk_lane(id, s.forced ? INFINITY : -INFINITY, s.valid, p.K, lane);
                    const int parent = __shfl_sync(kFull, id, lane >> 1);
                    cand = lane < 2 * kept ? 2 * parent + (lane & 1) : -1;
                    continue;
                }
                need = s.vmask & ~fmask;
                break;
            }
            sm.cand[lane] = cand;
            if (lane == 0) {
                sm.level = l;
                sm.need = need;
            }
        }
        __syncthreads();
        const int lv = sm.level;
        if (lv < 2) break;
        {
            const unsigned need = sm.need;
            const int64_t span_child = (int64_t)p.C << (lv - 2);
            const float* child_lvl = P + p.geom.off[lv - 1] * D;
            const int sl = tid % TPRW;
#pragma unroll
            for (int r0 = 0; r0 < 64; r0 += RowsW) {
                const int rho = r0 + tid / TPRW, c = rho >> 1;
                const int64_t child = 2 * (int64_t)sm.cand[c] + (rho & 1);
                const bool ok = ((need >> c) & 1u) && child * span_child < n_keys;
                float acc[G];
#pragma unroll
                for (int h = 0; h < G; ++h) acc[h] = 0.f;
                if (ok) {
                    const float4* row = reinterpret_cast<const float4*>(child_lvl + child * D);
                    float4 x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = __ldg(row + sl + TPRW * k);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int e0 = (sl + TPRW * k) * 4;
#pragma unroll
                        for (int h = 0; h < G; ++h) {
                            const float4 qv = *reinterpret_cast<const float4*>(&s_q[h][e0]);
                            acc[h] = fmaf(qv.x, x[k].x, fmaf(qv.y, x[k].y, fmaf(qv.z, x[k].z, fmaf(qv.w, x[k].w, acc[h]))));
                        }
                    }
                }
#pragma unroll
                for (int o = 1; o < TPRW; o <<= 1)
#pragma unroll
                    for (int h = 0; h < G; ++h) acc[h] += __shfl_xor_sync(kFull, acc[h], o);
                if (sl == 0)
#pragma unroll
                    for (int h = 0; h < G; ++h) sm.dot[rho][h] = acc[h];
            }
        }
        __syncthreads();
        if (warp == 0) {  // scores (Eq.7, summed over the group: Eq.11) and the keep
            const LevelState s = level_state(cand, l, p.C, n_keys, t, 1, F);
            const bool mine = (sm.need >> lane) & 1u;
            float score = -INFINITY;
            if (mine) {
                const bool has1 = (2 * (int64_t)cand + 1) * ((int64_t)p.C << (l - 2)) < n_keys;
                score = 0.f;
#pragma unroll
                for (int h = 0; h < G; ++h)
                    score += pair_score(sm.dot[2 * lane][h], has1 ? sm.dot[2 * lane + 1][h] : -INFINITY, p.variant);
            }
            int id = cand;
            const int kept = keep_topk_lane(id, s.forced ? INFINITY : score, s.valid, p.K, lane);
            const int parent = __shfl_sync(kFull, id, lane >> 1);
            cand = lane < 2 * kept ? 2 * parent + (lane & 1) : -1;
            --l;
        }
    }
}

// Final Top-K by one warp (lane c: candidate leaf c, `rank` its score per head, s_lse its
// log-sum-exp): the kept leaves, ascending, to idx[0..K) and s_sel; s_kj: for each, its
// index among the scored leaves; s_Z: the normaliser per head. Returns this lane's leaf.
template <int G>
__device__ __forceinline__ int keep_leaves(int cand, int64_t n_keys, int64_t t, const Forced& F, const DecodeParams& p,
                                           int lane, const float (*rank)[G], const float (&s_lse)[32][G], int32_t* idx,
                                           int (&s_sel)[32], int (&s_kj)[32], int& s_nlist, float (&s_Z)[G]) {
    const LevelState s = level_state(cand, 1, p.C, n_keys, t, 1, F);
    float score = 0.f;  // summed over the group (Eq.11)
#pragma unroll
    for (int h = 0; h < G; ++h) score += s.valid ? rank[lane][h] : 0.f;
    int id = cand, kept;
    unsigned kmask;
    if (s.n <= p.K) {
        kmask = s.vmask;
        id = compact_by_rank(cand, s.vmask, lane);
        kept = s.n;
    } else {
        kept = keep_topk_lane(id, s.forced ? INFINITY : score, s.valid, p.K, lane);
        // kept-ness per candidate lane: the kept ids are in lanes 0..kept-1
        bool mine = false;
        for (int i = 0; i < kept; ++i) mine |= (__shfl_sync(kFull, id, i) == cand) && s.valid;
        kmask = __ballot_sync(kFull, mine);
    }
    const int out_id = lane < kept ? id : -1;
    if (lane < p.K) idx[lane] = out_id;
    if ((kmask >> lane) & 1u)  // kept candidate lane -> (its rank among the kept, among the scored)
        s_kj[__popc(kmask & ((1u << lane) - 1u))] = __popc(s.vmask & ((1u << lane) - 1u));
    s_sel[lane] = lane < p.K ? out_id : -1;
    if (lane == 0) s_nlist = min(kept, p.K);
#pragma unroll
    for (int h = 0; h < G; ++h) {
        const float x = ((kmask >> lane) & 1u) ? s_lse[lane][h] : -INFINITY;
        float m = x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        float e = x == -INFINITY ? 0.f : exp2f(x - m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) e += __shfl_xor_sync(kFull, e, o);
        if (lane == 0) s_Z[h] = e == 0.f ? INFINITY : m + log2f(e);  // logits of -inf alone: no key has weight
    }
    return out_id;
}

}  // namespace pisa
