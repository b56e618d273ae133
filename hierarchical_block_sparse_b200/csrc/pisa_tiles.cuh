// pisa_tiles.cuh -- one warp's tile of keys and values against the query heads of a
// group, in bf16 on the tensor cores (MmaTile) and in fp32 on the CUDA cores (FmaTile).
// The rows wait in shared memory, kTileBytes of keys and as many of values.
#pragma once

#include "pisa_device.cuh"
#include "tc.cuh"

namespace pisa {

constexpr int kTileBytes = 4096;
// A softmax's reference is set kRescale above the largest logit so far and moves only when a
// logit passes it, so most tiles need no rescaling; terms are at most 1, and those below
// 2^(kRescale - 126) of the largest vanish.
constexpr float kRescale = 8.f;
// the log-sum-exp in log2 units of terms that add up to `sum` at reference m
__device__ __forceinline__ float lse2(float m, float sum) { return (m - kRescale) + log2f(sum * 256.f); }
static_assert(kRescale == 8.f, "lse2 takes 2^kRescale");

__device__ __forceinline__ void cp_async16_if(uint32_t dst, const void* src, bool live) {
    const int bytes = live ? 16 : 0;  // 0: the 16 bytes become zeros, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), bf16
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same from zero
__device__ __forceinline__ void mma16816_0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// an 8 x 8 matrix of 16-bit elements, two neighbours of a row a lane, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

struct Pair {  // two floats in a 64-bit register
    uint64_t v;
};
__device__ __forceinline__ Pair pair_of(float a, float b) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b));
    return p;
}
__device__ __forceinline__ void unpair(const Pair& p, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ Pair fma2(const Pair& a, const Pair& b, const Pair& c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}
__device__ __forceinline__ Pair mul2(const Pair& a, const Pair& b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Pair add2(const Pair& a, const Pair& b) {
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}

// Byte offset of 16-byte chunk c of row r of a stage's keys (or values): runs of 128 bytes
// of all rows one after another, chunks XOR-swizzled by the row so that the 8 rows of
// one ldmatrix phase hit distinct banks (TMA's 128-byte swizzle; stages are 1 KB aligned).
template <int Rows>
__device__ __forceinline__ uint32_t ring_off(int r, int c) {
    return (uint32_t)((c >> 3) * Rows * 128 + r * 128 + (((c ^ r) & 7) << 4));
}

// ---- one warp's tile, bf16: tensor cores -------------------------------------------
//
// S^T = K Q^T and O^T += V^T P^T as m16n8k16 products: the keys (then the dims) are the
// 16 rows and the group's heads the 8 columns, so a group of up to 8 heads takes half
// of the products that heads as rows would (G <= 4: 16 instead of 32 a 16 keys). Decode
// needs 4 G products a key element against 4 bytes of it, far below what even these
// instructions do per byte of HBM traffic; what they cost is power, and the
// kernel runs at the power limit.
// P enters in three bf16 parts, 8 bits each of its 24, so that nothing of it is rounded.
// The parts are cut, not rounded, and a lower one is never below 2^-26 of P, so that an
// infinite value times each stays that infinity, and a P of zero adds nothing (a floor that
// does not shrink with P would weigh values near the type's largest). With G <= 2 the columns repeat the heads and carry
// the three parts in one product; with G = 4 one carries the first two and another half of
// the third twice; larger groups take three.
template <int D_, int G_>
struct MmaTile {
    using T = __nv_bfloat16;
    static constexpr int D = D_, G = G_;
    static constexpr int KT = kTileBytes / (D * 2);  // 16 (d = 128) or 32 (d = 64) keys
    static constexpr int RowBytes = D * 2;
    static constexpr int kScratchFloats = 0, kWeighFloats = 0;
    static constexpr int NT = G > 8 ? 2 : 1;    // column tiles
    static constexpr int kCols = G <= 2 ? 2 : G <= 4 ? 4 : 8;      // the heads repeat every kCols columns, a part of P each
    static constexpr int kProducts = G <= 2 ? 1 : G <= 4 ? 2 : 3;  // that P's parts take

    uint32_t qb[D / 16][NT][2];
    float o[D / 16][NT][4];  // dims 16 j + g (+ 8), columns 2 c, 2 c + 1 (g = lane / 4, c = lane % 4)
    float m[NT][2], l[NT][2];  // of this lane's columns; l is this lane's share

    static constexpr bool kAhead = NT == 1;  // registers for the next unit's queries
    uint32_t qn[kAhead ? D / 16 : 1][NT][2];

    static __device__ __forceinline__ void read_q(uint32_t (*to)[NT][2], const T* q, int lane) {
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int h = kCols < 8 ? g % kCols : 8 * t + g, e = k * 16 + 2 * c + 8 * i;
                    to[k][t][i] = h < G ? __ldg(reinterpret_cast<const unsigned*>(q + (size_t)h * D + e)) : 0u;
                }
    }
    __device__ __forceinline__ void load_q(const T* q, float, int lane) { read_q(qb, q, lane); }
    // the next unit's queries: fetched early, taken when their unit begins
    __device__ __forceinline__ void fetch_q(const T* q, int lane) {
        if constexpr (kAhead) read_q(qn, q, lane);
    }
    __device__ __forceinline__ void take_q(const T* q, float, int lane) {
        if constexpr (kAhead) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) qb[k][0][i] = qn[k][0][i];
        } else {
            read_q(qb, q, lane);
        }
    }
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[j][t][i] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[t][i] = -INFINITY;
                l[t][i] = 0.f;
            }
        }
    }
    // keys of this tile whose bit is set in `mask` count
    __device__ __forceinline__ void step(uint32_t kbuf, uint32_t vbuf, unsigned mask, float qscale, int lane, float*) {
        const int g = lane >> 2, c = lane & 3;
        float s[KT / 16][NT][4];
#pragma unroll
        for (int r = 0; r < KT / 16; ++r) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[r][t][i] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t a[4];
                ldsm4(kbuf + ring_off<KT>(16 * r + (lane & 15), 2 * k + (lane >> 4)), a);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816(s[r][t], a, qb[k][t][0], qb[k][t][1]);
            }
        }
        // The reference moves when a logit passes it (see kRescale): most tiles need neither
        // the exchange between lanes nor the rescaling of o.
        float mx[NT][2];
        bool move = false;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            mx[t][0] = mx[t][1] = -INFINITY;
#pragma unroll
            for (int r = 0; r < KT / 16; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool live = (mask >> (16 * r + g + 8 * (i >> 1))) & 1u;
                    s[r][t][i] = live ? s[r][t][i] * qscale : -INFINITY;
                    mx[t][i & 1] = fmaxf(mx[t][i & 1], s[r][t][i]);
                }
            move |= mx[t][0] > m[t][0] || mx[t][1] > m[t][1];
        }
        if (__any_sync(kFull, move)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x = mx[t][i];
                    x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
                    const float mn = x > m[t][i] ? x + kRescale : m[t][i];
                    const float a = mn == -INFINITY ? 1.f : exp2f(m[t][i] - mn);
                    m[t][i] = mn;
                    l[t][i] *= a;
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        o[j][t][i] *= a;
                        o[j][t][i + 2] *= a;
                    }
                }
        }
#pragma unroll
        for (int r = 0; r < KT / 16; ++r) {
            uint32_t pp[kProducts][NT][2];  // P^T: keys 0..7 and 8..15 of the 16
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float m0 = m[t][0] == -INFINITY ? 0.f : m[t][0], m1 = m[t][1] == -INFINITY ? 0.f : m[t][1];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float p0 = ex2_approx(s[r][t][2 * i] - m0), p1 = ex2_approx(s[r][t][2 * i + 1] - m1);
                    l[t][0] += p0;
                    l[t][1] += p1;
#pragma unroll
                    for (int u = 0; u < kProducts; ++u) pp[u][t][i] = transpose8(parts(p0, p1, u, 2 * c));
                }
            }
            accumulate(vbuf, r, pp, lane);
        }
    }
    __device__ __forceinline__ void poison() {
#pragma unroll
        for (int t = 0; t < NT; ++t) l[t][0] = l[t][1] = NAN;
    }

    // ---- the same in two passes, where the logits are kept: z[h * stride + key] = scaled logits ...
    __device__ __forceinline__ void logits(uint32_t kbuf, float qscale, float* z, int stride, int lane) {
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int r = 0; r < KT / 16; ++r) {
            float s[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[t][i] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t a[4];
                ldsm4(kbuf + ring_off<KT>(16 * r + (lane & 15), 2 * k + (lane >> 4)), a);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816(s[t], a, qb[k][t][0], qb[k][t][1]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int h = 8 * t + 2 * c + (i & 1);
                    if (h < G) z[h * stride + 16 * r + g + 8 * (i >> 1)] = s[t][i] * qscale;
                }
        }
    }
    // ... and o += 2^(z - Z) v over the first `rows` keys. l (its first entry) is then the sum
    // of this lane's keys for head 8 t + lane / 4 (where heads repeat: of that column's head).
    __device__ __forceinline__ void weigh(uint32_t vbuf, const float* z, int stride, const float* Z, int rows, int lane,
                                          float*) {
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int r = 0; r < KT / 16; ++r) {
            uint32_t pp[kProducts][NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int h = kCols < 8 ? g % kCols : 8 * t + g;
                const float top = h < G ? Z[h] : 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int key = 16 * r + 8 * i + 2 * c;
                    float2 x = make_float2(0.f, 0.f);
                    if (h < G) x = *reinterpret_cast<const float2*>(z + h * stride + key);
                    const float p0 = h < G && key < rows ? ex2_approx(x.x - top) : 0.f;
                    const float p1 = h < G && key + 1 < rows ? ex2_approx(x.y - top) : 0.f;
                    l[t][0] += p0 + p1;
#pragma unroll
                    for (int u = 0; u < kProducts; ++u) pp[u][t][i] = parts(p0, p1, u, g);
                }
            }
            accumulate(vbuf, r, pp, lane);
        }
    }
    // o (not yet divided) and the sums into a slot ([G][D], then [G])
    __device__ __forceinline__ void put_sums(float* slot, int lane) {
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float sum = l[t][0];
            sum += __shfl_xor_sync(kFull, sum, 1);
            sum += __shfl_xor_sync(kFull, sum, 2);
            if (c == 0 && 8 * t + g < G) slot[G * D + 8 * t + g] = sum;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int h = 8 * t + 2 * c + i;
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = whole(o[j][t][i + 2 * e]);
                        if (h < G && 2 * c < kCols) slot[h * D + 16 * j + 8 * e + g] = x;
                    }
            }
        }
    }

    // the first 8 bits of x, or 0
    static __device__ __forceinline__ float cut(float x, bool any) {
        return __uint_as_float(__float_as_uint(x) & (any ? 0xffff0000u : 0u));
    }
    // what product u has of p in column `col`: its part is the first 8 bits of that (all steps are exact)
    static __device__ __forceinline__ float share(float p, int u, int col) {
        const int part = kProducts == 3 ? u : u == 0 ? col / kCols : 2;
        float x = p - cut(p, part >= 1);
        x -= cut(x, part >= 2);
        return fmaxf(kProducts == 2 && u == 1 ? 0.5f * x : x, p * 0x1p-26f);
    }
    // of two neighbouring probabilities
    static __device__ __forceinline__ uint32_t parts(float p0, float p1, int u, int col) {
        return __byte_perm(__float_as_uint(share(p0, u, col)), __float_as_uint(share(p1, u, col)), 0x7632);
    }
    // an output's columns together (of use in the lanes of the first kCols columns)
    static __device__ __forceinline__ float whole(float x) {
        if (kCols == 2) {
            const float y = __shfl_xor_sync(kFull, x, 1), z = __shfl_xor_sync(kFull, x, 2);
            return x + y + z;
        }
        return kCols == 4 ? x + __shfl_xor_sync(kFull, x, 2) : x;
    }
    // o += V^T P^T over keys 16 r .. 16 r + 15. The sum over a tile's keys starts from zero and is added
    // rounded: adding on, the tensor cores cut what lies below the sum's last bit, and a
    // chain of n / 64 such cuts, all toward zero, is a bias (sums of weights that cancel over 64 K
    // keys came out at -6e-6, over 256 K at -6e-5). It costs 1% of the time of 64 x 16 K.
    __device__ __forceinline__ void accumulate(uint32_t vbuf, int r, const uint32_t (&pp)[kProducts][NT][2], int lane) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            uint32_t a[4];
            ldsm4_t(vbuf + ring_off<KT>(16 * r + (lane >> 4) * 8 + (lane & 7), 2 * j + ((lane >> 3) & 1)), a);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float s[4];
                mma16816_0(s, a, pp[0][t][0], pp[0][t][1]);
#pragma unroll
                for (int u = 1; u < kProducts; ++u) mma16816(s, a, pp[u][t][0], pp[u][t][1]);
#pragma unroll
                for (int i = 0; i < 4; i += 2)
                    unpair(add2(pair_of(o[j][t][i], o[j][t][i + 1]), pair_of(s[i], s[i + 1])), o[j][t][i], o[j][t][i + 1]);
            }
        }
    }
    // this warp's state into a merge slot ([G][D] o, then m[G], l[G]); `add`: merged with what is there
    __device__ __forceinline__ void put(float* slot, bool add, int lane) {
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int h = 8 * t + 2 * c + i;
                const bool mine = h < G && 2 * c < kCols;
                float sum = l[t][i];
                sum += __shfl_xor_sync(kFull, sum, 4);
                sum += __shfl_xor_sync(kFull, sum, 8);
                sum += __shfl_xor_sync(kFull, sum, 16);
                float a = 1.f, b = 0.f, mn = m[t][i];
                if (add && mine) {
                    const float ms = slot[G * D + h];
                    mn = fmaxf(mn, ms);
                    a = m[t][i] == -INFINITY ? 0.f : exp2f(m[t][i] - mn);
                    b = ms == -INFINITY ? 0.f : exp2f(ms - mn);
                    sum = a * sum + b * slot[G * D + G + h];
                }
                __syncwarp();
                if (mine && g == 0) {
                    slot[G * D + h] = mn;
                    slot[G * D + G + h] = sum;
                }
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = whole(o[j][t][i + 2 * e]);
                        float* p = slot + h * D + 16 * j + 8 * e + g;
                        if (mine) *p = add ? a * x + b * *p : x;
                    }
            }
    }
};

// ---- one warp's tile, fp32: CUDA cores -----------------------------------------------
//
// A lane owns 4 dims of a row (D / 4 lanes a row, 32 * 4 / D rows at a time);
// the G partial dots of several rows are summed across lanes in one
// reduce-scatter, and the probabilities come back through shared memory (each twice,
// as the operand of a packed product). Products are packed pairs (fma.rn.f32x2): with
// groups of 8 and 16 the kernel is bound by instructions, not by memory.

template <int D_, int G_>
struct FmaTile {
    using T = float;
    static constexpr int D = D_, G = G_;
    static constexpr int KT = kTileBytes / (D * 4);  // 8 (d = 128) or 16 (d = 64) keys
    static constexpr int RowBytes = D * 4;
    static constexpr int LR = D / 4;       // lanes a row
    static constexpr int RP = 32 / LR;     // rows at a time
    static constexpr int RI = KT / RP;     // rows a lane takes part in
    static constexpr int kScratchFloats = (3 * KT * G + G + 3) / 4 * 4;  // p twice, logits, factors
    static constexpr int kZ = 2 * KT * G, kA = 3 * KT * G;
    static constexpr int kWeighFloats = 2 * KT * G;  // of which weigh() needs these
    static constexpr int NB = RI * G < LR ? RI * G : LR;  // values of one reduce-scatter

    Pair q[G][2], o[G][2];
    float m, l;  // of head lane % G (G <= 16 lanes hold it several times over; l is a share)

    __device__ __forceinline__ void fetch_q(const T*, int) {}
    __device__ __forceinline__ void take_q(const T* src, float qscale, int lane) { load_q(src, qscale, lane); }
    __device__ __forceinline__ void load_q(const T* src, float qscale, int lane) {
        const int e = (lane % LR) * 4;
#pragma unroll
        for (int h = 0; h < G; ++h) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(src + (size_t)h * D + e));
            q[h][0] = pair_of(v.x * qscale, v.y * qscale);
            q[h][1] = pair_of(v.z * qscale, v.w * qscale);
        }
    }
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int h = 0; h < G; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) o[h][e] = pair_of(0.f, 0.f);
        m = -INFINITY;
        l = 0.f;
    }
    static __device__ __forceinline__ void row16(uint32_t buf, int r, int c, Pair (&x)[2]) {
        asm volatile("ld.shared.v2.b64 {%0,%1}, [%2];\n" : "=l"(x[0].v), "=l"(x[1].v) : "r"(buf + ring_off<KT>(r, c)) : "memory");
    }
    // z[h * hs + key * ks] = logits of the tile's keys
    __device__ __forceinline__ void dots(uint32_t kbuf, float* z, int hs, int ks, int lane) {
        const int sub = lane / LR, c = lane % LR;
        constexpr int RowsB = NB / G;  // rows (of this lane's) in one reduce-scatter
#pragma unroll
        for (int r0 = 0; r0 < RI; r0 += RowsB) {
            float v[NB];
#pragma unroll
            for (int r = 0; r < RowsB; ++r) {
                Pair x[2];
                row16(kbuf, (r0 + r) * RP + sub, c, x);
#pragma unroll
                for (int h = 0; h < G; ++h) {
                    float a, b;
                    unpair(fma2(q[h][0], x[0], mul2(q[h][1], x[1])), a, b);
                    v[r * G + h] = a + b;
                }
            }
            int n = NB;
#pragma unroll
            for (int w = LR / 2; w >= 1; w >>= 1) {
                if (n > 1) {
                    n >>= 1;
                    const bool hi = (lane & w) != 0;
#pragma unroll
                    for (int i = 0; i < NB / 2; ++i)
                        if (i < n) {
                            const float send = hi ? v[i] : v[i + n], keep = hi ? v[i + n] : v[i];
                            v[i] = keep + __shfl_xor_sync(kFull, send, w);
                        }
                } else {
                    v[0] += __shfl_xor_sync(kFull, v[0], w);
                }
            }
            const int i = (lane % LR) / (LR / NB);  // the value this lane ended with
            z[(i % G) * hs + ((r0 + i / G) * RP + sub) * ks] = v[0];
        }
    }
    // o += p v, p[2 * (key * G + h)] and the float behind it
    __device__ __forceinline__ void accumulate(uint32_t vbuf, const float* p, int lane) {
        const int sub = lane / LR, c = lane % LR;
#pragma unroll
        for (int r = 0; r < RI; ++r) {
            const int key = r * RP + sub;
            Pair x[2], w[G];
            row16(vbuf, key, c, x);
            const uint32_t at = tc::smem_u32(p + 2 * key * G);
            if constexpr (G == 1) {
                asm volatile("ld.shared.b64 %0, [%1];\n" : "=l"(w[0].v) : "r"(at) : "memory");
            } else {
#pragma unroll
                for (int h = 0; h < G; h += 2)
                    asm volatile("ld.shared.v2.b64 {%0,%1}, [%2];\n" : "=l"(w[h].v), "=l"(w[h + 1].v) : "r"(at + 8 * h) : "memory");
            }
#pragma unroll
            for (int h = 0; h < G; ++h)
#pragma unroll
                for (int e = 0; e < 2; ++e) o[h][e] = fma2(w[h], x[e], o[h][e]);
        }
    }
    static __device__ __forceinline__ void put_p(float* scratch, int key, int h, float p) {
        *reinterpret_cast<float2*>(scratch + 2 * (key * G + h)) = make_float2(p, p);
    }
    __device__ __forceinline__ void step(uint32_t kbuf, uint32_t vbuf, unsigned mask, float, int lane, float* scratch) {
        dots(kbuf, scratch + kZ, 1, G, lane);
        __syncwarp();
        // head h = lane % G, keys lane / G, lane / G + 32 / G, ...
        constexpr int PER = (KT * G + 31) / 32;
        const int h = lane % G;
        float z[PER], mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int key = lane / G + i * (32 / G);
            z[i] = key < KT && ((mask >> key) & 1u) ? scratch[kZ + key * G + h] : -INFINITY;
            mx = fmaxf(mx, z[i]);
        }
#pragma unroll
        for (int w = G; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, w));
        const bool move = __any_sync(kFull, mx > m);
        if (move) {
            const float mn = mx > m ? mx + kRescale : m;
            const float a = mn == -INFINITY ? 1.f : exp2f(m - mn);
            m = mn;
            l *= a;
            if (lane < G) scratch[kA + lane] = a;
        }
        const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int key = lane / G + i * (32 / G);
            if (key < KT) {
                const float p = exp2f(z[i] - mu);
                l += p;
                put_p(scratch, key, h, p);
            }
        }
        __syncwarp();
        if (move) {
#pragma unroll
            for (int hh = 0; hh < G; ++hh) {
                const Pair a = pair_of(scratch[kA + hh], scratch[kA + hh]);
#pragma unroll
                for (int e = 0; e < 2; ++e) o[hh][e] = mul2(o[hh][e], a);
            }
        }
        accumulate(vbuf, scratch, lane);
        __syncwarp();  // scratch is rewritten by the next tile
    }
    __device__ __forceinline__ float part_of(int h, int e) const {
        float a, b;
        unpair(o[h][e >> 1], a, b);
        return e & 1 ? b : a;
    }
    __device__ __forceinline__ void poison() { l = NAN; }

    // ---- in two passes (see MmaTile)
    __device__ __forceinline__ void logits(uint32_t kbuf, float, float* z, int stride, int lane) {
        dots(kbuf, z, stride, 1, lane);
    }
    __device__ __forceinline__ void weigh(uint32_t vbuf, const float* z, int stride, const float* Z, int rows, int lane,
                                          float* scratch) {
        const int h = lane % G;
#pragma unroll
        for (int i = 0; i < (KT * G + 31) / 32; ++i) {
            const int key = lane / G + i * (32 / G);
            if (key < KT) {
                const float p = key < rows ? exp2f(z[h * stride + key] - Z[h]) : 0.f;
                l += p;
                put_p(scratch, key, h, p);
            }
        }
        __syncwarp();
        accumulate(vbuf, scratch, lane);
        __syncwarp();
    }
    __device__ __forceinline__ void put_sums(float* slot, int lane) {
        float sum = l;
#pragma unroll
        for (int w = G; w < 32; w <<= 1) sum += __shfl_xor_sync(kFull, sum, w);
        if (lane < G) slot[G * D + lane] = sum;
#pragma unroll
        for (int h = 0; h < G; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = part_of(h, e);
                if (RP == 2) x += __shfl_xor_sync(kFull, x, LR);
                if (lane < LR) slot[h * D + lane * 4 + e] = x;
            }
    }
    __device__ __forceinline__ void put(float* slot, bool add, int lane) {
        float sum = l;
#pragma unroll
        for (int w = G; w < 32; w <<= 1) sum += __shfl_xor_sync(kFull, sum, w);
        float a = 1.f, b = 0.f, mn = m;
        if (add) {
            const float ms = slot[G * D + lane % G];
            mn = fmaxf(m, ms);
            a = m == -INFINITY ? 0.f : exp2f(m - mn);
            b = ms == -INFINITY ? 0.f : exp2f(ms - mn);
            sum = a * sum + b * slot[G * D + G + lane % G];
        }
        __syncwarp();
        if (lane < G) {
            slot[G * D + lane] = mn;
            slot[G * D + G + lane] = sum;
        }
#pragma unroll
        for (int h = 0; h < G; ++h) {
            const float ah = __shfl_sync(kFull, a, h), bh = __shfl_sync(kFull, b, h);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = part_of(h, e);
                if (RP == 2) x += __shfl_xor_sync(kFull, x, LR);  // the two rows' shares of a dim
                float* p = slot + h * D + (lane % LR) * 4 + e;
                if (lane < LR) *p = add ? ah * x + bh * *p : x;
            }
        }
    }
};

}  // namespace pisa
