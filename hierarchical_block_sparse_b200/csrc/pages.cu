// pages.cu -- the page table of a paged cache: room for new tokens, forking,
// freeing and compacting on the device, and the copies of page data they ask
// for. One table serves every layer of a model; the data copies run once a layer.
//
// Counts are changed by integer atomics (their order does not matter) and free
// pages are handed out lowest first, so every result is the same from run to run.
#include "pisa_internal.h"
#include "pisa_paged.cuh"

namespace pisa {

namespace {

constexpr unsigned kAll = 0xffffffffu;
// Up to this many table entries one block does all phases of a fork or a compaction: with
// 1024 entries a beam step takes 13.1 us (two launches: 13.8), with 2048 14.6 (14.1) and a launch
// less on the host, with 4096 18.2 (15.7).
constexpr int kSmallTable = 2048;

// drops one reference of a page; the last one frees it
__device__ __forceinline__ void drop(int32_t* refs, unsigned* bits, int page, int P) {
    if ((unsigned)page >= (unsigned)P) return;
    const int old = atomicSub(refs + page, 1);
    if (old == 1) atomicOr(bits + (page >> 5), 1u << (page & 31));
    else if (old <= 0) atomicAdd(refs + page, 1);  // a table that names a free page: leave the page free
}

// exclusive sums of N values over the 1024 threads of a block; total[i] gets the sums of all
template <int N>
__device__ __forceinline__ void block_scan(int64_t (&v)[N], int64_t (&warp_sums)[N][32], int64_t (&total)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x[N], s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = v[i];
#pragma unroll
    for (int w = 1; w < 32; w <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t y = __shfl_up_sync(kFull, x[i], w);
            if (lane >= w) x[i] += y;
        }
    if (lane == 31)
#pragma unroll
        for (int i = 0; i < N; ++i) warp_sums[i][warp] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = warp_sums[i][lane];
#pragma unroll
    for (int w = 1; w < 32; w <<= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int64_t y = __shfl_up_sync(kFull, s[i], w);
            if (lane >= w) s[i] += y;
        }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        total[i] = __shfl_sync(kFull, s[i], 31);
        const int64_t before = __shfl_sync(kFull, s[i], (warp + 31) & 31);
        v[i] = (warp == 0 ? 0 : before) + x[i] - v[i];
    }
}

__global__ void __launch_bounds__(256) pages_init_kernel(int32_t* __restrict__ state, int32_t* __restrict__ table,
                                                         int32_t* __restrict__ len, int P, int B, int64_t entries) {
    const PageState L(P);
    const int64_t step = (int64_t)gridDim.x * blockDim.x, i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    for (int64_t i = i0; i < L.p4; i += step) state[i] = 0;
    for (int64_t i = i0; i < L.b4; i += step) {
        const int64_t left = (int64_t)P - i * 32;
        state[L.bits() + i] = (int32_t)(left >= 32 ? kAll : left > 0 ? (1u << left) - 1u : 0u);
    }
    for (int64_t i = i0; i < entries; i += step) table[i] = -1;
    for (int64_t i = i0; i < B; i += step) len[i] = 0;
}

// Room for add[b] more tokens of every sequence, as if done one sequence after
// another: ceil((len + add) / S) - ceil(len / S) new pages, and a page of its own
// in place of a partial last page that others share (all but the last of its
// sharers in this call copy it when no one else holds it). All or nothing. One
// CTA: the integers are few (B lengths, P / 8 bytes of bitmap) and one block's
// barriers are cheaper than a second launch.
constexpr int kReserveIds = 2048;
constexpr int kReservePer = kReserveMaxSeqs / 1024;  // sequences a thread
__global__ void __launch_bounds__(1024) pages_reserve_kernel(const int32_t* __restrict__ add, int32_t* __restrict__ state,
                                                             int32_t* __restrict__ table, int32_t* __restrict__ len,
                                                             int32_t* __restrict__ grant, int32_t* __restrict__ moves,
                                                             int B, int N, int S, int P, int W) {
    __shared__ int64_t warp_sums[2][32];
    __shared__ int s_shared;                         // sequences with a shared partial last page
    __shared__ int s_ids[kReserveIds];               // the first pages handed out
    extern __shared__ int dyn[];                     // two arrays of that list, then four of the sequences
    int* l_seq = dyn;
    int* l_page = dyn + B;
    int* s_base = dyn + 2 * B;                       // first of the sequence's pages among those handed out
    int* s_need = dyn + 3 * B;
    int* s_have = dyn + 4 * B;
    int* s_tail = dyn + 5 * B;                       // page to copy, or -1
    const int tid = threadIdx.x;
    const PageState L(P);
    int32_t* refs = state;
    unsigned* bits = reinterpret_cast<unsigned*>(state + L.bits());
    int32_t* ids = state + L.map();
    // free pages, counted in order of their ids, a run of words a thread (the bitmap is
    // padded to 4 words); read first, so that the loads overlap the sequences'
    const int words = (P + 31) / 32, run = words <= 1024 ? 1 : ((words + 1023) / 1024 + 3) / 4 * 4;
    const int w0 = tid * run, w1 = min(w0 + run, words);
    int64_t found = 0;
    if (run == 1) {
        if (w0 < w1) found = __popc(bits[w0]);
    } else {
        for (int w = w0; w < w1; w += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(bits + w);
            found += __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w);
        }
    }
    if (tid == 0) s_shared = 0;
    __syncthreads();

    const int per = (B + 1023) / 1024, b0 = tid * per;
    int a[kReservePer], n[kReservePer], have[kReservePer], want[kReservePer], tail[kReservePer];
#pragma unroll
    for (int i = 0; i < kReservePer; ++i) {
        const int b = b0 + i;
        a[i] = n[i] = have[i] = want[i] = 0;
        tail[i] = -1;
        if (i >= per || b >= B) continue;
        n[i] = len[b];
        a[i] = add[b];
        if (a[i] <= 0 || n[i] < 0 || (int64_t)n[i] + a[i] > N) {
            a[i] = 0;
            continue;
        }
        have[i] = (int)(((int64_t)n[i] + S - 1) / S);
        want[i] = (int)(((int64_t)n[i] + a[i] + S - 1) / S);
        if (n[i] % S != 0) {
            const int page = table[(size_t)b * W + have[i] - 1];
            if ((unsigned)page >= (unsigned)P) {  // the cached tokens have no page: nothing to go on from
                a[i] = 0;
                want[i] = have[i];
            } else if (refs[page] > 1) {
                tail[i] = page;
                const int k = atomicAdd(&s_shared, 1);
                l_seq[k] = b;
                l_page[k] = page;
            }
        }
    }
    __syncthreads();
    int64_t sums[2] = {0, found}, all[2];  // copies << 48 | pages of this thread's sequences; its free pages
#pragma unroll
    for (int i = 0; i < kReservePer; ++i) {
        if (tail[i] >= 0) {
            int before = 0;
            for (int k = 0; k < s_shared; ++k) before += l_page[k] == tail[i] && l_seq[k] < b0 + i;
            if (before >= refs[tail[i]] - 1) tail[i] = -1;  // the last holder writes in place
        }
        sums[0] += (int64_t)(want[i] - have[i]) + (tail[i] >= 0 ? ((int64_t)1 << 48) + 1 : 0);
    }
    block_scan(sums, warp_sums, all);
    int64_t at = sums[0], rank = sums[1];
    const int64_t total = all[0] & (((int64_t)1 << 48) - 1), spare = all[1];
    const bool fits = total <= spare;
    if (tid == 0) {
        moves[0] = fits ? (int)(all[0] >> 48) : 0;
        moves[1] = fits ? 0 : (int)min(total - spare, (int64_t)INT32_MAX);
        moves[2] = (int)(P - spare + (fits ? total : 0));
        moves[3] = (int)(spare - (fits ? total : 0));
    }
    if (fits) {
        // the first `total` of them, a word at a time by a whole warp, a bit a lane
        const int lane = tid & 31;
        unsigned busy = __ballot_sync(kFull, found > 0 && rank < total);
        while (busy) {
            const int from = __ffs(busy) - 1;
            busy &= busy - 1;
            int64_t at_rank = __shfl_sync(kFull, rank, from);
            const int first = __shfl_sync(kFull, w0, from), last = __shfl_sync(kFull, w1, from);
            for (int w = first; w < last && at_rank < total; ++w) {
                const unsigned v = bits[w];
                const int64_t k = at_rank + __popc(v & ((1u << lane) - 1u));
                const bool mine = (v >> lane) & 1u, taken = mine && k < total;
                if (taken) {
                    if (k < kReserveIds) s_ids[k] = w * 32 + lane;
                    else ids[k] = w * 32 + lane;
                }
                const unsigned left = __ballot_sync(kFull, mine && !taken);
                if (lane == 0 && left != v) bits[w] = left;
                at_rank += __popc(v);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kReservePer; ++i) {
        const int b = b0 + i;
        if (i >= per || b >= B) continue;
        grant[b] = fits ? a[i] : 0;
        if (fits && a[i] > 0) len[b] = n[i] + a[i];
        const int copies = tail[i] >= 0, need = want[i] - have[i] + copies;
        s_base[b] = (int)(at & INT32_MAX);  // read only where all pages fit, so below 2^31
        s_need[b] = need;
        s_have[b] = have[i];
        s_tail[b] = tail[i];
        if (fits && copies) {
            const int k = kMovesHead + 2 * (int)(at >> 48);
            moves[k] = tail[i];  // the destination follows below
            l_seq[b] = k + 1;    // the list of shared pages is done with
        }
        at += need + ((int64_t)copies << 48);
    }
    __syncthreads();  // the ids, written to global memory by this block, are visible to it
    if (!fits) return;
    const int lane = tid & 31;
    for (int b = tid >> 5; b < B; b += 32) {
        const int need = s_need[b], base = s_base[b], t = s_tail[b], first = s_have[b] - (t >= 0 ? 1 : 0);
        for (int k = lane; k < need; k += 32) {
            const int page = base + k < kReserveIds ? s_ids[base + k] : ids[base + k];
            refs[page] = 1;
            table[(size_t)b * W + first + k] = page;
            if (k == 0 && t >= 0) {
                moves[l_seq[b]] = page;
                atomicSub(refs + t, 1);  // at least one holder is left
            }
        }
    }
}

// New table row b = old row parent[b]; every entry a new row takes over counts.
__device__ __forceinline__ void fork_entry(int b, int w, const int32_t* parent, int32_t* refs, const int32_t* table,
                                           const int32_t* len, int32_t* table_out, int32_t* len_out, int B, int P, int W) {
    const int from = parent[b];
    const bool ok = (unsigned)from < (unsigned)B;
    if (w == 0) len_out[b] = ok ? len[from] : 0;
    const int page = ok ? table[(size_t)from * W + w] : -1;
    table_out[(size_t)b * W + w] = page;
    if (from != b && (unsigned)page < (unsigned)P) atomicAdd(refs + page, 1);
}
// The old rows' entries, dropped after every new one is counted (a page that
// stays in use never passes through zero).
__device__ __forceinline__ void unfork_entry(int b, int w, const int32_t* parent, int32_t* refs, unsigned* bits,
                                             const int32_t* table, int P, int W) {
    if (parent[b] != b) drop(refs, bits, table[(size_t)b * W + w], P);
}
__global__ void __launch_bounds__(256) pages_fork_kernel(const int32_t* __restrict__ parent, int32_t* __restrict__ refs,
                                                         const int32_t* __restrict__ table, const int32_t* __restrict__ len,
                                                         int32_t* __restrict__ table_out, int32_t* __restrict__ len_out,
                                                         int B, int P, int W, int tiles) {
    const int b = blockIdx.x / tiles, w = (blockIdx.x % tiles) * 256 + threadIdx.x;
    if (w < W) fork_entry(b, w, parent, refs, table, len, table_out, len_out, B, P, W);
}
__global__ void __launch_bounds__(256) pages_unfork_kernel(const int32_t* __restrict__ parent, int32_t* __restrict__ refs,
                                                           unsigned* __restrict__ bits, const int32_t* __restrict__ table,
                                                           int P, int W, int tiles) {
    const int b = blockIdx.x / tiles, w = (blockIdx.x % tiles) * 256 + threadIdx.x;
    if (w < W) unfork_entry(b, w, parent, refs, bits, table, P, W);
}
// Both in one block, for tables of up to kSmallTable entries.
__global__ void __launch_bounds__(1024) pages_fork_small_kernel(const int32_t* __restrict__ parent, int32_t* __restrict__ refs,
                                                                unsigned* __restrict__ bits, const int32_t* __restrict__ table,
                                                                const int32_t* __restrict__ len,
                                                                int32_t* __restrict__ table_out,
                                                                int32_t* __restrict__ len_out, int B, int P, int W) {
    for (int i = threadIdx.x; i < B * W; i += 1024) fork_entry(i / W, i % W, parent, refs, table, len, table_out, len_out, B, P, W);
    __syncthreads();
    for (int i = threadIdx.x; i < B * W; i += 1024) unfork_entry(i / W, i % W, parent, refs, bits, table, P, W);
}

// Each entry is taken out of the table by an exchange, so that a sequence
// listed twice is freed once.
__global__ void __launch_bounds__(256) pages_free_kernel(const int32_t* __restrict__ seqs, int32_t* __restrict__ refs,
                                                         unsigned* __restrict__ bits, int32_t* __restrict__ table,
                                                         int32_t* __restrict__ len, int B, int P, int W, int tiles) {
    const int b = seqs[blockIdx.x / tiles], w = (blockIdx.x % tiles) * 256 + threadIdx.x;
    if ((unsigned)b >= (unsigned)B || w >= W) return;
    if (w == 0) len[b] = 0;
    int32_t* e = table + (size_t)b * W + w;
    if (*reinterpret_cast<volatile int32_t*>(e) == -1) return;
    drop(refs, bits, atomicExch(e, -1), P);
}

// Compaction, 1 of 3: live pages before each word of the bitmap, the bitmap as it
// was and as it will be (pages below the live count taken, the others free).
__device__ __forceinline__ void compact_scan(int32_t* state, int32_t* moves, int P, int64_t (&warp_sums)[1][32]) {
    const PageState L(P);
    unsigned* bits = reinterpret_cast<unsigned*>(state + L.bits());
    unsigned* old = reinterpret_cast<unsigned*>(state + L.old_bits());
    int32_t* before = state + L.before();
    const int tid = threadIdx.x, words = (P + 31) / 32, run = (words + 1023) / 1024;
    const int w0 = tid * run, w1 = min(w0 + run, words);
    auto taken = [&](int w) {  // live pages of word w
        const unsigned v = ~bits[w];
        const int left = P - w * 32;
        return left >= 32 ? v : v & ((1u << left) - 1u);
    };
    int64_t sums[1] = {0}, all[1];
    for (int w = w0; w < w1; ++w) sums[0] += __popc(taken(w));
    block_scan(sums, warp_sums, all);
    const int64_t live = all[0];
    int64_t at = sums[0];
    for (int w = w0; w < w1; ++w) {
        const unsigned v = taken(w);
        before[w] = (int)at;
        if (live >= (int64_t)w * 32 && live < (int64_t)w * 32 + 32) {  // the boundary lies in this word
            const int below = (int)at + __popc(v & ((1u << (live - (int64_t)w * 32)) - 1u));
            moves[0] = (int)live - below;
        }
        at += __popc(v);
        old[w] = ~v;
        const int64_t cut = live - (int64_t)w * 32;  // pages of this word below the live count
        unsigned free = cut >= 32 ? 0u : cut > 0 ? ~((1u << cut) - 1u) : kAll;
        const int left = P - w * 32;
        if (left < 32) free &= (1u << left) - 1u;
        bits[w] = free;
    }
    if (tid == 0) {
        if (live == (int64_t)words * 32) moves[0] = 0;  // no word holds the boundary: the pool is full
        before[words] = (int)live;
        moves[1] = 0;
        moves[2] = (int)live;
        moves[3] = (int)(P - live);
    }
}

// 2 of 3: the i-th live page at or past the live count moves to the i-th free one below it.
__device__ __forceinline__ void compact_move(int page, int live, int32_t* state, int32_t* moves, int P, int max_moves) {
    const PageState L(P);
    if (page >= P || page < live) return;
    const unsigned* old = reinterpret_cast<const unsigned*>(state + L.old_bits());
    const int32_t* before = state + L.before();
    if ((old[page >> 5] >> (page & 31)) & 1u) return;
    auto live_below = [&](int x) { return before[x >> 5] + __popc(~old[x >> 5] & ((1u << (x & 31)) - 1u)); };
    const int rank = live_below(page) - live_below(live);
    // the word in which the rank-th free page lies: free pages before word w are 32 w - before[w]
    int lo = 0, hi = live >> 5;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (mid * 32 - before[mid] <= rank) lo = mid;
        else hi = mid - 1;
    }
    unsigned v = old[lo];
    for (int k = rank - (lo * 32 - before[lo]); k > 0; --k) v &= v - 1;
    const int to = lo * 32 + __ffs(v) - 1;
    if (v == 0 || to >= live || rank < 0 || rank >= max_moves) return;  // a state that does not add up: nothing moves
    state[L.map() + page] = to;
    state[to] = state[page];
    state[page] = 0;
    moves[kMovesHead + 2 * rank] = page;
    moves[kMovesHead + 2 * rank + 1] = to;
}

// 3 of 3: the table's entries follow.
__device__ __forceinline__ void compact_entry(int32_t* entry, int live, const int32_t* map, int P) {
    const int page = *entry;
    if (page < live || page >= P) return;
    const int to = map[page];
    if ((unsigned)to < (unsigned)live) *entry = to;
}

__global__ void __launch_bounds__(1024) compact_scan_kernel(int32_t* __restrict__ state, int32_t* __restrict__ moves, int P) {
    __shared__ int64_t warp_sums[1][32];
    compact_scan(state, moves, P, warp_sums);
}
__global__ void __launch_bounds__(256) compact_move_kernel(int32_t* __restrict__ state, int32_t* __restrict__ moves,
                                                           int P, int max_moves) {
    compact_move(blockIdx.x * 256 + threadIdx.x, moves[2], state, moves, P, max_moves);
}
__global__ void __launch_bounds__(256) compact_table_kernel(const int32_t* __restrict__ map, int32_t* __restrict__ table,
                                                            const int32_t* __restrict__ moves, int P, int64_t entries) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < entries) compact_entry(table + i, moves[2], map, P);
}
// All three in one block, for tables of up to kSmallTable entries and as many pages.
__global__ void __launch_bounds__(1024) compact_small_kernel(int32_t* state, int32_t* table, int32_t* moves, int P, int entries,
                                                             int max_moves) {
    __shared__ int64_t warp_sums[1][32];
    compact_scan(state, moves, P, warp_sums);
    __syncthreads();
    const int live = moves[2];
    for (int i = live + threadIdx.x; i < P; i += 1024) compact_move(i, live, state, moves, P, max_moves);
    __syncthreads();
    const int32_t* map = state + PageState(P).map();
    for (int i = threadIdx.x; i < entries; i += 1024) compact_entry(table + i, live, map, P);
}

// Page data of the moves: a page of a pool is one run of bytes, cut into segments of
// kSegment (smaller pages are one segment). TEAM threads, as many as a segment's bytes keep
// busy (2 KB pages with all 512: 28 us, with 64: 9, for 3660 of them), take a
// segment at a time, up to 2 x 16 bytes a thread in flight, and far more blocks than fit at
// once even out the ends (grids of 8, 16, 64 a SM: 164, 149, 143 us for 3600 pages of
// 128 KB, 6.6 TB/s read and written at best).
constexpr int kSegment = 16384;
constexpr int kCopyThreads = 512, kCopyPer = kSegment / 16 / kCopyThreads;
template <int TEAM>
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const int32_t* __restrict__ moves, uint8_t* __restrict__ K,
                                                         uint8_t* __restrict__ V, int64_t page_bytes, int segments, int P,
                                                         int max_moves) {
    constexpr int kTeams = kCopyThreads / TEAM;
    const int64_t tasks = (int64_t)min(max(moves[0], 0), max_moves) * 2 * segments;
    const int me = threadIdx.x % TEAM, mine = kTeams == 1 ? 0 : threadIdx.x / TEAM;
    for (int64_t task = (int64_t)blockIdx.x * kTeams + mine; task < tasks; task += (int64_t)gridDim.x * kTeams) {
        const int seg = (int)(task % segments);
        const int64_t rest = task / segments;
        const int src = moves[kMovesHead + (rest & ~(int64_t)1)], dst = moves[kMovesHead + (rest & ~(int64_t)1) + 1];
        if ((unsigned)src >= (unsigned)P || (unsigned)dst >= (unsigned)P) continue;
        uint8_t* pool = (rest & 1) ? V : K;
        const int64_t off = (int64_t)seg * kSegment;
        const int chunks = (int)(min(page_bytes - off, (int64_t)kSegment) / 16);
        const uint4* from = reinterpret_cast<const uint4*>(pool + (int64_t)src * page_bytes + off);
        uint4* to = reinterpret_cast<uint4*>(pool + (int64_t)dst * page_bytes + off);
        uint4 v[kCopyPer];
#pragma unroll
        for (int i = 0; i < kCopyPer; ++i)
            if (me + i * TEAM < chunks) v[i] = __ldcs(from + me + i * TEAM);
#pragma unroll
        for (int i = 0; i < kCopyPer; ++i)
            if (me + i * TEAM < chunks) __stcs(to + me + i * TEAM, v[i]);
    }
}

// New rows into the pages: kAppendPer times 16 bytes of K and of V a thread, all
// loaded before the first is stored (1, 2, 4 times: 42.1, 42.7, 44.7 us for 4 x 8192 full
// rows of 8 heads, 54.1, 51.0, 52.5 us with the page calls where half of 32 sequences
// add 1 to 2 K rows). Sequence b's rows are one run [Hkv, T, d] of the input; row
// i < count[b] goes to token len[b] - count[b] + i.
constexpr int kAppendPer = 2;
__global__ void __launch_bounds__(256) paged_append_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                                                           const int32_t* __restrict__ count, uint4* __restrict__ K,
                                                           uint4* __restrict__ V, int T, int shift, int64_t per_seq,
                                                           int tiles, PagedParams p) {
    const int b = blockIdx.x / tiles;
    const int64_t i0 = (int64_t)(blockIdx.x % tiles) * (256 * kAppendPer) + threadIdx.x;
    const int n = p.len[b], m = count[b];
    if (m <= 0 || m > T || n > p.N || m > n) return;
    uint4 k[kAppendPer], v[kAppendPer];
    int64_t dst[kAppendPer];
#pragma unroll
    for (int u = 0; u < kAppendPer; ++u) {
        const int64_t i = i0 + u * 256, row = i >> shift;
        dst[u] = -1;
        if (i >= per_seq) continue;
        const int h = (int)(row / T), r = (int)(row % T);
        if (r >= m) continue;
        const int tok = n - m + r, page = __ldg(p.table + (size_t)b * p.W + tok / p.S);
        if ((unsigned)page >= (unsigned)p.P) continue;
        dst[u] = ((((int64_t)page * p.Hkv + h) * p.S + tok % p.S) << shift) + (i & ((1 << shift) - 1));
        k[u] = __ldcs(k_new + (size_t)b * per_seq + i);
        v[u] = __ldcs(v_new + (size_t)b * per_seq + i);
    }
#pragma unroll
    for (int u = 0; u < kAppendPer; ++u)
        if (dst[u] >= 0) {
            __stcs(K + dst[u], k[u]);
            __stcs(V + dst[u], v[u]);
        }
}

}  // namespace

cudaError_t launch_pages_init(int32_t* state, int32_t* table, int32_t* len, int B, int P, int W, cudaStream_t st) {
    const int64_t entries = (int64_t)B * W, most = entries > P ? entries : P, want = (most + 255) / 256;
    pages_init_kernel<<<(unsigned)(want < 1184 ? want : 1184), 256, 0, st>>>(state, table, len, P, B, entries);
    return cudaGetLastError();
}

cudaError_t launch_pages_reserve(const int32_t* add, int32_t* state, int32_t* table, int32_t* len, int32_t* grant,
                                 int32_t* moves, int B, int N, int S, int P, int W, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const int smem = 6 * B * (int)sizeof(int);
    const cudaError_t e = allow_smem(pages_reserve_kernel, 6 * kReserveMaxSeqs * (int)sizeof(int), done);
    if (e != cudaSuccess) return e;
    pages_reserve_kernel<<<1, 1024, smem, st>>>(add, state, table, len, grant, moves, B, N, S, P, W);
    return cudaGetLastError();
}

cudaError_t launch_pages_fork(const int32_t* parent, int32_t* state, const int32_t* table, const int32_t* len,
                              int32_t* table_out, int32_t* len_out, int B, int P, int W, cudaStream_t st) {
    const int tiles = (W + 255) / 256;
    const PageState L(P);
    if ((int64_t)B * W <= kSmallTable) {
        pages_fork_small_kernel<<<1, 1024, 0, st>>>(parent, state, reinterpret_cast<unsigned*>(state + L.bits()), table, len,
                                                    table_out, len_out, B, P, W);
        return cudaGetLastError();
    }
    pages_fork_kernel<<<(unsigned)((int64_t)B * tiles), 256, 0, st>>>(parent, state, table, len, table_out, len_out, B,
                                                                      P, W, tiles);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    pages_unfork_kernel<<<(unsigned)((int64_t)B * tiles), 256, 0, st>>>(
        parent, state, reinterpret_cast<unsigned*>(state + L.bits()), table, P, W, tiles);
    return cudaGetLastError();
}

cudaError_t launch_pages_free(const int32_t* seqs, int n, int32_t* state, int32_t* table, int32_t* len, int B, int P,
                              int W, cudaStream_t st) {
    const int tiles = (W + 255) / 256;
    const PageState L(P);
    pages_free_kernel<<<(unsigned)((int64_t)n * tiles), 256, 0, st>>>(
        seqs, state, reinterpret_cast<unsigned*>(state + L.bits()), table, len, B, P, W, tiles);
    return cudaGetLastError();
}

cudaError_t launch_pages_compact(int32_t* state, int32_t* table, int32_t* moves, int max_moves, int B, int P, int W,
                                 cudaStream_t st) {
    const int64_t entries = (int64_t)B * W;
    const PageState L(P);
    if (entries <= kSmallTable && P <= kSmallTable) {
        compact_small_kernel<<<1, 1024, 0, st>>>(state, table, moves, P, (int)entries, max_moves);
        return cudaGetLastError();
    }
    compact_scan_kernel<<<1, 1024, 0, st>>>(state, moves, P);
    compact_move_kernel<<<(unsigned)(((int64_t)P + 255) / 256), 256, 0, st>>>(state, moves, P, max_moves);
    compact_table_kernel<<<(unsigned)((entries + 255) / 256), 256, 0, st>>>(state + L.map(), table, moves, P, entries);
    return cudaGetLastError();
}

template <int TEAM>
static cudaError_t launch_copy(const int32_t* moves, int max_moves, void* K, void* V, int64_t page_bytes, int P, int sms,
                               cudaStream_t st) {
    if constexpr (TEAM > 32)
        if (page_bytes <= (int64_t)TEAM / 2 * kCopyPer * 16)
            return launch_copy<TEAM / 2>(moves, max_moves, K, V, page_bytes, P, sms, st);
    constexpr int kTeams = kCopyThreads / TEAM;
    const int segments = (int)((page_bytes + kSegment - 1) / kSegment);
    const int64_t want = ((int64_t)max_moves * 2 * segments + kTeams - 1) / kTeams, most = (int64_t)sms * 64;
    pages_copy_kernel<TEAM><<<(unsigned)(want < most ? want : most), kCopyThreads, 0, st>>>(
        moves, (uint8_t*)K, (uint8_t*)V, page_bytes, segments, P, max_moves);
    return cudaGetLastError();
}

cudaError_t launch_pages_copy(const int32_t* moves, int max_moves, void* K, void* V, int64_t page_bytes, int P, int sms,
                              cudaStream_t st) {
    return launch_copy<kCopyThreads>(moves, max_moves, K, V, page_bytes, P, sms, st);
}

cudaError_t launch_paged_append(int row_bytes, const void* k_new, const void* v_new, int T, const int32_t* count, void* K,
                                void* V, const PagedParams& p, cudaStream_t st) {
    int shift = 0;
    while ((16 << shift) < row_bytes) ++shift;  // row_bytes is 128, 256 or 512
    const int64_t per_seq = ((int64_t)p.Hkv * T) << shift, per_block = 256 * kAppendPer,
                  tiles = (per_seq + per_block - 1) / per_block;
    paged_append_kernel<<<(unsigned)(p.B * tiles), 256, 0, st>>>((const uint4*)k_new, (const uint4*)v_new, count,
                                                                 (uint4*)K, (uint4*)V, T, shift, per_seq, (int)tiles, p);
    return cudaGetLastError();
}

}  // namespace pisa
