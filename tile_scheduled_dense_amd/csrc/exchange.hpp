// exchange.hpp -- tokens to expert order and back: the sort of a router's
// choices, the gather of the tokens' rows, the weighted sum back, its gradient.
//
// All of it moves rows: every kernel here is bound by memory, so each reads its
// inputs once, writes its outputs once and holds sums in fp32 registers.
// Measured: sort, gather, combine, its gradient and the gather's, 8192 tokens x 2 choices x
// 2048 bf16, 95 us (4.9 TB/s, what a large copy reaches on this card); 1999 x 8 x 1001 fp32,
// rows off 16 bytes, 86 us (4.1 TB/s); 16 tokens x 1024 16 us, three calls' host time.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_rows.hpp"
#include "grid.hpp"

namespace tg {

// ---- typed 16-byte chunks ---------------------------------------------------------
// A chunk is 16 bytes of a row at any element boundary: rows of odd length start
// anywhere, and gfx950 serves an unaligned 128-bit access as one instruction.
typedef u32x4 __attribute__((aligned(2))) u32x4_any;

template <int DT>
struct Row {
    typedef typename ElemOf<DT>::type T;
    static constexpr int PER = 16 / (int)sizeof(T);     // elements per chunk
    typedef T vec __attribute__((ext_vector_type(PER)));

    // Chunk c of a row of `cols` elements.  A last chunk that the row's end cuts is moved
    // back to end with the row: its first elements are the previous chunk's once more,
    // read, and written with the same values.  Only a row shorter than a chunk goes
    // element by element.
    __device__ __forceinline__ static int64_t first(int64_t c, int64_t cols) {
        return (c + 1) * PER <= cols || cols < PER ? c * PER : cols - PER;
    }
    __device__ __forceinline__ static u32x4 load(const T *row, int64_t c, int64_t cols) {
        if (cols >= PER) return *reinterpret_cast<const u32x4_any *>(row + first(c, cols));
        vec v = {};
#pragma unroll
        for (int e = 0; e < PER - 1; ++e)
            if (e < cols) v[e] = row[e];
        return __builtin_bit_cast(u32x4, v);
    }
    // PAST: with the non-temporal hint
    template <bool PAST = false>
    __device__ __forceinline__ static void store(T *row, int64_t c, int64_t cols, u32x4 x) {
        if (cols >= PER) {
            u32x4_any *at = reinterpret_cast<u32x4_any *>(row + first(c, cols));
            if constexpr (PAST) __builtin_nontemporal_store(x, at);
            else *at = x;
            return;
        }
        const vec v = __builtin_bit_cast(vec, x);
#pragma unroll
        for (int e = 0; e < PER - 1; ++e)
            if (e < cols) row[e] = v[e];
    }
    __device__ __forceinline__ static void widen(u32x4 x, float (&f)[PER]) {
        const vec v = __builtin_bit_cast(vec, x);
#pragma unroll
        for (int e = 0; e < PER; ++e) f[e] = (float)v[e];
    }
    // one rounding to the storage type, to nearest even
    __device__ __forceinline__ static u32x4 narrow(const float (&f)[PER]) {
        vec v;
#pragma unroll
        for (int e = 0; e < PER; ++e) v[e] = (T)f[e];
        return __builtin_bit_cast(u32x4, v);
    }
};

// ---- sort --------------------------------------------------------------------------
// A stable counting sort on keys 0 .. experts (the last: no expert).  A wave
// takes 64 consecutive entries at a time; the lanes that share a key find each
// other with one ballot per key bit, a lane's rank among them is a population
// count, and the wave's own histogram in LDS carries the ranks from one 64 to
// the next, so the order is the entries'.  Waves of a block are joined by a scan
// over their histograms.  Blocks are joined by the counts of sort_count_kernel,
// which every block of sort_place_kernel sums for itself, one load of a lane each.
// No atomics.  (Every block counting all entries for itself, in LDS atomics and one
// launch, took 19 us for 16384 entries of 8 experts, against 11 in two launches.)
// Bound by latency: 16384 entries are 64 KiB; 4.8 us for the counts, 6.2 for the places,
// and 3.5 in one block for 32 entries.
constexpr int kSortBlocks = 64;
constexpr int kSortOnce = 4;       // steps a wave at most for one block to take them all
// waves of a sorting block: their histograms are waves * (experts + 1) ints of LDS, 32 KiB at most
inline int sort_waves(int64_t experts) { return experts < 512 ? 16 : 4; }

struct SortShape {
    int waves, iters;      // a wave takes iters * 64 consecutive entries
    int64_t blocks;
};
inline SortShape sort_shape(int64_t n, int64_t experts) {
    SortShape s;
    s.waves = sort_waves(experts);
    const int64_t step = s.waves * 64;
    const int64_t steps = (n + step - 1) / step;
    s.iters = (int)(steps <= kSortOnce ? (steps > 1 ? steps : 1) : (steps + kSortBlocks - 1) / kSortBlocks);
    s.blocks = n > step * s.iters ? (n + step * s.iters - 1) / (step * s.iters) : 1;
    return s;
}

struct SortParams {
    const int32_t *ids;
    int64_t ld_ids;
    int32_t *offsets, *entry_of_row, *row_of_entry, *counts;
    int n, top_k, experts, bits, iters, blocks;
};

__device__ __forceinline__ int sort_key(const SortParams &p, int entry) {
    int64_t at = entry;
    if (p.ld_ids != p.top_k) {
        const int t = entry / p.top_k;
        at = (int64_t)t * p.ld_ids + (entry - t * p.top_k);
    }
    const int id = p.ids[at];
    return (uint32_t)id < (uint32_t)p.experts ? id : p.experts;
}

// lanes of the wave with this lane's key, among the active ones
__device__ __forceinline__ uint64_t same_key(int key, int bits, uint64_t active) {
    uint64_t m = active;
    for (int b = 0; b < bits; ++b) {
        const uint64_t ones = __ballot((key >> b) & 1);
        m &= ((key >> b) & 1) ? ones : ~ones;
    }
    return m;
}

// One step of a wave: 64 entries into its histogram (a key has one leader among
// them); returns this lane's rank among the wave's entries of its key so far.
__device__ __forceinline__ int sort_step(int key, bool in, int bits, int lane, volatile int *hist) {
    const uint64_t m = same_key(key, bits, __ballot(in));
    const int seen = in ? hist[key] : 0;
    __builtin_amdgcn_wave_barrier();
    if (in && __builtin_ctzll(m) == lane) hist[key] = seen + __popcll(m);
    __builtin_amdgcn_wave_barrier();
    return seen + __popcll(m & ((1ull << lane) - 1));
}

static __global__ __launch_bounds__(1024) void sort_count_kernel(SortParams p) {
    extern __shared__ int sort_lds[];
    const int keys = p.experts + 1, wave = threadIdx.x >> 6, lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    for (int i = threadIdx.x; i < waves * keys; i += blockDim.x) sort_lds[i] = 0;
    __syncthreads();
    const int first = (blockIdx.x * waves + wave) * p.iters * 64;
    for (int i = 0; i < p.iters; ++i) {
        const int entry = first + i * 64 + lane;
        const bool in = entry < p.n;
        sort_step(in ? sort_key(p, entry) : p.experts, in, p.bits, lane, sort_lds + wave * keys);
    }
    __syncthreads();
    for (int k = threadIdx.x; k < keys; k += blockDim.x) {
        int sum = 0;
        for (int w = 0; w < waves; ++w) sum += sort_lds[w * keys + k];
        p.counts[k * p.blocks + blockIdx.x] = sum;      // a key's counts lie together
    }
}

// KEPT: a wave's steps are at most that many, their keys and ranks kept in
// registers (0: any number, found again for the second pass).
template <int KEPT>
static __global__ __launch_bounds__(1024) void sort_place_kernel(SortParams p) {
    extern __shared__ int sort_lds[];
    __shared__ int wave_sum[16];
    const int keys = p.experts + 1, wave = threadIdx.x >> 6, lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    int *hist = sort_lds;                     // [waves][keys]
    int *total = sort_lds + waves * keys;     // [keys]: entries of the key, then its first row
    int *before = total + keys;               // [keys]: those in earlier blocks
    for (int i = threadIdx.x; i < (waves + 2) * keys; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    const int first = (blockIdx.x * waves + wave) * p.iters * 64;
    volatile int *mine_hist = hist + wave * keys;
    int kept_key[KEPT ? KEPT : 1], kept_rank[KEPT ? KEPT : 1];
    if constexpr (KEPT > 0) {
#pragma unroll
        for (int i = 0; i < KEPT; ++i) {
            const int entry = first + i * 64 + lane;
            kept_key[i] = i < p.iters && entry < p.n ? sort_key(p, entry) : -1;
        }
#pragma unroll
        for (int i = 0; i < KEPT; ++i)
            if (i < p.iters)
                kept_rank[i] = sort_step(kept_key[i] < 0 ? p.experts : kept_key[i], kept_key[i] >= 0, p.bits, lane, mine_hist);
    } else {
        for (int i = 0; i < p.iters; ++i) {
            const int entry = first + i * 64 + lane;
            const bool in = entry < p.n;
            sort_step(in ? sort_key(p, entry) : p.experts, in, p.bits, lane, mine_hist);
        }
    }
    if (p.blocks > 1) {
        // groups of `span` lanes take a key each, a lane a block's count
        int span = 1;
        while (span < p.blocks) span *= 2;
        const int per = 64 / span, sub = lane / span, blk = lane % span;
        for (int k0 = wave * per; k0 < keys; k0 += waves * per) {
            const int k = k0 + sub;
            int c = 0;
            if (k < keys && blk < p.blocks && blk != (int)blockIdx.x) c = p.counts[k * p.blocks + blk];
            int b = blk < (int)blockIdx.x ? c : 0;
            for (int d = 1; d < span; d *= 2) {
                c += __shfl_xor(c, d);
                b += __shfl_xor(b, d);
            }
            if (k < keys && blk == 0) {
                total[k] = c;
                before[k] = b;
            }
        }
    }
    __syncthreads();
    // a key's waves in order: exclusive sums over the histograms; total: this block's too
    for (int k = threadIdx.x; k < keys; k += blockDim.x) {
        int sum = 0;
        for (int w = 0; w < waves; ++w) {
            const int c = hist[w * keys + k];
            hist[w * keys + k] = sum;
            sum += c;
        }
        total[k] += sum;
    }
    __syncthreads();
    // the first row of every key: an exclusive sum over the totals, `share` keys a thread
    const int share = (keys + (int)blockDim.x - 1) / (int)blockDim.x;
    int mine = 0;
    for (int i = 0; i < share; ++i) {
        const int k = threadIdx.x * share + i;
        if (k < keys) mine += total[k];
    }
    int incl = mine;
    for (int d = 1; d < 64; d *= 2) {
        const int up = __shfl_up(incl, d);
        if (lane >= d) incl += up;
    }
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    int at = incl - mine;
    for (int w = 0; w < wave; ++w) at += wave_sum[w];
    for (int i = 0; i < share; ++i) {
        const int k = threadIdx.x * share + i;
        if (k < keys) {
            const int c = total[k];
            total[k] = at;
            if (blockIdx.x == 0) p.offsets[k] = at;
            at += c;
        }
    }
    __syncthreads();
    auto place = [&](int entry, int key, int rank) {
        const int row = total[key] + before[key] + rank;
        p.entry_of_row[row] = key < p.experts ? entry : ~entry;
        p.row_of_entry[entry] = key < p.experts ? row : ~row;
    };
    if constexpr (KEPT > 0) {
#pragma unroll
        for (int i = 0; i < KEPT; ++i)
            if (kept_key[i] >= 0)
                place(first + i * 64 + lane, kept_key[i], mine_hist[kept_key[i]] + kept_rank[i]);
    } else {
        for (int i = 0; i < p.iters; ++i) {
            const int entry = first + i * 64 + lane;
            const bool in = entry < p.n;
            const int key = in ? sort_key(p, entry) : p.experts;
            const int rank = sort_step(key, in, p.bits, lane, mine_hist);   // on from the earlier waves'
            if (in) place(entry, key, rank);
        }
    }
}

// ---- rows ---------------------------------------------------------------------------
// `group` threads, 16 to 256, take a token's row, a chunk each at a time, and 256 /
// group tokens fill a workgroup.  From 64 on a wave has one token, and its table
// entries and weights are scalar loads; NARROW: fewer, for rows of up to 32 chunks
// (6508 x 118 bf16 of 8 choices and 91 experts: forward and backward 87 us with a wave
// for each 15 chunks, 39 us with 16 lanes).
inline int row_group(int64_t chunks) {
    return chunks > 128 ? 256 : (chunks > 64 ? 128 : (chunks > 32 ? 64 : (chunks > 16 ? 32 : 16)));
}
// whether a call that moves so many bytes stores past the caches (gather_kernel)
inline bool store_past(int64_t bytes) { return bytes > (int64_t(64) << 20); }
inline dim3 token_grid(int64_t tokens, int group) { return wide_grid((tokens + 256 / group - 1) / (256 / group)); }
template <bool NARROW>
__device__ __forceinline__ uint32_t token_of(int group) {
    const uint32_t t = wide_block() * (256 / group) + threadIdx.x / group;
    return NARROW ? t : __builtin_amdgcn_readfirstlane(t);
}

// PAST: results are stored past the caches, where a call moves more than 64 MiB:
// lines that one call leaves dirty in them are written back during the next call's
// reads.  A pass of gather, combine, its gradient and the gather's gradient, 8192 x
// 2048 bf16 of 2 choices, takes 113 us without the hint and 99 with it; 1999 x 1001
// fp32 of 8 choices 96 and 87 (where the gather alone, its rows off 16 bytes, takes 18
// in place of 15).  The hint on loads too: 106.
template <int DT, bool PAST, bool NARROW>
__global__ __launch_bounds__(256) void gather_kernel(const typename ElemOf<DT>::type *__restrict__ x, int64_t ldx,
                                                     const int32_t *__restrict__ row_of_entry,
                                                     typename ElemOf<DT>::type *__restrict__ rows, int64_t ldr,
                                                     int tokens, int top_k, int64_t cols, int group) {
    using R = Row<DT>;
    const uint32_t t = token_of<NARROW>(group);
    if (t >= (uint32_t)tokens) return;
    const int n = tokens * top_k;
    const int32_t *row = row_of_entry + (int64_t)t * top_k;
    const int64_t chunks = (cols + R::PER - 1) / R::PER;
    for (int64_t c = threadIdx.x % group; c < chunks; c += group) {
        const u32x4 v = R::load(x + (int64_t)t * ldx, c, cols);
        for (int j = 0; j < top_k; ++j) {
            const int r = row[j], at = r < 0 ? ~r : r;
            if (at < n) R::template store<PAST>(rows + (int64_t)at * ldr, c, cols, r < 0 ? u32x4{0, 0, 0, 0} : v);
        }
    }
}

// JB choices of a token and U chunks at a time, their loads in flight together.  A
// choice without an expert loads row 0 in its place (in cache after the first) and is
// left out of the sum by selection, so that what lies there, a NaN say, goes nowhere.
template <int DT, int JB, int U, bool PAST, bool NARROW>
__global__ __launch_bounds__(256) void combine_kernel(const typename ElemOf<DT>::type *__restrict__ y, int64_t ldy,
                                                      const int32_t *__restrict__ row_of_entry,
                                                      const float *__restrict__ weights, int64_t ld_w,
                                                      typename ElemOf<DT>::type *__restrict__ out, int64_t ldo,
                                                      int tokens, int top_k, int64_t cols, int group) {
    using R = Row<DT>;
    const uint32_t t = token_of<NARROW>(group);
    if (t >= (uint32_t)tokens) return;
    const int n = tokens * top_k;
    const int32_t *row = row_of_entry + (int64_t)t * top_k;
    const int64_t chunks = (cols + R::PER - 1) / R::PER;
    for (int64_t c = threadIdx.x % group; c < chunks; c += U * group) {
        float sum[U][R::PER] = {};
        for (int j0 = 0; j0 < top_k; j0 += JB) {
            u32x4 v[JB][U];
            float w[JB];
            bool has[JB];
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                const int r = j0 + j < top_k ? row[j0 + j] : -1;
                has[j] = (uint32_t)r < (uint32_t)n;
                w[j] = has[j] && weights ? weights[(int64_t)t * ld_w + j0 + j] : 1.0f;
                const typename ElemOf<DT>::type *from = y + (has[j] ? (int64_t)r * ldy : 0);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (u == 0 || c + u * group < chunks) v[j][u] = R::load(from, c + u * group, cols);
            }
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                if (!has[j]) continue;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float f[R::PER];
                    R::widen(v[j][u], f);
#pragma unroll
                    for (int e = 0; e < R::PER; ++e) sum[u][e] = __builtin_fmaf(w[j], f[e], sum[u][e]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u == 0 || c + u * group < chunks)
                R::template store<PAST>(out + (int64_t)t * ldo, c + u * group, cols, R::narrow(sum[u]));
    }
}

// `group` of 16, 32 or 64 lanes a token: the dot products are summed over them without LDS.
template <int DT, int JB, bool PAST, bool NARROW>
__global__ __launch_bounds__(256) void combine_grad_kernel(const typename ElemOf<DT>::type *__restrict__ d_out,
                                                           int64_t ldo,
                                                           const typename ElemOf<DT>::type *__restrict__ y,
                                                           int64_t ldy, const int32_t *__restrict__ row_of_entry,
                                                           const float *__restrict__ weights, int64_t ld_w,
                                                           typename ElemOf<DT>::type *__restrict__ d_y, int64_t ldd,
                                                           float *__restrict__ d_w, int64_t ld_dw, int tokens,
                                                           int top_k, int64_t cols, int group) {
    using R = Row<DT>;
    const uint32_t t = token_of<NARROW>(group);
    const int lane = threadIdx.x % group;
    if (t >= (uint32_t)tokens) return;
    const int n = tokens * top_k;
    const int32_t *row = row_of_entry + (int64_t)t * top_k;
    const int64_t chunks = (cols + R::PER - 1) / R::PER;
    for (int j0 = 0; j0 < top_k; j0 += JB) {
        float w[JB], dot[JB];
        int at[JB];           // the choice's row, or -1 past top_k or outside the table
        bool has[JB];
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            const int r = j0 + j < top_k ? row[j0 + j] : n;
            has[j] = (uint32_t)r < (uint32_t)n;
            at[j] = has[j] ? r : (r < 0 && ~r < n ? ~r : -1);
            w[j] = has[j] ? weights[(int64_t)t * ld_w + j0 + j] : 0.0f;
            dot[j] = 0.0f;
        }
        for (int64_t c = lane; c < chunks; c += group) {
            const int64_t again = cols >= R::PER ? c * R::PER - R::first(c, cols) : 0;   // elements of the previous chunk
            float g[R::PER];
            u32x4 v[JB];
            R::widen(R::load(d_out + (int64_t)t * ldo, c, cols), g);
#pragma unroll
            for (int j = 0; j < JB; ++j) v[j] = R::load(y + (has[j] ? (int64_t)at[j] * ldy : 0), c, cols);
#pragma unroll
            for (int j = 0; j < JB; ++j) {
                float f[R::PER], d[R::PER];
                R::widen(v[j], f);
#pragma unroll
                for (int e = 0; e < R::PER; ++e) {
                    dot[j] = has[j] && e >= again ? __builtin_fmaf(g[e], f[e], dot[j]) : dot[j];
                    d[e] = has[j] ? w[j] * g[e] : 0.0f;
                }
                if (at[j] >= 0) R::template store<PAST>(d_y + (int64_t)at[j] * ldd, c, cols, R::narrow(d));
            }
        }
#pragma unroll
        for (int j = 0; j < JB; ++j) {
            for (int d = group / 2; d > 0; d /= 2) dot[j] += __shfl_xor(dot[j], d);
            if (lane == 0 && j0 + j < top_k) d_w[(int64_t)t * ld_dw + j0 + j] = dot[j];
        }
    }
}

}  // namespace tg
