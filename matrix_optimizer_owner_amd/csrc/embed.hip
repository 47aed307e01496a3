// embed.hip - an embedding table that is one entry of an owner buffer:
// lookup with scaling, and the table's gradient, on gfx950.
//
//   lookup:  out[i] = scale * W[id_i - first];
//   grad:    G[v] (+)= scale * sum over i with id_i - first = v of dout[i].
#include <algorithm>
#include <string>

#include "device_util.h"
#include "plan_internal.h"

namespace mfsdp {
namespace {

// ---- ids and elements ----

// Row of position i, or `rows` for an id outside the table.  The difference is
// taken modulo 2^64: first is at most 2^62, so no id outside wraps into it.
__device__ __forceinline__ int row_of(const void* ids, int id_type, int64_t i, int64_t first, int rows) {
    const int64_t id = id_type == MFSDP_I64 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
    const uint64_t r = uint64_t(id) - uint64_t(first);
    return r < uint64_t(rows) ? int(r) : rows;
}

// A 16-byte word at any element address: rows of an odd width start anywhere,
// and global accesses of this width need no alignment here.
typedef unsigned int word_t __attribute__((ext_vector_type(4), aligned(2)));

// N consecutive elements of type DT as the words they are stored in.
template <int DT, int N> struct Raw {
    static constexpr int kWords = N * (DT == kBF16 ? 2 : 4) / 16;
    static constexpr int kSize = DT == kBF16 ? 2 : 4;
    u32x4_t w[kWords];
    // The first `width` of N elements at p, the end of a row; nothing behind it is read.  A row of N elements or more
    // (`wide`) is read by whole words: its last lane takes the N that end with the row, and settle() moves its own
    // down.  The two are apart so that a batch of loads is on its way before the first is waited for (4144 ids of
    // 2764 columns take 66 us with them together, or element by element).
    template <bool STREAM> __device__ __forceinline__ void load(const uint8_t* p, int width, bool wide) {
        if (width == N || wide) {
            const int back = N - width;
            const word_t* q = reinterpret_cast<const word_t*>(p - back * kSize);
#pragma unroll
            for (int k = 0; k < kWords; ++k) w[k] = STREAM ? __builtin_nontemporal_load(q + k) : q[k];
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) {
                uint32_t v = 0;
                if (k < width)
                    v = DT == kBF16 ? uint32_t(reinterpret_cast<const uint16_t*>(p)[k]) : reinterpret_cast<const uint32_t*>(p)[k];
                if (DT == kBF16)
                    w[k / 8][k / 2 % 4] = k % 2 ? w[k / 8][k / 2 % 4] | v << 16 : v;
                else
                    w[k / 4][k % 4] = v;
            }
        }
    }
    __device__ __forceinline__ void settle(int width, bool wide) {
        if (width == N || !wide) return;
#pragma unroll
        for (int step = N / 2; step > 0; step /= 2)
            if ((N - width) & step) move_down(step);
    }
    // element k becomes element k + n, for the elements that there are (n a compile-time power of two after unrolling)
    __device__ __forceinline__ void move_down(int n) {
        constexpr int kDwords = kWords * 4;
        if (DT == kBF16 && n == 1) {
#pragma unroll
            for (int d = 0; d < kDwords; ++d)
                w[d / 4][d % 4] = w[d / 4][d % 4] >> 16 | (d + 1 < kDwords ? w[(d + 1) / 4][(d + 1) % 4] << 16 : 0u);
            return;
        }
        const int dn = DT == kBF16 ? n / 2 : n;
#pragma unroll
        for (int d = 0; d < kDwords; ++d)
            if (d + dn < kDwords) w[d / 4][d % 4] = w[(d + dn) / 4][(d + dn) % 4];
    }
    __device__ __forceinline__ float get(int k) const {
        if (DT == kBF16) {
            const uint32_t x = w[k / 8][k / 2 % 4];
            return __uint_as_float(k % 2 ? x & 0xffff0000u : x << 16);
        }
        return __uint_as_float(w[k / 4][k % 4]);
    }
};

// N floats rounded once and stored as `width` elements of type DT.
template <int DT, int N, bool STREAM> __device__ __forceinline__ void store(void* p, int width, const float (&v)[N]) {
    if (width == N) {
        constexpr int kWords = Raw<DT, N>::kWords;
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            u32x4_t w;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = DT == kBF16 ? pack_bf16x2(v[(k * 8 + 2 * e) % N], v[(k * 8 + 2 * e + 1) % N])
                                   : __float_as_uint(v[(k * 4 + e) % N]);
            word_t* q = static_cast<word_t*>(p) + k;
            if (STREAM)
                __builtin_nontemporal_store(w, q);
            else
                *q = w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (k < width) store_elem(p, DT, k, v[k]);
    }
}

// ---- lookup ----

constexpr int kLookupThreads = 512;
constexpr int64_t kBlocksMax = (int64_t(1) << 23) - 1;  // a launch holds fewer than 2^32 threads

struct LookupArgs {
    const uint8_t* table;
    const void* ids;
    uint8_t* out;
    int64_t n, first, out_stride;
    int rows, cols;
    int id_type;
    int group_shift;  // 2^group_shift lanes a row; grid.y such groups side by side
    float scale;
};

// HBM-bound: each id's row is read and written once.  One word of the
// narrower type a thread and no loop, the shape that copies fastest here
// (grad.hip); 2^group_shift lanes share a position, so narrow rows fill the
// wave too.  Stores go past the caches and loads through them, which keeps
// the rows that many ids share: 16384 ids into 128256 x 4096 bf16 take 32 us
// (191 MB, 6.0 TB/s), 49 with ordinary stores, 47 with loads past the caches
// too.  first_block: the launch's first block.
template <int TD, int OD>
__global__ __launch_bounds__(kLookupThreads) void k_embed_lookup(LookupArgs a, int64_t first_block) {
    constexpr int N = TD == kF32 && OD == kF32 ? 4 : 8;
    const int64_t i = (first_block + blockIdx.x) * (kLookupThreads >> a.group_shift) + (threadIdx.x >> a.group_shift);
    const int lane = int(threadIdx.x) & ((1 << a.group_shift) - 1);
    const int c = ((int(blockIdx.y) << a.group_shift) + lane) * N;
    if (i >= a.n || c >= a.cols) return;
    const int r = row_of(a.ids, a.id_type, i, a.first, a.rows);
    const int width = a.cols - c < N ? a.cols - c : N;
    float v[N];
    if (r < a.rows) {
        Raw<TD, N> x;
        x.template load<false>(a.table + (int64_t(r) * a.cols + c) * Raw<TD, N>::kSize, width, a.cols >= N);
        x.settle(width, a.cols >= N);
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = a.scale * x.get(k);
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = 0.f;
    }
    store<OD, N, true>(a.out + (i * a.out_stride + c) * Raw<OD, N>::kSize, width, v);
}

// ---- gradient ----
//
// grad[v] (+)= scale * sum of dout[i] over the positions i of row v: fp32 sums
// in the order of the positions, cut at places that depend on the ids and
// sizes alone.  HBM-bound: dout is read once and every row written once.

struct GradArgs {
    uint8_t* grad;
    const void* ids;
    const uint8_t* dout;
    int64_t first, dout_stride;
    int rows, cols, n;
    int id_type;
    int group_shift, slabs;  // 2^group_shift lanes a row, `slabs` of them side by side
    float scale;
};

constexpr int kPer = 8;  // columns of a lane

template <int GD, bool ACC>
__device__ __forceinline__ void write_row(const GradArgs& a, int row, int c, int width, const float (&sum)[kPer]) {
    uint8_t* p = a.grad + (int64_t(row) * a.cols + c) * Raw<GD, kPer>::kSize;
    float v[kPer];
    if constexpr (ACC) {
        Raw<GD, kPer> old;
        old.template load<false>(p, width, a.cols >= kPer);
        old.settle(width, a.cols >= kPer);
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = __builtin_fmaf(a.scale, sum[k], old.get(k));
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = a.scale * sum[k];
    }
    store<GD, kPer, true>(p, width, v);
}

// The sum of dout rows at(0) .. at(count-1), columns c .. c + width, kUnroll loads in flight.
template <int OD, typename F>
__device__ __forceinline__ void sum_rows(const GradArgs& a, F at, int count, int c, int width, float (&acc)[kPer]) {
    constexpr int kUnroll = 8;
    for (int q = 0; q < count; q += kUnroll) {
        Raw<OD, kPer> x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (q + u < count)
                x[u].template load<true>(a.dout + (int64_t(at(q + u)) * a.dout_stride + c) * Raw<OD, kPer>::kSize, width,
                                            a.cols >= kPer);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (q + u < count) {
                x[u].settle(width, a.cols >= kPer);
#pragma unroll
                for (int k = 0; k < kPer; ++k) acc[k] += x[u].get(k);
            }
    }
}

// Every thread's acc, added over the groups of a block of THREADS: within a
// wave pairwise, then wave by wave (an order that the sizes alone fix).
// Valid in group 0.  All threads call it.
template <int THREADS> __device__ __forceinline__ void add_groups(float* red, int group_shift, float (&acc)[kPer]) {
    const int lane = threadIdx.x & 63, G = 1 << group_shift;
    for (int off = G; off < 64; off <<= 1)
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[k] += __shfl_xor(acc[k], off, 64);
    if (lane < G)
#pragma unroll
        for (int k = 0; k < kPer; ++k) red[k * THREADS + threadIdx.x] = acc[k];
    __syncthreads();
    if (threadIdx.x >= unsigned(G)) return;
    for (int w = 1; w < THREADS / 64; ++w)
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[k] += red[k * THREADS + w * 64 + lane];
}

// Zeros over the whole table's gradient: one word a thread, the shape that
// writes fastest here (6.9 TB/s; 5.9 with 128 KB a block).
constexpr int kZeroThreads = 256;
__device__ __forceinline__ void fill_zeros(uint8_t* grad, int64_t bytes, int64_t word) {
    const int64_t at = word * 16;
    if (at + 16 <= bytes)
        *reinterpret_cast<u32x4_t*>(grad + at) = u32x4_t{0u, 0u, 0u, 0u};
    else
        for (int64_t b = at; b < bytes; b += 2) *reinterpret_cast<uint16_t*>(grad + b) = 0;
}
__global__ __launch_bounds__(kZeroThreads) void k_embed_zero(uint8_t* grad, int64_t bytes, int64_t first_block) {
    fill_zeros(grad, bytes, (first_block + blockIdx.x) * kZeroThreads + threadIdx.x);
}

// Few ids: a block of position i looks through all of them, ends if an
// earlier one has the same row, and else sums that row's positions in order.
// No sort and no workspace; the work grows with n^2, so only up to kFewIds.
// A block has kFewSlabs groups' worth of columns: with one, every row is
// looked for once more per group of columns, with all, a hot row is summed by
// one block.  Added to 5000 rows of bf16, us with 1, 2, 3 and 4: 1000 ids of
// 4096 columns as in text 26, 18, 16, 19, spread evenly 32, 21, 17, 13, one id
// over and over 43, 63, 88, 116; 2000 of 1536 columns 21, 16, 20, 20, then 26,
// 21, 14, 14, then 64, 113, 167, 167.  So a batch of one id is what this is
// slow at (2000 of 512 columns 56 us, as in text 9).  512 threads (2000 ids of
// 1536 columns: 20 us, 31 with 256; spread evenly 14 and 11); past kFewIds the
// sort is faster (at 1500 ids of 256 columns this takes 9 us, the sort 22; at
// 4096 of 768 columns this 48, the sort 30).
constexpr int kFewIds = 2048, kFewThreads = 512, kFewSlabs = 3;

template <int T, int IDS, int OD, int GD, bool ACC>
__device__ __forceinline__ void few_ids(const GradArgs& a, int i, int part) {
    constexpr int kWaves = T / 64, kRounds = IDS / T;
    __shared__ int list[IDS];
    __shared__ int wave_first[kWaves], wave_n[kWaves];
    __shared__ float red[T * kPer];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = row_of(a.ids, a.id_type, i, a.first, a.rows);
    if (row == a.rows) return;
    // wave w has the positions from w * rounds * 64 on, in order
    const int rounds = (a.n + T - 1) / T;
    uint64_t hits[kRounds];
    int found = 0, first = INT32_MAX;
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const int p = (wave * rounds + k) * 64 + lane;
        hits[k] = __ballot(k < rounds && p < a.n && row_of(a.ids, a.id_type, k < rounds && p < a.n ? p : 0, a.first, a.rows) == row);
        if (hits[k] && first == INT32_MAX) first = p - lane + __builtin_ctzll(hits[k]);
        found += __popcll(hits[k]);
    }
    if (lane == 0) {
        wave_first[wave] = first;
        wave_n[wave] = found;
    }
    __syncthreads();
    int at = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (wave_first[w] < i) return;  // an earlier position's block has this row
        at += w < wave ? wave_n[w] : 0;
        total += wave_n[w];
    }
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        if (hits[k] >> lane & 1) list[at + __popcll(hits[k] & ((uint64_t(1) << lane) - 1))] = (wave * rounds + k) * 64 + lane;
        at += __popcll(hits[k]);
    }
    __syncthreads();
    const int slab0 = part * kFewSlabs, slab1 = a.slabs - slab0 < kFewSlabs ? a.slabs : slab0 + kFewSlabs;
    if (total <= 8) {  // a thread has them all in flight at once
        const int end = (slab1 << a.group_shift) * kPer < a.cols ? (slab1 << a.group_shift) * kPer : a.cols;
        for (int c = ((slab0 << a.group_shift) + int(threadIdx.x)) * kPer; c < end; c += T * kPer) {
            const int width = a.cols - c < kPer ? a.cols - c : kPer;
            float acc[kPer] = {};
            sum_rows<OD>(a, [&](int q) { return list[q]; }, total, c, width, acc);
            write_row<GD, ACC>(a, row, c, width, acc);
        }
        return;
    }
    const int g = threadIdx.x >> a.group_shift, groups = T >> a.group_shift;
    const int share = (total + groups - 1) / groups, lo = g * share;
    for (int slab = slab0; slab < slab1; ++slab) {
        const int c = ((slab << a.group_shift) + (int(threadIdx.x) & ((1 << a.group_shift) - 1))) * kPer;
        const int width = a.cols - c < kPer ? a.cols - c : kPer;
        float acc[kPer] = {};
        if (width > 0 && lo < total)
            sum_rows<OD>(a, [&](int q) { return list[lo + q]; }, total - lo < share ? total - lo : share, c, width, acc);
        add_groups<T>(red, a.group_shift, acc);
        if (g == 0 && width > 0) write_row<GD, ACC>(a, row, c, width, acc);
        __syncthreads();
    }
}

// Blocks of a position.
__host__ __device__ constexpr int few_parts(int slabs) { return (slabs + kFewSlabs - 1) / kFewSlabs; }

template <int OD, int GD, bool ACC> __global__ __launch_bounds__(kFewThreads) void k_embed_few(GradArgs a) {
    few_ids<kFewThreads, kFewIds, OD, GD, ACC>(a, int(blockIdx.x), int(blockIdx.y));
}

// The same with the zeros of the other rows beside it: a block has `span`
// whole rows of at most kSpanWords words, or a piece of that many of one
// longer row, and looks through the ids for its rows first.  A word that two
// rows share is the first one's.  One launch instead of two saves 3 us on a
// small table (500 ids into 61 MB: 12.6 us, 15.3 apart); past kFewBytes
// clearing without looking at ids wins (1.05 GB: 195 us, 183 apart).
constexpr int kSpanIds = 512, kSpanThreads = 256, kSpanWords = kSpanThreads * 2, kSpanRows = 1024;
constexpr int64_t kFewBytes = int64_t(128) << 20;

struct SpanArgs {
    int span, pieces;        // rows of a block, or blocks of a row
    int few_blocks;          // the launch's first ones
};

template <int GD> __device__ __forceinline__ void fill_span(const GradArgs& a, const SpanArgs& s, int block) {
    constexpr int kElems = GD == kBF16 ? 8 : 4, kSize = 16 / kElems;
    __shared__ uint8_t hit[kSpanRows + 4];
    const int g = block / s.pieces, piece = block - g * s.pieces, r0 = g * s.span;
    const int r1 = a.rows - r0 < s.span ? a.rows : r0 + s.span;
    int row[kSpanIds / kSpanThreads];
#pragma unroll
    for (int k = 0; k < kSpanIds / kSpanThreads; ++k) {
        const int p = k * kSpanThreads + int(threadIdx.x);
        row[k] = p < a.n ? row_of(a.ids, a.id_type, p, a.first, a.rows) : a.rows;
    }
    for (int r = threadIdx.x; r <= s.span; r += kSpanThreads) hit[r] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kSpanIds / kSpanThreads; ++k)
        if (row[k] >= r0 && row[k] <= r1 && row[k] < a.rows) hit[row[k] - r0] = 1;
    __syncthreads();
    const int64_t total = int64_t(a.rows) * a.cols, begin = int64_t(r0) * a.cols, end = int64_t(r1) * a.cols;
    const int64_t first = (begin + kElems - 1) / kElems + int64_t(piece) * kSpanWords + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kSpanWords / kSpanThreads; ++k) {
        const int64_t e = (first + k * kSpanThreads) * kElems;
        if (e >= end) return;
        const uint32_t x = uint32_t(e - begin);
        uint32_t r = x / uint32_t(a.cols), c = x - r * uint32_t(a.cols);
        if (c + kElems <= uint32_t(a.cols)) {  // a word of one row
            if (!hit[r]) *reinterpret_cast<u32x4_t*>(a.grad + e * kSize) = u32x4_t{0u, 0u, 0u, 0u};
            continue;
        }
        // a word over a row's end reaches into one more row (rows are at least a word wide here), at most into
        // r1, whose ids were looked for too
        for (int j = 0; j < kElems && e + j < total; ++j) {
            if (!hit[r]) store_elem(a.grad, GD, e + j, 0.f);
            if (++c == uint32_t(a.cols)) {
                c = 0;
                ++r;
            }
        }
    }
}

template <int OD, int GD> __global__ __launch_bounds__(kSpanThreads) void k_embed_few_fill(GradArgs a, SpanArgs s) {
    const int b = int(blockIdx.x);
    if (b < s.few_blocks)
        few_ids<kSpanThreads, kSpanIds, OD, GD, false>(a, b / few_parts(a.slabs), b % few_parts(a.slabs));
    else
        fill_span<GD>(a, s, b - s.few_blocks);
}

// More ids than that into few rows, or at least twice as many ids as rows: a
// block of each row (and `span` groups of columns) looks through all ids, each
// wave through its part, and sums what it finds; rows without an id get their
// zeros here too.  One launch: 9660 ids into 1218 x 15 take 17 us, sorted 51;
// 4144 into 154 x 2764 31 and 41; 1000 into 490 x 768 8.8, by the positions'
// blocks 11.3 (2000 into 2900 x 768 27 and 15).  The search grows with ids
// times rows (kRowsWork), and one block sums a row that most ids point to
// (kRowsHot: with 16000 ids and span 4, a tenth of them on one row, 218 us
// against 63), by more groups side by side if it is narrow, of at most
// 2^kRowsNarrow lanes (kRowsIds: 16000 of 96 columns 22 us, sorted 35; 12000
// of 256 fp32 columns 48 and 35).  Below these limits one id over and over is
// still one block's for each group of columns: 10240 times into 1000 x 512 it
// takes 273 us (as in text 38), where the sort takes 64 for a table of 50000
// rows; 8192 times into 2 x 768 it takes 112.
constexpr int kRowsThreads = 512, kRowsWaves = kRowsThreads / 64, kRowsHot = 10240, kRowsIds = 16384, kRowsNarrow = 4;
constexpr int64_t kRowsWork = int64_t(16) << 20;

// Ids of a wave, a multiple of 64.
__host__ __device__ constexpr int rows_part(int n) { return ((n + kRowsWaves - 1) / kRowsWaves + 63) / 64 * 64; }

template <int OD, int GD, bool ACC> __global__ __launch_bounds__(kRowsThreads) void k_embed_rows(GradArgs a, int span) {
    extern __shared__ uint16_t row_hits[];  // kRowsWaves parts
    __shared__ int wave_n[kRowsWaves];
    __shared__ float red[kRowsThreads * kPer];
    const int row = int(blockIdx.x), lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int part = rows_part(a.n), base = wave * part;
    uint16_t* const hits = row_hits + base;
    const int end = a.n - base < part ? a.n : base + part;
    int found = 0;
    constexpr int kUnroll = 8;
    for (int r = base; r < end; r += 64 * kUnroll) {
        int key[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int p = r + u * 64 + lane;
            key[u] = p < end ? row_of(a.ids, a.id_type, p, a.first, a.rows) : a.rows;
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint64_t m = __builtin_amdgcn_ballot_w64(key[u] == row);
            if (key[u] == row)
                hits[found + __popcll(m & ((uint64_t(1) << lane) - 1))] = uint16_t(r - base + u * 64 + lane);
            found += __popcll(m);
        }
    }
    if (lane == 0) wave_n[wave] = found;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < kRowsWaves; ++w) total += wave_n[w];
    const int slab0 = int(blockIdx.y) * span, slab1 = a.slabs - slab0 < span ? a.slabs : slab0 + span;
    if (total == 0) {
        if (ACC) return;
        const int last = (slab1 << a.group_shift) * kPer < a.cols ? (slab1 << a.group_shift) * kPer : a.cols;
        const float zero[kPer] = {};  // stored as they are: a product with a negative or infinite scale is no zero
        for (int c = ((slab0 << a.group_shift) + int(threadIdx.x)) * kPer; c < last; c += kRowsThreads * kPer)
            store<GD, kPer, true>(a.grad + (int64_t(row) * a.cols + c) * Raw<GD, kPer>::kSize,
                                  a.cols - c < kPer ? a.cols - c : kPer, zero);
        return;
    }
    // a wave's groups each take a stretch of what the wave found
    const int groups = 64 >> a.group_shift, g = lane >> a.group_shift;
    const int share = (found + groups - 1) / groups, lo = g * share;
    for (int slab = slab0; slab < slab1; ++slab) {
        const int c = ((slab << a.group_shift) + (lane & ((1 << a.group_shift) - 1))) * kPer;
        const int width = a.cols - c < kPer ? a.cols - c : kPer;
        float acc[kPer] = {};
        if (width > 0 && lo < found)
            sum_rows<OD>(a, [&](int q) { return base + int(hits[lo + q]); }, found - lo < share ? found - lo : share, c,
                         width, acc);
        add_groups<kRowsThreads>(red, a.group_shift, acc);
        if (int(threadIdx.x) < (1 << a.group_shift) && width > 0) write_row<GD, ACC>(a, row, c, width, acc);
        __syncthreads();
    }
}

// ---- many ids: sort positions by row, then sum runs of the sorted order ----
//
// The sort is a stable radix sort of (row, position), in one pass for fewer
// than 2048 rows and else in two over about half of the row's bits each: per
// pass one launch counts each tile's digits
// and one ranks and scatters.  Ids outside the table sort last, as row `rows`.

constexpr int kSortUnroll = 4, kOnePassBits = 11;

struct SortArgs {
    const void* ids;          // first pass; else keys_in and pos_in
    int64_t first;
    int rows, n, id_type;
    int tile, n_tiles;        // positions of a block, a multiple of 512
    int shift, bits;          // the pass's digit
    const int *keys_in, *pos_in;
    int* hist;                // [n_tiles][2^bits]
    int *keys_out, *pos_out;
    int* n_runs;              // cleared by the first launch
};

// Zeros beside the sort: the table's gradient is cleared by blocks that the
// sort's launches carry behind their own, an equal part each, so that the
// sort, which keeps a few CUs for some microseconds a launch, takes no time
// of its own.  One word a thread, the shape that writes fastest here.  (Clearing
// only the rows without an id, by a flag a row, saves their bytes but waits
// for the flag first: 4.1 TB/s instead of 6.9.)
struct FillArgs {
    uint8_t* grad;
    int64_t bytes;
    int64_t first_block;     // of one word a thread
};

template <bool FIRST> __device__ __forceinline__ int sort_key(const SortArgs& a, int p) {
    return FIRST ? row_of(a.ids, a.id_type, p, a.first, a.rows) : a.keys_in[p];
}

// Calls f(p, key, position) for the places p of [lo, lo + count) that are `stride`
// apart from lo + me on, kSortUnroll of them loaded at a time; f also runs
// (with p >= n) on lanes whose place is past the end.  POS: the position that
// goes with the key is loaded too.
template <bool FIRST, bool POS, typename F>
__device__ __forceinline__ void for_keys(const SortArgs& a, int lo, int count, int me, int stride, F f) {
    for (int r = 0; r < count; r += stride * kSortUnroll) {
        int key[kSortUnroll], pos[kSortUnroll];
#pragma unroll
        for (int u = 0; u < kSortUnroll; ++u) {
            const int p = lo + r + u * stride + me;
            const bool live = r + u * stride < count && p < a.n;
            key[u] = live ? sort_key<FIRST>(a, p) : 0;
            pos[u] = POS && !FIRST && live ? a.pos_in[p] : p;
        }
#pragma unroll
        for (int u = 0; u < kSortUnroll; ++u)
            if (r + u * stride < count) f(lo + r + u * stride + me, key[u], pos[u]);
    }
}

template <bool FIRST, int T> __global__ __launch_bounds__(T) void k_sort_count(SortArgs a, FillArgs f) {
    extern __shared__ int cnt[];
    if (int(blockIdx.x) >= a.n_tiles)
        return fill_zeros(f.grad, f.bytes, (f.first_block + blockIdx.x - a.n_tiles) * T + threadIdx.x);
    const int bins = 1 << a.bits;
    for (int d = threadIdx.x; d < bins; d += T) cnt[d] = 0;
    if (FIRST && blockIdx.x == 0 && threadIdx.x == 0) *a.n_runs = 0;
    __syncthreads();
    for_keys<FIRST, false>(a, int(blockIdx.x) * a.tile, a.tile, threadIdx.x, T, [&](int p, int key, int) {
        if (p < a.n) atomicAdd(&cnt[key >> a.shift & (bins - 1)], 1);
    });
    __syncthreads();
    for (int d = threadIdx.x; d < bins; d += T) a.hist[int64_t(blockIdx.x) * bins + d] = cnt[d];
}

// Exclusive sum of v over a block of WAVES waves; `sum` receives the total.
template <int WAVES> __device__ __forceinline__ int block_scan(int v, int* red, int& sum) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int x = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int y = __shfl_up(x, off, 64);
        if (lane >= off) x += y;
    }
    if (lane == 63) red[wave] = x;
    __syncthreads();
    int before = 0;
    sum = 0;
    for (int w = 0; w < WAVES; ++w) {
        if (w < wave) before += red[w];
        sum += red[w];
    }
    __syncthreads();
    return before + x - v;
}

// A wave's next 64 keys get their places: place[digit] is where the wave's next
// key of that digit goes, moved on by as many as there are here.  Equal
// digits keep their lanes' order.  Returns the lane's place (live lanes).
__device__ __forceinline__ int take_places(int* place, int digit, int bits, bool live) {
    // the live lanes whose digit agrees in every bit, in two halves: with t all
    // ones where the lane's bit is set, a lane agrees where m and t do
    const uint64_t all = __builtin_amdgcn_ballot_w64(live);
    uint32_t lo = uint32_t(all), hi = uint32_t(all >> 32);
    for (int b0 = 0; b0 < bits; b0 += 3)
#pragma unroll
        for (int b = 0; b < 3; ++b) {  // bits behind the digit's last are zero in every lane
            const bool set = digit & (1 << (b0 + b));
            const uint64_t m = __builtin_amdgcn_ballot_w64(set);
            const uint32_t t = set ? ~0u : 0u;
            lo &= ~(uint32_t(m) ^ t);
            hi &= ~(uint32_t(m >> 32) ^ t);
        }
    int at = 0;
    if (live) {
        const int rank = int(__builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0)));  // of them, in lower lanes
        // (relaxed atomics: LDS accesses that stay where they are; a volatile pointer would make them flat ones)
        at = __hip_atomic_load(place + digit, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT) + rank;
        __builtin_amdgcn_wave_barrier();  // every lane has read its place before the first of them moves it on
        if (rank == 0)
            __hip_atomic_store(place + digit, at + __popc(lo) + __popc(hi), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
    }
    __builtin_amdgcn_wave_barrier();
    return at;
}

// One tile of a pass.  Wave w of the block has a contiguous part of the tile;
// a key's place is the number of smaller digits, then of equal digits in
// earlier tiles, earlier waves, earlier rounds and lower lanes: stable.
template <bool FIRST, int T> __global__ __launch_bounds__(T) void k_sort_scatter(SortArgs a, FillArgs f) {
    constexpr int kWaves = T / 64;
    extern __shared__ int cnt[];
    __shared__ int red[kWaves];
    const int tile = int(blockIdx.x);
    if (tile >= a.n_tiles)
        return fill_zeros(f.grad, f.bytes, (f.first_block + tile - a.n_tiles) * T + threadIdx.x);
    const int bins = 1 << a.bits, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // the digits of all tiles for this thread's first bin, on their way while the tile's own are counted
    constexpr int kAhead = 32;
    int ahead[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        ahead[u] = u < a.n_tiles && int(threadIdx.x) < bins ? a.hist[int64_t(u) * bins + threadIdx.x] : 0;
    for (int d = threadIdx.x; d < kWaves * bins; d += T) cnt[d] = 0;
    __syncthreads();
    const int part = a.tile / kWaves, lo = tile * a.tile + wave * part;
    int* mine = cnt + wave * bins;
    for_keys<FIRST, false>(a, lo, part, lane, 64, [&](int p, int key, int) {
        if (p < a.n) atomicAdd(&mine[key >> a.shift & (bins - 1)], 1);
    });
    __syncthreads();
    int carry = 0;
    for (int d0 = 0; d0 < bins; d0 += T) {
        const int d = d0 + int(threadIdx.x);
        int before = 0, total = 0;
        auto add = [&](int t, int h) {
            total += h;
            before += t < tile ? h : 0;
        };
        if (d0 == 0)
#pragma unroll
            for (int u = 0; u < kAhead; ++u) add(u, ahead[u]);
        if (d < bins) {
            constexpr int kUnroll = 16;
            for (int t0 = d0 == 0 ? kAhead : 0; t0 < a.n_tiles; t0 += kUnroll) {
                int h[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) h[u] = t0 + u < a.n_tiles ? a.hist[int64_t(t0 + u) * bins + d] : 0;
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) add(t0 + u, h[u]);
            }
        }
        int sum;
        int at = carry + block_scan<kWaves>(total, red, sum) + before;
        carry += sum;
        if (d < bins) {
            int c[kWaves];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) c[w] = cnt[w * bins + d];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                cnt[w * bins + d] = at;
                at += c[w];
            }
        }
    }
    __syncthreads();
    for_keys<FIRST, true>(a, lo, part, lane, 64, [&](int p, int key, int pos) {
        const int at = take_places(mine, key >> a.shift & (bins - 1), a.bits, p < a.n);
        if (p < a.n) {
            a.keys_out[at] = key;
            a.pos_out[at] = pos;
        }
    });
}

// Up to kBlockIds ids into a table of fewer than 2^18 rows: both passes in one
// block, between them in LDS.  Of a whole gradient of 4096 ids of 768 columns
// this saves 11 of 43 us, of 8000 into 10000 x 256 3 of 40; at 16384 the block
// sorts for 42 us where the four launches take 24.  The zeros of a written
// gradient run before this sort, beside the other: in a large table that costs
// what the block saves (8192 ids into 128256 x 4096 take 208 us, 8193 190).
constexpr int kBlockThreads = 1024, kBlockWaves = kBlockThreads / 64, kBlockRounds = 8;
constexpr int kBlockIds = kBlockThreads * kBlockRounds, kBlockBits = 9;

__global__ __launch_bounds__(kBlockThreads) void k_sort_block(SortArgs a, int bits0, int bits1) {
    __shared__ int cnt[kBlockWaves << kBlockBits];
    __shared__ int skey[kBlockIds];
    __shared__ uint16_t spos[kBlockIds];
    __shared__ int red[kBlockWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int rounds = (a.n + kBlockThreads - 1) / kBlockThreads, lo = wave * rounds * 64 + lane;
    if (threadIdx.x == 0) *a.n_runs = 0;
    int key[kBlockRounds], pos[kBlockRounds];
#pragma unroll
    for (int r = 0; r < kBlockRounds; ++r) {
        pos[r] = lo + r * 64;
        key[r] = r < rounds && pos[r] < a.n ? row_of(a.ids, a.id_type, pos[r], a.first, a.rows) : 0;
    }
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        const int shift = pass ? bits0 : 0, bits = pass ? bits1 : bits0, bins = 1 << bits;
        for (int d = threadIdx.x; d < kBlockWaves * bins; d += kBlockThreads) cnt[d] = 0;
        __syncthreads();
        int* mine = cnt + wave * bins;
#pragma unroll
        for (int r = 0; r < kBlockRounds; ++r)
            if (r < rounds && lo + r * 64 < a.n) atomicAdd(&mine[key[r] >> shift & (bins - 1)], 1);
        __syncthreads();
        const int d = int(threadIdx.x);
        int total = 0, sum;
        int c[kBlockWaves];
#pragma unroll
        for (int w = 0; w < kBlockWaves; ++w) {
            c[w] = d < bins ? cnt[w * bins + d] : 0;
            total += c[w];
        }
        int at = block_scan<kBlockWaves>(total, red, sum);
        if (d < bins)
#pragma unroll
            for (int w = 0; w < kBlockWaves; ++w) {
                cnt[w * bins + d] = at;
                at += c[w];
            }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kBlockRounds; ++r) {
            if (r < rounds) {
                const bool live = lo + r * 64 < a.n;
                const int to = take_places(mine, key[r] >> shift & (bins - 1), bits, live);
                if (live && pass == 0) {
                    skey[to] = key[r];
                    spos[to] = uint16_t(pos[r]);
                } else if (live) {
                    a.keys_out[to] = key[r];
                    a.pos_out[to] = pos[r];
                }
            }
        }
        if (pass == 0) {
            __syncthreads();
#pragma unroll
            for (int r = 0; r < kBlockRounds; ++r) {
                const int p = lo + r * 64;
                if (r < rounds && p < a.n) {
                    key[r] = skey[p];
                    pos[r] = spos[p];
                }
            }
        }
    }
}

// Sums over the sorted order.  Work is cut into chunks of `chunk` sorted
// positions, so a batch of one id over and over is spread like any other.  A
// run of equal rows that crosses chunk borders belongs whole to the chunk it
// starts in if it has at most kRunMax positions; a longer one is summed in a
// piece for each chunk (slot 1 of the chunk it starts in, slot 0 of the
// others), and k_embed_join adds the pieces in order.  kRunMax: without it
// every border costs two rows of fp32 pieces, written and read.
constexpr int kSumThreads = 256, kRunMax = 16;

struct SumArgs {
    GradArgs g;
    const int *keys, *pos;
    float* parts;            // [n_chunks][2][width]
    int* n_runs;
    int2* runs;              // of each long run the chunk it starts in, and its row; in no order
    int width;               // columns rounded up to kPer
    int chunk, n_chunks;
};

// First index in the sorted K[lo..hi) with K[index] >= key, or hi.
__device__ __forceinline__ int lower_bound(const int* K, int lo, int hi, int key) {
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (K[mid] < key) lo = mid + 1; else hi = mid;
    }
    return lo;
}

template <int OD, int GD, bool ACC> __global__ __launch_bounds__(kSumThreads) void k_embed_sum(SumArgs s) {
    extern __shared__ int lds[];
    const GradArgs& a = s.g;
    const int C = s.chunk, G = 1 << a.group_shift, win = C + 2 * kRunMax;
    const int lane = int(threadIdx.x) & (G - 1), grp = threadIdx.x >> a.group_shift;
    const uint32_t item = blockIdx.x * uint32_t(kSumThreads >> a.group_shift) + grp;
    const int chunk = int(item / uint32_t(a.slabs)), slab = int(item % uint32_t(a.slabs));
    // the group's chunk of keys with kRunMax more on both sides, and its positions with kRunMax more
    int* K = lds + grp * (win + C + kRunMax);
    int* P = K + win;
    const int base = chunk * C;
    if (chunk < s.n_chunks) {
        for (int j = lane; j < win; j += G) {
            const int p = base - kRunMax + j;
            K[j] = p < 0 ? -1 : p < a.n ? s.keys[p] : INT32_MAX;
        }
        for (int j = lane; j < C + kRunMax; j += G) P[j] = base + j < a.n ? s.pos[base + j] : 0;
    }
    __syncthreads();
    const int c = ((slab << a.group_shift) + lane) * kPer;
    const int width = a.cols - c < kPer ? a.cols - c : kPer;
    if (chunk >= s.n_chunks || width <= 0) return;
    int q0 = 0, q1 = a.n - base < C ? a.n - base : C;
    const int kf = K[kRunMax], kt = K[kRunMax + q1 - 1];
    if (kf >= a.rows) return;
    bool head = false, tail = false;  // a piece of a long run at the chunk's start, at its end
    if (K[kRunMax - 1] == kf) {
        const int start = lower_bound(K, 0, kRunMax, kf);
        head = start == 0 || K[start + kRunMax] == kf;
        if (!head) q0 = lower_bound(K, kRunMax, win, kf + 1) - kRunMax;
    }
    if (kt >= a.rows) {
        q1 = lower_bound(K, kRunMax, kRunMax + q1, a.rows) - kRunMax;
    } else if (K[kRunMax + q1] == kt) {
        const int start = lower_bound(K, 0, kRunMax + q1, kt);
        tail = start == 0 || K[start + kRunMax] == kt;
        // a short run that started before the chunk has moved q0 past the chunk's end already
        if (!tail && q0 < q1) q1 = lower_bound(K, kRunMax + q1, win, kt + 1) - kRunMax;
    }
    // of ACC, what a finished row's sum is added to is on its way with the batch that finishes it; eight of both in
    // flight take the same time as four (65536 ids of 768 fp32 columns 74.4 us both, 4096 29.6 and 30.6)
    constexpr int kUnroll = ACC ? 4 : 8;
    float acc[kPer] = {};
    for (int q = q0; q < q1; q += kUnroll) {
        Raw<OD, kPer> x[kUnroll];
        Raw<GD, kPer> old[ACC ? kUnroll : 1];
        int key[kUnroll + 1];
        key[0] = K[kRunMax + q];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            key[u + 1] = q + u + 1 < q1 ? K[kRunMax + q + u + 1] : -1;
            if (q + u < q1) {
                x[u].template load<true>(a.dout + (int64_t(P[q + u]) * a.dout_stride + c) * Raw<OD, kPer>::kSize, width,
                                            a.cols >= kPer);
                if constexpr (ACC)
                    if (key[u + 1] != key[u])
                        old[u].template load<false>(a.grad + (int64_t(key[u]) * a.cols + c) * Raw<GD, kPer>::kSize, width,
                                                    a.cols >= kPer);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (q + u < q1) {
                x[u].settle(width, a.cols >= kPer);
#pragma unroll
                for (int k = 0; k < kPer; ++k) acc[k] += x[u].get(k);
            }
            if (q + u < q1 && key[u + 1] != key[u]) {
                if ((head && key[u] == kf) || (tail && key[u] == kt)) {
                    const int slot = head && key[u] == kf ? 0 : 1;
                    float* o = s.parts + (int64_t(chunk) * 2 + slot) * s.width + c;
                    if (slot == 1 && c == 0) s.runs[atomicAdd(s.n_runs, 1)] = make_int2(chunk, key[u]);
                    reinterpret_cast<f32x4_t*>(o)[0] = f32x4_t{acc[0], acc[1], acc[2], acc[3]};
                    reinterpret_cast<f32x4_t*>(o)[1] = f32x4_t{acc[4], acc[5], acc[6], acc[7]};
                } else {
                    float v[kPer];
                    if constexpr (ACC) old[u].settle(width, a.cols >= kPer);
#pragma unroll
                    for (int k = 0; k < kPer; ++k)
                        v[k] = ACC ? __builtin_fmaf(a.scale, acc[k], old[ACC ? u : 0].get(k)) : a.scale * acc[k];
                    store<GD, kPer, true>(a.grad + (int64_t(key[u]) * a.cols + c) * Raw<GD, kPer>::kSize, width, v);
                }
#pragma unroll
                for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
            }
        }
    }
}

// The long runs, one at a time to a block: its pieces are added in order (each
// group a stretch of them, then the groups).  The list's order differs from
// run to run, the sums do not.
constexpr int kJoinThreads = 256, kJoinBlocks = 1024;

template <int GD, bool ACC> __global__ __launch_bounds__(kJoinThreads) void k_embed_join(SumArgs s) {
    __shared__ float red[kJoinThreads * kPer];
    __shared__ int more;
    const GradArgs& a = s.g;
    const int t = int(threadIdx.x), slab = int(blockIdx.y);
    const int groups = kJoinThreads >> a.group_shift, g = t >> a.group_shift;
    const int c = ((slab << a.group_shift) + (t & ((1 << a.group_shift) - 1))) * kPer;
    const int width = a.cols - c < kPer ? a.cols - c : kPer;
    const int n_runs = *s.n_runs;
    for (int r = blockIdx.x; r < n_runs; r += int(gridDim.x)) {
        const int chunk = s.runs[r].x, key = s.runs[r].y;
        __syncthreads();
        if (t == 0) more = 0;
        __syncthreads();
        // how many chunks behind this one the run reaches
        int reach = 0;
        for (int j = chunk + 1 + t; j < s.n_chunks && s.keys[int64_t(j) * s.chunk] == key; j += kJoinThreads) ++reach;
        if (reach) atomicAdd(&more, reach);
        __syncthreads();
        const int pieces = 1 + more;
        const int share = (pieces + groups - 1) / groups, lo = g * share, hi = lo + share < pieces ? lo + share : pieces;
        float acc[kPer] = {};
        if (width > 0) {
            constexpr int kUnroll = 8;
            for (int j = lo; j < hi; j += kUnroll) {
                f32x4_t x[kUnroll], y[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const float* o = s.parts + (int64_t(chunk + j + u) * 2 + (j + u == 0 ? 1 : 0)) * s.width + c;
                    x[u] = y[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                    if (j + u < hi) {
                        x[u] = reinterpret_cast<const f32x4_t*>(o)[0];
                        y[u] = reinterpret_cast<const f32x4_t*>(o)[1];
                    }
                }
#pragma unroll
                for (int u = 0; u < kUnroll; ++u)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        acc[k] += x[u][k];
                        acc[4 + k] += y[u][k];
                    }
            }
        }
        add_groups<kJoinThreads>(red, a.group_shift, acc);
        if (g == 0 && width > 0) write_row<GD, ACC>(a, key, c, width, acc);
    }
}

// ---- host side ----

// Lanes of a group, 8 to `most` (as a shift): the most lanes that leave at
// most an eighth more of them idle than the best choice does.
int pick_group(int words, int most_shift) {
    auto padded = [&](int s) { return ((words + (1 << s) - 1) >> s) << s; };
    int best = 1 << 30;
    for (int s = 3; s <= most_shift; ++s) best = std::min(best, padded(s));
    for (int s = most_shift; s > 3; --s)
        if (padded(s) <= best + best / 8) return s;
    return 3;
}

// How a gradient of n ids is cut, and where its workspace regions lie.
struct GradShape {
    // which way positions are grouped by row: searched for by each position's or by each row's block, sorted by one
    // block, else sorted by several launches
    bool few, by_row, block;
    int group_shift, slabs, width;
    int span;                // by_row: groups of columns of a block
    int bits[2], tile, n_tiles, chunk, n_chunks;
    uint64_t keys[2], pos[2], hist, runs, parts, total;
};

GradShape grad_shape(const mfsdp_entry& e, int64_t n) {
    GradShape s = {};
    const int words = int((e.cols + kPer - 1) / kPer);
    s.group_shift = pick_group(std::max(words, 1), 6);
    s.slabs = std::max(1, (words + (1 << s.group_shift) - 1) >> s.group_shift);
    s.width = words * kPer;
    s.few = e.rows == 0 || e.cols == 0;
    if (s.few) return s;
    // a row's columns in as many blocks as keep the search small
    s.span = 1;
    s.by_row = n <= kRowsIds && n * e.rows <= kRowsWork;
    while (s.by_row && s.span < s.slabs && n * e.rows * ((s.slabs + s.span - 1) / s.span) > 2 * kRowsWork) ++s.span;
    s.by_row = s.by_row && n * s.span <= (s.group_shift <= kRowsNarrow ? kRowsIds : kRowsHot);
    // wide rows sooner go to the sort, where a hot row is spread over more blocks
    s.few = n <= (s.slabs > kFewSlabs ? kFewIds / 2 : kFewIds) && !(s.by_row && 2 * e.rows <= n);
    s.by_row = s.by_row && !s.few;
    if (s.few || s.by_row) return s;
    int bits = 2;  // of the largest key, `rows`
    while ((int64_t(1) << bits) <= e.rows) ++bits;
    s.block = n <= kBlockIds && bits <= 2 * kBlockBits;
    // one pass where LDS holds its counts and the fill beside it still has room, else two
    s.bits[0] = !s.block && bits <= kOnePassBits ? bits : (bits + 1) / 2;
    s.bits[1] = bits - s.bits[0];
    // at least 2048 positions a tile, at most 128 tiles (each adds up the
    // digits of all others)
    s.tile = int(std::max<int64_t>(2048, (n + 128 * 512 - 1) / (128 * 512) * 512));
    s.n_tiles = int((n + s.tile - 1) / s.tile);
    // The longest chunk that still makes 2048 waves (8 a CU; 65536 ids of 768
    // columns take 73.6 us so, 75.7 with 4096 or 8192 waves, 94 with 1024).
    auto parts = [&](int64_t len) { return (n + len - 1) / len; };
    const int longest = s.group_shift < 5 ? 64 : 256;
    const int64_t most = std::max<int64_t>(1, (int64_t(2 * 2048) * 64 >> s.group_shift) / s.slabs);
    s.chunk = 16;
    while (s.chunk < longest && parts(s.chunk) > most) s.chunk *= 2;
    s.n_chunks = int(parts(s.chunk));
    // a workspace for n ids serves fewer of them too: regions are sized by what any smaller batch may need
    const uint64_t max_chunks = uint64_t(std::min(parts(16), std::max(most, parts(longest))));
    const uint64_t max_tiles = uint64_t(std::min<int64_t>(128, parts(2048)));
    uint64_t off = 0;
    auto region = [&](uint64_t bytes) {
        const uint64_t at = off;
        off = align_up(off + bytes, kAlign);
        return at;
    };
    for (int k = 0; k < 2; ++k) {
        s.keys[k] = region(uint64_t(n) * 4);
        s.pos[k] = region(uint64_t(n) * 4);
    }
    s.hist = region((max_tiles * 4) << std::max(s.bits[0], s.bits[1]));
    s.runs = region((max_chunks + 1) * 8);  // their number, then the list
    s.parts = region(max_chunks * 2 * uint64_t(s.width) * 4);
    s.total = off;
    return s;
}

mfsdp_status hip_fail(hipError_t e, const char* what) {
    return fail(MFSDP_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

constexpr int64_t kMaxIds = int64_t(1) << 30, kMaxFirst = int64_t(1) << 62, kMaxStride = int64_t(1) << 40;

// Checks that the lookup and the gradient share.  `stride`: elements from one
// row of the activations to the next (0 stands for cols), set on success.
mfsdp_status check(mfsdp_plan_t plan, int64_t entry, const void* buffer, const void* ids, int64_t n_ids,
                   int32_t id_type, int32_t act_type, int64_t first_id, const void* act, int64_t* stride) {
    if (entry < 0 || entry >= int64_t(plan->entries.size()))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "entry index out of range");
    if (id_type != MFSDP_I32 && id_type != MFSDP_I64)
        return fail(MFSDP_ERR_UNSUPPORTED, "id_type must be MFSDP_I32 or MFSDP_I64");
    if (act_type != MFSDP_F32 && act_type != MFSDP_BF16)
        return fail(MFSDP_ERR_UNSUPPORTED, "activations must be MFSDP_F32 or MFSDP_BF16");
    if (n_ids < 0 || n_ids > kMaxIds) return fail(MFSDP_ERR_INVALID_ARGUMENT, "n_ids must be in 0..2^30");
    if (first_id < 0 || first_id > kMaxFirst) return fail(MFSDP_ERR_INVALID_ARGUMENT, "first_id must be in 0..2^62");
    const int64_t cols = plan->entries[size_t(entry)].cols;
    if (*stride == 0) *stride = cols;
    if (*stride < cols || *stride > kMaxStride) return fail(MFSDP_ERR_INVALID_ARGUMENT, "row stride below cols or above 2^40");
    if (!buffer || misaligned(buffer, 16)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "owner buffer is NULL or not 16-byte aligned");
    if (n_ids > 0) {
        if (!ids || misaligned(ids, id_type == MFSDP_I64 ? 8 : 4))
            return fail(MFSDP_ERR_INVALID_ARGUMENT, "ids is NULL or misaligned");
        if (!act || misaligned(act, act_type == MFSDP_BF16 ? 2 : 4))
            return fail(MFSDP_ERR_INVALID_ARGUMENT, "activations are NULL or misaligned");
    }
    return MFSDP_OK;
}

}  // namespace
}  // namespace mfsdp

using namespace mfsdp;

namespace mfsdp {
namespace {

template <int TD, int OD> hipError_t launch_lookup(LookupArgs a, hipStream_t stream) {
    constexpr int N = TD == kF32 && OD == kF32 ? 4 : 8;
    const int words = (a.cols + N - 1) / N;
    a.group_shift = pick_group(words, 9);
    const uint32_t slabs = uint32_t((words + (1 << a.group_shift) - 1) >> a.group_shift);
    const int64_t rows = kLookupThreads >> a.group_shift, blocks = (a.n + rows - 1) / rows;
    for (int64_t first = 0; first < blocks; first += kBlocksMax)
        k_embed_lookup<TD, OD>
            <<<dim3(uint32_t(std::min(blocks - first, kBlocksMax)), slabs), dim3(kLookupThreads), 0, stream>>>(a, first);
    return hipGetLastError();
}

hipError_t zero_table(uint8_t* grad, int64_t bytes, hipStream_t stream) {
    const int64_t blocks = (bytes + kZeroThreads * 16 - 1) / (kZeroThreads * 16);
    for (int64_t first = 0; first < blocks; first += kBlocksMax)
        k_embed_zero<<<dim3(uint32_t(std::min(blocks - first, kBlocksMax))), dim3(kZeroThreads), 0, stream>>>(grad, bytes, first);
    return hipGetLastError();
}

template <int OD, int GD, bool ACC> hipError_t launch_few(const GradArgs& a, hipStream_t stream) {
    if constexpr (!ACC) {
        constexpr int kSize = Raw<GD, kPer>::kSize, kElems = 16 / kSize * kSpanWords;
        const int64_t bytes = int64_t(a.rows) * a.cols * kSize;
        if (a.n <= kSpanIds && bytes <= kFewBytes && a.cols >= 16 / kSize) {
            SpanArgs s;
            s.span = std::clamp(kElems / a.cols, 1, kSpanRows);
            s.pieces = s.span > 1 ? 1 : (a.cols + kElems - 1) / kElems;
            s.few_blocks = a.n * few_parts(a.slabs);
            const int blocks = s.few_blocks + (a.rows + s.span - 1) / s.span * s.pieces;
            k_embed_few_fill<OD, GD><<<dim3(uint32_t(blocks)), dim3(kSpanThreads), 0, stream>>>(a, s);
            return hipGetLastError();
        }
        if (hipError_t e = zero_table(a.grad, bytes, stream); e != hipSuccess) return e;
    }
    if (a.n > 0) k_embed_few<OD, GD, ACC><<<dim3(uint32_t(a.n), uint32_t(few_parts(a.slabs))), dim3(kFewThreads), 0, stream>>>(a);
    return hipGetLastError();
}

// The sort, two launches a pass, each with an equal part of the zeros.
template <int T>
hipError_t launch_sort(SortArgs t, const GradShape& s, uint8_t* ws, uint8_t* grad, int64_t bytes, hipStream_t stream) {
    auto ints = [&](uint64_t off) { return reinterpret_cast<int*>(ws + off); };
    FillArgs f = {grad, bytes, 0};
    int64_t fill = (bytes + T * 16 - 1) / (T * 16);
    if (fill > kBlocksMax) {  // 34 GB (256 threads): more than a launch holds
        if (hipError_t e = zero_table(grad, bytes, stream); e != hipSuccess) return e;
        fill = 0;
    }
    const int passes = s.bits[1] > 0 ? 2 : 1;
    const int64_t part = (fill + 2 * passes - 1) / (2 * passes);
    auto grid = [&] { return dim3(uint32_t(s.n_tiles + std::max<int64_t>(0, std::min(part, fill - f.first_block)))); };
    for (int pass = 0; pass < passes; ++pass) {
        t.shift = pass ? s.bits[0] : 0;
        t.bits = s.bits[pass];
        t.keys_in = ints(s.keys[0]);
        t.pos_in = ints(s.pos[0]);
        t.keys_out = ints(s.keys[pass + 2 - passes]);
        t.pos_out = ints(s.pos[pass + 2 - passes]);
        const size_t row = size_t(4) << t.bits;
        if (pass == 0)
            k_sort_count<true, T><<<grid(), dim3(T), row, stream>>>(t, f);
        else
            k_sort_count<false, T><<<grid(), dim3(T), row, stream>>>(t, f);
        f.first_block += part;
        if (pass == 0)
            k_sort_scatter<true, T><<<grid(), dim3(T), row * (T / 64), stream>>>(t, f);
        else
            k_sort_scatter<false, T><<<grid(), dim3(T), row * (T / 64), stream>>>(t, f);
        f.first_block += part;
    }
    return hipGetLastError();
}

template <int OD, int GD, bool ACC>
hipError_t launch_sorted(const GradArgs& a, const GradShape& s, uint8_t* ws, hipStream_t stream) {
    auto ints = [&](uint64_t off) { return reinterpret_cast<int*>(ws + off); };
    SortArgs t = {};
    t.ids = a.ids;
    t.first = a.first;
    t.rows = a.rows;
    t.n = a.n;
    t.id_type = a.id_type;
    t.tile = s.tile;
    t.n_tiles = s.n_tiles;
    t.hist = ints(s.hist);
    t.n_runs = ints(s.runs);
    const int64_t bytes = ACC ? 0 : int64_t(a.rows) * a.cols * Raw<GD, kPer>::kSize;
    if (s.block) {
        if (bytes > 0)
            if (hipError_t e = zero_table(a.grad, bytes, stream); e != hipSuccess) return e;
        t.keys_out = ints(s.keys[1]);
        t.pos_out = ints(s.pos[1]);
        k_sort_block<<<dim3(1), dim3(kBlockThreads), 0, stream>>>(t, s.bits[0], s.bits[1]);
    } else {
        // 256 threads clear faster (6.7 TB/s in four parts, 6.2 with 512), 512 sort faster
        if (hipError_t e = ACC ? launch_sort<512>(t, s, ws, a.grad, bytes, stream) : launch_sort<256>(t, s, ws, a.grad, bytes, stream);
            e != hipSuccess)
            return e;
    }
    SumArgs u = {};
    u.g = a;
    u.keys = ints(s.keys[1]);
    u.pos = ints(s.pos[1]);
    u.parts = reinterpret_cast<float*>(ws + s.parts);
    u.width = s.width;
    u.n_runs = ints(s.runs);
    u.runs = reinterpret_cast<int2*>(u.n_runs) + 1;
    u.chunk = s.chunk;
    u.n_chunks = s.n_chunks;
    const int groups = kSumThreads >> a.group_shift;
    const int64_t items = int64_t(s.n_chunks) * a.slabs;
    const size_t lds = size_t(groups) * size_t(2 * s.chunk + 3 * kRunMax) * 4;
    k_embed_sum<OD, GD, ACC><<<dim3(uint32_t((items + groups - 1) / groups)), dim3(kSumThreads), lds, stream>>>(u);
    // a long run has more than kRunMax positions
    const int runs = int(std::min<int64_t>(kJoinBlocks, (a.n + kRunMax) / (kRunMax + 1)));
    k_embed_join<GD, ACC><<<dim3(uint32_t(runs), uint32_t(a.slabs)), dim3(kJoinThreads), 0, stream>>>(u);
    return hipGetLastError();
}

template <int OD, int GD, bool ACC>
hipError_t launch_grad(const GradArgs& a, const GradShape& s, uint8_t* ws, hipStream_t stream) {
    if (s.by_row) {
        const uint32_t parts = uint32_t((a.slabs + s.span - 1) / s.span);
        const size_t lds = size_t(rows_part(a.n)) * kRowsWaves * sizeof(uint16_t);
        k_embed_rows<OD, GD, ACC><<<dim3(uint32_t(a.rows), parts), dim3(kRowsThreads), lds, stream>>>(a, s.span);
        return hipGetLastError();
    }
    return s.few ? launch_few<OD, GD, ACC>(a, stream) : launch_sorted<OD, GD, ACC>(a, s, ws, stream);
}

}  // namespace
}  // namespace mfsdp

extern "C" mfsdp_status mfsdp_embed_lookup(mfsdp_plan_t plan, int64_t entry, const mfsdp_embed_lookup_args* args) {
    clear_error();
    if (!plan || !args) return fail(MFSDP_ERR_INVALID_ARGUMENT, "NULL plan or args");
    int64_t stride = args->out_stride;
    if (mfsdp_status st = check(plan, entry, args->params, args->ids, args->n_ids, args->id_type, args->out_type,
                                args->first_id, args->out, &stride);
        st != MFSDP_OK)
        return st;
    const mfsdp_entry& e = plan->entries[size_t(entry)];
    if (args->n_ids == 0 || e.cols == 0) return MFSDP_OK;
    LookupArgs a = {};
    a.table = static_cast<const uint8_t*>(args->params) + e.offset;
    a.ids = args->ids;
    a.out = static_cast<uint8_t*>(args->out);
    a.n = args->n_ids;
    a.first = args->first_id;
    a.out_stride = stride;
    a.rows = int(e.rows);
    a.cols = int(e.cols);
    a.id_type = args->id_type;
    a.scale = args->scale;
    hipStream_t stream = static_cast<hipStream_t>(args->stream);
    const bool tb = e.dtype == kBF16, ob = args->out_type == kBF16;
    const hipError_t err = tb ? (ob ? launch_lookup<kBF16, kBF16>(a, stream) : launch_lookup<kBF16, kF32>(a, stream))
                              : (ob ? launch_lookup<kF32, kBF16>(a, stream) : launch_lookup<kF32, kF32>(a, stream));
    if (err != hipSuccess) return hip_fail(err, "lookup launch");
    return MFSDP_OK;
}

extern "C" mfsdp_status mfsdp_plan_embed_workspace_bytes(mfsdp_plan_t plan, int64_t entry, int64_t n_ids,
                                                         uint64_t* bytes) {
    clear_error();
    if (!plan || !bytes) return fail(MFSDP_ERR_INVALID_ARGUMENT, "NULL argument");
    if (entry < 0 || entry >= int64_t(plan->entries.size()))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "entry index out of range");
    if (n_ids < 0 || n_ids > kMaxIds) return fail(MFSDP_ERR_INVALID_ARGUMENT, "n_ids must be in 0..2^30");
    *bytes = grad_shape(plan->entries[size_t(entry)], n_ids).total;
    return MFSDP_OK;
}

extern "C" mfsdp_status mfsdp_embed_grad(mfsdp_plan_t plan, int64_t entry, const mfsdp_embed_grad_args* args) {
    clear_error();
    if (!plan || !args) return fail(MFSDP_ERR_INVALID_ARGUMENT, "NULL plan or args");
    int64_t stride = args->dout_stride;
    if (mfsdp_status st = check(plan, entry, args->grads, args->ids, args->n_ids, args->id_type, args->dout_type,
                                args->first_id, args->dout, &stride);
        st != MFSDP_OK)
        return st;
    if (args->accumulate != 0 && args->accumulate != 1)
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "accumulate must be 0 or 1");
    const mfsdp_entry& e = plan->entries[size_t(entry)];
    if (e.rows == 0 || e.cols == 0 || (args->n_ids == 0 && args->accumulate)) return MFSDP_OK;
    const GradShape s = grad_shape(e, args->n_ids);
    if (s.total > 0) {
        if (!args->workspace || misaligned(args->workspace, kAlign))
            return fail(MFSDP_ERR_INVALID_ARGUMENT, "workspace is NULL or not 256-byte aligned");
        if (args->workspace_bytes < s.total)
            return fail(MFSDP_ERR_WORKSPACE_TOO_SMALL, "workspace has " + std::to_string(args->workspace_bytes) +
                                                           " bytes, " + std::to_string(args->n_ids) + " ids need " +
                                                           std::to_string(s.total));
    }
    GradArgs a = {};
    a.grad = static_cast<uint8_t*>(args->grads) + e.offset;
    a.ids = args->ids;
    a.dout = static_cast<const uint8_t*>(args->dout);
    a.first = args->first_id;
    a.dout_stride = stride;
    a.rows = int(e.rows);
    a.cols = int(e.cols);
    a.n = int(args->n_ids);
    a.id_type = args->id_type;
    a.group_shift = s.group_shift;
    a.slabs = s.slabs;
    a.scale = args->scale;
    uint8_t* ws = static_cast<uint8_t*>(args->workspace);
    hipStream_t stream = static_cast<hipStream_t>(args->stream);
    const int which = (args->dout_type == kBF16 ? 4 : 0) + (e.dtype == kBF16 ? 2 : 0) + args->accumulate;
    hipError_t err = hipSuccess;
    switch (which) {
        case 0: err = launch_grad<kF32, kF32, false>(a, s, ws, stream); break;
        case 1: err = launch_grad<kF32, kF32, true>(a, s, ws, stream); break;
        case 2: err = launch_grad<kF32, kBF16, false>(a, s, ws, stream); break;
        case 3: err = launch_grad<kF32, kBF16, true>(a, s, ws, stream); break;
        case 4: err = launch_grad<kBF16, kF32, false>(a, s, ws, stream); break;
        case 5: err = launch_grad<kBF16, kF32, true>(a, s, ws, stream); break;
        case 6: err = launch_grad<kBF16, kBF16, false>(a, s, ws, stream); break;
        case 7: err = launch_grad<kBF16, kBF16, true>(a, s, ws, stream); break;
    }
    if (err != hipSuccess) return hip_fail(err, "embedding gradient launch");
    return MFSDP_OK;
}
