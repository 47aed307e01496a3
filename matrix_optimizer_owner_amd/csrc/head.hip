// head.hip - the output head over a table of the owner buffer: log
// probabilities of given tokens under softmax(scale * x W^T), entropy, likely
// alternatives, and the gradients of x and W.
//
// Logits are formed in fp32 by MFMA, from bf16 operands or the bf16 planes of
// fp32 ones (tile_loop.h), and used in base 2, y = log2(e) scale x.W, which is
// what the exponential instruction takes.  They are never stored
// whole for the sums: the block that forms a tile of them reduces it, per
// token and part of the vocabulary, to
//
//   M = max y,  S = sum 2^(y-M),  W = sum 2^(y-M) (y-M),
//
// and parts join by M = max(Ma, Mb), S = Sa 2^(Ma-M) + Sb 2^(Mb-M),
// W = 2^(Ma-M) (Wa + (Ma-M) Sa) + the same of b.  Then
//   logp = ln2 (y_t - M - log2 S),  entropy = ln2 (log2 S - W/S).
// The k likeliest tokens of a row lie in the k parts with the largest M (ties
// to the lower part): where they are asked for, logits go to the workspace too
// and only those parts of them are read.
//
// Backward, with p = 2^(y-M)/S:
//   dz_j = scale (dlogp ([j = t] - p_j) - dH p_j (ln p_j + H)),
//   dx = dz W,  dW = dz^T x,
// dz from the logits formed again, stored once, then two more products.  With
// fp32 among the operands dz is three planes, else one, rounded to bf16.  Errors
// of half a step, independent from element to element, average out in sums of
// many alike, but not where a few entries carry a row, as its target does and
// a likely other token.  What rounding takes from the entries of a 32nd or more
// of a row's sum |dz_j| (kShare), of which there are at most 32, is kept in fp32
// and added where dx and dW are written (in bf16 for rows of the table that many
// tokens share); what is left of the rounding is at most 2^-8 |dz_j| each, in
// the 2-norm 2^-8 sqrt(1/32) of the row's sum.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "kernels.h"
#include "plan_internal.h"
#include "tile_loop.h"

// Products are rounded before they are added, but where __builtin_fmaf says
// otherwise (see reduce_column).
#pragma clang fp contract(off)

namespace mfsdp {
namespace {

constexpr float kLn2 = 0.693147180559945309f;
constexpr int kMaxTop = 64;             // a list of alternatives is one lane an entry
constexpr int kPackThreads = 256;
constexpr int kPadTokens = 256;         // rows of the packed batch: a multiple of both tile edges
constexpr int64_t kFewTokens = 64;      // batches up to this are read straight from x and the table
constexpr int64_t kCacheBytes = int64_t(256) << 20;  // the Infinity Cache
constexpr float kShare = 1.f / 32;      // of a row's sum of |dz|: entries from it on keep what rounding takes
constexpr int kMaxRests = 48;           // such entries of a row, and some more than there can be but for rounding

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// A logit of -inf, or one far below the largest, has probability 0 and no part
// in a sum: the exponent of its probability is kept where that is 0 already and
// its product with any sum is finite.  NaN stays NaN.
__device__ __forceinline__ float not_below(float y) { return __builtin_elementwise_maximum(y, -1024.f); }

// ---- token ids ----

struct Ids {
    const void* ids;   // NULL: every row counts and none has a target
    int64_t first;
    int type;          // mfsdp_id_type
};
struct Token {
    int target;        // row of the table, -1: not here
    bool live;         // not padding (a negative id)
};
__device__ __forceinline__ Token token_of(const Ids& a, int64_t i, int rows) {
    if (!a.ids) return Token{-1, true};
    const int64_t id = a.type == MFSDP_I64 ? static_cast<const int64_t*>(a.ids)[i] : static_cast<const int32_t*>(a.ids)[i];
    const int64_t t = id - a.first;
    return Token{id >= 0 && t >= 0 && t < rows ? int(t) : -1, id >= 0};
}

// ---- unaligned words ----

typedef unsigned int word_at_2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned int word_at_4_t __attribute__((ext_vector_type(4), aligned(4)));

// Elements k .. k + 16/sizeof(element) - 1 of a row of D at any address, as
// they lie; zeros past the last column.  Where a word crosses it, the word that
// ends with it is read and moved down.  INSIDE: no word crosses it; PAST: past
// the caches.
template <int D, bool INSIDE, bool PAST> __device__ __forceinline__ u32x4_t row_word(const uint8_t* row, int k, int cols) {
    constexpr int ES = D == kBF16 ? 2 : 4, N = 16 / ES;
    using Word = std::conditional_t<D == kBF16, word_at_2_t, word_at_4_t>;
    auto at = [&](int i) {
        const Word* p = reinterpret_cast<const Word*>(row + i * ES);
        return u32x4_t(PAST ? __builtin_nontemporal_load(p) : *p);
    };
    if (INSIDE || k + N <= cols) return at(k);
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (k >= cols) return v;
    if (cols >= N) {
        v = at(cols - N);
        const int bits = (k + N - cols) * ES * 8;  // 16 .. 112
        uint64_t lo = uint64_t(v[1]) << 32 | v[0], hi = uint64_t(v[3]) << 32 | v[2];
        lo = bits >= 64 ? hi >> (bits - 64) : lo >> bits | hi << (64 - bits);
        hi = bits >= 64 ? 0 : hi >> bits;
        return u32x4_t{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
    }
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (k + e < cols) {
            if constexpr (D == kF32)
                v[e] = reinterpret_cast<const uint32_t*>(row)[k + e];
            else
                v[e >> 1] |= uint32_t(reinterpret_cast<const uint16_t*>(row)[k + e]) << (16 * (e & 1));
        }
    return v;
}

// ---- packing ----

struct PackArgs {
    const uint8_t* src;
    uint8_t* dst;
    int64_t stride;     // elements of src from row to row
    int64_t rows;       // of src
    int64_t block;      // bytes of dst from column block to column block, whose rows are 128 bytes apart
    int64_t plane;      // bytes of dst from plane to plane
    int64_t words;      // 16-byte words of a plane of dst, over all its rows
    int per_row;        // of a row
    int cols;
    Ids ids;            // rows with a negative id become zeros
    int table_rows;
    int* zeros;         // these words become zeros
    int64_t n_zeros;
};

// An fp32 value as three bf16 ones that add up to it, each the nearest to what
// the ones before it leave (the first towards zero where the nearest is not
// finite).  A value that is not finite is the first alone.
struct Planes {
    uint16_t part[3];
};
__device__ __forceinline__ Planes planes_of(float v) {
    Planes p;
    p.part[0] = f32_to_bf16(v);
    const bool fine = fabsf(v) < INFINITY;
    if (fine && (p.part[0] & 0x7f80) == 0x7f80) p.part[0] = uint16_t(__float_as_uint(v) >> 16);
    const float r = fine ? v - bf16_to_f32(p.part[0]) : 0.f;
    p.part[1] = f32_to_bf16(r);
    p.part[2] = f32_to_bf16(r - bf16_to_f32(p.part[1]));
    return p;
}

// Rows of a matrix in the layout the tile loop takes, one plane of a bf16
// matrix or three of an fp32 one: zeros behind each row's end, for rows past
// the last and for padding tokens.  HBM: 50000 x 1000 bf16, 0.2 GB read and
// written, 30 us; 34950 x 702 fp32 40 us.
template <int D> __device__ __forceinline__ void pack_word(const PackArgs& a, int64_t block) {
    const int64_t w = block * kPackThreads + threadIdx.x;
    if (w >= a.words) return;
    const int64_t row = w / a.per_row;
    const int g = int(w % a.per_row), c = g * 8;
    const Token t = row < a.rows ? token_of(a.ids, row, a.table_rows) : Token{-1, false};
    for (int64_t i = w; i < a.n_zeros; i += a.words) a.zeros[i] = 0;
    const bool in = t.live && c < a.cols;
    const uint8_t* src = a.src + row * a.stride * (D == kBF16 ? 2 : 4);
    uint8_t* dst = a.dst + int64_t(g >> 3) * a.block + row * 128 + (g & 7) * 16;
    if constexpr (D == kBF16) {
        *reinterpret_cast<u32x4_t*>(dst) = in ? row_word<D, false, false>(src, c, a.cols) : u32x4_t{0u, 0u, 0u, 0u};
    } else {
        float v[8] = {};
        if (in) {
            const u32x4_t x = row_word<D, false, false>(src, c, a.cols), y = row_word<D, false, false>(src, c + 4, a.cols);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = __uint_as_float(x[k]);
                v[4 + k] = __uint_as_float(y[k]);
            }
        }
        u32x4_t o[3] = {};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const Planes p = planes_of(v[k]);
#pragma unroll
            for (int j = 0; j < 3; ++j) o[j][k >> 1] |= uint32_t(p.part[j]) << (16 * (k & 1));
        }
#pragma unroll
        for (int j = 0; j < 3; ++j) *reinterpret_cast<u32x4_t*>(dst + j * a.plane) = o[j];
    }
}
// One matrix, and another from block `second` on: the batch and the table in
// one launch.
template <int D, int D2>
__global__ __launch_bounds__(kPackThreads) void k_head_pack(PackArgs a, PackArgs b, uint32_t second) {
    if (blockIdx.x < second)
        pack_word<D>(a, blockIdx.x);
    else
        pack_word<D2>(b, blockIdx.x - second);
}

// The packed batch turned over, a plane's 64 x 64 elements a block: rows are
// its columns, contiguous along the tokens, so that dW reads this operand
// row-major, with one LDS read a fragment where K-major takes two (HBM: 4096 x
// 4096 bf16 in 15 us).
struct TurnArgs {
    const uint8_t* src;
    uint8_t* dst;
    int64_t src_block, dst_block, src_plane, dst_plane;
    uint32_t across, stages, blocks;  // 64-token and 64-column blocks, and all of them
};
__device__ __forceinline__ void turn_block(const TurnArgs& a, uint32_t block) {
    __shared__ uint16_t t[64][66];
    const uint32_t bx = block % a.across, by = block / a.across % a.stages, bz = block / a.across / a.stages;
    const uint8_t* src = a.src + bz * a.src_plane + by * a.src_block + int64_t(bx) * 8192;
    uint8_t* dst = a.dst + bz * a.dst_plane + bx * a.dst_block + int64_t(by) * 8192;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k = int(threadIdx.x) + i * 256, row = k >> 3, g = k & 7;
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(src + k * 16);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[g * 8 + e][row] = uint16_t(v[e >> 1] >> (16 * (e & 1)));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k = int(threadIdx.x) + i * 256, row = k >> 3, g = k & 7;
        u32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = uint32_t(t[row][g * 8 + 2 * e]) | uint32_t(t[row][g * 8 + 2 * e + 1]) << 16;
        *reinterpret_cast<u32x4_t*>(dst + k * 16) = v;
    }
}

// ---- tiles ----

// Tile (ti, tj) of a block: tiles run in strips 8 wide along the dimension
// with fewer of them, and blocks of one XCD (block index mod 8) take 32
// consecutive ones, 4 x 8 where the strip is 8 wide, whose operands share its
// L2.  What is left over a multiple of 256 blocks keeps the plain order.
__device__ __forceinline__ void tile_of(int b, int total, int tp, int tq, int& ti, int& tj) {
    int at = b;
    if (b < total / 256 * 256) at = (b / 256 * 8 + (b & 7)) * 32 + ((b & 255) >> 3);
    const int few = min(tp, tq), many = max(tp, tq);
    const int strip = at / (8 * many), in = at - strip * 8 * many;
    const int width = min(8, few - 8 * strip);
    const int across = 8 * strip + in % width, along = in / width;
    ti = tp <= tq ? across : along;
    tj = tp <= tq ? along : across;
}

struct LogitArgs {
    Operand table, x;
    int rows;            // of the table
    int64_t n;
    int stages;          // of the contraction
    int tp, tq;          // tiles along the vocabulary and the batch
    float c2;            // scale * log2(e)
    Ids ids;
    float4* parts;       // [part][n]: M, S, W of a token over BT/2 rows of the table
    float* targets;      // [n]: y of the target, written where it is here
    float* logits;       // NULL, or [part][n][rows of a part]: y
};

// f(MFMA row tile, accumulator, row) for the rows of a wave's block that a
// lane holds of one column.
template <int MM, typename F>
__device__ __forceinline__ void each_row(int fhalf, F&& f) {
#pragma unroll
    for (int mi = 0; mi < MM; ++mi)
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) f(mi, q * 4 + e, mi * 32 + q * 8 + fhalf * 4 + e);
}

// One column of a wave's logits, MM x 32 rows of the table from row0 on of
// which the lane and lane ^ 32 hold half each, `held` of them in the table:
// their sums (in both lanes), the target and, where asked for, the logits
// themselves.  RAGGED: held may be less than MM * 32.
template <int MM, bool RAGGED, typename A>
__device__ __forceinline__ void reduce_column(const LogitArgs& a, A& acc, int64_t token, int row0, int held, int64_t part,
                                              int fhalf) {
    const bool in = token < a.n;
    float most = NAN, sum[2] = {0.f, 0.f}, wsum[2] = {0.f, 0.f};
    const float sign = copysignf(1.f, a.c2);
    each_row<MM>(fhalf, [&](int mi, int e, int r) {
        if (!RAGGED || r < held) most = fmaxf(most, acc[mi][e] * sign);
    });
    most = fmaxf(most, __shfl_xor(most, 32, 64));
    // y less its largest, fused: what rounding takes from the largest y is in the sums then, and entropies have a third of
    // the error that rounded y leave (1.7e-7).  But of large y that is many powers of 2, more than an exponential holds,
    // and is taken off again.  A part of no number but NaN has a NaN for the largest, and so is not among the ones that may
    // hold alternatives; one with a -inf is.
    const float exact = most * sign;
    most = exact * a.c2;
    const float base = fmaxf(most, -FLT_MAX), over = fabsf(most) > 0x1p10f && fabsf(most) < INFINITY ? __builtin_fmaf(exact, a.c2, -most) : 0.f;
    each_row<MM>(fhalf, [&](int mi, int e, int r) {
        const float d = not_below(__builtin_fmaf(acc[mi][e], a.c2, -base) - over), p = exp2_fast(d);
        if (!RAGGED || r < held) {
            sum[e & 1] += p;
            wsum[e & 1] = __builtin_fmaf(p, d, wsum[e & 1]);
        }
    });
    float s = sum[0] + sum[1], w = wsum[0] + wsum[1];
    s += __shfl_xor(s, 32, 64);
    w += __shfl_xor(w, 32, 64);
    if (in && fhalf == 0) a.parts[part * a.n + token] = make_float4(most, s, w, 0.f);
    if (a.ids.ids) {
        const int t = in ? token_of(a.ids, token, a.rows).target - row0 : -1;
        if (__ballot(t >= 0 && t < MM * 32))
            each_row<MM>(fhalf, [&](int mi, int e, int r) {
                if (r == t) a.targets[token] = acc[mi][e] * a.c2;
            });
    }
    if (a.logits && in) {
        float* to = a.logits + (part * a.n + token) * (MM * 32);
#pragma unroll
        for (int mi = 0; mi < MM; ++mi)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = mi * 32 + q * 8 + fhalf * 4;
                if (!RAGGED || r < held)  // up to three values past the table's end, inside the part
                    *reinterpret_cast<float4*>(to + r) = make_float4(acc[mi][q * 4] * a.c2, acc[mi][q * 4 + 1] * a.c2,
                                                                     acc[mi][q * 4 + 2] * a.c2, acc[mi][q * 4 + 3] * a.c2);
            }
    }
}

// Column ni of the accumulators, as reduce_column indexes it.
template <int MM, int MN> struct Column {
    f32x16_t (&acc)[MM][MN];
    int ni;
    __device__ __forceinline__ f32x16_t& operator[](int mi) { return acc[mi][ni]; }
};

// A tile of logits, BT rows of the table by BT tokens, reduced over each
// wave's BT/2 rows.  Bound by the MFMAs at the clock they leave: 4096 tokens
// over 128256 x 4096 in 3.30 - 3.48 ms, by machine, 1.24 - 1.30 PFLOP/s (a library
// product of the shape, whose 1 GB of logits is not reduced, 3.00); 1024 over 50257 x 768 in 97 us,
// 12 stages, of which starting and reducing a tile takes a part; of 80 or 245
// tiles, one a CU, 0.5 us a stage, LDS reads and MFMAs in turn.
template <int BT>
__global__ __launch_bounds__(256, BT == 256 ? 1 : 2) void k_head_logits(LogitArgs a) {
    using S = Shape<BT, 4>;
    __shared__ __attribute__((aligned(16))) uint8_t lds[Pipe<BT, 4>::BYTES];
    int ti, tj;
    tile_of(int(blockIdx.x), a.tp * a.tq, a.tp, a.tq, ti, tj);
    f32x16_t acc[S::MM][S::MN];
    tile_loop<false, false, BT>(acc, a.table, a.x, int64_t(ti) * BT, int64_t(tj) * BT, 0, a.stages, lds);

    const int lane = threadIdx.x & 63, wave = uni(int(threadIdx.x) >> 6);
    const int wm = wave >> 1, wn = wave & 1, frow = lane & 31, fhalf = lane >> 5;
    const int row0 = ti * BT + wm * S::WTM, held = a.rows - row0;
    const int64_t part = int64_t(ti) * 2 + wm;
#pragma unroll
    for (int ni = 0; ni < S::MN; ++ni) {
        const int64_t token = int64_t(tj) * BT + wn * S::WTN + ni * 32 + frow;
        Column<S::MM, S::MN> col{acc, ni};
        if (held >= S::WTM)
            reduce_column<S::MM, false>(a, col, token, row0, held, part, fhalf);
        else
            reduce_column<S::MM, true>(a, col, token, row0, held, part, fhalf);
    }
}

// ---- few tokens: the table read once, straight into MFMA fragments ----

struct FewArgs {
    LogitArgs l;         // without operands
    const uint8_t* table;
    const uint8_t* x;
    int64_t x_pitch;     // bytes
    int64_t pitch;       // bytes of a row of the table
    int cols;
};

// The 16 bytes of T (bf16 or fp32) that elements k .. of a row of D make.
template <typename T, int D, bool INSIDE, bool PAST> __device__ __forceinline__ u32x4_t granule(const uint8_t* row, int k, int cols) {
    if constexpr (D == kF32 || sizeof(T) == 2) {
        return row_word<D, INSIDE, PAST>(row, k, cols);
    } else {
        typedef unsigned int half_t __attribute__((ext_vector_type(2), aligned(2)));
        u32x2_t r = {0u, 0u};
        if (INSIDE || k + 4 <= cols) {
            r = *reinterpret_cast<const half_t*>(row + 2 * k);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (k + e < cols) r[e >> 1] |= uint32_t(reinterpret_cast<const uint16_t*>(row)[k + e]) << (16 * (e & 1));
        }
        return u32x4_t{r[0] << 16, r[0] & 0xffff0000u, r[1] << 16, r[1] & 0xffff0000u};
    }
}

// Orders a wave's LDS writes before its reads and the other way round: lanes
// exchange values through a part of LDS that no other wave touches.
__device__ __forceinline__ void wave_exchange() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// RB * 32 rows of the table by NB * 32 tokens a block.  Its four waves share
// the contraction, 128 bytes of T in turn.  A wave loads its lines of both
// operands with 8 lanes a row, so that a load instruction takes whole lines (a
// load straight into the fragment's layout touches 64 of them for 16 bytes
// each: 410 us where this takes 205, 5.1 TB/s, 32 tokens over 128256 x 4096), several
// lines ahead, and turns them to fragments in an LDS tile of its own: no
// barrier until the end.  Every column of the product is one token's alone, so
// what padding or a row past the last holds goes nowhere.
template <int WD, int XD, int RB, int NB>
__global__ __launch_bounds__(256) void k_head_few(FewArgs f) {
    using T = std::conditional_t<WD == kBF16 && XD == kBF16, uint16_t, float>;
    constexpr int LINE = 128 / int(sizeof(T)), GE = 16 / int(sizeof(T));  // elements of a line and a granule
    constexpr int ROWS = (RB + NB) * 32;                                   // LDS rows of a wave's tile
    constexpr int AHEAD = RB + NB == 2 ? 4 : 2;                            // lines on their way
    constexpr int TILE = 4 * ROWS * 128, SUMS = 4 * RB * NB * 16 * 64 * 4;
    const LogitArgs& a = f.l;
    __shared__ __attribute__((aligned(16))) uint8_t lds[TILE > SUMS ? TILE : SUMS];
    const int lane = threadIdx.x & 63, wave = uni(int(threadIdx.x) >> 6);
    const int frow = lane & 31, fhalf = lane >> 5;
    const int row0 = int(blockIdx.x) * RB * 32;
    uint8_t* tile = lds + wave * ROWS * 128;
    const uint8_t *w[RB * 4], *x[NB * 4];  // the rows whose granules the lane loads
#pragma unroll
    for (int i = 0; i < RB * 4; ++i) w[i] = f.table + int64_t(min(row0 + i * 8 + (lane >> 3), a.rows - 1)) * f.pitch;
#pragma unroll
    for (int i = 0; i < NB * 4; ++i) x[i] = f.x + min(int64_t(i * 8 + (lane >> 3)), a.n - 1) * f.x_pitch;
    f32x16_t acc[RB][NB] = {};
    const int lines = (f.cols + LINE - 1) / LINE, mine = (lane & 7) * GE;
    struct Line {
        u32x4_t w[RB * 4], x[NB * 4];
    };
    auto load = [&](Line& to, int line, auto INSIDE) {
        const int k = line * LINE + mine;
#pragma unroll
        for (int i = 0; i < RB * 4; ++i) to.w[i] = granule<T, WD, decltype(INSIDE)::value, true>(w[i], k, f.cols);
#pragma unroll
        for (int i = 0; i < NB * 4; ++i) to.x[i] = granule<T, XD, decltype(INSIDE)::value, false>(x[i], k, f.cols);
    };
    auto multiply = [&](const Line& from) {
#pragma unroll
        for (int i = 0; i < (RB + NB) * 4; ++i) {
            const int r = i * 8 + (lane >> 3);
            *reinterpret_cast<u32x4_t*>(tile + r * 128 + swz_r<8>(r, lane & 7) * 16) = i < RB * 4 ? from.w[i] : from.x[i - RB * 4];
        }
        wave_exchange();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            u32x4_t fr[RB + NB];
#pragma unroll
            for (int j = 0; j < RB + NB; ++j) {
                const int r = j * 32 + frow;
                fr[j] = *reinterpret_cast<const u32x4_t*>(tile + r * 128 + swz_r<8>(r, 2 * kk + fhalf) * 16);
            }
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int j = 0; j < NB; ++j) Mfma<T>::step(acc[i][j], fr[i], fr[RB + j]);
        }
        wave_exchange();
    };
    // AHEAD lines on their way: one is multiplied, the one AHEAD lines of the wave further takes its registers (past
    // the last whole line, that line again)
    const int whole = f.cols / LINE;  // lines without zeros
    Line ring[AHEAD];
    int line = wave;
    if (line < whole) {
#pragma unroll
        for (int l = 0; l < AHEAD; ++l) load(ring[l], min(line + 4 * l, whole - 1), std::true_type{});
        while (line < whole) {
#pragma unroll
            for (int l = 0; l < AHEAD; ++l) {
                if (line < whole) {
                    multiply(ring[l]);
                    load(ring[l], min(line + 4 * AHEAD, whole - 1), std::true_type{});
                    line += 4;
                }
            }
        }
    }
    if (line < lines) {
        load(ring[0], line, std::false_type{});
        multiply(ring[0]);
    }
    __syncthreads();
    float* sums = reinterpret_cast<float*>(lds);  // [wave][i, j, accumulator][lane]
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) sums[((wave * RB * NB + i * NB + j) * 16 + e) * 64 + lane] = acc[i][j][e];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < RB * NB; ++q) {
        if (q % 4 != wave) continue;
        f32x16_t col[1];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            auto of = [&](int v) { return sums[((v * RB * NB + q) * 16 + e) * 64 + lane]; };
            col[0][e] = (of(0) + of(1)) + (of(2) + of(3));
        }
        const int first = row0 + q / NB * 32;
        if (first < a.rows)
            reduce_column<1, true>(a, col, q % NB * 32 + frow, first, a.rows - first, int64_t(blockIdx.x) * RB + q / NB, fhalf);
    }
}

// The same for bf16 rows of whole 128-byte lines at 16-byte addresses: WV waves
// with 32 rows of the table each, over the whole contraction, and NB * 32
// tokens that they share.  Both operands come by direct global->LDS loads, a
// line of every row a stage, into a ring of 3 stages: loads on their way take
// no registers, waves share x, and none waits for the others' sums at the end.
// One token over 50257 x 768: 14.8 us, 19.7 with the kernel above; 64 tokens
// over 128256 x 4096: 217 and 232.  But 32 tokens there: 200 and 186, of a
// table that does not fit the Infinity Cache; the kernel above has four lines
// of a row on their way at once.
template <int WV, int NB>
__global__ __launch_bounds__(64 * WV) void k_head_stream(FewArgs f) {
    constexpr int ROWS = WV * 32 + NB * 32, STAGE = ROWS * 128, SLOTS = 3;
    constexpr int LP = ROWS / 8 / WV;  // loads a wave and stage: 8 rows each, the first 4 of the table
    static_assert(ROWS / 8 % WV == 0, "whole loads");
    const LogitArgs& a = f.l;
    __shared__ __attribute__((aligned(16))) uint8_t lds[SLOTS * STAGE];
    const int lane = threadIdx.x & 63, wave = uni(int(threadIdx.x) >> 6);
    const int frow = lane & 31, fhalf = lane >> 5;
    const int row0 = int(blockIdx.x) * WV * 32;
    const uint8_t* from[LP];  // rows past the last are the last again
#pragma unroll
    for (int i = 0; i < LP; ++i) {
        const int r = (i * WV + wave) * 8 + (lane >> 3);
        from[i] = (i < 4 ? f.table + int64_t(min(row0 + r, a.rows - 1)) * f.pitch
                         : f.x + min(int64_t(r - WV * 32), a.n - 1) * f.x_pitch) +
                  swz_r<8>(r, lane & 7) * 16;
    }
    const int stages = f.cols / 64;
    auto load = [&](int t) {
        const int at = min(t, stages - 1) * 128;
        uint8_t* to = lds + t % SLOTS * STAGE + wave * 1024;
#pragma unroll
        for (int i = 0; i < LP; ++i) {
            if (i < 4)  // the table past the caches (the last argument's bit 1)
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(from[i] + at),
                                                 (__attribute__((address_space(3))) void*)(to + i * WV * 1024), 16, 0, 2);
            else
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(from[i] + at),
                                                 (__attribute__((address_space(3))) void*)(to + i * WV * 1024), 16, 0, 0);
        }
    };
    f32x16_t acc[NB] = {};
#pragma unroll
    for (int t = 0; t < SLOTS - 1; ++t) load(t);
    for (int t = 0; t < stages; ++t) {
        // this wave's loads of stage t have landed, then everyone's, and nobody reads stage t - 1 any more
        waitcnt_seen<(SLOTS - 2) * LP, 0>();
        __builtin_amdgcn_s_barrier();
        load(t + SLOTS - 1);
        const uint8_t* slot = lds + t % SLOTS * STAGE;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            auto fragment = [&](int r) { return *reinterpret_cast<const u32x4_t*>(slot + r * 128 + swz_r<8>(r, 2 * kk + fhalf) * 16); };
            const u32x4_t w = fragment(wave * 32 + frow);
#pragma unroll
            for (int j = 0; j < NB; ++j) Mfma<uint16_t>::step(acc[j], w, fragment(WV * 32 + j * 32 + frow));
        }
    }
    wait_vmcnt<0>();  // the loads past the end, before LDS is released
    const int first = row0 + wave * 32, held = a.rows - first;
    if (held <= 0) return;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
        f32x16_t col[1] = {acc[j]};
        if (held >= 32)
            reduce_column<1, false>(a, col, j * 32 + frow, first, held, int64_t(blockIdx.x) * WV + wave, fhalf);
        else
            reduce_column<1, true>(a, col, j * 32 + frow, first, held, int64_t(blockIdx.x) * WV + wave, fhalf);
    }
}

// ---- rows: parts joined, alternatives ----

struct Sums {
    float m, s, w;
};
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
    if (b.s == 0.f) return a;  // no part: NaN sums are not equal to 0
    if (a.s == 0.f) return b;
    const float m = fmaxf(a.m, b.m), da = not_below(a.m - m), db = not_below(b.m - m);  // da * s stays finite
    const float fa = exp2_fast(da), fb = exp2_fast(db);
    return Sums{m, __builtin_fmaf(a.s, fa, b.s * fb),
                __builtin_fmaf(fa, __builtin_fmaf(da, a.s, a.w), fb * __builtin_fmaf(db, b.s, b.w))};
}
__device__ __forceinline__ Sums shuffled(const Sums& a, int off) {
    return Sums{__shfl_xor(a.m, off, 64), __shfl_xor(a.s, off, 64), __shfl_xor(a.w, off, 64)};
}

// A wave's list of the k largest values, largest first, ties to the lower
// index: lane i holds entry i.  An empty entry is (-inf, INT_MAX).
struct TopList {
    float v;
    int id;
    int k, lane;
    __device__ __forceinline__ TopList(int k_, int lane_) : v(-INFINITY), id(INT32_MAX), k(k_), lane(lane_) {}
    static __device__ __forceinline__ bool before(float a, int ia, float b, int ib) { return a > b || (a == b && ia < ib); }
    // the value in a lane (the same lane for all), and each lane's neighbour's
    static __device__ __forceinline__ int read(int x, int from) { return __builtin_amdgcn_readlane(x, from); }
    static __device__ __forceinline__ float read(float x, int from) { return __int_as_float(read(__float_as_int(x), from)); }
    static __device__ __forceinline__ int shifted(int x) { return __builtin_amdgcn_mov_dpp(x, 0x138, 0xf, 0xf, false); }
    // every lane offers one value (or none); NaN is never before anything
    __device__ __forceinline__ void offer(float x, int ix, bool valid) {
        float last = read(v, k - 1);
        int ilast = read(id, k - 1);
        uint64_t mask = __ballot(valid && before(x, ix, last, ilast));
        while (mask) {
            const int src = __ffsll(static_cast<unsigned long long>(mask)) - 1;
            mask &= mask - 1;
            const float c = read(x, src);
            const int ic = read(ix, src);
            if (!before(c, ic, last, ilast)) continue;  // the list has grown since (the same in every lane)
            const int pos = __popcll(__ballot(before(v, id, c, ic)));
            const float pv = __int_as_float(shifted(__float_as_int(v)));  // of lane - 1
            const int pi = shifted(id);
            if (lane > pos) {
                v = pv;
                id = pi;
            } else if (lane == pos) {
                v = c;
                id = ic;
            }
            last = read(v, k - 1);
            ilast = read(id, k - 1);
        }
    }
};

struct RowArgs {
    const float4* parts;
    const float* targets;
    const float* logits;
    int64_t n;
    int n_parts, part_rows, rows;
    Ids ids;
    int64_t first_id;    // id of the table's row 0
    mfsdp_head_record* records;
    float *logp, *entropy;
    int top_k;
    int64_t* top_ids;
    float *top_logp, *top_logits;
};

__device__ __forceinline__ float nat(float y2) { return y2 * kLn2; }

// A token's sums, known to a whole wave, and what follows from them.
struct Row {
    Token t;
    Sums sum;
    float ls;   // log2 of the sum
    __device__ __forceinline__ float logp(float y) const { return nat((y - sum.m) - ls); }
};
__device__ __forceinline__ Row finish_row(const RowArgs& a, int64_t token, const Token& t, const Sums& sum, bool writes) {
    const Row r = {t, sum, sum.s == 0.f ? 0.f : log2f(sum.s)};
    if (writes) {
        const float y = t.target >= 0 ? a.targets[token] : 0.f;
        a.records[token] = mfsdp_head_record{t.live ? sum.m : 0.f, t.live ? sum.s : 0.f, t.live ? sum.w : 0.f, y, t.target >= 0, t.live};
        if (a.logp) a.logp[token] = t.target >= 0 ? r.logp(y) : 0.f;
        if (a.entropy) a.entropy[token] = t.live && sum.s != 0.f ? nat(r.ls - sum.w / sum.s) : 0.f;
    }
    return r;
}
__device__ __forceinline__ void put_top(const RowArgs& a, int64_t token, const Row& r, int place, float y, int id) {
    const int64_t at = token * a.top_k + place;
    const bool some = id != INT32_MAX;
    a.top_ids[at] = some ? a.first_id + id : -1;
    if (a.top_logits) a.top_logits[at] = some ? y : -INFINITY;
    if (a.top_logp) a.top_logp[at] = some ? r.logp(y) : -INFINITY;
}
// Joined over the lanes that lie BY apart among N neighbouring ones, in all of them.
template <int N, int BY = 1> __device__ __forceinline__ Sums wave_join(Sums mine, int lane) {
#pragma unroll
    for (int off = BY; off < N; off <<= 1) {
        const Sums other = shuffled(mine, off);
        mine = (lane & off) ? join(other, mine) : join(mine, other);
    }
    return mine;
}

// A token's alternatives by one wave: the parts with the largest M in a list,
// then those parts' rows in another.
__device__ __forceinline__ void top_by_lists(const RowArgs& a, int64_t token, const Row& r, int lane) {
    TopList parts(a.top_k, lane), top(a.top_k, lane);
    if (r.t.live)
        for (int p0 = 0; p0 < a.n_parts; p0 += 64) {
            const int p = p0 + lane;
            parts.offer(p < a.n_parts ? a.parts[int64_t(p) * a.n + token].x : 0.f, p, p < a.n_parts);
        }
    // the rows of the chosen parts, 64 at a time over all of them, four loads on their way
    const int total = r.t.live ? a.top_k * a.part_rows : 0;
    for (int at = 0; at < total; at += 256) {
        float y4[4];
        int row4[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = at + u * 64 + lane, k = i / a.part_rows;
            const int p = __shfl(parts.id, min(k, 63), 64);
            const int64_t row = int64_t(p) * a.part_rows + i % a.part_rows;
            row4[u] = i < total && p != INT32_MAX && row < a.rows ? int(row) : -1;  // fewer parts, the table's end
            y4[u] = row4[u] >= 0 ? a.logits[(int64_t(p) * a.n + token) * a.part_rows + i % a.part_rows] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) top.offer(y4[u], row4[u], row4[u] >= 0);
    }
    if (lane < a.top_k) put_top(a, token, r, lane, top.v, top.id);
}

// Rows of a batch, eight a block: 64 threads a row join the parts they stride
// over in order, then by a butterfly, the same order for the same sizes.  A
// wave's lanes take eight rows by eight parts, so that each load takes whole
// 128-byte lines of the parts, four on their way (4096 rows of 1002 parts:
// 17.1 us, by a wave a row 34.1).
constexpr int kRowsBlock = 8;
__global__ __launch_bounds__(64 * kRowsBlock) void k_head_rows(RowArgs a) {
    __shared__ Sums sums[kRowsBlock][kRowsBlock];  // [wave][row]
    const int lane = threadIdx.x & 63, wave = int(threadIdx.x) >> 6;
    const int64_t first = int64_t(blockIdx.x) * kRowsBlock;
    const int64_t row = min(first + (lane & 7), a.n - 1);  // past the last: the last again
    Sums mine = {-INFINITY, 0.f, 0.f};
    constexpr int kAtOnce = 4;
    for (int p0 = wave * 8 + (lane >> 3); p0 < a.n_parts; p0 += 64 * kAtOnce) {
        float4 v[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int64_t p = p0 + i * 64;
            v[i] = p < a.n_parts ? a.parts[p * a.n + row] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) mine = join(mine, Sums{v[i].x, v[i].y, v[i].z});
    }
    mine = wave_join<64, 8>(mine, lane);
    if (lane < 8) sums[wave][lane] = mine;
    __syncthreads();
    const int64_t token = first + wave;  // a wave a row from here on
    if (token >= a.n) return;
    mine = wave_join<8>(sums[lane & 7][wave], lane);
    const Row r = finish_row(a, token, token_of(a.ids, token, a.rows), mine, lane == 0);
    if (a.top_k) top_by_lists(a, token, r, lane);
}

// Tokens of a batch that is not large, a block of 16 waves each: latency, of
// reading the parts and the logits of the best ones.  Alternatives without a
// serial list: the k-th largest of 64 groups' largest M is at most the k-th
// largest logit, so the parts whose M reaches it hold all alternatives, and so
// do their logits that reach it, which a second such threshold thins out where
// they are many; each one left finds its place by counting the ones before it.
// (One token over 50257 rows, 5 alternatives: 10.8 us, by lists 29.)  More parts
// or logits than there is room for, as where most logits are equal, go through
// the lists.
constexpr int kRowWaves = 16, kRoomParts = 512, kRoomRows = 1024;
__global__ __launch_bounds__(64 * kRowWaves) void k_head_few_rows(RowArgs a) {
    __shared__ Sums sums[kRowWaves];
    __shared__ float group_most[64];
    __shared__ int parts[kRoomParts];
    __shared__ float2 rows[kRoomRows], best[kRoomRows];  // y and the row's number
    __shared__ int n_parts, n_rows, n_best;
    const int lane = threadIdx.x & 63, wave = int(threadIdx.x) >> 6;
    const int64_t token = blockIdx.x;
    Sums mine = {-INFINITY, 0.f, 0.f};
    float most = -INFINITY;
    // 16 threads a group, parts dealt out to the 64 groups in turn
    const int dealt = int(threadIdx.x) / 16 + int(threadIdx.x) % 16 * 64;
    constexpr int kTurn = 64 * kRowWaves, kAtOnce = 4;  // parts on their way at once
    float largest[kAtOnce];                             // of the last ones
    for (int p0 = 0; p0 < a.n_parts; p0 += kAtOnce * kTurn) {
        float4 v[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int64_t p = p0 + i * kTurn + dealt;
            v[i] = p < a.n_parts ? a.parts[p * a.n + token] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            mine = join(mine, Sums{v[i].x, v[i].y, v[i].z});
            most = fmaxf(most, v[i].x);
            largest[i] = v[i].x;
        }
    }
    mine = wave_join<64>(mine, lane);
    if (lane == 0) sums[wave] = mine;
    if (a.top_k) {
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
        if ((lane & 15) == 0) group_most[wave * 4 + lane / 16] = most;
        if (threadIdx.x == 0) n_parts = n_rows = n_best = 0;
    }
    __syncthreads();
    mine = wave_join<kRowWaves>(sums[lane % kRowWaves], lane);
    const Row r = finish_row(a, token, token_of(a.ids, token, a.rows), mine, threadIdx.x == 0);
    if (!a.top_k) return;
    if (!r.t.live) {
        if (int(threadIdx.x) < a.top_k) put_top(a, token, r, threadIdx.x, 0.f, INT32_MAX);
        return;
    }
    // the k-th largest of the groups' values, by each one's place among them
    auto least_of_groups = [&] {
        const float g = group_most[lane];
        int place = 0;
#pragma unroll 8
        for (int k = 0; k < 64; ++k) place += TopList::before(TopList::read(g, k), k, g, lane);
        return TopList::read(g, __ffsll(static_cast<unsigned long long>(__ballot(place == a.top_k - 1))) - 1);
    };
    float least = least_of_groups();
    for (int p0 = 0; p0 < a.n_parts; p0 += kAtOnce * kTurn)
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int64_t p = p0 + i * kTurn + dealt;
            if (p >= a.n_parts) continue;
            const float m = a.n_parts > kAtOnce * kTurn ? a.parts[p * a.n + token].x : largest[i];
            if (m >= least) {
                const int at = atomicAdd(&n_parts, 1);  // their order does not matter
                if (at < kRoomParts) parts[at] = int(p);
            }
        }
    __syncthreads();
    const int total = n_parts * a.part_rows;
    if (n_parts <= kRoomParts)
        for (int i = threadIdx.x; i < total; i += 64 * kRowWaves) {
            const int64_t p = parts[i / a.part_rows], row = p * a.part_rows + i % a.part_rows;
            const float y = row < a.rows ? a.logits[(p * a.n + token) * a.part_rows + i % a.part_rows] : 0.f;
            if (row < a.rows && y >= least) {
                const int at = atomicAdd(&n_rows, 1);
                if (at < kRoomRows) rows[at] = make_float2(y, __int_as_float(int(row)));
            }
        }
    __syncthreads();
    if (n_parts > kRoomParts || n_rows > kRoomRows) {
        if (wave == 0) top_by_lists(a, token, r, lane);
        return;
    }
    // many of them (a table of few parts): once more, by groups of them
    const float2* list = rows;
    int count = n_rows;
    const float2 mine_row = dealt < count ? rows[dealt] : make_float2(-INFINITY, 0.f);
    if (count > 4 * a.top_k) {
        most = mine_row.x;
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) most = fmaxf(most, __shfl_xor(most, off, 64));
        if ((lane & 15) == 0) group_most[wave * 4 + lane / 16] = most;
        __syncthreads();
        least = least_of_groups();
        if (dealt < count && mine_row.x >= least) best[atomicAdd(&n_best, 1)] = mine_row;
        __syncthreads();
        list = best;
        count = n_best;
    }
    if (int(threadIdx.x) < count) {
        const float2 v = list[threadIdx.x];
        int before = 0;
#pragma unroll 8
        for (int k = 0; k < count; ++k) {
            const float2 o = list[k];
            before += TopList::before(o.x, __float_as_int(o.y), v.x, __float_as_int(v.y));
        }
        if (before < a.top_k) put_top(a, token, r, before, v.x, __float_as_int(v.y));
    }
    if (int(threadIdx.x) >= count && int(threadIdx.x) < a.top_k) put_top(a, token, r, threadIdx.x, 0.f, INT32_MAX);
}

struct TotalArgs {
    const mfsdp_head_record* parts;
    int count;
    int64_t n;
    mfsdp_head_record* records;
    float *logp, *entropy;
    int top_k;
    const int64_t* part_ids;
    const float* part_logits;
    int64_t* top_ids;
    float *top_logp, *top_logits;
};

// Records of several tables joined in their order, a wave a token.
// Alternatives: an entry's place in the parts' lists stands for its id, so
// that equal logits keep the parts' order.
__global__ __launch_bounds__(256) void k_head_total(TotalArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t token = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (token >= a.n) return;
    Sums all = {-INFINITY, 0.f, 0.f};
    float target = 0.f;
    int found = 0, active = 0;
    for (int c = 0; c < a.count; ++c) {
        const mfsdp_head_record r = a.parts[c * a.n + token];
        all = join(all, Sums{r.max, r.sum, r.wsum});
        if (r.found) target = r.target;
        found |= r.found;
        active |= r.active;
    }
    const float ls = all.s == 0.f ? 0.f : log2f(all.s);
    TopList top(a.top_k ? a.top_k : 1, lane);
    for (int c = 0; a.top_k && c < a.count; ++c) {
        const int64_t at = (c * a.n + token) * a.top_k + lane;
        const bool in = lane < a.top_k && a.part_ids[at] >= 0;
        top.offer(in ? a.part_logits[at] : 0.f, c * a.top_k + lane, in);
    }
    // every record of the token has been read before one is written
    if (lane == 0) {
        a.records[token] = mfsdp_head_record{active ? all.m : 0.f, all.s, all.w, target, found, active};
        if (a.logp) a.logp[token] = found ? nat((target - all.m) - ls) : 0.f;
        if (a.entropy) a.entropy[token] = active && all.s != 0.f ? nat(ls - all.w / all.s) : 0.f;
    }
    if (lane < a.top_k) {
        const int64_t at = token * a.top_k + lane;
        const bool some = top.id != INT32_MAX;
        const int64_t from = some ? (int64_t(top.id / a.top_k) * a.n + token) * a.top_k + top.id % a.top_k : 0;
        a.top_ids[at] = some ? a.part_ids[from] : -1;
        if (a.top_logits) a.top_logits[at] = top.v;
        if (a.top_logp) a.top_logp[at] = some ? nat((top.v - all.m) - ls) : -INFINITY;
    }
}

// Records of an empty table: nothing in the sums, no target.
__global__ __launch_bounds__(256) void k_head_empty(RowArgs a) {
    const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
    if (i >= a.n) return;
    const bool live = token_of(a.ids, i, 0).live;
    a.records[i] = mfsdp_head_record{live ? -INFINITY : 0.f, 0.f, 0.f, 0.f, 0, live};
    if (a.logp) a.logp[i] = 0.f;
    if (a.entropy) a.entropy[i] = 0.f;
    for (int k = 0; k < a.top_k; ++k) {
        a.top_ids[i * a.top_k + k] = -1;
        if (a.top_logits) a.top_logits[i * a.top_k + k] = -INFINITY;
        if (a.top_logp) a.top_logp[i * a.top_k + k] = -INFINITY;
    }
}

// ---- backward ----

// What rounding to bf16 took from the large entries of dz, a token's in no
// order: the k-th at [k][token].  A token that counts more than kMaxRests (the
// records were not of these operands) has none.
constexpr int kListRows = 128;
struct Rests {
    int* counts;      // [token]
    int* groups;      // [128 rows of the table]: entries found there, those of tokens that have none among them
    int* rows;        // [kMaxRests][token]: of the table
    float* values;
    int64_t tokens;   // from k to k + 1
    __device__ __forceinline__ int count(int64_t token) const {
        const int c = counts[token];
        return c <= kMaxRests ? c : 0;
    }
    // places of `some` more of a token's entries, from the one returned on (their order is settled where they are read)
    __device__ __forceinline__ int places(int64_t token, int some) const { return atomicAdd(&counts[token], some); }
    __device__ __forceinline__ void put(int k, int64_t token, int row, float value) const {
        if (k >= kMaxRests) return;
        rows[k * tokens + token] = row;
        values[k * tokens + token] = value;
    }
};

struct DzArgs {
    LogitArgs l;
    const mfsdp_head_record* records;
    const float *dlogp, *dentropy;
    float scale;
    uint8_t* dz;       // [plane][64 rows of the table][tokens, whole tiles][64] bf16
    int64_t block;     // bytes from 64 rows to the next 64
    int planes;
    int64_t plane;
    Rests rests;       // one plane
};

// dz of a tile: formed in the accumulators, staged in LDS as [token][row of
// the table] in bf16, a plane at a time, and written in whole 16-byte words.
// Zeros for tokens and rows past the last, and for padding.  Bound as
// k_head_logits: 3.54 - 3.62 ms for 4096 tokens over 128256 x 4096 (1.19 - 1.22
// PFLOP/s, and 1 GB of dz written), 115 - 134 us for 1024 over 50257 x 768.
template <int BT>
__global__ __launch_bounds__(256, BT == 256 ? 1 : 2) void k_head_dz(DzArgs d) {
    using S = Shape<BT, 4>;
    const LogitArgs& a = d.l;
    __shared__ __attribute__((aligned(16))) uint8_t lds[Pipe<BT, 4>::BYTES];
    int ti, tj;
    tile_of(int(blockIdx.x), a.tp * a.tq, a.tp, a.tq, ti, tj);
    f32x16_t acc[S::MM][S::MN];
    tile_loop<false, false, BT>(acc, a.table, a.x, int64_t(ti) * BT, int64_t(tj) * BT, 0, a.stages, lds);

    constexpr int RB = BT * 2, GPR = RB / 16;  // bytes and 16-byte words of a staged row
    static_assert(BT * RB <= Pipe<BT, 4>::BYTES, "staging area");
    const int lane = threadIdx.x & 63, wave = uni(int(threadIdx.x) >> 6);
    const int wm = wave >> 1, wn = wave & 1, frow = lane & 31, fhalf = lane >> 5;
    const int row0 = ti * BT + wm * S::WTM, held = a.rows - row0;
    int found = 0;  // large entries of the wave, all in one group of rows
    static_assert(kListRows % S::WTM == 0, "a wave's rows lie in one group");
#pragma unroll
    for (int ni = 0; ni < S::MN; ++ni) {
        const int64_t token = int64_t(tj) * BT + wn * S::WTN + ni * 32 + frow;
        float m = 0.f, ls = 0.f, b = 0.f, c = 0.f, hit = 0.f, least = NAN;  // least: of large entries, NaN where none is kept
        int t = -1;
        bool live = false;
        if (token < a.n) {
            const Token tok = token_of(a.ids, token, a.rows);
            const mfsdp_head_record r = d.records[token];
            live = tok.live && r.active;
            const float up = r.found ? d.dlogp[token] : 0.f, dh = d.dentropy ? d.dentropy[token] : 0.f;
            m = r.max;
            ls = log2f(r.sum);
            // dz = hit - p (b + c lp), lp = log2 p; NaN where the sum is none
            b = d.scale * (d.dentropy ? __builtin_fmaf(dh, nat(ls - r.wsum / r.sum), up) : up);
            if (!(r.sum > 0.f)) b = NAN;
            c = d.scale * dh * kLn2;
            if (d.planes == 1 && live) {
                // sum |dz_j| is at most |scale| (|dlogp| 2 (1 - p_t) + |dH| 2 H); 1 - p_t and H as far as roundings leave them
                const float pt = r.found ? exp2_fast(fminf((r.target - m) - ls, 0.f)) : 1.f;
                const float h = d.dentropy ? fmaxf(nat(ls - r.wsum / r.sum), 0x1p-15f) : 0.f;
                least = 2.f * kShare * fabsf(d.scale) * (fabsf(up) * fmaxf(1.f - pt, 0x1p-15f) + fabsf(dh) * h);
                if (least == 0.f) least = NAN;  // no gradient
            }
            if (tok.target >= 0 && r.found && live) {
                t = tok.target - row0;
                hit = d.scale * up;
            }
        }
        each_row<S::MM>(fhalf, [&](int mi, int e, int) {
            // y rounded: the largest less m is 0 however large it is; and at most 0, since y is formed again, in another
            // order than by k_head_few, and may pass the largest by its rounding
            const float lp = __builtin_amdgcn_fmed3f((acc[mi][ni][e] * a.c2 - m) - ls, -1024.f, 0.f);
            const float v = -exp2_fast(lp) * __builtin_fmaf(c, lp, b);
            acc[mi][ni][e] = live ? v : 0.f;
        });
        if (held < S::WTM)
            each_row<S::MM>(fhalf, [&](int mi, int e, int r) {
                if (r >= held) acc[mi][ni][e] = 0.f;
            });
        if (__ballot(t >= 0 && t < S::WTM))
            each_row<S::MM>(fhalf, [&](int mi, int e, int r) {
                if (r == t) acc[mi][ni][e] += hit;
            });
        float most = 0.f;
        each_row<S::MM>(fhalf, [&](int mi, int e, int) { most = fmaxf(most, fabsf(acc[mi][ni][e])); });
        if (!__ballot(most >= least)) continue;
        // the large ones, a bit each; then one a lane at a time, while their places are on their way
        uint64_t large = 0;
        each_row<S::MM>(fhalf, [&](int mi, int e, int) {
            large |= fabsf(acc[mi][ni][e]) >= least ? uint64_t(1) << (mi * 16 + e) : 0;
        });
        int place = large ? d.rests.places(token, __popcll(large)) : 0;
        while (const uint64_t some = __ballot(large != 0)) {
            const int q = large ? __ffsll(static_cast<unsigned long long>(large)) - 1 : -1;
            large &= large - 1;
            float v = 0.f;
            each_row<S::MM>(fhalf, [&](int mi, int e, int) { v = q == mi * 16 + e ? acc[mi][ni][e] : v; });
            const float rest = v - bf16_to_f32(f32_to_bf16(v));
            if (q >= 0)
                d.rests.put(place++, token, row0 + (q >> 4) * 32 + (q >> 2 & 3) * 8 + fhalf * 4 + (q & 3), fabsf(rest) < INFINITY ? rest : 0.f);
            found += __popcll(some);
        }
    }
    if (found > 0 && lane == 0) atomicAdd(&d.rests.groups[row0 / kListRows], found);
    for (int plane = 0; plane < d.planes; ++plane) {
        __syncthreads();  // the operands' stages, or the plane before, have been read
#pragma unroll
        for (int ni = 0; ni < S::MN; ++ni) {
            const int cl = wn * S::WTN + ni * 32 + frow;
#pragma unroll
            for (int mi = 0; mi < S::MM; ++mi)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int rl = wm * S::WTM + mi * 32 + q * 8 + fhalf * 4;
                    const uint2 w = make_uint2(pack_bf16x2(acc[mi][ni][q * 4], acc[mi][ni][q * 4 + 1]),
                                               pack_bf16x2(acc[mi][ni][q * 4 + 2], acc[mi][ni][q * 4 + 3]));
                    if (d.planes > 1) {
                        acc[mi][ni][q * 4] -= __uint_as_float(w.x << 16);
                        acc[mi][ni][q * 4 + 1] -= __uint_as_float(w.x & 0xffff0000u);
                        acc[mi][ni][q * 4 + 2] -= __uint_as_float(w.y << 16);
                        acc[mi][ni][q * 4 + 3] -= __uint_as_float(w.y & 0xffff0000u);
                    }
                    *reinterpret_cast<uint2*>(lds + cl * RB + ((rl >> 3) ^ (cl & (GPR - 1))) * 16 + ((rl >> 2) & 1) * 8) = w;
                }
        }
        __syncthreads();
        uint8_t* to = d.dz + plane * d.plane + int64_t(ti) * (BT / 64) * d.block + int64_t(tj) * BT * 128;
#pragma unroll 8
        for (int i = 0; i < BT * GPR / 256; ++i) {
            const int k = int(threadIdx.x) + i * 256, b = k / (BT * 8), r = k / 8 % BT, j = b * 8 + k % 8;
            *reinterpret_cast<u32x4_t*>(to + b * d.block + (k % (BT * 8)) * 16) =
                *reinterpret_cast<const u32x4_t*>(lds + r * RB + (j ^ (r & (GPR - 1))) * 16);
        }
    }
}

// A tile of fp32 accumulators, handed on in the order of its columns: through
// LDS in passes of BT*BT*4 / 128 KB, where row c of the staging area is tile
// column c of the pass, its 16-byte words j at j ^ (c % 32).  fix(pass,
// staging area) may change it (the block is in step before and after), then
// before(c, r) and out(c, r, what before gave, eight values) see the values of
// tile rows r .. r+7 of tile column c, `before` of a whole pass ahead of its
// staging, so that what it loads is on its way meanwhile.
struct Values {
    float4 a, b;
};
template <int BT> struct Staging {
    static constexpr int PASSES = BT == 256 ? 2 : 1, COLS = BT / PASSES, BYTES = COLS * BT * 4;
    static_assert(BYTES <= Pipe<BT, 4>::BYTES, "staging area");
    float* at;
    __device__ __forceinline__ float4& word(int c, int j) const {  // c in the pass
        return *reinterpret_cast<float4*>(at + c * BT + ((j ^ (c & 31)) * 4));
    }
};
// (Barriers of LDS accesses alone, so that a pass does not wait for the stores
// of the one before it.)
template <int BT, typename FIX, typename BEFORE, typename OUT>
__device__ __forceinline__ void walk_columns(const f32x16_t (&acc)[BT / 64][BT / 64], uint8_t* lds, FIX&& fix,
                                             BEFORE&& before, OUT&& out) {
    using S = Shape<BT, 4>;
    using G = Staging<BT>;
    constexpr int NCH = BT / 8, TURNS = G::COLS * NCH / 256;
    constexpr int STEP = 256 / NCH;  // columns from turn to turn
    const int c0 = int(threadIdx.x) / NCH, r = int(threadIdx.x) % NCH * 8;
    const G st = {reinterpret_cast<float*>(lds)};
    const int lane = threadIdx.x & 63, wave = uni(int(threadIdx.x) >> 6);
    const int wm = wave >> 1, wn = wave & 1, frow = lane & 31, fhalf = lane >> 5;
    stage_barrier();  // every wave is done with the operands' stages
#pragma unroll
    for (int h = 0; h < G::PASSES; ++h) {
        decltype(before(0, 0)) early[TURNS];
#pragma unroll
        for (int i = 0; i < TURNS; ++i) early[i] = before(h * G::COLS + c0 + i * STEP, r);
        if (G::PASSES == 1 || wn == h) {
#pragma unroll
            for (int mi = 0; mi < S::MM; ++mi)
#pragma unroll
                for (int ni = 0; ni < S::MN; ++ni)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int rl = wm * S::WTM + mi * 32 + q * 8 + fhalf * 4;
                        const int cl = wn * S::WTN + ni * 32 + frow - h * G::COLS;
                        const f32x16_t& v = acc[mi][ni];
                        st.word(cl, rl >> 2) = make_float4(v[q * 4], v[q * 4 + 1], v[q * 4 + 2], v[q * 4 + 3]);
                    }
        }
        stage_barrier();
        fix(h, st);
#pragma unroll
        for (int i = 0; i < TURNS; ++i) {
            const int c = c0 + i * STEP;
            out(h * G::COLS + c, r, early[i], Values{st.word(c, r / 4), st.word(c, r / 4 + 1)});
        }
        if (h + 1 < G::PASSES) stage_barrier();
    }
}

// Eight consecutive elements of a row as they lie, from column c on, n of them
// inside (the others 0); as whole vectors where `vector` says that rows are
// aligned for it.  Stores go past the caches.
template <int D> struct Eight;
template <> struct Eight<kBF16> {
    u32x4_t v;
    __device__ __forceinline__ void load(const uint8_t* row, int c, int n, bool vector) {
        if (n >= 8 && vector) {
            v = *reinterpret_cast<const u32x4_t*>(row + c * 2);
            return;
        }
        const uint16_t* e = reinterpret_cast<const uint16_t*>(row) + c;
        v = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) v[k >> 1] |= uint32_t(e[k]) << (16 * (k & 1));
    }
    __device__ __forceinline__ Values get() const {
        auto lo = [&](int k) { return __uint_as_float(v[k] << 16); };
        auto hi = [&](int k) { return __uint_as_float(v[k] & 0xffff0000u); };
        return Values{make_float4(lo(0), hi(0), lo(1), hi(1)), make_float4(lo(2), hi(2), lo(3), hi(3))};
    }
    static __device__ __forceinline__ void store(uint8_t* row, int c, const Values& x) {
        __builtin_nontemporal_store(u32x4_t{pack_bf16x2(x.a.x, x.a.y), pack_bf16x2(x.a.z, x.a.w), pack_bf16x2(x.b.x, x.b.y),
                                            pack_bf16x2(x.b.z, x.b.w)},
                                    reinterpret_cast<u32x4_t*>(row + c * 2));
    }
};
template <> struct Eight<kF32> {
    Values v;
    __device__ __forceinline__ void load(const uint8_t* row, int c, int n, bool vector) {
        const float* e = reinterpret_cast<const float*>(row) + c;
        if (n >= 8 && vector) {
            v = Values{reinterpret_cast<const float4*>(e)[0], reinterpret_cast<const float4*>(e)[1]};
            return;
        }
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = k < n ? e[k] : 0.f;
        v = Values{make_float4(x[0], x[1], x[2], x[3]), make_float4(x[4], x[5], x[6], x[7])};
    }
    __device__ __forceinline__ Values get() const { return v; }
    static __device__ __forceinline__ void store(uint8_t* row, int c, const Values& x) {
        f32x4_t* p = reinterpret_cast<f32x4_t*>(row + c * 4);
        __builtin_nontemporal_store(f32x4_t{x.a.x, x.a.y, x.a.z, x.a.w}, p);
        __builtin_nontemporal_store(f32x4_t{x.b.x, x.b.y, x.b.z, x.b.w}, p + 1);
    }
};
template <int D> __device__ __forceinline__ void put8(uint8_t* row, int c, int n, bool vector, const Values& v) {
    if (n >= 8 && vector) {
        Eight<D>::store(row, c, v);
    } else {
        const float e[8] = {v.a.x, v.a.y, v.a.z, v.a.w, v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) store_elem(row, D, c + k, e[k]);
    }
}
__device__ __forceinline__ float4 fma4(float f, const float4& a, const float4& b) {
    return make_float4(__builtin_fmaf(f, a.x, b.x), __builtin_fmaf(f, a.y, b.y), __builtin_fmaf(f, a.z, b.z),
                       __builtin_fmaf(f, a.w, b.w));
}
__device__ __forceinline__ Values fma8(float f, const Values& x, const Values& y) {
    return Values{fma4(f, x.a, y.a), fma4(f, x.b, y.b)};
}

struct DxArgs {
    Operand table, dz;
    int64_t n;
    int cols, rows;
    int tp, tq;           // tiles along the columns and the batch
    int stages, splits;   // of the contraction over the vocabulary, and the parts it is cut into
    Ids ids;
    const float* rests;   // NULL, or [n][ld]: what the large entries' rests add
    uint8_t* dx;
    int64_t stride;
    int vector;
    float* sums;          // splits > 1: [split][n][ld], ld a multiple of 8
    int64_t ld;
};

// dx = dz W: P is W, read K-major (its rows are the contraction).  Its result
// is small and its contraction long, so that it is cut into parts (dx_cut).
// Bound by the MFMAs: 3.23 - 3.33 ms for 4096 tokens over 128256 x 4096 (1.29 - 1.33
// PFLOP/s), 84 - 97 + 8 us for 1024 over 50257 x 768 (0.93; 9 parts).
template <int D, int BT>
__global__ __launch_bounds__(256, BT == 256 ? 1 : 2) void k_head_dx(DxArgs a) {
    using S = Shape<BT, 4>;
    __shared__ __attribute__((aligned(16))) uint8_t lds[Pipe<BT, 4>::BYTES];
    // parts one after another on an XCD (block index mod 8), whose L2 the tiles of a part share
    const int tiles = a.tp * a.tq;
    int split = 0, ti, tj;
    if (a.splits > 1) {
        const int all = tiles * a.splits, per = (all + 7) / 8;
        const int at = int(blockIdx.x & 7) * per + int(blockIdx.x >> 3);
        if (int(blockIdx.x >> 3) >= per || at >= all) return;
        split = at / tiles;
        ti = (at - split * tiles) % a.tp;
        tj = (at - split * tiles) / a.tp;
    } else {
        tile_of(int(blockIdx.x), tiles, a.tp, a.tq, ti, tj);
    }
    const int k0 = int(int64_t(a.stages) * split / a.splits), k1 = int(int64_t(a.stages) * (split + 1) / a.splits);
    f32x16_t acc[S::MM][S::MN];
    tile_loop<true, false, BT>(acc, a.table, a.dz, int64_t(ti) * BT, int64_t(tj) * BT, k0, k1, lds);
    walk_columns<BT>(
        acc, lds, [](int, const Staging<BT>&) {},
        [&](int c, int r) {
            const int64_t token = int64_t(tj) * BT + c;
            const int col = ti * BT + r;
            Eight<kF32> x = {};
            if (a.rests && a.splits == 1 && token < a.n && col < a.cols)
                x.load(reinterpret_cast<const uint8_t*>(a.rests + token * a.ld), col, 8, true);  // ld: of 8
            return x;
        },
        [&](int c, int r, const Eight<kF32>& x, Values v) {
            const int64_t token = int64_t(tj) * BT + c;
            const int col = ti * BT + r;
            if (token >= a.n || col >= a.cols) return;
            if (a.splits > 1) {
                float4* to = reinterpret_cast<float4*>(a.sums + (split * a.n + token) * a.ld + col);  // ld: of 8
                to[0] = v.a;
                to[1] = v.b;
            } else {
                if (a.rests) v = fma8(1.f, x.get(), v);
                if (!token_of(a.ids, token, a.rows).live) v = Values{};
                put8<D>(a.dx + token * a.stride * (D == kBF16 ? 2 : 4), col, a.cols - col, a.vector, v);
            }
        });
}

// The parts of dx added up: SLICES groups of consecutive parts, each in its
// order, by as many threads, then the groups' sums in theirs.  (8 tokens of 512
// columns in 117 parts are 512 words of work: 30 us with one thread each, all
// of it one load after another, 6.8 with 8.)
template <int D, int SLICES>
__global__ __launch_bounds__(256) void k_head_dx_sum(DxArgs a) {
    constexpr int WORDS = 256 / SLICES;
    __shared__ Values sums[SLICES][WORDS];
    const int slice = int(threadIdx.x) / WORDS, in = int(threadIdx.x) % WORDS;
    const int64_t w = int64_t(blockIdx.x) * WORDS + in, per = a.ld / 8;
    const int64_t token = w / per;
    const int col = int(w % per) * 8;
    const bool here = token < a.n;
    Values v = {};
    if (here && a.rests && slice == 0) {
        const float4* from = reinterpret_cast<const float4*>(a.rests + token * a.ld + col);
        v = Values{from[0], from[1]};
    }
    if (here) {
        const int end = a.splits * (slice + 1) / SLICES;
#pragma unroll 8
        for (int s = a.splits * slice / SLICES; s < end; ++s) {
            const float4* from = reinterpret_cast<const float4*>(a.sums + (s * a.n + token) * a.ld + col);
            v = fma8(1.f, Values{from[0], from[1]}, v);
        }
    }
    if constexpr (SLICES > 1) {
        sums[slice][in] = v;
        __syncthreads();
        if (slice > 0) return;
#pragma unroll
        for (int s = 1; s < SLICES; ++s) v = fma8(1.f, sums[s][in], v);
    }
    if (!here) return;
    if (!token_of(a.ids, token, a.rows).live) v = Values{};
    put8<D>(a.dx + token * a.stride * (D == kBF16 ? 2 : 4), col, a.cols - col, a.vector, v);
}

// What the rests of a token's large entries add to dx, a wave a token: times
// their rows of the table, in the rows' order, so that sums do not depend on
// which was found first.  HBM: the rows' bytes, and n x cols fp32 written.
struct GatherArgs {
    Rests rests;
    Operand table;     // one plane
    int64_t n;
    int64_t ld;        // of 8, and at most whole column blocks
    float* out;        // [n][ld]
    uint32_t blocks;
};
__device__ __forceinline__ void gather_block(const GatherArgs& a, uint32_t block) {
    const int lane = threadIdx.x & 63;
    const int64_t token = int64_t(block) * 4 + uni(int(threadIdx.x) >> 6);
    if (token >= a.n) return;
    const int count = uni(a.rests.count(token));
    static_assert(kMaxRests <= 64, "a lane an entry");
    int row = lane < count ? a.rests.rows[lane * a.rests.tokens + token] : 0;
    float value = lane < count ? a.rests.values[lane * a.rests.tokens + token] : 0.f;
    int place = 0;  // among the rows, which differ
    for (int k = 0; k < count; ++k) place += __builtin_amdgcn_readlane(row, k) < row;
    if (lane >= count) place = lane;
    row = __builtin_amdgcn_ds_permute(place * 4, row);
    value = __int_as_float(__builtin_amdgcn_ds_permute(place * 4, __float_as_int(value)));
    for (int64_t col = lane * 8; col < a.ld; col += 512) {
        Values v = {};
        for (int k = 0; k < count; k += 4) {  // four rows on their way
            Eight<kBF16> w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                w[u].load(a.table.at(__builtin_amdgcn_readlane(row, min(k + u, count - 1)), int(col)), 0, 8, true);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (k + u < count) v = fma8(__int_as_float(__builtin_amdgcn_readlane(__float_as_int(value), k + u)), w[u].get(), v);
        }
        float4* to = reinterpret_cast<float4*>(a.out + token * a.ld + col);
        to[0] = v.a;
        to[1] = v.b;
    }
}

struct DwArgs {
    Operand turned, dz;  // x with its columns as rows
    Operand x;
    int64_t n;
    int rows, cols;
    int tp, tq;          // tiles along the columns and the vocabulary
    int stages;          // of the contraction over the batch
    const int2* bounds;  // NULL, or of the lists below (x then has one plane)
    const uint2* list;
    const uint8_t* dense;
    uint8_t* grad;
    int vector;
    int add;
};

// For dW, the large entries of dz by a tile's rows of the table, 1 or 2 groups
// of 128 (span): as lists, or, where more entries than a quarter of the tokens
// lie in them, as a second plane of dz there, rests in bf16, which the tile then
// multiplies in a run of its own.  An entry of a list takes its tile 1/32 us, a
// run 1/128 us a token and up to three times that, so lists alone would cost
// hot rows (a likely token of every row; a table of 256 rows: the gradients of
// 4096 tokens of 768 columns 838 us, 114 so) far more than all other work, and
// planes alone all tiles as much again.  At most 32 entries a row make at most 128 such tiles.
struct ListArgs {
    Rests rests;
    int n, rows;
    int span;            // groups of a tile of dW
    int capacity;        // of the list
    int2* bounds;        // [group]: first entry in the list and past the last; or -1 and the plane's number
    uint2* list;
    uint8_t* dense;      // [plane][64 rows][token][64] bf16
    uint32_t units, planes, chunks;  // tiles of dW along the rows, planes there is room for, pieces of a plane
};
constexpr int kMostPlanes = 128, kPiece = 256;  // tokens of a piece
static_assert(kPadTokens % kPiece == 0, "whole pieces");
__device__ __forceinline__ int unit_entries(const ListArgs& a, int unit) {
    const int groups = (a.rows + kListRows - 1) / kListRows, g = unit * a.span;
    return a.rests.groups[g] + (a.span > 1 && g + 1 < groups ? a.rests.groups[g + 1] : 0);
}
__device__ __forceinline__ bool is_dense(const ListArgs& a, int entries) { return entries > a.n / 4; }

// One group's list, in an order that sizes and the entries alone fix: each the
// row in the group << 24 | the token (at most 2^22 of them), and the rest.  The
// block looks through all tokens, kLook times 256 at a time, each token's
// entries from the lowest row up; the first two of the next ones are on their
// way meanwhile.  Latency: a turn is a load, a barrier and the counts.
constexpr int kLook = 4;
__device__ __forceinline__ void list_block(const ListArgs& a, uint32_t block) {
    __shared__ int4 turns[2][kLook];
    int(&counts)[2][kLook][4] = reinterpret_cast<int(&)[2][kLook][4]>(turns);  // [.][.][wave]
    const int lane = threadIdx.x & 63, wave = int(threadIdx.x) >> 6;
    const int first = int(block) * kListRows, unit = int(block) / a.span;
    // a sum over the block, `most` at most (twice that is a whole number of 32 bits)
    auto block_sum = [&](int x, int most) {
        for (int off = 1; off < 64; off <<= 1) x = min(x + __shfl_xor(x, off, 64), most);
        if (lane == 0) counts[0][0][wave] = x;
        __syncthreads();
        const int4 c = turns[0][0];
        return min(min(c.x + c.y, most) + min(c.z + c.w, most), most);
    };
    if (is_dense(a, unit_entries(a, unit))) {
        int before = 0;  // such tiles before
        for (int u = threadIdx.x; u < unit; u += 256) before += is_dense(a, unit_entries(a, u));
        const int plane = block_sum(before, kMostPlanes);
        if (plane < int(a.planes)) {
            if (threadIdx.x == 0) a.bounds[block] = make_int2(-1, plane);
            return;
        }
        __syncthreads();
    }
    struct Ahead {
        int count, rows[2];
    };
    auto load = [&](int i) {
        Ahead h = {0, {0, 0}};
        if (i < a.n) h = Ahead{a.rests.counts[i], {a.rests.rows[i], a.rests.rows[a.rests.tokens + i]}};  // held or not
        return h;
    };
    Ahead next_ones[kLook];
#pragma unroll
    for (int u = 0; u < kLook; ++u) next_ones[u] = load(u * 256 + int(threadIdx.x));
    int below = 0;  // entries of the groups before
    for (int g = threadIdx.x; g < int(block); g += 256) below = min(below + a.rests.groups[g], a.capacity);
    const int start = block_sum(below, a.capacity);
    int at = start, turn = 0;
    for (int i0 = 0; i0 < a.n; i0 += kLook * 256) {
        Ahead h[kLook];
        int last[kLook];  // the row in the group that this token's entries up to it are listed
#pragma unroll
        for (int u = 0; u < kLook; ++u) {
            h[u] = next_ones[u];
            next_ones[u] = load(i0 + (kLook + u) * 256 + int(threadIdx.x));
            last[u] = -1;
        }
        for (bool more = true; more;) {
            int next[kLook], from[kLook], left[kLook];
            uint64_t mask[kLook], again = 0;
#pragma unroll
            for (int u = 0; u < kLook; ++u) {
                const int c = h[u].count <= kMaxRests ? h[u].count : 0;
                next[u] = kListRows;
                from[u] = left[u] = 0;
                auto look = [&](int k, int row) {
                    const int r = row - first;
                    if (r <= last[u] || r >= kListRows) return;
                    ++left[u];
                    if (r < next[u]) {
                        next[u] = r;
                        from[u] = k;
                    }
                };
                if (c > 0) look(0, h[u].rows[0]);
                if (c > 1) look(1, h[u].rows[1]);
                for (int k = 2; k < c; ++k) look(k, a.rests.rows[k * a.rests.tokens + i0 + u * 256 + int(threadIdx.x)]);
                mask[u] = __ballot(left[u] > 0);
                again |= __ballot(left[u] > 1);
            }
            turn ^= 1;  // one barrier a turn: counts of the last are still read
            if (lane == 0)
#pragma unroll
                for (int u = 0; u < kLook; ++u) counts[turn][u][wave] = __popcll(mask[u]) | (u == 0 && again ? 1 << 16 : 0);
            __syncthreads();
            more = false;
#pragma unroll
            for (int u = 0; u < kLook; ++u) {
                const int4 c = turns[turn][u];
                const int before = ((wave > 0 ? c.x : 0) + (wave > 1 ? c.y : 0) + (wave > 2 ? c.z : 0)) & 0xffff;
                const int all = c.x + c.y + c.z + c.w, to = at + before + __popcll(mask[u] & ((uint64_t(1) << lane) - 1));
                const int64_t i = i0 + u * 256 + int(threadIdx.x);
                if (left[u] > 0 && to < a.capacity)
                    a.list[to] = make_uint2(uint32_t(next[u]) << 24 | uint32_t(i), __float_as_uint(a.rests.values[from[u] * a.rests.tokens + i]));
                at += all & 0xffff;
                more |= all >> 16 != 0;
                last[u] = next[u];
            }
        }
    }
    if (threadIdx.x == 0) a.bounds[block] = make_int2(start, min(at, a.capacity));
}

// A piece of one plane, whose tile is the one with as many before it.
__device__ __forceinline__ void dense_block(const ListArgs& a, uint32_t block) {
    __shared__ int counts[4], found;
    const int lane = threadIdx.x & 63, wave = int(threadIdx.x) >> 6;
    const uint32_t plane = block / a.chunks, chunk = block % a.chunks;
    if (threadIdx.x == 0) found = -1;
    int seen = 0;
    for (uint32_t u0 = 0; u0 < a.units; u0 += 256) {
        const uint32_t u = u0 + threadIdx.x;
        const bool it = u < a.units && is_dense(a, unit_entries(a, int(u)));
        const uint64_t mask = __ballot(it);
        __syncthreads();
        if (lane == 0) counts[wave] = __popcll(mask);
        __syncthreads();
        int place = seen;
        for (int w = 0; w < wave; ++w) place += counts[w];
        if (it && place + __popcll(mask & ((uint64_t(1) << lane) - 1)) == int(plane)) found = int(u);
        seen += counts[0] + counts[1] + counts[2] + counts[3];
    }
    __syncthreads();
    if (found < 0) return;
    // a token a thread: zeros, then its entries in them
    const int held = a.span * kListRows, row0 = found * held;
    const int64_t token = int64_t(chunk) * kPiece + threadIdx.x, line = a.rests.tokens * 128;
    uint8_t* to = a.dense + int64_t(plane) * (held / 64) * line + token * 128;
    const int c = token < a.n ? a.rests.count(token) : 0;
    typedef u32x4_t __attribute__((may_alias)) any_word_t;
    for (int w = 0; w < held / 8; ++w) *reinterpret_cast<any_word_t*>(to + w / 8 * line + w % 8 * 16) = any_word_t{0u, 0u, 0u, 0u};
    for (int k = 0; k < c; ++k) {
        const int r = a.rests.rows[k * a.rests.tokens + token] - row0;
        if (r < 0 || r >= held) continue;
        typedef uint16_t __attribute__((may_alias)) any_half_t;
        *reinterpret_cast<any_half_t*>(to + r / 64 * line + r % 64 * 2) = f32_to_bf16(a.rests.values[k * a.rests.tokens + token]);
    }
}

// What dx and dW need besides dz, in one launch: the rests' part of dx, x turned
// over, planes and lists.  Latency, of a list's turns: 48 us for 4096 tokens over
// 128256 x 4096, 10 for 1024 over 50257 x 768.
__global__ __launch_bounds__(256) void k_head_turn(TurnArgs t, ListArgs l, GatherArgs g) {
    uint32_t block = blockIdx.x;
    if (block < g.blocks) return gather_block(g, block);
    block -= g.blocks;
    if (block < t.blocks) return turn_block(t, block);
    block -= t.blocks;
    if (block < l.planes * l.chunks)
        dense_block(l, block);
    else
        list_block(l, block - l.planes * l.chunks);
}

// What rounding took from the large entries of dz, times x, added to the staged
// rows of the table's gradient: the wave that a row falls to (row mod 4) adds
// its entries in the list's order, so sums do not depend on timing.
template <int BT>
__device__ __forceinline__ void add_rests(const DwArgs& a, const Staging<BT>& st, int first, int end, int first_col) {
    static_assert(Staging<BT>::COLS == kListRows, "a pass is a group");
    const int lane = threadIdx.x & 63, wave = uni(int(threadIdx.x) >> 6);
    const int col = first_col + lane * 4;
    const bool holds = lane * 4 < BT && col < a.cols;
    for (int e0 = first; e0 < end; e0 += 64) {
        const uint2 mine = e0 + lane < end ? a.list[e0 + lane] : make_uint2(0u, 0u);
        uint64_t own = __ballot(e0 + lane < end && int(mine.x >> 24 & 3) == wave);
        while (own) {  // eight entries' loads on their way: text has rows with hundreds of tokens
            constexpr int N = 8;
            uint2 x[N];
            float rest[N];
            int c[N];
#pragma unroll
            for (int u = 0; u < N; ++u) {
                c[u] = -1;
                x[u] = make_uint2(0u, 0u);
                rest[u] = 0.f;
                if (own) {
                    const int from = __ffsll(static_cast<unsigned long long>(own)) - 1;
                    const uint32_t entry = __builtin_amdgcn_readlane(mine.x, from);
                    own &= own - 1;
                    const int64_t token = entry & 0xffffff;
                    c[u] = int(entry >> 24);
                    if (holds) x[u] = *reinterpret_cast<const uint2*>(a.x.at(token, col));
                    rest[u] = __uint_as_float(__builtin_amdgcn_readlane(mine.y, from));
                }
            }
#pragma unroll
            for (int u = 0; u < N; ++u)
                if (c[u] >= 0 && holds) {
                    float4& v = st.word(c[u], lane);
                    v = fma4(rest[u], make_float4(__uint_as_float(x[u].x << 16), __uint_as_float(x[u].x & 0xffff0000u),
                                                  __uint_as_float(x[u].y << 16), __uint_as_float(x[u].y & 0xffff0000u)), v);
                }
        }
    }
    stage_barrier();  // the staged rows are whole
}

// dW = dz^T x: P is x turned over, Q is dz, read K-major (its rows are the
// contraction).  Bound by the MFMAs and what the walk adds, the table's size
// read or written: 3.66 - 3.78 ms for 4096 tokens over 128256 x 4096 (1.14 - 1.18
// PFLOP/s), 101 - 118 us for 1024 over 50257 x 768, added to 77 MB of gradients.
template <int D, int BT>
__global__ __launch_bounds__(256, BT == 256 ? 1 : 2) void k_head_dw(DwArgs a) {
    using S = Shape<BT, 4>;
    __shared__ __attribute__((aligned(16))) uint8_t lds[Pipe<BT, 4>::BYTES];
    int ti, tj;
    tile_of(int(blockIdx.x), a.tp * a.tq, a.tp, a.tq, ti, tj);
    int2 bounds[Staging<BT>::PASSES] = {};
    if (a.bounds)
#pragma unroll
        for (int h = 0; h < Staging<BT>::PASSES; ++h) {
            const int g = tj * Staging<BT>::PASSES + h;
            if (g * kListRows < a.rows) bounds[h] = make_int2(uni(a.bounds[g].x), uni(a.bounds[g].y));
        }
    Operand dz = a.dz;
    const bool dense = bounds[0].x < 0;  // the tile's large entries are a plane
    if (dense) {
        dz.planes = 2;
        dz.plane = a.dense + int64_t(bounds[0].y) * (BT / 64) * dz.block - (dz.base + int64_t(tj) * (BT / 64) * dz.block);
    }
    f32x16_t acc[S::MM][S::MN];
    tile_loop<false, true, BT>(acc, a.turned, dz, int64_t(ti) * BT, int64_t(tj) * BT, 0, a.stages, lds);
    const int left = a.cols - ti * BT, under = a.rows - tj * BT;  // columns and rows from the tile's first on
    const uint32_t pitch = uint32_t(a.cols) * (D == kBF16 ? 2 : 4);  // at most 2^22
    uint8_t* to = a.grad + int64_t(tj) * BT * pitch + int64_t(ti) * BT * (D == kBF16 ? 2 : 4);
    walk_columns<BT>(
        acc, lds,
        [&](int h, const Staging<BT>& st) {
            if (a.bounds && !dense) add_rests<BT>(a, st, bounds[h].x, bounds[h].y, ti * BT);
        },
        [&](int c, int r) {
            Eight<D> old = {};
            if (a.add && c < under && r < left) old.load(to + uint32_t(c) * pitch, r, left - r, a.vector);
            return old;
        },
        [&](int c, int r, const Eight<D>& old, const Values& v) {
            if (c < under && r < left) put8<D>(to + uint32_t(c) * pitch, r, left - r, a.vector, a.add ? fma8(1.f, old.get(), v) : v);
        });
}

// Zeros in rows of `cols` elements of es bytes, `stride` elements apart: what
// an empty batch or an empty table gives.
__global__ __launch_bounds__(256) void k_head_zero(uint8_t* to, int64_t rows, int64_t cols, int64_t stride, int es) {
    const int64_t all = rows * cols;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < all; i += int64_t(gridDim.x) * 256) {
        uint8_t* p = to + (i / cols * stride + i % cols) * es;
        if (es == 2)
            *reinterpret_cast<uint16_t*>(p) = 0;
        else
            *reinterpret_cast<uint32_t*>(p) = 0;
    }
}

// ---- host side ----

hipError_t fill_zeros(uint8_t* to, int64_t rows, int64_t cols, int64_t stride, int32_t type, hipStream_t stream) {
    if (rows * cols == 0) return hipSuccess;
    const int64_t blocks = std::min<int64_t>((rows * cols + 255) / 256, 1 << 16);
    k_head_zero<<<dim3(uint32_t(blocks)), dim3(256), 0, stream>>>(to, rows, cols, stride, type == kBF16 ? 2 : 4);
    return hipGetLastError();
}

mfsdp_status hip_fail(hipError_t e, const char* what) {
    return fail(MFSDP_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

constexpr int64_t kMaxTokens = int64_t(1) << 22, kMaxFirst = int64_t(1) << 62, kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxCols = int64_t(1) << 20;         // byte offsets inside a stage stay below 2^31 (rows: a plan's 2^22)
constexpr int64_t kMaxTiles = (int64_t(1) << 32) / 256 - 1;  // a launch has fewer than 2^32 threads
constexpr int kCusHead = 256;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tile edge of a product with p x q results over `stages` of the contraction.
// Microseconds of a round: 256-tiles, one block a CU, 1.45 a stage and 10 for
// what comes before and after the loop; 128-tiles, two blocks a CU, 1.03 a
// stage, the rest hidden by the other block.  (50257 rows, 1024 tokens: 12
// stages 101 us with 256-tiles, 83 with 128; 128256 rows, 4096 tokens: 64
// stages 3270 and 4140.)
int pick_tile(int64_t p, int64_t q, int stages) {
    const int64_t large = ceil_div(p, 256) * ceil_div(q, 256), small = ceil_div(p, 128) * ceil_div(q, 128);
    return double(ceil_div(large, kCusHead)) * (1.45 * stages + 10) <= double(ceil_div(small, 2 * kCusHead)) * (1.03 * stages + 2)
               ? 256
               : 128;
}

// Tile edge of dx, and the parts its contraction over the vocabulary is cut
// into, of at least 4 stages: the least of the rounds, as above, and what the
// parts' sums cost, written and read at 4 TB/s.
struct DxCut {
    int tile, splits;
};
DxCut dx_cut(const mfsdp_entry& e, int64_t n, int runs) {
    const int64_t stages = ceil_div(e.rows, 64);
    DxCut best = {256, 1};
    double least = INFINITY;
    for (int t : {256, 128}) {
        const int64_t tiles = ceil_div(e.cols, t) * ceil_div(n, t), slots = t == 256 ? kCusHead : 2 * kCusHead;
        const int64_t most = std::clamp<int64_t>(slots / tiles, 1, std::max<int64_t>(1, stages / 4));
        for (int64_t s = 1; s <= most; ++s) {
            const double one = double(ceil_div(stages, s) * runs) * (t == 256 ? 1.45 : 1.03) + (t == 256 ? 25 : 10);
            const double us = double(ceil_div(tiles * s, slots)) * one + (s > 1 ? 5 + double(s * n * e.cols) * 8 / 4e6 : 0);
            if (us < least) {
                least = us;
                best = {t, int(s)};
            }
        }
    }
    return best;
}
// Rows of sums that dx_cut may ask for with up to n tokens: never falls as n grows.
int64_t dx_sum_rows(const mfsdp_entry& e, int64_t n) {
    const int64_t stages = ceil_div(e.rows, 64);
    int64_t rows = 0;
    for (int t : {256, 128}) {
        const int64_t across = ceil_div(e.cols, t), slots = t == 256 ? kCusHead : 2 * kCusHead;
        const int64_t most = std::min(slots / across, std::max<int64_t>(1, stages / 4));  // parts of one row of tiles
        if (most > 1) rows = std::max(rows, std::min(most * n, slots / across * t));
    }
    return rows;
}

// How a batch of n tokens is laid out and cut over one entry.
struct HeadShape {
    int x_planes, table_planes, dz_planes;
    int stages;               // 128-byte column blocks of a row of x or the table
    bool direct;              // the table is read where it lies
    int64_t np, vp;           // padded tokens and rows of the table
    bool few;
    int tile;                 // edge of the logits' tiles
    int part_rows;
    int64_t n_parts;
    int tile_dw;
    DxCut dx;
    uint64_t x, turned, table, parts, targets, logits, dz, counts, rows, values, bounds, list, dense, sums, rests, total;
    int planes;               // of large entries that there is room for
    uint64_t x_plane, table_plane, dz_plane;   // bytes of a plane (turned over: as x)
};

HeadShape head_shape(const mfsdp_entry& e, int64_t n, int x_type, int top_k, bool grad) {
    HeadShape s = {};
    if (n == 0 || e.rows == 0 || e.cols == 0) return s;
    s.x_planes = x_type == kBF16 ? 1 : 3;
    s.table_planes = e.dtype == kBF16 ? 1 : 3;
    s.dz_planes = s.x_planes + s.table_planes > 2 ? 3 : 1;
    const int64_t kp = int64_t(align_up(uint64_t(e.cols), 64));
    s.stages = int(kp / 64);
    s.direct = s.table_planes == 1 && kp == e.cols;
    s.np = int64_t(align_up(uint64_t(n), kPadTokens));
    s.vp = int64_t(align_up(uint64_t(e.rows), 256));
    s.few = !grad && n <= kFewTokens;
    const int pairs = s.x_planes * s.table_planes;
    s.tile = pick_tile(e.rows, n, s.stages * (pairs == 9 ? 6 : pairs));
    s.part_rows = s.few ? 32 : s.tile / 2;
    s.n_parts = s.few ? ceil_div(e.rows, 32) : 2 * ceil_div(e.rows, s.tile);
    uint64_t off = 0;
    auto region = [&](uint64_t bytes) {
        const uint64_t at = off;
        off = align_up(off + bytes, kAlign);
        return at;
    };
    s.x_plane = uint64_t(s.np) * uint64_t(kp) * 2;
    s.table_plane = uint64_t(e.rows) * uint64_t(kp) * 2;
    // few tokens read x and the table where they lie
    s.x = region(s.few ? 0 : uint64_t(s.x_planes) * s.x_plane);
    s.table = region(s.few || s.direct ? 0 : uint64_t(s.table_planes) * s.table_plane);
    if (grad) {
        if (s.dz_planes == 1) {
            s.counts = region((uint64_t(s.np) + uint64_t(ceil_div(e.rows, kListRows))) * 4);  // of tokens, then of groups
            s.rows = region(uint64_t(s.np) * kMaxRests * 4);
            s.values = region(uint64_t(s.np) * kMaxRests * 4);
            s.bounds = region(uint64_t(ceil_div(e.rows, kListRows)) * 8);
            s.list = region(uint64_t(s.np) * kMaxRests * 8);
            // room for either tile edge of dW
            s.dense = region(uint64_t(std::min<int64_t>(kMostPlanes * 256, s.vp)) * uint64_t(s.np) * 2);
            s.rests = region(uint64_t(n) * align_up(uint64_t(e.cols), 8) * 4);
        }
        s.turned = region(uint64_t(s.x_planes) * s.x_plane);
        s.dz_plane = uint64_t(s.np) * uint64_t(s.vp) * 2;
        s.dz = region(uint64_t(s.dz_planes) * s.dz_plane);
        const int of_dx = s.dz_planes * s.table_planes, of_dw = s.dz_planes * s.x_planes;
        s.dx = dx_cut(e, n, of_dx == 9 ? 6 : of_dx);
        s.tile_dw = pick_tile(e.rows, e.cols, int(ceil_div(n, 64)) * (of_dw == 9 ? 6 : of_dw));
        s.planes = s.dz_planes == 1 ? int(std::min<int64_t>(kMostPlanes, ceil_div(e.rows, s.tile_dw))) : 0;
        s.sums = region(uint64_t(dx_sum_rows(e, n)) * align_up(uint64_t(e.cols), 8) * 4);
    } else {
        s.targets = region(uint64_t(s.np) * 4);
        // the most that either edge, or a smaller batch in another form, needs
        s.parts = region(16 * std::max(uint64_t(2 * ceil_div(e.rows, 128)) * uint64_t(n),
                                       uint64_t(ceil_div(e.rows, 32)) * uint64_t(std::min(n, kFewTokens))));
        s.logits = region(top_k > 0 ? uint64_t(n) * uint64_t(s.vp) * 4 : 0);
    }
    s.total = off;
    return s;
}

mfsdp_status check_common(mfsdp_plan_t plan, int64_t entry, int64_t n, int32_t x_type, int32_t top_k) {
    if (entry < 0 || entry >= int64_t(plan->entries.size()))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "entry index out of range");
    if (x_type != MFSDP_F32 && x_type != MFSDP_BF16)
        return fail(MFSDP_ERR_UNSUPPORTED, "x must be MFSDP_F32 or MFSDP_BF16");
    if (n < 0 || n > kMaxTokens) return fail(MFSDP_ERR_INVALID_ARGUMENT, "n must be in 0..2^22");
    if (top_k < 0 || top_k > kMaxTop) return fail(MFSDP_ERR_INVALID_ARGUMENT, "top_k must be in 0..64");
    const mfsdp_entry& e = plan->entries[size_t(entry)];
    if (e.cols > kMaxCols) return fail(MFSDP_ERR_UNSUPPORTED, "a table of more than 2^20 columns");
    if (ceil_div(e.rows, 128) * ceil_div(n, 128) > kMaxTiles || ceil_div(e.rows, 128) * ceil_div(e.cols, 128) > kMaxTiles)
        return fail(MFSDP_ERR_UNSUPPORTED, "more than 2^24 - 1 tiles of 128 x 128 logits or table elements: cut the batch or the table");
    // k_head_turn's blocks
    if (ceil_div(e.cols, 64) * ceil_div(n, kPadTokens) * (kPadTokens / 64) * 3 + ceil_div(e.rows, kListRows) + 1 > kMaxTiles)
        return fail(MFSDP_ERR_UNSUPPORTED, "more than a third of 2^24 tiles of 64 x 64 elements of x: cut the batch");
    return MFSDP_OK;
}

mfsdp_status check_batch(const mfsdp_entry& e, const void* params, const void* x, int64_t n, int32_t x_type,
                         int64_t* stride, const void* ids, int32_t id_type, int64_t first_id, float scale) {
    if (id_type != MFSDP_I32 && id_type != MFSDP_I64)
        return fail(MFSDP_ERR_UNSUPPORTED, "id_type must be MFSDP_I32 or MFSDP_I64");
    if (first_id < 0 || first_id > kMaxFirst) return fail(MFSDP_ERR_INVALID_ARGUMENT, "first_id must be in 0..2^62");
    if (!std::isfinite(scale)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "scale is not finite");
    if (*stride == 0) *stride = e.cols;
    if (*stride < e.cols || *stride > kMaxStride) return fail(MFSDP_ERR_INVALID_ARGUMENT, "row stride below cols or above 2^40");
    if (!params || misaligned(params, 16)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "params is NULL or not 16-byte aligned");
    if (n > 0) {
        if (!x || misaligned(x, x_type == MFSDP_BF16 ? 2 : 4)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "x is NULL or misaligned");
        if (ids && misaligned(ids, id_type == MFSDP_I64 ? 8 : 4)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "ids is misaligned");
    }
    return MFSDP_OK;
}

mfsdp_status check_space(const void* workspace, uint64_t have, uint64_t need) {
    if (need == 0) return MFSDP_OK;
    if (!workspace || misaligned(workspace, kAlign))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "workspace is NULL or not 256-byte aligned");
    if (have < need)
        return fail(MFSDP_ERR_WORKSPACE_TOO_SMALL,
                    "workspace has " + std::to_string(have) + " bytes, the call needs " + std::to_string(need));
    return MFSDP_OK;
}

// a launch has fewer than 2^32 threads: whole rows each
constexpr int64_t kMostWords = ((int64_t(1) << 32) / kPackThreads - 2) * kPackThreads;

void launch_pack(const PackArgs& a, int a_type, const PackArgs& b, int b_type, hipStream_t stream) {
    const uint32_t second = uint32_t(ceil_div(a.words, kPackThreads));
    const dim3 grid(second + uint32_t(ceil_div(b.words, kPackThreads))), block(kPackThreads);
    if (a_type == kBF16)
        b_type == kBF16 ? k_head_pack<kBF16, kBF16><<<grid, block, 0, stream>>>(a, b, second)
                        : k_head_pack<kBF16, kF32><<<grid, block, 0, stream>>>(a, b, second);
    else
        b_type == kBF16 ? k_head_pack<kF32, kBF16><<<grid, block, 0, stream>>>(a, b, second)
                        : k_head_pack<kF32, kF32><<<grid, block, 0, stream>>>(a, b, second);
}

// A matrix of any size, by launches of whole rows.
void launch_pack(const PackArgs& a, int type, hipStream_t stream) {
    const int64_t per_row = a.per_row, chunk = kMostWords / per_row * per_row;
    for (int64_t w = 0; w < a.words; w += chunk) {
        PackArgs b = a;
        const int64_t row = w / per_row;
        b.words = std::min(chunk, a.words - w);
        b.src = a.src + row * a.stride * (type == kBF16 ? 2 : 4);
        b.dst = a.dst + row * 128;
        b.rows = std::max<int64_t>(0, a.rows - row);
        if (a.ids.ids) b.ids.ids = static_cast<const uint8_t*>(a.ids.ids) + row * (a.ids.type == MFSDP_I64 ? 8 : 4);
        if (w > 0) b.n_zeros = 0;
        launch_pack(b, type, PackArgs{}, type, stream);
    }
}

struct Batch {
    const uint8_t* table;   // the entry's first element
    const void* x;
    int64_t n, stride;
    int x_type;
    Ids ids;
    float scale;
    uint8_t* ws;
    hipStream_t stream;
};

LogitArgs logit_args(const mfsdp_entry& e, const HeadShape& s, const Batch& b) {
    LogitArgs a = {};
    a.rows = int(e.rows);
    a.n = b.n;
    a.stages = s.stages;
    a.tp = int(ceil_div(e.rows, s.tile));
    a.tq = int(ceil_div(b.n, s.tile));
    a.c2 = float(double(b.scale) * 1.44269504088896340736);
    a.ids = b.ids;
    return a;
}

// The batch, and a table that cannot be read in place, in the tile loop's
// layout, and n_zeros words of zeros.
void pack_operands(const mfsdp_entry& e, const HeadShape& s, const Batch& b, int* zeros, int64_t n_zeros, LogitArgs& a) {
    PackArgs p = {};
    p.src = static_cast<const uint8_t*>(b.x);
    p.dst = b.ws + s.x;
    p.stride = b.stride;
    p.rows = b.n;
    p.block = s.np * 128;
    p.plane = int64_t(s.x_plane);
    p.per_row = s.stages * 8;
    p.words = s.np * p.per_row;
    p.cols = int(e.cols);
    p.ids = b.ids;
    p.table_rows = int(e.rows);
    p.zeros = zeros;
    p.n_zeros = n_zeros;
    const PackArgs x = p;
    a.x = Operand{p.dst, 128, p.block, s.np, s.stages, s.x_planes, p.plane};
    a.table = Operand{b.table, e.cols * 2, 128, e.rows, s.stages, 1, 0};
    if (s.direct) return launch_pack(x, b.x_type, b.stream);
    p.src = b.table;
    p.dst = b.ws + s.table;
    p.stride = e.cols;
    p.rows = e.rows;
    p.block = e.rows * 128;
    p.plane = int64_t(s.table_plane);
    p.words = e.rows * p.per_row;
    p.ids = Ids{};
    p.n_zeros = 0;
    if (x.words + p.words <= kMostWords) {
        launch_pack(x, b.x_type, p, e.dtype, b.stream);
    } else {
        launch_pack(x, b.x_type, b.stream);
        launch_pack(p, e.dtype, b.stream);
    }
    a.table = Operand{p.dst, 128, p.block, e.rows, s.stages, s.table_planes, p.plane};
}

template <int WD, int XD> void launch_few(const FewArgs& f, hipStream_t stream) {
    // Rows of a block: 64 where that leaves two blocks a CU, since x is then read half as often; for more than 32 tokens
    // 32, as measured (60 tokens over 50000 x 1000: 60 us, 66 with 64 rows; over 50000 x 1001 fp32 129 and 145; 40 over
    // 128256 x 1001 179 and 174).  Registers leave two blocks a CU either way.
    const bool two = f.l.n <= 32 && f.l.rows >= 64 * 2 * kCusHead;
    const dim3 grid(uint32_t(ceil_div(f.l.rows, two ? 64 : 32)));
    if (f.l.n > 32)
        k_head_few<WD, XD, 1, 2><<<grid, dim3(256), 0, stream>>>(f);
    else if (two)
        k_head_few<WD, XD, 2, 1><<<grid, dim3(256), 0, stream>>>(f);
    else
        k_head_few<WD, XD, 1, 1><<<grid, dim3(256), 0, stream>>>(f);
}

// Rows of a block of k_head_stream: 128 where that leaves three blocks a CU.
void launch_stream(const FewArgs& f, hipStream_t stream) {
    const bool large = f.l.rows >= 128 * 3 * kCusHead;
    const dim3 grid(uint32_t(ceil_div(f.l.rows, large ? 128 : 64))), block(large ? 256 : 128);
    if (f.l.n <= 32)
        large ? k_head_stream<4, 1><<<grid, block, 0, stream>>>(f) : k_head_stream<2, 1><<<grid, block, 0, stream>>>(f);
    else
        large ? k_head_stream<4, 2><<<grid, block, 0, stream>>>(f) : k_head_stream<2, 2><<<grid, block, 0, stream>>>(f);
}

hipError_t launch_logprob(const mfsdp_entry& e, const HeadShape& s, const Batch& b, RowArgs r) {
    LogitArgs a = logit_args(e, s, b);
    a.parts = reinterpret_cast<float4*>(b.ws + s.parts);
    a.targets = reinterpret_cast<float*>(b.ws + s.targets);
    a.logits = r.top_k > 0 ? reinterpret_cast<float*>(b.ws + s.logits) : nullptr;
    if (s.few) {
        const int xs = b.x_type == kBF16 ? 2 : 4, es = e.dtype == kBF16 ? 2 : 4;
        const FewArgs f = {a, b.table, static_cast<const uint8_t*>(b.x), b.stride * xs, e.cols * es, int(e.cols)};
        const bool lines = s.direct && xs == 2 && !misaligned(b.x, 16) && b.stride % 8 == 0;
        if (lines && (b.n > 32 || e.rows * e.cols * es <= kCacheBytes))
            launch_stream(f, b.stream);
        else if (e.dtype == kBF16)
            b.x_type == kBF16 ? launch_few<kBF16, kBF16>(f, b.stream) : launch_few<kBF16, kF32>(f, b.stream);
        else
            b.x_type == kBF16 ? launch_few<kF32, kBF16>(f, b.stream) : launch_few<kF32, kF32>(f, b.stream);
    } else {
        pack_operands(e, s, b, nullptr, 0, a);
        const dim3 grid(uint32_t(a.tp) * uint32_t(a.tq));
        if (s.tile == 256)
            k_head_logits<256><<<grid, dim3(256), 0, b.stream>>>(a);
        else
            k_head_logits<128><<<grid, dim3(256), 0, b.stream>>>(a);
    }
    r.parts = a.parts;
    r.targets = a.targets;
    r.logits = a.logits;
    r.n_parts = int(s.n_parts);
    r.part_rows = s.part_rows;
    // A block a token for few tokens, and up to 1024 with alternatives, which one wave finds in series (20 of
    // 9291 rows: 182 tokens 13.8 us by blocks, 45 by waves).
    if (s.few || (r.top_k > 0 && b.n <= 4 * kCusHead))
        k_head_few_rows<<<dim3(uint32_t(b.n)), dim3(64 * kRowWaves), 0, b.stream>>>(r);
    else
        k_head_rows<<<dim3(uint32_t(ceil_div(b.n, kRowsBlock))), dim3(64 * kRowsBlock), 0, b.stream>>>(r);
    return hipGetLastError();
}

struct GradOut {
    const mfsdp_head_record* records;
    const float *dlogp, *dentropy;
    uint8_t* dx;
    int64_t dx_stride;
    uint8_t* grad;      // the entry's gradient
    int add;
};

template <int D> void launch_dx(const DxArgs& a, int tile, hipStream_t stream) {
    const uint32_t blocks = uint32_t(a.tp) * uint32_t(a.tq) * uint32_t(a.splits);
    const dim3 grid(a.splits > 1 ? uint32_t(align_up(blocks, 8)) : blocks);
    if (tile == 256)
        k_head_dx<D, 256><<<grid, dim3(256), 0, stream>>>(a);
    else
        k_head_dx<D, 128><<<grid, dim3(256), 0, stream>>>(a);
    const int64_t words = a.n * (a.ld / 8);
    if (a.splits >= 16)  // fewer are all on their way at once
        k_head_dx_sum<D, 8><<<dim3(uint32_t(ceil_div(words, 32))), dim3(256), 0, stream>>>(a);
    else if (a.splits > 1)
        k_head_dx_sum<D, 1><<<dim3(uint32_t(ceil_div(words, 256))), dim3(256), 0, stream>>>(a);
}

template <int D> void launch_dw(const DwArgs& a, int tile, hipStream_t stream) {
    const dim3 grid(uint32_t(a.tp) * uint32_t(a.tq));
    if (tile == 256)
        k_head_dw<D, 256><<<grid, dim3(256), 0, stream>>>(a);
    else
        k_head_dw<D, 128><<<grid, dim3(256), 0, stream>>>(a);
}

hipError_t launch_grad(const mfsdp_entry& e, const HeadShape& s, const Batch& b, const GradOut& g) {
    const bool kept = s.dz_planes == 1;  // what rounding takes from large entries
    const int64_t ld = int64_t(align_up(uint64_t(e.cols), 8));
    const int64_t groups = kept ? ceil_div(e.rows, kListRows) : 0;
    Rests rests = {};
    if (kept) {
        int* counts = reinterpret_cast<int*>(b.ws + s.counts);
        rests = Rests{counts, counts + s.np, reinterpret_cast<int*>(b.ws + s.rows), reinterpret_cast<float*>(b.ws + s.values), s.np};
    }
    DzArgs d = {};
    d.l = logit_args(e, s, b);
    pack_operands(e, s, b, rests.counts, kept ? s.np + groups : 0, d.l);
    d.records = g.records;
    d.dlogp = g.dlogp;
    d.dentropy = g.dentropy;
    d.scale = b.scale;
    d.dz = b.ws + s.dz;
    d.block = s.np * 128;
    d.planes = s.dz_planes;
    d.plane = int64_t(s.dz_plane);
    d.rests = rests;
    const dim3 grid(uint32_t(d.l.tp) * uint32_t(d.l.tq));
    if (s.tile == 256)
        k_head_dz<256><<<grid, dim3(256), 0, b.stream>>>(d);
    else
        k_head_dz<128><<<grid, dim3(256), 0, b.stream>>>(d);
    // tokens and vocabulary rows that dz was written for
    const Operand dz = {d.dz, 128, d.block, int64_t(d.l.tq) * s.tile, d.l.tp * (s.tile / 64), s.dz_planes, d.plane};
    TurnArgs t = {};
    ListArgs l = {};
    GatherArgs of_dx = {};
    int64_t blocks = 0;  // of x turned over, lists, pieces of planes
    if (g.grad) {
        const int64_t kp = int64_t(s.stages) * 64;
        const uint32_t across = uint32_t(s.np / 64);
        t = TurnArgs{d.l.x.base, b.ws + s.turned, d.l.x.block, kp * 128, d.l.x.plane, d.l.x.plane,
                     across, uint32_t(s.stages), across * uint32_t(s.stages) * uint32_t(s.x_planes)};
        if (kept)
            l = ListArgs{rests, int(b.n), int(e.rows), s.tile_dw / kListRows, int(s.np) * kMaxRests,
                         reinterpret_cast<int2*>(b.ws + s.bounds), reinterpret_cast<uint2*>(b.ws + s.list), b.ws + s.dense,
                         uint32_t(ceil_div(e.rows, s.tile_dw)), uint32_t(s.planes), uint32_t(s.np / kPiece)};
        blocks = int64_t(t.blocks) + groups + int64_t(l.planes) * l.chunks;
    }
    if (g.dx && kept)
        of_dx = GatherArgs{rests, d.l.table, b.n, ld, reinterpret_cast<float*>(b.ws + s.rests), uint32_t(ceil_div(b.n, 4))};
    blocks += of_dx.blocks;  // with one plane of x a third of 2^24 at most, 2^15, 2^21 and 2^20
    if (blocks > 0) k_head_turn<<<dim3(uint32_t(blocks)), dim3(256), 0, b.stream>>>(t, l, of_dx);
    if (g.dx) {
        DxArgs a = {};
        const int tile = s.dx.tile, xs = b.x_type == kBF16 ? 2 : 4;
        a.table = d.l.table;
        a.dz = dz;
        a.n = b.n;
        a.cols = int(e.cols);
        a.rows = int(e.rows);
        a.tp = int(ceil_div(e.cols, tile));
        a.tq = int(ceil_div(b.n, tile));
        a.stages = int(ceil_div(e.rows, 64));
        a.splits = s.dx.splits;
        a.ids = b.ids;
        a.rests = kept ? reinterpret_cast<const float*>(b.ws + s.rests) : nullptr;
        a.dx = g.dx;
        a.stride = g.dx_stride;
        a.vector = !misaligned(g.dx, 16) && g.dx_stride * xs % 16 == 0;
        a.sums = reinterpret_cast<float*>(b.ws + s.sums);
        a.ld = ld;
        b.x_type == kBF16 ? launch_dx<kBF16>(a, tile, b.stream) : launch_dx<kF32>(a, tile, b.stream);
    }
    if (g.grad) {
        DwArgs a = {};
        a.turned = Operand{t.dst, 128, t.dst_block, int64_t(s.stages) * 64, int(s.np / 64), s.x_planes, t.dst_plane};
        a.x = d.l.x;
        a.dz = dz;
        a.n = b.n;
        a.rows = int(e.rows);
        a.cols = int(e.cols);
        a.tp = int(ceil_div(e.cols, s.tile_dw));
        a.tq = int(ceil_div(e.rows, s.tile_dw));
        a.stages = int(ceil_div(b.n, 64));
        a.bounds = kept ? l.bounds : nullptr;
        a.list = l.list;
        a.dense = l.dense;
        a.grad = g.grad;
        a.vector = e.cols * (e.dtype == kBF16 ? 2 : 4) % 16 == 0;  // the entry is 16-byte aligned
        a.add = g.add;
        e.dtype == kBF16 ? launch_dw<kBF16>(a, s.tile_dw, b.stream) : launch_dw<kF32>(a, s.tile_dw, b.stream);
    }
    return hipGetLastError();
}

}  // namespace
}  // namespace mfsdp

using namespace mfsdp;

extern "C" mfsdp_status mfsdp_plan_head_workspace_bytes(mfsdp_plan_t plan, int64_t entry, int64_t n, int32_t x_type,
                                                        int32_t top_k, int32_t grad, uint64_t* bytes) {
    clear_error();
    if (!plan || !bytes) return fail(MFSDP_ERR_INVALID_ARGUMENT, "NULL argument");
    if (mfsdp_status st = check_common(plan, entry, n, x_type, top_k); st != MFSDP_OK) return st;
    if (grad != 0 && grad != 1) return fail(MFSDP_ERR_INVALID_ARGUMENT, "grad must be 0 or 1");
    const mfsdp_entry& e = plan->entries[size_t(entry)];
    // one workspace serves the call forward too
    uint64_t most = head_shape(e, n, x_type, top_k, false).total;
    if (grad) most = std::max(most, head_shape(e, n, x_type, 0, true).total);
    *bytes = most;
    return MFSDP_OK;
}

extern "C" mfsdp_status mfsdp_head_logprob(mfsdp_plan_t plan, int64_t entry, const mfsdp_head_logprob_args* args) {
    clear_error();
    if (!plan || !args) return fail(MFSDP_ERR_INVALID_ARGUMENT, "NULL plan or args");
    if (mfsdp_status st = check_common(plan, entry, args->n, args->x_type, args->top_k); st != MFSDP_OK) return st;
    const mfsdp_entry& e = plan->entries[size_t(entry)];
    int64_t stride = args->x_stride;
    if (mfsdp_status st = check_batch(e, args->params, args->x, args->n, args->x_type, &stride, args->ids, args->id_type,
                                      args->first_id, args->scale);
        st != MFSDP_OK)
        return st;
    if (args->n == 0) return MFSDP_OK;
    if (!args->records || misaligned(args->records, 8))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "records is NULL or not 8-byte aligned");
    if (misaligned(args->logp, 4) || misaligned(args->entropy, 4) || misaligned(args->top_logp, 4) ||
        misaligned(args->top_logits, 4) || misaligned(args->top_ids, 8))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "an output is misaligned");
    if (args->top_k > 0 && !args->top_ids) return fail(MFSDP_ERR_INVALID_ARGUMENT, "top_ids is NULL");
    const HeadShape s = head_shape(e, args->n, args->x_type, args->top_k, false);
    if (mfsdp_status st = check_space(args->workspace, args->workspace_bytes, s.total); st != MFSDP_OK) return st;
    RowArgs r = {};
    r.n = args->n;
    r.rows = int(e.rows);
    r.ids = Ids{args->ids, args->first_id, args->id_type};
    r.first_id = args->first_id;
    r.records = args->records;
    r.logp = args->logp;
    r.entropy = args->entropy;
    r.top_k = args->top_k;
    r.top_ids = args->top_ids;
    r.top_logp = args->top_logp;
    r.top_logits = args->top_logits;
    hipStream_t stream = static_cast<hipStream_t>(args->stream);
    hipError_t err;
    if (e.rows == 0 || e.cols == 0) {
        k_head_empty<<<dim3(uint32_t(ceil_div(args->n, 256))), dim3(256), 0, stream>>>(r);
        err = hipGetLastError();
    } else {
        const Batch b = {static_cast<const uint8_t*>(args->params) + e.offset, args->x, args->n, stride, args->x_type, r.ids,
                         args->scale, static_cast<uint8_t*>(args->workspace), stream};
        err = launch_logprob(e, s, b, r);
    }
    if (err != hipSuccess) return hip_fail(err, "log probability launch");
    return MFSDP_OK;
}

extern "C" mfsdp_status mfsdp_head_total(const mfsdp_head_total_args* args) {
    clear_error();
    if (!args) return fail(MFSDP_ERR_INVALID_ARGUMENT, "NULL args");
    if (args->count < 1 || args->count > 65536) return fail(MFSDP_ERR_INVALID_ARGUMENT, "count must be in 1..65536");
    if (args->n < 0 || args->n > kMaxTokens) return fail(MFSDP_ERR_INVALID_ARGUMENT, "n must be in 0..2^22");
    if (args->top_k < 0 || args->top_k > kMaxTop) return fail(MFSDP_ERR_INVALID_ARGUMENT, "top_k must be in 0..64");
    if (args->n == 0) return MFSDP_OK;
    if (!args->parts || misaligned(args->parts, 8) || !args->records || misaligned(args->records, 8))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "parts or records is NULL or not 8-byte aligned");
    if (misaligned(args->logp, 4) || misaligned(args->entropy, 4) || misaligned(args->top_logp, 4) ||
        misaligned(args->top_logits, 4) || misaligned(args->top_ids, 8) || misaligned(args->part_top_ids, 8) ||
        misaligned(args->part_top_logits, 4))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "a buffer is misaligned");
    if (args->top_k > 0 && (!args->top_ids || !args->part_top_ids || !args->part_top_logits))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "top_ids, part_top_ids or part_top_logits is NULL");
    TotalArgs a = {};
    a.parts = args->parts;
    a.count = int(args->count);
    a.n = args->n;
    a.records = args->records;
    a.logp = args->logp;
    a.entropy = args->entropy;
    a.top_k = args->top_k;
    a.part_ids = args->part_top_ids;
    a.part_logits = args->part_top_logits;
    a.top_ids = args->top_ids;
    a.top_logp = args->top_logp;
    a.top_logits = args->top_logits;
    k_head_total<<<dim3(uint32_t(ceil_div(a.n, 4))), dim3(256), 0, static_cast<hipStream_t>(args->stream)>>>(a);
    if (hipError_t err = hipGetLastError(); err != hipSuccess) return hip_fail(err, "head total launch");
    return MFSDP_OK;
}

extern "C" mfsdp_status mfsdp_head_grad(mfsdp_plan_t plan, int64_t entry, const mfsdp_head_grad_args* args) {
    clear_error();
    if (!plan || !args) return fail(MFSDP_ERR_INVALID_ARGUMENT, "NULL plan or args");
    if (mfsdp_status st = check_common(plan, entry, args->n, args->x_type, 0); st != MFSDP_OK) return st;
    const mfsdp_entry& e = plan->entries[size_t(entry)];
    int64_t stride = args->x_stride, dx_stride = args->dx_stride == 0 ? e.cols : args->dx_stride;
    if (mfsdp_status st = check_batch(e, args->params, args->x, args->n, args->x_type, &stride, args->ids, args->id_type,
                                      args->first_id, args->scale);
        st != MFSDP_OK)
        return st;
    if (args->accumulate != 0 && args->accumulate != 1)
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "accumulate must be 0 or 1");
    if (dx_stride < e.cols || dx_stride > kMaxStride)
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "dx row stride below cols or above 2^40");
    if (misaligned(args->grads, 16)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "grads is not 16-byte aligned");
    if (misaligned(args->dx, args->x_type == MFSDP_BF16 ? 2 : 4)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "dx is misaligned");
    if (args->n > 0) {
        if (!args->records || misaligned(args->records, 8))
            return fail(MFSDP_ERR_INVALID_ARGUMENT, "records is NULL or not 8-byte aligned");
        if (!args->dlogp || misaligned(args->dlogp, 4) || misaligned(args->dentropy, 4))
            return fail(MFSDP_ERR_INVALID_ARGUMENT, "dlogp is NULL, or dlogp or dentropy misaligned");
    }
    hipStream_t stream = static_cast<hipStream_t>(args->stream);
    uint8_t* grad = args->grads ? static_cast<uint8_t*>(args->grads) + e.offset : nullptr;
    const HeadShape s = head_shape(e, args->n, args->x_type, 0, true);
    if (mfsdp_status st = check_space(args->workspace, args->workspace_bytes, s.total); st != MFSDP_OK) return st;
    hipError_t err = hipSuccess;
    if (e.cols == 0 || (args->n == 0 && (e.rows == 0 || args->accumulate || !grad))) return MFSDP_OK;
    if (args->n == 0) {
        err = fill_zeros(grad, e.rows, e.cols, e.cols, e.dtype, stream);
    } else if (e.rows == 0) {
        if (args->dx) err = fill_zeros(static_cast<uint8_t*>(args->dx), args->n, e.cols, dx_stride, args->x_type, stream);
    } else {
        const Batch b = {static_cast<const uint8_t*>(args->params) + e.offset, args->x, args->n, stride, args->x_type,
                         Ids{args->ids, args->first_id, args->id_type}, args->scale, static_cast<uint8_t*>(args->workspace),
                         stream};
        const GradOut g = {args->records, args->dlogp, args->dentropy, static_cast<uint8_t*>(args->dx), dx_stride, grad,
                           args->accumulate};
        err = launch_grad(e, s, b, g);
    }
    if (err != hipSuccess) return hip_fail(err, "head gradient launch");
    return MFSDP_OK;
}
