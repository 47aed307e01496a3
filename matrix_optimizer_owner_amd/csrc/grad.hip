// grad.hip - the global gradient norm over every tensor of an owner buffer,
// and clipping, on gfx950.
//
//   sumsq = sum g^2;  norm = sqrt(sumsq);  scale = min(1, max_norm/(norm+eps));
//   out <- RNE(scale * g).
//
// Both passes are bound by HBM: the norm reads each gradient once, clipping
// reads and writes it once.  The host cuts the table into runs of one tensor
// each (grad_layout.h), so a launch covers every tensor whatever its size.
#include <algorithm>
#include <cmath>
#include <string>

#include "device_util.h"
#include "plan_internal.h"

namespace mfsdp {
namespace {

constexpr int kNormThreads = 512, kNormUnroll = 8;
constexpr int kNormWaves = kNormThreads / 64;
constexpr int kClipThreads = int(kGradSlice / 16);
constexpr int64_t kClipBlocksMax = (int64_t(1) << 23) - 1;  // a launch holds fewer than 2^32 threads

// Adds the squares of one 16-byte word, in fp64: gradients over the whole range
// of their type neither overflow nor vanish, and the conversions and FMAs
// hide behind the loads (a 1.7 GB read takes 281 us with them, 280 with fp32).
template <int DT> __device__ __forceinline__ void add_squares(u32x4_t w, double (&s)[2]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (DT == kBF16) {
            const double lo = double(__uint_as_float(w[k] << 16)), hi = double(__uint_as_float(w[k] & 0xffff0000u));
            s[0] = __builtin_fma(lo, lo, s[0]);
            s[1] = __builtin_fma(hi, hi, s[1]);
        } else {
            const double v = double(__uint_as_float(w[k]));
            s[k & 1] = __builtin_fma(v, v, s[k & 1]);
        }
    }
}

// Sum over the norm's block in a fixed order; the result is valid in thread 0.
__device__ __forceinline__ double block_sum(double v, double* red) {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0)
        for (int k = 0; k < kNormWaves; ++k) t += red[k];
    __syncthreads();
    return t;
}

// One thread's share of a run's sum of squares, added to s: batches of kNormUnroll
// independent 16-byte loads, past the caches (nothing here is read twice:
// 1.7 GB take 251 us with nontemporal loads and 281 with plain ones).
template <int DT> __device__ __forceinline__ void run_squares(const uint8_t* p, uint64_t numel, double (&s)[2]) {
    constexpr uint32_t PER = DT == kBF16 ? 8 : 4;
    constexpr uint64_t BATCH = kNormThreads * kNormUnroll;
    const uint64_t words = numel / PER;
    const u32x4_t* q = reinterpret_cast<const u32x4_t*>(p) + threadIdx.x;
    const u32x4_t* const full = q + words / BATCH * BATCH;
    for (; q != full; q += BATCH) {
        u32x4_t w[kNormUnroll];
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) w[u] = __builtin_nontemporal_load(q + u * kNormThreads);
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) add_squares<DT>(w[u], s);
    }
    const uint32_t left = uint32_t(words % BATCH);
    if (left > 0) {
        u32x4_t w[kNormUnroll];
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) {
            w[u] = u32x4_t{0u, 0u, 0u, 0u};
            if (threadIdx.x + u * kNormThreads < left) w[u] = __builtin_nontemporal_load(q + u * kNormThreads);
        }
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) add_squares<DT>(w[u], s);
    }
    const uint64_t i = words * PER + threadIdx.x;
    if (i < numel) {
        const double v = double(load_elem(p, DT, int64_t(i)));
        s[0] = __builtin_fma(v, v, s[0]);
    }
}

__device__ __forceinline__ void write_stats(mfsdp_grad_stats* out, double sumsq, double max_norm, double eps) {
    const double norm = sqrt(sumsq);
    const double f = max_norm / (norm + eps);
    out->sumsq = sumsq;
    out->norm = float(norm);
    // a NaN norm gives a NaN scale; an infinite max_norm never scales
    out->scale = isinf(max_norm) || f >= 1.0 ? 1.f : float(f);
}

// A piece's partial sum, written by one block and read by another of the same
// launch, possibly on another XCD: device-scope accesses on both sides, which
// go through to memory.  The writer waits for its stores before it counts
// itself as finished, so the block that sees the full count sees them all.
// (A release and an acquire at device scope would order them too, but write
// back and invalidate the XCD's whole L2 in each of 1024 blocks: 20 us on the
// 1.7 GB share, 14 us on a 7 MB table.)
__device__ __forceinline__ void put_partial(double* p, double v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double get_partial(const double* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Whether this is the last block of the launch to get here.  The counters are 0
// before and after.  With more than kNormGroups * 2 blocks they count in
// groups first: balanced blocks finish together, and 1022 of them on one
// counter took 24 us of the 1.7 GB share's 277.
__device__ __forceinline__ bool last_to_finish(uint32_t* counters) {
    const uint32_t n = gridDim.x, g = blockIdx.x % kNormGroups;
    auto count = [&](uint32_t* c, uint32_t of) {
        const bool full = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == of - 1;
        if (full) __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        return full;
    };
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this thread's partial sums are in memory
    if (n <= kNormGroups * 2) return count(counters, n);
    return count(counters + (1 + g) * kNormCounterPitch, (n - g + kNormGroups - 1) / kNormGroups) &&
           count(counters, kNormGroups);
}

struct NormArgs {
    const NormBlock* blocks;
    const GradRun* pieces;
    const int32_t *entry_begin, *large;
    const uint8_t* grads;
    double* partials;
    uint32_t* counters;
    float* entry_norms;  // or NULL
    mfsdp_grad_stats* stats;
    double max_norm, eps;
    int n_pieces, n_entries, n_large;
};

// The norm in one launch: every block sums its pieces, and the block that
// finishes last adds the partial sums, always in the same order whichever
// block that is.  One launch instead of two saves about 3 us, a third of the
// time of a small table.
__global__ __launch_bounds__(kNormThreads) void k_grad_norm(NormArgs a) {
    __shared__ double red[kNormWaves];
    __shared__ bool last;
    const NormBlock b = a.blocks[blockIdx.x];
    GradRun r = b.first;
    for (int p = b.begin; p < b.end; ++p) {
        GradRun next = r;
        if (p + 1 < b.end) next = a.pieces[p + 1];
        double s[2] = {0.0, 0.0};
        if (r.dtype == kBF16)
            run_squares<kBF16>(a.grads + r.off, r.numel, s);
        else
            run_squares<kF32>(a.grads + r.off, r.numel, s);
        const double sum = block_sum(s[0] + s[1], red);
        if (threadIdx.x == 0) put_partial(a.partials + p, sum);
        r = next;
    }
    if (threadIdx.x == 0) last = last_to_finish(a.counters);
    __syncthreads();
    if (!last) return;

    // an entry of at most kNormFew pieces is one thread's; the first 512 start on their way before the total's sum
    auto small_entry = [&](int e, int b0, int b1) {
        if (e >= a.n_entries || b1 - b0 > kNormFew) return;
        double v[kNormFew], t = 0.0;
#pragma unroll
        for (int k = 0; k < kNormFew; ++k) v[k] = b0 + k < b1 ? get_partial(a.partials + b0 + k) : 0.0;
#pragma unroll
        for (int k = 0; k < kNormFew; ++k) t += v[k];
        a.entry_norms[e] = float(sqrt(t));
    };
    const int e0 = threadIdx.x;
    const bool mine = a.entry_norms && e0 < a.n_entries;
    const int b0 = mine ? a.entry_begin[e0] : 0, b1 = mine ? a.entry_begin[e0 + 1] : 0;
    double s = 0.0;
    for (int i = threadIdx.x; i < a.n_pieces; i += kNormThreads * kNormUnroll) {
        double v[kNormUnroll];
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u)
            v[u] = i + u * kNormThreads < a.n_pieces ? get_partial(a.partials + i + u * kNormThreads) : 0.0;
#pragma unroll
        for (int u = 0; u < kNormUnroll; ++u) s += v[u];
    }
    if (mine) small_entry(e0, b0, b1);
    s = block_sum(s, red);
    if (threadIdx.x == 0) write_stats(a.stats, s, a.max_norm, a.eps);
    if (!a.entry_norms) return;
    for (int e = e0 + kNormThreads; e < a.n_entries; e += kNormThreads) small_entry(e, a.entry_begin[e], a.entry_begin[e + 1]);
    // one of more is 16 lanes', 32 entries at a time (a wave for each took 35
    // us for the 28 matrices of the 1.7 GB share)
    const int lane = int(threadIdx.x & 15);
    for (int k = int(threadIdx.x >> 4); k < a.n_large; k += kNormThreads / 16) {
        const int e = a.large[k], b1 = a.entry_begin[e + 1];
        double t = 0.0;
        for (int i = a.entry_begin[e] + lane; i < b1; i += 16 * kNormFew) {
            double v[kNormFew];
#pragma unroll
            for (int u = 0; u < kNormFew; ++u) v[u] = i + 16 * u < b1 ? get_partial(a.partials + i + 16 * u) : 0.0;
#pragma unroll
            for (int u = 0; u < kNormFew; ++u) t += v[u];
        }
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) t += __shfl_xor(t, off, 16);
        if (lane == 0) a.entry_norms[e] = float(sqrt(t));
    }
}

// One thread, a record after another: a call takes 4.3 us for 8 owners, 4.5
// for 64, 166 for 4096.
__global__ void k_grad_total(const mfsdp_grad_stats* parts, int count, mfsdp_grad_stats* stats, double max_norm,
                             double eps) {
    double s = 0.0;
    for (int i = 0; i < count; ++i) s += parts[i].sumsq;
    write_stats(stats, s, max_norm, eps);
}

// One 16-byte word a thread, one 8 KB slice a block, no loop, loads past the
// caches.  Of the shapes tried on the 1.7 GB share (1, 2, 4 or 8 words a
// thread, 64 to 1024 threads, fixed grids that walk longer chunks), 512
// threads of one word copy at 6.65 TB/s, 256 at 6.57, 1024 at 6.46; two words
// a thread reach 6.1, four 6.0, a fixed grid over 128 KB chunks 5.3, and the
// same body inside a loop over slices 6.0.  first: the launch's first slice.
__global__ __launch_bounds__(kClipThreads) void k_grad_clip(const GradRun* chunks, int64_t first, int slice_shift,
                                                            const uint8_t* grads, uint8_t* out, const float* scale) {
    const int64_t b = first + blockIdx.x;
    const GradRun c = chunks[b >> slice_shift];
    const float f = *scale;
    if (f == 1.f && grads == out) return;
    const bool bf = c.dtype == kBF16;
    const uint32_t slice = uint32_t(b) & ((1u << slice_shift) - 1u);
    const uint32_t per = bf ? 8 : 4, numel = uint32_t(c.numel), words = numel / per;
    const uint32_t i = slice * kClipThreads + threadIdx.x;
    const u32x4_t* q = reinterpret_cast<const u32x4_t*>(grads + c.off);
    u32x4_t* o = reinterpret_cast<u32x4_t*>(out + c.off);
    if (i < words) {
        u32x4_t w = __builtin_nontemporal_load(q + i);
        if (f != 1.f) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = bf ? pack_bf16x2(f * __uint_as_float(w[k] << 16), f * __uint_as_float(w[k] & 0xffff0000u))
                          : __float_as_uint(f * __uint_as_float(w[k]));
        }
        o[i] = w;
    } else if (i == words) {
        // the elements behind the last whole word
        for (uint32_t k = words * per; k < numel; ++k) {
            if (bf) {
                const uint16_t v = reinterpret_cast<const uint16_t*>(q)[k];
                reinterpret_cast<uint16_t*>(o)[k] = f == 1.f ? v : f32_to_bf16(f * bf16_to_f32(v));
            } else {
                const float v = reinterpret_cast<const float*>(q)[k];
                reinterpret_cast<float*>(o)[k] = f == 1.f ? v : f * v;
            }
        }
    }
}

mfsdp_status hip_fail(hipError_t e, const char* what) {
    return fail(MFSDP_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// Checks shared by the norm and clipping, then the descriptor upload.
mfsdp_status ready(const GradTables& t, const void* grads, void* workspace, uint64_t workspace_bytes, uint32_t flags,
                   void* stream) {
    if (!workspace || misaligned(workspace, kAlign))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "workspace is NULL or not 256-byte aligned");
    if (t.n_chunks > 0 && !grads) return fail(MFSDP_ERR_INVALID_ARGUMENT, "grads is NULL");
    if (misaligned(grads, 16)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "grads must be 16-byte aligned");
    if (flags & ~MFSDP_STEP_DESCRIPTORS_RESIDENT) return fail(MFSDP_ERR_INVALID_ARGUMENT, "unknown flag");
    if (workspace_bytes < t.total_bytes)
        return fail(MFSDP_ERR_WORKSPACE_TOO_SMALL, "workspace has " + std::to_string(workspace_bytes) +
                                                       " bytes, the table needs " + std::to_string(t.total_bytes));
    if (!(flags & MFSDP_STEP_DESCRIPTORS_RESIDENT)) {
        const hipError_t e = hipMemcpyAsync(workspace, t.blob.data(), t.blob.size(), hipMemcpyHostToDevice,
                                            static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return hip_fail(e, "descriptor upload");
    }
    return MFSDP_OK;
}

mfsdp_status check_limit(double max_norm, double eps) {
    if (!(max_norm > 0.0)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "max_norm must be above 0");
    if (!(eps >= 0.0) || std::isinf(eps)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
    return MFSDP_OK;
}

}  // namespace
}  // namespace mfsdp

using namespace mfsdp;

extern "C" mfsdp_status mfsdp_grad_norm(mfsdp_plan_t plan, const mfsdp_grad_norm_args* args) {
    clear_error();
    if (!plan || !args) return fail(MFSDP_ERR_INVALID_ARGUMENT, "NULL plan or args");
    if (!args->stats || misaligned(args->stats, 16))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "stats is NULL or not 16-byte aligned");
    if (misaligned(args->entry_norms, 4)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "entry_norms must be 4-byte aligned");
    if (mfsdp_status st = check_limit(args->max_norm, args->eps); st != MFSDP_OK) return st;
    const GradTables* t = nullptr;
    if (mfsdp_status st = grad_tables(plan, &t); st != MFSDP_OK) return st;
    if (mfsdp_status st = ready(*t, args->grads, args->workspace, args->workspace_bytes, args->flags, args->stream);
        st != MFSDP_OK)
        return st;
    uint8_t* ws = static_cast<uint8_t*>(args->workspace);
    NormArgs a;
    a.pieces = reinterpret_cast<const GradRun*>(ws + t->off_pieces);
    a.blocks = reinterpret_cast<const NormBlock*>(ws + t->off_blocks);
    a.entry_begin = reinterpret_cast<const int32_t*>(ws + t->off_entry_begin);
    a.grads = static_cast<const uint8_t*>(args->grads);
    a.partials = reinterpret_cast<double*>(ws + t->off_partials);
    a.counters = reinterpret_cast<uint32_t*>(ws + t->off_counters);
    a.entry_norms = args->entry_norms;
    a.stats = args->stats;
    a.max_norm = args->max_norm;
    a.eps = args->eps;
    a.n_pieces = t->n_pieces;
    a.n_entries = t->n_entries;
    a.large = reinterpret_cast<const int32_t*>(ws + t->off_large);
    a.n_large = t->n_large;
    k_grad_norm<<<dim3(t->n_blocks), dim3(kNormThreads), 0, static_cast<hipStream_t>(args->stream)>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return hip_fail(e, "gradient norm launch");
    return MFSDP_OK;
}

extern "C" mfsdp_status mfsdp_grad_total(const mfsdp_grad_stats* parts, int64_t count, double max_norm, double eps,
                                         mfsdp_grad_stats* stats, void* stream) {
    clear_error();
    if (!parts || !stats || misaligned(parts, 16) || misaligned(stats, 16))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "parts or stats is NULL or not 16-byte aligned");
    if (count < 1 || count > 65536) return fail(MFSDP_ERR_INVALID_ARGUMENT, "count must be in 1..65536");
    if (mfsdp_status st = check_limit(max_norm, eps); st != MFSDP_OK) return st;
    k_grad_total<<<dim3(1), dim3(1), 0, static_cast<hipStream_t>(stream)>>>(parts, int(count), stats, max_norm, eps);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return hip_fail(e, "gradient total launch");
    return MFSDP_OK;
}

extern "C" mfsdp_status mfsdp_grad_clip(mfsdp_plan_t plan, const mfsdp_grad_clip_args* args) {
    clear_error();
    if (!plan || !args) return fail(MFSDP_ERR_INVALID_ARGUMENT, "NULL plan or args");
    if (!args->scale || misaligned(args->scale, 4))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "scale is NULL or not 4-byte aligned");
    const GradTables* t = nullptr;
    if (mfsdp_status st = grad_tables(plan, &t); st != MFSDP_OK) return st;
    const uintptr_t g = reinterpret_cast<uintptr_t>(args->grads), o = reinterpret_cast<uintptr_t>(args->out);
    if (t->n_chunks > 0 && !args->out) return fail(MFSDP_ERR_INVALID_ARGUMENT, "out is NULL");
    if (misaligned(args->out, 16)) return fail(MFSDP_ERR_INVALID_ARGUMENT, "out must be 16-byte aligned");
    if (g != o && (g < o ? o - g : g - o) < plan->max_param_end)
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "grads and out overlap in part");
    if (mfsdp_status st = ready(*t, args->grads, args->workspace, args->workspace_bytes, args->flags, args->stream);
        st != MFSDP_OK)
        return st;
    if (t->n_chunks == 0) return MFSDP_OK;
    const int64_t n_slices = int64_t(t->n_chunks) << t->slice_shift;
    for (int64_t first = 0; first < n_slices; first += kClipBlocksMax)  // one launch below 68 GB
        k_grad_clip<<<dim3(uint32_t(std::min(n_slices - first, kClipBlocksMax))), dim3(kClipThreads), 0,
                      static_cast<hipStream_t>(args->stream)>>>(
            static_cast<const GradRun*>(args->workspace), first, t->slice_shift,
            static_cast<const uint8_t*>(args->grads), static_cast<uint8_t*>(args->out), args->scale);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return hip_fail(e, "clip launch");
    return MFSDP_OK;
}
