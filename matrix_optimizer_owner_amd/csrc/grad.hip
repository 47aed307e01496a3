// grad.hip - the global gradient norm over every tensor of an owner buffer,
// and clipping, on gfx950.
//
//   sumsq = sum g^2;  norm = sqrt(sumsq);  scale = min(1, max_norm/(norm+eps));
//   out <- RNE(scale * g).
//
// Both passes are bound by HBM: the norm reads each gradient once, clipping
// reads and writes it once.  One block takes one chunk of one tensor
// (grad_layout.h), so a launch covers every tensor whatever its size.
#include <cmath>
#include <string>

#include "device_util.h"
#include "plan_internal.h"

namespace mfsdp {
namespace {

constexpr int kGradThreads = 256;

// sum of squares of one 16-byte word, in fp64
template <int DT> __device__ __forceinline__ double sq16(u32x4_t w) {
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (DT == kBF16) {
            const double lo = double(__uint_as_float(w[k] << 16)), hi = double(__uint_as_float(w[k] & 0xffff0000u));
            s = __builtin_fma(lo, lo, s);
            s = __builtin_fma(hi, hi, s);
        } else {
            const double v = double(__uint_as_float(w[k]));
            s = __builtin_fma(v, v, s);
        }
    }
    return s;
}

// Sum over the block in a fixed order; the result is valid in thread 0.
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double red[kGradThreads / 64];
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0)
        for (int k = 0; k < kGradThreads / 64; ++k) t += red[k];
    return t;
}

template <int DT> __device__ __forceinline__ double chunk_sumsq(const uint8_t* p, uint32_t numel) {
    constexpr uint32_t PER = DT == kBF16 ? 8 : 4;
    const u32x4_t* q = reinterpret_cast<const u32x4_t*>(p);
    const uint32_t words = numel / PER;
    double s = 0.0;
    for (uint32_t i = threadIdx.x; i < words; i += kGradThreads) s += sq16<DT>(q[i]);
    const uint32_t i = words * PER + threadIdx.x;
    if (i < numel) {
        const double v = double(load_elem(p, DT, i));
        s = __builtin_fma(v, v, s);
    }
    return s;
}

__global__ __launch_bounds__(kGradThreads) void k_grad_partials(const GradChunk* chunks, const uint8_t* grads,
                                                                double* partials) {
    const GradChunk c = chunks[blockIdx.x];
    const uint8_t* p = grads + c.off;
    const double s = block_sum(c.dtype == kBF16 ? chunk_sumsq<kBF16>(p, c.numel) : chunk_sumsq<kF32>(p, c.numel));
    if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

__device__ __forceinline__ void write_stats(mfsdp_grad_stats* out, double sumsq, double max_norm, double eps) {
    const double norm = sqrt(sumsq);
    const double f = max_norm / (norm + eps);
    out->sumsq = sumsq;
    out->norm = float(norm);
    // a NaN norm gives a NaN scale; an infinite max_norm never scales
    out->scale = isinf(max_norm) || f >= 1.0 ? 1.f : float(f);
}

// Block 0: the whole table; block 1 + e: entry e.
__global__ __launch_bounds__(kGradThreads) void k_grad_finalize(const double* partials, const int32_t* entry_begin,
                                                                int n_chunks, float* entry_norms,
                                                                mfsdp_grad_stats* stats, double max_norm, double eps) {
    const int e = int(blockIdx.x) - 1;
    const int b0 = e < 0 ? 0 : entry_begin[e], b1 = e < 0 ? n_chunks : entry_begin[e + 1];
    double s = 0.0;
    for (int i = b0 + int(threadIdx.x); i < b1; i += kGradThreads) s += partials[i];
    s = block_sum(s);
    if (threadIdx.x != 0) return;
    if (e < 0)
        write_stats(stats, s, max_norm, eps);
    else
        entry_norms[e] = float(sqrt(s));
}

__global__ void k_grad_total(const mfsdp_grad_stats* parts, int count, mfsdp_grad_stats* stats, double max_norm,
                             double eps) {
    double s = 0.0;
    for (int i = 0; i < count; ++i) s += parts[i].sumsq;
    write_stats(stats, s, max_norm, eps);
}

__global__ __launch_bounds__(kGradThreads) void k_grad_clip(const GradChunk* chunks, const uint8_t* grads, uint8_t* out,
                                                            const float* scale) {
    const float f = *scale;
    if (f == 1.f && grads == out) return;
    const GradChunk c = chunks[blockIdx.x];
    const uint32_t per = c.dtype == kBF16 ? 8 : 4, words = c.numel / per;
    const u32x4_t* q = reinterpret_cast<const u32x4_t*>(grads + c.off);
    u32x4_t* o = reinterpret_cast<u32x4_t*>(out + c.off);
    for (uint32_t i = threadIdx.x; i < words; i += kGradThreads) {
        u32x4_t w = q[i];
        if (f != 1.f) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = c.dtype == kBF16 ? pack_bf16x2(f * __uint_as_float(w[k] << 16), f * __uint_as_float(w[k] & 0xffff0000u))
                                        : __float_as_uint(f * __uint_as_float(w[k]));
        }
        o[i] = w;
    }
    const uint32_t i = words * per + threadIdx.x;
    if (i < c.numel) {
        if (c.dtype == kBF16) {
            const uint16_t v = reinterpret_cast<const uint16_t*>(q)[i];
            reinterpret_cast<uint16_t*>(o)[i] = f == 1.f ? v : f32_to_bf16(f * bf16_to_f32(v));
        } else {
            const float v = reinterpret_cast<const float*>(q)[i];
            reinterpret_cast<float*>(o)[i] = f == 1.f ? v : f * v;
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
    const uint8_t* ws = static_cast<const uint8_t*>(args->workspace);
    const GradChunk* chunks = reinterpret_cast<const GradChunk*>(ws);
    const int32_t* begin = reinterpret_cast<const int32_t*>(ws + t->off_entry_begin);
    double* partials = reinterpret_cast<double*>(static_cast<uint8_t*>(args->workspace) + t->off_partials);
    hipStream_t stream = static_cast<hipStream_t>(args->stream);
    if (t->n_chunks > 0) {
        k_grad_partials<<<dim3(t->n_chunks), dim3(kGradThreads), 0, stream>>>(
            chunks, static_cast<const uint8_t*>(args->grads), partials);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return hip_fail(e, "gradient norm launch");
    }
    k_grad_finalize<<<dim3(1 + (args->entry_norms ? t->n_entries : 0)), dim3(kGradThreads), 0, stream>>>(
        partials, begin, t->n_chunks, args->entry_norms, args->stats, args->max_norm, args->eps);
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
    k_grad_clip<<<dim3(t->n_chunks), dim3(kGradThreads), 0, static_cast<hipStream_t>(args->stream)>>>(
        static_cast<const GradChunk*>(args->workspace), static_cast<const uint8_t*>(args->grads),
        static_cast<uint8_t*>(args->out), args->scale);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return hip_fail(e, "clip launch");
    return MFSDP_OK;
}
