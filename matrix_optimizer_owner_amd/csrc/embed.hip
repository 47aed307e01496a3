// embed.hip - an embedding table that is one entry of an owner buffer:
// lookup with scaling, and the table's gradient, on gfx950.
//
//   lookup:  out[i] = scale * W[id_i - first];
//   grad:    G[v] (+)= scale * sum over i with id_i - first = v of dout[i].
#include <string>

#include "device_util.h"
#include "plan_internal.h"

namespace mfsdp {
namespace {

constexpr int kEmbedThreads = 256;

// Row of position i, or -1 for an id outside the table.  The difference is
// taken modulo 2^64: first is at most 2^62, so no id outside wraps into it.
__device__ __forceinline__ int64_t row_of(const void* ids, int id_type, int64_t i, int64_t first, int64_t rows) {
    const int64_t id = id_type == MFSDP_I64 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
    const uint64_t r = uint64_t(id) - uint64_t(first);
    return r < uint64_t(rows) ? int64_t(r) : -1;
}

struct LookupArgs {
    const void* table;
    const void* ids;
    void* out;
    int64_t rows, cols, first, out_stride;
    int table_type, id_type, out_type;
    float scale;
};

__global__ __launch_bounds__(kEmbedThreads) void k_embed_lookup(LookupArgs a) {
    const int64_t i = blockIdx.x;
    const int64_t r = row_of(a.ids, a.id_type, i, a.first, a.rows);
    for (int64_t c = threadIdx.x; c < a.cols; c += kEmbedThreads) {
        const float v = r < 0 ? 0.f : a.scale * load_elem(a.table, a.table_type, r * a.cols + c);
        store_elem(a.out, a.out_type, i * a.out_stride + c, v);
    }
}

struct GradArgs {
    void* grad;
    const void* ids;
    const void* dout;
    int64_t rows, cols, first, dout_stride;
    int n, grad_type, id_type, dout_type, accumulate;
    float scale;
};

// One block per table row: it finds the row's positions in order, and sums.
__global__ __launch_bounds__(kEmbedThreads) void k_embed_grad(GradArgs a) {
    __shared__ int list[kEmbedThreads];
    __shared__ int wave_n[kEmbedThreads / 64];
    const int64_t v = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int64_t c0 = 0; c0 < a.cols; c0 += kEmbedThreads) {
        const int64_t c = c0 + threadIdx.x;
        float acc = 0.f;
        bool any = false;
        for (int base = 0; base < a.n; base += kEmbedThreads) {
            const int i = base + int(threadIdx.x);
            const bool hit = i < a.n && row_of(a.ids, a.id_type, i, a.first, a.rows) == v;
            const uint64_t m = __ballot(hit);
            if (lane == 0) wave_n[wave] = __popcll(m);
            __syncthreads();
            int at = __popcll(m & ((uint64_t(1) << lane) - 1)), total = 0;
            for (int w = 0; w < kEmbedThreads / 64; ++w) {
                if (w < wave) at += wave_n[w];
                total += wave_n[w];
            }
            if (hit) list[at] = i;
            __syncthreads();
            any = any || total > 0;
            if (c < a.cols)
                for (int k = 0; k < total; ++k) acc += load_elem(a.dout, a.dout_type, int64_t(list[k]) * a.dout_stride + c);
            __syncthreads();
        }
        if (c < a.cols && (any || !a.accumulate)) {
            const float old = a.accumulate ? load_elem(a.grad, a.grad_type, v * a.cols + c) : 0.f;
            store_elem(a.grad, a.grad_type, v * a.cols + c, __builtin_fmaf(a.scale, acc, old));
        }
    }
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
    LookupArgs a{static_cast<const uint8_t*>(args->params) + e.offset, args->ids, args->out, e.rows, e.cols,
                 args->first_id, stride, e.dtype, args->id_type, args->out_type, args->scale};
    k_embed_lookup<<<dim3(uint32_t(args->n_ids)), dim3(kEmbedThreads), 0, static_cast<hipStream_t>(args->stream)>>>(a);
    if (hipError_t err = hipGetLastError(); err != hipSuccess) return hip_fail(err, "lookup launch");
    return MFSDP_OK;
}

extern "C" mfsdp_status mfsdp_plan_embed_workspace_bytes(mfsdp_plan_t plan, int64_t entry, int64_t n_ids,
                                                         uint64_t* bytes) {
    clear_error();
    if (!plan || !bytes) return fail(MFSDP_ERR_INVALID_ARGUMENT, "NULL argument");
    if (entry < 0 || entry >= int64_t(plan->entries.size()))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "entry index out of range");
    if (n_ids < 0 || n_ids > kMaxIds) return fail(MFSDP_ERR_INVALID_ARGUMENT, "n_ids must be in 0..2^30");
    *bytes = 0;
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
    GradArgs a{static_cast<uint8_t*>(args->grads) + e.offset, args->ids, args->dout, e.rows, e.cols, args->first_id,
               stride, int(args->n_ids), e.dtype, args->id_type, args->dout_type, args->accumulate, args->scale};
    k_embed_grad<<<dim3(uint32_t(e.rows)), dim3(kEmbedThreads), 0, static_cast<hipStream_t>(args->stream)>>>(a);
    if (hipError_t err = hipGetLastError(); err != hipSuccess) return hip_fail(err, "embedding gradient launch");
    return MFSDP_OK;
}
