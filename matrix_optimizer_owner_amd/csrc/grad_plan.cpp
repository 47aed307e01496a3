// grad_plan.cpp - lowering of an owner table to the gradient operators' work
// list.  Host only: this file makes no HIP call.
#include <cstring>
#include <new>

#include "plan_internal.h"

namespace mfsdp {
namespace {

std::unique_ptr<GradTables> lower(const mfsdp_plan_s& plan) {
    auto t = std::make_unique<GradTables>();
    auto count = [&](int64_t len) {
        int64_t c = 0;
        for (const mfsdp_entry& e : plan.entries) c += (e.rows * e.cols + len - 1) / len;
        return c;
    };
    int64_t len = kGradChunkMin;
    while (len < kGradChunkMax && count(len) > kGradChunks) len *= 2;
    if (count(len) > int64_t(INT32_MAX)) return t;  // refused below: n_chunks stays 0
    std::vector<GradChunk> chunks;
    std::vector<int32_t> begin(1, 0);
    for (const mfsdp_entry& e : plan.entries) {
        const int64_t numel = e.rows * e.cols;
        const uint64_t es = e.dtype == kBF16 ? 2 : 4;
        for (int64_t at = 0; at < numel; at += len)
            chunks.push_back(GradChunk{e.offset + uint64_t(at) * es, uint32_t(numel - at < len ? numel - at : len), e.dtype});
        begin.push_back(int32_t(chunks.size()));
    }
    t->n_chunks = int32_t(chunks.size());
    t->n_entries = int32_t(plan.entries.size());
    t->off_entry_begin = align_up(chunks.size() * sizeof(GradChunk), kAlign);
    const uint64_t desc = t->off_entry_begin + align_up(begin.size() * sizeof(int32_t), kAlign);
    t->off_partials = desc;
    t->total_bytes = desc + align_up(chunks.size() * sizeof(double), kAlign);
    t->blob.assign(size_t(desc), 0);
    if (!chunks.empty()) std::memcpy(t->blob.data(), chunks.data(), chunks.size() * sizeof(GradChunk));
    std::memcpy(t->blob.data() + t->off_entry_begin, begin.data(), begin.size() * sizeof(int32_t));
    return t;
}

}  // namespace

mfsdp_status grad_tables(mfsdp_plan_t plan, const GradTables** out) {
    try {
        std::call_once(plan->grad_once, [&] { plan->grad_tables = lower(*plan); });
    } catch (const std::bad_alloc&) {
        return fail(MFSDP_ERR_INTERNAL, "out of host memory");
    } catch (...) {
        return fail(MFSDP_ERR_INTERNAL, "unexpected exception in the gradient tables");
    }
    if (plan->grad_tables->total_bytes == 0)
        return fail(MFSDP_ERR_UNSUPPORTED, "owner buffer too large for the gradient operators");
    *out = plan->grad_tables.get();
    return MFSDP_OK;
}

}  // namespace mfsdp

using namespace mfsdp;

extern "C" mfsdp_status mfsdp_plan_grad_workspace_bytes(mfsdp_plan_t plan, uint64_t* bytes) {
    clear_error();
    if (!plan || !bytes) return fail(MFSDP_ERR_INVALID_ARGUMENT, "NULL argument");
    const GradTables* t = nullptr;
    if (mfsdp_status st = grad_tables(plan, &t); st != MFSDP_OK) return st;
    *bytes = t->total_bytes;
    return MFSDP_OK;
}
