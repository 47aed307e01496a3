// grad_plan.cpp - lowering of an owner table to the gradient operators' work
// list.  Host only: this file makes no HIP call.
#include <algorithm>
#include <cstring>
#include <new>

#include "plan_internal.h"

namespace mfsdp {
namespace {

std::unique_ptr<GradTables> lower(const mfsdp_plan_s& plan) {
    auto t = std::make_unique<GradTables>();
    auto es = [](const mfsdp_entry& e) { return int64_t(e.dtype == kBF16 ? 2 : 4); };
    auto count = [&](int64_t len) {
        int64_t c = 0;
        for (const mfsdp_entry& e : plan.entries) c += (e.rows * e.cols * es(e) + len - 1) / len;
        return c;
    };
    int64_t held = 0;  // tensors that are not empty
    for (const mfsdp_entry& e : plan.entries) held += e.rows * e.cols > 0;
    int64_t len = kGradSlice;
    while (len < kGradChunkMax && count(len) > kGradChunks + 2 * held) len *= 2;
    if (count(len) > int64_t(INT32_MAX)) return t;  // refused below: total_bytes stays 0
    for (int64_t l = kGradSlice; l < len; l *= 2) ++t->slice_shift;
    const int64_t cost = count(kGradSlice) + held * kNormPieceCost;
    const int64_t share = std::max(kNormShareMin, kNormPieceCost + (cost + kNormBlocks - 1) / kNormBlocks);
    std::vector<GradRun> chunks, pieces;
    std::vector<int32_t> block_begin(1, 0), entry_begin(1, 0), large;
    int64_t left = share;  // cost that the current share still takes
    auto close = [&] {
        block_begin.push_back(int32_t(pieces.size()));
        left = share;
    };
    for (const mfsdp_entry& e : plan.entries) {
        const int64_t numel = e.rows * e.cols, per = kGradSlice / es(e);
        auto run = [&](int64_t at, int64_t n) {
            return GradRun{e.offset + uint64_t(at * es(e)), uint64_t(std::min(numel - at, n)), e.dtype, 0};
        };
        for (int64_t at = 0; at < numel; at += len / es(e)) chunks.push_back(run(at, len / es(e)));
        for (int64_t at = 0; at < numel;) {
            if (left <= kNormPieceCost) close();
            const int64_t take = std::min(left - kNormPieceCost, (numel - at + per - 1) / per);
            pieces.push_back(run(at, take * per));
            at += take * per;
            left -= kNormPieceCost + take;
        }
        if (int64_t(pieces.size()) - entry_begin.back() > kNormFew) large.push_back(int32_t(entry_begin.size()) - 1);
        entry_begin.push_back(int32_t(pieces.size()));
    }
    if (block_begin.back() != int32_t(pieces.size())) close();
    t->n_entries = int32_t(plan.entries.size());
    t->n_chunks = int32_t(chunks.size());
    t->n_pieces = int32_t(pieces.size());
    std::vector<NormBlock> blocks;
    for (size_t b = 0; b + 1 < block_begin.size(); ++b)
        blocks.push_back(NormBlock{pieces[size_t(block_begin[b])], block_begin[b], block_begin[b + 1]});
    if (blocks.empty()) blocks.push_back(NormBlock{});
    t->n_blocks = int32_t(blocks.size());
    t->n_large = int32_t(large.size());
    uint64_t off = 0;
    auto put = [&](const auto& v) {
        const uint64_t at = off, bytes = v.size() * sizeof(v[0]);
        off = align_up(off + bytes, kAlign);
        t->blob.resize(size_t(off), 0);
        if (bytes) std::memcpy(t->blob.data() + at, v.data(), bytes);
        return at;
    };
    put(chunks);
    t->off_blocks = put(blocks);
    t->off_pieces = put(pieces);
    t->off_entry_begin = put(entry_begin);
    t->off_large = put(large);
    t->off_counters = put(std::vector<uint32_t>((kNormGroups + 1) * kNormCounterPitch, 0));
    t->off_partials = off;
    t->total_bytes = off + align_up(pieces.size() * sizeof(double), kAlign);
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
