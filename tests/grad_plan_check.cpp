// grad_plan_check.cpp - host-only check of the gradient operators' work list
// (built with g++ against plan.cpp and grad_plan.cpp; no HIP).  For the tables
// below and seeded random ones: chunks and pieces each cover every element of
// every entry exactly once, in order, at 16-byte aligned places; a chunk fits
// its slices; the blocks split the pieces, each knows its first one, and no
// block costs more than a share; entry ranges and the list of large entries
// are right; the counters are zero.  Prints "OK <tables>" or the first failure.
#include <cstdio>
#include <cstring>
#include <random>

#include "plan_internal.h"

using namespace mfsdp;

#define EXPECT(c, ...)                                       \
    do {                                                     \
        if (!(c)) {                                          \
            std::printf("FAIL table %d %s: ", tables, #c);   \
            std::printf(__VA_ARGS__);                        \
            std::printf("\n");                               \
            return 1;                                        \
        }                                                    \
    } while (0)

static int tables = 0;

static int check(const std::vector<mfsdp_entry>& entries, uint64_t bytes) {
    ++tables;
    mfsdp_hparams hp = {};
    hp.ns_steps = 5;
    hp.ns_eps = 1e-7f;
    mfsdp_plan_t plan = nullptr;
    EXPECT(mfsdp_plan_create(entries.data(), int64_t(entries.size()), bytes, &hp, &plan) == MFSDP_OK, "%s",
           mfsdp_last_error_message());
    const GradTables* t = nullptr;
    EXPECT(grad_tables(plan, &t) == MFSDP_OK, "%s", mfsdp_last_error_message());
    uint64_t ws = 0;
    EXPECT(mfsdp_plan_grad_workspace_bytes(plan, &ws) == MFSDP_OK && ws == t->total_bytes, "%llu", (unsigned long long)ws);
    const uint8_t* blob = t->blob.data();
    const GradRun* chunks = reinterpret_cast<const GradRun*>(blob);
    const NormBlock* blocks = reinterpret_cast<const NormBlock*>(blob + t->off_blocks);
    const GradRun* pieces = reinterpret_cast<const GradRun*>(blob + t->off_pieces);
    const int32_t* begin = reinterpret_cast<const int32_t*>(blob + t->off_entry_begin);
    const int32_t* large = reinterpret_cast<const int32_t*>(blob + t->off_large);
    const uint32_t* counters = reinterpret_cast<const uint32_t*>(blob + t->off_counters);
    EXPECT(t->blob.size() <= t->off_partials && t->off_partials + uint64_t(t->n_pieces) * 8 <= ws, "regions");
    EXPECT(t->off_counters + (kNormGroups + 1) * kNormCounterPitch * 4 <= t->blob.size(), "counters");
    for (uint32_t k = 0; k < (kNormGroups + 1) * kNormCounterPitch; ++k) EXPECT(counters[k] == 0, "counter %u", k);

    int32_t c = 0, p = 0, n_large = 0;
    for (size_t i = 0; i < entries.size(); ++i) {
        const mfsdp_entry& e = entries[i];
        const uint64_t es = e.dtype == kBF16 ? 2 : 4, numel = uint64_t(e.rows) * uint64_t(e.cols);
        auto cover = [&](const GradRun* runs, int32_t& k, int32_t n) {
            uint64_t at = 0;
            while (at < numel) {
                if (k >= n || runs[k].off != e.offset + at * es || runs[k].off % 16 != 0 || runs[k].numel == 0 ||
                    runs[k].numel > numel - at || runs[k].dtype != e.dtype)
                    return false;
                at += runs[k++].numel;
            }
            return true;
        };
        const int32_t c0 = c;
        EXPECT(cover(chunks, c, t->n_chunks), "chunks of entry %zu", i);
        for (int32_t k = c0; k < c; ++k)
            EXPECT(chunks[k].numel * es <= uint64_t(kGradSlice) << t->slice_shift, "chunk %d", k);
        EXPECT(begin[i] == p, "entry %zu", i);
        EXPECT(cover(pieces, p, t->n_pieces), "pieces of entry %zu", i);
        if (p - begin[i] > kNormFew) {
            EXPECT(n_large < t->n_large && large[n_large] == int32_t(i), "large entry %zu", i);
            ++n_large;
        }
    }
    EXPECT(c == t->n_chunks && p == t->n_pieces && begin[entries.size()] == p && n_large == t->n_large, "counts");
    EXPECT(t->n_blocks >= 1 && t->n_blocks <= kNormBlocks + 1, "%d blocks", t->n_blocks);
    int32_t at = 0;
    int64_t most = 0, sum = 0;
    for (int32_t b = 0; b < t->n_blocks; ++b) {
        EXPECT(blocks[b].begin == at && blocks[b].end >= at, "block %d", b);
        EXPECT(blocks[b].end > at || t->n_pieces == 0, "block %d is empty", b);
        if (blocks[b].end > at) EXPECT(std::memcmp(&blocks[b].first, &pieces[at], sizeof(GradRun)) == 0, "block %d", b);
        int64_t cost = 0;
        for (; at < blocks[b].end; ++at)
            cost += kNormPieceCost + int64_t((pieces[at].numel * (pieces[at].dtype == kBF16 ? 2 : 4) + kGradSlice - 1) / kGradSlice);
        most = cost > most ? cost : most;
        sum += cost;
    }
    EXPECT(at == t->n_pieces, "blocks");
    EXPECT(most <= kNormShareMin || most <= 2 * kNormPieceCost + (sum + kNormBlocks - 1) / kNormBlocks, "%lld of %lld",
           (long long)most, (long long)sum);
    mfsdp_plan_destroy(plan);
    return 0;
}

int main() {
    auto table = [](const std::vector<std::vector<int64_t>>& shapes, uint64_t gap, uint64_t& bytes) {
        std::vector<mfsdp_entry> out;
        bytes = gap;
        for (const auto& s : shapes) {
            out.push_back(mfsdp_entry{bytes, s[0], s[1], int32_t(s[2]), MFSDP_ROLE_ADAMW});
            bytes += (uint64_t(s[0] * s[1]) * (s[2] == kBF16 ? 2 : 4) + 15) / 16 * 16 + gap;
        }
        return out;
    };
    uint64_t bytes;
    const std::vector<std::vector<std::vector<int64_t>>> fixed = {
        {}, {{0, 5, 1}, {3, 0, 0}}, {{1, 1, 1}}, {{1, 4096, 1}, {1, 4097, 1}, {1, 2047, 0}, {1, 2048, 0}, {1, 2049, 0}},
        {{4096, 4096, 1}, {14336, 4096, 1}, {1024, 4096, 0}}, {{128256, 4096, 1}}, {{int64_t(1) << 20, int64_t(1) << 20, 0}},
        std::vector<std::vector<int64_t>>(3000, {1, 7, 0}), std::vector<std::vector<int64_t>>(40000, {3, 50, 1})};
    for (const auto& f : fixed) {
        const auto t = table(f, 16, bytes);
        if (check(t, bytes)) return 1;
    }
    std::mt19937_64 rng(11);
    for (int k = 0; k < 300; ++k) {
        std::vector<std::vector<int64_t>> shapes;
        const int n = 1 + int(rng() % 60);
        for (int i = 0; i < n; ++i) {
            const int big = int(rng() % 14);
            shapes.push_back({int64_t(rng() % ((uint64_t(1) << big) + 1)), int64_t(rng() % 3000), int64_t(rng() % 2)});
        }
        const auto t = table(shapes, 16 * (rng() % 5), bytes);
        if (check(t, bytes)) return 1;
    }
    std::printf("OK %d\n", tables);
    return 0;
}
