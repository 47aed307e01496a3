// clip_plan_check.cpp - host-only check of the clipping work list's length
// (built with g++ against plan.cpp and grad_plan.cpp; no HIP).  Clipping
// launches a block for each slice of each chunk, empty ones too: for the
// tables below and seeded random ones the blocks are at most three times the
// slices that hold elements, and the list has at most kGradChunks chunks and
// two more for each tensor.  Prints "OK <tables>" or the first failure.
#include <cstdio>
#include <random>

#include "plan_internal.h"

using namespace mfsdp;

static int tables = 0;

static int check(const std::vector<std::vector<int64_t>>& shapes) {
    ++tables;
    std::vector<mfsdp_entry> entries;
    uint64_t bytes = 0;
    int64_t useful = 0, held = 0;
    for (const auto& s : shapes) {
        entries.push_back(mfsdp_entry{bytes, s[0], s[1], int32_t(s[2]), MFSDP_ROLE_ADAMW});
        const int64_t size = s[0] * s[1] * (s[2] == kBF16 ? 2 : 4);
        bytes += uint64_t(size + 15) / 16 * 16;
        useful += (size + kGradSlice - 1) / kGradSlice;
        held += size > 0;
    }
    mfsdp_hparams hp = {};
    hp.ns_steps = 5;
    hp.ns_eps = 1e-7f;
    mfsdp_plan_t plan = nullptr;
    const GradTables* t = nullptr;
    if (mfsdp_plan_create(entries.data(), int64_t(entries.size()), bytes, &hp, &plan) != MFSDP_OK ||
        grad_tables(plan, &t) != MFSDP_OK) {
        std::printf("FAIL table %d: %s\n", tables, mfsdp_last_error_message());
        return 1;
    }
    const int64_t blocks = int64_t(t->n_chunks) << t->slice_shift;
    if (blocks < useful || blocks > 3 * useful || t->n_chunks > kGradChunks + 2 * held) {
        std::printf("FAIL table %d (%zu tensors): %lld blocks for %lld slices, %d chunks\n", tables, shapes.size(),
                    (long long)blocks, (long long)useful, t->n_chunks);
        return 1;
    }
    mfsdp_plan_destroy(plan);
    return 0;
}

int main() {
    const std::vector<int64_t> small = {3, 50, kBF16};
    for (size_t n : {0, 1, 100, 16383, 16384, 16385, 40000, 100000})
        if (check(std::vector<std::vector<int64_t>>(n, small))) return 1;
    for (size_t n : {100, 10000, 16000, 16384, 40000}) {
        std::vector<std::vector<int64_t>> mixed(n, small);
        mixed.push_back({128256, 4096, kBF16});
        if (check(mixed)) return 1;
        for (int k = 0; k < 40; ++k) mixed.push_back({int64_t(1) << 22, 700, kF32});
        if (check(mixed)) return 1;
    }
    std::mt19937_64 rng(12);
    for (int k = 0; k < 100; ++k) {
        std::vector<std::vector<int64_t>> shapes;
        const int n = 1 << (rng() % 17), top = 1 + int(rng() % 20);
        for (int i = 0; i < n; ++i)
            shapes.push_back({int64_t(rng() % ((uint64_t(1) << (rng() % top)) + 1)), int64_t(rng() % 3000), int64_t(rng() % 2)});
        if (check(shapes)) return 1;
    }
    std::printf("OK %d\n", tables);
    return 0;
}
