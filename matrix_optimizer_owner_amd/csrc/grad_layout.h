// grad_layout.h - the gradient operators' work list, shared by the host
// lowering (grad_plan.cpp) and the kernels (grad.hip).
//
// Workspace map (byte offsets, 256-byte aligned):
//   [desc]      GradChunk[n_chunks], int32 entry_begin[n_entries + 1]
//   [partials]  double[n_chunks]: sum of g^2 of one chunk
#pragma once
#include <stdint.h>

#include <vector>

namespace mfsdp {

// A run of one entry's elements, the work of one block.  Its first byte is
// 16-byte aligned: entry offsets are, and a chunk starts a multiple of the
// chunk length (a power of two of at least 1024 elements) into its entry.
struct GradChunk {
    uint64_t off;      // bytes into params / grads
    uint32_t numel;    // 1 .. chunk length
    int32_t dtype;
};
static_assert(sizeof(GradChunk) == 16, "GradChunk layout");

struct GradTables {
    std::vector<uint8_t> blob;  // [desc], uploaded by one copy
    uint64_t off_entry_begin = 0, off_partials = 0, total_bytes = 0;
    int32_t n_chunks = 0, n_entries = 0;
};

// Chunk lengths: the smallest power of two from kGradChunkMin to
// kGradChunkMax that cuts the table into at most kGradChunks chunks.
constexpr int64_t kGradChunkMin = 4096;
constexpr int64_t kGradChunkMax = int64_t(1) << 24;
constexpr int64_t kGradChunks = 16384;

}  // namespace mfsdp
