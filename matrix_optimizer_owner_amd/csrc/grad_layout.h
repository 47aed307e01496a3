// grad_layout.h - the gradient operators' work list, shared by the host
// lowering (grad_plan.cpp) and the kernels (grad.hip).
//
// Workspace map (byte offsets, 256-byte aligned):
//   [desc]      GradRun[n_chunks] (clipping), NormBlock[n_blocks],
//               GradRun[n_pieces], int32 entry_begin[n_entries + 1] and
//               large[n_large] (norm), and the norm's counters of finished
//               blocks (0 between calls): kNormGroups + 1 uint32 at a pitch of
//               kNormCounterPitch
//   [partials]  double[n_pieces]: sum of g^2 of one piece
#pragma once
#include <stdint.h>

#include <vector>

namespace mfsdp {

// A run of one entry's elements.  Its first byte is 16-byte aligned: entry
// offsets are, and a run starts a multiple of kGradSlice into its entry.
struct GradRun {
    uint64_t off;      // bytes into params / grads
    uint64_t numel;    // at least 1
    int32_t dtype;
    int32_t pad_;
};
static_assert(sizeof(GradRun) == 24, "GradRun layout");

// A block's share of the norm: pieces begin .. end-1, the first one here too,
// so that a block of one piece starts on it a load earlier.
struct NormBlock {
    GradRun first;
    int32_t begin, end;
};
static_assert(sizeof(NormBlock) == 32, "NormBlock layout");

struct GradTables {
    std::vector<uint8_t> blob;  // [desc], uploaded by one copy
    uint64_t off_blocks = 0, off_pieces = 0, off_entry_begin = 0, off_large = 0, off_counters = 0,
             off_partials = 0;
    uint64_t total_bytes = 0;
    int32_t n_entries = 0;
    // Clipping: chunk c is 2^slice_shift slices of kGradSlice bytes (its last
    // ones may be empty), one slice a block.
    int32_t n_chunks = 0, slice_shift = 0;
    // The norm: the blocks' pieces cut the table into n_blocks shares of the
    // same cost (a piece ends where its share or its entry does; an empty table
    // has one block of no piece).  Entry e is pieces entry_begin[e] ..
    // entry_begin[e+1]-1; `large` are the entries of more than kNormFew.
    int32_t n_pieces = 0, n_blocks = 0, n_large = 0;
};

constexpr int64_t kGradSlice = 8192;
// A chunk is the smallest power of two of bytes (at most kGradChunkMax) that
// cuts the table into at most kGradChunks chunks and two more for each tensor
// that is not empty: few enough for a short list, short enough not to leave
// many empty slices behind small tensors.  With N tensors and S slices that
// hold elements, half the length would make more than kGradChunks + 2 N
// chunks, so S / (slices of half a chunk) > kGradChunks + N, and the empty
// slices, less than a chunk's for each tensor, are fewer than 2 S.
constexpr int64_t kGradChunks = 16384;
constexpr int64_t kGradChunkMax = int64_t(1) << 30;
// The norm's shares.  Cost counts slices, and kNormPieceCost more for each
// piece (about what its descriptor, its sum and its drained loads take), so
// that many small tensors spread over more blocks.  One share for every
// kNormShareMin of cost, at most kNormBlocks.  (65 tensors of 16 KB take 5.6,
// 5.5, 6.2 and 8.2 us with a kNormShareMin of 2, 4, 8 and 16; 71 ragged ones,
// 7.1 MB, 7.3, 7.4, 7.5 and 12.1.)
constexpr int64_t kNormPieceCost = 2;
constexpr int64_t kNormShareMin = 8;
constexpr int64_t kNormBlocks = 1024;
constexpr int kNormFew = 8;
constexpr uint32_t kNormGroups = 32;
constexpr uint32_t kNormCounterPitch = 64;  // 256 bytes: no two share a cache line

}  // namespace mfsdp
