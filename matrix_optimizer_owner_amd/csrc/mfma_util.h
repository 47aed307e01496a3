// mfma_util.h - what the MFMA contraction kernels share: matrix instructions
// by storage type, LDS swizzles and transposing reads, the shape of a block's
// pipeline, waits and direct-to-LDS loads.
#pragma once
#include "device_util.h"

namespace mfsdp {
namespace {

// Wave-uniform copies (scalar registers) of values every lane agrees on.
__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }
template <typename P>
__device__ __forceinline__ P* uni_ptr(P* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(uint32_t(v)), hi = __builtin_amdgcn_readfirstlane(uint32_t(v >> 32));
    return reinterpret_cast<P*>((uint64_t(hi) << 32) | lo);
}

template <typename T> struct Mfma;
template <> struct Mfma<uint16_t> {
    __device__ __forceinline__ static void step(f32x16_t& acc, const u32x4_t& a, const u32x4_t& b) {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                      __builtin_bit_cast(bf16x8_t, b), acc, 0, 0, 0);
    }
    // a * b with a zero accumulator input
    __device__ __forceinline__ static f32x16_t first(const u32x4_t& a, const u32x4_t& b) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), f32x16_t{}, 0, 0, 0);
    }
};
template <> struct Mfma<float> {
    __device__ __forceinline__ static void step(f32x16_t& acc, const u32x4_t& a, const u32x4_t& b) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a[t]), __uint_as_float(b[t]), acc, 0, 0, 0);
    }
};

// Physical granule of logical granule g in LDS row `row`.  Tiles stored
// row-major along the contraction are read back with 16-byte fragment reads
// of 32 consecutive rows.  With 128-byte rows (8 granules): g ^ ((row / 2) %
// 8).  With 64-byte rows (4 granules) two rows share a 128-byte bank window;
// the 2-bit mask (bit 1: row bit 2; bit 0: row bit 1 xor row bit 3) spreads
// both 8 consecutive rows over a 128-byte window and 16 over 256 bytes.
// K-major tiles (128-byte rows, read with transposing reads of 4 consecutive
// rows x 32 bytes per 16 lanes): g ^ (((row % 4) * 2) | ((row / 4) % 2)).
// The 128-byte forms were chosen among alternatives by measuring
// SQ_LDS_BANK_CONFLICT on gfx950: zero conflicts.
template <int GR>
__device__ __forceinline__ int swz_r(int row, int g) {
    if constexpr (GR == 8) return g ^ ((row >> 1) & 7);
    else return g ^ ((((row >> 2) & 1) << 1) | (((row >> 1) ^ (row >> 3)) & 1));
}
__device__ __forceinline__ int swz_k(int row, int g) { return g ^ (((row & 3) << 1) | ((row >> 2) & 1)); }

// Word 3 of a raw buffer resource on gfx950: 32-bit data format, no
// swizzle, no index stride.
constexpr int kRsrcWord3 = 0x00020000;

typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));

// ds_read_b64_tr_b16: within each group of 16 lanes, lane i receives element
// i % 4 of the 8-byte words addressed by lanes i/4, 4 + i/4, 8 + i/4 and
// 12 + i/4 (confirmed by an in-bounds probe on gfx950).  So if lane s of a
// group addresses (k0 + s/4, c0 + 4*(s%4)) of a K-major tile, lane i gets
// the 4 consecutive k0..k0+3 of column c0 + i.
__device__ __forceinline__ u32x2_t ds_read_tr16(const uint8_t* lds_byte_addr) {
    const i16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) i16x4_t*)(lds_byte_addr));
    return __builtin_bit_cast(u32x2_t, v);
}

// Block shape: BT x BT output tile, NW wave64s in a 2 x (NW/2) grid; a wave
// owns a (BT/2) x (2*BT/NW) block of MFMA 32x32 tiles.
template <int BT, int NW>
struct Shape {
    static constexpr int kThreads = 64 * NW;
    static constexpr int WC = NW / 2;            // wave columns
    static constexpr int WTM = BT / 2;           // wave tile rows
    static constexpr int WTN = BT / WC;          // wave tile columns
    static constexpr int MM = WTM / 32;          // MFMA tiles per wave along rows
    static constexpr int MN = WTN / 32;          // MFMA tiles per wave along columns
};

// Main-loop pipeline: stages of KSB = 128 bytes of contraction index (four
// MFMA sub-steps of 32 bytes) in split stage rings of 3 P slots and 2 Q
// slots (5 operand stages of LDS: 160 KB for 256 tiles, 80 KB for 128
// tiles).  On the Llama-3-8B share, 64-byte stages with more look-ahead
// (twice the barriers) measured 10-20% slower.
template <int BT, int NW>
struct Pipe {
    static constexpr int KSB = 128;                // bytes of contraction index per stage
    static constexpr int SUBS = KSB / 32;          // MFMA sub-steps per stage
    static constexpr int GR = KSB / 16;            // 16-byte granules per row-major LDS row
    static constexpr int OPB = BT * KSB;           // bytes of one operand's stage
    static constexpr int LP = OPB / (1024 * NW);   // direct-to-LDS loads per wave, operand and stage
    static constexpr int BYTES = 5 * OPB;          // the two rings
    static_assert(SUBS % 2 == 0 && LP >= 1 && OPB % (1024 * NW) == 0 && 2 * LP <= 63, "pipeline shape");
};

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Block barrier between main-loop stages.  __syncthreads() is a workgroup
// release fence and waits for every outstanding vector-memory load
// (vmcnt(0)), which would also wait for look-ahead loads of later stages;
// the loads a stage needs are waited for explicitly (wait_vmcnt) before it,
// so this barrier only waits for the wave's LDS reads (the slot they read
// may be refilled after it).
__device__ __forceinline__ void stage_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// s_waitcnt vmcnt(VM) lgkmcnt(LGKM) through the builtin (gfx9 encoding:
// vmcnt bits 3:0 and 15:14, expcnt 6:4, lgkmcnt 11:8), so the compiler's own
// wait insertion knows which reads have returned; an inline-asm wait is
// invisible to it and it then adds a full wait of its own at the next use.
template <int VM, int LGKM>
__device__ __forceinline__ void waitcnt_seen() {
    static_assert(VM >= 0 && VM <= 63 && LGKM >= 0 && LGKM <= 15, "waitcnt range");
    __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4) | (LGKM << 8));
}

// Direct-to-LDS load of 16 bytes per lane (buffer resource words rs in
// scalar registers, LDS destination lds_addr in M0) issued through inline
// assembly.  The compiler cannot tell its LDS reads from the LDS writes of
// an outstanding direct-to-LDS load when the reads are the transposing
// ones, and then waits for every outstanding load before each such read,
// look-ahead loads included; loads it does not see are not ordered that way.
// Completion is the caller's explicit vmcnt wait.  Nothing else in the
// kernels that use it keeps a value in M0 (checked in the generated code);
// the hazard after writing M0 takes one wait state.
typedef int i32x4_t __attribute__((ext_vector_type(4)));
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16_unseen(i32x4_t rs, uint32_t lds_addr, uint32_t voff, int soff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds_addr), "v"(voff),
                 "s"(rs), "s"(soff)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

}  // namespace
}  // namespace mfsdp
