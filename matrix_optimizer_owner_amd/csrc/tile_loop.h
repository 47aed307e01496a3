// tile_loop.h - one output tile of a product C = P Q^T of two bf16 matrices in
// memory, on gfx950 MFMA: BT x BT per block of 4 waves, each with a
// BT/2 x BT/2 block of 32 x 32 MFMA tiles in registers.
//
// An operand is read in stages of 64 contraction indices, either
//   row-major: its rows are tile rows, contiguous along the contraction, or
//   K-major:   its rows are the contraction index, contiguous along tile rows.
// Both reach LDS by direct global->LDS loads of 16 bytes a lane into rings of
// stage slots, 3 for P and 2 for Q, whose rows are 128 bytes, swizzled on the
// global side; K-major is read back with the transposing LDS read.  Rows are
// 16-byte aligned.  In a plain matrix the 128-byte column blocks of a row follow
// one another; in one made for this loop each column block is a matrix of its
// own, its rows 128 bytes apart, so that a stage is one piece of memory (a
// K-major one 4 or 2), and a tile's stages do not sweep over the pages of the
// whole matrix.  Nothing past an
// operand's last row or last 128-byte column block is read: a load that would
// lie there reads the last one instead, and what it brings has to be
// multiplied by zeros (contraction) or left out (tile rows).
//
// An fp32 operand is three bf16 planes that add up to it exactly (bits 1-8,
// 9-16 and 17-24 of its significand).  A product of planes is exact in fp32,
// so with the pairs whose weights reach 2^-16, smallest first, a product of
// two fp32 operands takes 6 runs over the contraction and one of fp32 and bf16
// 3.  What is left out is under 2^-22 of a product's magnitude (values below
// 2^-109 lose bits under 2^-133, the smallest bf16).  Against
// v_mfma_f32_32x32x2_f32, 16 times slower than bf16, that is 2.7 and 5.3 times
// the rate.
#pragma once
#include <type_traits>

#include "mfma_util.h"

namespace mfsdp {
namespace {

struct Operand {
    const uint8_t* base;
    int64_t pitch;    // bytes from one row to the next
    int64_t block;    // bytes from one 128-byte column block of a row to the next
    int64_t rows;     // rows that may be read
    int blocks;       // column blocks that may be read
    int planes;       // 1 or 3; Q beside a P of one plane: also 2
    int64_t plane;    // bytes from one plane to the next
    // element (row, col), inside plane 0
    __device__ __forceinline__ const uint8_t* at(int64_t row, int col) const {
        return base + row * pitch + int64_t(col >> 6) * block + (col & 63) * 2;
    }
};

// The runs over the contraction: (plane of P, plane of Q) of each, 4 bits.
struct Runs {
    uint32_t list;
    int count;
    __device__ __forceinline__ Runs(int p, int q) {
        if (p == 1 && q == 1) {
            list = 0x0;
            count = 1;
        } else if (q == 1) {
            list = 0x012;
            count = 3;
        } else if (q == 2) {  // of one plane by two
            list = 0x04;
            count = 2;
        } else if (p == 1) {
            list = 0x048;
            count = 3;
        } else {  // (2,0) (1,1) (0,2) (1,0) (0,1) (0,0)
            list = 0x041852;
            count = 6;
        }
    }
    __device__ __forceinline__ int p(int run) const { return (list >> (4 * run)) & 3; }
    __device__ __forceinline__ int q(int run) const { return (list >> (4 * run + 2)) & 3; }
};

// One operand's loads: per-lane byte offsets from a stage's first byte, the
// same for every stage but a K-major operand's last, and where the next stage
// to be loaded lies (wave-uniform).
template <int BT, bool KM, bool IS_P>
struct StageLoads {
    using PP = Pipe<BT, 4>;
    static constexpr int LP = PP::LP;           // loads a wave and stage
    static constexpr int KST = PP::KSB / 2;     // contraction indices a stage
    const uint8_t* at;      // the stage to be loaded next
    const uint8_t* base;    // stage k0 of plane 0
    int64_t step, plane;    // bytes from one stage, one plane to the next
    int kt, run;
    uint32_t off[LP];       // lane's offset of load i
    int32_t back[LP];       // K-major: what the ragged stage's offsets differ by (<= 0)
    int ragged;             // the stage with rows past the end, or -1

    __device__ __forceinline__ void set(const Operand& o, const Runs& runs, int64_t row0, int k0, int lane, int wave) {
        if constexpr (KM) {
            step = int64_t(KST) * o.pitch;
            const int block0 = int(row0 / 64);
            base = o.base + k0 * step + block0 * o.block;
            const int last = int(o.rows % KST);
            ragged = last ? int(o.rows / KST) : -1;
#pragma unroll
            for (int i = 0; i < LP; ++i) {
                const int r = (i * 4 + wave) * 8 + (lane >> 3), blk = r / KST, k = r % KST;
                const uint32_t col = uint32_t(min(blk, o.blocks - 1 - block0)) * uint32_t(o.block) + uint32_t(swz_k(r, lane & 7)) * 16u;
                off[i] = uint32_t(k) * uint32_t(o.pitch) + col;
                back[i] = last && k >= last ? -int32_t(uint32_t(k - (last - 1)) * uint32_t(o.pitch)) : 0;
            }
        } else {
            step = o.block;
            base = o.base + row0 * o.pitch + k0 * step;
            ragged = -1;
            const int last = int(min(o.rows - row0, int64_t(BT))) - 1;
#pragma unroll
            for (int i = 0; i < LP; ++i) {
                const int r = (i * 4 + wave) * 8 + (lane >> 3);
                off[i] = uint32_t(min(r, last)) * uint32_t(o.pitch) + uint32_t(swz_r<8>(r, lane & 7)) * 16u;
                back[i] = 0;
            }
        }
        base = uni_ptr(base);
        plane = o.plane;
        kt = k0;
        run = 0;
        at = base + (IS_P ? runs.p(0) : runs.q(0)) * plane;
    }
    // to the next stage, of the next run after k1 - 1; the very last one stays
    __device__ __forceinline__ void next(const Runs& runs, int k0, int k1) {
        if (kt + 1 < k1) {
            ++kt;
            at += step;
        } else if (run + 1 < runs.count) {
            ++run;
            kt = k0;
            at = base + (IS_P ? runs.p(run) : runs.q(run)) * plane;
        }
    }
    __device__ __forceinline__ uint32_t offset(int i) const {
        if constexpr (KM) return off[i] + uint32_t(back[i] & (kt == ragged ? -1 : 0));
        return off[i];
    }
    // load i of the stage into LDS at `to`; UNSEEN: by dma16_unseen
    template <bool UNSEEN> __device__ __forceinline__ void load(int i, uint8_t* to) const {
        if constexpr (UNSEEN) {
            const uint64_t a = reinterpret_cast<uint64_t>(uni_ptr(at));
            const i32x4_t rs = {int(uint32_t(a)), int(uint32_t(a >> 32)), 0x7fffffff, kRsrcWord3};
            const uint32_t l = uint32_t(uni(int(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)to))));
            dma16_unseen(rs, l, offset(i), 0);
        } else {
            const __amdgpu_buffer_rsrc_t rs =
                __builtin_amdgcn_make_buffer_rsrc(uni_ptr(const_cast<uint8_t*>(at)), 0, 0x7fffffff, kRsrcWord3);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(to), 16, int(offset(i)), 0,
                                                     0, 0);
        }
    }
};

// acc <- P Q^T over stages [k0, k1) of the contraction, k0 < k1.  acc element e
// of MFMA tile (mi, ni) is tile row wm*BT/2 + 32*mi + 8*(e/4) + 4*(lane/32) +
// e%4, tile column wn*BT/2 + 32*ni + lane%32, where wm = wave/2, wn = wave%2.
// All loads have landed when it returns; the block's other waves may still
// read their LDS.
//
// The instruction order is fixed, as in the Newton-Schulz loop: a stage's four
// groups of MFMAs (the previous stage's last sub-step, then its own first
// three) carry the next sub-step's fragment reads and the stage's loads
// between them, Q of stage t+1 and P of stage t+2 into the slots that stage
// t-1 released; then a wave waits for its loads of stage t+1, all but its LP
// most recent, and the barrier makes every wave's visible.
template <bool PK, bool QK, int BT>
__device__ __forceinline__ void tile_loop(f32x16_t (&acc)[BT / 64][BT / 64], const Operand& P, const Operand& Q,
                                          int64_t row0, int64_t col0, int k0, int k1, uint8_t* lds) {
    using S = Shape<BT, 4>;
    using PP = Pipe<BT, 4>;
    using M = Mfma<uint16_t>;
    constexpr int MM = S::MM, MN = S::MN, LP = PP::LP, KSB = PP::KSB, OPB = PP::OPB;
    constexpr int KST = KSB / 2, CB = 64, GE = 8;
    constexpr bool kUnseen = PK || QK;  // the compiler waits for loads it sees before each transposing read
    constexpr int NF = MM * MN;                                 // MFMAs of a group
    constexpr int RP = (PK ? 2 : 1) * MM, NR = RP + (QK ? 2 : 1) * MN;  // LDS read instructions of a sub-step
    const int lane = threadIdx.x & 63, wave = uni(int(threadIdx.x) >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int frow = lane & 31, fhalf = lane >> 5;

    const Runs runs(P.planes, Q.planes);
    const int stages = runs.count * (k1 - k0);
    StageLoads<BT, PK, true> lp;
    StageLoads<BT, QK, false> lq;
    lp.set(P, runs, row0, k0, lane, wave);
    lq.set(Q, runs, col0, k0, lane, wave);

    auto load_p = [&](int i, int slot) { lp.template load<kUnseen>(i, lds + slot + (i * 4 + wave) * 1024); };
    auto load_q = [&](int i, int slot) { lq.template load<kUnseen>(i, lds + slot + (i * 4 + wave) * 1024); };
    // half h (contraction indices k..k+3, k+4..k+7 of the lane's) of a K-major fragment from tile row c on, sub-step kk
    auto kmajor_half = [&](int slot, int c, int kk, int h) -> u32x2_t {
        const int g16 = lane >> 4, sl = lane & 15;
        const int col = c + 16 * (g16 & 1) + 4 * (sl & 3);
        const int k = kk * 16 + 8 * (g16 >> 1) + (sl >> 2) + 4 * h;
        const int r = (col / CB) * KST + k;
        const int gr = (col % CB) / GE, e = (col % GE) * 2;
        return ds_read_tr16(lds + slot + r * 128 + swz_k(r, gr) * 16 + e);
    };
    auto rowmajor_frag = [&](int slot, int r, int kk) -> u32x4_t {
        return *reinterpret_cast<const u32x4_t*>(lds + slot + r * KSB + swz_r<8>(r, 2 * kk + fhalf) * 16);
    };
    // read instruction r of sub-step kk's fragments
    auto read_one = [&](int r, int oP, int oQ, int kk, u32x4_t (&fa)[MM], u32x4_t (&fb)[MN]) {
        if (r < RP) {
            if constexpr (PK) {
                const u32x2_t v = kmajor_half(oP, wm * S::WTM + (r >> 1) * 32, kk, r & 1);
                fa[r >> 1][2 * (r & 1)] = v[0];
                fa[r >> 1][2 * (r & 1) + 1] = v[1];
            } else {
                fa[r] = rowmajor_frag(oP, wm * S::WTM + r * 32 + frow, kk);
            }
        } else {
            const int s = r - RP;
            if constexpr (QK) {
                const u32x2_t v = kmajor_half(oQ, wn * S::WTN + (s >> 1) * 32, kk, s & 1);
                fb[s >> 1][2 * (s & 1)] = v[0];
                fb[s >> 1][2 * (s & 1) + 1] = v[1];
            } else {
                fb[s] = rowmajor_frag(oQ, wn * S::WTN + s * 32 + frow, kk);
            }
        }
    };
    using F0 = std::false_type;
    using F1 = std::true_type;
    // MFMA m of (fa, fb), FIRST: starting the accumulators, NONE: none; then side operations t with t*span/n == m
    auto group = [&](auto FIRST, auto NONE, const u32x4_t (&fa)[MM], const u32x4_t (&fb)[MN], int n, int span, auto&& side) {
#pragma unroll
        for (int m = 0; m < NF; ++m) {
            if constexpr (decltype(FIRST)::value)
                acc[m / MN][m % MN] = M::first(fa[m / MN], fb[m % MN]);
            else if constexpr (!decltype(NONE)::value)
                M::step(acc[m / MN][m % MN], fa[m / MN], fb[m % MN]);
#pragma unroll
            for (int t = 0; t < n; ++t)
                if (t * span / n == m) side(t);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

#pragma unroll
    for (int i = 0; i < LP; ++i) load_p(i, 0);
#pragma unroll
    for (int i = 0; i < LP; ++i) load_q(i, 3 * OPB);
    lp.next(runs, k0, k1);
    lq.next(runs, k0, k1);
#pragma unroll
    for (int i = 0; i < LP; ++i) load_p(i, OPB);
    lp.next(runs, k0, k1);
    waitcnt_seen<LP, 0>();
    __builtin_amdgcn_s_barrier();
    u32x4_t fa0[MM], fb0[MN], fa1[MM], fb1[MN];
#pragma unroll
    for (int r = 0; r < NR; ++r) read_one(r, 0, 3 * OPB, 0, fa0, fb0);
    __builtin_amdgcn_sched_barrier(0);
    int sp = 0, sq = 0;  // P and Q slots of the stage
    auto stage = [&](auto FIRST) {
        const int sp2 = sp == 0 ? 2 : sp - 1;
        const int oP = sp * OPB, oQ = (3 + sq) * OPB, oQn = (3 + (sq ^ 1)) * OPB, oPn = sp2 * OPB;
        constexpr int LP1 = LP / 2, LP2 = LP - LP1;
        group(F0{}, FIRST, fa1, fb1, LP, NF, [&](int t) { load_q(t, oQn); });
        group(FIRST, F0{}, fa0, fb0, NR + LP1, NF, [&](int t) {
            if (t < NR)
                read_one(t, oP, oQ, 1, fa1, fb1);
            else
                load_p(t - NR, oPn);
        });
        group(F0{}, F0{}, fa1, fb1, NR + LP2, NF, [&](int t) {
            if (t < NR)
                read_one(t, oP, oQ, 2, fa0, fb0);
            else
                load_p(LP1 + t - NR, oPn);
        });
        group(F0{}, F0{}, fa0, fb0, NR, NF / 2, [&](int t) { read_one(t, oP, oQ, 3, fa1, fb1); });
        lq.next(runs, k0, k1);
        lp.next(runs, k0, k1);
        waitcnt_seen<LP, 0>();
        __builtin_amdgcn_s_barrier();
        sp = sp == 2 ? 0 : sp + 1;
        sq ^= 1;
#pragma unroll
        for (int r = 0; r < NR; ++r) read_one(r, sp * OPB, (3 + sq) * OPB, 0, fa0, fb0);
        __builtin_amdgcn_sched_barrier(0);
    };
    stage(F1{});
    for (int s = 1; s < stages; ++s) stage(F0{});
#pragma unroll
    for (int m = 0; m < NF; ++m) M::step(acc[m / MN][m % MN], fa1[m / MN], fb1[m % MN]);
    wait_vmcnt<0>();
}

}  // namespace
}  // namespace mfsdp
