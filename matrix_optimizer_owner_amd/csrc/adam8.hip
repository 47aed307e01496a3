// adam8.hip - AdamW with its moments in 8 bits, and those moments as values.
//
// A group of 128 consecutive elements of a tensor shares two fp32 scales, the
// largest magnitude of the first moment m and of the second's root r = sqrt(v)
// in it.  Each is held as the square of a whole number times its scale,
//
//   m = scale_m * c |c| / 127^2,  c in -127 .. 127;
//   r = scale_r * (d / 255)^2,    d in 0 .. 255;  v = r^2,
//
// so steps are finest where values are small: next to the group's largest
// value they are 1.6% (m) and 0.8% (r) of it, and the smallest value held is
// 6e-5 (m) and 1.5e-5 (r) of it, where even steps of 1/127 would round m of a
// group with one large element to zero or to many times its size.  A group's
// largest value is its scale, exactly.  d is at least 1 where r > 0: a second
// moment that rounded to 0 beside a first one that did not would give an
// update of m / eps.
//
// The step rounds a code down after adding a dither in (0, 1) that step,
// tensor and element fix.  With beta2 = 0.999 a step moves v by
// about 0.1%, a tenth of half a code step: rounded to nearest it would never
// move at all; with the dither its mean does.  A moment that stays the same
// share of its scale keeps its code (the dither keeps 1/512 away from 0 and
// 1, over 60 times the fp32 error of the share), so in idle rows only scales
// move, by the betas and fp32 roundings.
//
// A group with a moment that is not finite gets the scale NaN and is NaN from
// then on.  Moments are formed in fp32 as the 32-bit step forms them, but r is
// held and not v, and small values are squared at 2^100 times their size, so
// that gradients down to the fp32 range's end have a second moment: within a
// few roundings, or half of 2^-149 each where values are subnormal.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "device_util.h"
#include "kernels.h"
#include "plan_internal.h"

namespace mfsdp {
namespace {

constexpr int kPer = 8;                         // consecutive elements of a thread
constexpr int kThreads = kTailChunk / kPer;     // of a block, which owns one chunk
constexpr int kLanes = kGroup / kPer;           // lanes of a group: one DPP row
static_assert(kLanes == 16, "a group's reduction stays inside 16 lanes");
constexpr int64_t kBlocksMax = (int64_t(1) << 32) / kThreads - 1;  // a launch has fewer than 2^32 threads

typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));

// kPer elements as fp32, from whole vectors past the caches (bf16 or fp32).
template <int D> __device__ __forceinline__ void load8(const void* p, float (&v)[kPer]) {
    if constexpr (D == kBF16) {
        const u32x4_t r = __builtin_nontemporal_load(static_cast<const u32x4_t*>(p));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[2 * k] = __uint_as_float(r[k] << 16);
            v[2 * k + 1] = __uint_as_float(r[k] & 0xffff0000u);
        }
    } else {
        const f32x4_t a = __builtin_nontemporal_load(static_cast<const f32x4_t*>(p));
        const f32x4_t b = __builtin_nontemporal_load(static_cast<const f32x4_t*>(p) + 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = a[k];
            v[4 + k] = b[k];
        }
    }
}
template <int D> __device__ __forceinline__ void store8(void* p, const float (&v)[kPer]) {
    if constexpr (D == kBF16) {
        __builtin_nontemporal_store(u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7])},
                                    static_cast<u32x4_t*>(p));
    } else {
        __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, static_cast<f32x4_t*>(p));
        __builtin_nontemporal_store(f32x4_t{v[4], v[5], v[6], v[7]}, static_cast<f32x4_t*>(p) + 1);
    }
}
// The first `n` of kPer elements, the others 0; whole vectors where n allows.
template <int D> __device__ __forceinline__ void load_n(const uint8_t* base, int64_t i, int n, float (&v)[kPer]) {
    if (n == kPer) {
        load8<D>(base + i * (D == kBF16 ? 2 : 4), v);
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = k < n ? load_elem(base, D, i + k) : 0.f;
    }
}
template <int D> __device__ __forceinline__ void store_n(uint8_t* base, int64_t i, int n, const float (&v)[kPer]) {
    if (n == kPer) {
        store8<D>(base + i * (D == kBF16 ? 2 : 4), v);
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (k < n) store_elem(base, D, i + k, v[k]);
    }
}

// Largest of a word over the 16 lanes of a group, in every lane: four DPP row
// rotations, no LDS.
template <int CTRL> __device__ __forceinline__ uint32_t max_rotated(uint32_t x) {
    return max(x, uint32_t(__builtin_amdgcn_mov_dpp(int(x), CTRL, 0xf, 0xf, false)));
}
__device__ __forceinline__ uint32_t group_max(uint32_t x) {
    x = max_rotated<0x128>(x);  // row_ror:8
    x = max_rotated<0x124>(x);
    x = max_rotated<0x122>(x);
    return max_rotated<0x121>(x);
}

// The finaliser of MurmurHash3 (Austin Appleby, public domain).
__device__ __forceinline__ uint32_t mix(uint32_t h) {
    h = (h ^ (h >> 16)) * 0x85ebca6bu;
    h = (h ^ (h >> 13)) * 0xc2b2ae35u;
    return h ^ (h >> 16);
}

// A group's scale and what its codes are formed with.  Magnitudes are compared
// as bit patterns, which orders them and puts Inf and NaN above the rest.
struct Scale {
    float value;      // stored: the largest magnitude, NaN where one is not finite
    float pre, inv;   // |x| * pre * inv is |x| / value; pre keeps 1 / value a normal number, and is 0 with a NaN
};
__device__ __forceinline__ Scale group_scale(const float (&x)[kPer]) {
    uint32_t most = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) most = max(most, __float_as_uint(x[k]) & 0x7fffffffu);
    most = group_max(most);
    Scale s;
    s.value = most < 0x7f800000u ? __uint_as_float(most) : __uint_as_float(0x7fc00000u);
    s.pre = s.value > 0x1p100f ? 0x1p-30f : s.value < 0x1p-90f && s.value > 0.f ? 0x1p60f : s.value >= 0.f ? 1.f : 0.f;
    const float v = s.value * s.pre;
    s.inv = v > 0.f ? __builtin_amdgcn_rcpf(v) : 0.f;
    return s;
}

// Code of a magnitude in bits 8 and up.  DITHER: floor(256 * count * sqrt(|x| /
// value) + 1/2) + byte, whose 256th part rounded down is the code with the
// dither (byte + 1/2) / 256; else without the 1/2, so that byte 128 gives the
// nearest code.  The root is at most 1 + 2^-22: no code exceeds count.
// PRE: the scale's pre is not 1 somewhere in the wave.  A group that is NaN
// has shares of 0: what is no number has no code.
template <bool DITHER, bool PRE>
__device__ __forceinline__ uint32_t code_of(float x, const Scale& s, float count, uint32_t byte) {
    const float share = !PRE ? fabsf(x) * s.inv : s.pre > 0.f ? fabsf(x) * s.pre * s.inv : 0.f;
    return uint32_t(__builtin_fmaf(__builtin_amdgcn_sqrtf(share), 256.f * count, DITHER ? 0.5f : 0.f)) + byte;
}

// Both moments' codes; word: the dither's 32 bits of elements 2j and 2j + 1.
struct Packed {
    u32x2_t first, root;
};
template <bool DITHER, bool PRE>
__device__ __forceinline__ Packed pack_codes(const float (&m)[kPer], const Scale& sm, const float (&r)[kPer], const Scale& sr,
                                             const uint32_t (&word)[kPer / 2]) {
    Packed p;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t c[4], d[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = h * 4 + j;
            const uint32_t w = word[k / 2];
            const int sign = __float_as_int(m[k]) >> 31;
            const uint32_t v = code_of<DITHER, PRE>(m[k], sm, 127.f, (w >> (16 * (k & 1))) & 0xff);
            c[j] = uint32_t((int(v >> 8 & 0xff) ^ sign) - sign);
            d[j] = max(code_of<DITHER, PRE>(r[k], sr, 255.f, (w >> (16 * (k & 1) + 8)) & 0xff), r[k] > 0.f ? 256u : 0u);
        }
        p.first[h] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[3], c[2], 0x0c0c0400), __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400), 0x05040100);
        p.root[h] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(d[3], d[2], 0x0c0c0501), __builtin_amdgcn_perm(d[1], d[0], 0x0c0c0501), 0x05040100);
    }
    return p;
}
template <bool DITHER>
__device__ __forceinline__ Packed pack(const float (&m)[kPer], const Scale& sm, const float (&r)[kPer], const Scale& sr,
                                       const uint32_t (&word)[kPer / 2]) {
    if (__any(sm.pre != 1.f || sr.pre != 1.f)) return pack_codes<DITHER, true>(m, sm, r, sr, word);
    return pack_codes<DITHER, false>(m, sm, r, sr, word);
}
// A code's share first, then the scale: a group's largest value is its scale,
// bit for bit, since 16129 * fl(1/16129) and 65025 * fl(1/65025) round to 1, and
// no factor of a value is below the fp32 range's normal numbers unless the value
// is.  (scale / 16129 first would save a product a value, and is subnormal from
// 1.9e-34 down.)
__device__ __forceinline__ void unpack_first(u32x2_t w, float scale, float (&m)[kPer]) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const float c = float(int8_t(w[k >> 2] >> (8 * (k & 3))));
        m[k] = c * fabsf(c) * (1.f / 16129.f) * scale;
    }
}
__device__ __forceinline__ void unpack_root(u32x2_t w, float scale, float (&r)[kPer]) {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const float d = float(uint8_t(w[k >> 2] >> (8 * (k & 3))));
        r[k] = d * d * (1.f / 65025.f) * scale;
    }
}

// Where one moment of a tensor lies in the state (Codes).
struct Place {
    uint8_t* codes;
    float* scales;
};
__device__ __forceinline__ Place place(uint8_t* state, uint64_t off, int64_t numel) {
    const uint64_t pad = (uint64_t(numel) + kAlign - 1) / kAlign * kAlign;
    return Place{state + off, reinterpret_cast<float*>(state + off + pad)};
}

struct Adam8Args {
    const TailDesc* tails;
    const int32_t* tail_begin;
    int n_tail;
    int first_chunk;           // the launch's first chunk
    uint32_t step;
    uint8_t* params;
    const uint8_t* grads;
    uint8_t* state;
    float b1, b2, omb1, omb2;  // betas and 1 - betas
    float root_bc2;            // sqrt(1/(1 - beta2^t))
    float lr_bc1;              // lr/(1 - beta1^t)
    float lrwd, eps;
    const float* gscale;       // SCALED kernel: the factor of every gradient
};

// One chunk of a tensor by a block, 8 consecutive elements a thread, a group
// by 16 lanes; every lane takes part in its group's reduction, with zeros
// behind the tensor's end.  Codes behind the end are written as zeros, inside
// the tensor's own code bytes.  WHOLE: the chunk has no such end.
// HBM: 10 bytes of a bf16 element and 14 of an fp32 one, 16 a group; 525 M bf16
// elements in 830 - 990 us (5.4 - 6.4 TB/s, by machine; in 32 bits 22 bytes,
// 1919 us), and next to it the codes' arithmetic, 8 elements a thread so that
// roots, reciprocals and hashes of neighbours overlap.
template <int D, bool SCALED, bool WHOLE>
__device__ __forceinline__ void step_chunk(const Adam8Args& a, const TailDesc& t, int64_t begin) {
    float gs = 1.f;
    if constexpr (SCALED) gs = *a.gscale;
    uint8_t* w = a.params + t.param_off;
    const uint8_t* g = a.grads + t.param_off;
    const Place pm = place(a.state, t.m1_off, t.numel), pr = place(a.state, t.m2_off, t.numel);
    const int64_t i = begin + int64_t(threadIdx.x) * kPer;
    const int n = WHOLE ? kPer : int(min(max(t.numel - i, int64_t(0)), int64_t(kPer)));
    float gv[kPer] = {}, wv[kPer] = {}, m[kPer] = {}, r[kPer] = {};
    if (n > 0) {
        load_n<D>(g, i, n, gv);
        load_n<D>(w, i, n, wv);
        const u32x2_t cm = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(pm.codes + i));
        const u32x2_t cr = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(pr.codes + i));
        unpack_first(cm, pm.scales[i / kGroup], m);
        unpack_root(cr, pr.scales[i / kGroup], r);
    }
    // behind the end g, m and r are zeros (codes there are written as zeros; the state is zero-filled at first)
    uint32_t least = ~0u;  // of the magnitudes that are not zero, as a bit pattern less 1
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if constexpr (SCALED) gv[k] *= gs;
        if (!WHOLE && k >= n) m[k] = r[k] = 0.f;
        m[k] = __builtin_fmaf(a.b1, m[k], a.omb1 * gv[k]);
        least = min(least, __float_as_uint(fmaxf(r[k], fabsf(gv[k]))) - 1);
    }
    if (__any(least < __float_as_uint(0x1p-40f) - 1)) {
        // small values are squared at 2^100 times their size: the least there is, 2^-149, has a normal square
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const bool small = fmaxf(r[k], fabsf(gv[k])) < 0x1p-40f;
            const float up = small ? 0x1p100f : 1.f, rk = r[k] * up, gk = gv[k] * up;
            r[k] = __builtin_amdgcn_sqrtf(__builtin_fmaf(a.b2, rk * rk, a.omb2 * (gk * gk))) * (small ? 0x1p-100f : 1.f);
        }
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            r[k] = __builtin_amdgcn_sqrtf(__builtin_fmaf(a.b2, r[k] * r[k], a.omb2 * (gv[k] * gv[k])));
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        // sqrt and reciprocal to 1 ulp each: 2e-7 of an update that is rounded with the parameter
        const float upd = m[k] * __builtin_amdgcn_rcpf(__builtin_fmaf(r[k], a.root_bc2, a.eps));
        wv[k] = __builtin_fmaf(-a.lr_bc1, upd, __builtin_fmaf(-a.lrwd, wv[k], wv[k]));
    }
    const Scale sm = group_scale(m), sr = group_scale(r);
    // one hashed word for two elements, a byte for each of their codes
    const uint32_t key = mix(a.step + 0x9e3779b9u * uint32_t(t.entry + 1));
    uint32_t word[kPer / 2];
#pragma unroll
    for (int j = 0; j < kPer / 2; ++j) {
        const uint64_t pair = uint64_t(i) / 2 + j;
        word[j] = mix(uint32_t(pair) + uint32_t(pair >> 32) * 0x9e3779b9u + key);
    }
    const Packed p = pack<true>(m, sm, r, sr, word);
    if (n <= 0) return;
    store_n<D>(w, i, n, wv);
    __builtin_nontemporal_store(p.first, reinterpret_cast<u32x2_t*>(pm.codes + i));
    __builtin_nontemporal_store(p.root, reinterpret_cast<u32x2_t*>(pr.codes + i));
    if (threadIdx.x % kLanes == 0) {
        pm.scales[i / kGroup] = sm.value;
        pr.scales[i / kGroup] = sr.value;
    }
}

template <bool SCALED>
__global__ __launch_bounds__(kThreads) void k_adamw8(Adam8Args a) {
    const int chunk = a.first_chunk + int(blockIdx.x);
    const int ti = upper_index(a.tail_begin, a.n_tail, chunk);
    const TailDesc t = a.tails[ti];
    const int64_t begin = int64_t(chunk - a.tail_begin[ti]) * kTailChunk;
    const bool whole = begin + kTailChunk <= t.numel;
    if (t.dtype == kBF16)
        whole ? step_chunk<kBF16, SCALED, true>(a, t, begin) : step_chunk<kBF16, SCALED, false>(a, t, begin);
    else
        whole ? step_chunk<kF32, SCALED, true>(a, t, begin) : step_chunk<kF32, SCALED, false>(a, t, begin);
}

// ---- moments as values ----

struct MomentArgs {
    uint8_t* state;
    uint64_t m1_off, m2_off;
    int64_t numel;
    uint8_t* first;
    uint8_t* second;
    int64_t first_block;
};

// CODES: the state holds codes, else fp32 values.  D: type of the values.
// HBM: 39 M moments of each kind out of codes in 38 us as bf16 and into them
// from fp32 in 68 (6.1 and 5.9 TB/s).
template <int D, bool CODES>
__global__ __launch_bounds__(kThreads) void k_moments_read(MomentArgs a) {
    const int64_t i = (a.first_block + blockIdx.x) * kTailChunk + int64_t(threadIdx.x) * kPer;
    if (i >= a.numel) return;
    const int n = int(min(a.numel - i, int64_t(kPer)));
    float m[kPer], v[kPer];
    if constexpr (CODES) {
        const Place pm = place(a.state, a.m1_off, a.numel), pr = place(a.state, a.m2_off, a.numel);
        const u32x2_t cm = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(pm.codes + i));
        const u32x2_t cr = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(pr.codes + i));
        unpack_first(cm, pm.scales[i / kGroup], m);
        unpack_root(cr, pr.scales[i / kGroup], v);
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] *= v[k];
    } else {
        load_n<kF32>(a.state + a.m1_off, i, n, m);
        load_n<kF32>(a.state + a.m2_off, i, n, v);
    }
    store_n<D>(a.first, i, n, m);
    store_n<D>(a.second, i, n, v);
}

template <int D, bool CODES>
__global__ __launch_bounds__(kThreads) void k_moments_write(MomentArgs a) {
    const int64_t i = (a.first_block + blockIdx.x) * kTailChunk + int64_t(threadIdx.x) * kPer;
    const int n = int(min(max(a.numel - i, int64_t(0)), int64_t(kPer)));
    float m[kPer] = {}, v[kPer] = {};
    if (n > 0) {
        load_n<D>(a.first, i, n, m);
        load_n<D>(a.second, i, n, v);
    }
    if constexpr (CODES) {
        const Place pm = place(a.state, a.m1_off, a.numel), pr = place(a.state, a.m2_off, a.numel);
#pragma unroll
        for (int k = 0; k < kPer; ++k) v[k] = sqrtf(v[k]);  // correctly rounded: the root of a square is the value again
        const Scale sm = group_scale(m), sr = group_scale(v);
        const uint32_t half[kPer / 2] = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};
        const Packed p = pack<false>(m, sm, v, sr, half);
        if (n <= 0) return;
        __builtin_nontemporal_store(p.first, reinterpret_cast<u32x2_t*>(pm.codes + i));
        __builtin_nontemporal_store(p.root, reinterpret_cast<u32x2_t*>(pr.codes + i));
        if (threadIdx.x % kLanes == 0) {
            pm.scales[i / kGroup] = sm.value;
            pr.scales[i / kGroup] = sr.value;
        }
    } else {
        if (n <= 0) return;
        store_n<kF32>(a.state + a.m1_off, i, n, m);
        store_n<kF32>(a.state + a.m2_off, i, n, v);
    }
}

template <bool READ, int D> void launch_moments(MomentArgs a, bool codes, hipStream_t stream) {
    const int64_t blocks = (a.numel + kTailChunk - 1) / kTailChunk;
    for (a.first_block = 0; a.first_block < blocks; a.first_block += kBlocksMax) {
        const dim3 grid(uint32_t(std::min(blocks - a.first_block, kBlocksMax)));
        if (READ)
            codes ? k_moments_read<D, true><<<grid, dim3(kThreads), 0, stream>>>(a)
                  : k_moments_read<D, false><<<grid, dim3(kThreads), 0, stream>>>(a);
        else
            codes ? k_moments_write<D, true><<<grid, dim3(kThreads), 0, stream>>>(a)
                  : k_moments_write<D, false><<<grid, dim3(kThreads), 0, stream>>>(a);
    }
}

template <bool READ>
mfsdp_status moments(mfsdp_plan_t plan, int64_t entry, const mfsdp_moments_args* args) {
    clear_error();
    if (!plan || !args) return fail(MFSDP_ERR_INVALID_ARGUMENT, "NULL plan or args");
    if (entry < 0 || entry >= int64_t(plan->entries.size()))
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "entry index out of range");
    if (args->type != MFSDP_F32 && args->type != MFSDP_BF16)
        return fail(MFSDP_ERR_UNSUPPORTED, "type must be MFSDP_F32 or MFSDP_BF16");
    const mfsdp_entry_info& inf = plan->info[size_t(entry)];
    if (inf.role == -1) return MFSDP_OK;  // an empty shard
    if (inf.role != MFSDP_ROLE_ADAMW && inf.role != MFSDP_ROLE_ADAMW8)
        return fail(MFSDP_ERR_UNSUPPORTED, "entry " + std::to_string(entry) + " has no AdamW moments");
    if (!args->state || reinterpret_cast<uintptr_t>(args->state) % kAlign != 0)
        return fail(MFSDP_ERR_INVALID_ARGUMENT, "state is NULL or not 256-byte aligned");
    for (const void* p : {args->first, args->second})
        if (!p || reinterpret_cast<uintptr_t>(p) % 16 != 0)
            return fail(MFSDP_ERR_INVALID_ARGUMENT, "first or second is NULL or not 16-byte aligned");
    MomentArgs a = {};
    a.state = static_cast<uint8_t*>(args->state);
    a.m1_off = inf.state_offset;
    a.m2_off = inf.state_offset2;
    a.numel = plan->entries[size_t(entry)].rows * plan->entries[size_t(entry)].cols;
    a.first = static_cast<uint8_t*>(args->first);
    a.second = static_cast<uint8_t*>(args->second);
    const bool codes = inf.role == MFSDP_ROLE_ADAMW8;
    hipStream_t stream = static_cast<hipStream_t>(args->stream);
    if (args->type == MFSDP_BF16)
        launch_moments<READ, kBF16>(a, codes, stream);
    else
        launch_moments<READ, kF32>(a, codes, stream);
    if (hipError_t e = hipGetLastError(); e != hipSuccess)
        return fail(MFSDP_ERR_HIP, std::string("moments launch: ") + hipGetErrorString(e));
    return MFSDP_OK;
}

}  // namespace

hipError_t launch_adamw8(const WorkspaceMap& map, const mfsdp_hparams& hp, int64_t step, const StepBuffers& b,
                         hipStream_t stream) {
    Adam8Args a = {};
    a.tails = reinterpret_cast<const TailDesc*>(b.ws + map.off_tail8);
    a.tail_begin = reinterpret_cast<const int32_t*>(b.ws + map.off_tail8_begin);
    a.n_tail = map.n_tail8;
    a.step = uint32_t(uint64_t(step));
    a.params = b.params;
    a.grads = b.grads;
    a.state = b.state;
    a.b1 = hp.adam_beta1;
    a.b2 = hp.adam_beta2;
    a.omb1 = float(1.0 - double(hp.adam_beta1));
    a.omb2 = float(1.0 - double(hp.adam_beta2));
    a.root_bc2 = float(1.0 / std::sqrt(1.0 - std::pow(double(hp.adam_beta2), double(step))));
    a.lr_bc1 = float(double(hp.adam_lr) / (1.0 - std::pow(double(hp.adam_beta1), double(step))));
    a.lrwd = float(double(hp.adam_lr) * double(hp.adam_weight_decay));
    a.eps = hp.adam_eps;
    a.gscale = b.grad_scale;
    for (int64_t first = 0; first < map.n_tail8_chunks; first += kBlocksMax) {
        a.first_chunk = int(first);
        const dim3 grid(uint32_t(std::min(map.n_tail8_chunks - first, kBlocksMax)));
        if (a.gscale)
            k_adamw8<true><<<grid, dim3(kThreads), 0, stream>>>(a);
        else
            k_adamw8<false><<<grid, dim3(kThreads), 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace mfsdp

extern "C" mfsdp_status mfsdp_moments_read(mfsdp_plan_t plan, int64_t entry, const mfsdp_moments_args* args) {
    return mfsdp::moments<true>(plan, entry, args);
}

extern "C" mfsdp_status mfsdp_moments_write(mfsdp_plan_t plan, int64_t entry, const mfsdp_moments_args* args) {
    return mfsdp::moments<false>(plan, entry, args);
}
