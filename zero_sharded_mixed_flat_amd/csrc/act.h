// Device and host helpers of the 8-bit activation checkpoints, shared by
// act.hip (checkpoint, gated activation, norm) and act_grad.hip (weight
// gradient).  The format is defined in include/zero_flat.h.
#pragma once

#include "device.h"

namespace zf {
namespace {

constexpr int kActBlock = ZERO_QBLOCK;
// A lane handles an oct: 8 consecutive elements of a row starting at a multiple
// of 8 (16 bytes of 16-bit values, 8 code bytes).  Half a wave holds one
// quantisation block.
constexpr int kOct = 8;
constexpr int kOctsPerBlock = kActBlock / kOct;
static_assert(kOctsPerBlock == 32, "a quantisation block is half a wave of octs");

// Rows of 16-bit matrices start at any 2-byte address.  gfx950 reads and
// writes global memory at any alignment (the compiler's unaligned access mode
// is on for this target), so an oct is always one 16-byte access.
typedef u4 u4_any __attribute__((aligned(2)));
typedef u2 u2_any __attribute__((aligned(2)));
typedef uint32_t u1_any __attribute__((aligned(2)));
typedef float f2 __attribute__((ext_vector_type(2)));

// The last oct of a row, n < 8 elements, in pieces of 4, 2 and 1; the rest of
// the oct reads as zero.
__device__ __forceinline__ u4 load_short_oct(const uint16_t* p, int n) {
    u2 a{0u, 0u};
    uint32_t b = 0, c = 0;
    if (n & 4) a = *reinterpret_cast<const u2_any*>(p);
    if (n & 2) b = *reinterpret_cast<const u1_any*>(p + (n & 4));
    if (n & 1) c = p[n & 6];
    const u2 t = (n & 2) ? u2{b, c} : u2{c, 0u};
    return (n & 4) ? u4{a.x, a.y, t.x, t.y} : u4{t.x, t.y, 0u, 0u};
}

// The oct of elements c.. of a row of `cols` (c < cols), read once: a streaming load.
__device__ __forceinline__ u4 load_oct(const uint16_t* row, int c, int cols) {
    if (c + kOct <= cols) return __builtin_nontemporal_load(reinterpret_cast<const u4_any*>(row + c));
    return load_short_oct(row + c, cols - c);
}

// As load_oct, for arrays that other blocks read too (no streaming hint).
__device__ __forceinline__ u4 load_oct_shared(const uint16_t* row, int c, int cols) {
    if (c + kOct <= cols) return *reinterpret_cast<const u4_any*>(row + c);
    return load_short_oct(row + c, cols - c);
}

__device__ __forceinline__ void store_oct(uint16_t* row, int c, int cols, const u4& w) {
    if (c + kOct <= cols) {
        __builtin_nontemporal_store(w, reinterpret_cast<u4_any*>(row + c));
        return;
    }
    const int n = cols - c;
    uint16_t* p = row + c;
    const u2 t = (n & 4) ? u2{w.z, w.w} : u2{w.x, w.y};
    if (n & 4) *reinterpret_cast<u2_any*>(p) = u2{w.x, w.y};
    if (n & 2) *reinterpret_cast<u1_any*>(p + (n & 4)) = t.x;
    if (n & 1) p[n & 6] = static_cast<uint16_t>((n & 2) ? t.y : t.x);
}

template <int DT>
__device__ __forceinline__ void widen_oct(const u4& w, float (&v)[kOct]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (DT == ZERO_BF16) {
            v[2 * k] = __uint_as_float(w[k] << 16);
            v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        } else {
            v[2 * k] = widen<DT>(w[k] & 0xffffu);
            v[2 * k + 1] = widen<DT>(w[k] >> 16);
        }
    }
}

// Two fp32 values rounded to nearest even into a packed pair (the hardware
// conversions; a NaN stays a NaN).
template <int DT>
__device__ __forceinline__ uint32_t narrow_pair(float a, float b) {
    if constexpr (DT == ZERO_BF16) {
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
    } else {
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, h2));
    }
}

template <int DT>
__device__ __forceinline__ u4 narrow_oct(const float (&v)[kOct]) {
    return u4{narrow_pair<DT>(v[0], v[1]), narrow_pair<DT>(v[2], v[3]), narrow_pair<DT>(v[4], v[5]),
              narrow_pair<DT>(v[6], v[7])};
}

// ---------------------------------------------------------------------------
// 8-bit blocks
// ---------------------------------------------------------------------------

template <int FMT>
constexpr float act_qmax() {
    return FMT == ZERO_ACT_INT8 ? 127.0f : 448.0f;
}

// Larger of two packed pairs of unsigned 16-bit values, half by half.
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
    typedef uint16_t s2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t,
                              __builtin_elementwise_max(__builtin_bit_cast(s2, a), __builtin_bit_cast(s2, b)));
}

// Scale of the block whose octs the 32 lanes of this half-wave hold: sign-free
// 16-bit patterns order like their magnitudes, with infinity and NaN above
// every finite value, so one integer maximum finds both the largest magnitude
// and a non-finite value (-> NaN).
template <int DT, int FMT>
__device__ __forceinline__ float block_scale(const u4& w) {
    uint32_t m = max_pair(max_pair(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                          max_pair(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    for (int off = 16; off > 0; off >>= 1) m = max_pair(m, __shfl_xor(m, off, 64));
    const uint32_t top = max(m & 0xffffu, m >> 16);
    if (!finite16<DT>(top)) return __uint_as_float(0x7fc00000u);
    return widen<DT>(top) / act_qmax<FMT>();
}

// Codes of an oct.  With y = 1 / scale correctly rounded, q0 = x y and one
// correction q = q0 + (x - q0 scale) y give the IEEE quotient wherever the code
// depends on its last bit: scale is A / qmax rounded, with A a 16-bit value
// (an 11-bit significand at most), so x / scale = qmax x / A (1 + e),
// |e| <= 2^-24, lies either at least 2^-19 (relative; 2^-16 for bf16 or E4M3) from
// every rounding boundary of the code or, but for e, on one; those finitely many
// cases are compared exhaustively by the tests.  This is 3 operations instead of about 10
// for a division, whose cost would exceed the memory time of the kernel.  Below
// 2^-60 (reached by bf16 blocks of magnitudes under 1e-16 only) the residual may
// leave the normal range and the division itself is used.  An INT8 code is the
// low byte of q + 1.5 * 2^23: the sum rounds q to an integer, ties to even.
template <int FMT>
__device__ __forceinline__ u2 encode_oct(const float (&v)[kOct], float scale) {
    float q[kOct];
    if (scale > 0x1p-60f) {
        const float y = 1.0f / scale;
#pragma unroll
        for (int k = 0; k < kOct; ++k) {
            const float q0 = v[k] * y;
            q[k] = __builtin_fmaf(__builtin_fmaf(-q0, scale, v[k]), y, q0);
            // -0 comes out of the correction as +0; INT8 has no sign of zero
            if constexpr (FMT == ZERO_ACT_E4M3) q[k] = __builtin_copysignf(q[k], v[k]);
        }
    } else if (scale > 0.0f) {
#pragma unroll
        for (int k = 0; k < kOct; ++k)
            q[k] = fminf(fmaxf(v[k] / scale, -act_qmax<FMT>()), act_qmax<FMT>());
    } else {  // a block of zeros, or a NaN scale
        return u2{0u, 0u};
    }
    u2 out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if constexpr (FMT == ZERO_ACT_INT8) {
            uint32_t b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) b[k] = __float_as_uint(q[4 * h + k] + 12582912.0f);
            const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
            const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
            out[h] = lo | hi;
        } else {
            int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], w, true);
            out[h] = static_cast<uint32_t>(w);
        }
    }
    return out;
}

// Four codes of a word as fp32.
template <int FMT>
__device__ __forceinline__ void decode_word(uint32_t w, float (&v)[4]) {
    if constexpr (FMT == ZERO_ACT_INT8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = static_cast<float>(static_cast<int>(w << (24 - 8 * k)) >> 24);
    } else {
        const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
        const f2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
        v[0] = a.x;
        v[1] = a.y;
        v[2] = b.x;
        v[3] = b.y;
    }
}

// The restored 16-bit oct: round16(code * scale).
template <int DT, int FMT>
__device__ __forceinline__ u4 decode_oct(const u2& codes, float scale) {
    u4 out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float v[4];
        decode_word<FMT>(codes[h], v);
        out[2 * h] = narrow_pair<DT>(v[0] * scale, v[1] * scale);
        out[2 * h + 1] = narrow_pair<DT>(v[2] * scale, v[3] * scale);
    }
    return out;
}

__device__ __forceinline__ void store_codes(uint8_t* row, int c, const u2& w) {
    __builtin_nontemporal_store(w, reinterpret_cast<u2*>(row + c));
}

__device__ __forceinline__ u2 load_codes(const uint8_t* row, int c) {
    return __builtin_nontemporal_load(reinterpret_cast<const u2*>(row + c));
}

// n / d for n < 2^31 by a multiplication: shift = ceil(log2 d), mult =
// ceil(2^(31 + shift) / d) < 2^32 exceeds the true ratio by less than d <= 2^shift,
// so n times the excess stays below 2^(31 + shift) and the quotient is exact.
struct FastDiv {
    uint32_t d, mult, shift;
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        return static_cast<uint32_t>((uint64_t(n) * mult) >> (31 + shift));
    }
};

inline FastDiv fast_div(uint32_t d) {
    uint32_t s = 0;
    while ((uint64_t(1) << s) < d) ++s;
    const uint64_t m = ((uint64_t(1) << (31 + s)) + d - 1) / d;
    return FastDiv{d, static_cast<uint32_t>(m), s};
}

// ---------------------------------------------------------------------------
// Host-side checks
// ---------------------------------------------------------------------------

inline int64_t act_pitch(int64_t cols) { return ceil_div(cols, 16) * 16; }
inline int64_t act_blocks(int64_t cols) { return ceil_div(cols, int64_t(kActBlock)); }

inline bool valid_format(int f) { return f == ZERO_ACT_INT8 || f == ZERO_ACT_E4M3; }

// rows * (cols rounded up to a block) within ZERO_MAX_ELEMS and cols within
// ZERO_ACT_MAX_COLS: block indices then fit 26 bits and columns an int.
inline bool act_size_ok(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || rows > ZERO_MAX_ELEMS || cols > ZERO_ACT_MAX_COLS) return false;
    if (rows == 0 || cols == 0) return true;
    return rows <= (ZERO_MAX_ELEMS / kActBlock) / act_blocks(cols);
}

// Largest distance from a matrix's first to its last element.
constexpr int64_t kMaxSpan = int64_t(1) << 52;

inline bool stride_ok(int64_t rows, int64_t cols, int64_t stride) {
    if (stride < cols) return false;
    return rows <= 1 || stride <= (kMaxSpan - cols) / (rows - 1);
}

// A region an argument covers: `rows` pieces of `row_bytes`, `pitch` bytes apart.
struct Area {
    const char* name;
    const void* p;
    int64_t rows, row_bytes, pitch;
    bool out;
};

inline Area mat16(const char* name, const void* p, int64_t rows, int64_t cols, int64_t stride, bool out) {
    return Area{name, p, rows, 2 * cols, 2 * stride, out};
}
inline Area flat(const char* name, const void* p, int64_t bytes, bool out) { return Area{name, p, 1, bytes, bytes, out}; }

// Whether two regions may share a byte.  Regions of equal pitch whose spans
// meet are compared column by column (interleaved halves of one matrix do not
// overlap); regions of unequal pitch whose spans meet count as overlapping.
inline bool areas_overlap(const Area& a, const Area& b) {
    if (a.p == nullptr || b.p == nullptr || a.rows <= 0 || b.rows <= 0 || a.row_bytes <= 0 || b.row_bytes <= 0)
        return false;
    const int64_t sa = (a.rows - 1) * a.pitch + a.row_bytes, sb = (b.rows - 1) * b.pitch + b.row_bytes;
    if (!overlaps(a.p, sa, b.p, sb)) return false;
    if ((a.rows == 1 && b.rows == 1) || a.pitch != b.pitch) return true;
    const uintptr_t s = uintptr_t(a.pitch);
    const uintptr_t d = addr(b.p) >= addr(a.p) ? (addr(b.p) - addr(a.p)) % s : (s - (addr(a.p) - addr(b.p)) % s) % s;
    return !(d >= uintptr_t(a.row_bytes) && d + uintptr_t(b.row_bytes) <= s);
}

// Every output against every other region; `same` names a pair that may be
// exactly the same region.
inline int check_overlaps(const char* fn, const Area* areas, int n, const char* same_out = "", const char* same_in = "") {
    for (int i = 0; i < n; ++i) {
        if (!areas[i].out) continue;
        for (int j = 0; j < n; ++j) {
            if (i == j || (areas[j].out && j < i) || !areas_overlap(areas[i], areas[j])) continue;
            const bool pair = std::string(areas[i].name) == same_out && std::string(areas[j].name) == same_in;
            if (pair && areas[i].p == areas[j].p && areas[i].pitch == areas[j].pitch) continue;
            return fail(ZERO_EALIAS, std::string(fn) + ": " + areas[i].name + " overlaps " + areas[j].name);
        }
    }
    return ZERO_OK;
}

inline bool bad_ptr(const void* p, int align) { return p == nullptr || (addr(p) & uintptr_t(align - 1)); }

// The checks every entry point starts with; a negative status has been reported.
inline int check_sizes(const char* fn, int64_t rows, int64_t cols, int dtype, int format) {
    if (!act_size_ok(rows, cols))
        return fail(ZERO_EINVAL, std::string(fn) + ": rows and cols must be >= 0, cols <= 2^30 and rows * (cols rounded "
                                                   "up to 256) <= 2^34");
    if (!valid_dtype(dtype)) return fail(ZERO_EINVAL, std::string(fn) + ": dtype must be ZERO_F16 or ZERO_BF16");
    if (!valid_format(format)) return fail(ZERO_EINVAL, std::string(fn) + ": format must be ZERO_ACT_INT8 or ZERO_ACT_E4M3");
    return ZERO_OK;
}

inline int check_matrix(const char* fn, const char* name, const void* p, int64_t rows, int64_t cols, int64_t stride) {
    if (bad_ptr(p, 2)) return fail(ZERO_EINVAL, std::string(fn) + ": " + name + " NULL or not 2-byte aligned");
    if (!stride_ok(rows, cols, stride))
        return fail(ZERO_EINVAL, std::string(fn) + ": " + name + "'s stride is less than cols or too large");
    return ZERO_OK;
}

inline int check_checkpoint(const char* fn, const char* name, const void* codes, const float* scales) {
    if (bad_ptr(codes, 16)) return fail(ZERO_EINVAL, std::string(fn) + ": " + name + "codes NULL or not 16-byte aligned");
    if (bad_ptr(scales, 4)) return fail(ZERO_EINVAL, std::string(fn) + ": " + name + "scales NULL or misaligned");
    return ZERO_OK;
}

inline const uint16_t* in16(const void* p) { return static_cast<const uint16_t*>(p); }
inline uint16_t* out16(void* p) { return static_cast<uint16_t*>(p); }
inline const uint8_t* in8(const void* p) { return static_cast<const uint8_t*>(p); }
inline uint8_t* out8(void* p) { return static_cast<uint8_t*>(p); }

// Calls f with the types as integral constants.
template <typename F>
hipError_t with_dtype(int dtype, F&& f) {
    if (dtype == ZERO_F16) return f(std::integral_constant<int, ZERO_F16>{});
    return f(std::integral_constant<int, ZERO_BF16>{});
}

template <typename F>
hipError_t with_types(int dtype, int format, F&& f) {
    return with_dtype(dtype, [&](auto dt) {
        if (format == ZERO_ACT_INT8) return f(dt, std::integral_constant<int, ZERO_ACT_INT8>{});
        return f(dt, std::integral_constant<int, ZERO_ACT_E4M3>{});
    });
}

}  // namespace
}  // namespace zf
