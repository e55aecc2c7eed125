// 8-bit activation checkpoints for MI355X (gfx950, wave64): the checkpoint
// itself, the gated activation and the residual norm that write and read it,
// and their C-ABI entry points.  The formulas are in include/zero_flat.h.
//
//   act_save_kernel / act_restore_kernel    16-bit matrix <-> codes + scales
//   glu_forward_kernel / glu_backward_kernel
//   norm_forward_kernel / norm_backward_kernel, fold_columns_kernel
//
// All of them stream: every array is read or written once, nothing is a
// contraction, and the bound is HBM (reads near 7 TB/s, writes near 6).
//
// Pages cited by short name:
//   L18 notes  CMU 11-868 Lecture 18 notes, "Memory Optimization in Distributed Training: ZeRO" (semidirectx.com)

#include "act.h"

namespace zf {
namespace {

// ---------------------------------------------------------------------------
// Block-wise streaming kernels: checkpoint and gated activation
// ---------------------------------------------------------------------------

// Quantisation blocks are numbered row by row; a wave takes PAIRS consecutive
// pairs of them, one block per half-wave, so a load of a wave covers one
// contiguous KiB of a row.
constexpr int kActWaves = 4;
constexpr int kActThreads = 64 * kActWaves;

struct Place {
    int64_t row;
    int col;  // first element of this lane's oct
    uint32_t block;
    bool live;
};

template <int PAIRS>
__device__ __forceinline__ Place place_of(int u, uint32_t nblocks, const FastDiv& per_row) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Place p;
    p.block = ((blockIdx.x * kActWaves + wave) * PAIRS + u) * 2 + (lane >> 5);
    p.live = p.block < nblocks;
    const uint32_t b = p.live ? p.block : 0u;
    const uint32_t row = per_row.div(b);
    p.row = row;
    p.col = int(b - row * per_row.d) * kActBlock + kOct * (lane & 31);
    return p;
}

inline dim3 act_grid(int64_t nblocks, int pairs) {
    return dim3{unsigned(ceil_div(nblocks, int64_t(2) * pairs * kActWaves))};
}

// Pairs of blocks per wave: 2 for large matrices (16384 x 16384: 128 us and 6.3 TB/s, with
// 1 154, with 4 130), 1 where the launch is all there is (one row of 1600: 2.2 us, with 2 2.8).
constexpr int64_t kSaveOnePair = 2048;  // up to as many blocks

template <int DT, int FMT, int PAIRS>
__global__ __launch_bounds__(kActThreads) void act_save_kernel(const uint16_t* __restrict__ x, int64_t stride,
                                                               int cols, uint32_t nblocks, FastDiv per_row,
                                                               uint8_t* __restrict__ codes, int64_t pitch,
                                                               float* __restrict__ scales) {
    u4 w[PAIRS];
    Place p[PAIRS];
#pragma unroll
    for (int u = 0; u < PAIRS; ++u) {
        p[u] = place_of<PAIRS>(u, nblocks, per_row);
        w[u] = u4{0u, 0u, 0u, 0u};
        if (p[u].live && p[u].col < cols) w[u] = load_oct(x + p[u].row * stride, p[u].col, cols);
    }
#pragma unroll
    for (int u = 0; u < PAIRS; ++u) {
        const float scale = block_scale<DT, FMT>(w[u]);
        if (!p[u].live) continue;
        float v[kOct];
        widen_oct<DT>(w[u], v);
        const u2 q = encode_oct<FMT>(v, scale);
        if ((threadIdx.x & 31) == 0) scales[p[u].block] = scale;
        if (p[u].col < pitch) store_codes(codes + p[u].row * pitch, p[u].col, q);
    }
}

constexpr int kRestorePairs = 2;  // 16384 x 16384: 127 us (6.4 TB/s), with 4 132

template <int DT, int FMT>
__global__ __launch_bounds__(kActThreads) void act_restore_kernel(const uint8_t* __restrict__ codes, int64_t pitch,
                                                                  const float* __restrict__ scales, int cols,
                                                                  uint32_t nblocks, FastDiv per_row,
                                                                  uint16_t* __restrict__ y, int64_t stride) {
    u2 q[kRestorePairs];
    float scale[kRestorePairs];
    Place p[kRestorePairs];
#pragma unroll
    for (int u = 0; u < kRestorePairs; ++u) {
        p[u] = place_of<kRestorePairs>(u, nblocks, per_row);
        p[u].live = p[u].live && p[u].col < cols;
        if (p[u].live) {
            q[u] = load_codes(codes + p[u].row * pitch, p[u].col);
            scale[u] = scales[p[u].block];
        }
    }
#pragma unroll
    for (int u = 0; u < kRestorePairs; ++u)
        if (p[u].live) store_oct(y + p[u].row * stride, p[u].col, cols, decode_oct<DT, FMT>(q[u], scale[u]));
}

// ---------------------------------------------------------------------------
// Activation functions
// ---------------------------------------------------------------------------

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }

// exp(a^2/2) P(-a) for a >= 0, with P the normal distribution function: t p(t),
// t = 1 / (1 + 0.32 a), with p a degree-7 polynomial fitted to it over t for the
// least largest relative error on [0, 60] (5.0e-7 with its coefficients in fp32, 8e-7
// evaluated in fp32).
__device__ __forceinline__ float normal_tail(float a) {
    const float t = rcp_hw(__builtin_fmaf(0.32f, a, 1.0f));
    float p = 0x1.1acb3cp-5f;
    p = __builtin_fmaf(p, t, -0x1.f57a54p-4f);
    p = __builtin_fmaf(p, t, 0x1.b2a5c6p-4f);
    p = __builtin_fmaf(p, t, 0x1.fed612p-7f);
    p = __builtin_fmaf(p, t, 0x1.8ed7dap-4f);
    p = __builtin_fmaf(p, t, 0x1.d0a53ep-4f);
    p = __builtin_fmaf(p, t, 0x1.05991ap-3f);
    p = __builtin_fmaf(p, t, 0x1.05728cp-3f);
    return t * p;
}

// The tanh form's z and z' of a g within [-30, 30].
__device__ __forceinline__ void tanh_arg(float g, float& z, float& zp) {
    const float g2 = g * g;
    z = 1.5957691216057308f * g * __builtin_fmaf(0.044715f, g2, 1.0f);
    zp = 1.5957691216057308f * __builtin_fmaf(0.134145f, g2, 1.0f);
}

// f(g) and, with GRAD, f'(g) in fp32.  The hardware exp2 and reciprocal are
// good to about an fp32 ulp; every result is rounded to 16 bits next.
//
// SiLU and tanh-GELU are g s(z) with s the logistic function, z = g and
// z = 2 sqrt(2/pi) (g + 0.044715 g^3) (as (1 + tanh(z/2)) / 2 = s(z)), and
// f' = s + g s (1 - s) z'.  1 - s is taken as e s, e = exp(-z), for z > 0, where
// the subtraction would cancel.
//
// GELU is g P(g), P(-a) = exp(-a^2/2) normal_tail(a) for a >= 0 and P(a) = 1 - P(-a).
// The left tail keeps its relative accuracy.
template <int FN, bool GRAD>
__device__ __forceinline__ void act_eval(float g, float& f, float& df) {
    if constexpr (FN == ZERO_GLU_GELU) {
        const float a = fabsf(g);
        const float e = exp2_hw(-0.5f * kLog2e * a * a);
        const float tail = e * normal_tail(a);
        const float cdf = g > 0.0f ? 1.0f - tail : tail;
        f = g * cdf;
        // where the density is 0, 0 * g is 0 for every finite g
        if constexpr (GRAD) df = __builtin_fmaf(e * 0.3989422804014327f, g, cdf);
    } else {
        float z = g, zp = 1.0f, gc = g;
        if constexpr (FN == ZERO_GLU_GELU_TANH) {
            // beyond |g| = 30, s is 0 or 1 in fp32; clamping keeps g^2 and z' finite
            gc = fminf(fmaxf(g, -30.0f), 30.0f);
            tanh_arg(gc, z, zp);
        }
        const float e = exp2_hw(-kLog2e * z);
        const float s = rcp_hw(1.0f + e);
        f = g * s;
        if constexpr (GRAD) {
            const float c = z > 0.0f ? e * s : 1.0f - s;
            df = s * __builtin_fmaf(gc * c, zp, 1.0f);
            if constexpr (FN == ZERO_GLU_GELU_TANH) df += 0.0f * (g - gc);  // a NaN stays a NaN
        }
    }
}

// The far left tail.  The hardware exp2 and reciprocal flush subnormal results to zero,
// but f and f' there, up to 2^-119, are bf16 values (f(-87.5) = -8.7e-37 for SiLU) and may be
// multiplied by a large up.  So below kFar (z below -78, or the density near 2^-113) exp(z) or
// exp(-g^2/2) is taken times 2^64 (s(z) equals exp(z) there, and 1 - s is 1), and 2^-64 comes
// last: under the normal range the result is fp32's.  fp16 ends at 2^-25 and up at 2^16,
// where zero is right.
template <int FN>
constexpr float kFar = FN == ZERO_GLU_SILU ? -80.0f : FN == ZERO_GLU_GELU ? -12.5f : -9.625f;

template <int FN, bool GRAD>
__device__ __forceinline__ void act_tail(float g, float& f, float& df) {
    if constexpr (FN == ZERO_GLU_GELU) {
        const float a = -g;
        const float e = exp2_hw(__builtin_fmaf(-0.5f * kLog2e * a, a, 64.0f));
        const float tail = e * normal_tail(a);
        f = g * tail * 0x1p-64f;
        if constexpr (GRAD) df = __builtin_fmaf(e * 0.3989422804014327f, g, tail) * 0x1p-64f;
    } else {
        float z = g, zp = 1.0f, gc = g;
        if constexpr (FN == ZERO_GLU_GELU_TANH) {
            gc = fmaxf(g, -30.0f);
            tanh_arg(gc, z, zp);
        }
        const float s = exp2_hw(__builtin_fmaf(kLog2e, z, 64.0f));
        f = g * s * 0x1p-64f;
        if constexpr (GRAD) {
            df = s * __builtin_fmaf(gc, zp, 1.0f) * 0x1p-64f;
            if constexpr (FN == ZERO_GLU_GELU_TANH) df += 0.0f * (g - gc);
        }
    }
}

// Whether an oct of 16-bit patterns has a value below kFar.  Its block's scale rules most
// out (not where it is NaN; a hundredth covers its roundings).  Patterns of negative values
// order like their magnitudes and lie above those of positive ones, so one integer maximum
// tells the rest (or finds a NaN, which is then not below kFar).  Ordinary data has none, so
// the tail stands behind a branch: computed for every element and selected, it made 262 x 9
// 9% and 8192 x 16384 up to 9% slower.  Branched over, it costs the GELU forms' forward pass
// 1 to 3% at 8192 x 16384 and a few hundredths of a microsecond elsewhere.
template <int DT, int FMT, int FN>
__device__ __forceinline__ bool any_far(const u4& w, float scale) {
    if (DT != ZERO_BF16 || scale < -0.99f * kFar<FN> / act_qmax<FMT>()) return false;
    constexpr uint32_t far = __builtin_bit_cast(uint32_t, kFar<FN>) >> 16;
    const uint32_t m = max_pair(max_pair(w[0], w[1]), max_pair(w[2], w[3]));
    return max(m & 0xffffu, m >> 16) > far;
}

// One pair of blocks per wave: 8192 x 16384 gated forward 172 us (with 2 it took 9 us more,
// with 4 15).
template <int DT, int FMT, int FN, bool GATED>
__global__ __launch_bounds__(kActThreads) void glu_forward_kernel(
    const uint16_t* __restrict__ gate, int64_t gate_stride, const uint16_t* __restrict__ up, int64_t up_stride,
    int cols, uint32_t nblocks, FastDiv per_row, uint16_t* __restrict__ h, int64_t h_stride,
    uint8_t* __restrict__ gate_codes, float* __restrict__ gate_scales, uint8_t* __restrict__ up_codes,
    float* __restrict__ up_scales, int64_t pitch) {
    const Place p = place_of<1>(0, nblocks, per_row);
    u4 wg{0u, 0u, 0u, 0u}, wu{0u, 0u, 0u, 0u};
    if (p.live && p.col < cols) {
        wg = load_oct(gate + p.row * gate_stride, p.col, cols);
        if constexpr (GATED) wu = load_oct(up + p.row * up_stride, p.col, cols);
    }
    const float gs = block_scale<DT, FMT>(wg);
    float us = 0.0f;
    if constexpr (GATED) us = block_scale<DT, FMT>(wu);
    if (!p.live) return;
    float g[kOct], u[kOct], o[kOct];
    widen_oct<DT>(wg, g);
    if constexpr (GATED) widen_oct<DT>(wu, u);
    const auto value = [&](int i, float f) { o[i] = GATED ? f * u[i] : f; };
#pragma unroll
    for (int i = 0; i < kOct; ++i) {
        float f, df;
        act_eval<FN, false>(g[i], f, df);
        value(i, f);
    }
    // in one piece with f: behind the branch, 262 x 9 took 4.1 us instead of 3.7
    const u2 cg = encode_oct<FMT>(g, gs);
    u2 cu{0u, 0u};
    if constexpr (GATED) cu = encode_oct<FMT>(u, us);
    if (any_far<DT, FMT, FN>(wg, gs)) {
#pragma unroll
        for (int i = 0; i < kOct; ++i) {
            if (!(g[i] < kFar<FN>)) continue;
            float f, df;
            act_tail<FN, false>(g[i], f, df);
            value(i, f);
        }
    }
    if (p.col < cols) store_oct(h + p.row * h_stride, p.col, cols, narrow_oct<DT>(o));
    if ((threadIdx.x & 31) == 0) {
        gate_scales[p.block] = gs;
        if constexpr (GATED) up_scales[p.block] = us;
    }
    if (p.col < pitch) {
        store_codes(gate_codes + p.row * pitch, p.col, cg);
        if constexpr (GATED) store_codes(up_codes + p.row * pitch, p.col, cu);
    }
}

// Bound by memory too (8192 x 16384 gated with h: 212 us, 6.3 TB/s): about 50 operations per
// element hide behind 10 bytes.
template <int DT, int FMT, int FN, bool GATED>
__global__ __launch_bounds__(kActThreads) void glu_backward_kernel(
    const uint8_t* __restrict__ gate_codes, const float* __restrict__ gate_scales,
    const uint8_t* __restrict__ up_codes, const float* __restrict__ up_scales, int64_t pitch, int cols,
    uint32_t nblocks, FastDiv per_row, const uint16_t* __restrict__ dh, int64_t dh_stride,
    uint16_t* __restrict__ dgate, int64_t dgate_stride, uint16_t* __restrict__ dup, int64_t dup_stride,
    uint16_t* __restrict__ h, int64_t h_stride) {
    const Place p = place_of<1>(0, nblocks, per_row);
    if (!p.live || p.col >= cols) return;
    const u4 wd = load_oct(dh + p.row * dh_stride, p.col, cols);
    const u2 qg = load_codes(gate_codes + p.row * pitch, p.col);
    const float sg = gate_scales[p.block];
    float d[kOct], g[kOct], u[kOct], f[kOct], df[kOct], a[kOct], b[kOct], o[kOct];
    if constexpr (GATED) {
        const u2 qu = load_codes(up_codes + p.row * pitch, p.col);
        widen_oct<DT>(decode_oct<DT, FMT>(qu, up_scales[p.block]), u);
    }
    widen_oct<DT>(wd, d);
    const u4 wg = decode_oct<DT, FMT>(qg, sg);
    widen_oct<DT>(wg, g);
#pragma unroll
    for (int i = 0; i < kOct; ++i) act_eval<FN, true>(g[i], f[i], df[i]);
    if (any_far<DT, FMT, FN>(wg, sg)) {
#pragma unroll
        for (int i = 0; i < kOct; ++i)
            if (g[i] < kFar<FN>) act_tail<FN, true>(g[i], f[i], df[i]);
    }
#pragma unroll
    for (int i = 0; i < kOct; ++i) {
        a[i] = (GATED ? d[i] * u[i] : d[i]) * df[i];
        b[i] = d[i] * f[i];
        o[i] = GATED ? f[i] * u[i] : f[i];
    }
    store_oct(dgate + p.row * dgate_stride, p.col, cols, narrow_oct<DT>(a));
    if constexpr (GATED) store_oct(dup + p.row * dup_stride, p.col, cols, narrow_oct<DT>(b));
    if (h != nullptr) store_oct(h + p.row * h_stride, p.col, cols, narrow_oct<DT>(o));
}

// ---------------------------------------------------------------------------
// Residual norm
// ---------------------------------------------------------------------------

// T threads hold a row in registers, V octs each: oct v of thread t starts at
// column (v T + t) 8, so the accesses of a wave are contiguous and every
// quantisation block lies in one half-wave.  Rows of up to 512 columns are a
// wave's (4 rows per block, no barrier); longer ones a block's.  The statistics take
// two passes over the registers (mean, then squared distances), which costs no
// memory time: 16384 x 4096 with a branch, 101 us and 6.0 TB/s forward, 123 us
// backward with both parameter gradients (4.9 TB/s: the row's two sums stand
// between its loads and its stores).  The backward pass of more than 8192 columns (two
// octs per thread at 1024 threads) keeps 9 registers in scratch memory.
template <int T>
constexpr int norm_rows() {
    return T >= 256 ? 1 : 256 / T;
}
template <int T>
constexpr int norm_threads() {
    return T >= 256 ? T : 256;
}

// Which of a block's rows this thread is on: the same in a whole wave, so that
// row addresses stay scalar.
template <int T>
__device__ __forceinline__ int row_in_block() {
    return norm_rows<T>() > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / T) : 0;
}

// Sum over the T threads of a row, the same in all of them: a butterfly in
// each wave, then the wave sums in wave order.  `slot` alternates between
// calls so that one barrier per call is enough.
template <int T, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int slot) {
#pragma unroll
    for (int k = 0; k < N; ++k)
        for (int off = 32; off > 0; off >>= 1) v[k] += __shfl_xor(v[k], off, 64);
    if constexpr (T > 64) {
        constexpr int kWaves = T / 64;
        __shared__ float part[2][N][kWaves];
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < N; ++k) part[slot][k][threadIdx.x >> 6] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float s = part[slot][k][0];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) s += part[slot][k][w];
            v[k] = s;
        }
    }
}

// x + alpha b in two fp32 roundings (no fused multiply-add): the residual
// stream is compared and checkpointed bit for bit.
__device__ __forceinline__ float add_scaled(float x, float alpha, float b) {
#pragma clang fp contract(off)
    return x + alpha * b;
}

template <int DT, int FMT, int T, int V>
__global__ __launch_bounds__(norm_threads<T>()) void norm_forward_kernel(
    const uint16_t* x, int64_t x_stride, const uint16_t* __restrict__ branch, int64_t branch_stride, float alpha,
    const uint16_t* __restrict__ weight, const uint16_t* __restrict__ bias, int64_t rows, int cols, int layer,
    float eps, uint16_t* res, int64_t res_stride, uint16_t* __restrict__ y, int64_t y_stride,
    uint8_t* __restrict__ codes, int64_t pitch, float* __restrict__ scales, int blocks_per_row,
    float* __restrict__ mean_out, float* __restrict__ rstd_out) {
    const int64_t row = int64_t(blockIdx.x) * norm_rows<T>() + row_in_block<T>();
    const int t = threadIdx.x % T;
    if (row >= rows) return;  // uniform over a wave; a block's only row exists
    u4 w[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * T + t) * kOct;
        w[v] = u4{0u, 0u, 0u, 0u};
        if (c < cols) w[v] = load_oct(x + row * x_stride, c, cols);
    }
    if (branch != nullptr) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + t) * kOct;
            if (c >= cols) continue;
            float a[kOct], b[kOct];
            widen_oct<DT>(w[v], a);
            widen_oct<DT>(load_oct(branch + row * branch_stride, c, cols), b);
#pragma unroll
            for (int k = 0; k < kOct; ++k) a[k] = add_scaled(a[k], alpha, b[k]);
            w[v] = narrow_oct<DT>(a);
            store_oct(res + row * res_stride, c, cols, w[v]);
        }
    }
    const float inv_n = 1.0f / float(cols);
    float mean = 0.0f;
    if (layer) {
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float a[kOct];
            widen_oct<DT>(w[v], a);
#pragma unroll
            for (int k = 0; k < kOct; ++k) s[0] += a[k];
        }
        row_sums<T, 1>(s, 0);
        mean = s[0] * inv_n;
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * T + t) * kOct;
        float a[kOct];
        widen_oct<DT>(w[v], a);
#pragma unroll
        for (int k = 0; k < kOct; ++k) {
            const float d = a[k] - mean;
            if (c + k < cols) q[0] = __builtin_fmaf(d, d, q[0]);
        }
    }
    row_sums<T, 1>(q, 1);
    const float rstd = 1.0f / sqrtf(__builtin_fmaf(q[0], inv_n, eps));
    if (t == 0) {
        rstd_out[row] = rstd;
        if (layer) mean_out[row] = mean;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * T + t) * kOct;
        const float scale = block_scale<DT, FMT>(w[v]);
        float a[kOct];
        widen_oct<DT>(w[v], a);
        if (c < pitch) {
            if ((t & 31) == 0) scales[row * blocks_per_row + c / kActBlock] = scale;
            store_codes(codes + row * pitch, c, encode_oct<FMT>(a, scale));
        }
        if (c >= cols) continue;
#pragma unroll
        for (int k = 0; k < kOct; ++k) a[k] = (a[k] - mean) * rstd;
        if (weight != nullptr) {
            float g[kOct];
            widen_oct<DT>(load_oct_shared(weight, c, cols), g);
#pragma unroll
            for (int k = 0; k < kOct; ++k) a[k] *= g[k];
        }
        if (bias != nullptr) {
            float b[kOct];
            widen_oct<DT>(load_oct_shared(bias, c, cols), b);
#pragma unroll
            for (int k = 0; k < kOct; ++k) a[k] += b[k];
        }
        store_oct(y + row * y_stride, c, cols, narrow_oct<DT>(a));
    }
}

// Block b does rows [b chunk, (b + 1) chunk), loading each row while the one
// before is computed (rows of up to 8192 columns).  Its threads keep the column
// sums of dy n and dy for their columns over all of them, and write the wanted ones
// to the workspace as partial b: [blocks][sums][cols8] fp32 (cols8: cols rounded up
// to an oct), added up by fold_columns_kernel.
template <int DT, int FMT, int T, int V>
__global__ __launch_bounds__(norm_threads<T>()) void norm_backward_kernel(
    const uint8_t* __restrict__ codes, int64_t pitch, const float* __restrict__ scales, int blocks_per_row,
    const float* __restrict__ mean_in, const float* __restrict__ rstd_in, const uint16_t* __restrict__ weight,
    int64_t rows, int64_t chunk, int cols, int layer, const uint16_t* __restrict__ dy, int64_t dy_stride,
    const uint16_t* dres, int64_t dres_stride, float alpha, uint16_t* dx, int64_t dx_stride,
    uint16_t* __restrict__ dbranch, int64_t dbranch_stride, float* __restrict__ partials, int sum_n, int sum_dy) {
    constexpr int R = norm_rows<T>();
    const int t = threadIdx.x % T;
    const float inv_n = 1.0f / float(cols);
    struct Row {
        u2 q[V];
        u4 d[V], r[V];
        float scale[V], rstd, mean;
    };
    const auto load = [&](int64_t row) {
        Row w;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + t) * kOct;
            w.q[v] = u2{0u, 0u};
            w.d[v] = w.r[v] = u4{0u, 0u, 0u, 0u};
            w.scale[v] = 0.0f;
            if (c < cols) {
                w.q[v] = load_codes(codes + row * pitch, c);
                w.scale[v] = scales[row * blocks_per_row + c / kActBlock];
                w.d[v] = load_oct(dy + row * dy_stride, c, cols);
                if (dres != nullptr) w.r[v] = load_oct(dres + row * dres_stride, c, cols);
            }
        }
        w.rstd = rstd_in[row];
        w.mean = layer ? mean_in[row] : 0.0f;
        return w;
    };
    // The loop's bounds are uniform over the T threads of a row (a wave, or the block).
    const int64_t first = int64_t(blockIdx.x) * chunk;
    const int64_t last = first + chunk < rows ? first + chunk : rows;
    int64_t row = first + row_in_block<T>();
    constexpr bool kAhead = V == 1;  // the registers for a second row are there
    Row next{};
    if (kAhead && row < last) next = load(row);
    u4 wt[V];
    float sn[V][kOct], sy[V][kOct];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * T + t) * kOct;
        wt[v] = u4{0u, 0u, 0u, 0u};
        if (weight != nullptr && c < cols) wt[v] = load_oct_shared(weight, c, cols);
#pragma unroll
        for (int k = 0; k < kOct; ++k) sn[v][k] = sy[v][k] = 0.0f;
    }
    int slot = 0;
    for (; row < last; row += R, slot ^= 1) {
        Row w;
        if constexpr (kAhead) {
            w = next;
            if (row + R < last) next = load(row + R);
        } else {
            w = load(row);
        }
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float r[kOct], d[kOct], g[kOct];
            widen_oct<DT>(decode_oct<DT, FMT>(w.q[v], w.scale[v]), r);
            widen_oct<DT>(w.d[v], d);
            widen_oct<DT>(wt[v], g);
#pragma unroll
            for (int k = 0; k < kOct; ++k) {
                const float n = (r[k] - w.mean) * w.rstd;
                sn[v][k] = __builtin_fmaf(d[k], n, sn[v][k]);
                sy[v][k] += d[k];
                const float dw = weight != nullptr ? d[k] * g[k] : d[k];
                s[0] = __builtin_fmaf(dw, n, s[0]);
                s[1] += dw;
            }
            // Decoded again below rather than kept in fp32 across the barrier: without the
            // empty asm a row of 8192 columns took 194 registers (2 waves per SIMD).
            asm("" : "+v"(w.q[v]), "+v"(w.d[v]));
        }
        row_sums<T, 2>(s, slot);
        const float mn = s[0] * inv_n;
        const float md = layer ? s[1] * inv_n : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (v * T + t) * kOct;
            if (c >= cols) continue;
            float r[kOct], d[kOct], g[kOct], o[kOct];
            widen_oct<DT>(decode_oct<DT, FMT>(w.q[v], w.scale[v]), r);
            widen_oct<DT>(w.d[v], d);
            widen_oct<DT>(wt[v], g);
            widen_oct<DT>(w.r[v], o);
#pragma unroll
            for (int k = 0; k < kOct; ++k) {
                const float n = (r[k] - w.mean) * w.rstd;
                const float dw = weight != nullptr ? d[k] * g[k] : d[k];
                o[k] = __builtin_fmaf(w.rstd, __builtin_fmaf(-n, mn, dw - md), o[k]);
            }
            store_oct(dx + row * dx_stride, c, cols, narrow_oct<DT>(o));
            if (dbranch != nullptr) {
#pragma unroll
                for (int k = 0; k < kOct; ++k) o[k] *= alpha;
                store_oct(dbranch + row * dbranch_stride, c, cols, narrow_oct<DT>(o));
            }
        }
    }
    if (sum_n + sum_dy == 0) return;
    const int cols8 = (cols + kOct - 1) / kOct * kOct;
    float* out = partials + int64_t(blockIdx.x) * (sum_n + sum_dy) * cols8;
    if constexpr (R > 1) {
        // The waves of a block hold the same columns: added in wave order.
        __shared__ float acc[2][T * V * kOct];
        for (int wv = 0; wv < R; ++wv) {
            if (row_in_block<T>() == wv) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = (v * T + t) * kOct;
#pragma unroll
                    for (int k = 0; k < kOct; ++k) {
                        if (wv > 0) {
                            sn[v][k] += acc[0][c + k];
                            sy[v][k] += acc[1][c + k];
                        }
                        acc[0][c + k] = sn[v][k];
                        acc[1][c + k] = sy[v][k];
                    }
                }
            }
            __syncthreads();
        }
        if (row_in_block<T>() != R - 1) return;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (v * T + t) * kOct;
        if (c >= cols8) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (sum_n)
                *reinterpret_cast<f4*>(out + c + 4 * h) =
                    f4{sn[v][4 * h], sn[v][4 * h + 1], sn[v][4 * h + 2], sn[v][4 * h + 3]};
            if (sum_dy)
                *reinterpret_cast<f4*>(out + sum_n * cols8 + c + 4 * h) =
                    f4{sy[v][4 * h], sy[v][4 * h + 1], sy[v][4 * h + 2], sy[v][4 * h + 3]};
        }
    }
}

// Column sums of the partials, in a fixed order: 32 threads per column take
// every 32nd partial, 8 loads in flight, then add up in a tree.  blockIdx.y is the
// sum: dweight's first if both are wanted.
constexpr int kFoldCols = 32, kFoldWays = 32, kFoldThreads = kFoldCols * kFoldWays;

template <int DT>
__global__ __launch_bounds__(kFoldThreads) void fold_columns_kernel(const float* __restrict__ partials, int count,
                                                                    int cols, int cols8, uint16_t* first,
                                                                    uint16_t* second, int accumulate) {
    __shared__ float sums[kFoldWays][kFoldCols];
    uint16_t* out = blockIdx.y == 0 ? first : second;
    const int c = blockIdx.x * kFoldCols + threadIdx.x % kFoldCols;
    const int way = threadIdx.x / kFoldCols;
    const int64_t stride = int64_t(gridDim.y) * cols8;
    float s = 0.0f;
    if (c < cols) {
        const float* p = partials + int64_t(blockIdx.y) * cols8 + c;
        for (int i = way; i < count; i += 8 * kFoldWays) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = i + k * kFoldWays < count ? p[(i + k * kFoldWays) * stride] : 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k];
        }
    }
    sums[way][threadIdx.x % kFoldCols] = s;
    __syncthreads();
    for (int half = kFoldWays / 2; half > 0; half >>= 1) {
        if (way < half) sums[way][threadIdx.x % kFoldCols] += sums[way + half][threadIdx.x % kFoldCols];
        __syncthreads();
    }
    if (way == 0 && c < cols) {
        float total = sums[0][threadIdx.x];
        if (accumulate) total += widen<DT>(out[c]);
        out[c] = static_cast<uint16_t>(narrow<DT>(total));
    }
}

// ---------------------------------------------------------------------------
// Launch glue
// ---------------------------------------------------------------------------

// Threads per row, and rows a block takes in one pass.
inline int norm_row_threads(int64_t cols) { return cols <= 512 ? 64 : cols <= 2048 ? 256 : cols <= 4096 ? 512 : 1024; }

struct NormShape {
    int64_t chunk, blocks;  // the backward pass's rows per block and blocks
    int64_t most_blocks;    // never falls as rows grow
};

// One round of blocks of 1024 threads per CU: more blocks mean more partial sums to
// write and fold (16384 x 4096: 512 blocks 123 us, 1024 blocks 126, 256 blocks 137).
// With fewer than 4 passes for each the partials outweigh the rows' own data, and
// 256 blocks do (1024 x 1600: 12.6 us with 256, 17.6 with 1024).
inline NormShape norm_shape(int64_t rows, int64_t cols) {
    const int threads = norm_row_threads(cols), per_pass = threads >= 256 ? 1 : 256 / threads;
    const int64_t passes = ceil_div(rows, int64_t(per_pass));
    const int64_t most = threads <= 256 ? 1024 : 262144 / threads;
    const int64_t target = passes < 4 * most ? 256 : most;
    NormShape s;
    s.chunk = std::max<int64_t>(1, ceil_div(passes, target)) * per_pass;
    s.blocks = ceil_div(rows, s.chunk);
    s.most_blocks = std::min(passes, target);
    return s;
}

// Both sums' partials; a workspace for the longest batch serves all.
inline int64_t norm_workspace(int64_t rows, int64_t cols) {
    if (rows == 0 || cols == 0) return 0;
    return norm_shape(rows, cols).most_blocks * 2 * ceil_div(cols, int64_t(kOct)) * kOct * 4;
}

// Calls f with the row shape <T, V> for `cols`.  A thread has one oct where it can:
// a wave per row of up to 2048 columns (4 octs per lane) took 9.3 us instead of 5.7
// for 1024 x 1600 forward and 63 instead of 37 for 8192 x 1600 backward.  The forward
// pass of 4097 to 8192 columns is faster with 512 threads of 2 (27 against 31 us at 2000 x 5001).
template <bool FORWARD, typename F>
hipError_t with_shape(int64_t cols, F&& f) {
    if (cols <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    if (cols <= 2048) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
    if (cols <= 4096) return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 1>{});
    if (cols <= 8192) {
        if constexpr (FORWARD) return f(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
        else return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 1>{});
    }
    return f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}

template <typename F>
hipError_t with_fn(int fn, bool gated, F&& f) {
    const auto pick = [&](auto k) { return gated ? f(k, std::true_type{}) : f(k, std::false_type{}); };
    if (fn == ZERO_GLU_SILU) return pick(std::integral_constant<int, ZERO_GLU_SILU>{});
    if (fn == ZERO_GLU_GELU) return pick(std::integral_constant<int, ZERO_GLU_GELU>{});
    return pick(std::integral_constant<int, ZERO_GLU_GELU_TANH>{});
}

}  // namespace
}  // namespace zf

using namespace zf;

extern "C" {

int64_t zero_act_code_bytes(int64_t rows, int64_t cols) {
    if (!act_size_ok(rows, cols)) {
        fail(ZERO_EINVAL, "zero_act_code_bytes: rows or cols out of range");
        return -1;
    }
    ok();
    return rows * act_pitch(cols);
}

int64_t zero_act_scale_count(int64_t rows, int64_t cols) {
    if (!act_size_ok(rows, cols)) {
        fail(ZERO_EINVAL, "zero_act_scale_count: rows or cols out of range");
        return -1;
    }
    ok();
    return rows * act_blocks(cols);
}

int zero_act_save(const void* x, int64_t x_stride, int dtype, int64_t rows, int64_t cols, int format, void* codes,
                  float* scales, void* stream) {
    const char* fn = "zero_act_save";
    if (int rc = check_sizes(fn, rows, cols, dtype, format)) return rc;
    if (rows == 0 || cols == 0) return ok();
    if (int rc = check_matrix(fn, "x", x, rows, cols, x_stride)) return rc;
    if (int rc = check_checkpoint(fn, "", codes, scales)) return rc;
    const int64_t pitch = act_pitch(cols), nb = rows * act_blocks(cols);
    const Area areas[] = {mat16("x", x, rows, cols, x_stride, false), flat("codes", codes, rows * pitch, true),
                          flat("scales", scales, 4 * nb, true)};
    if (int rc = check_overlaps(fn, areas, 3)) return rc;
    const FastDiv per_row = fast_div(uint32_t(act_blocks(cols)));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = with_types(dtype, format, [&](auto dt, auto fmt) {
        constexpr int D = decltype(dt)::value, M = decltype(fmt)::value;
        return nb <= kSaveOnePair
                   ? launch(act_save_kernel<D, M, 1>, act_grid(nb, 1), dim3(kActThreads), s, in16(x), x_stride, int(cols),
                            uint32_t(nb), per_row, out8(codes), pitch, scales)
                   : launch(act_save_kernel<D, M, 2>, act_grid(nb, 2), dim3(kActThreads), s, in16(x), x_stride, int(cols),
                            uint32_t(nb), per_row, out8(codes), pitch, scales);
    });
    return hip_status(e, fn);
}

int zero_act_restore(const void* codes, const float* scales, int format, int64_t rows, int64_t cols, void* y,
                     int64_t y_stride, int dtype, void* stream) {
    const char* fn = "zero_act_restore";
    if (int rc = check_sizes(fn, rows, cols, dtype, format)) return rc;
    if (rows == 0 || cols == 0) return ok();
    if (int rc = check_checkpoint(fn, "", codes, scales)) return rc;
    if (int rc = check_matrix(fn, "y", y, rows, cols, y_stride)) return rc;
    const int64_t pitch = act_pitch(cols), nb = rows * act_blocks(cols);
    const Area areas[] = {mat16("y", y, rows, cols, y_stride, true), flat("codes", codes, rows * pitch, false),
                          flat("scales", scales, 4 * nb, false)};
    if (int rc = check_overlaps(fn, areas, 3)) return rc;
    const FastDiv per_row = fast_div(uint32_t(act_blocks(cols)));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = with_types(dtype, format, [&](auto dt, auto fmt) {
        return launch(act_restore_kernel<decltype(dt)::value, decltype(fmt)::value>, act_grid(nb, kRestorePairs),
                      dim3(kActThreads), s, in8(codes), pitch, scales, int(cols), uint32_t(nb), per_row, out16(y), y_stride);
    });
    return hip_status(e, fn);
}

int zero_act_glu_forward(const void* gate, int64_t gate_stride, const void* up, int64_t up_stride, int dtype,
                         int64_t rows, int64_t cols, int fn_id, int format, void* h, int64_t h_stride,
                         void* gate_codes, float* gate_scales, void* up_codes, float* up_scales, void* stream) {
    const char* fn = "zero_act_glu_forward";
    if (int rc = check_sizes(fn, rows, cols, dtype, format)) return rc;
    if (fn_id < ZERO_GLU_SILU || fn_id > ZERO_GLU_GELU_TANH)
        return fail(ZERO_EINVAL, std::string(fn) + ": fn must be ZERO_GLU_SILU, ZERO_GLU_GELU or ZERO_GLU_GELU_TANH");
    if (rows == 0 || cols == 0) return ok();  // arrays without elements may be NULL, whatever they stand for
    const bool gated = up != nullptr;
    if (!gated && (up_codes != nullptr || up_scales != nullptr))
        return fail(ZERO_EINVAL, std::string(fn) + ": up_codes and up_scales must be NULL when up is");
    if (int rc = check_matrix(fn, "gate", gate, rows, cols, gate_stride)) return rc;
    if (int rc = check_matrix(fn, "h", h, rows, cols, h_stride)) return rc;
    if (int rc = check_checkpoint(fn, "gate_", gate_codes, gate_scales)) return rc;
    if (gated) {
        if (int rc = check_matrix(fn, "up", up, rows, cols, up_stride)) return rc;
        if (int rc = check_checkpoint(fn, "up_", up_codes, up_scales)) return rc;
    }
    const int64_t pitch = act_pitch(cols), nb = rows * act_blocks(cols);
    const Area areas[] = {mat16("gate", gate, rows, cols, gate_stride, false),
                          mat16("up", up, rows, cols, up_stride, false),
                          mat16("h", h, rows, cols, h_stride, true),
                          flat("gate_codes", gate_codes, rows * pitch, true),
                          flat("gate_scales", gate_scales, 4 * nb, true),
                          flat("up_codes", up_codes, rows * pitch, true),
                          flat("up_scales", up_scales, 4 * nb, true)};
    if (int rc = check_overlaps(fn, areas, 7)) return rc;
    const FastDiv per_row = fast_div(uint32_t(act_blocks(cols)));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = with_types(dtype, format, [&](auto dt, auto fmt) {
        return with_fn(fn_id, gated, [&](auto f, auto g) {
            constexpr int D = decltype(dt)::value, M = decltype(fmt)::value, N = decltype(f)::value;
            return launch(glu_forward_kernel<D, M, N, decltype(g)::value>, act_grid(nb, 1), dim3(kActThreads), s,
                          in16(gate), gate_stride, in16(up), up_stride, int(cols), uint32_t(nb), per_row, out16(h),
                          h_stride, out8(gate_codes), gate_scales, out8(up_codes), up_scales, pitch);
        });
    });
    return hip_status(e, fn);
}

int zero_act_glu_backward(const void* gate_codes, const float* gate_scales, const void* up_codes,
                          const float* up_scales, int format, int64_t rows, int64_t cols, int fn_id, const void* dh,
                          int64_t dh_stride, int dtype, void* dgate, int64_t dgate_stride, void* dup,
                          int64_t dup_stride, void* h, int64_t h_stride, void* stream) {
    const char* fn = "zero_act_glu_backward";
    if (int rc = check_sizes(fn, rows, cols, dtype, format)) return rc;
    if (fn_id < ZERO_GLU_SILU || fn_id > ZERO_GLU_GELU_TANH)
        return fail(ZERO_EINVAL, std::string(fn) + ": fn must be ZERO_GLU_SILU, ZERO_GLU_GELU or ZERO_GLU_GELU_TANH");
    if (rows == 0 || cols == 0) return ok();  // arrays without elements may be NULL, whatever they stand for
    const bool gated = up_codes != nullptr;
    if ((up_scales != nullptr) != gated || (dup != nullptr) != gated)
        return fail(ZERO_EINVAL, std::string(fn) + ": up_codes, up_scales and dup are given together or all NULL");
    if (int rc = check_checkpoint(fn, "gate_", gate_codes, gate_scales)) return rc;
    if (int rc = check_matrix(fn, "dh", dh, rows, cols, dh_stride)) return rc;
    if (int rc = check_matrix(fn, "dgate", dgate, rows, cols, dgate_stride)) return rc;
    if (gated) {
        if (int rc = check_checkpoint(fn, "up_", up_codes, up_scales)) return rc;
        if (int rc = check_matrix(fn, "dup", dup, rows, cols, dup_stride)) return rc;
    }
    if (h != nullptr)
        if (int rc = check_matrix(fn, "h", h, rows, cols, h_stride)) return rc;
    const int64_t pitch = act_pitch(cols), nb = rows * act_blocks(cols);
    const Area areas[] = {flat("gate_codes", gate_codes, rows * pitch, false),
                          flat("gate_scales", gate_scales, 4 * nb, false),
                          flat("up_codes", up_codes, rows * pitch, false),
                          flat("up_scales", up_scales, 4 * nb, false),
                          mat16("dh", dh, rows, cols, dh_stride, false),
                          mat16("dgate", dgate, rows, cols, dgate_stride, true),
                          mat16("dup", dup, rows, cols, dup_stride, true),
                          mat16("h", h, rows, cols, h_stride, true)};
    if (int rc = check_overlaps(fn, areas, 8)) return rc;
    const FastDiv per_row = fast_div(uint32_t(act_blocks(cols)));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = with_types(dtype, format, [&](auto dt, auto fmt) {
        return with_fn(fn_id, gated, [&](auto f, auto g) {
            constexpr int D = decltype(dt)::value, M = decltype(fmt)::value, N = decltype(f)::value;
            return launch(glu_backward_kernel<D, M, N, decltype(g)::value>, act_grid(nb, 1), dim3(kActThreads), s,
                          in8(gate_codes), gate_scales, in8(up_codes), up_scales, pitch, int(cols), uint32_t(nb), per_row,
                          in16(dh), dh_stride, out16(dgate), dgate_stride, out16(dup), dup_stride, out16(h), h_stride);
        });
    });
    return hip_status(e, fn);
}

int zero_act_norm_forward(const void* x, int64_t x_stride, const void* branch, int64_t branch_stride, float alpha,
                          const void* weight, const void* bias, int dtype, int64_t rows, int64_t cols, int kind,
                          float eps, int format, void* res, int64_t res_stride, void* y, int64_t y_stride, void* codes,
                          float* scales, float* mean, float* rstd, void* stream) {
    const char* fn = "zero_act_norm_forward";
    if (int rc = check_sizes(fn, rows, cols, dtype, format)) return rc;
    if (cols > ZERO_NORM_MAX_COLS) return fail(ZERO_EINVAL, std::string(fn) + ": cols exceeds ZERO_NORM_MAX_COLS");
    if (kind != ZERO_NORM_RMS && kind != ZERO_NORM_LAYER)
        return fail(ZERO_EINVAL, std::string(fn) + ": kind must be ZERO_NORM_RMS or ZERO_NORM_LAYER");
    if (!(eps > 0.0f) || !std::isfinite(eps)) return fail(ZERO_EINVAL, std::string(fn) + ": eps must be positive and finite");
    if (branch != nullptr && !std::isfinite(alpha)) return fail(ZERO_EINVAL, std::string(fn) + ": alpha must be finite");
    if (rows == 0 || cols == 0) return ok();  // arrays without elements may be NULL, whatever they stand for
    if ((branch != nullptr) != (res != nullptr))
        return fail(ZERO_EINVAL, std::string(fn) + ": branch and res are given together or both NULL");
    if ((kind == ZERO_NORM_RMS) != (mean == nullptr))
        return fail(ZERO_EINVAL, std::string(fn) + ": mean is given for ZERO_NORM_LAYER and NULL for ZERO_NORM_RMS");
    if (int rc = check_matrix(fn, "x", x, rows, cols, x_stride)) return rc;
    if (branch != nullptr) {
        if (int rc = check_matrix(fn, "branch", branch, rows, cols, branch_stride)) return rc;
        if (int rc = check_matrix(fn, "res", res, rows, cols, res_stride)) return rc;
    }
    if (int rc = check_matrix(fn, "y", y, rows, cols, y_stride)) return rc;
    if (int rc = check_checkpoint(fn, "", codes, scales)) return rc;
    if ((weight != nullptr && (addr(weight) & 1)) || (bias != nullptr && (addr(bias) & 1)))
        return fail(ZERO_EINVAL, std::string(fn) + ": weight or bias not 2-byte aligned");
    if (bad_ptr(rstd, 4) || (mean != nullptr && (addr(mean) & 3)))
        return fail(ZERO_EINVAL, std::string(fn) + ": rstd NULL, or rstd or mean misaligned");
    const int64_t pitch = act_pitch(cols), bpr = act_blocks(cols);
    const Area areas[] = {mat16("x", x, rows, cols, x_stride, false),
                          mat16("branch", branch, rows, cols, branch_stride, false),
                          flat("weight", weight, 2 * cols, false),
                          flat("bias", bias, 2 * cols, false),
                          mat16("res", res, rows, cols, res_stride, true),
                          mat16("y", y, rows, cols, y_stride, true),
                          flat("codes", codes, rows * pitch, true),
                          flat("scales", scales, 4 * rows * bpr, true),
                          flat("mean", mean, 4 * rows, true),
                          flat("rstd", rstd, 4 * rows, true)};
    if (int rc = check_overlaps(fn, areas, 10, "res", "x")) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = with_types(dtype, format, [&](auto dt, auto fmt) {
        return with_shape<true>(cols, [&](auto t, auto v) {
            constexpr int D = decltype(dt)::value, M = decltype(fmt)::value, T = decltype(t)::value;
            // A launch's work-items are counted in 32 bits: 2^21 blocks of at most 1024 at a time.
            constexpr int64_t kSlice = (int64_t(1) << 21) * norm_rows<T>();
            for (int64_t r = 0; r < rows; r += kSlice) {
                const int64_t n = std::min(kSlice, rows - r);
                const dim3 grid{unsigned(ceil_div(n, int64_t(norm_rows<T>())))};
                const hipError_t err = launch(
                    norm_forward_kernel<D, M, T, decltype(v)::value>, grid, dim3(norm_threads<T>()), s,
                    in16(x) + r * x_stride, x_stride, branch ? in16(branch) + r * branch_stride : nullptr, branch_stride,
                    alpha, in16(weight), in16(bias), n, int(cols), int(kind == ZERO_NORM_LAYER), eps,
                    res ? out16(res) + r * res_stride : nullptr, res_stride, out16(y) + r * y_stride, y_stride,
                    out8(codes) + r * pitch, pitch, scales + r * bpr, int(bpr), mean ? mean + r : nullptr, rstd + r);
                if (err != hipSuccess) return err;
            }
            return hipSuccess;
        });
    });
    return hip_status(e, fn);
}

int64_t zero_act_norm_workspace_bytes(int64_t rows, int64_t cols) {
    if (!act_size_ok(rows, cols) || cols > ZERO_NORM_MAX_COLS) {
        fail(ZERO_EINVAL, "zero_act_norm_workspace_bytes: rows or cols out of range");
        return -1;
    }
    ok();
    return norm_workspace(rows, cols);
}

int zero_act_norm_backward(const void* codes, const float* scales, int format, const float* mean, const float* rstd,
                           const void* weight, int64_t rows, int64_t cols, int kind, const void* dy, int64_t dy_stride,
                           const void* dres, int64_t dres_stride, float alpha, int dtype, void* dx, int64_t dx_stride,
                           void* dbranch, int64_t dbranch_stride, int accumulate, void* dweight, void* dbias,
                           void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "zero_act_norm_backward";
    if (int rc = check_sizes(fn, rows, cols, dtype, format)) return rc;
    if (cols > ZERO_NORM_MAX_COLS) return fail(ZERO_EINVAL, std::string(fn) + ": cols exceeds ZERO_NORM_MAX_COLS");
    if (kind != ZERO_NORM_RMS && kind != ZERO_NORM_LAYER)
        return fail(ZERO_EINVAL, std::string(fn) + ": kind must be ZERO_NORM_RMS or ZERO_NORM_LAYER");
    if (dbranch != nullptr && !std::isfinite(alpha)) return fail(ZERO_EINVAL, std::string(fn) + ": alpha must be finite");
    if ((dweight != nullptr && (addr(dweight) & 1)) || (dbias != nullptr && (addr(dbias) & 1)) ||
        (weight != nullptr && (addr(weight) & 1)))
        return fail(ZERO_EINVAL, std::string(fn) + ": weight, dweight or dbias not 2-byte aligned");
    if (cols == 0) return ok();
    const bool sums = dweight != nullptr || dbias != nullptr;
    const int64_t pitch = act_pitch(cols), bpr = act_blocks(cols), wb = sums ? norm_workspace(rows, cols) : 0;
    if (rows > 0) {
        if ((kind == ZERO_NORM_RMS) != (mean == nullptr))
            return fail(ZERO_EINVAL, std::string(fn) + ": mean is given for ZERO_NORM_LAYER and NULL for ZERO_NORM_RMS");
        if (int rc = check_checkpoint(fn, "", codes, scales)) return rc;
        if (int rc = check_matrix(fn, "dy", dy, rows, cols, dy_stride)) return rc;
        if (dres != nullptr)
            if (int rc = check_matrix(fn, "dres", dres, rows, cols, dres_stride)) return rc;
        if (int rc = check_matrix(fn, "dx", dx, rows, cols, dx_stride)) return rc;
        if (dbranch != nullptr)
            if (int rc = check_matrix(fn, "dbranch", dbranch, rows, cols, dbranch_stride)) return rc;
        if (bad_ptr(rstd, 4) || (mean != nullptr && (addr(mean) & 3)))
            return fail(ZERO_EINVAL, std::string(fn) + ": rstd NULL, or rstd or mean misaligned");
        if (wb > 0 && (bad_ptr(workspace, 16) || workspace_bytes < wb))
            return fail(ZERO_EINVAL, std::string(fn) + ": workspace NULL, not 16-byte aligned or too small");
    }
    const Area areas[] = {flat("codes", codes, rows * pitch, false),
                          flat("scales", scales, 4 * rows * bpr, false),
                          flat("mean", mean, 4 * rows, false),
                          flat("rstd", rstd, 4 * rows, false),
                          flat("weight", weight, 2 * cols, false),
                          mat16("dy", dy, rows, cols, dy_stride, false),
                          mat16("dres", dres, rows, cols, dres_stride, false),
                          mat16("dx", dx, rows, cols, dx_stride, true),
                          mat16("dbranch", dbranch, rows, cols, dbranch_stride, true),
                          flat("dweight", dweight, 2 * cols, true),
                          flat("dbias", dbias, 2 * cols, true),
                          flat("workspace", workspace, wb, true)};
    if (int rc = check_overlaps(fn, areas, 12, "dx", "dres")) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const NormShape shape = norm_shape(rows, cols);
    float* partials = sums ? static_cast<float*>(workspace) : nullptr;
    if (rows > 0) {
        const hipError_t e = with_types(dtype, format, [&](auto dt, auto fmt) {
            return with_shape<false>(cols, [&](auto t, auto v) {
                constexpr int D = decltype(dt)::value, M = decltype(fmt)::value, T = decltype(t)::value;
                return launch(norm_backward_kernel<D, M, T, decltype(v)::value>, dim3(unsigned(shape.blocks)),
                              dim3(norm_threads<T>()), s, in8(codes), pitch, scales, int(bpr), mean, rstd,
                              in16(weight), rows, shape.chunk, int(cols), int(kind == ZERO_NORM_LAYER), in16(dy),
                              dy_stride, in16(dres), dres_stride, alpha, out16(dx), dx_stride, out16(dbranch),
                              dbranch_stride, partials, int(dweight != nullptr), int(dbias != nullptr));
            });
        });
        if (e != hipSuccess) return hip_status(e, fn);
    }
    if (!sums || (rows == 0 && accumulate)) return ok();
    const hipError_t e = with_dtype(dtype, [&](auto dt) {
        return launch(fold_columns_kernel<decltype(dt)::value>,
                      dim3(unsigned(ceil_div(cols, int64_t(kFoldCols))), dweight != nullptr && dbias != nullptr ? 2 : 1),
                      dim3(kFoldThreads), s, partials, rows > 0 ? int(shape.blocks) : 0, int(cols),
                      int(ceil_div(cols, int64_t(kOct)) * kOct), out16(dweight != nullptr ? dweight : dbias),
                      out16(dbias), accumulate);
    });
    return hip_status(e, fn);
}

}  // extern "C"
