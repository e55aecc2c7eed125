// Weight and bias gradient of a linear layer from the 8-bit checkpoint of its
// input, for MI355X (gfx950, wave64), and its C-ABI entry point.  The formulas
// are in include/zero_flat.h.
//
//   weight_grad_kernel   a tile of dW = dY^T X, X restored from the checkpoint
//   join_kernel          adds the partial tiles of a product split over tokens
//
// The contraction runs over tokens, the slow axis of both operands: a matrix
// instruction wants 8 consecutive tokens of one column per lane.  Tiles of 64
// tokens are staged in LDS as they lie in memory ([token][column], 16 bits) and
// read with the transposing LDS load (ds_read_b64_tr_b16: 16 lanes read 4 rows
// of 16 columns and each lane receives one column of the 4 rows).  The codes are
// decoded once per block on their way into LDS, between the matrix
// instructions of the previous tile.

#include "act.h"

namespace zf {
namespace {

typedef short s4v __attribute__((ext_vector_type(4)));
typedef short s8v __attribute__((ext_vector_type(8)));
typedef __bf16 b8v __attribute__((ext_vector_type(8)));
typedef _Float16 h8v __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));

constexpr int kTokens = 64;       // tokens per staged tile
constexpr int kGradThreads = 256; // four waves, two by two

// A block's tile: TILE outputs x TILE inputs; a wave does a quarter of it in
// FRAGS x FRAGS 32 x 32 fragments.  LDS rows are TILE 16-bit values in segments of
// 32 columns (64 bytes), segment s of token t kept at s ^ (t mod 4): the four rows
// that a transposing read touches then lie in different quarters of the 256 bytes
// that the banks span.
template <int TILE>
struct GradTile {
    static constexpr int kRowBytes = 2 * TILE;
    static constexpr int kOperandBytes = kTokens * kRowBytes;
    static constexpr int kStageBytes = 2 * kOperandBytes;
    static constexpr int kWave = TILE / 2;
    static constexpr int kFrags = kWave / 32;
    static constexpr int kOcts = TILE / kOct;                    // per row
    static constexpr int kRowsPerPass = kGradThreads / kOcts;
    static constexpr int kPasses = kTokens / kRowsPerPass;
};

struct GradArgs {
    const uint16_t* dy;
    int64_t dy_stride;
    const uint8_t* codes;
    int64_t pitch;
    const float* scales;
    int blocks_per_row;
    int64_t rows;
    int in_cols, out_cols;
    int in_tiles, out_tiles;
    int splits;
    int64_t split_rows;  // tokens per split, a multiple of kTokens
    int accumulate;
    uint16_t* dweight;
    uint16_t* dbias;
    float* partials;       // splits > 1: [splits][out_cols][in8] fp32, then
    float* bias_partials;  // [splits][out_cols]
};

// Order of a 16-token step's instructions: after each matrix instruction, which
// keeps the matrix unit busy for 8 issue slots, one LDS read and a few of the
// others, so that a lone wave per SIMD never leaves it idle.
template <bool BIAS>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);          // MFMA
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);          // LDS read
        __builtin_amdgcn_sched_group_barrier(0x002, BIAS ? 6 : 4, 0);  // VALU
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);          // LDS write
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);          // global load
    }
}

template <int DT>
__device__ __forceinline__ f16v mfma32(const s8v& a, const s8v& b, const f16v& c) {
    if constexpr (DT == ZERO_BF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8v, a), __builtin_bit_cast(b8v, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8v, a), __builtin_bit_cast(h8v, b), c, 0, 0, 0);
}

// 8 tokens of one column per lane: two transposing reads, 4 tokens each.
template <int ROW_BYTES>
__device__ __forceinline__ s8v read_frag(const char* p) {
    typedef __attribute__((address_space(3))) s4v* lds4;
    const s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p));
    const s4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 4 * ROW_BYTES));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// How a run of staged tiles is loaded.  kWhole: every token and column of it
// lies in the operands.  kGuarded: some may lie outside and are staged as zero.
enum { kWhole, kGuarded };

// Staged tiles t0, t0 + 64, .. of `tiles` into acc and, with BIAS, the column
// sums of dY.  While tile k is multiplied, tile k + 1 goes from registers to the
// other LDS stage and tile k + 2 is loaded into the registers this frees, so a
// load has a whole tile's time (2048 cycles of matrix instructions at 256 x 256) to
// arrive.  The fragments of 16 tokens are read while the previous 16 are
// multiplied; the barrier stands before the last 16 of a tile, whose fragments
// are in registers by then, so that the next tile's first ones can be read under
// their multiplication.
template <int DT, int FMT, int TILE, int MODE, bool BIAS>
__device__ __forceinline__ void grad_loop(const GradArgs& g, char* smem, int o0, int i0, int64_t t0, int tiles,
                                          int64_t t_end, float (&bsum)[kOct],
                                          f16v (&acc)[GradTile<TILE>::kFrags][GradTile<TILE>::kFrags]) {
    using G = GradTile<TILE>;
    constexpr int F = G::kFrags, P = G::kPasses, kSteps = kTokens / 16;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int oct = tid % G::kOcts, row = tid / G::kOcts;
    // where this thread's octs go, and where its fragments start
    const int put = row * G::kRowBytes + (((oct >> 2) ^ (row & 3)) << 6) + ((oct & 3) << 4);
    const int l = lane & 15, grp = lane >> 4;
    const int frag_row = (grp >> 1) * 8 + (l >> 2);
    const int inner = ((grp & 1) * 16 + (l & 3) * 4) * 2;
    int fa[F], fb[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
        const int sa = (wave >> 1) * F + f, sb = (wave & 1) * F + f;
        fa[f] = frag_row * G::kRowBytes + ((sa ^ (l >> 2)) << 6) + inner;
        fb[f] = G::kOperandBytes + frag_row * G::kRowBytes + ((sb ^ (l >> 2)) << 6) + inner;
    }

    u4 a[P];
    u2 b[P];
    float s[P];
    // kWhole: one uniform base per operand and a constant 32-bit offset per pass
    uint32_t oa[P], ob[P], os[P];
    const char* pa = reinterpret_cast<const char*>(g.dy + t0 * g.dy_stride + o0);
    const char* pb = reinterpret_cast<const char*>(g.codes + t0 * g.pitch + i0);
    const char* ps = reinterpret_cast<const char*>(g.scales + t0 * g.blocks_per_row + i0 / kActBlock);
    if constexpr (MODE == kWhole) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const uint32_t r = uint32_t(row + j * G::kRowsPerPass);
            oa[j] = (r * uint32_t(g.dy_stride) + oct * kOct) * 2u;
            ob[j] = r * uint32_t(g.pitch) + oct * kOct;
            os[j] = r * uint32_t(g.blocks_per_row) * 4u;
        }
    }
    const auto load = [&](int tile, int j) {
        if constexpr (MODE == kGuarded) {
            const int64_t t = t0 + int64_t(tile) * kTokens + j * G::kRowsPerPass + row;
            const int o = o0 + oct * kOct, i = i0 + oct * kOct;
            a[j] = u4{0u, 0u, 0u, 0u};
            b[j] = u2{0u, 0u};
            s[j] = 0.0f;
            if (t < t_end) {
                if (o < g.out_cols) a[j] = load_oct_shared(g.dy + t * g.dy_stride, o, g.out_cols);
                if (i < g.in_cols) {
                    b[j] = *reinterpret_cast<const u2*>(g.codes + t * g.pitch + i);
                    s[j] = g.scales[t * g.blocks_per_row + i / kActBlock];
                }
            }
        } else {
            a[j] = *reinterpret_cast<const u4_any*>(pa + oa[j]);
            b[j] = *reinterpret_cast<const u2*>(pb + ob[j]);
            s[j] = *reinterpret_cast<const float*>(ps + os[j]);
        }
    };
    const auto advance = [&](bool more) {
        pa += more ? 2 * kTokens * g.dy_stride : 0;
        pb += more ? kTokens * g.pitch : 0;
        ps += more ? int64_t(4) * kTokens * g.blocks_per_row : 0;
    };
    const auto store = [&](char* stage, int j) {
        char* p = stage + put + j * G::kRowsPerPass * G::kRowBytes;
        *reinterpret_cast<u4*>(p) = a[j];
        *reinterpret_cast<u4*>(p + G::kOperandBytes) = decode_oct<DT, FMT>(b[j], s[j]);
    };
    // `keep` is all ones, or 0 for a tile that is only staged again
    const auto sum = [&](int j, uint32_t keep) {
        if constexpr (BIAS) {
            float v[kOct];
            widen_oct<DT>(a[j] & keep, v);
#pragma unroll
            for (int k = 0; k < kOct; ++k) bsum[k] += v[k];
        }
    };
    s8v x[2][F], y[2][F];
    const auto read = [&](const char* stage, int ks, int set) {
#pragma unroll
        for (int f = 0; f < F; ++f) y[set][f] = read_frag<G::kRowBytes>(stage + fa[f] + ks * 16 * G::kRowBytes);
#pragma unroll
        for (int f = 0; f < F; ++f) x[set][f] = read_frag<G::kRowBytes>(stage + fb[f] + ks * 16 * G::kRowBytes);
    };

#pragma unroll
    for (int j = 0; j < P; ++j) load(0, j);
    advance(tiles > 1);
#pragma unroll
    for (int j = 0; j < P; ++j) {
        store(smem, j);
        sum(j, ~0u);
        load(tiles > 1 ? 1 : 0, j);
    }
    __syncthreads();
    read(smem, 0, 0);
    for (int it = 0; it < tiles; ++it) {
        const char* cur = smem + (it & 1) * G::kStageBytes;
        char* nxt = smem + ((it & 1) ^ 1) * G::kStageBytes;
        // past the end the last tile is staged again and never used
        advance(it + 2 < tiles);
        const int ahead = it + 2 < tiles ? it + 2 : tiles - 1;
        const uint32_t keep = it + 1 < tiles ? ~0u : 0u;
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
            if (ks == kSteps - 1) __syncthreads();
            read(ks == kSteps - 1 ? nxt : cur, (ks + 1) % kSteps, (ks + 1) & 1);
#pragma unroll
            for (int m = 0; m < F; ++m)
#pragma unroll
                for (int n = 0; n < F; ++n) acc[m][n] = mfma32<DT>(y[ks & 1][m], x[ks & 1][n], acc[m][n]);
            // the passes are spread over all but the last 16 tokens
            if (ks < kSteps - 1) {
#pragma unroll
                for (int j = ks * P / (kSteps - 1); j < (ks + 1) * P / (kSteps - 1); ++j) {
                    store(nxt, j);
                    sum(j, keep);
                    load(ahead, j);
                }
            }
            if constexpr (MODE == kWhole && TILE == 256) interleave<BIAS>();
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    __syncthreads();
}

// Blocks are dispatched round-robin to the 8 XCDs; each XCD takes a contiguous
// run of tiles, ordered so that about 32 tiles in flight form a patch of 8
// output tiles by 4 input tiles that share operand panels in its L2.
__device__ __forceinline__ void place_tile(int id, int count, int out_tiles, int in_tiles, int& o, int& i) {
    constexpr int kXcds = 8, kGroup = 8;
    const int per = count / kXcds, extra = count % kXcds;
    const int x = id % kXcds, k = id / kXcds;
    const int t = x * per + (x < extra ? x : extra) + k;
    const int group = t / (kGroup * in_tiles);
    const int first = group * kGroup;
    const int height = out_tiles - first < kGroup ? out_tiles - first : kGroup;
    const int r = t - first * in_tiles;
    o = first + r % height;
    i = r / height;
}

template <int DT, int FMT, int TILE>
__global__ __launch_bounds__(kGradThreads) void weight_grad_kernel(GradArgs g) {
    using G = GradTile<TILE>;
    constexpr int F = G::kFrags;
    __shared__ __attribute__((aligned(16))) char smem[2 * G::kStageBytes];
    const int tiles = g.in_tiles * g.out_tiles;
    const int split = blockIdx.x / tiles;
    int ot, in;
    place_tile(blockIdx.x % tiles, tiles, g.out_tiles, g.in_tiles, ot, in);
    const int o0 = ot * TILE, i0 = in * TILE;
    const int64_t t0 = split * g.split_rows;
    const int64_t t_end = t0 + g.split_rows < g.rows ? t0 + g.split_rows : g.rows;
    f16v acc[F][F];
#pragma unroll
    for (int m = 0; m < F; ++m)
#pragma unroll
        for (int n = 0; n < F; ++n) acc[m][n] = f16v{};
    float bsum[kOct] = {};
    const bool bias = g.dbias != nullptr && in == 0;
    // Tiles that lie inside the operands take the unguarded loads, with 32-bit
    // offsets within 64 tokens; the last tokens and the edges the guarded ones.
    const bool inside = o0 + TILE <= g.out_cols && i0 + TILE <= g.pitch && g.dy_stride < (int64_t(1) << 24) &&
                        g.pitch < (int64_t(1) << 24);
    const int all = int((t_end - t0 + kTokens - 1) / kTokens);
    const int whole = inside ? int((t_end - t0) / kTokens) : 0;
    if (whole > 0) {
        if (bias)
            grad_loop<DT, FMT, TILE, kWhole, true>(g, smem, o0, i0, t0, whole, t_end, bsum, acc);
        else
            grad_loop<DT, FMT, TILE, kWhole, false>(g, smem, o0, i0, t0, whole, t_end, bsum, acc);
    }
    if (all > whole)
        grad_loop<DT, FMT, TILE, kGuarded, true>(g, smem, o0, i0, t0 + int64_t(whole) * kTokens, all - whole, t_end, bsum,
                                                 acc);

    // Through LDS in fp32, 32 rows of a wave's quarter at a time, into octs of a row.
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int in8 = (g.in_cols + kOct - 1) / kOct * kOct;
    float* strip = reinterpret_cast<float*>(smem) + wave * 32 * G::kWave;
#pragma unroll
    for (int m = 0; m < F; ++m) {
        __syncthreads();
#pragma unroll
        for (int n = 0; n < F; ++n)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                strip[(8 * (r / 4) + 4 * (lane >> 5) + r % 4) * G::kWave + 32 * n + (lane & 31)] = acc[m][n][r];
        __syncthreads();
        constexpr int kOctsW = G::kWave / kOct, kRows = 64 / kOctsW;
#pragma unroll
        for (int p = 0; p < 32 / kRows; ++p) {
            const int r = p * kRows + lane / kOctsW;
            const int o = o0 + (wave >> 1) * G::kWave + 32 * m + r;
            const int c = i0 + (wave & 1) * G::kWave + (lane % kOctsW) * kOct;
            if (o >= g.out_cols || c >= g.in_cols) continue;
            const f4* src = reinterpret_cast<const f4*>(strip + r * G::kWave + (lane % kOctsW) * kOct);
            const f4 lo = src[0], hi = src[1];
            if (g.splits > 1) {
                f4* dst = reinterpret_cast<f4*>(g.partials + (int64_t(split) * g.out_cols + o) * in8 + c);
                dst[0] = lo;
                dst[1] = hi;
                continue;
            }
            float v[kOct] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint16_t* out = g.dweight + int64_t(o) * g.in_cols;
            if (g.accumulate) {
                float old[kOct];
                widen_oct<DT>(load_oct(out, c, g.in_cols), old);
#pragma unroll
                for (int k = 0; k < kOct; ++k) v[k] += old[k];
            }
            store_oct(out, c, g.in_cols, narrow_oct<DT>(v));
        }
    }
    if (!bias) return;
    // The threads of a column's octs, added in row order.
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);
    const int oct = tid % G::kOcts, row = tid / G::kOcts;
#pragma unroll
    for (int k = 0; k < kOct; ++k) sums[row * TILE + oct * kOct + k] = bsum[k];
    __syncthreads();
    const int o = o0 + tid;
    if (tid >= TILE || o >= g.out_cols) return;
    float total = sums[tid];
    for (int r = 1; r < G::kRowsPerPass; ++r) total += sums[r * TILE + tid];
    if (g.splits > 1) {
        g.bias_partials[int64_t(split) * g.out_cols + o] = total;
        return;
    }
    if (g.accumulate) total += widen<DT>(g.dbias[o]);
    g.dbias[o] = static_cast<uint16_t>(narrow<DT>(total));
}

// Adds the splits' partial gradients in split order; an oct per thread.  The
// last threads do the bias, one element each.
constexpr int kJoinThreads = 256;

template <int DT>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(GradArgs g) {
    const int in_octs = (g.in_cols + kOct - 1) / kOct;
    const int64_t octs = int64_t(in_octs) * g.out_cols;
    const int64_t id = int64_t(blockIdx.x) * kJoinThreads + threadIdx.x;
    if (id < octs) {
        const int64_t o = id / in_octs;
        const int c = int(id % in_octs) * kOct;
        const float* p = g.partials + (o * in_octs + c / kOct) * kOct;
        float v[kOct] = {};
        for (int s = 0; s < g.splits; ++s) {
            const f4* q = reinterpret_cast<const f4*>(p + s * octs * kOct);
            const f4 lo = q[0], hi = q[1];
            v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
            v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
        }
        uint16_t* out = g.dweight + o * g.in_cols;
        if (g.accumulate) {
            float old[kOct];
            widen_oct<DT>(load_oct(out, c, g.in_cols), old);
#pragma unroll
            for (int k = 0; k < kOct; ++k) v[k] += old[k];
        }
        store_oct(out, c, g.in_cols, narrow_oct<DT>(v));
    } else if (g.dbias != nullptr && id - octs < g.out_cols) {
        const int o = int(id - octs);
        float total = 0.0f;
        for (int s = 0; s < g.splits; ++s) total += g.bias_partials[int64_t(s) * g.out_cols + o];
        if (g.accumulate) total += widen<DT>(g.dbias[o]);
        g.dbias[o] = static_cast<uint16_t>(narrow<DT>(total));
    }
}

// ---------------------------------------------------------------------------
// Launch glue
// ---------------------------------------------------------------------------

struct GradShape {
    int tile, in_tiles, out_tiles, splits;
    int64_t split_rows;
};

constexpr int kCus = 256;

inline GradShape grad_shape(int64_t rows, int64_t in_cols, int64_t out_cols) {
    const auto tiles = [&](int tile) {
        return std::max<int64_t>(1, ceil_div(in_cols, int64_t(tile))) * ceil_div(out_cols, int64_t(tile));
    };
    GradShape s;
    s.tile = tiles(256) >= kCus ? 256 : 128;
    s.in_tiles = int(std::max<int64_t>(1, ceil_div(in_cols, int64_t(s.tile))));
    s.out_tiles = int(ceil_div(out_cols, int64_t(s.tile)));
    const int64_t n = tiles(s.tile), steps = std::max<int64_t>(1, ceil_div(rows, int64_t(kTokens)));
    // few tiles and many tokens: enough splits for two blocks per CU, of at least 8 staged tiles each
    int64_t want = n >= kCus ? 1 : std::min(ceil_div(2 * kCus, n), std::max<int64_t>(1, steps / 8));
    s.split_rows = ceil_div(steps, want) * kTokens;
    s.splits = int(std::max<int64_t>(1, ceil_div(rows, s.split_rows)));
    return s;
}

inline bool weight_grad_sizes_ok(int64_t rows, int64_t in_cols, int64_t out_cols) {
    return act_size_ok(rows, in_cols) && act_size_ok(rows, out_cols) &&
           (in_cols == 0 || out_cols <= ZERO_MAX_ELEMS / in_cols);
}

inline int64_t partial_floats(const GradShape& s, int64_t in_cols, int64_t out_cols) {
    return s.splits > 1 ? int64_t(s.splits) * out_cols * ceil_div(in_cols, int64_t(kOct)) * kOct : 0;
}

inline int64_t weight_grad_workspace(int64_t rows, int64_t in_cols, int64_t out_cols) {
    if (rows == 0 || out_cols == 0) return 0;
    const GradShape s = grad_shape(rows, in_cols, out_cols);
    return s.splits > 1 ? 4 * (partial_floats(s, in_cols, out_cols) + s.splits * out_cols) : 0;
}

}  // namespace
}  // namespace zf

using namespace zf;

extern "C" {

int64_t zero_act_weight_grad_workspace_bytes(int64_t rows, int64_t in_cols, int64_t out_cols) {
    if (!weight_grad_sizes_ok(rows, in_cols, out_cols)) {
        fail(ZERO_EINVAL, "zero_act_weight_grad_workspace_bytes: rows, in_cols or out_cols out of range");
        return -1;
    }
    ok();
    return weight_grad_workspace(rows, in_cols, out_cols);
}

int zero_act_weight_grad(const void* dy, int64_t dy_stride, int dtype, const void* codes, const float* scales,
                         int format, int64_t rows, int64_t in_cols, int64_t out_cols, int accumulate, void* dweight,
                         void* dbias, void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "zero_act_weight_grad";
    if (int rc = check_sizes(fn, rows, in_cols, dtype, format)) return rc;
    if (!weight_grad_sizes_ok(rows, in_cols, out_cols))
        return fail(ZERO_EINVAL, std::string(fn) + ": rows * out_cols or in_cols * out_cols out of range");
    if (out_cols == 0) return ok();
    if ((in_cols > 0 && bad_ptr(dweight, 2)) || (dbias != nullptr && (addr(dbias) & 1)))
        return fail(ZERO_EINVAL, std::string(fn) + ": dweight NULL, or dweight or dbias not 2-byte aligned");
    const int64_t wb = weight_grad_workspace(rows, in_cols, out_cols);
    if (rows > 0) {
        if (int rc = check_matrix(fn, "dy", dy, rows, out_cols, dy_stride)) return rc;
        if (in_cols > 0)
            if (int rc = check_checkpoint(fn, "", codes, scales)) return rc;
        if (wb > 0 && (bad_ptr(workspace, 16) || workspace_bytes < wb))
            return fail(ZERO_EINVAL, std::string(fn) + ": workspace NULL, not 16-byte aligned or less than zero_act_weight_grad_workspace_bytes");
    }
    const int64_t pitch = act_pitch(in_cols), bpr = act_blocks(in_cols);
    const Area areas[] = {mat16("dy", dy, rows, out_cols, dy_stride, false),
                          flat("codes", codes, rows * pitch, false),
                          flat("scales", scales, 4 * rows * bpr, false),
                          flat("dweight", dweight, 2 * in_cols * out_cols, true),
                          flat("dbias", dbias, 2 * out_cols, true),
                          flat("workspace", workspace, wb, true)};
    if (int rc = check_overlaps(fn, areas, 6)) return rc;
    if ((rows == 0 && accumulate) || (in_cols == 0 && dbias == nullptr)) return ok();
    hipStream_t s = static_cast<hipStream_t>(stream);
    const GradShape sh = grad_shape(rows, in_cols, out_cols);
    float* partials = static_cast<float*>(workspace);
    const GradArgs args{in16(dy), dy_stride, in8(codes), pitch, scales, int(bpr), rows, int(in_cols), int(out_cols),
                        sh.in_tiles, sh.out_tiles, sh.splits, sh.split_rows, accumulate, out16(dweight), out16(dbias),
                        partials, sh.splits > 1 ? partials + partial_floats(sh, in_cols, out_cols) : nullptr};
    const dim3 grid(unsigned(int64_t(sh.in_tiles) * sh.out_tiles * sh.splits));
    hipError_t e = with_types(dtype, format, [&](auto dt, auto fmt) {
        constexpr int D = decltype(dt)::value, M = decltype(fmt)::value;
        return sh.tile == 256 ? launch(weight_grad_kernel<D, M, 256>, grid, dim3(kGradThreads), s, args)
                              : launch(weight_grad_kernel<D, M, 128>, grid, dim3(kGradThreads), s, args);
    });
    if (e != hipSuccess || sh.splits <= 1) return hip_status(e, fn);
    const int64_t threads = ceil_div(in_cols, int64_t(kOct)) * out_cols + (dbias != nullptr ? out_cols : 0);
    e = with_dtype(dtype, [&](auto dt) {
        return launch(join_kernel<decltype(dt)::value>, dim3(unsigned(ceil_div(threads, int64_t(kJoinThreads)))),
                      dim3(kJoinThreads), s, args);
    });
    return hip_status(e, fn);
}

}  // extern "C"
