// Weight and bias gradient of a linear layer from the 8-bit checkpoint of its
// input, for MI355X (gfx950, wave64), and its C-ABI entry point.  The formulas
// are in include/zero_flat.h.
//
//   weight_grad_kernel   a tile of dW = dY^T X, X restored from the checkpoint
//   join_kernel          adds the partial tiles of a product split over tokens
//
// The contraction runs over tokens, the slow axis of both operands: a matrix
// instruction wants 8 consecutive tokens of one column per lane.  Tiles of 32
// tokens are staged in LDS as they lie in memory ([token][column], 16 bits) and
// read with the transposing LDS load (ds_read_b64_tr_b16: 16 lanes read 4 rows
// of 16 columns and each lane receives one column of the 4 rows).  The codes are
// decoded on their way into LDS, between the matrix instructions of the previous
// tile, or for large products beforehand, once for all blocks.
//
// Large products: 16384 tokens, 4096 -> 16384 in bf16 take 1610-1680 us, 1310-1370
// TFLOP/s, where 16384^3 by the library reaches 1584 and the library's product of this
// shape (both operands transposed in memory) takes 1820-1860 us.  Two things bound it.
// At the full clock of 2.1 GHz the matrix units are busy 60-62% of the cycles: one wave
// per SIMD issues everything else between its own matrix instructions.  Over a run of such
// calls the clock falls to 1.6-1.9 GHz with the power drawn and the share rises to
// 66-68%, so the energy around the products counts too.

#include "act.h"

namespace zf {
namespace {

typedef short s4v __attribute__((ext_vector_type(4)));
typedef short s8v __attribute__((ext_vector_type(8)));
typedef __bf16 b8v __attribute__((ext_vector_type(8)));
typedef _Float16 h8v __attribute__((ext_vector_type(8)));

constexpr int kTokens = 32;       // tokens per staged tile: one matrix instruction's depth
constexpr int kGradThreads = 256; // four waves, two by two

// A block's tile: TILE outputs x TILE inputs; a wave does a quarter of it in
// FRAGS x FRAGS 16 x 16 fragments (the 16 x 16 x 32 instruction: 2040 TFLOP/s
// sustained on random operands held in registers, where 32 x 32 x 16 reaches 1785,
// as the clock falls with the power drawn).  LDS rows are TILE 16-bit values in units
// of 16 columns (32 bytes); token t's units are kept at unit ^ x(t), x(t) = t mod 4
// + 4 (t / 8 mod 2), so that the 16 rows which a transposing read touches spread
// evenly over the banks.
template <int TILE>
struct GradTile {
    static constexpr int kRowBytes = 2 * TILE;
    static constexpr int kOperandBytes = kTokens * kRowBytes;
    static constexpr int kStageBytes = 2 * kOperandBytes;
    static constexpr int kWave = TILE / 2;
    static constexpr int kFrags = kWave / 16;
    static constexpr int kOcts = TILE / kOct;                    // per row
    static constexpr int kRowsPerPass = kGradThreads / kOcts;
    static constexpr int kPasses = kTokens / kRowsPerPass;
};

// The input operand: codes (FMT a ZERO_ACT_* format, decoded while staged) or, for
// kDecoded, 16-bit values that a pass over the checkpoint restored beforehand.
constexpr int kDecoded = 0;

struct GradArgs {
    const uint16_t* dy;
    int64_t dy_stride;
    const uint8_t* input;
    int64_t pitch;  // bytes from row to row of the input
    const float* scales;
    int blocks_per_row;
    int64_t rows;
    int in_cols, out_cols;
    int in_tiles, out_tiles;
    int splits;
    int64_t split_rows;  // tokens per split, a multiple of kTokens
    int unchecked;  // the strides allow kWhole's loads
    int accumulate;
    uint16_t* dweight;
    uint16_t* dbias;
    float* partials;       // splits > 1: [splits][out_cols][in8] fp32, then
    float* bias_partials;  // [splits][out_cols]
};

// Order of a step's instructions: after every two matrix instructions, which keep
// the matrix unit busy for 8 issue slots, its share of the LDS reads (one of 32 at
// 256 x 256, two of 16 at 128 x 128) and a few of the others, so that a lone wave per
// SIMD does not leave it idle.  Without it 16384 tokens, 4096 -> 16384, take 1907
// instead of 1613 us and 4096 tokens, 1600 -> 6400, 113 instead of 105.
template <int F, int VALU>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int i = 0; i < F * F / 2; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);             // MFMA
        __builtin_amdgcn_sched_group_barrier(0x100, 8 / F, 0);         // LDS read
        __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);          // VALU
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);             // LDS write
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);             // global load
    }
}

template <int DT>
__device__ __forceinline__ f4 mfma16(const s8v& a, const s8v& b, const f4& c) {
    if constexpr (DT == ZERO_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8v, a), __builtin_bit_cast(b8v, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8v, a), __builtin_bit_cast(h8v, b), c, 0, 0, 0);
}

// 8 tokens of one column per lane: two transposing reads, 4 tokens each.
template <int ROW_BYTES>
__device__ __forceinline__ s8v read_frag(const char* p) {
    typedef __attribute__((address_space(3))) s4v* lds4;
    const s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p));
    const s4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(p + 4 * ROW_BYTES));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ constexpr int swizzle(int token) { return (token & 3) | ((token >> 1) & 4); }

constexpr int kUncheckedTokens = 4 * kTokens;

// How a block's tokens are loaded.  kGuarded: every load is checked against the
// operands' edges, and what lies outside is staged as zero.  kWhole, for at least
// 128 tokens: only the last 64 tokens, which are staged first, are checked.  The
// other loads need no check: an oct that lies outside the columns reads the row's
// first columns instead and one that straddles the end of a row reads on into the
// next row (these columns of the product are not stored), and the rows exist.
enum { kWhole, kGuarded };

// One tile of dW over tokens [t0, t_end), BIAS: with the column sums of dY.
//
// Tokens are staged 32 at a time, in pairs of such steps; the last pair comes
// first.  While step k is multiplied from registers, the fragments of step k + 1
// are read from one LDS stage, step k + 2 goes from registers to the other (whose
// step k every wave has read before the barrier at the start), and step k + 4 is
// loaded into the registers this frees: two steps' time for a load to arrive, and
// one barrier per step.
template <int DT, int FMT, int TILE, int MODE, bool BIAS>
__device__ __forceinline__ void grad_tile(const GradArgs& g, char* smem, int o0, int i0, int64_t t0, int64_t t_end,
                                          int split) {
    using G = GradTile<TILE>;
    constexpr int F = G::kFrags, P = G::kPasses;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int oct = tid % G::kOcts, row = tid / G::kOcts;
    const int l = lane & 15, grp = lane >> 4;
    // first of this lane's rows in a fragment, and its 4 columns there
    const int frag = (grp * 8 + (l >> 2)) * G::kRowBytes + (l & 3) * 8;
    const int frag_x = swizzle(grp * 8 + (l >> 2));
    int fa[F], fb[F];
#pragma unroll
    for (int f = 0; f < F; ++f) {
        fa[f] = frag + ((((wave >> 1) * F + f) ^ frag_x) << 5);
        fb[f] = frag + ((((wave & 1) * F + f) ^ frag_x) << 5) + G::kOperandBytes;
    }
    // at least one pair: without tokens it is staged as zeros
    const int pairs = int((t_end - t0 + 2 * kTokens - 1) / (2 * kTokens));
    const int steps = 2 * (pairs > 0 ? pairs : 1);

    constexpr int kBytes = FMT == kDecoded ? 2 : 1;  // per input element
    typedef std::conditional_t<FMT == kDecoded, u4, u2> InputOct;
    u4 a[2][P];
    InputOct b[2][P];
    float s[2][P];
    const int o = o0 + oct * kOct, i = i0 + oct * kOct;
    const auto load_checked = [&](int step, int set, int j) {
        const int64_t t = t0 + int64_t(step) * kTokens + j * G::kRowsPerPass + row;
        a[set][j] = u4{0u, 0u, 0u, 0u};
        b[set][j] = InputOct{};
        s[set][j] = 0.0f;
        if (t < t_end) {
            if (o < g.out_cols) a[set][j] = load_oct_shared(g.dy + t * g.dy_stride, o, g.out_cols);
            if (i < g.in_cols) {
                b[set][j] = *reinterpret_cast<const InputOct*>(g.input + t * g.pitch + i * kBytes);
                if constexpr (FMT != kDecoded) s[set][j] = g.scales[t * g.blocks_per_row + i / kActBlock];
            }
        }
    };
    // kWhole: a uniform base per operand and pass, and constant 32-bit offsets
    const char* pa = reinterpret_cast<const char*>(g.dy + t0 * g.dy_stride);
    const char* pb = reinterpret_cast<const char*>(g.input + t0 * g.pitch);
    const char* ps = reinterpret_cast<const char*>(g.scales + t0 * g.blocks_per_row + i0 / kActBlock);
    const uint32_t oa = (uint32_t(row) * uint32_t(g.dy_stride) + (o < g.out_cols ? o : 0)) * 2u;
    const uint32_t ob = uint32_t(row) * uint32_t(g.pitch) + (i < g.in_cols ? i : 0) * kBytes;
    const uint32_t os = uint32_t(row) * uint32_t(g.blocks_per_row) * 4u;
    int loaded = 0;
    // pass j of the next step to load, into `set`
    const auto load = [&](int set, int j) {
        if constexpr (MODE == kGuarded) {
            load_checked(loaded, set, j);
        } else {
            constexpr int64_t rp = G::kRowsPerPass;
            a[set][j] = *reinterpret_cast<const u4_any*>(pa + 2 * j * rp * g.dy_stride + oa);
            b[set][j] = *reinterpret_cast<const InputOct*>(pb + j * rp * g.pitch + ob);
            if constexpr (FMT != kDecoded)
                s[set][j] = *reinterpret_cast<const float*>(ps + 4 * j * rp * g.blocks_per_row + os);
        }
    };
    // on to the step after it, or past the end the last one again (staged but never used)
    const auto advance = [&]() {
        ++loaded;
        const bool more = loaded < steps - 2;
        pa += more ? 2 * kTokens * g.dy_stride : 0;
        pb += more ? kTokens * g.pitch : 0;
        ps += more ? int64_t(4) * kTokens * g.blocks_per_row : 0;
    };
    float bsum[kOct] = {};
    const auto store = [&](int set, int j, bool fresh) {
        const int r = row + j * G::kRowsPerPass;
        char* p = smem + set * G::kStageBytes + r * G::kRowBytes + (((oct >> 1) ^ swizzle(r)) << 5) + ((oct & 1) << 4);
        *reinterpret_cast<u4*>(p) = a[set][j];
        if constexpr (FMT == kDecoded)
            *reinterpret_cast<u4*>(p + G::kOperandBytes) = b[set][j];
        else
            *reinterpret_cast<u4*>(p + G::kOperandBytes) = decode_oct<DT, FMT>(b[set][j], s[set][j]);
        if constexpr (BIAS) {
            float v[kOct];
            widen_oct<DT>(a[set][j] & (fresh ? ~0u : 0u), v);
#pragma unroll
            for (int k = 0; k < kOct; ++k) bsum[k] += v[k];
        }
    };

    s8v y[2][F], x[F];  // outputs' and inputs' fragments
#pragma unroll
    for (int set = 0; set < 2; ++set)
#pragma unroll
        for (int j = 0; j < P; ++j) load_checked(steps - 2 + set, set, j);
#pragma unroll
    for (int set = 0; set < 2; ++set) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            store(set, j, true);
            load(set, j);
        }
        advance();
        // the loop's waits assume the loads in this order
        __builtin_amdgcn_sched_barrier(0);
    }
    f4 acc[F][F];
#pragma unroll
    for (int m = 0; m < F; ++m)
#pragma unroll
        for (int n = 0; n < F; ++n) {
            // The empty asm makes each zero a value of its own: accumulators that start from one
            // shared constant were moved between registers in every pass of the loop.
            acc[m][n] = f4{};
            asm("" : "+a"(acc[m][n]));
        }
    __syncthreads();
#pragma unroll
    for (int f = 0; f < F; ++f) {
        y[0][f] = read_frag<G::kRowBytes>(smem + fa[f]);
        x[f] = read_frag<G::kRowBytes>(smem + fb[f]);
    }
    const auto step = [&](int k, auto parity) {
        constexpr int S = decltype(parity)::value;
        const char* next = smem + (S ^ 1) * G::kStageBytes;
        __syncthreads();
#pragma unroll
        for (int n = 0; n < F; ++n) {
            y[S ^ 1][n] = read_frag<G::kRowBytes>(next + fa[n]);
#pragma unroll
            for (int m = 0; m < F; ++m) acc[m][n] = mfma16<DT>(y[S][m], x[n], acc[m][n]);
            x[n] = read_frag<G::kRowBytes>(next + fb[n]);
            constexpr int every = F / P;
            if (n % every == every - 1) {
                store(S, n / every, k + 2 < steps);
                load(S, n / every);
            }
        }
        advance();
        if constexpr (MODE == kWhole) interleave<F, (FMT == kDecoded ? 1 : 3) + (BIAS ? 2 : 0)>();
        __builtin_amdgcn_sched_barrier(0);
    };
    for (int k = 0; k < steps; k += 2) {
        step(k, std::integral_constant<int, 0>{});
        step(k + 1, std::integral_constant<int, 1>{});
    }

    // Through LDS in fp32, 16 rows of a wave's quarter at a time, into octs of a row.
    // Each wave has a strip of its own and LDS serves a wave in order, so within a
    // wave only the compiler has to keep the order (the fences).  Rows are 4 floats
    // longer than needed: the four groups of rows a write touches differ in banks.
    constexpr int kStrip = G::kWave + 4;
    static_assert(4 * 16 * kStrip * 4 <= 2 * G::kStageBytes, "the strips fit the stages");
    const int in8 = (g.in_cols + kOct - 1) / kOct * kOct;
    float* strip = reinterpret_cast<float*>(smem) + wave * 16 * kStrip;
    __syncthreads();
#pragma unroll
    for (int m = 0; m < F; ++m) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int n = 0; n < F; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) strip[(4 * (lane >> 4) + r) * kStrip + 16 * n + (lane & 15)] = acc[m][n][r];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        constexpr int kOctsW = G::kWave / kOct, kRows = 64 / kOctsW;
#pragma unroll
        for (int p = 0; p < 16 / kRows; ++p) {
            const int r = p * kRows + lane / kOctsW;
            const int oo = o0 + (wave >> 1) * G::kWave + 16 * m + r;
            const int c = i0 + (wave & 1) * G::kWave + (lane % kOctsW) * kOct;
            if (oo >= g.out_cols || c >= g.in_cols) continue;
            const f4* src = reinterpret_cast<const f4*>(strip + r * kStrip + (lane % kOctsW) * kOct);
            const f4 lo = src[0], hi = src[1];
            if (g.splits > 1) {
                f4* dst = reinterpret_cast<f4*>(g.partials + (int64_t(split) * g.out_cols + oo) * in8 + c);
                dst[0] = lo;
                dst[1] = hi;
                continue;
            }
            float v[kOct] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            uint16_t* out = g.dweight + int64_t(oo) * g.in_cols;
            if (g.accumulate) {
                float old[kOct];
                widen_oct<DT>(load_oct(out, c, g.in_cols), old);
#pragma unroll
                for (int k = 0; k < kOct; ++k) v[k] += old[k];
            }
            store_oct(out, c, g.in_cols, narrow_oct<DT>(v));
        }
    }
    if (!BIAS || g.dbias == nullptr || i0 != 0) return;
    // The threads of a column's octs, added in row order.
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int k = 0; k < kOct; ++k) sums[row * TILE + oct * kOct + k] = bsum[k];
    __syncthreads();
    const int oo = o0 + tid;
    if (tid >= TILE || oo >= g.out_cols) return;
    float total = sums[tid];
    for (int r = 1; r < G::kRowsPerPass; ++r) total += sums[r * TILE + tid];
    if (g.splits > 1) {
        g.bias_partials[int64_t(split) * g.out_cols + oo] = total;
        return;
    }
    if (g.accumulate) total += widen<DT>(g.dbias[oo]);
    g.dbias[oo] = static_cast<uint16_t>(narrow<DT>(total));
}

// Blocks are dispatched round-robin to the 8 XCDs; each XCD takes a contiguous
// run of tiles, ordered so that the 32 tiles in flight (one per CU) form a patch of
// 4 output tiles by 8 input tiles that share operand panels in its L2 (8 by 4 was
// 4% slower at 16384 tokens, 4096 -> 16384).
__device__ __forceinline__ void place_tile(int id, int count, int out_tiles, int in_tiles, int& o, int& i) {
    constexpr int kXcds = 8, kGroup = 4;
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
    __shared__ __attribute__((aligned(16))) char smem[2 * G::kStageBytes];
    const int tiles = g.in_tiles * g.out_tiles;
    const int split = blockIdx.x / tiles;
    int ot, in;
    place_tile(blockIdx.x % tiles, tiles, g.out_tiles, g.in_tiles, ot, in);
    const int o0 = ot * TILE, i0 = in * TILE;
    const int64_t t0 = split * g.split_rows;
    const int64_t t_end = t0 + g.split_rows < g.rows ? t0 + g.split_rows : g.rows;
    // TILE 256 is launched for unchecked calls in one split of at least 128 tokens only.
    // 256 accumulators and two sets of fragments and loads leave 9 or 10 registers of its
    // loop in scratch memory (40 or 44 bytes per lane); with a checked loop beside it the
    // kernel kept 157 to 229 there.
    if (TILE == 128 && !(g.unchecked && t_end - t0 >= kUncheckedTokens)) {
        if constexpr (TILE == 128) grad_tile<DT, FMT, TILE, kGuarded, true>(g, smem, o0, i0, t0, t_end, split);
    } else if (g.dbias != nullptr && in == 0) {
        grad_tile<DT, FMT, TILE, kWhole, true>(g, smem, o0, i0, t0, t_end, split);
    } else {
        grad_tile<DT, FMT, TILE, kWhole, false>(g, smem, o0, i0, t0, t_end, split);
    }
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
    int64_t split_rows, most_splits;  // the latter never falls as rows grow
    bool decode;                      // restore the input first
};

constexpr int kCus = 256;

// Restoring the input first costs a launch (3 us) and 3 bytes per element, and saves
// every output tile the decoding, which draws issue slots and power from the matrix
// units.  Measured without and with (us), INT8:
//   256 x 256 tiles  16384 tokens 4096 -> 16384 1839 / 1631; 16384 tokens 16384 -> 2048
//                    898 / 917, -> 1024 456 / 526; 2048 tokens 4096 -> 4096 64 / 64;
//                    512 tokens 4096 -> 4096 24 / 28
//   128 x 128 tiles  4096 tokens 1600 -> 6400 120 / 105, 6400 -> 1600 120 / 116; 16384
//                    tokens 2048 -> 1024 89 / 109; 48 tokens 1600 -> 4800 8 / 10
constexpr int64_t kDecodeOutputs = 1536;       // with 128 x 128 tiles
constexpr int64_t kDecodeOutputsLarge = 2048;  // with 256 x 256 tiles, which decode half as often
constexpr int64_t kDecodeProducts = 10000000000;

inline GradShape grad_shape(int64_t rows, int64_t in_cols, int64_t out_cols) {
    const auto tiles = [&](int tile) {
        return std::max<int64_t>(1, ceil_div(in_cols, int64_t(tile))) * ceil_div(out_cols, int64_t(tile));
    };
    GradShape s;
    // 256 x 256 tiles where they give every CU one (128 x 128 tiles take 2124 instead of 1613
    // us for 16384 tokens, 4096 -> 16384; 256 x 256 ones 143 instead of 105 us for 4096 tokens,
    // 1600 -> 6400) and the unchecked loop runs.
    s.tile = rows >= kUncheckedTokens && tiles(256) >= kCus ? 256 : 128;
    s.in_tiles = int(std::max<int64_t>(1, ceil_div(in_cols, int64_t(s.tile))));
    s.out_tiles = int(ceil_div(out_cols, int64_t(s.tile)));
    const int64_t n = tiles(s.tile), steps = std::max<int64_t>(1, ceil_div(rows, int64_t(kTokens)));
    // few tiles and many tokens: enough splits for two blocks per CU, of at least 16 staged tiles each
    s.most_splits = n >= kCus ? 1 : std::min(ceil_div(2 * kCus, n), std::max<int64_t>(1, steps / 16));
    s.split_rows = ceil_div(steps, s.most_splits) * kTokens;
    s.splits = int(std::max<int64_t>(1, ceil_div(rows, s.split_rows)));
    const int64_t outputs = tiles(256) >= kCus ? kDecodeOutputsLarge : kDecodeOutputs;
    s.decode = out_cols >= outputs && rows > 0 && in_cols * out_cols >= kDecodeProducts / rows;
    return s;
}

inline bool weight_grad_sizes_ok(int64_t rows, int64_t in_cols, int64_t out_cols) {
    return act_size_ok(rows, in_cols) && act_size_ok(rows, out_cols) &&
           (in_cols == 0 || out_cols <= ZERO_MAX_ELEMS / in_cols);
}

inline int64_t partial_floats(const GradShape& s, int64_t in_cols, int64_t out_cols) {
    return s.splits > 1 ? int64_t(s.splits) * out_cols * ceil_div(in_cols, int64_t(kOct)) * kOct : 0;
}

inline int64_t decoded_bytes(const GradShape& s, int64_t rows, int64_t in_cols) {
    return s.decode ? 2 * rows * act_pitch(in_cols) : 0;
}

// The restored input, if there is one, then the partial gradients.  Sized by what
// never falls as rows grow, so that a workspace for the longest batch serves all.
inline int64_t weight_grad_workspace(int64_t rows, int64_t in_cols, int64_t out_cols) {
    if (rows == 0 || out_cols == 0) return 0;
    const GradShape s = grad_shape(rows, in_cols, out_cols);
    const int64_t in8 = ceil_div(in_cols, int64_t(kOct)) * kOct;
    return decoded_bytes(s, rows, in_cols) + (s.most_splits > 1 ? 4 * s.most_splits * out_cols * (in8 + 1) : 0);
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
            return fail(ZERO_EINVAL, std::string(fn) + ": workspace NULL, not 16-byte aligned or too small");
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
    GradShape sh = grad_shape(rows, in_cols, out_cols);
    const int64_t in_pitch = sh.decode ? 2 * pitch : pitch;
    const int64_t far = int64_t(1) << 24;  // a pass's offsets stay within 32 bits
    const bool unchecked = in_cols > 0 && dy_stride >= kOct && dy_stride < far && in_pitch < far;
    if (sh.tile == 256 && !unchecked) {  // (one split; the workspace stays as it was sized)
        sh.tile = 128;
        sh.in_tiles = int(std::max<int64_t>(1, ceil_div(in_cols, int64_t(128))));
        sh.out_tiles = int(ceil_div(out_cols, int64_t(128)));
    }
    char* ws = static_cast<char*>(workspace);
    float* partials = reinterpret_cast<float*>(ws + decoded_bytes(sh, rows, in_cols));
    if (sh.decode)
        if (int rc = zero_act_restore(codes, scales, format, rows, in_cols, ws, pitch, dtype, stream)) return rc;
    const GradArgs args{in16(dy), dy_stride, sh.decode ? in8(ws) : in8(codes), in_pitch, scales,
                        int(bpr), rows, int(in_cols), int(out_cols), sh.in_tiles, sh.out_tiles, sh.splits,
                        sh.split_rows, int(unchecked), accumulate, out16(dweight), out16(dbias), partials,
                        sh.splits > 1 ? partials + partial_floats(sh, in_cols, out_cols) : nullptr};
    const dim3 grid(unsigned(int64_t(sh.in_tiles) * sh.out_tiles * sh.splits));
    const auto run = [&](auto dt, auto fmt) {
        constexpr int D = decltype(dt)::value, M = decltype(fmt)::value;
        return sh.tile == 256 ? launch(weight_grad_kernel<D, M, 256>, grid, dim3(kGradThreads), s, args)
                              : launch(weight_grad_kernel<D, M, 128>, grid, dim3(kGradThreads), s, args);
    };
    const auto run_decoded = [&](auto dt) { return run(dt, std::integral_constant<int, kDecoded>{}); };
    hipError_t e = sh.decode ? with_dtype(dtype, run_decoded) : with_types(dtype, format, run);
    if (e != hipSuccess || sh.splits <= 1) return hip_status(e, fn);
    const int64_t threads = ceil_div(in_cols, int64_t(kOct)) * out_cols + (dbias != nullptr ? out_cols : 0);
    e = with_dtype(dtype, [&](auto dt) {
        return launch(join_kernel<decltype(dt)::value>, dim3(unsigned(ceil_div(threads, int64_t(kJoinThreads)))),
                      dim3(kJoinThreads), s, args);
    });
    return hip_status(e, fn);
}

}  // extern "C"
