// Weight and bias gradient of a linear layer from the 8-bit checkpoint of its
// input, for MI355X (gfx950, wave64), and its C-ABI entry point.  The formulas
// are in include/zero_flat.h.
//
//   weight_grad_kernel   dW = dY^T X, X restored from the checkpoint

#include "act.h"

namespace zf {
namespace {

// A block does a 64 x 64 tile of dW, 16 tokens at a time, in fp32.
constexpr int kTile = 64, kTokens = 16, kGradThreads = 256;

template <int DT, int FMT>
__global__ __launch_bounds__(kGradThreads) void weight_grad_kernel(
    const uint16_t* __restrict__ dy, int64_t dy_stride, const uint8_t* __restrict__ codes, int64_t pitch,
    const float* __restrict__ scales, int blocks_per_row, int64_t rows, int64_t in_cols, int64_t out_cols,
    int accumulate, uint16_t* dweight, uint16_t* dbias) {
    __shared__ float a[kTokens][kTile], b[kTokens][kTile];
    const int64_t i0 = int64_t(blockIdx.x) * kTile, o0 = int64_t(blockIdx.y) * kTile;
    const int ti = threadIdx.x % 16, to = threadIdx.x / 16;
    float acc[4][4] = {}, bias[4] = {};
    for (int64_t t0 = 0; t0 < rows; t0 += kTokens) {
        for (int e = threadIdx.x; e < kTokens * kTile; e += kGradThreads) {
            const int r = e / kTile, c = e % kTile;
            const int64_t t = t0 + r;
            a[r][c] = t < rows && o0 + c < out_cols ? widen<DT>(dy[t * dy_stride + o0 + c]) : 0.0f;
            float x = 0.0f;
            if (t < rows && i0 + c < in_cols) {
                float v[4];
                decode_word<FMT>(codes[t * pitch + i0 + c], v);
                x = widen<DT>(narrow_pair<DT>(v[0] * scales[t * blocks_per_row + (i0 + c) / kActBlock], 0.0f) & 0xffffu);
            }
            b[r][c] = x;
        }
        __syncthreads();
        for (int r = 0; r < kTokens; ++r) {
            float x[4], y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                y[k] = a[r][4 * to + k];
                x[k] = b[r][4 * ti + k];
                bias[k] += y[k];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[j][k] = __builtin_fmaf(y[j], x[k], acc[j][k]);
        }
        __syncthreads();
    }
    for (int j = 0; j < 4; ++j) {
        const int64_t o = o0 + 4 * to + j;
        if (o >= out_cols) continue;
        for (int k = 0; k < 4; ++k) {
            const int64_t i = i0 + 4 * ti + k;
            if (i >= in_cols) continue;
            uint16_t* out = dweight + o * in_cols + i;
            *out = static_cast<uint16_t>(narrow<DT>(accumulate ? acc[j][k] + widen<DT>(*out) : acc[j][k]));
        }
        if (dbias != nullptr && i0 == 0 && ti == 0)
            dbias[o] = static_cast<uint16_t>(narrow<DT>(accumulate ? bias[j] + widen<DT>(dbias[o]) : bias[j]));
    }
}

inline bool weight_grad_sizes_ok(int64_t rows, int64_t in_cols, int64_t out_cols) {
    return act_size_ok(rows, in_cols) && act_size_ok(rows, out_cols) &&
           (in_cols == 0 || out_cols <= ZERO_MAX_ELEMS / in_cols);
}

inline int64_t weight_grad_workspace(int64_t rows, int64_t in_cols, int64_t out_cols) { return 0; }

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
    if (rows == 0 && accumulate) return ok();
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid(unsigned(std::max<int64_t>(1, ceil_div(in_cols, int64_t(kTile)))),
                    unsigned(ceil_div(out_cols, int64_t(kTile))));
    const hipError_t e = with_types(dtype, format, [&](auto dt, auto fmt) {
        return launch(weight_grad_kernel<decltype(dt)::value, decltype(fmt)::value>, grid, dim3(kGradThreads), s,
                      in16(dy), dy_stride, in8(codes), pitch, scales, int(bpr), rows, in_cols, out_cols, accumulate,
                      out16(dweight), out16(dbias));
    });
    return hip_status(e, fn);
}

}  // extern "C"
