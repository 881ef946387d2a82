// Residual addition, root-mean-square norm and 8-bit quantisation of a block's
// activations in one pass: eq_rmsnorm.
//
//   h[t, c]   = x[t, c] + res[t, c]                 (fp32)
//   rstd[t]   = 1 / sqrt(mean_c h[t, c]^2 + eps)    (fp32 sum)
//   bf16:       out = bf16(h gamma rstd)
//   8 bits:     p = fp32(h gamma), m[t] = max_c |p|, Q = 127 (Int8) or 448 (E4M3)
//               out = round_to_nearest_even(p * (Q / m)),  scale[t] = m rstd / Q
// The token's scale is the absolute maximum of its normalised values over Q,
// and rstd, a factor of every value and of the maximum, cancels out of the
// codes: they come from one maximum and two fp32 roundings, so they do not
// depend on the order in which the squares are summed.
//
// Squares leave the fp32 range long before the values do.  A row whose sum of
// squares reaches 2^126 (or is no number) is normalised from h 2^-80, an exact
// scaling that cancels out of the output and of the scale:
//   rstd = 2^-80 / sqrt(mean (h 2^-80)^2 + eps 2^-160)
// It rounds only what is below 2^-46, 100 binary orders under the row's own
// root mean square.  Rows of ordinary size pay one comparison per thread and one per row.
//
// Bound by memory: x and res are read once, res_out, out and the scale written
// once; a thread keeps its part of a token's h between the sum and the output.  One
// row (token) is shared by T threads that hold E values each, as vectors of 8
// consecutive columns (16-byte loads and stores) where the buffers allow it, else
// column by column (coalesced, any width and address).  Up to 16 values (16384
// columns) they stay in registers, column by column up to 8; with 32 values, and
// with 16 column by column, 8 to 264 bytes per thread go through local memory.
// Measured (B200): 8192 tokens x 8192, fp32 x, bf16 residual, E4M3 out: 102 us,
// 5.9 TB/s, 0.9 of a plain copy's rate; one token x 8192: 3.1 us, the launch.  With a
// block of 512 threads and more, few blocks fit an SM: 2000 x 16384, the same types, 61 us
// (0.74), 2000 x 28672 in bf16 91 us (0.68).
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "eqw_internal.h"
#include "eqw_launch.cuh"

namespace {

constexpr uint32_t kMaxThreads = 1024;
constexpr uint32_t kMaxPerThread = 32;
constexpr uint32_t kMaxNormCols = kMaxThreads * kMaxPerThread;
constexpr float kLargeSum = 0x1p126f;  // of squares, from which a row is scaled
constexpr float kScaleDown = 0x1p-80f;  // 32768 squares of 2^128 2^-80 stay in range

struct NormParams {
    const void *x;
    const void *res;      // nullptr: none
    void *res_out;
    const uint16_t *gamma;  // nullptr: ones
    void *out;
    float *out_scale;
    uint64_t x_stride, res_stride, res_out_stride, out_stride;  // elements
    uint32_t tokens, cols, out_type;
    uint32_t row_threads;  // T, a multiple of 32
    float eps;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// A value read once (evicted first).  Not through the read-only path: this grid may be resident before the
// kernel that writes the value has ended.
template <class T>
__device__ __forceinline__ T load_once(const T *p) {
    return __ldcs(p);
}

// The larger of two values, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <bool F32>
__device__ __forceinline__ void load8(const void *p, uint64_t at, float (&v)[8]) {
    if constexpr (F32) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
        const float4 a = load_once(q), b = load_once(q + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 a = load_once(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at));
        v[0] = bf16_lo(a.x), v[1] = bf16_hi(a.x), v[2] = bf16_lo(a.y), v[3] = bf16_hi(a.y);
        v[4] = bf16_lo(a.z), v[5] = bf16_hi(a.z), v[6] = bf16_lo(a.w), v[7] = bf16_hi(a.w);
    }
}

template <bool F32>
__device__ __forceinline__ float load1(const void *p, uint64_t at) {
    if constexpr (F32) return load_once(static_cast<const float *>(p) + at);
    return __uint_as_float((uint32_t)load_once(static_cast<const uint16_t *>(p) + at) << 16);
}

template <bool F32>
__device__ __forceinline__ void store8(void *p, uint64_t at, const float (&v)[8]) {
    if constexpr (F32) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at) =
            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    }
}

template <bool F32>
__device__ __forceinline__ void store1(void *p, uint64_t at, float v) {
    if constexpr (F32)
        static_cast<float *>(p)[at] = v;
    else
        static_cast<__nv_bfloat16 *>(p)[at] = __float2bfloat16_rn(v);
}

// The T threads of the block's row `sub`; a block whose rows have several warps each holds at most two.
__device__ __forceinline__ void row_sync(uint32_t sub, uint32_t T) {
    __syncwarp();
    if (sub == 0)
        asm volatile("bar.sync 1, %0;" ::"r"(T) : "memory");
    else
        asm volatile("bar.sync 2, %0;" ::"r"(T) : "memory");
}

// Codes of already scaled values (|v| <= Q up to one rounding), round to nearest even.
__device__ __forceinline__ uint32_t code_int8(float v) { return (uint32_t)__float2int_rn(v) & 0xFFu; }
__device__ __forceinline__ uint32_t code_e4m3(float v) { return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3); }
__device__ __forceinline__ uint32_t code_e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// How a thread's 8 neighbouring columns lie in memory.
//   kAligned  on 16-byte boundaries in every row
//   kShifted  vectors of 8 elements counted from the buffers' starts, which all
//             buffers' rows cut alike (row strides congruent modulo 8): a row's
//             first and last vector may be partly another row's, and those
//             elements are taken one by one
//   kScalar   a thread's columns are T apart and taken one by one
enum : int { kAligned = 0, kShifted = 1, kScalar = 2 };

// XF, RF: x / residual in fp32 (else bf16).  E: values per thread.
template <bool XF, bool RF, int MODE, int E>
__global__ void __launch_bounds__(kMaxThreads, 1) eq_rmsnorm_kernel(const NormParams P) {
    constexpr int NV = E / 8;
    __shared__ float sum_s[32], max_s[32];
    next_kernel_may_start();
    const uint32_t T = P.row_threads;
    const uint32_t sub = threadIdx.x / T, i = threadIdx.x % T;  // row of the block, place in the row
    const uint32_t token = blockIdx.x * (blockDim.x / T) + sub;
    const bool live = token < P.tokens;  // a block's last rows may be past the end: they only join the barrier
    const bool has_res = P.res != nullptr, narrow = P.out_type != EQ_BF16;
    const int cols = live ? (int)P.cols : 0;
    // value k of this thread is column col(k) of the row
    const int off = MODE == kShifted ? (int)((token * P.x_stride) & 7u) : 0;  // the row's start within a vector
    const auto vec_col = [&](int j) { return (int)(j * T + i) * 8 - off; };
    const auto whole = [&](int c) { return c >= 0 && c + 8 <= cols; };
    const auto col = [&](int k) { return MODE == kScalar ? (int)(k * T + i) : vec_col(k / 8) + k % 8; };
    const auto in_row = [&](int c) { return c >= 0 && c < cols; };
    float h[E];
#pragma unroll
    for (int k = 0; k < E; ++k) h[k] = 0.f;
    previous_kernel_done();
    if constexpr (MODE == kScalar) {
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (in_row(col(k))) h[k] = load1<XF>(P.x, token * P.x_stride + col(k));
        if (has_res) {
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (in_row(col(k))) h[k] = __fadd_rn(h[k], load1<RF>(P.res, token * P.res_stride + col(k)));
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (in_row(col(k))) store1<RF>(P.res_out, token * P.res_out_stride + col(k), h[k]);
        }
    } else {
        // loads of all vectors first, then the sums
        float r[E];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = vec_col(j);
            float(&hv)[8] = *reinterpret_cast<float(*)[8]>(h + 8 * j);
            if (whole(c)) {
                load8<XF>(P.x, token * P.x_stride + c, hv);
            } else if (MODE == kShifted) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (in_row(c + k)) hv[k] = load1<XF>(P.x, token * P.x_stride + c + k);
            }
        }
        if (has_res) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = vec_col(j);
                float(&rv)[8] = *reinterpret_cast<float(*)[8]>(r + 8 * j);
#pragma unroll
                for (int k = 0; k < 8; ++k) rv[k] = 0.f;
                if (whole(c)) {
                    load8<RF>(P.res, token * P.res_stride + c, rv);
                } else if (MODE == kShifted) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (in_row(c + k)) rv[k] = load1<RF>(P.res, token * P.res_stride + c + k);
                }
            }
#pragma unroll
            for (int k = 0; k < E; ++k) h[k] = __fadd_rn(h[k], r[k]);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = vec_col(j);
                float(&hv)[8] = *reinterpret_cast<float(*)[8]>(h + 8 * j);
                if (whole(c)) {
                    store8<RF>(P.res_out, token * P.res_out_stride + c, hv);
                } else if (MODE == kShifted) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (in_row(c + k)) store1<RF>(P.res_out, token * P.res_out_stride + c + k, hv[k]);
                }
            }
        }
    }
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < E; ++k) sum = fmaf(h[k], h[k], sum);
    float own = sum;  // this thread's squares, scaled where its values are
    const bool scaled = !(own < kLargeSum);
    if (scaled) {
        own = 0.f;
#pragma unroll
        for (int k = 0; k < E; ++k) {
            h[k] *= kScaleDown;
            own = fmaf(h[k], h[k], own);
        }
    }
    // h becomes p = h gamma (absent columns stay 0)
    if (P.gamma) {
        if constexpr (MODE == kAligned) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = vec_col(j);
                if (whole(c)) {
                    const uint4 g = *reinterpret_cast<const uint4 *>(P.gamma + c);
                    const uint32_t w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        h[8 * j + 2 * k] = __fmul_rn(h[8 * j + 2 * k], bf16_lo(w[k]));
                        h[8 * j + 2 * k + 1] = __fmul_rn(h[8 * j + 2 * k + 1], bf16_hi(w[k]));
                    }
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (in_row(col(k))) h[k] = __fmul_rn(h[k], __uint_as_float((uint32_t)P.gamma[col(k)] << 16));
        }
    }
    float top = 0.f;
    const auto maximum = [&]() {
        top = 0.f;
        if (narrow) {
#pragma unroll
            for (int k = 0; k < E; ++k) top = max_nan(top, fabsf(h[k]));
        }
    };
    // sum and maximum over the row's T threads: warps, then the warps' results
    const auto over_row = [&](bool again) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
            top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        }
        if (T > 32) {
            const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, warps = T / 32;
            if (again) row_sync(sub, T);  // the first results have been read
            if (lane == 0) {
                sum_s[warp] = sum;
                max_s[warp] = top;
            }
            if (again)
                row_sync(sub, T);
            else
                __syncthreads();
            const uint32_t first = sub * warps;
            sum = lane < warps ? sum_s[first + lane] : 0.f;
            top = lane < warps ? max_s[first + lane] : 0.f;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
                top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            }
        }
    };
    maximum();
    over_row(false);
    float eps = P.eps;
    // A scaled thread's own sum is part of the row's, so this branch, the same for all of a row's threads, is
    // taken wherever one has scaled its values.
    if (!(sum < kLargeSum)) {
        eps = eps * kScaleDown * kScaleDown;
        if (!scaled) {
            own = own * kScaleDown * kScaleDown;
#pragma unroll
            for (int k = 0; k < E; ++k) h[k] *= kScaleDown;
        }
        sum = own;
        maximum();
        over_row(true);
    }
    if (!live) return;
    const float rstd = __frsqrt_rn(__fdiv_rn(sum, (float)P.cols) + eps);
    if (!narrow) {
#pragma unroll
        for (int k = 0; k < E; ++k) h[k] = __fmul_rn(h[k], rstd);
        if constexpr (MODE == kScalar) {
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (in_row(col(k))) store1<false>(P.out, token * P.out_stride + col(k), h[k]);
        } else {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int c = vec_col(j);
                float(&hv)[8] = *reinterpret_cast<float(*)[8]>(h + 8 * j);
                if (whole(c)) {
                    store8<false>(P.out, token * P.out_stride + c, hv);
                } else if (MODE == kShifted) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (in_row(c + k)) store1<false>(P.out, token * P.out_stride + c + k, hv[k]);
                }
            }
        }
        return;
    }
    const bool int8 = P.out_type == EQ_INT8;
    const float q = int8 ? 127.f : 448.f;
    if (i == 0) P.out_scale[token] = __fdiv_rn(__fmul_rn(top, rstd), q);
    // Q / m would overflow below 2^-119: such a row is scaled up (exactly) first
    if (top < 0x1p-100f) {
        top *= 0x1p100f;
#pragma unroll
        for (int k = 0; k < E; ++k) h[k] *= 0x1p100f;
    }
    const float inv = top == 0.f ? 0.f : __fdiv_rn(q, top);  // a row of zeros: codes and scale 0
    uint8_t *out = static_cast<uint8_t *>(P.out) + token * P.out_stride;
#pragma unroll
    for (int k = 0; k < E; ++k) h[k] = __fmul_rn(h[k], inv);
    const auto code = [&](float v) { return (uint8_t)(int8 ? code_int8(v) : code_e4m3(v)); };
    if constexpr (MODE == kScalar) {
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (in_row(col(k))) out[col(k)] = code(h[k]);
    } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = vec_col(j);
            const float *v = h + 8 * j;
            if (whole(c)) {
                uint2 o;
                if (int8) {
                    o.x = code_int8(v[0]) | code_int8(v[1]) << 8 | code_int8(v[2]) << 16 | code_int8(v[3]) << 24;
                    o.y = code_int8(v[4]) | code_int8(v[5]) << 8 | code_int8(v[6]) << 16 | code_int8(v[7]) << 24;
                } else {
                    o.x = code_e4m3x2(v[0], v[1]) | code_e4m3x2(v[2], v[3]) << 16;
                    o.y = code_e4m3x2(v[4], v[5]) | code_e4m3x2(v[6], v[7]) << 16;
                }
                *reinterpret_cast<uint2 *>(out + c) = o;
            } else if (MODE == kShifted) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (in_row(c + k)) out[c + k] = code(v[k]);
            }
        }
    }
}

using NormKernel = void (*)(NormParams);

template <int MODE, int E>
NormKernel norm_kernel(bool xf, bool rf) {
    if (xf) return rf ? eq_rmsnorm_kernel<true, true, MODE, E> : eq_rmsnorm_kernel<true, false, MODE, E>;
    return rf ? eq_rmsnorm_kernel<false, true, MODE, E> : eq_rmsnorm_kernel<false, false, MODE, E>;
}

template <int MODE>
NormKernel norm_kernel(uint32_t e, bool xf, bool rf) {
    return e == 8 ? norm_kernel<MODE, 8>(xf, rf) : e == 16 ? norm_kernel<MODE, 16>(xf, rf) : norm_kernel<MODE, 32>(xf, rf);
}

bool real_type(uint32_t t) { return t == EQ_BF16 || t == EQ_F32; }

bool aligned(const void *p, uint64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

}  // namespace

extern "C" EQW_API int eq_rmsnorm(const eq_rmsnorm_args *a, cudaStream_t s) {
    const eqw::NvtxScope nvtx_range("eq_rmsnorm");
    if (!a || !real_type(a->x_type) || !std::isfinite(a->eps) || !(a->eps > 0.f)) return EQ_ERR_INVALID_ARG;
    const bool narrow = a->out_type == EQ_INT8 || a->out_type == EQ_E4M3;
    if (!narrow && a->out_type != EQ_BF16) return EQ_ERR_INVALID_ARG;
    if (a->res && !real_type(a->res_type)) return EQ_ERR_INVALID_ARG;
    if (!a->tokens || !a->cols) return EQ_OK;
    if (!a->x || !a->out || (narrow && !a->out_scale) || (a->res != nullptr) != (a->res_out != nullptr))
        return EQ_ERR_INVALID_ARG;
    if (a->x_stride < a->cols || a->out_stride < a->cols ||
        (a->res && (a->res_stride < a->cols || a->res_out_stride < a->cols)))
        return EQ_ERR_INVALID_ARG;
    const bool xf = a->x_type == EQ_F32, rf = a->res && a->res_type == EQ_F32;
    const uint64_t xb = xf ? 4 : 2, rb = rf ? 4 : 2, ob = narrow ? 1 : 2;
    if (!aligned(a->x, xb) || !aligned(a->out, ob) || !aligned(a->gamma, 2) || !aligned(a->out_scale, 4) ||
        (a->res && (!aligned(a->res, rb) || !aligned(a->res_out, rb))))
        return EQ_ERR_INVALID_ARG;
    if (a->cols > kMaxNormCols) return EQ_ERR_UNSUPPORTED;
    // vectors of 8 columns where every buffer starts on a vector and all rows cut the vectors alike
    const bool bases = aligned(a->x, 16) && aligned(a->out, 8 * ob) && (!a->res || (aligned(a->res, 16) && aligned(a->res_out, 16)));
    const auto like_x = [&](uint64_t stride) { return stride % 8 == a->x_stride % 8; };
    const bool shifted = bases && like_x(a->out_stride) && (!a->res || (like_x(a->res_stride) && like_x(a->res_out_stride)));
    int mode = kScalar;
    if (shifted && a->x_stride % 8 == 0 && a->cols % 8 == 0 && aligned(a->gamma, 16))
        mode = kAligned;
    else if (shifted && a->cols + 7 <= kMaxNormCols)  // a row may start inside a vector
        mode = kShifted;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return EQ_ERR_CUDA;
    // Values per thread: few while there are few rows per SM (a row's latency counts), else twice as many
    // (half the barriers' weight).  515 x 5121 bf16 + fp32: 10.2 us with 8, 12.2 with 16; 8192 x 8192 fp32 + bf16:
    // 114 and 103; 1111 x 4096: 10.1 and 9.5.  Rows only are counted, not how many blocks of their width fit: the
    // first takes two rounds of blocks (two of 672 threads per SM), the last too (five of 256).
    uint32_t e = a->tokens <= 4 * (uint32_t)sms ? 8 : 16;
    const uint32_t span = a->cols + (mode == kShifted ? 7 : 0);
    while (e < kMaxPerThread && (uint64_t)e * kMaxThreads < span) e *= 2;
    NormParams P;
    P.x = a->x, P.res = a->res, P.res_out = a->res_out, P.gamma = static_cast<const uint16_t *>(a->gamma);
    P.out = a->out, P.out_scale = a->out_scale;
    P.x_stride = a->x_stride, P.res_stride = a->res_stride, P.res_out_stride = a->res_out_stride;
    P.out_stride = a->out_stride;
    P.tokens = a->tokens, P.cols = a->cols, P.out_type = a->out_type, P.eps = a->eps;
    P.row_threads = (span + 32 * e - 1) / (32 * e) * 32;
    const uint32_t rows_per_block = std::max(1u, 128u / P.row_threads);
    const uint32_t grid = (uint32_t)(((uint64_t)a->tokens + rows_per_block - 1) / rows_per_block);
    if (grid > 0x7FFFFFFFu) return EQ_ERR_UNSUPPORTED;
    const NormKernel fn = mode == kAligned ? norm_kernel<kAligned>(e, xf, rf)
                          : mode == kShifted ? norm_kernel<kShifted>(e, xf, rf) : norm_kernel<kScalar>(e, xf, rf);
    void *args[] = {&P};
    return launch_overlapped((const void *)fn, grid, P.row_threads * rows_per_block, 0, 0, args, s) ? EQ_OK : EQ_ERR_CUDA;
}
