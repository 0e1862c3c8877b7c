// norm.cu -- root-mean-square norm with the residual's addition, in bf16 or as
// MXFP8 codes with E8M0 block scales, and its backward pass.
//
//   h = bf16(x + residual)          (h = x without a residual)
//   rstd = 1 / sqrt(mean(h^2) + eps)
//   y = h * rstd * w
// The statistic is taken over h as stored, so that the backward pass, which
// reads h, differentiates the function the forward pass computed.  y stays in
// FP32 until its one rounding, to bf16 or to MXFP8.
//
//   n = h * rstd,  c = mean(w * dy * n)
//   dx = dh + rstd * (w * dy - n * c)     (the gradient of x and of residual)
//   dw = sum over rows of dy * n
#include "common.cuh"

#include <algorithm>

namespace nvfp4 {
namespace {

constexpr int kMaxCols = 32768;  // 1024 threads x 4 vectors of 8 elements
constexpr int max_threads(int per) { return per == 4 ? 1024 : 256 * per; }

struct NormArgs {
    const uint4* x;
    const uint4* residual;  // NULL = none
    const void* weight;
    uint4* h;               // NULL without a residual
    uint4* y;               // NULL = not wanted
    float* rstd;
    uint32_t* amax;
    uint2* mx_q;
    uint8_t* mx_sf;
    int64_t ldx, ldr, ldh, ldy;  // in 16-byte vectors
    int64_t rows, padded_rows;
    int nvec;                    // 16-byte vectors per row
    float eps;
    int mx_tiled;
};

template <bool W32>
__device__ __forceinline__ void load_weight(const void* w, int v, float (&f)[8])
{
    if constexpr (W32) {
        const float4 a = static_cast<const float4*>(w)[2 * v], b = static_cast<const float4*>(w)[2 * v + 1];
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
        unpack8(static_cast<const uint4*>(w)[v], f);
    }
}

// Sum over the block, the same value in every thread; `s` holds one number per
// warp and is free again after the call's second barrier.
template <typename T>
__device__ __forceinline__ T block_sum(T v, T* s)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    T t = (threadIdx.x & 31) < warps ? s[threadIdx.x & 31] : T(0);
#pragma unroll
    for (int d = 16; d; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
    __syncthreads();
    return t;
}

// One CTA per row, V 16-byte vectors (8 elements) per thread held in registers
// between the statistic and the output: every tensor is read and written once.
template <int V, bool W32>
__global__ void __launch_bounds__(max_threads(V)) rmsnorm_kernel(const NormArgs a)
{
    __shared__ float s_sum[32];
    __shared__ double s_wide[32];
    float top = 0.0f;  // largest |y| as stored
    bool nan = false;
    for (int64_t row = blockIdx.x; row < a.padded_rows; row += gridDim.x) {
        if (row >= a.rows) {  // padding rows of the tiled scale layout: zero bytes
            for (int g = threadIdx.x; g < a.nvec / 16; g += blockDim.x)
                *reinterpret_cast<uint32_t*>(a.mx_sf + sf_mma_offset(row, 4 * g, a.nvec / 4)) = 0u;
            continue;
        }
        uint4 h[V];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            h[i] = v < a.nvec ? a.x[row * a.ldx + v] : make_uint4(0, 0, 0, 0);
        }
        if (a.residual) {
            uint4 r[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = threadIdx.x + i * blockDim.x;
                r[i] = v < a.nvec ? a.residual[row * a.ldr + v] : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int v = threadIdx.x + i * blockDim.x;
                float f[8], g[8];
                unpack8(h[i], f);
                unpack8(r[i], g);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] += g[j];
                h[i] = pack8(f);
                if (v < a.nvec) a.h[row * a.ldh + v] = h[i];
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float f[8];
            unpack8(h[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
        }
        sum = block_sum(sum, s_sum);
        float rstd = __frsqrt_rn(__fdiv_rn(sum, static_cast<float>(8 * a.nvec)) + a.eps);
        if (!(sum < 0x1p120f) || (sum < 0x1p-100f && a.eps < 0x1p-100f)) {
            // squares out of FP32's range (the whole row's CTA takes this branch)
            double wide = 0.0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float f[8];
                unpack8(h[i], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) wide += static_cast<double>(f[j]) * f[j];
            }
            wide = block_sum(wide, s_wide);
            rstd = static_cast<float>(1.0 / sqrt(wide / (8.0 * a.nvec) + static_cast<double>(a.eps)));
        }
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            const bool in = v < a.nvec;
            float f[8], w[8];
            unpack8(h[i], f);
            if (in) {
                load_weight<W32>(a.weight, v, w);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * w[j];
            if (a.y) {
                const uint4 p = pack8(f);
                if (in) a.y[row * a.ldy + v] = p;
                if (a.amax) {
                    float q[8];
                    unpack8(p, q);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        top = fmaxf(top, fabsf(q[j]));
                        nan |= q[j] != q[j];
                    }
                }
            }
            if (a.mx_q) {
                // four lanes hold a 32-element block; nvec is a multiple of 4, so a
                // block's lanes are all inside the row or all outside
                float m = absmax3(absmax3(f[0], f[1], f[2]), absmax3(f[3], f[4], f[5]), absmax3(f[6], f[7], 0.0f));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                // floor(log2 m) - 8, at least -127: from the exponent field (0 and
                // subnormal m have field 0)
                const int e = max(static_cast<int>(__float_as_uint(m) >> 23) - 135, -127);
                const float inv = __uint_as_float(e == -127 ? 0x7F000000u : static_cast<uint32_t>(127 - e) << 23);
                uint32_t byte = static_cast<uint32_t>(e + 127);
                uint2 c;
                c.x = e4m3x2_rne_sat(f[1] * inv, f[0] * inv) | e4m3x2_rne_sat(f[3] * inv, f[2] * inv) << 16;
                c.y = e4m3x2_rne_sat(f[5] * inv, f[4] * inv) | e4m3x2_rne_sat(f[7] * inv, f[6] * inv) << 16;
                if (in) a.mx_q[row * a.nvec + v] = c;
                if (a.mx_tiled) {  // nvec is a multiple of 16: one word of four scales per 16 lanes
                    byte |= __shfl_down_sync(0xffffffffu, byte, 4) << 8;
                    byte |= __shfl_down_sync(0xffffffffu, byte, 8) << 16;
                    if (in && (v & 15) == 0)
                        *reinterpret_cast<uint32_t*>(a.mx_sf + sf_mma_offset(row, v / 4, a.nvec / 4)) = byte;
                } else if (in && (v & 3) == 0) {
                    a.mx_sf[row * (a.nvec / 4) + v / 4] = static_cast<uint8_t>(byte);
                }
            }
        }
    }
    if (a.amax) {
        if (nan) top = __uint_as_float(0x7FC00000u);
        uint32_t t = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
        if ((threadIdx.x & 31) == 0) atomicMax(a.amax, t);
    }
}

struct NormBackArgs {
    const uint4* dy;
    const uint4* h;
    const uint4* dh;  // NULL = none
    const void* weight;
    const float* rstd;
    uint4* dx;
    float* partial;   // [gridDim.x, cols]; NULL = dw not wanted
    int64_t lddy, ldh, lddh, lddx;
    int64_t rows;
    int nvec;
};

// One CTA per row at a time; the columns' dy * n sums stay in registers over
// all the CTA's rows and go out once, as one row of `partial`.
template <int V, bool W32>
__global__ void __launch_bounds__(max_threads(V)) rmsnorm_backward_kernel(const NormBackArgs a)
{
    __shared__ float s_sum[32];
    float dw[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        uint4 h[V], dy[V], dh[V];
        const float rstd = a.rstd[row];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            const uint4 zero = make_uint4(0, 0, 0, 0);
            h[i] = v < a.nvec ? a.h[row * a.ldh + v] : zero;
            dy[i] = v < a.nvec ? a.dy[row * a.lddy + v] : zero;
            dh[i] = v < a.nvec && a.dh ? a.dh[row * a.lddh + v] : zero;
        }
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            float n[8], g[8], w[8];
            unpack8(h[i], n);
            unpack8(dy[i], g);
            if (v < a.nvec) {
                load_weight<W32>(a.weight, v, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    n[j] *= rstd;
                    dw[i][j] = fmaf(g[j], n[j], dw[i][j]);
                    sum = fmaf(g[j] * w[j], n[j], sum);
                }
            }
        }
        const float c = __fdiv_rn(block_sum(sum, s_sum), static_cast<float>(8 * a.nvec));
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v >= a.nvec) continue;
            float n[8], g[8], w[8], r[8];
            unpack8(h[i], n);
            unpack8(dy[i], g);
            unpack8(dh[i], r);
            load_weight<W32>(a.weight, v, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[j] = fmaf(rstd, g[j] * w[j] - n[j] * rstd * c, r[j]);
            a.dx[row * a.lddx + v] = pack8(r);
        }
    }
    if (!a.partial) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= a.nvec) continue;
        float4* dst = reinterpret_cast<float4*>(a.partial + (static_cast<int64_t>(blockIdx.x) * a.nvec + v) * 8);
        dst[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
        dst[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    }
}

// dw[c] = sum over the parts, 32 columns per CTA, its 8 warps over the parts in
// a fixed order.
template <bool W32>
__global__ void __launch_bounds__(256) rmsnorm_dw_kernel(const float* partial, int parts, int cols, void* dw)
{
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < cols)
        for (int p = warp; p < parts; p += 8) v += partial[static_cast<int64_t>(p) * cols + c];
    s[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < cols) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += s[i][lane];
        if (W32)
            static_cast<float*>(dw)[c] = t;
        else
            static_cast<__nv_bfloat16*>(dw)[c] = __float2bfloat16_rn(t);
    }
}

// Threads and vectors per thread of a row of nvec vectors.
void row_shape(int nvec, int* threads, int* per)
{
    *per = nvec <= 256 ? 1 : nvec <= 1024 ? 2 : 4;
    *threads = ((nvec + *per - 1) / *per + 31) / 32 * 32;
}

constexpr size_t kNormWorkspaceHead = 256;

// CTAs of the backward pass, each with one row of partial sums in the workspace.
constexpr int kMaxSms = 160;
int backward_grid(int64_t rows, int64_t cols, int sms)
{
    int threads, per;
    row_shape(static_cast<int>(cols / 8), &threads, &per);
    return static_cast<int>(std::min<int64_t>(
        rows, static_cast<int64_t>(std::min(sms, kMaxSms)) * std::max(1, 1024 / threads)));
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_rmsnorm(const void* x_bf16, int64_t ldx, const void* residual_bf16, int64_t ldr,
                                      const void* weight, int weight_dtype, float eps, int64_t rows,
                                      int64_t cols, void* h_bf16, int64_t ldh, void* y_bf16, int64_t ldy,
                                      float* rstd, float* amax_out, uint8_t* mx_q, uint8_t* mx_sf,
                                      int mx_sf_layout, void* stream)
{
    if (!weight || !(eps >= 0.0f)) return NVFP4_ERR_INVALID_ARG;
    if (weight_dtype != NVFP4_OUT_F32 && weight_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_INVALID_ARG;
    if (rows > 0) {  // an empty tensor has no address
        if (!x_bf16 || (!y_bf16 && !mx_q) || (mx_q == nullptr) != (mx_sf == nullptr) ||
            (residual_bf16 == nullptr) != (h_bf16 == nullptr) || (amax_out && !y_bf16))
            return NVFP4_ERR_INVALID_ARG;
    }
    if (mx_sf_layout != NVFP4_SF_ROWMAJOR && mx_sf_layout != NVFP4_SF_MMA) return NVFP4_ERR_INVALID_ARG;
    if (rows < 0 || cols <= 0 || cols % 8 || cols > kMaxCols || ldx < cols) return NVFP4_ERR_SHAPE;
    if ((residual_bf16 && (ldr < cols || ldh < cols)) || (y_bf16 && ldy < cols)) return NVFP4_ERR_SHAPE;
    if (mx_q && cols % (mx_sf_layout == NVFP4_SF_MMA ? 128 : 32)) return NVFP4_ERR_SHAPE;
    if (off16(x_bf16) || off16(residual_bf16) || off16(weight) || off16(h_bf16) || off16(y_bf16) || off16(mx_q) ||
        (reinterpret_cast<uintptr_t>(mx_sf) & 3u) || (reinterpret_cast<uintptr_t>(rstd) & 3u) ||
        (reinterpret_cast<uintptr_t>(amax_out) & 3u) || ldx % 8 || (residual_bf16 && (ldr % 8 || ldh % 8)) ||
        (y_bf16 && ldy % 8))
        return NVFP4_ERR_ALIGN;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
    const int sms = sm100_sms(dev);
    if (!sms) return NVFP4_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (amax_out && cudaMemsetAsync(amax_out, 0, 4, st) != cudaSuccess) return NVFP4_ERR_CUDA;
    if (rows == 0) return NVFP4_OK;
    NormArgs a{};
    a.x = static_cast<const uint4*>(x_bf16), a.residual = static_cast<const uint4*>(residual_bf16);
    a.weight = weight;
    a.h = static_cast<uint4*>(h_bf16), a.y = static_cast<uint4*>(y_bf16);
    a.rstd = rstd, a.amax = reinterpret_cast<uint32_t*>(amax_out);
    a.mx_q = reinterpret_cast<uint2*>(mx_q), a.mx_sf = mx_sf;
    a.ldx = ldx / 8, a.ldr = ldr / 8, a.ldh = ldh / 8, a.ldy = ldy / 8;
    a.rows = rows, a.nvec = static_cast<int>(cols / 8), a.eps = eps;
    a.mx_tiled = mx_q && mx_sf_layout == NVFP4_SF_MMA;
    a.padded_rows = a.mx_tiled ? (rows + 127) / 128 * 128 : rows;
    int threads, per;
    row_shape(a.nvec, &threads, &per);
    const int grid = static_cast<int>(std::min<int64_t>(a.padded_rows, static_cast<int64_t>(sms) * std::max(1, 2048 / threads)));
    const bool w32 = weight_dtype == NVFP4_OUT_F32;
    const auto go = [&](auto kernel) { kernel<<<grid, threads, 0, st>>>(a); };
    if (per == 1) w32 ? go(rmsnorm_kernel<1, true>) : go(rmsnorm_kernel<1, false>);
    else if (per == 2) w32 ? go(rmsnorm_kernel<2, true>) : go(rmsnorm_kernel<2, false>);
    else w32 ? go(rmsnorm_kernel<4, true>) : go(rmsnorm_kernel<4, false>);
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

extern "C" size_t nvfp4_rmsnorm_backward_workspace_size(int64_t rows, int64_t cols)
{
    if (rows <= 0 || cols <= 0 || cols > kMaxCols) return kNormWorkspaceHead;
    const int64_t parts = backward_grid(rows, cols, kMaxSms);
    return kNormWorkspaceHead + static_cast<size_t>(parts * cols) * 4;
}

extern "C" nvfp4_status nvfp4_rmsnorm_backward(const void* dy_bf16, int64_t lddy, const void* h_bf16, int64_t ldh,
                                               const void* dh_bf16, int64_t lddh, const void* weight,
                                               int weight_dtype, const float* rstd, int64_t rows, int64_t cols,
                                               void* dx_bf16, int64_t lddx, void* dweight, void* workspace,
                                               size_t ws_bytes, void* stream)
{
    if (!weight || (rows > 0 && (!dy_bf16 || !h_bf16 || !rstd || !dx_bf16))) return NVFP4_ERR_INVALID_ARG;
    if (weight_dtype != NVFP4_OUT_F32 && weight_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_INVALID_ARG;
    if (rows < 0 || cols <= 0 || cols % 8 || cols > kMaxCols || lddy < cols || ldh < cols || lddx < cols ||
        (dh_bf16 && lddh < cols))
        return NVFP4_ERR_SHAPE;
    if (off16(dy_bf16) || off16(h_bf16) || off16(dh_bf16) || off16(weight) || off16(dx_bf16) || off16(dweight) ||
        (reinterpret_cast<uintptr_t>(rstd) & 3u) || lddy % 8 || ldh % 8 || lddx % 8 || (dh_bf16 && lddh % 8))
        return NVFP4_ERR_ALIGN;
    if (dweight && (!workspace || off16(workspace) || ws_bytes < nvfp4_rmsnorm_backward_workspace_size(rows, cols)))
        return NVFP4_ERR_WORKSPACE;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
    const int sms = sm100_sms(dev);
    if (!sms) return NVFP4_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool w32 = weight_dtype == NVFP4_OUT_F32;
    if (workspace && ws_bytes >= 16 &&
        cudaMemsetAsync(static_cast<uint32_t*>(workspace) + 2, 0, 4, st) != cudaSuccess)
        return NVFP4_ERR_CUDA;
    if (rows == 0) {
        if (dweight && cudaMemsetAsync(dweight, 0, cols * (w32 ? 4 : 2), st) != cudaSuccess) return NVFP4_ERR_CUDA;
        return NVFP4_OK;
    }
    NormBackArgs a{};
    a.dy = static_cast<const uint4*>(dy_bf16), a.h = static_cast<const uint4*>(h_bf16);
    a.dh = static_cast<const uint4*>(dh_bf16), a.weight = weight, a.rstd = rstd;
    a.dx = static_cast<uint4*>(dx_bf16);
    a.partial = dweight ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kNormWorkspaceHead) : nullptr;
    a.lddy = lddy / 8, a.ldh = ldh / 8, a.lddh = lddh / 8, a.lddx = lddx / 8;
    a.rows = rows, a.nvec = static_cast<int>(cols / 8);
    int threads, per;
    row_shape(a.nvec, &threads, &per);
    const int grid = backward_grid(rows, cols, sms);
    const auto go = [&](auto kernel) { kernel<<<grid, threads, 0, st>>>(a); };
    if (per == 1) w32 ? go(rmsnorm_backward_kernel<1, true>) : go(rmsnorm_backward_kernel<1, false>);
    else if (per == 2) w32 ? go(rmsnorm_backward_kernel<2, true>) : go(rmsnorm_backward_kernel<2, false>);
    else w32 ? go(rmsnorm_backward_kernel<4, true>) : go(rmsnorm_backward_kernel<4, false>);
    if (cudaGetLastError() != cudaSuccess) return NVFP4_ERR_CUDA;
    if (dweight) {
        const int blocks = static_cast<int>((cols + 31) / 32);
        if (w32)
            rmsnorm_dw_kernel<true><<<blocks, 256, 0, st>>>(a.partial, grid, static_cast<int>(cols), dweight);
        else
            rmsnorm_dw_kernel<false><<<blocks, 256, 0, st>>>(a.partial, grid, static_cast<int>(cols), dweight);
    }
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
