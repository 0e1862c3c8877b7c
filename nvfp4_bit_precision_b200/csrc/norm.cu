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
constexpr int kNormThreads = 1024;

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
    int mx_tiled, w32;
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

// Sum over the block in warp order, the same value in every thread.  `s` holds
// two rows of one float per warp, used in turn (`turn` flips), so that one barrier
// a sum is enough.
__device__ __forceinline__ float block_sum_turn(float v, float (*s)[32], int& turn)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    float* const row = s[turn];
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) row[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
    for (int w = 0; w < warps; w += 4) {  // (the places past the last warp are zero)
        const float4 q = *reinterpret_cast<const float4*>(row + w);
        t += (q.x + q.y) + (q.z + q.w);
    }
    return t;
}

// bf16(a + b), one rounding: the FP32 sum rounded to bf16 is the same number (it
// is exact unless one addend is below 2^-16 of the other, far from any midpoint).
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

constexpr int kOutY = 1, kOutMx = 2;

// One CTA per row at a time, V 16-byte vectors (8 elements) per thread held in
// registers between the statistic and the output: every tensor is read and written
// once.  The weight stays in registers over the CTA's rows (read again for V = 4,
// whose registers it would not fit), pairs of values go through packed FP32
// arithmetic, and a row costs one barrier, which other CTAs of the SM fill.
//
// What bounds it: HBM.  16384 x 5120 with a residual to MXFP8 (590 MB): 96 us, 6.1
// TB/s; 8191 x 4096 with a residual to bf16 (268 MB): 41 us, 6.5 TB/s; one row of
// 5120: 3.3 us, a launch and two dependent loads.  Unpacked arithmetic with the
// weight loaded for every row took 262 instructions per vector and 123 us.
template <int V, bool RES, int OUT>
__global__ void __launch_bounds__(kNormThreads) rmsnorm_kernel(const NormArgs a)
{
    __shared__ __align__(16) float s_sum[2][32];
    __shared__ double s_wide[32];
    constexpr bool kKeepW = V <= 2;
    wait_for_previous_kernel();
    let_next_kernel_start();
    for (int i = threadIdx.x; i < 64; i += blockDim.x) s_sum[i >> 5][i & 31] = 0.0f;
    __syncthreads();
    const auto weight = [&](int v, float (&w)[8]) {
        if (v >= a.nvec) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 0.0f;
        } else if (a.w32) {
            load_weight<true>(a.weight, v, w);
        } else {
            load_weight<false>(a.weight, v, w);
        }
    };
    float w[kKeepW ? V : 1][8];
    if constexpr (kKeepW) {
#pragma unroll
        for (int i = 0; i < V; ++i) weight(threadIdx.x + i * blockDim.x, w[i]);
    }
    const float cols = static_cast<float>(8 * a.nvec);
    float top = 0.0f;  // largest |y| as stored
    bool nan = false;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.padded_rows; row += gridDim.x) {
        if (row >= a.rows) {  // padding rows of the tiled scale layout: zero bytes
            for (int g = threadIdx.x; g < a.nvec / 16; g += blockDim.x)
                *reinterpret_cast<uint32_t*>(a.mx_sf + sf_mma_offset(row, 4 * g, a.nvec / 4)) = 0u;
            continue;
        }
        uint4 h[V];
        const uint4* const px = a.x + row * a.ldx + threadIdx.x;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const bool in = static_cast<int>(threadIdx.x + i * blockDim.x) < a.nvec;
            h[i] = in ? px[i * blockDim.x] : make_uint4(0, 0, 0, 0);
        }
        if constexpr (RES) {
            const uint4* const pr = a.residual + row * a.ldr + threadIdx.x;
            uint4 r[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool in = static_cast<int>(threadIdx.x + i * blockDim.x) < a.nvec;
                r[i] = in ? pr[i * blockDim.x] : make_uint4(0, 0, 0, 0);
            }
            uint4* const ph = a.h + row * a.ldh + threadIdx.x;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                h[i].x = add_bf16x2(h[i].x, r[i].x), h[i].y = add_bf16x2(h[i].y, r[i].y);
                h[i].z = add_bf16x2(h[i].z, r[i].z), h[i].w = add_bf16x2(h[i].w, r[i].w);
                if (static_cast<int>(threadIdx.x + i * blockDim.x) < a.nvec) ph[i * blockDim.x] = h[i];
            }
        }
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float f[8];
            unpack8(h[i], f);
#pragma unroll
            for (int j = 0; j < 8; j += 2) fma2(s0, s1, f[j], f[j + 1], f[j], f[j + 1]);
        }
        const float sum = block_sum_turn(s0 + s1, s_sum, turn);
        float rstd = __frsqrt_rn(__fdiv_rn(sum, cols) + a.eps);
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
            float f[8];
            unpack8(h[i], f);
            if constexpr (!kKeepW) weight(v, w[0]);
            const float* const wi = w[kKeepW ? i : 0];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                mul2(f[j], f[j + 1], f[j], f[j + 1], rstd, rstd);
                mul2(f[j], f[j + 1], f[j], f[j + 1], wi[j], wi[j + 1]);
            }
            if constexpr ((OUT & kOutY) != 0) {
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
            if constexpr ((OUT & kOutMx) != 0) {
                // four lanes hold a 32-element block; nvec is a multiple of 4, so a
                // block's lanes are all inside the row or all outside
                float m = absmax3(absmax3(f[0], f[1], f[2]), absmax3(f[3], f[4], f[5]), absmax3(f[6], f[7], 0.0f));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                // floor(log2 m) - 8, at least -127, from the exponent field (0 and
                // subnormal m have field 0): the byte is the field - 8, at least 0
                const uint32_t byte = static_cast<uint32_t>(max(static_cast<int>(__float_as_uint(m) >> 23) - 8, 0));
                const float inv = __uint_as_float((254u - byte) << 23);
#pragma unroll
                for (int j = 0; j < 8; j += 2) mul2(f[j], f[j + 1], f[j], f[j + 1], inv, inv);
                uint2 c;
                c.x = e4m3x2_rne_sat(f[1], f[0]) | e4m3x2_rne_sat(f[3], f[2]) << 16;
                c.y = e4m3x2_rne_sat(f[5], f[4]) | e4m3x2_rne_sat(f[7], f[6]) << 16;
                if (in) a.mx_q[row * a.nvec + v] = c;
                if (a.mx_tiled) {  // nvec is a multiple of 16: one word of four scales per 16 lanes
                    uint32_t four = byte | __shfl_down_sync(0xffffffffu, byte, 4) << 8;
                    four |= __shfl_down_sync(0xffffffffu, four, 8) << 16;
                    if (in && (v & 15) == 0)
                        *reinterpret_cast<uint32_t*>(a.mx_sf + sf_mma_offset(row, v / 4, a.nvec / 4)) = four;
                } else if (in && (v & 3) == 0) {
                    a.mx_sf[row * (a.nvec / 4) + v / 4] = static_cast<uint8_t>(byte);
                }
            }
        }
    }
    if (a.amax) {
        if (nan) top = __uint_as_float(0x7FC00000u);
        const uint32_t t = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
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
    uint32_t* status;
    int64_t lddy, ldh, lddh, lddx;
    int64_t rows;
    int nvec;
};

// One CTA per row at a time; the columns' dy * n sums stay in registers over all
// the CTA's rows and go out once, as one row of `partial`.  At 64 registers a
// thread 1024 threads of an SM take part; more registers per thread, and fewer of
// them, were slower (8191 x 4096: 71 registers 66 us, 64 registers 50 us).
//
// What bounds it: HBM.  2^26 elements (h, dy, dh in, dx out, 537 MB) of 4096
// columns: 79 us without dw, 6.8 TB/s, and 85 us with it: the CTAs' rows of
// `partial` (592 x 4096 floats) are written and read once more.
template <int V, bool W32>
__global__ void __launch_bounds__(kNormThreads) rmsnorm_backward_kernel(const NormBackArgs a)
{
    __shared__ __align__(16) float s_sum[2][32];
    int turn = 0;
    for (int i = threadIdx.x; i < 64; i += blockDim.x) s_sum[i >> 5][i & 31] = 0.0f;
    wait_for_previous_kernel();
    let_next_kernel_start();
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.status) *a.status = 0u;
    __syncthreads();
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
        const float c = __fdiv_rn(block_sum_turn(sum, s_sum, turn), static_cast<float>(8 * a.nvec));
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

// dw[c] = sum over the parts, 32 columns per CTA: eight lanes hold a part's 32
// columns, 128 of them take the parts in turn, and their sums meet in shared
// memory in a fixed order.  Launched early (see wait_for_previous_kernel).
template <bool W32>
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(const float* partial, int parts, int cols, void* dw)
{
    __shared__ __align__(16) float s[128][36];
    const int v = threadIdx.x & 7, p0 = threadIdx.x >> 3;
    const int c = blockIdx.x * 32 + 4 * v;
    float4 t = make_float4(0, 0, 0, 0);
    wait_for_previous_kernel();
    let_next_kernel_start();
    if (c < cols) {
#pragma unroll 4
        for (int p = p0; p < parts; p += 128) {
            const float4 q = *reinterpret_cast<const float4*>(partial + static_cast<int64_t>(p) * cols + c);
            t.x += q.x, t.y += q.y, t.z += q.z, t.w += q.w;
        }
    }
    *reinterpret_cast<float4*>(&s[p0][4 * v]) = t;
    __syncthreads();
    // warp w adds rows 4 w .. 4 w + 3, then the first warp the 32 results
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float four = (s[4 * warp][lane] + s[4 * warp + 1][lane]) + (s[4 * warp + 2][lane] + s[4 * warp + 3][lane]);
    __syncthreads();
    s[warp][lane] = four;
    __syncthreads();
    const int col = blockIdx.x * 32 + lane;
    if (warp == 0 && col < cols) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) sum += s[i][lane];
        if (W32)
            static_cast<float*>(dw)[col] = sum;
        else
            static_cast<__nv_bfloat16*>(dw)[col] = __float2bfloat16_rn(sum);
    }
}

// Vectors per thread of a row of nvec vectors, and its threads.  Two, at up to
// 1024 threads (2^26 elements at 512 to 8192 columns: 80 to 93 us forward, 97 to
// 115 us backward; one: 96 to 170 and 107 to 155 us; four: 81 to 100 and 126 to
// 157 us); four for longer rows, and for the MXFP8 output of many rows from 2056
// columns on, whose arithmetic gains most from few threads per row (4096 to 8192
// columns: 81 to 83 us against 87 to 93).  What the rule does not serve: below 512
// columns a row is less than a warp's two vectors a lane (2^26 elements at 128 columns
// 133 us forward, 192 us backward; at 256 73 and 105; at 512 49 and 84), and from
// 16392 columns on the backward pass spills 284 to 312 bytes a thread (2^26 elements
// at 16384 columns 102 us, at 32768 146).
int row_vectors(int nvec) { return nvec <= 2 * kNormThreads ? 2 : 4; }
int row_threads(int nvec, int per) { return ((nvec + per - 1) / per + 31) / 32 * 32; }

constexpr size_t kNormWorkspaceHead = 256;

// CTAs of the backward pass, each with one row of partial sums in the workspace.
constexpr int kMaxSms = 160;
int backward_grid(int64_t rows, int64_t cols, int sms)
{
    const int nvec = static_cast<int>(cols / 8), threads = row_threads(nvec, row_vectors(nvec));
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
    int per = row_vectors(a.nvec);
    if (mx_q && a.nvec > 256 && rows > sms) per = 4;
    const int threads = row_threads(a.nvec, per);
    a.w32 = weight_dtype == NVFP4_OUT_F32;
    const int out = (y_bf16 ? kOutY : 0) | (mx_q ? kOutMx : 0);
    // one wave of CTAs takes all rows: as many as 64 registers a thread leave room for
    const int fit = std::max(1, 1024 / threads);
    const int grid = static_cast<int>(std::min<int64_t>(a.padded_rows, static_cast<int64_t>(sms) * fit));
    cudaError_t err = cudaSuccess;
    const auto go = [&](auto kernel) { err = launch_early(!amax_out, kernel, grid, threads, 0, st, a); };
#define NVFP4_NORM(V, RES)                                                               \
    out == kOutY ? go(rmsnorm_kernel<V, RES, kOutY>)                                     \
                 : out == kOutMx ? go(rmsnorm_kernel<V, RES, kOutMx>) : go(rmsnorm_kernel<V, RES, kOutY | kOutMx>)
    if (residual_bf16) {
        if (per == 2) NVFP4_NORM(2, true);
        else NVFP4_NORM(4, true);
    } else {
        if (per == 2) NVFP4_NORM(2, false);
        else NVFP4_NORM(4, false);
    }
#undef NVFP4_NORM
    return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
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
    if ((workspace && (off16(workspace) || ws_bytes < 16)) ||
        (dweight && (!workspace || ws_bytes < nvfp4_rmsnorm_backward_workspace_size(rows, cols))))
        return NVFP4_ERR_WORKSPACE;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
    const int sms = sm100_sms(dev);
    if (!sms) return NVFP4_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool w32 = weight_dtype == NVFP4_OUT_F32;
    uint32_t* const status = workspace ? static_cast<uint32_t*>(workspace) + 2 : nullptr;
    if (rows == 0) {
        if (status && cudaMemsetAsync(status, 0, 4, st) != cudaSuccess) return NVFP4_ERR_CUDA;
        if (dweight && cudaMemsetAsync(dweight, 0, cols * (w32 ? 4 : 2), st) != cudaSuccess) return NVFP4_ERR_CUDA;
        return NVFP4_OK;
    }
    NormBackArgs a{};
    a.dy = static_cast<const uint4*>(dy_bf16), a.h = static_cast<const uint4*>(h_bf16);
    a.dh = static_cast<const uint4*>(dh_bf16), a.weight = weight, a.rstd = rstd;
    a.dx = static_cast<uint4*>(dx_bf16);
    a.partial = dweight ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kNormWorkspaceHead) : nullptr;
    a.lddy = lddy / 8, a.ldh = ldh / 8, a.lddh = lddh / 8, a.lddx = lddx / 8;
    a.rows = rows, a.nvec = static_cast<int>(cols / 8), a.status = status;
    const int per = row_vectors(a.nvec), threads = row_threads(a.nvec, per);
    const int grid = backward_grid(rows, cols, sms);
    cudaError_t err = cudaSuccess;
    const auto go = [&](auto kernel) { err = launch_early(true, kernel, grid, threads, 0, st, a); };
    if (per == 2) w32 ? go(rmsnorm_backward_kernel<2, true>) : go(rmsnorm_backward_kernel<2, false>);
    else w32 ? go(rmsnorm_backward_kernel<4, true>) : go(rmsnorm_backward_kernel<4, false>);
    if (err != cudaSuccess || cudaGetLastError() != cudaSuccess) return NVFP4_ERR_CUDA;
    if (dweight) {
        const float* const partial = a.partial;
        if (launch_early(true, w32 ? rmsnorm_dw_kernel<true> : rmsnorm_dw_kernel<false>, (cols + 31) / 32, 1024, 0, st,
                         partial, grid, static_cast<int>(cols), dweight) != cudaSuccess)
            return NVFP4_ERR_CUDA;
    }
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
