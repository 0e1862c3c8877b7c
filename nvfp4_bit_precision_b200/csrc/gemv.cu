// gemv.cu -- a few bf16 rows times NVFP4 matrices, dense or one per expert.
//
//   D[i][j] = g * sum_k x[i][k] * (e2m1(q[j][k]) * e4m3(sf[j][k/16]))
//
// The matrices are the ones the block-scaled GEMMs read (codes row-major, scale
// bytes in the tiled order); x stays in bf16 values and sums are FP32.  At this
// few rows the weights' bytes are the work (9/16 byte each); the arithmetic is
// kept below that on the warp-level tensor core instructions:
//  - a code pair becomes two FP16 values in one conversion, and one packed
//    multiply by the block scale gives e2m1 * e4m3 (6 significant bits, between
//    2^-10 and 2688 or zero): exact in FP16;
//  - x is brought into FP16's range by a power of two per token and 128
//    columns, its largest magnitude to [2^14, 2^15): exact for values down to
//    2^-32 of that largest one, and off by at most 2^-40 of it below;
//  - products and their sums are FP32; each 128 columns' sum is scaled back and
//    added in FP32.
#include "common.cuh"

#include <algorithm>

namespace nvfp4 {
namespace {

constexpr int kGemvThreads = 256;
constexpr int kGemvWarps = kGemvThreads / 32;
constexpr int kUnitRows = 64;   // weight rows of a unit: 16 rows of each 32 of a 128-row scale block
constexpr int kChunk = 128;     // columns of a step, 32 per lane
constexpr int kTokStride = 68;  // floats per token in the reduction buffer (64 rows, padded off the banks)
constexpr int kMaxGemvGroups = 256;

struct GemvArgs {
    const uint16_t* x;
    int64_t ldx;
    const int32_t* row_index;      // NULL: row i of x
    int64_t src_rows;
    const int32_t* group_offsets;  // NULL: one matrix
    int groups;
    int64_t rows;
    const uint8_t* q;
    const uint8_t* sf;
    const float* g;
    int64_t n, k;
    int64_t sf_bytes;              // scale bytes of one matrix
    void* out;
    int64_t ldd;
    uint32_t* status;
};

__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&p)[4])
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
        : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// The two E4M3 scales of 32 elements, each in both halves of a register.
__device__ __forceinline__ void scale_pair(uint32_t two, uint32_t& first, uint32_t& second)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    first = __byte_perm(h, 0, 0x1010);
    second = __byte_perm(h, 0, 0x3232);
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_once(const void* p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Lane (r, t) = (lane / 4, lane % 4) of a warp holds, of each 16-row tile, rows
// r and r + 8, and of each 128-column step the 32 columns from 32 t on: one
// 16-byte load of codes a row.  The columns' order inside a matrix instruction
// does not matter as long as both operands agree, so a code word's pairs go in
// as they lie.  The tiles of a unit are rows 32 i + 16 h + 0..15 (i < 4) of a
// 128-row block, whose scales one 16-byte load a lane row holds.
template <int NT, bool F32>
__global__ void __launch_bounds__(kGemvThreads, NT == 1 ? 2 : 1) gemv_kernel(const GemvArgs a)
{
    extern __shared__ float s_red[];  // [warps][8 NT tokens][kTokStride]
    __shared__ int s_first[kMaxGemvGroups], s_rows[kMaxGemvGroups];
    __shared__ int16_t s_group[kMaxGemvGroups];
    __shared__ int s_active;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, t = lane & 3;
    // groups that have rows, in order
    if (warp == 0) {
        int active = 0;
        for (int e0 = 0; e0 < a.groups; e0 += 32) {
            const int e = e0 + lane;
            int64_t lo = 0, hi = 0;
            if (e < a.groups) {
                lo = a.group_offsets ? a.group_offsets[e] : 0;
                hi = a.group_offsets ? a.group_offsets[e + 1] : a.rows;
                lo = min(max(lo, static_cast<int64_t>(0)), a.rows);
                hi = min(hi, a.rows);
            }
            const unsigned has = __ballot_sync(0xffffffffu, hi > lo);
            if (hi > lo) {
                const int at = active + __popc(has & ((1u << lane) - 1));
                s_group[at] = static_cast<int16_t>(e);
                s_first[at] = static_cast<int>(lo);
                s_rows[at] = static_cast<int>(hi - lo);
            }
            active += __popc(has);
        }
        if (lane == 0) s_active = active;
    }
    __syncthreads();
    const int tiles = static_cast<int>((a.n + 127) / 128) * 2;
    const int64_t units = static_cast<int64_t>(s_active) * tiles;
    const int chunks = static_cast<int>((a.k + kChunk - 1) / kChunk);
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int which = static_cast<int>(u / tiles), tile = static_cast<int>(u - static_cast<int64_t>(which) * tiles);
        const int64_t e = s_group[which];
        const int64_t n0 = static_cast<int64_t>(tile >> 1) * 128 + (tile & 1) * 16;  // first row of tile 0
        const uint8_t* q = a.q + (e * a.n + n0) * (a.k / 2);
        const uint8_t* sf = a.sf + e * a.sf_bytes + static_cast<int64_t>(tile >> 1) * (a.k / 64) * 512 + (tile & 1) * 256;
        const float gs = a.g[e];
        for (int tok0 = 0; tok0 < s_rows[which]; tok0 += 8 * NT) {
            const int toks = min(8 * NT, s_rows[which] - tok0);
            const int64_t row0 = s_first[which] + static_cast<int64_t>(tok0);
            const uint16_t* xr[NT];
#pragma unroll
            for (int b = 0; b < NT; ++b) {
                xr[b] = nullptr;
                if (8 * b + r < toks) {
                    int64_t src = row0 + 8 * b + r;
                    if (a.row_index) src = a.row_index[src];
                    if (src < 0 || src >= a.src_rows)
                        record_status(a.status, NVFP4_ERR_INDEX);
                    else
                        xr[b] = a.x + src * a.ldx;
                }
            }
            float acc[4][NT][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int b = 0; b < NT; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][b][j] = 0.0f;
            for (int c = warp; c < chunks; c += kGemvWarps) {
                const int64_t k0 = static_cast<int64_t>(c) * kChunk + 32 * t;
                const bool in = k0 < a.k;
                const uint4 zero = make_uint4(0, 0, 0, 0);
                uint4 code[4][2], sc[2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool have = in && n0 + 32 * i < a.n;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        code[i][h] = have ? load_once(q + (32 * i + r + 8 * h) * (a.k / 2) + k0 / 2) : zero;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sc[h] = in ? load_once(sf + (k0 / 64) * 512 + (r + 8 * h) * 16) : zero;
                // x: 32 columns of token 8 b + r, scaled into FP16's range
                uint32_t xf[NT][16];
                float back[NT];
#pragma unroll
                for (int b = 0; b < NT; ++b) {
                    uint32_t m = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 v = in && xr[b] ? *reinterpret_cast<const uint4*>(xr[b] + k0 + 8 * j) : zero;
                        xf[b][4 * j] = v.x, xf[b][4 * j + 1] = v.y, xf[b][4 * j + 2] = v.z, xf[b][4 * j + 3] = v.w;
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) m = __vmaxu2(m, xf[b][j] & 0x7FFF7FFFu);
                    m = max(m & 0xFFFFu, m >> 16);
                    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                    const uint32_t ex = m >> 7;  // exponent field of the largest magnitude
                    const bool finite = ex < 255;
                    const uint32_t low = max(ex, 15u);
                    const float up = finite ? __uint_as_float((268u - low) << 23) : 1.0f;
                    back[b] = finite ? __uint_as_float((low - 14u) << 23) : 1.0f;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const __half2 h = __floats2half2_rn(bf16_lo(xf[b][j]) * up, bf16_hi(xf[b][j]) * up);
                        xf[b][j] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                }
                float part[4][NT][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int b = 0; b < NT; ++b)
#pragma unroll
                        for (int j = 0; j < 4; ++j) part[i][b][j] = 0.0f;
                    uint32_t s[2][2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t w = i == 0 ? sc[h].x : i == 1 ? sc[h].y : i == 2 ? sc[h].z : sc[h].w;
                        scale_pair(w >> (16 * (t & 1)), s[h][0], s[h][1]);
                    }
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t p[2][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4& cw = code[i][h];
                            e2m1x8_f16(w == 0 ? cw.x : w == 1 ? cw.y : w == 2 ? cw.z : cw.w, p[h]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) p[h][j] = mul_f16x2(p[h][j], s[h][w >> 1]);
                        }
#pragma unroll
                        for (int b = 0; b < NT; ++b) {
                            mma_16816(part[i][b], p[0][0], p[1][0], p[0][1], p[1][1], xf[b][4 * w], xf[b][4 * w + 1]);
                            mma_16816(part[i][b], p[0][2], p[1][2], p[0][3], p[1][3], xf[b][4 * w + 2],
                                      xf[b][4 * w + 3]);
                        }
                    }
                }
                // columns 2 t and 2 t + 1 of a sum are tokens 8 b + 2 t, 8 b + 2 t + 1
#pragma unroll
                for (int b = 0; b < NT; ++b) {
                    const float even = __shfl_sync(0xffffffffu, back[b], 8 * t);
                    const float odd = __shfl_sync(0xffffffffu, back[b], 8 * t + 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[i][b][j] = fmaf(part[i][b][j], (j & 1) ? odd : even, acc[i][b][j]);
                }
            }
            // the warps' sums, in warp order
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int b = 0; b < NT; ++b)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s_red[(warp * 8 * NT + 8 * b + 2 * t + (j & 1)) * kTokStride + 16 * i + r + 8 * (j >> 1)] =
                            acc[i][b][j];
            __syncthreads();
            for (int o = threadIdx.x; o < toks * kUnitRows; o += kGemvThreads) {
                const int tok = o / kUnitRows, row = o % kUnitRows;
                const int64_t n = n0 + 32 * (row >> 4) + (row & 15);
                if (n >= a.n) continue;
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < kGemvWarps; ++w) v += s_red[(w * 8 * NT + tok) * kTokStride + row];
                v *= gs;
                const int64_t at = (row0 + tok) * a.ldd + n;
                if (F32)
                    static_cast<float*>(a.out)[at] = v;
                else
                    static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
            }
            __syncthreads();
        }
    }
}

nvfp4_status launch_gemv(const GemvArgs& in, int out_dtype, void* workspace, size_t ws_bytes, void* stream)
{
    GemvArgs a = in;
    if (!a.q || !a.sf || !a.g) return NVFP4_ERR_INVALID_ARG;
    if (out_dtype != NVFP4_OUT_F32 && out_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_INVALID_ARG;
    if (a.rows < 0 || a.rows > 0x7fffffffll || a.n <= 0 || a.n % 16 || a.n > (1ll << 30) || a.k <= 0 || a.k % 64 ||
        a.k > (1ll << 30) || a.ldx < a.k || a.ldd < a.n)
        return NVFP4_ERR_SHAPE;
    if (a.rows > 0 && (!a.x || !a.out || a.src_rows <= 0)) return NVFP4_ERR_INVALID_ARG;
    if (off16(a.x) || a.ldx % 8 || off16(a.q) || off16(a.sf) || (reinterpret_cast<uintptr_t>(a.g) & 3u) ||
        (reinterpret_cast<uintptr_t>(a.out) & (out_dtype == NVFP4_OUT_F32 ? 3u : 1u)) ||
        (reinterpret_cast<uintptr_t>(a.row_index) & 3u) || (reinterpret_cast<uintptr_t>(a.group_offsets) & 3u))
        return NVFP4_ERR_ALIGN;
    if (workspace && (ws_bytes < 16 || off16(workspace))) return NVFP4_ERR_WORKSPACE;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
    const int sms = sm100_sms(dev);
    if (!sms) return NVFP4_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    a.status = workspace ? static_cast<uint32_t*>(workspace) + 2 : nullptr;
    if (a.status && cudaMemsetAsync(a.status, 0, 4, st) != cudaSuccess) return NVFP4_ERR_CUDA;
    if (a.rows == 0) return NVFP4_OK;
    a.sf_bytes = static_cast<int64_t>(nvfp4_sf_mma_bytes(a.n, a.k));
    const int64_t tiles = (a.n + 127) / 128 * 2;
    // two 8-token columns once a matrix is expected to meet more than 8 rows
    const bool two = a.rows > 8 * static_cast<int64_t>(a.groups);
    const int64_t units = tiles * std::min<int64_t>(a.groups, a.rows);
    const int grid = static_cast<int>(std::min<int64_t>(units, static_cast<int64_t>(sms) * (two ? 1 : 2)));
    const size_t smem = sizeof(float) * kGemvWarps * (two ? 16 : 8) * kTokStride;
    const auto go = [&](auto kernel) { kernel<<<grid, kGemvThreads, smem, st>>>(a); };
    if (out_dtype == NVFP4_OUT_F32)
        two ? go(gemv_kernel<2, true>) : go(gemv_kernel<1, true>);
    else
        two ? go(gemv_kernel<2, false>) : go(gemv_kernel<1, false>);
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_gemv(const void* x_bf16, int64_t ldx, int64_t rows, const uint8_t* q,
                                   const uint8_t* sf, const float* g, int64_t N, int64_t K, int out_dtype, void* D,
                                   int64_t ldd, void* stream)
{
    GemvArgs a{};
    a.x = static_cast<const uint16_t*>(x_bf16), a.ldx = ldx, a.rows = rows, a.src_rows = rows;
    a.groups = 1;
    a.q = q, a.sf = sf, a.g = g, a.n = N, a.k = K, a.out = D, a.ldd = ldd;
    return launch_gemv(a, out_dtype, nullptr, 0, stream);
}

extern "C" nvfp4_status nvfp4_grouped_gemv(int G, const int32_t* group_offsets, int64_t total_rows,
                                           const void* x_bf16, int64_t ldx, int64_t src_rows,
                                           const int32_t* row_index, const uint8_t* q, const uint8_t* sf,
                                           const float* g, int64_t N, int64_t K, int out_dtype, void* D, int64_t ldd,
                                           void* workspace, size_t ws_bytes, void* stream)
{
    if (G < 1 || G > kMaxGemvGroups || !group_offsets) return NVFP4_ERR_INVALID_ARG;
    if (N % 128) return NVFP4_ERR_SHAPE;
    if (!row_index && src_rows < total_rows) return NVFP4_ERR_SHAPE;
    GemvArgs a{};
    a.x = static_cast<const uint16_t*>(x_bf16), a.ldx = ldx, a.src_rows = src_rows, a.row_index = row_index;
    a.group_offsets = group_offsets, a.groups = G, a.rows = total_rows;
    a.q = q, a.sf = sf, a.g = g, a.n = N, a.k = K, a.out = D, a.ldd = ldd;
    return launch_gemv(a, out_dtype, workspace, ws_bytes, stream);
}
