// combine.cu -- the weighted sum of a token's expert rows, and its gradients.
//
//   out[t] = base[t] + sum_j weight[t][j] * rows[slot_row[t][j]]
//   drows[slot_row[t][j]] = weight[t][j] * dout[t]
//   dweight[t][j] = <dout[t], rows[slot_row[t][j]]>        (dbase = dout)
//
// FP32 sums in slot order, one rounding to bf16 at the end; slots with a
// negative row are left out.  All three are one pass over the data.
#include "common.cuh"

#include <algorithm>

namespace nvfp4 {
namespace {

template <bool F32>
struct RowVec;  // eight elements of a row
template <>
struct RowVec<false> {
    uint4 v;
    __device__ __forceinline__ void load(const void* rows, int64_t vec) { v = static_cast<const uint4*>(rows)[vec]; }
    __device__ __forceinline__ void get(float (&f)[8]) const { unpack8(v, f); }
    static __device__ __forceinline__ void store(void* rows, int64_t vec, const float (&f)[8])
    {
        static_cast<uint4*>(rows)[vec] = pack8(f);
    }
};
template <>
struct RowVec<true> {
    float4 a, b;
    __device__ __forceinline__ void load(const void* rows, int64_t vec)
    {
        a = static_cast<const float4*>(rows)[2 * vec];
        b = static_cast<const float4*>(rows)[2 * vec + 1];
    }
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    static __device__ __forceinline__ void store(void* rows, int64_t vec, const float (&f)[8])
    {
        static_cast<float4*>(rows)[2 * vec] = make_float4(f[0], f[1], f[2], f[3]);
        static_cast<float4*>(rows)[2 * vec + 1] = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// A slot's row, -1 for none; an index past the rows is reported and left out.
__device__ __forceinline__ int32_t slot_of(const int32_t* slot_row, int64_t slot, int64_t n_rows, uint32_t* status)
{
    const int32_t r = slot_row[slot];
    if (r >= n_rows) {
        record_status(status, NVFP4_ERR_INDEX);
        return -1;
    }
    return r < 0 ? -1 : r;
}

// One thread = 8 columns of a token; four slots' loads in flight.
//
// What bounds it: HBM.  16384 tokens x 4096 of four bf16 rows each (671 MB): 112 us,
// 6.0 TB/s; eight tokens of FP32 rows: 2.5 us.
template <bool F32>
__global__ void __launch_bounds__(256) combine_kernel(const void* rows, int64_t n_rows, int64_t nvec,
                                                      const int32_t* slot_row, const float* weight, int64_t tokens,
                                                      int k, const uint4* base, uint4* out, uint32_t* status)
{
    wait_for_previous_kernel();
    let_next_kernel_start();
    for (int64_t u = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; u < tokens * nvec;
         u += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t t = u / nvec, c = u - t * nvec;
        float acc[8];
        if (base) {
            unpack8(base[u], acc);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
        }
        for (int j0 = 0; j0 < k; j0 += 4) {
            int32_t r[4];
            RowVec<F32> v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                r[j] = j0 + j < k ? slot_of(slot_row, t * k + j0 + j, n_rows, status) : -1;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (r[j] >= 0) v[j].load(rows, r[j] * nvec + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (r[j] < 0) continue;
                const float w = weight[t * k + j0 + j];
                float f[8];
                v[j].get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, f[i], acc[i]);
            }
        }
        out[u] = pack8(acc);
    }
}

// With used_rows every row of drows is defined: those that no slot names are zeroed
// before the gradients are written.  Which rows slots name needs no memory of its
// own: mark_rows_kernel leaves each slot's number at a place of the row it names, and
// a row is named if the number found at its place is that of a slot with this row,
// whatever bytes lay there before.  The places are dweight's, which is written later,
// and for rows past its end (all rows where dweight is weight itself) the first bytes
// of the rows.  (Marks in the rows alone
// take 4.5 us more at 65536 rows of 8 KB, whose pages and sectors are all touched.)
struct Marks {
    int32_t* place;   // dweight
    int64_t places;
    uint8_t* rows;    // drows
    int64_t row_bytes;
    __device__ __forceinline__ int32_t* of(int64_t r) const
    {
        return r < places ? place + r : reinterpret_cast<int32_t*>(rows + r * row_bytes);
    }
};

__global__ void __launch_bounds__(256) mark_rows_kernel(const int32_t* slot_row, int64_t slots, int64_t n_rows, Marks marks)
{
    wait_for_previous_kernel();
    let_next_kernel_start();
    for (int64_t s = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; s < slots;
         s += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int32_t r = slot_row[s];
        if (r >= 0 && r < n_rows) *marks.of(r) = static_cast<int32_t>(s);
    }
}

// A warp looks at `per` rows at a time, a lane at each, and zeroes those of them that
// no slot names (from *used_rows on none does).  The gradients' kernel is not let in
// before the end: its CTAs would crowd where room comes first (16384 tokens x 256,
// top-4: 36 us in all against 23).
//
// The marks and this cost 4.5 us at 65536 rows, two launches: 184.1 -> 188.9 us with
// the gradients at 4096 columns, 19 -> 23 us at 256, 3.2 -> 5.7 us at 256 rows.
__global__ void __launch_bounds__(256) zero_unnamed_rows_kernel(const int32_t* slot_row, int64_t slots, int64_t n_rows,
                                                                const int32_t* used_rows, int per, Marks marks)
{
    const int lane = threadIdx.x & 31;
    const int64_t warp = blockIdx.x * static_cast<int64_t>(blockDim.x >> 5) + (threadIdx.x >> 5);
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    wait_for_previous_kernel();
    const int64_t used = *used_rows;
    for (int64_t r0 = warp * per; r0 < n_rows; r0 += warps * per) {
        const int64_t r = r0 + lane;
        bool unnamed = lane < per && r < n_rows;
        if (unnamed && r < used) {
            const int32_t s = *marks.of(r);
            unnamed = !(s >= 0 && s < slots && slot_row[s] == r);
        }
        for (unsigned left = __ballot_sync(0xffffffffu, unnamed); left; left &= left - 1) {
            uint4* const row = reinterpret_cast<uint4*>(marks.rows + (r0 + __ffs(left) - 1) * marks.row_bytes);
            for (int64_t v = lane; v < marks.row_bytes / 16; v += 32) row[v] = make_uint4(0, 0, 0, 0);
        }
    }
}

// What bounds it: HBM at wide rows; the gradients of the same tokens read dout and the
// rows and write the rows' gradients once (1.21 GB): 184 us, 6.6 TB/s.  At narrow ones
// (one warp a token, eight an SM) it is a token's chain of slots, rows, sums and
// barriers: 19 us at 256 columns, 75 MB.
//
// One CTA of W warps per token; each thread keeps the products' sums of four
// slots over its columns (bf16 rows within 64 registers: left to itself the compiler
// took 59, and 1 us more).  With `seen` (one bit a row, cleared by the call) a slot
// whose row an earlier one has named is reported and left out: the row's gradient
// would be a sum that two slots write.
template <bool F32>
__global__ void __launch_bounds__(256, F32 ? 1 : 4) combine_backward_kernel(
    const uint4* dout, const void* rows, int64_t n_rows, int nvec, const int32_t* slot_row, const float* weight,
    int64_t tokens, int k, void* drows, float* dweight, uint32_t* seen, uint32_t* status)
{
    __shared__ float s_dot[4][8];
    __shared__ int32_t s_row[4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    wait_for_previous_kernel();
    let_next_kernel_start();
    for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
        for (int j0 = 0; j0 < k; j0 += 4) {
            __syncthreads();
            if (threadIdx.x < 4) {
                const int j = threadIdx.x;
                int32_t r = j0 + j < k ? slot_of(slot_row, t * k + j0 + j, n_rows, status) : -1;
                if (r >= 0 && seen && (atomicOr(&seen[r >> 5], 1u << (r & 31)) >> (r & 31)) & 1u) {
                    record_status(status, NVFP4_ERR_INDEX);
                    r = -1;
                }
                s_row[j] = r;
            }
            __syncthreads();
            int32_t r[4];
            float w[4], dot[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r[j] = s_row[j];
                w[j] = r[j] >= 0 ? weight[t * k + j0 + j] : 0.0f;
                dot[j] = 0.0f;
            }
            for (int c = threadIdx.x; c < nvec; c += blockDim.x) {
                RowVec<F32> v[4];
                const uint4 dv = dout[t * nvec + c];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r[j] >= 0) v[j].load(rows, static_cast<int64_t>(r[j]) * nvec + c);
                float d[8];
                unpack8(dv, d);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (r[j] < 0) continue;
                    float f[8];
                    v[j].get(f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dot[j] = fmaf(d[i], f[i], dot[j]);
                        f[i] = w[j] * d[i];
                    }
                    RowVec<F32>::store(drows, static_cast<int64_t>(r[j]) * nvec + c, f);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int d = 16; d; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
                if (lane == 0) s_dot[j][warp] = dot[j];
            }
            __syncthreads();
            if (threadIdx.x < 4 && j0 + threadIdx.x < k) {
                float sum = 0.0f;
                for (int i = 0; i < warps; ++i) sum += s_dot[threadIdx.x][i];
                dweight[t * k + j0 + threadIdx.x] = sum;
            }
        }
    }
}

constexpr size_t kCombineWorkspaceHead = 256;

nvfp4_status combine_common(const void* rows, int rows_dtype, int64_t n_rows, int64_t cols, const int32_t* slot_row,
                            const float* weight, int64_t tokens, int k)
{
    if (rows_dtype != NVFP4_OUT_F32 && rows_dtype != NVFP4_OUT_BF16) return NVFP4_ERR_INVALID_ARG;
    if (k < 1 || k > 64) return NVFP4_ERR_INVALID_ARG;
    if (n_rows < 0 || n_rows > 0x7fffffffll || tokens < 0 || cols <= 0 || cols % 8 || cols > (1ll << 30))
        return NVFP4_ERR_SHAPE;
    if ((n_rows > 0 && !rows) || (tokens > 0 && (!slot_row || !weight))) return NVFP4_ERR_INVALID_ARG;
    if (off16(rows) || (reinterpret_cast<uintptr_t>(slot_row) & 3u) || (reinterpret_cast<uintptr_t>(weight) & 3u))
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

// Two arrays of as many bytes share some.
bool overlap(const void* a, const void* b, int64_t bytes)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return (x < y ? y - x : x - y) < static_cast<uint64_t>(bytes);
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_combine(const void* rows, int rows_dtype, int64_t n_rows, int64_t cols,
                                      const int32_t* slot_row, const float* weight, int64_t tokens, int k,
                                      const void* base_bf16, void* out_bf16, void* workspace, size_t ws_bytes,
                                      void* stream)
{
    if (const nvfp4_status s = combine_common(rows, rows_dtype, n_rows, cols, slot_row, weight, tokens, k)) return s;
    if (tokens > 0 && !out_bf16) return NVFP4_ERR_INVALID_ARG;
    if (off16(base_bf16) || off16(out_bf16)) return NVFP4_ERR_ALIGN;
    if (workspace && (ws_bytes < 16 || off16(workspace))) return NVFP4_ERR_WORKSPACE;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
    const int sms = sm100_sms(dev);
    if (!sms) return NVFP4_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint32_t* status = workspace ? static_cast<uint32_t*>(workspace) + 2 : nullptr;
    if (status && cudaMemsetAsync(status, 0, 4, st) != cudaSuccess) return NVFP4_ERR_CUDA;
    if (tokens == 0) return NVFP4_OK;
    const int64_t nvec = cols / 8;
    const int grid = static_cast<int>(std::min<int64_t>((tokens * nvec + 255) / 256, static_cast<int64_t>(sms) * 8));
    cudaError_t err = cudaSuccess;
    const auto go = [&](auto kernel) {
        err = launch_early(!status, kernel, grid, 256, 0, st, rows, n_rows, nvec, slot_row, weight, tokens, k,
                           static_cast<const uint4*>(base_bf16), static_cast<uint4*>(out_bf16), status);
    };
    rows_dtype == NVFP4_OUT_F32 ? go(combine_kernel<true>) : go(combine_kernel<false>);
    return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

extern "C" size_t nvfp4_combine_backward_workspace_size(int64_t n_rows)
{
    return kCombineWorkspaceHead + (n_rows > 0 ? static_cast<size_t>((n_rows + 31) / 32) * 4 : 0);
}

extern "C" nvfp4_status nvfp4_combine_backward(const void* dout_bf16, const void* rows, int rows_dtype,
                                               int64_t n_rows, int64_t cols, const int32_t* slot_row,
                                               const float* weight, int64_t tokens, int k, const int32_t* used_rows,
                                               void* drows, float* dweight, void* workspace, size_t ws_bytes,
                                               void* stream)
{
    if (const nvfp4_status s = combine_common(rows, rows_dtype, n_rows, cols, slot_row, weight, tokens, k)) return s;
    if ((tokens > 0 && (!dout_bf16 || !dweight)) || (n_rows > 0 && !drows)) return NVFP4_ERR_INVALID_ARG;
    if (off16(dout_bf16) || off16(drows) || (reinterpret_cast<uintptr_t>(dweight) & 3u) ||
        (reinterpret_cast<uintptr_t>(used_rows) & 3u))
        return NVFP4_ERR_ALIGN;
    if (workspace && (off16(workspace) || ws_bytes < nvfp4_combine_backward_workspace_size(n_rows)))
        return NVFP4_ERR_WORKSPACE;
    const int64_t row_bytes = cols * (rows_dtype == NVFP4_OUT_F32 ? 4 : 2);
    if (used_rows && tokens > 0x7fffffffll / k) return NVFP4_ERR_SHAPE;  // a mark is a slot's number
    // marks go where nothing is still to be read: not over weights, and not over rows
    const int64_t places = used_rows && !overlap(weight, dweight, tokens * k * 4) ? tokens * k : 0;
    if (used_rows && n_rows > places && overlap(rows, drows, n_rows * row_bytes)) return NVFP4_ERR_INVALID_ARG;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
    const int sms = sm100_sms(dev);
    if (!sms) return NVFP4_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (workspace && cudaMemsetAsync(workspace, 0, nvfp4_combine_backward_workspace_size(n_rows), st) != cudaSuccess)
        return NVFP4_ERR_CUDA;
    cudaError_t err = cudaSuccess;
    bool early = !workspace;
    if (used_rows && n_rows > 0) {
        const int64_t slots = tokens * k;
        const Marks marks{reinterpret_cast<int32_t*>(dweight), places, static_cast<uint8_t*>(drows), row_bytes};
        const auto ctas = [&](int64_t threads) {
            return std::min<int64_t>((threads + 255) / 256, static_cast<int64_t>(sms) * 8);
        };
        if (slots > 0) {
            err = launch_early(early, mark_rows_kernel, ctas(slots), 256, 0, st, slot_row, slots, n_rows, marks);
            early = true;
        }
        const int64_t grid = ctas(n_rows * 32);
        const int per = static_cast<int>(std::min<int64_t>((n_rows + grid * 8 - 1) / (grid * 8), 32));
        if (err == cudaSuccess)
            err = launch_early(early, zero_unnamed_rows_kernel, grid, 256, 0, st, slot_row, slots, n_rows, used_rows, per,
                               marks);
        early = true;
        if (err != cudaSuccess) return NVFP4_ERR_CUDA;
    }
    if (tokens == 0) return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
    const int nvec = static_cast<int>(cols / 8);
    const int threads = std::min(256, std::max(1, (nvec + 31) / 32) * 32);
    const int grid = static_cast<int>(std::min<int64_t>(tokens, static_cast<int64_t>(sms) * 8));
    uint32_t* const status = workspace ? static_cast<uint32_t*>(workspace) + 2 : nullptr;
    uint32_t* const seen =
        workspace ? reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + kCombineWorkspaceHead) : nullptr;
    const auto go = [&](auto kernel) {
        err = launch_early(early, kernel, grid, threads, 0, st, static_cast<const uint4*>(dout_bf16), rows, n_rows, nvec,
                           slot_row, weight, tokens, k, drows, dweight, seen, status);
    };
    rows_dtype == NVFP4_OUT_F32 ? go(combine_backward_kernel<true>) : go(combine_backward_kernel<false>);
    return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
