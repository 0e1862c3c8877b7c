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
//  - x is brought into FP16's range by a power of two per row, its largest
//    magnitude to [2^14, 2^15): exact for values down to 2^-32 of that largest one,
//    and off by at most 2^-40 of it below;
//  - products and their sums are FP32; the tensor cores' sums of 256 columns are
//    added in FP32, and the total is scaled back.
//
// What bounds it.  Bytes, with what comes before the first of them: a plain read of
// as many bytes takes 12.1 us (59 MB) and 20.6 us (133 MB) a launch here.  One row x
// 20480 x 5120 (59 MB) 16.0 us; 32 tokens' rows through four experts of 4096 x 1536
// each (133 MB) 36 us; eight tokens' through 1536 x 4096 (60 MB)
// 21.6 us, of which 3 us pass before the routing has been read and the first weights
// are asked for.  At more rows it is bringing x into each SM's shared memory, a row
// about as dear as a 16-row tile: 13 rows x 4096 x 4096 11 us, 32 rows x 5120 x 20480
// 75 us.  Steps on the way, at the one row: warps of 64 matrix
// rows loading into registers 24.9 us; a copy ring and 16-row tiles in equal runs
// 18.1 us; the first weights asked for behind x instead of before it, and no group
// scan for a single matrix, 15.7 us.  Decoding by shifts and masks into bf16 (15
// integer operations per eight codes against four conversions) ran at 37 codes a
// clock and SM with the matrix instructions, below the 41 that HBM delivers; the
// conversions run at 65.  Asking for a CTA's later tiles ahead by bulk prefetches
// into L2 was slower (one row: 16.9 to 19.4 us): x waits behind them.
#include "common.cuh"
#include "gemv_plan.h"

#include <algorithm>

namespace nvfp4 {
namespace {

constexpr int kGemvWarps = 16;
constexpr int kStep = 256;               // columns of a step, 64 per lane
constexpr int kStageBytes = 2048 + 256;  // a 16-row tile's codes and scales
constexpr int kRedStride = 20;           // floats per token of a tile's sums (16 rows, off the banks)
constexpr int kMaxGemvGroups = 256;
constexpr int kMaxSegments = 16;         // segments whose x rows are in shared memory together
constexpr size_t kGemvSmem = 216 * 1024;  // dynamic; 11.2 KB more are not, of 227 KB in all

// Steps in a warp's ring, all but one copied ahead.
__host__ __device__ constexpr int ring_stages(int nt) { return nt == 1 ? 3 : 2; }

// Bytes of the rings and of the tiles' sums that warps hand on.
__host__ __device__ constexpr size_t gemv_fixed(int nt)
{
    return kGemvWarps * (ring_stages(nt) * kStageBytes + 2 * sizeof(float) * 8 * nt * kRedStride);
}

// Tiles whose sums over several panels a CTA keeps, and the bytes of one.
constexpr int kPanelTiles = 24;
__host__ __device__ constexpr size_t tile_sum_bytes(int nt) { return sizeof(float) * 16 * 8 * nt; }

// Most (x row, step) pairs in shared memory, 512 bytes each.
__host__ __device__ constexpr int max_x_pairs(int nt, bool panels)
{
    return static_cast<int>((kGemvSmem - gemv_fixed(nt) - (panels ? kPanelTiles * tile_sum_bytes(nt) : 0)) / 512);
}

// Division of 0 <= n < 2^31 by a number known on the host.  With 2^s >= d and
// m = floor(2^(31 + s) / d) + 1, n m / 2^(31 + s) exceeds n / d by at most
// n / 2^(31 + s) < 2^-s <= 1 / d, too little to reach the next whole number.
struct Divisor {
    uint32_t m = 0;
    int shift = 0, d = 1;
    Divisor() = default;
    explicit Divisor(int by) : d(by)
    {
        int s = 0;
        while ((1ll << s) < by) ++s;
        m = static_cast<uint32_t>((1ull << (31 + s)) / static_cast<uint64_t>(by) + 1);
        shift = 31 + s;
    }
    __device__ __forceinline__ int operator()(int n) const
    {
        return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(n)) * m >> shift);
    }
};

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
    int tiles, steps;              // 16-row tiles of a matrix, 256-column steps of a row
    int seg_rows;                  // most x rows of a segment
    int whole;                     // no tile or step reaches past the matrix
    int x_rows;                    // x rows that shared memory holds
    int panel_steps;               // steps of x in shared memory at a time: all, or a panel of them
    Divisor by_tiles, by_steps, by_seg_rows;
    Divisor by_grid;               // CTAs; of one matrix those of a segment
    int each, more;                // one matrix's tiles over them: each, and one more for the first CTAs
    void* out;
    int out_f32;
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

// The E4M3 scales of four 16-blocks, each in both halves of a register.
__device__ __forceinline__ void four_scales(uint32_t word, uint32_t (&s)[4])
{
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(word));
    s[0] = __byte_perm(lo, 0, 0x1010);
    s[1] = __byte_perm(lo, 0, 0x3232);
    s[2] = __byte_perm(hi, 0, 0x1010);
    s[3] = __byte_perm(hi, 0, 0x3232);
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The exponent field by which a row of x is scaled, from its largest magnitude (bf16
// bits).  With an infinity or a NaN in the row it is that of the largest finite
// numbers: they, too, then fit into FP16, and a sum is infinite or NaN by those alone.
__device__ __forceinline__ uint32_t x_exponent(uint32_t top) { return min(max(top >> 7, 15u), 254u); }

// Asynchronous copies to shared memory; zeros where there is nothing to read.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 load_shared(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

// Work is cut into 16-row weight tiles; tile 8 b + u of a matrix is rows
// 128 b + 32 i + 4 u + 0..3 (i < 4), whose scales of 64 columns lie together.  A
// segment is a matrix with up to seg_rows of its x rows; all segments have the
// same number of tiles, and the CTAs take equal runs of the list of all (segment,
// tile) pairs.  A CTA brings the x rows of the segments it works on into shared
// memory as FP16, in the order in which lanes read them; its warps take equal
// runs of the tiles' 256-column steps.  A tile that lies inside one warp's run is
// stored by that warp; of a tile that several runs share, the warp with its first
// step adds the sums in warp order.
//
// Lane (r, t) = (lane / 4, lane % 4) works on rows r and r + 8 of a tile (row m is
// i = m / 4, row m % 4 of its four) and, of each step, on the 64 columns from 64 t
// on: two 16-byte vectors of codes and four scale bytes a row.  The columns' order
// inside a matrix instruction does not matter as long as both operands agree, so
// a code word's pairs go in as they lie.  Each warp copies its steps into a ring
// of its own, some steps ahead and into the next tile too, in whole 64-byte runs
// of a row, and waits for no other warp.
//
// With PANELS (one matrix), x comes in panels of columns: the CTA goes over at most
// kPanelTiles tiles panel by panel and keeps their sums in shared memory.
template <int NT, bool PANELS>
__global__ void __launch_bounds__(32 * kGemvWarps, 1) gemv_kernel(const GemvArgs a)
{
    constexpr int kStages = ring_stages(NT);
    constexpr int kRed = 8 * NT * kRedStride;  // floats of a tile's sums
    extern __shared__ __align__(16) uint8_t s_dyn[];
    __shared__ int s_first[kMaxGemvGroups], s_rows[kMaxGemvGroups], s_end[kMaxGemvGroups];
    __shared__ int16_t s_group[kMaxGemvGroups];
    __shared__ int2 s_count[kGemvWarps];
    __shared__ int s_seg_e[kMaxSegments], s_seg_row[kMaxSegments], s_seg_n[kMaxSegments], s_seg_x[kMaxSegments + 1];
    __shared__ int s_run[4];  // this CTA's tiles [0, 1) of the list, segments in shared memory, tile of the first one
    __shared__ uint4 s_zero[4];
    // of each x row in shared memory: its row of x (-1 for a bad index), its place in
    // s_x, the bytes from one of its pieces to the next, its matrix; its largest magnitude
    // (bf16 bits)
    __shared__ int4 s_x_row[kMaxSegments * 8 * NT];
    __shared__ uint32_t s_top[kMaxSegments * 8 * NT];
    __shared__ float2 s_scale[kMaxSegments * 8 * NT];  // the factors on its sums: the matrix's g, its own power of two
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, t = lane & 3;
    const int tiles = a.tiles, steps = a.steps;
    uint8_t* const my_ring = s_dyn + warp * kStages * kStageBytes;
    const uint32_t ring = smem_addr(my_ring);
    float* const s_sums = reinterpret_cast<float*>(s_dyn + kGemvWarps * kStages * kStageBytes);  // [2][warps][kRed]
    float* const my_head = s_sums + warp * kRed;                        // sums of a tile that an earlier warp began
    float* const my_sums = s_sums + (kGemvWarps + warp) * kRed;         // sums of a tile that this one began
    float* const s_acc = s_sums + 2 * kGemvWarps * kRed;  // with panels: [kPanelTiles][8 NT][16]
    uint8_t* const s_x = reinterpret_cast<uint8_t*>(s_acc) + (PANELS ? kPanelTiles * tile_sum_bytes(NT) : 0);
    const int panel_steps = PANELS ? a.panel_steps : steps;

    wait_for_previous_kernel();
    let_next_kernel_start();
    int active = 0;  // groups that have rows
    const bool one = !a.group_offsets;  // one matrix: a CTA has tiles of one segment
    if (one) {
        const int part = a.by_grid(blockIdx.x), b = blockIdx.x - part * a.by_grid.d, first = part * a.seg_rows;
        const int rows = min(a.seg_rows, static_cast<int>(a.rows) - first), xr = threadIdx.x;
        if (xr < rows) {
            s_x_row[xr] = make_int4(first + xr, xr * 64, rows * 64, 0);
            s_top[xr] = 0;
        }
        if (xr < 4) s_zero[xr] = make_uint4(0, 0, 0, 0);
        if (xr == 0) {
            s_run[0] = s_run[3] = b * a.each + min(b, a.more);
            s_run[1] = s_run[0] + a.each + (b < a.more ? 1 : 0);
            s_run[2] = 1;
            s_seg_e[0] = s_seg_x[0] = 0;
            s_seg_row[0] = first;
            s_seg_n[0] = s_seg_x[1] = rows;
        }
    } else {
        // those groups in order, with the segments up to and with each: thread e looks
        // at group e, its warp counts, and the warps' counts are added up
        static_assert(kMaxGemvGroups <= 32 * kGemvWarps, "a thread for each group");
        const int rows = static_cast<int>(a.rows), e = threadIdx.x;
        int lo = 0, hi = 0;
        if (e < a.groups) lo = a.group_offsets[e], hi = a.group_offsets[e + 1];
        const int first = min(max(lo, 0), rows), count = min(hi, rows) - first;
        const unsigned has = __ballot_sync(0xffffffffu, count > 0);
        int upto = count > 0 ? a.by_seg_rows(count - 1) + 1 : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += v;
        }
        if (lane == 31) s_count[warp] = make_int2(upto, __popc(has));
        if (e < 4) s_zero[e] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        int at = __popc(has & ((1u << lane) - 1)), all = 0;
#pragma unroll
        for (int w = 0; w < kMaxGemvGroups / 32; ++w) {
            const int2 n = s_count[w];
            if (w < warp) upto += n.x, at += n.y;
            all += n.x, active += n.y;
        }
        if (count > 0) {
            s_group[at] = static_cast<int16_t>(e);
            s_first[at] = first;
            s_rows[at] = count;
            s_end[at] = upto;
        }
        if (e == 0) {
            all *= tiles;
            const int b = blockIdx.x, each = a.by_grid(all), more = all - each * static_cast<int>(gridDim.x);
            s_run[0] = b * each + min(b, more);
            s_run[1] = s_run[0] + each + (b < more ? 1 : 0);
        }
        __syncthreads();
    }
#pragma unroll 1
    for (int f0 = -1;;) {
        if (warp == 0 && !one) {
            if (f0 < 0) f0 = s_run[0];
            const int f1 = s_run[1];
            // the segments from f0's on whose rows fit
            const int seg0 = a.by_tiles(f0), want = f1 > f0 ? a.by_tiles(f1 - 1) - seg0 + 1 : 0;
            int e = 0, row = 0, n = 0;
            if (lane < min(want, kMaxSegments)) {
                int g = 0;
#pragma unroll 1
                for (int step = 128; step; step >>= 1)  // groups whose segments all lie before
                    if (g + step <= active && s_end[g + step - 1] <= seg0 + lane) g += step;
                const int part = seg0 + lane - (g ? s_end[g - 1] : 0);
                e = s_group[g];
                row = s_first[g] + part * a.seg_rows;
                n = min(a.seg_rows, s_rows[g] - part * a.seg_rows);
            }
            int upto = n;
#pragma unroll 1
            for (int d = 1; d < kMaxSegments; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, d);
                if (lane >= d) upto += v;
            }
            const int fit = __popc(__ballot_sync(0xffffffffu, n > 0 && upto <= a.x_rows));
            if (lane < kMaxSegments) {
                s_seg_e[lane] = e, s_seg_row[lane] = row, s_seg_n[lane] = n;
                s_seg_x[lane + 1] = upto;
            }
            if (lane == 0) s_run[2] = fit, s_run[3] = f0 - seg0 * tiles, s_seg_x[0] = 0;
            __syncwarp();
#pragma unroll 1
            for (int xr = lane; xr < s_seg_x[fit]; xr += 32) {
                int s = 0;
                while (s_seg_x[s + 1] <= xr) ++s;
                int src = s_seg_row[s] + xr - s_seg_x[s];
                if (a.row_index) {
                    src = a.row_index[src];
                    if (src < 0 || src >= a.src_rows) {
                        record_status(a.status, NVFP4_ERR_INDEX);
                        src = -1;
                    }
                }
                const int x0 = s_seg_x[s];
                s_x_row[xr] = make_int4(src, x0 * steps * 512 + (xr - x0) * 64, s_seg_n[s] * 64, s_seg_e[s]);
                s_top[xr] = 0;
            }
        }
        __syncthreads();
        if (f0 < 0) f0 = s_run[0];
        // (with PANELS `one` holds; without the test here the loop over the steps came out a
        // sixth slower: 32 rows x 5120 x 20480 87 us against 75)
        const int segs = s_run[2], f1 = s_run[1], tile0 = PANELS && one ? f0 : s_run[3];
        if (f0 >= f1) return;
        const int fe = min(min(f1, f0 - tile0 + segs * tiles), PANELS ? f0 + kPanelTiles : f1);

#pragma unroll 1
        for (int p0 = 0;;) {
        const int psteps = PANELS ? min(panel_steps, steps - p0) : steps;
        // this warp's run of steps: items [j0, j1) of the (fe - f0) tiles' steps
        const int items = (fe - f0) * psteps;
        const auto run_start = [&](int w) { return (items / kGemvWarps) * w + min(w, items % kGemvWarps); };
        const int j0 = run_start(warp), j1 = run_start(warp + 1);
        const int skip = psteps == panel_steps ? a.by_steps(j0) : j0 / psteps, first_step = j0 - skip * psteps;
        int seg = 0, tile = tile0 + skip;
        while (tile >= tiles) tile -= tiles, ++seg;

        // A row's 128 bytes of a step are eight vectors; vector v of row r lies at
        // place v ^ (r & 1), so that lanes reading vectors 2 t or 2 t + 1 of two rows
        // meet eight different ones.
        int left = j1 - j0, pc = first_step, pslot = 0, pseg = seg, ptile = tile;
        bool have0 = true, have8 = true;  // rows r and r + 8 lie in the matrix
        const int64_t row_bytes = a.k / 2;
        const uint8_t *tq = nullptr, *ts = nullptr;                  // this lane's first codes (row r), scales of the tile
        const uint8_t *pq = nullptr, *pq8 = nullptr, *ps = nullptr;  // those of the step
        const auto rows_there = [&]() {
            if (a.whole) return;
            const int64_t n = static_cast<int64_t>(ptile >> 3) * 128 + 32 * (r >> 2) + 4 * (ptile & 7) + (r & 3);
            have0 = n < a.n;
            have8 = n + 64 < a.n;
        };
        const auto aim = [&]() {  // at tile ptile of segment pseg
            const int64_t e = s_seg_e[pseg], block = ptile >> 3;
            const int u = ptile & 7;
            tq = a.q + (e * a.n + block * 128 + 32 * (r >> 2) + 4 * u + (r & 3)) * row_bytes + 16 * t;
            ts = a.sf + e * a.sf_bytes + block * (a.k / 64) * 512 + (lane & 15) / 4 * 512 + (4 * u + (lane & 3)) * 16;
            rows_there();
        };
        const auto at_step = [&]() {
            pq = tq + (p0 + pc) * (kStep / 2);
            pq8 = pq + 64 * row_bytes;  // from row m to row m + 8: i + 2
            ps = ts + static_cast<int64_t>(p0 + pc) * 2048;
        };
        if (left > 0) {
            aim();
            at_step();
        }
        const uint32_t put = ring + r * 128 + (t ^ (r & 1)) * 16, put_sc = ring + 2048 + (lane & 15) * 16;
        const auto copy_step = [&]() {
            if (left > 0) {
                const uint32_t dst = put + pslot * kStageBytes, dst_sc = put_sc + pslot * kStageBytes;
                if (a.whole) {
                    copy16_async(dst, pq);
                    copy16_async(dst + 64, pq + 64);
                    copy16_async(dst + 1024, pq8);
                    copy16_async(dst + 1088, pq8 + 64);
                    if (lane < 16) copy16_async(dst_sc, ps);
                } else {
                    const int k = (p0 + pc) * kStep + 32 * t;
                    const bool in0 = k < a.k, in1 = k + 128 < a.k;
                    copy16_async(dst, in0 && have0 ? pq : a.q, in0 && have0);
                    copy16_async(dst + 64, in1 && have0 ? pq + 64 : a.q, in1 && have0);
                    copy16_async(dst + 1024, in0 && have8 ? pq8 : a.q, in0 && have8);
                    copy16_async(dst + 1088, in1 && have8 ? pq8 + 64 : a.q, in1 && have8);
                    const bool in = (p0 + pc) * kStep + 64 * ((lane & 15) >> 2) < a.k;
                    if (lane < 16) copy16_async(dst_sc, in ? ps : a.sf, in);
                }
                --left;
                pq += kStep / 2;
                pq8 += kStep / 2;
                ps += 2048;
                if (++pc == psteps && left > 0) {
                    pc = 0;
                    if (++ptile == tiles) {
                        ptile = 0, ++pseg;
                        aim();
                    } else {  // four rows on, or the next 128-row block
                        const bool next_block = (ptile & 7) == 0;
                        tq += (next_block ? 100 : 4) * row_bytes;
                        ts += next_block ? (a.k / 64) * 512 - 448 : 64;
                        rows_there();
                    }
                    at_step();
                }
            }
            pslot = pslot + 1 == kStages ? 0 : pslot + 1;
            asm volatile("cp.async.commit_group;" ::: "memory");
        };

        // x rows of the segments as FP16, each at the power of two that brings its
        // largest magnitude to [2^14, 2^15): of segment s (n rows) and a step, [8
        // pieces][n][4 lanes t] vectors of 16 bytes.  A warp takes the (row, step) pairs
        // warp, warp + 16, ... in row order; lane (r, t) brings piece r of the columns
        // that lanes t read, and converts it in place once the largest magnitude is known.
        const int x_rows = s_seg_x[segs];
        float g = 0.0f;  // of the x row that is this thread's index
        if (static_cast<int>(threadIdx.x) < x_rows) g = a.g[s_x_row[threadIdx.x].w];
        const auto next = [&](int& xr, int& c) {
            c += kGemvWarps;
            while (c >= psteps) c -= psteps, ++xr;
        };
        {
            constexpr int kAhead = 4 * NT;  // loads in flight together
            int xr = 0, c = warp - kGemvWarps;
            next(xr, c);
            bool primed = false;
#pragma unroll 1
            do {
                uint4 v[kAhead];
                int at[kAhead], of[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int4 row = s_x_row[min(xr, x_rows - 1)];
                    const int k = (p0 + c) * kStep + 64 * t + 8 * r;
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (xr < x_rows && row.x >= 0 && k < a.k) v[i] = *reinterpret_cast<const uint4*>(a.x + row.x * a.ldx + k);
                    at[i] = row.y + (c * 8 + r) * row.z + t * 16;
                    of[i] = xr;
                    next(xr, c);
                }
                if (!primed) {  // the first weights, behind the first x
#pragma unroll 1
                    for (int s = 0; s < kStages - 1; ++s) copy_step();
                    primed = true;
                }
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    if (of[i] >= x_rows) break;
                    *reinterpret_cast<uint4*>(s_x + at[i]) = v[i];
                    const uint32_t m = __vmaxu2(
                        __vimax3_u16x2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu, v[i].z & 0x7FFF7FFFu), v[i].w & 0x7FFF7FFFu);
                    const uint32_t top = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
                    if (lane == 0) atomicMax(&s_top[of[i]], top);
                }
            } while (xr < x_rows);
        }
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < x_rows) {
            s_scale[threadIdx.x] = make_float2(g, __uint_as_float((x_exponent(s_top[threadIdx.x]) - 14u) << 23));
        }
        {
            int xr = 0, c = warp - kGemvWarps;
            next(xr, c);
#pragma unroll 2
            while (xr < x_rows) {
                const int4 row = s_x_row[xr];
                uint4* const at = reinterpret_cast<uint4*>(s_x + t * 16 + row.y + (c * 8 + r) * row.z);
                const float up = __uint_as_float((268u - x_exponent(s_top[xr])) << 23);
                float f[8];
                unpack8(*at, f);
                __half2 h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mul2(f[2 * j], f[2 * j + 1], f[2 * j], f[2 * j + 1], up, up);
                    h[j] = __floats2half2_rn(f[2 * j], f[2 * j + 1]);
                }
                *at = *reinterpret_cast<const uint4*>(h);
                next(xr, c);
            }
        }
        if (j0 == j1)  // an empty run adds nothing to the tile that goes past it
            for (int i = lane; i < kRed; i += 32) my_head[i] = 0.0f;
        __syncthreads();
        if (PANELS && static_cast<int>(threadIdx.x) < x_rows) s_top[threadIdx.x] = 0;  // for the next panel

        int slot = 0, c = first_step;
        bool begun = first_step == 0, open = false;  // the tile was begun by this warp; its run ends inside it
        float acc[NT][4];
        // of the segment: this lane's x vectors, piece p of step c at x0 + (8 c + p) *
        // xstep; the factors on the sums of tokens 8 b + 2 t + 0, 1, and which are there
        uint32_t x0[NT], xp[NT], xstep[NT];
        float2 factor[NT][2];
        bool there[NT][2];
        int64_t row0 = 0;
        const auto enter = [&]() {
            const int n = s_seg_n[seg], first = s_seg_x[seg];
            row0 = s_seg_row[seg];
#pragma unroll
            for (int b = 0; b < NT; ++b) {
                const bool is = 8 * b + r < n;
                xstep[b] = is ? n * 64 : 0;
                x0[b] = is ? smem_addr(s_x) + first * panel_steps * 512 + (8 * b + r) * 64 + t * 16 : smem_addr(s_zero + t);
                xp[b] = x0[b] + c * 8 * xstep[b];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int tok = 8 * b + 2 * t + i;
                    there[b][i] = tok < n;
                    factor[b][i] = tok < n ? s_scale[first + tok] : make_float2(0.0f, 0.0f);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[b][i] = 0.0f;
            }
        };
        // a sum of token tok to weight row m of the tile (g first: the power of two
        // may leave few bits to a product of both factors)
        const auto store = [&](int tok, int m, float v, float2 by) {
            v = v * by.x * by.y;
            if (PANELS) {
                float* const sum = s_acc + ((tile - tile0) * 8 * NT + tok) * 16 + m;
                if (p0 > 0) v += *sum;
                if (p0 + psteps < steps) {
                    *sum = v;
                    return;
                }
            }
            const int64_t n = static_cast<int64_t>(tile >> 3) * 128 + 4 * (tile & 7) + 32 * (m >> 2) + (m & 3);
            if (n >= a.n) return;
            const int64_t at = (row0 + tok) * a.ldd + n;
            if (a.out_f32)
                static_cast<float*>(a.out)[at] = v;
            else
                static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
        };
        if (j0 < j1) enter();
#pragma unroll 1
        for (int j = j0; j < j1; ++j) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            __syncwarp();  // this step has come for every lane, and every lane is done with the last one
            copy_step();
            const uint8_t* const stage = my_ring + slot * kStageBytes;
            slot = slot + 1 == kStages ? 0 : slot + 1;
            uint4 code[2][2];
            uint32_t sc[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t* const row = stage + h * 1024 + r * 128 + t * 32;
                code[h][0] = *reinterpret_cast<const uint4*>(row + (r & 1) * 16);
                code[h][1] = *reinterpret_cast<const uint4*>(row + 16 - (r & 1) * 16);
                four_scales(*reinterpret_cast<const uint32_t*>(stage + 2048 + t * 64 + (r & 3) * 16 + ((r >> 2) + 2 * h) * 4),
                            sc[h]);
            }
            float part[2][NT][4] = {};
#pragma unroll
            for (int p = 0; p < 8; ++p) {
                uint4 x[NT];
#pragma unroll
                for (int b = 0; b < NT; ++b) {
                    x[b] = load_shared(xp[b]);
                    xp[b] += xstep[b];
                }
                uint32_t v[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4& cw = code[h][p >> 2];
                    e2m1x8_f16((p & 3) == 0 ? cw.x : (p & 3) == 1 ? cw.y : (p & 3) == 2 ? cw.z : cw.w, v[h]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[h][i] = mul_f16x2(v[h][i], sc[h][p >> 1]);
                }
#pragma unroll
                for (int b = 0; b < NT; ++b) {
                    mma_16816(part[0][b], v[0][0], v[1][0], v[0][1], v[1][1], x[b].x, x[b].y);
                    mma_16816(part[1][b], v[0][2], v[1][2], v[0][3], v[1][3], x[b].z, x[b].w);
                }
            }
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[b][i] += part[0][b][i] + part[1][b][i];
            if (++c < psteps && j + 1 < j1) continue;
            // the tile or the run ends: columns 2 t and 2 t + 1 of the sums are tokens
            // 8 b + 2 t, 8 b + 2 t + 1
            open = begun && c < psteps;
            if (begun && !open) {
#pragma unroll
                for (int b = 0; b < NT; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (there[b][i & 1])
                            store(8 * b + 2 * t + (i & 1), r + 8 * (i >> 1), acc[b][i], factor[b][i & 1]);
            } else {
                float* const to = begun ? my_sums : my_head;
#pragma unroll
                for (int b = 0; b < NT; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        to[(8 * b + 2 * t + (i & 1)) * kRedStride + r + 8 * (i >> 1)] = acc[b][i];
            }
            if (j + 1 < j1) {
                c = 0;
                begun = true;
                if (++tile == tiles) {
                    tile = 0, ++seg;
                    enter();
                } else {
#pragma unroll
                    for (int b = 0; b < NT; ++b) {
                        xp[b] = x0[b];
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[b][i] = 0.0f;
                    }
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        if (open) {  // this warp's sums and those of the warps that went on with the tile
            const int end = j1 - c + psteps;  // the item behind the tile's last
            int others = 0;
            while (run_start(warp + others + 1) < end) ++others;
            for (int o = lane; o < 16 * s_seg_n[seg]; o += 32) {
                const int at = (o >> 4) * kRedStride + (o & 15);
                float v = my_sums[at];
                for (int w = 1; w <= others; ++w) v += my_head[w * kRed + at];
                store(o >> 4, o & 15, v, s_scale[s_seg_x[seg] + (o >> 4)]);
            }
        }
        if (fe == f1 && (!PANELS || p0 + psteps == steps)) return;
        __syncthreads();  // the next panel or the next segments' rows take the place of these
        if (!PANELS || (p0 += psteps) == steps) break;
        }
        f0 = fe;
    }
}

template <int NT, bool PANELS>
nvfp4_status start_gemv(GemvArgs a, const Plan& plan, int sms, cudaStream_t st)
{
    const int64_t tiles = a.tiles, steps = a.steps;
    int64_t grid;
    if (a.group_offsets) {
        const int64_t fit = max_x_pairs(NT, false) / steps;
        a.seg_rows = static_cast<int>(std::min<int64_t>(8 * NT, fit));
        a.x_rows = static_cast<int>(std::min<int64_t>(fit, std::min<int64_t>(a.rows, 8 * NT * kMaxSegments)));
        // (no more segments than one unfinished for each group, and the full ones)
        grid = std::min<int64_t>(sms, tiles * (std::min<int64_t>(a.groups, a.rows) + a.rows / a.seg_rows));
        a.by_grid = Divisor(static_cast<int>(grid));
    } else {
        a.seg_rows = a.x_rows = plan.seg_rows;
        grid = plan.ctas * ((a.rows + plan.seg_rows - 1) / plan.seg_rows);
        a.by_grid = Divisor(plan.ctas);
        a.each = a.tiles / plan.ctas, a.more = a.tiles % plan.ctas;
    }
    a.panel_steps = a.steps;
    if (PANELS) {
        const int64_t most = max_x_pairs(NT, true) / a.x_rows, count = (steps + most - 1) / most;
        a.panel_steps = static_cast<int>((steps + count - 1) / count);
    }
    const size_t smem = gemv_fixed(NT) + (PANELS ? kPanelTiles * tile_sum_bytes(NT) : 0) +
                        static_cast<size_t>(a.panel_steps) * 512 * a.x_rows;
    static bool raised[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
    if (!raised[dev & 63]) {
        if (cudaFuncSetAttribute(reinterpret_cast<const void*>(gemv_kernel<NT, PANELS>),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kGemvSmem)) != cudaSuccess)
            return NVFP4_ERR_CUDA;
        raised[dev & 63] = true;
    }
    a.by_tiles = Divisor(a.tiles), a.by_steps = Divisor(a.panel_steps), a.by_seg_rows = Divisor(a.seg_rows);
    a.whole = a.n % 128 == 0 && a.k % kStep == 0;
    if (launch_early(!a.status, gemv_kernel<NT, PANELS>, static_cast<int>(grid), 32 * kGemvWarps, smem, st, a) != cudaSuccess)
        return NVFP4_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
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
    const int64_t tiles = (a.n + 127) / 128 * 8, steps = (a.k + kStep - 1) / kStep;
    if (a.rows > 0) {
        if (steps > max_x_pairs(1, false)) return NVFP4_ERR_SHAPE;            // one row does not fit
        if (a.rows > 0x7fffffffll / (tiles * steps)) return NVFP4_ERR_SHAPE;  // indexes are 31-bit on the device
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
    const int sms = sm100_sms(dev);
    if (!sms) return NVFP4_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    a.status = workspace ? static_cast<uint32_t*>(workspace) + 2 : nullptr;
    if (a.status && cudaMemsetAsync(a.status, 0, 4, st) != cudaSuccess) return NVFP4_ERR_CUDA;
    if (a.rows == 0) return NVFP4_OK;
    a.sf_bytes = static_cast<int64_t>(nvfp4_sf_mma_bytes(a.n, a.k));
    a.out_f32 = out_dtype == NVFP4_OUT_F32;
    a.tiles = static_cast<int>(tiles), a.steps = static_cast<int>(steps);
    const auto at_once = [&](int nt) { return std::min<int64_t>(8 * nt, max_x_pairs(nt, false) / steps); };
    if (a.group_offsets) {
        // 16 columns of x at a time where that saves a third of the passes over a matrix
        // (16 experts of 4096 x 1536: 9 rows each 24 us against 29, 32 rows 40 against 49, but
        // 8 rows 23.5 against 21.3; of 1536 x 4096, 16 rows, two passes either way, 44 against
        // 38, and 9 rows, where the rule loses, 34 against 31.5)
        const int64_t mean = (a.rows + a.groups - 1) / a.groups;
        const auto passes = [&](int nt) { return (mean + at_once(nt) - 1) / at_once(nt); };
        const bool two = 3 * passes(2) <= 2 * passes(1);
        return two ? start_gemv<2, false>(a, Plan(), sms, st) : start_gemv<1, false>(a, Plan(), sms, st);
    }
    const Form form = cheapest_form(a.rows, tiles, at_once(1), at_once(2), sms);
    if (form.panels) return start_gemv<1, true>(a, form.plan, sms, st);
    return form.columns == 8 ? start_gemv<1, false>(a, form.plan, sms, st) : start_gemv<2, false>(a, form.plan, sms, st);
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
