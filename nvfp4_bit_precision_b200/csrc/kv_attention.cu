// kv_attention.cu -- attention of a few query tokens per sequence over a paged NVFP4
// cache.
//
//   x_j = scale * <q, k_j>,  o = sum_j exp(x_j) v_j / sum_j exp(x_j),  lse = log sum_j exp(x_j)
// over the cached tokens j that a query sees.  One pass over the cache with the running
// maximum and sum of the softmax; work is split over the length, and the parts of a
// head are joined by a second kernel.
//
// The rows of a key head, its queries times the heads of its group, share each read of a
// key and a value.  Arithmetic, on the warp-level tensor core instructions:
//  - a code pair becomes two FP16 values in one conversion, and one packed multiply by the
//    block scale gives e2m1 * e4m3: exact in FP16;
//  - queries are FP16 at a power of two per row, exact down to 2^-32 of the row's largest;
//  - products are keys times queries (16 tokens x 8 rows), so that eight rows fill an
//    instruction; the exponentials change places by an 8x8 transpose in registers;
//  - two tokens' codes are interleaved by nibbles before their conversion, which gives the
//    operand's pairs of tokens without touching the converted values;
//  - products and sums are FP32; an exponential goes into the second product as FP16.
//
// What bounds it.  64 sequences of 5120 tokens on average, 40 heads over 8 key heads of 128
// (383 MB): 79.3 us on the device, 4.8 TB/s; four long ones 88.7 us at 450 MB.  The copies
// alone take 63 us (at 428 MB 66.5: the copy rate), the join 6; decoding and products overlap
// with the copies all but about 10 us: 1060 instructions a warp and 64 tokens at 58% of the
// issue slots, the ALU pipe (conversions) 48% busy.  With pages of 16, looked up and copied
// run by run, 101 us.  One sequence of 1000 tokens 9.3 to 10 us, 3.8 of them the join.
// Steps on the way, for the 64 sequences: four-warp CTAs with one softmax each and 16-byte
// copies 106 us; steps of 64 tokens instead of 32, three CTAs a multiprocessor 95; a worker
// a warp, copies ahead across items 85; joins a warp a row instead of a CTA a row 82.5;
// codes copied to places free of bank conflicts (bulk copies, whose lanes take turns,
// before) 80; the maximum raised only where it must be 78.5; scores of any size and pages
// gone before a window, which the forms up to there did not take, 79.3.  Products held apart by two
// sums each, values decoded ahead of the softmax, 8, 14 or 16 warps: none faster.
#include "kv_cache.cuh"

#include <algorithm>

namespace nvfp4 {
namespace {

// Exponentials are taken from a running maximum that is raised only where a product passes it by
// kSlack in the exponent: they are 2^9 at that maximum and at most 2^15, within FP16, whose
// eleven bits they have down to 2^-23 of it.
// (The sum takes them before that rounding, and so does the log-sum: of many equal products the
// result is off by the rounding that they share, 2^-11 at most, and the log-sum by none.)
constexpr float kUp = 9.0f, kSlack = 6.0f;
constexpr int kLeastSlice = 32;
constexpr size_t kHeadBytes = 256;        // of the workspace, the status word among them
constexpr float kMinusInf = -__builtin_huge_valf();

struct AttendArgs {
    CacheView cache;
    const uint16_t* q;
    int64_t ldb, ldi, ldh;     // of q: from sequence to sequence, token to token, head to head, in elements
    uint16_t* out;             // [sequences][queries][heads][dim]
    float* lse;                // [sequences][queries][heads] or NULL
    const int32_t* table;
    int64_t ldt;
    const int32_t* lengths;
    int sequences, table_pages, queries, heads, group;
    int rows, blocks, block_rows;  // rows (query, head of the group) of a key head, cut into blocks of so many
    int window;
    float scale;
    int by_item;               // records are counted by items, else by workers
    int4* records;             // of the items that a worker begins: item, its first and last worker, sequence (first < 0: one worker's)
    int* bad;                  // of each CTA: what is to be reported
    float2* part_ml;           // [2 workers][block_rows] maximum and sum of a part
    float* part_o;             // [2 workers][block_rows][dim]
    uint32_t* status;
};

__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t two)
{
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(two)));
    return d;
}

// Each half of a register in both halves of another (which the products take as they read it).
__device__ __forceinline__ void both_halves(uint32_t two, uint32_t& lo, uint32_t& hi)
{
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tmov.b32 %0, {l, l};\n\tmov.b32 %1, {h, h};\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(two));
}

// An 8x8 matrix of 16-bit numbers, a row in four lanes, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a)
{
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a sequence's rows see of it: tokens [begin, length), from a slice's boundary on, as slices.
struct Span {
    int begin, length, slices;
};
template <int SLICE>
__device__ __forceinline__ Span span_of(const AttendArgs& a, int seq, int* bad)
{
    const int64_t most = static_cast<int64_t>(a.table_pages) << a.cache.page_shift;
    int n = a.lengths[seq];
    if (n < 0 || n > most) {
        *bad = NVFP4_ERR_INDEX;
        n = n < 0 ? 0 : static_cast<int>(most);
    }
    int begin = 0;
    if (a.window > 0) begin = max(0, n - a.queries + 1 - a.window) & ~(SLICE - 1);
    return {begin, n, max(1, (n - begin + SLICE - 1) / SLICE)};
}

// Rows that work on a slice together: one matrix instruction's.  (Sixteen, with eight warps for their
// registers: 16 heads a key head over 32 sequences of 5120 47 us against 49.5, but 12 rows over four
// short ones 15.8 against 15.4, and 20 rows of five drafts 25.9 against 23.5.)
constexpr int kRows = 8;
// Warps of a CTA, one CTA a multiprocessor: 168 registers a thread with 12, 255 with 8.  (Heads of 256 41.5
// us with 8 and 50.4 with 12, where registers spill; heads of 128 94 and 80.)
constexpr int warps_of(int dim) { return dim == 256 ? 8 : 12; }
template <int DIM, int SLICE>  // SLICE: tokens of a warp's step
struct Shape {
    static constexpr int kSlice = SLICE;
    static constexpr int kWarps = warps_of(DIM);
    static constexpr int kCodes = kSlice * DIM / 2, kScales = kSlice * DIM / 16;
    static constexpr int kStage = 2 * (kCodes + kScales);
    static constexpr int kStages = kStage * kWarps * 3 > 224000 ? 2 : kStage > 2500 ? 3 : 4;
    static constexpr int kRing = kStages * kStage;
    static constexpr size_t kSmem = static_cast<size_t>(kWarps) * kRing;
    // Where the 16-byte vector `col` of token `tok`'s codes lies: the tokens of a slice in order, and the
    // vectors of eight of them so that the reads of keys (by neighbouring tokens) and of values (by tokens 0, 3, 4, 7
    // and 1, 2, 5, 6, a 16-block each lane) meet every bank once.
    static __device__ __forceinline__ int vector_of(int tok, int col)
    {
        if (DIM == 64) return (tok ^ (tok >> 2 & 1)) * 2 + col;
        if (DIM == 128) return tok * 4 + (col ^ (tok >> 1 & 2));
        return tok * 8 + (col ^ (tok & 7));
    }
};

// Each warp is a worker of its own: it takes an equal run of all slices of all (sequence,
// key head, block of rows) items, keeps its own maximum, sums and copies on their way, and
// leaves an item's result, or its part of one that other workers share.
template <int DIM, int SLICE>
__global__ void __launch_bounds__(32 * Shape<DIM, SLICE>::kWarps, 1) attend_kernel(const AttendArgs a)
{
    using S = Shape<DIM, SLICE>;
    constexpr int kWarps = S::kWarps, kSlice = SLICE, kM = kSlice / 16;
    constexpr int kSteps = DIM / 16;       // matrix instructions over the head dimension; 16-blocks of a token
    constexpr int kLaneCodes = DIM / 8;    // bytes of a token's keys that a lane reads
    constexpr int kThreads = 32 * kWarps;
    extern __shared__ __align__(128) uint8_t s_dyn[];
    __shared__ int s_sum[kWarps];
    __shared__ int s_upto[kThreads];
    __shared__ int s_bad;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, t = lane & 3;
    uint8_t* const my = s_dyn + warp * S::kRing;
    const uint32_t ring = smem_addr(my);
    const int items = a.cache.kv_heads * a.blocks;  // of a sequence

    if (threadIdx.x == 0) s_bad = 0;
    wait_for_previous_kernel();
    let_next_kernel_start();
    __syncthreads();
    // All slices of all items, sequence by sequence: each thread adds up some sequences.
    const int per = (a.sequences + kThreads - 1) / kThreads;
    int all = 0;
    {
        const int s0 = min(a.sequences, static_cast<int>(threadIdx.x) * per), s1 = min(a.sequences, s0 + per);
        int upto = 0;
#pragma unroll 1
        for (int s = s0; s < s1; ++s) upto += span_of<kSlice>(a, s, &s_bad).slices * items;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += v;
        }
        if (lane == 31) s_sum[warp] = upto;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) upto += s_sum[w];
            all += s_sum[w];
        }
        s_upto[threadIdx.x] = upto;
    }
    __syncthreads();
    // This worker's run; neighbours are on different multiprocessors.  Where items are long and few, the
    // join of their parts costs as much as their slices: runs are at least the root of a sixteenth of an
    // item's slices (one head over 131072 tokens 26.6 us, with runs of two slices 54; eight heads over
    // 32768 21.3 and 24.2; two over 4096 10.4, with a slice 11, with three 11.8).
    int least = 1;
    while (16 * (least + 1) * (least + 1) <= all / (a.sequences * items)) ++least;
    const int workers = min(static_cast<int>(gridDim.x) * kWarps, (all + least - 1) / least);
    const int worker = warp * gridDim.x + blockIdx.x;
    const int each = all / workers, more = all - each * workers;
    int left = worker < workers ? each + (worker < more ? 1 : 0) : 0;
    if (left == 0 && lane == 0 && !a.by_item) a.records[worker] = make_int4(0, -1, 0, 0);
    int seq = 0, rel = 0;  // where it begins: the sequence, the slice in it
    if (left > 0) {
        const int f = worker * each + min(worker, more);
        int before = 0;  // threads whose sequences lie before
#pragma unroll
        for (int i = 0; i < kThreads; i += 32) before += __popc(__ballot_sync(0xffffffffu, s_upto[i + lane] <= f));
        seq = before * per, rel = f - (before ? s_upto[before - 1] : 0);
#pragma unroll 1
        for (;; ++seq) {
            const int n = span_of<kSlice>(a, seq, &s_bad).slices * items;
            if (rel < n) break;
            rel -= n;
        }
    }

    // Copies, ahead of the work and across the items: the codes and scales of a slice's tokens'
    // keys and values.  The pages of 32 runs of tokens that lie together are at hand at a time, one in
    // each lane; where a slice is one run, its pointers are taken once.
    constexpr int kCopies = S::kCodes / 512;           // of a slice's keys or values, 32 vectors each
    constexpr int kCopyTokens = 1024 / DIM;            // of one copy
    const int run_shift = min(a.cache.page_shift, kSlice == 64 ? 6 : 5);
    const int runs = kSlice >> run_shift;  // of a slice
    const int in_page = (1 << a.cache.page_shift) - 1;
    const int64_t half_codes = a.cache.half * (DIM / 2), half_scales = a.cache.half * (DIM / 16);
    const auto place_of = [&](int i) {  // of this lane's vector of copy i: the place repeats every eight tokens
        return (S::vector_of((i * kCopyTokens + lane / (DIM / 32)) & 7, lane % (DIM / 32)) - (i * kCopyTokens & 7) * (DIM / 32)) * 16 +
               (DIM == 64 ? (lane / 2 & 8) * 32 : 0);
    };
    const uint32_t even_place = ring + place_of(0), odd_place = DIM == 256 ? ring + place_of(1) : even_place;
    // The first token that a sequence's queries see: the pages before it, of which a slice may hold some, may be gone.
    const auto first_seen = [&](int s) {
        if (a.window == 0) return 0;
        const int64_t most = static_cast<int64_t>(a.table_pages) << a.cache.page_shift;
        return static_cast<int>(min(static_cast<int64_t>(a.lengths[s]), most)) - a.queries + 1 - a.window;
    };
    int put = 0;                                      // stage of the ring
    int c_left = left, c_seq = seq, c_rel = rel;      // slices to copy; where the next item's begin
    int c_part = 0, c_token = 0, c_end = 0, c_head = 0, c_of = 0;  // of the item at hand: slices left, next token, end, head, sequence
    int page = -1, known = 0;                         // pages at hand, and how many of them are used
    const auto at_page = [&](int p, int token) {
        return ((static_cast<int64_t>(p) * a.cache.kv_heads + c_head) << a.cache.page_shift) + (token & in_page);
    };
    const auto copy_slice = [&]() {
        if (c_left > 0) {
            --c_left;
            if (c_part == 0) {
                const Span span = span_of<kSlice>(a, c_seq, &s_bad);
                const int item = c_rel / span.slices, first = c_rel - item * span.slices;
                c_part = min(span.slices - first, c_left + 1);
                c_head = item / a.blocks, c_of = c_seq;
                c_token = span.begin + first * kSlice, c_end = min(span.length, c_token + c_part * kSlice);
                c_rel += c_part;
                if (c_rel == span.slices * items) ++c_seq, c_rel = 0;
                known = 32;
            }
            --c_part;
            if (known + runs > 32) {
                const int token = c_token + (lane << run_shift);
                page = -1;
                if (token < c_end) {
                    page = a.table[c_of * a.ldt + (token >> a.cache.page_shift)];
                    if (page < 0 || page >= a.cache.pages) {
                        if (token + (1 << run_shift) > first_seen(c_of)) s_bad = NVFP4_ERR_INDEX;
                        page = -1;
                    }
                }
                known = 0;
            }
            const uint32_t stage = put * S::kStage;
            const int p0 = __shfl_sync(0xffffffffu, page, known);
            if (runs == 1 && p0 >= 0) {
                const int64_t at = at_page(p0, c_token);
                const uint8_t* const q = a.cache.q + at * (DIM / 2) + lane * 16;
                const uint8_t* const sf = a.cache.sf + at * (DIM / 16) + lane * 16;
#pragma unroll
                for (int i = 0; i < kCopies; ++i) {
                    const uint32_t to = (i & 1 ? odd_place : even_place) + stage + i * 512;
                    copy16_async(to, q + i * 512);
                    copy16_async(to + S::kCodes, q + half_codes + i * 512);
                }
#pragma unroll
                for (int i = 0; i < S::kScales; i += 512) {
                    if (lane * 16 + i < S::kScales) {
                        copy16_async(ring + stage + 2 * S::kCodes + lane * 16 + i, sf + i);
                        copy16_async(ring + stage + 2 * S::kCodes + S::kScales + lane * 16 + i, sf + half_scales + i);
                    }
                }
            } else {  // several runs, or zeros in a missing page's place
#pragma unroll 1
                for (int i = 0; i < kCopies; ++i) {
                    const int run = i * kCopyTokens >> run_shift, p = __shfl_sync(0xffffffffu, page, known + run);
                    const uint8_t* const q = a.cache.q + (p < 0 ? 0 : at_page(p, c_token + i * kCopyTokens) * (DIM / 2) + lane * 16);
                    const uint32_t to = (i & 1 ? odd_place : even_place) + stage + i * 512;
                    copy16_async(to, q, p >= 0);
                    copy16_async(to + S::kCodes, p < 0 ? q : q + half_codes, p >= 0);
                }
#pragma unroll
                for (int i = 0; i < S::kScales; i += 512) {
                    const int token = (lane * 16 + i) / (DIM / 16), p = __shfl_sync(0xffffffffu, page, known + (token >> run_shift));
                    if (lane * 16 + i < S::kScales) {
                        const uint8_t* const sf = a.cache.sf + (p < 0 ? 0 : at_page(p, c_token + token) * (DIM / 16));
                        copy16_async(ring + stage + 2 * S::kCodes + lane * 16 + i, sf, p >= 0);
                        copy16_async(ring + stage + 2 * S::kCodes + S::kScales + lane * 16 + i, p < 0 ? sf : sf + half_scales, p >= 0);
                    }
                }
            }
            known += runs;
            c_token += kSlice;
            put = put + 1 == S::kStages ? 0 : put + 1;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < S::kStages; ++i) copy_slice();

    int get = 0;                // stage that is worked on
    float unused, gk, gv;
    global_scales(a.cache.amax[0], unused, gk);
    global_scales(a.cache.amax[1], unused, gv);
#pragma unroll 1
    while (left > 0) {
        const Span span = span_of<kSlice>(a, seq, &s_bad);
        const int item = rel / span.slices, first = rel - item * span.slices;
        const int take = min(span.slices - first, left);
        const int head = item / a.blocks, row0 = (item - head * a.blocks) * a.block_rows;
        const int rows = min(a.block_rows, a.rows - row0);
        const int begin = span.begin + first * kSlice, end = min(span.length, begin + take * kSlice);

        // Queries as FP16, each row at the power of two that brings its largest magnitude
        // to [2^14, 2^15) (as in the few-token products): of step s, lane (r, t) has row r's
        // elements t DIM / 4 + 4 s + 0..3.  A negative scale turns their signs, so that the
        // factors on the products are positive.
        uint32_t qf[kSteps][2];
        float by[2];       // factors on the products of rows 2 t, 2 t + 1: to base-2 logarithms
        {
            const int i = (row0 + r) / a.group, h = (row0 + r) - i * a.group;
            uint4 v[kSteps / 2];
            uint32_t top = 0;
#pragma unroll
            for (int s = 0; s < kSteps / 2; ++s) {
                v[s] = make_uint4(0, 0, 0, 0);
                if (r < rows)
                    v[s] = *reinterpret_cast<const uint4*>(a.q + seq * a.ldb + i * a.ldi + (head * a.group + h) * a.ldh +
                                                           t * (DIM / 4) + 8 * s);
                const uint32_t m = __vmaxu2(
                    __vimax3_u16x2(v[s].x & 0x7FFF7FFFu, v[s].y & 0x7FFF7FFFu, v[s].z & 0x7FFF7FFFu), v[s].w & 0x7FFF7FFFu);
                top = max(top, max(m & 0xFFFFu, m >> 16));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const uint32_t ex = min(max(top >> 7, 15u), 254u);
            const float up = copysignf(__uint_as_float((268u - ex) << 23), a.scale);
#pragma unroll
            for (int s = 0; s < kSteps / 2; ++s) {
                float x[8];
                unpack8(v[s], x);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __half2 two = __floats2half2_rn(x[2 * j] * up, x[2 * j + 1] * up);
                    qf[2 * s + j / 2][j & 1] = *reinterpret_cast<const uint32_t*>(&two);
                }
            }
            // |scale| g log2(e), then the row's power of two; never zero, so that 0 x infinity does not arise
            const float down = __uint_as_float((ex - 14u) << 23);
            const float f2 = fabsf(a.scale) * gk * 1.44269502162933349609375f;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                by[j] = fmaxf(f2 * __shfl_sync(0xffffffffu, down, (2 * t + j) * 4), 1.17549435082228750797e-38f);
        }
        // the tokens that row 2 t + j sees, [last + 1 - window, last] of the part's; what every row sees
        // (rows are in the queries' order)
        const auto last_of = [&](int n) { return span.length - a.queries + (row0 + min(n, rows - 1)) / a.group; };
        const int all_to = min(last_of(0) + 1, end);
        const int all_from = a.window > 0 ? last_of(rows) + 1 - a.window : 0;
        // top: the running maximum of the products, from_top: the same, 0 before there is one, limit: the product that
        // raises it.  (Next to the maximum a product less it is exact, whatever their size.  Fused, as by x - (by top) with
        // the second rounded, was 0.5% faster, but off by a 2^-24 of the score: past 2^26 that left FP16.)
        float top[2], from_top[2], limit[2], sum[2], o[kSteps][4];
        top[0] = top[1] = limit[0] = limit[1] = kMinusInf;
        from_top[0] = from_top[1] = sum[0] = sum[1] = 0.0f;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;

        // The tokens of a row of eight of a matrix instruction, in an order in which neighbouring
        // lanes' reads of keys and of values meet other banks: row 2 j, 2 j + 1 has tokens 2 j and 2 j +
        // 1, or the other way round.
        const int my_token = r ^ (r >> 1 & 1), even_token = 2 * t ^ (t & 1), odd_token = (2 * t + 1) ^ (t & 1);
#pragma unroll 1
        for (int place = begin, k = take; k > 0; --k, place += kSlice) {  // place: of the slice's first token
            asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 1) : "memory");
            __syncwarp();  // this slice has come for every lane
            const uint8_t* const stage = my + get * S::kStage;
            const bool edge = place < all_from || place + kSlice > all_to;

            // products: the slice's tokens x rows; lane (r, t): tokens (my_token) + 8 h + 16 m, rows 2 t, 2 t + 1
            float x[kM][4] = {};
#pragma unroll
            for (int m = 0; m < kM; ++m) {
                uint32_t code[2][kLaneCodes / 4], sc[2][DIM / 64];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int tok = 16 * m + 8 * h + my_token;
                    const uint8_t* const codes = stage + (16 * m + 8 * h) * (DIM / 2);
                    const uint8_t* const scales = stage + 2 * S::kCodes + tok * kSteps + t * (DIM / 64);
                    if constexpr (DIM == 64) {
                        const uint2 w = *reinterpret_cast<const uint2*>(codes + S::vector_of(my_token, t >> 1) * 16 + (t & 1) * 8);
                        code[h][0] = w.x, code[h][1] = w.y;
                        uint32_t unused_half;
                        both_halves(e4m3x2_f16(*scales), sc[h][0], unused_half);
                    } else {
#pragma unroll
                        for (int v = 0; v < DIM / 128; ++v) {
                            const uint4 w = reinterpret_cast<const uint4*>(codes)[S::vector_of(my_token, t * (DIM / 128) + v)];
                            code[h][4 * v] = w.x, code[h][4 * v + 1] = w.y, code[h][4 * v + 2] = w.z, code[h][4 * v + 3] = w.w;
                            both_halves(e4m3x2_f16(reinterpret_cast<const uint16_t*>(scales)[v]), sc[h][2 * v], sc[h][2 * v + 1]);
                        }
                    }
                }
#pragma unroll
                for (int w = 0; w < kLaneCodes / 4; ++w) {
                    uint32_t v[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        e2m1x8_f16(code[h][w], v[h]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[h][i] = mul_f16x2(v[h][i], sc[h][w / 2]);
                    }
                    mma_16816(x[m], v[0][0], v[1][0], v[0][1], v[1][1], qf[2 * w][0], qf[2 * w][1]);
                    mma_16816(x[m], v[0][2], v[1][2], v[0][3], v[1][3], qf[2 * w + 1][0], qf[2 * w + 1][1]);
                }
            }
            uint32_t p[kM][2];  // exponentials, FP16: row r, tokens of rows 2 t, 2 t + 1 (+ 8)
            if (edge) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int last = last_of(2 * t + j), from = a.window > 0 ? last + 1 - a.window : 0;
#pragma unroll
                    for (int m = 0; m < kM; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int at = place + 16 * m + 8 * h + my_token;
                            if (at < from || at > last || at >= end) x[m][2 * h + j] = kMinusInf;
                        }
                }
            }
            float high[2];
            bool rises = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                high[i] = fmaxf(x[0][i], x[0][2 + i]);
#pragma unroll
                for (int m = 1; m < kM; ++m) high[i] = fmaxf(high[i], fmaxf(x[m][i], x[m][2 + i]));
                rises |= high[i] > limit[i];
            }
            if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float now = fmaxf(top[i], high[i]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, d));
                    const float less = now == top[i] ? 1.0f : exp2_fast((top[i] - now) * by[i]);  // (0 from nothing seen)
                    top[i] = now;
                    if (now > kMinusInf) from_top[i] = now, limit[i] = now + __fdividef(kSlack, by[i]);
                    sum[i] *= less;
#pragma unroll
                    for (int s = 0; s < kSteps; ++s) o[s][i] *= less, o[s][2 + i] *= less;
                }
            }
#pragma unroll
            for (int m = 0; m < kM; ++m) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[m][i] = exp2_fast(fmaf(x[m][i] - from_top[i & 1], by[i & 1], kUp));
                    sum[i & 1] += x[m][i];
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const __half2 two = __floats2half2_rn(x[m][2 * h], x[m][2 * h + 1]);
                    p[m][h] = transpose8x8(*reinterpret_cast<const uint32_t*>(&two));
                }
            }
            // o += p v.  Lane (r, t) reads, of the tokens of rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9, the 16-block (half
            // of one, two) number r: the pairs of tokens that an operand register holds are put
            // together from two tokens' codes before these are converted.
#pragma unroll
            for (int m = 0; m < kM; ++m) {
                constexpr int kWords = DIM / 64;  // of a token, eight codes each
                constexpr int kBlocks = DIM == 256 ? 2 : 1;
                uint32_t code[4][kWords], byte[4][kBlocks];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int of_eight = (j & 1) ? odd_token : even_token, tok = 16 * m + 8 * (j >> 1) + of_eight;
                    const uint8_t* const codes = stage + S::kCodes + (16 * m + 8 * (j >> 1)) * (DIM / 2);
                    const uint8_t* const scales = stage + 2 * S::kCodes + S::kScales + tok * kSteps;
                    if constexpr (DIM == 64) {
                        code[j][0] = *reinterpret_cast<const uint32_t*>(codes + S::vector_of(of_eight, r >> 2) * 16 + (r & 3) * 4);
                        byte[j][0] = scales[r >> 1];
                    } else if constexpr (DIM == 128) {
                        const uint2 w = *reinterpret_cast<const uint2*>(codes + S::vector_of(of_eight, r >> 1) * 16 + (r & 1) * 8);
                        code[j][0] = w.x, code[j][1] = w.y;
                        byte[j][0] = scales[r];
                    } else {
                        const uint4 w = reinterpret_cast<const uint4*>(codes)[S::vector_of(of_eight, r)];
                        code[j][0] = w.x, code[j][1] = w.y, code[j][2] = w.z, code[j][3] = w.w;
                        const uint32_t two = reinterpret_cast<const uint16_t*>(scales)[r];
                        byte[j][0] = two & 0xFFu, byte[j][1] = two >> 8;
                    }
                }
                if (edge) {
                    // Tokens that no row sees count as zeros.  A scale that is NaN must not reach, as 0 x NaN,
                    // rows that do not see its token: it goes to those that do here.
#pragma unroll
                    for (int k2 = 0; k2 < kBlocks; ++k2) {
                        uint32_t bad = 0;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int at = 8 * (j >> 1) + ((j & 1) ? odd_token : even_token);
                            if (place + 16 * m + at >= end) byte[j][k2] = 0;
                            if ((byte[j][k2] & 0x7Fu) == 0x7Fu) bad |= 1u << at, byte[j][k2] = 0;
                        }
                        bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
                        bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
                        if (bad) {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int last = last_of(2 * t + i), from = a.window > 0 ? last + 1 - a.window : 0;
                                bool sees = false;
#pragma unroll 1
                                for (int at = 0; at < 16; ++at) {
                                    const int token = place + 16 * m + at;
                                    sees |= (bad >> at & 1) && token >= from && token <= last;
                                }
                                if (sees) {
#pragma unroll
                                    for (int s = k2 * (kSteps / kBlocks); s < (k2 + 1) * (kSteps / kBlocks); ++s)
                                        o[s][i] = o[s][2 + i] = __int_as_float(0x7fffffff);
                                }
                            }
                        }
                    }
                }
                uint32_t sc[2][kBlocks];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k2 = 0; k2 < kBlocks; ++k2) sc[h][k2] = e4m3x2_f16(byte[2 * h][k2] | byte[2 * h + 1][k2] << 8);
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    uint32_t even[2][4], odd[2][4];  // elements 2 i and 2 i + 1 of eight
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t one = code[2 * h][w], two = code[2 * h + 1][w];
                        e2m1x8_f16((one & 0x0F0F0F0Fu) | ((two << 4) & 0xF0F0F0F0u), even[h]);
                        e2m1x8_f16(((one >> 4) & 0x0F0F0F0Fu) | (two & 0xF0F0F0F0u), odd[h]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            even[h][i] = mul_f16x2(even[h][i], sc[h][w * kBlocks / kWords]);
                            odd[h][i] = mul_f16x2(odd[h][i], sc[h][w * kBlocks / kWords]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_16816(o[4 * w + i], even[0][i], odd[0][i], even[1][i], odd[1][i], p[m][0], p[m][1]);
                }
            }
            get = get + 1 == S::kStages ? 0 : get + 1;
            __syncwarp();  // every lane is done with this stage
            copy_slice();
        }

        // The result, or a part: lane (r, t) has elements r DIM / 8.. of rows 2 t, 2 t + 1.
        const bool whole = take == span.slices;
        const int slot = 2 * worker + (first == 0 ? 1 : 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float l = sum[i];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
            const float high = top[i] == kMinusInf ? kMinusInf : top[i] * by[i];
            const int row = 2 * t + i;
            if (row >= rows) continue;
            if (whole) {
                const float n = l == 0.0f ? 0.0f : gv / l;
                const int query = (row0 + row) / a.group, h = (row0 + row) - query * a.group;
                const int64_t at = (static_cast<int64_t>(seq) * a.queries + query) * a.heads + head * a.group + h;
                uint2* const to = reinterpret_cast<uint2*>(a.out + at * DIM + r * (DIM / 8));
#pragma unroll
                for (int s = 0; s < kSteps; s += 2)
                    to[s / 2] = make_uint2(pack2(o[s][i] * n, o[s][2 + i] * n), pack2(o[s + 1][i] * n, o[s + 1][2 + i] * n));
                if (a.lse && r == 0) a.lse[at] = 0.693147182464599609375f * (high + (log2f(l) - kUp));
            } else {
                const int64_t at = static_cast<int64_t>(slot) * a.block_rows + row;
                float4* const to = reinterpret_cast<float4*>(a.part_o + at * DIM + r * (DIM / 8));
#pragma unroll
                for (int s = 0; s < kSteps; s += 2)
                    to[s / 2] = make_float4(o[s][i], o[s][2 + i], o[s + 1][i], o[s + 1][2 + i]);
                if (r == 0) a.part_ml[at] = make_float2(high, l);
            }
        }
        left -= take;
        // the worker that begins an item says who else has a part of it
        if (lane == 0 && first == 0 && (a.by_item || left == 0)) {
            const int end_at = worker * each + min(worker, more) + (each + (worker < more ? 1 : 0)) - left - take + span.slices - 1;
            const int cut = more * (each + 1);
            const int last = end_at < cut ? end_at / (each + 1) : more + (end_at - cut) / each;
            a.records[a.by_item ? seq * items + item : worker] = make_int4(item, whole ? -1 : worker, last, seq);
        } else if (lane == 0 && left == 0 && !a.by_item) {
            a.records[worker] = make_int4(0, -1, 0, 0);
        }
        rel += take;
        if (rel == span.slices * items) ++seq, rel = 0;
    }
    __syncthreads();
    if (threadIdx.x == 0) a.bad[blockIdx.x] = s_bad;
}

// The parts of the items that several workers share: a warp (half of one, the same twice)
// takes a row, or with few rows a share of its parts.  A CTA has one row where gridDim.y
// counts rows, else all of an item's.
constexpr int kJoinWarps = 8;
template <int DIM>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const AttendArgs a, int ctas)
{
    constexpr int kVecs = DIM / 4;                          // of a row
    constexpr int kEach = kVecs > 32 ? kVecs / 32 : 1;      // of a lane
    constexpr int kRowLanes = kVecs < 32 ? kVecs : 32;
    constexpr int kUnits = 32 * kJoinWarps / kRowLanes;     // rows, or shares of them, at a time
    constexpr int kParts = 8;                               // whose loads are in flight together
    __shared__ float4 s_v[kUnits][kVecs];
    __shared__ float2 s_ml[kUnits];
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int4 record = a.records[blockIdx.x];
    if (blockIdx.x == 0 && blockIdx.y == 0) {  // the call's status
        const int bad = static_cast<int>(threadIdx.x) < ctas ? a.bad[threadIdx.x] : NVFP4_OK;
        const int index = __syncthreads_or(bad);
        if (threadIdx.x == 0) *a.status = index ? NVFP4_ERR_INDEX : NVFP4_OK;
    }
    const int head = record.x / a.blocks, row0 = (record.x - head * a.blocks) * a.block_rows;
    const int first = record.y, parts = record.z - first + 1;
    if (first < 0) return;
    const int from = gridDim.y > 1 ? blockIdx.y : 0;
    const int rows = min(gridDim.y > 1 ? from + 1 : a.block_rows, a.rows - row0) - from;
    if (rows <= 0) return;
    int shares = 1;  // of a row's parts
    while (2 * shares * rows <= kUnits) shares *= 2;
    const int unit = threadIdx.x / kRowLanes, d = threadIdx.x % kRowLanes;
    float unused, gv;
    global_scales(a.cache.amax[1], unused, gv);
#pragma unroll 1
    for (int u0 = 0; u0 < rows * shares; u0 += kUnits) {
        const int u = u0 + unit, share = u % shares, row = from + u / shares;
        float high = kMinusInf, l = 0.0f;
        float4 v[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) v[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const auto add = [&](float2 ml, const float4 (&w)[kEach]) {
            const float now = fmaxf(high, ml.x), base = now == kMinusInf ? 0.0f : now;
            const float mine = exp2_fast(high - base), part = exp2_fast(ml.x - base);
            high = now;
            l = l * mine + ml.y * part;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                v[e].x = v[e].x * mine + w[e].x * part, v[e].y = v[e].y * mine + w[e].y * part;
                v[e].z = v[e].z * mine + w[e].z * part, v[e].w = v[e].w * mine + w[e].w * part;
            }
        };
        if (u < rows * shares) {
#pragma unroll 1
            for (int i0 = share; i0 < parts; i0 += kParts * shares) {
                float2 ml[kParts];
                float4 w[kParts][kEach];
#pragma unroll
                for (int i = 0; i < kParts; ++i) {
                    const int part = min(i0 + i * shares, parts - 1);
                    const int64_t at = static_cast<int64_t>(part == 0 ? 2 * first + 1 : 2 * (first + part)) * a.block_rows + row;
                    ml[i] = a.part_ml[at];
#pragma unroll
                    for (int e = 0; e < kEach; ++e) w[i][e] = reinterpret_cast<const float4*>(a.part_o + at * DIM)[d + 32 * e];
                }
#pragma unroll
                for (int i = 0; i < kParts; ++i)
                    if (i0 + i * shares < parts) add(ml[i], w[i]);
            }
        }
        if (shares > 1) {  // (then one turn takes all)
#pragma unroll
            for (int e = 0; e < kEach; ++e) s_v[unit][d + 32 * e] = v[e];
            if (d == 0) s_ml[unit] = make_float2(high, l);
            __syncthreads();
            if (share > 0) continue;
#pragma unroll 1
            for (int i = 1; i < shares; ++i) {
                float4 w[kEach];
#pragma unroll
                for (int e = 0; e < kEach; ++e) w[e] = s_v[unit + i][d + 32 * e];
                add(s_ml[unit + i], w);
            }
        }
        if (u >= rows * shares) continue;
        const float n = l == 0.0f ? 0.0f : gv / l;
        const int i = (row0 + row) / a.group, h = (row0 + row) - i * a.group;
        const int64_t at = (static_cast<int64_t>(record.w) * a.queries + i) * a.heads + head * a.group + h;
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            reinterpret_cast<uint2*>(a.out + at * DIM)[d + 32 * e] =
                make_uint2(pack2(v[e].x * n, v[e].y * n), pack2(v[e].z * n, v[e].w * n));
        if (a.lse && d == 0) a.lse[at] = 0.693147182464599609375f * (high + (log2f(l) - kUp));
    }
}

// Rows of a block, the CTAs of the attention and its records.
struct Cut {
    int rows, blocks, block_rows;
    int slice;     // tokens of a step
    int64_t ctas, workers, records;
};
Cut cut_of(int64_t sequences, int queries, int heads, int kv_heads, int dim, int64_t capacity, int sms)
{
    Cut c;
    c.rows = queries * (heads / kv_heads);
    c.blocks = (c.rows + kRows - 1) / kRows;
    c.block_rows = (c.rows + c.blocks - 1) / c.blocks;
    const int64_t items = sequences * kv_heads * c.blocks;
    // Steps of 64 tokens save a tenth of the instructions, those of 32 share out short work better: one
    // sequence of 32768 tokens 22.1 us with 32 and 23.9 with 64; 64 sequences of 5120 95 and 82.5.  The
    // host knows the table's width and not the lengths, so short sequences in a wide table take 64 (one of
    // 1000 tokens 9.3 us, in a table for 131072 10.1; eight of 300 10.2 and 10.5).
    c.slice = dim == 256 || items * (capacity / 64 + 1) <= 8000 ? 32 : 64;
    c.ctas = std::min<int64_t>(sms, items * (capacity / kLeastSlice + 2));  // (no more than there can be slices)
    c.workers = c.ctas * warps_of(dim);
    c.records = std::min(items, c.workers);
    return c;
}

constexpr int64_t kMostRows = 1 << 24;  // of a key head

// Slices of all items are counted in 31 bits on the device.
bool counts_fit(int64_t sequences, int queries, int heads, int kv_heads, int64_t capacity)
{
    const int64_t rows = static_cast<int64_t>(queries) * (heads / kv_heads);
    return rows <= kMostRows && capacity / kLeastSlice + 2 <= 0x7fffffffll / (sequences * kv_heads) / ((rows + kRows - 1) / kRows);
}

constexpr int kMostSms = 192;  // of the workspace's size, which is known without a device

template <int DIM, int SLICE>
nvfp4_status start(const AttendArgs& a, const Cut& cut, cudaStream_t st)
{
    using S = Shape<DIM, SLICE>;
    static bool raised[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
    if (!raised[dev & 63]) {
        if (cudaFuncSetAttribute(reinterpret_cast<const void*>(attend_kernel<DIM, SLICE>),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem)) != cudaSuccess)
            return NVFP4_ERR_CUDA;
        raised[dev & 63] = true;
    }
    if (launch_early(true, attend_kernel<DIM, SLICE>, cut.ctas, 32 * S::kWarps, S::kSmem, st, a) != cudaSuccess)
        return NVFP4_ERR_CUDA;
    // a CTA for each row while that fills no more than the multiprocessors
    const bool apart = cut.records * cut.block_rows <= 4 * cut.ctas;
    const dim3 grid(static_cast<unsigned>(cut.records), apart ? static_cast<unsigned>(cut.block_rows) : 1);
    if (launch_early(true, join_kernel<DIM>, grid, 32 * kJoinWarps, 0, st, a, static_cast<int>(cut.ctas)) != cudaSuccess)
        return NVFP4_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

size_t workspace_bytes(const Cut& c, int dim)
{
    const size_t parts = 2 * static_cast<size_t>(c.workers) * c.block_rows;
    return kHeadBytes + kMostSms * 4 + static_cast<size_t>(c.records) * sizeof(int4) + parts * (sizeof(float2) + 4 * static_cast<size_t>(dim)) + 16;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" size_t nvfp4_kv_attention_workspace_size(int64_t sequences, int queries, int heads, int kv_heads, int dim,
                                                    int64_t capacity)
{
    if (sequences < 1 || queries < 1 || kv_heads < 1 || heads < kv_heads || capacity < 0 ||
        (dim != 64 && dim != 128 && dim != 256) || sequences > (1 << 20) || queries > (1 << 20) || heads > 65536 ||
        !counts_fit(sequences, queries, heads, kv_heads, capacity))
        return kHeadBytes;  // (nothing to do, or sizes that the call refuses)
    return workspace_bytes(cut_of(sequences, queries, heads, kv_heads, dim, capacity, kMostSms), dim);
}

extern "C" nvfp4_status nvfp4_kv_attention(const void* q_bf16, int64_t ldb, int64_t ldi, int64_t ldh, int64_t sequences,
                                           int queries, int heads, const nvfp4_kv_cache* cache, const int32_t* table,
                                           int64_t ldt, int64_t table_pages, const int32_t* lengths, float scale,
                                           int64_t window, void* out_bf16, float* lse, void* workspace, size_t ws_bytes,
                                           void* stream)
{
    AttendArgs a{};
    const nvfp4_status bad = check_cache(cache, &a.cache);
    if (bad != NVFP4_OK) return bad;
    const int dim = cache->dim, kv = cache->kv_heads;
    if (sequences < 0 || sequences > (1 << 20) || queries < 1 || queries > (1 << 20) || heads < 1 || heads > 65536 || heads % kv ||
        table_pages < 0 || table_pages > 0x7fffffffll || ldt < table_pages || window < 0)
        return NVFP4_ERR_SHAPE;
    if (!(scale == scale) || scale - scale != 0.0f) return NVFP4_ERR_INVALID_ARG;
    if (sequences > 0 && (!q_bf16 || !out_bf16 || !lengths || (table_pages > 0 && !table))) return NVFP4_ERR_INVALID_ARG;
    if (ldb < 0 || ldi < 0 || (heads > 1 && ldh < dim)) return NVFP4_ERR_SHAPE;
    const int64_t capacity = table_pages * cache->page_size;
    // (places in a sequence are 31-bit numbers, and so are they less the queries and a window)
    if (capacity > 0x7f000000ll) return NVFP4_ERR_SHAPE;
    if (off16(q_bf16) || off16(out_bf16) || ldb % 8 || ldi % 8 || ldh % 8 ||
        ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(lengths) | reinterpret_cast<uintptr_t>(lse)) & 3u))
        return NVFP4_ERR_ALIGN;
    if (!workspace || off16(workspace) || ws_bytes < kHeadBytes) return NVFP4_ERR_WORKSPACE;
    if (static_cast<int64_t>(queries) * (heads / kv) > kMostRows) return NVFP4_ERR_SHAPE;
    if (sequences > 0 && !counts_fit(sequences, queries, heads, kv, capacity)) return NVFP4_ERR_SHAPE;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
    const int sms = sm100_sms(dev);
    if (!sms) return NVFP4_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (sequences == 0) {
        return cudaMemsetAsync(static_cast<uint8_t*>(workspace) + 8, 0, 4, st) == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
    }
    const Cut cut = cut_of(sequences, queries, heads, kv, dim, capacity, std::min(sms, kMostSms));
    if (ws_bytes < workspace_bytes(cut, dim)) return NVFP4_ERR_WORKSPACE;
    a.q = static_cast<const uint16_t*>(q_bf16), a.ldb = ldb, a.ldi = ldi, a.ldh = ldh;
    a.out = static_cast<uint16_t*>(out_bf16), a.lse = lse;
    a.table = table, a.ldt = ldt, a.lengths = lengths;
    a.sequences = static_cast<int>(sequences), a.table_pages = static_cast<int>(table_pages);
    a.queries = queries, a.heads = heads, a.group = heads / kv;
    a.rows = cut.rows, a.blocks = cut.blocks, a.block_rows = cut.block_rows;
    a.window = window >= capacity ? 0 : static_cast<int>(window);
    a.scale = scale;
    a.by_item = cut.records < cut.workers;
    uint8_t* at = static_cast<uint8_t*>(workspace) + kHeadBytes;
    a.bad = reinterpret_cast<int*>(at);
    at += kMostSms * 4;
    a.records = reinterpret_cast<int4*>(at);
    at += cut.records * sizeof(int4);
    a.part_o = reinterpret_cast<float*>(at);
    at += static_cast<size_t>(2 * cut.workers) * cut.block_rows * dim * 4;
    a.part_ml = reinterpret_cast<float2*>(at);
    a.status = static_cast<uint32_t*>(workspace) + 2;
    if (dim == 256) return start<256, 32>(a, cut, st);
    if (dim == 128) return cut.slice == 32 ? start<128, 32>(a, cut, st) : start<128, 64>(a, cut, st);
    return cut.slice == 32 ? start<64, 32>(a, cut, st) : start<64, 64>(a, cut, st);
}
