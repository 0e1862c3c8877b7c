// kv_append.cu -- keys and values of new tokens into a paged NVFP4 cache, with the
// rotation of keys and queries by their position on the way.
//
//   (a, b) -> (a cos - b sin, b cos + a sin)      for each pair of a head's first `rot` elements
//   S = 2688 / amax,  scale byte = E4M3((amax_block / 6) * S),  code = E2M1(x * (S / scale))
// The turned keys are rounded to bf16, once, and quantised as nvfp4_quantize does it
// from a given amax; so a cache holds the same bits whether a model turns its keys
// itself or leaves that to this call.
//
// The one rounding.  A product of a bf16 and an FP32 number is exact in FP64, and the
// sum of two is then rounded to odd in FP32 (FP64's own rounding lies 29 bits below)
// and to nearest in bf16.  Almost always FP32 is enough: its result r, of two or three
// roundings, is off by less than 2^-23 t (|a| + |b|) + 2^-148, t the largest |cos| or |sin|
// of the thread's pairs, and the sums r - d and r + d by less than 2^-24 (t + 2^-22) (|a| + |b|)
// more.  Where these, with d = 1.6 * 2^-23 t (|a| + |b|) + 2^-126, round to the same bf16 number,
// so does what lies between them.  Otherwise (about one number in 2000) the FP64 form decides.
//
// What bounds it: instructions and HBM alike where there is much to do.  16384 tokens with 32
// query and 8 key heads of 128 (354 MB, 54 us at the copy rate) 79.4 us on the device, 4.5
// TB/s: 290 instructions a warp and head, of which turning is 40%, fill two thirds of the
// issue slots.  Keys and values alone, not turned (86 MB), 23.6 us.  64 tokens with 40 query
// heads 3.7 us, one token 3, a launch and three loads that wait for one another.  The 80
// registers that leave room for three CTAs spill 24 or 32 bytes, 2% of the instructions.
// Steps on the way (with the cache read back, 16 us): every lane quantising, what it turned
// and what it did not, 150 us; packed arithmetic, S / d from a table, queries apart from keys
// and values 120; the next four heads' numbers on their way through shared memory 102; with
// nvfp4_dequantize's later steps 95.5.
#include "kv_cache.cuh"

#include <algorithm>

namespace nvfp4 {
namespace {

struct AppendArgs {
    CacheView cache;
    const uint16_t *k, *v, *q;
    int64_t ldk, hsk, ldv, hsv, ldq, hsq;  // from token to token, from head to head, in elements
    uint16_t* q_out;
    int64_t ldo, hso;
    int64_t tokens;
    int heads;                   // query heads, 0 without queries
    int per_thread;              // heads that a thread goes over
    const int32_t* table;
    int64_t ldt;
    int sequences, table_pages;
    const int32_t *position, *sequence;  // sequence NULL: token t belongs to sequence t
    const float *cos, *sin;      // [angles][rot / 2]
    int64_t angles;
    uint32_t* status;
};

constexpr int kAhead = 4;  // heads whose numbers are on their way
constexpr float kLeast = 1.17549435082228750797e-38f;  // 2^-126

// bf16 of a c - b s, rounded once.
__device__ __noinline__ uint32_t turn_exactly(float a, float c, float b, float s)
{
    const double d = __dadd_rn(__dmul_rn(static_cast<double>(a), static_cast<double>(c)),
                               -__dmul_rn(static_cast<double>(b), static_cast<double>(s)));
    float f = __double2float_rz(d);
    if (static_cast<double>(f) != d && d == d) f = __uint_as_float(__float_as_uint(f) | 1u);
    return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

// Eight consecutive numbers of a cached head, the other half of whose 16-block is the
// neighbouring lane's: four bytes of codes at q, the scale byte (by the even lane) at sf.
// by: S / d for each scale byte.
__device__ __forceinline__ void hold8(uint4 x, float S, const float* by, uint8_t* q, uint8_t* sf, bool writes)
{
    const uint32_t m2 = __vmaxu2(__vimax3_u16x2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu, x.z & 0x7FFF7FFFu), x.w & 0x7FFF7FFFu);
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const uint32_t byte = e4m3_rne_sat(__fmul_rn(div6_rn(__uint_as_float(m << 16)), S));
    const float r = by[byte & 127];
    float f[8];
    unpack8(x, f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) mul2(f[i], f[i + 1], f[i], f[i + 1], r, r);
    const uint32_t codes = e2m1x8_rne(f);
    if (!writes) return;
    *reinterpret_cast<uint32_t*>(q) = codes;
    if ((threadIdx.x & 1) == 0) *sf = static_cast<uint8_t>(byte);
}

// DIM / 16 lanes a head: lane j has elements 8 j.. and rot / 2 + 8 j.. of the turned
// part, or the like of the rest, so that it has both numbers of each of its pairs (with
// NEIGHBOURS a pair's numbers are next to one another).  A thread goes over several
// heads of its token with the same sines and cosines, the next ones' numbers on their
// way; the lanes of a warp have the same heads of neighbouring tokens, so that all of
// them turn queries or all quantise.
template <int DIM, bool NEIGHBOURS>
__global__ void __launch_bounds__(256, 3) append_kernel(const AppendArgs a, const int rot)
{
    constexpr int kLanes = DIM / 16;
    __shared__ float s_by[2][128];
    __shared__ uint4 s_ahead[kAhead * 512];
    wait_for_previous_kernel();
    let_next_kernel_start();
    float S[2], g;
    global_scales(a.cache.amax[0], S[0], g);
    global_scales(a.cache.amax[1], S[1], g);
    {
        const int which = threadIdx.x >> 7;
        const float d = e4m3_value(threadIdx.x & 127);
        s_by[which][threadIdx.x & 127] = d > 0.0f ? __fdiv_rn(S[which], d) : 0.0f;
    }
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / kLanes;
    const int lane = threadIdx.x % kLanes;
    const int turned = rot / 16;  // lanes of the turned part
    const bool turns = lane < turned;
    const int first = turns ? 8 * lane : rot + 8 * (lane - turned);
    const int second = first + (turns ? rot : DIM - rot) / 2;

    int64_t at = -1, pos = -1;  // the token's place in a page's row of tokens, as tokens x heads
    if (t < a.tokens) {
        pos = a.position[t];
        const int64_t seq = a.sequence ? a.sequence[t] : t;
        if (pos >= 0 && seq >= 0) {
            const int64_t index = pos >> a.cache.page_shift;
            int64_t page = -1;
            if (seq < a.sequences && index < a.table_pages && (!a.cos || pos < a.angles)) page = a.table[seq * a.ldt + index];
            if (page < 0 || page >= a.cache.pages) {
                if (lane == 0 && blockIdx.y == 0) record_status(a.status, NVFP4_ERR_INDEX);
            } else {
                at = (page * a.cache.kv_heads << a.cache.page_shift) + (pos & ((1 << a.cache.page_shift) - 1));
            }
        }
    }
    const bool kept = at >= 0;
    const int keys = a.heads, values = a.heads + a.cache.kv_heads, all = values + a.cache.kv_heads;
    const int h0 = blockIdx.y * a.per_thread, h1 = min(h0 + a.per_thread, all);
    // the numbers of the next heads, each thread's for itself
    const uint32_t mine = smem_addr(s_ahead + threadIdx.x);
    const auto fetch = [&](int h) {
        if (kept && h < h1) {
            const uint16_t* const from = h < keys     ? a.q + t * a.ldq + h * a.hsq
                                         : h < values ? a.k + t * a.ldk + (h - keys) * a.hsk
                                                      : a.v + t * a.ldv + (h - values) * a.hsv;
            const uint32_t to = mine + (h - h0) % kAhead * (512 * 16);
            copy16_async(to, from + first);
            copy16_async(to + 256 * 16, from + second);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(h0 + i);
    float c[8], ns[8], k = 0.0f;  // cosines, sines negated, 1.6 * 2^-23 of the largest
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.0f, ns[i] = 0.0f;
    if (turns && kept && h0 < values) {
        // pairs 0..3 and 4..7: at the first and the second place of NEIGHBOURS' pairs, else one after another
        const float* const pc = a.cos + pos * (rot / 2);
        const float* const ps = a.sin + pos * (rot / 2);
        const int p0 = NEIGHBOURS ? first / 2 : first, p1 = NEIGHBOURS ? second / 2 : first + 4;
        const float4 c0 = *reinterpret_cast<const float4*>(pc + p0), c1 = *reinterpret_cast<const float4*>(pc + p1);
        const float4 s0 = *reinterpret_cast<const float4*>(ps + p0), s1 = *reinterpret_cast<const float4*>(ps + p1);
        c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
        ns[0] = -s0.x, ns[1] = -s0.y, ns[2] = -s0.z, ns[3] = -s0.w, ns[4] = -s1.x, ns[5] = -s1.y, ns[6] = -s1.z, ns[7] = -s1.w;
#pragma unroll
        for (int i = 0; i < 8; ++i) k = fmaxf(k, fmaxf(fabsf(c[i]), fabsf(ns[i])));
        k *= 1.9073486328125e-7f;
    }
    __syncthreads();
#pragma unroll 1
    for (int h = h0; h < h1; ++h) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (kept) {
            const uint4* const from = s_ahead + (h - h0) % kAhead * 512 + threadIdx.x;
            x = from[0], y = from[256];
        }
        fetch(h + kAhead);
        if (turns && kept && h < values) {
            float u[8], w[8];  // the pairs' numbers
            if constexpr (NEIGHBOURS) {
                float f[8], e[8];
                unpack8(x, f);
                unpack8(y, e);
#pragma unroll
                for (int j = 0; j < 4; ++j) u[j] = f[2 * j], w[j] = f[2 * j + 1], u[4 + j] = e[2 * j], w[4 + j] = e[2 * j + 1];
            } else {
                unpack8(x, u);
                unpack8(y, w);
            }
            uint32_t p[8], differ = 0;
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float r0, r1, q0, q1, m0, m1, l[4], g[4];
                mul2(r0, r1, w[j], w[j + 1], ns[j], ns[j + 1]);
                fma2(r0, r1, u[j], u[j + 1], c[j], c[j + 1]);
                mul2(q0, q1, w[j], w[j + 1], c[j], c[j + 1]);
                mul2(m0, m1, u[j], u[j + 1], ns[j], ns[j + 1]);
                sub2(q0, q1, q0, q1, m0, m1);
                float d0 = kLeast, d1 = kLeast;
                fma2(d0, d1, fabsf(u[j]) + fabsf(w[j]), fabsf(u[j + 1]) + fabsf(w[j + 1]), k, k);
                sub2(l[0], l[1], r0, r1, d0, d1);
                add2(g[0], g[1], r0, r1, d0, d1);
                sub2(l[2], l[3], q0, q1, d0, d1);
                add2(g[2], g[3], q0, q1, d0, d1);
                // words as they are stored: neighbours' pairs one after another, or the pairs' first and then their second numbers
                if constexpr (NEIGHBOURS) {
                    p[j] = pack2(l[0], l[2]), p[j + 1] = pack2(l[1], l[3]);
                    differ |= (p[j] ^ pack2(g[0], g[2])) | (p[j + 1] ^ pack2(g[1], g[3]));
                } else {
                    p[j / 2] = pack2(l[0], l[1]), p[4 + j / 2] = pack2(l[2], l[3]);
                    differ |= (p[j / 2] ^ pack2(g[0], g[1])) | (p[4 + j / 2] ^ pack2(g[2], g[3]));
                }
            }
            if (differ) {  // the pairs that FP32 left open, looked for again (products may come out fused here or above)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float r = fmaf(u[j], c[j], w[j] * ns[j]), q = w[j] * c[j] - u[j] * ns[j];
                    const float d = fmaf(fabsf(u[j]) + fabsf(w[j]), k, kLeast);
                    uint32_t both = pack2(r - d, q - d);
                    if (both != pack2(r + d, q + d))
                        both = turn_exactly(u[j], c[j], w[j], -ns[j]) | turn_exactly(w[j], c[j], u[j], ns[j]) << 16;
                    if constexpr (NEIGHBOURS) {
                        p[j] = both;
                    } else {
                        p[j >> 1] = __byte_perm(p[j >> 1], both, j & 1 ? 0x5410 : 0x3254);
                        p[4 + (j >> 1)] = __byte_perm(p[4 + (j >> 1)], both, j & 1 ? 0x7610 : 0x3276);
                    }
                }
            }
            x = make_uint4(p[0], p[1], p[2], p[3]), y = make_uint4(p[4], p[5], p[6], p[7]);
        }
        if (h < keys) {
            if (kept) {
                uint16_t* const to = a.q_out + t * a.ldo + h * a.hso;
                *reinterpret_cast<uint4*>(to + first) = x;
                *reinterpret_cast<uint4*>(to + second) = y;
            }
        } else {  // (the lanes of a block meet in hold8: all lanes have the same head)
            const int which = h >= values;
            const int64_t token = kept ? (which ? a.cache.half : 0) + at + (static_cast<int64_t>(h - (which ? values : keys)) << a.cache.page_shift) : 0;
            uint8_t* const q = a.cache.q + token * (DIM / 2);
            uint8_t* const sf = a.cache.sf + token * (DIM / 16);
            hold8(x, S[which], s_by[which], q + first / 2, sf + first / 16, kept);
            hold8(y, S[which], s_by[which], q + second / 2, sf + second / 16, kept);
        }
    }
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_kv_append(const nvfp4_kv_cache* cache, const void* k_bf16, int64_t ldk, int64_t hsk,
                                        const void* v_bf16, int64_t ldv, int64_t hsv, int64_t tokens,
                                        const int32_t* table, int64_t ldt, int64_t sequences, int64_t table_pages,
                                        const int32_t* position, const int32_t* sequence, const float* cos,
                                        const float* sin, int64_t angles, int rot, int neighbours, const void* q_bf16,
                                        int64_t ldq, int64_t hsq, int heads, void* q_out, int64_t ldo, int64_t hso,
                                        void* workspace, size_t ws_bytes, void* stream)
{
    AppendArgs a{};
    const nvfp4_status bad = check_cache(cache, &a.cache);
    if (bad != NVFP4_OK) return bad;
    const int dim = cache->dim, kv = cache->kv_heads;
    if (tokens < 0 || tokens > 0x7fffffffll || sequences < 0 || sequences > 0x7fffffffll || table_pages < 0 ||
        table_pages > 0x7fffffffll || ldt < table_pages || heads < 0 || heads > 32768 || angles < 0)
        return NVFP4_ERR_SHAPE;
    if ((neighbours != 0 && neighbours != 1) || !cos != !sin || (heads > 0 && !cos)) return NVFP4_ERR_INVALID_ARG;
    // (tensors without a token may have no address)
    if (tokens > 0 && ((!q_bf16) != (!q_out) || (heads > 0) != (q_bf16 != nullptr))) return NVFP4_ERR_INVALID_ARG;
    if (cos ? rot < 32 || rot > dim || rot % 32 : rot != 0) return NVFP4_ERR_SHAPE;
    if (tokens > 0 && (!k_bf16 || !v_bf16 || !table || !position || sequences < 1 || table_pages < 1))
        return NVFP4_ERR_INVALID_ARG;
    if (!sequence && sequences < tokens) return NVFP4_ERR_SHAPE;
    const auto strides_ok = [&](int64_t ld, int64_t hs, int n) { return ld >= 0 && (n == 1 || hs >= dim); };
    if (!strides_ok(ldk, hsk, kv) || !strides_ok(ldv, hsv, kv) ||
        (q_bf16 && (!strides_ok(ldq, hsq, heads) || (tokens > 1 && ldo < dim) || (heads > 1 && hso < dim))))
        return NVFP4_ERR_SHAPE;
    if (off16(k_bf16) || off16(v_bf16) || off16(q_bf16) || off16(q_out) || off16(cos) || off16(sin) || ldk % 8 || hsk % 8 ||
        ldv % 8 || hsv % 8 || (q_bf16 && (ldq % 8 || hsq % 8 || ldo % 8 || hso % 8)) ||
        ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(position) | reinterpret_cast<uintptr_t>(sequence)) & 3u))
        return NVFP4_ERR_ALIGN;
    // the heads that are written lie apart: a token's within its stride, or the tokens of a head within the heads'
    if (q_bf16 && tokens > 1 && heads > 1 && (ldo - dim) / (heads - 1) < hso && (hso - dim) / (tokens - 1) < ldo)
        return NVFP4_ERR_SHAPE;
    if (workspace && (ws_bytes < 16 || off16(workspace))) return NVFP4_ERR_WORKSPACE;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
    const int sms = sm100_sms(dev);
    if (!sms) return NVFP4_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    a.status = workspace ? static_cast<uint32_t*>(workspace) + 2 : nullptr;
    if (a.status && cudaMemsetAsync(a.status, 0, 4, st) != cudaSuccess) return NVFP4_ERR_CUDA;
    if (tokens == 0) return NVFP4_OK;
    a.k = static_cast<const uint16_t*>(k_bf16), a.ldk = ldk, a.hsk = hsk;
    a.v = static_cast<const uint16_t*>(v_bf16), a.ldv = ldv, a.hsv = hsv;
    a.q = static_cast<const uint16_t*>(q_bf16), a.ldq = ldq, a.hsq = hsq, a.heads = heads;
    a.q_out = static_cast<uint16_t*>(q_out), a.ldo = ldo, a.hso = hso;
    a.tokens = tokens, a.table = table, a.ldt = ldt;
    a.sequences = static_cast<int>(sequences), a.table_pages = static_cast<int>(table_pages);
    a.position = position, a.sequence = sequence, a.cos = cos, a.sin = sin, a.angles = angles;
    const int all = heads + 2 * kv, lanes = dim / 16;
    // several heads a thread once every multiprocessor has its threads
    const int64_t rounds = tokens * all * lanes / (static_cast<int64_t>(sms) * 768);
    const int per = static_cast<int>(std::min<int64_t>(std::max<int64_t>(rounds, 1), 8));
    a.per_thread = per;
    const dim3 grid(static_cast<unsigned>((tokens * lanes + 255) / 256), static_cast<unsigned>((all + per - 1) / per));
    cudaError_t err = cudaSuccess;
    const auto go = [&](auto kernel) { err = launch_early(!a.status, kernel, grid, 256, 0, st, a, rot); };
    if (dim == 64) neighbours ? go(append_kernel<64, true>) : go(append_kernel<64, false>);
    else if (dim == 128) neighbours ? go(append_kernel<128, true>) : go(append_kernel<128, false>);
    else neighbours ? go(append_kernel<256, true>) : go(append_kernel<256, false>);
    return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
