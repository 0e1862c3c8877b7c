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
// and to nearest in bf16.  Almost always FP32 is enough: with p = RN(b sin), r = RN(a
// cos - p) is off by at most 2^-24 (|p| + |r|) and 2^-149 for each of the two roundings,
// and where r - d and r + d, d = 2^-22 (|p| + |r|) + 2^-126, round to the same bf16
// number, so does what lies between them.  Otherwise (about one number in 5000) the
// FP64 form decides.
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
    int groups;                  // threads' head groups of a token
    const int32_t* table;
    int64_t ldt;
    int sequences, table_pages;
    const int32_t *position, *sequence;  // sequence NULL: token t belongs to sequence t
    const float *cos, *sin;      // [angles][rot / 2]
    int64_t angles;
    uint32_t* status;
};

// bf16 of a c - b s, rounded once.
__device__ __noinline__ uint32_t turn_exactly(float a, float c, float b, float s)
{
    const double d = __dadd_rn(__dmul_rn(static_cast<double>(a), static_cast<double>(c)),
                               -__dmul_rn(static_cast<double>(b), static_cast<double>(s)));
    float f = __double2float_rz(d);
    if (static_cast<double>(f) != d && d == d) f = __uint_as_float(__float_as_uint(f) | 1u);
    return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

// Two pairs' a' (or, with the roles exchanged and s negated, b') as packed bf16.
__device__ __forceinline__ uint32_t turn2(float a0, float c0, float b0, float s0, float a1, float c1, float b1, float s1)
{
    const float p0 = __fmul_rn(b0, s0), p1 = __fmul_rn(b1, s1);
    const float r0 = __fmaf_rn(a0, c0, -p0), r1 = __fmaf_rn(a1, c1, -p1);
    const float small = 1.17549435082228750797e-38f, part = 2.384185791015625e-7f;  // 2^-126, 2^-22
    const float d0 = __fmaf_rn(fabsf(p0) + fabsf(r0), part, small), d1 = __fmaf_rn(fabsf(p1) + fabsf(r1), part, small);
    const uint32_t lo = pack2(r0 - d0, r1 - d1), hi = pack2(r0 + d0, r1 + d1);
    if (lo == hi) return lo;
    return turn_exactly(a0, c0, b0, s0) | turn_exactly(a1, c1, b1, s1) << 16;
}

// Eight consecutive numbers of a cached head, the other half of whose 16-block is the
// neighbouring lane's: four bytes of codes at q, the scale byte (by the even lane) at sf.
__device__ __forceinline__ void hold8(uint4 x, float S, uint8_t* q, uint8_t* sf, bool writes)
{
    float f[8];
    unpack8(x, f);
    float m = absmax3(absmax3(absmax3(fabsf(f[0]), f[1], f[2]), f[3], f[4]), f[5], absmax3(fabsf(f[6]), f[7], 0.0f));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const uint32_t byte = e4m3_rne_sat(__fmul_rn(__fdiv_rn(m, 6.0f), S));
    const float d = e4m3_value(byte);
    const float by = d > 0.0f ? __fdiv_rn(S, d) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) mul2(f[i], f[i + 1], f[i], f[i + 1], by, by);
    const uint32_t codes = e2m1x8_rne(f);
    if (!writes) return;
    *reinterpret_cast<uint32_t*>(q) = codes;
    if ((threadIdx.x & 1) == 0) *sf = static_cast<uint8_t>(byte);
}

// DIM / 16 lanes a head: lane j has elements 8 j.. and ROT / 2 + 8 j.. of the turned
// part, or the like of the rest, so that it has both numbers of each of its pairs
// (ROT = -1: pairs of neighbours, any turned part).  A thread goes over several heads
// of its token with the same sines and cosines.
template <int DIM, bool NEIGHBOURS>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a, const int rot)
{
    constexpr int kLanes = DIM / 16;
    wait_for_previous_kernel();
    let_next_kernel_start();
    const int64_t item = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / kLanes;
    const int lane = threadIdx.x % kLanes;
    const int64_t t = item / a.groups;
    const int group = static_cast<int>(item - t * a.groups);
    const bool there = t < a.tokens;
    const int turned = rot / 16;  // lanes of the turned part
    const bool turns = lane < turned;
    const int first = turns ? 8 * lane : rot + 8 * (lane - turned);
    const int second = first + (turns ? rot : DIM - rot) / 2;

    int64_t at = -1, pos = -1;  // the token's place in a page's row of tokens, as tokens x heads
    if (there) {
        pos = a.position[t];
        const int64_t seq = a.sequence ? a.sequence[t] : t;
        if (pos >= 0 && seq >= 0) {
            const int64_t index = pos >> a.cache.page_shift;
            int64_t page = -1;
            if (seq < a.sequences && index < a.table_pages && (!a.cos || pos < a.angles)) page = a.table[seq * a.ldt + index];
            if (page < 0 || page >= a.cache.pages) {
                if (lane == 0 && group == 0) record_status(a.status, NVFP4_ERR_INDEX);
            } else {
                at = (page * a.cache.kv_heads << a.cache.page_shift) + (pos & ((1 << a.cache.page_shift) - 1));
            }
        }
    }
    const bool kept = at >= 0;
    float c[8], s[8];
    if (turns && kept) {
        const int64_t row = pos * (rot / 2);
        if constexpr (NEIGHBOURS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = a.cos[row + first / 2 + i], s[i] = a.sin[row + first / 2 + i];
                c[4 + i] = a.cos[row + second / 2 + i], s[4 + i] = a.sin[row + second / 2 + i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 x = *reinterpret_cast<const float4*>(a.cos + row + first + i);
                const float4 y = *reinterpret_cast<const float4*>(a.sin + row + first + i);
                c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
                s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
            }
        }
    }
    float S[2], g;
    global_scales(a.cache.amax[0], S[0], g);
    global_scales(a.cache.amax[1], S[1], g);
    const int all = a.heads + 2 * a.cache.kv_heads;
#pragma unroll 1
    for (int i = 0; i < a.per_thread; ++i) {
        const int h = group * a.per_thread + i;
        const bool mine = kept && h < all;
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (mine) {
            const uint16_t* from = h < a.heads                       ? a.q + t * a.ldq + h * a.hsq
                                   : h < a.heads + a.cache.kv_heads ? a.k + t * a.ldk + (h - a.heads) * a.hsk
                                                                    : a.v + t * a.ldv + (h - a.heads - a.cache.kv_heads) * a.hsv;
            x = *reinterpret_cast<const uint4*>(from + first);
            y = *reinterpret_cast<const uint4*>(from + second);
        }
        if (mine && turns && h < a.heads + a.cache.kv_heads) {
            float u[8], w[8];
            unpack8(x, u);
            unpack8(y, w);
            uint32_t p[4], r[4];
            if constexpr (NEIGHBOURS) {
                uint32_t e[4], o[4];  // the even and odd elements of pairs 2 j, 2 j + 1
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    e[j] = turn2(u[4 * j], c[2 * j], u[4 * j + 1], s[2 * j], u[4 * j + 2], c[2 * j + 1], u[4 * j + 3], s[2 * j + 1]);
                    o[j] = turn2(u[4 * j + 1], c[2 * j], u[4 * j], -s[2 * j], u[4 * j + 3], c[2 * j + 1], u[4 * j + 2], -s[2 * j + 1]);
                    e[2 + j] = turn2(w[4 * j], c[4 + 2 * j], w[4 * j + 1], s[4 + 2 * j], w[4 * j + 2], c[5 + 2 * j], w[4 * j + 3], s[5 + 2 * j]);
                    o[2 + j] = turn2(w[4 * j + 1], c[4 + 2 * j], w[4 * j], -s[4 + 2 * j], w[4 * j + 3], c[5 + 2 * j], w[4 * j + 2], -s[5 + 2 * j]);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    p[2 * j] = __byte_perm(e[j], o[j], 0x5410), p[2 * j + 1] = __byte_perm(e[j], o[j], 0x7632);
                    r[2 * j] = __byte_perm(e[2 + j], o[2 + j], 0x5410), r[2 * j + 1] = __byte_perm(e[2 + j], o[2 + j], 0x7632);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    p[j] = turn2(u[2 * j], c[2 * j], w[2 * j], s[2 * j], u[2 * j + 1], c[2 * j + 1], w[2 * j + 1], s[2 * j + 1]);
                    r[j] = turn2(w[2 * j], c[2 * j], u[2 * j], -s[2 * j], w[2 * j + 1], c[2 * j + 1], u[2 * j + 1], -s[2 * j + 1]);
                }
            }
            x = make_uint4(p[0], p[1], p[2], p[3]), y = make_uint4(r[0], r[1], r[2], r[3]);
        }
        if (mine && h < a.heads) {
            uint16_t* const to = a.q_out + t * a.ldo + h * a.hso;
            *reinterpret_cast<uint4*>(to + first) = x;
            *reinterpret_cast<uint4*>(to + second) = y;
        }
        // (the lanes of a block meet in hold8: all lanes come here)
        const bool holds = mine && h >= a.heads;
        const bool values = h >= a.heads + a.cache.kv_heads;
        const int head = holds ? h - a.heads - (values ? a.cache.kv_heads : 0) : 0;
        const int64_t token = holds ? (values ? a.cache.half : 0) + at + (static_cast<int64_t>(head) << a.cache.page_shift) : 0;
        uint8_t* const q = a.cache.q + token * (DIM / 2);
        uint8_t* const sf = a.cache.sf + token * (DIM / 16);
        hold8(x, S[values], q + first / 2, sf + first / 16, holds);
        hold8(y, S[values], q + second / 2, sf + second / 16, holds);
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
        table_pages > 0x7fffffffll || ldt < table_pages || heads < 0 || heads > 65536 || angles < 0)
        return NVFP4_ERR_SHAPE;
    if ((neighbours != 0 && neighbours != 1) || !cos != !sin || (!q_bf16) != (!q_out) || (heads > 0) != (q_bf16 != nullptr) ||
        (heads > 0 && !cos))
        return NVFP4_ERR_INVALID_ARG;
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
    // several heads a thread once every multiprocessor has its 2048 threads
    const int64_t rounds = tokens * all * lanes / (static_cast<int64_t>(sms) * 2048);
    a.per_thread = static_cast<int>(std::min<int64_t>(std::max<int64_t>(rounds, 1), 8));
    a.groups = (all + a.per_thread - 1) / a.per_thread;
    const int64_t threads = tokens * a.groups * lanes, grid = (threads + 255) / 256;
    if (grid > 0x7fffffffll) return NVFP4_ERR_SHAPE;
    cudaError_t err = cudaSuccess;
    const auto go = [&](auto kernel) { err = launch_early(!a.status, kernel, grid, 256, 0, st, a, rot); };
    if (dim == 64) neighbours ? go(append_kernel<64, true>) : go(append_kernel<64, false>);
    else if (dim == 128) neighbours ? go(append_kernel<128, true>) : go(append_kernel<128, false>);
    else neighbours ? go(append_kernel<256, true>) : go(append_kernel<256, false>);
    return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}
