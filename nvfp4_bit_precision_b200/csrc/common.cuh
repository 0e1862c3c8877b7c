// common.cuh -- device helpers shared by the NVFP4 kernels (sm_100a only).
//
// Everything here is written for Blackwell: mbarrier-tracked bulk copies into
// shared memory, hardware FP8/FP4 conversions, and bounded waits that give up
// after a wall-clock limit instead of hanging the GPU.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include <mutex>

#include "nvfp4.h"

#if defined(__CUDA_ARCH__) && (__CUDA_ARCH__ < 1000)
#error "this library targets sm_100a (B200) only"
#endif

namespace nvfp4 {

// --------------------------------------------------------------------------
// Bounded waits.  Every spin on an mbarrier gives up after this many
// nanoseconds of %globaltimer, records NVFP4_ERR_TIMEOUT in the status word
// and lets the kernel return normally.
// --------------------------------------------------------------------------
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s

__device__ __forceinline__ uint64_t global_timer_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count)
                 : "memory");
}

// Make initialised barriers visible to the async (bulk copy / tensor core) proxy.
__device__ __forceinline__ void fence_barrier_init()
{
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void fence_proxy_async_smem()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Wait for the phase with the given parity to complete; false once limit_ns
// of %globaltimer have passed.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity,
                                          uint64_t limit_ns = kWaitLimitNs)
{
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (global_timer_ns() - t0 > limit_ns) return false;
    }
}

// Test hook for the timeout path (host side).  When the environment variable
// NVFP4_TEST_UNSIGNALLED_WAIT_NS holds a positive number of nanoseconds, the
// next launches of the quantiser's passes and of the GEMMs issue no copy at
// all, so every consumer waits on a barrier that nothing signals, gives up
// after that many nanoseconds, records NVFP4_ERR_TIMEOUT and returns; nothing
// is in flight when the kernel exits.  Outputs are left unwritten.  Unset (the
// normal case), the waits keep their 2 s limit and the copies run.
inline void wait_test_hook(uint64_t* limit_ns, int* no_copies)
{
    *limit_ns = kWaitLimitNs;
    *no_copies = 0;
    if (const char* e = getenv("NVFP4_TEST_UNSIGNALLED_WAIT_NS")) {
        const unsigned long long v = strtoull(e, nullptr, 10);
        if (v > 0) {
            *limit_ns = v;
            *no_copies = 1;
        }
    }
}

// One-dimensional bulk copy global -> shared, completing on `bar`.
// dst, src 16-byte aligned; bytes a multiple of 16.
__device__ __forceinline__ void bulk_copy_g2s(void* dst, const void* src, uint32_t bytes,
                                              uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            smem_addr(dst)),
        "l"(src), "r"(bytes), "r"(smem_addr(bar))
        : "memory");
}

// Two-dimensional TMA tile load (box given by the tensor map) completing on
// `bar`.  x is the innermost coordinate in elements; x * element size must be
// a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int32_t x, int32_t y,
                                            uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void st_shared_v4(void* p, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(smem_addr(p)), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}

// Two-dimensional TMA store of the box at `src` (this CTA's shared memory) to
// coordinates (x, y) of the map's tensor; parts past the tensor are not
// written.  x * element size must be a multiple of 16 bytes and x, y >= 0.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int32_t x,
                                             int32_t y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(smem_addr(src))
                 : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }

// The issuing thread's committed bulk stores have finished reading shared memory.
__device__ __forceinline__ void bulk_wait_read0()
{
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// The issuing thread's committed bulk stores have completed.
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// cuTensorMapEncodeTiled through the runtime's driver entry point (host).
inline PFN_cuTensorMapEncodeTiled_v12000 encode_tiled_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static bool looked = false;
    if (!looked) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        looked = true;
    }
    return fn;
}

__device__ __forceinline__ void record_status(uint32_t* status, uint32_t code)
{
    if (status) atomicCAS(status, 0u, code);
}

// --------------------------------------------------------------------------
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC'11): two 32x32->64 products
// per round, Weyl key schedule, ten rounds.
// --------------------------------------------------------------------------
struct U4 {
    uint32_t x, y, z, w;
};

__device__ __forceinline__ U4 philox4x32_10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                             uint32_t k0, uint32_t k1)
{
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        // one 32x32 -> 64-bit product gives both halves
        const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
        const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        const uint32_t n0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
        const uint32_t n2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
        c0 = n0;
        c1 = static_cast<uint32_t>(p1);
        c2 = n2;
        c3 = static_cast<uint32_t>(p0);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return U4{c0, c1, c2, c3};
}

// The ten round keys of one seed (key words after 0..9 Weyl steps), computed
// once on the host and passed as kernel parameters, so each round's XOR reads
// its key from the constant bank instead of recomputing it.
struct PhiloxKeys {
    uint32_t k0[10], k1[10];
};

inline void philox_round_keys(uint64_t seed, PhiloxKeys* k)
{
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
    for (int r = 0; r < 10; ++r) {
        k->k0[r] = k0;
        k->k1[r] = k1;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
}

// Philox4x32-10 with precomputed round keys (same result as philox4x32_10
// with key (k->k0[0], k->k1[0])).
__device__ __forceinline__ U4 philox4x32_10_keyed(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                                   const PhiloxKeys& k)
{
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
        const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        const uint32_t n0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k.k0[r];
        const uint32_t n2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k.k1[r];
        c0 = n0;
        c1 = static_cast<uint32_t>(p1);
        c2 = n2;
        c3 = static_cast<uint32_t>(p0);
    }
    return U4{c0, c1, c2, c3};
}

// Two Philox4x32-10 blocks that differ only in the first two counter words,
// computed round by round side by side (two independent dependency chains for
// the scheduler to interleave).  Same results as two philox4x32_10_keyed calls.
__device__ __forceinline__ void philox4x32_10_keyed_x2(uint32_t a0, uint32_t a1, uint32_t b0,
                                                       uint32_t b1, uint32_t c2, uint32_t c3,
                                                       const PhiloxKeys& k, U4& ra, U4& rb)
{
    uint32_t x0 = a0, x1 = a1, x2 = c2, x3 = c3;
    uint32_t y0 = b0, y1 = b1, y2 = c2, y3 = c3;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = static_cast<uint64_t>(x0) * 0xD2511F53u;
        const uint64_t p1 = static_cast<uint64_t>(x2) * 0xCD9E8D57u;
        const uint64_t q0 = static_cast<uint64_t>(y0) * 0xD2511F53u;
        const uint64_t q1 = static_cast<uint64_t>(y2) * 0xCD9E8D57u;
        x0 = static_cast<uint32_t>(p1 >> 32) ^ x1 ^ k.k0[r];
        x2 = static_cast<uint32_t>(p0 >> 32) ^ x3 ^ k.k1[r];
        x1 = static_cast<uint32_t>(p1);
        x3 = static_cast<uint32_t>(p0);
        y0 = static_cast<uint32_t>(q1 >> 32) ^ y1 ^ k.k0[r];
        y2 = static_cast<uint32_t>(q0 >> 32) ^ y3 ^ k.k1[r];
        y1 = static_cast<uint32_t>(q1);
        y3 = static_cast<uint32_t>(q0);
    }
    ra = U4{x0, x1, x2, x3};
    rb = U4{y0, y1, y2, y3};
}

// Four Philox4x32-10 blocks with consecutive 64-bit counters j .. j+3 in the
// first two words, computed round by round side by side.
__device__ __forceinline__ void philox4x32_10_keyed_x4(uint64_t j, uint32_t c2, uint32_t c3,
                                                       const PhiloxKeys& k, U4 (&r)[4])
{
    uint32_t x0[4], x1[4], x2[4], x3[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        x0[b] = static_cast<uint32_t>(j + b);
        x1[b] = static_cast<uint32_t>((j + b) >> 32);
        x2[b] = c2;
        x3[b] = c3;
    }
#pragma unroll
    for (int rd = 0; rd < 10; ++rd) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint64_t p0 = static_cast<uint64_t>(x0[b]) * 0xD2511F53u;
            const uint64_t p1 = static_cast<uint64_t>(x2[b]) * 0xCD9E8D57u;
            x0[b] = static_cast<uint32_t>(p1 >> 32) ^ x1[b] ^ k.k0[rd];
            x2[b] = static_cast<uint32_t>(p0 >> 32) ^ x3[b] ^ k.k1[rd];
            x1[b] = static_cast<uint32_t>(p1);
            x3[b] = static_cast<uint32_t>(p0);
        }
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) r[b] = U4{x0[b], x1[b], x2[b], x3[b]};
}

// MXFP8 stream: random bits for elements idx8*8 .. idx8*8+7; element j takes
// the 16-bit half (j % 2) of word j / 2.
__device__ __forceinline__ U4 sr_block8(const PhiloxKeys& k, uint32_t offset, uint32_t stream,
                                        uint64_t idx8)
{
    return philox4x32_10_keyed(static_cast<uint32_t>(idx8), static_cast<uint32_t>(idx8 >> 32), stream,
                               offset, k);
}

// NVFP4 streams: the four words for elements idx16*16 .. idx16*16+15; word q
// drives elements 4q .. 4q+3 through the stochastic-rounding conversion.
__device__ __forceinline__ U4 sr_block16(const PhiloxKeys& k, uint32_t offset, uint32_t stream,
                                         uint64_t idx16)
{
    return philox4x32_10_keyed(static_cast<uint32_t>(idx16), static_cast<uint32_t>(idx16 >> 32),
                               stream, offset, k);
}

// Stochastic rounding of four scaled values onto E2M1 with Blackwell's
// conversion (saturating at 6).  Element k of the group rounds up iff
// floor(f * 2^16) + v_k >= 2^16, where f is its position between its two grid
// neighbours and v_k is a 16-bit value the conversion assembles from two bytes
// of `rbits` (B2:B0, rev B0:rev B2, B3:B1, rev B1:rev B3 for k = 0..3).
// Returns the four codes, element 0 in the low nibble.
__device__ __forceinline__ uint32_t e2m1x4_sr(const float* y, uint32_t rbits)
{
    uint16_t d;
    asm("cvt.rs.satfinite.e2m1x4.f32 %0, {%1, %2, %3, %4}, %5;"
        : "=h"(d)
        : "f"(y[3]), "f"(y[2]), "f"(y[1]), "f"(y[0]), "r"(rbits));
    return d;
}

__device__ __forceinline__ uint32_t u16_of(const U4& w, int j)
{
    const uint32_t word = (j >> 1) == 0 ? w.x : (j >> 1) == 1 ? w.y : (j >> 1) == 2 ? w.z : w.w;
    return (j & 1) ? (word >> 16) : (word & 0xFFFFu);
}

// Hadamard sign bits: bit i set -> sign i is -1.  Word 0 of Philox(counter
// (0,0,3,0), key = seed); depends on the seed only.
__device__ __forceinline__ uint32_t rht_sign_bits(uint64_t seed)
{
    return philox4x32_10(0u, 0u, 3u, 0u, static_cast<uint32_t>(seed),
                         static_cast<uint32_t>(seed >> 32))
        .x;
}

// --------------------------------------------------------------------------
// Packed FP32 pairs: sm_100a's add/sub/mul .f32x2 perform two IEEE binary32
// operations (round to nearest even) per instruction, lane by lane.
// --------------------------------------------------------------------------
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1, float b0, float b1)
{
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

__device__ __forceinline__ void sub2(float& d0, float& d1, float a0, float a1, float b0, float b1)
{
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "sub.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1)
{
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// max(|a|, |b|, |c|) in one instruction (exact).
__device__ __forceinline__ float absmax3(float a, float b, float c)
{
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// max |v_i| over 16 values, starting from m (m >= 0).  A tree of three-input
// maxima (depth 3 instead of a chain of 8); max is exact, so the order does not
// change the result.
__device__ __forceinline__ float absmax16(const float* v, float m)
{
    const float a = absmax3(v[0], v[1], v[2]), b = absmax3(v[3], v[4], v[5]);
    const float c = absmax3(v[6], v[7], v[8]), d = absmax3(v[9], v[10], v[11]);
    const float e = absmax3(v[12], v[13], v[14]), f = absmax3(v[15], m, 0.0f);
    return absmax3(absmax3(a, b, c), absmax3(d, e, f), 0.0f);
}

// Butterfly stages h = 1, 2, 4, 8 of the 16-point Hadamard (IEEE add/sub in a
// fixed order) on two vectors at once, one per lane of the packed pairs.  The
// random sign flip is applied by the caller when it unpacks the inputs, and
// the transform's factor 1/4 is NOT applied: callers fold it into the scale
// arithmetic, which is exact -- every value the butterflies produce is a
// multiple of 2^-133 (sums of bf16 values) or a normal float, so dividing it by
// 4 never rounds.
__device__ __forceinline__ void hadamard16x2_times4(float (&a)[16], float (&b)[16])
{
#pragma unroll
    for (int h = 1; h < 16; h <<= 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i & h) continue;
            float s0, s1, d0, d1;
            add2(s0, s1, a[i], b[i], a[i + h], b[i + h]);
            sub2(d0, d1, a[i], b[i], a[i + h], b[i + h]);
            a[i] = s0;
            b[i] = s1;
            a[i + h] = d0;
            b[i + h] = d1;
        }
    }
}

// bf16 pair (element 0 in the low half) -> two floats with the sign bit
// flipped by `flip` (0 or 0x80000000).
__device__ __forceinline__ void unpack_bf16x2(uint32_t w, uint32_t flip, float& lo, float& hi)
{
    lo = __uint_as_float(w * 65536u + flip);  // low bf16 into the high half; + flip == xor bit 31
    hi = __uint_as_float((w & 0xFFFF0000u) ^ flip);
}

// --------------------------------------------------------------------------
// Conversions (hardware, exact where stated).
// --------------------------------------------------------------------------
__device__ __forceinline__ float bf16_lo(uint32_t packed) { return __uint_as_float(packed << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t packed)
{
    return __uint_as_float(packed & 0xFFFF0000u);
}

// Eight bf16 values of a 16-byte vector <-> floats (pack8 rounds to nearest even).
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8])
{
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z);
    f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// E4M3 round-to-nearest-even, saturating to +-448; returns the byte.
__device__ __forceinline__ uint32_t e4m3_rne_sat(float v)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0xFFu;
}

// Two E4M3 bytes in one 16-bit value: hi -> upper byte, lo -> lower byte.
__device__ __forceinline__ uint32_t e4m3x2_rne_sat(float hi, float lo)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Value of an E4M3 byte (exact).
__device__ __forceinline__ float e4m3_value(uint32_t byte)
{
    uint32_t h2;
    const uint16_t b = static_cast<uint16_t>(byte & 0xFFu);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(b));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h2 & 0xFFFFu)));
}

// Eight floats -> eight E2M1 codes (RNE, saturating), packed with element 0 in
// the low nibble of byte 0.
__device__ __forceinline__ uint32_t e2m1x8_rne(const float* v)
{
    uint32_t out;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(out)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]),
          "f"(v[7]));
    return out;
}

// Stochastic rounding onto the E4M3 grid (MXFP8 elements), returning the grid
// value (exact, so a following RNE conversion only encodes it): P(up) =
// floor(f * 2^16) / 2^16 with f the position of |y| between its neighbours.
// The 16 bits of the fraction the grid drops are added to (0xFFFF - u) and a
// carry rounds up; values below 2^-6 are first lifted by 2^-6 (truncating) so
// that the grid step equals the float's kept-bit step.  Saturates at 448.
__device__ __forceinline__ float e4m3_sr_value(float y, uint32_t u16)
{
    const float a = fabsf(y);
    const float lift = 0.015625f;  // 2^-6, the smallest normal E4M3 value
    const bool small = a < lift;
    const float a2 = small ? __fadd_rz(a, lift) : a;
    const uint32_t noise = (0xFFFFu - u16) << 4;
    float r = __uint_as_float((__float_as_uint(a2) + noise) & 0xFFF00000u);
    r = small ? __fsub_rn(r, lift) : r;
    r = fminf(r, 448.0f);
    return copysignf(r, y);
}

// --------------------------------------------------------------------------
// Global scale: S = 2688/amax, g = amax/2688 (IEEE single divisions); amax 0
// gives 1, 1; S is capped at 2^118 (g = 2^-118).
// --------------------------------------------------------------------------
__device__ __forceinline__ void global_scales(float amax, float& S, float& g)
{
    if (amax == 0.0f) {
        S = 1.0f;
        g = 1.0f;
        return;
    }
    const float cap = 3.32306998946228968226e+35f;  // 2^118
    const float s = __fdiv_rn(2688.0f, amax);
    if (!(s <= cap)) {
        S = cap;
        g = 3.00926553346026563215e-36f;  // 2^-118
        return;
    }
    S = s;
    g = __fdiv_rn(amax, 2688.0f);
}

// Offset of scale byte (row r, 16-block b) in the tiled tensor-core layout of
// an operand whose rows hold k16 = K/16 blocks: 128x4 atoms of 512 bytes,
// atoms ordered with the K group fastest.
__host__ __device__ __forceinline__ int64_t sf_mma_offset(int64_t r, int64_t b, int64_t k16)
{
    const int64_t atom = (r >> 7) * (k16 >> 2) + (b >> 2);
    return atom * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (b & 3);
}

// SM count of an sm_100 device, 0 for any other (host).
inline int sm100_sms(int dev)
{
    static int sms[64];
    static std::once_flag flags[64];
    std::call_once(flags[dev & 63], [dev]() {
        int major = 0, n = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) == cudaSuccess && major == 10 &&
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
            sms[dev & 63] = n;
    });
    return sms[dev & 63];
}

// Not on a 16-byte boundary.
inline bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// Programmatic dependent launch: a kernel launched with launch_early may start
// while the one before it in the stream still runs (its launch is then hidden), and
// calls wait_for_previous_kernel before it touches anything the other writes: all
// of the other kernel is done by then and its writes are visible.  The earlier
// kernel's let_next_kernel_start only says when the start may come; it comes once
// all of that kernel's CTAs have said so, so none of them is kept from starting.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// (`early` false: an ordinary launch, as after a memset, which is no kernel.)
template <typename... Params, typename... Args>
inline cudaError_t launch_early(bool early, void (*kernel)(Params...), int64_t grid, int block, size_t smem,
                                cudaStream_t stream, Args... args)
{
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid)), cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.dynamicSmemBytes = smem, cfg.stream = stream;
    cfg.attrs = &attr, cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace nvfp4
