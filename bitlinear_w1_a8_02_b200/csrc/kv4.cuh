// The 4-bit cache format and the batch description shared by the attention-side
// kernels (append, read, attention).
//
// A cached value is c * step, c = n - 8 with n in 0..15 and step of five
// significant bits. Dequantisation to bf16 is one multiply-add on pairs: with n
// in the top four mantissa bits of 1.0, fma(1 + n/16, 16 step, -24 step) =
// (n - 8) step; 16 step, 24 step (two more bits than step has) and the result
// (three bits times five) are bf16 numbers, so nothing is rounded.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"

namespace bl {

constexpr int kKvGroup = 32;                 // dims that share a step
constexpr int kKv4MaxSeqs = 4096;            // sequences of a batch
constexpr unsigned kErrTimeout = 1u;         // bits of the device error word
constexpr unsigned kErrBadBatch = 2u;
constexpr float kKvHuge = 1.329227995784916e36f;   // 2^120: vectors that reach it are marked
constexpr float kKvTiny = 7.888609052210118e-31f;  // 2^-100: groups below it are zero

// fl(A / 7) rounded to five significant bits, ties to even.
__device__ __forceinline__ float kv4_step(float amax) {
    if (amax < kKvTiny) return 0.0f;
    unsigned b = __float_as_uint(__fdiv_rn(amax, 7.0f));
    b += 0x3FFFFu + ((b >> 19) & 1u);
    return __uint_as_float(b & ~0x7FFFFu);
}

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN stays
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Eight values of a group -> the word of their codes, n = 8 + rint(fl(x / step)) in bits 4j; step > 0, all finite.
//
// The quotient needs no division: q0 = fl(x r), r = fl(1 / step), and one Newton step q = fl(q0 + fl(x - q0 step) r)
// give rint's argument to within 2^-46 before the last rounding, and that is enough for the same code. A tie is
// x = T = (c + 1/2) step exactly, and then q = c + 1/2 exactly. Any other x is at least one unit of its last place
// from T, which is mant(c + 1/2) / mant(T) units of c + 1/2's, and T has at most 9 bits: more than 0.5009 of a unit, so
// neither the quotient nor q rounds onto the tie.
// Adding 1.5 * 2^23 + 8 leaves n in the low bits; the words' upper parts add up to a constant.
__device__ __forceinline__ uint32_t kv4_word(const float (&x)[8], float step) {
    const float r = __frcp_rn(step);
    uint32_t w = 0;
#pragma unroll
    for (int j = 7; j >= 0; --j) {
        const float q0 = __fmul_rn(x[j], r);
        const float q = __fmaf_rn(__fmaf_rn(-q0, step, x[j]), r, q0);
        w = w * 16u + __float_as_uint(__fadd_rn(q, 12582920.0f));
    }
    constexpr uint32_t upper = 0x4B400000u * 0x11111111u;  // sum of 0x4B400000 * 16^j, mod 2^32
    return w - upper;
}

__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// (lo, hi) -> bf16 pair
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bulk copy of global to shared memory, completion counted on `bar`; addresses and size multiples of 16.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// (a & b) | c as one instruction. With two immediates the compiler makes two of it; the constants are passed as
// registers so that it does not.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// Nibbles i (low half) and i + 4 (high half) of `w` as the bf16 pair 1 + n/16.
template <int I>
__device__ __forceinline__ uint32_t kv4_unit_pair(uint32_t w) {
    const uint32_t sh = I == 0 ? w << 3 : w >> (4 * I - 3);
    return and_or(sh, 0x00780078u, 0x3F803F80u);
}

constexpr uint32_t kBf16x2Sixteen = 0x41804180u;    // (16, 16)
constexpr uint32_t kBf16x2MinusTwentyFour = 0xC1C0C1C0u;  // (-24, -24)

// The public structs as the kernels take them.
struct Kv4View {
    uint8_t* kc;
    uint16_t* ks;
    uint8_t* vc;
    uint16_t* vs;
    int num_pages;
    int page_shift;  // page size = 1 << page_shift
    int hkv;
};

struct Kv4Seqs {
    const int* q_start;
    const int* kv_len;
    const int* table;
    int64_t table_stride;
    int S;
    int W;
};

// Vector index ((page * Hkv + head) * P + offset) of position `pos` of sequence s.
// The caller has checked pos < W * P; a page id out of range gives -1.
__device__ __forceinline__ int64_t kv4_vector(const Kv4View& c, const Kv4Seqs& b, int s, int pos, int head) {
    const int page = b.table[s * b.table_stride + (pos >> c.page_shift)];
    if (page < 0 || page >= c.num_pages) return -1;
    return ((((int64_t)page * c.hkv + head) << c.page_shift)) + (pos & ((1 << c.page_shift) - 1));
}

// Sequence that row `m` belongs to (S: none, a padding row); all 32 lanes call it.
__device__ __forceinline__ int kv4_seq_of_row(const Kv4Seqs& b, int m) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int s0 = 0; s0 < b.S; s0 += 32) {
        const bool before = s0 + lane < b.S && b.q_start[s0 + lane + 1] <= m;
        const int k = __popc(__ballot_sync(0xffffffffu, before));
        n += k;
        if (k < 32) break;
    }
    return min(n, b.S);
}

}  // namespace bl
