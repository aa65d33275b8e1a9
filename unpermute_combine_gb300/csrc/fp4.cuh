// fp4.cuh -- e2m1 codes with a scale for each block, as the quantizers and the
// grouped products in 4-bit floating point share them.
//
// A block of 16 elements has an e4m3 scale and, for the whole tensor, a float g:
// x stands for code * scale * g, scale = e4m3(amax / (6 g)), 6 being e2m1's
// largest value.  A block of 32 has a power of two, scale = 2^(floor(log2 amax) - 2)
// in an exponent byte (biased by 127, at least 0), and no g.
#pragma once

#include "common.cuh"

namespace moe {

// e4m3's and the exponent byte's NaN: the scale of a block that holds a NaN or an
// infinity, which e2m1 has no code for; every element of such a block reads as NaN.
constexpr uint32_t kNanScaleE4M3 = 0x7Fu;
constexpr uint32_t kNanScaleE8M0 = 0xFFu;
constexpr uint32_t kMostScaleE4M3 = 0x7Eu;       // 448

// Eight floats to eight e2m1 codes, the first in the lowest bits: to nearest,
// ties to the even code, saturated at 6.
__device__ __forceinline__ uint32_t e2m1x8(const float* q) {
    uint32_t r;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(r) : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]),
          "f"(q[7]));
    return r;
}

// The float of an e4m3 byte (exact).
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    float a, b;
    e4m3x2_to_f32(byte, a, b);
    return a;
}

// The float of an exponent byte: 2^(byte - 127); 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    if (byte == kNanScaleE8M0) return __uint_as_float(0x7FC00000u);
    return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// What the scales of a tensor's blocks need of its g.
struct Fp4Unit {
    float g, six, inv_six;        // g, 6 g and its reciprocal
    bool normal;                  // 6 g is far from the ends of float32's range
};

__device__ __forceinline__ bool far_from_ends(float v) { return v >= 0x1p-100f && v <= 0x1p100f; }

__device__ __forceinline__ Fp4Unit fp4_unit(const float* global_scale) {
    Fp4Unit u;
    u.g = global_scale ? __ldg(global_scale) : 1.0f;
    u.six = 6.0f * u.g;
    u.inv_six = __frcp_rn(u.six);
    u.normal = far_from_ends(u.six);
    return u;
}

// a / b for a correctly rounded r = 1 / b, by one step of Markstein's correction
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990): the remainder of the first quotient is exact in an FMA.  For
// b far from the ends of the range and quotients that do not overflow; three
// instructions, where a division takes about ten and the rows come at 14 an
// element (one SM's share of the memory bandwidth).
__device__ __forceinline__ float quotient(float a, float b, float r) {
    const float q = __fmul_rn(a, r);
    return __fmaf_rn(__fmaf_rn(-q, b, a), r, q);
}
// Two at once, negated: -(a / b), less = -r.  A zero comes out with the sign that -(a / b)
// has, where the steps as above would make -0 into 0: -0 * r - (-0 * b - a) is 0.
__device__ __forceinline__ float2 less_quotient2(float2 a, float2 b, float2 less) {
    const float2 q = mul2(a, less);
    return fma2(fma2(q, b, a), less, q);
}

// Scale byte of a block whose largest magnitude has the bits `amax` (they order
// like the magnitudes, NaN above infinity), and in `step` the float scale * g by
// which elements are divided: NaN for a NaN scale, 0 where the scale is 0.
template <int BLOCK>
__device__ __forceinline__ uint32_t fp4_scale(uint32_t amax, const Fp4Unit& u, float& step) {
    static_assert(BLOCK == 16 || BLOCK == 32, "a block's size names its scale's type");
    if (BLOCK == 32) {
        const uint32_t e = amax >> 23;
        const uint32_t byte = amax >= 0x7F800000u ? kNanScaleE8M0 : e > 2 ? e - 2 : 0u;
        step = e8m0_value(byte);
        return byte;
    }
    const float a = __uint_as_float(amax);
    float q = __fmul_rn(a, u.inv_six);
    if (!u.normal) q = amax ? __fdiv_rn(a, u.six) : 0.0f;       // (zeros may have a g of 0)
    else if (q < 1024.0f) q = quotient(a, u.six, u.inv_six);    // above, it saturates
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(q));
    const uint32_t byte = amax >= 0x7F800000u ? kNanScaleE4M3 : uint32_t(two) & 0xFFu;
    step = __fmul_rn(e4m3_value(byte), u.g);
    return byte;
}

// Codes of N elements of one block: e2m1 of the float quotient v / step.  Where
// the step is 0 or NaN they are 0.
template <int BLOCK, int N>
__device__ __forceinline__ void fp4_codes(const float* v, uint32_t scale, float step,
                                          uint32_t* out) {
    float q[N];
    uint32_t sign = 0;          // where q is the negated quotient: the sign bits of eight codes
    if (BLOCK == 32) {          // a power of two: the product with its inverse is the quotient
        const bool nan = scale == kNanScaleE8M0;
        const float2 inv = both(__uint_as_float((254u - scale) << 23));
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 p = mul2(make_float2(v[i], v[i + 1]), inv);
            q[i] = nan ? 0.0f : p.x, q[i + 1] = nan ? 0.0f : p.y;
        }
    } else if (far_from_ends(step) && scale != kMostScaleE4M3) {   // |v / step| <= 9
        sign = 0x88888888u;
        const float2 b = both(step), less = both(-__frcp_rn(step));
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 p = less_quotient2(make_float2(v[i], v[i + 1]), b, less);
            q[i] = p.x, q[i + 1] = p.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) q[i] = step > 0.0f ? __fdiv_rn(v[i], step) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < N / 8; ++i) out[i] = e2m1x8(q + 8 * i) ^ sign;
}

// Largest magnitude bits of N floats.
template <int N>
__device__ __forceinline__ uint32_t amax_bits(const float* v) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    return m;
}

// ------------------------------------------------- where weights keep their scales
// Blocks of 128 rows x 256 columns, all chunks of columns of a block of rows one
// after another; in a chunk 512-byte parts of four scale bytes along the row, in
// the order in which a copy to tensor memory lays 128 rows over 32 lanes and four
// 32-bit columns: row r's word at (r % 32) * 16 + (r / 32) * 4.
constexpr int kScaleRows = 128;
constexpr int kScaleCols = 256;
constexpr int kScalePart = 512;

__host__ __device__ constexpr int scale_chunk_bytes(int block) {
    return kScaleRows * kScaleCols / block;
}

// Bytes of the scales of one expert's [N, K] weights.
__host__ __device__ inline int64_t packed_scale_bytes(int64_t N, int64_t K, int block) {
    return (N + kScaleRows - 1) / kScaleRows * ((K + kScaleCols - 1) / kScaleCols) *
           scale_chunk_bytes(block);
}

// Offset of row r's scale c within them.
__device__ __forceinline__ int64_t packed_scale_at(int64_t r, int64_t c, int64_t K, int block) {
    const int64_t per = kScaleCols / block, chunks = (K + kScaleCols - 1) / kScaleCols;
    const int in_row = int(r % kScaleRows), in_chunk = int(c % per);
    return (r / kScaleRows * chunks + c / per) * scale_chunk_bytes(block) +
           in_chunk / 4 * kScalePart + in_row % 32 * 16 + in_row / 32 * 4 + in_chunk % 4;
}

}  // namespace moe
