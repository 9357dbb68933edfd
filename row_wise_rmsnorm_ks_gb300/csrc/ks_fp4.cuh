// Groups of 16 values held in 4 bits each with an 8-bit scale.
//
// A code is a sign and one of the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 (e2m1); value 2i of a group is the low half of
// byte i. A group's scale s is an e4m3 number, 0 .. 448, and the pool has a factor g. With A the group's largest
// magnitude:
//     s = A / (6 g) to the nearest, ties to the even code, at most 448
//     u = s g, rounded to FP32
//     code = x / u to the nearest, ties to the even code, at most 6 (0 where s is 0); its sign that of x, none for -0
// A group with a NaN has the scale NaN, and reads back as NaN.
//
// A code times a scale has at most 6 significant bits and lies in 2^-10 .. 2688: fp16 holds it exactly. The
// attention's products therefore take codes times scales as fp16 without a rounding, whatever the queries' type, and
// the factors in FP32 with the scores' scale and the output's: u's own rounding, 2^-24 with a factor that is no power of
// two, is not in them.
#pragma once

#include "ks_decode.cuh"
#include "ks_strided.h"

namespace ks {

// A pool as the kernels address it: bytes, strides in bytes.
struct Pool4 {
    uint8_t *codes, *scales;
    int64_t code_page, code_slot, code_head;
    int64_t scale_page, scale_slot, scale_head;
    float factor;
};

inline Pool4 pool4(const ks_pages_4bit_t &p) {
    return {(uint8_t *)p.codes, (uint8_t *)p.scales, p.code_page_stride, p.code_slot_stride, p.code_head_stride,
            p.scale_page_stride, p.scale_slot_stride, p.scale_head_stride, p.factor};
}

// A pool's codes, or its scales, for the checks of shared memory.
inline Strided strided4(const ks_pages_4bit_t &p, bool scales, int64_t pages, int64_t page_size, int64_t heads, int64_t dim) {
    if (scales)
        return {p.scales, dim / 16, {pages, page_size, heads}, {p.scale_page_stride, p.scale_slot_stride, p.scale_head_stride}};
    return {p.codes, dim / 2, {pages, page_size, heads}, {p.code_page_stride, p.code_slot_stride, p.code_head_stride}};
}

// What can be wrong with the two pools of a call, whose other sizes are checked; `written`: their rows have to be
// apart and the pools too. Sets the alignment of all code and scale addresses (the OR of them and the strides used).
ks_status_t check_pools4(const ks_pages_4bit_t &k, const ks_pages_4bit_t &v, int64_t pages, int64_t page_size,
                         int64_t heads, int64_t dim, bool written, uintptr_t *code_align, uintptr_t *scale_align);
// Whether n bytes from p, first to last, cross either pool.
bool crosses_pools4(const ks_pages_4bit_t &k, const ks_pages_4bit_t &v, int64_t pages, int64_t page_size, int64_t heads,
                    int64_t dim, const void *p, int64_t n);

// ---- reading

// The 8 codes of a word as fp16 pairs: pair i from byte i.
__device__ __forceinline__ void fp4_to_half(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

// Two scales (the low two bytes) as an fp16 pair.
__device__ __forceinline__ uint32_t e4m3_to_half(uint32_t bytes) {
    uint32_t h;
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(h) : "r"(bytes));
    return h;
}

__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
    const uint32_t h = e4m3_to_half(byte);
    __half2 x;
    memcpy(&x, &h, 4);
    return __low2float(x);
}

__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// ---- writing

// The code of two magnitudes, that of a in the low half of the byte.
__device__ __forceinline__ uint32_t fp4_codes(float a, float b) {
    uint32_t c;
    asm("{\n\t.reg .b8 x;\n\tcvt.rn.satfinite.e2m1x2.f32 x, %2, %1;\n\tcvt.u32.u8 %0, x;\n\t}" : "=r"(c) : "f"(a), "f"(b));
    return c;
}

// The codes of a (low byte) and b.
__device__ __forceinline__ uint32_t e4m3_codes(float a, float b) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(c) : "f"(a), "f"(b));
    return c;
}

__device__ __forceinline__ float fp4_magnitude(uint32_t code) {  // of a code without its sign
    return code < 2 ? 0.5f * (float)code : (code & 1 ? 1.5f : 1.0f) * (float)(1 << ((code >> 1) - 1));
}

// How a product compares with a value, its sign exactly: FP32 by the one rounding of a fused multiply-add, double
// because its factors have few bits (at most 7 and 24).
__device__ __forceinline__ float product_less(float a, float b, float x) { return __fmaf_rn(a, b, -x); }
__device__ __forceinline__ double product_less(float a, float b, double x) { return (double)a * (double)b - x; }

// The group's scale, given that the quotient A / (6 g) lies in [low, high], FP32 numbers whose codes are one or
// neighbours: then A itself decides.
template <typename F>
__device__ __forceinline__ uint32_t fp4_scale(float low, float high, F A, float g) {
    const uint32_t c = e4m3_codes(fminf(fmaxf(low, 0.0f), 512.0f), fminf(high, 512.0f));
    uint32_t lo = c & 0xFF;
    const uint32_t hi = c >> 8;
    if (lo != hi) {
        const float border = 0.5f * (e4m3_to_float(lo) + e4m3_to_float(hi));
        const auto d = product_less(border * 6.0f, g, A);  // < 0: A is above the border
        if (d < 0 || (d == 0 && (lo & 1))) lo = hi;
    }
    return lo;
}

// The code of x, given that |x| / u lies in [low, high] and their codes are neighbours or one.
template <typename F>
__device__ __forceinline__ uint32_t fp4_decide(uint32_t lo, uint32_t hi, F x, float u) {
    if (lo == hi) return lo;
    const auto d = product_less(0.5f * (fp4_magnitude(lo) + fp4_magnitude(hi)), u, x);
    return d < 0 || (d == 0 && (lo & 1)) ? hi : lo;
}

}  // namespace ks
