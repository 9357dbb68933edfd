// Rotary positions with the keys and values landing in a cache held in 4 bits (ks_rotary_to_pages_4bit), and the rows
// of such a cache read back (ks_pages_4bit_to_rows).
//
// Writing. Some CTAs turn a token's queries as ks_rotary does, others take keys and values, a thread per group of 16: it
// loads its group and, for a key, the group of its pairs' partners, turns in FP32, and finds the group's scale and codes.
// These are those of the real numbers: the angles have 64 bits, the turn's FP32 error is bounded by
// 2^-21 (|x| + |y|) |scale| for a pair (x, y), and where the scale or a code could differ within the bound (about one
// group in five thousand; every tie of an unturned value) it is decided exactly, in double for turned values, by the sign
// of a fused multiply-add for the others.
//
// Bound by memory where there are many tokens: the queries are read and written once, keys and values read once, 9/16 byte
// written for each. Measured, 8192 tokens of 56 + 8 + 8 heads of 128, fp16, with the read-back: 84 us, 46 at the copy rate:
// 42 the queries (4.5 TB/s while the cache ends in L2), 30 the groups (issue: a quotient, two windows and their codes for each
// value; at 80 registers, three CTAs an SM, 24 to 156 bytes of them spill), 13 the read-back. 64 tokens with the read-back 8.4 us,
// two launches and a chain of loads each.
#include <cuda_runtime.h>

#include "ks_rotary.cuh"

namespace ks {
namespace {

constexpr float kTurnError = 4.76837158203125e-07f;    // 2^-21
constexpr float kRoundError = 2.384185791015625e-07f;  // 2^-22: a quotient by two roundings, or three

struct Rotary4Args {
    RotaryArgs r;
    Pool4 k, v;
    int32_t q_parts;                  // CTAs of a token's queries
    int32_t kv_tokens;                // tokens that a CTA of pages4_kernel takes
    Divisor per_head, per_token;      // groups of a head, and of a token's keys and values
};

struct Group4 {
    uint32_t scale, lo, hi;  // the scale's code, the codes of values 0 .. 7 and 8 .. 15
};

// Value d of a row, turned, in double: for what FP32 does not decide. (FP64 is slow here, a value takes about two
// microseconds; about one of 10^5 values asks for it.)
template <typename T, bool kHalf>
__device__ __noinline__ double turned_exact(const ks_rotary_args_t &a, const T *row, int d, uint64_t position) {
    const int rot = (int)a.rotary_dim, half = rot / 2;
    const double x = Elem<T>::load1(row, d);
    if (d >= rot) return x;
    const int j = kHalf ? (d < half ? d : d - half) : d / 2;
    const bool second = kHalf ? d >= half : d & 1;
    const double z = Elem<T>::load1(row, kHalf ? (second ? d - half : d + half) : d ^ 1);
    if (x == 0.0 && z == 0.0) return 0.0;  // rows may have many
    double s, c;
    sincospi((double)(int64_t)(position * (uint64_t)a.steps[j]) * 1.0842021724855044e-19, &s, &c);  // 2^-63
    return (second ? x * c + z * s : x * c - z * s) * (double)a.scale;
}

// NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float c;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
    return c;
}

// Codes of 8 signed quotients, value i in bits 4 i on.
__device__ __forceinline__ uint32_t fp4_word(const float2 *t) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(t[0].x), "f"(t[0].y), "f"(t[1].x), "f"(t[1].y), "f"(t[2].x), "f"(t[2].y), "f"(t[3].x), "f"(t[3].y));
    return w;
}

// 1 / x within 2^-23 of it: the windows of quotients have room for that.
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A group's values in FP32, each off by at most `off` (kExact: not at all). A quotient's code is taken at both ends
// of what it may be. A quotient's own error is at most 2^-23 + 2^-24 of it: for kExact both ends are multiples of it, of its
// sign (-0, which is not below 0, having been made +0). Otherwise the ends are a distance apart, the error being below
// 2^-19 of quotients below 10, and a zero's sign may be what is in doubt.
template <typename T, bool kHalf, bool kExact>
__device__ __forceinline__ Group4 group4(const ks_rotary_args_t &a, const T *row, int group, uint64_t position, float g,
                                         float2 (&y)[8], float off) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max_nan(top, max_nan(fabsf(y[i].x), fabsf(y[i].y)));
    if (top != top) return {0x7Fu, 0, 0};
    if constexpr (kExact) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fadd2_rn(y[i], make_float2(0.0f, 0.0f));
    }
    const float per = reciprocal(6.0f * g);
    const float low = (top - off) * per * (1.0f - 2 * kRoundError), high = (top + off) * per * (1.0f + 2 * kRoundError);
    Group4 out = {0, 0, 0};
    if constexpr (kExact) {
        out.scale = fp4_scale(low, high, top, g);
    } else {
        const uint32_t c = e4m3_codes(fminf(fmaxf(low, 0.0f), 512.0f), fminf(high, 512.0f));
        out.scale = c & 0xFF;
        if (out.scale != c >> 8) {
            // those that may be the largest, as a rule one
            uint32_t may = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (!(fabsf(i % 2 ? y[i / 2].y : y[i / 2].x) + off < top - off)) may |= 1u << i;
            double most = 0.0;
            for (; may; may &= may - 1)
                most = fmax(most, fabs(turned_exact<T, kHalf>(a, row, group * 16 + __ffs(may) - 1, position)));
            const float v = (float)(most / (6.0 * (double)g));
            out.scale = fp4_scale(v * (1.0f - kRoundError), v * (1.0f + kRoundError), most, g);
        }
    }
    const float u = __fmul_rn(e4m3_to_float(out.scale), g);
    if (!(u > 0.0f)) return out;
    const float inv = reciprocal(u);
    const float2 inv2 = make_float2(inv, inv);
    float2 t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = __fmul2_rn(y[i], inv2);
    if (out.scale == 126) {  // the largest: quotients may be of any size
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t[i].x = fminf(fmaxf(t[i].x, -8.0f), 8.0f);
            t[i].y = fminf(fmaxf(t[i].y, -8.0f), 8.0f);
        }
    }
    const float w = kExact ? 4.76837158203125e-07f : off * inv + 1.9073486328125e-06f;  // 2^-21, 2^-19
    const float2 more = kExact ? make_float2(1.0f + w, 1.0f + w) : make_float2(w, w);
    const float2 less = kExact ? make_float2(1.0f - w, 1.0f - w) : make_float2(-w, -w);
    uint32_t lo[2], hi[2];
    {
        float2 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = kExact ? __fmul2_rn(t[i], more) : __fadd2_rn(t[i], more);
        hi[0] = fp4_word(v), hi[1] = fp4_word(v + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = kExact ? __fmul2_rn(t[i], less) : __fadd2_rn(t[i], less);
        lo[0] = fp4_word(v), lo[1] = fp4_word(v + 4);
    }
    // (A window of infinite ends has no codes to compare.)
    const bool wide = !kExact && !(w < 0.125f);
    if (lo[0] != hi[0] || lo[1] != hi[1] || wide) {
        if constexpr (kExact) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int at = 4 * (i % 8);
                const uint32_t d = (lo[i / 8] ^ hi[i / 8]) >> at & 7;
                if (d) {
                    const float x = i % 2 ? y[i / 2].y : y[i / 2].x;
                    const uint32_t one = lo[i / 8] >> at & 7, other = one ^ d, small = min(one, other);
                    const uint32_t code = fp4_decide(small, small + 1, fabsf(x), u) | (x < 0.0f ? 8u : 0u);
                    lo[i / 8] = (lo[i / 8] & ~(15u << at)) | code << at;
                }
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < 16; ++i) {
                const int at = 4 * (i % 8);
                if (!wide && ((i < 8 ? lo[0] ^ hi[0] : lo[1] ^ hi[1]) >> at & 15) == 0) continue;
                const double x = turned_exact<T, kHalf>(a, row, group * 16 + i, position), size = fabs(x);
                // the window may be wider than two codes: of a group that its pairs all but cancel
                const float q = fminf((float)(size / (double)u), 8.0f);
                const uint32_t c = fp4_codes(q * (1.0f - kRoundError), q * (1.0f + kRoundError));
                const uint32_t code = fp4_decide(c & 7, c >> 4 & 7, size, u) | (x < 0.0 ? 8u : 0u);
                if (i < 8) lo[0] = (lo[0] & ~(15u << at)) | code << at;
                else lo[1] = (lo[1] & ~(15u << at)) | code << at;
            }
        }
    }
    out.lo = lo[0];
    out.hi = lo[1];
    return out;
}

template <typename T, bool kVec>
__device__ __forceinline__ void load16(const T *p, float2 (&x)[8]) {
    if constexpr (kVec) {
        constexpr int P = Elem<T>::kPerVec / 2;
        uint4 v[8 / P];
#pragma unroll
        for (int i = 0; i < 8 / P; ++i) v[i] = reinterpret_cast<const uint4 *>(p)[i];
#pragma unroll
        for (int i = 0; i < 8 / P; ++i) {
            float2 f[P];
            Elem<T>::unpack2(v[i], f);
#pragma unroll
            for (int k = 0; k < P; ++k) x[i * P + k] = f[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = make_float2(Elem<T>::load1(p, 2 * i), Elem<T>::load1(p, 2 * i + 1));
    }
}

// Cosines and sines for the groups, apart, 4 places free behind every 16: eight lanes with a group each read 16 bytes
// of theirs without a conflict.
constexpr int kTable = kRotMaxDim / 2 / 16 * 20;
__device__ __forceinline__ int table_at(int j) { return j + (j >> 4) * 4; }
__device__ __forceinline__ float2 pair_at(const float *table, int i) { return *reinterpret_cast<const float2 *>(table + i); }

constexpr int kMostTokens = 4;  // whose groups a CTA takes

// Where a token's rows go, and what it is turned by.
struct Place4 {
    int64_t k_codes, k_scales, v_codes, v_scales;  // k_codes -1: nowhere
    uint64_t position;  // negated where the turn is the inverse one
};

// A CTA's part of the groups of `tokens` tokens from `first` on, a thread a group. Rows are asked for before all else.
template <typename T, bool kHalf, bool kVec>
__device__ __forceinline__ void pages4_groups(const Rotary4Args &args, int64_t first, int tokens, int part, int parts, float *cosines,
                                              float *sines, Place4 *places) {
    const ks_rotary_args_t &a = args.r.a;
    const int rot = (int)a.rotary_dim, half = rot / 2, groups = (int)a.head_dim / 16;
    const int per_token = (int)(2 * a.kv_heads) * groups, total = tokens * per_token;
    struct Item {
        float2 x[8], z[8];  // the group, and (kHalf && kVec) its pairs' partners
    };
    struct Which {
        int of, group, head;
        bool value, turned;
        const T *row;
    };
    // Angles are a multiple of the position, so the inverse turn is that by the position negated, exactly.
    const bool inverse = (a.flags & KS_ROTARY_INVERSE) != 0;
    auto position = [&](int of) {
        const uint64_t at = (uint64_t)a.positions[first + of];
        return inverse ? 0 - at : at;
    };
    auto which = [&](int item) {
        Which w;
        w.of = (int)args.per_token.quotient((uint32_t)item);
        const int in = item - w.of * per_token, r = (int)args.per_head.quotient((uint32_t)in);
        w.group = in - r * groups;
        w.value = r >= a.kv_heads;
        w.head = w.value ? r - (int)a.kv_heads : r;
        w.turned = !w.value && w.group * 16 < rot;
        w.row = w.value ? (const T *)a.v + (first + w.of) * a.v_token_stride + w.head * a.v_head_stride
                        : (const T *)a.k + (first + w.of) * a.k_token_stride + w.head * a.k_head_stride;
        return w;
    };
    auto load = [&](const Which &w, Item &it) {
        load16<T, kVec>(w.row + w.group * 16, it.x);
        if (kHalf && kVec && w.turned) load16<T, true>(w.row + (w.group * 16 >= half ? w.group * 16 - half : w.group * 16 + half), it.z);
    };
    int item = part * blockDim.x + threadIdx.x;
    Which w = which(item < total ? item : 0);
    Item it;
    if (item < total) load(w, it);
    for (int i = threadIdx.x; i < tokens; i += blockDim.x) {
        const int64_t slot = a.slots[first + i];
        Place4 p = {-1, 0, 0, 0, rot > 0 ? position(i) : 0};
        if (slot >= 0) {
            const int64_t page = quotient(slot, a.page_size), place = slot - page * a.page_size;
            if (page < a.pages) {
                p.k_codes = page * args.k.code_page + place * args.k.code_slot;
                p.k_scales = page * args.k.scale_page + place * args.k.scale_slot;
                p.v_codes = page * args.v.code_page + place * args.v.code_slot;
                p.v_scales = page * args.v.scale_page + place * args.v.scale_slot;
            } else {
                atomicOr(&g_fault_flags, kFaultBadIndex);
            }
        }
        places[i] = p;
    }
    for (int i = threadIdx.x; i < tokens * half; i += blockDim.x) {
        const int of = i / half, j = i - of * half;
        const float2 c = turn_cos_sin(position(of) * (uint64_t)a.steps[j], a.scale);
        cosines[table_at(i)] = c.x;
        sines[table_at(i)] = c.y;
    }
    __syncthreads();
    while (item < total) {
        const int next = item + parts * blockDim.x;
        const Which now = w;
        Item cur = it;
        if (next < total) {
            w = which(next);
            load(w, it);
        }
        item = next;
        const Place4 &p = places[now.of];
        if (p.k_codes < 0) continue;
        const Pool4 &pool = now.value ? args.v : args.k;
        Group4 out;
        if (!now.turned) {
            out = group4<T, kHalf, true>(a, now.row, now.group, p.position, pool.factor, cur.x, 0.0f);
        } else {
            float2 y[8];
            float size = 0.0f;  // the largest |x| + |y| of the group's pairs
            if constexpr (kHalf && kVec) {
                const bool second = now.group * 16 >= half;
                const int j = table_at(now.of * half + (second ? now.group * 16 - half : now.group * 16));
                const float2 sign = make_float2(second ? 1.0f : -1.0f, second ? 1.0f : -1.0f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 x = cur.x[i], z = cur.z[i];
                    size = fmaxf(size, fmaxf(fabsf(x.x) + fabsf(z.x), fabsf(x.y) + fabsf(z.y)));
                    y[i] = __ffma2_rn(x, pair_at(cosines, j + 2 * i), __fmul2_rn(__fmul2_rn(z, pair_at(sines, j + 2 * i)), sign));
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int d = now.group * 16 + i;
                    float &to = i % 2 ? y[i / 2].y : y[i / 2].x;
                    const float m = i % 2 ? cur.x[i / 2].y : cur.x[i / 2].x;
                    to = m;
                    if (d < rot) {
                        const bool second = kHalf ? d >= half : i & 1;
                        const int j = table_at(now.of * half + (kHalf ? (second ? d - half : d) : d / 2));
                        const float z = kHalf ? Elem<T>::load1(now.row, second ? d - half : d + half)
                                              : i % 2 ? cur.x[i / 2].x : cur.x[i / 2].y;
                        to = fmaf(m, cosines[j], second ? z * sines[j] : -z * sines[j]);
                        size = fmaxf(size, fabsf(m) + fabsf(z));
                    }
                }
            }
            out = group4<T, kHalf, false>(a, now.row, now.group, p.position, pool.factor, y, size * (fabsf(a.scale) * kTurnError));
        }
        *reinterpret_cast<uint2 *>(pool.codes + (now.value ? p.v_codes : p.k_codes) + now.head * pool.code_head + now.group * 8) =
            make_uint2(out.lo, out.hi);
        pool.scales[(now.value ? p.v_scales : p.k_scales) + now.head * pool.scale_head + now.group] = (uint8_t)out.scale;
    }
}

// Few tokens: CTAs (token, part), the first parts for the queries, the others for the groups.
template <typename T, bool kHalf, bool kVec>
__global__ void __launch_bounds__(kRotThreads) rotary_4bit_kernel(const __grid_constant__ Rotary4Args args) {
    __shared__ __align__(16) float tables[2 * kTable];
    __shared__ Place4 places[kMostTokens];
    static_assert(sizeof(tables) >= kRotMaxDim / 2 * sizeof(float2), "the queries' table fits");
    float2 *cs = reinterpret_cast<float2 *>(tables);
    grid_dependency_wait();
    allow_dependents_launch();
    const int part = blockIdx.y;
    if (part < args.q_parts) {
        const int first = part * args.r.heads_per_y, last = min((int)args.r.a.q_heads, first + args.r.heads_per_y);
        if constexpr (kVec) rot_heads_vec<T, kHalf, false>(args.r, blockIdx.x, first, last, cs);
        else rot_heads_scalar<T, kHalf, false>(args.r, blockIdx.x, first, last, cs);
    } else {
        pages4_groups<T, kHalf, kVec>(args, blockIdx.x, 1, part - args.q_parts, gridDim.y - args.q_parts, tables, tables + kTable, places);
    }
}

// Many tokens: the queries are ks_rotary's kernel, the groups this one, for kv_tokens tokens a CTA. (Both in one kernel
// have its registers in common: measured at 8192 tokens of 56 + 8 + 8 heads, 88 us and more for 42 and 29.) It is
// launched to start while the queries' last CTAs run: those began after all earlier work was done, and of their own
// they write nothing that is read here. It ends after them. (`alone`: without queries, or where the queries' kernel may
// itself start before earlier work's end, it waits at its beginning.) Taken from 1024 tokens on. (Measured with cold caches, us, one
// kernel and two, at 512, 1024 and 2048 tokens, bf16: 32 + 8 + 8 heads of 128 18.6, 27.8, 44.3 and 18.8, 21.6, 30.9; 0 + 8 + 8 15.5,
// 22.2, 32.4 and 15.0, 16.0, 22.6; 8 + 1 + 1 12.4, 14.5, 19.6 and 13.4, 15.5, 18.5; 16 + 16 + 16 of 64 13.5, 15.5, 21.7 and 15.5, 17.5,
// 23.7, equal at 1536.)
template <typename T, bool kHalf, bool kVec>
__global__ void __launch_bounds__(kRotThreads, 3) pages4_kernel(const __grid_constant__ Rotary4Args args, int alone) {
    __shared__ __align__(16) float tables[2 * kTable];
    __shared__ Place4 places[kMostTokens];
    if (alone) grid_dependency_wait();
    const int64_t first = (int64_t)blockIdx.x * args.kv_tokens;
    pages4_groups<T, kHalf, kVec>(args, first, (int)min((int64_t)args.kv_tokens, args.r.a.tokens - first), 0, 1, tables,
                                  tables + kTable, places);
    if (!alone) grid_dependency_wait();
    else allow_dependents_launch();
}

template <typename T>
const void *pick_groups(bool vec, bool half) {
    if (vec) return half ? (const void *)pages4_kernel<T, true, true> : (const void *)pages4_kernel<T, false, true>;
    return half ? (const void *)pages4_kernel<T, true, false> : (const void *)pages4_kernel<T, false, false>;
}

template <typename T>
const void *pick(bool vec, bool half) {
    if (vec) return half ? (const void *)rotary_4bit_kernel<T, true, true> : (const void *)rotary_4bit_kernel<T, false, true>;
    return half ? (const void *)rotary_4bit_kernel<T, true, false> : (const void *)rotary_4bit_kernel<T, false, false>;
}

// ------------------------------------------------------------------------------- reading back

struct Rows4Args {
    ks_pages_4bit_rows_args_t a;
    Pool4 k, v;
    int32_t lanes;   // threads per token
    int32_t tokens;  // tokens at once in a CTA
};

// Whether a product of u and a code, rounded to FP32, may look like a tie of a 16-bit type without being one. Codes are 1 or
// 1.5 times a power of two, and a tie's last 12 bits are 0 (fp16's; 15 for bf16, more for subnormal numbers).
__device__ __forceinline__ bool twice_rounded(float u) {
    const float p = __fmul_rn(u, 1.5f);
    return (__float_as_uint(p) & 0xFFFu) == 0 && __fmaf_rn(u, 1.5f, -p) != 0.0f;
}

// u times a code for a 16-bit type: where FP32 does not hold it, FP32's neighbour towards 0 with its last bit set, which no
// later rounding takes for a tie or for a number of that type. (A product has at most 26 bits: 24 of u, which is s times a
// factor of any bits, and 2 of the code.)
__device__ __forceinline__ float times_odd(float code, float u) {
    const float p = __fmul_rz(code, u);
    return __uint_as_float(__float_as_uint(p) | (__fmaf_rn(code, u, -p) != 0.0f ? 1u : 0u));
}

constexpr int kRowsThreads = 256;
constexpr int kRowsEach = 8;  // tokens that a thread has in flight

// A thread per some values of a group and some tokens. Bound by the rows that are written: so where a token's rows lie in
// the pools is found once per token, in shared memory, and a group's FP32 unit multiplies its values two at a time; and a
// thread makes one 16-byte store of a row where the rows allow it, so that a warp's store is 512 bytes on end. (Measured,
// 131001 tokens of 8 + 8 heads of 128 to bf16: 113 us, 102 us at the copy rate; 138 with a group,
// two stores, a thread; 131 with four tokens a thread or with six CTAs an SM, 120 with four. Five leave 48 registers, of which
// 24 to 44 bytes a thread spill.)
// kOdd: a factor has more than 18 bits, u then more than 22, and FP32 may round a product that its type rounds again: looked at
// once a group, and one group in some thousands has its products rounded to odd first (factor 0.3: 116 us without, 120 with,
// 140 with every product rounded to odd; a factor of 1 would take 118 to 120 here).
template <typename T, bool kVec, bool kOdd>
__global__ void __launch_bounds__(kRowsThreads, 5) pages4_rows_kernel(const __grid_constant__ Rows4Args args) {
    constexpr int kVals = kVec ? 16 / (int)sizeof(T) : 16, kParts = 16 / kVals;
    extern __shared__ __align__(16) int64_t at_token[][4];  // k's codes and scales, v's; -1: nowhere
    grid_dependency_wait();
    allow_dependents_launch();
    const ks_pages_4bit_rows_args_t &a = args.a;
    const int per_cta = args.tokens * kRowsEach;
    const int64_t first = (int64_t)blockIdx.x * per_cta;
    for (int i = threadIdx.x; i < per_cta; i += kRowsThreads) {
        const int64_t slot = first + i < a.tokens ? a.slots[first + i] : -1;
        at_token[i][0] = -1;
        if (slot < 0) continue;
        const int64_t page = quotient(slot, a.page_size), place = slot - page * a.page_size;
        if (page >= a.pages) {
            atomicOr(&g_fault_flags, kFaultBadIndex);
            continue;
        }
        at_token[i][0] = page * args.k.code_page + place * args.k.code_slot;
        at_token[i][1] = page * args.k.scale_page + place * args.k.scale_slot;
        at_token[i][2] = page * args.v.code_page + place * args.v.code_slot;
        at_token[i][3] = page * args.v.scale_page + place * args.v.scale_slot;
    }
    __syncthreads();
    const int parts = (int)a.head_dim / kVals, total = (int)(2 * a.kv_heads * parts);
    const int lane = threadIdx.x % args.lanes, in_cta = threadIdx.x / args.lanes;
    if (in_cta >= args.tokens) return;
    for (int item = lane; item < total; item += args.lanes) {
        const int row_index = item / parts, part = item - row_index * parts;
        const bool value = row_index >= a.kv_heads;
        const int64_t head = value ? row_index - a.kv_heads : row_index;
        const Pool4 &pool = value ? args.v : args.k;
        const uint8_t *from_codes = pool.codes + head * pool.code_head + part * (kVals / 2);
        const uint8_t *from_scales = pool.scales + head * pool.scale_head + part / kParts;
        const int64_t stride = value ? a.v_token_stride : a.k_token_stride;
        T *dst = (value ? (T *)a.v_out + head * a.v_head_stride : (T *)a.k_out + head * a.k_head_stride) + part * kVals +
                 (first + in_cta) * stride;
        uint2 codes[kRowsEach];
        uint32_t scale[kRowsEach];
#pragma unroll
        for (int u = 0; u < kRowsEach; ++u) {
            const int i = in_cta + u * args.tokens;
            codes[u] = make_uint2(0, 0);
            scale[u] = 0;
            if (at_token[i][0] < 0) continue;
            const uint8_t *p = from_codes + at_token[i][value ? 2 : 0];
            if constexpr (kVals == 16) codes[u] = __ldg(reinterpret_cast<const uint2 *>(p));
            else if constexpr (kVals == 8) codes[u].x = __ldg(reinterpret_cast<const uint32_t *>(p));
            else codes[u].x = __ldg(reinterpret_cast<const uint16_t *>(p));
            scale[u] = __ldg(from_scales + at_token[i][value ? 3 : 1]);
        }
#pragma unroll
        for (int u = 0; u < kRowsEach; ++u) {
            if (first + in_cta + u * args.tokens >= a.tokens) break;
            const float unit = __fmul_rn(e4m3_to_float(scale[u]), pool.factor);
            const float2 units = make_float2(unit, unit);
            float2 f[kVals / 2];
            auto values = [&](auto times) {
#pragma unroll
                for (int w = 0; w < (kVals + 7) / 8; ++w) {
                    uint32_t h[4];
                    fp4_to_half(w ? codes[u].y : codes[u].x, h);
#pragma unroll
                    for (int i = 0; i < 4 && 4 * w + i < kVals / 2; ++i) {
                        __half2 x;
                        memcpy(&x, &h[i], 4);
                        f[4 * w + i] = times(__half22float2(x));
                    }
                }
            };
            if (kOdd && twice_rounded(unit)) values([&](float2 x) { return make_float2(times_odd(x.x, unit), times_odd(x.y, unit)); });
            else values([&](float2 x) { return __fmul2_rn(x, units); });
            T *to = dst + u * args.tokens * stride;
            if constexpr (kVec) {
                __stcs(reinterpret_cast<uint4 *>(to), Elem<T>::pack2(f));
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) Elem<T>::store1(to, i, i % 2 ? f[i / 2].y : f[i / 2].x);
            }
        }
    }
}

template <typename T>
const void *pick_rows(bool vec, bool odd) {
    if (vec) return odd ? (const void *)pages4_rows_kernel<T, true, true> : (const void *)pages4_rows_kernel<T, true, false>;
    return odd ? (const void *)pages4_rows_kernel<T, false, true> : (const void *)pages4_rows_kernel<T, false, false>;
}

// Strides whose product with their count, and a factor, that the kernels' arithmetic holds.
bool pool4_fits(const ks_pages_4bit_t &p, int64_t pages, int64_t page_size, int64_t heads) {
    const int64_t strides[6] = {p.code_page_stride, p.code_slot_stride, p.code_head_stride,
                                p.scale_page_stride, p.scale_slot_stride, p.scale_head_stride};
    const int64_t counts[3] = {pages, page_size, heads};
    for (int i = 0; i < 6; ++i)
        if (strides[i] < 0 || (__int128)strides[i] * counts[i % 3] > ((__int128)1 << 60)) return false;
    return true;
}

int64_t span4(const Strided &v) { return strided_span(v, StridedOrder(v, v)); }

}  // namespace

ks_status_t check_pools4(const ks_pages_4bit_t &k, const ks_pages_4bit_t &v, int64_t pages, int64_t page_size,
                         int64_t heads, int64_t dim, bool written, uintptr_t *code_align, uintptr_t *scale_align) {
    const ks_pages_4bit_t *pools[2] = {&k, &v};
    *code_align = *scale_align = 0;
    for (const ks_pages_4bit_t *p : pools)
        if (!(p->factor >= 5.421010862427522e-20f && p->factor <= 1.8446744073709552e19f))
            return fail(KS_ERR_INVALID_ARGUMENT, "a pool's factor must be in 2^-64 .. 2^64 (got %g)", (double)p->factor);
    if (pages <= 0) return KS_SUCCESS;
    Strided all[4];
    for (int i = 0; i < 2; ++i) {
        const ks_pages_4bit_t &p = *pools[i];
        if (!p.codes || !p.scales) return fail(KS_ERR_INVALID_ARGUMENT, "NULL codes or scales");
        if (!pool4_fits(p, pages, page_size, heads))
            return fail(KS_ERR_INVALID_ARGUMENT, "a pool's strides are negative or it is too large");
        all[2 * i] = strided4(p, false, pages, page_size, heads, dim);
        all[2 * i + 1] = strided4(p, true, pages, page_size, heads, dim);
        *code_align |= (uintptr_t)p.codes;
        *scale_align |= (uintptr_t)p.scales;
        for (int s = 0; s < 3; ++s) {
            *code_align |= (uintptr_t)all[2 * i].step(s);
            *scale_align |= (uintptr_t)all[2 * i + 1].step(s);
        }
    }
    if (*code_align & 7u)
        return fail(KS_ERR_INVALID_ARGUMENT, "codes must be aligned to 8 bytes, their strides multiples of 8");
    if (written)
        for (int i = 0; i < 4; ++i) {
            if (!strided_rows_apart(all[i])) return fail(KS_ERR_OVERLAP, "rows of a pool share storage");
            for (int j = 0; j < i; ++j)
                if (strided_cross(all[i], all[j])) return fail(KS_ERR_OVERLAP, "the pools' codes and scales share storage");
        }
    return KS_SUCCESS;
}

bool crosses_pools4(const ks_pages_4bit_t &k, const ks_pages_4bit_t &v, int64_t pages, int64_t page_size, int64_t heads,
                    int64_t dim, const void *p, int64_t n) {
    if (pages <= 0) return false;
    for (const ks_pages_4bit_t *pool : {&k, &v})
        for (int part = 0; part < 2; ++part) {
            const Strided s = strided4(*pool, part != 0, pages, page_size, heads, dim);
            if (overlaps(s.p, span4(s), p, n)) return true;
        }
    return false;
}

cudaError_t rotary_4bit_launch(const RotaryArgs &args, const ks_rotary_4bit_args_t &four, bool vec, bool half, int parts,
                               int threads, cudaStream_t stream) {
    Rotary4Args k_args;
    k_args.r = args;
    k_args.k = pool4(four.k_pages);
    k_args.v = pool4(four.v_pages);
    k_args.q_parts = parts;
    const int64_t groups = args.a.head_dim / 16, items = 2 * args.a.kv_heads * groups, half_dim = args.a.rotary_dim / 2;
    k_args.per_head = Divisor::of((uint32_t)groups);
    k_args.per_token = Divisor::of((uint32_t)items);
    k_args.kv_tokens = 1;
    const int dtype = args.a.dtype;
    if (parts <= 1 && args.a.tokens >= 1024) {
        // as many tokens a CTA as have their sines fit its tables
        k_args.kv_tokens = kMostTokens;
        while (k_args.kv_tokens > 1 && k_args.kv_tokens * half_dim > kRotMaxDim / 2) --k_args.kv_tokens;
        const bool queries = parts > 0;
        int alone = !queries || launch_pdl_enabled();
        if (queries) {
            const cudaError_t ce = rotary_queries_launch(args, vec, half, threads, stream);
            if (ce != cudaSuccess) return ce;
        }
        const void *f = dtype == KS_DTYPE_BF16  ? pick_groups<__nv_bfloat16>(vec, half)
                        : dtype == KS_DTYPE_F16 ? pick_groups<__half>(vec, half)
                                                : pick_groups<float>(vec, half);
        void *kp[] = {&k_args, &alone};
        return launch_kernel(f, dim3((unsigned)((args.a.tokens + k_args.kv_tokens - 1) / k_args.kv_tokens)), dim3(kRotThreads), 0, kp,
                             stream, queries || launch_pdl_enabled());
    }
    const int64_t most = (items + threads - 1) / threads;
    const void *f = dtype == KS_DTYPE_BF16  ? pick<__nv_bfloat16>(vec, half)
                    : dtype == KS_DTYPE_F16 ? pick<__half>(vec, half)
                                            : pick<float>(vec, half);
    void *kp[] = {&k_args};
    return launch_kernel(f, dim3((unsigned)args.a.tokens, (unsigned)(parts + (most < 64 ? most : 64))), dim3((unsigned)threads), 0, kp,
                         stream, launch_pdl_enabled());
}

int fault_flags_rotary_4bit(bool clear) { return fault_flags_t(clear); }

}  // namespace ks

using namespace ks;

extern "C" ks_status_t ks_pages_4bit_to_rows(const ks_pages_4bit_rows_args_t *args, ks_stream_t stream) {
    if (!args) return fail(KS_ERR_INVALID_ARGUMENT, "args is NULL");
    const ks_pages_4bit_rows_args_t &a = *args;
    const int e = elem_bytes((ks_dtype_t)a.dtype);
    if (e == 0) return fail(KS_ERR_UNSUPPORTED_DTYPE, "dtype code %d is not a ks_dtype_t", (int)a.dtype);
    if (a.tokens < 0 || a.tokens > 0x7fffffff)
        return fail(KS_ERR_INVALID_ARGUMENT, "tokens must be in 0 .. 2^31-1 (got %lld)", (long long)a.tokens);
    if (a.head_dim < 16 || a.head_dim > kRotMaxDim || a.head_dim % 16)
        return fail(KS_ERR_INVALID_ARGUMENT, "head_dim must be a multiple of 16 in 16 .. %d (got %lld)", kRotMaxDim, (long long)a.head_dim);
    if (a.kv_heads < 1 || a.kv_heads > 65536 || a.page_size < 1 || a.pages < 0)
        return fail(KS_ERR_INVALID_ARGUMENT, "a cache needs kv_heads in 1 .. 65536, page_size >= 1 and pages >= 0");
    if (a.tokens == 0) return KS_SUCCESS;
    if (!a.k_out || !a.v_out || !a.slots) return fail(KS_ERR_INVALID_ARGUMENT, "NULL pointer with tokens > 0");
    if (misaligned(e, a.k_out, a.v_out) || misaligned(8, a.slots))
        return fail(KS_ERR_INVALID_ARGUMENT, "outputs must be aligned to the element, slots to 8 bytes");
    uintptr_t code_align, scale_align;
    ks_status_t st = check_pools4(a.k_pages, a.v_pages, a.pages, a.page_size, a.kv_heads, a.head_dim, false, &code_align, &scale_align);
    if (st != KS_SUCCESS) return st;
    Strided out[2];
    uintptr_t align = 0;
    for (int i = 0; i < 2; ++i) {
        const int64_t token = i ? a.v_token_stride : a.k_token_stride, head = i ? a.v_head_stride : a.k_head_stride;
        if (token < 0 || head < 0 || ((__int128)a.tokens * token + (__int128)a.kv_heads * head + a.head_dim) * e > ((__int128)1 << 60))
            return fail(KS_ERR_INVALID_ARGUMENT, "a stride is negative or a tensor too large");
        out[i] = {i ? a.v_out : a.k_out, a.head_dim * e, {a.tokens, a.kv_heads, 1}, {token * e, head * e, 0}};
        if (!strided_rows_apart(out[i])) return fail(KS_ERR_OVERLAP, "rows of an output share storage");
        if (crosses_pools4(a.k_pages, a.v_pages, a.pages, a.page_size, a.kv_heads, a.head_dim, out[i].p, span4(out[i])))
            return fail(KS_ERR_OVERLAP, "an output overlaps the cache");
        if (strided_cross(out[i], {a.slots, a.tokens * 8, {1, 1, 1}, {0, 0, 0}}))
            return fail(KS_ERR_OVERLAP, "an output overlaps slots");
        align |= (uintptr_t)out[i].p | (uintptr_t)out[i].step(0) | (uintptr_t)out[i].step(1);
    }
    if (strided_cross(out[0], out[1])) return fail(KS_ERR_OVERLAP, "k_out and v_out storage overlap");
    Rows4Args k_args;
    k_args.a = a;
    k_args.k = pool4(a.k_pages);
    k_args.v = pool4(a.v_pages);
    const bool vec = (align & 15u) == 0;
    const int64_t items = 2 * a.kv_heads * (a.head_dim / (vec ? 16 / e : 16));
    k_args.lanes = items < kRowsThreads ? (int32_t)items : kRowsThreads;
    k_args.tokens = kRowsThreads / k_args.lanes;
    const int64_t per_cta = (int64_t)k_args.tokens * kRowsEach;
    auto bits = [](float factor) {  // up to 18 of a number's 24 bits: the last 6 are 0
        uint32_t w;
        memcpy(&w, &factor, 4);
        return w;
    };
    const bool odd = ((bits(a.k_pages.factor) | bits(a.v_pages.factor)) & 63u) != 0;
    const void *f = a.dtype == KS_DTYPE_BF16  ? pick_rows<__nv_bfloat16>(vec, odd)
                    : a.dtype == KS_DTYPE_F16 ? pick_rows<__half>(vec, odd)
                    : vec                     ? (const void *)pages4_rows_kernel<float, true, false>
                                              : (const void *)pages4_rows_kernel<float, false, false>;
    void *kp[] = {&k_args};
    const cudaError_t ce = launch_kernel(f, dim3((unsigned)((a.tokens + per_cta - 1) / per_cta)), dim3(kRowsThreads),
                                         (size_t)per_cta * 32, kp, static_cast<cudaStream_t>(stream), launch_pdl_enabled());
    if (ce != cudaSuccess) return fail(KS_ERR_CUDA, "launch: %s", cudaGetErrorString(ce));
    return KS_SUCCESS;
}
