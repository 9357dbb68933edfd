// Rotary positions with the keys and values landing in a cache held in 4 bits (ks_rotary_to_pages_4bit), and the rows
// of such a cache read back (ks_pages_4bit_to_rows).
//
// Writing. CTAs (token, part): the first parts turn the token's queries as ks_rotary does, the last takes its keys and
// values, a thread per group of 16: it loads its group and, for a key, the group of its pairs' partners, turns in
// FP32, and finds the group's scale and codes. These are those of the real numbers: the angles have 64 bits, the
// turn's FP32 error is bounded by 2^-21 (|x| + |y|) |scale| for a pair (x, y), and where the scale or a code could
// differ within the bound (about one group in ten thousand; every tie of an unturned value) it is decided
// exactly, in double for turned values, by the sign of a fused multiply-add for the others.
//
// Bound by memory: the queries are read and written once, keys and values read once, 9/16 byte written for each.
#include <cuda_runtime.h>

#include "ks_rotary.cuh"

namespace ks {
namespace {

constexpr float kTurnError = 4.76837158203125e-07f;    // 2^-21
constexpr float kRoundError = 2.384185791015625e-07f;  // 2^-22: a quotient by two roundings, or three

struct Rotary4Args {
    RotaryArgs r;
    Pool4 k, v;
    int32_t q_parts;
};

struct Group4 {
    uint32_t scale, lo, hi;  // the scale's code, the codes of values 0 .. 7 and 8 .. 15
};

// The group of turned values in double, for those that FP32 does not decide.
template <typename T, bool kHalf>
__device__ __noinline__ Group4 group4_exact(const ks_rotary_args_t &a, const T *row, int group, uint64_t position, float g) {
    const int rot = (int)a.rotary_dim, half = rot / 2;
    double y[16], top = 0.0;
    for (int i = 0; i < 16; ++i) {
        const int d = group * 16 + i;
        double x = Elem<T>::load1(row, d);
        if (d < rot) {
            const int j = kHalf ? (d < half ? d : d - half) : d / 2;
            const bool second = kHalf ? d >= half : d & 1;
            const double z = Elem<T>::load1(row, kHalf ? (second ? d - half : d + half) : d ^ 1);
            double s, c;
            sincospi((double)(int64_t)(position * (uint64_t)a.steps[j]) * 1.0842021724855044e-19, &s, &c);  // 2^-63
            x = (second ? x * c + z * s : x * c - z * s) * (double)a.scale;
        }
        y[i] = x;
        top = fmax(top, fabs(x));
    }
    Group4 out = {0, 0, 0};
    const float v = (float)(top / (6.0 * (double)g));
    out.scale = fp4_scale(v * (1.0f - kRoundError), v * (1.0f + kRoundError), top, g);
    const float u = __fmul_rn(e4m3_to_float(out.scale), g);
    if (u > 0.0f)
        for (int i = 0; i < 16; ++i) {
            const double size = fabs(y[i]);
            const float t = fminf((float)(size / (double)u), 8.0f);
            const uint32_t c = fp4_codes(t * (1.0f - kRoundError), t * (1.0f + kRoundError));
            const uint32_t code = fp4_decide(c & 7, c >> 4 & 7, size, u) | (y[i] < 0.0 ? 8u : 0u);
            if (i < 8) out.lo |= code << (4 * i);
            else out.hi |= code << (4 * (i - 8));
        }
    return out;
}

// A group's values in FP32, off by at most error[i] (all 0: exact).
template <typename T, bool kHalf, bool kExact>
__device__ __forceinline__ Group4 group4(const ks_rotary_args_t &a, const T *row, int group, uint64_t position, float g,
                                         const float (&y)[16], const float (&error)[16]) {
    float top = 0.0f, off = 0.0f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        top = fmaxf(top, fabsf(y[i]));
        nan |= y[i] != y[i];
        if (!kExact) off = fmaxf(off, error[i]);
    }
    if (nan) return {0x7Fu, 0, 0};
    const float per = __frcp_rn(6.0f * g);
    const float low = (top - off) * per * (1.0f - 2 * kRoundError), high = (top + off) * per * (1.0f + 2 * kRoundError);
    if (!kExact) {
        const uint32_t c = e4m3_codes(fminf(fmaxf(low, 0.0f), 512.0f), fminf(high, 512.0f));
        if ((c & 0xFF) != c >> 8) return group4_exact<T, kHalf>(a, row, group, position, g);
    }
    Group4 out = {fp4_scale(low, high, top, g), 0, 0};
    const float u = __fmul_rn(e4m3_to_float(out.scale), g);
    if (!(u > 0.0f)) return out;
    const float inv = __frcp_rn(u);
    uint32_t lo[2] = {0, 0}, hi[2] = {0, 0}, sign[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        float t[2], w[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            t[k] = fminf(fabsf(y[i + k]) * inv, 8.0f);
            w[k] = t[k] * kRoundError;
            if (!kExact) w[k] = fmaf(error[i + k], inv, w[k]);
            if (y[i + k] < 0.0f) sign[i / 8] |= 8u << (4 * (i % 8 + k));
        }
        lo[i / 8] |= fp4_codes(fmaxf(t[0] - w[0], 0.0f), fmaxf(t[1] - w[1], 0.0f)) << (4 * (i % 8));
        hi[i / 8] |= fp4_codes(t[0] + w[0], t[1] + w[1]) << (4 * (i % 8));
    }
    if (lo[0] != hi[0] || lo[1] != hi[1]) {
        if constexpr (!kExact) {
            return group4_exact<T, kHalf>(a, row, group, position, g);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int at = 4 * (i % 8);
                const uint32_t l = lo[i / 8] >> at & 7, h = hi[i / 8] >> at & 7;
                if (l != h) lo[i / 8] ^= (l ^ fp4_decide(l, h, fabsf(y[i]), u)) << at;
            }
        }
    }
    out.lo = lo[0] | sign[0];
    out.hi = lo[1] | sign[1];
    return out;
}

template <typename T, bool kVec>
__device__ __forceinline__ void load16(const T *p, float (&x)[16]) {
    if constexpr (kVec) {
        constexpr int V = Elem<T>::kPerVec;
        uint4 v[16 / V];
#pragma unroll
        for (int i = 0; i < 16 / V; ++i) v[i] = reinterpret_cast<const uint4 *>(p)[i];
#pragma unroll
        for (int i = 0; i < 16 / V; ++i) {
            float f[V];
            Elem<T>::unpack(v[i], f);
#pragma unroll
            for (int k = 0; k < V; ++k) x[i * V + k] = f[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = Elem<T>::load1(p, i);
    }
}

template <typename T, bool kHalf, bool kVec>
__device__ __forceinline__ void pages4_groups(const Rotary4Args &args, int64_t token, int first, int step, float2 *cs) {
    const ks_rotary_args_t &a = args.r.a;
    const int groups = (int)a.head_dim / 16, rot = (int)a.rotary_dim, half = rot / 2;
    const RotToken t = rot_token<true>(a, token);
    rot_table(a, t, cs);
    __syncthreads();
    if (t.slot < 0) return;
    const int64_t page = quotient(t.slot, a.page_size), place = t.slot - page * a.page_size;
    if (page >= a.pages) {
        if (threadIdx.x == 0) atomicOr(&g_fault_flags, kFaultBadIndex);
        return;
    }
    const int total = (int)(2 * a.kv_heads * groups);
    for (int item = first + threadIdx.x; item < total; item += step) {
        const int row_index = item / groups, group = item - row_index * groups;
        const bool value = row_index >= a.kv_heads;
        const int64_t head = value ? row_index - a.kv_heads : row_index;
        const T *row = value ? (const T *)a.v + token * a.v_token_stride + head * a.v_head_stride
                             : (const T *)a.k + token * a.k_token_stride + head * a.k_head_stride;
        const Pool4 &pool = value ? args.v : args.k;
        float x[16];
        load16<T, kVec>(row + group * 16, x);
        Group4 out;
        const bool turned = !value && group * 16 < rot;
        if (!turned) {
            const float none[16] = {};
            out = group4<T, kHalf, true>(a, row, group, t.position, pool.factor, x, none);
        } else {
            float z[16], y[16], error[16];
            if (!kHalf) {
#pragma unroll
                for (int i = 0; i < 16; ++i) z[i] = x[i ^ 1];
            } else if (kVec) {
                load16<T, true>(row + (group * 16 < half ? group * 16 + half : group * 16 - half), z);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int d = group * 16 + i;
                    z[i] = d < rot ? Elem<T>::load1(row, d < half ? d + half : d - half) : 0.0f;
                }
            }
            const float size = fabsf(a.scale) * kTurnError;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int d = group * 16 + i;
                const bool second = kHalf ? d >= half : i & 1;
                y[i] = x[i];
                error[i] = 0.0f;
                if ((kHalf && kVec) || d < rot) {
                    const float2 turn = cs[kHalf ? (second ? d - half : d) : d / 2];
                    y[i] = fmaf(x[i], turn.x, second ? z[i] * turn.y : -z[i] * turn.y);
                    error[i] = (fabsf(x[i]) + fabsf(z[i])) * size;
                }
            }
            out = group4<T, kHalf, false>(a, row, group, t.position, pool.factor, y, error);
        }
        uint8_t *codes = pool.codes + page * pool.code_page + place * pool.code_slot + head * pool.code_head + group * 8;
        *reinterpret_cast<uint2 *>(codes) = make_uint2(out.lo, out.hi);
        pool.scales[page * pool.scale_page + place * pool.scale_slot + head * pool.scale_head + group] = (uint8_t)out.scale;
    }
}

template <typename T, bool kHalf, bool kVec>
__global__ void __launch_bounds__(kRotThreads) rotary_4bit_kernel(const __grid_constant__ Rotary4Args args) {
    __shared__ float2 cs[kRotMaxDim / 2];
    grid_dependency_wait();
    allow_dependents_launch();
    const int part = blockIdx.y;
    if (part < args.q_parts) {
        const int first = part * args.r.heads_per_y, last = min((int)args.r.a.q_heads, first + args.r.heads_per_y);
        if constexpr (kVec) rot_heads_vec<T, kHalf, false>(args.r, blockIdx.x, first, last, cs);
        else rot_heads_scalar<T, kHalf, false>(args.r, blockIdx.x, first, last, cs);
    } else {
        const int y = part - args.q_parts, parts = gridDim.y - args.q_parts;
        pages4_groups<T, kHalf, kVec>(args, blockIdx.x, y * blockDim.x, parts * blockDim.x, cs);
    }
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

constexpr int kRowsThreads = 256;
constexpr int kRowsEach = 4;  // tokens a thread has in flight

// A thread per group and four tokens: 9 bytes in, 16 values out. Bound by the rows that are written.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kRowsThreads) pages4_rows_kernel(const __grid_constant__ Rows4Args args) {
    grid_dependency_wait();
    allow_dependents_launch();
    const ks_pages_4bit_rows_args_t &a = args.a;
    const int groups = (int)a.head_dim / 16, total = (int)(2 * a.kv_heads * groups);
    const int lane = threadIdx.x % args.lanes, in_cta = threadIdx.x / args.lanes;
    if (in_cta >= args.tokens) return;
    const int64_t first = (int64_t)blockIdx.x * args.tokens * kRowsEach + in_cta;
    int64_t page[kRowsEach], place[kRowsEach];
#pragma unroll
    for (int u = 0; u < kRowsEach; ++u) {
        const int64_t token = first + u * args.tokens;
        const int64_t slot = token < a.tokens ? a.slots[token] : -1;
        page[u] = -1;
        place[u] = 0;
        if (slot < 0) continue;
        page[u] = quotient(slot, a.page_size);
        place[u] = slot - page[u] * a.page_size;
        if (page[u] >= a.pages) {
            atomicOr(&g_fault_flags, kFaultBadIndex);
            page[u] = -1;
        }
    }
    for (int item = lane; item < total; item += args.lanes) {
        const int row_index = item / groups, group = item - row_index * groups;
        const bool value = row_index >= a.kv_heads;
        const int64_t head = value ? row_index - a.kv_heads : row_index;
        const Pool4 &pool = value ? args.v : args.k;
        uint2 codes[kRowsEach];
        uint32_t scale[kRowsEach];
#pragma unroll
        for (int u = 0; u < kRowsEach; ++u) {
            codes[u] = make_uint2(0, 0);
            scale[u] = 0;
            if (page[u] < 0) continue;
            codes[u] = *reinterpret_cast<const uint2 *>(pool.codes + page[u] * pool.code_page + place[u] * pool.code_slot +
                                                        head * pool.code_head + group * 8);
            scale[u] = pool.scales[page[u] * pool.scale_page + place[u] * pool.scale_slot + head * pool.scale_head + group];
        }
#pragma unroll
        for (int u = 0; u < kRowsEach; ++u) {
            const int64_t token = first + u * args.tokens;
            if (token >= a.tokens) break;
            const float unit = __fmul_rn(e4m3_to_float(scale[u]), pool.factor);
            float f[16];
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                uint32_t h[4];
                fp4_to_half(w ? codes[u].y : codes[u].x, h);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    __half2 x;
                    memcpy(&x, &h[i], 4);
                    const float2 p = __half22float2(x);
                    f[8 * w + 2 * i] = p.x * unit;
                    f[8 * w + 2 * i + 1] = p.y * unit;
                }
            }
            T *dst = value ? (T *)a.v_out + token * a.v_token_stride + head * a.v_head_stride
                           : (T *)a.k_out + token * a.k_token_stride + head * a.k_head_stride;
            dst += group * 16;
            if constexpr (kVec) {
                constexpr int V = Elem<T>::kPerVec;
#pragma unroll
                for (int i = 0; i < 16 / V; ++i) {
                    float x[V];
#pragma unroll
                    for (int k = 0; k < V; ++k) x[k] = f[i * V + k];
                    reinterpret_cast<uint4 *>(dst)[i] = Elem<T>::pack(x);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) Elem<T>::store1(dst, i, f[i]);
            }
        }
    }
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
    const int64_t items = 2 * args.a.kv_heads * (args.a.head_dim / 16);
    // Few tokens: enough threads for all of a token's groups.
    int kv_parts = 1;
    if (args.a.tokens < 1024) kv_parts = (int)((items + threads - 1) / threads < 64 ? (items + threads - 1) / threads : 64);
    const void *f = args.a.dtype == KS_DTYPE_BF16  ? pick<__nv_bfloat16>(vec, half)
                    : args.a.dtype == KS_DTYPE_F16 ? pick<__half>(vec, half)
                                                   : pick<float>(vec, half);
    void *kp[] = {&k_args};
    return launch_kernel(f, dim3((unsigned)args.a.tokens, (unsigned)(parts + kv_parts)), dim3((unsigned)threads), 0, kp, stream,
                         launch_pdl_enabled());
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
    const int64_t items = 2 * a.kv_heads * (a.head_dim / 16);
    k_args.lanes = items < kRowsThreads ? (int32_t)items : kRowsThreads;
    k_args.tokens = kRowsThreads / k_args.lanes;
    const int64_t per_cta = (int64_t)k_args.tokens * kRowsEach;
    const bool vec = (align & 15u) == 0;
    const void *f;
    switch (a.dtype) {
    case KS_DTYPE_BF16: f = vec ? (const void *)pages4_rows_kernel<__nv_bfloat16, true> : (const void *)pages4_rows_kernel<__nv_bfloat16, false>; break;
    case KS_DTYPE_F16: f = vec ? (const void *)pages4_rows_kernel<__half, true> : (const void *)pages4_rows_kernel<__half, false>; break;
    default: f = vec ? (const void *)pages4_rows_kernel<float, true> : (const void *)pages4_rows_kernel<float, false>; break;
    }
    void *kp[] = {&k_args};
    const cudaError_t ce = launch_kernel(f, dim3((unsigned)((a.tokens + per_cta - 1) / per_cta)), dim3(kRowsThreads), 0, kp,
                                         static_cast<cudaStream_t>(stream), launch_pdl_enabled());
    if (ce != cudaSuccess) return fail(KS_ERR_CUDA, "launch: %s", cudaGetErrorString(ce));
    return KS_SUCCESS;
}
