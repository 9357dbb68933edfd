// Rotary positions, plain (ks_rotary) or with the key and value rows landing in their slots of a
// paged cache (ks_rotary_to_pages).
//
// Mathematics. Pair j of a head is rotated by the angle position * f_j. The frequency comes as a
// 64-bit fixed-point fraction of a turn, step_j = f_j / (2 pi) * 2^64, so position * step_j
// mod 2^64 is the angle's fraction of a turn with no range reduction to get wrong: the integer
// product wraps exactly, and the only error is step_j's own rounding times the position. The top
// 32 bits give the quadrant and a remainder of at most an eighth of a turn, whose sine and cosine
// (sincospif) carry FP32 accuracy; an FP32 product position * f_j would be off by 0.03 radians at
// position 2^19. The rotation runs in FP32 and is rounded once.
//
// Layout. A CTA takes one token (and, where there are fewer tokens than SMs, a part of its heads):
// its threads first issue every load that does not hang on another (position, slot, step and their
// first vectors), then compute the token's rotary_dim/2 sines and cosines once into shared memory,
// then rotate every head with them. A thread keeps one
// column of the head (a 16-byte vector, or the two vectors of a half-split pair), so no index
// division is left in the loop. Bound by memory: each value is read once and written once. Measured:
// bf16, 16384 tokens of 64 + 8 heads of 128, 87 us or 6.9 TB/s; into the cache, fp16, 8192 tokens of
// 56 + 8 + 8 heads, 49 us or 6.2 TB/s.
#include <cuda_runtime.h>

#include <cmath>

#include "ks_rotary.cuh"
#include "ks_strided.h"

namespace ks {
namespace {

template <typename T, bool kHalf, bool kPages, bool kVec>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotaryArgs args) {
    __shared__ float2 cs[kRotMaxDim / 2];
    const ks_rotary_args_t &a = args.a;
    grid_dependency_wait();
    allow_dependents_launch();
    const int total = (int)(a.q_heads + a.kv_heads * (kPages ? 2 : 1));
    const int first = blockIdx.y * args.heads_per_y;
    const int last = min(total, first + args.heads_per_y);
    if constexpr (kVec) rot_heads_vec<T, kHalf, kPages>(args, blockIdx.x, first, last, cs);
    else rot_heads_scalar<T, kHalf, kPages>(args, blockIdx.x, first, last, cs);
}

template <typename T, bool kPages>
const void *rotary_pick(bool vec, bool half) {
    if (vec) return half ? (const void *)rotary_kernel<T, true, kPages, true>
                         : (const void *)rotary_kernel<T, false, kPages, true>;
    return half ? (const void *)rotary_kernel<T, true, kPages, false>
                : (const void *)rotary_kernel<T, false, kPages, false>;
}

// One packed tensor [tokens, heads, head_dim]: what the host checks need of it.
struct View {
    const void *p;
    int64_t token, head, heads;
};

// Bytes from the view's first to past its last element, and whether it lies within int64.
bool view_span(const View &v, int64_t tokens, int64_t dim, int e, int64_t *span) {
    if (v.token < 0 || v.head < 0) return false;
    const __int128 last = (__int128)(tokens - 1) * v.token + (__int128)(v.heads - 1) * v.head + dim;
    if (last * e > ((__int128)1 << 62)) return false;
    *span = (int64_t)last * e;
    return true;
}

Strided strided(const View &v, int64_t tokens, int64_t dim, int e) {
    return {v.p, dim * e, {tokens, v.heads, 1}, {v.token * e, v.head * e, 0}};
}

struct PoolView {
    const void *p;
    int64_t page, slot, head;
};

Strided strided(const PoolView &v, const ks_rotary_args_t &a, int e) {
    return {v.p, a.head_dim * e, {a.pages, a.page_size, a.kv_heads}, {v.page * e, v.slot * e, v.head * e}};
}

// The pool's span, and that its rows are apart, whatever the order of its axes.
bool pool_span(const PoolView &v, const ks_rotary_args_t &a, int e, int64_t *span) {
    if (v.page < 0 || v.slot < 0 || v.head < 0) return false;
    const __int128 last = (__int128)(a.pages - 1) * v.page + (__int128)(a.page_size - 1) * v.slot +
                          (__int128)(a.kv_heads - 1) * v.head + a.head_dim;
    if (last * e > ((__int128)1 << 62)) return false;
    *span = (int64_t)last * e;
    return strided_rows_apart(strided(v, a, e));
}

// Whether a tensor shares memory with the positions, the steps or the slots that the call reads. Every
// CTA reads them for itself while others write.
bool crosses_indices(const ks_rotary_args_t &a, bool pages, const Strided &v) {
    auto crosses = [&](const void *p, int64_t n) { return strided_cross(v, {p, n, {1, 1, 1}, {0, 0, 0}}); };
    return (a.rotary_dim > 0 && (crosses(a.positions, a.tokens * 8) || crosses(a.steps, a.rotary_dim / 2 * 8))) ||
           (pages && crosses(a.slots, a.tokens * 8));
}

// `four`: with `pages`, the 4-bit pools that the keys and values go to instead of args' own.
ks_status_t rotary(const ks_rotary_args_t *args, bool pages, const ks_rotary_4bit_args_t *four, ks_stream_t stream) {
    if (!args) return fail(KS_ERR_INVALID_ARGUMENT, "args is NULL");
    const ks_rotary_args_t &a = *args;
    const int e = elem_bytes((ks_dtype_t)a.dtype);
    if (e == 0) return fail(KS_ERR_UNSUPPORTED_DTYPE, "dtype code %d is not a ks_dtype_t", (int)a.dtype);
    if (a.tokens < 0 || a.tokens > 0x7fffffff)
        return fail(KS_ERR_INVALID_ARGUMENT, "tokens must be in 0 .. 2^31-1 (got %lld)", (long long)a.tokens);
    if (a.head_dim < 1 || a.head_dim > kRotMaxDim)
        return fail(KS_ERR_INVALID_ARGUMENT, "head_dim must be in 1 .. %d (got %lld)", kRotMaxDim, (long long)a.head_dim);
    if (a.rotary_dim < 0 || a.rotary_dim > a.head_dim || a.rotary_dim % 2)
        return fail(KS_ERR_INVALID_ARGUMENT, "rotary_dim must be even, in 0 .. head_dim (got %lld)", (long long)a.rotary_dim);
    if (a.q_heads < 0 || a.kv_heads < 0 || a.q_heads > 65536 || a.kv_heads > 65536 || a.q_heads + a.kv_heads == 0)
        return fail(KS_ERR_INVALID_ARGUMENT, "head counts must be in 0 .. 65536, not both 0");
    if (a.flags & ~(KS_ROTARY_INTERLEAVED | KS_ROTARY_INVERSE))
        return fail(KS_ERR_INVALID_ARGUMENT, "unknown rotary flags 0x%x", (unsigned)a.flags);
    if (!std::isfinite(a.scale)) return fail(KS_ERR_INVALID_ARGUMENT, "scale must be finite");
    if (pages && (a.kv_heads == 0 || a.page_size < 1 || a.pages < 0))
        return fail(KS_ERR_INVALID_ARGUMENT, "a cache needs kv_heads >= 1, page_size >= 1 and pages >= 0");
    if (four && a.head_dim % 16)
        return fail(KS_ERR_INVALID_ARGUMENT, "4-bit pages take head_dims of whole groups of 16 (got %lld)", (long long)a.head_dim);
    if (a.tokens == 0) return KS_SUCCESS;
    if ((a.rotary_dim > 0 && (!a.positions || !a.steps)) || (a.q_heads > 0 && (!a.q || !a.q_out)) ||
        (a.kv_heads > 0 && (!a.k || (!pages && !a.k_out))) || (pages && (!a.v || !a.slots)) ||
        (pages && !four && a.pages > 0 && (!a.k_pages || !a.v_pages)))
        return fail(KS_ERR_INVALID_ARGUMENT, "NULL pointer with tokens > 0");
    if (misaligned(8, a.positions, a.steps, a.slots))
        return fail(KS_ERR_INVALID_ARGUMENT, "positions, steps and slots must be aligned to 8 bytes");

    const View q = {a.q, a.q_token_stride, a.q_head_stride, a.q_heads};
    const View qo = {a.q_out, a.q_out_token_stride, a.q_out_head_stride, a.q_heads};
    const View k = {a.k, a.k_token_stride, a.k_head_stride, a.kv_heads};
    const View ko = {a.k_out, a.k_out_token_stride, a.k_out_head_stride, a.kv_heads};
    const View v = {a.v, a.v_token_stride, a.v_head_stride, a.kv_heads};
    const View *in[3] = {a.q_heads ? &q : nullptr, a.kv_heads ? &k : nullptr, pages ? &v : nullptr};
    const View *out[2] = {a.q_heads ? &qo : nullptr, a.kv_heads && !pages ? &ko : nullptr};
    const int64_t T = a.tokens, D = a.head_dim;
    uintptr_t align = 0;  // every address and stride that the vector kernel uses, in bytes
    int64_t span = 0;
    for (const View *w : {in[0], in[1], in[2], out[0], out[1]}) {
        if (!w) continue;
        if (misaligned(e, w->p))
            return fail(KS_ERR_INVALID_ARGUMENT, "a pointer is not aligned to the %d-byte element", e);
        if (!view_span(*w, T, D, e, &span))
            return fail(KS_ERR_INVALID_ARGUMENT, "a stride is negative or a tensor too large");
        align |= (uintptr_t)w->p | (uintptr_t)(w->token * e) | (uintptr_t)(w->head * e);
    }
    for (int i = 0; i < 2; ++i) {
        if (!out[i]) continue;
        if (!strided_rows_apart(strided(*out[i], T, D, e)))
            return fail(KS_ERR_OVERLAP, "rows of an output share storage");
        if (crosses_indices(a, pages, strided(*out[i], T, D, e)))
            return fail(KS_ERR_OVERLAP, "an output overlaps positions, steps or slots");
        for (int j = 0; j < 3; ++j) {
            if (!in[j]) continue;
            const bool same = i == j && out[i]->p == in[j]->p && (T == 1 || out[i]->token == in[j]->token) &&
                              (out[i]->heads == 1 || out[i]->head == in[j]->head);
            if (!same && strided_cross(strided(*out[i], T, D, e), strided(*in[j], T, D, e)))
                return fail(KS_ERR_OVERLAP, "an output overlaps an input without being exactly it");
        }
    }
    if (out[0] && out[1] && strided_cross(strided(qo, T, D, e), strided(ko, T, D, e)))
        return fail(KS_ERR_OVERLAP, "q_out and k_out storage overlap");
    if (four) {
        uintptr_t code_align = 0, scale_align = 0;
        const ks_status_t st = check_pools4(four->k_pages, four->v_pages, a.pages, a.page_size, a.kv_heads, D, true,
                                            &code_align, &scale_align);
        if (st != KS_SUCCESS) return st;
        if (a.pages > 0) {
            for (const ks_pages_4bit_t *p : {&four->k_pages, &four->v_pages})
                for (int part = 0; part < 2; ++part)
                    if (crosses_indices(a, pages, strided4(*p, part != 0, a.pages, a.page_size, a.kv_heads, D)))
                        return fail(KS_ERR_OVERLAP, "the cache overlaps positions, steps or slots");
            for (const View *w : {in[0], in[1], in[2], out[0]}) {
                if (!w) continue;
                view_span(*w, T, D, e, &span);
                if (crosses_pools4(four->k_pages, four->v_pages, a.pages, a.page_size, a.kv_heads, D, w->p, span))
                    return fail(KS_ERR_OVERLAP, "the cache overlaps q, k, v or q_out");
            }
        }
    } else if (pages && a.pages > 0) {
        const PoolView pools[2] = {{a.k_pages, a.k_page_stride, a.k_slot_stride, a.k_pages_head_stride},
                                   {a.v_pages, a.v_page_stride, a.v_slot_stride, a.v_pages_head_stride}};
        int64_t n[2] = {0, 0};
        for (int i = 0; i < 2; ++i) {
            if (misaligned(e, pools[i].p))
                return fail(KS_ERR_INVALID_ARGUMENT, "a pointer is not aligned to the %d-byte element", e);
            if (!pool_span(pools[i], a, e, &n[i]))
                return fail(KS_ERR_INVALID_ARGUMENT, "the cache's strides are negative, too large or let rows share storage");
            align |= (uintptr_t)pools[i].p | (uintptr_t)(pools[i].page * e) | (uintptr_t)(pools[i].slot * e) |
                     (uintptr_t)(pools[i].head * e);
            if (crosses_indices(a, pages, strided(pools[i], a, e)))
                return fail(KS_ERR_OVERLAP, "the cache overlaps positions, steps or slots");
            for (const View *w : {in[0], in[1], in[2], out[0]}) {
                if (!w) continue;
                view_span(*w, T, D, e, &span);
                if (overlaps(pools[i].p, n[i], w->p, span))
                    return fail(KS_ERR_OVERLAP, "the cache overlaps q, k, v or q_out");
            }
        }
        if (strided_cross(strided(pools[0], a, e), strided(pools[1], a, e)))
            return fail(KS_ERR_OVERLAP, "k_pages and v_pages storage overlap");
    }

    const int V = 16 / e;
    const bool half = (a.flags & KS_ROTARY_INTERLEAVED) == 0;
    bool vec = (align & 15u) == 0 && D % V == 0 && (half ? (a.rotary_dim / 2) % V == 0 : a.rotary_dim % V == 0);
    if (four && half && a.rotary_dim % 32) vec = false;  // a group's partners are then not one group
    RotaryArgs k_args;
    k_args.a = a;
    k_args.columns = (int32_t)(vec ? (half ? (D - a.rotary_dim / 2) / V : D / V) : D - a.rotary_dim / 2);
    const int total = (int)(a.q_heads + (four ? 0 : a.kv_heads * (pages ? 2 : 1)));
    // Few tokens: a token's heads are split over CTAs until the SMs are covered (each repeats the
    // token's sines, 64 of them for a head of 128).
    int sms = 0;
    ks_status_t st = device_sms(&sms);
    if (st != KS_SUCCESS) return st;
    const int lanes = vec ? kRotThreads / k_args.columns : 8;
    int parts = (int)((sms + T - 1) / T);
    const int most = (total + lanes - 1) / lanes;
    parts = parts > most ? most : parts;
    k_args.heads_per_y = parts ? (total + parts - 1) / parts : 0;  // no queries (4-bit pools alone): no parts
    parts = parts ? (total + k_args.heads_per_y - 1) / k_args.heads_per_y : 0;
    // As many threads as do the CTA's heads in equal rounds: with 72 heads of 8 columns, 3 rounds of 192
    // threads, not 2 of 256 and a third of 64.
    int threads = kRotThreads;
    if (vec && parts) {
        const int rounds = (k_args.heads_per_y + lanes - 1) / lanes;
        threads = ((k_args.heads_per_y + rounds - 1) / rounds * k_args.columns + 31) / 32 * 32;
        threads = threads < 64 ? 64 : threads;
    }
    if (four) {
        const cudaError_t ce = rotary_4bit_launch(k_args, *four, vec, half, parts, threads, static_cast<cudaStream_t>(stream));
        if (ce != cudaSuccess) return fail(KS_ERR_CUDA, "launch: %s", cudaGetErrorString(ce));
        return KS_SUCCESS;
    }
    const void *f;
    switch (a.dtype) {
    case KS_DTYPE_BF16: f = pages ? rotary_pick<__nv_bfloat16, true>(vec, half) : rotary_pick<__nv_bfloat16, false>(vec, half); break;
    case KS_DTYPE_F16: f = pages ? rotary_pick<__half, true>(vec, half) : rotary_pick<__half, false>(vec, half); break;
    default: f = pages ? rotary_pick<float, true>(vec, half) : rotary_pick<float, false>(vec, half); break;
    }
    void *kp[] = {&k_args};
    cudaError_t ce = launch_kernel(f, dim3((unsigned)T, (unsigned)parts), dim3((unsigned)threads), 0, kp,
                                   static_cast<cudaStream_t>(stream), launch_pdl_enabled());
    if (ce != cudaSuccess) return fail(KS_ERR_CUDA, "launch: %s", cudaGetErrorString(ce));
    return KS_SUCCESS;
}

}  // namespace

cudaError_t rotary_queries_launch(const RotaryArgs &args, bool vec, bool half, int threads, cudaStream_t stream) {
    RotaryArgs k_args = args;
    k_args.a.kv_heads = 0;
    const void *f = args.a.dtype == KS_DTYPE_BF16  ? rotary_pick<__nv_bfloat16, false>(vec, half)
                    : args.a.dtype == KS_DTYPE_F16 ? rotary_pick<__half, false>(vec, half)
                                                   : rotary_pick<float, false>(vec, half);
    void *kp[] = {&k_args};
    return launch_kernel(f, dim3((unsigned)args.a.tokens), dim3((unsigned)threads), 0, kp, stream, launch_pdl_enabled());
}

int fault_flags_rotary(bool clear) { return fault_flags_t(clear); }

}  // namespace ks

extern "C" {

ks_status_t ks_rotary(const ks_rotary_args_t *args, ks_stream_t stream) {
    return ks::rotary(args, false, nullptr, stream);
}

ks_status_t ks_rotary_to_pages(const ks_rotary_args_t *args, ks_stream_t stream) {
    return ks::rotary(args, true, nullptr, stream);
}

ks_status_t ks_rotary_to_pages_4bit(const ks_rotary_4bit_args_t *args, ks_stream_t stream) {
    if (!args) return ks::fail(KS_ERR_INVALID_ARGUMENT, "args is NULL");
    return ks::rotary(&args->rotary, true, args, stream);
}

}  // extern "C"
