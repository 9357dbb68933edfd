// What the rotary kernels share: angles, addresses, and the turning of a token's heads. Mathematics and layout are
// described in ks_rotary.cu.
#pragma once

#include "ks_decode.cuh"
#include "ks_fp4.cuh"

namespace ks {

constexpr int kRotThreads = 256;
constexpr int kRotMaxDim = 1024;  // head_dim limit: rotary_dim / 2 sines and cosines in shared memory

struct RotaryArgs {
    ks_rotary_args_t a;
    int32_t columns;     // vectors, or pairs of vectors, per head
    int32_t heads_per_y; // head slots per CTA (all of a token's, or a part)
};

// cos and sin of (t / 2^64) turns times scale, t taken mod 2^64.
__device__ __forceinline__ float2 turn_cos_sin(uint64_t t, float scale) {
    const uint32_t hi = (uint32_t)(t >> 32);
    const uint32_t quadrant = (hi + 0x20000000u) >> 30;
    const int32_t rest = (int32_t)(hi - (quadrant << 30));  // within an eighth of a turn
    float s, c;
    sincospif((float)rest * 4.656612873077393e-10f, &s, &c);  // rest / 2^31 half turns
    const float cc = (quadrant & 1) ? s : c, ss = (quadrant & 1) ? c : s;
    const bool neg_c = quadrant == 1 || quadrant == 2, neg_s = quadrant >= 2;
    return make_float2((neg_c ? -cc : cc) * scale, (neg_s ? -ss : ss) * scale);
}

// Where a head slot's row is read and written. Slots 0 .. q_heads-1 are the query's heads, then the
// keys', then (with a cache) the values', which are not rotated.
template <typename T>
__device__ __forceinline__ const T *rot_src(const ks_rotary_args_t &a, int64_t token, int slot) {
    if (slot < a.q_heads) return (const T *)a.q + token * a.q_token_stride + slot * a.q_head_stride;
    const int64_t h = slot - a.q_heads;
    if (h < a.kv_heads) return (const T *)a.k + token * a.k_token_stride + h * a.k_head_stride;
    return (const T *)a.v + token * a.v_token_stride + (h - a.kv_heads) * a.v_head_stride;
}

// The token's rows in the cache: NULL where they are not written (a negative slot, or one past the
// pool, which is also reported in the fault word).
template <typename T>
struct RotPage {
    T *k, *v;
};

template <typename T>
__device__ __forceinline__ RotPage<T> rot_page(const ks_rotary_args_t &a, int64_t slot) {
    RotPage<T> p = {nullptr, nullptr};
    const int64_t size = a.page_size;
    if (slot < 0) return p;
    int64_t page, in_page;
    if (((uint64_t)slot | (uint64_t)size) >> 32 == 0) {  // a 32-bit division takes a fifth of the time
        page = (uint32_t)slot / (uint32_t)size;
        in_page = (uint32_t)slot - (uint32_t)page * (uint32_t)size;
    } else {
        page = slot / size;
        in_page = slot - page * size;
    }
    if (page >= a.pages) {
        if (threadIdx.x == 0) atomicOr(&g_fault_flags, kFaultBadIndex);
        return p;
    }
    p.k = (T *)a.k_pages + page * a.k_page_stride + in_page * a.k_slot_stride;
    p.v = (T *)a.v_pages + page * a.v_page_stride + in_page * a.v_slot_stride;
    return p;
}

template <typename T, bool kPages>
__device__ __forceinline__ T *rot_dst(const ks_rotary_args_t &a, int64_t token, int slot, const RotPage<T> &p) {
    if (slot < a.q_heads) return (T *)a.q_out + token * a.q_out_token_stride + slot * a.q_out_head_stride;
    const int64_t h = slot - a.q_heads;
    if (!kPages) return (T *)a.k_out + token * a.k_out_token_stride + h * a.k_out_head_stride;
    if (!p.k) return nullptr;
    if (h < a.kv_heads) return p.k + h * a.k_pages_head_stride;
    return p.v + (h - a.kv_heads) * a.v_pages_head_stride;
}

// What a token's work hangs on, all loaded at once: its position, its slot, and the step of the angle
// that this thread computes.
struct RotToken {
    uint64_t position, step;
    int64_t slot;
};

template <bool kPages>
__device__ __forceinline__ RotToken rot_token(const ks_rotary_args_t &a, int64_t token) {
    RotToken t = {0, 0, -1};
    if (a.rotary_dim > 0) {  // otherwise nothing is turned, and positions and steps may be NULL
        t.position = (uint64_t)a.positions[token];
        if (threadIdx.x < a.rotary_dim / 2) t.step = (uint64_t)a.steps[threadIdx.x];
    }
    if (kPages) t.slot = a.slots[token];
    return t;
}

__device__ __forceinline__ void rot_table(const ks_rotary_args_t &a, const RotToken &t, float2 *cs) {
    const bool inverse = (a.flags & KS_ROTARY_INVERSE) != 0;
    uint64_t step = t.step;
    for (int j = threadIdx.x; j < (int)(a.rotary_dim / 2); j += blockDim.x) {
        if (j != threadIdx.x) step = (uint64_t)a.steps[j];
        const uint64_t angle = t.position * step;
        cs[j] = turn_cos_sin(inverse ? 0 - angle : angle, a.scale);
    }
}

// 16-byte vectors. kHalf: pair (j, j + rotary_dim/2); otherwise pair (2j, 2j + 1). kU: vectors
// (or pairs of them) a thread has in flight; measured (us): 1, 2 and 3 of them, 16384 tokens of 64 + 8
// heads 88.4, 88.0, 87.1; 8192 tokens of 56 + 8 + 8 into the cache, where addresses take more registers,
// 52.6, 48.9, 51.9.
template <typename T, bool kHalf, bool kPages>
__device__ __forceinline__ void rot_heads_vec(const RotaryArgs &args, int64_t token, int first, int last, float2 *cs) {
    constexpr int V = Elem<T>::kPerVec;
    constexpr int kU = kPages ? 2 : 3;
    const ks_rotary_args_t &a = args.a;
    const int column = threadIdx.x % args.columns, lane = threadIdx.x / args.columns;
    const int lanes = blockDim.x / args.columns;
    // the column's first element, and its partner's for a half-split pair
    const int pairs = (int)(a.rotary_dim / 2) / V;            // columns that are pairs (kHalf)
    const int turned = kHalf ? pairs : (int)a.rotary_dim / V; // columns that are rotated
    const bool mine = column < turned;
    const int at = (!kHalf || mine) ? column * V : (column + pairs) * V;
    const int at2 = at + pairs * V;

    uint4 x[kU], y[kU];
    const bool active = lane < lanes;
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int slot = base + u * lanes;
            if (active && slot < last) {
                const T *src = rot_src<T>(a, token, slot);
                x[u] = *reinterpret_cast<const uint4 *>(src + at);
                if (kHalf && mine) y[u] = *reinterpret_cast<const uint4 *>(src + at2);
            }
        }
    };
    const RotToken t = rot_token<kPages>(a, token);
    load(first + lane);
    rot_table(a, t, cs);
    RotPage<T> page = {};
    if (kPages) page = rot_page<T>(a, t.slot);
    __syncthreads();
    float2 turn[V];
    if (mine) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (kHalf) turn[i] = cs[column * V + i];
            else if (i < V / 2) turn[i] = cs[column * (V / 2) + i];
        }
    }
    for (int base = first + lane; base < last; base += kU * lanes) {
        if (base != first + lane) load(base);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int slot = base + u * lanes;
            if (!active || slot >= last) break;
            T *dst = rot_dst<T, kPages>(a, token, slot, page);
            if (kPages && dst == nullptr) continue;
            if (mine && (!kPages || slot < a.q_heads + a.kv_heads)) {
                float p[V];
                Elem<T>::unpack(x[u], p);
                if (kHalf) {
                    float q[V];
                    Elem<T>::unpack(y[u], q);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float c = turn[i].x, s = turn[i].y, m = p[i], n = q[i];
                        p[i] = fmaf(m, c, -n * s);
                        q[i] = fmaf(n, c, m * s);
                    }
                    y[u] = Elem<T>::pack(q);
                } else {
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float c = turn[i].x, s = turn[i].y, m = p[2 * i], n = p[2 * i + 1];
                        p[2 * i] = fmaf(m, c, -n * s);
                        p[2 * i + 1] = fmaf(n, c, m * s);
                    }
                }
                x[u] = Elem<T>::pack(p);
            }
            *reinterpret_cast<uint4 *>(dst + at) = x[u];
            if (kHalf && mine) *reinterpret_cast<uint4 *>(dst + at2) = y[u];
        }
    }
}

// Element loads, any rotary_dim and alignment: a thread per pair, or per value that is not rotated.
template <typename T, bool kHalf, bool kPages>
__device__ __forceinline__ void rot_heads_scalar(const RotaryArgs &args, int64_t token, int first, int last, float2 *cs) {
    const ks_rotary_args_t &a = args.a;
    const RotToken t = rot_token<kPages>(a, token);
    RotPage<T> page = {};
    if (kPages) page = rot_page<T>(a, t.slot);
    rot_table(a, t, cs);
    __syncthreads();
    const int pairs = (int)(a.rotary_dim / 2);
    const int n = (last - first) * args.columns;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int slot = first + i / args.columns, column = i % args.columns;
        const T *src = rot_src<T>(a, token, slot);
        T *dst = rot_dst<T, kPages>(a, token, slot, page);
        if (kPages && dst == nullptr) continue;
        if (column >= pairs) {  // not rotated
            dst[column + pairs] = src[column + pairs];
            continue;
        }
        const int i0 = kHalf ? column : 2 * column, i1 = kHalf ? column + pairs : 2 * column + 1;
        const T x = src[i0], y = src[i1];
        if (kPages && slot >= a.q_heads + a.kv_heads) {
            dst[i0] = x;
            dst[i1] = y;
            continue;
        }
        const float c = cs[column].x, s = cs[column].y;
        const float m = Elem<T>::load1(&x, 0), k = Elem<T>::load1(&y, 0);
        Elem<T>::store1(dst, i0, fmaf(m, c, -k * s));
        Elem<T>::store1(dst, i1, fmaf(k, c, m * s));
    }
}

// Rotary into 4-bit pools (ks_rotary_4bit.cu). `args` is filled in for the queries: vec, the vectors and head counts
// that a CTA does.
cudaError_t rotary_4bit_launch(const RotaryArgs &args, const ks_rotary_4bit_args_t &four, bool vec, bool half, int parts,
                               int threads, cudaStream_t stream);

// The queries alone, a CTA a token: ks_rotary's kernel (`args` without keys).
cudaError_t rotary_queries_launch(const RotaryArgs &args, bool vec, bool half, int threads, cudaStream_t stream);

}  // namespace ks
