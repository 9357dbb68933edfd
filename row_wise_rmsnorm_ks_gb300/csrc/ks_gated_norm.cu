// The norm after a block, its gate, the scaled residual add and the norm before the next block, in one pass
// (ks_gated_add_rms_norm). Per row, in FP32:
//     n = x * rsqrt(mean(x^2) + eps) * post_weight,  s = residual_scale * r + block_scale * gate * n,
//     r = cast(s),  x = cast(s * rsqrt(mean(s^2) + eps) * weight)
// Two sums over the row, the second of what the first gives: the row has to stay at hand between them. Rows of up to
// 4096 16-byte vectors lie in a CTA's registers, x and r each read and written once, which bounds the operator by
// memory (4 values a place), or in a CTA's registers by smaller words where no vector fits (bound by instructions, a load or
// store for one to four values); wider rows are read three times, the second and third time mostly from L2.
//
// What counts is how many bytes are on their way while rows are summed, so a thread holds x as it was read, packed,
// until the second sum's values take its place, and asks for the weights where they are used: 64 registers at four
// vectors a thread, 1024 threads an SM. (Measured, bf16 [16383, 8192], both norms, a gate per sequence: 176 us, 158 us
// at the copy rate; 207 with x unpacked and the weights asked for ahead, 216 through a ring of bulk copies, which is
// slower yet for narrower rows. bf16 [4, 1536], gate per channel: 3.1 us by graph replay, the two sums' latency.)
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "ks_decode.cuh"

namespace ks {
namespace {

struct GatedArgs {
    ks_gated_norm_args_t a;
    int64_t hv;  // vectors of a row
};

// The gate's row of a row, NULL without a gate.
template <typename T>
__device__ __forceinline__ const T *gate_row(const ks_gated_norm_args_t &a, int64_t row) {
    if (!a.gate) return nullptr;
    return (const T *)a.gate + (a.rows_per_gate == a.rows ? 0 : quotient(row, a.rows_per_gate)) * a.gate_row_stride;
}

template <int N>
__device__ __forceinline__ void fill(float (&f)[N], float v) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = v;
}

template <bool kPair, int P>
__device__ __forceinline__ void times(float2 (&s)[P], float v) {
    const float2 w = make_float2(v, v);
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = pair_mul<kPair>(s[i], w);
}
template <bool kPair, int P>
__device__ __forceinline__ void times(float2 (&s)[P], const float2 (&w)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = pair_mul<kPair>(s[i], w[i]);
}

// n bytes on their way from memory to L2.
__device__ __forceinline__ void prefetch_l2(const void *p, int n) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(n) : "memory");
}

// What a thread does with its vectors of a row. kAhead asks for weights and gate before the sums that they wait for, at
// the cost of their registers; without it, x stays packed until the second sum, so that more rows are on their way.
template <typename T, int V, int kTeam, bool kAhead>
__device__ __forceinline__ void gated_row(const ks_gated_norm_args_t &a, int64_t row, int hv, int t, int g, uint4 (&xv)[V],
                                          const uint4 (&rv)[V], float (&red)[2][32], int &slot) {
    using E = Elem<T>;
    constexpr int P = E::kPerVec / 2;
    constexpr bool kPair = E::kPairMath;
    constexpr int A = kAhead ? V : 1;
    const float hidden = (float)a.hidden;
    uint4 *xr = (uint4 *)a.x + row * hv, *rr = (uint4 *)a.residual + row * hv;
    auto get = [&](const void *p, int k) {
        const int c = t + k * g;
        return c < hv ? __ldg((const uint4 *)p + c) : make_uint4(0, 0, 0, 0);
    };
    auto ask = [&](const void *p, uint4 (&v)[A]) {
        if constexpr (kAhead) {
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = get(p, k);
        }
    };
    auto apply = [&](const void *p, const uint4 (&v)[A], int k, float2 (&s)[P]) {
        float2 w[P];
        E::unpack2(kAhead ? v[kAhead ? k : 0] : get(p, k), w);
        times<kPair>(s, w);
    };
    float factor = a.block_scale;
    uint4 post[A], gate[A], weight[A];
    const T *const of = gate_row<T>(a, row);
    const bool gates = of && a.gate_column_stride;
    if (a.post_weight) ask(a.post_weight, post);
    if (gates) ask(of, gate);
    else if (of) factor *= E::load1(of, 0);
    float scale = 1.0f;
    if (a.post_weight) {
        PairSumSq<kPair> acc;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float2 x[P];
            E::unpack2(xv[k], x);
            acc.add(x);
        }
        scale = row_scale(team_sum<kTeam>(acc.total(), red[slot ^= 1]), hidden, a.eps);
    }
    ask(a.weight, weight);
    float2 s[V][P];
    PairSumSq<kPair> acc;
    const float2 f2 = make_float2(factor, factor), r2 = make_float2(a.residual_scale, a.residual_scale);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int c = t + k * g;
        if (!kAhead) opaque(xv[k]);  // unpacked again
        E::unpack2(xv[k], s[k]);
        if (a.post_weight) {
            times<kPair>(s[k], scale);
            apply(a.post_weight, post, k, s[k]);
        }
        if (gates) apply(of, gate, k, s[k]);
        float2 r[P];
        E::unpack2(rv[k], r);
#pragma unroll
        for (int i = 0; i < P; ++i) s[k][i] = pair_fma<kPair>(r[i], r2, pair_mul<kPair>(s[k][i], f2));
        if (c < hv) {
            __stcs(rr + c, E::pack2(s[k]));
            acc.add(s[k]);
        }
    }
    const float out_scale = row_scale(team_sum<kTeam>(acc.total(), red[slot ^= 1]), hidden, a.eps);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int c = t + k * g;
        times<kPair>(s[k], out_scale);
        apply(a.weight, weight, k, s[k]);
        if (c < hv) __stcs(xr + c, E::pack2(s[k]));
    }
}

// A row per team, V vectors a thread: a warp (kTeam 32), several of them a CTA, or the CTA (0).
template <typename T, int V, int kTeam, bool kAhead>
__global__ void __launch_bounds__(kTeam ? 256 : 512, (V <= 4 && !kAhead ? 2 : 1) * (kTeam ? 2 : 1))
gated_rows_kernel(const __grid_constant__ GatedArgs args) {
    __shared__ float red[2][32];
    const ks_gated_norm_args_t &a = args.a;
    const int g = kTeam ? kTeam : blockDim.x, t = kTeam ? threadIdx.x % 32 : threadIdx.x;
    const int teams = kTeam ? blockDim.x / 32 : 1, team = kTeam ? threadIdx.x / 32 : 0;
    const int hv = (int)args.hv;
    int slot = 0;  // of `red`: every sum takes the other one
    grid_dependency_wait();
    allow_dependents_launch();
    for (int64_t row = (int64_t)blockIdx.x * teams + team; row < a.rows; row += (int64_t)gridDim.x * teams) {
        uint4 xv[V], rv[V];
        load_row<V>((const uint4 *)a.x + row * hv, t, g, hv, xv);
        load_row<V>((const uint4 *)a.residual + row * hv, t, g, hv, rv);
        if (V == 8) {
            const int64_t next = row + gridDim.x;
            if (t == 0 && next < a.rows) {
                prefetch_l2((const uint4 *)a.x + next * hv, hv * 16);
                prefetch_l2((const uint4 *)a.residual + next * hv, hv * 16);
            }
        }
        gated_row<T, V, kTeam, kAhead>(a, row, hv, t, g, xv, rv, red, slot);
    }
}

// N values that lie together, N a power of two of up to 8 bytes.
template <typename T, int N>
struct Few {
    static constexpr int kBytes = N * (int)sizeof(T);
    using Word = typename std::conditional<kBytes == 8, uint2, typename std::conditional<kBytes == 4, uint32_t, uint16_t>::type>::type;
    static_assert(sizeof(Word) == kBytes, "2, 4 or 8 bytes");
    __device__ __forceinline__ static void unpack(Word w, float (&f)[N]) {
        T v[N];
        memcpy(v, &w, kBytes);
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = Elem<T>::load1(v, i);
    }
    __device__ __forceinline__ static Word pack(const float (&f)[N]) {
        T v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) Elem<T>::store1(v, i, f[i]);
        Word w;
        memcpy(&w, v, kBytes);
        return w;
    }
};

// Rows that no 16-byte vector fits, kValues for each thread: N values an access, the row in registers between its sums as
// above (64 at most; of one value an access and 16 a thread, 24 to 32 bytes of them spill).
template <typename T, int N, int kValues>
__global__ void __launch_bounds__(1024, 1) gated_odd_kernel(const __grid_constant__ GatedArgs args) {
    using F = Few<T, N>;
    using Word = typename F::Word;
    constexpr int K = kValues / N;
    __shared__ float red[2][32];
    const ks_gated_norm_args_t &a = args.a;
    const int n = (int)a.hidden / N, g = blockDim.x, t = threadIdx.x;
    const float hidden = (float)a.hidden;
    int slot = 0;  // of `red`: every sum takes the other one
    grid_dependency_wait();
    allow_dependents_launch();
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        Word *x = (Word *)((T *)a.x + row * a.hidden), *r = (Word *)((T *)a.residual + row * a.hidden);
        Word xv[K], rv[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = t + k * g;
            xv[k] = rv[k] = Word{};
            if (c < n) {
                xv[k] = __ldcs(x + c);
                rv[k] = __ldcs(r + c);
            }
        }
        float factor = a.block_scale, scale = 1.0f;
        const T *const gate = gate_row<T>(a, row);
        const bool gates = gate && a.gate_column_stride;
        if (gate && !gates) factor *= Elem<T>::load1(gate, 0);
        auto times_at = [&](const void *p, int c, float (&s)[N]) {
            float w[N];
            F::unpack(__ldg((const Word *)p + c), w);
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] *= w[i];
        };
        if (a.post_weight) {
            SumSq acc;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                float f[N];
                F::unpack(xv[k], f);
                acc.add(f);
            }
            scale = row_scale(team_sum<0>(acc.total(), red[slot ^= 1]), hidden, a.eps);
        }
        float s[K][N];
        SumSq acc;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = t + k * g;
            float f[N];
            F::unpack(xv[k], s[k]);
            F::unpack(rv[k], f);
            if (c < n) {
                if (a.post_weight) {
#pragma unroll
                    for (int i = 0; i < N; ++i) s[k][i] *= scale;
                    times_at(a.post_weight, c, s[k]);
                }
                if (gates) times_at(gate, c, s[k]);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) s[k][i] = fmaf(f[i], a.residual_scale, s[k][i] * factor);
            if (c < n) {
                __stcs(r + c, F::pack(s[k]));
                acc.add(s[k]);
            }
        }
        const float out_scale = row_scale(team_sum<0>(acc.total(), red[slot ^= 1]), hidden, a.eps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = t + k * g;
            if (c < n) {
#pragma unroll
                for (int i = 0; i < N; ++i) s[k][i] *= out_scale;
                times_at(a.weight, c, s[k]);
                __stcs(x + c, F::pack(s[k]));
            }
        }
    }
}

// s of some places, in place of x: `scale` is the first norm's (1 without one).
template <int N>
__device__ __forceinline__ void gated_sum(float (&x)[N], const float (&r)[N], float scale, const float (&post)[N], const float (&gate)[N],
                                          float residual_scale, float block_scale) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = fmaf(r[i], residual_scale, x[i] * scale * post[i] * gate[i] * block_scale);
}

// Any width and alignment: the row read up to three times, vector by vector or value by value.
template <typename T, bool kVec>
__global__ void __launch_bounds__(512) gated_wide_kernel(const __grid_constant__ GatedArgs args) {
    using E = Elem<T>;
    constexpr int N = kVec ? E::kPerVec : 1;
    __shared__ float red[2][32];
    const ks_gated_norm_args_t &a = args.a;
    const int64_t n = kVec ? args.hv : a.hidden;
    const float hidden = (float)a.hidden;
    int slot = 0;  // of `red`: every sum takes the other one
    grid_dependency_wait();
    allow_dependents_launch();
    auto load = [](const T *p, int64_t c, float (&f)[N]) {
        if constexpr (kVec) E::unpack(reinterpret_cast<const uint4 *>(p)[c], f);
        else f[0] = E::load1(p, c);
    };
    auto store = [](T *p, int64_t c, const float (&f)[N]) {
        if constexpr (kVec) reinterpret_cast<uint4 *>(p)[c] = E::pack(f);
        else E::store1(p, c, f[0]);
    };
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        T *x = (T *)a.x + row * a.hidden, *r = (T *)a.residual + row * a.hidden;
        const T *gate = gate_row<T>(a, row);
        float scale = 1.0f;
        if (a.post_weight) {
            SumSq acc;
            for (int64_t c = threadIdx.x; c < n; c += blockDim.x) {
                float f[N];
                load(x, c, f);
                acc.add(f);
            }
            scale = row_scale(team_sum<0>(acc.total(), red[slot ^= 1]), hidden, a.eps);
        }
        auto sum = [&](int64_t c, float (&s)[N]) {
            float rv[N], post[N], gt[N];
            load(x, c, s);
            load(r, c, rv);
            fill(post, 1.0f);
            fill(gt, 1.0f);
            if (a.post_weight) load((const T *)a.post_weight, c, post);
            if (gate) {
                if (a.gate_column_stride) load(gate, c, gt);
                else fill(gt, E::load1(gate, 0));
            }
            gated_sum(s, rv, scale, post, gt, a.residual_scale, a.block_scale);
        };
        SumSq acc;
        for (int64_t c = threadIdx.x; c < n; c += blockDim.x) {
            float s[N];
            sum(c, s);
            acc.add(s);
        }
        const float out_scale = row_scale(team_sum<0>(acc.total(), red[slot ^= 1]), hidden, a.eps);
        for (int64_t c = threadIdx.x; c < n; c += blockDim.x) {
            float s[N], w[N];
            sum(c, s);
            store(r, c, s);
            load((const T *)a.weight, c, w);
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = s[i] * out_scale * w[i];
            store(x, c, s);
        }
    }
}

template <typename T, int N>
const void *odd_kernel(bool small) {
    return small ? (const void *)gated_odd_kernel<T, N, 4> : (const void *)gated_odd_kernel<T, N, 16>;
}

// The kernel for rows of hv vectors (0: no vector fits, rows and pointers are aligned to `align` bytes): threads of a CTA, and
// rows that one does at once.
template <typename T>
const void *pick(int64_t hv, int64_t hidden, int align, bool few, int *block, int *rows) {
    *rows = 1;
    if (hv == 0 && hidden <= 1024 * 16) {
        // Sixteen values a thread, so that an SM holds more rows; for few rows, a few values of an access a thread each.
        // (Measured, bf16, many rows GB/s and 100 rows us: 1001 places 16 values 2239, 6.8, 4 values 2153, 4.3; 404 3567, 3.7,
        // and 2121, 3.2; 4098 2799, 6.2. In three passes 656, 5.2 for 1001.)
        const int n = align / (int)sizeof(T), most = 8 / (int)sizeof(T), each = n < most ? n : most;
        const bool small = few && hidden <= 1024 * 4;
        const int64_t threads = few ? hidden / each : (hidden + 15) / 16;
        *block = (int)(threads < 1024 ? (threads + 31) / 32 * 32 : 1024);
        return each == 4   ? odd_kernel<T, sizeof(T) == 2 ? 4 : 2>(small)
               : each == 2 ? odd_kernel<T, 2>(small)
                           : odd_kernel<T, 1>(small);
    }
    if (hv == 0 || hv > 4096) {
        *block = 512;
        return hv ? (const void *)gated_wide_kernel<T, true> : (const void *)gated_wide_kernel<T, false>;
    }
    // Rows that fill no GPU: latency counts, so a vector a thread where that fits, and everything asked for at once.
    if (few) {
        const int v = hv <= 512 ? 1 : hv <= 1024 ? 2 : hv <= 2048 ? 4 : 8;
        *block = (int)((hv + v - 1) / v + 31) / 32 * 32;
        return v == 1   ? (const void *)gated_rows_kernel<T, 1, 0, true>
               : v == 2 ? (const void *)gated_rows_kernel<T, 2, 0, true>
               : v == 4 ? (const void *)gated_rows_kernel<T, 4, 0, true>
                        : (const void *)gated_rows_kernel<T, 8, 0, false>;
    }
    // Many rows: a warp's sums wait for no other warp, and from four vectors a thread on enough bytes are on their way.
    // (Measured, bf16 with both norms and a gate, 192 MB a tensor, GB/s by vectors a thread, w: a warp a row:
    //  32 vectors a row w1 5352, w2 4615, 1 4762; 64 w2 6512, 2 6208, w4 5457; 128 2 6049, 4 5821, w4 5986;
    //  192 2 5892, 4 6070; 448 2 5487, 4 6343; 1024 2 5200, 4 6238, 8 6186; 2048 4 6248, 8 6020.)
    // Rows of more than 2048 vectors have an SM to themselves: the next one is fetched into L2 meanwhile. (3584 vectors,
    // fp32, 6182 for 4830 without; up to 2048 within 3 % either way.)
    if (hv <= 64) {
        *block = 256;
        *rows = 8;
        return hv <= 32 ? (const void *)gated_rows_kernel<T, 1, 32, false> : (const void *)gated_rows_kernel<T, 2, 32, false>;
    }
    const int v = hv <= 160 ? 2 : hv <= 2048 ? 4 : 8;
    *block = (int)((hv + v - 1) / v + 31) / 32 * 32;
    return v == 2   ? (const void *)gated_rows_kernel<T, 2, 0, false>
           : v == 4 ? (const void *)gated_rows_kernel<T, 4, 0, false>
                    : (const void *)gated_rows_kernel<T, 8, 0, false>;
}

}  // namespace

}  // namespace ks

using namespace ks;

extern "C" ks_status_t ks_gated_add_rms_norm(const ks_gated_norm_args_t *args, ks_stream_t stream) {
    if (!args) return fail(KS_ERR_INVALID_ARGUMENT, "args is NULL");
    const ks_gated_norm_args_t &a = *args;
    const int e = elem_bytes((ks_dtype_t)a.dtype);
    if (e == 0) return fail(KS_ERR_UNSUPPORTED_DTYPE, "dtype code %d is not a ks_dtype_t", (int)a.dtype);
    if (a.hidden <= 0) return fail(KS_ERR_INVALID_ARGUMENT, "hidden must be > 0 (got %lld)", (long long)a.hidden);
    if (a.rows < 0) return fail(KS_ERR_INVALID_ARGUMENT, "rows must be >= 0 (got %lld)", (long long)a.rows);
    if (!std::isfinite(a.eps) || !(a.eps > 0.0f))
        return fail(KS_ERR_INVALID_ARGUMENT, "eps must be finite and > 0 (got %g)", (double)a.eps);
    if (!std::isfinite(a.residual_scale) || !std::isfinite(a.block_scale))
        return fail(KS_ERR_INVALID_ARGUMENT, "residual_scale and block_scale must be finite");
    if ((__int128)a.rows * a.hidden * e > ((__int128)1 << 62))
        return fail(KS_ERR_INVALID_ARGUMENT, "rows*hidden*element size is too large");
    if (a.rows == 0) return KS_SUCCESS;
    if (!a.x || !a.residual || !a.weight) return fail(KS_ERR_INVALID_ARGUMENT, "NULL pointer with rows > 0");
    if (misaligned(e, a.x, a.residual, a.weight) || misaligned(e, a.post_weight, a.gate))
        return fail(KS_ERR_INVALID_ARGUMENT, "a pointer is not aligned to the %d-byte element", e);
    const int64_t n = a.rows * a.hidden * e, w = a.hidden * e;
    if (overlaps(a.x, n, a.residual, n)) return fail(KS_ERR_OVERLAP, "x and residual storage overlap");
    uintptr_t align = (uintptr_t)a.x | (uintptr_t)a.residual | (uintptr_t)a.weight | (uintptr_t)a.post_weight;
    int64_t gate_bytes = 0;
    if (a.gate) {
        if (a.rows_per_gate < 1 || a.gate_row_stride < 0 || a.gate_column_stride < 0 || a.gate_column_stride > 1)
            return fail(KS_ERR_INVALID_ARGUMENT, "the gate needs rows_per_gate >= 1, a row stride >= 0 and a column stride of 0 or 1");
        const int64_t gates = (a.rows - 1) / a.rows_per_gate + 1;
        const __int128 last = (__int128)(gates - 1) * a.gate_row_stride + (a.hidden - 1) * a.gate_column_stride + 1;
        if (last * e > ((__int128)1 << 62)) return fail(KS_ERR_INVALID_ARGUMENT, "the gate is too large");
        gate_bytes = (int64_t)last * e;
        if (a.gate_column_stride) align |= (uintptr_t)a.gate | (uintptr_t)(gates > 1 ? a.gate_row_stride * e : 0);
    }
    for (const void *p : {(const void *)a.x, (const void *)a.residual})
        if (overlaps(p, n, a.weight, w) || (a.post_weight && overlaps(p, n, a.post_weight, w)) ||
            (a.gate && overlaps(p, n, a.gate, gate_bytes)))
            return fail(KS_ERR_OVERLAP, "x or residual overlaps a weight or the gate");
    int sms = 0;
    const ks_status_t st = device_sms(&sms);
    if (st != KS_SUCCESS) return st;
    GatedArgs k_args;
    k_args.a = a;
    const bool vec = (align & 15u) == 0 && w % 16 == 0;
    k_args.hv = vec ? w / 16 : 0;
    const uintptr_t bits = align | (uintptr_t)w | 16u;
    const int lowest = (int)(bits & (~bits + 1));
    int block = 0, at_once = 1;
    const bool few = a.rows <= sms;
    const void *f = a.dtype == KS_DTYPE_BF16  ? pick<__nv_bfloat16>(k_args.hv, a.hidden, lowest, few, &block, &at_once)
                    : a.dtype == KS_DTYPE_F16 ? pick<__half>(k_args.hv, a.hidden, lowest, few, &block, &at_once)
                                              : pick<float>(k_args.hv, a.hidden, lowest, few, &block, &at_once);
    int64_t most = (int64_t)sms * (2048 / block > 32 ? 32 : 2048 / block);
    // Rows read more than once: no more at a time than leave half of L2 to others' reads, while every SM has one. (Measured,
    // fp32, GB/s with and without: 20480 places a row 5390, 4688; 32768 4724, 4085. 131072, of which no SM's fit: 2806, 3092.)
    const int64_t room = ((int64_t)64 << 20) / (2 * w);
    if (k_args.hv > 4096 && room >= sms && room < most) most = room;
    const int64_t want = (a.rows + at_once - 1) / at_once, grid = want < most ? want : most;
    void *kp[] = {&k_args};
    const cudaError_t ce = launch_kernel(f, dim3((unsigned)grid), dim3((unsigned)block), 0, kp, static_cast<cudaStream_t>(stream),
                                         launch_pdl_enabled());
    if (ce != cudaSuccess) return fail(KS_ERR_CUDA, "launch: %s", cudaGetErrorString(ce));
    return KS_SUCCESS;
}
