// Attention of new tokens over a paged cache held in 4 bits: the kernel for few rows per key/value head, and the C
// entry points. The division of the work, the running maximum and the join are those of ks_attention.cu.
//
// Keys and values are fp16 numbers exactly (ks_fp4.cuh), so both products run as fp16 with FP32 sums. A bf16 query row
// is brought to a largest magnitude of 1 .. 2 by a power of two, which its scores are given back: values down to
// 2^-14 of the largest stay exact, smaller ones lose at most 2^-25 of it, less than an FP32 sum of the row's
// products does. Probabilities are fp16 too, 2^15 times as large as they are (as in ks_attention.cu).
//
// Few rows make this a stream of the cache, 144 bytes per key of 128 values, and of the instructions that make fp16 of
// it: each pair of codes is a conversion and a product with its group's scale. So the matrix instructions
// take the cache as their 16-row operand, straight from registers, and the query rows as the 8 columns: S^T = K Q^T
// and O^T += V^T P^T. Nothing passes through shared memory on the way:
//   - K: a product's sum runs over any order of the dims, so the lane quad's member t takes dims t D / 4 and on of
//     keys g and g + 8 (g = lane / 4): one contiguous load a key. Queries lie in registers in the same order.
//   - V^T: rows may be any dims, so lane row g has dims g D / 8 and on, of the keys 2 t, 2 t + 1, 2 t + 8 and
//     2 t + 9 that the operand's pairs want: the codes of two keys are merged by nibbles, and a conversion then
//     gives a pair over keys.
//   - P^T comes from S^T by one 8x8 transposition of a matrix of 16-bit values for 8 keys.
// A warp runs alone on every fourth 32-key step, and loads the next step's keys as soon as this step's are used.
#include <cuda_runtime.h>

#include <cmath>
#include <mutex>
#include <unordered_map>

#include "ks_attention_4bit.cuh"

namespace ks {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kStep = 32;                // keys of a warp's step
constexpr int kUnit = kWarps * kStep;    // keys of a unit
constexpr int kTileCost = 3;             // units that beginning and ending a row tile costs
constexpr int kSlotRows = 16;            // rows of a partial slot
constexpr float kLift = 32768.0f;        // what a row's largest probability counts

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_half(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}

// 16-bit values as floats, either type.
__device__ __forceinline__ float2 unpack16(uint32_t w, bool bf16) {
    if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    __half2 h;
    memcpy(&h, &w, 4);
    return __half22float2(h);
}

__device__ __forceinline__ uint32_t pack16(float x, float y, bool bf16) {
    if (!bf16) return pack_half(x, y);
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}

// kN words of codes. Whole: aligned to their size; otherwise in groups of two, those at and past `room` zeros.
template <int kN, bool kWhole>
__device__ __forceinline__ void load_codes(uint32_t (&w)[kN], const uint8_t *p, int room) {
    if constexpr (kWhole && kN % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kN / 4; ++i) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p) + i);
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        }
    } else if constexpr (kN % 2 == 0) {
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) {
            uint2 x = make_uint2(0, 0);
            if (kWhole || 2 * i < room) x = __ldg(reinterpret_cast<const uint2 *>(p) + i);
            w[2 * i] = x.x, w[2 * i + 1] = x.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) w[i] = kWhole || i < room ? __ldg(reinterpret_cast<const uint32_t *>(p) + i) : 0;
    }
}

// kN scales, one a byte of the result. Whole: aligned to kN bytes where kN is 2 or 4.
template <int kN, bool kWhole>
__device__ __forceinline__ uint32_t load_scales(const uint8_t *p, int room) {
    if constexpr (kWhole && kN == 4) return __ldg(reinterpret_cast<const uint32_t *>(p));
    if constexpr (kWhole && kN == 2) return __ldg(reinterpret_cast<const uint16_t *>(p));
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if (kWhole || i < room) x |= (uint32_t)__ldg(p + i) << (8 * i);
    return x;
}

// kR: 64 dims each; kTiles: tiles of 8 query rows; kWhole: head_dim is 64 kR, and rows of codes and scales are aligned
// to what a lane loads of them, and pages are whole blocks of 16 keys.
template <int kR, int kTiles, bool kWhole>
__global__ void __launch_bounds__(kThreads)
attn4_rows_kernel(const __grid_constant__ Attn4Args args) {
    constexpr int kWords = 2 * kR;                 // of a key's codes, for a quad's member
    constexpr int kVScales = (kR + 1) / 2;         // of a value's row, for a lane row
    constexpr int kRows = 8 * kTiles;
    constexpr int kPitch = 64 * kR + 4;
    __shared__ __align__(16) float ow[kWarps][kRows][kPitch];  // written and read in pairs
    __shared__ float mw[kWarps][kRows], lw[kWarps][kRows];
    const AttnArgs &s = args.s;
    const ks_attention_args_t &a = s.a;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int ctas = gridDim.x, cta = blockIdx.x;
    grid_dependency_wait();
    allow_dependents_launch();
    if (threadIdx.x == 0) attn_joins(s, ctas)[cta].pieces = 0;
    AttnCursor cur = attn_begin<kThreads>(s, cta, ctas);
    if (cur.left <= 0) return;
    AttnSeq q = attn_seq(a, cur.seq);

    const int dim = (int)a.head_dim, page_size = (int)a.page_size;
    const bool bf16 = a.dtype == KS_DTYPE_BF16, causal = (a.flags & KS_ATTENTION_CAUSAL) != 0;
    const int k_first = t * kR;                    // the lane's first group of a key
    const int v_first = g * kR;                    // its first word (8 dims) of a value
    const int k_room = 2 * (dim / 16 - k_first), v_room = dim / 8 - v_first;
    const int v_group = v_first / 2;

    while (true) {
        const AttnSpan span = attn_span(s, cur, q);
        const int units = span.units, first = span.first, last = span.last;
        if (first >= last) break;  // the share ends in the tile's extra cost
        const int sees = attn_tile_keys(s, q, cur.row_tile);
        const int kv_head = cur.head / s.head_splits;
        const uint8_t *k_codes = args.k.codes + kv_head * args.k.code_head + k_first * 8;
        const uint8_t *k_scales = args.k.scales + kv_head * args.k.scale_head + k_first;
        const uint8_t *v_codes = args.v.codes + kv_head * args.v.code_head + v_first * 4;
        const uint8_t *v_scales = args.v.scales + kv_head * args.v.scale_head + v_group;
        const int32_t *table = a.page_table + (int64_t)cur.seq * a.table_stride;

        uint32_t kc[4][kWords], ks[4];             // keys g, g + 8, g + 16, g + 24
        uint32_t vc[8][kR], vs[8];                 // values 2 t, 2 t + 1, 2 t + 8, 2 t + 9, then those 16 on
        // The page and the place of key `lane` of a step; page -1: no such key, or its page is not in the pool.
        auto look_up = [&](int key0, int &page, int &place) {
            const int key = key0 + lane;
            page = -1;
            place = 0;
            if (key < sees) {
                const int index = key / page_size;
                page = __ldg(table + index);
                place = key - index * page_size;
                if ((uint32_t)page >= (uint64_t)a.pages) {
                    atomicOr(&g_fault_flags, kFaultBadIndex);
                    page = -1;
                }
            }
        };
        auto load_keys = [&](int page, int place) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = 8 * i + g;
                const int64_t p = __shfl_sync(0xFFFFFFFFu, page, at), r = __shfl_sync(0xFFFFFFFFu, place, at);
#pragma unroll
                for (int j = 0; j < kWords; ++j) kc[i][j] = 0;
                ks[i] = 0;
                if (p >= 0) {
                    load_codes<kWords, kWhole>(kc[i], k_codes + p * args.k.code_page + r * args.k.code_slot, k_room);
                    ks[i] = load_scales<kR, kWhole>(k_scales + p * args.k.scale_page + r * args.k.scale_slot, k_room / 2);
                }
            }
        };
        auto load_values = [&](int page, int place) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = 16 * (i / 4) + 8 * (i / 2 % 2) + 2 * t + i % 2;
                const int64_t p = __shfl_sync(0xFFFFFFFFu, page, at), r = __shfl_sync(0xFFFFFFFFu, place, at);
#pragma unroll
                for (int j = 0; j < kR; ++j) vc[i][j] = 0;
                vs[i] = 0;
                if (p >= 0) {
                    load_codes<kR, kWhole>(vc[i], v_codes + p * args.v.code_page + r * args.v.code_slot, v_room);
                    vs[i] = load_scales<kVScales, false>(v_scales + p * args.v.scale_page + r * args.v.scale_slot,
                                                         kWhole ? kVScales : dim / 16 - v_group);
                }
            }
        };

        int key0 = first * kUnit + warp * kStep;
        int page, place;
        look_up(key0, page, place);
        load_keys(page, place);
        load_values(page, place);

        // the query rows as the products' columns, zeros where the tile has none, and what their scores count
        uint32_t qf[kTiles][4 * kR][2];
        float mul[kTiles][2];
        int limit[kTiles][2];
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
            int token, head;
            const bool real = attn_row(s, q.q0, q.n, cur.head, cur.row_tile, n * 8 + g, &token, &head);
            const uint16_t *row = (const uint16_t *)a.q + token * a.q_token_stride + head * a.q_head_stride;
            float big = 0.0f;
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
                if (real && (kWhole || 2 * r < k_room)) {
                    x[0] = *reinterpret_cast<const uint4 *>(row + (k_first + r) * 16);
                    x[1] = *reinterpret_cast<const uint4 *>(row + (k_first + r) * 16 + 8);
                }
                const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    qf[n][4 * r + i / 2][i % 2] = w[i];
                    const float2 f = unpack16(w[i], true);
                    big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
            float unit = 1.0f;  // the power of two that the row is multiplied by is 1 / unit
            if (bf16) {
                big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
                // 2^-126 .. 2^126, so that its inverse is a normal number too
                const uint32_t e = min(max(__float_as_uint(big) >> 23, 1u), 253u);
                unit = __uint_as_float(e << 23);
                const float inverse = __uint_as_float((254u - e) << 23);
#pragma unroll
                for (int i = 0; i < 4 * kR; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float2 f = unpack16(qf[n][i][j], true);
                        qf[n][i][j] = pack_half(f.x * inverse, f.y * inverse);
                    }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float row_unit = __shfl_sync(0xFFFFFFFFu, unit, 8 * t + 4 * i);  // of row 2 t + i
                mul[n][i] = fminf(fmaxf(s.scale_log2 * row_unit, -3.4e38f), 3.4e38f);
                const int in_seq = cur.row_tile * s.tile_tokens + (n * 8 + 2 * t + i) / s.tile_heads;
                limit[n][i] = causal ? min(sees, q.keys - q.n + in_seq + 1) : sees;
            }
        }
        const int all_see = causal ? min(sees, q.keys - q.n + cur.row_tile * s.tile_tokens + 1) : sees;

        float o[kTiles][4 * kR][4];
        float m[kTiles][2], l[kTiles][2];
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < 4 * kR; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;
        }

        for (int unit = first; unit < last; ++unit, key0 += kUnit) {
            if (key0 >= sees) break;  // the tile's last unit may end before this warp's step
            int next_page = -1, next_place = 0;
            if (unit + 1 < last) look_up(key0 + kUnit, next_page, next_place);
            // ---- scores of 32 keys: key 16 b + g (and 8 on), rows 2 t and 2 t + 1
            float sc[2][kTiles][4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int n = 0; n < kTiles; ++n) sc[b][n][0] = sc[b][n][1] = sc[b][n][2] = sc[b][n][3] = 0.0f;
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    uint32_t scale[2], h[2][8];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t byte = ks[2 * b + i] >> (8 * r) & 0xFF;
                        scale[i] = e4m3_to_half(byte | byte << 8);
                        uint32_t x[4];
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            fp4_to_half(kc[2 * b + i][2 * r + w], x);
#pragma unroll
                            for (int j = 0; j < 4; ++j) h[i][4 * w + j] = half2_mul(x[j], scale[i]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t f[4] = {h[0][2 * j], h[1][2 * j], h[0][2 * j + 1], h[1][2 * j + 1]};
#pragma unroll
                        for (int n = 0; n < kTiles; ++n) mma16816(sc[b][n], f, qf[n][4 * r + j][0], qf[n][4 * r + j][1]);
                    }
                }
            }
            load_keys(next_page, next_place);
            // ---- probabilities
            const bool masked = key0 + kStep > all_see;
            uint32_t p[2][kTiles][2];
#pragma unroll
            for (int n = 0; n < kTiles; ++n) {
                float top[2] = {m[n][0], m[n][1]};
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float x = sc[b][n][i] * mul[n][i & 1];
                        if (masked && key0 + 16 * b + 8 * (i / 2) + g >= limit[n][i & 1]) x = -INFINITY;
                        sc[b][n][i] = x;
                        top[i & 1] = fmaxf(top[i & 1], x);
                    }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 4));
                    top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 8));
                    top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 16));
                }
                if (__any_sync(0xFFFFFFFFu, top[0] != m[n][0] || top[1] != m[n][1])) {
                    const float f0 = exp2_approx(m[n][0] - attn_base(top[0])), f1 = exp2_approx(m[n][1] - attn_base(top[1]));
                    l[n][0] *= f0;
                    l[n][1] *= f1;
#pragma unroll
                    for (int i = 0; i < 4 * kR; ++i) {
                        o[n][i][0] *= f0;
                        o[n][i][1] *= f1;
                        o[n][i][2] *= f0;
                        o[n][i][3] *= f1;
                    }
                    m[n][0] = top[0];
                    m[n][1] = top[1];
                }
                const float b0 = attn_base(m[n][0]), b1 = attn_base(m[n][1]);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const float x0 = exp2_approx(sc[b][n][0] - b0) * kLift, x1 = exp2_approx(sc[b][n][1] - b1) * kLift;
                    const float x2 = exp2_approx(sc[b][n][2] - b0) * kLift, x3 = exp2_approx(sc[b][n][3] - b1) * kLift;
                    l[n][0] += x0 + x2;
                    l[n][1] += x1 + x3;
                    p[b][n][0] = transposed(pack_half(x0, x1));
                    p[b][n][1] = transposed(pack_half(x2, x3));
                }
            }
            // ---- outputs: dims 8 kR g + 2 j (and the next), rows 2 t and 2 t + 1
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t scale[kVScales][2];
#pragma unroll
                for (int i = 0; i < kVScales; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        scale[i][k] = e4m3_to_half((vs[4 * b + 2 * k] >> (8 * i) & 0xFF) |
                                                   (vs[4 * b + 2 * k + 1] >> (8 * i) & 0xFF) << 8);
#pragma unroll
                for (int w = 0; w < kR; ++w) {
                    // the word's group among the lane's scales; with kR odd it depends on whether v_first is
                    const int i0 = kR % 2 ? w / 2 : w / 2, i1 = kR % 2 ? (w + 1) / 2 : w / 2;
                    uint32_t h[2][2][4];  // [pair of keys][even, odd dims][byte]
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t x = vc[4 * b + 2 * k][w], y = vc[4 * b + 2 * k + 1][w];
                        const uint32_t u = i0 == i1 || !(v_first & 1) ? scale[i0 < kVScales ? i0 : 0][k]
                                                                      : scale[i1 < kVScales ? i1 : 0][k];
                        fp4_to_half((x & 0x0F0F0F0Fu) | (y << 4 & 0xF0F0F0F0u), h[k][0]);
                        fp4_to_half((x >> 4 & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), h[k][1]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            h[k][0][j] = half2_mul(h[k][0][j], u);
                            h[k][1][j] = half2_mul(h[k][1][j], u);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t f[4] = {h[0][0][j], h[0][1][j], h[1][0][j], h[1][1][j]};
#pragma unroll
                        for (int n = 0; n < kTiles; ++n) mma16816(o[n][4 * w + j], f, p[b][n][0], p[b][n][1]);
                    }
                }
            }
            load_values(next_page, next_place);
        }
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 4);
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 8);
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 16);
            }

        // Join the four warps.
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = n * 8 + 2 * t + i;
#pragma unroll
                for (int j = 0; j < 4 * kR; ++j)
                    *reinterpret_cast<float2 *>(&ow[warp][r][8 * kR * g + 2 * j]) = make_float2(o[n][j][i], o[n][j][2 + i]);
                if (g == 0) {
                    mw[warp][r] = m[n][i];
                    lw[warp][r] = l[n][i];
                }
            }
        __syncthreads();
        const bool whole = first == 0 && last == units;
        float *part = attn_slot(s, cta, first == 0 ? 1 : 0);
        for (int c = warp; c < dim / 8; c += kWarps) {  // 8 columns
            float ll[2] = {}, mm[2] = {-INFINITY, -INFINITY}, acc[4] = {};
#pragma unroll
            for (int k = 0; k < kTiles; ++k) {
                const int r = g + 8 * k;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) mm[k] = fmaxf(mm[k], mw[w][r]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = exp2_approx(mw[w][r] - attn_base(mm[k]));
                    const float2 x = *reinterpret_cast<const float2 *>(&ow[w][r][c * 8 + 2 * t]);
                    ll[k] += f * lw[w][r];
                    acc[2 * k] += f * x.x;
                    acc[2 * k + 1] += f * x.y;
                }
            }
            if (!whole) *attn_part(s, part, 0, c, lane) = make_float4(acc[0], acc[1], acc[2], acc[3]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = g + 8 * k;
                int token, head;
                if (whole && k < kTiles && attn_row(s, q.q0, q.n, cur.head, cur.row_tile, r, &token, &head)) {
                    const float inv = attn_inverse(ll[k]) * s.out_scale;
                    *reinterpret_cast<uint32_t *>((uint16_t *)a.out + token * a.out_token_stride + head * a.out_head_stride +
                                                  c * 8 + t * 2) = pack16(acc[2 * k] * inv, acc[2 * k + 1] * inv, bf16);
                }
                if (!whole && c == 0 && t == 0) {
                    part[kSlotRows * dim + r] = mm[k];
                    part[kSlotRows * dim + kSlotRows + r] = ll[k];
                }
            }
        }
        if (!whole && first == 0 && threadIdx.x == 0) {
            AttnJoin j = {};
            j.pieces = attn_pieces(s, cur, span, cta);
            j.seq = cur.seq;
            j.head = cur.head;
            j.row_tile = cur.row_tile;
            j.q0 = q.q0;
            j.q_len = q.n;
            attn_joins(s, ctas)[cta] = j;
        }
        cur.at += span.cost;
        cur.left -= span.cost;
        if (cur.left <= 0) break;
        attn_next(s, cur, q);
        __syncthreads();  // the join's reads are done before the next row tile's outputs are written
    }
}

// ------------------------------------------------------------------------------- host side

struct Attn4Plan {
    Attn4Args args;
    int ctas;
    const void *kernel;  // NULL: the tensor-core kernel
};

template <bool kWhole>
const void *rows_kernel(int r, int tiles) {
    switch (r) {
    case 1: return tiles == 1 ? (const void *)attn4_rows_kernel<1, 1, kWhole> : (const void *)attn4_rows_kernel<1, 2, kWhole>;
    case 2: return tiles == 1 ? (const void *)attn4_rows_kernel<2, 1, kWhole> : (const void *)attn4_rows_kernel<2, 2, kWhole>;
    case 3: return (const void *)attn4_rows_kernel<3, 1, kWhole>;
    default: return (const void *)attn4_rows_kernel<4, 1, kWhole>;
    }
}

// CTAs of a kernel that an SM holds, asked once per kernel and device.
int resident(const void *f) {
    static std::mutex mu;
    static std::unordered_map<uint64_t, int> known;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const uint64_t key = (uint64_t)(uintptr_t)f ^ (uint64_t)dev << 56;
    std::lock_guard<std::mutex> lock(mu);
    auto it = known.find(key);
    if (it != known.end()) return it->second;
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, f, kThreads, 0) != cudaSuccess) return 0;
    if (n > 0) known.emplace(key, n);
    return n;
}

// Query rows of a tile, in eights: 16 where head_dim leaves the registers and a sequence may have more than 8; 32,
// those of the tensor-core kernel, where it may have more than 16.
constexpr int kTc = 32;
int row_tiles(const ks_attention_args_t &a) {
    const int64_t q_len = a.max_q_len > 0 && a.max_q_len < a.tokens ? a.max_q_len : a.tokens;
    const int64_t rows = q_len * (a.q_heads / a.kv_heads);
    return a.head_dim > 128 || rows <= 8 ? 1 : rows <= 16 ? 2 : kTc;
}

ks_status_t plan4(const ks_attention_4bit_args_t &a, int tiles, uintptr_t code_align, uintptr_t scale_align, Attn4Plan *p) {
    AttnArgs &s = p->args.s;
    s.a = a.attention;
    s.scale_log2 = (float)((double)a.attention.scale * 1.4426950408889634 * (double)a.k_pages.factor);
    s.out_scale = a.v_pages.factor;
    p->args.k = pool4(a.k_pages);
    p->args.v = pool4(a.v_pages);
    const int dim = (int)s.a.head_dim, r = (dim + 63) / 64;
    int sms = 0;
    const ks_status_t st = device_sms(&sms);
    if (st != KS_SUCCESS) return st;
    if (tiles == kTc) {
        p->kernel = nullptr;
        attn_shape(&s, attn_tc_rows(), attn_tc_unit(), attn_tc_tile_cost());
        p->ctas = attn_ctas(s, sms);
        return KS_SUCCESS;
    }
    const uintptr_t codes = r % 4 == 0 || r == 2 ? 15 : 7, scales = r == 2 ? 1 : r == 4 ? 3 : 0;
    const bool whole = dim == 64 * r && (code_align & codes) == 0 && (scale_align & scales) == 0;
    p->kernel = whole ? rows_kernel<true>(r, tiles) : rows_kernel<false>(r, tiles);
    attn_shape(&s, 8 * tiles, kUnit, kTileCost);
    s.rows = kSlotRows;
    const int per_sm = resident(p->kernel);
    if (per_sm <= 0) return fail(KS_ERR_CUDA, "the attention kernel cannot be resident");
    p->ctas = attn_ctas(s, (int64_t)sms * per_sm);
    return KS_SUCCESS;
}

ks_status_t check_sizes4(const ks_attention_args_t &a) {
    const ks_status_t st = attn_check_sizes(a);
    if (st != KS_SUCCESS) return st;
    if (a.head_dim % 16) return fail(KS_ERR_INVALID_ARGUMENT, "4-bit pages take head_dims of whole groups of 16 (got %lld)", (long long)a.head_dim);
    return KS_SUCCESS;
}

ks_status_t check_tensors4(const ks_attention_4bit_args_t &args, uintptr_t *code_align, uintptr_t *scale_align) {
    const ks_attention_args_t &a = args.attention;
    if (!std::isfinite((float)((double)a.scale * 1.4426950408889634 * (double)args.k_pages.factor)) || !std::isfinite(a.scale))
        return fail(KS_ERR_INVALID_ARGUMENT, "scale (times log2 e and the keys' factor) must be finite");
    const ks_status_t st = check_pools4(args.k_pages, args.v_pages, a.tokens && a.seqs ? a.pages : 0, a.page_size, a.kv_heads,
                                        a.head_dim, false, code_align, scale_align);
    if (st != KS_SUCCESS || a.tokens == 0 || a.seqs == 0) return st;
    if (!a.out || !a.q || !a.kv_lens || !a.q_starts || (a.table_pages > 0 && !a.page_table))
        return fail(KS_ERR_INVALID_ARGUMENT, "NULL pointer with tokens > 0");
    if (misaligned(4, a.kv_lens, a.q_starts, a.page_table))
        return fail(KS_ERR_INVALID_ARGUMENT, "kv_lens, q_starts and page_table must be aligned to 4 bytes");
    const int64_t strides[] = {a.q_token_stride, a.q_head_stride, a.out_token_stride, a.out_head_stride};
    for (int i = 0; i < 4; ++i) {
        const int64_t count = i % 2 ? a.q_heads : a.tokens;
        if (strides[i] < 0 || (__int128)strides[i] * count > ((__int128)1 << 60))
            return fail(KS_ERR_INVALID_ARGUMENT, "a stride is negative or a tensor too large");
        if (count > 1 && strides[i] % 8)
            return fail(KS_ERR_INVALID_ARGUMENT, "strides of q and out must be multiples of 8 elements (16 bytes)");
    }
    if ((__int128)a.table_stride * a.seqs > ((__int128)1 << 60))
        return fail(KS_ERR_INVALID_ARGUMENT, "the page table is too large");
    if (((uintptr_t)a.q | (uintptr_t)a.out) & 15u)
        return fail(KS_ERR_INVALID_ARGUMENT, "q and out must be aligned to 16 bytes");
    if (!attn_out_apart(a)) return fail(KS_ERR_OVERLAP, "rows of out share storage");
    const int64_t out_bytes = attn_rows_bytes(a, a.out_token_stride, a.out_head_stride);
    if (overlaps(a.out, out_bytes, a.q, attn_rows_bytes(a, a.q_token_stride, a.q_head_stride)) ||
        crosses_pools4(args.k_pages, args.v_pages, a.pages, a.page_size, a.kv_heads, a.head_dim, a.out, out_bytes))
        return fail(KS_ERR_OVERLAP, "out overlaps q or the cache");
    if (attn_crosses_indices(a, {a.out, a.head_dim * 2, {a.tokens, a.q_heads, 1}, {a.out_token_stride * 2, a.out_head_stride * 2, 0}}))
        return fail(KS_ERR_OVERLAP, "out overlaps the page table, kv_lens or q_starts");
    return KS_SUCCESS;
}

}  // namespace

int fault_flags_attention_4bit(bool clear) { return fault_flags_t(clear); }

}  // namespace ks

using namespace ks;

extern "C" {

ks_status_t ks_paged_attention_4bit_workspace(const ks_attention_4bit_args_t *args, int64_t *bytes) {
    if (!args || !bytes) return fail(KS_ERR_INVALID_ARGUMENT, "args or bytes is NULL");
    *bytes = 0;
    ks_status_t st = check_sizes4(args->attention);
    if (st != KS_SUCCESS || args->attention.tokens == 0 || args->attention.seqs == 0) return st;
    // whichever kernel the pools' alignment, or fewer tokens, pick
    for (int tiles = row_tiles(args->attention); tiles > 0; tiles = tiles == kTc ? 2 : tiles - 1)
        for (uintptr_t align : {(uintptr_t)0, (uintptr_t)8}) {
            Attn4Plan p;
            if ((st = plan4(*args, tiles, align, align ? 1 : 0, &p)) != KS_SUCCESS) return st;
            const int64_t need = attn_workspace_bytes(p.args.s, p.ctas);
            *bytes = *bytes > need ? *bytes : need;
        }
    return KS_SUCCESS;
}

ks_status_t ks_paged_attention_4bit(const ks_attention_4bit_args_t *args, ks_stream_t stream) {
    if (!args) return fail(KS_ERR_INVALID_ARGUMENT, "args is NULL");
    const ks_attention_args_t &a = args->attention;
    uintptr_t code_align = 0, scale_align = 0;
    ks_status_t st = check_sizes4(a);
    if (st == KS_SUCCESS) st = check_tensors4(*args, &code_align, &scale_align);
    if (st != KS_SUCCESS || a.tokens == 0 || a.seqs == 0) return st;
    if (!a.workspace || ((uintptr_t)a.workspace & 15u))
        return fail(KS_ERR_INVALID_ARGUMENT, "the workspace must be device memory aligned to 16 bytes");
    Attn4Plan p;
    int tiles = row_tiles(a);
    if (tiles == kTc && !attn4_tc_fits(a)) tiles = 2;
    if ((st = plan4(*args, tiles, code_align, scale_align, &p)) != KS_SUCCESS) return st;
    const int64_t need = attn_workspace_bytes(p.args.s, p.ctas);
    if (a.workspace_bytes < need)
        return fail(KS_ERR_INVALID_ARGUMENT, "the workspace has %lld bytes, %lld are needed", (long long)a.workspace_bytes,
                    (long long)need);
    if (overlaps(a.workspace, need, a.out, attn_rows_bytes(a, a.out_token_stride, a.out_head_stride)) ||
        overlaps(a.workspace, need, a.q, attn_rows_bytes(a, a.q_token_stride, a.q_head_stride)) ||
        crosses_pools4(args->k_pages, args->v_pages, a.pages, a.page_size, a.kv_heads, a.head_dim, a.workspace, need) ||
        attn_crosses_indices(a, {a.workspace, need, {1, 1, 1}, {0, 0, 0}}))
        return fail(KS_ERR_OVERLAP, "the workspace overlaps out or what the call reads");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    void *kp[] = {&p.args};
    cudaError_t ce = p.kernel ? launch_kernel(p.kernel, dim3((unsigned)p.ctas), dim3(kThreads), 0, kp, s, launch_pdl_enabled())
                              : attn4_tc_launch(p.args, code_align, scale_align, p.ctas, s, launch_pdl_enabled());
    if (ce == cudaSuccess && p.ctas > 1) ce = attn_join_launch(p.args.s, p.ctas, s);
    if (ce != cudaSuccess) return fail(KS_ERR_CUDA, "launch: %s", cudaGetErrorString(ce));
    return KS_SUCCESS;
}

}  // extern "C"
