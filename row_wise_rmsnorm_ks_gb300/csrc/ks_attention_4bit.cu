// Attention of new tokens over a paged cache held in 4 bits: the kernel for few rows per key/value head, and the C
// entry points. The division of the work, the running maximum and the join are those of ks_attention.cu.
//
// Keys and values are fp16 numbers exactly (ks_fp4.cuh), so both products run as fp16 with FP32 sums. A bf16 query row
// is brought to a largest magnitude of 1 .. 2 by a power of two, which its scores are given back: values down to
// 2^-14 of the largest stay exact, smaller ones lose at most 2^-25 of it, less than an FP32 sum of the row's
// products does. Probabilities are fp16 too, 2^11 times as large as they are when a row's base is taken, and up to 2^15
// times as later scores outgrow it (kLift, kGrowth). The pools' factors go into the scores' scale and the output's, in FP32.
//
// Few rows make this a stream of the cache, 144 bytes per key of 128 values, and of the instructions that make fp16 of
// it: each pair of codes is a conversion and a product with its group's scale. So the matrix instructions
// take the cache as their 16-row operand, straight from registers, and the query rows as the 8 columns: S^T = K Q^T
// and O^T += V^T P^T, fp16 values never leaving the registers:
//   - K: a product's sum runs over any order of the dims, so the lane quad's member t takes dims t D / 4 and on of
//     two keys: one contiguous load a key. Queries lie in registers in the same order.
//   - V^T: rows may be any dims, so lane row g = lane / 4 has dims g D / 8 and on, of the four keys that the operand's
//     pairs want: the codes of two keys are merged by nibbles, and a conversion then gives a pair over keys.
//   - P^T comes from S^T by one 8x8 transposition of a matrix of 16-bit values for 8 keys.
// Row 2 t + e of a product's first 8 is key t + 4 e of its block, and so for the last 8, so that the lanes of a load have
// neighbouring keys.
// A warp runs alone on every fourth 32-key step, with its own ring of asynchronous copies in shared memory (no barrier
// in the loop; one ring for eight warps, which then wait for each other, takes 1.4 times as long; bulk copies, which
// lanes issue one after the other, take as many instructions as these). Pools that copies cannot take are loaded to
// registers a step ahead (kAny).
//
// Bound by instructions and latency together, at 60 % of the DRAM's cycles: a 32-key step is 588 instructions for 4608
// bytes of cache, an SM's 16 warps issue 2.4 a cycle, and finding the work, the first keys and the join take 20 us that no
// split shortens. Measured, 8 key/value heads of 128: 64 contexts of 700..8100 keys 83 us (53 at the copy rate; 203 with
// 16-bit pages), 4 of 131000 keys 128 us (87; 320), 1 token over 1001 keys 9.8 us (11.5). Heads with CTAs of their own
// read a page's heads together (where they lie token by token, 196 us become 128), and rings of asynchronous copies take 94
// where registers a step ahead take 98 and, with the bases kept and places looked up 16 at a time, 83.
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
// Exponentials are taken to a row's base, which lies kLift below the maximum of the scores when it was taken (in powers
// of two). It stays until a lane's probabilities outgrow it: most steps need no maximum. fp16 ends at 65504 and is
// normal down to 2^-14, so probabilities keep their precision down to 2^-25 of the row's largest and end at 2^-36.
constexpr float kLift = 11.0f, kGrowth = 32768.0f;

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
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

// kN words of codes, in groups of two where kN is even; those at and past `room` are zeros.
template <int kN>
__device__ __forceinline__ void load_codes(uint32_t (&w)[kN], const uint8_t *p, int room) {
    if constexpr (kN % 2 == 0) {
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) {
            uint2 x = make_uint2(0, 0);
            if (2 * i < room) x = __ldg(reinterpret_cast<const uint2 *>(p) + i);
            w[2 * i] = x.x, w[2 * i + 1] = x.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) w[i] = i < room ? __ldg(reinterpret_cast<const uint32_t *>(p) + i) : 0;
    }
}

// kN scales, one a byte of the result.
template <int kN>
__device__ __forceinline__ uint32_t load_scales(const uint8_t *p, int room) {
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if (i < room) x |= (uint32_t)__ldg(p + i) << (8 * i);
    return x;
}

// How pools lie:
//   kAny     any strides and page sizes, rows of any number of groups: each key's page is looked up on its own
//   kBlocks  head_dim is 64 kR, rows of codes and scales are aligned to what is copied of them at once, pages are whole
//            blocks of 16 keys, both pools have the same strides, those of the scales an eighth of the codes': a
//            block has one address. Copied by 16 bytes of codes and rows of scales.
//   kRuns    kBlocks with a head's keys one behind the other: a warp copies 512 bytes of a block's codes at once
enum { kAny, kBlocks, kRuns };

// (of a row's m below 8; rows 8 on are 8 keys on)
__device__ __forceinline__ int place(int m) { return (m >> 1) + 4 * (m & 1); }

// A warp's ring of steps: keys' codes, values' codes, keys' scales, values' scales.
template <int kR>
struct Ring {
    static constexpr int kStages = 3;
    static constexpr int kRow = 32 * kR, kScaleRow = 4 * kR;  // bytes of a key
    static constexpr int kCodes = kStep * kRow, kScales = kStep * kScaleRow;
    static constexpr int kStageBytes = 2 * (kCodes + kScales);
    // Byte of a 16-byte piece of a key's codes. Rows of 128 bytes all begin on one bank: where pieces are copied one by
    // one, they change places.
    template <int kPool>
    __device__ __forceinline__ static uint32_t piece(int key, int c) {
        return key * kRow + ((kR == 4 && kPool == kBlocks ? c ^ (key & 7) : c) << 4);
    }
};

template <int kR, int kTiles, int kPool>
struct Shared {
    static constexpr int kPitch = 64 * kR + 4;
    static constexpr int kJoin = kWarps * 8 * kTiles * kPitch * 4;  // the warps' outputs, over the rings
    static constexpr int kRingBytes = kPool != kAny ? kWarps * Ring<kR>::kStages * Ring<kR>::kStageBytes : 0;
    static constexpr int kBytes = kJoin > kRingBytes ? kJoin : kRingBytes;
};

template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, int n) {  // n of them, zeros behind
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(n) : "memory");
}

template <int kN>
__device__ __forceinline__ void shared_words(uint32_t (&w)[kN], const uint8_t *p) {
    if constexpr (kN == 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else if constexpr (kN == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x, w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
    }
}
template <int kN, bool kAligned = true>
__device__ __forceinline__ uint32_t shared_bytes(const uint8_t *p) {
    if constexpr (kN == 4) return *reinterpret_cast<const uint32_t *>(p);
    if constexpr (kN == 2 && kAligned) return *reinterpret_cast<const uint16_t *>(p);
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i) x |= (uint32_t)p[i] << (8 * i);
    return x;
}

// kR: 64 dims each; kTiles: tiles of 8 query rows.
template <int kR, int kTiles, int kPool>
__global__ void __launch_bounds__(kThreads, kPool == kAny ? (kR * kTiles == 1 ? 4 : kR * kTiles == 2 ? 3 : 2)
                                                          : (kR * kTiles <= 2 ? 4 : 2))
attn4_rows_kernel(const __grid_constant__ Attn4Args args) {
    using C = Ring<kR>;
    constexpr bool kWhole = kPool != kAny;
    constexpr int kWords = 2 * kR;                 // of a key's codes, for a quad's member
    constexpr int kVScales = (kR + 1) / 2;         // of a value's row, for a lane row
    constexpr int kRows = 8 * kTiles;
    constexpr int kPitch = Shared<kR, kTiles, kPool>::kPitch;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float mw[kWarps][kRows], lw[kWarps][kRows];
    float *ow = reinterpret_cast<float *>(smem);   // [kWarps][kRows][kPitch]
    const AttnArgs &s = args.s;
    const ks_attention_args_t &a = s.a;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int ctas = gridDim.x, cta = blockIdx.x;
    grid_dependency_wait();
    allow_dependents_launch();
    if (threadIdx.x == 0) attn_joins(s, ctas)[cta].pieces = 0;
    AttnCursor cur = attn_begin<kThreads>(s, cta, ctas);
    if (cur.left <= 0) return;
    uint32_t stage = 0;  // of the next step in the warp's ring
    AttnSeq q = attn_seq(a, cur.seq);

    const int dim = (int)a.head_dim, page_size = (int)a.page_size;
    const bool bf16 = a.dtype == KS_DTYPE_BF16, causal = (a.flags & KS_ATTENTION_CAUSAL) != 0;
    const int k_first = t * kR;                    // the lane's first group of a key
    const int v_first = g * kR;                    // its first word (8 dims) of a value
    const int k_room = 2 * (dim / 16 - k_first), v_room = dim / 8 - v_first;
    const int v_group = v_first / 2;
    uint8_t *ring = smem + warp * C::kStages * C::kStageBytes;
    // Where in a stage this lane's codes and scales of the first keys and values are.
    const int k_row = place(g), v_row = t;
    const uint32_t k_lane = k_row * C::kRow + (kR == 4 ? 0 : t * 8 * kR), v_lane = C::kCodes + v_row * C::kRow + (kR == 4 ? 0 : g * 4 * kR);
    const uint32_t k_scale_lane = 2 * C::kCodes + k_row * C::kScaleRow + k_first;
    const uint32_t v_scale_lane = 2 * C::kCodes + C::kScales + v_row * C::kScaleRow + v_group;
    // kR 4: the 16-byte pieces, which change places by the key's low bits (8 and 4 keys on: all of them, and one)
    auto piece = [&](int key, int c) { return (uint32_t)(kPool == kBlocks ? c ^ (key & 7) : c) << 4; };

    while (true) {
        const AttnSpan span = attn_span(s, cur, q);
        const int units = span.units, first = span.first, last = span.last;
        if (first >= last) break;  // the share ends in the tile's extra cost
        const int sees = attn_tile_keys(s, q, cur.row_tile);
        const int kv_head = cur.head / s.head_splits;
        const uint8_t *k_codes = args.k.codes + kv_head * args.k.code_head, *k_scales = args.k.scales + kv_head * args.k.scale_head;
        const uint8_t *v_codes = args.v.codes + kv_head * args.v.code_head, *v_scales = args.v.scales + kv_head * args.v.scale_head;
        if (!kWhole) {
            k_codes += k_first * 8;
            k_scales += k_first;
            v_codes += v_first * 4;
            v_scales += v_group;
        }
        const int32_t *table = a.page_table + (int64_t)cur.seq * a.table_stride;

        uint32_t kc[kWhole ? 2 : 4][kWords], ks[kWhole ? 2 : 4];  // kAny: of a step; otherwise of a block of 16
        uint32_t vc[kWhole ? 4 : 8][kR], vs[kWhole ? 4 : 8];
        const bool whole = first == 0 && last == units;
        const int end = min(sees, last * kUnit);  // steps at and past it are not this CTA's
        // ---- kAny: the page and the slot of key `lane` of a step, page -1 where there is no such key or its page is not
        // in the pool
        struct Where {
            int page, slot;
        };
        auto look_up = [&](int key_at) {
            Where w = {-1, 0};
            const int key = key_at + lane;
            if (!kWhole && key_at < end && key < sees) {
                const int index = key / page_size;
                w.slot = key - index * page_size;
                w.page = __ldg(table + index);
                if ((uint32_t)w.page >= (uint64_t)a.pages) {
                    atomicOr(&g_fault_flags, kFaultBadIndex);
                    w.page = -1;
                }
            }
            return w;
        };
        // ---- Otherwise the place of a block of 16 in the pool, in 16 bytes of codes or 2 of scales; kNone where there
        // is no key, or its page is not in the pool. A warp looks up those of 16 steps at once, two lanes a step, and as
        // many steps ahead: on its way through the steps a copy's address is then one multiplication.
        constexpr uint32_t kNone = 0xFFFFFFFFu;
        auto find = [&](int batch) {
            // (no sign: it looks some thousands of keys past the last, which may be the largest int but 1024)
            const uint32_t key = (uint32_t)first * kUnit + warp * kStep + (batch * 16 + lane / 2) * kUnit + lane % 2 * 16;
            if (key >= (uint32_t)end) return kNone;
            const uint32_t index = args.page_blocks.quotient(key >> 4);
            const int page = __ldg(table + index), slot = (int)(key - index * page_size);
            if ((uint32_t)page >= (uint64_t)a.pages) {
                atomicOr(&g_fault_flags, kFaultBadIndex);
                return kNone;
            }
            return (uint32_t)page * args.page_units + (uint32_t)slot * args.slot_units;
        };
        // What a lane copies: 16 bytes of codes kR times a block (kBlocks: of keys 16 / kR apart), of keys and values
        // each; scales by rows of a key (kBlocks) or 16 bytes (kRuns: keys' of both blocks, then values').
        constexpr int kScaleBytes = kPool == kRuns ? 16 : kR == 3 ? 4 : C::kScaleRow;
        constexpr int kPtrs = kPool == kRuns ? 1 : kR;
        const uint8_t *k_from[kPtrs], *v_from[kPtrs];
        uint32_t code_at[kR];  // in a block of the stage's codes
#pragma unroll
        for (int i = 0; i < kR; ++i) {
            const int in = i * 32 + lane, key = in / (2 * kR), c = in % (2 * kR);
            code_at[i] = C::template piece<kPool>(key, c);
            if (i < kPtrs) {
                const int64_t off = kPool == kRuns ? in * 16 : key * args.k.code_slot + c * 16;
                k_from[i] = k_codes + off;
                v_from[i] = v_codes + off;
            }
        }
        const uint8_t *ks_from = k_scales + lane % 16 * args.k.scale_slot, *vs_from = v_scales + lane % 16 * args.k.scale_slot;
        auto copy_step = [&](uint32_t places, int step, uint32_t to_stage) {
            const uint32_t to = smem_addr(ring) + to_stage * C::kStageBytes;
            uint32_t at[2] = {__shfl_sync(0xFFFFFFFFu, places, step % 16 * 2), __shfl_sync(0xFFFFFFFFu, places, step % 16 * 2 + 1)};
            auto copy = [&](const int (&n)[2]) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < kR; ++i) {
                        const uint32_t dst = to + b * 16 * C::kRow + code_at[i];
                        const int j = kPool == kRuns ? 0 : i, more = kPool == kRuns ? i * 512 : 0;
                        copy_async<16>(dst, k_from[j] + at[b] * 16ull + more, n[b]);
                        copy_async<16>(dst + C::kCodes, v_from[j] + at[b] * 16ull + more, n[b]);
                    }
                const uint32_t units = to + 2 * C::kCodes;
                if constexpr (kPool == kRuns) {
#pragma unroll
                    for (int i = 0; i < (kR + 1) / 2; ++i) {
                        const int in = i * 32 + lane, part = in / (4 * kR);
                        if (kR % 2 == 0 || in < 16 * kR)
                            copy_async<16>(units + in * 16,
                                           (part < 2 ? k_scales : v_scales) + (part & 1 ? at[1] : at[0]) * 2ull + in % (4 * kR) * 16,
                                           part & 1 ? n[1] : n[0]);
                    }
                } else {
                    const int of = (lane < 16 ? n[0] : n[1]) ? kScaleBytes : 0;
                    const uint64_t off = (lane < 16 ? at[0] : at[1]) * 2ull;
#pragma unroll
                    for (int i = 0; i < C::kScaleRow / kScaleBytes; ++i) {
                        const uint32_t dst = units + lane * C::kScaleRow + i * kScaleBytes;
                        copy_async<kScaleBytes>(dst, ks_from + off + i * kScaleBytes, of);
                        copy_async<kScaleBytes>(dst + C::kScales, vs_from + off + i * kScaleBytes, of);
                    }
                }
            };
            if (at[0] != kNone && at[1] != kNone) {
                copy({16, 16});
            } else {  // blocks without a place come out as zeros
                const int n[2] = {at[0] != kNone ? 16 : 0, at[1] != kNone ? 16 : 0};
                if (!n[0]) at[0] = 0;
                if (!n[1]) at[1] = 0;
                copy(n);
            }
        };
        auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
        // ---- kAny: loads of a step to registers
        auto load_keys = [&](const Where &w) {
#pragma unroll
            for (int i = 0; i < (kWhole ? 0 : 4); ++i) {
                const int at = 8 * i + place(g);
                const int64_t p = __shfl_sync(0xFFFFFFFFu, w.page, at), r = __shfl_sync(0xFFFFFFFFu, w.slot, at);
#pragma unroll
                for (int j = 0; j < kWords; ++j) kc[i][j] = 0;
                ks[i] = 0;
                if (p >= 0) {
                    load_codes<kWords>(kc[i], k_codes + p * args.k.code_page + r * args.k.code_slot, k_room);
                    ks[i] = load_scales<kR>(k_scales + p * args.k.scale_page + r * args.k.scale_slot, k_room / 2);
                }
            }
        };
        auto load_values = [&](const Where &w) {
#pragma unroll
            for (int i = 0; i < (kWhole ? 0 : 8); ++i) {
                const int at = 8 * (i / 2) + t + 4 * (i % 2);
                const int64_t p = __shfl_sync(0xFFFFFFFFu, w.page, at), r = __shfl_sync(0xFFFFFFFFu, w.slot, at);
#pragma unroll
                for (int j = 0; j < kR; ++j) vc[i][j] = 0;
                vs[i] = 0;
                if (p >= 0) {
                    load_codes<kR>(vc[i], v_codes + p * args.v.code_page + r * args.v.code_slot, v_room);
                    vs[i] = load_scales<kVScales>(v_scales + p * args.v.scale_page + r * args.v.scale_slot,
                                                         dim / 16 - v_group);
                }
            }
        };

        int key0 = first * kUnit + warp * kStep;
        Where next = {-1, 0};
        uint32_t places = kNone, more_places = kNone;
        int copied = 0;  // steps
        auto copy_next = [&](uint32_t to_stage) {
            if (copied && copied % 16 == 0) {
                places = more_places;
                more_places = find(copied / 16 + 1);
            }
            copy_step(places, copied++, to_stage);
        };
        if constexpr (kWhole) {
            places = find(0);
            more_places = find(1);
#pragma unroll
            for (int i = 0; i < C::kStages - 1; ++i) {
                copy_next(stage + i < C::kStages ? stage + i : stage + i - C::kStages);
                commit();
            }
        } else {
            next = look_up(key0);
            load_keys(next);
            load_values(next);
        }

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

        for (; key0 < end; key0 += kUnit) {
            const uint8_t *tile = ring + stage * C::kStageBytes;
            if constexpr (kWhole) {
                if (key0 + (C::kStages - 1) * kUnit < end) copy_next(stage ? stage - 1 : C::kStages - 1);
                commit();
                asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 1) : "memory");
                __syncwarp();
                if (++stage == C::kStages) stage = 0;
            } else {
                next = look_up(key0 + kUnit);
            }
            // ---- scores of 32 keys: key place(g) of block b (and 8 on), rows 2 t and 2 t + 1
            float sc[2][kTiles][4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int of = kWhole ? 0 : 2 * b;  // the block's keys among those in registers
                if constexpr (kWhole) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint8_t *at = tile + k_lane + (16 * b + 8 * i) * C::kRow;
                        if constexpr (kR == 4) {
                            uint32_t x[4], y[4];
                            shared_words(x, at + piece(k_row, 2 * t));
                            shared_words(y, at + piece(k_row, 2 * t + 1));
#pragma unroll
                            for (int j = 0; j < 4; ++j) kc[i][j] = x[j], kc[i][4 + j] = y[j];
                        } else if constexpr (kR == 3) {
#pragma unroll
                            for (int j = 0; j < 3; ++j) {
                                uint32_t x[2];
                                shared_words(x, at + 8 * j);
                                kc[i][2 * j] = x[0], kc[i][2 * j + 1] = x[1];
                            }
                        } else {
                            shared_words(kc[i], at);
                        }
                        ks[i] = shared_bytes<kR>(tile + k_scale_lane + (16 * b + 8 * i) * C::kScaleRow);
                    }
                }
#pragma unroll
                for (int n = 0; n < kTiles; ++n) sc[b][n][0] = sc[b][n][1] = sc[b][n][2] = sc[b][n][3] = 0.0f;
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    uint32_t scale[2], h[2][8];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        scale[i] = e4m3_to_half(__byte_perm(ks[of + i], 0, r | r << 4));
                        uint32_t x[4];
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            fp4_to_half(kc[of + i][2 * r + w], x);
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
            if (!kWhole) load_keys(next);
            // ---- probabilities
            const bool masked = key0 + kStep > all_see;
            uint32_t p[2][kTiles][2];
#pragma unroll
            for (int n = 0; n < kTiles; ++n) {
                float sum[2];
                // to the rows' old bases; again, with new ones, where a row has outgrown its base or has none yet
                bool fresh = false;
                while (true) {
                    const float base[2] = {attn_base(m[n][0]), attn_base(m[n][1])};
                    float x[2][4];
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[b][i] = __fmaf_rn(sc[b][n][i], mul[n][i & 1], -base[i & 1]);
                    if (masked) {
                        __syncwarp();
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (key0 + 16 * b + 8 * (i / 2) + k_row >= limit[n][i & 1]) x[b][i] = -INFINITY;
                    }
                    sum[0] = sum[1] = 0.0f;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            x[b][i] = exp2_approx(x[b][i]);
                            sum[i & 1] += x[b][i];
                        }
                        p[b][n][0] = pack_half(x[b][0], x[b][1]);
                        p[b][n][1] = pack_half(x[b][2], x[b][3]);
                    }
                    if (fresh || !__any_sync(0xFFFFFFFFu, !(fmaxf(sum[0], sum[1]) <= kGrowth) ||
                                                              fminf(m[n][0], m[n][1]) == -INFINITY))
                        break;
                    fresh = true;
                    float f[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float top = -INFINITY;
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int i = k; i < 4; i += 2) {
                                const float y = sc[b][n][i] * mul[n][k];
                                if (!masked || key0 + 16 * b + 8 * (i / 2) + k_row < limit[n][k]) top = fmaxf(top, y);
                            }
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
                        top = fmaxf(m[n][k], fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16)) - kLift);
                        f[k] = exp2_approx(m[n][k] - attn_base(top));
                        l[n][k] *= f[k];
                        m[n][k] = top;
                    }
#pragma unroll
                    for (int i = 0; i < 4 * kR; ++i) {
                        o[n][i][0] *= f[0];
                        o[n][i][1] *= f[1];
                        o[n][i][2] *= f[0];
                        o[n][i][3] *= f[1];
                    }
                }
                l[n][0] += sum[0];
                l[n][1] += sum[1];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    p[b][n][0] = transposed(p[b][n][0]);
                    p[b][n][1] = transposed(p[b][n][1]);
                }
            }
            // ---- outputs: dims 8 kR g + 2 j (and the next), rows 2 t and 2 t + 1
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int of = kWhole ? 0 : 4 * b;
                if constexpr (kWhole) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = 16 * b + 8 * (i / 2) + 4 * (i % 2);  // and v_row on
                        shared_words(vc[i], tile + v_lane + key * C::kRow + (kR == 4 ? piece(v_row + 4 * (i % 2), g) : 0));
                        vs[i] = shared_bytes<kVScales, kR % 2 == 0>(tile + v_scale_lane + key * C::kScaleRow);
                    }
                    // A scale behind the last key that the tile sees may be anything, and a probability of 0 would let
                    // a NaN through. (Its key's score is masked whatever it is.)
                    if (key0 + kStep > sees) {
                        __syncwarp();  // a branch, not selections in every step
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (key0 + 16 * b + 8 * (i / 2) + 4 * (i % 2) + v_row >= sees) vs[i] = 0;
                    }
                }
                uint32_t scale[kVScales][2];
#pragma unroll
                for (int i = 0; i < kVScales; ++i)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        scale[i][k] = e4m3_to_half(__byte_perm(vs[of + 2 * k], vs[of + 2 * k + 1], i | (4 + i) << 4));
#pragma unroll
                for (int w = 0; w < kR; ++w) {
                    // the word's group among the lane's scales; with kR odd it depends on whether v_first is
                    const int i0 = w / 2, i1 = kR % 2 ? (w + 1) / 2 : w / 2;
                    uint32_t h[2][2][4];  // [pair of keys][even, odd dims][byte]
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t x = vc[of + 2 * k][w], y = vc[of + 2 * k + 1][w];
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
            if (kWhole) __syncwarp();  // all lanes have read the stage before it is refilled
            else load_values(next);
        }
        if (kWhole) asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 4);
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 8);
                l[n][i] += __shfl_xor_sync(0xFFFFFFFFu, l[n][i], 16);
            }

        // Join the four warps, over the rings.
        if (kWhole) __syncthreads();
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = n * 8 + 2 * t + i;
#pragma unroll
                for (int j = 0; j < 4 * kR; ++j)
                    *reinterpret_cast<float2 *>(ow + (warp * kRows + r) * kPitch + 8 * kR * g + 2 * j) =
                        make_float2(o[n][j][i], o[n][j][2 + i]);
                if (g == 0) {
                    mw[warp][r] = m[n][i];
                    lw[warp][r] = l[n][i];
                }
            }
        __syncthreads();
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
                    const float2 x = *reinterpret_cast<const float2 *>(ow + (w * kRows + r) * kPitch + c * 8 + 2 * t);
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
    int smem;
};

template <int kR, int kTiles, int kPool>
const void *rows_kernel(int *smem) {
    *smem = Shared<kR, kTiles, kPool>::kBytes;
    return (const void *)attn4_rows_kernel<kR, kTiles, kPool>;
}

template <int kPool>
const void *rows_kernel(int r, int tiles, int *smem) {
    switch (r) {
    case 1: return tiles == 1 ? rows_kernel<1, 1, kPool>(smem) : rows_kernel<1, 2, kPool>(smem);
    case 2: return tiles == 1 ? rows_kernel<2, 1, kPool>(smem) : rows_kernel<2, 2, kPool>(smem);
    case 3: return rows_kernel<3, 1, kPool>(smem);
    default: return rows_kernel<4, 1, kPool>(smem);
    }
}

// CTAs of a kernel that an SM holds, asked once per kernel and device.
int resident(const void *f, int smem) {
    static std::mutex mu;
    static std::unordered_map<uint64_t, int> known;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const uint64_t key = (uint64_t)(uintptr_t)f ^ (uint64_t)dev << 56;
    std::lock_guard<std::mutex> lock(mu);
    auto it = known.find(key);
    if (it != known.end()) return it->second;
    int n = 0;
    if (!allow_smem(f, (size_t)smem)) return 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, f, kThreads, (size_t)smem) != cudaSuccess) return 0;
    if (n > 0) known.emplace(key, n);
    return n;
}

// Query rows of a tile, in eights: 16 where head_dim leaves the registers and a sequence may have more than 8; 32, the
// tensor-core kernel's, where it may have more than `most`: its row tiles begin and end in the time of 5 of their steps, and it
// makes fp16 tiles of all keys for however few rows, where each 16 rows of the other kernel read and convert them again.
// Above 128 dims, which no tensor-core kernel takes, 8 rows whatever their number: at 256 dims two tiles take all 255 registers
// and spill 88 to 692 bytes. (Measured, us, 8 rows and 16. 256 dims, 32 / 2 heads: one context of 100000 keys 46, 52; 64 of
// 4000 keys 76, 63; 16 / 4 heads, 2048 tokens over 8192 keys 1441, 997; 192 dims 1160, 757. So 16 rows would pay but for one
// context, and tensor cores more for prompts; both are left.)
constexpr int kTc = 32;
int row_tiles(const ks_attention_args_t &a, int most) {
    const int64_t q_len = a.max_q_len > 0 && a.max_q_len < a.tokens ? a.max_q_len : a.tokens;
    const int64_t rows = q_len * (a.q_heads / a.kv_heads);
    return a.head_dim > 128 || rows <= 8 ? 1 : rows <= most ? 2 : kTc;
}

// Whether both pools have the same strides, those of the scales an eighth of the codes', and a place in them is 32 bits of
// 16-byte units.
bool pools_alike(const ks_attention_4bit_args_t &args) {
    const ks_attention_args_t &a = args.attention;
    const ks_pages_4bit_t &k = args.k_pages, &v = args.v_pages;
    // an axis of one entry has any stride
    auto same = [](int64_t count, int64_t x, int64_t y, int64_t xs, int64_t ys) {
        return count == 1 || (x == y && xs == ys && x == 8 * xs && x % 16 == 0);
    };
    return a.pages > 0 && same(a.pages, k.code_page_stride, v.code_page_stride, k.scale_page_stride, v.scale_page_stride) &&
           same(a.page_size, k.code_slot_stride, v.code_slot_stride, k.scale_slot_stride, v.scale_slot_stride) &&
           (((__int128)(a.pages - 1) * k.code_page_stride + (a.page_size - 1) * k.code_slot_stride) >> 4) < 0xFFFFFFFFll;
}

// How the pools of a call lie, given the alignment of their addresses.
int pool_kind(const ks_attention_4bit_args_t &args, uintptr_t code_align, uintptr_t scale_align) {
    const ks_attention_args_t &a = args.attention;
    const ks_pages_4bit_t &k = args.k_pages, &v = args.v_pages;
    const int64_t r = a.head_dim / 64;
    if (a.head_dim % 64 || a.page_size % 16 || !pools_alike(args)) return kAny;
    const uintptr_t scales = r == 2 ? 7 : r == 4 ? 15 : 3;
    if ((code_align & 15) || (scale_align & scales)) return kAny;
    if (k.code_slot_stride != 32 * r) return kBlocks;
    uintptr_t runs = 0;  // a block of scales is copied by 16 bytes too
    for (const ks_pages_4bit_t *p : {&k, &v})
        runs |= (uintptr_t)p->scales | (uintptr_t)(a.pages > 1 ? p->scale_page_stride : 0) |
                (uintptr_t)(a.kv_heads > 1 ? p->scale_head_stride : 0);
    return runs & 15 ? kBlocks : kRuns;
}

// Rows up to which 16-row tiles pay. (Measured, us, 16-row tiles and tensor cores, 64 contexts of 4000 keys, 32 / 8 heads,
// pages of 16 keys, or of 24 where it says so. Rings: 128 dims, 32 rows 171, 210; 48 245, 212; 64 dims, 48 151, 174; 64 192, 175.
// Where 16-row tiles load to registers and the tensor cores' codes come by maps: 96 dims, 24 rows 384, 207; 32 dims 192, 172; by 16
// bytes: 128 dims in 24s, 24 rows 396, 205; 64 dims in 24s 204, 161; by 8: 96 dims in 24s, 32 rows 380, 457; 48 557, 460; 128 dims,
// unaligned, 32 415, 467; 48 611, 469; 80 dims, 32 381, 454; 48 556, 455; 48 dims, 32 200, 241; 48 287, 242.)
int most_rows(const ks_attention_4bit_args_t &args, int pool, uintptr_t code_align, uintptr_t scale_align) {
    const ks_attention_args_t &a = args.attention;
    if (pool != kAny) return a.head_dim > 64 ? 32 : 48;
    return attn4_tc_copies(a, pool4(args.k_pages), pool4(args.v_pages), pools_alike(args), code_align, scale_align) == kCopyBy8 ? 32 : 16;
}

ks_status_t plan4(const ks_attention_4bit_args_t &a, int tiles, int pool, Attn4Plan *p) {
    AttnArgs &s = p->args.s;
    s.a = a.attention;
    s.scale_log2 = (float)((double)a.attention.scale * 1.4426950408889634 * (double)a.k_pages.factor);
    s.out_scale = a.v_pages.factor;
    s.lanes = 1;
    p->args.k = pool4(a.k_pages);
    p->args.v = pool4(a.v_pages);
    const int dim = (int)s.a.head_dim, r = (dim + 63) / 64;
    int sms = 0;
    const ks_status_t st = device_sms(&sms);
    if (st != KS_SUCCESS) return st;
    p->args.alike = pools_alike(a);
    p->args.page_units = (uint32_t)(a.k_pages.code_page_stride / 16);
    p->args.slot_units = (uint32_t)(a.k_pages.code_slot_stride / 16);
    if (tiles == kTc) {
        p->kernel = nullptr;
        attn_shape(&s, attn_tc_rows(), attn_tc_unit(), attn4_tc_tile_cost());
        p->ctas = attn_ctas(s, sms);
        return KS_SUCCESS;
    }
    p->kernel = pool == kRuns     ? rows_kernel<kRuns>(r, tiles, &p->smem)
                : pool == kBlocks ? rows_kernel<kBlocks>(r, tiles, &p->smem)
                                  : rows_kernel<kAny>(r, tiles, &p->smem);
    p->args.page_blocks = Divisor::of((uint32_t)(s.a.page_size / 16));
    attn_shape(&s, 8 * tiles, kUnit, kTileCost);
    s.rows = kSlotRows;
    const int per_sm = resident(p->kernel, p->smem);
    if (per_sm <= 0) return fail(KS_ERR_CUDA, "the attention kernel cannot be resident");
    p->ctas = attn_ctas(s, (int64_t)sms * per_sm);
    // Heads with CTAs of their own, unless that leaves more than a tenth of the CTAs without work.
    const int64_t heads = s.a.kv_heads * s.head_splits, used = p->ctas / heads * heads;
    if (heads > 1 && used * 10 >= (int64_t)p->ctas * 9) {
        p->ctas = (int)used;
        s.lanes = (int)heads;
    }
    return KS_SUCCESS;
}

ks_status_t check_sizes4(const ks_attention_args_t &a) {
    const ks_status_t st = attn_check_sizes(a);
    if (st != KS_SUCCESS) return st;
    if (a.head_dim % 16)
        return fail(KS_ERR_INVALID_ARGUMENT, "4-bit pages take head_dims of whole groups of 16 (got %lld)", (long long)a.head_dim);
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
    // whichever kernel the pools' layout, or fewer tokens, pick
    for (int tiles = row_tiles(args->attention, 16); tiles > 0; tiles = tiles == kTc ? 2 : tiles - 1)
        for (int pool : {kAny, kBlocks, kRuns}) {
            Attn4Plan p;
            if ((st = plan4(*args, tiles, pool, &p)) != KS_SUCCESS) return st;
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
    const int pool = pool_kind(*args, code_align, scale_align);
    int tiles = row_tiles(a, most_rows(*args, pool, code_align, scale_align));
    if (tiles == kTc && !attn4_tc_fits(a)) tiles = 2;
    if ((st = plan4(*args, tiles, pool, &p)) != KS_SUCCESS) return st;
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
    cudaError_t ce = p.kernel ? launch_kernel(p.kernel, dim3((unsigned)p.ctas), dim3(kThreads), (size_t)p.smem, kp, s,
                                              launch_pdl_enabled())
                              : attn4_tc_launch(p.args, code_align, scale_align, p.ctas, s, launch_pdl_enabled());
    if (ce == cudaSuccess && p.ctas > 1) ce = attn_join_launch(p.args.s, p.ctas, s);
    if (ce != cudaSuccess) return fail(KS_ERR_CUDA, "launch: %s", cudaGetErrorString(ce));
    return KS_SUCCESS;
}

}  // extern "C"
