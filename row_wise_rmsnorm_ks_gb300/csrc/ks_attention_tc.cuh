// Paged attention on the fifth-generation tensor cores: the kernel, for caches of 16 and of 4 bits. Its structure is
// described in ks_attention_tc.cu, what 4-bit pages change in ks_attention_4bit_tc.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "ks_attention.cuh"
#include "ks_fp4.cuh"

namespace ks {

// The queries as columns, heads, tokens; boxes of 64 columns, a row tile's heads and its tokens.
bool attn_query_map(CUtensorMap *map, const AttnArgs &s);
// A pool's codes as bytes of a row, slots, heads, pages; boxes of a head's rows that lie together.
bool attn_codes_map(CUtensorMap *map, const AttnArgs &s, const Pool4 &pool);

namespace {

constexpr int kTile = 128;         // rows of a matrix tile
constexpr int kRows = 2 * kTile;   // rows of a row tile
constexpr int kKeys = 128;         // keys of a step
constexpr int kTileThreads = 2 * kTile;  // softmax threads of a tile: 16 rows a warp
constexpr int kSoftmaxWarps = 2 * kTileThreads / 32;
constexpr int kMma = kSoftmaxWarps, kCopy = kMma + 1, kTail = kMma + 3;  // the other warps (kMma + 2: see there)
constexpr int kConvert = kMma + 4, kConvertWarps = 4;  // the warps that make 16-bit tiles of 4-bit pages
// Threads and registers. 16-bit pages: 640 threads launch with 96 registers each; the softmax warpgroups take 104
// (64 scores a thread and their probabilities), the last keeps 64. 4-bit pages: 768 launch with 80.
template <bool k4>
struct Split {
    static constexpr int kThreads = 2 * kTileThreads + 128 + (k4 ? kConvertWarps * 32 : 0);
    static constexpr int kLaunchRegs = k4 ? 80 : 96, kSoftmaxRegs = k4 ? 96 : 104, kOtherRegs = k4 ? 40 : 64;
    static constexpr int kConvertRegs = 56;
    static_assert(2 * kTileThreads * kSoftmaxRegs + 128 * kOtherRegs + (k4 ? kConvertWarps * 32 * kConvertRegs : 0) <=
                      kThreads * kLaunchRegs, "the split draws on the launch's registers");
};
// What a kernel reads keys and values from.
struct Pages16 {
    static constexpr bool k4 = false;
    CUtensorMap k, v;
};
struct Pages4 {
    static constexpr bool k4 = true;
    Pool4 k, v;
    // Rows are kDim / 2 bytes of codes at 16-byte boundaries and kDim / 16 of scales at as many, both pools lie alike, and a
    // place has 32 bits of 16-byte units: the strides of pages and slots in those.
    int32_t whole;
    uint32_t page_units, slot_units;
    // A step's keys are whole pages or part of one, rows of codes are at 16-byte boundaries, of scales at 2: the copying warp
    // brings the codes, by these maps.
    int32_t by_map;
    CUtensorMap k_map, v_map;
};
constexpr int kHalfBytes = kKeys * 128;  // 128 rows of 64 values
constexpr int kTileCost = 3;       // steps that beginning and ending a row tile costs
// The exponent of a probability at the base, and the most that a lane's 32 to an old base may sum to.
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 8.0f : 0.0f;
template <typename T>
constexpr float kGrowth = std::is_same<T, __half>::value ? 65504.0f : 16384.0f;

template <int kDim, bool k4 = false>
struct Tc {
    static constexpr int kHalves = kDim / 64;
    static constexpr int kTileBytes = kHalves * kHalfBytes;  // a tile of Q, K or V
    static constexpr int kStages = kDim == 128 ? (k4 ? 4 : 5) : (k4 ? 8 : 10);
    static constexpr int kBars = (k4 ? 2 : 3) * kStages + 14 + (k4 ? 2 * 3 : 0);
    // 4-bit pages: each converting warp's ring of rows as the pools hold them, codes and scales; rows 16 bytes apart from a
    // multiple of 32, so that eight lanes read 16 bytes of theirs without a conflict.
    static constexpr int kRawStages = 3, kRawRow = kDim / 2 + 16;
    // In one ring for all of them, what the copies by map bring: rows end to end, 16-byte pieces swizzled.
    static constexpr int kRawAt = (2 + kStages) * kTileBytes + (kBars * 8 + 16 + 511) / 512 * 512;
    static constexpr int kRawTile = kKeys * kDim / 2;
    static_assert(kRawTile <= kConvertWarps * 32 * kRawRow, "both rings lie in the same place");
    static constexpr int kSmem = 1024 + (k4 ? kRawAt + kConvertWarps * kRawStages * 32 * kRawRow
                                            : (2 + kStages) * kTileBytes + (kBars * 8 + 16));
    static constexpr uint32_t kO = 256;  // tensor-memory columns: S0 0, S1 128, then the O tiles
};

// ---- tensor-core primitives

// Shared-memory operands are described by two words. Low: the address and, for an operand whose rows
// are the product's K dimension, the distance of its 64-value blocks (both over 16); an offset within
// the tile is added to it. High: 128-byte swizzle, groups of 8 rows 1024 bytes apart.
constexpr uint32_t kDescHigh = 1024 >> 4 | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lead) { return addr >> 4 | (lead >> 4) << 16; }

// FP32 accumulators, both operands of T, M = 128, N = n; bit 16: B's rows are its K dimension.
template <typename T>
__host__ __device__ constexpr uint32_t mma_shape(int n, bool b_by_rows) {
    const uint32_t t = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    return 1u << 4 | t << 7 | t << 10 | (b_by_rows ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 |
           (uint32_t)(kTile / 16) << 24;
}

// One step of 16 along K: D (+)= A B, A in shared or tensor memory.
template <bool kAdd>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t shape) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %5, 0;\n\t"
        "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "n"(kDescHigh),
        "r"(shape), "n"((int)kAdd)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t shape, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 y, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "n"(kDescHigh),
        "r"(shape), "r"(add)
        : "memory");
}
// Arrives on `bar` when all matrix instructions this thread issued so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define KS_R4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
#define KS_W4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])

// 16 rows of tensor memory: the quad lane / 4 has rows lane / 4 and lane / 4 + 8. Of every 8 columns a
// lane has columns 2 (lane % 4) and the next of the first row, then those of the second. 64 columns.
__device__ __forceinline__ void tmem_load_rows32(uint32_t (&r)[32], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : KS_W4(r, 0), KS_W4(r, 4), KS_W4(r, 8), KS_W4(r, 12), KS_W4(r, 16), KS_W4(r, 20), KS_W4(r, 24), KS_W4(r, 28)
        : "r"(addr));
}
// 32 columns.
__device__ __forceinline__ void tmem_load_rows16(uint32_t (&r)[16], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : KS_W4(r, 0), KS_W4(r, 4), KS_W4(r, 8), KS_W4(r, 12)
        : "r"(addr));
}
// 32 columns of two 16-bit values each: of every 4, a lane has column lane % 4 of both rows, which is
// where the pairs it loaded belong.
__device__ __forceinline__ void tmem_store_rows16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(addr),
        KS_R4(r, 0), KS_R4(r, 4), KS_R4(r, 8), KS_R4(r, 12)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the lane's two rows times f and g, in place.
__device__ __forceinline__ void tmem_scale_rows(uint32_t addr, float f, float g) {
    uint32_t r[16];
    tmem_load_rows16(r, addr);
    tmem_wait_load();
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * (i & 2 ? g : f));
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(addr),
        KS_R4(r, 0), KS_R4(r, 4), KS_R4(r, 8), KS_R4(r, 12)
        : "memory");
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int col, int slot, int head, int page,
                                         uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst), "l"(map), "r"(col), "r"(slot), "r"(head), "r"(page), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void bar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// One arrival for the warp: 32 arrivals of lanes would be worked off one after the other, in shared
// memory that the matrix instructions read from (measured: a fifth of the kernel's time).
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if (threadIdx.x % 32 == 0) bar_arrive(bar);
}

// One try that may sleep up to 20 us: warps that wait take no issue slots from those that compute.
__device__ __forceinline__ bool bar_sleep(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return done != 0;
}

// Waits for phase `parity`; false when the wait's limit passed or another role gave up. The role
// then leaves its loop: everybody meets at the kernel's end, with the fault word set.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *gave_up) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (!bar_sleep(bar, parity)) {
        if (*gave_up) return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            atomicOr(&g_fault_flags, kFaultWaitTimeout);
            *gave_up = 1;
            return false;
        }
    }
    return true;
}

// The same by a whole warp, with one answer for all lanes.
__device__ __forceinline__ bool bar_wait_warp(uint64_t *bar, uint32_t parity, volatile uint32_t *gave_up) {
    return __all_sync(0xFFFFFFFFu, bar_wait(bar, parity, gave_up));
}

// Lane 0's value, which the compiler then knows to be the same in all lanes: what the matrix
// instructions are given stays in uniform registers.
__device__ __forceinline__ int warp_uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float x, float y) {
    uint32_t w;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        memcpy(&w, &h, 4);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        memcpy(&w, &h, 4);
    }
    return w;
}

// Word i of lane q of a quad becomes word q of lane i.
__device__ __forceinline__ void quad_transpose(uint32_t (&y)[4], int q) {
    // pairs of words between lanes two apart, then words between neighbours
    const uint32_t a = __shfl_xor_sync(0xFFFFFFFFu, q & 2 ? y[0] : y[2], 2);
    const uint32_t b = __shfl_xor_sync(0xFFFFFFFFu, q & 2 ? y[1] : y[3], 2);
    if (q & 2) {
        y[0] = a;
        y[1] = b;
    } else {
        y[2] = a;
        y[3] = b;
    }
    const uint32_t c = __shfl_xor_sync(0xFFFFFFFFu, q & 1 ? y[0] : y[1], 1);
    const uint32_t d = __shfl_xor_sync(0xFFFFFFFFu, q & 1 ? y[2] : y[3], 1);
    if (q & 1) {
        y[0] = c;
        y[2] = d;
    } else {
        y[1] = c;
        y[3] = d;
    }
}

// A place in the ring of tiles and the phase of its barriers there.
template <int kStages>
struct RingAt {
    uint32_t stage = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// Each warp keeps its place in the CTA's work in shared memory: it is needed once per row tile, and the
// softmax has no registers to spare for it.
struct Place {
    AttnCursor cur;
    AttnSeq q;
};

// Whether the row tile's second tile has rows.
__device__ __forceinline__ bool second_tile(const AttnArgs &s, const Place &p) {
    return min(s.tile_tokens, p.q.n - p.cur.row_tile * s.tile_tokens) * s.tile_heads > kTile;
}

// Goes on to the CTA's next row tile; false when its share is done. All lanes of the warp call it.
__device__ __forceinline__ bool next_tile(const AttnArgs &s, Place &p, int cost) {
    __syncwarp();
    if (threadIdx.x % 32 == 0) {
        p.cur.at += cost;
        p.cur.left -= cost;
        if (p.cur.left > 0) attn_next(s, p.cur, p.q);
    }
    __syncwarp();
    return p.cur.left > 0;
}

// bf16 queries made fp16 where they lie: a warp's 16 rows from `first` on, two lanes a row. A row is multiplied by the
// power of two that brings its largest magnitude to 1 .. 2; its inverse is the row's unit (2^-126 .. 2^126). Returns
// the units of the rows lane / 4 and lane / 4 + 8.
template <int kDim>
__device__ __forceinline__ void make_queries(uint8_t *q_tile, int first, float (&unit)[2]) {
    constexpr int kChunks = kDim / 16;  // 16-byte pieces of a lane: half of a row
    const int lane = threadIdx.x % 32, row = first + lane % 16, part = lane / 16;
    uint8_t *at = q_tile + (kDim == 128 ? part * kRows * 128 : 0) + row * 128;
    const int c0 = kDim == 128 ? 0 : part * kChunks;
    uint4 x[kChunks];
    float big = 0.0f;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        x[c] = *reinterpret_cast<const uint4 *>(at + (((c0 + c) ^ (row & 7)) << 4));
        float f[8];
        Elem<__nv_bfloat16>::unpack(x[c], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(f[i]));
    }
    big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 16));
    const uint32_t e = min(max(__float_as_uint(big) >> 23, 1u), 253u);
    const float inverse = __uint_as_float((254u - e) << 23);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        float f[8];
        Elem<__nv_bfloat16>::unpack(x[c], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= inverse;
        *reinterpret_cast<uint4 *>(at + (((c0 + c) ^ (row & 7)) << 4)) = Elem<__half>::pack(f);
    }
    const float mine = __uint_as_float(e << 23);
    unit[0] = __shfl_sync(0xFFFFFFFFu, mine, lane / 4);
    unit[1] = __shfl_sync(0xFFFFFFFFu, mine, lane / 4 + 8);
}

// A row of 4-bit values made fp16 in the layout that the matrix instructions read: `piece` gives 16 bytes of codes.
template <int kDim, typename Piece>
__device__ __forceinline__ void convert_row(uint8_t *tile, int row, const uint32_t (&scales)[kDim / 64], Piece piece) {
#pragma unroll
    for (int i = 0; i < kDim / 32; ++i) {  // two groups
        const uint4 x = piece(i);
        const uint32_t words[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = 4 * i + k, g = c / 2;
            const uint32_t scale = e4m3_to_half(__byte_perm(scales[g / 4], 0, (g % 4) | (g % 4) << 4));
            uint32_t h[4];
            fp4_to_half(words[k], h);
#pragma unroll
            for (int n = 0; n < 4; ++n) h[n] = half2_mul(h[n], scale);
            *reinterpret_cast<uint4 *>(tile + row * 128 + c / 8 * kHalfBytes + ((c % 8 ^ (row & 7)) << 4)) =
                make_uint4(h[0], h[1], h[2], h[3]);
        }
    }
}

// The converting warps where the copying warp brings the codes: a thread per key of a step, which reads the row's scales a
// step ahead. Rows behind the last key that the row tile sees get scales of 0, whatever lies in their place.
template <int kDim, bool kWhole>
__device__ __forceinline__ void convert_copied(const AttnArgs &s, const Pages4 &pages, Place &place, bool more, uint8_t *ring,
                                               const uint8_t *raw, uint64_t *full, uint64_t *empty, uint64_t *raw_full,
                                               uint64_t *raw_empty, volatile uint32_t *gave_up) {
    using C = Tc<kDim, true>;
    constexpr int kWords = kDim / 64;
    const ks_attention_args_t &a = s.a;
    const int lane = threadIdx.x % 32, row = (threadIdx.x / 32 - kConvert) * 32 + lane;
    const int page_size = (int)a.page_size, pairs = (int)a.head_dim / 32;
    uint32_t at = 0;  // tiles made so far: K and V of each step in turn
    RingAt<C::kRawStages> from;
    while (more) {
        const AttnSpan span = attn_span(s, place.cur, place.q);
        const int head = place.cur.head / s.head_splits, sees = attn_tile_keys(s, place.q, place.cur.row_tile);
        const int32_t *table = a.page_table + (int64_t)place.cur.seq * a.table_stride;
        const uint8_t *k_scales = pages.k.scales + head * pages.k.scale_head, *v_scales = pages.v.scales + head * pages.v.scale_head;
        // The next step's, words of whole rows; of others (96 dims, or unaligned) pairs, joined when their turn comes.
        constexpr int kNext = kWhole ? kWords : 2 * kWords;
        uint32_t next[2][kNext];
        auto read_scales = [&](int j) {
#pragma unroll
            for (int i = 0; i < kNext; ++i) next[0][i] = next[1][i] = 0;
            const int key = j * kKeys + row;
            if (j >= span.last || key >= sees) return;
            const int index = key / page_size;
            const uint32_t page = (uint32_t)__ldg(table + index);
            if (page >= (uint64_t)a.pages) return;  // the copying warp reports it
            const uint64_t e = (uint64_t)(page * pages.page_units + (uint32_t)(key - index * page_size) * pages.slot_units) * 2;
            if constexpr (!kWhole) {
#pragma unroll
                for (int i = 0; i < kNext; ++i)
                    if (i < pairs) {
                        next[0][i] = __ldg(reinterpret_cast<const uint16_t *>(k_scales + e) + i);
                        next[1][i] = __ldg(reinterpret_cast<const uint16_t *>(v_scales + e) + i);
                    }
            } else if constexpr (kWords == 2) {
                const uint2 x = __ldg(reinterpret_cast<const uint2 *>(k_scales + e));
                const uint2 y = __ldg(reinterpret_cast<const uint2 *>(v_scales + e));
                next[0][0] = x.x;
                next[0][1] = x.y;
                next[1][0] = y.x;
                next[1][1] = y.y;
            } else {
                next[0][0] = __ldg(reinterpret_cast<const uint32_t *>(k_scales + e));
                next[1][0] = __ldg(reinterpret_cast<const uint32_t *>(v_scales + e));
            }
        };
        read_scales(span.first);
        bool ok = true;
        for (int j = span.first; j < span.last && ok; ++j) {
            uint32_t scales[2][kWords];
#pragma unroll
            for (int v = 0; v < 2; ++v)
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    if constexpr (kWhole) scales[v][i] = next[v][i];
                    else scales[v][i] = next[v][2 * i] | next[v][2 * i + 1] << 16;
                }
            read_scales(j + 1);
#pragma unroll
            for (int v = 0; v < 2; ++v, ++at) {
                const uint32_t stage = at % C::kStages;
                ok = ok && bar_wait_warp(empty + stage, (at / C::kStages & 1) ^ 1, gave_up) &&
                     bar_wait_warp(raw_full + from.stage, from.phase, gave_up);
                if (!ok) break;
                const uint8_t *codes = raw + from.stage * C::kRawTile + row * (kDim / 2);
                const int turn = kDim == 128 ? row >> 1 & 3 : row >> 2 & 1;
                convert_row<kDim>(ring + stage * C::kTileBytes, row, scales[v],
                                  [&](int i) { return *reinterpret_cast<const uint4 *>(codes + ((i ^ turn) << 4)); });
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(full + stage);
                    bar_arrive(raw_empty + from.stage);
                }
                from.next();
            }
        }
        more = ok && next_tile(s, place, span.cost);
    }
}

// The converting warps where they copy for themselves: a thread per key of a step, a warp for 32 of them. A warp copies its
// keys' codes and scales to a ring of its own, two tiles ahead, neighbouring lanes neighbouring bytes (with loads to registers,
// a key a thread, the long prompt takes 1.3 times as long); a thread then makes its row fp16 in the layout that the matrix
// instructions read.
// Rows behind the last key that the row tile sees are zeros.
template <int kDim, bool kWhole>
__device__ __forceinline__ void convert_pages(const AttnArgs &s, const Pages4 &pages, Place &place, bool more, uint8_t *ring, uint8_t *raw,
                                              uint64_t *full, uint64_t *empty, volatile uint32_t *gave_up) {
    using C = Tc<kDim, true>;
    constexpr int kGroups = kDim / 16;
    constexpr uint32_t kNone = 0xFFFFFFFFu;
    const ks_attention_args_t &a = s.a;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32 - kConvert, row = warp * 32 + lane;
    const int groups = (int)a.head_dim / 16, page_size = (int)a.page_size;
    uint8_t *mine = raw + warp * C::kRawStages * 32 * C::kRawRow;
    uint32_t at = 0;  // tiles made so far: K and V of each step in turn
    uint32_t raw_at = 0;
    while (more) {
        const AttnSpan span = attn_span(s, place.cur, place.q);
        const int head = place.cur.head / s.head_splits, sees = attn_tile_keys(s, place.q, place.cur.row_tile);
        const int32_t *table = a.page_table + (int64_t)place.cur.seq * a.table_stride;
        // The place of this thread's key of a step: whole pools, in 16 bytes of codes (2 of scales); others, its page, and its
        // slot. kNone: no key, or its page is not in the pool.
        auto look_up = [&](int j, uint32_t &slot) {
            const int key = j * kKeys + row;
            slot = 0;
            if (j >= span.last || key >= sees) return kNone;
            const int index = key / page_size;
            const uint32_t page = (uint32_t)__ldg(table + index);
            slot = (uint32_t)(key - index * page_size);
            if (page >= (uint64_t)a.pages) {
                atomicOr(&g_fault_flags, kFaultBadIndex);
                return kNone;
            }
            return kWhole ? page * pages.page_units + slot * pages.slot_units : page;
        };
        // A tile's codes (and scales, of whole pools) to the raw ring; zeros where there is no key.
        auto copy = [&](const Pool4 &pool, uint32_t where, uint32_t slots, uint32_t to) {
            const uint32_t dst = smem_addr(mine) + to * 32 * C::kRawRow;
            const uint8_t *codes = pool.codes + head * pool.code_head;
            if constexpr (kWhole) {
                constexpr int kPieces = kDim / 32;  // of 16 bytes in a row
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int key = i * (32 / kPieces) + lane / kPieces, c = lane % kPieces;
                    const uint32_t w = __shfl_sync(0xFFFFFFFFu, where, key);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + key * C::kRawRow + c * 16),
                                 "l"(codes + c * 16 + (w == kNone ? 0 : w) * 16ull), "r"(w == kNone ? 0 : 16) : "memory");
                }
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst + lane * C::kRawRow + kDim / 2),
                             "l"(pool.scales + head * pool.scale_head + (where == kNone ? 0 : where) * 2ull), "n"(kGroups),
                             "r"(where == kNone ? 0 : kGroups) : "memory");
            } else {
#pragma unroll 1
                for (int i = 0; i < kGroups; ++i) {
                    const int key = i * 32 / kGroups + lane / kGroups, g = lane % kGroups;
                    const uint32_t w = __shfl_sync(0xFFFFFFFFu, where, key), r = __shfl_sync(0xFFFFFFFFu, slots, key);
                    const bool in = w != kNone && g < groups;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst + key * C::kRawRow + g * 8),
                                 "l"(in ? codes + w * pool.code_page + r * pool.code_slot + g * 8 : pool.codes), "r"(in ? 8 : 0)
                                 : "memory");
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // Scales of rows that no copy takes, a byte a register so that nothing waits for them before they are used.
        uint32_t next_scales[kWhole ? 1 : kGroups];
        auto read_scales = [&](const Pool4 &pool, uint32_t w, uint32_t r) {
            const uint8_t *e = pool.scales + head * pool.scale_head + (int64_t)w * pool.scale_page + r * pool.scale_slot;
#pragma unroll
            for (int g = 0; g < (kWhole ? 0 : kGroups); ++g) next_scales[g] = w != kNone && g < groups ? __ldg(e + g) : 0;
        };
        uint32_t slot[2];  // of this step and the next
        uint32_t where[2];
        where[0] = look_up(span.first, slot[0]);
        copy(pages.k, where[0], slot[0], raw_at);
        copy(pages.v, where[0], slot[0], raw_at + 1 < C::kRawStages ? raw_at + 1 : raw_at + 1 - C::kRawStages);
        where[1] = look_up(span.first + 1, slot[1]);
        if constexpr (!kWhole) read_scales(pages.k, where[0], slot[0]);
        bool ok = true;
        for (int j = span.first; j < span.last && ok; ++j) {
            const uint32_t now = where[0], now_slot = slot[0];
            where[0] = where[1];
            slot[0] = slot[1];
            where[1] = look_up(j + 2, slot[1]);
#pragma unroll
            for (int v = 0; v < 2; ++v, ++at) {
                const Pool4 &pool = v ? pages.v : pages.k;
                copy(pool, where[0], slot[0], raw_at ? raw_at - 1 : C::kRawStages - 1);  // the next step's tile, two on
                const uint32_t stage = at % C::kStages;
                ok = ok && bar_wait_warp(empty + stage, (at / C::kStages & 1) ^ 1, gave_up);
                if (!ok) break;
                uint32_t scales[kGroups / 4] = {};
                if constexpr (!kWhole) {  // this tile's, read while the one before was made; the next one's
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) scales[g / 4] |= next_scales[g] << (8 * (g % 4));
                    if (v) read_scales(pages.k, where[0], slot[0]);
                    else read_scales(pages.v, now, now_slot);
                }
                asm volatile("cp.async.wait_group 2;" ::: "memory");
                __syncwarp();
                const uint8_t *from = mine + (raw_at * 32 + lane) * C::kRawRow;
                if constexpr (kWhole) {
#pragma unroll
                    for (int i = 0; i < kGroups / 4; ++i) scales[i] = reinterpret_cast<const uint32_t *>(from + kDim / 2)[i];
                }
                convert_row<kDim>(ring + stage * C::kTileBytes, row, scales,
                                  [&](int i) { return *reinterpret_cast<const uint4 *>(from + i * 16); });
                fence_async_smem();
                __syncwarp();
                if (lane == 0) bar_arrive(full + stage);
                if (++raw_at == C::kRawStages) raw_at = 0;
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");  // those of no step among them
        __syncwarp();
        more = ok && next_tile(s, place, span.cost);
    }
}

template <typename T, int kDim, typename Pages>
__global__ void __launch_bounds__(Split<Pages::k4>::kThreads, 1)
attn_tc_kernel(const __grid_constant__ AttnArgs s, const __grid_constant__ CUtensorMap q_map,
               const __grid_constant__ Pages pages) {
    constexpr bool k4 = Pages::k4;
    using C = Tc<kDim, k4>;
    using P = typename std::conditional<k4, __half, T>::type;  // of the products' operands
    constexpr bool kMakeQ = k4 && !std::is_same<T, P>::value;  // queries are made P's in shared memory
    constexpr int kThreads = Split<k4>::kThreads;
    extern __shared__ uint8_t raw[];
    const ks_attention_args_t &a = s.a;
    const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
    uint8_t *smem = raw + (base - smem_addr(raw));
    const uint32_t q_addr = base, ring = base + 2 * C::kTileBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + (2 + C::kStages) * C::kTileBytes);
    uint64_t *full = bars, *empty = bars + C::kStages;
    uint64_t *q_full = empty + C::kStages, *q_free = q_full + 1, *s_full = q_full + 2, *p_full = s_full + 2;
    uint64_t *o_full = p_full + 2;
    uint64_t *turn = o_full + 2, *done = turn + 2, *q_made = done + 2, *tail = q_made + 2;
    uint64_t *raw_full = tail, *raw_empty = tail + C::kRawStages;  // in place of the tails'
    uint32_t *tmem_at = reinterpret_cast<uint32_t *>(bars + C::kBars);
    volatile uint32_t *gave_up = tmem_at + 1;
    const int warp = warp_uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const int cta = blockIdx.x, ctas = gridDim.x;

    if (threadIdx.x == kThreads - 1) {  // the maps' descriptors, which the first copies would wait for
        prefetch_map(&q_map);
        if constexpr (!k4) {
            prefetch_map(&pages.k);
            prefetch_map(&pages.v);
        } else if (pages.by_map) {
            prefetch_map(&pages.k_map);
            prefetch_map(&pages.v_map);
        }
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(full + i, k4 ? kConvertWarps : 1);
            mbar_init(empty + i, k4 ? 2 : 3);  // the issuing warps and the one that clears tails
            if (!k4) mbar_init(tail + i, 1);
        }
        if (k4) {
            for (int i = 0; i < C::kRawStages; ++i) {
                mbar_init(raw_full + i, 1);
                mbar_init(raw_empty + i, kConvertWarps);
            }
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(s_full + w, 1);
            mbar_init(p_full + w, kTileThreads / 32);
            mbar_init(o_full + w, 1);
            mbar_init(turn + w, 1);
            mbar_init(done + w, 1);
            mbar_init(q_made + w, kTileThreads / 32);
        }
        mbar_init(q_full, 1);
        mbar_init(q_free, 2);
        bar_arrive(turn);  // tile 0 begins
        *gave_up = 0;
        fence_mbar_init();
    }
    if (warp == kMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(tmem_at))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = warp_uniform(*tmem_at);
    grid_dependency_wait();
    allow_dependents_launch();
    if (threadIdx.x == 0) attn_joins(s, ctas)[cta].pieces = 0;
    __shared__ Place places[kThreads / 32];
    Place &place = places[warp];
    bool more;
    {
        const AttnCursor &c = attn_begin<kThreads>(s, cta, ctas);
        more = c.left > 0;
        if (more && lane == 0) {
            place.cur = c;
            place.q = attn_seq(a, c.seq);
        }
        __syncwarp();
    }

    if (k4 && warp >= kConvert) {
        if constexpr (k4) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Split<k4>::kConvertRegs));
            uint8_t *tiles = smem + 2 * C::kTileBytes, *rows = smem + C::kRawAt;
            if (pages.by_map && pages.whole)
                convert_copied<kDim, true>(s, pages, place, more, tiles, rows, full, empty, raw_full, raw_empty, gave_up);
            else if (pages.by_map)
                convert_copied<kDim, false>(s, pages, place, more, tiles, rows, full, empty, raw_full, raw_empty, gave_up);
            else if (pages.whole) convert_pages<kDim, true>(s, pages, place, more, tiles, rows, full, empty, gave_up);
            else convert_pages<kDim, false>(s, pages, place, more, tiles, rows, full, empty, gave_up);
        }
    } else if (warp >= kSoftmaxWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Split<k4>::kOtherRegs));
        if (warp == kCopy) {
            // ---- copies
            // A copy's keys; with 4-bit pages, tiles go to the ring of codes, and a lane's copy has whole rows.
            constexpr int kParts = k4 ? 1 : C::kHalves, kTo = k4 ? C::kRawStages : C::kStages;
            constexpr int kToTile = k4 ? C::kRawTile : C::kTileBytes, kRowBytes = k4 ? kDim / 2 : 128;
            uint64_t *to_full = k4 ? raw_full : full, *to_empty = k4 ? raw_empty : empty;
            const uint32_t to = k4 ? base + C::kRawAt : ring;
            const int page_size = (int)a.page_size, in_tile = min(page_size, kKeys);
            const int part = lane / kParts, half = lane % kParts;
            uint32_t at = 0;  // tiles copied so far: K and V of each step in turn
            uint32_t queries = 0;
            // A row tile's queries, as soon as the tile before has had its last product with its own: a
            // box of tile_heads heads and tile_tokens tokens comes in the rows' order. Rows behind the
            // sequence hold other tokens' queries (or zeros behind the last); no row touches another.
            auto copy_queries = [&](int head) {
                if (!bar_wait_warp(q_free, (queries++ & 1) ^ 1, gave_up)) return false;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, C::kHalves * s.tile_heads * s.tile_tokens * 128);
                    const int first_head = head * s.group + place.cur.head % s.head_splits * s.tile_heads;
                    const int token = place.q.q0 + place.cur.row_tile * s.tile_tokens;
                    for (int h = 0; h < C::kHalves; ++h)
                        tma_load3(q_addr + h * kRows * 128, &q_map, h * 64, first_head, token, smem_addr(q_full));
                }
                __syncwarp();
                return true;
            };
            while (more) {
                const AttnSpan span = attn_span(s, place.cur, place.q);
                const int head = place.cur.head / s.head_splits, keys = place.q.keys;
                const int32_t *table = a.page_table + (int64_t)place.cur.seq * a.table_stride;
                bool ok = true;
                // The first row tile's queries are copied before all else, later ones behind their first keys
                // and values, which need not wait.
                const uint32_t tile = queries;
                if (tile == 0 && span.first < span.last) ok = copy_queries(head);
                int last = span.last;
                if constexpr (k4) {
                    if (!pages.by_map) {  // the pages are the converting warps' work
                        if (tile > 0 && span.first < span.last) ok = copy_queries(head);
                        last = span.first;
                    }
                }
                for (int j = span.first; j < last && ok; ++j) {
                    const int key = j * kKeys + part * in_tile;
                    const bool wanted = part * in_tile < kKeys && key < keys;
                    int page = 0, slot = 0;
                    if (wanted) {
                        page = __ldg(table + key / page_size);
                        slot = key % page_size;
                        if ((uint32_t)page >= (uint64_t)a.pages) {  // past the pool: the copy fills zeros
                            atomicOr(&g_fault_flags, kFaultBadIndex);
                            page = (int)a.pages;
                        }
                    }
                    const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xFFFFFFFFu, wanted)) * in_tile * kRowBytes;
                    for (int v = 0; v < 2 && ok; ++v, ++at) {
                        const uint32_t stage = at % kTo;
                        ok = bar_wait_warp(to_empty + stage, (at / kTo & 1) ^ 1, gave_up);
                        if (!ok) break;
                        if (lane == 0) mbar_arrive_expect_tx(to_full + stage, bytes);
                        __syncwarp();
                        const CUtensorMap *map;
                        if constexpr (k4) map = v ? &pages.v_map : &pages.k_map;
                        else map = v ? &pages.v : &pages.k;
                        if (wanted)
                            tma_load(to + stage * kToTile + half * kHalfBytes + part * in_tile * kRowBytes, map, half * 64, slot,
                                     head, page, smem_addr(to_full + stage));
                    }
                    if (tile > 0 && j == span.first) ok = ok && copy_queries(head);
                }
                more = ok && next_tile(s, place, span.cost);
            }
            if (queries) (void)mbar_wait_bounded(q_full, (queries - 1) & 1);
            // nothing of this CTA's is in flight when it ends, also after a wait that gave up
            const uint32_t from = at > (uint32_t)kTo ? at - kTo : 0;
            for (uint32_t i = from; i < at; ++i) (void)mbar_wait_bounded(to_full + i % kTo, i / kTo & 1);
        } else if (warp == kMma || warp == kMma + 2) {
            // ---- matrix instructions of tile w, issued by one thread: for each step P V, then Q K of the
            // next step. The two warps take turns, a whole batch each: the other tile's softmax runs beside
            // a batch, and a warp has done its waiting when its turn comes. (Without turns the batches
            // interleave, both softmaxes run at once and the tensor cores wait for them; one warp for both
            // tiles spends a third of its time on barriers while the few instructions it can issue ahead
            // run out. Measured at 8192 tokens over 16384 keys: both 1.2 to 1.4 ms.)
            const int w = warp == kMma ? 0 : 1;
            constexpr uint32_t qk = mma_shape<P>(kKeys, false), pv = mma_shape<P>(kDim, true);
            const uint32_t s_at = tmem + w * 128, o_at = tmem + C::kO + w * 128;
            const uint32_t q_low = desc_low(q_addr + w * kTile * 128, 16);
            RingAt<C::kStages> k_at, v_at;  // the next step's keys, this step's values
            uint32_t q_uses = 0, p_uses = 0, turns = 0;
            uint32_t tails = 0;             // phase of each stage's tail barrier, a bit each
            auto issue_qk = [&](uint32_t stage) {
                const uint32_t k_low = desc_low(ring + stage * C::kTileBytes, 16);
                mma_ss<false>(s_at, q_low, k_low, qk);
#pragma unroll
                for (int i = 1; i < kDim / 16; ++i)
                    mma_ss<true>(s_at, q_low + ((i / 4 * kRows * 128 + i % 4 * 32) >> 4),
                                 k_low + ((i / 4 * kHalfBytes + i % 4 * 32) >> 4), qk);
                mma_commit(smem_addr(s_full + w));
            };
            while (more) {
                const AttnSpan span = attn_span(s, place.cur, place.q);
                const int first = warp_uniform(span.first), end = warp_uniform(span.last);
                const int keys = warp_uniform(attn_tile_keys(s, place.q, place.cur.row_tile));
                const bool two = warp_uniform(second_tile(s, place)) != 0;
                if (first >= end) break;  // the share ends in the tile's extra cost
                bool ok = bar_wait_warp(kMakeQ ? q_made + w : q_full, q_uses++ & 1, gave_up);
                if (w == 1 && !two) {  // this tile has no rows: its share of the stages is given back
                    if (ok && lane == 0) bar_arrive(q_free);
                    for (int i = 2 * (end - first); i > 0 && ok; --i) {
                        ok = bar_wait_warp(full + k_at.stage, k_at.phase, gave_up);
                        if (!k4 && i == 1 && keys < end * kKeys) tails ^= 1u << k_at.stage;
                        if (ok && lane == 0) bar_arrive(empty + k_at.stage);
                        k_at.next();
                    }
                    more = ok && next_tile(s, place, span.cost);
                    continue;
                }
                ok = ok && bar_wait_warp(full + k_at.stage, k_at.phase, gave_up) &&
                     (!two || bar_wait_warp(turn + w, turns++ & 1, gave_up));
                if (!ok) break;
                fence_after();
                if (elect_one()) {
                    issue_qk(k_at.stage);
                    if (two) bar_arrive(turn + 1 - w);
                    mma_commit(smem_addr(empty + k_at.stage));
                    if (first + 1 == end) mma_commit(smem_addr(q_free));
                }
                __syncwarp();
                v_at = k_at;
                v_at.next();
                for (int j = first; j < end; ++j) {
                    const bool last = j + 1 == end;
                    k_at = v_at;
                    k_at.next();
                    ok = bar_wait_warp(full + v_at.stage, v_at.phase, gave_up);
                    if (!k4 && ok && keys < (j + 1) * kKeys) {
                        ok = bar_wait_warp(tail + v_at.stage, tails >> v_at.stage & 1, gave_up);
                        tails ^= 1u << v_at.stage;
                    }
                    if (!last) ok = ok && bar_wait_warp(full + k_at.stage, k_at.phase, gave_up);
                    // the probabilities last: they come later than the turn, and the products wait for them
                    if (two) ok = ok && bar_wait_warp(turn + w, turns++ & 1, gave_up);
                    ok = ok && bar_wait_warp(p_full + w, p_uses++ & 1, gave_up);
                    if (!ok) break;
                    fence_after();
                    if (elect_one()) {
                        const uint32_t v_low = desc_low(ring + v_at.stage * C::kTileBytes, kHalfBytes);
                        mma_ts(o_at, s_at, v_low, pv, j > first);
#pragma unroll
                        for (int i = 1; i < kKeys / 16; ++i) mma_ts(o_at, s_at + i * 8, v_low + i * (2048 >> 4), pv, 1u);
                        if (last) mma_commit(smem_addr(o_full + w));
                        else issue_qk(k_at.stage);
                        if (two) bar_arrive(turn + 1 - w);
                        mma_commit(smem_addr(empty + v_at.stage));
                        if (!last) mma_commit(smem_addr(empty + k_at.stage));
                        if (j + 2 == end) mma_commit(smem_addr(q_free));
                    }
                    __syncwarp();
                    v_at = k_at;
                    v_at.next();
                }
                // k_at is the tile after the row tile's last values: the next row tile's first keys
                more = ok && next_tile(s, place, span.cost);
            }
            // every instruction and arrival of this warp is done when it ends, also after a wait that gave up
            if (elect_one()) mma_commit(smem_addr(done + w));
            __syncwarp();
            (void)mbar_wait_bounded(done + w, 0);
        } else if (!k4 && warp == kTail) {
            // ---- the step a row tile's keys end in: value rows behind the last key that a row of it sees may
            // hold anything (later tokens' values, or no token's), and a product with their probability 0 would
            // let a NaN through, so they are set to 0. This warp follows every tile through the ring (a
            // barrier's phases can be told apart one apart, no further).
            uint32_t at = 0;
            while (more) {
                const AttnSpan span = attn_span(s, place.cur, place.q);
                const int valid = attn_tile_keys(s, place.q, place.cur.row_tile) - (span.last - 1) * kKeys;
                bool ok = true;
                for (uint32_t end = at + 2 * (span.last - span.first); at < end && ok; ++at) {
                    const uint32_t stage = at % C::kStages;
                    ok = bar_wait_warp(full + stage, at / C::kStages & 1, gave_up);
                    if (!ok) break;
                    if (at + 1 == end && valid < kKeys) {  // the row tile's last values
                        uint8_t *v_tile = smem + (2 + stage) * C::kTileBytes;
                        for (int h = 0; h < C::kHalves; ++h)
                            for (uint32_t b = (uint32_t)max(valid, 0) * 128 + lane * 16; b < (uint32_t)kHalfBytes; b += 512)
                                *reinterpret_cast<uint4 *>(v_tile + h * kHalfBytes + b) = make_uint4(0, 0, 0, 0);
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) bar_arrive(tail + stage);
                    }
                    if (lane == 0) bar_arrive(empty + stage);
                }
                more = ok && next_tile(s, place, span.cost);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Split<k4>::kSoftmaxRegs));
        // ---- softmax: a warp has 16 rows, a quad of lanes a row pair (r0, r0 + 8): the layout in which the
        // 16-row loads of tensor memory hand out scores, so that maxima and sums need two shuffles and
        // warps nothing of each other
        const int w = warp / 8, sub = warp % 4 * 32 + warp / 4 % 2 * 16, quad = lane % 4;
        const uint32_t s_at = tmem + ((uint32_t)sub << 16) + w * 128, o_at = s_at - w * 128 + C::kO + w * 128;
        const int r0 = w * kTile + sub + lane / 4;
        const int dim = (int)a.head_dim;
        const bool causal = (a.flags & KS_ATTENTION_CAUSAL) != 0;
        // The exponents are made with |scale|: a negative one turns the scores' signs. 0 becomes the least
        // normal number, whose products with finite scores vanish and which leaves -inf as it is.
        // Queries that were made fp16 have a unit for each row.
        float scale[2], unit[2] = {1.0f, 1.0f};
        const bool negative = s.scale_log2 < 0.0f;
        // the thread's rows' tokens and heads within a row tile
        const int r_token[2] = {r0 / s.tile_heads, (r0 + 8) / s.tile_heads};
        const int r_head[2] = {r0 % s.tile_heads, (r0 + 8) % s.tile_heads};
        const int warp_token = (w * kTile + sub) / s.tile_heads;
        uint32_t s_uses = 0, o_uses = 0, q_uses = 0;
        bool q_taken = false;
        auto take_queries = [&]() {
            if (!bar_wait_warp(q_full, q_uses++ & 1, gave_up)) return false;
            make_queries<kDim>(smem, w * kTile + sub, unit);
            fence_async_smem();
            warp_arrive(q_made + w);
            return true;
        };
        while (more) {
            const AttnSpan span = attn_span(s, place.cur, place.q);
            if (span.first >= span.last) break;  // the share ends in the tile's extra cost
            if (kMakeQ && !q_taken && !take_queries()) break;
            q_taken = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) scale[i] = fminf(fmaxf(fabsf(s.scale_log2) * unit[i], 1.17549435e-38f), 3.4e38f);
            if (w == 1 && !second_tile(s, place)) {
                more = next_tile(s, place, span.cost);
                continue;
            }
            // keys that this thread's rows see, and all rows of the warp; the threads' rows in the output
            int limit[2], all_see;
            T *dst[2];
            bool real[2];
            {
                const AttnSeq q = place.q;
                const int row_tile = place.cur.row_tile, sees = attn_tile_keys(s, q, row_tile);
                const int first = q.keys - q.n + row_tile * s.tile_tokens + 1;
                all_see = causal ? min(sees, first + warp_token) : sees;
                int kv_head = place.cur.head, split = 0;
                if (s.head_splits > 1) {
                    kv_head /= s.head_splits;
                    split = place.cur.head - kv_head * s.head_splits;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int in_seq = row_tile * s.tile_tokens + r_token[i], in_group = split * s.tile_heads + r_head[i];
                    real[i] = r_token[i] < s.tile_tokens && in_seq < q.n && in_group < s.group;
                    limit[i] = causal ? min(sees, first + r_token[i]) : sees;
                    dst[i] = (T *)a.out + (q.q0 + in_seq) * a.out_token_stride +
                             (kv_head * s.group + in_group) * a.out_head_stride;
                }
            }

            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
            bool ok = true;
            for (int j = span.first; j < span.last; ++j) {
                ok = bar_wait_warp(s_full + w, s_uses++ & 1, gave_up);
                if (!ok) break;
                fence_after();
                const int key0 = j * kKeys;
                uint32_t p[2][16];
                float2 sum[2];
                // The exponentials are taken to the rows' old base at once; their sums tell whether a score
                // has outgrown it (a maximum over the scores would take as long as the exponentials). Then,
                // and for the first step and rows that saw no key yet, the maxima are taken and the
                // exponentials again: the scores are still in tensor memory.
                bool rebase = j == span.first ||
                              __any_sync(0xFFFFFFFFu, (real[0] && m[0] == -INFINITY) || (real[1] && m[1] == -INFINITY));
                while (true) {
                    uint32_t x[2][32];  // [64 keys][of 8 keys two of each row, ...]
                    tmem_load_rows32(x[0], s_at);
                    tmem_load_rows32(x[1], s_at + 64);
                    tmem_wait_load();
                    if (negative) {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[c][i] ^= 0x80000000u;
                    }
                    if (key0 + kKeys > all_see) {
#pragma unroll
                        for (int g8 = 0; g8 < kKeys / 8; ++g8) {
                            if (key0 + g8 * 8 + 8 <= all_see) continue;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (key0 + g8 * 8 + quad * 2 + i % 2 >= limit[i / 2]) x[g8 / 8][g8 % 8 * 4 + i] = 0xFF800000u;  // -inf
                        }
                    }
                    if (rebase) {
                        float f[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float best = m[k];
#pragma unroll
                            for (int c = 0; c < 2; ++c)
#pragma unroll
                                for (int i = 2 * k; i < 32; i += 4)
                                    best = fmaxf(best, fmaxf(__uint_as_float(x[c][i]), __uint_as_float(x[c][i + 1])) * scale[k]);
                            best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, 1));
                            best = fmaxf(best, __shfl_xor_sync(0xFFFFFFFFu, best, 2));
                            // a base to which the lift adds exactly, so that old and new offsets differ by
                            // as much as the bases
                            if (kLift<P> != 0.0f) best = kLift<P> - (kLift<P> - best);
                            f[k] = exp2_approx(m[k] - attn_base(best));
                            l[k] *= f[k];
                            m[k] = best;
                        }
                        if (j > span.first) {
#pragma unroll 1
                            for (int c = 0; c < kDim / 32; ++c) tmem_scale_rows(o_at + c * 32, f[0], f[1]);
                        }
                    }
                    const float2 mul[2] = {make_float2(scale[0], scale[0]), make_float2(scale[1], scale[1])};
                    const float2 off[2] = {make_float2(kLift<P> - attn_base(m[0]), kLift<P> - attn_base(m[0])),
                                           make_float2(kLift<P> - attn_base(m[1]), kLift<P> - attn_base(m[1]))};
                    sum[0] = sum[1] = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 y = make_float2(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1]));
                            y = pair_fma<true>(y, mul[i & 1], off[i & 1]);
                            y.x = exp2_approx(y.x);
                            y.y = exp2_approx(y.y);
                            sum[i & 1] = pair_add<true>(sum[i & 1], y);
                            p[c][i] = pack_pair<P>(y.x, y.y);
                        }
                    sum[0].x += sum[0].y;
                    sum[1].x += sum[1].y;
                    if (rebase || !__any_sync(0xFFFFFFFFu, (real[0] && !(sum[0].x <= kGrowth<P>)) ||
                                                               (real[1] && !(sum[1].x <= kGrowth<P>))))
                        break;
                    rebase = true;
                }
                tmem_store_rows16(s_at, p[0]);
                tmem_store_rows16(s_at + 32, p[1]);
                tmem_wait_store();
                fence_before();
                warp_arrive(p_full + w);
                l[0] += sum[0].x;
                l[1] += sum[1].x;
            }
            if (!ok) break;
            // What is left to do without the output is done before the wait for it.
            const bool whole = span.first == 0 && span.last == span.units;
            float *part = attn_slot(s, cta, span.first == 0 ? 1 : 0);
            float inv[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
                l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
                inv[i] = attn_inverse(l[i]) * s.out_scale;
                if (!whole && quad == 0) {
                    part[kRows * dim + r0 + 8 * i] = m[i];
                    part[kRows * dim + kRows + r0 + 8 * i] = l[i];
                }
            }
            if (!whole && span.first == 0 && threadIdx.x == 0) {
                AttnJoin j = {};
                j.pieces = attn_pieces(s, place.cur, span, cta);
                j.seq = place.cur.seq;
                j.head = place.cur.head;
                j.row_tile = place.cur.row_tile;
                j.q0 = place.q.q0;
                j.q_len = place.q.n;
                attn_joins(s, ctas)[cta] = j;
            }
            more = next_tile(s, place, span.cost);
            if (kMakeQ && more) {  // the next row tile's queries first: its products wait for them
                const AttnSpan next = attn_span(s, place.cur, place.q);
                if (next.first < next.last) {
                    ok = q_taken = take_queries();
                    if (!ok) break;
                }
            }
            ok = bar_wait_warp(o_full + w, o_uses++ & 1, gave_up);
            if (!ok) break;
            fence_after();
            uint32_t o[kDim / 64][32];
#pragma unroll
            for (int c = 0; c < kDim / 64; ++c) tmem_load_rows32(o[c], o_at + c * 64);
            tmem_wait_load();
            fence_before();  // O is read before the next row tile's first product overwrites it
            if (!whole) {
#pragma unroll
                for (int c = 0; c < kDim / 8; ++c)
                    if (c * 8 < dim) {
                        const uint32_t *y = o[c / 8] + c % 8 * 4;
                        *attn_part(s, part, r0 / 16, c, lane) = make_float4(__uint_as_float(y[0]), __uint_as_float(y[1]),
                                                                            __uint_as_float(y[2]), __uint_as_float(y[3]));
                    }
                continue;
            }
#pragma unroll
            for (int c = 0; c < kDim / 32; ++c) {
                const uint32_t *x = o[c / 2] + c % 2 * 16;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // A lane has two columns of each of the chunk's four groups of 8; after the exchange
                    // lane q of the quad has the 8 columns of group q, 16 bytes.
                    uint32_t y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        y[i] = pack_pair<T>(__uint_as_float(x[4 * i + 2 * k]) * inv[k],
                                            __uint_as_float(x[4 * i + 2 * k + 1]) * inv[k]);
                    quad_transpose(y, quad);
                    const int col = c * 32 + quad * 8;
                    if (real[k] && col < dim) *reinterpret_cast<uint4 *>(dst[k] + col) = make_uint4(y[0], y[1], y[2], y[3]);
                }
            }
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

}  // namespace
}  // namespace ks
