// Attention of new tokens over a paged key/value cache: the kernel for few rows per key/value head
// (single tokens, short drafts), the join of split rows, and the C entry points.
//
// Mathematics, per query row with scores s_j = scale * q.k_j over the keys it sees:
//   m = max s_j, l = sum exp(s_j - m), o = sum exp(s_j - m) v_j / l
// in one pass with a running maximum: when m grows, l and o are scaled by exp(m_old - m_new).
// Scores, maxima, sums and outputs are FP32. The probabilities are rounded to the inputs' 16-bit
// type for the second matrix product, at most half a step relative to each (2^-9 for bf16, 2^-12 for
// fp16); the sum l adds them before that rounding. fp16 is normal down to 2^-14 only, so that its
// probabilities are taken 2^15 times as large as they are (l and o with them, which the quotient does
// not depend on): they keep their precision down to 2^-29 of the row's largest and end at 2^-40.
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "ks_attention.cuh"

namespace ks {
namespace {

constexpr int kRows = 16;                 // rows of a tile: one mma.m16n8k16 tile
constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTileCost = 4;              // units that beginning and ending a row tile costs
constexpr int kSub = 16;                  // keys of a warp's step
constexpr int kUnit = kWarps * kSub;      // keys of a unit: a step of each warp (a power of two)
template <typename T>
constexpr float kLift = std::is_same<T, __half>::value ? 32768.0f : 1.0f;  // what a row's largest probability counts

// Few rows make this a stream of the cache: per key of 128 values 512 bytes, 16 query rows cost
// two 16x8x16 matrix instructions, a tenth of the time its bytes take. Each warp therefore runs
// alone on every fourth 16-key step, with its own ring of asynchronous 16-byte copies in shared
// memory (no barrier in the loop), its own maximum, sum and output registers; the four are joined
// when the row tile ends. Bound by DRAM: 64 contexts of 700 to 8100 keys, 8 heads of 128, one token of
// 64 query heads each, 198 to 207 us or 6.1 to 6.4 TB/s; 4 of 131000 keys 315 to 327 us or 6.4 to 6.7 TB/s.
template <int kDim>
struct Rows16 {
    static constexpr int kStages = kDim == 64 ? 4 : 3;
    static constexpr int kStepBytes = 2 * kSub * kDim * 2;  // keys and values of a step
    static constexpr int kRingBytes = kWarps * kStages * kStepBytes;
    static constexpr int kQBytes = kRows * kDim * 2;
    static constexpr int kSmem = kRingBytes + kQBytes;
    static constexpr int kCtasPerSm = kDim == 64 ? 3 : kDim == 128 ? 2 : 1;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    const int n = valid ? 16 : 0;  // 0: the 16 bytes are filled with zeros, src is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float x, float y);
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}

// Shared-memory address of 16-byte chunk c of row r in a tile of kDim 16-bit values a row: chunks
// are exchanged within a row by the row's low bits, so that ldmatrix reads eight rows without
// bank conflicts.
template <int kDim>
__device__ __forceinline__ uint32_t tile_addr(uint32_t base, int r, int c) {
    return base + (uint32_t)(r * (kDim * 2) + ((c ^ (r & 7)) << 4));
}

template <typename T, int kDim>
__global__ void __launch_bounds__(kThreads, Rows16<kDim>::kCtasPerSm)
attn_rows16_kernel(const __grid_constant__ AttnArgs s) {
    using C = Rows16<kDim>;
    constexpr bool kQRegs = kDim <= 128;  // above, the output registers leave no room for them
    constexpr int kSteps = kDim / 16;
    extern __shared__ __align__(1024) uint8_t smem[];
    const ks_attention_args_t &a = s.a;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int ctas = gridDim.x, cta = blockIdx.x;
    grid_dependency_wait();
    allow_dependents_launch();
    if (threadIdx.x == 0) attn_joins(s, ctas)[cta].pieces = 0;
    AttnCursor cur = attn_begin<kThreads>(s, cta, ctas);
    if (cur.left <= 0) return;
    AttnSeq q = attn_seq(a, cur.seq);

    const int dim = (int)a.head_dim, chunks = dim / 8;
    const uint32_t ring = smem_addr(smem) + warp * C::kStages * C::kStepBytes;
    uint8_t *q_smem = smem + C::kRingBytes;
    const uint32_t q_addr = smem_addr(q_smem);
    const int page_size = (int)a.page_size;

    while (true) {
        const AttnSpan span = attn_span(s, cur, q);
        const int units = span.units, first = span.first, last = span.last;
        if (first >= last) break;  // the share ends in the tile's extra cost
        const int sees = attn_tile_keys(s, q, cur.row_tile);
        const int kv_head = cur.head / s.head_splits;
        const T *k_base = (const T *)a.k_pages + kv_head * a.k_head_stride;
        const T *v_base = (const T *)a.v_pages + kv_head * a.v_head_stride;
        const int32_t *table = a.page_table + (int64_t)cur.seq * a.table_stride;

        // Page of the lane's key (lanes 0..15: the step's 16 keys), read one step ahead.
        auto look_up = [&](int unit) -> int {
            const int key = unit * kUnit + warp * kSub + (lane & 15);
            return unit < last && key < sees ? __ldg(table + key / page_size) : -1;
        };
        auto load_step = [&](int unit, int stage, int page) {
            const int key = unit * kUnit + warp * kSub + (lane & 15);
            const bool wanted = unit < last && key < sees;
            const bool good = wanted && (uint32_t)page < (uint64_t)a.pages;
            if (wanted && !good) atomicOr(&g_fault_flags, kFaultBadIndex);
            const int slot = key % page_size;
            const int64_t ko = good ? page * a.k_page_stride + slot * a.k_slot_stride : -1;
            const int64_t vo = good ? page * a.v_page_stride + slot * a.v_slot_stride : -1;
            const uint32_t kt = ring + stage * C::kStepBytes, vt = kt + kSub * kDim * 2;
            constexpr int kLanes = kDim / 8 < 8 ? kDim / 8 : 8;  // lanes per row: 128 bytes
            constexpr int kRowsAtOnce = 32 / kLanes;
#pragma unroll
            for (int r0 = 0; r0 < kSub; r0 += kRowsAtOnce) {
                const int r = r0 + lane / kLanes;
                const int64_t kr = __shfl_sync(0xFFFFFFFFu, ko, r), vr = __shfl_sync(0xFFFFFFFFu, vo, r);
#pragma unroll
                for (int c0 = 0; c0 < kDim / 8; c0 += kLanes) {
                    const int c = c0 + lane % kLanes;
                    const bool in = kr >= 0 && c < chunks;
                    cp_async16(tile_addr<kDim>(kt, r, c), in ? (const void *)(k_base + kr + c * 8) : a.q, in);
                    cp_async16(tile_addr<kDim>(vt, r, c), in ? (const void *)(v_base + vr + c * 8) : a.q, in);
                }
            }
        };

        int page = look_up(first);
#pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i) {
            const int next = look_up(first + i + 1);
            load_step(first + i, i, page);
            cp_async_commit();
            page = next;
        }
        // the query rows, zeros where the tile has none
        for (int i = threadIdx.x; i < kRows * (kDim / 8); i += kThreads) {
            const int r = i / (kDim / 8), c = i % (kDim / 8);
            int token, head;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (attn_row(s, q.q0, q.n, cur.head, cur.row_tile, r, &token, &head) && c < chunks)
                x = *reinterpret_cast<const uint4 *>((const T *)a.q + token * a.q_token_stride +
                                                     head * a.q_head_stride + c * 8);
            *reinterpret_cast<uint4 *>(q_smem + (tile_addr<kDim>(0, r, c))) = x;
        }
        __syncthreads();
        uint32_t qf[kQRegs ? kSteps : 1][4];
        auto load_q = [&](uint32_t (&f)[4], int k) {
            ldmatrix4(f, tile_addr<kDim>(q_addr, lane & 15, k * 2 + (lane >> 4)));
        };
        if (kQRegs) {
#pragma unroll
            for (int k = 0; k < kSteps; ++k) load_q(qf[kQRegs ? k : 0], k);
        }

        // keys that this thread's two rows see
        int limit[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int in_seq = cur.row_tile * s.tile_tokens + (lane / 4 + 8 * i) / s.tile_heads;
            limit[i] = (a.flags & KS_ATTENTION_CAUSAL) ? min(sees, q.keys - q.n + in_seq + 1) : sees;
        }
        const int all_see = (a.flags & KS_ATTENTION_CAUSAL)
                                ? min(sees, q.keys - q.n + cur.row_tile * s.tile_tokens + 1) : sees;

        float o[kDim / 8][4];
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kDim / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;

        int stage = 0;
        for (int unit = first; unit < last; ++unit) {
            {
                const int ahead = unit + C::kStages - 1;
                const int to = stage == 0 ? C::kStages - 1 : stage - 1;
                const int next = look_up(ahead + 1);
                load_step(ahead, to, page);
                cp_async_commit();
                page = next;
            }
            cp_async_wait<C::kStages - 1>();
            __syncwarp();
            const uint32_t kt = ring + stage * C::kStepBytes, vt = kt + kSub * kDim * 2;
            const int key0 = unit * kUnit + warp * kSub;
            if (key0 < sees) {
                float sc[2][4] = {};
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    uint32_t b[4];
                    ldmatrix4(b, tile_addr<kDim>(kt, (lane & 7) + ((lane >> 4) << 3), k * 2 + ((lane >> 3) & 1)));
                    if (!kQRegs) load_q(qf[0], k);
                    mma16816<T>(sc[0], qf[kQRegs ? k : 0], b[0], b[1]);
                    mma16816<T>(sc[1], qf[kQRegs ? k : 0], b[2], b[3]);
                }
                const bool masked = key0 + kSub > all_see;
                float top[2] = {m[0], m[1]};
#pragma unroll
                for (int t = 0; t < 2; ++t) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float x = sc[t][i] * s.scale_log2;
                        if (masked && key0 + t * 8 + (lane % 4) * 2 + (i & 1) >= limit[i / 2]) x = -INFINITY;
                        sc[t][i] = x;
                        top[i / 2] = fmaxf(top[i / 2], x);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
                    top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
                }
                if (__any_sync(0xFFFFFFFFu, top[0] != m[0] || top[1] != m[1])) {
                    const float f0 = exp2_approx(m[0] - attn_base(top[0])), f1 = exp2_approx(m[1] - attn_base(top[1]));
                    l[0] *= f0;
                    l[1] *= f1;
#pragma unroll
                    for (int i = 0; i < kDim / 8; ++i) {
                        o[i][0] *= f0;
                        o[i][1] *= f0;
                        o[i][2] *= f1;
                        o[i][3] *= f1;
                    }
                    m[0] = top[0];
                    m[1] = top[1];
                }
                const float b0 = attn_base(m[0]), b1 = attn_base(m[1]);
                uint32_t p[4];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float x0 = exp2_approx(sc[t][0] - b0) * kLift<T>, x1 = exp2_approx(sc[t][1] - b0) * kLift<T>;
                    const float x2 = exp2_approx(sc[t][2] - b1) * kLift<T>, x3 = exp2_approx(sc[t][3] - b1) * kLift<T>;
                    l[0] += x0 + x1;
                    l[1] += x2 + x3;
                    p[2 * t] = pack16<T>(x0, x1);
                    p[2 * t + 1] = pack16<T>(x2, x3);
                }
#pragma unroll
                for (int d = 0; d < kDim / 16; ++d) {
                    uint32_t b[4];
                    ldmatrix4_trans(b, tile_addr<kDim>(vt, (lane & 7) + (((lane >> 3) & 1) << 3), d * 2 + (lane >> 4)));
                    mma16816<T>(o[2 * d], p, b[0], b[1]);
                    mma16816<T>(o[2 * d + 1], p, b[2], b[3]);
                }
            }
            __syncwarp();  // all lanes have read this stage before it is refilled
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
        }
        cp_async_wait<0>();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
            l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
        }

        // Join the four warps in shared memory, over the ring.
        constexpr int kPitch = kDim + 4;
        float *ow = reinterpret_cast<float *>(smem);  // [kWarps][kRows][kPitch]
        float *mw = ow + kWarps * kRows * kPitch;      // [kWarps][kRows], then the sums
        static_assert((kWarps * kRows * (kPitch + 2)) * 4 <= C::kRingBytes, "the join fits the ring");
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kDim / 8; ++i) {
            float *at = ow + (warp * kRows + lane / 4) * kPitch + i * 8 + (lane % 4) * 2;
            at[0] = o[i][0];
            at[1] = o[i][1];
            at[8 * kPitch] = o[i][2];
            at[8 * kPitch + 1] = o[i][3];
        }
        if (lane % 4 == 0) {
            mw[warp * kRows + lane / 4] = m[0];
            mw[warp * kRows + lane / 4 + 8] = m[1];
            mw[(kWarps + warp) * kRows + lane / 4] = l[0];
            mw[(kWarps + warp) * kRows + lane / 4 + 8] = l[1];
        }
        __syncthreads();
        const bool whole = first == 0 && last == units;
        float *part = attn_slot(s, cta, first == 0 ? 1 : 0);
        for (int g = warp; g < chunks; g += kWarps) {  // 8 columns
            float ll[2], mm[2], acc[4];
            const float *src = ow + (lane / 4) * kPitch + g * 8 + (lane % 4) * 2;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = lane / 4 + 8 * k;
                mm[k] = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) mm[k] = fmaxf(mm[k], mw[w * kRows + r]);
                ll[k] = acc[2 * k] = acc[2 * k + 1] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = exp2_approx(mw[w * kRows + r] - attn_base(mm[k]));
                    const float2 x = *reinterpret_cast<const float2 *>(src + (w * kRows + 8 * k) * kPitch);
                    ll[k] += f * mw[(kWarps + w) * kRows + r];
                    acc[2 * k] += f * x.x;
                    acc[2 * k + 1] += f * x.y;
                }
            }
            if (!whole) *attn_part(s, part, 0, g, lane) = make_float4(acc[0], acc[1], acc[2], acc[3]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = lane / 4 + 8 * k;
                int token, head;
                if (whole && attn_row(s, q.q0, q.n, cur.head, cur.row_tile, r, &token, &head)) {
                    const float inv = attn_inverse(ll[k]);
                    *reinterpret_cast<uint32_t *>((T *)a.out + token * a.out_token_stride + head * a.out_head_stride +
                                                  g * 8 + lane % 4 * 2) = pack16<T>(acc[2 * k] * inv, acc[2 * k + 1] * inv);
                }
                if (!whole && g == 0 && lane % 4 == 0) {
                    part[kRows * dim + r] = mm[k];
                    part[kRows * dim + kRows + r] = ll[k];
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
        __syncthreads();  // the join's reads are done before the ring is filled again
    }
}

// A piece of a row, its output to base pm and its sum, added to what there is.
__device__ __forceinline__ void attn_add(float &m, float &l, float &x, float &y, float pm, float pl, float px, float py) {
    const float top = fmaxf(m, pm), base = attn_base(top);
    const float f = exp2_approx(m - base), g = exp2_approx(pm - base);
    m = top;
    l = l * f + pl * g;
    x = x * f + px * g;
    y = y * f + py * g;
}

// Joins the row tiles that several CTAs shared: blocks (c, y) take the tile that CTA c began, a warp 16
// rows and 8 columns at a time, a lane two columns of two rows. Where there are many pieces the block's
// warps share them out; either way the pieces are added in one fixed order. It is a chain of two loads,
// so each warp has four pieces in flight.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads)
attn_join_kernel(const __grid_constant__ AttnArgs s, int ctas) {
    constexpr int kJoinWarps = kJoinThreads / 32;
    __shared__ float shared[kJoinWarps][32][8];  // outputs, maxima and sums of a warp's share
    grid_dependency_wait();
    allow_dependents_launch();
    const ks_attention_args_t &a = s.a;
    const int c = blockIdx.x, dim = (int)a.head_dim, groups = dim / 8;
    const AttnJoin j = attn_joins(s, ctas)[c];
    if (j.pieces <= 0) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rows = min(s.tile_tokens, j.q_len - j.row_tile * s.tile_tokens) * s.tile_heads;
    const int items = (rows + 15) / 16 * groups;
    // Warps that share the pieces of one item: what leaves a warp the fewest chains of loads, its items
    // times the fours of pieces that it takes of each.
    int shares = 1, chains = 0x7fffffff;
#pragma unroll
    for (int n = 1; n <= kJoinWarps; n *= 2) {
        const int at_once = gridDim.y * (kJoinWarps / n), fours = (j.pieces + 4 * n - 1) / (4 * n);
        const int mine = (items + at_once - 1) / at_once * fours;
        if (mine < chains) {
            chains = mine;
            shares = n;
        }
    }
    const int share = warp % shares, at_once = kJoinWarps / shares;
    for (int first = blockIdx.y * at_once; first < items; first += gridDim.y * at_once) {
        const int item = first + warp / shares, group = item / groups, col = item % groups;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f}, acc[4] = {};
        if (item < items) {
            const int r = group * 16 + lane / 4;
            for (int i0 = share; i0 < j.pieces; i0 += 4 * shares) {
                float4 x[4];
                float pm[4][2], pl[4][2];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int i = i0 + u * shares;
                    if (i >= j.pieces) continue;
                    float *part = attn_slot(s, c + i * s.lanes, i == 0 ? 1 : 0);
                    x[u] = *attn_part(s, part, group, col, lane);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        pm[u][k] = part[s.rows * dim + r + 8 * k];
                        pl[u][k] = part[s.rows * dim + s.rows + r + 8 * k];
                    }
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (i0 + u * shares >= j.pieces) continue;
                    const float v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                    for (int k = 0; k < 2; ++k) attn_add(m[k], l[k], acc[2 * k], acc[2 * k + 1], pm[u][k], pl[u][k], v[2 * k], v[2 * k + 1]);
                }
            }
        }
        if (shares > 1) {
            float *mine = shared[warp][lane];
            for (int k = 0; k < 4; ++k) mine[k] = acc[k];
            for (int k = 0; k < 2; ++k) {
                mine[4 + k] = m[k];
                mine[6 + k] = l[k];
            }
            __syncthreads();
            if (share == 0)
                for (int w = 1; w < shares; ++w) {
                    const float *other = shared[warp + w][lane];
                    for (int k = 0; k < 2; ++k)
                        attn_add(m[k], l[k], acc[2 * k], acc[2 * k + 1], other[4 + k], other[6 + k], other[2 * k], other[2 * k + 1]);
                }
            __syncthreads();
        }
        if (share == 0 && item < items) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                int token, head;
                if (!attn_row(s, j.q0, j.q_len, j.head, j.row_tile, group * 16 + lane / 4 + 8 * k, &token, &head)) continue;
                const float inv = attn_inverse(l[k]) * s.out_scale;
                *reinterpret_cast<uint32_t *>((T *)a.out + token * a.out_token_stride + head * a.out_head_stride + col * 8 +
                                              lane % 4 * 2) = pack16<T>(acc[2 * k] * inv, acc[2 * k + 1] * inv);
            }
        }
    }
}

// ------------------------------------------------------------------------------- host side

int64_t ceil_to(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How a call is launched: the row-tile height, the keys of a unit and the CTAs. Depends on
// host-known sizes only.
struct AttnPlan {
    AttnArgs s;
    int ctas;
    const void *kernel;  // the 16-row kernel, NULL for the tensor-core one
    int smem;
};

template <typename T>
const void *rows16_kernel(int dim, int *smem, int *per_sm) {
    if (dim <= 64) {
        *smem = Rows16<64>::kSmem;
        *per_sm = Rows16<64>::kCtasPerSm;
        return (const void *)attn_rows16_kernel<T, 64>;
    }
    if (dim <= 128) {
        *smem = Rows16<128>::kSmem;
        *per_sm = Rows16<128>::kCtasPerSm;
        return (const void *)attn_rows16_kernel<T, 128>;
    }
    *smem = Rows16<256>::kSmem;
    *per_sm = Rows16<256>::kCtasPerSm;
    return (const void *)attn_rows16_kernel<T, 256>;
}

// Up to 16 rows per key/value head fill one tile of the 16-row kernel; more go to the tensor-core
// kernel where it takes the call's pages.
bool attn_many_rows(const ks_attention_args_t &a) {
    const int64_t q_len = a.max_q_len > 0 && a.max_q_len < a.tokens ? a.max_q_len : a.tokens;
    return q_len * (a.q_heads / a.kv_heads) > kRows;
}

void attn_plan(const ks_attention_args_t &a, bool tc, int sms, AttnPlan *p) {
    p->s.a = a;
    p->s.scale_log2 = a.scale * 1.4426950408889634f;
    p->s.out_scale = 1.0f;
    p->s.lanes = 1;
    if (tc) attn_shape(&p->s, attn_tc_rows(), attn_tc_unit(), attn_tc_tile_cost());
    else attn_shape(&p->s, kRows, kUnit, kTileCost);
    int per_sm = 1;
    p->smem = 0;
    p->kernel = nullptr;
    if (!tc) p->kernel = a.dtype == KS_DTYPE_BF16 ? rows16_kernel<__nv_bfloat16>((int)a.head_dim, &p->smem, &per_sm)
                                         : rows16_kernel<__half>((int)a.head_dim, &p->smem, &per_sm);
    p->ctas = attn_ctas(p->s, (int64_t)sms * per_sm);
}

}  // namespace

void attn_shape(AttnArgs *s, int rows, int unit, int tile_cost) {
    const ks_attention_args_t &a = s->a;
    s->group = (int32_t)(a.q_heads / a.kv_heads);
    s->rows = rows;
    s->tile_cost = tile_cost;
    s->unit_shift = 0;
    while (1 << s->unit_shift < unit) ++s->unit_shift;
    s->head_splits = (int32_t)ceil_to(s->group, rows);
    s->tile_heads = (int32_t)ceil_to(s->group, s->head_splits);
    s->tile_tokens = s->head_splits > 1 ? 1 : rows / s->tile_heads;
}

int attn_ctas(const AttnArgs &s, int64_t most) {
    const ks_attention_args_t &a = s.a;
    const int64_t tiles = ceil_to(a.tokens, s.tile_tokens) + a.seqs;
    const int64_t tile_units = ceil_to(a.table_pages * a.page_size, 1 << s.unit_shift) + 1 + s.tile_cost;
    const int64_t heads = a.kv_heads * s.head_splits;
    if (tile_units < most && tiles < most && heads < most && tile_units * tiles * heads < most)
        return (int)(tile_units * tiles * heads);
    return (int)most;
}

int64_t attn_workspace_bytes(const AttnArgs &s, int ctas) {
    return ctas * (2 * attn_slot_floats(s.rows, s.a.head_dim) * (int64_t)sizeof(float) + (int64_t)sizeof(AttnJoin));
}

ks_status_t attn_check_sizes(const ks_attention_args_t &a) {
    if (a.dtype == KS_DTYPE_F32)
        return fail(KS_ERR_UNSUPPORTED_DTYPE, "paged attention takes float16 and bfloat16 (its products run on the tensor cores)");
    const int e = elem_bytes((ks_dtype_t)a.dtype);
    if (e == 0) return fail(KS_ERR_UNSUPPORTED_DTYPE, "dtype code %d is not a ks_dtype_t", (int)a.dtype);
    if (a.tokens < 0 || a.tokens > kMaxTokens || a.seqs < 0 || a.seqs > kMaxSeqs)
        return fail(KS_ERR_INVALID_ARGUMENT, "tokens must be in 0 .. %d and seqs in 0 .. %d", kMaxTokens, kMaxSeqs);
    if (a.head_dim < 8 || a.head_dim > 256 || a.head_dim % 8)
        return fail(KS_ERR_INVALID_ARGUMENT, "head_dim must be a multiple of 8 in 8 .. 256 (got %lld)", (long long)a.head_dim);
    if (a.kv_heads < 1 || a.q_heads < 1 || a.q_heads > 65536 || a.q_heads % a.kv_heads)
        return fail(KS_ERR_INVALID_ARGUMENT, "q_heads must be a multiple of kv_heads, both in 1 .. 65536");
    if (a.page_size < 1 || a.page_size > (1 << 20) || a.pages < 0 || a.pages > 0x7fffffff)
        return fail(KS_ERR_INVALID_ARGUMENT, "page_size must be in 1 .. 2^20 and pages in 0 .. 2^31-1");
    if (a.table_pages < 0 || a.table_pages > 0x7fffffff || a.table_stride < 0)
        return fail(KS_ERR_INVALID_ARGUMENT, "the page table's sizes are out of range");
    if (a.max_q_len < 0) return fail(KS_ERR_INVALID_ARGUMENT, "max_q_len must be >= 0");
    if (a.flags & ~KS_ATTENTION_CAUSAL) return fail(KS_ERR_INVALID_ARGUMENT, "unknown attention flags 0x%x", (unsigned)a.flags);
    return KS_SUCCESS;
}

int64_t attn_rows_bytes(const ks_attention_args_t &a, int64_t token, int64_t head) {
    return ((a.tokens - 1) * token + (a.q_heads - 1) * head + a.head_dim) * 2;
}

bool attn_out_apart(const ks_attention_args_t &a) {
    const int64_t D = a.head_dim, T = a.tokens;
    const bool heads_inner = (a.q_heads == 1 || a.out_head_stride >= D) &&
                             (T == 1 || a.out_token_stride >= (a.q_heads - 1) * a.out_head_stride + D);
    const bool tokens_inner = (T == 1 || a.out_token_stride >= D) &&
                              (a.q_heads == 1 || a.out_head_stride >= (T - 1) * a.out_token_stride + D);
    return heads_inner || tokens_inner;
}

namespace {

int64_t attn_pool_bytes(const ks_attention_args_t &a, int64_t page, int64_t slot, int64_t head) {
    return a.pages > 0 ? ((a.pages - 1) * page + (a.page_size - 1) * slot + (a.kv_heads - 1) * head + a.head_dim) * 2 : 0;
}

// Whether n bytes at p cross q or the cache.
bool attn_crosses_inputs(const ks_attention_args_t &a, const void *p, int64_t n) {
    return overlaps(p, n, a.q, attn_rows_bytes(a, a.q_token_stride, a.q_head_stride)) ||
           (a.pages > 0 &&
            (overlaps(p, n, a.k_pages, attn_pool_bytes(a, a.k_page_stride, a.k_slot_stride, a.k_head_stride)) ||
             overlaps(p, n, a.v_pages, attn_pool_bytes(a, a.v_page_stride, a.v_slot_stride, a.v_head_stride))));
}

}  // namespace

// The kernels read these while other blocks write the output and the workspace, and every block has to
// read the same.
// (The table's rows are an axis that v does not have.)
bool attn_crosses_indices(const ks_attention_args_t &a, const Strided &v) {
    return (a.table_pages > 0 &&
            strided_cross(v, {a.page_table, a.table_pages * 4, {1, 1, a.seqs}, {0, 0, a.table_stride * 4}})) ||
           strided_cross(v, {a.kv_lens, a.seqs * 4, {1, 1, 1}, {0, 0, 0}}) ||
           strided_cross(v, {a.q_starts, (a.seqs + 1) * 4, {1, 1, 1}, {0, 0, 0}});
}

namespace {

ks_status_t attn_check_tensors(const ks_attention_args_t &a) {
    if (!std::isfinite(a.scale * 1.4426950408889634f))
        return fail(KS_ERR_INVALID_ARGUMENT, "scale (times log2 e) must be finite");
    if (a.tokens == 0 || a.seqs == 0) return KS_SUCCESS;
    if (!a.out || !a.q || !a.kv_lens || !a.q_starts || (a.table_pages > 0 && !a.page_table) ||
        (a.pages > 0 && (!a.k_pages || !a.v_pages)))
        return fail(KS_ERR_INVALID_ARGUMENT, "NULL pointer with tokens > 0");
    if (misaligned(4, a.kv_lens, a.q_starts, a.page_table))
        return fail(KS_ERR_INVALID_ARGUMENT, "kv_lens, q_starts and page_table must be aligned to 4 bytes");
    const int64_t strides[] = {a.q_token_stride, a.q_head_stride, a.out_token_stride, a.out_head_stride,
                               a.k_page_stride, a.k_slot_stride, a.k_head_stride,
                               a.v_page_stride, a.v_slot_stride, a.v_head_stride};
    const int64_t counts[] = {a.tokens, a.q_heads, a.tokens, a.q_heads, a.pages, a.page_size, a.kv_heads,
                              a.pages, a.page_size, a.kv_heads};
    for (int i = 0; i < 10; ++i) {
        if (strides[i] < 0 || (__int128)strides[i] * counts[i] > ((__int128)1 << 60))
            return fail(KS_ERR_INVALID_ARGUMENT, "a stride is negative or a tensor too large");
        if (counts[i] > 1 && strides[i] % 8)
            return fail(KS_ERR_INVALID_ARGUMENT, "strides must be multiples of 8 elements (16 bytes)");
    }
    if ((__int128)a.table_stride * a.seqs > ((__int128)1 << 60))
        return fail(KS_ERR_INVALID_ARGUMENT, "the page table is too large");
    if (((uintptr_t)a.q | (uintptr_t)a.out | (uintptr_t)a.k_pages | (uintptr_t)a.v_pages) & 15u)
        return fail(KS_ERR_INVALID_ARGUMENT, "q, out and the cache must be aligned to 16 bytes");
    if (!attn_out_apart(a)) return fail(KS_ERR_OVERLAP, "rows of out share storage");
    if (attn_crosses_inputs(a, a.out, attn_rows_bytes(a, a.out_token_stride, a.out_head_stride)))
        return fail(KS_ERR_OVERLAP, "out overlaps q or the cache");
    if (attn_crosses_indices(a, {a.out, a.head_dim * 2, {a.tokens, a.q_heads, 1}, {a.out_token_stride * 2, a.out_head_stride * 2, 0}}))
        return fail(KS_ERR_OVERLAP, "out overlaps the page table, kv_lens or q_starts");
    return KS_SUCCESS;
}

}  // namespace

cudaError_t attn_join_launch(const AttnArgs &s, int ctas, cudaStream_t stream) {
    // The join is scheduled while the last CTAs finish and waits for them on the device.
    AttnArgs args = s;
    void *jp[] = {&args, &ctas};
    const void *f = s.a.dtype == KS_DTYPE_BF16 ? (const void *)attn_join_kernel<__nv_bfloat16>
                                               : (const void *)attn_join_kernel<__half>;
    // Half a block for each of a tile's items, without more blocks than start at once (measured, one
    // token over 1000 keys: 11.6 us, with half as many blocks the same, with twice 13.3).
    const int items = s.rows / 16 * (int)(s.a.head_dim / 8), blocks = items / 2 < 32 ? items / 2 : 32;
    return launch_kernel(f, dim3((unsigned)ctas, (unsigned)(blocks < 1 ? 1 : blocks)), dim3(kJoinThreads), 0, jp, stream,
                         true);
}

int fault_flags_attention(bool clear) { return fault_flags_t(clear); }

}  // namespace ks

using namespace ks;

extern "C" {

ks_status_t ks_paged_attention_workspace(const ks_attention_args_t *args, int64_t *bytes) {
    if (!args || !bytes) return fail(KS_ERR_INVALID_ARGUMENT, "args or bytes is NULL");
    *bytes = 0;
    ks_status_t st = attn_check_sizes(*args);
    if (st != KS_SUCCESS || args->tokens == 0 || args->seqs == 0) return st;
    int sms = 0;
    if ((st = device_sms(&sms)) != KS_SUCCESS) return st;
    AttnPlan p;
    attn_plan(*args, false, sms, &p);
    *bytes = attn_workspace_bytes(p.s, p.ctas);
    if (attn_many_rows(*args) && attn_tc_sizes(*args)) {
        attn_plan(*args, true, sms, &p);
        const int64_t more = attn_workspace_bytes(p.s, p.ctas);
        *bytes = *bytes > more ? *bytes : more;
    }
    return KS_SUCCESS;
}

ks_status_t ks_paged_attention(const ks_attention_args_t *args, ks_stream_t stream) {
    if (!args) return fail(KS_ERR_INVALID_ARGUMENT, "args is NULL");
    ks_status_t st = attn_check_sizes(*args);
    if (st == KS_SUCCESS) st = attn_check_tensors(*args);
    if (st != KS_SUCCESS || args->tokens == 0 || args->seqs == 0) return st;
    if (!args->workspace || ((uintptr_t)args->workspace & 15u))
        return fail(KS_ERR_INVALID_ARGUMENT, "the workspace must be device memory aligned to 16 bytes");
    int sms = 0;
    if ((st = device_sms(&sms)) != KS_SUCCESS) return st;
    AttnPlan p;
    attn_plan(*args, attn_many_rows(*args) && attn_tc_fits(*args), sms, &p);
    const int64_t need = attn_workspace_bytes(p.s, p.ctas);
    if (args->workspace_bytes < need)
        return fail(KS_ERR_INVALID_ARGUMENT, "the workspace has %lld bytes, %lld are needed",
                    (long long)args->workspace_bytes, (long long)need);
    if (overlaps(args->workspace, need, args->out, attn_rows_bytes(*args, args->out_token_stride, args->out_head_stride)) ||
        attn_crosses_inputs(*args, args->workspace, need) || attn_crosses_indices(*args, {args->workspace, need, {1, 1, 1}, {0, 0, 0}}))
        return fail(KS_ERR_OVERLAP, "the workspace overlaps out or what the call reads");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t ce;
    if (p.kernel) {
        if (!allow_smem(p.kernel, (size_t)p.smem)) return fail(KS_ERR_CUDA, "shared memory of %d bytes refused", p.smem);
        void *kp[] = {&p.s};
        ce = launch_kernel(p.kernel, dim3((unsigned)p.ctas), dim3(kThreads), (size_t)p.smem, kp, s, launch_pdl_enabled());
    } else {
        ce = attn_tc_launch(p.s, p.ctas, s, launch_pdl_enabled());
    }
    if (ce == cudaSuccess && p.ctas > 1) ce = attn_join_launch(p.s, p.ctas, s);
    if (ce != cudaSuccess) return fail(KS_ERR_CUDA, "launch: %s", cudaGetErrorString(ce));
    return KS_SUCCESS;
}

}  // extern "C"
