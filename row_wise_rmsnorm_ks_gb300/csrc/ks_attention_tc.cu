// Paged attention on the fifth-generation tensor cores, for many query rows per key/value head
// (chunks of a prompt, batches of chunks and single tokens).
//
// A CTA works on a row tile of 256 query rows, two tiles of 128 that share every 128-key step of
// the cache: S = Q K^T and O += P V are tcgen05.mma with S, P and O in tensor memory, which they
// fill exactly (two 128-column S, over which P is written, two 128-column O). Twenty warps:
//   warps 0-7, 8-15  softmax of tile 0 and 1, 16 rows a warp: S to registers, running maximum,
//                    exponentials, P back to tensor memory; at the end of a row tile O to the output or
//                    the workspace;
//   warps 16 and 18  issue the matrix instructions of tile 0 and 1: P V, then Q K(next), which
//                    overwrites S and P behind it in order;
//   warp 17          copies queries and pages to shared memory by TMA, for pages one lane per page and
//                    64 columns;
//   warp 19          clears value rows behind the last key that the row tile sees.
// While one tile is in its softmax, the matrix instructions of the other run. A row's base is the
// maximum of the first scores it saw until later probabilities outgrow it (kGrowth): only then is it
// raised and O scaled. The quotient does not depend on the base, and FP32 sums and bf16 probabilities
// keep their relative precision at any size. fp16 ends at 65504 and is normal down to 2^-14: a probability to the
// base counts 2^8 there (kLift), which leaves the base to be outgrown by 2^8, keeps the precision of
// probabilities down to 2^-22 of the row's largest and loses none above 2^-33 of it.
//
// Bound by the tensor cores for long chunks: a step of both tiles is 32 instructions of 64 cycles at
// dim 128. Measured: 8192 tokens over 16384 keys, 32 query and 8 key/value heads of 128, bf16, 0.92 ms
// or 1.79 PFLOP/s (2580 cycles a step; the softmax of a tile is 850 to 1100 of them, beside the other
// tile's products); called back to back, at the power limit's clock, 1.01 ms. Few rows of a tile make it a
// stream of the cache: 64 contexts of 6000 keys, 20 rows, 296 us or 5.3 TB/s, 4 of 30000 103 us or 4.8. What
// holds these below the copy rate is not known: 152 rings of 160 KB are 3.7 us of that rate, more than a
// copy's latency, but a step's page numbers are read only when its turn to be copied has come.
#include <mutex>

#include "ks_attention_tc.cuh"

namespace ks {
namespace {

// ------------------------------------------------------------------------------- host side

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static std::once_flag once;
    static EncodeTiled f = nullptr;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) == cudaSuccess &&
            found == cudaDriverEntryPointSuccess)
            f = (EncodeTiled)p;
        else
            (void)cudaGetLastError();
    });
    return f;
}

// The pool as a 4-dimensional tensor, columns, slots, heads, pages; boxes of 64 columns and as many
// slots as a step takes of a page. Columns past head_dim and pages past the pool read as zeros.
bool pool_map(CUtensorMap *map, const ks_attention_args_t &a, const void *p, int64_t page, int64_t slot, int64_t head) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.page_size, (cuuint64_t)a.kv_heads, (cuuint64_t)a.pages};
    // a dimension of one entry has no stride of its own: any valid one
    const cuuint64_t strides[3] = {(cuuint64_t)(a.page_size > 1 ? slot * 2 : 16 * ((a.head_dim + 7) / 8)),
                                   (cuuint64_t)(a.kv_heads > 1 ? head * 2 : 16 * ((a.head_dim + 7) / 8)),
                                   (cuuint64_t)(a.pages > 1 ? page * 2 : 16 * ((a.head_dim + 7) / 8))};
    const cuuint32_t box[4] = {64, (cuuint32_t)(a.page_size < kKeys ? a.page_size : kKeys), 1, 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    return encode(map, a.dtype == KS_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                  const_cast<void *>(p), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool attn_query_map(CUtensorMap *map, const AttnArgs &s) {
    const ks_attention_args_t &a = s.a;
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t row = 16 * ((a.head_dim + 7) / 8);
    const cuuint64_t dims[3] = {(cuuint64_t)a.head_dim, (cuuint64_t)a.q_heads, (cuuint64_t)a.tokens};
    const cuuint64_t strides[2] = {a.q_heads > 1 ? (cuuint64_t)a.q_head_stride * 2 : row,
                                   a.tokens > 1 ? (cuuint64_t)a.q_token_stride * 2 : row};
    const cuuint32_t box[3] = {64, (cuuint32_t)s.tile_heads, (cuuint32_t)s.tile_tokens};
    const cuuint32_t steps[3] = {1, 1, 1};
    return encode(map, a.dtype == KS_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                  const_cast<void *>(a.q), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool attn_codes_map(CUtensorMap *map, const AttnArgs &s, const Pool4 &pool) {
    const ks_attention_args_t &a = s.a;
    const EncodeTiled encode = encode_tiled();
    if (!encode) return false;
    const cuuint64_t row = (cuuint64_t)(a.head_dim <= 64 ? 32 : 64);  // places past head_dim read as zeros
    const cuuint64_t dims[4] = {(cuuint64_t)a.head_dim / 2, (cuuint64_t)a.page_size, (cuuint64_t)a.kv_heads, (cuuint64_t)a.pages};
    const cuuint64_t strides[3] = {a.page_size > 1 ? (cuuint64_t)pool.code_slot : row, a.kv_heads > 1 ? (cuuint64_t)pool.code_head : row,
                                   a.pages > 1 ? (cuuint64_t)pool.code_page : row};
    const cuuint32_t box[4] = {(cuuint32_t)row, (cuuint32_t)(a.page_size < kKeys ? a.page_size : kKeys), 1, 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t *>(pool.codes), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

template <typename T>
const void *tc_kernel(int dim, int *smem) {
    *smem = dim <= 64 ? Tc<64>::kSmem : Tc<128>::kSmem;
    return dim <= 64 ? (const void *)attn_tc_kernel<T, 64, Pages16> : (const void *)attn_tc_kernel<T, 128, Pages16>;
}

}  // namespace

bool attn_tc_sizes(const ks_attention_args_t &a) {
    // a copy's box begins on an 8-row group of the swizzled tile, and a step is whole pages or part of one
    return a.head_dim <= 128 && a.page_size % 8 == 0 && (kKeys % a.page_size == 0 || a.page_size % kKeys == 0);
}

bool attn_tc_fits(const ks_attention_args_t &a) {
    if (!attn_tc_sizes(a)) return false;
    // the tensor map's strides are below 2^40 bytes and not zero
    const int64_t strides[8] = {a.k_page_stride, a.k_slot_stride, a.k_head_stride, a.v_page_stride,
                                a.v_slot_stride, a.v_head_stride, a.q_token_stride, a.q_head_stride};
    const int64_t counts[8] = {a.pages, a.page_size, a.kv_heads, a.pages, a.page_size, a.kv_heads, a.tokens, a.q_heads};
    for (int i = 0; i < 8; ++i)
        if (counts[i] > 1 && (strides[i] == 0 || strides[i] >= (1ll << 39))) return false;
    return a.pages > 0;
}

int attn_tc_rows() { return kRows; }
int attn_tc_unit() { return kKeys; }
int attn_tc_tile_cost() { return kTileCost; }

cudaError_t attn_tc_launch(const AttnArgs &s, int ctas, cudaStream_t stream, bool pdl) {
    const ks_attention_args_t &a = s.a;
    AttnArgs args = s;
    CUtensorMap q_map;
    Pages16 pages;
    if (!attn_query_map(&q_map, s) ||
        !pool_map(&pages.k, a, a.k_pages, a.k_page_stride, a.k_slot_stride, a.k_head_stride) ||
        !pool_map(&pages.v, a, a.v_pages, a.v_page_stride, a.v_slot_stride, a.v_head_stride))
        return cudaErrorInvalidValue;
    int smem = 0;
    const void *f = a.dtype == KS_DTYPE_BF16 ? tc_kernel<__nv_bfloat16>((int)a.head_dim, &smem)
                                             : tc_kernel<__half>((int)a.head_dim, &smem);
    if (!allow_smem(f, (size_t)smem)) return cudaErrorInvalidConfiguration;
    void *kp[] = {&args, &q_map, &pages};
    return launch_kernel(f, dim3((unsigned)ctas), dim3(Split<false>::kThreads), (size_t)smem, kp, stream, pdl);
}

int fault_flags_attention_tc(bool clear) { return fault_flags_t(clear); }

}  // namespace ks
