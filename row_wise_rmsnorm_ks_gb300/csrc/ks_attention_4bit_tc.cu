// Paged attention over 4-bit pages on the fifth-generation tensor cores: the kernel of ks_attention_tc.cu, its operands
// fp16, with four more warps that make the tiles of keys and values.
//
// Code times scale is an fp16 number exactly, and so enters the matrix instructions without a rounding; the pools'
// factors go into the scores' scale and the output's. A thread of the four warps has one key of a step: 64 bytes of codes
// become 256 bytes in the swizzled layout, 64 conversions of a pair and as many products a tile. bf16 queries become fp16 in
// shared memory, each row times a power of two, by the warps that read their scores; fp16 probabilities follow.
//   - Where a step is whole pages or part of one, and rows of codes lie 16 bytes aligned (heads of any 32), the copying warp
//     brings the codes by tensor maps to a ring of three tiles, in 16-byte pieces swizzled for the threads' reads; the scales,
//     8 bytes a key, are read a step ahead. Other pools (any page size, odd heads of 16, unaligned rows) are copied by the four
//     warps themselves, two tiles ahead (1.07 times the time where rows are aligned; with 80 dims, whose rows are copied by 8
//     bytes, twice: 64 contexts of 4000 keys, 64 rows, 424 us for 210).
//   - 768 threads launch with 80 registers each; the softmax takes 96 (104 with 16-bit pages; 64 to 232 bytes a thread spill), the
//     four warps 56, the other four 40. Four tiles of 128 keys in the ring instead of five make room for the codes.
// Bound by issue and the chain of a step: 8192 tokens over 16384 keys, 32 query and 8 key/value heads of 128, bf16, 1.08 ms,
// 1.52 PFLOP/s; the same without making tiles 0.98, with 16-bit pages 0.92 (bf16) and 0.97 (fp16, whose probabilities need the
// lift). About 3000 cycles a step, 2048 of them products. With loads of the codes to registers 1.42, by the warps' own copies 1.16.
#include "ks_attention_tc.cuh"
#include "ks_attention_4bit.cuh"

namespace ks {

bool attn4_tc_fits(const ks_attention_args_t &a) {
    if (a.head_dim > 128 || a.pages <= 0) return false;
    // the queries' tensor map takes strides below 2^40 bytes and not zero
    const int64_t strides[2] = {a.q_token_stride, a.q_head_stride}, counts[2] = {a.tokens, a.q_heads};
    for (int i = 0; i < 2; ++i)
        if (counts[i] > 1 && (strides[i] == 0 || strides[i] >= (1ll << 39))) return false;
    return true;
}

int attn4_tc_copies(const ks_attention_args_t &a, const Pool4 &k, const Pool4 &v, bool alike, uintptr_t code_align, uintptr_t scale_align) {
    const int64_t dim = a.head_dim;
    if ((code_align & 15) != 0 || !alike) return kCopyBy8;
    bool map = dim % 32 == 0 && (scale_align & 1) == 0 && a.page_size % 8 == 0 && (kKeys % a.page_size == 0 || a.page_size % kKeys == 0);
    // the maps' strides are below 2^40 bytes and not zero
    const int64_t counts[3] = {a.pages, a.page_size, a.kv_heads};
    for (const Pool4 *p : {&k, &v}) {
        const int64_t strides[3] = {p->code_page, p->code_slot, p->code_head};
        for (int i = 0; i < 3; ++i)
            if (counts[i] > 1 && (strides[i] <= 0 || strides[i] >= (1ll << 39))) map = false;
    }
    return map ? kCopyByMap : (dim == 64 || dim == 128) && (scale_align & (dim / 16 - 1)) == 0 ? kCopyBy16 : kCopyBy8;
}

// Steps that beginning and ending a row tile costs: more than with 16-bit pages, whose next tile's first keys are there
// sooner. (Measured, us with 2, 3, 5 and 8: 16 sequences of 1..517 tokens over 392..4439 keys 212, 188, 177, 184; of sequences of
// one length, 16 of 128 tokens over 2000 keys 99, 99, 97, 97; 64 of 20 over 1000 110, 108, 106, 106; 40 of 65 over 300, 64 dims, 67,
// 67, 69, 67; 3 of 700 over 5000, 64 dims, 79, 79, 81, 85. The long prompt's does not change.)
int attn4_tc_tile_cost() { return 5; }

cudaError_t attn4_tc_launch(const Attn4Args &args, uintptr_t code_align, uintptr_t scale_align, int ctas, cudaStream_t stream,
                            bool pdl) {
    AttnArgs s = args.s;
    CUtensorMap q_map;
    if (!attn_query_map(&q_map, s)) return cudaErrorInvalidValue;
    Pages4 pages;
    pages.k = args.k;
    pages.v = args.v;
    const int dim = (int)s.a.head_dim;
    pages.whole = (dim == 64 || dim == 128) && (code_align & 15) == 0 && (scale_align & (dim / 16 - 1)) == 0 && args.alike;
    pages.page_units = args.page_units;
    pages.slot_units = args.slot_units;
    pages.by_map = attn4_tc_copies(s.a, args.k, args.v, args.alike, code_align, scale_align) == kCopyByMap;
    if (pages.by_map && (!attn_codes_map(&pages.k_map, s, args.k) || !attn_codes_map(&pages.v_map, s, args.v)))
        return cudaErrorInvalidValue;
    const bool bf16 = s.a.dtype == KS_DTYPE_BF16;
    const void *f = dim <= 64 ? (bf16 ? (const void *)attn_tc_kernel<__nv_bfloat16, 64, Pages4>
                                      : (const void *)attn_tc_kernel<__half, 64, Pages4>)
                              : (bf16 ? (const void *)attn_tc_kernel<__nv_bfloat16, 128, Pages4>
                                      : (const void *)attn_tc_kernel<__half, 128, Pages4>);
    const int smem = dim <= 64 ? Tc<64, true>::kSmem : Tc<128, true>::kSmem;
    if (!allow_smem(f, (size_t)smem)) return cudaErrorInvalidConfiguration;
    void *kp[] = {&s, &q_map, &pages};
    return launch_kernel(f, dim3((unsigned)ctas), dim3(Split<true>::kThreads), (size_t)smem, kp, stream, pdl);
}

int fault_flags_attention_4bit_tc(bool clear) { return fault_flags_t(clear); }

}  // namespace ks
