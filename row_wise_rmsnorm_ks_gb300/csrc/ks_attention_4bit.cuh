// What the kernels of the attention over 4-bit pages share.
#pragma once

#include "ks_attention.cuh"
#include "ks_fp4.cuh"

namespace ks {

struct Attn4Args {
    AttnArgs s;
    Pool4 k, v;
    Divisor page_blocks;  // page_size / 16, where pages are whole blocks of 16 keys
    bool alike;  // both pools have the same strides, those of the scales an eighth of the codes', and places 32 bits:
    uint32_t page_units, slot_units;  // strides of the codes' pages and slots, in 16 bytes
};

// The tensor-core kernel (ks_attention_4bit_tc.cu): whether it takes a call, how the codes of one come (by 8 bytes, by whole
// rows of 16 bytes each, by tensor maps), the steps that a row tile costs beyond its own, and its launch.
bool attn4_tc_fits(const ks_attention_args_t &a);
enum { kCopyBy8, kCopyBy16, kCopyByMap };
int attn4_tc_copies(const ks_attention_args_t &a, const Pool4 &k, const Pool4 &v, bool alike, uintptr_t code_align, uintptr_t scale_align);
int attn4_tc_tile_cost();
cudaError_t attn4_tc_launch(const Attn4Args &args, uintptr_t code_align, uintptr_t scale_align, int ctas, cudaStream_t stream,
                            bool pdl);

}  // namespace ks
