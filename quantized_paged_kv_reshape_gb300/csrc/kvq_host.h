// Host helpers shared by the translation units that implement the C ABI.
#pragma once

#include <cstdint>

#include "../../include/kvq.h"
#include "kvq_common.cuh"

namespace kvq {

// Records a message for kvq_last_error() and returns `st`; ok() clears it.
kvq_status fail(kvq_status st, const char* fmt, ...);
kvq_status ok();

bool fmt_ok(kvq_format f);
int side_of(kvq_format f, int side);
const Codebooks& codebooks();
int sm_count();                 // of the current device, 0 on error
bool aligned16(const void* p);
int rmax_for(int rep);          // GQA ratio rounded up to a power of two, 0 above 8

// What queries that become 16-bit operands before the score scale are
// multiplied by, a power of two (no bits change; the rest of the scale is taken
// after the products).  1 beside BF16 keys, and for score scales between 2^-14
// and 4, so for any of a usual model.  Otherwise queries of ordinary scores may
// lie outside fp16's range (an FP8 scale or sm_scale far from one): the rest of
// the scale is then in [2^-6, 2^-5), which leaves such queries around one.
float query_factor(int k_side, float score_scale);

// kvq_paged_decode that also stores each row's base-2 log-sum-exp of the
// scaled scores (-inf for a row that attends to nothing) when lse is not null.
kvq_status decode_with_lse(const void* q, kvq_dtype q_dtype, int64_t q_stride, const void* k_cache,
                           const void* v_cache, void* out, kvq_dtype out_dtype, float* lse,
                           const int32_t* block_tables, int32_t max_blocks, const int32_t* seq_lens,
                           int32_t num_seqs, int64_t num_blocks, int32_t nq, int32_t nkv, int32_t hd, int32_t bs,
                           int64_t k_bstride, int64_t v_bstride, float sm_scale, float k_scale, float v_scale,
                           int32_t window, float sparse_v_threshold, void* workspace, size_t workspace_bytes,
                           kvq_format fmt, int32_t* error_flag, void* stream);

}  // namespace kvq
