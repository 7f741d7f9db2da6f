// Launchers of the quantised cache's write and read-back (kv_mx.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace tt {

// Where the rows of a cache are: [B, Hkv, cap, D] (table null) or pages [num_pages, Hkv,
// 1 << page_shift, D] with table [B, pages_per_seq]; `cap` positions per sequence either way.
struct MxRows {
  uint8_t *k, *v;             // e4m3, D bytes per row
  uint8_t *k_scale, *v_scale; // D / 32 bytes per row
  const int32_t* table;
  int page_shift, pages_per_seq, num_pages;
  int cap, Hkv, D;
};

// Write rows [L_n, L_n + count_n) of every sequence from bf16 rows [B, T, Hkv, D]; counts null: T
// each.  advance: L_n += count_n once every block has read it (ticket: a zeroed counter that the
// launch leaves at zero).
cudaError_t launch_kv_append_mx(const void* k_new, const void* v_new, const MxRows& m, int32_t* ctx_lens,
                                const int32_t* counts, int B, int T, int advance, unsigned* ticket,
                                unsigned* err_word, int sms, cudaStream_t stream);
// Positions [starts[n], starts[n] + T) below ctx_lens[n] as bf16 into [B, Hkv, T, D].
cudaError_t launch_kv_read_mx(const MxRows& m, const int32_t* ctx_lens, const int32_t* starts, int B, int T,
                              void* k_out, void* v_out, unsigned* err_word, int sms, cudaStream_t stream);

}  // namespace tt
