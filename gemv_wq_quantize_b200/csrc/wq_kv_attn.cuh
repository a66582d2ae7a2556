// wq_kv_attn.cuh -- arguments and entry points shared by the kernels of kv_attention.
#pragma once
#include <stdint.h>

#include "wq_host.h"
#include "wq_kv.h"

namespace wq {

struct KvAttnArgs {
    const void *q;
    void *out;
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *cu_q, *seq_len, *block_table;
    int64_t num_pages;
    int n_seqs, max_pages, M;
    int q_heads, kv_heads, group, head_dim;
    int page_shift, pitch, capacity;
    float sm_scale;
    int few_rows;         // sequences with more rows per key head go to the tile kernel
    int by_rows;          // its items are counted by rows: few_rows, or 0 (see kv_row_item)
    // The kernel for few rows, launched behind the tile kernel of the same call, runs beside it: every
    // block of the tile kernel has waited for the kernels before when it lets the next grid start,
    // so the one started needs no wait of its own for them.  It waits for the tile kernel's end at
    // its own end, so that what follows has both behind it.
    bool behind_tiles;
    float *partials;      // nullptr: every tile is walked by one block
    unsigned *arrivals;
};

// The cache's codes as tensor maps of boxes of `rows` keys by 128 bytes, swizzled as wide, and a
// launch with (key map, value map, arguments).
wq_status encode_cache(CUtensorMap *km, CUtensorMap *vm, const KvAttnArgs &a, int rows);
void set_attn_launch(PreparedLaunch &L, const void *fn, unsigned blocks, int threads, size_t smem, const CUtensorMap &km,
                     const CUtensorMap &vm, const KvAttnArgs &a);

// Few rows per key head: split over the whole GPU by key ranges (wq_kv_attn.cu).
wq_status kv_attn_rows(const KvAttnArgs &a, bool bf16, bool f8, cudaStream_t st);
size_t kv_attn_rows_workspace();

// Many rows per key head (prefill): 256-row tiles on the tensor cores (wq_kv_tiles.cu).
wq_status kv_attn_tiles(KvAttnArgs a, bool bf16, bool f8, cudaStream_t st);

}  // namespace wq
