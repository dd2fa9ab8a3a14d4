// kq_attn.h — what the attention kernel and its entry point share.
#pragma once

#include "kq_layer.h"

namespace kq {

constexpr int kAttnWarps = 8;
constexpr int kChunk = 32;         // keys per chunk
// Bytes of the ring per warp: one unit in hand and one on its way (64 KB per SM
// on their way keep the memory busy; with 128 KB the 131072-key call took 94 us
// instead of 92, since what the warps themselves wait for queues behind them).
// Warps that share a stream share its ring.
constexpr int kRingAlone = 16384, kRingShared = 12288;
// Chunks' worth of work that beginning a pair is counted as when the sequence
// is cut: 256 requests of 5 to 1500 keys took 41, 31, 27, 28 us with 0, 1, 2, 3.
constexpr int kPairCost = 2;
constexpr int kMostKeys = INT32_MAX - 1023;  // of a request: key numbers a batch of pages further still fit
constexpr int kMaxBlocks = 160;    // of an attention launch

struct AttnArgs {
    int R, max_q, n_q, n_kv, G, shift, max_pages, window, tiles, vec, inv_g;
    int64_t T, ldq, ldo, table_ld, page_stride, n_pages;
    float scale;                   // times log2(e): the softmax is taken in powers of two
    const float* q;
    const void *k, *v;
    const int32_t *lens, *q_start, *table;
    float* out;
    int32_t* status;
    int4* head;                    // per block: {a pair continues in later blocks, its first column, columns,
                                   // kv head}, {the block that it ends in}
    float* part;                   // partial results (see kPart)
    int* fault;                    // device fault word (a wait that ran out)
    unsigned long long wait_ns;    // limit of a wait
    int test_hold;                 // test hook: the first block's keys of this chunk (from 1) are not handed on; 0: none
};

// More rows per pair than kTileRows always take the kernel for many rows
// (kq_attn_wide.cuh); more than half as many take it where a request may have
// kWideKeys keys.  Measured, tiles against it (us): 20 rows of 4096 keys 61 / 67,
// 32 rows 61 / 67; 40 rows of 4096 keys 86 / 64, of 1000 to 1400 62 / 52, of
// 20 to 400 50 / 61; 64 rows of 8000 keys 84 / 62, of 20 to 400 50 / 64;
// 128 rows of 4000 keys 109 / 52, 96 rows of 20 to 400 80 / 73.
constexpr int kTileRows = 64, kWideKeys = 1024;

// Runs an attention call of head_dim D on `blocks` blocks.
template <int D, bool BF16>
cudaError_t launch_attn(const AttnArgs& a, int blocks, cudaStream_t s);
template <int D, bool BF16>
cudaError_t launch_attn_wide(const AttnArgs& a, int blocks, cudaStream_t s);

}  // namespace kq
