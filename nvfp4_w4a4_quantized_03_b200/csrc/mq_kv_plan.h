// mq_kv_plan.h -- how mq_kv_attention splits a batch over the device: the rows
// of a block, the chunks of a sequence's keys, and where its workspace holds
// what.  A function of the call's sizes alone, so the workspace's size is too.
#pragma once
#include <algorithm>
#include <cstdint>

#include "mq_internal.h"

namespace mq {

constexpr int KV_BY_LENGTH_MAX = 128;     // sequences

struct KvPlan {
    int nt;                   // n-tiles of 8 rows per block (form for few rows)
    bool prefill;             // the tcgen05 form, 256 rows per block
    bool by_length;           // its blocks in the order of the keys they see
    int64_t block_rows;
    int64_t row_tiles;        // tiles of rows (new token x head of the group) per (sequence, kv head)
    int64_t cells;            // (sequence, row tile, kv head)
    int64_t chunks;           // chunks of keys per cell at max_len
    int64_t chunk_tokens;
    int64_t tickets_off, part_off, bytes;
};

inline KvPlan kv_plan(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t head_dim, int64_t max_q,
                      int64_t max_len) {
    constexpr int64_t SMS = 148, TICKETS = 4 * SMS;
    KvPlan p{};
    const int64_t rows = max_q * (q_heads / kv_heads);
    // The form for few rows has n-tiles for 16 rows per block: 16 rows take 99 us
    // in it (16 sequences of 8K, 8 kv heads of 128), 17 to 128 rows 157 to 160 in
    // the tcgen05 form, 256 rows 174.  No form in between was built.
    p.prefill = rows > 16;
    p.nt = p.prefill ? 0 : rows <= 8 ? 1 : 2;
    p.block_rows = p.prefill ? 256 : 8 * p.nt;
    p.row_tiles = (rows + p.block_rows - 1) / p.block_rows;
    p.cells = batch * p.row_tiles * kv_heads;
    // One chunk where the cells fill the device.  Else enough chunks to do so:
    // of the tcgen05 form (one block per SM) as many as run at once, of 512
    // tokens at least (the last block to finish a cell reads back 128 KB per
    // chunk); of the other (four blocks per SM) of 128 to 1024 tokens, but
    // never more than 128 of them.
    int64_t c = std::max<int64_t>(max_len, 128);
    if (p.prefill && p.cells < SMS) {
        const int64_t n = std::min<int64_t>(SMS / p.cells, 64);
        c = std::max<int64_t>((max_len + n - 1) / n, 512);
    } else if (!p.prefill && p.cells < TICKETS) {
        const int64_t want = (p.cells * max_len + TICKETS - 1) / TICKETS;
        c = std::max({std::min<int64_t>(want, 1024), (max_len + 127) / 128, (int64_t)128});
    }
    p.chunk_tokens = (c + 127) / 128 * 128;
    if (!p.prefill) p.chunk_tokens = (c + 63) / 64 * 64;
    p.chunks = std::max<int64_t>(1, (max_len + p.chunk_tokens - 1) / p.chunk_tokens);
    // More than one wave of several sequences: as they come and longest first
    // (32 / 8 heads of 128): 16 x 512 new tokens on 4K, ragged, 298 and
    // 269 us; 64 x 256 on 8K, ragged, 828 and 744; 8 prompts of 1024 tokens all
    // alike 155 and 157 (the block's look at the batch).  Beyond 128 sequences
    // the search would take longer and the last blocks weigh less.
    p.by_length = p.prefill && p.cells > SMS && batch > 1 && batch <= KV_BY_LENGTH_MAX;
    // the tickets lie where they lie for every size, so a workspace serves calls of all sizes
    p.tickets_off = (int64_t)WS_HEADER_BYTES;
    p.part_off = p.tickets_off + TICKETS * 4 / 256 * 256 + 256;
    p.bytes = p.part_off + (p.chunks > 1 ? p.cells * p.chunks * p.block_rows * (head_dim + 2) * 4 : 0);
    return p;
}

}  // namespace mq
