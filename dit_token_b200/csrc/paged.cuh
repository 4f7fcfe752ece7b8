// paged.cuh -- device helpers of the attention kernels over a paged cache:
// tiles of a ragged batch, the keys a query sees, and where a token's keys lie.
#pragma once

#include <cmath>

#include "common.cuh"
#include "launch.h"

namespace dit {

// The queries of one sequence and one key head form a matrix of
// rows (token, head of the group), token-major: row i is token i / G, q head
// kvh * G + i % G.  Tiles of R such rows never cross a sequence.
struct QueryTile {
    int seq;
    int first;      // first row of the tile (token * G + head)
    int rows;       // rows of the tile that exist (1 .. R)
    int n;          // tokens of the sequence's chunk
    int row0;       // padded row of the sequence's first token
    int ordinal0;   // valid-row ordinal of the sequence's first token
    int kv_len;     // keys the sequence claims
    int kv_end;     // keys that the table can name (<= kv_len)
};

// Rows of sequence b's chunk: those that are valid and have a padded row; 0 for a
// sequence that does not lie inside the buffer, which is skipped whole.  Every
// kernel asks here, so that they agree on which rows exist.
__device__ __forceinline__ int chunk_rows(const PagedParams& p, int b, int& ordinal0, int& row0)
{
    ordinal0 = __ldg(p.pk.cu_seqlens + b);
    row0 = __ldg(p.pk.cu_seqlens_padded + b);
    const int n = min(__ldg(p.pk.cu_seqlens + b + 1) - ordinal0, __ldg(p.pk.cu_seqlens_padded + b + 1) - row0);
    if (row0 < 0 || ordinal0 < 0 || n <= 0 || (long long)row0 + n > p.pk.num_rows_padded ||
        (long long)ordinal0 + n > p.pk.num_rows_padded)
        return 0;
    return n;
}

// Tile t of the batch, or false past the last one.  Warp-collective: 32
// sequences per round, their tile counts summed by a shuffle scan.
__device__ __forceinline__ bool map_query_tile(int t, const PagedParams& p, int R, int lane, QueryTile& q)
{
    int before = 0;
    for (int base = 0; base < p.pk.num_seqs; base += kWarp) {
        const int b = base + lane;
        int n = 0, tiles = 0, c0 = 0, row0 = 0, kv = 0;
        if (b < p.pk.num_seqs) {
            kv = __ldg(p.kv_lens + b);
            n = chunk_rows(p, b, c0, row0);
            tiles = (long long)n * p.group <= p.skip_rows ? 0 : (int)(((long long)n * p.group + R - 1) / R);
        }
        int sum = tiles;
#pragma unroll
        for (int o = 1; o < kWarp; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o)
                sum += up;
        }
        const unsigned m = __ballot_sync(0xffffffffu, t < before + sum);
        if (m != 0u) {
            const int l = __ffs(m) - 1;
            const int excl = __shfl_sync(0xffffffffu, sum - tiles, l);
            q.seq = base + l;
            q.n = __shfl_sync(0xffffffffu, n, l);
            q.row0 = __shfl_sync(0xffffffffu, row0, l);
            q.ordinal0 = __shfl_sync(0xffffffffu, c0, l);
            q.first = (t - before - excl) * R;
            q.rows = min(R, q.n * p.group - q.first);
            q.kv_len = max(__shfl_sync(0xffffffffu, kv, l), 0);
            q.kv_end = (int)min((long long)q.kv_len, (long long)p.max_pages * p.page_size);
            return true;
        }
        before += __shfl_sync(0xffffffffu, sum, kWarp - 1);
    }
    return false;
}

// Keys [lo, hi) that token i of the chunk sees: its own position is
// kv_len - n + i (the chunk's tokens are the cache's last ones).
__device__ __forceinline__ void visible_keys(const PagedParams& p, const QueryTile& q, int token, int& lo, int& hi)
{
    const int pos = q.kv_len - q.n + token;
    hi = p.causal ? min(pos, q.kv_end - 1) + 1 : q.kv_end;
    lo = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
}

// The entry of a sequence's table that holds a token.
__device__ __forceinline__ unsigned page_of(const PagedParams& p, int key)
{
    return (unsigned)(((unsigned long long)(unsigned)key * p.page_mul) >> p.page_shift);
}

// Element offset of a token's slot in the cache, or -1 where the table names
// no page of the cache.
__device__ __forceinline__ int64_t key_offset(const PagedParams& p, const int32_t* table, int key)
{
    const unsigned entry = page_of(p, key);
    const int page = __ldg(table + entry);
    if (page < 0 || page >= p.num_pages)
        return -1;
    return (int64_t)page * p.page_stride + (int64_t)(key - (int)entry * p.page_size) * p.slot_stride;
}

// 16 bytes from global to shared memory, or 16 zero bytes: keys behind the
// last token must read as zeros, because the cache may hold anything there
// and 0 * NaN would reach the sums.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Partial results of one split, per (valid-row ordinal, q head): the
// unnormalised sum over its keys and (largest score, sum of exponentials), in
// powers of two.
__device__ __forceinline__ int64_t partial_index(const PagedParams& p, int ordinal, int head, int split)
{
    return ((int64_t)ordinal * p.num_q_heads + head) * p.splits + split;
}

constexpr float kLn2 = 0.69314718055994530942f;

}  // namespace dit
