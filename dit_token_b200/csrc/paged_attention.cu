// paged_attention.cu -- attention of a chunk of new tokens over a paged cache
// on the warp-level matrix instructions, and the join of split key ranges.
//
//   s_ij = scale q_i . k_j over the keys j that row i sees,
//   o_i = sum_j exp(s_ij) v_j / sum_j exp(s_ij),  lse_i = ln sum_j exp(s_ij)
// in one pass over the keys: running maximum m, sum l and unnormalised o, all
// fp32; exp(s - m) is rounded to bf16 for its product with v (by at most 2^-8 of
// it, independently between keys); l adds the unrounded values.  A row that sees no key gives o = 0 and
// lse = -inf.
//
// The rows of a tile are the (token, head) pairs that share a key head, so
// grouped heads read each key once.  A block takes 64 of them, 16 per warp,
// and every warp all keys of a tile.  This is the kernel of the chunks that the
// tensor-memory kernel does not take (caches whose strides or page size TMA
// cannot follow); paged_attention_narrow.cu is that of next tokens.
// Key and value tiles arrive by 16-byte asynchronous copies, which take any
// page size and stride and write zeros for keys that are not there.  Bound by
// the warp-level matrix instructions and what feeds them: 163 TFLOP/s on the
// video chunk (2.74 TFLOP in 16.8 ms, 4,132 rows over 32,360 keys, 40 heads).
#include "paged_mma.cuh"
#include "paged_splits.h"

namespace dit {
namespace {

template <int D>
struct Shape {
    static constexpr int kWarps = 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRows = 16 * kWarps;
    static constexpr int kKeys = 64;                // of a tile
    static constexpr int kStages = D == 256 ? 2 : 3;
    static constexpr int kTile = kKeys * D * 2;     // bytes of a key (or value) tile
    static constexpr int kQ = kRows * D * 2;
    static constexpr int kOStride = D + 4;          // floats
    static constexpr int kO = kRows * kOStride * 4;
    static constexpr int kRing = 2 * kStages * kTile;
    static constexpr int kOffs = 2 * kKeys * 8;
    static constexpr int kMl = kRows * 8;
    static constexpr int kSmem = kQ + (kRing > kO ? kRing : kO) + kOffs + kMl;
};

template <int D>
__global__ void __launch_bounds__(Shape<D>::kThreads) paged_attention_kernel(const __grid_constant__ PagedParams p)
{
    using S = Shape<D>;
    constexpr int BN = S::kKeys, STAGES = S::kStages;
    constexpr int CH = D / 8;       // 16-byte chunks per row
    extern __shared__ __align__(128) unsigned char smem[];
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int kvh = blockIdx.y, split = blockIdx.z;
    QueryTile q;
    if (!map_query_tile(blockIdx.x, p, S::kRows, lane, q))
        return;
    unsigned char* s_q = smem;
    unsigned char* s_ring = smem + S::kQ;
    int64_t* s_offs = reinterpret_cast<int64_t*>(smem + S::kQ + (S::kRing > S::kO ? S::kRing : S::kO));
    float2* s_ml = reinterpret_cast<float2*>(reinterpret_cast<unsigned char*>(s_offs) + S::kOffs);
    const uint32_t a_q = (uint32_t)__cvta_generic_to_shared(s_q);
    const uint32_t a_ring = (uint32_t)__cvta_generic_to_shared(s_ring);

    // Keys of the tile: from the first row's lowest to the last row's highest,
    // cut into runs of split_keys; the last split takes what is left.
    int lo, hi, unused;
    visible_keys(p, q, q.first / p.group, lo, unused);
    visible_keys(p, q, (q.first + q.rows - 1) / p.group, unused, hi);
    if (p.splits > 1) {
        const long long from = lo + (long long)split * p.split_keys;
        if (split + 1 < p.splits)
            hi = (int)min((long long)hi, from + p.split_keys);
        lo = (int)min(from, (long long)hi);
    }
    const int tiles = hi > lo ? (hi - lo + BN - 1) / BN : 0;
    const int32_t* table = p.block_table + (int64_t)q.seq * p.table_stride;
    const uint16_t* kc = p.k_cache + (int64_t)kvh * p.head_stride;
    const uint16_t* vc = p.v_cache + (int64_t)kvh * p.head_stride;

    // queries: rows that do not exist read as zeros
    for (int i = tid; i < S::kRows * CH; i += S::kThreads) {
        const int r = i / CH, c = i % CH, at = q.first + r;
        const bool there = r < q.rows;
        const int token = there ? at / p.group : 0, head = kvh * p.group + (there ? at % p.group : 0);
        cp_async16(a_q + tile_off<D>(r, c), p.q + (int64_t)(q.row0 + token) * p.q_row_stride + head * D + c * 8, there);
    }

    auto offset_of = [&](int tile) -> int64_t {  // by thread: key tid of the tile
        const int key = lo + tile * BN + tid;
        return tid < BN && key < hi ? key_offset(p, table, key) : -1;
    };
    auto issue = [&](int tile) {
        const int64_t* offs = s_offs + (tile & 1) * BN;
        const uint32_t to = a_ring + (uint32_t)(tile % STAGES) * (2 * S::kTile);
#pragma unroll
        for (int i = 0; i < BN * CH / S::kThreads; ++i) {
            const int e = tid + i * S::kThreads, r = e / CH, c = e % CH;
            const int64_t o = offs[r];
            const bool there = o >= 0;
            const int64_t at = (there ? o : 0) + c * 8;
            cp_async16(to + tile_off<D>(r, c), kc + at, there);
            cp_async16(to + S::kTile + tile_off<D>(r, c), vc + at, there);
        }
    };
#pragma unroll 1
    for (int t = 0; t < STAGES - 1; ++t) {
        if (tid < BN)
            s_offs[(t & 1) * BN + tid] = offset_of(t);
        __syncthreads();
        if (t < tiles)
            issue(t);
        cp_async_commit();  // the first group holds the queries too
    }
    if (tid < BN)
        s_offs[((STAGES - 1) & 1) * BN + tid] = offset_of(STAGES - 1);

    // the thread's two rows: g and g + 8 of the warp's 16
    const int g = lane >> 2;
    int rlo[2], rhi[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = warp * 16 + g + 8 * i;
        visible_keys(p, q, (q.first + min(r, q.rows - 1)) / p.group, rlo[i], rhi[i]);
    }
    int full_lo, full_hi;  // keys that every row of the tile sees
    visible_keys(p, q, (q.first + q.rows - 1) / p.group, full_lo, unused);
    visible_keys(p, q, q.first / p.group, unused, full_hi);

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    // Queries stay in registers up to heads of 128; at 256 they would leave
    // none for the sums, and are read from shared memory for every tile.
    constexpr bool kKeepQ = D <= 128;
    uint32_t qf[kKeepQ ? D / 16 : 1][4];

#pragma unroll 1
    for (int t = 0; t < tiles; ++t) {
        cp_async_wait<STAGES - 2>();
        __syncthreads();
        if (t + STAGES - 1 < tiles)
            issue(t + STAGES - 1);
        cp_async_commit();
        const int64_t next_off = offset_of(t + STAGES);
        if (kKeepQ && t == 0) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                ldsm4(a_q + tile_off<D>(warp * 16 + (lane & 15), 2 * ks + (lane >> 4)), qf[kKeepQ ? ks : 0]);
        }
        const uint32_t ak = a_ring + (uint32_t)(t % STAGES) * (2 * S::kTile), av = ak + S::kTile;
        const int k0 = lo + t * BN;

        float s[BN / 8][4];
#pragma unroll
        for (int i = 0; i < BN / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[i][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t qr[4];
            if (kKeepQ) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    qr[e] = qf[kKeepQ ? ks : 0][e];
            } else {
                ldsm4(a_q + tile_off<D>(warp * 16 + (lane & 15), 2 * ks + (lane >> 4)), qr);
            }
#pragma unroll
            for (int nt = 0; nt < BN / 16; ++nt) {
                uint32_t b[4];  // keys 16 nt .. + 15, elements 16 ks .. + 15
                ldsm4(ak + tile_off<D>(nt * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)), b);
                mma16816(s[2 * nt], qr, b[0], b[1]);
                mma16816(s[2 * nt + 1], qr, b[2], b[3]);
            }
        }
        const bool clear = k0 >= full_lo && k0 + BN <= full_hi && k0 + BN <= hi;
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < BN / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = s[i][e] * p.scale_log2;
                if (!clear) {
                    const int key = k0 + i * 8 + (lane & 3) * 2 + (e & 1);
                    if (key < rlo[e >> 1] || key >= rhi[e >> 1] || key >= hi)
                        x = -INFINITY;
                }
                s[i][e] = x;
                top[e >> 1] = fmaxf(top[e >> 1], x);
            }
        float fix[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
            top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
            const float mn = fmaxf(m[i], top[i]);
            const float base = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: exp2(-inf) = 0 everywhere
            fix[i] = exp2f(m[i] - base);
            m[i] = mn;
            l[i] *= fix[i];
            top[i] = base;
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[i][e] *= fix[e >> 1];
#pragma unroll
        for (int nt = 0; nt < BN / 16; ++nt) {
            uint32_t a[4];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                float e4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    e4[e] = exp2f(s[2 * nt + hh][e] - top[e >> 1]);
                    l[e >> 1] += e4[e];
                }
                a[2 * hh] = pack2(e4[0], e4[1]);
                a[2 * hh + 1] = pack2(e4[2], e4[3]);
            }
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) {
                uint32_t b[4];  // keys 16 nt .. + 15, elements 16 dt .. + 15
                ldsm4_t(av + tile_off<D>(nt * 16 + (lane & 15), 2 * dt + (lane >> 4)), b);
                mma16816(o[2 * dt], a, b[0], b[1]);
                mma16816(o[2 * dt + 1], a, b[2], b[3]);
            }
        }
        if (tid < BN)
            s_offs[((t + STAGES) & 1) * BN + tid] = next_off;
    }
    cp_async_wait<0>();
    __syncthreads();  // the ring becomes the exchange buffer

    float* s_o = reinterpret_cast<float*>(s_ring);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        const int r = warp * 16 + g + 8 * i;
        float* row = s_o + r * S::kOStride + (lane & 3) * 2;
#pragma unroll
        for (int dt = 0; dt < D / 8; ++dt)
            *reinterpret_cast<float2*>(row + dt * 8) = make_float2(o[dt][2 * i], o[dt][2 * i + 1]);
        if ((lane & 3) == 0)
            s_ml[r] = make_float2(m[i], l[i]);
    }
    __syncthreads();
    // one warp per row: the output or the partial
    for (int r = warp; r < q.rows; r += S::kWarps) {
        const float mm = s_ml[r].x, ll = s_ml[r].y;
        const int at = q.first + r, token = at / p.group, head = kvh * p.group + at % p.group;
        const bool last = p.splits == 1;
        const float inv = last ? (ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll)) : 1.f;
        const int64_t part = partial_index(p, q.ordinal0 + token, head, split);
        uint16_t* out = p.out + (int64_t)(q.row0 + token) * p.out_row_stride + head * D;
        if (!last && tiles == 0) {
            if (lane == 0)
                p.part_ml[part] = make_float2(-INFINITY, 0.f);
            continue;
        }
        for (int c = lane * 4; c < D; c += 128) {
            const float4 v = *reinterpret_cast<const float4*>(s_o + r * S::kOStride + c);
            if (last)
                *reinterpret_cast<uint2*>(out + c) = make_uint2(pack2(v.x * inv, v.y * inv), pack2(v.z * inv, v.w * inv));
            else
                *reinterpret_cast<float4*>(p.part_o + part * D + c) = v;
        }
        if (lane == 0) {
            if (!last)
                p.part_ml[part] = make_float2(mm, ll);
            else if (p.lse != nullptr)
                p.lse[(int64_t)(q.row0 + token) * p.num_q_heads + head] = (mm + log2f(ll)) * kLn2;
        }
    }
}

// The splits of a (row, head) joined: one warp each.  Bound by reading the
// partials that hold keys (512 bytes each at heads of 128).
template <int D>
__global__ void __launch_bounds__(128) paged_join_kernel(const __grid_constant__ PagedParams p)
{
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const long long task = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int v = (int)(task / p.num_q_heads), head = (int)(task - (long long)v * p.num_q_heads);
    RowSlot s;
    if (!map_valid_row(v, p.pk.cu_seqlens, p.pk.cu_seqlens_padded, p.pk.num_seqs, p.pk.num_rows_padded, lane, s))
        return;
    int ordinal0, row0;
    const int n = chunk_rows(p, s.seq, ordinal0, row0);
    if (s.local >= n || (long long)n * p.group <= p.skip_rows)
        return;  // no block wrote its parts: skipped, or the narrow kernel's
    const int64_t part = partial_index(p, v, head, 0);
    float mm = -INFINITY;
    for (int i = lane; i < p.splits; i += 32)
        mm = fmaxf(mm, p.part_ml[part + i].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    const float base = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    constexpr int E = D / 32;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        acc[e] = 0.f;
    for (int i0 = 0; i0 < p.splits; i0 += 32) {
        const float2 ml = i0 + lane < p.splits ? p.part_ml[part + i0 + lane] : make_float2(-INFINITY, 0.f);
        const float w = exp2f(ml.x - base);
        ll += w * ml.y;
        unsigned live = __ballot_sync(0xffffffffu, ml.x != -INFINITY);
        while (live != 0u) {
            const int i = __ffs(live) - 1;
            live &= live - 1;
            const float f = __shfl_sync(0xffffffffu, w, i);
            const float* from = p.part_o + (part + i0 + i) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 x = *reinterpret_cast<const float2*>(from + e);
                acc[e] = fmaf(f, x.x, acc[e]);
                acc[e + 1] = fmaf(f, x.y, acc[e + 1]);
            }
        }
    }
    ll = group_sum<32>(ll);
    const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);
    uint16_t* out = p.out + (int64_t)s.row * p.out_row_stride + head * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(out + e) = pack2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[(int64_t)s.row * p.num_q_heads + head] = (mm + log2f(ll)) * kLn2;
}

template <int D>
cudaError_t launch_wide(const PagedParams& p, int tiles, cudaStream_t stream)
{
    using S = Shape<D>;
    const cudaError_t e = cudaFuncSetAttribute(paged_attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess)
        return e;
    return launch_kernel(paged_attention_kernel<D>, dim3((unsigned)tiles, (unsigned)p.num_kv_heads, (unsigned)p.splits),
                         S::kThreads, S::kSmem, stream, p);
}

template <int D>
cudaError_t launch_d(const PagedParams& p, const PagedPlan& plan, cudaStream_t stream)
{
    const cudaError_t e = plan.kind == kPagedTc ? launch_paged_attention_tc(p, plan.tiles, D, stream)
                                                : launch_wide<D>(p, plan.tiles, stream);
    if (e != cudaSuccess || p.splits == 1)
        return e;
    const long long warps = (long long)p.pk.num_rows_padded * p.num_q_heads;
    return launch_kernel(paged_join_kernel<D>, dim3((unsigned)((warps + 3) / 4)), 128, 0, stream, p);
}

}  // namespace

// The kernel, and the cut of the key axis, for a call's sizes.
bool paged_plan(int64_t rows, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int64_t max_chunk,
                int64_t max_kv_len, int64_t window, bool regular, PagedPlan& plan)
{
    const int64_t group = num_q_heads / num_kv_heads;
    const int64_t chunk = max_chunk > 0 && max_chunk < rows ? max_chunk : rows;
    plan = PagedPlan{};
    const int64_t narrow = paged_narrow_slots(head_dim);
    if (chunk * group <= kNarrowRows) {
        plan.kind = kPagedNarrow;
        plan.splits = 1;
        plan.part_rows = narrow;
        plan.bytes = plan.most_bytes = narrow * (head_dim * 4 + 8);
        return true;
    }
    // Next tokens beside chunks would each take a whole block per key head of
    // the chunk kernel, one row of 256: they go to the narrow kernel first (a
    // chunk of 2,000 rows and 31 next tokens over 3,000 to 27,000 keys: 664 us
    // -> 532).  Where a batch turns out to hold none its launches cost 5 us, so
    // not where the rows given leave no sequence that short.
    plan.mixed = num_seqs > 1 && rows <= (num_seqs - 1) * chunk + kNarrowRows;
    plan.kind = regular ? kPagedTc : kPagedWide;
    plan.tile_rows = plan.kind == kPagedWide ? 64 : (head_dim == 256 ? 128 : 256);
    // ceil over each sequence adds at most one tile per sequence
    const int64_t tiles = rows * group / plan.tile_rows + (num_seqs < rows ? num_seqs : rows);
    if (tiles > INT32_MAX)
        return false;
    plan.tiles = (int)tiles;
    const int64_t part = rows * num_q_heads * (head_dim * 4 + 8);  // bytes of one split's results
    int64_t keys = max_kv_len;
    if (window > 0 && window + plan.tile_rows < keys)
        keys = window + plan.tile_rows;
    int64_t splits;
    if (plan.kind == kPagedTc) {
        // Tiles the batch is expected to have: chunks that are all as long as the
        // longest, or ragged ones whose last tiles are half full on the average.
        const int64_t longest = num_seqs * ((chunk * group + plan.tile_rows - 1) / plan.tile_rows);
        int64_t expected = rows * group / plan.tile_rows + (num_seqs + 1) / 2;
        expected = expected > num_seqs ? expected : num_seqs;
        if (expected > longest || num_seqs * chunk <= rows)
            expected = longest;
        splits = tc_splits(expected * num_kv_heads, keys, part);
    } else {
        // several short blocks per SM: enough of them for the GPU several times
        // over, no run shorter than 128 keys
        const int64_t full = rows * group / plan.tile_rows;
        const int64_t blocks = (full > num_seqs ? full : num_seqs) * num_kv_heads;
        splits = (148 * 8 + blocks - 1) / blocks;
        const int64_t most = (keys + 127) / 128;
        splits = splits < most ? splits : most;
    }
    if (splits > 128)
        splits = 128;
    if (splits < 1)
        splits = 1;
    // splits only falls below its value here, and that grows with the keys:
    // what one workspace must hold for every window and shorter length
    const int64_t narrow_part = plan.mixed ? narrow * (head_dim * 4 + 8) : 0;
    plan.most_bytes = narrow_part + (splits == 1 ? 0 : part * splits);
    int64_t run = (keys + splits - 1) / splits;
    run = (run + 127) / 128 * 128;
    if (run < 128)
        run = 128;
    splits = (keys + run - 1) / run;
    plan.splits = (int)(splits < 1 ? 1 : splits);
    plan.split_keys = (int)(run > INT32_MAX ? INT32_MAX : run);
    plan.part_rows = (plan.mixed ? narrow : 0) + (plan.splits == 1 ? 0 : rows * num_q_heads * plan.splits);
    plan.bytes = narrow_part + (plan.splits == 1 ? 0 : part * plan.splits);
    return true;
}

cudaError_t launch_paged_attention(const PagedParams& p, const PagedPlan& plan, int head_dim, cudaStream_t stream)
{
    PagedParams few = p;
    few.narrow_rows = plan.kind == kPagedNarrow ? INT32_MAX : kNarrowRows;
    if (plan.kind == kPagedNarrow || plan.mixed) {
        const cudaError_t e = launch_paged_attention_narrow(few, plan.mixed, head_dim, stream);
        if (e != cudaSuccess || plan.kind == kPagedNarrow)
            return e;
    }
    PagedParams many = p;
    many.skip_rows = plan.mixed ? kNarrowRows : 0;
    if (plan.mixed) {
        const int64_t slots = paged_narrow_slots(head_dim);
        many.part_o += slots * head_dim;
        many.part_ml += slots;
    }
    switch (head_dim) {
    case 64: return launch_d<64>(many, plan, stream);
    case 128: return launch_d<128>(many, plan, stream);
    case 256: return launch_d<256>(many, plan, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace dit
