// paged_attention_narrow.cu -- attention of next tokens (and of chunks of a
// few rows) over a paged cache.
//
// The mathematics is paged_attention.cu's.  A call of this kind reads every
// cached key and value once and computes little with each: it is bound by
// HBM, as long as every SM reads all the time.  Requests' caches differ
// in length by orders of magnitude, so the key axis is not cut per request:
// the key tiles of all (sequence, 16-row tile, key head) triples
// are numbered through, and each block takes an equal run of that list,
// whatever it crosses.  The lengths are read on the device, so a captured
// call keeps its balance as caches grow.  A triple that lies within one run is
// written at once; one that several runs share leaves a part per run (its
// unnormalised sums, maximum and sum of exponentials), and a second kernel
// joins them in the order of the keys: results are bitwise reproducible.  A
// run has at most one part that began before it and one that goes on behind
// it, so two slots per block are the whole workspace.
//
// A block's warps share 16 rows and part each tile's keys; the next tile is
// under way by 16-byte asynchronous copies, which take any page size and
// stride and write zeros for keys that are not there.  (TMA boxes took 185
// against 153 us for heads of 64, whose rows are 128 bytes in a slot-major
// cache, and 249 against 239 for 128.)
#include "paged_mma.cuh"

namespace dit {
namespace {

constexpr int kNRows = 16;

template <int D>
struct NShape {
    // A stage is 32 KB of keys and values (D 64, 128 and 256: 128, 64 and 32
    // keys), 16 keys per warp and more where a row is short; two stages and
    // three blocks per SM (48 ragged requests, 40 q and 8 key heads of 128: 234 us
    // among other passes, 92 % of the measured copy rate; 239 with three stages and
    // two blocks, 415 with four and one).
    static constexpr int kWarps = D == 256 ? 2 : 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kKeys = 8192 / D;
    static constexpr int kStages = 2;
    static constexpr int kPerSm = 3;  // blocks
    static constexpr int kBlocks = 148 * kPerSm;
    static constexpr int kTile = kKeys * D * 2;
    static constexpr int kQ = kNRows * D * 2;
    static constexpr int kRing = 2 * kStages * kTile;
    static constexpr int kOStride = D + 4;
    static constexpr int kO = kWarps * kNRows * kOStride * 4;
    static constexpr int kMain = kRing > kO ? kRing : kO;
    static constexpr int kOffs = 2 * kKeys * 8;
    static constexpr int kSmem = kQ + kMain + kOffs + kWarps * kNRows * 8;
};

// A sequence in the list: its tiles of 16 rows and, for each of them and each
// key head, the same number of key tiles (those its chunk's rows see together;
// one where they see none, so that their rows are written).
struct Listed {
    int n, row0, ordinal0, kv_len, kv_end;
    int q_tiles, lo, k_tiles;
    __device__ __forceinline__ long long count(const PagedParams& p) const
    {
        return (long long)q_tiles * p.num_kv_heads * k_tiles;
    }
};

template <int D>
__device__ __forceinline__ Listed list_seq(const PagedParams& p, int b)
{
    Listed s{};
    if (b >= p.pk.num_seqs)
        return s;
    s.kv_len = max(__ldg(p.kv_lens + b), 0);
    s.n = chunk_rows(p, b, s.ordinal0, s.row0);
    if (s.n == 0 || (long long)s.n * p.group > p.narrow_rows)
        return Listed{};
    s.kv_end = (int)min((long long)s.kv_len, (long long)p.max_pages * p.page_size);
    s.q_tiles = (int)(((long long)s.n * p.group + kNRows - 1) / kNRows);
    QueryTile q{};
    q.n = s.n;
    q.kv_len = s.kv_len;
    q.kv_end = s.kv_end;
    int hi, unused;
    visible_keys(p, q, 0, s.lo, unused);
    visible_keys(p, q, s.n - 1, unused, hi);
    s.k_tiles = hi > s.lo ? (hi - s.lo + NShape<D>::kKeys - 1) / NShape<D>::kKeys : 1;
    return s;
}

__device__ __forceinline__ long long shfl_ll(long long v, int src)
{
    return (long long)__shfl_sync(0xffffffffu, (unsigned long long)v, src);
}

// Warp-collective: the list's entries before sequence `until` (all of it for
// num_seqs).
template <int D>
__device__ __forceinline__ long long listed_before(const PagedParams& p, int until, int lane)
{
    long long sum = 0;
    for (int base = 0; base < until; base += kWarp)
        if (base + lane < until)
            sum += list_seq<D>(p, base + lane).count(p);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        sum += (long long)__shfl_xor_sync(0xffffffffu, (unsigned long long)sum, o);
    return sum;
}

// Warp-collective: the sequence that holds entry `at` (0 <= at < the list's
// length), and the entries before it.
template <int D>
__device__ __forceinline__ int find_listed(const PagedParams& p, long long at, int lane, long long& before)
{
    before = 0;
    for (int base = 0; base < p.pk.num_seqs; base += kWarp) {
        const long long c = list_seq<D>(p, base + lane).count(p);
        long long sum = c;
#pragma unroll
        for (int o = 1; o < kWarp; o <<= 1) {
            const long long up = (long long)__shfl_up_sync(0xffffffffu, (unsigned long long)sum, o);
            if (lane >= o)
                sum += up;
        }
        const unsigned m = __ballot_sync(0xffffffffu, at < before + sum);
        if (m != 0u) {
            const int l = __ffs(m) - 1;
            before += shfl_ll(sum - c, l);
            return base + l;
        }
        before += shfl_ll(sum, kWarp - 1);
    }
    return -1;
}

// Quotient of counts that nearly always fit 32 bits.
__device__ __forceinline__ long long div_count(long long a, long long b)
{
    return ((unsigned long long)(a | b) >> 31) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

__device__ __forceinline__ Listed shfl_listed(const Listed& s, int src)
{
    Listed r;
    r.n = __shfl_sync(0xffffffffu, s.n, src);
    r.row0 = __shfl_sync(0xffffffffu, s.row0, src);
    r.ordinal0 = __shfl_sync(0xffffffffu, s.ordinal0, src);
    r.kv_len = __shfl_sync(0xffffffffu, s.kv_len, src);
    r.kv_end = __shfl_sync(0xffffffffu, s.kv_end, src);
    r.q_tiles = __shfl_sync(0xffffffffu, s.q_tiles, src);
    r.lo = __shfl_sync(0xffffffffu, s.lo, src);
    r.k_tiles = __shfl_sync(0xffffffffu, s.k_tiles, src);
    return r;
}

// The whole list of a batch of up to 32 sequences, one per lane, read in one
// round: a few next tokens are bound by such rounds (the one-token call 16.5
// us with three of them before its first key, 15.8 with one).
struct WholeList {
    Listed mine;
    long long before;  // entries before the lane's sequence
    long long total;
};
template <int D>
__device__ __forceinline__ WholeList whole_list(const PagedParams& p, int lane)
{
    WholeList w;
    w.mine = list_seq<D>(p, lane);
    const long long c = w.mine.count(p);
    long long sum = c;
#pragma unroll
    for (int o = 1; o < kWarp; o <<= 1) {
        const long long up = (long long)__shfl_up_sync(0xffffffffu, (unsigned long long)sum, o);
        if (lane >= o)
            sum += up;
    }
    w.before = sum - c;
    w.total = shfl_ll(sum, kWarp - 1);
    return w;
}

// Entries per block: an equal share, and two tiles at least.
template <int D>
__device__ __forceinline__ long long run_length(long long total)
{
    const long long share = div_count(total + NShape<D>::kBlocks - 1, NShape<D>::kBlocks);
    return share > 2 ? share : 2;
}

template <int D>
__global__ void __launch_bounds__(NShape<D>::kThreads) paged_narrow_kernel(const __grid_constant__ PagedParams p)
{
    using S = NShape<D>;
    constexpr int kKeys = S::kKeys, kNWarps = S::kWarps, kNThreads = S::kThreads;
    constexpr int NK = kKeys / kNWarps, CH = D / 8, ST = S::kStages;
    extern __shared__ __align__(128) unsigned char smem[];
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool few = p.pk.num_seqs <= kWarp;
    WholeList w{};
    if (few)
        w = whole_list<D>(p, lane);
    const long long total = few ? w.total : listed_before<D>(p, p.pk.num_seqs, lane);
    const long long run = run_length<D>(total);
    const long long begin = blockIdx.x * run, end = min(begin + run, total);
    if (begin >= end)
        return;
    unsigned char* s_ring = smem + S::kQ;
    int64_t* s_offs = reinterpret_cast<int64_t*>(smem + S::kQ + S::kMain);
    float2* s_ml = reinterpret_cast<float2*>(smem + S::kQ + S::kMain + S::kOffs);
    const uint32_t a_q = (uint32_t)__cvta_generic_to_shared(smem);
    const uint32_t a_ring = a_q + S::kQ;

    long long at = begin, before;
    int seq;
    Listed ls;
    if (few) {
        seq = __ffs(__ballot_sync(0xffffffffu, at < w.before + w.mine.count(p))) - 1;
        if (seq < 0)
            return;
        before = shfl_ll(w.before, seq);
        ls = shfl_listed(w.mine, seq);
    } else {
        seq = find_listed<D>(p, at, lane, before);
        if (seq < 0)
            return;
        ls = list_seq<D>(p, seq);
    }
    while (at < end) {
        while (at >= before + ls.count(p)) {  // the next sequence that has entries
            before += ls.count(p);
            if (++seq >= p.pk.num_seqs)
                return;
            ls = list_seq<D>(p, seq);
        }
        const long long triple = div_count(at - before, ls.k_tiles);
        const int t0 = (int)(at - before - triple * ls.k_tiles);
        const int t1 = (int)min((long long)ls.k_tiles, t0 + (end - at));
        const long long q_tile = div_count(triple, p.num_kv_heads);
        const int kvh = (int)(triple - q_tile * p.num_kv_heads);
        QueryTile q;
        q.seq = seq;
        q.first = (int)q_tile * kNRows;
        q.rows = min(kNRows, ls.n * p.group - q.first);
        q.n = ls.n;
        q.row0 = ls.row0;
        q.kv_len = ls.kv_len;
        q.kv_end = ls.kv_end;
        int tile_hi, unused;
        visible_keys(p, q, (q.first + q.rows - 1) / p.group, unused, tile_hi);
        const int lo = ls.lo + t0 * kKeys;
        const int hi = t1 == ls.k_tiles ? tile_hi : min(tile_hi, ls.lo + t1 * kKeys);
        const int tiles = hi > lo ? (hi - lo + kKeys - 1) / kKeys : 0;
        const int32_t* table = p.block_table + (int64_t)seq * p.table_stride;
        const uint16_t* kc = p.k_cache + (int64_t)kvh * p.head_stride;
        const uint16_t* vc = p.v_cache + (int64_t)kvh * p.head_stride;

        // queries: rows that do not exist read as zeros
        for (int i = tid; i < kNRows * CH; i += kNThreads) {
            const int r = i / CH, c = i % CH, row = q.first + r;
            const bool there = r < q.rows;
            const int token = there ? row / p.group : 0, head = kvh * p.group + (there ? row % p.group : 0);
            cp_async16(a_q + tile_off<D>(r, c), p.q + (int64_t)(q.row0 + token) * p.q_row_stride + head * D + c * 8, there);
        }
        auto offset_of = [&](int tile) -> int64_t {  // by thread: key tid of the tile
            const int key = lo + tile * kKeys + tid;
            return tid < kKeys && key < hi ? key_offset(p, table, key) : -1;
        };
        auto issue = [&](int tile) {
            const int64_t* offs = s_offs + (tile & 1) * kKeys;
            const uint32_t to = a_ring + (uint32_t)(tile % ST) * (2 * S::kTile);
#pragma unroll
            for (int i = 0; i < kKeys * CH / kNThreads; ++i) {
                const int e = tid + i * kNThreads, r = e / CH, c = e % CH;
                const int64_t o = offs[r];
                const bool there = o >= 0;
                const int64_t from = (there ? o : 0) + c * 8;
                cp_async16(to + tile_off<D>(r, c), kc + from, there);
                cp_async16(to + S::kTile + tile_off<D>(r, c), vc + from, there);
            }
        };
#pragma unroll 1
        for (int t = 0; t < ST - 1; ++t) {
            if (tid < kKeys)
                s_offs[(t & 1) * kKeys + tid] = offset_of(t);
            __syncthreads();
            if (t < tiles)
                issue(t);
            cp_async_commit();  // the first group holds the queries too
        }
        if (tid < kKeys)
            s_offs[((ST - 1) & 1) * kKeys + tid] = offset_of(ST - 1);

        const int g = lane >> 2;  // the thread's rows: g and g + 8
        int rlo[2], rhi[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            visible_keys(p, q, (q.first + min(g + 8 * i, q.rows - 1)) / p.group, rlo[i], rhi[i]);
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
        // Queries stay in registers up to heads of 128; at 256 they are read
        // from shared memory for every tile.
        constexpr bool kKeepQ = D <= 128;
        uint32_t qf[kKeepQ ? D / 16 : 1][4];

#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
            cp_async_wait<ST - 2>();
            __syncthreads();
            if (t + ST - 1 < tiles)
                issue(t + ST - 1);
            cp_async_commit();
            const int64_t next_off = offset_of(t + ST);
            if (kKeepQ && t == 0) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    ldsm4(a_q + tile_off<D>(lane & 15, 2 * ks + (lane >> 4)), qf[kKeepQ ? ks : 0]);
            }
            const uint32_t ak = a_ring + (uint32_t)(t % ST) * (2 * S::kTile), av = ak + S::kTile;
            const int k0 = lo + t * kKeys + warp * NK;  // the warp's first key
            float s[NK / 8][4];
#pragma unroll
            for (int i = 0; i < NK / 8; ++i)
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
                    ldsm4(a_q + tile_off<D>(lane & 15, 2 * ks + (lane >> 4)), qr);
                }
#pragma unroll
                for (int nt = 0; nt < NK / 16; ++nt) {
                    uint32_t b[4];  // 16 of the warp's keys, elements 16 ks .. + 15
                    ldsm4(ak + tile_off<D>(warp * NK + nt * 16 + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1)), b);
                    mma16816(s[2 * nt], qr, b[0], b[1]);
                    mma16816(s[2 * nt + 1], qr, b[2], b[3]);
                }
            }
            const bool clear = k0 >= full_lo && k0 + NK <= full_hi && k0 + NK <= hi;
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < NK / 8; ++i)
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
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
            }
            if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
                float fix[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float mn = fmaxf(m[i], top[i]);
                    fix[i] = mn == m[i] ? 1.f : exp2f(m[i] - mn);  // 0 for the first key seen
                    m[i] = mn;
                    l[i] *= fix[i];
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[i][e] *= fix[e >> 1];
            }
            // nothing seen yet: exp2(-inf - 0) = 0 everywhere
            const float base[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
            for (int nt = 0; nt < NK / 16; ++nt) {
                uint32_t a[4];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    float e4[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        e4[e] = exp2f(s[2 * nt + hh][e] - base[e >> 1]);
                        l[e >> 1] += e4[e];
                    }
                    a[2 * hh] = pack2(e4[0], e4[1]);
                    a[2 * hh + 1] = pack2(e4[2], e4[3]);
                }
#pragma unroll
                for (int dt = 0; dt < D / 16; ++dt) {
                    uint32_t b[4];  // 16 of the warp's keys, elements 16 dt .. + 15
                    ldsm4_t(av + tile_off<D>(warp * NK + nt * 16 + (lane & 15), 2 * dt + (lane >> 4)), b);
                    mma16816(o[2 * dt], a, b[0], b[1]);
                    mma16816(o[2 * dt + 1], a, b[2], b[3]);
                }
            }
            if (tid < kKeys)
                s_offs[((t + ST) & 1) * kKeys + tid] = next_off;
        }
        cp_async_wait<0>();
        __syncthreads();  // the ring becomes the exchange buffer

        float* s_o = reinterpret_cast<float*>(s_ring);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            const int r = g + 8 * i;
            float* row = s_o + (warp * kNRows + r) * S::kOStride + (lane & 3) * 2;
#pragma unroll
            for (int dt = 0; dt < D / 8; ++dt)
                *reinterpret_cast<float2*>(row + dt * 8) = make_float2(o[dt][2 * i], o[dt][2 * i + 1]);
            if ((lane & 3) == 0)
                s_ml[warp * kNRows + r] = make_float2(m[i], l[i]);
        }
        __syncthreads();
        // one warp per row: the four parts joined, then the output or the run's part
        const bool whole = t0 == 0 && t1 == ls.k_tiles;
        const int slot = 2 * blockIdx.x + (t0 > 0 ? 0 : 1);
        for (int r = warp; r < q.rows; r += kNWarps) {
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < kNWarps; ++w)
                mm = fmaxf(mm, s_ml[w * kNRows + r].x);
            const float base = mm == -INFINITY ? 0.f : mm;
            float ll = 0.f, f[kNWarps];
#pragma unroll
            for (int w = 0; w < kNWarps; ++w) {
                const float2 ml = s_ml[w * kNRows + r];
                f[w] = exp2f(ml.x - base);
                ll += f[w] * ml.y;
            }
            const int row = q.first + r, token = row / p.group, head = kvh * p.group + row % p.group;
            const float inv = whole ? (ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll)) : 1.f;
            uint16_t* out = p.out + (int64_t)(q.row0 + token) * p.out_row_stride + head * D;
            float* part = p.part_o + ((int64_t)slot * kNRows + r) * D;
            for (int c = lane * 4; c < D; c += 128) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kNWarps; ++w) {
                    const float4 x = *reinterpret_cast<const float4*>(s_o + (w * kNRows + r) * S::kOStride + c);
                    v.x = fmaf(f[w], x.x, v.x);
                    v.y = fmaf(f[w], x.y, v.y);
                    v.z = fmaf(f[w], x.z, v.z);
                    v.w = fmaf(f[w], x.w, v.w);
                }
                if (whole)
                    *reinterpret_cast<uint2*>(out + c) = make_uint2(pack2(v.x * inv, v.y * inv), pack2(v.z * inv, v.w * inv));
                else
                    *reinterpret_cast<float4*>(part + c) = v;
            }
            if (lane == 0) {
                if (!whole)
                    p.part_ml[(int64_t)slot * kNRows + r] = make_float2(mm, ll);
                else if (p.lse != nullptr)
                    p.lse[(int64_t)(q.row0 + token) * p.num_q_heads + head] = (mm + log2f(ll)) * kLn2;
            }
        }
        __syncthreads();  // the exchange buffer becomes the ring
        at += t1 - t0;
    }
}

// The parts of the triples that several runs share, joined: W warps per (row,
// head) take the parts in turn; rows of whole triples are done.  W is 4 where
// there are few rows (a single sequence's keys lie in hundreds of parts: one
// token over 21,065 keys of 2 heads of 256 took 87 us with one warp per row, 44
// with four), and 1 where there are many, each with a few parts (48 requests of
// 40 heads, back to back: 234 us against 292).
template <int D, int W>
__global__ void __launch_bounds__(128) paged_narrow_join_kernel(const __grid_constant__ PagedParams p, int tokens)
{
    __shared__ float s_acc[W][W > 1 ? D : 1];
    __shared__ float s_l[W];
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % W;
    const long long task = (long long)blockIdx.x * (4 / W) + (threadIdx.x >> 5) / W;
    const int v = (int)(task / p.num_q_heads), head = (int)(task - (long long)v * p.num_q_heads);
    // token `local` of sequence `seq`: of a mixed batch token v % tokens of
    // sequence v / tokens, else valid row v
    int seq = tokens > 0 ? v / tokens : -1, local = tokens > 0 ? v - seq * tokens : 0;
    if (seq >= p.pk.num_seqs)
        return;
    Listed ls;
    long long before, total;
    if (p.pk.num_seqs <= kWarp) {
        const WholeList w = whole_list<D>(p, lane);
        if (tokens == 0) {
            seq = __ffs(__ballot_sync(0xffffffffu, v >= w.mine.ordinal0 && v < w.mine.ordinal0 + w.mine.n)) - 1;
            if (seq < 0)
                return;
            local = v - __shfl_sync(0xffffffffu, w.mine.ordinal0, seq);
        }
        ls = shfl_listed(w.mine, seq);
        before = shfl_ll(w.before, seq);
        total = w.total;
    } else {
        if (tokens == 0) {
            RowSlot s;
            if (!map_valid_row(v, p.pk.cu_seqlens, p.pk.cu_seqlens_padded, p.pk.num_seqs, p.pk.num_rows_padded, lane, s))
                return;
            seq = s.seq;
            local = s.local;
        }
        ls = list_seq<D>(p, seq);
        before = listed_before<D>(p, seq, lane);
        total = listed_before<D>(p, p.pk.num_seqs, lane);
    }
    if (local >= ls.n)
        return;
    const long long run = run_length<D>(total);
    const int row = local * p.group + head % p.group, r = row % kNRows;
    const long long first = before + ((long long)(row / kNRows) * p.num_kv_heads + head / p.group) * ls.k_tiles;
    const int b0 = (int)div_count(first, run), b1 = (int)div_count(first + ls.k_tiles - 1, run);
    if (b0 == b1)
        return;
    auto part_of = [&](int b) { return (int64_t)(2 * b + (first < b * run ? 0 : 1)) * kNRows + r; };
    float mm = -INFINITY;
    for (int b = b0 + lane; b <= b1; b += 32)
        mm = fmaxf(mm, p.part_ml[part_of(b)].x);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    const float base = mm == -INFINITY ? 0.f : mm;
    constexpr int E = D / 32;
    float ll = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        acc[e] = 0.f;
    for (int c0 = b0 + warp; c0 <= b1; c0 += 32 * W) {  // the warp's parts: every W-th
        const int mine = c0 + lane * W;
        const float2 ml = mine <= b1 ? p.part_ml[part_of(mine)] : make_float2(-INFINITY, 0.f);
        const float w = exp2f(ml.x - base);
        ll += w * ml.y;
        const int count = min(32, (b1 - c0) / W + 1);
#pragma unroll 8
        for (int i = 0; i < count; ++i) {
            const float f = __shfl_sync(0xffffffffu, w, i);
            const float* from = p.part_o + part_of(c0 + i * W) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 x = *reinterpret_cast<const float2*>(from + e);
                acc[e] = fmaf(f, x.x, acc[e]);
                acc[e + 1] = fmaf(f, x.y, acc[e + 1]);
            }
        }
    }
    ll = group_sum<32>(ll);
    const int64_t out_row = ls.row0 + local;
    uint16_t* out = p.out + out_row * p.out_row_stride + head * D;
    if constexpr (W > 1) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            s_acc[warp][lane * E + e] = acc[e];
        if (lane == 0)
            s_l[warp] = ll;
        __syncthreads();  // W is the block's 4 warps: every one is here
        if (warp != 0)
            return;
        ll = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            ll += s_l[w];
#pragma unroll
            for (int e = 0; e < E; ++e)
                acc[e] += s_acc[w][lane * E + e];
        }
    }
    const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(out + lane * E + e) = pack2(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0 && p.lse != nullptr)
        p.lse[out_row * p.num_q_heads + head] = (mm + log2f(ll)) * kLn2;
}

template <int D>
cudaError_t launch_n(const PagedParams& p, bool mixed, cudaStream_t stream)
{
    using S = NShape<D>;
    cudaError_t e = cudaFuncSetAttribute(paged_narrow_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e == cudaSuccess)
        e = launch_kernel(paged_narrow_kernel<D>, dim3(S::kBlocks), S::kThreads, S::kSmem, stream, p);
    if (e != cudaSuccess)
        return e;
    const int tokens = mixed ? (kNarrowRows + p.group - 1) / p.group : 0;
    const long long rows = (mixed ? (long long)p.pk.num_seqs * tokens : p.pk.num_rows_padded) * p.num_q_heads;
    if (rows <= 4 * 148)
        return launch_kernel(paged_narrow_join_kernel<D, 4>, dim3((unsigned)rows), 128, 0, stream, p, tokens);
    return launch_kernel(paged_narrow_join_kernel<D, 1>, dim3((unsigned)((rows + 3) / 4)), 128, 0, stream, p, tokens);
}

}  // namespace

int64_t paged_narrow_slots(int head_dim)
{
    return 2 * kNRows * (int64_t)(head_dim == 64 ? NShape<64>::kBlocks : (head_dim == 128 ? NShape<128>::kBlocks
                                                                                         : NShape<256>::kBlocks));
}

cudaError_t launch_paged_attention_narrow(const PagedParams& p, bool mixed, int head_dim, cudaStream_t stream)
{
    switch (head_dim) {
    case 64: return launch_n<64>(p, mixed, stream);
    case 128: return launch_n<128>(p, mixed, stream);
    case 256: return launch_n<256>(p, mixed, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace dit
