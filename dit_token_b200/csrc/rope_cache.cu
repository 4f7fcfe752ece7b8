// rope_cache.cu -- rotary positions of q and k from a table of frequencies
// (scaled for long contexts, over the first R elements of a head), optionally
// behind the per-head RMSNorm, and the same on the way into a paged cache:
// k rotated into its pages, v copied beside it.
//
//   y = x * rsqrt(mean(x^2) + eps) * w          (or x, without weights)
//   (o_a, o_b) = g (y_a c - y_b s, y_a s + y_b c),  c, s = cos, sin(p f_j)
// for the pairs j < R / 2: elements (2j, 2j + 1) interleaved, (j, j + R/2)
// half-split; elements R .. D - 1 keep y.
//
// Bound: HBM, 4 bytes per element (read once, written once).  One warp per
// row and run of heads: D / 8 lanes hold a head, 8 elements per lane, so a
// lane needs the angles of the same 4 pairs for every head and forms them once
// (the fp64 product p f_j, reduced, then the hardware sine and cosine).  The
// heads go in batches of 4 steps, a batch's loads in flight while the one
// before is computed.  A batch of few rows (next tokens) cannot fill the
// GPU with whole rows: its rows' batches are spread over up to as many warps,
// which repeats the angles and shortens the chain of loads (launch_rc).  q, k
// and v are batched apart, so a batch has one weight vector and one
// destination.  Measured among other passes (behind an L2 that holds nothing to
// write back): 61,888 rows of 16 + 16 heads of 128 in 168 us, 6.0 TB/s (161),
// four ragged prompts of 53,619 rows of 40 + 8 heads in 239 us, 5.5 (225), 20,819
// rows of 40 + 8 + 8 heads into pages of 16 in 103 us, 5.8 (97.5).
#include "common.cuh"
#include "launch.h"
#include "rope.cuh"

#include <type_traits>

namespace dit {
namespace {

constexpr int kRcWarps = 4;  // warps per CTA

// Offset of the lane's first or second quad of a head's elements.  A half-
// split lane whose pairs turn holds 4 li .. and R/2 + 4 li ..; every other
// lane holds 8 consecutive elements, which are its four interleaved pairs
// (with R a multiple of 8 the lanes li < R / 8 turn and the rest pass).
template <int MODE>
__device__ __forceinline__ int quad_off(int li, int part, bool turns, int half)
{
    if (MODE == kRopeHalf && turns)
        return part * half + 4 * li;
    return 8 * li + 4 * part;
}

template <int MODE>
__device__ __forceinline__ uint4 load_quads(const uint16_t* head, int o0, int o1)
{
    if (MODE == kRopeHalf) {
        const uint2 a = __ldcs(reinterpret_cast<const uint2*>(head + o0));
        const uint2 b = __ldcs(reinterpret_cast<const uint2*>(head + o1));
        return make_uint4(a.x, a.y, b.x, b.y);
    }
    return ld_stream(head + o0);
}

// Cache pages are read again soon by the attention over them, so they keep
// the default policy; rows of q and k go out evict-first like the other
// operators' activations.
template <int MODE>
__device__ __forceinline__ void store_quads(uint16_t* head, int o0, int o1, uint4 v, bool keep)
{
    if (MODE == kRopeHalf) {
        uint2* a = reinterpret_cast<uint2*>(head + o0);
        uint2* b = reinterpret_cast<uint2*>(head + o1);
        if (keep) {
            *a = make_uint2(v.x, v.y);
            *b = make_uint2(v.z, v.w);
        } else {
            __stcs(a, make_uint2(v.x, v.y));
            __stcs(b, make_uint2(v.z, v.w));
        }
        return;
    }
    if (keep)
        *reinterpret_cast<uint4*>(head + o0) = v;
    else
        st_stream(head + o0, v);
}

// What a pair's elements are multiplied by: with weights these are folded into
// the rotation, (o_a, o_b) = r (x_a c0 + x_b c1, x_a c2 + x_b c3), so that a
// normed and turned pair costs two products, two fused ones and r.  A lane that
// passes has c0 = w_a, c3 = w_b and zeros.  q's and k's coefficients are both
// kept: registers decide how many warps hide the loads, and with a head's stride
// known (D) for all but the cache's writes they fit in 96.  The long video, single
// calls behind a clean L2: 161 us; weights applied on their own 186, one kernel
// for both destinations (126 registers) 197, one set folded again between q and k
// 174, without weights (one set) 154.
struct PairCoef {
    float c0[4], c1[4], c2[4], c3[4];
};

template <int MODE>
__device__ __forceinline__ void pair_regs(int e, int& a, int& z)
{
    a = MODE == kRopeHalf ? e : 2 * e;
    z = MODE == kRopeHalf ? 4 + e : 2 * e + 1;
}

template <int MODE, bool NORM>
__device__ __forceinline__ void fold(PairCoef& pc, const float (&c)[4], const float (&s)[4], bool turns,
                                     const uint16_t* w, int o0, int o1)
{
    float wf[8];
    if (NORM) {
        const uint2 wa = __ldg(reinterpret_cast<const uint2*>(w + o0));
        const uint2 wb = __ldg(reinterpret_cast<const uint2*>(w + o1));
        unpack8(make_uint4(wa.x, wa.y, wb.x, wb.y), wf);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        int a, z;
        pair_regs<MODE>(e, a, z);
        const float wa = NORM ? wf[a] : 1.f, wz = NORM ? wf[z] : 1.f;
        pc.c0[e] = wa * c[e];
        pc.c1[e] = NORM && !turns ? 0.f : -wz * s[e];
        pc.c2[e] = NORM && !turns ? 0.f : wa * s[e];
        pc.c3[e] = wz * c[e];
    }
}

template <int D, int MODE, bool NORM, int U>
__device__ __forceinline__ void turn_batch(uint16_t* to, int64_t step, int heads, int h0, int o0, int o1, bool keep,
                                           bool turns, float eps, const PairCoef& pc, const uint4 (&x)[U])
{
    constexpr int LPH = D / 8, HPW = kWarp / LPH;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int h = h0 + u * HPW;
        float r = 1.f;
        if (NORM) {
            const uint32_t wd[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            f32x2 ss2 = f2_make(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x2 xx = f2_from_bf16x2(wd[e]);
                ss2 = f2_fma(xx, xx, ss2);
            }
            const float ss = group_sum<LPH>(ss2.x + ss2.y);  // every lane of the warp takes part
            r = rsqrtf(ss * (1.0f / (float)D) + eps);
        }
        float v[8], o[8];
        unpack8(x[u], v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            int a, z;
            pair_regs<MODE>(e, a, z);
            // What passes has no part in its neighbour: 0 times an infinite one
            // would not be 0.  (Two selects per pair, 1 % of the ragged prompts'
            // time; a branch where r is 0, as an infinite element makes it, 2 %.)
            const float va = NORM && !turns ? 0.f : v[a], vz = NORM && !turns ? 0.f : v[z];
            const float oa = fmaf(vz, pc.c1[e], v[a] * pc.c0[e]), oz = fmaf(v[z], pc.c3[e], va * pc.c2[e]);
            o[a] = NORM ? r * oa : oa;
            o[z] = NORM ? r * oz : oz;
        }
        uint4 out = pack8(o);
        if (!NORM && !turns)
            out = x[u];  // passes bit for bit
        if (h < heads)
            store_quads<MODE>(to + (int64_t)h * step, o0, o1, out, keep);
    }
}

// PART: only the first rotary_dim elements of a head turn (or none), else all do,
// and nothing is asked of a lane (the long video 176 us with the question, 172
// without; it costs nothing where there are no weights).
template <int D, int MODE, bool NORM, bool APPEND, int U, bool PART>
__global__ void __launch_bounds__(kRcWarps * kWarp) rope_cache_kernel(const __grid_constant__ RopeCacheParams p)
{
    constexpr int LPH = D / 8;          // lanes per head
    constexpr int HPW = kWarp / LPH;    // heads per step
    constexpr int HB = HPW * U;         // heads per batch
    grid_dependency_wait();
    const int lane = threadIdx.x & (kWarp - 1);
    const long long task = (long long)blockIdx.x * kRcWarps + (threadIdx.x >> 5);
    const int v_row = (int)(task / p.runs_per_row);
    const int run = (int)(task - (long long)v_row * p.runs_per_row);
    RowSlot s;
    if (!map_valid_row(v_row, p.pk.cu_seqlens, p.pk.cu_seqlens_padded, p.pk.num_seqs, p.pk.num_rows_padded, lane, s))
        return;
    const int sub = lane / LPH, li = lane % LPH;
    const int nq = (p.num_q_heads + HB - 1) / HB, nk = (p.num_k_heads + HB - 1) / HB;
    const int total = nq + nk + (APPEND ? nk : 0);
    const int b0 = run * p.batches_per_run, b1 = min(b0 + p.batches_per_run, total);
    if (b0 >= b1)
        return;
    const bool turns = !PART || li < (p.rotary_dim >> 3);
    const int half = p.rotary_dim >> 1;
    const int o0 = quad_off<MODE>(li, 0, turns, half), o1 = quad_off<MODE>(li, 1, turns, half);

    // Where the row's k and v go: the rows' own outputs, or the token's slot
    // in the cache.  A token whose slot the table does not name is dropped.
    const int before = APPEND ? max(__ldg(p.cache_lens + s.seq), 0) : 0;
    uint16_t* k_to = nullptr;
    uint16_t* v_to = nullptr;
    if (APPEND) {
        const long long slot = (long long)before + s.local;
        const long long entry = slot / p.page_size;
        if (entry < p.max_pages) {
            const int page = __ldg(p.block_table + (int64_t)s.seq * p.table_stride + entry);
            if (page >= 0 && page < p.num_pages) {
                const int64_t at = (int64_t)page * p.page_stride + (slot - entry * p.page_size) * p.slot_stride;
                k_to = p.k_cache + at;
                v_to = p.v_cache + at;
            }
        }
    } else {
        k_to = p.k_out + (int64_t)s.row * p.k_out_stride;
    }
    const uint16_t* q_from = p.q + (int64_t)s.row * p.q_row_stride;
    const uint16_t* k_from = p.k + (int64_t)s.row * p.k_row_stride;
    const uint16_t* v_from = p.v + (int64_t)s.row * p.v_row_stride;
    uint16_t* q_to = p.q_out + (int64_t)s.row * p.q_out_stride;

    auto load = [&](int b, uint4 (&x)[U]) {
        const uint16_t* from = b < nq ? q_from : (b < nq + nk ? k_from : v_from);
        const int heads = b < nq ? p.num_q_heads : p.num_k_heads;
        const int h0 = (b < nq ? b : (b < nq + nk ? b - nq : b - nq - nk)) * HB + sub;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * HPW;
            x[u] = h < heads ? load_quads<MODE>(from + (int64_t)h * D, o0, o1) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    uint4 cur[U];
    load(b0, cur);

    // cos and sin (times g) of the lane's four pairs
    float c[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (turns && b0 < nq + nk) {
        const int off = p.pos_offset != nullptr ? max(__ldg(p.pos_offset + s.seq), 0) : before;
        const RowPosition rp = row_position((long long)s.local + off,
                                            p.rope_grid != nullptr ? p.rope_grid + 3 * s.seq : nullptr);
        const double2* table = reinterpret_cast<const double2*>(rp.is3d ? p.grid_freqs : p.freqs) + 2 * li;
        const double2 f01 = __ldg(table), f23 = __ldg(table + 1);
        const double f[4] = {f01.x, f01.y, f23.x, f23.y};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = 4 * li + e;
            const long long at = !rp.is3d ? rp.line : (j < p.sec_pairs[0] ? rp.t
                                                       : (j < p.sec_pairs[0] + p.sec_pairs[1] ? rp.h : rp.w));
            pair_cos_sin((double)at * f[e], c[e], sn[e]);
            c[e] *= p.attn_scale;
            sn[e] *= p.attn_scale;
        }
    }
    PairCoef pq, pk;
    fold<MODE, NORM>(pq, c, sn, turns, p.q_weight, o0, o1);
    if (NORM)
        fold<MODE, NORM>(pk, c, sn, turns, p.k_weight, o0, o1);

    for (int b = b0; b < b1; ++b) {
        uint4 nxt[U];
        if (b + 1 < b1)
            load(b + 1, nxt);
        if (b < nq) {
            turn_batch<D, MODE, NORM, U>(q_to, D, p.num_q_heads, b * HB + sub, o0, o1, false, turns, p.eps, pq, cur);
        } else if (!APPEND) {
            turn_batch<D, MODE, NORM, U>(k_to, D, p.num_k_heads, (b - nq) * HB + sub, o0, o1, false, turns, p.eps,
                                         NORM ? pk : pq, cur);
        } else if (k_to != nullptr) {
            const int h0 = (b - nq - (b < nq + nk ? 0 : nk)) * HB + sub;
            if (b < nq + nk) {
                turn_batch<D, MODE, NORM, U>(k_to, p.head_stride, p.num_k_heads, h0, o0, o1, true, turns, p.eps,
                                             NORM ? pk : pq, cur);
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (h0 + u * HPW < p.num_k_heads)
                        store_quads<MODE>(v_to + (h0 + u * HPW) * p.head_stride, o0, o1, cur[u], true);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            cur[u] = nxt[u];
    }
}

// A runtime choice as a compile-time one.
template <typename F>
cudaError_t with_bool(bool b, F f)
{
    return b ? f(std::true_type{}) : f(std::false_type{});
}

template <int D, int U>
cudaError_t launch_rc(RopeCacheParams p, int mode, cudaStream_t stream)
{
    constexpr int HB = (kWarp / (D / 8)) * U;
    const int nk = (p.num_k_heads + HB - 1) / HB;
    const int total = (p.num_q_heads + HB - 1) / HB + nk + (p.v != nullptr ? nk : 0);
    // Runs per row: one warp takes a whole row once the rows alone give every
    // SM 16 warps; below that a row's batches are spread over more warps.
    const long long want = (148LL * 16 + p.pk.num_rows_padded - 1) / p.pk.num_rows_padded;
    const int runs = (int)(want < total ? want : total);
    p.batches_per_run = (total + runs - 1) / runs;
    p.runs_per_row = (total + p.batches_per_run - 1) / p.batches_per_run;
    const unsigned grid = (unsigned)(((long long)p.pk.num_rows_padded * p.runs_per_row + kRcWarps - 1) / kRcWarps);
    const bool norm = p.k_weight != nullptr;
    auto launch = [&](auto* kernel) { return launch_kernel(kernel, grid, kRcWarps * kWarp, 0, stream, p); };
    auto pick = [&](auto norm_, auto append_, auto half_, auto part_) {
        constexpr bool kNorm = decltype(norm_)::value, kPart = !kNorm || decltype(part_)::value;
        constexpr int kMode = decltype(half_)::value ? kRopeHalf : kRopeInterleaved;
        return launch(rope_cache_kernel<D, kMode, kNorm, decltype(append_)::value, U, kPart>);
    };
    const bool half = mode == kRopeHalf, append = p.block_table != nullptr, part = p.rotary_dim < D;
    return with_bool(norm, [&](auto n) {
        return with_bool(append, [&](auto a) {
            return with_bool(half, [&](auto h) { return with_bool(part, [&](auto t) { return pick(n, a, h, t); }); });
        });
    });
}

// Steps per batch: 4, or 1 where 4-step batches would leave over half of their
// head slots empty (a few heads per row, as one rank's share has them): a
// batch of one step needs half the registers, so that twice the warps are
// resident (60,456 rows of 3 + 1 + 1 heads of 128: 98 -> 76 us).
template <int D>
cudaError_t launch_u(const RopeCacheParams& p, int mode, cudaStream_t stream)
{
    constexpr int kBatch = 4 * (kWarp / (D / 8));
    const int slots = ((p.num_q_heads + kBatch - 1) / kBatch + (p.num_k_heads + kBatch - 1) / kBatch) * kBatch;
    return 2 * (p.num_q_heads + p.num_k_heads) < slots ? launch_rc<D, 1>(p, mode, stream) : launch_rc<D, 4>(p, mode, stream);
}

}  // namespace

cudaError_t launch_rope_cache(const RopeCacheParams& p, int head_dim, int rope_mode, cudaStream_t stream)
{
    switch (head_dim) {
    case 64: return launch_u<64>(p, rope_mode, stream);
    case 128: return launch_u<128>(p, rope_mode, stream);
    case 256: return launch_u<256>(p, rope_mode, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace dit
