// paged_attention_tc.cu -- attention of a chunk of new tokens over a paged
// cache on the fifth-generation tensor cores (tcgen05, accumulators in tensor
// memory).
//
// The mathematics is paged_attention.cu's: one pass over the keys with the
// running maximum m, sum l and unnormalised o of a softmax, in fp32, the
// probabilities rounded to bf16 for their product with v.  The running
// maximum may lag: o and l are rescaled only when a row's maximum has grown
// by more than 2^8 since the last time, so probabilities reach at most 2^8
// (bf16 has fp32's range: the relative rounding is unchanged) and almost every
// tile skips the rescale.
//
// One block takes 256 rows, two tiles of 128 (a row is a (token, head) pair of
// one key head's group), over 128 keys at a time:
//   warps 0-3, 4-7  softmax of tile 0 and of tile 1; a thread owns a row, so
//                   row maxima and sums need no exchange
//   warp 8          issues the products: s = q k^T (both from shared memory)
//                   and o += p v (p from tensor memory)
//   warp 9, warp 10 fetch k and v with TMA, in boxes of rows that never cross a
//                   page: of 64 elements, the largest power of two rows that
//                   divides the page size, 4 to 128, or of whole heads, 8 rows,
//                   where those are fewer; warp 10 also writes zeros over the
//                   last step's rows of v behind the block's keys: the cache may
//                   hold anything behind the last token, and 0 * NaN must not
//                   reach the sums
//   warp 11         writes zeros over the first step's rows of v that lie before
//                   every row's window, whose tokens may be gone
// A box costs its warp some 40 cycles, whatever it holds.  (Heads of 256 in
// pages of 40: 154 us in boxes of 64 elements, 92 in whole heads, 81 by two
// warps; the video chunk in pages of 100, boxes of 4 rows: 5936 us by one warp,
// 3224 by two.)
// The softmax warps first copy q.  (Fetching k and v with 16-byte asynchronous
// copies by three warps held the video chunk at 3584 us, 2.8 us a step, and
// gathering TMA copies of four rows at 6210; without any copies it took 2611.)
// Steps begin at multiples of 128 keys, so boxes keep their alignment.
// The two tiles alternate: while one's softmax runs, the other's products do.
// Tensor memory (512 columns of 128 lanes x 32 bits): s0, s1 (128 each), o0,
// o1 (D each; heads of 256 leave room for one tile per block); p takes the
// second half of its s, once the row is in registers.
// The products of one tile are issued in the order o(i), s(i+1), and a
// commit covers everything issued before it, so "s(i+1) is there" also says
// that o(i) is complete and p(i) is free.
//
// Every wait is bounded: a wait that gives up raises a flag that ends the
// block's other waits, and the block's rows become NaN.  Whatever gave up,
// the fetching warps stay until their copies have landed and the issuing warp
// until its products have ended (bounded too), so that neither writes to shared
// or tensor memory that is no longer the block's.
#include <cuda.h>

#include "paged.cuh"

namespace dit {
namespace {

constexpr int kTcRows = 128;   // rows per tile
constexpr int kTcKeys = 128;   // keys per step
constexpr int kTcThreads = 384;
constexpr uint32_t kBlockBytes = kTcKeys * 128;  // 128 rows of 64 elements
constexpr float kTcLag = 8.f;  // log2 of how far probabilities may pass 1
constexpr long long kDrainCycles = 4000000000ll;  // about two seconds
// DIT_STALL=1 at build time, for tests: each of the first four key heads has
// barriers that never complete, and waits give up after a tenth of a millisecond
// instead of two seconds.
#ifndef DIT_STALL
#define DIT_STALL 0
#endif
constexpr long long kWaitCycles = DIT_STALL ? 200000ll : kDrainCycles;

// WHOLE: boxes of 8 rows of whole heads, else of 64 elements.  (A template:
// with strides read at run time the issuing warp fell behind, 2355 -> 2473 us
// for the video chunk.)
template <int D, bool WHOLE>
struct TcShape {
    static constexpr int kTiles = D == 256 ? 1 : 2;              // query tiles of a block
    static constexpr int kSlots = D == 256 ? 2 : (D == 128 ? 4 : 8);  // key or value tiles in shared memory
    static constexpr uint32_t kTile = (D / 64) * kBlockBytes;    // bytes of a tile (q, k or v)
    static constexpr uint32_t kGroup = WHOLE ? 1024 * (D / 64) : 1024;   // between a tile's 8-row groups
    static constexpr uint32_t kBlock = WHOLE ? 1024 : kBlockBytes;       // and its 64-element blocks
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kRing = kTiles * kTile;
    static constexpr uint32_t kBars = kRing + kSlots * kTile;
    static constexpr int kNumBars = 2 * kSlots + 12;
    static constexpr uint32_t kTmemPtr = kBars + kNumBars * 8;
    static constexpr uint32_t kAbort = kTmemPtr + 4;
    static constexpr uint32_t kSmem = kAbort + 4;
};

// ------------------------------------------------------------- barriers
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity, volatile int* abort)
{
    const long long from = clock64();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try(bar, parity))
                return true;
        if (*abort != 0)
            return false;
        if (clock64() - from > kWaitCycles) {
            *abort = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort)
{
    return mbar_try(bar, parity) || mbar_wait_long(bar, parity, abort);
}

// Until the phase is over, whether or not the block has given up.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity)
{
    const long long from = clock64();
    while (!mbar_try(bar, parity) && clock64() - from < kDrainCycles) {
    }
}

__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// A box of rows of 64 elements, from column x and row y.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
                 "[%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
// The same over whole heads: column block z on.
__device__ __forceinline__ void tma_box3(uint32_t dst, const CUtensorMap* map, int y, int z, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
                 "[%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(map), "r"(0), "r"(y), "r"(z), "r"(bar) : "memory");
}
// This thread's writes to shared memory, visible to the tensor cores' proxy.
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one != 0;
}

// ------------------------------------------------------------- tcgen05
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// d (+)= a b^T, a and b in shared memory
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
                 "r"((uint32_t)add) : "memory");
}
// d (+)= a b, a in tensor memory, b in shared memory
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
                 "r"((uint32_t)add) : "memory");
}

// 32 columns of the thread's lane.
__device__ __forceinline__ void tc_ld32(uint32_t addr, float* r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
                   "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]),
                   "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]),
                   "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]),
                   "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
                 : "r"(addr));
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t* r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
                 "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
                 "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]) : "memory");
}
// The loads before have landed.  The registers pass through, so that nothing
// that reads them moves above the wait.
__device__ __forceinline__ void tc_tie32(float* r)
{
    asm volatile("" : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]),
                       "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]),
                       "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]), "+f"(r[16]), "+f"(r[17]),
                       "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]),
                       "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]),
                       "+f"(r[30]), "+f"(r[31]));
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor, rows of 128 bytes permuted in 16-byte chunks
// by the row's low 3 bits (128-byte swizzle), 8-row groups `group` bytes apart.
// `lead` is the distance of 64-element blocks along the contiguous axis, read
// only where that axis is the product's outer one (v).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t group, uint32_t lead)
{
    return (uint64_t)((addr >> 4) & 0x3fffu) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(group >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: bf16 operands, fp32 accumulator, M x N, b along its
// inner axis (s = q k^T) or its outer one (o = p v).
template <int M, int N, bool B_OUTER>
struct TcIdesc {
    static constexpr uint32_t value = (1u << 4) | (1u << 7) | (1u << 10) | ((B_OUTER ? 1u : 0u) << 16) |
                                      ((uint32_t)(N / 8) << 17) | ((uint32_t)(M / 16) << 24);
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Probabilities 2^(s scale - base) of 64 scores of a row, to tensor memory as
// bf16; their sum.  The special-function units make 16 exponentials a cycle
// and SM: 1024 cycles for a tile.  (A polynomial on the FMA units for 1 to 5 of
// 8 pairs made the kernel slower, 2352 us -> 2420 for 1 of 8: its instructions
// cost what they save.)
__device__ __forceinline__ float exponentials(const float* s, float scale, float base, uint32_t to)
{
    const f32x2 scale2 = f2_make(scale, scale), base2 = f2_make(-base, -base);
    f32x2 sum[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
    uint32_t pk[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) {
        f32x2 e = f2_fma(f2_make(s[2 * c], s[2 * c + 1]), scale2, base2);
        e.x = ex2(e.x);
        e.y = ex2(e.y);
        sum[c & 1] = f2_add(sum[c & 1], e);
        pk[c] = f2_to_bf16x2(e);
    }
    tc_st32(to, pk);
    sum[0] = f2_add(sum[0], sum[1]);
    return sum[0].x + sum[0].y;
}

// Scores that the row does not see become -inf; their maximum is returned.
// keys: of the first score, from the row's first and to its last key.
__device__ __forceinline__ float mask_and_top(float* s, bool clear, int from, int to)
{
    if (!clear) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
            if (c < from || c >= to)
                s[c] = -INFINITY;
    }
    float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int c = 4; c < 64; c += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            top[e] = c + 4 + e < 64 ? fmaxf(top[e], fmaxf(s[c + e], s[c + 4 + e])) : fmaxf(top[e], s[c + e]);
    return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
}

__device__ __forceinline__ void hand_over(uint32_t bar)
{
    tc_wait_st();
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(bar);
}

// Byte offset of 16-byte chunk c of row r in a tile of 128 rows.
__device__ __forceinline__ uint32_t tc_off(int r, int c)
{
    return (uint32_t)(c >> 3) * kBlockBytes + (uint32_t)(r * 128 + (((c ^ r) & 7) << 4));
}

template <int D, bool WHOLE>
__global__ void __launch_bounds__(kTcThreads, 1) paged_attention_tc_kernel(const __grid_constant__ PagedParams p, const __grid_constant__ CUtensorMap k_map,
                          const __grid_constant__ CUtensorMap v_map)
{
    using S = TcShape<D, WHOLE>;
    constexpr int NS = S::kSlots;
    extern __shared__ __align__(1024) unsigned char smem[];
    grid_dependency_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int kvh = blockIdx.y, split = blockIdx.z;
    QueryTile q;
    // later tiles of a causal chunk see more keys: they go first
    if (!map_query_tile((int)(gridDim.x - 1 - blockIdx.x), p, S::kTiles * kTcRows, lane, q))
        return;
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + S::kAbort);
    const uint32_t bars = base + S::kBars;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (NS + s); };
    const uint32_t q_full = bars + 8u * (2 * NS);
    auto s_full = [&](int t) { return bars + 8u * (2 * NS + 1 + t); };
    auto o_full = [&](int t) { return bars + 8u * (2 * NS + 3 + t); };
    auto p_full = [&](int t, int h) { return bars + 8u * (2 * NS + 5 + 2 * t + h); };
    const uint32_t drained = bars + 8u * (2 * NS + 9), clean = bars + 8u * (2 * NS + 10);
    const uint32_t first_landed = bars + 8u * (2 * NS + 11);

    if (tid == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&k_map) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&v_map) : "memory");
        auto never = [&](int head) { return DIT_STALL && kvh == head ? 1u : 0u; };  // one arrival too many asked for
        for (int s = 0; s < NS; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1 + never(1));
        }
        mbar_init(q_full, S::kTiles * kTcRows + never(0));
        for (int t = 0; t < 2; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(p_full(t, 0), 4);
            mbar_init(p_full(t, 1), 4 + never(2));
            mbar_init(o_full(t), 1 + never(3));
        }
        mbar_init(drained, 1);
        mbar_init(clean, 1);
        mbar_init(first_landed, 1);
        *abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        proxy_fence();
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + S::kTmemPtr) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    // all 512 columns are the block's own, so its addresses start at 0
    constexpr uint32_t tmem = 0;

    // Keys of the two tiles, the block's share of them, and each tile's steps
    // [first, last) of the block's.
    int lo[2], hi[2], rows[2], unused;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        rows[t] = min(max(q.rows - t * kTcRows, 0), kTcRows);
        lo[t] = 0;
        hi[t] = 0;
        if (rows[t] > 0) {
            visible_keys(p, q, (q.first + t * kTcRows) / p.group, lo[t], unused);
            visible_keys(p, q, (q.first + t * kTcRows + rows[t] - 1) / p.group, unused, hi[t]);
        }
    }
    int k_lo = lo[0] / kTcKeys * kTcKeys, k_hi = max(hi[0], hi[1]);
    if (p.splits > 1) {
        const long long from = k_lo + (long long)split * p.split_keys;
        if (split + 1 < p.splits)
            k_hi = (int)min((long long)k_hi, from + p.split_keys);
        k_lo = (int)min(from, (long long)max(k_hi, 0));
    }
    int first[2], last[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int top = min(hi[t], k_hi);
        first[t] = max(lo[t] - k_lo, 0) / kTcKeys;
        last[t] = top > k_lo ? (top - k_lo + kTcKeys - 1) / kTcKeys : 0;
        if (rows[t] == 0 || last[t] <= first[t])
            first[t] = last[t] = 0;
    }
    const int steps = max(last[0], last[1]);
    // the last step's first row behind the block's keys: not fetched, or not
    // of a token; zeroed
    const int behind = min(k_hi - (k_lo + (steps - 1) * kTcKeys), kTcKeys);
    // the first step's rows that no row of the block sees; zeroed
    const int before = max(lo[0] - k_lo, 0);
    // by a whole warp, behind the copies into the slot
    auto zero_rows_of_v = [&](int slot, int from, int to, uint32_t bar) {
        for (int c = 0; c < D / 64; ++c)
            for (int e = from * 8 + lane; e < to * 8; e += 32) {
                const int r = e >> 3;
                *reinterpret_cast<uint4*>(smem + S::kRing + slot * S::kTile + c * S::kBlock + (r >> 3) * S::kGroup +
                                          (r & 7) * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
        proxy_fence();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar);
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 8) {
            // The whole warp walks the steps and one lane issues: operands
            // that every lane shares stay in uniform registers.  (With one
            // lane alone in the loop each product's operands were moved there
            // first, some 100 cycles per product of 64: the video chunk's
            // products alone 2036 us against 1781.)
            constexpr uint32_t kIdescS = TcIdesc<kTcRows, kTcKeys, false>::value;
            constexpr uint32_t kIdescO = TcIdesc<kTcRows, D, true>::value;
            auto in = [&](int t, int i) { return i >= first[t] && i < last[t]; };
            auto scores = [&](int t, int slot) {
                const uint32_t a = base + S::kQ + t * S::kTile, b = base + S::kRing + slot * S::kTile;
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t c = ks >> 2, in = (ks & 3) * 32;
                        tc_mma_ss(t * kTcKeys, smem_desc(a + c * kBlockBytes + in, 1024, 16),
                                  smem_desc(b + c * S::kBlock + in, S::kGroup, 16), kIdescS, ks > 0);
                    }
                    tc_commit(s_full(t));
                }
                __syncwarp();
            };
            auto products = [&](int t, int slot, int h, bool add) {
                const uint32_t b = base + S::kRing + slot * S::kTile;
                if (elect_one()) {
#pragma unroll
                    for (int ks = h * (kTcKeys / 32); ks < (h + 1) * (kTcKeys / 32); ++ks)
                        tc_mma_ts(2 * kTcKeys + t * D, t * kTcKeys + kTcKeys / 2 + ks * 8, smem_desc(b + ks * 2 * S::kGroup, S::kGroup, S::kBlock),
                                  kIdescO, add || ks > 0);
                }
                __syncwarp();
            };
            auto commit = [&](uint32_t bar) {
                if (elect_one())
                    tc_commit(bar);
                __syncwarp();
            };
            auto wait = [&](uint32_t bar, uint32_t parity) {
                return (bool)__all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
            };
            bool go = steps > 0 && wait(q_full, 0) && wait(full(0), 0);
            if (go) {
                tc_fence_after();
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (in(t, 0))
                        scores(t, 0);
                commit(empty(0));
            }
            for (int i = 0; go && i < steps; ++i) {
                const int vt = 2 * i + 1, kt = 2 * i + 2;
                const int vs = vt % NS, ks = kt % NS;
                go = wait(full(vs), (uint32_t)(vt / NS) & 1u);
                if (go && i + 1 == steps && behind < kTcKeys)
                    go = wait(clean, 0);
                if (go && i + 1 < steps)
                    go = wait(full(ks), (uint32_t)(kt / NS) & 1u);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (go && in(t, i)) {
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (go && (go = wait(p_full(t, h), (uint32_t)(i - first[t]) & 1u))) {
                                tc_fence_after();
                                products(t, vs, h, i > first[t]);
                            }
                        if (go && i + 1 == last[t])
                            commit(o_full(t));
                    }
                    if (go && t == 1)
                        commit(empty(vs));
                    if (go && in(t, i + 1))
                        scores(t, ks);
                }
                if (go && i + 1 < steps)
                    commit(empty(ks));
            }
            if (steps > 0) {  // what was issued ends before the memory is freed
                commit(drained);
                mbar_drain(drained, 0);
                __syncwarp();
            }
        } else if (warp < 11) {
            const int of_v = warp - 9;  // 0: k, 1: v
            const CUtensorMap* map = of_v ? &v_map : &k_map;
            // Lane e fetches the box of rows e * box of every tile, where there
            // is one.  Page numbers are read a step ahead.
            const int32_t* table = p.block_table + (int64_t)q.seq * p.table_stride;
            const int head_row = kvh * p.head_rows, x = kvh * p.head_cols;
            const int box = p.box_rows;
            int page = -1, slot_in = 0, row = 0;
            bool next = false, there = false;
            auto look_up = [&](int i) {
                const int key = k_lo + i * kTcKeys + lane * box;
                next = lane * box < kTcKeys && key < k_hi;
                if (next) {
                    const unsigned entry = page_of(p, key);
                    slot_in = key - (int)entry * p.page_size;
                    page = __ldg(table + entry);
                }
            };
            if (steps > 0)
                look_up(0);
            int i = 0;
            for (; i < steps; ++i) {
                const int j = 2 * i + of_v, slot = j % NS;
                there = next;
                // a page outside the cache: rows outside the map, which read as zeros
                row = page >= 0 && page < p.num_pages ? page * p.page_rows + slot_in + head_row : -kTcKeys;
                if (i + 1 < steps)
                    look_up(i + 1);
                if (j >= NS && !__all_sync(0xffffffffu, mbar_wait(empty(slot), (uint32_t)(j / NS - 1) & 1u, abort)))
                    break;
                // a first tile that warp 11 has to look at reports to it
                const uint32_t bar = of_v && i == 0 && before > 0 ? first_landed : full(slot);
                const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, there));
                if (lane == 0)
                    mbar_expect(bar, boxes * (uint32_t)box * (D * 2));
                __syncwarp();
                if (there) {
                    const uint32_t to = base + S::kRing + slot * S::kTile + (uint32_t)lane * (WHOLE ? S::kGroup : (uint32_t)box * 128);
                    if (WHOLE) {
                        tma_box3(to, map, row, x / 64, bar);
                    } else {
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tma_box(to + c * kBlockBytes, map, x + 64 * c, row, bar);
                    }
                }
                __syncwarp();
            }
            // The last tile of v: this warp has seen the slot's previous use end,
            // so the parity it waits for is the tile's own.
            if (of_v && i == steps && behind < kTcKeys && steps > 0) {
                const int j = 2 * steps - 1, slot = j % NS;
                if (__all_sync(0xffffffffu, mbar_wait(full(slot), (uint32_t)(j / NS) & 1u, abort)))
                    zero_rows_of_v(slot, behind, kTcKeys, clean);
            }
            // the copies under way land before the block ends
            for (int e = max(i - NS / 2, 0); lane == 0 && e < i; ++e) {
                const int j = 2 * e + of_v;
                mbar_drain(full(j % NS), (uint32_t)(j / NS) & 1u);
            }
        } else if (steps > 0 && before > 0) {
            // v's first tile, the second one fetched; behind this it counts as there
            mbar_drain(first_landed, 0);
            __syncwarp();
            zero_rows_of_v(1, 0, before, full(1));
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int t = warp >> 2;
        const int r = tid & (kTcRows - 1);
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's 32 lanes: bits 16 and up, times 32
        const uint32_t s_at = tmem + t * kTcKeys + lanes, o_at = tmem + 2 * kTcKeys + t * D + lanes;
        const uint32_t p_at = s_at + kTcKeys / 2;
        const int have = t ? rows[1] : rows[0];
        const bool mine = r < have;
        const int at = q.first + t * kTcRows + min(r, max(have - 1, 0));
        const int token = at / p.group, head = kvh * p.group + at % p.group;
        if (steps > 0 && t < S::kTiles) {
            // a warp copies the queries of its own 32 rows, RPI rows at a time
            constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte chunks per row, rows per instruction
            const int64_t mine_at = (int64_t)(q.row0 + token) * p.q_row_stride + head * D;
            const uint32_t there = __ballot_sync(0xffffffffu, mine);
            const uint32_t to = base + S::kQ + t * S::kTile;
#pragma unroll
            for (int e = 0; e < 32; e += RPI) {
                const int row = e + lane / CH, c = lane % CH;
                const int64_t from = __shfl_sync(0xffffffffu, mine_at, row);
                cp_async16(to + tc_off((r & ~31) + row, c), p.q + from + c * 8, (there >> row) & 1u);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            proxy_fence();
            mbar_arrive(q_full);
        }
        int r_lo, r_hi;
        visible_keys(p, q, token, r_lo, r_hi);
        r_hi = min(r_hi, k_hi);
        float m = -INFINITY, l = 0.f;
        bool go = true;
        const int n0 = t ? first[1] : first[0], n1 = t ? last[1] : last[0];
        for (int i = n0; i < n1; ++i) {
            go = mbar_wait(s_full(t), (uint32_t)(i - n0) & 1u, abort);
            go = __all_sync(0xffffffffu, go);
            if (!go)
                break;
            tc_fence_after();
            // The exponentials take the last step's m, before this step's
            // maximum is known; a maximum that has outgrown it (the first
            // step's always has) brings the sums up to date and repeats the
            // first half, which is handed over only then.
            const int k0 = k_lo + i * kTcKeys;
            const bool clear = __all_sync(0xffffffffu, r_lo <= k0 && r_hi >= k0 + kTcKeys);
            float s[kTcKeys];
#pragma unroll
            for (int c = 0; c < kTcKeys; c += 32)
                tc_ld32(s_at + c, s + c);
            tc_wait_ld();
#pragma unroll
            for (int c = 0; c < kTcKeys; c += 32)
                tc_tie32(s + c);
            float mx = fmaxf(mask_and_top(s, clear, r_lo - k0, r_hi - k0),
                             mask_and_top(s + 64, clear, r_lo - k0 - 64, r_hi - k0 - 64)) * p.scale_log2;
            float base_m = m == -INFINITY ? 0.f : m;
            float part = exponentials(s, p.scale_log2, base_m, p_at);
            if (__any_sync(0xffffffffu, mx > m + kTcLag)) {
                const float mn = mx > m + kTcLag ? mx : m;
                const float f = m == mn ? 1.f : ex2(m - mn);  // -inf stays -inf until a key is seen
                m = mn;
                base_m = m == -INFINITY ? 0.f : m;
                l *= f;
                if (i > n0) {
#pragma unroll
                    for (int c = 0; c < D; c += 32) {
                        float o[32];
                        tc_ld32(o_at + c, o);
                        tc_wait_ld();
                        tc_tie32(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] *= f;
                        tc_st32(o_at + c, reinterpret_cast<const uint32_t*>(o));
                    }
                }
                float again[64];  // the first half's scores: p has only taken the second half's place
                tc_ld32(s_at, again);
                tc_ld32(s_at + 32, again + 32);
                tc_wait_ld();
                tc_tie32(again);
                tc_tie32(again + 32);
                mask_and_top(again, clear, r_lo - k0, r_hi - k0);
                tc_wait_st();  // two stores to the same columns keep no order of their own
                part = exponentials(again, p.scale_log2, base_m, p_at);
            }
            hand_over(p_full(t, 0));
            part += exponentials(s + 64, p.scale_log2, base_m, p_at + 32);
            l += part;
            hand_over(p_full(t, 1));
        }
        if (go && n1 > n0) {
            go = mbar_wait(o_full(t), 0, abort);
            go = __all_sync(0xffffffffu, go);
            tc_fence_after();
        }
        if (!go)
            m = NAN;  // and with it lse, or the split's weight in the join
        // the thread's row: output, or the split's part
        const bool whole = p.splits == 1;
        const float inv = whole ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : 1.f;
        const int64_t part = partial_index(p, q.ordinal0 + token, head, split);
        uint16_t* out = p.out + (int64_t)(q.row0 + token) * p.out_row_stride + head * D;
        float* part_o = whole ? nullptr : p.part_o + part * D;
        if (n1 > n0 || whole) {
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                float o[32];
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    o[e] = 0.f;
                if (n1 > n0) {  // uniform over the warpgroup
                    tc_ld32(o_at + c, o);
                    tc_wait_ld();
                    tc_tie32(o);
                }
                if (!go)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = NAN;
                if (!mine)
                    continue;
                if (whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4*>(out + c + e) =
                            make_uint4(pack2(o[e] * inv, o[e + 1] * inv), pack2(o[e + 2] * inv, o[e + 3] * inv),
                                       pack2(o[e + 4] * inv, o[e + 5] * inv), pack2(o[e + 6] * inv, o[e + 7] * inv));
                } else {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<float4*>(part_o + c + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                }
            }
        }
        if (mine) {
            if (!whole)
                p.part_ml[part] = make_float2(n1 > n0 ? m : -INFINITY, l);
            else if (p.lse != nullptr)
                p.lse[(int64_t)(q.row0 + token) * p.num_q_heads + head] = (m + log2f(l)) * kLn2;
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 8)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// The cache as rows of one head's elements, slot_stride apart: element x of row
// g * page_rows + s (+ head_rows per head) is what the caller calls page g,
// slot s, with a head's columns from h * head_cols.
bool cache_map(CUtensorMap& map, const PagedParams& p, const uint16_t* cache, int head_dim, bool whole,
               const CacheRows& c)
{
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<Encode>(fn);
    }();
    const cuuint64_t heads[3] = {64, (cuuint64_t)c.rows, (cuuint64_t)c.cols / 64};
    const cuuint64_t flat[2] = {(cuuint64_t)c.cols, (cuuint64_t)c.rows};
    const cuuint64_t strides[2] = {(cuuint64_t)p.slot_stride * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.box_rows, (cuuint32_t)head_dim / 64}, step[3] = {1, 1, 1};
    return encode != nullptr &&
           encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, whole ? 3 : 2, const_cast<uint16_t*>(cache),
                  whole ? heads : flat, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool WHOLE>
cudaError_t launch_tc_boxes(PagedParams p, const CacheRows& c, int tiles, cudaStream_t stream)
{
    CUtensorMap k_map, v_map;
    p.page_rows = c.page_rows;
    p.head_rows = c.head_rows;
    p.head_cols = c.head_cols;
    p.box_rows = WHOLE ? 8 : c.box_rows;
    if (!cache_map(k_map, p, p.k_cache, D, WHOLE, c) || !cache_map(v_map, p, p.v_cache, D, WHOLE, c))
        return cudaErrorInvalidValue;
    auto* kernel = paged_attention_tc_kernel<D, WHOLE>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TcShape<D, WHOLE>::kSmem);
    if (e != cudaSuccess)
        return e;
    return launch_kernel(kernel, dim3((unsigned)tiles, (unsigned)p.num_kv_heads, (unsigned)p.splits), kTcThreads,
                         TcShape<D, WHOLE>::kSmem, stream, p, k_map, v_map);
}

template <int D>
cudaError_t launch_tc(const PagedParams& p, int tiles, cudaStream_t stream)
{
    CacheRows c;
    if (!cache_rows(p.page_stride, p.slot_stride, p.head_stride, p.num_pages, p.page_size, p.num_kv_heads, D, c))
        return cudaErrorInvalidValue;
    // whole heads where they make fewer boxes of a tile
    if constexpr (D > 64)
        if (c.box_rows >= 8 && kTcKeys / c.box_rows * (D / 64) > kTcKeys / 8 && c.head_cols % 64 == 0)
            return launch_tc_boxes<D, true>(p, c, tiles, stream);
    return launch_tc_boxes<D, false>(p, c, tiles, stream);
}

}  // namespace

bool cache_rows(int64_t page_stride, int64_t slot_stride, int64_t head_stride, int num_pages, int page_size,
                int num_kv_heads, int head_dim, CacheRows& c)
{
    const int64_t pages = num_pages > 0 ? num_pages : 1;
    if (page_size % 4 != 0)  // 32 boxes of a tile, one per lane of the fetching warp
        return false;
    int64_t head_rows = 0, head_cols = 0;
    if (num_kv_heads > 1) {  // heads lie within a row (slot-major pages) or whole rows apart (head-major)
        if (head_stride * (num_kv_heads - 1) + head_dim <= slot_stride)
            head_cols = head_stride;
        else if (head_stride % slot_stride == 0)
            head_rows = head_stride / slot_stride;
        else
            return false;
    }
    if (pages > 1 && page_stride % slot_stride != 0)
        return false;
    const int64_t page_rows = pages > 1 ? page_stride / slot_stride : 0;
    const int64_t rows = (pages - 1) * page_rows + (num_kv_heads - 1) * head_rows + page_size;
    const int64_t cols = (num_kv_heads - 1) * head_cols + head_dim;
    if (rows > INT32_MAX || cols > INT32_MAX || slot_stride >= (1ll << 38))
        return false;
    const int32_t power = page_size & -page_size;
    c = CacheRows{(int32_t)page_rows, (int32_t)head_rows, (int32_t)head_cols, power < kTcKeys ? power : kTcKeys, rows, cols};
    return true;
}

cudaError_t launch_paged_attention_tc(const PagedParams& p, int tiles, int head_dim, cudaStream_t stream)
{
    switch (head_dim) {
    case 64: return launch_tc<64>(p, tiles, stream);
    case 128: return launch_tc<128>(p, tiles, stream);
    case 256: return launch_tc<256>(p, tiles, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace dit
