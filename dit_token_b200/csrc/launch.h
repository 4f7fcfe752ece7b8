// launch.h -- internal interface between the C ABI (api.cu) and the kernel
// translation units.  Arguments reaching these launchers are already
// validated; every launcher only enqueues and returns cudaGetLastError().
#pragma once

#include <cstdint>
#include <utility>

#include <cuda_runtime.h>

namespace dit {

// Programmatic dependent launch.  Every kernel of the library starts with
// grid_dependency_wait() (common.cuh) before its first global-memory access
// -- the packing descriptors included -- and then lets its own dependents
// launch.  So each launch may carry the programmatic-serialization attribute:
// when the previous kernel on the stream lets it, this kernel's CTAs are
// placed and resident while that kernel drains, and start the moment it
// completes (its writes visible), instead of after a full launch gap.  A
// kernel launched after one that does not take part simply starts when that
// one completes, as without the attribute.  DIT_PDL=0 at build time launches
// plainly (for comparison).
#ifndef DIT_PDL
#define DIT_PDL 1
#endif

// A 32-byte boundary (the 256-bit row accesses need one).
inline bool aligned32(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 31u) == 0; }

template <typename... KArgs, typename... Args>
inline cudaError_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                 cudaStream_t stream, Args&&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = DIT_PDL ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

struct Packing {
    const int32_t* cu_seqlens;
    const int32_t* cu_seqlens_padded;
    int32_t num_seqs;
    int32_t num_rows_padded;
};


// Rotary layouts of dit_qk_rmsnorm_rope_ex (the DIT_ROPE_* values of the ABI).
constexpr int kRopeInterleaved = 0;
constexpr int kRopeHalf = 1;
constexpr int kRopeNone = 2;

struct QkParams {
    uint16_t* q;
    uint16_t* k;
    const uint16_t* q_weight;
    const uint16_t* k_weight;
    const int32_t* rope_grid;
    const int32_t* pos_offset;  // [num_seqs] start of each sequence's rows in the whole sequence, or null
    int64_t q_row_stride;
    int64_t k_row_stride;
    Packing pk;
    int32_t num_q_heads;
    int32_t num_k_heads;
    float eps;
    // Rotary frequency bases, fp64 from the host: pair j of a 1D row turns
    // at base_1d^j = theta^(-2j/D); on a 3D row pair j lies in section s (the
    // first sec_pairs[0] pairs t, the next sec_pairs[1] h, the rest w) and
    // turns at base_3d[s]^j' = theta^(-2j'/d_s), j' its index in the section.
    double base_1d;
    double base_3d[3];
    int32_t sec_pairs[3];
};

struct AdalnParams {
    const uint16_t* x;
    uint16_t* out;
    const void* shift;  // bf16 or fp32 (mod_f32)
    const void* scale;
    int64_t x_row_stride;
    int64_t out_row_stride;
    int64_t mod_seq_stride;
    Packing pk;
    int32_t hidden;
    float eps;
    int32_t mod_f32;
};

struct GatedParams {
    const uint16_t* x;
    const uint16_t* y;
    const void* gate;  // bf16 or fp32 (gate_f32)
    uint16_t* out;
    int64_t x_row_stride;
    int64_t y_row_stride;
    int64_t gate_seq_stride;
    int64_t out_row_stride;
    Packing pk;
    int32_t hidden;
    int32_t gate_f32;
};

struct FusedParams {
    const uint16_t* x;
    const uint16_t* y;
    const void* gate;  // gate, shift, scale: bf16 or fp32 (mod_f32)
    const void* shift;
    const void* scale;
    uint16_t* res_out;
    uint16_t* norm_out;
    int64_t x_row_stride;
    int64_t y_row_stride;
    int64_t gate_seq_stride;
    int64_t mod_seq_stride;
    int64_t res_row_stride;
    int64_t norm_row_stride;
    Packing pk;
    int32_t hidden;
    float eps;
    int32_t mod_f32;
};

struct SwigluParams {
    const uint16_t* a;
    const uint16_t* b;
    uint16_t* out;
    int64_t a_row_stride;
    int64_t b_row_stride;
    int64_t out_row_stride;
    Packing pk;
    int32_t inner;
};

struct FramesParams {
    const float* x;
    uint8_t* out;
    int64_t B, C, T, H, W;
    int32_t layout;
};

// dit_qk_rope_scaled (block_table null: k goes to k_out, no v) and
// dit_qkv_rope_append (k and v go to the cache).  Without rotation
// rotary_dim is 0 and every lane passes.
struct RopeCacheParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;  // null: none
    uint16_t* q_out;
    uint16_t* k_out;
    uint16_t* k_cache;
    uint16_t* v_cache;
    const uint16_t* q_weight;  // both null: no RMSNorm
    const uint16_t* k_weight;
    const double* freqs;       // [rotary_dim / 2] pair frequencies of 1D rows
    const double* grid_freqs;  // [rotary_dim / 2] of 3D rows, t, h, w pairs in order
    const int32_t* rope_grid;
    const int32_t* pos_offset;
    const int32_t* block_table;
    const int32_t* cache_lens;
    int64_t q_row_stride, k_row_stride, v_row_stride, q_out_stride, k_out_stride;
    int64_t page_stride, slot_stride, head_stride;
    int64_t table_stride;
    Packing pk;
    int32_t num_q_heads, num_k_heads;
    int32_t rotary_dim;
    int32_t sec_pairs[2];  // pairs of the t and h sections
    int32_t num_pages, page_size, max_pages;
    float eps, attn_scale;
    int32_t runs_per_row, batches_per_run;  // set by the launcher
};

// dit_paged_attention.
struct PagedParams {
    const uint16_t* q;
    const uint16_t* k_cache;
    const uint16_t* v_cache;
    uint16_t* out;
    float* lse;  // [num_rows_padded][num_q_heads] or null
    const int32_t* block_table;
    const int32_t* kv_lens;
    float* part_o;    // partial sums of the splits, see partial_index
    float2* part_ml;
    int64_t q_row_stride, out_row_stride;
    int64_t page_stride, slot_stride, head_stride;
    int64_t table_stride;
    Packing pk;
    int32_t num_q_heads, num_kv_heads, group;  // group = q heads per key head
    int32_t num_pages, page_size, max_pages;
    uint32_t page_mul, page_shift;  // key / page_size = key * page_mul >> page_shift
    float scale_log2;               // softmax scale times log2(e)
    int32_t causal, window;         // window 0: none
    int32_t splits, split_keys;
    // Which sequences a launch takes, by their rows (tokens times group): a
    // mixed batch's few-row ones go to the narrow kernel (narrow_rows at most),
    // the others (more than skip_rows) to the one for chunks.
    int32_t narrow_rows, skip_rows;
    int32_t page_rows, head_rows, head_cols, box_rows;  // see CacheRows; set by the launcher that uses them
};

// A cache whose strides make it a matrix of rows slot_stride apart: slot s of
// page g, head h is row g * page_rows + s + h * head_rows, columns from
// h * head_cols.  box_rows: the largest power of two, at most 128, that divides
// the page size.  false: its strides do not, or the page size is no multiple of 4.
struct CacheRows {
    int32_t page_rows, head_rows, head_cols, box_rows;
    int64_t rows, cols;
};
bool cache_rows(int64_t page_stride, int64_t slot_stride, int64_t head_stride, int num_pages, int page_size,
                int num_kv_heads, int head_dim, CacheRows& c);

// Which kernel a call takes, and how the key axis is cut.
constexpr int kPagedNarrow = 0;
constexpr int kPagedWide = 1;
constexpr int kPagedTc = 2;
constexpr int kNarrowRows = 32;  // rows (tokens times group) the narrow kernel is for: two tiles
struct PagedPlan {
    int kind;
    bool mixed;      // the narrow kernel runs before the other, for the few-row sequences
    int tile_rows;
    int tiles;       // upper bound of the batch's query tiles
    int splits;
    int split_keys;
    int64_t part_rows;   // rows of partial sums in the workspace, the narrow kernel's first
    int64_t bytes;       // workspace of this call
    int64_t most_bytes;  // of any window and shorter key axis at these sizes
};
// false: the batch has more tiles than a launch can name
// regular: cache_rows holds for the cache
bool paged_plan(int64_t rows, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int64_t max_chunk,
                int64_t max_kv_len, int64_t window, bool regular, PagedPlan& plan);
cudaError_t launch_paged_attention_tc(const PagedParams& p, int tiles, int head_dim, cudaStream_t stream);
int64_t paged_narrow_slots(int head_dim);  // rows of partial sums it wants
// mixed: narrow_rows leaves the batch's other sequences out
cudaError_t launch_paged_attention_narrow(const PagedParams& p, bool mixed, int head_dim, cudaStream_t stream);
cudaError_t launch_paged_attention(const PagedParams& p, const PagedPlan& plan, int head_dim, cudaStream_t stream);

cudaError_t launch_rope_cache(const RopeCacheParams& p, int head_dim, int rope_mode, cudaStream_t stream);
cudaError_t launch_frames_to_u8(const FramesParams& p, cudaStream_t stream);
cudaError_t launch_qk_rmsnorm_rope(const QkParams& p, int head_dim, int rope_mode, cudaStream_t stream);
cudaError_t launch_adaln_modulate(const AdalnParams& p, cudaStream_t stream);

// How dit_adaln_modulate lays a row out: 2, 4 or 8 words (8-, 16- or 32-byte
// accesses) per lane vector, a row per warp (team 1) or per CTA of 2, 4 or 8
// warps, and whether the per-sequence vectors are read 32 bytes at a time.
// adaln_shape picks it for a call; launch_adaln_shape runs a given one (every
// shape computes the same result up to the order of the row statistics).
struct AdalnShape {
    int row_words;
    int team;
    bool wide_vectors;
};
AdalnShape adaln_shape(const AdalnParams& p);
cudaError_t launch_adaln_shape(const AdalnParams& p, const AdalnShape& shape, cudaStream_t stream);
cudaError_t launch_gated_residual(const GatedParams& p, cudaStream_t stream);
cudaError_t launch_swiglu(const SwigluParams& p, cudaStream_t stream);
cudaError_t launch_gated_residual_adaln(const FusedParams& p, cudaStream_t stream);
cudaError_t launch_av_stream_seqlens(const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                                     const int32_t* rope_grid, const int32_t* pos_offset, int32_t num_seqs,
                                     int32_t* out_cu_seqlens, int32_t* out_cu_seqlens_padded, cudaStream_t stream);
cudaError_t launch_validate_seqlens(const Packing& pk, int64_t num_rows_padded, int32_t* flag,
                                    cudaStream_t stream);

// Largest hidden size dit_adaln_modulate supports (8 warps x 8 vectors x 32 lanes x 8).
constexpr int kMaxAdalnHidden = 16384;

// Key heads of dit_paged_attention: a launch's second grid axis.
constexpr int kMaxKvHeads = 65535;

}  // namespace dit
