// api.cu -- the C ABI declared in include/dit_token.h and dit_paged.h: host-side argument
// checks, the rotary frequency bases, and the launches.  Nothing here
// allocates or synchronizes; the only state is thread-local: the last CUDA
// error.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "dit_paged.h"
#include "dit_token.h"
#include "launch.h"

static_assert(DIT_ROPE_INTERLEAVED == dit::kRopeInterleaved && DIT_ROPE_HALF == dit::kRopeHalf &&
                  DIT_ROPE_NONE == dit::kRopeNone,
              "rotary mode codes");

namespace {

thread_local int32_t g_last_cuda_error = 0;

// The rotary frequency bases of p, in fp64: theta^(-2/D) for 1D rows (pair j
// turns at its j-th power, theta^(-2j/D)); on 3D rows pair j lies in the t, h
// or w section of d_s elements (d_s / 2 pairs) and turns at
// theta^(-2j'/d_s), the j'-th power of theta^(-2/d_s), j' its index inside
// the section.  The kernel forms each pair's frequency from these.
void rope_bases(dit::QkParams& p, float rope_theta, int32_t head_dim, int32_t sec_t, int32_t sec_h, int32_t sec_w,
                bool grid)
{
    const double theta = (double)rope_theta;
    const int32_t sec[3] = {sec_t, sec_h, sec_w};
    p.base_1d = std::pow(theta, -2.0 / head_dim);
    for (int s = 0; s < 3; ++s) {
        const bool used = grid && sec[s] > 0;
        p.base_3d[s] = used ? std::pow(theta, -2.0 / sec[s]) : 0.0;
        p.sec_pairs[s] = grid ? sec[s] / 2 : 0;
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool mult8(int64_t v) { return (v & 7) == 0; }

// A per-sequence vector stride keeps every sequence's vector 16-byte aligned:
// a multiple of 8 bf16 or of 4 fp32 elements.
bool mod_stride_ok(int64_t v, bool f32) { return f32 ? (v & 3) == 0 : mult8(v); }

bool known_dtype(int32_t d) { return d == DIT_DTYPE_BF16 || d == DIT_DTYPE_F32; }

dit_status from_cuda(cudaError_t e)
{
    if (e == cudaSuccess)
        return DIT_OK;
    g_last_cuda_error = (int32_t)e;
    return DIT_ERR_CUDA;
}

// Checks shared by every operator: sizes, then the descriptor pointers.
// Returns DIT_OK and sets *nothing_to_do when the batch is empty.
dit_status check_packing(const int32_t* cs, const int32_t* cp, int32_t num_seqs, int64_t num_rows_padded,
                         bool* nothing_to_do)
{
    if (num_seqs < 0 || num_rows_padded < 0 || num_rows_padded > INT32_MAX)
        return DIT_ERR_SHAPE;
    *nothing_to_do = (num_seqs == 0 || num_rows_padded == 0);
    if (*nothing_to_do)
        return DIT_OK;
    if (!cs || !cp)
        return DIT_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(cs) & 3u) || (reinterpret_cast<uintptr_t>(cp) & 3u))
        return DIT_ERR_ALIGN;
    return DIT_OK;
}

dit::Packing packing(const int32_t* cs, const int32_t* cp, int32_t num_seqs, int64_t num_rows_padded)
{
    return dit::Packing{cs, cp, num_seqs, (int32_t)num_rows_padded};
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Checks shared by the two calls that turn q and k by a frequency table.
dit_status check_rope_table(int32_t num_q_heads, int32_t num_k_heads, int32_t head_dim, int32_t rotary_dim,
                            const int32_t* rope_grid, int32_t sec_t, int32_t sec_h, int32_t sec_w, float attn_scale,
                            float eps, int32_t rope_mode)
{
    if (num_q_heads < 0 || num_k_heads < 0 || head_dim <= 0)
        return DIT_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return DIT_ERR_UNSUPPORTED;
    if (rope_mode != DIT_ROPE_INTERLEAVED && rope_mode != DIT_ROPE_HALF && rope_mode != DIT_ROPE_NONE)
        return DIT_ERR_UNSUPPORTED;
    if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(attn_scale))
        return DIT_ERR_SHAPE;
    if (rope_mode == DIT_ROPE_NONE)
        return DIT_OK;
    if (rotary_dim < 8 || rotary_dim > head_dim || (rotary_dim & 7))
        return DIT_ERR_SHAPE;
    if (rope_grid && (sec_t < 0 || sec_h < 0 || sec_w < 0 || (sec_t | sec_h | sec_w) & 1 ||
                      (int64_t)sec_t + sec_h + sec_w != rotary_dim))
        return DIT_ERR_SHAPE;
    return DIT_OK;
}

// The cache's sizes and strides.
dit_status check_cache(int32_t head_dim, int64_t page_stride, int64_t slot_stride, int64_t head_stride,
                       int32_t num_pages, int32_t page_size, int64_t table_stride, int32_t max_pages)
{
    if (num_pages < 0 || page_size <= 0 || max_pages < 0 || table_stride < max_pages || page_stride < 0 ||
        slot_stride < head_dim || head_stride < head_dim)
        return DIT_ERR_SHAPE;
    if (!mult8(page_stride) || !mult8(slot_stride) || !mult8(head_stride))
        return DIT_ERR_ALIGN;
    return DIT_OK;
}

void set_rope_table(dit::RopeCacheParams& p, const double* freqs, const double* grid_freqs, int32_t rotary_dim,
                    const int32_t* rope_grid, const int32_t* pos_offset, int32_t sec_t, int32_t sec_h, int32_t rope_mode)
{
    const bool turns = rope_mode != DIT_ROPE_NONE;
    p.freqs = freqs;
    p.grid_freqs = grid_freqs;
    p.rotary_dim = turns ? rotary_dim : 0;
    p.rope_grid = turns ? rope_grid : nullptr;
    p.pos_offset = pos_offset;
    p.sec_pairs[0] = sec_t / 2;
    p.sec_pairs[1] = sec_h / 2;
}

}  // namespace

extern "C" {

dit_status dit_qk_rmsnorm_rope(void* q, int64_t q_row_stride, void* k, int64_t k_row_stride,
                               const void* q_weight, const void* k_weight,
                               const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                               int32_t num_seqs, int64_t num_rows_padded,
                               int32_t num_q_heads, int32_t num_k_heads, int32_t head_dim,
                               const int32_t* rope_grid, int32_t sec_t, int32_t sec_h, int32_t sec_w,
                               float rope_theta, float eps, void* stream)
{
    if (head_dim != 64 && head_dim != 128 && head_dim > 0)
        return DIT_ERR_UNSUPPORTED;  // the original entry point keeps its documented range
    return dit_qk_rmsnorm_rope_ex(q, q_row_stride, k, k_row_stride, q_weight, k_weight, cu_seqlens,
                                  cu_seqlens_padded, num_seqs, num_rows_padded, num_q_heads, num_k_heads,
                                  head_dim, rope_grid, sec_t, sec_h, sec_w, rope_theta, eps,
                                  DIT_ROPE_INTERLEAVED, stream);
}

dit_status dit_qk_rmsnorm_rope_ex(void* q, int64_t q_row_stride, void* k, int64_t k_row_stride,
                                  const void* q_weight, const void* k_weight,
                                  const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                                  int32_t num_seqs, int64_t num_rows_padded,
                                  int32_t num_q_heads, int32_t num_k_heads, int32_t head_dim,
                                  const int32_t* rope_grid, int32_t sec_t, int32_t sec_h, int32_t sec_w,
                                  float rope_theta, float eps, int32_t rope_mode, void* stream)
{
    return dit_qk_rmsnorm_rope_shard(q, q_row_stride, k, k_row_stride, q_weight, k_weight, cu_seqlens,
                                     cu_seqlens_padded, num_seqs, num_rows_padded, num_q_heads, num_k_heads,
                                     head_dim, rope_grid, sec_t, sec_h, sec_w, rope_theta, eps, rope_mode, nullptr,
                                     stream);
}

dit_status dit_qk_rmsnorm_rope_shard(void* q, int64_t q_row_stride, void* k, int64_t k_row_stride,
                                     const void* q_weight, const void* k_weight,
                                     const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                                     int32_t num_seqs, int64_t num_rows_padded,
                                     int32_t num_q_heads, int32_t num_k_heads, int32_t head_dim,
                                     const int32_t* rope_grid, int32_t sec_t, int32_t sec_h, int32_t sec_w,
                                     float rope_theta, float eps, int32_t rope_mode, const int32_t* pos_offset,
                                     void* stream)
{
    bool empty = false;
    dit_status st = check_packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded, &empty);
    if (st != DIT_OK)
        return st;
    if (num_q_heads < 0 || num_k_heads < 0 || head_dim <= 0)
        return DIT_ERR_SHAPE;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return DIT_ERR_UNSUPPORTED;
    if (rope_mode != DIT_ROPE_INTERLEAVED && rope_mode != DIT_ROPE_HALF && rope_mode != DIT_ROPE_NONE)
        return DIT_ERR_UNSUPPORTED;
    if (q_row_stride < (int64_t)num_q_heads * head_dim || k_row_stride < (int64_t)num_k_heads * head_dim)
        return DIT_ERR_SHAPE;
    if (!(rope_theta > 0.f) || !(eps >= 0.f) || !std::isfinite(rope_theta) || !std::isfinite(eps))
        return DIT_ERR_SHAPE;
    if (rope_grid && rope_mode != DIT_ROPE_NONE) {
        if (sec_t < 0 || sec_h < 0 || sec_w < 0 || (sec_t | sec_h | sec_w) & 1 ||
            (int64_t)sec_t + sec_h + sec_w != head_dim)
            return DIT_ERR_SHAPE;
    }
    if (empty || num_q_heads + num_k_heads == 0)
        return DIT_OK;
    if (!q || !k || !q_weight || !k_weight)
        return DIT_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_weight) || !aligned16(k_weight) ||
        !mult8(q_row_stride) || !mult8(k_row_stride) ||
        (rope_grid && (reinterpret_cast<uintptr_t>(rope_grid) & 3u)) ||
        (pos_offset && (reinterpret_cast<uintptr_t>(pos_offset) & 3u)))
        return DIT_ERR_ALIGN;

    dit::QkParams p{};
    p.q = static_cast<uint16_t*>(q);
    p.k = static_cast<uint16_t*>(k);
    p.q_weight = static_cast<const uint16_t*>(q_weight);
    p.k_weight = static_cast<const uint16_t*>(k_weight);
    p.rope_grid = rope_mode == DIT_ROPE_NONE ? nullptr : rope_grid;
    p.pos_offset = rope_mode == DIT_ROPE_NONE ? nullptr : pos_offset;
    p.q_row_stride = q_row_stride;
    p.k_row_stride = k_row_stride;
    p.pk = packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded);
    p.num_q_heads = num_q_heads;
    p.num_k_heads = num_k_heads;
    p.eps = eps;
    rope_bases(p, rope_theta, head_dim, sec_t, sec_h, sec_w, p.rope_grid != nullptr);
    return from_cuda(dit::launch_qk_rmsnorm_rope(p, head_dim, rope_mode, static_cast<cudaStream_t>(stream)));
}

dit_status dit_adaln_modulate(const void* x, int64_t x_row_stride, void* out, int64_t out_row_stride,
                              const void* shift, const void* scale, int64_t mod_seq_stride,
                              const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                              int32_t num_seqs, int64_t num_rows_padded, int32_t hidden, float eps,
                              void* stream)
{
    return dit_adaln_modulate_ex(x, x_row_stride, out, out_row_stride, shift, scale, mod_seq_stride, cu_seqlens,
                                 cu_seqlens_padded, num_seqs, num_rows_padded, hidden, eps, DIT_DTYPE_BF16,
                                 stream);
}

dit_status dit_adaln_modulate_ex(const void* x, int64_t x_row_stride, void* out, int64_t out_row_stride,
                                 const void* shift, const void* scale, int64_t mod_seq_stride,
                                 const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                                 int32_t num_seqs, int64_t num_rows_padded, int32_t hidden, float eps,
                                 int32_t mod_dtype, void* stream)
{
    if (!known_dtype(mod_dtype))
        return DIT_ERR_UNSUPPORTED;
    const bool f32 = mod_dtype == DIT_DTYPE_F32;
    bool empty = false;
    dit_status st = check_packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded, &empty);
    if (st != DIT_OK)
        return st;
    if (hidden <= 0 || x_row_stride < hidden || out_row_stride < hidden || mod_seq_stride < 0 ||
        !(eps >= 0.f) || !std::isfinite(eps))
        return DIT_ERR_SHAPE;
    if (hidden > dit::kMaxAdalnHidden)
        return DIT_ERR_UNSUPPORTED;
    if (empty)
        return DIT_OK;
    if (!x || !out || !shift || !scale)
        return DIT_ERR_NULL;
    if (!aligned16(x) || !aligned16(out) || !aligned16(shift) || !aligned16(scale) || !mult8(hidden) ||
        !mult8(x_row_stride) || !mult8(out_row_stride) || !mod_stride_ok(mod_seq_stride, f32))
        return DIT_ERR_ALIGN;
    dit::AdalnParams p{static_cast<const uint16_t*>(x), static_cast<uint16_t*>(out), shift, scale,
                       x_row_stride, out_row_stride, mod_seq_stride,
                       packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded), hidden, eps,
                       f32 ? 1 : 0};
    return from_cuda(dit::launch_adaln_modulate(p, static_cast<cudaStream_t>(stream)));
}

dit_status dit_gated_residual(const void* x, int64_t x_row_stride, const void* y, int64_t y_row_stride,
                              const void* gate, int64_t gate_seq_stride, void* out, int64_t out_row_stride,
                              const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                              int32_t num_seqs, int64_t num_rows_padded, int32_t hidden, void* stream)
{
    return dit_gated_residual_ex(x, x_row_stride, y, y_row_stride, gate, gate_seq_stride, out, out_row_stride,
                                 cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded, hidden, DIT_DTYPE_BF16,
                                 stream);
}

dit_status dit_gated_residual_ex(const void* x, int64_t x_row_stride, const void* y, int64_t y_row_stride,
                                 const void* gate, int64_t gate_seq_stride, void* out, int64_t out_row_stride,
                                 const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                                 int32_t num_seqs, int64_t num_rows_padded, int32_t hidden, int32_t gate_dtype,
                                 void* stream)
{
    if (!known_dtype(gate_dtype))
        return DIT_ERR_UNSUPPORTED;
    const bool f32 = gate_dtype == DIT_DTYPE_F32;
    bool empty = false;
    dit_status st = check_packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded, &empty);
    if (st != DIT_OK)
        return st;
    if (hidden <= 0 || x_row_stride < hidden || y_row_stride < hidden || out_row_stride < hidden ||
        gate_seq_stride < 0)
        return DIT_ERR_SHAPE;
    if (empty)
        return DIT_OK;
    if (!x || !y || !gate || !out)
        return DIT_ERR_NULL;
    if (!aligned16(x) || !aligned16(y) || !aligned16(gate) || !aligned16(out) || !mult8(hidden) ||
        !mult8(x_row_stride) || !mult8(y_row_stride) || !mult8(out_row_stride) ||
        !mod_stride_ok(gate_seq_stride, f32))
        return DIT_ERR_ALIGN;
    dit::GatedParams p{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(y), gate,
                       static_cast<uint16_t*>(out), x_row_stride, y_row_stride, gate_seq_stride, out_row_stride,
                       packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded), hidden, f32 ? 1 : 0};
    return from_cuda(dit::launch_gated_residual(p, static_cast<cudaStream_t>(stream)));
}

dit_status dit_gated_residual_adaln(const void* x, int64_t x_row_stride, const void* y, int64_t y_row_stride,
                                    const void* gate, int64_t gate_seq_stride,
                                    const void* shift, const void* scale, int64_t mod_seq_stride,
                                    void* res_out, int64_t res_row_stride, void* norm_out, int64_t norm_row_stride,
                                    const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                                    int32_t num_seqs, int64_t num_rows_padded, int32_t hidden, float eps,
                                    void* stream)
{
    return dit_gated_residual_adaln_ex(x, x_row_stride, y, y_row_stride, gate, gate_seq_stride, shift, scale,
                                       mod_seq_stride, res_out, res_row_stride, norm_out, norm_row_stride,
                                       cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded, hidden, eps,
                                       DIT_DTYPE_BF16, stream);
}

dit_status dit_gated_residual_adaln_ex(const void* x, int64_t x_row_stride, const void* y, int64_t y_row_stride,
                                       const void* gate, int64_t gate_seq_stride,
                                       const void* shift, const void* scale, int64_t mod_seq_stride,
                                       void* res_out, int64_t res_row_stride, void* norm_out,
                                       int64_t norm_row_stride, const int32_t* cu_seqlens,
                                       const int32_t* cu_seqlens_padded, int32_t num_seqs,
                                       int64_t num_rows_padded, int32_t hidden, float eps, int32_t mod_dtype,
                                       void* stream)
{
    if (!known_dtype(mod_dtype))
        return DIT_ERR_UNSUPPORTED;
    const bool f32 = mod_dtype == DIT_DTYPE_F32;
    bool empty = false;
    dit_status st = check_packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded, &empty);
    if (st != DIT_OK)
        return st;
    if (hidden <= 0 || x_row_stride < hidden || y_row_stride < hidden || res_row_stride < hidden ||
        norm_row_stride < hidden || gate_seq_stride < 0 || mod_seq_stride < 0 || !(eps >= 0.f) ||
        !std::isfinite(eps))
        return DIT_ERR_SHAPE;
    if (hidden > dit::kMaxAdalnHidden)
        return DIT_ERR_UNSUPPORTED;
    if (empty)
        return DIT_OK;
    if (!x || !y || !gate || !shift || !scale || !res_out || !norm_out)
        return DIT_ERR_NULL;
    if (!aligned16(x) || !aligned16(y) || !aligned16(gate) || !aligned16(shift) || !aligned16(scale) ||
        !aligned16(res_out) || !aligned16(norm_out) || !mult8(hidden) || !mult8(x_row_stride) ||
        !mult8(y_row_stride) || !mult8(res_row_stride) || !mult8(norm_row_stride) ||
        !mod_stride_ok(gate_seq_stride, f32) || !mod_stride_ok(mod_seq_stride, f32))
        return DIT_ERR_ALIGN;
    dit::FusedParams p{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(y), gate, shift, scale,
                       static_cast<uint16_t*>(res_out), static_cast<uint16_t*>(norm_out), x_row_stride,
                       y_row_stride, gate_seq_stride, mod_seq_stride, res_row_stride, norm_row_stride,
                       packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded), hidden, eps,
                       f32 ? 1 : 0};
    return from_cuda(dit::launch_gated_residual_adaln(p, static_cast<cudaStream_t>(stream)));
}

dit_status dit_swiglu(const void* a, int64_t a_row_stride, const void* b, int64_t b_row_stride,
                      void* out, int64_t out_row_stride,
                      const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                      int32_t num_seqs, int64_t num_rows_padded, int32_t inner, void* stream)
{
    bool empty = false;
    dit_status st = check_packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded, &empty);
    if (st != DIT_OK)
        return st;
    if (inner <= 0 || a_row_stride < inner || b_row_stride < inner || out_row_stride < inner)
        return DIT_ERR_SHAPE;
    if (empty)
        return DIT_OK;
    if (!a || !b || !out)
        return DIT_ERR_NULL;
    if (!aligned16(a) || !aligned16(b) || !aligned16(out) || !mult8(inner) || !mult8(a_row_stride) ||
        !mult8(b_row_stride) || !mult8(out_row_stride))
        return DIT_ERR_ALIGN;
    dit::SwigluParams p{static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(b),
                        static_cast<uint16_t*>(out), a_row_stride, b_row_stride, out_row_stride,
                        packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded), inner};
    return from_cuda(dit::launch_swiglu(p, static_cast<cudaStream_t>(stream)));
}

dit_status dit_frames_to_u8(const float* x, int64_t batch, int64_t channels, int64_t frames, int64_t height,
                            int64_t width, int32_t layout, uint8_t* out, void* stream)
{
    if (batch < 0 || channels < 0 || frames < 0 || height < 0 || width < 0)
        return DIT_ERR_SHAPE;
    if (layout != DIT_FRAMES_BTHWC && layout != DIT_FRAMES_BTCHW)
        return DIT_ERR_UNSUPPORTED;
    if (batch == 0 || channels == 0 || frames == 0 || height == 0 || width == 0)
        return DIT_OK;
    const double total = (double)batch * channels * frames * height * width;
    if (total > 9.0e15)
        return DIT_ERR_SHAPE;
    if (!x || !out)
        return DIT_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(x) & 3u)
        return DIT_ERR_ALIGN;
    dit::FramesParams p{x, out, batch, channels, frames, height, width, layout};
    return from_cuda(dit::launch_frames_to_u8(p, static_cast<cudaStream_t>(stream)));
}

dit_status dit_validate_seqlens(const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                                int32_t num_seqs, int64_t num_rows_padded, int32_t* flag, void* stream)
{
    if (num_seqs < 0 || num_rows_padded < 0 || num_rows_padded > INT32_MAX)
        return DIT_ERR_SHAPE;
    if (!cu_seqlens || !cu_seqlens_padded || !flag)
        return DIT_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) || (reinterpret_cast<uintptr_t>(cu_seqlens_padded) & 3u) ||
        (reinterpret_cast<uintptr_t>(flag) & 3u))
        return DIT_ERR_ALIGN;
    dit::Packing pk = packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded);
    return from_cuda(dit::launch_validate_seqlens(pk, num_rows_padded, flag, static_cast<cudaStream_t>(stream)));
}

dit_status dit_av_stream_seqlens(const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                                 const int32_t* rope_grid, const int32_t* pos_offset, int32_t num_seqs,
                                 int32_t* out_cu_seqlens, int32_t* out_cu_seqlens_padded, void* stream)
{
    if (num_seqs < 0 || num_seqs > (INT32_MAX - 1) / 2)
        return DIT_ERR_SHAPE;
    if (!cu_seqlens || !cu_seqlens_padded || !out_cu_seqlens || !out_cu_seqlens_padded ||
        (num_seqs > 0 && !rope_grid))
        return DIT_ERR_NULL;
    const uintptr_t any = reinterpret_cast<uintptr_t>(cu_seqlens) | reinterpret_cast<uintptr_t>(cu_seqlens_padded) |
                          reinterpret_cast<uintptr_t>(rope_grid) | reinterpret_cast<uintptr_t>(pos_offset) |
                          reinterpret_cast<uintptr_t>(out_cu_seqlens) |
                          reinterpret_cast<uintptr_t>(out_cu_seqlens_padded);
    if (any & 3u)
        return DIT_ERR_ALIGN;
    return from_cuda(dit::launch_av_stream_seqlens(cu_seqlens, cu_seqlens_padded, rope_grid, pos_offset, num_seqs,
                                                   out_cu_seqlens, out_cu_seqlens_padded,
                                                   static_cast<cudaStream_t>(stream)));
}

dit_status dit_rope_frequencies(int32_t rotary_dim, double theta, int32_t scaling, double factor,
                                int64_t original_len, double beta_fast, double beta_slow, double* freqs,
                                float* attn_scale)
{
    if (rotary_dim <= 0 || (rotary_dim & 1) || !(theta > 0.0) || !std::isfinite(theta))
        return DIT_ERR_SHAPE;
    if (scaling < DIT_ROPE_SCALE_NONE || scaling > DIT_ROPE_SCALE_YARN)
        return DIT_ERR_UNSUPPORTED;
    if (scaling != DIT_ROPE_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
        return DIT_ERR_SHAPE;
    if (scaling == DIT_ROPE_SCALE_YARN &&
        (original_len <= 0 || !(theta > 1.0) || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) ||
         !std::isfinite(beta_fast)))
        return DIT_ERR_SHAPE;
    if (!freqs || !attn_scale)
        return DIT_ERR_NULL;
    const double R = rotary_dim;
    double base = theta, lo = 0.0, hi = 0.0;
    if (scaling == DIT_ROPE_SCALE_NTK && rotary_dim > 2)
        base = theta * std::pow(factor, R / (R - 2.0));
    if (scaling == DIT_ROPE_SCALE_YARN) {
        constexpr double kTwoPi = 6.283185307179586476925286766559;
        auto pair_at = [&](double turns) {
            return R * std::log((double)original_len / (kTwoPi * turns)) / (2.0 * std::log(theta));
        };
        lo = std::fmax(std::floor(pair_at(beta_fast)), 0.0);
        hi = std::fmin(std::ceil(pair_at(beta_slow)), R - 1.0);
    }
    for (int32_t j = 0; j < rotary_dim / 2; ++j) {
        double f = std::pow(base, -2.0 * j / R);
        if (scaling == DIT_ROPE_SCALE_LINEAR)
            f /= factor;
        if (scaling == DIT_ROPE_SCALE_YARN) {
            const double r = std::fmin(std::fmax((j - lo) / std::fmax(hi - lo, 0.001), 0.0), 1.0);
            f = f / factor * r + f * (1.0 - r);
        }
        freqs[j] = f;
    }
    *attn_scale = scaling == DIT_ROPE_SCALE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return DIT_OK;
}

dit_status dit_qk_rope_scaled(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, void* q_out,
                              int64_t q_out_stride, void* k_out, int64_t k_out_stride, const void* q_weight,
                              const void* k_weight, const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                              int32_t num_seqs, int64_t num_rows_padded, int32_t num_q_heads, int32_t num_k_heads,
                              int32_t head_dim, const double* freqs, int32_t rotary_dim, const int32_t* rope_grid,
                              const double* grid_freqs, int32_t sec_t, int32_t sec_h, int32_t sec_w,
                              const int32_t* pos_offset, float attn_scale, float eps, int32_t rope_mode, void* stream)
{
    bool empty = false;
    dit_status st = check_packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded, &empty);
    if (st != DIT_OK)
        return st;
    st = check_rope_table(num_q_heads, num_k_heads, head_dim, rotary_dim, rope_grid, sec_t, sec_h, sec_w, attn_scale,
                          eps, rope_mode);
    if (st != DIT_OK)
        return st;
    if (!q_out)
        q_out_stride = q_row_stride;
    if (!k_out)
        k_out_stride = k_row_stride;
    const int64_t qw = (int64_t)num_q_heads * head_dim, kw = (int64_t)num_k_heads * head_dim;
    if (q_row_stride < qw || q_out_stride < qw || k_row_stride < kw || k_out_stride < kw)
        return DIT_ERR_SHAPE;
    if (empty || num_q_heads + num_k_heads == 0)
        return DIT_OK;
    const bool turns = rope_mode != DIT_ROPE_NONE;
    if ((num_q_heads > 0 && !q) || (num_k_heads > 0 && !k) || (q_weight == nullptr) != (k_weight == nullptr) ||
        (turns && !freqs) || (turns && rope_grid && !grid_freqs))
        return DIT_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(q_weight) ||
        !aligned16(k_weight) || !aligned16(freqs) || !aligned16(grid_freqs) || !mult8(q_row_stride) ||
        !mult8(k_row_stride) || !mult8(q_out_stride) || !mult8(k_out_stride) || !aligned4(rope_grid) ||
        !aligned4(pos_offset))
        return DIT_ERR_ALIGN;
    dit::RopeCacheParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.q_out = static_cast<uint16_t*>(q_out ? q_out : const_cast<void*>(q));
    p.k_out = static_cast<uint16_t*>(k_out ? k_out : const_cast<void*>(k));
    p.q_weight = static_cast<const uint16_t*>(q_weight);
    p.k_weight = static_cast<const uint16_t*>(k_weight);
    p.q_row_stride = q_row_stride;
    p.k_row_stride = k_row_stride;
    p.q_out_stride = q_out_stride;
    p.k_out_stride = k_out_stride;
    p.pk = packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded);
    p.num_q_heads = num_q_heads;
    p.num_k_heads = num_k_heads;
    p.eps = eps;
    p.attn_scale = attn_scale;
    set_rope_table(p, freqs, grid_freqs, rotary_dim, rope_grid, pos_offset, sec_t, sec_h, rope_mode);
    return from_cuda(dit::launch_rope_cache(p, head_dim, rope_mode, static_cast<cudaStream_t>(stream)));
}

dit_status dit_qkv_rope_append(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                               const void* v, int64_t v_row_stride, void* q_out, int64_t q_out_stride,
                               const void* q_weight, const void* k_weight, void* k_cache, void* v_cache,
                               int64_t page_stride, int64_t slot_stride, int64_t head_stride, int32_t num_pages,
                               int32_t page_size, const int32_t* block_table, int64_t table_stride, int32_t max_pages,
                               const int32_t* cache_lens, const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                               int32_t num_seqs, int64_t num_rows_padded, int32_t num_q_heads, int32_t num_kv_heads,
                               int32_t head_dim, const double* freqs, int32_t rotary_dim, const int32_t* rope_grid,
                               const double* grid_freqs, int32_t sec_t, int32_t sec_h, int32_t sec_w,
                               const int32_t* pos_offset, float attn_scale, float eps, int32_t rope_mode, void* stream)
{
    bool empty = false;
    dit_status st = check_packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded, &empty);
    if (st != DIT_OK)
        return st;
    st = check_rope_table(num_q_heads, num_kv_heads, head_dim, rotary_dim, rope_grid, sec_t, sec_h, sec_w, attn_scale,
                          eps, rope_mode);
    if (st != DIT_OK)
        return st;
    if (!q_out)
        q_out_stride = q_row_stride;
    const int64_t qw = (int64_t)num_q_heads * head_dim, kw = (int64_t)num_kv_heads * head_dim;
    if (num_kv_heads <= 0 || q_row_stride < qw || q_out_stride < qw || k_row_stride < kw || v_row_stride < kw)
        return DIT_ERR_SHAPE;
    st = check_cache(head_dim, page_stride, slot_stride, head_stride, num_pages, page_size, table_stride, max_pages);
    if (st != DIT_OK)
        return st;
    if (empty)
        return DIT_OK;
    const bool turns = rope_mode != DIT_ROPE_NONE;
    if ((num_q_heads > 0 && !q) || !k || !v || (q_weight == nullptr) != (k_weight == nullptr) || !k_cache ||
        !v_cache || !block_table || !cache_lens || (turns && !freqs) || (turns && rope_grid && !grid_freqs))
        return DIT_ERR_NULL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(q_weight) ||
        !aligned16(k_weight) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(freqs) ||
        !aligned16(grid_freqs) || !mult8(q_row_stride) || !mult8(k_row_stride) || !mult8(v_row_stride) ||
        !mult8(q_out_stride) || !aligned4(rope_grid) || !aligned4(pos_offset) || !aligned4(block_table) ||
        !aligned4(cache_lens))
        return DIT_ERR_ALIGN;
    dit::RopeCacheParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.q_out = static_cast<uint16_t*>(q_out ? q_out : const_cast<void*>(q));
    p.k_cache = static_cast<uint16_t*>(k_cache);
    p.v_cache = static_cast<uint16_t*>(v_cache);
    p.q_weight = static_cast<const uint16_t*>(q_weight);
    p.k_weight = static_cast<const uint16_t*>(k_weight);
    p.block_table = block_table;
    p.cache_lens = cache_lens;
    p.q_row_stride = q_row_stride;
    p.k_row_stride = k_row_stride;
    p.v_row_stride = v_row_stride;
    p.q_out_stride = q_out_stride;
    p.page_stride = page_stride;
    p.slot_stride = slot_stride;
    p.head_stride = head_stride;
    p.table_stride = table_stride;
    p.pk = packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded);
    p.num_q_heads = num_q_heads;
    p.num_k_heads = num_kv_heads;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.max_pages = max_pages;
    p.eps = eps;
    p.attn_scale = attn_scale;
    set_rope_table(p, freqs, grid_freqs, rotary_dim, rope_grid, pos_offset, sec_t, sec_h, rope_mode);
    return from_cuda(dit::launch_rope_cache(p, head_dim, rope_mode, static_cast<cudaStream_t>(stream)));
}

dit_status dit_paged_attention_workspace(int64_t num_rows_padded, int32_t num_seqs, int32_t num_q_heads,
                                         int32_t num_kv_heads, int32_t head_dim, int64_t max_chunk,
                                         int64_t max_kv_len, int64_t* bytes)
{
    if (num_seqs < 0 || num_rows_padded < 0 || num_rows_padded > INT32_MAX || num_q_heads <= 0 || num_kv_heads <= 0 ||
        num_q_heads % num_kv_heads != 0 || max_kv_len <= 0 || max_kv_len > INT32_MAX || head_dim <= 0)
        return DIT_ERR_SHAPE;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || num_kv_heads > dit::kMaxKvHeads)
        return DIT_ERR_UNSUPPORTED;
    if (!bytes)
        return DIT_ERR_NULL;
    *bytes = 0;
    if (num_seqs == 0 || num_rows_padded == 0)
        return DIT_OK;
    dit::PagedPlan plan{};
    // whatever the cache's strides let it take
    for (const bool regular : {false, true}) {
        if (!dit::paged_plan(num_rows_padded, num_seqs, num_q_heads, num_kv_heads, head_dim, max_chunk, max_kv_len, 0,
                             regular, plan))
            return DIT_ERR_SHAPE;
        *bytes = plan.most_bytes > *bytes ? plan.most_bytes : *bytes;
    }
    return DIT_OK;
}

dit_status dit_paged_attention(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache,
                               int64_t page_stride, int64_t slot_stride, int64_t head_stride, int32_t num_pages,
                               int32_t page_size, const int32_t* block_table, int64_t table_stride, int32_t max_pages,
                               const int32_t* kv_lens, const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded,
                               int32_t num_seqs, int64_t num_rows_padded, int32_t num_q_heads, int32_t num_kv_heads,
                               int32_t head_dim, float softmax_scale, int32_t causal, int32_t window,
                               int64_t max_chunk, int64_t max_kv_len, void* out, int64_t out_row_stride, float* lse,
                               void* workspace, int64_t workspace_bytes, void* stream)
{
    bool empty = false;
    dit_status st = check_packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded, &empty);
    if (st != DIT_OK)
        return st;
    if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 || head_dim <= 0 ||
        !(softmax_scale > 0.f) || !std::isfinite(softmax_scale) || window < 0 || workspace_bytes < 0 ||
        q_row_stride < (int64_t)num_q_heads * head_dim || out_row_stride < (int64_t)num_q_heads * head_dim)
        return DIT_ERR_SHAPE;
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || num_kv_heads > dit::kMaxKvHeads)
        return DIT_ERR_UNSUPPORTED;
    st = check_cache(head_dim, page_stride, slot_stride, head_stride, num_pages, page_size, table_stride, max_pages);
    if (st != DIT_OK)
        return st;
    if (empty)
        return DIT_OK;
    if (!q || !k_cache || !v_cache || !block_table || !kv_lens || !out)
        return DIT_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(workspace) ||
        !mult8(q_row_stride) || !mult8(out_row_stride) || !aligned4(block_table) || !aligned4(kv_lens) ||
        !aligned4(lse))
        return DIT_ERR_ALIGN;
    const int64_t capacity = (int64_t)max_pages * page_size;
    if (capacity > INT32_MAX - 4096)  // key numbers, a tile beyond the last, are 32-bit
        return DIT_ERR_UNSUPPORTED;
    int64_t keys = max_kv_len > 0 && max_kv_len < capacity ? max_kv_len : capacity;
    keys = keys < 1 ? 1 : (keys > INT32_MAX ? INT32_MAX : keys);
    dit::PagedPlan plan{};
    dit::CacheRows as_rows;
    const bool regular = dit::cache_rows(page_stride, slot_stride, head_stride, num_pages, page_size, num_kv_heads,
                                         head_dim, as_rows);
    if (!dit::paged_plan(num_rows_padded, num_seqs, num_q_heads, num_kv_heads, head_dim, max_chunk, keys, window,
                         regular, plan))
        return DIT_ERR_SHAPE;
    if (plan.bytes > workspace_bytes)
        return DIT_ERR_SHAPE;
    if (plan.bytes > 0 && !workspace)
        return DIT_ERR_NULL;
    dit::PagedParams p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k_cache = static_cast<const uint16_t*>(k_cache);
    p.v_cache = static_cast<const uint16_t*>(v_cache);
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.block_table = block_table;
    p.kv_lens = kv_lens;
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) +
                                          plan.part_rows * head_dim * 4);
    p.q_row_stride = q_row_stride;
    p.out_row_stride = out_row_stride;
    p.page_stride = page_stride;
    p.slot_stride = slot_stride;
    p.head_stride = head_stride;
    p.table_stride = table_stride;
    p.pk = packing(cu_seqlens, cu_seqlens_padded, num_seqs, num_rows_padded);
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.num_pages = num_pages;
    p.page_size = page_size;
    p.max_pages = max_pages;
    // key / page_size = key * ceil(2^s / page_size) >> s with 2^(s - 31) >= page_size:
    // exact for keys below 2^31
    uint32_t log2_up = 0;
    while ((1ull << log2_up) < (uint64_t)page_size)
        ++log2_up;
    p.page_shift = 31 + log2_up;
    p.page_mul = (uint32_t)(((1ull << p.page_shift) + (uint64_t)page_size - 1) / (uint64_t)page_size);
    constexpr float kLog2e = 1.4426950408889634f;
    p.scale_log2 = softmax_scale * kLog2e;
    p.causal = causal != 0;
    p.window = window;
    p.splits = plan.splits;
    p.split_keys = plan.split_keys;
    return from_cuda(dit::launch_paged_attention(p, plan, head_dim, static_cast<cudaStream_t>(stream)));
}

const char* dit_status_string(dit_status s)
{
    switch (s) {
    case DIT_OK: return "DIT_OK";
    case DIT_ERR_NULL: return "DIT_ERR_NULL: a required pointer is NULL";
    case DIT_ERR_SHAPE: return "DIT_ERR_SHAPE: invalid size, stride or rope sections";
    case DIT_ERR_ALIGN: return "DIT_ERR_ALIGN: pointer not 16-byte aligned or size/stride not a multiple of 8";
    case DIT_ERR_UNSUPPORTED: return "DIT_ERR_UNSUPPORTED: unsupported head_dim or hidden size";
    case DIT_ERR_SEQLENS: return "DIT_ERR_SEQLENS: malformed cu_seqlens / cu_seqlens_padded";
    case DIT_ERR_CUDA: return "DIT_ERR_CUDA: kernel launch failed";
    default: return "unknown dit_status";
    }
}

int32_t dit_last_cuda_error(void) { return g_last_cuda_error; }

int32_t dit_abi_version(void) { return DIT_ABI_VERSION; }

}  // extern "C"
