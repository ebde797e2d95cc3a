/*
 * rows_api.cu — the C ABI of the operators on single heads of single tokens: attn_qk_norm_rope and
 * its gradient, attn_append_paged and attn_append_paged_fp8 (attn.h). Argument checks and launches;
 * none of them allocates or keeps anything between calls.
 */
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "attn.h"
#include "kernels.h"

namespace attn_b200 {

// The workspace that callers size by the macro holds a partial of both weights' gradients for every block.
static_assert(ATTN_QK_NORM_ROPE_BWD_WORKSPACE(128) == kNormRopeBwdBlocks * 2u * 128u * sizeof(float), "workspace of the gradient");

namespace {

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// {batch, head, row} element strides, as attn_fwd_strided takes them.
bool read_strides(const long long *s, TensorStrides *out)
{
    for (int i = 0; i < 3; ++i)
        if (s[i] < 1 || s[i] % 8 != 0 || s[i] >= (1LL << 38))
            return false;
    *out = TensorStrides{s[0], s[1], s[2]};
    return true;
}

// The norm's and the rotation's arguments.
int check_row_args(const void *q_weight, const void *k_weight, const float *cos, const float *sin, int D, int rot_dim,
                   int max_pos, int interleaved, float eps)
{
    if (interleaved != 0 && interleaved != 1)
        return ATTN_ERR_SHAPE;
    if (rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0 || (rot_dim > 0 && max_pos < 1))
        return ATTN_ERR_ROTATION;
    if (rot_dim > 0 && (!cos || !sin))
        return ATTN_ERR_NULL;
    if (!aligned(q_weight, 16) || !aligned(k_weight, 16) || (rot_dim > 0 && (!aligned(cos, 16) || !aligned(sin, 16))))
        return ATTN_ERR_ALIGN;
    if (!(eps >= 0.f) || !std::isfinite(eps))
        return ATTN_ERR_EPS;
    return ATTN_OK;
}

int norm_rope(const void *q, const void *k, const void *q_weight, const void *k_weight, const float *cos,
              const float *sin, const int *positions, const void *dq_out, const void *dk_out, void *q_to, void *k_to,
              float *dq_weight, float *dk_weight, void *workspace, int B, int Hq, int Hkv, int S, int D,
              const long long *const (&strides)[6], int rot_dim, int max_pos, int interleaved, float eps, bool backward,
              void *stream)
{
    // Without a norm the gradient does not need the inputs.
    const bool norm = q_weight != nullptr;
    if (!q_to || !k_to || ((!backward || norm) && (!q || !k)) || (backward && (!dq_out || !dk_out)))
        return ATTN_ERR_NULL;
    if (norm != (k_weight != nullptr) || (!norm && (dq_weight || dk_weight)))
        return ATTN_ERR_NULL;
    const bool want_dw = dq_weight || dk_weight;
    if (want_dw && !workspace)
        return ATTN_ERR_NULL;
    const bool uses[6] = {q != nullptr, k != nullptr, backward, backward, true, true};
    for (int i = 0; i < 6; ++i)
        if (!strides[i] && uses[i])
            return ATTN_ERR_NULL;
    if (B < 1 || Hq < 1 || Hkv < 1 || S < 1 || D < 1)
        return ATTN_ERR_SHAPE;
    if (D != 32 && D != 64 && D != 128)
        return ATTN_ERR_HEADDIM;
    const long long H = Hq > Hkv ? Hq : Hkv;
    if (static_cast<long long>(B) * S > kMaxHeadRows / H)
        return ATTN_ERR_SHAPE;
    const int rc = check_row_args(q_weight, k_weight, cos, sin, D, rot_dim, max_pos, interleaved, eps);
    if (rc != ATTN_OK)
        return rc;
    NormRopeArgs a;
    a.q = NormRopeSide{q, q_weight, dq_out, q_to, Hq, {}, {}, {}};
    a.k = NormRopeSide{k, k_weight, dk_out, k_to, Hkv, {}, {}, {}};
    TensorStrides *to[6] = {&a.q.xs, &a.k.xs, &a.q.zs, &a.k.zs, &a.q.os, &a.k.os};
    for (int i = 0; i < 6; ++i)
        if (strides[i] && !read_strides(strides[i], to[i]))
            return ATTN_ERR_ALIGN;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(dq_out, 16) || !aligned(dk_out, 16) || !aligned(q_to, 16) ||
        !aligned(k_to, 16) || !aligned(dq_weight, 16) || !aligned(dk_weight, 16) || !aligned(workspace, 16) ||
        !aligned(positions, 4))
        return ATTN_ERR_ALIGN;
    int sms = 0;
    const int dev = check_device(&sms);
    if (dev != ATTN_OK)
        return dev;
    a.cos = cos;
    a.sin = sin;
    a.positions = positions;
    a.B = B;
    a.S = S;
    a.D = D;
    a.rot_dim = rot_dim;
    a.max_pos = max_pos;
    a.interleaved = interleaved;
    a.eps = eps;
    a.backward = backward;
    a.sm_count = sms;
    a.partials = want_dw ? static_cast<float *>(workspace) : nullptr;
    a.dwq = dq_weight;
    a.dwk = dk_weight;
    if (launch_norm_rope(a, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_LAUNCH;
    }
    return ATTN_OK;
}

int append_paged(const void *q, const void *k, const void *v, const void *q_weight, const void *k_weight,
                 const float *cos, const float *sin, const int *positions, const int *seq_lens, const int *new_lens,
                 const int *block_table, void *q_out, void *k_pages, void *v_pages, const float *k_scale,
                 const float *v_scale, int B, int Hq, int Hkv, int Sq, const long long *q_strides,
                 const long long *k_strides, const long long *v_strides, const long long *q_out_strides, int num_pages,
                 int page_size, int pages_per_seq, int rot_dim, int max_pos, int interleaved, float eps, bool fp8,
                 void *stream)
{
    if (!k || !v || !seq_lens || !block_table || !k_pages || !v_pages || !k_strides || !v_strides ||
        (fp8 && (!k_scale || !v_scale)))
        return ATTN_ERR_NULL;
    if ((q != nullptr) != (q_out != nullptr) || (q && (!q_strides || !q_out_strides)))
        return ATTN_ERR_NULL;
    // A norm of the keys takes one of the queries with it; with no queries there is no weight for them.
    if (q ? (q_weight != nullptr) != (k_weight != nullptr) : q_weight != nullptr)
        return ATTN_ERR_NULL;
    if (B < 1 || Hkv < 1 || Sq < 1 || (q ? Hq < 1 : Hq != 0) || num_pages < 1 || pages_per_seq < 1)
        return ATTN_ERR_SHAPE;
    const bool page_ok = page_size == 16 || page_size == 32 || page_size == 64 ||
                         (page_size >= 128 && page_size % 128 == 0);
    if (!page_ok)
        return ATTN_ERR_SHAPE;
    const long long H = Hq > Hkv ? Hq : Hkv;
    if (static_cast<long long>(B) * Sq > kMaxHeadRows / H || static_cast<long long>(num_pages) * Hkv > INT_MAX ||
        static_cast<long long>(B) * pages_per_seq > INT_MAX ||
        static_cast<long long>(pages_per_seq) * page_size > INT_MAX)
        return ATTN_ERR_SHAPE;
    const int rc = check_row_args(q_weight, k_weight, cos, sin, 128, rot_dim, max_pos, interleaved, eps);
    if (rc != ATTN_OK)
        return rc;
    AppendArgs a;
    if (!read_strides(k_strides, &a.ks) || !read_strides(v_strides, &a.vs) ||
        (q && (!read_strides(q_strides, &a.qs) || !read_strides(q_out_strides, &a.qos))))
        return ATTN_ERR_ALIGN;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_pages, 16) ||
        !aligned(v_pages, 16) || !aligned(k_scale, 16) || !aligned(v_scale, 16) || !aligned(positions, 4) ||
        !aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(block_table, 4))
        return ATTN_ERR_ALIGN;
    int sms = 0;
    const int dev = check_device(&sms);
    if (dev != ATTN_OK)
        return dev;
    if (!q)
        a.qs = a.qos = TensorStrides{0, 0, 0};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.cos = cos;
    a.sin = sin;
    a.positions = positions;
    a.seq_lens = seq_lens;
    a.new_lens = new_lens;
    a.block_table = block_table;
    a.q_out = q_out;
    a.k_pages = k_pages;
    a.v_pages = v_pages;
    a.k_scale = fp8 ? k_scale : nullptr;
    a.v_scale = fp8 ? v_scale : nullptr;
    a.B = B;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.S = Sq;
    a.num_pages = num_pages;
    a.page_size = page_size;
    a.pages_per_seq = pages_per_seq;
    a.rot_dim = rot_dim;
    a.max_pos = max_pos;
    a.interleaved = interleaved;
    a.eps = eps;
    a.sm_count = sms;
    if (launch_append(a, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return ATTN_ERR_LAUNCH;
    }
    return ATTN_OK;
}

}  // namespace
}  // namespace attn_b200

using namespace attn_b200;

extern "C" int attn_qk_norm_rope(const void *q, const void *k, const void *q_weight, const void *k_weight,
                                 const float *cos, const float *sin, const int *positions, void *q_out, void *k_out,
                                 int B, int Hq, int Hkv, int S, int D, const long long *q_strides,
                                 const long long *k_strides, const long long *q_out_strides,
                                 const long long *k_out_strides, int rot_dim, int max_pos, int interleaved, float eps,
                                 void *stream)
{
    const long long *strides[6] = {q_strides, k_strides, nullptr, nullptr, q_out_strides, k_out_strides};
    return norm_rope(q, k, q_weight, k_weight, cos, sin, positions, nullptr, nullptr, q_out, k_out, nullptr, nullptr,
                     nullptr, B, Hq, Hkv, S, D, strides, rot_dim, max_pos, interleaved, eps, false, stream);
}

extern "C" int attn_qk_norm_rope_bwd(const void *q, const void *k, const void *q_weight, const void *k_weight,
                                     const float *cos, const float *sin, const int *positions, const void *dq_out,
                                     const void *dk_out, void *dq, void *dk, float *dq_weight, float *dk_weight,
                                     void *workspace, int B, int Hq, int Hkv, int S, int D, const long long *q_strides,
                                     const long long *k_strides, const long long *dq_out_strides,
                                     const long long *dk_out_strides, const long long *dq_strides,
                                     const long long *dk_strides, int rot_dim, int max_pos, int interleaved, float eps,
                                     void *stream)
{
    const long long *strides[6] = {q_strides, k_strides, dq_out_strides, dk_out_strides, dq_strides, dk_strides};
    return norm_rope(q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, dq, dk, dq_weight, dk_weight,
                     workspace, B, Hq, Hkv, S, D, strides, rot_dim, max_pos, interleaved, eps, true, stream);
}

extern "C" int attn_append_paged(const void *q, const void *k, const void *v, const void *q_weight,
                                 const void *k_weight, const float *cos, const float *sin, const int *positions,
                                 const int *seq_lens, const int *new_lens, const int *block_table, void *q_out,
                                 void *k_pages, void *v_pages, int B, int Hq, int Hkv, int Sq,
                                 const long long *q_strides, const long long *k_strides, const long long *v_strides,
                                 const long long *q_out_strides, int num_pages, int page_size, int pages_per_seq,
                                 int rot_dim, int max_pos, int interleaved, float eps, void *stream)
{
    return append_paged(q, k, v, q_weight, k_weight, cos, sin, positions, seq_lens, new_lens, block_table, q_out,
                        k_pages, v_pages, nullptr, nullptr, B, Hq, Hkv, Sq, q_strides, k_strides, v_strides,
                        q_out_strides, num_pages, page_size, pages_per_seq, rot_dim, max_pos, interleaved, eps, false,
                        stream);
}

extern "C" int attn_append_paged_fp8(const void *q, const void *k, const void *v, const void *q_weight,
                                     const void *k_weight, const float *cos, const float *sin, const int *positions,
                                     const int *seq_lens, const int *new_lens, const int *block_table, void *q_out,
                                     void *k_pages, void *v_pages, const float *k_scale, const float *v_scale, int B,
                                     int Hq, int Hkv, int Sq, const long long *q_strides, const long long *k_strides,
                                     const long long *v_strides, const long long *q_out_strides, int num_pages,
                                     int page_size, int pages_per_seq, int rot_dim, int max_pos, int interleaved,
                                     float eps, void *stream)
{
    return append_paged(q, k, v, q_weight, k_weight, cos, sin, positions, seq_lens, new_lens, block_table, q_out,
                        k_pages, v_pages, k_scale, v_scale, B, Hq, Hkv, Sq, q_strides, k_strides, v_strides,
                        q_out_strides, num_pages, page_size, pages_per_seq, rot_dim, max_pos, interleaved, eps, true,
                        stream);
}
