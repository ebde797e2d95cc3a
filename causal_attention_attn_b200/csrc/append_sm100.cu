/*
 * append_sm100.cu — new tokens' keys and values written to their slots of a paged K/V cache, the
 * keys normalised and rotated on the way, and the same tokens' queries normalised and rotated for the
 * attention that follows (attn_append_paged and attn_append_paged_fp8 in attn.h). One kernel, so a
 * decode step needs one launch between its projection and its attention.
 *
 * Row arithmetic as in norm_rope_sm100.cu. With an e4m3 cache a key or value element x is stored as
 * the code nearest to x / coefficient (ties to even, saturating at +-448), from the fp32 value: a key
 * is rounded once, not to bf16 first. Ties are as common as short coefficients are, so the quotient
 * is corrected by its remainder (quotient_codes): without it 84 of 8.4 million codes, every bf16 value over 128
 * short coefficients, fell on the wrong side of a tie. It costs 3 of 72 us for 16384 tokens.
 *
 * Bound by memory (each new row read and written once), and for a few tokens by the launch and one
 * chain of dependent loads: length, block-table entry and angles, store. The persistent blocks and
 * their rings are norm_rope_sm100.cu's; a unit's length and block-table entry are looked up when its
 * rows are sent for.
 */
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "head_row.cuh"
#include "kernels.h"

namespace attn_b200 {
namespace {

constexpr int kD = 128;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
using R = RowLanes<kD>;

enum Kind : int { kQ = 0, kK = 1, kV = 2 };

// One of q, k and v, in pairs of neighbouring heads of one token (as in norm_rope_sm100.cu).
struct Source {
    const __nv_bfloat16 *x, *w;
    TensorStrides xs;
    FastDiv pairs_per_token;
    int heads, pairs, units;
};

struct AppendParams {
    Source src[3];
    __nv_bfloat16 *q_out;
    TensorStrides qos;
    void *pages[2];         // k, v
    const float *coef[2];   // e4m3: [Hkv][128]
    RopeTable table;
    const int *positions, *seq_lens, *new_lens, *block_table;
    FastDiv seq, page_size;
    int Hkv, num_pages, pages_per_seq;
    long long cap;  // slots of a block-table row
    float eps;
};

constexpr int kStages = 3;
constexpr int kAngles = 2 * kRowSlots;  // a stage: two rows, then the angles
constexpr int kStageBytes = (kAngles + kAngleSlots) * kSlotBytes;
constexpr int kSmem = kWarps * kStages * kStageBytes;

// The e4m3 codes of x / c for two elements. With r the hardware's reciprocal of c (within a unit in the last
// place), q = x r is within three units of the quotient; its remainder x - q c is exact in one fused
// multiply-add, and q + (x - q c) r rounds once (Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990). Everything is computed negated, so that only the sign bits of the codes
// are turned at the end and zeros keep theirs; q stops at +-512, beyond every code, so that no infinity
// meets another.
__device__ __forceinline__ float negative_reciprocal(float c)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(-c));
    return r;
}

__device__ __forceinline__ uint32_t quotient_codes(float x0, float x1, float c0, float c1)
{
    const float2 x = make_float2(x0, x1), c = make_float2(c0, c1);
    const float2 r = make_float2(negative_reciprocal(c0), negative_reciprocal(c1));
    float2 q = __fmul2_rn(x, r);
    q = make_float2(fminf(fmaxf(q.x, -512.f), 512.f), fminf(fmaxf(q.y, -512.f), 512.f));
    q = __ffma2_rn(__ffma2_rn(q, c, x), r, q);
    return __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3) ^ 0x8080u;
}

template <bool kInterleaved, bool kFp8>
__global__ void __launch_bounds__(kThreads, 2) append_kernel(const AppendParams p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane & (R::kLanes - 1), group = lane / R::kLanes;
    const LaneElems le = lane_elems<kInterleaved>(l, p.table.rot);
    const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp * kStages * kStageBytes + lane * 16);
    const int n_q = p.src[kQ].units, n_qk = n_q + p.src[kK].units, n_units = n_qk + p.src[kV].units;
    const int step = gridDim.x * kWarps, first = blockIdx.x * kWarps + warp;
    auto kind_of = [&](int unit) { return unit < n_q ? kQ : unit < n_qk ? kK : kV; };

    struct At {
        bool live0, live1;  // the pair's rows exist
        bool token;         // their token has a slot and a position
        uint32_t b, i, h, slot;
        int page;
    } at[kStages];
    auto issue = [&](int unit, int s) {
        if (unit < n_units) {
            const Kind kind = kind_of(unit);
            const Source &sc = p.src[kind];
            At &a = at[s];
            const int pair = (unit - (kind == kQ ? 0 : kind == kK ? n_q : n_qk)) * R::kRows + group;
            a.live0 = pair < sc.pairs;
            const uint32_t n = a.live0 ? static_cast<uint32_t>(pair) : 0u;
            const uint32_t tok = sc.pairs_per_token.quot(n);
            a.h = 2 * (n - tok * sc.pairs_per_token.d);
            a.live1 = a.live0 && static_cast<int>(a.h) + 1 < sc.heads;
            a.b = p.seq.quot(tok);
            a.i = tok - a.b * p.seq.d;
            const uint32_t base = ring + static_cast<uint32_t>(s * kStageBytes);
            const __nv_bfloat16 *x = sc.x + (a.b * sc.xs.b + a.h * sc.xs.h + a.i * sc.xs.s);
            const int S = static_cast<int>(p.seq.d);
            // Rows of padding are not read. (Without new_lens the rows wait for no length.)
            const bool fresh = !p.new_lens || static_cast<int>(a.i) >= S - min(max(__ldg(p.new_lens + a.b), 0), S);
            copy_row(base, x, le, a.live0 && fresh);
            copy_row(base + kRowSlots * kSlotBytes, a.live1 ? x + sc.xs.h : x, le, a.live1 && fresh);
            const long long place = static_cast<long long>(__ldg(p.seq_lens + a.b)) - S + a.i;
            a.token = a.live0 && fresh && place >= 0 && place < p.cap;
            const int pos = p.positions ? __ldg(p.positions + tok) : static_cast<int>(a.token ? place : 0);
            a.token = a.token && p.table.has(pos);
            a.page = -1;
            a.slot = 0;
            if (a.token) {
                const uint32_t e = p.page_size.quot(static_cast<uint32_t>(place));
                a.slot = static_cast<uint32_t>(place) - e * p.page_size.d;
                a.page = __ldg(p.block_table + static_cast<size_t>(a.b) * p.pages_per_seq + e);
                if (kind != kV && le.rotated)
                    copy_angles(base + kAngles * kSlotBytes, p.table, pos, l);
            }
        }
        copy_commit();
    };

    // The weight of the kind that the warp is at (q, then k, then v): read once for each.
    Pairs w;
    Kind have_w = kV;
    auto consume = [&](int unit, int s) {
        const Kind kind = kind_of(unit);
        const Source &sc = p.src[kind];
        const uint32_t base = ring + static_cast<uint32_t>(s * kStageBytes);
        const At a = at[s];
        const bool write = a.token && a.page >= 0 && a.page < p.num_pages;
        const bool norm = sc.w != nullptr, turn = kind != kV && le.rotated && a.token;
        if (norm && kind != have_w) {
            w = unpack_pairs<kInterleaved>(load_row(sc.w, le));
            have_w = kind;
        }
        // Everything of the stage is read, and the row sums of both rows are taken, before anything is
        // stored: the two rows' chains then overlap.
        Pairs x[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            x[k] = unpack_pairs<kInterleaved>(read_row(base + k * kRowSlots * kSlotBytes));
        if (norm) {
            float r[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                r[k] = row_sum<kD>(pairs_dot(x[k], x[k]));
#pragma unroll
            for (int k = 0; k < 2; ++k)
                scale_pairs(x[k], rsqrtf(r[k] * (1.f / kD) + p.eps), w);
        }
        if (turn) {
            const Angles ang = read_angles(base + kAngles * kSlotBytes);
            rotate_pairs<false>(x[0], ang);
            rotate_pairs<false>(x[1], ang);
        }
        if (kind == kQ) {
            __nv_bfloat16 *out = p.q_out + (a.b * p.qos.b + a.h * p.qos.h + a.i * p.qos.s);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (k ? a.live1 : a.live0)
                    store_row(out + (k ? p.qos.h : 0), le, write ? pack_pairs<kInterleaved>(x[k]) : zero_row());
            return;
        }
        if (!write)
            return;
        const size_t dst = ((static_cast<size_t>(a.page) * p.Hkv + a.h) * p.page_size.d + a.slot) * kD;
        const size_t next_head = static_cast<size_t>(p.page_size.d) * kD;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (!(k ? a.live1 : a.live0))
                continue;
            if constexpr (kFp8) {
                const float *cf = p.coef[kind - kK] + (a.h + k) * kD;
                uint32_t codes[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {  // four elements at a time, in element order
                    const float4 f = __ldg(reinterpret_cast<const float4 *>(cf + (j < 2 ? le.e0 : le.e1) + 4 * (j & 1)));
                    float v[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int e = 4 * j + t;  // of the lane's sixteen
                        v[t] = kInterleaved ? ((e & 1) ? x[k].B[e >> 1] : x[k].A[e >> 1]) : (e < 8 ? x[k].A[e & 7] : x[k].B[e & 7]);
                    }
                    // The first element in the low byte.
                    codes[j] = quotient_codes(v[0], v[1], f.x, f.y) | (quotient_codes(v[2], v[3], f.z, f.w) << 16);
                }
                uint8_t *out = static_cast<uint8_t *>(p.pages[kind - kK]) + dst + (k ? next_head : 0);
                *reinterpret_cast<uint2 *>(out + le.e0) = make_uint2(codes[0], codes[1]);
                *reinterpret_cast<uint2 *>(out + le.e1) = make_uint2(codes[2], codes[3]);
            } else {
                store_row(static_cast<__nv_bfloat16 *>(p.pages[kind - kK]) + dst + (k ? next_head : 0), le,
                          pack_pairs<kInterleaved>(x[k]));
            }
        }
    };

    int next = first;
#pragma unroll
    for (int s = 0; s < kStages; ++s, next += step)
        issue(next, s);
    for (int unit = first; unit < n_units;) {
#pragma unroll
        for (int s = 0; s < kStages; ++s) {
            if (unit >= n_units)
                break;
            copy_wait<kStages - 1>();
            consume(unit, s);
            issue(next, s);
            unit += step;
            next += step;
        }
    }
    copy_wait<0>();
}

template <bool kInterleaved, bool kFp8>
cudaError_t launch(const AppendArgs &a, cudaStream_t stream)
{
    AppendParams p;
    const int heads[3] = {a.q ? a.Hq : 0, a.Hkv, a.Hkv};
    const void *x[3] = {a.q, a.k, a.v};
    const void *w[3] = {a.q_weight, a.k_weight, nullptr};
    const TensorStrides xs[3] = {a.qs, a.ks, a.vs};
    for (int i = 0; i < 3; ++i) {
        p.src[i].x = static_cast<const __nv_bfloat16 *>(x[i]);
        p.src[i].w = static_cast<const __nv_bfloat16 *>(w[i]);
        p.src[i].xs = xs[i];
        const int per_token = (heads[i] + 1) / 2;
        p.src[i].pairs_per_token = FastDiv(static_cast<uint32_t>(per_token > 0 ? per_token : 1));
        p.src[i].heads = heads[i];
        p.src[i].pairs = a.B * a.S * per_token;
        p.src[i].units = (p.src[i].pairs + R::kRows - 1) / R::kRows;
    }
    p.q_out = static_cast<__nv_bfloat16 *>(a.q_out);
    p.qos = a.qos;
    p.pages[0] = a.k_pages;
    p.pages[1] = a.v_pages;
    p.coef[0] = a.k_scale;
    p.coef[1] = a.v_scale;
    p.table = RopeTable{a.cos, a.sin, a.rot_dim, a.max_pos};
    p.positions = a.positions;
    p.seq_lens = a.seq_lens;
    p.new_lens = a.new_lens;
    p.block_table = a.block_table;
    p.seq = FastDiv(static_cast<uint32_t>(a.S));
    p.page_size = FastDiv(static_cast<uint32_t>(a.page_size));
    p.Hkv = a.Hkv;
    p.num_pages = a.num_pages;
    p.pages_per_seq = a.pages_per_seq;
    p.cap = static_cast<long long>(a.pages_per_seq) * a.page_size;
    p.eps = a.eps;
    // Per device, as for the other kernels: the attribute applies to the device current when it is set.
    static bool attr_set[kMaxDevices] = {};
    const int dev = current_device_index();
    if (dev < 0)
        return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        const cudaError_t e =
            cudaFuncSetAttribute(append_kernel<kInterleaved, kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess)
            return e;
        attr_set[dev] = true;
    }
    const long long units = static_cast<long long>(p.src[0].units) + p.src[1].units + p.src[2].units;
    const long long want = (units + kWarps - 1) / kWarps, most = 2LL * a.sm_count;
    append_kernel<kInterleaved, kFp8>
        <<<static_cast<unsigned>(want < most ? want : most), kThreads, kSmem, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, cudaStream_t stream)
{
    if (a.k_scale)
        return a.interleaved ? launch<true, true>(a, stream) : launch<false, true>(a, stream);
    return a.interleaved ? launch<true, false>(a, stream) : launch<false, false>(a, stream);
}

}  // namespace attn_b200
