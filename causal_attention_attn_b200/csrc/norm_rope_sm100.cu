/*
 * norm_rope_sm100.cu — the norm and position rotation of queries and keys, head by head, in one
 * pass over them, and its gradient (attn_qk_norm_rope and attn_qk_norm_rope_bwd in attn.h).
 *
 * Forward, per row x (one head of one token, D elements):
 *   r = (mean(x^2) + eps)^(-1/2),  y = x r w,  z = R(pos) y.
 * Backward, given dz:
 *   dy = R(pos)^T dz,  g = w dy,  dx = r (g - x r^2 mean(g x)),  dw = sum over rows of dy x r.
 * Without weights there is no norm: z = R x and dx = R^T dz.
 *
 * Bound by memory: forward reads and writes each row once, backward reads two and writes one, with
 * about a dozen operations an element. So the design is about bytes in flight and instructions per
 * byte: head_row.cuh has the layout of rows over lanes and the ring that keeps kStages units of every
 * warp on their way. Blocks are persistent (two per SM), their warps take every (number of warps)-th
 * unit of q, then of k. The weight's gradient stays in registers over all units of a warp, then
 * goes through shared memory to one partial per block; a second small kernel adds the partials in a
 * fixed order, so the result does not depend on timing (no atomics).
 */
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "head_row.cuh"
#include "kernels.h"

namespace attn_b200 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// One of q and k. A pair is two neighbouring heads of one token (the second may be missing), numbered
// token * ceil(H / 2) + pair, token = b * S + i; a unit is the kRows pairs that a warp takes at once.
struct Side {
    const __nv_bfloat16 *x, *w, *dz;
    __nv_bfloat16 *out;  // z, or dx
    TensorStrides xs, zs, os;
    FastDiv pairs_per_token;
    int heads, pairs, units;
};

struct NormRopeParams {
    Side side[2];  // q, k
    RopeTable table;
    const int *positions;  // [B][S], or null: the row index
    FastDiv seq;           // S
    float eps;
    float *partials;  // backward: [block][2][D]
};

// A lane's place: one pair of rows.
struct PairAt {
    bool live0, live1;  // the pair's rows exist
    bool has;           // their position has angles (or there is no rotation)
    uint32_t b, i, h;
    __device__ __forceinline__ long long offset(const TensorStrides &s) const { return b * s.b + h * s.h + i * s.s; }
};

__device__ __forceinline__ PairAt locate_pair(const Side &sd, const FastDiv &seq, int pair, uint32_t *tok)
{
    PairAt r;
    r.live0 = pair < sd.pairs;
    const uint32_t n = r.live0 ? static_cast<uint32_t>(pair) : 0u;
    *tok = sd.pairs_per_token.quot(n);
    r.h = 2 * (n - *tok * sd.pairs_per_token.d);
    r.live1 = r.live0 && static_cast<int>(r.h) + 1 < sd.heads;
    r.b = seq.quot(*tok);
    r.i = *tok - r.b * seq.d;
    return r;
}

template <bool kBackward>
struct Ring {
    // Forward: 3 stages of 4 KB a warp; backward (x and dz): 2 of 6 KB. Either way 96 KB of shared
    // memory a block, two blocks an SM, and 96 to 128 KB of rows in flight on each SM.
    static constexpr int kStages = kBackward ? 2 : 3;
    static constexpr int kX = 0, kDz = 2 * kRowSlots;
    static constexpr int kAngles = kBackward ? 4 * kRowSlots : 2 * kRowSlots;
    static constexpr int kStageBytes = (kAngles + kAngleSlots) * kSlotBytes;
    static constexpr int kBytes = kWarps * kStages * kStageBytes;
};

template <int D, bool kInterleaved, bool kBackward>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_kernel(const NormRopeParams p)
{
    using R = RowLanes<D>;
    using G = Ring<kBackward>;
    extern __shared__ __align__(16) uint8_t smem[];
    if (kBackward)
        asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane & (R::kLanes - 1), group = lane / R::kLanes;
    const LaneElems le = lane_elems<kInterleaved>(l, p.table.rot);
    const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp * G::kStages * G::kStageBytes + lane * 16);
    const int n_q = p.side[0].units, n_units = n_q + p.side[1].units;
    const int step = gridDim.x * kWarps;
    const int first = blockIdx.x * kWarps + warp;

    // Starts the copies of one unit into stage s; an empty group behind the last unit. What is left for
    // consume: where the pair's output goes, and whether its rows exist and their position has angles.
    struct Sent {
        long long out;
        bool live0, live1, has;
    } sent[G::kStages];
    auto issue = [&](int unit, int s) {
        if (unit < n_units) {
            const bool is_k = unit >= n_q;
            const Side &sd = p.side[is_k ? 1 : 0];
            uint32_t tok;
            PairAt a = locate_pair(sd, p.seq, (unit - (is_k ? n_q : 0)) * R::kRows + group, &tok);
            const uint32_t base = ring + static_cast<uint32_t>(s * G::kStageBytes);
            const int pos = p.positions ? __ldg(p.positions + tok) : static_cast<int>(a.i);
            a.has = p.table.has(pos);
            // A row that does not exist, or whose position has no row of the tables, arrives as zeros; consume
            // takes r as 0 there, which keeps it out of dw, and stores zeros (0 times a weight need not be 0; by a
            // branch: a select of the packed row cost the gradient 0.4 us of 27).
            const bool on0 = a.live0 && a.has, on1 = a.live1 && a.has;
            if (kBackward) {
                const __nv_bfloat16 *dz = sd.dz + a.offset(sd.zs);
                copy_row(base + G::kDz * kSlotBytes, dz, le, on0);
                copy_row(base + (G::kDz + kRowSlots) * kSlotBytes, on1 ? dz + sd.zs.h : dz, le, on1);
            }
            if (!kBackward || sd.w) {
                const __nv_bfloat16 *x = sd.x + a.offset(sd.xs);
                copy_row(base + G::kX * kSlotBytes, x, le, on0);
                copy_row(base + (G::kX + kRowSlots) * kSlotBytes, on1 ? x + sd.xs.h : x, le, on1);
            }
            if (le.rotated && a.has)
                copy_angles(base + G::kAngles * kSlotBytes, p.table, pos, l);
            sent[s] = Sent{a.offset(sd.os), a.live0, a.live1, a.has};
        }
        copy_commit();
    };

    // The weight of the side that the warp is at (units of q come first): read once for each.
    // (Backward keeps it packed: its unpacked registers would not fit.)
    Pairs w;
    RawRow wraw;
    auto load_weight = [&](int side) {
        if (p.side[side].w) {
            wraw = load_row(p.side[side].w, le);
            if constexpr (!kBackward)
                w = unpack_pairs<kInterleaved>(wraw);
        }
    };

    Pairs dw;
    float *red = reinterpret_cast<float *>(smem + G::kBytes);  // backward: [side][warp][D] sums
    // The sums of one side: over the lanes that hold the same channels, then to the warp's row.
    auto flush_dw = [&](int side) {
        if constexpr (kBackward) {
            float *mine = red + (side * kWarps + warp) * D;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
#pragma unroll
                for (int o = R::kLanes; o < 32; o <<= 1) {
                    dw.A[u] += __shfl_xor_sync(0xffffffffu, dw.A[u], o);
                    dw.B[u] += __shfl_xor_sync(0xffffffffu, dw.B[u], o);
                }
                if (group == 0) {
                    mine[elem_a<kInterleaved>(le, u)] = dw.A[u];
                    mine[elem_b<kInterleaved>(le, u)] = dw.B[u];
                }
                dw.A[u] = dw.B[u] = 0.f;
            }
        }
    };
    if constexpr (kBackward) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
            dw.A[u] = dw.B[u] = 0.f;
    }

    auto consume = [&](int unit, int s) {
        const bool is_k = unit >= n_q;
        const Side &sd = p.side[is_k ? 1 : 0];
        const bool norm = sd.w != nullptr;
        const uint32_t base = ring + static_cast<uint32_t>(s * G::kStageBytes);
        const Sent a = sent[s];
        const bool turn = le.rotated && a.has;
        __nv_bfloat16 *out = sd.out + a.out;
        // Everything of the stage is read, and the row sums of both rows are taken, before anything is
        // stored: the two rows' chains then overlap.
        if constexpr (!kBackward) {
            Pairs x[2];
            float r[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                x[k] = unpack_pairs<kInterleaved>(read_row(base + (G::kX + k * kRowSlots) * kSlotBytes));
            Angles ang;
            if (turn)
                ang = read_angles(base + G::kAngles * kSlotBytes);
            if (norm) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    r[k] = row_sum<D>(pairs_dot(x[k], x[k]));
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    scale_pairs(x[k], a.has ? rsqrtf(r[k] * (1.f / D) + p.eps) : 0.f, w);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (turn)
                    rotate_pairs<false>(x[k], ang);
                if (k ? a.live1 : a.live0) {
                    if (a.has)
                        store_row(out + (k ? sd.os.h : 0), le, pack_pairs<kInterleaved>(x[k]));
                    else
                        store_row(out + (k ? sd.os.h : 0), le, zero_row());
                }
            }
        } else {
            // (One row after the other: both at once need more than 128 registers, and spilling took 1.7
            // times as long.)
            Angles ang;
            if (turn)
                ang = read_angles(base + G::kAngles * kSlotBytes);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const bool live = k ? a.live1 : a.live0;
                Pairs dy = unpack_pairs<kInterleaved>(read_row(base + (G::kDz + k * kRowSlots) * kSlotBytes));
                if (turn)
                    rotate_pairs<true>(dy, ang);
                if (norm) {
                    const Pairs x = unpack_pairs<kInterleaved>(read_row(base + (G::kX + k * kRowSlots) * kSlotBytes));
                    Pairs g = dy;
                    mul_pairs(g, unpack_pairs<kInterleaved>(wraw));
                    const float xx = row_sum<D>(pairs_dot(x, x)), gx = row_sum<D>(pairs_dot(g, x));
                    const float r = live && a.has ? rsqrtf(xx * (1.f / D) + p.eps) : 0.f;
                    const float f = -r * r * (gx * (1.f / D));
                    const float2 rr = make_float2(r, r), ff = make_float2(f, f);
#pragma unroll
                    for (int u = 0; u < 8; u += 2) {
                        put_two(dw.A + u, __ffma2_rn(two(dy.A + u), __fmul2_rn(two(x.A + u), rr), two(dw.A + u)));
                        put_two(dw.B + u, __ffma2_rn(two(dy.B + u), __fmul2_rn(two(x.B + u), rr), two(dw.B + u)));
                        put_two(dy.A + u, __fmul2_rn(rr, __ffma2_rn(ff, two(x.A + u), two(g.A + u))));
                        put_two(dy.B + u, __fmul2_rn(rr, __ffma2_rn(ff, two(x.B + u), two(g.B + u))));
                    }
                }
                if (live) {
                    if (a.has)
                        store_row(out + (k ? sd.os.h : 0), le, pack_pairs<kInterleaved>(dy));
                    else
                        store_row(out + (k ? sd.os.h : 0), le, zero_row());
                }
            }
        }
    };

    int next = first;
#pragma unroll
    for (int s = 0; s < G::kStages; ++s, next += step)
        issue(next, s);
    bool on_k = first >= n_q;
    load_weight(on_k ? 1 : 0);
    for (int unit = first; unit < n_units;) {
#pragma unroll
        for (int s = 0; s < G::kStages; ++s) {
            if (unit >= n_units)
                break;
            copy_wait<G::kStages - 1>();
            if (!on_k && unit >= n_q) {  // this warp's first unit of k
                flush_dw(0);
                load_weight(1);
                on_k = true;
            }
            consume(unit, s);
            issue(next, s);
            unit += step;
            next += step;
        }
    }
    copy_wait<0>();
    if constexpr (kBackward) {
        flush_dw(on_k ? 1 : 0);
        if (!p.partials)
            return;
        if (!on_k || first >= n_q)
            flush_dw(on_k ? 0 : 1);  // no unit of the other side: zeros
        // The block's partial: the warps' sums in order.
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
            const int side = i / D, d = i % D;
            float t = 0.f;
#pragma unroll
            for (int v = 0; v < kWarps; ++v)
                t += red[(side * kWarps + v) * D + d];
            p.partials[static_cast<size_t>(blockIdx.x) * 2 * D + i] = t;
        }
    }
}

// dw[side][d] = the blocks' partials added up: one block per side and 32 channels, eight lanes to a partial
// (four channels each), 128 partials at a time; then the four partials of a warp and the warps' sums in order.
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float *partials, int blocks, int D, float *dwq, float *dwk)
{
    __shared__ float4 red[32][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int side = blockIdx.y, d0 = blockIdx.x * 32;
    float *dst = side ? dwk : dwq;
    // Launched while the gradient's last blocks still run (see the launch): their partials are complete
    // only behind this.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!dst)
        return;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 5  // all of them at once: kNormRopeBwdBlocks / 128
    for (int b = 4 * warp + (lane >> 3); b < blocks; b += 128) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(partials + (static_cast<size_t>(b) * 2 + side) * D + d0) + (lane & 7));
        t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
        t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
        t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
        t.z += __shfl_xor_sync(0xffffffffu, t.z, o);
        t.w += __shfl_xor_sync(0xffffffffu, t.w, o);
    }
    if (lane < 8)
        red[warp][lane] = t;
    __syncthreads();
    if (warp == 0) {
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < 32; ++v)
            sum += reinterpret_cast<const float *>(red[v])[lane];
        dst[d0 + lane] = sum;
    }
}

void fill_side(Side &sd, const NormRopeSide &a, int B, int S, int rows)
{
    sd.x = static_cast<const __nv_bfloat16 *>(a.x);
    sd.w = static_cast<const __nv_bfloat16 *>(a.w);
    sd.dz = static_cast<const __nv_bfloat16 *>(a.dz);
    sd.out = static_cast<__nv_bfloat16 *>(a.out);
    sd.xs = a.xs;
    sd.zs = a.zs;
    sd.os = a.os;
    const int per_token = (a.H + 1) / 2;
    sd.pairs_per_token = FastDiv(static_cast<uint32_t>(per_token));
    sd.heads = a.H;
    sd.pairs = B * S * per_token;
    sd.units = (sd.pairs + rows - 1) / rows;
}

template <int D, bool kInterleaved, bool kBackward>
cudaError_t launch(const NormRopeArgs &a, cudaStream_t stream)
{
    using R = RowLanes<D>;
    NormRopeParams p;
    fill_side(p.side[0], a.q, a.B, a.S, R::kRows);
    fill_side(p.side[1], a.k, a.B, a.S, R::kRows);
    p.table = RopeTable{a.cos, a.sin, a.rot_dim, a.max_pos};
    p.positions = a.positions;
    p.seq = FastDiv(static_cast<uint32_t>(a.S));
    p.eps = a.eps;
    p.partials = a.partials;
    constexpr int kSmem = Ring<kBackward>::kBytes + (kBackward ? 2 * kWarps * D * 4 : 0);
    // Per device, as for the other kernels: the attribute applies to the device current when it is set.
    static bool attr_set[kMaxDevices] = {};
    const int dev = current_device_index();
    if (dev < 0)
        return cudaErrorInvalidDevice;
    if (!attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(norm_rope_kernel<D, kInterleaved, kBackward>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess)
            return e;
        attr_set[dev] = true;
    }
    const long long want = (static_cast<long long>(p.side[0].units) + p.side[1].units + kWarps - 1) / kWarps;
    const long long most = 2LL * a.sm_count < kNormRopeBwdBlocks ? 2LL * a.sm_count : kNormRopeBwdBlocks;
    const int blocks = static_cast<int>(want < most ? want : most);
    norm_rope_kernel<D, kInterleaved, kBackward><<<static_cast<unsigned>(blocks), kThreads, kSmem, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !kBackward || !a.partials)
        return e;
    // The second kernel's launch overlaps the first one's end.
    return launch_behind(weight_grad_kernel, dim3(D / 32, 2), 1024, stream, static_cast<const float *>(a.partials), blocks, D,
                         a.dwq, a.dwk);
}

template <int D>
cudaError_t launch_d(const NormRopeArgs &a, cudaStream_t stream)
{
    if (a.backward)
        return a.interleaved ? launch<D, true, true>(a, stream) : launch<D, false, true>(a, stream);
    return a.interleaved ? launch<D, true, false>(a, stream) : launch<D, false, false>(a, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a, cudaStream_t stream)
{
    switch (a.D) {
    case 32:
        return launch_d<32>(a, stream);
    case 64:
        return launch_d<64>(a, stream);
    case 128:
        return launch_d<128>(a, stream);
    default:
        return cudaErrorInvalidValue;
    }
}

}  // namespace attn_b200
