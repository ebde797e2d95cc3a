/*
 * kernels.h — internal launch interface between the C-ABI layer (attn_api.cu) and the two kernels.
 * Not part of the public ABI.
 */
#pragma once

#include <cuda_runtime.h>

#include "fast_div.h"

namespace attn_b200 {

// Devices the library keeps state for (function attributes, occupancy, workspaces), by index.
constexpr int kMaxDevices = 64;

// Launches `kernel` programmatically behind the kernel before it on the stream: it may start once that
// one's blocks all run (or have called griddepcontrol.launch_dependents), and what it needs of it lies
// behind its own griddepcontrol.wait.
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t stream, const Args &...args)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// `total` units laid end to end, cut into `parts` ranges whose lengths differ by one at most (the first
// total % parts are the longer ones): with fewer units than parts the last ranges are empty.
struct EvenRange {
    unsigned base, rem;
    __host__ __device__ EvenRange(unsigned total, unsigned parts) : base(total / parts), rem(total - base * parts) {}
    __host__ __device__ unsigned begin(unsigned c) const { return c * base + (c < rem ? c : rem); }
    // The range that holds unit g < total.
    __host__ __device__ unsigned part_of(unsigned g) const
    {
        const unsigned longer = rem * (base + 1);
        return g < longer ? g / (base + 1) : rem + (g - longer) / base;
    }
};

// Index of the current device, or -1 if it cannot be read or is kMaxDevices or beyond. Function
// attributes such as the dynamic shared-memory limit take effect on the device that is current
// when they are set, so the launchers keep them per device.
inline int current_device_index()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return -1;
    }
    return (dev >= 0 && dev < kMaxDevices) ? dev : -1;
}

// Device status word values: 0 = fine, otherwise the site of the first wait that ran out.
enum WaitSite : int {
    kSiteNone = 0,
    kSitePrefillTmaEmpty = 1,
    kSitePrefillMmaQ = 2,
    kSitePrefillMmaFull = 3,
    kSitePrefillMmaSFree = 4,
    kSitePrefillMmaPFull = 5,
    kSitePrefillSoftmaxSFull = 6,
    kSitePrefillSoftmaxODone = 7,
    kSitePrefillEpilogue = 8,
    kSitePrefillDrain = 9,
    kSiteDecodeProducer = 16,
    kSiteDecodeConsumer = 17,
    kSiteBwd = 24,
    kSiteFp8Prefill = 32,
    kSiteSuffix = 40,
};

// Element strides of a [batch][head][row][dim] tensor with a contiguous dim (see tma_host.h).
struct TensorStrides {
    long long b, h, s;
};

struct PrefillArgs {
    const void *q, *k, *v;
    void *o;
    float *lse;  // [B][Hq][Sq], contiguous
    int B, Hq, Hkv, Sq, Skv, D;
    float scale;
    int causal;
    int *status;       // device status word
    int sm_count = 0;  // SMs of the device: the persistent grid's size
    TensorStrides qs, ks, vs, os;  // element strides of q, k, v, o
    // Paged, variable-length cache (seq_lens != nullptr; head dim 128): k, v are
    // [num_pages][Hkv][page_size][D]; sequence b holds min(max(seq_lens[b], 0), cap) keys, cap =
    // min(max_seq_len, pages_per_seq * page_size), in pages block_table[b][...]; Skv is unused.
    const int *seq_lens = nullptr;
    const int *block_table = nullptr;
    int num_pages = 0, page_size = 0, pages_per_seq = 0, max_seq_len = 0;
};

// How a decode (Sq == 1) is spread over persistent CTAs. A "pair" is one (batch, kv head, group of
// G query heads); its keys are cut into `cpp` chunks of `ck` keys; CTA c of `ctas` takes units
// [c*total/ctas, (c+1)*total/ctas) of the pairs' chunks laid end to end.
struct DecodePlan {
    int G;                  // query heads per pair
    int head_groups;        // (Hq / Hkv) / G
    long long pairs;        // B * Hkv * head_groups
    int ck;                 // keys per chunk
    int cpp;                // chunks per pair
    long long total;        // pairs * cpp
    int ctas;               // CTAs launched
    int max_contrib;        // most CTAs that can share one pair
    size_t partial_floats;  // workspace floats for shared pairs' partials (0 if no pair is shared)
};

struct DecodeArgs {
    const void *q, *k, *v;
    void *o;
    float *lse;
    // Element strides of q, k, v and o (dense cache, tensor-core kernel); `strided` false: the
    // contiguous [B][H][S][D] layouts, which the CUDA-core kernel requires.
    bool strided = false;
    TensorStrides qs{}, ks{}, vs{}, os{};
    int B, Hq, Hkv, Skv, D;
    float scale;
    DecodePlan plan;
    float *ws;          // plan.partial_floats floats (may be null when that is 0)
    int *counters;      // plan.pairs arrival counters, zero between calls
    int *status;        // device status word
    // Paged, variable-length cache (tensor-core decode only; seq_lens == nullptr: the dense cache
    // above). k, v are then [num_pages][Hkv][page_size][D]; block_table [B][pages_per_seq] and
    // seq_lens [B] are device int32 arrays; lengths are clamped to [0, min(max_seq_len, capacity)].
    const int *seq_lens = nullptr;
    const int *block_table = nullptr;
    int num_pages = 0, page_size = 0, pages_per_seq = 0, max_seq_len = 0;
    // e4m3 cache (tensor-core decode only): k, v hold e4m3 codes; k_scale, v_scale are device fp32
    // [Hkv][D] coefficients (value = code * coefficient of its kv head and channel).
    bool fp8 = false;
    const float *k_scale = nullptr, *v_scale = nullptr;
};

// ATTN_OK with the current device's SM count, or the attn_status that says why it cannot be used.
int check_device(int *sm_count);

// Returns a cudaError_t value (cudaSuccess on success); never synchronises.
cudaError_t launch_prefill(const PrefillArgs &a, cudaStream_t stream, int *encode_error);

// Prefill over an e4m3 K/V cache (head dim 128): k8, v8 [B][Hkv][Skv][D] codes, k_scale, v_scale
// [Hkv][D] fp32 coefficients; q, o [B][Hq][Sq][D] bf16, lse [B][Hq][Sq]; contiguous.
struct PrefillFp8Args {
    const void *q, *k8, *v8;
    const float *k_scale, *v_scale;
    void *o;
    float *lse;
    int B, Hq, Hkv, Sq, Skv, D;
    float scale;
    int causal;
    int *status;  // device status word
};
cudaError_t launch_prefill_fp8(const PrefillFp8Args &a, cudaStream_t stream, int *encode_error);

// The suffixes' part of a decode over a shared prefix: query heads of a pair (see suffix_sm100.cuh), and pairs of a kv head.
struct SuffixPlan {
    int heads_per_pair, head_groups;
};
SuffixPlan suffix_plan(int Hq, int Hkv);

// The shared-prefix part of a decode over paged caches (head dim 128): B sequences, one new token each,
// over the prefix's keys. The packed rows of one kv head make tiles of 128, two tiles share a list of KV
// tiles, and the lists are cut over blocks of the grid (prefix_split.cuh); every (list, block) segment
// leaves fp32 partials in slot list + block: part_o [slots][2][128][128] normalised, part_lse
// [slots][2][128] in log2 units.
struct PrefixPlan {
    int group, sub_groups;  // query heads of a row tile's group; parts of a group above 128 heads
    int heads;              // kv heads times sub_groups
    int tile_seqs;          // sequences in a tile
    int tile_pairs;         // per head
    int odd;                // a head's last pair has one tile only
    long long lists;
    int grid;               // blocks for prefix and suffixes together
    // The splits to choose from (prefix_split.cuh): the first by_head of 32 give every head equally many
    // blocks, from tile_pairs to steps more.
    int by_head, steps;
    float suffix_unit_us;
    FastDiv by_steps, by_share, by_rest;
};
PrefixPlan prefix_plan(int B, int Hq, int Hkv, int sm_count);

// How one call divides the grid.
struct PrefixSplit {
    int ctas;                // blocks of the prefix
    int per_list, per_last;  // of each list, and of a head's last list; per_last 0: cut end to end
    __host__ __device__ int per_head(int tile_pairs) const { return (tile_pairs - 1) * per_list + per_last; }
};
// The choice for a prefix of `tiles` KV tiles and suffixes of `work` units, the pairs' own included; its time.
double choose_split(const PrefixPlan &plan, long long tiles, long long work, PrefixSplit *split);
constexpr double kFixedSplitUs = 16.0;  // see prefix_split.cuh
struct PrefixArgs {
    const void *q, *k_pages, *v_pages;
    const int *prefix_table, *prefix_len;  // [prefix_pages], [1]
    int B, Hq, Hkv, num_pages, page_size, prefix_pages, cap;  // cap: most keys of the prefix
    float scale;
    PrefixPlan plan;
    bool find;  // the split is chosen on the device; otherwise `fixed`
    PrefixSplit fixed;
    float *part_o, *part_lse;
    int *status;
};

// The suffixes of a shared-prefix decode (head dim 128, paged bf16 cache): each sequence's token over its
// own keys. A pair is one (sequence, kv head, up to 16 query heads), its keys are units of 16; all pairs'
// units, sequence by sequence, are cut evenly over the workers (warps). Whole pairs leave their result
// in o (fp32 [B][Hq][128], normalised) and lse (log2 units); a worker's first and last piece of a shared
// pair are at pieces + (2 worker + (0 or 1)) * suffix_piece(heads_per_pair): O rows, then LSEs.
constexpr int kSuffixWarps = 12;      // workers of a CTA
constexpr int kSuffixUnitKeys = 16;
// Ranges are cut by units and so many more for each pair: what its start and end cost the worker. (16,884
// units of uneven suffixes on 34 SMs, their prefix on the others: 69.7 us without, 58.3, 58.1, 58.1 with 1, 2
// and 4; 100 suffixes of 300 keys at most 17.4, 16.7, 16.9 and 17.8.)
constexpr int kSuffixPairUnits = 2;
constexpr int kSuffixMinUnits = 2;    // units a worker has at least, while there are fewer than workers
// Workers that share `total` units, the pairs' own included, in a grid of `ctas`.
__host__ __device__ inline int suffix_workers(int total, int ctas)
{
    const int want = (total + kSuffixMinUnits - 1) / kSuffixMinUnits, most = ctas * kSuffixWarps;
    return want < most ? want : most;
}
// Floats of one piece; a multiple of four, so that every O row can be read 16 bytes at a time.
__host__ __device__ inline int suffix_piece(int heads_per_pair) { return heads_per_pair * 128 + (heads_per_pair + 3) / 4 * 4; }
struct SuffixArgs {
    const void *q, *k_pages, *v_pages;
    const int *seq_lens, *block_table;
    float *o, *lse, *pieces;
    int B, Hq, Hkv, num_pages, page_size, pages_per_seq, cap;
    float scale;
    SuffixPlan plan;
    int *status;
};
// Prefix and suffixes in one grid: the prefix's blocks first, then (own not null) the suffixes'.
cudaError_t launch_prefix_decode(const PrefixArgs &a, const SuffixArgs *own, cudaStream_t stream, int *encode_error);

// Joins the prefix's segments and the suffixes' results into o (bf16) and lse (natural log).
struct PrefixMergeArgs {
    PrefixPlan plan;
    bool find;  // as PrefixArgs
    PrefixSplit fixed;
    int B, Hq, Hkv, cap;
    const int *prefix_len;
    const float *part_o, *part_lse;
    const float *o_suffix, *lse_suffix, *pieces;  // null: no suffixes
    SuffixPlan suffix;
    const int *seq_lens;
    int suffix_cap;
    void *o;
    float *lse;
    FastDiv by_hq, by_tile_seqs, by_tile_group, by_group, by_pair;  // set by launch_prefix_merge
};
cudaError_t launch_prefix_merge(const PrefixMergeArgs &a, cudaStream_t stream);

// Backward pass (head dim 128): dq, dk, dv from q, k, v, o, dout and the forward's lse.
struct BwdArgs {
    const void *q, *k, *v, *o, *dout;
    const float *lse;
    void *dq, *dk, *dv;
    int B, Hq, Hkv, Sq, Skv, D;
    float scale;
    int causal;
    void *ws;      // bwd_workspace_bytes(B, Hq, Sq, D) bytes, 256-byte aligned
    int *status;   // device status word
    int sm_count;  // SMs of the device (chooses the head split)
};
size_t bwd_workspace_bytes(int B, int Hq, int Sq, int D);
cudaError_t launch_bwd(const BwdArgs &a, cudaStream_t stream, int *encode_error);

// LSE merge of a partial result (bf16 o_part, fp32 lse_part) into an fp32 accumulator, rows x D
// (D in {32, 64, 128}); o_out (bf16, may be null) receives the merged O.
cudaError_t launch_lse_merge(float *o_acc, float *lse_acc, const void *o_part, const float *lse_part, void *o_out,
                             long long rows, int D, int sm_count, cudaStream_t stream);

// Norm and rotation of q and k (head dim 32, 64 or 128) and its gradient. Rows are the heads of the
// B * S tokens; B * S * H stays below kMaxHeadRows, so that row numbers never pass 32 bits.
constexpr long long kMaxHeadRows = 2147483647LL - 4096;
constexpr int kNormRopeBwdBlocks = 592;  // blocks of the gradient at most: one partial of dw each
struct NormRopeSide {
    const void *x, *w, *dz;  // input, weight [D] (null: no norm), gradient of the output (backward)
    void *out;               // the output, or the input's gradient
    int H;
    TensorStrides xs, zs, os;  // of x, dz and out
};
struct NormRopeArgs {
    NormRopeSide q, k;
    const float *cos, *sin;  // [max_pos][rot_dim / 2]
    const int *positions;    // [B][S], or null: the row's index
    int B, S, D, rot_dim, max_pos, interleaved;
    float eps;
    bool backward;
    int sm_count;
    float *partials;   // backward with norm: [kNormRopeBwdBlocks][2][D], or null: no dw
    float *dwq, *dwk;  // [D], either may be null
};
cudaError_t launch_norm_rope(const NormRopeArgs &a, cudaStream_t stream);

// Append of B * S new tokens to a paged cache (head dim 128), keys normalised and rotated on the way,
// queries too when given.
struct AppendArgs {
    const void *q, *k, *v;     // q may be null
    const void *q_weight, *k_weight;
    const float *cos, *sin;
    const int *positions, *seq_lens, *new_lens, *block_table;  // positions, new_lens may be null
    void *q_out, *k_pages, *v_pages;
    const float *k_scale, *v_scale;  // e4m3 cache: [Hkv][128]; null: bf16 cache
    int B, Hq, Hkv, S, num_pages, page_size, pages_per_seq, rot_dim, max_pos, interleaved;
    float eps;
    int sm_count;
    TensorStrides qs, ks, vs, qos;
};
cudaError_t launch_append(const AppendArgs &a, cudaStream_t stream);

// Decode planning and launch. requested_ctas <= 0 means one CTA per resident slot on the device.
int decode_heads_per_cta(int group, int D);  // G: 1, 2, 4 or 8 (up to 16 for D = 128)
// fp8: plan for the e4m3-cache variant of the tensor-core kernel (its own occupancy).
cudaError_t decode_plan(int B, int Hq, int Hkv, int Skv, int D, int requested_ctas, int sm_count, DecodePlan *plan,
                        bool fp8 = false);
cudaError_t launch_decode(const DecodeArgs &a, cudaStream_t stream);

// Head dim 128 decodes on the tensor core (decode_tc_sm100.cu); launch_decode routes there.
int decode_tc_heads_per_pair(int group);  // G: largest power of two dividing the group, at most 16
int decode_tc_chunk_keys();               // keys per chunk (128)
cudaError_t decode_tc_ctas_per_sm(int G, bool fp8, int *ctas_per_sm);
size_t decode_tc_partial_floats(int G, int ctas);  // workspace floats for shared pairs' partials
constexpr int kPagedMaxBatch = 1024;  // batch entries a paged decode may have (per-CTA scan in shared memory)
// Plan of a paged, variable-length decode: lengths are only known on the device, so the plan holds
// upper bounds (cpp from max_seq_len; total is computed by each CTA); every pair may be shared.
cudaError_t decode_plan_paged(int B, int Hq, int Hkv, int max_seq_len, int requested_ctas, int sm_count,
                              DecodePlan *plan, bool fp8 = false);
cudaError_t launch_decode_tc(const DecodeArgs &a, cudaStream_t stream);

// The status word of attn_decode_noalloc's fixed scratch array on the current device, or nullptr
// if that entry point has not run on it (its address is only looked up by its first call there).
int *noalloc_status_word();

}  // namespace attn_b200
