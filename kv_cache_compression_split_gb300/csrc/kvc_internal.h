// kvc_internal.h -- host-side glue shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/kvc.h"

namespace kvc {

constexpr int TILE = 64;           // tokens per pipeline stage of the decode kernels
constexpr int H2O_ONCHIP_MAX_SLOTS = KVC_H2O_ONCHIP_MAX_SLOTS;   // fused H2O, logits on chip
constexpr int KIVI_G = KVC_KIVI_GROUP;

// Device status word of the current device (set-up once per device).
int *dev_status_ptr();

// SM count of the current device.
int sm_count();

// Raise the dynamic shared-memory limit of kernel `func` to `bytes` on the current
// device, once per (kernel, device); thread safe.  Returns the attribute call's error.
cudaError_t set_smem_once(const void *func, int bytes);

// Let kernel `func` run in clusters of more than 8 CTAs on the current device, likewise once.
cudaError_t allow_large_clusters_once(const void *func);

// CTAs of `func` (threads per CTA, dynamic shared memory) resident on all SMs of the
// current device together (at least one per SM), cached per (kernel, device).
int resident_ctas(const void *func, int threads, int smem);

// cuTensorMapEncodeTiled through the runtime's driver entry point.
bool encode_tmap_2d_f16(CUtensorMap *map, const void *base, uint64_t inner, uint64_t rows,
                        uint32_t box_inner, uint32_t box_rows);

// Rank-4 map of binary16 data (dims and box innermost first, byte strides of dims 1..3);
// swizzled over the bytes of the box's rows, 64 or 128.
bool encode_tmap_4d_f16(CUtensorMap *map, const void *base, const uint64_t dims[4],
                        const uint64_t strides[3], const uint32_t box[4]);

struct SlotAttendPlan {
    int splits;
    int tiles_per_split;
};

// Split plan shared by kvc_workspace_size and kvc_decode_attend (at most
// max_splits splits when none are requested).
SlotAttendPlan plan_attend(int units, int tiles_per_unit, int requested_splits, int max_splits = 64);

// Splits of one unit that the slot attention merges inside a thread-block cluster.
constexpr int SLOT_CLUSTER_MAX = 8;

// ---- launchers (each returns a cudaError_t of the launch) ----

struct AttendLaunch {
    int B, Hq, Hkv, D, C;
    const uint16_t *q;
    uint16_t *o;
    const uint16_t *K, *V;
    const int32_t *n;
    float *logits, *lse;
    float *part_o, *part_ml;
    int splits, tiles_per_split;
    float scale;
    float *h2o_scores;
    float h2o_keep, h2o_add;   // scores = keep * scores + add * p
    bool cluster;              // 2..8 splits merged in a cluster (no workspace)
    const int32_t *block_table; // paged layout (nullptr: dense)
    int num_pages;
};
cudaError_t launch_attend_slots(const AttendLaunch &a, cudaStream_t s);

// One decode step of H2O (scores != nullptr) or StreamingLLM in one launch of the slot
// attention kernel (one split): the new token joins the attention and takes one slot.
struct StepLaunch {
    kvc_slot_cache c;
    int Hq;
    const uint16_t *q;
    uint16_t *o;
    float *lse;
    const uint16_t *k_new, *v_new;
    float *scores;
    float h2o_keep, h2o_add;
    int n_heavy, n_recent, n_sink;
    float scale;
};
cudaError_t launch_decode_step(const StepLaunch &a, cudaStream_t s);

struct KiviAttendLaunch {
    int B, Hq, Hkv, D, bits, R, Cq;
    const uint16_t *q;
    uint16_t *o;
    const uint8_t *kb, *vb;
    const uint16_t *k_res, *v_res;
    const int32_t *len;
    float *lse;
    float *part_o, *part_ml;
    int splits, tiles_per_split;
    int full_units;              // with splits > 1: units 0 .. full_units-1 run unsplit
    float scale;
    const int32_t *block_table;  // paged group blocks (nullptr: dense)
    int num_pages;
    const uint8_t *kg, *vg;      // GEAR side blocks (nullptr: KIVI)
};
cudaError_t launch_attend_kivi(const KiviAttendLaunch &a, cudaStream_t s);

// Merge the split partials of units unit0 .. unit0 + n_units - 1 (partial rows
// indexed from unit0) into o and lse.
cudaError_t launch_combine(int B, int Hq, int Hkv, int D, int splits, int unit0, int n_units,
                           const float *part_o, const float *part_ml, uint16_t *o, float *lse,
                           cudaStream_t s);

// Attention of many query tokens per sequence.  Keys are the sequence's own tokens
// (n == nullptr: a causal prompt) or a unit's n slots, whose last ones hold the
// sequence's query tokens (a chunk over the slot cache).
struct TokensLaunch {
    int B, Hq, Hkv, D;
    int L;                     // packed: tokens of all sequences; padded: tokens per sequence
    const uint16_t *q, *k, *v;
    uint16_t *o;
    float *lse;                // may be nullptr
    long qs[3], ks[3], vs[3], os[3];   // element strides: sequence, head, token
    long ls[2];                // lse: sequence, head (tokens adjacent)
    const int32_t *cu;         // packed: first token of each sequence, [B + 1]
    const int32_t *lens;       // padded: tokens of each sequence (nullptr: L)
    const int32_t *n;          // chunk: slots of each unit
    int C;                     // chunk: slots per unit
    const int32_t *block_table; // chunk: paged layout (nullptr: dense)
    int num_pages;
    int kv_rows;               // chunk: rows of the K / V arrays (set by the launcher)
    int tiles;                 // chunk: tiles per item
    int splits;                // key ranges per item, merged by a second launch when above 1
    int ordered;               // chunk: items of long units first (set by the launcher)
    float *part_o;             // [splits, Hkv, D / 4, L * g, 4]: sums of the values, fp32
    float2 *part_ml;           // [splits, Hkv, L * g]: reference and sum
    int *broken;               // whether some sequence's range is bad, for the merge
    const uint64_t *mask;      // tree: [L, words] which nodes a node sees (nullptr: no tree)
    int words;
    float scale_log2;
    int *status;
};
cudaError_t launch_attend_tokens(const TokensLaunch &p, cudaStream_t s);

// Form (tiles per item) and key ranges per unit of a chunk of T tokens in all (requested > 0:
// that many ranges).
struct TokensPlan {
    int tiles, splits;
};
TokensPlan plan_tokens(int T, int B, int Hq, int Hkv, int D, int C, int requested);

// Page tables, slot map, positions and lengths of a ragged batch of new tokens.
struct PlanLaunch {
    int B, Hkv, C, T, num_pages;
    const int32_t *cu, *n, *seqlen, *table, *pages, *free_list, *count;
    int32_t *n_out, *seqlen_out, *table_out, *pages_out, *free_out, *count_out, *pos, *slot_map;
    int release;
    int *status;
};
cudaError_t launch_append_plan(const PlanLaunch &p, cudaStream_t s);

// Trees of drafted tokens: masks and positions, the walk over the accepted nodes, and the
// cache back on their path.
struct TreePlanLaunch {
    int B, T, words;
    const int32_t *cu, *parent, *seqlen;
    uint64_t *mask;
    int32_t *pos;
    int *status;
};
cudaError_t launch_tree_plan(const TreePlanLaunch &p, cudaStream_t s);

struct VerifyLaunch {
    int B, T, V;
    const int32_t *cu, *parent, *tokens;
    const float *p, *q, *u, *u_next;
    long ps, qs;
    int32_t *path, *count, *next_token;
    int max_path;
    int *status;
};
cudaError_t launch_draft_verify(const VerifyLaunch &p, cudaStream_t s);

struct CommitLaunch {
    int B, Hkv, D, C, T, max_path, num_pages;
    uint16_t *K, *V;
    const int32_t *cu, *path, *count, *slot_map, *n, *seqlen, *table;
    int32_t *n_out, *seqlen_out;
    int *status;
};
cudaError_t launch_draft_commit(const CommitLaunch &p, cudaStream_t s);

// New rows to the slots of a slot map (rows of the cache's K / V arrays, -1: skipped).
struct PackedLaunch {
    int T, Hkv, D;
    long rows;                 // rows of the K / V arrays
    const uint16_t *k_new, *v_new;
    long ks[2], vs[2];         // element strides: token, head
    uint16_t *K, *V;
    const int32_t *slot_map;
    int *status;
};
cudaError_t launch_append_packed(const PackedLaunch &p, cudaStream_t s);

cudaError_t launch_append_slots(const kvc_slot_cache &c, const uint16_t *k_new,
                                const uint16_t *v_new, int n_new, cudaStream_t s);
cudaError_t launch_append_quant(const kvc_quant_cache &c, const uint16_t *k_new,
                                const uint16_t *v_new, int n_new, cudaStream_t s);
cudaError_t launch_stream_append(const kvc_slot_cache &c, const uint16_t *k_new,
                                 const uint16_t *v_new, int n_sink, int n_recent, cudaStream_t s);

// Weights of the decode score update scores = keep * scores + add * p for a
// decay of 0 (plain: 1, 1) or lambda in (0, 1) (lambda, 1 - lambda); false
// for any other decay.
bool h2o_decay_weights(float decay, float *keep, float *add);
cudaError_t launch_h2o_decode_acc(const kvc_h2o_args &a, cudaStream_t s);
// Two tcgen05 passes over the causal prompt; lse_ws holds B*Hq*ceil(L/128)*128 floats.
cudaError_t launch_h2o_prefill(const kvc_h2o_args &a, float *lse_ws, cudaStream_t s);

enum EvictKind { EVICT_H2O = 0, EVICT_STREAM = 1, EVICT_RANDOM = 2 };
struct EvictLaunch {
    EvictKind kind;
    kvc_slot_cache c;
    float *scores;
    int n_heavy, n_recent, n_sink, prompt_len;
    int trigger;   // H2O: only units with n >= trigger are evicted (0: all)
    double keep_ratio;
    uint64_t seed;
    uint32_t epoch;
};
cudaError_t launch_evict(const EvictLaunch &e, cudaStream_t s);

} // namespace kvc
