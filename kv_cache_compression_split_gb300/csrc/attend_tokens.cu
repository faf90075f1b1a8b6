// attend_tokens.cu -- attention of many query tokens per sequence: whole prompts
// (kvc_prompt_attend) and chunks of new tokens over the slot cache
// (kvc_chunk_attend), on the 5th-generation tensor cores.
//
// For query token i of a sequence and query head h of KV head hk
//   s_j = scale q_i . k_j over the keys j < e_i,   m = max s, l = sum exp(s - m),
//   o_i = sum_j exp(s_j - m) v_j / l,              lse_i = m + log l
// with e_i = i + 1 in a prompt and e_i = n - m_b + i + 1 over a unit's n slots, of
// which the last m_b hold the chunk.  A row that sees nothing gives o = 0 and
// lse = -inf.
//
// Rows.  A tile is 128 rows of tcgen05.mma's M: (token, head of the group) pairs,
// token-major, so the query heads of one KV head share every key they read.  Two forms:
//   TILES = 2  one CTA per SM, a work item is two tiles of one (sequence, KV head): two
//              consecutive token ranges that share the K and V blocks, or, when its
//              tokens fit one tile, the same rows twice with the 128-key blocks dealt
//              out alternately.  Two independent softmax chains run per SM, and the
//              tensor cores work on one while the other's scores become probabilities.
//   TILES = 1  two CTAs per SM, one tile each: batches whose sequences bring few tokens,
//              where an item is a few key blocks and most of its time is latency.
//
// Pipeline.  The grid has a CTA per item; one that runs takes over the items of CTAs that
// have not started (cluster launch control), so work is balanced without a counter in
// memory and the pipeline does not drain between items.  A warp asks for the next item and looks
// it up: its sequence, its unit's slots, its part of the page table.  It does so when the
// producer has LEAD blocks of the item before left to load.  Asked for at that item's start, an
// item is held back by a CTA that may be busy for long: 16 trees over 1000 to 8192 slots 232 us
// then, 212 with 2 to 6 blocks left, 4 chunks of 257 to 512 tokens over such caches 178 and 155,
// 4 prompts of 2048 tokens of 32 heads 120 and 115.  A producer warp (TMA: query
// tiles, and K and V blocks through a ring), an MMA warp, and a warpgroup per tile in
// which a thread owns a row.  S = Q K^T (128 x 128, fp32) lands in TMEM; the row's
// thread reads it, keeps the running reference m and sum l in registers, and writes
// the probabilities back over S as binary16, from where they are the A operand of
// O += P V with O in TMEM.  The MMA warp issues O_t(j) and S_t(j + 1) of one tile
// back to back, so when S_t(j + 1) is complete O_t is at rest and its rows may be
// rescaled by their threads.  They rarely are: the reference follows the maximum only
// when that has grown by 2^8, and it lies 2^7 below the maximum that set it.  Probabilities
// then stay within 2^15, inside binary16, and are rounded by 2^-11 relative down to 2^-21 of
// the row's largest and by 2^-32 of it below that: with the reference at the maximum itself a
// weight under 2^-25 of the largest became 0, and 131 071 such keys were 0.3% of a row, whose
// sum had them and whose values had not.  Results leave through a
// small area of shared memory per warp, so that a warp stores whole rows: a thread that
// stores its own row touches 32 lines per instruction, which took 7000 clocks a tile.
//
// Code size.  The warps' roles run side by side, and what runs once per item comes from the
// instruction cache's far levels.  So prompts and chunks are kernels of their own, and loops
// that run a few times per item stay rolled: 74 KB instead of 105 took 187 us instead of 200
// for eight prompts of 152 to 2047 tokens, 29.6 instead of 31.9 for a batch of drafts.
//
// What bounds it.  Per 128 x 128 block of D = 128 the two products take 1070 clocks of the
// tensor pipe (a 128 x 128 x 16 product was measured at 64.5 to 67 clocks), the
// exponentials 520 of the SFU.  The two-tile form spends 1250 to 1310 clocks a block once it
// runs: a row's thread needs 1300 for its block (reading 30, maximum 300, exponentials and
// packing 800, storing 35) while the tensor cores do the other tile's.  8192 tokens of
// 64 / 8 heads: 654 to 737 us over GPUs and clocks, 1490 to 1680 TFLOP/s, 0.79 to 0.89 of the
// measured burst rate and 0.88 to 0.99 of the sustained one; back to back under the power cap
// 724 us at 1.64 GHz.  Shorter prompts pay about 3000 clocks per item between its last product
// and the next one's: one MMA warp serves both tiles in order, so both end and are stored
// together.  A batch of few tokens over long caches is HBM bound in the middle (64 KB per SM
// in 2700 clocks) and spends the rest on the start, the last round and the merge: 131 MB in
// 30 us in a graph, 33 us by single calls.  Heads of 64 channels: a block's products take half
// as long and its row threads as long as before, whose chain of loads, maximum, exponentials
// and stores bounds them: 2 x 8192 tokens of 16 heads 279 us, 985 TFLOP/s.
//
// Non-finite values.  A masked score is replaced, not added to, so keys behind a
// row's range never matter.  A masked value row would enter as 0 * v: rows behind the
// sequence's last key are cleared in shared memory, and a row whose result is not
// finite although its sum is gets it again from memory (rows_again).
#include "kvc_device.cuh"
#include "kvc_internal.h"

#include <math.h>

namespace kvc {

namespace {

constexpr int TM = 128;                   // rows of a tile
constexpr int BOX = 64;                   // keys of one TMA box (a page of the cache)
constexpr int NI = 2;                     // slots of the item feed
constexpr float LN2 = 0.6931471805599453f;
// The reference is log2 BELOW under the maximum that set it and moves when the maximum has
// grown by log2 GROWTH: probabilities reach 2^15, inside binary16.
constexpr float BELOW = 7.f, GROWTH = 8.f;

template <int D, int TILES> struct TokCfg {
    static constexpr int W_TMA = 4 * TILES, W_MMA = W_TMA + 1, W_NEXT = W_TMA + 2;   // one more is idle
    static constexpr int NTHR = 128 * (TILES + 1);
    static constexpr int CTAS = 3 - TILES;                 // per SM
    // keys of a block, and score buffers in TMEM: one per tile, or two for the only tile, so
    // that a block's scores are there when the row's threads have done the one before
    static constexpr int TK = 64 * TILES;
    static constexpr int NBOX = D / 64;
    static constexpr int QBOX_BYTES = TM * 128, QTILE_BYTES = NBOX * QBOX_BYTES;
    static constexpr int BOX_BYTES = TK * 128, TILE_BYTES = NBOX * BOX_BYTES;
    static constexpr int NS = D == 128 ? 4 : 8;   // ring stages (one K or V block each)
    static constexpr int LEAD = 4;   // blocks of an item that are still to be loaded when the next is asked for
    // output area of a row warp: buffers of 32 rows of 64 bytes
    static constexpr int OUT_BUF = 32 * 64, OUT_BUFS = TILES;
    static constexpr int OUT_BYTES = OUT_BUFS * OUT_BUF;
    static constexpr int ML_BYTES = TM * 8;
    static constexpr int SMEM = TILES * QTILE_BYTES + NS * TILE_BYTES + 4 * TILES * OUT_BYTES + ML_BYTES + 1024 + 1024;
    static constexpr uint32_t IDESC_QK = idesc_f16_f32(TM, TK);
    static constexpr uint32_t IDESC_PV = idesc_f16_f32_bmn(TM, D);
    static constexpr uint32_t COL_O = 2 * TK;              // TMEM: two score buffers, then O_t
    static constexpr uint32_t TMEM_COLS = 256 * TILES;
    // Registers.  384 threads are launched with 168 each, 256 (two CTAs per SM) with 128.
    // A row's thread holds its 128 scores and needs more; the last warpgroup gives what it
    // does not use.
    static constexpr int REGS = TILES == 2 ? 168 : 128;
    static constexpr int REGS_ROW = TILES == 2 ? 208 : 168, REGS_IO = 88;
    static_assert(128 * (TILES * REGS_ROW + REGS_IO) <= NTHR * REGS, "register split");
    static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory");
};

template <int N> struct Int {
    static constexpr int value = N;
};

struct TokItem {
    int b, hk;
    int tok0, ntok;      // tokens of the sequence
    int start;           // the sequence's first token in the tensors
    int shift;           // token i sees the keys j <= i + shift
    int keys;            // of the sequence or unit
    int j0, j1;          // key blocks
    int split;
    int two;             // one tile of rows, its blocks dealt to both warpgroups
};

struct TokMaps {
    CUtensorMap q, k, v, o;
};

// First token and length of sequence b; a range that leaves [0, L] counts as an
// empty sequence and is reported, and so does a tree of more nodes than its masks have bits.
template <bool TREE>
__device__ __forceinline__ void seq_range(const TokensLaunch &p, int b, int &start, int &len)
{
    start = p.cu ? p.cu[b] : 0;
    len = p.cu ? p.cu[b + 1] - start : p.lens ? p.lens[b] : p.L;
    if (start < 0 || start > p.L || len < 0 || len > p.L - start || (TREE && len > 64 * p.words)) {
        flag_error(p.status, DEV_CAPACITY);
        start = len = 0;
    }
}

// Walks the items in order: sequences, token ranges from the last (longest) to the
// first, KV heads, splits.  Every lane of the warp calls it.  It goes on from the
// sequences of the last call, since the work is handed out in order.
// Over a cache the sequences' slots may differ by far, and an item that is long and starts late
// runs while other SMs have nothing left.  So up to 32 sequences, one per lane, whose items do
// not all run at once are walked in four rounds, those of most slots first (by the first
// head's): 16 trees over 1000 to 8192 slots of 32 heads 217 us as they come, 215 in this order, 4
// chunks of 257 to 512 tokens over 2000 to 8192 slots 178 and 155.  More than 32 sequences, and
// the heads of a sequence, are walked as they come.
struct ItemWalk {
    static constexpr int ROUNDS = 4;
    int b0 = 0, round = 0;
    unsigned base = 0;   // items before it
    int s = 0, n = 0, own_round = -1;
    // tiles: per item; keys: per block
    template <bool CHUNK, bool TREE>
    __device__ bool find(const TokensLaunch &p, int tpt, int tiles, int keys, unsigned idx,
                         TokItem &it)
    {
        const int lane = threadIdx.x & 31;
        const unsigned splits = CHUNK ? p.splits : 1, Hkv = p.Hkv;
        const bool ordered = CHUNK && p.ordered;
        if (idx < base) {
            b0 = round = 0;
            base = 0;
        }
        if (ordered && own_round < 0) {
            own_round = ROUNDS;
            if (lane < p.B) {
                const unsigned slots = (unsigned)p.n[lane * p.Hkv];
                seq_range<TREE>(p, lane, s, n);
                own_round = ROUNDS - 1 - min(slots / (p.C / ROUNDS + 1u), ROUNDS - 1u);
            }
        }
        const int all = n;
#pragma unroll 1
        for (;; b0 += 32) {
            if (b0 >= p.B) {
                if (!ordered || ++round >= ROUNDS)
                    break;
                b0 = 0;
            }
            int s = this->s, n = all;
            if (ordered) {
                if (own_round != round)
                    n = 0;
                if (!__any_sync(0xffffffffu, n > 0))
                    continue;
            } else {
                s = n = 0;
                if (b0 + lane < p.B)
                    seq_range<TREE>(p, b0 + lane, s, n);
            }
            const unsigned ranges = (unsigned)(n + tiles * tpt - 1) / (unsigned)(tiles * tpt);
            unsigned sum = ranges * Hkv * splits;
            // ranges that overlap may add up to more than the grid: sums stop at the largest
            // number
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, sum, off);
                if (lane >= off)
                    sum = sum + y < y ? 0xffffffffu : sum + y;
            }
            sum = sum + base < base ? 0xffffffffu : sum + base;
            const unsigned here = __ballot_sync(0xffffffffu, sum > idx);
            if (!here) {
                base = __shfl_sync(0xffffffffu, sum, 31);
                continue;
            }
            const int src = __ffs(here) - 1;
            const unsigned before = __shfl_sync(0xffffffffu, sum, max(src - 1, 0));
            const unsigned r = idx - (src ? before : base);
            const int per = __shfl_sync(0xffffffffu, ranges, src);
            const int len = __shfl_sync(0xffffffffu, n, src);
            it.start = __shfl_sync(0xffffffffu, s, src);
            it.b = b0 + src;
            const unsigned q = r / splits, range = q / Hkv;
            it.split = r - q * splits;
            it.hk = q - range * Hkv;
            it.tok0 = (per - 1 - (int)range) * tiles * tpt;
            it.ntok = min(tiles * tpt, len - it.tok0);
            it.two = tiles == 2 && it.ntok <= tpt;
            int n_keys = len;
            if (CHUNK) {
                n_keys = p.n[it.b * p.Hkv + it.hk];
                if (n_keys < 0 || n_keys > p.C) {
                    flag_error(p.status, DEV_CAPACITY);
                    n_keys = 0;
                }
            }
            it.keys = n_keys;
            it.shift = n_keys - len;
            const int end = max(0, it.shift + it.tok0 + it.ntok);
            const int blocks = (end + keys - 1) / keys;
            const int chunk = (blocks + splits - 1) / splits;
            it.j0 = min(blocks, it.split * chunk);
            it.j1 = min(blocks, it.j0 + chunk);
            return true;
        }
        return false;
    }
};

// Keys before `end` that tile t of the item sees, and its share of the blocks.
template <int TK> struct TileRange {
    int tok, ntok;       // tokens of the tile
    int end;             // keys its last token sees
    int j, step, count;  // blocks j, j + step, ...
    __device__ TileRange(const TokItem &it, int t, int tpt)
    {
        tok = it.tok0 + (it.two ? 0 : t * tpt);
        ntok = it.two ? it.ntok : t ? it.ntok - tpt : min(tpt, it.ntok);
        end = max(0, it.shift + tok + ntok);
        const int j1 = min(it.j1, (end + TK - 1) / TK);
        step = it.two ? 2 : 1;
        j = it.j0 + (it.two ? t : 0);
        count = max(0, (j1 - j + step - 1) / step);
    }
};

template <bool CHUNK>
__device__ __forceinline__ const uint16_t *key_row(const TokensLaunch &p, const uint16_t *base,
                                                   const long *st, const TokItem &it, int j)
{
    if (!CHUNK)
        return base + (p.cu ? 0 : it.b) * st[0] + it.hk * st[1] + (long)(it.start + j) * st[2];
    const long row = SlotRows{p.block_table, p.C, p.num_pages}.row(it.b * p.Hkv + it.hk, j);
    return row < 0 ? nullptr : base + row * p.D;
}

// Scores behind the row's range (column > lim) become -inf.
__device__ __forceinline__ void mask64(float (&x)[64], int lim)
{
#pragma unroll
    for (int c = 0; c < 64; ++c)
        x[c] = c <= lim ? x[c] : -INFINITY;
}

// Which of the 64 columns that begin with node `off` of its tree a row sees: all in front of
// the tree (off may be negative), then its mask's, none behind column lim.
__device__ __forceinline__ uint64_t tree_columns(const uint64_t *mask, int words, int off, int lim)
{
    if (lim < 0)
        return 0;
    uint64_t x = ~0ull;
    if (off > -64) {
        const int w = off >> 6, s = off & 63;
        const uint64_t lo = w < 0 ? ~0ull : w < words ? mask[w] : 0;
        const uint64_t hi = w + 1 < words ? mask[w + 1] : 0;
        x = s ? lo >> s | hi << (64 - s) : lo;
    }
    return lim < 63 ? x & ((2ull << lim) - 1) : x;
}

__device__ __forceinline__ void mask64(float (&x)[64], uint64_t columns)
{
    const uint32_t lo = (uint32_t)columns, hi = (uint32_t)(columns >> 32);
#pragma unroll
    for (int c = 0; c < 32; ++c) {
        x[c] = lo >> c & 1 ? x[c] : -INFINITY;
        x[32 + c] = hi >> c & 1 ? x[32 + c] : -INFINITY;
    }
}

__device__ __forceinline__ float max64(const float (&x)[64])
{
    float c0 = fmax3f(x[0], x[1], x[2]), c1 = fmax3f(x[16], x[17], x[18]);
    float c2 = fmax3f(x[32], x[33], x[34]), c3 = fmax3f(x[48], x[49], x[50]);
#pragma unroll
    for (int c = 3; c < 15; c += 2) {
        c0 = fmax3f(c0, x[c], x[c + 1]);
        c1 = fmax3f(c1, x[16 + c], x[17 + c]);
        c2 = fmax3f(c2, x[32 + c], x[33 + c]);
        c3 = fmax3f(c3, x[48 + c], x[49 + c]);
    }
    return fmaxf(fmax3f(c0, c1, x[15]), fmax3f(c2, c3, fmax3f(x[31], x[47], x[63])));
}

// Probabilities 2^(x scale - ref) of 64 scores into TMEM (two per column, binary16: they
// are an operand of the second product), and their sum before that rounding.
__device__ __forceinline__ float prob64(uint32_t taddr, const float (&x)[64], float2 scale,
                                        float2 nref)
{
    float2 a0 = make_float2(0.f, 0.f), a1 = a0;
#pragma unroll
    for (int c = 0; c < 64; c += 32) {
        uint32_t w[16];
#pragma unroll
        for (int u = 0; u < 16; u += 2) {
            const float2 y0 = ffma2(make_float2(x[c + 2 * u], x[c + 2 * u + 1]), scale, nref);
            const float2 y1 = ffma2(make_float2(x[c + 2 * u + 2], x[c + 2 * u + 3]), scale, nref);
            const float2 e0 = make_float2(ex2(y0.x), ex2(y0.y));
            const float2 e1 = make_float2(ex2(y1.x), ex2(y1.y));
            a0 = fadd2(a0, e0);
            a1 = fadd2(a1, e1);
            w[u] = pack_half2(e0.x, e0.y);
            w[u + 1] = pack_half2(e1.x, e1.y);
        }
        tmem_st16(taddr + c / 2, w);
    }
    const float2 a = fadd2(a0, a1);
    return a.x + a.y;
}

// 4 (D = 128) or 2 (D = 64) channels of a row: a lane's share when a warp reads it whole.
template <int CH> struct Channels {
    uint32_t w[CH / 2];
    __device__ void load(const uint16_t *row)
    {
        if constexpr (CH == 4) {
            const uint2 x = *reinterpret_cast<const uint2 *>(row);
            w[0] = x.x;
            w[1] = x.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t *>(row);
        }
    }
    __device__ uint16_t bits(int c) const { return (uint16_t)(w[c / 2] >> 16 * (c & 1)); }
    __device__ float value(int c) const { return __half2float(__ushort_as_half(bits(c))); }
    // Not 0 when some channel is not finite (an exponent of ones).
    __device__ uint32_t odd() const
    {
        uint32_t x = 0;
#pragma unroll
        for (int i = 0; i < CH / 2; ++i)
            x |= ((w[i] & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
        return x;
    }
};

// The results of the rows `rows` (bits: lanes) of a warp whose tensor-core result is not
// finite although their sum is: some value row of the keys [first, end) that the tile went
// through is not.  The warp looks for such values first, every lane in its own channels.  A
// channel in which a row attends one has its result by that alone: NaN, or an infinity where
// all that it attends have one sign.  Only a row with a channel whose values of that kind all
// lie behind it (they entered as 0 * v) is computed again, R rows together: a key's scores per
// lane, then the lane's channels over the 32 keys.  So a value that is not finite costs the
// rows behind it a pass over the values, and only the rows of its own tile are computed again:
// 200 003 tokens of 8 heads over one of 128 channels take 46 ms, 600 ms with a NaN in the last
// tile and 480 ms with one in the first.
// In a tree, a row attends every key before it.shift and then those of its mask: the first are
// looked through for all rows together, the others, few, for each row by itself.
template <int D, bool CHUNK, bool TREE>
__device__ __noinline__ void rows_again(const TokensLaunch &p, const TokItem &it, unsigned rows,
                                        const uint16_t *q, int first, int end, int last,
                                        const uint64_t *mask, float ref, float scale, uint16_t *o,
                                        float4 *part, long stride, volatile uint32_t *active)
{
    constexpr int CH = D / 32, U = 8, R = 2;
    constexpr unsigned ALL = 0xffffffffu;
    constexpr int NEVER = 0x7fffffff;
    using Vec = Channels<CH>;
    const int lane = threadIdx.x & 31, c0 = CH * lane;
    auto from = [&](auto *ptr, int src) {
        return reinterpret_cast<decltype(ptr)>(
            __shfl_sync(ALL, reinterpret_cast<unsigned long long>(ptr), src));
    };
    // per channel: the first key with a NaN, +inf, -inf, and the last key with any of them
    int nan_at[CH], pos_at[CH], neg_at[CH], any_at[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        nan_at[c] = pos_at[c] = neg_at[c] = NEVER;
        any_at[c] = -1;
    }
    const int tree = TREE ? min(end, max(first, it.shift)) : end;   // the item's first node
#pragma unroll 1
    for (int j = first; j < tree; j += 2 * U) {
        still_active(active);
        Vec x[2 * U];
        uint32_t odd = 0;
#pragma unroll
        for (int u = 0; u < 2 * U; ++u) {
            const uint16_t *v = j + u < tree ? key_row<CHUNK>(p, p.v, p.vs, it, j + u) : nullptr;
            x[u] = Vec{};
            if (v)
                x[u].load(v + c0);
        }
#pragma unroll
        for (int u = 0; u < 2 * U; ++u)
            odd |= x[u].odd();
        if (odd)
#pragma unroll
            for (int u = 0; u < 2 * U; ++u)
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const uint32_t h = x[u].bits(c);
                    if ((h & 0x7c00u) != 0x7c00u)
                        continue;
                    any_at[c] = j + u;
                    const bool nan = h & 0x3ffu, neg = h & 0x8000u;
                    nan_at[c] = min(nan_at[c], nan ? j + u : NEVER);
                    pos_at[c] = min(pos_at[c], nan || neg ? NEVER : j + u);
                    neg_at[c] = min(neg_at[c], nan || !neg ? NEVER : j + u);
                }
    }
    auto sees = [&](int j, int lim, const uint64_t *row_mask) {
        if (!TREE || j < it.shift)
            return j <= lim;
        return j <= lim && (row_mask[(j - it.shift) >> 6] >> (j - it.shift & 63) & 1);
    };
    // Per channel of this lane what the row of lane `src` meets: NaN, +inf and -inf that it
    // attends, and any of them that it does not.
    constexpr uint32_t HAS_NAN = 1, HAS_POS = 2, HAS_NEG = 4, ATTENDED = 7, BEHIND = 8;
    auto meets = [&](int src, uint32_t (&st)[CH]) {
        const int lim = __shfl_sync(ALL, last, src);
#pragma unroll
        for (int c = 0; c < CH; ++c)
            st[c] = (nan_at[c] <= lim ? HAS_NAN : 0) | (pos_at[c] <= lim ? HAS_POS : 0) |
                    (neg_at[c] <= lim ? HAS_NEG : 0) | (any_at[c] > lim ? BEHIND : 0);
        if constexpr (TREE) {
            const uint64_t *row_mask = from(mask, src);
            still_active(active);
#pragma unroll 1
            for (int j = tree; j < end; ++j) {
                const uint16_t *v = key_row<CHUNK>(p, p.v, p.vs, it, j);
                Vec x{};
                if (v)
                    x.load(v + c0);
                if (!x.odd())
                    continue;
                const bool in = sees(j, lim, row_mask);
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const uint32_t h = x.bits(c);
                    if ((h & 0x7c00u) == 0x7c00u)
                        st[c] |= !in ? BEHIND : h & 0x3ffu ? HAS_NAN : h & 0x8000u ? HAS_NEG : HAS_POS;
                }
            }
        }
    };
    auto store = [&](uint16_t *to, float4 *to4, int c, float x) {
        if (to4)
            reinterpret_cast<float *>(to4 + (c0 + c) / 4 * stride)[(c0 + c) % 4] = x;
        else
            to[c0 + c] = __half_as_ushort(__float2half_rn(x));
    };
    unsigned again = 0;
#pragma unroll 1
    for (unsigned left = rows; left; left &= left - 1) {
        const int src = __ffs(left) - 1;
        uint16_t *to = from(o, src);
        float4 *to4 = from(part, src);
        uint32_t st[CH];
        meets(src, st);
        bool behind = false;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const bool neg = st[c] & HAS_NEG, pos = st[c] & HAS_POS;
            const bool nan = (st[c] & HAS_NAN) || (neg && pos);
            behind |= !(st[c] & ATTENDED) && (st[c] & BEHIND);
            if (st[c] & ATTENDED)
                store(to, to4, c, nan ? NAN : pos ? INFINITY : -INFINITY);
        }
        if (__any_sync(ALL, behind))
            again |= 1u << src;
    }
#pragma unroll 1
    while (again) {
        int src[R], lim[R], most = -1;   // rows that there are not: the last one once more
        const uint16_t *qr[R];
        const uint64_t *row_mask[R];
        float m[R], acc[R][CH];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            src[r] = again ? __ffs(again) - 1 : src[r ? r - 1 : 0];
            again &= again - 1;
            lim[r] = __shfl_sync(ALL, last, src[r]);
            m[r] = __shfl_sync(ALL, ref, src[r]);
            qr[r] = from(q, src[r]);
            row_mask[r] = TREE ? from(mask, src[r]) : nullptr;
            most = max(most, lim[r]);
#pragma unroll
            for (int c = 0; c < CH; ++c)
                acc[r][c] = 0.f;
        }
        const int stop = min(end, most + 1);
#pragma unroll 1
        for (int j0 = first; j0 < stop; j0 += 32) {
            still_active(active);
            const int j = j0 + lane;
            const uint16_t *k = j < stop ? key_row<CHUNK>(p, p.k, p.ks, it, j) : nullptr;
            const uint16_t *v = k ? key_row<CHUNK>(p, p.v, p.vs, it, j) : nullptr;
            float w[R] = {};
            if (k) {
#pragma unroll 4
                for (int d = 0; d < D; d += 8) {
                    const uint4 b = *reinterpret_cast<const uint4 *>(k + d);
                    const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const uint4 a = *reinterpret_cast<const uint4 *>(qr[r] + d);
                        const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&aw[i]));
                            const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&bw[i]));
                            w[r] = fmaf(y.x, z.x, fmaf(y.y, z.y, w[r]));
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < R; ++r)
                    w[r] = sees(j, lim[r], row_mask[r]) ? ex2(w[r] * p.scale_log2 - m[r]) : 0.f;
            }
#pragma unroll 1
            for (int i = 0; i < 32; i += U) {
                Vec y[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint16_t *vr = from(v, i + u);
                    y[u] = Vec{};
                    if (vr)
                        y[u].load(vr + c0);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool odd = y[u].odd();   // behind the row, or its channel has its result
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float wi = __shfl_sync(ALL, w[r], i + u);
#pragma unroll
                        for (int c = 0; c < CH; ++c) {
                            const float x = y[u].value(c);
                            acc[r][c] = fmaf(wi, odd && !(fabsf(x) < INFINITY) ? 0.f : x, acc[r][c]);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float f = __shfl_sync(ALL, scale, src[r]);
            uint16_t *to = from(o, src[r]);
            float4 *to4 = from(part, src[r]);
            uint32_t st[CH];
            meets(src[r], st);
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (!(st[c] & ATTENDED))
                    store(to, to4, c, acc[r][c] * f);
        }
    }
    still_active(active);
}

template <int D, int TILES, bool CHUNK, bool TREE>
__global__ void __launch_bounds__(TokCfg<D, TILES>::NTHR, TokCfg<D, TILES>::CTAS)
    k_attend_tokens(const __grid_constant__ TokMaps maps, const __grid_constant__ TokensLaunch p)
{
    using Cfg = TokCfg<D, TILES>;
    constexpr int NS = Cfg::NS, TK = Cfg::TK, W_TMA = Cfg::W_TMA, W_MMA = Cfg::W_MMA;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_align1024(smem_raw);
    uint8_t *sq = smem;                                      // query tiles
    uint8_t *ring = sq + TILES * Cfg::QTILE_BYTES;            // NS blocks of K or V
    uint8_t *s_out = ring + NS * Cfg::TILE_BYTES;            // an output area per row warp
    float2 *s_ml = reinterpret_cast<float2 *>(s_out + 4 * TILES * Cfg::OUT_BYTES);
    uint64_t *bars = reinterpret_cast<uint64_t *>(s_ml) + TM;
    uint64_t *kv_full = bars, *kv_empty = kv_full + NS;
    uint64_t *q_full = kv_empty + NS, *q_empty = q_full + 1;
    uint64_t *s_full = q_empty + 1, *p_full = s_full + 2, *o_full = p_full + 2;
    uint64_t *it_full = o_full + 2, *it_empty = it_full + NI;
    uint64_t *mrg_full = it_empty + NI, *mrg_empty = mrg_full + 4;
    uint64_t *mma_done = mrg_empty + 4;
    uint64_t *clc_full = mma_done + 1, *next = clc_full + 1;
    uint4 *clc = reinterpret_cast<uint4 *>(bars + 64);       // a 16-byte answer
    TokItem *s_item = reinterpret_cast<TokItem *>(clc + 1);
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(s_item + NI);
    volatile int *abort = reinterpret_cast<int *>(s_tmem + 1);
    // when a warp was last seen computing rows again
    volatile uint32_t *active = s_tmem + 2;

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int g = p.Hq / p.Hkv, tpt = TM / g;
    const bool packed = CHUNK || p.cu;

    asm volatile("griddepcontrol.launch_dependents;");
    if (threadIdx.x == 0) {
        *abort = 0;
        *active = 0;
        for (int i = 0; i < NS; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&kv_empty[i], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 4);
            mbar_init(&o_full[t], 1);
        }
        for (int i = 0; i < NI; ++i) {
            mbar_init(&it_full[i], 1);
            mbar_init(&it_empty[i], 2 + 4 * TILES);   // the TMA, the MMA and the row warps
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&mrg_full[i], 1);
            mbar_init(&mrg_empty[i], 1);
        }
        mbar_init(mma_done, 1);
        mbar_init(clc_full, 1);
        mbar_init(next, 1);
        fence_mbar_init();
    }
    if (warp == W_MMA) {
        tmem_alloc(s_tmem, Cfg::TMEM_COLS);
        tmem_relinquish();
    }
    // What the set-up above wrote is there behind this, which every warp calls once.
    auto set_up = [&] {
        tc_fence_before();
        asm volatile("bar.sync 1, %0;" ::"n"(Cfg::NTHR) : "memory");
        tc_fence_after();
        return *s_tmem;
    };

    // The others' waits run out only when no warp has been computing rows again for as long.
    auto spin = [&](uint64_t *bar, uint32_t parity) {
        return mbar_wait_or_abort(bar, parity, abort, active);
    };
    auto rest = [&](uint64_t *bar, uint32_t parity) {
        return mbar_sleep_or_abort(bar, parity, abort, active);
    };

    // The k-th item of the feed; false at the end (or after a wait that ran out).
    auto feed_get = [&](int k, TokItem &it) -> bool {
        const int slot = k % NI;
        const bool got = rest(&it_full[slot], (k / NI) & 1);
        if (!__all_sync(0xffffffffu, got))
            return false;
        it = s_item[slot];
        __syncwarp();
        mbar_arrive_warp(&it_empty[slot]);
        return it.b >= 0;
    };

    if (warp >= W_TMA) {
    regs_dec<Cfg::REGS_IO>();
    if (warp == Cfg::W_NEXT) {
        // ------------------------------------------------ the feed: which item comes next
        // An item is asked for when the one before has LEAD blocks left to load, so that its own loads
        // follow without the latency of sequence range, slot count and page table; and not
        // before, so that no CTA holds an item back while others have none.
        ItemWalk walk;
        int idx = blockIdx.x;
        bool ok = true, first = true;
        int n_clc = 0;
        int asked = -1;   // the launch-control request whose answer is still to come
        for (int k = 0; ok;) {
            TokItem it;
            it.b = -1;
            if (idx >= 0 && !walk.find<CHUNK, TREE>(p, tpt, TILES, TK, idx, it))
                it.j0 = it.j1 = it.two = 0;   // the grid is an upper bound
            if (first)   // the first item was looked up while the others set up
                set_up();
            first = false;
            if (idx < 0 || it.b >= 0) {
                const int slot = k % NI;
                if (lane == 0) {
                    ok = k < NI || rest(&it_empty[slot], ((k / NI) & 1) ^ 1);
                    if (ok) {
                        s_item[slot] = it;
                        mbar_arrive(&it_full[slot]);
                    }
                }
                ++k;
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok || idx < 0)
                    break;
            }
            if (CHUNK && p.block_table && it.b >= 0) {   // the item's part of the page table into L1
                const int per = p.C / PAGE_SLOTS;
                const int32_t *table = p.block_table + (size_t)(it.b * p.Hkv + it.hk) * per;
#pragma unroll 1
                for (int i = TK / BOX * it.j0 + 32 * lane; i < min(per, TK / BOX * it.j1); i += 1024)
                    asm volatile("prefetch.global.L1 [%0];" ::"l"(table + i));
            }
            if (CHUNK && idx == 0 && p.splits > 1) {
                // once per call, for the merge: ranges out of order cannot be bisected
                bool bad = false;
#pragma unroll 1
                for (int b = lane; b < p.B; b += 32) {
                    const int c0 = p.cu[b], c1 = p.cu[b + 1];
                    bad |= c0 < 0 || c1 < c0 || c1 > p.L;
                }
                bad = __any_sync(0xffffffffu, bad);
                if (lane == 0)
                    *p.broken = bad;
            }
            int to = -1;
            if (lane == 0) {
                // take over a CTA that has not started
                ok = it.b < 0 || rest(next, (k - 1) & 1);
                if (ok) {
                    clc_request(clc, clc_full);
                    asked = n_clc;
                    ok = rest(clc_full, n_clc & 1);
                }
                if (ok) {
                    to = clc_answer(clc);
                    asked = -1;
                }
            }
            ++n_clc;
            ok = __shfl_sync(0xffffffffu, ok, 0);
            idx = __shfl_sync(0xffffffffu, to, 0);
        }
        // the answer to a request after which a wait ran out has landed before the CTA leaves
        if (lane == 0 && asked >= 0)
            mbar_wait(clc_full, asked & 1);
    } else if (warp == W_TMA) {
        // ------------------------------------------------ producer
        if (lane == 0) {
            prefetch_tmap(&maps.q);
            prefetch_tmap(&maps.k);
            prefetch_tmap(&maps.v);
            prefetch_tmap(&maps.o);
        }
        set_up();
        int n_it = 0, n_q = 0;   // ring slots and query loads
        bool ok = true;
        TokItem it;
        for (int k = 0; ok && feed_get(k, it); ++k) {
            const int n = it.j1 - it.j0;
            if (n <= Cfg::LEAD)
                mbar_arrive_warp(next);
            const int unit = it.b * p.Hkv + it.hk;
            const int per = p.C / PAGE_SLOTS;
            if (lane == 0 && n > 0) {
                const int n_keys = it.keys;
                auto load = [&](const CUtensorMap *map, int j) {
                    const int st = n_it % NS;
                    if (n_it >= NS)
                        ok = ok && rest(&kv_empty[st], ((n_it / NS) & 1) ^ 1);
                    if (!ok)
                        return;
                    mbar_arrive_expect_tx(&kv_full[st], Cfg::TILE_BYTES);
                    uint8_t *dst = ring + st * Cfg::TILE_BYTES;
                    for (int h = 0; h < TK / BOX; ++h) {
                        const int j_key = j * TK + h * BOX;
                        if (CHUNK) {
                            // a box without a key, or without a page, reads as zeros: its
                            // row lies behind the last one
                            int row = p.kv_rows;
                            if (j_key < n_keys) {
                                if (!p.block_table) {
                                    row = unit * p.C + j_key;
                                } else {
                                    const int pg =
                                        __ldg(p.block_table + (size_t)unit * per + j_key / PAGE_SLOTS);
                                    if (pg >= 0 && pg < p.num_pages)
                                        row = pg * PAGE_SLOTS;
                                    else
                                        flag_error(p.status, DEV_CAPACITY);
                                }
                            }
                            for (int c = 0; c < Cfg::NBOX; ++c)
                                tma_load_2d(dst + c * Cfg::BOX_BYTES + h * (BOX * 128), map,
                                            &kv_full[st], 64 * c, row);
                        } else {
                            for (int c = 0; c < Cfg::NBOX; ++c)
                                tma_load_4d(dst + c * Cfg::BOX_BYTES + h * (BOX * 128), map,
                                            &kv_full[st], 64 * c, it.hk, it.start + j_key,
                                            packed ? 0 : it.b);
                        }
                    }
                    ++n_it;
                };
                // The order in which the MMA warp takes them: the first keys, then the query
                // tile (its place is free when the last item's scores are done), then values,
                // which wait for a place in the ring behind the last item's.
                const int ahead = TILES == 1 || it.two ? 2 : 1;
#pragma unroll 1
                for (int i = 0; ok && i < ahead && i < n; ++i)
                    load(&maps.k, it.j0 + i);
                if (ok && n_q > 0)
                    ok = rest(q_empty, (n_q - 1) & 1);
                if (ok) {
                    const int tiles = it.ntok > tpt ? 2 : 1;
                    mbar_arrive_expect_tx(q_full, tiles * Cfg::NBOX * tpt * g * 128);
#pragma unroll 1
                    for (int t = 0; t < tiles; ++t)
                        for (int c = 0; c < Cfg::NBOX; ++c)
                            tma_load_4d(sq + t * Cfg::QTILE_BYTES + c * Cfg::QBOX_BYTES, &maps.q,
                                        q_full, 64 * c, it.hk * g, it.start + it.tok0 + t * tpt,
                                        packed ? 0 : it.b);
                    ++n_q;
                }
                for (int i = 0; ok && i < n; ++i) {
                    if (i + Cfg::LEAD == n - 1)
                        mbar_arrive(next);
                    load(&maps.v, it.j0 + i);
                    if (ok && i + ahead < n)
                        load(&maps.k, it.j0 + i + ahead);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        // every copy has landed before the CTA leaves
        if (lane == 0) {
#pragma unroll 1
            for (int i = n_it > NS ? n_it - NS : 0; i < n_it; ++i)
                mbar_wait(&kv_full[i % NS], (i / NS) & 1);
            if (n_q > 0)
                mbar_wait(q_full, (n_q - 1) & 1);
        }
    } else if (warp == W_MMA) {
        // ------------------------------------------------ MMA issuer (an elected lane issues)
        int n_it = 0, n_q = 0;
        int n_p[2] = {0, 0};
        const Int<0> T0;
        const Int<1> T1;
        bool ok = true;
        TokItem it;
        const uint32_t tm = __shfl_sync(0xffffffffu, set_up(), 0);
        // descriptors differ in the start address alone (bits 0..13, in 16 bytes)
        const uint64_t q_desc = sdesc_k_sw128(smem_u32(sq));
        const uint64_t k_desc = sdesc_k_sw128(smem_u32(ring));
        const uint64_t v_desc = sdesc_mn_sw128(smem_u32(ring), Cfg::BOX_BYTES);
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, spin(bar, parity));
        };
        // t as a type: its TMEM columns and barrier are constants then
        auto qk = [&](auto t_, int tile, int st) {   // S_t = Q_tile K^T, K in ring stage st
            constexpr int t = decltype(t_)::value;
            const uint64_t qd = q_desc + tile * (Cfg::QTILE_BYTES >> 4);
            const uint64_t kd = k_desc + (uint32_t)st * (Cfg::TILE_BYTES >> 4);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t qo = ((kk >> 2) * Cfg::QBOX_BYTES + (kk & 3) * 32) >> 4;
                    const uint32_t ko = ((kk >> 2) * Cfg::BOX_BYTES + (kk & 3) * 32) >> 4;
                    umma_f16(tm + TK * t, qd + qo, kd + ko, Cfg::IDESC_QK, kk > 0 ? 1u : 0u);
                }
                umma_commit(&s_full[t]);
            }
            __syncwarp();
        };
        auto pv = [&](auto t_, int st, int keys, bool first) {   // O (+)= P_t V
            constexpr int t = decltype(t_)::value;
            const uint64_t vd = v_desc + (uint32_t)st * (Cfg::TILE_BYTES >> 4);
            const uint32_t od = tm + Cfg::COL_O + (TILES == 2 ? D * t : 0), pd = tm + TK * t;
            const uint32_t acc = first ? 0u : 1u;
            const int steps = (keys + 15) / 16;
            if (elect_one()) {
                if (steps >= TK / 16) {
#pragma unroll
                    for (int kk = 0; kk < TK / 16; ++kk)
                        umma_f16_ts(od, pd + 8 * kk, vd + kk * (2048 >> 4), Cfg::IDESC_PV,
                                    kk > 0 ? 1u : acc);
                } else {
#pragma unroll 1
                    for (int kk = 0; kk < steps; ++kk)
                        umma_f16_ts(od, pd + 8 * kk, vd + kk * (2048 >> 4), Cfg::IDESC_PV,
                                    kk > 0 ? 1u : acc);
                }
            }
            __syncwarp();
        };
        auto commit = [&](uint64_t *bar) {
            if (elect_one())
                umma_commit(bar);
            __syncwarp();
        };
        for (int k = 0; ok && feed_get(k, it); ++k) {
            // the same in every lane, and known to be
            it.tok0 = __shfl_sync(0xffffffffu, it.tok0, 0);
            it.ntok = __shfl_sync(0xffffffffu, it.ntok, 0);
            it.shift = __shfl_sync(0xffffffffu, it.shift, 0);
            it.j0 = __shfl_sync(0xffffffffu, it.j0, 0);
            it.j1 = __shfl_sync(0xffffffffu, it.j1, 0);
            it.two = __shfl_sync(0xffffffffu, it.two, 0);
            const int n = it.j1 - it.j0;
            if (n <= 0)
                continue;
            const TileRange<TK> r0(it, 0, tpt), r1(it, TILES - 1, tpt);
            const int ahead = TILES == 1 || it.two ? 2 : 1;
            wait(q_full, n_q & 1);
            ++n_q;
            // first scores of both tiles
#pragma unroll 1
            for (int i = 0; ok && i < ahead && i < n; ++i, ++n_it) {
                wait(&kv_full[n_it % NS], (n_it / NS) & 1);
                if (!ok)
                    break;
                tc_fence_after();
                const int kb = n_it % NS;
                if (TILES == 1 || it.two) {
                    if (i == 0)
                        qk(T0, 0, kb);
                    else
                        qk(T1, 0, kb);
                } else {
                    if (r0.count > 0)
                        qk(T0, 0, kb);
                    qk(T1, 1, kb);
                }
                commit(&kv_empty[n_it % NS]);
            }
            if (n <= ahead)
                commit(q_empty);
            for (int i = 0; ok && i < n; ++i) {
                const int j = it.j0 + i;
                const int vs = n_it++;
                const int ks = i + ahead < n ? n_it++ : -1;
                wait(&kv_full[vs % NS], (vs / NS) & 1);
                if (!ok)
                    break;
                const int vb = vs % NS;
                const int keys = min(TK, r1.end - j * TK);
                if (keys & 15) {   // rows behind the last key of the item: cleared
                    const int rows = 16 - (keys & 15);
#pragma unroll 1
                    for (int x = lane; x < rows * Cfg::NBOX * 8; x += 32) {
                        const int c = x / (rows * 8), y = x % (rows * 8);
                        *reinterpret_cast<uint4 *>(ring + (vs % NS) * Cfg::TILE_BYTES +
                                                   c * Cfg::BOX_BYTES + (keys + y / 8) * 128 +
                                                   (y & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                    __syncwarp();
                }
                if (TILES == 1 || it.two) {
                    auto one = [&](auto t) {
                        constexpr int T = decltype(t)::value;
                        wait(&p_full[T], n_p[T] & 1);
                        if (!ok)
                            return;
                        ++n_p[T];
                        tc_fence_after();
                        pv(t, vb, keys, i < TILES);
                        commit(&kv_empty[vs % NS]);
                        if (TILES == 1)   // each step of the only accumulator
                            commit(&o_full[T]);
                        if (ks >= 0) {
                            wait(&kv_full[ks % NS], (ks / NS) & 1);
                            if (!ok)
                                return;
                            tc_fence_after();
                            qk(t, 0, ks % NS);
                            commit(&kv_empty[ks % NS]);
                            if (i + ahead == n - 1)
                                commit(q_empty);
                        } else if (TILES == 2) {
                            commit(&o_full[T]);
                        }
                    };
                    if (!(i & 1))
                        one(T0);
                    else
                        one(T1);
                    continue;
                }
                if (i < r0.count) {
                    wait(&p_full[0], n_p[0] & 1);
                    if (!ok)
                        break;
                    ++n_p[0];
                    tc_fence_after();
                    pv(T0, vb, min(TK, r0.end - j * TK), i == 0);
                    if (i + 1 < r0.count) {
                        wait(&kv_full[ks % NS], (ks / NS) & 1);
                        if (!ok)
                            break;
                        tc_fence_after();
                        qk(T0, 0, ks % NS);
                    } else {
                        commit(&o_full[0]);
                    }
                }
                wait(&p_full[1], n_p[1] & 1);
                if (!ok)
                    break;
                ++n_p[1];
                tc_fence_after();
                pv(T1, vb, keys, i == 0);
                commit(&kv_empty[vs % NS]);
                if (ks >= 0) {
                    wait(&kv_full[ks % NS], (ks / NS) & 1);
                    if (!ok)
                        break;
                    tc_fence_after();
                    qk(T1, 1, ks % NS);
                    commit(&kv_empty[ks % NS]);
                    if (i + 2 == n)
                        commit(q_empty);
                } else {
                    commit(&o_full[1]);
                }
            }
        }
        // every product has finished before TMEM is released
        commit(mma_done);
        mbar_wait(mma_done, 0);
        __syncwarp();
    } else {
        set_up();
    }
    } else {
        // ------------------------------------------------ softmax: a thread per row
        regs_inc<Cfg::REGS_ROW>();
        const uint32_t tmem = set_up();
        const int t = warp >> 2, quarter = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t o_col = lanes + Cfg::COL_O + D * t;
        const int r = 32 * quarter + lane;
        const int r_tok = r / g, r_head = r - r_tok * g;
        const int w_tok = 32 * quarter / g;   // token of the warp's first row
        const float scale = p.scale_log2;
        int n_s[2] = {0, 0}, n_o[2] = {0, 0}, n_m = 0;   // phases: s_full, o_full, hand-over
        bool ok = true;
        TokItem it;
        for (int k = 0; ok && feed_get(k, it); ++k) {
            const TileRange<TK> rg(it, t, tpt);
            const bool real = r_tok < min(rg.ntok, tpt);
            const int last = real ? it.shift + rg.tok + r_tok : -1;
            const bool idle = w_tok >= rg.ntok;                   // no row of the warp is real
            const bool full = 32 % g == 0 && w_tok + 32 / g <= rg.ntok;
            const int first_last = it.shift + rg.tok + w_tok;
            // a row that is not real looks at no mask
            const uint64_t *mask = nullptr;
            if (TREE && real) {
                mask = p.mask + (size_t)(it.start + rg.tok + r_tok) * p.words;
                asm volatile("prefetch.global.L1 [%0];" ::"l"(mask));
            }
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < rg.count; ++i) {
                const int k0 = (rg.j + i * rg.step) * TK;
                // score buffer and its phase
                const int sb = TILES == 2 ? t : i & 1;
                const uint32_t s_col = lanes + TK * sb;
                const int ph = TILES == 2 || !sb ? n_s[0]++ : n_s[1]++;
                const bool got = spin(&s_full[sb], ph & 1);
                if (!__all_sync(0xffffffffu, got)) {
                    ok = false;
                    break;
                }
                if (idle) {
                    mbar_arrive_warp(&p_full[sb]);
                    continue;
                }
                tc_fence_after();
                float lo[64], hi[TILES == 2 ? 64 : 1];
                const int lim = last - k0;
                // ends behind some row's range, or behind some row's first node
                const bool cut = TREE ? k0 + TK > it.shift : k0 + TK - 1 > first_last;
                tmem_ld64(s_col, lo);
                if (cut) {
                    if constexpr (TREE)
                        mask64(lo, tree_columns(mask, p.words, k0 - it.shift, lim));
                    else
                        mask64(lo, lim);
                }
                float top = max64(lo);
                if constexpr (TILES == 2) {
                    tmem_ld64(s_col + 64, hi);
                    if (cut) {
                        if constexpr (TREE)
                            mask64(hi, tree_columns(mask, p.words, k0 + 64 - it.shift, lim - 64));
                        else
                            mask64(hi, lim - 64);
                    }
                    top = fmaxf(top, max64(hi));
                }
                const float mx = scale * top;
                const bool grow = mx > m + (BELOW + GROWTH);
                if (__any_sync(0xffffffffu, grow)) {
                    const float to = grow ? mx - BELOW : m;
                    const float f = grow ? ex2(m - to) : 1.f;   // 0 at the row's first key
                    m = to;
                    l *= f;
                    // two tiles: the scores were computed after the last product into O; one
                    // tile: they may be ahead of it
                    if (TILES == 1 && i > 0) {
                        const int e = (i - 1) & 1;   // the product before: its barrier and phase
                        const bool done =
                            spin(&o_full[e], ((e ? n_o[1] : n_o[0]) + ((i - 1) >> 1)) & 1);
                        if (!__all_sync(0xffffffffu, done)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                    }
                    if (i > 0) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float v[32];
                            tmem_ld32(o_col + c, v);
#pragma unroll
                            for (int u = 0; u < 32; ++u)
                                v[u] *= f;
                            tmem_st32(o_col + c, v);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m;
                const float2 sc2 = make_float2(scale, scale), nr2 = make_float2(-ref, -ref);
                l += prob64(s_col, lo, sc2, nr2);
                if constexpr (TILES == 2)
                    l += prob64(s_col + 32, hi, sc2, nr2);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                mbar_arrive_warp(&p_full[sb]);
            }
            if (!ok)
                break;
            if (rg.count > 0) {
                // One tile: the products into O alternate between two barriers.  The last
                // scores were issued after the last product but two, so on the last one's
                // barrier nothing but it can be outstanding, and a parity tells enough.
                bool got;
                if (TILES == 2) {
                    got = spin(&o_full[t], n_o[0]++ & 1);
                } else {
                    const int e = (rg.count - 1) & 1;
                    n_o[0] += (rg.count + 1) / 2;
                    n_o[1] += rg.count / 2;
                    got = spin(&o_full[e], ((e ? n_o[1] : n_o[0]) - 1) & 1);
                }
                if (!__all_sync(0xffffffffu, got))
                    break;
                tc_fence_after();
            }
            // ---- results
            const int head = it.hk * g + r_head;
            const int tok = it.start + rg.tok + r_tok;
            // Parts: of a split and KV head, the references and sums of its rows, and its rows'
            // values four channels at a time, so that a warp's rows are adjacent.
            const long rows = (long)p.L * g;
            auto part_at = [&](long per) {   // of `per` entries per row
                return ((long)it.split * p.Hkv + it.hk) * per * rows +
                       (long)(it.start + rg.tok) * g + r;
            };
            auto part_o = [&] { return reinterpret_cast<float4 *>(p.part_o) + part_at(D / 4); };
            auto o_row = [&] {
                return p.o + (packed ? 0 : it.b) * p.os[0] + head * p.os[1] + tok * p.os[2];
            };
            const bool part = CHUNK && p.splits > 1;
            if (elect_one())
                bulk_wait_read<0>();   // the last item's stores have read the area
            __syncwarp();
            float *hand = reinterpret_cast<float *>(s_out + (4 + quarter) * Cfg::OUT_BYTES) + lane;
            if (TILES == 2 && it.two && t == 1) {
                // second part of the blocks: handed over 32 channels at a time.  Each is read
                // before the warp goes on: its area takes the next item's results.
#pragma unroll 1
                for (int c = 0; c < D; c += 32, ++n_m) {
                    if (c == 0)
                        s_ml[r] = make_float2(m, l);
                    if (rg.count > 0 && !idle) {
                        float v[32];
                        tmem_ld32(o_col + c, v);
#pragma unroll
                        for (int u = 0; u < 32; ++u)
                            hand[32 * u] = v[u];
                    }
                    __syncwarp();
                    mbar_arrive_warp(&mrg_full[quarter]);
                    const bool got = spin(&mrg_empty[quarter], n_m & 1);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                }
                tc_fence_before();
                continue;
            }
            bool bad = false;
            float fa = 1.f, fb = 0.f;        // weights of the two parts of the blocks
            float inv = 1.f, lsum = l;
            // The area's rows are swizzled as TMA does it: 16-byte chunk ch of row r lies at
            // chunk ch ^ (r / 2 % 4).
            uint8_t *const area = s_out + warp * Cfg::OUT_BYTES;
            auto chunk = [&](uint8_t *buf, int ch) {
                return reinterpret_cast<uint4 *>(buf + lane * 64 + ((ch ^ (lane >> 1 & 3)) << 4));
            };
            if (!it.two && !part && rg.count > 0 && full) {
                // The common case: all 32 rows are real and whole tokens, so one TMA store
                // takes 32 channels of them.  A short loop: this code runs once per item and
                // comes from the instruction cache's far levels.
                inv = l > 0.f ? rcp(l) : 0.f;
                const int o_y = __shfl_sync(0xffffffffu, it.hk * g, 0);
                const int o_z = __shfl_sync(0xffffffffu, it.start + rg.tok + w_tok, 0);
                const int o_w = __shfl_sync(0xffffffffu, packed ? 0 : it.b, 0);
                const float2 inv2 = make_float2(inv, inv), zero2 = make_float2(0.f, 0.f);
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint8_t *buf = area + c / 32 % Cfg::OUT_BUFS * Cfg::OUT_BUF;
                    float v[32];
                    tmem_ld32(o_col + c, v);
                    if (c >= 32 * Cfg::OUT_BUFS) {
                        if (elect_one())
                            bulk_wait_read<Cfg::OUT_BUFS - 1>();
                        __syncwarp();
                    }
                    float2 z0 = zero2, z1 = zero2;   // not 0 when a value is not finite
#pragma unroll
                    for (int u = 0; u < 32; u += 8) {
                        const float2 v0 = make_float2(v[u], v[u + 1]);
                        const float2 v1 = make_float2(v[u + 2], v[u + 3]);
                        const float2 v2 = make_float2(v[u + 4], v[u + 5]);
                        const float2 v3 = make_float2(v[u + 6], v[u + 7]);
                        z0 = ffma2(v0, zero2, z0);
                        z1 = ffma2(v1, zero2, z1);
                        z0 = ffma2(v2, zero2, z0);
                        z1 = ffma2(v3, zero2, z1);
                        const float2 w0 = fmul2(v0, inv2), w1 = fmul2(v1, inv2);
                        const float2 w2 = fmul2(v2, inv2), w3 = fmul2(v3, inv2);
                        *chunk(buf, u / 8) =
                            make_uint4(pack_half2(w0.x, w0.y), pack_half2(w1.x, w1.y),
                                       pack_half2(w2.x, w2.y), pack_half2(w3.x, w3.y));
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (elect_one()) {
                        tma_store_4d(&maps.o, buf, c, o_y, o_z, o_w);
                        bulk_commit();
                    }
                    const float2 z = fadd2(z0, z1);
                    bad |= z.x + z.y != 0.f;
                }
            } else {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                if (TILES == 2 && it.two) {
                    const bool got = spin(&mrg_full[quarter], n_m & 1);
                    if (!__all_sync(0xffffffffu, got)) {
                        ok = false;
                        break;
                    }
                    ++n_m;
                    if (c == 0) {
                        const float2 other = s_ml[r];
                        const float mm = fmaxf(m, other.x);
                        fa = m == -INFINITY ? 0.f : ex2(m - mm);
                        fb = other.x == -INFINITY ? 0.f : ex2(other.x - mm);
                        lsum = l * fa + other.y * fb;
                        m = mm;
                    }
                }
                if (c == 0)
                    inv = part ? 1.f : lsum > 0.f ? rcp(lsum) : 0.f;
                float v[32];
                if (rg.count > 0 && !idle)
                    tmem_ld32(o_col + c, v);
                if (rg.count == 0 || idle || lsum == 0.f) {
#pragma unroll
                    for (int u = 0; u < 32; ++u)
                        v[u] = 0.f;
                }
                if (TILES == 2 && it.two) {
                    if (lsum != 0.f) {
#pragma unroll
                        for (int u = 0; u < 32; ++u) {
                            const float y = hand[32 * u];
                            v[u] = fmaf(fb, fb > 0.f ? y : 0.f, v[u] * fa);
                        }
                    }
                    __syncwarp();
                    mbar_arrive_warp(&mrg_empty[quarter]);
                }
                if (idle)
                    continue;
                float2 probe = make_float2(0.f, 0.f);   // not 0 when a value is not finite
#pragma unroll
                for (int u = 0; u < 32; u += 2)
                    probe = ffma2(make_float2(v[u], v[u + 1]), make_float2(0.f, 0.f), probe);
                bad |= probe.x + probe.y != 0.f;
                // parts of rows, and tiles that end inside a warp's rows: each thread stores
                // its own row
                if (real && part) {
                    float4 *to = part_o() + c / 4 * rows;
#pragma unroll
                    for (int u = 0; u < 32; u += 4)
                        to[u / 4 * rows] = make_float4(v[u], v[u + 1], v[u + 2], v[u + 3]);
                } else if (real) {
                    uint16_t *to = o_row() + c;
#pragma unroll
                    for (int u = 0; u < 32; u += 8)
                        *reinterpret_cast<uint4 *>(to + u) =
                            make_uint4(pack_half2(v[u] * inv, v[u + 1] * inv),
                                       pack_half2(v[u + 2] * inv, v[u + 3] * inv),
                                       pack_half2(v[u + 4] * inv, v[u + 5] * inv),
                                       pack_half2(v[u + 6] * inv, v[u + 7] * inv));
                }
            }
            }
            if (!ok)
                break;
            if (real) {
                if (part)
                    p.part_ml[part_at(1)] = make_float2(m, lsum);
                else if (p.lse)
                    p.lse[(packed ? 0 : it.b) * p.ls[0] + head * p.ls[1] + tok] =
                        lsum > 0.f ? (m + __log2f(lsum)) * LN2 : lsum == 0.f ? -INFINITY : lsum;
            }
            const bool again = real && bad && lsum < INFINITY;   // false for a sum that is NaN
            if (__any_sync(0xffffffffu, again)) {
                if (elect_one())
                    bulk_wait_all();   // what is stored again comes after what was stored
                __syncwarp();
                const uint16_t *q = p.q + (packed ? 0 : it.b) * p.qs[0] + head * p.qs[1] +
                                    tok * p.qs[2];
                const int end = max(0, it.shift + it.tok0 + it.ntok);   // keys of the item
                const TokItem item = it;   // it stays in registers
                rows_again<D, CHUNK, TREE>(p, item, __ballot_sync(0xffffffffu, again), q,
                                           it.j0 * TK, min(end, it.j1 * TK), last, mask,
                                           m == -INFINITY ? 0.f : m, inv, o_row(),
                                           part ? part_o() : nullptr, rows, active);
            }
            tc_fence_before();
        }
        if (elect_one())
            bulk_wait_read<0>();   // no store reads shared memory after the CTA has left
    }

    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) {
        tc_fence_after();
        tmem_dealloc(*s_tmem, Cfg::TMEM_COLS);
    }
    if (threadIdx.x == 0 && *abort)
        flag_error(p.status, DEV_TIMEOUT);
}

// Merges the splits.  A warp takes eight rows of a KV head and 16 channels, a lane four
// channels of a row.  WARPS = 4: the CTA's warps take every fourth split and meet in shared
// memory; WARPS = 1: each has channels of its own.  References, sums and values of U splits
// are in flight together, none waits for another.  The kernel runs once through code that
// no cache holds, so a split too many in U costs as much as a round of loads: U = 8 for the
// 8 splits of 2048 rows, two per warp, takes 1.7 us more than U = 4, and U = 4 for 38 splits
// 1.1 us more than U = 8.  Launched so that it may start while the attention still runs; it
// waits before it reads the parts.
constexpr int MAX_SPLITS = 64;
template <int D, int WARPS, int U>
__global__ void __launch_bounds__(128) k_combine_tokens(const TokensLaunch p, const int g)
{
    __shared__ float2 s_ml[WARPS][32];
    __shared__ float4 s_acc[WARPS][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split0 = WARPS > 1 ? warp : 0;
    const int c4 = 4 * (WARPS > 1 ? blockIdx.z : 4 * blockIdx.z + warp) + (lane >> 3);
    const int rows = p.L * g, row = blockIdx.x * 8 + (lane & 7);
    const int tok = (unsigned)row / (unsigned)g, head = blockIdx.y * g + row - tok * g;
    int lo = 0, hi = p.B;   // the first sequence that ends behind the token
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (p.cu[mid + 1] <= tok)
            lo = mid + 1;
        else
            hi = mid;
    }
    bool real = false;
    if (lo < p.B && row < rows) {
        const int start = p.cu[lo], end = p.cu[lo + 1];
        // as the attention took it
        real = start >= 0 && start <= tok && end <= p.L && (!p.words || end - start <= 64 * p.words);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!real && row < rows && *p.broken)
#pragma unroll 1
        for (int b = 0; b < p.B && !real; ++b) {
            const int start = p.cu[b], end = p.cu[b + 1];
            real = start >= 0 && start <= tok && tok < end && end <= p.L &&
                   (!p.words || end - start <= 64 * p.words);
        }
    const long step = (long)p.Hkv * rows;   // entries of a split
    const float2 *ml = p.part_ml + split0 * step + (long)blockIdx.y * rows + row;
    const float4 *part = reinterpret_cast<const float4 *>(p.part_o) + split0 * step * (D / 4) +
                         ((long)blockIdx.y * (D / 4) + c4) * rows + row;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float w, float lw, const float4 &x) {
        l = fmaf(w, lw, l);
        acc.x = fmaf(w, x.x, acc.x);
        acc.y = fmaf(w, x.y, acc.y);
        acc.z = fmaf(w, x.z, acc.z);
        acc.w = fmaf(w, x.w, acc.w);
    };
#pragma unroll 1
    for (int s0 = split0; s0 < p.splits; s0 += U * WARPS) {
        float2 y[U];
        float4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = s0 + u * WARPS < p.splits && real;
            y[u] = in ? *ml : make_float2(-INFINITY, 0.f);
            x[u] = in ? *part : make_float4(0.f, 0.f, 0.f, 0.f);
            ml += WARPS * step;
            part += WARPS * step * (D / 4);
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < U; ++u)
            top = fmaxf(top, y[u].x);
        // a range without a key of the row has the reference -inf, the sum 0 and zeros
        const float ref = top == -INFINITY ? 0.f : top, f = ex2(m - ref);
        m = top;
        l *= f;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
        for (int u = 0; u < U; ++u)
            add(ex2(y[u].x - ref), y[u].y, x[u]);
    }
    if (WARPS > 1) {
        s_ml[warp][lane] = make_float2(m, l);
        s_acc[warp][lane] = acc;
        __syncthreads();
        if (warp > 0)
            return;
#pragma unroll
        for (int i = 1; i < WARPS; ++i)
            m = fmaxf(m, s_ml[i][lane].x);
        l = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int i = 0; i < WARPS; ++i)
            add(ex2(s_ml[i][lane].x - ref), s_ml[i][lane].y, s_acc[i][lane]);
    }
    if (!real)
        return;
    const float inv = l != 0.f ? rcp(l) : 0.f;
    *reinterpret_cast<uint2 *>(p.o + head * p.os[1] + (long)tok * p.os[2] + 4 * c4) =
        make_uint2(pack_half2(acc.x * inv, acc.y * inv), pack_half2(acc.z * inv, acc.w * inv));
    if (p.lse && c4 == 0)
        p.lse[head * p.ls[1] + tok] = l > 0.f ? (m + __log2f(l)) * LN2 : l == 0.f ? -INFINITY : l;
}

template <int D, int TILES, bool CHUNK, bool TREE = false>
cudaError_t attend_tokens_impl(TokensLaunch p, cudaStream_t s)
{
    using Cfg = TokCfg<D, TILES>;
    const int g = p.Hq / p.Hkv, tpt = TM / g;
    TokMaps maps;
    const uint64_t seqs = p.cu ? 1 : p.B;
    const uint64_t D_ = D, L_ = p.L;
    auto map4 = [&](CUtensorMap *m, const uint16_t *base, const long *st, int heads, int box_heads,
                    int box_tok, uint32_t box_d = 64) {
        const uint64_t dims[4] = {D_, (uint64_t)heads, L_, seqs};
        const uint64_t str[3] = {(uint64_t)st[1] * 2, (uint64_t)st[2] * 2,
                                 (uint64_t)(seqs > 1 ? st[0] : st[2]) * 2};
        const uint32_t box[4] = {box_d, (uint32_t)box_heads, (uint32_t)box_tok, 1};
        return encode_tmap_4d_f16(m, base, dims, str, box);
    };
    bool ok = map4(&maps.q, p.q, p.qs, p.Hq, g, tpt) &&
              map4(&maps.o, p.o, p.os, p.Hq, g, 32 / g, 32);
    if (CHUNK) {
        p.kv_rows = p.block_table ? p.num_pages * PAGE_SLOTS : p.B * p.Hkv * p.C;
        ok = ok && encode_tmap_2d_f16(&maps.k, p.k, D, p.kv_rows, 64, BOX) &&
             encode_tmap_2d_f16(&maps.v, p.v, D, p.kv_rows, 64, BOX);
    } else {
        ok = ok && map4(&maps.k, p.k, p.ks, p.Hkv, 1, BOX) &&
             map4(&maps.v, p.v, p.vs, p.Hkv, 1, BOX);
    }
    if (!ok)
        return cudaErrorInvalidValue;
    cudaError_t e =
        set_smem_once(reinterpret_cast<const void *>(k_attend_tokens<D, TILES, CHUNK, TREE>), Cfg::SMEM);
    if (e != cudaSuccess)
        return e;
    // packed: every sequence ends in at most one partial range
    const int range = TILES * tpt;
    const long ranges =
        p.cu ? (long)p.L / range + p.B : (long)((p.L + range - 1) / range) * p.B;
    const long items = ranges * p.Hkv * p.splits;
    if (items > 0x7fffffffL)
        return cudaErrorInvalidValue;
    // Where all CTAs run at once, no order is better than another, and looking the order up costs
    // a start 1.2 us (3 x 1 to 130 tokens over 1000 slots, split: 10.5 us without, 11.7 with).
    p.ordered = CHUNK && p.B > 1 && p.B <= 32 && p.splits == 1 &&
                items > (long)Cfg::CTAS * sm_count();
    k_attend_tokens<D, TILES, CHUNK, TREE><<<(unsigned)items, Cfg::NTHR, Cfg::SMEM, s>>>(maps, p);
    e = cudaGetLastError();
    if (!CHUNK || e != cudaSuccess || p.splits == 1)
        return e;
    // The warps share the splits of a row where there are few rows: 40 rows of 8 heads and 38
    // splits, the whole call, 32.4 us against 36.2 with a warp for all of them; 512 rows and 8
    // splits 29.7 against 25.2.
    const bool many = p.splits > 4 && (long)p.L * p.Hq * D < 16L * 128 * sm_count();
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(((long)p.L * g + 7) / 8), p.Hkv, many ? D / 16 : D / 64);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (many)   // U by the splits of a warp
        return p.splits > 16 ? cudaLaunchKernelEx(&cfg, k_combine_tokens<D, 4, 8>, p, g)
                             : cudaLaunchKernelEx(&cfg, k_combine_tokens<D, 4, 4>, p, g);
    return p.splits > 2 ? cudaLaunchKernelEx(&cfg, k_combine_tokens<D, 1, 4>, p, g)
                        : cudaLaunchKernelEx(&cfg, k_combine_tokens<D, 1, 2>, p, g);
}

} // namespace

// Form and splits of a chunk, by what a call takes in microseconds: a start, then each round of
// CTAs its key blocks and an item's start and end, then the merge.  How many tokens a sequence
// brings is known on the GPU alone.  So the rounds are a mean of two estimates: of sequences of one
// length, whose rounds end together and count whole, and, with up to half the weight (one sequence
// has one length), of sequences a quarter longer or shorter, whose rounds run into one another.
// Both follow T without regard to what divides it.  The numbers are fitted to 1700 batches of 1 to
// 96 sequences of 1 to 400 tokens over 128 to 32768 slots, of one length or ragged, over caches of
// one length or ragged.  On 1110 others (220 of them of 200 to 4096 tokens over up to 65536
// slots), each with both forms and up to 17 numbers of splits, the choice was 2.5% above the best
// on average and over 10% above it on 88; by the first estimate alone, with numbers fitted to it,
// 3.1% and 109, by the second where B does not divide T 4.0% and 150.  Of 48 sequences of 2 to
// 4 tokens over 1024 slots, 192 items of one tile, the second takes two tiles for 23.4 us, one takes
// 19.5; of 64 trees of 8 to 24 nodes over 576 slots the first takes two for 49 us, one takes 40.  A
// block's time does not depend on D.  The slots that a unit holds are known on the GPU alone too:
// the capacity stands for them and every unit gets as many ranges.  64 sequences of 4 tokens, one
// over 32000 slots and the others over 300 to 610 of 32768, are not split and take 359 us, 88 us
// with num_splits = 8.
TokensPlan plan_tokens(int T, int B, int Hq, int Hkv, int D, int C, int requested)
{
    const int tpt = TM / (Hq / Hkv), sms = sm_count();
    const long rows = (long)T * Hq;
    const float weight = 0.5f - 0.5f / B;   // of the uneven estimate
    auto ceil_div = [](long x, long y) { return (x + y - 1) / y; };
    TokensPlan best{1, 1};
    float least = INFINITY;
    for (int tiles = D == 128 ? 2 : 1; tiles >= 1; --tiles) {
        const int keys = 64 * tiles, slots = sms * (3 - tiles);
        const int blocks = (C + keys - 1) / keys;
        const long range = (long)B * tiles * tpt;   // a range of tokens in every sequence
        const long items = (long)B * Hkv * ceil_div(T, range);
        const float uneven =
            0.5f * B * Hkv * (ceil_div(3L * T, 4 * range) + ceil_div(5L * T, 4 * range));
        // CTAs of the one-tile form share an SM
        auto shared = [&](float ctas) { return tiles == 1 && ctas > sms ? 1.2f : 1.f; };
        for (int s = requested > 0 ? requested : 1;; s += 1 + s / 16) {
            const int splits = s < MAX_SPLITS ? s : MAX_SPLITS;
            const long ctas = items * splits;
            const float more = uneven * splits;
            const float rounds = (1.f - weight) * ceil_div(ctas, slots) * shared(ctas) +
                                 weight * fmaxf(1.f, more / slots) * shared(more);
            const int per = (blocks + splits - 1) / splits;
            float us = rounds * (tiles == 2 ? 1.3f * per + 5.f : 0.7f * per + 3.f);
            if (splits > 1)
                us += 2.5f + 0.08f * splits + (float)rows * splits * D * 1.35e-6f;
            if (us < least) {
                least = us;
                best = TokensPlan{tiles, splits};
            }
            // more splits than fill the card twice only add to the merge
            if (requested > 0 || s >= MAX_SPLITS || s >= blocks || ctas >= 2 * slots)
                break;
        }
    }
    return best;
}

cudaError_t launch_attend_tokens(const TokensLaunch &p, cudaStream_t s)
{
    // Which form: two tiles share the K and V blocks and win once an item is long; the one-tile
    // form's second CTA per SM works through the start and the end of the first one's items,
    // and its smaller items fill the card when there are few.  Uniform prompts of 16 / 2 heads
    // of 128, one against two tiles, us: 16 x 512 tokens 27.4 / 29.2, 8 x 1024 40.1 / 41.6,
    // 8 x 2048 113 / 110, 4 x 4096 200 / 185, 2 x 8192 379 / 349, but 1 x 2048 29.7 / 32.9;
    // 16 / 16 heads: 35.9 / 37.9, 44.1 / 45.6, 118 / 114, 214 / 193, 404 / 364, but 1 x 2048
    // 25.8 / 29.8.  Heads of 64 channels, whose time goes to the row threads, were faster with
    // one tile throughout (2 x 8192: 276 / 298).  A chunk's form comes with its plan.
    const long seqs = p.cu ? p.B : 1, pair = 2 * (TM / (p.Hq / p.Hkv));
    const bool few = (p.L / pair + seqs) * p.Hkv * (p.cu ? 1 : p.B) <= sm_count();
    const bool one = p.n ? p.tiles == 1 : p.L <= 1024 * seqs || few;
    if (p.mask)
        return p.D == 64 ? attend_tokens_impl<64, 1, true, true>(p, s)
               : one     ? attend_tokens_impl<128, 1, true, true>(p, s)
                         : attend_tokens_impl<128, 2, true, true>(p, s);
    if (p.n)
        return p.D == 64 ? attend_tokens_impl<64, 1, true>(p, s)
               : one     ? attend_tokens_impl<128, 1, true>(p, s)
                         : attend_tokens_impl<128, 2, true>(p, s);
    return p.D == 64 ? attend_tokens_impl<64, 1, false>(p, s)
           : one     ? attend_tokens_impl<128, 1, false>(p, s)
                     : attend_tokens_impl<128, 2, false>(p, s);
}

} // namespace kvc
