// draft.cu -- trees of drafted tokens around their attention: the nodes' masks and positions
// (kvc_tree_plan), which nodes the target's probabilities accept and the token behind them
// (kvc_draft_verify), and the cache back on the accepted path (kvc_draft_commit).
#include "kvc_device.cuh"
#include "kvc_internal.h"

#include <math.h>

namespace kvc {

namespace {

constexpr int MAX_NODES = KVC_TREE_MAX_NODES;
constexpr unsigned ALL = 0xffffffffu;

// First token and nodes of sequence b; a range that leaves [0, T] or is longer than `most`
// counts as empty and is reported.
__device__ __forceinline__ void node_range(const int32_t *cu, int b, int T, int most, int *status,
                                           int &start, int &len)
{
    start = cu[b];
    const int end = cu[b + 1];
    len = 0;
    if (start >= 0 && start <= end && end <= T && end - start <= most)
        len = end - start;
    else if (threadIdx.x == 0)
        flag_error(status, DEV_CAPACITY);
}

// ------------------------------------------------------------------ masks and positions

// A CTA per sequence, its parents in shared memory; each thread walks from its node to the
// root, setting a bit per node on the way.
constexpr int PLAN_THREADS = 128;

__global__ void __launch_bounds__(PLAN_THREADS) k_tree_plan(const TreePlanLaunch p)
{
    constexpr int WORDS = MAX_NODES / 64;
    __shared__ int16_t s_parent[MAX_NODES];
    int start, len;
    node_range(p.cu, blockIdx.x, p.T, 64 * p.words, p.status, start, len);
    const int base = p.seqlen ? p.seqlen[blockIdx.x] : 0;
    for (int i = threadIdx.x; i < len; i += PLAN_THREADS) {
        int x = p.parent[start + i];
        if (x < -1 || x >= i) {
            flag_error(p.status, DEV_CAPACITY);
            x = -1;
        }
        s_parent[i] = (int16_t)x;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < len; i += PLAN_THREADS) {
        uint64_t bits[WORDS] = {};
        int depth = -1;
        for (int x = i; x >= 0; x = s_parent[x]) {
#pragma unroll
            for (int w = 0; w < WORDS; ++w)
                bits[w] |= x >> 6 == w ? 1ull << (x & 63) : 0ull;
            ++depth;
        }
        uint64_t *to = p.mask + (size_t)(start + i) * p.words;
#pragma unroll
        for (int w = 0; w < WORDS; ++w)
            if (w < p.words)
                to[w] = bits[w];
        if (p.pos)
            p.pos[start + i] = base + depth;
    }
}

// ------------------------------------------------------------------ verification

// A cluster of CTAs per sequence.  Every CTA walks the tree by itself, from the same numbers
// and so to the same end; the cluster's CTAs share the passes over rows of the vocabulary.
//
// Sums.  A running sum of V probabilities decides between neighbours that are 2^-24 apart and
// less, and there are V borders: with 32-bit sums (off by 10^-8) one token in a few hundred would
// be another one than 64-bit arithmetic draws.  So a weight is taken apart exactly: with
// t = w + 1 the bits of t count units of 2^-23, what is left counts units of 2^-46 in the same
// way, and what is left of that is below 2^-47 and summed in 32 bits.  A thread's three
// sums become one 64-bit number of units 2^-52, and these add up in any order to the same.
constexpr int VER_THREADS = 256, VER_WARPS = VER_THREADS / 32;
constexpr int VER_UNROLL = 4;                 // strips of 32 vectors in flight per warp
constexpr uint64_t ONE = 1ull << 52;          // a weight of 1 in fixed point

__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, 0.f), 1.f); }

// Weight p - a q of a token, where positive, as a sum of two floats; a is a sum of two, too.
struct Weight {
    float w, rest;
    __device__ Weight(float p, float q, float ah, float al)
    {
        const float h = __fmul_rn(ah, q), l = __fmaf_rn(ah, q, -h);
        const float d = __fsub_rn(p, h), b = __fsub_rn(d, p);
        const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(h, b));
        const float lo = __fmaf_rn(-al, q, __fsub_rn(e, l));
        const float s = __fadd_rn(d, lo);
        w = s > 0.f ? s : 0.f;
        rest = s > 0.f ? __fsub_rn(lo, __fsub_rn(s, d)) : 0.f;
    }
    __device__ explicit Weight(float p) : w(p), rest(0.f) {}
};

struct Sum {
    uint32_t hi = 0, lo = 0;
    float rest = 0.f;
    __device__ void add(const Weight &x)
    {
        constexpr float M = 1.5f / (1 << 23);
        const float t = __fadd_rn(x.w, 1.f);
        hi += __float_as_uint(t) - __float_as_uint(1.f);
        const float l = __fadd_rn(__fsub_rn(x.w, __fsub_rn(t, 1.f)), x.rest);
        const float t2 = __fadd_rn(l, M);
        lo += __float_as_uint(t2) - __float_as_uint(M);
        rest = __fadd_rn(rest, __fsub_rn(l, __fsub_rn(t2, M)));
    }
    // not negative but for a rounding of weights near 0
    __device__ uint64_t fixed() const
    {
        const long long x = ((long long)hi << 29) + ((long long)(int32_t)lo << 6) +
                            __float2ll_rn(rest * 4503599627370496.f);
        return x > 0 ? (uint64_t)x : 0;
    }
};

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t x, int m)
{
    return __shfl_xor_sync(ALL, (unsigned long long)x, m);
}

// A row of the vocabulary in vectors of four entries that begin on 16-byte boundaries: vector
// v holds the entries 4 v - off .. 4 v - off + 3, of which those in [0, V) count.
struct Row {
    const float *at;
    int off, V;
    __device__ Row(const float *row, int V_) : at(row), V(V_)
    {
        off = (int)(reinterpret_cast<uintptr_t>(row) >> 2 & 3);
    }
    __device__ int vectors() const { return (V + off + 3) / 4; }
    // entries i0 .. i0 + 3; this row's own vectors are loaded whole
    __device__ float4 load(int i0) const
    {
        if (i0 >= 0 && i0 + 3 < V && ((i0 + off) & 3) == 0)
            return *reinterpret_cast<const float4 *>(at + i0);
        float4 x;
        x.x = i0 >= 0 && i0 < V ? at[i0] : 0.f;
        x.y = i0 + 1 >= 0 && i0 + 1 < V ? at[i0 + 1] : 0.f;
        x.z = i0 + 2 >= 0 && i0 + 2 < V ? at[i0 + 2] : 0.f;
        x.w = i0 + 3 >= 0 && i0 + 3 < V ? at[i0 + 3] : 0.f;
        return x;
    }
};

struct VerShared {
    int parent[MAX_NODES], token[MAX_NODES];
    float u[MAX_NODES], p[MAX_NODES], q[MAX_NODES];
    int path[MAX_NODES], gone[MAX_NODES];
    uint64_t warp[VER_WARPS];
    uint64_t total[2];       // this CTA's, read by the cluster; two, used in turn
    int cur, count, n_gone, ask;
    float ah, al;
};

__device__ __forceinline__ uint64_t ld_cluster_u64(const uint64_t *local, uint32_t rank)
{
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(local)), "r"(rank));
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(ra) : "memory");
    return v;
}

// The weights of a row, dealt to the cluster's warps in contiguous ranges of vectors.
struct Weights {
    Row p, q;
    bool residual;           // p - a q; else p
    float ah, al;
    const int *gone;         // tokens whose weight is 0
    int n_gone;
    int v0, v1;              // this warp's vectors

    __device__ __forceinline__ void load(int v, float4 &x, float4 &y) const
    {
        const int i0 = 4 * v - p.off;
        x = y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (v < v1) {
            x = p.load(i0);
            if (residual)
                y = q.load(i0);
        }
    }
    __device__ __forceinline__ float4 kept(int v, float4 x) const
    {
        const int i0 = 4 * v - p.off;
        for (int k = 0; k < n_gone; ++k) {
            const int i = gone[k] - i0;
            x.x = i == 0 ? 0.f : x.x;
            x.y = i == 1 ? 0.f : x.y;
            x.z = i == 2 ? 0.f : x.z;
            x.w = i == 3 ? 0.f : x.w;
        }
        return x;
    }
    __device__ __forceinline__ Weight weight(float x, float y) const
    {
        return residual ? Weight(clean(x), clean(y), ah, al) : Weight(clean(x));
    }
    // Sum of this warp's weights (at most 2, which no distribution reaches).
    __device__ uint64_t sum() const
    {
        const int lane = threadIdx.x & 31;
        uint64_t all = 0;
        for (int v = v0 + lane; v - lane < v1; v += 32 * VER_UNROLL) {
            float4 x[VER_UNROLL], y[VER_UNROLL];
#pragma unroll
            for (int u = 0; u < VER_UNROLL; ++u)
                load(v + 32 * u, x[u], y[u]);
            Sum s;
#pragma unroll
            for (int u = 0; u < VER_UNROLL; ++u) {
                if (n_gone)
                    x[u] = kept(v + 32 * u, x[u]);
                s.add(weight(x[u].x, y[u].x));
                s.add(weight(x[u].y, y[u].y));
                s.add(weight(x[u].z, y[u].z));
                s.add(weight(x[u].w, y[u].w));
            }
            all = min(all + s.fixed(), 2 * ONE);
        }
#pragma unroll
        for (int m = 16; m; m >>= 1)
            all += shfl_xor64(all, m);
        return min(all, 2 * ONE);
    }
    // First token of this warp's range at which the running sum (which is `below` before it)
    // exceeds `line`; the range's last token with a weight if roundings hide it.
    __device__ int find(uint64_t below, uint64_t line) const
    {
        const int lane = threadIdx.x & 31;
        int last = -1;
        for (int v = v0 + lane; v - lane < v1; v += 32) {
            float4 x, y;
            load(v, x, y);
            x = kept(v, x);
            const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
            uint64_t f[4], own = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const Weight w = weight(xs[c], ys[c]);
                Sum s;
                s.add(w);
                f[c] = s.fixed();
                own += f[c];
                last = w.w > 0.f ? 4 * v - p.off + c : last;
            }
            uint64_t upto = own;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint64_t o = __shfl_up_sync(ALL, (unsigned long long)upto, off);
                upto += lane >= off ? o : 0;
            }
            const unsigned over = __ballot_sync(ALL, below + upto > line);
            if (over) {
                uint64_t at = below + upto - own;
                int token = -1;
#pragma unroll
                for (int c = 3; c >= 0; --c) {
                    uint64_t to = at;
#pragma unroll
                    for (int k = 0; k <= c; ++k)
                        to += f[k];
                    token = to > line ? 4 * v - p.off + c : token;
                }
                return __shfl_sync(ALL, token, __ffs(over) - 1);
            }
            below += __shfl_sync(ALL, (unsigned long long)upto, 31);
        }
#pragma unroll
        for (int m = 16; m; m >>= 1)
            last = max(last, __shfl_xor_sync(ALL, last, m));
        return last;
    }
};

__global__ void __launch_bounds__(VER_THREADS) k_draft_verify(const VerifyLaunch p, const int size)
{
    __shared__ VerShared s;
    const int b = blockIdx.x / size, rank = blockIdx.x - b * size;
    const int warp = __shfl_sync(ALL, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const bool drawn = p.q != nullptr;
    int start, len;
    node_range(p.cu, b, p.T, MAX_NODES, p.status, start, len);
    for (int i = threadIdx.x; i < len; i += VER_THREADS) {
        int up = p.parent ? p.parent[start + i] : i - 1;
        const int x = p.tokens[start + i];
        if (up < -1 || up >= i) {
            flag_error(p.status, DEV_CAPACITY);
            up = -1;
        }
        const bool in = up >= 0 && x >= 0 && x < p.V;
        s.parent[i] = up;
        s.token[i] = x;
        s.u[i] = p.u[start + i];
        s.p[i] = in ? clean(p.p[(start + up) * p.ps + x]) : 0.f;
        s.q[i] = in && drawn ? clean(p.q[(start + up) * p.qs + x]) : 0.f;
    }
    __syncthreads();

    int phase = 0;           // which of the two totals is in use
    uint64_t below = 0;      // sum of the weights in front of this warp's range
    Weights w{Row(nullptr, 0), Row(nullptr, 0), false, 0.f, 0.f, s.gone, 0, 0, 0};
    // Sum over the row of node c; in every thread of the cluster.
    auto row_sum = [&](int c, bool residual, float ah, float al, int n_gone) -> uint64_t {
        w.p = Row(p.p + (start + c) * p.ps, p.V);
        w.q = Row(residual ? p.q + (start + c) * p.qs : nullptr, p.V);
        w.residual = residual;
        w.ah = ah;
        w.al = al;
        w.n_gone = n_gone;
        const int vectors = w.p.vectors();
        const int per = ((vectors + size * VER_WARPS - 1) / (size * VER_WARPS) + 31) / 32 * 32;
        w.v0 = min(vectors, (rank * VER_WARPS + warp) * per);
        w.v1 = min(vectors, w.v0 + per);
        const uint64_t mine = w.sum();
        if (lane == 0)
            s.warp[warp] = mine;
        __syncthreads();
        uint64_t total = 0;
        below = 0;
#pragma unroll
        for (int i = 0; i < VER_WARPS; ++i) {
            const uint64_t x = s.warp[i];
            below += i < warp ? x : 0;
            total += x;
        }
        if (size > 1) {
            s.total[phase] = total;
            cluster_sync_all();
            total = 0;
            for (int i = 0; i < size; ++i) {
                const uint64_t x = ld_cluster_u64(&s.total[phase], i);
                below += i < rank ? x : 0;
                total += x;
            }
            phase ^= 1;
        }
        __syncthreads();     // s.warp is free again
        return total;
    };

    // The walk, by warp 0: what lies behind (cur, j) is the same in all its lanes.
    int cur = 0, j = 0, count = len > 0 ? 1 : 0, n_gone = 0;
    double a = 0.0, left = 1.0;
    bool have = true;        // `left` is that of a
    if (threadIdx.x == 0)
        s.path[0] = 0;
    for (;;) {
        if (warp == 0) {
            bool ask = false;
            while (count > 0 && count < p.max_path) {
                int child = -1;
                for (int i = j + 1; i < len && child < 0; i += 32) {
                    const unsigned hit = __ballot_sync(ALL, i + lane < len && s.parent[i + lane] == cur);
                    child = hit ? i + __ffs(hit) - 1 : -1;
                }
                if (child < 0)
                    break;
                if (!have) {
                    ask = true;      // the residual's mass, from everybody
                    break;
                }
                const int x = s.token[child];
                const double u = s.u[child], qx = s.q[child];
                double wx = s.p[child];
                bool take;
                if (drawn) {
                    wx -= a * qx;
                    take = wx > 0.0 && u * qx * left < wx;
                } else {
                    bool again = false;
                    for (int k = lane; k < n_gone; k += 32)
                        again |= s.gone[k] == x;
                    if (__any_sync(ALL, again))
                        wx = 0.0;
                    take = wx > 0.0 && u * left < wx;
                }
                j = child;
                if (take) {
                    cur = child;
                    a = 0.0;
                    left = 1.0;
                    n_gone = 0;
                    if (lane == 0)
                        s.path[count] = child;
                    ++count;
                } else if (drawn) {
                    a += left;
                    have = false;
                } else {
                    left -= wx;
                    if (lane == 0)
                        s.gone[n_gone] = x;
                    ++n_gone;
                }
                __syncwarp();
            }
            if (lane == 0) {
                s.ask = ask;
                s.cur = cur;
                s.count = count;
                s.n_gone = n_gone;
                s.ah = (float)a;
                s.al = (float)(a - (double)(float)a);
            }
        }
        __syncthreads();
        if (!s.ask)
            break;
        const uint64_t sum = row_sum(s.cur, true, s.ah, s.al, 0);
        left = (double)sum * (1.0 / (double)ONE);
        have = true;
    }

    // The next token, and the path.
    uint64_t total = 0;
    if (len > 0) {
        const bool residual = s.ah > 0.f;
        total = row_sum(s.cur, residual, s.ah, s.al, s.n_gone);
        if (total == 0 && (residual || s.n_gone))
            total = row_sum(s.cur, false, 0.f, 0.f, 0);
    }
    if (total > 0) {
        const float u = fminf(fmaxf(p.u_next[b], 0.f), 0x1.fffffep-1f);
        const uint64_t line = __umul64hi(__float2ull_rz(u * 18446744073709551616.f), total);
        if (line >= below && line - below < s.warp[warp]) {
            const int token = w.find(below, line);
            if (lane == 0)
                p.next_token[b] = token;
        }
    }
    if (rank == 0) {
        if (threadIdx.x == 0) {
            p.count[b] = s.count;
            if (total == 0)
                p.next_token[b] = -1;
        }
        for (int i = threadIdx.x; i < p.max_path; i += VER_THREADS)
            p.path[(size_t)b * p.max_path + i] = i < s.count ? s.path[i] : -1;
    }
    if (size > 1)
        cluster_sync_all();  // a CTA's totals are read by the others
}

// ------------------------------------------------------------------ the accepted path's rows

// A CTA per unit.  Rows move down (path[i] >= i), so a group of rows is read whole before it is
// written, and the rows that later groups read lie behind it.
constexpr int COMMIT_THREADS = 128, COMMIT_UNROLL = 4;

template <int D>
__global__ void __launch_bounds__(COMMIT_THREADS) k_draft_commit(const CommitLaunch p)
{
    constexpr int CHUNKS = D / 8;                               // of 16 bytes per row
    constexpr int AT_ONCE = COMMIT_THREADS / (2 * CHUNKS);      // rows of K and V per step
    const int unit = blockIdx.x, b = unit / p.Hkv;
    const int start = p.cu[b], end = p.cu[b + 1], count = p.count[b];
    const int n = p.n[unit], seqlen = p.seqlen[b];
    const int m = end - start;
    const int32_t *path = p.path + (size_t)b * p.max_path;
    bool ok = start >= 0 && start <= end && end <= p.T && count >= 0 && count <= m &&
              count <= p.max_path;
    if (ok)
        for (int i = threadIdx.x; i < count; i += COMMIT_THREADS) {
            const int x = path[i], before = i ? path[i - 1] : -1;
            ok = ok && x > before && x < m;
        }
    ok = !__syncthreads_or(!ok);
    const bool refused = ok && m > 0 && p.slot_map && p.slot_map[(size_t)start * p.Hkv + unit % p.Hkv] < 0;
    const bool fits = n >= m && n <= p.C;
    if (threadIdx.x == 0) {
        if (!ok || (!refused && !fits))
            flag_error(p.status, DEV_CAPACITY);
        p.n_out[unit] = ok && fits && !refused ? n - m + count : n;
        if (unit % p.Hkv == 0)
            p.seqlen_out[b] = ok ? seqlen - m + count : seqlen;
    }
    if (!ok || refused || !fits)
        return;
    const int row = threadIdx.x / (2 * CHUNKS), part = threadIdx.x % (2 * CHUNKS);
    uint16_t *base = (part < CHUNKS ? p.K : p.V) + part % CHUNKS * 8;
    const SlotRows rows{p.table, p.C, p.num_pages};
    for (int i0 = 0; i0 < count; i0 += AT_ONCE * COMMIT_UNROLL) {
        uint4 x[COMMIT_UNROLL];
        long to[COMMIT_UNROLL];
#pragma unroll
        for (int u = 0; u < COMMIT_UNROLL; ++u) {
            const int i = i0 + u * AT_ONCE + row;
            to[u] = -1;
            if (i < count && path[i] != i) {
                const long from = rows.row(unit, n - m + path[i]);
                to[u] = rows.row(unit, n - m + i);
                if (from < 0 || to[u] < 0) {
                    flag_error(p.status, DEV_CAPACITY);
                    to[u] = -1;
                } else {
                    x[u] = *reinterpret_cast<const uint4 *>(base + from * D);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < COMMIT_UNROLL; ++u)
            if (to[u] >= 0)
                *reinterpret_cast<uint4 *>(base + to[u] * D) = x[u];
    }
}

} // namespace

cudaError_t launch_tree_plan(const TreePlanLaunch &p, cudaStream_t s)
{
    k_tree_plan<<<p.B, PLAN_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_draft_verify(const VerifyLaunch &p, cudaStream_t s)
{
    const int size = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.B * size);
    cfg.blockDim = dim3(VER_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = size;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_draft_verify, p, size);
}

cudaError_t launch_draft_commit(const CommitLaunch &p, cudaStream_t s)
{
    if (p.D == 64)
        k_draft_commit<64><<<p.B * p.Hkv, COMMIT_THREADS, 0, s>>>(p);
    else
        k_draft_commit<128><<<p.B * p.Hkv, COMMIT_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

} // namespace kvc
