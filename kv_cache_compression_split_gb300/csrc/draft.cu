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
// be another one than 64-bit arithmetic draws.  64-bit floating point runs at two operations per
// clock and SM here, so a thread adds in pairs of 32-bit numbers: each addition's exact rounding
// error (Knuth's two-sum: six additions, without a branch) goes into a second sum, which is
// rounded itself.  Of a sum of N entries up to N^2 2^-49 of it is lost, 2^-37 at 64, and as a rule
// some 2^-48; 32-bit sums lose N 2^-25.  The pair becomes one 64-bit number of units 2^-52, and from there on all sums are
// integers, which add up in any order to the same.  The mass of the residual max(p - a q, 0) is
// sum p - a sum q over the tokens with p > a q: two such sums, a multiplied in once.  A token
// that the rounding of a moves across that border has a weight of 2^-24 of its probability.
constexpr int VER_THREADS = 256, VER_WARPS = VER_THREADS / 32;
constexpr int VER_UNROLL = 4;   // strips of 32 vectors in flight per warp
constexpr int MAX_CLUSTER = 16;
constexpr uint64_t ONE = 1ull << 52;          // a weight of 1 in fixed point
constexpr uint64_t A_MOST = 1024 * ONE;       // no distributions get there

// To [0, 1]; NaN becomes 0.
__device__ __forceinline__ float clean(float x) { return __saturatef(x); }

__device__ __forceinline__ uint64_t to_fixed(float x)
{
    return (uint64_t)__float2ll_rn(x * 4503599627370496.f);   // exact down to 2^-28, then rounded
}

// a times x, both of 2^-52, x at most 2
__device__ __forceinline__ uint64_t mul_fixed(uint64_t a, uint64_t x)
{
    return __umul64hi(a, x) << 12 | (a * x) >> 52;
}

__device__ __forceinline__ uint64_t less_fixed(uint64_t x, uint64_t y) { return x > y ? x - y : 0; }

// Sum of pairs of numbers with the rounding errors of its additions.
struct Sum2 {
    float2 sum = make_float2(0.f, 0.f), err = make_float2(0.f, 0.f);
    __device__ __forceinline__ void add(float2 x)
    {
        const float2 s = fadd2(sum, x), b = fsub2(s, sum);
        err = fadd2(err, fadd2(fsub2(sum, fsub2(s, b)), fsub2(x, b)));
        sum = s;
    }
    // both halves, at most 2
    __device__ __forceinline__ uint64_t fixed() const
    {
        const float s = __fadd_rn(sum.x, sum.y), b = __fsub_rn(s, sum.x);
        const float r = __fadd_rn(__fsub_rn(sum.x, __fsub_rn(s, b)), __fsub_rn(sum.y, b));
        const long long v = (long long)to_fixed(fminf(s, 2.f)) +
                            (long long)to_fixed(__fadd_rn(r, __fadd_rn(err.x, err.y)));
        return v < 0 ? 0 : min((uint64_t)v, 2 * ONE);
    }
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t x)
{
#pragma unroll
    for (int m = 16; m; m >>= 1)
        x += __shfl_xor_sync(ALL, (unsigned long long)x, m);
    return x;
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
    __device__ int vectors() const { return (int)(((unsigned)V + off + 3) / 4); }
    // entries i0 .. i0 + 3, those outside 0
    __device__ float4 load(int i0) const
    {
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
    uint64_t warp[2][VER_WARPS];
    uint64_t total[2][MAX_CLUSTER];   // the cluster's CTAs', written by them; two, used in turn
    float u_next;
    // the walk: at node cur, whose children up to node last have been refused
    uint64_t a;
    long long left;
    int cur, last, count, n_gone, ask;
};

// To the shared memory of CTA `rank` of this cluster, at the offset that `local` has in this CTA's.
__device__ __forceinline__ void st_cluster_u64(uint64_t *local, uint32_t rank, uint64_t v)
{
    uint32_t ra;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(smem_u32(local)), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(ra), "l"(v) : "memory");
}

// The weights of a row: max(p - a q, 0), or with a = 0 those of p without some tokens.  Of a
// range of vectors [v0, v1), by a warp.
struct Weights {
    Row p, q;
    uint64_t a;
    float ah;                // a in 32 bits
    const int *gone;         // tokens whose weight is 0
    int n_gone;

    // whether some token of the range is gone
    __device__ __forceinline__ bool patched(int v0, int v1) const
    {
        bool some = false;
        for (int k = threadIdx.x & 31; k < n_gone; k += 32) {
            const int v = (gone[k] + p.off) >> 2;
            some |= v >= v0 && v < v1;
        }
        return __any_sync(ALL, some);
    }
    __device__ __forceinline__ void keep(float4 &x, int i0) const
    {
#pragma unroll 1
        for (int k = 0; k < n_gone; ++k) {
            const int i = gone[k] - i0;
            x.x = i == 0 ? 0.f : x.x;
            x.y = i == 1 ? 0.f : x.y;
            x.z = i == 2 ? 0.f : x.z;
            x.w = i == 3 ? 0.f : x.w;
        }
    }
    // 1 where the weight is positive
    __device__ __forceinline__ float2 positive(float2 x, float2 y) const
    {
        const float2 d = ffma2(make_float2(-ah, -ah), y, x);
        return make_float2(d.x > 0.f ? 1.f : 0.f, d.y > 0.f ? 1.f : 0.f);
    }
    // p and q of the tokens that count
    __device__ __forceinline__ void split(float4 x, float4 y, float2 (&ps)[2], float2 (&qs)[2]) const
    {
        const float2 x0 = make_float2(clean(x.x), clean(x.y)), x1 = make_float2(clean(x.z), clean(x.w));
        const float2 y0 = make_float2(clean(y.x), clean(y.y)), y1 = make_float2(clean(y.z), clean(y.w));
        const float2 m0 = positive(x0, y0), m1 = positive(x1, y1);
        ps[0] = fmul2(x0, m0);
        ps[1] = fmul2(x1, m1);
        qs[0] = fmul2(y0, m0);
        qs[1] = fmul2(y1, m1);
    }
    // Vector v of any place and alignment.
    __device__ __forceinline__ void any_vector(int v, float2 (&ps)[2], float2 (&qs)[2]) const
    {
        const int i0 = 4 * v - p.off;
        float4 x = p.load(i0), y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (a)
            y = q.load(i0);
        keep(x, i0);
        split(x, y, ps, qs);
    }
    // Sum of the range's weights: whole vectors several strips of 32 at a time, the others (the row's
    // ends, the range's last strips, a q of another alignment than p's) strip by strip.  The last
    // strips in a predicated group took 75 us for 512 chains of 128000 tokens instead of 71.
    __device__ __forceinline__ uint64_t sum(int v0, int v1) const
    {
        constexpr int U = VER_UNROLL, W = 2 * U;     // as many loads in flight without q
        const int lane = threadIdx.x & 31;
        Sum2 sp, sq;
        int v = v0;
        float2 ps[2], qs[2];
        if (v < v1 && v == 0 && p.off) {         // the row's first vector is not whole
            if (lane < v1) {
                any_vector(lane, ps, qs);
                sp.add(ps[0]);
                sp.add(ps[1]);
                sq.add(qs[0]);
                sq.add(qs[1]);
            }
            v = min(32, v1);
        }
        const int whole = min(v1, (p.V + p.off) / 4);
        if (a && p.off == q.off) {
            const float4 *xs = reinterpret_cast<const float4 *>(p.at - p.off) + lane;
            const float4 *ys = reinterpret_cast<const float4 *>(q.at - q.off) + lane;
#pragma unroll 1
            for (; v + 32 * U <= whole; v += 32 * U) {
                float4 x[U], y[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    x[u] = xs[v + 32 * u];
                    y[u] = ys[v + 32 * u];
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    split(x[u], y[u], ps, qs);
                    sp.add(ps[0]);
                    sq.add(qs[0]);
                    sp.add(ps[1]);
                    sq.add(qs[1]);
                }
            }
        } else if (!a) {
            const bool patch = n_gone > 0 && patched(v0, v1);
            const float4 *xs = reinterpret_cast<const float4 *>(p.at - p.off) + lane;
#pragma unroll 1
            for (; v + 32 * W <= whole; v += 32 * W) {
                float4 x[W];
#pragma unroll
                for (int u = 0; u < W; ++u)
                    x[u] = xs[v + 32 * u];
                if (patch)
#pragma unroll
                    for (int u = 0; u < W; ++u)
                        keep(x[u], 4 * (v + 32 * u + lane) - p.off);
#pragma unroll
                for (int u = 0; u < W; ++u) {
                    sp.add(make_float2(clean(x[u].x), clean(x[u].y)));
                    sp.add(make_float2(clean(x[u].z), clean(x[u].w)));
                }
            }
        }
#pragma unroll 1
        for (v += lane; v < v1; v += 32) {
            any_vector(v, ps, qs);
            sp.add(ps[0]);
            sp.add(ps[1]);
            sq.add(qs[0]);
            sq.add(qs[1]);
        }
        const uint64_t total = min(warp_sum64(sp.fixed()), 2 * ONE);
        if (!a)
            return total;
        return less_fixed(total, mul_fixed(a, min(warp_sum64(sq.fixed()), 2 * ONE)));
    }
    // First token of the range at which the running sum (which is `below` before it) exceeds
    // `line`; the range's last token with a weight if roundings hide it.
    __device__ __forceinline__ int find(int v0, int v1, uint64_t below, uint64_t line) const
    {
        const int lane = threadIdx.x & 31;
        int last = -1;
#pragma unroll 1
        for (int v = v0; v < v1; v += 32) {
            const int i0 = 4 * (v + lane) - p.off;
            float2 ps[2], qs[2];
            if (v + lane < v1)
                any_vector(v + lane, ps, qs);
            else
                ps[0] = ps[1] = qs[0] = qs[1] = make_float2(0.f, 0.f);
            const float x[4] = {ps[0].x, ps[0].y, ps[1].x, ps[1].y};
            const float y[4] = {qs[0].x, qs[0].y, qs[1].x, qs[1].y};
            uint64_t w[4], upto = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                w[c] = to_fixed(x[c]);
                if (a)
                    w[c] = less_fixed(w[c], mul_fixed(a, to_fixed(y[c])));
                upto += w[c];
                last = x[c] > 0.f ? i0 + c : last;
            }
            const uint64_t mine = upto;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint64_t o = __shfl_up_sync(ALL, (unsigned long long)upto, off);
                upto += lane >= off ? o : 0;
            }
            const unsigned over = __ballot_sync(ALL, below + upto > line);
            if (over) {
                uint64_t run = below + upto - mine;
                int c = 0;
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    run += w[i];
                    c += run <= line;
                }
                return __shfl_sync(ALL, i0 + c, __ffs(over) - 1);
            }
            below += __shfl_sync(ALL, (unsigned long long)upto, 31);
        }
#pragma unroll
        for (int m = 16; m; m >>= 1)
            last = max(last, __shfl_xor_sync(ALL, last, m));
        return last;
    }
};

// Vectors of part `i` of `parts` of [v0, v1): whole strips of 32.  Returns the length of the first
// part, which no other one exceeds.
__device__ __forceinline__ int part_of(int &v0, int &v1, int i, int parts)
{
    const int per = ((v1 - v0 + parts - 1) / parts + 31) / 32 * 32;
    v0 = (int)min((long)v1, v0 + (long)i * per);
    v1 = min(v1, v0 + per);
    return per;
}

__global__ void __launch_bounds__(VER_THREADS, 4) k_draft_verify(const VerifyLaunch p, const int size)
{
    __shared__ VerShared s;
    const int b = blockIdx.x / size, rank = blockIdx.x - b * size;
    const int warp = __shfl_sync(ALL, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const bool drawn = p.q != nullptr;
    if (size > 1)
        cluster_arrive();        // waited for before the first store to another CTA
    bool joined = size == 1;
    int start, len;
    node_range(p.cu, b, p.T, MAX_NODES, p.status, start, len);
    if (threadIdx.x == 0 && len > 0)
        s.u_next = p.u_next[b];
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

    // The walk is warp 0's; its state waits in shared memory during the passes over a row: for the
    // residual's mass, then for the next token.
    if (threadIdx.x == 0) {
        s.path[0] = s.cur = s.last = s.n_gone = 0;
        s.count = len > 0 ? 1 : 0;
        s.a = 0;
        s.left = ONE;
    }
    Weights w{Row(nullptr, 0), Row(nullptr, 0), 0, 0.f, s.gone, 0};
    int phase = 0;               // which of the two totals is in use
    uint64_t at = 0, line = 0;   // sum in front of this CTA's, the owner's, the finder's range; the draw
    int owner = -1;              // the CTA's warp in whose range the next token lies
    int v0, v1;                  // this warp's range of vectors
    bool finder = false, none = true, plain = false;
    for (;;) {
        if (warp == 0 && owner < 0 && !plain) {
            __syncwarp();
            int cur = s.cur, j = s.last, count = s.count, n_gone = s.n_gone;
            uint64_t a = s.a;            // of 2^-52, like `left`, the mass S; of given tokens 0
            long long left = s.left;
            bool ask = false, have = true;   // `left` is that of a
            while (count > 0 && count < p.max_path) {
                int child = -1;
                for (int i = j + 1; i < len && child < 0; i += 32) {
                    const unsigned hit = __ballot_sync(ALL, i + lane < len && s.parent[i + lane] == cur);
                    child = hit ? i + __ffs(hit) - 1 : -1;
                }
                if (child < 0)
                    break;
                if (!have) {
                    ask = true;          // the residual's mass, from everybody
                    break;
                }
                // accepted iff u q S < p - a q; of given tokens q is 1 and a 0
                const int x = s.token[child];
                const float u = s.u[child], qx = drawn ? s.q[child] : 1.f;
                float px = s.p[child];
                if (n_gone > 0) {
                    bool again = false;
                    for (int k = lane; k < n_gone; k += 32)
                        again |= s.gone[k] == x;
                    px = __any_sync(ALL, again) ? 0.f : px;
                }
                bool take;
                if (a == 0 && left == (long long)ONE) {
                    take = __fmaf_rn(u, qx, -px) < 0.f;      // one rounding: the sign is exact
                } else {
                    // 32 bits where they are enough: 64-bit products take hundreds of clocks here
                    const float af = (float)a * (1.f / ONE), rhs = __fmaf_rn(-af, qx, px);
                    const float lhs = u * qx * ((float)left * (1.f / ONE));
                    take = lhs < rhs;
                    if (fabsf(lhs - rhs) <= (fabsf(lhs) + px + af * qx) * (1.f / (1 << 21))) {
                        const double wx = (double)px - (double)a * (1.0 / (double)ONE) * (double)qx;
                        take = wx > 0.0 && (double)u * (double)qx * ((double)left * (1.0 / (double)ONE)) < wx;
                    }
                }
                take = take && px > 0.f;
                j = child;
                if (take) {
                    cur = child;
                    a = 0;
                    left = ONE;
                    n_gone = 0;
                    if (lane == 0)
                        s.path[count] = child;
                    ++count;
                } else if (drawn) {
                    a = min(a + (uint64_t)left, A_MOST);
                    have = false;
                } else {
                    left -= (long long)to_fixed(px);
                    if (lane == 0)
                        s.gone[n_gone] = x;
                    ++n_gone;
                }
                __syncwarp();
            }
            if (lane == 0) {
                s.ask = ask;
                s.cur = cur;
                s.last = j;
                s.count = count;
                s.n_gone = n_gone;
                s.a = a;
            }
        }
        __syncthreads();
        if (len == 0)
            break;
        // Sum of the weights of node cur's row, in every thread of the cluster; or, when the next
        // token's place is known to lie in warp `owner`'s range, of the parts of that range.
        w.a = plain ? 0 : s.a;
        w.ah = (float)w.a * (1.f / ONE);
        w.n_gone = plain ? 0 : s.n_gone;
        w.p = Row(p.p + (start + s.cur) * p.ps, p.V);
        w.q = Row(w.a ? p.q + (start + s.cur) * p.qs : nullptr, p.V);
        v0 = 0;
        v1 = w.p.vectors();
        const int per = part_of(v0, v1, rank * VER_WARPS + (owner < 0 ? warp : owner), size * VER_WARPS);
        if (owner >= 0)
            part_of(v0, v1, warp, VER_WARPS);
        const uint64_t mine = w.sum(v0, v1);
        if (lane == 0)
            s.warp[owner >= 0][warp] = mine;
        __syncthreads();
        if (owner >= 0) {
            int part = -1;
            uint64_t from = at;
#pragma unroll
            for (int i = 0; i < VER_WARPS; ++i) {
                const uint64_t x = s.warp[1][i];
                if (part < 0) {
                    if (line - from < x)
                        part = i;
                    else
                        from += x;
                }
            }
            if (part >= 0) {
                at = from;
            } else {             // roundings of the parts hide it: the whole range
                v0 = 0;
                v1 = w.p.vectors();
                part_of(v0, v1, rank * VER_WARPS + owner, size * VER_WARPS);
            }
            finder = warp == max(part, 0);
            break;
        }
        uint64_t total = 0;
#pragma unroll
        for (int i = 0; i < VER_WARPS; ++i)
            total += s.warp[0][i];
        at = 0;
        if (size > 1) {
            if (!joined)         // every CTA of the cluster runs: its shared memory may be written
                cluster_wait();
            joined = true;
            if (threadIdx.x < size)
                st_cluster_u64(&s.total[phase][rank], threadIdx.x, total);
            cluster_sync_all();
            total = 0;
#pragma unroll 4
            for (int i = 0; i < size; ++i) {
                const uint64_t x = s.total[phase][i];
                at += i < rank ? x : 0;
                total += x;
            }
            phase ^= 1;
        }
        if (s.ask) {
            if (threadIdx.x == 0)
                s.left = (long long)total;
        } else if (total > 0) {
            none = false;
            const float u = fminf(fmaxf(s.u_next, 0.f), 0x1.fffffep-1f);
            line = __umul64hi(__float2ull_rz(u * 18446744073709551616.f), total);
            if (line < at)
                break;
#pragma unroll
            for (int i = 0; i < VER_WARPS; ++i) {
                const uint64_t x = s.warp[0][i];
                if (owner < 0) {
                    if (line - at < x)
                        owner = i;
                    else
                        at += x;
                }
            }
            finder = warp == owner;
            if (owner < 0 || per <= 32 * VER_UNROLL)   // another CTA's, or short: no parts
                break;
        } else {
            if (!w.a && !w.n_gone)
                break;
            plain = true;        // nothing of p is left: p itself
        }
        __syncthreads();         // what warp 0 wrote, and the warps' sums, have been read
    }

    if (finder) {
        const int token = w.find(v0, v1, at, line);
        if (lane == 0)
            p.next_token[b] = token;
    }
    if (rank == 0) {
        if (threadIdx.x == 0) {
            p.count[b] = s.count;
            if (none)
                p.next_token[b] = -1;
        }
        for (int i = threadIdx.x; i < p.max_path; i += VER_THREADS)
            p.path[(size_t)b * p.max_path + i] = i < s.count ? s.path[i] : -1;
    }
    if (!joined)
        cluster_wait();
}

// ------------------------------------------------------------------ the accepted path's rows

// A CTA per unit.  Rows move down (path[i] >= i), so a group of rows is read whole before it is
// written, and the rows that later groups read lie behind it.  What bounds it is the chain of
// loads: range, counts and path together, then the page table, then the rows.
constexpr int COMMIT_THREADS = 128, COMMIT_UNROLL = 2;

template <int D>
__global__ void __launch_bounds__(COMMIT_THREADS) k_draft_commit(const CommitLaunch p)
{
    constexpr int CHUNKS = D / 8;                               // of 16 bytes per row
    constexpr int AT_ONCE = COMMIT_THREADS / (2 * CHUNKS);      // rows of K and V per step
    __shared__ int s_path[COMMIT_THREADS];                      // the path's first nodes
    const int unit = blockIdx.x, b = unit / p.Hkv;
    const int32_t *path = p.path + (size_t)b * p.max_path;
    const int start = p.cu[b], end = p.cu[b + 1], count = p.count[b];
    const int n = p.n[unit], seqlen = p.seqlen[b];
    int x = -1, before = -1;
    if (threadIdx.x < p.max_path) {
        x = path[threadIdx.x];
        before = threadIdx.x ? path[threadIdx.x - 1] : -1;
    }
    s_path[threadIdx.x] = x;
    const int m = end - start;
    bool ok = start >= 0 && start <= end && end <= p.T && count >= 0 && count <= m &&
              count <= p.max_path;
    const bool fits = n >= m && n <= p.C;
    bool refused = ok && m > 0 && p.slot_map &&
                   p.slot_map[(size_t)start * p.Hkv + unit % p.Hkv] < 0;
    const SlotRows rows{p.table, p.C, p.num_pages};
    if (refused && fits && p.table) {
        // A unit whose first new slot lies on no page has no row for node 0 either, and took its
        // nodes.  In its case every node without a row is on such a slot; of a refused unit the
        // slots looked at are older ones, on pages that it holds.
        bool page = false;
        for (int i = threadIdx.x; i < m; i += COMMIT_THREADS)
            page |= p.slot_map[(size_t)(start + i) * p.Hkv + unit % p.Hkv] < 0 &&
                    rows.row(unit, n - m + i) >= 0;
        refused = __syncthreads_or(page);
    }
    if (ok) {
        if (threadIdx.x < count)
            ok = x > before && x < m;
        for (int i = threadIdx.x + COMMIT_THREADS; i < count; i += COMMIT_THREADS)
            ok = ok && path[i] > path[i - 1] && path[i] < m;
    }
    ok = !__syncthreads_or(!ok);
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
    for (int i0 = 0; i0 < count; i0 += AT_ONCE * COMMIT_UNROLL) {
        uint4 y[COMMIT_UNROLL];
        long from[COMMIT_UNROLL], to[COMMIT_UNROLL];
#pragma unroll
        for (int u = 0; u < COMMIT_UNROLL; ++u) {
            const int i = i0 + u * AT_ONCE + row;
            from[u] = to[u] = -1;
            if (i < count) {
                const int node = i < COMMIT_THREADS ? s_path[i] : path[i];
                if (node != i) {
                    from[u] = rows.row(unit, n - m + node);
                    to[u] = rows.row(unit, n - m + i);
                    if (from[u] < 0 || to[u] < 0) {
                        flag_error(p.status, DEV_CAPACITY);
                        to[u] = -1;
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < COMMIT_UNROLL; ++u)
            if (to[u] >= 0)
                y[u] = *reinterpret_cast<const uint4 *>(base + from[u] * D);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < COMMIT_UNROLL; ++u)
            if (to[u] >= 0)
                *reinterpret_cast<uint4 *>(base + to[u] * D) = y[u];
    }
}

} // namespace

cudaError_t launch_tree_plan(const TreePlanLaunch &p, cudaStream_t s)
{
    k_tree_plan<<<p.B, PLAN_THREADS, 0, s>>>(p);
    return cudaGetLastError();
}

// CTAs per sequence.  A pass over a row costs a cluster barrier and what a CTA reads, and many
// sequences fill the card by themselves: the more there are, the longer a CTA's part has to be.
// Measured in a graph, us, with 1 / 2 / 4 / 8 / 16 CTAs (drawn trees of up to 6 nodes): one sequence
// of 32000 tokens 9.4 / 8.7 / 7.7 / 8.3 / 7.0, of 128000 18.3 / 15.5 / 10.9 / 8.8 / 8.1; 64 sequences
// of 32000 22.6 / 18.5 / 15.6 / 16.1 / 24.2, of 128000 73 / 47 / 31 / 24 / 29; 512 of 32000
// 41 / 40 / 48 / 78 / 153, of 128000 96 / 80 / 68 / 79 / 133; 1000 tokens take one CTA at any number.
int verify_ctas(int B, int V)
{
    const int part = 1900 + 64 * (B < 256 ? B : 256), most = B >= 128 ? 4 : B > 32 ? 8 : MAX_CLUSTER;
    int size = 1;
    while (2 * size <= most && V / part >= 2 * size)
        size *= 2;
    return size;
}

cudaError_t launch_draft_verify(const VerifyLaunch &p, cudaStream_t s)
{
    const int size = verify_ctas(p.B, p.V);
    const void *kernel = reinterpret_cast<const void *>(k_draft_verify);
    if (size > 8) {
        const cudaError_t e = allow_large_clusters_once(kernel);
        if (e != cudaSuccess)
            return e;
    }
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
