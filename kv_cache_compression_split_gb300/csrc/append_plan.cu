// append_plan.cu -- where the new tokens of a ragged batch go.
//
// kvc_append_plan: per (sequence, KV head) unit with n slots and m new tokens
//   need = ceil((n + m) / 64) pages, grow = max(0, need - held),
//   back = max(0, held - need) when pages are to be released.
// A unit's new pages are the next `grow` ones from the top of the free stack, in
// unit order, so every unit needs the sum of grow over the units before it; the
// returned pages go on what is left of the stack, placed by the same sum of back.
// Integer work of a few bytes per unit and token: latency bound.  One thread-block
// cluster scans the units, since the sums run over all of them: every CTA its range, the
// totals through distributed shared memory.  The outputs may be the inputs: of the old state
// only the stack's taken pages and the table's returned entries are read after the cluster
// barrier, the latter by the thread that then writes them, and a second barrier lies between
// the taking and the returned pages that go on the same stack.  What has many words is dealt
// evenly over threads that find their unit by bisecting the sums.
// 512 sequences of 8 heads, one new token each: 10.4 to 10.7 us in a graph, of which an empty
// batch takes 7 (the cluster's start, one round of loads, the barrier) and the copy of the
// 0.5 MB table and the 0.5 MB stack to other arrays, by these eight SMs, most of the rest; 96
// ragged prompts, 33 K tokens: 12.3 to 12.9 us (a kernel on all SMs writes their slot map).
//
// kvc_append_packed: one 16-byte chunk of a K and of a V row per thread and step,
// written to the row that the slot map names.  HBM bound: 2 D bytes read and
// written per row, twice.  35 K tokens of 8 heads of 128: 291 MB in 46.5 us in a graph,
// 6.2 TB/s, 0.92 of the measured copy rate, and 48.5 us by single calls, 0.88.
#include "kvc_device.cuh"
#include "kvc_internal.h"

namespace kvc {

namespace {

constexpr int CTAS = 8;        // one cluster (16 CTAs start 2.6 us later)
constexpr int THREADS = 1024;
constexpr int CU_CACHE = 2048; // sequence starts held in shared memory
constexpr int HEADS = 8;       // heads of a token whose loads are in flight together
// Tokens whose slot map the cluster writes itself: beyond the first of each unit, single
// words in many lines, which eight SMs take long over (8 x 1024 tokens of 8 heads: 79 us,
// 12 us with the second kernel; 128 x 4 tokens 17.4 against 16.8; 64 x 1 11.9 against 12.4).
constexpr int CLUSTER_TOKENS = 512;
constexpr int PLAN_MAX_SPAN = KVC_PLAN_MAX_UNITS / (CTAS * THREADS);

__device__ __forceinline__ int ld_cluster_s32(const int *local, uint32_t rank)
{
    return __float_as_int(ld_cluster_f32(reinterpret_cast<const float *>(local), rank));
}

// New tokens of sequence b: 0 when its range leaves [0, T].
__device__ __forceinline__ int new_tokens(const PlanLaunch &p, int b, int &start)
{
    start = p.cu[b];
    const int m = p.cu[b + 1] - start;
    return start < 0 || start > p.T || m < 0 || m > p.T - start ? 0 : m;
}

// Whether a unit of n slots has room for m more.
__device__ __forceinline__ bool fits(const PlanLaunch &p, int n, int m)
{
    return n >= 0 && n <= p.C - m;
}

// Exclusive scans of three counts over the CTA's threads, and their totals.
__device__ __forceinline__ void scan3(int (&x)[3], int (&total)[3])
{
    __shared__ int s_x[3][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int in[3] = {x[0], x[1], x[2]};
#pragma unroll
    for (int off = 1; off < 32; off <<= 1)
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int y = __shfl_up_sync(0xffffffffu, in[k], off);
            in[k] += lane >= off ? y : 0;
        }
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < 3; ++k)
            s_x[k][warp] = in[k];
    __syncthreads();
    if (warp < 3) {
        int w = s_x[warp][lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, off);
            w += lane >= off ? y : 0;
        }
        s_x[warp][lane] = w;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        x[k] = in[k] - x[k] + (warp ? s_x[k][warp - 1] : 0);
        total[k] = s_x[k][31];
    }
}

// dst[i] = src[i] for i in [0, n), by the whole cluster, 16 bytes at a time where both are
// aligned, four loads in flight per thread.
__device__ __forceinline__ void copy_i32(int32_t *dst, const int32_t *src, long n, int gtid)
{
    constexpr int U = 4;
    const long gsize = CTAS * THREADS;
    long done = 0;
    if (((reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(src)) & 15) == 0) {
        const long n4 = n / 4;
        for (long i = gtid; i < n4; i += U * gsize) {
            int4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u * gsize < n4)
                    x[u] = reinterpret_cast<const int4 *>(src)[i + u * gsize];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i + u * gsize < n4)
                    reinterpret_cast<int4 *>(dst)[i + u * gsize] = x[u];
        }
        done = 4 * n4;
    }
    for (long i = done + gtid; i < n; i += gsize)
        dst[i] = src[i];
}

// The last index whose value is at most x, in v[0] = 0, v[1], ..., v[n], none smaller than
// the one before it.
__device__ __forceinline__ int last_at_most(const int *v, int n, int x)
{
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (v[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Row of the cache's arrays that slot `slot` of unit u is, by its page table; -1 (and
// reported) when the entry is not a page.
__device__ __forceinline__ int slot_row(const PlanLaunch &p, int u, int slot)
{
    if (!p.table)
        return u * p.C + slot;
    const int pg = p.table_out[(size_t)u * (p.C / PAGE_SLOTS) + slot / PAGE_SLOTS];
    if (pg >= 0 && pg < p.num_pages)
        return pg * PAGE_SLOTS + slot % PAGE_SLOTS;
    flag_error(p.status, DEV_CAPACITY);
    return -1;
}

// A thread owns SPAN consecutive units, so CTAS * THREADS * SPAN units at most.  What the
// CTA's units are, for its threads that write new pages, returned pages and tokens: those
// are dealt evenly over the threads, who find their unit by bisecting the sums.
template <int SPAN> struct PlanSmem {
    static constexpr int N = THREADS * SPAN;
    int grow[N + 1], back[N + 1], toks[N + 1];   // pages taken, given back, tokens, before each unit
    int held[N];                                 // pages before
    int base[N];                                 // first new slot; -1: the unit is refused
    int start[N], pos[N];                        // first new token and its position
};

template <int SPAN>
__global__ void __launch_bounds__(THREADS) k_append_plan(const PlanLaunch p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    using Smem = PlanSmem<SPAN>;
    Smem &sm = *reinterpret_cast<Smem *>(smem);
    __shared__ int s_sum[4];   // this CTA's pages asked for, given back, granted; a bad range
    const int rank = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const int gtid = rank * THREADS + tid;
    const int units = p.B * p.Hkv;
    const int per = p.C / PAGE_SLOTS;
    const int u0 = gtid * SPAN, cta_u0 = rank * Smem::N;
    const bool paged = p.table != nullptr;
    asm volatile("griddepcontrol.launch_dependents;");

    // ---- the old counts, lengths and held pages, all of them: they may be replaced after the
    // cluster barrier below
    const int given = paged ? *p.count : 0, count = min(max(given, 0), p.num_pages);
    if (given != count && gtid == 0)
        flag_error(p.status, DEV_CAPACITY);
    int held[SPAN], now[SPAN], n[SPAN], m[SPAN], seqlen[SPAN];   // now: pages after
    int sum[3] = {0, 0, 0};
    bool fit[SPAN], broken = false;
#pragma unroll
    for (int i = 0; i < SPAN; ++i) {
        held[i] = now[i] = n[i] = m[i] = seqlen[i] = 0;
        fit[i] = false;
        const int u = u0 + i, b = u / p.Hkv;
        if (u < units) {
            const int c0 = p.cu[b], c1 = p.cu[b + 1];
            n[i] = p.n[u];
            seqlen[i] = p.seqlen[b];
            held[i] = now[i] = paged ? p.pages[u] : 0;
            const bool bad = c0 < 0 || c1 < c0 || c1 > p.T;
            broken |= bad;
            m[i] = bad ? 0 : c1 - c0;
            sm.start[tid * SPAN + i] = c0;
            fit[i] = fits(p, n[i], m[i]) && held[i] >= 0 && held[i] <= per;
            if (fit[i] && paged) {
                const int need = (n[i] + m[i] + PAGE_SLOTS - 1) / PAGE_SLOTS;
                now[i] = p.release || need > held[i] ? need : held[i];
            }
            if (!fit[i] || bad)
                flag_error(p.status, DEV_CAPACITY);
        }
        sum[0] += max(0, now[i] - held[i]);
        sum[1] += max(0, held[i] - now[i]);
        sum[2] += m[i];
    }
    if (paged && p.table_out != p.table)   // entries that change are written again below
        copy_i32(p.table_out, p.table, (long)units * per, gtid);
    broken = __syncthreads_or(broken);
    int total[3];
    scan3(sum, total);
#pragma unroll
    for (int i = 0; i < SPAN; ++i) {
        const int x = tid * SPAN + i;
        sm.held[x] = held[i];
        sm.grow[x] = sum[0];
        sm.back[x] = sum[1];
        sm.toks[x] = sum[2];
        sm.pos[x] = seqlen[i];
        sum[0] += max(0, now[i] - held[i]);
        sum[1] += max(0, held[i] - now[i]);
        sum[2] += m[i];
    }
    if (tid == 0) {
        s_sum[0] = sm.grow[Smem::N] = total[0];
        s_sum[1] = sm.back[Smem::N] = total[1];
        s_sum[2] = 0;
        s_sum[3] = broken;
        sm.toks[Smem::N] = total[2];
    }
    cluster_sync_all();
    // pages asked for and given back in all, and before this CTA's first unit
    const bool one = lane < CTAS;
    const int r_ask = one ? ld_cluster_s32(&s_sum[0], lane) : 0;
    const int r_back = one ? ld_cluster_s32(&s_sum[1], lane) : 0;
    broken = __any_sync(0xffffffffu, one && ld_cluster_s32(&s_sum[3], lane) != 0);
    const int asked = __reduce_add_sync(0xffffffffu, r_ask);
    const int before = __reduce_add_sync(0xffffffffu, lane < rank ? r_ask : 0);
    const int back0 = __reduce_add_sync(0xffffffffu, lane < rank ? r_back : 0);
    const int n_back = __reduce_add_sync(0xffffffffu, r_back);
    cluster_arrive();   // a CTA may leave once every other one has read its sums

    // ---- grants: a unit that the stack cannot serve in full keeps what it has.  Units are
    // served in order, so those served are the ones up to some unit and those that ask for
    // nothing.
    int granted = 0;
#pragma unroll
    for (int i = 0; i < SPAN; ++i) {
        const int x = tid * SPAN + i, u = u0 + i, g = max(0, now[i] - held[i]);
        bool ok = fit[i];
        if (g && before + sm.grow[x] + g > count) {
            ok = false;
            now[i] = held[i];
            flag_error(p.status, DEV_CAPACITY);
        } else {
            granted += g;
        }
        sm.base[x] = ok ? n[i] : -1;
        if (u < units) {
            p.n_out[u] = ok ? n[i] + m[i] : n[i];
            if (paged)
                p.pages_out[u] = now[i];
            if (u % p.Hkv == 0)
                p.seqlen_out[u / p.Hkv] = seqlen[i] + m[i];
        }
    }
    int taken = asked, mine = total[0];   // pages taken in all, and by this CTA
    if (asked > count) {   // the same on every CTA of the cluster
        cluster_wait();
        granted = __reduce_add_sync(0xffffffffu, granted);
        if (lane == 0)
            atomicAdd(&s_sum[2], granted);
        cluster_sync_all();
        taken = __reduce_add_sync(0xffffffffu, one ? ld_cluster_s32(&s_sum[2], lane) : 0);
        mine = s_sum[2];
        cluster_arrive();
    }
    const int left = count - taken;   // pages left on the stack
    if (paged && gtid == 0)
        *p.count_out = min(left + n_back, p.num_pages);
    // ---- new pages of the CTA's units, the next ones of the stack
    for (int x = tid; x < mine; x += THREADS) {
        const int i = last_at_most(sm.grow, Smem::N, x);
        p.table_out[(size_t)(cta_u0 + i) * per + sm.held[i] + x - sm.grow[i]] =
            p.free_list[count - 1 - before - x];
    }
    if (paged && p.free_out != p.free_list)
        copy_i32(p.free_out, p.free_list, left, gtid);
    // ---- tokens of no sequence
    const int first = broken ? p.T : min(p.cu[0], p.T), end = broken ? p.T : max(0, p.cu[p.B]);
    for (long x = gtid; x < (long)first * p.Hkv; x += CTAS * THREADS)
        p.slot_map[x] = -1;
    for (long x = (long)end * p.Hkv + gtid; x < (long)p.T * p.Hkv; x += CTAS * THREADS)
        p.slot_map[x] = -1;
    if (broken) {   // ranges may overlap what was just filled
        cluster_wait();
        cluster_sync_all();
        cluster_arrive();
    }
    __syncthreads();   // the CTA's pages are in the table, its units' slots known
    // ---- slot map and positions: every token of the CTA's units, or the first one of each
    // (k_plan_tokens follows with the others)
    const bool all = p.T <= CLUSTER_TOKENS;
    for (int x = tid; x < (all ? total[2] : Smem::N); x += THREADS) {
        const int i = all ? last_at_most(sm.toks, Smem::N, x) : x;
        const int u = cta_u0 + i, step = all ? x - sm.toks[i] : 0;
        if (step >= sm.toks[i + 1] - sm.toks[i])
            continue;
        int row = -1;
        if (sm.base[i] >= 0) {
            const int slot = sm.base[i] + step;
            row = slot_row(p, u, slot);
            p.pos[(size_t)u * p.C + slot] = sm.pos[i] + step;
        }
        p.slot_map[(size_t)(sm.start[i] + step) * p.Hkv + u % p.Hkv] = row;
    }
    // ---- returned pages go on the stack in unit order, when every page has been taken
    if (n_back > 0 && p.free_out == p.free_list) {
        cluster_wait();
        cluster_sync_all();
        cluster_arrive();
    }
    for (int x = tid; x < total[1]; x += THREADS) {
        const int i = last_at_most(sm.back, Smem::N, x);
        const int gave = sm.back[i + 1] - sm.back[i];
        const size_t e = (size_t)(cta_u0 + i) * per + sm.held[i] - gave + x - sm.back[i];
        const int pg = p.table[e], to = left + back0 + x;
        p.table_out[e] = -1;
        if (to < p.num_pages)
            p.free_out[to] = pg;
        else
            flag_error(p.status, DEV_CAPACITY);
    }
    cluster_wait();
}

// Whether a unit takes its tokens although the first one has no row: the entry of the first
// new slot is then not a page, and the plan has set that slot's position.  A refused unit's
// slot there is an older one, on a page that it holds.
__device__ __forceinline__ bool takes_behind_bad_page(const PlanLaunch &p, int u, int slot, int pos)
{
    const int pg = p.table_out[(size_t)u * (p.C / PAGE_SLOTS) + slot / PAGE_SLOTS];
    return (pg < 0 || pg >= p.num_pages) && p.pos[(size_t)u * p.C + slot] == pos;
}

// The other tokens of a large batch, a thread per token and eight heads' loads in flight
// together.  Launched so that its CTAs may start while the plan still runs: they wait for
// it before they read what it wrote.  The counts are the new ones by then, and the first
// token of each unit is done: its row says that the unit takes its tokens.  Ranges
// that run backwards cannot be bisected: then the first sequence that holds the token is
// looked for one by one.
__global__ void __launch_bounds__(256) k_plan_tokens(const PlanLaunch p)
{
    __shared__ int s_cu[CU_CACHE];
    bool backwards = false;
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
        const int c0 = p.cu[b], c1 = p.cu[b + 1];
        backwards |= c1 < c0;
        if (b < CU_CACHE)
            s_cu[b] = c0;
    }
    backwards = __syncthreads_or(backwards);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int t = blockIdx.x * blockDim.x + threadIdx.x;
    if (t >= p.T)
        return;
    int b = 0, start = 0, m = 0;
    if (!backwards) {
        // of sequences without tokens, the last
        b = last_at_most(p.B <= CU_CACHE ? s_cu : p.cu, p.B - 1, t);
        m = new_tokens(p, b, start);
    } else {
        for (; b < p.B; ++b) {
            m = new_tokens(p, b, start);
            if (t >= start && t < start + m)
                break;
        }
    }
    const int step = t - start;
    if (b >= p.B || step <= 0 || step >= m)
        return;   // of no sequence, or the first one: written by the plan
    const int per = p.C / PAGE_SLOTS;
    const int P = p.seqlen_out[b] - m + step;
    int *map = p.slot_map + (size_t)t * p.Hkv;
    for (int h0 = 0; h0 < p.Hkv; h0 += HEADS) {
        const int nh = min(HEADS, p.Hkv - h0), u = b * p.Hkv + h0;
        // each step loads for all heads before any value is used
        int n[HEADS], first[HEADS], row[HEADS];
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            n[h] = h < nh ? p.n_out[u + h] - m : -1;
            first[h] = h < nh ? p.slot_map[(size_t)start * p.Hkv + h0 + h] : -1;
        }
        unsigned ok = 0;   // heads that take the token
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            bool takes = fits(p, n[h], m);
            if (takes && first[h] < 0)
                takes = p.table && takes_behind_bad_page(p, u + h, n[h], P - step);
            ok |= (unsigned)takes << h;
            n[h] += step;   // the token's slot
        }
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            row[h] = -1;
            if (ok >> h & 1)
                row[h] = p.table ? p.table_out[(size_t)(u + h) * per + n[h] / PAGE_SLOTS]
                                 : (u + h) * p.C + n[h];
        }
        bool bad = false;
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            if (ok >> h & 1)
                p.pos[(size_t)(u + h) * p.C + n[h]] = P;
            if (p.table) {
                const bool page = row[h] >= 0 && row[h] < p.num_pages;
                bad |= (ok >> h & 1) && !page;
                row[h] = page ? row[h] * PAGE_SLOTS + n[h] % PAGE_SLOTS : -1;
            }
        }
        if (bad)
            flag_error(p.status, DEV_CAPACITY);
        if (nh == HEADS && p.Hkv % 4 == 0 && (reinterpret_cast<uintptr_t>(p.slot_map) & 15) == 0) {
            *reinterpret_cast<int4 *>(map + h0) = make_int4(row[0], row[1], row[2], row[3]);
            *reinterpret_cast<int4 *>(map + h0 + 4) = make_int4(row[4], row[5], row[6], row[7]);
        } else {
#pragma unroll
            for (int h = 0; h < HEADS; ++h)
                if (h < nh)
                    map[h0 + h] = row[h];
        }
    }
}

// Rows of the packed new tokens to the cache.  Each thread copies 16 bytes of K and
// of V per step.
__global__ void __launch_bounds__(256) k_append_packed(const PackedLaunch p)
{
    const int cpr = p.D / 8;   // 16-byte chunks per row
    const long total = (long)p.T * p.Hkv * cpr;
    for (long i = (long)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (long)gridDim.x * blockDim.x) {
        const long r = i / cpr;
        const int ch = (int)(i - r * cpr);
        const long t = r / p.Hkv;
        const int h = (int)(r - t * p.Hkv);
        const int row = p.slot_map[r];
        if (row < 0 || row >= p.rows) {
            if (row != -1 && ch == 0)
                flag_error(p.status, DEV_CAPACITY);
            continue;
        }
        const uint4 k = *reinterpret_cast<const uint4 *>(p.k_new + t * p.ks[0] + h * p.ks[1] + 8 * ch);
        const uint4 v = *reinterpret_cast<const uint4 *>(p.v_new + t * p.vs[0] + h * p.vs[1] + 8 * ch);
        *reinterpret_cast<uint4 *>(p.K + (long)row * p.D + 8 * ch) = k;
        *reinterpret_cast<uint4 *>(p.V + (long)row * p.D + 8 * ch) = v;
    }
}

} // namespace

template <int SPAN> static cudaError_t plan_impl(const PlanLaunch &p, cudaStream_t s)
{
    const void *f = reinterpret_cast<const void *>(k_append_plan<SPAN>);
    cudaError_t e = set_smem_once(f, sizeof(PlanSmem<SPAN>));
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(CTAS);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = sizeof(PlanSmem<SPAN>);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = CTAS;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_append_plan<SPAN>, p);
    if (e != cudaSuccess || p.T <= CLUSTER_TOKENS)
        return e;
    cfg.gridDim = dim3((p.T + 255) / 256);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    return cudaLaunchKernelEx(&cfg, k_plan_tokens, p);
}

cudaError_t launch_append_plan(const PlanLaunch &p, cudaStream_t s)
{
    return (long)p.B * p.Hkv <= (long)CTAS * THREADS ? plan_impl<1>(p, s)
                                                     : plan_impl<PLAN_MAX_SPAN>(p, s);
}

cudaError_t launch_append_packed(const PackedLaunch &p, cudaStream_t s)
{
    const long total = (long)p.T * p.Hkv * (p.D / 8);
    long grid = (total + 255) / 256;
    const long cap = 16L * sm_count();
    if (grid > cap)
        grid = cap;
    k_append_packed<<<(unsigned)grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

} // namespace kvc
