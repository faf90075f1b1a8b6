// append_plan.cu -- where the new tokens of a ragged batch go.
//
// kvc_append_plan: per (sequence, KV head) unit with n slots and m new tokens
//   need = ceil((n + m) / 64) pages, grow = max(0, need - held),
//   back = max(0, held - need) when pages are to be released.
// A unit's new pages are the next `grow` ones from the top of the free stack, in
// unit order, so every unit needs the sum of grow over the units before it; the
// returned pages go on what is left of the stack, placed by the same sum of back.
// Integer work of a few bytes per unit and token: latency bound.  One thread-block
// cluster does it in one launch, because the sums run over all units and the
// outputs may be the inputs: every CTA scans its range of units, the totals cross
// through distributed shared memory, and cluster barriers part the reads of the
// old state from the writes of the new.
//
// kvc_append_packed: one 16-byte chunk of a K and of a V row per thread and step,
// written to the row that the slot map names.  HBM bound: 2 D bytes read and
// written per row, twice.
#include "kvc_device.cuh"
#include "kvc_internal.h"

namespace kvc {

namespace {

constexpr int CTAS = 16;       // one cluster
constexpr int THREADS = 1024;
constexpr int CU_CACHE = 2048; // sequence starts held in shared memory
constexpr int HEADS = 8;       // heads of a token whose loads are in flight together
// Tokens whose slot map the cluster writes itself; more go to a second kernel on all SMs
// (scattered words: TODO).
constexpr int CLUSTER_TOKENS = 2048;
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

// Exclusive scans of two counts over the CTA's threads, and their totals.
__device__ __forceinline__ void scan2(int &x, int &y, int &tx, int &ty)
{
    __shared__ int s_x[32], s_y[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int ix = x, iy = y;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int ux = __shfl_up_sync(0xffffffffu, ix, off);
        const int uy = __shfl_up_sync(0xffffffffu, iy, off);
        if (lane >= off) {
            ix += ux;
            iy += uy;
        }
    }
    if (lane == 31) {
        s_x[warp] = ix;
        s_y[warp] = iy;
    }
    __syncthreads();
    if (warp == 0) {
        int wx = s_x[lane], wy = s_y[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int ux = __shfl_up_sync(0xffffffffu, wx, off);
            const int uy = __shfl_up_sync(0xffffffffu, wy, off);
            if (lane >= off) {
                wx += ux;
                wy += uy;
            }
        }
        s_x[lane] = wx;
        s_y[lane] = wy;
    }
    __syncthreads();
    x = ix - x + (warp ? s_x[warp - 1] : 0);
    y = iy - y + (warp ? s_y[warp - 1] : 0);
    tx = s_x[31];
    ty = s_y[31];
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

// Whether unit u takes its m new tokens, once its pages are granted.
__device__ __forceinline__ bool takes(const PlanLaunch &p, int u, int n, int m)
{
    return fits(p, n, m) && (!p.table || p.pages_out[u] * (long)PAGE_SLOTS >= n + m);
}

// Row of unit u's slot, once its pages are granted; -1 when its table entry is not a page.
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

// Slot map and positions of token t for every head.  `starts` are the sequences' first
// tokens (cu, or a copy).  Ranges that run backwards cannot be bisected: then the first
// sequence that holds the token is looked for one by one.
// AFTER: the counts are already the new ones, and the first token of each unit is done: its
// entry says whether the unit takes its tokens.
template <bool AFTER>
__device__ __forceinline__ void plan_token(const PlanLaunch &p, int t, const int *starts,
                                           bool backwards)
{
    int b = 0, start = 0, m = 0;
    if (!backwards) {
        b = last_at_most(starts, p.B - 1, t);   // of sequences without tokens, the last
        m = new_tokens(p, b, start);
    } else {
        for (; b < p.B; ++b) {
            m = new_tokens(p, b, start);
            if (t >= start && t < start + m)
                break;
        }
    }
    const bool inside = b < p.B && t >= start && t < start + m;
    const int step = t - start;
    if (AFTER && inside && step == 0)
        return;
    const int P = inside ? (AFTER ? p.seqlen_out[b] - m : p.seqlen[b]) + step : 0;
    int *map = p.slot_map + (size_t)t * p.Hkv;
    const int per = p.C / PAGE_SLOTS;
    for (int h0 = 0; h0 < p.Hkv; h0 += HEADS) {
        const int nh = min(HEADS, p.Hkv - h0), u = b * p.Hkv + h0;
        // each step loads for all heads before any value is used
        int n[HEADS], x[HEADS], row[HEADS];
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            const bool here = inside && h < nh;
            n[h] = here ? (AFTER ? p.n_out : p.n)[u + h] : -1;
            // what tells whether the unit takes its tokens: its pages, or its first entry
            x[h] = !here ? -1
                   : AFTER ? p.slot_map[(size_t)start * p.Hkv + h0 + h]
                           : p.table ? p.pages_out[u + h] : per;
        }
        unsigned ok = 0;   // heads that take the token
#pragma unroll
        for (int h = 0; h < HEADS; ++h) {
            n[h] -= AFTER ? m : 0;
            const bool room = !p.table || x[h] * (long)PAGE_SLOTS >= n[h] + m;
            ok |= (unsigned)(fits(p, n[h], m) && (AFTER ? x[h] >= 0 : room)) << h;
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

// A thread owns SPAN consecutive units, so CTAS * THREADS * SPAN units at most.
template <int SPAN> struct PlanSmem {
    int cu[CU_CACHE];
    int grow[THREADS * SPAN + 1];   // pages taken by the CTA's units before each unit
    int back[THREADS * SPAN + 1];   // pages given back
    int held[THREADS * SPAN];
};

template <int SPAN>
__global__ void __launch_bounds__(THREADS) k_append_plan(const PlanLaunch p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    PlanSmem<SPAN> &sm = *reinterpret_cast<PlanSmem<SPAN> *>(smem);
    __shared__ int s_sum[3];   // this CTA's pages asked for, given back and granted
    const int rank = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const int gtid = rank * THREADS + tid, gsize = CTAS * THREADS;
    const int units = p.B * p.Hkv;
    const int per = p.C / PAGE_SLOTS;
    const int u0 = gtid * SPAN, cta_u0 = rank * THREADS * SPAN;
    int left = 0, n_back = 0;      // pages left on the stack, pages given back

    asm volatile("griddepcontrol.launch_dependents;");

    bool backwards = false;
    for (int b = tid; b < p.B; b += THREADS) {
        const int c0 = p.cu[b], c1 = p.cu[b + 1];
        backwards |= c1 < c0;
        if (b < CU_CACHE)
            sm.cu[b] = c0;
    }

    if (p.table) {
        if (p.table_out != p.table)   // entries that change are written again below
            copy_i32(p.table_out, p.table, (long)units * per, gtid);
        // ---- scan: pages asked for and given back by the units before each unit
        const int given = *p.count, count = min(max(given, 0), p.num_pages);
        if (given != count && gtid == 0)
            flag_error(p.status, DEV_CAPACITY);
        int held[SPAN], now[SPAN];     // pages before and after
        int ask = 0, back = 0;
#pragma unroll
        for (int i = 0; i < SPAN; ++i) {
            held[i] = now[i] = 0;
            if (u0 + i < units) {
                int st;
                const int m = new_tokens(p, (u0 + i) / p.Hkv, st), n = p.n[u0 + i];
                const int h = p.pages[u0 + i];
                held[i] = now[i] = h;
                if (fits(p, n, m) && h >= 0 && h <= per) {
                    const int need = (n + m + PAGE_SLOTS - 1) / PAGE_SLOTS;
                    now[i] = p.release || need > h ? need : h;
                } else {
                    flag_error(p.status, DEV_CAPACITY);
                }
                ask += max(0, now[i] - h);
                back += max(0, h - now[i]);
            }
        }
        int tx, ty;
        scan2(ask, back, tx, ty);
#pragma unroll
        for (int i = 0; i < SPAN; ++i) {
            sm.held[tid * SPAN + i] = held[i];
            sm.grow[tid * SPAN + i] = ask;
            sm.back[tid * SPAN + i] = back;
            ask += max(0, now[i] - held[i]);
            back += max(0, held[i] - now[i]);
        }
        if (tid == 0) {
            s_sum[0] = tx;
            s_sum[1] = ty;
            s_sum[2] = 0;
            sm.grow[THREADS * SPAN] = tx;
            sm.back[THREADS * SPAN] = ty;
        }
        cluster_sync_all();
        // pages asked for and given back in all, and before this CTA's first unit
        const int r_ask = lane < CTAS ? ld_cluster_s32(&s_sum[0], lane) : 0;
        const int r_back = lane < CTAS ? ld_cluster_s32(&s_sum[1], lane) : 0;
        const int total = __reduce_add_sync(0xffffffffu, r_ask);
        const int before = __reduce_add_sync(0xffffffffu, lane < rank ? r_ask : 0);
        const int back0 = __reduce_add_sync(0xffffffffu, lane < rank ? r_back : 0);
        n_back = __reduce_add_sync(0xffffffffu, r_back);
        // ---- grants: a unit that the stack cannot serve in full keeps what it has.  Units
        // are served in order, so those served are the ones up to some unit and those that
        // ask for nothing.
        int granted = 0;
#pragma unroll
        for (int i = 0; i < SPAN; ++i) {
            const int g = max(0, now[i] - held[i]);
            if (g && before + sm.grow[tid * SPAN + i] + g > count) {
                now[i] = held[i];
                flag_error(p.status, DEV_CAPACITY);
            } else {
                granted += g;
            }
            if (u0 + i < units)
                p.pages_out[u0 + i] = now[i];
        }
        int taken = total, mine = tx;   // pages taken in all, and by this CTA
        if (total > count) {   // the same on every CTA of the cluster
            granted = __reduce_add_sync(0xffffffffu, granted);
            if (lane == 0)
                atomicAdd(&s_sum[2], granted);
            cluster_sync_all();
            taken = __reduce_add_sync(0xffffffffu,
                                      lane < CTAS ? ld_cluster_s32(&s_sum[2], lane) : 0);
            mine = s_sum[2];
        }
        left = count - taken;
        // ---- new pages of the CTA's units, the next ones of the stack
        for (int x = tid; x < mine; x += THREADS) {
            const int i = last_at_most(sm.grow, THREADS * SPAN, x);
            p.table_out[(size_t)(cta_u0 + i) * per + sm.held[i] + x - sm.grow[i]] =
                p.free_list[count - 1 - before - x];
        }
        if (p.free_out != p.free_list)
            copy_i32(p.free_out, p.free_list, left, gtid);
        cluster_sync_all();   // every new page is taken, every page count written
        // ---- returned pages go on the stack in unit order
        for (int x = tid; x < ty; x += THREADS) {
            const int i = last_at_most(sm.back, THREADS * SPAN, x);
            const int gave = sm.back[i + 1] - sm.back[i];
            const size_t e = (size_t)(cta_u0 + i) * per + sm.held[i] - gave + x - sm.back[i];
            const int pg = p.table[e], to = left + back0 + x;
            p.table_out[e] = -1;
            if (to < p.num_pages)
                p.free_out[to] = pg;
            else
                flag_error(p.status, DEV_CAPACITY);
        }
    } else {
        for (int u = gtid; u < units; u += gsize) {
            int st;
            if (!fits(p, p.n[u], new_tokens(p, u / p.Hkv, st)))
                flag_error(p.status, DEV_CAPACITY);
        }
    }

    // ---- slot map and positions
    backwards = __syncthreads_or(backwards);
    if (p.T <= CLUSTER_TOKENS) {
        // a thread per token, warps dealt to the CTAs in turn
        for (int t = ((tid >> 5) * CTAS + rank) * 32 + lane; t < p.T; t += gsize)
            plan_token<false>(p, t, p.B <= CU_CACHE ? sm.cu : p.cu, backwards);
    } else {
        // the first token of each unit; k_plan_tokens follows with the others
        for (int u = gtid; u < units; u += gsize) {
            int start;
            const int b = u / p.Hkv, m = new_tokens(p, b, start), n = p.n[u];
            if (m == 0)
                continue;
            int row = -1;
            if (takes(p, u, n, m)) {
                row = slot_row(p, u, n);
                p.pos[(size_t)u * p.C + n] = p.seqlen[b];
            }
            p.slot_map[(size_t)start * p.Hkv + u - b * p.Hkv] = row;
        }
    }
    cluster_sync_all();   // the old counts have been read everywhere

    // ---- counts
    for (int u = gtid; u < units; u += gsize) {
        int st;
        const int m = new_tokens(p, u / p.Hkv, st), n = p.n[u];
        p.n_out[u] = takes(p, u, n, m) ? n + m : n;
    }
    for (int b = gtid; b < p.B; b += gsize) {
        int st;
        const int m = new_tokens(p, b, st);
        const int before = p.cu[b], after = p.cu[b + 1];
        if (after != before && m == 0)
            flag_error(p.status, DEV_CAPACITY);   // a range outside the batch
        p.seqlen_out[b] = p.seqlen[b] + m;
    }
    if (p.table && gtid == 0)
        *p.count_out = min(left + n_back, p.num_pages);
}

// The other tokens of a large batch, a thread per token.  Launched so that its CTAs may
// start while the plan still runs: they wait for it before they read what it wrote.
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
    if (t < p.T)
        plan_token<true>(p, t, p.B <= CU_CACHE ? s_cu : p.cu, backwards);
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
    cudaError_t e = set_smem_once(f, sizeof(PlanSmem<SPAN>), true);
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
