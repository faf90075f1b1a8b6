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

constexpr int CTAS = 8;        // one portable cluster
constexpr int THREADS = 1024;
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

// Units a thread owns: SPAN consecutive ones, so 8192 * SPAN units at most.
template <int SPAN>
__global__ void __cluster_dims__(CTAS, 1, 1) __launch_bounds__(THREADS)
    k_append_plan(const PlanLaunch p)
{
    __shared__ int s_sum[3];   // this CTA's pages asked for, given back and granted
    const int rank = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    const int gtid = rank * THREADS + tid, gsize = CTAS * THREADS;
    const int units = p.B * p.Hkv;
    const int per = p.C / PAGE_SLOTS;
    const int u0 = gtid * SPAN;
    int left = 0, n_back = 0;      // pages left on the stack, pages given back
    int held[SPAN], now[SPAN], at[SPAN];   // pages before and after; place in the stack

    if (p.table) {
        // ---- scan: pages asked for and given back by the units before each unit
        const int count = min(max(*p.count, 0), p.num_pages);
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
        if (tid == 0) {
            s_sum[0] = tx;
            s_sum[1] = ty;
            s_sum[2] = 0;
        }
        cluster_sync_all();
        int total = 0;
        for (int r = 0; r < CTAS; ++r) {
            const int a = ld_cluster_s32(&s_sum[0], r), k = ld_cluster_s32(&s_sum[1], r);
            ask += r < rank ? a : 0;
            back += r < rank ? k : 0;
            total += a;
            n_back += k;
        }
        // ---- grants: a unit that the stack cannot serve in full keeps what it has
        int granted = 0;
#pragma unroll
        for (int i = 0; i < SPAN; ++i) {
            const int g = max(0, now[i] - held[i]), k = max(0, held[i] - now[i]);
            at[i] = g ? count - 1 - ask : back;
            if (g && ask + g > count) {
                now[i] = held[i];
                flag_error(p.status, DEV_CAPACITY);
            } else {
                granted += g;
            }
            ask += g;
            back += k;
        }
        int taken = total;
        if (total > count) {   // the same on every CTA of the cluster
            granted = __reduce_add_sync(0xffffffffu, granted);
            if (lane == 0)
                atomicAdd(&s_sum[2], granted);
            cluster_sync_all();
            taken = 0;
            for (int r = 0; r < CTAS; ++r)
                taken += ld_cluster_s32(&s_sum[2], r);
        }
        left = count - taken;
        // ---- table rows, a warp per row: kept entries, then the new pages
        const bool copy = p.table_out != p.table;
#pragma unroll
        for (int i = 0; i < SPAN; ++i) {
            for (int l = 0; l < 32; ++l) {
                const int u = __shfl_sync(0xffffffffu, u0, l) + i;
                if (u >= units)
                    break;
                const int h = __shfl_sync(0xffffffffu, held[i], l);
                const int w = __shfl_sync(0xffffffffu, now[i], l);
                const int top = __shfl_sync(0xffffffffu, at[i], l);
                const int32_t *src = p.table + (size_t)u * per;
                int32_t *dst = p.table_out + (size_t)u * per;
                for (int j = (copy ? 0 : h) + lane; j < (copy ? per : w); j += 32) {
                    if (j >= h && j < w)
                        dst[j] = p.free_list[top - (j - h)];
                    else if (j < w || j >= h)   // entries that go back are written below
                        dst[j] = src[j];
                }
            }
            if (u0 + i < units)
                p.pages_out[u0 + i] = now[i];
        }
        if (p.free_out != p.free_list)
            for (int i = gtid; i < left; i += gsize)
                p.free_out[i] = p.free_list[i];
        cluster_sync_all();   // every new page is taken, every row and page count written
        // ---- returned pages go on the stack in unit order
#pragma unroll
        for (int i = 0; i < SPAN; ++i) {
            unsigned any = __ballot_sync(0xffffffffu, now[i] < held[i]);
            while (any) {
                const int l = __ffs(any) - 1;
                any &= any - 1;
                const int u = __shfl_sync(0xffffffffu, u0, l) + i;
                const int h = __shfl_sync(0xffffffffu, held[i], l);
                const int w = __shfl_sync(0xffffffffu, now[i], l);
                const int to = left + __shfl_sync(0xffffffffu, at[i], l);
                for (int j = w + lane; j < h; j += 32) {
                    const int pg = p.table[(size_t)u * per + j];
                    p.table_out[(size_t)u * per + j] = -1;
                    if (to + j - w < p.num_pages)
                        p.free_out[to + j - w] = pg;
                    else
                        flag_error(p.status, DEV_CAPACITY);
                }
            }
        }
    } else {
        for (int u = gtid; u < units; u += gsize) {
            int st;
            if (!fits(p, p.n[u], new_tokens(p, u / p.Hkv, st)))
                flag_error(p.status, DEV_CAPACITY);
        }
    }

    // ---- slot map and positions: a thread per token.  Ranges that run backwards cannot be
    // bisected: then the first sequence that holds the token is looked for one by one.
    bool backwards = false;
    for (int b = tid; b < p.B; b += THREADS)
        backwards |= p.cu[b + 1] < p.cu[b];
    backwards = __syncthreads_or(backwards);
    for (int t = gtid; t < p.T; t += gsize) {
        int lo = 0, hi = p.B;   // the first sequence that starts behind t, less one
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (p.cu[mid + 1] <= t)
                lo = mid + 1;
            else
                hi = mid;
        }
        int start = 0;
        int m = lo < p.B && !backwards ? new_tokens(p, lo, start) : 0;
        for (int b = 0; backwards && b < p.B; ++b) {
            m = new_tokens(p, b, start);
            lo = b;
            if (t >= start && t < start + m)
                break;
        }
        const bool inside = t >= start && t < start + m;
        const int step = t - start;
        const int P = inside ? p.seqlen[lo] + step : 0;
        for (int h = 0; h < p.Hkv; ++h) {
            int row = -1;
            if (inside) {
                const int u = lo * p.Hkv + h, n = p.n[u], slot = n + step;
                if (fits(p, n, m) && (!p.table || p.pages_out[u] * (long)PAGE_SLOTS >= n + m)) {
                    if (!p.table) {
                        row = u * p.C + slot;
                    } else {
                        const int pg = p.table_out[(size_t)u * per + slot / PAGE_SLOTS];
                        if (pg >= 0 && pg < p.num_pages)
                            row = pg * PAGE_SLOTS + slot % PAGE_SLOTS;
                        else
                            flag_error(p.status, DEV_CAPACITY);
                    }
                    p.pos[(size_t)u * p.C + slot] = P;
                }
            }
            p.slot_map[(size_t)t * p.Hkv + h] = row;
        }
    }
    cluster_sync_all();   // the old counts have been read everywhere

    // ---- counts
    for (int u = gtid; u < units; u += gsize) {
        int st;
        const int m = new_tokens(p, u / p.Hkv, st), n = p.n[u];
        const bool ok =
            fits(p, n, m) && (!p.table || p.pages_out[u] * (long)PAGE_SLOTS >= n + m);
        p.n_out[u] = ok ? n + m : n;
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

cudaError_t launch_append_plan(const PlanLaunch &p, cudaStream_t s)
{
    if ((long)p.B * p.Hkv <= (long)CTAS * THREADS)
        k_append_plan<1><<<CTAS, THREADS, 0, s>>>(p);
    else
        k_append_plan<PLAN_MAX_SPAN><<<CTAS, THREADS, 0, s>>>(p);
    return cudaGetLastError();
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
