// attend_tokens.cu -- attention of many query tokens per sequence: whole prompts
// (kvc_prompt_attend) and chunks of new tokens over the slot cache
// (kvc_chunk_attend).
//
// For query token i of a sequence and query head h of KV head hk
//   s_j = scale q_i . k_j over the keys j < e_i,   m = max s, l = sum exp(s - m),
//   o_i = sum_j exp(s_j - m) v_j / l,              lse_i = m + log l
// with e_i = i + 1 in a prompt and e_i = n - m_b + i + 1 over a unit's n slots, of
// which the last m_b hold the chunk.  A row that sees nothing gives o = 0 and
// lse = -inf.
//
// A tile's rows are (token, head of the group) pairs, token-major, so the query
// heads of one KV head share every key they read.  One CTA of four warps takes
// 64 rows; keys stream through shared memory 64 at a time, and each warp keeps
// the running maximum, sum and weighted values of its 16 rows in registers.
#include "kvc_device.cuh"
#include "kvc_internal.h"

#include <math.h>

namespace kvc {

namespace {

constexpr int ROWS = 64;
constexpr int KEYS = 64;
constexpr float LN2 = 0.6931471805599453f;

// First token and length of sequence b; a range that leaves [0, L] counts as an
// empty sequence and is reported.
__device__ __forceinline__ void seq_range(const TokensLaunch &p, int b, int &start, int &len)
{
    start = p.cu ? p.cu[b] : 0;
    len = p.cu ? p.cu[b + 1] - start : p.lens ? p.lens[b] : p.L;
    if (start < 0 || start > p.L || len < 0 || len > p.L - start) {
        flag_error(p.status, DEV_CAPACITY);
        start = len = 0;
    }
}

// Sequence and tile of tile number idx, counted over the sequences in order
// (tiles of `tokens` tokens).  Every lane of the warp calls it; b = -1 when idx
// lies behind the last tile.
__device__ __forceinline__ void find_tile(const TokensLaunch &p, int tokens, int idx, int &b,
                                          int &tile, int &start, int &len)
{
    const int lane = threadIdx.x & 31;
    long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
        int s = 0, n = 0;
        if (b0 + lane < p.B)
            seq_range(p, b0 + lane, s, n);
        const int t = (n + tokens - 1) / tokens;
        int sum = t;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off)
                sum += y;
        }
        const unsigned here = __ballot_sync(0xffffffffu, base + sum > idx);
        if (here) {
            const int src = __ffs(here) - 1;
            b = b0 + src;
            tile = (int)(idx - base) - __shfl_sync(0xffffffffu, sum - t, src);
            start = __shfl_sync(0xffffffffu, s, src);
            len = __shfl_sync(0xffffffffu, n, src);
            return;
        }
        base += __shfl_sync(0xffffffffu, sum, 31);
    }
    b = -1;
}

template <int D>
__global__ void __launch_bounds__(128) k_attend_tokens(const TokensLaunch p)
{
    constexpr int LD = D + 8;   // padded row of a key tile: conflict-free ldmatrix
    constexpr int NK = D / 16;
    __shared__ __align__(16) uint16_t sk[KEYS * LD];
    __shared__ __align__(16) uint16_t sv[KEYS * LD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = p.Hq / p.Hkv, tokens = ROWS / g;
    const int hk = blockIdx.y;
    const SlotRows rows{p.block_table, p.C, p.num_pages};
    int b, tile, start, len;
    find_tile(p, tokens, blockIdx.x, b, tile, start, len);
    if (b < 0)
        return;
    const int tok0 = tile * tokens, n_tok = min(tokens, len - tok0);
    const int unit = b * p.Hkv + hk;
    int n_keys = len;   // keys the sequence's last token sees
    if (p.n) {
        n_keys = p.n[unit];
        if (n_keys < 0 || n_keys > p.C) {
            if (threadIdx.x == 0)
                flag_error(p.status, DEV_CAPACITY);
            n_keys = 0;
        }
    }
    const int shift = n_keys - len;               // token i sees keys j <= i + shift
    const int end = min(n_keys, shift + tok0 + n_tok);

    // this thread's two rows of the warp's 16
    int tok[2], head[2], last[2];
    bool real[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int r = 16 * warp + (lane >> 2) + 8 * u;
        tok[u] = tok0 + r / g;
        head[u] = hk * g + r % g;
        real[u] = r < n_tok * g;
        last[u] = real[u] ? tok[u] + shift : -1;
    }
    const long qb = p.cu ? 0 : b;
    uint32_t qf[NK][4];
#pragma unroll
    for (int kk = 0; kk < NK; ++kk)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint16_t *row = p.q + qb * p.qs[0] + head[u] * p.qs[1] +
                                  (long)(start + tok[u]) * p.qs[2] + 16 * kk + 2 * (lane & 3);
            qf[kk][u] = real[u] ? *reinterpret_cast<const uint32_t *>(row) : 0u;
            qf[kk][u + 2] = real[u] ? *reinterpret_cast<const uint32_t *>(row + 8) : 0u;
        }
    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
        acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int k0 = 0; k0 < end; k0 += KEYS) {
        __syncthreads();
        for (int i = threadIdx.x; i < KEYS * (D / 8); i += blockDim.x) {
            const int j = i / (D / 8), ch = i % (D / 8);
            uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
            if (k0 + j < end) {
                const uint16_t *ks, *vs;
                bool ok = true;
                if (p.n) {
                    const long row = rows.row(unit, k0 + j);
                    ok = row >= 0;
                    ks = p.k + row * D;
                    vs = p.v + row * D;
                } else {
                    ks = p.k + qb * p.ks[0] + hk * p.ks[1] + (long)(start + k0 + j) * p.ks[2];
                    vs = p.v + qb * p.vs[0] + hk * p.vs[1] + (long)(start + k0 + j) * p.vs[2];
                }
                if (ok) {
                    kx = *reinterpret_cast<const uint4 *>(ks + 8 * ch);
                    vx = *reinterpret_cast<const uint4 *>(vs + 8 * ch);
                } else if (ch == 0) {
                    flag_error(p.status, DEV_CAPACITY);
                }
            }
            *reinterpret_cast<uint4 *>(&sk[j * LD + 8 * ch]) = kx;
            *reinterpret_cast<uint4 *>(&sv[j * LD + 8 * ch]) = vx;
        }
        __syncthreads();
        float s[KEYS / 8][4];
#pragma unroll
        for (int nb = 0; nb < KEYS / 8; ++nb) {
            s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < NK; kk += 2) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4(smem_u32(&sk[(8 * nb + (lane & 7)) * LD + 16 * kk + 8 * (lane >> 3)]), b0,
                        b1, b2, b3);
                mma16816(s[nb], qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3], b0, b1);
                mma16816(s[nb], qf[kk + 1][0], qf[kk + 1][1], qf[kk + 1][2], qf[kk + 1][3], b2, b3);
            }
        }
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int nb = 0; nb < KEYS / 8; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = k0 + 8 * nb + 2 * (lane & 3) + (e & 1), u = e >> 1;
                s[nb][e] = j <= last[u] && j < end ? s[nb][e] * p.scale_log2 : -INFINITY;
                mx[u] = fmaxf(mx[u], s[nb][e]);
            }
        float corr[2], ref[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
            mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
            ref[u] = mx[u] == -INFINITY ? 0.f : mx[u];
            corr[u] = ex2(m[u] - ref[u]);
            m[u] = mx[u];
            l[u] *= corr[u];
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[i][e] *= corr[e >> 1];
        uint32_t pf[KEYS / 8][2];
#pragma unroll
        for (int nb = 0; nb < KEYS / 8; ++nb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[nb][e] = ex2(s[nb][e] - ref[e >> 1]);
                l[e >> 1] += s[nb][e];
            }
            pf[nb][0] = pack_half2(s[nb][0], s[nb][1]);
            pf[nb][1] = pack_half2(s[nb][2], s[nb][3]);
        }
#pragma unroll
        for (int kb = 0; kb < KEYS / 16; ++kb)
#pragma unroll
            for (int nd = 0; nd < D / 16; ++nd) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4_t(smem_u32(&sv[(16 * kb + (lane & 15)) * LD + 16 * nd + 8 * (lane >> 4)]),
                          b0, b1, b2, b3);
                mma16816(acc[2 * nd], pf[2 * kb][0], pf[2 * kb][1], pf[2 * kb + 1][0],
                         pf[2 * kb + 1][1], b0, b1);
                mma16816(acc[2 * nd + 1], pf[2 * kb][0], pf[2 * kb][1], pf[2 * kb + 1][0],
                         pf[2 * kb + 1][1], b2, b3);
            }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
        if (!real[u])
            continue;
        const float inv = l[u] > 0.f ? 1.f / l[u] : 0.f;
        uint16_t *row = p.o + qb * p.os[0] + head[u] * p.os[1] + (long)(start + tok[u]) * p.os[2];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<uint32_t *>(row + 8 * i + 2 * (lane & 3)) =
                pack_half2(acc[i][2 * u] * inv, acc[i][2 * u + 1] * inv);
        if (p.lse && (lane & 3) == 0)
            p.lse[qb * p.ls[0] + head[u] * p.ls[1] + start + tok[u]] =
                l[u] > 0.f ? (m[u] + log2f(l[u])) * LN2 : -INFINITY;
    }
}

} // namespace

cudaError_t launch_attend_tokens(const TokensLaunch &p, cudaStream_t s)
{
    const int g = p.Hq / p.Hkv, tokens = ROWS / g;
    const long per = (p.L + tokens - 1) / tokens;
    // packed: every sequence ends in at most one partial tile
    const long tiles = p.cu ? (long)p.L / tokens + p.B : per * p.B;
    if (tiles > 0x7fffffffL)
        return cudaErrorInvalidValue;
    const dim3 grid((unsigned)tiles, (unsigned)p.Hkv);
    if (p.D == 128)
        k_attend_tokens<128><<<grid, 128, 0, s>>>(p);
    else
        k_attend_tokens<64><<<grid, 128, 0, s>>>(p);
    return cudaGetLastError();
}

} // namespace kvc
