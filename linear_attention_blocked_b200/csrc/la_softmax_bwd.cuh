// la_softmax_bwd.cuh -- gradients of causal softmax attention for sm_100a.
//
// With P_ts = exp(scale q_t . k_s - lse_t) for s <= t (0 otherwise), g_t = dL/do_t
// and delta_t = g_t . o_t:
//
//     dS_ts = P_ts (g_t . v_s - delta_t)
//     dq_t  = scale sum_s dS_ts k_s
//     dk_s  = scale sum_t dS_ts q_t,   dv_s = sum_t P_ts g_t
//
// (dk, dv summed over the query heads of the group).  P is formed again from
// the scores and lse, so nothing of the scores' size is kept.
//
// Two kernels, each of which owns its sums: one CTA per key block walks the
// query blocks behind it (dk, dv), one per query block walks the key blocks
// before it (dq).  That is seven products of 128 x 128 x 128 per pair of
// blocks where five would do with dq added up across CTAs; it needs no
// atomics, so the gradients do not depend on timing, and no fp32 copy of dq
// in memory.  P and dS go from registers to TMEM as bf16, where the products
// that sum over them take them as their first operand: shared memory holds
// only what TMA brought.
//
// delta_t = g_t . o_t is off by the rounding of o to bf16.  In a row of few keys, or
// of one heavy key, g_t . v_s - delta_t may be much smaller than either, so the first
// 128 rows of a sequence, which meet all their keys in one step, take
// delta_t = sum_s P_ts (g_t . v_s) from that step, in fp32: with sequences of 2 tokens
// dq is off by 0.0023 of its norm instead of 0.0037 (dS and the result, rounded to
// bf16, alone make 0.0023).  8 sequences of 60, 64 heads over 8: 3.7 us more.
//
// 8192 tokens, 16 heads over 2: dk and dv 447 us at 1.62 GHz, 1229 TFLOP/s, tensor pipe
// busy 66 %; dq 299 us at 1.58 GHz, 1377 TFLOP/s, 75 %.  What is left is the way from a product
// through TMEM, the exponentials or the sums and back to the next product.
#pragma once
#include "la_softmax.cuh"

namespace la {

constexpr int SB_THREADS = 384;  // warpgroup 0: loads, MMA; 1 and 2: columns [0, 64) and [64, 128) of a tile
constexpr uint32_t ID_SS = idesc_bf16_f32(BLK, BLK, 0, 0);  // both operands K-major
constexpr uint32_t ID_TS = idesc_bf16_f32(BLK, D, 0, 1);    // TMEM x MN-major

struct SoftmaxBwdParams {
    const float *lse2, *delta;    // [H, T]: lse * log2 e, g . o
    __nv_bfloat16 *dq, *dk, *dv;
    float *parts;                 // [nparts][2][T, Hkv, D] fp32 sums of dk, dv, or null (nparts = 1)
    int *hdr;
    const int4 *entries;
    int T, H, Hkv, G;
    int nparts;                   // CTAs that share a key block's query heads
    int by_length;                // entries are in order of length: all heads of an entry in turn
    float scale, scale_log2;
    unsigned long long wait_limit_ns;
    int *status;
};

// bf16 pairs of 64 fp32 values -> 32 TMEM columns
__device__ __forceinline__ void tmem_st_bf16x64(uint32_t taddr, const float (&x)[64]) {
    uint32_t b[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) b[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    tmem_st32(taddr, b);
}
// A operand in TMEM written as two halves of 64 columns by the two
// warpgroups, each inside its own half of the fp32 tile that it replaces
__device__ __forceinline__ uint32_t half_cols(int kk) { return (uint32_t)((kk >> 2) * 64 + (kk & 3) * 8); }

// delta_t = g_t . o_t and lse_t log2 e, both as [H, T]: 16 lanes per (token, head).
// The first block is the scheduler, beside the others: a launch less (1 to 2 us).
__global__ void __launch_bounds__(SCHED_THREADS, 2)
la_softmax_rows_kernel(const SoftmaxScheduleParams s, const __nv_bfloat16 *out, const __nv_bfloat16 *dout,
                       const float *lse, float *lse2, float *delta, int T, int H) {
    pdl_wait();    // before the kernel behind may start: it reads what came before this one
    pdl_launch();
    if (blockIdx.x == 0) {
        softmax_schedule(s);
        return;
    }
    const long long total = (long long)T * H, step = ((long long)(gridDim.x - 1) * SCHED_THREADS) >> 4;
    const int l16 = threadIdx.x & 15, half = (threadIdx.x >> 4) & 1;
    // A warp has two rows; both halves stay in the loop as long as one has a row, since
    // the sums' shuffles name all 32 lanes (with odd T H the last warp has one row).
    for (long long first = ((long long)(blockIdx.x - 1) * SCHED_THREADS + (threadIdx.x & ~31u)) >> 4; first < total;
         first += step) {
        const long long e = first + half;
        const bool has = e < total;
        const uint4 none = make_uint4(0, 0, 0, 0);
        const uint4 a = has ? reinterpret_cast<const uint4 *>(out + e * D)[l16] : none;
        const uint4 b = has ? reinterpret_cast<const uint4 *>(dout + e * D)[l16] : none;
        const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x = fmaf(__uint_as_float(av[i] << 16), __uint_as_float(bv[i] << 16), x);
            x = fmaf(__uint_as_float(av[i] & 0xffff0000u), __uint_as_float(bv[i] & 0xffff0000u), x);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o, 16);
        if (has && l16 == 0) {
            const long long t = e / H, h = e - t * H;
            delta[h * T + t] = x;
            lse2[h * T + t] = lse[e] * 1.44269504088896341f;
        }
    }
}

// ---------------------------------------------------------------------------
// dk and dv.  Per step (query head, query block) of a key block, all 128 x 128
// with key rows and query columns:
//     S^T = K Q^T,  dP^T = V g^T           (SS MMAs)
//     P^T = 2^(c S^T - lse2[t])            -> TMEM, bf16
//     dv += P^T g                          (TS MMA)
//     dS^T = P^T (dP^T - delta[t])         -> TMEM, bf16
//     dk += dS^T Q                         (TS MMA)
// issued as S, dP | dv, S' | dk, dP' | ...: while dS is formed the tensor pipe
// has dv and the next S to do, while P is formed dk and the next dP.
// TMEM: S^T | dP^T | dv | dk.  Warps: 0 Q and g tiles, 1 MMA, 2 K and V tiles,
// 3 lse2 and delta of the step's rows (and zeros behind the sequence's end).
// ---------------------------------------------------------------------------
constexpr int DKV_K = 0, DKV_V = TILE_BYTES, DKV_RING = 2 * TILE_BYTES;  // ring: 2 x (Q, g)
constexpr int DKV_ROWS = DKV_RING + 4 * TILE_BYTES;                      // 2 x (lse2 [128], delta [128])
constexpr int DKV_CTRL = DKV_ROWS + 2 * 2 * BLK * 4;
constexpr int DKV_SUMS = DKV_CTRL + 512;                                 // [2][4 warps][64 columns]
constexpr int DKV_SMEM = DKV_SUMS + 2 * 4 * 64 * 4;
constexpr int SB_SLOTS = 4;

struct DkvCtrl {
    uint64_t q_full[2], q_empty[2];       // [1], [1]
    uint64_t rows_full[2];                // [1] lse2, delta (and zeroed rows) of the step
    uint64_t kv_full, kv_empty;           // [1], [1]
    uint64_t s_full, p_full;              // [1], [8]
    uint64_t dp_full, ds_full;            // [1], [8]
    uint64_t sum_full[2];                 // [4] a warpgroup's exact delta: sums of its warps, then joined
    uint64_t acc_full;                    // [1] an item's dv and dk are complete
    uint64_t item_full[SB_SLOTS], item_empty[SB_SLOTS];  // [1], [11]
    uint64_t fin;
    int item[SB_SLOTS][8];
    uint32_t tmem_base;
    volatile int abort;
};
static_assert(sizeof(DkvCtrl) <= 512, "control block");

enum { BI_VALID = 0, BI_TOK0, BI_LEN, BI_BLK, BI_KVH, BI_G0, BI_G1, BI_PART, BI_FIELDS };

template <class Ctrl>
__device__ __forceinline__ bool sb_next(uint32_t &it, int (&item)[BI_FIELDS], int lane, unsigned long long limit_ns,
                                        int *status, Ctrl *cb) {
    const int slot = it % SB_SLOTS;
    item[BI_VALID] = 0;
    if (!ctrl_warp_wait(&cb->item_full[slot], (it / SB_SLOTS) & 1, limit_ns, status, cb)) return false;
#pragma unroll
    for (int f = 0; f < BI_FIELDS; ++f) item[f] = __shfl_sync(0xffffffffu, cb->item[slot][f], 0);
    if (lane == 0) mbar_arrive(&cb->item_empty[slot]);
    ++it;
    return item[BI_VALID] != 0;
}

// Zero rows [valid, 128) of a swizzled tile (a warp; the caller fences)
__device__ __forceinline__ void zero_rows(uint8_t *tile, int valid, int lane) {
    const int nbytes = (BLK - valid) * 128;
    for (int hh = 0; hh < 2; ++hh)
        for (int o = lane * 16; o < nbytes; o += 32 * 16)
            *reinterpret_cast<uint4 *>(tile + hh * HALF_BYTES + valid * 128 + o) = make_uint4(0, 0, 0, 0);
}

__global__ void __launch_bounds__(SB_THREADS, 1)
la_softmax_dkv_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmg,
                      const __grid_constant__ SoftmaxBwdParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    DkvCtrl *cb = reinterpret_cast<DkvCtrl *>(smem + DKV_CTRL);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t sbase = smem_u32(smem);
    if (sbase & 1023) {
        if (threadIdx.x == 0) record_status(p.status, ST_CUDA);
        return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&cb->q_full[s], 1);
            mbar_init(&cb->q_empty[s], 1);
            mbar_init(&cb->rows_full[s], 1);
        }
        mbar_init(&cb->kv_full, 1);
        mbar_init(&cb->kv_empty, 1);
        mbar_init(&cb->s_full, 1);
        mbar_init(&cb->p_full, 8);
        mbar_init(&cb->dp_full, 1);
        mbar_init(&cb->ds_full, 8);
        mbar_init(&cb->sum_full[0], 4);
        mbar_init(&cb->sum_full[1], 4);
        mbar_init(&cb->acc_full, 1);
        for (int s = 0; s < SB_SLOTS; ++s) {
            mbar_init(&cb->item_full[s], 1);
            mbar_init(&cb->item_empty[s], 11);  // MMA, K/V, rows and 8 softmax warps
        }
        mbar_init(&cb->fin, 1);
        cb->abort = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
        tma_prefetch_desc(&tmg);
    }
    if (warp == 1) {
        tmem_alloc(&cb->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, cb->tmem_base, 0);
    const uint32_t TS = tmem, TDP = tmem + 128, TDV = tmem + 256, TDK = tmem + 384;
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return ctrl_warp_wait(bar, parity, p.wait_limit_ns, p.status, cb);
    };
    auto next = [&](uint32_t &it, int (&item)[BI_FIELDS]) -> bool {
        return sb_next(it, item, lane, p.wait_limit_ns, p.status, cb);
    };
    pdl_wait();  // every warp, before its first wait with a limit: the tables and rows are written

    if (warp < 4) {
        reg_dec<72>();
        if (warp == 0) {
            // ===================== items, Q and g tiles =====================
            const uint64_t pol = policy_evict_last();
            // What this thread has waited for is handed on to dq, which does not wait for this
            // kernel's end: the word is behind all that the kernels in front have written.
            if (blockIdx.x == 0 && lane == 0)
                asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(p.hdr + HDR_READY), "r"(1) : "memory");
            pdl_launch();  // dq, which needs nothing of this kernel, fills the SMs that run out of items
            const int ne = p.hdr[HDR_G];
            const long long total = (long long)ne * p.Hkv * p.nparts;
            uint32_t it = 0, n = 0;
            bool ok = true;
            while (ok) {
                const int slot = it % SB_SLOTS;
                if (!wait(&cb->item_empty[slot], ((it / SB_SLOTS) & 1) ^ 1)) { ok = false; break; }
                int im[BI_FIELDS] = {};
                if (lane == 0) {
                    const int t = atomicAdd(&p.hdr[HDR_TICKET], 1);
                    if (t < total) {
                        const int per = (p.by_length ? p.Hkv : ne) * p.nparts, outer = t / per, rest = t - outer * per;
                        const int inner = rest / p.nparts, part = rest - inner * p.nparts;
                        const int kvh = p.by_length ? inner : outer;
                        const int4 en = p.entries[p.by_length ? outer : inner];
                        im[BI_VALID] = 1;
                        im[BI_TOK0] = en.y;
                        im[BI_LEN] = en.z;
                        im[BI_BLK] = (en.z + BLK - 1) / BLK - 1 - en.w;  // the longest walk first
                        im[BI_KVH] = kvh;
                        im[BI_G0] = (int)((long long)p.G * part / p.nparts);
                        im[BI_G1] = (int)((long long)p.G * (part + 1) / p.nparts);
                        im[BI_PART] = part;
                    }
#pragma unroll
                    for (int f = 0; f < BI_FIELDS; ++f) cb->item[slot][f] = im[f];
                    mbar_arrive(&cb->item_full[slot]);
                }
#pragma unroll
                for (int f = 0; f < BI_FIELDS; ++f) im[f] = __shfl_sync(0xffffffffu, im[f], 0);
                ++it;
                if (!im[BI_VALID]) break;
                const int nblk = (im[BI_LEN] + BLK - 1) / BLK;
                for (int g = im[BI_G0]; g < im[BI_G1] && ok; ++g)
                    for (int i = im[BI_BLK]; i < nblk; ++i) {
                        const int s = n & 1;
                        if (!wait(&cb->q_empty[s], ((n >> 1) & 1) ^ 1)) { ok = false; break; }
                        if (lane == 0) {
                            const int h = im[BI_KVH] * p.G + g, row = im[BI_TOK0] + i * BLK;
                            uint8_t *at = smem + DKV_RING + s * 2 * TILE_BYTES;
                            mbar_expect_tx(&cb->q_full[s], 2 * TILE_BYTES);
                            tma_load_4d(at, &tmq, &cb->q_full[s], 0, h, row, 0, pol);
                            tma_load_4d(at + TILE_BYTES, &tmg, &cb->q_full[s], 0, h, row, 0, pol);
                        }
                        ++n;
                    }
            }
            for (uint32_t i = n > 2 ? n - 2 : 0; i < n; ++i) {  // copies land before the CTA exits
                drain_wait(&cb->q_full[i & 1], (i >> 1) & 1);
            }
            if (!ok) cb->abort = 1;
        } else if (warp == 1) {
            // ===================== MMA issuer =====================
            uint32_t it = 0, n = 0, items = 0;
            int cur[BI_FIELDS], nxt[BI_FIELDS];
            const uint32_t kt = sbase + DKV_K, vt = sbase + DKV_V;
            auto qt = [&](uint32_t m) -> uint32_t { return sbase + DKV_RING + (m & 1) * 2 * TILE_BYTES; };
            auto steps = [&](const int (&im)[BI_FIELDS]) -> int {
                return (im[BI_G1] - im[BI_G0]) * ((im[BI_LEN] + BLK - 1) / BLK - im[BI_BLK]);
            };
            // S^T of step m, the first of its item or not
            auto issue_s = [&](uint32_t m, bool first) -> bool {
                if (first) {
                    if (!wait(&cb->kv_full, items & 1)) return false;
                    ++items;
                }
                if (!wait(&cb->q_full[m & 1], (m >> 1) & 1) || !wait(&cb->rows_full[m & 1], (m >> 1) & 1)) return false;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss_w(TS, desc_kmajor(kt, kk), desc_kmajor(qt(m), kk), ID_SS, kk > 0 ? 1u : 0u);
                tc_commit_w(&cb->s_full);
                return true;
            };
            auto issue_dp = [&](uint32_t m, bool last) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss_w(TDP, desc_kmajor(vt, kk), desc_kmajor(qt(m) + TILE_BYTES, kk), ID_SS, kk > 0 ? 1u : 0u);
                tc_commit_w(&cb->dp_full);
                if (last) tc_commit_w(&cb->kv_empty);
            };
            bool ok = next(it, cur);
            int ns = ok ? steps(cur) : 0;
            if (ok) {
                ok = issue_s(0, true);
                if (ok) issue_dp(0, ns == 1);
            }
            while (ok) {
                bool more = false;
                int nns = 0;
                for (int j = 0; j < ns && ok; ++j, ++n) {
                    const bool last = j == ns - 1;
                    if (!wait(&cb->p_full, n & 1)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < BLK / 16; ++kk)
                        mma_ts_w(TDV, TS + half_cols(kk), desc_mnmajor(qt(n) + TILE_BYTES, kk), ID_TS, (j > 0 || kk > 0) ? 1u : 0u);
                    if (last) {
                        more = next(it, nxt);
                        nns = more ? steps(nxt) : 0;
                        if (cb->abort) { ok = false; break; }
                    }
                    if (!last || more) {
                        if (!issue_s(n + 1, last)) { ok = false; break; }
                    }
                    if (!wait(&cb->ds_full, n & 1)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < BLK / 16; ++kk)
                        mma_ts_w(TDK, TDP + half_cols(kk), desc_mnmajor(qt(n), kk), ID_TS, (j > 0 || kk > 0) ? 1u : 0u);
                    tc_commit_w(&cb->q_empty[n & 1]);
                    if (last) tc_commit_w(&cb->acc_full);
                    if (!last || more) issue_dp(n + 1, last ? nns == 1 : j + 1 == ns - 1);
                }
                if (!more) break;
                ns = nns;
#pragma unroll
                for (int f = 0; f < BI_FIELDS; ++f) cur[f] = nxt[f];
            }
            tc_commit_w(&cb->fin);
            drain_wait(&cb->fin, 0);
        } else if (warp == 2) {
            // ===================== K and V tiles =====================
            const uint64_t pol = policy_evict_first();
            uint32_t it = 0, n = 0;
            int im[BI_FIELDS];
            while (next(it, im)) {
                if (!wait(&cb->kv_empty, (n & 1) ^ 1)) break;
                if (lane == 0) {
                    const int row = im[BI_TOK0] + im[BI_BLK] * BLK;
                    mbar_expect_tx(&cb->kv_full, 2 * TILE_BYTES);
                    tma_load_4d(smem + DKV_K, &tmk, &cb->kv_full, 0, im[BI_KVH], row, 0, pol);
                    tma_load_4d(smem + DKV_V, &tmv, &cb->kv_full, 0, im[BI_KVH], row, 0, pol);
                }
                ++n;
            }
            if (n > 0) {
                drain_wait(&cb->kv_full, (n - 1) & 1);
            }
        } else {
            // ===================== rows of the steps =====================
            // A query row behind the sequence's end: lse2 = +inf makes its P zero, and
            // its Q and g rows (another sequence's) are zeroed.
            uint32_t it = 0, n = 0;
            int im[BI_FIELDS];
            bool ok = true;
            while (ok && next(it, im)) {
                const int nblk = (im[BI_LEN] + BLK - 1) / BLK;
                for (int g = im[BI_G0]; g < im[BI_G1] && ok; ++g)
                    for (int i = im[BI_BLK]; i < nblk; ++i, ++n) {
                        const int h = im[BI_KVH] * p.G + g, valid = min(BLK, im[BI_LEN] - i * BLK);
                        const size_t at = (size_t)h * p.T + im[BI_TOK0] + i * BLK;
                        float a[4], b[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int r = lane + 32 * k;
                            a[k] = r < valid ? p.lse2[at + r] : INFINITY;
                            b[k] = r < valid ? p.delta[at + r] : 0.f;
                        }
                        const int s = n & 1;
                        // (Q of the step landed, so the step two before has been used up)
                        if (!wait(&cb->q_full[s], (n >> 1) & 1)) { ok = false; break; }
                        float *rows = reinterpret_cast<float *>(smem + DKV_ROWS) + s * 2 * BLK;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            rows[lane + 32 * k] = a[k];
                            rows[BLK + lane + 32 * k] = b[k];
                        }
                        if (valid < BLK) {
                            uint8_t *tile = smem + DKV_RING + s * 2 * TILE_BYTES;
                            zero_rows(tile, valid, lane);
                            zero_rows(tile + TILE_BYTES, valid, lane);
                            fence_proxy_async_smem();
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&cb->rows_full[s]);
                    }
            }
        }
    } else {
        // ===================== P and dS: 64 query columns per warpgroup =====================
        reg_inc<216>();
        const int wg = (warp - 4) >> 2;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t trow = (uint32_t)(warp & 3) << 21;
        const uint32_t ts = TS + trow + wg * 64, tdp = TDP + trow + wg * 64;
        const float c = p.scale_log2;
        const bool wide = aligned32(wg ? p.dk : p.dv);
        uint32_t it = 0, n = 0, items = 0;
        int im[BI_FIELDS];
        bool ok = true;
        while (ok && next(it, im)) {
            const int nblk = (im[BI_LEN] + BLK - 1) / BLK;
            for (int g = im[BI_G0]; g < im[BI_G1] && ok; ++g)
                for (int i = im[BI_BLK]; i < nblk; ++i, ++n) {
                    const int s = n & 1;
                    const float4 *rows = reinterpret_cast<const float4 *>(smem + DKV_ROWS + s * 2 * BLK * 4) + wg * 16;
                    if (!wait(&cb->rows_full[s], (n >> 1) & 1) || !wait(&cb->s_full, n & 1)) { ok = false; break; }
                    tc_fence_after();
                    uint32_t x[64];
                    tmem_ld_cols<64>(ts, x);
                    float pr[64];
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const float4 ls = rows[q];
                        pr[4 * q] = ex2(fmaf(__uint_as_float(x[4 * q]), c, -ls.x));
                        pr[4 * q + 1] = ex2(fmaf(__uint_as_float(x[4 * q + 1]), c, -ls.y));
                        pr[4 * q + 2] = ex2(fmaf(__uint_as_float(x[4 * q + 2]), c, -ls.z));
                        pr[4 * q + 3] = ex2(fmaf(__uint_as_float(x[4 * q + 3]), c, -ls.w));
                    }
                    if (i == im[BI_BLK]) {  // the diagonal: a query sees the keys up to its own
                        const int lim = r - wg * 64;
#pragma unroll
                        for (int q = 0; q < 64; ++q)
                            if (q < lim) pr[q] = 0.f;
                    }
                    tmem_st_bf16x64(ts, pr);  // one rounding to bf16, for the tensor cores
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&cb->p_full);
                    if (!wait(&cb->dp_full, n & 1)) { ok = false; break; }
                    tc_fence_after();
                    tmem_ld_cols<64>(tdp, x);
                    if (i == 0) {  // a sequence's first rows: delta from this step, into its place among the rows
                        float *sums = reinterpret_cast<float *>(smem + DKV_SUMS) + wg * 4 * 64;
                        const int lim = r < im[BI_LEN] ? r - wg * 64 : 64;  // (a key behind the end may hold anything)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float v[32];
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                v[k] = half * 32 + k < lim ? 0.f : pr[half * 32 + k] * __uint_as_float(x[half * 32 + k]);
                            // over the warp's keys: lane l ends with column half * 32 + l
#pragma unroll
                            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                                for (int k = 0; k < o; ++k) {
                                    const float keep = lane & o ? v[k + o] : v[k], send = lane & o ? v[k] : v[k + o];
                                    v[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                                }
                            sums[(warp & 3) * 64 + half * 32 + lane] = v[0];
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&cb->sum_full[wg]);
                        if (!wait(&cb->sum_full[wg], 0)) { ok = false; break; }
                        if ((warp & 3) < 2) {
                            const int q = (warp & 3) * 32 + lane;
                            reinterpret_cast<float *>(smem + DKV_ROWS)[s * 2 * BLK + BLK + wg * 64 + q] =
                                (sums[q] + sums[64 + q]) + (sums[128 + q] + sums[192 + q]);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&cb->sum_full[wg]);
                        if (!wait(&cb->sum_full[wg], 1)) { ok = false; break; }
                    }
                    // On the diagonal what is hidden stays 0, also where its dP - delta is not
                    // finite.  (8 sequences of 60: 0.7 us; set to 0 once more, 1.3 us.)
                    auto times_dp = [&](int lim) {
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            const float4 de = rows[32 + q];
                            if (4 * q >= lim) pr[4 * q] *= __uint_as_float(x[4 * q]) - de.x;
                            if (4 * q + 1 >= lim) pr[4 * q + 1] *= __uint_as_float(x[4 * q + 1]) - de.y;
                            if (4 * q + 2 >= lim) pr[4 * q + 2] *= __uint_as_float(x[4 * q + 2]) - de.z;
                            if (4 * q + 3 >= lim) pr[4 * q + 3] *= __uint_as_float(x[4 * q + 3]) - de.w;
                        }
                    };
                    if (i == im[BI_BLK]) times_dp(r - wg * 64);
                    else times_dp(0);
                    tmem_st_bf16x64(tdp, pr);  // likewise one rounding
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&cb->ds_full);
                }
            if (!ok) break;
            // the sums: warpgroup 0 writes dv, warpgroup 1 dk (the next item's first
            // product into them waits for P and dS, which these warps deliver later)
            if (!wait(&cb->acc_full, items & 1)) break;
            ++items;
            tc_fence_after();
            const int row = im[BI_BLK] * BLK + r;
            const bool mine = row < im[BI_LEN];
            const size_t at = (((size_t)im[BI_TOK0] + row) * p.Hkv + im[BI_KVH]) * D;
            const float f = wg ? p.scale : 1.f;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld_wait32((wg ? TDK : TDV) + trow + q * 32, o);
                if (mine && p.parts) {
                    scale32(o, f);
                    float *to = p.parts + ((size_t)im[BI_PART] * 2 + wg) * p.T * p.Hkv * D + at + q * 32;
#pragma unroll
                    for (int k = 0; k < 4; ++k) st_global_v8(to + 8 * k, o + 8 * k);  // (the workspace is 256-byte aligned)
                } else if (mine) {
                    store_row32((wg ? p.dk : p.dv) + at + q * 32, o, f, wide);
                }
            }
            tc_fence_before();
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// dk, dv = the sums of their parts, in order (4 elements a thread)
__global__ void __launch_bounds__(256) la_softmax_dkv_sum_kernel(const int *hdr, const float *parts, int nparts,
                                                                 long long n, __nv_bfloat16 *dk, __nv_bfloat16 *dv) {
    if (hdr[HDR_G] == 0) return;  // the tables were refused
    const long long quads = n / 4;
    for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < 2 * quads; e += (long long)gridDim.x * 256) {
        const int which = e >= quads;  // 0: dv, 1: dk
        const long long i = e - which * quads;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int q = 0; q < nparts; ++q) {
            const float4 x = reinterpret_cast<const float4 *>(parts + ((size_t)q * 2 + which) * n)[i];
            s.x += x.x;
            s.y += x.y;
            s.z += x.z;
            s.w += x.w;
        }
        reinterpret_cast<uint2 *>(which ? dk : dv)[i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
    }
}

// ---------------------------------------------------------------------------
// dq.  Per key block of a query block, query rows and key columns:
//     S = Q K^T (two buffers),  dP = g V^T      (SS MMAs)
//     dS = 2^(c S - lse2) (dP - delta)          -> TMEM, bf16
//     dq += dS K                                (TS MMA)
// issued as dq, dP', S'' | ...: P of the next block is formed while the tensor
// pipe adds this one's dq.  TMEM: S0 | S1 | dP | dq.  (Slower, 16000 tokens and 2
// heads, 157 us: one S buffer with Q and g in TMEM, where a first operand takes no
// shared-memory bandwidth, 164; one S buffer, g in TMEM and columns of its own for
// dS, so that the next dP does not wait for dq, 175.)
// ---------------------------------------------------------------------------
constexpr int DQ_STAGES = 5;
constexpr int DQ_Q = 0, DQ_G = TILE_BYTES, DQ_RING = 2 * TILE_BYTES;
constexpr int DQ_CTRL = DQ_RING + DQ_STAGES * TILE_BYTES;
constexpr int DQ_SUMS = DQ_CTRL + 512;               // [2][128] rows
constexpr int DQ_SMEM = DQ_SUMS + 2 * BLK * 4;
static_assert(DKV_SMEM <= 227 * 1024 && DQ_SMEM <= 227 * 1024, "shared memory of one CTA");

struct DqCtrl {
    uint64_t kv_full[DQ_STAGES], kv_empty[DQ_STAGES];
    uint64_t q_full, q_empty;             // [1], [1]
    uint64_t s_full[2];                   // [1]
    uint64_t dp_full, ds_full;            // [1], [8]
    uint64_t sum_full;                    // [8] the halves of exact deltas
    uint64_t acc_full;                    // [1]
    uint64_t item_full[SB_SLOTS], item_empty[SB_SLOTS];  // [1], [10]
    uint64_t fin;
    int item[SB_SLOTS][8];
    uint32_t tmem_base;
    volatile int abort;
};
static_assert(sizeof(DqCtrl) <= 512, "control block");

__global__ void __launch_bounds__(SB_THREADS, 1)
la_softmax_dq_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmg,
                     const __grid_constant__ SoftmaxBwdParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    DqCtrl *cb = reinterpret_cast<DqCtrl *>(smem + DQ_CTRL);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t sbase = smem_u32(smem);
    if (sbase & 1023) {
        if (threadIdx.x == 0) record_status(p.status, ST_CUDA);
        return;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < DQ_STAGES; ++s) {
            mbar_init(&cb->kv_full[s], 1);
            mbar_init(&cb->kv_empty[s], 1);
        }
        mbar_init(&cb->q_full, 1);
        mbar_init(&cb->q_empty, 1);
        mbar_init(&cb->s_full[0], 1);
        mbar_init(&cb->s_full[1], 1);
        mbar_init(&cb->dp_full, 1);
        mbar_init(&cb->ds_full, 8);
        mbar_init(&cb->sum_full, 8);
        mbar_init(&cb->acc_full, 1);
        for (int s = 0; s < SB_SLOTS; ++s) {
            mbar_init(&cb->item_full[s], 1);
            mbar_init(&cb->item_empty[s], 10);  // MMA, Q and 8 softmax warps
        }
        mbar_init(&cb->fin, 1);
        cb->abort = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
        tma_prefetch_desc(&tmg);
        // The tables, lse2, delta and the inputs come from kernels in front of the one of dk and
        // dv, whose end this one does not wait for here.  That one's first CTA has waited for
        // them and released HDR_READY before this kernel could start, so the acquire succeeds
        // at once; it orders, through the barrier below, all reads of this CTA behind them.
        // (Beside the allocation of TMEM: 0 to 0.3 us a call; behind it 0.1 to 0.8.)
        const uint64_t deadline = globaltimer_ns() + p.wait_limit_ns;
        for (int ready = 0;;) {
            asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(ready) : "l"(p.hdr + HDR_READY) : "memory");
            if (ready == 1) break;
            if (globaltimer_ns() > deadline) {
                record_status(p.status, ST_TIMEOUT);
                cb->abort = 1;
                break;
            }
        }
    }
    if (warp == 1) {
        tmem_alloc(&cb->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, cb->tmem_base, 0);
    const uint32_t TS = tmem, TDP = tmem + 256, TDQ = tmem + 384;  // S of step m: TS + (m & 1) * 128
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return ctrl_warp_wait(bar, parity, p.wait_limit_ns, p.status, cb);
    };
    auto next = [&](uint32_t &it, int (&item)[BI_FIELDS]) -> bool {
        return sb_next(it, item, lane, p.wait_limit_ns, p.status, cb);
    };

    if (warp < 4) {
        reg_dec<72>();
        if (warp == 0) {
            // ===================== items, K and V tiles =====================
            const uint64_t pol = policy_evict_last();
            bool ok = __shfl_sync(0xffffffffu, cb->abort, 0) == 0;
            const int ne = ok ? p.hdr[HDR_G] : 0;
            const long long total = (long long)ne * p.H;
            uint32_t it = 0, n = 0;
            while (ok) {
                const int slot = it % SB_SLOTS;
                if (!wait(&cb->item_empty[slot], ((it / SB_SLOTS) & 1) ^ 1)) { ok = false; break; }
                int im[BI_FIELDS] = {};
                if (lane == 0) {
                    const int t = atomicAdd(&p.hdr[HDR_TICKET2], 1);
                    if (t < total) {
                        const int per = (p.by_length ? p.Hkv : ne) * p.G, outer = t / per, rest = t - outer * per;
                        const int inner = rest / p.G;
                        const int kvh = p.by_length ? inner : outer;
                        const int4 en = p.entries[p.by_length ? outer : inner];
                        im[BI_VALID] = 1;
                        im[BI_TOK0] = en.y;
                        im[BI_LEN] = en.z;
                        im[BI_BLK] = en.w;
                        im[BI_KVH] = kvh;
                        im[BI_G0] = rest % p.G;
                    }
#pragma unroll
                    for (int f = 0; f < BI_FIELDS; ++f) cb->item[slot][f] = im[f];
                    mbar_arrive(&cb->item_full[slot]);
                }
#pragma unroll
                for (int f = 0; f < BI_FIELDS; ++f) im[f] = __shfl_sync(0xffffffffu, im[f], 0);
                ++it;
                if (!im[BI_VALID]) break;
                for (int j = 0; j <= im[BI_BLK] && ok; ++j)
                    for (int kv = 0; kv < 2; ++kv) {
                        const int s = n % DQ_STAGES;
                        if (!wait(&cb->kv_empty[s], ((n / DQ_STAGES) & 1) ^ 1)) { ok = false; break; }
                        if (lane == 0) {
                            mbar_expect_tx(&cb->kv_full[s], TILE_BYTES);
                            tma_load_4d(smem + DQ_RING + s * TILE_BYTES, kv ? &tmv : &tmk, &cb->kv_full[s], 0,
                                        im[BI_KVH], im[BI_TOK0] + j * BLK, 0, pol);
                        }
                        ++n;
                    }
            }
            for (uint32_t i = n > DQ_STAGES ? n - DQ_STAGES : 0; i < n; ++i) {
                drain_wait(&cb->kv_full[i % DQ_STAGES], (i / DQ_STAGES) & 1);
            }
            if (!ok) cb->abort = 1;
        } else if (warp == 1) {
            // ===================== MMA issuer =====================
            // Steps are counted across items; step m has K at ring position 2 m and V
            // at 2 m + 1.  S is issued up to two steps ahead, into the item behind too.
            uint32_t it = 0, items = 0;
            int cur[BI_FIELDS], nxt[BI_FIELDS];
            auto tile = [&](uint32_t pos) -> uint32_t { return sbase + DQ_RING + (pos % DQ_STAGES) * TILE_BYTES; };
            auto landed = [&](uint32_t pos) -> bool {
                return wait(&cb->kv_full[pos % DQ_STAGES], (pos / DQ_STAGES) & 1);
            };
            auto issue_s = [&](uint32_t m, bool first) -> bool {
                if (first) {
                    if (!wait(&cb->q_full, items & 1)) return false;
                    ++items;
                }
                if (!landed(2 * m)) return false;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss_w(TS + (m & 1) * 128, desc_kmajor(sbase + DQ_Q, kk), desc_kmajor(tile(2 * m), kk), ID_SS, kk > 0 ? 1u : 0u);
                tc_commit_w(&cb->s_full[m & 1]);
                return true;
            };
            auto issue_dp = [&](uint32_t m, bool last) -> bool {
                if (!landed(2 * m + 1)) return false;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss_w(TDP, desc_kmajor(sbase + DQ_G, kk), desc_kmajor(tile(2 * m + 1), kk), ID_SS, kk > 0 ? 1u : 0u);
                tc_commit_w(&cb->dp_full);
                tc_commit_w(&cb->kv_empty[(2 * m + 1) % DQ_STAGES]);
                if (last) tc_commit_w(&cb->q_empty);  // every S of the item came before
                return true;
            };
            uint32_t n = 0;
            bool ok = next(it, cur);
            while (ok) {
                // Q and g are the item's own, so S runs ahead inside an item only
                const int ns = cur[BI_BLK] + 1;
                ok = issue_s(n, true) && (ns == 1 || issue_s(n + 1, false)) && issue_dp(n, ns == 1);
                for (int j = 0; j < ns && ok; ++j, ++n) {
                    const bool last = j == ns - 1;
                    const int valid = cur[BI_LEN] - cur[BI_BLK] * BLK;
                    if (last && valid < BLK) {  // key rows behind the sequence's end meet dS = 0
                        zero_rows(smem + DQ_RING + ((2 * n) % DQ_STAGES) * TILE_BYTES, valid, lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (!wait(&cb->ds_full, n & 1)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < BLK / 16; ++kk)
                        mma_ts_w(TDQ, TDP + half_cols(kk), desc_mnmajor(tile(2 * n), kk), ID_TS, (j > 0 || kk > 0) ? 1u : 0u);
                    tc_commit_w(&cb->kv_empty[(2 * n) % DQ_STAGES]);
                    if (last) {
                        tc_commit_w(&cb->acc_full);
                    } else {
                        ok = issue_dp(n + 1, j + 1 == ns - 1);
                        if (ok && j + 2 < ns) ok = issue_s(n + 2, false);
                    }
                }
                if (!ok || !next(it, nxt)) break;
#pragma unroll
                for (int f = 0; f < BI_FIELDS; ++f) cur[f] = nxt[f];
            }
            tc_commit_w(&cb->fin);
            drain_wait(&cb->fin, 0);
        } else if (warp == 2) {
            // ===================== Q and g tiles =====================
            const uint64_t pol = policy_evict_first();
            uint32_t it = 0, n = 0;
            int im[BI_FIELDS];
            while (next(it, im)) {
                if (!wait(&cb->q_empty, (n & 1) ^ 1)) break;
                if (lane == 0) {
                    const int h = im[BI_KVH] * p.G + im[BI_G0], row = im[BI_TOK0] + im[BI_BLK] * BLK;
                    mbar_expect_tx(&cb->q_full, 2 * TILE_BYTES);
                    tma_load_4d(smem + DQ_Q, &tmq, &cb->q_full, 0, h, row, 0, pol);
                    tma_load_4d(smem + DQ_G, &tmg, &cb->q_full, 0, h, row, 0, pol);
                }
                ++n;
            }
            if (n > 0) {
                drain_wait(&cb->q_full, (n - 1) & 1);
            }
        }
    } else {
        // ===================== dS: 64 key columns per warpgroup =====================
        reg_inc<216>();
        const int wg = (warp - 4) >> 2;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t trow = (uint32_t)(warp & 3) << 21;
        const uint32_t tdp = TDP + trow + wg * 64;
        const float c = p.scale_log2;
        const bool wide = aligned32(p.dq);
        uint32_t it = 0, n = 0, items = 0, firsts = 0;
        int im[BI_FIELDS];
        bool ok = true;
        while (ok && next(it, im)) {
            const int h = im[BI_KVH] * p.G + im[BI_G0], row = im[BI_BLK] * BLK + r;
            const bool mine = row < im[BI_LEN];
            const size_t st = (size_t)h * p.T + im[BI_TOK0] + row;
            const float ls = mine ? p.lse2[st] : 0.f;
            float de = mine ? p.delta[st] : 0.f;
            const int ns = im[BI_BLK] + 1;
            for (int j = 0; j < ns; ++j, ++n) {
                // each S buffer's phase advances once per two steps
                if (!wait(&cb->s_full[n & 1], (n >> 1) & 1)) { ok = false; break; }
                tc_fence_after();
                uint32_t x[64];
                tmem_ld_cols<64>(TS + trow + (n & 1) * 128 + wg * 64, x);
                float pr[64];
#pragma unroll
                for (int q = 0; q < 64; ++q) pr[q] = ex2(fmaf(__uint_as_float(x[q]), c, -ls));
                if (!wait(&cb->dp_full, n & 1)) { ok = false; break; }
                tc_fence_after();
                tmem_ld_cols<64>(tdp, x);
                if (ns == 1) {  // a sequence's first rows: delta from this step
                    float *sums = reinterpret_cast<float *>(smem + DQ_SUMS);
                    const int lim = r - wg * 64;
                    float sum = 0.f;
#pragma unroll
                    for (int q = 0; q < 64; ++q)
                        if (q <= lim) sum = fmaf(pr[q], __uint_as_float(x[q]), sum);
                    // (read by both warpgroups before ds_full, and so before the next item's)
                    sums[wg * BLK + r] = sum;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&cb->sum_full);
                    if (!wait(&cb->sum_full, firsts & 1)) { ok = false; break; }
                    ++firsts;
                    de = sums[r] + sums[BLK + r];
                }
#pragma unroll
                for (int q = 0; q < 64; ++q) pr[q] *= __uint_as_float(x[q]) - de;
                if (j == ns - 1) {  // the diagonal; what it hides may hold anything
                    const int lim = r - wg * 64;
#pragma unroll
                    for (int q = 0; q < 64; ++q)
                        if (q > lim) pr[q] = 0.f;
                }
                tmem_st_bf16x64(tdp, pr);  // one rounding to bf16, for the tensor cores
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&cb->ds_full);
            }
            if (!ok) break;
            if (!wait(&cb->acc_full, items & 1)) break;
            ++items;
            tc_fence_after();
            __nv_bfloat16 *to = p.dq + (((size_t)im[BI_TOK0] + row) * p.H + h) * D + wg * 64;
#pragma unroll 1
            for (int q = 0; q < 2; ++q) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld_wait32(TDQ + trow + wg * 64 + q * 32, o);
                if (mine) store_row32(to + q * 32, o, p.scale, wide);
            }
            tc_fence_before();
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
    // This kernel may have run beside the one of dk and dv; it ends no earlier.
    pdl_wait();
}

}  // namespace la
