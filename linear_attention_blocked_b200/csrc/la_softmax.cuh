// la_softmax.cuh -- causal softmax attention over whole prompts for sm_100a,
// with grouped key/value heads, on packed sequences or behind a paged cache.
//
// Per sequence and query head, with past cached tokens in front of its n new
// ones and pos(t) = past + t:
//
//     o_t = sum_{s <= pos(t)} p_ts v_s,   p_ts = exp(scale q_t . k_s - lse_t)
//     lse_t = log sum_{s <= pos(t)} exp(scale q_t . k_s)
//
// in one pass over the keys with a running maximum m and sum l per row:
//     x = Q K_j^T,  m' = max(m, rowmax x),  P = 2^(c x - c m'),  c = scale log2 e
//     l <- 2^(c m - c m') l + rowsum P,  O <- 2^(c m - c m') O + P V_j.
// m may lag behind the true maximum as long as 2^(c x - c m) stays small: a row
// rescales O only when its maximum has grown by more than 2^RESCALE_LOG2 since
// the m in use (P then stays below 2^8, exact in fp32 sums; bf16 P has the same
// relative rounding at any magnitude), which after the first tiles is rare.
//
// One CTA works on a pair of query tiles (128 rows of one query head each)
// that read the same K and V tiles: two query heads of the same key/value
// head and the same rows, or, where a group has an odd number of heads, the
// pairs that its heads' tiles over 256 rows fall into.  Every step of a tile
// is S = Q K_j^T (SS MMA), softmax by one warpgroup (a thread per row), and
// O += P V_j (TS MMA, P as bf16 in TMEM over its scores).  The two tiles take
// turns: the tensor pipe runs P V and the next S of one while the other is in
// its softmax, so neither waits as long as a softmax is no slower than two
// products (1024 cycles at 128 x 128 x 128).
//
// The tensor pipe runs MMAs in issue order, so S_{j+1} may be issued over the
// buffer that P V_j reads, right behind it.
//
// Warp roles (512 threads, registers split by setmaxnreg):
//   warp 0       items and K/V tiles (TMA)         warpgroup 0: 48 registers
//   warp 1       TMEM allocator + MMA issuer
//   warp 2       Q tiles (TMA)
//   warp 3       (small chunks) new tokens into their pages
//   warps 4-7    softmax of tile 0                 192 registers
//   warps 8-11   softmax of tile 1                 192 registers
//   warps 12-15  output: O / l, lse                80 registers
// Shared memory: Q 2 x 32 KiB | ring of 5 x 32 KiB K and V tiles in turn |
// barriers.  TMEM (512 columns): S0 | S1 | O0 | O1.
//
// What bounds it: the exponentials (16 a cycle and SM) take as many cycles as the two
// products, and an S product reads both operands from shared memory, at little more
// than half its rate.  8192 tokens, 16 heads over 2: 215 us, 1278 TFLOP/s of causal
// pairs, both units busy 63 % of the cycles.  32768 tokens, 32 heads over 4: 7.0 to
// 7.5 ms, 1170 to 1250 TFLOP/s, at the power limit (clock near 1.6 of 1.965 GHz).
// Slower or no faster there: a polynomial for part of the exponentials, four softmax
// warpgroups of half a row, two MMA warps, P handed over in halves.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include "la_prefill.cuh"
#include "la_ptx.cuh"

namespace la {

constexpr int ST_CUDA = 3;  // device status code (matches la_status)

constexpr int SMX_THREADS = 512;
constexpr int SMX_STAGES = 5;
constexpr int SMX_Q = 0;
constexpr int SMX_KV = 2 * TILE_BYTES;
constexpr int SMX_CTRL = SMX_KV + SMX_STAGES * TILE_BYTES;
constexpr int SMX_STAT = SMX_CTRL + 576;                    // {c m, l} of both tiles' rows
constexpr int SMX_SMEM = SMX_STAT + 2 * BLK * 8;            // (1024-byte aligned as it is)
static_assert(SMX_SMEM <= 227 * 1024, "shared memory of one CTA");
constexpr uint32_t SMX_TM_S = 0, SMX_TM_O = 256;            // tile t: + 128 t
constexpr int HDR_TICKET2 = 3;                              // second ticket counter of the workspace header
constexpr int HDR_READY = 4;                                // gradients: dkv has seen the tables and rows
constexpr int SMX_SLOTS = 4;                                // item queue
constexpr float RESCALE_LOG2 = 8.f;
constexpr int SMX_CTAS = 148;                               // split: runs of key tiles
constexpr int SMX_PART = D + 4;                             // floats of a row's part: O, c m, l

// Entries: the row blocks of every sequence, sequence by sequence, each from
// its last block (the longest row of keys) to its first, or (by_length) those of
// all sequences from the longest row of keys to the shortest.
struct SoftmaxScheduleParams {
    const int *cu;            // device cu_seqlens [nseq + 1]
    const int *past;          // device [nseq] cached tokens, or null (none)
    int nseq, T, max_seqlen;
    long long max_keys;       // bound on past + new tokens of a sequence (paged)
    int rows;                 // rows per entry: 128 or 256
    int items_per_entry;
    int by_length;
    int *hdr;                 // workspace header
    int *prefix;              // [nseq + 1] entries before each sequence
    int4 *entries;            // {sequence, first token, length, block}
    int *status;
};

struct SoftmaxPrefillParams {
    __nv_bfloat16 *out;       // [T, H, D]
    float *lse;               // [T, H]
    int *hdr;
    const int4 *entries;
    const int *past;          // device [nseq] or null
    const int *pages;         // device [nseq, max_pages] page table, or null (no cache)
    int max_pages, n_pages, page, page_shift;
    // direct: every CTA has one item at most and finds it in cu itself; split: it
    // has a run of key tiles, equal to the others', of whichever items they are of
    int direct, split;
    float *parts;             // split: [SMX_CTAS][2][2 tiles][128][SMX_PART] O, m, l of cut items
    int4 *info;               // split: [SMX_CTAS][3] the item cut at the CTA's end
    const int *cu;            // device [nseq + 1] (direct, append)
    int nseq, T, max_seqlen;
    long long max_keys;       // room of a sequence's pages
    // new tokens that this kernel writes into their pages (direct), or null
    const __nv_bfloat16 *new_k, *new_v;
    __nv_bfloat16 *kc, *vc;
    int H, Hkv, G;
    int pairs;                // pairs of query tiles per entry
    int rows;
    int by_length;            // entries are in order of length: all heads of an entry in turn
    float scale_log2;         // scale * log2(e)
    unsigned long long wait_limit_ns;
    int *status;
};

// item fields
enum { SI_VALID = 0, SI_H0, SI_H1, SI_B0, SI_B1, SI_N0, SI_N1, SI_TOK0, SI_LEN, SI_PAST, SI_KVH, SI_SEQ, SI_J0, SI_PART, SI_FIELDS };
// N0, N1: key tiles of the two query tiles: those of the cached tokens, then those
// of the new ones up to the query tile's own rows.  A piece of an item (split) has
// N0, N1 of them from tile J0 on; PART: the slot for its part of the sums, or -1.

struct SoftmaxCtrl {
    uint64_t kv_full[SMX_STAGES], kv_empty[SMX_STAGES];
    uint64_t q_full[2], q_empty[2];   // per tile
    uint64_t s_full[2];               // [1] scores of the tile's next step
    uint64_t p_full[2];               // [4] P of the step in TMEM (and O rescaled)
    uint64_t o_full[2];               // [1] all of an item's P V added to O
    uint64_t o_empty[2];              // [4] output warps have read O
    uint64_t stat_full[2];            // [4] m and l of the tile's rows written
    uint64_t stat_empty[2];           // [4] output warps have read them
    uint64_t item_full[SMX_SLOTS];    // [1]
    uint64_t item_empty[SMX_SLOTS];   // [14] Q, MMA, 8 softmax and 4 output warps
    uint64_t fin;                     // [1] tear-down: every MMA done
    int item[SMX_SLOTS][16];
    uint32_t tmem_base;
    volatile int abort;
};
static_assert(sizeof(SoftmaxCtrl) <= 576, "control block");
static_assert(SI_FIELDS <= 16, "item fields");

// Programmatic dependent launch: wait for the kernel before this one in the
// stream to end (when it was launched so; else a no-op); let the next one start.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// 2^x (the PTX instruction: relative error 2^-22, 0 for -inf)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---- pairs of fp32 values in one 64-bit register (packed fp32 instructions) ----
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// One thread's row of 32 fp32 TMEM columns, times f, as bf16.  Whole sectors where
// the tensor's address allows it (wide: 32-byte aligned; rows are then, too): in
// 16-byte stores 48 prompts of 512 tokens, 64 heads over 8, take 416 us instead of
// 396, 12 of up to 4059 1396 instead of 1367.
__device__ __forceinline__ bool aligned32(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }
__device__ __forceinline__ void store_row32(__nv_bfloat16 *to, uint32_t (&o)[32], float f, bool wide) {
    scale32(o, f);
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
    if (wide) {
        st_global_v8(to, w);
        st_global_v8(to + 16, w + 8);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<uint4 *>(to)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
}

// Bounded waits of a control block with `abort`: as wait_or_abort above.
template <class Ctrl>
__device__ __forceinline__ bool ctrl_wait(uint64_t *bar, uint32_t parity, unsigned long long limit_ns, int *status,
                                          Ctrl *cb) {
    if (mbar_try_wait(bar, parity)) return true;
    if (la_wait(bar, parity, globaltimer_ns() + limit_ns, &cb->abort)) return true;
    cb->abort = 1;
    record_status(status, ST_TIMEOUT);
    return false;
}
template <class Ctrl>
__device__ __forceinline__ bool ctrl_warp_wait(uint64_t *bar, uint32_t parity, unsigned long long limit_ns,
                                               int *status, Ctrl *cb) {
    return __all_sync(0xffffffffu, ctrl_wait(bar, parity, limit_ns, status, cb)) != 0;
}

// Before a CTA ends, what it has in flight does: copies into its shared memory, products
// into its TMEM.  They end by themselves, also where a wait has run out, and take
// microseconds; so this wait has a limit of its own, which no setting shortens.
constexpr unsigned long long DRAIN_NS = 2000000000ull;
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity) {
    int go_on = 0;
    la_wait(bar, parity, globaltimer_ns() + DRAIN_NS, &go_on);
}

// The next item of the queue; a role reads the fields of its MASK.
template <uint32_t MASK>
__device__ __forceinline__ bool smx_next(uint32_t &it, int (&item)[SI_FIELDS], int lane,
                                         const SoftmaxPrefillParams &p, SoftmaxCtrl *cb) {
    const int slot = it % SMX_SLOTS;
    item[SI_VALID] = 0;
    if (!ctrl_warp_wait(&cb->item_full[slot], (it / SMX_SLOTS) & 1, p.wait_limit_ns, p.status, cb)) return false;
#pragma unroll
    for (int f = 0; f < SI_FIELDS; ++f)
        if (f == SI_VALID || ((MASK >> f) & 1)) item[f] = __shfl_sync(0xffffffffu, cb->item[slot][f], 0);
    if (lane == 0) mbar_arrive(&cb->item_empty[slot]);
    ++it;
    return item[SI_VALID] != 0;
}

// The item of (key/value head, entry, pair of tiles).
__device__ __forceinline__ void smx_item(int kvh, int4 en, int pair, const SoftmaxPrefillParams &p, int *item) {
    const int past = p.past ? p.past[en.x] : 0;
    const int bpe = p.rows / BLK;  // blocks per entry
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int u = 2 * pair + w;
        const int b = en.w * bpe + u / p.G;
        item[SI_H0 + w] = kvh * p.G + u % p.G;
        item[SI_B0 + w] = b;
        item[SI_N0 + w] = (u < bpe * p.G && b * BLK < en.z) ? (past + BLK - 1) / BLK + b + 1 : 0;
    }
    item[SI_TOK0] = en.y;
    item[SI_LEN] = en.z;
    item[SI_PAST] = past;
    item[SI_KVH] = kvh;
    item[SI_SEQ] = en.x;
    item[SI_J0] = 0;
    item[SI_PART] = -1;
}

// Is sequence i of the tables as the header asks?
__device__ __forceinline__ bool smx_sequence_ok(int i, int a, int b, const int *past, int T, int max_seqlen,
                                                long long max_keys) {
    if (a < 0 || b < a || b > T || b - a > max_seqlen) return false;
    if (!past || b == a) return true;
    return past[i] >= 0 && (long long)past[i] + (b - a) <= max_keys;
}

// Entry e by a warp's own walk over cu_seqlens, checking all of it as the
// scheduler does: its number of entries, 0 when the tables are refused.
__device__ __forceinline__ int smx_find(int e, int lane, const SoftmaxPrefillParams &p, int4 &en) {
    int at = 0;
    bool bad = lane == 0 && (p.cu[0] != 0 || p.cu[p.nseq] != p.T);
    for (int base = 0; base < p.nseq; base += 32) {
        const int i = base + lane;
        int a = 0, b = 0;
        if (i < p.nseq) {
            a = p.cu[i];
            b = p.cu[i + 1];
            if (!smx_sequence_ok(i, a, b, p.past, p.T, p.max_seqlen, p.max_keys)) {
                bad = true;
                b = a;
            }
        }
        const int n = (b - a + p.rows - 1) / p.rows;
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        const int first = at + x - n;
        const uint32_t hit = __ballot_sync(0xffffffffu, e >= first && e < first + n);
        if (hit) {
            const int src = __ffs(hit) - 1;
            en = make_int4(base + src, __shfl_sync(0xffffffffu, a, src), __shfl_sync(0xffffffffu, b - a, src),
                           __shfl_sync(0xffffffffu, first + n - 1 - e, src));
        }
        at += __shfl_sync(0xffffffffu, x, 31);
    }
    if (__any_sync(0xffffffffu, bad)) {
        if (lane == 0) record_status(p.status, ST_INVALID);
        return 0;
    }
    return at;
}

// Split: the key tiles of all items are laid end to end, entry by entry, all items
// of an entry with as many tiles as its longest, and cut into equal runs.
struct SplitCursor {
    int seq, blk, tok0, len, past, cost;  // the entry, and tiles of each of its items
    int rest, j;                          // item of the entry, tile of the item
    int n;                                // CTAs with a run
    long long u, u1, total;               // this run's place and end among all tiles
};

__device__ __forceinline__ int smx_cost(int blk, int len, int past, int bpe) {
    return (past + BLK - 1) / BLK + min((blk + 1) * bpe, (len + BLK - 1) / BLK);
}

// A warp finds its CTA's run; false without one.  Checks the tables like smx_find.
__device__ __forceinline__ bool smx_split(SplitCursor &c, int lane, const SoftmaxPrefillParams &p) {
    const int bpe = p.rows / BLK;
    const long long hp = (long long)p.Hkv * p.pairs;
    bool bad = lane == 0 && (p.cu[0] != 0 || p.cu[p.nseq] != p.T);
    long long at = 0;
    c.total = 0;
    for (int pass = 0; pass < 2; ++pass) {  // the sum, then the run's first entry
        for (int base = 0; base < p.nseq; base += 32) {
            const int i = base + lane;
            long long mine = 0;
            int a = 0, len = 0, past = 0;
            if (i < p.nseq) {
                a = p.cu[i];
                const int b = p.cu[i + 1];
                if (smx_sequence_ok(i, a, b, p.past, p.T, p.max_seqlen, p.max_keys)) {
                    len = b - a;
                    past = p.past && len ? p.past[i] : 0;
                } else {
                    bad = true;
                }
                for (int blk = 0; blk < (len + p.rows - 1) / p.rows; ++blk) mine += smx_cost(blk, len, past, bpe);
            }
            long long incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            if (pass == 0) {
                c.total += __shfl_sync(0xffffffffu, incl, 31) * hp;
                continue;
            }
            const long long first = (at + incl - mine) * hp;
            const uint32_t hit = __ballot_sync(0xffffffffu, c.u >= first && c.u < first + mine * hp);
            at += __shfl_sync(0xffffffffu, incl, 31);
            if (!hit) continue;
            const int src = __ffs(hit) - 1;
            c.seq = base + src;
            c.tok0 = __shfl_sync(0xffffffffu, a, src);
            c.len = __shfl_sync(0xffffffffu, len, src);
            c.past = __shfl_sync(0xffffffffu, past, src);
            long long rem = c.u - __shfl_sync(0xffffffffu, first, src);
            for (c.blk = (c.len + p.rows - 1) / p.rows - 1;; --c.blk) {
                c.cost = smx_cost(c.blk, c.len, c.past, bpe);
                if (rem < c.cost * hp) break;
                rem -= c.cost * hp;
            }
            c.rest = (int)(rem / c.cost);
            c.j = (int)(rem % c.cost);
            return true;
        }
        if (pass == 0) {
            if (__any_sync(0xffffffffu, bad)) {
                if (lane == 0) record_status(p.status, ST_INVALID);
                return false;
            }
            // (a run of less than four tiles would not pay)
            c.n = (int)min((long long)gridDim.x, (c.total + 3) / 4);
            if ((int)blockIdx.x >= c.n) return false;
            c.u = c.total * blockIdx.x / c.n;
            c.u1 = c.total * (blockIdx.x + 1) / c.n;
        }
    }
    return false;
}

// The run's next piece into `item` (one thread); false at its end.
__device__ __forceinline__ bool smx_piece(SplitCursor &c, const SoftmaxPrefillParams &p, int *item) {
    const int bpe = p.rows / BLK;
    while (c.u < c.u1) {
        const int j0 = c.j, take = (int)min((long long)(c.cost - c.j), c.u1 - c.u);
        smx_item(c.rest / p.pairs, make_int4(c.seq, c.tok0, c.len, c.blk), c.rest % p.pairs, p, item);
        const int n0 = item[SI_N0], n1 = item[SI_N1], nmax = max(n0, n1);
        const long long begin = c.u - j0;  // the item's first tile among all
        c.u += take;
        c.j += take;
        if (c.j == c.cost) {
            c.j = 0;
            if (++c.rest == p.Hkv * p.pairs && c.u < c.u1) {
                c.rest = 0;
                if (--c.blk < 0) {
                    do {
                        ++c.seq;
                        c.tok0 = p.cu[c.seq];
                        c.len = p.cu[c.seq + 1] - c.tok0;
                    } while (c.len == 0);
                    c.past = p.past ? p.past[c.seq] : 0;
                    c.blk = (c.len + p.rows - 1) / p.rows - 1;
                }
                c.cost = smx_cost(c.blk, c.len, c.past, bpe);
            }
        }
        if (j0 >= nmax) continue;  // this item has fewer tiles than the entry's longest
        item[SI_N0] = max(0, min(n0 - j0, take));
        item[SI_N1] = max(0, min(n1 - j0, take));
        item[SI_J0] = j0;
        if (j0 == 0 && take >= nmax) return true;  // whole
        item[SI_PART] = j0 == 0 ? 1 : 0;           // (a run cuts one item at either end)
        if (j0 == 0) {
            const int parts = (int)(((begin + nmax) * c.n - 1) / c.total) - (int)blockIdx.x + 1;
            int4 *in = p.info + 3 * blockIdx.x;
            in[0] = make_int4(parts, item[SI_TOK0], item[SI_LEN], 0);
            in[1] = make_int4(item[SI_H0], item[SI_H1], item[SI_B0], item[SI_B1]);
            in[2] = make_int4(n0, n1, 0, 0);
        }
        return true;
    }
    return false;
}

// The pages that hold keys [key0, key0 + 128) of a sequence with `keys` cached
// ones, as one K or V tile.  Called by a whole warp: lane i brings page i of the
// tile (both halves); what lies behind the last key's page is not loaded.
__device__ __forceinline__ void smx_load_pages(uint8_t *dst, const CUtensorMap *tm, uint64_t *bar, int kvh, int key0,
                                               int keys, int pid, int lane, uint64_t pol,
                                               const SoftmaxPrefillParams &p) {
    const int np = (min(keys - key0, BLK) + p.page - 1) >> p.page_shift;
    if (lane == 0) mbar_expect_tx(bar, (uint32_t)(np * p.page * D * 2));
    __syncwarp();
    if (lane < np) {
        const int r = (int)(((long long)pid * p.Hkv + kvh) << p.page_shift);
        uint8_t *at = dst + lane * p.page * 128;
        tma_load_3d(at, tm, bar, 0, r, 0, pol);
        tma_load_3d(at + HALF_BYTES, tm, bar, 0, r, 1, pol);
    }
}

// 16 bytes of k and of v of the new tokens into their pages: piece e of
// T x Hkv x 16, token t of sequence b going to position past[b] + t.
struct AppendTables {
    const __nv_bfloat16 *k, *v;   // [T, Hkv, D]
    __nv_bfloat16 *kc, *vc;       // [n_pages, Hkv, page, D]
    const int *cu, *pages, *past;
    int nseq, Hkv, max_pages, n_pages, page, page_shift;
    int *status;
};
__device__ __forceinline__ void append_piece(long long e, const AppendTables &p) {
    const int ch = (int)(e % (D / 8));
    const long long th = e / (D / 8);
    const int h = (int)(th % p.Hkv), t = (int)(th / p.Hkv);
    const size_t from = (size_t)th * D + ch * 8;
    const uint4 kx = *reinterpret_cast<const uint4 *>(p.k + from), vx = *reinterpret_cast<const uint4 *>(p.v + from);
    int lo = 0, hi = p.nseq - 1;  // the last sequence that starts at or before t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    const int pos = p.past[lo] + t - p.cu[lo];
    const int pid = p.pages[(size_t)lo * p.max_pages + (pos >> p.page_shift)];
    if (pid < 0 || pid >= p.n_pages) {  // nothing outside the pool is written
        record_status(p.status, ST_INVALID);
        return;
    }
    const size_t to = ((((size_t)pid * p.Hkv + h) << p.page_shift) + (pos & (p.page - 1))) * D + ch * 8;
    *reinterpret_cast<uint4 *>(p.kc + to) = kx;
    *reinterpret_cast<uint4 *>(p.vc + to) = vx;
}

__global__ void __launch_bounds__(SMX_THREADS, 1)
la_softmax_prefill_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                          const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmkc,
                          const __grid_constant__ CUtensorMap tmvc, const __grid_constant__ SoftmaxPrefillParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    SoftmaxCtrl *cb = reinterpret_cast<SoftmaxCtrl *>(smem + SMX_CTRL);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t sbase = smem_u32(smem);
    if (sbase & 1023) {  // the swizzle needs it; dynamic shared memory starts there when there is no static
        if (threadIdx.x == 0) record_status(p.status, ST_CUDA);
        return;
    }

    if (threadIdx.x == 0) {
        for (int s = 0; s < SMX_STAGES; ++s) {
            mbar_init(&cb->kv_full[s], 1);
            mbar_init(&cb->kv_empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&cb->q_full[t], 1);
            mbar_init(&cb->q_empty[t], 1);
            mbar_init(&cb->s_full[t], 1);
            mbar_init(&cb->p_full[t], 4);
            mbar_init(&cb->o_full[t], 1);
            mbar_init(&cb->o_empty[t], 4);
            mbar_init(&cb->stat_full[t], 4);
            mbar_init(&cb->stat_empty[t], 4);
        }
        for (int s = 0; s < SMX_SLOTS; ++s) {
            mbar_init(&cb->item_full[s], 1);
            mbar_init(&cb->item_empty[s], 14);
        }
        mbar_init(&cb->fin, 1);
        cb->abort = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (warp == 1) {
        tmem_alloc(&cb->tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, cb->tmem_base, 0);
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return ctrl_warp_wait(bar, parity, p.wait_limit_ns, p.status, cb);
    };
    // Every warp: what came before has ended.  The waits below have a limit, which must
    // not run while the kernel in front still does.
    pdl_wait();

    if (warp < 4) {
        reg_dec<48>();
        if (warp == 0) {
            // ===================== items, K and V tiles =====================
            const uint64_t pol = policy_evict_last();
            int total = 0, ne = 0;
            int4 own = make_int4(0, 0, 0, 0);
            SplitCursor run;
            pdl_launch();  // the kernel behind may be set up (it waits for this one's end)
            if (p.split) {
                if (lane == 0) p.info[3 * blockIdx.x] = make_int4(0, 0, 0, 0);
                total = smx_split(run, lane, p) ? 0x7fffffff : 0;
            } else if (p.direct) {
                const int e = blockIdx.x / (p.Hkv * p.pairs);
                total = e < smx_find(e, lane, p, own) ? 1 : 0;
            } else {
                total = p.hdr[HDR_TOTAL];
                ne = p.hdr[HDR_G];
            }
            uint32_t it = 0, n = 0;
            bool ok = true;
            for (;;) {
                const int slot = it % SMX_SLOTS;
                if (!wait(&cb->item_empty[slot], ((it / SMX_SLOTS) & 1) ^ 1)) { ok = false; break; }
                int t = 0;
                if (lane == 0 && p.split) {
                    if (total == 0 || !smx_piece(run, p, cb->item[slot])) t = total;
                    cb->item[slot][SI_VALID] = t < total;
                } else if (lane == 0) {
                    int kvh, rest;
                    if (p.direct) {
                        t = (int)it;
                        rest = blockIdx.x % (p.Hkv * p.pairs);
                        kvh = rest / p.pairs;
                    } else {
                        t = atomicAdd(&p.hdr[HDR_TICKET], 1);
                        int e;
                        if (p.by_length) {
                            const int per_entry = p.Hkv * p.pairs;
                            e = t / per_entry;
                            rest = t - e * per_entry;
                            kvh = rest / p.pairs;
                        } else {
                            // key/value head outermost, so that the CTAs at work share its keys in L2
                            const int per_head = max(1, ne * p.pairs);
                            kvh = t / per_head;
                            rest = t - kvh * per_head;
                            e = rest / p.pairs;
                        }
                        if (t < total) own = p.entries[e];
                    }
                    cb->item[slot][SI_VALID] = t < total;
                    if (t < total) smx_item(kvh, own, rest % p.pairs, p, cb->item[slot]);
                }
                t = __shfl_sync(0xffffffffu, t, 0);
                __syncwarp();
                const int n0 = cb->item[slot][SI_N0], n1 = cb->item[slot][SI_N1];
                const int kvh = cb->item[slot][SI_KVH], tok0 = cb->item[slot][SI_TOK0];
                const int past = cb->item[slot][SI_PAST], seq = cb->item[slot][SI_SEQ];
                const int j0 = cb->item[slot][SI_J0];
                __syncwarp();
                if (lane == 0) mbar_arrive(&cb->item_full[slot]);
                ++it;
                if (t >= total) break;
                const int nmax = max(n0, n1), np = (past + BLK - 1) / BLK;
                for (int j = j0; j < j0 + nmax && ok; ++j) {
                    int pid = 0;
                    if (j < np) {
                        const int i = (j << (7 - p.page_shift)) + lane;  // page of this lane in the tile
                        if (lane < (BLK >> p.page_shift) && (i << p.page_shift) < past) {
                            pid = p.pages[(size_t)seq * p.max_pages + i];
                            if (pid < 0 || pid >= p.n_pages) {  // nothing outside the pool is read
                                record_status(p.status, ST_INVALID);
                                pid = 0;
                            }
                        }
                    }
                    for (int kv = 0; kv < 2; ++kv) {
                        const int s = n % SMX_STAGES;
                        uint8_t *dst = smem + SMX_KV + s * TILE_BYTES;
                        if (!wait(&cb->kv_empty[s], ((n / SMX_STAGES) & 1) ^ 1)) { ok = false; break; }
                        if (j < np) {
                            smx_load_pages(dst, kv ? &tmvc : &tmkc, &cb->kv_full[s], kvh, j * BLK, past, pid, lane, pol, p);
                        } else if (lane == 0) {
                            mbar_expect_tx(&cb->kv_full[s], TILE_BYTES);
                            tma_load_4d(dst, kv ? &tmv : &tmk, &cb->kv_full[s], 0, kvh, tok0 + (j - np) * BLK, 0, pol);
                        }
                        ++n;
                    }
                }
                if (!ok) break;
            }
            // every issued copy must land before the CTA exits
            const uint32_t first = n > SMX_STAGES ? n - SMX_STAGES : 0;
            for (uint32_t i = first; i < n; ++i) {
                drain_wait(&cb->kv_full[i % SMX_STAGES], (i / SMX_STAGES) & 1);
            }
            if (!ok) cb->abort = 1;
        } else if (warp == 1) {
            // ===================== MMA issuer =====================
            constexpr uint32_t ID_QK = idesc_bf16_f32(BLK, BLK, 0, 0);  // Q (K-major) x K (K-major)
            constexpr uint32_t ID_PV = idesc_bf16_f32(BLK, D, 0, 1);    // P (TMEM) x V (MN-major)
            uint32_t it = 0;
            int cur[SI_FIELDS], nxt[SI_FIELDS];
            uint32_t base = 0;                 // ring position of the current item's first K tile
            // bit t: phase of the tile's Q, P and O barriers
            uint32_t qph = 0, pph = 0, oph = 0;
            uint32_t pend = 3;                 // bit t: first scores of the tile's next item not issued yet
            constexpr uint32_t MASK = 1u << SI_N0 | 1u << SI_N1 | 1u << SI_PAST | 1u << SI_LEN | 1u << SI_J0;
            bool ok = smx_next<MASK>(it, cur, lane, p, cb);
            // S_t of step j of an item whose first K tile is at ring position rb
            auto scores = [&](int t, const int (&im)[SI_FIELDS], uint32_t rb, int j) -> bool {
                const uint32_t pos = rb + 2 * j, s = pos % SMX_STAGES;
                const int nt = t ? im[SI_N1] : im[SI_N0], n1 = im[SI_N1];
                if (j == 0) {
                    if (!wait(&cb->q_full[t], (qph >> t) & 1)) return false;
                    qph ^= 1u << t;
                }
                if (!wait(&cb->kv_full[s], (pos / SMX_STAGES) & 1)) return false;
                tc_fence_after();
                const uint32_t qt = sbase + SMX_Q + t * TILE_BYTES, kt = sbase + SMX_KV + s * TILE_BYTES;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss_w(tmem + SMX_TM_S + t * 128, desc_kmajor(qt, kk), desc_kmajor(kt, kk), ID_QK, kk > 0 ? 1u : 0u);
                tc_commit_w(&cb->s_full[t]);
                if (t == 1 || j >= n1) tc_commit_w(&cb->kv_empty[s]);  // last reader of the K tile
                if (j == nt - 1) tc_commit_w(&cb->q_empty[t]);
                return true;
            };
            while (ok) {
                const int n0 = cur[SI_N0], n1 = cur[SI_N1], nmax = max(n0, n1);
                // tile j of the piece is tile j + J0 of the item: cached keys up to np
                const int np = (cur[SI_PAST] + BLK - 1) / BLK - cur[SI_J0];
                const int past = cur[SI_PAST] - cur[SI_J0] * BLK;
                bool have_nxt = false, nxt_valid = false;
                for (int t = 0; t < 2 && ok; ++t) {
                    if (((pend >> t) & 1) && (t ? n1 : n0) > 0) {
                        ok = scores(t, cur, base, 0);
                        pend &= ~(1u << t);
                    }
                }
                for (int j = 0; j < nmax && ok; ++j) {
                    for (int t = 0; t < 2 && ok; ++t) {
                        const int nt = t ? n1 : n0;
                        if (j >= nt) continue;
                        const uint32_t pos = base + 2 * j + 1, s = pos % SMX_STAGES;
                        uint8_t *vp = smem + SMX_KV + s * TILE_BYTES;
                        if (!wait(&cb->kv_full[s], (pos / SMX_STAGES) & 1)) { ok = false; break; }
                        const int valid = j < np ? past - j * BLK : cur[SI_LEN] - (j - np) * BLK;
                        if (valid < BLK && (t == 0 || j >= n0)) {
                            // rows behind the last key meet P = 0, which keeps out what they
                            // hold only if it is finite: zero them
                            const int nbytes = (BLK - valid) * 128;
                            for (int hh = 0; hh < 2; ++hh)
                                for (int o = lane * 16; o < nbytes; o += 32 * 16)
                                    *reinterpret_cast<uint4 *>(vp + hh * HALF_BYTES + valid * 128 + o) = make_uint4(0, 0, 0, 0);
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        if (j == 0) {
                            if (!wait(&cb->o_empty[t], ((oph >> t) & 1) ^ 1)) { ok = false; break; }
                            oph ^= 1u << t;
                        }
                        if (!wait(&cb->p_full[t], (pph >> t) & 1)) { ok = false; break; }
                        pph ^= 1u << t;
                        tc_fence_after();
                        const uint32_t vt = smem_u32(vp);
#pragma unroll
                        for (int kk = 0; kk < BLK / 16; ++kk)
                            mma_ts_w(tmem + SMX_TM_O + t * 128, tmem + SMX_TM_S + t * 128 + kk * 8, desc_mnmajor(vt, kk),
                                     ID_PV, (j > 0 || kk > 0) ? 1u : 0u);
                        if (t == 1 || j >= n1) tc_commit_w(&cb->kv_empty[s]);  // last reader of the V tile
                        if (j + 1 < nt) {
                            ok = scores(t, cur, base, j + 1);
                        } else {
                            tc_commit_w(&cb->o_full[t]);
                            if (!have_nxt) {
                                have_nxt = true;
                                nxt_valid = smx_next<MASK>(it, nxt, lane, p, cb);
                                if (cb->abort) ok = false;
                            }
                            pend |= 1u << t;
                            // (tile 0's scores come first: tile 1's release the K tile)
                            const bool behind = t == 1 && (pend & 1) && nxt[SI_N0] > 0;
                            if (ok && nxt_valid && !behind && (t ? nxt[SI_N1] : nxt[SI_N0]) > 0) {
                                ok = scores(t, nxt, base + 2 * nmax, 0);
                                pend &= ~(1u << t);
                            }
                        }
                    }
                }
                if (!ok) break;
                if (!have_nxt) nxt_valid = smx_next<MASK>(it, nxt, lane, p, cb);
                base += 2 * nmax;
                if (!nxt_valid) break;
#pragma unroll
                for (int f = 0; f < SI_FIELDS; ++f)
                    if ((MASK >> f) & 1) cur[f] = nxt[f];
            }
            tc_commit_w(&cb->fin);
            drain_wait(&cb->fin, 0);
        } else if (warp == 2) {
            // ===================== Q tiles =====================
            const uint64_t pol = policy_evict_first();
            constexpr uint32_t MASK = ~(1u << SI_PAST | 1u << SI_KVH | 1u << SI_SEQ | 1u << SI_LEN);
            uint32_t it = 0, n[2] = {0, 0};
            int im[SI_FIELDS];
            bool ok = true;
            while (ok && smx_next<MASK>(it, im, lane, p, cb)) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if ((t ? im[SI_N1] : im[SI_N0]) == 0) continue;
                    if (!wait(&cb->q_empty[t], (n[t] & 1) ^ 1)) { ok = false; break; }
                    if (lane == 0) {
                        mbar_expect_tx(&cb->q_full[t], TILE_BYTES);
                        tma_load_4d(smem + SMX_Q + t * TILE_BYTES, &tmq, &cb->q_full[t], 0, t ? im[SI_H1] : im[SI_H0],
                                    im[SI_TOK0] + (t ? im[SI_B1] : im[SI_B0]) * BLK, 0, pol);
                    }
                    ++n[t];
                }
            }
            for (int t = 0; t < 2; ++t)
                if (n[t] > 0) {
                    drain_wait(&cb->q_full[t], (n[t] - 1) & 1);
                }
        } else if (p.new_k) {
            // ===================== new tokens into their pages =====================
            // (no CTA reads them there: their tiles come from the packed tensors)
            int4 unused;
            if (smx_find(-1, lane, p, unused) > 0) {
                const AppendTables at = {p.new_k, p.new_v, p.kc, p.vc, p.cu, p.pages, p.past, p.nseq,
                                         p.Hkv, p.max_pages, p.n_pages, p.page, p.page_shift, p.status};
                const long long total = (long long)p.T * p.Hkv * (D / 8);
#pragma unroll 2
                for (long long e = (long long)blockIdx.x * 32 + lane; e < total; e += (long long)gridDim.x * 32)
                    append_piece(e, at);
            }
        }
    } else if (warp < 12) {
        // ===================== softmax of tile t =====================
        reg_inc<192>();
        const int t = (warp - 4) >> 2;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(warp & 3) << 21);  // lanes of this warp's quarter
        const uint32_t ts = trow + SMX_TM_S + t * 128, to = trow + SMX_TM_O + t * 128;
        float2 *stat = reinterpret_cast<float2 *>(smem + SMX_STAT) + t * BLK;
        const float c = p.scale_log2;
        uint32_t it = 0, sn = 0, in = 0;
        int im[SI_FIELDS];
        bool ok = true;
        constexpr uint32_t MASK = 1u << SI_N0 | 1u << SI_N1 | 1u << SI_B0 | 1u << SI_B1 | 1u << SI_PAST | 1u << SI_J0;
        while (ok && smx_next<MASK>(it, im, lane, p, cb)) {
            const int nt = t ? im[SI_N1] : im[SI_N0];
            if (nt == 0) continue;
            // tile j of the piece is tile j + J0 of the item: cached keys up to np, then new
            // ones up to the diagonal
            const int past = im[SI_PAST] - im[SI_J0] * BLK, np = (im[SI_PAST] + BLK - 1) / BLK - im[SI_J0];
            const int diag = np + (t ? im[SI_B1] : im[SI_B0]);
            float m = -INFINITY, l = 0.f;           // m: maximum in use
            for (int j = 0; j < nt; ++j) {
                if (!wait(&cb->s_full[t], sn & 1)) { ok = false; break; }
                tc_fence_after();
                uint32_t x[128];
                tmem_ld_cols<128>(ts, x);
                // the last tile of cached keys may be ragged, that of the own rows is the diagonal
                if (j == diag || (j < np && past - j * BLK < BLK)) {
                    const int lim = j < np ? past - j * BLK - 1 : r;  // columns [0, lim] are seen
#pragma unroll
                    for (int q = 0; q < 4; ++q) {  // (tests of a mask's bits; 48 prompts of 512: 1 % less than compares)
                        const int seen = min(max(lim + 1 - 32 * q, 0), 32);
                        const uint32_t hidden = seen == 32 ? 0u : 0xffffffffu << seen;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (hidden & (1u << i)) x[32 * q + i] = 0xff800000u;  // -inf
                    }
                }
                float mt[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 128; i += 2)  // (three-input maxima)
                    mt[(i >> 1) & 3] = fmaxf(mt[(i >> 1) & 3], fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 1])));
                const float tile_max = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3]));
                if (j == 0) {
                    m = tile_max;
                } else {
                    const bool grow = (tile_max - m) * c > RESCALE_LOG2;
                    if (__any_sync(0xffffffffu, grow)) {
                        const float alpha = grow ? ex2((m - tile_max) * c) : 1.f;
                        if (grow) m = tile_max;
                        l *= alpha;
                        // O is complete up to the previous step: these scores were
                        // issued, and so committed, behind its P V
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            uint32_t o[32];
                            tmem_ld_wait32(to + q * 32, o);
                            scale32(o, alpha);
                            tmem_st32(to + q * 32, o);
                        }
                    }
                }
                const float mc = m == -INFINITY ? 0.f : -m * c;  // (only scores of -inf so far: no weight)
                const f32x2 c2 = pack2(c, c), mc2 = pack2(mc, mc);
                f32x2 s2[2] = {0ull, 0ull};
#pragma unroll
                for (int q = 0; q < 4; ++q) {  // 32 columns at a time: 16 TMEM columns of bf16 pairs
                    uint32_t b[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int k = q * 32 + 2 * i;
                        float e0, e1;
                        unpack2(fma2(pack2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), c2, mc2), e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        s2[i & 1] = add2(s2[i & 1], pack2(e0, e1));
                        b[i] = pack_bf16x2(e0, e1);  // one rounding to bf16, for the tensor cores
                    }
                    tmem_st16(ts + q * 16, b);
                }
                float sa, sb;
                unpack2(add2(s2[0], s2[1]), sa, sb);
                l += sa + sb;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&cb->p_full[t]);
                ++sn;
            }
            if (!ok) break;
            if (!wait(&cb->stat_empty[t], (in & 1) ^ 1)) break;
            stat[r] = make_float2(m * c, l);
            __syncwarp();
            if (lane == 0) mbar_arrive(&cb->stat_full[t]);
            ++in;
        }
    } else {
        // ===================== output =====================
        reg_dec<80>();
        const int r = (warp & 3) * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(warp & 3) << 21);
        uint32_t it = 0, n[2] = {0, 0};
        int im[SI_FIELDS];
        bool ok = true;
        const bool wide = aligned32(p.out);
        constexpr uint32_t MASK = ~(1u << SI_PAST | 1u << SI_KVH | 1u << SI_SEQ);
        while (ok && smx_next<MASK>(it, im, lane, p, cb)) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                // a part of a cut item goes to the workspace, as it is
                float *part = im[SI_PART] < 0 ? nullptr
                    : p.parts + (((size_t)blockIdx.x * 2 + im[SI_PART]) * 2 + t) * BLK * SMX_PART + (size_t)r * SMX_PART;
                if ((t ? im[SI_N1] : im[SI_N0]) == 0) {
                    if (part) *reinterpret_cast<float2 *>(part + D) = make_float2(-INFINITY, 0.f);  // none of the tile's keys
                    continue;
                }
                const float2 *stat = reinterpret_cast<const float2 *>(smem + SMX_STAT) + t * BLK;
                if (!wait(&cb->stat_full[t], n[t] & 1)) { ok = false; break; }
                const float2 ml = stat[r];
                __syncwarp();
                if (lane == 0) mbar_arrive(&cb->stat_empty[t]);
                if (!wait(&cb->o_full[t], n[t] & 1)) { ok = false; break; }
                ++n[t];
                tc_fence_after();
                const int row = (t ? im[SI_B1] : im[SI_B0]) * BLK + r, h = t ? im[SI_H1] : im[SI_H0];
                const bool mine = row < im[SI_LEN];  // rows behind the sequence are left as they are
                const size_t at = ((size_t)im[SI_TOK0] + row) * p.H + h;
                const float inv = 1.f / ml.y;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    uint32_t o[32];
                    __syncwarp();
                    tmem_ld_wait32(trow + SMX_TM_O + t * 128 + q * 32, o);
                    if (mine && part) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            reinterpret_cast<uint4 *>(part + q * 32)[i] =
                                make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    } else if (mine) {
                        store_row32(p.out + at * D + q * 32, o, inv, wide);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&cb->o_empty[t]);
                if (part) *reinterpret_cast<float2 *>(part + D) = ml;
                else if (mine && p.lse) p.lse[at] = (ml.x + log2f(ml.y)) * 0.69314718055994531f;  // ln 2
            }
        }
    }

    // ===================== tear-down =====================
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Split: joins the parts of the items that the runs' borders cut.  Block (c, tile,
// z) has rows 8 z to 8 z + 7, a warp each, of the item that starts in CTA c's run
// and goes on, if one does; a lane has four features, and the m and l of every
// 32nd part.  (A block per row: 35 us for its 38000 blocks, most with nothing to do.)
constexpr int SPLIT_JOIN_ROWS = 8;

__global__ void __launch_bounds__(32 * SPLIT_JOIN_ROWS)
la_softmax_split_join_kernel(const __grid_constant__ SoftmaxPrefillParams p) {
    pdl_wait();
    pdl_launch();
    const int c = blockIdx.x, t = blockIdx.y, lane = threadIdx.x & 31;
    const int r = blockIdx.z * SPLIT_JOIN_ROWS + (threadIdx.x >> 5);
    const int4 a = p.info[3 * c], hb = p.info[3 * c + 1], n = p.info[3 * c + 2];
    if (a.x == 0) return;
    const int h = t ? hb.y : hb.x, row = (t ? hb.w : hb.z) * BLK + r;
    if ((t ? n.y : n.x) == 0 || row >= a.z) return;
    // first part: slot 1 of CTA c; the others: slot 0 of the CTAs behind it
    auto part = [&](int i) -> const float * {
        return p.parts + (((size_t)(c + i) * 2 + (i == 0)) * 2 + t) * BLK * SMX_PART + (size_t)r * SMX_PART;
    };
    float m = -INFINITY, l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = 0; base < a.x; base += 32) {
        const int i = base + lane, count = min(32, a.x - base);
        const float2 ml = i < a.x ? *reinterpret_cast<const float2 *>(part(i) + D) : make_float2(-INFINITY, 0.f);
        float mm = fmaxf(m, ml.x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
        const float u = mm == -INFINITY ? 0.f : mm;
        const float old = m == -INFINITY ? 0.f : ex2(m - u), w = ml.x == -INFINITY ? 0.f : ex2(ml.x - u);
        float s = ml.y * w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        l = fmaf(l, old, s);
        m = mm;
        x.x *= old;
        x.y *= old;
        x.z *= old;
        x.w *= old;
#pragma unroll 8
        for (int k = 0; k < count; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            if (wk != 0.f) {  // (a part without keys of this tile holds nothing)
                const float4 o = reinterpret_cast<const float4 *>(part(base + k))[lane];
                x.x = fmaf(o.x, wk, x.x);
                x.y = fmaf(o.y, wk, x.y);
                x.z = fmaf(o.z, wk, x.z);
                x.w = fmaf(o.w, wk, x.w);
            }
        }
    }
    const size_t at = ((size_t)a.y + row) * p.H + h;
    const float inv = 1.f / l;
    reinterpret_cast<uint2 *>(p.out + at * D)[lane] =
        make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
    if (lane == 0 && p.lse) p.lse[at] = (m + log2f(l)) * 0.69314718055994531f;  // ln 2
}

// Entries of at most SCHED_THREADS sequences of at most SCHED_THREADS blocks each,
// by block number (which is what a query block has keys before it, in blocks)
// from the largest down: with m(w) sequences of more than w blocks, block w's
// entries are the m(w) longest sequences'.
__device__ __forceinline__ void schedule_by_length(const SoftmaxScheduleParams &s, int tid) {
    __shared__ int nb[SCHED_THREADS], order[SCHED_THREADS], first[SCHED_THREADS + 1], warp_sums2[SCHED_THREADS / 32];
    int n = 0;
    if (tid < s.nseq) {
        n = (s.cu[tid + 1] - s.cu[tid] + s.rows - 1) / s.rows;
        nb[tid] = n;
    }
    __syncthreads();
    if (tid < s.nseq) {
        int rank = 0;
        for (int j = 0; j < s.nseq; ++j) rank += nb[j] > n || (nb[j] == n && j < tid);
        order[rank] = tid;
    }
    __syncthreads();
    // thread x stands for block w = SCHED_THREADS - 1 - x: m(w), then a scan over x
    const int w = SCHED_THREADS - 1 - tid;
    int lo = 0, hi = s.nseq;  // the first of the ordered sequences with no more than w blocks
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (nb[order[mid]] > w) lo = mid + 1;
        else hi = mid;
    }
    int x = lo;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if ((tid & 31) >= o) x += y;
    }
    if ((tid & 31) == 31) warp_sums2[tid >> 5] = x;
    __syncthreads();
    for (int v = 0; v < (tid >> 5); ++v) x += warp_sums2[v];
    first[tid] = x - lo;
    if (tid == SCHED_THREADS - 1) first[SCHED_THREADS] = x;
    __syncthreads();
    const int ne = first[SCHED_THREADS];
    for (int e = tid; e < ne; e += SCHED_THREADS) {
        int a = 0, b = SCHED_THREADS - 1;  // the last x whose first entry is at or before e
        while (a < b) {
            const int mid = (a + b + 1) >> 1;
            if (first[mid] <= e) a = mid;
            else b = mid - 1;
        }
        const int seq = order[e - first[a]], at = s.cu[seq];
        s.entries[e] = make_int4(seq, at, s.cu[seq + 1] - at, SCHED_THREADS - 1 - a);
    }
    if (tid == 0) {
        s.hdr[HDR_G] = ne;
        s.hdr[HDR_TOTAL] = ne * s.items_per_entry;
    }
}

// Scheduler of the softmax kernels: checks cu_seqlens and the cached lengths,
// writes the entries and resets the tickets.  One block.
__device__ __forceinline__ void softmax_schedule(const SoftmaxScheduleParams &s) {
    __shared__ int warp_sums[SCHED_THREADS / 32];
    __shared__ int carry_sh;
    const int tid = threadIdx.x;
    int bad = 0;
    if (tid == 0 && (s.cu[0] != 0 || s.cu[s.nseq] != s.T)) bad = 1;
    for (int i = tid; i < s.nseq; i += SCHED_THREADS)
        if (!smx_sequence_ok(i, s.cu[i], s.cu[i + 1], s.past, s.T, s.max_seqlen, s.max_keys)) bad = 1;
    bad = __syncthreads_or(bad);
    if (tid == 0) {
        s.hdr[HDR_TICKET] = 0;
        s.hdr[HDR_TICKET2] = 0;
        s.hdr[HDR_READY] = 0;
        carry_sh = 0;
        if (bad) {
            s.hdr[HDR_TOTAL] = 0;
            s.hdr[HDR_G] = 0;
            atomicCAS(s.status, 0, ST_INVALID);
        }
    }
    if (bad) return;
    if (s.by_length) {
        schedule_by_length(s, tid);
        return;
    }
    __syncthreads();
    for (int base = 0; base < s.nseq; base += SCHED_THREADS) {  // exclusive scan of entry counts
        const int i = base + tid;
        const int n = i < s.nseq ? (s.cu[i + 1] - s.cu[i] + s.rows - 1) / s.rows : 0;
        int x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if ((tid & 31) >= o) x += y;
        }
        if ((tid & 31) == 31) warp_sums[tid >> 5] = x;
        __syncthreads();
        if (tid < 32) {
            int w = warp_sums[tid];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, w, o);
                if (tid >= o) w += y;
            }
            warp_sums[tid] = w;
        }
        __syncthreads();
        if (i < s.nseq) s.prefix[i] = carry_sh + x - n + ((tid >> 5) ? warp_sums[(tid >> 5) - 1] : 0);
        __syncthreads();
        if (tid == 0) carry_sh += warp_sums[SCHED_THREADS / 32 - 1];
        __syncthreads();
    }
    const int ne = carry_sh;
    for (int e = tid; e < ne; e += SCHED_THREADS) {
        int lo = 0, hi = s.nseq - 1;  // the last sequence whose first entry is at or before e
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s.prefix[mid] <= e) lo = mid;
            else hi = mid - 1;
        }
        const int a = s.cu[lo], len = s.cu[lo + 1] - a;
        const int nb = (len + s.rows - 1) / s.rows;
        s.entries[e] = make_int4(lo, a, len, nb - 1 - (e - s.prefix[lo]));
    }
    if (tid == 0) {
        s.hdr[HDR_G] = ne;
        s.hdr[HDR_TOTAL] = ne * s.items_per_entry;
    }
}

__global__ void __launch_bounds__(SCHED_THREADS, 1) la_softmax_schedule_kernel(const SoftmaxScheduleParams s) {
    pdl_wait();    // before the kernel behind may start: it reads what came before this one
    pdl_launch();
    softmax_schedule(s);
}

}  // namespace la
