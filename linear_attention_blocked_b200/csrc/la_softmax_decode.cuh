// la_softmax_decode.cuh -- softmax attention of one new token per sequence on
// a paged key/value cache, and the kernels that keep the cache.
//
// For request b with len cached tokens, every key/value head and the G query
// heads of its group:  write the new token's k, v at position len, then
//
//     o = sum_{s <= len} p_s v_s,   p_s = exp(scale q . k_s - lse).
//
// The cache is read once and nothing else is large, so HBM bounds the step:
// 512 bytes a key and key/value head.  The keys of all (request, head) rows
// are laid end to end in tiles of 64, and every CTA takes an equal run of tiles
// whatever the rows' lengths; a row that a run's border cuts is joined from
// its parts by a second, small kernel.  The lengths stay on the device.
//
// A CTA streams its tiles through a ring of TMA loads (two CTAs of 3 x 32 KiB
// per SM keep some 190 KB in flight, four times latency x bandwidth).  Four
// warps take 16 keys of a tile each, with sums and maxima of their own
// that are joined when the row ends.  The group's heads are the rows of one
// m16n8k16 product (up to 16; larger groups are cut into chunks of 16): with
// 16 rows instead of 128, tcgen05 tiles would be 7/8 empty and need the same
// bytes, while mma.sync from registers takes a fifth of the time the tile's
// bytes take.  The weights meet V as a bf16 pair hi + lo (2^-17 of each), so
// the output is as exact as its own type.
#pragma once
#include "la_softmax.cuh"

namespace la {

constexpr int SD_THREADS = 160;      // warps 0-3: 16 keys each; warp 4: loads
constexpr int SD_KEYS = 64;          // keys per tile
constexpr int SD_STAGES = 3;
constexpr int SD_HALF = SD_KEYS * 128;         // 64 features of the tile's keys
constexpr int SD_TILE = 2 * SD_HALF;           // one of K, V
constexpr int SD_CTAS = 2 * 148;               // equal runs of tiles
constexpr int SD_HEADS = 16;                   // query heads per row of tiles
constexpr int SD_RED = SD_STAGES * 2 * SD_TILE;             // two [16][128] fp32 buffers
constexpr int SD_SMEM = SD_RED + 2 * SD_HEADS * D * 4;      // 114688: two CTAs per SM
constexpr int SD_PART = SD_HEADS * D + 2 * SD_HEADS;        // floats of one part: O, m, l

struct SoftmaxDecodeParams {
    const __nv_bfloat16 *q, *k, *v;   // [B, H, D], [B, Hkv, D]
    __nv_bfloat16 *kc, *vc;           // [n_pages, Hkv, page, D]
    const int *pages;                 // [B, max_pages]
    const int *lens;                  // [B] cached tokens before the step; -1: no request
    void *out;                        // [B, H, D]
    float *lse;                       // [B, H] or null
    float *parts;                     // [SD_CTAS][2][SD_PART]
    int4 *info;                       // [SD_CTAS] {request, row, parts, 0}: the row cut at the CTA's end
    int out_fp32;
    int B, H, Hkv, G, chunks;         // chunks of 16 heads in a group
    int max_pages, n_pages, page, page_shift;
    long long max_keys;               // max_pages * page
    float scale_log2;
    unsigned long long wait_limit_ns;
    int *status;
};

struct SoftmaxDecodeCtrl {
    uint64_t full[SD_STAGES], empty[SD_STAGES];
    volatile int abort;
};

__device__ __forceinline__ int sd_tiles(int len, long long max_keys) {  // tiles of a request's row
    return (len < 0 || (long long)len + 1 > max_keys) ? 0 : len / SD_KEYS + 1;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Where a run of tiles starts: request, row of the request (head and chunk), tile
struct DecodeCursor {
    int b, row, tile, nt, len;
};

__device__ __forceinline__ void sd_next_request(DecodeCursor &c, const SoftmaxDecodeParams &p) {
    do {
        ++c.b;
        c.len = c.b < p.B ? p.lens[c.b] : 0;
        c.nt = c.b < p.B ? sd_tiles(c.len, p.max_keys) : 1;
    } while (c.nt == 0);
    c.row = 0;
    c.tile = 0;
}

// Shared memory of a decode CTA next to its ring and sum buffers
struct SoftmaxDecodeShared {
    SoftmaxDecodeCtrl cb;
    int stop;
    float m[4][SD_HEADS], l[4][SD_HEADS];  // of each warp, per head
};

// The loads of one tile of a row (request b with len cached tokens, row = head
// and chunk): the whole warp, lane (kv, half, page of the tile) issuing one box
// of 64 features of up to 64 keys.
struct DecodeLoader {
    int bx_shift, nbx, g, bx;
    const CUtensorMap *tm;
    uint64_t pol;
    __device__ DecodeLoader(const CUtensorMap *tmk, const CUtensorMap *tmv, const SoftmaxDecodeParams &p, int lane) {
        pol = policy_evict_first();
        bx_shift = p.page_shift < 6 ? p.page_shift : 6;  // keys per box
        nbx = SD_KEYS >> bx_shift;                        // boxes of a tile's half: 1, 2 or 4
        g = lane / nbx;                                   // 0, 1: K halves; 2, 3: V halves
        bx = lane - g * nbx;
        tm = g & 2 ? tmv : tmk;
    }
    __device__ bool load(int b, int len, int row, int tile, uint32_t it, uint8_t *smem, SoftmaxDecodeCtrl *cb,
                         const SoftmaxDecodeParams &p, int lane) const {
        const int key = tile * SD_KEYS + (bx << bx_shift);  // first key of this lane's box
        const bool has = g < 4 && key <= len;
        int pid = 0;
        if (has) {
            pid = p.pages[(size_t)b * p.max_pages + (key >> p.page_shift)];
            if (pid < 0 || pid >= p.n_pages) {  // nothing outside the pool is read
                record_status(p.status, ST_INVALID);
                pid = 0;
            }
        }
        const int s = it % SD_STAGES;
        if (!ctrl_warp_wait(&cb->empty[s], ((it / SD_STAGES) & 1) ^ 1, p.wait_limit_ns, p.status, cb)) return false;
        const int nb = __popc(__ballot_sync(0xffffffffu, has));
        if (lane == 0) mbar_expect_tx(&cb->full[s], (uint32_t)(nb << bx_shift) * 128u);
        __syncwarp();
        if (has) {
            const int r = (int)((((long long)pid * p.Hkv + row / p.chunks) << p.page_shift) + (key & (p.page - 1)));
            tma_load_3d(smem + s * 2 * SD_TILE + g * SD_HALF + (bx << bx_shift) * 128, tm, &cb->full[s], 0, r, g & 1, pol);
        }
        return true;
    }
};

__device__ __forceinline__ void sd_drain(uint32_t it, SoftmaxDecodeCtrl *cb, const SoftmaxDecodeParams &p) {
    for (uint32_t i = it > SD_STAGES ? it - SD_STAGES : 0; i < it; ++i) {  // copies land before the CTA exits
        int dummy = 0;
        la_wait(&cb->full[i % SD_STAGES], (i / SD_STAGES) & 1, globaltimer_ns() + p.wait_limit_ns, &dummy);
    }
}

// Maximum and sum of a head over the four warps
__device__ __forceinline__ void sd_joined(const SoftmaxDecodeShared *sh, int head, float &m, float &l) {
    m = fmaxf(fmaxf(sh->m[0][head], sh->m[1][head]), fmaxf(sh->m[2][head], sh->m[3][head]));
    const float u = m == -INFINITY ? 0.f : m;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) l += sh->l[w][head] * ex2(sh->m[w][head] - u);
}

// Column of feature d of a head in the sum buffers: spreads the heads over the banks
__device__ __forceinline__ int sd_col(int head, int d) { return d ^ ((head & 7) << 3); }

// The four attention warps over tiles [tile0, tile1) of a row.  Leaves, behind
// a barrier, each warp's m and l in `sh` and the joined sums of O (relative to
// the joined m) in two buffers of smem + SD_RED to be added, and in sh->stop
// whether a wait ran out.  The caller has the warps meet again before the next
// call.
__device__ __forceinline__ void sd_piece(const SoftmaxDecodeParams &p, uint8_t *smem, SoftmaxDecodeShared *sh, int b,
                                         int len, int crow, int tile0, int tile1, uint32_t &it, int warp, int lane) {
    const uint32_t sbase = smem_u32(smem);
    SoftmaxDecodeCtrl *cb = &sh->cb;
    const int g = lane >> 2, t4 = lane & 3;
    float *red = reinterpret_cast<float *>(smem + SD_RED);
    const int kvh = crow / p.chunks, chunk = crow - kvh * p.chunks, h0 = kvh * p.G + chunk * SD_HEADS;
    const int nh = min(SD_HEADS, p.G - chunk * SD_HEADS);  // heads of this row
    // Q as the A operand: rows g, g + 8, columns 16 kk + 2 t4 (+ 8)
    uint32_t qa[8][4];
    const __nv_bfloat16 *qr = p.q + ((size_t)b * p.H + h0) * D;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = g + (i & 1) * 8, col = kk * 16 + t4 * 2 + (i >> 1) * 8;
            qa[kk][i] = row < nh ? *reinterpret_cast<const uint32_t *>(qr + (size_t)row * D + col) : 0u;
        }
    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows g, g + 8 (l: this thread's keys)
    for (int tile = tile0; tile < tile1; ++tile) {
        const int s = it % SD_STAGES;
        if (!ctrl_warp_wait(&cb->full[s], (it / SD_STAGES) & 1, p.wait_limit_ns, p.status, cb)) break;
        uint8_t *kt = smem + s * 2 * SD_TILE, *vt = kt + SD_TILE;
        const int key0 = tile * SD_KEYS + warp * 16;  // this warp's 16 keys
        const bool tail = key0 + 16 > len;
        if (tail) {
            // the warp's keys hold or lie behind the new token: its row goes into the
            // tile and the cache, rows behind it are zeroed (P = 0 keeps out what
            // they hold only if it is finite)
            if (len >= key0) {
                const int rr = warp * 16 + len - key0, ch = lane & 15;
                const size_t src = ((size_t)b * p.Hkv + kvh) * D;
                const uint4 val = *reinterpret_cast<const uint4 *>((lane < 16 ? p.k : p.v) + src + ch * 8);
                *reinterpret_cast<uint4 *>((lane < 16 ? kt : vt) + (ch >> 3) * SD_HALF + rr * 128 +
                                           (((ch & 7) ^ (rr & 7)) << 4)) = val;
                if (chunk == 0) {
                    const int pid = p.pages[(size_t)b * p.max_pages + (len >> p.page_shift)];
                    if (pid >= 0 && pid < p.n_pages)
                        *reinterpret_cast<uint4 *>((lane < 16 ? p.kc : p.vc) +
                                                   ((((size_t)pid * p.Hkv + kvh) << p.page_shift) + (len & (p.page - 1))) * D +
                                                   ch * 8) = val;
                }
            }
            for (int e = lane; e < 16 * 16; e += 32) {
                const int rr = e >> 4, ch = e & 15;
                if (key0 + rr > len)
                    *reinterpret_cast<uint4 *>(vt + (ch >> 3) * SD_HALF + (warp * 16 + rr) * 128 + ((ch & 7) << 4)) =
                        make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
        }
        // S = Q K^T for 16 keys
        float sc[2][4] = {};
        const uint32_t ka = sbase + (uint32_t)(kt - smem), va = sbase + (uint32_t)(vt - smem);
        {
            const int rr = warp * 16 + (lane & 7) + ((lane >> 4) << 3);  // key of this lane's address
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                const int ch = 2 * kk + ((lane >> 3) & 1);
                uint32_t bf[4];
                ldsm4(bf, ka + (ch >> 3) * SD_HALF + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4));
                mma16816(sc[0], qa[kk], bf[0], bf[1]);
                mma16816(sc[1], qa[kk], bf[2], bf[3]);
            }
        }
        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int key = key0 + i * 8 + t4 * 2 + (k & 1);
                sc[i][k] = key <= len ? sc[i][k] * p.scale_log2 : -INFINITY;
                if (k < 2) x0 = fmaxf(x0, sc[i][k]);
                else x1 = fmaxf(x1, sc[i][k]);
            }
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
        if (__any_sync(0xffffffffu, x0 > m0 || x1 > m1)) {
            const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
            const float a0 = n0 == -INFINITY ? 1.f : ex2(m0 - n0), a1 = n1 == -INFINITY ? 1.f : ex2(m1 - n1);
            m0 = n0;
            m1 = n1;
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                o[i][0] *= a0;
                o[i][1] *= a0;
                o[i][2] *= a1;
                o[i][3] *= a1;
            }
        }
        const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float e0 = ex2(sc[i][0] - u0), e1 = ex2(sc[i][1] - u0);
            const float e2 = ex2(sc[i][2] - u1), e3 = ex2(sc[i][3] - u1);
            l0 += e0 + e1;
            l1 += e2 + e3;
            hi[2 * i] = pack_bf16x2(e0, e1);
            hi[2 * i + 1] = pack_bf16x2(e2, e3);
            lo[2 * i] = pack_bf16x2(e0 - __uint_as_float(hi[2 * i] << 16), e1 - __uint_as_float(hi[2 * i] & 0xffff0000u));
            lo[2 * i + 1] = pack_bf16x2(e2 - __uint_as_float(hi[2 * i + 1] << 16),
                                        e3 - __uint_as_float(hi[2 * i + 1] & 0xffff0000u));
        }
        // O += P V
        {
            const int rr = warp * 16 + (lane & 15);
#pragma unroll
            for (int dd = 0; dd < 8; ++dd) {
                const int ch = 2 * dd + (lane >> 4);
                uint32_t bf[4];
                ldsm4_t(bf, va + (ch >> 3) * SD_HALF + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4));
                mma16816(o[2 * dd], hi, bf[0], bf[1]);
                mma16816(o[2 * dd + 1], hi, bf[2], bf[3]);
                mma16816(o[2 * dd], lo, bf[0], bf[1]);
                mma16816(o[2 * dd + 1], lo, bf[2], bf[3]);
            }
        }
        if (tail) fence_proxy_async_smem();  // this thread's writes before the next TMA load
        __syncwarp();
        if (lane == 0) mbar_arrive(&cb->empty[s]);
        ++it;
    }
    // ---- join the four warps ----
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    if (t4 == 0) {
        sh->m[warp][g] = m0;
        sh->m[warp][g + 8] = m1;
        sh->l[warp][g] = l0;
        sh->l[warp][g + 8] = l1;
    }
    named_bar_sync(1, 128);
    if (warp == 0 && lane == 0) sh->stop = cb->abort;  // one decision for the four warps
    float M0, M1, L;
    sd_joined(sh, g, M0, L);
    sd_joined(sh, g + 8, M1, L);
    const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - M0), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M1);
    float *buf = red + (warp & 1) * SD_HEADS * D;
    for (int turn = 0; turn < 2; ++turn) {  // warps 0, 1 store; warps 2, 3 add
        if ((warp >> 1) == turn) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int col = sd_col(g, i * 8 + t4 * 2);
                float2 *d0 = reinterpret_cast<float2 *>(buf + g * D + col);
                float2 *d1 = reinterpret_cast<float2 *>(buf + (g + 8) * D + col);
                float2 x = make_float2(o[i][0] * f0, o[i][1] * f0), y = make_float2(o[i][2] * f1, o[i][3] * f1);
                if (turn) {
                    x.x += d0->x;
                    x.y += d0->y;
                    y.x += d1->x;
                    y.y += d1->y;
                }
                *d0 = x;
                *d1 = y;
            }
        }
        named_bar_sync(1, 128);
    }
}

__device__ __forceinline__ void sd_store(const SoftmaxDecodeParams &p, size_t at, float x) {
    if (p.out_fp32) reinterpret_cast<float *>(p.out)[at] = x;
    else reinterpret_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(x);
}
__device__ __forceinline__ float sd_lse(float m, float l) { return (m + log2f(l)) * 0.69314718055994531f; }  // ln 2

__device__ __forceinline__ void sd_init(SoftmaxDecodeCtrl *cb) {
    for (int s = 0; s < SD_STAGES; ++s) {
        mbar_init(&cb->full[s], 1);
        mbar_init(&cb->empty[s], 4);
    }
    cb->abort = 0;
    fence_mbarrier_init();
}

__global__ void __launch_bounds__(SD_THREADS, 2)
la_softmax_decode_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                         const __grid_constant__ SoftmaxDecodeParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ SoftmaxDecodeShared sh;
    __shared__ long long sh_sum[5];
    __shared__ DecodeCursor sh_start;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    pdl_wait();                      // the cache and lengths as the kernels before leave them
    pdl_launch();                    // the join kernel may be set up meanwhile (it waits for this one's end)
    if (smem_u32(smem) & 1023) {     // the swizzle's atoms
        if (tid == 0) {
            record_status(p.status, ST_CUDA);
            p.info[blockIdx.x] = make_int4(0, 0, 0, 0);
        }
        return;
    }

    // ---- this CTA's run of tiles ----
    const int R = p.Hkv * p.chunks;  // rows of a request
    const int per = (p.B + 127) / 128;
    long long mine = 0, incl;
    if (tid < 128)
        for (int i = tid * per; i < min(p.B, (tid + 1) * per); ++i) {
            const int len = p.lens[i], nt = sd_tiles(len, p.max_keys);
            mine += nt;
            if (blockIdx.x == 0 && nt == 0 && len != -1) record_status(p.status, ST_INVALID);
        }
    incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sh_sum[warp] = incl;
    if (tid == 0) sd_init(&sh.cb);
    __syncthreads();
    const long long total = (sh_sum[0] + sh_sum[1] + sh_sum[2] + sh_sum[3]) * R;
    const int n = (int)(total < SD_CTAS ? total : SD_CTAS);
    if (tid == 0) p.info[blockIdx.x] = make_int4(0, 0, 0, 0);
    if ((int)blockIdx.x >= n) return;
    const long long t0 = total * blockIdx.x / n, t1 = total * (blockIdx.x + 1) / n;
    for (int w = 0; w < warp; ++w) incl += sh_sum[w];
    if (tid < 128 && (incl - mine) * R <= t0 && t0 < incl * R) {
        long long at = (incl - mine) * R;
        for (int i = tid * per;; ++i) {
            const int nt = sd_tiles(p.lens[i], p.max_keys);
            if (t0 < at + (long long)nt * R) {
                const long long rem = t0 - at;
                sh_start.b = i;
                sh_start.row = (int)(rem / nt);
                sh_start.tile = (int)(rem % nt);
                sh_start.nt = nt;
                sh_start.len = p.lens[i];
                break;
            }
            at += (long long)nt * R;
        }
    }
    __syncthreads();
    DecodeCursor c = sh_start;
    long long left = t1 - t0;
    auto advance = [&](int tile) {  // to tile `tile` of the row, or the next row
        c.tile = tile;
        if (c.tile == c.nt) {
            c.tile = 0;
            if (++c.row == R && left > 0) sd_next_request(c, p);
        }
    };

    if (warp == 4) {
        const DecodeLoader ld(&tmk, &tmv, p, lane);
        uint32_t it = 0;
        while (left > 0 && ld.load(c.b, c.len, c.row, c.tile, it, smem, &sh.cb, p, lane)) {
            ++it;
            --left;
            advance(c.tile + 1);
        }
        sd_drain(it, &sh.cb, p);
    } else {
        const float *red = reinterpret_cast<const float *>(smem + SD_RED);
        long long at = t0;  // tile number of the piece's first tile
        uint32_t it = 0;
        while (left > 0) {
            const int tile0 = c.tile, tile1 = (int)min((long long)c.nt, tile0 + left);
            sd_piece(p, smem, &sh, c.b, c.len, c.row, tile0, tile1, it, warp, lane);
            const int kvh = c.row / p.chunks, chunk = c.row - kvh * p.chunks;
            const int nh = min(SD_HEADS, p.G - chunk * SD_HEADS);
            const size_t at_o = (size_t)c.b * p.H + kvh * p.G + chunk * SD_HEADS;
            const bool whole = tile0 == 0 && tile1 == c.nt;
            // a cut row: part 0 when the row began in an earlier CTA, else part 1
            const long long row_at = at - tile0;  // tile number of the row's first tile
            float *part = p.parts + ((size_t)blockIdx.x * 2 + (row_at < t0 ? 0 : 1)) * SD_PART;
            for (int row = 0; row < nh; ++row) {
                const int col = sd_col(row, tid);
                const float x = red[row * D + col] + red[SD_HEADS * D + row * D + col];
                if (whole) {
                    float m, l;
                    sd_joined(&sh, row, m, l);
                    sd_store(p, (at_o + row) * D + tid, x / l);
                    if (tid == 0 && p.lse) p.lse[at_o + row] = sd_lse(m, l);
                } else {
                    part[row * D + tid] = x;
                }
            }
            if (!whole && tid < SD_HEADS) {
                float m, l;
                sd_joined(&sh, tid, m, l);
                part[SD_HEADS * D + tid] = m;
                part[SD_HEADS * D + SD_HEADS + tid] = l;
            }
            if (!whole && tid == 0 && row_at >= t0) {  // the row starts here and goes on: its parts
                const long long last = row_at + c.nt;   // one behind the row's last tile
                const int c1 = (int)((last * n - 1) / total);
                p.info[blockIdx.x] = make_int4(c.b, c.row, c1 - (int)blockIdx.x + 1, 0);
            }
            const bool stop = sh.stop != 0;
            named_bar_sync(1, 128);  // the buffers may be used again
            if (stop) break;
            left -= tile1 - tile0;
            at += tile1 - tile0;
            advance(tile1);
        }
    }
}

// Few, short rows: a cluster of CTAs per row, each with an equal share of the
// row's tiles, that join their parts through distributed shared memory.  One
// launch and no parts in memory, where the form above needs a second kernel.
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t local, uint32_t rank) {
    uint32_t a;
    float x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
    return x;
}

template <int SD_CLUSTER>
__global__ void __launch_bounds__(SD_THREADS, 2)
la_softmax_decode_cluster_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                                 const __grid_constant__ SoftmaxDecodeParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ SoftmaxDecodeShared sh;
    __shared__ float sh_ml[2][SD_HEADS];  // this CTA's m and l per head
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int rank = blockIdx.x % SD_CLUSTER, cl = blockIdx.x / SD_CLUSTER;
    const int R = p.Hkv * p.chunks, b = cl / R, crow = cl - b * R;
    if (tid == 0) sd_init(&sh.cb);
    pdl_wait();    // the cache and lengths as the kernels before leave them
    pdl_launch();  // the kernel behind may be set up (it waits for this one's end)
    const int len = p.lens[b], nt = sd_tiles(len, p.max_keys);
    if (smem_u32(smem) & 1023) {  // (the same in every CTA)
        if (tid == 0) record_status(p.status, ST_CUDA);
        return;
    }
    if (nt == 0) {  // no request in this row: the whole cluster leaves
        if (tid == 0 && crow == 0 && rank == 0 && len != -1) record_status(p.status, ST_INVALID);
        return;
    }
    __syncthreads();
    const int tile0 = (int)((long long)nt * rank / SD_CLUSTER), tile1 = (int)((long long)nt * (rank + 1) / SD_CLUSTER);
    const float *red = reinterpret_cast<const float *>(smem + SD_RED);
    if (warp == 4) {
        const DecodeLoader ld(&tmk, &tmv, p, lane);
        uint32_t it = 0;
        for (int tile = tile0; tile < tile1; ++tile, ++it)
            if (!ld.load(b, len, crow, tile, it, smem, &sh.cb, p, lane)) break;
        sd_drain(it, &sh.cb, p);
    } else {
        uint32_t it = 0;
        sd_piece(p, smem, &sh, b, len, crow, tile0, tile1, it, warp, lane);
        if (tid < SD_HEADS) sd_joined(&sh, tid, sh_ml[0][tid], sh_ml[1][tid]);
    }
    __syncthreads();
    cluster_sync_all();
    // CTA `rank` joins features [16 rank, 16 rank + 16) of every head
    const int kvh = crow / p.chunks, chunk = crow - kvh * p.chunks, nh = min(SD_HEADS, p.G - chunk * SD_HEADS);
    const size_t at_o = (size_t)b * p.H + kvh * p.G + chunk * SD_HEADS;
    constexpr int SHARE = D / SD_CLUSTER;
    for (int e = tid; e < nh * SHARE; e += SD_THREADS) {
        const int head = e / SHARE, d = rank * SHARE + e % SHARE;
        float mm[SD_CLUSTER], m = -INFINITY;
#pragma unroll
        for (int r = 0; r < SD_CLUSTER; ++r) {
            mm[r] = ld_cluster_f32(smem_u32(&sh_ml[0][head]), r);
            m = fmaxf(m, mm[r]);
        }
        const float u = m == -INFINITY ? 0.f : m;
        float l = 0.f, x = 0.f;
#pragma unroll
        for (int r = 0; r < SD_CLUSTER; ++r) {
            const float f = ex2(mm[r] - u);
            const float *src = red + head * D + sd_col(head, d);
            l = fmaf(ld_cluster_f32(smem_u32(&sh_ml[1][head]), r), f, l);
            x = fmaf(ld_cluster_f32(smem_u32(src), r) + ld_cluster_f32(smem_u32(src + SD_HEADS * D), r), f, x);
        }
        sd_store(p, (at_o + head) * D + d, x / l);
        if (d == 0 && p.lse) p.lse[at_o + head] = sd_lse(m, l);
    }
    cluster_sync_all();  // no CTA leaves while another reads its shared memory
}

// Joins the parts of the rows that the CTAs' borders cut: block (c, head) has
// the row that starts in CTA c, if one does, and thread d its feature d.
__global__ void __launch_bounds__(D) la_softmax_join_kernel(const __grid_constant__ SoftmaxDecodeParams p) {
    pdl_wait();
    const int4 in = p.info[blockIdx.x];
    if (in.z == 0) return;
    const int head = blockIdx.y, chunk = in.y % p.chunks;
    if (chunk * SD_HEADS + head >= p.G) return;
    const int h = (in.y / p.chunks) * p.G + chunk * SD_HEADS + head;
    // first part: slot 1 of CTA c; the others: slot 0 of the CTAs behind it
    const float *first = p.parts + ((size_t)blockIdx.x * 2 + 1) * SD_PART;
    auto part = [&](int i) -> const float * { return i == 0 ? first : first + ((size_t)2 * i - 1) * SD_PART; };
    float m = -INFINITY;
    for (int i = 0; i < in.z; ++i) m = fmaxf(m, part(i)[SD_HEADS * D + head]);
    const float u = m == -INFINITY ? 0.f : m;
    float l = 0.f, x = 0.f;
#pragma unroll 4
    for (int i = 0; i < in.z; ++i) {
        const float *pt = part(i);
        const float f = ex2(pt[SD_HEADS * D + head] - u);
        l = fmaf(pt[SD_HEADS * D + SD_HEADS + head], f, l);
        x = fmaf(pt[head * D + threadIdx.x], f, x);
    }
    const size_t at = (size_t)in.x * p.H + h;
    sd_store(p, at * D + threadIdx.x, x / l);
    if (threadIdx.x == 0 && p.lse) p.lse[at] = sd_lse(m, l);
}

// ---------------------------------------------------------------------------
// The cache: new tokens into their pages, pages copied inside the pool.
// ---------------------------------------------------------------------------

// The new tokens of a prompt chunk into their pages.
constexpr int APPEND_THREADS = 256;

__global__ void __launch_bounds__(APPEND_THREADS) la_cache_append_kernel(const AppendTables p, int T, const int *hdr) {
    pdl_launch();
    pdl_wait();
    if (hdr[HDR_G] == 0) return;  // the scheduler refused the tables
    const long long total = (long long)T * p.Hkv * (D / 8);
    for (long long e = (long long)blockIdx.x * APPEND_THREADS + threadIdx.x; e < total;
         e += (long long)gridDim.x * APPEND_THREADS)
        append_piece(e, p);
}

// Page src[i] -> page dst[i] of both caches.  A block copies 16 KiB pieces, 64
// bytes a thread in four loads that are in flight together.
constexpr int COPY_THREADS = 256;
constexpr int COPY_PIECE = COPY_THREADS * 64;

__global__ void __launch_bounds__(COPY_THREADS) la_cache_copy_kernel(uint8_t *kc, uint8_t *vc, const int *src,
                                                                     const int *dst, int n, int n_pages,
                                                                     long long page_bytes, int *status) {
    pdl_wait();
    pdl_launch();
    const int pieces = (int)((page_bytes + COPY_PIECE - 1) / COPY_PIECE);
    const long long total = 2LL * n * pieces;
    for (long long e = blockIdx.x; e < total; e += gridDim.x) {
        const int piece = (int)(e % pieces);
        const long long ci = e / pieces;
        const int i = (int)(ci >> 1);
        uint8_t *c = ci & 1 ? vc : kc;
        const int a = src[i], b = dst[i];
        if (a < 0 || a >= n_pages || b < 0 || b >= n_pages) {
            if (threadIdx.x == 0) record_status(status, ST_INVALID);
            continue;
        }
        const long long at = (long long)piece * COPY_PIECE + threadIdx.x * 16;
        const uint8_t *from = c + a * page_bytes;
        uint8_t *to = c + b * page_bytes;
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (at + k * COPY_THREADS * 16 < page_bytes)
                x[k] = __ldcs(reinterpret_cast<const uint4 *>(from + at + k * COPY_THREADS * 16));
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (at + k * COPY_THREADS * 16 < page_bytes)
                __stcs(reinterpret_cast<uint4 *>(to + at + k * COPY_THREADS * 16), x[k]);
    }
}

}  // namespace la
