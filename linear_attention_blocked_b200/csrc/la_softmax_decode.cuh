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
// per SM keep some 190 KB in flight, four times latency x bandwidth).  A warp
// takes 16 keys of a tile, with sums and maxima of its own that are joined when
// the row ends.  The group's heads are the rows or columns of m16n8k16 products:
// with 8 or 16 of them, tcgen05 tiles of 128 rows would be 7/8 empty and need the
// same bytes, while mma.sync from registers stays below the time the tile's bytes
// take.  The weights meet V as a bf16 pair hi + lo (within 2^-16 of each), so the
// output is nearly as exact as its own type.
//
// 64 requests of 8192 keys, 64 heads over 8: 2.15 GB at 6.8 TB/s, 83 % of what DRAM
// could nominally do, tensor pipe busy 16 %.  256 requests of up to 8192: 0.645 ms,
// 6.7 TB/s; one request of 524288 keys 0.327 ms, 6.6 TB/s: 90 % of what a kernel that
// only reads gets.
#pragma once
#include "la_softmax.cuh"

namespace la {

constexpr int SD_KEYS = 64;          // keys per tile
constexpr int SD_HALF = SD_KEYS * 128;         // 64 features of the tile's keys
constexpr int SD_TILE = 2 * SD_HALF;           // one of K, V
constexpr int SD_CTAS = 2 * 148;               // equal runs of tiles
// What a row costs next to its tiles, in tiles (Q, the join of the warps, the
// output: some 3 us, a tile 0.5): runs are equal in tiles + this per row.  (Runs of
// equal tiles left 9 requests of lengths up to 4000 at 52 us, against 18.)
constexpr int SD_ROW_COST = 5;
constexpr int SD_PART = 16 * D + 2 * 16;       // floats of one part: O, m, l of up to 16 heads

// The shape of a CTA.  HEADS, query heads in a row of tiles: wide, up to 16, the
// rows of m16n8k16 products; narrow, for groups of up to 8, the products turned
// over, S^T = K Q^T and O^T = V^T P^T with the heads as their 8 columns, which halves
// their number.  STAGES, tiles of the ring: 3, with 4 warps that take 16 keys of
// each tile, lets two CTAs share an SM; where there are no more CTAs than SMs, 6
// keep as much in flight, and 8 warps in two groups take the tiles in turn (a
// warp's 16 keys take it some 1000 cycles from K to O, one after another).  A stage
// of the ring then always belongs to the same group, which so waits for each of
// its fills in order: a barrier's phase is told by its parity alone.
template <int HEADS_, int STAGES_>
struct DecodeShape {
    static constexpr int HEADS = HEADS_, STAGES = STAGES_;
    static constexpr int GROUPS = STAGES == 6 ? 2 : 1;
    static constexpr int WARPS = 4 * GROUPS;
    static constexpr int THREADS = 32 * WARPS + 32;       // and a warp that loads
    static constexpr int BUFS = 32 / HEADS;               // sum buffers of [HEADS][128] fp32
    static constexpr int RED = STAGES * 2 * SD_TILE;
    static constexpr int SMEM = RED + BUFS * HEADS * D * 4;
    static_assert(STAGES % GROUPS == 0 && WARPS % BUFS == 0, "");
};
constexpr int SD_WIDE = 16, SD_NARROW = 8;

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
    int B, H, Hkv, G, chunks;         // chunks: rows of a request per key/value head
    int max_pages, n_pages, page, page_shift;
    long long max_keys;               // max_pages * page
    float scale_log2;
    unsigned long long wait_limit_ns;
    int *status;
};

struct SoftmaxDecodeCtrl {
    uint64_t full[6], empty[6];
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
template <class S>
struct SoftmaxDecodeShared {
    SoftmaxDecodeCtrl cb;
    int stop;
    float m[S::WARPS * S::HEADS], l[S::WARPS * S::HEADS];  // of each warp, per head
    float mj[S::HEADS], lj[S::HEADS];                      // joined
};

// The loads of a row's tiles (request b with len cached tokens, row = head and
// chunk): the whole warp, lane (kv, half, page of the tile) issuing one box of 64
// features of up to 64 keys.
template <class S>
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
    __device__ int key_of(int tile) const { return tile * SD_KEYS + (bx << bx_shift); }  // first key of the lane's box
    // The lane's page of a tile, as the table has it
    __device__ int page(int b, int len, int tile, const SoftmaxDecodeParams &p) const {
        const int key = key_of(tile);
        return g < 4 && key <= len ? p.pages[(size_t)b * p.max_pages + (key >> p.page_shift)] : 0;
    }
    __device__ bool load(int len, int row, int tile, int pid, uint32_t it, uint8_t *smem, SoftmaxDecodeCtrl *cb,
                         const SoftmaxDecodeParams &p, int lane) const {
        const int key = key_of(tile);
        const bool has = g < 4 && key <= len;
        const int s = it % S::STAGES;
        if (!ctrl_warp_wait(&cb->empty[s], ((it / S::STAGES) & 1) ^ 1, p.wait_limit_ns, p.status, cb)) return false;
        const int nb = __popc(__ballot_sync(0xffffffffu, has));
        if (lane == 0) mbar_expect_tx(&cb->full[s], (uint32_t)(nb << bx_shift) * 128u);
        __syncwarp();
        if (has) {
            if (pid < 0 || pid >= p.n_pages) {  // nothing outside the pool is read
                record_status(p.status, ST_INVALID);
                pid = 0;
            }
            const int r = (int)((((long long)pid * p.Hkv + row / p.chunks) << p.page_shift) + (key & (p.page - 1)));
            tma_load_3d(smem + s * 2 * SD_TILE + g * SD_HALF + (bx << bx_shift) * 128, tm, &cb->full[s], 0, r, g & 1, pol);
        }
        return true;
    }
    // Tiles [tile0, tile1) of a row; the next tile's page is fetched while the ring
    // is full.  False when a wait ran out.
    __device__ bool run(int b, int len, int row, int tile0, int tile1, uint32_t &it, uint8_t *smem,
                        SoftmaxDecodeCtrl *cb, const SoftmaxDecodeParams &p, int lane) const {
        int pid = page(b, len, tile0, p);
        for (int tile = tile0; tile < tile1; ++tile, ++it) {
            const int next = tile + 1 < tile1 ? page(b, len, tile + 1, p) : 0;
            if (!load(len, row, tile, pid, it, smem, cb, p, lane)) return false;
            pid = next;
        }
        return true;
    }
};

static_assert(sizeof(SoftmaxDecodeShared<DecodeShape<16, 3>>) <= 900 &&
              sizeof(SoftmaxDecodeShared<DecodeShape<8, 3>>) <= 900, "with the dynamic 112 KiB, two CTAs per SM");

template <class S>
__device__ __forceinline__ void sd_drain(uint32_t it, SoftmaxDecodeCtrl *cb, const SoftmaxDecodeParams &p) {
    for (uint32_t i = it > S::STAGES ? it - S::STAGES : 0; i < it; ++i) {  // copies land before the CTA exits
        drain_wait(&cb->full[i % S::STAGES], (i / S::STAGES) & 1);
    }
}

// Maximum and sum of a head over the warps
template <class S>
__device__ __forceinline__ void sd_joined(const SoftmaxDecodeShared<S> *sh, int head, float &m, float &l) {
    m = -INFINITY;
#pragma unroll
    for (int w = 0; w < S::WARPS; ++w) m = fmaxf(m, sh->m[w * S::HEADS + head]);
    const float u = m == -INFINITY ? 0.f : m;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < S::WARPS; ++w) l += sh->l[w * S::HEADS + head] * ex2(sh->m[w * S::HEADS + head] - u);
}

// Column of feature d of a head in the sum buffers: spreads the heads over the banks
__device__ __forceinline__ int sd_col(int head, int d) { return d ^ ((head & 7) << 3); }

// O of a head and feature, from the sum buffers
template <class S>
__device__ __forceinline__ float sd_sum(const float *red, int head, int d) {
    const float *at = red + head * D + sd_col(head, d);
    float x = at[0];
#pragma unroll
    for (int i = 1; i < S::BUFS; ++i) x += at[i * S::HEADS * D];
    return x;
}

// bf16 pairs hi + lo of two weights e >= 0, hi the next bf16 below e.  lo is then above
// zero whenever e is, at most 2^-7 e, and rounded by at most 2^-16 e.  With the nearest
// bf16 for hi, rounded by half of that, lo would be zero or negative for half of the
// weights, and with an infinite value hi v + lo v would be NaN where the sum is infinite.
__device__ __forceinline__ uint32_t sd_below(float e) {
    const uint32_t bits = __float_as_uint(e);
    return max(bits, 1u) - 1u;  // (0 stays 0)
}
__device__ __forceinline__ void sd_hi_lo(float a, float b, uint32_t &hi, uint32_t &lo) {
    const uint32_t x = sd_below(a), y = sd_below(b);
    hi = __byte_perm(x, y, 0x7632);  // the upper halves
    lo = pack_bf16x2(a - __uint_as_float(x & 0xffff0000u), b - __uint_as_float(y & 0xffff0000u));
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {  // an 8 x 8 bf16 matrix over the warp, transposed
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The warp's 16 keys [key0, key0 + 16) hold or lie behind the new token (position
// len): its row goes into the tile and, once, into the cache; rows of V behind it
// are zeroed (P = 0 keeps out what they hold only if it is finite).
__device__ __forceinline__ void sd_tail(const SoftmaxDecodeParams &p, uint8_t *kt, uint8_t *vt, int b, int len, int kvh,
                                        bool write, int key0, int row0, int lane) {
    if (len >= key0) {
        const int rr = row0 + len - key0, ch = lane & 15;
        const size_t src = ((size_t)b * p.Hkv + kvh) * D;
        const uint4 val = *reinterpret_cast<const uint4 *>((lane < 16 ? p.k : p.v) + src + ch * 8);
        *reinterpret_cast<uint4 *>((lane < 16 ? kt : vt) + (ch >> 3) * SD_HALF + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)) = val;
        if (write) {
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
            *reinterpret_cast<uint4 *>(vt + (ch >> 3) * SD_HALF + (row0 + rr) * 128 + ((ch & 7) << 4)) = make_uint4(0, 0, 0, 0);
    }
    __syncwarp();
}

// A warp's running state over its keys of a row, and the products for 16 keys.
// The layouts are those of the m16n8k16 fragments; g = lane / 4, t = lane % 4.
template <int HEADS>
struct DecodeWarp;

template <>
struct DecodeWarp<16> {  // heads g, g + 8 are rows of S and O
    uint32_t q[8][4];
    float o[16][4], m[2], l[2];
    __device__ void init(const __nv_bfloat16 *qr, int nh, int lane) {
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = g + (i & 1) * 8, col = kk * 16 + t4 * 2 + (i >> 1) * 8;
                q[kk][i] = row < nh ? *reinterpret_cast<const uint32_t *>(qr + (size_t)row * D + col) : 0u;
            }
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }
    __device__ void keys16(uint32_t ka, uint32_t va, int row0, int key0, int len, float scale_log2, int lane) {
        const int t4 = lane & 3;
        float sc[2][4] = {};
        const int rk = row0 + (lane & 7) + ((lane >> 4) << 3);  // key of this lane's address
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            const int ch = 2 * kk + ((lane >> 3) & 1);
            uint32_t bf[4];
            ldsm4(bf, ka + (ch >> 3) * SD_HALF + rk * 128 + (((ch & 7) ^ (rk & 7)) << 4));
            mma16816(sc[0], q[kk], bf[0], bf[1]);
            mma16816(sc[1], q[kk], bf[2], bf[3]);
        }
        float x[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int key = key0 + i * 8 + t4 * 2 + (k & 1);
                sc[i][k] = key <= len ? sc[i][k] * scale_log2 : -INFINITY;
                x[k >> 1] = fmaxf(x[k >> 1], sc[i][k]);
            }
#pragma unroll
        for (int o2 = 1; o2 < 4; o2 <<= 1) {
            x[0] = fmaxf(x[0], __shfl_xor_sync(0xffffffffu, x[0], o2));
            x[1] = fmaxf(x[1], __shfl_xor_sync(0xffffffffu, x[1], o2));
        }
        if (__any_sync(0xffffffffu, x[0] > m[0] || x[1] > m[1])) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float n = fmaxf(m[r], x[r]), a = n == -INFINITY ? 1.f : ex2(m[r] - n);
                m[r] = n;
                l[r] *= a;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    o[i][2 * r] *= a;
                    o[i][2 * r + 1] *= a;
                }
            }
        }
        const float u0 = m[0] == -INFINITY ? 0.f : m[0], u1 = m[1] == -INFINITY ? 0.f : m[1];
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float e0 = ex2(sc[i][0] - u0), e1 = ex2(sc[i][1] - u0);
            const float e2 = ex2(sc[i][2] - u1), e3 = ex2(sc[i][3] - u1);
            l[0] += e0 + e1;
            l[1] += e2 + e3;
            sd_hi_lo(e0, e1, hi[2 * i], lo[2 * i]);
            sd_hi_lo(e2, e3, hi[2 * i + 1], lo[2 * i + 1]);
        }
        const int rv = row0 + (lane & 15);
#pragma unroll
        for (int dd = 0; dd < 8; ++dd) {
            const int ch = 2 * dd + (lane >> 4);
            uint32_t bf[4];
            ldsm4_t(bf, va + (ch >> 3) * SD_HALF + rv * 128 + (((ch & 7) ^ (rv & 7)) << 4));
            mma16816(o[2 * dd], hi, bf[0], bf[1]);
            mma16816(o[2 * dd + 1], hi, bf[2], bf[3]);
            mma16816(o[2 * dd], lo, bf[0], bf[1]);
            mma16816(o[2 * dd + 1], lo, bf[2], bf[3]);
        }
    }
    __device__ int head(int r, int lane) const { return (lane >> 2) + 8 * r; }
    template <class S>
    __device__ void stats(SoftmaxDecodeShared<S> *sh, int warp, int lane) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if ((lane & 3) == 0) {
                sh->m[warp * 16 + head(r, lane)] = m[r];
                sh->l[warp * 16 + head(r, lane)] = l[r];
            }
        }
    }
    __device__ void add(float *buf, const float (&f)[2], bool add_in, int lane) const {
        const int t4 = lane & 3;
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int h = head(r, lane);
                float2 *at = reinterpret_cast<float2 *>(buf + h * D + sd_col(h, i * 8 + t4 * 2));
                float2 x = make_float2(o[i][2 * r] * f[r], o[i][2 * r + 1] * f[r]);
                if (add_in) {
                    x.x += at->x;
                    x.y += at->y;
                }
                *at = x;
            }
    }
};

template <>
struct DecodeWarp<8> {  // heads 2 t, 2 t + 1 are columns of S^T and O^T
    uint32_t q[8][2];
    float o[8][4], m[2], l[2];
    __device__ void init(const __nv_bfloat16 *qr, int nh, int lane) {
        const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                q[kk][i] = g < nh ? *reinterpret_cast<const uint32_t *>(qr + (size_t)g * D + kk * 16 + t4 * 2 + i * 8) : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }
    __device__ void keys16(uint32_t ka, uint32_t va, int row0, int key0, int len, float scale_log2, int lane) {
        const int g = lane >> 2;
        float s0[4] = {}, s1[4] = {};  // two chains of sums
        const int rk = row0 + (lane & 15);  // key of this lane's address
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
            const int ch = 2 * kk + (lane >> 4);
            uint32_t a[4];
            ldsm4(a, ka + (ch >> 3) * SD_HALF + rk * 128 + (((ch & 7) ^ (rk & 7)) << 4));
            mma16816(kk & 1 ? s1 : s0, a, q[kk][0], q[kk][1]);
        }
        float x[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            s0[k] = key0 + g + (k >> 1) * 8 <= len ? (s0[k] + s1[k]) * scale_log2 : -INFINITY;
            x[k & 1] = fmaxf(x[k & 1], s0[k]);
        }
#pragma unroll
        for (int o2 = 4; o2 < 32; o2 <<= 1) {
            x[0] = fmaxf(x[0], __shfl_xor_sync(0xffffffffu, x[0], o2));
            x[1] = fmaxf(x[1], __shfl_xor_sync(0xffffffffu, x[1], o2));
        }
        if (__any_sync(0xffffffffu, x[0] > m[0] || x[1] > m[1])) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float n = fmaxf(m[r], x[r]), a = n == -INFINITY ? 1.f : ex2(m[r] - n);
                m[r] = n;
                l[r] *= a;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o[i][r] *= a;
                    o[i][r + 2] *= a;
                }
            }
        }
        const float u0 = m[0] == -INFINITY ? 0.f : m[0], u1 = m[1] == -INFINITY ? 0.f : m[1];
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // keys g + 8 i
            const float e0 = ex2(s0[2 * i] - u0), e1 = ex2(s0[2 * i + 1] - u1);
            l[0] += e0;
            l[1] += e1;
            sd_hi_lo(e0, e1, hi[i], lo[i]);
            hi[i] = movmatrix_t(hi[i]);  // keys x heads -> the operand with keys along its pairs
            lo[i] = movmatrix_t(lo[i]);
        }
        const int rv = row0 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
        for (int dd = 0; dd < 8; ++dd) {
            const int ch = 2 * dd + ((lane >> 3) & 1);
            uint32_t a[4];
            ldsm4_t(a, va + (ch >> 3) * SD_HALF + rv * 128 + (((ch & 7) ^ (rv & 7)) << 4));
            mma16816(o[dd], a, hi[0], hi[1]);
            mma16816(o[dd], a, lo[0], lo[1]);
        }
    }
    __device__ int head(int r, int lane) const { return (lane & 3) * 2 + r; }
    template <class S>
    __device__ void stats(SoftmaxDecodeShared<S> *sh, int warp, int lane) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
            for (int o2 = 4; o2 < 32; o2 <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o2);
            if (lane < 4) {
                sh->m[warp * 8 + head(r, lane)] = m[r];
                sh->l[warp * 8 + head(r, lane)] = l[r];
            }
        }
    }
    __device__ void add(float *buf, const float (&f)[2], bool add_in, int lane) const {
        const int g = lane >> 2;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int h = head(k & 1, lane);
                float *at = buf + h * D + sd_col(h, i * 16 + g + (k >> 1) * 8);
                const float x = o[i][k] * f[k & 1];
                *at = add_in ? *at + x : x;
            }
    }
};

// The attention warps over tiles [tile0, tile1) of a row.  Leaves, behind a
// barrier, the joined m and l in `sh`, the sums of O (relative to the joined m) in
// the buffers of smem + RED to be added (sd_sum), and in sh->stop whether a
// wait ran out.  The caller has the warps meet again before the next call; with two
// groups there is one call (the ring's first tile is the row's).
template <class S>
__device__ __forceinline__ void sd_piece(const SoftmaxDecodeParams &p, uint8_t *smem, SoftmaxDecodeShared<S> *sh, int b,
                                         int len, int crow, int tile0, int tile1, uint32_t &it, int warp, int lane) {
    constexpr int HEADS = S::HEADS;
    const uint32_t sbase = smem_u32(smem);
    SoftmaxDecodeCtrl *cb = &sh->cb;
    const int kvh = crow / p.chunks, chunk = crow - kvh * p.chunks;
    const int nh = min(HEADS, p.G - chunk * HEADS);  // heads of this row
    DecodeWarp<HEADS> w;
    w.init(p.q + ((size_t)b * p.H + kvh * p.G + chunk * HEADS) * D, nh, lane);
    const int group = warp >> 2, row0 = (warp & 3) * 16;
    for (int tile = tile0 + group; tile < tile1; tile += S::GROUPS) {
        const uint32_t n = it + (uint32_t)(tile - tile0);
        const int s = n % S::STAGES;
        if (!ctrl_warp_wait(&cb->full[s], (n / S::STAGES) & 1, p.wait_limit_ns, p.status, cb)) break;
        uint8_t *kt = smem + s * 2 * SD_TILE, *vt = kt + SD_TILE;
        const int key0 = tile * SD_KEYS + row0;
        const bool tail = key0 + 16 > len;
        if (tail) sd_tail(p, kt, vt, b, len, kvh, chunk == 0, key0, row0, lane);
        w.keys16(sbase + (uint32_t)(kt - smem), sbase + (uint32_t)(vt - smem), row0, key0, len, p.scale_log2, lane);
        if (tail) fence_proxy_async_smem();  // this thread's writes before the next TMA load
        __syncwarp();
        if (lane == 0) mbar_arrive(&cb->empty[s]);
    }
    it += (uint32_t)(tile1 - tile0);
    w.stats(sh, warp, lane);
    named_bar_sync(1, 32 * S::WARPS);
    if (warp == 0 && lane == 0) sh->stop = cb->abort;  // one decision for all warps
    if (warp == 1 && lane < HEADS) sd_joined<S>(sh, lane, sh->mj[lane], sh->lj[lane]);
    float f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < S::WARPS; ++i) m = fmaxf(m, sh->m[i * HEADS + w.head(r, lane)]);
        f[r] = w.m[r] == -INFINITY ? 0.f : ex2(w.m[r] - m);
    }
    float *buf = reinterpret_cast<float *>(smem + S::RED) + (warp % S::BUFS) * HEADS * D;
    for (int turn = 0; turn < S::WARPS / S::BUFS; ++turn) {  // the first BUFS warps store, the others add
        if (warp / S::BUFS == turn) w.add(buf, f, turn > 0, lane);
        named_bar_sync(1, 32 * S::WARPS);
    }
}

__device__ __forceinline__ void sd_store(const SoftmaxDecodeParams &p, size_t at, float x) {
    if (p.out_fp32) reinterpret_cast<float *>(p.out)[at] = x;
    else reinterpret_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(x);
}
__device__ __forceinline__ float sd_lse(float m, float l) { return (m + log2f(l)) * 0.69314718055994531f; }  // ln 2

__device__ __forceinline__ void sd_init(SoftmaxDecodeCtrl *cb) {
    for (int s = 0; s < 6; ++s) {
        mbar_init(&cb->full[s], 1);
        mbar_init(&cb->empty[s], 4);
    }
    cb->abort = 0;
    fence_mbarrier_init();
}

template <int HEADS>
__global__ void __launch_bounds__(DecodeShape<HEADS, 3>::THREADS, 2)
la_softmax_decode_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                         const __grid_constant__ SoftmaxDecodeParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using S = DecodeShape<HEADS, 3>;
    __shared__ SoftmaxDecodeShared<S> sh;
    __shared__ long long sh_sum[4];
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
            mine += nt ? nt + SD_ROW_COST : 0;
            if (blockIdx.x == 0 && nt == 0 && len != -1) record_status(p.status, ST_INVALID);
        }
    incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31 && warp < 4) sh_sum[warp] = incl;
    if (tid == 0) sd_init(&sh.cb);
    __syncthreads();
    const long long total = (sh_sum[0] + sh_sum[1] + sh_sum[2] + sh_sum[3]) * R;
    const int n = (int)(total < SD_CTAS ? total : SD_CTAS);
    if (tid == 0) p.info[blockIdx.x] = make_int4(0, 0, 0, 0);
    if ((int)blockIdx.x >= n) return;
    const long long t0 = total * blockIdx.x / n, t1 = total * (blockIdx.x + 1) / n;
    for (int w = 0; w < min(warp, 4); ++w) incl += sh_sum[w];
    if (tid < 128 && (incl - mine) * R <= t0 && t0 < incl * R) {
        long long at = (incl - mine) * R;
        for (int i = tid * per;; ++i) {
            const int nt = sd_tiles(p.lens[i], p.max_keys), units = nt ? nt + SD_ROW_COST : 0;
            if (t0 < at + (long long)units * R) {
                const long long rem = t0 - at;
                sh_start.b = i;
                sh_start.row = (int)(rem / units);
                sh_start.tile = (int)(rem % units) - SD_ROW_COST;
                sh_start.nt = nt;
                sh_start.len = p.lens[i];
                break;
            }
            at += (long long)units * R;
        }
    }
    __syncthreads();
    DecodeCursor c = sh_start;  // (tile -SD_ROW_COST: the row's first unit)
    // The run's pieces in order: tiles [tile0, tile1) of c's row, the row's first
    // unit at row_at.  False when the run is through.
    long long at = t0;
    int tile0 = 0, tile1 = 0;
    long long row_at = 0;
    auto piece = [&]() -> bool {
        for (;;) {
            if (at >= t1) return false;
            row_at = at - (c.tile + SD_ROW_COST);
            tile0 = max(c.tile, 0);
            tile1 = (int)min((long long)c.nt, c.tile + (t1 - at));
            if (tile1 > tile0) return true;
            at = t1;  // the run ends before the row's first tile
        }
    };
    auto next_piece = [&]() {
        at += tile1 - c.tile;
        c.tile = tile1;
        if (c.tile == c.nt) {
            c.tile = -SD_ROW_COST;
            if (++c.row == R && at < t1) {
                sd_next_request(c, p);
                c.tile = -SD_ROW_COST;
            }
        }
    };

    if (warp == S::WARPS) {
        const DecodeLoader<S> ld(&tmk, &tmv, p, lane);
        uint32_t it = 0;
        for (; piece(); next_piece())
            if (!ld.run(c.b, c.len, c.row, tile0, tile1, it, smem, &sh.cb, p, lane)) break;
        sd_drain<S>(it, &sh.cb, p);
    } else {
        const float *red = reinterpret_cast<const float *>(smem + S::RED);
        uint32_t it = 0;
        for (; piece(); next_piece()) {
            sd_piece<S>(p, smem, &sh, c.b, c.len, c.row, tile0, tile1, it, warp, lane);
            const int kvh = c.row / p.chunks, chunk = c.row - kvh * p.chunks;
            const int nh = min(HEADS, p.G - chunk * HEADS);
            const size_t at_o = (size_t)c.b * p.H + kvh * p.G + chunk * HEADS;
            const bool whole = tile0 == 0 && tile1 == c.nt;
            // a cut row: part 0 when its tiles began in an earlier CTA, else part 1
            const bool begins = tile0 == 0;
            float *part = p.parts + ((size_t)blockIdx.x * 2 + (begins ? 1 : 0)) * SD_PART;
            const int d = tid % D;
            for (int row = tid / D; row < nh; row += 32 * S::WARPS / D) {
                const float x = sd_sum<S>(red, row, d);
                if (whole) {
                    const float m = sh.mj[row], l = sh.lj[row];
                    sd_store(p, (at_o + row) * D + d, x / l);
                    if (d == 0 && p.lse) p.lse[at_o + row] = sd_lse(m, l);
                } else {
                    part[row * D + d] = x;
                }
            }
            if (!whole && tid < HEADS) {
                part[16 * D + tid] = sh.mj[tid];
                part[16 * D + 16 + tid] = sh.lj[tid];
            }
            if (!whole && tid == 0 && begins) {  // the row goes on in the CTAs behind: its parts
                const long long last = row_at + SD_ROW_COST + c.nt;  // one behind the row's last unit
                const int c1 = (int)((last * n - 1) / total);
                p.info[blockIdx.x] = make_int4(c.b, c.row, c1 - (int)blockIdx.x + 1, 0);
            }
            const bool stop = sh.stop != 0;
            named_bar_sync(1, 32 * S::WARPS);  // the buffers may be used again
            if (stop) break;
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

template <int HEADS, int STAGES, int SD_CLUSTER>
__global__ void __launch_bounds__(DecodeShape<HEADS, STAGES>::THREADS, STAGES == 6 ? 1 : 2)
la_softmax_decode_cluster_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                                 const __grid_constant__ SoftmaxDecodeParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using S = DecodeShape<HEADS, STAGES>;
    __shared__ SoftmaxDecodeShared<S> sh;
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
    const float *red = reinterpret_cast<const float *>(smem + S::RED);
    if (warp == S::WARPS) {
        const DecodeLoader<S> ld(&tmk, &tmv, p, lane);
        uint32_t it = 0;
        ld.run(b, len, crow, tile0, tile1, it, smem, &sh.cb, p, lane);
        sd_drain<S>(it, &sh.cb, p);
    } else {
        uint32_t it = 0;
        sd_piece<S>(p, smem, &sh, b, len, crow, tile0, tile1, it, warp, lane);
    }
    const int kvh = crow / p.chunks, chunk = crow - kvh * p.chunks, nh = min(HEADS, p.G - chunk * HEADS);
    const size_t at_o = (size_t)b * p.H + kvh * p.G + chunk * HEADS;
    __syncthreads();
    if (SD_CLUSTER == 1) {
        for (int e = tid; e < nh * D; e += S::THREADS) {
            const int head = e / D, d = e % D;
            sd_store(p, (at_o + head) * D + d, sd_sum<S>(red, head, d) / sh.lj[head]);
            if (d == 0 && p.lse) p.lse[at_o + head] = sd_lse(sh.mj[head], sh.lj[head]);
        }
        return;
    }
    cluster_sync_all();
    // CTA `rank` joins its share of every head's features
    constexpr int SHARE = D / SD_CLUSTER;
    for (int e = tid; e < nh * SHARE; e += S::THREADS) {
        const int head = e / SHARE, d = rank * SHARE + e % SHARE;
        float mm[SD_CLUSTER], m = -INFINITY;
#pragma unroll
        for (int r = 0; r < SD_CLUSTER; ++r) {
            mm[r] = ld_cluster_f32(smem_u32(&sh.mj[head]), r);
            m = fmaxf(m, mm[r]);
        }
        const float u = m == -INFINITY ? 0.f : m;
        float l = 0.f, x = 0.f;
#pragma unroll
        for (int r = 0; r < SD_CLUSTER; ++r) {
            const float f = ex2(mm[r] - u);
            const float *src = red + head * D + sd_col(head, d);
            float y = ld_cluster_f32(smem_u32(src), r);
#pragma unroll
            for (int i = 1; i < S::BUFS; ++i) y += ld_cluster_f32(smem_u32(src + i * HEADS * D), r);
            l = fmaf(ld_cluster_f32(smem_u32(&sh.lj[head]), r), f, l);
            x = fmaf(y, f, x);
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
    const int heads = p.G > SD_NARROW ? SD_WIDE : SD_NARROW;  // of a row
    const int head = blockIdx.y, chunk = in.y % p.chunks;
    if (chunk * heads + head >= p.G) return;
    const int h = (in.y / p.chunks) * p.G + chunk * heads + head;
    // first part: slot 1 of CTA c; the others: slot 0 of the CTAs behind it
    const float *first = p.parts + ((size_t)blockIdx.x * 2 + 1) * SD_PART;
    auto part = [&](int i) -> const float * { return i == 0 ? first : first + ((size_t)2 * i - 1) * SD_PART; };
    float m = -INFINITY;
    for (int i = 0; i < in.z; ++i) m = fmaxf(m, part(i)[16 * D + head]);
    const float u = m == -INFINITY ? 0.f : m;
    float l = 0.f, x = 0.f;
#pragma unroll 4
    for (int i = 0; i < in.z; ++i) {
        const float *pt = part(i);
        const float f = ex2(pt[16 * D + head] - u);
        l = fmaf(pt[16 * D + 16 + head], f, l);
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
// bytes a thread in four loads that are in flight together.  3001 pages of 128 KiB
// in both: 257 us, 6.1 TB/s read and written, 94 % of a plain copy.
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
