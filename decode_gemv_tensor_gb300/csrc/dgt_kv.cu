// dgt_kv.cu -- the paged 8-bit cache: quantising append, reading back, and the
// page operations (copy, fork, reserve with copy on write, free, compact).
//
// An append reads the new rows of a block once, into registers: the largest
// magnitude (of the bf16 bits, two at a time) gives the power-of-two scale, the
// codes follow by one multiplication and one rounding (exact scaling, so the
// result depends on no order).  Values are transposed four by four through
// shared memory.  Page copies move whole pages, bytes untouched.  Page
// bookkeeping is integer work on a few words per sequence, done by one CTA in
// the order of the list.
//
// Bounds: a step's append is latency (16 sequences, append and read back 7.3
// us); a prompt's the loads in flight (three of up to 3001 rows, 8 heads of
// 256, append and read back 35.8 us, 55 % of the measured copy rate); copies
// HBM (160 pages of 28 layers, 1.17 GB: 184 us, 95 %).
#include "dgt_kv.cuh"

#include "dgt_device.cuh"

namespace dgt {

// Smallest e with amax <= 448 * 2^e, clamped to KV_EMIN (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_exp(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int x = (int)(u >> 23) - 127;             // subnormals: -127, below the clamp
    const int e = x - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return e < KV_EMIN ? KV_EMIN : e;
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
    return (uint16_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// The code byte pair to two floats.
__device__ __forceinline__ float2 e4m3x2_f32(uint16_t c) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3);
    return __half22float2(__half2(h));
}

// A bf16 pair with what is not finite set to zero.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
    return w;
}

// Value tiles in shared memory, 64 tokens of D / 4 words (four dimensions
// each): the words of a row permuted by its sixteen-token quarter, so that the
// four quarters of a word, read together, fall into different banks.
__device__ __forceinline__ uint32_t tile_word(uint32_t D, uint32_t t, uint32_t w) {
    return t * (D / 4) + (w ^ (8 * ((t >> 4) & (D >= 128 ? 3 : 1))));
}

// Four words of four bytes, transposed.
__device__ __forceinline__ void transpose4(uint32_t (&x)[4]) {
    const uint32_t a = prmt(x[0], x[1], 0x5140u), b = prmt(x[2], x[3], 0x5140u);   // bytes 0 and 1 of each pair
    const uint32_t c = prmt(x[0], x[1], 0x7362u), d = prmt(x[2], x[3], 0x7362u);   // bytes 2 and 3
    x[0] = prmt(a, b, 0x5410u);
    x[1] = prmt(a, b, 0x7632u);
    x[2] = prmt(c, d, 0x5410u);
    x[3] = prmt(c, d, 0x7632u);
}

struct AppendArgs {
    dgt_kv_cache c;
    uint32_t layer, batch;
    uint64_t tokens;
    dgt_heads x[2];
    const int32_t *seqs, *start, *cu;
    int32_t *status;
};

constexpr uint32_t AP_THREADS = 128;

// One CTA: (block item, head, keys or values).
template <uint32_t D>
__global__ void __launch_bounds__(AP_THREADS) k_kv_append(AppendArgs a) {
    __shared__ uint32_t red[AP_THREADS / 32];
    __shared__ __align__(16) uint32_t tile[KV_P * D / 4];
    pdl_trigger();
    pdl_wait();
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t head = blockIdx.y, side = blockIdx.z;
    uint32_t b = blockIdx.x, blk = 0, row0 = blockIdx.x, n = 1;
    int32_t cu0 = 0;
    if (a.cu) {
        cu0 = a.cu[0];   // the numbering begins at the first entry's rows: 0
        b = item_entry(a.cu, a.batch, blockIdx.x, KV_P, 2);
        blk = blockIdx.x - item_base(a.cu, b, KV_P, 2);
        row0 = (uint32_t)a.cu[b];
        n = (uint32_t)(a.cu[b + 1] - a.cu[b]);
    }
    if (n == 0 && cu0 == 0) return;
    const int32_t seq = a.seqs[b], start = a.start[b];
    if (cu0 != 0 || (uint64_t)row0 + n > a.tokens || seq < 0 || (uint32_t)seq >= a.c.max_seqs || start < 0 ||
        (uint64_t)start + n > (uint64_t)a.c.max_pages * KV_P) {
        if (tid == 0) set_status(a.status, DGT_ERR_ARG);
        return;
    }
    const uint32_t pi = (uint32_t)start / KV_P + blk;
    if ((uint64_t)pi * KV_P >= (uint64_t)start + n) return;   // an empty number
    const int32_t page = a.c.table[(uint64_t)seq * a.c.max_pages + pi];
    if (page < 0 || (uint32_t)page >= a.c.pages) {
        if (tid == 0) set_status(a.status, DGT_ERR_ARG);
        return;
    }
    const uint32_t t0 = pi * KV_P;
    const uint32_t lo = blk == 0 ? (uint32_t)start - t0 : 0;
    const uint32_t hi = min(KV_P, (uint32_t)start + n - t0);
    const dgt_heads &x = a.x[side];
    const uint16_t *src = x.data + (int64_t)head * x.head_stride +
                          (int64_t)(row0 + (t0 + lo - (uint32_t)start)) * x.token_stride;
    const uint64_t bi = kv_block(a.c, a.layer, (uint32_t)page, head);
    uint8_t *dst = (side ? a.c.v : a.c.k) + bi * (KV_P * D);
    float *scale_p = (side ? a.c.v_scale : a.c.k_scale) + bi;

    // the new rows, and their largest magnitude
    constexpr uint32_t CH = D / 16;                          // 16-element chunks of a row
    constexpr uint32_t N = KV_P * CH / AP_THREADS;           // chunks of a thread
    const uint32_t chunks = (hi - lo) * CH;
    uint4 u[N][2];
#pragma unroll
    for (uint32_t k = 0; k < N; k++) {
        const uint32_t i = tid + k * AP_THREADS;
        u[k][0] = u[k][1] = make_uint4(0, 0, 0, 0);
        if (i < chunks) {
            const uint4 *p = reinterpret_cast<const uint4 *>(src + (int64_t)(i / CH) * x.token_stride + (i % CH) * 16);
            u[k][0] = p[0];
            u[k][1] = p[1];
        }
    }
    const float s_old = lo ? *scale_p : 0.0f;   // read by all before thread 0 writes it
    const int32_t holders = a.c.refs[page];
    auto largest = [&]() {
        uint32_t m = 0;
#pragma unroll
        for (uint32_t k = 0; k < N; k++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const uint4 v = u[k][e];
                m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                         __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
            }
        m = __reduce_max_sync(DGT_FULL, max(m & 0xFFFFu, m >> 16));
        if (lane == 0) red[warp] = m;
        __syncthreads();
        m = 0;
#pragma unroll
        for (uint32_t i = 0; i < AP_THREADS / 32; i++) m = max(m, red[i]);
        return m;
    };
    uint32_t top = largest();
    if (holders > 1) {   // other sequences read this page
        if (tid == 0) set_status(a.status, DGT_ERR_ARG);
        return;
    }
    bool bad = top >= 0x7F80u;
    if (bad) {
        // a value that is not finite: the block's scale will say so; its finite values as ever
#pragma unroll
        for (uint32_t k = 0; k < N; k++)
#pragma unroll
            for (int e = 0; e < 2; e++) {
                uint4 &v = u[k][e];
                v = make_uint4(finite_pair(v.x), finite_pair(v.y), finite_pair(v.z), finite_pair(v.w));
            }
        __syncthreads();
        top = largest();
    }
    const float amax = __uint_as_float(top << 16);
    int e = scale_exp(amax);
    bool grow = false;
    float down = 1.0f;
    if (lo) {
        if (s_old != s_old) {
            bad = true;
        } else {
            const int eo = (int)(__float_as_uint(s_old) >> 23) - 127;
            if (eo >= e) {
                e = eo;
            } else {
                grow = true;
                down = s_old / exp2_int(e);   // a power of two below 1
            }
        }
    }
    const float inv = exp2_int(-e);
    if (tid == 0) *scale_p = bad ? __uint_as_float(0x7FC00000u) : exp2_int(e);

    // tokens that were there, to the new scale: two codes of a word at a time
    if (grow) {
        const uint32_t words = side ? D * KV_P / 4 : KV_P * D / 4;
        for (uint32_t i = tid; i < words; i += AP_THREADS) {
            // the four bytes of a value word are four tokens of a dimension,
            // those of a key word four dimensions of a token
            uint32_t keep = 0xFFFFFFFFu;   // bytes that stay as they are
            if (side) {
                const uint32_t t = (i * 4) % KV_P;
                if (t >= lo) continue;
                keep = lo - t >= 4 ? 0u : 0xFFFFFFFFu << (8 * (lo - t));
            } else {
                const uint32_t t = D == 64 ? (i * 4) / 64 : ((i * 4) % (KV_P * 128)) / 128;
                if (t >= lo) continue;
                keep = 0u;
            }
            uint32_t *wp = reinterpret_cast<uint32_t *>(dst) + i;
            const uint32_t w = *wp;
            const float2 f0 = e4m3x2_f32((uint16_t)w), f1 = e4m3x2_f32((uint16_t)(w >> 16));
            const uint32_t r = (uint32_t)e4m3x2(f0.x * down, f0.y * down) |
                               (uint32_t)e4m3x2(f1.x * down, f1.y * down) << 16;
            *wp = (w & keep) | (r & ~keep);
        }
        __syncthreads();   // a value word may hold old and new tokens
    }

    // codes: a chunk of keys is 16 bytes of its row; values go through the tile
#pragma unroll
    for (uint32_t k = 0; k < N; k++) {
        const uint32_t i = tid + k * AP_THREADS;
        if (i >= chunks) break;
        const uint32_t r = i / CH, c = i % CH;
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint4 v = u[k][j / 2];
            const uint32_t w0 = j & 1 ? v.z : v.x, w1 = j & 1 ? v.w : v.y;
            o[j] = (uint32_t)e4m3x2(bf16lo(w0) * inv, bf16hi(w0) * inv) |
                   (uint32_t)e4m3x2(bf16lo(w1) * inv, bf16hi(w1) * inv) << 16;
        }
        if (side == 0)
            *reinterpret_cast<uint4 *>(dst + kv_k_off(D, lo + r, c * 16)) = make_uint4(o[0], o[1], o[2], o[3]);
        else
            *reinterpret_cast<uint4 *>(&tile[tile_word(D, lo + r, 4 * c)]) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (side == 0) return;
    __syncthreads();
    if (lo == 0 && hi == KV_P) {
        // four dimensions by sixteen tokens a thread, four rows of 16 bytes out
        for (uint32_t i = tid; i < D; i += AP_THREADS) {
            const uint32_t q = i & 3, w = i >> 2;
            uint32_t y[4][4];   // [word of four tokens][dimension]
#pragma unroll
            for (uint32_t j = 0; j < 4; j++) {
#pragma unroll
                for (uint32_t t = 0; t < 4; t++) y[j][t] = tile[tile_word(D, 16 * q + 4 * j + t, w)];
                transpose4(y[j]);
            }
#pragma unroll
            for (uint32_t d = 0; d < 4; d++)
                *reinterpret_cast<uint4 *>(dst + kv_v_off(16 * q, 4 * w + d)) = make_uint4(y[0][d], y[1][d], y[2][d], y[3][d]);
        }
        return;
    }
    // a part of a block: whole words of four tokens where they are new, bytes at the ends
    const uint8_t *tb = reinterpret_cast<const uint8_t *>(tile);
    const uint32_t w0 = lo / 4, nw = (hi + 3) / 4 - w0;
    for (uint32_t i = tid; i < D * nw; i += AP_THREADS) {
        const uint32_t d = i / nw, t = (w0 + i % nw) * 4;
        uint8_t *q = dst + kv_v_off(t, d);
        uint32_t w = 0;
#pragma unroll
        for (uint32_t j = 0; j < 4; j++) w |= (uint32_t)tb[4 * tile_word(D, t + j, d / 4) + d % 4] << (8 * j);
        if (t >= lo && t + 4 <= hi) {
            *reinterpret_cast<uint32_t *>(q) = w;
        } else {
            for (uint32_t j = 0; j < 4; j++)
                if (t + j >= lo && t + j < hi) q[j] = (uint8_t)(w >> (8 * j));
        }
    }
}

struct ReadArgs {
    dgt_kv_cache c;
    uint32_t layer0, layers, batch;
    uint64_t tokens;
    const int32_t *seqs, *first, *cu;
    uint16_t *out[2];
    int32_t *status;
};

constexpr uint32_t RD_THREADS = 128;

// Four codes of a word, times the scale, to four bf16 (exact).
__device__ __forceinline__ uint2 decode4(uint32_t w, float s) {
    const float2 a = e4m3x2_f32((uint16_t)w), b = e4m3x2_f32((uint16_t)(w >> 16));
    uint2 r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.x) : "f"(a.y * s), "f"(a.x * s));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.y) : "f"(b.y * s), "f"(b.x * s));
    return r;
}

// One CTA: (block item, head, layer and keys or values).
template <uint32_t D>
__global__ void __launch_bounds__(RD_THREADS) k_kv_read(ReadArgs a) {
    __shared__ __align__(16) uint32_t tile[KV_P * D / 4];
    pdl_trigger();
    pdl_wait();
    const uint32_t tid = threadIdx.x;
    const uint32_t head = blockIdx.y, side = blockIdx.z & 1, layer = a.layer0 + blockIdx.z / 2;
    if (!a.out[side]) return;
    uint32_t b = blockIdx.x, blk = 0, row0 = blockIdx.x, n = 1;
    int32_t cu0 = 0;
    if (a.cu) {
        cu0 = a.cu[0];   // the numbering begins at the first entry's rows: 0
        b = item_entry(a.cu, a.batch, blockIdx.x, KV_P, 2);
        blk = blockIdx.x - item_base(a.cu, b, KV_P, 2);
        row0 = (uint32_t)a.cu[b];
        n = (uint32_t)(a.cu[b + 1] - a.cu[b]);
    }
    if (n == 0 && cu0 == 0) return;
    const int32_t seq = a.seqs[b], first = a.first[b];
    if (cu0 != 0 || (uint64_t)row0 + n > a.tokens || seq < 0 || (uint32_t)seq >= a.c.max_seqs || first < 0 ||
        (uint64_t)first + n > (uint64_t)a.c.max_pages * KV_P) {
        if (tid == 0) set_status(a.status, DGT_ERR_ARG);
        return;
    }
    const uint32_t pi = (uint32_t)first / KV_P + blk;
    if ((uint64_t)pi * KV_P >= (uint64_t)first + n) return;
    const int32_t page = a.c.table[(uint64_t)seq * a.c.max_pages + pi];
    if (page < 0 || (uint32_t)page >= a.c.pages) {
        if (tid == 0) set_status(a.status, DGT_ERR_ARG);
        return;
    }
    const uint32_t t0 = pi * KV_P;
    const uint32_t lo = blk == 0 ? (uint32_t)first - t0 : 0;
    const uint32_t hi = min(KV_P, (uint32_t)first + n - t0);
    const uint64_t bi = kv_block(a.c, layer, (uint32_t)page, head);
    const uint8_t *src = (side ? a.c.v : a.c.k) + bi * (KV_P * D);
    const float s = (side ? a.c.v_scale : a.c.k_scale)[bi];
    uint16_t *out = a.out[side] + (((uint64_t)(layer - a.layer0) * a.tokens + row0 + (t0 + lo - (uint32_t)first)) *
                                       a.c.kv_heads + head) * D;
    if (side) {
        // rows of tokens out of rows of dimensions: four dimensions by sixteen tokens a thread
        for (uint32_t i = tid; i < D; i += RD_THREADS) {
            const uint32_t q = i & 3, w = i >> 2;
            uint4 v[4];
#pragma unroll
            for (uint32_t d = 0; d < 4; d++) v[d] = *reinterpret_cast<const uint4 *>(src + kv_v_off(16 * q, 4 * w + d));
#pragma unroll
            for (uint32_t j = 0; j < 4; j++) {
                uint32_t y[4];
#pragma unroll
                for (uint32_t d = 0; d < 4; d++) y[d] = j == 0 ? v[d].x : j == 1 ? v[d].y : j == 2 ? v[d].z : v[d].w;
                transpose4(y);
#pragma unroll
                for (uint32_t t = 0; t < 4; t++) tile[tile_word(D, 16 * q + 4 * j + t, w)] = y[t];
            }
        }
        __syncthreads();
    }
    constexpr uint32_t CH = D / 16;
#pragma unroll 2
    for (uint32_t i = tid; i < (hi - lo) * CH; i += RD_THREADS) {
        const uint32_t r = i / CH, c = (i % CH) * 16;
        const uint4 w = side ? *reinterpret_cast<const uint4 *>(&tile[tile_word(D, lo + r, c / 4)])
                             : *reinterpret_cast<const uint4 *>(src + kv_k_off(D, lo + r, c));
        const uint2 a0 = decode4(w.x, s), a1 = decode4(w.y, s), a2 = decode4(w.z, s), a3 = decode4(w.w, s);
        uint4 *o = reinterpret_cast<uint4 *>(out + (uint64_t)r * a.c.kv_heads * D + c);
        o[0] = make_uint4(a0.x, a0.y, a1.x, a1.y);
        o[1] = make_uint4(a2.x, a2.y, a3.x, a3.y);
    }
}

// ---- pages ------------------------------------------------------------------
// Copy list on the device: n pairs, or *count of them; a pair with a negative
// source or destination is skipped, one out of range reported.
struct CopyArgs {
    dgt_kv_cache c;
    const int32_t *src, *dst, *count;
    uint32_t n;
    int32_t *status;
};

constexpr uint32_t CP_THREADS = 256;

// A load that is not kept in L1.  Not the read-only path: the grid may have
// started before the kernel that writes these pages has ended, and writes to
// the same pool itself.
__device__ __forceinline__ uint4 ld_once16(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// Item: (pair, layer, keys or values), one page of one layer and side, the
// scales with it.  CTAs walk the items.
__global__ void __launch_bounds__(CP_THREADS) k_kv_copy(CopyArgs a) {
    pdl_trigger();
    pdl_wait();
    const uint32_t n = a.count ? min(a.n, (uint32_t)max(*a.count, 0)) : a.n;
    const uint64_t items = (uint64_t)n * a.c.layers * 2;
    const uint32_t quads = a.c.kv_heads * (KV_P * a.c.head_dim / 16);
    for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const uint32_t side = (uint32_t)(it & 1), layer = (uint32_t)(it / 2 % a.c.layers);
        const uint64_t i = it / 2 / a.c.layers;
        const int32_t s = a.src[i], d = a.dst[i];
        if (s < 0 && d < 0) continue;
        if (s < 0 || d < 0 || (uint32_t)s >= a.c.pages || (uint32_t)d >= a.c.pages) {
            if (threadIdx.x == 0) set_status(a.status, DGT_ERR_ARG);
            continue;
        }
        if (s == d) continue;
        const uint64_t bs = kv_block(a.c, layer, (uint32_t)s, 0), bd = kv_block(a.c, layer, (uint32_t)d, 0);
        uint8_t *base = side ? a.c.v : a.c.k;
        float *sc = side ? a.c.v_scale : a.c.k_scale;
        const uint4 *from = reinterpret_cast<const uint4 *>(base + bs * (KV_P * a.c.head_dim));
        uint4 *to = reinterpret_cast<uint4 *>(base + bd * (KV_P * a.c.head_dim));
        // eight loads in flight (a page of one layer and side is a multiple of 4 KB)
        constexpr uint32_t UN = 8;
        uint32_t q = threadIdx.x;
        for (; q + (UN - 1) * CP_THREADS < quads; q += UN * CP_THREADS) {
            uint4 v[UN];
#pragma unroll
            for (uint32_t i = 0; i < UN; i++) v[i] = ld_once16(from + q + i * CP_THREADS);
#pragma unroll
            for (uint32_t i = 0; i < UN; i++) to[q + i * CP_THREADS] = v[i];
        }
        for (; q < quads; q += CP_THREADS) to[q] = from[q];
        for (uint32_t h = threadIdx.x; h < a.c.kv_heads; h += CP_THREADS) sc[bd + h] = sc[bs + h];
    }
}

// One CTA per pair: the target's table row becomes the source's, every page
// of it one reference more.
__global__ void __launch_bounds__(256) k_kv_fork(dgt_kv_cache c, const int32_t *from, const int32_t *to,
                                                int32_t *status) {
    pdl_trigger();
    pdl_wait();
    const int32_t f = from[blockIdx.x], t = to[blockIdx.x];
    if (f < 0 || t < 0 || (uint32_t)f >= c.max_seqs || (uint32_t)t >= c.max_seqs || f == t) {
        if (threadIdx.x == 0) set_status(status, DGT_ERR_ARG);
        return;
    }
    int32_t *dst = c.table + (uint64_t)t * c.max_pages;
    const int32_t *src = c.table + (uint64_t)f * c.max_pages;
    if (dst[0] >= 0 || c.lens[t] != 0) {
        if (threadIdx.x == 0) set_status(status, DGT_ERR_ARG);
        return;
    }
    __syncthreads();   // every thread has looked before any writes
    for (uint32_t i = threadIdx.x; i < c.max_pages; i += blockDim.x) {
        const int32_t p = src[i];
        if (p >= 0 && (uint32_t)p < c.pages) {
            dst[i] = p;
            atomicAdd(&c.refs[p], 1);
        }
    }
    if (threadIdx.x == 0) c.lens[t] = c.lens[f];
}

// One CTA per sequence.
__global__ void __launch_bounds__(256) k_kv_free(dgt_kv_cache c, const int32_t *seqs, int32_t *status) {
    pdl_trigger();
    pdl_wait();
    const int32_t s = seqs[blockIdx.x];
    if (s < 0 || (uint32_t)s >= c.max_seqs) {
        if (threadIdx.x == 0) set_status(status, DGT_ERR_ARG);
        return;
    }
    int32_t *row = c.table + (uint64_t)s * c.max_pages;
    for (uint32_t i = threadIdx.x; i < c.max_pages; i += blockDim.x) {
        // an exchange: a sequence that the list holds twice gives each page up once
        if (row[i] < 0) continue;
        const int32_t p = atomicExch(&row[i], -1);
        if (p >= 0 && (uint32_t)p < c.pages) atomicSub(&c.refs[p], 1);
    }
    if (threadIdx.x == 0) c.lens[s] = 0;
}

constexpr uint32_t PG_THREADS = 1024;
constexpr uint32_t PG_MAX = 1024;   // sequences of one reserve call

// Exclusive prefix sum over the CTA (PG_THREADS threads); *total its sum.
__device__ __forceinline__ uint32_t cta_excl_scan(uint32_t v, uint32_t *total, uint32_t *part) {
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t wsum;
    const uint32_t x = warp_excl_scan(v, &wsum);
    if (lane == 0) part[warp] = wsum;
    __syncthreads();
    uint32_t all;
    const uint32_t before = warp_excl_scan(part[lane], &all);
    const uint32_t base = __shfl_sync(DGT_FULL, before, warp);
    __syncthreads();
    *total = all;
    return base + x;
}

struct ReserveArgs {
    dgt_kv_cache c;
    const int32_t *seqs, *count;
    uint32_t n;
    int32_t *start, *src, *dst, *free, *old;   // workspace: copy pairs [n], free pages found and what they replace
    int32_t *status;
};

// Copy on write in list order: of the listed sequences that share a partly
// filled last page, the k-th (from 0) finds refs - k references left, and
// copies it when that is more than its own.  Pages that a row lists past its
// length (it was lowered) and that no other row does serve again; the others
// are replaced like empty entries, and lose this row's reference.
__global__ void __launch_bounds__(PG_THREADS) k_kv_reserve(ReserveArgs a) {
    __shared__ int32_t seq_s[PG_MAX], last_s[PG_MAX];
    __shared__ uint32_t part[32];
    pdl_trigger();
    pdl_wait();
    const uint32_t t = threadIdx.x;
    const dgt_kv_cache &c = a.c;
    int32_t seq = -1, len = 0, cnt = 0, last = -1;
    uint32_t have = 0, add = 0, need = 0, bad = 0, full = 0, listed = 0;   // listed: pages past the length
    if (t < a.n) {
        seq = a.seqs[t];
        cnt = a.count[t];
        if (seq < 0 || (uint32_t)seq >= c.max_seqs || cnt < 0) {
            bad = 1;
            seq = -1;
        } else {
            len = c.lens[seq];
            if (len < 0 || (uint64_t)len > (uint64_t)c.max_pages * KV_P) {
                bad = 1;
            } else {
                have = ((uint32_t)len + KV_P - 1) / KV_P;
                const uint64_t want = ((uint64_t)len + (uint32_t)cnt + KV_P - 1) / KV_P;
                if (want > c.max_pages) full = 1;
                else need = add = (uint32_t)want - have;
                const int32_t *row = c.table + (uint64_t)seq * c.max_pages;
                const int32_t end = have ? row[have - 1] : -1;   // on its way with the entries behind it
                for (uint32_t i = 0; i < add; i++) {
                    const int32_t p = row[have + i];
                    if (p < 0) break;   // a row's pages stand together
                    listed = 1;
                    if ((uint32_t)p >= c.pages) bad = 1;
                    else if (c.refs[p] == 1) need--;
                }
                if (have) {
                    if (end < 0 || (uint32_t)end >= c.pages) bad = 1;
                    else if (((uint32_t)len & (KV_P - 1)) && cnt > 0) last = end;
                }
            }
        }
    }
    if (t < PG_MAX) {
        seq_s[t] = seq;
        last_s[t] = last;
    }
    const bool anylisted = __syncthreads_or(listed);
    uint32_t rank = 0;
    if (t < a.n)
        for (uint32_t j = 0; j < t; j++) {
            if (seq >= 0 && seq_s[j] == seq) bad = 1;
            rank += last >= 0 && last_s[j] == last;
        }
    const uint32_t copy = last >= 0 && c.refs[last] - (int32_t)rank > 1 ? 1u : 0u;
    const uint32_t anybad = __syncthreads_or(bad);
    const uint32_t anyfull = __syncthreads_or(full);
    uint32_t total;
    const uint32_t base = cta_excl_scan(bad || full ? 0 : need + copy, &total, part);
    // the lowest free pages, in order
    uint32_t found = 0;
    if (!anybad && !anyfull && total <= c.pages) {
        for (uint64_t p0 = 0; p0 < c.pages && found < total; p0 += PG_THREADS * 4) {
            uint32_t m = 0;
            const uint64_t p = p0 + 4 * t;
#pragma unroll
            for (uint32_t j = 0; j < 4; j++)
                if (p + j < c.pages && c.refs[p + j] == 0) m |= 1u << j;
            uint32_t here;
            uint32_t at = found + cta_excl_scan(__popc(m), &here, part);
#pragma unroll
            for (uint32_t j = 0; j < 4; j++)
                if ((m >> j) & 1u) {
                    if (at < total) a.free[at] = (int32_t)(p + j);
                    at++;
                }
            found += here;
        }
    }
    __syncthreads();
    const bool ok = !anybad && !anyfull && found >= total;
    if (t < a.n) {
        a.src[t] = a.dst[t] = -1;
        if (!ok) {
            a.start[t] = -1;
        } else {
            a.start[t] = len;
            c.lens[seq] = len + cnt;
            int32_t *row = c.table + (uint64_t)seq * c.max_pages;
            uint32_t at = base;
            if (__builtin_expect(anylisted, 0)) {
                // references change below, when every row has been read
                if (copy) {
                    const int32_t p = a.free[at];
                    a.src[t] = last;
                    a.dst[t] = p;
                    row[have - 1] = p;
                    a.old[at++] = last;
                }
                bool more = true;
                for (uint32_t i = 0; i < add; i++) {
                    const int32_t p = more ? row[have + i] : -1, r = p < 0 ? 0 : c.refs[p];
                    more = p >= 0;
                    if (r == 1) continue;
                    row[have + i] = a.free[at];
                    a.old[at++] = r > 1 ? p : -1;
                }
                add = 0;
            } else if (copy) {
                const int32_t p = a.free[at++];
                a.src[t] = last;
                a.dst[t] = p;
                row[have - 1] = p;
                atomicSub(&c.refs[last], 1);
                c.refs[p] = 1;
            }
            for (uint32_t i = 0; i < add; i++) {
                const int32_t p = a.free[at + i];
                row[have + i] = p;
                c.refs[p] = 1;
            }
        }
    }
    if (__builtin_expect(ok && anylisted, 0)) {
        __syncthreads();
        for (uint32_t k = t; k < total; k += PG_THREADS) {
            c.refs[a.free[k]] = 1;
            if (a.old[k] >= 0) atomicSub(&c.refs[a.old[k]], 1);
        }
    }
    if (!ok && t == 0) set_status(a.status, anybad ? DGT_ERR_ARG : DGT_ERR_FULL);
}

struct CompactArgs {
    dgt_kv_cache c;
    int32_t *src, *dst, *count, *map;   // workspace: moves, how many, page -> new page
    int32_t *live;
};

// Counts the used pages, pairs the k-th used page past that count with the
// k-th free page below it, and moves refs.
__global__ void __launch_bounds__(PG_THREADS) k_kv_compact_plan(CompactArgs a) {
    __shared__ uint32_t part[32];
    pdl_trigger();
    pdl_wait();
    const dgt_kv_cache &c = a.c;
    const uint32_t t = threadIdx.x;
    uint32_t mine = 0, live;
    for (uint64_t p = t; p < c.pages; p += PG_THREADS) mine += c.refs[p] > 0;
    cta_excl_scan(mine, &live, part);
    uint32_t holes = 0, movers = 0;
    for (uint64_t p0 = 0; p0 < c.pages; p0 += PG_THREADS) {
        const uint64_t p = p0 + t;
        const bool used = p < c.pages && c.refs[p] > 0;
        const uint32_t hole = p < live && !used, mover = p >= live && used;
        uint32_t nh, nm;
        const uint32_t ih = holes + cta_excl_scan(hole, &nh, part);
        const uint32_t im = movers + cta_excl_scan(mover, &nm, part);
        if (hole) a.dst[ih] = (int32_t)p;
        if (mover) a.src[im] = (int32_t)p;
        holes += nh;
        movers += nm;
    }
    __syncthreads();
    for (uint64_t p = t; p < c.pages; p += PG_THREADS) a.map[p] = (int32_t)p;
    __syncthreads();
    for (uint32_t i = t; i < movers; i += PG_THREADS) {
        const int32_t s = a.src[i], d = a.dst[i];
        a.map[s] = d;
        c.refs[d] = c.refs[s];
        c.refs[s] = 0;
    }
    if (t == 0) {
        *a.count = (int32_t)movers;
        if (a.live) *a.live = (int32_t)live;
    }
}

__global__ void __launch_bounds__(256) k_kv_compact_tables(dgt_kv_cache c, const int32_t *map) {
    pdl_trigger();
    pdl_wait();
    const uint64_t n = (uint64_t)c.max_seqs * c.max_pages;
    for (uint64_t i = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (uint64_t)gridDim.x * blockDim.x) {
        const int32_t p = c.table[i];
        if (p >= 0 && (uint32_t)p < c.pages) c.table[i] = map[p];
    }
}

static int launched(cudaError_t e) { return e == cudaSuccess ? DGT_OK : DGT_ERR_CUDA; }

static int copy_launch(const CopyArgs &a, cudaStream_t st) {
    DeviceInfo di;
    if (device_info(&di) != DGT_OK) return DGT_ERR_CUDA;
    const uint64_t items = (uint64_t)a.n * a.c.layers * 2, most = (uint64_t)di.sms * 8;
    return launched(launch_pdl(k_kv_copy, dim3((unsigned)(items < most ? items : most)), dim3(CP_THREADS), 0, st, a));
}

}  // namespace dgt

using namespace dgt;

extern "C" int dgt_kv_append(const dgt_kv_cache *cache, uint32_t layer, const dgt_heads *k, const dgt_heads *v,
                             uint64_t tokens, const int32_t *d_seqs, const int32_t *d_start, const int32_t *d_cu,
                             uint32_t batch, int32_t *d_status, void *stream) {
    int rc = kv_check(cache);
    if (rc != DGT_OK) return rc;
    if (layer >= cache->layers) return DGT_ERR_ARG;
    if ((rc = batch_check(tokens, batch, d_cu)) != DGT_OK) return rc;
    if (tokens == 0 || batch == 0) return DGT_OK;
    if (!d_seqs || !d_start) return DGT_ERR_ARG;
    if ((rc = heads_check(k, cache->kv_heads)) != DGT_OK || (rc = heads_check(v, cache->kv_heads)) != DGT_OK) return rc;
    AppendArgs a{*cache, layer, batch, tokens, {*k, *v}, d_seqs, d_start, d_cu, d_status};
    const unsigned items = d_cu ? (unsigned)(tokens / KV_P + 2ull * batch) : batch;
    const dim3 grid(items, cache->kv_heads, 2);
    auto fn = cache->head_dim == 64 ? k_kv_append<64> : cache->head_dim == 128 ? k_kv_append<128> : k_kv_append<256>;
    return launched(launch_pdl(fn, grid, dim3(AP_THREADS), 0, (cudaStream_t)stream, a));
}

extern "C" int dgt_kv_read(const dgt_kv_cache *cache, int32_t layer, const int32_t *d_seqs, const int32_t *d_first,
                           const int32_t *d_cu, uint32_t batch, uint64_t tokens, uint16_t *d_k, uint16_t *d_v,
                           int32_t *d_status, void *stream) {
    int rc = kv_check(cache);
    if (rc != DGT_OK) return rc;
    if (layer < -1 || (layer >= 0 && (uint32_t)layer >= cache->layers)) return DGT_ERR_ARG;
    if ((rc = batch_check(tokens, batch, d_cu)) != DGT_OK) return rc;
    if (tokens == 0 || batch == 0 || (!d_k && !d_v)) return DGT_OK;
    if (!d_seqs || !d_first || !aligned16(d_k) || !aligned16(d_v)) return DGT_ERR_ARG;
    const uint32_t layers = layer < 0 ? cache->layers : 1;
    if (layers > 32767) return DGT_ERR_SHAPE;
    ReadArgs a{*cache, layer < 0 ? 0u : (uint32_t)layer, layers, batch, tokens, d_seqs, d_first, d_cu, {d_k, d_v},
               d_status};
    const unsigned items = d_cu ? (unsigned)(tokens / KV_P + 2ull * batch) : batch;
    const dim3 grid(items, cache->kv_heads, 2 * layers);
    auto fn = cache->head_dim == 64 ? k_kv_read<64> : cache->head_dim == 128 ? k_kv_read<128> : k_kv_read<256>;
    return launched(launch_pdl(fn, grid, dim3(RD_THREADS), 0, (cudaStream_t)stream, a));
}

extern "C" int dgt_kv_copy_pages(const dgt_kv_cache *cache, const int32_t *d_src, const int32_t *d_dst, uint32_t n,
                                 int32_t *d_status, void *stream) {
    const int rc = kv_check(cache);
    if (rc != DGT_OK) return rc;
    if (n == 0) return DGT_OK;
    if (!d_src || !d_dst) return DGT_ERR_ARG;
    return copy_launch(CopyArgs{*cache, d_src, d_dst, nullptr, n, d_status}, (cudaStream_t)stream);
}

extern "C" int dgt_kv_fork(const dgt_kv_cache *cache, const int32_t *d_from, const int32_t *d_to, uint32_t n,
                           int32_t *d_status, void *stream) {
    const int rc = kv_check(cache);
    if (rc != DGT_OK) return rc;
    if (n == 0) return DGT_OK;
    if (!d_from || !d_to) return DGT_ERR_ARG;
    return launched(launch_pdl(k_kv_fork, dim3(n), dim3(256), 0, (cudaStream_t)stream, *cache, d_from, d_to, d_status));
}

extern "C" int dgt_kv_free(const dgt_kv_cache *cache, const int32_t *d_seqs, uint32_t n, int32_t *d_status,
                           void *stream) {
    const int rc = kv_check(cache);
    if (rc != DGT_OK) return rc;
    if (n == 0) return DGT_OK;
    if (!d_seqs) return DGT_ERR_ARG;
    return launched(launch_pdl(k_kv_free, dim3(n), dim3(256), 0, (cudaStream_t)stream, *cache, d_seqs, d_status));
}

// Workspace: a reserve's copy pairs, free list and what it replaces, or a
// compaction's moves, map and count.
extern "C" size_t dgt_kv_pages_workspace_bytes(const dgt_kv_cache *cache) {
    if (!cache) return 0;
    const size_t reserve = 2 * (size_t)PG_MAX + 2 * (size_t)cache->pages, compact = 3 * (size_t)cache->pages + 1;
    return 4 * (reserve > compact ? reserve : compact);
}

extern "C" int dgt_kv_reserve(const dgt_kv_cache *cache, const int32_t *d_seqs, const int32_t *d_count, uint32_t n,
                              int32_t *d_start, void *d_ws, size_t ws_bytes, int32_t *d_status, void *stream) {
    int rc = kv_check(cache);
    if (rc != DGT_OK) return rc;
    if (n > PG_MAX) return DGT_ERR_SHAPE;
    if (n == 0) return DGT_OK;
    if (!d_seqs || !d_count || !d_start || !d_ws || ws_bytes < dgt_kv_pages_workspace_bytes(cache)) return DGT_ERR_ARG;
    int32_t *w = (int32_t *)d_ws;
    const ReserveArgs a{*cache, d_seqs, d_count, n, d_start, w, w + PG_MAX, w + 2 * PG_MAX,
                        w + 2 * PG_MAX + cache->pages, d_status};
    rc = launched(launch_pdl(k_kv_reserve, dim3(1), dim3(PG_THREADS), 0, (cudaStream_t)stream, a));
    if (rc != DGT_OK) return rc;
    return copy_launch(CopyArgs{*cache, a.src, a.dst, nullptr, n, d_status}, (cudaStream_t)stream);
}

extern "C" int dgt_kv_compact(const dgt_kv_cache *cache, int32_t *d_live, void *d_ws, size_t ws_bytes,
                              int32_t *d_status, void *stream) {
    int rc = kv_check(cache);
    if (rc != DGT_OK) return rc;
    if (!d_ws || ws_bytes < dgt_kv_pages_workspace_bytes(cache)) return DGT_ERR_ARG;
    int32_t *w = (int32_t *)d_ws;
    const size_t P = cache->pages;
    const CompactArgs a{*cache, w, w + P, w + 3 * P, w + 2 * P, d_live};
    DeviceInfo di;
    if (device_info(&di) != DGT_OK) return DGT_ERR_CUDA;
    rc = launched(launch_pdl(k_kv_compact_plan, dim3(1), dim3(PG_THREADS), 0, (cudaStream_t)stream, a));
    if (rc != DGT_OK) return rc;
    rc = copy_launch(CopyArgs{*cache, a.src, a.dst, a.count, (uint32_t)(P / 2 + 1), d_status}, (cudaStream_t)stream);
    if (rc != DGT_OK) return rc;
    const uint64_t entries = (uint64_t)cache->max_seqs * cache->max_pages, most = (uint64_t)di.sms * 8;
    const uint64_t g = (entries + 255) / 256;
    return launched(launch_pdl(k_kv_compact_tables, dim3((unsigned)(g < most ? g : most)), dim3(256), 0,
                               (cudaStream_t)stream, *cache, (const int32_t *)a.map));
}
