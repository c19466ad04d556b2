// dgt_beam.cu -- beam search's selection: the best n of
//   score[b] + l[b, v] - log sum_v e^l[b, v]
// over the beams b and the vocabulary v of an entry, in one pass over the
// logits.
//
// A beam's row is cut into segments, a CTA each.  A CTA keeps, beside the
// running maximum and sum of its part, the best n of its logits: within a row
// the order of the totals is that of the logits.  The first tile gives a
// threshold, the n-th of the threads' largest; what lies above it later is
// rare and goes to a list in shared memory, which is cut back to its best n,
// with a new threshold, when it is full.  The CTA that ends an entry's last
// segment joins its parts.
//
// Totals are compared in fp64.  Sums of fp32 terms are off by up to 2^-18, so
// where totals of two beams are closer than that and it matters, the entry's
// sums are made again, from terms of about 2^-35 (a table of 2^(j/32), a short
// polynomial, three floats) added as whole numbers: rows of the same logits in
// any order then have the same sum, and beams that tie are seen to.
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/dgt.h"
#include "dgt_device.cuh"
#include "dgt_launch.h"

namespace dgt {

constexpr uint32_t BM_THREADS = 256, BM_WARPS = BM_THREADS / 32;
constexpr uint32_t BM_MAX_N = 64, BM_MAX_BEAMS = 64, BM_MAX_JOIN = 2048;   // the last: beams times n
constexpr uint32_t BM_EPT = 32;                                   // elements of a tile a thread
constexpr uint32_t BM_CAP = BM_MAX_N * BM_EPT + BM_MAX_N;         // of the list
constexpr float BM_LOG2E = 1.4426950408889634f;

struct BeamArgs {
    const void *logits;
    int64_t stride;
    const float *scores;
    const uint8_t *done;
    int32_t eos;
    uint32_t batch, beams, vocab, n, segs, seg_pieces;
    int32_t *parent, *token;
    float *total;
    uint8_t *done_out;
    // workspace
    int32_t *entry_count, *row_count;   // arrivals at an entry and at a row, zero between calls
    float2 *seg_sum;                    // (maximum, sum) of a segment, and its best n
    uint64_t *seg_keys;
    double2 *row_sum;                   // (log of the sum, maximum) of a row, and its best n
    uint64_t *row_keys;
};

// A logit and its place as one whole number: greater for a greater logit, and
// for the lower of two places with one logit.
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(float v, uint32_t i) { return (uint64_t)order_of(v) << 32 | ~i; }
__device__ __forceinline__ float key_value(uint64_t k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
constexpr uint64_t BM_NONE = 0x007FFFFFull << 32 | 0xFFFFFFFFull;   // -inf at place 0: only greater keys are candidates

__device__ __forceinline__ float beam_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float beam_base(float m) { return m == -INFINITY ? 0.0f : m; }

// The row of a beam as 16-byte pieces of V elements: the first and the last
// may be cut, what lies outside reads as -inf.
template <bool F32>
struct BeamRow {
    static constexpr uint32_t V = F32 ? 4 : 8;
    const uint8_t *base;   // the first piece, aligned
    uint32_t off, vocab;   // elements of the first piece before the row
    __device__ __forceinline__ BeamRow(const void *logits, int64_t stride, uint64_t row, uint32_t vocab_) : vocab(vocab_) {
        const uintptr_t p = (uintptr_t)logits + row * stride * (F32 ? 4 : 2);
        base = (const uint8_t *)(p & ~(uintptr_t)15);
        off = (uint32_t)(p & 15) / (F32 ? 4 : 2);
    }
    __device__ __forceinline__ uint32_t pieces() const { return (vocab + off + V - 1) / V; }
    __device__ __forceinline__ bool whole(uint32_t c) const { return c * V >= off && (c + 1) * V <= off + vocab; }
    __device__ __forceinline__ uint4 edge(uint32_t c) const {
        uint32_t w[4];
#pragma unroll
        for (uint32_t i = 0; i < 4; i++) {
            if (F32) {
                const uint32_t e = c * V + i;
                w[i] = e >= off && e < off + vocab ? reinterpret_cast<const uint32_t *>(base)[e] : 0xFF800000u;
            } else {
                const uint32_t e = c * V + 2 * i;
                const uint16_t *q = reinterpret_cast<const uint16_t *>(base);
                const uint32_t lo = e >= off && e < off + vocab ? q[e] : 0xFF80u;
                const uint32_t hi = e + 1 >= off && e + 1 < off + vocab ? q[e + 1] : 0xFF80u;
                w[i] = lo | hi << 16;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ uint4 load(uint32_t c, uint32_t end) const {
        if (c >= end) return F32 ? make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u)
                                 : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
        return whole(c) ? ldg_stream16(base + (uint64_t)c * 16) : edge(c);
    }
    static __device__ __forceinline__ float value(const uint4 &x, uint32_t i) {
        const uint32_t w = F32 ? (i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w)
                               : (i / 2 == 0 ? x.x : i / 2 == 1 ? x.y : i / 2 == 2 ? x.z : x.w);
        return F32 ? __uint_as_float(w) : i & 1 ? bf16hi(w) : bf16lo(w);
    }
    // the place in the row of element i of piece c
    __device__ __forceinline__ uint32_t place(uint32_t c, uint32_t i) const { return c * V + i - off; }
};

struct BeamShared {
    union {
        uint64_t list[BM_CAP];
        struct {   // of an entry's join
            double total[BM_MAX_JOIN], lse[BM_MAX_BEAMS];
            uint32_t token[BM_MAX_JOIN];
            float logit[BM_MAX_JOIN];
            uint16_t beam[BM_MAX_JOIN];
        };
    };
    uint64_t best[BM_MAX_N];
    uint64_t top[BM_THREADS];
    float2 part[BM_WARPS];
    uint64_t thr;
    uint32_t count, last, refine;
};

// The list's best n (fewer, when it has fewer) to its beginning, in order; the
// n-th becomes the threshold.  The whole CTA.
__device__ __forceinline__ void cut_list(BeamShared &s, uint32_t n) {
    __syncthreads();
    const uint32_t count = s.count;
    for (uint32_t i = threadIdx.x; i < count; i += BM_THREADS) {
        const uint64_t k = s.list[i];
        uint32_t rank = 0;
        for (uint32_t j = 0; j < count; j++) rank += s.list[j] > k;
        if (rank < n) s.best[rank] = k;
    }
    __syncthreads();
    const uint32_t left = min(count, n);
    if (threadIdx.x < left) s.list[threadIdx.x] = s.best[threadIdx.x];
    if (threadIdx.x == 0) {
        s.count = left;
        if (left == n) s.thr = s.best[n - 1];
    }
    __syncthreads();
}

// A threshold that n keys at least reach, and n * BM_EPT at most: the n-th of
// the threads' largest (0 counts as none).
__device__ __forceinline__ uint64_t tile_threshold(BeamShared &s, uint64_t mine, uint32_t n) {
    __syncthreads();
    s.top[threadIdx.x] = mine;
    __syncthreads();
    uint32_t rank = 0;
#pragma unroll 8
    for (uint32_t j = 0; j < BM_THREADS; j++) rank += s.top[j] > mine;
    __syncthreads();
    if (threadIdx.x == 0) s.top[0] = 0;
    __syncthreads();
    if (rank == n - 1 && mine) s.top[0] = mine;
    __syncthreads();
    return s.top[0];
}

// The tile's elements from key `at` on to the list.
template <bool F32>
__device__ __forceinline__ void push(BeamShared &s, const BeamRow<F32> &row, const uint4 (&x)[BM_EPT / BeamRow<F32>::V],
                                     uint32_t c0, uint64_t at) {
    constexpr uint32_t V = BeamRow<F32>::V;
    const float v0 = key_value(at);
#pragma unroll
    for (uint32_t u = 0; u < BM_EPT / V; u++)
#pragma unroll
        for (uint32_t i = 0; i < V; i++) {
            const float v = BeamRow<F32>::value(x[u], i);
            if (!(v >= v0)) continue;
            const uint64_t k = key_of(v, row.place(c0 + u * BM_THREADS + threadIdx.x, i));
            if (k < at || k <= BM_NONE) continue;
            const uint32_t p = atomicAdd(&s.count, 1u);
            if (p < BM_CAP) s.list[p] = k;
        }
}

template <bool F32>
__device__ __forceinline__ float2 scan_segment(const BeamArgs &a, BeamShared &s, uint64_t r, uint32_t seg) {
    constexpr uint32_t V = BeamRow<F32>::V, U = BM_EPT / V;
    const BeamRow<F32> row(a.logits, a.stride, r, a.vocab);
    const uint32_t c_begin = seg * a.seg_pieces, c_end = min(c_begin + a.seg_pieces, row.pieces());
    float m = -INFINITY, sum = 0.0f, low = 0.0f;   // sum + low
    if (threadIdx.x == 0) s.count = 0, s.thr = 0;
    bool first = true;
    for (uint32_t c0 = c_begin; c0 < c_end; c0 += BM_THREADS * U) {
        uint4 x[U];
#pragma unroll
        for (uint32_t u = 0; u < U; u++) x[u] = row.load(c0 + u * BM_THREADS + threadIdx.x, c_end);
        float top = -INFINITY;
#pragma unroll
        for (uint32_t u = 0; u < U; u++)
#pragma unroll
            for (uint32_t i = 0; i < V; i++) top = fmaxf(top, BeamRow<F32>::value(x[u], i));
        const float mn = fmaxf(m, top), b = beam_base(mn);
        float tile = 0.0f;
#pragma unroll
        for (uint32_t u = 0; u < U; u++)
#pragma unroll
            for (uint32_t i = 0; i < V; i++) tile += beam_ex2((BeamRow<F32>::value(x[u], i) - b) * BM_LOG2E);
        const float f = m == mn ? 1.0f : beam_ex2((m - b) * BM_LOG2E);
        sum *= f, low *= f;
        m = mn;
        // sum + low + tile, the error of the sum kept
        const float t = sum + tile, back = t - sum;
        low += (sum - (t - back)) + (tile - back);
        sum = t;

        if (first) {
            // the thread's largest as a key: its lowest place
            uint64_t mine = 0;
            if (top > -INFINITY) {
#pragma unroll
                for (uint32_t u = 0; u < U; u++)
#pragma unroll
                    for (uint32_t i = 0; i < V; i++) {
                        const uint64_t k = key_of(BeamRow<F32>::value(x[u], i), row.place(c0 + u * BM_THREADS + threadIdx.x, i));
                        if (BeamRow<F32>::value(x[u], i) == top && k > mine) mine = k;
                    }
            }
            const uint64_t at = tile_threshold(s, mine, a.n);
            push<F32>(s, row, x, c0, at ? at : BM_NONE);
            cut_list(s, a.n);
            first = false;
            continue;
        }
        // later places with the threshold's logit come behind it
        const uint64_t thr = s.thr;
        const float v0 = key_value(thr);
        const bool above = thr ? top > v0 : top > -INFINITY;
        if (!__syncthreads_or(above)) continue;
        const uint32_t before = s.count;
        __syncthreads();
        if (above) push<F32>(s, row, x, c0, thr ? thr + 1 : BM_NONE);
        __syncthreads();
        if (s.count <= BM_CAP) continue;
        // too many: cut what was there, and take the best of the tile alone
        __syncthreads();
        if (threadIdx.x == 0) s.count = before;
        cut_list(s, a.n);
        uint64_t mine = 0;
#pragma unroll
        for (uint32_t u = 0; u < U; u++)
#pragma unroll
            for (uint32_t i = 0; i < V; i++) {
                const uint64_t k = key_of(BeamRow<F32>::value(x[u], i), row.place(c0 + u * BM_THREADS + threadIdx.x, i));
                if (BeamRow<F32>::value(x[u], i) == top && k > mine && k > BM_NONE) mine = k;
            }
        const uint64_t at = tile_threshold(s, mine, a.n);
        const uint64_t from = at > s.thr ? at : s.thr + 1;
        push<F32>(s, row, x, c0, from > BM_NONE ? from : BM_NONE);
        cut_list(s, a.n);
    }
    cut_list(s, a.n);

    // the threads' maxima and sums to one
    float mm = m;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(DGT_FULL, mm, d));
    float ss = (sum + low) * beam_ex2((m - beam_base(mm)) * BM_LOG2E);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) ss += __shfl_xor_sync(DGT_FULL, ss, d);
    if (lane_id() == 0) s.part[threadIdx.x >> 5] = make_float2(mm, ss);
    __syncthreads();
    float M = -INFINITY, S = 0.0f;
    for (uint32_t w = 0; w < BM_WARPS; w++) M = fmaxf(M, s.part[w].x);
    for (uint32_t w = 0; w < BM_WARPS; w++) S += s.part[w].y * beam_ex2((s.part[w].x - beam_base(M)) * BM_LOG2E);
    return make_float2(M, S);
}

// This CTA's arrival at a counter: true for the last of `all`, which then sees
// what the others stored before theirs.  The whole CTA.
__device__ __forceinline__ bool arrive(BeamShared &s, int32_t *count, uint32_t all) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        int32_t was;
        asm volatile("atom.add.acq_rel.gpu.s32 %0, [%1], 1;" : "=r"(was) : "l"(count) : "memory");
        s.last = was == (int32_t)all - 1;
        if (s.last) *count = 0;
    }
    __syncthreads();
    const bool last = s.last;
    __syncthreads();
    if (last) __threadfence();
    return last;
}

// The segments of a row to one: its best n to s.list, its sum.
__device__ __forceinline__ void join_row(const BeamArgs &a, BeamShared &s, uint64_t r, float &M, double &S) {
    if (threadIdx.x == 0) s.count = 0;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < a.segs * a.n; i += BM_THREADS) {
        const uint64_t k = __ldcg(&a.seg_keys[r * a.segs * a.n + i]);
        if (k) s.list[atomicAdd(&s.count, 1u)] = k;
    }
    cut_list(s, a.n);
    M = -INFINITY;
    for (uint32_t g = lane_id(); g < a.segs; g += 32) M = fmaxf(M, __ldcg(&a.seg_sum[r * a.segs + g]).x);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) M = fmaxf(M, __shfl_xor_sync(DGT_FULL, M, d));
    S = 0.0;
    for (uint32_t g = lane_id(); g < a.segs; g += 32) {
        const float2 p = __ldcg(&a.seg_sum[r * a.segs + g]);
        S += (double)(p.y * beam_ex2((p.x - beam_base(M)) * BM_LOG2E));
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) S += __shfl_xor_sync(DGT_FULL, S, d);
}

// log sum e^l of a row: e^(l - M) = 2^(k / 32) e^r with the table of 2^(j / 32)
// in two floats and e^r by its series (after P. T. P. Tang's table-driven
// exponential, 1989), in units of 2^-62.
template <bool F32>
__device__ __forceinline__ double sum_again(const BeamArgs &a, uint64_t r, float M, uint64_t (*scratch)[2],
                                            const float2 *table) {
    const BeamRow<F32> row(a.logits, a.stride, r, a.vocab);
    uint64_t low = 0, high = 0;   // high 2^64 + low
    auto plus = [&](uint64_t l, uint64_t h) {
        low += l;
        high += h + (low < l);
    };
    const uint32_t end = row.pieces();
    for (uint32_t c = threadIdx.x; c < end; c += BM_THREADS) {
        const uint4 x = row.load(c, end);
#pragma unroll
        for (uint32_t i = 0; i < BeamRow<F32>::V; i++) {
            const float v = BeamRow<F32>::value(x, i);
            const float d = v - M, back = d - v, e = (v - (d - back)) - (M + back);   // d + e = v - M
            if (!(d > -60.0f)) continue;   // below 2^-86 of the largest
            const float k = rintf(d * 46.16624130844683f);   // 32 / ln 2
            // ln 2 / 32 in two parts, the first of nine bits: its product with k is exact
            const float q0 = fmaf(k, -0.02166748046875f, d), q1 = k * 6.631076251709805e-06f;
            const float q = q0 + q1, ql = (q1 - (q - q0)) + e;
            const int ki = (int)k;
            const float2 t = table[ki & 31];
            // t.x (1 + q + ql + q^2 (1/2 + q/6 + q^2/24)) + t.y (1 + q)
            const float p = t.x * q, pl = fmaf(t.x, q, -p);
            const float rest = fmaf(t.x, fmaf(q * q, fmaf(q, fmaf(q, 1.0f / 24.0f, 1.0f / 6.0f), 0.5f), ql), fmaf(t.y, q, t.y) + pl);
            const float unit = __uint_as_float((uint32_t)((ki >> 5) + 62 + 127) << 23);
            const int64_t term = __float2ll_rn(t.x * unit) + __float2ll_rn(p * unit) + __float2ll_rn(rest * unit);
            plus((uint64_t)term, 0);
        }
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        const uint64_t l = __shfl_xor_sync(DGT_FULL, low, d), h = __shfl_xor_sync(DGT_FULL, high, d);
        plus(l, h);
    }
    __syncthreads();
    if (lane_id() == 0) scratch[threadIdx.x >> 5][0] = low, scratch[threadIdx.x >> 5][1] = high;
    __syncthreads();
    low = high = 0;
    for (uint32_t w = 0; w < BM_WARPS; w++) plus(scratch[w][0], scratch[w][1]);
    return (double)M + log((double)high * 4.0 + (double)low * 0x1p-62);
}

// A total as a whole number in the same order (0: none).
__device__ __forceinline__ uint64_t order_of(double t) {
    const uint64_t b = (uint64_t)__double_as_longlong(t + 0.0);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

template <bool F32>
__device__ __forceinline__ void join_entry(const BeamArgs &a, BeamShared &s, uint32_t entry) {
    const uint32_t tid = threadIdx.x, n = a.n;
    const uint64_t r0 = (uint64_t)entry * a.beams;
    auto reads = [&](uint32_t b) { return fabsf(a.scores[r0 + b]) < INFINITY && !(a.done && a.done[r0 + b]); };
    if (tid == 0) s.count = 0, s.refine = 0;
    // a beam without a score, without a finite sum, or at its end offers nothing of its row
    for (uint32_t b = tid; b < a.beams; b += BM_THREADS)
        s.lse[b] = reads(b) ? __ldcg(&a.row_sum[r0 + b]).x : (double)INFINITY;
    __syncthreads();
    constexpr double OFF = 1.0 / (1 << 18);
    auto candidate = [&](uint32_t c, double &t, uint32_t &b, uint32_t &v, float &x) {
        b = c / n;
        const double lse = s.lse[b];
        if (!(fabs(lse) < (double)INFINITY)) return false;
        const uint64_t k = __ldcg(&a.row_keys[r0 * n + c]);
        v = ~(uint32_t)k;
        x = key_value(k);
        t = (double)a.scores[r0 + b] + ((double)x - lse);
        return k != 0;
    };
    // the n-th of the threads' largest leaves out most of what cannot be among the best n
    uint64_t mine = 0;
    double t;
    uint32_t b, v;
    float x;
    for (uint32_t c = tid; c < a.beams * n; c += BM_THREADS)
        if (candidate(c, t, b, v, x)) mine = max(mine, order_of(t));
    mine = mine ? (mine & ~255ull) | (255u - tid) : 0;   // distinct
    const uint64_t at = tile_threshold(s, mine, n) & ~255ull;
    double from = -INFINITY;
    if (at) from = __longlong_as_double((int64_t)(at & 0x8000000000000000ull ? at ^ 0x8000000000000000ull : ~at)) - 2 * OFF;
    auto add = [&](double t, uint32_t b, uint32_t v, float x) {
        const uint32_t p = atomicAdd(&s.count, 1u);
        s.total[p] = t, s.beam[p] = (uint16_t)b, s.token[p] = v, s.logit[p] = x;
    };
    for (uint32_t c = tid; c < a.beams * n; c += BM_THREADS)
        if (candidate(c, t, b, v, x) && t >= from) add(t, b, v, x);
    // a beam at its end offers its end token at its own score
    if (a.done && tid < a.beams && a.done[r0 + tid] && fabsf(a.scores[r0 + tid]) < INFINITY)
        add((double)a.scores[r0 + tid], tid, (uint32_t)a.eos, 0.0f);
    __syncthreads();
    const uint32_t count = s.count;
    auto rank_of = [&](uint32_t i, bool &close) {
        const double ti = s.total[i];
        const uint32_t bi = s.beam[i], vi = s.token[i];
        uint32_t rank = 0;
        for (uint32_t j = 0; j < count; j++) {
            const double tj = s.total[j];
            const uint32_t bj = s.beam[j];
            rank += tj > ti || (tj == ti && (bj < bi || (bj == bi && s.token[j] < vi)));
            close |= bj != bi && fabs(tj - ti) <= 2 * OFF;
        }
        return rank;
    };
    for (uint32_t i = tid; i < count; i += BM_THREADS) {
        bool close = false;
        if (rank_of(i, close) < n && close) s.refine = 1;
    }
    __syncthreads();
    if (s.refine) {
        // totals of two beams that may be the other way round
        float2 *table = reinterpret_cast<float2 *>(s.top);
        uint64_t(*scratch)[2] = reinterpret_cast<uint64_t(*)[2]>(s.top + 32);
        if (tid < 32) {
            const double e = exp2(tid / 32.0);
            table[tid] = make_float2((float)e, (float)(e - (double)(float)e));
        }
        __syncthreads();
        for (uint32_t beam = 0; beam < a.beams; beam++) {
            if (!(fabs(s.lse[beam]) < (double)INFINITY)) continue;
            const double lse = sum_again<F32>(a, r0 + beam, (float)__ldcg(&a.row_sum[r0 + beam]).y, scratch, table);
            for (uint32_t i = tid; i < count; i += BM_THREADS)
                if (s.beam[i] == beam) s.total[i] = (double)a.scores[r0 + beam] + ((double)s.logit[i] - lse);
        }
        __syncthreads();
    }
    const uint64_t o = (uint64_t)entry * n;
    for (uint32_t i = tid; i < count; i += BM_THREADS) {
        bool close;
        const uint32_t rank = rank_of(i, close);
        if (rank >= n) continue;
        a.parent[o + rank] = (int32_t)s.beam[i];
        a.token[o + rank] = (int32_t)s.token[i];
        a.total[o + rank] = (float)s.total[i];
        if (a.done_out) a.done_out[o + rank] = a.done[r0 + s.beam[i]] || (int32_t)s.token[i] == a.eos;
    }
    for (uint32_t i = count + tid; i < n; i += BM_THREADS) {
        a.parent[o + i] = -1;
        a.token[o + i] = -1;
        a.total[o + i] = -INFINITY;
        if (a.done_out) a.done_out[o + i] = 0;
    }
}

template <bool F32>
__global__ void __launch_bounds__(BM_THREADS) k_beam_select(BeamArgs a) {
    __shared__ BeamShared s;
    pdl_trigger();
    pdl_wait();
    const uint32_t seg = blockIdx.x % a.segs;
    const uint64_t r = blockIdx.x / a.segs;
    const uint32_t entry = (uint32_t)(r / a.beams);
    if (fabsf(a.scores[r]) < INFINITY && !(a.done && a.done[r])) {
        const float2 p = scan_segment<F32>(a, s, r, seg);
        float M = p.x;
        double S = p.y;
        if (a.segs > 1) {
            const uint64_t at = r * a.segs + seg;
            if (threadIdx.x == 0) a.seg_sum[at] = p;
            for (uint32_t i = threadIdx.x; i < a.n; i += BM_THREADS) a.seg_keys[at * a.n + i] = i < s.count ? s.list[i] : 0ull;
            if (!arrive(s, &a.row_count[r], a.segs)) return;
            join_row(a, s, r, M, S);
        }
        if (threadIdx.x == 0) a.row_sum[r] = make_double2((double)M + log(S), (double)M);
        for (uint32_t i = threadIdx.x; i < a.n; i += BM_THREADS) a.row_keys[r * a.n + i] = i < s.count ? s.list[i] : 0ull;
    } else if (seg) {
        return;
    }
    if (arrive(s, &a.entry_count[entry], a.beams)) join_entry<F32>(a, s, entry);
}

// Segments of a row: as many as fill the SMs with four CTAs each, of 4096
// elements at least; their best n fit the list.
static uint32_t beam_segments(uint64_t rows, uint32_t vocab, uint32_t n, uint32_t sms) {
    const uint64_t want = (4ull * sms) / rows, most = (vocab + 4095) / 4096, fit = 2048 / n;
    const uint64_t s = std::min(std::min(want, most), fit);
    return (uint32_t)std::max<uint64_t>(s, 1);
}
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Where the parts of a workspace begin; the last is its size.  The counters
// have room for every call's, so that one workspace serves all sizes: an entry
// each, and a row each where rows have segments, which are 2 BM_MAX_SMS rows
// at most.
constexpr uint32_t BM_MAX_SMS = 160;
constexpr uint32_t BM_MAX_BATCH = 65536;
struct BeamSpace {
    size_t row_count, row_sum, row_keys, seg_sum, seg_keys, bytes;
    BeamSpace(uint32_t batch, uint32_t beams, uint32_t n, uint64_t segs) {
        const uint64_t rows = (uint64_t)batch * beams;
        row_count = up256(4 * (size_t)BM_MAX_BATCH);
        row_sum = row_count + up256(4 * 2 * BM_MAX_SMS);
        row_keys = row_sum + up256(16 * rows);
        seg_sum = row_keys + up256(8 * rows * n);
        seg_keys = seg_sum + up256(8 * rows * segs);
        bytes = seg_keys + 8 * rows * segs * n;
    }
};

}  // namespace dgt

using namespace dgt;

extern "C" size_t dgt_beam_workspace_bytes(uint32_t batch, uint32_t beams, uint32_t vocab, uint32_t n) {
    if (!batch || !beams || !vocab || !n || n > BM_MAX_N) return 0;
    return BeamSpace(batch, beams, n, beam_segments((uint64_t)batch * beams, vocab, n, BM_MAX_SMS)).bytes;
}

extern "C" int dgt_beam_select(const void *d_logits, uint32_t f32, int64_t stride, const float *d_scores,
                               const uint8_t *d_done, int32_t eos, uint32_t batch, uint32_t beams, uint32_t vocab,
                               uint32_t n, int32_t *d_parent, int32_t *d_token, float *d_total, uint8_t *d_done_out,
                               void *d_ws, size_t ws_bytes, void *stream) {
    if (f32 > 1) return DGT_ERR_ARG;
    if (beams == 0 || beams > BM_MAX_BEAMS || n == 0 || n > BM_MAX_N || beams * n > BM_MAX_JOIN || vocab == 0 ||
        vocab > (1u << 24) || batch > 65536)
        return DGT_ERR_SHAPE;
    if (batch == 0) return DGT_OK;
    if (!d_logits || !d_scores || !d_parent || !d_token || !d_total || ((uintptr_t)d_logits & (f32 ? 3 : 1)) ||
        (((uintptr_t)d_scores | (uintptr_t)d_parent | (uintptr_t)d_token | (uintptr_t)d_total) & 3))
        return DGT_ERR_ARG;
    if ((d_done && (eos < 0 || (uint32_t)eos >= vocab)) || (d_done_out && !d_done)) return DGT_ERR_ARG;
    if (!d_ws || ((uintptr_t)d_ws & 255) || ws_bytes < dgt_beam_workspace_bytes(batch, beams, vocab, n)) return DGT_ERR_ARG;
    DeviceInfo di;
    if (device_info(&di) != DGT_OK) return DGT_ERR_CUDA;
    const uint64_t rows = (uint64_t)batch * beams;
    const uint32_t segs = beam_segments(rows, vocab, n, std::min((uint32_t)di.sms, BM_MAX_SMS)), V = f32 ? 4 : 8;
    const BeamSpace at(batch, beams, n, segs);
    uint8_t *w = (uint8_t *)d_ws;
    const BeamArgs a{d_logits, stride, d_scores, d_done, eos, batch, beams, vocab, n, segs,
                     ((vocab + 2 * V - 2) / V + segs - 1) / segs,   // a row that begins inside a piece may touch one more
                     d_parent, d_token, d_total, d_done_out, (int32_t *)w, (int32_t *)(w + at.row_count),
                     (float2 *)(w + at.seg_sum), (uint64_t *)(w + at.seg_keys), (double2 *)(w + at.row_sum),
                     (uint64_t *)(w + at.row_keys)};
    const dim3 grid((unsigned)(rows * segs)), block(BM_THREADS);
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = f32 ? launch_pdl(k_beam_select<true>, grid, block, 0, st, a)
                              : launch_pdl(k_beam_select<false>, grid, block, 0, st, a);
    return e == cudaSuccess ? DGT_OK : DGT_ERR_CUDA;
}
