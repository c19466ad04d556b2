// dgt_attn.cuh -- what the attention kernels share: arguments, row tiles, and
// how the work is cut.
//
// Work is cut evenly over the CTAs whatever the lengths: a segment is one tile
// of query rows and one kv head, its units are the pages that the tile sees,
// and CTA c of C takes units [c U / C, (c + 1) U / C) of all U.  A segment that
// ends up in several CTAs leaves partial sums in the workspace; the CTA that
// arrives last adds them in page order, so results do not depend on timing.
// Lengths are read on the device: a captured graph follows them.
#pragma once
#include "dgt_kv.cuh"

#include "dgt_device.cuh"

namespace dgt {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr uint32_t AT_CHUNK = 64;      // row tiles described in shared memory at a time
constexpr uint32_t AT_MAX_CTAS = 320;

struct AttnArgs {
    dgt_kv_cache c;
    uint32_t layer, batch, q_heads, window, sinks, group, slots, per_entry;
    uint64_t tokens;
    dgt_heads q;
    const int32_t *seqs, *cu;
    float scale_log2;   // scale * log2(e)
    uint16_t *out;
    float *lse;
    int32_t *count;     // workspace: arrivals at the segment that CTA c begins and others end, zero between calls
    float *part;        // workspace: two partial results per CTA
    int32_t *status;
    uint32_t min_units, spin;
};

// A tile of query rows: rows [row0, row0 + rows) of its entry's flattened
// (token, head of the group) rows, at positions pos0 + row / group.
struct Slot {
    uint32_t base, np;          // first unit (of the chunk's), pages per head (0: none is seen)
    uint32_t sp, wp;            // pages seen before the window's, the window's first page
    int32_t seq, pos0;          // table row; position of the entry's first row
    uint32_t tok0, row0, rows;  // entry's first token row, tile's first flattened row, row count
    __device__ __forceinline__ uint32_t per_head() const { return np ? np : 1; }
    __device__ __forceinline__ uint32_t page_index(uint32_t i) const { return i < sp ? i : wp + i - sp; }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two fp32 to bf16, nearest with ties to even.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.0f : m; }

// Two e4m3 codes (the low or high half of w) as two fp16.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// The row tile of number `slot`, RT rows each; units 0 for an empty number.
__device__ __forceinline__ Slot slot_info(const AttnArgs &a, uint32_t slot, uint32_t RT, uint32_t *units) {
    Slot s{};
    uint32_t b, rt, n = 1;
    *units = 0;
    if (a.cu) {
        b = item_entry(a.cu, a.batch, slot, RT, 1, a.group);
        rt = slot - item_base(a.cu, b, RT, 1, a.group);
        s.tok0 = (uint32_t)a.cu[b];
        n = (uint32_t)(a.cu[b + 1] - a.cu[b]);
        if ((uint64_t)s.tok0 + n > a.tokens) {
            set_status(a.status, DGT_ERR_ARG);
            return s;
        }
    } else {
        b = slot / a.per_entry;
        rt = slot % a.per_entry;
        s.tok0 = b;
    }
    const uint64_t all = (uint64_t)n * a.group, first = (uint64_t)rt * RT;
    if (first >= all) return s;
    s.row0 = (uint32_t)first;
    s.rows = (uint32_t)min((uint64_t)RT, all - first);
    *units = a.c.kv_heads;
    s.seq = a.seqs[b];
    int32_t len = 0;
    if (s.seq < 0 || (uint32_t)s.seq >= a.c.max_seqs) {
        set_status(a.status, DGT_ERR_ARG);
        return s;
    }
    len = a.c.lens[s.seq];
    if (len < 0 || (uint64_t)len > (uint64_t)a.c.max_pages * KV_P) {
        set_status(a.status, DGT_ERR_ARG);
        len = 0;
    }
    s.pos0 = len > 0 ? len - (int32_t)n : -0x40000000;
    const int32_t pf = s.pos0 + (int32_t)(s.row0 / a.group);
    const int32_t pl = s.pos0 + (int32_t)((s.row0 + s.rows - 1) / a.group);
    if (pl < 0) return s;
    const uint32_t lo = a.window && pf >= 0 && (uint32_t)pf >= a.window ? (uint32_t)pf - a.window + 1 : 0;
    s.wp = lo / KV_P;
    s.sp = min((min(a.sinks, lo) + KV_P - 1) / KV_P, s.wp);
    s.np = s.sp + (uint32_t)pl / KV_P - s.wp + 1;
    *units = a.c.kv_heads * s.np;
    return s;
}

// Many rows (dgt_prompt.cu): the rows of its tile, and its launch.
uint32_t prompt_rows(uint32_t head_dim);
int prompt_launch(const AttnArgs &a, cudaStream_t st);

// All units of a call, summed by a CTA of WARPS warps.
template <uint32_t WARPS>
__device__ __forceinline__ uint64_t all_units(const AttnArgs &a, uint32_t RT, uint64_t *usum) {
    uint64_t sum = 0;
    uint32_t units;
    for (uint32_t s = threadIdx.x; s < a.slots; s += WARPS * 32) {
        slot_info(a, s, RT, &units);
        sum += units;
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(DGT_FULL, sum, d);
    if (lane_id() == 0) usum[threadIdx.x >> 5] = sum;
    __syncthreads();
    uint64_t U = 0;
#pragma unroll
    for (uint32_t w = 0; w < WARPS; w++) U += usum[w];
    return U;
}

// The row tiles s0 .. s0 + AT_CHUNK - 1 into shared memory; returns their units.
template <uint32_t WARPS>
__device__ __forceinline__ uint32_t describe(const AttnArgs &a, uint32_t RT, uint32_t s0, Slot *slots, uint32_t *wsum) {
    const uint32_t tid = threadIdx.x, warp = tid >> 5;
    __syncthreads();   // the tiles described before are done with
    Slot s{};
    uint32_t units = 0, before = 0;
    if (warp < AT_CHUNK / 32) {
        if (s0 + tid < a.slots) s = slot_info(a, s0 + tid, RT, &units);
        uint32_t wtot;
        before = warp_excl_scan(units, &wtot);
        if (lane_id() == 0) wsum[warp] = wtot;
    }
    __syncthreads();
    uint32_t tot = 0;
#pragma unroll
    for (uint32_t w = 0; w < AT_CHUNK / 32; w++) {
        if (w < warp) before += wsum[w];
        tot += wsum[w];
    }
    if (warp < AT_CHUNK / 32) {
        s.base = before;
        slots[tid] = s;
    }
    __syncthreads();
    return tot;
}

// A run of pages [pa, pe) of head h's segment of a described tile, beginning
// at unit u and ending by unit u1; `slot`: a tile at or before it.
struct Run {
    uint32_t u, slot, h, pa, pe;
};
__device__ __forceinline__ Run run_at(const Slot *slots, uint32_t nslots, uint32_t u, uint32_t u1, uint32_t slot) {
    Run r;
    while (slot + 1 < nslots && slots[slot + 1].base <= u) slot++;
    const Slot &s = slots[slot];
    const uint32_t n = s.per_head();
    r.u = u, r.slot = slot, r.h = (u - s.base) / n, r.pa = (u - s.base) % n;
    r.pe = min(n, r.pa + (u1 - u));
    return r;
}

// One element of a finished row: v its numerator, M, MU, L its maxima and
// denominator, weights of up to 2^wlog2.
template <uint32_t D>
__device__ __forceinline__ void write_out(const AttnArgs &a, const Slot &s, uint32_t h, uint32_t row, uint32_t d,
                                          float v, float M, float MU, float L, float wlog2) {
    const uint32_t flat = s.row0 + row;
    const uint64_t at = (uint64_t)(s.tok0 + flat / a.group) * a.q_heads + h * a.group + flat % a.group;
    const bool none = M == -INFINITY && L == 0.0f;
    a.out[at * D + d] = f32_to_bf16_rne(none ? 0.0f : v * ex2(finite_base(MU) - finite_base(M) - wlog2) / L);
    if (a.lse && d == 0) a.lse[at] = none ? -INFINITY : (M + __log2f(L)) * LN2;
}

// Rows that see nothing: out 0, lse -inf.
template <uint32_t D>
__device__ __forceinline__ void write_none(const AttnArgs &a, const Slot &s, uint32_t h, uint32_t t, uint32_t threads) {
    for (uint32_t i = t; i < s.rows * (D / 8); i += threads) {
        const uint32_t flat = s.row0 + i / (D / 8);
        const uint64_t at = (uint64_t)(s.tok0 + flat / a.group) * a.q_heads + h * a.group + flat % a.group;
        reinterpret_cast<uint4 *>(a.out + at * D)[i % (D / 8)] = make_uint4(0, 0, 0, 0);
        if (a.lse && i % (D / 8) == 0) a.lse[at] = -INFINITY;
    }
}

// The parts of a segment, left by the CTAs c0..c1 that hold its units (two
// parts of PART floats a CTA: a row's M, MU, L, then its numerators), added in
// page order by `threads` threads, this one number t, which all call it; sync
// is their barrier, sh shared memory of join_floats(RT) floats.  The parts'
// statistics come in blocks, a load per thread; then four elements at a time
// are weighted and added, several loads in flight.
constexpr uint32_t JOIN_PARTS = 32;   // parts of a block, when rows are few
__host__ __device__ constexpr uint32_t join_block(uint32_t RT) { return RT >= 128 ? 2 : JOIN_PARTS * 8 / RT; }
__host__ __device__ constexpr uint32_t join_floats(uint32_t RT) { return join_block(RT) * RT * 3 + 4 * RT; }
template <uint32_t D, uint32_t PART, uint32_t RT, typename Sync>
__device__ __forceinline__ void join_parts(const AttnArgs &a, const Slot &s, uint32_t h, uint64_t c0, uint64_t c1,
                                           uint32_t t, uint32_t threads, float wlog2, float *sh, Sync sync) {
    constexpr uint32_t KB = join_block(RT);
    float *rows = sh + KB * RT * 3;   // per row M, MU, L, then the quotient's factor
    const uint32_t parts = (uint32_t)(c1 - c0 + 1);
    // part 0 is the one that begins the segment, at the end of its CTA's work
    auto at = [&](uint32_t k, uint32_t row) { return a.part + (2 * (c0 + k) + (k == 0 ? 1 : 0)) * PART + row * (D + 4); };
    auto load_block = [&](uint32_t k0) {
        for (uint32_t i = t; i < KB * RT; i += threads) {
            const uint32_t k = k0 + i / RT, row = i % RT;
            if (k < parts && row < s.rows) {
                const float4 st = __ldcg(reinterpret_cast<const float4 *>(at(k, row)));
                sh[3 * i] = st.x, sh[3 * i + 1] = st.y, sh[3 * i + 2] = st.z;
            }
        }
        sync();
    };
    for (uint32_t k0 = 0; k0 < parts; k0 += KB) {
        if (k0) sync();
        load_block(k0);
        for (uint32_t row = t; row < s.rows; row += threads) {
            float *r = rows + 4 * row;
            float M = k0 ? r[0] : -INFINITY, MU = k0 ? r[1] : -INFINITY, L = k0 ? r[2] : 0.0f;
            const uint32_t n = min(KB, parts - k0);
            float m = M;
            for (uint32_t k = 0; k < n; k++) {
                m = fmaxf(m, sh[3 * (k * RT + row)]);
                MU = fmaxf(MU, sh[3 * (k * RT + row) + 1]);
            }
            const float b = finite_base(m);
            L *= ex2(M - b);
            for (uint32_t k = 0; k < n; k++) L += sh[3 * (k * RT + row) + 2] * ex2(sh[3 * (k * RT + row)] - b);
            r[0] = m, r[1] = MU, r[2] = L;
            if (k0 + KB >= parts) {
                const bool none = m == -INFINITY && L == 0.0f;
                r[3] = none ? 0.0f : ex2(finite_base(MU) - b - wlog2) / L;
                if (a.lse) {
                    const uint32_t flat = s.row0 + row;
                    a.lse[(uint64_t)(s.tok0 + flat / a.group) * a.q_heads + h * a.group + flat % a.group] =
                        none ? -INFINITY : (m + __log2f(L)) * LN2;
                }
            }
        }
    }
    sync();
    const bool one = parts <= KB;   // the statistics of every part are still here
    constexpr uint32_t Q = D / 4, B = RT >= 128 ? 4 : 1, UN = RT >= 128 ? 2 : 8;   // B elements of four in flight, UN parts
    const uint32_t all = s.rows * Q;
    for (uint32_t i0 = t; i0 < all; i0 += B * threads) {
        float v[B][4] = {};
#pragma unroll UN
        for (uint32_t k = 0; k < parts; k++) {
            float mu[B];
            float4 x[B];
#pragma unroll
            for (uint32_t b = 0; b < B; b++) {
                const uint32_t i = min(i0 + b * threads, all - 1), row = i / Q;
                const float *p = at(k, row);
                mu[b] = one ? sh[3 * (k * RT + row) + 1] : __ldcg(p + 1);
                x[b] = __ldcg(reinterpret_cast<const float4 *>(p + 4 + (i % Q) * 4));
            }
#pragma unroll
            for (uint32_t b = 0; b < B; b++) {
                const float f = ex2(mu[b] - finite_base(rows[4 * (min(i0 + b * threads, all - 1) / Q) + 1]));
                v[b][0] += x[b].x * f, v[b][1] += x[b].y * f, v[b][2] += x[b].z * f, v[b][3] += x[b].w * f;
            }
        }
#pragma unroll
        for (uint32_t b = 0; b < B; b++) {
            const uint32_t i = i0 + b * threads;
            if (i >= all) break;
            const float quot = rows[4 * (i / Q) + 3];
            const uint32_t flat = s.row0 + i / Q;
            const uint64_t o = (uint64_t)(s.tok0 + flat / a.group) * a.q_heads + h * a.group + flat % a.group;
            *reinterpret_cast<uint2 *>(a.out + o * D + (i % Q) * 4) =
                make_uint2(bf16x2(v[b][0] * quot, v[b][1] * quot), bf16x2(v[b][2] * quot, v[b][3] * quot));
        }
    }
    sync();   // sh and the parts are done with
}

}  // namespace dgt
