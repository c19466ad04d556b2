// dgt_attn.cuh -- what the attention kernels share: arguments, row tiles, and
// how the work is cut.
//
// Work is cut evenly over the CTAs whatever the lengths.  A segment is one tile
// of query rows and one kv head, its units are the pages that the tile sees and
// `end` more, which come first, for what a segment costs besides its pages.
// Where that comes out even enough, every segment is cut into equal parts, a
// CTA for each; otherwise CTA c of C takes units [c U / C, (c + 1) U / C) of
// all U, a cut close to a segment's border moved there.  A segment that ends up
// in several CTAs leaves partial sums in the workspace; the CTA that arrives
// last adds them in page order, so results do not depend on timing.  Lengths
// are read on the device: a captured graph follows them.
#pragma once
#include <algorithm>

#include "dgt_kv.cuh"

#include "dgt_device.cuh"

namespace dgt {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr uint32_t AT_CHUNK = 64;      // row tiles described in shared memory at a time
constexpr uint32_t AT_MAX_SMS = 160;   // a workspace has room for so many

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
    uint32_t min_units, slack;   // pages of a part at least; pages that parts may be above an even share
    uint32_t end;                // what a segment costs besides its pages, in pages
    float join;                  // what a part costs the join, in pages
    uint32_t spin;
};

// A tile of query rows: rows [row0, row0 + rows) of its entry's flattened
// (token, head of the group) rows, at positions pos0 + row / group.
struct Slot {
    uint32_t base, np;          // first unit (of the chunk's), pages per head (0: none is seen, counted as one)
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
    *units = a.c.kv_heads * (1 + a.end);
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
    *units = a.c.kv_heads * (s.np + a.end);
    return s;
}

// Many rows (dgt_prompt.cu): the rows of its tile, and its launch.
uint32_t prompt_rows(uint32_t head_dim);
int prompt_launch(const AttnArgs &a, cudaStream_t st);

// Units and row tiles that hold rows, counted together.
struct Units {
    uint64_t packed;   // units below, tiles from bit 40 on
    __device__ __forceinline__ uint64_t units() const { return packed & ((1ull << 40) - 1); }
    __device__ __forceinline__ uint32_t tiles() const { return (uint32_t)(packed >> 40); }
};

// All of a call's, summed by a CTA of WARPS warps.
template <uint32_t WARPS>
__device__ __forceinline__ Units all_units(const AttnArgs &a, uint32_t RT, uint64_t *usum) {
    uint64_t sum = 0;
    uint32_t units;
    for (uint32_t s = threadIdx.x; s < a.slots; s += WARPS * 32) {
        slot_info(a, s, RT, &units);
        if (units) sum += units + (1ull << 40);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(DGT_FULL, sum, d);
    if (lane_id() == 0) usum[threadIdx.x >> 5] = sum;
    __syncthreads();
    Units u{0};
#pragma unroll
    for (uint32_t w = 0; w < WARPS; w++) u.packed += usum[w];
    return u;
}

// The row tiles s0 .. s0 + AT_CHUNK - 1 into shared memory; returns their units.
template <uint32_t WARPS>
__device__ __forceinline__ Units describe(const AttnArgs &a, uint32_t RT, uint32_t s0, Slot *slots, uint64_t *usum) {
    const uint32_t tid = threadIdx.x, warp = tid >> 5;
    __syncthreads();   // the tiles described before are done with
    Slot s{};
    uint32_t units = 0, before = 0;
    if (warp < AT_CHUNK / 32) {
        if (s0 + tid < a.slots) s = slot_info(a, s0 + tid, RT, &units);
        uint32_t wtot;
        before = warp_excl_scan(units, &wtot);
        const uint32_t tiles = __popc(__ballot_sync(DGT_FULL, units != 0));
        if (lane_id() == 0) usum[warp] = wtot + ((uint64_t)tiles << 40);
    }
    __syncthreads();
    Units u{0};
#pragma unroll
    for (uint32_t w = 0; w < AT_CHUNK / 32; w++) {
        if (w < warp) before += (uint32_t)usum[w];
        u.packed += usum[w];
    }
    if (warp < AT_CHUNK / 32) {
        s.base = before;
        slots[tid] = s;
    }
    __syncthreads();
    return u;
}

// A run of pages [pa, pe) of head h's segment of a described tile: `units`
// units from u on, ending by unit u1.
struct Run {
    uint32_t u, units, slot, h, pa, pe;
};
__device__ __forceinline__ Run run_at(const Slot *slots, uint32_t nslots, uint32_t end, uint32_t u, uint32_t u1) {
    uint32_t lo = 0, hi = nslots;   // the last tile that begins at or before u
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if (slots[mid].base <= u) lo = mid;
        else hi = mid;
    }
    Run r;
    const Slot &s = slots[lo];
    const uint32_t n = s.per_head() + end, from = (u - s.base) % n, to = min(n, from + (u1 - u));
    r.u = u, r.units = to - from, r.slot = lo, r.h = (u - s.base) / n;
    r.pa = from > end ? from - end : 0;
    r.pe = to > end ? to - end : 0;
    return r;
}

// Where the CTAs' shares begin.
struct Cuts {
    uint64_t U;
    uint32_t C, tol, end;     // CTA c at unit c U / C, or at a segment's border within tol of that
    bool parts;               // or: one part of one segment, units [u0, u1) of the only chunk,
    uint32_t u0, u1, c0, c1;  // the segment's other parts with the CTAs c0..c1
    __device__ __forceinline__ uint64_t raw(uint32_t c) const {
        return U < (1u << 22) ? (uint32_t)U * c / C : U * c / C;   // C < 2^10
    }
    // unit u of a described chunk, moved to a segment's border
    __device__ __forceinline__ uint32_t snap(const Slot *slots, uint32_t nslots, uint32_t u) const {
        const Run r = run_at(slots, nslots, end, u, u + 1);
        const uint32_t n = slots[r.slot].per_head() + end, below = (u - slots[r.slot].base) % n, above = n - below;
        return below <= end + tol || above <= tol ? (below <= end + above ? u - below : u + above) : u;
    }
    // this CTA's units of the chunk [base, base + tot)
    __device__ __forceinline__ void share(const Slot *slots, uint32_t nslots, uint64_t base, uint32_t tot, uint32_t &a,
                                          uint32_t &b) const {
        if (parts) {
            a = u0, b = u1;
            return;
        }
        const uint64_t ua = raw(blockIdx.x), ub = raw(blockIdx.x + 1);
        a = ua <= base ? 0 : ua >= base + tot ? tot : snap(slots, nslots, (uint32_t)(ua - base));
        b = ub >= base + tot ? tot : ub <= base ? 0 : snap(slots, nslots, (uint32_t)(ub - base));
    }
    // the CTAs first..last that hold units of the segment [sa, sb)
    __device__ __forceinline__ void holders(uint64_t sa, uint64_t sb, uint32_t &first, uint32_t &last) const {
        if (parts) {
            first = c0, last = c1;
            return;
        }
        // cuts c with sa + end + tol < raw(c) < sb - tol stay inside
        first = (uint32_t)(((sa + end + tol + 1) * C + U - 1) / U) - 1;
        last = sb <= tol ? 0u : (uint32_t)(((sb - tol) * C + U - 1) / U) - 1;
    }
};

// How a call is cut over `grid` CTAs.  Parts: of at most T pages, T the least
// for which all parts have a CTA, min_units, and what balances a part's pages
// against the join of many parts; taken while T is no more than
// `slack` pages above an even share, because a second segment in a CTA costs a
// segment's end.  Otherwise even shares, whose cuts move by an eighth of a
// share at most, or past the units that stand for the segment's end.
__device__ __forceinline__ Cuts cut_plan(const AttnArgs &a, Units all, const Slot *slots, uint32_t grid) {
    const uint64_t U = all.units(), S = (uint64_t)all.tiles() * a.c.kv_heads, P = U - S * a.end;
    const uint32_t lane = lane_id(), heads = a.c.kv_heads;
    Cuts k;
    k.U = U;
    k.C = (uint32_t)min((uint64_t)grid, U);   // shares of one unit at least: cuts inside a segment are distinct
    k.end = a.end;
    // (U below 2^22: a segment's pages and T then are below 2^23)
    k.parts = a.slots <= AT_CHUNK && S <= grid && U && U < (1u << 22);
    auto shares = [&]() {
        k.parts = false;
        k.tol = U >= 32ull * grid ? 4u : (uint32_t)U / (8 * grid);
        return k;
    };
    if (!k.parts) return shares();
    // two tiles a lane
    uint32_t n[2], p[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint32_t s = 2 * lane + i;
        // a number without rows has no units: as far as the next begins
        const uint32_t next = s + 1 < a.slots ? slots[s + 1].base : (uint32_t)U;
        n[i] = s < a.slots && next > slots[s].base ? slots[s].per_head() : 0;
    }
    auto pieces = [](uint32_t x, uint32_t T, float inv) {   // ceil(x / T), x below 2^23
        x += T - 1;
        uint32_t q = (uint32_t)((float)x * inv);
        if (q * T > x) q--;
        if ((q + 1) * T <= x) q++;
        return q;
    };
    // T pages take T, their n / T parts' join n / T times the cost of a part: least at the root
    const uint32_t nmax = __reduce_max_sync(DGT_FULL, max(n[0], n[1]));
    const uint32_t T0 = max(max(((uint32_t)P + grid - 1) / grid, a.min_units), (uint32_t)sqrtf(a.join * (float)nmax));
    // rolled, and left at the first T that fits: the code runs once a call, from a cold instruction cache
    uint32_t i = 0;
#pragma unroll 1
    for (; i < 6; i++) {
        const uint32_t t = T0 + a.slack * i / 5;
        const float inv = __fdividef(1.0f, (float)t);
        p[0] = pieces(n[0], t, inv), p[1] = pieces(n[1], t, inv);
        if (__reduce_add_sync(DGT_FULL, (p[0] + p[1]) * heads) <= grid) break;
    }
    if (i == 6) return shares();
    uint32_t cnt;
    const uint32_t ex = warp_excl_scan((p[0] + p[1]) * heads, &cnt);
    k.C = cnt;
    // the tile of this CTA's part
    const uint32_t cta = blockIdx.x, mid = ex + p[0] * heads;
    const uint32_t who = __ballot_sync(DGT_FULL, cta >= ex && cta < mid + p[1] * heads);
    if (!who) {
        k.u0 = k.u1 = 0;
        return k;
    }
    const int src = __ffs(who) - 1;
    const bool second = cta >= mid;
    const uint32_t first = __shfl_sync(DGT_FULL, second ? mid : ex, src);
    const uint32_t parts = __shfl_sync(DGT_FULL, second ? p[1] : p[0], src), pages = __shfl_sync(DGT_FULL, second ? n[1] : n[0], src);
    const uint32_t slot = 2 * src + __shfl_sync(DGT_FULL, (uint32_t)second, src);
    const uint32_t h = (cta - first) / parts, j = (cta - first) % parts, at = slots[slot].base + h * (pages + a.end);
    k.u0 = at + (j ? a.end + j * pages / parts : 0);
    k.u1 = at + a.end + (j + 1) * pages / parts;
    k.c0 = first + h * parts;
    k.c1 = k.c0 + parts - 1;
    return k;
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
// is their barrier, sh shared memory of join_floats(RT) floats.  First a warp
// per row, a part per lane, finds the row's maxima and denominator; then four
// elements at a time are weighted and added, the parts' loads in flight
// together.
constexpr uint32_t JOIN_PARTS = 32;
__host__ __device__ constexpr uint32_t join_floats(uint32_t RT) { return (JOIN_PARTS + 2) * RT; }
template <uint32_t D, uint32_t PART, uint32_t RT, typename Sync>
__device__ __forceinline__ void join_parts(const AttnArgs &a, const Slot &s, uint32_t h, uint32_t c0, uint32_t c1,
                                           uint32_t t, uint32_t threads, float wlog2, float *sh, Sync sync) {
    float2 *rows = reinterpret_cast<float2 *>(sh);   // per row MU, the quotient's factor
    float *weight = sh + 2 * RT;                     // per part and row
    const uint32_t parts = c1 - c0 + 1;
    // part 0 is the one that begins the segment, at the end of its CTA's work
    auto at = [&](uint32_t k, uint32_t row) {
        return a.part + (2 * (uint64_t)(c0 + k) + (k == 0 ? 1 : 0)) * PART + row * (D + 4);
    };
    auto finish = [&](uint32_t row, float M, float MU, float L) {
        const bool none = M == -INFINITY && L == 0.0f;
        rows[row] = make_float2(finite_base(MU), none ? 0.0f : ex2(finite_base(MU) - finite_base(M) - wlog2) / L);
        if (a.lse) {
            const uint32_t flat = s.row0 + row;
            a.lse[(uint64_t)(s.tok0 + flat / a.group) * a.q_heads + h * a.group + flat % a.group] =
                none ? -INFINITY : (M + __log2f(L)) * LN2;
        }
    };
    // RPW rows a warp, their loads together
    constexpr uint32_t RPW = RT / 4;
    const uint32_t lane = t & 31, warp = t >> 5;
    float M[RPW], MU[RPW], L[RPW], mu0[RPW];
#pragma unroll
    for (uint32_t i = 0; i < RPW; i++) M[i] = MU[i] = -INFINITY, L[i] = 0.0f;
    for (uint32_t k0 = 0; k0 < parts; k0 += 32) {
        float4 st[RPW];
#pragma unroll
        for (uint32_t i = 0; i < RPW; i++) {
            st[i] = make_float4(-INFINITY, -INFINITY, 0.0f, 0.0f);
            if (k0 + lane < parts && warp + 4 * i < s.rows)
                st[i] = __ldcg(reinterpret_cast<const float4 *>(at(k0 + lane, warp + 4 * i)));
        }
#pragma unroll
        for (uint32_t i = 0; i < RPW; i++) {
            if (k0 == 0) mu0[i] = st[i].y;
            float m = fmaxf(M[i], st[i].x), u = st[i].y;
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) {
                m = fmaxf(m, __shfl_xor_sync(DGT_FULL, m, d));
                u = fmaxf(u, __shfl_xor_sync(DGT_FULL, u, d));
            }
            const float b = finite_base(m);
            float l = st[i].z * ex2(st[i].x - b);
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(DGT_FULL, l, d);
            L[i] = L[i] * ex2(M[i] - b) + l;
            M[i] = m;
            MU[i] = fmaxf(MU[i], u);
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < RPW; i++) {
        const uint32_t row = warp + 4 * i;
        if (row >= s.rows) break;
        weight[lane * RT + row] = ex2(mu0[i] - finite_base(MU[i]));
        if (lane == 0) finish(row, M[i], MU[i], L[i]);
    }
    sync();
    constexpr uint32_t Q = D / 4, B = RT / 8, UN = RT <= 8 ? 8 : 4;   // B elements of four in flight, UN parts
    const uint32_t all = s.rows * Q;
    for (uint32_t i0 = t; i0 < all; i0 += B * threads) {
        float v[B][4] = {};
        float2 ro[B];
#pragma unroll
        for (uint32_t b = 0; b < B; b++) ro[b] = rows[min(i0 + b * threads, all - 1) / Q];
        // UN parts' loads together; past the last part the last again, with weight 0
        for (uint32_t k0 = 0; k0 < parts; k0 += UN) {
            float f[UN][B];
            float4 x[UN][B];
#pragma unroll
            for (uint32_t j = 0; j < UN; j++)
#pragma unroll
                for (uint32_t b = 0; b < B; b++) {
                    const uint32_t i = min(i0 + b * threads, all - 1), row = i / Q, k = min(k0 + j, parts - 1);
                    const float *p = at(k, row);
                    x[j][b] = __ldcg(reinterpret_cast<const float4 *>(p + 4 + (i % Q) * 4));
                    f[j][b] = k0 < JOIN_PARTS ? weight[k * RT + row] : __ldcg(p + 1) - ro[b].x;
                }
#pragma unroll
            for (uint32_t j = 0; j < UN; j++)
#pragma unroll
                for (uint32_t b = 0; b < B; b++) {
                    const float w = k0 + j >= parts ? 0.0f : k0 < JOIN_PARTS ? f[j][b] : ex2(f[j][b]);
                    v[b][0] += x[j][b].x * w, v[b][1] += x[j][b].y * w, v[b][2] += x[j][b].z * w, v[b][3] += x[j][b].w * w;
                }
        }
#pragma unroll
        for (uint32_t b = 0; b < B; b++) {
            const uint32_t i = i0 + b * threads;
            if (i >= all) break;
            const uint32_t flat = s.row0 + i / Q;
            const uint64_t o = (uint64_t)(s.tok0 + flat / a.group) * a.q_heads + h * a.group + flat % a.group;
            *reinterpret_cast<uint2 *>(a.out + o * D + (i % Q) * 4) =
                make_uint2(bf16x2(v[b][0] * ro[b].y, v[b][1] * ro[b].y), bf16x2(v[b][2] * ro[b].y, v[b][3] * ro[b].y));
        }
    }
    sync();   // sh and the parts are done with
}

// A CTA's arrival at a segment's counter, after a barrier behind its part's
// stores: true for the last of `parts` to arrive, which then sees all parts
// (behind another barrier for the other threads).
__device__ __forceinline__ bool arrive_last(int32_t *count, uint32_t parts) {
    int32_t was;
    asm volatile("atom.add.acq_rel.gpu.s32 %0, [%1], 1;" : "=r"(was) : "l"(count) : "memory");
    if (was != (int32_t)(parts - 1)) return false;
    *count = 0;
    return true;
}

}  // namespace dgt
