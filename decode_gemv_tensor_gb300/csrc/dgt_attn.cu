// dgt_attn.cu -- attention over the paged 8-bit cache.
//
// For a query row q at position p and the positions j that it sees,
//   t_j = scale * q . k_j,   out = sum_j e^(t_j - m) v_j / sum_j e^(t_j - m),
// in one pass over the cache with the running maximum m: when a page raises
// it, the sums so far are multiplied by e^(old - new).  Exponentials are in
// base 2, with log2(e) inside the scale.
//
// The values' scales differ from page to page, so two maxima run: m of the
// scores (the denominator l counts exp2(t - m)) and mu of score + log2(value
// scale) (the numerator sums codes times exp2(t + log2 vs - mu)).  Then no
// page's weight is lost to another page's scale, and the quotient is
// exp2(mu - m) * numerator / l.
//
// What bounds it: with many long sequences HBM (48 of up to 6007 tokens, 8 kv
// heads of 128: 62 us, 5.8 TB/s, 87 % of the measured copy rate; two of 131072
// and 93523, 8 heads of 256: 138 us, 99 %); with few pages a warp the chain of
// dependent steps from the tables to the join (one sequence of 778 tokens: 9.1
// us, of which its bytes are 0.2).
#include "dgt_attn.cuh"

namespace dgt {

constexpr float W_LOG2 = 12.0f;        // weights of the numerator reach 2^12 (fp16 holds them to 2^-24)
constexpr uint32_t AT_WARPS = 4;

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// The queries: rows of up to eight per n-tile (NT of them) are the N side of
// the matrix instructions, a page's 64 tokens their M side for S = K Q^T, and
// 16 dimensions at a time for O += V^T P^T; the accumulators of S, packed and
// transposed eight by eight, are the operand P^T.  Which token stands in which
// row of S is free, and so chosen that a lane's value word (four tokens of a
// dimension) is what the second product wants, and which dimension in which
// step likewise, so that keys and values are read 16 bytes at a time without
// bank conflicts (see kv_k_off).
//
// Every warp works alone on its share of a CTA's pages with its own ring of
// bulk copies (one item: 64 tokens by up to 128 dimensions of one side), and
// looks ahead into the CTA's next segment; warps meet only at a segment's end.

// CTAs an SM: what the registers allow without spills.  64 dimensions and up to
// eight rows, three against two: 48 sequences of up to 6000 tokens, 4 kv heads
// 24 and 29 us, 200 of 300 20 and 23 us, one of 500 9.1 and 8.8 us; with 16
// rows, spilling, 37 and 39, 30 and 32, 12.0 and 11.2 us, 2 of 60000 33 and 29.
__host__ __device__ constexpr uint32_t attn_ctas(uint32_t D, uint32_t nt) { return D == 64 && nt == 1 ? 3 : 2; }

template <uint32_t D, uint32_t NT>
struct AttnCfg {
    static constexpr uint32_t PD = D < 128 ? D : 128, PAN = D / PD;
    static constexpr uint32_t IB = KV_P * PD, IPP = 2 * PAN;
    static constexpr uint32_t CTAS = attn_ctas(D, NT);
    static constexpr uint32_t NS = D == 64 ? (CTAS == 3 ? 3 : 4) : 2;   // deeper rings were no faster
    static constexpr uint32_t RT = 8 * NT;
    static constexpr uint32_t KSTEPS = D / 16;           // k-steps of the first product; their operands stay in registers
    static_assert(NT * D <= 256, "which more rows would not");
    static constexpr uint32_t RS = D + 4;                // row of the merge scratch, padded
    static constexpr uint32_t ring = 0, scratch = AT_WARPS * NS * IB, q = scratch + AT_WARPS * 8 * RS * 4,
                              bytes = q + KSTEPS * NT * 256;
    static constexpr uint32_t PART = RT * (D + 4);       // floats of a partial result
};

template <uint32_t D, uint32_t NT>
__global__ void __launch_bounds__(AT_WARPS * 32, attn_ctas(D, NT)) k_kv_attention(AttnArgs a) {
    using Cfg = AttnCfg<D, NT>;
    constexpr uint32_t RT = Cfg::RT, NS = Cfg::NS, IB = Cfg::IB, PD = Cfg::PD, PAN = Cfg::PAN, IPP = Cfg::IPP;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bar[AT_WARPS][NS];
    __shared__ Slot slots[AT_CHUNK];
    __shared__ float stat[AT_WARPS][RT][3];
    __shared__ float rowstat[RT][3];
    __shared__ float rowfac[RT];
    __shared__ uint64_t usum[AT_WARPS];
    __shared__ int last_flag;
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    if (tid < AT_WARPS * NS) mbar_init(smem_u32(&bar[tid / NS][tid % NS]), 1);
    fence_mbarrier_init();
    __syncthreads();
    pdl_trigger();
    pdl_wait();

    // ---- the CTA's units
    Units here = describe<AT_WARPS>(a, RT, 0, slots, usum);
    const Units all = a.slots <= AT_CHUNK ? here : all_units<AT_WARPS>(a, RT, usum);
    const Cuts cut = cut_plan(a, all, slots, gridDim.x);
    if (blockIdx.x >= cut.C) return;
    const uint64_t ub = cut.parts ? cut.U : cut.raw(blockIdx.x + 1);

    const uint32_t ring = smem_u32(smem) + warp * NS * IB;
    float *scratch = reinterpret_cast<float *>(smem + Cfg::scratch);
    const uint32_t qs = smem_u32(smem + Cfg::q);
    // pages are read once: they leave L2 first, tables, lengths and queries stay
    const uint64_t once = l2_evict_first();
    uint32_t issued = 0, taken = 0;   // items of this warp's ring
    bool dead = false;                // a wait ran out: no more work from this warp

    uint64_t base0 = 0;
    for (uint32_t s0 = 0; s0 < a.slots && base0 < ub; s0 += AT_CHUNK) {
        // ---- describe the next row tiles
        if (s0) here = describe<AT_WARPS>(a, RT, s0, slots, usum);
        const uint32_t tot = (uint32_t)here.units();
        const uint32_t nslots = min(AT_CHUNK, a.slots - s0);
        const uint64_t chunk_base = base0;
        base0 += tot;
        uint32_t u0, u1;
        cut.share(slots, nslots, chunk_base, tot, u0, u1);
        if (u0 >= u1) continue;

        struct Share : Run {
            uint32_t wa, wb;   // this warp's pages
        };
        auto make_run = [&](uint32_t u) {
            Share r;
            static_cast<Run &>(r) = run_at(slots, nslots, a.end, u, u1);
            const uint32_t cnt = slots[r.slot].np ? r.pe - r.pa : 0;
            r.wa = r.pa + warp * cnt / AT_WARPS, r.wb = r.pa + (warp + 1) * cnt / AT_WARPS;
            return r;
        };

        // a row's elements 2 lane + 64 j and the next
        auto load_row = [&](const Slot &s, uint32_t h, uint32_t row, uint32_t (&bits)[D / 64]) {
            const uint32_t flat = s.row0 + row;
            const bool live = row < s.rows;
            const uint16_t *qp = a.q.data + (int64_t)(s.tok0 + flat / a.group) * a.q.token_stride +
                                 (int64_t)(h * a.group + flat % a.group) * a.q.head_stride;
#pragma unroll
            for (uint32_t j = 0; j < D / 64; j++)
                bits[j] = live ? reinterpret_cast<const uint32_t *>(qp)[lane + 32 * j] : 0u;
        };
        // ---- issue side: page numbers and scales of up to 32 pages in the lanes
        Share ir = make_run(u0);
        // the first run's queries travel while its pages are looked up
        uint32_t ahead[D / 64];
        load_row(slots[ir.slot], ir.h, warp, ahead);
        bool at_hand = true;
        uint32_t ix = ir.wa, ik = 0, ibs = ir.wa, ibe = ir.wa;
        bool more = true, fresh = false;   // fresh: a batch that the consuming side has not taken over
        int bpid = -1;
        float bks = 0.0f, bvs = 0.0f;
        auto load_batch = [&]() {
            const Slot &s = slots[ir.slot];
            ibs = ix;
            ibe = min(ix + 32, ir.wb);
            bpid = -1;
            if (ix + lane < ibe) {
                const int32_t p = a.c.table[(uint64_t)s.seq * a.c.max_pages + s.page_index(ix + lane)];
                if (p < 0 || (uint32_t)p >= a.c.pages) {
                    set_status(a.status, DGT_ERR_ARG);
                } else {
                    bpid = p;
                    const uint64_t bi = kv_block(a.c, a.layer, (uint32_t)p, ir.h);
                    bks = a.c.k_scale[bi];
                    bvs = a.c.v_scale[bi];
                }
            }
            fresh = true;
        };
        auto issue = [&]() {
            while (more && issued - taken < NS) {
                if (ix == ibe) {
                    if (fresh) break;
                    while (ix == ir.wb) {
                        const uint32_t next = ir.u + ir.units;
                        if (next >= u1) {
                            more = false;
                            break;
                        }
                        ir = make_run(next);
                        ix = ir.wa;
                    }
                    if (!more) break;
                    load_batch();
                }
                const int p = __shfl_sync(DGT_FULL, bpid, ix - ibs);
                if (lane == 0) {
                    // a page that is not there is passed over when its turn comes; page 0 stands in
                    const uint64_t bi = kv_block(a.c, a.layer, p < 0 ? 0u : (uint32_t)p, ir.h);
                    const uint8_t *src = (ik < PAN ? a.c.k : a.c.v) + bi * (KV_P * D) + (ik % PAN) * IB;
                    const uint32_t st = issued % NS, fb = smem_u32(&bar[warp][st]);
                    fence_proxy_async_smem();
                    mbar_arrive_expect_tx(fb, IB);
                    bulk_g2s_once(ring + st * IB, src, IB, fb, once);
                }
                issued++;
                if (++ik == IPP) {
                    ik = 0;
                    ix++;
                }
            }
        };
        // the next item's stage once it has arrived; false when the wait ran out
        auto arrive = [&](uint32_t &addr) {
            const uint32_t st = taken % NS;
            addr = ring + st * IB;
            // a lane that saw the phase end speaks for all
            if (__any_sync(DGT_FULL, mbar_wait_n(smem_u32(&bar[warp][st]), (taken / NS) & 1u, a.spin))) return true;
            if (lane == 0) set_status(a.status, DGT_ERR_TIMEOUT);
            return false;
        };
        auto release = [&]() {
            __syncwarp();
            taken++;
            issue();
        };
        if (dead) more = false;
        issue();

        // ---- consume the CTA's runs of this chunk
        for (uint32_t u = u0; u < u1;) {
            const Share r = make_run(u);
            u += r.units;
            const Slot s = slots[r.slot];

            if (s.np == 0) {
                write_none<D>(a, s, r.h, tid, AT_WARPS * 32);
                at_hand = false;
                continue;
            }
            // queries: a row per warp at a time, scaled to its exponent, in fragment order
            __syncthreads();
            uint32_t rows[RT / AT_WARPS][D / 64];   // all loads first
#pragma unroll
            for (uint32_t i = 0; i < RT / AT_WARPS; i++) {
                if (i == 0 && at_hand) {
#pragma unroll
                    for (uint32_t j = 0; j < D / 64; j++) rows[0][j] = ahead[j];
                } else {
                    load_row(s, r.h, warp + i * AT_WARPS, rows[i]);
                }
            }
#pragma unroll
            for (uint32_t i = 0; i < RT / AT_WARPS; i++) {
                const uint32_t row = warp + i * AT_WARPS;
                const uint32_t(&bits)[D / 64] = rows[i];
                float x[D / 32], amax = 0.0f;
#pragma unroll
                for (uint32_t j = 0; j < D / 64; j++) {
                    x[2 * j] = bf16lo(bits[j]);
                    x[2 * j + 1] = bf16hi(bits[j]);
                    // by bits, so that a NaN counts as the largest
                    amax = __uint_as_float(max(__float_as_uint(amax), max(__float_as_uint(x[2 * j]) & 0x7FFFFFFFu,
                                                                         __float_as_uint(x[2 * j + 1]) & 0x7FFFFFFFu)));
                }
                const uint32_t top = __reduce_max_sync(DGT_FULL, __float_as_uint(amax)) >> 23;
                // the largest element to [2^14, 2^15): exact in fp16 down to 2^-31 of it
                const int up = 14 + 127 - (int)top, up0 = min(up, 100);
                const float f0 = top == 255 ? 0.0f : __uint_as_float((uint32_t)(up0 + 127) << 23);
                const float f1 = __uint_as_float((uint32_t)(up - up0 + 127) << 23);
                if (lane == 0)
                    rowfac[row] = top == 255 ? __uint_as_float(0x7FC00000u) : ldexpf(a.scale_log2, -up);
#pragma unroll
                for (uint32_t j = 0; j < D / 64; j++) {
                    const uint32_t d = 2 * (lane + 32 * j);   // the pair's first dimension
                    uint32_t step, cc;
                    if (D == 64) {
                        cc = d >> 4;
                        step = (d & 15) >> 2;
                    } else {
                        cc = (d & 127) >> 5;
                        step = (d >> 7) * 8 + ((d & 31) >> 2);
                    }
                    const uint32_t fr = ((step * NT + row / 8) * 32 + (row & 7) * 4 + cc) * 8 + ((d >> 1) & 1) * 4;
                    // not finite: the row's factor says so, the operand stays clean
                    const float lo = top == 255 ? 0.0f : x[2 * j] * f0 * f1, hi = top == 255 ? 0.0f : x[2 * j + 1] * f0 * f1;
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(qs + fr), "r"(f16_pair(lo, hi)) : "memory");
                }
            }
            __syncthreads();

            at_hand = false;
            uint2 qf[Cfg::KSTEPS * NT];
#pragma unroll
            for (uint32_t i = 0; i < Cfg::KSTEPS * NT; i++)
                asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(qf[i].x), "=r"(qf[i].y) : "r"(qs + (i * 32 + lane) * 8));
            // per column (query row 8 nt + 2 c + e): factor, position, window start, maxima, sum
            float fac[NT][2], m[NT][2], mu[NT][2], l[NT][2];
            float o[D / 16][NT][4];
            int32_t pos[NT][2];
#pragma unroll
            for (uint32_t nt = 0; nt < NT; nt++)
#pragma unroll
                for (uint32_t e = 0; e < 2; e++) {
                    const uint32_t row = 8 * nt + 2 * c + e;
                    fac[nt][e] = rowfac[row];
                    pos[nt][e] = row < s.rows ? s.pos0 + (int32_t)((s.row0 + row) / a.group) : -1;
                    m[nt][e] = mu[nt][e] = -INFINITY;
                    l[nt][e] = 0.0f;
                }
#pragma unroll
            for (uint32_t i = 0; i < D / 16; i++)
#pragma unroll
                for (uint32_t nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int j = 0; j < 4; j++) o[i][nt][j] = 0.0f;
            const int32_t pf = s.pos0 + (int32_t)(s.row0 / a.group);
            const int32_t pl = s.pos0 + (int32_t)((s.row0 + s.rows - 1) / a.group);

            int cpid = -1;
            float cks = 0.0f, cvs = 0.0f;
            uint32_t cbs = r.wa, cbe = r.wa;
            for (uint32_t x = r.wa; x < r.wb && !dead; x++) {
                if (x == cbe) {
                    cpid = bpid, cks = bks, cvs = bvs, cbs = ibs, cbe = ibe;
                    fresh = false;
                    issue();
                }
                const int pid = __shfl_sync(DGT_FULL, cpid, x - cbs);
                const float ks = __shfl_sync(DGT_FULL, cks, x - cbs), vs = __shfl_sync(DGT_FULL, cvs, x - cbs);
                uint32_t addr;
                float sc[4][NT][4];
#pragma unroll
                for (int t = 0; t < 4; t++)
#pragma unroll
                    for (uint32_t nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int j = 0; j < 4; j++) sc[t][nt][j] = 0.0f;

                // S: m-tile t holds tokens 16 (i / 2) + 4 t + i % 2 (rows i < 8) and those + 2 (rows 8 + i)
#pragma unroll
                for (uint32_t pan = 0; pan < PAN; pan++) {
                    if (!dead && !arrive(addr)) dead = true;
                    if (!dead && pid >= 0) {
#pragma unroll
                        for (uint32_t t = 0; t < 4; t++) {
                            const uint32_t ta = 16 * (g >> 1) + 4 * t + (g & 1), tb = ta + 2;
#pragma unroll
                            for (uint32_t i = 0; i < PD / 64; i++) {
                                const uint32_t ch = PD == 64 ? c : 2 * c + i;
                                const uint4 ua4 = lds16(addr + ta * PD + ((ch ^ (PD == 64 ? (ta >> 1) & 3 : ta & 7)) << 4));
                                const uint4 ub4 = lds16(addr + tb * PD + ((ch ^ (PD == 64 ? (tb >> 1) & 3 : tb & 7)) << 4));
                                const uint32_t wa[4] = {ua4.x, ua4.y, ua4.z, ua4.w}, wb[4] = {ub4.x, ub4.y, ub4.z, ub4.w};
#pragma unroll
                                for (uint32_t w = 0; w < 4; w++) {
                                    const uint32_t a0 = e4m3_lo(wa[w]), a2 = e4m3_hi(wa[w]);
                                    const uint32_t a1 = e4m3_lo(wb[w]), a3 = e4m3_hi(wb[w]);
#pragma unroll
                                    for (uint32_t nt = 0; nt < NT; nt++) {
                                        const uint2 b = qf[(pan * 8 + i * 4 + w) * NT + nt];
                                        mma16816(sc[t][nt], a0, a1, a2, a3, b.x, b.y);
                                    }
                                }
                            }
                        }
                    }
                    if (!dead) release();
                }
                if (dead) break;
                if (pid < 0) {
#pragma unroll
                    for (uint32_t pan = 0; pan < PAN; pan++) {
                        if (!dead && !arrive(addr)) dead = true;
                        if (!dead) release();
                    }
                    continue;
                }

                // weights; a page that every row sees whole needs no comparisons
                const int32_t t0 = (int32_t)(s.page_index(x) * KV_P);
                const bool whole = t0 + (int32_t)KV_P - 1 <= pf &&
                                   (!a.window || t0 > pl - (int32_t)a.window || (uint32_t)t0 + KV_P <= a.sinks);
                // log2 of the values' scale, a power of two (0, never written: 2^-127 does as well)
                const float ev = (float)((int)(__float_as_uint(vs) >> 23) - 127);
                uint32_t pw[4][NT][2];
#pragma unroll
                for (uint32_t nt = 0; nt < NT; nt++) {
                    float tm[2] = {-INFINITY, -INFINITY}, al[2], ao[2], bs[2], cw[2];
#pragma unroll
                    for (uint32_t t = 0; t < 4; t++)
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            float v = sc[t][nt][j] * (fac[nt][j & 1] * ks);
                            if (!whole) {
                                const int32_t tok = t0 + (int32_t)(16 * (g >> 1) + 4 * t + (g & 1) + 2 * (j >> 1));
                                const int32_t p = pos[nt][j & 1];
                                const bool see = tok <= p && (!a.window || (int64_t)tok > (int64_t)p - a.window ||
                                                              (uint32_t)tok < a.sinks);
                                if (!see) v = -INFINITY;
                            }
                            sc[t][nt][j] = v;
                            tm[j & 1] = fmaxf(tm[j & 1], v);
                        }
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        tm[e] = fmaxf(tm[e], __shfl_xor_sync(DGT_FULL, tm[e], 4));
                        tm[e] = fmaxf(tm[e], __shfl_xor_sync(DGT_FULL, tm[e], 8));
                        tm[e] = fmaxf(tm[e], __shfl_xor_sync(DGT_FULL, tm[e], 16));
                        const float mn = fmaxf(m[nt][e], tm[e]), un = fmaxf(mu[nt][e], tm[e] + ev);
                        bs[e] = finite_base(mn);
                        const float ubs = finite_base(un);
                        al[e] = ex2(m[nt][e] - bs[e]);
                        ao[e] = ex2(mu[nt][e] - ubs);
                        cw[e] = vs != vs ? vs : ex2(fminf(bs[e] + ev - ubs + W_LOG2, 126.0f));
                        m[nt][e] = mn;
                        mu[nt][e] = un;
                    }
                    float ps[2] = {0.0f, 0.0f};
#pragma unroll
                    for (uint32_t t = 0; t < 4; t++) {
                        float w[4];
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const float p = ex2(sc[t][nt][j] - bs[j & 1]);
                            ps[j & 1] += p;
                            w[j] = p * cw[j & 1];
                            // a token that the row does not see has no weight, whatever its value's scale is
                            if (!whole && sc[t][nt][j] == -INFINITY) w[j] = 0.0f;
                        }
                        pw[t][nt][0] = transpose8x8(f16_pair(w[0], w[1]));
                        pw[t][nt][1] = transpose8x8(f16_pair(w[2], w[3]));
                    }
                    l[nt][0] = l[nt][0] * al[0] + ps[0];
                    l[nt][1] = l[nt][1] * al[1] + ps[1];
                    if (__any_sync(DGT_FULL, ao[0] != 1.0f || ao[1] != 1.0f)) {
#pragma unroll
                        for (uint32_t i = 0; i < D / 16; i++) {
                            o[i][nt][0] *= ao[0];
                            o[i][nt][1] *= ao[1];
                            o[i][nt][2] *= ao[0];
                            o[i][nt][3] *= ao[1];
                        }
                    }
                }

                // O: 16 dimensions at a time, k-step t the tokens of m-tile t
#pragma unroll
                for (uint32_t pan = 0; pan < PAN; pan++) {
                    if (!dead && !arrive(addr)) dead = true;
                    if (!dead) {
#pragma unroll
                        for (uint32_t i = 0; i < PD / 16; i++) {
                            const uint4 ua4 = lds16(addr + (16 * i + g) * KV_P + 16 * c);
                            const uint4 ub4 = lds16(addr + (16 * i + g + 8) * KV_P + 16 * c);
                            const uint32_t wa[4] = {ua4.x, ua4.y, ua4.z, ua4.w}, wb[4] = {ub4.x, ub4.y, ub4.z, ub4.w};
#pragma unroll
                            for (uint32_t t = 0; t < 4; t++) {
                                const uint32_t a0 = e4m3_lo(wa[t]), a2 = e4m3_hi(wa[t]);
                                const uint32_t a1 = e4m3_lo(wb[t]), a3 = e4m3_hi(wb[t]);
#pragma unroll
                                for (uint32_t nt = 0; nt < NT; nt++)
                                    mma16816(o[pan * (PD / 16) + i][nt], a0, a1, a2, a3, pw[t][nt][0], pw[t][nt][1]);
                            }
                        }
                        release();
                    }
                }
            }
            if (dead) {
                // let every copy in flight land before the CTA can end
                more = false;
                for (uint32_t i = taken; i < issued; i++) mbar_wait(smem_u32(&bar[warp][i % NS]), (i / NS) & 1u);
                issued = taken;
            }

            // ---- the warps' sums to one
#pragma unroll
            for (uint32_t nt = 0; nt < NT; nt++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float v = l[nt][e];
                    v += __shfl_xor_sync(DGT_FULL, v, 4);
                    v += __shfl_xor_sync(DGT_FULL, v, 8);
                    v += __shfl_xor_sync(DGT_FULL, v, 16);
                    if (g == 0) {
                        float *st = stat[warp][8 * nt + 2 * c + e];
                        st[0] = m[nt][e], st[1] = mu[nt][e], st[2] = v;
                    }
                }
            __syncthreads();
            if (warp < NT) {
                // a row per four lanes, a warp's sums in each
                const float *st = stat[c][8 * warp + g];
                float M = st[0], MU = st[1];
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) {
                    M = fmaxf(M, __shfl_xor_sync(DGT_FULL, M, d));
                    MU = fmaxf(MU, __shfl_xor_sync(DGT_FULL, MU, d));
                }
                float L = st[2] * ex2(st[0] - finite_base(M));
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) L += __shfl_xor_sync(DGT_FULL, L, d);
                if (c == 0) {
                    float *o2 = rowstat[8 * warp + g];
                    o2[0] = M, o2[1] = MU, o2[2] = L;
                }
            }
            const uint32_t n = s.per_head();
            const bool complete = r.pa == 0 && r.pe == n;
            float *part = a.part + (2 * (uint64_t)blockIdx.x + (r.pa == 0 ? 1 : 0)) * Cfg::PART;
#pragma unroll
            for (uint32_t nt = 0; nt < NT; nt++) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    float MU = -INFINITY;
                    for (uint32_t w = 0; w < AT_WARPS; w++) MU = fmaxf(MU, stat[w][8 * nt + 2 * c + e][1]);
                    f[e] = ex2(mu[nt][e] - finite_base(MU));
                }
                __syncthreads();
#pragma unroll
                for (uint32_t i = 0; i < D / 16; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        scratch[(warp * 8 + 2 * c + (j & 1)) * Cfg::RS + 16 * i + g + 8 * (j >> 1)] = o[i][nt][j] * f[j & 1];
                __syncthreads();
                // four elements a thread
                const uint32_t live = s.rows > 8 * nt ? min(8u, s.rows - 8 * nt) : 0u;
#pragma unroll 2
                for (uint32_t i = tid; i < live * (D / 4); i += AT_WARPS * 32) {
                    const uint32_t rr = i / (D / 4), row = 8 * nt + rr, d = (i % (D / 4)) * 4;
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (uint32_t w = 0; w < AT_WARPS; w++) {
                        const float4 x = *reinterpret_cast<const float4 *>(&scratch[(w * 8 + rr) * Cfg::RS + d]);
                        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
                    }
                    const float *st = rowstat[row];
                    if (complete) {
                        const bool none = st[0] == -INFINITY && st[2] == 0.0f;
                        const float q = none ? 0.0f : ex2(finite_base(st[1]) - finite_base(st[0]) - W_LOG2) / st[2];
                        const uint32_t flat = s.row0 + row;
                        const uint64_t at = (uint64_t)(s.tok0 + flat / a.group) * a.q_heads + r.h * a.group + flat % a.group;
                        *reinterpret_cast<uint2 *>(a.out + at * D + d) = make_uint2(bf16x2(v.x * q, v.y * q), bf16x2(v.z * q, v.w * q));
                        if (a.lse && d == 0) a.lse[at] = none ? -INFINITY : (st[0] + __log2f(st[2])) * LN2;
                    } else {
                        float *pr = part + row * (D + 4);
                        *reinterpret_cast<float4 *>(pr + 4 + d) = v;
                        if (d == 0) *reinterpret_cast<float4 *>(pr) = make_float4(st[0], st[1], st[2], 0.0f);
                    }
                }
            }
            if (complete) continue;

            // ---- partial: the last CTA of the segment to arrive adds its parts in page order
            const uint64_t sa = chunk_base + s.base + (uint64_t)r.h * (n + a.end), sb = sa + n + a.end;   // the segment's units
            uint32_t c0, c1;
            cut.holders(sa, sb, c0, c1);
            __syncthreads();
            if (tid == 0) last_flag = arrive_last(&a.count[c0], c1 - c0 + 1);
            __syncthreads();
            if (!last_flag) continue;
            join_parts<D, Cfg::PART, RT>(a, s, r.h, c0, c1, tid, AT_WARPS * 32, W_LOG2, scratch, [] { __syncthreads(); });
        }
        more = false;   // everything of this chunk has been taken
    }
}

template <uint32_t D, uint32_t NT>
static int attn_launch(const AttnArgs &a, cudaStream_t st) {
    DeviceInfo di;
    if (device_info(&di) != DGT_OK) return DGT_ERR_CUDA;
    constexpr uint32_t smem = AttnCfg<D, NT>::bytes;
    auto fn = k_kv_attention<D, NT>;
    static std::atomic<uint64_t> ready;   // devices that allow the shared memory
    const uint64_t bit = di.device < 64 ? 1ull << di.device : 0;
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
            cudaSuccess)
            return DGT_ERR_CUDA;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    const unsigned grid = AttnCfg<D, NT>::CTAS * std::min((unsigned)di.sms, AT_MAX_SMS);
    return launch_pdl(fn, dim3(grid), dim3(AT_WARPS * 32), smem, st, a) == cudaSuccess ? DGT_OK : DGT_ERR_CUDA;
}

// Rows of a tile, by an entry's rows (the mean of a batch): in n-tiles of
// eight, as many as they fill, while that is the faster form; more rows go to
// the tensor-core tiles.  Measured on both sides, n-tiles of eight first (1
// sequence of 500 tokens, 8 of up to 8003 with 4 kv heads):
//   64 dimensions, 24 rows: 14 and 12, 23 and 27 us (2 of 60000: 32 and 41);
//     32 rows: 21 and 13, 33 and 28 us;
//   128 dimensions, 16 rows: 13 and 13, 23 and 29 us (2 of 60000: 37 and 42);
//     24 rows: 20 and 14, 35 and 29 us;
//   256 dimensions, 8 rows: 14 and 18, 26 and 38 us; 10 rows: 20 and 18, 41
//     and 39 us.
struct Plan {
    uint32_t nt, RT;   // nt 0: tensor-core tiles
};
static Plan attn_plan(uint32_t head_dim, uint32_t group, uint32_t batch, uint64_t tokens) {
    const uint64_t rows = group * ((tokens + batch - 1) / batch);
    const uint64_t most = head_dim == 64 ? 24 : head_dim == 128 ? 16 : 8;
    if (rows > most) return {0, prompt_rows(head_dim)};
    const uint32_t nt = (uint32_t)((rows + 7) / 8);
    return {nt, 8 * nt};
}
static uint64_t slot_count(uint32_t RT, uint32_t group, uint32_t batch, uint64_t tokens, bool ragged) {
    if (!ragged) return (uint64_t)batch * ((group + RT - 1) / RT);
    return tokens * group / RT + batch;
}

}  // namespace dgt

using namespace dgt;

// Arrival counters, then two partial results per CTA.
constexpr size_t AT_COUNT_BYTES = (3 * AT_MAX_SMS * 4 + 255) / 256 * 256;   // a counter a CTA
extern "C" size_t dgt_kv_attention_workspace_bytes(const dgt_kv_cache *cache, uint32_t q_heads, uint32_t batch,
                                                   uint64_t tokens) {
    if (!cache || cache->kv_heads == 0 || batch == 0 || q_heads < cache->kv_heads) return 0;
    const Plan p = attn_plan(cache->head_dim, q_heads / cache->kv_heads, batch, tokens);
    return AT_COUNT_BYTES + (size_t)AT_MAX_SMS * (p.nt ? attn_ctas(cache->head_dim, p.nt) : 1) * 2 * p.RT * (cache->head_dim + 4) * 4;
}

extern "C" int dgt_kv_attention_ex(const dgt_kv_cache *cache, uint32_t layer, const dgt_heads *q, uint64_t tokens,
                                   const int32_t *d_seqs, const int32_t *d_cu, uint32_t batch, float scale,
                                   uint32_t window, uint32_t sinks, uint16_t *d_out, float *d_lse, void *d_ws,
                                   size_t ws_bytes, int32_t *d_status, unsigned flags, void *stream) {
    int rc = kv_check(cache);
    if (rc != DGT_OK) return rc;
    if (!q || layer >= cache->layers) return DGT_ERR_ARG;
    if (flags & ~(DGT_TEST_SHORT_WAITS | DGT_TEST_WAIT_POLLS(0xFFFF))) return DGT_ERR_ARG;
    if ((rc = batch_check(tokens, batch, d_cu)) != DGT_OK) return rc;
    if (tokens == 0 || batch == 0) return DGT_OK;
    if (!d_seqs || !d_out || !aligned16(d_out)) return DGT_ERR_ARG;
    if (q->heads == 0 || q->heads % cache->kv_heads || q->heads / cache->kv_heads > 64) return DGT_ERR_SHAPE;
    if ((rc = heads_check(q, q->heads)) != DGT_OK) return rc;
    if (!d_ws || ((uintptr_t)d_ws & 255) ||
        ws_bytes < dgt_kv_attention_workspace_bytes(cache, q->heads, batch, tokens))
        return DGT_ERR_ARG;
    AttnArgs a{};
    a.c = *cache;
    a.layer = layer, a.batch = batch, a.q_heads = q->heads, a.tokens = tokens;
    // a window past every position is none
    a.window = window < 0x40000000u ? window : 0u;
    a.sinks = a.window ? (sinks < 0x40000000u ? sinks : 0x40000000u) : 0u;
    a.group = q->heads / cache->kv_heads;
    a.q = *q, a.seqs = d_seqs, a.cu = d_cu, a.scale_log2 = scale * LOG2E, a.out = d_out, a.lse = d_lse;
    a.status = d_status;
    const Plan plan = attn_plan(cache->head_dim, a.group, batch, tokens);
    const uint32_t nt = plan.nt, RT = plan.RT;
    const uint64_t slots = slot_count(RT, a.group, batch, tokens, d_cu != nullptr);
    a.slots = (uint32_t)slots;
    a.per_entry = (a.group + RT - 1) / RT;
    a.count = (int32_t *)d_ws;
    a.part = (float *)((uint8_t *)d_ws + AT_COUNT_BYTES);
    // A page a warp (64 dimensions, 4001 tokens: 10.6 us; 2 or 8 pages 11.6); in prompts eight pages (200 rows of 128
    // dimensions over 500 tokens 18.2 us; 4 pages 21.4).
    a.min_units = nt ? 4 : 8;
    // 30 sequences of up to 1501 tokens, 8 kv heads of 128: 17.1 us (24 pages 18.5); 4 prompts of up to 300 rows over
    // 2300 tokens 42 us (10 pages 46, 24 pages 44).
    a.slack = nt ? 12 : 16;
    // Measured against min_units alone, one sequence of 60000 tokens, one kv head of 64, 128 and 256 dimensions: 4
    // rows 28 and 19, 29 and 20, 49 and 31 us (0.5: 21, 22, 35); 240 rows over 120020 tokens 104 and 76, 218 and
    // 107, 143 and 108 us (0.75: 72, 113, 114).
    a.join = nt ? 0.25f : 1.5f;
    // Measured against shares of equal pages: 100 sequences of up to 300 tokens (64 dimensions) 28 and 22 us, 200
    // of 1000 65 and 52 us (12 instead of 8: the same within 4%); a prompt of 8192 rows (128 dimensions) 770 and
    // 379 us (6: 439, 15: 389).
    a.end = nt ? 8 : 10;
    a.spin = wait_limit_from_flags(flags);
    cudaStream_t st = (cudaStream_t)stream;
    if (nt == 0) return prompt_launch(a, st);
    switch (cache->head_dim) {
        case 64: return nt == 1 ? attn_launch<64, 1>(a, st) : nt == 2 ? attn_launch<64, 2>(a, st) : attn_launch<64, 3>(a, st);
        case 128: return nt == 1 ? attn_launch<128, 1>(a, st) : attn_launch<128, 2>(a, st);
        default: return attn_launch<256, 1>(a, st);
    }
}

extern "C" int dgt_kv_attention(const dgt_kv_cache *cache, uint32_t layer, const dgt_heads *q, uint64_t tokens,
                                const int32_t *d_seqs, const int32_t *d_cu, uint32_t batch, float scale,
                                uint32_t window, uint32_t sinks, uint16_t *d_out, float *d_lse, void *d_ws,
                                size_t ws_bytes, int32_t *d_status, void *stream) {
    return dgt_kv_attention_ex(cache, layer, q, tokens, d_seqs, d_cu, batch, scale, window, sinks, d_out, d_lse, d_ws,
                               ws_bytes, d_status, 0, stream);
}
