// dgt_prompt.cu -- attention of many query rows over the paged 8-bit cache, on
// the 5th-generation tensor cores.
//
// S = Q K^T takes the cache's e4m3 keys as they lie in a page (kv_k_off is the
// operand tile's swizzle), so no key is converted: a bf16 query has eight
// significant bits and e4m3 four, so q = hi + lo with two e4m3 parts, exactly
// while |q| is within 2^-9 of the row's largest element and to 2^-17 of that
// below.  The two parts are two runs of the same matrix instructions into the
// same accumulator; at e4m3's double rate that costs what one fp16 product
// would.  O = P V wants more bits of P than that: P is fp16 (2^-11), in tensor
// memory where the scores were, and four warps turn value pages into fp16
// operand tiles once for all the rows of a CTA.
//
// Per CTA two tiles of 128 rows (head_dim 256: one) share every page: while
// one tile's 128 threads (a row each) take exponentials, the tensor cores work
// on the other.  The numerator's reference maximum moves only when a row has
// grown by 2^8 past it, so the accumulators are rarely rescaled.
#include "dgt_attn.cuh"

#include "dgt_tc.cuh"

namespace dgt {

constexpr float PR_W_LOG2 = 4.0f;    // weights at the reference; 2^8 above it they reach 2^12
constexpr float PR_GROW = 8.0f;
constexpr uint32_t PR_WARPS = 14;    // 0-7 rows, 8-11 values to fp16, 12 matrix instructions, 13 copies
constexpr uint32_t PR_META = 8;

template <uint32_t D>
struct PromptCfg {
    static constexpr uint32_t NSTR = D <= 128 ? 2 : 1;   // row tiles of 128
    static constexpr uint32_t TP = D <= 128 ? 2 : 1;     // pages of a key tile
    static constexpr uint32_t TN = KV_P * TP, RT = 128 * NSTR;
    static constexpr uint32_t RB = D < 128 ? 64 : 128, PAN = D / RB;   // operand row bytes, panels
    static constexpr uint32_t PB = KV_P * D;                           // bytes of a page's block
    static constexpr uint32_t KS = 3, VS = 2, WS = 2;                  // stages: keys, values, fp16 values
    static constexpr uint32_t QP = 128 * D;                            // one part of a row tile
    static constexpr uint32_t q = 0, k = q + NSTR * 2 * QP, v = k + KS * TP * PB, w = v + VS * TP * PB,
                              bytes = w + WS * TP * PB * 2 + 1024;
    static constexpr uint32_t SCOL = 256, SSTEP = TN;                  // score columns: a buffer of TN per tile
    static constexpr uint32_t PART = RT * (D + 4);
};

// What a key tile is: its pages' scales (a page that is not there: used 0).
struct TileMeta {
    float ks[2], vs[2];
    uint32_t used[2];
};

__device__ __forceinline__ void bar_rows() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Sixteen scaled query elements to their two e4m3 parts.
__device__ __forceinline__ void split16(const uint32_t (&bits)[8], float f0, float f1, uint4 &hi, uint4 &lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        float x[4];
        x[0] = bf16lo(bits[2 * j]) * f0 * f1, x[1] = bf16hi(bits[2 * j]) * f0 * f1;
        x[2] = bf16lo(bits[2 * j + 1]) * f0 * f1, x[3] = bf16hi(bits[2 * j + 1]) * f0 * f1;
        h[j] = l[j] = 0;
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * e], x[2 * e + 1]), __NV_SATFINITE,
                                                                     __NV_E4M3);
            const float2 y = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3)));
            const __nv_fp8x2_storage_t r = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * e] - y.x, x[2 * e + 1] - y.y),
                                                                     __NV_SATFINITE, __NV_E4M3);
            h[j] |= (uint32_t)c << (16 * e);
            l[j] |= (uint32_t)r << (16 * e);
        }
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

template <uint32_t D>
__global__ void __launch_bounds__(PR_WARPS * 32, 1) k_kv_prompt(AttnArgs a) {
    using Cfg = PromptCfg<D>;
    constexpr uint32_t NSTR = Cfg::NSTR, TP = Cfg::TP, TN = Cfg::TN, RT = Cfg::RT, RB = Cfg::RB, PAN = Cfg::PAN,
                       PB = Cfg::PB, QP = Cfg::QP, KS = Cfg::KS, VS = Cfg::VS, WS = Cfg::WS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t kfull[KS], kfree[KS], vfull[VS], vfree[VS], wfull[WS], wfree[WS];
    __shared__ __align__(8) uint64_t sfull[2], pfull[2], ofull[2], qfull[2], mfull[PR_META], drained;
    __shared__ TileMeta meta[PR_META];
    __shared__ Slot slots[AT_CHUNK];
    __shared__ uint64_t usum[PR_WARPS];
    __shared__ uint32_t wsum[PR_WARPS];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, last_flag;
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    if (tid == 0) {
        for (uint32_t i = 0; i < KS; i++) mbar_init(smem_u32(&kfull[i]), 1), mbar_init(smem_u32(&kfree[i]), 1);
        for (uint32_t i = 0; i < VS; i++) mbar_init(smem_u32(&vfull[i]), 1), mbar_init(smem_u32(&vfree[i]), 4);
        for (uint32_t i = 0; i < WS; i++) mbar_init(smem_u32(&wfull[i]), 4), mbar_init(smem_u32(&wfree[i]), 1);
        for (uint32_t i = 0; i < 2; i++) {
            mbar_init(smem_u32(&sfull[i]), 1);
            mbar_init(smem_u32(&pfull[i]), 4);
            mbar_init(smem_u32(&ofull[i]), 1);
            mbar_init(smem_u32(&qfull[i]), 4);
        }
        for (uint32_t i = 0; i < PR_META; i++) mbar_init(smem_u32(&mfull[i]), 1);
        mbar_init(smem_u32(&drained), 1);
        abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == 12) {
        tmem_alloc(smem_u32(&tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    pdl_wait();
    const uint32_t tm = tmem_slot;
    volatile int *abortp = &abort_flag;

    Slot si{};
    uint32_t units0;
    const uint64_t U = all_units<PR_WARPS>(a, RT, usum, si, units0);
    const uint64_t most = (U + a.min_units - 1) / a.min_units;
    const uint64_t C = most < gridDim.x ? most : gridDim.x;
    const uint64_t ua = C ? blockIdx.x * U / C : 0, ub = blockIdx.x < C ? (blockIdx.x + 1) * U / C : 0;

    bool dead = false;   // a wait ran out, here or elsewhere in the CTA: no more work from this warp
    // a whole warp's wait
    auto wait = [&](uint64_t &bar, uint32_t parity) {
        if (!dead && !__any_sync(DGT_FULL, wait_or_abort(smem_u32(&bar), parity, abortp, a.spin))) {
            dead = true;
            if (lane == 0) set_status(a.status, DGT_ERR_TIMEOUT);
            *abortp = 1;
        }
        __syncwarp();   // the lane that saw the phase end has seen it for all
        return !dead;
    };
    uint32_t it = 0;               // key tiles so far, the same in every role
    uint32_t qc[2] = {0, 0};       // per row tile: segments, key tiles so far
    uint32_t sc[2] = {0, 0};
    uint32_t kissued = 0, vissued = 0;   // the copying warp's items

    uint64_t base0 = 0;
    for (uint32_t s0 = 0; s0 < a.slots && base0 < ub; s0 += AT_CHUNK) {
        const uint32_t tot = describe<PR_WARPS>(a, RT, s0, si, units0, slots, wsum);
        const uint64_t first = base0 > ua ? base0 : ua, end = base0 + tot < ub ? base0 + tot : ub;
        const uint32_t u0 = (uint32_t)(first - base0), u1 = end > first ? (uint32_t)(end - base0) : u0;
        const uint64_t chunk_base = base0;
        const uint32_t nslots = min(AT_CHUNK, a.slots - s0);
        base0 += tot;
        for (uint32_t u = u0, hint = 0; u < u1;) {
            const Run r = run_at(slots, nslots, u, u1, hint);
            hint = r.slot;
            u += r.pe - r.pa;
            const Slot &s = slots[r.slot];
            const uint32_t n = s.per_head();
            const uint32_t T = s.np ? (r.pe - r.pa + TP - 1) / TP : 0;
            const uint32_t ns = NSTR == 2 && s.rows > 128 ? 2 : 1;   // row tiles that hold rows

            if (warp == 13) {
                // ---- copies
                int pid = -1;
                float ks = 0.0f, vs = 0.0f;
                for (uint32_t j = 0; j < T && !dead; j++) {
                    const uint32_t x = r.pa + j * TP, c = it + j;
                    if ((j * TP) % 32 == 0) {
                        pid = -1;
                        if (x + lane < r.pe) {
                            const int32_t p = a.c.table[(uint64_t)s.seq * a.c.max_pages + s.page_index(x + lane)];
                            if (p < 0 || (uint32_t)p >= a.c.pages) {
                                set_status(a.status, DGT_ERR_ARG);
                            } else {
                                pid = p;
                                const uint64_t bi = kv_block(a.c, a.layer, (uint32_t)p, r.h);
                                ks = a.c.k_scale[bi];
                                vs = a.c.v_scale[bi];
                            }
                        }
                    }
                    if (c >= KS && !wait(kfree[c % KS], (c / KS - 1) & 1u)) break;
                    uint64_t bi[TP];
                    uint32_t have = 0;
#pragma unroll
                    for (uint32_t p = 0; p < TP; p++) {
                        const uint32_t from = (j * TP + p) % 32;
                        const int id = __shfl_sync(DGT_FULL, pid, from);
                        const float kk = __shfl_sync(DGT_FULL, ks, from), vv = __shfl_sync(DGT_FULL, vs, from);
                        bi[p] = kv_block(a.c, a.layer, id < 0 ? 0u : (uint32_t)id, r.h);
                        if (id >= 0) have |= 1u << p;
                        if (lane == 0) {
                            TileMeta &m = meta[c % PR_META];
                            m.ks[p] = id < 0 ? 1.0f : kk, m.vs[p] = id < 0 ? 1.0f : vv, m.used[p] = id >= 0;
                        }
                    }
                    if (lane == 0) {
                        const uint32_t bytes = __popc(have) * PB;
                        mbar_arrive(smem_u32(&mfull[c % PR_META]));
                        const uint32_t kb = smem_u32(&kfull[c % KS]);
                        mbar_arrive_expect_tx(kb, bytes);
#pragma unroll
                        for (uint32_t p = 0; p < TP; p++)
                            if ((have >> p) & 1u)
                                bulk_g2s(base + Cfg::k + ((c % KS) * TP + p) * PB, a.c.k + bi[p] * PB, PB, kb);
                    }
                    kissued = c + 1;
                    if (c >= VS && !wait(vfree[c % VS], (c / VS - 1) & 1u)) break;
                    if (lane == 0) {
                        const uint32_t bytes = __popc(have) * PB, vb = smem_u32(&vfull[c % VS]);
                        mbar_arrive_expect_tx(vb, bytes);
#pragma unroll
                        for (uint32_t p = 0; p < TP; p++)
                            if ((have >> p) & 1u)
                                bulk_g2s(base + Cfg::v + ((c % VS) * TP + p) * PB, a.c.v + bi[p] * PB, PB, vb);
                    }
                    vissued = c + 1;
                    __syncwarp();
                }
            } else if (warp == 12) {
                // ---- matrix instructions, one lane
                constexpr uint32_t idesc_s = (1u << 4) | ((TN >> 3) << 17) | ((128u >> 4) << 24);
                constexpr uint32_t idesc_o = (1u << 4) | ((D >> 3) << 17) | ((128u >> 4) << 24);
                auto desc = [&](uint32_t addr) { return RB == 128 ? sw128_desc(addr) : sw64_desc(addr); };
                auto scores = [&](uint32_t t, uint32_t c, uint32_t col) {
                    if (lane == 0) {
                        const uint32_t kt = base + Cfg::k + (c % KS) * TP * PB;
#pragma unroll
                        for (uint32_t part = 0; part < 2; part++)
#pragma unroll
                            for (uint32_t pan = 0; pan < PAN; pan++) {
                                const uint64_t ad = desc(base + Cfg::q + (2 * t + part) * QP + pan * 128 * RB);
                                const uint64_t bd = desc(kt + pan * KV_P * RB);
#pragma unroll
                                for (uint32_t i = 0; i < RB / 32; i++)
                                    mma_e4m3(tm + col, ad + 2 * i, bd + 2 * i, idesc_s, part + pan + i > 0 ? 1u : 0u);
                            }
                    }
                };
                auto values = [&](uint32_t t, uint32_t c, uint32_t col, bool accumulate) {
                    if (lane == 0) {
#pragma unroll
                        for (uint32_t p = 0; p < TP; p++) {
                            const uint64_t bd = sw128_desc(base + Cfg::w + ((c % WS) * TP + p) * PB * 2);
#pragma unroll
                            for (uint32_t i = 0; i < 4; i++)
                                mma_f16_ta(tm + t * D, tm + col + p * 32 + i * 8, bd + 2 * i, idesc_o,
                                           accumulate || p + i > 0 ? 1u : 0u);
                        }
                    }
                };
                auto commit = [&](uint64_t &bar) {
                    if (lane == 0) mma_commit(smem_u32(&bar));
                    __syncwarp();
                };
                if (NSTR == 2) {
                    if (T && wait(kfull[it % KS], (it / KS) & 1u)) {
                        for (uint32_t t = 0; t < ns; t++) {
                            if (!wait(qfull[t], qc[t] & 1u)) break;
                            tc_fence_after();
                            scores(t, it, Cfg::SCOL + t * Cfg::SSTEP);
                            commit(sfull[t]);
                        }
                        commit(kfree[it % KS]);
                    }
                    for (uint32_t j = 0; j < T && !dead; j++) {
                        const uint32_t c = it + j;
                        for (uint32_t t = 0; t < ns && !dead; t++) {
                            if (!wait(pfull[t], (sc[t] + j) & 1u) || (t == 0 && !wait(wfull[c % WS], (c / WS) & 1u))) break;
                            tc_fence_after();
                            values(t, c, Cfg::SCOL + t * Cfg::SSTEP, j > 0);
                            commit(ofull[t]);
                            if (j + 1 < T) {
                                if (t == 0 && !wait(kfull[(c + 1) % KS], ((c + 1) / KS) & 1u)) break;
                                scores(t, c + 1, Cfg::SCOL + t * Cfg::SSTEP);
                                commit(sfull[t]);
                            }
                        }
                        if (dead) break;
                        commit(wfree[c % WS]);
                        if (j + 1 < T) commit(kfree[(c + 1) % KS]);
                    }
                } else {
                    // one row tile, two score buffers: the next tile's scores before this one's values
                    if (T && wait(kfull[it % KS], (it / KS) & 1u) && wait(qfull[0], qc[0] & 1u)) {
                        tc_fence_after();
                        scores(0, it, Cfg::SCOL + (it & 1) * Cfg::SSTEP);
                        commit(sfull[it & 1]);
                        commit(kfree[it % KS]);
                    }
                    for (uint32_t j = 0; j < T && !dead; j++) {
                        const uint32_t c = it + j, b = c & 1;
                        if (j + 1 < T) {
                            if (!wait(kfull[(c + 1) % KS], ((c + 1) / KS) & 1u)) break;
                            scores(0, c + 1, Cfg::SCOL + (1 - b) * Cfg::SSTEP);
                            commit(sfull[1 - b]);
                            commit(kfree[(c + 1) % KS]);
                        }
                        if (!wait(pfull[b], (c >> 1) & 1u) || !wait(wfull[c % WS], (c / WS) & 1u)) break;
                        tc_fence_after();
                        values(0, c, Cfg::SCOL + b * Cfg::SSTEP, j > 0);
                        commit(ofull[0]);
                        commit(wfree[c % WS]);
                    }
                }
            } else if (warp >= 8) {
                // ---- value pages to fp16 operand tiles: rows of 64 tokens, 128-byte swizzle
                const uint32_t ct = tid - 256;
                for (uint32_t j = 0; j < T && !dead; j++) {
                    const uint32_t c = it + j;
                    if (!wait(vfull[c % VS], (c / VS) & 1u)) break;
                    if (c >= WS && !wait(wfree[c % WS], (c / WS - 1) & 1u)) break;
                    const TileMeta &m = meta[c % PR_META];
#pragma unroll
                    for (uint32_t p = 0; p < TP; p++) {
                        const uint32_t src = base + Cfg::v + ((c % VS) * TP + p) * PB;
                        const uint32_t dst = base + Cfg::w + ((c % WS) * TP + p) * PB * 2;
                        const bool used = m.used[p] != 0;
#pragma unroll 4
                        for (uint32_t i = ct; i < D * 4; i += 128) {
                            const uint32_t row = i >> 2, q = i & 3;
                            uint4 x = make_uint4(0, 0, 0, 0);
                            if (used) x = lds128(src + row * KV_P + q * 16);
                            const uint32_t o = dst + row * 128;
                            sts128(o + (((2 * q) ^ (row & 7)) << 4), e4m3_lo(x.x), e4m3_hi(x.x), e4m3_lo(x.y), e4m3_hi(x.y));
                            sts128(o + (((2 * q + 1) ^ (row & 7)) << 4), e4m3_lo(x.z), e4m3_hi(x.z), e4m3_lo(x.w), e4m3_hi(x.w));
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_u32(&wfull[c % WS]));
                        mbar_arrive(smem_u32(&vfree[c % VS]));
                    }
                }
            } else {
                // ---- a query row per thread
                const uint32_t t = NSTR == 2 ? warp >> 2 : 0, quad = warp & 3;
                const bool mine = NSTR == 2 ? t < ns : warp < 4;
                const uint32_t row = t * 128 + quad * 32 + lane, tl = quad << 21;   // lanes 32 quad .. of tensor memory
                const bool live = mine && row < s.rows;
                const uint32_t flat = s.row0 + row;
                const int32_t pos = live ? s.pos0 + (int32_t)(flat / a.group) : -1;
                float m = -INFINITY, mu = -INFINITY, l = 0.0f, fac = 0.0f;
                if (mine && T) {
                    const uint16_t *qp = a.q.data + (int64_t)(s.tok0 + flat / a.group) * a.q.token_stride +
                                         (int64_t)(r.h * a.group + flat % a.group) * a.q.head_stride;
                    uint32_t top = 0;
                    if (live)
#pragma unroll 4
                        for (uint32_t i = 0; i < D / 8; i++) {
                            const uint4 x = reinterpret_cast<const uint4 *>(qp)[i];
                            top = max(top, max(max(x.x & 0x7FFFu, x.x >> 16 & 0x7FFFu), max(x.y & 0x7FFFu, x.y >> 16 & 0x7FFFu)));
                            top = max(top, max(max(x.z & 0x7FFFu, x.z >> 16 & 0x7FFFu), max(x.w & 0x7FFFu, x.w >> 16 & 0x7FFFu)));
                        }
                    top >>= 7;
                    // the largest element to [2^7, 2^8)
                    const bool bad = top == 255;
                    const int up = 7 + 127 - (int)top, up0 = min(up, 100);
                    float f0 = bad ? 0.0f : __uint_as_float((uint32_t)(up0 + 127) << 23);
                    const float f1 = __uint_as_float((uint32_t)(up - up0 + 127) << 23);
                    if (a.scale_log2 < 0.0f) f0 = -f0;
                    fac = bad ? __uint_as_float(0x7FC00000u) : ldexpf(fabsf(a.scale_log2), -up);
                    const uint32_t q0 = base + Cfg::q + 2 * t * QP, rr = row & 127;
#pragma unroll 2
                    for (uint32_t i = 0; i < D / 16; i++) {
                        uint32_t bits[8] = {};
                        if (live && !bad) {
                            const uint4 x = reinterpret_cast<const uint4 *>(qp)[2 * i], y = reinterpret_cast<const uint4 *>(qp)[2 * i + 1];
                            bits[0] = x.x, bits[1] = x.y, bits[2] = x.z, bits[3] = x.w;
                            bits[4] = y.x, bits[5] = y.y, bits[6] = y.z, bits[7] = y.w;
                        }
                        uint4 hi, lo;
                        split16(bits, f0, f1, hi, lo);
                        const uint32_t pan = i / (RB / 16), ch = i % (RB / 16);
                        const uint32_t at = pan * 128 * RB + rr * RB + ((ch ^ (RB == 128 ? rr & 7 : (rr >> 1) & 3)) << 4);
                        sts128(q0 + at, hi.x, hi.y, hi.z, hi.w);
                        sts128(q0 + QP + at, lo.x, lo.y, lo.z, lo.w);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&qfull[t]));
                }
                const int32_t pf = s.pos0 + (int32_t)(s.row0 / a.group);
                const int32_t pl = s.pos0 + (int32_t)((s.row0 + s.rows - 1) / a.group);
                for (uint32_t j = 0; mine && j < T && !dead; j++) {
                    const uint32_t c = it + j, sb = NSTR == 2 ? t : c & 1;
                    const uint32_t sp = NSTR == 2 ? (sc[t] + j) & 1u : (c >> 1) & 1u;
                    if (!wait(mfull[c % PR_META], (c / PR_META) & 1u) || !wait(sfull[sb], sp)) break;
                    tc_fence_after();
                    const uint32_t st = tm + tl + Cfg::SCOL + sb * Cfg::SSTEP;
                    float f[TP], ev[TP], vsc[TP], tmx[TP];
                    uint32_t see[TP][2];
                    bool whole[TP];
                    uint32_t sv[2][32];
                    float mn = m, un = mu;
#pragma unroll
                    for (uint32_t p = 0; p < TP; p++) {
                        const TileMeta &mt = meta[c % PR_META];
                        const bool used = mt.used[p] != 0;
                        f[p] = fac * mt.ks[p];
                        vsc[p] = mt.vs[p];
                        ev[p] = (float)((int)(__float_as_uint(vsc[p]) >> 23) - 127);
                        // which of the page's 64 tokens the row sees
                        const int32_t t0 = (int32_t)(s.page_index(r.pa + j * TP + p) * KV_P);
                        whole[p] = used && t0 + (int32_t)KV_P - 1 <= pf &&
                                   (!a.window || t0 > pl - (int32_t)a.window || (uint32_t)t0 + KV_P <= a.sinks);
                        see[p][0] = see[p][1] = 0xFFFFFFFFu;
                        if (!whole[p]) {
                            const int32_t hi = used ? min(max(pos - t0 + 1, 0), 64) : 0;   // tokens [0, hi) are not ahead of the row
                            const int32_t lo = a.window ? min(max(pos - (int32_t)a.window + 1 - t0, 0), 64) : 0;
                            const int32_t sk = a.window ? min(max((int32_t)a.sinks - t0, 0), 64) : 0;
                            const uint64_t one = 1ull;
                            const uint64_t below_hi = hi >= 64 ? ~0ull : (one << hi) - 1;
                            const uint64_t below_lo = lo >= 64 ? ~0ull : (one << lo) - 1;
                            const uint64_t below_sk = sk >= 64 ? ~0ull : (one << sk) - 1;
                            const uint64_t v = below_hi & (~below_lo | below_sk);
                            see[p][0] = (uint32_t)v, see[p][1] = (uint32_t)(v >> 32);
                        }
                        tmem_ld32(st + p * KV_P, sv[0]);
                        tmem_ld32(st + p * KV_P + 32, sv[1]);
                        tmem_wait_ld();
                        float mx = -INFINITY;
                        if (whole[p]) {
#pragma unroll
                            for (int i = 0; i < 32; i++)
                                mx = fmaxf(mx, fmaxf(__uint_as_float(sv[0][i]), __uint_as_float(sv[1][i])));
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i++) {
                                if ((see[p][0] >> i) & 1u) mx = fmaxf(mx, __uint_as_float(sv[0][i]));
                                if ((see[p][1] >> i) & 1u) mx = fmaxf(mx, __uint_as_float(sv[1][i]));
                            }
                        }
                        tmx[p] = mx == -INFINITY ? mx : mx * f[p];
                        mn = fmaxf(mn, tmx[p]);
                        un = fmaxf(un, tmx[p] + ev[p]);
                    }
                    const float bm = finite_base(mn);
                    l *= ex2(m - bm);
                    m = mn;
                    const bool grow = un > mu + PR_GROW || (mu == -INFINITY && un > -INFINITY);
                    const float ao = grow ? ex2(mu - un) : 1.0f;
                    if (grow) mu = un;
                    const float bu = finite_base(mu);
                    if (j > 0 && __any_sync(DGT_FULL, grow)) {
                        // this row tile's accumulators: the products of the tile before are done
                        if (NSTR == 1 && !wait(ofull[0], (sc[0] + j - 1) & 1u)) break;
                        tc_fence_after();
#pragma unroll
                        for (uint32_t d0 = 0; d0 < D; d0 += 32) {
                            uint32_t o[32];
                            tmem_ld32(tm + tl + t * D + d0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * ao);
                            tmem_st32(tm + tl + t * D + d0, o);
                        }
                    }
#pragma unroll
                    for (uint32_t p = 0; p < TP; p++) {
                        if (TP > 1) {
                            tmem_ld32(st + p * KV_P, sv[0]);
                            tmem_ld32(st + p * KV_P + 32, sv[1]);
                            tmem_wait_ld();
                        }
                        const float lc = bm + ev[p] - bu + PR_W_LOG2;
                        uint32_t pk[32];
                        float sum = 0.0f;
                        if (__all_sync(DGT_FULL, fabsf(lc) < 40.0f && vsc[p] == vsc[p])) {
                            // weights with the value's scale inside the exponent, their sum without it
                            const float b = lc - bm;
#pragma unroll
                            for (int h = 0; h < 2; h++)
#pragma unroll
                                for (int i = 0; i < 16; i++) {
                                    float x = ex2(fmaf(__uint_as_float(sv[h][2 * i]), f[p], b));
                                    float y = ex2(fmaf(__uint_as_float(sv[h][2 * i + 1]), f[p], b));
                                    if (!whole[p]) {
                                        x = (see[p][h] >> (2 * i)) & 1u ? x : 0.0f;
                                        y = (see[p][h] >> (2 * i + 1)) & 1u ? y : 0.0f;
                                    }
                                    sum += x;
                                    sum += y;
                                    pk[16 * h + i] = f16_pair(x, y);
                                }
                            l += sum * ex2(-lc);
                        } else {
                            const float cw = vsc[p] != vsc[p] ? vsc[p] : ex2(fminf(lc, 126.0f));
#pragma unroll
                            for (int h = 0; h < 2; h++)
#pragma unroll
                                for (int i = 0; i < 16; i++) {
                                    float w[2];
#pragma unroll
                                    for (int e = 0; e < 2; e++) {
                                        const bool v = (see[p][h] >> (2 * i + e)) & 1u;
                                        const float x = ex2(fmaf(__uint_as_float(sv[h][2 * i + e]), f[p], -bm));
                                        sum += v ? x : 0.0f;
                                        w[e] = v ? x * cw : 0.0f;
                                    }
                                    pk[16 * h + i] = f16_pair(w[0], w[1]);
                                }
                            l += sum;
                        }
                        tmem_st32(st + p * 32, pk);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&pfull[sb]));
                }

                // ---- the segment's end: this row's quotient, or its part
                const bool complete = r.pa == 0 && r.pe == n;
                if (mine && T) wait(ofull[t], (sc[t] + T - 1) & 1u);
                tc_fence_after();
                float *part = a.part + (2 * (uint64_t)blockIdx.x + (r.pa == 0 ? 1 : 0)) * Cfg::PART + row * (D + 4);
                const bool none = m == -INFINITY && l == 0.0f;
                const uint64_t at = (uint64_t)(s.tok0 + flat / a.group) * a.q_heads + r.h * a.group + flat % a.group;
                const float quot = none ? 0.0f : ex2(finite_base(mu) - finite_base(m) - PR_W_LOG2) / l;
                if (mine && !dead) {
#pragma unroll 1
                    for (uint32_t d0 = 0; d0 < D; d0 += 32) {
                        uint32_t o[32] = {};
                        if (T) {
                            tmem_ld32(tm + tl + t * D + d0, o);
                            tmem_wait_ld();
                        }
                        if (!live) continue;
                        if (complete) {
#pragma unroll
                            for (int i = 0; i < 32; i += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int e = 0; e < 4; e++) {
                                    const float x = none ? 0.0f : __uint_as_float(o[i + 2 * e]) * quot;
                                    const float y = none ? 0.0f : __uint_as_float(o[i + 2 * e + 1]) * quot;
                                    w[e] = (uint32_t)f32_to_bf16_rne(x) | (uint32_t)f32_to_bf16_rne(y) << 16;
                                }
                                *reinterpret_cast<uint4 *>(a.out + at * D + d0 + i) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                *reinterpret_cast<uint4 *>(part + 4 + d0 + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        }
                    }
                    if (live && complete && a.lse) a.lse[at] = none ? -INFINITY : (m + __log2f(l)) * LN2;
                    if (live && !complete) *reinterpret_cast<float4 *>(part) = make_float4(m, mu, l, 0.0f);
                }
                tc_fence_before();
                if (!complete) {
                    // the last CTA of the segment to arrive adds its parts in page order
                    const uint64_t sa = chunk_base + s.base + (uint64_t)r.h * n, sb = sa + n;
                    const uint64_t c0 = ((sa + 1) * C - 1) / U, c1 = (sb * C - 1) / U;
                    __threadfence();
                    bar_rows();
                    if (tid == 0) {
                        const int32_t was = atomicAdd(&a.count[c0], 1);
                        last_flag = was == (int32_t)(c1 - c0);
                        if (last_flag) a.count[c0] = 0;
                    }
                    bar_rows();
                    if (last_flag) {
                        __threadfence();
                        join_parts<D, Cfg::PART>(a, s, r.h, c0, c1, tid, 256, PR_W_LOG2);
                    }
                }
            }
            it += T;
            for (uint32_t t = 0; t < ns; t++) sc[t] += T, qc[t] += T ? 1 : 0;
        }
    }

    // copies land and matrix instructions end before shared and tensor memory are given back
    if (warp == 13) {
        for (uint32_t i = kissued > KS ? kissued - KS : 0; i < kissued; i++)
            mbar_wait(smem_u32(&kfull[i % KS]), (i / KS) & 1u);
        for (uint32_t i = vissued > VS ? vissued - VS : 0; i < vissued; i++)
            mbar_wait(smem_u32(&vfull[i % VS]), (i / VS) & 1u);
    }
    if (warp == 12 && lane == 0) {
        mma_commit(smem_u32(&drained));
        mbar_wait(smem_u32(&drained), 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc(tm, 512);
}

template <uint32_t D>
static int prompt_launch_d(const AttnArgs &a, cudaStream_t st) {
    DeviceInfo di;
    if (device_info(&di) != DGT_OK) return DGT_ERR_CUDA;
    auto fn = k_kv_prompt<D>;
    static std::atomic<uint64_t> ready;   // devices that allow the shared memory
    const uint64_t bit = di.device < 64 ? 1ull << di.device : 0;
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        if (cudaFuncSetAttribute((const void *)fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)PromptCfg<D>::bytes) != cudaSuccess)
            return DGT_ERR_CUDA;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    const unsigned grid = (unsigned)di.sms < AT_MAX_CTAS ? (unsigned)di.sms : AT_MAX_CTAS;
    return launch_pdl(fn, dim3(grid), dim3(PR_WARPS * 32), PromptCfg<D>::bytes, st, a) == cudaSuccess ? DGT_OK
                                                                                                      : DGT_ERR_CUDA;
}

uint32_t prompt_rows(uint32_t head_dim) { return head_dim <= 128 ? 256 : 128; }

int prompt_launch(const AttnArgs &a, cudaStream_t st) {
    switch (a.c.head_dim) {
        case 64: return prompt_launch_d<64>(a, st);
        case 128: return prompt_launch_d<128>(a, st);
        default: return prompt_launch_d<256>(a, st);
    }
}

}  // namespace dgt
