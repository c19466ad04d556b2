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
// Per CTA two tiles of 128 rows (head_dim 256: one) share every page.  Each has
// two score buffers in tensor memory, so that the scores of the page after
// next are made while its 128 threads (a row each) take exponentials, and the
// threads never wait for a product.  The numerator's reference maximum moves
// only when a row has grown by 2^8 past it, so the accumulators are rarely
// rescaled.
//
// What bounds it: the row threads' exponentials and conversions and the
// dependent steps of a page (issue slots 49 % used, tensor pipe 47 %).  Two
// prompts of 2048 and 1461 rows over 7048 and 5028 tokens, 24 heads of 128:
// 213 us, 1.07 PFLOP/s by what causality leaves of the two products, 55 % of
// the measured bf16 peak.  One of 8192 rows from an empty cache: 373 us.
#include "dgt_attn.cuh"

#include "dgt_tc.cuh"

namespace dgt {

constexpr float PR_W_LOG2 = 4.0f;    // weights at the reference; 2^8 above it they reach 2^12
constexpr float PR_GROW = 8.0f;
constexpr uint32_t PR_WARPS = 15;    // 0-7 rows, 8-11 values to fp16, 12-13 matrix instructions, 14 copies
constexpr uint32_t PR_CONV = 128;    // threads that convert values
constexpr uint32_t PR_META = 16;

template <uint32_t D>
struct PromptCfg {
    static constexpr uint32_t NSTR = D <= 128 ? 2 : 1, RT = 128 * NSTR;   // row tiles of 128
    static constexpr uint32_t RB = D < 128 ? 64 : 128, PAN = D / RB;       // operand row bytes, panels
    static constexpr uint32_t PB = KV_P * D;                               // bytes of a page's block
    static constexpr uint32_t KS = D <= 128 ? 6 : 3, VS = D <= 128 ? 4 : 2, WS = VS;   // stages: keys, values, fp16 values
    static constexpr uint32_t QP = 128 * D;                                // one part of a row tile
    static constexpr uint32_t q = 0, k = q + NSTR * 2 * QP, v = k + KS * PB, w = v + VS * PB,
                              bytes = w + WS * PB * 2 + 1024;
    static constexpr uint32_t SCOL = 256;   // score columns: two buffers of 64 per row tile
    static constexpr uint32_t PART = RT * (D + 4);
};

// A place in a ring of barriers: stage and phase.
struct Ring {
    uint32_t st, ph;
    __device__ __forceinline__ void next(uint32_t n) {
        if (++st == n) st = 0, ph ^= 1;
    }
};

// A page's scales (used 0: it is not there).
struct PageMeta {
    float ks, vs;
    uint32_t used;
};

// Pairs of fp32, two operations an instruction.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(f32x2 x, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void bar_rows() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Two query elements times f0 and f1, to their two e4m3 parts (16 bits each).
// The scaled pair is exact in fp16, down to 2^-31 of the row's largest element.
__device__ __forceinline__ void split2(uint32_t bits, f32x2 f0, f32x2 f1, uint32_t &hi, uint32_t &lo) {
    float x, y;
    unpack2(mul2(mul2(pack2(bf16lo(bits), bf16hi(bits)), f0), f1), x, y);
    const uint32_t h = f16_pair(x, y);
    asm("{\n\t.reg .b16 c, e;\n\t.reg .b32 b, d;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 c, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 b, c;\n\t"
        "sub.rn.f16x2 d, %2, b;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 e, d;\n\t"
        "cvt.u32.u16 %0, c;\n\t"
        "cvt.u32.u16 %1, e;\n\t}"
        : "=r"(hi), "=r"(lo)
        : "r"(h));
}

// A lane's N words of a row, and to shared memory N halfwords.
template <uint32_t N>
__device__ __forceinline__ void load_words(const uint16_t *p, uint32_t (&x)[N]) {
    if constexpr (N == 1) {
        x[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        x[0] = v.x, x[1] = v.y;
    } else {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    }
}
template <uint32_t N>
__device__ __forceinline__ void store_halves(uint32_t addr, const uint32_t (&x)[N]) {
    if constexpr (N == 1)
        asm volatile("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tst.shared.b16 [%0], h;\n\t}" ::"r"(addr), "r"(x[0]) : "memory");
    else if constexpr (N == 2)
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(x[0] | x[1] << 16) : "memory");
    else
        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(x[0] | x[1] << 16), "r"(x[2] | x[3] << 16) : "memory");
}

template <uint32_t D>
__global__ void __launch_bounds__(PR_WARPS * 32, 1) k_kv_prompt(AttnArgs a) {
    using Cfg = PromptCfg<D>;
    constexpr uint32_t NSTR = Cfg::NSTR, RT = Cfg::RT, RB = Cfg::RB, PAN = Cfg::PAN, PB = Cfg::PB, QP = Cfg::QP,
                       KS = Cfg::KS, VS = Cfg::VS, WS = Cfg::WS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t kfull[KS], kfree[KS], vfull[VS], vfree[VS], wfull[WS], wfree[WS];
    __shared__ __align__(8) uint64_t sfull[4], pfull[4], ofull[2], ofin[2], qfull[2], drained;
    __shared__ PageMeta meta[PR_META];
    __shared__ Slot slots[AT_CHUNK];
    __shared__ uint64_t usum[PR_WARPS];
    __shared__ uint32_t tmem_slot;
    __shared__ Cuts shared_cut;
    __shared__ int abort_flag, last_flag;
    // the warp's number out of a shuffle: the compiler then knows that it is the warp's
    const uint32_t tid = threadIdx.x, warp = __shfl_sync(DGT_FULL, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
    if (tid == 0) {
        for (uint32_t i = 0; i < KS; i++) mbar_init(smem_u32(&kfull[i]), 1), mbar_init(smem_u32(&kfree[i]), NSTR);
        for (uint32_t i = 0; i < VS; i++) mbar_init(smem_u32(&vfull[i]), 1), mbar_init(smem_u32(&vfree[i]), PR_CONV / 32);
        for (uint32_t i = 0; i < WS; i++) mbar_init(smem_u32(&wfull[i]), PR_CONV / 32), mbar_init(smem_u32(&wfree[i]), NSTR);
        for (uint32_t i = 0; i < 4; i++) {
            mbar_init(smem_u32(&sfull[i]), 2);
            mbar_init(smem_u32(&pfull[i]), 4);
        }
        for (uint32_t i = 0; i < 2; i++) {
            mbar_init(smem_u32(&ofull[i]), 1);
            mbar_init(smem_u32(&ofin[i]), 1);
            mbar_init(smem_u32(&qfull[i]), 4);
        }
        mbar_init(smem_u32(&drained), NSTR);
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

    Units here = describe<PR_WARPS>(a, RT, 0, slots, usum);
    const Units all = a.slots <= AT_CHUNK ? here : all_units<PR_WARPS>(a, RT, usum);
    // found by one warp, and kept in shared memory: registers are short here
    if (warp == 0) {
        const Cuts k = cut_plan(a, all, slots, gridDim.x);
        if (lane == 0) shared_cut = k;
    }
    __syncthreads();
    const Cuts &cut = shared_cut;
    const uint64_t ub = blockIdx.x >= cut.C ? 0 : cut.parts ? cut.U : cut.raw(blockIdx.x + 1);

    bool dead = false;   // a wait ran out, here or elsewhere in the CTA: no more work from this warp
    // a whole warp's wait for two phases (or one, given twice): the tries overlap
    auto wait_both = [&](uint32_t bar, uint32_t parity, uint32_t bar2, uint32_t parity2) {
        if (dead) return false;
        for (uint32_t i = 0; i < a.spin; i++) {
            bool ok = mbar_try_wait(bar, parity);
            if (bar2 != bar) ok &= mbar_try_wait(bar2, parity2);
            if (__all_sync(DGT_FULL, ok)) return true;
            if ((i & 63) == 63 && *abortp) break;
        }
        dead = true;
        if (lane == 0) set_status(a.status, DGT_ERR_TIMEOUT);
        *abortp = 1;
        return false;
    };
    auto wait_at = [&](uint32_t bar, uint32_t parity) { return wait_both(bar, parity, bar, parity); };
    auto wait = [&](uint64_t &bar, uint32_t parity) { return wait_at(smem_u32(&bar), parity); };
    Ring kr{0, 0}, wr{0, 0};       // the matrix instructions' next stages of keys and fp16 values
    uint32_t it = 0;               // pages so far, the same in every role
    uint32_t qc[2] = {0, 0};       // per row tile: segments, pages so far
    uint32_t sc[2] = {0, 0};
    uint32_t kissued = 0, vissued = 0;   // the copying warp's items

    uint64_t base0 = 0;
    for (uint32_t s0 = 0; s0 < a.slots && base0 < ub; s0 += AT_CHUNK) {
        if (s0) here = describe<PR_WARPS>(a, RT, s0, slots, usum);
        const uint32_t tot = (uint32_t)here.units();
        const uint32_t nslots = min(AT_CHUNK, a.slots - s0);
        const uint64_t chunk_base = base0;
        base0 += tot;
        uint32_t u0, u1;
        cut.share(slots, nslots, chunk_base, tot, u0, u1);
        for (uint32_t u = u0; u < u1;) {
            const Run r = run_at(slots, nslots, a.end, u, u1);
            u += r.units;
            const Slot &s = slots[r.slot];
            const uint32_t n = s.per_head();
            const uint32_t T = s.np ? r.pe - r.pa : 0;
            const uint32_t ns = NSTR == 2 && s.rows > 128 ? 2 : 1;   // row tiles that hold rows

            if (warp == 14) {
                // ---- copies
                int pid = -1;
                float ks = 0.0f, vs = 0.0f;
                for (uint32_t j = 0; j < T && !dead; j++) {
                    const uint32_t x = r.pa + j, c = it + j;
                    if (j % 32 == 0) {
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
                    const int id = __shfl_sync(DGT_FULL, pid, j % 32);
                    const float kk = __shfl_sync(DGT_FULL, ks, j % 32), vv = __shfl_sync(DGT_FULL, vs, j % 32);
                    const uint64_t bi = kv_block(a.c, a.layer, id < 0 ? 0u : (uint32_t)id, r.h);
                    const uint32_t kb = smem_u32(&kfull[c % KS]), vb = smem_u32(&vfull[c % VS]);
                    if (lane == 0) {
                        PageMeta &m = meta[c % PR_META];
                        m.ks = id < 0 ? 1.0f : kk, m.vs = id < 0 ? 1.0f : vv, m.used = id >= 0;
                        if (id >= 0) {
                            mbar_arrive_expect_tx(kb, PB);
                            bulk_g2s(base + Cfg::k + (c % KS) * PB, a.c.k + bi * PB, PB, kb);
                        } else {
                            mbar_arrive(kb);
                        }
                    }
                    kissued = c + 1;
                    if (c >= VS && !wait(vfree[c % VS], (c / VS - 1) & 1u)) break;
                    if (lane == 0) {
                        if (id >= 0) {
                            mbar_arrive_expect_tx(vb, PB);
                            bulk_g2s(base + Cfg::v + (c % VS) * PB, a.c.v + bi * PB, PB, vb);
                        } else {
                            mbar_arrive(vb);
                        }
                    }
                    vissued = c + 1;
                    __syncwarp();
                }
            } else if (warp >= 12) {
                // ---- matrix instructions, a warp for each row tile.  The whole warp walks the pages, one
                // lane issues: page and buffer numbers out of shuffles keep the descriptors in uniform
                // registers (computed by the issuing lane alone they cost 70 cycles an instruction, twice
                // what it runs).
                constexpr uint32_t idesc_s = (1u << 4) | ((KV_P >> 3) << 17) | ((128u >> 4) << 24);
                constexpr uint32_t idesc_o = (1u << 4) | ((D >> 3) << 17) | ((128u >> 4) << 24);
                const uint32_t t = warp - 12;
                const bool leader = elect_one();
                const uint32_t tmu = __shfl_sync(DGT_FULL, tm, 0);
                auto desc = [&](uint32_t addr) { return RB == 128 ? sw128_desc(addr) : sw64_desc(addr); };
                auto commit = [&](uint32_t bar) {
                    if (leader) mma_commit(bar);
                };
                const uint32_t kb0 = smem_u32(kfull), kf0 = smem_u32(kfree), wb0 = smem_u32(wfull), wf0 = smem_u32(wfree);
                const uint32_t sf0 = smem_u32(sfull) + 16 * t, pf0 = smem_u32(pfull) + 16 * t;
                const uint32_t scol = tmu + Cfg::SCOL + 2 * t * KV_P;
                const uint64_t qd = desc(base + Cfg::q + 2 * t * QP), kd = desc(base + Cfg::k);
                const uint64_t wd = sw128_desc(base + Cfg::w);
                // scores with the keys' stage st into buffer n
                auto scores = [&](uint32_t st, uint32_t n) {
                    const uint64_t k0 = kd + st * (PB / 16);
                    const uint32_t col = scol + n * KV_P;
                    if (leader) {
#pragma unroll
                        for (uint32_t part = 0; part < 2; part++)
#pragma unroll
                            for (uint32_t pan = 0; pan < PAN; pan++)
#pragma unroll
                                for (uint32_t i = 0; i < RB / 32; i++)
                                    mma_e4m3(col, qd + (part * QP + pan * 128 * RB) / 16 + 2 * i,
                                             k0 + pan * KV_P * RB / 16 + 2 * i, idesc_s, part + pan + i > 0 ? 1u : 0u);
                        mma_commit(sf0 + 8 * n);
                        // the page's scales, seen here with its keys, are seen behind this barrier too
                        mbar_arrive(sf0 + 8 * n);
                        mma_commit(kf0 + 8 * st);
                    }
                };
                if (t < ns) {
                    // The pipe runs a warp's instructions in order: a buffer's next scores are issued behind
                    // the products that read its weights.
                    for (uint32_t j = 0; j < 2 && j < T; j++) {
                        const uint32_t x = __shfl_sync(DGT_FULL, kr.st | ((sc[t] + j) & 1) << 8, 0);
                        if (!wait_at(kb0 + 8 * kr.st, kr.ph) || (j == 0 && !wait(qfull[t], qc[t] & 1u))) break;
                        tc_fence_after();
                        scores(x & 255, x >> 8);
                        kr.next(KS);
                    }
                    for (uint32_t j = 0; j < T && !dead; j++) {
                        const uint32_t n = sc[t] + j;
                        const uint32_t x = __shfl_sync(DGT_FULL, kr.st | wr.st << 8 | (n & 1) << 16 | (j ? 1u << 24 : 0u), 0);
                        const uint32_t ks = x & 255, ws = x >> 8 & 255, nb = x >> 16 & 1, more = x >> 24;
                        const uint32_t wbar = wb0 + 8 * ws;
                        if (!wait_both(j + 2 < T ? kb0 + 8 * ks : wbar, j + 2 < T ? kr.ph : wr.ph, wbar, wr.ph) ||
                            !wait_at(pf0 + 8 * nb, (n >> 1) & 1u))
                            break;
                        tc_fence_after();
#pragma unroll
                        for (uint32_t i = 0; i < 4; i++)
                            if (leader)
                                mma_f16_ta(tmu + t * D, scol + nb * KV_P + i * 8, wd + ws * (PB * 2 / 16) + 2 * i, idesc_o,
                                           i > 0 ? 1u : more);
                        commit(smem_u32(&ofull[t]));
                        commit(wf0 + 8 * ws);
                        wr.next(WS);
                        if (j + 2 < T) {
                            scores(ks, nb);
                            kr.next(KS);
                        } else if (j + 1 == T) {
                            commit(smem_u32(&ofin[t]));
                        }
                    }
                } else if (t < NSTR) {
                    // no rows: give the pages back as they come
                    for (uint32_t j = 0; j < T; j++) {
                        if (!wait_at(kb0 + 8 * kr.st, kr.ph) || !wait_at(wb0 + 8 * wr.st, wr.ph)) break;
                        if (leader) {
                            mbar_arrive(kf0 + 8 * kr.st);
                            mbar_arrive(wf0 + 8 * wr.st);
                        }
                        kr.next(KS);
                        wr.next(WS);
                    }
                }
                __syncwarp();
            } else if (warp >= 8) {
                // ---- value pages to fp16 operand tiles: rows of 64 tokens, 128-byte swizzle
                const uint32_t ct = tid - 256;
                for (uint32_t j = 0; j < T && !dead; j++) {
                    const uint32_t c = it + j;
                    const uint32_t vb = smem_u32(&vfull[c % VS]), wb = smem_u32(&wfree[c % WS]);
                    if (!wait_both(vb, (c / VS) & 1u, c >= WS ? wb : vb, c >= WS ? (c / WS - 1) & 1u : 0u)) break;
                    const uint32_t src = base + Cfg::v + (c % VS) * PB, dst = base + Cfg::w + (c % WS) * PB * 2;
                    const bool used = meta[c % PR_META].used != 0;
                    // 16 bytes a thread: row ct / 4 (and every 32nd from there), tokens 16 (ct % 4) ..
                    constexpr uint32_t B = D * 4 / PR_CONV < 4 ? D * 4 / PR_CONV : 4;
                    static_assert(D * 4 % (B * PR_CONV) == 0, "a page's pieces divide evenly over the threads");
                    const uint32_t row = ct >> 2, q = ct & 3, o0 = dst + row * 128 + (((2 * q) ^ (row & 7)) << 4);
                    const uint32_t o1 = dst + row * 128 + (((2 * q + 1) ^ (row & 7)) << 4);
#pragma unroll
                    for (uint32_t i0 = 0; i0 < D * 4 / PR_CONV; i0 += B) {
                        uint4 x[B];
#pragma unroll
                        for (uint32_t i = 0; i < B; i++) {
                            x[i] = make_uint4(0, 0, 0, 0);
                            if (used) x[i] = lds128(src + ct * 16 + (i0 + i) * PR_CONV * 16);
                        }
#pragma unroll
                        for (uint32_t i = 0; i < B; i++) {
                            const uint32_t k = (i0 + i) * (PR_CONV / 4) * 128;
                            sts128(o0 + k, e4m3_lo(x[i].x), e4m3_hi(x[i].x), e4m3_lo(x[i].y), e4m3_hi(x[i].y));
                            sts128(o1 + k, e4m3_lo(x[i].z), e4m3_hi(x[i].z), e4m3_lo(x[i].w), e4m3_hi(x[i].w));
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
                const uint32_t qt = base + Cfg::q + 2 * t * QP;   // the row tile's operand, later its output
                if (mine && T) {
                    // A row by the whole warp, so that a load touches one row's lines, IN rows in flight.  With a
                    // thread per row every load touched 32 lines and a segment of 128 dimensions took 9000 to
                    // 11000 cycles here; so it takes 6500 to 7000.
                    constexpr uint32_t W = D / 64, IN = 32 / W;
                    const uint32_t first = t * 128 + quad * 32, f0 = s.row0 + first;
                    const uint32_t count = s.rows > first ? min(s.rows - first, 32u) : 0;
                    uint32_t head = f0 % a.group, mytop = 0;
                    const uint16_t *qp = a.q.data + (int64_t)(s.tok0 + f0 / a.group) * a.q.token_stride +
                                         (int64_t)(r.h * a.group + head) * a.q.head_stride + lane * 2 * W;
                    const int64_t wrap = a.q.token_stride - (int64_t)(a.group - 1) * a.q.head_stride;
                    const uint32_t d = lane * 2 * W, chunk = (d % RB) / 16;   // the lane's first dimension
                    const uint32_t col = qt + d / RB * 128 * RB + d % 16;
#pragma unroll 1
                    for (uint32_t i0 = 0; i0 < 32; i0 += IN) {
                        uint32_t x[IN][W];
#pragma unroll
                        for (uint32_t i = 0; i < IN; i++) {
                            if (i0 + i < count) {
                                load_words<W>(qp, x[i]);
                                const bool last = ++head == a.group;
                                qp += last ? wrap : a.q.head_stride;
                                if (last) head = 0;
                            } else {
#pragma unroll
                                for (uint32_t k = 0; k < W; k++) x[i][k] = 0;
                            }
                        }
#pragma unroll
                        for (uint32_t i = 0; i < IN; i++) {
                            uint32_t top = x[i][0] & 0x7FFF7FFFu;
#pragma unroll
                            for (uint32_t k = 1; k < W; k++) top = __vmaxu2(top, x[i][k] & 0x7FFF7FFFu);
                            top = __reduce_max_sync(DGT_FULL, max(top & 0xFFFFu, top >> 16)) >> 7;
                            if (lane == i0 + i) mytop = top;
                            // the largest element to [2^7, 2^8); one that is not finite: the row's factor says so
                            const int up = 7 + 127 - (int)top, up0 = min(up, 100);
                            float a0 = __uint_as_float((uint32_t)(up0 + 127) << 23);
                            const float a1 = __uint_as_float((uint32_t)(up - up0 + 127) << 23);
                            if (a.scale_log2 < 0.0f) a0 = -a0;
                            const f32x2 m0 = pack2(a0, a0), m1 = pack2(a1, a1);
                            uint32_t hi[W], lo[W];
#pragma unroll
                            for (uint32_t k = 0; k < W; k++) split2(top == 255 ? 0u : x[i][k], m0, m1, hi[k], lo[k]);
                            const uint32_t rr = quad * 32 + i0 + i, sw = RB == 128 ? rr & 7 : (rr >> 1) & 3;
                            const uint32_t at = col + rr * RB + ((chunk ^ sw) << 4);
                            store_halves<W>(at, hi);
                            store_halves<W>(at + QP, lo);
                        }
                    }
                    fac = mytop == 255 ? __uint_as_float(0x7FC00000u) : ldexpf(fabsf(a.scale_log2), (int)mytop - 134);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&qfull[t]));
                }
                const int32_t pf = s.pos0 + (int32_t)(s.row0 / a.group);
                const int32_t pl = s.pos0 + (int32_t)((s.row0 + s.rows - 1) / a.group);
                for (uint32_t j = 0; mine && j < T && !dead; j++) {
                    const uint32_t c = it + j, sn = sc[t] + j, sb = 2 * t + (sn & 1);
                    if (!wait(sfull[sb], (sn >> 1) & 1u)) break;
                    tc_fence_after();
                    const uint32_t st = tm + tl + Cfg::SCOL + sb * KV_P;
                    uint32_t sv[64];
                    tmem_ld64(st, sv);
                    // the page's factors, and which of its 64 tokens the row sees
                    const PageMeta &mt = meta[c % PR_META];
                    const float vs = mt.vs, ev = (float)((int)(__float_as_uint(vs) >> 23) - 127);
                    float f = fac * mt.ks;
                    if (f == 0.0f) f = 1e-30f;   // scores of zero, also for what is set to -inf below
                    const bool used = mt.used != 0;
                    const int32_t t0 = (int32_t)(s.page_index(r.pa + j) * KV_P);
                    const bool whole = used && t0 + (int32_t)KV_P - 1 <= pf &&
                                       (!a.window || t0 > pl - (int32_t)a.window || (uint32_t)t0 + KV_P <= a.sinks);
                    uint64_t see = ~0ull;
                    if (!whole) {
                        const int32_t hi = used ? min(max(pos - t0 + 1, 0), 64) : 0;   // tokens [0, hi) are not ahead of the row
                        const int32_t lo = a.window ? min(max(pos - (int32_t)a.window + 1 - t0, 0), 64) : 0;
                        const int32_t sk = a.window ? min(max((int32_t)a.sinks - t0, 0), 64) : 0;
                        const uint64_t below_hi = hi >= 64 ? ~0ull : (1ull << hi) - 1;
                        const uint64_t below_lo = lo >= 64 ? ~0ull : (1ull << lo) - 1;
                        const uint64_t below_sk = sk >= 64 ? ~0ull : (1ull << sk) - 1;
                        see = below_hi & (~below_lo | below_sk);
                    }
                    tmem_wait_ld();
                    if (!whole) {
#pragma unroll
                        for (int i = 0; i < 64; i++)
                            if (!((see >> i) & 1u)) sv[i] = 0xFF800000u;
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 64; i += 8)
#pragma unroll
                        for (int k = 0; k < 4; k++)
                            mx[k] = fmaxf(fmaxf(mx[k], __uint_as_float(sv[i + k])), __uint_as_float(sv[i + 4 + k]));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    const float tx = top == -INFINITY ? top : top * f;
                    const float mn = fmaxf(m, tx), un = fmaxf(mu, tx + ev);
                    const float bm = finite_base(mn);
                    l *= ex2(m - bm);
                    m = mn;
                    const bool grow = un > mu + PR_GROW || (mu == -INFINITY && un > -INFINITY);
                    const float ao = grow ? ex2(mu - un) : 1.0f;
                    if (grow) mu = un;
                    const float bu = finite_base(mu);
                    // weights: the value's scale inside the exponent, and their sum freed of it
                    const float lc = bm + ev - bu + PR_W_LOG2;
                    const bool fast = __all_sync(DGT_FULL, fabsf(lc) < 40.0f && vs == vs && f == f);
                    const float bb = fast ? lc - bm : -bm;
                    const f32x2 f2 = pack2(f, f), b2 = pack2(bb, bb);
                    f32x2 sum[2] = {0ull, 0ull};
                    uint32_t pk[32];
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        float x, y;
                        unpack2(fma2(pack2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])), f2, b2), x, y);
                        x = ex2(x);
                        y = ex2(y);
                        sv[2 * i] = __float_as_uint(x);
                        sv[2 * i + 1] = __float_as_uint(y);
                        sum[i & 1] = add2(sum[i & 1], pack2(x, y));
                        pk[i] = f16_pair(x, y);
                    }
                    float all;
                    {
                        float x, y;
                        unpack2(add2(sum[0], sum[1]), x, y);
                        all = x + y;
                    }
                    if (!fast) {
                        // scales that are not finite or far apart: weights and their sum one by one, and none
                        // for a token that the row does not see, whatever its scales are
                        const float cw = vs != vs ? vs : ex2(fminf(lc, 126.0f));
                        all = 0.0f;
#pragma unroll
                        for (int i = 0; i < 32; i++) {
                            const float x = (see >> (2 * i)) & 1u ? __uint_as_float(sv[2 * i]) : 0.0f;
                            const float y = (see >> (2 * i + 1)) & 1u ? __uint_as_float(sv[2 * i + 1]) : 0.0f;
                            all += x + y;
                            pk[i] = f16_pair((see >> (2 * i)) & 1u ? x * cw : 0.0f, (see >> (2 * i + 1)) & 1u ? y * cw : 0.0f);
                        }
                    }
                    tmem_st32(st, pk);
                    l += fast ? all * ex2(-lc) : all;
                    if (j > 0 && __any_sync(DGT_FULL, grow)) {
                        // The accumulators may move once the products of the page before are done.  Those of
                        // the page before that are: this page's scores came behind them, so the phase is the
                        // next of the barrier or the one just past.
                        if (!wait(ofull[t], (sn - 1) & 1u)) break;
                        tc_fence_after();
#pragma unroll 1
                        for (uint32_t d0 = 0; d0 < D; d0 += 32) {
                            uint32_t o[32];
                            tmem_ld32(tm + tl + t * D + d0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * ao);
                            tmem_st32(tm + tl + t * D + d0, o);
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&pfull[sb]));
                }
                tmem_wait_st();   // weights of a page whose wait ran out

                // ---- the segment's end: this row's quotient, or its part
                const bool complete = r.pa == 0 && r.pe == n;
                if (mine && T) wait(ofin[t], qc[t] & 1u);
                tc_fence_after();
                const bool none = m == -INFINITY && l == 0.0f;
                const uint32_t orow = (s.tok0 + flat / a.group) * a.q_heads + r.h * a.group + flat % a.group;
                // Output rows pass through the warp's 32 rows of the operand, which nothing reads any more, and
                // leave it a row's lines at a time.
                auto chunk_at = [&](uint32_t row, uint32_t e) {   // 16 bytes of output row `row` of the tile
                    const uint32_t rr = row & 127, c = (e % (RB / 16)) ^ (RB == 128 ? rr & 7 : (rr >> 1) & 3);
                    return base + Cfg::q + row / 128 * 2 * QP + e / (RB / 16) * 128 * RB + rr * RB + (c << 4);
                };
                auto put = [&](uint32_t row, uint32_t d0, const float (&o)[32], float f) {
#pragma unroll
                    for (uint32_t i = 0; i < 4; i++)
                        sts128(chunk_at(row, d0 / 8 + i), bf16x2(o[8 * i] * f, o[8 * i + 1] * f),
                               bf16x2(o[8 * i + 2] * f, o[8 * i + 3] * f), bf16x2(o[8 * i + 4] * f, o[8 * i + 5] * f),
                               bf16x2(o[8 * i + 6] * f, o[8 * i + 7] * f));
                };
                auto put_out = [&]() {
                    __syncwarp();
#pragma unroll 4
                    for (uint32_t k = 0; k < D / 8; k++) {
                        const uint32_t i = (k * 32 + lane) / (D / 8), e = (k * 32 + lane) % (D / 8), ri = t * 128 + quad * 32 + i;
                        const uint32_t o = __shfl_sync(DGT_FULL, orow, i);
                        const uint4 x = lds128(chunk_at(ri, e));
                        if (ri < s.rows) reinterpret_cast<uint4 *>(a.out + (uint64_t)o * D)[e] = x;
                    }
                    __syncwarp();
                };
                // A part: four dimensions of all rows after four, then M, MU, L of all rows.
                float4 *part = reinterpret_cast<float4 *>(a.part + (2 * (uint64_t)blockIdx.x + (r.pa == 0 ? 1 : 0)) * Cfg::PART) + row;
                if (mine && !dead) {
                    const float quot = none ? 0.0f : ex2(finite_base(mu) - finite_base(m) - PR_W_LOG2) / l;
#pragma unroll 1
                    for (uint32_t d0 = 0; d0 < D; d0 += 32) {
                        float o[32] = {};
                        if (T) {
                            uint32_t w[32];
                            tmem_ld32(tm + tl + t * D + d0, w);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i++) o[i] = __uint_as_float(w[i]);
                        }
                        if (complete) {
                            put(row, d0, o, quot);
                        } else if (live) {
#pragma unroll
                            for (int i = 0; i < 8; i++)
                                part[(d0 / 4 + i) * RT] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        }
                        __syncwarp();   // the next load is the whole warp's
                    }
                    if (complete) put_out();
                    if (live && complete && a.lse) a.lse[orow] = none ? -INFINITY : (m + __log2f(l)) * LN2;
                    if (live && !complete) part[D / 4 * RT] = make_float4(m, mu, l, 0.0f);
                }
                tc_fence_before();
                if (!complete) {
                    // The last CTA of the segment to arrive adds its parts in page order: GR threads a row, each
                    // for D / GR of its dimensions, as many as the tile's rows leave.
                    const uint64_t sa = chunk_base + s.base + (uint64_t)r.h * (n + a.end), sb = sa + n + a.end;
                    uint32_t c0, c1;
                    cut.holders(sa, sb, c0, c1);
                    bar_rows();
                    if (tid == 0) last_flag = arrive_last(&a.count[c0], c1 - c0 + 1);
                    bar_rows();
                    if (last_flag) {
                        const uint32_t lrows = s.rows > 128 ? 8 : s.rows > 64 ? 7 : s.rows > 32 ? 6 : 5;   // log2 of rows, padded
                        const uint32_t jr = tid & ((1u << lrows) - 1), gr = tid >> lrows, groups = 256u >> lrows;
                        const bool jlive = jr < s.rows;
                        // part 0 is the one that begins the segment, at the end of its CTA's work
                        const float4 *p0 = reinterpret_cast<const float4 *>(a.part + (2 * (uint64_t)c0 + 1) * Cfg::PART) + (jlive ? jr : 0);
                        const float4 *p1 = reinterpret_cast<const float4 *>(a.part + 2 * ((uint64_t)c0 + 1) * Cfg::PART) + (jlive ? jr : 0);
                        const uint32_t parts = c1 - c0 + 1;
                        auto at = [&](uint32_t k) { return k ? p1 + (uint64_t)(k - 1) * (2 * Cfg::PART / 4) : p0; };
                        auto out_row = [&](uint32_t row) {
                            const uint32_t f = s.row0 + row;
                            return (uint64_t)(s.tok0 + f / a.group) * a.q_heads + r.h * a.group + f % a.group;
                        };
                        float M = -INFINITY, MU = -INFINITY, L = 0.0f;
#pragma unroll 8
                        for (uint32_t k = 0; k < parts; k++) {
                            const float4 st = __ldcg(at(k) + D / 4 * RT);
                            const float mn = fmaxf(M, st.x), bm = finite_base(mn);
                            L = L * ex2(M - bm) + st.z * ex2(st.x - bm);
                            M = mn;
                            MU = fmaxf(MU, st.y);
                        }
                        const bool nothing = M == -INFINITY && L == 0.0f;
                        const float bu = finite_base(MU), quot = nothing ? 0.0f : ex2(bu - finite_base(M) - PR_W_LOG2) / L;
                        if (jlive && gr == 0 && a.lse) a.lse[out_row(jr)] = nothing ? -INFINITY : (M + __log2f(L)) * LN2;
#pragma unroll 1
                        for (uint32_t d0 = gr * 32; jlive && d0 < D; d0 += groups * 32) {
                            float o[32] = {};
#pragma unroll 2
                            for (uint32_t k = 0; k < parts; k++) {
                                const float4 *p = at(k);
                                float4 x[8];
#pragma unroll
                                for (uint32_t i = 0; i < 8; i++) x[i] = __ldcg(p + (d0 / 4 + i) * RT);
                                const float w = ex2(__ldcg(p + D / 4 * RT).y - bu);
#pragma unroll
                                for (uint32_t i = 0; i < 8; i++) {
                                    o[4 * i] += x[i].x * w, o[4 * i + 1] += x[i].y * w;
                                    o[4 * i + 2] += x[i].z * w, o[4 * i + 3] += x[i].w * w;
                                }
                            }
                            put(jr, d0, o, quot);
                        }
                        bar_rows();
                        for (uint32_t i = tid; i < s.rows * (D / 8); i += 256) {
                            const uint32_t row = i / (D / 8), e = i % (D / 8);
                            reinterpret_cast<uint4 *>(a.out + out_row(row) * D)[e] = lds128(chunk_at(row, e));
                        }
                        bar_rows();   // the rows' places are free for the next queries
                    }
                }
            }
            it += T;
            for (uint32_t t = 0; t < ns; t++) sc[t] += T, qc[t] += T ? 1 : 0;
        }
    }

    // copies land and matrix instructions end before shared and tensor memory are given back
    if (warp == 14) {
        for (uint32_t i = kissued > KS ? kissued - KS : 0; i < kissued; i++)
            mbar_wait(smem_u32(&kfull[i % KS]), (i / KS) & 1u);
        for (uint32_t i = vissued > VS ? vissued - VS : 0; i < vissued; i++)
            mbar_wait(smem_u32(&vfull[i % VS]), (i / VS) & 1u);
    }
    if (warp >= 12 && warp < 12 + NSTR) {
        // committed by the lane that issued the instructions
        if (elect_one()) mma_commit(smem_u32(&drained));
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
    const unsigned grid = std::min((unsigned)di.sms, AT_MAX_SMS);
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
