// dgt_attn.cu -- attention over the paged 8-bit cache.
//
// For a query row q at position p and the positions j that it sees,
//   t_j = scale * q . k_j,   out = sum_j e^(t_j - m) v_j / sum_j e^(t_j - m),
// in one pass over the cache with the running maximum m: when a page raises
// it, the sums so far are multiplied by e^(old - new).
#include "dgt_kv.cuh"

#include "dgt_device.cuh"

namespace dgt {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

struct AttnArgs {
    dgt_kv_cache c;
    uint32_t layer, batch, q_heads, window, sinks;
    uint64_t tokens;
    dgt_heads q;
    const int32_t *seqs, *cu;
    float scale_log2;   // scale * log2(e)
    uint16_t *out;
    float *lse;
    int32_t *status;
};

__device__ __forceinline__ float e4m3_f32(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)c, __NV_E4M3)));
}

// One warp per (row, query head).  Lane l scores tokens l and l + 32 of a
// page, then owns dimensions l, l + 32, ... of the output.
template <uint32_t D>
__global__ void __launch_bounds__(128) k_kv_attention_rows(AttnArgs a) {
    __shared__ float qs[4][D];
    __shared__ float ps[4][KV_P];
    pdl_trigger();
    pdl_wait();
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t item = (uint64_t)blockIdx.x * 4 + warp;
    if (item >= a.tokens * a.q_heads) return;
    const uint64_t row = item / a.q_heads;
    const uint32_t h = (uint32_t)(item % a.q_heads), hk = h / (a.q_heads / a.c.kv_heads);
    uint32_t b = (uint32_t)row, i = 0, n = 1;
    if (a.cu) {
        uint32_t lo = 0, hi = a.batch;   // the last entry that starts at or before the row
        while (hi - lo > 1) {
            const uint32_t mid = (lo + hi) >> 1;
            if ((uint64_t)a.cu[mid] <= row) lo = mid;
            else hi = mid;
        }
        b = lo;
        i = (uint32_t)row - (uint32_t)a.cu[b];
        n = (uint32_t)(a.cu[b + 1] - a.cu[b]);
    }
    const int32_t seq = a.seqs[b];
    int64_t pos = -1;
    if (seq < 0 || (uint32_t)seq >= a.c.max_seqs) {
        if (lane == 0) set_status(a.status, DGT_ERR_ARG);
    } else {
        int64_t len = a.c.lens[seq];
        if (len < 0 || len > (int64_t)a.c.max_pages * KV_P) {
            if (lane == 0) set_status(a.status, DGT_ERR_ARG);
            len = 0;
        }
        if (len > 0) pos = len - n + i;
    }
    const uint16_t *q = a.q.data + (int64_t)row * a.q.token_stride + (int64_t)h * a.q.head_stride;
    for (uint32_t d = lane; d < D; d += 32) qs[warp][d] = __uint_as_float((uint32_t)q[d] << 16);
    __syncwarp();
    float m = -INFINITY, l = 0.0f, acc[D / 32];
#pragma unroll
    for (uint32_t j = 0; j < D / 32; j++) acc[j] = 0.0f;
    const int64_t lo = a.window && pos >= (int64_t)a.window ? pos - a.window + 1 : 0;   // the window's first position
    const int64_t sinks = min((int64_t)a.sinks, lo);
    for (int64_t t0 = 0; t0 <= pos; t0 += KV_P) {
        if (t0 >= sinks && t0 + KV_P <= lo) {
            t0 = lo / KV_P * KV_P;
            if (t0 > pos) break;
        }
        const int32_t page = a.c.table[(uint64_t)seq * a.c.max_pages + t0 / KV_P];
        if (page < 0 || (uint32_t)page >= a.c.pages) {
            if (lane == 0) set_status(a.status, DGT_ERR_ARG);
            continue;
        }
        const uint64_t bi = kv_block(a.c, a.layer, (uint32_t)page, hk);
        const uint8_t *kb = a.c.k + bi * (KV_P * D), *vb = a.c.v + bi * (KV_P * D);
        const float ks = a.c.k_scale[bi], vs = a.c.v_scale[bi];
        float t[2], mx = m;
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const uint32_t tok = lane + 32 * e;
            float s = 0.0f;
            for (uint32_t d = 0; d < D; d += 16) {
                const uint4 u = *reinterpret_cast<const uint4 *>(kb + kv_k_off(D, tok, d));
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 16; j++)
                    s = fmaf(qs[warp][d + j], e4m3_f32((uint8_t)(w[j / 4] >> (8 * (j & 3)))), s);
            }
            const int64_t j = t0 + tok;
            const bool see = j <= pos && (j >= lo || j < sinks);
            t[e] = see ? s * (ks * a.scale_log2) : -INFINITY;
            mx = fmaxf(mx, t[e]);
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(DGT_FULL, mx, d));
        const float base = mx == -INFINITY ? 0.0f : mx;
        const float alpha = exp2f(m - base);
        m = mx;
        __syncwarp();
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 2; e++) {
            const float p = exp2f(t[e] - base);
            ps[warp][lane + 32 * e] = p;
            sum += p;
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(DGT_FULL, sum, d);
        l = l * alpha + sum;
        __syncwarp();
#pragma unroll
        for (uint32_t j = 0; j < D / 32; j++) {
            const uint32_t d = lane + 32 * j;
            float s = 0.0f;
            for (uint32_t tok = 0; tok < KV_P; tok += 16) {
                const uint4 u = *reinterpret_cast<const uint4 *>(vb + kv_v_off(tok, d));
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int k = 0; k < 16; k++)
                    s = fmaf(ps[warp][tok + k], e4m3_f32((uint8_t)(w[k / 4] >> (8 * (k & 3)))), s);
            }
            acc[j] = acc[j] * alpha + (sum == 0.0f ? 0.0f : s * vs);   // a page that the row sees nothing of adds nothing
        }
    }
    uint16_t *out = a.out + (row * a.q_heads + h) * D;
    const bool none = m == -INFINITY && l == 0.0f;
#pragma unroll
    for (uint32_t j = 0; j < D / 32; j++) out[lane + 32 * j] = f32_to_bf16_rne(none ? 0.0f : acc[j] / l);
    if (a.lse && lane == 0) a.lse[row * a.q_heads + h] = none ? -INFINITY : (m + log2f(l)) * LN2;
}

}  // namespace dgt

using namespace dgt;

extern "C" size_t dgt_kv_attention_workspace_bytes(const dgt_kv_cache *cache, uint32_t q_heads, uint32_t batch,
                                                   uint64_t tokens) {
    (void)cache, (void)q_heads, (void)batch, (void)tokens;
    return 0;
}

extern "C" int dgt_kv_attention(const dgt_kv_cache *cache, uint32_t layer, const dgt_heads *q, uint64_t tokens,
                                const int32_t *d_seqs, const int32_t *d_cu, uint32_t batch, float scale,
                                uint32_t window, uint32_t sinks, uint16_t *d_out, float *d_lse, void *d_ws,
                                size_t ws_bytes, int32_t *d_status, void *stream) {
    int rc = kv_check(cache);
    if (rc != DGT_OK) return rc;
    if (!q || layer >= cache->layers) return DGT_ERR_ARG;
    if ((rc = batch_check(tokens, batch, d_cu)) != DGT_OK) return rc;
    if (tokens == 0 || batch == 0) return DGT_OK;
    if (!d_seqs || !d_out || !aligned16(d_out)) return DGT_ERR_ARG;
    if (q->heads == 0 || q->heads % cache->kv_heads || q->heads / cache->kv_heads > 64) return DGT_ERR_SHAPE;
    if ((rc = heads_check(q, q->heads)) != DGT_OK) return rc;
    if (ws_bytes < dgt_kv_attention_workspace_bytes(cache, q->heads, batch, tokens)) return DGT_ERR_ARG;
    (void)d_ws;
    AttnArgs a{*cache, layer, batch, q->heads, window, window ? sinks : 0u, tokens, *q, d_seqs, d_cu, scale * LOG2E,
               d_out, d_lse, d_status};
    auto fn = cache->head_dim == 64    ? k_kv_attention_rows<64>
              : cache->head_dim == 128 ? k_kv_attention_rows<128>
                                       : k_kv_attention_rows<256>;
    const uint64_t items = tokens * q->heads;
    return launch_pdl(fn, dim3((unsigned)((items + 3) / 4)), dim3(128), 0, (cudaStream_t)stream, a) == cudaSuccess
               ? DGT_OK
               : DGT_ERR_CUDA;
}
