// dgt_kv.cuh -- the paged 8-bit cache as its kernels see it: block layout,
// sequence lookup, and the checks every entry point shares.
#pragma once
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dgt.h"
#include "dgt_launch.h"

namespace dgt {

constexpr uint32_t KV_P = DGT_KV_PAGE;
constexpr int KV_EMIN = -100;   // smallest exponent of a scale
constexpr uint64_t KV_MAX_TOKENS = 1ull << 24;
constexpr uint32_t KV_MAX_BATCH = 65536;

// Byte of (token t, dimension d) in a key block: panels of 128 dimensions (one
// of 64 when D is 64), the 16-byte chunks of a row permuted by its token so
// that eight rows read at one chunk, or 16-byte chunks of neighbouring rows,
// fall into different shared-memory banks.  It is the 128-byte (64-byte)
// swizzle of the tensor cores' operand tiles: a block copied to shared memory
// as it stands is one.
__host__ __device__ inline uint32_t kv_k_off(uint32_t D, uint32_t t, uint32_t d) {
    if (D == 64) return t * 64 + ((((d >> 4) ^ (t >> 1)) & 3) << 4) + (d & 15);
    return (d >> 7) * (KV_P * 128) + t * 128 + (((((d >> 4) & 7) ^ t) & 7) << 4) + (d & 15);
}

// Byte of (token t, dimension d) in a value block.
__host__ __device__ inline uint32_t kv_v_off(uint32_t t, uint32_t d) { return d * KV_P + t; }

// Block index of (layer, page, head); a block is KV_P * head_dim bytes.
__host__ __device__ inline uint64_t kv_block(const dgt_kv_cache &c, uint32_t layer, uint32_t page, uint32_t head) {
    return ((uint64_t)layer * c.pages + page) * c.kv_heads + head;
}

static inline int kv_check(const dgt_kv_cache *c) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->refs || !c->table || !c->lens) return DGT_ERR_ARG;
    if (!aligned16(c->k) || !aligned16(c->v)) return DGT_ERR_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return DGT_ERR_SHAPE;
    if (c->kv_heads == 0 || c->kv_heads > 256 || c->layers == 0 || c->layers > (1u << 16)) return DGT_ERR_SHAPE;
    if (c->pages == 0 || c->pages > (1u << 22)) return DGT_ERR_SHAPE;
    if (c->max_seqs == 0 || c->max_seqs > (1u << 20) || c->max_pages == 0 || c->max_pages > (1u << 16))
        return DGT_ERR_SHAPE;
    return DGT_OK;
}

// A strided tensor of `heads` heads that 16-byte loads can walk.
static inline int heads_check(const dgt_heads *x, uint32_t heads) {
    if (!x || !x->data || !aligned16(x->data) || (x->token_stride & 7) || (x->head_stride & 7)) return DGT_ERR_ARG;
    if (x->heads != heads) return DGT_ERR_ARG;
    return DGT_OK;
}

static inline int batch_check(uint64_t tokens, uint32_t batch, const int32_t *cu) {
    if (tokens > KV_MAX_TOKENS || batch > KV_MAX_BATCH) return DGT_ERR_SHAPE;
    if ((!cu || batch == 0) && tokens != batch) return DGT_ERR_ARG;
    return DGT_OK;
}

// Items of up to `step` rows cut from the entries of a batch (each of their
// tokens `mult` rows), numbered without a prefix sum: entry b's items are
// numbered from floor(cu[b] * mult / step) + per * b on.  Consecutive entries
// are then at least floor(rows_b / step) + per numbers apart, so `per` = 1 has
// room for the ceil(rows_b / step) pieces of an entry and per = 2 for the
// blocks that it touches wherever it starts; numbers past an entry's pieces
// are empty.  The count of numbers is known on the host:
// floor(tokens * mult / step) + per * batch.
__device__ __forceinline__ uint32_t item_base(const int32_t *cu, uint32_t b, uint32_t step, uint32_t per,
                                              uint32_t mult = 1) {
    return (uint32_t)((uint64_t)(uint32_t)cu[b] * mult / step) + per * b;
}
__device__ __forceinline__ uint32_t item_entry(const int32_t *cu, uint32_t batch, uint32_t item, uint32_t step,
                                               uint32_t per, uint32_t mult = 1) {
    uint32_t lo = 0, hi = batch;   // the last b with item_base(b) <= item
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if (item_base(cu, mid, step, per, mult) <= item) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace dgt
