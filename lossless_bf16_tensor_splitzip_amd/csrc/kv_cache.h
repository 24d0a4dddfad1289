// kv_cache.h -- what the kernels and entry points of the paged key-value cache
// have in common: the cache as kernels see it, divisions by a constant of the
// launch, wave scans, and the checks of a cache's arguments.
#ifndef SPLITZIP_CSRC_KV_CACHE_H
#define SPLITZIP_CSRC_KV_CACHE_H

#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "splitzip_kv.h"

namespace {

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31 as a multiplication: with
// s = ceil(log2 d) and m = floor(2^(31+s) / d) + 1, m d exceeds 2^(31+s) by at
// most d <= 2^s, so n m / 2^(31+s) exceeds n / d by less than n / (2^31 d) <
// 1 / d and has the same floor.
struct Div {
    uint32_t m, sh, d;
};
inline Div make_div(uint32_t d) {
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    return Div{(uint32_t)(((unsigned __int128)1 << (31 + s)) / d + 1), 31 + s, d};
}
__device__ inline uint32_t div(uint32_t n, Div v) {
    return (uint32_t)(((uint64_t)n * v.m) >> v.sh);
}

// A cache as the kernels see it (strides in elements).
struct Cache {
    uint16_t *k, *v;
    uint64_t ks[3], vs[3];
    const int32_t *table;
    uint64_t table_stride;
    int32_t *lens;
    Div page;
    uint32_t num_pages, kv_heads, dim, batch, max_len;
};

__device__ inline void report(int32_t *status, int32_t bits) {
    if (status) atomicOr(status, bits);
}

// The sequence's length, within what its table holds.
__device__ inline uint32_t seq_len(const Cache &c, uint32_t b, int32_t *status = nullptr) {
    const int32_t n = c.lens[b];
    if (n < 0 || (uint32_t)n > c.max_len) {
        report(status, SPLITZIP_KV_BAD_LEN);
        return n < 0 ? 0u : c.max_len;
    }
    return (uint32_t)n;
}

// Page and slot of token t < max_len of sequence b; false for a page number
// outside the pool.
__device__ inline bool locate(const Cache &c, uint32_t b, uint32_t t, uint32_t &page,
                              uint32_t &slot) {
    const uint32_t p = div(t, c.page);
    slot = t - p * c.page.d;
    page = (uint32_t)c.table[b * c.table_stride + p];
    return page < c.num_pages;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Until every vector memory operation this wave issued has completed.
// (The builtin, which the compiler counts; after an asm it would wait again
// before every load into a register that a store has read.)
__device__ inline void wait_vector_memory() { __builtin_amdgcn_s_waitcnt(0); }

// 16 bytes that nothing reads again soon.
__device__ inline u32x4 load_once(const uint16_t *p) { return __builtin_nontemporal_load((const u32x4 *)p); }
__device__ inline void store_away(uint16_t *p, u32x4 x) { __builtin_nontemporal_store(x, (u32x4 *)p); }

// Running sum over the wave's lanes: within rows of 16 by shifts, then the
// rows before.
__device__ inline uint32_t wave_scan(uint32_t x) {
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xf, 0xf, false);    // row_shr:1
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xf, 0xf, false);    // row_shr:2
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xf, 0xf, false);    // row_shr:4
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xf, 0xf, false);    // row_shr:8
    const uint32_t r0 = __builtin_amdgcn_readlane(x, 15), r1 = __builtin_amdgcn_readlane(x, 31),
                   r2 = __builtin_amdgcn_readlane(x, 47), row = (threadIdx.x & 63) >> 4;
    return x + (row == 0 ? 0 : row == 1 ? r0 : row == 2 ? r0 + r1 : r0 + r1 + r2);
}

// Set lanes of the mask below this one.
__device__ inline uint32_t lanes_below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

inline int launched() { return hipGetLastError() == hipSuccess ? SPLITZIP_OK : SPLITZIP_ERR_HIP; }

constexpr uint64_t kMaxOffset = 1ull << 40;      // elements

// count - 1 steps of `stride` stay below the limit (no overflow on the way)
inline bool spans(uint64_t stride, uint64_t count) {
    return count <= 1 || stride <= kMaxOffset / (count - 1);
}

inline bool shape_ok(const splitzip_kv_cache *c) {
    return c && c->head_dim >= 8 && c->head_dim <= SPLITZIP_KV_MAX_DIM && c->head_dim % 8 == 0 &&
           c->kv_heads >= 1 && c->kv_heads <= SPLITZIP_KV_MAX_KV_HEADS && c->page_size >= 1 &&
           c->page_size <= SPLITZIP_KV_MAX_PAGE && c->batch <= SPLITZIP_KV_MAX_BATCH &&
           (uint64_t)c->max_pages * c->page_size < (1ull << 31) &&
           (c->dtype == SPLITZIP_KV_BF16 || c->dtype == SPLITZIP_KV_FP16);
}

inline bool cache_ok(const splitzip_kv_cache *c) {
    if (!shape_ok(c)) return false;
    if (c->num_pages < 1 || c->num_pages > 0x7fffffffu || !c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
        return false;
    const uint64_t counts[3] = {c->num_pages, c->kv_heads, c->page_size};
    uint64_t ke = 0, ve = 0;
    for (int i = 0; i < 3; ++i) {
        if (c->k_stride[i] % 8 || c->v_stride[i] % 8 || !spans(c->k_stride[i], counts[i]) || !spans(c->v_stride[i], counts[i]))
            return false;
        ke += c->k_stride[i] * (counts[i] - 1);
        ve += c->v_stride[i] * (counts[i] - 1);
    }
    if (ke + c->head_dim > kMaxOffset || ve + c->head_dim > kMaxOffset) return false;
    return c->batch == 0 || (c->lens && aligned(c->lens, 4) && aligned(c->table, 4) && (c->table || c->max_pages == 0) &&
                             (c->batch == 1 || c->table_stride >= c->max_pages) && c->table_stride <= kMaxOffset);
}

inline Cache view(const splitzip_kv_cache *c) {
    Cache v{};
    v.k = c->k;
    v.v = c->v;
    for (int i = 0; i < 3; ++i) {
        v.ks[i] = c->k_stride[i];
        v.vs[i] = c->v_stride[i];
    }
    v.table = c->table;
    v.table_stride = c->table_stride;
    v.lens = c->lens;
    v.page = make_div(c->page_size);
    v.num_pages = c->num_pages;
    v.kv_heads = c->kv_heads;
    v.dim = c->head_dim;
    v.batch = c->batch;
    v.max_len = c->max_pages * c->page_size;
    return v;
}

}  // namespace

#endif  // SPLITZIP_CSRC_KV_CACHE_H
