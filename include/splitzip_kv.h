/*
 * splitzip_kv.h -- C ABI of the paged key-value cache on MI355X (gfx950): the
 * cache that decoded KV tensors go into, the attention of one new token per
 * sequence over it, and the eviction of the tokens that drew the least
 * attention.  Library: libsplitzip_kv.so.
 *
 * A cache is two pools of pages (K and V), a table of page numbers per
 * sequence and the sequences' lengths.  Token t of sequence b lies in slot
 * t % page_size of page table[b][t / page_size]; element d of its KV head h is
 *   k[page * k_stride[0] + h * k_stride[1] + slot * k_stride[2] + d]
 * (v alike), so a pool may be stored [page][head][slot][dim], as the codec's
 * KV tensors are, [page][slot][head][dim], or inside a larger array.
 *
 * Conventions as in splitzip.h: all work is enqueued asynchronously on
 * `stream` of the calling thread's current device, no entry point
 * synchronises, allocates or frees memory, every buffer is the caller's, and
 * every call enqueues kernels only, so it can be captured in a HIP graph.  The
 * return value reports argument errors and launch failures (the codes of
 * enum splitzip_status; nothing is enqueued on an argument error).  Structs
 * live in host memory and are read before the call returns; the pointers in
 * them are device pointers (or pinned host memory).
 *
 * What only the device can see is checked there: a page number outside
 * [0, num_pages), a length outside [0, max_pages * page_size], a row range
 * outside the rows given.  Such a token is left out (neither read nor
 * written), such a length is taken as the nearest one allowed, and where
 * d_status is given the bits below are ORed into it.
 * Table, lengths and row ranges must not change while a call runs.
 */
#ifndef SPLITZIP_KV_H
#define SPLITZIP_KV_H

#include <stddef.h>
#include <stdint.h>

#include "splitzip.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPLITZIP_KV_BF16 0u
#define SPLITZIP_KV_FP16 1u

/* d_status bits */
#define SPLITZIP_KV_BAD_PAGE 1   /* a page number outside the pool               */
#define SPLITZIP_KV_BAD_LEN 2    /* a length outside the table                   */
#define SPLITZIP_KV_BAD_ROWS 4   /* row ranges that decrease or leave the rows,
                                    or a first position below 0 or rows that
                                    pass the table's end                         */

/* No window: every cached token is visible. */
#define SPLITZIP_KV_ALL 0xffffffffu

#define SPLITZIP_KV_MAX_DIM 256u
#define SPLITZIP_KV_MAX_PAGE 65536u
#define SPLITZIP_KV_MAX_BATCH 65535u
#define SPLITZIP_KV_MAX_KV_HEADS 4096u
#define SPLITZIP_KV_MAX_HEADS 65535u
#define SPLITZIP_KV_MAX_ROWS 0x7fffffffu

/* Limits: head_dim a multiple of 8 in 8..256; all strides multiples of 8 (16
 * bytes) and pools 16-byte aligned; 1..65536 slots a page; max_pages *
 * page_size below 2^31; rows of the table at least max_pages apart;
 * num_pages in 1..2^31-1; batch 0..65535; 1..4096 KV heads; the pools'
 * largest offset below 2^40 elements.  A page that the table names twice (for
 * two sequences or in one) may be read, not written. */
typedef struct splitzip_kv_cache {
    uint16_t *k, *v;             /* pools (bf16 or fp16 bit patterns)            */
    uint64_t k_stride[3];        /* elements between pages, heads, slots         */
    uint64_t v_stride[3];
    const int32_t *table;        /* page numbers, row b at table + b * table_stride */
    uint64_t table_stride;
    int32_t *lens;               /* cached tokens per sequence [batch]           */
    uint32_t num_pages;
    uint32_t page_size;
    uint32_t kv_heads;
    uint32_t head_dim;
    uint32_t batch;
    uint32_t max_pages;          /* entries of a table row                       */
    uint32_t dtype;              /* SPLITZIP_KV_BF16 or SPLITZIP_KV_FP16         */
    uint32_t reserved;
} splitzip_kv_cache;

/* Rows outside the cache: element d of row r, head h is
 * k[r * k_stride[0] + h * k_stride[1] + d].  Rows cu[b] .. cu[b+1]-1 belong to
 * sequence b and to its positions start[b], start[b]+1, ... (lens is not looked
 * at then); with start NULL they are its last ones, start[b] = lens[b] -
 * (cu[b+1] - cu[b]). */
typedef struct splitzip_kv_rows {
    uint16_t *k, *v;
    uint64_t k_stride[2];        /* elements between rows, heads (multiples of 8) */
    uint64_t v_stride[2];
    uint32_t rows;
    uint32_t reserved;
    const int32_t *cu;           /* [batch + 1], ascending                       */
    const int32_t *start;        /* [batch] or NULL                              */
} splitzip_kv_rows;

/* One new token's queries per sequence. */
typedef struct splitzip_kv_query {
    const uint16_t *q;           /* element d of sequence b, head i at q + b *
                                    q_stride[0] + i * q_stride[1] + d; query head
                                    i reads KV head i / (heads / kv_heads)       */
    uint64_t q_stride[2];        /* multiples of 8                               */
    uint16_t *out;               /* laid out like q, with strides of its own; may
                                    be q itself, and else shares no memory with it */
    uint64_t out_stride[2];
    float *lse;                  /* NULL, or [batch][heads]: log of the sum of
                                    exp(logit); -inf where nothing is visible    */
    const float *mass;           /* NULL, or attention weight gathered so far:
                                    token t, KV head h at b * mass_stride[0] +
                                    h * mass_stride[1] + t                       */
    float *mass_out;             /* NULL, or mass plus this call's weights; may
                                    be mass itself                               */
    uint64_t mass_stride[2];
    uint64_t mass_out_stride[2];
    uint32_t heads;              /* a multiple of kv_heads                       */
    uint32_t window;             /* last tokens visible, SPLITZIP_KV_ALL: all    */
    uint32_t sinks;              /* first tokens visible beside the window       */
    float scale;                 /* logit = scale * (q . k)                      */
    uint32_t mass_len;           /* entries of mass and mass_out per head; a
                                    longer sequence's other tokens are left out
                                    of them (SPLITZIP_KV_BAD_LEN)                */
    uint32_t reserved;
} splitzip_kv_query;

/* Which tokens an eviction keeps. */
typedef struct splitzip_kv_budget {
    const float *mass;           /* as in splitzip_kv_query                      */
    float *mass_out;             /* NULL, or the kept tokens' mass in their new
                                    places, 0 from there to the old length; may
                                    be mass itself                               */
    uint64_t mass_stride[2];
    uint64_t mass_out_stride[2];
    int32_t *kept;               /* [batch][kv_heads][budget]: the old position of
                                    each kept token, ascending; -1 behind them   */
    uint32_t budget;
    uint32_t sinks;              /* first tokens, always kept                    */
    uint32_t recent;             /* last tokens, always kept                     */
    uint32_t mass_len;           /* entries of mass and mass_out per head; a
                                    longer length is taken as this
                                    (SPLITZIP_KV_BAD_LEN)                        */
} splitzip_kv_budget;

/* sizeof of the four structs above, in their order, as compiled into the
 * library. */
void splitzip_kv_struct_sizes(size_t sizes[4]);

/* Copy rows into the cache / cached tokens into rows.  With start NULL, lens
 * already counts the appended tokens.  Rows behind cu[batch] are left alone (an
 * append does not read them, a gather does not write them).  Bit-exact copies.
 * What is written shares no memory with what is read, nor its K with its V
 * (where both pools are one, K and V rows may be one).
 * Errors: INVALID, HIP. */
int splitzip_kv_append(const splitzip_kv_cache *cache, const splitzip_kv_rows *rows,
                       int32_t *d_status, void *stream);
int splitzip_kv_gather(const splitzip_kv_cache *cache, const splitzip_kv_rows *rows,
                       int32_t *d_status, void *stream);

/* Bytes of workspace that splitzip_kv_attend needs for caches of this shape
 * (batch, kv_heads, head_dim; no pointer is read), `heads` query heads and,
 * where mass is asked for, up to mass_len entries (0: none); 0 for invalid
 * shapes.  A larger workspace serves too.  Its content between calls does not
 * matter; one workspace must not be used by two calls that can run at the same
 * time. */
size_t splitzip_kv_attend_workspace_size(const splitzip_kv_cache *cache, uint32_t heads,
                                         uint32_t mass_len);

/* Attention of one new token per sequence over the cached ones (its own K and
 * V appended before).  Of a sequence of length n, token t is visible when
 * t >= n - window or t < sinks.  With x[t] = scale * (q . k[t]) over the
 * visible tokens, out = sum_t exp(x[t] - lse) v[t], lse = log sum_t exp(x[t]).
 * A sequence with no visible token gives zeros and lse = -inf.  Logits and the
 * sum before its division are held in 32 bits: where they pass 3.4e38 (bf16
 * values near the type's largest) the result is not finite.  With mass_out,
 * mass_out[t] = mass[t] + the sum of exp(x[t] - lse) over the query heads of
 * the KV head for visible tokens, mass[t] for the others, up to the sequence's
 * length (mass NULL: 0); entries behind it are left alone.
 * Errors: INVALID, WORKSPACE, HIP. */
int splitzip_kv_attend(const splitzip_kv_cache *cache, const splitzip_kv_query *query, void *d_ws,
                       size_t ws_bytes, int32_t *d_status, void *stream);

/* Evict: every KV head of a sequence longer than `budget` keeps the first
 * `sinks` tokens, the last `recent` ones and, of those between, the budget -
 * sinks - recent of the largest mass (equal masses: the lower position; NaN
 * counts as larger than any number), in their order; shorter sequences stay
 * whole.  The kept tokens' K and V are copied to positions 0, 1, ... of `to`,
 * and to->lens becomes min(length, budget).  `to` has the cache's batch,
 * kv_heads, head_dim and dtype.  It is the cache itself (same table, pools and
 * lens: compaction in place) or pages and lens that share no memory with it;
 * a `to` that shares its table or lens or a pool's start with the cache is
 * taken as in place and must be equal to it in all fields.  Its K and V pools
 * share no memory in place.  to's table must
 * hold budget tokens, or its width the whole cache's.
 * Errors: INVALID (also sinks + recent > budget, budget 0), HIP. */
int splitzip_kv_evict(const splitzip_kv_cache *cache, const splitzip_kv_cache *to,
                      const splitzip_kv_budget *budget, int32_t *d_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPLITZIP_KV_H */
