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

#define SPLITZIP_KV_NO_PAGE 8    /* no page left: a sequence is shorter than asked for */
#define SPLITZIP_KV_BAD_PARENT 16 /* a parent outside the batch: the sequence is left */

/* No window: every cached token is visible. */
#define SPLITZIP_KV_ALL 0xffffffffu

#define SPLITZIP_KV_MAX_DIM 256u
#define SPLITZIP_KV_MAX_PAGE 65536u
#define SPLITZIP_KV_MAX_BATCH 65535u
#define SPLITZIP_KV_MAX_KV_HEADS 4096u
#define SPLITZIP_KV_MAX_HEADS 65535u
#define SPLITZIP_KV_MAX_ROWS 0x7fffffffu
#define SPLITZIP_KV_MAX_PAGES 0x1000000u  /* of the operators on pages */
#define SPLITZIP_KV_MAX_LAYERS 1024u

/* Limits: head_dim a multiple of 8 in 8..256; all strides multiples of 8 (16
 * bytes) and pools 16-byte aligned; 1..65536 slots a page; max_pages *
 * page_size below 2^31; rows of the table at least max_pages apart;
 * num_pages in 1..2^31-1; batch 0..65535; 1..4096 KV heads; the pools'
 * largest offset below 2^40 elements.  A page that the table names twice (for
 * two sequences or in one) may be read, not written; splitzip_kv_pages_resize
 * sees to it that none is. */
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
 * hold budget tokens, or its width the whole cache's.  Caches of several layers
 * that have one lens: in place the first call sets it, and what it was is put
 * back before each further one.
 * Errors: INVALID (also sinks + recent > budget, budget 0), HIP. */
int splitzip_kv_evict(const splitzip_kv_cache *cache, const splitzip_kv_cache *to,
                      const splitzip_kv_budget *budget, int32_t *d_status, void *stream);

/* Sequences with their first tokens in common: group g has sequences cu[g] ..
 * cu[g+1]-1 of the batch, and of them the first shared[g] tokens (no more than
 * its first sequence has) are the same.  Sequences in no group have none. */
typedef struct splitzip_kv_groups {
    const int32_t *cu;           /* [groups + 1], ascending                        */
    const int32_t *shared;       /* [groups]                                       */
    uint32_t groups;             /* 0..65535                                       */
    uint32_t reserved;
} splitzip_kv_groups;

size_t splitzip_kv_groups_struct_size(void);

/* As splitzip_kv_attend_workspace_size, for splitzip_kv_attend_shared with up
 * to `groups` groups. */
size_t splitzip_kv_shared_workspace_size(const splitzip_kv_cache *cache, uint32_t heads, uint32_t groups);

/* What splitzip_kv_attend computes (window ALL, no mass), where K and V of the
 * tokens that a group has in common are read through the table row of its first
 * sequence: the others need only have the same values there, mostly in the same
 * pages.  They are read once for as many query rows of a KV head as a workgroup
 * takes: 128 of the group's sequences, or 16 or 32 where little would be read
 * again; by every sequence where those have no room for two of them, or where a
 * KV head's tokens are few.  A sequence that is shorter than the tokens in common
 * attends on its own; when the first one ends, so do all, until cu begins a group
 * with one that goes on.  With 128 rows the weights of the tokens in common are
 * rounded to the cache's type once (half a step of it each); all other sums, and
 * those of the other forms, are held as in splitzip_kv_attend.  The form goes by
 * the shapes, the number of groups and what the table can hold, not by lengths,
 * which are on the device: a table much wider than its sequences takes the form
 * for long ones.  Ranges that decrease or leave the
 * batch: BAD_ROWS, no tokens in common (where ranges overlap by that, outputs
 * mean nothing); shared below 0: BAD_LEN, taken as 0.
 * Errors: INVALID (also a window or mass), WORKSPACE, HIP. */
int splitzip_kv_attend_shared(const splitzip_kv_cache *cache, const splitzip_kv_query *query,
                              const splitzip_kv_groups *groups, void *d_ws, size_t ws_bytes, int32_t *d_status,
                              void *stream);

/* Who has which pages: the pools of a model's layers, which share one table
 * and lengths, and how many table entries name each page.  A page that none
 * names is free.  The cache gives table, lens, shape and strides of all
 * layers (its own k and v are not looked at); table and lens are written. */
typedef struct splitzip_kv_pages {
    const splitzip_kv_cache *cache;
    uint16_t *const *k, *const *v;   /* [layers], in host memory: the layers' pools   */
    uint32_t layers;                 /* 1..SPLITZIP_KV_MAX_LAYERS                     */
    uint32_t reserved;
    void *state;                     /* device memory; its first num_pages int32 are
                                        the counts, to be read; the rest, and the
                                        counts between calls, are the operators'     */
    size_t state_bytes;
} splitzip_kv_pages;

size_t splitzip_kv_pages_struct_size(void);

/* Bytes of state for caches of this shape (batch and num_pages; no pointer is
 * read), 0 for invalid shapes: more than SPLITZIP_KV_MAX_PAGES pages, pages of
 * 32 GiB.  Calls on one state must run one after another.  batch * max_pages
 * must be below 2^31, the layers' pools share no memory. */
size_t splitzip_kv_pages_state_size(const splitzip_kv_cache *cache);

/* Count: the state from the table.  Entries within a sequence's length name
 * its pages, those behind are set to -1.  The first call on a state, and the
 * one after the table has been written by others.  (An entry outside the pool
 * within a length becomes -1: SPLITZIP_KV_BAD_PAGE.)
 * Errors of all page operators: INVALID, WORKSPACE (a state too small), HIP. */
int splitzip_kv_pages_count(const splitzip_kv_pages *pages, int32_t *d_status, void *stream);

/* Fork: sequence b becomes a copy of sequence parents[b], all at once: the
 * same pages, also the last one that is not full, and the length.  Parent -1
 * frees the sequence (no page, length 0), b itself leaves it.  Nothing is
 * copied but table and lengths. */
int splitzip_kv_pages_fork(const splitzip_kv_pages *pages, const int32_t *parents, int32_t *d_status, void *stream);

/* Resize: the sequences' lengths become lens (device memory; may be the
 * cache's own, which frees the pages behind them).  Pages behind a sequence's
 * new length, or behind its old one where that is shorter (a length that was cut
 * in place, as an eviction does), are freed first.  Then, in the order of sequences, each is given the pages
 * that positions up to its new length need, and where it grows from within a
 * page that others name, a page of its own first, to which the slots in use
 * are copied in every layer (of the sequences that all grow in one page that
 * no other names the first keeps it).  The pages given are the free ones in
 * ascending order.  When they run out a sequence's length becomes what its
 * pages hold, or stays as it was if its copy could not be had, or if it would
 * have kept a page that another still reads because that one's copy could not
 * be had (SPLITZIP_KV_NO_PAGE).  The tokens from the old length on are the
 * caller's to append.  The old length is the cache's, or, where that was made
 * greater in place since (lens += 1, and then resized to itself), the one that
 * the last of these calls left.  Between two of them a length is cut in place or
 * made greater, not the one and then the other: a growth back over pages that
 * others name is not seen. */
int splitzip_kv_pages_resize(const splitzip_kv_pages *pages, const int32_t *lens, int32_t *d_status, void *stream);

/* Compact: with n pages in use, the pages in use from n on move to the free
 * ones below, the last to the first, in every layer; table and counts follow.
 * moved (NULL or [num_pages]): the new number of each page, -1 for free ones;
 * used (NULL or one int32): n. */
int splitzip_kv_pages_compact(const splitzip_kv_pages *pages, int32_t *moved, int32_t *used, int32_t *d_status,
                              void *stream);

/* Copy: K and V of pages src[i] of `from` to pages dst[i] of `to`, i < n, in
 * every layer, whatever the strides.  Both have the same layers, page_size,
 * kv_heads, head_dim and dtype; tables, lengths and state are not looked at.
 * No page is named in dst twice, nor in dst and src where `to` has the pools
 * of `from`; other pools share no memory.  Pairs with a page outside its pool
 * are left out (SPLITZIP_KV_BAD_PAGE). */
int splitzip_kv_pages_copy(const splitzip_kv_pages *from, const splitzip_kv_pages *to, const int32_t *src,
                           const int32_t *dst, uint32_t n, int32_t *d_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPLITZIP_KV_H */
