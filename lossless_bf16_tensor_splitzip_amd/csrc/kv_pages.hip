// kv_pages.hip -- who has which pages of a paged key-value cache: HIP kernels
// and the C ABI of the page operators declared in include/splitzip_kv.h.
//
//   k_clear, k_names, k_free   counts of all pages from the table (count)
//   k_fork                     table rows become copies of others
//   k_want, k_choose, k_give   pages freed, chosen and given, shared ones copied (resize)
//   k_holes, k_fill            pages in use to the front of the pools (compact)
//   k_copy                     pages to other pages (copy)
//
// A page is free when no table entry names it (its count is 0).  Beside the
// counts the state keeps how many of every 256 pages are free, so that pages
// are found by reading the blocks that have some and no others.  All of it is
// kept by integer additions, which no order changes, and pages are given in the
// order of their numbers: results depend on the arguments alone.
//
// Chains of dependent loads and the launches bound the bookkeeping, memory the
// moves of pages.

#include "kv_cache.h"

namespace {

constexpr uint32_t kBlock = 256;          // pages a free count is of
constexpr uint32_t kMaxPools = 128;       // pools (K and V of 64 layers) a launch moves pages of

// What resize knows of a sequence.
struct Want {
    uint32_t first, need;     // entries to be filled: first .. need - 1
    uint32_t page;            // the page that is begun and will be written, or kNoPage
    uint32_t old_len, new_len;
    uint32_t before;          // pages wanted by the sequences before it
    uint32_t copies;          // 1: the begun page is shared, a copy is wanted before the entries
    uint32_t slots;           // in use of the begun page; before one is found, the cache's length
};
constexpr uint32_t kNoPage = 0xffffffffu;

struct State {
    int32_t *refs;            // [pages] table entries that name the page
    int32_t *free_in;         // [pages / kBlock] of them free
    int32_t *writers, *lowest;// [pages] sequences about to write the page, the first of them; 0 and INT_MAX between calls
    uint32_t *list;           // [pages] free pages, ascending
    uint32_t *from;           // [pages] pages to be moved, from the top
    uint32_t *rank;           // [pages] a moved page's place in from
    uint32_t *words;          // 0: pages in use; 1: moves; 2: pages given; 3: pages wanted; 4: 1 if rows have gaps
    Want *want;               // [batch]
    int32_t *left;            // [batch] lengths as the last call left them
};

struct PageArgs {
    Cache c;                  // strides are those of every layer
    int32_t *table;
    State s;
    const int32_t *arg;       // lengths or parents
    int32_t *status;
};

__device__ inline void drop_name(const State &s, uint32_t page, int32_t n) {
    if (atomicSub(&s.refs[page], n) == n) atomicAdd(&s.free_in[page / kBlock], 1);
}

__device__ inline uint32_t pages_for(const Cache &c, uint32_t n) { return n ? div(n - 1, c.page) + 1 : 0; }

// ---------------------------------------------------------------------------
// Pages' contents
// ---------------------------------------------------------------------------

// How a page of one pool becomes a page of another: n0 x n1 runs of `run`
// 16-byte pieces, in the order in which the source has them.
struct Geometry {
    uint64_t s0, s1, d0, d1;      // strides of source and destination, elements
    Div run, n1;
    uint32_t total, per_slot;     // pieces of a page, of a slot
    bool slot_first;              // n0 counts slots (and n1 heads, or nothing)
};

struct Pools {
    uint16_t *p[kMaxPools];
};

constexpr int kCopyThreads = 256;
constexpr int kCopyAhead = 4;     // pieces a thread has under way

// The workgroup copies the first `slots` slots of a page.
template <int AHEAD = kCopyAhead>
__device__ inline void copy_page(const uint16_t *src, uint16_t *dst, const Geometry &g, uint32_t slots) {
    const uint32_t total = g.slot_first ? slots * g.per_slot : g.total;
    for (uint32_t i0 = threadIdx.x; i0 < total; i0 += kCopyThreads * AHEAD) {
        u32x4 x[AHEAD];
        uint64_t to[AHEAD];
        bool ok[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const uint32_t i = i0 + u * kCopyThreads;
            const uint32_t row = div(i, g.run), piece = i - row * g.run.d;
            const uint32_t r0 = div(row, g.n1), r1 = row - r0 * g.n1.d;
            ok[u] = i < total && (g.slot_first || r1 < slots);
            to[u] = r0 * g.d0 + r1 * g.d1 + piece * 8;
            if (ok[u]) x[u] = load_once(src + r0 * g.s0 + r1 * g.s1 + piece * 8);
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
            if (ok[u]) store_away(dst + to[u], x[u]);
    }
}

// ---------------------------------------------------------------------------
// count
// ---------------------------------------------------------------------------

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void k_clear(PageArgs a) {
    for (uint32_t p = blockIdx.x * kThreads + threadIdx.x; p < a.c.num_pages; p += gridDim.x * kThreads) {
        a.s.refs[p] = 0;
        a.s.writers[p] = 0;
        a.s.lowest[p] = 0x7fffffff;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.s.words[4] = 0;
}

// A row's entries within the sequence's length name their pages, those behind it none.
__global__ __launch_bounds__(kThreads) void k_names(PageArgs a, uint32_t width, uint32_t parts) {
    for (uint32_t w = blockIdx.x; w < a.c.batch * parts; w += gridDim.x) {
        const uint32_t b = w / parts, part = w - b * parts;
        const bool first = part == 0 && threadIdx.x == 0;
        const uint32_t len = seq_len(a.c, b, first ? a.status : nullptr), held = pages_for(a.c, len);
        if (first) a.s.left[b] = (int32_t)len;
        int32_t *row = a.table + b * a.c.table_stride;
        for (uint32_t i = part * kThreads + threadIdx.x; i < width; i += parts * kThreads) {
            const uint32_t page = (uint32_t)row[i];
            if (i < held && page < a.c.num_pages) {
                atomicAdd(&a.s.refs[page], 1);
            } else {
                if (i < held) {
                    report(a.status, SPLITZIP_KV_BAD_PAGE);
                    a.s.words[4] = 1;
                }
                row[i] = -1;
            }
        }
    }
}

__global__ __launch_bounds__(kThreads) void k_free(PageArgs a, uint32_t blocks) {
    __shared__ uint32_t part[kThreads / 64];
    static_assert(kThreads == kBlock, "a thread a page");
    for (uint32_t k = blockIdx.x; k < blocks; k += gridDim.x) {
        const uint32_t p = k * kBlock + threadIdx.x;
        const uint64_t is_free = __ballot(p < a.c.num_pages && a.s.refs[p] == 0);
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = __popcll(is_free);
        __syncthreads();
        if (threadIdx.x == 0) a.s.free_in[k] = part[0] + part[1] + part[2] + part[3];
        __syncthreads();
    }
}

constexpr uint32_t kSmallPages = 16384, kSmallEntries = 4096;
constexpr int kSmallThreads = 1024;

// The same by one workgroup, with the counts in LDS (a pool of 64 pages and 4
// rows of 13 entries: one launch instead of three).
__global__ __launch_bounds__(kSmallThreads) void k_count(PageArgs a, uint32_t width) {
    __shared__ int32_t n[kSmallPages];
    __shared__ uint32_t s_gaps;
    const uint32_t tid = threadIdx.x;
    if (tid == 0) s_gaps = 0;
    for (uint32_t p = tid; p < a.c.num_pages; p += kSmallThreads) n[p] = 0;
    for (uint32_t b = tid; b < a.c.batch; b += kSmallThreads) a.s.left[b] = (int32_t)seq_len(a.c, b);
    __syncthreads();
    for (uint32_t i = tid; i < a.c.batch * width; i += kSmallThreads) {
        const uint32_t b = i / width, at = i - b * width;
        const uint32_t held = pages_for(a.c, seq_len(a.c, b, at == 0 ? a.status : nullptr));
        int32_t *entry = a.table + b * a.c.table_stride + at;
        const uint32_t page = (uint32_t)*entry;
        if (at < held && page < a.c.num_pages) {
            atomicAdd(&n[page], 1);
        } else {
            if (at < held) {
                report(a.status, SPLITZIP_KV_BAD_PAGE);
                s_gaps = 1;
            }
            *entry = -1;
        }
    }
    __syncthreads();
    if (tid == 0) a.s.words[4] = s_gaps;
    for (uint32_t p = tid; p < a.c.num_pages; p += kSmallThreads) {
        a.s.refs[p] = n[p];
        a.s.writers[p] = 0;
        a.s.lowest[p] = 0x7fffffff;
    }
    // a wave for every 256 pages
    for (uint32_t k = tid >> 6; k * kBlock < a.c.num_pages; k += kSmallThreads / 64) {
        uint32_t is_free = 0;
        for (uint32_t q = 0; q < kBlock; q += 64) {
            const uint32_t p = k * kBlock + q + (tid & 63);
            is_free += __popcll(__ballot(p < a.c.num_pages && n[p] == 0));
        }
        if ((tid & 63) == 0) a.s.free_in[k] = is_free;
    }
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------

constexpr int kForkThreads = 1024;

// A workgroup has some columns of the table for all sequences (the last one
// the lengths): it reads what the rows will be, and then writes them, so that
// rows can be copies of each other in any order without a second table.  A
// row's pages are named by as many rows as have it as parent, instead of by
// itself: one addition for all of them, and none where rows change places.  A
// thread has U rows of one column, one below the other, whose additions to one
// page are one.  (64 beams of up to 2048 tokens 5.2 us; naming and dropping
// entry by entry, 15.)
template <int U>
__global__ __launch_bounds__(kForkThreads) void k_fork(PageArgs a, uint32_t width, uint32_t columns) {
    extern __shared__ uint32_t s_children[];      // [batch / 2 + 1], 16 bits each
    const uint32_t batch = a.c.batch;
    for (uint32_t k = threadIdx.x; k < batch / 2 + 1; k += blockDim.x) s_children[k] = 0;
    __syncthreads();
    const bool is_lens = blockIdx.x == gridDim.x - 1;
    auto parent_of = [&](uint32_t b) {
        const int32_t p = a.arg[b];
        return p >= -1 && p < (int32_t)batch ? p : (int32_t)b;
    };
    for (uint32_t b = threadIdx.x; b < batch; b += blockDim.x) {
        const int32_t p = parent_of(b);
        if (is_lens && p != a.arg[b]) report(a.status, SPLITZIP_KV_BAD_PARENT);
        // (a sum of up to 65535 stays within its half)
        if (p >= 0) atomicAdd(&s_children[p >> 1], p & 1 ? 1u << 16 : 1u);
    }
    const uint32_t per_row = is_lens ? 1 : columns;       // a power of two
    const uint32_t i = blockIdx.x * columns + (threadIdx.x & (per_row - 1));
    const uint32_t b0 = threadIdx.x / per_row * U;
    const bool mine = is_lens || i < width;
    int32_t next[U], was[U];
    uint64_t changed = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t b = b0 + u;
        was[u] = next[u] = -1;
        if (!mine || b >= batch) continue;
        const int32_t parent = parent_of(b);
        if (is_lens) next[u] = parent < 0 ? 0 : a.c.lens[parent];
        else was[u] = a.table[b * a.c.table_stride + i];
        if (parent == (int32_t)b) continue;
        changed |= 1ull << u;
        if (!is_lens && parent >= 0) next[u] = a.table[parent * a.c.table_stride + i];
    }
    __syncthreads();
    if (!is_lens) {
        int32_t sum = 0, add[U], before[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t b = b0 + u;
            add[u] = before[u] = 0;
            if ((uint32_t)was[u] < a.c.num_pages) sum += (int32_t)(s_children[b >> 1] >> (b & 1 ? 16 : 0) & 0xffff) - 1;
            if (u + 1 < U && was[u + 1] == was[u]) continue;
            add[u] = sum;
            sum = 0;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (add[u]) before[u] = atomicAdd(&a.s.refs[was[u]], add[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (add[u] && before[u] + add[u] == 0) atomicAdd(&a.s.free_in[(uint32_t)was[u] / kBlock], 1);
            else if (add[u] && before[u] == 0) atomicSub(&a.s.free_in[(uint32_t)was[u] / kBlock], 1);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (is_lens && b0 + u < batch) a.s.left[b0 + u] = next[u];
        if (changed >> u & 1) {
            if (is_lens) a.c.lens[b0 + u] = next[u];
            else a.table[(b0 + u) * a.c.table_stride + i] = next[u];
        }
    }
}

// ---------------------------------------------------------------------------
// resize
// ---------------------------------------------------------------------------

// A sequence keeps the pages that its old or its new length needs, whichever is
// shorter.  Entries behind an old length that was cut in the caches hold no
// token, and a fork may have given them to others, who would write them too.
// Pages are held from a row's start without a gap, so what a sequence drops and
// misses is looked for from the border of what it keeps.  A wave looks at 64
// entries a time: drops those behind, and returns the first that is missing.
// Where the count found page numbers outside the pool rows may have gaps, and all
// that lies behind is looked at.
__device__ inline uint32_t drop_and_find(const PageArgs &a, int32_t *row, uint32_t keep, uint32_t width, bool gaps) {
    const uint32_t lane = threadIdx.x & 63;
    for (uint32_t i0 = keep; i0 < width; i0 += 64) {
        const int32_t page = i0 + lane < width ? row[i0 + lane] : -1;
        if (page >= 0) {
            if ((uint32_t)page < a.c.num_pages) drop_name(a.s, page, 1);
            row[i0 + lane] = -1;
        }
        if (!gaps && !__ballot(page >= 0)) break;
    }
    uint32_t first = keep;
    while (first) {
        const uint32_t n = min(first, 64u), i = first - n + lane;
        const uint64_t held = __ballot(lane < n && row[i] >= 0);
        if (held) return first - n + 64 - __builtin_clzll(held);
        first -= n;
    }
    return 0;
}

// Lengths asked for and old, and what is kept (in `first`).  A sequence that was
// made longer in the cache (lens += 1 before the call) grows from the length that
// the last call left: what lies behind is written after this one.
__device__ inline Want want_of(const PageArgs &a, uint32_t b, bool tell) {
    const uint32_t len = seq_len(a.c, b, tell ? a.status : nullptr);
    const int32_t asked = a.arg[b];
    const uint32_t new_len = asked < 0 ? 0 : min((uint32_t)asked, a.c.max_len);
    if (tell && (int32_t)new_len != asked) report(a.status, SPLITZIP_KV_BAD_LEN);
    return Want{pages_for(a.c, min(len, new_len)), pages_for(a.c, new_len), kNoPage, min(len, (uint32_t)a.s.left[b]), new_len, 0, 0, len};
}

// The page that is begun and will be written, whose writers are counted.
__device__ inline void begin_writing(const PageArgs &a, uint32_t b, const int32_t *row, Want &w) {
    const uint32_t at = div(w.old_len, a.c.page);
    if (w.new_len <= w.old_len || w.old_len == at * a.c.page.d) return;      // else `at` is kept
    const uint32_t page = (uint32_t)row[at];
    if (page < a.c.num_pages) {
        w.page = page;
        w.slots = min(w.slots - at * a.c.page.d, a.c.page.d);
        atomicAdd(&a.s.writers[page], 1);
        atomicMin(&a.s.lowest[page], (int32_t)b);
    } else {
        report(a.status, SPLITZIP_KV_BAD_PAGE);
    }
}

// A wave per sequence.
__global__ __launch_bounds__(kThreads) void k_want(PageArgs a, uint32_t width) {
    const uint32_t b = blockIdx.x * (kThreads / 64) + threadIdx.x / 64, lane = threadIdx.x & 63;
    if (b >= a.c.batch) return;
    int32_t *row = a.table + b * a.c.table_stride;
    Want w = want_of(a, b, lane == 0);
    w.first = drop_and_find(a, row, w.first, width, a.s.words[4] != 0);
    if (lane == 0) {
        begin_writing(a, b, row, w);
        a.s.want[b] = w;
    }
}

constexpr int kChooseThreads = 1024;

// Sum of x over the threads up to this one; `all` gets the whole sum.
__device__ inline uint32_t group_scan(uint32_t x, uint32_t *part, uint32_t &all) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t upto = wave_scan(x);
    __syncthreads();       // part has been read
    if (lane == 63) part[wave] = upto;
    __syncthreads();
    const uint32_t waves = wave_scan(lane < kChooseThreads / 64 ? part[lane] : 0);
    all = __builtin_amdgcn_readlane(waves, 63);
    return upto + (wave ? __builtin_amdgcn_readlane(waves, wave - 1) : 0);
}

// Counts that this launch's additions changed: past the caches.
__device__ inline int32_t latest(const int32_t *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// One workgroup: how many pages the sequences want, each its place among them,
// and the first so many free pages, in order.  WANT: with what k_want does for
// up to kChooseThreads sequences, a thread each where a sequence drops a page
// at most (a step's tokens), else a wave.  (64 sequences with 8
// drafts each, given back and made room for: 15.6 us, with k_want 20.8 to 25.5.)
template <bool WANT>
__global__ __launch_bounds__(kChooseThreads) void k_choose(PageArgs a, uint32_t width, uint32_t blocks) {
    __shared__ uint32_t part[64], s_block[kChooseThreads], s_before[kChooseThreads], s_take[kChooseThreads], s_slow;
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint32_t total = 0;
    Want mine{};
    if (WANT) {
        if (tid == 0) s_slow = 0;
        __syncthreads();
        int32_t *row = a.table + tid * a.c.table_stride;
        const bool gaps = a.s.words[4] != 0;
        bool slow = false;
        if (tid < a.c.batch) {
            mine = want_of(a, tid, true);
            const uint32_t keep = mine.first;
            const int32_t before2 = keep > 1 ? row[keep - 2] : 0, before1 = keep ? row[keep - 1] : 0;
            const int32_t behind1 = keep < width ? row[keep] : -1, behind2 = keep + 1 < width ? row[keep + 1] : -1;
            slow = gaps || behind2 >= 0 || (before1 < 0 && before2 < 0);
            if (slow) {
                s_take[atomicAdd(&s_slow, 1u)] = tid;
            } else {
                if (before1 < 0) mine.first = keep - 1;
                if (behind1 >= 0) {
                    if ((uint32_t)behind1 < a.c.num_pages) drop_name(a.s, behind1, 1);
                    row[keep] = -1;
                }
            }
        }
        __syncthreads();
        for (uint32_t i = wave; i < s_slow; i += kChooseThreads / 64) {
            const uint32_t b = s_take[i];
            const uint32_t first = drop_and_find(a, a.table + b * a.c.table_stride, want_of(a, b, false).first, width, gaps);
            if (lane == 0) s_before[b] = first;
        }
        __syncthreads();
        if (slow) mine.first = s_before[tid];
        if (tid < a.c.batch) begin_writing(a, tid, row, mine);
        wait_vector_memory();      // the additions have been made
        __syncthreads();
    }
    for (uint32_t b0 = 0; b0 < a.c.batch; b0 += kChooseThreads) {
        const uint32_t b = b0 + tid;
        uint32_t n = 0, copies = 0;
        Want w{};
        if (b < a.c.batch) {
            w = WANT ? mine : a.s.want[b];
            // the sequences that write a page leave it to the first of them, if no other names it
            if (w.page != kNoPage) {
                const int32_t refs = latest(&a.s.refs[w.page]);
                copies = refs > 1 && !(latest(&a.s.writers[w.page]) == refs && latest(&a.s.lowest[w.page]) == (int32_t)b);
            }
            n = w.need - w.first + copies;
        }
        uint32_t all;
        const uint32_t upto = group_scan(n, part, all);
        if (b < a.c.batch) {
            w.before = total + upto - n;
            w.copies = copies;
            a.s.want[b] = w;
        }
        total += all;
    }
    uint32_t found = 0;
    for (uint32_t k0 = 0; k0 < blocks && found < total; k0 += kChooseThreads) {
        const uint32_t n = k0 + tid < blocks ? (uint32_t)latest(&a.s.free_in[k0 + tid]) : 0;
        uint32_t all, used;
        const uint32_t before = found + group_scan(n, part, all) - n;
        const bool here = n && before < total;
        const uint32_t at = group_scan(here, part, used) - here;
        if (here) {
            s_block[at] = k0 + tid;
            s_before[at] = before;
            s_take[at] = min(n, total - before);
            a.s.free_in[k0 + tid] = (int32_t)(n - s_take[at]);
        }
        __syncthreads();
        for (uint32_t j = wave; j < used; j += kChooseThreads / 64) {
            const uint32_t p0 = s_block[j] * kBlock, take = s_take[j], at0 = s_before[j];
            uint64_t free4[kBlock / 64];
#pragma unroll
            for (uint32_t q = 0; q < kBlock / 64; ++q) {
                const uint32_t p = p0 + q * 64 + lane;
                free4[q] = __ballot(p < a.c.num_pages && latest(&a.s.refs[p]) == 0);
            }
            uint32_t done = 0;
#pragma unroll
            for (uint32_t q = 0; q < kBlock / 64; ++q) {
                const uint32_t rank = done + lanes_below(free4[q]);
                if ((free4[q] >> lane & 1) && rank < take && at0 + rank < a.c.num_pages) a.s.list[at0 + rank] = p0 + q * 64 + lane;
                done += __popcll(free4[q]);
            }
        }
        found += all;
        __syncthreads();
    }
    if (tid == 0) {
        a.s.words[2] = min(found, total);
        a.s.words[3] = total;
    }
}

// (A state that was written to may name anything: a page number is compared
// with the pool's size wherever it comes from the state.)
// The chosen pages are entered and the shared ones' slots in use copied, a
// workgroup for every sequence and pool, of which the first sees to the table.
// (64 sequences that copy no page 2.7 us; 7 MB of copies in 16 layers 8 to 9, a chain
// of three loads in each of 2048 workgroups.)
__global__ __launch_bounds__(kCopyThreads) void k_give(PageArgs a, Pools pools, Geometry gk, Geometry gv,
                                                       uint64_t page_k, uint64_t page_v, bool first_launch) {
    const uint32_t b = blockIdx.x, pool = blockIdx.y, tid = threadIdx.x;
    const Want w = a.s.want[b];
    const uint32_t given = min(a.s.words[2], a.c.num_pages);
    bool copied = w.copies && w.before < given;
    const uint32_t copy = copied ? a.s.list[w.before] : 0;
    copied = copied && copy < a.c.num_pages;
    if (pool == 0 && first_launch) {
        int32_t *row = a.table + b * a.c.table_stride;
        // A sequence that keeps the page it shared must not write it where another
        // got no page for its copy and still reads it.
        bool kept = false;
        if (given < a.s.words[3] && w.page != kNoPage && !w.copies) {
            for (uint32_t other = tid; other < a.c.batch; other += kCopyThreads) {
                const Want x = a.s.want[other];
                kept = kept || (x.page == w.page && x.copies && x.before >= given);
            }
            kept = __syncthreads_or(kept);
        }
        for (uint32_t i = w.first + tid; i < w.need; i += kCopyThreads) {
            const uint32_t rank = w.before + w.copies + (i - w.first);
            if (rank < given) {
                const uint32_t page = a.s.list[rank];
                if (page >= a.c.num_pages) continue;
                if (kept) {
                    atomicAdd(&a.s.free_in[page / kBlock], 1);
                } else {
                    row[i] = (int32_t)page;
                    a.s.refs[page] = 1;
                }
            }
        }
        if (tid == 0) {
            const uint32_t begin = w.before + w.copies, n = w.need - w.first;
            const uint32_t got = given > begin ? min(n, given - begin) : 0;
            uint32_t len = min(w.new_len, got < n ? (w.first + got) * a.c.page.d : a.c.max_len);
            if (copied) {
                row[div(w.old_len, a.c.page)] = (int32_t)copy;
                a.s.refs[copy] = 1;
                drop_name(a.s, w.page, 1);
            } else if (w.copies || kept) {
                len = w.old_len;
            }
            if (got < n || kept || (w.copies && !copied)) report(a.status, SPLITZIP_KV_NO_PAGE);
            a.c.lens[b] = a.s.left[b] = (int32_t)len;
            if (w.page != kNoPage) {
                a.s.writers[w.page] = 0;
                a.s.lowest[w.page] = 0x7fffffff;
            }
        }
    }
    if (!copied) return;
    const uint64_t step = pool & 1 ? page_v : page_k;
    copy_page<8>(pools.p[pool] + w.page * step, pools.p[pool] + copy * step, pool & 1 ? gv : gk, w.slots);
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------

// With n pages in use, the free pages below n are the holes and the pages in
// use from n on fill them, the last one the first hole.  A page's rank among
// them follows from how many free pages come before it.
__global__ __launch_bounds__(kThreads) void k_holes(PageArgs a, uint32_t blocks, int32_t *moved, int32_t *used_out) {
    __shared__ uint32_t s_before[kThreads / 64], s_all[kThreads / 64], part[kThreads / 64];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t per = (blocks - 1) / gridDim.x + 1, k0 = min(blocks, blockIdx.x * per), k1 = min(blocks, k0 + per);
    uint32_t before = 0, all = 0;
    for (uint32_t k = tid; k < blocks; k += kThreads) {
        const uint32_t n = (uint32_t)a.s.free_in[k];
        all += n;
        if (k < k0) before += n;
    }
    before = wave_scan(before);
    all = wave_scan(all);
    if (lane == 63) {
        s_before[wave] = before;
        s_all[wave] = all;
    }
    __syncthreads();
    before = s_before[0] + s_before[1] + s_before[2] + s_before[3];
    const uint32_t used = a.c.num_pages - (s_all[0] + s_all[1] + s_all[2] + s_all[3]);
    if (blockIdx.x == 0 && tid == 0) {
        a.s.words[0] = used;
        if (used == 0) a.s.words[1] = 0;
        if (used_out) *used_out = (int32_t)used;
    }
    for (uint32_t k = k0; k < k1; ++k) {
        const uint32_t p = k * kBlock + tid;
        const bool in = p < a.c.num_pages, is_free = in && a.s.refs[p] == 0;
        const uint64_t frees = __ballot(is_free);
        if (lane == 0) part[wave] = __popcll(frees);
        __syncthreads();
        uint32_t at = before + lanes_below(frees);
        for (uint32_t w = 0; w < wave; ++w) at += part[w];
        before += part[0] + part[1] + part[2] + part[3];
        if (in) {
            // (the comparisons with num_pages keep counts that were written to from leading outside)
            if (p < used) {
                if (is_free && at < a.c.num_pages) a.s.list[at] = p;
            } else if (!is_free) {
                const uint32_t j = used - (p - at) - 1;
                if (j < a.c.num_pages) a.s.from[j] = p;
                a.s.rank[p] = j;
            }
            if (p == used - 1) a.s.words[1] = at + is_free;
            if (moved && (p < used || is_free)) moved[p] = is_free ? -1 : (int32_t)p;
        }
        __syncthreads();
    }
}

// The table renamed, counts and pages moved (475 MB read and written in 196 us,
// 4.8 TB/s; a workgroup a page and pool at a time, whose rows are one run).
__global__ __launch_bounds__(kCopyThreads) void k_fill(PageArgs a, Pools pools, uint32_t count, Geometry gk, Geometry gv,
                                                       uint64_t page_k, uint64_t page_v, uint32_t width, uint32_t blocks,
                                                       int32_t *moved, bool first_launch) {
    const uint32_t used = a.s.words[0], moves = min(a.s.words[1], a.c.num_pages);
    if (first_launch) {
        const uint32_t id = blockIdx.x * kCopyThreads + threadIdx.x, step = gridDim.x * kCopyThreads;
        for (uint32_t k = id; k < blocks; k += step) {
            const uint32_t end = min((k + 1) * kBlock, a.c.num_pages);
            a.s.free_in[k] = (int32_t)(end - min(end, max(used, k * kBlock)));
        }
        for (uint32_t m = id; m < moves; m += step) {
            const uint32_t source = a.s.from[m], target = a.s.list[m];
            if (source >= a.c.num_pages || target >= a.c.num_pages) continue;
            a.s.refs[target] = a.s.refs[source];
            a.s.refs[source] = 0;
            if (moved) moved[source] = (int32_t)target;
        }
        if (moves)
            for (uint64_t i = id; i < (uint64_t)a.c.batch * width; i += step) {
                const uint32_t b = (uint32_t)(i / width);
                int32_t *entry = a.table + b * a.c.table_stride + (i - (uint64_t)b * width);
                const uint32_t page = (uint32_t)*entry;
                if (page < used || page >= a.c.num_pages) continue;
                const uint32_t rank = a.s.rank[page];
                if (rank < moves) *entry = (int32_t)a.s.list[rank];
            }
    }
    for (uint64_t i = blockIdx.x; i < (uint64_t)moves * count; i += gridDim.x) {
        const uint32_t m = (uint32_t)(i / count), pool = (uint32_t)(i - (uint64_t)m * count);
        const uint32_t source = a.s.from[m], target = a.s.list[m];
        if (source >= a.c.num_pages || target >= a.c.num_pages) continue;
        const uint64_t step = pool & 1 ? page_v : page_k;
        copy_page(pools.p[pool] + source * step, pools.p[pool] + target * step, pool & 1 ? gv : gk, a.c.page.d);
    }
}

// ---------------------------------------------------------------------------
// copy
// ---------------------------------------------------------------------------

struct CopyArgs {
    const int32_t *src, *dst;
    uint32_t n, from_pages, to_pages, slots, count;
    uint64_t from_k, from_v, to_k, to_v;      // elements between pages
    int32_t *status;
};

// A workgroup a page and pool: 537 MB read and written in 209 us, 5.1 TB/s (a
// large device-to-device copy 4.9); 19 pages of 32 layers, 40 MB, in 16.
__global__ __launch_bounds__(kCopyThreads) void k_copy(CopyArgs a, Pools from, Pools to, Geometry gk, Geometry gv) {
    for (uint64_t i = blockIdx.x; i < (uint64_t)a.n * a.count; i += gridDim.x) {
        const uint32_t m = (uint32_t)(i / a.count), pool = (uint32_t)(i - (uint64_t)m * a.count);
        const uint32_t source = (uint32_t)a.src[m], target = (uint32_t)a.dst[m];
        if (source >= a.from_pages || target >= a.to_pages) {
            if (threadIdx.x == 0) report(a.status, SPLITZIP_KV_BAD_PAGE);
            continue;
        }
        copy_page(from.p[pool] + source * (pool & 1 ? a.from_v : a.from_k), to.p[pool] + target * (pool & 1 ? a.to_v : a.to_k),
                  pool & 1 ? gv : gk, a.slots);
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

inline uint32_t blocks_of(uint32_t pages) { return (pages - 1) / kBlock + 1; }

bool pages_shape_ok(const splitzip_kv_cache *c) {
    return shape_ok(c) && c->num_pages >= 1 && c->num_pages <= SPLITZIP_KV_MAX_PAGES;
}

size_t place_state(const splitzip_kv_cache *c, void *base, State &s) {
    uint8_t *p = reinterpret_cast<uint8_t *>(base);
    const size_t n = up16(4 * (size_t)c->num_pages);
    s.refs = reinterpret_cast<int32_t *>(p);
    s.writers = reinterpret_cast<int32_t *>(p + n);
    s.lowest = reinterpret_cast<int32_t *>(p + 2 * n);
    s.list = reinterpret_cast<uint32_t *>(p + 3 * n);
    s.from = reinterpret_cast<uint32_t *>(p + 4 * n);
    s.rank = reinterpret_cast<uint32_t *>(p + 5 * n);
    s.words = reinterpret_cast<uint32_t *>(p + 6 * n);
    s.want = reinterpret_cast<Want *>(p + 6 * n + 32);
    size_t at = 6 * n + 32 + sizeof(Want) * (size_t)c->batch;
    s.free_in = reinterpret_cast<int32_t *>(p + at);
    at += up16(4 * (size_t)blocks_of(c->num_pages));
    s.left = reinterpret_cast<int32_t *>(p + at);
    return at + up16(4 * (size_t)c->batch);
}

// The pools alone: shape, strides, alignment, reach.
bool pools_ok(const splitzip_kv_pages *p) {
    if (!p || !p->cache || !p->k || !p->v || p->layers < 1 || p->layers > SPLITZIP_KV_MAX_LAYERS) return false;
    splitzip_kv_cache c = *p->cache;
    if (!pages_shape_ok(&c) || (uint64_t)c.page_size * c.kv_heads * (c.head_dim / 8) >> 31) return false;
    c.batch = 0;
    c.k = p->k[0];
    c.v = p->v[0];
    if (!cache_ok(&c)) return false;
    for (uint32_t i = 1; i < p->layers; ++i)      // shape and strides are those of all layers
        if (!p->k[i] || !p->v[i] || !aligned(p->k[i], 16) || !aligned(p->v[i], 16)) return false;
    return true;
}

int prepare(const splitzip_kv_pages *p, const int32_t *arg, int32_t *d_status, PageArgs &a) {
    if (!pools_ok(p) || (d_status && !aligned(d_status, 4)) || !aligned(arg, 4)) return SPLITZIP_ERR_INVALID;
    splitzip_kv_cache c = *p->cache;
    c.k = p->k[0];
    c.v = p->v[0];
    if ((uint64_t)c.batch * c.max_pages >> 31) return SPLITZIP_ERR_INVALID;
    if (!cache_ok(&c) || !p->state || !aligned(p->state, 16)) return SPLITZIP_ERR_INVALID;
    if (p->state_bytes < place_state(&c, p->state, a.s)) return SPLITZIP_ERR_WORKSPACE;
    a.c = view(&c);
    a.table = const_cast<int32_t *>(c.table);
    a.arg = arg;
    a.status = d_status;
    return SPLITZIP_OK;
}

// Pages of `from` as pages of `to`, whose shapes are equal; `part`: the first
// slots alone may be copied.
Geometry geometry(const splitzip_kv_cache *from, const splitzip_kv_cache *to, bool v, bool part) {
    const uint64_t *s = v ? from->v_stride : from->k_stride, *d = v ? to->v_stride : to->k_stride;
    // strides of a dimension of one entry mean nothing
    const bool slot_first = from->page_size > 1 && (from->kv_heads == 1 || s[1] < s[2]);
    uint32_t n0 = slot_first ? from->page_size : from->kv_heads, n1 = slot_first ? from->kv_heads : from->page_size;
    Geometry g{};
    g.s0 = s[slot_first ? 2 : 1], g.s1 = s[slot_first ? 1 : 2];
    g.d0 = d[slot_first ? 2 : 1], g.d1 = d[slot_first ? 1 : 2];
    uint32_t run = from->head_dim / 8;
    g.per_slot = from->kv_heads * run;
    g.total = n0 * n1 * run;
    // rows that follow each other in both are one run
    auto joins = [&](uint32_t n, uint64_t ss, uint64_t ds) { return n == 1 || (ss == run * 8ull && ds == ss); };
    if ((slot_first || !part) && joins(n1, g.s1, g.d1)) {
        run *= n1;
        n1 = 1;
        if (!part && joins(n0, g.s0, g.d0)) {
            run *= n0;
            n0 = 1;
        }
    }
    g.slot_first = slot_first;
    g.run = make_div(run);
    g.n1 = make_div(n1);
    return g;
}

// Calls launch(pools from the layer, layers) for as many layers a time as a
// launch takes.
template <typename F>
int by_layers(const splitzip_kv_pages *p, F launch) {
    for (uint32_t l0 = 0; l0 < p->layers; l0 += kMaxPools / 2) {
        const uint32_t n = p->layers - l0 < kMaxPools / 2 ? p->layers - l0 : kMaxPools / 2;
        launch(l0, n);
        const int rc = launched();
        if (rc) return rc;
    }
    return SPLITZIP_OK;
}

Pools pools_from(const splitzip_kv_pages *p, uint32_t l0, uint32_t n) {
    Pools q{};
    for (uint32_t i = 0; i < n; ++i) {
        q.p[2 * i] = p->k[l0 + i];
        q.p[2 * i + 1] = p->v[l0 + i];
    }
    return q;
}

constexpr uint32_t kGrid = 2048;     // workgroups of the loops over many items: eight a compute unit

inline uint32_t grid_for(uint64_t items) { return items < kGrid ? (items ? (uint32_t)items : 1) : kGrid; }

}  // namespace

extern "C" {

size_t splitzip_kv_pages_struct_size(void) { return sizeof(splitzip_kv_pages); }

size_t splitzip_kv_pages_state_size(const splitzip_kv_cache *cache) {
    State s;
    return pages_shape_ok(cache) ? place_state(cache, nullptr, s) : 0;
}

int splitzip_kv_pages_count(const splitzip_kv_pages *pages, int32_t *d_status, void *stream) {
    PageArgs a{};
    if (const int rc = prepare(pages, nullptr, d_status, a)) return rc;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const uint32_t width = pages->cache->max_pages, blocks = blocks_of(a.c.num_pages);
    if (a.c.num_pages <= kSmallPages && (uint64_t)a.c.batch * width <= kSmallEntries) {
        k_count<<<1, kSmallThreads, 0, s>>>(a, width);
        return launched();
    }
    k_clear<<<grid_for(blocks), kThreads, 0, s>>>(a);
    int rc = launched();
    if (!rc && a.c.batch && width) {
        // eight entries a thread of the widest rows
        const uint32_t parts = (width - 1) / (8 * kThreads) + 1;
        k_names<<<grid_for((uint64_t)a.c.batch * parts), kThreads, 0, s>>>(a, width, parts);
        rc = launched();
    }
    if (!rc) {
        k_free<<<grid_for(blocks), kThreads, 0, s>>>(a, blocks);
        rc = launched();
    }
    return rc;
}

int splitzip_kv_pages_fork(const splitzip_kv_pages *pages, const int32_t *parents, int32_t *d_status, void *stream) {
    PageArgs a{};
    if (const int rc = prepare(pages, parents, d_status, a)) return rc;
    if (a.c.batch == 0) return SPLITZIP_OK;
    if (!parents) return SPLITZIP_ERR_INVALID;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const uint32_t width = pages->cache->max_pages, batch = a.c.batch;
    // Rows a thread: four, and as many more as leave a workgroup at least one
    // column; 16 columns, a cache line, as far as that goes.
    const int u = batch <= 4 * kForkThreads ? 4 : batch <= 16 * kForkThreads ? 16 : 64;
    const uint32_t ways = (batch - 1) / u + 1;      // threads a column
    uint32_t columns = 16;
    while (columns > 1 && ways > kForkThreads / columns) columns >>= 1;
    uint32_t threads = ways * columns;
    threads = threads <= 64 ? 64 : (threads + 63) / 64 * 64;
    const uint32_t grid = (width ? (width - 1) / columns + 1 : 0) + 1;
    if (u == 4) k_fork<4><<<grid, threads, (batch / 2 + 1) * 4, s>>>(a, width, columns);
    else if (u == 16) k_fork<16><<<grid, threads, (batch / 2 + 1) * 4, s>>>(a, width, columns);
    else k_fork<64><<<grid, threads, (batch / 2 + 1) * 4, s>>>(a, width, columns);
    return launched();
}

int splitzip_kv_pages_resize(const splitzip_kv_pages *pages, const int32_t *lens, int32_t *d_status, void *stream) {
    PageArgs a{};
    if (const int rc = prepare(pages, lens, d_status, a)) return rc;
    if (a.c.batch == 0) return SPLITZIP_OK;
    if (!lens) return SPLITZIP_ERR_INVALID;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const uint32_t width = pages->cache->max_pages, blocks = blocks_of(a.c.num_pages);
    if (a.c.batch <= kChooseThreads) {
        k_choose<true><<<1, kChooseThreads, 0, s>>>(a, width, blocks);
    } else {
        k_want<<<(a.c.batch - 1) / (kThreads / 64) + 1, kThreads, 0, s>>>(a, width);
        if (const int rc = launched()) return rc;
        k_choose<false><<<1, kChooseThreads, 0, s>>>(a, width, blocks);
    }
    if (const int rc = launched()) return rc;
    const splitzip_kv_cache *c = pages->cache;
    const Geometry gk = geometry(c, c, false, true), gv = geometry(c, c, true, true);
    return by_layers(pages, [&](uint32_t l0, uint32_t n) {
        k_give<<<dim3(a.c.batch, 2 * n), kCopyThreads, 0, s>>>(a, pools_from(pages, l0, n), gk, gv, c->k_stride[0], c->v_stride[0],
                                                               l0 == 0);
    });
}

int splitzip_kv_pages_compact(const splitzip_kv_pages *pages, int32_t *moved, int32_t *used, int32_t *d_status, void *stream) {
    PageArgs a{};
    if (!aligned(moved, 4) || !aligned(used, 4)) return SPLITZIP_ERR_INVALID;
    if (const int rc = prepare(pages, nullptr, d_status, a)) return rc;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const uint32_t blocks = blocks_of(a.c.num_pages);
    k_holes<<<blocks < 1024 ? blocks : 1024, kThreads, 0, s>>>(a, blocks, moved, used);
    const int rc = launched();
    if (rc) return rc;
    const splitzip_kv_cache *c = pages->cache;
    const Geometry gk = geometry(c, c, false, false), gv = geometry(c, c, true, false);
    return by_layers(pages, [&](uint32_t l0, uint32_t n) {
        // at most half of the pages move; the table is renamed by the same workgroups
        const uint64_t items = (uint64_t)(a.c.num_pages / 2) * 2 * n, entries = ((uint64_t)a.c.batch * c->max_pages) / kCopyThreads + 1;
        k_fill<<<grid_for(items > entries ? items : entries), kCopyThreads, 0, s>>>(
            a, pools_from(pages, l0, n), 2 * n, gk, gv, c->k_stride[0], c->v_stride[0], c->max_pages, blocks, moved, l0 == 0);
    });
}

int splitzip_kv_pages_copy(const splitzip_kv_pages *from, const splitzip_kv_pages *to, const int32_t *src, const int32_t *dst,
                           uint32_t n, int32_t *d_status, void *stream) {
    if (!pools_ok(from) || !pools_ok(to) || !aligned(src, 4) || !aligned(dst, 4) || (d_status && !aligned(d_status, 4)))
        return SPLITZIP_ERR_INVALID;
    const splitzip_kv_cache *f = from->cache, *t = to->cache;
    if (from->layers != to->layers || f->page_size != t->page_size || f->kv_heads != t->kv_heads || f->head_dim != t->head_dim ||
        f->dtype != t->dtype || n > 0x7fffffffu)
        return SPLITZIP_ERR_INVALID;
    if (n == 0) return SPLITZIP_OK;
    if (!src || !dst) return SPLITZIP_ERR_INVALID;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    CopyArgs a{src, dst, n, f->num_pages, t->num_pages, f->page_size, 0, f->k_stride[0], f->v_stride[0], t->k_stride[0], t->v_stride[0],
               d_status};
    const Geometry gk = geometry(f, t, false, false), gv = geometry(f, t, true, false);
    return by_layers(from, [&](uint32_t l0, uint32_t layers) {
        a.count = 2 * layers;
        const uint64_t items = (uint64_t)n * a.count;
        const uint32_t most = 1u << 20;
        k_copy<<<items < most ? (uint32_t)items : most, kCopyThreads, 0, s>>>(a, pools_from(from, l0, layers), pools_from(to, l0, layers), gk, gv);
    });
}

}  // extern "C"
