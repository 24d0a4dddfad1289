// kv.hip -- paged key-value cache for MI355X (gfx950): HIP kernels and the C
// ABI declared in include/splitzip_kv.h.
//
//   k_rows    rows <-> pages (append and gather), 16-byte copies
//   k_attend, k_join  (kv_attend.h) attention of one new token per sequence
//   k_select  per KV head, which tokens an eviction keeps
//   k_move    the kept tokens' K and V to their new places
//
// Memory bounds all of them where there is work to fill the GPU, and chains of
// dependent loads (a length, page numbers, rows) where there is not.  Every
// page number and length is checked where it is read.  Times below are of one
// MI355X, a pass among others with inputs that change from pass to pass.

#include "kv_attend.h"
#include "kv_cache.h"

namespace {

// ---------------------------------------------------------------------------
// append / gather
// ---------------------------------------------------------------------------

struct RowArgs {
    Cache c;
    uint16_t *k, *v;
    uint64_t ks[2], vs[2];
    uint32_t rows, per_wg, groups;   // rows a workgroup takes at a time; groups of that many
    const int32_t *cu, *start;
    int32_t *status;
    Div chunks, items;    // 16-byte pieces of a head's row; of a whole row
};

constexpr int kRowThreads = 256;
constexpr int kRowMax = 64;      // rows a workgroup

// A workgroup copies per_wg rows: one thread per row finds its place, then
// all threads copy 16-byte pieces, neighbouring threads neighbouring pieces.
// Memory bounds it: 268 MB move in 48 us (5.6 TB/s), with loads and stores that
// leave the caches alone where nothing reads the bytes again soon.
template <bool GATHER>
__global__ __launch_bounds__(kRowThreads) void k_rows(RowArgs a) {
    __shared__ uint64_t at_k[kRowMax], at_v[kRowMax];
    constexpr uint64_t kNone = ~0ull;
    for (uint32_t wg = blockIdx.x; wg < a.groups; wg += gridDim.x) {
        const uint32_t r0 = wg * a.per_wg;
        const uint32_t count = min(a.per_wg, a.rows - r0);
        if (threadIdx.x < count) {
            const uint32_t r = r0 + threadIdx.x;
            // first entry of cu above r
            uint32_t lo = 0, hi = a.c.batch + 1;
            while (lo < hi) {
                const uint32_t mid = (lo + hi) >> 1;
                if (a.cu[mid] > (int64_t)r) hi = mid; else lo = mid + 1;
            }
            uint64_t pk = kNone, pv = kNone;
            if (lo > 0 && lo <= a.c.batch) {
                const uint32_t b = lo - 1;
                const int64_t first = a.cu[b], end = a.cu[b + 1];
                // with first positions given, a length need not be set yet
                const int64_t from = a.start ? (int64_t)a.start[b] : (int64_t)seq_len(a.c, b, a.status) - (end - first);
                const int64_t pos = from + ((int64_t)r - first);
                uint32_t page, slot;
                if (first < 0 || first > (int64_t)r || end > (int64_t)a.rows || pos < 0 || pos >= (int64_t)a.c.max_len) {
                    report(a.status, SPLITZIP_KV_BAD_ROWS);
                } else if (!locate(a.c, b, (uint32_t)pos, page, slot)) {
                    report(a.status, SPLITZIP_KV_BAD_PAGE);
                } else {
                    pk = page * a.c.ks[0] + slot * a.c.ks[2];
                    pv = page * a.c.vs[0] + slot * a.c.vs[2];
                }
            }
            at_k[threadIdx.x] = pk;
            at_v[threadIdx.x] = pv;
        }
        __syncthreads();
        const uint32_t total = count * a.items.d;
        for (uint32_t i = threadIdx.x; i < total; i += kRowThreads) {
            const uint32_t r = div(i, a.items), j = i - r * a.items.d;
            const uint32_t h = div(j, a.chunks), d = (j - h * a.chunks.d) * 8;
            if (at_k[r] == kNone) continue;
            uint16_t *pk = a.c.k + at_k[r] + h * a.c.ks[1] + d;
            uint16_t *pv = a.c.v + at_v[r] + h * a.c.vs[1] + d;
            uint16_t *rk = a.k + (uint64_t)(r0 + r) * a.ks[0] + h * a.ks[1] + d;
            uint16_t *rv = a.v + (uint64_t)(r0 + r) * a.vs[0] + h * a.vs[1] + d;
            // pages are read for this once, new rows may still be in a cache
            const u32x4 xk = GATHER ? load_once(pk) : *(const u32x4 *)rk;
            const u32x4 xv = GATHER ? load_once(pv) : *(const u32x4 *)rv;
            store_away(GATHER ? rk : pk, xk);
            store_away(GATHER ? rv : pv, xv);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// evict
// ---------------------------------------------------------------------------

struct EvictArgs {
    Cache c, to;
    const float *mass;
    float *mass_out;
    uint64_t ms[2], mos[2];
    int32_t *kept;
    uint32_t budget, sinks, recent, mass_len;
    int32_t *status;
    uint32_t chunk, chunks, per_wg;   // k_move: 16-byte pieces of a column, columns, rows a workgroup
};

constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;

// The masses as unsigned integers of the same order: -0 as 0, NaN above all
// numbers; above NaN the tokens that stay whatever their mass, and below all
// keys (-inf has 0x007fffff) what is no token.
constexpr uint32_t kKeyAlways = 0xffffffffu, kKeyNan = 0xfffffffeu, kKeyNone = 0;

__device__ inline uint32_t mass_key(float m) {
    const uint32_t u = __float_as_uint(m + 0.f);   // -0 + 0 = 0
    const uint32_t key = u ^ (0x80000000u | (uint32_t)((int32_t)u >> 31));
    return m != m ? kKeyNan : key;
}

// Sum of part[0 .. wave - 1], of up to 16 waves: one look at LDS, a scan over
// 16 lanes.
__device__ inline uint32_t sum_before(const uint32_t *part, uint32_t wave) {
    uint32_t x = part[threadIdx.x & (kSelWaves - 1)];
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xf, 0xf, false);    // row_shr:1
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xf, 0xf, false);    // row_shr:2
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xf, 0xf, false);    // row_shr:4
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xf, 0xf, false);    // row_shr:8
    return wave ? __builtin_amdgcn_readlane(x, wave - 1) : 0u;
}
static_assert(kSelWaves == 16, "a DPP row holds a count of every wave");

// The threshold is found by its bits from the top, kSelDigits[i] of them a
// pass: a histogram in LDS of the keys that agree so far, and its suffix sums.
// The first digit of 11 bits is sign, exponent and two bits below, so that
// masses, which crowd into a few powers of two, spread over more than a few
// counters (LDS adds to one address take turns).
constexpr int kSelBits = 11, kSelBins = 1 << kSelBits, kSelPasses = 3;
// Copies of the first pass's histogram, by lane (32768 masses counted in 2.6 us
// with 8, 4.0 with 4, and more of them to clear and sum); later digits are
// spread enough for one.
constexpr int kSelCopies = 8;
constexpr int kSelHeld = 32;       // masses a thread can hold

// One workgroup per sequence and KV head: 8 us for 4096 tokens, 19 us for 32768
// (3 until the masses are there, 4.5, 2 and 2 for the passes, 5.5 to count and
// place what stays; the instructions of one compute unit bound it), 180 us for
// 131072, whose masses are read again by every pass.  Wave w has the run of tokens from
// w * span; lane l its tokens l, l + 64, ..., HELD of them in registers (all
// of them where span is at most 64 HELD, and then the masses are read once);
// HELD 0: read again by every pass.
template <int HELD>
__global__ __launch_bounds__(kSelThreads) void k_select(EvictArgs a) {
    __shared__ __align__(16) uint32_t hist[kSelBins * kSelCopies];
    __shared__ uint32_t part[kSelWaves], part2[kSelWaves];
    __shared__ uint32_t s_prefix, s_need;
    const uint32_t b = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int32_t *status = tid == 0 && h == 0 ? a.status : nullptr;
    uint32_t n = seq_len(a.c, b, status);
    if (n > a.mass_len) {
        report(status, SPLITZIP_KV_BAD_LEN);
        n = a.mass_len;
    }
    const float *mass = a.mass + b * a.ms[0] + h * a.ms[1];
    float *out = a.mass_out ? a.mass_out + b * a.mos[0] + h * a.mos[1] : nullptr;
    int32_t *kept = a.kept + ((uint64_t)b * a.c.kv_heads + h) * a.budget;
    if (n <= a.budget) {
        for (uint32_t t = tid; t < a.budget; t += kSelThreads) kept[t] = t < n ? (int32_t)t : -1;
        if (out && out != mass)
            for (uint32_t t = tid; t < n; t += kSelThreads) out[t] = mass[t];
        return;
    }
    const uint32_t span = ((n + kSelThreads - 1) / kSelThreads) * 64;
    const uint32_t w0 = min(n, wave * span), w1 = min(n, w0 + span);
    auto key_of = [&](uint32_t t, float m) {
        return t >= w1 ? kKeyNone : t < a.sinks || t >= n - a.recent ? kKeyAlways : mass_key(m);
    };
    float held[HELD ? HELD : 1];
    uint32_t keys[HELD ? HELD : 1];
    if (HELD) {
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const uint32_t t = w0 + i * 64 + lane;
            held[i] = t < w1 ? mass[t] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < HELD; ++i) keys[i] = key_of(w0 + i * 64 + lane, held[i]);
    }
    // f(token, mass, key) over the wave's run, in order
    auto each = [&](auto f) {
        if (HELD) {
#pragma unroll
            for (int i = 0; i < HELD; ++i)
                if (w0 + i * 64 < w1) f(w0 + i * 64 + lane, held[i], keys[i]);
        } else {
            for (uint32_t t = w0 + lane; t - lane < w1; t += 64) {
                const float m = t < w1 ? mass[t] : 0.f;
                f(t, m, key_of(t, m));
            }
        }
    };
    uint32_t prefix = 0, need = a.budget;
    for (int pass = 0; pass < kSelPasses; ++pass) {
        // the last digit repeats a bit of the one before, which is agreed on
        const int left = 32 - pass * kSelBits, shift = left > kSelBits ? left - kSelBits : 0;
        const uint32_t agreed = pass ? 0xffffffffu << left : 0u;
        const uint32_t copies = pass ? 1 : kSelCopies, copy = lane & (copies - 1);
        for (uint32_t k = tid; k < kSelBins / 4 * copies; k += kSelThreads) ((u32x4 *)hist)[k] = u32x4{0, 0, 0, 0};
        __syncthreads();
        each([&](uint32_t, float, uint32_t key) {
            if ((key & agreed) == prefix)
                atomicAdd(&hist[(key >> shift & (kSelBins - 1)) * copies + copy], 1u);
        });
        __syncthreads();
        // every mass is in registers now
        if (HELD && pass == 0 && out)
            for (uint32_t t = a.budget + tid; t < n; t += kSelThreads) out[t] = 0.f;
        // thread i has bins 2i and 2i + 1, counted from the top bin down
        const uint32_t top = kSelBins - 1 - 2 * tid;
        uint32_t c0, c1;
        if (pass) {
            const u32x2 both = *(const u32x2 *)&hist[top - 1];
            c0 = both[1], c1 = both[0];
        } else {
            u32x4 h0{0, 0, 0, 0}, h1 = h0;
#pragma unroll
            for (int k = 0; k < kSelCopies; k += 4) {
                h0 += *(const u32x4 *)&hist[top * kSelCopies + k];
                h1 += *(const u32x4 *)&hist[(top - 1) * kSelCopies + k];
            }
            c0 = h0[0] + h0[1] + h0[2] + h0[3], c1 = h1[0] + h1[1] + h1[2] + h1[3];
        }
        const uint32_t upto = wave_scan(c0 + c1);
        if (lane == 63) part[wave] = upto;
        __syncthreads();
        uint32_t above = upto - c0 - c1 + sum_before(part, wave);
        if (above < need && above + c0 >= need) {
            s_prefix = prefix | top << shift;
            s_need = need - above;
        }
        above += c0;
        if (above < need && above + c1 >= need) {
            s_prefix = prefix | (top - 1) << shift;
            s_need = need - above;
        }
        __syncthreads();
        prefix = s_prefix;
        need = s_need;
    }
    // Kept: the keys above the threshold, and the first `need` of those equal to
    // it.  A wave counts its own, then places them from where the waves before
    // it end.
    uint32_t mine = 0, ties = 0;
    each([&](uint32_t, float, uint32_t key) {
        mine += __popcll(__ballot(key > prefix));
        ties += __popcll(__ballot(key == prefix));
    });
    if (lane == 0) {
        part[wave] = mine;
        part2[wave] = ties;
    }
    __syncthreads();
    uint32_t at = sum_before(part, wave), eq = sum_before(part2, wave);
    at += min(eq, need);
    // mostly all of the equal ones stay, and one comparison tells
    const bool some = sum_before(part2, kSelWaves) > need;
    const uint32_t least = some ? prefix + 1 : prefix;
    // In place a mass moves to a position at or below its own; with all of
    // them in registers that is free of order, else see below.
    each([&](uint32_t t, float m, uint32_t key) {
        uint64_t all = __ballot(key >= least);
        if (const uint64_t same = some ? __ballot(key == prefix) : 0) {
            const uint32_t rank = eq + lanes_below(same);
            all |= __ballot(key == prefix && rank < need);
            eq += __popcll(same);
        }
        if (all >> lane & 1) {
            const uint32_t to = at + lanes_below(all);
            kept[to] = (int32_t)t;
            if (HELD && out) out[to] = m;
        }
        at += __popcll(all);
    });
    if (HELD || !out) return;
    // step by step upwards, a step's masses read before any of it is written
    __syncthreads();
    for (uint32_t t0 = 0; t0 < a.budget; t0 += kSelThreads) {
        const uint32_t t = t0 + tid;
        float m = 0.f;
        if (t < a.budget) m = mass[kept[t]];
        __syncthreads();
        if (t < a.budget) out[t] = m;
    }
    __syncthreads();
    for (uint32_t t = a.budget + tid; t < n; t += kSelThreads) out[t] = 0.f;
}

constexpr int kMoveThreads = 512;
// Rows a thread moves at a time: apart from the source, where workgroups are
// many, and in place, where one has a whole column (one sequence of 32768
// tokens, 8 KV heads of 128, all masses distinct: to 8192 98 us with 2, 70 with
// 4, 55 with 8, to 32000 366, 242 and 186).
constexpr int kMoveApart = 4, kMoveInPlace = 8;
constexpr uint32_t kMoveParts = 65536;
constexpr uint32_t kMoveRows = 64;      // most rows side by side in a workgroup
__host__ __device__ inline uint32_t move_rows(uint32_t chunk) { return kMoveThreads / chunk < kMoveRows ? kMoveThreads / chunk : kMoveRows; }

// A workgroup moves a column of one pool: `chunk` 16-byte pieces of the rows
// of a sequence's KV head.  Row i comes from row kept[i] >= i, so within a
// column, step by step upwards, a step's writes can only meet sources of the
// step itself: they wait until all its loads have arrived (the barrier), and
// steps need no other order.  Columns share nothing.  Memory bounds it where
// there are workgroups enough: 16 x 4096 tokens of 8 heads of 128 to half,
// 268 MB, in 54 us, in place too.  In place with few columns a step's three loads
// in turn do (one sequence of 32768 tokens of 8 heads to 8192 in 55 us, selection
// included); looking the next step's places up ahead gained nothing.
template <bool LINES, int U>
__global__ __launch_bounds__(kMoveThreads) void k_move(EvictArgs a) {
    __shared__ uint64_t from[kMoveRows * U], dest[kMoveRows * U];
    const uint32_t b = blockIdx.z, tid = threadIdx.x;
    const uint32_t h = blockIdx.y / (2 * a.chunks), col = blockIdx.y % (2 * a.chunks);
    const bool is_v = col >= a.chunks;
    const uint32_t piece0 = (is_v ? col - a.chunks : col) * a.chunk;
    const uint32_t width = min(a.chunk, a.c.dim / 8 - piece0);
    const uint32_t n = min(min(seq_len(a.c, b), a.mass_len), a.budget);
    const uint16_t *src = (is_v ? a.c.v : a.c.k) + h * (is_v ? a.c.vs[1] : a.c.ks[1]) + piece0 * 8;
    uint16_t *dst = (is_v ? a.to.v : a.to.k) + h * (is_v ? a.to.vs[1] : a.to.ks[1]) + piece0 * 8;
    const int32_t *kept = a.kept + ((uint64_t)b * a.c.kv_heads + h) * a.budget;
    const uint32_t lane_rows = move_rows(a.chunk), step = lane_rows * U;
    const uint32_t row = tid / a.chunk, piece = tid % a.chunk;
    const uint64_t begin = (uint64_t)blockIdx.x * a.per_wg, end = min((uint64_t)n, begin + a.per_wg);
    const bool same = a.to.k == a.c.k, mine = row < lane_rows && piece < width;
    constexpr uint64_t kNone = ~0ull;
    static_assert(kMoveRows * U <= kMoveThreads, "a thread per row of a step");
    for (uint64_t i0 = begin; i0 < end; i0 += step) {
        if (tid < step) {
            uint64_t f = kNone, d = kNone;
            if (i0 + tid < end) {
                const uint32_t i = (uint32_t)(i0 + tid), t = (uint32_t)kept[i];
                uint32_t p0, s0, p1, s1;
                // kept is as the selection left it: -1 where a length has grown since
                const bool here = t < a.c.max_len && locate(a.c, b, t, p0, s0), there = locate(a.to, b, i, p1, s1);
                if (!here || !there) {
                    report(a.status, SPLITZIP_KV_BAD_PAGE);
                } else if (!(same && t == i)) {
                    f = p0 * (is_v ? a.c.vs[0] : a.c.ks[0]) + s0 * (is_v ? a.c.vs[2] : a.c.ks[2]);
                    d = p1 * (is_v ? a.to.vs[0] : a.to.ks[0]) + s1 * (is_v ? a.to.vs[2] : a.to.ks[2]);
                }
            }
            from[tid] = f;
            dest[tid] = d;
        }
        __syncthreads();
        u32x4 x[U];
        bool ok[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t j = u * lane_rows + row;
            ok[u] = mine && from[j] != kNone;
            if (ok[u]) {
                const uint16_t *p = src + from[j] + piece * 8;
                x[u] = LINES ? load_once(p) : *(const u32x4 *)p;
            }
        }
        wait_vector_memory();
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (ok[u]) {
                uint16_t *p = dst + dest[u * lane_rows + row] + piece * 8;
                if (LINES) store_away(p, x[u]);
                else *(u32x4 *)p = x[u];
            }
        __syncthreads();
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) a.to.lens[b] = (int32_t)n;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

constexpr uint32_t kMaxGrid = 1u << 20;

int copy_rows(const splitzip_kv_cache *cache, const splitzip_kv_rows *r, int32_t *d_status, bool gather,
              void *stream) {
    if (!cache_ok(cache) || !r || (d_status && !aligned(d_status, 4))) return SPLITZIP_ERR_INVALID;
    if (r->rows > SPLITZIP_KV_MAX_ROWS) return SPLITZIP_ERR_INVALID;
    for (int i = 0; i < 2; ++i) {
        const uint64_t count = i == 0 ? r->rows : cache->kv_heads;
        if (r->k_stride[i] % 8 || r->v_stride[i] % 8 || !spans(r->k_stride[i], count) || !spans(r->v_stride[i], count))
            return SPLITZIP_ERR_INVALID;
    }
    if (r->rows == 0 || cache->batch == 0) return SPLITZIP_OK;
    if (!r->k || !r->v || !aligned(r->k, 16) || !aligned(r->v, 16) || !r->cu || !aligned(r->cu, 4) || !aligned(r->start, 4))
        return SPLITZIP_ERR_INVALID;
    RowArgs a{};
    a.c = view(cache);
    a.k = r->k;
    a.v = r->v;
    for (int i = 0; i < 2; ++i) {
        a.ks[i] = r->k_stride[i];
        a.vs[i] = r->v_stride[i];
    }
    a.rows = r->rows;
    a.cu = r->cu;
    a.start = r->start;
    a.status = d_status;
    a.chunks = make_div(cache->head_dim / 8);
    a.items = make_div(cache->kv_heads * (cache->head_dim / 8));
    // One piece of each pool a thread: 32768 rows of 8 x 128 gathered in 48 us
    // with one, 53 with two, 57 with four.
    uint32_t per = kRowThreads / a.items.d;
    if (per < 1) per = 1;
    if (per > (uint32_t)kRowMax) per = kRowMax;
    a.per_wg = per;
    a.groups = (r->rows - 1) / per + 1;
    const uint32_t grid = a.groups < kMaxGrid ? a.groups : kMaxGrid;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (gather) k_rows<true><<<grid, kRowThreads, 0, s>>>(a);
    else k_rows<false><<<grid, kRowThreads, 0, s>>>(a);
    return launched();
}

bool mass_strides_ok(const uint64_t s[2]) { return s[0] <= kMaxOffset && s[1] <= kMaxOffset; }

}  // namespace

extern "C" {

void splitzip_kv_struct_sizes(size_t sizes[4]) {
    sizes[0] = sizeof(splitzip_kv_cache);
    sizes[1] = sizeof(splitzip_kv_rows);
    sizes[2] = sizeof(splitzip_kv_query);
    sizes[3] = sizeof(splitzip_kv_budget);
}

int splitzip_kv_append(const splitzip_kv_cache *cache, const splitzip_kv_rows *rows, int32_t *d_status,
                       void *stream) {
    return copy_rows(cache, rows, d_status, false, stream);
}

int splitzip_kv_gather(const splitzip_kv_cache *cache, const splitzip_kv_rows *rows, int32_t *d_status,
                       void *stream) {
    return copy_rows(cache, rows, d_status, true, stream);
}

size_t splitzip_kv_attend_workspace_size(const splitzip_kv_cache *cache, uint32_t heads, uint32_t mass_len) {
    AttendPlan p;
    if (!shape_ok(cache) || !attend_plan(cache, heads, mass_len, p)) return 0;
    return p.bytes;
}

int splitzip_kv_attend(const splitzip_kv_cache *cache, const splitzip_kv_query *query, void *d_ws,
                       size_t ws_bytes, int32_t *d_status, void *stream) {
    if (!cache_ok(cache) || !query || (d_status && !aligned(d_status, 4))) return SPLITZIP_ERR_INVALID;
    const splitzip_kv_query &Q = *query;
    AttendPlan P;
    if (!attend_plan(cache, Q.heads, Q.mass_out ? Q.mass_len : 0, P) || !(Q.scale * kLog2e - Q.scale * kLog2e == 0.f))
        return SPLITZIP_ERR_INVALID;      // also a scale that is not finite in base 2
    for (int i = 0; i < 2; ++i)
        if (Q.q_stride[i] % 8 || Q.out_stride[i] % 8 || Q.q_stride[i] > kMaxOffset || Q.out_stride[i] > kMaxOffset)
            return SPLITZIP_ERR_INVALID;
    if (!mass_strides_ok(Q.mass_stride) || !mass_strides_ok(Q.mass_out_stride) || (Q.mass && !Q.mass_out) ||
        !aligned(Q.mass, 4) || !aligned(Q.mass_out, 4) || !aligned(Q.lse, 4))
        return SPLITZIP_ERR_INVALID;
    if (cache->batch == 0) return SPLITZIP_OK;
    if (!Q.q || !Q.out || !aligned(Q.q, 16) || !aligned(Q.out, 16) || !d_ws || !aligned(d_ws, 16))
        return SPLITZIP_ERR_INVALID;
    if (ws_bytes < P.bytes) return SPLITZIP_ERR_WORKSPACE;
    AttendArgs a{};
    a.c = view(cache);
    a.q = Q.q;
    a.out = Q.out;
    a.lse = Q.lse;
    a.mass = Q.mass;
    a.mass_out = Q.mass_out;
    for (int i = 0; i < 2; ++i) {
        a.qs[i] = Q.q_stride[i];
        a.os[i] = Q.out_stride[i];
        a.ms[i] = Q.mass_stride[i];
        a.mos[i] = Q.mass_out_stride[i];
    }
    a.heads = Q.heads;
    a.group = P.group;
    a.row_tiles = P.row_tiles;
    a.rows = P.rows;
    a.window = Q.window;
    a.sinks = Q.sinks;
    a.scale2 = Q.scale * kLog2e;
    a.mass_len = Q.mass_len;
    a.status = d_status;
    uint8_t *ws = reinterpret_cast<uint8_t *>(d_ws);
    a.splits = reinterpret_cast<uint32_t *>(ws);
    a.share_o = reinterpret_cast<float *>(ws + P.o_at);
    a.share_ml = reinterpret_cast<float *>(ws + P.ml_at);
    if (Q.mass_out && P.logit_stride) {
        a.lse2 = reinterpret_cast<float *>(ws + P.lse2_at);
        a.logits = reinterpret_cast<float *>(ws + P.logits_at);
        a.logit_stride = P.logit_stride;
        a.logit_len = (uint32_t)P.logit_stride;
    }
    // no sequence sees more than this
    const uint64_t window = (uint64_t)Q.window + Q.sinks;
    const uint64_t seen = Q.window == SPLITZIP_KV_ALL || window > a.c.max_len ? a.c.max_len : window;
    const uint32_t grid_x = lay_out(a, P, seen);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool bf16 = cache->dtype == SPLITZIP_KV_BF16;
    if (bf16) launch_attend<true>(a, P.blocks, grid_x, s);
    else launch_attend<false>(a, P.blocks, grid_x, s);
    int rc = launched();
    if (rc) return rc;
    // a mass of no tokens: one part that reports the sequences that have some
    const uint32_t parts = a.logits ? (uint32_t)((P.logit_stride - 1) / kMassTokens + 1) : Q.mass_out ? 1 : 0;
    if (a.runs || parts) {
        const dim3 grid((a.runs ? Q.heads : 0) + parts * cache->kv_heads, cache->batch);
        if (bf16) k_join<true><<<grid, kJoinThreads, 0, s>>>(a);
        else k_join<false><<<grid, kJoinThreads, 0, s>>>(a);
        rc = launched();
    }
    return rc;
}

int splitzip_kv_evict(const splitzip_kv_cache *cache, const splitzip_kv_cache *to,
                      const splitzip_kv_budget *budget, int32_t *d_status, void *stream) {
    if (!cache_ok(cache) || !cache_ok(to) || !budget || (d_status && !aligned(d_status, 4)))
        return SPLITZIP_ERR_INVALID;
    const splitzip_kv_budget &B = *budget;
    if (to->batch != cache->batch || to->kv_heads != cache->kv_heads || to->head_dim != cache->head_dim || to->dtype != cache->dtype)
        return SPLITZIP_ERR_INVALID;
    if (B.budget == 0 || B.budget > 0x7fffffffu || B.sinks > B.budget || B.recent > B.budget - B.sinks)
        return SPLITZIP_ERR_INVALID;
    const uint64_t all = (uint64_t)cache->max_pages * cache->page_size;
    if ((uint64_t)to->max_pages * to->page_size < (all < B.budget ? all : B.budget)) return SPLITZIP_ERR_INVALID;
    if (cache->batch == 0) return SPLITZIP_OK;
    const bool share = to->table == cache->table || to->lens == cache->lens || to->k == cache->k || to->v == cache->v;
    if (share) {
        bool same = to->k == cache->k && to->v == cache->v && to->table == cache->table && to->table_stride == cache->table_stride &&
                    to->lens == cache->lens && to->num_pages == cache->num_pages && to->page_size == cache->page_size && to->max_pages == cache->max_pages;
        for (int i = 0; i < 3; ++i) same = same && to->k_stride[i] == cache->k_stride[i] && to->v_stride[i] == cache->v_stride[i];
        if (!same) return SPLITZIP_ERR_INVALID;
    }
    if (!B.mass || !B.kept || !aligned(B.mass, 4) || !aligned(B.mass_out, 4) || !aligned(B.kept, 4) ||
        !mass_strides_ok(B.mass_stride) || !mass_strides_ok(B.mass_out_stride))
        return SPLITZIP_ERR_INVALID;
    EvictArgs a{};
    a.c = view(cache);
    a.to = view(to);
    a.mass = B.mass;
    a.mass_out = B.mass_out;
    for (int i = 0; i < 2; ++i) {
        a.ms[i] = B.mass_stride[i];
        a.mos[i] = B.mass_out_stride[i];
    }
    a.kept = B.kept;
    a.budget = B.budget;
    a.sinks = B.sinks;
    a.recent = B.recent;
    a.mass_len = B.mass_len;
    a.status = d_status;
    const uint32_t pieces = cache->head_dim / 8;
    // columns of 256 bytes; in place, where a column is one workgroup's, of 128
    const uint32_t wide = share ? 8 : 16;
    a.chunk = pieces < wide ? pieces : wide;
    a.chunks = (pieces + a.chunk - 1) / a.chunk;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const dim3 heads(cache->kv_heads, cache->batch);
    // By the longest there can be; the lengths are on the device.  16 x 4096 tokens
    // in a table and masses for 4096, 16384 and 131072: 7.2, 12.1 and 10.5 us, one
    // sequence of 32768 in those for 32768 and 131072 19 and 45.
    const uint64_t longest = all < B.mass_len ? all : B.mass_len;
    if (longest <= 4 * kSelThreads) k_select<4><<<heads, kSelThreads, 0, s>>>(a);
    else if (longest <= kSelHeld * kSelThreads) k_select<kSelHeld><<<heads, kSelThreads, 0, s>>>(a);
    else k_select<0><<<heads, kSelThreads, 0, s>>>(a);
    const int rc = launched();
    if (rc) return rc;
    const uint32_t most = (uint32_t)(all < B.budget ? all : B.budget);
    uint32_t parts = 1;
    a.per_wg = most ? most : 1;
    if (!share) {
        const uint32_t step = move_rows(a.chunk) * kMoveApart;
        const uint32_t steps = most ? (most - 1) / step + 1 : 1;
        a.per_wg = (steps - 1) / kMoveParts + 1;
        parts = (steps - 1) / a.per_wg + 1;
        a.per_wg *= step;
    }
    const dim3 grid(parts, cache->kv_heads * 2 * a.chunks, cache->batch);
    // Apart, rows of whole cache lines pass the caches by, as in k_attend; in place
    // they go through them (8 heads of 128, all masses distinct, through and past
    // them: 32768 to 8192 tokens 55 and 68 us, to 32000 186 and 209, 16 x 4096 to
    // 2048 59 and 62, 64 x 4096 to 4000 438 and 433).
    if (share) k_move<false, kMoveInPlace><<<grid, kMoveThreads, 0, s>>>(a);
    else if (cache->head_dim % 64 == 0) k_move<true, kMoveApart><<<grid, kMoveThreads, 0, s>>>(a);
    else k_move<false, kMoveApart><<<grid, kMoveThreads, 0, s>>>(a);
    return launched();
}

}  // extern "C"
