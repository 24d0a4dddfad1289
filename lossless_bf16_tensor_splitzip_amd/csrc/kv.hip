// kv.hip -- paged key-value cache for MI355X (gfx950): HIP kernels and the C
// ABI declared in include/splitzip_kv.h.
//
//   k_rows    rows <-> pages (append and gather), 16-byte copies
//   k_attend  attention of one new token per sequence over its cached tokens
//   k_select  per KV head, which tokens an eviction keeps
//   k_move    the kept tokens' K and V to their new places

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
                const uint32_t len = seq_len(a.c, b, a.status);
                const int64_t pos = (a.start ? (int64_t)a.start[b] : (int64_t)len - (end - first)) + ((int64_t)r - first);
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
#pragma unroll 4
        for (uint32_t i = threadIdx.x; i < total; i += kRowThreads) {
            const uint32_t r = div(i, a.items), j = i - r * a.items.d;
            const uint32_t h = div(j, a.chunks), d = (j - h * a.chunks.d) * 8;
            if (at_k[r] == kNone) continue;
            uint16_t *pk = a.c.k + at_k[r] + h * a.c.ks[1] + d;
            uint16_t *pv = a.c.v + at_v[r] + h * a.c.vs[1] + d;
            uint16_t *rk = a.k + (uint64_t)(r0 + r) * a.ks[0] + h * a.ks[1] + d;
            uint16_t *rv = a.v + (uint64_t)(r0 + r) * a.vs[0] + h * a.vs[1] + d;
            const u32x4 xk = *(const u32x4 *)(GATHER ? pk : rk);
            const u32x4 xv = *(const u32x4 *)(GATHER ? pv : rv);
            *(u32x4 *)(GATHER ? rk : pk) = xk;
            *(u32x4 *)(GATHER ? rv : pv) = xv;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// attend
// ---------------------------------------------------------------------------

struct AttendArgs {
    Cache c;
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    const float *mass;
    float *mass_out;
    uint64_t qs[2], os[2], ms[2], mos[2];
    uint32_t heads, group, window, sinks, mass_len;
    float scale;
    float *weights;
    int32_t *status;
};

template <bool BF16>
__device__ inline float to_float(uint16_t x) {
    if (BF16) return __uint_as_float((uint32_t)x << 16);
    return (float)__builtin_bit_cast(_Float16, x);
}
template <bool BF16>
__device__ inline uint16_t from_float(float x) {
    if (BF16) return __builtin_bit_cast(uint16_t, (__bf16)x);
    return __builtin_bit_cast(uint16_t, (_Float16)x);
}

constexpr int kAttendThreads = 256;

template <bool MAX>
__device__ inline float block_reduce(float x, float *part) {
    for (int k = 32; k; k >>= 1) {
        const float y = __shfl_xor(x, k);
        x = MAX ? fmaxf(x, y) : x + y;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    x = part[0];
    for (int w = 1; w < kAttendThreads / 64; ++w) x = MAX ? fmaxf(x, part[w]) : x + part[w];
    return x;
}

// One workgroup per sequence and KV head, the group's query heads one after
// another: a thread takes a token's logit, then an element of the output.
template <bool BF16>
__global__ __launch_bounds__(kAttendThreads) void k_attend(AttendArgs a) {
    __shared__ float q[SPLITZIP_KV_MAX_DIM], p[kAttendThreads], part[kAttendThreads / 64];
    __shared__ uint64_t at[kAttendThreads];
    const uint32_t b = blockIdx.x, h = blockIdx.y, D = a.c.dim;
    const uint32_t n = seq_len(a.c, b, threadIdx.x == 0 && h == 0 ? a.status : nullptr);
    const uint32_t first = a.window >= n ? 0 : n - a.window;
    const uint32_t s = min(a.sinks, first), seen = s + (n - first);
    for (uint32_t g = 0; g < a.group; ++g) {
        const uint32_t head = h * a.group + g;
        __syncthreads();
        for (uint32_t d = threadIdx.x; d < D; d += kAttendThreads)
            q[d] = to_float<BF16>(a.q[b * a.qs[0] + head * a.qs[1] + d]);
        __syncthreads();
        auto logit = [&](uint32_t i, uint64_t &v_at) {
            if (i >= seen) return -INFINITY;
            const uint32_t t = i < s ? i : first + (i - s);
            uint32_t page, slot;
            if (!locate(a.c, b, t, page, slot)) {
                report(a.status, SPLITZIP_KV_BAD_PAGE);
                return -INFINITY;
            }
            const uint16_t *k = a.c.k + page * a.c.ks[0] + h * a.c.ks[1] + slot * a.c.ks[2];
            v_at = page * a.c.vs[0] + h * a.c.vs[1] + slot * a.c.vs[2];
            float x = 0.f;
            for (uint32_t d = 0; d < D; ++d) x = fmaf(q[d], to_float<BF16>(k[d]), x);
            return x * a.scale;
        };
        float m = -INFINITY, l = 0.f, o = 0.f;
        for (uint32_t i0 = 0; i0 < seen; i0 += kAttendThreads) {
            uint64_t v_at = ~0ull;
            const float x = logit(i0 + threadIdx.x, v_at);
            const float m1 = fmaxf(m, block_reduce<true>(x, part));
            const float e = v_at == ~0ull || m1 == -INFINITY ? 0.f : expf(x - m1);
            const float r = m == -INFINITY ? 0.f : expf(m - m1);
            l = l * r + block_reduce<false>(e, part);
            __syncthreads();
            p[threadIdx.x] = e;
            at[threadIdx.x] = v_at;
            __syncthreads();
            o *= r;
            if (threadIdx.x < D)
                for (uint32_t j = 0; j < kAttendThreads; ++j)
                    if (at[j] != ~0ull) o = fmaf(p[j], to_float<BF16>(a.c.v[at[j] + threadIdx.x]), o);
            m = m1;
        }
        const float lse = l == 0.f ? -INFINITY : m + logf(l);   // NaN stays NaN
        if (threadIdx.x < D)
            a.out[b * a.os[0] + head * a.os[1] + threadIdx.x] = from_float<BF16>(l == 0.f ? 0.f : o / l);
        if (a.lse && threadIdx.x == 0) a.lse[b * (uint64_t)a.heads + head] = lse;
        if (!a.mass_out) continue;
        const uint32_t nm = min(n, a.mass_len);
        if (n > a.mass_len && g == 0 && h == 0 && threadIdx.x == 0) report(a.status, SPLITZIP_KV_BAD_LEN);
        // the weights are summed over the group first, then added to the mass
        float *w = a.weights + ((uint64_t)b * a.c.kv_heads + h) * min(a.mass_len, a.c.max_len);
        if (g == 0)
            for (uint32_t t = threadIdx.x; t < nm; t += kAttendThreads) w[t] = 0.f;
        __syncthreads();
        for (uint32_t i0 = 0; i0 < seen; i0 += kAttendThreads) {
            uint64_t v_at = ~0ull;
            const uint32_t i = i0 + threadIdx.x;
            const float x = logit(i, v_at);
            const uint32_t t = i < s ? i : first + (i - s);
            if (v_at != ~0ull && l != 0.f && t < nm) w[t] += expf(x - lse);
        }
        __syncthreads();
        if (g + 1 < a.group) continue;
        const float *mi = a.mass ? a.mass + b * a.ms[0] + h * a.ms[1] : nullptr;
        float *mo = a.mass_out + b * a.mos[0] + h * a.mos[1];
        for (uint32_t t = threadIdx.x; t < nm; t += kAttendThreads) mo[t] = (mi ? mi[t] : 0.f) + w[t];
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
constexpr int kSelCopies = 16;

// The masses as unsigned integers of the same order: -0 as 0, NaN above all.
__device__ inline uint32_t mass_key(float m) {
    if (m != m) return 0xffffffffu;
    const uint32_t u = __float_as_uint(m + 0.f);   // -0 + 0 = 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One workgroup per sequence and KV head: the threshold key by four
// passes over its bytes from the top (a histogram in LDS of the keys that
// agree so far), then every wave places what it keeps of a run of tokens of
// its own, in order.
__global__ __launch_bounds__(kSelThreads) void k_select(EvictArgs a) {
    __shared__ uint32_t hist[256 * kSelCopies];
    __shared__ uint32_t above_w[kSelWaves], equal_w[kSelWaves];
    __shared__ uint32_t s_prefix, s_need;
    const uint32_t b = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
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
        if (out)
            for (uint32_t t = tid; t < n; t += kSelThreads) out[t] = mass[t];
        return;
    }
    const uint32_t lo = a.sinks, hi = n - a.recent, take = a.budget - a.sinks - a.recent;
    uint32_t prefix = 0, need = take;
    if (take) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (uint32_t k = tid; k < 256 * kSelCopies; k += kSelThreads) hist[k] = 0;
            __syncthreads();
            const uint32_t seen = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            for (uint32_t t = lo + tid; t < hi; t += kSelThreads) {
                const uint32_t key = mass_key(mass[t]);
                if ((key & seen) == prefix)
                    atomicAdd(&hist[((key >> shift) & 255u) * kSelCopies + (lane & (kSelCopies - 1))], 1u);
            }
            __syncthreads();
            if (wave == 0) {
                // lane l holds bins 4l .. 4l+3; suffix sums over the lanes
                uint32_t bin[4], sum = 0;
                for (int k = 0; k < 4; ++k) {
                    bin[k] = 0;
                    for (int j = 0; j < kSelCopies; ++j) bin[k] += hist[(lane * 4 + k) * kSelCopies + j];
                    sum += bin[k];
                }
                uint32_t suf = sum;
                for (int d = 1; d < 64; d <<= 1) {
                    const uint32_t y = __shfl_down(suf, d);
                    if (lane + d < 64) suf += y;
                }
                uint32_t above = suf - sum;      // keys in higher lanes' bins
                for (int k = 3; k >= 0; --k) {
                    if (above < need && above + bin[k] >= need) {
                        s_prefix = prefix | ((lane * 4 + k) << shift);
                        s_need = need - above;
                    }
                    above += bin[k];
                }
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;
        }
    }
    // Of [lo, hi): keys above prefix stay, and the first `need` equal to it.
    const uint32_t span = (hi - lo + kSelWaves - 1) / kSelWaves;
    const uint32_t w0 = min(hi, lo + wave * span), w1 = min(hi, w0 + span);
    uint32_t above = 0, equal = 0;
    if (take)
        for (uint32_t t0 = w0; t0 < w1; t0 += 64) {
            const uint32_t t = t0 + lane;
            const uint32_t key = t < w1 ? mass_key(mass[t]) : 0u;
            above += __popcll(__ballot(t < w1 && key > prefix));
            equal += __popcll(__ballot(t < w1 && key == prefix));
        }
    if (lane == 0) {
        above_w[wave] = above;
        equal_w[wave] = equal;
    }
    __syncthreads();
    uint32_t at = a.sinks, eq = 0;
    for (uint32_t w = 0; w < wave; ++w) {
        at += above_w[w];
        eq += equal_w[w];
    }
    at += min(eq, need);
    // In place, a kept mass moves to a position that is not above its own, which
    // an earlier wave may not have read yet: the tokens are placed first,
    // then their masses copied in order.
    for (uint32_t t = tid; t < lo; t += kSelThreads) kept[t] = (int32_t)t;
    for (uint32_t t = tid; t < a.recent; t += kSelThreads) kept[a.budget - a.recent + t] = (int32_t)(hi + t);
    if (take)
        for (uint32_t t0 = w0; t0 < w1; t0 += 64) {
            const uint32_t t = t0 + lane;
            const uint32_t key = t < w1 ? mass_key(mass[t]) : 0u;
            const uint64_t below = (1ull << lane) - 1;
            const uint64_t gt = __ballot(t < w1 && key > prefix), same = __ballot(t < w1 && key == prefix);
            const uint32_t rank = eq + __popcll(same & below);
            const bool tie = (same >> lane & 1) && rank < need;
            const uint64_t keep = gt | __ballot(tie);
            if (keep >> lane & 1) kept[at + __popcll(keep & below)] = (int32_t)t;
            at += __popcll(keep);
            eq += __popcll(same);
        }
    if (!out) return;
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
constexpr int kMoveUnroll = 4;
constexpr uint32_t kMaxMoveParts = 65536;

// A workgroup moves a column of one pool: `chunk` 16-byte pieces of the rows
// of a sequence's KV head. Row i comes from row kept[i] >= i, so within a
// column, step by step upwards, a step's writes can only meet sources of the
// step itself: they wait until all its loads have arrived (the barrier), and
// steps need no other order. Columns share nothing.
__global__ __launch_bounds__(kMoveThreads) void k_move(EvictArgs a) {
    __shared__ uint64_t from[kMoveThreads * kMoveUnroll], dest[kMoveThreads * kMoveUnroll];
    const uint32_t b = blockIdx.z, tid = threadIdx.x;
    const uint32_t h = blockIdx.y / (2 * a.chunks), col = blockIdx.y % (2 * a.chunks);
    const bool is_v = col >= a.chunks;
    const uint32_t piece0 = (is_v ? col - a.chunks : col) * a.chunk;
    const uint32_t width = min(a.chunk, a.c.dim / 8 - piece0);
    const uint32_t n = min(min(seq_len(a.c, b), a.mass_len), a.budget);
    const uint16_t *src = (is_v ? a.c.v : a.c.k) + h * (is_v ? a.c.vs[1] : a.c.ks[1]) + piece0 * 8;
    uint16_t *dst = (is_v ? a.to.v : a.to.k) + h * (is_v ? a.to.vs[1] : a.to.ks[1]) + piece0 * 8;
    const int32_t *kept = a.kept + ((uint64_t)b * a.c.kv_heads + h) * a.budget;
    const uint32_t lane_rows = kMoveThreads / a.chunk, step = lane_rows * kMoveUnroll;
    const uint32_t row = tid / a.chunk, piece = tid % a.chunk;
    const uint64_t begin = (uint64_t)blockIdx.x * a.per_wg;
    const uint32_t end = (uint32_t)min((uint64_t)n, begin + a.per_wg);
    const bool same = a.to.k == a.c.k;
    constexpr uint64_t kNone = ~0ull;
    for (uint64_t i0 = begin; i0 < end; i0 += step) {
        for (uint32_t j = tid; j < step; j += kMoveThreads) {
            uint64_t f = kNone, d = kNone;
            if (i0 + j < end) {
                const uint32_t i = (uint32_t)(i0 + j), t = (uint32_t)kept[i];
                uint32_t p0, s0, p1, s1;
                if (locate(a.c, b, t, p0, s0) && locate(a.to, b, i, p1, s1)) {
                    if (!(same && t == i)) {
                        f = p0 * (is_v ? a.c.vs[0] : a.c.ks[0]) + s0 * (is_v ? a.c.vs[2] : a.c.ks[2]);
                        d = p1 * (is_v ? a.to.vs[0] : a.to.ks[0]) + s1 * (is_v ? a.to.vs[2] : a.to.ks[2]);
                    }
                } else {
                    report(a.status, SPLITZIP_KV_BAD_PAGE);
                }
            }
            from[j] = f;
            dest[j] = d;
        }
        __syncthreads();
        u32x4 x[kMoveUnroll];
        bool ok[kMoveUnroll];
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u) {
            const uint32_t j = u * lane_rows + row;
            ok[u] = row < lane_rows && piece < width && from[j] != kNone;
            if (ok[u]) x[u] = *(const u32x4 *)(src + from[j] + piece * 8);
        }
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kMoveUnroll; ++u)
            if (ok[u]) *(u32x4 *)(dst + dest[u * lane_rows + row] + piece * 8) = x[u];
        __syncthreads();
    }
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) a.to.lens[b] = (int32_t)n;
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

constexpr uint32_t kMaxGrid = 1u << 20;

inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline int launched() { return hipGetLastError() == hipSuccess ? SPLITZIP_OK : SPLITZIP_ERR_HIP; }

constexpr uint64_t kMaxOffset = 1ull << 40;      // elements

// count - 1 steps of `stride` stay below the limit (no overflow on the way)
inline bool spans(uint64_t stride, uint64_t count) {
    return count <= 1 || stride <= kMaxOffset / (count - 1);
}

bool shape_ok(const splitzip_kv_cache *c) {
    return c && c->head_dim >= 8 && c->head_dim <= SPLITZIP_KV_MAX_DIM && c->head_dim % 8 == 0 &&
           c->kv_heads >= 1 && c->kv_heads <= SPLITZIP_KV_MAX_KV_HEADS && c->page_size >= 1 &&
           c->page_size <= SPLITZIP_KV_MAX_PAGE && c->batch <= SPLITZIP_KV_MAX_BATCH &&
           (uint64_t)c->max_pages * c->page_size < (1ull << 31) &&
           (c->dtype == SPLITZIP_KV_BF16 || c->dtype == SPLITZIP_KV_FP16);
}

bool cache_ok(const splitzip_kv_cache *c) {
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
                             (c->batch == 1 || c->table_stride >= c->max_pages) && c->table_stride <= kMaxOffset / 65536);
}

Cache view(const splitzip_kv_cache *c) {
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
    // about 2048 pieces a workgroup, while that leaves 1024 workgroups
    uint32_t per = 2048 / a.items.d;
    if (per > r->rows / 1024) per = r->rows / 1024;
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

bool mass_strides_ok(const uint64_t s[2]) { return s[0] <= kMaxOffset / 65536 && s[1] <= kMaxOffset / 65536; }

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
    if (!shape_ok(cache) || heads == 0 || heads > SPLITZIP_KV_MAX_HEADS || heads % cache->kv_heads) return 0;
    const uint32_t all = cache->max_pages * cache->page_size;
    if (mass_len > all) mass_len = all;      // no sequence is longer
    const double logits = 4.0 * cache->batch * heads * mass_len;
    if (logits > 1e15) return 0;
    return 16 + 4ull * cache->batch * heads * mass_len;
}

int splitzip_kv_attend(const splitzip_kv_cache *cache, const splitzip_kv_query *query, void *d_ws,
                       size_t ws_bytes, int32_t *d_status, void *stream) {
    if (!cache_ok(cache) || !query || (d_status && !aligned(d_status, 4))) return SPLITZIP_ERR_INVALID;
    const splitzip_kv_query &Q = *query;
    const size_t need = splitzip_kv_attend_workspace_size(cache, Q.heads, Q.mass_out ? Q.mass_len : 0);
    if (!need || !(Q.scale - Q.scale == 0.f)) return SPLITZIP_ERR_INVALID;
    for (int i = 0; i < 2; ++i)
        if (Q.q_stride[i] % 8 || Q.out_stride[i] % 8 || Q.q_stride[i] > kMaxOffset / 65536 || Q.out_stride[i] > kMaxOffset / 65536)
            return SPLITZIP_ERR_INVALID;
    if (!mass_strides_ok(Q.mass_stride) || !mass_strides_ok(Q.mass_out_stride) || (Q.mass && !Q.mass_out) ||
        !aligned(Q.mass, 4) || !aligned(Q.mass_out, 4) || !aligned(Q.lse, 4))
        return SPLITZIP_ERR_INVALID;
    if (cache->batch == 0) return SPLITZIP_OK;
    if (!Q.q || !Q.out || !aligned(Q.q, 16) || !aligned(Q.out, 16) || !d_ws || !aligned(d_ws, 16))
        return SPLITZIP_ERR_INVALID;
    if (ws_bytes < need) return SPLITZIP_ERR_WORKSPACE;
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
    a.group = Q.heads / cache->kv_heads;
    a.window = Q.window;
    a.sinks = Q.sinks;
    a.scale = Q.scale;
    a.mass_len = Q.mass_len;
    a.weights = reinterpret_cast<float *>(d_ws);
    a.status = d_status;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const dim3 grid(cache->batch, cache->kv_heads);
    if (cache->dtype == SPLITZIP_KV_BF16) k_attend<true><<<grid, kAttendThreads, 0, s>>>(a);
    else k_attend<false><<<grid, kAttendThreads, 0, s>>>(a);
    return launched();
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
    a.chunk = pieces < 8 ? pieces : 8;
    a.chunks = (pieces + a.chunk - 1) / a.chunk;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    k_select<<<dim3(cache->batch, cache->kv_heads), kSelThreads, 0, s>>>(a);
    const int rc = launched();
    if (rc) return rc;
    const uint32_t most = (uint32_t)(all < B.budget ? all : B.budget);
    uint32_t parts = 1;
    a.per_wg = most ? most : 1;
    if (!share) {
        const uint32_t step = kMoveThreads / a.chunk * kMoveUnroll;
        const uint32_t steps = most ? (most - 1) / step + 1 : 1;
        a.per_wg = (steps - 1) / kMaxMoveParts + 1;
        parts = (steps - 1) / a.per_wg + 1;
        a.per_wg *= step;
    }
    k_move<<<dim3(parts, cache->kv_heads * 2 * a.chunks, cache->batch), kMoveThreads, 0, s>>>(a);
    return launched();
}

}  // extern "C"
