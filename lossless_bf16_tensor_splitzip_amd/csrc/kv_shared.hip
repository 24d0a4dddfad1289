// kv_shared.hip -- attention of one new token per sequence where the sequences
// of a group have their first tokens in common: HIP kernels and the C ABI of
// splitzip_kv_attend_shared.
//
//   k_shared       the tokens in common, for the query rows of a whole group
//   k_attend REST  (kv_attend.h) every sequence's other tokens
//   k_join_shared  the shares of both joined
//
// With x = scale q k over a part of the tokens, a share is m >= max x (in base
// 2), l = sum 2^(x - m) and o = sum 2^(x - m) v; shares join as
// M = max m, out = sum o 2^(m - M) / sum l 2^(m - M).

#include <type_traits>

#include "kv_attend.h"
#include "kv_cache.h"

namespace {

constexpr uint32_t kRows = 128;        // query rows a workgroup takes: 32 a wave
constexpr int kSharedThreads = 256;
constexpr uint32_t kSharedRuns = 512;

// Tokens a tile of K or V has, 16 KB of it or less.
constexpr int tile_tokens(int dp) { return dp <= 128 ? 64 : 32; }

struct SharedArgs {
    Cache c;
    const uint16_t *q;
    uint64_t qs[2];
    const int32_t *cu, *shared;
    uint32_t groups, heads, group;     // group: query heads of a KV head
    uint32_t members, parts;           // sequences a row tile has; row tiles a sequence's heads are cut into (one of them is 1)
    uint32_t rows;                     // rows of a full row tile
    float scale2;                      // |scale| log2(e)
    uint32_t negate;                   // 0x80008000 where the scale is negative
    uint32_t runs;
    Div by_runs, by_group;
    uint32_t *from;                    // [batch] tokens that were attended for the group
    uint32_t *notes;                   // [batch][kv_heads][parts][4]: see Note
    float *slot_o, *slot_ml;           // [runs][2] shares of [rows][dim] and [rows][2]
    float *whole_o, *whole_ml;         // [batch][heads] of [dim] and [2]: row tiles that were one run's
    int32_t *status;
};

// Where a sequence's rows of a KV head are: runs first .. first + n - 1 have
// shares of them, at `row` of the row tile, the first as its second share if it
// is late; with n = 1 they are in whole_o.
struct Note {
    uint32_t first, n2_late, row, reserved;
};

// A group's sequences, and how many tokens they have in common.
struct Group {
    uint32_t first, size, len;
};

__device__ inline Group group_of(const SharedArgs &a, uint32_t g, int32_t *status) {
    const int32_t c0 = a.cu[g], c1 = a.cu[g + 1], n = a.shared[g];
    if (c0 < 0 || c1 < c0 || c1 > (int32_t)a.c.batch) {
        report(status, SPLITZIP_KV_BAD_ROWS);
        return Group{0, 0, 0};
    }
    if (n < 0) report(status, SPLITZIP_KV_BAD_LEN);
    // one sequence alone has its tokens to itself
    if (n <= 0 || c1 - c0 < 2) return Group{(uint32_t)c0, (uint32_t)(c1 - c0), 0};
    return Group{(uint32_t)c0, (uint32_t)(c1 - c0), min((uint32_t)n, seq_len(a.c, c0))};
}

// The groups in blocks of 64, one a lane, and running sums of their units (of
// one KV head).
struct Block64Groups {
    uint32_t base;
    Group group;
    uint32_t units, tiles, before, upto, total;
};

template <int T>
__device__ inline void group_units(const SharedArgs &a, const Group &g, uint32_t &units, uint32_t &tiles) {
    units = g.len ? (g.len - 1) / T + 1 : 0;
    tiles = ((g.size + a.members - 1) / a.members) * a.parts;
}

template <int T>
__device__ inline void load_groups(const SharedArgs &a, uint32_t base, uint32_t carry, Block64Groups &k, int32_t *status) {
    const uint32_t g = base + (threadIdx.x & 63);
    k.base = base;
    k.group = g < a.groups ? group_of(a, g, status) : Group{0, 0, 0};
    group_units<T>(a, k.group, k.units, k.tiles);
    const uint32_t n = k.units * k.tiles, sum = wave_scan(n);
    k.before = carry + sum - n;
    k.upto = carry + sum;
    k.total = __builtin_amdgcn_readlane(k.upto, 63);
}

// The work -- all row tiles of all groups in tiles of T tokens, for every KV
// head -- is cut into equal runs, one a workgroup.  A workgroup's four waves
// have 32 query rows each and meet the same tokens, which are staged in LDS:
// the loads of a tile are under way while the one before is worked on.  Both
// products are the matrix cores' (see k_attend for the operands' layouts).
//
// The weights enter the second product as one 16-bit number each: with many
// rows the matrix cores bound this kernel, and a second number would cost half
// as much again.  The error, half a step of the type for each weight, is as
// large as that of rounding the output where V has no mean (1.4 times that
// error together), and smaller where it has.
template <bool BF16, int DP, bool EXACT>
__global__ __launch_bounds__(kSharedThreads, DP <= 192 ? 2 : 1) void k_shared(SharedArgs a) {
    constexpr int T = tile_tokens(DP);
    constexpr int KS = DP / 32;              // steps of the K product
    constexpr int P16 = DP / 128, P8 = (DP % 128) / 64, VC = DP / 16;      // as in k_attend
    constexpr int PR = DP / 8;               // 16-byte pieces of a row
    constexpr int NP = T * PR / kSharedThreads;      // pieces a thread stages of K, of V
    constexpr int ST = T / 16;
    // fp16 weights are held times 2^11, up to 2^4 above what the maximum of before
    // allows: no more than 2^15, and steps of 2^-35 of the largest or less.
    constexpr float kSlack = 4.f, kLift = BF16 ? 0.f : 11.f;
    auto at_least = [](float p) { return BF16 ? p : __builtin_amdgcn_fmed3f(p, p * 0x1p102f, 0x1p-24f); };
    // A row's pieces are stored in an order of its own, so that 16 lanes that
    // read one piece of 16 rows meet all banks.
    auto spot = [](uint32_t row, uint32_t piece) {
        return row * PR + (DP % 128 == 0 ? piece ^ (row & 15) : piece ^ (row >> 1 & 7));
    };
    __shared__ u32x4 s_k[2][T * PR], s_v[2][T * PR];
    __shared__ uint64_t off_k[4][T], off_v[4][T], s_valid[4];      // of tiles, in turn
    uint32_t *s_block = (uint32_t *)s_k;
    static_assert(sizeof s_k >= 4 * kMaxBlocks, "sums of all blocks");
    const uint32_t tid = threadIdx.x, lane = tid & 63, c16 = lane & 15, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t D = EXACT ? DP : a.c.dim, kvh = a.c.kv_heads;
    // This lane's places in a tile: where it puts its pieces, and what it reads
    // of the first 16 rows (further ones are a constant away).
    uint32_t put[NP], k_at[KS], v_at[4], v8_at[4];
#pragma unroll
    for (int k = 0; k < NP; ++k) put[k] = spot((tid + k * kSharedThreads) / PR, (tid + k * kSharedThreads) % PR);
#pragma unroll
    for (int j = 0; j < KS; ++j) k_at[j] = spot(c16, j * 4 + g);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v_at[i] = spot(g * 4 + i, c16);
        v8_at[i] = spot(g * 4 + i, P16 * 16 + (c16 >> 1)) * 2 + (c16 & 1);
    }

    if (blockIdx.x >= a.runs) {      // what every sequence has in common with its group
        const uint32_t b = (blockIdx.x - a.runs) * kSharedThreads + tid;
        if (b >= a.c.batch) return;
        uint32_t lo = 0, hi = a.groups;      // the last group that begins at b or before
        while (lo < hi) {
            const uint32_t mid = (lo + hi) >> 1;
            if (a.cu[mid] <= (int32_t)b) lo = mid + 1; else hi = mid;
        }
        uint32_t len = 0;
        if (lo) {
            const Group of = group_of(a, lo - 1, nullptr);
            if (b - of.first < of.size && seq_len(a.c, b) >= of.len) len = of.len;
        }
        a.from[b] = len;
        return;
    }

    // this workgroup's run
    Block64Groups blk{};
    uint32_t total = 0;
    int32_t *status0 = blockIdx.x == 0 ? a.status : nullptr;
    const uint32_t blocks = (a.groups + 63) / 64;
    if (blocks == 1) {
        load_groups<T>(a, 0, 0, blk, status0);
        total = blk.total;
    } else {
        for (uint32_t i = wave; i < blocks; i += kWaves) {
            Block64Groups one;
            load_groups<T>(a, i * 64, 0, one, status0);
            if (lane == 63) s_block[i] = one.total;
        }
        __syncthreads();
        for (uint32_t f = 0; f < blocks; f += 64)
            total += __builtin_amdgcn_readlane(wave_scan(f + lane < blocks ? s_block[f + lane] : 0), 63);
    }
    const Cut cut = cut_of(total * kvh, a.by_runs);
    if (blockIdx.x >= cut.runs) return;
    const uint32_t u_begin = cut.begin(blockIdx.x), u_end = cut.begin(blockIdx.x + 1);
    if (blocks > 1) {
        uint32_t first = 0, carry = 0;
        for (uint32_t f = 0; f < blocks; f += 64) {
            const uint32_t sum = f + lane < blocks ? s_block[f + lane] : 0, upto = carry + wave_scan(sum);
            const uint64_t past = __ballot(upto * kvh > u_begin);
            if (past) {
                const uint32_t i = (uint32_t)__builtin_ctzll(past);
                first = (f + i) * 64;
                carry = __builtin_amdgcn_readlane(upto - sum, i);
                break;
            }
            carry = __builtin_amdgcn_readlane(upto, 63);
        }
        load_groups<T>(a, first, carry, blk, nullptr);
    }

    for (uint32_t u = u_begin; u < u_end;) {
        uint64_t past;
        while (!(past = __ballot(blk.upto * kvh > u))) {
            if (blk.base + 64 >= a.groups) return;      // cu or lengths that change meanwhile
            load_groups<T>(a, blk.base + 64, blk.total, blk, nullptr);
        }
        const uint32_t at = (uint32_t)__builtin_ctzll(past);
        const uint32_t first = __builtin_amdgcn_readlane(blk.group.first, at), size = __builtin_amdgcn_readlane(blk.group.size, at),
                       len = __builtin_amdgcn_readlane(blk.group.len, at), units = __builtin_amdgcn_readlane(blk.units, at),
                       tiles = __builtin_amdgcn_readlane(blk.tiles, at), rel = u - __builtin_amdgcn_readlane(blk.before, at) * kvh;
        const uint32_t pair = rel / units, unit0 = rel - pair * units, count = min(units - unit0, u_end - u);
        const uint32_t h = pair / tiles, tile = pair - h * tiles;
        if (h >= kvh) return;
        const bool whole = count == units;
        const uint32_t member0 = tile / a.parts * a.members, part = tile % a.parts;
        const uint32_t members = min(a.members, size - member0);
        const uint32_t rows = a.parts == 1 ? members * a.group : min(a.rows, a.group - part * a.rows);
        const uint32_t end = min(len, (unit0 + count) * T);
        const int32_t *table = a.c.table + first * a.c.table_stride;
        // member and query head of a row
        auto locate_row = [&](uint32_t r, uint32_t &b, uint32_t &head) {
            const uint32_t i = part * a.rows + r, m = div(i, a.by_group);
            b = first + member0 + m;
            head = h * a.group + i - m * a.group;
        };

        u32x4 q[2][KS];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t r = wave * 32 + t * 16 + c16;
            uint32_t b = 0, head = 0;
            if (r < rows) locate_row(r, b, head);
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                const uint32_t d = j * 32 + g * 8;
                q[t][j] = u32x4{0, 0, 0, 0};
                if (r < rows && (EXACT || d < D)) q[t][j] = *(const u32x4 *)(a.q + b * a.qs[0] + head * a.qs[1] + d) ^ a.negate;
            }
        }
        f32x4 o[2][VC];
        float m[2], l[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            m[t] = -INFINITY;
            l[t] = 0.f;
#pragma unroll
            for (int j = 0; j < VC; ++j) o[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        // Staging: this thread's pieces of a tile.  A row's place is found by one
        // lane, two tiles ahead (the waves take turns), from a page number loaded
        // a tile before; the pieces' threads take it from LDS.
        const uint16_t *k_head = a.c.k + h * a.c.ks[1], *v_head = a.c.v + h * a.c.vs[1];
        u32x4 kx[NP], vx[NP];
        auto row_of = [&](int k) { return (tid + k * kSharedThreads) / PR; };
        auto piece_of = [&](int k) { return (tid + k * kSharedThreads) % PR; };
        const uint32_t tile0 = unit0, tile_end = (end - 1) / T + 1;
        auto page_at = [&](uint32_t n) {
            const uint32_t t = n * T + lane;
            return lane < T && t < end ? (uint32_t)table[div(t, a.c.page)] : 0xffffffffu;
        };
        auto place = [&](uint32_t n, uint32_t page) {
            const uint32_t t = n * T + lane;
            const bool in = lane < T && t < end, ok = in && page < a.c.num_pages;
            if (in && !ok) report(a.status, SPLITZIP_KV_BAD_PAGE);
            const uint32_t slot = t - div(t, a.c.page) * a.c.page.d;
            if (lane < T) {
                off_k[n & 3][lane] = ok ? page * a.c.ks[0] + slot * a.c.ks[2] : 0;
                off_v[n & 3][lane] = ok ? page * a.c.vs[0] + slot * a.c.vs[2] : 0;
            }
            const uint64_t mask = __ballot(ok);
            if (lane == 0) s_valid[n & 3] = mask;
        };
        auto valid_of = [&](uint32_t n) {
            const uint64_t x = s_valid[n & 3];
            return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(x >> 32)) << 32 |
                   (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)x);
        };
        auto fetch = [&](uint32_t n) {
            const uint64_t valid = valid_of(n);
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const uint32_t row = row_of(k), piece = piece_of(k);
                kx[k] = vx[k] = u32x4{0, 0, 0, 0};
                if (!(valid >> row & 1) || (!EXACT && piece * 8 >= D)) continue;
                kx[k] = *(const u32x4 *)(k_head + off_k[n & 3][row] + piece * 8);
                vx[k] = *(const u32x4 *)(v_head + off_v[n & 3][row] + piece * 8);
            }
        };

        __syncthreads();        // the piece of work before, and the sums of blocks, have been read
        const uint32_t turn = (wave - tile0) & 3;      // of the first four tiles this one is this wave's
        uint32_t page = page_at(tile0 + turn);
        if (turn < 2) {
            place(tile0 + turn, page);
            page = page_at(tile0 + turn + 4);
        }
        if (unit0 == 0 && tid < members) {
            const uint32_t shares = whole ? 1 : cut.owner(u + units - 1) - blockIdx.x + 1;
            ((u32x4 *)a.notes)[((uint64_t)(first + member0 + tid) * kvh + h) * a.parts + part] =
                u32x4{blockIdx.x, shares * 2 + (u != u_begin), tid * a.group, 0};
        }
        __syncthreads();
        fetch(tile0);
        for (uint32_t n = tile0; n < tile_end; ++n) {
            u32x4 *const now_k = s_k[n & 1], *const now_v = s_v[n & 1];
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                now_k[put[k]] = kx[k];
                now_v[put[k]] = vx[k];
            }
            if (((n + 2) & 3) == wave) {
                place(n + 2, page);
                page = page_at(n + 6);
            }
            __syncthreads();
            if (n + 1 < tile_end) fetch(n + 1);
            if (wave * 32 >= rows) continue;
            f32x4 x[2][ST];
#pragma unroll
            for (int s = 0; s < ST; ++s) {
                x[0][s] = x[1][s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    const u32x4 y = now_k[k_at[j] + s * 16 * PR];
                    x[0][s] = mfma<BF16>(y, q[0][j], x[0][s]);
                    x[1][s] = mfma<BF16>(y, q[1][j], x[1][s]);
                }
            }
            const uint64_t valid = valid_of(n);
            if (~valid << (64 - T)) {       // the last tile's end, or a page number outside the pool
                const uint64_t mine = valid >> (g * 4);
#pragma unroll
                for (int s = 0; s < ST; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!(mine >> (s * 16 + i) & 1)) x[0][s][i] = x[1][s][i] = -INFINITY;
            }
            u32x4 p[2][ST / 2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float top = -INFINITY;
#pragma unroll
                for (int s = 0; s < ST; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = fmaxf(top, x[t][s][i]);
                top = row_reduce<true>(top) * a.scale2 - kLift;
                // The sums are rescaled only where weights would pass 2^(kLift + kSlack):
                // rarely, after a run's first tiles.
                if (__any(top > m[t] + kSlack)) {
                    const float m_new = fmaxf(m[t], top), r = __builtin_amdgcn_exp2f(m[t] - (m_new == -INFINITY ? 0.f : m_new));
                    l[t] *= r;
#pragma unroll
                    for (int j = 0; j < VC; ++j) o[t][j] *= r;
                    m[t] = m_new;
                }
                const float use = m[t] == -INFINITY ? 0.f : m[t];
#pragma unroll
                for (int s = 0; s < ST; ++s)
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][s][i], a.scale2, -use));
                        const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][s][i + 1], a.scale2, -use));
                        l[t] += p0 + p1;
                        p[t][s >> 1][(s & 1) * 2 + i / 2] = pack2<BF16>(at_least(p0), at_least(p1));
                    }
            }
            // 32 tokens a time: the lane's 8 tokens' pieces, halves of words exchanged
#pragma unroll
            for (int s = 0; s < ST / 2; ++s) {
#pragma unroll
                for (int w0 = 0; w0 < P16; ++w0) {
                    u32x4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = now_v[v_at[i & 3] + (s * 32 + (i >> 2) * 16) * PR + w0 * 16];
#pragma unroll
                    for (int w = 0; w < 4; ++w)
#pragma unroll
                        for (int odd = 0; odd < 2; ++odd) {
                            u32x4 col;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                col[i] = __builtin_amdgcn_perm(v[2 * i + 1][w], v[2 * i][w], odd ? 0x07060302u : 0x05040100u);
                            o[0][w0 * 8 + 2 * w + odd] = mfma<BF16>(col, p[0][s], o[0][w0 * 8 + 2 * w + odd]);
                            o[1][w0 * 8 + 2 * w + odd] = mfma<BF16>(col, p[1][s], o[1][w0 * 8 + 2 * w + odd]);
                        }
                }
                if constexpr (P8 > 0) {
                    u32x2 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] = ((const u32x2 *)now_v)[v8_at[i & 3] + (s * 32 + (i >> 2) * 16) * PR * 2];
#pragma unroll
                    for (int w = 0; w < 2; ++w)
#pragma unroll
                        for (int odd = 0; odd < 2; ++odd) {
                            u32x4 col;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                col[i] = __builtin_amdgcn_perm(v[2 * i + 1][w], v[2 * i][w], odd ? 0x07060302u : 0x05040100u);
                            o[0][P16 * 8 + 2 * w + odd] = mfma<BF16>(col, p[0][s], o[0][P16 * 8 + 2 * w + odd]);
                            o[1][P16 * 8 + 2 * w + odd] = mfma<BF16>(col, p[1][s], o[1][P16 * 8 + 2 * w + odd]);
                        }
                }
            }
        }

        const uint32_t slot = blockIdx.x * 2 + (u != u_begin);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            l[t] = row_reduce<false>(l[t]);
            const uint32_t r = wave * 32 + t * 16 + c16;
            if (r >= rows) continue;
            uint32_t b, head;
            locate_row(r, b, head);
            const uint64_t row = whole ? b * (uint64_t)a.heads + head : (uint64_t)slot * a.rows + r;
            float *to = (whole ? a.whole_o : a.slot_o) + row * D;
            if (g == 0) *(f32x2 *)((whole ? a.whole_ml : a.slot_ml) + row * 2) = f32x2{m[t], l[t]};
#pragma unroll
            for (int w0 = 0; w0 < P16 + P8; ++w0) {
                const int wide = w0 < P16 ? 8 : 4;       // columns of a piece
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < wide; j += 4) {
                        f32x4 y;
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = o[t][w0 * 8 + j + e][i];
                        const uint32_t d = w0 * 128 + (g * 4 + i) * wide + j;
                        if (EXACT || d < D) *(f32x4 *)(to + d) = y;
                    }
            }
        }
        u += count;
    }
}

constexpr uint32_t kMaxShares = kSharedRuns + 1024;      // of a query head: runs of both kernels

struct JoinArgs {
    SharedArgs s;
    AttendArgs r;          // the rest
};

// One workgroup per query head of a sequence.
template <bool BF16>
__global__ __launch_bounds__(kJoinThreads) void k_join_shared(JoinArgs ja) {
    __shared__ float s_w[kJoinThreads / 64][kMaxShares];
    __shared__ f32x4 s_o[kJoinThreads];
    const SharedArgs &a = ja.s;
    const AttendArgs &r = ja.r;
    const uint32_t tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, b = blockIdx.y, head = blockIdx.x, dim = a.c.dim;
    const uint32_t h = head / a.group, in_group = head - h * a.group, part = in_group / a.rows;
    const uint64_t whole = b * (uint64_t)a.heads + head;
    uint32_t first = 0, n0 = 0, row = 0, late = 0;
    if (a.from[b]) {
        const u32x4 note = ((const u32x4 *)a.notes)[((uint64_t)b * a.c.kv_heads + h) * a.parts + part];
        // within the workspace also where arguments that changed meanwhile left it unwritten
        first = min(note[0], a.runs - 1), n0 = min(note[1] >> 1, a.runs - first), late = note[1] & 1;
        row = min(note[2] + in_group - part * a.rows, a.rows - 1);
    }
    uint32_t rest_first = 0, n1 = 1, rest_row = 0, rest_late = 0;
    if (r.runs) {
        const Shares sh(r, b, h, in_group);
        rest_first = sh.first, n1 = sh.n, rest_row = sh.row, rest_late = sh.late;
    }
    const uint32_t n = n0 + n1;
    // rows of a share, and whose array they are in
    auto place = [&](uint32_t j, const float *&o, const float *&ml) {
        uint64_t at = whole;
        if (j < n0) {
            if (n0 > 1) at = (uint64_t)((first + j) * 2 + (j == 0 ? late : 0)) * a.rows + row;
            o = n0 > 1 ? a.slot_o : a.whole_o;
            ml = n0 > 1 ? a.slot_ml : a.whole_ml;
        } else {
            j -= n0;
            if (n1 > 1) at = (uint64_t)((rest_first + j) * 2 + (j == 0 ? rest_late : 0)) * r.rows + rest_row;
            o = n1 > 1 ? r.share_o : r.whole_o;
            ml = n1 > 1 ? r.share_ml : r.whole_ml;
        }
        o += at * dim;
        ml += at * 2;
    };
    float top = -INFINITY, sum = 0.f;
    for (uint32_t j = lane; j < n; j += 64) {
        const float *o, *ml;
        place(j, o, ml);
        top = fmaxf(top, ml[0]);
    }
    top = wave_reduce<true>(top);
    for (uint32_t j = lane; j < n; j += 64) {
        const float *o, *ml;
        place(j, o, ml);
        // a share with m = -inf saw no finite logit: its sum is 0, or NaN, which stays
        const float w = ml[0] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml[0] - top);
        s_w[wave][j] = w;
        sum += ml[1] * w;
    }
    sum = wave_reduce<false>(sum);
    __builtin_amdgcn_wave_barrier();
    const uint32_t pieces = dim / 4, ways = kJoinThreads / pieces;
    const uint32_t way = tid / pieces, d = (tid - way * pieces) * 4;
    f32x4 y{0.f, 0.f, 0.f, 0.f};
    if (way < ways)
        for (uint32_t j = way; j < n; j += ways) {
            const float *o, *ml;
            place(j, o, ml);
            y += *(const f32x4 *)(o + d) * s_w[wave][j];
        }
    s_o[tid] = y;
    __syncthreads();
    if (tid < pieces) {
        for (uint32_t w = 1; w < ways; ++w) y += s_o[w * pieces + tid];
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        u32x2 z{pack2<BF16>(y[0] * inv, y[1] * inv), pack2<BF16>(y[2] * inv, y[3] * inv)};
        *(u32x2 *)(r.out + b * r.os[0] + head * r.os[1] + d) = z;
        if (tid == 0 && r.lse) r.lse[whole] = (sum == 0.f ? -INFINITY : top + log2f(sum)) * kLn2;
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

struct SharedPlan {
    AttendPlan rest;
    uint32_t members, parts, rows, runs;
    size_t from_at, notes_at, slot_at, slot_ml_at, whole_at, whole_ml_at, rest_whole_at, rest_whole_ml_at, rest_at, bytes;
};

bool shared_plan(const splitzip_kv_cache *c, uint32_t heads, uint32_t groups, SharedPlan &p) {
    if (groups > SPLITZIP_KV_MAX_BATCH || !attend_plan(c, heads, 0, p.rest)) return false;
    const uint32_t group = p.rest.group;
    p.members = group <= kRows ? kRows / group : 1;
    p.parts = (group - 1) / kRows + 1;
    p.rows = p.parts == 1 ? p.members * group : (group - 1) / p.parts + 1;
    const uint64_t all = (uint64_t)c->max_pages * c->page_size;
    const uint32_t tokens = tile_tokens((c->head_dim + 63) / 64 * 64);
    const uint64_t units = (all / tokens + 1) * c->batch * p.parts * c->kv_heads;
    if (units >> 31) return false;
    // a group has two sequences at least
    const uint64_t most = groups ? units : 0, runs = c->head_dim <= 192 ? kSharedRuns : kSharedRuns / 2;
    p.runs = (uint32_t)(most < runs ? most : runs);
    if (p.runs < 1) p.runs = 1;
    const size_t row = (size_t)c->head_dim * 4, per = (size_t)c->batch * heads, slots = (size_t)p.runs * 2 * p.rows;
    p.from_at = 0;
    p.notes_at = up16((size_t)c->batch * 4);
    p.slot_at = p.notes_at + (size_t)c->batch * c->kv_heads * p.parts * sizeof(Note);
    p.slot_ml_at = p.slot_at + slots * row;
    p.whole_at = up16(p.slot_ml_at + slots * 8);
    p.whole_ml_at = p.whole_at + per * row;
    p.rest_whole_at = up16(p.whole_ml_at + per * 8);
    p.rest_whole_ml_at = p.rest_whole_at + per * row;
    p.rest_at = up16(p.rest_whole_ml_at + per * 8);
    p.bytes = p.rest_at + p.rest.bytes;
    return true;
}

template <bool BF16>
void launch_shared(const SharedArgs &a, uint32_t grid, hipStream_t s) {
    auto go = [&](auto dp) {
        constexpr int DP = decltype(dp)::value;
        if (a.c.dim == DP) k_shared<BF16, DP, true><<<grid, kSharedThreads, 0, s>>>(a);
        else k_shared<BF16, DP, false><<<grid, kSharedThreads, 0, s>>>(a);
    };
    if (a.c.dim <= 64) go(std::integral_constant<int, 64>{});
    else if (a.c.dim <= 128) go(std::integral_constant<int, 128>{});
    else if (a.c.dim <= 192) go(std::integral_constant<int, 192>{});
    else go(std::integral_constant<int, 256>{});
}

}  // namespace

extern "C" {

size_t splitzip_kv_groups_struct_size(void) { return sizeof(splitzip_kv_groups); }

size_t splitzip_kv_shared_workspace_size(const splitzip_kv_cache *cache, uint32_t heads, uint32_t groups) {
    SharedPlan p;
    if (!shape_ok(cache) || !shared_plan(cache, heads, groups, p)) return 0;
    return p.bytes;
}

int splitzip_kv_attend_shared(const splitzip_kv_cache *cache, const splitzip_kv_query *query, const splitzip_kv_groups *groups,
                              void *d_ws, size_t ws_bytes, int32_t *d_status, void *stream) {
    if (!cache_ok(cache) || !query || !groups || (d_status && !aligned(d_status, 4))) return SPLITZIP_ERR_INVALID;
    const splitzip_kv_query &Q = *query;
    SharedPlan P;
    if (!shared_plan(cache, Q.heads, groups->groups, P) || !(Q.scale * kLog2e - Q.scale * kLog2e == 0.f)) return SPLITZIP_ERR_INVALID;
    for (int i = 0; i < 2; ++i)
        if (Q.q_stride[i] % 8 || Q.out_stride[i] % 8 || Q.q_stride[i] > kMaxOffset || Q.out_stride[i] > kMaxOffset)
            return SPLITZIP_ERR_INVALID;
    if (Q.mass || Q.mass_out || Q.window != SPLITZIP_KV_ALL || !aligned(Q.lse, 4)) return SPLITZIP_ERR_INVALID;
    if (groups->groups && (!groups->cu || !groups->shared || !aligned(groups->cu, 4) || !aligned(groups->shared, 4)))
        return SPLITZIP_ERR_INVALID;
    if (cache->batch == 0) return SPLITZIP_OK;
    if (!Q.q || !Q.out || !aligned(Q.q, 16) || !aligned(Q.out, 16) || !d_ws || !aligned(d_ws, 16)) return SPLITZIP_ERR_INVALID;
    if (ws_bytes < P.bytes) return SPLITZIP_ERR_WORKSPACE;
    uint8_t *ws = reinterpret_cast<uint8_t *>(d_ws);
    JoinArgs ja{};
    SharedArgs &a = ja.s;
    a.c = view(cache);
    a.q = Q.q;
    a.cu = groups->cu;
    a.shared = groups->shared;
    a.groups = groups->groups;
    a.heads = Q.heads;
    a.group = P.rest.group;
    a.members = P.members;
    a.parts = P.parts;
    a.rows = P.rows;
    // a scale of 0 makes no order of logits: every sequence on its own
    a.scale2 = (Q.scale < 0 ? -Q.scale : Q.scale) * kLog2e;
    if (a.scale2 == 0.f) a.groups = 0;
    a.negate = Q.scale < 0 ? 0x80008000u : 0;
    a.runs = P.runs;
    a.by_runs = make_div(P.runs);
    a.by_group = make_div(a.group);
    a.from = reinterpret_cast<uint32_t *>(ws + P.from_at);
    a.notes = reinterpret_cast<uint32_t *>(ws + P.notes_at);
    a.slot_o = reinterpret_cast<float *>(ws + P.slot_at);
    a.slot_ml = reinterpret_cast<float *>(ws + P.slot_ml_at);
    a.whole_o = reinterpret_cast<float *>(ws + P.whole_at);
    a.whole_ml = reinterpret_cast<float *>(ws + P.whole_ml_at);
    a.status = d_status;
    AttendArgs &r = ja.r;
    r.c = a.c;
    r.q = Q.q;
    r.out = Q.out;
    r.lse = Q.lse;
    for (int i = 0; i < 2; ++i) {
        a.qs[i] = r.qs[i] = Q.q_stride[i];
        r.os[i] = Q.out_stride[i];
    }
    r.heads = Q.heads;
    r.group = P.rest.group;
    r.row_tiles = P.rest.row_tiles;
    r.rows = P.rest.rows;
    r.window = SPLITZIP_KV_ALL;
    r.scale2 = Q.scale * kLog2e;
    r.status = d_status;
    r.from = a.from;
    uint8_t *rest = ws + P.rest_at;
    r.splits = reinterpret_cast<uint32_t *>(rest);
    r.share_o = reinterpret_cast<float *>(rest + P.rest.o_at);
    r.share_ml = reinterpret_cast<float *>(rest + P.rest.ml_at);
    r.whole_o = reinterpret_cast<float *>(ws + P.rest_whole_at);
    r.whole_ml = reinterpret_cast<float *>(ws + P.rest_whole_ml_at);
    const uint32_t grid = lay_out(r, P.rest, r.c.max_len);
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool bf16 = cache->dtype == SPLITZIP_KV_BF16;
    const uint32_t grid_shared = P.runs + (cache->batch - 1) / kSharedThreads + 1;
    if (bf16) launch_shared<true>(a, grid_shared, s);
    else launch_shared<false>(a, grid_shared, s);
    int rc = launched();
    if (rc) return rc;
    if (bf16) launch_attend<true, true>(r, P.rest.blocks, grid, s);
    else launch_attend<false, true>(r, P.rest.blocks, grid, s);
    rc = launched();
    if (rc) return rc;
    const dim3 joins(Q.heads, cache->batch);
    if (bf16) k_join_shared<true><<<joins, kJoinThreads, 0, s>>>(ja);
    else k_join_shared<false><<<joins, kJoinThreads, 0, s>>>(ja);
    return launched();
}

}  // extern "C"
