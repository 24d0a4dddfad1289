// kv_shared.hip -- attention of one new token per sequence where the sequences
// of a group have their first tokens in common: HIP kernels and the C ABI of
// splitzip_kv_attend_shared.
//
//   k_both    the tokens in common, for the query rows of a group, and every
//             sequence's other tokens, where query rows are few; or all tokens
//             of every sequence, where little would be read once instead
//   k_shared  the tokens in common where they are many (k_both then has the
//             other tokens alone)
//   k_join_shared  the shares of both joined
//
// With x = scale q k over a part of the tokens, a share is m (near max x, in
// base 2), l = sum 2^(x - m) and o = sum 2^(x - m) v; shares join as
// M = max m, out = sum o 2^(m - M) / sum l 2^(m - M).

#include <type_traits>

#include "kv_attend.h"
#include "kv_cache.h"

namespace {

constexpr int kSharedWaves = 4, kSharedThreads = 64 * kSharedWaves;
constexpr uint32_t kRows = 32 * kSharedWaves;      // query rows a workgroup of k_shared takes
constexpr uint32_t kSharedRuns = 512;  // of k_shared: as many as are resident (wide heads: half of that)
constexpr uint32_t kGroupsHere = 2048; // groups that k_both holds in LDS
// Tiles of a run, at least: one writes up to 128 rows of shares of every row
// tile that it has part of, which few tokens do not repay (8 KV heads of 128, 128
// query rows each, us with runs of at least 1, 2, 4 and 8 tiles: 1024 tokens 26,
// 25, 27 and 33, 4096 39, 33, 32 and 36, 12000 48, 49, 40 and 44).
constexpr uint32_t kLeast = 4;

// Tokens that k_shared's workgroups take at a time: 16 KB of K and of V, or less.
constexpr int tile_tokens(int dp) { return dp <= 128 ? 64 : 32; }

// How query rows are put together: sequences a row tile has, and row tiles a
// sequence's query heads of a KV head are cut into (one of the two is 1).
struct Tiling {
    uint32_t members, parts, rows;     // rows: of a full row tile
};

// Where the shares of a sequence's rows of a KV head lie, for the first row of
// the part: share 0 at row first, share j at row rest + j * 2 rows; whether the
// sequence has tokens in common with others (in the note of its other tokens).
struct Note {
    uint32_t first, rest, n, common;
};

struct SharedArgs {
    Cache c;
    const uint16_t *q;
    uint64_t qs[2];
    const int32_t *cu, *shared;
    uint32_t groups, heads, group;     // group: query heads of a KV head
    Tiling of, alone;                  // of groups, of sequences alone (members 1)
    float scale2;                      // scale * log2(e)
    uint32_t runs, most;               // runs 0: a workgroup for each sequence's KV head; most: units of groups that do not overlap, at most
    Div by_runs, by_group, by_pairs;
    uint16_t *out;                     // rows of the query heads and their lse
    uint64_t os[2];
    float *lse;
    uint32_t *from;                    // [batch] tokens that k_shared attended for the group; NULL: k_both attends them
    Note *of_notes, *alone_notes;      // [batch][kv_heads][of.parts], [alone.parts]
    float *o, *ml;                     // rows of [dim] and [2]: shares
    uint32_t slots, slot_rows;         // the launch's first row of [runs][2][slot_rows] for row tiles that several runs have
    uint32_t of_whole, alone_whole;    // first rows of [batch][heads]: row tiles that one run has
    int32_t *status;
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

template <int UNIT>
__device__ inline void scan_groups(const SharedArgs &a, uint32_t base, uint32_t carry, Group group, Block64Groups &k) {
    k.base = base;
    k.group = group;
    k.units = group.len ? (group.len - 1) / UNIT + 1 : 0;
    k.tiles = ((group.size + a.of.members - 1) / a.of.members) * a.of.parts;
    const uint32_t n = k.units * k.tiles, sum = wave_scan(n);
    k.before = carry + sum - n;
    k.upto = carry + sum;
    k.total = __builtin_amdgcn_readlane(k.upto, 63);
}

template <int UNIT>
__device__ inline void load_groups(const SharedArgs &a, uint32_t base, uint32_t carry, Block64Groups &k, int32_t *status) {
    const uint32_t g = base + (threadIdx.x & 63);
    scan_groups<UNIT>(a, base, carry, g < a.groups ? group_of(a, g, status) : Group{0, 0, 0}, k);
}

// One row tile's work on one KV head: some units of its tokens.
struct Piece {
    uint32_t first, len, from;       // the sequence whose table row is read, its tokens from .. len - 1
    uint32_t h, unit0, count, units; // KV head; units of those tokens here, and all of them
    uint32_t row0, rows;             // rows of the row tile: query heads row0 .. of the sequences from first on, in turn
    uint32_t part;
    uint32_t split, source;          // tokens before split are those of the table row of sequence source
};

// The piece of a group at unit u of the groups' work, from the block that
// has it; of no unit where ranges that overlap made the running sums wrap.
__device__ inline Piece group_piece(const SharedArgs &a, const Block64Groups &blk, uint32_t at, uint32_t u, uint32_t u_end) {
    auto lane_of = [&](uint32_t x) { return (uint32_t)__builtin_amdgcn_readlane(x, at); };
    const uint32_t size = lane_of(blk.group.size), tiles = lane_of(blk.tiles);
    Piece p{lane_of(blk.group.first), lane_of(blk.group.len), 0, 0, 0, 0, lane_of(blk.units), 0, 0, 0, 0, 0};
    if (!p.units || !tiles) return p;
    const uint32_t rel = u - lane_of(blk.before) * a.c.kv_heads, pair = rel / p.units;
    p.unit0 = rel - pair * p.units;
    p.count = min(p.units - p.unit0, u_end - u);
    p.h = pair / tiles;
    const uint32_t tile = pair - p.h * tiles, member0 = tile / a.of.parts * a.of.members;
    p.part = tile % a.of.parts;
    p.row0 = member0 * a.group + p.part * a.of.rows;
    p.rows = a.of.parts == 1 ? min(a.of.members, size - member0) * a.group : min(a.of.rows, a.group - p.part * a.of.rows);
    return p;
}

// Sequence and query head of a row.
__device__ inline void locate_row(const SharedArgs &a, const Piece &p, uint32_t row, uint32_t &b, uint32_t &head) {
    const uint32_t i = p.row0 + row, m = div(i, a.by_group);
    b = p.first + m;
    head = p.h * a.group + i - m * a.group;
}

// The run that begins a row tile tells the join where its shares will be.
__device__ inline void note_shares(const SharedArgs &a, const Piece &p, const Cut &cut, uint32_t u, bool late, bool of_group,
                                   bool common) {
    const uint32_t members = of_group && a.of.parts == 1 ? p.rows / a.group : 1;
    if (p.unit0 || threadIdx.x >= members) return;
    const uint32_t n = p.count == p.units ? 1 : cut.owner(u + p.units - 1) - blockIdx.x + 1;
    const uint32_t row = threadIdx.x * a.group;      // the member's first
    uint32_t b, head;
    locate_row(a, p, row, b, head);
    const uint32_t rest = a.slots + blockIdx.x * 2 * a.slot_rows + row;
    const uint32_t first = n > 1 ? rest + (late ? a.slot_rows : 0) : (of_group ? a.of_whole : a.alone_whole) + b * a.heads + head;
    const uint32_t parts = of_group ? a.of.parts : a.alone.parts;
    u32x4 *notes = (u32x4 *)(of_group ? a.of_notes : a.alone_notes);
    notes[((uint64_t)b * a.c.kv_heads + p.h) * parts + p.part] = u32x4{first, rest, n, common};
}

// The row of a share's arrays that a row of the piece has.
__device__ inline uint64_t share_row(const SharedArgs &a, const Piece &p, uint32_t row, bool late, bool of_group) {
    if (p.count != p.units) return a.slots + (uint64_t)(blockIdx.x * 2 + late) * a.slot_rows + row;
    uint32_t b, head;
    locate_row(a, p, row, b, head);
    return (of_group ? a.of_whole : a.alone_whole) + (uint64_t)b * a.heads + head;
}

// ---------------------------------------------------------------------------
// few query rows
// ---------------------------------------------------------------------------

struct Block64Rest {
    uint32_t base, len, from, first, units, before, upto, total;
};

template <bool BF16>
__device__ inline void write_head(const SharedArgs &a, uint32_t b, uint32_t head, uint32_t d, f32x4 o, float top, float sum) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    u32x2 z{pack2<BF16>(o[0] * inv, o[1] * inv), pack2<BF16>(o[2] * inv, o[3] * inv)};
    *(u32x2 *)(a.out + b * a.os[0] + head * a.os[1] + d) = z;
    if (d == 0 && a.lse) a.lse[b * (uint64_t)a.heads + head] = (sum == 0.f ? -INFINITY : top + log2f(sum)) * kLn2;
}

// Groups' tokens in common and sequences' other tokens in units of kUnit, all
// of them cut into equal runs.  Every workgroup looks all groups and lengths
// over to find its run; which of the groups a sequence belongs to is looked up
// in LDS.  APART: every sequence attends all of its tokens.  (4 beams of 546
// tokens 8.4 us, chains of loads; the other tokens of 64 sequences, 83 MB, 25
// us; 24 groups of up to 8192 tokens, 103 MB, 32: runs of many short pieces end
// 10 us after the average one.  In one launch with the tokens in common the
// beams take 12 us, in two 19.)
template <bool BF16, int DP, int NT, bool EXACT, bool APART>
__global__ __launch_bounds__(kAttendThreads) void k_both(SharedArgs a) {
    __shared__ AttendLds<DP, NT> lds;
    __shared__ uint32_t s_block[kMaxBlocks];
    __shared__ int32_t s_cu[kGroupsHere + 1];
    __shared__ uint32_t s_len[kGroupsHere];
    const uint32_t tid = threadIdx.x, lane = tid & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t D = EXACT ? DP : a.c.dim, kvh = a.c.kv_heads;
    int32_t *status0 = blockIdx.x == 0 ? a.status : nullptr;
    const bool unseen = APART && a.groups > kGroupsHere;      // more than are looked up: every sequence on its own
    const uint32_t groups = a.from || unseen ? 0 : a.groups;  // that are looked up here
    if (unseen && status0)
        for (uint32_t g = tid; g < a.groups; g += kAttendThreads) group_of(a, g, status0);

    Block64Groups gblk{};
    auto block_of_groups = [&](uint32_t base, uint32_t carry) {
        const uint32_t g = base + lane;
        Group x{0, 0, 0};
        if (g < groups) x = Group{(uint32_t)s_cu[g], (uint32_t)(s_cu[g + 1] - s_cu[g]), s_len[g]};
        scan_groups<kUnit>(a, base, carry, x, gblk);
    };
    uint32_t group_units = 0;
    if (groups) {
        for (uint32_t g = tid; g < groups; g += kAttendThreads) {
            const Group x = group_of(a, g, status0);
            s_cu[g] = a.cu[g];
            s_len[g] = x.len;
            if (g == groups - 1) s_cu[groups] = a.cu[groups];
        }
        __syncthreads();
        if (!APART) {
            for (uint32_t base = 0; base < groups; base += 64) {
                block_of_groups(base, group_units);
                group_units = gblk.total;
            }
            if (groups > 64) block_of_groups(0, 0);
        }
        group_units *= kvh;
        if (group_units > a.most) group_units = 0;      // ranges that overlap
    }

    Block64Rest blk{};
    auto block_of_rest = [&](uint32_t base, uint32_t carry, int32_t *status) {
        const uint32_t b = base + lane;
        blk.base = base;
        blk.len = b < a.c.batch ? seq_len(a.c, b, status) : 0;
        blk.from = blk.first = 0;
        if (a.from) {
            if (b < a.c.batch) blk.from = min(a.from[b], blk.len);
        } else {
            uint32_t lo = 0, hi = groups;        // the last group that begins at b or before
            while (lo < hi) {
                const uint32_t mid = (lo + hi) >> 1;
                if (s_cu[mid] <= (int32_t)b) lo = mid + 1; else hi = mid;
            }
            if (lo && (int32_t)b < s_cu[lo] && s_len[lo - 1] <= blk.len) {
                blk.from = s_len[lo - 1];
                blk.first = s_cu[lo - 1];
            }
        }
        const uint32_t from = APART ? 0 : blk.from;
        // an empty rest is one unit's work, so that every sequence has a share
        blk.units = b < a.c.batch ? (blk.len > from ? (blk.len - from - 1) / kUnit + 1 : 1) : 0;
        const uint32_t sum = wave_scan(blk.units);
        blk.before = carry + sum - blk.units;
        blk.upto = carry + sum;
        blk.total = __builtin_amdgcn_readlane(blk.upto, 63);
    };
    const uint32_t blocks = (a.c.batch + 63) / 64, pairs = kvh * a.alone.parts;
    const bool whole = APART && !a.runs;
    uint32_t rest_units = 0;
    auto piece_of_rest = [&](uint32_t at, uint32_t pair) {
        auto lane_of = [&](uint32_t x) { return (uint32_t)__builtin_amdgcn_readlane(x, at); };
        const uint32_t from = lane_of(blk.from);
        Piece p{blk.base + at, lane_of(blk.len), APART ? 0 : from, 0, 0, 0, lane_of(blk.units), 0, 0, 0, APART ? from : 0, lane_of(blk.first)};
        p.h = pair / a.alone.parts;
        p.part = pair - p.h * a.alone.parts;
        p.row0 = p.part * a.alone.rows;
        p.rows = min(a.alone.rows, a.group - p.row0);
        return p;
    };
    Cut cut{};
    uint32_t u_begin = 0, u_end = 1;
    bool found = blocks == 1;       // blk is the block of the rest that the run is in, or one before it
    if (!whole) {
        if (blocks == 1) {
            block_of_rest(0, 0, status0);
            rest_units = blk.total;
        } else {
            for (uint32_t i = wave; i < blocks; i += kWaves) {
                block_of_rest(i * 64, 0, status0);
                if (lane == 63) s_block[i] = blk.total;
            }
            __syncthreads();
            for (uint32_t f = 0; f < blocks; f += 64)
                rest_units += __builtin_amdgcn_readlane(wave_scan(f + lane < blocks ? s_block[f + lane] : 0), 63);
        }
        cut = cut_of(group_units + rest_units * pairs, a.by_runs);
        if (blockIdx.x >= cut.runs) return;
        u_begin = cut.begin(blockIdx.x);
        u_end = cut.begin(blockIdx.x + 1);
    }

    for (uint32_t u = u_begin; u < u_end;) {
        const bool of_group = u < group_units, late = u != u_begin;
        Piece p;
        uint64_t past;
        if (whole) {
            const uint32_t b = div(blockIdx.x, a.by_pairs), pair = blockIdx.x - b * pairs;
            block_of_rest(b & ~63u, 0, pair == 0 ? a.status : nullptr);
            p = piece_of_rest(b & 63, pair);
            p.count = p.units;
        } else if (of_group) {
            while (!(past = __ballot(gblk.upto * kvh > u))) {
                if (gblk.base + 64 >= groups) return;
                block_of_groups(gblk.base + 64, gblk.total);
            }
            p = group_piece(a, gblk, (uint32_t)__builtin_ctzll(past), u, u_end);
        } else {
            const uint32_t v = u - group_units;
            if (!found) {
                uint32_t first = 0, carry = 0;
                for (uint32_t f = 0; f < blocks; f += 64) {
                    const uint32_t sum = f + lane < blocks ? s_block[f + lane] : 0, upto = carry + wave_scan(sum);
                    if ((past = __ballot(upto * pairs > v))) {
                        const uint32_t i = (uint32_t)__builtin_ctzll(past);
                        first = (f + i) * 64;
                        carry = __builtin_amdgcn_readlane(upto - sum, i);
                        break;
                    }
                    carry = __builtin_amdgcn_readlane(upto, 63);
                }
                block_of_rest(first, carry, nullptr);
                found = true;
            }
            while (!(past = __ballot(blk.upto * pairs > v))) {
                if (blk.base + 64 >= a.c.batch) return;      // lengths that another stream changes meanwhile
                block_of_rest(blk.base + 64, blk.total, nullptr);
            }
            const uint32_t at = (uint32_t)__builtin_ctzll(past);
            const uint32_t rel = v - (uint32_t)__builtin_amdgcn_readlane(blk.before, at) * pairs;
            const uint32_t units = __builtin_amdgcn_readlane(blk.units, at), pair = rel / units;
            p = piece_of_rest(at, pair);
            p.unit0 = rel - pair * units;
            p.count = min(units - p.unit0, u_end - u);
        }
        if (!p.count || p.h >= kvh) return;
        const Seen seen{0, p.from, p.len - p.from};
        const int32_t *own = a.c.table + p.first * a.c.table_stride;
        const int32_t *common = APART ? a.c.table + p.source * a.c.table_stride : own;
        attend_tokens<BF16, DP, NT, EXACT>(
            lds, a.c, p.h, seen, p.unit0, min(seen.count, (p.unit0 + p.count) * kUnit), p.rows, a.scale2, a.status,
            [&](uint32_t t, uint32_t i) { return (APART && t < p.split ? common : own)[i]; },
            [&](uint32_t row) {
                uint32_t b, head;
                locate_row(a, p, row, b, head);
                return a.q + b * a.qs[0] + head * a.qs[1];
            },
            [&] {
                if (!whole) note_shares(a, p, cut, u, late, of_group, p.from != 0);
            },
            false, [](uint32_t, uint32_t, f32x4) {},
            [&](uint32_t row, uint32_t d, f32x4 y, float top, float sum) {
                if (whole) {
                    write_head<BF16>(a, p.first, p.h * a.group + p.row0 + row, d, y, top, sum);
                    return;
                }
                const uint64_t at = share_row(a, p, row, late, of_group);
                *(f32x4 *)(a.o + at * D + d) = y;
                if (d == 0) *(f32x2 *)(a.ml + at * 2) = f32x2{top, sum};
            });
        if (whole) return;
        u += p.count;
    }
}

// ---------------------------------------------------------------------------
// many query rows
// ---------------------------------------------------------------------------

// 16 or 4 bytes a lane from memory into LDS, the lanes' one after another from
// `to` on, without registers.  The compiler does not know of these: what waits
// for them is written out (until_loads), and the loop that has them under way
// has no other loads from memory.  (M0 holds the place in LDS, and is read one
// state after it is written; the compiler reserves it and keeps nothing in it.)
__device__ inline uint32_t lds_place(const void *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}
__device__ inline void load_to_lds16(const void *from, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(from) : "memory");
}
__device__ inline void load_to_lds4(const void *from, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(from) : "memory");
}
__device__ inline void until_loads() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0f70);      // vmcnt(0)
    asm volatile("" ::: "memory");
}

// Until all waves of the workgroup are here and their LDS stores have been
// made; loads from memory stay under way.
__device__ inline void meet() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The work -- all row tiles of all groups in tiles of T tokens, for every KV
// head -- is cut into equal runs, one a workgroup.  A workgroup's four waves
// have 32 query rows each and meet the same tokens, which are staged in LDS:
// the loads of a tile are under way while the one before is worked on.  Both
// products are the matrix cores' (see k_attend for the operands' layouts).
// (512 query rows a KV head, 8 heads of 128, 32768 tokens: 105 us, 650 TFLOP/s,
// of which the loads alone take 57 and the arithmetic alone 77.  Tiles through
// registers instead of straight into LDS took 120, 64 rows a wave 165.)
//
// The weights enter the second product as one 16-bit number each.  A second one
// is not hidden, though the matrix cores are busy for a quarter of the time only:
// a wave's loads, products and weights come one after another, and the two waves
// of a SIMD overlap little of them.  The whole call, us, with one number and with
// two (64 sequences behind 32768 tokens): bf16 131 and 153, fp16 137 and 167,
// heads of 64 82 and 99, 2 KV heads of 256 120 and 130.  The error of one, half a
// step of the type for each weight, is as large as that of rounding the output
// where V has no mean (1.4 times that error together), and smaller where it has:
// against 64 bits 0.00197 of the outputs' size, with two numbers 0.00165, what
// rounding the output alone leaves.
template <bool BF16, int DP, bool EXACT>
__global__ __launch_bounds__(kSharedThreads, DP <= 128 ? 2 : 1) void k_shared(SharedArgs a) {
    constexpr int NT = 2;                    // blocks of 16 query rows a wave has
    constexpr int T = tile_tokens(DP), ST = T / 16;
    constexpr int KS = DP / 32;              // steps of the K product
    constexpr int P16 = DP / 128, P8 = (DP % 128) / 64, VC = DP / 16;      // as in k_attend
    constexpr int PR = DP / 8;               // 16-byte pieces of a row
    constexpr int NP = T * PR / kSharedThreads;      // pieces a thread stages of K, of V
    // fp16 weights are held times 2^11, up to 2^4 above what the maximum of before
    // allows: no more than 2^15, and steps of 2^-35 of the largest or less.
    constexpr float kSlack = 4.f, kLift = BF16 ? 0.f : 11.f;
    auto at_least = [](float p) { return BF16 ? p : __builtin_amdgcn_fmed3f(p, p * 0x1p102f, 0x1p-24f); };
    // A row's pieces are stored in an order of its own, so that 16 lanes that
    // read one piece of 16 rows meet all banks.
    auto spot = [](uint32_t row, uint32_t piece) {
        return row * PR + (DP % 128 == 0 ? piece ^ (row & 15) : piece ^ (row >> 1 & 7));
    };
    __shared__ u32x4 s_k[2][T * PR], s_v[2][T * PR];      // two tiles, in turn
    __shared__ uint64_t off_k[4][T], off_v[4][T];         // of four tiles: rows' places, bytes
    __shared__ uint64_t s_valid[4];                       // which of their tokens are there
    __shared__ uint32_t s_page[4][64];                    // page numbers
    uint32_t *s_block = (uint32_t *)s_k;
    static_assert(sizeof s_k >= 4 * kMaxBlocks, "sums of all blocks");
    const uint32_t tid = threadIdx.x, lane = tid & 63, c16 = lane & 15, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t D = EXACT ? DP : a.c.dim, kvh = a.c.kv_heads;
    // Logits are compared before they are scaled: a negative scale is the queries'.
    const uint32_t negate = a.scale2 < 0.f ? 0x80008000u : 0;
    const float scale2 = fabsf(a.scale2);
    // This lane's places in a tile, of the first 16 rows (further ones are a
    // constant away).
    uint32_t k_at[KS], v_at[4], v8_at[4];
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
        for (uint32_t i = wave; i < blocks; i += kSharedWaves) {
            Block64Groups one;
            load_groups<T>(a, i * 64, 0, one, status0);
            if (lane == 63) s_block[i] = one.total;
        }
        __syncthreads();
        for (uint32_t f = 0; f < blocks; f += 64)
            total += __builtin_amdgcn_readlane(wave_scan(f + lane < blocks ? s_block[f + lane] : 0), 63);
    }
    const uint32_t units = total * kvh;
    if (units > a.most) return;      // ranges that overlap
    const Cut cut = units < kLeast * a.runs ? Cut{units, (units + kLeast - 1) / kLeast, kLeast, 0} : cut_of(units, a.by_runs);
    if (blockIdx.x >= cut.runs) return;
    const uint32_t u_begin = cut.begin(blockIdx.x), u_end = min(units, cut.begin(blockIdx.x + 1));
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

    if (!EXACT) {       // columns behind head_dim
        __syncthreads();
        for (uint32_t i = tid; i < 2 * T * PR; i += kSharedThreads) s_k[0][i] = s_v[0][i] = u32x4{0, 0, 0, 0};
    }

    for (uint32_t u = u_begin; u < u_end;) {
        uint64_t past;
        while (!(past = __ballot(blk.upto * kvh > u))) {
            if (blk.base + 64 >= a.groups) return;      // cu or lengths that change meanwhile
            load_groups<T>(a, blk.base + 64, blk.total, blk, nullptr);
        }
        const Piece p = group_piece(a, blk, (uint32_t)__builtin_ctzll(past), u, u_end);
        if (!p.count || p.h >= kvh) return;
        const bool late = u != u_begin;
        const uint32_t rows = p.rows, end = min(p.len, (p.unit0 + p.count) * T);
        const int32_t *table = a.c.table + p.first * a.c.table_stride;

        u32x4 q[NT][KS];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const uint32_t r = (wave * NT + t) * 16 + c16;
            uint32_t b = 0, head = 0;
            if (r < rows) locate_row(a, p, r, b, head);
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                const uint32_t d = j * 32 + g * 8;
                q[t][j] = u32x4{0, 0, 0, 0};
                if (r < rows && (EXACT || d < D)) q[t][j] = *(const u32x4 *)(a.q + b * a.qs[0] + head * a.qs[1] + d) ^ negate;
            }
        }
        f32x4 o[NT][VC];
        float m[NT], l[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t] = -INFINITY;
            l[t] = 0.f;
#pragma unroll
            for (int j = 0; j < VC; ++j) o[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        // Tile n's K and V are loaded a tile ahead.  A row's place is found by one
        // lane, three tiles ahead (the waves take turns), from a page number loaded
        // a tile before, and taken to the registers of the threads that load the
        // row's pieces a tile later.
        const uint8_t *k_head = (const uint8_t *)(a.c.k + p.h * a.c.ks[1]), *v_head = (const uint8_t *)(a.c.v + p.h * a.c.vs[1]);
        const uint32_t tile0 = p.unit0, tile_end = (end - 1) / T + 1;
        auto load_pages = [&](uint32_t n) {
            const uint32_t t = n * T + lane;
            const uint32_t to = lds_place(s_page[n & 3]);
            if (lane < T && t < end) load_to_lds4(table + div(t, a.c.page), to);
        };
        auto place = [&](uint32_t n) {
            const uint32_t t = n * T + lane, page = s_page[n & 3][lane];
            const bool in = lane < T && t < end, ok = in && page < a.c.num_pages;
            if (in && !ok) report(a.status, SPLITZIP_KV_BAD_PAGE);
            const uint32_t slot = t - div(t, a.c.page) * a.c.page.d;
            if (lane < T) {      // a token that is not there: the pool's first, stored over with zeros
                off_k[n & 3][lane] = ok ? 2 * (page * a.c.ks[0] + slot * a.c.ks[2]) : 0;
                off_v[n & 3][lane] = ok ? 2 * (page * a.c.vs[0] + slot * a.c.vs[2]) : 0;
            }
            const uint64_t mask = __ballot(ok);
            if (lane == 0) s_valid[n & 3] = mask;
        };
        auto missing_of = [&](uint32_t n) {      // its tokens that are not there
            const uint64_t x = ~s_valid[n & 3] << (64 - T) >> (64 - T);
            return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(x >> 32)) << 32 |
                   (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)x);
        };
        // Piece k of this thread: its place in the tile is tid + 256 k, and what belongs there.
        auto row_of = [&](int k) { return (tid + k * kSharedThreads) / PR; };
        auto piece_of = [&](int k) {
            const uint32_t row = row_of(k);
            return spot(row, (tid + k * kSharedThreads) % PR) - row * PR;
        };
        auto load_tile = [&](uint32_t n) {
            const uint32_t to_k = lds_place(s_k[n & 1]) + wave * 1024, to_v = lds_place(s_v[n & 1]) + wave * 1024;
            uint64_t from_k[NP], from_v[NP];      // all read before the first load, which nothing moves across
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                from_k[k] = off_k[n & 3][row_of(k)];
                from_v[k] = off_v[n & 3][row_of(k)];
            }
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const uint32_t piece = piece_of(k);
                if (!EXACT && piece * 8 >= D) continue;      // zeros since the start
                load_to_lds16(k_head + from_k[k] + piece * 16, to_k + k * kSharedThreads * 16);
                load_to_lds16(v_head + from_v[k] + piece * 16, to_v + k * kSharedThreads * 16);
            }
        };
        auto clear_rows = [&](uint32_t n, uint64_t missing) {
#pragma unroll
            for (int k = 0; k < NP; ++k)
                if (missing >> row_of(k) & 1) s_k[n & 1][tid + k * kSharedThreads] = s_v[n & 1][tid + k * kSharedThreads] = u32x4{0, 0, 0, 0};
        };
        const bool active = wave * (16 * NT) < rows;

        __syncthreads();        // the piece of work before, and the sums of blocks, have been read
        load_pages(tile0 + wave);
        note_shares(a, p, cut, u, late, true, true);
        until_loads();
        if (wave < 3) place(tile0 + wave);
        meet();
        uint64_t missing = missing_of(tile0);
        load_tile(tile0);
        for (uint32_t n = tile0; n < tile_end; ++n) {
            until_loads();
            if (missing) clear_rows(n, missing);
            meet();
            if (n + 1 < tile_end) load_tile(n + 1);
            if (((n - tile0) & (kSharedWaves - 1)) == wave && n + 3 < tile_end) place(n + 3);
            if (((n - tile0 + 1) & (kSharedWaves - 1)) == wave && n + 4 < tile_end) load_pages(n + 4);
            const uint64_t here = missing;
            if (active) {
                const u32x4 *const now_k = s_k[n & 1], *const now_v = s_v[n & 1];
                f32x4 x[NT][ST];
#pragma unroll
                for (int s = 0; s < ST; ++s) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) x[t][s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < KS; ++j) {
                        const u32x4 y = now_k[k_at[j] + s * 16 * PR];
#pragma unroll
                        for (int t = 0; t < NT; ++t) x[t][s] = mfma<BF16>(y, q[t][j], x[t][s]);
                    }
                }
                if (here) {       // the last tile's end, or a page number outside the pool
                    const uint64_t mine = here >> (g * 4);
#pragma unroll
                    for (int s = 0; s < ST; ++s)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (mine >> (s * 16 + i) & 1)
#pragma unroll
                                for (int t = 0; t < NT; ++t) x[t][s][i] = -INFINITY;
                }
                // The sums are rescaled only where weights would pass 2^(kLift + kSlack):
                // rarely, after a run's first tiles.
                float top[NT];
                bool far = false;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    top[t] = -INFINITY;
#pragma unroll
                    for (int s = 0; s < ST; ++s)
#pragma unroll
                        for (int i = 0; i < 4; ++i) top[t] = fmaxf(top[t], x[t][s][i]);
                    far = far || top[t] * scale2 > m[t] + (kLift + kSlack);
                }
                if (__any(far)) {
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const float m_new = fmaxf(m[t], row_reduce<true>(top[t]) * scale2 - kLift);
                        const float r = __builtin_amdgcn_exp2f(m[t] - (m_new == -INFINITY ? 0.f : m_new));
                        l[t] *= r;
#pragma unroll
                        for (int j = 0; j < VC; ++j) o[t][j] *= r;
                        m[t] = m_new;
                    }
                }
                u32x4 w[NT][ST / 2];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const float use = m[t] == -INFINITY ? 0.f : m[t];
#pragma unroll
                    for (int s = 0; s < ST; ++s)
#pragma unroll
                        for (int i = 0; i < 4; i += 2) {
                            const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][s][i], scale2, -use));
                            const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[t][s][i + 1], scale2, -use));
                            l[t] += p0 + p1;
                            w[t][s >> 1][(s & 1) * 2 + i / 2] = pack2<BF16>(at_least(p0), at_least(p1));
                        }
                }
                // 32 tokens a time: the lane's 8 tokens' pieces, halves of words exchanged
                auto add_columns = [&](int s, int c0, const auto &v, int words) {
#pragma unroll
                    for (int k = 0; k < words; ++k)
#pragma unroll
                        for (int odd = 0; odd < 2; ++odd) {
                            u32x4 col;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                col[i] = __builtin_amdgcn_perm(v[2 * i + 1][k], v[2 * i][k], odd ? 0x07060302u : 0x05040100u);
#pragma unroll
                            for (int t = 0; t < NT; ++t) o[t][c0 + 2 * k + odd] = mfma<BF16>(col, w[t][s], o[t][c0 + 2 * k + odd]);
                        }
                };
#pragma unroll
                for (int s = 0; s < ST / 2; ++s) {
#pragma unroll
                    for (int w0 = 0; w0 < P16; ++w0) {
                        u32x4 v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = now_v[v_at[i & 3] + (s * 32 + (i >> 2) * 16) * PR + w0 * 16];
                        add_columns(s, w0 * 8, v, 4);
                    }
                    if constexpr (P8 > 0) {
                        u32x2 v[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = ((const u32x2 *)now_v)[v8_at[i & 3] + (s * 32 + (i >> 2) * 16) * PR * 2];
                        add_columns(s, P16 * 8, v, 2);
                    }
                }
            }
            missing = missing_of(n + 1);
        }

#pragma unroll
        for (int t = 0; t < NT; ++t) {
            l[t] = row_reduce<false>(l[t]);
            const uint32_t r = (wave * NT + t) * 16 + c16;
            if (r >= rows) continue;
            const uint64_t row = share_row(a, p, r, late, true);
            float *to = a.o + row * D;
            if (g == 0) *(f32x2 *)(a.ml + row * 2) = f32x2{m[t], l[t]};
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
        u += p.count;
    }
}

// ---------------------------------------------------------------------------
// join
// ---------------------------------------------------------------------------

// Shares of a query head: of its group's tokens, from k_shared or k_both, and of
// its own, from k_both; a run has one of each at most.
constexpr uint32_t kMaxOwn = most_runs(), kMaxOf = kSharedRuns > kMaxOwn ? kSharedRuns : kMaxOwn;
constexpr uint32_t kJoinWaves = kJoinThreads / 64;
constexpr int kAhead = 12;                               // shares a thread loads before their weights are known

struct JoinArgs {
    SharedArgs s;
    uint32_t rows, of_step, alone_step;      // rows there are; rows from a share to the next
    uint32_t per;                            // query heads a workgroup has: kJoinWaves, or 1
};

// Where a query head's shares are: n0 of its group's tokens, the others of its own.
struct HeadShares {
    uint32_t n0, n, of_first, of_rest, of_step, alone_first, alone_rest, alone_step, last;

    __device__ HeadShares(const JoinArgs &j, uint32_t b, uint32_t head) {
        const SharedArgs &a = j.s;
        const uint32_t h = head / a.group, in_group = head - h * a.group;
        const uint32_t of_part = in_group / a.of.rows, alone_part = in_group / a.alone.rows;
        const uint64_t pair = (uint64_t)b * a.c.kv_heads + h;
        const u32x4 of = ((const u32x4 *)a.of_notes)[pair * a.of.parts + of_part];
        const u32x4 alone = ((const u32x4 *)a.alone_notes)[pair * a.alone.parts + alone_part];
        // (bounded, where arguments that changed meanwhile left notes unwritten)
        n0 = alone[3] ? min(of[2], kMaxOf) : 0;
        n = n0 + min(alone[2], kMaxOwn);
        const uint32_t of_row = in_group - of_part * a.of.rows, alone_row = in_group - alone_part * a.alone.rows;
        of_first = of[0] + of_row, of_rest = of[1] + of_row, of_step = j.of_step;
        alone_first = alone[0] + alone_row, alone_rest = alone[1] + alone_row, alone_step = j.alone_step;
        last = j.rows - 1;
    }
    __device__ uint64_t row(uint32_t i) const {
        const bool of = i < n0;
        const uint32_t k = of ? i : i - n0;
        return min(k ? (of ? of_rest + k * of_step : alone_rest + k * alone_step) : of ? of_first : alone_first, last);
    }
};

// The weights of n shares into w, and the joined sum, by a wave.
__device__ inline void weigh(const float *shares_ml, const HeadShares &sh, float *w, float &top, float &sum) {
    const uint32_t lane = threadIdx.x & 63;
    f32x2 ml{-INFINITY, 0.f};
    if (lane < sh.n) ml = *(const f32x2 *)(shares_ml + sh.row(lane) * 2);
    top = ml[0];
    for (uint32_t k = lane + 64; k < sh.n; k += 64) top = fmaxf(top, shares_ml[sh.row(k) * 2]);
    top = wave_reduce<true>(top);
    // a share with m = -inf saw no finite logit: its sum is 0, or NaN, which stays
    auto weight = [&](float m) { return m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top); };
    const float v = weight(ml[0]);
    sum = ml[1] * v;
    if (lane < sh.n) w[lane] = v;
    for (uint32_t k = lane + 64; k < sh.n; k += 64) {
        const f32x2 more = *(const f32x2 *)(shares_ml + sh.row(k) * 2);
        const float u = weight(more[0]);
        w[k] = u;
        sum += more[1] * u;
    }
    sum = wave_reduce<false>(sum);
}

// A wave per query head of a sequence: its shares, rescaled to their common
// maximum.  A chain of two loads: where they are; maxima, sums and outputs
// together.  Heads of more shares than a wave loads at once are all four waves',
// one after another; where heads are few a workgroup has one.  (96 x 32 heads
// of 64 columns with 2 to 4 shares 5.1 us, a workgroup each 9.6; 12 x 24 of 256
// with 13 and more, a workgroup each 5.2, four a workgroup 12.9.)
template <bool BF16>
__global__ __launch_bounds__(kJoinThreads) void k_join_shared(JoinArgs j) {
    __shared__ float s_w[kMaxOf + kMaxOwn];
    __shared__ f32x4 s_o[kJoinThreads];
    __shared__ float s_top, s_sum;
    __shared__ bool s_many[kJoinWaves];
    const SharedArgs &a = j.s;
    const uint32_t tid = threadIdx.x, lane = tid & 63, b = blockIdx.y, dim = a.c.dim;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t pieces = dim / 4;      // 4-column pieces of a row
    // shares summed side by side, and those that a thread loads before their weights are known
    auto load = [&](const HeadShares &sh, uint32_t t, uint32_t ways, f32x4 (&y)[kAhead]) {
        const uint32_t way = t / pieces, d = (t - way * pieces) * 4;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const uint32_t k = way + i * ways;
            y[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            if (way < ways && k < sh.n) y[i] = *(const f32x4 *)(a.o + sh.row(k) * dim + d);
        }
    };
    auto add = [&](const HeadShares &sh, uint32_t t, uint32_t ways, const f32x4 (&y)[kAhead], const float *w) {
        const uint32_t way = t / pieces, d = (t - way * pieces) * 4;
        f32x4 o{0.f, 0.f, 0.f, 0.f};
        if (way >= ways) return o;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (way + i * ways < sh.n) o += y[i] * w[way + i * ways];
        for (uint32_t k = way + kAhead * ways; k < sh.n; k += ways) o += *(const f32x4 *)(a.o + sh.row(k) * dim + d) * w[k];
        return o;
    };
    f32x4 y[kAhead];
    float top, sum;
    const uint32_t mine = blockIdx.x * kJoinWaves + wave, ways = 64 / pieces;
    bool many = j.per == 1 && wave == 0;
    if (j.per != 1 && mine < a.heads) {
        const HeadShares sh(j, b, mine);
        many = sh.n > min(ways * kAhead, 64u);
        if (!many) {
            float *w = s_w + wave * 64;
            load(sh, lane, ways, y);
            weigh(a.ml, sh, w, top, sum);
            __builtin_amdgcn_wave_barrier();
            f32x4 o = add(sh, lane, ways, y, w);
            s_o[tid] = o;
            __builtin_amdgcn_wave_barrier();
            if (lane < pieces) {
                for (uint32_t k = 1; k < ways; ++k) o += s_o[wave * 64 + k * pieces + lane];
                write_head<BF16>(a, b, mine, lane * 4, o, top, sum);
            }
        }
    }
    if (lane == 0) s_many[wave] = many;
    __syncthreads();
    for (uint32_t i = 0; i < kJoinWaves; ++i) {
        if (!s_many[i]) continue;
        const uint32_t head = blockIdx.x * j.per + i, all = kJoinThreads / pieces;
        const HeadShares sh(j, b, head);
        load(sh, tid, all, y);
        if (wave == 0) {
            weigh(a.ml, sh, s_w, top, sum);
            if (lane == 0) {
                s_top = top;
                s_sum = sum;
            }
        }
        __syncthreads();
        f32x4 o = add(sh, tid, all, y, s_w);
        s_o[tid] = o;
        __syncthreads();
        if (tid < pieces) {
            for (uint32_t k = 1; k < all; ++k) o += s_o[k * pieces + tid];
            write_head<BF16>(a, b, head, tid * 4, o, s_top, s_sum);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

struct SharedPlan {
    uint32_t group, blocks, both_runs, shared_runs;     // blocks of 16 rows in k_both; shared_runs 0: no k_shared
    bool apart, whole;                                  // k_both has all tokens of every sequence; by a workgroup for each KV head
    Tiling of, alone;
    uint32_t most;                                      // units of the groups' tokens, at most
    uint32_t of_whole, both_slots, alone_whole, rows, slot_rows;
    size_t from_at, of_notes_at, alone_notes_at, ml_at, o_at, bytes;
};

Tiling tiling(uint32_t group, uint32_t most) {
    Tiling t{};
    t.members = group <= most ? most / group : 1;
    t.parts = (group - 1) / most + 1;
    t.rows = t.parts == 1 ? t.members * group : (group - 1) / t.parts + 1;
    return t;
}

// many: with k_shared; most: query rows a workgroup of k_both takes.
bool lay_out(const splitzip_kv_cache *c, uint32_t heads, bool many, uint32_t most, SharedPlan &p) {
    const uint32_t group = heads / c->kv_heads, batch = c->batch;
    p.group = group;
    p.blocks = most / 16;
    p.alone = tiling(group, most);
    p.alone.members = 1;
    p.alone.rows = p.alone.parts == 1 ? group : p.alone.rows;
    p.of = tiling(group, many ? kRows : most);
    const uint64_t all = (uint64_t)c->max_pages * c->page_size;
    const uint64_t tiles = (uint64_t)batch * p.of.parts * c->kv_heads;      // of groups, at most
    const uint64_t units = (all / (many ? tile_tokens((int)c->head_dim) : kUnit) + 1) * tiles, shared = many ? units : 0;
    const uint64_t both = (all / kUnit + 1) * batch * p.alone.parts * c->kv_heads + (many ? 0 : units);
    if (both >> 31 || units >> 31) return false;
    p.most = (uint32_t)units;
    const uint32_t runs = runs_for(c->head_dim, p.blocks), more = c->head_dim <= 128 ? kSharedRuns : kSharedRuns / 2;
    p.both_runs = both < runs ? (uint32_t)both : runs;
    p.shared_runs = shared < more ? (uint32_t)shared : more;
    p.slot_rows = p.of.rows > p.alone.rows ? p.of.rows : p.alone.rows;
    if (many) p.slot_rows = p.alone.rows;
    const uint64_t per = (uint64_t)batch * heads, of_slots = (uint64_t)p.shared_runs * 2 * p.of.rows,
                   both_slots = (uint64_t)p.both_runs * 2 * p.slot_rows, rows = of_slots + both_slots + 2 * per;
    if (rows >> 31) return false;
    p.of_whole = (uint32_t)of_slots;
    p.both_slots = p.of_whole + (uint32_t)per;
    p.alone_whole = p.both_slots + (uint32_t)both_slots;
    p.rows = (uint32_t)rows;
    p.from_at = 0;
    p.of_notes_at = up16((size_t)batch * 4);
    p.alone_notes_at = p.of_notes_at + (size_t)batch * c->kv_heads * p.of.parts * sizeof(Note);
    p.ml_at = p.alone_notes_at + (size_t)batch * c->kv_heads * p.alone.parts * sizeof(Note);
    p.o_at = up16(p.ml_at + rows * 8);
    p.bytes = p.o_at + rows * c->head_dim * 4;
    if (p.bytes < 16) p.bytes = 16;
    return true;
}

bool shape_fits(const splitzip_kv_cache *c, uint32_t heads, uint32_t groups) {
    return groups <= SPLITZIP_KV_MAX_BATCH && heads && heads <= SPLITZIP_KV_MAX_HEADS && heads % c->kv_heads == 0;
}

// Which kernel has the tokens in common.  k_both reads them again for every 32
// query rows, k_shared for every 128, with another launch and larger shares.  By
// what k_both would read, with groups of average size and of all tokens that the
// table holds (sizes and lengths are on the device).  One group, us, k_both and
// k_shared: 8 KV heads of 128, 32 query rows a KV head, 4096 tokens (17 MB) 18
// and 25, 32768 (134 MB) 52 and 41; 64 rows, 4096 (34 MB) 25 and 28; 128 rows,
// 1024 (17 MB) 21 and 27, 4096 (67 MB) 36 and 32; 512 rows, 512 (34 MB) 50 and
// 48, 32768 (2.1 GB) 723 and 120.  2 KV heads of 256: 256 rows, 4096 (67 MB) 39
// and 45; 512 rows, 4096 (134 MB) 49 and 51; 1024 rows, 4096 (268 MB) 97 and 60;
// 64 rows, 32768 (134 MB) 51 and 54; 128 rows (268 MB) 85 and 62.
bool shared_plan(const splitzip_kv_cache *c, uint32_t heads, uint32_t groups, SharedPlan &p) {
    if (!shape_fits(c, heads, groups)) return false;
    const uint32_t group = heads / c->kv_heads;
    const uint64_t average = groups ? (uint64_t)c->batch * group / groups : 0;
    const double read = 4.0 * c->max_pages * c->page_size * c->kv_heads * c->head_dim * groups * (double)((average + 31) / 32);
    const bool many = groups > kGroupsHere || (average > 16 && read > (c->head_dim <= 128 ? 56e6 : 160e6));
    // Row tiles of k_both: of 16 rows for few rows, and for wide heads where that
    // leaves a tile two sequences (2 groups of 6, 4096 tokens, 2 KV heads of 256, us
    // with 16 and 32 rows: 8 query heads each 22.7 and 28.3, 12 each 33.3 and 28.1).
    // Where no tile has two sequences, each attends all of its tokens (2 groups of 6,
    // 5000 tokens, one KV head of 256 with 24 query heads 22.3 us, with the tokens in
    // common apart 26.5), and few units a KV head are one workgroup's, without a join
    // (4 groups of 8, 256 tokens in common of 512, 8 KV heads of 128: 15.0, 26.8).
    const uint64_t all = (uint64_t)c->max_pages * c->page_size;
    const bool whole = !many && whole_heads((uint64_t)c->batch * c->kv_heads * ((group - 1) / 32 + 1), all ? (uint32_t)((all - 1) / kUnit + 1) : 1);
    if (!lay_out(c, heads, many, group <= 16 && (many || whole || average <= 16 || (c->head_dim > 128 && group <= 8)) ? 16 : 32, p)) return false;
    p.whole = whole;
    p.apart = whole || (!many && p.of.members == 1);
    return true;
}

template <bool BF16>
void launch_both(const SharedArgs &a, uint32_t blocks, bool apart, hipStream_t s) {
    const uint32_t grid = a.runs ? a.runs : a.c.batch * a.c.kv_heads * a.alone.parts;
    auto go = [&](auto dp, auto nt) {
        constexpr int DP = decltype(dp)::value, NT = decltype(nt)::value;
        auto with = [&](auto exact, auto each) {
            k_both<BF16, DP, NT, decltype(exact)::value, decltype(each)::value><<<grid, kAttendThreads, 0, s>>>(a);
        };
        if (a.c.dim == DP) apart ? with(std::true_type{}, std::true_type{}) : with(std::true_type{}, std::false_type{});
        else apart ? with(std::false_type{}, std::true_type{}) : with(std::false_type{}, std::false_type{});
    };
    auto with = [&](auto dp) {
        if (blocks == 1) go(dp, std::integral_constant<int, 1>{});
        else go(dp, std::integral_constant<int, 2>{});
    };
    if (a.c.dim <= 64) with(std::integral_constant<int, 64>{});
    else if (a.c.dim <= 128) with(std::integral_constant<int, 128>{});
    else if (a.c.dim <= 192) with(std::integral_constant<int, 192>{});
    else with(std::integral_constant<int, 256>{});
}

template <bool BF16>
void launch_shared(const SharedArgs &a, hipStream_t s) {
    const uint32_t grid = a.runs + (a.c.batch - 1) / kSharedThreads + 1;
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
    if (!shape_ok(cache) || !shape_fits(cache, heads, groups)) return 0;
    size_t bytes = 0;
    for (int way = 0; way < 4; ++way) {      // a call with fewer groups goes another way
        SharedPlan p;
        if (!lay_out(cache, heads, way & 1, way & 2 ? 32 : 16, p)) return 0;
        if (p.bytes > bytes) bytes = p.bytes;
    }
    return bytes;
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
    SharedArgs a{};
    a.c = view(cache);
    a.q = Q.q;
    a.cu = groups->cu;
    a.shared = groups->shared;
    a.groups = groups->groups;
    a.heads = Q.heads;
    a.group = P.group;
    a.of = P.of;
    a.alone = P.alone;
    a.by_pairs = make_div(cache->kv_heads * P.alone.parts);
    a.out = Q.out;
    a.lse = Q.lse;
    a.scale2 = Q.scale * kLog2e;
    a.most = P.most;
    a.by_group = make_div(P.group);
    a.of_notes = reinterpret_cast<Note *>(ws + P.of_notes_at);
    a.alone_notes = reinterpret_cast<Note *>(ws + P.alone_notes_at);
    a.ml = reinterpret_cast<float *>(ws + P.ml_at);
    a.o = reinterpret_cast<float *>(ws + P.o_at);
    a.of_whole = P.of_whole;
    a.alone_whole = P.alone_whole;
    a.status = d_status;
    for (int i = 0; i < 2; ++i) {
        a.qs[i] = Q.q_stride[i];
        a.os[i] = Q.out_stride[i];
    }
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool bf16 = cache->dtype == SPLITZIP_KV_BF16;
    // a scale of 0 makes no order of logits, which k_shared goes by: every sequence on its own
    const bool many = P.shared_runs && a.groups && a.scale2 != 0.f;
    const bool apart = P.apart || (P.shared_runs && !many);
    if (many) {
        a.from = reinterpret_cast<uint32_t *>(ws + P.from_at);
        a.runs = P.shared_runs;
        a.by_runs = make_div(a.runs);
        a.slots = 0;
        a.slot_rows = P.of.rows;
        if (bf16) launch_shared<true>(a, s);
        else launch_shared<false>(a, s);
        const int rc = launched();
        if (rc) return rc;
    }
    a.runs = P.whole ? 0 : P.both_runs;
    a.by_runs = make_div(a.runs ? a.runs : 1);
    a.slots = P.both_slots;
    a.slot_rows = P.slot_rows;
    if (bf16) launch_both<true>(a, P.blocks, apart, s);
    else launch_both<false>(a, P.blocks, apart, s);
    const int rc = launched();
    if (rc || P.whole) return rc;
    JoinArgs j{a, P.rows, 2 * (many ? P.of.rows : P.slot_rows), 2 * P.slot_rows,
               (uint64_t)Q.heads * cache->batch >= 1024 ? kJoinWaves : 1};
    const dim3 joins((Q.heads - 1) / j.per + 1, cache->batch);
    if (bf16) k_join_shared<true><<<joins, kJoinThreads, 0, s>>>(j);
    else k_join_shared<false><<<joins, kJoinThreads, 0, s>>>(j);
    return launched();
}

}  // extern "C"
