// kv_attend.h -- attention of one new token per sequence over a paged cache:
//   k_attend  the work of all sequences cut into equal runs
//   k_join    joins the shares of KV heads that several runs had, and adds the
//             attention weights to the tokens' mass
// and how they are laid out.  Times are of one MI355X, a pass among others
// with inputs that change from pass to pass.
#ifndef SPLITZIP_CSRC_KV_ATTEND_H
#define SPLITZIP_CSRC_KV_ATTEND_H

#include "kv_cache.h"

namespace {

// ---------------------------------------------------------------------------
// attend
// ---------------------------------------------------------------------------
//
// Per KV head: logits x = scale q k for its group of query heads, weights
// p = exp(x - lse), out = sum p v, over the visible tokens, which are numbered
// 0, 1, ... (the sinks first, then the window).  Each K and V row is read
// once and meets at most a few dozen query rows, so memory bounds it: the
// matrix cores do both products, with the operands loaded from memory straight
// into their registers.
//
//   x^T = K q^T    mfma 16x16x32: 16 tokens by 16 query rows.  A lane loads
//                  8 elements of a K row (16 bytes); it receives 4 tokens'
//                  logits of one query row.
//   out^T = V^T p^T  32 tokens a time.  The lane's 8 weights (of two 16-token
//                  products) are the operand's 8 in the order it has them, so
//                  no weight moves between lanes; its V operand is those 8
//                  tokens' values of one column, which it gets from whole
//                  16-byte pieces of their rows by exchanging halves of words.
//
// The four waves of a workgroup take tiles in turn, each with a maximum, sum
// and output of its own, joined in LDS at the end: no barrier while tokens are
// read.  The next tile's K loads are issued as soon as the K product has read
// this one's, V's after the V product, so that each wave has 8 to 16 KB under
// way (dim 128).
//
// The work of a launch -- every sequence's tokens in units of kUnit, for every
// KV head -- is cut into equal runs, one a workgroup, whatever the lengths.  A
// run that begins or ends inside a KV head's tokens leaves its share (maximum,
// sum, unnormalised output) in the workspace, and k_join joins the shares.  (A
// join by the last workgroup to arrive, without a second launch, was slower:
// its stores, counter and loads pass the L2s of eight XCDs one after another,
// 32768 tokens of one sequence 37 us against 30.)
//
// 32 sequences of 32768 tokens, 8 KV heads of 128, 8 query heads each: 4.30 GB
// in 642 us, 6.7 TB/s, the rate of a bare read stream.  One sequence: 30 us, 26
// of them here and 4.5 in the join's launch.  48 sequences of 0 to 8192: 44 us.
// A run without any token takes 4 (dim 64) to 6.5 us (24 rows of dim 256).

constexpr int kWaves = 4;
constexpr int kAttendThreads = 64 * kWaves;
constexpr uint32_t kTile = 32;                  // tokens a wave takes at a time
constexpr uint32_t kUnit = kTile * kWaves;      // tokens a workgroup takes at a time
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct AttendArgs {
    Cache c;
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    uint64_t qs[2], os[2];
    uint32_t heads, group, window, sinks;
    uint32_t row_tiles, rows;     // row tiles a group is cut into, query rows a tile
    float scale2;                 // scale * log2(e): logits in base 2
    uint32_t runs;                // workgroups of k_attend; 0: one for every row tile of every KV head, nothing split
    Div by_runs, by_row_tiles, by_pairs;    // divisors: runs, row_tiles, kv_heads * row_tiles
    float *share_o, *share_ml;    // [runs][2] shares of [rows][dim] and [rows][2]
    uint32_t *splits;             // [batch][kv_heads][row_tiles][2]: see Shares
    float *logits;                // [batch][heads][logit_stride], by visible number (mass only)
    float *lse2;                  // [batch][heads] (mass only)
    uint64_t logit_stride;
    uint32_t logit_len;
    const float *mass;
    float *mass_out;
    uint64_t ms[2], mos[2];
    uint32_t mass_len;
    int32_t *status;
};

struct Seen {
    uint32_t sinks, shift, count;    // token of visible number v: v < sinks ? v : v + shift
};

__device__ inline Seen seen_of(uint32_t n, uint32_t window, uint32_t sinks) {
    const uint32_t first = window >= n ? 0 : n - window;
    const uint32_t s = min(sinks, first);
    return Seen{s, first - s, s + (n - first)};
}

__device__ inline uint32_t units_of(uint32_t n, uint32_t window, uint32_t sinks) {
    const uint32_t seen = seen_of(n, window, sinks).count;
    return seen ? (seen - 1) / kUnit + 1 : 1;    // an empty sequence's outputs are one unit's work
}

// The sequences in blocks of 64, one a lane: lengths and running sums of units.
struct Block64 {
    uint32_t first, len, before, upto;     // first sequence; the lane's length, units before and with it
    uint32_t total;                        // units with the block's last
};

__device__ inline void load_block(const AttendArgs &a, uint32_t first, uint32_t carry, Block64 &k,
                                  int32_t *status) {
    const uint32_t lane = threadIdx.x & 63, b = first + lane;
    k.first = first;
    k.len = b < a.c.batch ? seq_len(a.c, b, status) : 0;
    const uint32_t units = b < a.c.batch ? units_of(k.len, a.window, a.sinks) : 0;
    const uint32_t sum = wave_scan(units);
    k.before = carry + sum - units;
    k.upto = carry + sum;
    k.total = __builtin_amdgcn_readlane(k.upto, 63);
}

constexpr uint32_t kMaxBlocks = (SPLITZIP_KV_MAX_BATCH + 63) / 64;

// Units of a launch, and how they are cut into runs: the first `extra` runs
// have size + 1 of them, the others size.
struct Cut {
    uint32_t units, runs, size, extra;
    __device__ uint32_t begin(uint32_t run) const { return run * size + min(run, extra); }
    __device__ uint32_t owner(uint32_t u) const {
        const uint32_t big = extra * (size + 1);
        return u < big ? u / (size + 1) : extra + (u - big) / size;
    }
};

__device__ inline Cut cut_of(uint32_t units, Div runs) {
    if (units < runs.d) return Cut{units, units, 1, 0};
    const uint32_t size = div(units, runs);
    return Cut{units, runs.d, size, units - size * runs.d};
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

template <bool BF16>
__device__ inline f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <bool BF16>
__device__ inline uint32_t pack2(float x, float y) {
    if constexpr (BF16) return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x, (__bf16)y});
    else return __builtin_bit_cast(uint32_t, f16x2{(_Float16)x, (_Float16)y});
}

template <bool BF16>
__device__ inline void unpack2(uint32_t w, float &x, float &y) {
    if constexpr (BF16) {
        x = __uint_as_float(w << 16);
        y = __uint_as_float(w & 0xffff0000u);
    } else {
        const f16x2 h = __builtin_bit_cast(f16x2, w);
        x = (float)h[0];
        y = (float)h[1];
    }
}

typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Two values with infinities and NaN replaced by the largest finite number of
// their sign, as integers: positive ones compare as signed, negative ones are
// the upper half of the unsigned.
template <bool BF16>
__device__ inline uint32_t finite2(uint32_t w) {
    constexpr uint16_t top = BF16 ? 0x7f7f : 0x7bff;
    const i16x2 x = __builtin_elementwise_min(__builtin_bit_cast(i16x2, w), i16x2{(int16_t)top, (int16_t)top});
    constexpr uint16_t low = 0x8000 | top;
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(u16x2, x), u16x2{low, low}));
}

// Over the four lanes that hold a query row's tokens (16 apart).
template <bool MAX>
__device__ inline float row_reduce(float x) {
    const u32x2 a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    const float y0 = __uint_as_float(a[0]), y1 = __uint_as_float(a[1]);
    x = MAX ? fmaxf(y0, y1) : y0 + y1;
    const u32x2 b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    const float z0 = __uint_as_float(b[0]), z1 = __uint_as_float(b[1]);
    return MAX ? fmaxf(z0, z1) : z0 + z1;
}

// What attend_tokens keeps in LDS.  The query rows stay in registers, or here
// where those would spill.
template <int DP, int NT>
struct AttendLds {
    static constexpr bool kQueries = NT * (DP / 32) >= 12;
    static constexpr int LQ = DP + 8;
    __align__(16) uint16_t q[kQueries ? NT * 16 * LQ : 8];
    uint64_t off_k[kWaves][2][kTile], off_v[kWaves][2][kTile];
    __align__(16) float o[kWaves][16][DP + 4];
    float m[kWaves][NT * 16], l[kWaves][NT * 16], top[16], sum[16];
};

// A workgroup's work on one KV head's tokens for up to 16 NT query rows: the
// visible numbers from unit0 * kUnit to v_end of a table row.
//   page_at(t, i)                entry i of the row, of token t
//   query_at(row)                address of a query row
//   meanwhile()                  called while the first K and V are on their way
//   logits(row, v, x[4])         (keep_logits) logits in base 2 of four visible numbers from v on
//   emit(row, d, o[4], m, l)     four columns from d on of the sum of 2^(x - m) v, not divided by l
// DP: head_dim rounded up to a multiple of 64.  NT: blocks of 16 query rows.
// EXACT: head_dim is DP.
template <bool BF16, int DP, int NT, bool EXACT, typename PageAt, typename Query, typename Meanwhile, typename Logits, typename Emit>
__device__ __forceinline__ void attend_tokens(AttendLds<DP, NT> &lds, const Cache &c, uint32_t h, const Seen &seen, uint32_t unit0,
                                              uint32_t v_end, uint32_t rows, float scale2, int32_t *status, PageAt page_at,
                                              Query query_at, Meanwhile meanwhile, bool keep_logits, Logits logits, Emit emit) {
    constexpr int KS = DP / 32;             // steps of the K product
    constexpr int P16 = DP / 128;           // 16-byte pieces of a V row a lane takes: columns 128 i + 8 (lane % 16)
    constexpr int P8 = (DP % 128) / 64;     // and an 8-byte one: 128 P16 + 4 (lane % 16)
    constexpr int VW = 4 * P16 + 2 * P8;    // words of them
    constexpr int VC = 2 * VW;              // columns
    constexpr bool QLDS = AttendLds<DP, NT>::kQueries;
    constexpr int LQ = AttendLds<DP, NT>::LQ;
    // fp16 weights are held times 2^15: their smallest normal step then lies 2^-29
    // below the largest weight instead of 2^-14.
    constexpr float kLift = BF16 ? 0.f : 15.f;
    // The first part of a weight is 0 only where the weight is, so that an
    // infinity in V comes out as one: fp16 would round weights below 2^-40 of the
    // largest to 0, and 0 times infinity is a NaN.  The median of p, 2^102 p and
    // the type's smallest step is p, or that step, or 0; the second part then
    // takes the step away again.
    auto at_least = [](float p) { return BF16 ? p : __builtin_amdgcn_fmed3f(p, p * 0x1p102f, 0x1p-24f); };
    const uint32_t tid = threadIdx.x, lane = tid & 63, c16 = lane & 15, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t D = EXACT ? DP : c.dim;

    u32x4 q[QLDS ? 1 : NT][QLDS ? 1 : KS];
    constexpr int kStage = QLDS ? NT * 16 * (DP / 8) / kAttendThreads : 1;
    u32x4 stage[kStage];
    if constexpr (QLDS) {
#pragma unroll
        for (int k = 0; k < kStage; ++k) {
            const uint32_t i = tid + k * kAttendThreads, row = i / (DP / 8), d = i % (DP / 8) * 8;
            stage[k] = u32x4{0, 0, 0, 0};
            if (row < rows && (EXACT || d < D)) stage[k] = *(const u32x4 *)(query_at(row) + d);
        }
    } else {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                q[t][j] = u32x4{0, 0, 0, 0};
                const uint32_t d = j * 32 + g * 8;
                if (t * 16 + c16 < rows && (EXACT || d < D)) q[t][j] = *(const u32x4 *)(query_at(t * 16 + c16) + d);
            }
    }
    auto query = [&](int t, int j) {
        if constexpr (QLDS) return *(const u32x4 *)&lds.q[(t * 16 + c16) * LQ + j * 32 + g * 8];
        else return q[t][j];
    };
    f32x4 o[NT][VC];
    float m[NT], l[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        m[t] = -INFINITY;
        l[t] = 0.f;
#pragma unroll
        for (int j = 0; j < VC; ++j) o[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // Bases of this lane's pieces; columns behind head_dim (EXACT false)
    // are read from column 0 and stay unused.
    const uint16_t *k_lane[EXACT ? 1 : KS], *v_lane[P16 + P8];
    const uint16_t *k_head = c.k + h * c.ks[1], *v_head = c.v + h * c.vs[1];
#pragma unroll
    for (int j = 0; j < (EXACT ? 1 : KS); ++j) {
        const uint32_t d = j * 32 + g * 8;
        k_lane[j] = k_head + (EXACT || d < D ? d : 0);
    }
#pragma unroll
    for (int i = 0; i < P16 + P8; ++i) {
        const uint32_t d = i < P16 ? i * 128 + c16 * 8 : P16 * 128 + c16 * 4;
        v_lane[i] = v_head + (EXACT || d < D ? d : 0);
    }

    // The page number of lane t's token of the wave's tile at v0 (lanes
    // 32.. repeat 0..31), and from it the places of K and V.
    auto token = [&](uint32_t v) { return v < seen.sinks ? v : v + seen.shift; };
    auto page_of = [&](uint32_t v0) {
        const uint32_t v = v0 + (lane & 31), t = token(v);
        return v < v_end ? (uint32_t)page_at(t, div(t, c.page)) : 0xffffffffu;
    };
    auto place = [&](uint32_t v0, uint32_t page, int buf) {
        const uint32_t v = v0 + (lane & 31), t = token(v);
        const bool in = v < v_end, ok = in && page < c.num_pages;
        if (in && !ok) report(status, SPLITZIP_KV_BAD_PAGE);
        const uint32_t p = ok ? page : 0, slot = ok ? t - div(t, c.page) * c.page.d : 0;
        if (lane < 32) {
            lds.off_k[wave][buf][lane] = p * c.ks[0] + slot * c.ks[2];
            lds.off_v[wave][buf][lane] = p * c.vs[0] + slot * c.vs[2];
        }
        __builtin_amdgcn_wave_barrier();      // the wave's own LDS: in order without a wait
        return (uint32_t)__ballot(ok);
    };
    // Rows of whole cache lines pass the caches by (32 sequences of 32768 tokens
    // 642 us, through them 722); others share lines with their neighbours and
    // go through them (dim 80, 16 x 8192 tokens: 70 us, past them 88).
    auto load_kv = [](const uint16_t *p) { return EXACT ? load_once(p) : *(const u32x4 *)p; };
    auto load_kv8 = [](const uint16_t *p) {
        return EXACT ? __builtin_nontemporal_load((const u32x2 *)p) : *(const u32x2 *)p;
    };
    u32x4 kr[2][KS];
    u32x4 v16[8][P16 ? P16 : 1];
    u32x2 v8[8];
    auto word = [&](int i, int w) { return w < 4 * P16 ? v16[i][w / 4][w % 4] : v8[i][w - 4 * P16]; };
    auto load_k = [&](int buf) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint64_t off = lds.off_k[wave][buf][s * 16 + c16];
#pragma unroll
            for (int j = 0; j < KS; ++j)
                kr[s][j] = load_kv(EXACT ? k_lane[0] + off + j * 32 : k_lane[j] + off);
        }
    };
    auto load_v = [&](int buf) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t off = lds.off_v[wave][buf][(i >> 2) * 16 + g * 4 + (i & 3)];
#pragma unroll
            for (int p = 0; p < P16; ++p) v16[i][p] = load_kv(v_lane[p] + off);
            if constexpr (P8 > 0) v8[i] = load_kv8(v_lane[P16] + off);
        }
    };

    uint32_t v0 = unit0 * kUnit + wave * kTile;
    uint32_t page = 0xffffffffu, valid = 0, valid_next = 0;
    int buf = 0;
    if (v0 < v_end) {
        page = page_of(v0);
        valid = place(v0, page, 0);
        load_k(0);
        load_v(0);
        page = page_of(v0 + kUnit);
    }
    if constexpr (QLDS) {      // K and V are on their way; the row tile before has been read (its last barriers)
#pragma unroll
        for (int k = 0; k < kStage; ++k) {
            const uint32_t i = tid + k * kAttendThreads;
            *(u32x4 *)&lds.q[i / (DP / 8) * LQ + i % (DP / 8) * 8] = stage[k];
        }
        __syncthreads();
    }
    meanwhile();
    for (; v0 < v_end; v0 += kUnit) {
        const bool more = v0 + kUnit < v_end;
        if (more) {
            valid_next = place(v0 + kUnit, page, buf ^ 1);
            page = page_of(v0 + 2 * kUnit);
        }
        if (!EXACT) {
#pragma unroll
            for (int j = 0; j < KS; ++j)
                if (j * 32 + g * 8 >= D) kr[0][j] = kr[1][j] = u32x4{0, 0, 0, 0};
        }
        f32x4 x[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            x[t][0] = x[t][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                const u32x4 y = query(t, j);
                x[t][0] = mfma<BF16>(kr[0][j], y, x[t][0]);
                x[t][1] = mfma<BF16>(kr[1][j], y, x[t][1]);
            }
        }
        if (more) load_k(buf ^ 1);

        u32x4 hi[NT], lo[NT], rest[BF16 ? NT : 1];
        const uint32_t mine = (valid >> (g * 4) & 15u) | (valid >> (16 + g * 4) & 15u) << 4;     // of its 8 tokens
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float y[8], top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[i] = x[t][i >> 2][i & 3] * scale2;
                if (valid != 0xffffffffu && !(mine >> i & 1)) y[i] = -INFINITY;
                top = fmaxf(top, y[i]);
            }
            if (keep_logits && t * 16 + c16 < rows) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    logits(t * 16 + c16, v0 + s * 16 + g * 4, f32x4{y[4 * s], y[4 * s + 1], y[4 * s + 2], y[4 * s + 3]});
            }
            const float m_new = fmaxf(m[t], row_reduce<true>(top) - kLift);
            const float use = m_new == -INFINITY ? 0.f : m_new;
            if (__any(m_new > m[t])) {
                const float r = __builtin_amdgcn_exp2f(m[t] - use);
                l[t] *= r;
#pragma unroll
                for (int j = 0; j < VC; ++j) o[t][j] *= r;
                m[t] = m_new;
            }
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                // The weight as a sum of 16-bit numbers, as many as hold the
                // bits that 32 have: three of 8 in bf16, two of 11 in fp16.
                // One alone would add an error as large as the output's own
                // rounding, two in bf16 one of 2^-16, which moved 0.1 % of the
                // outputs by a step.  The further products are hidden behind
                // the loads (second 0 to 3 %, third 0 to 1; with 32 and 64
                // rows a KV head 62.3 us become 65.4 and 79.8 85.1).
                const float p0 = __builtin_amdgcn_exp2f(y[i] - use), p1 = __builtin_amdgcn_exp2f(y[i + 1] - use);
                l[t] += p0 + p1;
                float r0, r1;
                hi[t][i / 2] = pack2<BF16>(at_least(p0), at_least(p1));
                unpack2<BF16>(hi[t][i / 2], r0, r1);
                lo[t][i / 2] = pack2<BF16>(p0 - r0, p1 - r1);
                if constexpr (BF16) {
                    float s0, s1;
                    unpack2<BF16>(lo[t][i / 2], s0, s1);
                    rest[t][i / 2] = pack2<BF16>(p0 - r0 - s0, p1 - r1 - s1);
                }
            }
        }
        if (valid != 0xffffffffu) {
            // weight 0 does not silence an infinity or a NaN
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!(mine >> i & 1)) {
#pragma unroll
                    for (int p = 0; p < P16; ++p) v16[i][p] = u32x4{0, 0, 0, 0};
                    if constexpr (P8 > 0) v8[i] = u32x2{0, 0};
                }
        }
#pragma unroll
        for (int w = 0; w < VW; ++w)
#pragma unroll
            for (int odd = 0; odd < 2; ++odd) {
                // An infinity in V counts once, with the first part: times
                // another that is 0 or negative it would make a NaN.
                u32x4 col, fin;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    col[i] = __builtin_amdgcn_perm(word(2 * i + 1, w), word(2 * i, w), odd ? 0x07060302u : 0x05040100u);
                    fin[i] = finite2<BF16>(col[i]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    o[t][2 * w + odd] = mfma<BF16>(col, hi[t], o[t][2 * w + odd]);
                    o[t][2 * w + odd] = mfma<BF16>(fin, lo[t], o[t][2 * w + odd]);
                    if constexpr (BF16) o[t][2 * w + odd] = mfma<BF16>(fin, rest[t], o[t][2 * w + odd]);
                }
            }
        if (more) load_v(buf ^ 1);
        buf ^= 1;
        valid = valid_next;
    }

    // The waves' shares joined: common maximum, rescaled sums.
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        l[t] = row_reduce<false>(l[t]);
        if (lane < 16) {
            lds.m[wave][t * 16 + lane] = m[t];
            lds.l[wave][t * 16 + lane] = l[t];
        }
    }
    __syncthreads();
    for (int t = 0; t < NT && t * 16 < (int)rows; ++t) {
        // a lane's row c16: the waves' maximum and sum
        float M = -INFINITY, L = 0.f, mw[kWaves], lw[kWaves];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            mw[w] = lds.m[w][t * 16 + c16];
            lw[w] = lds.l[w][t * 16 + c16];
            M = fmaxf(M, mw[w]);
        }
#pragma unroll
        for (int w = 0; w < kWaves; ++w) L += mw[w] == -INFINITY ? lw[w] : lw[w] * __builtin_amdgcn_exp2f(mw[w] - M);
        if (tid < 16) {
            lds.top[tid] = M;
            lds.sum[tid] = L;
        }
        // o[t] is indexed by a constant: one of the NT blocks is taken
#pragma unroll
        for (int tt = 0; tt < NT; ++tt)
            if (tt == t) {
                const float r = m[tt] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[tt] - M);
#pragma unroll
                for (int p = 0; p < P16 + P8; ++p) {
                    const int wide = p < P16 ? 8 : 4;      // columns of the piece
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < wide; j += 4) {
                            const int at_col = p * 8 + j;
                            f32x4 y;
#pragma unroll
                            for (int e = 0; e < 4; ++e) y[e] = o[tt][at_col + e][i] * r;
                            *(f32x4 *)&lds.o[wave][c16][p * 128 + (g * 4 + i) * wide + j] = y;
                        }
                }
            }
        __syncthreads();
        constexpr int kItems = 16 * (DP / 4) / kAttendThreads;
        f32x4 y[kItems];
        float top[kItems], sum[kItems];
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const uint32_t item = tid + k * kAttendThreads, row = item / (DP / 4), d = item % (DP / 4) * 4;
            top[k] = lds.top[row];
            sum[k] = lds.sum[row];
            y[k] = *(const f32x4 *)&lds.o[0][row][d];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) y[k] += *(const f32x4 *)&lds.o[w][row][d];
        }
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const uint32_t item = tid + k * kAttendThreads, row = item / (DP / 4), d = item % (DP / 4) * 4;
            const uint32_t gr = t * 16 + row;
            if (gr >= rows || d >= D) continue;
            emit(gr, d, y[k], top[k], sum[k]);
        }
        __syncthreads();
    }
}

// (Bounded to 168 registers, for a third workgroup on a compute unit, dim 128
// spills: 30 us become 36.)
template <bool BF16, int DP, int NT, bool EXACT>
__global__ __launch_bounds__(kAttendThreads) void k_attend(AttendArgs a) {
    __shared__ AttendLds<DP, NT> lds;
    uint32_t *s_block = (uint32_t *)lds.o;      // while the run is looked up, before any output
    static_assert(sizeof lds.o >= 4 * kMaxBlocks, "sums of all blocks");
    const uint32_t tid = threadIdx.x, lane = tid & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t D = EXACT ? DP : a.c.dim;
    const uint32_t pairs = a.c.kv_heads * a.row_tiles;     // of a sequence

    // this workgroup's run of units
    Block64 blk{};
    Cut cut{};
    uint32_t at = 0, u_begin = 0, u_end = 1;
    if (a.runs) {
        int32_t *status0 = blockIdx.x == 0 ? a.status : nullptr;
        const uint32_t blocks = (a.c.batch + 63) / 64;
        uint32_t total = 0;
        if (blocks == 1) {
            load_block(a, 0, 0, blk, status0);
            total = blk.total;
        } else {
            // Every wave sums some blocks, then all of them look at the sums
            // (1024 sequences of 64 tokens in a table for 8192: 96 us, and 214
            // where every wave and every join read all of the lengths).
            for (uint32_t i = wave; i < blocks; i += kWaves) {
                const uint32_t b = i * 64 + lane;
                const uint32_t sum = wave_scan(b < a.c.batch ? units_of(seq_len(a.c, b, status0), a.window, a.sinks) : 0);
                if (lane == 63) s_block[i] = sum;
            }
            __syncthreads();
            for (uint32_t f = 0; f < blocks; f += 64)
                total += __builtin_amdgcn_readlane(wave_scan(f + lane < blocks ? s_block[f + lane] : 0), 63);
        }
        cut = cut_of(total * pairs, a.by_runs);
        if (blockIdx.x >= cut.runs) return;
        u_begin = cut.begin(blockIdx.x);
        u_end = cut.begin(blockIdx.x + 1);
        if (blocks > 1) {
            uint32_t first = 0, carry = 0;
            for (uint32_t f = 0;; f += 64) {
                const uint32_t sum = f + lane < blocks ? s_block[f + lane] : 0, upto = carry + wave_scan(sum);
                const uint64_t past = __ballot(upto * pairs > u_begin);
                if (past) {       // before the last block's end: u_begin < total * pairs
                    const uint32_t i = (uint32_t)__builtin_ctzll(past);
                    first = (f + i) * 64;
                    carry = __builtin_amdgcn_readlane(upto - sum, i);
                    break;
                }
                carry = __builtin_amdgcn_readlane(upto, 63);
            }
            load_block(a, first, carry, blk, nullptr);
        }
        const uint64_t past = __ballot(blk.upto * pairs > u_begin);
        at = past ? (uint32_t)__builtin_ctzll(past) : 64;      // the sequence's lane
    }

    for (uint32_t u = u_begin; u < u_end;) {
        uint32_t b, n, units, pair, unit0 = 0, count;
        if (a.runs) {
            while (at >= 64) {
                load_block(a, blk.first + 64, blk.total, blk, nullptr);
                at -= 64;
            }
            b = blk.first + at;
            n = __builtin_amdgcn_readlane(blk.len, at);
            const uint32_t before = __builtin_amdgcn_readlane(blk.before, at), rel = u - before * pairs;
            units = __builtin_amdgcn_readlane(blk.upto, at) - before;
            pair = rel / units;
            if (b >= a.c.batch || pair >= pairs) break;      // lengths that another stream changes meanwhile
            unit0 = rel - pair * units;
            count = min(units - unit0, u_end - u);
        } else {
            b = div(blockIdx.x, a.by_pairs);
            pair = blockIdx.x - b * pairs;
            n = __builtin_amdgcn_readfirstlane(seq_len(a.c, b, pair == 0 && wave == 0 ? a.status : nullptr));
            count = units = units_of(n, a.window, a.sinks);
        }
        const bool whole = count == units;
        const uint32_t h = div(pair, a.by_row_tiles), row0 = (pair - h * a.row_tiles) * a.rows;     // rows of the group
        const uint32_t rows = min(a.rows, a.group - row0), head0 = h * a.group + row0;
        const Seen seen = seen_of(n, a.window, a.sinks);
        const uint32_t v_end = min(seen.count, (unit0 + count) * kUnit);
        const int32_t *table = a.c.table + b * a.c.table_stride;

        const uint32_t slot = blockIdx.x * 2 + (u != u_begin);
        attend_tokens<BF16, DP, NT, EXACT>(
            lds, a.c, h, seen, unit0, v_end, rows, a.scale2, a.status, [&](uint32_t, uint32_t i) { return table[i]; },
            [&](uint32_t row) { return a.q + b * a.qs[0] + (head0 + row) * a.qs[1]; },
            [&] {
                if (a.runs && unit0 == 0 && tid == 0) {      // here its divisions are waited for by nothing
                    const uint32_t shares = whole ? 1 : cut.owner(u + units - 1) - blockIdx.x + 1;
                    ((u32x2 *)a.splits)[(uint64_t)b * pairs + pair] = u32x2{blockIdx.x, shares * 2 + (u != u_begin)};
                }
            },
            a.logits != nullptr,
            [&](uint32_t row, uint32_t v, f32x4 x) {
                float *to = a.logits + (b * (uint64_t)a.heads + head0 + row) * a.logit_stride;
                if (v < a.logit_len) *(f32x4 *)(to + v) = x;
            },
            [&](uint32_t row, uint32_t d, f32x4 y, float top, float sum) {
                if (whole) {
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    u32x2 z{pack2<BF16>(y[0] * inv, y[1] * inv), pack2<BF16>(y[2] * inv, y[3] * inv)};
                    *(u32x2 *)(a.out + b * a.os[0] + (head0 + row) * a.os[1] + d) = z;
                    if (d == 0) {
                        const float e = sum == 0.f ? -INFINITY : top + log2f(sum);
                        if (a.lse) a.lse[b * (uint64_t)a.heads + head0 + row] = e * kLn2;
                        if (a.lse2) a.lse2[b * (uint64_t)a.heads + head0 + row] = e;
                    }
                } else {
                    *(f32x4 *)(a.share_o + ((uint64_t)slot * a.rows + row) * D + d) = y;
                    if (d == 0) *(f32x2 *)(a.share_ml + ((uint64_t)slot * a.rows + row) * 2) = f32x2{top, sum};
                }
            });
        u += a.runs ? count : 1;
        if (pair == pairs - 1 && unit0 + count == units) ++at;
    }
}

// Over all lanes of the wave.
template <bool MAX>
__device__ inline float wave_reduce(float x) {
    auto with = [](float x, float y) { return MAX ? fmaxf(x, y) : x + y; };
    x = with(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x128, 0xf, 0xf, false)));    // row_ror:8
    x = with(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x124, 0xf, 0xf, false)));    // row_ror:4
    x = with(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x122, 0xf, 0xf, false)));    // row_ror:2
    x = with(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x121, 0xf, 0xf, false)));    // row_ror:1
    return row_reduce<MAX>(x);
}

constexpr int kJoinThreads = 256;
constexpr int kJoinAhead = 12;      // shares a thread loads before their weights are known
constexpr uint32_t kMaxRuns = 1024;

// A query head's shares: runs first .. first + n - 1 have them, at its row in
// the row tile, the first as its second share if it is late.  The run that
// began the row tile left first and n * 2 + late in splits.
struct Shares {
    uint32_t first, n, row, late;

    __device__ Shares(const AttendArgs &a, uint32_t b, uint32_t h, uint32_t in_group) {
        const uint32_t tile = in_group / a.rows;
        const u32x2 x = ((const u32x2 *)a.splits)[((uint64_t)b * a.c.kv_heads + h) * a.row_tiles + tile];
        // within the workspace also where lengths that changed meanwhile left it unwritten
        first = min(x[0], a.runs - 1), n = min(x[1] >> 1, a.runs - first), late = x[1] & 1, row = in_group - tile * a.rows;
    }
    __device__ uint64_t at(const AttendArgs &a, uint32_t j) const {
        return (uint64_t)((first + j) * 2 + (j == 0 ? late : 0)) * a.rows + row;
    }
};

// Largest share's maximum and the joined sum of the head looked up, over the
// lanes of a wave; keep(j, weight) for every share.
template <typename F>
__device__ inline void weigh(const AttendArgs &a, const Shares &sh, float &top, float &sum, F keep) {
    const uint32_t lane = threadIdx.x & 63;
    // a share with m = -inf saw no finite logit: its sum is 0, or NaN, which stays
    auto weight = [&](float m) { return m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top); };
    f32x2 ml{-INFINITY, 0.f};
    if (lane < sh.n) ml = *(const f32x2 *)(a.share_ml + sh.at(a, lane) * 2);
    top = ml[0];
    for (uint32_t j = lane + 64; j < sh.n; j += 64) top = fmaxf(top, a.share_ml[sh.at(a, j) * 2]);
    top = wave_reduce<true>(top);
    const float w = weight(ml[0]);
    if (lane < sh.n) keep(lane, w);
    sum = ml[1] * w;
    for (uint32_t j = lane + 64; j < sh.n; j += 64) {
        const f32x2 more = *(const f32x2 *)(a.share_ml + sh.at(a, j) * 2);
        const float v = weight(more[0]);
        keep(j, v);
        sum += more[1] * v;
    }
    sum = wave_reduce<false>(sum);
}

constexpr int kMassAhead = 4;                                   // tokens a thread, and query rows loaded ahead
constexpr uint32_t kMassTokens = kMassAhead * kJoinThreads;     // a workgroup
constexpr uint32_t kMassRows = 64;                              // query rows it takes at a time

// mass_out = mass + the group's weights, for one KV head's tokens from `part`
// on.  Each workgroup works the rows' lse out for itself from their shares (or
// takes them where one run had all).
__device__ inline void add_mass(const AttendArgs &a, uint32_t b, uint32_t h, uint32_t part) {
    __shared__ float s_lse[kMassRows];
    const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t n = seq_len(a.c, b);
    const Seen seen = seen_of(n, a.window, a.sinks);
    if (n > a.mass_len) {
        if (part == 0 && h == 0 && tid == 0) report(a.status, SPLITZIP_KV_BAD_LEN);
        n = a.mass_len;
    }
    const uint32_t t0 = part * kMassTokens + tid;
    if (part * kMassTokens >= n) return;
    const float *x = a.logits + (b * (uint64_t)a.heads + h * a.group) * a.logit_stride;
    const float *in = a.mass ? a.mass + b * a.ms[0] + h * a.ms[1] : nullptr;
    float *out = a.mass_out + b * a.mos[0] + h * a.mos[1];
    // the masses and the first rows' logits are under way while the lse are found
    float w[kMassAhead], old[kMassAhead], ahead[kMassAhead][kMassAhead];
    uint32_t v[kMassAhead];
#pragma unroll
    for (int k = 0; k < kMassAhead; ++k) {
        const uint32_t t = t0 + k * kJoinThreads;
        const bool hidden = t >= n || (t >= seen.sinks && t - seen.sinks < seen.shift);
        v[k] = hidden ? 0xffffffffu : t < seen.sinks ? t : t - seen.shift;
        w[k] = 0.f;
        old[k] = in && t < n ? in[t] : 0.f;
#pragma unroll
        for (int r = 0; r < kMassAhead; ++r)
            ahead[k][r] = hidden || r >= (int)a.group ? -INFINITY : x[r * a.logit_stride + v[k]];
    }
    for (uint32_t r0 = 0; r0 < a.group; r0 += kMassRows) {
        const uint32_t rows = min(kMassRows, a.group - r0);
        __syncthreads();
        for (uint32_t r = wave; r < rows; r += kJoinThreads / 64) {
            const uint32_t head = h * a.group + r0 + r;
            float e;
            if (!a.runs) {
                e = a.lse2[b * (uint64_t)a.heads + head];
            } else if (const Shares sh(a, b, h, r0 + r); sh.n == 1) {
                e = a.lse2[b * (uint64_t)a.heads + head];
            } else {
                float top, sum;
                weigh(a, sh, top, sum, [](uint32_t, float) {});
                e = sum == 0.f ? -INFINITY : top + log2f(sum);
            }
            // where nothing weighs, no logit does
            if (lane == 0) s_lse[r] = e == -INFINITY ? INFINITY : e;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kMassAhead; ++k) {
            if (v[k] == 0xffffffffu) continue;
            uint32_t r = 0;
            if (r0 == 0) {
#pragma unroll
                for (int i = 0; i < kMassAhead; ++i)
                    if (i < (int)rows) w[k] += __builtin_amdgcn_exp2f(ahead[k][i] - s_lse[i]);
                r = kMassAhead;
            }
#pragma unroll 4
            for (; r < rows; ++r) w[k] += __builtin_amdgcn_exp2f(x[(r0 + r) * a.logit_stride + v[k]] - s_lse[r]);
        }
    }
#pragma unroll
    for (int k = 0; k < kMassAhead; ++k)
        if (t0 + k * kJoinThreads < n) out[t0 + k * kJoinThreads] = old[k] + w[k];
}

// One workgroup per query head of a sequence: nothing to do where one run
// held all of its tokens; else the runs' shares, rescaled to their common
// maximum.  It is a chain of two loads (which shares; their maxima, sums and
// outputs together), and every wave works the weights out for itself instead
// of waiting for another.  The workgroups behind them add the mass.
template <bool BF16>
__global__ __launch_bounds__(kJoinThreads) void k_join(AttendArgs a) {
    __shared__ float s_w[kJoinThreads / 64][kMaxRuns];
    __shared__ f32x4 s_o[kJoinThreads];
    const uint32_t tid = threadIdx.x, wave = tid >> 6, b = blockIdx.y, head = blockIdx.x;
    const uint32_t joins = a.runs ? a.heads : 0;
    if (head >= joins) {
        const uint32_t i = head - joins, part = i / a.c.kv_heads;
        add_mass(a, b, i - part * a.c.kv_heads, part);
        return;
    }
    const uint32_t h = head / a.group;
    const Shares sh(a, b, h, head - h * a.group);
    const uint32_t n = sh.n;
    if (n <= 1) return;
    const uint32_t pieces = a.c.dim / 4;             // 4-column pieces of a row
    const uint32_t ways = kJoinThreads / pieces;     // shares summed side by side
    const uint32_t way = tid / pieces, d = (tid - way * pieces) * 4;
    f32x4 y[kJoinAhead];
#pragma unroll
    for (int i = 0; i < kJoinAhead; ++i) {
        const uint32_t j = way + i * ways;
        y[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (way < ways && j < n) y[i] = *(const f32x4 *)(a.share_o + sh.at(a, j) * a.c.dim + d);
    }
    float top, sum;
    weigh(a, sh, top, sum, [&](uint32_t j, float w) { s_w[wave][j] = w; });
    __builtin_amdgcn_wave_barrier();
    f32x4 o{0.f, 0.f, 0.f, 0.f};
    if (way < ways) {
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) {
            const uint32_t j = way + i * ways;
            if (j < n) o += y[i] * s_w[wave][j];
        }
        for (uint32_t j = way + kJoinAhead * ways; j < n; j += ways)
            o += *(const f32x4 *)(a.share_o + sh.at(a, j) * a.c.dim + d) * s_w[wave][j];
    }
    s_o[tid] = o;
    __syncthreads();
    if (tid < pieces) {
        for (uint32_t w = 1; w < ways; ++w) o += s_o[w * pieces + tid];
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        u32x2 z{pack2<BF16>(o[0] * inv, o[1] * inv), pack2<BF16>(o[2] * inv, o[3] * inv)};
        *(u32x2 *)(a.out + b * a.os[0] + head * a.os[1] + d) = z;
        if (tid == 0) {
            const float e = sum == 0.f ? -INFINITY : top + log2f(sum);
            if (a.lse) a.lse[b * (uint64_t)a.heads + head] = e * kLn2;
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// How an attention is laid out: query rows a workgroup, runs, workspace.
struct AttendPlan {
    uint32_t group, row_tiles, rows, blocks, runs;
    uint64_t logit_stride;
    size_t o_at, ml_at, lse2_at, logits_at, bytes;
};

// As many runs as workgroups are resident on 256 compute units, which the
// registers of k_attend decide.  16 sequences of 8192 tokens, 8 KV heads, us with
// 256, 512, 768 and 1024 runs: dim 64 71, 54, 52, 57; dim 128 96, 91, 94, 92;
// dim 256 171, 175, 185, 185; 2 sequences, dim 256 31, 36, 43, 48.
constexpr uint32_t runs_for(uint32_t dim, uint32_t blocks) {
    return dim <= 64 ? (blocks == 1 ? 768 : blocks == 2 ? 512 : 256) : dim <= 128 && blocks == 1 ? 512 : 256;
}
constexpr uint32_t most_runs() {
    uint32_t most = 0;
    for (uint32_t dim = 64; dim <= 256; dim += 64)
        for (uint32_t blocks = 1; blocks <= 4; blocks *= 2)
            if (runs_for(dim, blocks) > most) most = runs_for(dim, blocks);
    return most;
}
static_assert(most_runs() <= kMaxRuns, "a query head's shares fit the joins");

inline bool attend_plan(const splitzip_kv_cache *c, uint32_t heads, uint32_t mass_len, AttendPlan &p) {
    if (heads == 0 || heads > SPLITZIP_KV_MAX_HEADS || heads % c->kv_heads) return false;
    p.group = heads / c->kv_heads;
    const uint32_t all = c->max_pages * c->page_size;
    const uint64_t kv_units = (uint64_t)(all ? (all - 1) / kUnit + 1 : 1) * c->batch * c->kv_heads;
    // K and V are read once for every row tile: of 64 rows, or 32 where the
    // accumulators of 64 would not fit the registers, or where there is so little
    // to read that more and shorter workgroups win (64 rows against 32, dim 128,
    // 64 rows a KV head, us: 256 units 24 and 18, 512 26 and 24, 768 35.3 and
    // 33.9, 8192 147 and 213).  Units are of what the table can hold: the lengths
    // are on the device.
    const uint32_t most = c->head_dim <= 128 && kv_units >= 1024 ? 64 : 32;
    p.row_tiles = (p.group - 1) / most + 1;
    p.rows = (p.group - 1) / p.row_tiles + 1;
    p.row_tiles = (p.group - 1) / p.rows + 1;
    p.blocks = p.rows > 32 ? 4 : p.rows > 16 ? 2 : 1;
    const uint64_t units = kv_units * p.row_tiles;
    if (units >> 31) return false;
    const uint32_t runs = runs_for(c->head_dim, p.blocks);
    p.runs = units < runs ? (uint32_t)units : runs;
    if (mass_len > all) mass_len = all;      // no sequence is longer
    p.logit_stride = ((uint64_t)mass_len + 3) & ~3ull;
    if ((double)p.logit_stride * c->batch * heads > 1e15) return false;
    if ((p.logit_stride / kMassTokens + 1) * c->kv_heads + heads >= 1ull << 24) return false;      // k_join's grid
    p.o_at = up16((size_t)c->batch * c->kv_heads * p.row_tiles * 8);
    p.ml_at = up16(p.o_at + (size_t)p.runs * 2 * p.rows * c->head_dim * 4);
    p.lse2_at = up16(p.ml_at + (size_t)p.runs * 2 * p.rows * 8);
    p.logits_at = up16(p.lse2_at + (p.logit_stride ? (size_t)c->batch * heads * 4 : 0));
    p.bytes = p.logits_at + 4 * p.logit_stride * c->batch * heads;
    if (p.bytes < 16) p.bytes = 16;
    return true;
}

// Whole, with few units a KV head: no join (5 us), no search for the run's
// place.  Split/whole in us, KV heads by units (dim 128, batches of equal and
// of ragged lengths): 64 x 2 11.1/8.5 and 10.5/7.8, 64 x 4 11.5/14.1 and
// 11.1/13.2, 256 x 4 20.0/16.1 and 13.1/13.6, 256 x 8 30.3/27.3 and 16.1/23.6,
// 2048 x 4 96/89 and 41/38, 2048 x 32 650/643 and 123/155.
inline bool whole_heads(uint64_t tiles, uint32_t units) {
    return tiles < 1u << 24 && (units <= 2 || (units <= 4 && tiles >= 256));      // a grid's limit
}

// How many runs a launch has, where no sequence sees more than `seen` tokens;
// its workgroups.
inline uint32_t lay_out(AttendArgs &a, const AttendPlan &P, uint64_t seen) {
    const uint32_t units = seen ? (uint32_t)((seen - 1) / kUnit + 1) : 1;
    const uint64_t tiles = (uint64_t)a.c.batch * a.c.kv_heads * P.row_tiles;
    const bool whole = whole_heads(tiles, units);
    a.runs = whole ? 0 : tiles * units < P.runs ? (uint32_t)(tiles * units) : P.runs;
    a.by_runs = make_div(a.runs ? a.runs : 1);
    a.by_row_tiles = make_div(P.row_tiles);
    a.by_pairs = make_div(a.c.kv_heads * P.row_tiles);
    return a.runs ? a.runs : (uint32_t)tiles;
}

template <bool BF16, int DP, int NT>
void launch_attend(const AttendArgs &a, uint32_t grid, hipStream_t s) {
    if (a.c.dim == DP) k_attend<BF16, DP, NT, true><<<grid, kAttendThreads, 0, s>>>(a);
    else k_attend<BF16, DP, NT, false><<<grid, kAttendThreads, 0, s>>>(a);
}

template <bool BF16>
void launch_attend(const AttendArgs &a, uint32_t blocks, uint32_t grid, hipStream_t s) {
    const uint32_t d = (a.c.dim + 63) / 64;
    if (blocks == 1) {
        if (d == 1) launch_attend<BF16, 64, 1>(a, grid, s);
        else if (d == 2) launch_attend<BF16, 128, 1>(a, grid, s);
        else if (d == 3) launch_attend<BF16, 192, 1>(a, grid, s);
        else launch_attend<BF16, 256, 1>(a, grid, s);
    } else if (blocks == 4) {
        if (d == 1) launch_attend<BF16, 64, 4>(a, grid, s);
        else launch_attend<BF16, 128, 4>(a, grid, s);
    } else {
        if (d == 1) launch_attend<BF16, 64, 2>(a, grid, s);
        else if (d == 2) launch_attend<BF16, 128, 2>(a, grid, s);
        else if (d == 3) launch_attend<BF16, 192, 2>(a, grid, s);
        else launch_attend<BF16, 256, 2>(a, grid, s);
    }
}

}  // namespace

#endif  // SPLITZIP_CSRC_KV_ATTEND_H
