// attention.hip -- attention of packed query rows over the paged MXFP4 cache.
//
// Mathematics. Query i of a sequence with n queries and l cached tokens sits at
// position p = l - n + i and sees the tokens max(0, p - window + 1) .. p (all l
// without a mask). With s_j = scale log2(e) q . k_j, out = sum_j 2^(s_j - m) v_j /
// (sum_j 2^(s_j - m) + 2^(sink log2(e) - m)) for any m: one pass over the tokens
// with m a running maximum. Ranges of a sequence's tokens are worked on apart
// and joined by the same rule: sums scaled to the larger m and added. A query
// that sees no token gives zeros.
//
// gfx950 design. The tile of work of a wave is 16 NQ query rows of one kv head
// (row = query token x head of the group, so a group's heads share the tokens
// they read) against steps of 32 tokens.
//   * Scores: v_mfma_scale_f32_16x16x128_f8f6f4 takes the cache's own bytes: 16
//     tokens' E2M1 codes as the A operand, one 16-byte load a lane, their E8M0
//     bytes as its scales, so keys are never decoded. Queries, times scale
//     log2(e), are the B operand, as a sum of three E2M3 (6-bit) parts with block
//     scales 2^e, 2^(e-4), 2^(e-9), which leave 2^-13 of a block's largest
//     magnitude (two parts: 2^-9). 4- and 6-bit operands run at twice the rate of
//     8-bit ones, so the three products take 3/4 of the time of bf16 keys, and no
//     key is unpacked. The accumulator starts at minus the top in use (below): the
//     result is the exponent of the weight. Heads of 64 channels fill half of the
//     instruction's 128: the other half takes the second part of the same keys.
//   * The scores come out transposed (a lane has 8 tokens of one query row), which
//     is what the values' product takes as an operand: the weights never leave
//     their lane. The values are its other operand, 8 tokens of 2 channels a lane:
//     a lane loads the codes of D / 16 channels of 8 tokens, and
//     v_cvt_scalef32_pk_bf16_fp4 decodes two channels of one token with the
//     token's scale. A dense product wants two tokens of one channel side by side;
//     here the contraction runs over (token, channel parity) instead and the
//     weights are a 2:4 sparse operand (v_smfmac_f32_16x16x64_bf16) that is zero
//     for the other parity: two products, of the even and of the odd channels, take
//     the same registers with two index words, in the time of dense ones over the
//     tokens, and nothing is permuted. Half an operation an element, for all NQ
//     tiles. The weights' sum is one more such product, with ones.
//   * Weights are powers of two below a top that lies 8 above the maximum when it is
//     set, and is set anew only when a score passes it (a vote per step): the usual
//     step has no exchange between lanes and no rescaling. Weights are at most 1, so
//     the fp32 sums stay below the sum of the values' magnitudes, and the largest is
//     2^-8 or more: those that pass below the smallest normal number are 2^-118 of it.
// Weights are rounded to bf16 for the matrix cores: half a step is 2^-8 of a
// weight, in the sum as in the product, and the errors of a row's weights are
// independent: the result's own rounding is larger.
// No LDS and no barrier in the loop: the bytes of a step are few (4352 for 32
// tokens of 128 channels), waves that share tokens find them in the L1, and the
// loads of the next step are on their way into a second set of registers. (Measured
// before the offsets and shares of today, all else alike: a ring of steps in LDS,
// filled by direct-to-LDS loads, took 6 % longer for packed prompts and for 64
// ragged sequences, three or four sets of registers 13 to 28 % for the latter.)
//
// Bounds. One token of many sequences: HBM, 304 MB (64 sequences of 512 to 8192
// tokens) in 69 us, 4.4 TB/s; 64 of 16384 tokens 200 us, 5.7 TB/s. Prompts: issue,
// since vector instructions hardly overlap matrix ones here (a 16x16x32 product takes 20
// cycles, with two fma 24; the conversion of two values 6.6, an exp 9): per 32 tokens
// and 32 rows of 128 channels 12 + 16 + 2 matrix and about 100 vector instructions:
// 8192 new tokens 545 us, 1.01 PFLOP/s where the library's bf16 product of 8192^3
// reaches 1.23. Little of both: latency, of two reads one after the other (lengths,
// page numbers), a step and the joins: 777 tokens 10.8 us, 32 tokens 4.7.
// Two tiles of 128 channels (three of 64) fill 256 registers; four need the second
// half of the register file, and 35 moves a tile and step (slower); three waves a
// SIMD spill.
#include "device.hpp"
#include "kernels.hpp"

namespace e2m1 {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kRowWaves = 4;       // of a workgroup of attention_rows_kernel
constexpr int kStep = 32;          // tokens a wave takes at a time
constexpr float kSlack = 8.0f;     // how far the top lies above the maximum when it is set (0: packed prompts 419 us, not 355)
constexpr int kFarRight = 0x7FFFFFFF;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x6 __attribute__((ext_vector_type(6)));
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x32 __attribute__((ext_vector_type(32)));

// Quotients of numbers below 2^29 by `d` below 2^13 (Granlund and Montgomery): with 2^bits >= d and mul =
// ceil(2^(29 + bits) / d), n mul / 2^(29 + bits) exceeds n / d by less than 1 / d.
struct Divisor {
    uint32_t mul;
    int bits;
};

Divisor divisor_of(uint32_t d) {
    Divisor v = {0, 0};
    while ((1u << v.bits) < d) ++v.bits;
    v.mul = (uint32_t)((((uint64_t)1 << (29 + v.bits)) + d - 1) / d);
    return v;
}

__device__ __forceinline__ int divide(int n, const Divisor& d) {
    return (int)(__umulhi((uint32_t)n << 3, d.mul) >> d.bits);
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// The same number, but nothing that is made of it is made earlier: addresses of results, which would be kept in registers (and
// then out of them) through all steps. Two tiles of 128 channels: 50 spilled registers, 7 us a launch.
__device__ __forceinline__ int not_before(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

// ------------------------------------------------------------------- plan --

// What a sequence asks for.
struct Span {
    int first;   // its first query row
    int n;       // queries
    int len;     // cached tokens, also where the table has no room for them: positions go by it
};

// The tokens that a sequence's pages have room for.
__device__ __forceinline__ int table_room(const Attention& a, int page_bits) { return (int)(a.table_width << page_bits); }

__device__ __forceinline__ Span make_span(const Attention& a, int page_bits, int o0, int o1, int len) {
    const int tokens = (int)a.tokens;
    Span r;
    r.first = min(max(o0, 0), tokens);
    r.n = min(max(o1, r.first), tokens) - r.first;
    r.len = max(len, 0);
    if (len > table_room(a, page_bits) && r.n > 0 && a.err_flag) *a.err_flag = 1;
    return r;
}

__device__ __forceinline__ Span span_of(const Attention& a, int page_bits, int s) {
    return make_span(a, page_bits, a.q_offsets[s], a.q_offsets[s + 1], a.kv_lens[s]);
}

// The first token that query i of a sequence sees.
__device__ __forceinline__ int first_seen(const Attention& a, const Span& s, int i) {
    const int pos = s.len - s.n + i, window = (int)a.window;
    return window > 0 && window <= pos ? pos - window + 1 : 0;
}

__device__ __forceinline__ uint32_t tiles_of(const Span& s, int group, int rows) {
    return (uint32_t)(s.n * group + rows - 1) / (uint32_t)rows;
}

// Units of 2^unit_bits tokens of every tile of a sequence.
__device__ __forceinline__ uint32_t units_of(const Attention& a, int page_bits, const Span& s, int unit_bits) {
    const int hi = min(s.len, table_room(a, page_bits)), lo = min(first_seen(a, s, 0), hi) & ~(kStep - 1);
    return max(1u, ((uint32_t)(hi - lo) + (1u << unit_bits) - 1) >> unit_bits);
}

template <int kCtrl, int kRowMask>
__device__ __forceinline__ uint32_t shifted(uint32_t v) {   // 0 where there is no lane to take from
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, kRowMask, 0xF, false);
}

// Sums over the lanes up to each one's own.
__device__ __forceinline__ uint32_t scan(uint32_t v) {
    v += shifted<0x111, 0xF>(v);   // row_shr:1, 2, 4, 8
    v += shifted<0x112, 0xF>(v);
    v += shifted<0x114, 0xF>(v);
    v += shifted<0x118, 0xF>(v);
    v += shifted<0x142, 0xA>(v);   // row_bcast:15 to rows 1 and 3
    v += shifted<0x143, 0xC>(v);   // row_bcast:31 to rows 2 and 3
    return v;
}

__device__ __forceinline__ int from_lane(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// Sequences laid end to end by weight. Up to 64 are read once and kept, one a lane. Of more, a lane has the sum of a run of
// whole rounds of the wave (64 sequences side by side, four rounds on their way), and the run that holds a place is gone
// through again.
struct Plan {
    const Attention& a;
    int page_bits, lane, per;
    Span mine;                 // of the lane's sequence, where each lane has one
    uint32_t before, total;
    bool ok;                   // no offset is below the one before it: then no query row belongs to two sequences

    __device__ __forceinline__ int begin() const { return lane * per; }
    __device__ __forceinline__ int end(int owner) const { return (int)min((int64_t)(owner + 1) * per, a.seqs); }

    // The weights of the lane's run.
    template <typename F>
    __device__ __forceinline__ uint32_t run_sum(F weight, bool& bad) const {
        constexpr int kRounds = 4;
        uint32_t sum = 0;
        const int seqs = (int)a.seqs;
        for (int s0 = 0; s0 < seqs; s0 += kRounds * kWave) {
            int o0[kRounds], o1[kRounds], len[kRounds];
#pragma unroll
            for (int i = 0; i < kRounds; ++i) {
                const int s = min(s0 + i * kWave + lane, seqs - 1);
                o0[i] = a.q_offsets[s];
                o1[i] = a.q_offsets[s + 1];
                len[i] = a.kv_lens[s];
            }
#pragma unroll
            for (int i = 0; i < kRounds; ++i) {
                const int s = s0 + i * kWave;
                const uint32_t w = s + lane < seqs ? weight(make_span(a, page_bits, o0[i], o1[i], len[i])) : 0;
                const uint32_t all = (uint32_t)from_lane((int)scan(w), kWave - 1);
                if (s >= begin() && s < begin() + per) sum += all;
                bad |= o1[i] < o0[i];
            }
        }
        return sum;
    }

    template <typename F>
    __device__ __forceinline__ Plan(const Attention& a_, int page_bits_, int lane_, F weight)
        : a(a_), page_bits(page_bits_), lane(lane_) {
        per = a.seqs <= kWave ? 1 : (int)((a.seqs + kWave * kWave - 1) / (kWave * kWave)) * kWave;
        mine = {0, 0, 0};
        uint32_t sum = 0;
        bool bad = false;
        if (per == 1) {
            if (lane < a.seqs) {
                mine = span_of(a, page_bits, lane);
                bad = a.q_offsets[lane + 1] < a.q_offsets[lane];
            }
            sum = weight(mine);
        } else {
            sum = run_sum(weight, bad);
        }
        ok = !__any(bad);
        if (bad && a.err_flag) *a.err_flag = 1;
        const uint32_t after = scan(sum);
        before = after - sum;
        total = (uint32_t)from_lane((int)after, kWave - 1);
    }

    // Another weight's sum over the sequences before `seq`, and over all.
    template <typename F>
    __device__ __forceinline__ uint32_t sum_before(int seq, F weight, uint32_t& all) const {
        bool bad = false;
        const uint32_t sum = per == 1 ? weight(mine) : run_sum(weight, bad);
        const uint32_t after = scan(sum);
        all = (uint32_t)from_lane((int)after, kWave - 1);
        const int owner = (int)((uint32_t)seq / (uint32_t)per);
        uint32_t part = (uint32_t)from_lane((int)(after - sum), owner);
        for (int s = owner * per; s < seq; s += kWave) {
            const uint32_t w = s + lane < seq ? weight(span_of(a, page_bits, s + lane)) : 0;
            part += (uint32_t)from_lane((int)scan(w), kWave - 1);
        }
        return part;
    }

    // A sequence, the same for every lane.
    __device__ __forceinline__ Span span(int seq) const {
        if (per == 1) return {from_lane(mine.first, seq), from_lane(mine.n, seq), from_lane(mine.len, seq)};
        const Span s = span_of(a, page_bits, seq);
        return {uniform(s.first), uniform(s.n), uniform(s.len)};
    }

    // The sequence that holds place `at` < total, and where it begins.
    template <typename F>
    __device__ __forceinline__ int find(uint32_t at, uint32_t& begins, F weight) const {
        // the last lane whose run begins at or before it: empty runs before it begin at the same place
        const int owner = 63 - __builtin_clzll(__ballot(before <= at && begin() < end(lane)));
        begins = (uint32_t)from_lane((int)before, owner);
        if (per == 1) return owner;
        const int last = end(owner);
        for (int s = owner * per;; s += kWave) {
            const uint32_t w = s + lane < last ? weight(span_of(a, page_bits, s + lane)) : 0;
            const uint32_t after = scan(w);
            const uint64_t past = __ballot(begins + after > at);
            if (past != 0 || s + kWave >= last) {
                const int i = past != 0 ? __builtin_ctzll(past) : last - 1 - s;
                begins += (uint32_t)from_lane((int)(after - w), i);
                return s + i;
            }
            begins += (uint32_t)from_lane((int)after, kWave - 1);
        }
    }
};

// ------------------------------------------------------------------- step --
// Tokens of a step: as scores, lane group g has 8 g + 4 t + r (r = 0..3) of product t; as values, 16 t + 4 g + r. Halves of
// 16 tokens lie in one page each.

// Where a step's halves are: rows of the cache's [pages, heads, page]; ok: they are there and some row sees a token.
struct Place {
    int64_t row[2];
    bool ok[2];
    int base;   // first token
};

template <int D>
struct Keys {
    u32x4 k[2];       // 32 channels of the token of row lane % 16 of product t
    uint32_t ks[2];   // their scale byte
};

template <int D>
struct Values {
    uint32_t v[8];            // D / 16 channels of each token
    uint32_t vs[2][D / 32];   // the tokens' scale bytes
};

// A wave's rows.
template <int NQ>
struct Rows {
    i32x8 q[NQ][3];       // the parts of 32 channels of row lane % 16
    uint32_t qs[NQ];      // their scale bytes, one a part
    int lo[NQ], hi[NQ];   // the tokens that row lane % 16 sees
    int lo_all, hi_all;   // the tokens that some row sees
    int lo_max, hi_min;   // the tokens that every row sees
};

// o: channels D / 16 (lane % 16) + 2 b + c of rows 4 g + r; l: the weights' sums of these rows. Of row lane % 16: minus the
// top (four times, as the scores' accumulator) and how far above it a score may be: nothing before there is one, then 0.
template <int D, int NQ>
struct Sums {
    f32x4 o[NQ][D / 16];
    f32x4 l[NQ];
    f32x4 less[NQ];
    float slack[NQ];
    __device__ __forceinline__ float top(int i) const { return slack[i] < 0.0f ? -INFINITY : -less[i][0]; }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            slack[i] = -INFINITY;
            l[i] = less[i] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[i][j] = f32x4{0, 0, 0, 0};
        }
    }
};

// Lane constants of the loads: byte offsets in a run of 16 tokens.
template <int D>
struct Lane {
    int lane, n, g;
    uint32_t k, ks, v, vs;
    uint32_t turn;   // rotation that brings the scale of the lane's channels to an exponent field
    int own;         // the block of its channels
    __device__ __forceinline__ Lane(int lane_) : lane(lane_) {
        n = lane % 16;
        g = lane / 16;
        const int block = D == 128 ? g : g & 1;
        const int token = 8 * (n / 4 % 2) + n % 4;   // of product 0; 4 on in product 1
        k = token * (D / 2) + block * 16;
        ks = token * (D / 32) + block;
        v = 4 * g * (D / 2) + n * (D / 32);
        vs = 4 * g * (D / 32);
        own = n * (D / 16) / 32;
        turn = 8 * own + 9;
    }
};

// Where a wave's next 32 steps are: lane 2 i + t holds the page of half t of step at + i stride, -1 where no row sees a token
// of it or the page is not there.
__device__ __forceinline__ int pages_ahead(const Attention& a, const CacheView& c, const int32_t* table, int at, int stride,
                                           int lo_all, int hi_all, int lane) {
    const int64_t tb = (int64_t)(at + (lane / 2) * stride) * kStep + (lane % 2) * 16;
    if (tb >= hi_all || tb + 16 <= lo_all) return -1;
    const int pg = table[tb >> c.page_bits];
    if (pg >= 0 && ((int64_t)pg << c.page_bits) < c.slots) return pg;
    if (a.err_flag) *a.err_flag = 1;
    return -1;
}

// The `i`-th step that `pages` holds; halves that are not there are read as the cache's first tokens.
__device__ __forceinline__ Place place_of(const CacheView& c, int pages, int i, int head, int base) {
    Place p;
    p.base = base;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int pg = from_lane(pages, 2 * i + t);
        p.ok[t] = pg >= 0;
        p.row[t] = p.ok[t] ? ((((int64_t)pg * c.heads + head) << c.page_bits) + ((base + 16 * t) & ((1 << c.page_bits) - 1)))
                           : 0;
    }
    return p;
}

template <int D>
__device__ __forceinline__ void load_keys(Keys<D>& s, const CacheView& c, const Place& p, const Lane<D>& ln) {
    const int64_t row = ln.n < 8 ? p.row[0] : p.row[1];
    const uint8_t* k = c.k_codes + row * (D / 2) + ln.k;
    const uint8_t* x = c.k_scales + row * (D / 32) + ln.ks;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        s.k[t] = *reinterpret_cast<const u32x4*>(k + t * 4 * (D / 2));
        s.ks[t] = x[t * 4 * (D / 32)];
    }
}

template <int D>
__device__ __forceinline__ void load_values(Values<D>& s, const CacheView& c, const Place& p, const Lane<D>& ln) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint8_t* v = c.v_codes + p.row[t] * (D / 2);
        const uint8_t* x = c.v_scales + p.row[t] * (D / 32);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if constexpr (D == 128) s.v[4 * t + r] = *reinterpret_cast<const uint32_t*>(v + ln.v + r * 64);
            else s.v[4 * t + r] = *reinterpret_cast<const uint16_t*>(v + ln.v + r * 32);
        }
        if constexpr (D == 128) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(x + ln.vs);
#pragma unroll
            for (int r = 0; r < 4; ++r) s.vs[t][r] = w[r];
        } else {
            const u32x2 w = *reinterpret_cast<const u32x2*>(x + ln.vs);
            s.vs[t][0] = w.x;
            s.vs[t][1] = w.y;
        }
    }
}

// Scale bytes of token r of a half: one word (128 channels) or half of one.
template <int D>
__device__ __forceinline__ uint32_t scale_bytes(const uint32_t (&vs)[D / 32], int r) {
    if constexpr (D == 128) return vs[r];
    else return (vs[r / 2] >> (16 * (r % 2))) & 0xFFFFu;
}

template <int D>
__device__ __forceinline__ void clear_token(Values<D>& s, int t, int r, bool clear) {
    s.v[4 * t + r] = clear ? 0u : s.v[4 * t + r];
    if constexpr (D == 128) s.vs[t][r] = clear ? 0u : s.vs[t][r];
    else s.vs[t][r / 2] &= clear ? (r % 2 ? 0x0000FFFFu : 0xFFFF0000u) : 0xFFFFFFFFu;
}

__device__ __forceinline__ uint32_t pack_weights(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Scores of a step's tokens, less the top.
template <int D, int NQ>
__device__ __forceinline__ void score(f32x4 (&x)[NQ][2], const Keys<D>& s, const Rows<NQ>& rows, const Sums<D, NQ>& sums) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const i32x8 k = {(int)s.k[t].x, (int)s.k[t].y, (int)s.k[t].z, (int)s.k[t].w, 0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            f32x4 z = sums.less[i];
            z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, rows.q[i][0], z, 4, 2, 0, s.ks[t], 0, rows.qs[i]);
            z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, rows.q[i][1], z, 4, 2, 0, s.ks[t], 1, rows.qs[i]);
            if constexpr (D == 128)
                z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, rows.q[i][2], z, 4, 2, 0, s.ks[t], 2, rows.qs[i]);
            x[i][t] = z;
        }
    }
}

// Bits [lo, hi) of 32.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
    const uint32_t upto = hi <= 0 ? 0u : hi >= 32 ? 0xFFFFFFFFu : (1u << hi) - 1;
    const uint32_t under = lo <= 0 ? 0u : lo >= 32 ? 0xFFFFFFFFu : (1u << lo) - 1;
    return upto & ~under;
}

// Values with scale byte 255 in a step that not all rows see whole: NaN for the rows that see the token, in its block's
// channels, and zeros for the product with the others' weights.
template <int D, int NQ>
__device__ __forceinline__ void values_not_finite(Values<D>& s, const Rows<NQ>& rows, Sums<D, NQ>& sums, int base,
                                                  const Lane<D>& ln) {
    uint32_t bad = 0;   // bit 16 t + 4 g + r: that token, in the block of the lane's channels
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint32_t w = scale_bytes<D>(s.vs[t], r);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t there = (uint32_t)from_lane((int)w, 16 * g);
                bad |= ((there >> (8 * ln.own)) & 255u) == 255u ? 1u << (16 * t + 4 * g + r) : 0u;
            }
            clear_token<D>(s, t, r, ((w >> (8 * ln.own)) & 255u) == 255u);
        }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        f32x4 z;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int lo = __shfl(rows.lo[i], 4 * ln.g + e, kWave), hi = __shfl(rows.hi[i], 4 * ln.g + e, kWave);
            z[e] = (bad & bits_between(lo - base, hi - base)) ? __uint_as_float(0x7FC00000u) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j) sums.o[i][j] += z;
    }
}

// Weights of a step's tokens, and their products with its values.
template <int D, int NQ>
__device__ __forceinline__ void take_step(const Keys<D>& keys, Values<D>& s, const Place& p, const Rows<NQ>& rows,
                                          Sums<D, NQ>& sums, const Lane<D>& ln) {
    constexpr int NJ = D / 16;
    f32x4 x[NQ][2];
    score<D, NQ>(x, keys, rows, sums);
    if (p.base < rows.lo_max || p.base + kStep > rows.hi_min || !(p.ok[0] && p.ok[1])) {   // not every row sees every token
        const bool there = ln.g < 2 ? p.ok[0] : p.ok[1];
        bool high = false;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = p.base + 8 * ln.g + 4 * t + r;
#pragma unroll
                for (int i = 0; i < NQ; ++i)
                    x[i][t][r] = there && j >= rows.lo[i] && j < rows.hi[i] ? x[i][t][r] : -INFINITY;
                // values that no row sees stay finite whatever is there
                const int jv = p.base + 16 * t + 4 * ln.g + r;
                clear_token<D>(s, t, r, !(p.ok[t] && jv >= rows.lo_all && jv < rows.hi_all));
                const uint32_t w = scale_bytes<D>(s.vs[t], r);
                high |= (w & (w << 1) & 0x80808080u) != 0;   // bytes from 192 on: rare enough to be looked at one by one
            }
        if (__any(high)) values_not_finite<D, NQ>(s, rows, sums, p.base, ln);
    }
    // the top is left alone until a score is above it
    bool past = false;
    float top[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        float v = fmaxf(fmaxf(x[i][0][0], x[i][0][1]), x[i][0][2]);
        v = fmaxf(fmaxf(v, x[i][0][3]), x[i][1][0]);
        v = fmaxf(fmaxf(v, x[i][1][1]), x[i][1][2]);
        top[i] = fmaxf(v, x[i][1][3]);
        past |= top[i] > sums.slack[i];
    }
    if (__any(past)) {
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            float v = fmaxf(top[i], __shfl_xor(top[i], 16, kWave));
            v = fmaxf(v, __shfl_xor(v, 32, kWave));
            const bool none = sums.slack[i] < 0.0f;
            v += kSlack;
            const float by = v == -INFINITY ? 0.0f : none ? v : fmaxf(v, 0.0f);   // 16 rows at once: each to its maximum
            const float f = none ? 1.0f : exp2_raw(-by);
            if (v != -INFINITY) sums.slack[i] = 0.0f;
            sums.less[i] -= by;
#pragma unroll
            for (int t = 0; t < 2; ++t) x[i][t] -= by;
            const f32x4 f4 = {__shfl(f, 4 * ln.g, kWave), __shfl(f, 4 * ln.g + 1, kWave), __shfl(f, 4 * ln.g + 2, kWave),
                              __shfl(f, 4 * ln.g + 3, kWave)};   // of the rows that this lane has the sums of
            sums.l[i] *= f4;
#pragma unroll
            for (int j = 0; j < NJ; ++j) sums.o[i][j] *= f4;
        }
    }
    constexpr int kEven = (int)0x88888888u, kOdd = (int)0xDDDDDDDDu;   // places 0 and 2, 1 and 3 of every four
    const uint32_t one = 0x3F803F80u;
    const u32x4 ones = {one, one, one, one};
    bf16x8 w[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        float e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = exp2_raw(x[i][k / 4][k % 4]);
        const u32x4 pk = {pack_weights(e[0], e[1]), pack_weights(e[2], e[3]), pack_weights(e[4], e[5]),
                          pack_weights(e[6], e[7])};
        w[i] = __builtin_bit_cast(bf16x8, pk);
        sums.l[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], __builtin_bit_cast(bf16x8, ones), sums.l[i], 0, 0, 0);
    }
    // values: a byte (two channels) of all eight tokens at a time
    float sc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = D == 128 ? s.vs[e / 4][e % 4] : s.vs[e / 4][(e % 4) / 2];
        sc[e] = __uint_as_float(__builtin_amdgcn_alignbit(b, b, D == 128 ? ln.turn : ln.turn + 16 * (e % 2)));
    }
#pragma unroll
    for (int b = 0; b < NJ / 2; ++b) {
        u32x8 d;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            bf16x2 v;
            if (b == 0) v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.v[e], sc[e], 0);
            else if (b == 1) v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.v[e], sc[e], 1);
            else if (b == 2) v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.v[e], sc[e], 2);
            else v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.v[e], sc[e], 3);
            d[e] = __builtin_bit_cast(uint32_t, v);
        }
        const bf16x16 both = __builtin_bit_cast(bf16x16, d);
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            sums.o[i][2 * b] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(w[i], both, sums.o[i][2 * b], kEven, 0, 0);
            sums.o[i][2 * b + 1] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(w[i], both, sums.o[i][2 * b + 1], kOdd, 0, 0);
        }
    }
}

// ---------------------------------------------------------------- queries --

// x <- by x - part: what a part leaves, in units `by` times smaller.
__device__ __forceinline__ void take_off(float (&x)[32], float by, const f16x32& part) {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __builtin_fmaf(x[i], by, -(float)part[i]);
}

__device__ __forceinline__ f16x32 as_f16(const float (&x)[32]) {
    f16x32 h;
#pragma unroll
    for (int i = 0; i < 32; ++i) h[i] = (_Float16)x[i];
    return h;
}

__device__ __forceinline__ i32x8 widen(const u32x6& v) {
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], (int)v[4], (int)v[5], 0, 0};
}

// The three parts of a lane's 32 channels times `scale`, in units 2^e where the largest magnitude lies in (3.75, 7.5] (7.5 is
// E2M3's largest). The first part leaves at most 1/4 (half of its largest step), the second, in units of 2^-4, at most 2^-7,
// the third, in 2^-9, 2^-12: less than 2^-13 of the largest. Remainders are fp32, each in its part's unit, and go through fp16
// on their way to a part, which may pass a border between two of its values by no more than half a step of fp16: 2^-9 of the
// first unit, 2^-10 of the others. What is left stays within 1/4 + 2^-9, 2^-7 + 2^-14 and 2^-12 + 2^-19: the next part's value
// nearest to it is the last one before its steps grow (through bf16 2^-6 can be left for the third part, past its end, and 2^-10
// by it; the conversion from fp32, 2xpk16, gets its result on its operands' registers from this compiler, and spoils two of them).
// A block that holds a NaN or an infinity gets the scale NaN.
template <int D>
__device__ __forceinline__ void split_query(const u32x4 (&w)[4], float scale, int g, i32x8 (&q)[3], uint32_t& scales) {
    u16x2 top = {0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[i / 4][i % 4] & 0x7FFF7FFFu));
    const float largest = __uint_as_float(max((uint32_t)top.x, (uint32_t)top.y) << 16) * scale;
    const uint32_t most = __float_as_uint(largest) & 0x7FFFFFFFu;
    const uint32_t field = (most + 0xFFFFFu) >> 23;   // past 1.875 2^n: of 2^(n+1)
    const uint32_t e = max(field, 11u) - 2u;
    const float unit = __uint_as_float((254u - e) << 23);   // 2^-e
    float x[32];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t v = w[i / 4][i % 4];
        x[2 * i] = __uint_as_float(v << 16) * scale * unit;
        x[2 * i + 1] = __uint_as_float(v & 0xFFFF0000u) * scale * unit;
    }
    const u32x6 p0 = __builtin_amdgcn_cvt_scalef32_pk32_fp6_f16(as_f16(x), 1.0f);
    take_off(x, 16.0f, __builtin_amdgcn_cvt_scalef32_pk32_f16_fp6(p0, 16.0f));
    const u32x6 p1 = __builtin_amdgcn_cvt_scalef32_pk32_fp6_f16(as_f16(x), 1.0f);
    take_off(x, 32.0f, __builtin_amdgcn_cvt_scalef32_pk32_f16_fp6(p1, 32.0f));
    const u32x6 p2 = __builtin_amdgcn_cvt_scalef32_pk32_fp6_f16(as_f16(x), 1.0f);
    if constexpr (D == 128) {
        q[0] = widen(p0);
        q[1] = widen(p1);
        q[2] = widen(p2);
        scales = e | (e - 4u) << 8 | (e - 9u) << 16;
    } else {   // the upper half of the lanes has the same channels: the second part, and nothing
        const bool up = g >= 2;
        u32x6 first, second;
#pragma unroll
        for (int i = 0; i < 6; ++i) {
            first[i] = up ? p1[i] : p0[i];
            second[i] = up ? 0u : p2[i];
        }
        q[0] = widen(first);
        q[1] = widen(second);
        q[2] = q[1];   // not used
        scales = (up ? e - 4u : e) | (e - 9u) << 8;
    }
    if (most >= 0x7F800000u) scales = 0xFFFFFFFFu;
}

// The rows [row0, row0 + 16 NQ) of a sequence's (query, head of the group) pairs; rows past the last one see what it sees.
template <int D, int NQ>
__device__ __forceinline__ void set_ranges(Rows<NQ>& rows, const Attention& a, int room, const Span& s, int group,
                                           const Divisor& by, int row0, const Lane<D>& ln) {
    const int last = s.n * group - 1;
    const int i_first = divide(row0, by), i_last = divide(min(row0 + 16 * NQ - 1, last), by);
    const int p0 = s.len - s.n;   // position of query 0
    if (a.causal) {
        rows.lo_all = first_seen(a, s, i_first);
        rows.lo_max = first_seen(a, s, i_last);
        rows.hi_all = max(0, min(p0 + i_last + 1, room));
        rows.hi_min = max(0, min(p0 + i_first + 1, room));
    } else {
        rows.lo_all = rows.lo_max = 0;
        rows.hi_all = rows.hi_min = min(s.len, room);
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int q = divide(min(row0 + 16 * i + ln.n, last), by);
        rows.lo[i] = a.causal ? first_seen(a, s, q) : 0;
        rows.hi[i] = max(0, min(a.causal ? p0 + q + 1 : s.len, room));
    }
}

// Steps first, first + stride, .. below `last` of a wave's rows. The bytes of the steps to come are on their way while
// one is worked on.
template <int D, int NQ>
__device__ __forceinline__ void run_steps(const Attention& a, const CacheView& c, const int32_t* table, const Span& s,
                                          int kv_head, int group, const Divisor& by, int row0, int first, int last,
                                          int stride, Sums<D, NQ>& sums, const Lane<D>& ln) {
    Rows<NQ> rows;
    set_ranges<D, NQ>(rows, a, table_room(a, c.page_bits), s, group, by, row0, ln);
    sums.clear();
    // steps with a token that some row sees
    int at = first;
    const int low = rows.lo_all / kStep;
    if (at < low) at += (low - at + stride - 1) & ~(stride - 1);   // stride: a power of two
    const int end = min(last, (int)(((uint32_t)rows.hi_all + kStep - 1) / kStep));
    if (at >= end) return;
    if (c.slots == 0) {   // no page is there
        if (a.err_flag) *a.err_flag = 1;
        return;
    }
    // the queries' bytes first: their parts are made while the first tokens are on their way
    u32x4 w[NQ][4];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int row = min(row0 + 16 * i + ln.n, s.n * group - 1);
        const int q = divide(row, by);
        const int block = D == 128 ? ln.g : ln.g & 1;
        const uint16_t* p =
            a.q + (int64_t)(s.first + q) * a.q_stride + (int64_t)(kv_head * group + (row - q * group)) * D + block * 32;
#pragma unroll
        for (int b = 0; b < 4; ++b) w[i][b] = *reinterpret_cast<const u32x4*>(p + 8 * b);
    }
    const int lane = threadIdx.x % kWave;
    int pages = pages_ahead(a, c, table, at, stride, rows.lo_all, rows.hi_all, lane);
    int later = pages_ahead(a, c, table, at + 32 * stride, stride, rows.lo_all, rows.hi_all, lane);
    int i = 0;       // place in `pages` of the step whose keys are loaded next
    int ahead = at;  // and the step; past the end they are the cache's first tokens or a neighbour's, and not used
    auto next_place = [&] {
        const Place p = place_of(c, pages, i, kv_head, ahead * kStep);
        ahead += stride;
        if (++i == 32) {
            i = 0;
            pages = later;
            later = pages_ahead(a, c, table, ahead + 32 * stride, stride, rows.lo_all, rows.hi_all, lane);
        }
        return p;
    };
    Keys<D> keys[2];
    Values<D> values[2];
    Place p0 = next_place(), p1;
    load_keys<D>(keys[0], c, p0, ln);
    load_values<D>(values[0], c, p0, ln);
#pragma unroll
    for (int b = 0; b < NQ; ++b) {
        split_query<D>(w[b], a.scale * kLog2e, ln.g, rows.q[b], rows.qs[b]);
        __builtin_amdgcn_sched_barrier(0);   // a tile's parts after the other's: packed prompts 355 us, 361 without
    }
    for (;;) {
        p1 = next_place();
        load_keys<D>(keys[1], c, p1, ln);
        load_values<D>(values[1], c, p1, ln);
        take_step<D, NQ>(keys[0], values[0], p0, rows, sums, ln);
        if ((at += stride) >= end) return;
        p0 = next_place();
        load_keys<D>(keys[0], c, p0, ln);
        load_values<D>(values[0], c, p0, ln);
        take_step<D, NQ>(keys[1], values[1], p1, rows, sums, ln);
        if ((at += stride) >= end) return;
    }
}

// ---------------------------------------------------------------- results --

__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.0f : m; }

// What sums with maximum m and total l are to be multiplied by, the sink counted in.
__device__ __forceinline__ float last_factor(float m, float l, const float* sinks, int head) {
    float f = 1.0f;
    if (sinks) {
        const float s = sinks[head] * kLog2e;
        const float mn = finite_or_zero(fmaxf(m, s));
        f = exp2_raw(m - mn);
        l = l * f + exp2_raw(s == mn ? 0.0f : s - mn);   // equal: of infinities too
    }
    return l == 0.0f ? 0.0f : f * __builtin_amdgcn_rcpf(l);
}

template <int NJ>
__device__ __forceinline__ void store_out(uint16_t* p, const float (&v)[NJ]) {
    uint32_t w[NJ / 2 + 1];
#pragma unroll
    for (int j = 0; j < NJ / 2; ++j) w[j] = pack_weights(v[2 * j], v[2 * j + 1]);
    if constexpr (NJ == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (NJ == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (NJ == 2) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *p = (uint16_t)pack_weights(v[0], v[0]);
}

// Where a segment (a tile of a sequence) was cut: its parts are the second one of worker `from` and the first ones of the
// workers up to `to`.
struct Record {
    int row0, first;    // the tile's first row, the sequence's first query
    int from, to;       // from == to: nothing to join
    int rows, head;
    int pad[2];
};

// A worker has room for two parts (of the segment it begins in and of the one it ends in): 16 NQ rows of D sums, then
// maximum and total of each.
template <int D, int NQ>
constexpr size_t part_floats() { return (size_t)16 * NQ * (D + 2); }

// Split form: workers take equal shares of all units (2^unit_bits tokens of a tile), in a row. A worker is kW waves, which
// take every kW-th step of its share and join in LDS. Without records every segment is one unit, and nothing is left to join.
// Shares are cut at single steps: at every fourth, 64 sequences of 4352 tokens took 68.5 us instead of 63.5.
template <int D, int NQ, int kW>
__global__ __launch_bounds__(kW * kWave, 2) void attention_split_kernel(Attention a, CacheView c, float* parts,
                                                                        Record* records, int workers, int unit_bits,
                                                                        int record_count, bool by_segment, Divisor by) {
    constexpr int NJ = D / 16;
    constexpr int kRows = 16 * NQ;
    __shared__ f32x4 lo_o[kW == 1 ? 1 : kW][kW == 1 ? 1 : NJ][kWave];   // the waves' sums
    __shared__ __attribute__((aligned(16))) float lo_m[kW][16];
    __shared__ f32x4 lo_l[kW][4];
    const int lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
    const int group = a.heads / c.heads;

    auto segments = [&](const Span& s) { return tiles_of(s, group, kRows) * c.heads; };
    auto weight = [&](const Span& s) { return segments(s) * units_of(a, c.page_bits, s, unit_bits); };
    const Plan plan(a, c.page_bits, lane, weight);
    // neighbours in the order of work on the same XCD, whose L2 then holds what they share; of more workgroups than segments the
    // first ones have work, so that all XCDs do
    const int per_xcd = (records ? workers : (int)min(plan.total, (uint32_t)workers)) / 8;
    const int id = (int)blockIdx.x < per_xcd * 8 ? (int)(blockIdx.x % 8) * per_xcd + (int)blockIdx.x / 8 : (int)blockIdx.x;
    if (!plan.ok) {
        if (threadIdx.x == 0 && id < record_count) records[id].from = records[id].to = 0;
        return;
    }
    // without records a worker has one segment
    const uint32_t share = records ? plan.total / (uint32_t)workers : 0;
    const uint32_t more = plan.total - share * workers;
    uint32_t u = id * share + min((uint32_t)id, more);
    const uint32_t u_end = u + share + ((uint32_t)id < more ? 1 : 0);
    const bool idle = u >= u_end;
    uint32_t begin = 0, segs_before = 0;
    int seq = idle ? 0 : plan.find(u, begin, weight);
    if (by_segment) {   // a record for every segment there could be: worker i also writes the i-th where there is none
        uint32_t all;
        segs_before = plan.sum_before(seq, segments, all);
        if (threadIdx.x == 0 && id < record_count && (uint32_t)id >= all) records[id].from = records[id].to = 0;
    } else if (idle) {
        if (threadIdx.x == 0 && id < record_count) records[id].from = records[id].to = 0;
    }
    if (idle) return;
    Span s = plan.span(seq);
    uint32_t units = units_of(a, c.page_bits, s, unit_bits), segs = segments(s);
    Record cut = {};
    while (u < u_end) {
        while (u >= begin + segs * units) {   // on to the next sequence that has queries
            begin += segs * units;
            segs_before += segs;
            s = plan.span(++seq);
            units = units_of(a, c.page_bits, s, unit_bits);
            segs = segments(s);
        }
        const uint32_t segment = units == 1 ? u - begin : (u - begin) / units;
        const uint32_t seg_begin = begin + segment * units;
        const int u0 = (int)(u - seg_begin);
        const int u1 = (int)min(units, u_end - seg_begin);
        const uint32_t tiles = tiles_of(s, group, kRows);
        const int head = (int)(tiles == 1 ? segment : segment / tiles);
        const int row0 = (int)(segment - head * tiles) * kRows;
        const int origin = first_seen(a, s, 0) / kStep, steps = unit_bits - 5;
        Sums<D, NQ> sums;
        run_steps<D, NQ>(a, c, a.page_table + seq * a.table_width, s, head, group, by, row0,
                         origin + (u0 << steps) + wave, origin + (u1 << steps), kW, sums, Lane<D>(lane));
        const Lane<D> ln(not_before(lane));
        const bool whole = u0 == 0 && u1 == (int)units;
        float* part = parts + (2 * (size_t)id + (u0 > 0 ? 0 : 1)) * part_floats<D, NQ>();
        const int rows_left = s.n * group - row0;
        // sums of row `at`, channels d on
        auto put = [&](auto& o, int at, int d, float m, float total) {
            constexpr int kN = sizeof(o) / sizeof(float);
            if (at >= rows_left) return;
            if (whole) {
                const int row = row0 + at, q = divide(row, by);
                const int h = head * group + (row - q * group);
                const float f = last_factor(m, total, a.sinks, h);
#pragma unroll
                for (int j = 0; j < kN; ++j) o[j] *= f;
                store_out<kN>(a.out + ((int64_t)(s.first + q) * a.heads + h) * D + d, o);
            } else {
#pragma unroll
                for (int j = 0; j < kN; ++j) part[(size_t)at * D + d + j] = o[j];
                if (d == 0) {
                    part[(size_t)kRows * D + 2 * at] = m;
                    part[(size_t)kRows * D + 2 * at + 1] = total;
                }
            }
        };
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            if (16 * i >= rows_left) break;
            if constexpr (kW == 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float m = __shfl(sums.top(i), 4 * ln.g + e, kWave);
                    float o[NJ];
#pragma unroll
                    for (int j = 0; j < NJ; ++j) o[j] = sums.o[i][j][e];
                    put(o, 16 * i + 4 * ln.g + e, NJ * ln.n, m, sums.l[i][e]);
                }
            } else {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < NJ; ++j) lo_o[wave][j][ln.lane] = sums.o[i][j];
                if (ln.lane < 16) lo_m[wave][ln.lane] = sums.top(i);
                if (ln.n == 0) lo_l[wave][ln.g] = sums.l[i];
                __syncthreads();
                // wave w joins channels [w kN, ..) of every run of NJ, for this lane's four rows
                constexpr int kN = NJ >= kW ? NJ / kW : 1;
                if (wave * kN < NJ) {
                    f32x4 m = *reinterpret_cast<const f32x4*>(&lo_m[0][4 * ln.g]);
#pragma unroll
                    for (int w = 1; w < kW; ++w) {
                        const f32x4 v = *reinterpret_cast<const f32x4*>(&lo_m[w][4 * ln.g]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) m[r] = fmaxf(m[r], v[r]);
                    }
                    f32x4 o[kN] = {}, total = {0, 0, 0, 0};
#pragma unroll
                    for (int w = 0; w < kW; ++w) {
                        const f32x4 v = *reinterpret_cast<const f32x4*>(&lo_m[w][4 * ln.g]);
                        f32x4 f;
#pragma unroll
                        for (int r = 0; r < 4; ++r) f[r] = exp2_raw(v[r] - finite_or_zero(m[r]));
                        total += f * lo_l[w][ln.g];
#pragma unroll
                        for (int j = 0; j < kN; ++j) o[j] += f * lo_o[w][wave * kN + j][ln.lane];
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float v[kN];
#pragma unroll
                        for (int j = 0; j < kN; ++j) v[j] = o[j][r];
                        put(v, 16 * i + 4 * ln.g + r, NJ * ln.n + wave * kN, m[r], total[r]);
                    }
                }
            }
        }
        if (u1 == (int)units) {   // the segment ends here
            Record r = {row0, s.first, 0, 0, min(kRows, rows_left), head, {0, 0}};
            if (u0 > 0) {
                const uint32_t edge = more * (share + 1);
                r.from = (int)(seg_begin < edge ? seg_begin / (share + 1) : more + (seg_begin - edge) / share);
                r.to = id;
                cut = r;
            }
            if (by_segment && threadIdx.x == 0) records[segs_before + segment] = r;
        }
        u = seg_begin + u1;
    }
    if (!by_segment && threadIdx.x == 0 && id < record_count) records[id] = cut;
}

constexpr int kJoinWaves = 4;
constexpr int kSpreadRecords = 64;   // 16 segments of 64 parts: a call of 36.7 us instead of 39; 640 of 4: 71.1 instead of 69.4

// Joins the parts of a segment: a wave a row, or, where there are few segments and so many parts of each, a workgroup a row
// (kSpread). Two parts at a time, half a wave each, sixteen of them on their way.
template <int D, int NQ, bool kSpread>
__global__ __launch_bounds__(kJoinWaves * kWave) void attention_join_kernel(Attention a, CacheView c, const float* parts,
                                                                            const Record* records, Divisor by) {
    constexpr int kRows = 16 * NQ;
    constexpr int kEach = D / 32;
    __shared__ float sums[kSpread ? kJoinWaves : 1][kEach + 1][32];
    const Record r = records[blockIdx.x];
    if (r.from == r.to) return;
    const int lane = threadIdx.x % kWave, half = lane / 32, place = lane % 32;
    const int wave = uniform(threadIdx.x / kWave);
    const int count = r.to - r.from + 1;
    const int group = a.heads / c.heads;
    constexpr int kStride = kSpread ? 1 : kJoinWaves;
    for (int at = blockIdx.y * kStride + (kSpread ? 0 : wave); at < r.rows; at += gridDim.y * kStride) {
        auto part_of = [&](int i) { return parts + (2 * (size_t)(r.from + i) + (i == 0 ? 1 : 0)) * part_floats<D, NQ>(); };
        float m = -INFINITY;
        for (int i = lane; i < count; i += kWave) m = fmaxf(m, part_of(i)[(size_t)kRows * D + 2 * at]);
        for (int x = 32; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor(m, x, kWave));
        const float m0 = finite_or_zero(m);
        float total = 0.0f, o[kEach] = {};
        for (int i0 = kSpread ? 16 * wave : 0; i0 < count; i0 += kSpread ? 16 * kJoinWaves : 16) {
            float v[8][kEach], ml[8][2];
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                const float* p = part_of(min(i0 + 2 * b + half, count - 1));
#pragma unroll
                for (int e = 0; e < kEach; ++e) v[b][e] = p[(size_t)at * D + place * kEach + e];
                ml[b][0] = p[(size_t)kRows * D + 2 * at];
                ml[b][1] = p[(size_t)kRows * D + 2 * at + 1];
            }
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                if (i0 + 2 * b + half < count) {
                    const float f = exp2_raw(ml[b][0] - m0);
                    total += f * ml[b][1];
#pragma unroll
                    for (int e = 0; e < kEach; ++e) o[e] += f * v[b][e];
                }
            }
        }
        total += __shfl_xor(total, 32, kWave);
#pragma unroll
        for (int e = 0; e < kEach; ++e) o[e] += __shfl_xor(o[e], 32, kWave);
        if constexpr (kSpread) {
            __syncthreads();   // the row before is done with
            if (half == 0) {
#pragma unroll
                for (int e = 0; e < kEach; ++e) sums[wave][e][place] = o[e];
                sums[wave][kEach][place] = total;
            }
            __syncthreads();
            total = 0.0f;
#pragma unroll
            for (int e = 0; e < kEach; ++e) o[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < kJoinWaves; ++w) {
                total += sums[w][kEach][place];
#pragma unroll
                for (int e = 0; e < kEach; ++e) o[e] += sums[w][e][place];
            }
        }
        const int row = r.row0 + at, q = divide(row, by);
        const int h = r.head * group + (row - q * group);
        const float f = last_factor(m, total, a.sinks, h);
        if (half == 0 && (!kSpread || wave == 0)) {
            uint16_t* out = a.out + ((int64_t)(r.first + q) * a.heads + h) * D + place * kEach;
            if constexpr (kEach == 4)
                *reinterpret_cast<uint2*>(out) = make_uint2(pack_weights(o[0] * f, o[1] * f), pack_weights(o[2] * f, o[3] * f));
            else *reinterpret_cast<uint32_t*>(out) = pack_weights(o[0] * f, o[1] * f);
        }
    }
}

// Many rows: a wave has a tile of its own and goes through all that it sees. Tile groups are taken from the last to the first,
// of a sequence those with the most tokens first, of sequences the last one, whatever its length: packed prompts of 5000, 3334,
// 1667 and 1 tokens 356 us, in the other order 350.
template <int D, int NQ>
__global__ __launch_bounds__(kRowWaves * kWave, 2) void attention_rows_kernel(Attention a, CacheView c, int round, Divisor by) {
    constexpr int NJ = D / 16;
    constexpr int kRows = 16 * NQ;
    const int lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
    const int group = a.heads / c.heads;
    auto weight = [&](const Span& s) { return tiles_of(s, group, kRows * kRowWaves); };
    const Plan plan(a, c.page_bits, lane, weight);
    // rounds of `round` tile groups, one a compute unit and head: every other one backwards, so that a unit that had the
    // longest of one round gets the shortest of the next
    int turn = (int)(blockIdx.x / (uint32_t)c.heads);
    if (const int k = turn / round; k % 2 == 1) turn = k * round + (round - 1 - (turn - k * round));
    const int at = (int)plan.total - 1 - turn;
    if (at < 0 || !plan.ok) return;
    const int head = (int)(blockIdx.x % (uint32_t)c.heads);
    uint32_t begin;
    const int seq = plan.find((uint32_t)at, begin, weight);
    const Span s = plan.span(seq);
    const int row0 = ((at - (int)begin) * kRowWaves + wave) * kRows;
    const int rows_left = s.n * group - row0;
    if (rows_left <= 0) return;
    Sums<D, NQ> sums;
    run_steps<D, NQ>(a, c, a.page_table + seq * a.table_width, s, head, group, by, row0, 0, kFarRight, 1, sums, Lane<D>(lane));
    const Lane<D> ln(not_before(lane));
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = 16 * i + 4 * ln.g + e;
            const float m = __shfl(sums.top(i), 4 * ln.g + e, kWave);
            if (r < rows_left) {
                const int row = row0 + r, q = divide(row, by);
                const int h = head * group + (row - q * group);
                const float f = last_factor(m, sums.l[i][e], a.sinks, h);
                float o[NJ];
#pragma unroll
                for (int j = 0; j < NJ; ++j) o[j] = sums.o[i][j][e] * f;
                store_out<NJ>(a.out + ((int64_t)(s.first + q) * a.heads + h) * D + NJ * ln.n, o);
            }
        }
}

// Tiles of `rows` rows that the sequences of a call can have.
int64_t most_tiles(int64_t tokens, int64_t seqs, int64_t group, int64_t rows) {
    return tokens * group / rows + (seqs < tokens ? seqs : tokens);
}

// How a call is worked on, from what the host knows: the numbers of rows and sequences, and how many tokens a row can see. The
// times below are of 32 query heads over 8 of 128 channels, in us; n: segments of 16 rows. The choice was taken from 70 calls
// (heads of 64 and 128 channels, 1 to 2048 queries, 1 to 256 sequences of 64 to 131072 tokens) timed in every form: it is 1 %
// above the fastest form on the mean, 14 % at most. In all of them the sequences had alike many queries and filled their
// tables. The host knows the mean of the queries and the width of the table only, and where they say little the choice is far
// off: 2048 queries after 6144 tokens beside 30 single ones after 8192 to 131072 go in tiles, each long sequence a wave's alone,
// 2770 us (in two calls 242 + 262); 64 single ones after 1000 take 22.0 with a table of 131072, 17.2 with one of their length.
enum Kind { kRowsForm, kWholeForm, kSplitForm };
struct Form {
    Kind kind;
    int nq;              // tiles of 16 rows a wave takes
    int waves;           // of a worker
    int workers;
    int64_t segments;    // at most
    int join_rows;       // workgroups a segment's rows are joined by
    int records() const { return kind == kSplitForm ? (int)(segments < workers ? segments : workers) : 0; }
};

// Equal shares. Waves of their own where there are segments enough that a worker's share is about one (64 ragged sequences of
// up to 8192: 69.5 against 77.8 in workgroups of four), else workgroups of four, with a quarter of the parts to join (four
// queries after 131072 tokens: 36.2 against 45.3).
Form split_of(int64_t tokens, int64_t seqs, int64_t heads, int64_t kv_heads, int nq) {
    const int64_t group = heads / kv_heads, cus = device_cu_count(), mean = (tokens + seqs - 1) / seqs * group;
    const int64_t segments = most_tiles(tokens, seqs, group, 16 * nq) * kv_heads;
    const int waves = segments >= cus / 2 && nq == 1 ? 1 : 4;
    return {kSplitForm, nq, waves, (int)(8 / waves * cus), segments,
            (int)(((mean < 16 * nq ? mean : 16 * nq) + kJoinWaves - 1) / kJoinWaves)};
}

Form form_of(int64_t tokens, int64_t seqs, int64_t heads, int64_t kv_heads, int64_t head_dim, int64_t length) {
    const int64_t group = heads / kv_heads, cus = device_cu_count();
    const int64_t queries = (tokens + seqs - 1) / seqs, mean = queries * group;
    const int64_t n = seqs * ((mean + 15) / 16) * kv_heads;   // if the sequences have alike many queries
    const int64_t steps = (length + kStep - 1) / kStep;
    const int wide = head_dim == 128 ? 2 : 3;
    // Rows enough to fill the chip twice with two or three tiles a wave: a prompt of 2048 56.7 (one tile a wave 61.5, shares
    // 95), 2048 tokens after 6144 242 (322, 304). With 64 rows a sequence or less half of a workgroup has none (16 queries of
    // 256 sequences: 150, one tile 135).
    // Every workgroup looks for its rows among all sequences, 3 us of 1024: where a tile has less to do than that, the few
    // workgroups of equal shares are better (64 tokens of 64 in 1024 sequences 436, tiles 522; in 256: 107, 100).
    const bool few = seqs <= kWave + 16 * steps;
    if (few && mean > 64 && most_tiles(tokens, seqs, group, 16 * wide * kRowWaves) * kv_heads >= 2 * cus)
        return {kRowsForm, wide, 0, 0, 0, 0};
    // One tile a wave. Few segments and tokens: one token of 64 sequences of 192 8.4 (four waves a segment 10.2), of 16: 7.6
    // (7.6). Many of both, as long as the chain of steps is short beside the number of tiles: the last 1024 of 4096 tokens 88
    // (shares 92.7), 512 after 1700 42.5 (35.8).
    if (n <= 2 * cus ? steps <= (n <= cus ? 5 : 12) : few && mean >= 48 && 16 * steps <= n) return {kRowsForm, 1, 0, 0, 0, 0};
    // Whole segments save the join, its launch and the parts' way through memory. With no more than two a compute unit all
    // are under way at once: one token after 1000 in 64 sequences 17.7 (shares 28.1), of 2048 in 16 15.5 in eight waves (16.2
    // in four, 16.9), of 2048 alone 14.2 (11.1: its eight segments leave the chip idle, which the estimates say, in 0.1 us). A
    // segment longer than the others keeps the call waiting, so chains longer than 32 steps are cut (64 sequences of 4352:
    // 63.5, whole 57). Of more segments, each a wave's: one token after 384 in 200 sequences 20.1 (30.8), 8 queries after 1000
    // in 256 84.7 (92.7), one token after 64 in 256 11.1 (13.2), in 1024 49.7 (32.8).
    Form f = split_of(tokens, seqs, heads, kv_heads, 1);
    auto whole = [&](int waves) {
        f.kind = kWholeForm;
        f.waves = waves;
        f.workers = (int)f.segments;
        return f;
    };
    if (n <= 2 * cus) {
        const int waves = n <= cus && steps > 32 ? 8 : 4;
        const int64_t chain = (steps + waves - 1) / waves;
        const int64_t as_whole = waves == 8 ? 93 + 7 * chain : 66 + 6 * chain;
        const int64_t as_shares = 110 + 50 * (n < 64 ? n : 64) / 64 + 7 * n * steps / (8 * cus);
        if (chain <= 32 && as_whole < as_shares) return whole(waves);
    } else if (mean < 48 && steps <= 32 && seqs <= 4 * kWave) {
        return whole(1);
    }
    // Two tiles share their tokens' bytes, and pay for it once a worker, with more to set up and to join: 512 tokens after
    // 15872 154 (one tile 201), 8 queries of 4 sequences of 16384 30.2 (27.5), 16 of 64 of 300 33.9 (21.5).
    if (mean > 16 && steps >= 64 && seqs * ((mean + 31) / 32) * kv_heads * steps >= 9 * 8 * cus)
        return split_of(tokens, seqs, heads, kv_heads, 2);
    return f;
}

size_t bytes_of(const Form& f, int64_t head_dim) {
    return f.records() * sizeof(Record) + (size_t)f.workers * 2 * 16 * f.nq * (head_dim + 2) * sizeof(float);
}

template <int D, int NQ, int kW>
hipError_t split_form(const Attention& a, const CacheView& c, const Form& f, void* workspace, hipStream_t stream) {
    Record* records = f.kind == kSplitForm ? static_cast<Record*>(workspace) : nullptr;
    float* parts = reinterpret_cast<float*>(records + f.records());
    // one step, more where the number of units would not fit 32 bits: the segments of 2^28 rows are fewer than 2^29
    int unit_bits = f.kind == kSplitForm ? 5 : 30;
    while (f.segments > ((int64_t)1 << 30) / (((a.table_width << c.page_bits) >> unit_bits) + 2)) ++unit_bits;
    attention_split_kernel<D, NQ, kW><<<f.workers, kW * kWave, 0, stream>>>(a, c, parts, records, f.workers, unit_bits,
                                                                            f.records(),
                                                                            records && f.segments <= f.workers,
                                                                            divisor_of(a.heads / c.heads));
    if (hipError_t e = hipGetLastError(); e != hipSuccess || !records) return e;
    const Divisor by = divisor_of(a.heads / c.heads);
    const int threads = kJoinWaves * kWave;
    if (f.records() <= kSpreadRecords)
        attention_join_kernel<D, NQ, true><<<dim3(f.records(), 16 * NQ), threads, 0, stream>>>(a, c, parts, records, by);
    else
        attention_join_kernel<D, NQ, false><<<dim3(f.records(), f.join_rows), threads, 0, stream>>>(a, c, parts, records, by);
    return hipGetLastError();
}

template <int D, int NQ>
hipError_t rows_form(const Attention& a, const CacheView& c, hipStream_t stream) {
    const int round = device_cu_count() > c.heads ? device_cu_count() / c.heads : 1;
    const int64_t tiles = most_tiles(a.tokens, a.seqs, a.heads / c.heads, 16 * NQ * kRowWaves);
    // whole rounds: see the kernel's order. Of 2^28 rows, with 48 or more a sequence: under 2^24 workgroups (a launch may
    // have 2^32 threads), at most 2^28 / 64 + 2^28 / 24 + 4096
    const int64_t grid = (tiles + round - 1) / round * round * c.heads;
    attention_rows_kernel<D, NQ><<<(unsigned)grid, kRowWaves * kWave, 0, stream>>>(a, c, round, divisor_of(a.heads / c.heads));
    return hipGetLastError();
}

template <int D>
hipError_t attend(const Attention& a, const CacheView& c, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const int64_t most = a.table_width << c.page_bits, seen = a.window + (a.tokens + a.seqs - 1) / a.seqs;
    const Form f = form_of(a.tokens, a.seqs, a.heads, c.heads, D, a.window > 0 && seen < most ? seen : most);
    if (f.kind == kSplitForm && bytes_of(f, D) > workspace_bytes) return hipErrorInvalidValue;
    if (f.kind == kRowsForm)
        return f.nq == 1 ? rows_form<D, 1>(a, c, stream) : rows_form<D, (D == 128 ? 2 : 3)>(a, c, stream);
    if (f.nq == 2) return split_form<D, 2, 4>(a, c, f, workspace, stream);
    if (f.waves == 1) return split_form<D, 1, 1>(a, c, f, workspace, stream);
    if (f.waves == 4) return split_form<D, 1, 4>(a, c, f, workspace, stream);
    return split_form<D, 1, 8>(a, c, f, workspace, stream);
}

}  // namespace

// For any length: the form depends on it, and the bytes of the shares with it.
size_t attention_workspace_bytes(int64_t tokens, int64_t seqs, int64_t heads, int64_t kv_heads, int64_t head_dim) {
    if (seqs <= kWave && form_of(tokens, seqs, heads, kv_heads, head_dim, 1).nq >= 2) return 0;   // wide rows whatever the length
    const size_t one = bytes_of(split_of(tokens, seqs, heads, kv_heads, 1), head_dim);
    const size_t two = bytes_of(split_of(tokens, seqs, heads, kv_heads, 2), head_dim);
    return one > two ? one : two;
}

hipError_t launch_attention(const Attention& a, const CacheView& c, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
    return c.head_dim == 128 ? attend<128>(a, c, workspace, workspace_bytes, stream)
                             : attend<64>(a, c, workspace, workspace_bytes, stream);
}

}  // namespace e2m1

extern "C" int e2m1_mxfp4_attention_form(int64_t tokens, int64_t seqs, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                         int64_t length) {
    const e2m1::Form f = e2m1::form_of(tokens, seqs, heads, kv_heads, head_dim, length);
    const bool by_worker = f.kind == e2m1::kSplitForm && f.segments > f.workers;
    const bool spread = f.kind == e2m1::kSplitForm && f.records() <= e2m1::kSpreadRecords;
    return 1000 * (spread ? 2 : by_worker ? 1 : 0) + 100 * f.kind + 10 * f.nq + f.waves;
}
