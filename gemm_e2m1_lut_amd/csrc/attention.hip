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
//     bytes as its scales, so keys are never decoded. Queries are the B operand,
//     as a sum of three E2M3 (6-bit) parts with block scales 2^e, 2^(e-4),
//     2^(e-10): a bf16 number has 8 significant bits, three parts keep every
//     element to 2^-16 of its block's largest (the second part alone leaves
//     2^-10). 4- and 6-bit operands run at twice the rate of 8-bit ones, so the three
//     products take 3/4 of the time of bf16 keys, and no key is unpacked. (Two E4M3 parts
//     would do too, at the rate of four E2M3 ones.) Heads of 64 channels fill half of the
//     instruction's 128: the other half takes the second part of the same keys.
//   * The scores come out transposed (a lane has 4 tokens of one query row), which
//     is what the values' product takes as its B operand: the weights never
//     leave their lane. Its A operand is the values transposed, 8 tokens of a
//     channel a lane: a lane loads the codes of 8 channels of its 8 tokens,
//     v_cvt_scalef32_pk_bf16_fp4 decodes pairs of channels with the token's scale
//     and v_perm_b32 pairs the tokens. One operation an element, for all NQ tiles.
//   * A maximum is replaced only when a score passes it by 2^8 (a vote per step):
//     weights are then at most 2^8, the sums fp32, and the usual step has no
//     exchange between lanes and no rescaling.
// Weights are rounded to bf16 for the matrix cores (half a step is 2^-8 of a weight, and the
// errors of a row's weights are independent: the result's own rounding is larger).
// No LDS and no barrier in the loop: the bytes of a step are few (4352 for 32
// tokens of 128 channels), and waves that share tokens find them in the L1.
#include "device.hpp"
#include "kernels.hpp"

namespace e2m1 {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kWaves = 4;          // of a workgroup
constexpr int kStep = 32;          // tokens a wave takes at a time
constexpr int kUnit = kWaves * kStep;
constexpr float kSlack = 8.0f;     // how far a score may pass the maximum in use, in powers of two
constexpr int kFarRight = 0x7FFFFFFF;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x6 __attribute__((ext_vector_type(6)));
typedef __bf16 bf16x32 __attribute__((ext_vector_type(32)));

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

// ------------------------------------------------------------------- plan --

// What a sequence asks for.
struct Span {
    int64_t first;   // its first query row
    int n;           // queries
    int len;         // cached tokens
};

__device__ __forceinline__ Span span_of(const Attention& a, int page_bits, int64_t s) {
    const int64_t o0 = a.q_offsets[s], o1 = a.q_offsets[s + 1];
    Span r;
    r.first = min(max(o0, (int64_t)0), a.tokens);
    r.n = (int)(min(max(o1, r.first), a.tokens) - r.first);
    const int64_t most = a.table_width << page_bits;
    const int64_t len = a.kv_lens[s];
    r.len = (int)min(max(len, (int64_t)0), most);
    if (len > most && r.n > 0 && a.err_flag) *a.err_flag = 1;
    return r;
}

// The first token that some query of [i0, ..) sees.
__device__ __forceinline__ int first_seen(const Attention& a, const Span& s, int i0) {
    return a.window > 0 ? (int)max((int64_t)0, (int64_t)s.len - s.n + i0 - a.window + 1) : 0;
}

// Units of kUnit tokens of every tile of a sequence.
__device__ __forceinline__ int units_of(const Attention& a, const Span& s) {
    const int lo = first_seen(a, s, 0) & ~(kStep - 1);
    return max(1, (s.len - lo + kUnit - 1) / kUnit);
}

__device__ __forceinline__ int64_t scan64(int64_t v, int lane) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int64_t o = __shfl_up((long long)v, d, kWave);
        if (lane >= d) v += o;
    }
    return v;
}

__device__ __forceinline__ int64_t uniform64(int64_t v, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// Sequences laid end to end by weight: each lane sums a run of them, a scan over the wave gives the runs' places.
template <typename F>
struct Layout {
    F weight;
    int64_t seqs, per, before, total;
    int lane;

    __device__ __forceinline__ Layout(F f, int64_t n, int lane_) : weight(f), seqs(n), lane(lane_) {
        per = (n + kWave - 1) / kWave;
        int64_t sum = 0;
        for (int64_t s = lane * per; s < min((lane + 1) * per, n); ++s) sum += weight(s);
        const int64_t end = scan64(sum, lane);
        before = end - sum;
        total = uniform64(end, kWave - 1);
        after = end;
    }
    int64_t after;

    // The sequence that holds place `at` < total, and where it begins.
    __device__ __forceinline__ void find(int64_t at, int64_t& seq, int64_t& begin) const {
        const uint64_t mine = __ballot(at >= before && at < after);
        const int owner = __builtin_ctzll(mine);
        int64_t s = lane * per, b = before;
        if (lane == owner) {
            for (;;) {
                const int64_t w = weight(s);
                if (at < b + w) break;
                b += w;
                ++s;
            }
        }
        seq = uniform64(s, owner);
        begin = uniform64(b, owner);
    }
};

// ------------------------------------------------------------------- step --

// The bytes of 32 tokens of a kv head, as loaded.
template <int D>
struct Stage {
    u32x4 k[2];       // 16 bytes of token lane % 16 of each half
    uint32_t ks[2];   // its scale byte
    uint32_t v[8];    // D / 16 codes each of tokens 4 g + r and 16 + 4 g + r
    uint32_t vs[2][D / 32];   // the scale bytes of these four tokens
    bool ok[2];       // whether the half holds tokens (uniform)
};

// A wave's rows.
template <int NQ>
struct Rows {
    i32x8 q[NQ][3];       // the parts of 32 channels of row lane % 16
    uint32_t qs[NQ];      // their scale bytes, one a part
    int lo[NQ], hi[NQ];   // the tokens that the lane's row sees
    int lo_all, hi_all;   // the tokens that some row sees
    int lo_max, hi_min;   // the tokens that every row sees
};

template <int D, int NQ>
struct Sums {
    f32x4 o[NQ][D / 16];
    float m[NQ], l[NQ];   // l: of the lane's own tokens
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[i][j] = f32x4{0, 0, 0, 0};
        }
    }
};

// Lane constants of the loads.
template <int D>
struct Lane {
    int n, g;
    uint32_t k, ks, v, vs;   // byte offsets in a run of 16 tokens
    uint32_t turn;           // rotation that brings the scale of the lane's channels to an exponent field
    __device__ __forceinline__ explicit Lane(int lane) {
        n = lane % 16;
        g = lane / 16;
        const int block = D == 128 ? g : g & 1;
        k = n * (D / 2) + block * 16;
        ks = n * (D / 32) + block;
        v = 4 * g * (D / 2) + n * (D / 32);
        vs = 4 * g * (D / 32);
        turn = 8 * (n * (D / 16) / 32) + 9;
    }
};

// First row (of the cache's [pages, heads, page]) of the 16 tokens from tb on; ok: they exist and some row sees them.
template <int NQ>
__device__ __forceinline__ int64_t half_row(const Attention& a, const CacheView& c, const int32_t* table, int head, int tb,
                                            int lo_all, int hi_all, bool& ok) {
    const bool in = tb < hi_all && tb + 16 > lo_all;
    const int at = in ? tb : 0;
    int pg = hi_all > lo_all ? uniform(table[at >> c.page_bits]) : 0;
    const bool there = pg >= 0 && ((int64_t)pg << c.page_bits) < c.slots;
    if (in && !there && a.err_flag) *a.err_flag = 1;
    ok = in && there;
    return ok ? ((((int64_t)pg * c.heads + head) << c.page_bits) + (at & ((1 << c.page_bits) - 1))) : 0;
}

template <int D, int NQ>
__device__ __forceinline__ void load_step(Stage<D>& s, const Attention& a, const CacheView& c, const int32_t* table,
                                          int head, int base, const Rows<NQ>& rows, const Lane<D>& ln) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int64_t row = half_row<NQ>(a, c, table, head, base + 16 * t, rows.lo_all, rows.hi_all, s.ok[t]);
        const uint8_t* kc = c.k_codes + row * (D / 2);
        const uint8_t* kx = c.k_scales + row * (D / 32);
        const uint8_t* vc = c.v_codes + row * (D / 2);
        const uint8_t* vx = c.v_scales + row * (D / 32);
        s.k[t] = *reinterpret_cast<const u32x4*>(kc + ln.k);
        s.ks[t] = kx[ln.ks];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if constexpr (D == 128) s.v[4 * t + r] = *reinterpret_cast<const uint32_t*>(vc + ln.v + r * 64);
            else s.v[4 * t + r] = *reinterpret_cast<const uint16_t*>(vc + ln.v + r * 32);
        }
        if constexpr (D == 128) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(vx + ln.vs);
#pragma unroll
            for (int r = 0; r < 4; ++r) s.vs[t][r] = w[r];
        } else {
            const u32x2 w = *reinterpret_cast<const u32x2*>(vx + ln.vs);
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
__device__ __forceinline__ void clear_token(Stage<D>& s, int t, int r, bool clear) {
    s.v[4 * t + r] = clear ? 0u : s.v[4 * t + r];
    if constexpr (D == 128) s.vs[t][r] = clear ? 0u : s.vs[t][r];
    else s.vs[t][r / 2] &= clear ? (r % 2 ? 0x0000FFFFu : 0xFFFF0000u) : 0xFFFFFFFFu;
}

__device__ __forceinline__ uint32_t pack_weights(float a, float b) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    const f2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

template <int D, int NQ>
__device__ __forceinline__ void take_step(Stage<D>& s, const Rows<NQ>& rows, Sums<D, NQ>& sums, float scale, int base,
                                          const Lane<D>& ln) {
    constexpr int NJ = D / 16;
    // scores of 2 x 16 tokens
    f32x4 x[NQ][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const i32x8 k = {(int)s.k[t].x, (int)s.k[t].y, (int)s.k[t].z, (int)s.k[t].w, 0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            f32x4 z = {0, 0, 0, 0};
            z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, rows.q[i][0], z, 4, 2, 0, s.ks[t], 0, rows.qs[i]);
            z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, rows.q[i][1], z, 4, 2, 0, s.ks[t], 1, rows.qs[i]);
            if constexpr (D == 128)
                z = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(k, rows.q[i][2], z, 4, 2, 0, s.ks[t], 2, rows.qs[i]);
            x[i][t] = z;
        }
    }
    const int j0 = base + 4 * ln.g;
    const bool edge = base < rows.lo_max || base + kStep > rows.hi_min || !(s.ok[0] && s.ok[1]);
    if (edge) {   // tokens that no row sees: values that stay finite whatever is there
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = j0 + 16 * t + r;
                clear_token<D>(s, t, r, !(s.ok[t] && j >= rows.lo_all && j < rows.hi_all));
            }
    }
    // A value's scale byte past 252: its token turns NaN in the scores, its values are left out. Bytes from 192 on are rare
    // enough to be looked at one by one.
    uint32_t high = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < D / 32; ++i) high |= s.vs[t][i] & (s.vs[t][i] << 1);
    if (__builtin_expect(__any((high & 0x80808080u) != 0), 0)) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t w = scale_bytes<D>(s.vs[t], r);
                bool bad = false;
#pragma unroll
                for (int b = 0; b < D / 32; ++b) bad |= ((w >> (8 * b)) & 255u) > 252u;
#pragma unroll
                for (int i = 0; i < NQ; ++i) x[i][t][r] = bad ? __uint_as_float(0x7FC00000u) : x[i][t][r];
                clear_token<D>(s, t, r, bad);
            }
    }
    if (edge) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = j0 + 16 * t + r;
#pragma unroll
                for (int i = 0; i < NQ; ++i)
                    x[i][t][r] = s.ok[t] && j >= rows.lo[i] && j < rows.hi[i] ? x[i][t][r] : -INFINITY;
            }
    }
    // maxima
    bool past = false;
    float top[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        top[i] = fmaxf(fmaxf(fmaxf(x[i][0][0], x[i][0][1]), fmaxf(x[i][0][2], x[i][0][3])),
                       fmaxf(fmaxf(x[i][1][0], x[i][1][1]), fmaxf(x[i][1][2], x[i][1][3]))) * scale;
        past |= top[i] > sums.m[i] + kSlack;
    }
    if (__any(past)) {
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            float v = fmaxf(top[i], __shfl_xor(top[i], 16, kWave));
            v = fmaxf(v, __shfl_xor(v, 32, kWave));
            const float mn = fmaxf(sums.m[i], v);
            const float f = mn == -INFINITY ? 1.0f : exp2_raw(sums.m[i] - mn);
            sums.m[i] = mn;
            sums.l[i] *= f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) sums.o[i][j] *= f;
        }
    }
    // weights
    bf16x8 p[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const float m = sums.m[i] == -INFINITY ? 0.0f : sums.m[i];
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = exp2_raw(__builtin_fmaf(x[i][e / 4][e % 4], scale, -m));
        sums.l[i] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
        const u32x4 pk = {pack_weights(w[0], w[1]), pack_weights(w[2], w[3]), pack_weights(w[4], w[5]),
                          pack_weights(w[6], w[7])};
        p[i] = __builtin_bit_cast(bf16x8, pk);
    }
    // values: a byte (two channels) of all eight tokens at a time
    float sc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t w = D == 128 ? s.vs[e / 4][e % 4] : s.vs[e / 4][(e % 4) / 2];
        sc[e] = __uint_as_float(__builtin_amdgcn_alignbit(w, w, D == 128 ? ln.turn : ln.turn + 16 * (e % 2)));
    }
#pragma unroll
    for (int b = 0; b < NJ / 2; ++b) {
        uint32_t d[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            bf16x2 v;
            if (b == 0) v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.v[e], sc[e], 0);
            else if (b == 1) v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.v[e], sc[e], 1);
            else if (b == 2) v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.v[e], sc[e], 2);
            else v = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(s.v[e], sc[e], 3);
            d[e] = __builtin_bit_cast(uint32_t, v);
        }
        u32x4 even, odd;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            even[e] = __builtin_amdgcn_perm(d[2 * e + 1], d[2 * e], 0x05040100u);
            odd[e] = __builtin_amdgcn_perm(d[2 * e + 1], d[2 * e], 0x07060302u);
        }
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            sums.o[i][2 * b] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, even), p[i], sums.o[i][2 * b], 0, 0, 0);
            sums.o[i][2 * b + 1] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, odd), p[i], sums.o[i][2 * b + 1], 0, 0, 0);
        }
    }
}

// ---------------------------------------------------------------- queries --

// x - y of bf16 pairs, exact where the difference fits bf16.
__device__ __forceinline__ bf16x32 difference(const bf16x32& x, const bf16x32& y) {
    typedef uint32_t u32x16 __attribute__((ext_vector_type(16)));
    const u32x16 a = __builtin_bit_cast(u32x16, x), b = __builtin_bit_cast(u32x16, y);
    u32x16 d;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float lo = __uint_as_float(a[i] << 16) - __uint_as_float(b[i] << 16);
        const float hi = __uint_as_float(a[i] & 0xFFFF0000u) - __uint_as_float(b[i] & 0xFFFF0000u);
        d[i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
    }
    return __builtin_bit_cast(bf16x32, d);
}

__device__ __forceinline__ i32x8 widen(const u32x6& v) {
    return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], (int)v[4], (int)v[5], 0, 0};
}

// The three parts of a lane's 32 channels. Their largest magnitude lies in [4, 8) of the first part's unit 2^e, so the
// first part leaves at most 1/2, the second, in units of 2^(e-4), at most 2^-8, the third, in 2^(e-10), 2^-14. Each
// remainder has at most the 8 significant bits it started with. A block that holds a NaN or an infinity gets the scale NaN.
template <int D>
__device__ __forceinline__ void split_query(const u32x4 (&w)[4], int g, i32x8 (&q)[3], uint32_t& scales) {
    typedef uint32_t u32x16 __attribute__((ext_vector_type(16)));
    u32x16 a;
    u16x2 top = {0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        a[i] = w[i / 4][i % 4];
        top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, a[i] & 0x7FFF7FFFu));
    }
    const uint32_t field = max((uint32_t)top.x, (uint32_t)top.y) >> 7;
    const uint32_t e = max(field, 12u) - 2u;
    const bf16x32 x = __builtin_bit_cast(bf16x32, a);
    const float s0 = __uint_as_float(e << 23), s1 = __uint_as_float((e - 4u) << 23), s2 = __uint_as_float((e - 10u) << 23);
    const u32x6 p0 = __builtin_amdgcn_cvt_scalef32_pk32_fp6_bf16(x, s0);
    const bf16x32 r0 = difference(x, __builtin_amdgcn_cvt_scalef32_pk32_bf16_fp6(p0, s0));
    const u32x6 p1 = __builtin_amdgcn_cvt_scalef32_pk32_fp6_bf16(r0, s1);
    const bf16x32 r1 = difference(r0, __builtin_amdgcn_cvt_scalef32_pk32_bf16_fp6(p1, s1));
    const u32x6 p2 = __builtin_amdgcn_cvt_scalef32_pk32_fp6_bf16(r1, s2);
    if constexpr (D == 128) {
        q[0] = widen(p0);
        q[1] = widen(p1);
        q[2] = widen(p2);
        scales = e | (e - 4u) << 8 | (e - 10u) << 16;
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
        scales = (up ? e - 4u : e) | (e - 10u) << 8;
    }
    if (field == 255u) scales = 0xFFFFFFFFu;
}

// The rows [row0, row0 + 16 NQ) of a sequence's (query, head of the group) pairs; rows past the last one see what it sees.
template <int D, int NQ>
__device__ __forceinline__ void set_ranges(Rows<NQ>& rows, const Attention& a, const Span& s, int group, int64_t row0,
                                           const Lane<D>& ln) {
    const int64_t last = (int64_t)s.n * group - 1;
    const int i_first = (int)(row0 / group), i_last = (int)(min(row0 + 16 * NQ - 1, last) / group);
    const int p0 = s.len - s.n;   // position of query 0
    if (a.causal) {
        rows.lo_all = first_seen(a, s, i_first);
        rows.lo_max = first_seen(a, s, i_last);
        rows.hi_all = max(0, p0 + i_last + 1);
        rows.hi_min = max(0, p0 + i_first + 1);
    } else {
        rows.lo_all = rows.lo_max = 0;
        rows.hi_all = rows.hi_min = s.len;
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int q = (int)(min(row0 + 16 * i + ln.n, last) / group);
        rows.lo[i] = a.causal ? first_seen(a, s, q) : 0;
        rows.hi[i] = a.causal ? max(0, p0 + q + 1) : s.len;
    }
}

template <int D, int NQ>
__device__ __forceinline__ void load_queries(Rows<NQ>& rows, const Attention& a, const Span& s, int kv_head, int group,
                                             int64_t row0, const Lane<D>& ln) {
    const int64_t last = (int64_t)s.n * group - 1;
    const int block = D == 128 ? ln.g : ln.g & 1;
    u32x4 w[NQ][4];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int64_t row = min(row0 + 16 * i + ln.n, last);
        const int64_t q = row / group;
        const uint16_t* p = a.q + (s.first + q) * a.q_stride + ((int64_t)kv_head * group + (row - q * group)) * D + block * 32;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            w[i][b] = *reinterpret_cast<const u32x4*>(p + 8 * b);
            if (a.scale == 0.0f) w[i][b] = u32x4{0, 0, 0, 0};
        }
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) split_query<D>(w[i], ln.g, rows.q[i], rows.qs[i]);
}

// Steps first, first + stride, .. below `last` of a wave's rows: the next step's bytes are on their way while one is worked on.
template <int D, int NQ>
__device__ __forceinline__ void run_steps(const Attention& a, const CacheView& c, const int32_t* table, const Span& s,
                                          int kv_head, int group, int64_t row0, int first, int last, int stride,
                                          Sums<D, NQ>& sums, const Lane<D>& ln) {
    Rows<NQ> rows;
    set_ranges<D, NQ>(rows, a, s, group, row0, ln);
    sums.clear();
    if (c.slots == 0) return;   // no page is there
    // 0 has to leave a masked score's -infinity alone: the queries become zeros instead
    const float scale = a.scale > 0.0f ? a.scale * kLog2e : 1.0f;
    // steps with a token that some row sees
    first = max(first, 0);
    int at = first;
    const int low = rows.lo_all / kStep;
    if (at < low) at += (low - at + stride - 1) / stride * stride;
    const int end = min(last, (rows.hi_all + kStep - 1) / kStep);
    if (at >= end) return;
    Stage<D> st[2];
    load_step<D, NQ>(st[0], a, c, table, kv_head, at * kStep, rows, ln);
    load_queries<D, NQ>(rows, a, s, kv_head, group, row0, ln);
    for (;;) {
        if (at + stride < end) load_step<D, NQ>(st[1], a, c, table, kv_head, (at + stride) * kStep, rows, ln);
        take_step<D, NQ>(st[0], rows, sums, scale, at * kStep, ln);
        at += stride;
        if (at >= end) break;
        if (at + stride < end) load_step<D, NQ>(st[0], a, c, table, kv_head, (at + stride) * kStep, rows, ln);
        take_step<D, NQ>(st[1], rows, sums, scale, at * kStep, ln);
        at += stride;
        if (at >= end) break;
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
        l = l * f + exp2_raw(s - mn);
    }
    return l == 0.0f ? 0.0f : f / l;
}

template <int NJ>
__device__ __forceinline__ void store_out(uint16_t* p, const float (&v)[NJ]) {
    uint32_t w[NJ / 2];
#pragma unroll
    for (int j = 0; j < NJ / 2; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
    if constexpr (NJ == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// A worker's place in the workspace: two partial results (of the segment it begins in and of the one it ends in), each
// 16 NQ rows of D sums, maximum and total; then a record for the joining kernel.
struct Record {
    int64_t row0, first;    // rows of the sequence, its first query
    int from, rows, head;   // from: the worker whose second part is the first one; -1: nothing to join
    int pad;
};

template <int D, int NQ>
constexpr size_t part_floats() { return (size_t)16 * NQ * (D + 2); }

// Split form: workers take equal shares of all units (kUnit tokens of a tile), in a row; the waves of one take every
// fourth step of its share and join in LDS.
template <int D, int NQ>
__global__ __launch_bounds__(kWaves * kWave) void attention_split_kernel(Attention a, CacheView c, float* parts,
                                                                         Record* records, int workers) {
    constexpr int NJ = D / 16;
    constexpr int kRows = 16 * NQ;
    __shared__ float lo_o[kWaves][4 * NJ][kWave];
    __shared__ float lo_ml[kWaves][16][2];
    const int lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
    // neighbours in the order of work on the same XCD, whose L2 then holds what they share
    const int per_xcd = workers / 8;
    const int id = (int)blockIdx.x < per_xcd * 8 ? (int)(blockIdx.x % 8) * per_xcd + (int)blockIdx.x / 8 : (int)blockIdx.x;
    const int group = a.heads / c.heads;
    const Lane<D> ln(lane);

    auto weight = [&](int64_t s) -> int64_t {
        const Span sp = span_of(a, c.page_bits, s);
        const int64_t tiles = ((int64_t)sp.n * group + kRows - 1) / kRows;
        return tiles * c.heads * units_of(a, sp);
    };
    const Layout<decltype(weight)> plan(weight, a.seqs, lane);
    const int64_t share = plan.total / workers, more = plan.total - share * workers;
    int64_t u = id * share + min((int64_t)id, more);
    const int64_t u_end = u + share + (id < more ? 1 : 0);
    if (u >= u_end) {
        if (threadIdx.x == 0) records[id].from = -1;
        return;
    }
    const int64_t u_begin = u;
    int64_t seq, begin;
    plan.find(u, seq, begin);
    Span s = span_of(a, c.page_bits, seq);
    s.first = uniform64(s.first, 0);
    s.n = uniform(s.n);
    s.len = uniform(s.len);
    int units = units_of(a, s);
    int64_t tiles = ((int64_t)s.n * group + kRows - 1) / kRows;
    int from = -1;
    Record rec = {0, 0, -1, 0, 0, 0};
    while (u < u_end) {
        while (u >= begin + tiles * c.heads * units) {   // on to the next sequence that has queries
            begin += tiles * c.heads * units;
            ++seq;
            s = span_of(a, c.page_bits, seq);
            s.first = uniform64(s.first, 0);
            s.n = uniform(s.n);
            s.len = uniform(s.len);
            units = units_of(a, s);
            tiles = ((int64_t)s.n * group + kRows - 1) / kRows;
        }
        const int64_t segment = (u - begin) / units;
        const int64_t seg_begin = begin + segment * units;
        const int u0 = (int)(u - seg_begin);
        const int u1 = (int)min((int64_t)units, u_end - seg_begin);
        const int head = (int)(segment / tiles);
        const int64_t row0 = (segment - head * tiles) * kRows;
        const int origin = (first_seen(a, s, 0) & ~(kStep - 1)) / kStep;
        Sums<D, NQ> sums;
        run_steps<D, NQ>(a, c, a.page_table + seq * a.table_width, s, head, group, row0, origin + u0 * kWaves + wave,
                         origin + u1 * kWaves, kWaves, sums, ln);
        const bool whole = u0 == 0 && u1 == units;
        const bool goes_on = u0 > 0;   // the segment's start is another worker's
        float* part = parts + (2 * (size_t)id + (goes_on ? 0 : 1)) * part_floats<D, NQ>();
        const int64_t rows_left = (int64_t)s.n * group - row0;
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            if (16 * i >= rows_left) break;
            float l = sums.l[i];
            l += __shfl_xor(l, 16, kWave);
            l += __shfl_xor(l, 32, kWave);
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) lo_o[wave][r * NJ + j][lane] = sums.o[i][j][r];
            if (lane < 16) {
                lo_ml[wave][lane][0] = sums.m[i];
                lo_ml[wave][lane][1] = l;
            }
            __syncthreads();
            float m = lo_ml[0][ln.n][0];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) m = fmaxf(m, lo_ml[w][ln.n][0]);
            const float m0 = finite_or_zero(m);
            float o[NJ] = {}, total = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float f = exp2_raw(lo_ml[w][ln.n][0] - m0);
                total += f * lo_ml[w][ln.n][1];
#pragma unroll
                for (int j = 0; j < NJ; ++j) o[j] += f * lo_o[w][wave * NJ + j][lane];
            }
            const int at = 16 * i + ln.n;
            const int d = NJ * (4 * ln.g + wave);   // this lane's channels of row `at`
            if (at < rows_left) {
                if (whole) {
                    const int64_t row = row0 + at, q = row / group;
                    const int h = head * group + (int)(row - q * group);
                    const float f = last_factor(m, total, a.sinks, h);
#pragma unroll
                    for (int j = 0; j < NJ; ++j) o[j] *= f;
                    store_out<NJ>(a.out + ((s.first + q) * a.heads + h) * D + d, o);
                } else {
#pragma unroll
                    for (int j = 0; j < NJ; j += 4)
                        *reinterpret_cast<f32x4*>(part + (size_t)at * D + d + j) = f32x4{o[j], o[j + 1], o[j + 2], o[j + 3]};
                    if (ln.g == 0 && wave == 0) {
                        part[(size_t)kRows * D + 2 * at] = m;
                        part[(size_t)kRows * D + 2 * at + 1] = total;
                    }
                }
            }
        }
        if (goes_on && u1 == units) {   // its last part: this worker's record names the join
            const int64_t edge = more * (share + 1);
            from = (int)(seg_begin < edge ? seg_begin / (share + 1) : more + (seg_begin - edge) / share);
            rec = {row0, s.first, from, (int)min((int64_t)kRows, rows_left), head, 0};
        }
        u = seg_begin + u1;
    }
    (void)u_begin;
    if (threadIdx.x == 0) records[id] = rec;
}

// Joins the parts of the segment that worker blockIdx.x ended: the second part of worker `from`, the first ones of the
// workers after it. A wave a row.
template <int D, int NQ>
__global__ __launch_bounds__(kWaves * kWave) void attention_join_kernel(Attention a, CacheView c, const float* parts,
                                                                        const Record* records) {
    constexpr int kRows = 16 * NQ;
    constexpr int kEach = D / kWave;
    const Record r = records[blockIdx.x];
    if (r.from < 0) return;
    const int lane = threadIdx.x % kWave;
    const int count = (int)blockIdx.x - r.from + 1;
    const int group = a.heads / c.heads;
    for (int at = blockIdx.y * kWaves + threadIdx.x / kWave; at < r.rows; at += gridDim.y * kWaves) {
        auto part_of = [&](int i) { return parts + (2 * (size_t)(r.from + i) + (i == 0 ? 1 : 0)) * part_floats<D, NQ>(); };
        float m = -INFINITY;
        for (int i = lane; i < count; i += kWave) m = fmaxf(m, part_of(i)[(size_t)kRows * D + 2 * at]);
        for (int x = 32; x > 0; x >>= 1) m = fmaxf(m, __shfl_xor(m, x, kWave));
        const float m0 = finite_or_zero(m);
        float total = 0.0f, o[kEach] = {};
        for (int i0 = 0; i0 < count; i0 += kWave) {
            float f = 0.0f;
            if (i0 + lane < count) {
                const float* ml = part_of(i0 + lane) + (size_t)kRows * D + 2 * at;
                f = exp2_raw(ml[0] - m0);
                total += f * ml[1];
            }
            const int here = min(kWave, count - i0);
#pragma unroll 8
            for (int i = 0; i < here; ++i) {
                const float* p = part_of(i0 + i) + (size_t)at * D + lane * kEach;
                const float w = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(f), i));
#pragma unroll
                for (int e = 0; e < kEach; ++e) o[e] += w * p[e];
            }
        }
        total = group_sum<kWave>(total);
        const int64_t row = r.row0 + at, q = row / group;
        const int h = r.head * group + (int)(row - q * group);
        const float f = last_factor(m, total, a.sinks, h);
        uint16_t* out = a.out + ((r.first + q) * a.heads + h) * D + lane * kEach;
        if constexpr (kEach == 2) *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(o[0] * f, o[1] * f);
        else *out = (uint16_t)f32_to_bf16_rne(o[0] * f);
    }
}

// Many rows: a wave has a tile of its own and goes through all that it sees; the tiles with the most tokens first.
template <int D, int NQ>
__global__ __launch_bounds__(kWaves * kWave) void attention_rows_kernel(Attention a, CacheView c) {
    constexpr int NJ = D / 16;
    constexpr int kRows = 16 * NQ;
    const int lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
    const int group = a.heads / c.heads;
    const Lane<D> ln(lane);
    auto weight = [&](int64_t s) -> int64_t {
        return ((int64_t)span_of(a, c.page_bits, s).n * group + kRows * kWaves - 1) / (kRows * kWaves);
    };
    const Layout<decltype(weight)> plan(weight, a.seqs, lane);
    const int64_t at = plan.total - 1 - (int64_t)blockIdx.x / c.heads;
    if (at < 0) return;
    const int head = (int)(blockIdx.x % c.heads);
    int64_t seq, begin;
    plan.find(at, seq, begin);
    Span s = span_of(a, c.page_bits, seq);
    s.first = uniform64(s.first, 0);
    s.n = uniform(s.n);
    s.len = uniform(s.len);
    const int64_t row0 = ((at - begin) * kWaves + wave) * kRows;
    const int64_t rows_left = (int64_t)s.n * group - row0;
    if (rows_left <= 0) return;
    Sums<D, NQ> sums;
    run_steps<D, NQ>(a, c, a.page_table + seq * a.table_width, s, head, group, row0, 0, kFarRight, 1, sums, ln);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int r = 16 * i + ln.n;
        float l = sums.l[i];
        l += __shfl_xor(l, 16, kWave);
        l += __shfl_xor(l, 32, kWave);
        if (r < rows_left) {
            const int64_t row = row0 + r, q = row / group;
            const int h = head * group + (int)(row - q * group);
            const float f = last_factor(sums.m[i], l, a.sinks, h);
            uint16_t* out = a.out + ((s.first + q) * a.heads + h) * D;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float o[NJ];
#pragma unroll
                for (int j = 0; j < NJ; ++j) o[j] = sums.o[i][j][e] * f;
                store_out<NJ>(out + NJ * (4 * ln.g + e), o);
            }
        }
    }
}

// Tiles of `rows` rows that the sequences of a call can have.
int64_t most_tiles(int64_t tokens, int64_t seqs, int64_t group, int64_t rows) {
    return tokens * group / rows + (seqs < tokens ? seqs : tokens);
}

struct Form {
    bool split;
    int nq;
    int workers;
};

// Which form a call takes, from what the host knows: rows a sequence on the average, tiles in all.
Form form_of(int64_t tokens, int64_t seqs, int64_t heads, int64_t kv_heads) {
    const int64_t group = heads / kv_heads, cus = device_cu_count();
    const int64_t mean = (tokens + seqs - 1) / seqs * group;
    const int64_t wide = most_tiles(tokens, seqs, group, 64 * kWaves) * kv_heads;
    if (mean > 64 && wide >= cus) return {false, 4, 0};
    if (mean > 32) return {true, 4, (int)(cus)};
    if (mean > 16) return {true, 2, (int)(2 * cus)};
    return {true, 1, (int)(3 * cus)};
}

template <int D, int NQ>
hipError_t split_form(const Attention& a, const CacheView& c, int workers, void* workspace, hipStream_t stream) {
    Record* records = static_cast<Record*>(workspace);
    float* parts = reinterpret_cast<float*>(records + workers);
    attention_split_kernel<D, NQ><<<workers, kWaves * kWave, 0, stream>>>(a, c, parts, records, workers);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    attention_join_kernel<D, NQ><<<dim3(workers, 4 * NQ), kWaves * kWave, 0, stream>>>(a, c, parts, records);
    return hipGetLastError();
}

template <int D>
hipError_t attend(const Attention& a, const CacheView& c, void* workspace, hipStream_t stream) {
    const Form f = form_of(a.tokens, a.seqs, a.heads, c.heads);
    if (!f.split) {
        const int64_t grid = most_tiles(a.tokens, a.seqs, a.heads / c.heads, 64 * kWaves) * c.heads;
        attention_rows_kernel<D, 4><<<(unsigned)grid, kWaves * kWave, 0, stream>>>(a, c);
        return hipGetLastError();
    }
    if (f.nq == 4) return split_form<D, 4>(a, c, f.workers, workspace, stream);
    if (f.nq == 2) return split_form<D, 2>(a, c, f.workers, workspace, stream);
    return split_form<D, 1>(a, c, f.workers, workspace, stream);
}

}  // namespace

size_t attention_workspace_bytes(int64_t tokens, int64_t seqs, int64_t heads, int64_t kv_heads, int64_t head_dim) {
    const Form f = form_of(tokens, seqs, heads, kv_heads);
    if (!f.split) return 0;
    return (size_t)f.workers * (sizeof(Record) + 2 * (size_t)16 * f.nq * (head_dim + 2) * sizeof(float));
}

hipError_t launch_attention(const Attention& a, const CacheView& c, void* workspace, hipStream_t stream) {
    return c.head_dim == 128 ? attend<128>(a, c, workspace, stream) : attend<64>(a, c, workspace, stream);
}

}  // namespace e2m1
