// cache.hip -- the paged MXFP4 cache of an attention layer: rows of keys and
// values into it (mxfp4_cache_write; norm_rope_mxfp4_cache_write from the rows
// of a fused q | k | v product, with the norm and rotation of the heads), and
// tokens of it back to bf16 by slot (mxfp4_cache_read).
//
// Mathematics. A head's row of d values is d / 32 blocks; a block with largest
// magnitude amax gets e = max(floor(log2 amax) - 2 + 127, 0) and each element
// the E2M1 code nearest to x / 2^(e - 127), ties to the even code, magnitudes
// above 6 to 6: the rule of mxfp4_quantize, applied to the fp32 value, so that
// a normed and rotated key is rounded once. A block that holds a NaN or an
// infinity gets scale byte 255 (the E8M0 NaN) and codes 0. With a norm,
// x <- x w / sqrt(mean(x^2) + eps) over the head's d channels, in fp32 (the sum
// of at most 128 squares, added in a tree). The rotation takes channel pairs
// (i, i + rot / 2), or (2 i, 2 i + 1) interleaved, through the angle of
// position and i: (a cos - b sin, b cos + a sin), with cos and sin read from the
// caller's fp32 table.
//
// gfx950 design. All three stream memory. A lane owns 8 channels (16 bytes of
// bf16 in, 4 bytes of codes out, or the reverse), 16 or 8 lanes a head, so a
// block is a quad of lanes (its maximum two DPP steps away) and a norm's sum or
// a rotation's partner at most 15 lanes away. In the fused writer the groups of
// a workgroup are tokens and its loop runs over heads: a group reads its
// token's angles once for all the heads it takes, and q, k and v heads part at
// a branch that the whole workgroup takes alike. The codes of a head are 64 (or
// 32) contiguous bytes and its scales 4 (or 2): [page][head][place], the layout
// in which attention reads a head's tokens in one run.
//
// Bounds. Many tokens: HBM; 8192 of 32 query and 8 + 8 kv heads of 128 through norm
// and rotation 40.6 us (181 MB, 4.5 TB/s: half of the issue slots are taken as well),
// 16384 of 8 heads of 128 read back 17.4 us (85 MB, 4.9 TB/s). Few: the latency of a
// slot's load, a row's load and the store, 2.4 us.
#include <limits.h>

#include "device.hpp"
#include "kernels.hpp"

namespace e2m1 {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kInfBits = 0x7F800000u;

// Eight channels of a row as they lie in memory.
template <typename T>
struct Raw;

template <>
struct Raw<uint16_t> {
    uint4 a;
    __device__ __forceinline__ void load(const uint16_t* p) { a = load_nt16(p); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};

template <>
struct Raw<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        // not streaming: the two halves of a line come with two instructions, and a streaming load would fetch it twice (4097
        // tokens of 8 heads of 64: 10.3 us with the read back instead of 14.4)
        a = *reinterpret_cast<const uint4*>(p);
        b = *reinterpret_cast<const uint4*>(p + 4);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    }
};

// Two bf16 numbers, rounded to nearest, ties to even.
__device__ __forceinline__ uint32_t round_bf16x2(float lo, float hi) {
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Rows that a group has on their way at a time (norm and rotation of 8192 tokens, read back: 50.8 us; 1: 52.8, 8: 51.9).
constexpr int kAtOnce = 4;

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true);
}

// The codes of a lane's eight values and the scale byte of its block (a quad of lanes).
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], uint32_t& e) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    m = max(m, dpp_u32<0xB1>(m));
    m = max(m, dpp_u32<0x4E>(m));
    e = (uint32_t)max((int)(m >> 23) - 2, 0);
    const float sc = __uint_as_float(e << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], sc, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], sc, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], sc, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], sc, 3);
    const bool bad = m >= kInfBits;
    e = bad ? 255u : e;
    return bad ? 0u : c;
}

template <int kCtrl>
__device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double,
                              (uint64_t)dpp_u32<kCtrl>((uint32_t)u) | ((uint64_t)dpp_u32<kCtrl>((uint32_t)(u >> 32)) << 32));
}

// A head's norm with the sum and the products in 64 bits, where the squares of every finite fp32 fit; a row of zeros
// stays one also where eps is 0.
template <int kLanes>
__device__ __forceinline__ void norm_wide(float (&x)[8], const float (&w)[8], float eps) {
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += (double)x[i] * x[i];
    ss += dpp_f64<0xB1>(ss);
    ss += dpp_f64<0x4E>(ss);
    ss += dpp_f64<0x141>(ss);
    if constexpr (kLanes == 16) ss += dpp_f64<0x140>(ss);
    const double f = ss == 0.0 ? 0.0 : 1.0 / sqrt(ss / (8 * kLanes) + (double)eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)((double)x[i] * f * w[i]);
}

template <typename T>
__device__ __forceinline__ void load_row(const T* p, float (&x)[8]) {
    Raw<T> raw;
    raw.load(p);
    raw.get(x);
}

template <int D>
__device__ __forceinline__ void store_row(const float (&x)[8], uint8_t* codes, uint8_t* scales, int64_t row, int lane,
                                          bool live) {
    uint32_t e;
    const uint32_t c = encode8(x, e);
    if (live) {
        *reinterpret_cast<uint32_t*>(codes + row * (D / 2) + lane * 4) = c;
        if (lane % 4 == 0) scales[row * (D / 32) + lane / 4] = (uint8_t)e;
    }
}

// Row of the cache's [pages, heads, page] that holds `slot` of `head`.
__device__ __forceinline__ int64_t cache_row(int64_t slot, int head, const CacheView& c) {
    return ((slot >> c.page_bits) * c.heads + head) * ((int64_t)1 << c.page_bits) +
           (slot & (((int64_t)1 << c.page_bits) - 1));
}

// Group g of a workgroup takes token blockIdx.x * groups + g and the rows [blockIdx.y * rows_per, ..) of its keys and
// then its values.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(const T* __restrict__ k, const T* __restrict__ v,
                                                               int64_t k_stride, int64_t v_stride,
                                                               const int64_t* __restrict__ slots, CacheView c,
                                                               int64_t tokens, int rows_per, int32_t* err_flag) {
    constexpr int kLanes = D / 8;
    const int lane = threadIdx.x % kLanes;
    const int64_t at = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    const bool in = at < tokens;
    const int64_t t = in ? at : tokens - 1;
    const int64_t slot = slots[t];
    const bool live = in && slot >= 0 && slot < c.slots;
    if (in && slot >= c.slots && err_flag) *err_flag = 1;
    const int first = blockIdx.y * rows_per, last = min(first + rows_per, 2 * c.heads);
    for (int r0 = first; r0 < last; r0 += kAtOnce) {
        Raw<T> raw[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int r = min(r0 + i, last - 1);
            raw[i].load((r >= c.heads ? v + t * v_stride + (r - c.heads) * D : k + t * k_stride + r * D) + lane * 8);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int r = r0 + i;
            if (r >= last) break;
            const bool is_v = r >= c.heads;
            float x[8];
            raw[i].get(x);
            store_row<D>(x, is_v ? c.v_codes : c.k_codes, is_v ? c.v_scales : c.k_scales,
                         cache_row(live ? slot : 0, is_v ? r - c.heads : r, c), lane, live);
        }
    }
}

// The same over a token's query, key and value heads, queries to q_out.
template <typename T, int D, bool kInterleaved>
__global__ __launch_bounds__(kThreads) void norm_rope_write_kernel(
    const T* __restrict__ qkv, int64_t stride, const T* __restrict__ q_weight, const T* __restrict__ k_weight, float eps,
    const float* __restrict__ cos_sin, int64_t max_pos, int rot, const int64_t* __restrict__ positions,
    const int64_t* __restrict__ slots, uint16_t* __restrict__ q_out, int heads, CacheView c, int64_t tokens, int rows_per,
    int32_t* err_flag) {
    constexpr int kLanes = D / 8;
    const int lane = threadIdx.x % kLanes;
    const int64_t at = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    const bool in = at < tokens;
    const int64_t t = in ? at : tokens - 1;
    const int64_t slot = slots[t];
    const int64_t pos = rot > 0 ? positions[t] : 0;
    const bool placed = rot == 0 || (pos >= 0 && pos < max_pos);
    const bool live = in && slot >= 0 && slot < c.slots && placed;
    if (in && (slot >= c.slots || (slot >= 0 && !placed)) && err_flag) *err_flag = 1;
    const int first = blockIdx.y * rows_per, last = min(first + rows_per, heads + 2 * c.heads);

    // angles of this lane's channels: eight of one half, or four pairs
    const bool turns = lane * 8 < rot && max_pos > 0;   // an empty table has no position, and nothing to read
    const bool high = !kInterleaved && lane * 8 >= rot / 2;
    const int partner = threadIdx.x % kWave + (high ? -rot / 16 : rot / 16);
    float cs[8], sn[8];
    if (turns && first < heads + c.heads) {
        const float* row = cos_sin + (placed ? pos : 0) * rot;
        const int i0 = kInterleaved ? lane * 4 : high ? lane * 8 - rot / 2 : lane * 8;
#pragma unroll
        for (int i = 0; i < (kInterleaved ? 4 : 8); i += 4) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(row + i0 + i);
            const f32x4 b = *reinterpret_cast<const f32x4*>(row + rot / 2 + i0 + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                cs[i + e] = a[e];
                sn[i + e] = kInterleaved || high ? b[e] : -b[e];
            }
        }
    }
    float wq[8], wk[8];   // the norms' weights
    if (q_weight && first < heads) load_row(q_weight + lane * 8, wq);
    if (k_weight && first < heads + c.heads && last > heads) load_row(k_weight + lane * 8, wk);
    const T* row = qkv + t * stride + lane * 8;
    for (int r0 = first; r0 < last; r0 += kAtOnce) {
        Raw<T> raw[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) raw[i].load(row + (int64_t)min(r0 + i, last - 1) * D);
#pragma unroll
        for (int n = 0; n < kAtOnce; ++n) {
            const int r = r0 + n;
            if (r >= last) break;
            float x[8];
            raw[n].get(x);
            const int kind = r < heads ? 0 : r < heads + c.heads ? 1 : 2;
            if (kind < 2) {
                if (kind == 0 ? q_weight != nullptr : k_weight != nullptr) {
                    float w[8], ss = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = kind == 0 ? wq[i] : wk[i];
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
                    ss = group_sum<kLanes>(ss);
                    if (ss > 0x1p-80f && ss < 0x1p100f) {
                        const float f = __builtin_amdgcn_rsqf(ss * (1.0f / D) + eps);
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = x[i] * f * w[i];
                    } else {
                        norm_wide<kLanes>(x, w, eps);   // squares past the fp32 range, or nearly so: the whole group alike
                    }
                }
                if (kInterleaved) {
                    if (turns) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float a = x[2 * i], b = x[2 * i + 1];
                            x[2 * i] = a * cs[i] - b * sn[i];
                            x[2 * i + 1] = b * cs[i] + a * sn[i];
                        }
                    }
                } else {
                    float o[8];   // every lane takes part in the exchange, those past rot for nothing
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = __shfl(x[i], partner & (kWave - 1), kWave);
                    if (turns) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = x[i] * cs[i] + o[i] * sn[i];
                    }
                }
            }
            if (kind == 0) {
                if (in) {
                    uint4 o = make_uint4(round_bf16x2(x[0], x[1]), round_bf16x2(x[2], x[3]), round_bf16x2(x[4], x[5]),
                                         round_bf16x2(x[6], x[7]));
                    if (!placed) o = make_uint4(0, 0, 0, 0);
                    store_nt16(q_out + (t * heads + r) * D + lane * 8, o.x, o.y, o.z, o.w);
                }
            } else {
                const int head = kind == 1 ? r - heads : r - heads - c.heads;
                store_row<D>(x, kind == 1 ? c.k_codes : c.v_codes, kind == 1 ? c.k_scales : c.v_scales,
                             cache_row(live ? slot : 0, head, c), lane, live);
            }
        }
    }
}

// Eight codes of a block with scale byte e as bf16 pairs; zero codes give +0, 255 NaN.
__device__ __forceinline__ uint4 decode8(uint32_t c, uint32_t e) {
    if (e == 255u) return make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
    c &= ~(0x88888888u & ~(c << 1 | c << 2 | c << 3));   // code 8 (-0) to code 0
    const float sc = __uint_as_float(e << 23);
    return make_uint4(fp4x2_to_bf16x2<0>(c, sc), fp4x2_to_bf16x2<1>(c, sc), fp4x2_to_bf16x2<2>(c, sc),
                      fp4x2_to_bf16x2<3>(c, sc));
}

// One group of lanes per token and head, keys and values together; a grid that does not cover all rows goes round.
template <int D>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(CacheView c, const int64_t* __restrict__ slots,
                                                              uint16_t* __restrict__ k_out, uint16_t* __restrict__ v_out,
                                                              int64_t rows, int32_t* err_flag) {
    constexpr int kLanes = D / 8;
    const int lane = threadIdx.x % kLanes;
    for (int64_t row = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kLanes; row < rows;
         row += (int64_t)gridDim.x * (kThreads / kLanes)) {
        const int64_t t = rows <= INT_MAX ? (int64_t)((uint32_t)row / (uint32_t)c.heads) : row / c.heads;
        const int head = (int)(row - t * c.heads);
        const int64_t slot = slots[t];
        uint4 ko = make_uint4(0, 0, 0, 0), vo = ko;
        if (slot >= 0 && slot < c.slots) {
            const int64_t at = cache_row(slot, head, c);
            const uint32_t kc = *reinterpret_cast<const uint32_t*>(c.k_codes + at * (D / 2) + lane * 4);
            const uint32_t vc = *reinterpret_cast<const uint32_t*>(c.v_codes + at * (D / 2) + lane * 4);
            const uint32_t ke = c.k_scales[at * (D / 32) + lane / 4], ve = c.v_scales[at * (D / 32) + lane / 4];
            ko = decode8(kc, ke);
            vo = decode8(vc, ve);
        } else if (slot >= 0 && err_flag) {
            *err_flag = 1;
        }
        store_nt16(k_out + row * D + lane * 8, ko.x, ko.y, ko.z, ko.w);
        store_nt16(v_out + row * D + lane * 8, vo.x, vo.y, vo.z, vo.w);
    }
}

// Heads a group takes one after another: all of a token's angles are read again by each of its groups, so a large call takes
// several heads a group (8192 tokens through norm and rotation, read back: 50.8 us, a head a group 101), and a small one a
// head each (64 tokens 5.8, eight a group 9.3).
int rows_per_group(int64_t token_groups, int rows) {
    int per = 1;
    while (per < 8 && token_groups * ((rows + per - 1) / per) > 8 * device_cu_count()) per *= 2;
    return per;
}

template <typename T, int D>
hipError_t write_rows(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int64_t* slots,
                      const CacheView& c, int64_t tokens, int32_t* err_flag, hipStream_t stream) {
    const int64_t gx = (tokens * (D / 8) + kThreads - 1) / kThreads;
    const int per = rows_per_group(gx, 2 * c.heads);
    const dim3 grid((unsigned)gx, (unsigned)((2 * c.heads + per - 1) / per));
    cache_write_kernel<T, D><<<grid, kThreads, 0, stream>>>(static_cast<const T*>(k), static_cast<const T*>(v), k_stride,
                                                            v_stride, slots, c, tokens, per, err_flag);
    return hipGetLastError();
}

template <typename T, int D, bool kInterleaved>
hipError_t norm_rope_rows(const NormRope& a, const CacheView& c, int64_t tokens, int32_t* err_flag, hipStream_t stream) {
    const int64_t gx = (tokens * (D / 8) + kThreads - 1) / kThreads;
    const int rows = a.heads + 2 * c.heads;
    const int per = rows_per_group(gx, rows);
    const dim3 grid((unsigned)gx, (unsigned)((rows + per - 1) / per));
    norm_rope_write_kernel<T, D, kInterleaved><<<grid, kThreads, 0, stream>>>(
        static_cast<const T*>(a.qkv), a.stride, static_cast<const T*>(a.q_weight), static_cast<const T*>(a.k_weight),
        a.eps, a.cos_sin, a.max_pos, a.rot, a.positions, a.slots, a.q_out, a.heads, c, tokens, per, err_flag);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t norm_rope_pairs(const NormRope& a, const CacheView& c, int64_t tokens, int32_t* err_flag,
                           hipStream_t stream) {
    return a.interleaved ? norm_rope_rows<T, D, true>(a, c, tokens, err_flag, stream)
                         : norm_rope_rows<T, D, false>(a, c, tokens, err_flag, stream);
}

}  // namespace

hipError_t launch_cache_write(const void* k, const void* v, bool bf16, int64_t k_stride, int64_t v_stride,
                              const int64_t* slots, const CacheView& c, int64_t tokens, int32_t* err_flag,
                              hipStream_t stream) {
    if (c.head_dim == 128)
        return bf16 ? write_rows<uint16_t, 128>(k, v, k_stride, v_stride, slots, c, tokens, err_flag, stream)
                    : write_rows<float, 128>(k, v, k_stride, v_stride, slots, c, tokens, err_flag, stream);
    return bf16 ? write_rows<uint16_t, 64>(k, v, k_stride, v_stride, slots, c, tokens, err_flag, stream)
                : write_rows<float, 64>(k, v, k_stride, v_stride, slots, c, tokens, err_flag, stream);
}

hipError_t launch_norm_rope_write(const NormRope& a, bool bf16, const CacheView& c, int64_t tokens, int32_t* err_flag,
                                  hipStream_t stream) {
    if (c.head_dim == 128)
        return bf16 ? norm_rope_pairs<uint16_t, 128>(a, c, tokens, err_flag, stream)
                    : norm_rope_pairs<float, 128>(a, c, tokens, err_flag, stream);
    return bf16 ? norm_rope_pairs<uint16_t, 64>(a, c, tokens, err_flag, stream)
                : norm_rope_pairs<float, 64>(a, c, tokens, err_flag, stream);
}

hipError_t launch_cache_read(const CacheView& c, const int64_t* slots, uint16_t* k_out, uint16_t* v_out, int64_t tokens,
                             int32_t* err_flag, hipStream_t stream) {
    const int64_t rows = tokens * c.heads;
    const int64_t need = (rows * (c.head_dim / 8) + kThreads - 1) / kThreads;
    const unsigned grid = (unsigned)(need < 1 << 20 ? need : 1 << 20);
    if (c.head_dim == 128)
        cache_read_kernel<128><<<grid, kThreads, 0, stream>>>(c, slots, k_out, v_out, rows, err_flag);
    else
        cache_read_kernel<64><<<grid, kThreads, 0, stream>>>(c, slots, k_out, v_out, rows, err_flag);
    return hipGetLastError();
}

}  // namespace e2m1
