// attention.hip -- attention of packed query rows over the paged MXFP4 cache.
//
// Mathematics. Query i of a sequence with n queries and l cached tokens sits at
// position p = l - n + i and sees the keys max(0, p - window + 1) .. p (all l
// without a mask). out = sum_j exp(s_j - m) v_j / (sum_j exp(s_j - m) +
// exp(sink - m)), s_j = scale q . k_j, m their running maximum: one pass over
// the keys. A query that sees none gives zeros.
#include "device.hpp"
#include "kernels.hpp"

namespace e2m1 {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// One wave per query row and head: a lane per key for the scores, two channels a lane for the values.
template <int D>
__global__ __launch_bounds__(kWave) void attention_plain_kernel(Attention a, CacheView c) {
    __shared__ float qs[D];
    __shared__ float ps[kWave];
    const int64_t t = blockIdx.x;
    const int head = blockIdx.y;
    const int lane = threadIdx.x;
    // the sequence of row t
    int64_t seq = -1;
    for (int64_t s = 0; s < a.seqs; ++s)
        if (t >= a.q_offsets[s] && t < a.q_offsets[s + 1]) { seq = s; break; }
    if (seq < 0) return;
    const int page = 1 << c.page_bits;
    int64_t len = a.kv_lens[seq];
    const int64_t most = a.table_width << c.page_bits;
    if (len > most) { len = most; if (a.err_flag) *a.err_flag = 1; }
    if (len < 0) len = 0;
    const int64_t n = (int64_t)a.q_offsets[seq + 1] - a.q_offsets[seq];
    const int64_t pos = len - n + (t - a.q_offsets[seq]);
    int64_t lo = 0, hi = len;
    if (a.causal) {
        hi = pos + 1;
        if (a.window > 0 && pos - a.window + 1 > 0) lo = pos - a.window + 1;
    }
    const int kvh = head / (a.heads / c.heads);
    const uint16_t* q = a.q + t * a.q_stride + (int64_t)head * D;
    for (int i = lane; i < D; i += kWave) qs[i] = __uint_as_float((uint32_t)q[i] << 16);
    __syncthreads();
    const float sc = a.scale * kLog2e;
    float m = -INFINITY, l = 0.0f, o[D / kWave] = {};
    for (int64_t j0 = lo; j0 < hi; j0 += kWave) {
        const int64_t j = j0 + lane;
        float s = -INFINITY;
        int64_t row = -1;
        if (j < hi) {
            const int64_t pg = a.page_table[seq * a.table_width + (j >> c.page_bits)];
            if (pg >= 0 && (pg << c.page_bits) < c.slots) row = ((pg * c.heads + kvh) << c.page_bits) + (j & (page - 1));
            else if (a.err_flag) *a.err_flag = 1;
        }
        if (row >= 0) {
            float acc = 0.0f;
            for (int b = 0; b < D / 32; ++b) {
                const uint32_t e = c.k_scales[row * (D / 32) + b];
                const float scale = __uint_as_float(e << 23);
                if (e == 255u || c.v_scales[row * (D / 32) + b] == 255u) acc = __uint_as_float(0x7FC00000u);
                for (int w = 0; w < 4; ++w) {
                    const uint32_t word = *reinterpret_cast<const uint32_t*>(c.k_codes + row * (D / 2) + b * 16 + w * 4);
                    const float* x = qs + b * 32 + w * 8;
                    const f32x2 v0 = fp4x2_to_f32x2<0>(word, scale), v1 = fp4x2_to_f32x2<1>(word, scale);
                    const f32x2 v2 = fp4x2_to_f32x2<2>(word, scale), v3 = fp4x2_to_f32x2<3>(word, scale);
                    acc += v0.x * x[0] + v0.y * x[1] + v1.x * x[2] + v1.y * x[3] + v2.x * x[4] + v2.y * x[5] +
                           v3.x * x[6] + v3.y * x[7];
                }
            }
            s = acc * sc;
        }
        float top = s;
        for (int i = 32; i > 0; i >>= 1) {
            const float other = __shfl_xor(top, i, kWave);
            top = (top != top || other != other) ? __uint_as_float(0x7FC00000u) : fmaxf(top, other);
        }
        const float mn = (m != m || top != top) ? __uint_as_float(0x7FC00000u) : fmaxf(m, top);
        if (mn == -INFINITY) continue;
        const float p = row >= 0 ? exp2f(s - mn) : 0.0f;
        const float f = exp2f(m - mn);
        m = mn;
        l = l * f + group_sum<kWave>(p);
        for (int i = 0; i < D / kWave; ++i) o[i] *= f;
        ps[lane] = p;
        __syncthreads();
        for (int x = 0; x < kWave && j0 + x < hi; ++x) {
            const int64_t r = __shfl((long long)row, x, kWave);
            if (r < 0) continue;
            for (int i = 0; i < D / kWave; ++i) {
                const int d = i * kWave + lane;
                const uint32_t e = c.v_scales[r * (D / 32) + d / 32];
                const uint32_t word = c.v_codes[r * (D / 2) + d / 2];
                const f32x2 v = fp4x2_to_f32x2<0>(word, __uint_as_float(min(e, 254u) << 23));
                o[i] += ps[x] * (d & 1 ? v.y : v.x);
            }
        }
        __syncthreads();
    }
    if (a.sinks && m != -INFINITY) {
        const float s = a.sinks[head] * kLog2e, mn = fmaxf(m, s), f = exp2f(m - mn);
        l = l * f + exp2f(s - mn);
        for (int i = 0; i < D / kWave; ++i) o[i] *= f;
    }
    for (int i = 0; i < D / kWave; ++i)
        a.out[(t * a.heads + head) * D + i * kWave + lane] = (uint16_t)f32_to_bf16_rne(m == -INFINITY ? 0.0f : o[i] / l);
}

}  // namespace

size_t attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_attention(const Attention& a, const CacheView& c, void*, hipStream_t stream) {
    const dim3 grid((unsigned)a.tokens, (unsigned)a.heads);
    if (c.head_dim == 128) attention_plain_kernel<128><<<grid, kWave, 0, stream>>>(a, c);
    else attention_plain_kernel<64><<<grid, kWave, 0, stream>>>(a, c);
    return hipGetLastError();
}

}  // namespace e2m1
