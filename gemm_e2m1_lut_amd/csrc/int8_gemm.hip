// int8_gemm.hip -- product of two int8 matrices with a scale per token and per
// output channel (int8_gemm).
//
// Mathematics: y[m][n] = (sum_k x[m][k] w[n][k]) x_scale[m] w_scale[n] + bias[n].
// The sum is exact: int8 products in int32 accumulators (|sum| <= 2^14 k, below
// 2^31 for k <= 131056). It is rounded to fp32 once, then multiplied by the two
// scales and added to the bias in fp32, and rounded to the output type once.
#include "device.hpp"
#include "kernels.hpp"

namespace e2m1 {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));

constexpr uint32_t kOutOfRange = 0xFFFFFFF0u;   // a buffer offset past any resource's range

__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t rsrc, uint32_t off) {
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, off, 0, 0));
}

// Four outputs of row m from column n0 on.
template <bool kBf16Out>
__device__ __forceinline__ void store4(void* y, int64_t idx, const f32x4& v, int count) {
    if constexpr (kBf16Out) {
        uint16_t* p = reinterpret_cast<uint16_t*>(y) + idx;
        if (count == 4 && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
            *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        } else {
            for (int j = 0; j < count; ++j) p[j] = (uint16_t)f32_to_bf16_rne(v[j]);
        }
    } else {
        float* p = reinterpret_cast<float*>(y) + idx;
        if (count == 4 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
            *reinterpret_cast<f32x4*>(p) = v;
        } else {
            for (int j = 0; j < count; ++j) p[j] = v[j];
        }
    }
}

// ------------------------------------------------------------ split form --
// A workgroup owns 16 NT rows of w and 16 MT rows of x; its waves split K
// (128-column steps dealt in turn) and the partial sums meet in LDS. Operands
// go straight from memory into the matrix cores' registers: lane 16 g + r holds
// columns 16 g .. + 15 of row r of a 64-column block.

template <int MT, int NT, bool kBf16Out>
__global__ __launch_bounds__(1024) void int8_gemm_split_kernel(
    const int8_t* __restrict__ x, const float* __restrict__ xs, const int8_t* __restrict__ w,
    const float* __restrict__ ws, const float* __restrict__ bias, void* __restrict__ y, int m, int n, int k) {
    extern __shared__ __attribute__((aligned(16))) int32_t part[];   // [wave][tile][lane][4]
    constexpr int kTiles = MT * NT;
    const int nwaves = blockDim.x / kWave;
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, g = lane >> 4;
    const int64_t tile_id = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int tiles_n = (n + 16 * NT - 1) / (16 * NT);
    const int n0 = (int)(tile_id % tiles_n) * 16 * NT;
    const int64_t mstart = tile_id / tiles_n * 16 * MT;
    if (mstart >= m) return;   // the grid's last row may run past the tiles
    const int m0 = (int)mstart;
    const int nt = min(16 * NT, n - n0), mt = min(16 * MT, m - m0);
    const __amdgpu_buffer_rsrc_t wres = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t*>(w + (int64_t)n0 * k), 0, nt * k, kBufferWord3);
    const __amdgpu_buffer_rsrc_t xres = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t*>(x + (int64_t)m0 * k), 0, mt * k, kBufferWord3);
    i32x4 acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

    const int steps = (k + 127) / 128;
    constexpr int kAhead = NT + MT <= 2 ? 4 : 2;   // steps whose loads are in flight together
    for (int s = wave; s < steps; s += nwaves * kAhead) {
        i32x4 a[kAhead][2][NT], b[kAhead][2][MT];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = 128 * (s + u * nwaves) + 64 * h + 16 * g;
                const bool live = c < k;   // past the row's end: zeros, no memory access
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    a[u][h][i] = load16(wres, live && 16 * i + r < nt ? (uint32_t)((16 * i + r) * k + c) : kOutOfRange);
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    b[u][h][j] = load16(xres, live && 16 * j + r < mt ? (uint32_t)((16 * j + r) * k + c) : kOutOfRange);
            }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < MT; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u][h][i], b[u][h][j], acc[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
            *reinterpret_cast<i32x4*>(part + ((wave * kTiles + i * MT + j) * kWave + lane) * 4) = acc[i][j];
    __syncthreads();
    // one quad (row m, four columns n) per thread and turn
    for (int qd = threadIdx.x; qd < kTiles * kWave; qd += blockDim.x) {
        i32x4 sum = {0, 0, 0, 0};
        for (int v = 0; v < nwaves; ++v) sum += *reinterpret_cast<const i32x4*>(part + (v * kTiles * kWave + qd) * 4);
        const int tile = qd / kWave, l = qd % kWave;
        const int mm = m0 + 16 * (tile % MT) + (l & 15);
        const int nn = n0 + 16 * (tile / MT) + 4 * (l >> 4);
        if (mm >= m || nn >= n) continue;
        const int count = min(4, n - nn);
        const float sx = xs[mm];
        f32x4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int c = min(nn + e, n - 1);
            v[e] = (float)sum[e] * sx * ws[c];
            if (bias != nullptr) v[e] += bias[c];
        }
        store4<kBf16Out>(y, (int64_t)mm * n + nn, v, count);
    }
}

// `tiles` workgroups in rows of 2^20 (a grid dimension holds fewer than 2^32 threads).
dim3 grid_of(int64_t tiles) {
    const int64_t gx = tiles < (1 << 20) ? tiles : 1 << 20;
    return dim3((unsigned)gx, (unsigned)((tiles + gx - 1) / gx));
}

template <int MT, int NT>
hipError_t launch_split(const int8_t* x, const float* xs, const int8_t* w, const float* ws, const float* bias, void* y,
                        bool out_bf16, int64_t m, int64_t n, int64_t k, int waves, hipStream_t stream) {
    const dim3 grid = grid_of(((n + 16 * NT - 1) / (16 * NT)) * ((m + 16 * MT - 1) / (16 * MT)));
    const unsigned lds = (unsigned)(waves * MT * NT * kWave * 16);
    if (out_bf16)
        int8_gemm_split_kernel<MT, NT, true><<<grid, waves * kWave, lds, stream>>>(x, xs, w, ws, bias, y, (int)m, (int)n, (int)k);
    else
        int8_gemm_split_kernel<MT, NT, false><<<grid, waves * kWave, lds, stream>>>(x, xs, w, ws, bias, y, (int)m, (int)n, (int)k);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_gemm(const int8_t* x, const float* x_scale, const int8_t* w, const float* w_scale,
                            const float* bias, void* y, bool out_bf16, int64_t m, int64_t n, int64_t k,
                            hipStream_t stream) {
    if (m <= 16) {
        const int64_t steps = (k + 127) / 128;
        const int waves = steps >= 64 ? 16 : steps >= 16 ? 8 : 4;
        return launch_split<1, 1>(x, x_scale, w, w_scale, bias, y, out_bf16, m, n, k, waves, stream);
    }
    return launch_split<4, 2>(x, x_scale, w, w_scale, bias, y, out_bf16, m, n, k, 4, stream);
}

}  // namespace e2m1
