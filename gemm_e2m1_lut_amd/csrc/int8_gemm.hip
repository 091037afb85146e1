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

// ------------------------------------------------------------- tile form --
// A workgroup owns a tile of 16 TN kWN rows of w x 16 TM kWM rows of x; each of
// its kWN x kWM waves 16 TN x 16 TM of it in 16x16x64 matrix-core tiles (A = w, B = x).
// K goes in steps of KS columns through a ring of NS LDS buffers that the
// memory pipeline fills itself (buffer_load ... lds: no registers, no LDS
// writes by the waves). In LDS a row's 16-byte chunks are permuted, chunk c of
// row r at slot c ^ (r / (256 / KS) % (KS / 16)), so that an operand read (16 rows, one
// chunk) meets every bank once; the requests' source addresses do that, as
// the LDS side of a request is contiguous.
// Operands are read one 64-column slice ahead of their MFMAs, over the step's
// border too: before the last slice's MFMAs of step s a wave waits until its own
// reads of the buffer and its requests of step s + 1 are done, passes the step's
// one barrier (with the previous slice's MFMAs still running), requests step s +
// NS into the buffer that is now free and reads the first slice of step s + 1.
// The sums leave through LDS too, one 16-row band of x at a time in an area of
// the wave's own, so that whole rows of y are scaled and stored.

// the lane's 16 bytes at byte offset voff of the buffer -> LDS lds + 16 * lane (M0 is set here and used
// by nothing else in these kernels)
__device__ __forceinline__ void lds_load16(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(lds), "v"(voff), "s"(rsrc) : "memory");
}

// This wave's LDS reads are done and at most kN of its requests are in flight; then the workgroup's barrier.
template <int kN>
__device__ __forceinline__ void step_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(kN) : "memory");
}

constexpr int kXcds = 8;

constexpr int KS = 128;   // columns per step: two slices (64-byte row segments read at half the L2 rate)

template <int kWN, int kWM, int TN, int TM, int NS, bool kBf16Out>
__global__ __launch_bounds__(kWave * kWN * kWM) void int8_gemm_tile_kernel(
    const int8_t* __restrict__ x, const float* __restrict__ xs, const int8_t* __restrict__ w,
    const float* __restrict__ ws, const float* __restrict__ bias, void* __restrict__ y, int m, int n, int k,
    int64_t tiles, int group_m) {
    constexpr int kWaves = kWN * kWM;
    constexpr int NR = 16 * TN * kWN, MR = 16 * TM * kWM;
    constexpr int kWLoads = NR / 8 / kWaves, kXLoads = MR / 8 / kWaves;   // 1 KB requests (8 rows) per wave and step
    constexpr int kSlices = KS / 64;
    static_assert(kWLoads * 8 * kWaves == NR && kXLoads * 8 * kWaves == MR, "requests");
    constexpr int kBufBytes = (NR + MR) * KS;
    constexpr int kOutBytes = 16 * 16 * TN * 4;                           // a wave's band of sums
    static_assert(kWaves * kOutBytes <= NS * kBufBytes && NS * kBufBytes <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(256))) uint8_t lds[NS * kBufBytes];

    // workgroup id -> tile: ids go round the XCDs, and each XCD gets a run of neighbouring tiles
    // (group_m tiles along x, then along w), which share their operands in its L2
    const int64_t per = (tiles + kXcds - 1) / kXcds;
    const int64_t id = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t tile = id % kXcds * per + id / kXcds;
    if (id / kXcds >= per || tile >= tiles) return;   // the whole workgroup
    const int tn = (n + NR - 1) / NR, tm = (m + MR - 1) / MR;
    const int64_t band = (int64_t)group_m * tn;
    const int mfirst = (int)(tile / band) * group_m;
    const int msize = min(group_m, tm - mfirst);
    const int n0 = (int)(tile % band / msize) * NR;
    const int m0 = (mfirst + (int)(tile % band % msize)) * MR;

    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, g = lane >> 4;
    const int wn = (wave % kWN) * 16 * TN, wm = (wave / kWN) * 16 * TM;
    const int nt = min(NR, n - n0), mt = min(MR, m - m0);
    const __amdgpu_buffer_rsrc_t wres = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t*>(w + (int64_t)n0 * k), 0, nt * k, kBufferWord3);
    const __amdgpu_buffer_rsrc_t xres = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t*>(x + (int64_t)m0 * k), 0, mt * k, kBufferWord3);

    // request i of a wave fills rows 8 (kLoads wave + i) .. + 7 of its operand; lane l fills slot l % 8 of row
    // l / 8, whose chunk is l % 8 ^ (row / 2 % 8): column col for every second request, col ^ 64 for the others.
    // Rows past the matrix read out of range: zeros, no memory access.
    const int col = 16 * ((lane % 8) ^ (lane >> 4));
    auto wcol = [&](int i) __attribute__((always_inline)) { return col ^ (64 * ((kWLoads * wave + i) & 1)); };
    auto xcol = [&](int i) __attribute__((always_inline)) { return col ^ (64 * ((kXLoads * wave + i) & 1)); };
    uint32_t woff[kWLoads], xoff[kXLoads];
#pragma unroll
    for (int i = 0; i < kWLoads; ++i)
        woff[i] = (uint32_t)(8 * (kWLoads * wave + i) + lane / 8) * (uint32_t)k + (uint32_t)wcol(i);
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
        xoff[i] = (uint32_t)(8 * (kXLoads * wave + i) + lane / 8) * (uint32_t)k + (uint32_t)xcol(i);
    const uint32_t base = (uint32_t)(uintptr_t)&lds[0];
    auto issue = [&](int st, int b) __attribute__((always_inline)) {
        const int c0 = st * KS;   // below 2^18: st <= steps + NS
        const uint32_t at = base + b * kBufBytes;
#pragma unroll
        for (int i = 0; i < kWLoads; ++i)   // columns (and whole steps) past K too
            lds_load16(wres, c0 + wcol(i) < k ? woff[i] + (uint32_t)c0 : kOutOfRange,
                       __builtin_amdgcn_readfirstlane(at + 1024u * (uint32_t)(kWLoads * wave + i)));
#pragma unroll
        for (int i = 0; i < kXLoads; ++i)
            lds_load16(xres, c0 + xcol(i) < k ? xoff[i] + (uint32_t)c0 : kOutOfRange,
                       __builtin_amdgcn_readfirstlane(at + NR * KS + 1024u * (uint32_t)(kXLoads * wave + i)));
    };
    // operand i of w / j of x: slice q of buffer b (row / 2 % 8 is r / 2 % 8: the tiles start at multiples of 16)
    const uint8_t* wrow = lds + (wn + r) * KS;
    const uint8_t* xrow = lds + NR * KS + (wm + r) * KS;
    const int slot[2] = {16 * (g ^ (r >> 1)), 16 * ((4 + g) ^ (r >> 1))};
    auto read_w = [&](int b, int q, int i) __attribute__((always_inline)) {
        return *reinterpret_cast<const i32x4*>(wrow + slot[q] + (b * kBufBytes + 16 * i * KS));
    };
    auto read_x = [&](int b, int q, int j) __attribute__((always_inline)) {
        return *reinterpret_cast<const i32x4*>(xrow + slot[q] + (b * kBufBytes + 16 * j * KS));
    };

    i32x4 a[TN], c[2][TM];
    i32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

    const int steps = (k + KS - 1) / KS;
    constexpr int kPerStep = kWLoads + kXLoads;
#pragma unroll
    for (int st = 0; st < NS; ++st) issue(st, st);
    step_barrier<kPerStep*(NS - 1)>();
#pragma unroll
    for (int j = 0; j < TM; ++j) c[0][j] = read_x(0, 0, j);
#pragma unroll
    for (int i = 0; i < TN; ++i) a[i] = read_w(0, 0, i);
    for (int s0 = 0; s0 < steps; s0 += NS) {   // unrolled by the ring, so that the buffers are static
#pragma unroll
        for (int b = 0; b < NS; ++b) {
            const int s = s0 + b;
            if (s >= steps) break;   // workgroup-uniform
#pragma unroll
            for (int q = 0; q < kSlices; ++q) {
                // the slice after this one (after the last step: read, never used)
                const int set = q & 1, nb = q + 1 < kSlices ? b : (b + 1) % NS, nq = (q + 1) % kSlices;
                __builtin_amdgcn_sched_barrier(0);
                if (q + 1 == kSlices) {
                    step_barrier<kPerStep*(NS - 2)>();
                    issue(s + NS, b);
                }
#pragma unroll
                for (int j = 0; j < TM; ++j) c[1 - set][j] = read_x(nb, nq, j);
#pragma unroll
                for (int i = 0; i < TN; ++i) {   // an operand of w is replaced as soon as its MFMAs are under way
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int j = 0; j < TM; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], c[set][j], acc[i][j], 0, 0, 0);
                    a[i] = read_w(nb, nq, i);
                }
            }
        }
    }
    step_barrier<0>();   // every request has landed and every read is done: the buffers are free

    // lane 16 g + r holds, of row wm + 16 j + r of x, rows wn + 16 i + 4 g .. + 3 of w: chunk 4 i + g of the
    // band's row, permuted like the operands' chunks so that 16 rows of one chunk meet every bank once
    auto mix = [](int row) __attribute__((always_inline)) { return TN >= 4 ? row : row >> 1; };
    static_assert(TN >= 2, "eight chunks in a band's row");
    constexpr int kLanesPerRow = 4 * TN;                 // lanes that store one row of the band, four outputs each
    constexpr int kRowsPer = kWave / kLanesPerRow;
    int32_t* area = reinterpret_cast<int32_t*>(lds + wave * kOutBytes);
    const int chunk = lane % kLanesPerRow;
    const int nn = n0 + wn + 4 * chunk;
    const int count = min(4, n - nn);                    // <= 0: nothing to store
    float sw[4], bb[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int col = min(nn + e, n - 1);
        sw[e] = ws[col];
        bb[e] = bias != nullptr ? bias[col] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < TM; ++j) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
            *reinterpret_cast<i32x4*>(area + r * 16 * TN + 4 * ((4 * i + g) ^ mix(r))) = acc[i][j];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int t = 0; t < 16 / kRowsPer; ++t) {
            const int br = t * kRowsPer + lane / kLanesPerRow;
            const int mm = m0 + wm + 16 * j + br;
            const i32x4 sum = *reinterpret_cast<const i32x4*>(area + br * 16 * TN + 4 * (chunk ^ mix(br)));
            if (mm < m && count > 0) {
                const float sx = xs[mm];
                f32x4 v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = (float)sum[e] * sx * sw[e] + bb[e];
                store4<kBf16Out>(y, (int64_t)mm * n + nn, v, count);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

template <int kWN, int kWM, int TN, int TM, int NS>
hipError_t launch_tile(const int8_t* x, const float* xs, const int8_t* w, const float* ws, const float* bias, void* y,
                       bool out_bf16, int64_t m, int64_t n, int64_t k, hipStream_t stream) {
    constexpr int NR = 16 * TN * kWN, MR = 16 * TM * kWM;
    const int64_t tiles = ((n + NR - 1) / NR) * ((m + MR - 1) / MR);
    const dim3 grid = grid_of((tiles + kXcds - 1) / kXcds * kXcds);
    constexpr int kGroupM = 4;
    if (out_bf16)
        int8_gemm_tile_kernel<kWN, kWM, TN, TM, NS, true>
            <<<grid, kWave * kWN * kWM, 0, stream>>>(x, xs, w, ws, bias, y, (int)m, (int)n, (int)k, tiles, kGroupM);
    else
        int8_gemm_tile_kernel<kWN, kWM, TN, TM, NS, false>
            <<<grid, kWave * kWN * kWM, 0, stream>>>(x, xs, w, ws, bias, y, (int)m, (int)n, (int)k, tiles, kGroupM);
    return hipGetLastError();
}

// Tile shapes and what one 128-column step of a tile takes with every compute unit busy (us, int8 codes of
// normal values; the two large ones at the clock the chip keeps under that load). The shape whose rounds of
// tiles over the compute units sum to the least is taken. Measured against it (us; 256 x 256, 256 x 128,
// 128 x 128, 64 x 128, 64 x 64 rows of w x x):
//   m 256,  n 4096,  k 4096:   49.0  29.9  23.3  15.5  10.9      m 128, n 14336, k 4096:  57.7  37.5  29.8  22.7  27.1
//   m 512,  n 4096,  k 4096:   49.5  30.3  24.1  16.6  19.3      m 256, n 14336, k 4096:  58.7  37.2  29.7  36.7  48.2
//   m 1024, n 4096,  k 4096:   50.5  30.9  25.5  30.7  36.1      m 512, n 14336, k 4096:  60.0  39.0  53.9  68.6  80.2
//   m 1024, n 14336, k 4096:   64.5  74.0  102.8 117.8 156.8     m 8192, n 8192, k 8192:  441   529   -     -     -
struct TileShape {
    int rows_w, rows_x;
    float step_us;
    hipError_t (*launch)(const int8_t*, const float*, const int8_t*, const float*, const float*, void*, bool, int64_t,
                         int64_t, int64_t, hipStream_t);
};
constexpr float kTileFixedUs = 2.5f;   // a round's first requests and its stores

const TileShape kShapes[] = {
    {256, 256, 1.6f, launch_tile<2, 4, 8, 4, 2>},
    {256, 128, 0.95f, launch_tile<4, 2, 4, 4, 3>},
    {128, 128, 0.66f, launch_tile<2, 2, 4, 4, 4>},
    {64, 128, 0.47f, launch_tile<2, 2, 2, 4, 6>},
    {64, 64, 0.28f, launch_tile<2, 2, 2, 2, 8>},
};

}  // namespace

hipError_t launch_int8_gemm(const int8_t* x, const float* x_scale, const int8_t* w, const float* w_scale,
                            const float* bias, void* y, bool out_bf16, int64_t m, int64_t n, int64_t k,
                            hipStream_t stream) {
    const int64_t steps = (k + 127) / 128;
    if (m <= 16) {
        const int waves = steps >= 64 ? 16 : steps >= 16 ? 8 : 4;
        return launch_split<1, 1>(x, x_scale, w, w_scale, bias, y, out_bf16, m, n, k, waves, stream);
    }
    const int64_t cus = device_cu_count();
    const TileShape* best = nullptr;
    float best_us = 0.f;
    for (const TileShape& s : kShapes) {
        const int64_t tiles = ((n + s.rows_w - 1) / s.rows_w) * ((m + s.rows_x - 1) / s.rows_x);
        const float us = (float)((tiles + cus - 1) / cus) * ((float)steps * s.step_us + kTileFixedUs);
        if (best == nullptr || us < best_us) {
            best = &s;
            best_us = us;
        }
    }
    return best->launch(x, x_scale, w, w_scale, bias, y, out_bf16, m, n, k, stream);
}

}  // namespace e2m1
