// int8_gemm.hip -- product of two int8 matrices with a scale per token and per
// output channel (int8_gemm).
//
// Mathematics: y[m][n] = (sum_k x[m][k] w[n][k]) x_scale[m] w_scale[n] + bias[n].
// The sum is exact: int8 products in int32 accumulators (|sum| <= 2^14 k, below
// 2^31 for k <= 131056). It is rounded to fp32 once, then multiplied by x_scale
// in fp32, by w_scale with the bias added in one fma, and rounded to the output
// type.
//
// gfx950 design. Few rows of x: the bytes of w bound the product, which are read
// at 5.3 to 5.6 TB/s (us in a graph: 4096 x 14336 10.6 for one row of x, 11.1 for
// 16; a plain read of the same bytes takes 8.8). The stream form takes it where
// its tiles of 16 or 32 rows of w are about one round over the compute units, 64
// x 64 tiles of the tile form where w has more rows (14336 x 4096, one row of x:
// 10.8, with 32 x 32 stream tiles 11.1, with 16 x 16 ones 11.7). Many rows: the
// matrix cores' work bounds it from below. A step of a 256 x 256 tile (128
// columns) takes 3200 cycles, 2050 of which its matrix instructions fill, at 1.6
// to 2.0 GHz: with the operands of real matrices the power limit lowers the clock
// (operands of zero: 2.4 GHz, 3550 cycles). 16x16x64 tiles take less energy
// than 32x32x32 ones (matrix cores alone, normal codes: 4.09 against 3.42 POP/s;
// 8192^3: 441 against 494 us), so they are used throughout: 8192^3 takes 430 to
// 450 us, 2048 x 28672 x 4096 217 to 226. Both forms feed the matrix cores from
// LDS rings that direct-to-LDS loads fill in 128-byte row segments (64-byte ones
// read at half the L2 rate: 66 against 130 GB/s a compute unit). What bounds the
// tiles in between is LDS traffic and a step's latency.
#include "device.hpp"
#include "kernels.hpp"

namespace e2m1 {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kOutOfRange = 0xFFFFFFF0u;   // a buffer offset past any resource's range

typedef float f32x2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

// bf16 patterns of two floats, nearest even, in the conversion instruction
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2v{lo, hi}), bf16x2v));
}

// One output. The same in every form, so that a row of y has the same bits whatever the other rows and their number.
__device__ __forceinline__ float output(int32_t sum, float sx, float sw, float bias) {
    return fmaf((float)sum * sx, sw, bias);
}

// v's first `count` (at most four) values to y from element idx on.
template <bool kBf16Out>
__device__ __forceinline__ void store4(void* y, int64_t idx, const f32x4& v, int count) {
    if constexpr (kBf16Out) {
        uint16_t* p = reinterpret_cast<uint16_t*>(y) + idx;
        if (count == 4 && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
            *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        } else {
            for (int j = 0; j < count; ++j) p[j] = (uint16_t)pack_bf16(v[j], 0.f);
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

// ----------------------------------------------------------- direct to LDS --

// the lane's 16 bytes at byte offset voff of the buffer -> LDS lds + 16 * lane (M0 is set here and used
// by nothing else in these kernels)
__device__ __forceinline__ void lds_load16(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(lds), "v"(voff), "s"(rsrc) : "memory");
}

// the lane's 4 bytes at p -> LDS lds + 4 * lane, active lanes only
__device__ __forceinline__ void lds_load4(const float* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" :: "s"(lds), "v"(p) : "memory");
}

// At most kN of this wave's requests are in flight.
template <int kN>
__device__ __forceinline__ void wait_vm() {
    asm volatile("s_waitcnt vmcnt(%0)" :: "n"(kN) : "memory");
}

// This wave's LDS accesses are done.
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// `tiles` workgroups (below 2^32) in rows of 2^20 (a grid dimension holds fewer than 2^32 threads).
dim3 grid_of(int64_t tiles) {
    const int64_t gx = tiles < (1 << 20) ? tiles : 1 << 20;
    return dim3((unsigned)gx, (unsigned)((tiles + gx - 1) / gx));
}

// ----------------------------------------------------------- stream form --
// For few rows of x: the weights' bytes bound it, so the kernel is a stream
// of w. A workgroup takes a tile of 16 NT rows of w x 16 MT rows of x. Its W
// waves split K, a run of 128-column steps each (runs spread a workgroup's
// requests over the row, and so over the memory channels: with the steps dealt
// out one by one, every workgroup is at the same columns of rows that lie 4096
// bytes apart, and 14336 x 4096 took 13.2 us in this form instead of 11.8).
// Each wave has an LDS ring of its own (kStages steps of its rows of w and of
// x, filled by direct-to-LDS requests of 8 rows x 128 bytes), so that no wave
// waits for another before the end. Lane 16 g + r takes columns 16 g .. + 15 of row r of
// a 64-column half step; 16x16x64 matrix-core tiles, A = w, B = x. The waves'
// sums meet in LDS. (Workgroups that go on to further tiles, with the requests
// of the next under way while one ends, measured the same.)

// Ring stages of a wave. Three or four, with one workgroup on a compute unit instead of two, measured 2 to 10 % slower.
// (By lines a step reads the next stage too, and there are three.)
template <bool kLines>
constexpr int kStagesOf = kLines ? 3 : 2;

// Chunks (16 bytes) by which row `row` of a matrix of `chunks` chunks a row at p starts past a 128-byte line.
__device__ __forceinline__ int past_line(const int8_t* p, uint32_t row, uint32_t chunks) {
    return (int)(((uint32_t)((uintptr_t)p / 16) + row * chunks) & 7);
}

// Column `col` (of 128) of a row's next 128, or the one 128 before it, if that is in the line where these start.
__device__ __forceinline__ int in_line(int col, int past) { return col / 16 + past >= 8 ? col - 128 : col; }

template <int W, int NT, int MT, bool kLines, bool kBf16Out>
__global__ __launch_bounds__(kWave * W) void int8_gemm_stream_kernel(
    const int8_t* __restrict__ x, const float* __restrict__ xs, const int8_t* __restrict__ w,
    const float* __restrict__ ws, const float* __restrict__ bias, void* __restrict__ y, int m, int n, int k,
    int tiles_n, int tiles_m) {
    constexpr int kStages = kStagesOf<kLines>;
    constexpr int kRequests = 2 * (NT + MT);            // 1 KB each: eight rows of w or of x
    constexpr int kStage = 1024 * kRequests;
    constexpr int kQuads = NT * MT;                     // 64 quads (four outputs) each
    static_assert(kQuads <= W && MT <= 2, "one block a wave, its scales in 64 lanes");
    __shared__ __attribute__((aligned(256))) uint8_t lds[W * kStages * kStage + (W - 1) * kQuads * 1024 + W * 256];
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, g = lane >> 4;
    // tiles along w first, then along x
    const uint32_t tile = blockIdx.y * gridDim.x + blockIdx.x;
    const int tile_m = __builtin_amdgcn_readfirstlane(tile / (uint32_t)tiles_n);
    if (tile_m >= tiles_m) return;                      // the grid's last row may run past the tiles
    const int n0 = (int)(tile - (uint32_t)tile_m * (uint32_t)tiles_n) * 16 * NT, m0 = tile_m * 16 * MT;
    // rows past n or m are out of range: zeros, no memory access
    const __amdgpu_buffer_rsrc_t wres = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t*>(w + (int64_t)n0 * k), 0, min(16 * NT, n - n0) * k, kBufferWord3);
    const __amdgpu_buffer_rsrc_t xres = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t*>(x + (int64_t)m0 * k), 0, min(16 * MT, m - m0) * k, kBufferWord3);
    const int steps = (k + 127) / 128;
    const int per = max((steps + W - 1) / W, 1);        // steps of a wave: wave * per on (some may lie past K)
    uint8_t* const ring = lds + wave * kStages * kStage;
    const uint32_t base = (uint32_t)(uintptr_t)ring;

    // request j of an operand fills rows 8 j .. + 7: lane l slot l % 8 of row l / 8, which holds chunk
    // l % 8 ^ (row / 2 % 8), so that an operand read (16 rows, one chunk) meets every LDS bank once
    const int col = 16 * ((lane % 8) ^ (lane >> 4));
    const uint32_t off = (uint32_t)(lane / 8) * (uint32_t)k;
    const uint32_t chunks = (uint32_t)k / 16;           // of a row
    const int pastw = kLines ? past_line(w, lane / 8, chunks) : 0, pastx = kLines ? past_line(x, lane / 8, chunks) : 0;
    auto issue = [&](int st) __attribute__((always_inline)) {
        const int c0 = 128 * (wave * per + st);
        const bool live = st < per + (kLines ? 1 : 0);
        auto from = [&](int c, int past) __attribute__((always_inline)) {
            const int at = c0 + (kLines ? in_line(c, past) : c);
            return live && (uint32_t)at < (uint32_t)k ? off + (uint32_t)at : kOutOfRange;
        };
        const uint32_t evenw = from(col, pastw), oddw = from(col ^ 64, pastw);
        const uint32_t evenx = kLines ? from(col, pastx) : evenw, oddx = kLines ? from(col ^ 64, pastx) : oddw;
        const uint32_t into = base + (st % kStages) * kStage;
#pragma unroll
        for (int j = 0; j < kRequests; ++j) {
            const bool of_w = j < 2 * NT;
            const int jj = of_w ? j : j - 2 * NT;
            const uint32_t o = of_w ? (j & 1 ? oddw : evenw) : (j & 1 ? oddx : evenx);
            // (selected once more: "out of range" plus a row offset would wrap)
            const uint32_t v = jj == 0 || o == kOutOfRange ? o : o + (uint32_t)(8 * jj) * (uint32_t)k;
            lds_load16(of_w ? wres : xres, v, __builtin_amdgcn_readfirstlane(into + 1024u * (uint32_t)j));
        }
    };

#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);
    // Wave b < kQuads adds up block b. Its scales and biases are requested like the operands (a wait for a vector
    // load would wait for the whole ring too): w_scale of the block's 16 rows in lanes 0 .. 15, bias in 16 .. 31,
    // x_scale of the tile's rows of x from lane 32 on. They have landed when the last step's rows have.
    uint8_t* const areas = lds + W * kStages * kStage;
    const float* const sc = reinterpret_cast<const float*>(areas + (W - 1) * kQuads * 1024 + wave * 256);
    if (wave < kQuads) {
        const int c = n0 + 16 * (wave / MT) + (lane & 15), row = m0 + (lane & 31);
        const uint32_t into = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)sc);
        const float* p = lane < 16 ? ws : bias;
        if (lane < 32 && c < n && p != nullptr) lds_load4(p + c, into);
        if (lane >= 32 && row < m) lds_load4(xs + row, into);
    }

    const int slot[2] = {r * 128 + 16 * (g ^ (r >> 1)), r * 128 + 16 * ((4 + g) ^ (r >> 1))};
    // whether chunk 4 h + g of the lane's row of w or x lies in the next stage
    const int fromw = kLines ? g + past_line(w, r, chunks) : 0, fromx = kLines ? g + past_line(x, r, chunks) : 0;
    i32x4 acc[NT][MT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    for (int s = 0; s < per; ++s) {
        issue(s + kStages - 1);                   // into the slot read in the last turn of this loop
        wait_vm<kRequests>();                     // this step's rows (by lines, the next one's) are in LDS
        const int here = (s % kStages) * kStage, next = ((s + 1) % kStages) * kStage;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t* pw = ring + (kLines && fromw + 4 * h >= 8 ? next : here) + slot[h];
            const uint8_t* px = ring + (kLines && fromx + 4 * h >= 8 ? next : here) + slot[h];
            i32x4 a[NT], b[MT];
#pragma unroll
            for (int i = 0; i < NT; ++i) a[i] = *reinterpret_cast<const i32x4*>(pw + 2048 * i);
#pragma unroll
            for (int j = 0; j < MT; ++j) b[j] = *reinterpret_cast<const i32x4*>(px + 2048 * (NT + j));
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], b[j], acc[i][j], 0, 0, 0);
        }
        wait_lds();                               // read: the slot may be filled again
    }

    i32x4 sum = {0, 0, 0, 0};
    uint8_t* const part = areas + lane * 16;      // [block][the other waves][lane]
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int block = i * MT + j;
            if (wave == block) sum = acc[i][j];
            else
                *reinterpret_cast<i32x4*>(part + 1024 * (block * (W - 1) + wave - (wave > block))) = acc[i][j];
        }
    wait_vm<0>();   // the requests past the last step have landed before the workgroup's LDS is released
    wait_lds();
    __syncthreads();
    if (wave >= kQuads) return;
#pragma unroll
    for (int v = 0; v < W - 1; ++v) sum += *reinterpret_cast<const i32x4*>(part + 1024 * (wave * (W - 1) + v));
    const f32x4 sw = *reinterpret_cast<const f32x4*>(sc + 4 * g);
    const f32x4 sb = *reinterpret_cast<const f32x4*>(sc + 16 + 4 * g);
    const float sx = sc[32 + 16 * (wave % MT) + r];
    const int mm = m0 + 16 * (wave % MT) + r, nn = n0 + 16 * (wave / MT) + 4 * g;
    if (mm >= m || nn >= n) return;
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = output(sum[e], sx, sw[e], bias != nullptr ? sb[e] : 0.f);
    store4<kBf16Out>(y, (int64_t)mm * n + nn, v, min(4, n - nn));
}

template <int W, int NT, int MT, bool kLines>
hipError_t launch_stream(const int8_t* x, const float* xs, const int8_t* w, const float* ws, const float* bias,
                         void* y, bool out_bf16, int64_t m, int64_t n, int64_t k, hipStream_t stream) {
    const int64_t tiles_n = (n + 16 * NT - 1) / (16 * NT), tiles_m = (m + 16 * MT - 1) / (16 * MT);
    const dim3 grid = grid_of(tiles_n * tiles_m);
    if (out_bf16)
        int8_gemm_stream_kernel<W, NT, MT, kLines, true><<<grid, kWave * W, 0, stream>>>(
            x, xs, w, ws, bias, y, (int)m, (int)n, (int)k, (int)tiles_n, (int)tiles_m);
    else
        int8_gemm_stream_kernel<W, NT, MT, kLines, false><<<grid, kWave * W, 0, stream>>>(
            x, xs, w, ws, bias, y, (int)m, (int)n, (int)k, (int)tiles_n, (int)tiles_m);
    return hipGetLastError();
}

// ------------------------------------------------------------- tile form --
// A workgroup owns a tile of 16 TN kWN rows of w x 16 TM kWM rows of x; each of
// its kWN x kWM waves 16 TN x 16 TM of it in 16x16x64 matrix-core tiles (A = w, B = x).
// K goes in steps of KS columns through a ring of NS LDS buffers that the
// memory pipeline fills itself (buffer_load ... lds: no registers, no LDS
// writes by the waves). In LDS a row's 16-byte chunks are permuted by the row,
// so that an operand read (16 rows, one chunk) meets every bank once; the
// requests' source addresses do that, as the LDS side of a request is contiguous.
// Operands are read one 64-column slice ahead of their MFMAs, over the step's
// border too: before the last slice's MFMAs of step s a wave waits until its own
// reads of the buffer and its requests of step s + 1 are done, passes the step's
// one barrier (with the previous slice's MFMAs still running), requests step s +
// NS into the buffer that is now free and reads the first slice of step s + 1.
// Rows that start inside a 128-byte line (k no multiple of 128) would have every
// request of a row touch two lines, a third of the time in mid-sized products.
// By lines (kLines), a request takes the row's line instead, so a step's chunks
// lie in its own buffer and the next one: the chunk's slot stays as it is, only
// the buffer depends on how far into a line the row starts, which is the same
// for all rows of a lane's operands of x, and one of two values for w.
// A lane's sums of two operands of w are eight neighbouring columns of y, which
// it scales and stores at once (through LDS instead, 4096 x 4096 x 512 took 17.5
// us, so 16.3). Stores past the caches (nontemporal) took 58 us where these take
// 57 (4096 x 4096 x 4096), and leave y for the next operator to fetch.
// Waves: as many as the registers and pairs of operands allow, though small ones
// read an operand from LDS more often; a step's latency (barrier, LDS reads,
// matrix instructions) is hidden by the other waves alone. 130 x 4096 x 4096 in
// 64 x 64 tiles: 13.0 us with two waves, 10.7 with four, 9.2 with eight (8.4 to
// 8.9 with the later steps); one round of 128 x 128 tiles of 4096 columns 35.6,
// 22.4 and, with sixteen, 15.7. A workgroup alone on its compute unit passes 38
// LDS bytes a cycle for them (64 x 64: 16 KB in 430 cycles at 2.2 GHz); the
// direct-to-LDS path at most 64. Ring buffers:
// as few as let a second workgroup onto the compute unit (64 x 64 with eight
// instead of four: 512 x 4096 x 4096 18.2 instead of 15.8 us).

// This wave's LDS reads are done and at most kN of its requests are in flight; then the workgroup's barrier.
template <int kN>
__device__ __forceinline__ void step_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(kN) : "memory");
}

constexpr int kXcds = 8;

constexpr int KS = 128;   // columns per step: two slices (64-byte row segments read at half the L2 rate)

template <int kWN, int kWM, int TN, int TM, int NS>
constexpr int tile_lds_bytes() {   // the ring; w_scale, bias and x_scale of the tile's rows
    return NS * 16 * (TN * kWN + TM * kWM) * KS + 4 * 16 * (2 * TN * kWN + TM * kWM);
}

// The tile from row n0 of w and row m0 of x on.
template <int kWN, int kWM, int TN, int TM, int NS, bool kLines, bool kBf16Out>
__device__ __forceinline__ void tile_body(uint8_t* lds, const int8_t* __restrict__ x, const float* __restrict__ xs,
                                          const int8_t* __restrict__ w, const float* __restrict__ ws,
                                          const float* __restrict__ bias, void* __restrict__ y, int m, int n, int k,
                                          int n0, int m0) {
    constexpr int kWaves = kWN * kWM;
    constexpr int NR = 16 * TN * kWN, MR = 16 * TM * kWM;
    constexpr int kWLoads = NR / 8 / kWaves, kXLoads = MR / 8 / kWaves;   // 1 KB requests (8 rows) per wave and step
    constexpr int kSlices = KS / 64;
    static_assert(kWLoads * 8 * kWaves == NR && kXLoads * 8 * kWaves == MR, "requests");
    constexpr int kBufBytes = (NR + MR) * KS;
    constexpr int kOutBytes = 16 * 16 * TN * 4;                           // a wave's band of sums
    static_assert(kWaves * kOutBytes <= NS * kBufBytes && tile_lds_bytes<kWN, kWM, TN, TM, NS>() <= 160 * 1024, "LDS");
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, g = lane >> 4;
    const int wn = (wave % kWN) * 16 * TN, wm = (wave / kWN) * 16 * TM;
    const int nt = min(NR, n - n0), mt = min(MR, m - m0);
    const __amdgpu_buffer_rsrc_t wres = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t*>(w + (int64_t)n0 * k), 0, nt * k, kBufferWord3);
    const __amdgpu_buffer_rsrc_t xres = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t*>(x + (int64_t)m0 * k), 0, mt * k, kBufferWord3);

    // request q of an operand fills rows 8 q .. + 7; lane l fills slot l % 8 of row l / 8, whose chunk is
    // l % 8 ^ (row / 2 % 8) for x and l % 8 ^ (2 (row / 8 % 4) + row / 2 % 2) for w; by lines, it is a chunk of the
    // step before if this one lies in the row's next line. Rows past the matrix and columns outside [0, k) read out of
    // range: zeros, no memory access.
    const uint32_t chunks = (uint32_t)k / 16;            // of a row
    auto past = [&](const int8_t* p, uint32_t row) __attribute__((always_inline)) {
        return kLines ? past_line(p, row, chunks) : 0;
    };
    const int colx = 16 * ((lane % 8) ^ (lane >> 4)), colw = 16 * ((lane % 8) ^ (lane >> 4 & 1));
    const int pastx = past(x, lane / 8), pastw = past(w, lane / 8);
    auto wcol = [&](int i) __attribute__((always_inline)) {
        const int col = colw ^ (32 * ((kWLoads * wave + i) & 3));
        return kLines ? in_line(col, pastw) : col;
    };
    auto xcol = [&](int i) __attribute__((always_inline)) {
        const int col = colx ^ (64 * ((kXLoads * wave + i) & 1));
        return kLines ? in_line(col, pastx) : col;
    };
    uint32_t woff[kWLoads], xoff[kXLoads];
#pragma unroll
    for (int i = 0; i < kWLoads; ++i)
        woff[i] = (uint32_t)(8 * (kWLoads * wave + i) + lane / 8) * (uint32_t)k + (uint32_t)wcol(i);
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
        xoff[i] = (uint32_t)(8 * (kXLoads * wave + i) + lane / 8) * (uint32_t)k + (uint32_t)xcol(i);
    const uint32_t base = (uint32_t)(uintptr_t)&lds[0];
    const int steps = (k + KS - 1) / KS;

    // w_scale [NR], bias [NR], x_scale [MR]: requested like the operands and before them, so landed with the first
    // step (loads in the epilogue would wait for its stores: their count is one)
    float* const factors = reinterpret_cast<float*>(lds + NS * kBufBytes);
    for (int q = wave; q < (2 * NR + MR + kWave - 1) / kWave; q += kWaves) {
        const int at = kWave * q + lane;
        const bool of_w = at < NR, of_bias = !of_w && at < 2 * NR;
        const int row = of_w ? at : of_bias ? at - NR : at - 2 * NR;
        const float* const from = of_w ? ws + n0 : of_bias ? bias + n0 : xs + m0;
        if ((!of_bias || bias != nullptr) && row < (of_w || of_bias ? nt : mt))   // mt <= MR: nor past the area
            lds_load4(from + row, __builtin_amdgcn_readfirstlane(base + NS * kBufBytes + 4u * kWave * (uint32_t)q));
    }

    auto issue = [&](int st, int b) __attribute__((always_inline)) {
        const int c0 = st * KS;   // below 2^18: st <= steps + NS
        const uint32_t at = base + b * kBufBytes;
#pragma unroll
        for (int i = 0; i < kWLoads; ++i)   // columns (and whole steps) past K too
            lds_load16(wres, (uint32_t)(c0 + wcol(i)) < (uint32_t)k ? woff[i] + (uint32_t)c0 : kOutOfRange,
                       __builtin_amdgcn_readfirstlane(at + 1024u * (uint32_t)(kWLoads * wave + i)));
#pragma unroll
        for (int i = 0; i < kXLoads; ++i)
            lds_load16(xres, (uint32_t)(c0 + xcol(i)) < (uint32_t)k ? xoff[i] + (uint32_t)c0 : kOutOfRange,
                       __builtin_amdgcn_readfirstlane(at + NR * KS + 1024u * (uint32_t)(kXLoads * wave + i)));
    };
    // Operand i of w takes rows 32 (i / 2) + 8 (r / 4) + 4 (i % 2) + r % 4 of the wave's, so that a lane's sums of two
    // operands are eight neighbouring columns of y; operand j of x rows 16 j + r.
    static_assert(TN % 2 == 0, "operands of w in pairs");
    const uint8_t* wrow = lds + (wn + 8 * (r >> 2) + (r & 3)) * KS;
    const uint8_t* xrow = lds + NR * KS + (wm + r) * KS;
    // chunk 4 q + g of a row that starts `chunks_past` into a line: in the next step's buffer where it is past the line
    struct Place { int here, last; };   // from the buffer of the step; of the ring's last buffer
    auto place = [&](int q, int chunks_past) __attribute__((always_inline)) {
        const int at = 16 * ((4 * q + g) ^ (r >> 1)), next = (4 * q + g + chunks_past) >> 3;
        return Place{at + next * kBufBytes, at - next * (NS - 1) * kBufBytes};
    };
    Place wat[kLines ? 2 : 1][kSlices], xat[kSlices];
#pragma unroll
    for (int q = 0; q < kSlices; ++q) {
        xat[q] = place(q, past(x, r));
#pragma unroll
        for (int h = 0; h < (kLines ? 2 : 1); ++h) wat[h][q] = place(q, past(w, (r & 3) + 4 * h));
    }
    auto read_w = [&](int b, int q, int i) __attribute__((always_inline)) {
        const Place& p = wat[kLines ? i % 2 : 0][q];
        return *reinterpret_cast<const i32x4*>(wrow + (b == NS - 1 ? p.last : p.here) +
                                               (b * kBufBytes + (32 * (i / 2) + 4 * (i % 2)) * KS));
    };
    auto read_x = [&](int b, int q, int j) __attribute__((always_inline)) {
        const Place& p = xat[q];
        return *reinterpret_cast<const i32x4*>(xrow + (b == NS - 1 ? p.last : p.here) + (b * kBufBytes + 16 * j * KS));
    };

    i32x4 a[TN], c[2][TM];
    i32x4 acc[TN][TM];
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

    constexpr int kPerStep = kWLoads + kXLoads;
    constexpr int kAhead = kLines ? 1 : 0;   // a step reads the next buffer too
    static_assert(NS >= 2 + kAhead, "ring");
#pragma unroll
    for (int st = 0; st < NS; ++st) issue(st, st);
    step_barrier<kPerStep*(NS - 1 - kAhead)>();
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
                    step_barrier<kPerStep*(NS - 2 - kAhead)>();
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
    // lane 16 g + r holds in acc[i][j], of row wm + 16 j + r of x, columns wn + 32 (i / 2) + 8 g + 4 (i % 2) on of y
    if (n % 4 == 0 && (reinterpret_cast<uintptr_t>(y) & (kBf16Out ? 7 : 15)) == 0) {
        const bool wide = kBf16Out && n % 8 == 0 && (reinterpret_cast<uintptr_t>(y) & 15) == 0;
        float sx[TM];
#pragma unroll
        for (int j = 0; j < TM; ++j) sx[j] = factors[2 * NR + wm + 16 * j + r];
#pragma unroll
        for (int i = 0; i < TN; i += 2) {
            const int row = wn + 16 * i + 8 * g, nn = n0 + row;
            float sw[8], bb[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sw[e] = factors[row + e];
                bb[e] = bias != nullptr ? factors[NR + row + e] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < TM; ++j) {
                const int mm = m0 + wm + 16 * j + r;
                f32x4 v[2];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e / 4][e % 4] = output(acc[i + e / 4][j][e % 4], sx[j], sw[e], bb[e]);
                if (mm < m && nn < n) {
                    const int64_t at = (int64_t)mm * n + nn;
                    if (wide) {
                        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(y) + at) =
                            make_uint4(pack_bf16(v[0][0], v[0][1]), pack_bf16(v[0][2], v[0][3]),
                                       pack_bf16(v[1][0], v[1][1]), pack_bf16(v[1][2], v[1][3]));
                    } else {
                        store4<kBf16Out>(y, at, v[0], 4);
                        if (nn + 4 < n) store4<kBf16Out>(y, at + 4, v[1], 4);
                    }
                }
            }
        }
        wait_vm<0>();   // the requests past the last step have landed before the workgroup's LDS is released
        return;
    }
    // Rows of y off the vector's alignment leave through LDS, one 16-row band of x at a time in an area of the wave's
    // own, its chunks permuted like the operands', to be stored side by side across the lanes (2048 x 4097 x 512:
    // 28.7 us with four a lane, stored one by one, 24.1 so; 2048 x 4100 x 512, in vectors: 19.0).
    step_barrier<0>();   // every request has landed and every read is done: the buffers are free
    auto mix = [](int row) __attribute__((always_inline)) { return TN >= 4 ? row : row >> 1; };
    constexpr int kSide = 16 * TN < kWave ? 16 * TN : kWave;
    constexpr int kSides = 16 * TN / kSide;
    float* area = reinterpret_cast<float*>(lds + wave * kOutBytes);
    float sw[kSides], bb[kSides];
#pragma unroll
    for (int e = 0; e < kSides; ++e) {
        const int row = wn + lane % kSide + kSide * e;
        sw[e] = factors[row];
        bb[e] = bias != nullptr ? factors[NR + row] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < TM; ++j) {
        const float sx = factors[2 * NR + wm + 16 * j + r];
#pragma unroll
        for (int i = 0; i < TN; ++i) {
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][j][e] * sx;
            *reinterpret_cast<f32x4*>(area + r * 16 * TN + 4 * ((8 * (i / 2) + 2 * g + i % 2) ^ mix(r))) = v;
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll 4
        for (int t = 0; t < 16 * kSide / kWave; ++t) {
            const int br = t * (kWave / kSide) + lane / kSide;
            const int mm = m0 + wm + 16 * j + br;
#pragma unroll
            for (int e = 0; e < kSides; ++e) {
                const int c = lane % kSide + kSide * e;
                const float v = fmaf(area[br * 16 * TN + 4 * ((c / 4) ^ mix(br)) + c % 4], sw[e], bb[e]);   // output()
                const int64_t at = (int64_t)mm * n + (n0 + wn + c);
                if (mm < m && n0 + wn + c < n) {
                    if constexpr (kBf16Out) reinterpret_cast<uint16_t*>(y)[at] = (uint16_t)pack_bf16(v, 0.f);
                    else reinterpret_cast<float*>(y)[at] = v;
                }
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// Tiles along x that workgroups of one XCD take before they go on along w.
constexpr int kBand = 4;

// First rows of tile `tile` (rows_w x rows_x of them each), numbered along x inside bands of kBand tiles, then along w.
__device__ __forceinline__ void tile_rows(uint32_t tile, int m, int n, int rows_w, int rows_x, int& n0, int& m0) {
    const uint32_t tn = (uint32_t)(n + rows_w - 1) / (uint32_t)rows_w;
    const uint32_t tm = (uint32_t)(m + rows_x - 1) / (uint32_t)rows_x;
    const uint32_t band = tile / (kBand * tn), in = tile - band * (kBand * tn);
    const uint32_t size = min((uint32_t)kBand, tm - band * kBand);
    n0 = __builtin_amdgcn_readfirstlane(in / size * (uint32_t)rows_w);
    m0 = __builtin_amdgcn_readfirstlane((band * kBand + in % size) * (uint32_t)rows_x);
}

// Workgroup id -> number: ids go round the XCDs, and each XCD gets a run of neighbouring numbers, whose tiles share
// operands in its L2. Not below count: no work.
__device__ __forceinline__ uint32_t xcd_number(uint32_t id, uint32_t count) {
    const uint32_t per = (count + kXcds - 1) / kXcds;
    return id / kXcds < per ? id % kXcds * per + id / kXcds : count;
}

template <int kWN, int kWM, int TN, int TM, int NS, bool kLines, bool kBf16Out>
__global__ __launch_bounds__(kWave * kWN * kWM) void int8_gemm_tile_kernel(
    const int8_t* __restrict__ x, const float* __restrict__ xs, const int8_t* __restrict__ w,
    const float* __restrict__ ws, const float* __restrict__ bias, void* __restrict__ y, int m, int n, int k,
    uint32_t tiles) {
    __shared__ __attribute__((aligned(256))) uint8_t lds[tile_lds_bytes<kWN, kWM, TN, TM, NS>()];
    const uint32_t tile = xcd_number(blockIdx.y * gridDim.x + blockIdx.x, tiles);
    if (tile >= tiles) return;   // the whole workgroup
    int n0, m0;
    tile_rows(tile, m, n, 16 * TN * kWN, 16 * TM * kWM, n0, m0);
    tile_body<kWN, kWM, TN, TM, NS, kLines, kBf16Out>(lds, x, xs, w, ws, bias, y, m, n, k, n0, m0);
}

// 256 x 256 tiles whose last round would leave at least half of the compute units idle: the last tiles, those from
// `whole` on, as two halves of 256 x 128 each. 2048 x 28672 x 4096 (896 tiles on 256 compute units): 239 us with
// whole tiles, 219 with 128 of them halved.
template <bool kBf16Out>
__global__ __launch_bounds__(512) void int8_gemm_mixed_kernel(
    const int8_t* __restrict__ x, const float* __restrict__ xs, const int8_t* __restrict__ w,
    const float* __restrict__ ws, const float* __restrict__ bias, void* __restrict__ y, int m, int n, int k,
    uint32_t tiles, uint32_t whole) {
    constexpr int kLds = tile_lds_bytes<2, 4, 8, 4, 2>() > tile_lds_bytes<4, 2, 4, 4, 3>()
                             ? tile_lds_bytes<2, 4, 8, 4, 2>() : tile_lds_bytes<4, 2, 4, 4, 3>();
    __shared__ __attribute__((aligned(256))) uint8_t lds[kLds];
    const uint32_t id = blockIdx.y * gridDim.x + blockIdx.x;
    const uint32_t ids = (whole + kXcds - 1) / kXcds * kXcds;   // of the whole tiles
    int n0, m0;
    if (id < ids) {
        const uint32_t tile = xcd_number(id, whole);
        if (tile >= whole) return;   // the whole workgroup
        tile_rows(tile, m, n, 256, 256, n0, m0);
        tile_body<2, 4, 8, 4, 2, false, kBf16Out>(lds, x, xs, w, ws, bias, y, m, n, k, n0, m0);
    } else {
        const uint32_t half = xcd_number(id - ids, 2 * (tiles - whole));
        if (half >= 2 * (tiles - whole)) return;
        tile_rows(whole + half / 2, m, n, 256, 256, n0, m0);
        m0 += 128 * (int)(half % 2);
        if (m0 >= m) return;
        tile_body<4, 2, 4, 4, 3, false, kBf16Out>(lds, x, xs, w, ws, bias, y, m, n, k, n0, m0);
    }
}

template <int kWN, int kWM, int TN, int TM, int NS, bool kLines>
hipError_t launch_tile(const int8_t* x, const float* xs, const int8_t* w, const float* ws, const float* bias, void* y,
                       bool out_bf16, int64_t m, int64_t n, int64_t k, hipStream_t stream) {
    constexpr int NR = 16 * TN * kWN, MR = 16 * TM * kWM;
    const int64_t tiles = ((n + NR - 1) / NR) * ((m + MR - 1) / MR);
    const dim3 grid = grid_of((tiles + kXcds - 1) / kXcds * kXcds);
    if (out_bf16)
        int8_gemm_tile_kernel<kWN, kWM, TN, TM, NS, kLines, true>
            <<<grid, kWave * kWN * kWM, 0, stream>>>(x, xs, w, ws, bias, y, (int)m, (int)n, (int)k, (uint32_t)tiles);
    else
        int8_gemm_tile_kernel<kWN, kWM, TN, TM, NS, kLines, false>
            <<<grid, kWave * kWN * kWM, 0, stream>>>(x, xs, w, ws, bias, y, (int)m, (int)n, (int)k, (uint32_t)tiles);
    return hipGetLastError();
}

// Whether the last of several rounds of 256 x 256 tiles fills at most half of the compute units.
bool halves_last_round(int64_t tiles, int64_t cus) {
    return tiles > cus && tiles % cus != 0 && 2 * (tiles % cus) <= cus;
}

// 256 x 256 tiles, such a last round's halved.
hipError_t launch_largest(const int8_t* x, const float* xs, const int8_t* w, const float* ws, const float* bias,
                          void* y, bool out_bf16, int64_t m, int64_t n, int64_t k, hipStream_t stream) {
    const int64_t tiles = ((n + 255) / 256) * ((m + 255) / 256), cus = device_cu_count();
    const int64_t rest = tiles % cus, whole = tiles - rest;
    if (!halves_last_round(tiles, cus))
        return launch_tile<2, 4, 8, 4, 2, false>(x, xs, w, ws, bias, y, out_bf16, m, n, k, stream);
    const dim3 grid = grid_of((whole + kXcds - 1) / kXcds * kXcds + (2 * rest + kXcds - 1) / kXcds * kXcds);
    if (out_bf16)
        int8_gemm_mixed_kernel<true>
            <<<grid, 512, 0, stream>>>(x, xs, w, ws, bias, y, (int)m, (int)n, (int)k, (uint32_t)tiles,
                                      (uint32_t)whole);
    else
        int8_gemm_mixed_kernel<false>
            <<<grid, 512, 0, stream>>>(x, xs, w, ws, bias, y, (int)m, (int)n, (int)k, (uint32_t)tiles,
                                      (uint32_t)whole);
    return hipGetLastError();
}

// The forms and tile shapes, and what a call takes: call_us, and round_us + step_us for every 128 columns of each
// round of tiles over the compute units (us; fitted to 310 calls of random sizes from 1 x 256 x 256 to 8192 x 32768 x
// 16384, with int8 codes of normal values; the largest at the clock that the chip keeps under that load). The least is
// taken: over those calls 0.7 % above the fastest shape's time, and each shape, left out, would cost 0.5 to 1.6 %.
struct Shape {
    int rows_w, rows_x;
    float call_us, round_us, step_us;
    hipError_t (*launch)(const int8_t*, const float*, const int8_t*, const float*, const float*, void*, bool, int64_t,
                         int64_t, int64_t, hipStream_t);
};

const Shape kShapes[] = {
    {16, 16, 2.1f, 0.8f, 0.052f, launch_stream<8, 1, 1, false>},
    {16, 32, 2.2f, 0.6f, 0.071f, launch_stream<4, 1, 2, false>},
    {32, 32, 2.3f, 0.7f, 0.118f, launch_stream<4, 2, 2, false>},
    {64, 64, 2.3f, 1.1f, 0.202f, launch_tile<2, 4, 2, 1, 4, false>},
    {64, 128, 2.3f, 1.5f, 0.311f, launch_tile<2, 4, 2, 2, 3, false>},
    {128, 128, 0.4f, 4.0f, 0.468f, launch_tile<4, 4, 2, 2, 3, false>},
    {256, 128, 0.4f, 6.5f, 0.772f, launch_tile<4, 4, 4, 2, 3, false>},
    {256, 256, 0.1f, 12.7f, 1.39f, launch_largest},
};

// The same where rows start inside 128-byte lines (370 calls of such sizes, 0.8 % above the fastest). All but the
// first and the last shape then read by lines, with a longer ring; against reading across lines, in a graph: 32 x 4096
// x 14352 13.4 instead of 17.1 us (k = 14336: 12.0), 130 x 4096 x 4112 9.7 instead of 12.0 (k = 4096: 8.8), 512 x 4096
// x 4112 14.5 instead of 18.2, 2048 x 4096 x 4112 35.9 instead of 39.2. 16 x 16 stream tiles, whose workgroups no
// longer share a compute unit with a longer ring, take 12.4 us across lines and 15.7 by lines for 1 x 14336 x 4112.
// The ring of 256 x 256 tiles has no room; across lines they take 262 us for 2048 x 28672 x 4112, 256 x 128 ones by
// lines 322.
const Shape kShapesInLines[] = {
    {16, 16, 1.9f, 0.72f, 0.065f, launch_stream<8, 1, 1, false>},
    {16, 32, 2.4f, 0.7f, 0.078f, launch_stream<4, 1, 2, true>},
    {32, 32, 1.4f, 1.9f, 0.126f, launch_stream<4, 2, 2, true>},
    {64, 64, 1.2f, 2.4f, 0.208f, launch_tile<2, 4, 2, 1, 6, true>},
    {64, 128, 1.0f, 3.0f, 0.294f, launch_tile<2, 4, 2, 2, 5, true>},
    {128, 128, 0.2f, 4.3f, 0.438f, launch_tile<4, 4, 2, 2, 4, true>},
    {256, 128, 0.0f, 5.6f, 0.93f, launch_tile<4, 4, 4, 2, 3, true>},
    {256, 256, 0.0f, 11.0f, 1.48f, launch_largest},
};

// A last round of halves takes this part of a round of 256 x 256 tiles.
constexpr float kHalvesRound = 0.6f;

// The entry of kShapes (whole_lines) or kShapesInLines that a call takes on a device of `cus` compute units.
const Shape& shape_of(int64_t m, int64_t n, int64_t k, bool whole_lines, int64_t cus) {
    const float steps = (float)((k + 127) / 128);
    const Shape* best = nullptr;
    float best_us = 0.f;
    for (const Shape& s : whole_lines ? kShapes : kShapesInLines) {
        const int64_t tiles = ((n + s.rows_w - 1) / s.rows_w) * ((m + s.rows_x - 1) / s.rows_x);
        float rounds = (float)((tiles + cus - 1) / cus);
        if (s.launch == launch_largest && halves_last_round(tiles, cus)) rounds -= 1.f - kHalvesRound;
        const float us = s.call_us + rounds * (s.round_us + steps * s.step_us);
        if (best == nullptr || us < best_us) {
            best = &s;
            best_us = us;
        }
    }
    return *best;
}

}  // namespace

hipError_t launch_int8_gemm(const int8_t* x, const float* x_scale, const int8_t* w, const float* w_scale,
                            const float* bias, void* y, bool out_bf16, int64_t m, int64_t n, int64_t k,
                            hipStream_t stream) {
    const bool whole_lines =
        k % 128 == 0 && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w)) & 127) == 0;
    return shape_of(m, n, k, whole_lines, device_cu_count())
        .launch(x, x_scale, w, w_scale, bias, y, out_bf16, m, n, k, stream);
}

}  // namespace e2m1

int e2m1_int8_gemm_variant(int64_t m, int64_t n, int64_t k, int whole_lines, int cus) {
    using namespace e2m1;
    const Shape& s = shape_of(m, n, k, whole_lines != 0, cus);
    const int at = (int)(&s - (whole_lines ? kShapes : kShapesInLines));
    const bool halved = s.launch == launch_largest && halves_last_round(((n + 255) / 256) * ((m + 255) / 256), cus);
    return at + (halved ? 1 : 0);
}
