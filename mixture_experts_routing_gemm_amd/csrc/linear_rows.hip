// The linear layer's forward for few rows (decoding steps, short prompts over
// many experts): bound by reading the weights once from HBM.
//
// A work-group of eight waves takes up to 64 rows of a group and 16 FB output
// columns. The waves split k between them, 128 bytes at a time in turn, so
// that together they read 1 KB runs of each weight row; the weights go
// straight from memory to the registers of the MFMAs (16x16x32 in bf16,
// 16x16x4 in float32; first operand: 16 weight rows; second: 16 rows of x),
// several steps ahead, because registers hold more bytes in flight than the
// LDS could. A lane fetches 32 consecutive bytes of a row; the k values of an
// MFMA are then not consecutive but the same ones in both operands, which is
// all a sum over k needs. The
// eight waves' sums are added through LDS, in wave order, and the epilogue
// runs on the total.
//
// Rows past the group's end are not read (their lanes hold zeros): one row
// costs 1/16 of the x traffic of 16. Measured: one row, 4096 -> 4096 in bf16,
// 8.9 us, 3.8 TB/s with the launch; wider columns, k contiguous per wave and
// non-temporal weight loads were no faster.
#include <algorithm>

#include "linear.h"

namespace moe {

constexpr int kRowsBM = 64;      // rows a work-group takes at most
constexpr int kRowsWaves = 8;

typedef float f32x4r __attribute__((ext_vector_type(4)));

// sums of JB blocks of 16 rows and FB of 16 columns over this wave's share of
// k; lane holds columns 4 (lane / 16) .. +3 of row lane % 16 of each block
template <typename T, int FB, int JB, int U>
__device__ __forceinline__ void rows_products(const T* __restrict__ x, const T* __restrict__ w, int K,
                                              int rows, int cols, int wave, int lane, f32x4r (&acc)[JB][FB]) {
    constexpr int V = 16 / sizeof(T), STEP = 8 * V;  // values of 16 and of 128 bytes
    const int r = lane & 15, q = lane >> 4;
    const T* xp[JB];
    const T* wp[FB];
#pragma unroll
    for (int j = 0; j < JB; ++j) xp[j] = x + static_cast<int64_t>(min(16 * j + r, rows - 1)) * K + 2 * V * q;
#pragma unroll
    for (int f = 0; f < FB; ++f) wp[f] = w + static_cast<int64_t>(min(16 * f + r, cols - 1)) * K + 2 * V * q;
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
        for (int f = 0; f < FB; ++f) acc[j][f] = f32x4r{0.0f, 0.0f, 0.0f, 0.0f};
    // U steps in flight: a step's registers are loaded again as soon as its
    // products are issued
    u32x4 wv[U][FB][2], xv[U][JB][2];
    auto load = [&](int u, int s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = STEP * s + V * h;
            // (both operands are zero past the end of k)
            const bool in = k + 2 * V * q < K;
#pragma unroll
            for (int f = 0; f < FB; ++f) wv[u][f][h] = in ? load16(wp[f] + k) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < JB; ++j)
                xv[u][j][h] = in && 16 * j + r < rows ? load16(xp[j] + k) : u32x4{0u, 0u, 0u, 0u};
        }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, wave + u * kRowsWaves);
    const int steps = (K + STEP - 1) / STEP;
    for (int s0 = wave; s0 < steps; s0 += kRowsWaves * U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < JB; ++j)
#pragma unroll
                    for (int f = 0; f < FB; ++f) {
                        if constexpr (sizeof(T) == 2) {
                            acc[j][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8, wv[u][f][h]), __builtin_bit_cast(bf16x8, xv[u][j][h]),
                                acc[j][f], 0, 0, 0);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc[j][f] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                    __uint_as_float(wv[u][f][h][i]), __uint_as_float(xv[u][j][h][i]), acc[j][f], 0, 0, 0);
                        }
                    }
            load(u, s0 + (u + U) * kRowsWaves);
        }
    }
}

// The products of one pass (16 FB columns from c0), the waves' sums put side by
// side in LDS as [wave][row][column] with rows padded by four floats, added in
// wave order, and the epilogue: a wave per 32 rows x 32 columns. Every thread
// of the work-group calls this.
template <typename T, int FB, int JB, int U>
__device__ __forceinline__ void rows_pass(const LinearArgs& a, const T* x, int g, int64_t row0, int n, int c0,
                                          float* sums) {
    constexpr int C = 16 * FB, P = C + 4, RB = 16 * JB;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int cols = min(C, a.N - c0);
    const T* w = reinterpret_cast<const T*>(a.b) + (static_cast<int64_t>(g) * a.N + c0) * a.K;
    f32x4r acc[JB][FB];
    rows_products<T, FB, JB, U>(x, w, a.K, n, cols, wave, lane, acc);
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
        for (int f = 0; f < FB; ++f)
            *reinterpret_cast<f32x4r*>(sums + (wave * RB + 16 * j + (lane & 15)) * P + 16 * f + 4 * (lane >> 4)) =
                acc[j][f];
    __syncthreads();
    constexpr int RW = (RB + 31) / 32, CW = (C + 31) / 32;  // waves along rows and columns
    const int rw = wave % RW, cw = wave / RW;
    if (cw >= CW || rw * 32 >= n || cw * 32 >= cols) return;
    const int lr = lane & 31, half = lane >> 5, m = rw * 32 + lr;
    float v[2][8];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int u = 0; u < 8; ++u) v[p][u] = 0.0f;
        if (16 * p < C && m < n) {
#pragma unroll
            for (int s = 0; s < kRowsWaves; ++s) {
                const float* from = sums + (s * RB + m) * P + 32 * cw + 16 * p + 8 * half;
#pragma unroll
                for (int u = 0; u < 8; u += 4) {
                    const f32x4r t = *reinterpret_cast<const f32x4r*>(from + u);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[p][u + i] += t[i];
                }
            }
        }
    }
    linear_epilogue32<T>(a, g, row0 + m, c0 + 32 * cw, half, m < n, v, c0 + cols);
}

template <typename T, int FB>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(FB == 1 ? 2 : 4, FB == 1 ? 2 : 4))) void
linear_rows_kernel(LinearArgs a) {
    constexpr int C = 16 * FB;
    extern __shared__ __attribute__((aligned(16))) float sums[];
    __shared__ GroupWalk walk;
    int g = 0, m0 = 0, rows = static_cast<int>(a.R), c0;
    int64_t row0 = 0;
    if (a.offsets != nullptr) {
        // the list of (row block, column block) is cut into eight runs, one
        // for each XCD: a group's columns share its rows of x in one L2
        walk_groups(walk, a.offsets, a.R, a.G, kRowsBM, blockIdx.x == 0 ? a.hdr : nullptr);
        const int total = __builtin_amdgcn_readfirstlane(walk.pre[a.G]) * a.ntn, xcd = blockIdx.x & 7;
        const auto eighth = [&](int i) { return (total >> 3) * i + ((total & 7) * i >> 3); };
        const int L = eighth(xcd) + static_cast<int>(blockIdx.x >> 3);
        if (L >= eighth(xcd + 1)) return;
        const int mt = L / a.ntn;
        c0 = (L - mt * a.ntn) * C;
        g = group_of(walk, a.G, mt);
        m0 = (mt - __builtin_amdgcn_readfirstlane(walk.pre[g])) * kRowsBM;
        row0 = __builtin_amdgcn_readfirstlane(walk.off[g]);
        rows = __builtin_amdgcn_readfirstlane(walk.off[g + 1]) - static_cast<int>(row0);
    } else {
        m0 = static_cast<int>(blockIdx.x) / a.ntn * kRowsBM;
        c0 = static_cast<int>(blockIdx.x) % a.ntn * C;
    }
    const int n = min(kRowsBM, rows - m0);
    row0 += m0;
    const T* x = reinterpret_cast<const T*>(a.a) + row0 * a.K;
    if (n <= 16) {
        rows_pass<T, FB, 1, 8 / FB>(a, x, g, row0, n, c0, sums);
    } else if (n <= 32) {
        rows_pass<T, FB, 2, 4 / FB>(a, x, g, row0, n, c0, sums);
    } else {
        rows_pass<T, FB, 4, 2 / FB>(a, x, g, row0, n, c0, sums);
    }
}

namespace {
template <typename T, int FB>
hipError_t launch(const LinearArgs& a, unsigned grid, hipStream_t st) {
    constexpr int lds = kRowsWaves * kRowsBM * (16 * FB + 4) * 4;
    static hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&linear_rows_kernel<T, FB>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (attr != hipSuccess) return attr;
    linear_rows_kernel<T, FB><<<grid, 512, lds, st>>>(a);
    return hipGetLastError();
}
}  // namespace

// fb: 16-column blocks a work-group (1 or 2; 8-bit codes need 2)
hipError_t launch_linear_rows(const LinearArgs& a0, int fb, bool f32, hipStream_t st) {
    LinearArgs a = a0;
    a.ntn = (a.N + 16 * fb - 1) / (16 * fb);
    const int64_t mt = a.offsets != nullptr ? a.R / kRowsBM + a.G : (a.R + kRowsBM - 1) / kRowsBM;
    const int64_t total = mt * a.ntn;
    if (total >= (int64_t(1) << 30)) return hipErrorInvalidValue;
    const unsigned grid = static_cast<unsigned>(a.offsets != nullptr ? (total + 7) & ~int64_t(7) : total);
    if (f32) return fb == 1 ? launch<float, 1>(a, grid, st) : launch<float, 2>(a, grid, st);
    return fb == 1 ? launch<bf16_t, 1>(a, grid, st) : launch<bf16_t, 2>(a, grid, st);
}

}  // namespace moe
