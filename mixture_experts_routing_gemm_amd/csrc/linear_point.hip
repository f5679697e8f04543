// The linear layer's kernels without a product: dz = dy fn'(zs) with the bias
// gradient's partial sums, those sums joined, and the sums of a product that
// was split along k joined (with the forward's epilogue, or as dx or dW).
// All are bound by HBM.
#include <algorithm>

#include "linear.h"

namespace moe {

constexpr int kDzCols = 256;

// A work-group takes 32 rows of one group and 256 columns: eight rows of 32
// lanes x 8 columns at a time. dz is rounded to the act type once (the
// products that read it need that type); the bias gradient sums it before the
// rounding, each thread its rows in order, then the eight threads of a column
// in order: no atomics, the same bits every call.
template <typename T>
__global__ __launch_bounds__(256) void linear_dz_kernel(DzArgs a) {
    __shared__ GroupWalk walk;
    __shared__ float sums[8][kDzCols];
    walk_groups(walk, a.offsets, a.R, a.G, kDzRows, nullptr);
    const int cl = (threadIdx.x & 31) * 8, rl = threadIdx.x >> 5;
    const int c = blockIdx.y * kDzCols + cl;
    const int nv = min(8, max(0, a.N - c));
    // (more than one round only past the largest grid)
    for (int mt = blockIdx.x; mt < walk.pre[a.G]; mt += gridDim.x) {
        const int g = group_of(walk, a.G, mt);
        const int m0 = (mt - walk.pre[g]) * kDzRows;
        const int rows = min(kDzRows, walk.off[g + 1] - walk.off[g] - m0);
        const int64_t row0 = walk.off[g] + m0;
        float s[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) s[u] = 0.0f;
        if (nv > 0) {
#pragma unroll 4
            for (int r = rl; r < rows; r += 8) {
                const int64_t row = row0 + r;
                float v[8], z[8];
                load8<T>(a.dy, row * a.N + c, nv, v);
                if (a.fn != MOE_FN_NONE) {
                    if (a.z != nullptr) {
                        load8<T>(a.z, row * a.N + c, nv, z);
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2*>(a.codes + row * a.n32 + c);
                        const float step = rows8_step(a.scales[row * (a.n32 / kRows8Block) + c / kRows8Block]);
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            z[u] = rows8_value(w.x, u, step);
                            z[4 + u] = rows8_value(w.y, u, step);
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 8; ++u) v[u] *= lin_slope(a.fn, z[u]);
                    store8<T>(a.dz, row * a.N + c, nv, v);
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) s[u] += v[u];
            }
        }
        if (a.db_part == nullptr) continue;
        __syncthreads();  // (the round before is done with the sums)
#pragma unroll
        for (int u = 0; u < 8; ++u) sums[rl][cl + u] = s[u];
        __syncthreads();
        const int col = blockIdx.y * kDzCols + threadIdx.x;
        if (col < a.N) {
            float t = 0.0f;
#pragma unroll
            for (int r = 0; r < 8; ++r) t += sums[r][threadIdx.x];
            a.db_part[static_cast<int64_t>(mt) * a.N + col] = t;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(512) void linear_db_kernel(DbArgs a) {
    linear_db_block<T, 8>(a, blockIdx.y, blockIdx.x);
}

// The parts' sums of 32 x 32 values, added part by part, then stored as the
// tile kernels store a block. A block is one wave's (SPLIT = 1), or four waves
// (SPLIT = 4) sum every fourth part each, in order, and then their sums in
// order: where many parts are added over few blocks, which are then as long as
// the loads that one wave has under way.
template <typename T, int PASS, int SPLIT>
__global__ __launch_bounds__(256) void linear_join_kernel(LinearArgs a) {
    __shared__ GroupWalk walk;
    __shared__ float sums[SPLIT > 1 ? SPLIT - 1 : 1][16][64];
    if constexpr (PASS != kLinDw) walk_groups(walk, a.offsets, a.R, a.G, 1, nullptr);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, half = lane >> 5;
    const int64_t all = PASS == kLinDw ? static_cast<int64_t>(a.G) * a.M : a.R;
    const int nblk = (a.N + 31) / 32;
    const int64_t blk = SPLIT > 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * 4 + wave;
    if (blk >= (all + 31) / 32 * nblk) return;  // (SPLIT > 1: never)
    const int c0 = static_cast<int>(blk % nblk) * 32;
    const int64_t row = blk / nblk * 32 + (lane & 31);
    bool ok = row < all;
    int g = 0;
    if constexpr (PASS != kLinDw) {
        // (rows of no group are left as they are)
        ok = ok && row >= walk.off[0] && row < walk.off[a.G];
        if (PASS == kLinForward && a.bias != nullptr && ok) {
            int lo = 0, hi = a.G - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (walk.off[mid] <= row) lo = mid;
                else hi = mid - 1;
            }
            g = lo;
        }
    }
    float v[2][8];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int u = 0; u < 8; ++u) v[p][u] = 0.0f;
        const int c = c0 + 16 * p + 8 * half, nv = min(8, a.N - c);
        if (ok && nv > 0) {
#pragma unroll 4
            for (int s = SPLIT > 1 ? wave : 0; s < a.parts; s += SPLIT) {
                float t[8];
                load8<float>(reinterpret_cast<const uint8_t*>(a.part_out), (s * all + row) * a.N + c, nv, t);
#pragma unroll
                for (int u = 0; u < 8; ++u) v[p][u] += t[u];
            }
        }
    }
    if constexpr (SPLIT > 1) {
        if (wave > 0) {
#pragma unroll
            for (int u = 0; u < 16; ++u) sums[wave - 1][u][lane] = v[u >> 3][u & 7];
        }
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int w = 0; w < SPLIT - 1; ++w)
#pragma unroll
            for (int u = 0; u < 16; ++u) v[u >> 3][u & 7] += sums[w][u][lane];
    }
    if constexpr (PASS == kLinForward) {
        linear_epilogue32<T>(a, g, row, c0, half, ok, v, a.N);
    } else if (PASS == kLinDw && a.out_f32) {
        plain_epilogue32<float>(a.out, row * a.N, a.N, c0, half, ok, v);
    } else {
        plain_epilogue32<T>(a.out, row * a.N, a.N, c0, half, ok, v);
    }
}

int64_t linear_db_tiles(int64_t R, int G) { return R / kDzRows + G; }

hipError_t launch_linear_dz(const DzArgs& a, bool f32, hipStream_t st) {
    // (a grid has at most 2^32 - 1 threads along x)
    const int64_t mt = std::min<int64_t>(linear_db_tiles(a.R, a.G), (int64_t(1) << 24) - 1);
    const dim3 grid(static_cast<unsigned>(mt), (a.N + kDzCols - 1) / kDzCols);
    if (f32)
        linear_dz_kernel<float><<<grid, 256, 0, st>>>(a);
    else
        linear_dz_kernel<bf16_t><<<grid, 256, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_linear_db(const DbArgs& a, bool f32, hipStream_t st) {
    const dim3 grid((a.N + 63) / 64, a.G);
    if (f32)
        linear_db_kernel<float><<<grid, 512, 0, st>>>(a);
    else
        linear_db_kernel<bf16_t><<<grid, 512, 0, st>>>(a);
    return hipGetLastError();
}

namespace {
template <typename T, int PASS>
hipError_t launch_join(const LinearArgs& a, hipStream_t st) {
    const int64_t all = PASS == kLinDw ? static_cast<int64_t>(a.G) * a.M : a.R;
    const int64_t blocks = (all + 31) / 32 * ((a.N + 31) / 32);
    if (blocks >= (int64_t(1) << 24)) return hipErrorInvalidValue;
    if (a.parts >= 8)
        linear_join_kernel<T, PASS, 4><<<static_cast<unsigned>(blocks), 256, 0, st>>>(a);
    else
        linear_join_kernel<T, PASS, 1><<<static_cast<unsigned>((blocks + 3) / 4), 256, 0, st>>>(a);
    return hipGetLastError();
}
}  // namespace

hipError_t launch_linear_join(int pass, const LinearArgs& a, bool f32, hipStream_t st) {
    switch (pass) {
        case kLinForward: return f32 ? launch_join<float, kLinForward>(a, st) : launch_join<bf16_t, kLinForward>(a, st);
        case kLinDx: return f32 ? launch_join<float, kLinDx>(a, st) : launch_join<bf16_t, kLinDx>(a, st);
        default: return f32 ? launch_join<float, kLinDw>(a, st) : launch_join<bf16_t, kLinDw>(a, st);
    }
}

}  // namespace moe
