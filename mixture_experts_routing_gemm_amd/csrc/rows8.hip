// Rows packed into the 8-bit checkpoint format, and read back (rows8.h).
// Bound by HBM: es + 33/32 bytes a value either way (32768 x 2048 bf16: pack 38
// us, 5.4 TB/s; unpack 31 us with the codes still in the cache).
#include <algorithm>

#include "rows8.h"

namespace moe {

// Four lanes share a block of 32 values, eight each: a wave packs 16 blocks
// (512 values) at a time. VEC: rows start on 16 bytes and n is a multiple of
// the values in them; else values move one by one.
template <typename T, bool VEC>
__device__ __forceinline__ void rows8_load(const T* x, int64_t at, int nv, float (&v)[8]) {
    if constexpr (VEC) {
        constexpr int N = ActVec<T>::N;
#pragma unroll
        for (int q = 0; q < 8 / N; ++q) {
            if (q * N < nv) {
                ActVec<T>::unpack(load16(x + at + q * N), v + q * N);
            } else {
#pragma unroll
                for (int u = 0; u < N; ++u) v[q * N + u] = 0.0f;
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            v[u] = 0.0f;
            if (u < nv) {
                if constexpr (sizeof(T) == 4) v[u] = x[at + u];
                else v[u] = bf16_to_f32(x[at + u]);
            }
        }
    }
}

template <typename T, bool VEC>
__global__ __launch_bounds__(256) void pack_rows8_kernel(const T* __restrict__ x, int64_t rows, int n, int n32,
                                                         uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    const int per_row = n32 / 8;
    const int64_t total = rows * per_row;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    // (stride is a multiple of 4: the four lanes of a block stay together)
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += stride) {
        const int64_t row = i / per_row;
        const int c = static_cast<int>(i - row * per_row) * 8;
        const int nv = min(8, max(0, n - c));
        float v[8];
        rows8_load<T, VEC>(x, row * n + c, nv, v);
        uint32_t top = 0u;
#pragma unroll
        for (int u = 0; u < 8; ++u) top = max(top, abs_bits(v[u]));
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 1, 64)));
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 2, 64)));
        const uint32_t scale = rows8_scale(top);
        const float inv = rows8_inverse(scale);
        uint2 w;
        w.x = rows8_code4(v[0], v[1], v[2], v[3], inv);
        w.y = rows8_code4(v[4], v[5], v[6], v[7], inv);
        *reinterpret_cast<uint2*>(codes + i * 8) = w;
        if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(scale);
    }
}

template <typename T, bool VEC>
__global__ __launch_bounds__(256) void unpack_rows8_kernel(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int64_t rows, int n,
                                                           int n32, T* __restrict__ x) {
    const int per_row = n32 / 8;
    const int64_t total = rows * per_row;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += stride) {
        const int64_t row = i / per_row;
        const int c = static_cast<int>(i - row * per_row) * 8;
        const int nv = min(8, max(0, n - c));
        const uint2 w = *reinterpret_cast<const uint2*>(codes + i * 8);
        const float step = rows8_step(scales[i >> 2]);
        float v[8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            v[u] = rows8_value(w.x, u, step);
            v[4 + u] = rows8_value(w.y, u, step);
        }
        if constexpr (VEC) {
            constexpr int N = ActVec<T>::N;
#pragma unroll
            for (int q = 0; q < 8 / N; ++q)
                if (q * N < nv) store16(x + row * n + c + q * N, ActVec<T>::pack(v + q * N));
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (u < nv) {
                    if constexpr (sizeof(T) == 4) x[row * n + c + u] = v[u];
                    else x[row * n + c + u] = f32_to_bf16(v[u]);
                }
        }
    }
}

namespace {
unsigned rows8_blocks(int64_t rows, int64_t n32) {
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((rows * (n32 / 8) + 255) / 256, 256 * 32)));
}
}  // namespace

hipError_t launch_pack_rows8(int64_t rows, int n, bool f32, const void* x, void* packed, hipStream_t st) {
    const int n32 = static_cast<int>(rows8_stride(n));
    uint8_t* codes = static_cast<uint8_t*>(packed);
    uint8_t* scales = codes + rows8_scales_at(rows, n);
    const unsigned b = rows8_blocks(rows, n32);
    if (f32) {
        const float* p = static_cast<const float*>(x);
        if (n % 4 == 0) pack_rows8_kernel<float, true><<<b, 256, 0, st>>>(p, rows, n, n32, codes, scales);
        else pack_rows8_kernel<float, false><<<b, 256, 0, st>>>(p, rows, n, n32, codes, scales);
    } else {
        const bf16_t* p = static_cast<const bf16_t*>(x);
        if (n % 8 == 0) pack_rows8_kernel<bf16_t, true><<<b, 256, 0, st>>>(p, rows, n, n32, codes, scales);
        else pack_rows8_kernel<bf16_t, false><<<b, 256, 0, st>>>(p, rows, n, n32, codes, scales);
    }
    return hipGetLastError();
}

hipError_t launch_unpack_rows8(int64_t rows, int n, bool f32, const void* packed, void* x, hipStream_t st) {
    const int n32 = static_cast<int>(rows8_stride(n));
    const uint8_t* codes = static_cast<const uint8_t*>(packed);
    const uint8_t* scales = codes + rows8_scales_at(rows, n);
    const unsigned b = rows8_blocks(rows, n32);
    if (f32) {
        float* p = static_cast<float*>(x);
        if (n % 4 == 0) unpack_rows8_kernel<float, true><<<b, 256, 0, st>>>(codes, scales, rows, n, n32, p);
        else unpack_rows8_kernel<float, false><<<b, 256, 0, st>>>(codes, scales, rows, n, n32, p);
    } else {
        bf16_t* p = static_cast<bf16_t*>(x);
        if (n % 8 == 0) unpack_rows8_kernel<bf16_t, true><<<b, 256, 0, st>>>(codes, scales, rows, n, n32, p);
        else unpack_rows8_kernel<bf16_t, false><<<b, 256, 0, st>>>(codes, scales, rows, n, n32, p);
    }
    return hipGetLastError();
}

}  // namespace moe
