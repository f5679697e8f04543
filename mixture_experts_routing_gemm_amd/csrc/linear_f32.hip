// The linear layer's products in float32: forward, dx and dW of a grouped (or
// dense) linear layer on the float32 matrix instruction (32x32x2, 256 FLOPs a
// cycle and CU: the part's float32 matrix peak, 157 TFLOP/s, is a sixteenth
// of the bf16 one). linear.h has the formulas and the tile list.
//
// BT x BT output tiles, four waves of (BT/2) x (BT/2), k in steps of 16.
// Operands go global -> registers -> LDS, the next step's loads in flight
// during the current step's MFMAs, and lie in LDS as [k][feature], so that a
// fragment (one value a lane: 32 features at two k) is one 4-byte read. A
// wave's four MFMAs at one k pair take 256 cycles against four such reads:
// LDS is never the bound here. Rows of 4 BT + 144 bytes: the transposed
// 4-byte writes of a k-contiguous operand (16 rows x 4 chunks a wave) fall on
// 64 distinct banks.
#include <algorithm>

#include "linear.h"

namespace moe {

int device_cus();

constexpr int kF32K = 16;

template <bool TR, int BT>
struct F32Operand {
    static constexpr int kPitch = BT + 36;
    static constexpr int N = BT / 64;  // 16-byte chunks a thread
    // chunk i of this thread of the step at k: `base` as for the bf16 kernel
    __device__ static u32x4 load(const float* base, int64_t ld, int i, int k, int kend, int valid) {
        if constexpr (TR) {
            const int u = threadIdx.x + 256 * i;
            const int kk = k + u / (BT / 4), c = 4 * (u % (BT / 4));
            if (kk >= kend || c >= valid) return u32x4{0u, 0u, 0u, 0u};
            return load16(base + kk * ld + c);
        } else {
            const int r = (threadIdx.x >> 2) + 64 * i, kk = k + 4 * (threadIdx.x & 3);
            if (kk >= kend || r >= valid) return u32x4{0u, 0u, 0u, 0u};
            return load16(base + r * ld + kk);
        }
    }
    __device__ static void store(float* op, int i, u32x4 v) {
        if constexpr (TR) {
            const int u = threadIdx.x + 256 * i;
            store16(op + u / (BT / 4) * kPitch + 4 * (u % (BT / 4)), v);
        } else {
            const int r = (threadIdx.x >> 2) + 64 * i, k = 4 * (threadIdx.x & 3);
#pragma unroll
            for (int j = 0; j < 4; ++j) op[(k + j) * kPitch + r] = __uint_as_float(v[j]);
        }
    }
};

template <int PASS, int BT>
__global__ __launch_bounds__(256, 2) void linear_f32_kernel(LinearArgs a) {
    typedef F32Operand<PASS == kLinDw, BT> OpA;
    typedef F32Operand<PASS != kLinForward, BT> OpB;
    constexpr int P = OpA::kPitch, MB = BT / 64, WB = BT / 2;
    __shared__ __attribute__((aligned(16))) float lds[2][2][kF32K * P];
    __shared__ GroupWalk walk;
    __shared__ GroupOrder order;
    walk_groups(walk, a.offsets, a.R, a.G, BT, a.hdr);
    if constexpr (PASS == kLinDw) order_groups(order, walk, a.G);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wm = wave >> 1, wn = wave & 1, lr = lane & 31, lg = lane >> 5;
    const int64_t lda = PASS == kLinDw ? a.M : a.K, ldb = PASS == kLinForward ? a.K : a.N;
    const float* const pa = reinterpret_cast<const float*>(a.a);
    const float* const pb = reinterpret_cast<const float*>(a.b);

    LinTile t;
    for (int it = 0; lin_tile<PASS, BT, BT>(a, walk, order, it, t); ++it) {
        const float *ta, *tb;
        int va, vb;  // valid rows (k-contiguous) or columns of the operands' tiles
        if constexpr (PASS == kLinDw) {
            ta = pa + t.m0;
            tb = pb + t.c0;
            va = a.M - t.m0;
            vb = a.N - t.c0;
        } else {
            ta = pa + (t.row0 + t.m0) * lda;
            va = t.rows - t.m0;
            const int64_t wg = static_cast<int64_t>(t.g) * a.N * a.K;
            tb = pb + wg + (PASS == kLinForward ? t.c0 * ldb : static_cast<int64_t>(t.c0));
            vb = a.N - t.c0;
        }
        u32x4 ra[OpA::N], rb[OpB::N];
        auto load = [&](int k) {
#pragma unroll
            for (int i = 0; i < OpA::N; ++i) ra[i] = OpA::load(ta, lda, i, k, t.k1, va);
#pragma unroll
            for (int i = 0; i < OpB::N; ++i) rb[i] = OpB::load(tb, ldb, i, k, t.k1, vb);
        };
        auto put = [&](int buf) {
#pragma unroll
            for (int i = 0; i < OpA::N; ++i) OpA::store(lds[buf][0], i, ra[i]);
#pragma unroll
            for (int i = 0; i < OpB::N; ++i) OpB::store(lds[buf][1], i, rb[i]);
        };
        f32x16 acc[MB][MB];
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < MB; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
        const int KT = (t.k1 - t.k0 + kF32K - 1) / kF32K;
        if (KT > 0) {
            load(t.k0);
            put(0);
            __syncthreads();
        }
        for (int kt = 0; kt < KT; ++kt) {
            if (kt + 1 < KT) load(t.k0 + (kt + 1) * kF32K);
            const float* As = lds[kt & 1][0] + wm * WB + lr;
            const float* Bs = lds[kt & 1][1] + wn * WB + lr;
#pragma unroll
            for (int k = 0; k < kF32K; k += 2) {
                float fa[MB], fb[MB];
#pragma unroll
                for (int i = 0; i < MB; ++i) fa[i] = As[(k + lg) * P + 32 * i];
#pragma unroll
                for (int i = 0; i < MB; ++i) fb[i] = Bs[(k + lg) * P + 32 * i];
#pragma unroll
                for (int i = 0; i < MB; ++i)
#pragma unroll
                    for (int j = 0; j < MB; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fb[j], fa[i], acc[i][j], 0, 0, 0);
            }
            if (kt + 1 < KT) put((kt + 1) & 1);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < MB; ++j) {
                const int c = t.c0 + wn * WB + 32 * j;
                if (c < a.N)
                    store_block<float, PASS>(a, t.g, t.part, t.row0, t.rows, t.m0 + wm * WB + 32 * i + lr, c, lg,
                                             acc[i][j]);
            }
    }
}

namespace {

template <int PASS, int BT>
hipError_t launch(const LinearArgs& a0, hipStream_t st) {
    LinearArgs a = a0;
    a.ntn = (a.N + BT - 1) / BT;
    a.mtiles = PASS == kLinDw ? (a.M + BT - 1) / BT : 0;
    const int64_t mt = PASS == kLinDw ? static_cast<int64_t>(a.G) * a.mtiles : a.R / BT + a.G;
    const int64_t tiles = mt * a.ntn * a.parts;
    if (tiles >= (int64_t(1) << 30)) return hipErrorInvalidValue;
    int64_t blocks = std::min<int64_t>(static_cast<int64_t>(device_cus()) * 2, tiles);
    blocks = std::max<int64_t>(8, (blocks + 7) & ~int64_t(7));
    linear_f32_kernel<PASS, BT><<<static_cast<unsigned>(blocks), 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

// shape: 0 128 x 128, 1 64 x 64 tiles
hipError_t launch_linear_f32(int pass, const LinearArgs& a, int shape, hipStream_t st) {
    switch (pass) {
        case kLinForward: return shape == 0 ? launch<kLinForward, 128>(a, st) : launch<kLinForward, 64>(a, st);
        case kLinDx: return shape == 0 ? launch<kLinDx, 128>(a, st) : launch<kLinDx, 64>(a, st);
        default: return shape == 0 ? launch<kLinDw, 128>(a, st) : launch<kLinDw, 64>(a, st);
    }
}

}  // namespace moe
