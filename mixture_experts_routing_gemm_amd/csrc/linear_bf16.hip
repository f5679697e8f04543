// The linear layer's products on the bf16 matrix cores: forward, dx and dW of
// a grouped (or dense) linear layer, with the bias, activation and residual in
// the forward's epilogue. linear.h has the formulas and the tile list.
//
// One persistent kernel for the three products. A work-group walks its list
// of BM x BN output tiles; the operands' slices of 32 k values go global ->
// LDS by direct 16-byte loads into a ring of four slots, three slices ahead,
// as one stream that runs on across tiles (while a tile's epilogue stores,
// the next tile's first slices arrive). Operands are staged as they lie in
// memory: one contiguous along k as rows of 64 bytes, read by 16-byte LDS
// reads; one contiguous along m or n as 32 rows of BM or BN values, read by
// the transposing LDS read. So neither the weights (dx) nor the rows (dW) are
// ever written out transposed.
//
// Each tile's requests go through buffer resources that start at the tile and
// end at its last row: 32-bit offsets however large the operands are, and
// rows past the end read as zeros. A slice that runs past the end of k masks
// the lanes of a k-contiguous operand by an offset beyond the resource, and
// the other kind's rows past k lie beyond it.
#include <algorithm>

#include "lds_ring.h"
#include "linear.h"

namespace moe {

int device_cus();

constexpr int kLinBK = 32;
constexpr int kLinSlots = 4;

typedef int i32x4lin __attribute__((ext_vector_type(4)));
typedef short v4i16lin __attribute__((ext_vector_type(4)));

// byte offset of 16-byte chunk c (0..3) of row r of a k-contiguous slice; the
// XOR spreads aligned runs of 8 rows over the banks
__device__ __forceinline__ int lin_swz(int r) { return ((r >> 1) & 3) ^ ((r >> 3) & 1); }
__device__ __forceinline__ int lin_koff(int r, int c) { return (r << 6) + ((c ^ lin_swz(r)) << 4); }
// chunk swizzle of slice row k of an m- or n-contiguous operand: the
// transposing reads (4 rows of 32 or 64 bytes at a time) hit distinct banks
__device__ __forceinline__ int lin_tsw(int k) { return (0xEA40 >> (4 * (k & 3))) & 15; }  // 0, 4, 10, 14

__device__ __forceinline__ uint32_t lin_lds_addr(const uint8_t* p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) uint8_t*)p));
}

// A buffer -> LDS request as inline asm without register results: issued
// through the builtin it counts as an LDS write to the compiler, which then
// drains the prefetched slices before LDS reads it cannot tell apart from it.
// (The counted waits and barriers of the kernel order it; s_nop 0: one wait
// state between a write of M0 and an LDS load.)
__device__ __forceinline__ void lin_dma16(i32x4lin rsrc, uint32_t voff, uint32_t ldsaddr) {
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "{m0}"(ldsaddr));
}
__device__ __forceinline__ i32x4lin lin_rsrc(const uint8_t* base, uint32_t bytes) {
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    i32x4lin r;
    r[0] = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(b)));
    r[1] = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(b >> 32) & 0xffffu));
    r[2] = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes));
    r[3] = kBufferFlags;
    return r;
}

// The tile shapes: BM x BN by waves of WM x WN; the first ISS waves issue the
// requests.
struct LinBig {
    static constexpr int BM = 256, BN = 256, WM = 128, WN = 64, ISS = 4, PER_CU = 1;
};
struct LinMid {
    static constexpr int BM = 128, BN = 128, WM = 64, WN = 64, ISS = 4, PER_CU = 2;
};
struct LinSmall {
    static constexpr int BM = 64, BN = 128, WM = 32, WN = 64, ISS = 4, PER_CU = 3;
};
template <class S>
constexpr int lin_threads() {
    return (S::BM / S::WM) * (S::BN / S::WN) * 64;
}
template <class S>
constexpr int lin_slot() {
    return (S::BM + S::BN) * kLinBK * 2;
}

// One operand's side of the request stream. TR: contiguous along m or n
// (columns col0 .. of rows k); else rows row0 .. contiguous along k.
template <bool TR, int W>
struct LinOperand {
    static constexpr int kBytes = W * kLinBK * 2;

    // this lane's byte offset in request i (1 KB of the slice): constant over
    // slices and tiles. ld: values a row.
    __device__ static uint32_t lane_offset(int i, int lane, int64_t ld) {
        if constexpr (TR) {
            constexpr int CH = W / 8;  // 16-byte chunks a row
            const int k = i * (64 / CH) + lane / CH;
            return static_cast<uint32_t>(k * ld * 2) + 16u * ((lane % CH) ^ lin_tsw(k));
        } else {
            const int r = 16 * i + (lane >> 2);
            return static_cast<uint32_t>(r * ld * 2) + 16u * ((lane & 3) ^ lin_swz(r));
        }
    }
    // resource of the slice at k: `base` points at row first of the operand's
    // tile (k-contiguous: its first row; else the row of k = 0 at the tile's
    // first column)
    __device__ static i32x4lin resource(const uint8_t* base, int64_t ld, int k, int kend, int valid) {
        if constexpr (TR) {
            const int n = min(kLinBK, kend - k);  // valid: columns from the tile's first one on
            const uint32_t bytes = n > 0 ? static_cast<uint32_t>(((n - 1) * ld + valid) * 2) : 0u;
            return lin_rsrc(base + k * ld * 2, bytes);
        } else {
            // valid: rows of the tile
            const uint32_t bytes = kend > k ? static_cast<uint32_t>((valid * ld - k) * 2) : 0u;
            return lin_rsrc(base + static_cast<int64_t>(k) * 2, bytes);
        }
    }
    // this lane's fragment offset within a slice, for features f0 .. f0+31 and
    // half-slice 0; half-slice 1 lies kHalf further (TR), or at the other
    // chunk (k-contiguous: half_offset)
    __device__ static uint32_t frag_offset(int f0, int ks, int lane) {
        if constexpr (TR) {
            const int g = lane >> 4, s = lane & 15;
            const int k = 16 * ks + 8 * (g >> 1) + (s >> 2);
            const int f = f0 + 16 * (g & 1) + 4 * (s & 3);
            return static_cast<uint32_t>(k * W * 2 + (((f >> 3) ^ lin_tsw(k)) << 4) + (f & 7) * 2);
        } else {
            return static_cast<uint32_t>(lin_koff(f0 + (lane & 31), 2 * ks + (lane >> 5)));
        }
    }
    // eight k values of one feature: k = 16 ks + 8 (lane / 32) ..
    __device__ static bf16x8 fragment(const uint8_t* lds, uint32_t at) {
        if constexpr (TR) {
            typedef __attribute__((address_space(3))) v4i16lin lv4;
            const __attribute__((address_space(3))) uint8_t* p =
                (const __attribute__((address_space(3))) uint8_t*)lds + at;
            const v4i16lin lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lv4*)p);
            const v4i16lin hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lv4*)(p + 4 * W * 2));
            return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            return *reinterpret_cast<const bf16x8*>(lds + at);
        }
    }
};

template <int PASS, class S>
__global__ __launch_bounds__(lin_threads<S>()) __attribute__((amdgpu_waves_per_eu(lin_threads<S>() / 256 * S::PER_CU,
                                                                                  lin_threads<S>() / 256 * S::PER_CU)))
void linear_bf16_kernel(LinearArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ GroupWalk walk;
    __shared__ GroupOrder order;
    constexpr int BM = S::BM, BN = S::BN;
    constexpr int WN_WAVES = BN / S::WN;
    constexpr int MB = S::WM / 32, NB = S::WN / 32;
    constexpr int RA = BM / 16 / S::ISS, RB = BN / 16 / S::ISS, REQS = RA + RB;
    constexpr int kSlot = lin_slot<S>();
    typedef LinOperand<PASS == kLinDw, BM> OpA;
    typedef LinOperand<PASS != kLinForward, BN> OpB;

    walk_groups(walk, a.offsets, a.R, a.G, BM, a.hdr);
    if constexpr (PASS == kLinDw) order_groups(order, walk, a.G);

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int wm = wave / WN_WAVES, wn = wave % WN_WAVES;
    const int lr = lane & 31, lg = lane >> 5;
    const bool issuer = wave < S::ISS;

    // row strides in values
    const int64_t lda = PASS == kLinDw ? a.M : a.K;
    const int64_t ldb = PASS == kLinForward ? a.K : a.N;

    // ---- the request stream ----
    uint32_t va[RA], vb[RB];
#pragma unroll
    for (int q = 0; q < RA; ++q) va[q] = OpA::lane_offset(wave * RA + q, lane, lda);
#pragma unroll
    for (int q = 0; q < RB; ++q) vb[q] = OpB::lane_offset(wave * RB + q, lane, ldb);
    // k offset, within a slice, of the chunk that this lane fetches of a
    // k-contiguous operand (the same in each of its requests: lin_swz takes
    // bits 1 to 3 of the row, which is 16 i + lane / 4)
    const int kc = 8 * ((lane & 3) ^ lin_swz(lane >> 2));
    int ilist = 0;         // next position of the list to request
    int ik = 0, ikend = 0; // next slice of the current tile; its end
    int ivalid_a = 0, ivalid_b = 0;
    const uint8_t* ia = a.a;
    const uint8_t* ib = a.b;
    auto next_source = [&]() {
        LinTile t;
        do {
            if (!lin_tile<PASS, BM, BN>(a, walk, order, ilist, t)) {
                ik = ikend = 0;  // nothing more: empty resources, zeros
                return;
            }
            ++ilist;
        } while (t.k1 <= t.k0);
        ik = t.k0;
        ikend = t.k1;
        if constexpr (PASS == kLinDw) {
            ia = a.a + static_cast<int64_t>(t.m0) * 2;
            ib = a.b + static_cast<int64_t>(t.c0) * 2;
            ivalid_a = a.M - t.m0;
            ivalid_b = a.N - t.c0;
        } else {
            ia = a.a + (t.row0 + t.m0) * lda * 2;
            ivalid_a = min(BM, t.rows - t.m0);
            const int64_t wbase = static_cast<int64_t>(t.g) * a.N * a.K;
            if constexpr (PASS == kLinForward) {
                ib = a.b + (wbase + t.c0 * ldb) * 2;
                ivalid_b = min(BN, a.N - t.c0);
            } else {
                ib = a.b + (wbase + t.c0) * 2;
                ivalid_b = a.N - t.c0;
            }
        }
    };
    i32x4lin rsa, rsb;
    uint32_t slot_addr;
    bool in_a, in_b;  // this lane's chunk lies before the end of k
    auto open_slice = [&](int slot) {
        rsa = OpA::resource(ia, lda, ik, ikend, ivalid_a);
        rsb = OpB::resource(ib, ldb, ik, ikend, ivalid_b);
        in_a = PASS == kLinDw || kc < ikend - ik;
        in_b = PASS != kLinForward || kc < ikend - ik;
        slot_addr = __builtin_amdgcn_readfirstlane(lin_lds_addr(lds) + slot * kSlot);
    };
    auto request = [&](auto I) {
        constexpr int i = decltype(I)::value;
        if constexpr (i < RA)
            lin_dma16(rsa, in_a ? va[i] : 0xfffffff0u,
                      __builtin_amdgcn_readfirstlane(slot_addr + 1024 * (wave * RA + i)));
        else
            lin_dma16(rsb, in_b ? vb[i - RA] : 0xfffffff0u,
                      __builtin_amdgcn_readfirstlane(slot_addr + OpA::kBytes + 1024 * (wave * RB + i - RA)));
    };
    auto close_slice = [&]() {
        ik += kLinBK;
        if (ik >= ikend) next_source();
    };

    // ---- fragments ----
    uint32_t fo_a[2], fo_b[2];  // of blocks 0, by half-slice; block i lies a constant further
    fo_a[0] = OpA::frag_offset(wm * S::WM, 0, lane);
    fo_a[1] = OpA::frag_offset(wm * S::WM, 1, lane);
    fo_b[0] = OpB::frag_offset(wn * S::WN, 0, lane) + OpA::kBytes;
    fo_b[1] = OpB::frag_offset(wn * S::WN, 1, lane) + OpA::kBytes;
    // (k-contiguous: 32 rows of 64 bytes, the same swizzle. Transposed: 32
    // features are 4 chunks, and the XOR with lin_tsw (values 0, 4, 10, 14)
    // does not commute with adding them: their offsets are kept.)
    uint32_t ta[PASS == kLinDw ? MB : 1], tb[PASS != kLinForward ? NB : 1];
    if constexpr (PASS == kLinDw) {
#pragma unroll
        for (int i = 0; i < MB; ++i) ta[i] = OpA::frag_offset(wm * S::WM + 32 * i, 0, lane);
    }
    if constexpr (PASS != kLinForward) {
#pragma unroll
        for (int i = 0; i < NB; ++i) tb[i] = OpB::frag_offset(wn * S::WN + 32 * i, 0, lane) + OpA::kBytes;
    }
    auto frag_a = [&](uint32_t slot_off, auto KS, int i) -> bf16x8 {
        constexpr int ks = decltype(KS)::value;
        if constexpr (PASS == kLinDw)
            return OpA::fragment(lds, slot_off + ta[i] + ks * 16 * BM * 2);
        else
            return OpA::fragment(lds, slot_off + fo_a[ks] + i * 2048);
    };
    auto frag_b = [&](uint32_t slot_off, auto KS, int i) -> bf16x8 {
        constexpr int ks = decltype(KS)::value;
        if constexpr (PASS != kLinForward)
            return OpB::fragment(lds, slot_off + tb[i] + ks * 16 * BN * 2);
        else
            return OpB::fragment(lds, slot_off + fo_b[ks] + i * 2048);
    };

    f32x16 acc[MB][NB];
    bf16x8 fa0[MB], fb0[NB], fa1[MB], fb1[NB];
    // the MFMAs on one half-slice (fa, fb), each followed by one request (in
    // the first half) and the read of one fragment of half-slice KS of a slot
    auto half = [&](bf16x8 (&fa)[MB], bf16x8 (&fb)[NB], uint32_t slot_off, auto KS, bf16x8 (&na)[MB],
                    bf16x8 (&nb)[NB], auto IDLE, auto ISSUE) {
        constexpr bool idle = decltype(IDLE)::value;
        constexpr int n1 = MB * NB > MB + NB ? MB * NB : MB + NB;
        constexpr int n = decltype(ISSUE)::value && REQS > n1 ? REQS : n1;
        static_for<0, n>([&](auto I) {
            constexpr int i = decltype(I)::value;
            if constexpr (!idle && i < MB * NB)
                acc[i / NB][i % NB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[i % NB], fa[i / NB],
                                                                              acc[i / NB][i % NB], 0, 0, 0);
            if constexpr (decltype(ISSUE)::value && i < REQS) {
                if (issuer) request(I);
            }
            if constexpr (i < NB)
                nb[i] = frag_b(slot_off, KS, i);
            else if constexpr (i < MB + NB)
                na[i - NB] = frag_a(slot_off, KS, i - NB);
            __builtin_amdgcn_sched_barrier(0);
        });
    };

    // prologue: three slices
    int slice = 0;  // slices computed so far (of all tiles)
    next_source();
    for (int s = 0; s < 3; ++s) {
        open_slice(s);
        if (issuer) static_for<0, REQS>(request);
        close_slice();
    }
    wait_vmcnt<2 * REQS>();
    ring_barrier();
    static_for<0, MB + NB>([&](auto I) {
        constexpr int i = decltype(I)::value;
        if constexpr (i < NB)
            fb0[i] = frag_b(0, ic<0>(), i);
        else
            fa0[i - NB] = frag_a(0, ic<0>(), i - NB);
    });

    for (int it = 0;; ++it) {
        LinTile t;
        if (!lin_tile<PASS, BM, BN>(a, walk, order, it, t)) break;
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
        const int KT = (t.k1 - t.k0 + kLinBK - 1) / kLinBK;
        // Step: slice s is in slot s % 4, its first fragments in fa0, fb0.
        // The first half computes on them, requests slice s + 3 into the slot
        // of s - 1 (read to its end before the last barrier) and reads the
        // second half's fragments; then slice s + 1 has to have landed (the
        // requests of s + 2 and s + 3 may be under way), and the second half
        // reads its first fragments, which may be the next tile's.
        // A wave without rows or columns in the tile (idle) computes nothing.
        auto steps = [&](auto IDLE) {
            for (int k = 0; k < KT; ++k, ++slice) {
                const uint32_t here = static_cast<uint32_t>(slice & 3) * kSlot;
                const uint32_t next = static_cast<uint32_t>((slice + 1) & 3) * kSlot;
                open_slice((slice + 3) & 3);
                half(fa0, fb0, here, ic<1>(), fa1, fb1, IDLE, std::true_type());
                wait_vmcnt<2 * REQS>();
                ring_barrier();
                __builtin_amdgcn_sched_barrier(0);
                half(fa1, fb1, next, ic<0>(), fa0, fb0, IDLE, std::false_type());
                close_slice();
            }
        };
        const int mw = t.m0 + wm * S::WM, cw = t.c0 + wn * S::WN;
        if (mw >= t.rows || cw >= a.N)
            steps(std::true_type());
        else
            steps(std::false_type());

        if (mw < t.rows) {
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    // (the 8-bit codes' padding ends with the block)
                    if (cw + 32 * nb < a.N)
                        store_block<bf16_t, PASS>(a, t.g, t.part, t.row0, t.rows, mw + 32 * mb + lr, cw + 32 * nb,
                                                  lg, acc[mb][nb]);
                }
        }
    }
    // the requests past the last tile (zeros) land before the LDS is released
    wait_vmcnt<0>();
}

namespace {

template <int PASS, class S>
hipError_t launch(const LinearArgs& a0, hipStream_t st) {
    constexpr int ring = kLinSlots * lin_slot<S>();
    static hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&linear_bf16_kernel<PASS, S>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, ring);
    if (attr != hipSuccess) return attr;
    LinearArgs a = a0;
    a.ntn = (a.N + S::BN - 1) / S::BN;
    a.mtiles = PASS == kLinDw ? (a.M + S::BM - 1) / S::BM : 0;
    const int64_t mt = PASS == kLinDw ? static_cast<int64_t>(a.G) * a.mtiles : a.R / S::BM + a.G;
    const int64_t tiles = mt * a.ntn * a.parts;
    if (tiles >= (int64_t(1) << 30)) return hipErrorInvalidValue;
    int64_t blocks = std::min<int64_t>(static_cast<int64_t>(device_cus()) * S::PER_CU, tiles);
    blocks = std::max<int64_t>(8, (blocks + 7) & ~int64_t(7));
    linear_bf16_kernel<PASS, S><<<static_cast<unsigned>(blocks), lin_threads<S>(), ring, st>>>(a);
    return hipGetLastError();
}

template <int PASS>
hipError_t launch_shape(const LinearArgs& a, int shape, hipStream_t st) {
    switch (shape) {
        case 0: return launch<PASS, LinBig>(a, st);
        case 1: return launch<PASS, LinMid>(a, st);
        default: return PASS == kLinDw ? launch<PASS, LinMid>(a, st) : launch<PASS, LinSmall>(a, st);
    }
}

}  // namespace

// shape: 0 256 x 256, 1 128 x 128, 2 64 x 128 tiles
hipError_t launch_linear_bf16(int pass, const LinearArgs& a, int shape, hipStream_t st) {
    switch (pass) {
        case kLinForward: return launch_shape<kLinForward>(a, shape, st);
        case kLinDx: return launch_shape<kLinDx>(a, shape, st);
        default: return launch_shape<kLinDw>(a, shape, st);
    }
}

}  // namespace moe
