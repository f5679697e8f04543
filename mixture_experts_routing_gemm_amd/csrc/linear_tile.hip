// The linear layer's products on the matrix cores: forward, dx and dW of a
// grouped (or dense) linear layer in bf16 or float32, with the bias,
// activation and residual in the forward's epilogue. linear.h has the
// formulas and the tile list.
//
// One persistent kernel for the three products. A work-group walks its list
// of BM x BN output tiles; the operands' slices (64 bytes of k: 32 bf16 or 16
// float32 values) go global -> LDS by direct 16-byte loads into a ring of
// slots, as one stream that runs on across tiles (while a tile's epilogue
// stores, the next tile's first slices arrive). Operands are staged as they
// lie in memory: one contiguous along k as rows of 64 bytes, read by 16-byte
// LDS reads; one contiguous along m or n as rows of BM or BN values, read by
// the transposing LDS read (bf16) or value by value (float32). So neither the
// weights (dx) nor the rows (dW) are ever written out transposed.
//
// Each tile's requests go through buffer resources that start at the tile and
// end at its last row: 32-bit offsets however large the operands are, and
// rows past the end read as zeros. A slice that runs past the end of k masks
// the lanes of a k-contiguous operand by an offset beyond the resource, and
// the other kind's rows past k lie beyond it.
//
// Measured (8192 x 4096 -> 4096, bf16, 256 x 256 tiles): forward 226 us, dx 218
// (1.22 and 1.26 PFLOP/s, the clock below its peak); smaller tiles are bound by
// L2 -> LDS, about 50 GB/s a unit. float32, 128 x 128 tiles: 132 TFLOP/s, bound
// by the matrix instructions.
#include <algorithm>

#include "lds_ring.h"
#include "linear.h"

namespace moe {

int device_cus();

typedef int i32x4lin __attribute__((ext_vector_type(4)));
typedef short v4i16lin __attribute__((ext_vector_type(4)));

// byte offset of 16-byte chunk c (0..3) of row r of a k-contiguous slice; the
// XOR spreads aligned runs of 8 rows over the banks
__device__ __forceinline__ int lin_swz(int r) { return ((r >> 1) & 3) ^ ((r >> 3) & 1); }
__device__ __forceinline__ int lin_koff(int r, int c) { return (r << 6) + ((c ^ lin_swz(r)) << 4); }
// chunk swizzle of slice row k of an m- or n-contiguous operand. bf16: the
// transposing reads (4 rows of 32 or 64 bytes at a time) hit distinct banks;
// float32: so do the two halves of a wave, which read rows four apart (rows of
// W >= 64 values; the 32 of a narrower one have the same banks in each row).
template <typename T, int W>
__device__ __forceinline__ int lin_tsw(int k) {
    if constexpr (sizeof(T) == 2) return (0xEA40 >> (4 * (k & 3))) & 15;  // 0, 4, 10, 14
    else return W >= 64 ? ((k >> 2) & 1) << 3 : 0;
}

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

// The tile shapes: BM x BN by waves of WM x WN, SLOTS slots of the ring, the
// first ISS waves issue the requests, PER_CU work-groups a compute unit; KG
// sets of such waves, each with a ring of its own and its share of the tile's
// k, whose sums are added in the end. A step of one set is a chain (barrier,
// LDS reads, products), in float32 twice as long as its products (64 x 64: 0.40
// us against 0.21): a second set on the unit takes its steps meanwhile, where
// there is no second tile to do so (0.28 us; bf16 tiles, bound by what arrives
// in LDS, gained 5 to 10 per cent at long k and nothing below).
struct LinBig {
    static constexpr int BM = 256, BN = 256, WM = 128, WN = 64, ISS = 8, SLOTS = 4, PER_CU = 1, KG = 1;
};
struct LinHalf {
    static constexpr int BM = 256, BN = 128, WM = 128, WN = 64, ISS = 4, SLOTS = 3, PER_CU = 2, KG = 1;
};
struct LinMid {
    static constexpr int BM = 128, BN = 128, WM = 64, WN = 64, ISS = 4, SLOTS = 4, PER_CU = 2, KG = 1;
};
struct LinSmall {
    static constexpr int BM = 64, BN = 128, WM = 32, WN = 64, ISS = 4, SLOTS = 4, PER_CU = 3, KG = 1;
};
struct LinTiny {
    static constexpr int BM = 64, BN = 64, WM = 32, WN = 32, ISS = 4, SLOTS = 4, PER_CU = 2, KG = 2;
};
struct LinSlim {
    static constexpr int BM = 64, BN = 32, WM = 32, WN = 32, ISS = 2, SLOTS = 4, PER_CU = 3, KG = 2;
};
// waves of a set, threads of a work-group
template <class S>
constexpr int lin_waves() {
    return (S::BM / S::WM) * (S::BN / S::WN);
}
template <class S>
constexpr int lin_threads() {
    return lin_waves<S>() * S::KG * 64;
}
template <class S>
constexpr int lin_slot() {
    return (S::BM + S::BN) * 64;
}
template <class S>
constexpr int lin_ring() {
    return S::KG * S::SLOTS * lin_slot<S>();
}
template <class S>
constexpr int lin_waves_per_simd() {
    return lin_threads<S>() * S::PER_CU / 256;
}

// One operand's side of the request stream. TR: contiguous along m or n
// (columns col0 .. of rows k); else rows row0 .. contiguous along k.
template <typename T, bool TR, int W>
struct LinOperand {
    static constexpr int ES = sizeof(T), SK = 64 / ES;  // k values a slice
    static constexpr int kBytes = W * 64;

    // this lane's byte offset in request i (1 KB of the slice): constant over
    // slices and tiles. ld: values a row.
    __device__ static uint32_t lane_offset(int i, int lane, int64_t ld) {
        if constexpr (TR) {
            constexpr int CH = W * ES / 16;  // 16-byte chunks a row
            const int k = i * (64 / CH) + lane / CH;
            return static_cast<uint32_t>(k * ld * ES) + 16u * ((lane % CH) ^ lin_tsw<T, W>(k));
        } else {
            const int r = 16 * i + (lane >> 2);
            return static_cast<uint32_t>(r * ld * ES) + 16u * ((lane & 3) ^ lin_swz(r));
        }
    }
    // resource of the slice at k: `base` points at the operand's tile
    // (k-contiguous: its first row; else the row of k = 0 at the tile's first
    // column)
    __device__ static i32x4lin resource(const uint8_t* base, int64_t ld, int k, int kend, int valid) {
        if constexpr (TR) {
            const int n = min(SK, kend - k);  // valid: columns from the tile's first one on
            const uint32_t bytes = n > 0 ? static_cast<uint32_t>(((n - 1) * ld + valid) * ES) : 0u;
            return lin_rsrc(base + k * ld * ES, bytes);
        } else {
            // valid: rows of the tile
            const uint32_t bytes = kend > k ? static_cast<uint32_t>((valid * ld - k) * ES) : 0u;
            return lin_rsrc(base + static_cast<int64_t>(k) * ES, bytes);
        }
    }
    // this lane's fragment offset within a slice, for features f0 .. f0+31 of
    // half-slice ks
    __device__ static uint32_t frag_offset(int f0, int ks, int lane) {
        if constexpr (!TR) {
            return static_cast<uint32_t>(lin_koff(f0 + (lane & 31), 2 * ks + (lane >> 5)));
        } else if constexpr (ES == 2) {
            const int g = lane >> 4, s = lane & 15;
            const int k = 16 * ks + 8 * (g >> 1) + (s >> 2);
            const int f = f0 + 16 * (g & 1) + 4 * (s & 3);
            return static_cast<uint32_t>(k * W * 2 + (((f >> 3) ^ lin_tsw<T, W>(k)) << 4) + (f & 7) * 2);
        } else {
            const int k = 8 * ks + 4 * (lane >> 5), f = f0 + (lane & 31);
            return static_cast<uint32_t>(k * W * 4 + (((f >> 2) ^ lin_tsw<T, W>(k)) << 4) + (f & 3) * 4);
        }
    }
    // 16 bytes of k values of one feature: bf16 k = 16 ks + 8 (lane / 32) ..
    // +7, float32 k = 8 ks + 4 (lane / 32) .. +3
    __device__ static u32x4 fragment(const uint8_t* lds, uint32_t at) {
        if constexpr (!TR) {
            return *reinterpret_cast<const u32x4*>(lds + at);
        } else if constexpr (ES == 2) {
            typedef __attribute__((address_space(3))) v4i16lin lv4;
            const __attribute__((address_space(3))) uint8_t* p =
                (const __attribute__((address_space(3))) uint8_t*)lds + at;
            const v4i16lin lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lv4*)p);
            const v4i16lin hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lv4*)(p + 4 * W * 2));
            return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            u32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const uint32_t*>(lds + at + j * W * 4);
            return v;
        }
    }
};

// acc += the products of one half-slice: first operand B (columns), second A
// (rows). float32: four 32x32x2 steps, each of them the j-th of the four k
// values that either half of the wave holds.
template <typename T>
__device__ __forceinline__ void lin_mma(const u32x4& fb, const u32x4& fa, f32x16& acc) {
    if constexpr (sizeof(T) == 2) {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, fb), __builtin_bit_cast(bf16x8, fa),
                                                      acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(fb[j]), __uint_as_float(fa[j]), acc, 0, 0, 0);
    }
}

// The tiles of work-group `bid` of `nblk`.
template <typename T, int PASS, class S>
__device__ __forceinline__ void linear_tiles(const LinearArgs& a, int bid, int nblk) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ GroupWalk walk;
    __shared__ GroupOrder order;
    // the bias of a tile's columns, by list position: the request stream is at
    // most three tiles ahead of the tile whose epilogue reads it
    __shared__ __attribute__((aligned(16))) float bias_lds[4][256];
    constexpr int BM = S::BM, BN = S::BN, SLOTS = S::SLOTS;
    constexpr int WN_WAVES = BN / S::WN;
    constexpr int MB = S::WM / 32, NB = S::WN / 32;
    constexpr int RA = BM / 16 / S::ISS, RB = BN / 16 / S::ISS, REQS = RA + RB;
    constexpr int kSlot = lin_slot<S>();
    typedef LinOperand<T, PASS == kLinDw, BM> OpA;
    typedef LinOperand<T, PASS != kLinForward, BN> OpB;
    constexpr int ES = sizeof(T), SK = 64 / ES;
    constexpr int KG = S::KG, WAVES = lin_waves<S>();
    // Outputs in bf16 go through LDS, 32 rows x 64 columns a wave at a time,
    // so that a store instruction writes 8 rows x 128 bytes (as the
    // accumulators hold them: 32 rows x 32 bytes, a quarter of each line).
    constexpr bool kStage = ES == 2 && S::WN == 64 && (KG > 1 || kSlot >= WAVES * 4096);
    // the other sets' sums (KG > 1), and the staging area behind them
    constexpr int kSums = (KG - 1) * WAVES * MB * NB * 4096;
    static_assert(KG == 1 || kSums + (kStage ? WAVES * 4096 : 0) <= lin_ring<S>(), "LDS of the epilogue");
    static_assert(KG == 1 || PASS <= kLinDw, "one segment");
    // stores of a full tile by a wave, at least (see the waits below)
    constexpr int kStores = kStage && KG == 1 ? 4 * MB : 0;

    walk_groups(walk, a.offsets, a.R, a.G, BM, bid == 0 ? a.hdr : nullptr);
    if constexpr (PASS == kLinDw) order_groups(order, walk, a.G);

    const int tid = threadIdx.x;
    const int wave_all = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    // the set, its ring, and the wave within it
    const int set = KG > 1 ? wave_all / WAVES : 0, wave = KG > 1 ? wave_all % WAVES : wave_all;
    const int ring = set * SLOTS * kSlot;
    const int wm = wave / WN_WAVES, wn = wave % WN_WAVES;
    const int lr = lane & 31, lg = lane >> 5;
    const bool issuer = S::ISS == WAVES || wave < S::ISS;

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
    const int kc = 16 / ES * ((lane & 3) ^ lin_swz(lane >> 2));
    // where the next slice comes from: operand bases of the tile, the rows or
    // columns that they hold, k and its end, and the next list position (kept
    // and returned by value: state changed through captured references went
    // through scratch memory, and the wait for it drained the slices in flight)
    struct Source {
        const uint8_t* a;
        const uint8_t* b;
        int valid_a, valid_b, k, kend, list;
        int first, g, c0;  // forward: this is the tile's first slice; its group and column
        int kb, seg;       // kLinDx2: k within the segment of b; the segment's number
    };
    // kLinDx2: the first row of segment i of the tile's k, at the tile's column
    auto segment = [&](int g, int i, int c0) {
        const uint8_t* w = (i & 1) != 0 ? a.b2 : a.b;
        return w + (static_cast<int64_t>(g + (i >> 1)) * a.seg * a.N + c0) * ES;
    };
    auto source_of = [&](const LinTile& t, bool more, int list) {
        Source src;
        src.list = list;
        src.first = more ? 1 : 0;
        src.g = t.g;
        src.c0 = t.c0;
        src.k = more ? t.k0 : 0;
        src.kend = more ? t.k1 : 0;  // nothing more: empty resources, zeros
        if constexpr (PASS == kLinDw) {
            src.a = a.a + static_cast<int64_t>(t.m0) * ES;
            src.b = a.b + static_cast<int64_t>(t.c0) * ES;
            src.valid_a = a.M - t.m0;
            src.valid_b = a.N - t.c0;
        } else {
            src.a = a.a + (t.row0 + t.m0) * lda * ES;
            src.valid_a = min(BM, t.rows - t.m0);
            const int64_t wbase = static_cast<int64_t>(t.g) * a.N * a.K;
            if constexpr (PASS == kLinForward) {
                src.b = a.b + (wbase + t.c0 * ldb) * ES;
                src.valid_b = min(BN, a.N - t.c0);
            } else {
                src.b = PASS == kLinDx2 ? segment(t.g, 0, t.c0) : a.b + (wbase + t.c0) * ES;
                src.valid_b = a.N - t.c0;
            }
        }
        src.kb = src.seg = 0;
        return src;
    };
    auto next_source = [&](int list) {
        LinTile t;
        bool more = lin_tile<PASS, BM, BN, SK>(a, walk, order, bid, nblk, list, t);
        ++list;
        while (more && t.k1 <= t.k0) {  // (a group without rows, or an empty part)
            more = lin_tile<PASS, BM, BN, SK>(a, walk, order, bid, nblk, list, t);
            ++list;
        }
        return source_of(t, more, list);
    };
    Source src;
    i32x4lin rsa, rsb;
    uint32_t slot_addr;
    bool in_a, in_b;  // this lane's chunk lies before the end of k
    auto open_slice = [&](int slot) {
        rsa = OpA::resource(src.a, lda, src.k, src.kend, src.valid_a);
        rsb = PASS == kLinDx2 ? OpB::resource(src.b, ldb, src.kb, src.kend > src.k ? a.seg : 0, src.valid_b)
                              : OpB::resource(src.b, ldb, src.k, src.kend, src.valid_b);
        in_a = PASS == kLinDw || kc < src.kend - src.k;
        in_b = PASS != kLinForward || kc < src.kend - src.k;
        slot_addr = __builtin_amdgcn_readfirstlane(lin_lds_addr(lds) + ring + slot * kSlot);
        if constexpr (PASS == kLinForward && kStage) {
            // the tile's bias (zeros without one) lands before its first slice
            if (wave_all == 0 && src.first != 0) {
                const uint32_t bytes = a.bias != nullptr ? min(BN, a.N - src.c0) * 4 : 0;
                lin_dma16(lin_rsrc(reinterpret_cast<const uint8_t*>(a.bias + static_cast<int64_t>(src.g) * a.N + src.c0), bytes),
                          16u * lane,
                          __builtin_amdgcn_readfirstlane(lin_lds_addr(reinterpret_cast<const uint8_t*>(bias_lds)) +
                                                         1024 * ((src.list - 1) & 3)));
            }
            src.first = 0;
        }
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
        src.k += SK;
        if constexpr (PASS == kLinDx2) {  // (seg is a multiple of SK)
            src.kb += SK;
            if (src.kb >= a.seg && src.k < src.kend) {
                src.kb = 0;
                ++src.seg;
                src.b = segment(src.g, src.seg, src.c0);
            }
        }
        // (several sets: past its share a set requests zeros)
        if (KG == 1 && src.k >= src.kend) src = next_source(src.list);
    };
    // slot numbers go round
    auto slot_after = [](int s, int n) { return s + n >= SLOTS ? s + n - SLOTS : s + n; };

    // ---- fragments ----
    // (k-contiguous: block i lies 32 rows of 64 bytes further, the swizzle is
    // the same, and the half-slices have an offset each. Transposed: the XOR
    // does not commute with adding blocks, so each block has its offset, and
    // half-slice 1 lies SK / 2 rows further with the same swizzle.)
    uint32_t fo_a[PASS == kLinDw ? MB : 2], fo_b[PASS != kLinForward ? NB : 2];
#pragma unroll
    for (int i = 0; i < (PASS == kLinDw ? MB : 2); ++i)
        fo_a[i] = PASS == kLinDw ? OpA::frag_offset(wm * S::WM + 32 * i, 0, lane) : OpA::frag_offset(wm * S::WM, i, lane);
#pragma unroll
    for (int i = 0; i < (PASS != kLinForward ? NB : 2); ++i)
        fo_b[i] = OpA::kBytes + (PASS != kLinForward ? OpB::frag_offset(wn * S::WN + 32 * i, 0, lane)
                                                     : OpB::frag_offset(wn * S::WN, i, lane));
    auto frag_a = [&](uint32_t slot_off, auto KS, int i) -> u32x4 {
        constexpr int ks = decltype(KS)::value;
        if constexpr (PASS == kLinDw)
            return OpA::fragment(lds, ring + slot_off + fo_a[i] + ks * 32 * BM);
        else
            return OpA::fragment(lds, ring + slot_off + fo_a[ks] + i * 2048);
    };
    auto frag_b = [&](uint32_t slot_off, auto KS, int i) -> u32x4 {
        constexpr int ks = decltype(KS)::value;
        if constexpr (PASS != kLinForward)
            return OpB::fragment(lds, ring + slot_off + fo_b[i] + ks * 32 * BN);
        else
            return OpB::fragment(lds, ring + slot_off + fo_b[ks] + i * 2048);
    };

    f32x16 acc[MB][NB];
    u32x4 fa0[MB], fb0[NB], fa1[MB], fb1[NB];
    // the MFMAs on one half-slice (fa, fb), each followed by one request (in
    // the first half) and the read of one fragment of half-slice KS of a slot
    auto half = [&](u32x4 (&fa)[MB], u32x4 (&fb)[NB], uint32_t slot_off, auto KS, u32x4 (&na)[MB], u32x4 (&nb)[NB],
                    auto IDLE, auto ISSUE) {
        constexpr bool idle = decltype(IDLE)::value;
        constexpr int n1 = MB * NB > MB + NB ? MB * NB : MB + NB;
        constexpr int n = decltype(ISSUE)::value && REQS > n1 ? REQS : n1;
        static_for<0, n>([&](auto I) {
            constexpr int i = decltype(I)::value;
            if constexpr (!idle && i < MB * NB) lin_mma<T>(fb[i % NB], fa[i / NB], acc[i / NB][i % NB]);
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

    auto first_fragments = [&](uint32_t slot_off) {
        static_for<0, MB + NB>([&](auto I) {
            constexpr int i = decltype(I)::value;
            if constexpr (i < NB)
                fb0[i] = frag_b(slot_off, ic<0>(), i);
            else
                fa0[i - NB] = frag_a(slot_off, ic<0>(), i - NB);
        });
    };
    // all slots but one
    auto fill_ring = [&]() {
        for (int s = 0; s < SLOTS - 1; ++s) {
            open_slice(s);
            if (issuer) static_for<0, REQS>(request);
            close_slice();
        }
        wait_vmcnt<(SLOTS - 2) * REQS>();
        ring_barrier();
        first_fragments(0);
    };
    if constexpr (KG == 1) {
        src = next_source(0);
        fill_ring();
    }

    int slot = 0;   // of the next slice to compute
    int relax = 0;  // steps left whose wait may leave the last tile's stores under way
    for (int it = 0;; ++it) {
        LinTile t;
        if (!lin_tile<PASS, BM, BN, SK>(a, walk, order, bid, nblk, it, t)) break;
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
        int KT = (t.k1 - t.k0 + SK - 1) / SK;
        if constexpr (KG > 1) {
            // a tile at a time: its sums go through the ring
            KT = (KT + KG - 1) / KG;
            LinTile mine = t;
            mine.k0 = min(t.k1, t.k0 + SK * KT * set);
            mine.k1 = min(t.k1, mine.k0 + SK * KT);
            src = source_of(mine, true, it + 1);
            slot = 0;
            fill_ring();
        }
        // Step: the slice in `slot`, its first fragments in fa0, fb0. The
        // first half computes on them, requests a slice into the slot before
        // (read to its end before the last barrier) and reads the second
        // half's fragments; then the next slice has to have landed (the
        // requests of the SLOTS - 2 after it may be under way), and the second
        // half reads its first fragments, which may be the next tile's.
        // Memory operations complete in order as far as the counter shows:
        // in the first SLOTS - 2 steps after an epilogue its stores come after
        // the slice waited for, and the wait leaves them under way too (where
        // their number is known: a tile without edges).
        // A wave without rows or columns in the tile (idle) computes nothing.
        auto steps = [&](auto IDLE) {
            for (int k = 0; k < KT; ++k) {
                const int nslot = slot_after(slot, 1);
                open_slice(slot_after(slot, SLOTS - 1));
                half(fa0, fb0, slot * kSlot, ic<1>(), fa1, fb1, IDLE, std::true_type());
                close_slice();
                if (kStores > 0 && relax > 0) {
                    wait_vmcnt<(SLOTS - 2) * REQS + kStores>();
                    --relax;
                } else {
                    wait_vmcnt<(SLOTS - 2) * REQS>();
                }
                ring_barrier();
                __builtin_amdgcn_sched_barrier(0);
                half(fa1, fb1, nslot * kSlot, ic<0>(), fa0, fb0, IDLE, std::false_type());
                slot = nslot;
            }
        };
        const int mw = t.m0 + wm * S::WM, cw = t.c0 + wn * S::WN;
        const bool idle = mw >= t.rows || cw >= a.N;
        if (idle)
            steps(std::true_type());
        else
            steps(std::false_type());

        if constexpr (KG > 1) {
            // the requests past the end (zeros) have landed; the other sets'
            // sums, added in their order
            wait_vmcnt<0>();
            ring_barrier();
            constexpr int NBLK = MB * NB;
            const auto sums = [&](int from, int i, int q) {
                return lds + ((((from - 1) * WAVES + wave) * NBLK + i) * 4 + q) * 1024 + 16 * lane;
            };
            if (set > 0 && !idle) {
#pragma unroll
                for (int i = 0; i < NBLK; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x16& v = acc[i / NB][i % NB];
                        *reinterpret_cast<f32x4*>(sums(set, i, q)) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                    }
            }
            wait_vmcnt<0>();
            ring_barrier();
            if (set == 0 && !idle) {
#pragma unroll
                for (int f = 1; f < KG; ++f)
#pragma unroll
                    for (int i = 0; i < NBLK; ++i)
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const f32x4 v = *reinterpret_cast<const f32x4*>(sums(f, i, q));
#pragma unroll
                            for (int u = 0; u < 4; ++u) acc[i / NB][i % NB][4 * q + u] += v[u];
                        }
            }
        }
        const bool store = !idle && set == 0;
        bool staged = false;
        if constexpr (kStage) staged = a.part_out == nullptr && !(PASS == kLinDw && a.out_f32);
        if (staged) {
            if constexpr (kStage) {
                // the slot before is free until the next step's requests
                if (store) {
                    uint8_t* stage = lds + (KG > 1 ? kSums : slot_after(slot, SLOTS - 1) * kSlot) + wave * 4096;
                    if constexpr (PASS == kLinDh8)
                        store_tile_dh8<MB, NB>(a, t, mw, cw, stage, lane, acc);
                    else
                        store_tile_staged<PASS, MB, NB>(a, t, mw, cw, stage, bias_lds[it & 3], lane, acc);
                }
                relax = !idle && mw + S::WM <= t.rows && cw + S::WN <= a.N ? SLOTS - 2 : 0;
                ring_barrier();  // every wave is done with its stage
                // (read again, so that they take no registers in the epilogue)
                if constexpr (KG == 1) first_fragments(slot * kSlot);
            }
        } else if (PASS <= kLinDw && store) {
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    // (the 8-bit codes' padding ends with the block)
                    if (cw + 32 * nb < a.N)
                        store_block<T, PASS, kStage>(a, t.g, t.part, t.row0, t.rows, mw + 32 * mb + lr, cw + 32 * nb, lg,
                                             acc[mb][nb]);
                }
        }
        if constexpr (KG > 1) {
            if (!staged) ring_barrier();  // (the next tile's slices go where the sums were)
        }
    }
    // the requests past the last tile (zeros) land before the LDS is released
    wait_vmcnt<0>();
}

template <typename T, int PASS, class S>
__global__ __launch_bounds__(lin_threads<S>())
    __attribute__((amdgpu_waves_per_eu(lin_waves_per_simd<S>(), lin_waves_per_simd<S>())))
void linear_tile_kernel(LinearArgs a) {
    linear_tiles<T, PASS, S>(a, blockIdx.x, gridDim.x);
}

// Two sets of tiles in one launch, `first` of the work-groups on the first (a
// multiple of 8): the routed experts' and the shared ones'.
template <typename T, int PASS, class S>
__global__ __launch_bounds__(lin_threads<S>())
    __attribute__((amdgpu_waves_per_eu(lin_waves_per_simd<S>(), lin_waves_per_simd<S>())))
void linear_pair_kernel(LinearArgs r, LinearArgs s, int first) {
    if (static_cast<int>(blockIdx.x) < first)
        linear_tiles<T, PASS, S>(r, blockIdx.x, first);
    else
        linear_tiles<T, PASS, S>(s, blockIdx.x - first, gridDim.x - first);
}

// dx, dW and db of a small layer in one launch: none needs another's result,
// and each alone leaves most units idle. Work-groups 0 .. nx-1 take dx's
// tiles, nx .. nx+nw-1 dW's, the rest db's columns (nx and nw multiples of 8).
template <typename T, class S>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(S::PER_CU, S::PER_CU)))
void linear_backward_kernel(LinearArgs x, LinearArgs w, DbArgs d, int nx, int nw) {
    static_assert(lin_threads<S>() == 256, "four waves");
    const int b = blockIdx.x;
    if (b < nx) {
        linear_tiles<T, kLinDx, S>(x, b, nx);
    } else if (b < nx + nw) {
        linear_tiles<T, kLinDw, S>(w, b - nx, nw);
    } else {
        const int cbs = (d.N + 63) / 64, i = b - nx - nw;
        linear_db_block<T, 4>(d, i / cbs, i % cbs);
    }
}

namespace {

// fills in the tile counts and gives the work-groups, or 0 for too many tiles
template <int PASS, class S>
unsigned tile_grid(LinearArgs& a) {
    a.ntn = (a.N + S::BN - 1) / S::BN;
    a.mtiles = PASS == kLinDw ? (a.M + S::BM - 1) / S::BM : 0;
    const int64_t mt = PASS == kLinDw ? static_cast<int64_t>(a.G) * a.mtiles
                                      : a.same_rows ? a.G * ((a.R + S::BM - 1) / S::BM) : a.R / S::BM + a.G;
    const int64_t tiles = mt * a.ntn * a.parts;
    if (tiles >= (int64_t(1) << 30)) return 0;
    const int64_t blocks = std::min<int64_t>(static_cast<int64_t>(device_cus()) * S::PER_CU, tiles);
    return static_cast<unsigned>(std::max<int64_t>(8, (blocks + 7) & ~int64_t(7)));
}

template <typename T, int PASS, class S>
hipError_t launch(const LinearArgs& a0, hipStream_t st) {
    constexpr int ring = lin_ring<S>();
    static hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&linear_tile_kernel<T, PASS, S>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, ring);
    if (attr != hipSuccess) return attr;
    LinearArgs a = a0;
    const unsigned blocks = tile_grid<PASS, S>(a);
    if (blocks == 0) return hipErrorInvalidValue;
    linear_tile_kernel<T, PASS, S><<<blocks, lin_threads<S>(), ring, st>>>(a);
    return hipGetLastError();
}

template <typename T, class S>
hipError_t launch_backward(const LinearArgs& x0, const LinearArgs& w0, const DbArgs& d, hipStream_t st) {
    constexpr int ring = lin_ring<S>();
    static hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&linear_backward_kernel<T, S>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, ring);
    if (attr != hipSuccess) return attr;
    LinearArgs x = x0, w = w0;
    const unsigned nx = x.out != nullptr ? tile_grid<kLinDx, S>(x) : 0, nw = w.out != nullptr ? tile_grid<kLinDw, S>(w) : 0;
    if ((x.out != nullptr && nx == 0) || (w.out != nullptr && nw == 0)) return hipErrorInvalidValue;
    const unsigned nb = d.db != nullptr ? static_cast<unsigned>(d.G) * ((d.N + 63) / 64) : 0;
    if (nx + nw + nb == 0) return hipSuccess;
    linear_backward_kernel<T, S><<<nx + nw + nb, 256, ring, st>>>(x, w, d, static_cast<int>(nx), static_cast<int>(nw));
    return hipGetLastError();
}

template <int PASS, class S>
hipError_t launch_pair(const LinearArgs& r0, const LinearArgs& s0, hipStream_t st) {
    constexpr int ring = lin_ring<S>();
    static hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&linear_pair_kernel<bf16_t, PASS, S>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, ring);
    if (attr != hipSuccess) return attr;
    LinearArgs r = r0, s = s0;
    unsigned nr = tile_grid<PASS, S>(r), ns = s.out != nullptr ? tile_grid<PASS, S>(s) : 0;
    if (nr == 0 || (s.out != nullptr && ns == 0)) return hipErrorInvalidValue;
    // where there are not units enough for both, they are shared out by work
    // (each set with a work-group for every unit, the second set's tiles began
    // when the first's were done: dx of 4096 tokens, eight experts of 32 and two
    // shared, whose tiles take twice as long, 558 us)
    const unsigned units = static_cast<unsigned>(device_cus() * S::PER_CU) & ~7u;
    if (ns > 0 && nr + ns > units) {
        const double wr = static_cast<double>(r.R) * r.K, ws = static_cast<double>(s.R) * s.K * (s.same_rows ? s.G : 1);
        const unsigned part = (static_cast<unsigned>(units * (ws / (wr + ws))) + 7) & ~7u;
        ns = std::min(ns, std::max(8u, std::min(part, units - 8)));
        nr = std::min(nr, units - ns);
    }
    linear_pair_kernel<bf16_t, PASS, S><<<nr + ns, lin_threads<S>(), ring, st>>>(r, s, static_cast<int>(nr));
    return hipGetLastError();
}

template <int PASS>
hipError_t launch_pair_shape(const LinearArgs& r, const LinearArgs& s, int shape, hipStream_t st) {
    switch (shape) {
        case kLinTileBig: return launch_pair<PASS, LinBig>(r, s, st);
        case kLinTileHalf: return launch_pair<PASS, LinHalf>(r, s, st);
        default: return launch_pair<PASS, LinMid>(r, s, st);
    }
}

template <int PASS>
hipError_t launch_pass(const LinearArgs& a, int shape, bool f32, hipStream_t st) {
    if (f32) {
        switch (shape) {
            case kLinTileMid: return launch<float, PASS, LinMid>(a, st);
            case kLinTileTiny: return launch<float, PASS, LinTiny>(a, st);
            default: return launch<float, PASS, LinSlim>(a, st);
        }
    }
    switch (shape) {
        case kLinTileBig: return launch<bf16_t, PASS, LinBig>(a, st);
        case kLinTileHalf: return launch<bf16_t, PASS, LinHalf>(a, st);
        case kLinTileSmall:
            if constexpr (PASS != kLinDw) return launch<bf16_t, PASS, LinSmall>(a, st);
            break;
        default: break;
    }
    return launch<bf16_t, PASS, LinMid>(a, st);
}

}  // namespace

// kLinDh8 or kLinDx2, the routed experts' tiles and (s.out not NULL) the shared
// experts'; bf16, Big, Half or Mid
hipError_t launch_linear_pair(int pass, const LinearArgs& r, const LinearArgs& s, int shape, hipStream_t st) {
    return pass == kLinDh8 ? launch_pair_shape<kLinDh8>(r, s, shape, st) : launch_pair_shape<kLinDx2>(r, s, shape, st);
}

// dx, dW and db together (out or db NULL: not computed), 128 x 128 tiles in
// bf16, 64 x 32 in float32, k not split
hipError_t launch_linear_backward(const LinearArgs& x, const LinearArgs& w, const DbArgs& d, bool f32, hipStream_t st) {
    return f32 ? launch_backward<float, LinSlim>(x, w, d, st) : launch_backward<bf16_t, LinMid>(x, w, d, st);
}

// shape: a LinTileShape (float32: Mid, Tiny or Slim; bf16: Big to Small; dW: not Small)
hipError_t launch_linear_tile(int pass, const LinearArgs& a, int shape, bool f32, hipStream_t st) {
    switch (pass) {
        case kLinForward: return launch_pass<kLinForward>(a, shape, f32, st);
        case kLinDx: return launch_pass<kLinDx>(a, shape, f32, st);
        default: return launch_pass<kLinDw>(a, shape, f32, st);
    }
}

}  // namespace moe
