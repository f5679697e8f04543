// What the linear layer's kernels share: the arguments, the walk over ragged
// groups, the activation functions and the epilogue.
//
// The layer: rows x [R, K] sorted by group, group g holding the rows
// offsets[g] .. offsets[g+1]-1 (one group of all R rows without offsets), and
//     z[r] = W_g x[r] + b_g,   y[r] = fn(z[r]) + residual[r]
// with W [G, N, K]; backward, with zs the pre-activation as it was saved,
//     dz = dy fn'(zs),  dx[r] = dz[r] W_g,  dW_g = sum_r dz[r] x[r]^T,
//     db_g = sum_r dz[r].
// One tile kernel computes C [M, N] = sum_k A(m, k) B(n, k) for all three:
//     forward  A = x rows,   B = W_g rows        (both contiguous along k)
//     dx       A = dz rows,  B = W_g columns     (B contiguous along n)
//     dW       A = dz cols,  B = x columns       (both contiguous along m / n,
//                                                 k runs over the group's rows)
#pragma once

#include "moe_device.h"
#include "rows8.h"

namespace moe {

constexpr int kMaxGroups = 256;

// For the SwiGLU experts' backward from 8 bits: kLinDh8 is dx of the
// down-projection, dhid = dy W2, with the SwiGLU backward in its epilogue;
// kLinDx2 is dx of the up-projections, [da | db] [W1; W3], k running over
// segments of W1 and W3 in turn.
enum LinearPass { kLinForward = 0, kLinDx = 1, kLinDw = 2, kLinDh8 = 3, kLinDx2 = 4 };
// output tiles: 256 x 256, 256 x 128, 128 x 128, 64 x 128, 64 x 64, 64 x 32
enum LinTileShape {
    kLinTileBig = 0,
    kLinTileHalf = 1,
    kLinTileMid = 2,
    kLinTileSmall = 3,
    kLinTileTiny = 4,
    kLinTileSlim = 5
};

struct LinearArgs {
    const uint8_t* a;        // x (forward), dz (dx, dW)
    const uint8_t* b;        // W (forward, dx), x (dW)
    const int32_t* offsets;  // [G+1], NULL: one group of R rows
    uint32_t* hdr;           // error flag of the workspace, or NULL
    int64_t R;
    int G;
    int M, N, K;             // M: dW only (n_out); K: forward and dx
    int mtiles, ntn;         // dW: m-tiles a group; n-tiles
    // epilogue
    int fn;
    const float* bias;       // [G, N] or NULL
    const uint8_t* residual; // [R, N] (act) or NULL
    uint8_t* out;            // y / dx [R, N] (act), dW [G, M, N] (act or float32)
    uint8_t* zsave;          // saved pre-activations [R, N] (act), or NULL
    uint8_t* codes;          // saved pre-activations in 8 bits, or NULL
    uint8_t* scales;
    int64_t n32;             // row stride of the codes
    int out_f32;             // dW: float32 output
    // split along k: part s of `parts` writes its float32 sums to
    // part_out [parts][rows][N] (rows: R, or G * M for dW), joined later
    float* part_out;
    int parts;
    // every group holds all R rows (the shared experts); without offsets only
    int same_rows;
    // kLinDh8: a and b in 8 bits and hid, rows of ldp values, group g's at
    // column g N (same_rows) or 0; out: [da | db] rows of 2 ldp values, group
    // g's at column 2 g N or 0
    const uint8_t* ca;
    const uint8_t* cb;
    const uint8_t* sa;
    const uint8_t* sb;
    uint8_t* hid;
    int ldp;
    // kLinDx2: b is W1 and b2 W3, segments of seg k values: W1 of the group,
    // its W3, then the next group's
    const uint8_t* b2;
    int seg;
};

// ------------------------------------------------------------ functions --
// (A 256 x 256 tile's epilogue is bound by its vector instructions, 4 cycles
// each and 16 for exp and rcp: 128 values a lane, two waves a SIMD. The forms
// below are the ones with the fewest.)
__device__ __forceinline__ float lin_sigmoid(float v) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504088896341f));
}

// Phi(-|v|), the normal distribution's tail, from Abramowitz and Stegun's
// formula 7.1.26 for erf (off by at most 1.5e-7): with x = |v| / sqrt(2) and
// t = 1 / (1 + 0.3275911 x), erfc(x) = t (a1 + t (a2 + t (a3 + t (a4 + t a5))))
// e^(-x x), and Phi(-|v|) = erfc(x) / 2 (the halves are in the coefficients).
// Also gives e = e^(-v v / 2) = 2^(-s s), s = v sqrt(log2(e) / 2).
__device__ __forceinline__ float normal_tail(float v, float& e) {
    const float s = v * 0.849321800288019f;
    e = __builtin_amdgcn_exp2f(-(s * s));
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.27273748f, __builtin_fabsf(s), 1.0f));
    float p = __builtin_fmaf(0.5307027145f, t, -0.7265760135f);
    p = __builtin_fmaf(p, t, 0.7107068705f);
    p = __builtin_fmaf(p, t, -0.142248368f);
    p = __builtin_fmaf(p, t, 0.127414796f);
    return p * t * e;
}

// (the bounds on z keep an infinity from meeting a zero factor: gelu(-inf) and
// silu(-inf) are 0, gelu(inf) is inf; a NaN stays one through the other factor)
__device__ __forceinline__ float lin_fn(int fn, float z) {
    if (fn == MOE_FN_RELU) return z < 0.0f ? 0.0f : z;
    if (fn == MOE_FN_GELU) {
        // z >= 0: z (1 - tail); z < 0: z tail
        float e;
        const float tail = normal_tail(z, e);
        return __builtin_fmaf(-__builtin_fminf(__builtin_fabsf(z), 64.0f), tail, __builtin_fmaxf(z, 0.0f));
    }
    if (fn == MOE_FN_SILU) return __builtin_fmaxf(z, -1e4f) * lin_sigmoid(z);
    return z;
}
__device__ __forceinline__ float lin_slope(int fn, float z) {
    if (fn == MOE_FN_RELU) return z > 0.0f ? 1.0f : (z <= 0.0f ? 0.0f : z);
    if (fn == MOE_FN_GELU) {
        // Phi(z) + z times the density, e / sqrt(2 pi)
        float e;
        const float tail = normal_tail(z, e);
        const float cdf = 0.5f + __builtin_copysignf(0.5f - tail, z);
        return __builtin_fmaf(__builtin_amdgcn_fmed3f(z, -64.0f, 64.0f) * e, 0.39894228040143268f, cdf);
    }
    if (fn == MOE_FN_SILU) {
        const float s = lin_sigmoid(z);
        return s * __builtin_fmaf(__builtin_amdgcn_fmed3f(z, -1e4f, 1e4f), 1.0f - s, 1.0f);
    }
    return 1.0f;
}

// ------------------------------------------------------------ group walk --
// Row ranges of the groups and the prefix of their m-tiles, in LDS. Offsets
// are taken into [0, R] and made non-decreasing (each becomes the largest so
// far), so that no row outside the buffers is ever touched; offsets that this
// changes are reported through the workspace's error flag.
struct GroupWalk {
    int off[kMaxGroups + 1];
    int pre[kMaxGroups + 1];
};

// by every thread of a work-group of at least one wave; ends with a barrier.
// hdr: the workspace's header (one work-group of a launch reports), or NULL
__device__ __forceinline__ void walk_groups(GroupWalk& w, const int32_t* __restrict__ offsets, int64_t R, int G,
                                            int bm, uint32_t* hdr) {
    const int R32 = static_cast<int>(R);
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        if (offsets == nullptr) {
            // (more than one group: groups that each hold all R rows)
            for (int g = lane; g <= G; g += 64) {
                w.off[g] = g * R32;
                w.pre[g] = g * ((R32 + bm - 1) / bm);
            }
        } else {
            // lane i holds entries per*i .. per*i + per-1 of the G + 1 offsets
            const int per = (G + 1 + 63) / 64;  // at most 5
            int v[5], run = 0;
            bool bad = false;
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                const int g = lane * per + i;
                v[i] = 0;
                if (i < per && g <= G) {
                    const int raw = offsets[g];
                    v[i] = min(max(raw, 0), R32);
                    bad |= raw != v[i] || v[i] < run;
                    run = max(run, v[i]);
                    v[i] = run;
                }
            }
            int top = run;  // running maximum over the lanes
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int t = __shfl_up(top, o, 64);
                if (lane >= o) top = max(top, t);
            }
            int before = __shfl_up(top, 1, 64);
            if (lane == 0) before = 0;
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                const int g = lane * per + i;
                if (i < per && g <= G) {
                    bad |= v[i] < before;
                    v[i] = max(v[i], before);
                    w.off[g] = v[i];
                }
            }
            if (bad) set_error(hdr, 1u);
            // (one wave: its LDS accesses complete in order)
            __builtin_amdgcn_wave_barrier();
            int sum = 0, t[5];
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                const int g = lane * per + i;
                t[i] = 0;
                if (i < per && g < G) t[i] = (w.off[g + 1] - w.off[g] + bm - 1) / bm;
                sum += t[i];
            }
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int u = __shfl_up(incl, o, 64);
                if (lane >= o) incl += u;
            }
            int acc = incl - sum;
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                const int g = lane * per + i;
                if (i < per && g <= G) w.pre[g] = acc;
                acc += t[i];
            }
        }
    }
    __syncthreads();
}

// the last g with pre[g] <= v (pre[0] = 0 <= v): every lane looks at every
// 64th group
__device__ __forceinline__ int group_of(const GroupWalk& w, int G, int v) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int i = 0; i < G; i += 64) {
        const bool le = i + lane < G && w.pre[min(i + lane, G)] <= v;
        n += __popcll(__ballot(le));
    }
    return __builtin_amdgcn_readfirstlane(n - 1);
}

// ------------------------------------------------------------- epilogue --
// Eight float32 values of one row, stored as the output type; nv (0 .. 8) of
// them exist (bf16: 0 or 8; float32: 0, 4 or 8).
template <typename T>
__device__ __forceinline__ void load8(const uint8_t* p, int64_t at, int nv, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<bf16_t>(const uint8_t* p, int64_t at, int, float (&v)[8]) {
    ActVec<bf16_t>::unpack(load16(p + at * 2), v);
}
template <>
__device__ __forceinline__ void load8<float>(const uint8_t* p, int64_t at, int nv, float (&v)[8]) {
    ActVec<float>::unpack(load16(p + at * 4), v);
    if (nv > 4) {
        ActVec<float>::unpack(load16(p + at * 4 + 16), v + 4);
    } else {
#pragma unroll
        for (int u = 4; u < 8; ++u) v[u] = 0.0f;
    }
}
template <typename T>
__device__ __forceinline__ void store8(uint8_t* p, int64_t at, int nv, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<bf16_t>(uint8_t* p, int64_t at, int, const float (&v)[8]) {
    store16(p + at * 2, ActVec<bf16_t>::pack(v));
}
template <>
__device__ __forceinline__ void store8<float>(uint8_t* p, int64_t at, int nv, const float (&v)[8]) {
    store16(p + at * 4, ActVec<float>::pack(v));
    if (nv > 4) store16(p + at * 4 + 16, ActVec<float>::pack(v + 4));
}

// The 32 columns c0 .. c0+31 of one row of the forward's output, held by two
// lanes (half = 0, 1): half h has columns c0 + 8 h .. +7 in v[0] and c0 + 16 +
// 8 h .. +7 in v[1]. Adds the bias, keeps the pre-activation, applies fn, adds
// the residual and stores. `ok`: the row exists (the same for both lanes; both
// call this, whether it exists or not); cend: the first column not to store.
template <typename T>
__device__ __forceinline__ void linear_epilogue32(const LinearArgs& a, int g, int64_t row, int c0, int half,
                                                  bool ok, float (&v)[2][8], int cend) {
    int nv[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        nv[p] = min(8, max(0, cend - (c0 + 16 * p + 8 * half)));
        if (!ok) nv[p] = 0;
        if (a.bias != nullptr && nv[p] > 0) {
            float b[8];
            load8<float>(reinterpret_cast<const uint8_t*>(a.bias), static_cast<int64_t>(g) * a.N + c0 + 16 * p + 8 * half,
                         nv[p], b);
#pragma unroll
            for (int u = 0; u < 8; ++u) v[p][u] += b[u];
        }
    }
    if (a.zsave != nullptr) {
#pragma unroll
        for (int p = 0; p < 2; ++p)
            if (nv[p] > 0) store8<T>(a.zsave, row * a.N + c0 + 16 * p + 8 * half, nv[p], v[p]);
    }
    if (a.codes != nullptr) {
        uint32_t top = 0u;
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int u = 0; u < 8; ++u) top = max(top, u < nv[p] ? abs_bits(v[p][u]) : 0u);
        top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32, 64)));
        if (ok && c0 < a.n32) {
            const uint32_t scale = rows8_scale(top);
            const float inv = rows8_inverse(scale);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float q[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) q[u] = u < nv[p] ? v[p][u] : 0.0f;  // the padding's codes are 0
                uint2 w;
                w.x = rows8_code4(q[0], q[1], q[2], q[3], inv);
                w.y = rows8_code4(q[4], q[5], q[6], q[7], inv);
                *reinterpret_cast<uint2*>(a.codes + row * a.n32 + c0 + 16 * p + 8 * half) = w;
            }
            if (half == 0) a.scales[row * (a.n32 / kRows8Block) + c0 / kRows8Block] = static_cast<uint8_t>(scale);
        }
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        if (nv[p] == 0) continue;
        const int64_t at = row * a.N + c0 + 16 * p + 8 * half;
        if (a.fn != MOE_FN_NONE) {
#pragma unroll
            for (int u = 0; u < 8; ++u) v[p][u] = lin_fn(a.fn, v[p][u]);
        }
        if (a.residual != nullptr) {
            float r[8];
            load8<T>(a.residual, at, nv[p], r);
#pragma unroll
            for (int u = 0; u < 8; ++u) v[p][u] += r[u];
        }
        store8<T>(a.out, at, nv[p], v[p]);
    }
}

// The same 32 columns of a row of dx (T), dW (T or float32) or of a part's
// sums: stored as they are. `base`: elements before the row.
template <typename T>
__device__ __forceinline__ void plain_epilogue32(uint8_t* out, int64_t base, int N, int c0, int half, bool ok,
                                                 const float (&v)[2][8]) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int c = c0 + 16 * p + 8 * half;
        const int nv = ok ? min(8, max(0, N - c)) : 0;
        if (nv > 0) store8<T>(out, base + c, nv, v[p]);
    }
}

// A 32x32 accumulator block, element 4 q + u of lane (lr, lg) being row lr and
// column 8 q + 4 lg + u, as the two runs of eight columns that the epilogues
// take: a half-wave swap per pair of column groups.
__device__ __forceinline__ void block_runs(const f32x16& acc, float (&v)[2][8]) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[8 * p + u]),
                                                            __float_as_uint(acc[8 * p + 4 + u]), false, false);
            v[p][u] = __uint_as_float(s[0]);
            v[p][4 + u] = __uint_as_float(s[1]);
        }
}

// The store of one 32x32 block of C at rows m0 + lr, columns c0 ..: `row0` is
// the first row of the group (forward, dx), `rows` the rows that exist.
// STAGED: of a kernel that stages its outputs, except for parts' sums and
// float32 weight gradients.
template <typename T, int PASS, bool STAGED>
__device__ __forceinline__ void store_block(const LinearArgs& a, int g, int part, int64_t row0, int rows, int m,
                                            int c0, int half, const f32x16& acc) {
    float v[2][8];
    block_runs(acc, v);
    const bool ok = m < rows;
    const int64_t row = row0 + m;
    if ((STAGED && PASS != kLinDw) || a.part_out != nullptr) {
        const int64_t all = PASS == kLinDw ? static_cast<int64_t>(a.G) * a.M : a.R;
        plain_epilogue32<float>(reinterpret_cast<uint8_t*>(a.part_out), (part * all + row) * a.N, a.N, c0, half, ok, v);
    } else if constexpr (PASS == kLinForward) {
        linear_epilogue32<T>(a, g, row, c0, half, ok, v, a.N);
    } else if constexpr (PASS == kLinDx) {
        plain_epilogue32<T>(a.out, row * a.N, a.N, c0, half, ok, v);
    } else {
        if (STAGED || a.out_f32)
            plain_epilogue32<float>(a.out, row * a.N, a.N, c0, half, ok, v);
        else
            plain_epilogue32<T>(a.out, row * a.N, a.N, c0, half, ok, v);
    }
}

// ------------------------------------------------------------ tile list --
// One output tile: rows m0 .. of the group's `rows` rows of C, the first of
// them row row0 of the output; columns c0 ..; k from k0 to k1 (dW: rows of x
// and dz).
struct LinTile {
    int g, part, m0, c0, rows, k0, k1;
    int64_t row0;
};

// groups by rows, descending (ties by index): dW's tiles go longest first
struct GroupOrder {
    int by_rank[kMaxGroups];
};
__device__ __forceinline__ void order_groups(GroupOrder& o, const GroupWalk& w, int G) {
    for (int g = threadIdx.x; g < G; g += blockDim.x) {
        const int n = w.off[g + 1] - w.off[g];
        int rank = 0;
        for (int q = 0; q < G; ++q) {
            const int nq = w.off[q + 1] - w.off[q];
            rank += (nq > n || (nq == n && q < g)) ? 1 : 0;
        }
        o.by_rank[rank] = g;
    }
    __syncthreads();
}

// Tiles go in supertiles of 4 x 4 within a group (n-blocks of four n-tiles,
// within those m-blocks of four m-tiles): tiles that run at the same time
// share operand panels in their XCD's L2.
__device__ __forceinline__ void lin_supertile(int M, int N, int j, int& m, int& nt) {
    const int nb = j / (4 * M);
    const int w = min(4, N - 4 * nb);
    const int r = j - nb * 4 * M;
    const int mb = r / (4 * w);
    const int hgt = min(4, M - 4 * mb);
    const int rr = r - mb * 4 * w;
    nt = 4 * nb + rr / hgt;
    m = 4 * mb + rr % hgt;
}

// k range of part s of `parts` of k values k_lo .. k_hi: whole slices of SK
template <int SK>
__device__ __forceinline__ void part_range(int k_lo, int k_hi, int s, int parts, int& k0, int& k1) {
    if (parts == 1) {
        k0 = k_lo;
        k1 = k_hi;
        return;
    }
    const int slices = (k_hi - k_lo + SK - 1) / SK;
    const int per = (slices + parts - 1) / parts;
    k0 = min(k_hi, k_lo + SK * per * s);
    k1 = min(k_hi, k0 + SK * per);
}

// The position `i` of the list of work-group `bid` of `nblk` (a multiple of 8,
// bid % 8 the XCD) -> tile, or false past its end. Forward and dx: the list of
// tiles (part by part, group by group) is cut into eight equal runs, one for
// each XCD (work-groups b with b % 8 = x), dealt round-robin to its
// work-groups: every m-tile takes equally long, and an XCD's L2 sees few
// groups' weights. dW: tiles take as long as their group has rows, so groups go
// longest first, and four tiles at a time to each XCD.
template <int PASS, int BM, int BN, int SK>
__device__ __forceinline__ bool lin_tile(const LinearArgs& a, const GroupWalk& w, const GroupOrder& o, int bid, int nblk,
                                         int i, LinTile& t) {
    t = LinTile{0, 0, 0, 0, 0, 0, 0, 0};
    const int xcd = bid & 7, per_xcd = nblk >> 3;
    const int c = (bid >> 3) + i * per_xcd;
    if constexpr (PASS == kLinDw) {
        const int per_group = a.mtiles * a.ntn;
        const int total = a.G * per_group * a.parts;
        // (one at a time where four would leave XCDs with more than others)
        const int L = total % 32 == 0 || total >= 4 * nblk ? ((c >> 2) * 8 + xcd) * 4 + (c & 3) : c * 8 + xcd;
        if (L >= total) return false;
        const int gp = L / per_group;
        const int rank = gp / a.parts;
        t.part = gp - rank * a.parts;
        t.g = __builtin_amdgcn_readfirstlane(o.by_rank[rank]);
        int m, nt;
        lin_supertile(a.mtiles, a.ntn, L - gp * per_group, m, nt);
        t.m0 = m * BM;
        t.c0 = nt * BN;
        t.rows = a.M;
        t.row0 = static_cast<int64_t>(t.g) * a.M;
        part_range<SK>(w.off[t.g], w.off[t.g + 1], t.part, a.parts, t.k0, t.k1);
    } else {
        // (the launch bounds the list to 2^30 tiles)
        const int per_part = __builtin_amdgcn_readfirstlane(w.pre[a.G]) * a.ntn, total = per_part * a.parts;
        const auto eighth = [&](int x) { return (total >> 3) * x + ((total & 7) * x >> 3); };
        const int L = eighth(xcd) + c;
        if (L >= eighth(xcd + 1)) return false;
        t.part = a.parts == 1 ? 0 : L / per_part;
        const int l = L - t.part * per_part;
        t.g = group_of(w, a.G, l / a.ntn);
        int m, nt;
        lin_supertile(w.pre[t.g + 1] - w.pre[t.g], a.ntn, l - w.pre[t.g] * a.ntn, m, nt);
        t.m0 = m * BM;
        t.c0 = nt * BN;
        t.rows = w.off[t.g + 1] - w.off[t.g];
        t.row0 = a.same_rows ? 0 : w.off[t.g];
        part_range<SK>(0, a.K, t.part, a.parts, t.k0, t.k1);
    }
    // (the same for every lane by construction)
    t.g = __builtin_amdgcn_readfirstlane(t.g);
    t.part = __builtin_amdgcn_readfirstlane(t.part);
    t.m0 = __builtin_amdgcn_readfirstlane(t.m0);
    t.c0 = __builtin_amdgcn_readfirstlane(t.c0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    t.k0 = __builtin_amdgcn_readfirstlane(t.k0);
    t.k1 = __builtin_amdgcn_readfirstlane(t.k1);
    t.row0 = static_cast<int64_t>(static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(t.row0)))) |
             (static_cast<int64_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(t.row0 >> 32))) << 32);
    return true;
}

// ------------------------------------------------------ staged epilogue --
// A wave's WM x 64 block of a bf16 output, 32 rows at a time through 4 KB of
// LDS (`stage`, this wave's own): lane (row, half) writes its runs of eight
// columns as 16-byte chunks, at position chunk ^ (row / 2) % 8 of the row, and
// reads back chunk lane % 8 of row lane / 8 + 8 i, so that a store writes 8
// rows x 128 bytes. The wave's LDS accesses complete in order. `bias`: the
// tile's bias in LDS (forward).
__device__ __forceinline__ uint8_t* stage_at(uint8_t* stage, int row, int chunk) {
    return stage + row * 128 + ((chunk ^ ((row >> 1) & 7)) << 4);
}
// the staged 32 x 64 block at rows m .. (below `rows`, counted from row0) and
// columns c .. (below `cols`) of a bf16 array with ld values a row
__device__ __forceinline__ void stage_out(const uint8_t* stage, uint8_t* out, int64_t row0, int rows, int ld, int cols,
                                          int m, int c, int lane) {
    u32x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = load16(stage_at(const_cast<uint8_t*>(stage), 8 * i + (lane >> 3), lane & 7));
    const int col = c + 8 * (lane & 7);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = m + 8 * i + (lane >> 3);
        if (r < rows && col < cols)
            *(__attribute__((address_space(1))) u32x4*)(out + ((row0 + r) * ld + col) * 2) = v[i];
    }
}

template <int PASS, int MB, int NB>
__device__ __forceinline__ void store_tile_staged(const LinearArgs& a, const LinTile& t, int mw, int cw, uint8_t* stage,
                                                  const float* bias, int lane, f32x16 (&acc)[MB][NB]) {
    static_assert(NB == 2, "64 columns a wave");
    static_assert(PASS != kLinDh8, "store_tile_dh8");
    // (the addresses below depend on the lane alone: computed before the tile
    // loop and kept, they took more registers than there are)
    asm volatile("" : "+v"(lane));
    const int lr = lane & 31, half = lane >> 5;
    if constexpr (PASS != kLinForward) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float v[2][8];
                block_runs(acc[mb][nb], v);
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    store16(stage_at(stage, lr, 4 * nb + 2 * p + half), ActVec<bf16_t>::pack(v[p]));
            }
            stage_out(stage, a.out, t.row0, t.rows, a.N, a.N, mw + 32 * mb, cw, lane);
        }
    } else {
        // this lane's columns: cw + 32 nb + 16 p + 8 half .. +7; z of one block
        const auto in = [&](int nb, int p) { return cw + 32 * nb + 16 * p + 8 * half < a.N; };
        auto z_runs = [&](int mb, int nb, float (&v)[2][8]) {
            // (computed anew for each use: kept from one to the next, z of a
            // whole block row cost 32 registers, and the compiler spilled)
            asm volatile("" : "+v"(acc[mb][nb]));
            block_runs(acc[mb][nb], v);
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const f32x4 b = *reinterpret_cast<const f32x4*>(bias + cw - t.c0 + 32 * nb + 16 * p + 8 * half + 4 * q);
#pragma unroll
                    for (int u = 0; u < 4; ++u) v[p][4 * q + u] += b[u];
                }
        };
        // the residual of the next 32 rows is loaded before this one's stores:
        // a load after them would complete after them
        u32x4 res[2][NB][2];
        auto load_residual = [&](int mb, u32x4 (&r)[NB][2]) {
            const int m = mw + 32 * mb + lr;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    r[nb][p] = u32x4{0u, 0u, 0u, 0u};
                    if (m < t.rows && in(nb, p))
                        r[nb][p] = *(const __attribute__((address_space(1))) u32x4*)(
                            a.residual + ((t.row0 + m) * a.N + cw + 32 * nb + 16 * p + 8 * half) * 2);
                }
        };
        if (a.residual != nullptr) load_residual(0, res[0]);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            if (a.residual != nullptr && mb + 1 < MB) load_residual(mb + 1, res[(mb + 1) & 1]);
            const int m = mw + 32 * mb;
            if (a.zsave != nullptr) {
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float v[2][8];
                    z_runs(mb, nb, v);
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        store16(stage_at(stage, lr, 4 * nb + 2 * p + half), ActVec<bf16_t>::pack(v[p]));
                }
                stage_out(stage, a.zsave, t.row0, t.rows, a.N, a.N, m, cw, lane);
            }
            if (a.codes != nullptr) {
                // 64 codes a row, 16 bytes at position chunk ^ (row / 2) % 4
                // (past N the weights and the bias read as zeros, and so z:
                // the padding's codes are 0)
                const int64_t nblk = a.n32 / kRows8Block;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float v[2][8];
                    z_runs(mb, nb, v);
                    uint32_t top = 0u;
#pragma unroll
                    for (int p = 0; p < 2; ++p)
#pragma unroll
                        for (int u = 0; u < 8; ++u) top = max(top, abs_bits(v[p][u]));
                    top = max(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32, 64)));
                    const uint32_t scale = rows8_scale(top);
                    const float inv = rows8_inverse(scale);
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        uint2 w;
                        w.x = rows8_code4(v[p][0], v[p][1], v[p][2], v[p][3], inv);
                        w.y = rows8_code4(v[p][4], v[p][5], v[p][6], v[p][7], inv);
                        *reinterpret_cast<uint2*>(stage + lr * 64 + (((2 * nb + p) ^ ((lr >> 1) & 3)) << 4) + 8 * half) = w;
                    }
                    if (half == 0 && m + lr < t.rows && cw + 32 * nb < a.N)
                        *(__attribute__((address_space(1))) uint8_t*)(
                            a.scales + (t.row0 + m + lr) * nblk + (cw + 32 * nb) / kRows8Block) =
                            static_cast<uint8_t>(scale);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 16 * i + (lane >> 2), c = lane & 3;
                    const u32x4 w = load16(stage + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
                    if (m + r < t.rows && cw + 16 * c < a.n32)
                        *(__attribute__((address_space(1))) u32x4*)(a.codes + (t.row0 + m + r) * a.n32 + cw + 16 * c) = w;
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float v[2][8];
                z_runs(mb, nb, v);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    if (a.fn != MOE_FN_NONE) {
#pragma unroll
                        for (int u = 0; u < 8; ++u) v[p][u] = lin_fn(a.fn, v[p][u]);
                    }
                    if (a.residual != nullptr) {
                        float r[8];
                        ActVec<bf16_t>::unpack(res[mb & 1][nb][p], r);
#pragma unroll
                        for (int u = 0; u < 8; ++u) v[p][u] += r[u];
                    }
                    store16(stage_at(stage, lr, 4 * nb + 2 * p + half), ActVec<bf16_t>::pack(v[p]));
                }
            }
            stage_out(stage, a.out, t.row0, t.rows, a.N, a.N, m, cw, lane);
        }
    }
}

// a staged 32 x 32 block (64 bytes a row, 16-byte chunk c at c ^ (row / 2) % 4)
// out to rows m .. (below `rows`, counted from row0), columns c .. of a bf16
// array with ld values a row
__device__ __forceinline__ uint8_t* stage32_at(uint8_t* stage, int row, int chunk) {
    return stage + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ void stage32_out(uint8_t* stage, uint8_t* out, int64_t row0, int rows, int ld, int m, int c,
                                            int lane) {
    u32x4 v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = load16(stage32_at(stage, 16 * i + (lane >> 2), lane & 3));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = m + 16 * i + (lane >> 2);
        if (r < rows)
            *(__attribute__((address_space(1))) u32x4*)(out + ((row0 + r) * ld + c + 8 * (lane & 3)) * 2) = v[i];
    }
}

// dhid of a wave's WM x 64 block -> da = dhid b s (1 + a (1 - s)) (s =
// sigmoid(a)), db = dhid silu(a) and hid = silu(a) b, from a and b in 8 bits.
// The codes of 32 rows x 64 columns come in 16 bytes a lane (row lane / 4 +
// 16 i, chunk lane % 4), through the staging area to the lanes that hold those
// columns; the next rows' are loaded before the last of this one's stores. The
// outputs go out 32 columns at a time, hid and da side by side in the staging
// area, then db: 64 columns of all three took more registers than there are.
// N % 64 == 0: a wave's columns all exist.
template <int MB, int NB>
__device__ __forceinline__ void store_tile_dh8(const LinearArgs& a, const LinTile& t, int mw, int cw, uint8_t* stage,
                                               int lane, f32x16 (&acc)[MB][NB]) {
    asm volatile("" : "+v"(lane));  // (as above)
    const int lr = lane & 31, half = lane >> 5;
    const int col = (a.same_rows ? t.g * a.N : 0) + cw;
    const int c2 = (a.same_rows ? 2 * t.g * a.N : 0) + cw;
    u32x4 cd[2][2];
    uint32_t sc[NB][2];
    auto load_codes = [&](int mb) {
        const int m = mw + 32 * mb, last = t.rows - 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t at = (t.row0 + min(m + 16 * i + (lane >> 2), last)) * a.ldp + col + 16 * (lane & 3);
            cd[0][i] = *(const __attribute__((address_space(1))) u32x4*)(a.ca + at);
            cd[1][i] = *(const __attribute__((address_space(1))) u32x4*)(a.cb + at);
        }
        const int64_t blk = ((t.row0 + min(m + lr, last)) * a.ldp + col) / kRows8Block;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            sc[nb][0] = *(const __attribute__((address_space(1))) uint8_t*)(a.sa + blk + nb);
            sc[nb][1] = *(const __attribute__((address_space(1))) uint8_t*)(a.sb + blk + nb);
        }
    };
    load_codes(0);
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
        const int m = mw + 32 * mb;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 2; ++i) store16(stage_at(stage, 16 * i + (lane >> 2), 4 * q + (lane & 3)), cd[q][i]);
        uint2 w[NB][2][2];  // this lane's codes: [block][a, b][run]
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    w[nb][q][p] = *reinterpret_cast<const uint2*>(stage_at(stage, lr, 4 * q + 2 * nb + p) + 8 * half);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            __builtin_amdgcn_sched_barrier(0);
            const float sa = rows8_step(sc[nb][0]), sb = rows8_step(sc[nb][1]);
            float dh[2][8];
            block_runs(acc[mb][nb], dh);
            u32x4 vb[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float da[8], db[8], hd[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float av = rows8_value(u < 4 ? w[nb][0][p].x : w[nb][0][p].y, u & 3, sa);
                    const float bv = rows8_value(u < 4 ? w[nb][1][p].x : w[nb][1][p].y, u & 3, sb);
                    const float sg = lin_sigmoid(av), sil = av * sg;
                    da[u] = dh[p][u] * bv * (sg * __builtin_fmaf(av, 1.0f - sg, 1.0f));
                    db[u] = dh[p][u] * sil;
                    hd[u] = sil * bv;
                }
                store16(stage32_at(stage, lr, 2 * p + half), ActVec<bf16_t>::pack(hd));
                store16(stage32_at(stage + 2048, lr, 2 * p + half), ActVec<bf16_t>::pack(da));
                vb[p] = ActVec<bf16_t>::pack(db);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (nb + 1 == NB && mb + 1 < MB) load_codes(mb + 1);
            stage32_out(stage, a.hid, t.row0, t.rows, a.ldp, m, col + 32 * nb, lane);
            stage32_out(stage + 2048, a.out, t.row0, t.rows, 2 * a.ldp, m, c2 + 32 * nb, lane);
#pragma unroll
            for (int p = 0; p < 2; ++p) store16(stage32_at(stage, lr, 2 * p + half), vb[p]);
            stage32_out(stage, a.out, t.row0, t.rows, 2 * a.ldp, m, c2 + a.N + 32 * nb, lane);
        }
    }
}

// ------------------------------------------------------- bias gradient --
// rows that one work-group of the dz kernel sums into one partial. (32768 x
// 1408: 64 us at 32 rows, 72 at 64, 86 at 128, where every work-group starts
// at once and they load and compute in step; 512 x 128: 8 against 15.)
constexpr int kDzRows = 32;

struct DzArgs {
    const int32_t* offsets;
    int64_t R;
    int G, N, fn;
    const uint8_t* dy;       // [R, N] (act)
    const uint8_t* z;        // [R, N] (act) or NULL
    const uint8_t* codes;    // [R, n32] or NULL
    const uint8_t* scales;
    int64_t n32;
    uint8_t* dz;             // [R, N] (act) or NULL
    float* db_part;          // [blocks of 32 rows of a group][N] or NULL
};

struct DbArgs {
    const int32_t* offsets;
    uint32_t* hdr;       // error flag of the workspace
    int64_t R;
    int G, N;
    const float* part;   // [blocks of kDzRows rows of a group][N], or NULL:
    const uint8_t* dy;   //   the sums are taken of dy [R, N] (act) itself
    void* db;            // [G, N]
    int db_f32;
};

// db of group g, columns 64 cb .. +63: SPLIT threads a column, each every
// SPLIT-th partial (or row) in order, then their sums in order. No atomics:
// the same bits every call. By 64 SPLIT threads.
template <typename T, int SPLIT>
__device__ __forceinline__ void linear_db_block(const DbArgs& a, int g, int cb) {
    __shared__ GroupWalk walk;
    __shared__ float sums[SPLIT][64];
    walk_groups(walk, a.offsets, a.R, a.G, kDzRows, g == 0 && cb == 0 ? a.hdr : nullptr);
    const int c = threadIdx.x & 63, col = cb * 64 + c, q = threadIdx.x >> 6;
    float s = 0.0f;
    if (col < a.N) {
        if (a.part != nullptr) {
            const int end = walk.pre[g + 1];
#pragma unroll 8
            for (int t = walk.pre[g] + q; t < end; t += SPLIT) s += a.part[static_cast<int64_t>(t) * a.N + col];
        } else {
            const int end = walk.off[g + 1];
            const T* dy = reinterpret_cast<const T*>(a.dy);
#pragma unroll 8
            for (int r = walk.off[g] + q; r < end; r += SPLIT) {
                const T v = dy[static_cast<int64_t>(r) * a.N + col];
                if constexpr (sizeof(T) == 4) s += v;
                else s += bf16_to_f32(v);
            }
        }
    }
    sums[q][c] = s;
    __syncthreads();
    if (q == 0 && col < a.N) {
        float t = sums[0][c];
#pragma unroll
        for (int i = 1; i < SPLIT; ++i) t += sums[i][c];
        const int64_t at = static_cast<int64_t>(g) * a.N + col;
        if (a.db_f32) static_cast<float*>(a.db)[at] = t;
        else static_cast<bf16_t*>(a.db)[at] = f32_to_bf16(t);
    }
}

}  // namespace moe
