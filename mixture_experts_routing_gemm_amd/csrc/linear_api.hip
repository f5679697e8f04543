// Host side of the linear layer's and the rows8 format's C entry points
// (include/moe.h): argument validation, workspace layout, the choice of tiles
// and the launch sequence. No call here allocates or synchronises.
#include <algorithm>

#include "api_common.h"
#include "linear.h"

namespace moe {

int device_cus();
hipError_t launch_linear_tile(int pass, const LinearArgs& a, int shape, bool f32, hipStream_t st);
hipError_t launch_linear_rows(const LinearArgs& a, int fb, bool f32, hipStream_t st);
hipError_t launch_linear_join(int pass, const LinearArgs& a, bool f32, hipStream_t st);
int64_t linear_db_tiles(int64_t R, int G);
hipError_t launch_linear_dz(const DzArgs& a, bool f32, hipStream_t st);
hipError_t launch_linear_db(const DbArgs& a, bool f32, hipStream_t st);
hipError_t launch_linear_pair(int pass, const LinearArgs& r, const LinearArgs& s, int shape, hipStream_t st);
hipError_t launch_linear_backward(const LinearArgs& x, const LinearArgs& w, const DbArgs& d, bool f32, hipStream_t st);
hipError_t launch_pack_rows8(int64_t rows, int n, bool f32, const void* x, void* packed, hipStream_t st);
hipError_t launch_unpack_rows8(int64_t rows, int n, bool f32, const void* packed, void* x, hipStream_t st);

}  // namespace moe

using namespace moe;

namespace {

int32_t check_linear(const moe_linear_shape* s, bool grouped) {
    if (s == nullptr) return MOE_ERR_INVALID_ARG;
    if (s->rows < 0 || s->n_in <= 0 || s->n_out <= 0 || s->groups <= 0 || s->fn < MOE_FN_NONE || s->fn > MOE_FN_SILU ||
        s->save < MOE_SAVE_NONE || s->save > MOE_SAVE_INT8 || (!grouped && s->groups != 1))
        return MOE_ERR_INVALID_ARG;
    if (s->act != MOE_F32 && s->act != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    if (s->grad != MOE_F32 && s->grad != s->act) return MOE_ERR_UNSUPPORTED;
    const int unit = s->act == MOE_F32 ? 4 : 8;
    // (row counts are rounded up to tiles and parts in 32 bits)
    if (s->rows > (int64_t(1) << 31) - 4096 || s->n_in > (1 << 20) || s->n_out > (1 << 20) || s->n_in % unit != 0 ||
        s->n_out % unit != 0 || s->groups > kMaxGroups)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

size_t act_size(const moe_linear_shape& s) { return s.act == MOE_F32 ? 4 : 2; }

size_t saved_size(const moe_linear_shape& s) {
    if (s.save == MOE_SAVE_ACT) return align256(static_cast<size_t>(s.rows) * s.n_out * act_size(s));
    if (s.save == MOE_SAVE_INT8) return rows8_bytes(s.rows, s.n_out);
    return 0;
}

// How a product is run: its tile shape and in how many parts k is split.
struct Plan {
    int shape, parts;
    float us;  // its estimate
};

// The microseconds that a compute unit takes for one slice of k (64 bytes) of
// one tile: `full` with every unit at work on as many tiles as it holds, `one`
// for a tile that has a unit to itself in a round that is not full. Measured
// at 4096 values of k on an MI355X (forward, dx and dW alike):
// bf16 256 x 256 tiles reach 1.13 PFLOP/s, 256 x 128 0.94, 128 x 128 0.82 and
// 64 x 128 0.63, float32 128 x 128 132 TFLOP/s, 64 x 64 119 and 64 x 32 109;
// smaller tiles win where the larger ones leave units idle (512 x 512 values
// of 4096 products in float32: 64 x 64 tiles 77 us, 64 x 32 51).
// `epilogue`: what an activation and saved pre-activations each add to a tile
// (two work-groups on a unit hide half of it in each other's products).
struct TileCost {
    int shape, bm, bn;
    float full, one, epilogue;
};
constexpr TileCost kBf16Tiles[] = {{kLinTileBig, 256, 256, 0.96f, 0.64f, 8.0f},
                                   {kLinTileHalf, 256, 128, 0.57f, 0.52f, 3.0f},
                                   {kLinTileMid, 128, 128, 0.345f, 0.33f, 1.5f},
                                   {kLinTileSmall, 64, 128, 0.215f, 0.24f, 0.8f}};
constexpr TileCost kF32Tiles[] = {{kLinTileMid, 128, 128, 1.01f, 1.0f, 1.0f},
                                  {kLinTileTiny, 64, 64, 0.283f, 0.29f, 0.5f},
                                  {kLinTileSlim, 64, 32, 0.157f, 0.19f, 0.3f}};

// The cheapest tile shape and number of parts by those costs: whole rounds of
// the units, the last one in between, and for parts the join: about 7 us, and
// its float32 sums written and read at 4 TB/s (dW of 128 x 128 weights over
// 30000 rows: 45 us in 8 parts, 29 in 16, 24 in 32 and in 64). The rows of a group are not
// known here: half a tile of each group is taken to be empty.
// smallest: the last tile shape to consider, with k whole (0: any, and parts)
Plan plan_of(const moe_linear_shape& s, int pass, int smallest = 0) {
    const bool f32 = s.act == MOE_F32;
    const TileCost* const first = f32 ? kF32Tiles : kBf16Tiles;
    const TileCost* const last = first + (f32 || pass == kLinDw ? 3 : 4);
    const int64_t units = device_cus(), sk = f32 ? 16 : 32;
    const int64_t n = pass == kLinForward ? s.n_out : s.n_in;
    const int64_t groups = std::min<int64_t>(s.groups, std::max<int64_t>(1, s.rows));
    const int64_t k = pass == kLinForward ? s.n_in : pass == kLinDx ? s.n_out : s.rows / groups;
    const int64_t slices = std::max<int64_t>(1, (k + sk - 1) / sk);
    const float values = static_cast<float>(pass == kLinDw ? static_cast<int64_t>(s.groups) * s.n_out : s.rows) * n;
    const float extras = pass != kLinForward ? 0.0f
                                             : static_cast<float>((s.fn != MOE_FN_NONE) + (s.save != MOE_SAVE_NONE));
    Plan best{first->shape, 1, -1.0f};
    for (const TileCost* c = first; c != last && (smallest == 0 || c->shape <= smallest); ++c) {
        const int64_t mt = pass == kLinDw ? groups * ((s.n_out + c->bm - 1) / c->bm)
                                          : s.groups == 1 ? (s.rows + c->bm - 1) / c->bm : s.rows / c->bm + (groups + 1) / 2;
        const int64_t tiles = mt * ((n + c->bn - 1) / c->bn);
        // 1, 2, 3, 4, 6, 8, 12 .. 64 parts
        for (int parts = 1; parts <= (smallest == 0 ? 64 : 1) && parts * 4 <= slices + 3;
             parts = parts < 4 ? parts + 1 : (parts & (parts - 1)) == 0 ? parts + parts / 2 : parts / 3 * 4) {
            if (parts > 1 && tiles * parts > 4 * units) break;
            const int64_t all = tiles * parts, rounds = all / units;
            const float rest = static_cast<float>(all - rounds * units) / units;
            const float round =
                std::max(c->one, rounds * c->full + (rest > 0.0f ? c->one + (c->full - c->one) * rest : 0.0f));
            float us = static_cast<float>((slices + parts - 1) / parts) * round;
            us += extras * c->epilogue * (parts > 1 ? 0 : rounds + (rest > 0.0f ? 1 : 0));
            if (parts > 1) us += 7.0f + values * parts * (8.0f / 4e6f);
            if (best.us < 0.0f || us < best.us) best = Plan{c->shape, parts, us};
        }
    }
    return best;
}

// The forward by the kernel for few rows: where the 64 x 128 tiles of all
// groups would leave units idle, that kernel's narrower columns keep them
// reading (one row, 4096 -> 4096: 9 us, the tiles in four parts 20; 8 groups of
// 4 rows, 2048 -> 1408: 16 against 19, of 16 rows 20 against 19).
bool few_rows(const moe_linear_shape& s) {
    const int64_t groups = std::min<int64_t>(s.groups, s.rows);
    return s.rows <= s.groups * int64_t(s.groups == 1 ? 32 : 8) &&
           groups * ((s.n_out + 127) / 128) < device_cus();
}

// The tile shape of the SwiGLU experts' backward products over the routed rows
// (n columns, k values), which take whole k and stage their outputs: the
// three largest shapes.
int pair_shape(const moe_shape& s, int n, int k) {
    const moe_linear_shape l{s.T * s.k, n, k, s.E, MOE_BF16, MOE_FN_NONE, MOE_SAVE_NONE, MOE_BF16};
    return plan_of(l, kLinDx, kLinTileMid).shape;
}

// dx, dW and db in one launch, on 128 x 128 (float32: 64 x 32) tiles, k not
// split: where the longer of the two products, or both together spread over
// the units, take less than one after the other by their own plans and the 6
// us that a launch takes to begin and end. Replayed from a graph: 512 rows of
// 64 -> 128, eight groups, in float32 6 us against 14 apart; in bf16 300 rows
// of 512 -> 512 11 against 22, 2048 rows of 1024 -> 2048 36 against 60; 8000
// rows of 256 -> 256, whose dW needs its parts, 83 against 37.
bool backward_together(const moe_linear_shape& s, const Plan& dx, const Plan& dw) {
    const bool f32 = s.act == MOE_F32;
    const TileCost& c = f32 ? kF32Tiles[2] : kBf16Tiles[2];
    const int64_t sk = f32 ? 16 : 32, groups = std::min<int64_t>(s.groups, std::max<int64_t>(1, s.rows));
    const int64_t nt = (s.n_in + c.bn - 1) / c.bn;
    const float sx = static_cast<float>((s.n_out + sk - 1) / sk), sw = static_cast<float>((s.rows / groups + sk - 1) / sk);
    const float tx = static_cast<float>((s.rows / c.bm + groups) * nt);
    const float tw = static_cast<float>(s.groups) * ((s.n_out + c.bm - 1) / c.bm) * nt;
    const float both = std::max(std::max(sx, sw) * c.one, (tx * sx + tw * sw) * c.full / device_cus());
    return both < dx.us + dw.us + 6.0f;
}

struct LinLayout {
    size_t dz = 0, db = 0, part = 0, total = 0;
    Plan fwd{0, 1, 0.0f}, dx{0, 1, 0.0f}, dw{0, 1, 0.0f};
    bool together = false;  // dx, dW and db in one launch
};
LinLayout linear_layout(const moe_linear_shape& s, bool backward) {
    LinLayout L;
    size_t off = kHeaderBytes;
    auto take = [&](size_t n) {
        const size_t at = off;
        off = align256(off + n);
        return at;
    };
    auto parts = [](const Plan& p, size_t rows, size_t n) { return p.parts > 1 ? p.parts * rows * n * 4 : 0; };
    const size_t R = static_cast<size_t>(s.rows), ni = s.n_in, no = s.n_out;
    if (backward) {
        L.dx = plan_of(s, kLinDx);
        L.dw = plan_of(s, kLinDw);
        L.together = backward_together(s, L.dx, L.dw);
        L.dz = take(s.fn != MOE_FN_NONE ? R * no * act_size(s) : 0);
        L.db = take(static_cast<size_t>(linear_db_tiles(s.rows, s.groups)) * no * 4);
        // (a caller may ask for one of the two alone: room for its own plan)
        L.part = take(std::max(parts(L.dx, R, ni), parts(L.dw, s.groups * no, ni)));
    } else {
        L.fwd = plan_of(s, kLinForward);
        L.part = take(parts(L.fwd, R, no));
    }
    L.total = off;
    return L;
}

int32_t check_linear_ws(size_t need, const void* ws, size_t ws_bytes) {
    if (ws == nullptr || !aligned256(ws) || ws_bytes < need) return MOE_ERR_WORKSPACE;
    return MOE_OK;
}

int32_t check_saved(const moe_linear_shape& s, const void* saved, size_t saved_bytes) {
    if (s.save == MOE_SAVE_NONE) return MOE_OK;
    if (saved == nullptr || !aligned256(saved) || saved_bytes < saved_size(s)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

hipError_t run_product(const Plan& p, int pass, LinearArgs a, bool f32, void* ws, size_t part_at, hipStream_t st) {
    a.parts = p.parts;
    a.part_out = p.parts > 1 ? at<float>(ws, part_at) : nullptr;
    const hipError_t e = launch_linear_tile(pass, a, p.shape, f32, st);
    if (e != hipSuccess || p.parts == 1) return e;
    return launch_linear_join(pass, a, f32, st);
}

int32_t linear_forward(const moe_linear_shape* s, const void* x, const int32_t* offsets, bool grouped, const void* w,
                       const float* bias, const void* residual, void* y, void* saved, size_t saved_bytes, void* ws,
                       size_t ws_bytes, void* stream) {
    MOE_TRY(check_linear(s, grouped));
    if (s->rows == 0) return MOE_OK;
    MOE_TRY(check_ptrs({x, w, y}));
    if (grouped) MOE_TRY(check_ptrs({offsets}));
    MOE_TRY(check_opt({bias, residual}));
    MOE_TRY(check_saved(*s, saved, saved_bytes));
    const LinLayout L = linear_layout(*s, false);
    MOE_TRY(check_linear_ws(L.total, ws, ws_bytes));
    LinearArgs a{};
    a.a = static_cast<const uint8_t*>(x);
    a.b = static_cast<const uint8_t*>(w);
    a.offsets = offsets;
    a.hdr = static_cast<uint32_t*>(ws);
    a.R = s->rows;
    a.G = s->groups;
    a.N = s->n_out;
    a.K = s->n_in;
    a.fn = s->fn;
    a.bias = bias;
    a.residual = static_cast<const uint8_t*>(residual);
    a.out = static_cast<uint8_t*>(y);
    if (s->save == MOE_SAVE_ACT) {
        a.zsave = static_cast<uint8_t*>(saved);
    } else if (s->save == MOE_SAVE_INT8) {
        a.codes = static_cast<uint8_t*>(saved);
        a.scales = a.codes + rows8_scales_at(s->rows, s->n_out);
        a.n32 = rows8_stride(s->n_out);
    }
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (few_rows(*s)) {
        // 16 columns a work-group where 32 would leave compute units idle
        // (8-bit codes need 32: a block)
        a.parts = 1;
        const int64_t blocks = std::min<int64_t>(s->groups, s->rows) * ((s->n_out + 31) / 32);
        return hip_status(launch_linear_rows(a, s->save != MOE_SAVE_INT8 && blocks < device_cus() ? 1 : 2,
                                             s->act == MOE_F32, st));
    }
    return hip_status(run_product(L.fwd, kLinForward, a, s->act == MOE_F32, ws, L.part, st));
}

int32_t linear_backward(const moe_linear_shape* s, const void* x, const int32_t* offsets, bool grouped, const void* w,
                        const void* saved, size_t saved_bytes, const void* dy, void* dx, void* dw, void* db, void* ws,
                        size_t ws_bytes, void* stream) {
    MOE_TRY(check_linear(s, grouped));
    if (s->fn != MOE_FN_NONE && s->save == MOE_SAVE_NONE) return MOE_ERR_INVALID_ARG;
    MOE_TRY(check_opt({x, w, dy, dx, dw, db, offsets}));
    if (s->rows > 0) {
        MOE_TRY(check_ptrs({dy}));
        if (dx != nullptr) MOE_TRY(check_ptrs({w}));
        if (dw != nullptr) MOE_TRY(check_ptrs({x}));
        if (grouped) MOE_TRY(check_ptrs({offsets}));
        if (s->fn != MOE_FN_NONE) MOE_TRY(check_saved(*s, saved, saved_bytes));
    }
    const LinLayout L = linear_layout(*s, true);
    MOE_TRY(check_linear_ws(L.total, ws, ws_bytes));
    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool f32 = s->act == MOE_F32;
    // (without rows the offsets are not read: every group is empty)
    const int32_t* off = offsets;
    const uint8_t* dz = static_cast<const uint8_t*>(dy);
    // without an activation dz is dy, and where that is short db sums it itself
    const bool direct = s->fn == MOE_FN_NONE && s->rows <= 2048;
    if (s->rows > 0 && (s->fn != MOE_FN_NONE || (db != nullptr && !direct))) {
        DzArgs d{};
        d.offsets = off;
        d.R = s->rows;
        d.G = s->groups;
        d.N = s->n_out;
        d.fn = s->fn;
        d.dy = static_cast<const uint8_t*>(dy);
        if (s->fn != MOE_FN_NONE) {
            if (s->save == MOE_SAVE_ACT) {
                d.z = static_cast<const uint8_t*>(saved);
            } else {
                d.codes = static_cast<const uint8_t*>(saved);
                d.scales = d.codes + rows8_scales_at(s->rows, s->n_out);
                d.n32 = rows8_stride(s->n_out);
            }
            d.dz = at<uint8_t>(ws, L.dz);
            dz = d.dz;
        }
        d.db_part = db != nullptr ? at<float>(ws, L.db) : nullptr;
        MOE_TRY(hip_status(launch_linear_dz(d, f32, st)));
    }
    LinearArgs x_args{}, w_args{};
    x_args.a = w_args.a = dz;
    x_args.offsets = w_args.offsets = off;
    x_args.hdr = w_args.hdr = static_cast<uint32_t*>(ws);
    x_args.R = w_args.R = s->rows;
    x_args.G = w_args.G = s->groups;
    x_args.N = w_args.N = s->n_in;
    x_args.parts = w_args.parts = 1;
    if (s->rows > 0 && dx != nullptr) {
        x_args.b = static_cast<const uint8_t*>(w);
        x_args.K = s->n_out;
        x_args.out = static_cast<uint8_t*>(dx);
    }
    if (dw != nullptr) {
        w_args.b = static_cast<const uint8_t*>(x);
        w_args.M = s->n_out;
        w_args.out = static_cast<uint8_t*>(dw);
        w_args.out_f32 = s->grad == MOE_F32 ? 1 : 0;
    }
    DbArgs b_args{};
    b_args.offsets = off;
    b_args.hdr = static_cast<uint32_t*>(ws);
    b_args.R = s->rows;
    b_args.G = s->groups;
    b_args.N = s->n_out;
    b_args.part = direct ? nullptr : at<float>(ws, L.db);
    b_args.dy = static_cast<const uint8_t*>(dy);
    b_args.db = db;
    b_args.db_f32 = s->grad == MOE_F32 ? 1 : 0;
    if (L.together) return hip_status(launch_linear_backward(x_args, w_args, b_args, f32, st));
    if (x_args.out != nullptr) MOE_TRY(hip_status(run_product(L.dx, kLinDx, x_args, f32, ws, L.part, st)));
    if (w_args.out != nullptr) MOE_TRY(hip_status(run_product(L.dw, kLinDw, w_args, f32, ws, L.part, st)));
    if (db != nullptr) MOE_TRY(hip_status(launch_linear_db(b_args, f32, st)));
    return MOE_OK;
}

int32_t check_rows8(int64_t rows, int32_t n, int32_t dtype, const void* x, const void* packed, size_t bytes) {
    if (rows < 0 || n < 1) return MOE_ERR_INVALID_ARG;
    if (n > (1 << 20) || rows >= (int64_t(1) << 40)) return MOE_ERR_UNSUPPORTED;
    if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
    if (rows == 0) return MOE_OK;
    MOE_TRY(check_ptrs({x, packed}));
    if (!aligned256(packed) || bytes < rows8_bytes(rows, n)) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

}  // namespace

namespace moe {

// dhid = dy W2 and the SwiGLU backward of every routed row and shared-expert
// block, from a and b in 8 bits (saved8): [da | db] rows and hid rows
hipError_t launch_ffn_dh8(const moe_shape& s, const int32_t* offsets, const void* w2, const void* dy_perm,
                          const void* dy_sh, const void* saved8, void* h_r, void* h_s, void* dd_r, void* dd_s,
                          hipStream_t st) {
    const Saved8Layout L = saved8_layout(s);
    const uint8_t* sv = static_cast<const uint8_t*>(saved8);
    const int64_t wgroup = static_cast<int64_t>(s.d) * s.h * 2;
    LinearArgs r{}, q{};
    r.a = static_cast<const uint8_t*>(dy_perm);
    r.b = static_cast<const uint8_t*>(w2);
    r.offsets = offsets;
    r.R = s.T * s.k;
    r.G = s.E;
    r.N = s.h;
    r.K = s.d;
    r.parts = 1;
    r.out = static_cast<uint8_t*>(dd_r);
    r.ca = sv + L.a_r;
    r.cb = sv + L.b_r;
    r.sa = r.ca + L.scales_r;
    r.sb = r.cb + L.scales_r;
    r.hid = static_cast<uint8_t*>(h_r);
    r.ldp = s.h;
    if (s.S > 0) {
        q = r;
        q.a = static_cast<const uint8_t*>(dy_sh);
        q.b = r.b + s.E * wgroup;
        q.offsets = nullptr;
        q.same_rows = 1;
        q.R = s.T;
        q.G = s.S;
        q.out = static_cast<uint8_t*>(dd_s);
        q.ca = sv + L.a_s;
        q.cb = sv + L.b_s;
        q.sa = q.ca + L.scales_s;
        q.sb = q.cb + L.scales_s;
        q.hid = static_cast<uint8_t*>(h_s);
        q.ldp = s.S * s.h;
    }
    return launch_linear_pair(kLinDh8, r, q, pair_shape(s, s.h, s.d), st);
}

// dv = [da | db] [W1; W3] of every routed row; the shared experts' blocks side
// by side along k, so that their sum is the product's own
hipError_t launch_ffn_dx2(const moe_shape& s, const int32_t* offsets, const void* w1, const void* w3, const void* dd_r,
                          const void* dd_s, void* dx_perm, void* dx_sh, hipStream_t st) {
    const int64_t wgroup = static_cast<int64_t>(s.d) * s.h * 2;
    LinearArgs r{}, q{};
    r.a = static_cast<const uint8_t*>(dd_r);
    r.b = static_cast<const uint8_t*>(w1);
    r.b2 = static_cast<const uint8_t*>(w3);
    r.seg = s.h;
    r.offsets = offsets;
    r.R = s.T * s.k;
    r.G = s.E;
    r.N = s.d;
    r.K = 2 * s.h;
    r.parts = 1;
    r.out = static_cast<uint8_t*>(dx_perm);
    if (s.S > 0) {
        q = r;
        q.a = static_cast<const uint8_t*>(dd_s);
        q.b = r.b + s.E * wgroup;
        q.b2 = r.b2 + s.E * wgroup;
        q.offsets = nullptr;
        q.R = s.T;
        q.G = 1;
        q.K = 2 * s.S * s.h;
        q.out = static_cast<uint8_t*>(dx_sh);
    }
    return launch_linear_pair(kLinDx2, r, q, pair_shape(s, s.d, 2 * s.h), st);
}

}  // namespace moe

extern "C" {

size_t moe_linear_workspace_bytes(const moe_linear_shape* s, int32_t stage) {
    if (check_linear(s, true) != MOE_OK) return 0;
    if (stage != MOE_STAGE_LINEAR && stage != MOE_STAGE_LINEAR_BACKWARD) return 0;
    return linear_layout(*s, stage == MOE_STAGE_LINEAR_BACKWARD).total;
}

size_t moe_linear_saved_bytes(const moe_linear_shape* s) {
    return check_linear(s, true) == MOE_OK ? saved_size(*s) : 0;
}

int32_t moe_grouped_linear(const moe_linear_shape* s, const void* x, const int32_t* offsets, const void* w,
                           const float* bias, const void* residual, void* y, void* saved, size_t saved_bytes, void* ws,
                           size_t ws_bytes, void* stream) {
    return linear_forward(s, x, offsets, true, w, bias, residual, y, saved, saved_bytes, ws, ws_bytes, stream);
}

int32_t moe_linear(const moe_linear_shape* s, const void* x, const void* w, const float* bias, const void* residual,
                   void* y, void* saved, size_t saved_bytes, void* ws, size_t ws_bytes, void* stream) {
    return linear_forward(s, x, nullptr, false, w, bias, residual, y, saved, saved_bytes, ws, ws_bytes, stream);
}

int32_t moe_grouped_linear_backward(const moe_linear_shape* s, const void* x, const int32_t* offsets, const void* w,
                                    const void* saved, size_t saved_bytes, const void* dy, void* dx, void* dw, void* db,
                                    void* ws, size_t ws_bytes, void* stream) {
    return linear_backward(s, x, offsets, true, w, saved, saved_bytes, dy, dx, dw, db, ws, ws_bytes, stream);
}

int32_t moe_linear_backward(const moe_linear_shape* s, const void* x, const void* w, const void* saved,
                            size_t saved_bytes, const void* dy, void* dx, void* dw, void* db, void* ws, size_t ws_bytes,
                            void* stream) {
    return linear_backward(s, x, nullptr, false, w, saved, saved_bytes, dy, dx, dw, db, ws, ws_bytes, stream);
}

size_t moe_rows8_bytes(int64_t rows, int32_t n) {
    if (rows < 0 || rows >= (int64_t(1) << 40) || n < 1 || n > (1 << 20)) return 0;
    return rows8_bytes(rows, n);
}

int32_t moe_pack_rows8(int64_t rows, int32_t n, int32_t dtype, const void* x, void* packed, size_t packed_bytes,
                       void* stream) {
    MOE_TRY(check_rows8(rows, n, dtype, x, packed, packed_bytes));
    if (rows == 0) return MOE_OK;
    return hip_status(launch_pack_rows8(rows, n, dtype == MOE_F32, x, packed, static_cast<hipStream_t>(stream)));
}

int32_t moe_unpack_rows8(int64_t rows, int32_t n, int32_t dtype, const void* packed, size_t packed_bytes, void* x,
                         void* stream) {
    MOE_TRY(check_rows8(rows, n, dtype, x, packed, packed_bytes));
    if (rows == 0) return MOE_OK;
    return hip_status(launch_unpack_rows8(rows, n, dtype == MOE_F32, packed, x, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
