// Internal launch interface between the C-ABI layer (zr_abi.cpp,
// zr_sched.cpp) and the HIP kernels. Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zr.h"

namespace zr {

constexpr int kMaxRanks = ZR_MAX_RANKS;
constexpr int kAgSegsPerLaunch = 32;   // segments carried in one all-gather launch
constexpr int kFlatPtrsPerLaunch = 256;    // source pointers of fragments in one flatten launch
constexpr int kFlatEntriesPerLaunch = 32;  // fragments in one flatten launch
constexpr int kRsfPtrsPerLaunch = 256;   // rank pointers of fragments in one discrete-RS launch
constexpr int kRsfEntriesPerLaunch = 32; // fragments in one discrete-RS launch
constexpr int kRsfSegsPerLaunch = 96;    // (fragment, chunk) segments in one discrete-RS launch

// Rank pointer tables travel by value in kernel arguments (K <= 64 -> 512 B).
struct ConstPtrs {
    const void* p[kMaxRanks];
};
struct MutPtrs {
    void* p[kMaxRanks];
};

// One fragment of a flatten or a discrete reduce-scatter: its K rank
// pointers (all null for the zero padding after the last fragment), its
// offset in the (virtual) bucket, and its size.
struct FragEntry {
    const void* ptr[kMaxRanks];
    int64_t off, n;
};

// Knobs read once from the environment (for tuning sweeps and tests);
// defaults are the measured best.
// Debugging aids among them: ZR_FORCE_PATH overrides the kernels' choice of
// access path or tile shape where they have one, and ZR_DEBUG makes every call
// wait for its stream after its launches (outside stream capture), so a fault
// in a kernel is reported by the call that launched it.
enum ForcePath {
    kPathAuto = 0,     // each kernel's own choice
    kPathElement = 1,  // element-wise folds and copies (reduce-scatter, discrete
                       // reduce-scatter, all-reduce, all-gather)
    kPathSmall = 2,    // one-slice tiles for every ring-order reduce-scatter
    kPathLarge = 3,    // full tiles for every reduce-scatter, however small
};
struct Tuning {
    int ar_nontemporal;    // fused all-reduce: streaming (non-temporal) loads and stores
    int ag_nontemporal;    // all-gather
    int max_grid;          // blocks per launch at most (ZR_MAX_GRID, default 2^30): every
                           // kernel launches one block per tile up to it, and its blocks
                           // stride over the tiles beyond it
    int force_path;        // ZR_FORCE_PATH: element | small | large (a ForcePath)
    int rs_pairs;          // ZR_RS_PAIRS: reduce-scatter tiles by pairs of chunks (1) or chunk by chunk (0)
    int debug;             // ZR_DEBUG: 1 = wait for the stream after each call's launches
};
const Tuning& tuning();
// Blocks of `threads` threads for a launch of `tiles` tiles: one per tile, at
// most tuning().max_grid, and fewer than 2^32 threads in all (HIP refuses more).
inline int grid_for(int64_t tiles, int threads = 256) {
    const int64_t most = (((int64_t)1 << 32) - 1) / threads;
    const int64_t cap = tuning().max_grid < most ? tuning().max_grid : most;
    return (int)(tiles < cap ? tiles : cap);
}
int device_cu_count();  // CUs of the current device (cached per device)

// flags: ZR_AVERAGE | ZR_ACCUMULATE
hipError_t launch_reduce_scatter(int K, const ConstPtrs& in, zr_dtype in_dt, int64_t N,
                                 const MutPtrs& out, zr_dtype out_dt, int shift, int flags,
                                 zr_order order, hipStream_t stream);

// A reduce-scatter prepared once (launch geometry and kernel chosen) and
// launched many times. rs_plan_build returns NULL when host memory runs out.
struct RsPlan;
RsPlan* rs_plan_build(int K, const ConstPtrs& in, zr_dtype in_dt, int64_t N, const MutPtrs& out,
                      zr_dtype out_dt, int shift, int flags, zr_order order);
hipError_t rs_plan_launch(const RsPlan* plan, hipStream_t stream);
void rs_plan_free(RsPlan* plan);

hipError_t launch_allreduce_fused(int K, const ConstPtrs& in, const MutPtrs& out, zr_dtype dt,
                                  int64_t N, int average, zr_order order, hipStream_t stream);

// segs: up to kAgSegsPerLaunch segments per call.
hipError_t launch_all_gather(int K, const ConstPtrs& shards, const MutPtrs& fulls, zr_dtype dt,
                             const zr_seg* segs, int n_segs, int shift, hipStream_t stream);
// Any number of segments in one launch, their table staged to `ws` (at least
// ag_table_bytes(n_segs) bytes) on `stream` first.
hipError_t launch_all_gather_ws(int K, const ConstPtrs& shards, const MutPtrs& fulls, zr_dtype dt,
                                const zr_seg* segs, int n_segs, int shift, void* ws,
                                hipStream_t stream);

// Device descriptor tables. A call whose fragment (or segment) table does not
// fit one kernel-argument block either goes out as several argument launches
// or, given a workspace, as one launch that reads the whole table from it.
// The host builds the table as a byte image whose internal pointers already
// hold the workspace's device addresses; staging copies the image there.
// Every table is laid out in 8-byte words (sizes below in bytes).
constexpr size_t kWsAlign = 256;

// Discrete reduce-scatter: first tiles int64[nseg + 1], segment records
// int32[3 * nseg] (entry, chunk, head), entry records int64[2 * nent]
// (offset, size), rank pointers [K * nent].
struct RsfLayout {
    size_t tile0, seg, ent, ptr, bytes;
    RsfLayout(int K, int64_t nent, int64_t nseg) {
        tile0 = 0;
        seg = tile0 + 8 * (size_t)(nseg + 1);
        ent = seg + ((12 * (size_t)nseg + 7) & ~(size_t)7);
        ptr = ent + 16 * (size_t)nent;
        bytes = ptr + 8 * (size_t)K * (size_t)nent;
    }
};
// Flatten: first tiles int64[nent + 1], tiles per rank int64[nent], entry
// records int64[2 * nent] (offset, size), source pointers [K * nent].
struct FlatLayout {
    size_t tile0, tpr, ent, src, bytes;
    FlatLayout(int K, int64_t nent) {
        tile0 = 0;
        tpr = tile0 + 8 * (size_t)(nent + 1);
        ent = tpr + 8 * (size_t)nent;
        src = ent + 16 * (size_t)nent;
        bytes = src + 8 * (size_t)K * (size_t)nent;
    }
};
// All-gather: first tiles int64[nseg + 1], then kAgSegBytes per segment record.
constexpr size_t kAgSegBytes = 48;
inline size_t rsf_table_bytes(int K, int64_t n_entries, int64_t n_segs) {
    return RsfLayout(K, n_entries, n_segs).bytes;
}
inline size_t flatten_table_bytes(int K, int64_t n_entries) { return FlatLayout(K, n_entries).bytes; }
inline size_t ag_table_bytes(int64_t n_segs) { return 8 * (size_t)(n_segs + 1) + kAgSegBytes * (size_t)n_segs; }
// Copies a table image to the workspace: asynchronously on `stream`, or with a
// blocking copy when `stream_order` is false (plan creation).
hipError_t stage_table(void* ws, const void* image, size_t bytes, hipStream_t stream, bool stream_order);

// Discrete reduce-scatter over fragment entries (any count): a plan holds the
// launches' argument blocks, built once and launched many times. With `ws`
// non-null and more than one argument launch needed, the plan instead holds
// one launch whose table image (table_bytes, host copy in table_image) is to
// be staged to `ws` before the launch. rsf_plan_build returns NULL when host
// memory runs out.
struct RsfPlan;
RsfPlan* rsf_plan_build(int K, const FragEntry* entries, int n_entries, int64_t N, zr_dtype in_dt,
                        const MutPtrs& out, zr_dtype out_dt, int shift, int flags, zr_order order,
                        void* ws);
size_t rsf_plan_table_bytes(const RsfPlan* plan);   // 0: argument launches only
const void* rsf_plan_table_image(const RsfPlan* plan);
int rsf_plan_launch_count(const RsfPlan* plan);
hipError_t rsf_plan_launch(const RsfPlan* plan, hipStream_t stream);
void rsf_plan_free(RsfPlan* plan);

// Device address, on the current device, of the file-scope staging array of
// ZR_NOALLOC_TABLE_BYTES bytes that zr_reduce_scatter_frags_noalloc stages its
// table in (looked up once per device with hipGetSymbolAddress).
constexpr int kMaxDevices = 64;
hipError_t noalloc_scratch(void** ptr);

// Bucket flatten over fragment entries, planned the same way: argument
// launches of kFlatEntriesPerLaunch (or fewer) entries, an entry of more than
// 2^28 / K tiles of 4 KiB per rank cut into pieces of that many (so tile
// numbers fit 32 bits), or, with `ws`, one launch over a staged table of the
// uncut entries.
struct FlatPlan;
FlatPlan* flat_plan_build(int K, const FragEntry* entries, int n_entries, const MutPtrs& buckets,
                          int elem_bytes, void* ws);
size_t flat_plan_table_bytes(const FlatPlan* plan);
const void* flat_plan_table_image(const FlatPlan* plan);
int flat_plan_launch_count(const FlatPlan* plan);
hipError_t flat_plan_launch(const FlatPlan* plan, hipStream_t stream);
void flat_plan_free(FlatPlan* plan);

// Layer norm and 8-bit checkpoints. The launches are declared weak so that a
// build of the C-ABI layer alone (argument validation, no kernels) links; its
// calls then report that the kernels are missing.
#define ZR_KERNELS __attribute__((weak))

struct NormFwd {
    const void *x, *weight, *bias;
    zr_dtype x_dt, param_dt, y_dt, ckpt_format;
    int64_t rows, cols, ld_x, ld_y;
    float eps;
    void *y, *ckpt_x, *ckpt_y;
    float *mean, *rstd;
};
ZR_KERNELS hipError_t launch_layernorm_fwd(const NormFwd& f, hipStream_t stream);

struct NormBwd {
    const void *dy, *x, *weight;
    const float *mean, *rstd;
    zr_dtype dy_dt, x_dt, param_dt, dx_dt, grad_dt;
    int64_t rows, cols, ld_dy, ld_x, ld_dx;
    void *dx, *dweight, *dbias;
    int accumulate, add_dx;
    void* workspace;  // of layernorm_workspace() floats
};
ZR_KERNELS hipError_t launch_layernorm_bwd(const NormBwd& f, hipStream_t stream);
// Strips of rows that a backward pass leaves partial parameter gradients of:
// one block each, as many as the chip holds at once, and no more than there
// are steps of rows (a block takes 16, 4 or 1 rows at once). Up to kNormOne
// elements one block, with more rows at once, walks over all rows and writes the
// gradients itself: it takes longer than several would, but saves the joining
// launch.
constexpr int64_t kNormOne = 16384;
inline int layernorm_strips(int64_t rows, int64_t cols) {
    if (rows > 0 && rows * cols <= kNormOne) return 1;
    const int64_t per = cols <= 128 ? 16 : (cols <= 1024 ? 4 : 1), n = (rows + per - 1) / per;
    const int64_t places = cols <= 4096 ? 512 : 256, most = tuning().max_grid < places ? tuning().max_grid : places;
    return (int)(n < most ? n : most);
}
// Floats of workspace for them.
inline int64_t layernorm_workspace(int64_t rows, int64_t cols) {
    const int64_t strips = layernorm_strips(rows, cols);
    return strips > 1 || cols > 12288 ? strips * 2 * cols : 0;
}

ZR_KERNELS hipError_t launch_ckpt_pack(const void* x, zr_dtype dt, int64_t rows, int64_t cols, int64_t ld, zr_dtype fmt,
                                       void* ckpt, hipStream_t stream);
ZR_KERNELS hipError_t launch_ckpt_unpack(const void* ckpt, zr_dtype fmt, int64_t rows, int64_t cols, void* x,
                                         zr_dtype dt, int64_t ld, hipStream_t stream);

// How a weight gradient is cut. Both forms' times come from a model fitted to
// sweeps with bf16 dY over 11 shapes (rows 128 to 65,536, dW 128 x 128 to 4096 x
// 4096; its choices were within 10% of the best measured), and the smaller one is
// taken. fp32 dY, of three products, is cut by the same numbers, though a slab of
// it takes a small block about 4.9 us (1001x777x1000: 20 us for 4 slabs), so where
// tiles are few it gets fewer parts than would be best:
//  - a slab of 64 rows takes a small block 0.95 us alone, 1.05 with one block
//    on every CU and 1.4 with two; a large block 1.46 alone, 1.9 with all;
//  - joining costs 5 us and 0.35 us per MB of parts (more than it does where the
//    parts are small: 9.4 us for 1001x777x1000's, which take 5.2).
//
// Small form: tiles of 128 x 128, the sum over rows in `splits` parts of `span`
// rows. More parts fill the chip where there are few tiles, but each writes
// and reads dW once more in fp32.
constexpr int kWgradTile = 128, kWgradBig = 256;
constexpr float kWgradJoinUs = 5.0f, kWgradMbUs = 0.35f;
struct WgradCut {
    int splits;
    int64_t span;
    float us;
};
inline WgradCut wgrad_cut(int64_t rows, int64_t out, int64_t in) {
    const int64_t tiles = ((out + kWgradTile - 1) / kWgradTile) * ((in + kWgradTile - 1) / kWgradTile);
    const int64_t slabs = (rows + 63) / 64, places = 512;
    auto slab_us = [](int64_t blocks) {  // one slab of each of up to `places` blocks
        return blocks > 256 ? 1.4f : 0.95f + 0.1f * (float)blocks / 256.0f;
    };
    WgradCut best{1, (slabs > 0 ? slabs : 1) * 64, 0.0f};
    for (int64_t n = 1; n <= 64 && (n == 1 || n <= slabs); ++n) {
        const int64_t per = (slabs + n - 1) / n;
        if (n > 1 && (slabs + per - 1) / per != n) continue;  // the same parts as a smaller n
        const int64_t blocks = tiles * n, rounds = blocks / places, rest = blocks % places;
        float us = (float)per * ((float)rounds * slab_us(places) + (rest ? slab_us(rest) : 0.0f));
        if (n > 1) us += kWgradJoinUs + kWgradMbUs * 4e-6f * (float)n * (float)out * (float)in;
        if (n == 1 || us < best.us) best = WgradCut{(int)n, (per > 0 ? per : 1) * 64, us};
    }
    return best;
}

// Large form: tiles of 256 x 256, of which whole rounds of 256 take one block
// each; the slabs of the `rest` tiles are split into `parts` of `share` slabs,
// joined from the workspace, where part p of rest tile t has slot p * rest + t.
// (Sharing the rest's slabs out evenly, a block's share beginning anywhere in a
// tile, would fill the last round too, but blocks at different rows have no
// slabs in common in their L2: 16384x11008x4096, 176 rest tiles, took 1,446 us
// against 1,428 unsplit.)
struct WgradShare {
    int64_t slabs, full, rest, parts, share;
    float us;
};
constexpr int64_t kWgradSlot = kWgradBig * kWgradBig + kWgradBig;  // floats: a tile and its bias
inline WgradShare wgrad_share(int64_t rows, int64_t out, int64_t in) {
    const int64_t tiles = ((out + kWgradBig - 1) / kWgradBig) * ((in + kWgradBig - 1) / kWgradBig);
    auto slab_us = [](int64_t blocks) { return 1.46f + 0.44f * (float)blocks / 256.0f; };
    WgradShare w;
    w.slabs = rows > 0 ? (rows + 63) / 64 : 1;
    w.full = tiles / 256 * 256;
    w.rest = tiles - w.full;
    w.parts = 1;
    w.share = w.slabs;
    float best = (float)w.slabs * slab_us(w.rest);
    for (int64_t n = 2; n * w.rest <= 256 && n <= w.slabs && w.rest > 0; ++n) {
        const int64_t share = (w.slabs + n - 1) / n;
        if ((w.slabs + share - 1) / share != n) continue;  // the same shares as a smaller n
        const float us = (float)share * slab_us(n * w.rest) + kWgradJoinUs + kWgradMbUs * 4e-6f * (float)(n * w.rest * kWgradSlot);
        if (us < best) {
            best = us;
            w.parts = n;
            w.share = share;
        }
    }
    w.us = (float)(w.full / 256) * (float)w.slabs * slab_us(256) + (w.rest > 0 ? best : 0.0f);
    return w;
}

struct Wgrad {
    const void *dy, *ckpt;
    zr_dtype dy_dt, format, grad_dt;
    int64_t rows, out, in, ld_dy, ld_dw;
    void *dw, *dbias;
    int accumulate;
    void* workspace;  // of wgrad_workspace() floats
};
// The large form needs dY in bf16, at least a chunk of it per row, and 32-bit
// offsets within a slab.
inline bool wgrad_can_be_large(const Wgrad& w) {
    return w.dy_dt == ZR_BF16 && w.out >= 8 && w.ld_dy <= (1 << 24) && w.in <= (1 << 24);
}
// Floats of workspace that either form needs.
inline int64_t wgrad_workspace(int64_t rows, int64_t out, int64_t in) {
    const WgradCut c = wgrad_cut(rows, out, in);
    const WgradShare s = wgrad_share(rows, out, in);
    const int64_t a = c.splits > 1 ? c.splits * (out * in + out) : 0;
    const int64_t b = s.parts > 1 ? s.parts * s.rest * kWgradSlot : 0;
    // the large form is taken only where it is the faster one
    return s.us < c.us && b > a ? b : a;
}
ZR_KERNELS hipError_t launch_ckpt_wgrad(const Wgrad& w, hipStream_t stream);

// Norm, scaling and AdamW over many tensors: a launch carries so many in its
// arguments (4 KiB at most), and a longer list goes out as several.
constexpr int kNormPer = 192, kScalePer = 128, kAdamPer = 64;
constexpr int kNormBlocks = 2048;  // partial sums of a launch at most
constexpr int kNormTile = 8192;    // elements
constexpr int kNormOneElems = 16384;  // in as many tiles as one block has groups of lanes: taken by it alone
constexpr int64_t kCachedBytes = 256ll << 20;  // of the last cache

struct GradNorm {
    int n;
    const void* const* grads;
    const int64_t* numels;
    zr_dtype dt;
    double scale, max_norm;
    float *norm, *coef;
    void* workspace;  // of grad_norm_parts() doubles
};
ZR_KERNELS hipError_t launch_grad_norm(const GradNorm& f, hipStream_t stream);
inline int64_t grad_norm_parts(int n) { return ((int64_t)n + kNormPer - 1) / kNormPer * kNormBlocks; }

struct GradScale {
    int n;
    const void* const* grads;
    const int64_t* numels;
    zr_dtype dt, out_dt;
    void* const* outs;  // null: in place
    const float* coef;
};
ZR_KERNELS hipError_t launch_grad_scale(const GradScale& f, hipStream_t stream);

struct AdamW {
    int n;
    const void* const* grads;
    const int64_t* numels;
    zr_dtype grad_dt;
    void *const *params, *const *exp_avg, *const *exp_avg_sq, *const *shards;  // shards may be null
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;
    const float* coef;
    int64_t* left_out;  // may be null
};
ZR_KERNELS hipError_t launch_adamw(const AdamW& f, hipStream_t stream);

struct RmsFwd {
    const void *x, *residual, *weight;
    zr_dtype x_dt, h_dt, param_dt, y_dt, ckpt_format;
    int64_t rows, cols, ld_x, ld_res, ld_h, ld_y;
    float eps;
    void *h, *y, *ckpt_h, *ckpt_y;
    float* rstd;
};
ZR_KERNELS hipError_t launch_rmsnorm_fwd(const RmsFwd& f, hipStream_t stream);

struct RmsBwd {
    const void *dy, *h, *weight;
    const float* rstd;
    zr_dtype dy_dt, h_dt, param_dt, dx_dt, grad_dt;
    int64_t rows, cols, ld_dy, ld_h, ld_dx;
    void *dx, *dweight;
    int accumulate, add_dx;
    void* workspace;  // of rmsnorm_workspace() floats
};
ZR_KERNELS hipError_t launch_rmsnorm_bwd(const RmsBwd& f, hipStream_t stream);
// The layer norm's strips; a strip leaves one row of sums.
inline int64_t rmsnorm_workspace(int64_t rows, int64_t cols) {
    const int64_t strips = layernorm_strips(rows, cols);
    return strips > 1 || cols > 12288 ? strips * cols : 0;
}

// Packing of e2m1 blocks, and of a transpose (of any format).
ZR_KERNELS hipError_t launch_pack_small(const void* x, zr_dtype dt, int64_t rows, int64_t cols, int64_t ld, void* ckpt,
                                        hipStream_t stream);
ZR_KERNELS hipError_t launch_unpack_small(const void* ckpt, int64_t rows, int64_t cols, void* x, zr_dtype dt, int64_t ld,
                                          hipStream_t stream);
ZR_KERNELS hipError_t launch_pack_t(const void* x, zr_dtype dt, int64_t rows, int64_t cols, int64_t ld, void* ckpt,
                                    zr_dtype fmt, hipStream_t stream);

struct Linear {
    const void *x, *w, *bias;
    zr_dtype x_format, w_format, bias_dt, z_dt;
    int64_t rows, in, out, ld_z;
    void* z;
    int accumulate;
    void* workspace;  // of linear_workspace() floats
};
ZR_KERNELS hipError_t launch_linear(const Linear& f, hipStream_t stream);

// How a product of packed matrices is cut: form 0 for few rows, tiles of 128 x 128
// (1) or 256 x 256 (2), and the columns in `parts` of `share` turns of 512, joined
// from the workspace. The fastest by a model fitted to sweeps of 20 shapes (70 to 16384
// rows) in both forms of tiles and up to 22 parts, where its choices took at most 13%
// longer than the best measured (decoded; 10% else), and 1% in the mean, and of 10 shapes
// of up to 64 rows in all forms, where they took 3% longer in the mean and up to 41% (8
// outer shapes that it was not fitted to: 2.5% and 49%, a single row by 100000x640):
//  - a tile takes kStart, which has the results' writing in it, and kTurn for every turn,
//    the first of each with few blocks on the chip, the second with all places taken
//    (512 of form 1, 256 of form 2: of a whole MI355X, whatever the current device has,
//    because the workspace's size follows from the cut and is asked for on the host), in us;
//  - joining costs 4 us and 0.4 us per MB of parts;
//  - form 0 reads the tokens again for every 16 outputs: 3.4 us, 0.44 for every 4096
//    outputs, and kFew for every turn of 16, 32 and 64 tokens (a little over half of it is
//    there without any), by as many times 4096 outputs as there are, for more blocks than
//    the chip has CUs (64 tokens of 11008x4096 took 34 us where tiles take 17; 17 tokens of
//    4096x11008 in 4 bits 10.4 for 13.8, and of 777x1000 in 8 bits 5.3 for 8.1).
constexpr int kLinearGroup = 512;         // columns of a turn, of a load of exponents
constexpr int64_t kLinearWide = 1 << 23;  // columns up to which a tile's rows lie within 32-bit offsets
// What multiplies: scaled instructions with e4m3 on a side, or with e2m1 on both, or
// bf16 instructions on decoded operands (fp32 results, as of kLinearFourWide).
enum LinearKind { kLinearScaled = 0, kLinearFour = 1, kLinearDecoded = 2, kLinearFourWide = 3 };
struct LinearCut {
    int form, parts;
    int64_t turns, share;
};
inline LinearCut linear_cut(int64_t rows, int64_t out, int64_t in, LinearKind kind) {
    static constexpr float kStart[2][4][2] = {{{4.7f, 4.7f}, {5.4f, 5.4f}, {5.0f, 7.0f}, {6.0f, 6.0f}},
                                              {{8.2f, 8.2f}, {8.7f, 8.7f}, {8.0f, 16.0f}, {8.0f, 16.0f}}};
    static constexpr float kTurn[2][4][2] = {{{1.5f, 4.2f}, {0.7f, 2.4f}, {2.4f, 6.6f}, {0.7f, 2.8f}},
                                             {{3.6f, 6.5f}, {1.9f, 4.0f}, {5.2f, 12.5f}, {1.7f, 4.2f}}};
    static constexpr float kFew[4][3] = {{0.38f, 0.60f, 1.09f}, {0.23f, 0.34f, 0.62f}, {0.50f, 0.70f, 1.25f}, {0.22f, 0.33f, 0.61f}};
    const int64_t turns = (in + kLinearGroup - 1) / kLinearGroup;
    LinearCut best{0, 1, turns, turns};
    if (in > kLinearWide) return best;
    const int most = rows <= 16 ? 0 : (rows <= 32 ? 1 : 2);
    const float token = kFew[kind][most] * (0.57f + 0.43f * (float)rows / (float)(16 << most));
    const float wide = (float)out / 4096.0f, blocks = wide > 1.0f ? wide : 1.0f;
    const float few = 3.4f + 0.44f * blocks + (float)turns * token * (1.1f * wide > 1.0f ? 1.1f * wide : 1.0f);
    float least = rows <= 64 ? few : 3e38f;
    for (int f = 0; f < 2; ++f) {
        const int64_t edge = f ? 256 : 128, places = f ? 256 : 512;
        const int64_t tiles = ((rows + edge - 1) / edge) * ((out + edge - 1) / edge);
        const float *s = kStart[f][kind], *t = kTurn[f][kind];
        for (int64_t n = 1; n <= 32 && n <= turns; ++n) {
            const int64_t share = (turns + n - 1) / n;
            if (n > 1 && ((turns + share - 1) / share != n || tiles * n > 2 * places)) continue;
            const int64_t blocks = tiles * n, rounds = blocks / places, rest = blocks % places;
            auto tile = [&](int64_t on) {
                const float full = (float)on / (float)places;
                return s[0] + (s[1] - s[0]) * full + (float)share * (t[0] + (t[1] - t[0]) * full);
            };
            float us = (float)rounds * tile(places) + (rest ? tile(rest) : 0.0f);
            if (n > 1) us += 4.0f + 1.6e-6f * (float)n * (float)rows * (float)out;
            if (us < least) {
                best = LinearCut{f + 1, (int)n, turns, share};
                least = us;
            }
        }
    }
    return best;
}
// Floats of workspace that the cut needs, whatever the formats.
inline int64_t linear_workspace(int64_t rows, int64_t out, int64_t in) {
    int64_t need = 0;
    for (LinearKind k : {kLinearScaled, kLinearFour, kLinearDecoded, kLinearFourWide}) {
        const LinearCut c = linear_cut(rows, out, in, k);
        const int64_t n = c.parts > 1 ? c.parts * rows * out : 0;
        need = n > need ? n : need;
    }
    return need;
}

}  // namespace zr
