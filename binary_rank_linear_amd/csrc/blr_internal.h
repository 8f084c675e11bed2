// Internal interface between the C ABI (blr_api.hip) and the kernels
// (blr_kernels.hip). Not installed; the public interface is include/blr.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace blr {

// Smallest row tile of the MFMA contraction kernels; the column reductions
// fused into the contractions write one partial row per row tile, so the
// partial buffers are sized for this tile.
constexpr int GEMM_BM_MIN = 64;
// Tokens per partial of the standalone column reduction.
constexpr int COLSUM_ROWS = 64;
// Tokens per row of the dl partial buffer as sized (every producer writes
// one row per 64 tokens, within this).
constexpr int PART_ROWS_MIN = 32;

// Kernel kinds, for per-kernel timing.
enum KernelId {
    K_EXPAND = 0,
    K_TRANSPOSE, // bitmap [rows][r/32] -> [r][rows/32]
    K_GEMM_F1,   // a = (x.g) S_V
    K_GEMM_F2,   // c = (a.l) S_U^T, y (+)= h.c
    K_GEMM_B1,   // db = (dy.h.gs) S_U / gs, partials of dl
    K_GEMM_B2,   // dx' = (db.l.gs) S_V^T / gs, dx (+)= g.dx', partials of dg
    K_COLSUM,    // partials of dh = sum_t dy.c from the stored c tape
    K_GEMM_DH,   // c recomputed as in F2, partials of dh = sum_t dy.c
    K_FINISH,    // sum of partials into dh / dl / dg
    K_GEMM_B1_DH, // B1 with dh fused (c recomputed per column block)
    K_GEMM_SIGNS, // sign gradients G_U, G_V (contractions over tokens)
    K_SUMSQ,      // sum-of-squares partials (finite check)
    K_GEMM_PLANE, // dense frozen f16 linear
    K_SIGNS_REDUCE, // sign gradients: the token ranges' partials summed in order
    K_ROUTE_COUNT,  // routing: pairs per expert of each range of pairs
    K_ROUTE_PLACE,  // routing: order, slot and offsets
    K_ROUTE_GATHER, // rows laid out by expert
    K_ROUTE_COMBINE, // experts' rows weighted and summed back
    K_ROUTE_COMBINE_BWD, // gradients of the experts' rows and of the weights
    K_ADAPT_DOWN,   // adapters: partials of s = x A^T
    K_ADAPT_UP,     // adapters: y (+)= c s B^T
    K_ADAPT_PREPARE, // adapters: the backward's A^T and B^T, the tape's panel
    K_ADAPT_DS,     // adapters: partials of ds = c dy B
    K_ADAPT_DX,     // adapters: dx (+)= ds A
    K_ADAPT_DY,     // adapters: partials of ds, and the gradient of B
    K_ADAPT_THIN,   // adapters: ds as the gradient's operand
    K_ADAPT_DX_GRAD, // adapters: dx, and the gradient of A
    K_ADAPT_REDUCE, // adapters: the ranges' partials summed in order
    K_COUNT
};
const char *kernel_name(int id);

// out[m][n] = (sum_k f16(A[m][k] * colscale[k] * ascale) * S[n][k]) * oscale
// with the +-1 plane S [N][K] given as a bitmap; every [M][N] array below
// has row stride N.
struct GemmArgs {
    const float *A;        // [M][lda] f32
    int64_t lda;
    const float *colscale; // [K]
    float ascale;          // power of two
    const uint32_t *Bbits; // sign bitmap of the plane [N][K]: row n, word k/32, bit k%32 (set = +1)
    const uint16_t *Bplane; // GEMM_PLANE: the f16 plane [N][K] itself (no column scale)
    int64_t M;
    int N, K;
    float oscale;          // power of two (1/ascale)
    float *out;            // [M][N] raw product (F1: tape a, F2: tape c, B1: db)
    float *out2;           // [M][N] out2 (+)= out2col[n] * product (F2: y, B2: dx)
    const float *out2col;
    int out2acc;
    const float *dot_other; // [M][N]: partial[mt][n] = sum_{m in tile} product * other
    float *dot_partial;     // [ceil(M/gemm_tile_rows(kind))][N]
    // B1 with the dh reduction fused (GEMM_B1_DH): c = (a.l) S_U^T is
    // recomputed per column block of dy and dh partials sum dy.c over the tile
    const uint32_t *dh_bits; // bitmap of S_U [K][N/32] (K = d_out, N = r)
    const float *dh_a;       // the a tape [M][N]
    const float *dh_l;       // l [N]
    float *dh_partial;       // [(N/BN) * ceil(M/BM)][K], row nt * ceil(M/BM) + mt
    // A layer of several paths (y = sum_p h_p . c_p); zero for one path.
    // Paths along N (F1, B1: the ranks of all paths side by side): path_n
    // columns per path; the tile of column n0 belongs to path n0 / path_n,
    // whose column scales start at colscale + path * cs_pstride and, for the
    // fused dh role, whose S_U bitmap is dh_bits + path * dh_pstride words
    // with dh_row_words words per row.
    int path_n;
    int64_t cs_pstride, dh_pstride;
    int dh_row_words;
    // Paths along K (GEMM_F2_MP, GEMM_B2_MP: K = paths * path_k): the
    // bitmap of path q is Bbits + q * b_pstride words, rows of path_k / 32
    // words; at the end of each path's ranks the product is scaled by
    // out2col + q * o2_pstride into a running sum (stored at the end), and
    // that path's column partials go to dot_partial + q * dot_pstride.
    int path_k;
    int64_t b_pstride, o2_pstride, dot_pstride;
};

// F2 writes the c tape and y (F2) or y only (F2_NOTAPE); DH repeats F2's
// contraction with the same tiles (so c is bit-identical) and sums dy.c.
enum GemmKind {
    GEMM_F1 = 0, GEMM_F2, GEMM_F2_NOTAPE, GEMM_B1, GEMM_B2, GEMM_DH, GEMM_B1_DH, GEMM_PLANE,
    GEMM_F2_MP,  // y (+)= sum_p h_p . c_p over paths along K (no c tape)
    GEMM_B2_MP   // dx (+)= sum_p g_p . dx'_p, partials of dg_p per path
};
// Most paths of one layer the fused launches serve.
constexpr int MAX_PATHS = 4;
// At most this many 64 x 256 tiles (half the CUs) leave the chip half idle
// or worse: F1, B1 and the fused B1_DH then take 128-column tiles.
constexpr int64_t SMALL_GRID = 128;
// GEMM_B1_DH tiles for M tokens and P paths of r ranks: rank columns and
// token rows per workgroup (0 where the fused launch does not serve r). The
// dh partials of a path have ceil(M / b1dh_tile_rows(r)) * (r /
// b1dh_cols(M, r, P)) rows, at most 4 * ceil(M / 64); the dl partials
// ceil(M / b1dh_tile_rows(r)).
int b1dh_cols(int64_t M, int64_t r, int64_t P);
int b1dh_tile_rows(int64_t r);

// Sign-plane expansion jobs (one bitmap each; pl and/or plt may be null).
struct ExpandJob {
    const uint32_t *bits;  // [rows][ceil(r/32)]
    int64_t rows, r;
    uint16_t *pl;   // f16 [rows][r]
    uint16_t *plt;  // f16 [r][rows]
};
struct ExpandJobs {
    ExpandJob job[2];
    int count;
};

// Column-sum finishing jobs: out[n] += sum_p partial[p][n].
struct FinishJob {
    const float *partial;
    int64_t nparts;
    int N;
    float *out;
};
struct FinishJobs {
    FinishJob job[2 * MAX_PATHS + 1];
    int blocks_before[2 * MAX_PATHS + 1];
    int count;
};

// Token-contraction jobs for the sign gradients:
//   out[m][n] (+)= (sum_t f16(A[t][m] acol[m] ascale) f16(B[t][n] bcol[n] bscale)) oscale
// A [T][lda] and B [T][ldb] row-major (columns Mo and No used); out
// [Mo][No]; Mo, No multiples of 128.
struct TnJob {
    const float *A;
    const float *acol;
    float ascale;
    const float *B;
    const float *bcol;
    float bscale;
    int Mo, No;
    float oscale;
    float *out;
    int acc;
    int tiles_before;  // filled by the launcher
    int64_t lda, ldb;  // row strides of A and B (elements)
    int64_t elems_before;  // filled by the launcher: sum of Mo * No of the jobs before
};
struct TnJobs {
    TnJob job[2 * MAX_PATHS];
    int count;
    int64_t T;
    // Partial sums of token ranges 1 .. splits-1 (range 0 writes out itself):
    // part[(s - 1) * part_stride + elems_before + m * No + n], with
    // part_stride = sum over jobs of Mo * No. Needed when sign_splits() > 1.
    float *part;
};
// Token ranges of the sign-gradient contraction on its 256 x 256 tiles:
// enough ranges (each at least 512 tokens) to give about 256 workgroups over
// `tiles256` output tiles, 1 when the tiles alone fill the GPU. Only shapes
// whose output sizes are all multiples of 256 take those tiles (and ranges).
int sign_splits(int64_t tiles256, int64_t T);

// Launchers: enqueue on `s`, return the launch error (hipSuccess if none).
hipError_t launch_gemm_tn(TnJobs jobs, hipStream_t s);
hipError_t launch_sumsq(const float *a, int64_t n, float *partials, int nparts, hipStream_t s);
hipError_t launch_expand(const ExpandJobs &jobs, hipStream_t s);
// out [r][rows/32]: bit (i % 32) of word i / 32 in row k is rank k of row i
// of bits [rows][r/32] (rows and r multiples of 32); for paths > 1, bits
// holds that many such bitmaps back to back and out their transposes.
hipError_t launch_transpose_bits(const uint32_t *bits, int64_t rows, int64_t r, uint32_t *out, hipStream_t s,
                                 int paths = 1);
hipError_t launch_gemm(GemmKind kind, const GemmArgs &a, hipStream_t s);
int gemm_tile_rows(GemmKind kind);
hipError_t launch_colsum(const float *A, const float *B, int64_t M, int N, float *partial, hipStream_t s);
hipError_t launch_finish(FinishJobs jobs, hipStream_t s);

// ---------------------------------------------------------------- routing --
// Most experts a sort takes (its counters lie in LDS, one table per wave).
constexpr int ROUTE_MAX_EXPERTS = 1024;
// Ranges of pairs of the sort: how many, and pairs per range (a multiple of
// 64). One range is placed by a single launch.
int64_t route_ranges(int64_t pairs, int64_t *per_range);
struct RouteSortArgs {
    const int32_t *ids;  // [pairs]
    int32_t *offsets;    // [experts + 1]
    int32_t *order, *slot;
    uint32_t *counts;    // [ranges][experts + 1], used when ranges > 1
    int pairs, experts, per_range, ranges;
};
hipError_t launch_route_sort(const RouteSortArgs &a, hipStream_t s);

// Rows of d elements; row pointers 16-byte aligned, d a multiple of 8.
struct RouteRows {
    const int32_t *placed;  // &offsets[experts]: pairs that have an expert
    const int32_t *slot;    // [T][k]
    const float *weights;   // [T][k] or null (all one)
    const void *a;          // gather: x; combine: z; backward: dy
    const void *z;          // backward: z (null when dw is)
    void *out;              // gather: rows; combine: y; backward: dz
    float *dw;              // backward: [T][k] or null
    int64_t T, d;
    int k, dtype, acc;
};
hipError_t launch_route_gather(const RouteRows &a, hipStream_t s);
hipError_t launch_route_combine(const RouteRows &a, hipStream_t s);
hipError_t launch_route_combine_backward(const RouteRows &a, hipStream_t s);

// --------------------------------------------------------------- adapters --
// Rows per tile of the adapter contractions, and the limits of a call.
constexpr int ADAPT_TM = 64;
constexpr int ADAPT_MAX_RANK = 128;
constexpr int ADAPT_MAX_SPLITS = 32;
// Rows grouped by adapter: position p of the plan belongs to adapter e when
// offsets[e] <= p < offsets[e + 1], and holds row order[p] (p itself when
// order is null). Positions from offsets[E] on have no adapter.
struct AdaptPlan {
    const int32_t *offsets;
    const int32_t *order;
    int M, E;
};
// part[split][p][r] = sum over the split's columns of X[row(p)][k] W_e[.][k]
// with W_e = W + e r K, [r][K].
struct AdaptShrink {
    AdaptPlan plan;
    const void *X, *W;
    float *part;
    int K, r, splits, act, wt;
    bool once;  // X is not worth keeping in the caches; set by the launcher of ds and grad_up
};
// out[row(p)][n] (+)= sum_k S[p][k] W_e[n][k], S[p] = scale_e sum over splits
// of part[.][p]; W_e: [N][r]. S goes to s_row by row, unscaled (unless null).
struct AdaptExpand {
    AdaptPlan plan;
    const float *part;
    const float *scale;
    const void *W;
    void *out;
    float *s_row;
    int N, r, splits, act, wt, acc;
};
// The gradients' thin operands, ds (scaled) and the tape s, as panels: of each
// tile of 64 positions, its ranks (rounded up to 16, 32, 64 or 128: r16) by 64
// positions, zero past the tile's end, in the order of the matrix operand; f32
// for rows of f32, three bf16 terms for rows of 16 bits.
struct AdaptThin {  // panels of ds alone
    AdaptPlan plan;
    const float *part, *scale;
    void *panel;
    int r, splits, act;
};
// dst_e [cols][rows] = the transpose of src_e [rows][cols] for the adapters that
// have rows, two tables; the tape's panels (tape null: none); zeros into grad_e
// of the adapters that have none (null: not).
struct AdaptPrepare {
    AdaptPlan plan;
    const void *src[2];
    void *dst[2];
    int rows[2], cols[2];
    const float *tape;
    void *panel;
    float *grad[2];
    int r, act, wt;
    int tiles[2], zeros, panels;  // pieces of each kind of work; filled by the launcher
};
constexpr int64_t adapt_r16(int64_t r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : 128; }
constexpr int64_t adapt_panel_bytes(int64_t r, int act) { return adapt_r16(r) * 64 * (act == 0 ? 4 : 6); }
// The two gradients, G_e (+)= scale_e sum over the adapter's rows of
// thin[.][k] X[row][n]: job 0 laid out [r][N], job 1 [N][r]. Ranges of `range`
// positions; an adapter of several ranges leaves partials in part[slot], which
// the reduction adds in range order.
constexpr int ADAPT_MAX_RANGE = 4096;  // its rows' numbers lie in LDS
struct AdaptGradJob {
    const void *X;
    const void *panel;
    const float *scale;  // null: no factor
    float *grad, *part;
    int N;
};
struct AdaptGrad {
    AdaptPlan plan;
    AdaptGradJob job[2];
    int r, act, acc, range;
    int64_t panels;  // that exist
    int64_t slots;   // partials that each `part` has room for
    bool once;       // job 0's X is not worth keeping in the caches; set by its launcher
};
hipError_t launch_adapt_prepare(const AdaptPrepare &a, hipStream_t s);
// id: the kernel kind that the launch is timed as.
hipError_t launch_adapt_shrink(const AdaptShrink &a, int id, hipStream_t s);
hipError_t launch_adapt_expand(const AdaptExpand &a, int id, hipStream_t s);
hipError_t launch_adapt_dy(const AdaptShrink &sh, const AdaptGrad &gr, hipStream_t s);  // ds, and job 1
hipError_t launch_adapt_thin(const AdaptThin &a, hipStream_t s);
hipError_t launch_adapt_dx(const AdaptExpand &ex, const AdaptGrad &gr, hipStream_t s);  // dx (out null: not), and job 0
hipError_t launch_adapt_reduce(const AdaptGrad &a, hipStream_t s);
// Ranges of columns of the expand, per tile.
int64_t adapt_chunks(int64_t M, int64_t E, int64_t N);
// Tiles of tm positions that M positions in at most E + 1 groups can need.
int64_t adapt_tiles(int64_t M, int64_t E, int64_t tm);
int adapt_splits(int64_t M, int64_t E, int64_t K);
int64_t adapt_range(int64_t M, int64_t d_in, int64_t d_out, int64_t r);
// Partials of ranges that a gradient over M rows can leave.
int64_t adapt_range_slots(int64_t M, int64_t E, int64_t range);

// Profiling hooks around each launch (no-ops unless enabled).
void prof_begin(int id, hipStream_t s);
void prof_end(hipStream_t s);

}  // namespace blr
