// C ABI of the `blr` layer (include/blr.h): argument validation, workspace
// layout and launch order on the caller's stream. The order of the steps is
// the one of `blr_forward` / `blr_backward` on the cortiq-engine page
// "src/gpu_wgpu/train_mm.rs"; their staging and scaling passes live inside
// the contraction kernels.
#include <math.h>
#include <string.h>

#include <mutex>
#include <vector>

#include "../../include/blr.h"
#include "blr_internal.h"

namespace blr {

// ------------------------------------------------------------ profiling --
namespace {
struct ProfState {
    bool on = false;
    std::vector<hipEvent_t> ev;  // pairs
    std::vector<int> ids;        // kernel id per recorded pair
    size_t used = 0;
    int pending_id = -1;
    int64_t counts[K_COUNT] = {};
    double total_ms[K_COUNT] = {};
};
ProfState g_prof;
std::mutex g_prof_mu;

void prof_release() {
    for (hipEvent_t e : g_prof.ev) (void)hipEventDestroy(e);
    g_prof.ev.clear();
    g_prof.ids.clear();
    g_prof.used = 0;
    g_prof.on = false;
}
}  // namespace

void prof_begin(int id, hipStream_t s) {
    if (!g_prof.on) return;
    g_prof.pending_id = -1;
    if (2 * (g_prof.used + 1) > g_prof.ev.size()) return;  // pool full: launch goes untimed
    (void)hipEventRecord(g_prof.ev[2 * g_prof.used], s);
    g_prof.pending_id = id;
}

void prof_end(hipStream_t s) {
    if (!g_prof.on || g_prof.pending_id < 0) return;
    (void)hipEventRecord(g_prof.ev[2 * g_prof.used + 1], s);
    g_prof.ids.push_back(g_prof.pending_id);
    g_prof.used += 1;
    g_prof.pending_id = -1;
}

// ------------------------------------------------------------ workspace --
namespace {
constexpr size_t ALIGN = 256;
size_t up(size_t v) { return (v + ALIGN - 1) / ALIGN * ALIGN; }

struct Layout {
    size_t bits_t;  // transposed bitmaps [P][r][max(d_in, d_out)/32] (u32)
    size_t db;      // f32 [M][P r]
    size_t part_h, part_l, part_g;
    size_t part_s;  // sign gradients: partials of token ranges 1.. (f32)
    size_t total;
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// P paths (1 for a plain layer); the paths' ranks lie side by side.
Layout layout(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t P = 1) {
    Layout L;
    size_t off = 0;
    L.bits_t = off;
    off += up((size_t)(P * r * ((d_in > d_out ? d_in : d_out) / 32)) * 4);
    L.db = off;
    off += up((size_t)(M * P * r) * 4);
    // dh partials per path: ceil(M/64) rows from the c-tape column sum or the
    // recomputed-c contraction, ceil(M/64) per rank tile from B1 with dh
    // fused (up to four tiles of 128 ranks); dl partials: one row per 32
    // tokens; dg partials: one row per 64 tokens and path
    const int64_t bc = b1dh_cols(M, r, P);
    const int64_t hrows = ceil_div(M, GEMM_BM_MIN) * (bc ? r / bc : 1);
    L.part_h = off;
    off += up((size_t)(P * hrows * d_out) * 4);
    L.part_l = off;
    off += up((size_t)(ceil_div(M, PART_ROWS_MIN) * P * r) * 4);
    L.part_g = off;
    off += up((size_t)(P * ceil_div(M, GEMM_BM_MIN) * d_in) * 4);
    // the sign gradients' token ranges past the first (256 x 256 tiles only):
    // (splits - 1) copies of G_U and G_V, under 64 MB whatever the shape
    // (splits * tiles stays near 256)
    L.part_s = off;
    if (d_in % 256 == 0 && d_out % 256 == 0 && r % 256 == 0) {
        const int64_t tiles = P * ((d_out / 256) * (r / 256) + (d_in / 256) * (r / 256));
        const int64_t splits = sign_splits(tiles, M);
        off += up((size_t)((splits - 1) * P * (d_out + d_in) * r) * 4);
    }
    L.total = off;
    return L;
}

// Sizes the kernels accept: d_in, d_out, r multiples of 128 (the page's GEMM
// contract), M >= 1, and everything small enough for 32-bit grid and column
// indices.
bool shape_ok(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t P = 1) {
    if (P < 1 || P > MAX_PATHS) return false;
    if (P > 1) {
        // the paths' ranks side by side are one operand dimension
        if (!shape_ok(M, d_in, d_out, P * r)) return false;
    }
    if (M < 1 || d_in < 128 || d_out < 128 || r < 128) return false;
    if (d_in % 128 || d_out % 128 || r % 128) return false;
    const int64_t LIM = (int64_t)1 << 24;  // ranks
    if (r > LIM) return false;
    if ((d_in + 63) / 64 > 65535 || (d_out + 63) / 64 > 65535) return false;  // expansion grid rows
    if (ceil_div(M, COLSUM_ROWS) > 65535) return false;
    // the contraction kernels address every operand with 32-bit byte offsets
    const int64_t widest = d_in > d_out ? (d_in > r ? d_in : r) : (d_out > r ? d_out : r);
    if (M * widest * 4 > (int64_t)0xFFFFFFFF) return false;
    if ((d_out / 128) * ceil_div(M, GEMM_BM_MIN) > ((int64_t)1 << 31) - 1) return false;
    if ((d_in / 128) * ceil_div(M, GEMM_BM_MIN) > ((int64_t)1 << 31) - 1) return false;
    return true;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

// Products are divided by s, as a product with its inverse: f32 has none below 2^-127.
bool pow2_scale_ok(float s) {
    if (!(s > 0.0f) || !isfinite(s) || !isfinite(1.0f / s)) return false;
    int e;
    return frexpf(s, &e) == 0.5f;
}

int g_supported[64];  // 0 unknown, 1 yes, -1 no
std::mutex g_dev_mu;

int current_device_ok() {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return BLR_ERR_HIP;
    if (dev < 0 || dev >= 64) return blr_device_supported(dev) ? BLR_OK : BLR_ERR_DEVICE;
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if (g_supported[dev] == 0) g_supported[dev] = blr_device_supported(dev) ? 1 : -1;
    return g_supported[dev] == 1 ? BLR_OK : BLR_ERR_DEVICE;
}

#define BLR_TRY(expr)                                   \
    do {                                                \
        if ((expr) != hipSuccess) return BLR_ERR_HIP;   \
    } while (0)
}  // namespace

}  // namespace blr

using namespace blr;

extern "C" {

const char *blr_status_string(int status) {
    switch (status) {
        case BLR_OK: return "ok";
        case BLR_ERR_NULL: return "a required pointer is NULL";
        case BLR_ERR_SHAPE: return "invalid shape (d_in, d_out, r must be multiples of 128; M >= 1)";
        case BLR_ERR_SCALE: return "gscale must be a power of two from 2^-127 to 2^127, eps finite and not below zero";
        case BLR_ERR_WORKSPACE: return "workspace missing or smaller than blr_workspace_bytes()";
        case BLR_ERR_DEVICE: return "the current device is not gfx950";
        case BLR_ERR_HIP: return "HIP runtime error";
        case BLR_ERR_ALIGN: return "a pointer is not 16-byte aligned";
        case BLR_ERR_DTYPE: return "element type (or pair of types) not supported by this call";
        case BLR_ERR_OVERLAP: return "an output shares memory with another argument";
        case BLR_ERR_SCRATCH: return "sizes need more than the allocation-free forward's scratch (r * d_in / 8 bytes)";
    }
    return "unknown status";
}

int blr_device_supported(int hip_device) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, hip_device) != hipSuccess) return 0;
    return strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 0;
}

size_t blr_workspace_bytes(int64_t M, int64_t d_in, int64_t d_out, int64_t r) {
    if (!shape_ok(M, d_in, d_out, r)) return 0;
    return layout(M, d_in, d_out, r).total;
}

int blr_expand_signs(const uint32_t *bits, int64_t rows, int64_t r, uint16_t *plane, uint16_t *plane_t,
                     void *stream) {
    if (bits == nullptr || (plane == nullptr && plane_t == nullptr)) return BLR_ERR_NULL;
    if (rows < 1 || r < 1 || (rows + 63) / 64 > 65535 || r > ((int64_t)1 << 30) || rows * r > ((int64_t)1 << 40))
        return BLR_ERR_SHAPE;
    if (!aligned4(bits) || (plane && !aligned16(plane)) || (plane_t && !aligned16(plane_t))) return BLR_ERR_ALIGN;
    int st = current_device_ok();
    if (st != BLR_OK) return st;
    ExpandJobs jobs = {};
    jobs.job[0] = {bits, rows, r, plane, plane_t};
    jobs.count = 1;
    return launch_expand(jobs, (hipStream_t)stream) == hipSuccess ? BLR_OK : BLR_ERR_HIP;
}

// A layer of P paths (P = 1: the plain layer). Path p's operands are the
// p-th blocks of bits_u [P][d_out][r/32], bits_v [P][d_in][r/32],
// h [P][d_out], l [P][r], g [P][d_in]; the a tape is [M][P r] (the paths'
// ranks side by side). F1 runs once over the concatenated ranks; F2 runs
// once with the paths along K (one flush per path) when P > 1.
// Arguments of the forward, workspace aside.
static int forward_check(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t P, const float *x,
                         const uint32_t *bits_u, const uint32_t *bits_v, const float *h, const float *l,
                         const float *g, const float *y, const float *tape_a, const float *tape_c) {
    if (!x || !bits_u || !bits_v || !h || !l || !g || !y || !tape_a) return BLR_ERR_NULL;
    if (!shape_ok(M, d_in, d_out, r, P)) return BLR_ERR_SHAPE;
    if (P > 1 && tape_c) return BLR_ERR_SHAPE;  // no c tape for several paths
    const void *f16a[] = {x, h, l, g, y, tape_a, tape_c ? tape_c : tape_a};
    for (const void *p : f16a)
        if (!aligned16(p)) return BLR_ERR_ALIGN;
    if (!aligned16(bits_u) || !aligned16(bits_v)) return BLR_ERR_ALIGN;
    return BLR_OK;
}

// The forward's launches, after validation. bits_vt: room for the
// transposed S_V bitmaps, [P][r][d_in/32] u32 (16-byte aligned), the only
// scratch the forward uses.
static int forward_launch(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t P, const float *x,
                          const uint32_t *bits_u, const uint32_t *bits_v, const float *h, const float *l,
                          const float *g, float *y, int accumulate_y, float *tape_a, float *tape_c,
                          uint32_t *bits_vt, hipStream_t s) {
    BLR_TRY(launch_transpose_bits(bits_v, d_in, r, bits_vt, s, (int)P));

    GemmArgs f1 = {};
    f1.A = x;
    f1.lda = d_in;
    f1.colscale = g;
    f1.ascale = 1.0f;
    f1.Bbits = bits_vt;
    f1.M = M;
    f1.N = (int)(P * r);
    f1.K = (int)d_in;
    f1.oscale = 1.0f;
    f1.out = tape_a;
    if (P > 1) {
        f1.path_n = (int)r;      // path n0 / r: x staged with g_p
        f1.cs_pstride = d_in;
    }
    BLR_TRY(launch_gemm(GEMM_F1, f1, s));

    GemmArgs f2 = {};
    f2.A = tape_a;
    f2.lda = P * r;
    f2.colscale = l;
    f2.ascale = 1.0f;
    f2.Bbits = bits_u;
    f2.M = M;
    f2.N = (int)d_out;
    f2.K = (int)(P * r);
    f2.oscale = 1.0f;
    f2.out = tape_c;
    f2.out2 = y;
    f2.out2col = h;
    f2.out2acc = accumulate_y ? 1 : 0;
    if (P > 1) {
        f2.path_k = (int)r;                 // S_U of path q: bits_u + q d_out r/32 words
        f2.b_pstride = d_out * (r / 32);
        f2.o2_pstride = d_out;              // h_q
        BLR_TRY(launch_gemm(GEMM_F2_MP, f2, s));
    } else {
        BLR_TRY(launch_gemm(tape_c ? GEMM_F2 : GEMM_F2_NOTAPE, f2, s));
    }
    return BLR_OK;
}

static int forward_impl(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t P, const float *x,
                        const uint32_t *bits_u, const uint32_t *bits_v, const float *h, const float *l,
                        const float *g, float *y, int accumulate_y, float *tape_a, float *tape_c, void *workspace,
                        size_t workspace_bytes, void *stream) {
    int st = forward_check(M, d_in, d_out, r, P, x, bits_u, bits_v, h, l, g, y, tape_a, tape_c);
    if (st != BLR_OK) return st;
    const Layout L = layout(M, d_in, d_out, r, P);
    if (workspace == nullptr || workspace_bytes < L.total) return BLR_ERR_WORKSPACE;
    if (!aligned16(workspace)) return BLR_ERR_ALIGN;
    st = current_device_ok();
    if (st != BLR_OK) return st;
    uint32_t *bits_vt = (uint32_t *)((char *)workspace + L.bits_t);  // S_V^T per path, [P][r][d_in/32]
    return forward_launch(M, d_in, d_out, r, P, x, bits_u, bits_v, h, l, g, y, accumulate_y, tape_a, tape_c, bits_vt,
                          (hipStream_t)stream);
}

int blr_forward(int64_t M, int64_t d_in, int64_t d_out, int64_t r, const float *x, const uint32_t *bits_u,
                const uint32_t *bits_v, const float *h, const float *l, const float *g, float *y, int accumulate_y,
                float *tape_a, float *tape_c, void *workspace, size_t workspace_bytes, void *stream) {
    return forward_impl(M, d_in, d_out, r, 1, x, bits_u, bits_v, h, l, g, y, accumulate_y, tape_a, tape_c, workspace,
                        workspace_bytes, stream);
}

// ------------------------------------------------------ no allocation --
// The allocation-free forward's scratch: room for the transposed S_V bitmap.
// Each GPU the library runs on holds its own copy until the process ends.
// In host code this name is not a device address: the address each device
// uses comes from hipGetSymbolAddress (scratch_on_device below).
static __device__ __align__(256) uint8_t scratch[BLR_NOALLOC_SCRATCH_BYTES];

namespace {
void *g_scratch_ptr[64];  // per device, looked up on its first call
std::mutex g_scratch_mu;

int scratch_on_device(void **out) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return BLR_ERR_HIP;
    if (dev < 0 || dev >= 64) return BLR_ERR_DEVICE;
    std::lock_guard<std::mutex> lk(g_scratch_mu);
    if (g_scratch_ptr[dev] == nullptr) {
        void *p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || p == nullptr) return BLR_ERR_HIP;
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return BLR_OK;
}
}  // namespace

int blr_forward_noalloc(int64_t M, int64_t d_in, int64_t d_out, int64_t r, const float *x, const uint32_t *bits_u,
                        const uint32_t *bits_v, const float *h, const float *l, const float *g, float *y,
                        int accumulate_y, float *tape_a, float *tape_c, void *stream) {
    int st = forward_check(M, d_in, d_out, r, 1, x, bits_u, bits_v, h, l, g, y, tape_a, tape_c);
    if (st != BLR_OK) return st;
    if ((uint64_t)r * (uint64_t)d_in / 8 > (uint64_t)BLR_NOALLOC_SCRATCH_BYTES) return BLR_ERR_SCRATCH;
    st = current_device_ok();
    if (st != BLR_OK) return st;
    void *bits_vt = nullptr;
    st = scratch_on_device(&bits_vt);
    if (st != BLR_OK) return st;
    return forward_launch(M, d_in, d_out, r, 1, x, bits_u, bits_v, h, l, g, y, accumulate_y, tape_a, tape_c,
                          (uint32_t *)bits_vt, (hipStream_t)stream);
}

int blr_forward_paths(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t paths, const float *x,
                      const uint32_t *bits_u, const uint32_t *bits_v, const float *h, const float *l, const float *g,
                      float *y, int accumulate_y, float *tape_a, void *workspace, size_t workspace_bytes,
                      void *stream) {
    return forward_impl(M, d_in, d_out, r, paths, x, bits_u, bits_v, h, l, g, y, accumulate_y, tape_a, nullptr,
                        workspace, workspace_bytes, stream);
}

size_t blr_workspace_bytes_paths(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t paths) {
    if (!shape_ok(M, d_in, d_out, r, paths)) return 0;
    return layout(M, d_in, d_out, r, paths).total;
}

// The backward of P paths, and with grad_u / grad_v the sign gradients
// after it (both or neither). dh [P][d_out], dl [P][r], dg [P][d_in],
// grad_u [P][d_out][r], grad_v [P][d_in][r].
static int backward_impl(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t P, const float *x,
                         const float *dy, const uint32_t *bits_u, const uint32_t *bits_v, const float *h,
                         const float *l, const float *g, const float *tape_a, const float *tape_c, float gscale,
                         float *dh, float *dl, float *dg, float *dx, int accumulate_dx, float *grad_u, float *grad_v,
                         int accumulate_signs, void *workspace, size_t workspace_bytes, void *stream) {
    if (!x || !dy || !bits_u || !bits_v || !h || !l || !g || !tape_a || !dh || !dl || !dg || !dx)
        return BLR_ERR_NULL;
    if ((grad_u == nullptr) != (grad_v == nullptr)) return BLR_ERR_NULL;
    if (grad_u && (!aligned16(grad_u) || !aligned16(grad_v))) return BLR_ERR_ALIGN;
    if (!shape_ok(M, d_in, d_out, r, P)) return BLR_ERR_SHAPE;
    if (P > 1 && tape_c) return BLR_ERR_SHAPE;
    if (!pow2_scale_ok(gscale)) return BLR_ERR_SCALE;
    const Layout L = layout(M, d_in, d_out, r, P);
    if (workspace == nullptr || workspace_bytes < L.total) return BLR_ERR_WORKSPACE;
    const void *f16a[] = {x, dy, h, l, g, tape_a, tape_c ? tape_c : tape_a, dh, dl, dg, dx, workspace};
    for (const void *p : f16a)
        if (!aligned16(p)) return BLR_ERR_ALIGN;
    if (!aligned16(bits_u) || !aligned16(bits_v)) return BLR_ERR_ALIGN;
    int st = current_device_ok();
    if (st != BLR_OK) return st;

    hipStream_t s = (hipStream_t)stream;
    char *ws = (char *)workspace;
    uint32_t *bits_ut = (uint32_t *)(ws + L.bits_t);  // S_U^T per path, [P][r][d_out/32]
    float *db = (float *)(ws + L.db);                 // [M][P r]
    float *part_h = (float *)(ws + L.part_h);
    float *part_l = (float *)(ws + L.part_l);
    float *part_g = (float *)(ws + L.part_g);
    const float inv = 1.0f / gscale;  // exact: gscale is a power of two
    const int64_t Pr = P * r;
    const int64_t b1dh_c = b1dh_cols(M, r, P);
    const bool fused = tape_c == nullptr && b1dh_c > 0;  // B1 with dh fused
    const int64_t mt_b1 = ceil_div(M, fused ? b1dh_tile_rows(r) : gemm_tile_rows(GEMM_B1));
    const int64_t mt_b2 = ceil_div(M, gemm_tile_rows(P > 1 ? GEMM_B2_MP : GEMM_B2));

    BLR_TRY(launch_transpose_bits(bits_u, d_out, r, bits_ut, s, (int)P));

    // partials of dh_p = sum_t dy.c_p, nparts_h rows per path: inside B1
    // below, from the stored tape, or with c recomputed by F2's contraction
    // (same tiles, so the same c)
    int64_t nparts_h = 0;
    if (fused) {
        nparts_h = mt_b1 * (r / b1dh_c);  // one row per (rank tile, row tile) of the path
    } else if (tape_c) {
        BLR_TRY(launch_colsum(dy, tape_c, M, (int)d_out, part_h, s));
        nparts_h = ceil_div(M, COLSUM_ROWS);
    } else {
        nparts_h = ceil_div(M, gemm_tile_rows(GEMM_DH));
        for (int64_t q = 0; q < P; ++q) {
            GemmArgs rc = {};
            rc.A = tape_a + q * r;
            rc.lda = Pr;
            rc.colscale = l + q * r;
            rc.ascale = 1.0f;
            rc.Bbits = bits_u + q * d_out * (r / 32);
            rc.M = M;
            rc.N = (int)d_out;
            rc.K = (int)r;
            rc.oscale = 1.0f;
            rc.dot_other = dy;
            rc.dot_partial = part_h + q * nparts_h * d_out;
            BLR_TRY(launch_gemm(GEMM_DH, rc, s));
        }
    }

    // db_p = f16(dy.h_p.gs) S_U,p / gs for all paths side by side; dl += sum_t a.db
    GemmArgs b1 = {};
    b1.A = dy;
    b1.lda = d_out;
    b1.colscale = h;
    b1.ascale = gscale;
    b1.Bbits = bits_ut;
    b1.M = M;
    b1.N = (int)Pr;
    b1.K = (int)d_out;
    b1.oscale = inv;
    b1.out = db;
    b1.dot_other = tape_a;
    b1.dot_partial = part_l;
    if (P > 1) {
        b1.path_n = (int)r;  // path n0 / r: dy staged with h_p
        b1.cs_pstride = d_out;
    }
    if (fused) {
        // and, per 32-column block of dy, c_p = f16(a_p.l_p) S_U,p^T recomputed
        // and dh partials sum_t dy.c_p (c is not stored)
        b1.dh_bits = bits_u;
        b1.dh_a = tape_a;
        b1.dh_l = l;
        b1.dh_partial = part_h;
        if (P > 1) {
            b1.dh_pstride = d_out * (r / 32);
            b1.dh_row_words = (int)(r / 32);
        }
        BLR_TRY(launch_gemm(GEMM_B1_DH, b1, s));
    } else {
        BLR_TRY(launch_gemm(GEMM_B1, b1, s));
    }

    // dx'_p = f16(db_p.l_p.gs) S_V,p^T / gs; dx (+)= sum_p g_p.dx'_p;
    // dg_p += sum_t x.dx'_p
    GemmArgs b2 = {};
    b2.A = db;
    b2.lda = Pr;
    b2.colscale = l;
    b2.ascale = gscale;
    b2.Bbits = bits_v;
    b2.M = M;
    b2.N = (int)d_in;
    b2.K = (int)Pr;
    b2.oscale = inv;
    b2.out2 = dx;
    b2.out2col = g;
    b2.out2acc = accumulate_dx ? 1 : 0;
    b2.dot_other = x;
    b2.dot_partial = part_g;
    if (P > 1) {
        b2.path_k = (int)r;
        b2.b_pstride = d_in * (r / 32);
        b2.o2_pstride = d_in;
        b2.dot_pstride = mt_b2 * d_in;
        BLR_TRY(launch_gemm(GEMM_B2_MP, b2, s));
    } else {
        BLR_TRY(launch_gemm(GEMM_B2, b2, s));
    }

    // dh_p, dl, dg_p += their partial sums, one launch
    FinishJobs fin = {};
    int nj = 0;
    for (int64_t q = 0; q < P; ++q) fin.job[nj++] = {part_h + q * nparts_h * d_out, nparts_h, (int)d_out, dh + q * d_out};
    fin.job[nj++] = {part_l, mt_b1, (int)Pr, dl};
    for (int64_t q = 0; q < P; ++q) fin.job[nj++] = {part_g + q * mt_b2 * d_in, mt_b2, (int)d_in, dg + q * d_in};
    fin.count = nj;
    BLR_TRY(launch_finish(fin, s));

    if (grad_u) {
        // G_U,p = diag(h_p) dy^T a_p diag(l_p) from f16(dy.h_p.gs) and
        // f16(a_p.l_p); G_V,p = diag(g_p) x^T db_p diag(l_p) from f16(x.g_p)
        // and f16(db_p.l_p.gs); both / gs. The a tape and db hold the paths
        // side by side, so path p's columns start at p r with row stride P r.
        TnJobs tj = {};
        tj.T = M;
        tj.count = 0;
        tj.part = (float *)(ws + L.part_s);
        for (int64_t q = 0; q < P; ++q) {
            tj.job[tj.count++] = {dy, h + q * d_out, gscale, tape_a + q * r, l + q * r, 1.0f, (int)d_out, (int)r, inv,
                                  grad_u + q * d_out * r, accumulate_signs ? 1 : 0, 0, d_out, Pr, 0};
            tj.job[tj.count++] = {x, g + q * d_in, 1.0f, db + q * r, l + q * r, gscale, (int)d_in, (int)r, inv,
                                  grad_v + q * d_in * r, accumulate_signs ? 1 : 0, 0, d_in, Pr, 0};
        }
        BLR_TRY(launch_gemm_tn(tj, s));
    }
    return BLR_OK;
}

int blr_backward(int64_t M, int64_t d_in, int64_t d_out, int64_t r, const float *x, const float *dy,
                 const uint32_t *bits_u, const uint32_t *bits_v, const float *h, const float *l, const float *g,
                 const float *tape_a, const float *tape_c, float gscale, float *dh, float *dl, float *dg, float *dx,
                 int accumulate_dx, void *workspace, size_t workspace_bytes, void *stream) {
    return backward_impl(M, d_in, d_out, r, 1, x, dy, bits_u, bits_v, h, l, g, tape_a, tape_c, gscale, dh, dl, dg,
                         dx, accumulate_dx, nullptr, nullptr, 0, workspace, workspace_bytes, stream);
}

int blr_backward_signs(int64_t M, int64_t d_in, int64_t d_out, int64_t r, const float *x, const float *dy,
                       const uint32_t *bits_u, const uint32_t *bits_v, const float *h, const float *l, const float *g,
                       const float *tape_a, const float *tape_c, float gscale, float *dh, float *dl, float *dg,
                       float *dx, int accumulate_dx, float *grad_u, float *grad_v, int accumulate_signs,
                       void *workspace, size_t workspace_bytes, void *stream) {
    if (!grad_u || !grad_v) return BLR_ERR_NULL;
    return backward_impl(M, d_in, d_out, r, 1, x, dy, bits_u, bits_v, h, l, g, tape_a, tape_c, gscale, dh, dl, dg,
                         dx, accumulate_dx, grad_u, grad_v, accumulate_signs, workspace, workspace_bytes, stream);
}

int blr_backward_paths(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t paths, const float *x,
                       const float *dy, const uint32_t *bits_u, const uint32_t *bits_v, const float *h,
                       const float *l, const float *g, const float *tape_a, float gscale, float *dh, float *dl,
                       float *dg, float *dx, int accumulate_dx, float *grad_u, float *grad_v, int accumulate_signs,
                       void *workspace, size_t workspace_bytes, void *stream) {
    return backward_impl(M, d_in, d_out, r, paths, x, dy, bits_u, bits_v, h, l, g, tape_a, nullptr, gscale, dh, dl,
                         dg, dx, accumulate_dx, grad_u, grad_v, accumulate_signs, workspace, workspace_bytes, stream);
}

int blr_plane_linear(int64_t M, int64_t n, int64_t k, const float *x, const uint16_t *plane, float *y, float scale,
                     void *stream) {
    if (!x || !plane || !y) return BLR_ERR_NULL;
    if (M < 1 || n < 128 || k < 128 || n % 128 || k % 128) return BLR_ERR_SHAPE;
    const int64_t widest = n > k ? n : k;
    if (M * widest * 4 > (int64_t)0xFFFFFFFF || n * k * 2 > (int64_t)0xFFFFFFFF) return BLR_ERR_SHAPE;
    if ((n / 128) * ceil_div(M, 64) > ((int64_t)1 << 31) - 1) return BLR_ERR_SHAPE;
    if (!pow2_scale_ok(scale)) return BLR_ERR_SCALE;
    if (!aligned16(x) || !aligned16(plane) || !aligned16(y)) return BLR_ERR_ALIGN;
    int st = current_device_ok();
    if (st != BLR_OK) return st;
    GemmArgs a = {};
    a.A = x;
    a.lda = k;
    a.ascale = scale;
    a.Bplane = plane;
    a.M = M;
    a.N = (int)n;
    a.K = (int)k;
    a.oscale = 1.0f / scale;  // exact: scale is a power of two
    a.out = y;
    BLR_TRY(launch_gemm(GEMM_PLANE, a, (hipStream_t)stream));
    return BLR_OK;
}

int blr_sumsq(const float *a, int64_t n, float *partials, int nparts, void *stream) {
    if (!a || !partials) return BLR_ERR_NULL;
    if (n < 1 || nparts < 1 || nparts > 1024) return BLR_ERR_SHAPE;
    if (!aligned16(a) || !aligned4(partials)) return BLR_ERR_ALIGN;
    int st = current_device_ok();
    if (st != BLR_OK) return st;
    BLR_TRY(launch_sumsq(a, n, partials, nparts, (hipStream_t)stream));
    return BLR_OK;
}

// --------------------------------------------------------------- routing --
namespace {
constexpr int64_t MAX_POSITIONS = ((int64_t)1 << 31) - 65536;  // int32 positions, with room for a grid's tail

// An argument's memory; an output must be apart from every other argument.
struct Span {
    const void *p;
    size_t bytes;
    bool out;
};

bool apart(const Span *s, int n) {
    for (int i = 0; i < n; ++i) {
        if (!s[i].out || !s[i].p) continue;
        const uintptr_t lo = (uintptr_t)s[i].p, hi = lo + s[i].bytes;
        for (int j = 0; j < n; ++j) {
            if (j == i || !s[j].p) continue;
            const uintptr_t l = (uintptr_t)s[j].p;
            if (l < hi && lo < l + s[j].bytes) return false;
        }
    }
    return true;
}

size_t size_of(int dtype) { return dtype == BLR_F32 ? 4 : 2; }

bool dtype_ok(int t) { return t == BLR_F32 || t == BLR_F16 || t == BLR_BF16; }

bool route_shape_ok(int64_t pairs, int64_t experts) {
    return pairs >= 1 && pairs < MAX_POSITIONS && experts >= 1 && experts <= ROUTE_MAX_EXPERTS;
}

// Checks that the three row calls share; T k is formed only once k is known to be small.
int route_rows_check(int64_t T, int64_t k, int64_t experts, int64_t d, int dtype, const void *a,
                     const int32_t *offsets, const int32_t *slot, const void *out) {
    if (!a || !offsets || !slot || !out) return BLR_ERR_NULL;
    if (!dtype_ok(dtype)) return BLR_ERR_DTYPE;
    if (T < 1 || T >= MAX_POSITIONS || k < 1 || k > 1024 || !route_shape_ok(T * k, experts)) return BLR_ERR_SHAPE;
    if (d < 8 || d % 8 || d > ((int64_t)1 << 20)) return BLR_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(out) || !aligned4(offsets) || !aligned4(slot)) return BLR_ERR_ALIGN;
    return BLR_OK;
}
}  // namespace

size_t blr_route_workspace_bytes(int64_t pairs, int64_t experts) {
    if (!route_shape_ok(pairs, experts)) return 0;
    return up((size_t)(route_ranges(pairs, nullptr) * (experts + 1)) * 4);
}

int blr_route_sort(int64_t pairs, int64_t experts, const int32_t *ids, int32_t *offsets, int32_t *order,
                   int32_t *slot, void *workspace, size_t workspace_bytes, void *stream) {
    if (!ids || !offsets || !order || !slot) return BLR_ERR_NULL;
    if (!route_shape_ok(pairs, experts)) return BLR_ERR_SHAPE;
    int64_t per = 0;
    const int64_t ranges = route_ranges(pairs, &per);
    const size_t need = ranges > 1 ? blr_route_workspace_bytes(pairs, experts) : 0;
    if (workspace_bytes < need || (need && workspace == nullptr)) return BLR_ERR_WORKSPACE;
    if (!aligned4(ids) || !aligned4(offsets) || !aligned4(order) || !aligned4(slot) || !aligned16(workspace))
        return BLR_ERR_ALIGN;
    const size_t list = (size_t)pairs * 4;
    const Span spans[] = {{ids, list, false}, {offsets, (size_t)(experts + 1) * 4, true}, {order, list, true},
                          {slot, list, true}, {need ? workspace : nullptr, need, true}};
    if (!apart(spans, 5)) return BLR_ERR_OVERLAP;
    int st = current_device_ok();
    if (st != BLR_OK) return st;
    RouteSortArgs a = {};
    a.ranges = (int)ranges;
    a.per_range = (int)per;
    a.ids = ids;
    a.offsets = offsets;
    a.order = order;
    a.slot = slot;
    a.counts = (uint32_t *)workspace;
    a.pairs = (int)pairs;
    a.experts = (int)experts;
    BLR_TRY(launch_route_sort(a, (hipStream_t)stream));
    return BLR_OK;
}

int blr_route_gather(int64_t T, int64_t k, int64_t experts, int64_t d, int dtype, const void *x,
                     const int32_t *offsets, const int32_t *slot, void *rows, void *stream) {
    int st = route_rows_check(T, k, experts, d, dtype, x, offsets, slot, rows);
    if (st != BLR_OK) return st;
    const size_t row = (size_t)d * size_of(dtype), list = (size_t)(T * k) * 4;
    const Span spans[] = {{x, T * row, false}, {offsets, (size_t)(experts + 1) * 4, false}, {slot, list, false},
                          {rows, T * k * row, true}};
    if (!apart(spans, 4)) return BLR_ERR_OVERLAP;
    st = current_device_ok();
    if (st != BLR_OK) return st;
    RouteRows a = {};
    a.placed = offsets + experts;
    a.slot = slot;
    a.a = x;
    a.out = rows;
    a.T = T;
    a.d = d;
    a.k = (int)k;
    a.dtype = dtype;
    BLR_TRY(launch_route_gather(a, (hipStream_t)stream));
    return BLR_OK;
}

int blr_route_combine(int64_t T, int64_t k, int64_t experts, int64_t d, int dtype, const void *z,
                      const int32_t *offsets, const int32_t *slot, const float *weights, void *y, int accumulate_y,
                      void *stream) {
    int st = route_rows_check(T, k, experts, d, dtype, z, offsets, slot, y);
    if (st != BLR_OK) return st;
    if (!aligned4(weights)) return BLR_ERR_ALIGN;
    const size_t row = (size_t)d * size_of(dtype), list = (size_t)(T * k) * 4;
    const Span spans[] = {{z, T * k * row, false}, {offsets, (size_t)(experts + 1) * 4, false}, {slot, list, false},
                          {weights, list, false}, {y, T * row, true}};
    if (!apart(spans, 5)) return BLR_ERR_OVERLAP;
    st = current_device_ok();
    if (st != BLR_OK) return st;
    RouteRows a = {};
    a.placed = offsets + experts;
    a.slot = slot;
    a.weights = weights;
    a.a = z;
    a.out = y;
    a.T = T;
    a.d = d;
    a.k = (int)k;
    a.dtype = dtype;
    a.acc = accumulate_y ? 1 : 0;
    BLR_TRY(launch_route_combine(a, (hipStream_t)stream));
    return BLR_OK;
}

int blr_route_combine_backward(int64_t T, int64_t k, int64_t experts, int64_t d, int dtype, const void *dy,
                               const void *z, const int32_t *offsets, const int32_t *slot, const float *weights,
                               void *dz, float *dw, void *stream) {
    if (dw && !z) return BLR_ERR_NULL;
    int st = route_rows_check(T, k, experts, d, dtype, dy, offsets, slot, dz);
    if (st != BLR_OK) return st;
    if (!aligned16(z) || !aligned4(weights) || !aligned4(dw)) return BLR_ERR_ALIGN;
    const size_t row = (size_t)d * size_of(dtype), list = (size_t)(T * k) * 4;
    const Span spans[] = {{dy, T * row, false}, {z, T * k * row, false}, {offsets, (size_t)(experts + 1) * 4, false},
                          {slot, list, false}, {weights, list, false}, {dz, T * k * row, true}, {dw, list, true}};
    if (!apart(spans, 7)) return BLR_ERR_OVERLAP;
    st = current_device_ok();
    if (st != BLR_OK) return st;
    RouteRows a = {};
    a.placed = offsets + experts;
    a.slot = slot;
    a.weights = weights;
    a.a = dy;
    a.z = z;
    a.out = dz;
    a.dw = dw;
    a.T = T;
    a.d = d;
    a.k = (int)k;
    a.dtype = dtype;
    BLR_TRY(launch_route_combine_backward(a, (hipStream_t)stream));
    return BLR_OK;
}

// -------------------------------------------------------------- adapters --
namespace {
bool adapt_shape_ok(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t E) {
    const int64_t D = (int64_t)1 << 20;
    return M >= 1 && M < MAX_POSITIONS && d_in >= 128 && d_in <= D && d_in % 128 == 0 && d_out >= 128 && d_out <= D &&
           d_out % 128 == 0 && r >= 8 && r <= ADAPT_MAX_RANK && r % 8 == 0 && E >= 1 && E <= ROUTE_MAX_EXPERTS;
}

// Workspace: the splits' partials of s or ds (f32 [splits][M][r]), then for
// the backward the transposes of down and up, the panels of ds and of the tape
// and the ranges' partials of both gradients.
struct AdaptLayout {
    size_t down_t, up_t, panel[2], part[2], total;
    int64_t range, slots;
};

AdaptLayout adapt_layout(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t E) {
    AdaptLayout L;
    const int si = adapt_splits(M, E, d_in), so = adapt_splits(M, E, d_out);
    size_t off = up((size_t)(si > so ? si : so) * M * r * 4);
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += up(bytes);
        return at;
    };
    // sized for the widest types, so that one workspace serves them all
    L.down_t = take((size_t)E * r * d_in * 4);
    L.up_t = take((size_t)E * r * d_out * 4);
    const size_t panels = (size_t)adapt_tiles(M, E, ADAPT_TM) * adapt_panel_bytes(r, BLR_BF16);
    L.panel[0] = take(panels);
    L.panel[1] = take(panels);
    L.range = adapt_range(M, d_in, d_out, r);
    L.slots = adapt_range_slots(M, E, L.range);
    L.part[0] = take((size_t)L.slots * r * d_in * 4);
    L.part[1] = take((size_t)L.slots * r * d_out * 4);
    L.total = off;
    return L;
}

// What the forward needs: the splits' partials of s. Up to a megabyte a buffer
// for both calls costs nobody anything, so below that the two sizes are one.
size_t adapt_forward_bytes(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t E) {
    const size_t own = up((size_t)adapt_splits(M, E, d_in) * M * r * 4), least = (size_t)1 << 20;
    const size_t both = adapt_layout(M, d_in, d_out, r, E).total;
    return own > least ? own : both < least ? both : least;
}

// Checks that both calls share.
int adapt_check(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t E, int act, int wt, const void *down,
                const void *up_, const int32_t *offsets, const int32_t *order, const float *scale,
                const void *workspace, size_t workspace_bytes, bool forward, size_t *need) {
    if (!down || !up_ || !offsets) return BLR_ERR_NULL;
    if (!dtype_ok(act) || !dtype_ok(wt) || (act != BLR_F32 && wt != act)) return BLR_ERR_DTYPE;
    if (!adapt_shape_ok(M, d_in, d_out, r, E)) return BLR_ERR_SHAPE;
    // whatever wt is
    *need = forward ? adapt_forward_bytes(M, d_in, d_out, r, E) : adapt_layout(M, d_in, d_out, r, E).total;
    if (workspace == nullptr || workspace_bytes < *need) return BLR_ERR_WORKSPACE;
    if (!aligned16(down) || !aligned16(up_) || !aligned4(offsets) || !aligned4(order) || !aligned4(scale) ||
        !aligned16(workspace))
        return BLR_ERR_ALIGN;
    return BLR_OK;
}
}  // namespace

size_t blr_adapters_workspace_bytes(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t adapters) {
    if (!adapt_shape_ok(M, d_in, d_out, r, adapters)) return 0;
    return adapt_layout(M, d_in, d_out, r, adapters).total;
}

size_t blr_adapters_forward_workspace_bytes(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t adapters) {
    if (!adapt_shape_ok(M, d_in, d_out, r, adapters)) return 0;
    return adapt_forward_bytes(M, d_in, d_out, r, adapters);
}

int blr_adapters_forward(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t adapters, int act, int wt,
                         const void *x, const void *down, const void *up, const int32_t *offsets,
                         const int32_t *order, const float *scale, void *y, int accumulate_y, float *tape_s,
                         void *workspace, size_t workspace_bytes, void *stream) {
    if (!x || !y) return BLR_ERR_NULL;
    size_t need = 0;
    int st = adapt_check(M, d_in, d_out, r, adapters, act, wt, down, up, offsets, order, scale, workspace,
                         workspace_bytes, true, &need);
    if (st != BLR_OK) return st;
    if (!aligned16(x) || !aligned16(y) || !aligned16(tape_s)) return BLR_ERR_ALIGN;
    const size_t a = size_of(act), w = (size_t)adapters * r * size_of(wt);
    const Span spans[] = {{x, M * d_in * a, false}, {down, w * d_in, false}, {up, w * d_out, false},
                          {offsets, (size_t)(adapters + 1) * 4, false}, {order, (size_t)M * 4, false},
                          {scale, (size_t)adapters * 4, false}, {y, M * d_out * a, true},
                          {tape_s, (size_t)M * r * 4, true}, {workspace, need, true}};
    if (!apart(spans, 9)) return BLR_ERR_OVERLAP;
    st = current_device_ok();
    if (st != BLR_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    AdaptShrink sh = {};
    sh.plan = {offsets, order, (int)M, (int)adapters};
    sh.X = x;
    sh.W = down;
    sh.part = (float *)workspace;
    sh.K = (int)d_in;
    sh.r = (int)r;
    sh.splits = adapt_splits(M, adapters, d_in);
    sh.act = act;
    sh.wt = wt;
    AdaptExpand ex = {};
    ex.plan = sh.plan;
    ex.part = sh.part;
    ex.scale = scale;
    ex.W = up;
    ex.out = y;
    ex.s_row = tape_s;
    ex.N = (int)d_out;
    ex.r = (int)r;
    ex.splits = sh.splits;
    ex.act = act;
    ex.wt = wt;
    ex.acc = accumulate_y ? 1 : 0;
    BLR_TRY(launch_adapt_shrink(sh, K_ADAPT_DOWN, s));
    BLR_TRY(launch_adapt_expand(ex, K_ADAPT_UP, s));
    return BLR_OK;
}

int blr_adapters_backward(int64_t M, int64_t d_in, int64_t d_out, int64_t r, int64_t adapters, int act, int wt,
                          const void *x, const void *dy, const void *down, const void *up, const int32_t *offsets,
                          const int32_t *order, const float *scale, const float *tape_s, float *grad_down,
                          float *grad_up, int accumulate_grads, void *dx, int accumulate_dx, void *workspace,
                          size_t workspace_bytes, void *stream) {
    if (!dy || (grad_down == nullptr) != (grad_up == nullptr) || (!grad_down && !dx)) return BLR_ERR_NULL;
    if (grad_down && (!x || !tape_s)) return BLR_ERR_NULL;
    size_t need = 0;
    int st = adapt_check(M, d_in, d_out, r, adapters, act, wt, down, up, offsets, order, scale, workspace,
                         workspace_bytes, false, &need);
    if (st != BLR_OK) return st;
    const void *arrays[] = {x, dy, tape_s, grad_down, grad_up, dx};
    for (const void *p : arrays)
        if (!aligned16(p)) return BLR_ERR_ALIGN;
    const size_t a = size_of(act), w = (size_t)adapters * r;
    const Span spans[] = {{x, M * d_in * a, false}, {dy, M * d_out * a, false}, {down, w * d_in * size_of(wt), false},
                          {up, w * d_out * size_of(wt), false}, {offsets, (size_t)(adapters + 1) * 4, false},
                          {order, (size_t)M * 4, false}, {scale, (size_t)adapters * 4, false},
                          {tape_s, (size_t)M * r * 4, false}, {grad_down, w * d_in * 4, true},
                          {grad_up, w * d_out * 4, true}, {dx, M * d_in * a, true}, {workspace, need, true}};
    if (!apart(spans, 12)) return BLR_ERR_OVERLAP;
    st = current_device_ok();
    if (st != BLR_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    const AdaptLayout L = adapt_layout(M, d_in, d_out, r, adapters);
    char *ws = (char *)workspace;
    AdaptPrepare pr = {};
    pr.plan = {offsets, order, (int)M, (int)adapters};
    pr.src[0] = down;
    pr.dst[0] = ws + L.down_t;
    pr.rows[0] = (int)r;
    pr.cols[0] = (int)d_in;
    pr.src[1] = up;
    pr.dst[1] = ws + L.up_t;
    pr.rows[1] = (int)d_out;
    pr.cols[1] = (int)r;
    pr.tape = grad_down ? tape_s : nullptr;
    pr.panel = ws + L.panel[1];
    pr.grad[0] = accumulate_grads ? nullptr : grad_down;
    pr.grad[1] = accumulate_grads ? nullptr : grad_up;
    pr.r = (int)r;
    pr.act = act;
    pr.wt = wt;
    BLR_TRY(launch_adapt_prepare(pr, s));
    // ds = c dy B: the contraction over d_out, then its splits' sum with dx
    AdaptShrink sh = {};
    sh.plan = pr.plan;
    sh.X = dy;
    sh.W = pr.dst[1];
    sh.part = (float *)ws;
    sh.K = (int)d_out;
    sh.r = (int)r;
    sh.splits = adapt_splits(M, adapters, d_out);
    sh.act = act;
    sh.wt = wt;
    AdaptExpand ex = {};
    ex.plan = sh.plan;
    ex.part = sh.part;
    ex.scale = scale;
    ex.W = pr.dst[0];
    ex.out = dx;
    ex.N = (int)d_in;
    ex.r = (int)r;
    ex.splits = sh.splits;
    ex.act = act;
    ex.wt = wt;
    ex.acc = accumulate_dx ? 1 : 0;
    if (!grad_down) {
        BLR_TRY(launch_adapt_shrink(sh, K_ADAPT_DS, s));
        BLR_TRY(launch_adapt_expand(ex, K_ADAPT_DX, s));
        return BLR_OK;
    }
    AdaptGrad gr = {};
    gr.plan = sh.plan;
    gr.r = (int)r;
    gr.act = act;
    gr.acc = accumulate_grads ? 1 : 0;
    gr.panels = adapt_tiles(M, adapters, ADAPT_TM);
    gr.range = (int)L.range;
    gr.slots = L.slots;
    void *ds_panel = ws + L.panel[0];
    gr.job[0] = {x, ds_panel, nullptr, grad_down, (float *)(ws + L.part[0]), (int)d_in};
    gr.job[1] = {dy, pr.panel, scale, grad_up, (float *)(ws + L.part[1]), (int)d_out};
    BLR_TRY(launch_adapt_dy(sh, gr, s));
    AdaptThin th = {sh.plan, sh.part, scale, ds_panel, (int)r, sh.splits, act};
    BLR_TRY(launch_adapt_thin(th, s));
    BLR_TRY(launch_adapt_dx(ex, gr, s));
    if (L.slots > 0) BLR_TRY(launch_adapt_reduce(gr, s));  // otherwise no adapter can have several ranges
    return BLR_OK;
}

// ---------------------------------------------------- norms, checkpoints --
namespace {
constexpr int64_t MAX_WIDTH = (int64_t)1 << 20;

bool rows_ok(int64_t M) { return M >= 1 && M < MAX_POSITIONS; }

int checkpoint(int64_t M, int64_t d, int dtype, const void *x, const int8_t *q, const uint8_t *b, bool save,
               void *stream) {
    if (!x || !q || !b) return BLR_ERR_NULL;
    if (!dtype_ok(dtype)) return BLR_ERR_DTYPE;
    if (!rows_ok(M) || d < 32 || d % 32 || d > MAX_WIDTH) return BLR_ERR_SHAPE;
    if (!aligned16(x) || !aligned16(q)) return BLR_ERR_ALIGN;
    const size_t n = (size_t)(M * d);
    const Span spans[] = {{x, n * size_of(dtype), !save}, {q, n, save}, {b, n / 32, save}};
    if (!apart(spans, 3)) return BLR_ERR_OVERLAP;
    const int st = current_device_ok();
    if (st != BLR_OK) return st;
    const Checkpoint a = {const_cast<void *>(x), const_cast<int8_t *>(q), const_cast<uint8_t *>(b), (int64_t)n, dtype};
    BLR_TRY(launch_checkpoint(a, save, (hipStream_t)stream));
    return BLR_OK;
}

bool norm_shape_ok(int64_t M, int64_t d, int64_t span) {
    return rows_ok(M) && d >= 8 && d % 8 == 0 && d <= NORM_MAX_D && span >= 1;
}

bool norm_types_ok(int xt, int ft, int nt) {
    return dtype_ok(xt) && dtype_ok(ft) && dtype_ok(nt) && (xt == BLR_F32 || (ft == xt && nt == xt));
}

// Sums of workgroups: of dw, of dw_after; of ranges, two gates' parts, where
// rows share gates.
struct NormLayout {
    size_t part_a, part_z, total;
    NormSplit split;
};
NormLayout norm_layout(int64_t M, int64_t d, int64_t span) {
    NormLayout L;
    L.split = norm_split(M, d);
    L.part_a = up((size_t)(L.split.blocks * d) * 4);
    L.part_z = 2 * L.part_a;
    L.total = L.part_z + (span > 1 ? up((size_t)(2 * L.split.ranges * d) * 4) : 0);
    return L;
}

// `a` all aligned to 16 bytes, and every output apart from the rest and from `more`.
int arrays_ok(const Span *a, int n, const Span *more, int extra) {
    Span spans[24];
    for (int i = 0; i < n; ++i) {
        if (!aligned16(a[i].p)) return BLR_ERR_ALIGN;
        spans[i] = a[i];
    }
    for (int i = 0; i < extra; ++i) spans[n + i] = more[i];
    return apart(spans, n + extra) ? BLR_OK : BLR_ERR_OVERLAP;
}
}  // namespace

int blr_checkpoint_save(int64_t M, int64_t d, int dtype, const void *x, int8_t *q, uint8_t *b, void *stream) {
    return checkpoint(M, d, dtype, x, q, b, true, stream);
}

int blr_checkpoint_load(int64_t M, int64_t d, int dtype, const int8_t *q, const uint8_t *b, void *x, void *stream) {
    return checkpoint(M, d, dtype, x, q, b, false, stream);
}

int blr_norm_forward(int64_t M, int64_t d, int xt, int ft, int nt, const void *x, const void *f, int norm_f,
                     const float *w_after, const void *gate, int gate_kind, int64_t span, float skip, float scale,
                     const float *w, float eps, void *out, void *n, float *stats, int8_t *q, uint8_t *b,
                     void *stream) {
    if (!x || (f == nullptr) != (out == nullptr) || (q == nullptr) != (b == nullptr)) return BLR_ERR_NULL;
    if (!f && !n && !stats && !q) return BLR_ERR_NULL;
    if (!norm_types_ok(xt, ft, nt) || gate_kind < BLR_GATE_LINEAR || gate_kind > BLR_GATE_SILU) return BLR_ERR_DTYPE;
    if (!norm_shape_ok(M, d, span) || (q && d % 32)) return BLR_ERR_SHAPE;
    if (!(eps >= 0.0f) || !isfinite(eps)) return BLR_ERR_SCALE;
    if (!aligned4(stats)) return BLR_ERR_ALIGN;
    if (!f) w_after = nullptr, gate = nullptr, norm_f = 0;
    if (span > M) span = M;
    const size_t rows = (size_t)(M * d), col = (size_t)d * 4;
    const Span arrays[] = {{x, rows * size_of(xt), false}, {f, rows * size_of(ft), false},
                            {gate, (size_t)(ceil_div(M, span) * d) * size_of(ft), false}, {w_after, col, false},
                            {w, col, false}, {out, rows * size_of(xt), true}, {n, rows * size_of(nt), true},
                            {q, rows, true}};
    const Span more[] = {{stats, (size_t)M * 8, true}, {b, rows / 32, true}};
    int st = arrays_ok(arrays, 8, more, 2);
    if (st != BLR_OK) return st;
    st = current_device_ok();
    if (st != BLR_OK) return st;
    NormForward a = {};
    a.x = x;
    a.f = f;
    a.gate = gate;
    a.w_after = w_after;
    a.w = w;
    a.out = out;
    a.n = n;
    a.stats = stats;
    a.q = q;
    a.b = b;
    a.M = M;
    a.d = d;
    a.span = (uint32_t)span;
    a.xt = xt;
    a.ft = ft;
    a.nt = nt;
    a.gate_kind = gate_kind;
    a.norm_f = norm_f ? 1 : 0;
    a.skip = skip;
    a.scale = scale;
    a.eps = eps;
    BLR_TRY(launch_norm_forward(a, (hipStream_t)stream));
    return BLR_OK;
}

size_t blr_norm_workspace_bytes(int64_t M, int64_t d, int64_t span) {
    return norm_shape_ok(M, d, span) ? norm_layout(M, d, span).total : 0;
}

int blr_norm_backward(int64_t M, int64_t d, int xt, int ft, int nt, const void *dn, const void *dout, const void *out,
                      const int8_t *out_q, const uint8_t *out_b, int has_f, const void *f, const int8_t *f_q,
                      const uint8_t *f_b, int norm_f, const float *w_after, const void *gate, int gate_kind,
                      int64_t span, float skip, float scale, const float *w, const float *stats, void *dx, void *df,
                      void *dgate, float *dw, float *dw_after, int accumulate_grads, void *workspace,
                      size_t workspace_bytes, void *stream) {
    if (!has_f) {
        // f's arguments mean nothing, and none of its gradients can be asked for
        if (df || dgate || dw_after) return BLR_ERR_NULL;
        f = f_q = nullptr, f_b = nullptr, norm_f = 0, w_after = nullptr, gate = nullptr, skip = 1.0f;
    }
    if ((out_q == nullptr) != (out_b == nullptr) || (f_q == nullptr) != (f_b == nullptr)) return BLR_ERR_NULL;
    if ((out && out_q) || (f && f_q)) return BLR_ERR_NULL;  // one form or the other
    if ((!dn && !dout) || (dn && !out && !out_q) || (dw && !dn) || (dgate && !gate)) return BLR_ERR_NULL;
    const bool need_f = has_f && (norm_f || dw_after || dgate);
    if (need_f && !f && !f_q) return BLR_ERR_NULL;
    if ((dn || norm_f) && !stats) return BLR_ERR_NULL;
    if (!dx && !df && !dgate && !dw && !dw_after) return BLR_ERR_NULL;
    if (!norm_types_ok(xt, ft, nt) || gate_kind < BLR_GATE_LINEAR || gate_kind > BLR_GATE_SILU) return BLR_ERR_DTYPE;
    if (!norm_shape_ok(M, d, span) || ((out_q || f_q) && d % 32)) return BLR_ERR_SHAPE;
    const NormLayout L = norm_layout(M, d, span);
    if (workspace == nullptr || workspace_bytes < L.total) return BLR_ERR_WORKSPACE;
    if (!aligned4(stats)) return BLR_ERR_ALIGN;
    const bool summed = span > 1;
    if (span > M) span = M;
    const size_t rows = (size_t)(M * d), col = (size_t)d * 4, x_size = rows * size_of(xt), f_size = rows * size_of(ft);
    const size_t gates = (size_t)(ceil_div(M, span) * d);
    const Span arrays[] = {{dn, rows * size_of(nt), false}, {dout, x_size, false}, {out, x_size, false},
                            {out_q, rows, false}, {f, f_size, false}, {f_q, rows, false},
                            {gate, gates * size_of(ft), false}, {w_after, col, false}, {w, col, false},
                            {dx, x_size, true}, {df, f_size, true}, {dgate, gates * (summed ? 4 : size_of(ft)), true},
                            {dw, col, true}, {dw_after, col, true}, {workspace, L.total, true}};
    const Span more[] = {{stats, (size_t)M * 8, false}, {out_b, rows / 32, false}, {f_b, rows / 32, false}};
    int st = arrays_ok(arrays, 15, more, 3);
    if (st != BLR_OK) return st;
    st = current_device_ok();
    if (st != BLR_OK) return st;
    NormBackward a = {};
    a.dn = dn;
    a.dout = dout;
    a.out = dn ? out : nullptr;
    a.out_q = out_q;
    a.out_b = out_b;
    a.f = f;
    a.f_q = f_q;
    a.f_b = f_b;
    a.gate = gate;
    a.w = w;
    a.w_after = w_after;
    a.stats = stats;
    a.dx = dx;
    a.df = df;
    a.dgate = dgate;
    a.dw = dw;
    a.dw_after = dw_after;
    a.part_w = (float *)workspace;
    a.part_a = (float *)((char *)workspace + L.part_a);
    a.part_z = (float *)((char *)workspace + L.part_z);
    a.M = M;
    a.d = d;
    a.per = L.split.per;
    a.ranges = L.split.ranges;
    a.blocks = L.split.blocks;
    a.span = (uint32_t)span;
    a.xt = xt;
    a.ft = ft;
    a.nt = nt;
    a.gate_kind = gate_kind;
    a.norm_f = norm_f ? 1 : 0;
    a.acc = accumulate_grads ? 1 : 0;
    a.need_f = need_f;
    a.summed = summed;
    a.skip = skip;
    a.scale = has_f ? scale : 0.0f;
    BLR_TRY(launch_norm_backward(a, (hipStream_t)stream));
    return BLR_OK;
}

// ---------------------------------------------------- gated feed-forward --
namespace {
bool gated_shape_ok(int64_t M, int64_t d, int64_t ff) {
    const int64_t most = (int64_t)1 << 24;  // tiles of 256 threads: a grid has room for 2^32
    return rows_ok(M) && d >= 128 && d % 128 == 0 && d <= MAX_WIDTH && ff >= 128 && ff % 128 == 0 && ff <= MAX_WIDTH &&
           ceil_div(M, 128) * (ff / 64) < most && ceil_div(M, 128) * (d / 128) < most;
}
// dg and du side by side, x out of its checkpoint, the sums of dx's splits.
struct GatedLayout {
    size_t rows, part, total;
};
GatedLayout gated_layout(int64_t M, int64_t d, int64_t ff) {
    GatedLayout L;
    int64_t steps;
    const int64_t splits = gated_splits(M, d, 2 * ff, &steps);
    L.rows = up((size_t)(M * ff) * 4);
    L.part = L.rows + up((size_t)(M * d) * 2);
    L.total = L.part + (splits > 1 ? up((size_t)(splits * M * d) * 4) : 0);
    return L;
}
bool half_type(int t) { return t == BLR_F16 || t == BLR_BF16; }
}  // namespace

int blr_gated_forward(int64_t M, int64_t d, int64_t ff, int dtype, int ht, const void *x, const void *w_gate,
                      const void *w_up, int act, void *h, int8_t *tape_q, uint8_t *tape_b, void *stream) {
    if (!x || !w_gate || !w_up || !h || (tape_q == nullptr) != (tape_b == nullptr)) return BLR_ERR_NULL;
    if (!half_type(dtype) || (ht != dtype && ht != BLR_F32) || act < BLR_ACT_SILU || act > BLR_ACT_GELU)
        return BLR_ERR_DTYPE;
    if (!gated_shape_ok(M, d, ff)) return BLR_ERR_SHAPE;
    const size_t w = (size_t)(ff * d) * 2, mid = (size_t)(M * ff);
    const Span arrays[] = {{x, (size_t)(M * d) * 2, false}, {w_gate, w, false}, {w_up, w, false},
                           {h, mid * size_of(ht), true}, {tape_q, 2 * mid, true}};
    const Span more[] = {{tape_b, mid / 16, true}};
    int st = arrays_ok(arrays, 5, more, 1);
    if (st != BLR_OK) return st;
    st = current_device_ok();
    if (st != BLR_OK) return st;
    GatedGemm a = {};
    a.A = x;
    a.B = w_gate;
    a.B2 = w_up;
    a.out = h;
    a.tape_q = tape_q;
    a.tape_b = tape_b;
    a.M = M;
    a.K = d;
    a.lda = d;
    a.ldb = d;
    a.ff = ff;
    a.dtype = dtype;
    a.kind = act;
    a.out_f32 = ht == BLR_F32;
    BLR_TRY(launch_gated_forward(a, (hipStream_t)stream));
    return BLR_OK;
}

size_t blr_gated_workspace_bytes(int64_t M, int64_t d, int64_t ff) {
    return gated_shape_ok(M, d, ff) ? gated_layout(M, d, ff).total : 0;
}

int blr_gated_backward(int64_t M, int64_t d, int64_t ff, int dtype, int ht, int gt, const void *x, const int8_t *x_q,
                       const uint8_t *x_b, const void *dh, const void *w_gate, const void *w_up, int act,
                       const int8_t *tape_q, const uint8_t *tape_b, float gscale, void *dx, int accumulate_dx,
                       void *dw_gate, void *dw_up, int accumulate_grads, void *workspace, size_t workspace_bytes,
                       void *stream) {
    if (!dh || !w_gate || !w_up || (tape_q == nullptr) != (tape_b == nullptr) || (x_q == nullptr) != (x_b == nullptr) ||
        (x && x_q) || (dw_gate == nullptr) != (dw_up == nullptr) || (!dx && !dw_gate))
        return BLR_ERR_NULL;
    if ((dw_gate || !tape_q) && !x && !x_q) return BLR_ERR_NULL;
    if (!half_type(dtype) || (ht != dtype && ht != BLR_F32) || (gt != dtype && gt != BLR_F32) || act < BLR_ACT_SILU ||
        act > BLR_ACT_GELU)
        return BLR_ERR_DTYPE;
    if (!gated_shape_ok(M, d, ff)) return BLR_ERR_SHAPE;
    if (!pow2_scale_ok(gscale)) return BLR_ERR_SCALE;
    const GatedLayout L = gated_layout(M, d, ff);
    const size_t need = L.total;
    if (workspace == nullptr || workspace_bytes < need) return BLR_ERR_WORKSPACE;
    const size_t n = (size_t)(ff * d), mid = (size_t)(M * ff), rows = (size_t)(M * d);
    const Span arrays[] = {{x, rows * 2, false}, {x_q, rows, false}, {dh, mid * size_of(ht), false},
                           {w_gate, n * 2, false}, {w_up, n * 2, false}, {tape_q, 2 * mid, false}, {dx, rows * 2, true},
                           {dw_gate, n * size_of(gt), true}, {dw_up, n * size_of(gt), true}, {workspace, need, true}};
    const Span more[] = {{x_b, rows / 32, false}, {tape_b, mid / 16, false}};
    int st = arrays_ok(arrays, 10, more, 2);
    if (st != BLR_OK) return st;
    st = current_device_ok();
    if (st != BLR_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    if (x_q && (dw_gate || !tape_q)) {
        void *rows_x = (char *)workspace + L.rows;
        const Checkpoint c = {rows_x, const_cast<int8_t *>(x_q), const_cast<uint8_t *>(x_b), M * d, dtype};
        BLR_TRY(launch_checkpoint(c, false, s));
        x = rows_x;
    }
    GatedGemm a = {};
    a.dtype = dtype;
    a.kind = act;
    a.ff = ff;
    // dg and du times gscale
    GatedGemm g = a;
    g.A = x;
    g.B = w_gate;
    g.B2 = w_up;
    g.dh = dh;
    g.out = workspace;
    g.tape_q = const_cast<int8_t *>(tape_q);
    g.tape_b = const_cast<uint8_t *>(tape_b);
    g.M = M;
    g.K = d;
    g.lda = d;
    g.ldb = d;
    g.out_f32 = ht == BLR_F32;
    g.scale = gscale;
    BLR_TRY(tape_q ? launch_gated_gradients(g, s) : launch_gated_again(g, s));
    a.scale = 1.0f / gscale;
    a.N = (int)d;
    a.A = workspace;
    a.lda = 2 * ff;
    a.ldb = d;
    if (dx) {
        GatedGemm v = a;
        v.B = w_gate;
        v.B2 = w_up;
        v.out = dx;
        v.M = M;
        v.K = 2 * ff;
        v.part = (float *)((char *)workspace + L.part);
        v.acc = accumulate_dx ? 1 : 0;
        BLR_TRY(launch_gated_dx(v, s));
    }
    if (dw_gate) {
        a.B = a.B2 = x;
        a.out = dw_gate;
        a.out2 = dw_up;
        a.M = 2 * ff;
        a.K = M;
        a.out_f32 = gt == BLR_F32;
        a.acc = accumulate_grads ? 1 : 0;
        BLR_TRY(launch_gated_dw(a, s));
    }
    return BLR_OK;
}

int blr_profile_enable(int max_launches) {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    prof_release();
    if (max_launches <= 0) return BLR_OK;
    g_prof.ev.resize(2 * (size_t)max_launches);
    for (size_t i = 0; i < g_prof.ev.size(); ++i) {
        if (hipEventCreate(&g_prof.ev[i]) != hipSuccess) {
            g_prof.ev.resize(i);
            prof_release();
            return BLR_ERR_HIP;
        }
    }
    g_prof.on = true;
    return BLR_OK;
}

int blr_profile_read(const char **names, int64_t *counts, double *total_ms, int max) {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    for (size_t q = 0; q < g_prof.used; ++q) {
        if (hipEventSynchronize(g_prof.ev[2 * q + 1]) != hipSuccess) return BLR_ERR_HIP;
        float ms = 0.0f;
        if (hipEventElapsedTime(&ms, g_prof.ev[2 * q], g_prof.ev[2 * q + 1]) != hipSuccess) return BLR_ERR_HIP;
        g_prof.counts[g_prof.ids[q]] += 1;
        g_prof.total_ms[g_prof.ids[q]] += ms;
    }
    g_prof.used = 0;
    g_prof.ids.clear();
    int n = 0;
    for (int id = 0; id < K_COUNT; ++id) {
        if (g_prof.counts[id] == 0) continue;
        if (n < max) {
            if (names) names[n] = kernel_name(id);
            if (counts) counts[n] = g_prof.counts[id];
            if (total_ms) total_ms[n] = g_prof.total_ms[id];
        }
        ++n;
    }
    return n;
}

int blr_profile_reset(void) {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    for (int id = 0; id < K_COUNT; ++id) {
        g_prof.counts[id] = 0;
        g_prof.total_ms[id] = 0.0;
    }
    return BLR_OK;
}

}  // extern "C"
