// Low-rank adapters: the backward with the adapters' gradients. Each of its two
// large launches pairs a contraction with the gradient beside it:
//
//   dy   ds = c dy B and dB, which both read dy: their workgroups take the rows
//        in the same order, so that of a small dy the second read finds the
//        last-level cache
//   dx   dx = ds A, which writes, and dA, whose read of x is the only one
//
// 8192 x 4096 -> 4096 f32, rank 16: 58 + 64 us; 30000 x 5120 -> 17408 bf16, rank
// 64: 425 + 196 us. Reads bound the first: dy passes twice, with the weights of
// every tile of 64 rows 2.7 GB of reads, 2 GB of them dy.
#include "blr_adapters.h"

namespace blr {

namespace {

// --------------------------------------------------------------- prepare --
// The backward's first launch; each workgroup does one of three things.
//
// Transpose: the backward contracts over the other side of A and B than the
// forward, so both are laid out transposed, 64 x 64 elements at a time through
// LDS; then every weight is read 16 consecutive bytes a lane, as in the
// forward. Adapters without rows are left out.
template <typename T>
__device__ void transpose_tile(const AdaptPrepare &a, int job, int e, int b, T (*tile)[64 + 16 / sizeof(T)]) {
    constexpr int n = 16 / sizeof(T);
    typedef T V __attribute__((ext_vector_type(n)));
    const int R = a.rows[job], C = a.cols[job], across = (C + 63) / 64;
    const int r0 = b / across * 64, c0 = b % across * 64;
    const T *src = reinterpret_cast<const T *>(a.src[job]) + (int64_t)e * R * C;
    T *dst = reinterpret_cast<T *>(a.dst[job]) + (int64_t)e * R * C;
    constexpr int per = 64 / n;  // vectors of a tile's row
    for (int i = threadIdx.x; i < 64 * per; i += 256) {
        const int r = i / per, c = i % per * n;
        if (r0 + r < R && c0 + c < C)  // R and C are multiples of 8
            *reinterpret_cast<V *>(&tile[r][c]) = *reinterpret_cast<const V *>(src + (int64_t)(r0 + r) * C + c0 + c);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * per; i += 256) {
        const int c = i / per, r = i % per * n;
        if (r0 + r < R && c0 + c < C) {
            V v;
#pragma unroll
            for (int j = 0; j < n; ++j) v[j] = tile[r + j][c];
            *reinterpret_cast<V *>(dst + (int64_t)(c0 + c) * R + r0 + r) = v;
        }
    }
}

// Workgroups of 64 KB of an adapter's two gradients: zeros, where it has no rows.
constexpr int ZERO_FLOATS = 16384;

template <typename TX, typename TW, int RT>
__global__ __launch_bounds__(256) void adapt_prepare_kernel(AdaptPrepare a) {
    typedef typename std::conditional<sizeof(TW) == 4, uint32_t, uint16_t>::type T;
    constexpr int T_BYTES = 64 * (64 * sizeof(T) + 16), S_BYTES = sizeof(float) * TM * (RT * 16 + 1);
    __shared__ __align__(16) char lds[T_BYTES > S_BYTES ? T_BYTES : S_BYTES];
    const int transposes = a.tiles[0] + a.tiles[1], per = transposes + a.zeros;
    const int64_t all = a.panels + (int64_t)a.plan.E * per;
    // the conditions below are the same in the whole workgroup
    for (int64_t b = blockIdx.x; b < all; b += gridDim.x, __syncthreads()) {
        if (b < a.panels) {
            // the tape's panel
            float(*S)[RT * 16 + 1] = reinterpret_cast<float(*)[RT * 16 + 1]>(lds);
            const Tile tile = find_tile<false>(a.plan, a.plan.E, TM, (int)b);
            if (tile.e < 0) continue;
            for (int i = threadIdx.x; i < TM * RT * 4; i += 256) {
                const int m = i / (RT * 4), k = i % (RT * 4) * 4;
                vf4 v = {0.f, 0.f, 0.f, 0.f};
                if (m < tile.cnt && k < a.r) {  // r is a multiple of 8
                    const int64_t row = row_of(a.plan, tile.p0 + m);
                    if (row >= 0) v = load4(a.tape + row * a.r + k);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) S[m][k + j] = v[j];
            }
            __syncthreads();
            write_panel<TX, RT>(a.panel, b, S);
            continue;
        }
        const int e = (int)((b - a.panels) / per), t = (int)((b - a.panels) % per);
        const bool empty = plan_rows(a.plan.offsets[e], a.plan.offsets[e + 1], a.plan.M) == 0;
        if (t < transposes) {
            const int job = t >= a.tiles[0];
            if (!empty)
                transpose_tile<T>(a, job, e, t - (job ? a.tiles[0] : 0),
                                  reinterpret_cast<T(*)[64 + 16 / sizeof(T)]>(lds));
        } else if (empty) {
            int64_t at = (int64_t)(t - transposes) * ZERO_FLOATS + threadIdx.x * 4;
            const int64_t size[2] = {(int64_t)a.rows[0] * a.cols[0], (int64_t)a.rows[1] * a.cols[1]};
            for (int i = 0; i < ZERO_FLOATS / 1024; ++i, at += 1024) {
                if (at < size[0])
                    store4(a.grad[0] + e * size[0] + at, vf4{0.f, 0.f, 0.f, 0.f});
                else if (at < size[0] + size[1])
                    store4(a.grad[1] + e * size[1] + at - size[0], vf4{0.f, 0.f, 0.f, 0.f});
            }
        }
    }
}

// The panel of ds, from the splits' partials.
template <typename TX, int RT>
__global__ __launch_bounds__(256) void adapt_thin_kernel(AdaptThin a) {
    __shared__ float S[TM][RT * 16 + 1];
    const Tile tile = find_tile<false>(a.plan, a.plan.E, TM, blockIdx.x);
    if (tile.e < 0) return;
    const float scale = a.scale ? a.scale[tile.e] : 1.f;
    const int64_t next = (int64_t)a.plan.M * a.r;
    for (int i = threadIdx.x; i < TM * RT * 4; i += 256) {
        const int m = i / (RT * 4), k = i % (RT * 4) * 4;
        vf4 v = {0.f, 0.f, 0.f, 0.f};
        if (m < tile.cnt && k < a.r && row_of(a.plan, tile.p0 + m) >= 0) {  // r is a multiple of 8
            const float *part = a.part + (int64_t)(tile.p0 + m) * a.r + k;
#pragma unroll 8
            for (int sp = 0; sp < a.splits; ++sp) v += load4(part + sp * next);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) S[m][k + j] = scale * v[j];
    }
    __syncthreads();
    write_panel<TX, RT>(a.panel, blockIdx.x, S);
}

// The two kinds of work of a launch, `one` workgroups of the first kind spread
// evenly among `two` of the second, eight of a kind at a time: one on each XCD
// (single ones left an XCD more of one kind than of the other: 468 us of the
// dy launch above, 451 in eights).
struct Mix {
    int one, two;
};

// Which kind workgroup b does, and its number in that kind; it does nothing
// where that is past the kind's count.
__device__ __forceinline__ bool is_first(const Mix &m, unsigned b, int *number) {
    const int64_t one = (m.one + 7) / 8, two = (m.two + 7) / 8, g = b / 8;
    const int64_t before = g * one / (one + two), upto = (g + 1) * one / (one + two);
    *number = (int)((upto > before ? before : g - before) * 8 + b % 8);
    return upto > before;
}

template <typename TX, typename TW, int RT>
__global__ __launch_bounds__(256, RT <= 4 ? 2 : 1) void adapt_dy_kernel(AdaptShrink sh, AdaptGrad gr, Mix mix) {
    constexpr int A = ShrinkBlock<TX, TW, RT>::BYTES, B = GradBlock<TX, RT>::BYTES;
    __shared__ __align__(16) char lds[A > B ? A : B];
    int b;
    const bool first = is_first(mix, blockIdx.x, &b);
    if (b >= (first ? mix.one : mix.two)) return;
    if (first)
        sh.once ? ShrinkBlock<TX, TW, RT>::template run<true>(sh, b, lds)
                : ShrinkBlock<TX, TW, RT>::template run<false>(sh, b, lds);
    else
        GradBlock<TX, RT>::template run<false>(gr, 1, b, lds);
}

template <typename TX, typename TW, int RT, bool ACC>
__global__ __launch_bounds__(256, RT <= 4 ? 2 : 1) void adapt_dx_kernel(AdaptExpand ex, AdaptGrad gr, int chunks,
                                                                       Mix mix) {
    constexpr int A = ExpandBlock<TX, TW, RT, ACC>::BYTES, B = GradBlock<TX, RT>::BYTES;
    __shared__ __align__(16) char lds[A > B ? A : B];
    int b;
    const bool first = is_first(mix, blockIdx.x, &b);
    if (b >= (first ? mix.one : mix.two)) return;
    if (first)
        ExpandBlock<TX, TW, RT, ACC>::run(ex, chunks, b, lds);
    else
        gr.once ? GradBlock<TX, RT>::template run<true>(gr, 0, b, lds)
                : GradBlock<TX, RT>::template run<false>(gr, 0, b, lds);
}

// The partials of an adapter of several ranges, added in range order.
// blockIdx.z: the gradient.
__global__ __launch_bounds__(256) void adapt_reduce_kernel(AdaptGrad a) {
    const AdaptGradJob &job = a.job[blockIdx.z];
    const int e = blockIdx.y;
    const int64_t size = (int64_t)a.r * job.N;
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if ((int64_t)blockIdx.x * 1024 >= size) return;
    auto rows = [&](int f) { return plan_rows(a.plan.offsets[f], a.plan.offsets[f + 1], a.plan.M); };
    const int cnt = rows(e);
    if (cnt <= a.range) return;
    // partials of the adapters before: every wave sums for itself
    const int lane = threadIdx.x & 63;
    int slot = 0;
    for (int base = 0; base < e; base += 64) {
        int several = 0;
        if (base + lane < e) {
            const int n = rows(base + lane);
            if (n > a.range) several = n / a.range + (n % a.range ? 1 : 0);
        }
        for (int o = 32; o > 0; o /= 2) several += __shfl_xor(several, o);
        slot += several;
    }
    const int of = cnt / a.range + (cnt % a.range ? 1 : 0);
    if (slot + of > a.slots) return;
    if (at >= size) return;
    float *g = job.grad + e * size + at;
    vf4 sum = a.acc ? load4(g) : vf4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int j = 0; j < of; ++j) sum += load4(job.part + (int64_t)(slot + j) * size + at);
    store4(g, sum);
}

template <typename TX, typename TW, int RT>
hipError_t prepare_t(AdaptPrepare a, hipStream_t s) {
    for (int j = 0; j < 2; ++j) a.tiles[j] = (a.rows[j] + 63) / 64 * ((a.cols[j] + 63) / 64);
    const int64_t floats = (int64_t)a.rows[0] * a.cols[0] + (int64_t)a.rows[1] * a.cols[1];
    a.zeros = a.grad[0] ? (int)((floats + ZERO_FLOATS - 1) / ZERO_FLOATS) : 0;
    a.panels = a.tape ? (int)adapt_tiles(a.plan.M, a.plan.E, TM) : 0;
    int64_t blocks = a.panels + (int64_t)a.plan.E * (a.tiles[0] + a.tiles[1] + a.zeros);
    if (blocks > ((int64_t)1 << 22)) blocks = (int64_t)1 << 22;  // the kernel steps on by the grid
    hipLaunchKernelGGL((adapt_prepare_kernel<TX, TW, RT>), dim3((unsigned)blocks), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <typename TX, int RT>
hipError_t thin_t(const AdaptThin &a, hipStream_t s) {
    hipLaunchKernelGGL((adapt_thin_kernel<TX, RT>), dim3((unsigned)adapt_tiles(a.plan.M, a.plan.E, TM)), dim3(256), 0,
                       s, a);
    return hipGetLastError();
}

int64_t grad_blocks(const AdaptGrad &a, int which) {
    return adapt_tiles(a.plan.M, a.plan.E, a.range) * ((a.job[which].N + 255) / 256);
}

unsigned mix_blocks(const Mix &m) { return (unsigned)(8 * ((m.one + 7) / 8 + (m.two + 7) / 8)); }

// Rows that the last-level cache (256 MB) cannot hold are read with loads that
// ask not to be kept where nothing reads them again while they could be there.
// dy by ds, which leaves the caches to the weights and panels: 30000 rows of
// 17408 bf16 (1 GB) 425 us, 451 with ordinary loads; smaller dy is still there
// when the gradient reads it: 8192 rows of 4096 f32 (134 MB) 58 us, 66 if not
// kept. x by its gradient, the call's only read of it, if over a quarter of the
// cache, which it shares with dy, dx and the next call's: 16384 rows of 4096 f32
// (268 MB), rank 16, 238 us a call, 242 with ordinary loads; 8192 rows 134 and 133,
// with a layer's backward on the same x 290 and 295; 4096 rows (67 MB) 84 and
// 79, with the layer 183 and 179.
constexpr int64_t CACHE_BYTES = (int64_t)256 << 20;

template <typename TX>
int64_t row_bytes(int64_t rows, int64_t columns) {
    return rows * columns * (int64_t)sizeof(TX);
}

template <typename TX, typename TW, int RT>
hipError_t dy_t(AdaptShrink sh, const AdaptGrad &gr, hipStream_t s) {
    sh.once = row_bytes<TX>(sh.plan.M, sh.K) > CACHE_BYTES;
    const Mix mix = {(int)(sh.splits * adapt_tiles(sh.plan.M, sh.plan.E, TM)), (int)grad_blocks(gr, 1)};
    hipLaunchKernelGGL((adapt_dy_kernel<TX, TW, RT>), dim3(mix_blocks(mix)), dim3(256), 0, s, sh, gr, mix);
    return hipGetLastError();
}

template <typename TX, typename TW, int RT>
hipError_t dx_t(const AdaptExpand &ex, AdaptGrad gr, hipStream_t s) {
    gr.once = row_bytes<TX>(gr.plan.M, gr.job[0].N) > CACHE_BYTES / 4;
    const int64_t chunks = adapt_chunks(ex.plan.M, ex.plan.E, ex.N);
    const int64_t expands = ex.out ? chunks * adapt_tiles(ex.plan.M, ex.plan.E, TM) : 0;
    const Mix mix = {(int)expands, (int)grad_blocks(gr, 0)};
    if (ex.acc)
        hipLaunchKernelGGL((adapt_dx_kernel<TX, TW, RT, true>), dim3(mix_blocks(mix)), dim3(256), 0, s, ex, gr,
                           (int)chunks, mix);
    else
        hipLaunchKernelGGL((adapt_dx_kernel<TX, TW, RT, false>), dim3(mix_blocks(mix)), dim3(256), 0, s, ex, gr,
                           (int)chunks, mix);
    return hipGetLastError();
}

#define BLR_BY_RANK1(r, F, TX, ...)                                                              \
    ((r) <= 16   ? F<TX, 1>(__VA_ARGS__)                                                         \
     : (r) <= 32 ? F<TX, 2>(__VA_ARGS__)                                                         \
     : (r) <= 64 ? F<TX, 4>(__VA_ARGS__)                                                         \
                 : F<TX, 8>(__VA_ARGS__))

}  // namespace

hipError_t launch_adapt_prepare(const AdaptPrepare &a, hipStream_t s) {
    prof_begin(K_ADAPT_PREPARE, s);
    hipError_t e = BLR_BY_TYPES(a, prepare_t, a, s);
    prof_end(s);
    return e;
}

hipError_t launch_adapt_dy(const AdaptShrink &sh, const AdaptGrad &gr, hipStream_t s) {
    prof_begin(K_ADAPT_DY, s);
    hipError_t e = BLR_BY_TYPES(sh, dy_t, sh, gr, s);
    prof_end(s);
    return e;
}

hipError_t launch_adapt_thin(const AdaptThin &a, hipStream_t s) {
    prof_begin(K_ADAPT_THIN, s);
    hipError_t e = a.act == 0   ? BLR_BY_RANK1(a.r, thin_t, float, a, s)
                   : a.act == 1 ? BLR_BY_RANK1(a.r, thin_t, _Float16, a, s)
                                : BLR_BY_RANK1(a.r, thin_t, __bf16, a, s);
    prof_end(s);
    return e;
}

hipError_t launch_adapt_dx(const AdaptExpand &ex, const AdaptGrad &gr, hipStream_t s) {
    prof_begin(K_ADAPT_DX_GRAD, s);
    hipError_t e = BLR_BY_TYPES(ex, dx_t, ex, gr, s);
    prof_end(s);
    return e;
}

hipError_t launch_adapt_reduce(const AdaptGrad &a, hipStream_t s) {
    const int N = a.job[0].N > a.job[1].N ? a.job[0].N : a.job[1].N;
    const int64_t blocks = ((int64_t)a.r * N / 4 + 255) / 256;
    prof_begin(K_ADAPT_REDUCE, s);
    hipLaunchKernelGGL(adapt_reduce_kernel, dim3((unsigned)blocks, (unsigned)a.plan.E, 2), dim3(256), 0, s, a);
    hipError_t e = hipGetLastError();
    prof_end(s);
    return e;
}

}  // namespace blr
