// Token routing for gfx950: pairs (token, choice) sorted by expert, rows laid
// out in that order, weighted back into tokens, and the gradient.
//
//   order    the stable sort of the pairs by expert id, pairs whose id is not
//            in [0, E) last; slot is its inverse; offsets[e] the first
//            position of expert e, offsets[E] the number of placed pairs
//   gather   rows[slot[t][j]] = x[t], zero for a pair that is not placed
//   combine  y[t] (+)= sum_j w[t][j] z[slot[t][j]] over the placed pairs
//   backward dz[slot[t][j]] = w[t][j] dy[t] (zero if not placed),
//            dw[t][j] = dy[t] . z[slot[t][j]] (zero if not placed)
//
// All three row kernels go token by token, so that x, y and dy cross HBM
// once and only the experts' rows are addressed through slot. They are copies
// with a little arithmetic, bound by HBM, where a 2 GiB device copy moves 4.9
// TB/s: 8192 tokens to 8 of 128 experts, rows of 8 KB, take 118 us in the gather
// (5.1 TB/s); 30000 back from 4 choices, rows of 10 KB, 302 us in the combine
// (5.1 TB/s); 8192 with 8 choices, rows of 16 KB, 480 us in the backward (4.8
// TB/s).
#include "blr_internal.h"
#include "blr_vec.h"

namespace blr {

namespace {

constexpr int SORT_WAVES = 16;
constexpr int SORT_THREADS = 64 * SORT_WAVES;
// Pairs that one workgroup places alone: a second workgroup needs the first's
// counts, hence a launch before. Both orders of size are bound by latency: one
// launch of 64 pairs takes 4 us, two of 65536 over 128 experts 4 and 9 us.
constexpr int64_t SORT_ONE = 8192;
constexpr int64_t SORT_RANGE_MIN = 4096;
constexpr int64_t SORT_RANGES_MAX = 256;

__device__ __forceinline__ int group_of(int id, int E) { return (unsigned)id < (unsigned)E ? id : E; }

__global__ __launch_bounds__(SORT_THREADS) void route_count_kernel(RouteSortArgs a) {
    __shared__ uint32_t cnt[ROUTE_MAX_EXPERTS + 1];
    const int E1 = a.experts + 1;
    for (int e = threadIdx.x; e < E1; e += SORT_THREADS) cnt[e] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * a.per_range;
    const int64_t hi = lo + a.per_range < a.pairs ? lo + a.per_range : a.pairs;
    for (int64_t p = lo + threadIdx.x; p < hi; p += SORT_THREADS) atomicAdd(&cnt[group_of(a.ids[p], a.experts)], 1u);
    __syncthreads();
    for (int e = threadIdx.x; e < E1; e += SORT_THREADS) a.counts[(int64_t)blockIdx.x * E1 + e] = cnt[e];
}

// One workgroup places one range. Each wave takes a contiguous part of it and
// counts it into its own table; a scan over experts, earlier ranges and
// earlier waves turns the counts into each wave's first positions, and a
// second walk hands them out: lanes of equal id find each other with one
// ballot per id bit, so equal ids keep their order (integer sums only: the
// result does not depend on any order of execution).
__global__ __launch_bounds__(SORT_THREADS) void route_place_kernel(RouteSortArgs a, int id_bits) {
    __shared__ uint32_t table[SORT_WAVES * (ROUTE_MAX_EXPERTS + 1)];
    __shared__ uint32_t total[ROUTE_MAX_EXPERTS + 1], before[ROUTE_MAX_EXPERTS + 1];
    __shared__ uint32_t wave_sum[SORT_WAVES];
    const int E = a.experts, E1 = E + 1;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int64_t lo = (int64_t)blockIdx.x * a.per_range;
    const int64_t hi = lo + a.per_range < a.pairs ? lo + a.per_range : a.pairs;
    const int64_t per_wave = ((hi - lo + SORT_WAVES - 1) / SORT_WAVES + 63) / 64 * 64;
    const int64_t w_lo = lo + w * per_wave;
    const int64_t w_hi = w_lo + per_wave < hi ? w_lo + per_wave : hi;
    uint32_t *mine = table + w * E1;

    for (int i = tid; i < SORT_WAVES * E1; i += SORT_THREADS) table[i] = 0;
    for (int e = tid; e < E1; e += SORT_THREADS) total[e] = before[e] = 0;
    __syncthreads();
    for (int64_t p = w_lo + lane; p < w_hi; p += 64) atomicAdd(&mine[group_of(a.ids[p], E)], 1u);
    if (a.ranges > 1) {
        // every range's counts: threads over (expert, part of the ranges)
        int lanes = 1;
        while (lanes < E1 && lanes < SORT_THREADS) lanes *= 2;
        const int parts = SORT_THREADS / lanes;
        for (int e = tid & (lanes - 1); e < E1; e += lanes) {
            uint32_t all = 0, early = 0;
            for (int b = tid / lanes; b < a.ranges; b += parts) {
                const uint32_t c = a.counts[(int64_t)b * E1 + e];
                all += c;
                early += b < (int)blockIdx.x ? c : 0u;
            }
            atomicAdd(&total[e], all);
            atomicAdd(&before[e], early);
        }
    }
    __syncthreads();
    if (a.ranges == 1) {
        for (int e = tid; e < E1; e += SORT_THREADS) {
            uint32_t all = 0;
            for (int v = 0; v < SORT_WAVES; ++v) all += table[v * E1 + e];
            total[e] = all;
        }
        __syncthreads();
    }
    // exclusive scan over the E <= 1024 experts, one per thread; the group of
    // the pairs without one starts behind them all
    const uint32_t own = tid < E ? total[tid] : 0u;
    uint32_t incl = own;
    for (int o = 1; o < 64; o *= 2) {
        const uint32_t v = __shfl_up(incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 63) wave_sum[w] = incl;
    __syncthreads();
    uint32_t base = incl - own, sum = 0;
    for (int v = 0; v < SORT_WAVES; ++v) {
        if (v < w) base += wave_sum[v];
        sum += wave_sum[v];
    }
    for (int e = tid; e < E1; e += SORT_THREADS) {
        uint32_t at = e < E ? base : sum;
        if (blockIdx.x == 0) a.offsets[e] = (int32_t)at;
        at += before[e];
        for (int v = 0; v < SORT_WAVES; ++v) {
            const uint32_t c = table[v * E1 + e];
            table[v * E1 + e] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t p0 = w_lo; p0 < w_hi; p0 += 64) {
        const int64_t p = p0 + lane;
        const bool in = p < w_hi;
        const int e = in ? group_of(a.ids[p], E) : E;
        uint64_t same = __ballot(in);
        for (int b = 0; b < id_bits; ++b) {
            const uint64_t set = __ballot((e >> b) & 1);
            same &= ((e >> b) & 1) ? set : ~set;
        }
        const int leader = __ffsll((unsigned long long)same) - 1;  // < 0 only for lanes outside
        uint32_t at = 0;
        if (in && lane == leader) at = atomicAdd(&mine[e], (uint32_t)__popcll(same));
        at = __shfl(at, leader < 0 ? 0 : leader);
        if (in) {
            at += (uint32_t)__popcll(same & ((1ull << lane) - 1));
            a.order[at] = (int32_t)p;
            a.slot[p] = (int32_t)at;
        }
    }
}

// Workgroups along the tokens; the kernels step on by the grid past it.
constexpr int64_t TOKEN_BLOCKS = (int64_t)1 << 22;
unsigned token_blocks(int64_t T, int64_t per) {
    const int64_t n = (T + per - 1) / per;
    return (unsigned)(n < TOKEN_BLOCKS ? n : TOKEN_BLOCKS);
}

// Threads of a workgroup over a row: tx (a power of two) take its vectors, the
// 256 / tx others further tokens.
int row_threads(int64_t nv) {
    int tx = 8;
    while (tx < 256 && tx < nv) tx *= 2;
    return tx;
}

__global__ __launch_bounds__(256) void route_gather_kernel(RouteRows a, int64_t nv) {
    const int64_t c = (int64_t)blockIdx.y * blockDim.x + threadIdx.x;
    if (c >= nv) return;
    const int placed = *a.placed;
    const int64_t pairs = a.T * a.k;
    for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < a.T; t += (int64_t)gridDim.x * blockDim.y) {
        const vf4 v = reinterpret_cast<const vf4 *>(a.a)[t * nv + c];
        for (int j = 0; j < a.k; ++j) {
            const int at = a.slot[t * a.k + j];
            if (at < 0 || at >= pairs) continue;
            reinterpret_cast<vf4 *>(a.out)[at * nv + c] = at < placed ? v : vf4{0.f, 0.f, 0.f, 0.f};
        }
    }
}

template <typename T>
__global__ __launch_bounds__(256) void route_combine_kernel(RouteRows a, int64_t nv) {
    constexpr int n = Vec<T>::n;
    typedef typename Vec<T>::v V;
    typedef float F __attribute__((ext_vector_type(n)));
    const int64_t c = (int64_t)blockIdx.y * blockDim.x + threadIdx.x;
    if (c >= nv) return;
    const int64_t pairs = a.T * a.k;
    const int64_t placed = *a.placed < pairs ? *a.placed : pairs;
    const V *z = reinterpret_cast<const V *>(a.a);
    for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < a.T; t += (int64_t)gridDim.x * blockDim.y) {
        V *y = reinterpret_cast<V *>(a.out) + t * nv + c;
        F sum = a.acc ? __builtin_convertvector(*y, F) : (F)(0.f);
#pragma unroll 4
        for (int j = 0; j < a.k; ++j) {
            const int at = a.slot[t * a.k + j];
            if (at < 0 || at >= placed) continue;  // nothing of its row or weight is read
            const float w = a.weights ? a.weights[t * a.k + j] : 1.f;
            sum += w * __builtin_convertvector(z[at * nv + c], F);
        }
        *y = __builtin_convertvector(sum, V);
    }
}

// W waves walk a token's row together (W = 1: four tokens a workgroup, for rows
// of up to 4 KB). Four choices at a time: their rows are in flight together, and dy's row is read
// once per four.
template <typename T, int W>
__global__ __launch_bounds__(256) void route_combine_backward_kernel(RouteRows a, int64_t nv) {
    constexpr int n = Vec<T>::n;
    typedef typename Vec<T>::v V;
    typedef float F __attribute__((ext_vector_type(n)));
    __shared__ float part[4][4];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t pairs = a.T * a.k;
    const int64_t placed = *a.placed < pairs ? *a.placed : pairs;
    const V *z = reinterpret_cast<const V *>(a.z);
    V *dz = reinterpret_cast<V *>(a.out);
    // W = 4: every wave takes the same tokens, so all meet at the barriers
    for (int64_t t = W == 1 ? (int64_t)blockIdx.x * 4 + w : (int64_t)blockIdx.x; t < a.T;
         t += (int64_t)gridDim.x * (4 / W)) {
        const V *dy = reinterpret_cast<const V *>(a.a) + t * nv;
        for (int j0 = 0; j0 < a.k; j0 += 4) {
            int at[4];
            float wt[4], dot[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool in = j0 + j < a.k;
                at[j] = in ? a.slot[t * a.k + j0 + j] : -1;
                if (at[j] >= pairs) at[j] = -1;
                wt[j] = at[j] >= 0 && at[j] < placed && a.weights ? a.weights[t * a.k + j0 + j] : 1.f;
                dot[j] = 0.f;
            }
            for (int64_t c = W == 1 ? lane : (int64_t)threadIdx.x; c < nv; c += 64 * W) {
                const F g = __builtin_convertvector(dy[c], F);
                if (a.dw) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (at[j] >= 0 && at[j] < placed) {
                            const F v = g * __builtin_convertvector(z[at[j] * nv + c], F);
#pragma unroll
                            for (int q = 0; q < n; ++q) dot[j] += v[q];
                        }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (at[j] >= 0)
                        dz[at[j] * nv + c] = at[j] < placed ? __builtin_convertvector(wt[j] * g, V) : (V)(T)0;
            }
            if (a.dw) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    for (int o = 32; o > 0; o /= 2) dot[j] += __shfl_xor(dot[j], o);
                if (W == 1) {
                    if (lane < 4 && j0 + lane < a.k)
                        a.dw[t * a.k + j0 + lane] =
                            lane == 0 ? dot[0] : lane == 1 ? dot[1] : lane == 2 ? dot[2] : dot[3];
                } else {
                    __syncthreads();  // the last four's sums have been read
                    if (lane == 0) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) part[w][j] = dot[j];
                    }
                    __syncthreads();
                    const int j = threadIdx.x;
                    if (j < 4 && j0 + j < a.k)
                        a.dw[t * a.k + j0 + j] = ((part[0][j] + part[1][j]) + part[2][j]) + part[3][j];
                }
            }
        }
    }
}

template <typename T>
hipError_t combine_t(const RouteRows &a, hipStream_t s) {
    const int64_t nv = a.d / Vec<T>::n;
    const int tx = row_threads(nv);
    const dim3 block(tx, 256 / tx), grid(token_blocks(a.T, block.y), (unsigned)((nv + tx - 1) / tx));
    hipLaunchKernelGGL((route_combine_kernel<T>), grid, block, 0, s, a, nv);
    return hipGetLastError();
}

template <typename T>
hipError_t combine_backward_t(const RouteRows &a, hipStream_t s) {
    const int64_t nv = a.d / Vec<T>::n;
    // rows of up to 256 vectors: a wave each, no barrier; longer ones: four
    if (nv <= 256)
        hipLaunchKernelGGL((route_combine_backward_kernel<T, 1>), dim3(token_blocks(a.T, 4)), dim3(256), 0, s, a, nv);
    else
        hipLaunchKernelGGL((route_combine_backward_kernel<T, 4>), dim3(token_blocks(a.T, 1)), dim3(256), 0, s, a, nv);
    return hipGetLastError();
}

}  // namespace

int64_t route_ranges(int64_t pairs, int64_t *per_range) {
    int64_t per = (pairs + SORT_RANGES_MAX - 1) / SORT_RANGES_MAX;
    per = pairs <= SORT_ONE ? SORT_ONE : per > SORT_RANGE_MIN ? (per + 63) / 64 * 64 : SORT_RANGE_MIN;
    if (per_range) *per_range = per;
    return (pairs + per - 1) / per;
}

hipError_t launch_route_sort(const RouteSortArgs &a, hipStream_t s) {
    if (a.ranges > 1) {
        prof_begin(K_ROUTE_COUNT, s);
        hipLaunchKernelGGL(route_count_kernel, dim3(a.ranges), dim3(SORT_THREADS), 0, s, a);
        hipError_t e = hipGetLastError();
        prof_end(s);
        if (e != hipSuccess) return e;
    }
    int bits = 0;
    while ((a.experts >> bits) != 0) ++bits;  // ids 0 .. E
    prof_begin(K_ROUTE_PLACE, s);
    hipLaunchKernelGGL(route_place_kernel, dim3(a.ranges), dim3(SORT_THREADS), 0, s, a, bits);
    hipError_t e = hipGetLastError();
    prof_end(s);
    return e;
}

hipError_t launch_route_gather(const RouteRows &a, hipStream_t s) {
    const int64_t nv = a.d * (a.dtype == 0 ? 4 : 2) / 16;
    const int tx = row_threads(nv);
    const dim3 block(tx, 256 / tx), grid(token_blocks(a.T, block.y), (unsigned)((nv + tx - 1) / tx));
    prof_begin(K_ROUTE_GATHER, s);
    hipLaunchKernelGGL(route_gather_kernel, grid, block, 0, s, a, nv);
    hipError_t e = hipGetLastError();
    prof_end(s);
    return e;
}

hipError_t launch_route_combine(const RouteRows &a, hipStream_t s) {
    prof_begin(K_ROUTE_COMBINE, s);
    hipError_t e = a.dtype == 0   ? combine_t<float>(a, s)
                   : a.dtype == 1 ? combine_t<_Float16>(a, s)
                                  : combine_t<__bf16>(a, s);
    prof_end(s);
    return e;
}

hipError_t launch_route_combine_backward(const RouteRows &a, hipStream_t s) {
    prof_begin(K_ROUTE_COMBINE_BWD, s);
    hipError_t e = a.dtype == 0   ? combine_backward_t<float>(a, s)
                   : a.dtype == 1 ? combine_backward_t<_Float16>(a, s)
                                  : combine_backward_t<__bf16>(a, s);
    prof_end(s);
    return e;
}

}  // namespace blr
