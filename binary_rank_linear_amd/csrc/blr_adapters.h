// Device code of the low-rank adapters of many requests at once, for gfx950
// (internal; blr_adapters.hip launches the forward, blr_adapters_backward.hip
// the backward). Row t with adapter e (A_e [r][d_in], B_e [d_out][r], factor
// c_e):
//
//   forward   s = x A_e^T          y (+)= c_e s B_e^T
//   backward  ds = c_e dy B_e      dx (+)= ds A_e
//             dA_e (+)= sum_t ds^T x      dB_e (+)= c_e sum_t dy^T s
//
// Rows are taken by the plan of the sort (blr_route.hip): a workgroup has a
// tile of rows of one adapter, found from offsets by every wave for itself.
// The rank is small, so a contraction of 16-bit rows is bound by the rows' bytes.
// So is one of f32 rows up to rank 32; 2 r flop for the 4 bytes of an element,
// at the 153.6 TFLOP/s and 4.92 TB/s of large products and copies, meet at rank
// 62, and ranks of 33 to 64 count as 64 here, larger ones as 128: there the
// matrix instructions bound all of them but the forward's expand, which reads
// y and writes it. A contraction takes its rows from memory once; ds and the
// gradient of B each read dy.
//
// Rows of f32 run on v_mfma_f32_16x16x4_f32 (D += A B: lane l = 16 q + c gives
// A[c][q] and B[q][c], and holds D[4 q + i][c], i < 4), with 16-bit adapters
// widened, which is exact. Rows of 16 bits run on the 16x16x32 instructions
// (lane gives eight k: A[c][8 q + j], B[8 q + j][c]; D as above), whose
// products are exact and whose sums are f32; s and ds, which are f32, enter
// them as three bf16 terms, so that all their 24 bits take part (see
// take_term). Which column of a product a k index stands for is free as long as
// A and B agree: the loads use that to read 16 consecutive bytes per lane.
#pragma once

#include <type_traits>

#include "blr_internal.h"
#include "blr_plan.h"
#include "blr_vec.h"

namespace blr {

namespace {

constexpr int TM = ADAPT_TM;
typedef uint32_t vu2 __attribute__((ext_vector_type(2)));
typedef uint32_t vu4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ vf4 mfma4(float a, float b, vf4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// The wave's number in its workgroup, in a scalar register.
__device__ __forceinline__ int wave() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)); }

// base + bytes: where base is the same in all lanes, the address needs one
// 32-bit register per lane.
template <typename T>
__device__ __forceinline__ const T *ahead(const T *base, unsigned bytes) {
    return reinterpret_cast<const T *>(reinterpret_cast<const char *>(base) + bytes);
}

// A vector V from p; ONCE: by a load that asks not to be kept in the caches.
template <bool ONCE, typename V, typename T>
__device__ __forceinline__ V fetch(const T *p) {
    const V *v = reinterpret_cast<const V *>(p);
    return ONCE ? __builtin_nontemporal_load(v) : *v;
}

// A tile of one group of the plan; group E is the rows without an adapter.
struct Tile {
    int e;      // -1: the grid has more tiles than the plan
    int p0;     // first position
    int cnt;    // positions
    int j, of;  // this tile is the j-th of the group's `of`
    int slot;   // tiles of earlier groups that have several
    int panel;  // tiles of 64 positions of earlier groups
};

// Sum over the lanes up to this one, of which only the first n are not zero.
__device__ __forceinline__ int scan(int v, int n, int lane) {
    for (int o = 1; o < 64 && o < n; o *= 2) {
        const int u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Tile b of tiles of tm positions over groups 0 .. groups-1 (wave-uniform);
// slot and panel only where RANGES. Offsets out of order or out of range
// cannot lead outside [0, M).
template <bool RANGES>
__device__ Tile find_tile(const AdaptPlan &plan, int groups, int tm, int b) {
    const int lane = threadIdx.x & 63;
    int run = 0, many = 0, panels = 0;
    for (int base = 0; base < groups; base += 64) {
        const int e = base + lane;
        int lo = 0, cnt = 0;
        if (e < groups) {
            const int offset = plan.offsets[e];
            lo = plan_at(offset, plan.M);
            cnt = plan_rows(offset, e < plan.E ? plan.offsets[e + 1] : plan.M, plan.M);
        }
        const int nt = cnt / tm + (cnt % tm ? 1 : 0);
        const int incl = scan(nt, groups - base, lane);
        const uint64_t past = __ballot(run + incl > b);
        const int l = past ? __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)past) - 1) : 63;
        const int of = __builtin_amdgcn_readlane(nt, l), upto = __builtin_amdgcn_readlane(incl, l);
        int slot = 0, panel = 0;
        if (RANGES) {
            const int several = nt > 1 ? nt : 0, np = cnt / TM + (cnt % TM ? 1 : 0);
            const int mincl = scan(several, groups - base, lane), pincl = scan(np, groups - base, lane);
            slot = many + __builtin_amdgcn_readlane(mincl, l) - __builtin_amdgcn_readlane(several, l);
            panel = panels + __builtin_amdgcn_readlane(pincl, l) - __builtin_amdgcn_readlane(np, l);
            many += __builtin_amdgcn_readlane(mincl, 63);
            panels += __builtin_amdgcn_readlane(pincl, 63);
        }
        if (past) {
            Tile t;
            t.e = base + l;
            t.of = of;
            t.j = b - run - (upto - of);
            t.p0 = __builtin_amdgcn_readlane(lo, l) + t.j * tm;
            const int left = __builtin_amdgcn_readlane(cnt, l) - t.j * tm;
            t.cnt = left < tm ? left : tm;
            t.slot = slot;
            t.panel = panel;
            return t;
        }
        run += upto;
    }
    return Tile{-1, 0, 0, 0, 0, 0, 0};
}

// The row of position p, -1 if the plan names none.
__device__ __forceinline__ int64_t row_of(const AdaptPlan &plan, int p) {
    const int row = plan.order ? plan.order[p] : p;
    return row >= 0 && row < plan.M ? row : -1;
}

// Matrix instructions on 16-bit operands.
__device__ __forceinline__ vf4 mfma8(vh8 a, vh8 b, vf4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ vf4 mfma8(vb8 a, vb8 b, vf4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Walks a wave's n steps with two register sets (DEEP): the next step's loads
// are in flight while one is used. The walk has no branch around a load (a
// wave's last extra load repeats its last step), or every wait would be for
// all; the barriers keep the compiler from moving the loads behind the
// products. Ranks over 64 leave no room for a second set.
template <typename Step, bool DEEP, typename Load, typename Use>
__device__ __forceinline__ void walk(int n, Load load, Use use) {
    if (n <= 0) return;
    if constexpr (!DEEP) {
        for (int i = 0; i < n; ++i) {
            Step st;
            load(st, i);
            use(st, i);
        }
    } else {
        Step one, two;
        load(one, 0);
        int i = 0;
        for (; i + 2 <= n; i += 2) {
            load(two, i + 1);
            __builtin_amdgcn_sched_barrier(0);
            use(one, i);
            __builtin_amdgcn_sched_barrier(0);
            load(one, i + 2 < n ? i + 2 : n - 1);
            __builtin_amdgcn_sched_barrier(0);
            use(two, i + 1);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (i < n) use(one, i);
    }
}

// ---------------------------------------------------------------- shrink --
// What a lane holds of one step: 128 bytes of a row, over the four lanes q, and
// the weights of the same columns. Rows of f32: 32 columns, lane q the columns
// 4 q .. 4 q + 3 and 16 + 4 q .. Rows of 16 bits: 64, lane q 8 q .. 8 q + 7 and
// 32 + 8 q ..
template <typename TX, typename TW, int RT>
struct ShrinkStep {
    static constexpr int COLS = 32;
    vf4 x[2];
    typename Vec<TW>::v4 w[RT][2];  // widened where they are used, or the wait for them would stand here

    __device__ __forceinline__ void load(const TX *row, const TW *W, int r, int K, int k0, int q, int c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) x[h] = load4(row + k0 + 16 * h + 4 * q);
#pragma unroll
        for (int n = 0; n < RT; ++n) {
            const int rank = n * 16 + c < r ? n * 16 + c : r - 1;  // columns past r of the product are not stored
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[n][h] = *reinterpret_cast<const typename Vec<TW>::v4 *>(
                    ahead(W + k0 + 16 * h, (unsigned)(rank * K + 4 * q) * (unsigned)sizeof(TW)));
        }
    }
    __device__ __forceinline__ void multiply(vf4 (&acc)[RT]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int n = 0; n < RT; ++n) acc[n] = mfma4(x[h][j], (float)w[n][h][j], acc[n]);
    }
};

template <typename T, int RT>
struct ShrinkStep16 {
    static constexpr int COLS = 64;
    typedef typename Vec<T>::v V;
    V x[2], w[RT][2];

    __device__ __forceinline__ void load(const T *row, const T *W, int r, int K, int k0, int q, int c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) x[h] = *reinterpret_cast<const V *>(row + k0 + 32 * h + 8 * q);
#pragma unroll
        for (int n = 0; n < RT; ++n) {
            const int rank = n * 16 + c < r ? n * 16 + c : r - 1;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[n][h] = *reinterpret_cast<const V *>(
                    ahead(W + k0 + 32 * h, (unsigned)(rank * K + 8 * q) * (unsigned)sizeof(T)));
        }
    }
    __device__ __forceinline__ void multiply(vf4 (&acc)[RT]) const {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < RT; ++n) acc[n] = mfma8(x[h], w[n][h], acc[n]);
    }
};
template <int RT>
struct ShrinkStep<_Float16, _Float16, RT> : ShrinkStep16<_Float16, RT> {};
template <int RT>
struct ShrinkStep<__bf16, __bf16, RT> : ShrinkStep16<__bf16, RT> {};

// A wave's steps (every fourth of [from, to)) over a tile of up to 16 rows,
// then the four waves' sums, in wave order, into red.
template <typename TX, typename TW, int RT>
__device__ void shrink_tile(const AdaptShrink &a, const Tile &tile, int from, int to, float (*red)[RT * 16 + 1]) {
    typedef ShrinkStep<TX, TW, RT> Step;
    const int lane = threadIdx.x & 63, w = wave();
    const int q = lane >> 4, c = lane & 15;
    const TW *W = reinterpret_cast<const TW *>(a.W) + (int64_t)tile.e * a.r * a.K;
    // rows past the tile, or not named by the plan, repeat one; not stored
    const int64_t row = row_of(a.plan, tile.p0 + (c < tile.cnt ? c : tile.cnt - 1));
    const TX *x = reinterpret_cast<const TX *>(a.X) + (row < 0 ? 0 : row) * a.K;
    vf4 acc[RT];
#pragma unroll
    for (int n = 0; n < RT; ++n) acc[n] = vf4{0.f, 0.f, 0.f, 0.f};
    const int first = from + w;
    walk<Step, RT <= 4>((to - first + 3) / 4,
                        [&](Step &s, int i) { s.load(x, W, a.r, a.K, (first + 4 * i) * Step::COLS, q, c); },
                        [&](const Step &s, int) { s.multiply(acc); });
    for (int v = 0; v < 4; ++v) {
        if (w == v) {
#pragma unroll
            for (int n = 0; n < RT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float *at = &red[4 * q + i][n * 16 + c];
                    *at = v == 0 ? acc[n][i] : *at + acc[n][i];
                }
        }
        __syncthreads();
    }
}

// The same for tiles of up to 64 rows, by way of LDS. A load instruction takes
// the vector cache one cycle for every four lanes if those lie together in
// memory, and one for every lane if not: lanes laid out for the matrix operand
// (each another row) cost four times the cycles, and that, not HBM, bounds the
// loads above. So eight lanes read 128 bytes of a row, and a wave turns its
// step of X and of the weights round through 16-byte slots of its own (slot
// h of row m stands at h ^ (m & 7), which spreads both sides over the banks);
// no barrier, since no other wave reads them. 28500 rows of 17408 bf16, rank
// 64: 237 us (4.2 TB/s, what reads alone reach here) against 288 by the loads
// above; 8192 of 4096 f32, rank 16: 41 against 44. Tiles of up to 16 rows keep
// the loads above: their 64 would be mostly repeats.
template <typename TX, typename TW, int RT>
struct ShrinkLds {
    static constexpr int COLS = 128 / sizeof(TX);
    static constexpr int X_BYTES = 64 * 128;
    static constexpr int W_ROW = COLS * sizeof(TW);  // 128, or 64 for 16-bit weights beside f32 rows
    static constexpr int W_BYTES = RT * 16 * W_ROW;
    static constexpr int W_LOADS = W_BYTES / 1024;
    static constexpr int BYTES = X_BYTES + W_BYTES;
    vu4 x[8], w[W_LOADS];

    template <bool ONCE>
    __device__ __forceinline__ void load(const TX *const *row, const TW *W, const unsigned *rank, int k0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fetch<ONCE, vu4>(row[i] + k0);
#pragma unroll
        for (int i = 0; i < W_LOADS; ++i) w[i] = *reinterpret_cast<const vu4 *>(ahead(W + k0, rank[i]));
    }
    __device__ __forceinline__ void stage(char *lds, int lane) const {
        const int m = lane >> 3, h = (lane & 7) ^ (m & 7);
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<vu4 *>(lds + (8 * i + m) * 128 + h * 16) = x[i];
        lds += X_BYTES;
        if constexpr (W_ROW == 128) {
#pragma unroll
            for (int i = 0; i < W_LOADS; ++i) *reinterpret_cast<vu4 *>(lds + (8 * i + m) * 128 + h * 16) = w[i];
        } else {
            const int n = lane >> 2, g = (lane & 3) ^ ((n >> 1) & 3);
#pragma unroll
            for (int i = 0; i < W_LOADS; ++i) *reinterpret_cast<vu4 *>(lds + (16 * i + n) * 64 + g * 16) = w[i];
        }
    }
    // All 64 rows against all ranks; all of the step's reads go out first.
    static __device__ __forceinline__ void multiply(const char *lds, vf4 (&acc)[4][RT], int q, int c) {
        typedef typename Vec<TX>::v V;
        V xv[2][4];
        typename std::conditional<W_ROW == 128, V, typename Vec<TW>::v4>::type wv[2][RT];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = ((4 * h + q) ^ (c & 7)) * 16;
#pragma unroll
            for (int n = 0; n < RT; ++n) {
                const char *p = lds + X_BYTES + (16 * n + c) * W_ROW;
                p += W_ROW == 128 ? at : ((2 * h + (q >> 1)) ^ ((c >> 1) & 3)) * 16 + 8 * (q & 1);
                wv[h][n] = *reinterpret_cast<decltype(&wv[0][0])>(const_cast<char *>(p));
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) xv[h][t] = *reinterpret_cast<const V *>(lds + (16 * t + c) * 128 + at);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (sizeof(TX) == 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int n = 0; n < RT; ++n)
#pragma unroll
                        for (int t = 0; t < 4; ++t) acc[t][n] = mfma4(xv[h][t][j], (float)wv[h][n][j], acc[t][n]);
            } else {
#pragma unroll
                for (int n = 0; n < RT; ++n)
#pragma unroll
                    for (int t = 0; t < 4; ++t) acc[t][n] = mfma8(xv[h][t], wv[h][n], acc[t][n]);
            }
        }
    }
};

// Orders a wave's own writes and reads of LDS (they execute in order; this
// keeps the compiler from moving one past the other).
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <typename TX, typename TW, int RT, bool ONCE>
__device__ void shrink_tile_lds(const AdaptShrink &a, const Tile &tile, int from, int to, char *lds,
                                float (*red)[RT * 16 + 1]) {
    typedef ShrinkLds<TX, TW, RT> Step;
    const int lane = threadIdx.x & 63, w = wave();
    const int q = lane >> 4, c = lane & 15;
    const TW *W = reinterpret_cast<const TW *>(a.W) + (int64_t)tile.e * a.r * a.K;
    const TX *x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // rows past the tile, or not named by the plan, repeat one; not stored
        const int m = 8 * i + (lane >> 3);
        const int64_t row = row_of(a.plan, tile.p0 + (m < tile.cnt ? m : tile.cnt - 1));
        x[i] = reinterpret_cast<const TX *>(a.X) + (row < 0 ? 0 : row) * a.K + (lane & 7) * (16 / sizeof(TX));
    }
    unsigned rank[Step::W_LOADS];
#pragma unroll
    for (int i = 0; i < Step::W_LOADS; ++i) {
        const int per = Step::W_ROW / 16;  // lanes of a rank's columns
        const int n = i * (64 / per) + lane / per;  // columns past r of the product are not stored
        rank[i] = (unsigned)((n < a.r ? n : a.r - 1) * a.K) * (unsigned)sizeof(TW) + (lane % per) * 16;
    }
    vf4 acc[4][RT];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int n = 0; n < RT; ++n) acc[t][n] = vf4{0.f, 0.f, 0.f, 0.f};
    char *mine = lds + w * Step::BYTES;
    const int first = from + w, n = (to - first + 3) / 4;
    if (n > 0) {
        Step st;
        st.template load<ONCE>(x, W, rank, first * Step::COLS);
        for (int i = 0; i < n; ++i) {
            st.stage(mine, lane);
            wave_lds_fence();
            const int next = i + 1 < n ? i + 1 : i;  // no branch: see walk
            st.template load<ONCE>(x, W, rank, (first + 4 * next) * Step::COLS);
            __builtin_amdgcn_sched_barrier(0);
            Step::multiply(mine, acc, q, c);
            wave_lds_fence();
        }
    }
    __syncthreads();  // red lies in the same memory
    for (int v = 0; v < 4; ++v) {
        if (w == v) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int n = 0; n < RT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float *at = &red[t * 16 + 4 * q + i][n * 16 + c];
                        *at = v == 0 ? acc[t][n][i] : *at + acc[t][n][i];
                    }
        }
        __syncthreads();
    }
}

// One workgroup's part of the grid: 64 rows x all r over one split of K, the
// splits of a tile next to each other (grids are one-dimensional: their other
// dimensions are short).
template <typename TX, typename TW, int RT>
struct ShrinkBlock {
    typedef ShrinkLds<TX, TW, RT> Lds;
    static constexpr int BYTES = 4 * Lds::BYTES;

    template <bool ONCE>
    static __device__ void run(const AdaptShrink &a, int block, char *lds) {
        float(*red)[RT * 16 + 1] = reinterpret_cast<float(*)[RT * 16 + 1]>(lds);
        static_assert(sizeof(float) * TM * (RT * 16 + 1) <= BYTES, "the sums fit");
        const int split = block % a.splits;
        const Tile tile = find_tile<false>(a.plan, a.plan.E, TM, block / a.splits);
        if (tile.e < 0) return;
        const int64_t steps = a.K / Lds::COLS;
        const int from = (int)(steps * split / a.splits), to = (int)(steps * (split + 1) / a.splits);
        if (tile.cnt <= 16)
            shrink_tile<TX, TW, RT>(a, tile, from, to, red);
        else
            shrink_tile_lds<TX, TW, RT, ONCE>(a, tile, from, to, lds, red);
        float *part = a.part + ((int64_t)split * a.plan.M + tile.p0) * a.r;
        const int per = a.r / 4;
        for (int i = threadIdx.x; i < tile.cnt * per; i += 256) {
            const int m = i / per, k = i % per * 4;
            store4(part + (int64_t)m * a.r + k, vf4{red[m][k], red[m][k + 1], red[m][k + 2], red[m][k + 3]});
        }
    }
};

// The bf16 nearest to v, and in v what it leaves; nothing where v is not
// finite, so that an infinity stays one. Three such terms hold the 24 bits of
// an f32 and two the 11 of an f16, whatever its size, since bf16 has f32's
// exponents: no element loses bits to a larger neighbour. (Two f16 terms with
// the row's largest element scaled near one lost every element 2^-25 below it;
// two products instead of five, 8192 rows of 4096 -> 4096 added to y, the whole
// call: 127 us against 147 at rank 128, 41 against 42 at rank 16. bf16 rows, two
// terms against three: 39.4 us and 40.0 at rank 16, 116 and 117 of 4096 -> 12288
// at rank 64.)
__device__ __forceinline__ __bf16 take_term(float &v) {
    const __bf16 t = (__bf16)v;
    const float left = v - (float)t;
    v = __builtin_isfinite(left) ? left : 0.f;
    return t;
}

// Element j of the three terms of an f32. A finite v past bf16's largest value,
// the last 2^-9 of f32's range, would round to an infinite first term; that
// term is the largest value then.
__device__ __forceinline__ void put_terms(float v, int j, vb8 (&term)[3]) {
    constexpr float largest = 0x1.fep127f;
    float first = __builtin_isfinite(v) ? fminf(fmaxf(v, -largest), largest) : v;
    term[0][j] = take_term(first);
    v -= (float)term[0][j];
    v = __builtin_isfinite(v) ? v : 0.f;
    term[1][j] = take_term(v);
    term[2][j] = take_term(v);
}

// 16-bit weights as bf16 operands: bf16 as they are, f16 as the upper half of
// the f32 of that value and what it leaves, both exact.
template <typename T>
constexpr int PARTS = __is_same(T, _Float16) ? 2 : 1;

__device__ __forceinline__ void split(vb8 w, vb8 (&part)[1]) { part[0] = w; }
__device__ __forceinline__ void split(vh8 w, vb8 (&part)[2]) {
    vu4 hi, lo;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float a = (float)w[2 * j], b = (float)w[2 * j + 1];
        const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
        const float la = a - __uint_as_float(ua & 0xffff0000u), lb = b - __uint_as_float(ub & 0xffff0000u);
        hi[j] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
        lo[j] = __builtin_amdgcn_perm(__float_as_uint(lb), __float_as_uint(la), 0x07060302u);
    }
    part[0] = __builtin_bit_cast(vb8, hi);
    part[1] = __builtin_bit_cast(vb8, lo);
}

// Terms of s that part p of a weight meets: all three, but of the second part,
// 2^-7 of the weight at most, only two (with the third, 2^-18 of s at most, it
// would add 2^-25 of the whole product).
__device__ constexpr int terms_for(int p) { return p == 0 ? 3 : 2; }

// ------------------------------------------------------------------ thin --
// A tile's ds or s, S[64][.] with zeros past the tile's end, as the gradients'
// panel: in the order of the matrix operand, a slot of 16 bytes a lane. f32
// for rows of f32: [16 rows][16 ranks][lane][4]. For rows of 16 bits three
// bf16 terms: [32 rows][term][16 ranks][lane][8].
template <typename TX, int RT, int STRIDE>
__device__ void write_panel(void *panels, int64_t tile, const float (*S)[STRIDE]) {
    if constexpr (sizeof(TX) == 4) {
        float *to = reinterpret_cast<float *>(panels) + tile * RT * 16 * TM;
        for (int i = threadIdx.x; i < 4 * RT * 64; i += 256) {
            const int lane = i & 63, n = (i >> 6) % RT, step = (i >> 6) / RT;
            const int k = n * 16 + (lane & 15), t = step * 16 + (lane >> 4) * 4;
            store4(to + i * 4, vf4{S[t][k], S[t + 1][k], S[t + 2][k], S[t + 3][k]});
        }
    } else {
        __bf16 *to = reinterpret_cast<__bf16 *>(panels) + 3 * tile * RT * 16 * TM;
        for (int i = threadIdx.x; i < 2 * RT * 64; i += 256) {
            const int lane = i & 63, n = (i >> 6) % RT, step = (i >> 6) / RT;
            const int k = n * 16 + (lane & 15), t = step * 32 + (lane >> 4) * 8;
            vb8 term[3];
#pragma unroll
            for (int j = 0; j < 8; ++j) put_terms(S[t + j][k], j, term);
#pragma unroll
            for (int h = 0; h < 3; ++h)
                *reinterpret_cast<vb8 *>(to + (((step * 3 + h) * RT + n) * 64 + lane) * 8) = term[h];
        }
    }
}

// ---------------------------------------------------------------- expand --
// For a tile of up to 16 rows: s is the B operand, kept for all columns; the
// weights of a step of columns are the A operand, its rows placed on columns so
// that lane (q, c) ends with 16 consecutive bytes of row c, next to those of
// the other lanes q: out never passes through LDS. `row` is the row to read
// (the last one repeated past the tile's end), `out` the row to write or null.
//
// Rows of f32: two tiles of 16 columns a step, tile h at 16 h.
template <typename TX, typename TW, int RT>
struct ExpandStep {
    static constexpr int COLS = 32;
    struct S {
        vf4 v[RT];
        __device__ __forceinline__ void load(const float (*tile)[RT * 16 + 4], int q, int c) {
#pragma unroll
            for (int n = 0; n < RT; ++n) v[n] = *reinterpret_cast<const vf4 *>(&tile[c][n * 16 + q * 4]);
        }
    };
    typename Vec<TW>::v4 w[2][RT];
    vf4 y[2];

    template <bool ACC>
    __device__ __forceinline__ void load(const TX *row, const TW *W, int r, int o0, int q, int c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (ACC) y[h] = load4(row + o0 + 16 * h + 4 * q);
#pragma unroll
            for (int n = 0; n < RT; ++n) {
                const int k = n * 16 + q * 4, kc = k < r ? k : 0;  // r is a multiple of 8
                w[h][n] = *reinterpret_cast<const typename Vec<TW>::v4 *>(
                    ahead(W + (int64_t)(o0 + 16 * h) * r, (unsigned)(c * r + kc) * (unsigned)sizeof(TW)));
            }
        }
    }
    template <bool ACC>
    __device__ __forceinline__ void multiply_store(const S &s, TX *out, int r, int o0, int q) const {
        vf4 v[2][RT], d[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int n = 0; n < RT; ++n) {
                v[h][n] = __builtin_convertvector(w[h][n], vf4);
                if (n * 16 + q * 4 >= r) v[h][n] = vf4{0.f, 0.f, 0.f, 0.f};  // s is zero there
            }
            d[h] = ACC ? y[h] : vf4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int n = 0; n < RT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) d[h] = mfma4(v[h][n][j], s.v[n][j], d[h]);
        if (out) {
#pragma unroll
            for (int h = 0; h < 2; ++h) store4(out + o0 + 16 * h + 4 * q, d[h]);
        }
    }
};

// Elements k .. k + 7 of a row of s of RT * 16 elements, zero past its end, in
// three terms.
template <int RT>
__device__ __forceinline__ void three_terms(const float *row, int k, vb8 (&term)[3]) {
    const bool in = RT > 1 || k < RT * 16;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float at = row[(in ? k : 0) + j];
        put_terms(in ? at : 0.f, j, term);
    }
}

// Rows of 16 bits: four tiles, 64 columns a step; column i of row 4 q' of tile
// 2 g + h is 32 g + 8 q' + 4 h + i.
template <typename T, int RT>
struct ExpandStep16 {
    static constexpr int COLS = 64;
    static constexpr int KS = (RT + 1) / 2;  // steps of 32 ranks
    typedef typename Vec<T>::v V;
    struct S {
        vb8 t[KS][3];
        __device__ __forceinline__ void load(const float (*tile)[RT * 16 + 4], int q, int c) {
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) three_terms<RT>(tile[c], kk * 32 + q * 8, t[kk]);
        }
    };
    V w[4][KS], y[2];

    template <bool ACC>
    __device__ __forceinline__ void load(const T *row, const T *W, int r, int o0, int q, int c) {
        if (ACC) {
#pragma unroll
            for (int g = 0; g < 2; ++g) y[g] = *reinterpret_cast<const V *>(row + o0 + 32 * g + 8 * q);
        }
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                const int k = kk * 32 + q * 8, kc = k < r ? k : 0;
                w[h][kk] = *reinterpret_cast<const V *>(
                    ahead(W + (int64_t)(o0 + 32 * (h >> 1) + 4 * (h & 1)) * r,
                          (unsigned)((8 * (c >> 2) + (c & 3)) * r + kc) * (unsigned)sizeof(T)));
            }
    }
    template <bool ACC>
    __device__ __forceinline__ void multiply_store(const S &s, T *out, int r, int o0, int q) const {
        typedef float F __attribute__((ext_vector_type(8)));
        vf4 d[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) d[h] = vf4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            const bool past = kk * 32 + q * 8 >= r;  // s is zero there
            vb8 v[4][PARTS<T>];
#pragma unroll
            for (int h = 0; h < 4; ++h) split(past ? (V)(T)0 : w[h][kk], v[h]);
#pragma unroll
            for (int p = 0; p < PARTS<T>; ++p)
#pragma unroll
                for (int i = 0; i < terms_for(p); ++i)
#pragma unroll
                    for (int h = 0; h < 4; ++h) d[h] = mfma8(v[h][p], s.t[kk][i], d[h]);
        }
        if (out) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const vf4 u = d[2 * g], v = d[2 * g + 1];
                F f = {u[0], u[1], u[2], u[3], v[0], v[1], v[2], v[3]};
                if (ACC) f += __builtin_convertvector(y[g], F);
                *reinterpret_cast<V *>(out + o0 + 32 * g + 8 * q) = __builtin_convertvector(f, V);
            }
        }
    }
};
template <int RT>
struct ExpandStep<_Float16, _Float16, RT> : ExpandStep16<_Float16, RT> {};
template <int RT>
struct ExpandStep<__bf16, __bf16, RT> : ExpandStep16<__bf16, RT> {};

// A wave's steps (every fourth of [from, to)) over a tile of up to 16 rows.
template <typename TX, typename TW, int RT, bool ACC>
__device__ void expand_tile(const AdaptExpand &a, const Tile &tile, int from, int to, const float (*S)[RT * 16 + 4]) {
    typedef ExpandStep<TX, TW, RT> Step;
    const int lane = threadIdx.x & 63, w = wave();
    const int q = lane >> 4, c = lane & 15;
    const int64_t at = row_of(a.plan, tile.p0 + (c < tile.cnt ? c : tile.cnt - 1));
    TX *row = reinterpret_cast<TX *>(a.out) + (at < 0 ? 0 : at) * a.N, *out = c < tile.cnt && at >= 0 ? row : nullptr;
    typename Step::S s;
    s.load(S, q, c);
    const TW *W = reinterpret_cast<const TW *>(a.W) + (int64_t)tile.e * a.r * a.N;
    const int first = from + w;
    walk<Step, RT <= 4>((to - first + 3) / 4,
                        [&](Step &st, int i) {
                            st.template load<ACC>(row, W, a.r, (first + 4 * i) * Step::COLS, q, c);
                        },
                        [&](const Step &st, int i) {
                            st.template multiply_store<ACC>(s, out, a.r, (first + 4 * i) * Step::COLS, q);
                        });
}

// The same for tiles of up to 64 rows, each wave its 16 of them, by way of
// LDS: the lanes of a load or store have to lie together in memory (see the
// shrink), so here the rows are the A operand and the columns the B operand,
// with column c of tile h standing for column 16 / size * c + h of the step:
// lane (q, c) ends with 16 consecutive bytes of each of rows 4 q .. 4 q + 3,
// 256 bytes of a row in 16 lanes. The step's weights, which lie together, are
// brought into operand order through LDS once for the four waves, in two
// buffers, one barrier a step. 7400 rows of 12288 f32, rank 64, added to y: 198
// us, of which the f32 matrix instructions are busy 83 and HBM 150; 295 by the
// loads above.
//
// Operand slots of 16 bytes: [part of an f16 weight][tile h][group of
// ranks][lane], the 16 lanes c of a q at c ^ (4 q + v) with v counting the
// pieces of four slots in the order they lie in memory: then both the writes
// (along the ranks) and the reads (along the lanes) spread over the banks.
template <typename TX, typename TW, int RT>
struct ExpandLds {
    static constexpr bool WIDE = sizeof(TX) == 4;  // f32 rows: 4 ranks a slot, else 8
    static constexpr int H = 16 / sizeof(TX);      // tiles of a step, and elements of 16 bytes of a row
    static constexpr int COLS = 16 * H;
    static constexpr int KS = WIDE ? RT : (RT + 1) / 2;
    static constexpr int KS_RANKS = WIDE ? 16 : 32;  // of each of the KS
    static constexpr int P = WIDE ? 1 : PARTS<TX>;   // of a weight
    static constexpr int SLOTS = H * KS * 64;
    static constexpr int PART = SLOTS + 64;  // and the spare ones
    static constexpr int BUFFER = P * PART;
    typedef typename Vec<TX>::v V;
    typedef typename std::conditional<WIDE, typename Vec<TW>::v4, vu4>::type Piece;  // a slot's ranks, as they lie
    static constexpr int RANKS = WIDE ? 4 : 8;
    static constexpr int PIECES = (COLS * RT * 16 / RANKS + 255) / 256;  // a thread's, at most

    // Thread i's pieces of the step: piece p holds ranks RANKS (p % per) ..
    // of column p / per, p = i + 256 j.
    static __device__ __forceinline__ void load(Piece (&w)[PIECES], const TW *W, int r, int o0) {
        const int total = COLS * r / RANKS;
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            const int p = threadIdx.x + 256 * j;
            w[j] = *reinterpret_cast<const Piece *>(
                ahead(W + (int64_t)o0 * r, (unsigned)(p < total ? p : 0) * (unsigned)(RANKS * sizeof(TW))));
        }
    }
    // Where they go; those past the step to a spare slot, so that no branch
    // stands before the write (its wait would be for the last step's stores).
    static __device__ __forceinline__ void places(int (&at)[PIECES], int r) {
        const int per = r / RANKS;
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            const int p = threadIdx.x + 256 * j, o = p / per, k = p % per;
            const int h = o % H, c = o / H;
            const int q = k % 4, v = (h * ((per + 3) / 4) + k / 4) & 3;
            at[j] = o < COLS ? (h * KS + k / 4) * 64 + q * 16 + (c ^ (4 * q + v)) : SLOTS;
        }
    }
    static __device__ __forceinline__ void stage(vu4 *lds, const Piece (&w)[PIECES], const int (&at)[PIECES]) {
#pragma unroll
        for (int j = 0; j < PIECES; ++j) {
            if constexpr (WIDE)
                *reinterpret_cast<vf4 *>(lds + at[j]) = __builtin_convertvector(w[j], vf4);
            else {
                vb8 part[P];
                split(__builtin_bit_cast(V, w[j]), part);
#pragma unroll
                for (int p = 0; p < P; ++p) lds[p * PART + at[j]] = __builtin_bit_cast(vu4, part[p]);
            }
        }
    }
};

// A wave's rows and what the next step needs of memory; the first step's loads
// go out before s is summed.
template <typename TX, typename TW, int RT, bool ACC>
struct ExpandRows {
    typedef ExpandLds<TX, TW, RT> L;
    typedef typename L::V V;
    TX *row[4];
    bool in[4];
    const TW *W;
    typename L::Piece piece[L::PIECES];
    V next[4];

    __device__ __forceinline__ void start(const AdaptExpand &a, const Tile &tile, int step) {
        const int lane = threadIdx.x & 63, q = lane >> 4, c = lane & 15;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = 16 * wave() + 4 * q + i;
            const int64_t at = row_of(a.plan, tile.p0 + (m < tile.cnt ? m : tile.cnt - 1));
            row[i] = reinterpret_cast<TX *>(a.out) + (at < 0 ? 0 : at) * a.N + L::H * c;
            in[i] = m < tile.cnt && at >= 0;
        }
        W = reinterpret_cast<const TW *>(a.W) + (int64_t)tile.e * a.r * a.N;
        load(a.r, step);
    }
    __device__ __forceinline__ void load(int r, int step) {
        L::load(piece, W, r, step * L::COLS);
        if (ACC) {
#pragma unroll
            for (int i = 0; i < 4; ++i) next[i] = *reinterpret_cast<const V *>(row[i] + step * L::COLS);
        }
    }
};

// FULL: every row of the tile is written.
template <typename TX, typename TW, int RT, bool ACC, bool FULL>
__device__ void expand_tile_lds(const AdaptExpand &a, ExpandRows<TX, TW, RT, ACC> &rows, int from, int to,
                                const float (*S)[RT * 16 + 4], vu4 *lds) {
    typedef ExpandLds<TX, TW, RT> L;
    typedef typename L::V V;
    typedef float F __attribute__((ext_vector_type(L::H)));
    const int lane = threadIdx.x & 63, w = wave();
    const int q = lane >> 4, c = lane & 15;
    const int spread = q * 16 + (c ^ (4 * q)), per4 = (a.r / L::RANKS + 3) / 4;  // the lane's slot: see ExpandLds
    // s of row c as the A operand: f32, or three terms
    const int m = 16 * w + c;
    vf4 s[RT];
    vb8 term[L::KS][3];
    if constexpr (L::WIDE) {
#pragma unroll
        for (int n = 0; n < RT; ++n) s[n] = *reinterpret_cast<const vf4 *>(&S[m][n * 16 + q * 4]);
    } else {
#pragma unroll
        for (int kk = 0; kk < L::KS; ++kk) three_terms<RT>(S[m], kk * 32 + q * 8, term[kk]);
    }
    __syncthreads();  // S lies in the same memory as the weights
    if (a.r < L::KS * L::KS_RANKS) {  // ranks past r stay zero
        for (int i = threadIdx.x; i < 2 * L::BUFFER; i += 256) lds[i] = vu4{0, 0, 0, 0};
        __syncthreads();
    }
    int place[L::PIECES];
    L::places(place, a.r);
    // What the next step needs is waited for and put in place behind this step's
    // stores: the loads are older than they, so nothing waits for them. (At the
    // loop's head the wait would have to hold for its first entry too.)
    V old[4];
    auto take = [&](int buffer) {
        L::stage(lds + buffer * L::BUFFER, rows.piece, place);
        if (ACC) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                old[i] = rows.next[i];
                asm volatile("" : "+v"(old[i]));
            }
        }
        __syncthreads();
    };
    if (from < to) take(0);
    for (int step = from; step < to; ++step) {
        const vu4 *buf = lds + ((step - from) & 1) * L::BUFFER;
        rows.load(a.r, step + 1 < to ? step + 1 : step);  // no branch: see walk
        __builtin_amdgcn_sched_barrier(0);
        vf4 d[L::H];
#pragma unroll
        for (int h = 0; h < L::H; ++h) {
            d[h] = vf4{0.f, 0.f, 0.f, 0.f};
            if constexpr (L::WIDE && ACC) {
#pragma unroll
                for (int i = 0; i < 4; ++i) d[h][i] = old[i][h];
            }
        }
        // groups of four tiles of one part; the next group's reads are in flight while one is multiplied
        constexpr int SETS = L::H / 4, GROUPS = L::KS * L::P * SETS;
        vu4 slot[2][4];
        auto read = [&](int g, int t) {
            const int kk = g / SETS / L::P, h = g % SETS * 4 + t;
            return buf[g / SETS % L::P * L::PART + (h * L::KS + kk) * 64 + (spread ^ ((h * per4 + kk) & 3))];
        };
#pragma unroll
        for (int t = 0; t < 4; ++t) slot[0][t] = read(0, t);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const int kk = g / SETS / L::P, h = g % SETS * 4;
            if (g + 1 < GROUPS) {
#pragma unroll
                for (int t = 0; t < 4; ++t) slot[(g + 1) & 1][t] = read(g + 1, t);
            }
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (L::WIDE) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        d[h + t] = mfma4(s[kk][j], __builtin_bit_cast(vf4, slot[g & 1][t])[j], d[h + t]);
            } else {
#pragma unroll
                for (int i = 0; i < terms_for(g / SETS % L::P); ++i)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        d[h + t] = mfma8(term[kk][i], __builtin_bit_cast(vb8, slot[g & 1][t]), d[h + t]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            F f;
#pragma unroll
            for (int h = 0; h < L::H; ++h) f[h] = d[h][i];
            if constexpr (!L::WIDE) {
                if (ACC) f += __builtin_convertvector(old[i], F);
            }
            if (FULL || rows.in[i])
                *reinterpret_cast<V *>(rows.row[i] + step * L::COLS) = __builtin_convertvector(f, V);
        }
        __builtin_amdgcn_sched_barrier(0);
        take((step + 1 - from) & 1);
    }
}

// A workgroup's share of the zeros in rows without an adapter.
template <typename TX>
__device__ void zero_rows(const AdaptExpand &a, const Tile &tile, int chunk, int chunks, int threads) {
    const int64_t n = (int64_t)a.N * sizeof(TX) / 16, lo = n * chunk / chunks, hi = n * (chunk + 1) / chunks;
    for (int m = 0; m < tile.cnt; ++m) {
        const int64_t row = row_of(a.plan, tile.p0 + m);
        if (row < 0) continue;
        vu4 *out = reinterpret_cast<vu4 *>(reinterpret_cast<TX *>(a.out) + row * a.N);
        for (int64_t i = lo + threadIdx.x; i < hi; i += threads) out[i] = vu4{0, 0, 0, 0};
    }
}

// One workgroup's part of the grid: 64 rows x a range of columns. The prologue
// adds the splits' partials; the workgroups of the first range also write s out.
template <typename TX, typename TW, int RT, bool ACC>
struct ExpandBlock {
    typedef ExpandLds<TX, TW, RT> Lds;
    static constexpr int S_BYTES = sizeof(float) * TM * (RT * 16 + 4), W_BYTES = 2 * 16 * Lds::BUFFER;
    static constexpr int SHARED = S_BYTES > W_BYTES ? S_BYTES : W_BYTES;  // s, then the weights
    static constexpr int BYTES = SHARED + 16;

    static __device__ void run(const AdaptExpand &a, int chunks, int block, char *lds) {
        float(*S)[RT * 16 + 4] = reinterpret_cast<float(*)[RT * 16 + 4]>(lds);
        int &named = *reinterpret_cast<int *>(lds + SHARED);
        const int chunk = block % chunks;
        const Tile tile = find_tile<false>(a.plan, a.plan.E + 1, TM, block / chunks);
        if (tile.e < 0) return;
        const bool none = tile.e == a.plan.E, large = tile.cnt > 16;
        const int64_t steps = a.N / Lds::COLS;
        const int from = (int)(steps * chunk / chunks), to = (int)(steps * (chunk + 1) / chunks);
        ExpandRows<TX, TW, RT, ACC> own;
        if (large && !none) own.start(a, tile, from < steps ? from : 0);
        const float scale = a.scale && !none ? a.scale[tile.e] : 1.f;
        if (threadIdx.x < TM) {  // one wave
            const bool ok = threadIdx.x < tile.cnt && row_of(a.plan, tile.p0 + threadIdx.x) >= 0;
            if (threadIdx.x == 0) named = 0;
            if (__ballot(ok) == ~0ull && threadIdx.x == 0) named = 1;
        }
        const int rows = tile.cnt <= 16 ? 16 : TM;
        for (int i = threadIdx.x; i < rows * RT * 4; i += 256) {
            const int m = i / (RT * 4), k = i % (RT * 4) * 4;
            vf4 sum = {0.f, 0.f, 0.f, 0.f};
            if (m < tile.cnt && k < a.r) {  // r is a multiple of 8
                if (!none) {
                    const float *part = a.part + (int64_t)(tile.p0 + m) * a.r + k;
                    const int64_t next = (int64_t)a.plan.M * a.r;
#pragma unroll 8
                    for (int sp = 0; sp < a.splits; ++sp) sum += load4(part + sp * next);
                }
                if (chunk == 0 && a.s_row) {
                    const int64_t row = row_of(a.plan, tile.p0 + m);
                    if (row >= 0) store4(a.s_row + row * a.r + k, sum);
                }
            }
            *reinterpret_cast<vf4 *>(&S[m][k]) = scale * sum;
        }
        if (none && ACC) return;
        __syncthreads();
        if (none) {
            zero_rows<TX>(a, tile, chunk, chunks, 256);
            return;
        }
        if (!large) {
            const int64_t steps = a.N / ExpandStep<TX, TW, RT>::COLS;
            const int from = (int)(steps * chunk / chunks), to = (int)(steps * (chunk + 1) / chunks);
            expand_tile<TX, TW, RT, ACC>(a, tile, from, to, S);
        } else if (named) {
            expand_tile_lds<TX, TW, RT, ACC, true>(a, own, from, to, S, reinterpret_cast<vu4 *>(lds));
        } else {
            expand_tile_lds<TX, TW, RT, ACC, false>(a, own, from, to, S, reinterpret_cast<vu4 *>(lds));
        }
    }
};

// -------------------------------------------------------------- gradients --
// Rows past a range's end: zeros, so that they add nothing whatever a real row
// holds. A wave reads up to 64 columns of a row.
__device__ float zero_row[64];  // never written; not const, or its loads would not be global ones

// X as the A operand, straight from its rows: lane (q, c) loads columns
// 4 c .. 4 c + 3, component u belonging to tile u of the output (so that row m
// of tile u stands for column 4 m + u), of the rows q of the step's k indices.
// The thin operand's panel gives B[k][rank] from LDS. D then holds
// G[column 4 (4 q + i) + u][rank c].
//
// Rows of f32: 16 a step, k index 4 q + j.
template <typename TX, int RT>
struct GradStep {
    static constexpr int ROWS = 16;
    static constexpr int SLOTS = RT * 64;  // of a step's panel
    vf4 x[4];

    template <bool ONCE>
    __device__ __forceinline__ void load(const TX *X, int N, const int *row, int q, int c) {
        const int4 at = *reinterpret_cast<const int4 *>(row + 4 * q);
        const int r[4] = {at.x, at.y, at.z, at.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] =
                fetch<ONCE, vf4>((r[j] < 0 ? reinterpret_cast<const TX *>(zero_row) : X + (int64_t)r[j] * N) + 4 * c);
    }
    __device__ __forceinline__ void multiply(const vu4 *panel, vf4 (&acc)[4][RT], int lane) const {
        vf4 t[RT];
#pragma unroll
        for (int n = 0; n < RT; ++n) t[n] = __builtin_bit_cast(vf4, panel[n * 64 + lane]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int n = 0; n < RT; ++n)
#pragma unroll
                for (int u = 0; u < 4; ++u) acc[u][n] = mfma4(x[j][u], t[n][j], acc[u][n]);
    }
};

// Rows of 16 bits: 32 a step, k index 8 q + j, on the bf16 instruction. The
// gradients are f32, so the thin operand takes part with 24 leading bits, in
// three bf16 terms; an f16 element of X is exactly two (11 bits in 8 + 3), and
// the product of its second with the third term, 2^-25 of the whole at most,
// is left out.
template <typename T, int RT>
struct GradStep16 {
    static constexpr int ROWS = 32;
    static constexpr int SLOTS = 3 * RT * 64;
    vu2 x[8];  // four elements

    template <bool ONCE>
    __device__ __forceinline__ void load(const T *X, int N, const int *row, int q, int c) {
        const int4 a = *reinterpret_cast<const int4 *>(row + 8 * q);
        const int4 b = *reinterpret_cast<const int4 *>(row + 8 * q + 4);
        const int r[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = fetch<ONCE, vu2>((r[j] < 0 ? reinterpret_cast<const T *>(zero_row) : X + (int64_t)r[j] * N) + 4 * c);
    }
    __device__ __forceinline__ void multiply(const vu4 *panel, vf4 (&acc)[4][RT], int lane) const {
        vb8 hi[4], lo[4];
        vu4 t[2][RT];  // the next term's reads are in flight while one is multiplied
#pragma unroll
        for (int n = 0; n < RT; ++n) t[0][n] = panel[n * 64 + lane];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if constexpr (__is_same(T, __bf16)) {
                vu4 pairs;  // element u of two rows each
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const vu2 even = x[2 * j], odd = x[2 * j + 1];
                    pairs[j] = __builtin_amdgcn_perm(u < 2 ? odd.x : odd.y, u < 2 ? even.x : even.y,
                                                     u & 1 ? 0x07060302u : 0x05040100u);
                }
                hi[u] = __builtin_bit_cast(vb8, pairs);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float v = (float)__builtin_bit_cast(vh4, x[j])[u];
                    hi[u][j] = take_term(v);
                    lo[u][j] = take_term(v);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 3; ++h) {
            if (h < 2) {
#pragma unroll
                for (int n = 0; n < RT; ++n) t[(h + 1) & 1][n] = panel[((h + 1) * RT + n) * 64 + lane];
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int n = 0; n < RT; ++n)
#pragma unroll
                for (int u = 0; u < 4; ++u) acc[u][n] = mfma8(hi[u], __builtin_bit_cast(vb8, t[h & 1][n]), acc[u][n]);
            if constexpr (!__is_same(T, __bf16)) {
                if (h < 2) {
#pragma unroll
                    for (int n = 0; n < RT; ++n)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            acc[u][n] = mfma8(lo[u], __builtin_bit_cast(vb8, t[h & 1][n]), acc[u][n]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
};
template <int RT>
struct GradStep<_Float16, RT> : GradStep16<_Float16, RT> {};
template <int RT>
struct GradStep<__bf16, RT> : GradStep16<__bf16, RT> {};

// One workgroup's part of the grid of job `which`: a range of one adapter's
// rows x 256 columns, wave w 64 of them. A panel of 64 rows is up to three
// times as many bytes as the 64 columns it meets, so the four waves share it
// through LDS (in two buffers, one barrier a panel); the next panel and one
// or three steps' rows are in flight while a step is multiplied. Both gradients
// of 28500 rows of 22528 columns in all, bf16, rank 64, took 360 us in a launch
// of their own (3.6 TB/s), 520 with panels read by each wave for itself and 3800
// on f32 instructions.
template <typename TX, int RT>
struct GradBlock {
    typedef GradStep<TX, RT> Step;
    static constexpr int STEPS = TM / Step::ROWS, SLOTS = STEPS * Step::SLOTS, PIECES = (SLOTS + 255) / 256;
    static constexpr int SETS = RT <= 2 ? 4 : 2;  // of rows in flight or use; more would spill
    static_assert(4 % STEPS == 0 && 4 % SETS == 0, "the sets go round with the panels");
    static constexpr int BYTES = 4 * ADAPT_MAX_RANGE + 2 * 16 * SLOTS;

    template <bool ONCE>
    static __device__ void run(const AdaptGrad &a, int which, int block, char *shared) {
        int *row = reinterpret_cast<int *>(shared);
        vu4(*lds)[SLOTS] = reinterpret_cast<vu4(*)[SLOTS]>(shared + 4 * ADAPT_MAX_RANGE);
        const AdaptGradJob &job = a.job[which];
        const int N = job.N, across = (N + 255) / 256, col = block % across;
        const Tile tile = find_tile<true>(a.plan, a.plan.E, a.range, block / across);
        if (tile.e < 0) return;
        const int first = tile.panel + tile.j * (a.range / TM), panels = (tile.cnt + TM - 1) / TM;
        // only offsets out of order can count more panels or partials than there are
        if (first + panels > a.panels || (tile.of > 1 && tile.slot + tile.j >= a.slots)) return;
        const int lane = threadIdx.x & 63, w = wave();
        const int q = lane >> 4, c = lane & 15;
        const int n0 = col * 256 + w * 64;
        // waves past the last column repeat column 0, for the barriers; not stored
        const TX *X = reinterpret_cast<const TX *>(job.X) + (n0 < N ? n0 : 0);
        const vu4 *panel = reinterpret_cast<const vu4 *>(job.panel) + (int64_t)first * SLOTS;
        vf4 acc[4][RT];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int n = 0; n < RT; ++n) acc[u][n] = vf4{0.f, 0.f, 0.f, 0.f};
        vu4 piece[PIECES];
        auto load_panel = [&](int p) {
#pragma unroll
            for (int j = 0; j < PIECES; ++j) {
                const unsigned i = threadIdx.x + 256 * j;
                piece[j] = *ahead(panel + (int64_t)p * SLOTS, (SLOTS % 256 == 0 || i < SLOTS ? i : 0) * 16u);
            }
        };
        load_panel(0);
        for (int i = threadIdx.x; i < panels * TM; i += 256)
            row[i] = i < tile.cnt ? (int)row_of(a.plan, tile.p0 + i) : -1;
        __syncthreads();
        // no branch around a load (see walk): past the end the last step again
        const int steps = panels * STEPS;
        Step set[SETS];
        auto load_rows = [&](Step &st, int step) {
            st.template load<ONCE>(X, N, row + (step < steps ? step : steps - 1) * Step::ROWS, q, c);
        };
#pragma unroll
        for (int i = 0; i < SETS - 1; ++i) load_rows(set[i], i);
        for (int p = 0; p < panels; p += 4 / STEPS) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int at = p + s / STEPS;  // the panel
                vu4 *buf = lds[at & 1];
                if (s % STEPS == 0) {
                    if (s > 0 && at >= panels) break;
#pragma unroll
                    for (int j = 0; j < PIECES; ++j) {
                        const int i = threadIdx.x + 256 * j;
                        if (SLOTS % 256 == 0 || i < SLOTS) buf[i] = piece[j];
                    }
                    __syncthreads();
                    load_panel(at + 1 < panels ? at + 1 : at);
                }
                load_rows(set[(s + SETS - 1) % SETS], p * STEPS + s + SETS - 1);
                __builtin_amdgcn_sched_barrier(0);
                set[s % SETS].multiply(buf + s % STEPS * Step::SLOTS, acc, lane);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (n0 >= N) return;
        const int64_t size = (int64_t)a.r * N;
        const bool alone = tile.of == 1;
        float *g = alone ? job.grad + tile.e * size : job.part + (tile.slot + tile.j) * size;
        const bool add = alone && a.acc;
        const float scale = job.scale ? job.scale[tile.e] : 1.f;
#pragma unroll
        for (int n = 0; n < RT; ++n) {
            const int k = n * 16 + c;
            if (k >= a.r) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const vf4 v = scale * vf4{acc[0][n][i], acc[1][n][i], acc[2][n][i], acc[3][n][i]};
                const int o = n0 + 16 * q + 4 * i;
                if (which == 0) {
                    float *at = g + (int64_t)k * N + o;
                    store4(at, add ? load4(at) + v : v);
                } else {
                    float *at = g + (int64_t)o * a.r + k;
#pragma unroll
                    for (int u = 0; u < 4; ++u) at[u * a.r] = add ? at[u * a.r] + v[u] : v[u];
                }
            }
        }
    }
};

// Calls F<TX, TW, RT> for the call's types and rank.
#define BLR_BY_RANK(r, F, TX, TW, ...)                                                          \
    ((r) <= 16   ? F<TX, TW, 1>(__VA_ARGS__)                                                     \
     : (r) <= 32 ? F<TX, TW, 2>(__VA_ARGS__)                                                     \
     : (r) <= 64 ? F<TX, TW, 4>(__VA_ARGS__)                                                     \
                 : F<TX, TW, 8>(__VA_ARGS__))
#define BLR_BY_TYPES(a, F, ...)                                                                  \
    ((a).act == 1   ? BLR_BY_RANK((a).r, F, _Float16, _Float16, __VA_ARGS__)                     \
     : (a).act == 2 ? BLR_BY_RANK((a).r, F, __bf16, __bf16, __VA_ARGS__)                         \
     : (a).wt == 1  ? BLR_BY_RANK((a).r, F, float, _Float16, __VA_ARGS__)                        \
     : (a).wt == 2  ? BLR_BY_RANK((a).r, F, float, __bf16, __VA_ARGS__)                          \
                    : BLR_BY_RANK((a).r, F, float, float, __VA_ARGS__))

}  // namespace
}  // namespace blr
