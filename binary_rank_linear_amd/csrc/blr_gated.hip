// The gated feed-forward for gfx950: h = act(g) * u, g = x Wg^T, u = x Wu^T,
// and its backward, with dense f16 or bf16 rows and weights.
//
//   forward   one contraction over d for both projections; h in its epilogue
//   backward  dg = dh u act'(g), du = dh act(g), side by side as D [M][2 ff]
//             (from the projections kept in 8 bits, or by the forward's
//             contraction again); then dx = D [Wg; Wu] and [dWg; dWu] = D^T x
//
// Products of 16-bit values are exact in the matrix instructions' f32 sums. D
// is rounded to the rows' type once (times gscale, as f16 needs it for small
// gradients): the products after it are of 16 bits. Its rounding, 1.7e-3 (bf16)
// or 2.1e-4 (f16) of a gradient in the 2-norm, is of the size of 16-bit results'
// own, which are off by 2.3e-3 or 2.9e-4 in all; in f32 gradients it is what
// is left.
//
// All three contractions are one kernel over tiles in LDS, bound by the matrix
// units. An operand lies in memory with the contracted index innermost (x and
// the weights of the forward, D of dx) or outermost (the weights of dx, both
// operands of the weights' gradients). Either is copied to LDS as it lies,
// 16 bytes a lane, without passing through registers; the first kind is read
// back 8 contracted values to a lane, the second through the LDS's transposing
// reads. Lanes copy their 16 bytes from a place XORed with the row, which spreads
// the first kind's reads over all banks; the second's of n take half the banks
// at a time (a quarter of dx's and dw's LDS cycles, by the counters).
//
// 8192 rows of bf16, 4096 -> 12288, HIP events: forward 1.31 ms (1.26 PFLOP/s; the
// library's product without the activation 1.29), dx 1.20 (1.37; 1.32), the weights'
// gradients 1.31 (1.26; 1.15); f16 1.37, 1.26 and 1.36. 30000 x 5120 -> 17408, bf16:
// 8.6 ms (1.24), 9.2 with a tape (1.16), dx 8.8 (1.21), the weights' 9.2 (1.16). Some
// cards are 5 % slower in all of them. Copies that always come out of L2 would make them 5,
// 8 and 14 % faster, no copies at all 15, 16 and 24 %: what is left is the matrix
// units' own rate, the LDS's, and the ends of tiles. One row of 4096 -> 12288 takes
// 39 us, its weights' bytes at 5.2 TB/s, one of 5120 -> 17408 84 (4.2).
#include <cfloat>
#include <type_traits>

#include "blr_internal.h"
#include "blr_keep8.h"
#include "blr_math.h"

namespace blr {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
#define LDS_PTR(T) __attribute__((address_space(3))) T *

__device__ __forceinline__ vf4 mma(s16x8 a, s16x8 b, vf4 c, _Float16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(vh8, a), __builtin_bit_cast(vh8, b), c, 0, 0, 0);
}
__device__ __forceinline__ vf4 mma(s16x8 a, s16x8 b, vf4 c, __bf16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(vb8, a), __builtin_bit_cast(vb8, b), c, 0, 0, 0);
}

// act(g) and its slope. gelu is the form with tanh: 0.5 g (1 + tanh y) is
// g sigmoid(2 y), y = sqrt(2 / pi) (g + 0.044715 g^3). Both ends stay finite:
// the exponential is of -|.|.
template <bool GELU>
__device__ __forceinline__ float act(float g, float *slope) {
    float y = g, dy = 1.0f;
    if constexpr (GELU) {
        const float a = 1.59576912160573071176f, b = 0.044715f;  // 2 sqrt(2 / pi)
        const float gg = g * g;
        y = a * g * fmaf(b, gg, 1.0f);
        dy = a * fmaf(3.0f * b, gg, 1.0f);
    }
    // past 200 the exponential is zero; y itself may be infinite. A NaN stays one.
    if (fabsf(y) > 200.0f) y = copysignf(200.0f, y);
    const float e = exp_of(-fabsf(y)), big = inverse(1.0f + e), small = e * big;
    const float s = y >= 0.0f ? big : small;
    // far out the slope's second term is zero, whatever y has grown to
    const float r = big * small;
    *slope = r == 0.0f ? s : fmaf(g * dy, r, s);
    return fmaxf(g, -FLT_MAX) * s;  // s is zero where g is minus infinity
}
// h = act(g) u of eight columns, in place of g. The kind is looked at once, so
// that the eight go through the long chain side by side.
__device__ __forceinline__ void products8(int kind, float *g, const float *u) {
    auto all = [&](auto gelu) {
        float unused;
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = act<decltype(gelu)::value>(g[i], &unused) * u[i];
    };
    if (kind)
        all(std::true_type());
    else
        all(std::false_type());
}
// dg = v u act'(g) and du = v act(g), in place of g and u. The slope is at most
// 1.13, so that its product with u stays in range where v u may not.
__device__ __forceinline__ void gradients8(int kind, const float *v, float *g, float *u) {
    auto all = [&](auto gelu) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float slope;
            const float a = act<decltype(gelu)::value>(g[i], &slope);
            g[i] = v[i] * (u[i] * slope);
            u[i] = v[i] * a;
        }
    };
    if (kind)
        all(std::true_type());
    else
        all(std::false_type());
}

// ------------------------------------------------------------ contraction --
// out[m][n] = sum_k A(m, k) B(n, k), tiles of BM x BN by 2 x BN / 64 waves, each
// BM / 2 rows by 64 columns, in steps of 64 over k. The matrix instruction's
// rows are n and its columns m, so that a lane holds neighbouring n of one m.
constexpr int BK = 64;

// n of row p (0 .. 15) of instruction tile j (0 .. 3) in a wave's 64 columns:
// a lane has rows 4 (lane / 16) + 0 .. 3 of each tile, which makes 16
// neighbouring columns; gated, 8 neighbouring columns of the gate (j = 0, 1)
// and the same 8 of up (j = 2, 3).
__device__ __forceinline__ int col_of(bool gated, int j, int p) {
    return gated ? (p >> 2) * 8 + (j & 1) * 4 + (p & 3) : (p >> 2) * 16 + j * 4 + (p & 3);
}

__device__ __forceinline__ i32x4 resource(const void *p, uint32_t bytes) {
    const uint64_t a = (uint64_t)p;
    i32x4 r = {__builtin_amdgcn_readfirstlane((int)(uint32_t)a), __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
    return r;
}
// 16 bytes a lane from rsrc + voff to LDS at lds + 16 lane; zeros from past the
// resource's end. It is complete after a wait for vmcnt.
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is always the compiler's; it is named below all the same
__device__ __forceinline__ void copy_to_lds(i32x4 rsrc, int voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(rsrc)
                 : "memory", "m0");
}
// All but the last N copies have arrived, and every read of LDS.
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void barrier() {
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

enum Role { FORWARD, AGAIN, DX, DW };

// XOR of a 16-byte place in an LDS row of the second kind, by its contracted
// index: rows of the matrix instruction's columns (m) take 32 bytes of each of
// 8 LDS rows at once, those of its rows (n) 8 bytes of 4 places in each.
__device__ __forceinline__ int twist_m(int k) { return ((k & 3) | ((k >> 1) & 4)) << 1; }
__device__ __forceinline__ int twist_n(int k) { return (k & 1) | (k & 8); }

// Eight elements of a product go out, scaled, and added to what is there where
// the call says so.
template <typename T>
__device__ __forceinline__ void put_product(const GatedGemm &a, char *out, int64_t at, float *v) {
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= a.scale;
    auto put = [&](auto *q) {
        using O = typename std::remove_pointer<decltype(q)>::type;
        if (a.acc) {
            widen8(raw8(q), o);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += o[e];
        }
        put8(q, narrow8<O>(v));
    };
    if (a.out_f32)
        put((float *)out + at);
    else
        put((T *)out + at);
}

template <typename T, Role R, int BM, int BN, int STEPS>
struct Tile {
    static constexpr bool gated = R == FORWARD || R == AGAIN;
    static constexpr bool a_inner = R != DW, b_inner = gated;  // contracted index innermost
    static constexpr int WN = BN / 64, WAVES = 2 * WN, MT = BM / 32;
    static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, STAGE = A_BYTES + B_BYTES;
    // copies of 1 KB by each wave: of either operand, and of both
    static constexpr int A_COPIES = A_BYTES / WAVES / 1024, B_COPIES = B_BYTES / WAVES / 1024, COPIES = A_COPIES + B_COPIES;
    static_assert(A_BYTES == A_COPIES * WAVES * 1024 && B_COPIES == 4, "copies fill the tiles, four of 8 rows of n each");
};

template <typename T, Role R, int BM, int BN, int STEPS>
__global__ __launch_bounds__(128 * (BN / 64)) void gated_kernel(GatedGemm a) {
    using G = Tile<T, R, BM, BN, STEPS>;
    __shared__ __attribute__((aligned(1024))) char smem[STEPS * G::STAGE];
    const uint32_t lds0 = (uint32_t)(uintptr_t)(LDS_PTR(char))smem;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = w % G::WN, wm = w / G::WN, p = lane & 15, g4 = lane >> 4;

    // tiles of one XCD lie together, a group of rows' tiles beside each column's
    int64_t tile = blockIdx.x;
    {
        const int64_t total = gridDim.x, per = total / 8, rest = total % 8, x = tile % 8;
        tile = x * per + (x < rest ? x : rest) + tile / 8;
    }
    const int64_t split = R == DX ? tile / (a.tiles_m * a.tiles_n) : 0;
    tile -= split * a.tiles_m * a.tiles_n;
    const int64_t group = tile / (a.group * a.tiles_n), in_group = tile % (a.group * a.tiles_n);
    const int64_t first = group * a.group, rows = a.tiles_m - first < a.group ? a.tiles_m - first : a.group;
    const int64_t m0 = (first + in_group % rows) * BM;
    const int n0 = (int)(in_group / rows) * (G::gated ? BN / 2 : BN);

    // what each lane copies: byte offsets from the tile's corner
    int off_a[G::A_COPIES], off_b[G::B_COPIES];
#pragma unroll
    for (int i = 0; i < G::A_COPIES; ++i) {
        const int c = w * G::A_COPIES + i;  // 1 KB of the tile
        if constexpr (G::a_inner) {
            const int row = c * 8 + (lane >> 3), at = (lane & 7) ^ (row & 7);
            const int64_t left = a.M - 1 - m0;
            const int64_t r = row < left ? row : left;  // rows past the last one are that one
            off_a[i] = (int)(r * a.lda * 2 + at * 16);
        } else {
            constexpr int PLACES = BM / 8;
            const int k = (c * 64 + lane) / PLACES, at = ((c * 64 + lane) % PLACES) ^ twist_m(k);
            off_a[i] = (int)(k * a.lda * 2 + at * 16);
            if (m0 + at * 8 >= a.M) off_a[i] = 0x7fffffff;  // past every resource's end: zeros
        }
    }
#pragma unroll
    for (int i = 0; i < G::B_COPIES; ++i) {
        const int c = w * G::B_COPIES + i;
        if constexpr (G::b_inner) {
            const int row = c * 8 + (lane >> 3), at = (lane & 7) ^ (row & 7);
            const int n = (row >> 6) * 32 + col_of(true, (row >> 4) & 3, row & 15);
            off_b[i] = (int)((int64_t)n * a.ldb * 2 + at * 16);
        } else {
            constexpr int PLACES = BN / 8;
            const int k = (c * 64 + lane) / PLACES, at = ((c * 64 + lane) % PLACES) ^ twist_n(k);
            off_b[i] = (int)(k * a.ldb * 2 + at * 16);
            if (n0 + at * 8 >= a.N) off_b[i] = 0x7fffffff;
        }
    }
    const char *pa = (const char *)a.A + (G::a_inner ? m0 * a.lda * 2 : m0 * 2);
    // forward: of the LDS rows that a wave copies all are of the gate or all of up
    const char *pb = (const char *)(G::b_inner && (w & 1) ? a.B2 : a.B) + (G::b_inner ? (int64_t)n0 * a.ldb * 2 : (int64_t)n0 * 2);
    const int64_t hop = (const char *)a.B2 - (const char *)a.B;

    // where a step's copies come from and go to
    struct Source {
        i32x4 a, b;
        uint32_t to;
    };
    auto source = [&](int64_t k0, int buf) {
        Source q;
        q.to = lds0 + buf * G::STAGE;
        const int64_t left = a.K - k0 < BK ? a.K - k0 : BK;
        q.a = G::a_inner ? resource(pa + k0 * 2, 0x7ffffffe)
                         : resource(pa + k0 * a.lda * 2, (uint32_t)((left * a.lda - m0) * 2));
        const char *b = pb;
        if constexpr (G::b_inner) {
            q.b = resource(b + k0 * 2, 0x7ffffffe);
        } else {
            // dx: the contraction runs through Wg, then Wu
            int64_t kb = k0;
            if (R == DX && k0 >= a.K / 2) b += hop, kb -= a.K / 2;
            q.b = resource(b + kb * a.ldb * 2, (uint32_t)((left * a.ldb - n0) * 2));
        }
        // a vector instruction may have written them last, and the copies, which
        // the compiler does not see as loads, need five cycles' distance from it
        asm volatile("s_nop 4" : "+s"(q.a), "+s"(q.b));
        return q;
    };
    auto copy = [&](const Source &q, int i) {
        if (i < G::A_COPIES)
            copy_to_lds(q.a, off_a[i], q.to + (w * G::A_COPIES + i) * 1024);
        else if (i < G::COPIES)
            copy_to_lds(q.b, off_b[i - G::A_COPIES], q.to + G::A_BYTES + (w * G::B_COPIES + i - G::A_COPIES) * 1024);
    };
    auto stage = [&](int64_t k0, int buf) {
        const Source q = source(k0, buf);
#pragma unroll
        for (int i = 0; i < G::COPIES; ++i) copy(q, i);
    };

    // an operand's 16 x 32 piece: lane = row (p), 8 contracted values (8 g4 on)
    auto frag_a = [&](const char *s, int i, int kk) -> s16x8 {
        if constexpr (G::a_inner) {
            const int row = wm * (BM / 2) + i * 16 + p, at = (kk * 4 + g4) ^ (p & 7);
            return *(const s16x8 *)(s + row * (BK * 2) + at * 16);
        } else {
            s16x8 v;
            const int r = p >> 2, c = p & 3;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = kk * 32 + g4 * 8 + h * 4 + r;
                const int at = ((wm * (BM / 2) + i * 16) / 8 + (c >> 1)) ^ twist_m(g4 * 8 + r);
                const s16x4 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (LDS_PTR(s16x4))(s + k * (BM * 2) + at * 16 + (c & 1) * 8));
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * h + e] = q[e];
            }
            return v;
        }
    };
    auto frag_b = [&](const char *s, int j, int kk) -> s16x8 {
        if constexpr (G::b_inner) {
            const int row = wn * 64 + j * 16 + p, at = (kk * 4 + g4) ^ (p & 7);
            return *(const s16x8 *)(s + row * (BK * 2) + at * 16);
        } else {
            s16x8 v;
            const int r = p >> 2, c = p & 3;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = kk * 32 + g4 * 8 + h * 4 + r;
                const int at = (wn * 8 + c * 2 + (j >> 1)) ^ twist_n(g4 * 8 + r);
                const s16x4 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (LDS_PTR(s16x4))(s + k * (BN * 2) + at * 16 + (j & 1) * 8));
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * h + e] = q[e];
            }
            return v;
        }
    };

    vf4 acc[G::MT][4];
#pragma unroll
    for (int i = 0; i < G::MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = vf4{};

    // this workgroup's steps of the contraction: all, or a split's
    const int64_t k_first = split * a.split_steps * BK;
    int steps = (int)((a.K - k_first + BK - 1) / BK);
    if (R == DX && steps > a.split_steps) steps = (int)a.split_steps;
    s16x8 xa[G::MT], xb[4], ya[G::MT], yb[4];
    // piece r of a half step's operands: n's four, then m's
    auto read = [&](s16x8 *fa, s16x8 *fb, int buf, int kk, int r) {
        const char *s = smem + buf * G::STAGE;
        if (r < 4)
            fb[r] = frag_b(s + G::A_BYTES, r, kk);
        else if (r < 4 + G::MT)
            fa[r - 4] = frag_a(s, r - 4, kk);
    };
    auto multiply = [&](const s16x8 *fa, const s16x8 *fb, int i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mma(fb[j], fa[i], acc[i][j], T());
    };
    // Reads and copies are handed out among the products, so that the matrix
    // units start at once after the barrier; the order is the one written.
    constexpr int ROWS = G::a_inner ? G::MT / 2 : G::MT * 3 / 4;  // rows of products that take reads
    constexpr int READS = (4 + G::MT + ROWS - 1) / ROWS;
    constexpr int COPIES = (G::COPIES + G::MT / 2 - 1) / (G::MT / 2);
    auto step = [&](int t, auto copies, auto reads) {
        const int buf = t % STEPS, next = (t + 1) % STEPS;
#pragma unroll
        for (int i = 0; i < G::MT; ++i) {
            if (i < ROWS)
#pragma unroll
                for (int r = 0; r < READS; ++r) read(ya, yb, buf, 1, i * READS + r);
            multiply(xa, xb, i);
            __builtin_amdgcn_sched_barrier(0);
        }
        // of the steps after the next one, as many as there are may be on their way
        if constexpr (decltype(copies)::value)
            wait_copies<G::COPIES *(STEPS - 2)>();
        else if (STEPS > 3 && t + 3 < steps)
            wait_copies<2 * G::COPIES>();
        else if (STEPS > 2 && t + 2 < steps)
            wait_copies<G::COPIES>();
        else
            wait_copies<0>();
        barrier();
        __builtin_amdgcn_sched_barrier(0);
        Source q;
        if constexpr (decltype(copies)::value) q = source(k_first + (int64_t)(t + STEPS) * BK, buf);
#pragma unroll
        for (int i = 0; i < G::MT; ++i) {
            if (decltype(copies)::value && i < G::MT / 2)
#pragma unroll
                for (int c = 0; c < COPIES; ++c) copy(q, i * COPIES + c);
            if (decltype(reads)::value && i < ROWS)
#pragma unroll
                for (int r = 0; r < READS; ++r) read(xa, xb, next, 0, i * READS + r);
            multiply(ya, yb, i);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    // A step's second half is read while the first multiplies, the next step's
    // first half while the second does; between them one barrier, at which the
    // step's buffer is free and the next one's copies have arrived. With STEPS
    // buffers a step's copies have STEPS - 1 steps to arrive in.
    using Yes = std::true_type;
    using No = std::false_type;
    static_assert(STEPS <= 4, "the waits at the end tell up to three steps apart");
    for (int i = 0; i < STEPS && i < steps; ++i) stage(k_first + (int64_t)i * BK, i);
    if (steps < STEPS)
        wait_copies<0>();
    else
        wait_copies<G::COPIES *(STEPS - 1)>();
    barrier();
#pragma unroll
    for (int r = 0; r < 4 + G::MT; ++r) read(xa, xb, 0, 0, r);
    int t = 0;
    for (; t + STEPS < steps; ++t) step(t, Yes(), Yes());
    for (; t + 1 < steps; ++t) step(t, No(), Yes());
    step(t, No(), No());

    // lane: row m, columns from n on
#pragma unroll
    for (int i = 0; i < G::MT; ++i) {
        const int64_t m = m0 + wm * (BM / 2) + i * 16 + p;
        if (m >= a.M) continue;  // whole quads of lanes with the same p
        if constexpr (G::gated) {
            const int n = n0 + wn * 32 + g4 * 8;
            float gate[8], up[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                gate[e] = acc[i][e >> 2][e & 3];
                up[e] = acc[i][2 + (e >> 2)][e & 3];
            }
            const int64_t at = m * a.ff + n;
            if constexpr (R == FORWARD) {
                if (a.tape_q) {
                    // the 32 columns of a block are those of the four lanes with this row
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float *v = h ? up : gate;
                        uint32_t top = top8(v);
                        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
                        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
                        const int b = keep_exponent(top, KEEP_MAX<float>);
                        *(uint2 *)(a.tape_q + h * a.M * a.ff + at) = keep8(v, b);
                        if (g4 == 0) a.tape_b[(h * a.M * a.ff + at) / 32] = (uint8_t)b;
                    }
                }
                products8(a.kind, gate, up);
                if (a.out_f32)
                    put8((float *)a.out + at, narrow8<float>(gate));
                else
                    put8((T *)a.out + at, narrow8<T>(gate));
            } else {
                float dh[8];
                if (a.out_f32)
                    widen8(raw8((const float *)a.dh + at), dh);
                else
                    widen8(raw8((const T *)a.dh + at), dh);
#pragma unroll
                for (int e = 0; e < 8; ++e) dh[e] *= a.scale;
                gradients8(a.kind, dh, gate, up);
                T *d = (T *)a.out + m * 2 * a.ff + n;
                put8(d, narrow8<T>(gate));
                put8(d + a.ff, narrow8<T>(up));
            }
        } else {
            const int n = n0 + wn * 64 + g4 * 16;
            if (n >= a.N) continue;  // N is a multiple of 16
            if (R == DX && a.splits > 1) {
                float *q = a.part + (split * a.M + m) * a.N + n;
#pragma unroll
                for (int j = 0; j < 4; ++j) ((vf4 *)q)[j] = acc[i][j];
                continue;
            }
            char *out = (char *)a.out;
            int64_t row = m;
            if (R == DW && m >= a.M / 2) {
                out = (char *)a.out2;
                row -= a.M / 2;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = acc[i][2 * h + (e >> 2)][e & 3];
                put_product<T>(a, out, row * a.N + n + 8 * h, v);
            }
        }
    }
}

// The splits' products summed in order.
template <typename T>
__global__ __launch_bounds__(256) void gated_sum_kernel(GatedGemm a) {
    const int64_t n = a.M * a.N, grid = (int64_t)gridDim.x * 2048;
    for (int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; at < n; at += grid) {
        float v[8], o[8];
        widen8(raw8(a.part + at), v);
        for (int q = 1; q < a.splits; ++q) {
            widen8(raw8(a.part + q * n + at), o);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += o[e];
        }
        put_product<T>(a, (char *)a.out, at, v);
    }
}

// D from the projections kept in 8 bits: rows down the grid's y, 8 columns a
// thread along x. Bound by HBM: 8192 x 12288 in 130 us, 6.2 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void gated_gradients_kernel(GatedGemm a) {
    const int64_t n = 8 * ((int64_t)blockIdx.x * blockDim.x + threadIdx.x), ups = a.M * a.ff;
    if (n >= a.ff) return;
    for (int64_t row = blockIdx.y; row < a.M; row += gridDim.y) {
        const int64_t at = row * a.ff + n;
        float gate[8], up[8], dh[8];
        if (a.out_f32)
            widen8(raw8((const float *)a.dh + at), dh);
        else
            widen8(raw8((const T *)a.dh + at), dh);
        kept8(*(const uint2 *)(a.tape_q + at), a.tape_b[at / 32], gate);
        kept8(*(const uint2 *)(a.tape_q + ups + at), a.tape_b[(ups + at) / 32], up);
#pragma unroll
        for (int e = 0; e < 8; ++e) dh[e] *= a.scale;
        gradients8(a.kind, dh, gate, up);
        T *d = (T *)a.out + row * 2 * a.ff + n;
        put8(d, narrow8<T>(gate));
        put8(d + a.ff, narrow8<T>(up));
    }
}

// Tiles of rows that lie beside each tile of columns, for the caches' sake: with
// 4, 8, 16 and 32 the forward of 30000 x 5120 -> 17408 takes 8.78, 8.66, 9.29
// and 9.67 ms, the weights' gradients of 8192 x 4096 -> 12288 1.32, 1.37, 1.37 and
// 1.39, dx of the former 8.93, 9.09, 9.33 and 9.68.
constexpr int64_t group_of(Role r) { return r == FORWARD || r == AGAIN ? 8 : 4; }

template <typename T, Role R, int BM, int BN, int STEPS>
hipError_t contract(int id, GatedGemm a, hipStream_t s) {
    using G = Tile<T, R, BM, BN, STEPS>;
    a.tiles_m = (a.M + BM - 1) / BM;
    const int64_t cols = G::gated ? BN / 2 : BN, N = G::gated ? a.ff : a.N;
    a.tiles_n = (N + cols - 1) / cols;
    a.group = a.tiles_m < group_of(R) ? a.tiles_m : group_of(R);
    prof_begin(id, s);
    gated_kernel<T, R, BM, BN, STEPS><<<dim3((unsigned)(a.tiles_m * a.tiles_n * a.splits)), dim3(64 * G::WAVES), 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    prof_end(s);
    return e;
}

int64_t tiles(int64_t m, int64_t n, int64_t bm, int64_t bn) { return (m + bm - 1) / bm * ((n + bn - 1) / bn); }

// Which tiles: times in us of the forward, 2048 -> 5504 bf16, for 64, 300, 400, 600
// and 1000 rows:
//   64 x 64, 4 buffers     15  30  41  54  79    256 x 256   46  53  --  --  57
//   64 x 128, 2 buffers    22  24  31  47  59
//   128 x 128, 2 buffers   25  30  32  34  53
// Up to 64 rows the first line ends at ff = 16384. Past it, the first two, bf16:
// 5120 -> 17408 82 against 84 (1 row), 94 against 97 (64); 8192 -> 28672 171 against 174
// and 187 against 169.
template <typename T, Role R>
hipError_t contract(int id, GatedGemm a, hipStream_t s) {
    constexpr bool gated = R == FORWARD || R == AGAIN;
    const int64_t N = gated ? 2 * a.ff : a.N;
    a.splits = 1;
    a.split_steps = (a.K + BK - 1) / BK;
    // A round is one tile of 256 on every CU, or two of 128, which together take
    // 0.62 of its time (8192 rows, 4096 x 12288: 1.27 PFLOP/s against 1.06).
    const int64_t large = (tiles(a.M, N, 256, 256) + 255) / 256, small = (tiles(a.M, N, 128, 128) + 511) / 512;
    if (8 * large <= 5 * small) return contract<T, R, 256, 256, 2>(id, a, s);
    if constexpr (gated) {
        // few rows: small tiles, all on the chip at once; the smallest, two on a
        // CU, with three steps on their way
        if (tiles(a.M, N, 64, 64) <= 512) return contract<T, R, 64, 64, 4>(id, a, s);
        if (tiles(a.M, N, 64, 128) <= 768) return contract<T, R, 64, 128, 2>(id, a, s);
    }
    if constexpr (R == DX) {
        a.splits = gated_splits(a.M, a.N, a.K, &a.split_steps);
        if (a.splits > 1) {
            const hipError_t e = contract<T, R, 128, 128, 2>(id, a, s);
            if (e != hipSuccess) return e;
            const int64_t n = (a.M * a.N / 8 + 255) / 256;
            prof_begin(K_GATED_SUM, s);
            gated_sum_kernel<T><<<dim3((unsigned)(n < 8192 ? n : 8192)), dim3(256), 0, s>>>(a);
            const hipError_t e2 = hipGetLastError();
            prof_end(s);
            return e2;
        }
    }
    return contract<T, R, 128, 128, 2>(id, a, s);
}

template <Role R>
hipError_t contract(int id, const GatedGemm &a, hipStream_t s) {
    return a.dtype == 1 ? contract<_Float16, R>(id, a, s) : contract<__bf16, R>(id, a, s);
}

}  // namespace

int64_t gated_splits(int64_t M, int64_t N, int64_t K, int64_t *steps) {
    // two tiles of 128 on every CU, none of fewer than eight steps
    const int64_t all = (K + BK - 1) / BK, t = tiles(M, N, 128, 128);
    int64_t most = 512 / t;
    if (most > all / 8) most = all / 8;
    if (most < 1) most = 1;
    *steps = (all + most - 1) / most;
    return (all + *steps - 1) / *steps;
}

hipError_t launch_gated_forward(const GatedGemm &a, hipStream_t s) { return contract<FORWARD>(K_GATED, a, s); }
hipError_t launch_gated_again(const GatedGemm &a, hipStream_t s) { return contract<AGAIN>(K_GATED_AGAIN, a, s); }
hipError_t launch_gated_dx(const GatedGemm &a, hipStream_t s) { return contract<DX>(K_GATED_DX, a, s); }
hipError_t launch_gated_dw(const GatedGemm &a, hipStream_t s) { return contract<DW>(K_GATED_DW, a, s); }

hipError_t launch_gated_gradients(const GatedGemm &a, hipStream_t s) {
    const int64_t lanes = a.ff / 8, threads = lanes < 256 ? (lanes + 63) / 64 * 64 : 256;
    const dim3 grid((unsigned)((lanes + threads - 1) / threads), (unsigned)(a.M < 16384 ? a.M : 16384)), block((unsigned)threads);
    prof_begin(K_GATED_GRADIENTS, s);
    if (a.dtype == 1)
        gated_gradients_kernel<_Float16><<<grid, block, 0, s>>>(a);
    else
        gated_gradients_kernel<__bf16><<<grid, block, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    prof_end(s);
    return e;
}

}  // namespace blr
