// Norms before and after a block for gfx950, and rows kept in 8 bits.
//
//   forward   v = (norm_f ? f rstd_f : f) w_after   out = skip x + scale phi(z) v   n = out rstd w
//             (without f: out is x), rstd = 1 / sqrt(mean(row^2) + eps)
//   backward  dO = dout + J(w dn; out, rstd)        dx = skip dO
//             p = scale phi(z) dO                   df = norm_f ? J(w_after p; f, rstd_f) : w_after p
//             dw = sum dn out rstd                  dw_after = sum p (norm_f ? f rstd_f : f)
//             dz = scale phi'(z) v dO, summed over the rows that share z
//             with J(v; x, r) = r (v - x^ mean(v x^)), x^ = x r
//
// Both are passes over rows, bound by HBM. A workgroup takes a row whole, each
// thread 8 C of its columns, in registers from the load to the last store, so
// that every array crosses memory once. Sums over a row are f32: along a wave
// by lane moves, over the row's waves through LDS, in a fixed order. The forward
// of 8192 x 4096, f32 stream and f, a gate a row, bf16 n takes 110 us (18 bytes a
// value, 5.5 TB/s); a 2 GiB copy runs at 5.0.
#include <cfloat>

#include "blr_internal.h"
#include "blr_keep8.h"
#include "blr_math.h"

namespace blr {

namespace {

constexpr int MAX_WAVES = 16;
constexpr int TEAMS = 4;  // rows of a workgroup where one wave holds a row

// lane's value plus the one that a lane move of the row of 16 brings
template <int CTRL>
__device__ __forceinline__ float plus_dpp(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// The sum over a wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
    v = plus_dpp<0xB1>(v);   // lane ^ 1
    v = plus_dpp<0x4E>(v);   // lane ^ 2
    v = plus_dpp<0x141>(v);  // mirrored within 8
    v = plus_dpp<0x140>(v);  // mirrored within 16
    const int i = __builtin_bit_cast(int, v);
    auto lane = [i](int l) { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(i, l)); };
    return (lane(0) + lane(16)) + (lane(32) + lane(48));
}

// phi(z) and its slope. With e = exp(-|z|), 1 / (1 + e) and e / (1 + e) are
// sigmoid(|z|) and sigmoid(-|z|), so that s (1 - s) loses nothing far out (it is
// zero where e is), and nothing overflows.
__device__ __forceinline__ float phi(int kind, float z, float *slope) {
    if (kind == 0) {
        *slope = 1.0f;
        return z;
    }
    // past 200 the exponential is zero, and z may be infinite; a NaN stays one
    const float e = exp_of(fabsf(z) > 200.0f ? -200.0f : -fabsf(z)), big = inverse(1.0f + e), small = e * big;
    const float s = z >= 0.0f ? big : small, r = big * small;
    *slope = kind == 1 ? r : r == 0.0f ? s : s + z * r;  // z may be infinite where r is zero
    return kind == 1 ? s : fmaxf(z, -FLT_MAX) * s;  // and s zero where z is minus infinity
}

// phi of eight values, and their slopes where asked for, both times scale; the
// kind is looked at once.
template <bool SLOPE>
__device__ __forceinline__ void phi8(int kind, float scale, float *z, float *slope) {
    auto all = [&](int kind) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float s;
            z[i] = scale * phi(kind, z[i], &s);
            if constexpr (SLOPE) slope[i] = scale * s;
        }
    };
    if (kind == 0)
        all(0);
    else if (kind == 1)
        all(1);
    else
        all(2);
}

struct Team {
    int tid, waves, team;
    __device__ Team() : tid(threadIdx.x), waves(blockDim.x >> 6), team(__builtin_amdgcn_readfirstlane(threadIdx.y)) {}
    // Sums of N values over the threads of a row; `slot` alternates between
    // calls, so that one barrier a call is enough.
    template <int N>
    __device__ void sum(float *v, float *lds, int slot) const {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
        if (waves == 1) return;
        float *at = lds + slot * N * MAX_WAVES;
        if ((tid & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) at[i * MAX_WAVES + (tid >> 6)] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.0f;
            for (int w = 0; w < waves; ++w) v[i] += at[i * MAX_WAVES + w];
        }
    }
};

template <typename XT, typename FT, typename NT, int C>
__global__ __launch_bounds__(64 * MAX_WAVES) void norm_forward_kernel(NormForward a) {
    __shared__ float red[2 * MAX_WAVES];
    const Team t;
    const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.y + t.team;
    if (row >= a.M) return;  // whole waves: a workgroup of several rows has one wave for each
    const int d = (int)a.d, chunks = d / 8, step = 64 * t.waves;
    const float inv_d = 1.0f / (float)d;
    const XT *x = (const XT *)a.x + row * d;
    float v[C][8];
    if (a.f) {
        const FT *f = (const FT *)a.f + row * d;
        const FT *z = (const FT *)a.gate + (a.gate ? (int64_t)((uint32_t)row / a.span) * d : 0);
        Raw8<XT> xr[C];
        Raw8<FT> fr[C], zr[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = t.tid + c * step;
            if (k < chunks) {
                fr[c] = raw8(f + 8 * k);
                xr[c] = raw8(x + 8 * k);
                if (a.gate) zr[c] = raw8(z + 8 * k);
            }
        }
        float rf = 1.0f;
        if (a.norm_f) {
            float s = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (t.tid + c * step < chunks) {
                    float e[8];
                    widen8(fr[c], e);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s += e[i] * e[i];
                }
            t.sum<1>(&s, red, 0);
            rf = 1.0f / sqrtf(s * inv_d + a.eps);
        }
        if (t.tid == 0 && a.stats) a.stats[a.M + row] = a.norm_f ? rf : 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = t.tid + c * step;
            if (k >= chunks) continue;
            float e[8], w[8], g[8];
            widen8(fr[c], e);
            if (a.w_after) {
                widen8(raw8(a.w_after + 8 * k), w);
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] = e[i] * rf * w[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] = e[i] * rf;
            }
            if (a.gate) {
                widen8(zr[c], g);
                float unused;
#pragma unroll
                for (int i = 0; i < 8; ++i) e[i] *= phi(a.gate_kind, g[i], &unused);
            }
            widen8(xr[c], v[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] = a.skip * v[c][i] + a.scale * e[i];
            const Raw8<XT> o = narrow8<XT>(v[c]);
            put8((XT *)a.out + row * d + 8 * k, o);
            widen8(o, v[c]);  // the norm, like the checkpoint, is of the rows as they are stored
        }
    } else {
        if (t.tid == 0 && a.stats) a.stats[a.M + row] = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (t.tid + c * step < chunks) widen8(raw8(x + 8 * (t.tid + c * step)), v[c]);
    }
    if (a.q)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = t.tid + c * step;
            if (k >= chunks) continue;  // four lanes together: d is a multiple of 32 here
            const int b = keep_exponent(top_of_quad(top8(v[c])), KEEP_MAX<XT>);
            *reinterpret_cast<uint2 *>(a.q + row * d + 8 * k) = keep8(v[c], b);
            if ((t.tid & 3) == 0) a.b[row * (d / 32) + k / 4] = (uint8_t)b;
        }
    if (!a.n && !a.stats) return;
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (t.tid + c * step < chunks)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[c][i] * v[c][i];
    t.sum<1>(&s, red, 1);
    const float r = 1.0f / sqrtf(s * inv_d + a.eps);
    if (t.tid == 0 && a.stats) a.stats[row] = r;
    if (!a.n) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int k = t.tid + c * step;
        if (k >= chunks) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= r;
        if (a.w) {
            float w[8];
            widen8(raw8(a.w + 8 * k), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] *= w[i];
        }
        put8((NT *)a.n + row * d + 8 * k, narrow8<NT>(v[c]));
    }
}

// What a row of the backward reads, in one chunk of 8 columns, and the values
// that its sums are of:
//   xh = out r   fh = f rf   o = dout + r w dn   z
template <typename XT, typename FT, typename NT, bool GATE>
struct NormRow {
    Raw8<XT> dout, out;
    Raw8<FT> f, z;
    Raw8<NT> dn;
    int out_b, f_b;

    __device__ __forceinline__ void load(const NormBackward &a, int64_t row, int64_t gate_row, int k) {
        const int64_t at = row * a.d + 8 * k;
        if (a.dout) dout = raw8((const XT *)a.dout + at);
        if (a.dn) {
            dn = raw8((const NT *)a.dn + at);
            if (a.out_q) {
                const uint2 q = *reinterpret_cast<const uint2 *>(a.out_q + at);
                __builtin_memcpy(&out, &q, 8);
                out_b = a.out_b[row * (a.d / 32) + k / 4];
            } else {
                out = raw8((const XT *)a.out + at);
            }
        }
        if (a.need_f) {
            if (a.f_q) {
                const uint2 q = *reinterpret_cast<const uint2 *>(a.f_q + at);
                __builtin_memcpy(&f, &q, 8);
                f_b = a.f_b[row * (a.d / 32) + k / 4];
            } else {
                f = raw8((const FT *)a.f + at);
            }
        }
        if constexpr (GATE) z = raw8((const FT *)a.gate + gate_row * a.d + 8 * k);
    }
    template <typename T>
    __device__ __forceinline__ static void rows(const Raw8<T> &r, bool kept, int b, float *o) {
        if (kept) {
            uint2 q;
            __builtin_memcpy(&q, &r, 8);
            kept8(q, b, o);
        } else {
            widen8(r, o);
        }
    }
    // g: dn
    __device__ __forceinline__ void values(const NormBackward &a, float r, float rf, const float *w, float *xh, float *fh,
                                           float *o, float *g) const {
        if (a.dn) {
            rows(out, a.out_q != nullptr, out_b, xh);
            widen8(dn, g);
        }
        if (a.dout) widen8(dout, o);
        if (a.need_f) rows(f, a.f_q != nullptr, f_b, fh);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (!a.dn) xh[i] = g[i] = 0.0f;
            if (!a.dout) o[i] = 0.0f;
            if (!a.need_f) fh[i] = 0.0f;
            xh[i] *= r;
            fh[i] *= rf;
            o[i] += r * (g[i] * w[i]);
        }
    }
    // scale phi(z) and scale phi'(z)
    template <bool SLOPE>
    __device__ __forceinline__ void gate(const NormBackward &a, float *ph, float *slope) const {
        if constexpr (GATE) {
            widen8(z, ph);
            phi8<SLOPE>(a.gate_kind, a.scale, ph, slope);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) ph[i] = a.scale;
        }
    }
};

__device__ __forceinline__ void put_sums(float *p, const float *v, bool add) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        vf4 *at = reinterpret_cast<vf4 *>(p) + h;
        vf4 s = {v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
        if (add) s += *at;
        *at = s;
    }
}

// A team (a workgroup, or one of its waves for short rows) takes a range of
// consecutive rows and keeps the sums over them in registers; a workgroup's go
// to the workspace, and the next launch adds those in order.
// m1 = mean(w dn x^) and the mean that df needs come out of one exchange:
// with k = scale w_after phi f^, sum(k dO) = sum(k (dout + r w dn)) - r m1 sum(k x^).
// HOLD: a row stays in registers from its sums to its results; with 16 columns a
// thread that is more than the 128 registers of 16 waves on a CU, and the row is
// read a second time, out of the caches. AHEAD: the next row is loaded
// meanwhile, which leaves no room for a gate.
// 8192 x 4096, f32 stream and f, bf16 n, the bytes of its rows: 117 us from
// checkpoints (16.06 bytes a value, 4.6 TB/s), 152 from rows (22, 4.8), 225 with a
// gate a row (30, 4.5); the finish takes 7 to 9 more. Wider rows are slower: 5120 bf16
// columns, ten of a CU's sixteen waves, 3.8 TB/s; 8192 f32 with a gate, 36 registers
// in memory, 640 us (3.1); 2048 x 16384 f32 with a gate, 168 of them, 680 us (1.5).
template <typename XT, typename FT, typename NT, int C, bool GATE, int WAVES = MAX_WAVES>
__global__ __launch_bounds__(64 * WAVES) void norm_backward_kernel(NormBackward a) {
    constexpr bool HOLD = C == 1, AHEAD = HOLD && !GATE;
    __shared__ float red[2 * 3 * MAX_WAVES];
    __shared__ vf4 fold[C == 1 ? TEAMS * 64 * 2 : 1];
    const Team t;
    const int64_t range = (int64_t)blockIdx.x * blockDim.y + t.team;
    const int64_t lo = range * a.per, hi = lo + a.per < a.M ? lo + a.per : a.M;  // past the last range lo >= hi
    const int d = (int)a.d, chunks = d / 8, step = 64 * t.waves;
    const float inv_d = 1.0f / (float)d;
    using Row = NormRow<XT, FT, NT, GATE>;
    float w[C][8], wa[C][8], sw[C][8], sa[C][8], sz[C][8];
    Row in[C];
    auto weights = [&](int c) {
        const int k = t.tid + c * step;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[c][i] = wa[c][i] = 1.0f;
        if (a.w) widen8(raw8(a.w + 8 * k), w[c]);
        if (a.w_after) widen8(raw8(a.w_after + 8 * k), wa[c]);
    };
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sw[c][i] = sa[c][i] = sz[c][i] = 0.0f;
        if (t.tid + c * step >= chunks || lo >= hi) continue;
        if (AHEAD) weights(c);
        if (AHEAD) in[c].load(a, lo, 0, t.tid + c * step);
    }
    const bool shared = GATE && a.dgate && a.summed;
    for (int64_t row = lo; row < hi; ++row) {
        const float r = a.dn ? a.stats[row] : 0.0f, rf = a.norm_f ? a.stats[a.M + row] : 1.0f;
        const int64_t group = GATE ? (uint32_t)row / a.span : 0;
        float xh[C][8], fh[C][8], o[C][8];
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = t.tid + c * step;
            if (k >= chunks) continue;
            float g[8], ph[8];
            if (!AHEAD) {
                weights(c);
                in[c].load(a, row, group, k);
            }
            in[c].values(a, r, rf, w[c], xh[c], fh[c], o[c], g);
            in[c].template gate<false>(a, ph, nullptr);
            if (AHEAD && row + 1 < hi) in[c].load(a, row + 1, 0, k);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sw[c][i] += g[i] * xh[c][i];
                s[0] += g[i] * w[c][i] * xh[c][i];
                const float q = wa[c][i] * ph[i] * fh[c][i];
                s[1] += q * o[c][i];
                s[2] += q * xh[c][i];
            }
            if (!HOLD) __builtin_amdgcn_sched_barrier(0);  // a chunk at a time
        }
        t.sum<3>(s, red, (int)(row & 1));
        const float m1 = r * s[0] * inv_d;
        const float m2 = (s[1] - m1 * s[2]) * inv_d;
        const bool last = shared && ((uint32_t)(row + 1) % a.span == 0 || row + 1 == hi);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int k = t.tid + c * step;
            if (k >= chunks) continue;
            float ph[8], slope[8];
            if (!HOLD) {
                // not to be taken for the loads above, whose results would be held
                asm volatile("" ::: "memory");
                weights(c);
                in[c].load(a, row, group, k);
                float g[8];
                in[c].values(a, r, rf, w[c], xh[c], fh[c], o[c], g);
            }
            in[c].template gate<true>(a, ph, slope);
            const int64_t at = row * d + 8 * k;
            float dx[8], df[8], dz[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float dO = o[c][i] - m1 * xh[c][i];
                const float p = ph[i] * dO;
                dx[i] = a.skip * dO;
                df[i] = wa[c][i] * p;
                if (a.norm_f) df[i] = rf * (df[i] - fh[c][i] * m2);
                sa[c][i] += p * fh[c][i];
                if constexpr (GATE) {
                    dz[i] = slope[i] * wa[c][i] * fh[c][i] * dO;
                    sz[c][i] += dz[i];
                }
            }
            if (a.dx) put8((XT *)a.dx + at, narrow8<XT>(dx));
            if (a.df) put8((FT *)a.df + at, narrow8<FT>(df));
            if (GATE && a.dgate && !shared) put8((FT *)a.dgate + at, narrow8<FT>(dz));
            if (last) {
                // the rows of this gate end here, or the range does: whole
                // gates go to their place, parts of one to the workspace,
                // slot 0 where it began before the range, 1 where it goes on
                const int64_t first = group * a.span, end = first + a.span < a.M ? first + a.span : a.M;
                if (first >= lo && end <= hi)
                    put_sums((float *)a.dgate + group * d + 8 * k, sz[c], a.acc);
                else
                    put_sums(a.part_z + (2 * range + (first >= lo ? 1 : 0)) * d + 8 * k, sz[c], false);
#pragma unroll
                for (int i = 0; i < 8; ++i) sz[c][i] = 0.0f;
            }
        }
    }
    // the workgroup's sums: its teams' in order, where it has several (one chunk
    // a thread then)
    if (C == 1 && blockDim.y > 1) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            float *mine = v ? sa[0] : sw[0];
            __syncthreads();
            put_sums((float *)(fold + (t.team * 64 + t.tid) * 2), mine, false);
            __syncthreads();
            if (t.team == 0)
                for (int q = 1; q < (int)blockDim.y; ++q)
#pragma unroll
                    for (int i = 0; i < 8; ++i) mine[i] += ((const float *)(fold + (q * 64 + t.tid) * 2))[i];
        }
        if (t.team) return;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int k = t.tid + c * step;
        if (k >= chunks) continue;
        const bool one = gridDim.x == 1;
        if (a.dw) put_sums((one ? a.dw : a.part_w + (int64_t)blockIdx.x * d) + 8 * k, sw[c], one && a.acc);
        if (a.dw_after) put_sums((one ? a.dw_after : a.part_a + (int64_t)blockIdx.x * d) + 8 * k, sa[c], one && a.acc);
    }
}

// The sums in order: 32 columns to a workgroup, 32 lines of its threads down
// the partial sums, then the lines. blockIdx.y: dw, dw_after, and from 2 on the
// gates whose rows lie in several ranges (by gate, or, if there are fewer
// ranges, by the range in which such a gate begins).
__global__ __launch_bounds__(256) void norm_finish_kernel(NormBackward a) {
    __shared__ vf4 line[32][8];
    const int d = (int)a.d, col = blockIdx.x * 32 + 4 * (threadIdx.x & 7), l = threadIdx.x >> 3;
    const bool in = col < d;
    const float *part;
    float *out;
    int64_t first, count, stride = d;
    if (blockIdx.y < 2) {
        part = blockIdx.y == 0 ? a.part_w : a.part_a;
        out = blockIdx.y == 0 ? a.dw : a.dw_after;
        if (!out || a.blocks == 1) return;
        first = 0;
        count = a.blocks;
    } else {
        int64_t group = blockIdx.y - 2;
        if (!a.by_gate) {
            const int64_t hi = (group + 1) * a.per < a.M ? (group + 1) * a.per : a.M;
            const int64_t lo = group * a.per;
            group = (hi - 1) / a.span;
            if (group * a.span < lo) return;
        }
        const int64_t begin = group * a.span, end = begin + a.span < a.M ? begin + a.span : a.M;
        first = begin / a.per;
        count = (end + a.per - 1) / a.per - first;
        if (count == 1) return;
        part = a.part_z;
        out = (float *)a.dgate + group * d;
        stride = 2 * d;
    }
    vf4 s = {};
    if (in)
#pragma unroll 8
        for (int64_t i = l; i < count; i += 32) {
            const float *p = part + (first + i) * stride + col;
            if (stride != d && i == 0) p += d;  // where the gate begins its sum lies in slot 1
            s += *reinterpret_cast<const vf4 *>(p);
        }
    line[l][threadIdx.x & 7] = s;
    __syncthreads();
    if (l || !in) return;
    s = a.acc ? *reinterpret_cast<vf4 *>(out + col) : vf4{};
    vf4 sum = {};
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += line[i][threadIdx.x & 7];
    *reinterpret_cast<vf4 *>(out + col) = s + sum;
}

template <typename T>
__global__ __launch_bounds__(256) void checkpoint_save_kernel(Checkpoint a) {
    const int64_t n = a.n / 8, grid = (int64_t)gridDim.x * 256;
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += grid) {  // n is a multiple of 4
        float v[8];
        widen8(raw8((const T *)a.x + 8 * k), v);
        const int b = keep_exponent(top_of_quad(top8(v)), KEEP_MAX<T>);
        *reinterpret_cast<uint2 *>(a.q + 8 * k) = keep8(v, b);
        if ((threadIdx.x & 3) == 0) a.b[k / 4] = (uint8_t)b;
    }
}

template <typename T>
__global__ __launch_bounds__(256) void checkpoint_load_kernel(Checkpoint a) {
    const int64_t n = a.n / 8, grid = (int64_t)gridDim.x * 256;
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += grid) {
        float v[8];
        kept8(*reinterpret_cast<const uint2 *>(a.q + 8 * k), a.b[k / 4], v);
        put8((T *)a.x + 8 * k, narrow8<T>(v));
    }
}

struct Shape {
    int c, waves, teams;
};
// Rows up to 512 C columns are one wave's, four rows to a workgroup; longer
// ones a workgroup's, with as few waves as hold them.
Shape shape_of(int64_t d, int c) {
    const int waves = (int)((d + 512 * c - 1) / (512 * c));
    return {c, waves, waves == 1 ? TEAMS : 1};
}
// Chunks of 8 columns per thread: one while 16 waves hold the row.
int chunks_of(int64_t d) { return d <= 512 * MAX_WAVES ? 1 : 2; }

template <typename F>
hipError_t with_types(int xt, int ft, int nt, F f) {
    if (xt == 1) return f(_Float16(), _Float16(), _Float16());
    if (xt == 2) return f(__bf16(), __bf16(), __bf16());
    auto third = [&](auto ftag) {
        return nt == 0 ? f(float(), ftag, float()) : nt == 1 ? f(float(), ftag, _Float16()) : f(float(), ftag, __bf16());
    };
    return ft == 0 ? third(float()) : ft == 1 ? third(_Float16()) : third(__bf16());
}

template <typename K, typename A>
hipError_t launch(int id, K kernel, dim3 grid, dim3 block, const A &a, hipStream_t s) {
    prof_begin(id, s);
    kernel<<<grid, block, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    prof_end(s);
    return e;
}

}  // namespace

hipError_t launch_norm_forward(const NormForward &a, hipStream_t s) {
    const Shape sh = shape_of(a.d, chunks_of(a.d));
    // a row (or four) to a workgroup; a grid has room for 2^32 threads along x
    const int64_t groups = (a.M + sh.teams - 1) / sh.teams, most = 1 << 20;
    const dim3 block(64 * sh.waves, sh.teams);
    const dim3 grid((unsigned)(groups < most ? groups : most), (unsigned)((groups + most - 1) / most));
    return with_types(a.xt, a.ft, a.nt, [&](auto x, auto f, auto n) {
        using X = decltype(x);
        using F = decltype(f);
        using N = decltype(n);
        return launch(K_NORM, sh.c == 1 ? norm_forward_kernel<X, F, N, 1> : norm_forward_kernel<X, F, N, 2>, grid, block,
                      a, s);
    });
}

NormSplit norm_split(int64_t M, int64_t d) {
    // as many as are on the chip at once, 16 waves on a CU: each takes its rows
    // in one go, and more partial sums cost more than they bring
    const Shape sh = shape_of(d, chunks_of(d));
    const int64_t most = 256 * (MAX_WAVES / sh.waves);
    NormSplit n;
    n.per = (M + most - 1) / most;
    n.ranges = (M + n.per - 1) / n.per;
    n.blocks = (n.ranges + sh.teams - 1) / sh.teams;
    return n;
}

hipError_t launch_norm_backward(NormBackward a, hipStream_t s) {
    const Shape sh = shape_of(a.d, chunks_of(a.d));
    const dim3 block(64 * sh.waves, sh.teams), grid((unsigned)a.blocks);
    const hipError_t e = with_types(a.xt, a.ft, a.nt, [&](auto x, auto f, auto n) {
        using X = decltype(x);
        using F = decltype(f);
        using N = decltype(n);
        if (a.gate)
            return launch(K_NORM_BWD,
                          // 12 waves, up to 6144 columns, leave it 168 registers: 227 us
                          // for 8192 x 4096 f32 against 308 with 128, some of them in memory
                          sh.c == 1 && sh.waves <= 12 ? norm_backward_kernel<X, F, N, 1, true, 12>
                          : sh.c == 1    ? norm_backward_kernel<X, F, N, 1, true>
                                         : norm_backward_kernel<X, F, N, 2, true>,
                          grid, block, a, s);
        return launch(K_NORM_BWD,
                      sh.c == 1 ? norm_backward_kernel<X, F, N, 1, false> : norm_backward_kernel<X, F, N, 2, false>,
                      grid, block, a, s);
    });
    const int64_t gates = a.dgate && a.summed ? (a.M + a.span - 1) / a.span : 0;
    if (e != hipSuccess || ((a.blocks == 1 || !(a.dw || a.dw_after)) && (!gates || a.ranges == 1))) return e;
    a.by_gate = gates <= a.ranges;
    return launch(K_NORM_FINISH, norm_finish_kernel,
                  dim3((unsigned)((a.d + 31) / 32), 2 + (unsigned)(a.by_gate ? gates : a.ranges)), dim3(256), a, s);
}

hipError_t launch_checkpoint(const Checkpoint &a, bool save, hipStream_t s) {
    const int64_t n = (a.n / 8 + 255) / 256, most = 256 * 32;
    const dim3 grid((unsigned)(n < most ? n : most)), block(256);
    auto run = [&](auto t) {
        using T = decltype(t);
        return save ? launch(K_CHECKPOINT_SAVE, checkpoint_save_kernel<T>, grid, block, a, s)
                    : launch(K_CHECKPOINT_LOAD, checkpoint_load_kernel<T>, grid, block, a, s);
    };
    return a.dtype == 0 ? run(float()) : a.dtype == 1 ? run(_Float16()) : run(__bf16());
}

}  // namespace blr
