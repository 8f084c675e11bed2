// Low-rank adapters: launches of the contractions that the forward uses, and
// of the backward's where no gradient of an adapter is asked for.
#include "blr_adapters.h"

namespace blr {

namespace {

// Workgroups that keep the chip busy: a few per CU.
constexpr int64_t FILL = 1024;

template <typename TX, typename TW, int RT>
__global__ __launch_bounds__(256, RT <= 4 ? 2 : 1) void adapt_shrink_kernel(AdaptShrink a) {
    __shared__ __align__(16) char lds[ShrinkBlock<TX, TW, RT>::BYTES];
    ShrinkBlock<TX, TW, RT>::template run<false>(a, blockIdx.x, lds);
}

// Two workgroups to a CU. At ranks over 64 the adding form spills 100 bytes a
// lane for it in bf16, and is the faster for it all the same (8192 rows of 4096 ->
// 4096, rank 128, the whole call: 107 us against 130; f32, without a spill, 210
// against 243). f16 weights of such ranks, in two parts and two buffers, take
// 133 KB of LDS, which leaves room for one.
template <typename TX, int RT>
constexpr int expand_per_cu = __is_same(TX, _Float16) && RT > 4 ? 1 : 2;

template <typename TX, typename TW, int RT, bool ACC>
__global__ __launch_bounds__(256, (expand_per_cu<TX, RT>)) void adapt_expand_kernel(AdaptExpand a, int chunks) {
    __shared__ __align__(16) char lds[ExpandBlock<TX, TW, RT, ACC>::BYTES];
    ExpandBlock<TX, TW, RT, ACC>::run(a, chunks, blockIdx.x, lds);
}

template <typename TX, typename TW, int RT>
hipError_t shrink_t(const AdaptShrink &a, hipStream_t s) {
    const dim3 grid((unsigned)(a.splits * adapt_tiles(a.plan.M, a.plan.E, TM)));
    hipLaunchKernelGGL((adapt_shrink_kernel<TX, TW, RT>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

template <typename TX, typename TW, int RT>
hipError_t expand_t(const AdaptExpand &a, hipStream_t s) {
    const int64_t chunks = adapt_chunks(a.plan.M, a.plan.E, a.N);
    const dim3 grid((unsigned)(chunks * adapt_tiles(a.plan.M, a.plan.E, TM)));
    if (a.acc)
        hipLaunchKernelGGL((adapt_expand_kernel<TX, TW, RT, true>), grid, dim3(256), 0, s, a, (int)chunks);
    else
        hipLaunchKernelGGL((adapt_expand_kernel<TX, TW, RT, false>), grid, dim3(256), 0, s, a, (int)chunks);
    return hipGetLastError();
}

}  // namespace

int64_t adapt_tiles(int64_t M, int64_t E, int64_t tm) {
    const int64_t groups = E + 1 < M ? E + 1 : M;  // that have rows
    const int64_t tiles = M / tm + groups;
    return tiles < M ? tiles : M;
}

int adapt_splits(int64_t M, int64_t E, int64_t K) {
    const int64_t tiles = adapt_tiles(M, E, TM), units = K / 128;  // a split has a step for each wave in f32
    int64_t sp = (FILL / 2 + tiles - 1) / tiles;
    sp = sp > units ? units : sp;
    return (int)(sp > ADAPT_MAX_SPLITS ? ADAPT_MAX_SPLITS : sp);
}

int64_t adapt_chunks(int64_t M, int64_t E, int64_t N) {
    const int64_t tiles = adapt_tiles(M, E, TM), units = N / 128;
    int64_t chunks = (FILL + tiles - 1) / tiles;
    chunks = chunks > units ? units : chunks;
    return chunks > 8 ? chunks / 8 * 8 : chunks;  // a range of columns then stays on one XCD
}

// Enough ranges to fill the chip, but none so short that its partial (r floats
// a column, written and read again) costs much beside its rows. 8192 rows of
// rank 16 over 4096 + 4096 columns in eight adapters: both gradients' launches
// and the reduction take 133 us with 256 rows a range, 140 with 512, 169 with
// 1024. Up to 512 rows there is one range: a second did not pay for the
// reduction's launch in the one case measured, 300 f16 rows of rank 24 (6 us of
// 36). Neither limit was measured for f32 at ranks over 32, where a range's
// products take longest and a narrow layer leaves few workgroups.
int64_t adapt_range(int64_t M, int64_t d_in, int64_t d_out, int64_t r) {
    const int64_t cols = (d_in + 255) / 256 + (d_out + 255) / 256;
    int64_t range = M * cols / FILL;
    const int64_t least = M <= 512 ? M : 8 * r > 256 ? 8 * r : 256;
    range = range < least ? least : range;
    range = range < ADAPT_MAX_RANGE ? range : ADAPT_MAX_RANGE;
    range = range < M ? range : M;
    return (range + 63) / 64 * 64;
}

int64_t adapt_range_slots(int64_t M, int64_t E, int64_t range) {
    if (M <= range) return 0;
    const int64_t twice = 2 * M / range, all = M / range + E;
    return twice < all ? twice : all;
}

hipError_t launch_adapt_shrink(const AdaptShrink &a, int id, hipStream_t s) {
    prof_begin(id, s);
    hipError_t e = BLR_BY_TYPES(a, shrink_t, a, s);
    prof_end(s);
    return e;
}

hipError_t launch_adapt_expand(const AdaptExpand &a, int id, hipStream_t s) {
    prof_begin(id, s);
    hipError_t e = BLR_BY_TYPES(a, expand_t, a, s);
    prof_end(s);
    return e;
}

}  // namespace blr
