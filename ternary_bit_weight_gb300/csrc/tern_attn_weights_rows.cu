// Attention weight that cached tokens receive from many query rows: the form of
// tern_attn_weights for windows of a prompt and whole prompts.
//
// Mathematics: as in tern_attn_weights.cu.  A key is a row of the product S = K Q^T
// and a query row and head a column, so a thread that has a key adds up what it
// receives without asking another.
//
// What bounds it: the tensor cores and beside them the warps that take a score out of
// tensor memory, its exponential and its sum; for windows of few rows what an item
// costs besides.  Measured, 40 / 8 heads of 128, bf16: a prompt of 4096 tokens 89 us (960
// TFLOP/s of the pairs that see one another; over codes the same), of 8192 305 us (1125),
// windows of 32 rows over 4 x 8191 tokens 35.3 us.  A tile of 192 columns costs the summing warps some 900
// cycles of exponentials and 500 of waits, accumulations and arrivals, so tiles are as
// wide as tensor memory allows.  Tried and slower, against 94 us for the prompt at the
// time: tiles of 128 columns in three buffers (115), twelve or sixteen summing warps
// instead of eight, in one team (95) or two (112), 256 keys to an item with clusters that
// share its columns (99), keys by way of shared memory (95; windows the same), a third of
// the exponentials by a polynomial (111: the unit for them is not what is busy).
//
// Work.  An item is 128 keys of one (sequence, key/value head), against the columns
// of all rows that see them, 192 or fewer at a time.  Items are dealt to one CTA per
// SM, there and back, a sequence's first keys, which most rows see, first.  The keys
// lie in tensor memory (codes exactly as 16-bit values, their factor being the
// thread's), which leaves shared memory to the queries alone.
//
// Roles, each a loop over the CTA's items:
//   warp 0       queries of a column tile by TMA, one box of heads x rows
//   warp 1       tcgen05.mma, scores into one of two buffers of tensor memory
//   warp 2       the columns' logarithms
//   warps 4-7    keys, one per thread, into one of two buffers of tensor memory,
//                an item ahead
//   warps 8-15   exponentials and sums: a thread has a key and half of the columns
// Every wait is bounded; after a timeout the weights not yet written become NaN.
//
// Sums with care.  A column tile with a logarithm far from zero or of a row that saw nothing,
// and every tile of an item with a key whose factor is out of the ordinary, go through a
// slower form of the sums, right for any size of values (see kFarLse, kFarScale).  Of codes
// it forms a score anew where their product with the query is beyond fp32: 0.3 ms a tile if
// all of them are, so that past 200000 rows of such values the waits would run out.

#include <float.h>
#include <math_constants.h>
#include <string.h>

#include "tern_attn_weights.cuh"

namespace tern {
namespace weights {
namespace {

constexpr int kKeys = 128;               // of an item
constexpr int kColumns = 192;            // of a column tile, at most
constexpr int kThreads = 512;
constexpr int kOffStages = 4;
// Column tiles in shared memory; so many that one CTA fills an SM.
template <int DP>
constexpr int kQStagesOf = DP == 64 ? 6 : 3;
constexpr int kHalfBytes = kColumns * 128;   // 64 dimensions of a column tile
constexpr int kSCol = 128;               // tensor memory: two key buffers of 64 columns, two of scores
constexpr int kTmemCols = 512;
// Scores are taken to base 2 by their scale, and the logarithms with them, each rounded at its
// own size, which moves a weight by 2^-23 |lse| of itself, as the roundings of the product's sum
// may.  A column tile that has a logarithm past this is summed with care: the difference alone is
// taken to base 2 (a prompt of 4096 tokens 142 us, over int8 codes 190; 89 without).
constexpr float kFarLse = 128.0f;
// So are the tiles of an item with a key whose factor times the scale is not within 2^-90 and 2^90.
constexpr float kFarScale = 0x1p90f;
static_assert(kSCol + 2 * kColumns <= kTmemCols, "tensor-memory budget");

// control block
constexpr int kMostQStages = 6;
constexpr int kBarQFull = 0, kBarQEmpty = kBarQFull + 8 * kMostQStages;
constexpr int kBarOffFull = kBarQEmpty + 8 * kMostQStages, kBarOffEmpty = kBarOffFull + 8 * kOffStages;
constexpr int kBarSFull = kBarOffEmpty + 8 * kOffStages, kBarSEmpty = kBarSFull + 16;
constexpr int kBarKFull = kBarSEmpty + 16, kBarKEmpty = kBarKFull + 16;
constexpr int kBarDrain = kBarKEmpty + 16;
constexpr int kTmemPtr = kBarDrain + 8, kAbort = kTmemPtr + 4;
constexpr int kPartial = 256;                          // [2][128] sums of the second halves
constexpr int kOff = kPartial + 2 * kKeys * 4;         // [stages][columns]
constexpr int kFar = kOff + kOffStages * kColumns * 4; // [stages] whether a tile is summed with care
constexpr int kCtrlBytes = kFar + kOffStages * 4;
static_assert(kAbort + 4 <= kPartial, "control block");

template <int DP>
constexpr int smem_bytes() {
    return 1024 + kQStagesOf<DP> * (DP / 64) * kHalfBytes + kCtrlBytes;
}
static_assert(smem_bytes<128>() <= 232448, "shared-memory budget");

struct Maps {
    CUtensorMap q;
};

// 128 keys of a sequence from j0, and the rows from i0 on that see some of them.
struct Item {
    int b, hk, j0, i0;
    int q0, nq, len;
};

// The CTA's items in turn; one warp.  Items that follow one another are mostly of one
// sequence, whose place is kept: every role takes this step for every item, and the
// search for the sequence alone made it 800 cycles.
struct Walker {
    Sequence mine = {0, 0, 0};      // of the 32 sequences from b0, one per lane
    int64_t incl = 0, base = 0;     // their items up to the lane's end, and those before
    int b0 = 0;
    int64_t index, step[2];         // there and back
    int64_t first = 0, each = 0;    // items before the sequence at hand, and its own
    int b = 0;
    Sequence s = {0, 0, 0};
    float inverse;                  // 1 / Hkv

    __device__ __forceinline__ void load(const Args& a, int lane) {
        mine = {0, 0, 0};
        if (b0 + lane < a.B) mine = sequence_at(a, b0 + lane);
        incl = tiles_of(a, mine, kKeys);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += up;
        }
    }
    __device__ __forceinline__ Walker(const Args& a, int lane) {
        load(a, lane);
        step[0] = 2 * static_cast<int64_t>(gridDim.x - 1 - blockIdx.x) + 1;
        step[1] = 2 * static_cast<int64_t>(blockIdx.x) + 1;
        index = static_cast<int64_t>(blockIdx.x) - step[1];
        inverse = 1.0f / static_cast<float>(a.Hkv);
    }
    __device__ __forceinline__ bool next(const Args& a, int lane, Item& o) {
        index += step[1];
        const int64_t t = step[0];
        step[0] = step[1];
        step[1] = t;
        if (index - first >= each) {   // (never below: indices grow)
            for (;;) {
                const uint32_t past = __ballot_sync(0xffffffffu, base + incl > index);
                if (past != 0) {
                    const int src = __ffs(past) - 1;
                    b = b0 + src;
                    s.q0 = __shfl_sync(0xffffffffu, mine.q0, src);
                    s.nq = __shfl_sync(0xffffffffu, mine.nq, src);
                    s.len = __shfl_sync(0xffffffffu, mine.len, src);
                    each = tiles_of(a, s, kKeys);
                    first = base + __shfl_sync(0xffffffffu, incl, src) - each;
                    break;
                }
                base += __shfl_sync(0xffffffffu, incl, 31);
                b0 += 32;
                if (b0 >= a.B) return false;
                load(a, lane);
            }
        }
        const int64_t in = index - first;
        int block, hk;
        if (in < (1 << 22)) {
            // (a quotient below 2^22 by fp32 is off by one at most)
            const int n = static_cast<int>(in);
            block = static_cast<int>(static_cast<float>(n) * inverse);
            hk = n - block * a.Hkv;
            if (hk < 0) {
                --block;
                hk += a.Hkv;
            } else if (hk >= a.Hkv) {
                ++block;
                hk -= a.Hkv;
            }
        } else {
            block = static_cast<int>(in / a.Hkv);
            hk = static_cast<int>(in - static_cast<int64_t>(block) * a.Hkv);
        }
        o.b = b;
        o.q0 = s.q0;
        o.nq = s.nq;
        o.len = s.len;
        o.hk = hk;
        o.j0 = block * kKeys;
        o.i0 = max(0, o.j0 - (o.len - o.nq));
        return true;
    }
};

// Four codes as two pairs of 16-bit values, exactly.
template <int KV, bool F16>
__device__ __forceinline__ void decode4_as(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (F16) {
        decode4<KV>(w, lo, hi);
    } else if constexpr (KV == kKvE4m3) {
        decode4<KV>(w, lo, hi);
        const float2 x = unpack_x2<true>(lo), y = unpack_x2<true>(hi);
        lo = pack_x2<false>(x.x, x.y);
        hi = pack_x2<false>(y.x, y.y);
    } else {
        // (128 + low 7 bits) - (128, or 256 where the code is negative)
        const uint32_t u = w & 0x7F7F7F7Fu, n = w & 0x80808080u;
        const uint32_t x = __byte_perm(u, 0x43434343u, 0x4140), y = __byte_perm(u, 0x43434343u, 0x4342);
        const uint32_t bx = __byte_perm(n, 0x43434343u, 0x4140), by = __byte_perm(n, 0x43434343u, 0x4342);
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(x), "r"(bx));
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(y), "r"(by));
    }
}

// The exponentials of 32 columns' scores, to `part` (pairs of sums).  MASKED: of columns from
// lo to hi only.
template <bool MASKED>
__device__ __forceinline__ void add_scores(const uint32_t (&v)[32], uint64_t ff, const ulonglong2* off, int lo, int hi, uint64_t (&part)[2]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const ulonglong2 o = off[j / 2];
        float x0, x1;
        unpair(fma_x2(pair(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), ff, j & 1 ? o.y : o.x), x0, x1);
        if (MASKED) {
            x0 = 2 * j >= lo && 2 * j < hi ? exp2_approx(x0) : 0.0f;
            x1 = 2 * j + 1 >= lo && 2 * j + 1 < hi ? exp2_approx(x1) : 0.0f;
        } else {
            x0 = exp2_approx(x0);
            x1 = exp2_approx(x1);
        }
        part[j & 1] = add_x2(part[j & 1], pair(x0, x1));
    }
}

// Whether a scale times a key's factor is too large or small for the usual sums.
__device__ __forceinline__ bool out_of_range(float scale, float factor) {
    const float size = fabsf(scale);
    return factor != 0.0f && (size < 1.0f / kFarScale || size > kFarScale);
}

// scale * q.k of a query and a coded key, whatever their sizes: the query times a power of two,
// so that its largest value lies in [1, 2).
template <int KV, bool F16>
__device__ __noinline__ double score_of_codes(const Args& a, const uint16_t* q, const uint8_t* codes, float factor) {
    float top = 0.0f;
    for (int d = 0; d < a.D; d += 16) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 u = *reinterpret_cast<const uint4*>(q + d + 8 * h);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = unpack_x2<F16>(w[i]);
                top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
            }
        }
    }
    const int e = top > 0.0f && top <= FLT_MAX ? -ilogbf(top) : 0;
    // in two steps: 2^e may pass fp32's range
    const float up0 = exp2f(static_cast<float>(e / 2)), up1 = exp2f(static_cast<float>(e - e / 2));
    float sum = 0.0f;
    for (int d = 0; d < a.D; d += 16) {
        const uint4 u = *reinterpret_cast<const uint4*>(codes + d);
        const uint32_t k[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint2 w = *reinterpret_cast<const uint2*>(q + d + 4 * i);
            uint32_t lo, hi;
            decode4<KV>(k[i], lo, hi);
            const float2 x = unpack_x2<F16>(w.x), y = unpack_x2<F16>(w.y), c = unpack_x2<true>(lo), f = unpack_x2<true>(hi);
            sum = fmaf(x.x * up0 * up1, c.x, sum);
            sum = fmaf(x.y * up0 * up1, c.y, sum);
            sum = fmaf(y.x * up0 * up1, f.x, sum);
            sum = fmaf(y.y * up0 * up1, f.y, sum);
        }
    }
    return static_cast<double>(sum) * factor * a.scale * scalbn(1.0, -e);
}

// What half a tile's columns, from c0 on, give the thread's key, those from lo to hi: `offs` times
// `unit` are the logarithms' negatives, +infinity where a row saw nothing.  Where a product of
// codes is out of fp32's range, 32 scores are formed anew; row0 is the tile's first row.
template <int KV, bool F16>
__device__ __noinline__ float sum_with_care(const Args& a, uint32_t scores, int c0, const float* offs, float unit, int lo, int hi,
                                            int64_t cell, int row0, int hk) {
    constexpr bool kCoded = KV != kKvX16;
    const float factor = !kCoded ? 1.0f : cell >= 0 ? a.kscale[cell] : 0.0f, scale = a.scale * factor;
    const uint64_t ff = pair(scale, scale), uu = pair(unit, unit), to2 = pair(kLog2e, kLog2e);
    float sum = 0.0f;
    for (int c = c0; c < min(hi, c0 + kColumns / 2); c += 32) {
        uint32_t v[32];
        tmem_ld32_sync(scores + c, v);
        const ulonglong2* off = reinterpret_cast<const ulonglong2*>(offs + c);
        const int first = lo - c, end = hi - c;
        uint64_t part[2] = {0, 0}, bad = 0;   // `bad` becomes NaN by a product that is not finite
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const ulonglong2 two = off[j / 2];
            const uint64_t o = mul_x2(j & 1 ? two.y : two.x, uu);
            float y0 = __uint_as_float(v[2 * j]), y1 = __uint_as_float(v[2 * j + 1]), x0, x1, o0, o1;
            unpair(mul_x2(fma_x2(pair(y0, y1), ff, o), to2), x0, x1);
            unpair(o, o0, o1);
            const bool in0 = 2 * j >= first && 2 * j < end && o0 != CUDART_INF_F, in1 = 2 * j + 1 >= first && 2 * j + 1 < end && o1 != CUDART_INF_F;
            part[j & 1] = add_x2(part[j & 1], pair(in0 ? exp2_approx(x0) : 0.0f, in1 ? exp2_approx(x1) : 0.0f));
            if (kCoded) bad = fma_x2(pair(in0 ? y0 : 0.0f, in1 ? y1 : 0.0f), 0, bad);
        }
        float p0, p1, b0, b1;
        unpair(add_x2(part[0], part[1]), p0, p1);
        unpair(bad, b0, b1);
        p0 += p1;
        if (kCoded && cell >= 0 && (b0 != 0.0f || b1 != 0.0f || out_of_range(scale, factor))) {
            p0 = 0.0f;
            for (int j = max(lo, c); j < min(hi, c + 32); ++j) {
                const int row = j / static_cast<uint32_t>(a.G);
                const uint16_t* q = a.q + (static_cast<int64_t>(row0) + row) * a.ldq + (hk * a.G + j - row * a.G) * a.D;
                if (offs[j] == CUDART_INF_F) continue;
                const double x = score_of_codes<KV, F16>(a, q, a.k + cell * a.D, factor) + offs[j] * unit;
                p0 += exp2_approx(static_cast<float>(x * kLog2e));
            }
        }
        sum += p0;
        __syncwarp();
    }
    return sum;
}

template <int DP, int KV, bool F16>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a,
                                                           const int R) {
    constexpr bool kCoded = KV != kKvX16;
    constexpr int kQStages = kQStagesOf<DP>;
    constexpr int kHalves = DP / 64, kStageBytes = kHalves * kHalfBytes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sq = smem_u32(smem);
    uint8_t* ctrl = smem + kQStages * kStageBytes;
    const uint32_t cb = smem_u32(ctrl);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + kAbort);
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(ctrl + kTmemPtr);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        prefetch_tensormap(&maps.q);
        for (int i = 0; i < kQStages; ++i) {
            mbar_init(cb + kBarQFull + 8 * i, 1);
            mbar_init(cb + kBarQEmpty + 8 * i, 1);
        }
        for (int i = 0; i < kOffStages; ++i) {
            mbar_init(cb + kBarOffFull + 8 * i, 1);
            mbar_init(cb + kBarOffEmpty + 8 * i, 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(cb + kBarSFull + 8 * i, 1);
            mbar_init(cb + kBarSEmpty + 8 * i, 8);
            mbar_init(cb + kBarKFull + 8 * i, 4);
            mbar_init(cb + kBarKEmpty + 8 * i, 1);
        }
        mbar_init(cb + kBarDrain, 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    grid_dependency_wait();
    // the next kernel is let in once this CTA has its tensor memory: one that took
    // tensor memory first and then waited for this one would never get to run
    if (warp == 3) {
        tmem_alloc(smem_u32(tmem_ptr), kTmemCols);
        tmem_relinquish();
        grid_launch_dependents();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_ptr;
    Item it = {};

    if (warp == 0) {
        // ------------------------------------------------------ queries
        Walker walk(a, lane);
        int n = 0;
        bool ok = true;
        while (ok && walk.next(a, lane, it)) {
            for (int i = it.i0; ok && i < it.nq; i += R, ++n) {
                const int st = n % kQStages;
                ok = mbar_wait(cb + kBarQEmpty + 8 * st, (n / kQStages + 1) & 1, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t bar = cb + kBarQFull + 8 * st;
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar, kHalves * R * a.G * 128);
#pragma unroll
                    for (int h = 0; h < kHalves; ++h)
                        tma_load_3d(sq + st * kStageBytes + h * kHalfBytes, &maps.q, 64 * h, it.hk * a.G, it.q0 + i, bar);
                }
                __syncwarp();
            }
        }
        // let the copies land: after a timeout elsewhere nobody else waits for the last ones
        volatile int no_abort = 0;
        for (int i = n < kQStages ? 0 : n - kQStages; i < n; ++i)
            (void)mbar_wait(cb + kBarQFull + 8 * (i % kQStages), (i / kQStages) & 1, &no_abort);
    } else if (warp == 1) {
        // ----------------------------------------------------- products
        Walker walk(a, lane);
        const int steps = a.D >> 4;
        int n = 0, k = 0;
        bool ok = true;
        while (ok && walk.next(a, lane, it)) {
            ok = __all_sync(0xffffffffu, mbar_wait(cb + kBarKFull + 8 * (k & 1), (k >> 1) & 1, abort_flag));
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t keys = tmem + (k & 1) * 64;
            for (int i = it.i0; ok && i < it.nq; i += R, ++n) {
                const int st = n % kQStages, sb = n & 1;
                // one vote for both: a wait costs some 170 cycles even where nothing is waited for
                ok = vote_wait(lane == 0 ? cb + kBarQFull + 8 * st : cb + kBarSEmpty + 8 * sb,
                               lane == 0 ? (n / kQStages) & 1 : ((n >> 1) + 1) & 1, lane < 2, abort_flag);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t columns = (min(R, it.nq - i) * a.G + 15) & ~15;
                const uint32_t idesc = F16 ? idesc_fp16_f32(128, columns) : idesc_bf16_f32(128, columns);
                const uint64_t bd = smem_desc_kmajor_sw128(sq + st * kStageBytes);
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < DP / 16; ++s)
                        if (s < steps)
                            umma_bf16_tmem_a(tmem + kSCol + sb * kColumns, keys + 8 * s, bd + (s >> 2) * (kHalfBytes >> 4) + (s & 3) * 2,
                                             idesc, s > 0);
                    umma_commit(cb + kBarQEmpty + 8 * st);
                    umma_commit(cb + kBarSFull + 8 * sb);
                }
                __syncwarp();
            }
            if (ok && elect_one()) umma_commit(cb + kBarKEmpty + 8 * (k & 1));
            __syncwarp();
            ++k;
        }
        // let the products finish: after a timeout elsewhere nobody else waits for the last ones
        volatile int no_abort = 0;
        if (elect_one()) umma_commit(cb + kBarDrain);
        __syncwarp();
        (void)mbar_wait(cb + kBarDrain, 0, &no_abort);
    } else if (warp == 2) {
        // --------------------------------------------------- logarithms
        // Loaded two tiles ahead: they come from L2, 1000 cycles away, and a tile takes not
        // much more.
        constexpr int kAhead = 3, kEach = kColumns / 32;
        Walker walk(a, lane);
        float* ring = reinterpret_cast<float*>(ctrl + kOff) + lane;
        int* far = reinterpret_cast<int*>(ctrl + kFar);
        int64_t place[kEach];   // of the lane's columns among the logarithms of a tile
        int row[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            row[e] = (lane + 32 * e) / static_cast<uint32_t>(a.G);
            place[e] = static_cast<int64_t>(row[e]) * a.Hq + (lane + 32 * e - row[e] * a.G);
        }
        const float* src = nullptr;
        float x[kAhead][kEach];
        int left = 0, have = 0, n = 0;   // rows of the item from the next tile on
        bool more = true, ok = true;
        auto load = [&](float (&y)[kEach]) {
            if (left <= 0 && more) {
                more = walk.next(a, lane, it);
                if (more) {
                    left = it.nq - it.i0;
                    src = a.lse + (static_cast<int64_t>(it.q0) + it.i0) * a.Hq + it.hk * a.G;
                }
            }
            if (!more) return;
            const int rows = min(R, left);
#pragma unroll
            for (int e = 0; e < kEach; ++e) y[e] = row[e] < rows ? src[place[e]] : 0.0f;
            src += static_cast<int64_t>(R) * a.Hq;
            left -= R;
            ++have;
        };
#pragma unroll
        for (int i = 0; i < kAhead - 1; ++i) load(x[i]);
        while (ok && n < have) {
            // (by turns, not moved along: a number that is moved is waited for)
#pragma unroll
            for (int now = 0; now < kAhead; ++now) {
                if (!ok || n >= have) break;
                load(x[(now + kAhead - 1) % kAhead]);
                const int st = n % kOffStages;
                ok = __all_sync(0xffffffffu, mbar_wait(cb + kBarOffEmpty + 8 * st, (n / kOffStages + 1) & 1, abort_flag));
                if (!ok) break;
                bool near = true;
#pragma unroll
                for (int e = 0; e < kEach; ++e) near = near && fabsf(x[now][e]) <= kFarLse;   // (not where a row saw nothing)
                near = __all_sync(0xffffffffu, near);
                const float unit = near ? kLog2e : 1.0f;
#pragma unroll
                for (int e = 0; e < kEach; ++e) ring[st * kColumns + 32 * e] = -x[now][e] * unit;
                if (lane == 0) far[st] = !near;
                __syncwarp();
                if (lane == 0) mbar_arrive(cb + kBarOffFull + 8 * st);
                ++n;
            }
        }
        // one more, of no columns: the sums look up a tile's `far` a tile ahead
        const int st = n % kOffStages;
        if (ok && __all_sync(0xffffffffu, mbar_wait(cb + kBarOffEmpty + 8 * st, (n / kOffStages + 1) & 1, abort_flag)) && lane == 0) {
            far[st] = 0;
            mbar_arrive(cb + kBarOffFull + 8 * st);
        }
    } else if (warp >= 4 && warp < 8) {
        // --------------------------------------------------------- keys
        Walker walk(a, lane);
        constexpr int kWords = DP / 2;                       // of a key in tensor memory
        constexpr int kRuns = DP * (kCoded ? 1 : 2) / 16;    // and in the cache
        const uint32_t lanes = tmem + ((warp & 3) << 21);
        const int bytes = a.D * (kCoded ? 1 : 2);
        int k = 0;
        bool ok = true;
        while (ok && walk.next(a, lane, it)) {
            const int key = it.j0 + 32 * (warp & 3) + lane;
            const uint8_t* src = nullptr;
            if (key < it.len) {
                const int page = a.table[it.b * a.max_pages + (key >> a.shift)];
                if (page >= 0 && page < a.num_pages)
                    src = a.k + (((static_cast<int64_t>(page) * a.Hkv + it.hk) << a.shift) + (key & ((1 << a.shift) - 1))) * bytes;
            }
            uint4 u[kRuns];
#pragma unroll
            for (int i = 0; i < kRuns; ++i)
                u[i] = src != nullptr && 16 * i < bytes ? __ldg(reinterpret_cast<const uint4*>(src + 16 * i)) : make_uint4(0, 0, 0, 0);
            ok = __all_sync(0xffffffffu, mbar_wait(cb + kBarKEmpty + 8 * (k & 1), ((k >> 1) + 1) & 1, abort_flag));
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll
            for (int h = 0; h < kWords / 32; ++h) {
                uint32_t v[32];
#pragma unroll
                for (int i = 0; i < 32 / (kCoded ? 8 : 4); ++i) {
                    const uint4& x = u[h * (kCoded ? 4 : 8) + i];
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (kCoded)
                            decode4_as<KV, F16>(w[j], v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
                        else
                            v[4 * i + j] = w[j];
                    }
                }
                tmem_st_32x32b_x32(lanes + (k & 1) * 64 + 32 * h, v);
            }
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(cb + kBarKFull + 8 * (k & 1));
            ++k;
        }
    } else if (warp >= 8) {
        // --------------------------------------------------------- sums
        Walker walk(a, lane);
        const int half = (warp - 8) >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t scores = tmem + kSCol + ((warp & 3) << 21);
        float* partial = reinterpret_cast<float*>(ctrl + kPartial);
        const float* ring = reinterpret_cast<const float*>(ctrl + kOff);
        const int* far_of = reinterpret_cast<const int*>(ctrl + kFar);
        int n = 0, k = 0;
        bool ok = __all_sync(0xffffffffu, mbar_wait(cb + kBarOffFull, 0, abort_flag));
        bool far = ok && far_of[0] != 0;   // of tile n
        while (walk.next(a, lane, it)) {
            const int key = it.j0 + row, before = it.len - it.nq;
            int64_t cell = -1;
            if (key < it.len) {
                const int page = a.table[it.b * a.max_pages + (key >> a.shift)];
                if (page >= 0 && page < a.num_pages)
                    cell = ((static_cast<int64_t>(page) * a.Hkv + it.hk) << a.shift) + (key & ((1 << a.shift) - 1));
            }
            float f = a.scale, old = 0.0f;
            bool wild;
            if constexpr (kCoded) {
                const float factor = cell >= 0 ? a.kscale[cell] : 0.0f;
                f *= factor;
                wild = __any_sync(0xffffffffu, out_of_range(f, factor));
            } else {
                wild = out_of_range(f, 1.0f);
            }
            bool had = false;
            if (half == 0 && cell >= 0) {
                had = key < (a.known == nullptr ? it.len : a.known[it.b]);
                if (had) old = a.weight[cell];
            }
            float sum = 0.0f;
            // Tiles in turn, those with care in a loop of their own (as a choice inside the one
            // loop they made it 5 % slower).  One vote for both: that scores of tile n have come,
            // and of tile n + 1 whether it is to be summed with care.
            for (int i = it.i0; ok && i < it.nq;) {
                for (; i < it.nq && !far && !wild; i += R, ++n) {
                    const int st = n % kOffStages, sb = n & 1, ahead = (n + 1) % kOffStages;
                    const int columns = min(R, it.nq - i) * a.G;
                    const bool full = it.j0 + kKeys - 1 <= before + i;   // every row of the tile sees every key
                    const int first = max(0, key - before - i) * a.G;    // column from which the key is seen
                    ok = ok && vote_wait(lane == 0 ? cb + kBarOffFull + 8 * ahead : cb + kBarSFull + 8 * sb,
                                         lane == 0 ? ((n + 1) / kOffStages) & 1 : (n >> 1) & 1, lane < 2, abort_flag);
                    __syncwarp();
                    if (!ok) break;
                    tc_fence_after_sync();
                    const int next_far = far_of[ahead];
                    uint64_t part[2] = {0, 0};   // pairs of sums
                    const uint64_t ff = pair(f * kLog2e, f * kLog2e);
#pragma unroll 1
                    for (int c = half * (kColumns / 2); c < min(columns, (half + 1) * (kColumns / 2)); c += 32) {
                        uint32_t v[32];
                        tmem_ld32_sync(scores + sb * kColumns + c, v);
                        const ulonglong2* off = reinterpret_cast<const ulonglong2*>(ring + st * kColumns + c);
                        if (full && c + 32 <= columns)
                            add_scores<false>(v, ff, off, 0, 0, part);
                        else   // columns before lo are of rows before the key, those from hi on of none
                            add_scores<true>(v, ff, off, first - c, columns - c, part);
                    }
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(cb + kBarSEmpty + 8 * sb);
                        mbar_arrive(cb + kBarOffEmpty + 8 * st);
                    }
                    float p0, p1;
                    unpair(add_x2(part[0], part[1]), p0, p1);
                    sum += p0 + p1;
                    far = next_far != 0;
                }
                for (; ok && i < it.nq && (far || wild); i += R, ++n) {
                    const int st = n % kOffStages, sb = n & 1, ahead = (n + 1) % kOffStages;
                    ok = vote_wait(lane == 0 ? cb + kBarOffFull + 8 * ahead : cb + kBarSFull + 8 * sb,
                                   lane == 0 ? ((n + 1) / kOffStages) & 1 : (n >> 1) & 1, lane < 2, abort_flag);
                    __syncwarp();
                    if (!ok) break;
                    tc_fence_after_sync();
                    const int next_far = far_of[ahead];
                    sum += sum_with_care<KV, F16>(a, scores + sb * kColumns, half * (kColumns / 2), ring + st * kColumns, far ? 1.0f : kLn2,
                                                  max(0, key - before - i) * a.G, min(R, it.nq - i) * a.G, cell, it.q0 + i, it.hk);
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(cb + kBarSEmpty + 8 * sb);
                        mbar_arrive(cb + kBarOffEmpty + 8 * st);
                    }
                    far = next_far != 0;
                }
            }
            if (!ok) sum = CUDART_NAN_F;
            if (half == 1) partial[(k & 1) * kKeys + row] = sum;
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (half == 0 && cell >= 0) {
                sum += partial[(k & 1) * kKeys + row];
                a.weight[cell] = had ? fmaf(a.decay, old, sum) : sum;
            }
            ++k;
        }
    }
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0 && a.err != nullptr) atomicOr(a.err, 1);
    if (warp == 3) tmem_dealloc(tmem, kTmemCols);
}

template <int DP, int KV, bool F16>
cudaError_t launch(const Args& a, int sm_count, cudaStream_t stream) {
    // rows of a column tile: as many as fit, spread evenly over a sequence's tiles
    const int64_t fit = kColumns / a.G, rows = ceil_div(a.Tq, a.B);
    const int R = static_cast<int>(rows < fit ? rows : ceil_div(rows, ceil_div(rows, fit)));
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    const EncodeTiledFn enc = encode_tiled_fn();
    if (enc == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.D), static_cast<cuuint64_t>(a.Hq), static_cast<cuuint64_t>(a.Tq)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.D) * 2, static_cast<cuuint64_t>(a.ldq) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(R)};
    const cuuint32_t estr[3] = {1, 1, 1};
    if (enc(&maps.q, F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<uint16_t*>(a.q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    static OncePerDevice once;
    const cudaError_t limit = allow_smem(once, rows_kernel<DP, KV, F16>, smem_bytes<DP>());
    if (limit != cudaSuccess) return limit;
    const int64_t items = static_cast<int64_t>(a.B) * a.Hkv * ceil_div(a.capacity, kKeys);
    const dim3 grid(static_cast<unsigned>(items < 1 ? 1 : items < sm_count ? items : sm_count));
    return launch_after(rows_kernel<DP, KV, F16>, grid, kThreads, smem_bytes<DP>(), stream, maps, a, R);
}

template <int DP, bool F16>
cudaError_t launch_kind(int kv, const Args& a, int sm_count, cudaStream_t stream) {
    if (kv == kKvX16) return launch<DP, kKvX16, F16>(a, sm_count, stream);
    if (kv == kKvE4m3) return launch<DP, kKvE4m3, F16>(a, sm_count, stream);
    return launch<DP, kKvI8, F16>(a, sm_count, stream);
}

}  // namespace

bool rows_form(const Args& a) {
    // the tensor map's stride stays below 2^40 bytes
    return by_tma(a) && a.G <= kColumns && a.ldq < (int64_t(1) << 39) && static_cast<int64_t>(a.Tq) * a.G > static_cast<int64_t>(a.B) * 16;
}

cudaError_t launch_rows(bool x_f16, int kv, const Args& a, int sm_count, cudaStream_t stream) {
    if (a.D > 64) return x_f16 ? launch_kind<128, true>(kv, a, sm_count, stream) : launch_kind<128, false>(kv, a, sm_count, stream);
    return x_f16 ? launch_kind<64, true>(kv, a, sm_count, stream) : launch_kind<64, false>(kv, a, sm_count, stream);
}

}  // namespace weights
}  // namespace tern
