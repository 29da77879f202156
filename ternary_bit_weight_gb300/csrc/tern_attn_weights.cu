// Attention weight that each cached token receives from the newest tokens of its
// sequence:
//   add[j] = sum over query rows i that see key j, and the query heads of the
//            key's group, of exp(scale q_i . k_j - lse_i),
// added to the token's weight in a plane that lies like the cache's factors.
//
// Mathematics.  The rows' logarithms are known, so a key's sum needs no other key
// and each key belongs to one warp: no partial results, no atomics, and sums in
// an order that does not depend on timing.  Exponentials are taken in base 2 of
// fma(q.k, scale log2(e), -lse log2(e)): one rounding, of a number that is small
// wherever the weight is not.
//
// What bounds it: for single tokens the keys, read once.
//
// Layout of the work.  An item is one (sequence, key/value head, 8 KB of keys);
// items are dealt to the warps of a persistent grid in turn.  A warp holds its
// keys as operands of mma.sync m16n8k16 (16 keys x 8 columns, a column being one
// query row and head; the order of dimensions inside a product is free, so a
// thread multiplies those it has loaded as 16-byte runs) and passes the columns
// by them.

#include <float.h>
#include <math_constants.h>

#include "tern_attn.cuh"
#include "tern_common.cuh"
#include "tern_internal.h"

namespace tern {
namespace {

constexpr int kWarps = 4;
constexpr int kItemBytes = 8192;     // of keys, per item
constexpr float kLog2e = 1.44269504088896340736f;

struct Args {
    const int32_t* cu_q;
    const int32_t* lens;
    const int32_t* known;
    const int32_t* table;
    const uint16_t* q;
    const float* lse;
    const uint8_t* k;
    const float* kscale;
    float* weight;
    int64_t ldq, max_pages, num_pages;
    int64_t capacity;      // max_pages * page_size
    int B, Tq, Hq, Hkv, G, D;
    int shift;
    float scale2;          // scale * log2(e)
    float decay;
};

struct Sequence {
    int q0, nq, len;
};
__device__ __forceinline__ Sequence sequence_at(const Args& a, int b) {
    Sequence s;
    if (a.cu_q == nullptr) {
        s.q0 = b;
        s.nq = 1;
    } else {
        s.q0 = min(max(a.cu_q[b], 0), a.Tq);
        s.nq = max(0, min(max(a.cu_q[b + 1], 0), a.Tq) - s.q0);
    }
    s.len = static_cast<int>(min(static_cast<int64_t>(max(a.lens[b], 0)), a.capacity));
    return s;
}

template <int DP, int KV, bool F16>
__global__ void __launch_bounds__(kWarps * 32) weights_kernel(const __grid_constant__ Args a) {
    constexpr bool kCoded = KV != kKvX16;
    constexpr bool kMma16 = kCoded || F16;
    constexpr int kElem = kCoded ? 1 : 2, kRowBytes = DP * kElem;
    constexpr int kPieces = kRowBytes / 64;            // 16-byte runs per lane and key
    constexpr int kSteps = DP / 16;
    constexpr int kPer = kSteps / kPieces;             // K-steps of a run
    constexpr int kTiles = kItemBytes / (16 * kRowBytes);
    constexpr int kKeys = 16 * kTiles;
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t step = (int64_t)gridDim.x * kWarps;
    int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int bytes = a.D * kElem;
    const int page_mask = (1 << a.shift) - 1;

    // 32 sequences at a time, one per lane: `incl` counts items up to its end
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        Sequence mine = {0, 0, 0};
        if (b0 + lane < a.B) mine = sequence_at(a, b0 + lane);
        const int64_t each = mine.nq == 0 ? 0 : static_cast<int64_t>((mine.len + (kKeys - 1)) / kKeys) * a.Hkv;
        int64_t incl = each;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += up;
        }
        for (;; item += step) {
            const uint32_t past = __ballot_sync(0xffffffffu, base + incl > item);
            if (past == 0) break;
            const int src = __ffs(past) - 1, b = b0 + src;
            const int len = __shfl_sync(0xffffffffu, mine.len, src), nq = __shfl_sync(0xffffffffu, mine.nq, src);
            const int q0 = __shfl_sync(0xffffffffu, mine.q0, src);
            const int64_t first = base + __shfl_sync(0xffffffffu, incl - each, src);
            const int blocks = (len + (kKeys - 1)) / kKeys;
            const int64_t in = item - first;
            const int hk = (in >> 32) == 0 ? static_cast<uint32_t>(in) / static_cast<uint32_t>(blocks) : static_cast<int>(in / blocks);
            const int j0 = static_cast<int>(in - static_cast<int64_t>(hk) * blocks) * kKeys;

            // ------------------------------------------------ the warp's keys
            uint4 k[kTiles][2][kPieces];
            float kf[kTiles][2];
            int64_t cell[kTiles][2];
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int key = j0 + 16 * m + 8 * r + g;
                    cell[m][r] = -1;
                    if (key < len) {
                        const int page = a.table[static_cast<int64_t>(b) * a.max_pages + (key >> a.shift)];
                        if (page >= 0 && page < a.num_pages)
                            cell[m][r] = ((static_cast<int64_t>(page) * a.Hkv + hk) << a.shift) + (key & page_mask);
                    }
                }
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    kf[m][r] = 1.0f;
                    if (kCoded && cell[m][r] >= 0) kf[m][r] = a.kscale[cell[m][r]];
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const int off = 64 * i + 16 * t;
                        k[m][r][i] = make_uint4(0, 0, 0, 0);
                        if (cell[m][r] >= 0 && off < bytes)
                            k[m][r][i] = __ldg(reinterpret_cast<const uint4*>(a.k + cell[m][r] * bytes + off));
                    }
                }
            const int known = a.known == nullptr ? len : a.known[b];
            float sum[kTiles][2];
#pragma unroll
            for (int m = 0; m < kTiles; ++m) sum[m][0] = sum[m][1] = 0.0f;

            // ------------------------------------------------- the columns
            const int before = len - nq;                 // row i sees keys up to before + i
            const int i0 = max(0, j0 - before);
            const int64_t columns = static_cast<int64_t>(nq) * a.G;
            for (int64_t c0 = static_cast<int64_t>(i0) * a.G; c0 < columns; c0 += 8) {
                // column c0 + g: its query, and what the scores' owners need of it
                const int64_t c = c0 + g;
                const int i = static_cast<int>(c / a.G), head = hk * a.G + static_cast<int>(c - static_cast<int64_t>(i) * a.G);
                const bool live = c < columns;
                uint32_t qb[kSteps][2];
                const uint16_t* src_q = a.q + (q0 + static_cast<int64_t>(i)) * a.ldq + static_cast<int64_t>(head) * a.D;
#pragma unroll
                for (int w = 0; w < kSteps; ++w) {
                    const int d = kCoded ? ((w / 4) * 4 + t) * 16 + (w % 4) * 4 : ((w / 2) * 4 + t) * 8 + (w % 2) * 4;
                    const uint2 u = live && d < a.D ? *reinterpret_cast<const uint2*>(src_q + d) : make_uint2(0, 0);
                    qb[w][0] = u.x;
                    qb[w][1] = u.y;
                }
                float f = a.scale2;
                if constexpr (kCoded) {
                    // times 2^e, so that the row's largest magnitude lies in [2^14, 2^15); or
                    // lower: beyond 2^120 the factor that undoes it would lose bits below
                    // fp32's normal range
                    float top = 0.0f;
#pragma unroll
                    for (int w = 0; w < kSteps; ++w) {
                        const float2 x = unpack_x2<F16>(qb[w][0]), y = unpack_x2<F16>(qb[w][1]);
                        top = fmaxf(top, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y))));
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const int e = top > 0.0f && top <= 3.4e38f ? min(14 - ilogbf(top), 120) : 0;
                    const float up0 = exp2f(static_cast<float>(e / 2)), up1 = exp2f(static_cast<float>(e - e / 2));
                    f = f * exp2f(static_cast<float>(-(e / 2))) * exp2f(static_cast<float>(-(e - e / 2)));
#pragma unroll
                    for (int w = 0; w < kSteps; ++w) {
                        const float2 x = unpack_x2<F16>(qb[w][0]), y = unpack_x2<F16>(qb[w][1]);
                        qb[w][0] = pack_x2<true>(x.x * up0 * up1, x.y * up0 * up1);
                        qb[w][1] = pack_x2<true>(y.x * up0 * up1, y.y * up0 * up1);
                    }
                }
                // last key that the column sees: none without a row, or where the row saw nothing
                const float lse = live ? a.lse[(q0 + static_cast<int64_t>(i)) * a.Hq + head] : -CUDART_INF_F;
                const int last = lse == -CUDART_INF_F ? -1 : before + i;
                float fac[2], off[2];
                int upto[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int from = 4 * (2 * t + h);
                    fac[h] = kCoded ? __shfl_sync(0xffffffffu, f, from) : f;
                    off[h] = __shfl_sync(0xffffffffu, -lse * kLog2e, from);
                    upto[h] = __shfl_sync(0xffffffffu, last, from);
                }
#pragma unroll
                for (int m = 0; m < kTiles; ++m) {
                    float s[2][4];
#pragma unroll
                    for (int n = 0; n < 8; ++n) s[n >> 2][n & 3] = 0.0f;
#pragma unroll
                    for (int p = 0; p < kPieces; ++p) {
                        const uint32_t w0[4] = {k[m][0][p].x, k[m][0][p].y, k[m][0][p].z, k[m][0][p].w};
                        const uint32_t w1[4] = {k[m][1][p].x, k[m][1][p].y, k[m][1][p].z, k[m][1][p].w};
#pragma unroll
                        for (int w = 0; w < kPer; ++w) {
                            uint32_t o[4];   // (key g, key g + 8) x (dimensions 0-1, 2-3)
                            if constexpr (kCoded) {
                                decode4<KV>(w0[w], o[0], o[2]);
                                decode4<KV>(w1[w], o[1], o[3]);
                            } else {
                                o[0] = w0[2 * w], o[2] = w0[2 * w + 1];
                                o[1] = w1[2 * w], o[3] = w1[2 * w + 1];
                            }
                            mma<kMma16>(s[w & 1], o, qb[p * kPer + w][0], qb[p * kPer + w][1]);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float x = s[0][2 * r + h] + s[1][2 * r + h];
                            if (kCoded) x *= kf[m][r];
                            const float p = exp2_approx(fmaf(x, fac[h], off[h]));
                            sum[m][r] += j0 + 16 * m + 8 * r + g <= upto[h] ? p : 0.0f;
                        }
                }
            }
            // -------------------------------------------------- the weights
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float x = sum[m][r];
                    x += __shfl_xor_sync(0xffffffffu, x, 1);
                    x += __shfl_xor_sync(0xffffffffu, x, 2);
                    if (t == r && cell[m][r] >= 0) {
                        float* w = a.weight + cell[m][r];
                        *w = j0 + 16 * m + 8 * r + g < known ? fmaf(a.decay, *w, x) : x;
                    }
                }
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
}

template <int DP, int KV, bool F16>
cudaError_t launch(const Args& a, int sm_count, cudaStream_t stream) {
    constexpr int kKeys = kItemBytes / (DP * (KV == kKvX16 ? 2 : 1));
    const int64_t items = static_cast<int64_t>(a.B) * a.Hkv * ceil_div(a.capacity, kKeys);
    const int64_t most = static_cast<int64_t>(sm_count) * 4;
    const int64_t ctas = ceil_div(items, kWarps);
    const dim3 grid(static_cast<unsigned>(ctas < 1 ? 1 : ctas < most ? ctas : most));
    return launch_after(weights_kernel<DP, KV, F16>, grid, kWarps * 32, 0, stream, a);
}

template <int DP, bool F16>
cudaError_t launch_kind(int kv, const Args& a, int sm_count, cudaStream_t stream) {
    if (kv == kKvX16) return launch<DP, kKvX16, F16>(a, sm_count, stream);
    if (kv == kKvE4m3) return launch<DP, kKvE4m3, F16>(a, sm_count, stream);
    return launch<DP, kKvI8, F16>(a, sm_count, stream);
}

}  // namespace

cudaError_t launch_weights(bool x_f16, const WeightsArgs& w, int sm_count, cudaStream_t stream) {
    Args a = {};
    a.cu_q = w.cu_q;
    a.lens = w.lens;
    a.known = w.known;
    a.table = w.table;
    a.q = w.q;
    a.lse = w.lse;
    a.k = static_cast<const uint8_t*>(w.cache.k);
    a.kscale = w.cache.kscale;
    a.weight = w.weight;
    a.ldq = w.ldq;
    a.max_pages = w.max_pages;
    a.num_pages = w.cache.num_pages;
    a.shift = w.cache.page_shift;
    a.capacity = w.max_pages << a.shift;
    a.B = w.B;
    a.Tq = w.Tq;
    a.Hq = w.Hq;
    a.Hkv = w.Hkv;
    a.G = w.Hq / w.Hkv;
    a.D = w.D;
    a.scale2 = w.scale * kLog2e;
    a.decay = w.decay;
    if (w.D > 64) return x_f16 ? launch_kind<128, true>(w.cache.kv, a, sm_count, stream) : launch_kind<128, false>(w.cache.kv, a, sm_count, stream);
    return x_f16 ? launch_kind<64, true>(w.cache.kv, a, sm_count, stream) : launch_kind<64, false>(w.cache.kv, a, sm_count, stream);
}

}  // namespace tern
