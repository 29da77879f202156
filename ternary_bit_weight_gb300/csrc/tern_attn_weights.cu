// Attention weight that each cached token receives from the newest tokens of its
// sequence:
//   add[j] = sum over query rows i that see key j, and the query heads of the
//            key's group, of exp(scale q_i . k_j - lse_i),
// added to the token's weight in a plane that lies like the cache's factors.
//
// Mathematics.  The rows' logarithms are known, so a key's sum needs no other key
// and each key belongs to one warp: no partial results, no atomics, and sums in
// an order that does not depend on timing.  An exponential's argument is
// fma(q.k, scale, -lse), rounded once, where it is small wherever the weight is not;
// only then is it taken to base 2.  (With scale log2(e) and lse log2(e), each rounded at
// its own size, one operation less: weights of equal scores of 9e6 were off by up to 38 %.)
//
// What bounds it: for single tokens the keys, read once.  Measured, 40 / 8 heads of 128:
// 128 sequences of 8192 over int8 codes 208 us (5.6 TB/s), in bf16 347 us (6.4 TB/s), 32 of up
// to 8192 over e4m3 codes 21 us, one of 701 in bf16 3.8 us a launch in a CUDA graph.
//
// Layout of the work.  The product is mma.sync m16n8k16 with 16 keys as its rows and 8
// columns, a column being one query row and head (tcgen05 would take 128 columns of which
// a single token has 1 to 16; many rows go there, see tern_attn_weights_rows.cu).  The order
// of dimensions inside a product is free, so a thread multiplies those it has loaded as
// 16-byte runs.
//   * stream_kernel: all tiles of 32 keys, one after the other, are cut into equal parts,
//     one for each warp of a persistent grid, which brings them by TMA into a ring of its
//     own; warps never wait for one another.  A tile's scalars (factor, weight so far) are
//     loaded a tile ahead, one key per lane.
//   * any_pages_kernel: pages of fewer than 16 tokens, which a copy does not take: 8 KB of keys
//     at a time straight into registers (the first form of the above: 762 us for the 128
//     sequences over int8 codes, 920 in pages of 8).

#include <float.h>
#include <math_constants.h>
#include <string.h>

#include "tern_attn_weights.cuh"

namespace tern {
namespace {

using weights::Args;
using weights::kLog2e;
using weights::Sequence;
using weights::sequence_at;
using weights::tiles_of;

constexpr int kWarps = 4;
constexpr int kItemBytes = 8192;     // of keys, per item
// A thread's part of 8 columns: operands of its column c0 + g, and what its scores'
// columns c0 + 2t, c0 + 2t + 1 need.
template <int DP>
struct Columns {
    uint32_t q[DP / 16][2];
    float fac[2], off[2];   // a product's weight is exp(product * fac + off)
    int upto[2];            // last key that the column sees
};

// The weight of a product of codes: the column's factor times the key's first, for the
// product times the key's factor could leave fp32's range (tiny queries, scaled up to fp16,
// against large keys) where the score does not.  The product of the two is kept finite: a
// score of zero stays one.
template <bool CODED>
__device__ __forceinline__ float weight_of(float product, float fac, float key, float off) {
    if constexpr (CODED) asm("min.NaN.f32 %0, %1, %2;" : "=f"(fac) : "f"(fac * key), "f"(FLT_MAX));
    return exp2_approx(fmaf(product, fac, off) * kLog2e);
}

// Column c is query row c / G of the sequence and head c mod G of the group.
template <int DP, int KV, bool F16>
__device__ __forceinline__ void load_columns(const Args& a, int q0, int nq, int before, int hk, int64_t c0, int lane, Columns<DP>& o) {
    constexpr bool kCoded = KV != kKvX16;
    constexpr int kSteps = DP / 16;
    const int g = lane >> 2, t = lane & 3;
    const int64_t c = c0 + g;
    const int64_t i = (c >> 32) == 0 ? static_cast<uint32_t>(c) / static_cast<uint32_t>(a.G) : c / a.G;
    const int head = hk * a.G + static_cast<int>(c - i * a.G);
    const bool live = i < nq;
    const uint16_t* src = a.q + (q0 + i) * a.ldq + static_cast<int64_t>(head) * a.D;
#pragma unroll
    for (int w = 0; w < kSteps; ++w) {
        const int d = kCoded ? ((w / 4) * 4 + t) * 16 + (w % 4) * 4 : ((w / 2) * 4 + t) * 8 + (w % 2) * 4;
        const uint2 u = live && d < a.D ? *reinterpret_cast<const uint2*>(src + d) : make_uint2(0, 0);
        o.q[w][0] = u.x;
        o.q[w][1] = u.y;
    }
    float f = a.scale;
    if constexpr (kCoded) {
        // times 2^e, so that the row's largest magnitude lies in [2^14, 2^15); or lower:
        // beyond 2^120 the factor that undoes it would lose bits below fp32's normal range
        float top = 0.0f;
#pragma unroll
        for (int w = 0; w < kSteps; ++w) {
            const float2 x = unpack_x2<F16>(o.q[w][0]), y = unpack_x2<F16>(o.q[w][1]);
            top = fmaxf(top, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = top > 0.0f && top <= 3.4e38f ? min(14 - ilogbf(top), 120) : 0;
        // in two steps: 2^e may pass fp32's range
        const float up0 = exp2f(static_cast<float>(e / 2)), up1 = exp2f(static_cast<float>(e - e / 2));
        f = f * exp2f(static_cast<float>(-(e / 2))) * exp2f(static_cast<float>(-(e - e / 2)));
#pragma unroll
        for (int w = 0; w < kSteps; ++w) {
            const float2 x = unpack_x2<F16>(o.q[w][0]), y = unpack_x2<F16>(o.q[w][1]);
            o.q[w][0] = pack_x2<true>(x.x * up0 * up1, x.y * up0 * up1);
            o.q[w][1] = pack_x2<true>(y.x * up0 * up1, y.y * up0 * up1);
        }
    }
    // no key without a row, or where the row saw nothing
    const float lse = live ? a.lse[(q0 + i) * a.Hq + head] : -CUDART_INF_F;
    const int last = lse == -CUDART_INF_F ? -1 : before + static_cast<int>(i);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int from = 4 * (2 * t + h);
        o.fac[h] = kCoded ? __shfl_sync(0xffffffffu, f, from) : f;
        o.off[h] = __shfl_sync(0xffffffffu, -lse, from);
        o.upto[h] = __shfl_sync(0xffffffffu, last, from);
    }
}

// Scores of 16 keys against 8 columns: k0, k1 hold the thread's runs of the key
// rows g and g + 8.
template <int DP, int KV, bool F16, int PIECES>
__device__ __forceinline__ void multiply(const uint4 (&k0)[PIECES], const uint4 (&k1)[PIECES], const uint32_t (&q)[DP / 16][2],
                                         float (&s)[2][4]) {
    constexpr bool kCoded = KV != kKvX16;
    constexpr int kPer = DP / 16 / PIECES;   // K-steps of a run
#pragma unroll
    for (int n = 0; n < 8; ++n) s[n >> 2][n & 3] = 0.0f;
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
        const uint32_t w0[4] = {k0[p].x, k0[p].y, k0[p].z, k0[p].w}, w1[4] = {k1[p].x, k1[p].y, k1[p].z, k1[p].w};
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
            mma<kCoded || F16>(s[w & 1], o, q[p * kPer + w][0], q[p * kPer + w][1]);
        }
    }
}

// -------------------------------------------------- keys that come by TMA

struct Maps {
    CUtensorMap k;
};

template <int DP, int KV, int COLS>
struct Ring {
    static constexpr int kElem = KV == kKvX16 ? 2 : 1;
    static constexpr int kWarps = 8, kThreads = kWarps * 32;
    static constexpr int kKeys = 32;                                 // of a tile
    static constexpr int kRowBytes = DP * kElem;
    static constexpr int kWidth = kRowBytes < 128 ? kRowBytes : 128; // bytes of a row in one block of the tile
    static constexpr int kBlocks = kRowBytes / kWidth;
    static constexpr int kPieces = kRowBytes / 64;                   // 16-byte runs per lane and key
    static constexpr int kStage = kKeys * kRowBytes;
    static constexpr int kCtas = kStage > 4096 || COLS > 1 ? 1 : 2;  // per SM
    static constexpr int kSmemMax = kCtas == 2 ? 115712 : 232448;
    static constexpr int kFit = (kSmemMax - 1024 - 64) / (kWarps * (kStage + 8));
    static constexpr int kStages = kFit < 4 ? kFit : 4;
    static constexpr int kSmem = 1024 + kWarps * kStages * (kStage + 8) + 64;
    static_assert(kStages >= 3 && kSmem <= kSmemMax, "shared-memory budget");
    // Byte `at` of row `row` (a multiple of 16).
    static __device__ __forceinline__ int place(int row, int at) {
        if (kWidth < 128) return row * kWidth + at;
        return (at >> 7) * (kKeys * 128) + row * 128 + ((at & 127) ^ ((row & 7) << 4));
    }
};

// 32 of a warp's tiles, one per lane.
struct Batch {
    int b, hk, j0;      // sequence, head, first key
    int len;            // keys of the sequence
    int pos[2];         // (page, head) index of the tile's halves, -1: not there
};

template <int DP, int KV, bool F16, int COLS>
__global__ void __launch_bounds__(Ring<DP, KV, COLS>::kThreads, Ring<DP, KV, COLS>::kCtas) stream_kernel(const __grid_constant__ Maps maps,
                                                                                  const __grid_constant__ Args a) {
    using R = Ring<DP, KV, COLS>;
    constexpr bool kCoded = KV != kKvX16;
    constexpr int kStages = R::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint8_t* ring = smem + warp * kStages * R::kStage;
    const uint32_t bars = smem_u32(smem + R::kWarps * kStages * R::kStage) + warp * kStages * 8;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + R::kWarps * kStages * (R::kStage + 8));
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        prefetch_tensormap(&maps.k);
    }
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(bars + 8 * i, 1);
        mbar_fence_init();
    }
    __syncthreads();
    grid_launch_dependents();
    grid_dependency_wait();

    // ------------------------------------------------- the warp's tiles [u0, u1)
    Sequence mine = {0, 0, 0};   // of the 32 sequences from b0, one per lane
    int64_t incl = 0, base = 0;  // their tiles up to the lane's end, and those before
    int b0 = 0, cur = 0;
    auto load_sequences = [&]() {
        mine = {0, 0, 0};
        if (b0 + lane < a.B) mine = sequence_at(a, b0 + lane);
        incl = tiles_of(a, mine, R::kKeys);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += up;
        }
    };
    load_sequences();
    int64_t total = __shfl_sync(0xffffffffu, incl, 31);
    if (a.B > 32) {
        int64_t more = 0;
        for (int b = 32 + lane; b < a.B; b += 32) more += tiles_of(a, sequence_at(a, b), R::kKeys);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) more += __shfl_xor_sync(0xffffffffu, more, d);
        total += more;
    }
    const uint32_t warps = gridDim.x * R::kWarps, w = blockIdx.x * R::kWarps + warp;
    int64_t u0, u1;
    if (total < (int64_t(1) << 31) / warps) {
        u0 = static_cast<uint32_t>(total) * w / warps;
        u1 = static_cast<uint32_t>(total) * (w + 1) / warps;
    } else {
        u0 = total * w / warps;
        u1 = total * (w + 1) / warps;
    }
    const int page_mask = (1 << a.shift) - 1;
    // the tiles from u on: each lane finds its own
    auto find = [&](int64_t u) {
        Batch o = {0, 0, 0, 0, {-1, -1}};
        u += lane;
        bool found = u >= u1;
        for (;;) {
            const int64_t end = base + __shfl_sync(0xffffffffu, incl, cur);
            const Sequence s = {__shfl_sync(0xffffffffu, mine.q0, cur), __shfl_sync(0xffffffffu, mine.nq, cur),
                                __shfl_sync(0xffffffffu, mine.len, cur)};
            if (!found && u < end) {
                found = true;
                const uint32_t tiles = (s.len + (R::kKeys - 1)) / R::kKeys;
                const int64_t in = u - (end - static_cast<int64_t>(tiles) * a.Hkv);
                o.hk = (in >> 32) == 0 ? static_cast<uint32_t>(in) / tiles : static_cast<int>(in / tiles);
                o.j0 = static_cast<int>(in - static_cast<int64_t>(o.hk) * tiles) * R::kKeys;
                o.b = b0 + cur;
                o.len = s.len;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int key = o.j0 + 16 * h;
                    if (key < s.len) {
                        const int page = a.table[o.b * a.max_pages + (key >> a.shift)];
                        if (page >= 0 && page < a.num_pages) o.pos[h] = page * a.Hkv + o.hk;
                    }
                }
            }
            if (__all_sync(0xffffffffu, found)) return o;
            if (++cur == 32) {   // tiles are left, so sequences are
                base += __shfl_sync(0xffffffffu, incl, 31);
                b0 += 32;
                cur = 0;
                load_sequences();
            }
        }
    };
    const int count = static_cast<int>(u1 - u0);
    if (count == 0) return;
    Batch now = find(u0), next = now;
    // field of tile i, which is in this batch (of tile c) or the next
    auto pick = [&](int c, int i, int Batch::*field) {
        return __shfl_sync(0xffffffffu, (i >> 5) == (c >> 5) ? now.*field : next.*field, i & 31);
    };
    auto pick_pos = [&](int c, int i, int h) {
        return __shfl_sync(0xffffffffu, (i >> 5) == (c >> 5) ? now.pos[h] : next.pos[h], i & 31);
    };
    auto issue = [&](int c, int i, int stage) {
        const int p0 = pick_pos(c, i, 0), p1 = pick_pos(c, i, 1), row = pick(c, i, &Batch::j0) & page_mask;
        const uint32_t st = smem_u32(ring + stage * R::kStage), bar = bars + 8 * stage;
        if (elect_one()) {
            mbar_arrive_expect_tx(bar, ((p0 >= 0) + (p1 >= 0)) * (R::kStage / 2));
#pragma unroll
            for (int n = 0; n < R::kBlocks; ++n) {
                const uint32_t dst = st + n * R::kKeys * R::kWidth;
                const int x = n * (R::kWidth / R::kElem);
                if (p0 >= 0) tma_load_3d(dst, &maps.k, x, row, p0, bar);
                if (p1 >= 0) tma_load_3d(dst + 16 * R::kWidth, &maps.k, x, (row + 16) & page_mask, p1, bar);
            }
        }
        __syncwarp();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        if (i < count) issue(0, i, i);

    // Rows of a 16-key product that are in one quarter of a shared-memory access
    // differ in bit 2 (runs are swizzled by the row), so row g is key kr.  A lane
    // has the scalars of key `own` of a tile.
    const int kr = (g >> 1) | ((g & 1) << 2), own = 16 * (t >> 1) + 8 * (t & 1) + kr;
    // cell, factor and weight so far of the lane's key of tile i (cell -1: not there)
    auto scalars = [&](int c, int i, int64_t& cell, float& factor, float& old) {
        const int key = pick(c, i, &Batch::j0) + own, len = pick(c, i, &Batch::len);
        const int p0 = pick_pos(c, i, 0), p1 = pick_pos(c, i, 1), p = t >> 1 ? p1 : p0;
        cell = key < len && p >= 0 ? (static_cast<int64_t>(p) << a.shift) + (key & page_mask) : -1;
        factor = kCoded && cell >= 0 ? a.kscale[cell] : 1.0f;
        old = cell >= 0 ? a.weight[cell] : 0.0f;
    };
    int64_t cell;
    float factor, old;
    scalars(0, 0, cell, factor, old);

    Columns<DP> cols[COLS];
    int seq = -1, head = -1, before = 0, known = 0;
    Sequence s = {0, 0, 0};
    int stage = 0, fill = kStages - 1;
    uint32_t phase = 0;
    for (int c = 0; c < count; ++c) {
        if (c > 0 && (c & 31) == 0) now = next;
        __syncwarp();   // every lane has read the stage that is filled now
        const int ahead = c + kStages - 1;
        if (ahead < count) {
            if ((ahead & 31) == 0) next = find(u0 + ahead);
            issue(c, ahead, fill);
        }
        if (++fill == kStages) fill = 0;
        int64_t next_cell = -1;
        float next_factor = 1.0f, next_old = 0.0f;
        if (c + 1 < count) scalars(c, c + 1, next_cell, next_factor, next_old);

        const int j0 = pick(c, c, &Batch::j0), b = pick(c, c, &Batch::b), hk = pick(c, c, &Batch::hk);
        const bool other = b != seq || hk != head;
        if (b != seq) {
            s = sequence_at(a, b);
            before = s.len - s.nq;
            known = a.known == nullptr ? s.len : a.known[b];
        }
        seq = b;
        head = hk;
        const bool got = mbar_wait(bars + 8 * stage, phase, abort_flag);
        __syncwarp();
        const uint8_t* st = ring + stage * R::kStage;
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
        }
        float sum[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
        const int64_t columns = static_cast<int64_t>(s.nq) * a.G;
        const bool held = columns <= 8 * COLS;   // they stay from tile to tile
        for (int64_t c0 = held ? 0 : static_cast<int64_t>(max(0, j0 - before)) * a.G; c0 < columns; c0 += 8 * COLS) {
            if (!held || other) {
#pragma unroll
                for (int n = 0; n < COLS; ++n) load_columns<DP, KV, F16>(a, s.q0, s.nq, before, hk, c0 + 8 * n, lane, cols[n]);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint4 k0[R::kPieces], k1[R::kPieces];
#pragma unroll
                for (int i = 0; i < R::kPieces; ++i) {
                    k0[i] = lds_v4(st + R::place(16 * m + kr, 64 * i + 16 * t));
                    k1[i] = lds_v4(st + R::place(16 * m + 8 + kr, 64 * i + 16 * t));
                }
                const float f0 = __shfl_sync(0xffffffffu, factor, 4 * g + 2 * m), f1 = __shfl_sync(0xffffffffu, factor, 4 * g + 2 * m + 1);
#pragma unroll
                for (int n = 0; n < COLS; ++n) {
                    float x[2][4];
                    multiply<DP, KV, F16, R::kPieces>(k0, k1, cols[n].q, x);
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float y = x[0][2 * r + h] + x[1][2 * r + h];
                            const float p = weight_of<kCoded>(y, cols[n].fac[h], r ? f1 : f0, cols[n].off[h]);
                            if (j0 + 16 * m + 8 * r + kr <= cols[n].upto[h]) sum[m][r] += p;
                        }
                }
            }
        }
        // the four lanes of a row have its sums; each keeps that of its own key
        float x = 0.0f;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float y = sum[m][r];
                y += __shfl_xor_sync(0xffffffffu, y, 1);
                y += __shfl_xor_sync(0xffffffffu, y, 2);
                if (t == 2 * m + r) x = y;
            }
        if (!got) {   // the keys did not come
            x = CUDART_NAN_F;
            if (lane == 0 && a.err != nullptr) atomicOr(a.err, 1);
        }
        if (cell >= 0) a.weight[cell] = j0 + own < known ? fmaf(a.decay, old, x) : x;
        cell = next_cell;
        factor = next_factor;
        old = next_old;
    }
    // copies are all consumed, unless a wait ran out: let them land
    if (*abort_flag) {
        volatile int no_abort = 0;
        for (int i = 0; i < kStages; ++i) {
            (void)mbar_wait(bars + 8 * i, 0, &no_abort);
            (void)mbar_wait(bars + 8 * i, 1, &no_abort);
        }
    }
}

// ------------------------------------------------------- keys of any pages

template <int DP, int KV, bool F16>
__global__ void __launch_bounds__(kWarps * 32) any_pages_kernel(const __grid_constant__ Args a) {
    constexpr bool kCoded = KV != kKvX16;
    constexpr int kElem = kCoded ? 1 : 2, kRowBytes = DP * kElem;
    constexpr int kPieces = kRowBytes / 64;            // 16-byte runs per lane and key
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
        const int64_t each = tiles_of(a, mine, kKeys);
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
            const int64_t columns = static_cast<int64_t>(nq) * a.G;
            for (int64_t c0 = static_cast<int64_t>(max(0, j0 - before)) * a.G; c0 < columns; c0 += 8) {
                Columns<DP> col;
                load_columns<DP, KV, F16>(a, q0, nq, before, hk, c0, lane, col);
#pragma unroll
                for (int m = 0; m < kTiles; ++m) {
                    float s[2][4];
                    multiply<DP, KV, F16, kPieces>(k[m][0], k[m][1], col.q, s);
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float x = s[0][2 * r + h] + s[1][2 * r + h];
                            const float p = weight_of<kCoded>(x, col.fac[h], kf[m][r], col.off[h]);
                            if (j0 + 16 * m + 8 * r + g <= col.upto[h]) sum[m][r] += p;
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

template <int DP, int KV, bool F16, int COLS>
cudaError_t launch_stream(const Args& a, int sm_count, cudaStream_t stream) {
    using R = Ring<DP, KV, COLS>;
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    const EncodeTiledFn enc = encode_tiled_fn();
    if (enc == nullptr) return cudaErrorNotSupported;
    const CUtensorMapDataType type = KV != kKvX16 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : F16        ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const cuuint64_t row = static_cast<cuuint64_t>(a.D) * R::kElem;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.D), static_cast<cuuint64_t>(1) << a.shift,
                                static_cast<cuuint64_t>(a.num_pages * a.Hkv)};
    const cuuint64_t strides[2] = {row, row << a.shift};
    const cuuint32_t box[3] = {R::kWidth / R::kElem, R::kKeys / 2, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    if (enc(&maps.k, type, 3, const_cast<uint8_t*>(a.k), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            R::kWidth == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    static OncePerDevice once;
    const cudaError_t limit = allow_smem(once, stream_kernel<DP, KV, F16, COLS>, R::kSmem);
    if (limit != cudaSuccess) return limit;
    // a CTA for every 8 tiles that there may be
    const int64_t ctas = ceil_div(static_cast<int64_t>(a.B) * a.Hkv * ceil_div(a.capacity, R::kKeys), R::kWarps);
    const int64_t most = static_cast<int64_t>(sm_count) * R::kCtas;
    const dim3 grid(static_cast<unsigned>(ctas < 1 ? 1 : ctas < most ? ctas : most));
    return launch_after(stream_kernel<DP, KV, F16, COLS>, grid, R::kThreads, R::kSmem, stream, maps, a);
}

template <int DP, int KV, bool F16>
cudaError_t launch(const Args& a, int sm_count, cudaStream_t stream) {
    if (weights::by_tma(a))
        return a.G <= 8 ? launch_stream<DP, KV, F16, 1>(a, sm_count, stream) : launch_stream<DP, KV, F16, 2>(a, sm_count, stream);
    constexpr int kKeys = kItemBytes / (DP * (KV == kKvX16 ? 2 : 1));
    const int64_t items = static_cast<int64_t>(a.B) * a.Hkv * ceil_div(a.capacity, kKeys);
    const int64_t most = static_cast<int64_t>(sm_count) * 4;
    const int64_t ctas = ceil_div(items, kWarps);
    const dim3 grid(static_cast<unsigned>(ctas < 1 ? 1 : ctas < most ? ctas : most));
    return launch_after(any_pages_kernel<DP, KV, F16>, grid, kWarps * 32, 0, stream, a);
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
    a.err = w.err;
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
    a.scale = w.scale;
    a.decay = w.decay;
    // many rows against many keys are the tensor cores' work
    if (weights::rows_form(a)) return weights::launch_rows(x_f16, w.cache.kv, a, sm_count, stream);
    if (w.D > 64) return x_f16 ? launch_kind<128, true>(w.cache.kv, a, sm_count, stream) : launch_kind<128, false>(w.cache.kv, a, sm_count, stream);
    return x_f16 ? launch_kind<64, true>(w.cache.kv, a, sm_count, stream) : launch_kind<64, false>(w.cache.kv, a, sm_count, stream);
}

}  // namespace tern
