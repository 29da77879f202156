// Attention of single tokens over the paged cache:
//   O = softmax(scale q K^T) V, one query row per sequence and head.
//
// Mathematics.  The softmax is taken in base 2 (s = scale log2(e) q.k) in one
// pass over the keys with a running reference m: a row keeps l = sum 2^(s-m)
// and o = sum 2^(s-m) v, both rescaled when m moves, and partial results
// (m, l, o) of disjoint key ranges add after rescaling to the larger m.  m
// follows the running maximum lazily: it moves only when a score passes it by
// 8, so weights stay below 2^8 and most tiles need one vote instead of a
// reduction.  With coded values v = c f (code times factor) the products with
// V use the codes, exact in fp16, and weights 2^((s - m) + log2 f - r) with a
// reference r of their own, so that factors of any size keep the weights
// within fp16; keys' factors multiply the scores.  (r is relative to m, and the
// difference s - m taken first: log2 f added to a large score is lost in its
// rounding.)  Queries are brought to fp16 by a power of two per row, which the
// scores' factor undoes.  Weights are rounded to 16 bits for that product, whose
// operands have one type; l sums them unrounded.  (Relative distance from 64 bits:
// bf16 values 0.0021, and 0.0017 with the output's rounding alone; fp16 weights over
// codes add nothing to 0.0017.)
//
// What bounds it: the bytes of the cache, read once (the G query heads of a
// key/value head are rows of the same products).
// Measured, 40 / 8 heads of 128: 128 sequences of 8192 over int8 codes 338 us
// (6.6 TB/s), two of 32768 in fp16 49.1 us (5.5 TB/s), 32 of up to 8192 over e4m3
// codes 39.3 us, one of 701 8.7 us, of which some 8 us are launch, start and join.
//
// Work.  An item is one (sequence, key/value head); its tiles of 16 keys are
// dealt to the CTAs in one of three ways (see Share), a segment being the part of
// an item that a CTA has.  Within a segment the warps take the tiles in turn;
// at its end their (m, l, o) meet in shared memory.  An item inside one CTA is
// then finished; otherwise the CTAs leave partial results in the workspace and
// the last to arrive adds them in CTA order (the result does not depend on
// timing).
//
// A warp's tiles land in a ring of its own, so warps never wait for one
// another inside a segment.  Pages of 16 tokens and more hold a tile as one
// block: two TMA copies per 128 bytes of a row's width bring it, 128-byte
// swizzled, issued by one lane.  (A copy per lane and 16 bytes instead costs
// some 60 instructions of a tile's 500 and fills the load/store queue.)
// Smaller pages take that per-lane form, cp.async to the same layout.
//
// The products are mma.sync m16n8k16 with the heads as the 8 columns:
// S^T = K q^T (16 keys x 8 heads), then o^T += V^T P^T (16 dimensions x 8
// heads), P transposed between the two by movmatrix.  With the heads as the 16
// rows instead, half of every product and accumulator is empty for groups of
// up to 8 heads.  The order of dimensions inside a product is free, so each
// thread multiplies the dimensions it has loaded: keys need no transposition,
// values only a byte or half-word interleave of two rows.  The order of keys in
// a tile is free too: kKey picks it so that the reads of keys and of values
// both meet every bank once.  (tcgen05 would take 128-row tiles of which 1 to
// 16 rows exist here.)

#include <cuda.h>
#include <float.h>
#include <math_constants.h>
#include <string.h>

#include "tern_attn.cuh"
#include "tern_common.cuh"
#include "tern_internal.h"
#include "tern_sm100.cuh"

namespace tern {
namespace {

constexpr int kTile = 16;              // keys per unit
constexpr int kRows = 16;              // query heads per pass over the keys
constexpr int kMinTiles = 8;           // of a CTA, one per warp
constexpr int kEnd = 8;                // what ending a segment costs, in tiles
constexpr int kJoin = 24;              // what a second segment and the joining of parts cost, in tiles
constexpr float kPart = 2.4f;          // what adding a part costs, against an eighth of a tile
constexpr int kFirst = 4;              // parts that a join loads before it knows their statistics
constexpr float kLazy = 8.0f;          // how far a score may pass the reference
constexpr float kNone = -FLT_MAX;      // reference before any key: no finite score is below it
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

struct Args {
    const int32_t* lens;
    const int32_t* table;
    const uint8_t* k;
    const uint8_t* v;
    const float* kscale;
    const float* vscale;
    const uint16_t* q;
    uint16_t* o;
    float* lse;
    int* err;
    int32_t* arrived;      // [grid], zero between calls
    float* slots;          // [2 * grid] partial results
    int64_t ldq, ldo, max_pages, num_pages;
    int64_t capacity;      // max_pages * page_size
    float slack;           // see share_of
    int B, D, G;           // G query heads share a key/value head
    int Hkv, passes, Hv;   // Hv = Hkv * passes: (key/value head, 16 of its query heads)
    int shift;
    int tma;               // tiles come by TMA (else a copy per lane)
    int narrow;            // all of the work's weight x CTAs is below 2^31
    float scale2;          // scale * log2(e)
};

struct Maps {
    CUtensorMap k, v;
};


// Key of the tile at row g (or slot g) of a product's 8-key half.  Rows are
// 128 bytes, their 16-byte runs swizzled by the row: run c of row r is at
// c ^ (r mod 8).  Keys are read as runs 0-3 (or 4-7) of rows kKey(2i) and
// kKey(2i + 1) together, which must differ in bit 2; values as runs 2i, 2i + 1
// of the four rows kKey(0, 2, 4, 6) (or 1, 3, 5, 7), which must differ above
// bit 0.
__device__ __forceinline__ int key_at(int g) { return (0x37156240u >> (4 * g)) & 7; }   // 0 4 2 6 5 1 7 3

// COLS: columns of heads, 8 each (1 for groups of up to 8 heads, else 2).
template <int DP, int KV, int COLS>
struct Shape {
    static constexpr int kElem = KV == kKvX16 ? 2 : 1;
    // Coded tiles are half the bytes and take twice the instructions per byte:
    // two CTAs of 8 warps and 128 registers on an SM, so that one streams while
    // the other ends a segment.  The rest needs the registers, or the ring, of one.
    static constexpr int kCtas = KV != kKvX16 && COLS == 1 ? 2 : 1;
    // SMs take tiles from L2 so much faster than all of them get them from memory
    static constexpr float kSlack = KV == kKvX16 ? 1.6f : KV == kKvE4m3 ? 1.2f : 1.05f;
    static constexpr int kWarps = 8;
    static constexpr int kSmemMax = kCtas == 2 ? 115712 : 232448;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kRowBytes = DP * kElem;
    static constexpr int kWidth = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a row in one block of the tile
    static constexpr int kBlocks = kRowBytes / kWidth;
    static constexpr int kKPieces = kRowBytes / 64;                   // 16-byte runs per lane and key row
    static constexpr int kVRun = kRowBytes / 8 < 16 ? kRowBytes / 8 : 16;
    static constexpr int kVPieces = kRowBytes / 8 / kVRun;            // runs per lane and value row
    static constexpr int kKBytes = kTile * kRowBytes;
    static constexpr int kStage = 2 * kKBytes;
    static constexpr int kScaleBytes = KV == kKvX16 ? 0 : 2 * kTile * 4;
    static constexpr int kSteps = DP / 16;                            // K-steps of a score, row tiles of the output
    static constexpr int kMerge = kWarps * 8 * DP * 4;
    static constexpr int kStat = kWarps * 8 * COLS * 3 * 4;
    static constexpr int kFit = (kSmemMax - 1024 - kMerge - kStat - 64) / (kWarps * (kStage + kScaleBytes + 8));
    static constexpr int kStages = kFit < 4 ? kFit : 4;
    static constexpr int kSmem = 1024 + kWarps * kStages * (kStage + kScaleBytes + 8) + kMerge + kStat + 64;
    static constexpr int kEach = 8 * DP / kThreads;                   // merged elements per thread
    static_assert(kStages >= 2 && (kEach == 2 || kEach == 4) && kWarps == 8 && kSmem <= kSmemMax, "shape");
    // Dimension of row g (half 0) or g + 8 (half 1) of output row tile j: a
    // thread's dimensions are those of the value runs it loads.
    static __device__ __forceinline__ int dim(int g, int half, int j) {
        return KV == kKvX16 && DP == 128 ? 64 * half + 8 * g + j : (DP / 8) * g + (DP / 16) * half + j;
    }
    // Byte `at` (a multiple of 16, or 8 in narrow rows) of a row of the tile.
    static __device__ __forceinline__ int place(int row, int at) {
        if (kWidth < 128) return row * kWidth + at;
        return (at >> 7) * (kTile * 128) + row * 128 + ((at & 127) ^ ((row & 7) << 4));
    }
    // Place of a key row's run 64 * i bytes after the one at `place` (i counts up
    // from the row's start).
    static __device__ __forceinline__ int k_run(int place, int i) { return (place ^ ((i & 1) * 64)) + (i >> 1) * kTile * 128; }
    // Element d of a head's row in a warp's merge block (spread over the banks).
    static __device__ __forceinline__ int merge_at(int row, int d) {
        return row * DP + ((((d >> 2) ^ (row >> 1)) << 2) | (d & 3));
    }
};

__host__ __device__ constexpr int slot_floats(int DP, int rows) { return rows * (DP + 3); }

// N (2 or 4) floats at once.
template <int N>
struct __align__(4 * N) Floats {
    float v[N];
};
template <int N>
__device__ __forceinline__ Floats<N> load_l2(const float* p) {
    Floats<N> x;
    if constexpr (N == 4) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(p));
        x.v[0] = u.x, x.v[1] = u.y, x.v[2] = u.z, x.v[3] = u.w;
    } else {
        const float2 u = __ldcg(reinterpret_cast<const float2*>(p));
        x.v[0] = u.x, x.v[1] = u.y;
    }
    return x;
}

template <int BYTES>
__device__ __forceinline__ void copy_async_or_zero(uint32_t dst, const void* src, bool there) {
    const int n = there ? BYTES : 0;   // the rest is filled with zeros
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values, thread (g, t) holding
// elements 2t, 2t + 1 of row g.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Count an arrival; what the CTA wrote before is visible to the CTAs that arrive
// later, and theirs before to this one.
__device__ __forceinline__ int arrive(int32_t* counter) {
    int before;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    return before;
}

// The larger of two references of the products with V, finite.
__device__ __forceinline__ float join_reference(float a, float b) { return fmaxf(fmaxf(a, b), kNone); }

__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float warp_add(float x) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}
__device__ __forceinline__ float log2_approx(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The four codes of a word as two fp16 pairs, exactly.
template <int KV>
__device__ __forceinline__ void decode4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (KV == kKvE4m3) {
        const __half2 a = e4m3x2_to_half2(w & 0xFFFFu), b = e4m3x2_to_half2(w >> 16);
        lo = *reinterpret_cast<const uint32_t*>(&a);
        hi = *reinterpret_cast<const uint32_t*>(&b);
    } else {
        // byte + 128 in the low mantissa bits of 1024.0, less 1152
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t x = __byte_perm(u, 0x64646464u, 0x4140), y = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
        const __half2 a = __hsub2(*reinterpret_cast<const __half2*>(&x), bias);
        const __half2 b = __hsub2(*reinterpret_cast<const __half2*>(&y), bias);
        lo = *reinterpret_cast<const uint32_t*>(&a);
        hi = *reinterpret_cast<const uint32_t*>(&b);
    }
}

// One segment: the tiles [begin, end) of item (b, hv).
struct Segment {
    int b, hv;
    int len, tiles;      // keys and tiles of sequence b
    int begin, end;
    int64_t start;       // dealing by weight: where the item starts
    int64_t left;        // and what is left of the CTA's part after it
    int64_t item;        // dealing whole items: what each takes of `left` (else 0)
};

// How the tiles are dealt to the CTAs.
//   * whole == 0, by weight: an item weighs its tiles and kEnd more, and the
//     items' weights, one after the other, are cut into equal parts, one per
//     CTA, so unequal lengths load the SMs equally.  The first kEnd of an item
//     stand for no tile: a cut that falls there splits no item.
//   * whole == q: an item of n tiles goes to ceil(n / q) CTAs of its own, one
//     segment each.
//   * several == k: a CTA has k items, whole.
// The last two have fewer segments and partial results than by weight, and less
// equal loads.  Where the loads are within `slack` of equal, and kJoin, they are
// faster, because the memory is what is busy, not every SM: bf16 cache of 18 sequences of 4064 (144
// items for 152 CTAs) 50.1 us against 55 by weight, 32 of 2272 (two items each) 51
// against 55; e4m3 codes of 30 of 3000 (240 for 304) 37.4 against 41.8, int8 of 32
// of 512 11.8 against 17.4.  (int8 codes of 128 of 8192 in fours, 1.19 times the
// equal load, 367 against 338: there the SMs are as busy as the memory.)
struct Share {
    int whole, several;
    int64_t weight;      // by weight: of all items
    int64_t ctas;        // that have a part
    int64_t items;
    uint32_t ctas0;      // dealing a CTA or more to an item: CTAs of an item of the lane's first sequence
};

__device__ __forceinline__ int length_of(const Args& a, int b) {
    return static_cast<int>(min(static_cast<int64_t>(max(a.lens[b], 0)), a.capacity));
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// The arithmetic of the start is done in T: 32 bits where the host has seen that
// the largest product fits (64-bit divisions and their code made the start of a
// short call 1 us longer), else 64 bits.
template <typename T>
__device__ __forceinline__ T warp_sum(T n) {
    if constexpr (sizeof(T) == 4) {
        return __reduce_add_sync(0xffffffffu, n);
    } else {
        const int64_t lo = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(n) & 0xFFFFFFu);
        const int64_t hi = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(n >> 24));   // n is below 2^51
        return lo + (hi << 24);
    }
}

// `mine` is the length of the lane's first sequence (0 where there is none).
template <typename T>
__device__ __forceinline__ Share share_of(const Args& a, int lane, int mine) {
    T tiles = 0;
    uint32_t some = 0, most = 0;
    for (int b = lane; b < a.B; b += 32) {
        const uint32_t n = tiles_of(b == lane ? mine : length_of(a, b));
        tiles += n;
        some += n > 0;
        most = max(most, n);
    }
    tiles = warp_sum<T>(tiles) * a.Hv;
    const T items = static_cast<T>(__reduce_add_sync(0xffffffffu, some)) * a.Hv;
    const T grid = gridDim.x;
    Share s;
    s.whole = s.several = 0;
    s.ctas0 = 0;
    const T weight = tiles + kEnd * items;
    s.weight = weight;
    T ctas = tiles == 0 ? T(0) : max(T(1), min(grid, max(items, weight / (kMinTiles + kEnd))));
    // the weight that a CTA may have when items are not cut by weight
    const float bound = a.slack * __fdividef(static_cast<float>(weight), static_cast<float>(ctas)) + kJoin;
    most = __reduce_max_sync(0xffffffffu, most);
    if (items >= grid) {
        const T k = (items + grid - 1) / grid;
        if (static_cast<float>(k) * static_cast<float>(most + kEnd) <= bound && k <= T(INT32_MAX)) {
            s.several = static_cast<int>(k);
            ctas = (items + k - 1) / k;
        }
    } else if (tiles > 0) {
        // an item's parts add up one after the other: n tiles are split no finer
        // than where a tile less per warp costs as much as the parts it adds
        const T even = static_cast<T>(sqrtf(kPart * __fdividef(static_cast<float>(tiles), static_cast<float>(items))));
        const T q = max(max(T(kMinTiles), even), (tiles + grid - items - 1) / (grid - items));
        if (most <= q) {   // a CTA per item
            if (static_cast<float>(most + kEnd) <= bound) {
                s.whole = static_cast<int>(most);
                s.ctas0 = mine > 0;
                ctas = items;
            }
        } else {   // so q is below 2^31
            T parts = 0;
            float load = 0.0f;   // the largest of a CTA
            for (int b = lane; b < a.B; b += 32) {
                const uint32_t n = tiles_of(b == lane ? mine : length_of(a, b));
                const uint32_t some = (n + static_cast<uint32_t>(q) - 1) / static_cast<uint32_t>(q);
                parts += some;
                if (b == lane) s.ctas0 = some;
                if (some > 0) load = fmaxf(load, __fdividef(static_cast<float>(n), static_cast<float>(some)));
            }
            if (warp_max(load) + kEnd <= bound) {
                s.whole = static_cast<int>(q);
                ctas = warp_sum<T>(parts) * a.Hv;
            }
        }
    }
    s.ctas = ctas;
    s.items = items;
    return s;
}

// The next item's part; the caller has seen that there is one (left > kEnd).
__device__ __forceinline__ void next_segment(const Args& a, Segment& s) {
    s.start += s.tiles + kEnd;
    if (++s.hv == a.Hv) {
        s.hv = 0;
        do {
            s.len = length_of(a, ++s.b);   // weight remains, so a sequence that has some follows
        } while (s.len == 0);
        s.tiles = tiles_of(s.len);
    }
    s.begin = 0;
    s.end = static_cast<int>(min(static_cast<int64_t>(s.tiles), s.left - kEnd));
    s.left -= s.item ? s.item : s.end + kEnd;
}

// The CTA's first segment (one warp); begin == end: it has none.
template <typename T>
__device__ __forceinline__ Segment first_segment(const Args& a, const Share& share, int lane, int mine) {
    Segment s;
    const T cta = blockIdx.x, weight = static_cast<T>(share.weight), ctas = static_cast<T>(share.ctas);
    const T k = share.several;
    const T u0 = share.whole ? cta : k ? cta * k : weight * cta / ctas;
    const T u1 = share.whole || k ? u0 + 1 : weight * (cta + 1) / ctas;
    s.item = 0;
    T base = 0;
    for (int b0 = 0;; b0 += 32) {
        const int len = b0 == 0 ? mine : b0 + lane < a.B ? length_of(a, b0 + lane) : 0;
        const uint32_t tiles = tiles_of(len);
        // CTAs, number (1) or weight of an item: below 2^28
        const uint32_t each = tiles == 0 ? 0 : k ? 1
                              : share.whole ? b0 == 0 ? share.ctas0 : (tiles + share.whole - 1) / static_cast<uint32_t>(share.whole) : tiles + kEnd;
        T incl = static_cast<T>(each) * a.Hv;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const T up = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += up;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, base + incl > u0);
        if (past != 0) {   // u0 is below the total, so some lane finds it
            const int src = __ffs(past) - 1;
            s.b = b0 + src;
            s.len = __shfl_sync(0xffffffffu, len, src);
            s.tiles = tiles_of(s.len);
            const T n = __shfl_sync(0xffffffffu, each, src);
            const T in = u0 - base - (__shfl_sync(0xffffffffu, incl, src) - n * a.Hv);
            s.hv = static_cast<int>(n == 1 ? in : in / n);
            const int at = static_cast<int>(in - s.hv * n);
            if (share.whole) {
                const int per = static_cast<int>((s.tiles + static_cast<uint32_t>(n) - 1) / static_cast<uint32_t>(n));
                s.start = cta - at;
                s.begin = at * per;
                s.end = min(s.tiles, s.begin + per);
                s.left = 0;
            } else if (k) {
                s.item = int64_t(1) << 32;   // more than an item weighs
                s.start = 0;
                s.begin = 0;
                s.end = s.tiles;
                s.left = (min(k, static_cast<T>(share.items) - u0) - 1) * s.item;
            } else {
                const int upto = static_cast<int>(min(n, at + (u1 - u0)));
                s.start = u0 - at;
                s.begin = max(0, at - kEnd);
                s.end = max(s.begin, upto - kEnd);
                s.left = (u1 - u0) - (upto - at);
                if (s.begin == s.end && s.left > kEnd) next_segment(a, s);
            }
            return s;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
}

// Share and first segment of the CTA; false: it has none.
template <typename T>
__device__ __forceinline__ bool start(const Args& a, int lane, int mine, Share& share, Segment& s) {
    share = share_of<T>(a, lane, mine);
    if (blockIdx.x >= share.ctas) return false;
    s = first_segment<T>(a, share, lane, mine);
    return s.begin != s.end;
}
__device__ __noinline__ bool start_wide(const Args& a, int lane, int mine, Share& share, Segment& s) {
    return start<int64_t>(a, lane, mine, share, s);
}

// CTAs that have a part of the segment's item.
template <typename T>
__device__ __forceinline__ void parts_of(const Share& share, const Segment& s, int& c0, int& c1) {
    if (share.whole) {
        c0 = static_cast<int>(s.start);
        c1 = c0 + static_cast<int>((static_cast<uint32_t>(s.tiles) + share.whole - 1) / static_cast<uint32_t>(share.whole)) - 1;
    } else {
        // the CTA that has weight unit u of the total W is the last c with W c / C <= u
        const T u = static_cast<T>(s.start) + kEnd, weight = static_cast<T>(share.weight), ctas = static_cast<T>(share.ctas);
        c0 = static_cast<int>(((u + 1) * ctas - 1) / weight);
        c1 = static_cast<int>(((u + s.tiles) * ctas - 1) / weight);
    }
}
__device__ __noinline__ void parts_of_wide(const Share& share, const Segment& s, int& c0, int& c1) {
    parts_of<int64_t>(share, s, c0, c1);
}

template <int DP, int KV, bool F16, int COLS>
__global__ void __launch_bounds__(Shape<DP, KV, COLS>::kThreads, Shape<DP, KV, COLS>::kCtas) decode_kernel(const __grid_constant__ Maps maps,
                                                                                const __grid_constant__ Args a) {
    using S = Shape<DP, KV, COLS>;
    constexpr bool kCoded = KV != kKvX16;
    constexpr bool kMma16 = kCoded || F16;       // products in fp16 (else bf16)
    constexpr int kWarps = S::kWarps, kThreads = S::kThreads, kSlotRows = 8 * COLS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint8_t* ring = smem + warp * S::kStages * S::kStage;
    uint8_t* factors = smem + kWarps * S::kStages * S::kStage + warp * S::kStages * S::kScaleBytes;
    float* merge = reinterpret_cast<float*>(smem + kWarps * S::kStages * (S::kStage + S::kScaleBytes));
    float* stat = merge + S::kMerge / 4;         // [warp][row][m, r, l]
    const uint32_t bars = smem_u32(stat + S::kStat / 4) + warp * S::kStages * 8;   // a warp's stages
    volatile int* last_flag = reinterpret_cast<volatile int*>(reinterpret_cast<uint8_t*>(stat) + S::kStat +
                                                             kWarps * S::kStages * 8);
    volatile int* part_info = last_flag + 2;     // [2][4]
    volatile int* abort_flag = last_flag + 10;
    if (threadIdx.x == 0) *abort_flag = 0;
    if (lane == 0) {
        for (int i = 0; i < S::kStages; ++i) mbar_init(bars + 8 * i, 1);
        mbar_fence_init();
    }
    if (threadIdx.x == 0 && a.tma) {
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
    }
    __syncthreads();

    grid_launch_dependents();
    grid_dependency_wait();

    const int mine0 = lane < a.B ? length_of(a, lane) : 0;   // the lane's first sequence
    // sequences of length zero see nothing
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (length_of(a, b) != 0) continue;
        const int n = a.Hkv * a.G * a.D;
        for (int i = threadIdx.x * 8; i < n; i += kThreads * 8)
            *reinterpret_cast<uint4*>(a.o + b * a.ldo + i) = make_uint4(0, 0, 0, 0);
        if (a.lse != nullptr)
            for (int h = threadIdx.x; h < a.Hkv * a.G; h += kThreads)
                a.lse[static_cast<int64_t>(b) * a.Hkv * a.G + h] = -CUDART_INF_F;
    }

    Share share;
    Segment seg;
    if (!(a.narrow ? start<uint32_t>(a, lane, mine0, share, seg) : start_wide(a, lane, mine0, share, seg))) return;

    // ---------------------------------------------------- loads of a warp
    // Page ids are looked up for a batch of up to 32 of the warp's tiles in one
    // load: lane i holds the (page, head) index of the batch's tile i, or -1
    // where its page is outside the cache.
    Segment ls = seg;                 // segment of the batch
    int lt = ls.begin + warp;         // first tile of the batch
    int batch = 0, taken = 0, pos = 0;
    int hk_at = 0;                    // (pages of fewer than 16 tokens look theirs up tile by tile)
    auto refill = [&]() {
        lt += taken * kWarps;
        taken = 0;
        while (lt >= ls.end) {
            if (ls.left <= kEnd) {
                batch = 0;
                return;
            }
            next_segment(a, ls);
            lt = warp;
        }
        batch = min(32, (ls.end - lt + kWarps - 1) / kWarps);
        hk_at = a.passes == 1 ? ls.hv : ls.hv / a.passes;
        if (a.tma) {
            const int key = min(lt + lane * kWarps, ls.end - 1) * kTile;
            const int page = a.table[static_cast<int64_t>(ls.b) * a.max_pages + (key >> a.shift)];
            pos = page >= 0 && page < a.num_pages ? page * a.Hkv + hk_at : -1;
        }
    };
    const int bytes = a.D * S::kElem;
    const int page_mask = (1 << a.shift) - 1;
    uint64_t masks = 0;   // 16 bits per tile in flight: its keys that exist
    auto issue = [&](int stage, int ahead) {
        if (taken == batch) refill();
        uint32_t mask = 0;
        if (batch > 0) {
            const uint32_t st = smem_u32(ring + stage * S::kStage), fs = smem_u32(factors + stage * S::kScaleBytes);
            const int key0 = (lt + taken * kWarps) * kTile;
            const int at = __shfl_sync(0xffffffffu, pos, taken);
            ++taken;
            if (a.tma) {
                // a tile lies in one page
                const bool there = at >= 0;
                mask = there ? 0xFFFFu >> max(0, key0 + kTile - ls.len) : 0u;
                const uint32_t bar = bars + 8 * stage;
                const int row = key0 & page_mask;
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar, there ? S::kStage + S::kScaleBytes : 0);
                    if (there) {
#pragma unroll
                        for (int i = 0; i < S::kBlocks; ++i) {
                            tma_load_3d(st + i * kTile * S::kWidth, &maps.k, i * (S::kWidth / S::kElem), row, at, bar);
                            tma_load_3d(st + S::kKBytes + i * kTile * S::kWidth, &maps.v, i * (S::kWidth / S::kElem), row, at, bar);
                        }
                        if constexpr (kCoded) {
                            const int64_t cell = (static_cast<int64_t>(at) << a.shift) + row;
                            bulk_load(fs, a.kscale + cell, kTile * 4, bar);
                            bulk_load(fs + kTile * 4, a.vscale + cell, kTile * 4, bar);
                        }
                    }
                }
                __syncwarp();
            } else {
                // cell of the lane's key (lane mod 16), negative where there is none
                const int key = key0 + (lane & 15);
                int64_t cell = -1;
                if (key < ls.len) {
                    const int page = a.table[static_cast<int64_t>(ls.b) * a.max_pages + (key >> a.shift)];
                    if (page >= 0 && page < a.num_pages)
                        cell = ((static_cast<int64_t>(page) * a.Hkv + hk_at) << a.shift) + (key & page_mask);
                }
                mask = __ballot_sync(0xffffffffu, cell >= 0) & 0xFFFFu;
                constexpr int kRuns = S::kRowBytes / 16, kAtOnce = 32 / kRuns;   // rows per step
#pragma unroll
                for (int i = 0; i < kTile / kAtOnce; ++i) {
                    const int row = i * kAtOnce + lane / kRuns, off = (lane % kRuns) * 16;
                    const int64_t c = __shfl_sync(0xffffffffu, cell, row);
                    const bool there = c >= 0 && off < bytes;
                    const int dst = S::place(row, off);
                    copy_async_or_zero<16>(st + dst, there ? a.k + c * bytes + off : a.k, there);
                    copy_async_or_zero<16>(st + S::kKBytes + dst, there ? a.v + c * bytes + off : a.v, there);
                }
                if constexpr (kCoded) {
                    const float* src = lane < 16 ? a.kscale : a.vscale;
                    copy_async_or_zero<4>(fs + lane * 4, cell >= 0 ? src + cell : src, cell >= 0);
                }
            }
        }
        if (!a.tma) copy_commit();
        masks |= static_cast<uint64_t>(mask) << (16 * ahead);
    };

#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) issue(i, i);
    const int kr = key_at(g);   // keys kr and kr + 8 are the thread's rows of the scores
    const int vr[4] = {key_at(2 * t), key_at(2 * t + 1), key_at(2 * t) + 8, key_at(2 * t + 1) + 8};
    // where the thread's runs lie in a tile (rows 8 apart are kWidth * 8 apart,
    // the swizzle being the same; a run 64 bytes on is the one with bit 6 turned)
    const int k_place = S::place(kr, t * 16), v_place[2] = {S::place(vr[0], g * S::kVRun), S::place(vr[1], g * S::kVRun)};
    int stage = 0, fill = S::kStages - 1;
    uint32_t phase = 0;

    // queries of head 8c + g: the four dimensions of each K-step that the thread's
    // key runs hold
    uint32_t qb[COLS][S::kSteps][2];
    auto load_queries = [&](const Segment& s) {
        const int hk = a.passes == 1 ? s.hv : s.hv / a.passes;
        const int head0 = (s.hv - hk * a.passes) * kRows;
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
            const bool live = 8 * c + g < min(kRows, a.G - head0);
            const uint16_t* src = a.q + s.b * a.ldq + (static_cast<int64_t>(hk) * a.G + head0 + 8 * c + g) * a.D;
#pragma unroll
            for (int w = 0; w < S::kSteps; ++w) {
                const int d = kCoded ? ((w / 4) * 4 + t) * 16 + (w % 4) * 4 : ((w / 2) * 4 + t) * 8 + (w % 2) * 4;
                const uint2 u = live && d < a.D ? *reinterpret_cast<const uint2*>(src + d) : make_uint2(0, 0);
                qb[c][w][0] = u.x;
                qb[c][w][1] = u.y;
            }
        }
    };
    load_queries(seg);
    // partial results left so far (in part_info: b, hv, first and last CTA of the
    // item).  The CTA arrives for them when its tiles are done: in mid-stream the
    // arrival waits for stores that queue with the loads of the SM, and its warp
    // fell 6 us behind.
    int parts = 0;

    // a warp stores the finished sums of one head
    auto finish = [&](const Segment& s, int head, const float (&sum)[S::kEach], float M, float R, float L) {
        const int hk = a.passes == 1 ? s.hv : s.hv / a.passes;
        const int64_t q_head = static_cast<int64_t>(hk) * a.G + (s.hv - hk * a.passes) * kRows + head;
        // (exact below 2^-126, too, which the reference of small values comes to)
        const float f = L == 0.0f ? 0.0f : exp2f(R) / L;
        const int d = lane * S::kEach;
        if (d < a.D) {
            uint16_t* dst = a.o + s.b * a.ldo + q_head * a.D + d;
            if constexpr (S::kEach == 4)
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack_x2<F16>(sum[0] * f, sum[1] * f), pack_x2<F16>(sum[2] * f, sum[3] * f));
            else
                *reinterpret_cast<uint32_t*>(dst) = pack_x2<F16>(sum[0] * f, sum[1] * f);
        }
        if (lane == 0 && a.lse != nullptr)
            a.lse[static_cast<int64_t>(s.b) * a.Hkv * a.G + q_head] = L == 0.0f ? -CUDART_INF_F : M * kLn2 + logf(L);
    };

    // ------------------------------------------------------------ segments
    for (;;) {
        const int hk = a.passes == 1 ? seg.hv : seg.hv / a.passes;
        const int head0 = (seg.hv - hk * a.passes) * kRows;               // first of the group's heads
        const int heads = min(kRows, a.G - head0);
        // the thread's heads: 8c + 2t, 8c + 2t + 1
        float m[COLS][2], r[COLS][2], l[COLS][2], fac[COLS][2];
        float o[COLS][S::kSteps][4];
        const bool mine = seg.begin + warp < seg.end;
        if (mine) {
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
                float f = a.scale2;
                if constexpr (kCoded) {
                    // times 2^e, so that the row's largest magnitude lies in [2^14, 2^15); or
                    // lower: beyond 2^120 the factor that undoes it would lose bits below
                    // fp32's normal range, and a row of bf16's smallest normal numbers is at
                    // 2^-6 by then, well inside fp16's
                    float top = 0.0f;
#pragma unroll
                    for (int w = 0; w < S::kSteps; ++w) {
                        const float2 x = unpack_x2<F16>(qb[c][w][0]), y = unpack_x2<F16>(qb[c][w][1]);
                        top = fmaxf(top, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y))));
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const int e = top > 0.0f && top <= 3.4e38f ? min(14 - ilogbf(top), 120) : 0;
                    // in two steps: 2^e may pass fp32's range
                    const float up0 = exp2f(static_cast<float>(e / 2)), up1 = exp2f(static_cast<float>(e - e / 2));
                    f = f * exp2f(static_cast<float>(-(e / 2))) * exp2f(static_cast<float>(-(e - e / 2)));
#pragma unroll
                    for (int w = 0; w < S::kSteps; ++w) {
                        const float2 x = unpack_x2<F16>(qb[c][w][0]), y = unpack_x2<F16>(qb[c][w][1]);
                        qb[c][w][0] = pack_x2<true>(x.x * up0 * up1, x.y * up0 * up1);
                        qb[c][w][1] = pack_x2<true>(y.x * up0 * up1, y.y * up0 * up1);
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    fac[c][h] = kCoded ? __shfl_sync(0xffffffffu, f, 4 * (2 * t + h)) : f;
                    m[c][h] = r[c][h] = kNone;
                    l[c][h] = 0.0f;
                }
#pragma unroll
                for (int j = 0; j < S::kSteps; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[c][j][i] = 0.0f;
            }
        }

        for (int tile = seg.begin + warp; tile < seg.end; tile += kWarps) {
            __syncwarp();   // every lane has read the stage that is filled now
            issue(fill, S::kStages - 1);
            if (++fill == S::kStages) fill = 0;
            if (a.tma) {
                // after a timeout the rest runs through without waiting
                if (!mbar_wait(bars + 8 * stage, phase, abort_flag) && lane == 0) atomicOr(a.err, 1);
            } else {
                copy_wait<S::kStages - 1>();
            }
            __syncwarp();   // the lanes' copies are visible to one another
            const uint8_t* st = ring + stage * S::kStage;
            const float* ks = reinterpret_cast<const float*>(factors + stage * S::kScaleBytes);
            if (++stage == S::kStages) {
                stage = 0;
                phase ^= 1u;
            }
            const uint32_t mask = static_cast<uint32_t>(masks) & 0xFFFFu;
            masks >>= 16;

            // ------------------------------------------------ scores
            // two chains of products, added at the end
            float s[COLS][2][4];
#pragma unroll
            for (int c = 0; c < COLS; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) s[c][i >> 2][i & 3] = 0.0f;
#pragma unroll
            for (int i = 0; i < S::kKPieces; ++i) {
                const uint4 u0 = *reinterpret_cast<const uint4*>(st + S::k_run(k_place, i));
                const uint4 u1 = *reinterpret_cast<const uint4*>(st + S::k_run(k_place, i) + 8 * S::kWidth);
                const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
                constexpr int kPer = kCoded ? 4 : 2;   // K-steps of a run
#pragma unroll
                for (int w = 0; w < kPer; ++w) {
                    uint32_t k[4];   // (key g, key g + 8) x (dimensions 0-1, 2-3)
                    if constexpr (kCoded) {
                        decode4<KV>(w0[w], k[0], k[2]);
                        decode4<KV>(w1[w], k[1], k[3]);
                    } else {
                        k[0] = w0[2 * w], k[2] = w0[2 * w + 1];
                        k[1] = w1[2 * w], k[3] = w1[2 * w + 1];
                    }
#pragma unroll
                    for (int c = 0; c < COLS; ++c) mma<kMma16>(s[c][w & 1], k, qb[c][i * kPer + w][0], qb[c][i * kPer + w][1]);
                }
            }
            // the thread's keys: kr, kr + 8
            float kf[2] = {1, 1}, vl[2] = {0, 0};
            if constexpr (kCoded) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    kf[k] = ks[kr + 8 * k];
                    vl[k] = log2_approx(ks[kTile + kr + 8 * k]);
                }
            }
            float x[COLS][4];   // [key][head]: key kr heads 2t, 2t+1; key kr + 8 the same
#pragma unroll
            for (int c = 0; c < COLS; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // rounded before the reference is taken off, which is one of them
                    x[c][i] = __fmul_rn(s[c][0][i] + s[c][1][i], fac[c][i & 1]);
                    if (kCoded) x[c][i] = __fmul_rn(x[c][i], kf[i >> 1]);
                }
            if (mask != 0xFFFFu) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (!((mask >> (kr + 8 * k)) & 1u)) {
                        vl[k] = 0.0f;
#pragma unroll
                        for (int c = 0; c < COLS; ++c) x[c][2 * k] = x[c][2 * k + 1] = -CUDART_INF_F;
                    }
            }
            // ------------------------------------------- references
            float top[COLS][2], topo[COLS][2];
            bool past = false;
#pragma unroll
            for (int c = 0; c < COLS; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    top[c][h] = fmaxf(x[c][h], x[c][2 + h]);
                    past = past || top[c][h] > m[c][h] + kLazy;
                    if (kCoded) {
                        topo[c][h] = fmaxf((x[c][h] - m[c][h]) + vl[0], (x[c][2 + h] - m[c][h]) + vl[1]);
                        past = past || topo[c][h] > r[c][h] + kLazy;
                    }
                }
            if (__any_sync(0xffffffffu, past)) {
#pragma unroll
                for (int c = 0; c < COLS; ++c) {
                    float f[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float up = top[c][h];   // over the lanes that share t
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, d));
                        up = fmaxf(m[c][h], up);
                        const float moved = m[c][h] - up;
                        f[h] = exp2_approx(moved);
                        l[c][h] *= f[h];
                        m[c][h] = up;
                        if (kCoded) {
                            up = fmaxf((x[c][h] - m[c][h]) + vl[0], (x[c][2 + h] - m[c][h]) + vl[1]);
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, d));
                            up = join_reference(r[c][h] + moved, up);
                            f[h] = exp2_approx(moved + (r[c][h] - up));
                            r[c][h] = up;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < S::kSteps; ++j) {
                        o[c][j][0] *= f[0], o[c][j][1] *= f[1];
                        o[c][j][2] *= f[0], o[c][j][3] *= f[1];
                    }
                }
            }
            // ---------------------------------------------- weights
            uint32_t p[COLS][2];
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float past_m = x[c][i] - m[c][i & 1];
                    w[i] = exp2_approx(past_m);
                    l[c][i & 1] += w[i];
                    if (kCoded) w[i] = exp2_approx((past_m + vl[i >> 1]) - r[c][i & 1]);
                }
                p[c][0] = transpose8(pack_x2<kMma16>(w[0], w[1]));
                p[c][1] = transpose8(pack_x2<kMma16>(w[2], w[3]));
            }
            // ----------------------------------------------- values
            // row tile j of the output: dimensions dim(g, 0, j) and dim(g, 1, j); an
            // operand register holds two keys of a dimension: slots 2t, 2t + 1 or 8 more
            const uint8_t* sv = st + S::kKBytes;
            if constexpr (kCoded) {
                constexpr int kWords = S::kVRun / 4, kHalf = kWords / 2;
                uint32_t v[4][kWords];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint8_t* src = sv + v_place[j & 1] + (j >> 1) * 8 * S::kWidth;
                    if constexpr (kWords == 4) {
                        const uint4 u = *reinterpret_cast<const uint4*>(src);
                        v[j][0] = u.x, v[j][1] = u.y, v[j][2] = u.z, v[j][3] = u.w;
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2*>(src);
                        v[j][0] = u.x, v[j][1] = u.y;
                    }
                }
                if (mask != 0xFFFFu) {   // what lies there for keys that do not exist must not meet a weight of zero
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < kWords; ++i) v[j][i] = (mask >> vr[j]) & 1u ? v[j][i] : 0u;
                }
#pragma unroll
                for (int q = 0; q < kHalf; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t sel = h ? 0x7362 : 0x5140;
                        uint32_t x0[2], x1[2], x2[2], x3[2];
                        decode4<KV>(__byte_perm(v[0][q], v[1][q], sel), x0[0], x0[1]);
                        decode4<KV>(__byte_perm(v[0][q + kHalf], v[1][q + kHalf], sel), x1[0], x1[1]);
                        decode4<KV>(__byte_perm(v[2][q], v[3][q], sel), x2[0], x2[1]);
                        decode4<KV>(__byte_perm(v[2][q + kHalf], v[3][q + kHalf], sel), x3[0], x3[1]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t av[4] = {x0[i], x1[i], x2[i], x3[i]};
#pragma unroll
                            for (int c = 0; c < COLS; ++c) mma<kMma16>(o[c][4 * q + 2 * h + i], av, p[c][0], p[c][1]);
                        }
                    }
            } else {
                uint32_t v[4][4 * S::kVPieces];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < S::kVPieces; ++i) {
                        const uint4 u = *reinterpret_cast<const uint4*>(sv + v_place[j & 1] + (j >> 1) * 8 * S::kWidth +
                                                                           i * kTile * 128);
                        v[j][4 * i] = u.x, v[j][4 * i + 1] = u.y, v[j][4 * i + 2] = u.z, v[j][4 * i + 3] = u.w;
                    }
                if (mask != 0xFFFFu) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < 4 * S::kVPieces; ++i) v[j][i] = (mask >> vr[j]) & 1u ? v[j][i] : 0u;
                }
                constexpr int kHalf = 2 * S::kVPieces;   // words from a tile's first dimension to its second
#pragma unroll
                for (int q = 0; q < kHalf; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t sel = h ? 0x7632 : 0x5410;
                        const uint32_t av[4] = {__byte_perm(v[0][q], v[1][q], sel),
                                                __byte_perm(v[0][q + kHalf], v[1][q + kHalf], sel),
                                                __byte_perm(v[2][q], v[3][q], sel),
                                                __byte_perm(v[2][q + kHalf], v[3][q + kHalf], sel)};
#pragma unroll
                        for (int c = 0; c < COLS; ++c) mma<kMma16>(o[c][2 * q + h], av, p[c][0], p[c][1]);
                    }
            }
        }

        // ------------------------------------------- the segment's sum
        // the next segment's queries are on their way meanwhile
        const Segment done = seg;
        const bool another = seg.left > kEnd;
        if (another) {
            next_segment(a, seg);
            load_queries(seg);
        }
        const int active = min(kWarps, done.end - done.begin);   // warps that had a tile
        const bool whole = done.begin == 0 && done.end == done.tiles;
        if (mine) {
#pragma unroll
            for (int c = 0; c < COLS; ++c)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l[c][h] += __shfl_xor_sync(0xffffffffu, l[c][h], d);
                    if (g == 0) {
                        float* dst = stat + (warp * kSlotRows + 8 * c + 2 * t + h) * 3;
                        dst[0] = m[c][h];
                        dst[1] = kCoded ? r[c][h] : 0.0f;
                        dst[2] = l[c][h];
                    }
                }
        }
        // partial results: the CTA that begins an item uses its odd slot, the
        // others their even one
        float* slot = a.slots + (2 * static_cast<int64_t>(blockIdx.x) + (done.begin == 0 ? 1 : 0)) * slot_floats(DP, kSlotRows);
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
            if (mine) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float* dst = merge + warp * 8 * DP;
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int j = 0; j < S::kSteps; j += 4)
                            *reinterpret_cast<float4*>(dst + S::merge_at(2 * t + h, S::dim(g, half, j))) =
                                make_float4(o[c][j][2 * half + h], o[c][j + 1][2 * half + h], o[c][j + 2][2 * half + h],
                                            o[c][j + 3][2 * half + h]);
                }
            }
            __syncthreads();
            const int head = 8 * c + warp;   // a warp adds up one head, a lane kEach of its elements
            if (head < heads) {
                const float* sp = stat + ((lane & 7) * kSlotRows + head) * 3;
                const bool had = lane < active;
                const float M = warp_max(had ? sp[0] : kNone);
                const float L = warp_add(had ? sp[2] * exp2_approx(sp[0] - M) : 0.0f);
                const float ri = had ? sp[1] + (sp[0] - M) : kNone, R = join_reference(kNone, warp_max(ri));
                const float fw = had ? exp2_approx(ri - R) : 0.0f;
                float sum[S::kEach];
#pragma unroll
                for (int i = 0; i < S::kEach; ++i) sum[i] = 0.0f;
                for (int w = 0; w < active; ++w) {
                    const float f = __shfl_sync(0xffffffffu, fw, w);
                    const Floats<S::kEach> x =
                        *reinterpret_cast<const Floats<S::kEach>*>(merge + w * 8 * DP + S::merge_at(warp, lane * S::kEach));
#pragma unroll
                    for (int i = 0; i < S::kEach; ++i) sum[i] += x.v[i] * f;
                }
                if (whole) {
                    finish(done, head, sum, M, R, L);
                } else {
                    Floats<S::kEach> x;
#pragma unroll
                    for (int i = 0; i < S::kEach; ++i) x.v[i] = sum[i];
                    *reinterpret_cast<Floats<S::kEach>*>(slot + head * DP + lane * S::kEach) = x;
                    if (lane == 0) {
                        float* dst = slot + kSlotRows * DP + head * 3;
                        dst[0] = M;
                        dst[1] = R;
                        dst[2] = L;
                    }
                }
            }
            __syncthreads();
        }
        if (!whole) {
            // at most two of a CTA's segments are parts of an item: its first and its last
            if (threadIdx.x == 0) {
                int c0, c1;
                if (a.narrow) parts_of<uint32_t>(share, done, c0, c1);
                else parts_of_wide(share, done, c0, c1);
                volatile int* info = part_info + 4 * (parts & 1);
                info[0] = done.b, info[1] = done.hv, info[2] = c0, info[3] = c1;
            }
            ++parts;
        }
        if (!another) break;
    }

    // the last CTA to arrive adds the parts of an item, in CTA order
    if (lane == 0 && warp < parts) {   // warp 0, which has just written it, takes the last part
        const int n = parts - 1 - warp;
        last_flag[n] = arrive(a.arrived + part_info[4 * n + 2]) == part_info[4 * n + 3] - part_info[4 * n + 2];
    }
    __syncthreads();
    for (int n = 0; n < parts; ++n) {
        if (!last_flag[n]) continue;
        Segment done;
        done.b = part_info[4 * n], done.hv = part_info[4 * n + 1];
        const int c0 = part_info[4 * n + 2], c1 = part_info[4 * n + 3];
        const int hk = a.passes == 1 ? done.hv : done.hv / a.passes;
        const int heads = min(kRows, a.G - (done.hv - hk * a.passes) * kRows);
        auto part = [&](int cta) {
            return a.slots + (2 * static_cast<int64_t>(cta) + (cta == c0 ? 1 : 0)) * slot_floats(DP, kSlotRows);
        };
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
            const int head = 8 * c + warp;
            if (head >= heads) continue;
            float M = kNone, R = kNone, L = 0.0f;
            float sum[S::kEach];
#pragma unroll
            for (int i = 0; i < S::kEach; ++i) sum[i] = 0.0f;
            for (int i0 = c0; i0 <= c1; i0 += 32) {   // a lane has one part's statistics
                const int count = min(32, c1 - i0 + 1);
                // the first parts are on their way with the statistics
                Floats<S::kEach> x0[kFirst];
#pragma unroll
                for (int k = 0; k < kFirst; ++k)
                    x0[k] = load_l2<S::kEach>(part(i0 + min(k, count - 1)) + head * DP + lane * S::kEach);
                const float* sp = part(i0 + min(lane, count - 1)) + kSlotRows * DP + head * 3;
                const bool had = lane < count;
                const float mi = had ? __ldcg(sp) : kNone, rp = had ? __ldcg(sp + 1) : kNone, li = had ? __ldcg(sp + 2) : 0.0f;
                const float up = fmaxf(M, warp_max(mi)), before = R + (M - up), ri = rp + (mi - up);
                R = join_reference(before, warp_max(had ? ri : kNone));
                const float keep = exp2_approx(before - R), f = exp2_approx(ri - R);
                L = L * exp2_approx(M - up) + li * exp2_approx(mi - up);
                M = up;
#pragma unroll
                for (int i = 0; i < S::kEach; ++i) sum[i] *= keep;
#pragma unroll
                for (int k = 0; k < kFirst; ++k) {
                    const float fk = k < count ? __shfl_sync(0xffffffffu, f, k) : 0.0f;
#pragma unroll
                    for (int i = 0; i < S::kEach; ++i)
                        if (k < count) sum[i] += x0[k].v[i] * fk;
                }
#pragma unroll 4
                for (int k = kFirst; k < count; ++k) {
                    const Floats<S::kEach> x = load_l2<S::kEach>(part(i0 + k) + head * DP + lane * S::kEach);
                    const float fk = __shfl_sync(0xffffffffu, f, k);
#pragma unroll
                    for (int i = 0; i < S::kEach; ++i) sum[i] += x.v[i] * fk;
                }
            }
            finish(done, head, sum, M, R, warp_add(L));
        }
        if (threadIdx.x == 0) a.arrived[c0] = 0;
    }
    // copies are all consumed, unless a wait ran out: let them land
    if (a.tma && *abort_flag) {
        volatile int no_abort = 0;
        for (int i = 0; i < S::kStages; ++i) {
            (void)mbar_wait(bars + 8 * i, 0, &no_abort);
            (void)mbar_wait(bars + 8 * i, 1, &no_abort);
        }
    }
}

int group_rows(int64_t G) { return G > 8 ? 16 : 8; }

// CTAs of a call; `most` is what the GPU holds at once.
int grid_size(int64_t B, int64_t Hv, int64_t max_len, int64_t most) {
    // one CTA per kMinTiles tiles, and one more per item for what is left over
    const int64_t ctas = B * Hv * (max_len / (kTile * kMinTiles) + 1);
    return static_cast<int>(ctas < 1 ? 1 : ctas < most ? ctas : most);
}

template <int DP, int KV, bool F16, int COLS>
cudaError_t launch(Args& a, const DecodeArgs& d, int sm_count, cudaStream_t stream) {
    using S = Shape<DP, KV, COLS>;
    const int grid = grid_size(d.B, a.Hv, a.capacity, static_cast<int64_t>(sm_count) * S::kCtas);
    a.slack = S::kSlack;
    a.narrow = static_cast<double>(d.B) * a.Hv * static_cast<double>(a.capacity / kTile + 1 + kEnd) * (grid + 1) < 2147483648.0;
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    // pages of a tile and more, whose (page, head) count fits a coordinate
    a.tma = d.cache.num_pages > 0 && a.shift >= 4 && d.cache.num_pages * d.Hkv <= INT32_MAX &&
            ((reinterpret_cast<uintptr_t>(a.kscale) | reinterpret_cast<uintptr_t>(a.vscale)) & 15) == 0;
    if (a.tma) {
        const EncodeTiledFn enc = encode_tiled_fn();
        if (enc == nullptr) return cudaErrorNotSupported;
        const CUtensorMapDataType type = KV != kKvX16 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                         : F16        ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        const cuuint64_t row = static_cast<cuuint64_t>(d.D) * S::kElem;
        const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d.D), static_cast<cuuint64_t>(1) << a.shift,
                                    static_cast<cuuint64_t>(d.cache.num_pages * d.Hkv)};
        const cuuint64_t strides[2] = {row, row << a.shift};
        const cuuint32_t box[3] = {S::kWidth / S::kElem, kTile, 1};
        const cuuint32_t estr[3] = {1, 1, 1};
        for (int i = 0; i < 2; ++i)
            if (enc(i ? &maps.v : &maps.k, type, 3, const_cast<void*>(i ? d.cache.v : d.cache.k), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, S::kWidth == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return cudaErrorInvalidValue;
    }
    static OncePerDevice once;
    const cudaError_t limit = allow_smem(once, decode_kernel<DP, KV, F16, COLS>, S::kSmem);
    if (limit != cudaSuccess) return limit;
    return launch_after(decode_kernel<DP, KV, F16, COLS>, dim3(static_cast<unsigned>(grid)), S::kThreads, S::kSmem, stream,
                        maps, a);
}

template <int DP, int KV, bool F16>
cudaError_t launch_cols(Args& a, const DecodeArgs& d, int sm_count, cudaStream_t stream) {
    return group_rows(a.G) == 16 ? launch<DP, KV, F16, 2>(a, d, sm_count, stream) : launch<DP, KV, F16, 1>(a, d, sm_count, stream);
}

template <int DP, bool F16>
cudaError_t launch_kind(int kv, Args& a, const DecodeArgs& d, int sm_count, cudaStream_t stream) {
    if (kv == kKvX16) return launch_cols<DP, kKvX16, F16>(a, d, sm_count, stream);
    if (kv == kKvE4m3) return launch_cols<DP, kKvE4m3, F16>(a, d, sm_count, stream);
    return launch_cols<DP, kKvI8, F16>(a, d, sm_count, stream);
}

constexpr int64_t kMostCtas = 2;   // per SM, any form: the workspace does not depend on the form

static_assert(kMostCtas <= kCountersPerSm, "an arrival counter per CTA");

}  // namespace

size_t decode_ws_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len, int sm_count) {
    const int64_t G = Hq / Hkv;
    const int grid = grid_size(B, Hkv * ceil_div(G, kRows), max_len, kMostCtas * (sm_count < 1 ? 1 : sm_count));
    return workspace_data(sm_count) + static_cast<size_t>(2 * grid) * slot_floats(D > 64 ? 128 : 64, group_rows(G)) * sizeof(float);
}

cudaError_t launch_decode(bool x_f16, const DecodeArgs& d, void* ws, int sm_count, cudaStream_t stream) {
    Args a = {};
    a.lens = d.lens;
    a.table = d.table;
    a.k = static_cast<const uint8_t*>(d.cache.k);
    a.v = static_cast<const uint8_t*>(d.cache.v);
    a.kscale = d.cache.kscale;
    a.vscale = d.cache.vscale;
    a.q = d.q;
    a.o = d.o;
    a.lse = d.lse;
    a.ldq = d.ldq;
    a.ldo = d.ldo;
    a.max_pages = d.max_pages;
    a.num_pages = d.cache.num_pages;
    a.shift = d.cache.page_shift;
    a.capacity = d.max_pages << a.shift;
    a.B = d.B;
    a.D = d.D;
    a.G = d.Hq / d.Hkv;
    a.Hkv = d.Hkv;
    a.passes = static_cast<int>(ceil_div(a.G, kRows));
    a.Hv = a.Hkv * a.passes;
    a.scale2 = d.scale * kLog2e;
    uint8_t* w = static_cast<uint8_t*>(ws);
    a.err = reinterpret_cast<int*>(w);
    a.arrived = reinterpret_cast<int32_t*>(w + kWorkspaceErrBytes);
    a.slots = reinterpret_cast<float*>(w + workspace_data(sm_count));
    if (d.D > 64) return x_f16 ? launch_kind<128, true>(d.cache.kv, a, d, sm_count, stream) : launch_kind<128, false>(d.cache.kv, a, d, sm_count, stream);
    return x_f16 ? launch_kind<64, true>(d.cache.kv, a, d, sm_count, stream) : launch_kind<64, false>(d.cache.kv, a, d, sm_count, stream);
}

}  // namespace tern
