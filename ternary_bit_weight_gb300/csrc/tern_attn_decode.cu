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
// V use the codes, exact in fp16, and weights 2^(s + log2 f - mo) under a
// reference mo of their own, so that factors of any size keep the weights
// within fp16; keys' factors multiply the scores.  Queries are brought to fp16
// by a power of two per row, which the scores' factor undoes.
//
// What bounds it: the bytes of the cache, read once (the G query heads of a
// key/value head are rows of the same products).
//
// Work.  A unit is a tile of 16 keys of one (sequence, key/value head); all
// units in that order are cut into equal contiguous ranges, one per CTA, so
// unequal lengths load the SMs equally.  Within a CTA a segment (the part of
// one item in its range) is dealt to the 8 warps tile by tile; at its end the
// warps' (m, l, o) meet in shared memory.  An item inside one CTA is then
// finished; otherwise the CTAs leave partial results in the workspace and the
// last to arrive adds them in CTA order (the result does not depend on
// timing).
//
// A warp's tile goes global -> shared by cp.async in a ring of its own, each
// lane writing and reading back its own 16-byte runs: no barrier and no bank
// conflict, and the ring holds what a memory latency needs beside the
// registers.  The products are mma.sync m16n8k16: heads are the 16 rows, keys
// the columns, and the score fragment of a thread is its weight fragment for
// the product with V.  The order of dimensions inside a product is free, so
// each thread multiplies the dimensions it has loaded: keys need no
// transposition, values only a byte or half-word interleave of two rows.
// (tcgen05 would take 128-row tiles of which 1 to 16 rows exist here.)

#include <math_constants.h>

#include "tern_attn.cuh"
#include "tern_common.cuh"
#include "tern_internal.h"
#include "tern_sm100.cuh"

namespace tern {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;              // keys per unit
constexpr int kRows = 16;              // query heads per pass over the keys
constexpr float kLazy = 8.0f;          // how far a score may pass the reference
constexpr float kNone = -1.0e38f;      // reference before any key
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;
constexpr int kSmemMax = 232448;

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
    int32_t* arrived;      // [grid], zero between calls
    float* slots;          // [2 * grid] partial results
    int64_t ldq, ldo, max_pages, num_pages;
    int64_t capacity;      // max_pages * page_size
    int B, D, G;           // G query heads share a key/value head
    int Hkv, passes, Hv;   // Hv = Hkv * passes: (key/value head, 16 of its query heads)
    int shift;
    float scale2;          // scale * log2(e)
};

template <int DP, int KV>
struct Shape {
    static constexpr int kElem = KV == kKvX16 ? 2 : 1;
    static constexpr int kRowBytes = DP * kElem;
    static constexpr int kKPieces = kRowBytes / 64;                   // 16-byte runs per lane and key row
    static constexpr int kVRun = kRowBytes / 8 < 16 ? kRowBytes / 8 : 16;
    static constexpr int kVPieces = kRowBytes / 8 / kVRun;            // runs per lane and value row
    static constexpr int kKBytes = kTile * kRowBytes;
    static constexpr int kScaleBytes = KV == kKvX16 ? 0 : 2 * kTile * 4;
    static constexpr int kStage = 2 * kKBytes + kScaleBytes + 16;     // + mask of the keys that exist
    static constexpr int kSteps = DP / 16;                            // K-steps of a score
    static constexpr int kCols = DP / 8;                              // column tiles of the output
    static constexpr int kMergeLd = DP + 4;
    static constexpr int kMerge = kWarps * 8 * kMergeLd * 4;
    static constexpr int kStat = kWarps * kRows * 3 * 4;
    static constexpr int kFit = (kSmemMax - kMerge - kStat - 16) / (kWarps * kStage);
    static constexpr int kStages = kFit < 6 ? kFit : 6;
    static constexpr int kSmem = kWarps * kStages * kStage + kMerge + kStat + 16;
    static_assert(kStages >= 3, "ring depth");
    // dimension of output column n (0..7) in column tile j
    static __device__ __forceinline__ int dim(int n, int j) {
        constexpr int run = KV == kKvX16 ? 8 : DP / 8;
        return (j / run) * 64 + n * run + j % run;
    }
};

__host__ __device__ constexpr int slot_floats(int DP, int rows) { return rows * DP + 3 * kRows; }

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool there) {
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

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

// One segment: the tiles [t, end) of item (b, hv) that lie in the CTA's range.
struct Segment {
    int b, hv;
    int len, tiles;      // keys and tiles of sequence b
    int begin, end;
    int64_t left;        // units of the range after this segment
};

__device__ __forceinline__ int length_of(const Args& a, int b) {
    return static_cast<int>(min(static_cast<int64_t>(max(a.lens[b], 0)), a.capacity));
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

__device__ __forceinline__ void next_segment(const Args& a, Segment& s) {
    if (++s.hv == a.Hv) {
        s.hv = 0;
        do {
            s.len = length_of(a, ++s.b);   // units remain, so a sequence that has some follows
        } while (s.len == 0);
        s.tiles = tiles_of(s.len);
    }
    s.begin = 0;
    s.end = static_cast<int>(min(static_cast<int64_t>(s.tiles), s.left));
    s.left -= s.end;
}

// Total units, and (by one warp) the segment at the front of the CTA's range.
__device__ __forceinline__ int64_t total_units(const Args& a, int lane) {
    int64_t n = 0;
    for (int b = lane; b < a.B; b += 32) n += tiles_of(length_of(a, b));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) n += __shfl_xor_sync(0xffffffffu, n, d);
    return n * a.Hv;
}
__device__ __forceinline__ Segment first_segment(const Args& a, int64_t u0, int64_t u1, int lane) {
    Segment s;
    int64_t base = 0;
    for (int b0 = 0;; b0 += 32) {
        const int len = b0 + lane < a.B ? length_of(a, b0 + lane) : 0;
        const int64_t units = static_cast<int64_t>(tiles_of(len)) * a.Hv;
        int64_t incl = units;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += up;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, base + incl > u0);
        if (past != 0) {   // u0 is below the total, so some lane finds it
            const int src = __ffs(past) - 1;
            s.b = b0 + src;
            s.len = __shfl_sync(0xffffffffu, len, src);
            const int64_t in = u0 - base - __shfl_sync(0xffffffffu, incl - units, src);
            s.tiles = tiles_of(s.len);
            s.hv = static_cast<int>(in / s.tiles);
            s.begin = static_cast<int>(in - static_cast<int64_t>(s.hv) * s.tiles);
            s.end = static_cast<int>(min(static_cast<int64_t>(s.tiles), s.begin + (u1 - u0)));
            s.left = u1 - u0 - (s.end - s.begin);
            return s;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
}

// A tile whose page id has been asked for.
struct Request {
    int page;        // lane's key (shift < 4: key of lane mod 16; else the tile's one page)
    int len, hk;
    int tile;        // -1: none
};

template <int DP, int KV, bool F16, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const Args a) {
    using S = Shape<DP, KV>;
    constexpr bool kCoded = KV != kKvX16;
    constexpr bool kMma16 = kCoded || F16;       // products in fp16 (else bf16)
    constexpr int kR = WIDE ? 2 : 1;             // rows per thread: head g, and g + 8
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * S::kStages * S::kStage;
    uint8_t* ring_ptr = smem + warp * S::kStages * S::kStage;
    float* merge = reinterpret_cast<float*>(smem + kWarps * S::kStages * S::kStage);
    float* stat = merge + S::kMerge / 4;         // [warp][row][m, mo, l]
    volatile int* last_flag = reinterpret_cast<volatile int*>(stat + S::kStat / 4);

    grid_launch_dependents();
    grid_dependency_wait();

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

    // a CTA's range holds a tile for every warp, or there are fewer CTAs
    const int64_t U = total_units(a, lane);
    const int64_t V = max(static_cast<int64_t>(1), min(static_cast<int64_t>(gridDim.x), (U + kWarps - 1) / kWarps));
    if (blockIdx.x >= V || U == 0) return;
    const int64_t u0 = U * blockIdx.x / V, u1 = U * (blockIdx.x + 1) / V;
    Segment seg = first_segment(a, u0, u1, lane);

    // ---------------------------------------------------- loads of a warp
    Segment ls = seg;                 // segment of the next request
    int lt = ls.begin + warp;         // and its tile
    bool more = true;
    auto request = [&]() {
        Request r;
        while (more && lt >= ls.end) {
            if (ls.left == 0) {
                more = false;
            } else {
                next_segment(a, ls);
                lt = warp;
            }
        }
        r.tile = -1;
        if (!more) return r;
        r.tile = lt;
        r.len = ls.len;
        r.hk = a.passes == 1 ? ls.hv : ls.hv / a.passes;
        const int key = a.shift >= 4 ? lt * kTile : min(lt * kTile + (lane & 15), ls.len - 1);
        r.page = a.table[static_cast<int64_t>(ls.b) * a.max_pages + (key >> a.shift)];
        lt += kWarps;
        return r;
    };
    const int bytes = a.D * S::kElem;
    auto issue = [&](const Request& r, int stage) {
        if (r.tile >= 0) {
            const uint32_t st = ring + stage * S::kStage;
            const int key0 = r.tile * kTile;
            // cell of the lane's key (lane mod 16), negative where there is none
            const int key = key0 + (lane & 15);
            int64_t cell = -1;
            if (key < r.len && r.page >= 0 && r.page < a.num_pages)
                cell = ((static_cast<int64_t>(r.page) * a.Hkv + r.hk) << a.shift) + (key & ((1 << a.shift) - 1));
            const uint32_t mask = __ballot_sync(0xffffffffu, cell >= 0) & 0xFFFFu;
#pragma unroll
            for (int r8 = 0; r8 < 2; ++r8) {
                const int64_t c = __shfl_sync(0xffffffffu, cell, g + 8 * r8);
#pragma unroll
                for (int i = 0; i < S::kKPieces; ++i) {
                    const int off = (i * 4 + t) * 16;
                    const bool there = c >= 0 && off < bytes;
                    copy_async<16>(st + ((i * 2 + r8) * 32 + lane) * 16, there ? a.k + c * bytes + off : a.k, there);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t c = __shfl_sync(0xffffffffu, cell, 2 * t + (j & 1) + 8 * (j >> 1));
#pragma unroll
                for (int i = 0; i < S::kVPieces; ++i) {
                    const int off = i * 128 + g * S::kVRun;
                    const bool there = c >= 0 && off < bytes;
                    copy_async<S::kVRun>(st + S::kKBytes + ((j * S::kVPieces + i) * 32 + lane) * S::kVRun,
                                         there ? a.v + c * bytes + off : a.v, there);
                }
            }
            if constexpr (kCoded) {
                const float* src = lane < 16 ? a.kscale : a.vscale;
                copy_async<4>(st + 2 * S::kKBytes + lane * 4, cell >= 0 ? src + cell : src, cell >= 0);
            }
            if (lane == 0)
                *reinterpret_cast<uint32_t*>(ring_ptr + stage * S::kStage + 2 * S::kKBytes + S::kScaleBytes) = mask;
        }
        copy_commit();
    };

    Request next = request();
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) {
        const Request now = next;
        next = request();
        issue(now, i);
    }
    int stage = 0, fill = S::kStages - 1;

    // ------------------------------------------------------------ segments
    for (bool first = true;; first = false) {
        if (!first) next_segment(a, seg);
        const int hk = a.passes == 1 ? seg.hv : seg.hv / a.passes;
        const int head0 = (seg.hv - hk * a.passes) * kRows;               // first of the group's heads
        const int heads = min(kRows, a.G - head0);
        const int64_t q_head = static_cast<int64_t>(hk) * a.G + head0;
        float m[kR], mo[kR], l[kR], fac[kR];
        float o[S::kCols][4];
        uint32_t qa[S::kSteps][4];
        const bool mine = seg.begin + warp < seg.end;
        if (mine) {
            // queries: the four dimensions of each K-step that the thread's key runs hold
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                uint2 u[S::kSteps];
                const bool live = r < kR && g + 8 * r < heads;
                const uint16_t* src = a.q + seg.b * a.ldq + (q_head + g + 8 * r) * a.D;
#pragma unroll
                for (int w = 0; w < S::kSteps; ++w) {
                    const int d = kCoded ? ((w / 4) * 4 + t) * 16 + (w % 4) * 4 : ((w / 2) * 4 + t) * 8 + (w % 2) * 4;
                    u[w] = live && d < a.D ? *reinterpret_cast<const uint2*>(src + d) : make_uint2(0, 0);
                }
                float f = a.scale2;
                if constexpr (kCoded) {
                    // times 2^e, so that the row's largest magnitude lies in [2^14, 2^15)
                    float top = 0.0f;
#pragma unroll
                    for (int w = 0; w < S::kSteps; ++w) {
                        const float2 x = unpack_x2<F16>(u[w].x), y = unpack_x2<F16>(u[w].y);
                        top = fmaxf(top, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y))));
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const int e = top > 0.0f && top <= 3.4e38f ? 14 - ilogbf(top) : 0;
                    // in two steps: 2^e may pass fp32's range
                    const float up0 = exp2f(static_cast<float>(e / 2)), up1 = exp2f(static_cast<float>(e - e / 2));
                    f = f * exp2f(static_cast<float>(-(e / 2))) * exp2f(static_cast<float>(-(e - e / 2)));
#pragma unroll
                    for (int w = 0; w < S::kSteps; ++w) {
                        const float2 x = unpack_x2<F16>(u[w].x), y = unpack_x2<F16>(u[w].y);
                        u[w].x = pack_x2<true>(x.x * up0 * up1, x.y * up0 * up1);
                        u[w].y = pack_x2<true>(y.x * up0 * up1, y.y * up0 * up1);
                    }
                }
#pragma unroll
                for (int w = 0; w < S::kSteps; ++w) {
                    qa[w][r] = u[w].x;
                    qa[w][2 + r] = u[w].y;
                }
                if (r < kR) {
                    fac[r] = f;
                    m[r] = mo[r] = kNone;
                    l[r] = 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < S::kCols; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[j][i] = 0.0f;
        }

        for (int tile = seg.begin + warp; tile < seg.end; tile += kWarps) {
            __syncwarp();   // every lane has read the stage that is filled now
            const Request now = next;
            next = request();
            issue(now, fill);
            if (++fill == S::kStages) fill = 0;
            copy_wait<S::kStages - 1>();
            __syncwarp();   // the lanes' copies and the mask are visible to one another
            const uint8_t* st = ring_ptr + stage * S::kStage;
            if (++stage == S::kStages) stage = 0;
            const uint32_t mask = *reinterpret_cast<const uint32_t*>(st + 2 * S::kKBytes + S::kScaleBytes);

            // ------------------------------------------------ scores
            float s[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int i = 0; i < S::kKPieces; ++i) {
                const uint4 u0 = *reinterpret_cast<const uint4*>(st + ((i * 2) * 32 + lane) * 16);
                const uint4 u1 = *reinterpret_cast<const uint4*>(st + ((i * 2 + 1) * 32 + lane) * 16);
                const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
                if constexpr (kCoded) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t lo, hi;
                        decode4<KV>(w0[w], lo, hi);
                        mma<kMma16>(s[0], qa[i * 4 + w], lo, hi);
                        decode4<KV>(w1[w], lo, hi);
                        mma<kMma16>(s[1], qa[i * 4 + w], lo, hi);
                    }
                } else {
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        mma<kMma16>(s[0], qa[i * 2 + w], w0[2 * w], w0[2 * w + 1]);
                        mma<kMma16>(s[1], qa[i * 2 + w], w1[2 * w], w1[2 * w + 1]);
                    }
                }
            }
            // the thread's keys: 2t, 2t+1, 8+2t, 9+2t
            float kf[4] = {1, 1, 1, 1}, vl[4] = {0, 0, 0, 0};
            if constexpr (kCoded) {
                const float* ks = reinterpret_cast<const float*>(st + 2 * S::kKBytes);
                const float2 k0 = *reinterpret_cast<const float2*>(ks + 2 * t), k1 = *reinterpret_cast<const float2*>(ks + 8 + 2 * t);
                const float2 v0 = *reinterpret_cast<const float2*>(ks + 16 + 2 * t), v1 = *reinterpret_cast<const float2*>(ks + 24 + 2 * t);
                kf[0] = k0.x, kf[1] = k0.y, kf[2] = k1.x, kf[3] = k1.y;
                vl[0] = log2_approx(v0.x), vl[1] = log2_approx(v0.y), vl[2] = log2_approx(v1.x), vl[3] = log2_approx(v1.y);
            }
            float x[kR][4];
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[r][i] = s[i >> 1][2 * r + (i & 1)] * fac[r];
                    if (kCoded) x[r][i] *= kf[i];
                }
            if (mask != 0xFFFFu) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!((mask >> (2 * t + (i & 1) + 8 * (i >> 1))) & 1u)) {
#pragma unroll
                        for (int r = 0; r < kR; ++r) x[r][i] = -CUDART_INF_F;
                    }
            }
            // ------------------------------------------- references
            float top[kR], topo[kR];
            bool past = false;
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                top[r] = fmaxf(fmaxf(x[r][0], x[r][1]), fmaxf(x[r][2], x[r][3]));
                past = past || top[r] > m[r] + kLazy;
                if (kCoded) {
                    topo[r] = fmaxf(fmaxf(x[r][0] + vl[0], x[r][1] + vl[1]), fmaxf(x[r][2] + vl[2], x[r][3] + vl[3]));
                    past = past || topo[r] > mo[r] + kLazy;
                }
            }
            if (__any_sync(0xffffffffu, past)) {
#pragma unroll
                for (int r = 0; r < kR; ++r) {
                    float up = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                    up = fmaxf(m[r], fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 2)));
                    l[r] *= exp2_approx(m[r] - up);
                    float f = exp2_approx(m[r] - up);
                    m[r] = up;
                    if (kCoded) {
                        up = fmaxf(topo[r], __shfl_xor_sync(0xffffffffu, topo[r], 1));
                        up = fmaxf(mo[r], fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 2)));
                        f = exp2_approx(mo[r] - up);
                        mo[r] = up;
                    }
#pragma unroll
                    for (int j = 0; j < S::kCols; ++j) {
                        o[j][2 * r] *= f;
                        o[j][2 * r + 1] *= f;
                    }
                }
            }
            // ---------------------------------------------- weights
            uint32_t p[4] = {0, 0, 0, 0};
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                float w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] = exp2_approx(x[r][i] - m[r]);
                    l[r] += w[i];
                    if (kCoded) w[i] = exp2_approx(x[r][i] + vl[i] - mo[r]);
                }
                p[r] = pack_x2<kMma16>(w[0], w[1]);
                p[2 + r] = pack_x2<kMma16>(w[2], w[3]);
            }
            // ----------------------------------------------- values
            const uint8_t* sv = st + S::kKBytes;
            if constexpr (kCoded) {
                constexpr int kWords = S::kVRun / 4;
                uint32_t v[4][kWords];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint8_t* src = sv + (j * 32 + lane) * S::kVRun;
                    if constexpr (kWords == 4) {
                        const uint4 u = *reinterpret_cast<const uint4*>(src);
                        v[j][0] = u.x, v[j][1] = u.y, v[j][2] = u.z, v[j][3] = u.w;
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2*>(src);
                        v[j][0] = u.x, v[j][1] = u.y;
                    }
                }
#pragma unroll
                for (int q = 0; q < kWords; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t b0[2], b1[2];
                        decode4<KV>(__byte_perm(v[0][q], v[1][q], h ? 0x7362 : 0x5140), b0[0], b0[1]);
                        decode4<KV>(__byte_perm(v[2][q], v[3][q], h ? 0x7362 : 0x5140), b1[0], b1[1]);
                        mma<kMma16>(o[4 * q + 2 * h], p, b0[0], b1[0]);
                        mma<kMma16>(o[4 * q + 2 * h + 1], p, b0[1], b1[1]);
                    }
            } else {
#pragma unroll
                for (int i = 0; i < S::kVPieces; ++i) {
                    uint32_t v[4][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 u = *reinterpret_cast<const uint4*>(sv + ((j * S::kVPieces + i) * 32 + lane) * 16);
                        v[j][0] = u.x, v[j][1] = u.y, v[j][2] = u.z, v[j][3] = u.w;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        mma<kMma16>(o[8 * i + 2 * q], p, __byte_perm(v[0][q], v[1][q], 0x5410),
                                    __byte_perm(v[2][q], v[3][q], 0x5410));
                        mma<kMma16>(o[8 * i + 2 * q + 1], p, __byte_perm(v[0][q], v[1][q], 0x7632),
                                    __byte_perm(v[2][q], v[3][q], 0x7632));
                    }
                }
            }
        }

        // ------------------------------------------- the segment's sum
        const int active = min(kWarps, seg.end - seg.begin);   // warps that had a tile
        const bool whole = seg.begin == 0 && seg.end == seg.tiles;
        if (mine) {
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                if (t == 0) {
                    float* dst = stat + (warp * kRows + g + 8 * r) * 3;
                    dst[0] = m[r];
                    dst[1] = kCoded ? mo[r] : m[r];
                    dst[2] = l[r];
                }
            }
        }
        // partial results: the CTA that begins an item uses its odd slot, the
        // others their even one
        constexpr int kSlotRows = 8 * kR;
        float* slot = a.slots + (2 * static_cast<int64_t>(blockIdx.x) + (seg.begin == 0 ? 1 : 0)) * slot_floats(DP, kSlotRows);
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            if (mine) {
                float* dst = merge + (warp * 8 + g) * S::kMergeLd;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < S::kCols; j += 4)
                        *reinterpret_cast<float4*>(dst + S::dim(2 * t + n, j)) =
                            make_float4(o[j][2 * r + n], o[j + 1][2 * r + n], o[j + 2][2 * r + n], o[j + 3][2 * r + n]);
            }
            __syncthreads();
            const int row = threadIdx.x / (DP / 4), d = (threadIdx.x % (DP / 4)) * 4, head = row + 8 * r;
            if (row < 8 && head < heads) {
                float M = kNone, MO = kNone, L = 0.0f;
                for (int w = 0; w < active; ++w) {
                    M = fmaxf(M, stat[(w * kRows + head) * 3]);
                    MO = fmaxf(MO, stat[(w * kRows + head) * 3 + 1]);
                }
                float4 sum = make_float4(0, 0, 0, 0);
                for (int w = 0; w < active; ++w) {
                    const float* sp = stat + (w * kRows + head) * 3;
                    L += sp[2] * exp2_approx(sp[0] - M);
                    const float f = exp2_approx(sp[1] - MO);
                    const float4 u = *reinterpret_cast<const float4*>(merge + (w * 8 + row) * S::kMergeLd + d);
                    sum.x += u.x * f, sum.y += u.y * f, sum.z += u.z * f, sum.w += u.w * f;
                }
                if (whole) {
                    const float f = L == 0.0f ? 0.0f : exp2_approx(MO - M) / L;
                    if (d < a.D)
                        *reinterpret_cast<uint2*>(a.o + seg.b * a.ldo + (q_head + head) * a.D + d) =
                            make_uint2(pack_x2<F16>(sum.x * f, sum.y * f), pack_x2<F16>(sum.z * f, sum.w * f));
                    if (d == 0 && a.lse != nullptr)
                        a.lse[static_cast<int64_t>(seg.b) * a.Hkv * a.G + q_head + head] =
                            L == 0.0f ? -CUDART_INF_F : M * kLn2 + logf(L);
                } else {
                    *reinterpret_cast<float4*>(slot + head * DP + d) = sum;
                    if (d == 0) {
                        float* dst = slot + kSlotRows * DP + head * 3;
                        dst[0] = M;
                        dst[1] = MO;
                        dst[2] = L;
                    }
                }
            }
            __syncthreads();
        }
        if (!whole) {
            // CTAs c0 .. c1 hold the item; the last to arrive adds their parts
            const int64_t before = u1 - seg.left - (seg.end - seg.begin) - seg.begin;   // first unit of the item
            const int c0 = static_cast<int>(((before + 1) * V - 1) / U);
            const int c1 = static_cast<int>(((before + seg.tiles) * V - 1) / U);
            if (threadIdx.x == 0) {
                __threadfence();
                const int32_t old = atomicAdd(a.arrived + c0, 1);
                *last_flag = old == c1 - c0;
                __threadfence();
            }
            __syncthreads();
            if (*last_flag) {
                for (int e = threadIdx.x; e < heads * (DP / 4); e += kThreads) {
                    const int head = e / (DP / 4), d = (e % (DP / 4)) * 4;
                    auto part = [&](int c) {
                        return a.slots + (2 * static_cast<int64_t>(c) + (c == c0 ? 1 : 0)) * slot_floats(DP, kSlotRows);
                    };
                    float M = kNone, MO = kNone, L = 0.0f;
                    for (int c = c0; c <= c1; ++c) {
                        const float* sp = part(c) + kSlotRows * DP + head * 3;
                        M = fmaxf(M, __ldcg(sp));
                        MO = fmaxf(MO, __ldcg(sp + 1));
                    }
                    float4 sum = make_float4(0, 0, 0, 0);
#pragma unroll 4
                    for (int c = c0; c <= c1; ++c) {
                        const float* sp = part(c) + kSlotRows * DP + head * 3;
                        const float4 u = __ldcg(reinterpret_cast<const float4*>(part(c) + head * DP + d));
                        L += __ldcg(sp + 2) * exp2_approx(__ldcg(sp) - M);
                        const float f = exp2_approx(__ldcg(sp + 1) - MO);
                        sum.x += u.x * f, sum.y += u.y * f, sum.z += u.z * f, sum.w += u.w * f;
                    }
                    const float f = L == 0.0f ? 0.0f : exp2_approx(MO - M) / L;
                    if (d < a.D)
                        *reinterpret_cast<uint2*>(a.o + seg.b * a.ldo + (q_head + head) * a.D + d) =
                            make_uint2(pack_x2<F16>(sum.x * f, sum.y * f), pack_x2<F16>(sum.z * f, sum.w * f));
                    if (d == 0 && a.lse != nullptr)
                        a.lse[static_cast<int64_t>(seg.b) * a.Hkv * a.G + q_head + head] =
                            L == 0.0f ? -CUDART_INF_F : M * kLn2 + logf(L);
                }
                if (threadIdx.x == 0) a.arrived[c0] = 0;
            }
            __syncthreads();   // last_flag is free again
        }
        if (seg.left == 0) break;
    }
    copy_wait<0>();
}

int group_rows(int64_t G) { return G > 8 ? 16 : 8; }

int grid_size(int64_t B, int64_t Hv, int64_t max_len, int sm_count) {
    const int64_t units = B * Hv * ceil_div(max_len, kTile);
    const int64_t ctas = ceil_div(units, kWarps);
    return static_cast<int>(ctas < 1 ? 1 : ctas < sm_count ? ctas : sm_count);
}

template <int DP, int KV, bool F16, bool WIDE>
cudaError_t launch(const Args& a, int grid, cudaStream_t stream) {
    using S = Shape<DP, KV>;
    static const cudaError_t limit = cudaFuncSetAttribute(decode_kernel<DP, KV, F16, WIDE>,
                                                          cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (limit != cudaSuccess) return limit;
    return launch_after(decode_kernel<DP, KV, F16, WIDE>, dim3(static_cast<unsigned>(grid)), kThreads, S::kSmem, stream, a);
}

template <int DP, int KV, bool F16>
cudaError_t launch_rows(const Args& a, int grid, cudaStream_t stream) {
    return group_rows(a.G) == 16 ? launch<DP, KV, F16, true>(a, grid, stream)
                                 : launch<DP, KV, F16, false>(a, grid, stream);
}

template <int DP, bool F16>
cudaError_t launch_kind(int kv, const Args& a, int grid, cudaStream_t stream) {
    if (kv == kKvX16) return launch_rows<DP, kKvX16, F16>(a, grid, stream);
    if (kv == kKvE4m3) return launch_rows<DP, kKvE4m3, F16>(a, grid, stream);
    return launch_rows<DP, kKvI8, F16>(a, grid, stream);
}

int64_t arrived_bytes(int grid) { return round_up(static_cast<int64_t>(grid) * 4, 256); }

}  // namespace

size_t decode_ws_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len, int sm_count) {
    const int64_t G = Hq / Hkv;
    const int grid = grid_size(B, Hkv * ceil_div(G, kRows), max_len, sm_count < 1 ? 1 : sm_count);
    return kWorkspaceErrBytes + static_cast<size_t>(arrived_bytes(grid)) +
           static_cast<size_t>(2 * grid) * slot_floats(D > 64 ? 128 : 64, group_rows(G)) * sizeof(float);
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
    const int grid = grid_size(d.B, a.Hv, a.capacity, sm_count);
    uint8_t* w = static_cast<uint8_t*>(ws) + kWorkspaceErrBytes;
    a.arrived = reinterpret_cast<int32_t*>(w);
    a.slots = reinterpret_cast<float*>(w + arrived_bytes(grid));
    if (d.D > 64) return x_f16 ? launch_kind<128, true>(d.cache.kv, a, grid, stream) : launch_kind<128, false>(d.cache.kv, a, grid, stream);
    return x_f16 ? launch_kind<64, true>(d.cache.kv, a, grid, stream) : launch_kind<64, false>(d.cache.kv, a, grid, stream);
}

}  // namespace tern
