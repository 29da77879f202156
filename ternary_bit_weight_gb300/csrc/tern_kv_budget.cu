// Keeping a paged key/value cache within a budget of tokens: the choice of the
// tokens to keep by their accumulated weight, and their move to the front.
//
// Mathematics.  Weights become 32-bit keys in the order of the numbers (a NaN, or
// a token of a page outside the cache, below all of them).  The smallest kept key
// is found digit by digit, 8 bits of its distance from the smallest key at a time, by
// counting; of the tokens that have it the first ones are kept.  Counts are whole
// numbers, so the result does not depend on the order of the atomics.  What bounds the
// choice: a chain of loads, counts and votes per row.  (512 of 577 tokens of 8 heads 3.1 us
// in a CUDA graph, 4096 of 8192 of 512 rows 21 us; digits of the keys themselves, whose counts
// meet in few places, and 128 registers a thread 52 us; a load for each token 33 us.)  The
// form goes by the table's room, not by the lengths: those 512 rows take 59 us with a table for
// 32768 tokens and 46 with one for 65536, rows of 600 tokens 5.4, 48 and 24.
//
// Moves.  A list of kept tokens ascends, so entry j is at or behind place j: tokens
// taken in order, a block of places at a time, never write what a later block
// still reads.  A CTA has one (sequence, head) and a slice of the row's bytes, reads
// a block of tokens, meets, and writes it; slices do not touch one another's bytes.
// What bounds the moves: DRAM, and that a block's list, page table and data follow from
// one another, which many CTAs on an SM hide (32 sequences of 8192 to 4096 tokens in bf16
// 205 us, 5.3 TB/s read and written; with the next block's loads ahead in registers fewer CTAs
// fit and it took 257 to 336, with whole rows instead of 64 bytes 249).

#include <float.h>
#include <math_constants.h>

#include "tern_attn.cuh"
#include "tern_common.cuh"
#include "tern_internal.h"

namespace tern {
namespace {

// -------------------------------------------------------------------- choice

struct KeepArgs {
    const float* weight;
    const int32_t* table;
    const int32_t* lens;
    int32_t* keep;
    int32_t* new_lens;
    int64_t max_pages, num_pages, capacity, budget;
    int first, recent;
    int Hkv, shift;
};

// Keys in the order of the numbers, -0 being 0, between 1 (NaN, or a hidden token)
// and that of infinity.
constexpr uint32_t kAbsent = 0, kLowest = 1, kMust = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) return kLowest;
    const uint32_t u = __float_as_uint(w == 0.0f ? 0.0f : w);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Whether the weights of four tokens are one access.
__host__ __device__ __forceinline__ bool by_four(const KeepArgs& a) {
    return a.shift >= 2 && (reinterpret_cast<uintptr_t>(a.weight) & 15) == 0;
}

// Four tokens beside one another are one lane's, one page look-up and one load (with a
// load for each of them half of the time of 512 rows went there); 128 of them are a
// step of the warp, which lists its tokens in order with votes.  EACH keys of a thread stay
// in registers; EACH == 0: more tokens than that, or pages and planes that do not take four
// weights in one access; each pass loads them again.
// Every warp works out a digit by itself from the counts, so a digit costs one barrier.
template <int EACH, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 4 : 1) keep_kernel(const KeepArgs a) {
    __shared__ __align__(16) uint32_t bins[4][256];
    __shared__ uint32_t ends[2][32];       // per warp: smallest and largest key
    __shared__ int above[32], equal[32];   // per warp
    grid_launch_dependents();
    grid_dependency_wait();
    const int b = blockIdx.x / static_cast<uint32_t>(a.Hkv), hk = blockIdx.x - b * a.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int len = static_cast<int>(min(static_cast<int64_t>(max(a.lens[b], 0)), a.capacity));
    int32_t* out = a.keep + static_cast<int64_t>(blockIdx.x) * a.budget;
    const int kept = static_cast<int>(min(static_cast<int64_t>(len), a.budget));
    if (hk == 0 && threadIdx.x == 0) a.new_lens[b] = kept;
    for (int64_t j = kept + threadIdx.x; j < a.budget; j += blockDim.x) out[j] = -1;
    if (len <= a.budget) {
        for (int j = threadIdx.x; j < len; j += blockDim.x) out[j] = j;
        return;
    }
    const int page_mask = (1 << a.shift) - 1;
    const int32_t* table = a.table + b * a.max_pages;
    const int lo = a.first, hi = len - a.recent;
    // the warp's run of tokens [j0, j1)
    const int run = ((len + warps - 1) / warps + 127) & ~127;
    const int j0 = min(len, warp * run), j1 = min(len, j0 + run);
    const bool wide = EACH > 0 || by_four(a);
    auto page_of = [&](int j) { return j < j1 ? table[j >> a.shift] : -1; };
    auto weights_of = [&](int page, int j) {   // NaN outside the cache
        return page >= 0 && page < a.num_pages ? a.weight + (((static_cast<int64_t>(page) * a.Hkv + hk) << a.shift) + (j & page_mask)) : nullptr;
    };
    auto load4 = [&](int j, int page, float4& w) {   // page: that of j
        w = make_float4(CUDART_NAN_F, CUDART_NAN_F, CUDART_NAN_F, CUDART_NAN_F);
        const float* src = weights_of(page, j);
        if (wide) {
            if (src != nullptr) w = *reinterpret_cast<const float4*>(src);
        } else {
            const float *s1 = weights_of(page_of(j + 1), j + 1), *s2 = weights_of(page_of(j + 2), j + 2), *s3 = weights_of(page_of(j + 3), j + 3);
            if (src != nullptr) w.x = *src;
            if (s1 != nullptr) w.y = *s1;
            if (s2 != nullptr) w.z = *s2;
            if (s3 != nullptr) w.w = *s3;
        }
    };
    auto key_of = [&](int j, float w) { return j >= j1 ? kAbsent : j < lo || j >= hi ? kMust : order_key(w); };
    uint32_t keys[EACH == 0 ? 1 : EACH];
    if constexpr (EACH > 0) {
        constexpr int kAtOnce = EACH < 16 ? EACH / 4 : 4;
#pragma unroll
        for (int i0 = 0; i0 < EACH / 4; i0 += kAtOnce) {
            int pages[kAtOnce];
            float4 w[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) pages[i] = page_of(j0 + 128 * (i0 + i) + 4 * lane);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) load4(j0 + 128 * (i0 + i) + 4 * lane, pages[i], w[i]);
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int j = j0 + 128 * (i0 + i) + 4 * lane, at = 4 * (i0 + i);
                keys[at] = key_of(j, w[i].x);
                keys[at + 1] = key_of(j + 1, w[i].y);
                keys[at + 2] = key_of(j + 2, w[i].z);
                keys[at + 3] = key_of(j + 3, w[i].w);
            }
        }
    }
    for (int i = threadIdx.x; i < 4 * 256; i += blockDim.x) bins[0][i] = 0;
    // what(j, keys of j .. j + 3) for the thread's tokens, the whole warp together
    auto each4 = [&](auto&& what) {
        if constexpr (EACH > 0) {
#pragma unroll
            for (int i = 0; i < EACH / 4; ++i) {
                const uint32_t k[4] = {keys[4 * i], keys[4 * i + 1], keys[4 * i + 2], keys[4 * i + 3]};
                what(j0 + 128 * i + 4 * lane, k);
            }
        } else {
            for (int at = j0; at < j1; at += 128) {
                const int j = at + 4 * lane;
                float4 w;
                load4(j, page_of(j), w);
                const uint32_t k[4] = {key_of(j, w.x), key_of(j + 1, w.y), key_of(j + 2, w.z), key_of(j + 3, w.w)};
                what(j, k);
            }
        }
    };
    auto each = [&](auto&& what) {
        each4([&](int, const uint32_t (&k)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) what(k[e]);
        });
    };
    // the key of which `take` are left to keep when all above it are kept: digits of the
    // distance from the smallest key, so that the first ones are spread over the counts
    uint32_t take = static_cast<uint32_t>(kept - a.first - a.recent), prefix = kMust - 1;   // take == 0: no key has it
    if (take > 0) {
        // (one less and one more, so that kAbsent and kMust are out of the way)
        uint32_t least = 0xFFFFFFFFu, most = 0;
        each([&](uint32_t k) {
            least = min(least, k - 1);
            most = max(most, k + 1);
        });
        least = __reduce_min_sync(0xffffffffu, least);
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) ends[0][warp] = least, ends[1][warp] = most;
        __syncthreads();   // (and the counts are zero)
        least = __reduce_min_sync(0xffffffffu, lane < warps ? ends[0][lane] : 0xFFFFFFFFu) + 1;
        most = __reduce_max_sync(0xffffffffu, lane < warps ? ends[1][lane] : 0u) - 1;
        prefix = least;
        uint32_t span = most - least;        // keys looked at: prefix to prefix + span
        int at = 32 - __clz(span);           // bits that are not known yet
        for (int turn = 0; at > 0; ++turn) {
            at = max(0, at - 8);
            uint32_t* count = bins[turn];
            each([&](uint32_t k) {
                if (k - prefix <= span) atomicAdd(&count[(k - prefix) >> at], 1u);
            });
            __syncthreads();
            // lane l has digits 255 - 8l - 7 .. 255 - 8l, the largest first
            uint32_t c[8], mine = 0;
            const uint4 c0 = *reinterpret_cast<const uint4*>(count + 248 - 8 * lane), c1 = *reinterpret_cast<const uint4*>(count + 252 - 8 * lane);
            c[7] = c0.x, c[6] = c0.y, c[5] = c0.z, c[4] = c0.w, c[3] = c1.x, c[2] = c1.y, c[1] = c1.z, c[0] = c1.w;
#pragma unroll
            for (int i = 0; i < 8; ++i) mine += c[i];
            uint32_t incl = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t up = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += up;
            }
            // the first lane whose count passes `take` has the digit
            const int src = __ffs(__ballot_sync(0xffffffffu, incl >= take)) - 1;
            uint32_t before = incl - mine, digit = 0, over = 0, held = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (before < take && before + c[i] >= take) {
                    digit = 255 - 8 * lane - i;
                    over = before;
                    held = c[i];
                }
                before += c[i];
            }
            prefix += __shfl_sync(0xffffffffu, digit, src) << at;
            take -= __shfl_sync(0xffffffffu, over, src);
            span = min(most - prefix, (1u << at) - 1);
            if (__shfl_sync(0xffffffffu, held, src) == take) {   // all that have the digits
                --prefix;
                take = 0;
                break;
            }
        }
    }

    int n_over = 0, n_same = 0;
    each([&](uint32_t k) {
        n_over += k > prefix;
        n_same += k == prefix;
    });
    n_over = __reduce_add_sync(0xffffffffu, n_over);
    n_same = __reduce_add_sync(0xffffffffu, n_same);
    if (lane == 0) above[warp] = n_over, equal[warp] = n_same;
    __syncthreads();
    // what the warps before list
    int over_before = lane < warp ? above[lane] : 0, same_before = lane < warp ? equal[lane] : 0;
    over_before = __reduce_add_sync(0xffffffffu, over_before);
    same_before = __reduce_add_sync(0xffffffffu, same_before);
    int place = over_before + min(same_before, static_cast<int>(take));
    const uint32_t below = (1u << lane) - 1;
    each4([&](int j, const uint32_t (&k)[4]) {
        uint32_t ins[4];
        bool in[4];
        if (take > 0) {
            int rank = same_before;   // of the lane's first token among those that have the smallest kept key
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t sames = __ballot_sync(0xffffffffu, k[e] == prefix);
                rank += __popc(sames & below);
                same_before += __popc(sames);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                in[e] = k[e] > prefix || (k[e] == prefix && rank < static_cast<int>(take));
                rank += k[e] == prefix;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) in[e] = k[e] > prefix;
        }
        int at = place;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            ins[e] = __ballot_sync(0xffffffffu, in[e]);
            at += __popc(ins[e] & below);
            place += __popc(ins[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (in[e]) out[at++] = j + e;
    });
}

// --------------------------------------------------------------------- moves

constexpr int kUnroll = 2;         // tokens of a thread in a block of places

struct MoveArgs {
    const int32_t* table;
    const int32_t* to;     // where place j goes (the same table: in place)
    const int32_t* keep;
    uint8_t* k;
    uint8_t* v;
    float* kscale;
    float* vscale;
    float* weight;
    int32_t* err;
    int64_t max_pages, to_pages, num_pages, capacity, budget;
    int Hkv, shift;
    int in_place;
    int bytes;             // of a row of keys or values
    int lanes;             // 16-byte runs of a slice
    int slices;            // of a row
};

// Runs of 16 bytes of the keys (or values) of one head, or its fp32 numbers.
template <int THREADS, typename T>
__device__ __forceinline__ void move(const MoveArgs& a, T* data, int64_t row_bytes, int64_t at, bool live, int width, int b, int hk,
                                     int start, int count) {
    const int per = THREADS / width;           // tokens at a time
    const int me = threadIdx.x / static_cast<uint32_t>(width);
    const int page_mask = (1 << a.shift) - 1;
    const int32_t* list = a.keep + (static_cast<int64_t>(b) * a.Hkv + hk) * a.budget;
    const int32_t* from_table = a.table + b * a.max_pages;
    const int32_t* to_table = a.to + b * a.to_pages;
    auto address = [&](const int32_t* table, int j) -> T* {
        const int page = table[j >> a.shift];
        if (page < 0 || page >= a.num_pages) return nullptr;
        const int64_t cell = ((static_cast<int64_t>(page) * a.Hkv + hk) << a.shift) + (j & page_mask);
        return reinterpret_cast<T*>(reinterpret_cast<uint8_t*>(data) + cell * row_bytes + at);
    };
    for (int j0 = start; j0 < count; j0 += per * kUnroll) {
        T x[kUnroll];
        T* dst[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int j = j0 + i * per + me;
            dst[i] = nullptr;
            if (live && j < count) {
                const T* src = address(from_table, list[j]);
                if (src != nullptr) {
                    dst[i] = address(to_table, j);
                    x[i] = *src;
                }
            }
        }
        __syncthreads();   // the block is read
#pragma unroll
        for (int i = 0; i < kUnroll; ++i)
            if (dst[i] != nullptr) *dst[i] = x[i];
    }
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) move_kernel(const MoveArgs a) {
    __shared__ int moved, ends, bad;
    grid_launch_dependents();
    grid_dependency_wait();
    const int each = 2 * a.slices + 1;             // CTAs of a head
    const uint32_t row = blockIdx.x / static_cast<uint32_t>(each);
    const int part = blockIdx.x - row * each;
    const int b = row / static_cast<uint32_t>(a.Hkv), hk = row - b * a.Hkv;
    const int32_t* list = a.keep + static_cast<int64_t>(row) * a.budget;
    if (threadIdx.x == 0) {
        moved = ends = INT32_MAX;
        bad = 0;
    }
    __syncthreads();
    // the first entry that moves, the list's end, and whether it is one
    const int budget = static_cast<int>(a.budget);
    int my_moved = INT32_MAX, my_end = budget;
    for (int j = threadIdx.x; j < budget; j += THREADS)
        if (list[j] < 0) {
            my_end = j;
            break;
        }
    atomicMin(&ends, my_end);
    __syncthreads();
    const int count = ends;
    bool wrong = false;
    for (int j = threadIdx.x; j < count; j += THREADS) {
        const int at = list[j];
        if (at >= a.capacity || (a.in_place && j > 0 && list[j - 1] >= at)) wrong = true;
        if (at != j && my_moved == INT32_MAX) my_moved = j;
    }
    if (wrong) bad = 1;
    atomicMin(&moved, my_moved);
    __syncthreads();
    if (bad) {
        if (part == 0 && threadIdx.x == 0 && a.err != nullptr) atomicAdd(a.err, 1);
        return;
    }
    const int start = a.in_place ? min(moved, count) : 0;
    if (part < 2 * a.slices) {
        const int slice = part < a.slices ? part : part - a.slices;
        const int run = slice * a.lanes + threadIdx.x % a.lanes;
        uint8_t* data = part < a.slices ? a.k : a.v;
        move<THREADS>(a, reinterpret_cast<uint4*>(data), a.bytes, 16 * run, 16 * run < a.bytes, a.lanes, b, hk, start, count);
    } else {
        if (a.kscale != nullptr) move<THREADS>(a, a.kscale, 4, 0, true, 1, b, hk, start, count);
        if (a.vscale != nullptr) move<THREADS>(a, a.vscale, 4, 0, true, 1, b, hk, start, count);
        if (a.weight != nullptr) move<THREADS>(a, a.weight, 4, 0, true, 1, b, hk, start, count);
    }
}

}  // namespace

cudaError_t launch_keep(const KeepCall& c, cudaStream_t stream) {
    KeepArgs a = {};
    a.weight = c.weight;
    a.table = c.table;
    a.lens = c.lens;
    a.keep = c.keep;
    a.new_lens = c.new_lens;
    a.max_pages = c.max_pages;
    a.num_pages = c.num_pages;
    a.capacity = c.max_pages << c.page_shift;
    a.budget = c.budget;
    a.first = static_cast<int>(c.first);
    a.recent = static_cast<int>(c.recent);
    a.Hkv = c.Hkv;
    a.shift = c.page_shift;
    // registers for every token that there may be; small sequences in few threads
    const dim3 grid(static_cast<unsigned>(c.B * c.Hkv));
    if (!by_four(a)) return launch_after(keep_kernel<0, 1024>, grid, 1024, 0, stream, a);
    if (a.capacity <= 1024) return launch_after(keep_kernel<4, 256>, grid, 256, 0, stream, a);
    if (a.capacity <= 2048) return launch_after(keep_kernel<8, 256>, grid, 256, 0, stream, a);
    if (a.capacity <= 4096) return launch_after(keep_kernel<16, 256>, grid, 256, 0, stream, a);
    if (a.capacity <= 8192) return launch_after(keep_kernel<32, 256>, grid, 256, 0, stream, a);
    if (a.capacity <= 16384) return launch_after(keep_kernel<32, 512>, grid, 512, 0, stream, a);
    if (a.capacity <= 32768) return launch_after(keep_kernel<32, 1024>, grid, 1024, 0, stream, a);
    return launch_after(keep_kernel<0, 1024>, grid, 1024, 0, stream, a);
}

cudaError_t launch_compact(const CompactCall& c, cudaStream_t stream) {
    MoveArgs a = {};
    a.table = c.table;
    a.to = c.to == nullptr ? c.table : c.to;
    a.keep = c.keep;
    a.k = static_cast<uint8_t*>(const_cast<void*>(c.cache.k));
    a.v = static_cast<uint8_t*>(const_cast<void*>(c.cache.v));
    a.kscale = c.cache.kv == kKvX16 ? nullptr : const_cast<float*>(c.cache.kscale);
    a.vscale = c.cache.kv == kKvX16 ? nullptr : const_cast<float*>(c.cache.vscale);
    a.weight = c.weight;
    a.err = c.err;
    a.max_pages = c.max_pages;
    a.to_pages = c.to == nullptr ? c.max_pages : c.to_pages;
    a.num_pages = c.cache.num_pages;
    a.capacity = c.max_pages << c.cache.page_shift;
    a.budget = c.budget;
    a.Hkv = c.Hkv;
    a.shift = c.cache.page_shift;
    a.in_place = a.to == a.table;
    a.bytes = c.D * (c.cache.kv == kKvX16 ? 2 : 1);
    const int runs = a.bytes / 16;
    // slices of 64 bytes, of 32 where there are few CTAs
    a.lanes = c.B * c.Hkv * 2 * ceil_div(runs, 4) < 2 * static_cast<int64_t>(device_sm_count()) ? 2 : 4;
    a.slices = static_cast<int>(ceil_div(runs, a.lanes));
    const int64_t ctas = c.B * c.Hkv * (2 * a.slices + 1);
    const dim3 grid(static_cast<unsigned>(ctas));
    // (tokens of fp8 codes, one sequence of 577: 4.3 us with 256 threads, 3.7 with 512; 32 of
    // 8192 in bf16: 205 and 218)
    if (ctas < 2 * static_cast<int64_t>(device_sm_count())) return launch_after(move_kernel<512>, grid, 512, 0, stream, a);
    return launch_after(move_kernel<256>, grid, 256, 0, stream, a);
}

}  // namespace tern
