// Keeping a paged key/value cache within a budget of tokens: the choice of the
// tokens to keep by their accumulated weight, and their move to the front.
//
// Mathematics.  Weights become 32-bit keys in the order of the numbers (a NaN, or
// a token of a page outside the cache, below all of them).  The smallest kept key
// is found digit by digit, 8 bits at a time, by counting; of the tokens that have
// it the first ones are kept.  Counts are whole numbers, so the result does not
// depend on the order of the atomics.
//
// Moves.  A list of kept tokens ascends, so entry j is at or behind place j: tokens
// taken in order, a block of places at a time, never write what a later block
// still reads.  A CTA has one (sequence, head) and a slice of the row's bytes, reads
// a block of tokens, meets, and writes it; slices do not touch one another's bytes.

#include <float.h>

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
    int stored;            // tokens whose keys fit in shared memory
};

// Order of the numbers; -0 is 0.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) return 0;
    const uint32_t u = __float_as_uint(w == 0.0f ? 0.0f : w);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(1024) keep_kernel(const KeepArgs a) {
    extern __shared__ uint32_t keys[];
    __shared__ uint32_t bins[256];
    __shared__ uint32_t found[2];          // digit, and how many above it
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
    auto load = [&](int j) -> uint32_t {
        const int page = a.table[b * a.max_pages + (j >> a.shift)];
        if (page < 0 || page >= a.num_pages) return 0;
        return order_key(a.weight[((static_cast<int64_t>(page) * a.Hkv + hk) << a.shift) + (j & page_mask)]);
    };
    for (int j = threadIdx.x; j < min(len, a.stored); j += blockDim.x) keys[j] = load(j);
    auto key = [&](int j) { return j < a.stored ? keys[j] : load(j); };

    // the key of which `take` are left to keep when all above it are kept
    const int lo = a.first, hi = len - a.recent;
    uint32_t take = static_cast<uint32_t>(kept - a.first - a.recent), prefix = 0;
    if (take > 0) {
        for (int at = 24; at >= 0; at -= 8) {
            __syncthreads();   // (the first time: the keys are there)
            for (int i = threadIdx.x; i < 256; i += blockDim.x) bins[i] = 0;
            __syncthreads();
            const uint32_t known = at == 24 ? 0u : 0xFFFFFFFFu << (at + 8);
            for (int j = lo + threadIdx.x; j < hi; j += blockDim.x) {
                const uint32_t k = key(j);
                if ((k & known) == prefix) atomicAdd(&bins[(k >> at) & 255], 1u);
            }
            __syncthreads();
            if (warp == 0) {
                // lane l has digits 255 - 8l - 7 .. 255 - 8l, the largest first
                uint32_t c[8], mine = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) mine += c[i] = bins[255 - 8 * lane - i];
                uint32_t incl = mine;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t up = __shfl_up_sync(0xffffffffu, incl, d);
                    if (lane >= d) incl += up;
                }
                uint32_t before = incl - mine;
                if (before < take && incl >= take) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (before < take && before + c[i] >= take) {
                            found[0] = 255 - 8 * lane - i;
                            found[1] = before;
                        }
                        before += c[i];
                    }
                }
            }
            __syncthreads();
            prefix |= found[0] << at;
            take -= found[1];
        }
    } else {
        prefix = 0xFFFFFFFFu;   // no key has it
        __syncthreads();
    }

    // each warp lists a run of tokens in order
    const int run = ((len + warps - 1) / warps + 31) & ~31;
    const int j0 = min(len, warp * run), j1 = min(len, j0 + run);
    auto kind = [&](int j, bool& over, bool& same) {
        over = same = false;
        if (j >= j1) return;
        if (j < lo || j >= hi) {
            over = true;
            return;
        }
        const uint32_t k = key(j);
        over = k > prefix;
        same = k == prefix;
    };
    int n_over = 0, n_same = 0;
    for (int j = j0; j < j1; j += 32) {
        bool over, same;
        kind(j + lane, over, same);
        n_over += __popc(__ballot_sync(0xffffffffu, over));
        n_same += __popc(__ballot_sync(0xffffffffu, same));
    }
    if (lane == 0) above[warp] = n_over, equal[warp] = n_same;
    __syncthreads();
    int over_before = 0, same_before = 0;
    for (int w = 0; w < warp; ++w) over_before += above[w], same_before += equal[w];
    int place = over_before + min(same_before, static_cast<int>(take));
    const uint32_t below = (1u << lane) - 1;
    for (int j = j0; j < j1; j += 32) {
        bool over, same;
        kind(j + lane, over, same);
        const uint32_t sames = __ballot_sync(0xffffffffu, same);
        const bool in = over || (same && same_before + __popc(sames & below) < static_cast<int>(take));
        const uint32_t ins = __ballot_sync(0xffffffffu, in);
        if (in) out[place + __popc(ins & below)] = j + lane;
        place += __popc(ins);
        same_before += __popc(sames);
    }
}

// --------------------------------------------------------------------- moves

constexpr int kMoveThreads = 256;
constexpr int kUnroll = 4;         // tokens of a thread in a block of places

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
template <typename T>
__device__ __forceinline__ void move(const MoveArgs& a, T* data, int64_t row_bytes, int64_t at, bool live, int width, int b, int hk,
                                     int start, int count) {
    const int per = kMoveThreads / width;           // tokens at a time
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

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveArgs a) {
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
    for (int j = threadIdx.x; j < budget; j += kMoveThreads)
        if (list[j] < 0) {
            my_end = j;
            break;
        }
    atomicMin(&ends, my_end);
    __syncthreads();
    const int count = ends;
    bool wrong = false;
    for (int j = threadIdx.x; j < count; j += kMoveThreads) {
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
        move(a, reinterpret_cast<uint4*>(data), a.bytes, 16 * run, 16 * run < a.bytes, a.lanes, b, hk, start, count);
    } else {
        if (a.kscale != nullptr) move(a, a.kscale, 4, 0, true, 1, b, hk, start, count);
        if (a.vscale != nullptr) move(a, a.vscale, 4, 0, true, 1, b, hk, start, count);
        if (a.weight != nullptr) move(a, a.weight, 4, 0, true, 1, b, hk, start, count);
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
    constexpr int kMostStored = 49152;
    a.stored = static_cast<int>(a.capacity < kMostStored ? a.capacity : kMostStored);
    static OncePerDevice once;
    const cudaError_t limit = allow_smem(once, keep_kernel, kMostStored * 4);
    if (limit != cudaSuccess) return limit;
    const unsigned threads = a.capacity <= 2048 ? 256 : a.capacity <= 8192 ? 512 : 1024;
    return launch_after(keep_kernel, dim3(static_cast<unsigned>(c.B * c.Hkv)), threads, static_cast<size_t>(a.stored) * 4, stream, a);
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
    a.lanes = 4;
    a.slices = static_cast<int>(ceil_div(runs, a.lanes));
    return launch_after(move_kernel, dim3(static_cast<unsigned>(c.B * c.Hkv * (2 * a.slices + 1))), kMoveThreads, 0, stream, a);
}

}  // namespace tern
