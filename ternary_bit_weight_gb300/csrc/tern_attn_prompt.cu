// Attention over packed prompts:
//   O = softmax(scale Q K^T, keys a query may see) V.
//
// Mathematics.  One pass over the keys in tiles of 128 with the softmax in
// base 2: a row keeps a reference m, l = sum 2^(s-m) and o = sum 2^(s-m) v
// (s = scale log2(e) q.k), rescaled when m moves.  m follows the running
// maximum lazily: it moves only when a tile's maximum passes it by 8, so
// weights stay below 2^8 and the rescaling of o is rare.  Weights are rounded
// to the 16-bit type for the product with V, the tensor cores taking both of its
// operands in one type; l sums them unrounded in fp32.  (With it the output of 8192
// bf16 tokens is 0.0021, relative, from 64 bits; with the output's rounding alone it
// would be 0.0016.)
//
// What bounds it: for long prompts the tensor cores (4 D flops per pair that
// attends) and, beside them, the exponential of every score; for short ones
// the launch and the chain load -> scores -> softmax -> values -> store.
//
// Rows of a tile.  A tile is `tok` tokens x `gs` of the heads that share one
// key/value head, gs * tok <= 128 rows (gs = 1: 128 tokens of one head).  With
// gs > 1 short sequences fill the tile with the group's heads; the host takes
// the gs that needs the fewest tiles.  A CTA works on two tiles of consecutive
// tokens against the same keys: while the softmax of one runs, the tensor
// cores multiply for the other.  For short sequences a CTA has one tile (10 warps,
// the load warp is the guard, too) and two CTAs share an SM (see plan_prompt).
// Measured, 40 / 8 heads of 128, causal, bf16: 8192 tokens 450-485 us (1.42-1.53
// PFLOP/s, with the power limit), 4096 137 us, 512 11.2 us, 32 prompts of 128 40 us.
//
// Roles (two tiles, 20 warps):
//   * warp 0 issues all tcgen05.mma: scores S_i = Q_i K_j^T (both operands in
//     shared memory) into tensor memory, and O_i += P_i V_j with P_i in tensor
//     memory over the columns of S_i (operations of one thread run in order,
//     so S_i of the next tile follows the product that reads P_i).  Per tile
//     and key tile it votes once over all barriers and issues both products: a
//     wait costs it some 170 cycles even when the barrier is complete, and the
//     tensor pipe runs dry meanwhile;
//   * warp 1 brings Q and the K and V tiles by TMA (128-byte swizzle);
//   * warp 2 makes V tiles safe that hold keys some row must not see: 0 * NaN
//     is NaN, so non-finite values there become 0 before the product, and the
//     epilogue adds them to the rows that do see them;
//   * warps 4-11 and 12-19, eight per tile: softmax, rescaling of O in tensor
//     memory, epilogue.  A warp has 16 rows, four threads sharing each (the
//     16-lane forms of tensor-memory access): the time from scores to weights
//     has to fit into the other tile's products, and with one thread per row it
//     was 1660 cycles against their 1024.
// Few rows against many keys: the keys are split over CTAs, which leave
// (m, l, o) in the workspace for a second kernel that adds them in split order.
// Every wait is bounded; a timeout raises the workspace error word.

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

constexpr int kTileM = 128, kTileN = 128;
constexpr int kHalf = kTileM * 128;           // 128 rows x 64 elements of 16 bits
constexpr int kMaxNT = 2;

// The two forms of the kernel: NT tiles per CTA.
template <int NT>
struct Form {
    static constexpr int kMmaWarp = 0, kLoadWarp = 1;
    static constexpr int kGuardWarp = NT == 2 ? 2 : -1;   // NT == 1: the load warp guards, too
    static constexpr int kSoftWarp0 = NT == 2 ? 4 : 2;    // any 4 warps in a row reach all tensor-memory lanes
    static constexpr int kThreads = (kSoftWarp0 + 8 * NT) * 32;
    static constexpr int kCtas = NT == 2 ? 1 : 2;         // per SM
    static constexpr int kSlots = NT == 2 ? 4 : 2;        // K and V tiles, alternating: K even, V odd
    static constexpr int kSCol = 0, kOCol = NT * kTileN;
    static constexpr int kTmemCols = NT == 2 ? 512 : 256;
    static_assert(NT * (kTileN + 128) <= kTmemCols, "tensor-memory budget");
};
constexpr int kShareBytes = kMaxNT * kTileM * 8;       // reference and sum of every row
constexpr int kShare = 256;
constexpr int kCtrlBytes = kShare + kShareBytes;
constexpr float kLazy = 8.0f;
constexpr float kNone = -FLT_MAX;     // reference before any key: no finite score is below it
constexpr float kFar = 2097152.0f;   // 2^21: from here on a reference's unit is 1/4 and more
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

// control block
constexpr int kMaxSlots = Form<2>::kSlots;
constexpr int kBarFull = 0;                          // [slots] tile landed
constexpr int kBarEmpty = kBarFull + 8 * kMaxSlots;     // [slots] tile consumed
constexpr int kBarRaw = kBarEmpty + 8 * kMaxSlots;      // [2] V tile landed that the guard looks over
constexpr int kBarSafe = kBarRaw + 8 * 2;            // [2] and is ready
constexpr int kBarQ = kBarSafe + 8 * 2;              // [NT]
constexpr int kBarS = kBarQ + 8 * kMaxNT;               // [NT] scores ready
constexpr int kBarP = kBarS + 8 * kMaxNT;               // [NT] weights ready
constexpr int kBarO = kBarP + 8 * kMaxNT;               // [NT] product with V done
constexpr int kBarDrain = kBarO + 8 * kMaxNT;
constexpr int kTmemPtr = kBarDrain + 8;
constexpr int kAbort = kTmemPtr + 4;
constexpr int kBad = kAbort + 4;                     // a value was taken out by the guard
constexpr int kItem = kBad + 4;                      // an Item
static_assert(kItem + 20 <= kShare, "control block");

template <int DP, int NT>
constexpr int smem_bytes() {
    return 1024 + (NT + Form<NT>::kSlots) * (DP / 64) * kHalf + kCtrlBytes;
}
static_assert(smem_bytes<128, 2>() <= 232448 && smem_bytes<128, 1>() <= 115712, "shared-memory budget");

struct Maps {
    CUtensorMap q, k, v;
};

struct Args {
    const int32_t* cu_q;
    const int32_t* cu_kv;
    const uint16_t* v;
    uint16_t* o;
    float* lse;
    float* part;          // split keys: [tile][split][D / 4][128 rows][4] unnormalised outputs
    float* part_ml;       // [tile][split][128 rows][2]: reference, sum
    int* err;
    int64_t ldv, ldo;
    int B, Tq, Tkv, Hq, G, D;
    int nt;               // tiles of a block
    int gs, tok, chunks;  // heads and tokens of a tile; chunks = ceil(G / gs)
    int HC;               // key/value heads x chunks
    int splits;
    int causal;
    float scale2;         // scale * log2(e)
};

// Where a block works: tokens [t0, t0 + nt * tok) of sequence b, its rows of Q
// from q0 and of K from k0.
struct Item {
    int q0, nq, k0, nk, t0;
};

__device__ __forceinline__ void clamp_range(const int32_t* cu, int b, int total, int& lo, int& n) {
    lo = min(max(cu[b], 0), total);
    n = max(0, min(max(cu[b + 1], 0), total) - lo);
}

// Block `index` of the sequences' token blocks in order; the blocks of a
// sequence run from its end, whose causal rows see most keys.  One warp; false
// past the last block.  A lane counts the blocks of RUN sequences, whose offsets
// it loads together.
template <int RUN>
__device__ __forceinline__ bool find_item(const Args& a, int index, int lane, Item& it) {
    int base = 0;
    const int step = a.nt * a.tok;
    for (int b0 = 0; b0 < a.B; b0 += 32 * RUN) {
        const int first = b0 + lane * RUN;
        int q0[RUN], nq[RUN], k0 = 0, nk = 0, mine = 0;
#pragma unroll
        for (int i = 0; i < RUN; ++i) {
            q0[i] = nq[i] = 0;
            if (first + i < a.B) clamp_range(a.cu_q, first + i, a.Tq, q0[i], nq[i]);
        }
        if (RUN == 1 && first < a.B) clamp_range(a.cu_kv, first, a.Tkv, k0, nk);
#pragma unroll
        for (int i = 0; i < RUN; ++i) mine += static_cast<uint32_t>(nq[i] + step - 1) / static_cast<uint32_t>(step);
        int incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += up;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, base + incl > index);
        if (past != 0) {
            const int src = __ffs(past) - 1;
            // the lane that has it finds the sequence of its run
            int end = base + incl - mine, b = first, q = q0[0], n = nq[0];
#pragma unroll
            for (int i = 0; i < RUN; ++i)
                if (end <= index) {
                    b = first + i;
                    q = q0[i];
                    n = nq[i];
                    end += static_cast<uint32_t>(n + step - 1) / static_cast<uint32_t>(step);
                }
            it.q0 = __shfl_sync(0xffffffffu, q, src);
            it.nq = __shfl_sync(0xffffffffu, n, src);
            it.t0 = (__shfl_sync(0xffffffffu, end, src) - 1 - index) * step;
            if (RUN > 1) clamp_range(a.cu_kv, __shfl_sync(0xffffffffu, b, src), a.Tkv, k0, nk);
            it.k0 = __shfl_sync(0xffffffffu, k0, src);
            it.nk = __shfl_sync(0xffffffffu, nk, src);
            return true;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
}

// Keys that token t of the item sees.
__device__ __forceinline__ int visible(const Args& a, const Item& it, int t) {
    return a.causal ? max(0, min(it.nk, t + 1 + it.nk - it.nq)) : it.nk;
}

// Wait for the phase with the given parity; false when *abort is set or after
// kWaitTimeoutNs, in which case it sets *abort.  Inline, unlike mbar_wait: a
// call would spill the row of scores that a softmax thread holds.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort) {
    bool got = mbar_test_wait(bar, parity);
    uint64_t t0 = 0;
    for (uint32_t i = 1; !got; ++i) {
        got = mbar_try_wait(bar, parity);
        if (!got && (i & 15u) == 0) {
            if (*abort) break;
            const uint64_t t = global_timer_ns();
            if (t0 == 0) {
                t0 = t;
            } else if (t - t0 > kWaitTimeoutNs) {
                *abort = 1;
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, got);
}

// D[tmem] (+)= A[smem] . B[smem]^T
__device__ __forceinline__ void umma_smem_a(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// MN-major operand in the 128-byte swizzle: rows of 64 elements along MN, one
// per K index, in atoms of 8 rows (1024 bytes): stride (bits 32-45) 1024 bytes
// between atoms along K, leading offset (16-29) between runs of 64 along MN.
__device__ __forceinline__ uint64_t smem_desc_mnmajor_sw128(uint32_t saddr, uint32_t next64) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((next64 >> 4) & 0x3FFFu) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
constexpr uint32_t kBMnMajor = 1u << 16;   // instruction descriptor: B is MN-major

// acc + 0 * w on both halves: a non-finite half makes its sum NaN for good.
template <bool F16>
__device__ __forceinline__ uint32_t times_zero(uint32_t w, uint32_t acc) {
    uint32_t d;
    if (F16)
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(w), "r"(0u), "r"(acc));
    else
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(w), "r"(0u), "r"(acc));
    return d;
}

template <bool F16>
__device__ __forceinline__ bool value_non_finite(uint16_t u) {
    constexpr uint16_t ones = F16 ? 0x7C00 : 0x7F80;
    return (u & ones) == ones;
}

template <int DP, bool F16, int NT>
__global__ void __launch_bounds__(Form<NT>::kThreads, Form<NT>::kCtas) prompt_kernel(const __grid_constant__ Maps maps,
                                                                                     const __grid_constant__ Args a) {
    using F = Form<NT>;
    constexpr int kNT = NT, kSlots = F::kSlots, kSCol = F::kSCol, kOCol = F::kOCol;
    constexpr int kHalves = DP / 64, kTileBytes = kHalves * kHalf;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t sq = smem_u32(smem), skv = sq + kNT * kTileBytes;
    uint8_t* ctrl = smem + (kNT + kSlots) * kTileBytes;
    const uint32_t cb = smem_u32(ctrl);
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(ctrl + kTmemPtr);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + kAbort);
    volatile int* bad_flag = reinterpret_cast<volatile int*>(ctrl + kBad);
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

    if (warp == F::kLoadWarp) {   // which uses them first
        if (lane < 3) prefetch_tensormap(lane == 0 ? &maps.q : lane == 1 ? &maps.k : &maps.v);
        if (elect_one()) {
            for (int i = 0; i < kSlots; ++i) {
                mbar_init(cb + kBarFull + 8 * i, 1);
                mbar_init(cb + kBarEmpty + 8 * i, 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(cb + kBarRaw + 8 * i, 1);
                mbar_init(cb + kBarSafe + 8 * i, 1);
            }
            for (int i = 0; i < kNT; ++i) {
                mbar_init(cb + kBarQ + 8 * i, 1);
                mbar_init(cb + kBarS + 8 * i, 1);
                mbar_init(cb + kBarP + 8 * i, 8);
                mbar_init(cb + kBarO + 8 * i, 1);
            }
            mbar_init(cb + kBarDrain, 1);
            *abort_flag = 0;
            *bad_flag = 0;
            mbar_fence_init();
        }
        __syncwarp();
    }
    const uint32_t rest = blockIdx.x / static_cast<uint32_t>(a.HC);
    const int hc = blockIdx.x - rest * a.HC;
    const int block = a.splits == 1 ? rest : rest / static_cast<uint32_t>(a.splits);
    const int split = rest - block * a.splits;
    grid_dependency_wait();
    // The next kernel is let in once this CTA has its tensor memory: a kernel that took
    // tensor memory first and then waited for this one would never get to run (the
    // allocation waits without a limit).
    auto allocate = [&]() {
        tmem_alloc(smem_u32(tmem_ptr), F::kTmemCols);
        tmem_relinquish();
        grid_launch_dependents();
    };
    Item it = {};
    if constexpr (NT == 1) {
        // One warp finds the item, the others get it with the barrier: short blocks
        // are many, and ten warps' loads of the same offsets held one another up (per
        // call in a CUDA graph, 32 queries of up to 48 tokens 6.9 us instead of 7.6, 200
        // prompts of 64 117 instead of 135).  With two tiles the loads are earlier when
        // nobody waits for a barrier.
        int* found = reinterpret_cast<int*>(ctrl + kItem);
        if (warp == F::kLoadWarp) {
            if (!(a.B <= 64 ? find_item<1>(a, block, lane, it) : find_item<4>(a, block, lane, it))) it.nq = 0;
            if (lane == 0) found[0] = it.q0, found[1] = it.nq, found[2] = it.k0, found[3] = it.nk, found[4] = it.t0;
        } else if (warp == F::kMmaWarp) {
            allocate();
        }
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
        it.q0 = found[0], it.nq = found[1], it.k0 = found[2], it.nk = found[3], it.t0 = found[4];
        if (it.nq == 0) {   // past the last block
            if (warp == F::kMmaWarp) tmem_dealloc(*tmem_ptr, F::kTmemCols);
            return;
        }
    } else {
        if (!find_item<1>(a, block, lane, it)) return;   // the whole CTA
    }

    const int hk = hc / a.chunks, head0 = hk * a.G + (hc - hk * a.chunks) * a.gs;
    const int heads = min(a.gs, (hk + 1) * a.G - head0);   // of the tile's gs, those that exist
    // key tiles: tile i works on [j0, e[i])
    int e[kNT], last[kNT];   // last: tokens of tile i
    // Key tile of which tile i sees at most half: products, softmax and guard take
    // that half only.  (32 queries of up to 48 tokens 0.4 us less of 8.0, 200 prompts
    // of 64 9 of 144.  With two tiles per CTA the branches cost the long
    // prompts 7 %, so only with one.)
    int shorter[kNT];
    int most = 0, keys_most = 0;
#pragma unroll
    for (int i = 0; i < kNT; ++i) {
        last[i] = min(a.tok, it.nq - it.t0 - i * a.tok);
        const int keys = last[i] > 0 ? visible(a, it, it.t0 + i * a.tok + last[i] - 1) : 0;
        e[i] = (keys + kTileN - 1) / kTileN;
        shorter[i] = NT == 1 && e[i] * kTileN - keys >= kTileN / 2 ? e[i] - 1 : -1;
        most = max(most, e[i]);
        keys_most = max(keys_most, keys);
    }
    int j0 = 0, j1 = most;
    if (a.splits > 1) {   // most < 2^24, splits <= 32
        j0 = static_cast<uint32_t>(most) * split / static_cast<uint32_t>(a.splits);
        j1 = static_cast<uint32_t>(most) * (split + 1) / static_cast<uint32_t>(a.splits);
    }
#pragma unroll
    for (int i = 0; i < kNT; ++i) e[i] = max(j0, min(e[i], j1));
    // first tile that holds a key which some row does not see
    const int jm = visible(a, it, it.t0) / kTileN;
    // guarded V tiles are jg, jg + 1, ...: they complete on barriers of their own,
    // two in turn, which count guarded tiles only
    const int jg = max(j0, jm);

    // K or V tile n of the loads (K and V of each key tile in turn).
    auto load_tile = [&](int n) {
        const int slot = n % kSlots, j = j0 + n / 2;
        const uint32_t bar = cb + ((n & 1) && j >= jm ? kBarRaw + 8 * ((j - jg) & 1) : kBarFull + 8 * slot);
        if (elect_one()) {
            mbar_arrive_expect_tx(bar, kTileBytes);
            for (int h = 0; h < kHalves; ++h)
                tma_load_3d(skv + slot * kTileBytes + h * kHalf, n & 1 ? &maps.v : &maps.k, 64 * h, hk, it.k0 + j * kTileN, bar);
        }
        __syncwarp();
    };
    // Make guarded V tile j safe (one warp): keys from `seen` on are hidden from some
    // row, those from nk on from all.
    const int seen = visible(a, it, it.t0);
    auto guard = [&](int j) {
        const int slot = (2 * (j - j0) + 1) % kSlots, bar = 8 * ((j - jg) & 1);
        if (!warp_wait(cb + kBarRaw + bar, ((j - jg) >> 1) & 1, abort_flag)) return false;
        const int lo = max(0, seen - j * kTileN), hi = min(kTileN, it.nk - j * kTileN);
        uint8_t* tile = smem + (kNT + slot) * kTileBytes + lane * 16;   // a row's 128 bytes are 8 lanes'
        uint32_t acc[4] = {0, 0, 0, 0};
        const uint32_t* first = reinterpret_cast<const uint32_t*>(tile);
        for (int h = 0; h < kHalves; ++h) {
#pragma unroll 8
            for (int row = lo & ~3; row < hi; row += 4) {
                const uint4 u = *reinterpret_cast<const uint4*>(first + (h * kHalf + row * 128) / 4);
                acc[0] = times_zero<F16>(u.x, acc[0]);
                acc[1] = times_zero<F16>(u.y, acc[1]);
                acc[2] = times_zero<F16>(u.z, acc[2]);
                acc[3] = times_zero<F16>(u.w, acc[3]);
            }
        }
        const uint32_t any = acc[0] | acc[1] | acc[2] | acc[3];
        bool wrote = false;
        if (__any_sync(0xffffffffu, (any & 0x7FFF7FFFu) != 0)) {
            wrote = true;
            uint16_t* value = reinterpret_cast<uint16_t*>(tile);
            for (int h = 0; h < kHalves; ++h)
                for (int row = lo & ~3; row < hi; row += 4)
                    for (int q = 0; q < 8; ++q)
                        if (row + (lane >> 3) >= lo && value_non_finite<F16>(value[(h * kHalf + row * 128) / 2 + q]))
                            value[(h * kHalf + row * 128) / 2 + q] = 0;
            if (lane == 0) *bad_flag = 1;
        }
        const int used = NT == 1 && keys_most - j * kTileN <= kTileN / 2 ? kTileN / 2 : kTileN;   // rows that the product takes
        if (hi < used) {
            wrote = true;
            for (int h = 0; h < kHalves; ++h)
                for (int row = hi & ~3; row < used; row += 4)
                    if (row + (lane >> 3) >= hi) *reinterpret_cast<uint4*>(tile + h * kHalf + row * 128) = make_uint4(0, 0, 0, 0);
        }
        if (wrote) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(cb + kBarSafe + bar);
        return true;
    };

    // the first loads
    if (warp == F::kLoadWarp && j1 > j0) {
        if (elect_one()) {
#pragma unroll
            for (int i = 0; i < kNT; ++i) {
                if (e[i] == j0) continue;
                mbar_arrive_expect_tx(cb + kBarQ + 8 * i, kHalves * a.gs * a.tok * 128);
                for (int h = 0; h < kHalves; ++h)
                    tma_load_3d(sq + i * kTileBytes + h * kHalf, &maps.q, 64 * h, head0, it.q0 + it.t0 + i * a.tok,
                                cb + kBarQ + 8 * i);
            }
        }
        __syncwarp();
        for (int n = 0; n < min(kSlots, 2 * (j1 - j0)); ++n) load_tile(n);
    }
    if constexpr (NT == 2) {
        if (warp == F::kMmaWarp) allocate();
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
    }
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_ptr, 0);   // uniform, and known to be

    if (warp < F::kSoftWarp0) {
        if (warp == F::kLoadWarp) {
            // ------------------------------------------------------------ loads
            if (j1 > j0) {
                bool ok = true;
                for (int n = 0; n < 2 * (j1 - j0) && ok; ++n) {
                    if (n >= kSlots) {
                        if (!(ok = warp_wait(cb + kBarEmpty + 8 * (n % kSlots), (n / kSlots - 1) & 1, abort_flag))) break;
                        load_tile(n);
                    }
                    if (F::kGuardWarp < 0 && (n & 1) && j0 + n / 2 >= jg) ok = guard(j0 + n / 2);
                }
                if (*abort_flag) {   // copies in flight must land before the CTA ends
                    volatile int no_abort = 0;
                    for (int s = 0; s < kSlots; ++s) {
                        (void)warp_wait(cb + kBarFull + 8 * s, 0, &no_abort);
                        (void)warp_wait(cb + kBarFull + 8 * s, 1, &no_abort);
                    }
                    for (int s = 0; s < 2; ++s) {
                        (void)warp_wait(cb + kBarRaw + 8 * s, 0, &no_abort);
                        (void)warp_wait(cb + kBarRaw + 8 * s, 1, &no_abort);
                    }
                    for (int i = 0; i < kNT; ++i) (void)warp_wait(cb + kBarQ + 8 * i, 0, &no_abort);
                }
            }
        } else if (warp == F::kMmaWarp) {
            // -------------------------------------------------------------- MMA
            const uint32_t type = F16 ? idesc_fp16_f32(128, 0) : idesc_bf16_f32(128, 0);
            const uint32_t idesc_s = type | ((kTileN >> 3) << 17), idesc_half = type | ((kTileN >> 4) << 17);
            const uint32_t idesc_o = type | (static_cast<uint32_t>(a.D >> 3) << 17) | kBMnMajor;
            const int steps = a.D / 16;
            // lane 0, which is elected, tests no barrier: its tests would wait behind its
            // own commits, that is, until its last products have completed
            auto scores = [&](int i, int n) {   // S_i = Q_i K^T, K in load n
                const uint32_t idesc = NT == 1 && j0 + n / 2 == shorter[i] ? idesc_half : idesc_s;
                const uint64_t ad = smem_desc_kmajor_sw128(sq + i * kTileBytes);
                const uint64_t bd = smem_desc_kmajor_sw128(skv + (n % kSlots) * kTileBytes);
#pragma unroll
                for (int s = 0; s < DP / 16; ++s)
                    if (s < steps) {
                        const uint32_t off = (s >> 2) * (kHalf / 16) + 2 * (s & 3);
                        umma_smem_a(tmem + kSCol + i * kTileN, ad + off, bd + off, idesc, s > 0);
                    }
                umma_commit(cb + kBarS + 8 * i);
            };
            bool ok = j1 > j0;
            if (ok) {
                const bool q = (lane == 1 && e[0] > j0) || (NT == 2 && lane == 2 && e[kNT - 1] > j0);
                ok = vote_wait(q ? cb + kBarQ + 8 * (lane - 1) : cb + kBarFull, 0, q || lane == 3, abort_flag);
                tc_fence_after_sync();
                if (ok && elect_one()) {
#pragma unroll
                    for (int i = 0; i < kNT; ++i)
                        if (e[i] > j0) scores(i, 0);
                    umma_commit(cb + kBarEmpty);
                }
                __syncwarp();
            }
            for (int j = j0; j < j1 && ok; ++j) {
                const int n = 2 * (j - j0) + 1, slot = n % kSlots, kslot = (n + 1) % kSlots;
                const bool next = j + 1 < j1;
                // a guarded tile is ready when the guard says so
                const uint32_t vbar = cb + (j >= jm ? kBarSafe + 8 * ((j - jg) & 1) : kBarFull + 8 * slot);
                const uint32_t vph = j >= jm ? ((j - jg) >> 1) & 1 : (n / kSlots) & 1;
                const uint64_t bd = smem_desc_mnmajor_sw128(skv + slot * kTileBytes, kHalf);
#pragma unroll
                for (int i = 0; i < kNT; ++i) {
                    if (j >= e[i]) continue;
                    // weights (lane 1), this V tile (2), the next K tile (3)
                    const uint32_t bar = lane == 1 ? cb + kBarP + 8 * i : lane == 2 ? vbar : cb + kBarFull + 8 * kslot;
                    const uint32_t par = lane == 1 ? (j - j0) & 1 : lane == 2 ? vph : ((n + 1) / kSlots) & 1;
                    if (!(ok = vote_wait(bar, par, lane == 1 || lane == 2 || (lane == 3 && next), abort_flag))) break;
                    tc_fence_after_sync();
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < kTileN / 16; ++s) {   // 16 keys: 16 rows of 128 bytes
                            if (NT == 1 && s == kTileN / 32 && j == shorter[i]) break;
                            umma_bf16_tmem_a(tmem + kOCol + i * DP, tmem + kSCol + i * kTileN + 8 * s, bd + s * (2048 / 16),
                                             idesc_o, (j > j0 || s > 0) ? 1u : 0u);
                        }
                        umma_commit(cb + kBarO + 8 * i);
                        if (j + 1 < e[i]) scores(i, n + 1);
                        if (i == kNT - 1 || j >= e[kNT - 1]) {   // the last tile that reads these
                            umma_commit(cb + kBarEmpty + 8 * slot);
                            if (next) umma_commit(cb + kBarEmpty + 8 * kslot);
                        }
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) umma_commit(cb + kBarDrain);
            __syncwarp();
            volatile int no_abort = 0;
            (void)warp_wait(cb + kBarDrain, 0, &no_abort);
        } else if (warp == F::kGuardWarp) {
            for (int j = jg; j < j1; ++j)
                if (!guard(j)) break;
        }
    } else {
        // ---------------------------------------------------------- softmax
        const int i = (warp - F::kSoftWarp0) >> 3;
        const int half = ((warp - F::kSoftWarp0) >> 2) & 1;      // which 16 of the quarter's 32 lanes; in the epilogue, which columns
        const uint32_t quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + quarter + (static_cast<uint32_t>(16 * half) << 16) + kSCol + i * kTileN;
        const uint32_t to = tmem + quarter + kOCol + i * DP, to16 = to + (static_cast<uint32_t>(16 * half) << 16);
        const int end = i == 0 ? e[0] : e[kNT - 1], half_tile = i == 0 ? shorter[0] : shorter[kNT - 1];
        const float scale2 = a.scale2;
        // the thread's rows r0 and r0 + 8: the keys they see, their references and sums
        const int r0 = (warp & 3) * 32 + half * 16 + (lane >> 2);
        int lim[2];
        float m[2] = {kNone, kNone}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int token = (r0 + 8 * q) / a.gs, head = r0 + 8 * q - token * a.gs;
            const bool live = token < last[i] && head < heads;
            lim[q] = live ? visible(a, it, it.t0 + i * a.tok + token) : 0;
            // a row that does not exist (its queries are whatever shared memory held)
            // never asks for a new reference, so the others' do not depend on it
            if (!live) m[q] = CUDART_INF_F;
        }
        float2* share = reinterpret_cast<float2*>(ctrl + kShare) + i * kTileM;
        // Scores far from zero are taken relative to a base of their row (in share[].x): a
        // reference is a rounded product, and the fused difference of a score and it would
        // give the row's largest score 2^(what the rounding dropped) as its weight, past 16
        // bits' range from 2^28 on.  `far`: some row of the warp has one.
        bool far = false;
        auto rebase = [&](float (&s)[kTileN / 2], int q, float base) {
            const float up = 1.0f / scale2;
#pragma unroll
            for (int c = 0; c < kTileN / 8; ++c)
#pragma unroll
                for (int k = 0; k < 2; ++k) s[4 * c + 2 * q + k] = (__fmul_rn(s[4 * c + 2 * q + k], scale2) - base) * up;
        };
        bool ok = true;
        for (int j = j0; j < end; ++j) {
            if (!(ok = warp_wait(cb + kBarS + 8 * i, (j - j0) & 1, abort_flag))) break;
            tc_fence_after_sync();
            float s[kTileN / 2];   // register 4c + 2q + k: row q, key 8c + 2 (lane mod 4) + k
            tmem_ld_16x256b_x16_sync(ts, reinterpret_cast<uint32_t*>(s));
            if (j >= jm) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int keys = lim[q] - j * kTileN - 2 * (lane & 3);
#pragma unroll
                    for (int c = 0; c < kTileN / 8; ++c) {
                        if (8 * c >= keys) s[4 * c + 2 * q] = -CUDART_INF_F;
                        if (8 * c + 1 >= keys) s[4 * c + 2 * q + 1] = -CUDART_INF_F;
                    }
                }
            }
            if (far) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float base = share[r0 + 8 * q].x;
                    float top = s[2 * q];
#pragma unroll
                    for (int c = 0; c < kTileN / 8; ++c) top = fmaxf(top, fmaxf(s[4 * c + 2 * q], s[4 * c + 2 * q + 1]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));   // (which also is the lanes' barrier)
                    top = __fmul_rn(fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)), scale2);
                    if (top <= FLT_MAX && top - base > FLT_MAX) {
                        // beyond fp32's range above the base: what the row has seen so far weighs
                        // nothing, and it starts again
                        m[q] = kNone;
                        if ((lane & 3) == 0) share[r0 + 8 * q].x = 0.0f;
                    } else if (base != 0.0f) {
                        rebase(s, q, base);
                    }
                }
                __syncwarp();
            }
            float mx[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float top[2] = {s[2 * q], s[2 * q + 1]};
#pragma unroll
                for (int c = 1; c < kTileN / 8; ++c) top[c & 1] = fmaxf(fmaxf(top[c & 1], s[4 * c + 2 * q]), s[4 * c + 2 * q + 1]);
                mx[q] = fmaxf(top[0], top[1]) * scale2;
            }
            if (__any_sync(0xffffffffu, mx[0] > m[0] + kLazy || mx[1] > m[1] + kLazy)) {
                float f[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float up = fmaxf(mx[q], __shfl_xor_sync(0xffffffffu, mx[q], 1));
                    up = fmaxf(m[q], fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 2)));
                    f[q] = exp2_approx(m[q] - up);
                    m[q] = up;
                    l[q] *= f[q];
                }
                // (not rows that have seen nothing or do not exist)
                auto is_far = [](float m) { return fabsf(m) >= kFar && fabsf(m) <= FLT_MAX && m != kNone; };
                if (__any_sync(0xffffffffu, is_far(m[0]) || is_far(m[1]))) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float before = far ? share[r0 + 8 * q].x : 0.0f, more = is_far(m[q]) ? m[q] : 0.0f;
                        __syncwarp();   // the four lanes of a row have read it
                        if ((lane & 3) == 0) share[r0 + 8 * q].x = before + more;
                        if (more != 0.0f) {
                            rebase(s, q, more);
                            m[q] = 0.0f;
                        }
                    }
                    __syncwarp();
                    far = true;
                }
                if (j > j0) {
                    if (!(ok = warp_wait(cb + kBarO + 8 * i, (j - j0 - 1) & 1, abort_flag))) break;
                    tc_fence_after_sync();
                    for (int c = 0; c < a.D; c += 16) {
                        uint32_t u[8];
                        tmem_ld_16x256b_x2_sync(to16 + c, u);
#pragma unroll
                        for (int q = 0; q < 8; ++q) u[q] = __float_as_uint(__uint_as_float(u[q]) * f[(q >> 1) & 1]);
                        tmem_st_16x256b_x2(to16 + c, u);
                    }
                }
            }
            const uint64_t scale_x2 = pair(scale2, scale2), minus_m[2] = {pair(-m[0], -m[0]), pair(-m[1], -m[1])};
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (NT == 1 && h == 1 && j == half_tile) break;   // (its scores are from before, masked)
                uint32_t p[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) {   // pair c of this half: row c & 1
                    float x, y;
                    unpair(fma_x2(pair(s[32 * h + 2 * c], s[32 * h + 2 * c + 1]), scale_x2, minus_m[c & 1]), x, y);
                    x = exp2_approx(x);
                    y = exp2_approx(y);
                    sum[c & 1] = add_x2(sum[c & 1], pair(x, y));
                    p[c] = pack_x2<F16>(x, y);
                }
                tmem_st_16x128b_x8(ts + 32 * h, p);
            }
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(cb + kBarP + 8 * i);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float x, y;
                unpair(sum[q], x, y);
                l[q] += x + y;
            }
        }
        // --------------------------------------------------------- epilogue
        // one thread per row of the quarter, the two warps half of the columns each
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (far) m[q] += share[r0 + 8 * q].x;
            __syncwarp();
            l[q] += __shfl_xor_sync(0xffffffffu, l[q], 1);
            l[q] += __shfl_xor_sync(0xffffffffu, l[q], 2);
            if ((lane & 3) == 0) share[r0 + 8 * q] = make_float2(m[q], l[q]);
        }
        if (end > j0 && ok) {
            ok = warp_wait(cb + kBarO + 8 * i, (end - j0 - 1) & 1, abort_flag);
            tc_fence_after_sync();
        }
        // (both warps come here, whatever their waits did)
        ok = !named_barrier_or(1 + 4 * i + (warp & 3), 64, !ok);
        const int r = (warp & 3) * 32 + lane;
        const int token = r / a.gs, head = r - token * a.gs;
        const bool live = token < last[i] && head < heads;
        const int t = it.t0 + i * a.tok + token;
        const float m_row = share[r].x, l_row = share[r].y;
        const int middle = (a.D + 63) / 64 * 32, c0 = half ? middle : 0, c1 = half ? a.D : middle;   // columns, by 32
        if (ok) {
            const bool bad = *bad_flag != 0;
            const bool split_keys = a.splits > 1;
            const int64_t part = ((static_cast<int64_t>(block) * a.HC + hc) * kNT + i) * a.splits + split;
            const int lim_row = live ? visible(a, it, t) : 0;
            const float inv = split_keys ? 1.0f : l_row > 0.0f ? 1.0f / l_row : l_row == 0.0f ? 0.0f : CUDART_NAN_F;
            uint8_t* stage = smem + i * kTileBytes;   // over the queries, whose products are done
            for (int c = c0; c < c1; c += 32) {   // (columns from D on are loaded, too, and dropped)
                float x[32];
                if (end > j0) {
                    tmem_ld32_sync(to + c, reinterpret_cast<uint32_t*>(x));
                } else {
#pragma unroll
                    for (int q = 0; q < 32; ++q) x[q] = 0.0f;
                }
#pragma unroll
                for (int q = 0; q < 32; ++q) x[q] *= inv;
                if (bad && live) {   // values taken out by the guard
                    for (int key = max(seen, j0 * kTileN); key < min(lim_row, j1 * kTileN); ++key) {
                        const uint16_t* src = a.v + (it.k0 + key) * a.ldv + static_cast<int64_t>(hk) * a.D + c;
#pragma unroll
                        for (int q = 0; q < 32; ++q) {
                            const uint32_t w = c + q < a.D ? src[q] : 0;
                            if (value_non_finite<F16>(static_cast<uint16_t>(w))) x[q] += unpack_x2<F16>(w).x;
                        }
                    }
                }
                if (split_keys) {   // [4 columns][row], so that a warp's rows lie together
                    float4* dst = reinterpret_cast<float4*>(a.part) + (part * (a.D / 4) + c / 4) * kTileM + r;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (c + 4 * q < a.D)
                            dst[q * kTileM] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
                } else {
                    // 16-byte runs spread over the banks by the row
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<uint4*>(stage + r * (DP * 2) + (((c / 8 + q) ^ (r & 7)) << 4)) =
                            make_uint4(pack_x2<F16>(x[8 * q], x[8 * q + 1]), pack_x2<F16>(x[8 * q + 2], x[8 * q + 3]),
                                       pack_x2<F16>(x[8 * q + 4], x[8 * q + 5]), pack_x2<F16>(x[8 * q + 6], x[8 * q + 7]));
                }
            }
            const int64_t row = it.q0 + t;
            if (half == 0) {
                if (split_keys)
                    reinterpret_cast<float2*>(a.part_ml)[part * kTileM + r] = make_float2(m_row, l_row);
                else if (live && a.lse != nullptr)
                    a.lse[row * a.Hq + head0 + head] = l_row == 0.0f ? -CUDART_INF_F : m_row * kLn2 + logf(l_row);
            }
            if (!split_keys) {
                // whole rows to memory, 16 of the quarter's 32 by each warp: a thread per
                // row would touch 32 lines with every store
                (void)named_barrier_or(1 + 4 * i + (warp & 3), 64, false);
                constexpr int kRuns = DP / 8, kAtOnce = 32 / kRuns;
                const int64_t at = row * a.ldo + static_cast<int64_t>(head0 + head) * a.D;
                const uint32_t live_rows = __ballot_sync(0xffffffffu, live);
                const int run = lane % kRuns;
#pragma unroll
                for (int q = 0; q < 16 / kAtOnce; ++q) {
                    const int rq = 16 * half + q * kAtOnce + lane / kRuns;   // of the quarter's rows
                    const int64_t dst = __shfl_sync(0xffffffffu, at, rq);
                    const uint4 u = *reinterpret_cast<const uint4*>(stage + ((warp & 3) * 32 + rq) * (DP * 2) + ((run ^ (rq & 7)) << 4));
                    if (((live_rows >> rq) & 1u) && run * 8 < a.D) *reinterpret_cast<uint4*>(a.o + dst + run * 8) = u;
                }
            }
        }
    }

    // -------------------------------------------------------------- teardown
    tc_fence_before_sync();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) atomicOr(a.err, 1);
    if (warp == 0) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, F::kTmemCols);
    }
}

// Sum of the splits' partial results in split order: `parts` CTAs per tile, a
// thread per row, 8 columns at a time, the rows of a warp one after the other as
// they were written.
constexpr int kCombineThreads = kTileM;
template <bool F16>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const Args a, int parts) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int r = threadIdx.x;
    const int64_t tile = blockIdx.x / parts, item = tile / a.nt;
    const int i = static_cast<int>(tile % a.nt);
    const int hc = static_cast<int>(item % a.HC), block = static_cast<int>(item / a.HC);
    Item it;
    if (!find_item<1>(a, block, threadIdx.x & 31, it)) return;
    const int hk = hc / a.chunks, head0 = hk * a.G + (hc - hk * a.chunks) * a.gs;
    const int token = r / a.gs, head = r - token * a.gs, t = it.t0 + i * a.tok + token;
    if (token >= a.tok || t >= it.nq || head >= min(a.gs, (hk + 1) * a.G - head0)) return;
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + tile * a.splits * kTileM + r;
    float M = kNone, L = 0.0f;
    for (int s = 0; s < a.splits; ++s) M = fmaxf(M, ml[s * kTileM].x);
    for (int s = 0; s < a.splits; ++s) L += ml[s * kTileM].y * exp2_approx(ml[s * kTileM].x - M);
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const int64_t row = it.q0 + t;
    const int h = head0 + head;
    for (int run = blockIdx.x % parts; run < a.D / 8; run += parts) {
        const float4* part = reinterpret_cast<const float4*>(a.part) + (tile * a.splits * (a.D / 4) + 2 * run) * kTileM + r;
        float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s) {
            const float2 x = ml[s * kTileM];
            const float4 u = part[static_cast<int64_t>(s) * (a.D / 4) * kTileM];
            const float4 v = part[(static_cast<int64_t>(s) * (a.D / 4) + 1) * kTileM];
            const float f = exp2_approx(x.x - M);
            if (x.y != 0.0f) {   // a split that the row sees nothing of adds nothing
                sum[0] += u.x * f, sum[1] += u.y * f, sum[2] += u.z * f, sum[3] += u.w * f;
                sum[4] += v.x * f, sum[5] += v.y * f, sum[6] += v.z * f, sum[7] += v.w * f;
            }
        }
        *reinterpret_cast<uint4*>(a.o + row * a.ldo + static_cast<int64_t>(h) * a.D + 8 * run) =
            make_uint4(pack_x2<F16>(sum[0] * inv, sum[1] * inv), pack_x2<F16>(sum[2] * inv, sum[3] * inv),
                       pack_x2<F16>(sum[4] * inv, sum[5] * inv), pack_x2<F16>(sum[6] * inv, sum[7] * inv));
        if (run == 0 && a.lse != nullptr) a.lse[row * a.Hq + h] = L == 0.0f ? -CUDART_INF_F : M * kLn2 + logf(L);
    }
}

// ---------------------------------------------------------------- host

// Heads [rows, ld] as a [rows][heads][D] tensor; a box is 64 elements x
// `box_heads` heads x `box_rows` rows.
bool encode_heads(CUtensorMap* map, bool f16, const uint16_t* p, int64_t rows, int64_t ld, int heads, int D, int box_heads,
                  int box_rows) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode_tiled_fn()(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                             const_cast<uint16_t*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int64_t kMostPartial = 96 << 20;   // bytes of partial results: they stay in L2

struct Plan {
    int nt, gs, tok, chunks, HC, splits;
    int64_t blocks;   // token blocks, at most
    size_t off_part, off_ml, ws_bytes;
};

Plan plan_prompt(int64_t B, int64_t Tq, int64_t Tkv, int64_t Hq, int64_t Hkv, int64_t D, bool causal, int sm_count) {
    Plan p = {};
    const int64_t G = Hq / Hkv, avg_q = ceil_div(Tq, B), avg_k = Tkv / B;
    // fewest tiles for sequences of the average length; of equals, the most heads
    int64_t best = INT64_MAX;
    for (int64_t gs = G < 128 ? G : 128; gs >= 1; --gs) {
        const int64_t tok = kTileM / gs, tiles = ceil_div(avg_q, tok) * ceil_div(G, gs);
        if (tiles < best) {
            best = tiles;
            p.gs = static_cast<int>(gs);
            p.tok = static_cast<int>(tok);
        }
    }
    p.chunks = static_cast<int>(ceil_div(G, p.gs));
    p.HC = static_cast<int>(Hkv) * p.chunks;
    // One tile per CTA and two CTAs per SM where the second tile of a block would be
    // empty, where a tile sees few keys, so that one CTA's start and end run beside
    // the other's products, and where short blocks fit the GPU at once and their
    // latency counts.  Two tiles against the same keys otherwise, which read K and V
    // half as often.  27B-class heads, us, one tile / two: 32 prompts of 128 39 / 61,
    // 64 of 256 156 / 192, 16 of 512 89 / 99, 16 of 768 154 / 160, 16 of 1024 234 / 235;
    // 24 documents of up to 1023, not causal, 56 / 54; 8 of 256 new tokens after 1000
    // 63 / 61; one prompt of 512 11.1 / 12.4, of 1500 31 / 27, of 4096 143 / 134.
    const int64_t single = B * ceil_div(avg_q, p.tok) * p.HC;
    const int64_t seen = causal ? avg_k - avg_q / 2 : avg_k;   // keys of a row, on average
    p.nt = avg_q <= p.tok || 2 * seen < 5 * kTileN || (avg_k < 6 * kTileN && single <= 2 * sm_count) ? 1 : 2;
    p.blocks = Tq / (p.nt * p.tok) + B;
    if (p.blocks > Tq) p.blocks = Tq;
    // Split the keys where that costs less by this estimate (us): waves of blocks,
    // each a key tile at a time and 4.5 beside them; partial results written and
    // read at 8 TB/s, and a second launch.  A split keeps at least four key tiles.
    // From four waves on blocks of unequal length fill the GPU by themselves.
    // 27B-class heads, us, split / not: 256 new tokens against 16384 74 / 183, 512
    // 143 / 185, 1024 278 / 351, 2048 490 / 515; 8 x 128 against 4128 117 / 120.
    const int64_t items = B * ceil_div(avg_q, p.nt * p.tok) * p.HC, places = static_cast<int64_t>(sm_count) * (p.nt == 1 ? 2 : 1);
    const double tiles = static_cast<double>(avg_k) / kTileN, step = p.nt == 1 ? 1.25 : 1.45;
    int64_t splits = 1;
    if (items < 4 * places) {
        double least = 0.0;
        for (int64_t s = 1; s <= 32 && (s == 1 || 4 * s <= tiles); ++s) {
            if (s > 1 && items * s * p.nt * kTileM * D * 4 > kMostPartial) break;
            const double waves = static_cast<double>(ceil_div(items * s, places));
            const double joined = s == 1 ? 0.0 : 3.0 + static_cast<double>(items * s * p.nt * kTileM * D) * 8.0 / 8.0e6;
            const double cost = waves * (step * tiles / static_cast<double>(s) + 4.5) + joined;
            if (s == 1 || cost < least) {
                least = cost;
                splits = s;
            }
        }
    }
    p.splits = static_cast<int>(splits);
    size_t off = kWorkspaceErrBytes;
    p.off_part = p.off_ml = off;
    if (splits > 1) {
        p.off_part = off = workspace_data(sm_count);
        const int64_t rows = p.blocks * p.HC * p.nt * kTileM * splits;
        off += static_cast<size_t>(rows * D) * sizeof(float);
        p.off_ml = off;
        off += static_cast<size_t>(rows) * 2 * sizeof(float);
    }
    p.ws_bytes = off;
    return p;
}

template <int DP, bool F16, int NT>
cudaError_t launch_form(const Maps& maps, const Args& a, int64_t grid, cudaStream_t stream) {
    static OncePerDevice once;
    const cudaError_t limit = allow_smem(once, prompt_kernel<DP, F16, NT>, smem_bytes<DP, NT>());
    if (limit != cudaSuccess) return limit;
    return launch_after(prompt_kernel<DP, F16, NT>, dim3(static_cast<unsigned>(grid)), Form<NT>::kThreads,
                        smem_bytes<DP, NT>(), stream, maps, a);
}

template <int DP, bool F16>
cudaError_t launch_tiles(const Maps& maps, const Args& a, int64_t grid, cudaStream_t stream) {
    const cudaError_t e = a.nt == 1 ? launch_form<DP, F16, 1>(maps, a, grid, stream) : launch_form<DP, F16, 2>(maps, a, grid, stream);
    if (e != cudaSuccess || a.splits == 1) return e;
    // one CTA per 8 columns, fewer where the tiles alone are many
    const int64_t tiles = grid / a.splits * a.nt;
    const int parts = tiles * (a.D / 8) <= 4096 ? a.D / 8 : 4;
    return launch_after(combine_kernel<F16>, dim3(static_cast<unsigned>(tiles * parts)), kCombineThreads, 0, stream, a, parts);
}

}  // namespace

size_t prompt_ws_bytes(int64_t B, int64_t Tq, int64_t Tkv, int64_t Hq, int64_t Hkv, int64_t D, int sm_count) {
    const int sms = sm_count < 1 ? 1 : sm_count;
    const size_t all = plan_prompt(B, Tq, Tkv, Hq, Hkv, D, false, sms).ws_bytes, causal = plan_prompt(B, Tq, Tkv, Hq, Hkv, D, true, sms).ws_bytes;
    return all > causal ? all : causal;
}

cudaError_t launch_prompt(bool x_f16, const PromptArgs& pa, void* ws, int sm_count, cudaStream_t stream) {
    const Plan p = plan_prompt(pa.B, pa.Tq, pa.Tkv, pa.Hq, pa.Hkv, pa.D, pa.causal, sm_count);
    const int64_t grid = p.blocks * p.HC * p.splits;
    if (grid > INT32_MAX / 8) return cudaErrorInvalidValue;
    if (encode_tiled_fn() == nullptr) return cudaErrorNotSupported;
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    bool ok = encode_heads(&maps.q, x_f16, pa.q, pa.Tq, pa.ldq, pa.Hq, pa.D, p.gs, p.tok);
    if (pa.Tkv > 0) {   // without keys there is nothing to load
        ok = ok && encode_heads(&maps.k, x_f16, pa.k, pa.Tkv, pa.ldk, pa.Hkv, pa.D, 1, kTileN);
        ok = ok && encode_heads(&maps.v, x_f16, pa.v, pa.Tkv, pa.ldv, pa.Hkv, pa.D, 1, kTileN);
    } else {
        maps.k = maps.v = maps.q;
    }
    if (!ok) return cudaErrorInvalidValue;
    uint8_t* w = static_cast<uint8_t*>(ws);
    Args a = {};
    a.cu_q = pa.cu_q;
    a.cu_kv = pa.cu_kv;
    a.v = pa.v;
    a.o = pa.o;
    a.lse = pa.lse;
    a.part = reinterpret_cast<float*>(w + p.off_part);
    a.part_ml = reinterpret_cast<float*>(w + p.off_ml);
    a.err = reinterpret_cast<int*>(w);
    a.ldv = pa.ldv;
    a.ldo = pa.ldo;
    a.B = pa.B;
    a.Tq = pa.Tq;
    a.Tkv = pa.Tkv;
    a.Hq = pa.Hq;
    a.G = pa.Hq / pa.Hkv;
    a.D = pa.D;
    a.nt = p.nt;
    a.gs = p.gs;
    a.tok = p.tok;
    a.chunks = p.chunks;
    a.HC = p.HC;
    a.splits = p.splits;
    a.causal = pa.causal ? 1 : 0;
    // a scale of zero as the smallest number: the largest product stays below 2^-20, and
    // keys that are not seen stay at minus infinity
    a.scale2 = fmaxf(pa.scale * kLog2e, FLT_TRUE_MIN);
    if (pa.D > 64) return x_f16 ? launch_tiles<128, true>(maps, a, grid, stream) : launch_tiles<128, false>(maps, a, grid, stream);
    return x_f16 ? launch_tiles<64, true>(maps, a, grid, stream) : launch_tiles<64, false>(maps, a, grid, stream);
}

}  // namespace tern
