// Rotary positions and the paged key/value cache (bandwidth-bound passes
// over token rows).
//
// Mathematics.  A rotation turns the pair (a, b) of a head by the angle
// p * f (position times the pair's frequency): (a cos - b sin, b cos + a sin).
// p * f reaches 10^5 radians and beyond, where an fp32 product is off by more
// than a 16-bit result's rounding; the angle is formed and reduced in
// double, in turns, and only the remainder goes to fp32.  A cached head of D
// values x is stored as codes round(x * (top / m)) with m = max |x| and the
// factor m / top, both divisions and the product IEEE fp32, so that any other
// implementation of the rule gets the same codes.
//
// Layout of the work: a head is one task of LANES lanes (4 for D <= 64, 8
// for D <= 128, 16 above; with 8 lanes for 48 heads of 64, half of them idle, 8191
// tokens took 23 us instead of 14), a lane owning two runs of 8 elements (16
// bytes each).  In the half layout the two runs are the partners of one another
// (elements 8j.. and rot/2 + 8j..), in the interleaved layout they are
// neighbours; either way lane j needs the angles of pairs 8j .. 8j+7 and a rotation stays inside a
// lane.  m is a butterfly over the task's lanes.  A warp serves one token, or
// a part of its heads when tokens are few: its lanes compute the token's angles
// once, keep them in registers for all heads, and walk the heads with two
// loads ahead (one where it quantises, too, which at 72 registers leaves 28 warps
// on an SM: 8191 tokens rotated and stored as int8 43 us, 6 less than with two).  A
// CTA is one warp, so that warps come and go one by one.  No barrier and no
// shared memory: with one CTA per token and the angles in shared memory, CTAs
// stood at barriers and start-up for most of their life (8191 tokens of 48 heads:
// 42 us, 4.8 TB/s, against 34 us, 5.9 TB/s).

#include <cuda_fp8.h>
#include <float.h>

#include "tern_attn.cuh"
#include "tern_common.cuh"
#include "tern_internal.h"

namespace tern {
namespace {

constexpr int kTokenThreads = 32;
constexpr int kTokenWarps = 8;     // per SM, at least, before a token's heads stay in one warp
constexpr int kReadThreads = 128;

struct TokenArgs {
    const int32_t* pos;
    const float* inv_freq;
    float amplitude;
    int interleaved;
    int D, rot;
    int Hq, Hk, Hv;            // heads rotated to qo, then keys, then values
    int64_t T;
    int parts;                 // warps per token, `per` heads each
    int per;
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    uint16_t* qo;
    uint16_t* ko;              // no cache: rotated keys
    int64_t ldq, ldk, ldv, ldqo, ldko;
    const int64_t* slots;
    int64_t capacity;          // num_pages * page_size
    int page_shift;
    uint8_t* kcache;
    uint8_t* vcache;
    float* kscale;
    float* vscale;
    int32_t* err;
};

// Rotation of pair angle `turns` (fraction of a full turn in double).
__device__ __forceinline__ float2 cos_sin(int32_t pos, float f, float amplitude) {
    const double turns = static_cast<double>(pos) * static_cast<double>(f) * 0.15915494309189533577;   // 1 / (2 pi)
    const float r = static_cast<float>(turns - rint(turns));   // [-1/2, 1/2]
    float s, c;
    sincospif(2.0f * r, &s, &c);
    return make_float2(c * amplitude, s * amplitude);
}

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_x2<F16>(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack_x2<F16>(x[0], x[1]), pack_x2<F16>(x[2], x[3]), pack_x2<F16>(x[4], x[5]),
                      pack_x2<F16>(x[6], x[7]));
}

// Largest magnitude of a head's values, 16 of them in each of its LANES lanes; a
// NaN among them stays.  Magnitudes are compared two by two as 16-bit values.
template <bool F16>
__device__ __forceinline__ uint32_t max_x2(uint32_t a, uint32_t b) {
    uint32_t d;
    if (F16)
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <int LANES, bool F16>
__device__ __forceinline__ float head_max(const uint4& ua, const uint4& ub) {
    const uint32_t sign = 0x7FFF7FFFu;
    uint32_t m = max_x2<F16>(max_x2<F16>(max_x2<F16>(ua.x & sign, ua.y & sign), max_x2<F16>(ua.z & sign, ua.w & sign)),
                             max_x2<F16>(max_x2<F16>(ub.x & sign, ub.y & sign), max_x2<F16>(ub.z & sign, ub.w & sign)));
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) m = max_x2<F16>(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float2 f = unpack_x2<F16>(m);
    return f.x != f.x ? f.x : f.y != f.y ? f.y : fmaxf(f.x, f.y);
}

// 8 codes of x * inv as two words.
template <int KV>
__device__ __forceinline__ uint2 encode8(const float* x, float inv) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __fmul_rn(x[4 * h + i], inv);
        if (KV == kKvE4m3) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
            w[h] = lo | (hi << 16);
        } else {
            w[h] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[h] |= (static_cast<uint32_t>(__float2int_rn(y[i])) & 0xFFu) << (8 * i);
        }
    }
    return make_uint2(w[0], w[1]);
}

__host__ __device__ constexpr bool coded(int kv) { return kv == kKvE4m3 || kv == kKvI8; }

// A lane's run of 8 elements: 16 bytes at `at`, or (SPLIT) 8 there and 8 at `at2`;
// likewise 8 codes.
template <bool SPLIT>
__device__ __forceinline__ uint4 load_run(const uint16_t* p, int at, int at2) {
    if constexpr (!SPLIT) return *reinterpret_cast<const uint4*>(p + at);
    const uint2 a = *reinterpret_cast<const uint2*>(p + at), b = *reinterpret_cast<const uint2*>(p + at2);
    return make_uint4(a.x, a.y, b.x, b.y);
}
template <bool SPLIT>
__device__ __forceinline__ void store_run(uint16_t* p, int at, int at2, const uint4& u) {
    if constexpr (!SPLIT) {
        *reinterpret_cast<uint4*>(p + at) = u;
    } else {
        *reinterpret_cast<uint2*>(p + at) = make_uint2(u.x, u.y);
        *reinterpret_cast<uint2*>(p + at2) = make_uint2(u.z, u.w);
    }
}
template <bool SPLIT>
__device__ __forceinline__ void store_codes(uint8_t* p, int at, int at2, const uint2& u) {
    if constexpr (!SPLIT) {
        *reinterpret_cast<uint2*>(p + at) = u;
    } else {
        *reinterpret_cast<uint32_t*>(p + at) = u.x;
        *reinterpret_cast<uint32_t*>(p + at2) = u.y;
    }
}

// One warp per token and part of its heads: rotate queries and keys, and
// (KV != kKvNone) store keys and values in the cache.  SPLIT: rot is an odd
// multiple of 8, so that one lane has four pairs that turn and four that do not,
// and runs are of 4 elements (8191 tokens, 48 heads of 80, half of each turned 28.5
// us, all of each 27.2).
template <int LANES, bool F16, int KV, bool SPLIT>
__global__ void __launch_bounds__(kTokenThreads, coded(KV) ? 28 : 0) token_kernel(const TokenArgs a) {
    constexpr int kSub = 32 / LANES;      // heads at a time
    constexpr int kOwn = 8 / kSub;        // pairs whose angle a lane computes
    constexpr int kAhead = coded(KV) ? 1 : 2;   // tasks loaded ahead
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t w = (int64_t)blockIdx.x * (kTokenThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = w / a.parts;
    if (t >= a.T) return;
    const int lane = threadIdx.x % LANES, sub = (threadIdx.x & 31) / LANES;
    const int first = static_cast<int>(w - t * a.parts) * a.per;
    const int tasks = min(a.Hq + a.Hk + a.Hv, first + a.per);
    const bool live = lane * 16 < a.D;
    const bool turned = live && lane * 16 < a.rot;
    const bool turned2 = SPLIT ? lane * 16 + 8 < a.rot : turned;   // pairs 4-7 of the lane
    // the lane's two runs of 8 elements (SPLIT: of 4 and 4)
    int ea = lane * 16, eb = ea + 8, ea2 = ea + 4, eb2 = eb + 4;
    if (!a.interleaved && turned) {
        ea = lane * 8;
        eb = a.rot / 2 + lane * 8;
        ea2 = ea + 4;
        eb2 = eb + 4;
        if (SPLIT && !turned2) {
            ea2 = lane * 16 + 8;
            eb2 = ea2 + 4;
        }
    }
    const uint16_t* qrow = a.q + t * a.ldq;
    const uint16_t* krow = a.k + t * a.ldk - (int64_t)a.Hq * a.D;
    const uint16_t* vrow = KV == kKvNone ? nullptr : a.v + t * a.ldv - (int64_t)(a.Hq + a.Hk) * a.D;
    auto load = [&](int h, uint4& ua, uint4& ub) {
        ua = ub = make_uint4(0, 0, 0, 0);
        if (h < tasks && live) {
            const uint16_t* src = (h < a.Hq ? qrow : h < a.Hq + a.Hk ? krow : vrow) + (int64_t)h * a.D;
            ua = load_run<SPLIT>(src, ea, ea2);
            ub = load_run<SPLIT>(src, eb, eb2);
        }
    };
    int h = first + sub;
    uint4 ua, ub, na, nb;
    load(h, ua, ub);
    if (kAhead == 2) load(h + kSub, na, nb);
    int64_t slot = -1;
    if (KV != kKvNone) {
        slot = a.slots[t];
        if (slot >= a.capacity) {
            if (first == 0 && (threadIdx.x & 31) == 0 && a.err != nullptr) atomicAdd(a.err, 1);
            slot = -1;
        }
    }
    // angles of pairs 8 lane .. 8 lane + 7, each computed by one of the lanes that need it
    float2 cs[8];
    if (a.rot > 0) {
        const int32_t p = a.pos[t];
        float2 own[kOwn];
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int pair = lane * 8 + sub * kOwn + i;
            own[i] = (SPLIT ? 2 * pair < a.rot : turned) ? cos_sin(p, a.inv_freq[pair], a.amplitude) : make_float2(0.0f, 0.0f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            cs[i].x = __shfl_sync(0xffffffffu, own[i % kOwn].x, (i / kOwn) * LANES + lane);
            cs[i].y = __shfl_sync(0xffffffffu, own[i % kOwn].y, (i / kOwn) * LANES + lane);
        }
    }
    const int64_t page = slot >> a.page_shift;
    const int64_t row = slot & ((int64_t(1) << a.page_shift) - 1);
    // the whole warp walks on while one of its tasks is left (for the butterfly)
    for (int h0 = first; h0 < tasks; h0 += kSub, h += kSub) {
        const bool mine = h < tasks && live;
        uint4 la, lb;
        load(h + kAhead * kSub, la, lb);
        const bool is_v = h >= a.Hq + a.Hk;
        if (turned && !is_v) {
            float x[16], y[16];
            unpack8<F16>(ua, x);
            unpack8<F16>(ub, x + 8);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // pair i of the lane: (x[i], x[8 + i]) or (x[2i], x[2i + 1])
                const float p0 = a.interleaved ? x[2 * i] : x[i], p1 = a.interleaved ? x[2 * i + 1] : x[8 + i];
                const float r0 = p0 * cs[i].x - p1 * cs[i].y, r1 = p1 * cs[i].x + p0 * cs[i].y;
                const bool turn = !SPLIT || i < 4 || turned2;
                if (a.interleaved) {
                    y[2 * i] = turn ? r0 : p0;
                    y[2 * i + 1] = turn ? r1 : p1;
                } else {
                    y[i] = turn ? r0 : p0;
                    y[8 + i] = turn ? r1 : p1;
                }
            }
            ua = pack8<F16>(y);
            ub = pack8<F16>(y + 8);
        }
        if (KV == kKvNone || h < a.Hq) {
            if (mine) {
                uint16_t* dst = h < a.Hq ? a.qo + t * a.ldqo + h * a.D : a.ko + t * a.ldko + (h - a.Hq) * a.D;
                store_run<SPLIT>(dst, ea, ea2, ua);
                store_run<SPLIT>(dst, eb, eb2, ub);
            }
        }
        if (KV != kKvNone && h0 + kSub > a.Hq) {   // some of the warp's tasks go to the cache
            const int g = is_v ? h - a.Hq - a.Hk : h - a.Hq;
            const int64_t cell = ((page * a.Hk + g) << a.page_shift) + row;
            const bool store = mine && h >= a.Hq && slot >= 0;
            uint8_t* cache = is_v ? a.vcache : a.kcache;
            if (KV == kKvX16) {
                if (store) {
                    uint16_t* dst = reinterpret_cast<uint16_t*>(cache) + cell * a.D;
                    store_run<SPLIT>(dst, ea, ea2, ua);
                    store_run<SPLIT>(dst, eb, eb2, ub);
                }
            } else {
                // codes from the values rounded to 16 bits, as a separate write sees them
                const float m = head_max<LANES, F16>(ua, ub);   // NaN or infinite with any such value
                if (store) {
                    const float top = KV == kKvE4m3 ? 448.0f : 127.0f;
                    const bool bad = !(m <= FLT_MAX);
                    float x[16];
                    unpack8<F16>(ua, x);
                    unpack8<F16>(ub, x + 8);
                    // m below top / FLT_MAX: the largest finite inverse keeps codes within the range
                    const float inv = m > 0.0f && !bad ? fminf(__fdiv_rn(top, m), FLT_MAX) : 0.0f;
                    if (bad) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = 0.0f;
                    }
                    uint8_t* dst = cache + cell * a.D;
                    store_codes<SPLIT>(dst, ea, ea2, encode8<KV>(x, inv));
                    store_codes<SPLIT>(dst, eb, eb2, encode8<KV>(x + 8, inv));
                    if (lane == 0) (is_v ? a.vscale : a.kscale)[cell] = bad ? __int_as_float(0x7fc00000) : __fdiv_rn(m, top);
                }
            }
        }
        if (kAhead == 2) {
            ua = na, ub = nb;
            na = la, nb = lb;
        } else {
            ua = la, ub = lb;
        }
    }
}

struct ReadArgs {
    int D, Hkv;
    int64_t T;
    const int64_t* slots;
    int64_t capacity;
    int page_shift;
    const uint8_t* kcache;
    const uint8_t* vcache;
    const float* kscale;
    const float* vscale;
    uint16_t* k;
    uint16_t* v;
    int64_t ldk, ldv;
};

// 16 codes -> 16 values of x_type, code * factor in fp32 rounded once.
template <bool F16, int KV>
__device__ __forceinline__ void decode16(const uint4& u, float factor, uint4& lo, uint4& hi) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    float x[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (KV == kKvE4m3) {
            const float2 p = __half22float2(e4m3x2_to_half2(w[i] & 0xFFFFu)), r = __half22float2(e4m3x2_to_half2(w[i] >> 16));
            x[4 * i] = p.x;
            x[4 * i + 1] = p.y;
            x[4 * i + 2] = r.x;
            x[4 * i + 3] = r.y;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * i + j] = static_cast<float>(static_cast<int8_t>((w[i] >> (8 * j)) & 0xFFu));
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], factor);
    lo = pack8<F16>(x);
    hi = pack8<F16>(x + 8);
}

// Eight lanes (four for D <= 64) per (token, head).  A lane has two runs of 8 elements, one in each
// half of the head, so that the lanes' stores of 16 bytes follow one another.  What
// bounds it: latency while the codes are in L2, DRAM beyond.  (8191 tokens of int8
// codes just written, 50 MB read and written, us: 7.0; 10.0 with two neighbouring
// runs, whose stores have half of every 32-byte sector each.  The passes above keep
// neighbours: bound by DRAM they gain nothing, and the start costs 1 us more.)
template <int LANES, bool F16, int KV>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const ReadArgs a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x % LANES;
    const int ea = lane * 8, eb = a.D / 2 + ea;
    if (eb >= a.D) return;
    const int64_t tasks = a.T * a.Hkv, step = (int64_t)gridDim.x * (kReadThreads / LANES);
    for (int64_t i = (int64_t)blockIdx.x * (kReadThreads / LANES) + threadIdx.x / LANES; i < tasks; i += step) {
        const int64_t t = ((i | a.Hkv) >> 32) == 0 ? static_cast<uint32_t>(i) / static_cast<uint32_t>(a.Hkv) : i / a.Hkv;
        const int g = static_cast<int>(i - t * a.Hkv);
        const int64_t slot = a.slots[t];
        uint4 k0 = make_uint4(0, 0, 0, 0), k1 = k0, v0 = k0, v1 = k0;
        if (slot >= 0 && slot < a.capacity) {
            const int64_t cell = (((slot >> a.page_shift) * a.Hkv + g) << a.page_shift) +
                                 (slot & ((int64_t(1) << a.page_shift) - 1));
            if (KV == kKvX16) {
                const uint16_t* ks = reinterpret_cast<const uint16_t*>(a.kcache) + cell * a.D;
                const uint16_t* vs = reinterpret_cast<const uint16_t*>(a.vcache) + cell * a.D;
                k0 = *reinterpret_cast<const uint4*>(ks + ea), k1 = *reinterpret_cast<const uint4*>(ks + eb);
                v0 = *reinterpret_cast<const uint4*>(vs + ea), v1 = *reinterpret_cast<const uint4*>(vs + eb);
            } else {
                const uint8_t* ks = a.kcache + cell * a.D;
                const uint8_t* vs = a.vcache + cell * a.D;
                const uint2 ka = *reinterpret_cast<const uint2*>(ks + ea), kb = *reinterpret_cast<const uint2*>(ks + eb);
                const uint2 va = *reinterpret_cast<const uint2*>(vs + ea), vb = *reinterpret_cast<const uint2*>(vs + eb);
                const float fk = a.kscale[cell], fv = a.vscale[cell];
                decode16<F16, KV>(make_uint4(ka.x, ka.y, kb.x, kb.y), fk, k0, k1);
                decode16<F16, KV>(make_uint4(va.x, va.y, vb.x, vb.y), fv, v0, v1);
            }
        }
        uint16_t* kd = a.k + t * a.ldk + g * a.D;
        uint16_t* vd = a.v + t * a.ldv + g * a.D;
        *reinterpret_cast<uint4*>(kd + ea) = k0, *reinterpret_cast<uint4*>(kd + eb) = k1;
        *reinterpret_cast<uint4*>(vd + ea) = v0, *reinterpret_cast<uint4*>(vd + eb) = v1;
    }
}

template <int LANES, bool F16, bool SPLIT>
cudaError_t launch_runs(int kv, TokenArgs a, int64_t T, cudaStream_t stream) {
    constexpr int kSub = 32 / LANES;
    const int64_t tasks = a.Hq + a.Hk + a.Hv, steps = ceil_div(tasks, kSub);
    // a warp walks all heads of a token, unless the tokens are too few to fill the SMs
    int64_t parts = ceil_div((int64_t)device_sm_count() * kTokenWarps, T);
    if (parts > steps) parts = steps;
    if (parts < 1) parts = 1;
    a.T = T;
    a.per = static_cast<int>(ceil_div(steps, parts)) * kSub;
    a.parts = static_cast<int>(ceil_div(tasks, a.per));
    const dim3 grid(static_cast<unsigned>(ceil_div(T * a.parts, kTokenThreads / 32)));
    if constexpr (LANES <= 8) {
        if (kv == kKvX16) return launch_after(token_kernel<LANES, F16, kKvX16, SPLIT>, grid, kTokenThreads, 0, stream, a);
        if (kv == kKvE4m3) return launch_after(token_kernel<LANES, F16, kKvE4m3, SPLIT>, grid, kTokenThreads, 0, stream, a);
        if (kv == kKvI8) return launch_after(token_kernel<LANES, F16, kKvI8, SPLIT>, grid, kTokenThreads, 0, stream, a);
    }
    return launch_after(token_kernel<LANES, F16, kKvNone, SPLIT>, grid, kTokenThreads, 0, stream, a);
}

template <int LANES, bool F16>
cudaError_t launch_token(int kv, const TokenArgs& a, int64_t T, cudaStream_t stream) {
    return a.rot % 16 == 0 ? launch_runs<LANES, F16, false>(kv, a, T, stream) : launch_runs<LANES, F16, true>(kv, a, T, stream);
}

TokenArgs token_args(const RopeArgs& r) {
    TokenArgs a = {};
    a.pos = r.pos;
    a.inv_freq = r.inv_freq;
    a.amplitude = r.amplitude;
    a.interleaved = r.interleaved ? 1 : 0;
    a.D = r.D;
    a.rot = r.rot;
    a.Hq = r.Hq;
    a.Hk = r.Hk;
    a.q = r.q;
    a.ldq = r.ldq;
    a.qo = r.qo;
    a.ldqo = r.ldqo;
    a.k = r.k;
    a.ldk = r.ldk;
    a.ko = r.ko;
    a.ldko = r.ldko;
    return a;
}

}  // namespace

cudaError_t launch_rope(bool x_f16, int64_t T, const RopeArgs& r, cudaStream_t stream) {
    const TokenArgs a = token_args(r);
    if (r.D <= 64)
        return x_f16 ? launch_token<4, true>(kKvNone, a, T, stream) : launch_token<4, false>(kKvNone, a, T, stream);
    if (r.D <= 128)
        return x_f16 ? launch_token<8, true>(kKvNone, a, T, stream) : launch_token<8, false>(kKvNone, a, T, stream);
    return x_f16 ? launch_token<16, true>(kKvNone, a, T, stream) : launch_token<16, false>(kKvNone, a, T, stream);
}

cudaError_t launch_kv_write(bool x_f16, int64_t T, const RopeArgs& r, const uint16_t* v, int64_t ldv,
                            const int64_t* slots, const KvCache& c, int32_t* err, cudaStream_t stream) {
    TokenArgs a = token_args(r);
    a.Hv = r.Hk;
    a.v = v;
    a.ldv = ldv;
    a.slots = slots;
    a.capacity = c.num_pages << c.page_shift;
    a.page_shift = c.page_shift;
    a.kcache = static_cast<uint8_t*>(const_cast<void*>(c.k));
    a.vcache = static_cast<uint8_t*>(const_cast<void*>(c.v));
    a.kscale = const_cast<float*>(c.kscale);
    a.vscale = const_cast<float*>(c.vscale);
    a.err = err;
    if (r.D <= 64) return x_f16 ? launch_token<4, true>(c.kv, a, T, stream) : launch_token<4, false>(c.kv, a, T, stream);
    return x_f16 ? launch_token<8, true>(c.kv, a, T, stream) : launch_token<8, false>(c.kv, a, T, stream);
}

template <int LANES, bool F16>
static cudaError_t launch_read_by(const ReadArgs& a, int kv, cudaStream_t stream) {
    const int64_t blocks = ceil_div(a.T * a.Hkv, kReadThreads / LANES);
    const dim3 grid(static_cast<unsigned>(blocks < (1 << 30) ? blocks : (1 << 30)));
    if (kv == kKvX16) return launch_after(kv_read_kernel<LANES, F16, kKvX16>, grid, kReadThreads, 0, stream, a);
    if (kv == kKvE4m3) return launch_after(kv_read_kernel<LANES, F16, kKvE4m3>, grid, kReadThreads, 0, stream, a);
    return launch_after(kv_read_kernel<LANES, F16, kKvI8>, grid, kReadThreads, 0, stream, a);
}

template <bool F16>
static cudaError_t launch_read(const ReadArgs& a, int kv, cudaStream_t stream) {
    return a.D <= 64 ? launch_read_by<4, F16>(a, kv, stream) : launch_read_by<8, F16>(a, kv, stream);
}

cudaError_t launch_kv_read(bool x_f16, int64_t T, int Hkv, int D, const int64_t* slots, const KvCache& c, uint16_t* k,
                           int64_t ldk, uint16_t* v, int64_t ldv, cudaStream_t stream) {
    const ReadArgs a = {D,   Hkv, T, slots, c.num_pages << c.page_shift, c.page_shift, static_cast<const uint8_t*>(c.k),
                        static_cast<const uint8_t*>(c.v), c.kscale, c.vscale, k, v, ldk, ldv};
    return x_f16 ? launch_read<true>(a, c.kv, stream) : launch_read<false>(a, c.kv, stream);
}

}  // namespace tern
