// Root-mean-square norm of rows with the residual's addition, 16-bit outputs or
// int8 codes with a scale per row.
//
// Mathematics.  s = x + r in fp32 (and S is s rounded once), y_k = s_k / sqrt(mean
// s^2 + eps) * (w_k + add).  A row's values stay in registers between the sum of
// squares and the outputs, so x and r are read once.  With codes, y is not
// rounded in between: a = max |y| / 127, q = rint(y * (127 / max |y|)).  Sums of
// squares are fp32 over at most 32 values a thread and then pairwise; rows whose
// squares leave fp32's range are summed again in double.
//
// What bounds it: DRAM for long prompts, launch and one chain load -> sum ->
// store for a few tokens.
//
// Measured: 8191 rows of 5120 in bf16 with the residual 50 us (6.7 TB/s), fp32 input and
// codes 61 us (6.2 TB/s), bf16 input and an fp32 stream 83 us (6.1 TB/s), 40 heads of 128 of
// 4095 tokens 15.1 us (5.5 TB/s; with a choice of type for every element, and twice the lanes
// to a row, instructions bounded it: 20.2), 16 rows 1.9 us a launch in a CUDA graph.
//
// Layout of the work: a thread holds NV runs of 8 elements.  Rows of up to 256
// elements are taken by 4 to 32 lanes, several rows to a warp, up to 1024 by a
// warp, longer ones by a CTA, whose warps meet once (twice with codes).

#include <float.h>

#include "tern_attn.cuh"
#include "tern_common.cuh"
#include "tern_internal.h"

namespace tern {
namespace {

constexpr int kRowThreads = 128;   // of a CTA whose warps have rows of their own

// Kinds of the residual stream.
constexpr int kResNone = 0, kRes16 = 1, kRes32 = 2;

struct Args {
    const void* x;
    const void* r;
    void* s;
    const uint16_t* w;
    uint16_t* y;
    int8_t* q;
    float* a;
    int64_t rows;              // tokens x heads
    int64_t ldx, ldr, lds, ldy;
    uint32_t H;
    int K;
    int x_f16, r_f16, y_f16;   // 16-bit types: fp16, else bf16
    float add, eps;
    float inverse;             // 1 / K
};

// (the type is the call's: one branch, not a choice for every element)
template <bool F16>
__device__ __forceinline__ void widen8_as(const uint4& u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_x2<F16>(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void widen8(const uint4& u, int f16, float (&v)[8]) {
    if (f16)
        widen8_as<true>(u, v);
    else
        widen8_as<false>(u, v);
}
__device__ __forceinline__ uint4 narrow8(const float (&v)[8], int f16) {
    if (f16)
        return make_uint4(pack_x2<true>(v[0], v[1]), pack_x2<true>(v[2], v[3]), pack_x2<true>(v[4], v[5]), pack_x2<true>(v[6], v[7]));
    return make_uint4(pack_x2<false>(v[0], v[1]), pack_x2<false>(v[2], v[3]), pack_x2<false>(v[4], v[5]), pack_x2<false>(v[6], v[7]));
}

// A run of 8 elements of 16 or 32 bits as it lies in memory.
template <bool WIDE>
struct Run {
    uint4 u[WIDE ? 2 : 1];
};
template <bool WIDE>
__device__ __forceinline__ Run<WIDE> load_run(const void* p, int64_t at) {
    Run<WIDE> r;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at * (WIDE ? 4 : 2));
    r.u[0] = src[0];
    if constexpr (WIDE) r.u[1] = src[1];
    return r;
}
template <bool WIDE>
__device__ __forceinline__ void values(const Run<WIDE>& r, int f16, float (&v)[8]) {
    if constexpr (WIDE) {
        const uint32_t w[8] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w, r.u[1].x, r.u[1].y, r.u[1].z, r.u[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
        widen8(r.u[0], f16, v);
    }
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Over the LANES lanes of a row (32: and over the CTA's warps, where CTA is set);
// every thread of the row gets the result.
template <int LANES, bool CTA, typename T, typename Op>
__device__ __forceinline__ T reduce(T v, T* meet, Op op) {
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, d));
    if constexpr (CTA) {
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) meet[threadIdx.x >> 5] = v;
        __syncthreads();
        v = meet[lane < warps ? lane : 0];
        // (a warp's place twice: sums count it once)
        if (lane >= warps) v = op.none();
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, d));
    }
    return v;
}
struct Sum {
    template <typename T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
    __device__ __forceinline__ float none() const { return 0.0f; }
};
struct Most {
    __device__ __forceinline__ float operator()(float a, float b) const { return max_nan(a, b); }
    __device__ __forceinline__ float none() const { return 0.0f; }
};

// CTAs of an SM, so that short rows' loads are many: as many as fit with spills of 48 bytes a
// thread at most (163800 rows of 128: 16.1 us at 58 registers a thread, 15.1 at 40).  CTAs of
// one row are held to 64 registers, whatever their size: their four-run form spills some 30
// bytes where there is no stream or all values have 16 bits, else 96 to 192.
template <bool X32, int RES, int LANES, int NV, bool CTA>
constexpr int kCtas = CTA || NV == 1 || LANES == 32 ? 1 : X32 || RES == kRes32 ? 8 : RES == kRes16 ? 10 : 12;

template <bool X32, int RES, bool I8, int LANES, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 1024 : kRowThreads, kCtas<X32, RES, LANES, NV, CTA>) norm_kernel(const Args a) {
    __shared__ float meet_sum[32], meet_max[32];
    __shared__ double meet_wide[32];
    grid_launch_dependents();
    grid_dependency_wait();
    const int threads = CTA ? blockDim.x : LANES;
    const int me = CTA ? threadIdx.x : threadIdx.x % LANES;
    constexpr int kGroups = CTA ? 1 : kRowThreads / LANES;
    const int64_t row = CTA ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kGroups + threadIdx.x / LANES;
    const bool real = CTA || row < a.rows;   // (the warp's other rows need its lanes)
    Run<X32> xr[NV];
    Run<RES == kRes32> rr[NV];
    uint4 wr[NV];
    int64_t tok = row;
    int head = 0;
    if (a.H > 1) {
        tok = (row >> 32) == 0 ? static_cast<uint32_t>(row) / a.H : row / a.H;
        head = static_cast<int>(row - tok * a.H);
    }
    const int64_t x0 = tok * a.ldx + (int64_t)head * a.K, r0 = tok * a.ldr + (int64_t)head * a.K;
    bool live[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int k = 8 * (me + i * threads);
        live[i] = k < a.K;
        if (!live[i] || !real) continue;
        xr[i] = load_run<X32>(a.x, x0 + k);
        if constexpr (RES != kResNone) rr[i] = load_run<RES == kRes32>(a.r, r0 + k);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (live[i] && a.w != nullptr) wr[i] = *reinterpret_cast<const uint4*>(a.w + 8 * (me + i * threads));
    const int64_t s0 = tok * a.lds + (int64_t)head * a.K;
    float v[NV][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (live[i] && real) {
            values<X32>(xr[i], a.x_f16, v[i]);
            if constexpr (RES != kResNone) {
                float r[8];
                values<RES == kRes32>(rr[i], a.r_f16, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += r[j];
            }
            if (a.s != nullptr) {
                const int64_t at = s0 + 8 * (me + i * threads);
                if constexpr (RES == kRes32) {
                    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.s) + at);
                    dst[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
                    dst[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
                } else {
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.s) + at) = narrow8(v[i], a.r_f16);
                }
            }
            uint64_t part = mul_x2(pair(v[i][0], v[i][1]), pair(v[i][0], v[i][1]));
#pragma unroll
            for (int j = 2; j < 8; j += 2) part = fma_x2(pair(v[i][j], v[i][j + 1]), pair(v[i][j], v[i][j + 1]), part);
            float even, odd;
            unpair(part, even, odd);
            ss += even + odd;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        }
    }
    ss = reduce<LANES, CTA>(ss, meet_sum, Sum());
    float scale = rsqrtf(fmaf(ss, a.inverse, a.eps));
    // Squares beyond fp32's range, or below it and not lost beside eps.  Uniform in
    // a row; the lanes of a warp's other rows take part.
    const bool wide = !(ss <= 1e37f) || (ss < 1e-25f && a.eps < 1e-25f);
    if (CTA ? wide : __any_sync(0xffffffffu, wide)) {
        double d = 0.0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) d += static_cast<double>(v[i][j]) * v[i][j];
        d = reduce<LANES, CTA>(d, meet_wide, Sum());
        // values times a power of two first: the scale may pass fp32's range
        const double inv = 1.0 / sqrt(d / a.K + a.eps);
        if (wide) {
            const double up = inv > 1e30 ? 0x1p100 : inv < 1e-30 ? 0x1p-100 : 1.0;
            scale = static_cast<float>(inv / up);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] *= static_cast<float>(up);
        }
    }
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!live[i] || !real) continue;
        float w[8];
        if (a.w != nullptr) {
            widen8(wr[i], a.y_f16, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] += a.add;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 1.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; j += 2)
            unpair(mul_x2(mul_x2(pair(v[i][j], v[i][j + 1]), pair(scale, scale)), pair(w[j], w[j + 1])), v[i][j], v[i][j + 1]);
        if constexpr (I8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) most = max_nan(most, fabsf(v[i][j]));
        } else {
            *reinterpret_cast<uint4*>(a.y + tok * a.ldy + (int64_t)head * a.K + 8 * (me + i * threads)) = narrow8(v[i], a.y_f16);
        }
    }
    if constexpr (I8) {
        most = reduce<LANES, CTA>(most, meet_max, Most());
        const bool bad = !(most <= FLT_MAX);
        // (below 127 / FLT_MAX the largest finite inverse keeps codes within the range)
        const float inv = most > 0.0f && !bad ? fminf(__fdiv_rn(127.0f, most), FLT_MAX) : 0.0f;
        if (real && me == 0) a.a[row] = bad ? __int_as_float(0x7fc00000) : __fdiv_rn(most, 127.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            // of 16 values the even ones lie first: the two threads that have them change halves
            uint32_t even = 0, odd = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = bad ? 0 : __float2int_rn(__fmul_rn(v[i][2 * j], inv));
                const int o = bad ? 0 : __float2int_rn(__fmul_rn(v[i][2 * j + 1], inv));
                even |= (static_cast<uint32_t>(e) & 0xFFu) << (8 * j);
                odd |= (static_cast<uint32_t>(o) & 0xFFu) << (8 * j);
            }
            const bool second = me & 1;
            const uint32_t other = __shfl_xor_sync(0xffffffffu, second ? even : odd, 1);
            if (live[i] && real)
                *reinterpret_cast<uint2*>(a.q + row * a.K + 8 * (me + i * threads)) =
                    second ? make_uint2(other, odd) : make_uint2(even, other);
        }
    }
}

template <bool X32, int RES, bool I8>
cudaError_t launch(const Args& a, cudaStream_t stream) {
    const int runs = a.K / 8;
    if (runs <= 128) {
        const int lanes = runs <= 4 ? 4 : runs <= 8 ? 8 : runs <= 16 ? 16 : 32;
        // two runs a lane where there are rows enough for all SMs: what a row costs besides
        // its elements is shared by fewer lanes (163800 rows of 128: 20.6 us with one run, 15.1
        // with two, 16.0 with four)
        const bool many = runs > 4 && runs <= 32 && a.rows * lanes >= (int64_t)device_sm_count() * 4096;
        const dim3 grid(static_cast<unsigned>(ceil_div(a.rows, kRowThreads / lanes * (many ? 2 : 1))));
        if (many) {
            if (lanes == 8) return launch_after(norm_kernel<X32, RES, I8, 4, 2, false>, grid, kRowThreads, 0, stream, a);
            if (lanes == 16) return launch_after(norm_kernel<X32, RES, I8, 8, 2, false>, grid, kRowThreads, 0, stream, a);
            return launch_after(norm_kernel<X32, RES, I8, 16, 2, false>, grid, kRowThreads, 0, stream, a);
        }
        if (lanes == 4) return launch_after(norm_kernel<X32, RES, I8, 4, 1, false>, grid, kRowThreads, 0, stream, a);
        if (lanes == 8) return launch_after(norm_kernel<X32, RES, I8, 8, 1, false>, grid, kRowThreads, 0, stream, a);
        if (lanes == 16) return launch_after(norm_kernel<X32, RES, I8, 16, 1, false>, grid, kRowThreads, 0, stream, a);
        if (runs <= 32) return launch_after(norm_kernel<X32, RES, I8, 32, 1, false>, grid, kRowThreads, 0, stream, a);
        if (runs <= 64) return launch_after(norm_kernel<X32, RES, I8, 32, 2, false>, grid, kRowThreads, 0, stream, a);
        return launch_after(norm_kernel<X32, RES, I8, 32, 4, false>, grid, kRowThreads, 0, stream, a);
    }
    const dim3 grid(static_cast<unsigned>(a.rows));
    // One run a thread for few rows, where the chain of one row is what counts; more of them,
    // in smaller CTAs, for many, so that an SM has rows in every phase (8191 rows of 5120 in
    // bf16 with the residual: 66 us with one run, 52 with two, 50 with four; fp32 input and
    // codes 78, 62, 79).
    const int few = runs <= 1024 ? 1 : runs <= 2048 ? 2 : 4;
    const int nv = a.rows < 4 * static_cast<int64_t>(device_sm_count()) ? few : X32 && runs <= 2048 ? 2 : 4;
    const unsigned threads = static_cast<unsigned>(round_up(ceil_div(runs, nv), 32));
    if (nv == 1) return launch_after(norm_kernel<X32, RES, I8, 32, 1, true>, grid, threads, 0, stream, a);
    if (nv == 2) return launch_after(norm_kernel<X32, RES, I8, 32, 2, true>, grid, threads, 0, stream, a);
    return launch_after(norm_kernel<X32, RES, I8, 32, 4, true>, grid, threads, 0, stream, a);
}

template <bool X32, int RES>
cudaError_t launch_out(const Args& a, cudaStream_t stream) {
    return a.q != nullptr ? launch<X32, RES, true>(a, stream) : launch<X32, RES, false>(a, stream);
}

template <bool X32>
cudaError_t launch_res(int kind, const Args& a, cudaStream_t stream) {
    if (kind == kRes16) return launch_out<X32, kRes16>(a, stream);
    if (kind == kRes32) return launch_out<X32, kRes32>(a, stream);
    return launch_out<X32, kResNone>(a, stream);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& n, cudaStream_t stream) {
    Args a = {};
    a.x = n.x;
    a.r = n.r;
    a.s = n.s;
    a.w = n.w;
    a.y = n.y;
    a.q = n.q;
    a.a = n.a;
    a.rows = n.T * n.H;
    a.ldx = n.ldx;
    a.ldr = n.ldr;
    a.lds = n.lds;
    a.ldy = n.ldy;
    a.H = static_cast<uint32_t>(n.H);
    a.K = static_cast<int>(n.K);
    a.x_f16 = n.x_type == kElemF16;
    a.r_f16 = n.res_type == kElemF16;
    a.y_f16 = n.y_f16;
    a.add = n.add;
    a.eps = n.eps;
    a.inverse = 1.0f / static_cast<float>(n.K);
    const int kind = n.r == nullptr ? kResNone : n.res_type == kElemF32 ? kRes32 : kRes16;
    return n.x_type == kElemF32 ? launch_res<true>(kind, a, stream) : launch_res<false>(kind, a, stream);
}

}  // namespace tern
