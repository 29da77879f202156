// Attention of single tokens over the paged cache.
//
// Plain form: one warp per (sequence, query head), each lane holding four of
// the head's elements; keys are taken one after the other with a running
// maximum and sum, all in fp32.

#include <math_constants.h>

#include "tern_attn.cuh"
#include "tern_common.cuh"
#include "tern_internal.h"

namespace tern {
namespace {

constexpr int kWarps = 8;

template <bool F16, int KV>
__device__ __forceinline__ float4 load4(const void* cache, int64_t cell, int D, int d, const float* factor) {
    if (KV == kKvX16) {
        const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(cache) + cell * D + d);
        const float2 a = unpack_x2<F16>(u.x), b = unpack_x2<F16>(u.y);
        return make_float4(a.x, a.y, b.x, b.y);
    }
    const uint32_t u = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(cache) + cell * D + d);
    const float f = factor[cell];
    if (KV == kKvE4m3) {
        const float2 a = __half22float2(e4m3x2_to_half2(u & 0xFFFFu)), b = __half22float2(e4m3x2_to_half2(u >> 16));
        return make_float4(a.x * f, a.y * f, b.x * f, b.y * f);
    }
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(static_cast<int8_t>((u >> (8 * i)) & 0xFFu)) * f;
    return make_float4(x[0], x[1], x[2], x[3]);
}

template <bool F16, int KV>
__global__ void __launch_bounds__(kWarps * 32) decode_kernel(const DecodeArgs a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int b = static_cast<int>(task / a.Hq), h = static_cast<int>(task % a.Hq);
    if (b >= a.B) return;
    const int64_t most = a.max_pages << a.cache.page_shift;
    const int len = static_cast<int>(min((int64_t)max(a.lens[b], 0), most));
    const int g = h / (a.Hq / a.Hkv), d = lane * 4;
    const bool live = d < a.D;
    const float4 zero = make_float4(0, 0, 0, 0);
    float4 q = zero;
    if (live) {
        const uint2 u = *reinterpret_cast<const uint2*>(a.q + (int64_t)b * a.ldq + h * a.D + d);
        const float2 x = unpack_x2<F16>(u.x), y = unpack_x2<F16>(u.y);
        q = make_float4(x.x, x.y, y.x, y.y);
    }
    float m = -CUDART_INF_F, l = 0.0f;
    float4 o = zero;
    for (int j = 0; j < len; ++j) {
        const int page = a.table[b * a.max_pages + (j >> a.cache.page_shift)];
        if (page < 0 || page >= a.cache.num_pages) continue;
        const int64_t cell = (((int64_t)page * a.Hkv + g) << a.cache.page_shift) + (j & ((1 << a.cache.page_shift) - 1));
        const float4 k = live ? load4<F16, KV>(a.cache.k, cell, a.D, d, a.cache.kscale) : zero;
        const float4 v = live ? load4<F16, KV>(a.cache.v, cell, a.D, d, a.cache.vscale) : zero;
        float s = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
        s *= a.scale;
        const float mn = fmaxf(m, s);
        const float keep = m == mn ? 1.0f : expf(m - mn), p = expf(s - mn);
        m = mn;
        l = l * keep + p;
        o = make_float4(o.x * keep + p * v.x, o.y * keep + p * v.y, o.z * keep + p * v.z, o.w * keep + p * v.w);
    }
    const float inv = l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : CUDART_NAN_F;
    if (live)
        *reinterpret_cast<uint2*>(a.o + (int64_t)b * a.ldo + h * a.D + d) =
            make_uint2(pack_x2<F16>(o.x * inv, o.y * inv), pack_x2<F16>(o.z * inv, o.w * inv));
    if (lane == 0 && a.lse != nullptr) a.lse[(int64_t)b * a.Hq + h] = l == 0.0f ? -CUDART_INF_F : m + logf(l);
}

template <bool F16>
cudaError_t launch(const DecodeArgs& a, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(ceil_div((int64_t)a.B * a.Hq, kWarps)));
    if (a.cache.kv == kKvX16) return launch_after(decode_kernel<F16, kKvX16>, grid, kWarps * 32, 0, stream, a);
    if (a.cache.kv == kKvE4m3) return launch_after(decode_kernel<F16, kKvE4m3>, grid, kWarps * 32, 0, stream, a);
    return launch_after(decode_kernel<F16, kKvI8>, grid, kWarps * 32, 0, stream, a);
}

}  // namespace

size_t decode_ws_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int) { return kWorkspaceErrBytes; }

cudaError_t launch_decode(bool x_f16, const DecodeArgs& a, void*, int, cudaStream_t stream) {
    return x_f16 ? launch<true>(a, stream) : launch<false>(a, stream);
}

}  // namespace tern
