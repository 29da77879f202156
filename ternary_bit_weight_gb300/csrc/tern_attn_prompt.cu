// Attention over packed prompts.
//
// Plain form: one warp per (query row, head), each lane holding four of the
// head's elements; keys are taken one after the other with a running maximum
// and sum (the softmax's numerator and denominator are rescaled whenever the
// maximum grows), all in fp32.

#include <math_constants.h>

#include "tern_attn.cuh"
#include "tern_common.cuh"
#include "tern_internal.h"

namespace tern {
namespace {

constexpr int kWarps = 8;

template <bool F16>
__device__ __forceinline__ float4 load4(const uint16_t* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = unpack_x2<F16>(u.x), b = unpack_x2<F16>(u.y);
    return make_float4(a.x, a.y, b.x, b.y);
}

template <bool F16>
__global__ void __launch_bounds__(kWarps * 32) prompt_kernel(const PromptArgs a) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int lane = threadIdx.x & 31;
    const int64_t task = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int row = static_cast<int>(task / a.Hq), h = static_cast<int>(task % a.Hq);
    if (row >= a.Tq) return;
    int k0 = 0, k1 = -1;
    for (int b = 0; b < a.B; ++b) {
        const int q0 = min(max(a.cu_q[b], 0), a.Tq), q1 = min(max(a.cu_q[b + 1], 0), a.Tq);
        if (row < q0 || row >= q1) continue;
        k0 = min(max(a.cu_kv[b], 0), a.Tkv);
        k1 = max(k0, min(max(a.cu_kv[b + 1], 0), a.Tkv));
        if (a.causal) k1 = max(k0, min(k1, k0 + (k1 - k0) - (q1 - q0) + (row - q0) + 1));
        break;
    }
    if (k1 < 0) return;   // a row of no sequence
    const int g = h / (a.Hq / a.Hkv), d = lane * 4;
    const bool live = d < a.D;
    const float4 zero = make_float4(0, 0, 0, 0);
    const float4 q = live ? load4<F16>(a.q + (int64_t)row * a.ldq + h * a.D + d) : zero;
    float m = -CUDART_INF_F, l = 0.0f;
    float4 o = zero;
    for (int j = k0; j < k1; ++j) {
        const float4 k = live ? load4<F16>(a.k + (int64_t)j * a.ldk + g * a.D + d) : zero;
        const float4 v = live ? load4<F16>(a.v + (int64_t)j * a.ldv + g * a.D + d) : zero;
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
        *reinterpret_cast<uint2*>(a.o + (int64_t)row * a.ldo + h * a.D + d) =
            make_uint2(pack_x2<F16>(o.x * inv, o.y * inv), pack_x2<F16>(o.z * inv, o.w * inv));
    if (lane == 0 && a.lse != nullptr) a.lse[(int64_t)row * a.Hq + h] = l == 0.0f ? -CUDART_INF_F : m + logf(l);
}

}  // namespace

size_t prompt_ws_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int) { return kWorkspaceErrBytes; }

cudaError_t launch_prompt(bool x_f16, const PromptArgs& a, void*, int, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(ceil_div((int64_t)a.Tq * a.Hq, kWarps)));
    return x_f16 ? launch_after(prompt_kernel<true>, grid, kWarps * 32, 0, stream, a)
                 : launch_after(prompt_kernel<false>, grid, kWarps * 32, 0, stream, a);
}

}  // namespace tern
