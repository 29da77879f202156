// What the kernels of the cached tokens' attention weights share.
#pragma once

#include "tern_attn.cuh"
#include "tern_common.cuh"
#include "tern_internal.h"

namespace tern {
namespace weights {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.693147180559945309417f;

struct Args {
    const int32_t* cu_q;
    const int32_t* lens;
    const int32_t* known;
    const int32_t* table;
    const uint16_t* q;
    const float* lse;
    const uint8_t* k;
    const float* kscale;
    float* weight;
    int32_t* err;
    int64_t ldq, max_pages, num_pages;
    int64_t capacity;      // max_pages * page_size
    int B, Tq, Hq, Hkv, G, D;
    int shift;
    float scale, decay;
};

struct Sequence {
    int q0, nq, len;
};
__device__ __forceinline__ Sequence sequence_at(const Args& a, int b) {
    Sequence s;
    if (a.cu_q == nullptr) {
        s.q0 = b;
        s.nq = 1;
    } else {
        s.q0 = min(max(a.cu_q[b], 0), a.Tq);
        s.nq = max(0, min(max(a.cu_q[b + 1], 0), a.Tq) - s.q0);
    }
    s.len = static_cast<int>(min(static_cast<int64_t>(max(a.lens[b], 0)), a.capacity));
    return s;
}

// Tiles of `keys` keys of a sequence, over all its heads.
__device__ __forceinline__ int64_t tiles_of(const Args& a, const Sequence& s, int keys) {
    return s.nq == 0 ? 0 : static_cast<int64_t>((s.len + (keys - 1)) / keys) * a.Hkv;
}

// Whether keys come by TMA, 16 at a time: they lie in one page, and the (page, head)
// count fits a coordinate.
inline bool by_tma(const Args& a) { return a.shift >= 4 && a.num_pages > 0 && a.num_pages * a.Hkv <= INT32_MAX; }

// Whether the form for many rows takes the call, and that form.
bool rows_form(const Args& a);
cudaError_t launch_rows(bool x_f16, int kv, const Args& a, int sm_count, cudaStream_t stream);

}  // namespace weights
}  // namespace tern
