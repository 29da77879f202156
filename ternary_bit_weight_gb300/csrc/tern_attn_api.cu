// Host entry points of the attention side (rotary positions, paged cache,
// attention; declared in include/tern.h): argument checks and launches.
// Nothing here allocates memory or keeps state between calls.

#include <math.h>

#include "tern.h"
#include "tern_common.cuh"
#include "tern_internal.h"

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxHeads = 4096;
constexpr int64_t kMaxHeadDim = 128;       // cache and attention
constexpr int64_t kMaxRopeDim = 256;
constexpr int64_t kMaxPageSize = 32768;
constexpr int64_t kMaxMoves = int64_t(1) << 25;   // (sequence, head) pairs of one compaction

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }
inline tern_status from_cuda(cudaError_t e) { return e == cudaSuccess ? TERN_OK : TERN_ERR_CUDA; }
inline bool valid_x_type(int x_type) { return x_type == TERN_X_BF16 || x_type == TERN_X_F16; }
inline bool valid_heads(int64_t H) { return H >= 1 && H <= kMaxHeads; }
inline bool valid_scale(float s) { return s >= 0.0f && isfinite(s); }
inline bool valid_dim(int64_t D, int64_t most) { return D >= 16 && D <= most && D % 16 == 0; }

// A [rows, ld] buffer of H heads of dimension D.
tern_status check_rows(const void* p, int64_t ld, int64_t H, int64_t D) {
    if (p == nullptr) return TERN_ERR_NULL;
    if (ld < H * D || ld > (int64_t(1) << 40)) return TERN_ERR_SHAPE;
    if (!aligned(p, 16) || ld % 8 != 0) return TERN_ERR_ALIGN;
    return TERN_OK;
}

#define TERN_TRY(expr)                              \
    do {                                            \
        const tern_status tern_try_status = (expr); \
        if (tern_try_status != TERN_OK) return tern_try_status; \
    } while (0)

tern_status check_rotation(int layout, int64_t rot_dim, int64_t D) {
    if (layout != TERN_ROPE_HALF && layout != TERN_ROPE_INTERLEAVED) return TERN_ERR_SHAPE;
    if (rot_dim < 0 || rot_dim > D || (rot_dim % 16 != 0 && 2 * rot_dim != D)) return TERN_ERR_SHAPE;
    return TERN_OK;
}

tern_status check_angles(const int32_t* d_pos, const float* d_inv_freq, int64_t rot_dim) {
    if (rot_dim == 0) return TERN_OK;
    if (d_pos == nullptr || d_inv_freq == nullptr) return TERN_ERR_NULL;
    if (!aligned(d_pos, 4) || !aligned(d_inv_freq, 4)) return TERN_ERR_ALIGN;
    return TERN_OK;
}

// Shape of a cache; *shift = log2(page_size).
tern_status check_pages(int kv_type, int64_t Hkv, int64_t D, int64_t num_pages, int64_t page_size, int* shift) {
    if (kv_type != TERN_KV_X16 && kv_type != TERN_KV_E4M3 && kv_type != TERN_KV_I8) return TERN_ERR_SHAPE;
    if (!valid_heads(Hkv) || !valid_dim(D, kMaxHeadDim)) return TERN_ERR_SHAPE;
    if (page_size < 1 || page_size > kMaxPageSize || (page_size & (page_size - 1)) != 0) return TERN_ERR_SHAPE;
    if (num_pages < 0 || num_pages > INT32_MAX) return TERN_ERR_SHAPE;
    *shift = 0;
    while ((int64_t(1) << *shift) < page_size) ++*shift;
    return TERN_OK;
}

tern_status check_cache(int kv_type, const void* k, const void* v, const float* kscale, const float* vscale) {
    if (k == nullptr || v == nullptr) return TERN_ERR_NULL;
    if (kv_type != TERN_KV_X16 && (kscale == nullptr || vscale == nullptr)) return TERN_ERR_NULL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(kscale, 4) || !aligned(vscale, 4)) return TERN_ERR_ALIGN;
    return TERN_OK;
}

const uint16_t* u16(const void* p) { return static_cast<const uint16_t*>(p); }

}  // namespace

extern "C" {

tern_status tern_rope_freqs(int64_t rot_dim, double base, int scaling, double factor, double trained_len,
                            double turns_low, double turns_high, float* h_inv_freq, float* h_amplitude) {
    if (rot_dim <= 0 || rot_dim % 2 != 0 || rot_dim > kMaxRopeDim) return TERN_ERR_SHAPE;
    if (!(base > 0.0) || !isfinite(base) || !(factor > 0.0) || !isfinite(factor)) return TERN_ERR_SHAPE;
    if (scaling < TERN_ROPE_SCALE_NONE || scaling > TERN_ROPE_SCALE_PARTS) return TERN_ERR_SHAPE;
    if (scaling == TERN_ROPE_SCALE_BASE && rot_dim <= 2) return TERN_ERR_SHAPE;
    if (scaling == TERN_ROPE_SCALE_PARTS && !(trained_len > 0.0 && turns_high > turns_low)) return TERN_ERR_SHAPE;
    if (h_inv_freq == nullptr || h_amplitude == nullptr) return TERN_ERR_NULL;
    const double r = static_cast<double>(rot_dim);
    if (scaling == TERN_ROPE_SCALE_BASE) base *= pow(factor, r / (r - 2.0));
    for (int64_t i = 0; i < rot_dim / 2; ++i) {
        double f = pow(base, -2.0 * static_cast<double>(i) / r);
        if (scaling == TERN_ROPE_SCALE_LINEAR) f /= factor;
        if (scaling == TERN_ROPE_SCALE_PARTS) {
            const double turns = trained_len * f / (2.0 * 3.14159265358979323846);
            double keep = (turns - turns_low) / (turns_high - turns_low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f *= keep + (1.0 - keep) / factor;
        }
        h_inv_freq[i] = static_cast<float>(f);
    }
    *h_amplitude = scaling == TERN_ROPE_SCALE_PARTS && factor > 1.0 ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.0f;
    return TERN_OK;
}

tern_status tern_rope(int x_type, int layout, int64_t T, int64_t D, int64_t rot_dim, const int32_t* d_pos,
                      const float* d_inv_freq, float amplitude, int64_t Hq, const void* d_Q, int64_t ldq,
                      void* d_Qo, int64_t ldqo, int64_t Hk, const void* d_K, int64_t ldk, void* d_Ko,
                      int64_t ldko, void* stream) {
    if (!valid_x_type(x_type) || T < 0 || T > kMaxRows) return TERN_ERR_SHAPE;
    if (!valid_dim(D, kMaxRopeDim) || !valid_heads(Hq) || (Hk != 0 && !valid_heads(Hk))) return TERN_ERR_SHAPE;
    TERN_TRY(check_rotation(layout, rot_dim, D));
    if (T == 0) return TERN_OK;
    TERN_TRY(check_angles(d_pos, d_inv_freq, rot_dim));
    TERN_TRY(check_rows(d_Q, ldq, Hq, D));
    TERN_TRY(check_rows(d_Qo, ldqo, Hq, D));
    if (Hk != 0) {
        TERN_TRY(check_rows(d_K, ldk, Hk, D));
        TERN_TRY(check_rows(d_Ko, ldko, Hk, D));
    }
    tern::RopeArgs r = {};
    r.interleaved = layout == TERN_ROPE_INTERLEAVED;
    r.D = static_cast<int>(D);
    r.rot = static_cast<int>(rot_dim);
    r.pos = d_pos;
    r.inv_freq = d_inv_freq;
    r.amplitude = amplitude;
    r.Hq = static_cast<int>(Hq);
    r.Hk = static_cast<int>(Hk);
    r.q = u16(d_Q);
    r.ldq = ldq;
    r.qo = static_cast<uint16_t*>(d_Qo);
    r.ldqo = ldqo;
    r.k = u16(d_K);
    r.ldk = ldk;
    r.ko = static_cast<uint16_t*>(d_Ko);
    r.ldko = ldko;
    return from_cuda(tern::launch_rope(x_type == TERN_X_F16, T, r, as_stream(stream)));
}

tern_status tern_rope_kv_write(int x_type, int kv_type, int layout, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                               int64_t rot_dim, const int32_t* d_pos, const float* d_inv_freq, float amplitude,
                               const void* d_Q, int64_t ldq, void* d_Qo, int64_t ldqo, const void* d_K, int64_t ldk,
                               const void* d_V, int64_t ldv, const int64_t* d_slots, int64_t num_pages,
                               int64_t page_size, void* d_kcache, void* d_vcache, float* d_kscale, float* d_vscale,
                               int32_t* d_err, void* stream) {
    int shift = 0;
    if (!valid_x_type(x_type) || T < 0 || T > kMaxRows || Hq < 0 || Hq > kMaxHeads) return TERN_ERR_SHAPE;
    TERN_TRY(check_pages(kv_type, Hkv, D, num_pages, page_size, &shift));
    TERN_TRY(check_rotation(layout, rot_dim, D));
    if (T == 0) return TERN_OK;
    TERN_TRY(check_angles(d_pos, d_inv_freq, rot_dim));
    if (Hq != 0) {
        TERN_TRY(check_rows(d_Q, ldq, Hq, D));
        TERN_TRY(check_rows(d_Qo, ldqo, Hq, D));
    }
    TERN_TRY(check_rows(d_K, ldk, Hkv, D));
    TERN_TRY(check_rows(d_V, ldv, Hkv, D));
    if (d_slots == nullptr) return TERN_ERR_NULL;
    if (!aligned(d_slots, 8) || (d_err != nullptr && !aligned(d_err, 4))) return TERN_ERR_ALIGN;
    TERN_TRY(check_cache(kv_type, d_kcache, d_vcache, d_kscale, d_vscale));
    tern::RopeArgs r = {};
    r.interleaved = layout == TERN_ROPE_INTERLEAVED;
    r.D = static_cast<int>(D);
    r.rot = static_cast<int>(rot_dim);
    r.pos = d_pos;
    r.inv_freq = d_inv_freq;
    r.amplitude = amplitude;
    r.Hq = static_cast<int>(Hq);
    r.Hk = static_cast<int>(Hkv);
    r.q = u16(d_Q);
    r.ldq = ldq;
    r.qo = static_cast<uint16_t*>(d_Qo);
    r.ldqo = ldqo;
    r.k = u16(d_K);
    r.ldk = ldk;
    const tern::KvCache c = {kv_type, num_pages, shift, d_kcache, d_vcache, d_kscale, d_vscale};
    return from_cuda(tern::launch_kv_write(x_type == TERN_X_F16, T, r, u16(d_V), ldv, d_slots, c, d_err,
                                           as_stream(stream)));
}

tern_status tern_kv_write(int x_type, int kv_type, int64_t T, int64_t Hkv, int64_t D, const void* d_K, int64_t ldk,
                          const void* d_V, int64_t ldv, const int64_t* d_slots, int64_t num_pages, int64_t page_size,
                          void* d_kcache, void* d_vcache, float* d_kscale, float* d_vscale, int32_t* d_err,
                          void* stream) {
    return tern_rope_kv_write(x_type, kv_type, TERN_ROPE_HALF, T, 0, Hkv, D, 0, nullptr, nullptr, 1.0f, nullptr, 0,
                              nullptr, 0, d_K, ldk, d_V, ldv, d_slots, num_pages, page_size, d_kcache, d_vcache,
                              d_kscale, d_vscale, d_err, stream);
}

tern_status tern_kv_read(int x_type, int kv_type, int64_t T, int64_t Hkv, int64_t D, const int64_t* d_slots,
                         int64_t num_pages, int64_t page_size, const void* d_kcache, const void* d_vcache,
                         const float* d_kscale, const float* d_vscale, void* d_K, int64_t ldk, void* d_V, int64_t ldv,
                         void* stream) {
    int shift = 0;
    if (!valid_x_type(x_type) || T < 0 || T > kMaxRows) return TERN_ERR_SHAPE;
    TERN_TRY(check_pages(kv_type, Hkv, D, num_pages, page_size, &shift));
    if (T == 0) return TERN_OK;
    TERN_TRY(check_rows(d_K, ldk, Hkv, D));
    TERN_TRY(check_rows(d_V, ldv, Hkv, D));
    if (d_slots == nullptr) return TERN_ERR_NULL;
    if (!aligned(d_slots, 8)) return TERN_ERR_ALIGN;
    TERN_TRY(check_cache(kv_type, d_kcache, d_vcache, d_kscale, d_vscale));
    const tern::KvCache c = {kv_type, num_pages, shift, d_kcache, d_vcache, d_kscale, d_vscale};
    return from_cuda(tern::launch_kv_read(x_type == TERN_X_F16, T, static_cast<int>(Hkv), static_cast<int>(D), d_slots,
                                          c, static_cast<uint16_t*>(d_K), ldk, static_cast<uint16_t*>(d_V), ldv,
                                          as_stream(stream)));
}

size_t tern_attn_prompt_workspace_bytes(int64_t B, int64_t Tq, int64_t Tkv, int64_t Hq, int64_t Hkv, int64_t D) {
    if (B <= 0 || B > kMaxRows || Tq <= 0 || Tq > kMaxRows || Tkv < 0 || Tkv > kMaxRows || !valid_heads(Hkv) ||
        !valid_heads(Hq) || Hq % Hkv != 0 || !valid_dim(D, kMaxHeadDim))
        return 0;
    return tern::prompt_ws_bytes(B, Tq, Tkv, Hq, Hkv, D, tern::device_sm_count());
}

tern_status tern_attn_prompt(int x_type, int64_t B, const int32_t* d_cu_q, const int32_t* d_cu_kv, int64_t Tq,
                             int64_t Tkv, int64_t Hq, int64_t Hkv, int64_t D, int causal, float scale, const void* d_Q,
                             int64_t ldq, const void* d_K, int64_t ldk, const void* d_V, int64_t ldv, void* d_O,
                             int64_t ldo, float* d_lse, void* d_ws, size_t ws_bytes, void* stream) {
    if (!valid_x_type(x_type) || B < 0 || B > kMaxRows || Tq < 0 || Tq > kMaxRows || Tkv < 0 || Tkv > kMaxRows)
        return TERN_ERR_SHAPE;
    if (!valid_heads(Hkv) || !valid_heads(Hq) || Hq % Hkv != 0 || !valid_dim(D, kMaxHeadDim)) return TERN_ERR_SHAPE;
    if (!valid_scale(scale)) return TERN_ERR_SHAPE;
    if (B == 0 || Tq == 0) return TERN_OK;
    if (d_cu_q == nullptr || d_cu_kv == nullptr) return TERN_ERR_NULL;
    if (!aligned(d_cu_q, 4) || !aligned(d_cu_kv, 4) || !aligned(d_lse, 4)) return TERN_ERR_ALIGN;
    TERN_TRY(check_rows(d_Q, ldq, Hq, D));
    if (Tkv > 0) {
        TERN_TRY(check_rows(d_K, ldk, Hkv, D));
        TERN_TRY(check_rows(d_V, ldv, Hkv, D));
    }
    TERN_TRY(check_rows(d_O, ldo, Hq, D));
    const int sms = tern::device_sm_count();
    if (sms <= 0) return TERN_ERR_UNSUPPORTED;
    if (d_ws == nullptr) return TERN_ERR_NULL;
    if (!aligned(d_ws, 256)) return TERN_ERR_ALIGN;
    if (ws_bytes < tern::prompt_ws_bytes(B, Tq, Tkv, Hq, Hkv, D, sms)) return TERN_ERR_SIZE;
    tern::PromptArgs a = {};
    a.B = static_cast<int>(B);
    a.cu_q = d_cu_q;
    a.cu_kv = d_cu_kv;
    a.Tq = static_cast<int>(Tq);
    a.Tkv = static_cast<int>(Tkv);
    a.Hq = static_cast<int>(Hq);
    a.Hkv = static_cast<int>(Hkv);
    a.D = static_cast<int>(D);
    a.causal = causal != 0;
    a.scale = scale;
    a.q = u16(d_Q);
    a.ldq = ldq;
    a.k = u16(d_K);
    a.ldk = ldk;
    a.v = u16(d_V);
    a.ldv = ldv;
    a.o = static_cast<uint16_t*>(d_O);
    a.ldo = ldo;
    a.lse = d_lse;
    return from_cuda(tern::launch_prompt(x_type == TERN_X_F16, a, d_ws, sms, as_stream(stream)));
}

size_t tern_attn_decode_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_len) {
    if (B <= 0 || B > kMaxRows || max_len < 0 || max_len > INT32_MAX || !valid_heads(Hkv) || !valid_heads(Hq) ||
        Hq % Hkv != 0 || !valid_dim(D, kMaxHeadDim))
        return 0;
    return tern::decode_ws_bytes(B, Hq, Hkv, D, max_len, tern::device_sm_count());
}

tern_status tern_attn_decode(int x_type, int kv_type, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, float scale,
                             const void* d_Q, int64_t ldq, int64_t num_pages, int64_t page_size, const void* d_kcache,
                             const void* d_vcache, const float* d_kscale, const float* d_vscale,
                             const int32_t* d_page_table, int64_t max_pages, const int32_t* d_lens, void* d_O,
                             int64_t ldo, float* d_lse, void* d_ws, size_t ws_bytes, void* stream) {
    int shift = 0;
    if (!valid_x_type(x_type) || B < 0 || B > kMaxRows) return TERN_ERR_SHAPE;
    TERN_TRY(check_pages(kv_type, Hkv, D, num_pages, page_size, &shift));
    if (!valid_heads(Hq) || Hq % Hkv != 0 || !valid_scale(scale)) return TERN_ERR_SHAPE;
    if (max_pages < 0 || max_pages > (INT32_MAX >> shift)) return TERN_ERR_SHAPE;
    if (B == 0) return TERN_OK;
    if (d_lens == nullptr || (max_pages > 0 && d_page_table == nullptr)) return TERN_ERR_NULL;
    if (!aligned(d_lens, 4) || !aligned(d_page_table, 4) || !aligned(d_lse, 4)) return TERN_ERR_ALIGN;
    TERN_TRY(check_rows(d_Q, ldq, Hq, D));
    TERN_TRY(check_rows(d_O, ldo, Hq, D));
    TERN_TRY(check_cache(kv_type, d_kcache, d_vcache, d_kscale, d_vscale));
    const int sms = tern::device_sm_count();
    if (sms <= 0) return TERN_ERR_UNSUPPORTED;
    if (d_ws == nullptr) return TERN_ERR_NULL;
    if (!aligned(d_ws, 256)) return TERN_ERR_ALIGN;
    if (ws_bytes < tern::decode_ws_bytes(B, Hq, Hkv, D, max_pages << shift, sms)) return TERN_ERR_SIZE;
    tern::DecodeArgs a = {};
    a.B = static_cast<int>(B);
    a.Hq = static_cast<int>(Hq);
    a.Hkv = static_cast<int>(Hkv);
    a.D = static_cast<int>(D);
    a.scale = scale;
    a.q = u16(d_Q);
    a.ldq = ldq;
    a.cache = {kv_type, num_pages, shift, d_kcache, d_vcache, d_kscale, d_vscale};
    a.table = d_page_table;
    a.max_pages = max_pages;
    a.lens = d_lens;
    a.o = static_cast<uint16_t*>(d_O);
    a.ldo = ldo;
    a.lse = d_lse;
    return from_cuda(tern::launch_decode(x_type == TERN_X_F16, a, d_ws, sms, as_stream(stream)));
}

tern_status tern_attn_weights(int x_type, int kv_type, int64_t B, const int32_t* d_cu_q, int64_t Tq, int64_t Hq,
                              int64_t Hkv, int64_t D, float scale, const void* d_Q, int64_t ldq, const float* d_lse,
                              int64_t num_pages, int64_t page_size, const void* d_kcache, const float* d_kscale,
                              const int32_t* d_page_table, int64_t max_pages, const int32_t* d_lens,
                              const int32_t* d_known, float decay, float* d_weight, int32_t* d_err, void* stream) {
    int shift = 0;
    if (!valid_x_type(x_type) || B < 0 || B > kMaxRows || Tq < 0 || Tq > kMaxRows) return TERN_ERR_SHAPE;
    TERN_TRY(check_pages(kv_type, Hkv, D, num_pages, page_size, &shift));
    if (!valid_heads(Hq) || Hq % Hkv != 0 || !valid_scale(scale) || !valid_scale(decay)) return TERN_ERR_SHAPE;
    if (max_pages < 0 || max_pages > (kMaxRows >> shift)) return TERN_ERR_SHAPE;   // (a token past a tile's end still counts in 32 bits)
    if (d_cu_q == nullptr && Tq != B) return TERN_ERR_SHAPE;
    if (B == 0 || Tq == 0) return TERN_OK;
    if (d_lse == nullptr || d_lens == nullptr || d_weight == nullptr || (max_pages > 0 && d_page_table == nullptr))
        return TERN_ERR_NULL;
    if (!aligned(d_cu_q, 4) || !aligned(d_lse, 4) || !aligned(d_lens, 4) || !aligned(d_known, 4) || !aligned(d_weight, 4) ||
        !aligned(d_page_table, 4) || !aligned(d_err, 4))
        return TERN_ERR_ALIGN;
    TERN_TRY(check_rows(d_Q, ldq, Hq, D));
    TERN_TRY(check_cache(kv_type, d_kcache, d_kcache, d_kscale, d_kscale));
    const int sms = tern::device_sm_count();
    if (sms <= 0) return TERN_ERR_UNSUPPORTED;
    tern::WeightsArgs w = {};
    w.B = static_cast<int>(B);
    w.cu_q = d_cu_q;
    w.Tq = static_cast<int>(Tq);
    w.Hq = static_cast<int>(Hq);
    w.Hkv = static_cast<int>(Hkv);
    w.D = static_cast<int>(D);
    w.scale = scale;
    w.decay = decay;
    w.q = u16(d_Q);
    w.ldq = ldq;
    w.lse = d_lse;
    w.cache = {kv_type, num_pages, shift, d_kcache, nullptr, d_kscale, nullptr};
    w.table = d_page_table;
    w.max_pages = max_pages;
    w.lens = d_lens;
    w.known = d_known;
    w.weight = d_weight;
    w.err = d_err;
    return from_cuda(tern::launch_weights(x_type == TERN_X_F16, w, sms, as_stream(stream)));
}

tern_status tern_kv_keep(int64_t B, int64_t Hkv, int64_t num_pages, int64_t page_size, const float* d_weight,
                         const int32_t* d_page_table, int64_t max_pages, const int32_t* d_lens, int64_t budget,
                         int64_t first, int64_t recent, int32_t* d_keep, int32_t* d_new_lens, void* stream) {
    int shift = 0;
    if (B < 0) return TERN_ERR_SHAPE;
    TERN_TRY(check_pages(TERN_KV_X16, Hkv, kMaxHeadDim, num_pages, page_size, &shift));
    if (B > kMaxRows / Hkv) return TERN_ERR_SHAPE;
    if (max_pages < 0 || max_pages > (kMaxRows >> shift)) return TERN_ERR_SHAPE;   // (a token past a tile's end still counts in 32 bits)
    if (budget < 1 || budget > kMaxRows || first < 0 || recent < 0 || first > budget || recent > budget - first)
        return TERN_ERR_SHAPE;
    if (B == 0) return TERN_OK;
    if (d_weight == nullptr || d_lens == nullptr || d_keep == nullptr || d_new_lens == nullptr ||
        (max_pages > 0 && d_page_table == nullptr))
        return TERN_ERR_NULL;
    if (!aligned(d_weight, 4) || !aligned(d_lens, 4) || !aligned(d_keep, 4) || !aligned(d_new_lens, 4) ||
        !aligned(d_page_table, 4))
        return TERN_ERR_ALIGN;
    if (d_new_lens == d_lens) return TERN_ERR_SHAPE;   // (every head of a sequence reads its length)
    const tern::KeepCall c = {B, static_cast<int>(Hkv), num_pages, shift, d_weight, d_page_table, max_pages, d_lens,
                              budget, first, recent, d_keep, d_new_lens};
    return from_cuda(tern::launch_keep(c, as_stream(stream)));
}

tern_status tern_kv_compact(int kv_type, int64_t B, int64_t Hkv, int64_t D, int64_t num_pages, int64_t page_size,
                            void* d_kcache, void* d_vcache, float* d_kscale, float* d_vscale, float* d_weight,
                            const int32_t* d_page_table, int64_t max_pages, const int32_t* d_keep, int64_t budget,
                            const int32_t* d_to_table, int64_t to_pages, int32_t* d_err, void* stream) {
    int shift = 0;
    if (B < 0) return TERN_ERR_SHAPE;
    TERN_TRY(check_pages(kv_type, Hkv, D, num_pages, page_size, &shift));
    if (B > kMaxMoves / Hkv) return TERN_ERR_SHAPE;
    if (max_pages < 0 || max_pages > (INT32_MAX >> shift)) return TERN_ERR_SHAPE;
    if (budget < 1 || budget > kMaxRows) return TERN_ERR_SHAPE;
    if (d_to_table != nullptr && (to_pages < 0 || to_pages > (INT32_MAX >> shift) || (to_pages << shift) < budget))
        return TERN_ERR_SHAPE;
    if (d_to_table != nullptr && d_to_table == d_page_table && to_pages != max_pages) return TERN_ERR_SHAPE;
    if (B == 0) return TERN_OK;
    if (d_keep == nullptr || (max_pages > 0 && d_page_table == nullptr)) return TERN_ERR_NULL;
    if (!aligned(d_weight, 4) || !aligned(d_keep, 4) || !aligned(d_page_table, 4) || !aligned(d_to_table, 4) ||
        !aligned(d_err, 4))
        return TERN_ERR_ALIGN;
    TERN_TRY(check_cache(kv_type, d_kcache, d_vcache, d_kscale, d_vscale));
    const tern::CompactCall c = {B, static_cast<int>(Hkv), static_cast<int>(D),
                                 {kv_type, num_pages, shift, d_kcache, d_vcache, d_kscale, d_vscale},
                                 d_weight, d_page_table, max_pages, d_keep, budget, d_to_table, to_pages, d_err};
    return from_cuda(tern::launch_compact(c, as_stream(stream)));
}

}  // extern "C"
