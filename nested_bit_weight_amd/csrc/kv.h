// kv.h -- what the key-value cache's kernels share: the launchers' arguments,
// the place of a slot in the pools, and the conversions of the element types.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nbw {

// A cache as the kernels take it (see nbw_kvcache in nbw.h).
struct KvCache {
    uint8_t *k, *v;         // pools [pages][heads][page][dim]
    int64_t pages;
    int heads, dim, fp8;
    int page_log2;          // slots of a page: 1 << page_log2
    const float *k_scale, *v_scale;  // fp8: [heads]
    const int32_t *table;   // [rows][table_ld]
    int rows, width;
    int64_t table_ld;
    int cap;                // width << page_log2
};

struct KvAppend {
    const uint16_t *k, *v, *q;
    uint16_t *q_out;
    int64_t k_ld, v_ld, q_ld, q_out_ld;
    int tokens, q_heads;
    float eps;
    const int32_t *cu, *lens, *positions;
    const float *rope;
    int64_t rope_rows;
    const uint16_t *q_norm, *k_norm;
    int32_t *pos;
    float *acc;
    int32_t *lens_out;
};

struct KvAttend {
    const uint16_t *q;
    uint16_t *out;
    int64_t q_ld, out_ld;
    int q_heads;
    float scale;
    const int32_t *lens;
    int max_len;
    const float *acc;
    float *acc_out;
    float decay;
    uint8_t *ws;
};

struct KvEvict {
    const float *acc;
    const int32_t *pos, *lens;
    int budget, sink, recent;
    float *acc_out;
    int32_t *pos_out, *lens_out;
    int max_len;
    uint8_t *ws;
};

// Work-items that a launch takes in a dimension.
constexpr int64_t MOST_ITEMS = ((int64_t)1 << 32) - 1;
constexpr bool fits_launch(int64_t groups, int threads) { return groups <= MOST_ITEMS / threads; }
constexpr int64_t APPEND_TOKENS = ((int64_t)1 << 24) - (1 << 13);  // 256 work-items each, and one for each row's length

hipError_t launch_kv_append(const KvCache &c, const KvAppend &a, hipStream_t stream);
int64_t kv_attend_workspace_bytes(const KvCache &c, int q_heads, int max_len, bool weights, int cu_count);
hipError_t launch_kv_attend(const KvCache &c, const KvAttend &a, int cu_count, hipStream_t stream);
int64_t kv_evict_workspace_bytes(const KvCache &c, int budget, int max_len);
hipError_t launch_kv_evict(const KvCache &c, const KvEvict &a, hipStream_t stream);

typedef uint32_t u32x2_kv __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_kv __attribute__((ext_vector_type(4)));

// A row's length within [0, bound].
__device__ __forceinline__ int kv_len(const int32_t *lens, int row, int bound) {
    const int n = lens[row];
    return n < 0 ? 0 : n > bound ? bound : n;
}

// The number of (row, head, slot)'s row in a pool, counted in rows of dim
// elements, or -1 where the table names no page of the pool.  64 bits: a long
// cache has more than 2^31 elements.
__device__ __forceinline__ int64_t kv_row(const KvCache &c, int row, int head, int slot) {
    const int32_t page = c.table[(int64_t)row * c.table_ld + (slot >> c.page_log2)];
    if (page < 0 || page >= c.pages) return -1;
    return (((int64_t)page * c.heads + head) << c.page_log2) + (slot & ((1 << c.page_log2) - 1));
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// fp32 to bf16, to nearest even; a NaN stays one.
__device__ __forceinline__ uint16_t to_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// Sums and other reductions over the 64 lanes of a wave, in six register-to-register
// steps: within rows of 16 lanes, from each row into the next, from the lower half
// into the upper.  (These sit on paths that small calls wait for; general shuffles go
// through LDS.  16 rows' attention 18.3 -> 17.8 us, ranking 120001 slots 56 -> 53.)
template <int CTRL, int ROWS>
__device__ __forceinline__ int32_t from_lane(int32_t none, int32_t x) {
    return __builtin_amdgcn_update_dpp(none, x, CTRL, ROWS, 0xF, false);
}
template <class Op>
__device__ __forceinline__ int32_t wave_running(int32_t x, int32_t none, Op op) {  // over this lane and those before it
    x = op(x, from_lane<0x111, 0xF>(none, x));
    x = op(x, from_lane<0x112, 0xF>(none, x));
    x = op(x, from_lane<0x114, 0xF>(none, x));
    x = op(x, from_lane<0x118, 0xF>(none, x));
    x = op(x, from_lane<0x142, 0xA>(none, x));
    return op(x, from_lane<0x143, 0xC>(none, x));
}
template <class Op>
__device__ __forceinline__ int32_t wave_all(int32_t x, int32_t none, Op op) {  // over all lanes, in each of them
    return __builtin_amdgcn_readlane(wave_running(x, none, op), 63);
}
struct OpSum { __device__ __forceinline__ int32_t operator()(int32_t a, int32_t b) const { return a + b; } };
struct OpMax { __device__ __forceinline__ int32_t operator()(int32_t a, int32_t b) const { return a > b ? a : b; } };
struct OpMaxU { __device__ __forceinline__ int32_t operator()(int32_t a, int32_t b) const { return (uint32_t)a > (uint32_t)b ? a : b; } };
struct OpMinU { __device__ __forceinline__ int32_t operator()(int32_t a, int32_t b) const { return (uint32_t)a < (uint32_t)b ? a : b; } };
__device__ __forceinline__ int32_t wave_running_sum(int32_t x) { return wave_running(x, 0, OpSum()); }
__device__ __forceinline__ int32_t wave_sum(int32_t x) { return wave_all(x, 0, OpSum()); }
__device__ __forceinline__ int32_t wave_max(int32_t x) { return wave_all(x, INT32_MIN, OpMax()); }
__device__ __forceinline__ uint32_t wave_max_u(uint32_t x) { return (uint32_t)wave_all((int32_t)x, 0, OpMaxU()); }
__device__ __forceinline__ uint32_t wave_min_u(uint32_t x) { return (uint32_t)wave_all((int32_t)x, -1, OpMinU()); }

// Four fp32 values, already divided by the head's factor, to the cache's 8 bits:
// limited to the largest finite value and rounded to nearest even, NaN kept.
__device__ __forceinline__ uint32_t to_fp8x4(float a, float b, float c, float d) {
    auto limit = [](float x) { return x > 448.f ? 448.f : x < -448.f ? -448.f : x; };
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(limit(a), limit(b), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(limit(c), limit(d), w, true);
    return (uint32_t)w;
}

}  // namespace nbw
