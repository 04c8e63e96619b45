// Declarations shared by the kernels of the 4-bit KV cache (recsa_kv4_*).
//
// A cache row is one token's key or value of one KV head, d = 64 or 128 dims in groups
// of 32.  A group holds lo + s * code: `lo` and `s` in bf16, one 4-bit code a dim:
//   lo = the largest bf16 <= min(x);  s = the smallest bf16 >= (max(x) - lo) / 15;
//   code = (x - lo) / s to the nearest integer, ties to even (s = 0: code 0).
// A group with a NaN or an infinity, or whose lo or s is no finite bf16, has lo = NaN
// and s = 0: every one of its dims reads back as NaN.
//
// Layout, per unit u = b * Hkv + h: codes [R][d/2] bytes (dim 2j in the low nibble of
// byte j), parameters [R][d/32] words (s in the low half, lo in the high half), token
// positions [R] int32 and accumulated weights [R] fp32; R is the capacity rounded up
// to whole tiles, so a tile of rows never leaves its unit.
#pragma once

#include <cuda_fp16.h>

#include "recsa_internal.cuh"

namespace recsa {

constexpr int kKv4Group = 32;        // dims that share a step and an offset
constexpr int kKv4RowPad = 128;      // R is a multiple of this many rows
constexpr float kKv4MinLog2 = -1e30f;   // running maximum before any token (log2 units)

struct Kv4View {
    uint8_t *kc, *vc;        // [U][R][D/2]
    uint32_t *kp, *vp;       // [U][R][D/32]
    int32_t* pos;            // [U][R]; 0 past the length
    float* w;                // [U][R]; 0 past the length
    int64_t* len;            // [B] rows in use
    int64_t* seen;           // [B] tokens appended so far: the next token's position
    uint32_t* kmax;          // [U] bits of the largest |value| written since the last build (a bound)
    uint32_t* vmax;
    uint32_t* kmin;          // [U] bits of the smallest group's largest |value| (but groups of 0)
    uint32_t* vmin;
    uint32_t* wide;          // [B] 1 where a unit's minimum lies 2^24 below its maximum: kv4_is_wide
    uint32_t* status;
    uint32_t* done;          // CTA arrival counter of append and evict (left at 0)
    int B, Hkv, Hq, G, D;
    int64_t R, cap;
    float scale;
};

struct Kv4Lengths { int64_t v[RECSA_MAX_BATCH]; };

// Source rows of build (strided, lengths from the host) and append (contiguous).
struct Kv4Source {
    const void *k, *v;
    int64_t s_b, s_h, s_t;   // element strides
    int64_t n;               // rows a sequence (append); the largest length (build)
    const int32_t* counts;   // append: rows in use of each sequence, or nullptr for n
    int append;
    int tiles;               // rows of a lane (set by the launcher)
};

// Scratch of the attention kernels.
struct Kv4Scratch {
    float* part;             // [2 * grid][rows a block][D + 2] split-softmax partials (both kernels')
    uint32_t* ucnt;          // [3 * grid] arrivals at the joins of split units (left at 0)
    float4* sum;             // kv4_launch_chunk: [grid][2][D / 4][128] sums of O, in large caches
    float2* stat;            // [U][rows] a row's reference m (log2 units) and 1 / sum of 2^(score - m)
};

// Rows of one attention wave: rows i0 .. i0 + w - 1 of every sequence's n rows.
struct Kv4Query {
    const void* q;           // [B][n][Hq][D]
    void* out;
    const int32_t* counts;   // rows in use of each sequence, or nullptr for n
    int n, i0, w;
    int acc_rows;            // the newest rows of each sequence whose weights accumulate
};

struct Kv4Maps { CUtensorMap k, v; };

cudaError_t kv4_launch_clear(const Kv4View& c, cudaStream_t s);
cudaError_t kv4_launch_build(const Kv4View& c, const Kv4Source& src, const Kv4Lengths& lens,
                             int dtype, cudaStream_t s);
cudaError_t kv4_launch_append(const Kv4View& c, const Kv4Source& src, int dtype, cudaStream_t s);
cudaError_t kv4_launch_read(const Kv4View& c, int64_t start, int64_t n, void* k, void* v, int dtype,
                            cudaStream_t s);
cudaError_t kv4_prepare_evict(const Kv4View& c);
cudaError_t kv4_launch_evict(const Kv4View& c, int64_t budget, int64_t n_first, int64_t n_recent,
                             int32_t* lists, cudaStream_t s);
int kv4_attend_counters();                              // words of Kv4Scratch::ucnt
size_t kv4_attend_part_floats(int D);                   // floats of Kv4Scratch::part
cudaError_t kv4_prepare_attend(int dtype, int D);
cudaError_t kv4_launch_attend(const Kv4View& c, const Kv4Query& qv, const Kv4Scratch& sc,
                              const Kv4Maps& maps, int chunk, int dtype, cudaStream_t s);
size_t kv4_chunk_part_floats(int D, int rows);          // the same for kv4_launch_chunk
size_t kv4_chunk_sum_floats(int D, int64_t R);          // floats of Kv4Scratch::sum
cudaError_t kv4_prepare_chunk(int D);
// bf16 with more than 8 rows a KV head: tensor-core products over blocks of rows, of keys and
// values as fp16; in fp32 for sequences whose magnitudes span more than that holds (wide)
cudaError_t kv4_launch_chunk(const Kv4View& c, const Kv4Query& qv, const Kv4Scratch& sc, cudaStream_t s);
// form_stat: after kv4_launch_chunk, which leaves no Kv4Scratch::stat (its scores come from
// keys rounded to fp16)
cudaError_t kv4_launch_weights(const Kv4View& c, const Kv4Query& qv, const Kv4Scratch& sc,
                               const Kv4Maps& maps, int chunk, int form_stat, int dtype, cudaStream_t s);

// A row's entry of Kv4Scratch::stat from its reference and sum (a row that sees no token: 0).
__device__ __forceinline__ float2 kv4_stat(float m, float l) {
    return l > 0.0f || l != l ? make_float2(m, 1.0f / l) : make_float2(0.0f, 0.0f);
}

// A launch that may start while the previous kernel of the stream finishes (every
// kernel of the cache passes pdl_wait() in all its threads before it touches memory).
template <typename... P, typename... A>
inline cudaError_t kv4_launch(void (*kern)(P...), dim3 grid, int threads, size_t smem,
                              cudaStream_t s, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at = pdl_attribute();
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// ---------------------------------------------------------------------------------
// device helpers
// ---------------------------------------------------------------------------------
__device__ __forceinline__ float kv4_step(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float kv4_off(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 2^x.  (Without .ftz every call is wrapped in the scaling of subnormal results.)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^e for a whole e, clamped to the normal range.
__device__ __forceinline__ float pow2i(int e) {
    e = e < -126 ? -126 : e > 127 ? 127 : e;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}
__device__ __forceinline__ float pow2z(int e) { return e < -126 ? 0.0f : pow2i(e); }
__device__ __forceinline__ int exponent_of(float x) {   // floor(log2 |x|), -127 for 0
    return (int)((__float_as_uint(x) >> 23) & 255u) - 127;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 y;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(y))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 y;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(y))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
          "l"(reinterpret_cast<uint64_t&>(c)));
    return y;
}

// Groups of keys or values from `least` to `most` in size: more than fp16 holds, scaled by `most`
// to 2^13?  (2^-24 of it is 2^-11 there, off by 2^-14 of itself; below, bits are lost.)
constexpr float kKv4Wide = 0x1p-24f;
__device__ __forceinline__ bool kv4_is_wide(float least, float most) { return least < most * kKv4Wide; }

// Rows of sequence b in a call of n rows (a count outside 0..n is recorded and taken as 0).
__device__ __forceinline__ int64_t kv4_count(const int32_t* counts, int b, int64_t n, uint32_t* st) {
    if (counts == nullptr) return n;
    const int64_t c = counts[b];
    if (c >= 0 && c <= n) return c;
    set_status(st, kStatusBadQuery);
    return 0;
}

}  // namespace recsa
