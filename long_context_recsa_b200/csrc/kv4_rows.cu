// Writing and reading rows of the 4-bit KV cache: quantisation (build, append) and
// dequantisation (read).  The format is in kv4.cuh.
//
// All three are bound by memory if the quantisation takes few instructions: a bf16 row of
// d = 128 is 256 bytes in and 80 out.  Two lanes own
// a group (16 dims each), so what is done once a group costs a sixteenth of it a dim, and
// the group's minimum and maximum take one exchange; arithmetic goes two dims at a time.
//
// Measured (B200, 131072 x 8 rows of bf16, d = 128): build 214 us for 705 MB, 3.3 TB/s: 314
// instructions a warp for 512 dims, issued in 70% of the cycles, the busiest pipe (ALU) half used:
// latency, and the instruction cache.  (Keeping the smallest group beside the largest value costs
// 6 us of it.)  Fewer or more rows in flight a lane than 2 (433 and 270 us) and another number of
// CTAs than 4 (231 to 275) were slower.  Read 105 us for 705 MB, 6.7 TB/s.
#include "kv4.cuh"

namespace recsa {

namespace {

constexpr int kThreadsRows = 256;
constexpr int kUnroll = 2;           // rows of a lane that are loaded before the first is used
constexpr int kTilesRows = 8;        // rows of a lane in all, at most
constexpr int kReadRows = 4;         // rows of a lane in the read back
constexpr uint32_t kInfBits = 0x7f800000u;

// 16 dims of a row as they are stored: two 16-byte words of bf16, four of fp32.
template <typename T> struct Raw { uint4 a[(int)sizeof(T)]; };

template <typename T>
__device__ __forceinline__ void load_raw(Raw<T>& r, const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) r.a[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
}

__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {   // of two bf16
    uint32_t y;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}

__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}

// The 16 values, and the smallest and largest of the group (lanes l and l ^ 1); both are
// NaN if one of the group is.
__device__ __forceinline__ void spread(const Raw<__nv_bfloat16>& r, float2 (&x)[8], float& mn,
                                       float& mx) {
    const uint32_t w[8] = {r.a[0].x, r.a[0].y, r.a[0].z, r.a[0].w,
                           r.a[1].x, r.a[1].y, r.a[1].z, r.a[1].w};
    uint32_t lo = w[0], hi = w[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        if (i > 0) {
            lo = min2_nan(lo, w[i]);
            hi = max2_nan(hi, w[i]);
        }
    }
    hi ^= 0x80008000u;                   // the largest as the smallest of the negated: one word
    uint32_t both = min2_nan(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
    both = min2_nan(both, __shfl_xor_sync(kFull, both, 1));
    mn = __uint_as_float(both << 16);
    mx = -__uint_as_float(both & 0xffff0000u);
}
__device__ __forceinline__ void spread(const Raw<float>& r, float2 (&x)[8], float& mn, float& mx) {
    float lo = __uint_as_float(r.a[0].x), hi = -lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = make_float2(__uint_as_float(r.a[i].x), __uint_as_float(r.a[i].y));
        x[2 * i + 1] = make_float2(__uint_as_float(r.a[i].z), __uint_as_float(r.a[i].w));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = min_nan(min_nan(lo, x[i].x), x[i].y);
        hi = min_nan(min_nan(hi, -x[i].x), -x[i].y);
    }
    mn = min_nan(lo, __shfl_xor_sync(kFull, lo, 1));
    mx = -min_nan(hi, __shfl_xor_sync(kFull, hi, 1));
}

__device__ __forceinline__ float2 twice(float a) { return make_float2(a, a); }

// bf16 bits (in the high half) of the largest bf16 <= x.
__device__ __forceinline__ uint32_t bf16_floor(float x) {
    const uint32_t u = __float_as_uint(x), cut = u & 0xffff0000u;
    return ((u >> 31) && u != cut) ? cut + 0x10000u : cut;
}

// 1 where x - lo < (k - 1/2) s in real arithmetic, or equal with k odd: code k is one too high.
__device__ __forceinline__ uint32_t too_high(float x, float lo, float k, float s) {
    const float half = (k - 0.5f) * s;
    if (__fsub_rd(x, lo) < half) return 1u;
    return __fsub_ru(x, lo) > half ? 0u : (uint32_t)((int)k & 1);
}

// Quantises the 16 dims of this lane (spread() above has the group's extremes).  `code`
// gets the lane's 16 nibbles, `par` the group's parameter word; returns the largest |value|
// of the group (0 for a group of NaN).
//
// Everything is decided as in real arithmetic, with fp32 operations only (fp64 ones took
// 397 us instead of 208 at 131072 x 8 bf16 rows).  A difference rounded up (down) is the
// smallest (largest) fp32 number not below (above) the real one, so it compares with a
// number of fp32 as the real difference does:
//   s: the smallest bf16 with 15 s >= mx - lo; 15 s is exact.  A product with 1 / 15 is off
//      by less than a step of bf16, two corrections suffice.
//   codes: the quotient is formed a few 1e-7 too large, so that rounding it may give a code
//      one too high but never one too low; the remainder x - lo - code s shows where that
//      may be (bf16 values lie on ties often), and too_high() decides.
__device__ __forceinline__ float quantize16(const float2 (&x)[8], float mn, float mx, uint2& code,
                                            uint32_t& par) {
    const uint32_t lob = bf16_floor(mn);
    const float lo = __uint_as_float(lob);
    const float range = __fsub_ru(mx, lo);
    uint32_t sb = __float_as_uint(range * (1.0f / 15.0f)) & 0xffff0000u;
    if (__uint_as_float(sb) * 15.0f < range) sb += 0x10000u;
    if (__uint_as_float(sb) * 15.0f < range) sb += 0x10000u;
    if (range > 1e38f) {
        // the range itself may pass fp32
        sb = __float_as_uint(__double2float_ru(((double)mx - (double)lo) / 15.0));
        if (sb & 0xffffu) sb = (sb & 0xffff0000u) + 0x10000u;
    }
    const float s = __uint_as_float(sb);
    uint32_t c[2] = {0, 0};
    float big = 0.0f;
    par = 0x7fc00000u;                   // lo = NaN, s = 0: a group that cannot be held
    if (fabsf(lo) <= 3.4e38f && s <= 3.4e38f) {
        par = (sb >> 16) | lob;
        big = fmaxf(fabsf(lo), fabsf(fmaf(s, 15.0f, lo)));
        if (s >= 1e-30f && range <= 1e38f) {
            // adding 1.5 * 2^23 rounds to a whole number, in the low bits
            constexpr float kRound = 12582912.0f;
            const float inv = __frcp_rn(s) * (1.0f + 0x1p-21f);
            float low = 0.0f;
            float2 r[8], e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 t = add2(x[i], twice(-lo));
                r[i] = fma2(t, twice(inv), twice(kRound));
                const float2 k = add2(r[i], twice(-kRound));
                e[i] = fma2(k, twice(-s), t);
                low = fminf(low, fminf(e[i].x, e[i].y));
                c[i >> 2] += __float_as_uint(r[i].x) * (1u << (8 * (i & 3)));
                c[i >> 2] += __float_as_uint(r[i].y) * (16u << (8 * (i & 3)));
            }
            // less the bits of 1.5 * 2^23 in each of the eight places
            c[0] -= 0x4b400000u * 0x11111111u;
            c[1] -= 0x4b400000u * 0x11111111u;
            const float near = -0.5f * s * (1.0f - 0x1p-21f);
            if (low <= near) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (e[i].x <= near)
                        c[i >> 2] -= too_high(x[i].x, lo, r[i].x - kRound, s) << (8 * (i & 3));
                    if (e[i].y <= near)
                        c[i >> 2] -= too_high(x[i].y, lo, r[i].y - kRound, s) << (8 * (i & 3) + 4);
                }
            }
        } else if (s > 0.0f) {
            // 1 / s or x - lo may overflow fp32
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const double a = rint(((double)x[i].x - (double)lo) / (double)s);
                const double b = rint(((double)x[i].y - (double)lo) / (double)s);
                c[i >> 2] |= (uint32_t)fmin(a, 15.0) << (8 * (i & 3));
                c[i >> 2] |= (uint32_t)fmin(b, 15.0) << (8 * (i & 3) + 4);
            }
        }
    }
    code = make_uint2(c[0], c[1]);
    return big;
}

}  // namespace

// Initial state, and the state before a build: weights and positions of every row and
// the largest-value bounds are 0 (with `all`), lengths 0.
__global__ void __launch_bounds__(kThreadsRows) kv4_clear_kernel(Kv4View c) {
    pdl_wait();
    const int64_t n = (int64_t)c.B * c.Hkv * c.R / 4;   // R is a multiple of 128
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    const int64_t i0 = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
    for (int64_t i = i0; i < n; i += step) {
        reinterpret_cast<int4*>(c.pos)[i] = make_int4(0, 0, 0, 0);
        reinterpret_cast<float4*>(c.w)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (i0 < c.B * c.Hkv) {
        c.kmax[i0] = c.vmax[i0] = 0;
        c.kmin[i0] = c.vmin[i0] = kInfBits;
    }
    if (i0 < c.B) {
        c.wide[i0] = 0;
        c.len[i0] = 0;
        c.seen[i0] = 0;
    }
    if (i0 == 0) {
        *c.status = 0;
        *c.done = 0;
    }
}

// Before a build: the rows past the new length lose their weight and position, and the
// bounds start from 0.  One CTA a unit; the lengths themselves are set by the rows
// kernel that follows.
__global__ void __launch_bounds__(kThreadsRows) kv4_reset_kernel(Kv4View c, Kv4Lengths lens) {
    pdl_wait();
    pdl_launch_dependents();
    const int u = blockIdx.x, b = u / c.Hkv;
    const int64_t old = c.len[b];
    for (int64_t i = lens.v[b] + threadIdx.x; i < old; i += blockDim.x) {
        c.pos[u * c.R + i] = 0;
        c.w[u * c.R + i] = 0.0f;
    }
    if (threadIdx.x == 0) {
        c.kmax[u] = c.vmax[u] = 0;
        c.kmin[u] = c.vmin[u] = kInfBits;
        if (u == b * c.Hkv) c.wide[b] = 0;
    }
}

// Quantises rows into the cache.  Grid: x = tiles of rows, y = unit, z = 0 keys, 1
// values.  Build: sequence b's rows 0 .. lens[b] - 1 go to slots of the same number.
// Append: its count rows go to the slots from len[b] on, and the last CTA of the grid
// advances the lengths (every CTA has read them by then).
template <typename T, int D>
__global__ void __launch_bounds__(kThreadsRows, 4) kv4_rows_kernel(Kv4View c, Kv4Source src,
                                                                   Kv4Lengths lens) {
    constexpr int LPR = D / 16;                // lanes a row
    constexpr int RPW = 32 / LPR;              // rows a warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rows_tile = (int)(blockDim.x >> 5) * RPW;
    const int u = blockIdx.y, b = u / c.Hkv, h = u % c.Hkv;
    const bool is_v = blockIdx.z != 0;
    pdl_wait();
    pdl_launch_dependents();
    int64_t n, slot0 = 0, pos0 = 0;
    if (src.append) {
        n = kv4_count(src.counts, b, src.n, c.status);
        slot0 = c.len[b];
        pos0 = c.seen[b];
        if (slot0 + n > c.cap || pos0 + n > 0x7fffffff) {
            if (threadIdx.x == 0) set_status(c.status, kStatusCapacity);
            n = 0;
        }
    } else {
        n = lens.v[b];
    }
    const T* base = reinterpret_cast<const T*>(is_v ? src.v : src.k) + b * src.s_b + h * src.s_h;
    uint2* codes = reinterpret_cast<uint2*>(is_v ? c.vc : c.kc) + u * c.R * LPR;
    uint32_t* pars = (is_v ? c.vp : c.kp) + u * c.R * (D / kKv4Group);
    const int sub = lane % LPR;
    const int64_t r0 = blockIdx.x * (int64_t)rows_tile * src.tiles;
    float big = 0.0f, small = INFINITY;        // of the groups' largest values
    Raw<T> raw[kUnroll];
#pragma unroll 1
    for (int tile = 0; tile < src.tiles; tile += kUnroll) {
        const int64_t r = r0 + (int64_t)tile * rows_tile + warp * RPW + lane / LPR;
        if (r - lane / LPR >= n) break;        // the same for the whole warp
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            // a row past the last one is read again in its place, and not stored
            const int64_t row = r + (int64_t)i * rows_tile;
            load_raw(raw[i], base + (row < n ? row : n - 1) * src.s_t + sub * 16);
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int64_t row = r + (int64_t)i * rows_tile;
            uint2 code;
            uint32_t par;
            float2 x[8];
            float mn, mx;
            spread(raw[i], x, mn, mx);
            const float most = quantize16(x, mn, mx, code, par);
            big = fmaxf(big, most);
            if (most > 0.0f) small = fminf(small, most);
            const int64_t slot = slot0 + row;
            if (row < n && in_bounds(slot >= 0 && slot < c.cap, c.status)) {
                codes[slot * LPR + sub] = code;
                if ((sub & 1) == 0) pars[slot * (D / kKv4Group) + (sub >> 1)] = par;
            }
        }
    }
    if (!is_v) {
        for (int64_t i = r0 + threadIdx.x; i < r0 + rows_tile * src.tiles && i < n; i += blockDim.x) {
            const int64_t slot = slot0 + i;
            if (!in_bounds(slot >= 0 && slot < c.cap, c.status)) continue;
            c.pos[u * c.R + slot] = (int32_t)(pos0 + i);
            c.w[u * c.R + slot] = 0.0f;
        }
    }
    // the CTA's largest and smallest, then one atomic each (neither depends on their order);
    // a check by every warp made all of them queue at the unit's one word
    __shared__ float2 warp_big[kThreadsRows / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        big = fmaxf(big, __shfl_xor_sync(kFull, big, o));
        small = fminf(small, __shfl_xor_sync(kFull, small, o));
    }
    if (lane == 0) warp_big[warp] = make_float2(big, small);
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < (int)(blockDim.x >> 5); ++i) {
            big = fmaxf(big, warp_big[i].x);
            small = fminf(small, warp_big[i].y);
        }
        volatile uint32_t *hi = (is_v ? c.vmax : c.kmax) + u, *lo = (is_v ? c.vmin : c.kmin) + u;
        const bool more = __float_as_uint(big) > *hi, less = __float_as_uint(small) < *lo;
        if (more) atomicMax((uint32_t*)hi, __float_as_uint(big));
        if (less) atomicMin((uint32_t*)lo, __float_as_uint(small));
        if (more || less) {
            // of two CTAs that bring the one and the other, the later sees both
            __threadfence();
            if (kv4_is_wide(__uint_as_float(*lo), __uint_as_float(*hi))) c.wide[b] = 1;
        }
    }
    if (!src.append) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
            for (int i = threadIdx.x; i < c.B; i += blockDim.x) {
                c.len[i] = lens.v[i];
                c.seen[i] = lens.v[i];
            }
        return;
    }
    __shared__ int last;
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t total = gridDim.x * gridDim.y * gridDim.z;
        __threadfence();
        last = atomicAdd(c.done, 1u) == total - 1;
    }
    __syncthreads();
    if (!last) return;
    for (int i = threadIdx.x; i < c.B; i += blockDim.x) {
        int64_t m = kv4_count(src.counts, i, src.n, c.status);
        const int64_t L = c.len[i], P = c.seen[i];
        if (L + m > c.cap || P + m > 0x7fffffff) m = 0;
        c.len[i] = L + m;
        c.seen[i] = P + m;
    }
    if (threadIdx.x == 0) *c.done = 0;
}

// Slots start .. start + n - 1 as values of the storage dtype, [B][Hkv][n][D]; a slot
// at or past the length gives zeros.  Grid: x = tiles of rows, y = unit, z = keys, values.
template <typename T, int D>
__global__ void __launch_bounds__(kThreadsRows) kv4_read_kernel(Kv4View c, int64_t start, int64_t n,
                                                                T* k_out, T* v_out) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int u = blockIdx.y, b = u / c.Hkv;
    const bool is_v = blockIdx.z != 0;
    T* out = is_v ? v_out : k_out;
    pdl_wait();
    pdl_launch_dependents();
    if (out == nullptr) return;
    const int64_t L = c.len[b];
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(is_v ? c.vc : c.kc) + u * c.R * (D / 8);
    const uint32_t* pars = (is_v ? c.vp : c.kp) + u * c.R * (D / kKv4Group);
    const int sub = lane % LPR;
    const int rows_cta = kThreadsRows / 32 * RPW * kReadRows;
    const int64_t r = blockIdx.x * (int64_t)rows_cta + (warp * kReadRows) * RPW + lane / LPR;
    uint32_t code[kReadRows], par[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        const int64_t slot = start + r + i * RPW;
        code[i] = par[i] = 0;
        if (r + i * RPW < n && slot < L && in_bounds(slot >= 0 && slot < c.cap, c.status)) {
            code[i] = codes[slot * (D / 8) + sub];
            par[i] = pars[slot * (D / kKv4Group) + (sub >> 2)];
        }
    }
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        const int64_t row = r + i * RPW;
        if (row >= n) continue;
        const float s = kv4_step(par[i]), lo = kv4_off(par[i]);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fmaf(s, (float)((code[i] >> (4 * j)) & 15u), lo);
        T* dst = out + ((int64_t)u * n + row) * D + sub * 8;
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(dst + 4) = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            uint4 w;
            __nv_bfloat162 p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
            w.x = *reinterpret_cast<uint32_t*>(&p[0]);
            w.y = *reinterpret_cast<uint32_t*>(&p[1]);
            w.z = *reinterpret_cast<uint32_t*>(&p[2]);
            w.w = *reinterpret_cast<uint32_t*>(&p[3]);
            *reinterpret_cast<uint4*>(dst) = w;
        }
    }
}

// ---------------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------------
cudaError_t kv4_launch_clear(const Kv4View& c, cudaStream_t s) {
    NvtxRange nv("recsa kv4 clear");
    const int64_t n = (int64_t)c.B * c.Hkv * c.R / 4;
    int64_t ctas = (n + kThreadsRows * 4 - 1) / (kThreadsRows * 4);
    const int64_t least = ((int64_t)c.B * c.Hkv + kThreadsRows - 1) / kThreadsRows;
    if (ctas < least) ctas = least;
    if (ctas > 148 * 32) ctas = 148 * 32;    // >= 65535 / 256 CTAs: the bounds are covered
    return kv4_launch(kv4_clear_kernel, dim3((unsigned)ctas), kThreadsRows, 0, s, c);
}

template <typename T, int D>
static cudaError_t rows_impl(const Kv4View& c, const Kv4Source& src, const Kv4Lengths& lens,
                             cudaStream_t s) {
    constexpr int per_warp = 32 / (D / 16);
    const int64_t n = src.n;
    // a lane takes 8 rows where that still fills the GPU, else 2
    const int64_t units = 2 * (int64_t)c.B * c.Hkv;
    Kv4Source sized = src;
    sized.tiles = n * units >= (int64_t)148 * 8 * (kThreadsRows / 32) * per_warp * kTilesRows
                      ? kTilesRows : kUnroll;
    int threads = kThreadsRows;
    while (threads > 32 && (int64_t)(threads / 64) * per_warp * sized.tiles >= n) threads /= 2;
    const int64_t rows_cta = (int64_t)(threads / 32) * per_warp * sized.tiles;
    const dim3 grid((unsigned)((n + rows_cta - 1) / rows_cta), (unsigned)(c.B * c.Hkv), 2);
    return kv4_launch(kv4_rows_kernel<T, D>, grid, threads, 0, s, c, sized, lens);
}

#define KV4_DISPATCH(FN, ...)                                                   \
    do {                                                                        \
        if (dtype == RECSA_BF16 && c.D == 128) return FN<__nv_bfloat16, 128>(__VA_ARGS__); \
        if (dtype == RECSA_BF16 && c.D == 64) return FN<__nv_bfloat16, 64>(__VA_ARGS__);   \
        if (dtype == RECSA_F32 && c.D == 128) return FN<float, 128>(__VA_ARGS__);          \
        if (dtype == RECSA_F32 && c.D == 64) return FN<float, 64>(__VA_ARGS__);            \
        return cudaErrorInvalidValue;                                           \
    } while (0)

cudaError_t kv4_launch_build(const Kv4View& c, const Kv4Source& src, const Kv4Lengths& lens,
                             int dtype, cudaStream_t s) {
    NvtxRange nv("recsa kv4 build");
    cudaError_t e = kv4_launch(kv4_reset_kernel, dim3((unsigned)(c.B * c.Hkv)), kThreadsRows, 0, s, c,
                               lens);
    if (e != cudaSuccess) return e;
    KV4_DISPATCH(rows_impl, c, src, lens, s);
}

cudaError_t kv4_launch_append(const Kv4View& c, const Kv4Source& src, int dtype, cudaStream_t s) {
    NvtxRange nv("recsa kv4 append");
    const Kv4Lengths none = {};
    KV4_DISPATCH(rows_impl, c, src, none, s);
}

template <typename T, int D>
static cudaError_t read_impl(const Kv4View& c, int64_t start, int64_t n, void* k, void* v,
                             cudaStream_t s) {
    constexpr int rows_cta = kThreadsRows / 32 * (32 / (D / 8)) * kReadRows;
    const dim3 grid((unsigned)((n + rows_cta - 1) / rows_cta), (unsigned)(c.B * c.Hkv), 2);
    return kv4_launch(kv4_read_kernel<T, D>, grid, kThreadsRows, 0, s, c, start, n, (T*)k, (T*)v);
}

cudaError_t kv4_launch_read(const Kv4View& c, int64_t start, int64_t n, void* k, void* v, int dtype,
                            cudaStream_t s) {
    NvtxRange nv("recsa kv4 read");
    KV4_DISPATCH(read_impl, c, start, n, k, v, s);
}

}  // namespace recsa
