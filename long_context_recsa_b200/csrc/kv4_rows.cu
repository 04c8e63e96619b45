// Writing and reading rows of the 4-bit KV cache: quantisation (build, append) and
// dequantisation (read).  The format is in kv4.cuh.
//
// All three are bound by memory: a bf16 row of d = 128 is 256 bytes in and 80 out.  Four
// lanes own a group (8 dims each, one 16-byte load of bf16), so a group's minimum and
// maximum take two shuffles, a lane's 8 codes are one word, and a warp's stores of codes
// are whole 128-byte lines.  Four rows a thread are loaded before the first is used.
#include "kv4.cuh"

namespace recsa {

namespace {

constexpr int kThreadsRows = 256;
constexpr int kUnroll = 4;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
    load16_nc<__nv_bfloat16>(p, x);
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
    load16_nc<float>(p, x);
    load16_nc<float>(p + 4, x + 4);
}

// bf16 bits (in the high half) of the largest bf16 <= x.
__device__ __forceinline__ uint32_t bf16_floor(float x) {
    const uint32_t u = __float_as_uint(x), cut = u & 0xffff0000u;
    return ((u >> 31) && u != cut) ? cut + 0x10000u : cut;
}
// bf16 bits (in the high half) of the smallest bf16 >= x, x >= 0.
__device__ __forceinline__ uint32_t bf16_ceil(double x) {
    uint32_t u = __float_as_uint(__double2float_ru(x));
    return (u & 0xffffu) ? (u & 0xffff0000u) + 0x10000u : u;
}

// Quantises the 8 dims of this lane; the group's four lanes are l, l^1, l^2, l^3.
// `code` gets the lane's 8 nibbles, `par` the group's parameter word; returns the
// largest |value| of the group (0 for a group of NaN).
//
// Codes follow the definition in real arithmetic: (x - lo) / s is formed in fp32 (off
// by less than 1e-5), and where that is within 1e-4 of a half, the sign of
// (x - lo) - (k + 1/2) s in fp64 decides.
__device__ __forceinline__ float quantize8(const float (&x)[8], uint32_t& code, uint32_t& par) {
    float mn = x[0], mx = x[0], bad = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        mn = fminf(mn, x[i]);
        mx = fmaxf(mx, x[i]);
        bad += x[i] * 0.0f;              // NaN for a NaN or an infinity
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(kFull, mn, o));
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
        bad += __shfl_xor_sync(kFull, bad, o);
    }
    const uint32_t lob = bf16_floor(mn);
    const float lo = __uint_as_float(lob);
    const uint32_t sb = bf16_ceil(((double)mx - (double)lo) / 15.0);
    const float s = __uint_as_float(sb);
    code = 0;
    if (bad != 0.0f || !(fabsf(lo) <= 3.4e38f) || !(s <= 3.4e38f)) {
        par = 0x7fc00000u;               // lo = NaN, s = 0
        return 0.0f;
    }
    par = (sb >> 16) | lob;
    if (s < 1e-30f) {
        // tiny steps: 1 / s may overflow fp32
        if (s > 0.0f)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const double r = rint(((double)x[i] - (double)lo) / (double)s);
                code |= (uint32_t)fmin(r, 15.0) << (4 * i);
            }
    } else {
        const float inv = 1.0f / s;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = (x[i] - lo) * inv;
            float r = rintf(q);
            if (fabsf(q - r) > 0.4999f) {
                const float k = floorf(q);
                const double e =
                    ((double)x[i] - (double)lo) - ((double)k + 0.5) * (double)s;
                const bool up = e > 0.0 || (e == 0.0 && ((int)k & 1));
                r = up ? k + 1.0f : k;
            }
            code |= (uint32_t)fminf(r, 15.0f) << (4 * i);
        }
    }
    return fmaxf(fabsf(lo), fabsf(fmaf(s, 15.0f, lo)));
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
        c.kmax[i0] = 0;
        c.vmax[i0] = 0;
    }
    if (i0 < c.B) {
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
        c.kmax[u] = 0;
        c.vmax[u] = 0;
    }
}

// Quantises rows into the cache.  Grid: x = tiles of rows, y = unit, z = 0 keys, 1
// values.  Build: sequence b's rows 0 .. lens[b] - 1 go to slots of the same number.
// Append: its count rows go to the slots from len[b] on, and the last CTA of the grid
// advances the lengths (every CTA has read them by then).
template <typename T, int D>
__global__ void __launch_bounds__(kThreadsRows) kv4_rows_kernel(Kv4View c, Kv4Source src,
                                                                Kv4Lengths lens) {
    constexpr int LPR = D / 8;                 // lanes a row
    constexpr int RPW = 32 / LPR;              // rows a warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rows_cta = (int)(blockDim.x >> 5) * RPW * kUnroll;
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
    const int64_t r0 = blockIdx.x * (int64_t)rows_cta;
    float big = 0.0f;
    if (r0 < n) {
        const T* base = reinterpret_cast<const T*>(is_v ? src.v : src.k) + b * src.s_b + h * src.s_h;
        uint32_t* codes = reinterpret_cast<uint32_t*>(is_v ? c.vc : c.kc) + u * c.R * (D / 8);
        uint32_t* pars = (is_v ? c.vp : c.kp) + u * c.R * (D / kKv4Group);
        const int sub = lane % LPR;
        const int64_t r = r0 + (warp * kUnroll) * RPW + lane / LPR;
        float x[kUnroll][8];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int64_t row = r + i * RPW;
            if (row < n) {
                load8<T>(base + row * src.s_t + sub * 8, x[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int64_t row = r + i * RPW;
            uint32_t code, par;
            big = fmaxf(big, quantize8(x[i], code, par));
            if (row < n) {
                const int64_t slot = slot0 + row;
                codes[slot * (D / 8) + sub] = code;
                if ((sub & 3) == 0) pars[slot * (D / kKv4Group) + (sub >> 2)] = par;
            }
        }
        if (!is_v) {
            for (int i = threadIdx.x; i < rows_cta && r0 + i < n; i += blockDim.x) {
                const int64_t slot = slot0 + r0 + i;
                c.pos[u * c.R + slot] = (int32_t)(pos0 + r0 + i);
                c.w[u * c.R + slot] = 0.0f;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(kFull, big, o));
        // the maximum does not depend on the order of the atomics
        if (lane == 0 && big > 0.0f) {
            uint32_t* m = (is_v ? c.vmax : c.kmax) + u;
            if (__float_as_uint(big) > *(volatile uint32_t*)m) atomicMax(m, __float_as_uint(big));
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
    const int rows_cta = kThreadsRows / 32 * RPW * kUnroll;
    const int64_t r = blockIdx.x * (int64_t)rows_cta + (warp * kUnroll) * RPW + lane / LPR;
    uint32_t code[kUnroll], par[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
        const int64_t slot = start + r + i * RPW;
        code[i] = par[i] = 0;
        if (r + i * RPW < n && slot < L) {
            code[i] = codes[slot * (D / 8) + sub];
            par[i] = pars[slot * (D / kKv4Group) + (sub >> 2)];
        }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
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
    constexpr int per_warp = 32 / (D / 8) * kUnroll;
    const int64_t n = src.n;
    int threads = kThreadsRows;
    while (threads > 32 && (threads / 64) * per_warp >= n) threads /= 2;   // few rows: few warps
    const int64_t rows_cta = (int64_t)(threads / 32) * per_warp;
    const dim3 grid((unsigned)((n + rows_cta - 1) / rows_cta), (unsigned)(c.B * c.Hkv), 2);
    return kv4_launch(kv4_rows_kernel<T, D>, grid, threads, 0, s, c, src, lens);
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
    constexpr int rows_cta = kThreadsRows / 32 * (32 / (D / 8)) * kUnroll;
    const dim3 grid((unsigned)((n + rows_cta - 1) / rows_cta), (unsigned)(c.B * c.Hkv), 2);
    return kv4_launch(kv4_read_kernel<T, D>, grid, kThreadsRows, 0, s, c, start, n, (T*)k, (T*)v);
}

cudaError_t kv4_launch_read(const Kv4View& c, int64_t start, int64_t n, void* k, void* v, int dtype,
                            cudaStream_t s) {
    NvtxRange nv("recsa kv4 read");
    KV4_DISPATCH(read_impl, c, start, n, k, v, s);
}

}  // namespace recsa
