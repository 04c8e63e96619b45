// Eviction from the 4-bit KV cache by accumulated attention weight.
//
// Per unit (sequence, KV head) of length L > budget, `budget` rows stay: the first
// n_first tokens, the newest n_recent ones, and of the others those of the largest
// weights (ties: the lower slot; a NaN weight ranks below every number).  Kept rows in
// slots >= budget (they "move") go into the slots < budget that became free, the j-th by
// slot into the j-th free one: sources and destinations are disjoint, so rows move in
// place, and only as many as leave.  Attention does not depend on the order of slots.
//
// One CTA a unit: a radix select over 32-bit order keys (4 passes of 8 bits: the
// threshold key and how many of its ties stay), a scan that lists free slots and movers
// in ascending order, and the copies.
#include "kv4.cuh"

namespace recsa {

namespace {

constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;

// Order key of a slot: ~0 for a protected token, else monotone in the weight.
__device__ __forceinline__ uint32_t evict_key(float w, int32_t pos, int64_t first, int64_t recent0) {
    if (pos < first || pos >= recent0) return 0xffffffffu;
    if (w != w) return 0u;
    return ordered_key(w);   // at most the key of +inf, below ~0; at least that of -inf, above 0
}

// Exclusive prefix of v over the CTA, and the total.
__device__ __forceinline__ int cta_scan(int v, int* tmp, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int y = tmp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(kFull, y, o);
            if (lane >= o) y += z;
        }
        tmp[lane] = y;
    }
    __syncthreads();
    total = tmp[kEvictWarps - 1];
    return x - v + (warp > 0 ? tmp[warp - 1] : 0);
}

}  // namespace

// lists: [U][R] int32; free slots from the front of a unit's part, movers from R / 2 on
// (neither can pass R / 2: both are at most min(budget, L - budget)).
template <int D>
__global__ void __launch_bounds__(kEvictThreads) kv4_evict_kernel(Kv4View c, int64_t budget,
                                                                  int64_t n_first, int64_t n_recent,
                                                                  int32_t* lists) {
    __shared__ int hist[256];
    __shared__ int scan_tmp[kEvictWarps];
    __shared__ uint32_t s_prefix;
    __shared__ int64_t s_need;
    __shared__ int last;
    const int u = blockIdx.x, b = u / c.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t L = c.len[b];
    if (L > budget) {
        const int64_t recent0 = c.seen[b] - n_recent;
        const float* w = c.w + u * c.R;
        const int32_t* pos = c.pos + u * c.R;
        uint32_t prefix = 0;
        int64_t need = budget;           // of the slots whose key starts with prefix
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (threadIdx.x < 256) hist[threadIdx.x] = 0;
            __syncthreads();
            for (int64_t i = threadIdx.x; i < L; i += kEvictThreads) {
                const uint32_t k = evict_key(w[i], pos[i], n_first, recent0);
                if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
                    atomicAdd(&hist[(k >> shift) & 255u], 1);
            }
            __syncthreads();
            if (warp == 0) {
                // from the top bin down: the bin in which the need-th key lies
                int mine[8], sum = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    mine[j] = hist[255 - (lane * 8 + j)];
                    sum += mine[j];
                }
                int x = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(kFull, x, o);
                    if (lane >= o) x += y;
                }
                int64_t before = x - sum;
                if (before < need && need <= x) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (before < need && need <= before + mine[j]) {
                            s_prefix = prefix | ((uint32_t)(255 - (lane * 8 + j)) << shift);
                            s_need = need - before;
                        }
                        before += mine[j];
                    }
                }
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;
        }
        // need slots with key == prefix stay, the lowest first
        int32_t* free_list = lists + u * c.R;
        int32_t* move_list = free_list + c.R / 2;
        int64_t ties = 0;
        int n_free = 0, n_move = 0;
        for (int64_t i0 = 0; i0 < L; i0 += kEvictThreads) {
            const int64_t i = i0 + threadIdx.x;
            uint32_t k = 0;
            if (i < L) k = evict_key(w[i], pos[i], n_first, recent0);
            const int eq = i < L && k == prefix;
            int total;
            const int rank = cta_scan(eq, scan_tmp, total);
            const bool kept = i < L && (k > prefix || (eq && ties + rank < need));
            ties += total;
            const int fr = i < L && i < budget && !kept, mv = i >= budget && kept;
            // one of the two is always 0 for a slot: a packed scan counts both
            const int both = cta_scan(fr | (mv << 16), scan_tmp, total);
            if (fr) free_list[n_free + (both & 0xffff)] = (int32_t)i;
            if (mv) move_list[n_move + (both >> 16)] = (int32_t)i;
            n_free += total & 0xffff;
            n_move += total >> 16;
        }
        __syncthreads();                 // the lists are read below by other threads
        // a row is 2 x (D / 2) bytes of codes and 2 x (D / 8) bytes of parameters
        constexpr int CK = D / 32, CH = 2 * CK + 2;   // 16-byte pieces of codes; + parameters
        uint4* kc = reinterpret_cast<uint4*>(c.kc) + u * c.R * CK;
        uint4* vc = reinterpret_cast<uint4*>(c.vc) + u * c.R * CK;
        uint32_t* kp = c.kp + u * c.R * CK;
        uint32_t* vp = c.vp + u * c.R * CK;
        for (int64_t x = threadIdx.x; x < (int64_t)n_move * CH; x += kEvictThreads) {
            const int j = (int)(x / CH), p = (int)(x % CH);
            const int64_t to = free_list[j], from = move_list[j];
            if (p < CK) {
                kc[to * CK + p] = kc[from * CK + p];
            } else if (p < 2 * CK) {
                vc[to * CK + p - CK] = vc[from * CK + p - CK];
            } else {
                uint32_t* a = p == 2 * CK ? kp : vp;
#pragma unroll
                for (int e = 0; e < CK; ++e) a[to * CK + e] = a[from * CK + e];
                if (p == 2 * CK) {
                    c.w[u * c.R + to] = c.w[u * c.R + from];
                    c.pos[u * c.R + to] = c.pos[u * c.R + from];
                }
            }
        }
        __syncthreads();
        for (int64_t i = budget + threadIdx.x; i < L; i += kEvictThreads) {
            c.w[u * c.R + i] = 0.0f;
            c.pos[u * c.R + i] = 0;
        }
    }
    // the last CTA sets the lengths: every CTA has read its own by then
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(c.done, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    for (int i = threadIdx.x; i < c.B; i += kEvictThreads)
        if (c.len[i] > budget) c.len[i] = budget;
    if (threadIdx.x == 0) *c.done = 0;
}

cudaError_t kv4_launch_evict(const Kv4View& c, int64_t budget, int64_t n_first, int64_t n_recent,
                             int32_t* lists, cudaStream_t s) {
    NvtxRange nv("recsa kv4 evict");
    const dim3 grid((unsigned)(c.B * c.Hkv));
    if (c.D == 128)
        return kv4_launch(kv4_evict_kernel<128>, grid, kEvictThreads, 0, s, c, budget, n_first,
                          n_recent, lists);
    return kv4_launch(kv4_evict_kernel<64>, grid, kEvictThreads, 0, s, c, budget, n_first, n_recent,
                      lists);
}

}  // namespace recsa
