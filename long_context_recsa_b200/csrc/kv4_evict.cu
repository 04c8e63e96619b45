// Eviction from the 4-bit KV cache by accumulated attention weight.
//
// Per unit (sequence, KV head) of length L > budget, `budget` rows stay: the first
// n_first tokens, the newest n_recent ones, and of the others those of the largest
// weights (ties: the lower slot; a NaN weight ranks below every number).  Kept rows in
// slots >= budget (they "move") go into the slots < budget that became free, the j-th by
// slot into the j-th free one: sources and destinations are disjoint, so rows move in
// place, and only as many as leave.  Attention does not depend on the order of slots.
//
// One CTA or one cluster of up to 8 a unit: CTA r owns an eighth (or so) of the slots, and
// reads their weights and positions once, into order keys in shared memory.  A radix select
// over the keys (four digits of 8 bits, counted by all, summed over the cluster) gives the
// threshold key and how many of its ties stay; every warp's counts of keys above and at
// the threshold, read by the whole cluster, give each warp its places in the ascending
// lists of free slots and movers; the cluster shares the copies.  What bounds it is the
// chain of these steps and their barriers, not the bytes.
#include <cooperative_groups.h>

#include "kv4.cuh"

namespace recsa {

namespace {

namespace cg = cooperative_groups;

constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kBins = 256;
constexpr int kEvictKeys = 49152;           // order keys a CTA's shared memory holds

// Order key of a slot: ~0 for a protected token, else monotone in the weight.
__device__ __forceinline__ uint32_t evict_key(float w, int32_t pos, int64_t first, int64_t recent0) {
    if (pos < first || pos >= recent0) return 0xffffffffu;
    if (w != w) return 0u;
    return ordered_key(w);   // at most the key of +inf, below ~0; at least that of -inf, above 0
}

__device__ __forceinline__ int warp_prefix(int v) {   // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// What a warp's run of slots holds: keys above the threshold and at it, in slots below the
// budget and behind, and the slots below the budget.
struct __align__(16) RunCounts { int above_lo, above_hi, ties_lo, ties_hi, slots_lo, pad[3]; };

}  // namespace

// lists: [U][R] int32; free slots from the front of a unit's part, movers from R / 2 on
// (neither can pass R / 2: both are at most min(budget, L - budget)).
template <int D>
__global__ void __launch_bounds__(kEvictThreads) kv4_evict_kernel(Kv4View c, int64_t budget,
                                                                  int64_t n_first, int64_t n_recent,
                                                                  int32_t* lists) {
    extern __shared__ uint32_t keys[];       // [min(segment, kEvictKeys)]
    __shared__ int hist[4][kBins];           // a pass each, so that none is cleared while it is read
    __shared__ int part[kEvictThreads];      // sums over some of the cluster's CTAs
    __shared__ RunCounts runs[kEvictWarps];  // read by the cluster
    __shared__ int2 place[kEvictWarps];      // of this CTA's warps: first free slot and mover
    __shared__ int tie_rank[kEvictWarps];
    __shared__ uint32_t s_digit;
    __shared__ int s_need, s_moves;
    __shared__ int last;
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int u = blockIdx.x / CS, b = u / c.Hkv;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t L = c.len[b];
    if (L > budget) {                        // the same for the whole cluster
        const int64_t recent0 = c.seen[b] - n_recent;
        const float* w = c.w + u * c.R;
        const int32_t* pos = c.pos + u * c.R;
        // this CTA's slots: seg0 .. seg0 + n - 1, whole warps of 16-byte words
        const int64_t seg = ((L + CS - 1) / CS + 127) / 128 * 128;
        const int64_t seg0 = rank * seg;
        const int n = (int)(seg0 >= L ? 0 : L - seg0 < seg ? L - seg0 : seg);
        const int held = n < kEvictKeys ? n : kEvictKeys;
        auto far_key = [&](int i) { return evict_key(w[seg0 + i], pos[seg0 + i], n_first, recent0); };
        auto key_at = [&](int i) { return i < held ? keys[i] : far_key(i); };

        // digits from the top: the need-th largest key, and how many of its ties stay
        uint32_t prefix = 0;
        int need = (int)budget;
        for (int i = threadIdx.x; i < 4 * kBins; i += kEvictThreads) hist[0][i] = 0;
        __syncthreads();
#pragma unroll 1
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            int* mine = hist[pass];
            if (pass == 0) {
                // R is a multiple of 128, so whole words stay inside the unit
                for (int i = threadIdx.x * 4; i < held; i += kEvictThreads * 4) {
                    const float4 x = *reinterpret_cast<const float4*>(w + seg0 + i);
                    const int4 p = *reinterpret_cast<const int4*>(pos + seg0 + i);
                    const uint4 k = make_uint4(evict_key(x.x, p.x, n_first, recent0),
                                               evict_key(x.y, p.y, n_first, recent0),
                                               evict_key(x.z, p.z, n_first, recent0),
                                               evict_key(x.w, p.w, n_first, recent0));
                    *reinterpret_cast<uint4*>(keys + i) = k;
                    atomicAdd(&mine[k.x >> 24], 1);
                    if (i + 1 < n) atomicAdd(&mine[k.y >> 24], 1);
                    if (i + 2 < n) atomicAdd(&mine[k.z >> 24], 1);
                    if (i + 3 < n) atomicAdd(&mine[k.w >> 24], 1);
                }
                for (int i = held + threadIdx.x; i < n; i += kEvictThreads)
                    atomicAdd(&mine[far_key(i) >> 24], 1);
            } else {
                for (int i = threadIdx.x; i < n; i += kEvictThreads) {
                    const uint32_t k = key_at(i);
                    if ((k ^ prefix) >> (shift + 8) == 0) atomicAdd(&mine[(k >> shift) & 255u], 1);
                }
            }
            if (CS > 1) {
                cluster.sync();
                // thread t: bin t & 255 of the CTAs t / 256, t / 256 + 4
                const int bin = threadIdx.x & 255;
                int sum = 0;
                for (int r = threadIdx.x >> 8; r < CS; r += 4)
                    sum += cluster.map_shared_rank(mine, r)[bin];
                part[threadIdx.x] = sum;
            }
            __syncthreads();
            if (warp == 0) {
                // from the top bin down, eight a lane: the bin in which the need-th key lies
                int count[8], sum = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int bin = 255 - (lane * 8 + j);
                    count[j] = CS > 1 ? part[bin] + part[bin + 256] + part[bin + 512] + part[bin + 768]
                                      : mine[bin];
                    sum += count[j];
                }
                int before = warp_prefix(sum) - sum;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (before < need && need <= before + count[j]) {
                        s_digit = (uint32_t)(255 - (lane * 8 + j));
                        s_need = need - before;
                    }
                    before += count[j];
                }
            }
            __syncthreads();
            prefix |= s_digit << shift;
            need = s_need;
        }

        // need slots with key == prefix stay, the lowest first.  A warp owns a run of slots.
        const int run = ((n + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;
        const int i0 = warp * run, i1 = i0 + run < n ? i0 + run : n;
        const int lo_end = (int)(budget - seg0 < 0 ? 0 : budget - seg0 < i1 ? budget - seg0 : i1);
        {
            RunCounts rc = {};
            for (int i = i0 + lane; i - lane < i1; i += 32) {
                const uint32_t k = i < i1 ? key_at(i) : 0u;
                const bool lo = i < lo_end;
                const uint32_t gt = __ballot_sync(kFull, i < i1 && k > prefix);
                const uint32_t eq = __ballot_sync(kFull, i < i1 && k == prefix);
                const uint32_t lm = __ballot_sync(kFull, lo);
                rc.above_lo += __popc(gt & lm);
                rc.above_hi += __popc(gt & ~lm);
                rc.ties_lo += __popc(eq & lm);
                rc.ties_hi += __popc(eq & ~lm);
                rc.slots_lo += __popc(lm);
            }
            if (lane == 0) runs[warp] = rc;
        }
        if (CS > 1) cluster.sync();
        else __syncthreads();
        if (warp < CS) {
            // warp r reads the counts of CTA r's warps: ties, then free slots and movers,
            // before each of them
            RunCounts rc;
            const int4* from = reinterpret_cast<const int4*>(
                CS > 1 ? cluster.map_shared_rank(&runs[0], warp) + lane : &runs[lane]);
            *reinterpret_cast<int4*>(&rc) = from[0];
            rc.slots_lo = from[1].x;
            const int ties = rc.ties_lo + rc.ties_hi;
            int tie0 = warp_prefix(ties);
            if (lane == 31) part[warp] = tie0;
            asm volatile("bar.sync 1, %0;" ::"r"(CS * 32) : "memory");
            tie0 -= ties;
            for (int r = 0; r < warp; ++r) tie0 += part[r];
            const int stay = need - tie0 < 0 ? 0 : need - tie0 < ties ? need - tie0 : ties;
            const int stay_lo = stay < rc.ties_lo ? stay : rc.ties_lo;
            const int fr = rc.slots_lo - rc.above_lo - stay_lo, mv = rc.above_hi + stay - stay_lo;
            int fr0 = warp_prefix(fr), mv0 = warp_prefix(mv);
            if (lane == 31) {
                part[8 + warp] = fr0;
                part[16 + warp] = mv0;
            }
            asm volatile("bar.sync 1, %0;" ::"r"(CS * 32) : "memory");
            fr0 -= fr;
            mv0 -= mv;
            int moves = 0;
            for (int r = 0; r < CS; ++r) {
                if (r < warp) {
                    fr0 += part[8 + r];
                    mv0 += part[16 + r];
                }
                moves += part[16 + r];
            }
            if (warp == rank) {
                tie_rank[lane] = tie0;
                place[lane] = make_int2(fr0, mv0);
                if (lane == 0) s_moves = moves;
            }
        }
        __syncthreads();
        const int moves = s_moves;
        const uint32_t below = (1u << lane) - 1u;
        int free0 = place[warp].x, move0 = place[warp].y, seen = tie_rank[warp];
        int32_t* free_list = lists + u * c.R;
        int32_t* move_list = free_list + c.R / 2;
        for (int i = i0 + lane; i - lane < i1; i += 32) {
            const uint32_t k = i < i1 ? key_at(i) : 0u;
            const bool eq = i < i1 && k == prefix;
            const uint32_t m = __ballot_sync(kFull, eq);
            const bool kept = i < i1 && (k > prefix || (eq && seen + __popc(m & below) < need));
            seen += __popc(m);
            const bool fr = i < lo_end && !kept, mv = i >= lo_end && kept;
            const uint32_t mf = __ballot_sync(kFull, fr), mm = __ballot_sync(kFull, mv);
            const int at_f = free0 + __popc(mf & below), at_m = move0 + __popc(mm & below);
            if (fr && in_bounds(at_f >= 0 && at_f < c.R / 2, c.status)) free_list[at_f] = (int32_t)(seg0 + i);
            if (mv && in_bounds(at_m >= 0 && at_m < c.R / 2, c.status)) move_list[at_m] = (int32_t)(seg0 + i);
            free0 += __popc(mf);
            move0 += __popc(mm);
        }
        if (CS > 1) cluster.sync();          // (a release and acquire over the cluster)
        else __syncthreads();                // the lists are read below by the whole cluster
        // a row is 2 x (D / 2) bytes of codes and 2 x (D / 8) bytes of parameters
        constexpr int CK = D / 32, CH = 2 * CK + 2;   // 16-byte pieces of codes; + parameters
        uint4* kc = reinterpret_cast<uint4*>(c.kc) + u * c.R * CK;
        uint4* vc = reinterpret_cast<uint4*>(c.vc) + u * c.R * CK;
        uint32_t* kp = c.kp + u * c.R * CK;
        uint32_t* vp = c.vp + u * c.R * CK;
        for (int64_t x = rank * kEvictThreads + threadIdx.x; x < (int64_t)moves * CH;
             x += CS * kEvictThreads) {
            const int j = (int)(x / CH), p = (int)(x % CH);
            const int64_t to = __ldcg(free_list + j), from = __ldcg(move_list + j);
            if (!in_bounds(to >= 0 && to < budget && from >= budget && from < L, c.status)) continue;
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
        if (CS > 1) cluster.sync();
        else __syncthreads();                // the moved rows' weights and positions are read
        for (int64_t i = budget + rank * kEvictThreads + threadIdx.x; i < L; i += CS * kEvictThreads) {
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

namespace {

// CTAs of a unit: one or a cluster of eight, by the capacity (the length is known on the device
// only) and by how often the clusters of all units fill the GPU.  One CTA / eight, us, where one
// row goes and where a fifth of them go:
//     units  4096           8192           16384           32768            131072
//         8  16/20  28/21   21/23  43/25   29/23   70/28   43/25  154/39    301/37  786/100
//        32  18/25  29/27   21/26  49/31   31/29   87/39   44/32  166/53    303/57  854/160
//       128  18/82  33/91   23/88  57/109  31/92  107/139  45/105 205/202
int evict_cluster(const Kv4View& c) {
    constexpr int kResident = 2 * 148;       // CTAs of this kernel at once
    const int64_t waves = ((int64_t)c.B * c.Hkv * 8 + kResident - 1) / kResident;
    return c.cap <= 6144 * waves && c.cap <= kEvictKeys ? 1 : 8;
}

size_t evict_smem(int64_t cap, int ctas) {
    const int64_t seg = ((cap + ctas - 1) / ctas + 127) / 128 * 128;
    return sizeof(uint32_t) * (size_t)(seg < kEvictKeys ? seg : kEvictKeys);
}

template <int D>
cudaError_t evict_impl(const Kv4View& c, int64_t budget, int64_t n_first, int64_t n_recent,
                       int32_t* lists, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    const int cs = evict_cluster(c);
    at[0] = pdl_attribute();
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cs;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(c.B * c.Hkv * cs));
    cfg.blockDim = dim3(kEvictThreads);
    cfg.dynamicSmemBytes = evict_smem(c.cap, cs);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kv4_evict_kernel<D>, c, budget, n_first, n_recent, lists);
}

}  // namespace

cudaError_t kv4_prepare_evict(const Kv4View& c) {
    return c.D == 128 ? cudaFuncSetAttribute(kv4_evict_kernel<128>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(sizeof(uint32_t) * kEvictKeys))
                      : cudaFuncSetAttribute(kv4_evict_kernel<64>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(sizeof(uint32_t) * kEvictKeys));
}

cudaError_t kv4_launch_evict(const Kv4View& c, int64_t budget, int64_t n_first, int64_t n_recent,
                             int32_t* lists, cudaStream_t s) {
    NvtxRange nv("recsa kv4 evict");
    return c.D == 128 ? evict_impl<128>(c, budget, n_first, n_recent, lists, s)
                      : evict_impl<64>(c, budget, n_first, n_recent, lists, s);
}

}  // namespace recsa
