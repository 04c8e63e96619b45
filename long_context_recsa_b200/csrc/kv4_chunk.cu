// Attention of a prompt's chunk over the 4-bit KV cache on the tensor cores (tcgen05), for
// bf16 tensors and more than 8 rows (chunk rows times heads of a group) a KV head:
//
//   o_r = sum_t p_rt V_t / sum_t p_rt,   p_rt = exp(scale q_r . K_t), over the t that r sees.
//
// A CTA (one per SM, persistent) works on two streams of 128 rows each, so that one's
// softmax runs under the other's products:
//   S_i  = Q_i K^T      128 rows x 128 tokens, fp32 in TMEM; Q and K fp16 in shared memory
//   P_i  = 2^(S_i - m)  by a warpgroup a stream, a thread a row, fp16 over S_i in TMEM
//   O_i += P_i V        fp32 in TMEM; V fp16 in shared memory, tokens x dims as it is read
// With more than 128 rows the streams are two blocks of rows over the same tokens, else the
// even and the odd tiles of the same rows, whose results are joined at the end.
//
// Eight warps turn the codes into fp16: (w & 0x000f000f) | 0x64006400 is 1024 + code in both
// halves, less 1024 is the code, and one HFMA2 gives lo + s * code, rounded once (2^-12 of
// the value).  K, V and q are scaled by powers of two into fp16's range (the largest |K|
// and |V| of a unit are kept by the writes); a bf16 q is exact there.  P is scaled to at most
// 2^14: its rounding is 2^-12 relative down to 2^-28 of the largest.  The running maximum m
// moves only when a score passes it by 6 (in log2), so O is seldom rescaled; m, the sum of
// P, S and O are fp32.
//
// Bound: 4 d flops a pair of row and token.  At 128 x 128 x 128 a tile and stream, products
// take 1024 cycles at the tensor cores' rate and the 16384 exponentials 1024 cycles at the
// SM's 16 a cycle.
//
// All tiles of all units (sequence, KV head, block of rows) form one list, cut evenly over
// the CTAs.  Tiles behind a block's last position are left out where slots are positions
// (nothing was evicted).  A unit that is cut leaves partial results (O, m, sum of P), which
// kv4_join_kernel adds in the order of the CTAs.
#include "kv4.cuh"

namespace recsa {

namespace {

constexpr int kTok = 128;                 // tokens of a tile
constexpr int kRowsStream = 128;
constexpr int kSoftWarps = 8;             // two warpgroups, a stream each
constexpr int kKWarp0 = 8, kVWarp0 = 12, kMmaWarp = 16;
constexpr int kChunkThreads = 17 * 32;
constexpr int kInfo = 4;                  // tiles whose positions are held (see the ring's use)
constexpr float kUp = 8.0f;               // P is scaled by 2^8, and stays below 2^14
constexpr float kGrow = 6.0f;

template <int D>
struct ChunkSmem {
    static constexpr int kSlab = 128 * 128;             // 128 rows of 64 fp16
    static constexpr int kTileBytes = kSlab * (D / 64);
    static constexpr int kQ = 0;                        // [2 streams]
    static constexpr int kK = 2 * kTileBytes;           // [2 stages]
    static constexpr int kV = 4 * kTileBytes;           // [2 stages]
    static constexpr int kBytes = 6 * kTileBytes + 1024;
};

// The list of tiles: sequence b has nrb[b] blocks of RB rows a KV head; block j sees
// tiles_of(b, j) tiles of the cache.  pre: running totals over b.
struct ChunkPlan {
    int64_t pre[RECSA_MAX_BATCH + 1];
    int64_t first[RECSA_MAX_BATCH];       // tokens that the first block's rows see, + 127; -1: all
    int tmax[RECSA_MAX_BATCH];            // tiles of the whole cache
    int nrb[RECSA_MAX_BATCH];
    int lg_step;                          // log2 of the positions a block adds
};

__device__ __forceinline__ int tiles_of(const ChunkPlan& p, int b, int j) {
    if (p.first[b] < 0) return p.tmax[b];
    const int64_t t = (p.first[b] + ((int64_t)j << p.lg_step)) >> 7;
    return (int)(t < p.tmax[b] ? t : p.tmax[b]);
}
// Tiles of blocks 0 .. k - 1; only the last block of all may be cut to tmax.
__device__ __forceinline__ int64_t tiles_before(const ChunkPlan& p, int b, int k) {
    if (p.first[b] < 0) return (int64_t)k * p.tmax[b];
    const bool all = k == p.nrb[b] && k > 0;
    if (all) --k;
    const int64_t a = p.first[b];
    int64_t sum = all ? tiles_of(p, b, k) : 0;
    if (p.lg_step >= 7)
        return sum + k * (a >> 7) + (((int64_t)k * (k - 1) / 2) << (p.lg_step - 7));
    const int q = 128 >> p.lg_step;       // blocks that add one tile together
    const int64_t U = k / q;
    const int v = k % q;
    for (int w = 0; w < q; ++w) {
        const int64_t t = (a + ((int64_t)w << p.lg_step)) >> 7;
        sum += U * t + U * (U - 1) / 2;
        if (w < v) sum += t + U;
    }
    return sum;
}

__device__ __forceinline__ void make_chunk_plan(ChunkPlan& pl, const Kv4View& c, const Kv4Query& qv,
                                                int RB, int lane) {
    // one warp, two sequences a lane
    const int lg_g = 31 - __clz(c.G);
    if (lane == 0) pl.lg_step = (RB == 256 ? 8 : 7) - lg_g;
    __syncwarp();
    int64_t v[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int b = 2 * lane + k;
        v[k] = 0;
        if (b < c.B) {
            const int64_t L = c.len[b], seen = c.seen[b];
            int n_b = (int)kv4_count(qv.counts, b, qv.n, c.status);
            if (n_b > seen) {             // more rows than tokens: none has a position
                set_status(c.status, kStatusBadQuery);
                n_b = 0;
            }
            int rows = n_b - qv.i0;
            rows = rows < 0 ? 0 : rows < qv.w ? rows : qv.w;
            pl.nrb[b] = (rows * c.G + RB - 1) / RB;
            pl.tmax[b] = (int)((L + kTok - 1) / kTok);
            pl.first[b] = L == seen ? seen - n_b + qv.i0 + ((int64_t)RB >> lg_g) + 127 : -1;
            v[k] = c.Hkv * tiles_before(pl, b, pl.nrb[b]);
        }
    }
    int64_t x = v[0] + v[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
    }
    const int64_t before = x - v[0] - v[1];
    if (2 * lane < c.B) pl.pre[2 * lane] = before;
    if (2 * lane + 1 < c.B) pl.pre[2 * lane + 1] = before + v[0];
    const int64_t total = __shfl_sync(kFull, x, 31);
    if (lane == 0) pl.pre[c.B] = total;
}

// (KV head, block) of sequence b in which tile `in_b` of the sequence's list lies, and the
// place of the unit's first tile in that list.
__device__ __forceinline__ void unit_at(const ChunkPlan& p, int b, int64_t in_b, int& h, int& rb,
                                        int64_t& start) {
    const int64_t per_h = tiles_before(p, b, p.nrb[b]);
    h = (int)(in_b / per_h);
    const int64_t x = in_b - h * per_h;
    int lo = 0, hi = p.nrb[b] - 1;        // the last block that starts at or before x
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (tiles_before(p, b, mid) <= x) lo = mid; else hi = mid - 1;
    }
    rb = lo;
    start = h * per_h + tiles_before(p, b, lo);
}

// ---- tcgen05 ------------------------------------------------------------------------
__device__ __forceinline__ void tc_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Shared-memory matrix descriptor with 128-byte swizzle.  K-major (Q, K): rows of 64 fp16,
// groups of 8 rows 1024 bytes apart.  MN-major (V): rows are tokens (the K dimension), 64
// dims contiguous, groups of 8 tokens 1024 bytes apart, the next 64 dims `lead` bytes on.
__device__ __forceinline__ uint64_t sw128(uint32_t addr, uint32_t lead) {
    return (uint64_t)((addr >> 4) & 0x3fffu) | ((uint64_t)((lead >> 4) & 0x3fffu) << 16) |
           ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}
// kind::f16, fp16 operands, fp32 accumulator, M = 128.
__host__ __device__ constexpr uint32_t f16_idesc(int N, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
// Arrives on `bar` when all products that this thread has issued are done.
__device__ __forceinline__ void commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void ld32(uint32_t t, float (&v)[32]) {
    uint32_t* u = reinterpret_cast<uint32_t*>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
          "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]),
          "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]),
          "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(t)
        : "memory");
}
__device__ __forceinline__ void ld_done() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_done() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st32(uint32_t t, const float (&v)[32]) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(v);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(t),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
        "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]),
        "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]), "r"(u[19]), "r"(u[20]), "r"(u[21]),
        "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]), "r"(u[28]),
        "r"(u[29]), "r"(u[30]), "r"(u[31])
        : "memory");
}
__device__ __forceinline__ void st16(uint32_t t, const uint32_t (&u)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(t),
        "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
        "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
        : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float pow2i(int e) {   // 2^e, clamped to the normal range
    e = e < -126 ? -126 : e > 127 ? 127 : e;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}
__device__ __forceinline__ int exponent_of(float x) {
    return (int)((__float_as_uint(x) >> 23) & 255u) - 127;
}
__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_u(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// Place of a 16-byte chunk (8 dims) of a row: slabs of 64 dims, swizzled.
__device__ __forceinline__ uint32_t chunk_of(int row, int ch) {
    return (uint32_t)((ch >> 3) * (128 * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
}

// The 8 values of a word of codes, in the order of dims 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 values8(uint32_t w, __half2 s, __half2 lo) {
    const __half2 k1024 = as_h2(0xe400e400u), k64 = as_h2(0xd400d400u);   // -1024, -64
    const uint32_t x = w >> 8;
    uint4 v;
    v.x = as_u(__hfma2(__hadd2(as_h2((w & 0x000f000fu) | 0x64006400u), k1024), s, lo));
    v.y = as_u(__hfma2(__hadd2(as_h2((w & 0x00f000f0u) | 0x54005400u), k64), s, lo));
    v.z = as_u(__hfma2(__hadd2(as_h2((x & 0x000f000fu) | 0x64006400u), k1024), s, lo));
    v.w = as_u(__hfma2(__hadd2(as_h2((x & 0x00f000f0u) | 0x54005400u), k64), s, lo));
    return v;
}

// What a thread of the dequantising warps holds of its token's row.
template <int D> struct TokenRow {
    uint4 codes[D / 32];
    uint32_t par[D / 32];
};
template <int D>
__device__ __forceinline__ void load_token(TokenRow<D>& t, const uint8_t* codes, const uint32_t* pars,
                                           int64_t row, bool there) {
    constexpr int NG = D / 32;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        t.codes[j] = make_uint4(0, 0, 0, 0);
        t.par[j] = 0;
    }
    if (!there) return;
    const uint4* p = reinterpret_cast<const uint4*>(codes) + row * NG;
#pragma unroll
    for (int j = 0; j < NG; ++j) t.codes[j] = __ldg(p + j);
    if constexpr (NG == 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(pars) + row);
        t.par[0] = v.x; t.par[1] = v.y; t.par[2] = v.z; t.par[3] = v.w;
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(pars) + row);
        t.par[0] = v.x; t.par[1] = v.y;
    }
}
template <int D>
__device__ __forceinline__ void put_token(unsigned char* tile, const TokenRow<D>& t, int row,
                                          float scale) {
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        const __half2 s = __float2half2_rn(kv4_step(t.par[j]) * scale);
        const __half2 lo = __float2half2_rn(kv4_off(t.par[j]) * scale);
        const uint32_t w[4] = {t.codes[j].x, t.codes[j].y, t.codes[j].z, t.codes[j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(tile + chunk_of(row, j * 4 + k)) = values8(w[k], s, lo);
    }
}

// Tiles a CTA takes; two at least, one for each stream.
__device__ __forceinline__ int64_t chunk_quota(int64_t total, int ctas) {
    const int64_t q = (total + ctas - 1) / ctas;
    return q < 2 ? 2 : q;
}

// 8 dims of an output row from the order 0 4 1 5 2 6 3 7 of the columns.
__device__ __forceinline__ uint4 out8(const float* o, float inv) {
    const __nv_bfloat162 a[4] = {__floats2bfloat162_rn(o[0] * inv, o[2] * inv),
                                 __floats2bfloat162_rn(o[4] * inv, o[6] * inv),
                                 __floats2bfloat162_rn(o[1] * inv, o[3] * inv),
                                 __floats2bfloat162_rn(o[5] * inv, o[7] * inv)};
    return *reinterpret_cast<const uint4*>(a);
}

constexpr uint32_t kNanPar = 0x7fc00000u;   // lo = NaN, s = 0

struct ChunkBars {
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full;
};

}  // namespace

// part: [2 * grid] of: O [D / 4][RB] float4, m [RB], l [RB].
template <int D>
__global__ void __launch_bounds__(kChunkThreads, 1) kv4_chunk_kernel(Kv4View c, Kv4Query qv,
                                                                     Kv4Scratch sc, int RB) {
    constexpr int NG = D / 32;
    using Sm = ChunkSmem<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ ChunkPlan pl;
    __shared__ ChunkBars bars;
    __shared__ __align__(16) int32_t pos_s[kInfo][kTok];
    __shared__ __align__(16) int32_t pos_max[kInfo][4];
    __shared__ uint32_t nan_s[kInfo][4][4];   // [tile][warp's 32 tokens][group of 32 dims]
    __shared__ __align__(16) uint32_t nan_any[kInfo][4];
    __shared__ float join_m[kRowsStream], join_l[kRowsStream];
    __shared__ uint32_t join_nan[kRowsStream];
    __shared__ int unit_h, unit_rb;
    __shared__ int64_t unit_start;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int failed;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool two_blocks = RB == 256;        // else the streams share their rows

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.k_full[i], 128);
            mbar_init(&bars.k_empty[i], 1);
            mbar_init(&bars.v_full[i], 128);
            mbar_init(&bars.v_empty[i], 1);
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_full[i], 128);
        }
        mbar_init(&bars.o_full, 1);
        mbar_fence_init();
        failed = 0;
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_u32(&tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) make_chunk_plan(pl, c, qv, RB, lane);
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = tmem_slot;
    const int64_t total = pl.pre[c.B];
    const int64_t quota = chunk_quota(total, gridDim.x);
    int64_t at = blockIdx.x * quota;
    const int64_t at_end = at + quota < total ? at + quota : total;

    // a wait of this CTA that gave up ends the CTA's work (all waits are bounded)
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_wait_bounded(bar, parity, c.status, failed ? kWaitPollsAfterFail : kWaitPolls))
            return failed == 0;
        failed = 1;
        return false;
    };

    // uses of each barrier so far give the parities
    uint32_t n_tiles = 0, n_x[2] = {0, 0}, n_units = 0;

    int b = 0;
    while (at < at_end) {
        while (pl.pre[b + 1] <= at) ++b;
        if (threadIdx.x == 0) {
            int h, rb;
            int64_t start;
            unit_at(pl, b, at - pl.pre[b], h, rb, start);
            unit_h = h;
            unit_rb = rb;
            unit_start = pl.pre[b] + start;
        }
        __syncthreads();
        const int h = unit_h, rb = unit_rb, u = b * c.Hkv + h;
        const int64_t start = unit_start;
        const int tiles = tiles_of(pl, b, rb), tile0 = (int)(at - start);
        const int T = (int)(at_end - at < tiles - tile0 ? at_end - at : tiles - tile0);
        const int64_t L = c.len[b], seen = c.seen[b];
        const int n_b = qv.counts ? qv.counts[b] : qv.n;
        const int w_end = qv.i0 + qv.w < n_b ? qv.i0 + qv.w : n_b;
        const int row0 = qv.i0 * c.G + rb * RB, row_end = w_end * c.G;
        const int ek = exponent_of(__uint_as_float(c.kmax[u])), ev = exponent_of(__uint_as_float(c.vmax[u]));
        // products of the two streams in turn: x = 0, 1, .. ; x's stream is x & 1
        const int X = two_blocks ? 2 * T : T;
        const int sh = two_blocks ? 1 : 0;        // tile of x: x >> sh

        // ---- Q: the softmax warps stage their rows ----
        int lim = -1;
        float rsc = 0.0f;
        const int stream = warp >> 2, r = threadIdx.x & 127;
        const int row = row0 + (two_blocks ? stream * kRowsStream : 0) + r;
        if (warp < kSoftWarps) {
            unsigned char* qs = smem + Sm::kQ + stream * Sm::kTileBytes;
            const bool live = row < row_end;
            uint4 raw[D / 8];
            float mx = 0.0f;
            if (live) {
                const int i = row / c.G, g = row % c.G;
                lim = (int)(seen - n_b + i);
                const uint4* q = reinterpret_cast<const uint4*>(
                    reinterpret_cast<const __nv_bfloat16*>(qv.q) +
                    (((int64_t)b * qv.n + i) * c.Hq + h * c.G + g) * D);
#pragma unroll
                for (int k = 0; k < D / 8; ++k) raw[k] = __ldg(q + k);
            } else {
#pragma unroll
                for (int k = 0; k < D / 8; ++k) raw[k] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[e] << 16)),
                                         fabsf(__uint_as_float(w[e] & 0xffff0000u))));
            }
            const int e0 = exponent_of(mx), eq = e0 < -116 ? -116 : e0;
            const float up = pow2i(10 - eq);
            rsc = fmaxf(fminf(c.scale * 1.4426950408889634f * pow2i(eq - 10 + ek - 13), 3e38f), 1e-38f);
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
                float x[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[2 * e] = __uint_as_float(w[e] << 16) * up;
                    x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u) * up;
                }
                uint4 y;
                y.x = as_u(__floats2half2_rn(x[0], x[4]));
                y.y = as_u(__floats2half2_rn(x[1], x[5]));
                y.z = as_u(__floats2half2_rn(x[2], x[6]));
                y.w = as_u(__floats2half2_rn(x[3], x[7]));
                *reinterpret_cast<uint4*>(qs + chunk_of(r, k)) = y;
            }
            fence_async_smem();
        }
        __syncthreads();

        if (warp >= kKWarp0 && warp < kMmaWarp) {
            // ---- codes to fp16: four warps K, four V, a thread a token ----
            const bool is_v = warp >= kVWarp0;
            const int tok = threadIdx.x & 127;
            const uint8_t* codes = (is_v ? c.vc : c.kc) + u * c.R * (D / 2);
            const uint32_t* pars = (is_v ? c.vp : c.kp) + u * c.R * NG;
            const uint32_t* vpars = c.vp + u * c.R * NG;
            const float scale = pow2i(13 - (is_v ? ev : ek));
            uint64_t* full = is_v ? bars.v_full : bars.k_full;
            uint64_t* empty = is_v ? bars.v_empty : bars.k_empty;
            unsigned char* ring = smem + (is_v ? Sm::kV : Sm::kK);
            TokenRow<D> cur, nxt;
            int64_t t_row = (int64_t)tile0 * kTok + tok;
            load_token<D>(nxt, codes, pars, t_row, t_row < L);
            for (int t = 0; t < T; ++t) {
                const uint32_t n = n_tiles + t;
                cur = nxt;
                const int64_t row_t = (int64_t)(tile0 + t) * kTok + tok;
                const bool there = row_t < L;
                int32_t pos = 0x7fffffff;
                uint32_t vnan = 0;
                if (!is_v && there) {
                    pos = __ldg(c.pos + u * c.R + row_t);
#pragma unroll
                    for (int j = 0; j < NG; ++j)
                        vnan |= (__ldg(vpars + row_t * NG + j) == kNanPar ? 1u : 0u) << j;
                }
                if (t + 1 < T) load_token<D>(nxt, codes, pars, row_t + kTok, row_t + kTok < L);
                const uint32_t st = n & 1;
                if (!wait(&empty[st], ((n >> 1) & 1) ^ 1)) break;
                if (is_v) {
                    // the rows that see a NaN group learn of it by nan_s; in a product
                    // it would reach all rows
#pragma unroll
                    for (int j = 0; j < NG; ++j)
                        if (cur.par[j] == kNanPar) cur.par[j] = 0;
                } else {
                    const int slot = n % kInfo, wq = warp - kKWarp0;
                    pos_s[slot][tok] = pos;
                    const int32_t most = __reduce_max_sync(kFull, pos);
                    const bool any = __any_sync(kFull, vnan != 0);
                    if (any) {
#pragma unroll
                        for (int j = 0; j < NG; ++j) {
                            const uint32_t m = __ballot_sync(kFull, (vnan >> j) & 1u);
                            if (lane == 0) nan_s[slot][wq][j] = m;
                        }
                    }
                    if (lane == 0) {
                        pos_max[slot][wq] = most;
                        nan_any[slot][wq] = any;
                    }
                }
                put_token<D>(ring + st * Sm::kTileBytes, cur, tok, scale);
                fence_async_smem();
                mbar_arrive(&full[st]);
            }
        } else if (warp == kMmaWarp) {
            // ---- products ----
            if (lane == 0) {
                constexpr uint32_t id_qk = f16_idesc(kTok, false), id_pv = f16_idesc(D, true);
                const uint32_t q0 = smem_u32(smem + Sm::kQ), k0 = smem_u32(smem + Sm::kK),
                               v0 = smem_u32(smem + Sm::kV);
                bool ok = true;
                auto qk = [&](int x) {
                    const uint32_t n = n_tiles + (x >> sh), st = n & 1;
                    ok = ok && wait(&bars.k_full[st], (n >> 1) & 1);
                    if (!ok) return;
                    tc_after();
                    const uint32_t qa = q0 + (x & 1) * Sm::kTileBytes, ka = k0 + st * Sm::kTileBytes;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = (k >> 2) * Sm::kSlab + (k & 3) * 32;
                        mma_ss(tmem + (x & 1) * 128, sw128(qa + off, 16), sw128(ka + off, 16), id_qk, k > 0);
                    }
                    commit(&bars.s_full[x & 1]);
                    if (!two_blocks || (x & 1)) commit(&bars.k_empty[st]);
                };
                qk(0);
                if (X > 1) qk(1);
                for (int x = 0; ok && x < X; ++x) {
                    const uint32_t n = n_tiles + (x >> sh), st = n & 1, i = x & 1;
                    ok = ok && wait(&bars.v_full[st], (n >> 1) & 1) &&
                         wait(&bars.p_full[i], (n_x[i] + (x >> 1)) & 1);
                    if (!ok) break;
                    tc_after();
#pragma unroll
                    for (int k = 0; k < kTok / 16; ++k)
                        mma_ts(tmem + 256 + i * 128, tmem + i * 128 + k * 8,
                               sw128(v0 + st * Sm::kTileBytes + k * 2048, Sm::kSlab), id_pv,
                               x > 1 || k > 0);
                    if (!two_blocks || i) commit(&bars.v_empty[st]);
                    if (x + 2 < X) qk(x + 2);
                }
                commit(&bars.o_full);
                // after a failure: what was issued is done before TMEM is given back
                if (!ok) mbar_wait_bounded(&bars.o_full, n_units & 1, c.status, kWaitPollsAfterFail);
            }
            __syncwarp();
        }
        if (warp < kSoftWarps) {
            // ---- softmax: a thread a row ----
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t ts = tmem + lanes + stream * 128, to = tmem + lanes + 256 + stream * 128;
            const int mine = (X - stream + 1) / 2;
            const bool some = __any_sync(kFull, lim >= 0);
            float m = kKv4MinLog2, l = 0.0f;
            uint32_t nanbits = 0;
            bool ok = true;
            for (int j = 0; j < mine; ++j) {
                const int x = 2 * j + stream;
                const uint32_t slot = (n_tiles + (x >> sh)) % kInfo;
                ok = ok && wait(&bars.s_full[stream], (n_x[stream] + j) & 1);
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                tc_after();
                if (some) {
                    const int4 pm = *reinterpret_cast<const int4*>(pos_max[slot]);
                    const int most = max(max(pm.x, pm.y), max(pm.z, pm.w));
                    const bool masked = __any_sync(kFull, most > lim && lim >= 0);
                    const uint4 na = *reinterpret_cast<const uint4*>(nan_any[slot]);
                    if (na.x | na.y | na.z | na.w) {
                        for (int q = 0; q < 4; ++q) {
                            if (!nan_any[slot][q]) continue;
                            for (int e = 0; e < 32; ++e)
                                if (pos_s[slot][q * 32 + e] <= lim)
                                    for (int g = 0; g < NG; ++g)
                                        nanbits |= ((nan_s[slot][q][g] >> e) & 1u) << g;
                        }
                    }
                    float s[32];
                    auto load_scores = [&](int k) {
                        ld32(ts + k * 32, s);
                        ld_done();
                        if (masked) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const int4 p = *reinterpret_cast<const int4*>(&pos_s[slot][k * 32 + e]);
                                if (p.x > lim) s[e] = -INFINITY;
                                if (p.y > lim) s[e + 1] = -INFINITY;
                                if (p.z > lim) s[e + 2] = -INFINITY;
                                if (p.w > lim) s[e + 3] = -INFINITY;
                            }
                        }
                    };
                    float mx = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        load_scores(k);
#pragma unroll
                        for (int e = 0; e < 32; e += 2) mx = fmaxf(mx, fmaxf(s[e], s[e + 1]));
                    }
                    mx *= rsc;
                    if (__any_sync(kFull, mx > m + kGrow)) {
                        const float mn = mx > m + kGrow ? mx : m;
                        const float f = ex2(m - mn);
                        m = mn;
                        l *= f;
                        if (j > 0) {
                            // the products before S are done (one thread issued both, and
                            // the barrier stands for all it had issued)
#pragma unroll 1
                            for (int k = 0; k < D; k += 32) {
                                float o[32];
                                ld32(to + k, o);
                                ld_done();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] *= f;
                                st32(to + k, o);
                            }
                        }
                    }
                    const float shift = kUp - m;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        load_scores(k);
                        uint32_t p[16];
                        float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float a = ex2(fmaf(s[e], rsc, shift)), z = ex2(fmaf(s[e + 1], rsc, shift));
                            l0 += a;
                            l1 += z;
                            p[e >> 1] = as_u(__floats2half2_rn(a, z));
                        }
                        l += l0 + l1;
                        st16(ts + k * 16, p);
                    }
                    st_done();
                }
                tc_before();
                mbar_arrive(&bars.p_full[stream]);
            }
            // ---- results ----
            ok = __all_sync(kFull, ok && wait(&bars.o_full, n_units & 1));
            tc_after();
            const int64_t cta0 = start / quota, cta1 = (start + tiles - 1) / quota;
            const bool whole = cta0 == cta1;
            float f0 = 1.0f, f1 = 0.0f;
            float4* other = reinterpret_cast<float4*>(smem + Sm::kK);   // [D / 4][128]: K is done
            if (!two_blocks) {
                // stream 1 leaves its part of the same rows to stream 0
                if (stream == 1) {
                    join_m[r] = m;
                    join_l[r] = l;
                    join_nan[r] = nanbits;
                    if (mine > 0 && some) {
#pragma unroll 1
                        for (int k = 0; k < D; k += 32) {
                            float o[32];
                            ld32(to + k, o);
                            ld_done();
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                other[(k + e) / 4 * 128 + r] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                        }
                    }
                }
                asm volatile("bar.sync 1, 256;" ::: "memory");
                if (stream == 0 && X > 1) {
                    const float m1 = join_m[r], mm = fmaxf(m, m1);
                    f0 = ex2(m - mm);
                    f1 = ex2(m1 - mm);
                    m = mm;
                    l = f0 * l + f1 * join_l[r];
                    nanbits |= join_nan[r];
                }
            }
            if ((two_blocks || stream == 0) && some && ok) {
                const bool live = row < row_end;
                const int i = row / c.G, g = row % c.G, rr = row - row0;
                const bool any = l > 0.0f || l != l;
                const float inv = any ? pow2i(ev - 13) / l : 0.0f;
                float* part = sc.part + (size_t)(2 * blockIdx.x + (tile0 == 0 ? 1 : 0)) * RB * (D + 2);
                __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(qv.out) +
                                     (((int64_t)b * qv.n + i) * c.Hq + h * c.G + g) * D;
#pragma unroll 1
                for (int k = 0; k < D; k += 32) {
                    float o[32];
                    ld32(to + k, o);
                    ld_done();
                    if (f1 != 0.0f) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 v = other[(k + e) / 4 * 128 + r];
                            o[e] = fmaf(f1, v.x, f0 * o[e]);
                            o[e + 1] = fmaf(f1, v.y, f0 * o[e + 1]);
                            o[e + 2] = fmaf(f1, v.z, f0 * o[e + 2]);
                            o[e + 3] = fmaf(f1, v.w, f0 * o[e + 3]);
                        }
                    } else if (f0 != 1.0f) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= f0;
                    }
                    if ((nanbits >> (k / 32)) & 1u) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = NAN;
                    }
                    if (!live) continue;
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4*>(out + k + e) = out8(&o[e], inv);
                    } else {
                        float4* po = reinterpret_cast<float4*>(part);
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            po[(size_t)((k + e) / 4) * RB + rr] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                if (live && whole) {
                    sc.lse[(int64_t)u * qv.w * c.G + row - qv.i0 * c.G] =
                        any ? m - kUp + log2f(l) : INFINITY;
                } else if (live) {
                    part[(size_t)RB * D + rr] = m;
                    part[(size_t)RB * D + RB + rr] = l;
                }
            }
        }
        at += T;
        n_tiles += T;
        n_x[0] += (X + 1) / 2;
        n_x[1] += X / 2;
        ++n_units;
        tc_before();
        __syncthreads();
        tc_after();
        if (failed) break;
    }
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Joins the parts of the units that were cut.  Grid: x = 32 rows, y = unit; a lane a row, a
// warp some of the 8-dim pieces.
template <int D>
__global__ void __launch_bounds__(256) kv4_join_kernel(Kv4View c, Kv4Query qv, Kv4Scratch sc, int RB,
                                                       int ctas) {
    __shared__ ChunkPlan pl;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) make_chunk_plan(pl, c, qv, RB, lane);
    __syncthreads();
    const int u = blockIdx.y, b = u / c.Hkv, h = u % c.Hkv;
    const int rel = blockIdx.x * 32, rb = rel / RB, rr = rel % RB + lane;
    if (rb >= pl.nrb[b]) return;
    const int64_t quota = chunk_quota(pl.pre[c.B], ctas);
    const int64_t start = pl.pre[b] + h * tiles_before(pl, b, pl.nrb[b]) + tiles_before(pl, b, rb);
    const int64_t cta0 = start / quota, cta1 = (start + tiles_of(pl, b, rb) - 1) / quota;
    if (cta0 == cta1) return;
    const int n_b = qv.counts ? qv.counts[b] : qv.n;
    const int w_end = qv.i0 + qv.w < n_b ? qv.i0 + qv.w : n_b;
    const int row = qv.i0 * c.G + rel + lane;
    if (row >= w_end * c.G) return;
    auto part = [&](int64_t cta) {
        return sc.part + (size_t)(2 * cta + (cta == cta0 ? 1 : 0)) * RB * (D + 2);
    };
    float m = kKv4MinLog2, l = 0.0f;
    for (int64_t k = cta0; k <= cta1; ++k) m = fmaxf(m, part(k)[(size_t)RB * D + rr]);
    for (int64_t k = cta0; k <= cta1; ++k) {
        const float* p = part(k) + (size_t)RB * D + rr;
        l = fmaf(ex2(p[0] - m), p[RB], l);
    }
    const bool any = l > 0.0f || l != l;
    const int ev = exponent_of(__uint_as_float(c.vmax[u]));
    const float inv = any ? pow2i(ev - 13) / l : 0.0f;
    const int i = row / c.G, g = row % c.G;
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(qv.out) +
                         (((int64_t)b * qv.n + i) * c.Hq + h * c.G + g) * D;
    for (int ch = warp; ch < D / 8; ch += 8) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.0f;
#pragma unroll 4
        for (int64_t k = cta0; k <= cta1; ++k) {
            const float* p = part(k);
            const float f = ex2(p[(size_t)RB * D + rr] - m);
            const float4 x = reinterpret_cast<const float4*>(p)[(size_t)(2 * ch) * RB + rr];
            const float4 y = reinterpret_cast<const float4*>(p)[(size_t)(2 * ch + 1) * RB + rr];
            o[0] = fmaf(f, x.x, o[0]); o[1] = fmaf(f, x.y, o[1]);
            o[2] = fmaf(f, x.z, o[2]); o[3] = fmaf(f, x.w, o[3]);
            o[4] = fmaf(f, y.x, o[4]); o[5] = fmaf(f, y.y, o[5]);
            o[6] = fmaf(f, y.z, o[6]); o[7] = fmaf(f, y.w, o[7]);
        }
        *reinterpret_cast<uint4*>(out + ch * 8) = out8(o, inv);
    }
    if (warp == 0)
        sc.lse[(int64_t)u * qv.w * c.G + row - qv.i0 * c.G] = any ? m - kUp + log2f(l) : INFINITY;
}

// ---------------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------------
namespace {

constexpr int kChunkGrid = 148;

// Rows of a unit's block: 256 (two streams) or 128 (two halves of the tiles).
int chunk_rows(int rows) { return rows > kRowsStream ? 2 * kRowsStream : kRowsStream; }

template <int D>
cudaError_t chunk_impl(const Kv4View& c, const Kv4Query& qv, const Kv4Scratch& sc, cudaStream_t s) {
    const int rows = qv.w * c.G, RB = chunk_rows(rows);
    cudaError_t e = kv4_launch(kv4_chunk_kernel<D>, dim3(kChunkGrid), kChunkThreads,
                               (size_t)ChunkSmem<D>::kBytes, s, c, qv, sc, RB);
    if (e != cudaSuccess) return e;
    return kv4_launch(kv4_join_kernel<D>, dim3((unsigned)((rows + 31) / 32), (unsigned)(c.B * c.Hkv)), 256,
                      0, s, c, qv, sc, RB, kChunkGrid);
}

}  // namespace

size_t kv4_chunk_part_floats(int D, int rows) {
    return (size_t)2 * kChunkGrid * chunk_rows(rows) * (D + 2);
}

cudaError_t kv4_prepare_chunk(int D) {
    return D == 128 ? cudaFuncSetAttribute(kv4_chunk_kernel<128>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           ChunkSmem<128>::kBytes)
                    : cudaFuncSetAttribute(kv4_chunk_kernel<64>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           ChunkSmem<64>::kBytes);
}

cudaError_t kv4_launch_chunk(const Kv4View& c, const Kv4Query& qv, const Kv4Scratch& sc, cudaStream_t s) {
    NvtxRange nv("recsa kv4 chunk");
    return c.D == 128 ? chunk_impl<128>(c, qv, sc, s) : chunk_impl<64>(c, qv, sc, s);
}

}  // namespace recsa
